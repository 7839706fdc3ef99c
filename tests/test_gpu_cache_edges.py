"""The rolling-cache operators on the GPU where they are easily wrong: large, small and
absurd score caps, NaN, unused rows and keys, positions and documents on every path.

Against the plain 64-bit implementations of the operators' main tests, with their
tolerances but for the cap, whose bound follows the score here (see capped_scores).
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import test_gpu_cache_ops as T  # noqa: E402
from test_gpu_cache_ops import P, at, check_attention, check_mass, docs, ints, lens, make, run_attention, run_mass, stream  # noqa: E402,F401


# ---------------------------------------------------------------- in place

@pytest.mark.parametrize("kw", [
    dict(B=3, Lq=1, Lk=700, Hq=4, Hkv=2, dh=128), dict(B=1, Lq=1, Lk=9000, Hq=2, Hkv=2, dh=64), dict(B=2, Lq=5, Lk=300, Hq=6, Hkv=2, dh=64),
    dict(B=2, Lq=400, Lk=600, Hq=6, Hkv=2, dh=128, causal=True, q_lens=[400, 133]), dict(B=1, Lq=60, Lk=9000, Hq=2, Hkv=2, dh=64),
    dict(B=1, Lq=270, Lk=4300, Hq=20, Hkv=20, dh=32, slopes=True), dict(B=2, Lq=9, Lk=90, Hq=2, Hkv=1, dh=7),
], ids=lambda k: f"L{k['Lq']}-{k['Lk']}-{k['dh']}")
def test_attention_in_place(P, kw):
    """o over q: every row is read before it is written, and rows that are not used keep their values."""
    c = make(**kw)
    o, lse = run_attention(P, c)
    q = c["q"].clone()
    got, got_lse = run_attention(P, c, o=c["q"])
    for b, n in enumerate(lens(c, "q_lens", c["Lq"])):
        assert torch.equal(got[b, :n], o[b, :n]) and torch.equal(got[b, n:], q[b, n:])
    assert torch.equal(got_lse, lse)


def test_packed_outputs_of_eviction(P):
    """Kept keys and values side by side in one buffer, row by row."""
    B, L, H, dh, n = 2, 130, 3, 64, 40
    kv, out = (torch.randn(B, m, H, 2, dh, device="cuda").to(torch.bfloat16) for m in (L, n))
    mass = torch.rand(B, H, L, device="cuda")
    mass_out, idx = torch.zeros(B, H, n, device="cuda"), torch.zeros(B, H, n, device="cuda", dtype=torch.int32)
    k, v, ko, vo = kv[..., 0, :], kv[..., 1, :], out[..., 0, :], out[..., 1, :]
    prob = P.evict_problem(P.PSV_DTYPE_BF16, (B, L, H, dh), n, 1, 5, k_stride=k.stride()[:3], v_stride=v.stride()[:3],
                           k_out_stride=ko.stride()[:3], v_out_stride=vo.stride()[:3])
    P.psv_cache_evict(prob, at(k), at(v), at(mass), at(ko), at(vo), at(mass_out), at(idx), stream())
    c = dict(n=[L] * B, budget=n, sinks=1, recent=5, mass=mass)
    for b in range(B):
        for h in range(H):
            w = torch.as_tensor(T.evict_reference(c, b, h), device="cuda")
            assert torch.equal(ko[b, :, h], k[b, w, h]) and torch.equal(vo[b, :, h], v[b, w, h])


# ------------------------------------------------------------- long pieces

def test_a_piece_of_over_two_seconds_is_no_timeout(P):
    """2^28 capped keys in one work item, two of which one pair of SMs does: it takes longer
    than a wait that makes no progress may."""
    L, Lq, dh, n = 1 << 28, 76 * 256 + 1, 8, 500
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    k = torch.zeros(1, L, 1, dh, device="cuda", dtype=torch.bfloat16)
    k[..., 0] = -220.0  # a score of -622 for every row, -60 under the cap: no weight
    v = torch.zeros_like(k)
    some = torch.randperm(1 << 20, device="cuda", generator=g)[:n].sort().values * 256 + 77
    k[0, some, 0] = torch.randn(n, dh, device="cuda", generator=g).to(k.dtype)
    v[0, some, 0] = torch.randn(n, dh, device="cuda", generator=g).to(k.dtype)
    q = torch.randn(1, Lq, 1, dh, device="cuda", generator=g).to(k.dtype)
    q[..., 0] = 8.0
    c = dict(make(B=1), B=1, Lq=Lq, Lk=L, Hq=1, Hkv=1, dh=dh, q=q, k=k, v=v, cap=60.0)
    o, lse = run_attention(P, c)
    few = dict(c, Lk=n, k=k[:, some], v=v[:, some])  # (the others' weight is below 2^28 e^-59)
    check_attention(few, o, lse)


def test_a_mass_piece_of_over_two_seconds_is_no_timeout(P):
    """2^30 rows for one tile of keys, two of which one pair of SMs does.  The rows overlap in
    memory: row (i, h) is row i + h of a buffer; 500 of them give weight."""
    Lq, H, Lk, dh, lse0 = 1 << 24, 64, 76 * 256 + 1, 8, 5.0
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    rows = torch.zeros(Lq + H - 1, dh, device="cuda", dtype=torch.bfloat16)
    rows[:, 0] = 8.0  # scores of -85: no weight
    some = torch.randperm(Lq + H - 1, device="cuda", generator=g)[:500].sort().values
    rows[some] = torch.randn(500, dh, device="cuda", generator=g).to(rows.dtype)
    rows[some, 0] = 0.0
    k = torch.randn(1, Lk, 1, dh, device="cuda", generator=g).to(torch.bfloat16)
    k[..., 0] = -30.0
    lse = torch.full((1, H, Lq), lse0, device="cuda")
    out = torch.zeros(1, 1, Lk, device="cuda")
    prob = P.cache_problem(P.PSV_DTYPE_BF16, (1, Lq, H, dh), k.shape, q_stride=(Lq * dh, dh, dh))
    n = P.psv_cache_scratch_bytes(prob)
    s = torch.zeros(n, dtype=torch.uint8, device="cuda")
    P.psv_cache_mass(prob, at(rows), at(k), at(lse), 0, at(out), at(s), n, stream())
    torch.cuda.synchronize()
    T.no_error(s)
    # how many (i, h) are row r
    times = torch.minimum(torch.minimum(some + 1, Lq + H - 1 - some), torch.full_like(some, H)).double()
    x = rows[some].double() @ k[0, :, 0].double().T / dh**0.5
    want = (torch.exp(x - lse0) * times[:, None]).sum(0)
    # Of the 32000 weights of a key each of its 32 sums gets about 1000, at most 2^11 (each addition
    # off by 2^-24 of the sum); a score's products, exp2 and its argument take 2^-17.
    tol = want * (2.0**-13 + 2.0**-17)
    d = (out[0, 0].double() - want).abs()
    assert (d <= tol).all(), float((d / tol).max())

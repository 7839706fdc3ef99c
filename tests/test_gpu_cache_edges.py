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

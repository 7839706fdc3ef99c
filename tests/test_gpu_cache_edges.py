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
from test_gpu_cache_ops import P, at, check_attention, check_mass, code, docs, ints, lens, make, run_attention, run_mass, stream  # noqa: E402,F401


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

# ------------------------------------------------------------------- caps

def capped_scores(c, b, h):
    """As the main tests' head_scores, but a cap over 128 costs 2^-21 of the capped score, not of the cap.

    Up to the cap the score is s P(z), z = (s / cap)^2: P is interpolated to 2^-24, z is off by three
    roundings (2^-22.4, of which P, whose logarithm changes at most a third as fast as z's, takes
    2^-24), P and its product round four times (2^-22).  Beyond it, t = (1 - a) / (1 + a), a = e^-2x <=
    0.14: a is off by (2 x + 2) 2^-23, of which t takes 0.28, the reciprocal by 2^-23, and t and its
    product round four times: 2^-21.2.  Caps up to 128 may take t = 1 - 2 / (1 + e^2x) throughout: e^2x
    off by (2 |x| + 2) 2^-23, the sum by 2^-24, the reciprocal by 2^-23, 2^-21 of the cap at most.
    """
    s, es, ok, nq, nk = T_head_scores(dict(c, cap=0.0, slopes=None), b, h)
    if c["cap"]:
        cap = float(np.float32(c["cap"]))
        s = cap * torch.tanh(s / cap)
        es = es + 2.0**-21 * (s.abs() if cap > 128 else cap)
    if c["slopes"] is not None:
        dev = s.device
        qp = c["q_pos"][b, :nq].long() if c["q_pos"] is not None else torch.arange(nq, device=dev) + nk - nq
        kp = c["k_pos"]
        kp = torch.arange(nk, device=dev) if kp is None else (kp[b, h // (c["Hq"] // c["Hkv"])] if kp.dim() == 3 else kp[b])[:nk].long()
        far = c["slopes"][h].double() * (qp[:, None] - kp).abs().double()
        s = s - far
        es = es + 2.0**-22 * far.abs() + 2.0**-22 * s.abs()
    return s, es, ok, nq, nk


T_head_scores = T.head_scores

CAP_SHAPES = {
    "token": dict(B=3, Lq=1, Lk=333, Hq=4, Hkv=4, dh=128, k_lens=[333, 1, 70]),
    "rows": dict(B=2, Lq=5, Lk=700, Hq=6, Hkv=2, dh=64, causal=True, dtype="f16"),
    "ragged": dict(B=3, Lq=40, Lk=300, Hq=4, Hkv=2, dh=128, q_lens=[40, 17, 1], k_lens=[300, 257, 40]),
    "many": dict(B=2, Lq=300, Lk=900, Hq=2, Hkv=1, dh=64, causal=True, slopes=True),
    "wide": dict(B=1, Lq=300, Lk=600, Hq=2, Hkv=2, dh=128, dtype="f16"),
    "general": dict(B=1, Lq=30, Lk=100, Hq=2, Hkv=1, dh=7, causal=True),
}


@pytest.mark.parametrize("cap", [1e-40, 1e-3, 2.0, 50.0, 300.0, 1e4, 1e6, 1e8, 1e20, 1e30, 3.4e38])
@pytest.mark.parametrize("shape", CAP_SHAPES)
def test_caps(P, monkeypatch, shape, cap):
    """Scores of deviation 1.5 and 8, and in one head a few far above the cap among small ones."""
    monkeypatch.setattr(T, "head_scores", capped_scores)
    for q_scale in (1.5, 8.0):
        c = make(**CAP_SHAPES[shape], cap=cap, q_scale=q_scale)
        c["q"][:, ::7, 0] *= 12.0
        o, lse = run_attention(P, c)
        check_attention(c, o, lse)
        mass_in = torch.rand(c["B"], c["Hkv"], c["Lk"], device="cuda")
        out = torch.full_like(mass_in, 3.0)
        run_mass(P, c, lse, mass_in, out)
        check_mass(c, lse, mass_in, out, torch.full_like(out, 3.0))


@pytest.mark.parametrize("Lq", [1, 40])
def test_a_large_cap_beside_far_larger_scores(P, monkeypatch, Lq):
    """One row's scores pass a cap of 1e6, the others' are small: each row's error follows its own."""
    monkeypatch.setattr(T, "head_scores", capped_scores)
    for dh in (64, 128):
        c = make(B=2, Lq=Lq, Lk=500, Hq=16, Hkv=4, dh=dh, cap=1e6, k_lens=[500, 333])
        c["q"][:, 0, 1::4] *= 1e6
        o, lse = run_attention(P, c)
        check_attention(c, o, lse)
        out = torch.zeros(2, 4, 500, device="cuda")
        run_mass(P, c, lse, None, out)
        check_mass(c, lse, None, out, torch.zeros_like(out))


def test_garbage_does_not_choose_how_scores_are_capped(P):
    """Unused rows and keys behind the lengths, however large, change no bit of the others."""
    for Lq, dh, cap in ((3, 64, 50.0), (3, 128, 1e6), (300, 128, 50.0), (300, 64, 20.0)):
        n, nq = [500, 301, 7], [Lq, Lq - 2, 1]
        c = make(B=3, Lq=Lq, Lk=500, Hq=4, Hkv=2, dh=dh, cap=cap, k_lens=n, q_lens=nq, q_scale=1.0)
        o, lse = run_attention(P, c)
        mass = torch.zeros(3, 2, 500, device="cuda")
        run_mass(P, c, lse, None, mass)
        for big in (3e38, float("inf"), float("nan"), 40.0):
            for b in range(3):
                c["k"][b, n[b]:] = big
                c["v"][b, n[b]:] = big
                c["q"][b, nq[b]:] = big
            got = run_attention(P, c)
            assert torch.equal(got[0], o) and torch.equal(got[1], lse)
            again = torch.zeros_like(mass)
            run_mass(P, c, lse, None, again)
            assert torch.equal(again, mass)

# -------------------------------------------------------------------- NaN

@pytest.mark.parametrize("kw", [
    dict(Lq=3, Lk=300, dh=128), dict(Lq=3, Lk=300, dh=64, cap=20.0), dict(Lq=3, Lk=70, dh=7),
    dict(Lq=60, Lk=300, dh=128), dict(Lq=60, Lk=9000, dh=64), dict(Lq=300, Lk=900, dh=64, slopes=True),
    dict(Lq=60, Lk=300, dh=128, cap=20.0, dtype="f16"), dict(Lq=60, Lk=90, dh=7, cap=5.0, slopes=True),
    dict(Lq=1, Lk=9000, dh=128),
], ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_nan_in_a_query_row_is_not_a_row_that_sees_nothing(P, kw):
    """Its output, lse and the weights of the keys it sees are NaN; no other row changes, and no
    weight of another sequence or kv head."""
    c = make(B=2, Hq=4, Hkv=2, causal=True, **kw)
    o, lse = run_attention(P, c)
    mass = torch.zeros(2, 2, c["Lk"], device="cuda")
    run_mass(P, c, lse, None, mass)
    i, h = c["Lq"] // 2, 3
    c["q"][1, i, h, 2] = float("nan")
    bad, bad_lse = run_attention(P, c)
    hit = torch.zeros(2, c["Lq"], 4, dtype=torch.bool, device="cuda")
    hit[1, i, h] = True
    assert bad[hit].isnan().all() and bad_lse.transpose(1, 2)[hit].isnan().all()
    assert torch.equal(bad[~hit], o[~hit]) and torch.equal(bad_lse.transpose(1, 2)[~hit], lse.transpose(1, 2)[~hit])

    def check(got):
        assert got[seen].isnan().all()
        assert torch.equal(got[0], mass[0]) and torch.equal(got[1, 0], mass[1, 0])
        rest = ~got[1, 1].isnan()
        assert torch.equal(got[1, 1][rest], mass[1, 1][rest])

    got = torch.zeros_like(mass)
    run_mass(P, c, bad_lse, None, got)
    seen = torch.zeros_like(mass, dtype=torch.bool)
    seen[1, 1, :c["Lk"] - c["Lq"] + i + 1] = True
    check(got)
    # an lse of NaN alone (the row itself is good) says the same
    c["q"][1, i, h, 2] = 0.25
    run_mass(P, c, bad_lse, None, got)
    check(got)


@pytest.mark.parametrize("Lq,dh", [(3, 64), (60, 128), (20, 7)])
def test_nan_in_a_key_that_a_row_sees(P, Lq, dh):
    doc = (np.arange(300) % 3)[None]
    c = make(B=1, Lq=Lq, Lk=300, Hq=2, Hkv=1, dh=dh, q_doc=(np.arange(Lq) % 3)[None], k_doc=doc)
    c["k"][0, 4] = float("nan")  # of document 1
    o, lse = run_attention(P, c)
    hit = torch.arange(Lq, device="cuda") % 3 == 1
    assert o[0, hit].isnan().all() and lse[0][:, hit].isnan().all()
    assert not o[0, ~hit].isnan().any() and not lse[0][:, ~hit].isnan().any()


# ------------------------------------------------------------------ status

def test_status_of_a_workspace(P):
    """0 after good calls; what a timed-out wait leaves in the first int; not within a capture."""
    c = make(B=2, Lq=40, Lk=300, Hq=2, Hkv=2, dh=64)
    prob = T.problem(P, c)
    scratch, n = T.scratch_for(P, prob)
    o, lse = torch.empty_like(c["q"]), torch.empty(2, 2, 40, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    P.psv_cache_attention(prob, at(c["q"]), at(c["k"]), at(c["v"]), at(o), at(lse), at(scratch), n, s.cuda_stream)
    assert P.psv_cache_status(at(scratch), s.cuda_stream) == 0
    assert P.psv_cache_status(at(scratch)) == 0
    scratch[:4].view(torch.int32).fill_(3)
    torch.cuda.synchronize()
    assert P.psv_cache_status(at(scratch), s.cuda_stream) == 3
    scratch.zero_()
    host = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(P.PSVError) as e:
        P.psv_cache_status((host.data_ptr() + 255) // 256 * 256, s.cuda_stream)
    assert e.value.code == P.PSV_EINVAL and "device memory" in str(e.value)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.psv_cache_attention(prob, at(c["q"]), at(c["k"]), at(c["v"]), at(o), at(lse), at(scratch), n, stream())
        with pytest.raises(P.PSVError) as e:
            P.psv_cache_status(at(scratch), stream())
        assert e.value.code == P.PSV_EINVAL and "captured" in str(e.value)
    want = o.clone()
    o.zero_()
    g.replay()
    assert P.psv_cache_status(at(scratch), stream()) == 0
    assert torch.equal(o, want)

# -------------------------------------------------------------------- rope

def test_rope_small_negative_frequencies_far_out(P):
    """A frequency just below zero turns as exactly as one just above it, up to positions of 2^31."""
    f = np.geomspace(1e-7, 1.0, 32)
    x = torch.zeros(1, 500, 1, 64, device="cuda")
    x[..., 0::2] = 1.0  # every pair becomes (cos, sin) of its angle: no rounding but theirs
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    pos = torch.randint(2**30, 2**31 - 1, (1, 500, 1), device="cuda", generator=g, dtype=torch.int32)
    # The turns per position are off by 2^-64 (2^-30 radians over 2^31 positions), of an angle 24 bits
    # are used (2^-23.3 radians), sine and cosine are good to 2 ulp (2^-23).
    tol = 2.0**-29 + 2.0**-23.3 + 2.0**-23
    for freqs in (f, -f):
        out = torch.empty_like(x)
        P.psv_rope(P.rope_problem(P.PSV_DTYPE_F32, x.shape, (64,), freqs=freqs), at(x), at(pos), at(out), stream())
        ref, _ = T.rope_reference(x.double(), pos, (64,), freqs=freqs)
        assert ((out.double() - ref).abs() <= tol).all(), float((out.double() - ref).abs().max())

# ---------------------------------------- masks and positions on every path

rng = np.random.default_rng(11)


def ring(n, turn, B=1):
    return np.broadcast_to((np.arange(n) + turn) % n, (B, n))


def heads(B, H, n):
    return np.stack([np.stack([rng.permutation(n) for _ in range(H)]) for _ in range(B)])


COVER = {
    # at most 16 rows a kv head
    "token-ring": dict(B=2, Lq=1, Lk=500, Hq=4, Hkv=2, dh=128, causal=True, k_pos=ring(500, 133, 2), q_pos=[[499], [250]]),
    "rows-ring-slopes": dict(B=2, Lq=4, Lk=333, Hq=4, Hkv=2, dh=64, causal=True, k_pos=ring(333, 100, 2), slopes=True,
                             k_lens=[333, 217], dtype="f16"),
    "rows-per-head": dict(B=2, Lq=3, Lk=500, Hq=6, Hkv=2, dh=80, causal=True, k_pos=heads(2, 2, 500), q_pos=[[3, 499, 200], [0, -4, 77]],
                          slopes=True),
    "rows-documents": dict(B=2, Lq=4, Lk=777, Hq=2, Hkv=2, dh=128, q_doc=[[0, 1, 2, 9], [2, 2, 0, 1]], k_doc=docs(2, 777, [1, 300, 640])),
    "rows-documents-per-head": dict(B=1, Lq=2, Lk=300, Hq=4, Hkv=2, dh=64, q_doc=[[1, 2]], k_doc=rng.integers(0, 4, (1, 2, 300)), cap=20.0),
    "rows-prefix": dict(B=3, Lq=4, Lk=260, Hq=2, Hkv=1, dh=128, causal=True, prefix=[100, 0, 9999], k_lens=[260, 33, 2], q_lens=[4, 1, 4]),
    "rows-all": dict(B=2, Lq=2, Lk=400, Hq=8, Hkv=1, dh=128, causal=True, prefix=[50, 7], cap=30.0, slopes=True, k_lens=[400, 399],
                     k_pos=ring(400, 31, 2), q_doc=[[0, 1], [1, 1]], k_doc=docs(2, 400, [200])),
    "rows-shares": dict(B=1, Lq=1, Lk=9001, Hq=2, Hkv=1, dh=64, causal=True, k_pos=ring(9001, 77), q_doc=[[1]], k_doc=docs(1, 9001, [4000, 8000])),
    # many rows, capped, with documents or positions
    "cap-documents": dict(B=2, Lq=600, Lk=600, Hq=2, Hkv=1, dh=64, cap=20.0, q_doc=docs(2, 600, [1, 100, 357]), k_doc=docs(2, 600, [1, 100, 357])),
    "cap-documents-wide": dict(B=1, Lq=700, Lk=700, Hq=2, Hkv=2, dh=128, cap=50.0, q_doc=docs(1, 700, [300, 301]), k_doc=docs(1, 700, [300, 301]),
                               dtype="f16", causal=True),
    "cap-ring": dict(B=2, Lq=300, Lk=1000, Hq=4, Hkv=2, dh=128, cap=30.0, causal=True, k_pos=ring(1000, 333, 2), k_lens=[1000, 700]),
    "cap-ring-slopes": dict(B=2, Lq=300, Lk=1000, Hq=4, Hkv=2, dh=128, cap=30.0, causal=True, k_pos=ring(1000, 333, 2), slopes=True),
    "cap-per-head-slopes": dict(B=1, Lq=260, Lk=700, Hq=4, Hkv=2, dh=64, cap=5.0, causal=True, k_pos=heads(1, 2, 700),
                                q_pos=rng.integers(-10, 800, (1, 260)), slopes=True, dtype="f16"),
    "cap-documents-slopes": dict(B=1, Lq=500, Lk=500, Hq=2, Hkv=1, dh=64, cap=10.0, slopes=True, q_doc=rng.integers(0, 3, (1, 500)),
                                 k_doc=rng.integers(0, 3, (1, 500))),
    "cap-prefix-lens": dict(B=3, Lq=300, Lk=600, Hq=2, Hkv=2, dh=128, cap=50.0, causal=True, prefix=[100, 0, 600], k_lens=[600, 300, 0],
                            q_lens=[300, 299, 12]),
    # the kernels for every layout
    "general-ring": dict(B=2, Lq=20, Lk=150, Hq=2, Hkv=1, dh=7, causal=True, k_pos=ring(150, 40, 2), slopes=True, k_lens=[150, 99]),
    "general-per-head": dict(B=1, Lq=9, Lk=100, Hq=4, Hkv=2, dh=256, causal=True, k_pos=heads(1, 2, 100), q_pos=rng.integers(0, 100, (1, 9)), cap=10.0),
    "general-documents": dict(B=2, Lq=33, Lk=120, Hq=2, Hkv=2, dh=130, q_doc=docs(2, 33, [5, 20]), k_doc=docs(2, 120, [50, 70]), dtype="f16"),
    "general-prefix": dict(B=2, Lq=40, Lk=90, Hq=2, Hkv=1, dh=36, causal=True, prefix=[60, 0], slopes=True, q_lens=[40, 3]),
    "general-groups": dict(Lq=2, Lk=60, Hq=160, Hkv=1, dh=64, causal=True, slopes=True),
}


@pytest.mark.parametrize("name", COVER)
def test_masks_and_positions(P, name):
    c = make(**COVER[name])
    o, lse = run_attention(P, c)
    check_attention(c, o, lse)
    mass_in = torch.rand(c["B"], c["Hkv"], c["Lk"], device="cuda")
    out = torch.full_like(mass_in, 3.0)
    run_mass(P, c, lse, mass_in, out)
    check_mass(c, lse, mass_in, out, torch.full_like(out, 3.0))


@pytest.mark.parametrize("kw", [
    dict(Lq=1, Hq=4, dh=128), dict(Lq=3, Hq=4, dh=64, cap=20.0), dict(Lq=2, Hq=16, dh=80, slopes=True, dtype="f16"),
    dict(Lq=1, Hq=2, dh=32, causal=True), dict(Lq=7, Hq=2, dh=36), dict(Lq=100, Hq=4, dh=128), dict(Lq=100, Hq=4, dh=64, cap=20.0),
    dict(Lq=300, Hq=6, dh=128, slopes=True, causal=True),
], ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_what_lies_behind_the_lengths_changes_nothing(P, kw):
    """NaN and infinities behind keys that end anywhere in a tile, and in unused rows: the same bits."""
    n = [300, 257, 256, 97, 33, 32, 31, 1, 0]
    Lq = kw["Lq"]
    nq = [Lq, max(1, Lq - 1), Lq, Lq // 2, Lq, 1, Lq, 0, Lq]
    c = make(B=len(n), Lk=300, Hkv=2, k_lens=n, q_lens=nq, **kw)
    o, lse = run_attention(P, c)
    check_attention(c, o, lse)
    mass = torch.full((len(n), 2, 300), 2.0, device="cuda")
    run_mass(P, c, lse, None, mass)
    check_mass(c, lse, None, mass, torch.full_like(mass, 2.0))
    for bad in (float("nan"), float("inf"), -float("inf")):
        for b in range(len(n)):
            c["k"][b, n[b]:] = bad
            c["v"][b, n[b]:] = bad
            c["v"][b, n[b]:, :, ::2] = float("nan")
            c["q"][b, nq[b]:] = bad
            lse[b, :, nq[b]:] = bad
        got = run_attention(P, c, lse=torch.where(torch.isfinite(lse) | (lse == -math.inf), lse, torch.full_like(lse, 9.0)))
        assert torch.equal(got[0], o)
        for b in range(len(n)):
            assert torch.equal(got[1][b, :, :nq[b]], lse[b, :, :nq[b]])
        again = torch.full_like(mass, 2.0)
        run_mass(P, c, lse, None, again)
        assert torch.equal(again, mass)


# ---------------------------------------------------------------- eviction

EVICT = {
    "8192": dict(B=1, L=8192, H=1, dh=8, budget=8000, sinks=4, recent=100),
    "8193": dict(B=2, L=8193, H=1, dh=32, budget=3000, sinks=1, recent=700, lens=[8193, 8192], values="ties"),
    "12480": dict(B=2, L=12480, H=3, dh=64, budget=9360, sinks=30, recent=1560, lens=[12480, 11000]),
    "16384": dict(B=1, L=16384, H=2, dh=32, budget=16383, sinks=0, recent=0),
    "16384-strange": dict(B=1, L=16384, H=1, dh=32, budget=700, sinks=3, recent=60, values="strange"),
    "16385": dict(B=2, L=16385, H=1, dh=32, budget=5000, sinks=3, recent=60, lens=[16385, 3], values="ties"),
    "20000": dict(B=2, L=20000, H=2, dh=64, budget=12000, sinks=4, recent=2000, lens=[20000, 12001]),
    "20002-zeros": dict(B=1, L=20002, H=1, dh=7, budget=9, sinks=4, recent=5, values="zeros"),
    "49152": dict(B=1, L=49152, H=1, dh=32, budget=30000, sinks=1, recent=1000, values="strange"),
    "49153": dict(B=1, L=49153, H=1, dh=32, budget=30001, sinks=1, recent=1000, values="ties"),
    "1023": dict(B=2, L=1023, H=2, dh=64, budget=600, sinks=1, recent=9, lens=[1023, 601], values="ties"),
    "4097": dict(B=1, L=4097, H=2, dh=128, budget=2049, sinks=1, recent=9),
}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("name", EVICT)
def test_evict_sizes(P, monkeypatch, name, dtype):
    monkeypatch.setitem(T.EVICT, name, EVICT[name])
    T.test_evict(P, name, dtype)


def test_evict_unaligned_mass_of_many_slots(P):
    """Rows of the mass that do not start on 16 bytes, in the selection with 32 slots a thread."""
    L, n = 12481, 5000
    k = torch.randn(1, L, 2, 32, device="cuda").half()
    mass = torch.rand(2 * L + 1, device="cuda")[1:].view(1, 2, L)
    ko, vo = (torch.zeros(1, n, 2, 32, device="cuda", dtype=torch.float16) for _ in range(2))
    mo, idx = torch.zeros(1, 2, n, device="cuda"), torch.zeros(1, 2, n, device="cuda", dtype=torch.int32)
    prob = P.evict_problem(P.PSV_DTYPE_F16, k.shape, n, 3, 1000)
    P.psv_cache_evict(prob, at(k), at(k), at(mass), at(ko), at(vo), at(mo), at(idx), stream())
    for h in range(2):
        w = torch.as_tensor(T.evict_reference(dict(n=[L], budget=n, sinks=3, recent=1000, mass=mass), 0, h), device="cuda")
        assert torch.equal(idx[0, h].long(), w) and torch.equal(mo[0, h], mass[0, h, w]) and torch.equal(ko[0, :, h], k[0, w, h])
        assert torch.equal(vo[0, :, h], ko[0, :, h])


# ------------------------------------------------------ captured and replayed

@pytest.mark.parametrize("kw", [
    dict(B=2, Lq=300, Lk=900, Hq=4, Hkv=2, dh=128, causal=True, slopes=True),
    dict(B=2, Lq=600, Lk=600, Hq=6, Hkv=3, dh=64, q_doc=docs(2, 600, [40, 41, 300]), k_doc=docs(2, 600, [40, 41, 300])),
    dict(B=1, Lq=270, Lk=4300, Hq=20, Hkv=20, dh=32),                                            # a last unit in shares
    dict(B=1, Lq=40, Lk=9000, Hq=2, Hkv=1, dh=128, cap=30.0, slopes=True),                       # shares of the keys
    dict(B=2, Lq=90, Lk=500, Hq=4, Hkv=2, dh=64, cap=1e5, causal=True, k_pos=ring(500, 99, 2)),  # a wide cap
    dict(B=2, Lq=9, Lk=200, Hq=2, Hkv=1, dh=7, causal=True),                                     # the general kernels
], ids=["bias", "documents", "last-unit", "shares", "wide-cap-ring", "general"])
def test_captured_many_rows(P, kw):
    """Attention, mass and rope in one graph, and a second graph on the same workspace, replayed in
    turn with other inputs and lengths: the eager calls' bits."""
    full = [kw["Lk"]] * kw["B"]
    c = make(k_lens=full, q_lens=[kw["Lq"]] * kw["B"], **kw)
    prob = T.problem(P, c)
    scratch, n = T.scratch_for(P, prob)
    pos = torch.randint(0, 500, (c["B"], c["Lq"], 1), device="cuda", dtype=torch.int32)
    dh = c["dh"] // 2 * 2
    turn = P.rope_problem(code(P, c["dtype"]), (c["B"], c["Lq"], c["Hq"], dh), (dh,)) if dh == c["dh"] else None
    raw = c["q"].clone()

    def buffers():
        return torch.zeros_like(c["q"]), torch.zeros(c["B"], c["Hq"], c["Lq"], device="cuda"), torch.zeros(c["B"], c["Hkv"], c["Lk"], device="cuda")

    def calls(o, lse, mass):
        if turn is not None:
            P.psv_rope(turn, at(raw), at(pos), at(c["q"]), stream())
        P.psv_cache_attention(prob, at(c["q"]), at(c["k"]), at(c["v"]), at(o), at(lse), at(scratch), n, stream())
        P.psv_cache_mass(prob, at(c["q"]), at(c["k"]), at(lse), 0, at(mass), at(scratch), n, stream())
        P.psv_cache_mass(prob, at(c["q"]), at(c["k"]), at(lse), at(mass), at(mass), at(scratch), n, stream())

    one, two, want = buffers(), buffers(), buffers()
    calls(*want)
    torch.cuda.synchronize()
    graphs = []
    for out in (one, two):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls(*out)
        graphs.append(g)
    for step in range(3):
        c["k_lens"].copy_(torch.tensor([max(0, x - 97 * step * (b + 1)) for b, x in enumerate(full)]))
        c["q_lens"].copy_(torch.tensor([max(0, c["Lq"] - 31 * step * b) for b in range(c["B"])]))
        (raw if turn is not None else c["q"]).normal_()
        pos.random_(0, 10000)
        for t in (*one, *two, *want):
            t.zero_()
        for _ in range(3):
            for g in graphs:
                g.replay()
        calls(*want)
        torch.cuda.synchronize()
        for got in (one, two):
            for x, y in zip(got, want):
                assert torch.equal(x, y)
    assert P.psv_cache_status(at(scratch), stream()) == 0


def test_captured_eviction(P):
    """A graph of an eviction follows the lengths and weights of its replay."""
    B, L, H, dh, n = 2, 9000, 2, 64, 4000
    k, v = (torch.randn(B, L, H, dh, device="cuda").to(torch.bfloat16) for _ in range(2))
    mass, kl = torch.rand(B, H, L, device="cuda"), ints([L, L])

    def buffers():
        return [torch.zeros(B, n, H, dh, device="cuda", dtype=torch.bfloat16) for _ in range(2)] + [
            torch.zeros(B, H, n, device="cuda"), torch.zeros(B, H, n, device="cuda", dtype=torch.int32), ints([0, 0])]

    def call(ko, vo, mo, idx, ln):
        prob = P.evict_problem(P.PSV_DTYPE_BF16, k.shape, n, 4, 500, k_lens=at(kl), lens_out=at(ln))
        P.psv_cache_evict(prob, at(k), at(v), at(mass), at(ko), at(vo), at(mo), at(idx), stream())

    got, want = buffers(), buffers()
    call(*got)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(*got)
    for new in ([L, L], [3999, 4001], [0, 8999]):
        kl.copy_(torch.tensor(new))
        mass.uniform_()
        for t in got + want:
            t.zero_()
        g.replay()
        call(*want)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


FIRST_CALLS = """
import sys
sys.path.insert(0, {root!r})
sys.path.insert(0, {tests!r})
import torch
import test_gpu_cache_ops as T
from autoregressive_denoising_dit_gb300 import _psv as P
c = T.make(B=2, Lq={Lq}, Lk=3000, Hq=4, Hkv=2, dh={dh}, causal=True, slopes={slopes}, cap={cap}, k_lens=[3000, 40])
prob = T.problem(P, c)
scratch, n = T.scratch_for(P, prob)
x, pos = torch.randn(2, 9, 3, 64, device="cuda"), torch.arange(18, device="cuda", dtype=torch.int32).view(2, 9, 1)
rope = P.rope_problem(P.PSV_DTYPE_F32, x.shape, (64,))
ev = P.evict_problem(P.PSV_DTYPE_BF16, c["k"].shape, 700, 4, 100, k_lens=T.at(c["k_lens"]))

def buffers():
    return (torch.zeros_like(c["q"]), torch.zeros(2, 4, {Lq}, device="cuda"), torch.zeros(2, 2, 3000, device="cuda"), torch.zeros_like(x),
            torch.zeros(2, 700, 2, {dh}, device="cuda", dtype=torch.bfloat16), torch.zeros(2, 700, 2, {dh}, device="cuda", dtype=torch.bfloat16),
            torch.zeros(2, 2, 700, device="cuda"), torch.zeros(2, 2, 700, device="cuda", dtype=torch.int32))

def calls(o, lse, mass, y, ko, vo, mo, idx):
    at, st = T.at, T.stream()
    P.psv_rope(rope, at(x), at(pos), at(y), st)
    P.psv_cache_attention(prob, at(c["q"]), at(c["k"]), at(c["v"]), at(o), at(lse), at(scratch), n, st)
    P.psv_cache_mass(prob, at(c["q"]), at(c["k"]), at(lse), 0, at(mass), at(scratch), n, st)
    P.psv_cache_evict(ev, at(c["k"]), at(c["v"]), at(mass), at(ko), at(vo), at(mo), at(idx), st)

got, want = buffers(), buffers()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls(*got)
g.replay()
calls(*want)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and float(want[1].abs().sum()) > 0
print("captured")
"""


@pytest.mark.parametrize("kw", [dict(Lq=1, dh=128, slopes=False, cap=0.0), dict(Lq=300, dh=128, slopes=False, cap=0.0),
                                dict(Lq=300, dh=64, slopes=True, cap=0.0), dict(Lq=90, dh=128, slopes=True, cap=500.0)],
                         ids=lambda k: f"{k['Lq']}-{k['dh']}-{k['cap']}")
def test_a_process_may_begin_with_a_capture(kw):
    """The first calls of a process, before any kernel is loaded, go into a graph."""
    import os
    import subprocess
    import sys

    tests = os.path.dirname(os.path.abspath(__file__))
    src = FIRST_CALLS.format(root=os.path.dirname(tests), tests=tests, **kw)
    r = subprocess.run([sys.executable, "-c", src], capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-1000:] + r.stderr[-3000:]


def test_calls_from_four_threads(P):
    """Calls at the same time, each thread with its own stream, workspace and outputs; errors stay with their thread."""
    import threading

    kinds = [dict(B=2, Lq=1, Lk=700, Hq=4, Hkv=2, dh=128), dict(B=1, Lq=300, Lk=900, Hq=2, Hkv=1, dh=64, causal=True),
             dict(B=1, Lq=40, Lk=5000, Hq=2, Hkv=2, dh=128, slopes=True), dict(B=2, Lq=90, Lk=600, Hq=2, Hkv=1, dh=64, cap=20.0)]
    cases = [make(seed=i, **kw) for i, kw in enumerate(kinds)]
    want = [run_attention(P, c) for c in cases]
    bad = []

    def work(i):
        try:
            c, s = cases[i], torch.cuda.Stream()
            prob = T.problem(P, c)
            scratch, n = T.scratch_for(P, prob)
            o, lse = torch.zeros_like(c["q"]), torch.zeros_like(want[i][1])
            torch.cuda.synchronize()
            for k in range(200):
                P.psv_cache_attention(prob, at(c["q"]), at(c["k"]), at(c["v"]), at(o), at(lse), at(scratch), n, s.cuda_stream)
                if k % 20 == i:
                    with pytest.raises(P.PSVError, match=f"scratch of {i} bytes"):
                        P.psv_cache_attention(prob, at(c["q"]), at(c["k"]), at(c["v"]), at(o), at(lse), at(scratch), i, s.cuda_stream)
            assert P.psv_cache_status(at(scratch), s.cuda_stream) == 0
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
        except BaseException as e:  # noqa: BLE001 (handed to the test's thread)
            bad.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad

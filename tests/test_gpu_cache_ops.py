"""The rolling-cache operators on the GPU against plain 64-bit implementations.

Tolerances are derived, element by element, from the roundings that the
operators make.  With u half a step of the operand type relative to the value
(bf16 2^-8, f16 2^-11, f32 2^-24):
  scores   dh products accumulated in f32, at worst one ulp (2^-23) lost a step:
           es = dh 2^-23 scale sum|q||k|, plus the cap's tanh to 2^-21 of the cap and the
           bias to 2^-22 of its size, plus 2^-22 of the score (exp2's argument)
  weights  exp(s) is off by a factor 1 + es + 2^-21, both in the numerator and the sum
  o        weights and output rounded once: u sum(p |v|) / l + u |o|, plus the weights' 2 es
  lse      es + 2^-21 + 2^-22 |lse|
  mass     (es + 2^-21 + rows 2^-24) of the added weight + 2^-23 of the result
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0**-8, "f16": 2.0**-11, "f32": 2.0**-24}
# Below 2^-14 f16 has a fixed step of 2^-24 (ten fraction bits at the exponent -14): half of it is
# the rounding there, whatever the value.  bf16 and f32 keep their relative step down to 2^-126.
STEP = {"bf16": 0.0, "f16": 2.0**-25, "f32": 0.0}


@pytest.fixture(scope="module")
def P():
    from autoregressive_denoising_dit_gb300 import _psv

    return _psv


def code(P, dtype):
    return {"bf16": P.PSV_DTYPE_BF16, "f16": P.PSV_DTYPE_F16, "f32": P.PSV_DTYPE_F32}[dtype]


def ints(a):
    return None if a is None else torch.as_tensor(np.array(a, order="C"), dtype=torch.int32, device="cuda")


def at(t):
    return 0 if t is None else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


# ------------------------------------------------------------------ rope

def rope_reference(x, pos, dims, theta=1e4, freqs=None, halves=False, inverse=False):
    """x [B, L, H, dh] float64, pos [B, L, axes]: rotated values and |a| + |b| of their pairs."""
    y, size = x.clone(), x.abs()
    R, first = sum(dims), 0
    for a, d in enumerate(dims):
        for j in range(d // 2):
            p = first + j
            f = freqs[p] if freqs is not None else theta ** (-2.0 * j / d)
            # the angle modulo 2 pi from whole turns in extended precision
            turns = pos[..., a].cpu().numpy().astype(np.longdouble) * (np.longdouble(f) / (2 * np.longdouble(np.pi) + 2 * np.longdouble(1.2246467991473532e-16)))
            th = torch.as_tensor(np.float64((turns - np.floor(turns)) * 2 * np.pi), device=x.device)[..., None]
            lo, hi = (p, p + R // 2) if halves else (2 * p, 2 * p + 1)
            c, s = torch.cos(th), torch.sin(th) * (-1.0 if inverse else 1.0)
            u, w = x[..., lo].clone(), x[..., hi].clone()
            y[..., lo], y[..., hi] = u * c - w * s, u * s + w * c
            size[..., lo] = size[..., hi] = u.abs() + w.abs()
        first += d // 2
    return y, size


ROPE = [
    dict(B=1, L=1, H=1, dh=2, dims=(2,)),
    dict(B=2, L=3, H=12, dh=128, dims=(44, 42, 42)),
    dict(B=3, L=101, H=3, dh=64, dims=(24, 20, 20), halves=True),
    dict(B=1, L=77, H=5, dh=80, dims=(16, 16), inverse=True),          # 48 values copied
    dict(B=2, L=50, H=2, dh=96, dims=(32, 16, 16), halves=True, inverse=True),  # halves, 32 copied
    dict(B=1, L=40, H=3, dh=50, dims=(20, 6, 4), halves=True),          # odd widths: value by value
    dict(B=1, L=33, H=2, dh=22, dims=(22,)),
    dict(B=1, L=9, H=2, dh=256, dims=(64, 64, 64, 64)),
    dict(B=4, L=1560, H=12, dh=128, dims=(44, 42, 42)),                 # several heads per thread
    dict(B=2, L=700, H=13, dh=128, dims=(64, 32, 32), halves=True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: f"B{c['B']}L{c['L']}H{c['H']}dh{c['dh']}")
def test_rope(P, case, dtype):
    c = dict(halves=False, inverse=False, **{k: v for k, v in case.items() if k not in ("halves", "inverse")})
    c.update({k: case[k] for k in ("halves", "inverse") if k in case})
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    shape = (c["B"], c["L"], c["H"], c["dh"])
    x = torch.randn(shape, device="cuda", generator=g).to(DT[dtype])
    pos = torch.randint(-100000, 100000, (c["B"], c["L"], len(c["dims"])), device="cuda", generator=g, dtype=torch.int32)
    out = torch.full_like(x, 7.0)
    prob = P.rope_problem(code(P, dtype), shape, c["dims"], halves=c["halves"], inverse=c["inverse"])
    P.psv_rope(prob, at(x), at(pos), at(out), stream())
    ref, size = rope_reference(x.double(), pos, c["dims"], halves=c["halves"], inverse=c["inverse"])
    # sin and cos to 2 ulp, angle to 2^-53 |pos| 2 pi + 2^-31, two products and a sum in f32
    tol = U[dtype] * ref.abs() + STEP[dtype] + size * (6 * 2.0**-24 + 2.0**-29)
    assert ((out.double() - ref).abs() <= tol).all()
    R = sum(c["dims"])
    assert torch.equal(out[..., R:], x[..., R:])
    y = x.clone()  # in place
    P.psv_rope(prob, at(y), at(pos), at(y), stream())
    assert torch.equal(y, out)


@pytest.mark.parametrize("offset", [0, 1])
def test_rope_strides_lengths_and_shared_positions(P, offset):
    B, L, H, dh = 3, 37, 4, 64
    base = torch.randn(B * L * 3 * H * dh + 8, device="cuda").to(torch.bfloat16)[offset:offset + B * L * 3 * H * dh]
    x = base.view(B, L, 3, H, dh)[:, :, 1]
    pos = torch.randint(0, 5000, (L, 2), device="cuda", dtype=torch.int32)
    out = torch.full((B, H, L, dh), -3.0, device="cuda", dtype=torch.bfloat16)  # heads before rows
    lens = ints([37, 0, 11])
    prob = P.rope_problem(P.PSV_DTYPE_BF16, (B, L, H, dh), (32, 32), x_stride=x.stride()[:3],
                          out_stride=(H * L * dh, dh, L * dh), pos_stride=(0, 2), lens=at(lens))
    P.psv_rope(prob, at(x), at(pos), at(out), stream())
    ref, size = rope_reference(x.double(), pos[None].expand(B, L, 2), (32, 32))
    got = out.transpose(1, 2)
    for b, n in enumerate((37, 0, 11)):
        tol = U["bf16"] * ref[b, :n].abs() + size[b, :n] * 2.0**-21
        assert ((got[b, :n].double() - ref[b, :n]).abs() <= tol).all()
        assert (got[b, n:] == -3.0).all()


def test_rope_far_positions_and_own_frequencies(P):
    B, L, H, dh = 1, 64, 2, 64
    freqs = np.concatenate([np.linspace(-3.0, 3.0, 16), np.geomspace(1e-6, 1.0, 16)])
    x = torch.randn(B, L, H, dh, device="cuda")
    pos = torch.randint(-2**31, 2**31 - 1, (B, L, 1), device="cuda", dtype=torch.int32)
    out = torch.empty_like(x)
    prob = P.rope_problem(P.PSV_DTYPE_F32, x.shape, (dh,), freqs=freqs)
    P.psv_rope(prob, at(x), at(pos), at(out), stream())
    ref, size = rope_reference(x.double(), pos, (dh,), freqs=freqs)
    # |pos| f 2^-53 of the reduced frequency: 2^31 * 3 * 2^-53 radians at most, both sides
    tol = U["f32"] * ref.abs() + size * (6 * 2.0**-24 + 2 * 3 * 2.0**-22)
    assert ((out.double() - ref).abs() <= tol).all()


def test_rope_inverse_is_the_gradient_and_undoes(P):
    """The rotation is orthogonal: <rope(x), g> = <x, inverse(g)>, and the gradient agrees with differences."""
    shape = (2, 19, 3, 64)
    x, g = torch.randn(shape, device="cuda"), torch.randn(shape, device="cuda")
    pos = torch.randint(0, 10000, (2, 19, 3), device="cuda", dtype=torch.int32)
    y, gx, back = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    fw = P.rope_problem(P.PSV_DTYPE_F32, shape, (24, 20, 20))
    bw = P.rope_problem(P.PSV_DTYPE_F32, shape, (24, 20, 20), inverse=True)
    P.psv_rope(fw, at(x), at(pos), at(y), stream())
    P.psv_rope(bw, at(g), at(pos), at(gx), stream())
    P.psv_rope(bw, at(y), at(pos), at(back), stream())
    assert (back - x).abs().max() <= 20 * 2.0**-24 * x.abs().max() * 2
    d = torch.randn(shape, device="cuda")
    z = torch.empty_like(x)
    P.psv_rope(fw, at(x + d), at(pos), at(z), stream())
    along = ((z.double() - y.double()) * g.double()).sum()
    # f32 roundings of each of the n terms, added at random and bounded by their sum of sizes
    assert abs(along - (d.double() * gx.double()).sum()) <= 2.0**-21 * ((z - y).abs() * g.abs()).double().sum() * 2


# ------------------------------------------------- attention over a cache

def make(dtype="bf16", B=1, Lq=1, Lk=1, Hq=1, Hkv=1, dh=64, seed=0, causal=False, prefix=None, cap=0.0, slopes=False,
         q_lens=None, k_lens=None, q_pos=None, k_pos=None, q_doc=None, k_doc=None, scale=0.0, q_scale=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rnd(*shape, s=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * s).to(DT[dtype])

    c = dict(dtype=dtype, B=B, Lq=Lq, Lk=Lk, Hq=Hq, Hkv=Hkv, dh=dh, causal=causal, cap=cap, scale=scale,
             q=rnd(B, Lq, Hq, dh, s=q_scale), k=rnd(B, Lk, Hkv, dh), v=rnd(B, Lk, Hkv, dh))
    if slopes is True:
        slopes = 2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)
    c["slopes"] = torch.tensor(slopes, dtype=torch.float32, device="cuda") if slopes is not False else None
    for name, value in dict(prefix=prefix, q_lens=q_lens, k_lens=k_lens, q_pos=q_pos, q_doc=q_doc).items():
        c[name] = ints(value)
    # [B][Lk] metadata is shared by the heads, [B][Hkv][Lk] is not
    c["k_pos"], c["k_doc"] = ints(k_pos), ints(k_doc)
    return c


def problem(P, c, **kw):
    meta = c["k_pos"] if c["k_pos"] is not None else c["k_doc"]
    ms = None
    if meta is not None:
        ms = (meta.stride(0), meta.stride(1)) if meta.dim() == 3 else (meta.stride(0), 0)
    return P.cache_problem(code(P, c["dtype"]), c["q"].shape, c["k"].shape, q_stride=c["q"].stride()[:3],
                           k_stride=c["k"].stride()[:3], v_stride=c["v"].stride()[:3], scale=c["scale"],
                           softcap=c["cap"], causal=c["causal"], q_lens=at(c["q_lens"]), k_lens=at(c["k_lens"]),
                           q_pos=at(c["q_pos"]), q_doc=at(c["q_doc"]), k_pos=at(c["k_pos"]), k_doc=at(c["k_doc"]),
                           k_meta_stride=ms, prefix=at(c["prefix"]), slopes=at(c["slopes"]), **kw)


def scratch_for(P, prob):
    n = P.psv_cache_scratch_bytes(prob)
    return torch.zeros(n, dtype=torch.uint8, device="cuda"), n


def no_error(scratch):
    assert int(scratch[:4].view(torch.int32).item()) == 0, "a device-side wait timed out"


def run_attention(P, c, o=None, lse=None, scratch=None, **kw):
    o = torch.full_like(c["q"].contiguous(), 5.0) if o is None else o
    lse = torch.full((c["B"], c["Hq"], c["Lq"]), 9.0, device="cuda") if lse is None else lse
    prob = problem(P, c, **kw)
    if scratch is None:
        scratch, n = scratch_for(P, prob)
    n = scratch.numel()
    P.psv_cache_attention(prob, at(c["q"]), at(c["k"]), at(c["v"]), at(o), at(lse), at(scratch), n, stream())
    torch.cuda.synchronize()
    no_error(scratch)
    return o, lse


def lens(c, name, full):
    return [full] * c["B"] if c[name] is None else [min(max(int(x), 0), full) for x in c[name].cpu()]


def head_scores(c, b, h):
    """Scores, their error bound and visibility of sequence b and head h in 64 bits (valid rows and keys)."""
    G = c["Hq"] // c["Hkv"]
    nq, nk = lens(c, "q_lens", c["Lq"])[b], lens(c, "k_lens", c["Lk"])[b]
    q, k = c["q"][b, :nq, h].double(), c["k"][b, :nk, h // G].double()
    scale = c["scale"] or 1.0 / math.sqrt(c["dh"])
    s = q @ k.T * scale
    es = c["dh"] * 2.0**-23 * scale * (q.abs() @ k.abs().T) + 2.0**-22 * s.abs()
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
        es = es + 2.0**-21 * c["cap"]

    def row(t):
        return (t[b, h // G] if t.dim() == 3 else t[b])[:nk].long()

    dev = s.device
    qp = c["q_pos"][b, :nq].long() if c["q_pos"] is not None else torch.arange(nq, device=dev) + nk - nq
    kp = row(c["k_pos"]) if c["k_pos"] is not None else torch.arange(nk, device=dev)
    if c["slopes"] is not None:
        far = c["slopes"][h].double() * (qp[:, None] - kp).abs().double()
        s = s - far
        es = es + 2.0**-22 * far.abs() + 2.0**-22 * s.abs()
    ok = torch.ones(nq, nk, dtype=torch.bool, device=dev)
    if c["causal"]:
        ok &= (kp <= qp[:, None]) | (kp < (int(c["prefix"][b]) if c["prefix"] is not None else -2**31))
    if c["k_doc"] is not None:
        ok &= c["q_doc"][b, :nq].long()[:, None] == row(c["k_doc"])
    return s, es, ok, nq, nk


def check_attention(c, o, lse, fill=5.0, lse_fill=9.0):
    G, u = c["Hq"] // c["Hkv"], U[c["dtype"]]
    for b in range(c["B"]):
        for h in range(c["Hq"]):
            s, es, ok, nq, nk = head_scores(c, b, h)
            assert (o[b, nq:, h] == fill).all() and (lse[b, h, nq:] == lse_fill).all()
            if nq == 0:
                continue
            v = c["v"][b, :nk, h // G].double()
            s = torch.where(ok, s, torch.full_like(s, -math.inf))
            m = s.amax(1, keepdim=True) if nk else torch.full((nq, 1), -math.inf, device=o.device, dtype=torch.float64)
            m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
            p = torch.exp(s - m0)
            l = p.sum(1, keepdim=True)
            some = l[:, 0] > 0
            got, gl = o[b, :nq, h].double(), lse[b, h, :nq].double()
            assert (got[~some] == 0).all() and (gl[~some] == -math.inf).all()
            if not some.any():
                continue
            p, l, es, m0 = p[some], l[some], torch.where(ok, es, torch.zeros_like(es))[some], m0[some]
            ref = p @ v / l
            worst = es.amax(1, keepdim=True)
            spread = p @ v.abs() / l
            tol = u * spread * 1.01 + u * ref.abs() * 1.01 + spread * (2 * worst + 2.0**-19) + 2.0**-25
            d = (got[some] - ref).abs()
            assert (d <= tol).all(), (b, h, float((d / tol).max()))
            want = (m0 + torch.log(l))[:, 0]
            tl = worst[:, 0] + 2.0**-21 + 2.0**-22 * want.abs()
            assert ((gl[some] - want).abs() <= tl).all(), (b, h, float(((gl[some] - want).abs() / tl).max()))


def docs(B, L, cuts):
    return np.broadcast_to(np.searchsorted(cuts, np.arange(L), side="right"), (B, L))


rng = np.random.default_rng(5)
ATTN = {
    "one": dict(),
    "one-key-many-rows": dict(Lq=300, Lk=1, dh=128),
    "token": dict(B=2, Lq=1, Lk=777, Hq=4, Hkv=4, dh=128),
    "token-long": dict(B=1, Lq=1, Lk=20011, Hq=2, Hkv=1, dh=128),
    "token-groups": dict(B=3, Lq=1, Lk=1000, Hq=16, Hkv=2, dh=128, dtype="f16", k_lens=[1000, 1, 513], causal=True),
    "draft": dict(B=2, Lq=5, Lk=600, Hq=6, Hkv=2, dh=64, causal=True, cap=30.0),
    "odd": dict(B=2, Lq=101, Lk=333, Hq=3, Hkv=3, dh=64, k_lens=[333, 257]),
    "tile": dict(Lq=256, Lk=256, Hq=2, Hkv=1, dh=128),
    "tile+1": dict(Lq=257, Lk=257, Hq=2, Hkv=1, dh=128, causal=True),
    "width32": dict(Lq=70, Lk=130, Hq=4, Hkv=4, dh=32, slopes=True),
    "width80": dict(Lq=70, Lk=300, Hq=2, Hkv=2, dh=80, dtype="f16"),
    "width40": dict(Lq=7, Lk=90, Hq=2, Hkv=2, dh=40, causal=True),
    "width256": dict(Lq=9, Lk=70, Hq=2, Hkv=1, dh=256),
    "width7": dict(Lq=5, Lk=40, Hq=2, Hkv=1, dh=7, cap=5.0),
    "groups3": dict(Lq=100, Lk=400, Hq=6, Hkv=2, dh=128, causal=True, slopes=True),
    "groups40": dict(Lq=11, Lk=300, Hq=40, Hkv=1, dh=64, causal=True),
    "groups128": dict(Lq=3, Lk=300, Hq=128, Hkv=1, dh=64),
    "groups160": dict(Lq=2, Lk=60, Hq=160, Hkv=1, dh=64),
    "causal-short-keys": dict(B=2, Lq=300, Lk=200, Hq=2, Hkv=2, dh=64, causal=True),  # rows that see nothing
    "causal-long": dict(Lq=700, Lk=1500, Hq=2, Hkv=1, dh=128, causal=True, dtype="f16"),
    "prefix": dict(B=2, Lq=500, Lk=500, Hq=2, Hkv=2, dh=64, causal=True, prefix=[130, 0]),
    "prefix-beyond": dict(B=2, Lq=300, Lk=300, Hq=1, Hkv=1, dh=64, causal=True, prefix=[100000, -5]),
    "cap": dict(Lq=200, Lk=600, Hq=2, Hkv=2, dh=128, cap=20.0, q_scale=12.0),
    "cap-huge": dict(Lq=200, Lk=300, Hq=2, Hkv=2, dh=128, cap=1.0, q_scale=60.0),
    "scale": dict(Lq=60, Lk=300, Hq=2, Hkv=2, dh=64, scale=0.5),
    "large-scores": dict(Lq=60, Lk=900, Hq=2, Hkv=2, dh=64, q_scale=100.0),
    "bias": dict(B=2, Lq=300, Lk=900, Hq=4, Hkv=2, dh=128, slopes=True, k_lens=[900, 400]),
    "bias-causal-cap": dict(B=1, Lq=300, Lk=900, Hq=4, Hkv=4, dh=128, slopes=True, causal=True, cap=50.0, dtype="f16"),
    "bias-both-sides": dict(B=2, Lq=1100, Lk=1300, Hq=2, Hkv=2, dh=128, slopes=True, k_lens=[1300, 1111]),
    "bias-both-sides-f16": dict(Lq=900, Lk=900, Hq=6, Hkv=2, dh=64, slopes=True, dtype="f16"),
    "bias-steep": dict(Lq=600, Lk=800, Hq=4, Hkv=4, dh=64, slopes=[3.0, 1e5, 0.0, 1e-4], dtype="f16"),
    "bias-signs": dict(Lq=600, Lk=800, Hq=4, Hkv=2, dh=64, slopes=[0.01, -0.01, 1e-7, 0.3], causal=True),
    "bias-rows": dict(Lq=1, Lk=800, Hq=4, Hkv=4, dh=64, slopes=[0.01, -0.01, 0.0, 1e4]),
    "lens": dict(B=5, Lq=200, Lk=700, Hq=2, Hkv=1, dh=64, k_lens=[0, 1, 256, 699, 5000], q_lens=[200, 1, 0, 129, 4000]),
    "lens-causal": dict(B=5, Lq=200, Lk=700, Hq=2, Hkv=1, dh=64, k_lens=[0, 1, 256, 700, -3], q_lens=[200, 100, 199, 129, 7],
                        causal=True, slopes=True),
    "docs": dict(B=2, Lq=600, Lk=600, Hq=2, Hkv=2, dh=64, q_doc=docs(2, 600, [1, 100, 357]), k_doc=docs(2, 600, [1, 100, 357])),
    "docs-causal": dict(B=1, Lq=900, Lk=900, Hq=2, Hkv=1, dh=128, q_doc=docs(1, 900, [300, 301, 640]),
                        k_doc=docs(1, 900, [300, 301, 640]), causal=True, slopes=True),
    "docs-unseen": dict(B=1, Lq=300, Lk=600, Hq=2, Hkv=1, dh=64, q_doc=np.arange(300)[None] // 50, k_doc=np.zeros((1, 600))),
    "docs-mixed": dict(B=2, Lq=300, Lk=1100, Hq=2, Hkv=1, dh=64, q_doc=rng.integers(0, 4, (2, 300)), k_doc=rng.integers(0, 4, (2, 1100))),
    "ring": dict(B=2, Lq=300, Lk=1000, Hq=4, Hkv=2, dh=128, causal=True, k_pos=np.broadcast_to((np.arange(1000) + 333) % 1000, (2, 1000)),
                 slopes=True),
    "positions-per-head": dict(B=2, Lq=40, Lk=500, Hq=4, Hkv=2, dh=64, causal=True, slopes=True,
                               k_pos=np.stack([np.stack([rng.permutation(500) for _ in range(2)]) for _ in range(2)]),
                               q_pos=rng.integers(-10, 600, (2, 40))),
    "positions-far": dict(Lq=70, Lk=300, Hq=2, Hkv=1, dh=64, causal=True, k_pos=np.arange(300)[None] + 2**30 - 400,
                          q_pos=np.arange(70)[None] + 2**30 - 150, slopes=True),
    "many-sequences": dict(B=70, Lq=3, Lk=100, Hq=4, Hkv=2, dh=64, causal=True),
}


@pytest.mark.parametrize("name", ATTN)
def test_attention(P, name):
    c = make(**ATTN[name])
    check_attention(c, *run_attention(P, c))


def test_attention_strides_and_no_lse(P):
    """q, k, v as slices of one projection, o with heads before rows, no lse."""
    B, L, H, dh = 2, 150, 3, 64
    c = make(B=B, Lq=L, Lk=L, Hq=H, Hkv=H, dh=dh, causal=True)
    qkv = torch.randn(B, L, 3, H, dh, device="cuda").to(torch.bfloat16)
    c["q"], c["k"], c["v"] = (qkv[:, :, i] for i in range(3))
    o = torch.full((B, H, L, dh), 5.0, device="cuda", dtype=torch.bfloat16)
    prob = problem(P, c, o_stride=(H * L * dh, dh, L * dh))
    s, n = scratch_for(P, prob)
    P.psv_cache_attention(prob, at(c["q"]), at(c["k"]), at(c["v"]), at(o), 0, at(s), n, stream())
    want, lse = run_attention(P, c)
    assert torch.equal(o.transpose(1, 2), want)
    check_attention(c, want, lse)


@pytest.mark.parametrize("which", ["q", "k", "v", "o"])
def test_attention_unaligned(P, which):
    """A base or a stride off 16 bytes takes the general kernel and gives the same result within tolerance."""
    c = make(B=2, Lq=20, Lk=150, Hq=2, Hkv=1, dh=64, causal=True)
    o = torch.full((2, 20, 2, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    kw = {}
    if which == "o":
        o = torch.full((2 * 20 * 2 * 64 + 1,), 5.0, device="cuda", dtype=torch.bfloat16)[1:].view(2, 20, 2, 64)
    else:
        t = c[which]
        wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 1, device="cuda", dtype=t.dtype)
        wide[..., :-1] = t
        c[which] = wide[..., :-1]
    lse = torch.full((2, 2, 20), 9.0, device="cuda")
    run_attention(P, c, o, lse, **kw)
    check_attention(c, o, lse)


def test_attention_broadcast_keys(P):
    """One cache read by every sequence (batch stride 0)."""
    c = make(B=3, Lq=30, Lk=400, Hq=2, Hkv=2, dh=64)
    c["k"] = c["k"][:1].expand(3, -1, -1, -1)
    c["v"] = c["v"][:1].expand(3, -1, -1, -1)
    check_attention(c, *run_attention(P, c))


def test_attention_ignores_what_lies_behind_the_keys(P):
    """NaN and infinities behind k_lens, and unused rows of q, change nothing."""
    for dh, L in ((64, 300), (128, 511), (128, 200)):
        c = make(B=3, Lq=40, Lk=L, Hq=4, Hkv=2, dh=dh, k_lens=[L - 3, 1, L // 2 + 7], q_lens=[40, 17, 1])
        want = run_attention(P, c)
        for b, (nk, nq) in enumerate(zip([L - 3, 1, L // 2 + 7], [40, 17, 1])):
            c["k"][b, nk:] = float("nan")
            c["v"][b, nk:] = float("inf")
            c["v"][b, nk:, :, ::2] = float("nan")
            c["q"][b, nq:] = float("nan")
        got = run_attention(P, c)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_masked_keys_may_be_infinite_scores(P):
    """A masked key's score is not used, whatever it is."""
    c = make(Lq=30, Lk=300, Hq=1, Hkv=1, dh=64, q_doc=np.zeros((1, 30)), k_doc=(np.arange(300) % 3 == 1)[None].astype(int))
    want = run_attention(P, c)
    hidden = torch.arange(300, device="cuda") % 3 == 1
    c["k"][0, hidden] = 3.0e38
    got = run_attention(P, c)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_no_keys_at_all(P):
    c = make(B=2, Lq=5, Lk=0, Hq=2, Hkv=1, dh=64)
    o, lse = run_attention(P, c)
    assert (o == 0).all() and (lse == -math.inf).all()


def test_attention_repeats_and_is_batch_invariant(P):
    """The same bits again, and for a sequence alone as in a batch."""
    c = make(B=4, Lq=33, Lk=3000, Hq=4, Hkv=2, dh=128, k_lens=[3000, 700, 2222, 1], causal=True)
    a, la = run_attention(P, c)
    b, lb = run_attention(P, c)
    assert torch.equal(a, b) and torch.equal(la, lb)
    one = dict(c, B=1, q=c["q"][2:3], k=c["k"][2:3], v=c["v"][2:3], k_lens=c["k_lens"][2:3].clone())
    o, lse = run_attention(P, one)
    assert torch.equal(o[0], a[2]) and torch.equal(lse[0], la[2])


@pytest.mark.parametrize("kw", [
    dict(Lq=300, Hq=20, Hkv=20, dh=32),
    dict(Lq=270, Hq=20, Hkv=20, dh=64, slopes=True, dtype="f16", q_lens=[270, 257, 256, 3]),
    dict(Lq=100, Hq=60, Hkv=20, dh=48, cap=20.0),
    dict(Lq=257, Hq=20, Hkv=20, dh=32, causal=False, k_pos=np.broadcast_to((np.arange(4300) + 999) % 4300, (4, 4300)), slopes=True),
], ids=["plain", "bias", "groups-cap", "ring"])
def test_attention_last_unit_in_shares(P, kw):
    """A last unit of few rows is done in shares of the keys (also empty ones), the same alone as in a batch."""
    n = [4300, 4100, 700, 0]
    c = make(B=4, Lk=4300, k_lens=n, **kw)
    o, lse = run_attention(P, c)
    check_attention(c, o, lse)
    for b in (1, 2):
        one = dict(c, B=1, **{x: c[x][b:b + 1].clone() for x in ("q", "k", "v", "k_lens", "q_lens", "k_pos") if c[x] is not None})
        a, la = run_attention(P, one)
        assert torch.equal(a[0], o[b]) and torch.equal(la[0], lse[b])


@pytest.mark.parametrize("Lq,G,dh", [(1, 1, 128), (3, 5, 64), (4, 2, 80)])
def test_tokens_alone_and_in_a_batch(P, Lq, G, dh):
    """Few rows: the shares of one sequence's few heads are joined elsewhere than those of many, to the same bits."""
    B, H = 12, 6
    c = make(B=B, Lq=Lq, Lk=2500, Hq=H * G, Hkv=H, dh=dh, k_lens=[2500 - 190 * b for b in range(B)], slopes=True)
    o, lse = run_attention(P, c)
    check_attention(c, o, lse)
    s, n = scratch_for(P, problem(P, c))
    for b in (0, 5, 11):
        one = dict(c, B=1, q=c["q"][b:b + 1], k=c["k"][b:b + 1], v=c["v"][b:b + 1], k_lens=c["k_lens"][b:b + 1].clone())
        for _ in range(3):  # one workspace for all of them
            a, la = run_attention(P, one, scratch=s)
            assert torch.equal(a[0], o[b]) and torch.equal(la[0], lse[b])


@pytest.mark.parametrize("kw", [
    dict(Lq=4400, Lk=8800, Hq=24, Hkv=8, dh=128, causal=True, prefix=[880], cap=50.0, dtype="f16"),
    dict(B=9, Lq=3, Lk=40, Hq=12, Hkv=12, dh=64, k_lens=[40, 1, 0, 7, 33, 39, 12, 40, 3]),
    dict(B=40, Lq=1, Lk=700, Hq=4, Hkv=4, dh=128, k_lens=list(range(660, 700))),
], ids=["long", "one-tile-pieces", "shares"])
def test_attention_many_pieces_many_times(P, kw):
    """Several work pieces per pair of SMs, launched over and over with and without a gap: the
    hand-over of pieces between the two SMs never mixes them up."""
    c = make(**kw)
    want = run_attention(P, c)
    prob = problem(P, c)
    scratch, n = scratch_for(P, prob)
    o, lse = torch.zeros_like(c["q"]), torch.zeros(c["B"], c["Hq"], c["Lq"], device="cuda")
    for i in range(300):
        P.psv_cache_attention(prob, at(c["q"]), at(c["k"]), at(c["v"]), at(o), at(lse), at(scratch), n, stream())
        if i % 2:
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    no_error(scratch)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("kw", [
    dict(B=2, Lq=2100, Lk=2100, Hq=40, Hkv=40, dh=32, k_lens=[2100, 1300], q_lens=[2100, 700]),  # more heads than sorted at a time
    dict(B=1, Lq=2500, Lk=2500, Hq=6, Hkv=2, dh=128, dtype="f16"),
], ids=["heads", "groups"])
def test_attention_uneven_documents(P, kw):
    """Units of rows that see far more keys than others are taken first; every one is done, once."""
    B, L = kw["B"], kw["Lk"]
    d = docs(B, L, [40, 1100, 1101, 1900])
    c = make(q_doc=d, k_doc=d, **kw)
    o, lse = run_attention(P, c)
    check_attention(c, o, lse)
    again = run_attention(P, c)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("kw", [
    dict(B=3, Lq=40, Lk=900, k_lens=[900, 1, 611], q_lens=[40, 17, 1]),
    dict(B=2, Lq=700, Lk=1500, k_lens=[1031, 520]),             # rows in the last tiles, or before the first key
    dict(B=1, Lq=700, Lk=1500, k_lens=[700]),                    # rows among the keys
    dict(B=1, Lq=40, Lk=9000, k_lens=[8000], cap=30.0),          # shares of the keys, with a cap
    dict(B=1, Lq=300, Lk=1500, k_lens=[1200], causal=True),
], ids=["short", "long", "square", "shares", "causal"])
def test_attention_biased_with_unused_keys(P, kw):
    """With a distance bias the tile behind which no keys lie is not the last one taken."""
    c = make(Hq=4, Hkv=2, dh=128, slopes=True, **kw)
    o, lse = run_attention(P, c)
    check_attention(c, o, lse)
    for b, nk in enumerate(kw["k_lens"]):
        c["k"][b, nk:] = float("nan")
        c["v"][b, nk:] = float("nan")
    got = run_attention(P, c)
    assert torch.equal(got[0], o) and torch.equal(got[1], lse)


def test_attention_long_cache_offsets(P):
    """A cache whose offsets pass 2^31 elements: the last sequence reads its own keys."""
    B, L, H, dh = 5, 36000, 100, 128
    k = torch.zeros(B, L, H, dh, device="cuda", dtype=torch.bfloat16)
    assert k.numel() > 2**31
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    k[-1, -700:] = torch.randn(700, H, dh, device="cuda", generator=g).to(k.dtype)
    v[-1, -700:] = torch.randn(700, H, dh, device="cuda", generator=g).to(k.dtype)
    q = torch.randn(B, 2, H, dh, device="cuda", generator=g).to(k.dtype)
    c = dict(make(B=1), B=B, Lq=2, Lk=L, Hq=H, Hkv=H, dh=dh, q=q, k=k, v=v)
    o, lse = run_attention(P, c)
    for h in (0, 57, 99):
        s = q[-1, :, h].double() @ k[-1, :, h].double().T / dh**0.5
        p = torch.softmax(s, 1)
        ref = p @ v[-1, :, h].double()
        tol = U["bf16"] * 1.01 * (p @ v[-1, :, h].double().abs() + ref.abs()) + 2.0**-16
        assert ((o[-1, :, h].double() - ref).abs() <= tol).all()
        assert (lse[-1, h].double() - torch.logsumexp(s, 1)).abs().max() <= 1e-4


# ------------------------------------------------------------------ mass

def run_mass(P, c, lse, mass_in, mass_out):
    prob = problem(P, c)
    s, n = scratch_for(P, prob)
    P.psv_cache_mass(prob, at(c["q"]), at(c["k"]), at(lse), at(mass_in), at(mass_out), at(s), n, stream())
    torch.cuda.synchronize()
    no_error(s)


def check_mass(c, lse, mass_in, got, fill):
    G = c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        for g in range(c["Hkv"]):
            nk = lens(c, "k_lens", c["Lk"])[b]
            assert (got[b, g, nk:] == fill[b, g, nk:]).all()
            add, err, rows = torch.zeros(nk, device="cuda", dtype=torch.float64), 0.0, 0
            for h in range(g * G, (g + 1) * G):
                s, es, ok, nq, _ = head_scores(c, b, h)
                l = lse[b, h, :nq, None].double()
                p = torch.where(ok & (l > -math.inf), torch.exp(s - torch.where(l == -math.inf, 0.0, l)), 0.0)
                add += p.sum(0)
                err = err + (p * (es + 2.0**-21 + 2.0**-22 * torch.where(l == -math.inf, 0.0, l).abs())).sum(0)
                rows += nq
            old = mass_in[b, g, :nk].double() if mass_in is not None else 0.0
            tol = err + add * rows * 2.0**-24 + 2.0**-23 * (old + add) + 2.0**-40
            d = (got[b, g, :nk].double() - old - add).abs()
            assert (d <= tol).all(), (b, g, float((d / tol).max()))


@pytest.mark.parametrize("name", ATTN)
def test_mass(P, name):
    c = make(**ATTN[name])
    _, lse = run_attention(P, c)
    mass_in = torch.rand(c["B"], c["Hkv"], c["Lk"], device="cuda")
    out = torch.full_like(mass_in, 3.0)
    run_mass(P, c, lse, mass_in, out)
    check_mass(c, lse, mass_in, out, torch.full_like(out, 3.0))
    zero = torch.full_like(mass_in, 3.0)
    run_mass(P, c, lse, None, zero)
    check_mass(c, lse, None, zero, torch.full_like(out, 3.0))
    acc = mass_in.clone()  # in place
    run_mass(P, c, lse, acc, acc)
    for b, n in enumerate(lens(c, "k_lens", c["Lk"])):
        assert torch.equal(acc[b, :, :n], out[b, :, :n])
        assert torch.equal(acc[b, :, n:], mass_in[b, :, n:])


def test_mass_adds_up_to_the_rows(P):
    """Every row that sees something gives a total weight of one."""
    c = make(B=2, Lq=150, Lk=900, Hq=6, Hkv=2, dh=64, causal=True, k_lens=[900, 100], cap=10.0)
    _, lse = run_attention(P, c)
    out = torch.zeros(2, 2, 900, device="cuda")
    run_mass(P, c, lse, None, out)
    rows = (lse > -math.inf).view(2, 2, 3 * 150).sum(2)
    for b, n in enumerate((900, 100)):
        assert (out[b, :, :n].double().sum(1) - rows[b]).abs().max() <= 1e-4 * 450


# ----------------------------------------------------------------- evict

def evict_reference(c, b, h):
    n = c["n"][b]
    m = min(n, c["budget"])
    w = c["mass"][b, h, :n].cpu().numpy().astype(np.float64)
    slot = np.arange(n)
    held = (slot < c["sinks"]) | (slot >= n - c["recent"])
    nan = np.isnan(w)
    order = np.lexsort((slot, -np.where(nan, 0.0, w), ~nan, ~held))
    return np.sort(order[:m])


EVICT = {
    "one": dict(B=1, L=1, H=1, dh=64, budget=1),
    "half": dict(B=2, L=100, H=3, dh=64, budget=50, sinks=4, recent=10),
    "all": dict(B=2, L=100, H=2, dh=128, budget=100, sinks=1, recent=1),
    "held-only": dict(B=1, L=300, H=2, dh=64, budget=30, sinks=10, recent=20),
    "lens": dict(B=5, L=700, H=2, dh=128, budget=333, sinks=3, recent=50, lens=[0, 1, 333, 334, 9999]),
    "long": dict(B=1, L=60001, H=1, dh=32, budget=40000, sinks=1, recent=1000),
    "window": dict(B=1, L=7800, H=4, dh=128, budget=4680, sinks=30, recent=1560),
    "odd-width": dict(B=1, L=90, H=2, dh=7, budget=31, sinks=0, recent=3),
    "ties": dict(B=2, L=3000, H=2, dh=64, budget=1000, values="ties"),
    "zeros": dict(B=1, L=500, H=1, dh=64, budget=100, values="zeros"),
    "strange": dict(B=1, L=400, H=2, dh=64, budget=150, values="strange"),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", EVICT)
def test_evict(P, name, dtype):
    c = dict(sinks=0, recent=0, lens=None, values="spread", **{k: v for k, v in EVICT[name].items() if k not in ("sinks", "recent", "lens", "values")})
    c.update({k: v for k, v in EVICT[name].items()})
    B, L, H, dh, n = (c[k] for k in ("B", "L", "H", "dh", "budget"))
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    k, v = (torch.randn(B, L, H, dh, device="cuda", generator=g).to(DT[dtype]) for _ in range(2))
    mass = torch.exp(2 * torch.randn(B, H, L, device="cuda", generator=g))
    if c["values"] == "ties":
        mass = (mass * 3).floor() / 3
    elif c["values"] == "zeros":
        mass = torch.zeros_like(mass)
        mass[..., ::3] = -0.0
    elif c["values"] == "strange":
        for i, x in enumerate((float("nan"), float("inf"), -float("inf"), -1.0, -0.0, 1e-42, -float("nan"))):
            mass[..., i::29] = x
    c["mass"], c["n"] = mass, [min(max(x, 0), L) for x in (c["lens"] or [L] * B)]
    kl = ints(c["lens"])
    pos = torch.randint(0, 1 << 20, (B, H, L), device="cuda", generator=g, dtype=torch.int32)
    doc = torch.randint(0, 9, (B, H, L), device="cuda", generator=g, dtype=torch.int32)
    k_out, v_out = (torch.full((B, n, H, dh), 8.0, device="cuda", dtype=DT[dtype]) for _ in range(2))
    mass_out = torch.full((B, H, n), 8.0, device="cuda")
    idx, pos_out, doc_out = (torch.full((B, H, n), -8, device="cuda", dtype=torch.int32) for _ in range(3))
    lens_out = torch.full((B,), -8, device="cuda", dtype=torch.int32)
    prob = P.evict_problem(code(P, dtype), k.shape, n, c["sinks"], c["recent"], k_lens=at(kl), k_pos=at(pos),
                           k_doc=at(doc), pos_out=at(pos_out), doc_out=at(doc_out), lens_out=at(lens_out))
    P.psv_cache_evict(prob, at(k), at(v), at(mass), at(k_out), at(v_out), at(mass_out), at(idx), stream())
    for b in range(B):
        m = min(c["n"][b], n)
        assert int(lens_out[b]) == m
        for h in range(H):
            want = evict_reference(c, b, h)
            np.testing.assert_array_equal(idx[b, h, :m].cpu().numpy(), want)
            w = torch.as_tensor(want, device="cuda")
            assert torch.equal(k_out[b, :m, h], k[b, w, h]) and torch.equal(v_out[b, :m, h], v[b, w, h])
            assert torch.equal(mass_out[b, h, :m].view(torch.int32), mass[b, h, w].view(torch.int32))
            assert torch.equal(pos_out[b, h, :m], pos[b, h, w]) and torch.equal(doc_out[b, h, :m], doc[b, h, w])
            for t, fill in ((k_out[b, m:, h], 8.0), (v_out[b, m:, h], 8.0), (mass_out[b, h, m:], 8.0), (idx[b, h, m:], -8),
                            (pos_out[b, h, m:], -8), (doc_out[b, h, m:], -8)):
                assert (t == fill).all()


def test_evict_strides_and_shared_positions(P):
    """K and V as halves of one buffer, heads before rows outside; slots as positions."""
    B, L, H, dh, n = 2, 130, 3, 64, 40
    kv = torch.randn(B, H, L, 2, dh, device="cuda").to(torch.bfloat16)
    k, v = kv[..., 0, :], kv[..., 1, :]
    st = (k.stride(0), k.stride(2), k.stride(1))
    mass = torch.rand(B, H, L, device="cuda")
    k_out, v_out = (torch.zeros(B, H, n, dh, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    mass_out = torch.zeros(B, H, n, device="cuda")
    idx, pos_out = (torch.zeros(B, H, n, device="cuda", dtype=torch.int32) for _ in range(2))
    so = (H * n * dh, dh, n * dh)
    prob = P.evict_problem(P.PSV_DTYPE_BF16, (B, L, H, dh), n, 1, 5, k_stride=st, v_stride=st, k_out_stride=so,
                           v_out_stride=so, pos_out=at(pos_out))
    P.psv_cache_evict(prob, at(k), at(v), at(mass), at(k_out), at(v_out), at(mass_out), at(idx), stream())
    c = dict(n=[L] * B, budget=n, sinks=1, recent=5, mass=mass)
    for b in range(B):
        for h in range(H):
            w = torch.as_tensor(evict_reference(c, b, h), device="cuda")
            assert torch.equal(idx[b, h].long(), w) and torch.equal(pos_out, idx)
            assert torch.equal(k_out[b, h], k[b, h, w]) and torch.equal(v_out[b, h], v[b, h, w])


# ------------------------------------------------------- used together

def step(P, st, q, k_new, v_new, pos, n, scratch):
    """One chunk: rotate, append, attend, add up the weights (all on the current stream)."""
    B, T, H, dh = k_new.shape
    kc, vc = st["k"], st["v"]
    dims = (24, 20, 20)
    qr = torch.empty_like(q)
    P.psv_rope(P.rope_problem(P.PSV_DTYPE_BF16, q.shape, dims), at(q), at(pos), at(qr), stream())
    slot = kc[:, n:n + T]
    P.psv_rope(P.rope_problem(P.PSV_DTYPE_BF16, k_new.shape, dims, out_stride=slot.stride()[:3]), at(k_new), at(pos),
               at(slot), stream())
    vc[:, n:n + T] = v_new
    prob = P.cache_problem(P.PSV_DTYPE_BF16, q.shape, kc.shape, k_lens=at(st["lens"]))
    o = torch.empty_like(q)
    lse = torch.empty(B, q.shape[2], T, device="cuda")
    P.psv_cache_attention(prob, at(qr), at(kc), at(vc), at(o), at(lse), at(scratch), scratch.numel(), stream())
    P.psv_cache_mass(prob, at(qr), at(kc), at(lse), at(st["mass"]), at(st["mass"]), at(scratch), scratch.numel(), stream())
    return qr, o, lse


def test_rolling_cache_with_eviction(P):
    """Five chunks through rope, append, attention, weights, and eviction to three chunks' worth, twice."""
    B, T, H, Hkv, dh, cap, budget = 2, 60, 4, 2, 64, 240, 120
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    kc, vc = (torch.zeros(B, cap, Hkv, dh, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    st = dict(k=kc, v=vc, mass=torch.zeros(B, Hkv, cap, device="cuda"), lens=ints([0] * B))
    scratch, _ = scratch_for(P, P.cache_problem(P.PSV_DTYPE_BF16, (B, T, H, dh), kc.shape))
    n = 0
    for chunk in range(5):
        q = torch.randn(B, T, H, dh, device="cuda", generator=g).to(torch.bfloat16)
        kn, vn = (torch.randn(B, T, Hkv, dh, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
        i = torch.arange(T, device="cuda", dtype=torch.int32)
        pos = torch.stack([torch.full_like(i, chunk), i // 10, i % 10], 1)[None].repeat(B, 1, 1).contiguous()
        st["lens"].fill_(n + T)
        before = st["mass"].clone()
        qr, o, lse = step(P, st, q, kn, vn, pos, n, scratch)
        n += T
        ref, size = rope_reference(kn.double(), pos, (24, 20, 20))
        assert ((st["k"][:, n - T:n].double() - ref).abs() <= U["bf16"] * ref.abs() + size * 2.0**-21).all()
        c = dict(make(B=1), B=B, Lq=T, Lk=cap, Hq=H, Hkv=Hkv, dh=dh, q=qr, k=st["k"], v=st["v"], k_lens=st["lens"])
        check_attention(c, o, lse)
        check_mass(c, lse, before, st["mass"], before)
        if n > budget + T - 1:
            ko, vo = torch.zeros_like(kc), torch.zeros_like(vc)
            mo = torch.zeros(B, Hkv, budget, device="cuda")
            idx = torch.zeros(B, Hkv, budget, device="cuda", dtype=torch.int32)
            prob = P.evict_problem(P.PSV_DTYPE_BF16, kc.shape, budget, 4, 30, k_out_stride=ko.stride()[:3],
                                   v_out_stride=vo.stride()[:3], k_lens=at(st["lens"]))
            P.psv_cache_evict(prob, at(st["k"]), at(st["v"]), at(st["mass"]), at(ko), at(vo), at(mo), at(idx), stream())
            e = dict(n=[n] * B, budget=budget, sinks=4, recent=30, mass=st["mass"])
            for b in range(B):
                for h in range(Hkv):
                    w = torch.as_tensor(evict_reference(e, b, h), device="cuda")
                    assert torch.equal(idx[b, h].long(), w)
                    assert torch.equal(ko[b, :budget, h], st["k"][b, w, h])
            st["k"], st["v"] = ko, vo
            st["mass"] = torch.zeros_like(st["mass"])
            st["mass"][:, :, :budget] = mo
            n = budget
    no_error(scratch)


def test_captured_calls_see_new_lengths(P):
    """Two graphs that share a workspace, replayed with other inputs, lengths and masses, give the eager bits."""
    c = make(B=2, Lq=4, Lk=900, Hq=4, Hkv=2, dh=128, k_lens=[900, 300], causal=True)
    prob = problem(P, c)
    scratch, n = scratch_for(P, prob)
    o, lse = torch.zeros_like(c["q"]), torch.zeros(2, 4, 4, device="cuda")
    mass = torch.zeros(2, 2, 900, device="cuda")

    def attend():
        P.psv_cache_attention(prob, at(c["q"]), at(c["k"]), at(c["v"]), at(o), at(lse), at(scratch), n, stream())

    def weigh():
        P.psv_cache_mass(prob, at(c["q"]), at(c["k"]), at(lse), 0, at(mass), at(scratch), n, stream())

    attend()
    weigh()
    torch.cuda.synchronize()
    graphs = []
    for f in (attend, weigh):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for kl in ([900, 300], [17, 900], [0, 257]):
        c["k_lens"].copy_(torch.tensor(kl))
        c["q"].normal_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone(), mass.clone()
        attend()
        weigh()
        torch.cuda.synchronize()
        for x, y in zip(got, (o, lse, mass)):
            assert torch.equal(x, y)
    no_error(scratch)


def test_calls_on_two_streams(P):
    """Two calls at once, each with its own stream and workspace."""
    cs = [make(B=2, Lq=64, Lk=2000, Hq=4, Hkv=4, dh=128, seed=s) for s in (1, 2)]
    want = [run_attention(P, c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = []
    torch.cuda.synchronize()
    for c, s in zip(cs, streams):
        prob = problem(P, c)
        scratch, n = scratch_for(P, prob)
        o, lse = torch.zeros_like(c["q"]), torch.zeros(2, 4, 64, device="cuda")
        torch.cuda.synchronize()
        outs.append((prob, scratch, n, o, lse))
    for _ in range(5):
        for c, s, (prob, scratch, n, o, lse) in zip(cs, streams, outs):
            P.psv_cache_attention(prob, at(c["q"]), at(c["k"]), at(c["v"]), at(o), at(lse), at(scratch), n, s.cuda_stream)
    torch.cuda.synchronize()
    for (prob, scratch, n, o, lse), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)
        no_error(scratch)


def test_host_memory_is_refused(P):
    c = make(Lq=4, Lk=8, dh=64)
    prob = problem(P, c)
    scratch, n = scratch_for(P, prob)
    host = torch.zeros(4 * 64, dtype=torch.bfloat16)
    with pytest.raises(P.PSVError) as e:
        P.psv_cache_attention(prob, host.data_ptr(), at(c["k"]), at(c["v"]), at(c["q"]), 0, at(scratch), n, stream())
    assert e.value.code == P.PSV_EINVAL and "device memory" in str(e.value)
    with pytest.raises(P.PSVError) as e:
        P.psv_cache_attention(prob, at(c["q"]), at(c["k"]), at(c["v"]), at(c["q"]), 0, at(scratch), n - 1, stream())
    assert e.value.code == P.PSV_EINVAL and "scratch" in str(e.value)

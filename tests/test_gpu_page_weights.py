"""Weights and query values far below the largest one in the attention over pages, against
64 bits.

A few keys have nearly all the weight and nothing in the columns that count, so that the output
is made of many small weights.  Tolerances, with the largest weight's reference at least 2^7
(the kernel's f16 weights reach 2^15 at most) and half of f16's fixed step 2^-25:
  a weight   2^-11 relative, and 2^-32 of the largest: of the row's largest p for f16 pages,
             of its largest p times a value's scale for 8-bit ones, whose codes it multiplies;
             for bf16 pages 2^-8 relative
  a score    dh products in f32, at worst one ulp a step: es = dh 2^-23 scale sum|q||k|, and
             2^-21 of the score for its further roundings; weights are off by 2^-20 more
  o          sums of these over the keys, and half a step of the output
  lse        es + 2^-20 + 2^-22 |lse|
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from test_gpu_page_ops import DT, STEP, U, Cache, quantised, run_attention  # noqa: E402

WIDE = 100000  # positions more than there are: shared groups are cut


@pytest.fixture(scope="module")
def P():
    from autoregressive_denoising_dit_gb300 import _psv

    return _psv


def large_keys(P, c, dtype, f, gap, width):
    """The cache, q, and o, lse with their tolerances: every 97th key `gap` above the others, whose
    scores spread over half a bit (so that whoever shares a long cache meets one); its value is
    1.25 in column 0 and zero elsewhere."""
    B, Lq, n, Hq, Hkv, dh = (c[x] for x in ("B", "Lq", "Lk", "Hq", "Hkv", "dh"))
    page = c["page"]
    cache = Cache(P, f, B, Hkv, dh, page, -(-n // page), width=(n + WIDE) // page if width else 0)
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.zeros(B, n, Hkv, dh, device="cuda")
    k[..., 0] = torch.rand(B, n, Hkv, device="cuda", generator=g) * 0.35 / gap
    k[:, ::97, :, 0] = 1.0 + 0.175 / gap
    v = 1.0 + 0.25 * torch.rand(B, n, Hkv, dh, device="cuda", generator=g)
    v[:, ::97] = 0
    v[:, ::97, :, 0] = 1.25
    k, v = k.to(DT[dtype]).double(), v.to(DT[dtype]).double()
    codes, vs = quantised(v, f)
    kk, vv = cache.fill(k, v, [n] * B)
    q = torch.zeros(B, Lq, Hq, dh, device="cuda", dtype=DT[dtype])
    q[..., 0] = gap
    G = Hq // Hkv
    # every query row of a kv head sees the same: [B, n, Hkv]
    s = q[0, 0, 0, 0].double() * kk[..., 0]
    es = (dh * 2.0**-23 + 2.0**-21) * s.abs().amax(1)
    top = s.amax(1, keepdim=True)
    p = torch.exp(s - top)
    l = p.sum(1)
    o = torch.einsum("bjh,bjhd->bhd", p, vv) / l[..., None]
    A = torch.einsum("bjh,bjhd->bhd", p, vv.abs()) / l[..., None]
    uw = U["bf16"] if f == "bf16" else U["f16"]
    least = (p * vs).amax(1)[..., None] * codes.abs().sum(1) * 2.0**-32 / l[..., None] if f != "bf16" else 0.0
    tol = (uw + 2 * es[..., None] + 2.0**-19) * A + least + U[dtype] * o.abs() + STEP[dtype]
    lse = torch.log(l) + top[:, 0]
    ltol = es + 2.0**-20 + 2.0**-22 * lse.abs()
    rows = [x.repeat_interleave(G, 1) for x in (o, tol, lse, ltol)]
    return cache, q, rows


CASES = [
    dict(B=1, Lq=1, Lk=131072, Hq=5, Hkv=1, dh=128, page=64),             # cut and joined
    dict(B=2, Lq=3, Lk=20000, Hq=4, Hkv=1, dh=128, page=64),              # 12 rows
    dict(B=2, Lq=8, Lk=20000, Hq=32, Hkv=8, dh=128, page=64),             # 32 rows: 16-bit pages once for all
    dict(B=1, Lq=1, Lk=1500, Hq=2, Hkv=2, dh=128, page=64),               # clusters
    dict(B=1, Lq=3, Lk=9000, Hq=4, Hkv=1, dh=64, page=24),
    dict(B=1, Lq=2, Lk=3000, Hq=2, Hkv=1, dh=80, page=7),
    dict(B=1, Lq=2, Lk=3000, Hq=2, Hkv=1, dh=200, page=16),
    dict(B=300, Lq=1, Lk=50, Hq=8, Hkv=4, dh=128, page=16),               # a warp a group
    dict(B=300, Lq=3, Lk=40, Hq=16, Hkv=4, dh=64, page=8),
    dict(B=1, Lq=1, Lk=2000, Hq=2, Hkv=1, dh=100, page=64),               # general kernel
]


@pytest.mark.parametrize("gap", [12.0, 16.0, 17.5])
@pytest.mark.parametrize("dtype,f", [("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "i8"), ("bf16", "bf16")])
@pytest.mark.parametrize("width", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"B{c['B']}q{c['Lq']}k{c['Lk']}H{c['Hq']}-{c['Hkv']}dh{c['dh']}")
def test_small_weights_beside_large_ones(P, case, dtype, f, gap, width):
    cache, q, (o, tol, lse, ltol) = large_keys(P, case, dtype, f, gap, width)
    got, got_lse = run_attention(P, dict(case, scale=1.0), cache, q, [case["Lk"]] * case["B"], [case["Lq"]] * case["B"], dtype)
    err = (got.double() - o[:, None]).abs() / tol[:, None]
    assert (err <= 1).all(), float(err.max())
    assert ((got_lse.double() - lse[..., None]).abs() <= ltol[..., None]).all()


@pytest.mark.parametrize("below", [20, 24, 30])
@pytest.mark.parametrize("f", ["e4m3", "i8", "bf16"])
@pytest.mark.parametrize("Lq,dh", [(1, 128), (5, 128), (12, 64), (2, 256)])
def test_small_values_of_a_query_row(P, f, Lq, dh, below):
    """A query's largest value meets zeros; one 2^-20 to 2^-30 of it makes the score, and keeps
    its eight bits (1 + 2^-7)."""
    n = 70
    cache = Cache(P, f, 1, 1, dh, 16, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    k = torch.zeros(1, n, 1, dh, device="cuda", dtype=torch.float64)
    k[0, :, 0, 1] = torch.randint(-8, 9, (n,), device="cuda", generator=g).double()
    k[0, :, 0, 9] = 16.0  # (met by zeros)
    v = torch.randn(1, n, 1, dh, device="cuda", generator=g).bfloat16().double()
    kk, vv = cache.fill(k, v, [n])
    q = torch.zeros(1, Lq, 1, dh, device="cuda", dtype=torch.bfloat16)
    q[..., 0], q[..., 1] = 2.0**below, 1.0 + 2.0**-7
    c = dict(scale=1.0)
    got, got_lse = run_attention(P, c, cache, q, [n], [Lq], "bf16")
    s = (1.0 + 2.0**-7) * kk[0, :, 0, 1]
    es = (dh * 2.0**-23 + 2.0**-21) * s.abs().max()
    lse = torch.logsumexp(s, 0)
    assert ((got_lse[0, 0].double() - lse).abs() <= es + 2.0**-20 + 2.0**-22 * lse.abs()).all()
    p = torch.softmax(s, 0)
    o, A = p @ vv[0, :, 0], p @ vv[0, :, 0].abs()
    # (f16 weights: 2^-32 of the largest for each code, at most 448 scales)
    _, vs = quantised(v, f)
    tol = ((U["bf16"] if f == "bf16" else U["f16"]) + 2 * es + 2.0**-19) * A + U["bf16"] * o.abs()
    tol = tol + (0.0 if f == "bf16" else n * 448 * 2.0**-32 * (p * vs[0, :, 0]).max())
    assert ((got[0, :, 0].double() - o).abs() <= tol).all()


@pytest.mark.parametrize("width", [False, True])
@pytest.mark.parametrize("Lq,dh", [(1, 128), (6, 64), (2, 256)])
def test_large_values_in_bf16_pages(P, Lq, dh, width):
    """Values of 2^118 to 2^119: their sums with weights of at most 2^2 of the first ones stay
    within f32 (70 x 2^119 x 2^2)."""
    n = 70
    cache = Cache(P, "bf16", 1, 2, dh, 16, 5, width=WIDE // 16 if width else 0)
    g = torch.Generator(device="cuda").manual_seed(11)
    k = torch.randn(1, n, 2, dh, device="cuda", generator=g).bfloat16().double() * 0.1
    v = ((1.0 + torch.rand(1, n, 2, dh, device="cuda", generator=g)) * 2.0**118).bfloat16().double()
    kk, vv = cache.fill(k, v, [n])
    q = torch.randn(1, Lq, 2, dh, device="cuda", generator=g).bfloat16()
    got, got_lse = run_attention(P, {}, cache, q, [n], [Lq], "bf16")
    s = torch.einsum("qhd,jhd->qhj", q[0].double(), kk[0]) * dh**-0.5
    assert (s.amax(-1) - s.amin(-1)).max() < 2.0 * 0.69  # weights within 2^2 of one another
    es = (dh * 2.0**-23 * torch.einsum("qhd,jhd->qhj", q[0].double().abs(), kk[0].abs()) * dh**-0.5).amax(-1) + 2.0**-20
    p = torch.softmax(s, -1)
    o = torch.einsum("qhj,jhd->qhd", p, vv[0])
    tol = (2 * U["bf16"] + 2 * es[..., None] + 2.0**-19) * o
    assert ((got[0].double() - o).abs() <= tol).all()
    assert ((got_lse[0].T.double() - torch.logsumexp(s, -1)).abs() <= es + 2.0**-20 + 2.0**-20).all()

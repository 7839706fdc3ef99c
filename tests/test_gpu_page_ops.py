"""The operators of a paged key/value cache on the GPU against plain 64-bit implementations.

Tolerances are derived, element by element, from the roundings that the operators make.
With u half a step of a type relative to the value (bf16 2^-8, f16 2^-11, f32 2^-24):
  scale    one division in f32: u32 of the scale
  code     M / size and x times it, each rounded in f32: 2 u32 of x M / size (and u32 for
           the size of the quotient that it is compared with), then the nearest code
  read     code times scale in f32, then the output type: u32 + u of the value
  scores   dh products accumulated in f32, at worst one ulp (2^-23) lost a step:
           es = dh 2^-23 scale sum|q||k|, four more roundings of the score, and the cap's
           tanh to 2^-21 of the cap (2^-21 of the capped score)
  weights  exp(s) is off by a factor 1 + es + 2^-20 (a value's scale enters by its
           logarithm: 2^-22 of an exponent of up to 16), in the numerator and the sum
  o        weights rounded to the operand type (f16 for 8-bit pages) uw, the output uo:
           uw sum(p |v|) / l + uo |o| + 2 (es + 2^-20) sum(p |v|) / l; f16 weights below 2^-14
           of the largest have a fixed half step of 2^-25 of it: n 2^-25 max(p |v|) / l
  lse      es + 2^-20 + 2^-22 |lse|
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0**-8, "f16": 2.0**-11, "f32": 2.0**-24}
STEP = {"bf16": 0.0, "f16": 2.0**-25, "f32": 0.0}  # half of f16's fixed step below 2^-14
MOST = {"e4m3": 448.0, "i8": 127.0}
INF = float("inf")


@pytest.fixture(scope="module")
def P():
    from autoregressive_denoising_dit_gb300 import _psv

    return _psv


def code(P, dtype):
    return {"bf16": P.PSV_DTYPE_BF16, "f16": P.PSV_DTYPE_F16, "f32": P.PSV_DTYPE_F32}[dtype]


def form(P, f):
    return {"bf16": P.PSV_PAGE_BF16, "f16": P.PSV_PAGE_F16, "e4m3": P.PSV_PAGE_E4M3, "i8": P.PSV_PAGE_I8}[f]


def ints(a):
    return None if a is None else torch.as_tensor(np.array(a, order="C"), dtype=torch.int32, device="cuda")


def at(t):
    return 0 if t is None else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


def quantised(x, f):
    """Codes as 64-bit numbers and scales of rows x [..., dh] in 64 bits, by f32 arithmetic as the header has it."""
    if f in DT:
        return x.to(DT[f]).double(), torch.ones(x.shape[:-1], device=x.device, dtype=torch.float64)
    x = x.float()
    size = x.abs().amax(-1)
    most = torch.full_like(size, MOST[f])
    turn = most / size
    y = x * turn[..., None]
    y = torch.where((torch.isfinite(size) & (size >= 2.0**-100))[..., None], y, torch.zeros_like(y))
    c = torch.round(y).double() if f == "i8" else y.to(torch.float8_e4m3fn).double()
    scale = torch.where(size < 2.0**-100, torch.zeros_like(size), size / most)
    return c, torch.where(torch.isfinite(size), scale, torch.full_like(scale, float("nan"))).double()


def stored(c, f):
    """Codes (64-bit numbers) as they are stored."""
    if f in DT:
        return c.to(DT[f])
    return c.to(torch.int8).view(torch.uint8) if f == "i8" else c.float().to(torch.float8_e4m3fn).view(torch.uint8)


def numbers(pages, f):
    if f in DT:
        return pages.double()
    return pages.view(torch.int8).double() if f == "i8" else pages.view(torch.float8_e4m3fn).double()


class Cache:
    """A pool of pages in which everything is NaN (codes 0x7f, scales NaN) but what is written."""

    def __init__(self, P, f, B, Hkv, dh, page, max_pages, spare=3, seed=0, layout="phrd", missing=(), packed=False,
                 width=0):
        """width: entries of the table, those behind max_pages without a page."""
        self.P, self.f, self.B, self.Hkv, self.dh, self.page = P, f, B, Hkv, dh, page
        self.max_pages = max(max_pages, width)
        self.n_pages = B * max_pages + spare
        g = torch.Generator().manual_seed(seed)
        t = torch.randperm(self.n_pages, generator=g)[:B * max_pages].view(B, max_pages).int()
        t = torch.cat([t, torch.full((B, self.max_pages - max_pages), -7, dtype=torch.int32)], 1)
        for b, i in missing:
            t[b, i] = -1 if (b + i) % 2 else self.n_pages + 5
        self.table = t.cuda()
        n = {"p": self.n_pages, "h": Hkv, "r": page, "d": dh}

        def pool(extra=()):
            shape = [n[x] for x in layout]
            if extra:
                shape = shape[:1] + [2] + shape[1:]
            if f in DT:
                return torch.full(shape, float("nan"), device="cuda", dtype=DT[f])
            return torch.full(shape, 0x7F, device="cuda", dtype=torch.uint8)

        order = [layout.index(x) for x in "phrd"]
        if packed:  # keys and values of a page next to each other
            both = pool(extra=(2,))
            self.k, self.v = both[:, 0].permute(order), both[:, 1].permute(order)
        else:
            self.k, self.v = pool().permute(order), pool().permute(order)
        self.scaled = f in MOST
        self.ks, self.vs = (torch.full((self.n_pages, Hkv, page), float("nan"), device="cuda") if self.scaled else None
                            for _ in range(2))

    def desc(self):
        s = lambda t: (t.stride(0), t.stride(2), t.stride(1))  # noqa: E731
        return self.P.page_cache(form(self.P, self.f), self.table.shape, self.n_pages, self.page, self.Hkv, self.dh,
                                 at(self.table), at(self.k), at(self.v), at(self.ks), at(self.vs), k_stride=s(self.k),
                                 v_stride=s(self.v))

    def where(self, b, pos):
        """(page, row) of a position, or None."""
        if not 0 <= pos < self.max_pages * self.page:
            return None
        e = int(self.table_host()[b, pos // self.page])
        return (e, pos % self.page) if 0 <= e < self.n_pages else None

    def table_host(self):
        return self.table.cpu()

    def fill(self, k, v, lens):
        """Keys and values [B, L, Hkv, dh] in 64 bits at positions 0.. of each sequence; what they are kept as."""
        kept = []
        table = self.table.long()
        for name, x in (("k", k), ("v", v)):
            c, s = quantised(x, self.f)
            pages, scales = getattr(self, name), getattr(self, name + "s")
            for b in range(self.B):
                pos = torch.arange(lens[b], device="cuda")
                e = table[b][pos // self.page]
                ok = (e >= 0) & (e < self.n_pages)
                pages[e[ok], :, (pos % self.page)[ok]] = stored(c[b, :lens[b]][ok], self.f)
                if self.scaled:
                    scales[e[ok], :, (pos % self.page)[ok]] = s[b, :lens[b]][ok].float()
            kept.append(c * s[..., None])
        return kept

    def there(self, b, n):
        pos = torch.arange(n, device="cuda")
        i = (pos // self.page).clamp(max=self.max_pages - 1)
        e = self.table.long()[b][i]
        return (e >= 0) & (e < self.n_pages) & (pos < self.max_pages * self.page)


# ------------------------------------------------------------ write, read

ROWS = [
    dict(B=1, L=1, Hkv=1, dh=128, page=64, starts=[0]),
    dict(B=8, L=1, Hkv=12, dh=128, page=64, starts=[0, 1, 62, 63, 64, 65, 127, 128]),
    dict(B=3, L=37, Hkv=3, dh=64, page=16, starts=[5, 0, 15], lens=[37, 0, 20]),
    dict(B=2, L=70, Hkv=5, dh=80, page=24, starts=[1, 23], missing=[(0, 2), (1, 0)]),
    dict(B=2, L=33, Hkv=2, dh=20, page=7, starts=[3, 0], lens=[40, 12]),       # value by value; a length over L
    dict(B=1, L=130, Hkv=2, dh=256, page=128, starts=[100], layout="prhd"),
    dict(B=2, L=19, Hkv=3, dh=33, page=1, starts=[0, 7], packed=True),
    dict(B=2, L=40, Hkv=4, dh=8, page=30, starts=[-5, 100], packed=True),      # rows before and behind the table
    dict(B=1, L=3, Hkv=7, dh=1, page=3, starts=[1], layout="rphd"),
    dict(B=2, L=1560, Hkv=12, dh=128, page=1560, starts=[0, 780]),
]


def new_rows(c, dtype, strided):
    g = torch.Generator(device="cuda").manual_seed(5)
    B, L, H, dh = c["B"], c["L"], c["Hkv"], c["dh"]
    if strided:  # between other projections of the same product
        x = torch.randn(B, L, 3 * H, dh, device="cuda", generator=g).to(DT[dtype])
        return x[:, :, H:2 * H], x[:, :, 2 * H:]
    return tuple(torch.randn(B, L, H, dh, device="cuda", generator=g).to(DT[dtype]) for _ in range(2))


def rows_of(c, b):
    n = c["L"] if c.get("lens") is None else min(c["lens"][b], c["L"])
    return [(i, c["starts"][b] + i) for i in range(n)]


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("dtype,f", [("bf16", "e4m3"), ("f16", "e4m3"), ("f32", "e4m3"), ("bf16", "i8"), ("f16", "i8"),
                                     ("f32", "i8"), ("bf16", "bf16"), ("f32", "bf16"), ("f16", "f16"), ("f32", "f16")])
@pytest.mark.parametrize("case", ROWS, ids=lambda c: f"B{c['B']}L{c['L']}H{c['Hkv']}dh{c['dh']}p{c['page']}")
def test_write_and_read(P, case, dtype, f, strided):
    c = case
    max_pages = -(-(max(c["starts"]) + c["L"]) // c["page"]) - (1 if -5 in c["starts"] else 0)
    cache = Cache(P, f, c["B"], c["Hkv"], c["dh"], c["page"], max_pages, layout=c.get("layout", "phrd"),
                  missing=c.get("missing", ()), packed=c.get("packed", False))
    k, v = new_rows(c, dtype, strided)
    before = {n: getattr(cache, n).clone() for n in ("k", "v") + (("ks", "vs") if cache.scaled else ())}
    starts, lens = ints(c["starts"]), ints(c.get("lens"))
    rows = P.page_rows(code(P, dtype), k.shape, k_stride=k.stride()[:3], v_stride=v.stride()[:3], starts=at(starts),
                       lens=at(lens))
    P.psv_page_write(cache.desc(), rows, at(k), at(v), stream())
    outs = {n: torch.full_like(x, 7.0) for n, x in (("k", k), ("v", v))}
    back = P.page_rows(code(P, dtype), k.shape, k_stride=outs["k"].stride()[:3], v_stride=outs["v"].stride()[:3],
                       starts=at(starts), lens=at(lens))
    P.psv_page_read(cache.desc(), back, at(outs["k"]), at(outs["v"]), stream())
    for name, x in (("k", k), ("v", v)):
        where = [(b, i, *w) for b in range(c["B"]) for i, pos in rows_of(c, b) if (w := cache.where(b, pos))]
        lost = [(b, i) for b in range(c["B"]) for i, pos in rows_of(c, b) if cache.where(b, pos) is None]
        b, i, e, r = (torch.tensor(t, dtype=torch.long, device="cuda") for t in (zip(*where) if where else ([],) * 4))
        x64 = x[b, i].double()
        got = numbers(getattr(cache, name)[e, :, r], f)
        want, want_scale = quantised(x64, f)
        assert torch.equal(got, want)
        kept = got
        if cache.scaled:
            scale = getattr(cache, name + "s")[e, :, r].double()
            assert torch.equal(scale, want_scale)
            # and against the definition: the nearest code of x / scale
            assert ((scale - x64.abs().amax(-1) / MOST[f]).abs() <= U["f32"] * scale).all()
            y = x64 / scale[..., None]
            half = torch.full_like(y, 0.5) if f == "i8" else 0.5 * torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)
            assert ((got - y).abs() <= half + 4 * U["f32"] * y.abs()).all()
            kept = got * scale[..., None]
        tol = kept.abs() * (U["f32"] + U[dtype]) + STEP[dtype]
        assert ((outs[name][b, i].double() - kept).abs() <= tol).all()
        for bb, ii in lost:
            assert (outs[name][bb, ii] == 0).all()
        for bb in range(c["B"]):
            n = len(rows_of(c, bb))
            assert (outs[name][bb, n:] == 7.0).all()
        # everything else in the pool is as it was
        pages, old = getattr(cache, name).clone(), before[name]
        pages[e, :, r] = old[e, :, r]
        assert torch.equal(pages.view(torch.uint8) if cache.scaled else pages.isnan(), old if cache.scaled else old.isnan())
        if cache.scaled:
            scales = getattr(cache, name + "s").clone()
            scales[e, :, r] = float("nan")
            assert scales.isnan().all()


@pytest.mark.parametrize("dh", [128, 20])
@pytest.mark.parametrize("f", ["e4m3", "i8"])
def test_rows_of_zeros_tiny_and_unbounded_values(P, f, dh):
    cache = Cache(P, f, 1, 1, dh, 16, 1)
    x = torch.randn(1, 10, 1, dh, device="cuda")
    x[0, 0] = 0
    x[0, 1] = -0.0
    x[0, 2] *= 2.0**-120                       # below the smallest size that is kept
    x[0, 3] = 1e-45
    x[0, 4] *= 2.0**-95
    x[0, 5, 0, 3] = float("nan")
    x[0, 6, 0, dh - 1] = -INF
    x[0, 7, 0, :2] = torch.tensor([float("nan"), INF], device="cuda")
    x[0, 8] *= 2.0**120
    x[0, 9, 0, 1] = 3.4e38
    x[0, 9, 0, 2] = 1.0
    v = x.flip(1).contiguous()
    rows = P.page_rows(P.PSV_DTYPE_F32, x.shape)
    P.psv_page_write(cache.desc(), rows, at(x), at(v), stream())
    k2, v2 = torch.zeros_like(x), torch.zeros_like(x)
    P.psv_page_read(cache.desc(), rows, at(k2), at(v2), stream())
    assert torch.equal(k2.flip(1).nan_to_num(5.0), v2.nan_to_num(5.0))
    assert (k2[0, :4] == 0).all() and k2[0, 5:8].isnan().all()
    for i in (4, 8, 9):
        size = x[0, i].abs().max().double()
        # half a step, of e4m3 relative to the value with the smallest step 2^-9 of a scale
        half = size / 254 if f == "i8" else (x[0, i].abs().double() * 2.0**-4).clamp(min=size / 448 * 2.0**-10)
        assert ((k2[0, i].double() - x[0, i].double()).abs() <= half + size * 2.0**-22).all()


# --------------------------------------------------------------- attention

def reference(cache, c, q, k, v, lens, rows):
    """o, lse and their tolerances in 64 bits. k, v: kept values [B, L, Hkv, dh]."""
    B, Lq, Hq, dh = q.shape
    G, f = Hq // cache.Hkv, cache.f
    uw = U["bf16"] if f == "bf16" else U["f16"]
    scale = c.get("scale") or dh ** -0.5
    out = []
    for b in range(B):
        n, ql = lens[b], rows[b]
        if not ql:
            out.append(None)
            continue
        qq = q[b, :ql].double()
        m = min(n, cache.max_pages * cache.page, k.shape[1])  # (there are no pages behind the kept ones)
        kk, vv = (x[b, :m].repeat_interleave(G, 1) for x in (k, v))
        j = torch.arange(m, device="cuda")[None]
        p = (n - ql + torch.arange(ql, device="cuda"))[:, None]
        see = cache.there(b, m)[None].expand(ql, m).clone()
        if c.get("causal"):
            see &= j <= p
        if c.get("window"):
            see &= (j > p - c["window"]) | (j < c.get("sinks", 0))
        hide = ~see[:, None]
        kk, vv = torch.nan_to_num(kk, 0, 0, 0), torch.nan_to_num(vv, 0, 0, 0)
        s = torch.einsum("ihd,jhd->ihj", qq, kk) * scale
        es = torch.einsum("ihd,jhd->ihj", qq.abs(), kk.abs()) * scale * dh * 2.0**-23 + s.abs() * 2.0**-21
        if c.get("cap"):
            s = c["cap"] * torch.tanh(s / c["cap"])
            es = es + 2.0**-21 * c["cap"]
        es = es.masked_fill(hide, 0).amax(2) if m else torch.zeros(ql, Hq, device="cuda", dtype=torch.float64)
        s = s.masked_fill(hide, -INF)
        top = s.amax(2, keepdim=True) if m else torch.full((ql, Hq, 1), -INF, device="cuda", dtype=torch.float64)
        e = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        l = e.sum(2, keepdim=True)
        l1 = torch.where(l == 0, torch.ones_like(l), l)
        o = torch.einsum("ihj,jhd->ihd", e, vv) / l1
        A = torch.einsum("ihj,jhd->ihd", e, vv.abs()) / l1
        big = (e * vv.abs().amax(2).T[None]).amax(2, keepdim=True) / l1 if m else torch.zeros_like(l)
        dt = {torch.bfloat16: "bf16", torch.float16: "f16"}[q.dtype]
        # (the largest weight times scale bounds every code's weight: a code of a row is at most MOST scales)
        tol = (uw + 2 * es[..., None] + 2.0**-19) * A + U[dt] * o.abs() + STEP[dt] + m * 2.0**-25 * big * (uw < 2.0**-9)
        lse = torch.where(l > 0, torch.log(l) + top, torch.full_like(l, -INF))[..., 0]
        ltol = es + 2.0**-20 + 2.0**-22 * torch.where(torch.isinf(lse), torch.zeros_like(lse), lse.abs())
        out.append((o, tol, lse, ltol))
    return out


def check(got_o, got_lse, ref, rows, fill):
    for b, r in enumerate(ref):
        n = rows[b]
        assert (got_o[b, n:] == fill).all() and (got_lse[b, :, n:] == fill).all()
        if not n:
            continue
        o, tol, lse, ltol = r
        err = (got_o[b, :n].double() - o).abs()
        assert (err <= tol).all(), (b, float((err / tol).max()))
        empty = torch.isinf(lse)
        gl = got_lse[b, :, :n].T.double()
        assert torch.equal(torch.isinf(gl), empty) and (gl[empty] == -INF).all()
        assert (got_o[b, :n][empty] == 0).all()
        el = (gl - lse)[~empty].abs()
        assert (el <= ltol[~empty]).all()


ATTN = [
    dict(B=1, Lq=1, Lk=1, Hq=1, Hkv=1, dh=128, page=64),
    dict(B=1, Lq=1, Lk=1560, Hq=12, Hkv=12, dh=128, page=64),
    dict(B=3, Lq=1, Lk=1000, Hq=4, Hkv=4, dh=128, page=64, lens=[1000, 0, 333]),
    dict(B=2, Lq=1, Lk=700, Hq=10, Hkv=2, dh=128, page=16, lens=[700, 17]),
    dict(B=2, Lq=4, Lk=321, Hq=6, Hkv=2, dh=128, page=32, causal=True, lens=[321, 3], rows=[4, 4]),  # rows before 0
    dict(B=2, Lq=3, Lk=500, Hq=8, Hkv=1, dh=64, page=64, lens=[500, 200], rows=[3, 2], causal=True),
    dict(B=1, Lq=2, Lk=90, Hq=64, Hkv=1, dh=128, page=24, causal=True),          # 128 rows a kv head
    dict(B=2, Lq=1, Lk=777, Hq=3, Hkv=3, dh=80, page=24),
    dict(B=2, Lq=2, Lk=555, Hq=4, Hkv=2, dh=32, page=7, causal=True),
    dict(B=2, Lq=1, Lk=130, Hq=4, Hkv=2, dh=128, page=1),
    dict(B=2, Lq=3, Lk=230, Hq=4, Hkv=2, dh=40, page=30, causal=True),           # rows of 8-byte pieces
    dict(B=2, Lq=1, Lk=630, Hq=12, Hkv=2, dh=72, page=64),
    dict(B=1, Lq=3, Lk=410, Hq=8, Hkv=2, dh=120, page=16, causal=True, window=300, missing=[(0, 13)]),
    dict(B=1, Lq=1, Lk=130, Hq=2, Hkv=2, dh=8, page=64),
    dict(B=2, Lq=2, Lk=90, Hq=2, Hkv=2, dh=24, page=9, causal=True),
    dict(B=1, Lq=2, Lk=150, Hq=2, Hkv=1, dh=21, page=64, causal=True),           # general kernel
    dict(B=1, Lq=1, Lk=100, Hq=2, Hkv=1, dh=100, page=32, window=40, sinks=5, missing=[(0, 2)], cap=3.0),  # general kernel
    dict(B=1, Lq=1, Lk=200, Hq=2, Hkv=1, dh=256, page=64),
    dict(B=2, Lq=3, Lk=700, Hq=8, Hkv=2, dh=256, page=24, causal=True, lens=[700, 60], rows=[3, 2]),
    dict(B=2, Lq=1, Lk=530, Hq=4, Hkv=4, dh=200, page=16, window=300, sinks=20),
    dict(B=1, Lq=5, Lk=260, Hq=4, Hkv=1, dh=136, page=7, causal=True, missing=[(0, 3)]),
    dict(B=2, Lq=1, Lk=900, Hq=4, Hkv=2, dh=128, page=64, causal=True, window=200, sinks=20),
    dict(B=2, Lq=5, Lk=900, Hq=2, Hkv=2, dh=128, page=48, causal=True, window=33, sinks=3, lens=[900, 20]),
    dict(B=1, Lq=9, Lk=400, Hq=4, Hkv=2, dh=64, page=64, window=5, lens=[400]),  # not causal
    dict(B=2, Lq=1, Lk=640, Hq=4, Hkv=2, dh=128, page=64, window=100000, sinks=4),
    dict(B=2, Lq=2, Lk=640, Hq=4, Hkv=2, dh=128, page=64, causal=True, window=1, sinks=0),
    dict(B=2, Lq=1, Lk=640, Hq=4, Hkv=2, dh=128, page=64, missing=[(0, 0), (0, 5), (1, 9)]),
    dict(B=2, Lq=2, Lk=100, Hq=4, Hkv=2, dh=128, page=10, causal=True, missing=[(0, i) for i in range(10)] + [(1, 3)]),
    dict(B=2, Lq=3, Lk=300, Hq=6, Hkv=2, dh=128, page=64, causal=True, cap=5.0),
    dict(B=1, Lq=1, Lk=300, Hq=6, Hkv=2, dh=64, page=64, cap=200.0, scale=2.0),
    dict(B=2, Lq=4, Lk=128, Hq=2, Hkv=2, dh=128, page=64, causal=True, append=True, lens=[126, 60], rows=[4, 1]),  # over the table
    dict(B=70, Lq=1, Lk=200, Hq=2, Hkv=1, dh=64, page=16, lens=[(b * 37) % 201 for b in range(70)]),
    dict(B=2, Lq=20, Lk=600, Hq=3, Hkv=1, dh=128, page=64, causal=True, rows=[20, 7]),
    # many short sequences: a warp has a group by itself
    dict(B=300, Lq=1, Lk=50, Hq=8, Hkv=4, dh=128, page=16, lens=[(b * 7) % 51 for b in range(300)]),
    dict(B=200, Lq=3, Lk=40, Hq=24, Hkv=6, dh=128, page=8, causal=True, lens=[40 - b % 40 for b in range(200)], rows=[b % 4 for b in range(200)]),
    dict(B=260, Lq=2, Lk=70, Hq=10, Hkv=5, dh=64, page=24, causal=True, window=20, sinks=3, missing=[(b, b % 3) for b in range(0, 260, 7)]),
    dict(B=250, Lq=1, Lk=37, Hq=6, Hkv=6, dh=72, page=7, cap=4.0),
    dict(B=300, Lq=5, Lk=33, Hq=8, Hkv=4, dh=64, page=16, causal=True),
    dict(B=300, Lq=1, Lk=33, Hq=8, Hkv=4, dh=200, page=16, lens=[b % 34 for b in range(300)]),
    dict(B=1, Lq=1, Lk=20000, Hq=4, Hkv=1, dh=128, page=64),
    dict(B=1, Lq=4, Lk=9000, Hq=16, Hkv=4, dh=64, page=32, causal=True),
]


def attention_case(P, c, dtype, f, seed=1, layout="phrd", packed=False, spread=1.0, width=0):
    B, Lq, Lk, Hq, Hkv, dh = (c[n] for n in ("B", "Lq", "Lk", "Hq", "Hkv", "dh"))
    g = torch.Generator(device="cuda").manual_seed(seed)
    max_pages = -(-Lk // c["page"])
    cache = Cache(P, f, B, Hkv, dh, c["page"], max_pages, missing=c.get("missing", ()), layout=layout, packed=packed,
                  width=width)
    lens, rows = c.get("lens", [Lk] * B), c.get("rows", [Lq] * B)
    total = [n + r for n, r in zip(lens, rows)] if c.get("append") else lens
    used = [min(n, max_pages * c["page"]) for n in total]
    if width and c.get("lens") is None:
        total = lens = used
    k, v = (torch.randn(B, max(used) or 1, Hkv, dh, device="cuda", generator=g) for _ in range(2))
    # rows of very different size, so that their scales differ
    k, v = (x * torch.exp(spread * torch.randn(x.shape[:2] + (Hkv, 1), device="cuda", generator=g)) for x in (k, v))
    k = k / (1 + spread)
    kept = cache.fill(k.to(DT[dtype]).double(), v.to(DT[dtype]).double(), used)
    q = (torch.randn(B, Lq, Hq, dh, device="cuda", generator=g) * 1.5).to(DT[dtype])
    for b in range(B):
        q[b, rows[b]:] = float("nan")  # rows not in use
    return cache, q, kept, lens, total, rows


def run_attention(P, c, cache, q, lens, rows, dtype, o=None, scratch=None):
    B, Lq, Hq, dh = q.shape
    o = torch.full_like(q, 9.0) if o is None else o
    lse = torch.full((B, Hq, Lq), 9.0, device="cuda")
    kl, ql = ints(lens), ints(rows) if "rows" in c else None
    query = P.page_query(code(P, dtype), q.shape, q_stride=q.stride()[:3], o_stride=o.stride()[:3],
                         causal=c.get("causal", False), window=c.get("window", 0), sinks=c.get("sinks", 0),
                         scale=c.get("scale", 0.0), softcap=c.get("cap", 0.0), q_lens=at(ql), k_lens=at(kl),
                         append=c.get("append", False))
    n = P.psv_page_scratch_bytes(cache.desc(), query)
    scratch = torch.zeros(n, dtype=torch.uint8, device="cuda") if scratch is None else scratch
    P.psv_page_attention(cache.desc(), query, at(q), at(o), at(lse), at(scratch), scratch.numel(), stream())
    torch.cuda.synchronize()
    return o, lse


@pytest.mark.parametrize("dtype,f", [("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "i8"), ("f16", "i8"), ("bf16", "bf16"),
                                     ("f16", "f16")])
@pytest.mark.parametrize("wide", [False, True])  # tables that cover much more than there is: shared groups are cut
@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"B{c['B']}q{c['Lq']}k{c['Lk']}H{c['Hq']}-{c['Hkv']}dh{c['dh']}p{c['page']}")
def test_attention(P, case, dtype, f, wide):
    cache, q, (k, v), lens, total, rows = attention_case(P, case, dtype, f, width=100000 // case["page"] if wide else 0)
    ref = reference(cache, case, q, k, v, total, rows)
    o, lse = run_attention(P, case, cache, q, lens, rows, dtype)
    check(o, lse, ref, rows, 9.0)
    o2, lse2 = run_attention(P, case, cache, q, lens, rows, dtype)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # repeats bit for bit


# Over 16 rows a kv head: four tiles of eight at a time, some of them without rows.
MANY_ROWS = [
    dict(B=2, Lq=1, Lk=700, Hq=34, Hkv=2, dh=128, page=64, lens=[700, 90]),                       # 17 rows
    dict(B=2, Lq=3, Lk=700, Hq=16, Hkv=2, dh=128, page=64, causal=True, lens=[700, 2], rows=[3, 1]),
    dict(B=1, Lq=4, Lk=3000, Hq=64, Hkv=8, dh=128, page=24, causal=True),
    dict(B=2, Lq=33, Lk=500, Hq=1, Hkv=1, dh=128, page=7, causal=True, window=60, sinks=3, rows=[33, 17], missing=[(0, 2), (1, 40)]),
    dict(B=2, Lq=5, Lk=400, Hq=16, Hkv=2, dh=64, page=64, causal=True, cap=5.0),                  # 40 rows
    dict(B=3, Lq=6, Lk=260, Hq=8, Hkv=1, dh=64, page=16, causal=True, lens=[260, 5, 100], rows=[6, 6, 0]),
    dict(B=2, Lq=25, Lk=330, Hq=2, Hkv=1, dh=32, page=40, causal=True, window=300),
    dict(B=2, Lq=2, Lk=640, Hq=20, Hkv=2, dh=72, page=64, missing=[(0, 0), (1, 9)]),
    dict(B=2, Lq=1, Lk=90, Hq=31, Hkv=1, dh=104, page=9, scale=1.5),
    dict(B=70, Lq=4, Lk=200, Hq=20, Hkv=4, dh=128, page=16, causal=True, lens=[(b * 37) % 201 for b in range(70)], rows=[b % 5 for b in range(70)]),
    dict(B=310, Lq=3, Lk=50, Hq=14, Hkv=2, dh=128, page=8, causal=True, append=True, lens=[b % 48 for b in range(310)]),
    dict(B=1, Lq=3, Lk=20000, Hq=6, Hkv=1, dh=128, page=64, causal=True),
    dict(B=2, Lq=4, Lk=16000, Hq=64, Hkv=8, dh=128, page=64, causal=True, lens=[15000, 70], cap=20.0),
    dict(B=2, Lq=9, Lk=4100, Hq=64, Hkv=8, dh=128, page=64, causal=True, lens=[4100, 9], rows=[9, 5], window=4000, sinks=30),  # 72 rows
]


@pytest.mark.parametrize("dtype,f", [("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "i8"), ("f16", "i8"), ("bf16", "bf16"),
                                     ("f16", "f16")])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("case", MANY_ROWS, ids=lambda c: f"B{c['B']}q{c['Lq']}k{c['Lk']}H{c['Hq']}-{c['Hkv']}dh{c['dh']}p{c['page']}")
def test_attention_of_many_rows(P, case, dtype, f, wide):
    test_attention(P, case, dtype, f, wide)


NARROW = [  # rows of 5, 6, 9 and 10 pieces
    dict(B=2, L=23, Hkv=5, dh=40, page=16, starts=[3, 0], lens=[23, 9]),
    dict(B=3, L=1, Hkv=12, dh=48, page=64, starts=[0, 63, 64]),
    dict(B=2, L=61, Hkv=3, dh=72, page=7, starts=[-2, 11], missing=[(0, 1)]),
    dict(B=1, L=333, Hkv=9, dh=80, page=64, starts=[40], layout="prhd"),
]


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("dtype,f", [("bf16", "e4m3"), ("f16", "i8"), ("f32", "e4m3"), ("f32", "i8"), ("bf16", "bf16"),
                                     ("f32", "f16")])
@pytest.mark.parametrize("case", NARROW, ids=lambda c: f"B{c['B']}L{c['L']}H{c['Hkv']}dh{c['dh']}p{c['page']}")
def test_write_and_read_of_narrow_rows(P, case, dtype, f, strided):
    test_write_and_read(P, case, dtype, f, strided)

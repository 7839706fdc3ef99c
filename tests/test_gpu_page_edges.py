"""The operators of a paged cache where they could go wrong together: values that are not
finite behind masks, long pools, many sequences, tables that several sequences share,
captured and replayed steps, side streams, and a run beside the rolling cache's operators."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from test_gpu_page_ops import (DT, INF, Cache, at, attention_case, check, code, form, ints, reference, run_attention,  # noqa: E402
                               stream)


@pytest.fixture(scope="module")
def P():
    from autoregressive_denoising_dit_gb300 import _psv

    return _psv


WIDE = 4096  # table entries: groups are cut


@pytest.mark.parametrize("width", [0, WIDE])
@pytest.mark.parametrize("dtype,f", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "i8")])
def test_keys_and_values_that_are_not_finite_behind_masks(P, dtype, f, width):
    """A drafted token's key and value are NaN or infinite: rows before it, and rows whose
    window has left it, do not notice."""
    c = dict(B=1, Lq=6, Lk=200, Hq=4, Hkv=2, dh=128, page=32, causal=True, window=60, sinks=3)
    cache, q, (k, v), lens, total, rows = attention_case(P, c, dtype, f, width=width)
    bad = [(197, "v"), (195, "k"), (137, "v"), (0, "v")]  # rows 194..199; 137 leaves the window at row 197
    for j, name in bad:
        e, r = int(cache.table[0, j // 32]), j % 32
        if f in DT:
            getattr(cache, name)[e, 1, r, 5] = INF if j == 137 else float("nan")
        else:
            getattr(cache, name)[e, 1, r] = 0
            getattr(cache, name + "s")[e, 1, r] = float("nan")
    o, lse = run_attention(P, c, cache, q, lens, rows, dtype)
    # query heads of kv head 0 see none of it
    assert torch.isfinite(o[0, :, :2].float()).all() and torch.isfinite(lse[0, :2]).all()
    # kv head 1: position 0 is a sink that every row sees
    if f in DT:
        assert torch.isnan(o[0, :, 2:, 5].float()).all()
        ok = [d for d in range(128) if d != 5]
        assert torch.isfinite(o[0, 0, 2:][:, ok].float()).all()      # row 194 sees neither 195 nor 197
        assert torch.isfinite(lse[0, 2:, 0]).all()
    else:
        assert torch.isnan(o[0, :, 2:].float()).all()
        assert torch.isfinite(lse[0, 2:, 0]).all()
    assert torch.isnan(lse[0, 2:, 1:]).all()                          # NaN scores from row 195 on
    # kv head 0 by the definition
    want_o, tol, want_lse, ltol = reference(cache, c, q, k, v, total, rows)[0]
    assert ((lse[0, :2].T.double() - want_lse[:, :2]).abs() <= ltol[:, :2]).all()
    assert ((o[0, :, :2].double() - want_o[:, :2]).abs() <= tol[:, :2]).all()


@pytest.mark.parametrize("width", [0, WIDE])
@pytest.mark.parametrize("f", ["bf16", "f16"])
def test_an_infinite_value_reaches_the_rows_that_see_it_only(P, f, width):
    c = dict(B=1, Lq=12, Lk=90, Hq=2, Hkv=2, dh=64, page=16, causal=True)
    cache, q, (k, v), lens, total, rows = attention_case(P, c, f, f, width=width)
    e, r = int(cache.table[0, 84 // 16]), 84 % 16
    cache.v[e, 0, r, 7] = INF
    cache.v[e, 1, r, 9] = float("nan")
    v2 = v.clone()
    v2[0, 84, 0, 7] = v2[0, 84, 1, 9] = 0
    o, lse = run_attention(P, c, cache, q, lens, rows, f)
    want_o, tol, want_lse, ltol = reference(cache, c, q, k, v2, total, rows)[0]
    first = 84 - 78  # rows stand at 78..89
    assert (o[0, first:, 0, 7] == INF).all() and torch.isnan(o[0, first:, 1, 9].float()).all()
    hit = torch.zeros(o.shape[1:], dtype=torch.bool, device="cuda")
    hit[first:, 0, 7] = hit[first:, 1, 9] = True
    assert ((o[0].double() - want_o).abs() <= tol)[~hit].all()
    assert ((lse[0].T.double() - want_lse).abs() <= ltol).all()


@pytest.mark.parametrize("width", [0, WIDE])
@pytest.mark.parametrize("f", ["e4m3", "i8"])
def test_scales_of_any_size(P, f, width):
    """Rows of zeros, rows from 2^-60 to 2^60: weights fit their type all the same."""
    c = dict(B=2, Lq=2, Lk=333, Hq=6, Hkv=2, dh=128, page=64, causal=True, lens=[333, 100])
    cache, q, _, lens, total, rows = attention_case(P, c, "bf16", f, width=width)
    g = torch.Generator(device="cuda").manual_seed(9)
    k, v = (torch.randn(2, 333, 2, 128, device="cuda", generator=g) for _ in range(2))
    v = v * torch.exp2(torch.randint(-60, 61, (2, 333, 2, 1), device="cuda", generator=g).float())
    k = k * torch.exp2(torch.randint(-40, 1, (2, 333, 2, 1), device="cuda", generator=g).float())
    v[:, ::7], k[:, ::11] = 0, 0
    k, v = cache.fill(k.double(), v.double(), lens)
    o, lse = run_attention(P, c, cache, q, lens, rows, "bf16")
    check(o, lse, reference(cache, c, q, k, v, total, rows), rows, 9.0)
    z = torch.zeros(2, 333, 2, 128, device="cuda", dtype=torch.float64)
    k, v = cache.fill(k, z, lens)  # every value zero
    o, lse = run_attention(P, c, cache, q, lens, rows, "bf16")
    check(o, lse, reference(cache, c, q, k, v, total, rows), rows, 9.0)
    assert (o[0] == 0).all()


@pytest.mark.parametrize("f", ["e4m3", "bf16"])
def test_queries_of_any_size(P, f):
    c = dict(B=1, Lq=3, Lk=150, Hq=4, Hkv=2, dh=128, page=64, causal=True, scale=1.0)
    cache, q, (k, v), lens, total, rows = attention_case(P, c, "bf16", f)
    q[0, 0] *= 2.0**-70
    q[0, 1, 0] = 0
    q[0, 1, 1, 3:] *= 2.0**-20
    q[0, 2, 2] *= 2.0**-126
    o, lse = run_attention(P, c, cache, q, lens, rows, "bf16")
    check(o, lse, reference(cache, c, q, k, v, total, rows), rows, 9.0)
    q[0, 2, 0, 0] = float("nan")
    o, lse = run_attention(P, c, cache, q, lens, rows, "bf16")
    assert torch.isnan(o[0, 2, 0].float()).all() and torch.isnan(lse[0, 0, 2])
    assert torch.isfinite(o[0, :2].float()).all() and torch.isfinite(o[0, 2, 1:].float()).all()


@pytest.mark.parametrize("f", ["e4m3", "f16"])
@pytest.mark.parametrize("layout,packed", [("prhd", False), ("phrd", True), ("hprd", False), ("rphd", False)])
@pytest.mark.parametrize("width", [0, WIDE])
def test_orders_of_the_indexes(P, f, layout, packed, width):
    c = dict(B=2, Lq=2, Lk=300, Hq=6, Hkv=3, dh=128, page=24, causal=True, lens=[300, 111])
    cache, q, (k, v), lens, total, rows = attention_case(P, c, "f16", f, layout=layout, packed=packed, width=width)
    # queries and outputs inside wider products; then the output in the queries' place
    wide = torch.zeros(2, 2, 10, 128, device="cuda", dtype=torch.float16)
    wide[:, :, 2:8] = q
    ref = reference(cache, c, q, k, v, total, rows)
    o, lse = run_attention(P, c, cache, wide[:, :, 2:8], lens, rows, "f16", o=torch.full((2, 6, 2, 128), 9.0, device="cuda", dtype=torch.float16).transpose(1, 2))
    check(o, lse, ref, rows, 9.0)
    o, lse = run_attention(P, c, cache, wide[:, :, 2:8], lens, rows, "f16", o=wide[:, :, 2:8])
    check(o, lse, ref, rows, 9.0)
    assert (wide[:, :, :2] == 0).all() and (wide[:, :, 8:] == 0).all()


def test_bases_that_are_not_aligned(P):
    """Two bytes off: the general kernel, the same answers."""
    c = dict(B=1, Lq=2, Lk=70, Hq=4, Hkv=2, dh=64, page=16, causal=True)
    cache, q, (k, v), lens, total, rows = attention_case(P, c, "bf16", "e4m3")
    ref = reference(cache, c, q, k, v, total, rows)
    buf = torch.zeros(q.numel() + 1, device="cuda", dtype=torch.bfloat16)
    q1 = buf[1:].view(q.shape)
    q1.copy_(q)
    o1 = torch.full((q.numel() + 1,), 9.0, device="cuda", dtype=torch.bfloat16)[1:].view(q.shape)
    check(*run_attention(P, c, cache, q1, lens, rows, "bf16", o=o1), ref, rows, 9.0)
    n = cache.k.numel()
    pool = torch.zeros(n + 1, device="cuda", dtype=torch.uint8)[1:].view(cache.k.shape)
    pool.copy_(cache.k)
    cache.k = pool
    check(*run_attention(P, c, cache, q, lens, rows, "bf16"), ref, rows, 9.0)


@pytest.mark.parametrize("f", ["e4m3", "i8", "bf16"])
def test_pages_far_apart(P, f):
    """Pages in a pool of over 4 GB, whose offsets pass 32 bits."""
    B, Hkv, dh, page, n_pages = 2, 2, 128, 64, 300000 if f != "bf16" else 150000
    dt = DT.get(f, torch.uint8)
    pools = [torch.empty(n_pages, Hkv, page, dh, device="cuda", dtype=dt) for _ in range(2)]
    scales = [torch.empty(n_pages, Hkv, page, device="cuda") if f not in DT else None for _ in range(2)]
    table = ints([[n_pages - 1, 3, n_pages // 2 + 7], [n_pages - 2, 140000, n_pages - 5]])
    cache = P.page_cache(form(P, f), table.shape, n_pages, page, Hkv, dh, at(table), at(pools[0]), at(pools[1]), at(scales[0]),
                         at(scales[1]))
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(B, 180, Hkv, dh, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    rows = P.page_rows(P.PSV_DTYPE_BF16, k.shape)
    P.psv_page_write(cache, rows, at(k), at(v), stream())
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    P.psv_page_read(cache, rows, at(k2), at(v2), stream())
    for x, y in ((k, k2), (v, v2)):
        # half a step of the format, by the row's largest value, and the output's rounding
        half = {"e4m3": 2.0**-4, "i8": 1 / 254, "bf16": 0.0}[f] * x.double().abs().amax(-1, keepdim=True)
        assert ((x.double() - y.double()).abs() <= half * (1 + 2.0**-8) + 2.0**-8 * y.double().abs()).all()
    q = torch.randn(B, 1, 4, dh, device="cuda", generator=g).to(torch.bfloat16)
    near = Cache(P, f, B, Hkv, dh, page, 3)
    kn, vn = near.fill(k.double(), v.double(), [180, 180])
    ref = reference(near, {}, q, kn, vn, [180, 180], [1, 1])
    o, lse, kl = torch.full_like(q, 9.0), torch.full((B, 4, 1), 9.0, device="cuda"), ints([180, 180])
    query = P.page_query(P.PSV_DTYPE_BF16, q.shape, k_lens=at(kl))
    scratch = torch.empty(P.psv_page_scratch_bytes(cache, query), dtype=torch.uint8, device="cuda")
    P.psv_page_attention(cache, query, at(q), at(o), at(lse), at(scratch), scratch.numel(), stream())
    check(o, lse, ref, [1, 1], 9.0)


@pytest.mark.parametrize("width", [0, 600])
@pytest.mark.parametrize("B", [33, 1000, 4099])
def test_many_sequences_of_uneven_length(P, B, width):
    """More than a warp looks at in one go; most hold nothing, some hold much."""
    rng = np.random.default_rng(B)
    lens = [int(n) for n in np.where(rng.random(B) < 0.4, 0, rng.integers(0, 25, B))]
    lens[B // 2] = 3000
    lens[B - 1] = 1700
    Hkv, dh, page = 2, 64, 16
    need = [-(-n // page) for n in lens]
    width = max(max(need), width)
    n_pages = sum(need) + 1
    order = rng.permutation(n_pages)[:sum(need)]
    table = np.full((B, width), -1)
    for b, start in enumerate(np.cumsum([0] + need[:-1])):
        table[b, :need[b]] = order[start:start + need[b]]
    cache = Cache.__new__(Cache)
    cache.P, cache.f, cache.B, cache.Hkv, cache.dh, cache.page, cache.max_pages, cache.n_pages, cache.scaled = P, "i8", B, Hkv, dh, page, width, n_pages, True
    cache.table = ints(table)
    cache.k, cache.v = (torch.full((n_pages, Hkv, page, dh), 0x7F, device="cuda", dtype=torch.uint8) for _ in range(2))
    cache.ks, cache.vs = (torch.full((n_pages, Hkv, page), float("nan"), device="cuda") for _ in range(2))
    rows = [0 if b % 5 == 2 else 1 for b in range(B)]
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(B, 1, 4, dh, device="cuda", generator=g).half()
    k, v = (torch.randn(B, 3000, Hkv, dh, device="cuda", generator=g).half().double() for _ in range(2)) if B < 100 else (None, None)
    if k is None:  # keys and values by the place in the pool
        k, v = torch.randn(n_pages, Hkv, page, dh, device="cuda", generator=g), torch.randn(n_pages, Hkv, page, dh, device="cuda", generator=g)
        from test_gpu_page_ops import quantised, stored
        (ck, sk), (cv, sv) = quantised(k, "i8"), quantised(v, "i8")
        cache.k, cache.v, cache.ks, cache.vs = stored(ck, "i8"), stored(cv, "i8"), sk.float(), sv.float()
        kk, vv = ck * sk[..., None], cv * sv[..., None]
        some = [b for b in range(B) if b in (0, 1, B // 2, B - 1, B - 2) or b % 97 == 0]
    else:
        kk, vv = cache.fill(k, v, lens)
        some = list(range(B))
    c = dict(rows=rows)
    o, lse = run_attention(P, c, cache, q, lens, rows, "f16")
    for b in some:
        n = lens[b]
        one = Cache.__new__(Cache)
        one.f, one.Hkv, one.page, one.max_pages, one.n_pages, one.table = "i8", Hkv, page, width, n_pages, cache.table[b:b + 1]
        if B >= 100:
            pos = torch.arange(n, device="cuda")
            e = cache.table[b].long()[pos // page]
            kb, vb = kk[e, :, pos % page][None], vv[e, :, pos % page][None]
        else:
            kb, vb = kk[b:b + 1], vv[b:b + 1]
        check(o[b:b + 1], lse[b:b + 1], reference(one, {}, q[b:b + 1], kb, vb, [n], [rows[b]]), [rows[b]], 9.0)


def test_shared_pages_and_tables(P):
    """Sequences that share a prefix's pages, and one table for all (stride 0)."""
    c = dict(B=3, Lq=1, Lk=128, Hq=4, Hkv=2, dh=128, page=32, lens=[128, 100, 64])
    cache, q, _, lens, total, rows = attention_case(P, c, "bf16", "e4m3")
    cache.table[1:] = cache.table[0]
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(1, 128, 2, 128, device="cuda", generator=g).expand(3, -1, -1, -1) for _ in range(2))
    k, v = cache.fill(k.double(), v.double(), [128, 0, 0])
    ref = reference(cache, c, q, k, v, total, rows)
    check(*run_attention(P, c, cache, q, lens, rows, "bf16"), ref, rows, 9.0)
    d = cache.desc()
    d.table_stride = 0
    cache.desc = lambda: d
    check(*run_attention(P, c, cache, q, lens, rows, "bf16"), ref, rows, 9.0)


class Decoder:
    """A program's step: rotate, write, look back; all on the device, lengths too."""

    def __init__(self, P, f="e4m3", B=3, Hq=8, Hkv=2, dh=128, page=16, max_pages=12, scratch=None, seed=0):
        self.P, self.B, self.Hkv = P, B, Hkv
        self.cache = Cache(P, f, B, Hkv, dh, page, max_pages, seed=seed)
        self.desc = self.cache.desc()
        z = lambda H: torch.zeros(B, 1, H, dh, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        self.q, self.k, self.v, self.o = z(Hq), z(Hkv), z(Hkv), z(Hq)
        self.lse = torch.zeros(B, Hq, 1, device="cuda")
        self.before = torch.zeros(B, device="cuda", dtype=torch.int32)
        self.rope = [P.rope_problem(P.PSV_DTYPE_BF16, x.shape, (dh,), pos_stride=(1, 1)) for x in (self.q, self.k)]
        self.rows = P.page_rows(P.PSV_DTYPE_BF16, self.k.shape, starts=at(self.before))
        self.query = P.page_query(P.PSV_DTYPE_BF16, self.q.shape, causal=True, k_lens=at(self.before), append=True)
        n = P.psv_page_scratch_bytes(self.desc, self.query)
        self.scratch = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") if scratch is None else scratch

    def step(self):
        P, s = self.P, stream()
        P.psv_rope(self.rope[0], at(self.q), at(self.before), at(self.q), s)
        P.psv_rope(self.rope[1], at(self.k), at(self.before), at(self.k), s)
        P.psv_page_write(self.desc, self.rows, at(self.k), at(self.v), s)
        P.psv_page_attention(self.desc, self.query, at(self.q), at(self.o), at(self.lse), at(self.scratch), self.scratch.numel(), s)
        self.before += 1

    def feed(self, g):
        for x in (self.q, self.k, self.v):
            x.copy_(torch.randn(x.shape, device="cuda", generator=g))


@pytest.mark.parametrize("max_pages", [12, WIDE])
@pytest.mark.parametrize("f", ["e4m3", "i8", "bf16"])
def test_a_captured_step_follows_its_lengths(P, f, max_pages):
    eager, graphed = (Decoder(P, f=f, max_pages=min(max_pages, 300)) for _ in range(2))
    start = ints([0, 30, 150])
    g1, g2 = (torch.Generator(device="cuda").manual_seed(7) for _ in range(2))
    side = torch.cuda.Stream()
    for d in (eager, graphed):
        x = torch.randn(3, 160, 2, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
        P.psv_page_write(d.desc, P.page_rows(P.PSV_DTYPE_BF16, x.shape, lens=at(start)), at(x), at(x), stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        graphed.feed(g2)
        with torch.cuda.graph(graph, stream=side):
            graphed.step()
    g2.manual_seed(7)
    graphed.before.copy_(start)
    eager.before.copy_(start)
    torch.cuda.synchronize()
    for _ in range(25):  # lengths pass pages, and more keys than at the capture
        eager.feed(g1)
        eager.step()
        graphed.feed(g2)
        graph.replay()
        assert torch.equal(eager.o, graphed.o) and torch.equal(eager.lse, graphed.lse)
    assert graphed.before.tolist() == [25, 55, 175]
    for name in ("k", "v"):
        assert torch.equal(getattr(eager.cache, name).view(torch.uint8), getattr(graphed.cache, name).view(torch.uint8))


def test_two_graphs_share_a_workspace(P):
    big = Decoder(P, Hq=24, max_pages=300)     # cut groups
    small = Decoder(P, B=2, Hq=2, scratch=big.scratch)  # clusters
    alone = [Decoder(P, Hq=24, max_pages=300), Decoder(P, B=2, Hq=2)]
    gens = [torch.Generator(device="cuda").manual_seed(i) for i in (1, 2, 1, 2)]
    graphs = []
    for d in (big, small):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            d.step()
        d.before.zero_()
        graphs.append(g)
    for _ in range(20):
        for d, g, gen in zip((big, small), graphs, gens):
            d.feed(gen)
            g.replay()
        for d, gen in zip(alone, gens[2:]):
            d.feed(gen)
            d.step()
        assert torch.equal(big.o, alone[0].o) and torch.equal(small.o, alone[1].o)


def test_two_streams_at_once(P):
    """Calls on two streams with workspaces of their own."""
    a, b = (Decoder(P, Hq=24, max_pages=300, seed=i) for i in range(2))
    c, d = (Decoder(P, Hq=24, max_pages=300, seed=i) for i in range(2))
    lens = ints([2500, 4700, 60])
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(3, 4700, 2, 128, device="cuda", generator=g).bfloat16()
    for t in (a, b, c, d):
        P.psv_page_write(t.desc, P.page_rows(P.PSV_DTYPE_BF16, x.shape, lens=at(lens)), at(x), at(x), stream())
        t.before.copy_(lens)
        t.feed(torch.Generator(device="cuda").manual_seed(5))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(30):
        for t, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                t.step()
    torch.cuda.synchronize()
    for _ in range(30):
        c.step()
    for _ in range(30):
        d.step()
    for t, u in ((a, c), (b, d)):
        assert torch.equal(t.o, u.o) and torch.equal(t.lse, u.lse) and torch.equal(t.before, u.before)


@pytest.mark.parametrize("f", ["e4m3", "i8", "bf16"])
def test_a_chunk_reads_back_what_tokens_look_at(P, f):
    """A run of the operators beside the rolling cache's: a chunk is rotated, written, read back
    with what is before it and attended to by its many rows (psv_cache_attention); its last rows
    get the same from the pages (psv_page_attention), to the two calls' roundings."""
    B, T, past, Hq, Hkv, dh, page = 2, 300, 430, 6, 2, 128, 64
    cache = Cache(P, f, B, Hkv, dh, page, -(-(past + T) // page))
    g = torch.Generator(device="cuda").manual_seed(8)
    randn = lambda L, H: torch.randn(B, L, H, dh, device="cuda", generator=g).bfloat16()  # noqa: E731
    old_k, old_v, k, v, q = randn(past, Hkv), randn(past, Hkv), randn(T, Hkv), randn(T, Hkv), randn(T, Hq)
    P.psv_page_write(cache.desc(), P.page_rows(P.PSV_DTYPE_BF16, old_k.shape), at(old_k), at(old_v), stream())
    pos = (past + torch.arange(T, device="cuda", dtype=torch.int32)).view(1, T, 1).expand(B, T, 1).contiguous()
    for x in (q, k):
        P.psv_rope(P.rope_problem(P.PSV_DTYPE_BF16, x.shape, (dh,)), at(x), at(pos), at(x), stream())
    starts = ints([past] * B)
    P.psv_page_write(cache.desc(), P.page_rows(P.PSV_DTYPE_BF16, k.shape, starts=at(starts)), at(k), at(v), stream())
    n = past + T
    kk, vv = (torch.zeros(B, n, Hkv, dh, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    P.psv_page_read(cache.desc(), P.page_rows(P.PSV_DTYPE_BF16, kk.shape), at(kk), at(vv), stream())
    o, lse = torch.zeros_like(q), torch.zeros(B, Hq, T, device="cuda")
    prob = P.cache_problem(P.PSV_DTYPE_BF16, q.shape, kk.shape, causal=True)
    m = P.psv_cache_scratch_bytes(prob)
    scratch = torch.zeros(m, dtype=torch.uint8, device="cuda")
    P.psv_cache_attention(prob, at(q), at(kk), at(vv), at(o), at(lse), at(scratch), m, stream())
    last = q[:, -5:].contiguous()
    o2, lse2 = torch.zeros_like(last), torch.zeros(B, Hq, 5, device="cuda")
    kl = ints([n] * B)
    query = P.page_query(P.PSV_DTYPE_BF16, last.shape, causal=True, k_lens=at(kl))
    w = torch.empty(P.psv_page_scratch_bytes(cache.desc(), query), dtype=torch.uint8, device="cuda")
    P.psv_page_attention(cache.desc(), query, at(last), at(o2), at(lse2), at(w), w.numel(), stream())
    # the chunk's keys and values are rounded to bf16 once more on their way (2^-8), its weights too
    e = torch.softmax(torch.einsum("bihd,bjhd->bihj", last.double(), kk.double().repeat_interleave(3, 2)) * dh**-0.5
                      + torch.triu(torch.full((5, n), -INF, device="cuda", dtype=torch.float64), n - 4)[None, :, None], -1)
    A = torch.einsum("bihj,bjhd->bihd", e, vv.double().abs().repeat_interleave(3, 2))
    es = 2.0**-8 * dh**-0.5 * torch.einsum("bihd,bjhd->bihj", last.double().abs(), kk.double().abs().repeat_interleave(3, 2)).amax(-1, keepdim=True)
    tol = (3 * 2.0**-8 + 2 * es) * A + 2 * 2.0**-8 * o2.double().abs()
    assert ((o2.double() - o[:, -5:].double()).abs() <= tol).all()
    assert ((lse2.transpose(1, 2) - lse[:, :, -5:].transpose(1, 2)).abs() <= es[..., 0] + 1e-4).all()


def test_host_memory_and_captures_that_fail(P):
    c = dict(B=1, Lq=1, Lk=40, Hq=2, Hkv=1, dh=64, page=16)
    cache, q, _, lens, _, rows = attention_case(P, c, "bf16", "e4m3")
    x = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16).pin_memory()
    y = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    r = P.page_rows(P.PSV_DTYPE_BF16, x.shape)
    plain = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    for call in (P.psv_page_write, P.psv_page_read):
        for bad in (x, plain):
            with pytest.raises(P.PSVError) as e:
                call(cache.desc(), r, at(bad), at(y), stream())
            assert e.value.code == P.PSV_EINVAL and "device" in str(e.value)
    query = P.page_query(P.PSV_DTYPE_BF16, q.shape)
    w = torch.empty(P.psv_page_scratch_bytes(cache.desc(), query), dtype=torch.uint8, device="cuda")
    with pytest.raises(P.PSVError):
        P.psv_page_attention(cache.desc(), query, at(q), at(plain), 0, at(w), w.numel(), stream())
    o, lse = run_attention(P, c, cache, q, lens, rows, "bf16")  # and the next call works
    assert torch.isfinite(o.float()).all()


def test_nothing_to_do_and_no_lse(P):
    c = dict(B=2, Lq=2, Lk=40, Hq=2, Hkv=1, dh=64, page=16, lens=[0, 0], rows=[0, 0])
    cache, q, _, lens, _, rows = attention_case(P, c, "bf16", "e4m3")
    o, lse = run_attention(P, c, cache, q, lens, rows, "bf16")
    assert (o == 9.0).all() and (lse == 9.0).all()
    o, lse = run_attention(P, dict(c, rows=[2, 1]), cache, torch.zeros_like(q), [0, 0], [2, 1], "bf16")
    assert (o[0] == 0).all() and (o[1, 0] == 0).all() and (o[1, 1] == 9.0).all()
    assert (lse[0] == -INF).all() and (lse[1, :, 0] == -INF).all()
    c = dict(B=2, Lq=1, Lk=400, Hq=2, Hkv=1, dh=64, page=16)
    cache, q, (k, v), lens, total, rows = attention_case(P, c, "bf16", "e4m3", width=WIDE)
    want, _ = run_attention(P, c, cache, q, lens, rows, "bf16")
    kl = ints(lens)
    query = P.page_query(P.PSV_DTYPE_BF16, q.shape, k_lens=at(kl))
    w = torch.empty(P.psv_page_scratch_bytes(cache.desc(), query), dtype=torch.uint8, device="cuda")
    o = torch.zeros_like(q)
    P.psv_page_attention(cache.desc(), query, at(q), at(o), 0, at(w), w.numel(), stream())
    assert torch.equal(o, want)


@pytest.mark.parametrize("width", [0, WIDE])
@pytest.mark.parametrize("f", ["e4m3", "i8"])
def test_pages_aligned_to_eight_bytes(P, f, width):
    """Heads of 128 whose pages begin, and whose rows lie, at odd multiples of eight bytes."""
    c = dict(B=2, Lq=3, Lk=210, Hq=4, Hkv=2, dh=128, page=16, causal=True, lens=[210, 37])
    cache, q, (k, v), lens, total, rows = attention_case(P, c, "bf16", f, width=width)
    ref = reference(cache, c, q, k, v, total, rows)
    n, h, r, d = cache.k.shape
    for name in ("k", "v"):
        wide = torch.full((n * h * r * 136 + 16,), 0x7F, device="cuda", dtype=torch.uint8)[8:8 + n * h * r * 136].view(n, h, r, 136)
        wide[..., :128] = getattr(cache, name)
        setattr(cache, name, wide[..., :128])
    check(*run_attention(P, c, cache, q, lens, rows, "bf16"), ref, rows, 9.0)


@pytest.mark.parametrize("dh", [64, 80])
def test_windows_and_lengths_at_the_ends_of_their_range(P, dh):
    c = dict(B=2, Lq=4, Lk=100, Hq=2, Hkv=1, dh=dh, page=16, causal=True, window=2**31 - 1, sinks=2**31 - 1, lens=[100, 2])
    cache, q, (k, v), lens, total, rows = attention_case(P, c, "f16", "i8")
    ref = reference(cache, dict(c, window=0, sinks=0), q, k, v, total, rows)
    check(*run_attention(P, c, cache, q, lens, rows, "f16"), ref, rows, 9.0)
    # lengths beyond what there is are cut to it; negative ones are nothing
    o, lse = run_attention(P, dict(c, window=0, sinks=0, rows=[2**31 - 1, -5]), cache, q, [2**31 - 1, 50], [2**31 - 1, -5], "f16")
    full = cache.max_pages * 16
    assert (o[1] == 9.0).all() and (lse[1] == 9.0).all()
    pos = torch.arange(full, device="cuda")
    e = cache.table[0].long()[pos // 16]
    cache.ks[e, :, pos % 16] = torch.nan_to_num(cache.ks[e, :, pos % 16], 0)  # rows behind the written ones: zeros
    cache.vs[e, :, pos % 16] = torch.nan_to_num(cache.vs[e, :, pos % 16], 0)
    o, lse = run_attention(P, dict(c, window=0, sinks=0, rows=[9, -5]), cache, q, [2**31 - 1, 50], [9, -5], "f16")
    pad = torch.zeros(2, full - 100, 1, dh, device="cuda", dtype=torch.float64)
    ref = reference(cache, dict(c, window=0, sinks=0), q, torch.cat([k, pad], 1), torch.cat([v, pad], 1), [full, 50], [4, 0])
    check(o, lse, ref, [4, 0], 9.0)


FIRST_CALLS = """
import sys
sys.path.insert(0, {root!r})
sys.path.insert(0, {tests!r})
import torch
from test_gpu_page_edges import Decoder
from autoregressive_denoising_dit_gb300 import _psv as P
d = Decoder(P, f={f!r}, Hq={Hq}, dh={dh}, max_pages={max_pages})
d.feed(torch.Generator(device="cuda").manual_seed(1))
x = torch.zeros(3, 4, 2, {dh}, device="cuda", dtype=torch.bfloat16)
r = P.page_rows(P.PSV_DTYPE_BF16, x.shape)
y = torch.zeros_like(x)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    d.step()
    P.psv_page_read(d.desc, r, x.data_ptr(), y.data_ptr(), torch.cuda.current_stream().cuda_stream)
d.before.zero_()
d.feed(torch.Generator(device="cuda").manual_seed(1))
g.replay()
torch.cuda.synchronize()
o, lse, kx = d.o.clone(), d.lse.clone(), x.clone()
d.before.zero_()
d.feed(torch.Generator(device="cuda").manual_seed(1))
d.step()
torch.cuda.synchronize()
assert torch.equal(o, d.o) and torch.equal(lse, d.lse) and float(o.abs().sum()) > 0 and float(kx[:, 0].abs().sum()) > 0
print("captured")
"""


@pytest.mark.parametrize("kw", [dict(f="e4m3", Hq=8, dh=128, max_pages=12), dict(f="i8", Hq=24, dh=64, max_pages=3000),
                                dict(f="bf16", Hq=2, dh=128, max_pages=3000), dict(f="e4m3", Hq=4, dh=20, max_pages=12)],
                         ids=lambda k: f"{k['f']}-{k['Hq']}-{k['dh']}-{k['max_pages']}")
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

    kinds = [dict(f="e4m3"), dict(f="i8", Hq=24, max_pages=300), dict(f="bf16", max_pages=300), dict(f="e4m3", dh=64, Hq=2)]
    bad = []
    lens = ints([20, 70, 150])

    def made(kw):
        d = Decoder(P, **kw)
        x = torch.randn(3, 150, 2, d.k.shape[3], device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
        P.psv_page_write(d.desc, P.page_rows(P.PSV_DTYPE_BF16, x.shape, lens=at(lens)), at(x), at(x), stream())
        d.before.copy_(lens)
        d.feed(torch.Generator(device="cuda").manual_seed(3))
        return d

    want, got = [made(kw) for kw in kinds], [made(kw) for kw in kinds]
    for d in want:
        for _ in range(25):
            d.step()
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for k in range(25):
                    got[i].step()
                    if k % 5 == i:
                        with pytest.raises(P.PSVError, match=f"scratch of {i} bytes"):
                            P.psv_page_attention(got[i].desc, got[i].query, at(got[i].q), at(got[i].o), 0, at(got[i].scratch), i, stream())
                torch.cuda.current_stream().synchronize()
            assert torch.equal(got[i].o, want[i].o) and torch.equal(got[i].lse, want[i].lse)
        except BaseException as e:  # noqa: BLE001 (handed to the test's thread)
            bad.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


@pytest.mark.parametrize("dh,Lq", [(128, 4), (64, 7), (256, 2)])
@pytest.mark.parametrize("f", ["bf16", "f16", "e4m3"])
def test_many_copies_of_a_sequence(P, f, dh, Lq):
    """700 copies (a warp has each): all the same, as the definition has it, infinite values that some rows see too."""
    dtype = "f16" if f == "f16" else "bf16"
    c = dict(B=1, Lq=Lq, Lk=60, Hq=4, Hkv=2, dh=dh, page=16, causal=True)
    cache, q, (k, v), lens, total, rows = attention_case(P, c, dtype, f)
    hit = torch.zeros(Lq, 4, dh, dtype=torch.bool, device="cuda")
    if f in DT:  # the last row's own value
        e, r = int(cache.table[0, 59 // 16]), 59 % 16
        cache.v[e, 0, r, 7], cache.v[e, 1, r, 9] = INF, float("nan")
        v[0, 59, 0, 7] = v[0, 59, 1, 9] = 0
        hit[-1, :2, 7] = hit[-1, 2:, 9] = True
    want_o, tol, want_lse, ltol = reference(cache, c, q, k, v, total, rows)[0]
    d = cache.desc()
    d.B, d.table_stride = 700, 0
    cache.desc = lambda: d
    o, lse = run_attention(P, dict(c, B=700), cache, q.expand(700, -1, -1, -1).contiguous(), lens * 700, rows * 700, dtype)
    assert torch.equal(torch.nan_to_num(o.float(), 3e4, 2e4), torch.nan_to_num(o[:1].float(), 3e4, 2e4).expand_as(o)) and torch.equal(lse, lse[:1].expand_as(lse))
    assert ((o[0].double() - want_o).abs() <= tol)[~hit].all() and not torch.isfinite(o[0][hit].float()).any()
    assert ((lse[0].T.double() - want_lse).abs() <= ltol).all()


def test_a_captured_step_of_many_sequences(P):
    eager, graphed = (Decoder(P, B=300, Hq=4, Hkv=2, max_pages=3) for _ in range(2))
    start = ints([b % 22 for b in range(300)])
    gens = [torch.Generator(device="cuda").manual_seed(7) for _ in range(2)]
    x = torch.randn(300, 22, 2, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    for d in (eager, graphed):
        P.psv_page_write(d.desc, P.page_rows(P.PSV_DTYPE_BF16, x.shape, lens=at(start)), at(x), at(x), stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for d in (eager, graphed):
        d.before.copy_(start)
    for _ in range(30):  # some pass the ends of their tables
        eager.feed(gens[0])
        eager.step()
        graphed.feed(gens[1])
        graph.replay()
        assert torch.equal(eager.o, graphed.o) and torch.equal(eager.lse, graphed.lse)


@pytest.mark.parametrize("width", [0, WIDE])
@pytest.mark.parametrize("f", ["bf16", "f16"])
@pytest.mark.parametrize("Lq", [24, 37])
def test_an_infinite_value_and_many_rows(P, f, width, Lq):
    c = dict(B=1, Lq=Lq, Lk=90, Hq=4, Hkv=4, dh=128, page=16, causal=True)
    cache, q, (k, v), lens, total, rows = attention_case(P, c, f, f, width=width)
    e, r = int(cache.table[0, 84 // 16]), 84 % 16
    cache.v[e, 0, r, 7] = INF
    cache.v[e, 1, r, 9] = float("nan")
    v2 = v.clone()
    v2[0, 84, 0, 7] = v2[0, 84, 1, 9] = 0
    o, lse = run_attention(P, c, cache, q, lens, rows, f)
    want_o, tol, want_lse, ltol = reference(cache, c, q, k, v2, total, rows)[0]
    first = 84 - (90 - Lq)
    assert (o[0, first:, 0, 7] == INF).all() and torch.isnan(o[0, first:, 1, 9].float()).all()
    hit = torch.zeros(o.shape[1:], dtype=torch.bool, device="cuda")
    hit[first:, 0, 7] = hit[first:, 1, 9] = True
    assert ((o[0].double() - want_o).abs() <= tol)[~hit].all()
    assert ((lse[0].T.double() - want_lse).abs() <= ltol).all()


@pytest.mark.parametrize("width", [0, WIDE])
@pytest.mark.parametrize("f", ["e4m3", "i8"])
def test_scales_of_any_size_and_many_rows(P, f, width):
    c = dict(B=2, Lq=7, Lk=333, Hq=6, Hkv=2, dh=64, page=64, causal=True, lens=[333, 100], rows=[7, 6])
    cache, q, _, lens, total, rows = attention_case(P, c, "f16", f, width=width)
    g = torch.Generator(device="cuda").manual_seed(9)
    k, v = (torch.randn(2, 333, 2, 64, device="cuda", generator=g) for _ in range(2))
    v = v * torch.exp2(torch.randint(-60, 0, (2, 333, 2, 1), device="cuda", generator=g).float())
    k = k * torch.exp2(torch.randint(-40, 1, (2, 333, 2, 1), device="cuda", generator=g).float())
    v[:, ::7], k[:, ::11] = 0, 0
    k, v = cache.fill(k.double(), v.double(), lens)
    o, lse = run_attention(P, c, cache, q, lens, rows, "f16")
    check(o, lse, reference(cache, c, q, k, v, total, rows), rows, 9.0)

"""Measured cases of libpsv's operators of a paged, quantised key/value cache.

Three operators that belong together: writing new keys and values into the pages of a
cache, in 8 bits with a scale for each token and head (psv_page_write), reading positions
back into plain tensors, as attention with many rows takes them (psv_page_read), and
attention of one new token, or a few, over the pages (psv_page_attention).

``listed()`` and ``draw()`` give cases, ``prepare()`` their inputs on the GPU, ``run()`` one
pass: in plain torch operations, or, where ``own`` is set, through the library's public
calls.  ``exact()`` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1, "i8": 1}
MOST_CODE = {"e4m3": 448.0, "i8": 127.0}
TINY = 2.0 ** -100  # a row whose largest size is below this is kept as zeros


def listed():
    return [
        # Eight streams that each add one token: the smallest call, bound by its launch.
        write("write token", "bf16", "e4m3", B=8, L=1, Hkv=12, dh=128, start=7800),
        # The keys and values of one wave: four chunks of 1560 tokens, appended at uneven places.
        write("write wave", "bf16", "e4m3", B=4, L=1560, Hkv=12, dh=128, start=4689, uneven=37),
        # Eight streams of a wide model whose rotated keys are still in 32 bits, a chunk a page.
        write("write chunks", "f32", "i8", B=8, L=1560, Hkv=40, dh=128, page=1560, start=1560),
        # One stream's window of five chunks as plain tensors, for the next chunk's attention.
        read("read window", "bf16", "e4m3", B=1, L=7800, Hkv=12, dh=128),
        # Eight streams of a wide model, unequal lengths, from a first position inside a page.
        read("read streams", "f16", "i8", B=8, L=6240, Hkv=40, dh=128, start=100, uneven=401),
        # One token against one chunk's cache: latency.
        attention("attention token", "bf16", "i8", B=1, Lq=1, Lk=1560, Hq=12, Hkv=12, dh=128),
        # One token of each of eight streams with caches of unequal length: bound by reading them.
        attention("attention tokens", "bf16", "e4m3", B=8, Lq=1, Lk=7800, Hq=12, Hkv=12, dh=128, ragged=371),
        # The same from pages that are not quantised, small ones.
        attention("attention pages of 16 bits", "bf16", "bf16", B=8, Lq=1, Lk=7800, Hq=12, Hkv=12, dh=128, page=16,
                  ragged=371),
        # Four drafted tokens behind a long cache, three query heads a kv head, capped scores.
        attention("attention draft", "f16", "i8", B=4, Lq=4, Lk=17600, Hq=24, Hkv=8, dh=128, causal=True, cap=50.0),
        # One long stream with shared heads: the cache is read by all SMs and joined.
        attention("attention long", "bf16", "e4m3", B=1, Lq=1, Lk=131072, Hq=40, Hkv=8, dh=128),
        # Many streams that see the last chunk and the first tokens; other pages are given back.
        attention("attention window", "bf16", "e4m3", B=64, Lq=1, Lk=7800, Hq=12, Hkv=12, dh=128, causal=True,
                  window=1560, sinks=52, ragged=53, dropped=True),
        # A step of eight streams: the new token's key and value are written, then it looks back.
        step("step", "bf16", "e4m3", B=8, Lk=3900, Hq=24, Hkv=12, dh=128, ragged=203),
    ]


def write(name, dtype, form, B, L, Hkv, dh, page=64, start=0, uneven=0):
    """start: the first position written; uneven: by what it differs from sequence to sequence."""
    return dict(op="write", name=name, dtype=dtype, form=form, B=B, L=L, Hkv=Hkv, dh=dh, page=page, start=start,
                uneven=uneven)


def read(name, dtype, form, **sizes):
    """uneven: what each further sequence reads less."""
    return dict(write(name, dtype, form, **sizes), op="read")


def attention(name, dtype, form, B, Lq, Lk, Hq, Hkv, dh, page=64, causal=False, window=0, sinks=0, cap=0.0, ragged=0,
              qcut=0, dropped=False):
    """ragged, qcut: what each further sequence has fewer in keys and rows; dropped: pages that no
    row sees have no entry in the table."""
    return dict(op="attention", name=name, dtype=dtype, form=form, B=B, Lq=Lq, Lk=Lk, Hq=Hq, Hkv=Hkv, dh=dh, page=page,
                causal=causal, window=window, sinks=sinks, cap=cap, ragged=ragged, qcut=qcut, dropped=dropped)


def step(name, dtype, form, **sizes):
    return dict(attention(name, dtype, form, Lq=1, causal=True, **sizes), op="step")


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["write", "read", "attention", "attention", "attention", "step"])
    form = rng.choice(["e4m3", "e4m3", "i8", "i8", "bf16", "f16"])
    dtype = form if form in DTYPES else rng.choice(["bf16", "f16"])
    dh, page = rng.choice([32, 64, 80, 128, 128, 128]), rng.choice([8, 16, 24, 64, 64, 128, 1560])
    B, Hkv = log(1, 64), rng.choice([1, 2, 5, 8, 12, 40])
    if op in ("write", "read"):
        if form not in DTYPES and rng.random() < 0.3:
            dtype = "f32"
        L = log(1, 12480)
        while B * Hkv * L > 8 * 40 * 1500:
            B, L = max(1, B // 2), max(1, L * 2 // 3)
        make = write if op == "write" else read
        c = make("", dtype, form, B=B, L=L, Hkv=Hkv, dh=dh, page=page, start=rng.choice([0, log(1, 8000)]),
                 uneven=rng.choice([0, rng.randint(1, max(1, L // 9))]))
    else:
        G, Lk = rng.choice([1, 1, 2, 3, 5, 8]), log(1, 131072)
        while B * Hkv * Lk > 8 * 131072:
            if B > 1:
                B //= 2
            elif Hkv > 8:
                Hkv //= 2
            else:
                Lk //= 2
        while G > 1 and B * Hkv * G * Lk > 5 * 8 * 131072:
            G -= 1
        sizes = dict(B=B, Lk=Lk, Hq=G * Hkv, Hkv=Hkv, dh=dh, page=page, cap=rng.choice([0.0, 0.0, 0.0, 30.0]),
                     ragged=rng.choice([0, Lk // (B + 1)]))
        if rng.random() < 0.3 and Lk > 64:
            sizes.update(window=log(16, Lk), sinks=rng.choice([0, 4, 52]), dropped=rng.random() < 0.5)
        if op == "step":
            c = step("", dtype, form, **sizes)
        else:
            Lq = rng.choice([1, 1, 1, 2, rng.randint(2, 9)])
            while Lq > 1 and B * Hkv * G * Lq * Lk > 5 * 8 * 131072:
                Lq -= 1
            c = attention("", dtype, form, Lq=Lq, causal="window" in sizes or rng.random() < 0.7,
                          qcut=rng.choice([0, 0, 1]) if Lq > 1 else 0, **sizes)
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes

def starts(c):
    if c["op"] == "write":
        return [c["start"] + b * c["uneven"] for b in range(c["B"])]
    return [c["start"]] * c["B"]


def row_lens(c):
    """Rows of each sequence that are written, read, or ask."""
    if c["op"] == "write":
        return [c["L"]] * c["B"]
    if c["op"] == "read":
        return [max(0, c["L"] - b * c["uneven"]) for b in range(c["B"])]
    return [max(0, c["Lq"] - b * c["qcut"]) for b in range(c["B"])]


def key_lens(c):
    """Keys of each sequence, those of the rows among them."""
    return [max(0, c["Lk"] - b * c["ragged"]) for b in range(c["B"])]


def positions(c):
    """Positions that the table of pages covers."""
    if c["op"] in ("write", "read"):
        return max(s + n for s, n in zip(starts(c), row_lens(c)))
    return c["Lk"]


def table_width(c):
    return -(-positions(c) // c["page"])


def spans(c, b):
    """What rows of sequence b see, by row: (first, end of the sinks, first of the rest, end)."""
    n, q = key_lens(c)[b], row_lens(c)[b]
    for i in range(q):
        qp = n - q + i
        end = max(0, min(n, qp + 1)) if c["causal"] else n
        first = max(0, qp - c["window"] + 1) if c["window"] else 0
        yield min(c["sinks"], end), min(max(first, min(c["sinks"], end)), end), end


def keys_seen(c):
    """Keys that some row sees and pairs of a row and a key that it sees, over all sequences, for one head."""
    keys = pairs = 0
    for b in range(c["B"]):
        got = list(spans(c, b))
        pairs += sum(s + e - f for s, f, e in got)
        if got:
            sinks, first, end = max(s for s, _, _ in got), min(f for _, f, _ in got), max(e for _, _, e in got)
            keys += sinks + max(0, end - max(first, sinks))
    return keys, pairs


def work(c):
    scale = 0 if c["form"] in DTYPES else 4
    row = c["dh"] * SIZE[c["form"]] + scale  # a key's or a value's bytes in its page
    if c["op"] in ("write", "read"):
        rows = 2 * sum(row_lens(c)) * c["Hkv"]
        return {"bytes": rows * (c["dh"] * SIZE[c["dtype"]] + row), "flops": (3 if c["op"] == "write" else 1) * rows * c["dh"]}
    keys, pairs = keys_seen(c)
    rows = sum(row_lens(c)) * c["Hq"]
    asked = rows * (2 * c["dh"] * SIZE[c["dtype"]] + 4)
    new = 2 * c["B"] * c["Hkv"] * (c["dh"] * SIZE[c["dtype"]] + row) if c["op"] == "step" else 0
    return {"bytes": asked + new + 2 * keys * c["Hkv"] * row, "flops": 4 * pairs * c["Hq"] * c["dh"]}


# ----------------------------------------------------------------- inputs

def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]

    def randn(*shape, scale=1.0):
        # heads differ in size, as keys of trained models do
        size = torch.exp(0.5 * torch.randn(shape[-2], 1, device="cuda", generator=g))
        return torch.randn(*shape, device="cuda", generator=g) * size * scale

    def ints(a):
        return torch.tensor(np.ascontiguousarray(a), dtype=torch.int32, device="cuda")

    B, Hkv, dh, page, width = c["B"], c["Hkv"], c["dh"], c["page"], table_width(c)
    s = {"case": c}
    # a pool shared by the sequences, with a few pages more than they use, in any order
    n_pages = B * width + 3
    order = torch.randperm(n_pages, device="cuda", generator=g)[:B * width].view(B, width).int()
    if c["op"] in ("attention", "step") and c["dropped"]:
        at = torch.arange(width, device="cuda")[None] * page
        n = ints([k - q for k, q in zip(key_lens(c), row_lens(c))])[:, None]
        order = torch.where((at + page <= n - c["window"]) & (at >= c["sinks"]), torch.full_like(order, -1), order)
    s["table"] = order.contiguous()
    filled = c["op"] != "write"
    for name in ("k", "v"):
        if filled:  # head by head, as a page holds them
            x = torch.cat([randn(n_pages, page, 1, dh) for _ in range(Hkv)], 2).transpose(1, 2).contiguous()
            s[name + "_pages"], s[name + "_scales"] = quantise(x.to(dt).float(), c["form"])
        else:
            s[name + "_pages"] = torch.zeros(n_pages, Hkv, page, dh, device="cuda", dtype=store_type(c["form"]))
            s[name + "_scales"] = None if c["form"] in DTYPES else torch.zeros(n_pages, Hkv, page, device="cuda")
    s["ql"] = ints(row_lens(c))
    if c["op"] in ("write", "read"):
        s["starts"] = ints(starts(c))
        s["lens"] = s["ql"] if c["op"] == "read" and c["uneven"] else None
        s["k"], s["v"] = ((randn(B, c["L"], Hkv, dh) if c["op"] == "write" else torch.zeros(B, c["L"], Hkv, dh, device="cuda")).to(dt)
                          for _ in range(2))
    else:
        s["kl"] = ints(key_lens(c))
        s["before"] = s["kl"] - s["ql"]
        s["q_lens"] = s["ql"] if c["qcut"] else None
        s["q"] = randn(B, c["Lq"], c["Hq"], dh, scale=1.3).to(dt)
        s["o"] = torch.zeros(B, c["Lq"], c["Hq"], dh, device="cuda", dtype=dt)
        s["lse"] = torch.zeros(B, c["Hq"], c["Lq"], device="cuda")
        if c["op"] == "step":  # keys and values come out of one product with the queries
            new = randn(B, 1, 2 * Hkv, dh).to(dt)
            s["k"], s["v"] = new[:, :, :Hkv], new[:, :, Hkv:]
    if own:
        s["plan"] = plan(s)
    return s


# ------------------------------------------------------------ plain forms

def store_type(form):
    return DTYPES.get(form, torch.uint8)


def quantise(x, form):
    """[..., dh] in 32 bits: what is stored, and a scale for each row."""
    if form in DTYPES:
        return x.to(DTYPES[form]), None
    most = torch.full((), MOST_CODE[form], device=x.device)
    size = x.abs().amax(-1)
    kept = size >= TINY
    turn = torch.where(kept & torch.isfinite(size), most / size, torch.zeros_like(size))
    y = torch.where(turn[..., None] > 0, x * turn[..., None], torch.zeros_like(x))
    scale = torch.where(torch.isfinite(size), size / most, torch.full_like(size, math.nan))
    scale = torch.where(size < TINY, torch.zeros_like(size), scale)
    code = y.to(torch.float8_e4m3fn).view(torch.uint8) if form == "e4m3" else torch.round(y).to(torch.int8).view(torch.uint8)
    return code, scale


def as_values(pages, form):
    """The stored bytes as numbers (a view)."""
    return pages if form in DTYPES else pages.view(torch.float8_e4m3fn if form == "e4m3" else torch.int8)


def at_positions(s, pos):
    """Page and row of positions [B, n], and whether the table names a page there."""
    c, table = s["case"], s["table"]
    p = torch.div(pos, c["page"], rounding_mode="floor")
    inside = (p >= 0) & (p < table.shape[1])
    entry = torch.gather(table.long(), 1, p.clamp(0, table.shape[1] - 1))
    ok = inside & (entry >= 0) & (entry < s["k_pages"].shape[0])
    return torch.where(ok, entry, torch.zeros_like(entry)), pos % c["page"], ok


def gathered(s, name, pos):
    """Values [B, n, Hkv, dh] in 32 bits at positions [B, n]; zeros where there is no page."""
    form = s["case"]["form"]
    page, row, ok = at_positions(s, pos)
    x = as_values(s[name + "_pages"][page, :, row], form).float()
    if s[name + "_scales"] is not None:
        x = x * s[name + "_scales"][page, :, row][..., None]
    return torch.where(ok[..., None, None], x, torch.zeros_like(x)), ok


def plain_write(s):
    c = s["case"]
    i = torch.arange(s["k"].shape[1], device="cuda")
    first = s["starts"] if c["op"] == "write" else s["before"]
    page, row, _ = at_positions(s, first.long()[:, None] + i)  # (each has a page of its own)
    for name in ("k", "v"):
        code, scale = quantise(s[name].float(), c["form"])
        s[name + "_pages"][page, :, row] = code
        if scale is not None:
            s[name + "_scales"][page, :, row] = scale
    return pages_of(s)


def pages_of(s):
    out = {}
    for name in ("k", "v"):
        out[name + "_pages"] = as_values(s[name + "_pages"], s["case"]["form"])
        if s[name + "_scales"] is not None:
            out[name + "_scales"] = s[name + "_scales"]
    return out


def plain_read(s):
    i = torch.arange(s["case"]["L"], device="cuda")
    pos = s["starts"].long()[:, None] + i
    there = (i < s["ql"][:, None])[..., None, None]
    return {name: torch.where(there, gathered(s, name, pos)[0].to(s[name].dtype), s[name]) for name in ("k", "v")}


def plain_attention(s):
    c = s["case"]
    B, Lq, Lk, Hq, Hkv, dh = (c[n] for n in ("B", "Lq", "Lk", "Hq", "Hkv", "dh"))
    i, j = torch.arange(Lq, device="cuda"), torch.arange(Lk, device="cuda")
    k, ok = gathered(s, "k", j.expand(B, -1))
    v, _ = gathered(s, "v", j.expand(B, -1))
    kl, ql = s["kl"].long(), s["ql"].long()
    qp = ((kl - ql)[:, None] + i)[:, :, None]
    ok = (ok & (j < kl[:, None]))[:, None] & (i < ql[:, None])[:, :, None]
    if c["causal"]:
        ok = ok & (j <= qp)
    if c["window"]:
        ok = ok & ((j > qp - c["window"]) | (j < c["sinks"]))
    q = s["q"].float().view(B, Lq, Hkv, Hq // Hkv, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, dh)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, Hq, Lq, Lk)
    x *= 1.0 / math.sqrt(dh)
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    x = x.masked_fill_(~ok[:, None], -math.inf)
    m = x.amax(3, keepdim=True)
    x -= torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.exp_()
    l = x.sum(3, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, -1, Lk), v.permute(0, 2, 1, 3)).view(B, Hq, Lq, dh)
    o = o / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + torch.log(l))[..., 0]
    there = i < ql[:, None]
    o = torch.where(there[:, :, None, None], o.transpose(1, 2).to(s["q"].dtype), s["o"])
    return {"o": o, "lse": torch.where(there[:, None], lse, s["lse"])}


def plain_step(s):
    pages = plain_write(s)
    return dict(plain_attention(s), **pages)


# ------------------------------------------------------------ own calls

def plan(s):
    """The descriptions and the workspace that a program keeps for its calls, and its stream."""
    from autoregressive_denoising_dit_gb300 import _psv as P

    c = s["case"]
    dtype = {"bf16": P.PSV_DTYPE_BF16, "f16": P.PSV_DTYPE_F16, "f32": P.PSV_DTYPE_F32}[c["dtype"]]
    form = {"bf16": P.PSV_PAGE_BF16, "f16": P.PSV_PAGE_F16, "e4m3": P.PSV_PAGE_E4M3, "i8": P.PSV_PAGE_I8}[c["form"]]

    def at(t):
        return 0 if t is None else t.data_ptr()

    # pages [n_pages][Hkv][page][dh]: strides of a page, a row, a head
    st = s["k_pages"].stride()
    cache = P.page_cache(form, s["table"].shape, s["k_pages"].shape[0], c["page"], c["Hkv"], c["dh"], at(s["table"]),
                         at(s["k_pages"]), at(s["v_pages"]), at(s["k_scales"]), at(s["v_scales"]),
                         k_stride=(st[0], st[2], st[1]), v_stride=(st[0], st[2], st[1]))
    p = {"P": P, "cache": cache, "stream": torch.cuda.current_stream().cuda_stream}
    if c["op"] in ("write", "read"):
        p["rows"] = P.page_rows(dtype, s["k"].shape, k_stride=s["k"].stride()[:3], v_stride=s["v"].stride()[:3],
                                starts=at(s["starts"]), lens=at(s["lens"]))
        return p
    append = c["op"] == "step"
    if append:
        p["rows"] = P.page_rows(dtype, s["k"].shape, k_stride=s["k"].stride()[:3], v_stride=s["v"].stride()[:3],
                                starts=at(s["before"]))
    p["query"] = P.page_query(dtype, s["q"].shape, causal=c["causal"], window=c["window"], sinks=c["sinks"],
                              softcap=c["cap"], q_lens=at(s["q_lens"]), k_lens=at(s["before"] if append else s["kl"]),
                              append=append)
    n = P.psv_page_scratch_bytes(cache, p["query"])
    p["scratch"], p["bytes"] = torch.zeros(n, dtype=torch.uint8, device="cuda"), n
    return p


def run_own(s):
    op, p = s["case"]["op"], s["plan"]
    P = p["P"]
    if op in ("write", "step"):
        P.psv_page_write(p["cache"], p["rows"], s["k"].data_ptr(), s["v"].data_ptr(), p["stream"])
        if op == "write":
            return pages_of(s)
    if op == "read":
        P.psv_page_read(p["cache"], p["rows"], s["k"].data_ptr(), s["v"].data_ptr(), p["stream"])
        return {"k": s["k"], "v": s["v"]}
    P.psv_page_attention(p["cache"], p["query"], s["q"].data_ptr(), s["o"].data_ptr(), s["lse"].data_ptr(),
                         p["scratch"].data_ptr(), p["bytes"], p["stream"])
    out = {"o": s["o"], "lse": s["lse"]}
    return out if op == "attention" else dict(out, **pages_of(s))


def run(s):
    if own:
        return run_own(s)
    return {"write": plain_write, "read": plain_read, "attention": plain_attention, "step": plain_step}[s["case"]["op"]](s)


# ------------------------------------------------------- the definition

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "write":
        return exact_write(c, s)[0]
    if c["op"] == "read":
        out = {}
        for name in ("k", "v"):
            out[name] = s[name].double()
            for b, (first, n) in enumerate(zip(starts(c), row_lens(c))):
                if n:
                    out[name][b, :n] = exact_rows(c, s, name, b, first, n)
        return out
    if c["B"] * c["Hq"] * c["Lq"] * c["Lk"] > 1e9:
        return None
    pages = {}
    if c["op"] == "step":
        pages, new = exact_write(c, s)
    o, lse = s["o"].double(), s["lse"].double()
    G = c["Hq"] // c["Hkv"]
    for b, (n, q) in enumerate(zip(key_lens(c), row_lens(c))):
        if not q:
            continue
        k, v = (exact_rows(c, s, name, b, 0, n) for name in ("k", "v"))
        if c["op"] == "step" and n:
            k[n - 1], v[n - 1] = new["k"][b], new["v"][b]
        entry = s["table"][b].long().repeat_interleave(c["page"])[:n]
        for h in range(c["Hq"]):
            x = s["q"][b, :q, h].double() @ k[:, h // G].T / c["dh"] ** 0.5
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            see = torch.zeros(q, n, dtype=torch.bool, device="cuda")
            for i, (sinks, first, end) in enumerate(spans(c, b)):
                see[i, :sinks] = True
                see[i, first:end] = True
            x = torch.where(see & (entry >= 0), x, torch.full_like(x, -math.inf))
            top = x.amax(1, keepdim=True) if n else torch.full((q, 1), -math.inf, device="cuda", dtype=torch.float64)
            e = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
            z = e.sum(1, keepdim=True)
            o[b, :q, h] = torch.where(z > 0, e @ v[:, h // G] / z, torch.zeros_like(z))
            lse[b, h, :q] = (torch.log(z) + top)[:, 0]
    return dict({"o": o, "lse": lse}, **pages)


def stored_numbers(pages, form):
    """Stored bytes as 64-bit numbers: sign, exponent and fraction taken apart."""
    if form in DTYPES:
        return pages.double()
    u = pages.to(torch.int64)
    if form == "i8":
        return torch.where(u < 128, u, u - 256).double()
    e, f = u // 8 % 16, (u % 8).double()
    size = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e.double() - 10))
    return torch.where(u < 128, size, -size)


def exact_rows(c, s, name, b, first, n):
    """Keys or values [n, Hkv, dh] of sequence b from position `first` on, page by page."""
    out = torch.zeros(n, c["Hkv"], c["dh"], device="cuda", dtype=torch.float64)
    table, at = s["table"][b].tolist(), first
    while at < first + n:
        end = min(first + n, (at // c["page"] + 1) * c["page"])
        page, r0 = table[at // c["page"]], at % c["page"]
        if page >= 0:
            x = stored_numbers(s[name + "_pages"][page, :, r0:r0 + end - at], c["form"])
            if s[name + "_scales"] is not None:
                x = x * s[name + "_scales"][page, :, r0:r0 + end - at, None].double()
            out[at - first:end - first] = x.transpose(0, 1)
        at = end
    return out


def exact_write(c, s):
    """The pages after the write, and the new rows' values as they are kept."""
    pages, new = {}, {}
    if c["op"] == "write":
        first, lens = starts(c), row_lens(c)
    else:
        first, lens = s["before"].tolist(), [1] * c["B"]
    for name in ("k", "v"):
        x = s[name].double()
        if c["form"] in DTYPES:
            code, scale = x.to(DTYPES[c["form"]]).double(), None
            kept = code
        else:
            size = x.abs().amax(-1)
            scale = size / MOST_CODE[c["form"]]
            y = x / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
            if c["form"] == "i8":
                code = torch.round(y)
            else:  # the nearest multiple of the step at y's size
                e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
                code = torch.round(y * torch.exp2(3 - e)) * torch.exp2(e - 3)
            kept = code * scale[..., None]
        held = stored_numbers(s[name + "_pages"], c["form"])
        scales = None if scale is None else s[name + "_scales"].double()
        for b in range(c["B"]):
            i = torch.arange(lens[b], device="cuda")
            if not len(i):
                continue
            pos = first[b] + i
            page = s["table"][b].long()[pos // c["page"]]
            there = page >= 0
            page, row = page[there], (pos % c["page"])[there]
            held[page, :, row] = code[b, i[there]]
            if scale is not None:
                scales[page, :, row] = scale[b, i[there]]
        pages[name + "_pages"] = held.to(torch.int8) if c["form"] == "i8" else held
        if scale is not None:
            pages[name + "_scales"] = scales
        # (what attention sees of the new token)
        new[name] = kept[:, 0] if c["op"] == "step" else None
    return pages, new

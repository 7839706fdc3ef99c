"""Measured cases of libpsv's kernel-level cache operators.

Four operators that a rolling key/value cache needs beside the window
attention: rotary positions with several axes (psv_rope), attention over a
cache with masks, a score cap and a distance bias (psv_cache_attention), the
attention weight that every cached key received (psv_cache_mass), and the
eviction of the keys that received least (psv_cache_evict).

``listed()`` and ``draw()`` give cases, ``prepare()`` their inputs on the GPU,
``run()`` one pass: in plain torch operations, or, where ``own`` is set, through
the library's public calls.  ``exact()`` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # Eight streams that each add one token: the smallest call, bound by its launch.
        rope("rope token", "bf16", B=8, L=1, H=12, dh=128, t0=7800),
        # The queries of one wave: four chunks of 30 x 52 latent tokens.
        rope("rope wave", "bf16", B=4, L=1560, H=12, dh=128, t0=400),
        # Keys of eight streams kept in 32 bits turned back to position zero, pairs as two halves.
        rope("rope back", "f32", B=8, L=1560, H=40, dh=128, t0=90000, halves=True, inverse=True),
        # One token against one chunk's cache: latency.
        attention("attention token", "bf16", B=1, Lq=1, Lk=1560, Hq=12, Hkv=12, dh=128),
        # One token of each of eight streams with caches of unequal length: bound by reading them.
        attention("attention tokens", "bf16", B=8, Lq=1, Lk=7800, Hq=12, Hkv=12, dh=128, ragged=371),
        # A wave of four chunks over five chunks' keys, nearer tokens favoured.
        attention("attention wave", "bf16", B=4, Lq=1560, Lk=7800, Hq=12, Hkv=12, dh=128, bias=True),
        # Causal rows behind a prefix that all see, shared heads, capped scores.
        attention("attention prefix", "f16", B=1, Lq=4400, Lk=17600, Hq=24, Hkv=8, dh=128, causal=True,
                  prefix=880, cap=50.0),
        # Streams of unequal length packed into one row, each seeing itself only.
        attention("attention documents", "bf16", B=1, Lq=12480, Lk=12480, Hq=12, Hkv=12, dh=128, docs=9),
        # The weight that one token of each of eight streams gave to its cache.
        mass("mass tokens", "bf16", B=8, Lq=1, Lk=7800, Hq=12, Hkv=12, dh=128, ragged=371),
        # The weight that a wave of four chunks gave to its window.
        mass("mass wave", "bf16", B=4, Lq=1560, Lk=7800, Hq=12, Hkv=12, dh=128),
        # One stream's window of five chunks cut to three.
        evict("evict window", "bf16", B=1, L=7800, Hkv=12, dh=128, budget=4680, sinks=30, recent=1560),
        # Eight streams of a wide model, unequal lengths, cut by one chunk, with positions.
        evict("evict streams", "bf16", B=8, L=7800, Hkv=40, dh=128, budget=6240, sinks=52, recent=1560,
              ragged=401, meta=True),
    ]


def rope(name, dtype, B, L, H, dh, t0=0, halves=False, inverse=False, axes=3, packed=False):
    """packed: q sits in a [B, L, 3, H, dh] product of one projection (strided rows)."""
    return dict(op="rope", name=name, dtype=dtype, B=B, L=L, H=H, dh=dh, t0=t0, halves=halves, inverse=inverse,
                axes=axes, packed=packed)


def attention(name, dtype, B, Lq, Lk, Hq, Hkv, dh, causal=False, prefix=0, cap=0.0, bias=False, docs=0, ragged=0,
              qcut=0, ring=0):
    """ragged, qcut: what each further sequence has fewer in keys and rows; ring: cache slots are
    in ring order, turned by that many, with their positions given."""
    return dict(op="attention", name=name, dtype=dtype, B=B, Lq=Lq, Lk=Lk, Hq=Hq, Hkv=Hkv, dh=dh, causal=causal,
                prefix=prefix, cap=cap, bias=bias, docs=docs, ragged=ragged, qcut=qcut, ring=ring)


def mass(name, dtype, **sizes):
    return dict(attention(name, dtype, **sizes), op="mass")


def evict(name, dtype, B, L, Hkv, dh, budget, sinks, recent, ragged=0, meta=False):
    return dict(op="evict", name=name, dtype=dtype, B=B, L=L, Hkv=Hkv, dh=dh, budget=budget, sinks=sinks,
                recent=recent, ragged=ragged, meta=meta)


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    dtype = rng.choice(["bf16", "bf16", "f16"])
    op = rng.choice(["rope", "attention", "attention", "mass", "evict"])
    if op == "rope":
        dtype = rng.choice(["bf16", "f16", "f32"])
        H, dh, B = rng.choice([1, 3, 12, 24, 40]), rng.choice([32, 64, 80, 128]), rng.randint(1, 8)
        L = min(log(1, 12480), 12480 * 40 * 128 // (B * H * dh))
        c = rope("", dtype, B=B, L=L, H=H, dh=dh, t0=log(1, 100000), halves=rng.random() < 0.4,
                 inverse=rng.random() < 0.3, axes=rng.randint(1, 3), packed=rng.random() < 0.3)
    elif op == "evict":
        L, B, Hkv = log(8, 32768), rng.randint(1, 8), rng.choice([1, 4, 8, 12, 40])
        while B * Hkv * L > 8 * 40 * 6000:
            B = max(1, B // 2)
            Hkv = max(1, Hkv // 2)
        budget = max(1, int(L * rng.uniform(0.2, 0.95)))
        recent = int(budget * rng.uniform(0, 0.5))
        c = evict("", dtype, B=B, L=L, Hkv=Hkv, dh=rng.choice([32, 64, 80, 128]), budget=budget,
                  sinks=min(rng.choice([0, 1, 4, 52]), budget - recent), recent=recent,
                  ragged=rng.choice([0, 0, L // 9]), meta=rng.random() < 0.5)
    else:
        G, Hkv, dh, B = rng.choice([1, 1, 2, 3, 8]), rng.choice([1, 2, 8, 12]), rng.choice([32, 64, 80, 128, 128]), rng.randint(1, 8)
        Lk = log(1, 32768)
        Lq = rng.choice([1, 1, rng.randint(2, 17), log(17, 8192), Lk])
        while B * Hkv * G * Lq * Lk > 12 * 9000 * 9000 or B * Hkv * Lk > 8 * 12 * 7800:
            if B > 1:
                B -= 1
            elif Hkv > 1:
                Hkv //= 2
            else:
                Lq = max(1, Lq // 2)
                G = 1
                Lk = min(Lk, 32768)
        mask = rng.choice(["full", "causal", "prefix", "docs", "causal docs"])
        c = attention("", dtype, B=B, Lq=Lq, Lk=Lk, Hq=G * Hkv, Hkv=Hkv, dh=dh, causal=mask not in ("full", "docs"),
                      prefix=rng.randint(1, Lk) if mask == "prefix" else 0, cap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                      bias=rng.random() < 0.4, docs=rng.randint(2, 12) if "docs" in mask and Lk >= 12 else 0,
                      ragged=rng.choice([0, Lk // 11]), qcut=rng.choice([0, Lq // 10]),
                      ring=rng.choice([0, 0, Lk // 3]))
        c["op"] = op
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes

def key_lens(c):
    Lk = c["L"] if c["op"] == "evict" else c["Lk"]
    return [max(0, Lk - b * c["ragged"]) for b in range(c["B"])]


def row_lens(c):
    return [max(0, c["Lq"] - b * c["qcut"]) for b in range(c["B"])]


def doc_of(c, pos):
    """The document that holds position pos (an array): unequal lengths."""
    cuts = [d * c["Lk"] // c["docs"] + (d * 37) % 5 for d in range(1, c["docs"])]
    return np.searchsorted(np.asarray(cuts), np.asarray(pos), side="right").astype(np.int32)


def pairs(c):
    """Pairs of a row and a key that it sees, over all sequences, for one head."""
    n = 0
    for kl, ql in zip(key_lens(c), row_lens(c)):
        qp = np.arange(kl - ql, kl)
        if c["ring"]:  # the slots in use hold any of the positions
            kp = np.sort((np.arange(kl) + c["ring"]) % c["Lk"])
        else:
            kp = np.arange(kl)
        if c["docs"]:
            kd, qd = doc_of(c, kp), doc_of(c, qp)
            lo, hi = np.searchsorted(kd, qd, "left"), np.searchsorted(kd, qd, "right")
        else:
            lo, hi = np.zeros(ql, np.int64), np.full(ql, kl)
        if c["causal"]:
            hi = np.minimum(hi, np.searchsorted(kp, np.maximum(qp, c["prefix"] - 1), "right"))
        n += int(np.maximum(hi - lo, 0).sum())
    return n


def work(c):
    w = SIZE[c["dtype"]]
    if c["op"] == "rope":
        n = c["B"] * c["L"] * c["H"] * c["dh"]
        return {"bytes": 2 * n * w + c["B"] * c["L"] * c["axes"] * 4, "flops": 3 * n}
    if c["op"] == "evict":
        lens = key_lens(c)
        kept = sum(min(n, c["budget"]) for n in lens) * c["Hkv"]
        seen = sum(lens) * c["Hkv"]
        return {"bytes": 4 * seen + kept * (4 * c["dh"] * w + 8 + (12 if c["meta"] else 0)), "flops": seen}
    keys, rows = sum(key_lens(c)), sum(row_lens(c))
    meta = (4 * keys if c["docs"] else 0) + (4 * keys if c["ring"] else 0)
    if c["op"] == "attention":
        return {"bytes": 2 * rows * c["Hq"] * c["dh"] * w + 4 * rows * c["Hq"] + 2 * keys * c["Hkv"] * c["dh"] * w + meta,
                "flops": 4 * pairs(c) * c["Hq"] * c["dh"]}
    return {"bytes": rows * c["Hq"] * (c["dh"] * w + 4) + keys * c["Hkv"] * (c["dh"] * w + 8) + meta,
            "flops": 2 * pairs(c) * c["Hq"] * c["dh"]}


def axis_dims(c):
    """Widths of the axes: all but time get an even third, as video models split a head."""
    if c["axes"] == 1:
        return [c["dh"]]
    rest = 2 * (c["dh"] // (2 * c["axes"]))
    return [c["dh"] - (c["axes"] - 1) * rest] + [rest] * (c["axes"] - 1)


# ----------------------------------------------------------------- inputs

def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dt)

    s = {"case": c}
    B, dh = c["B"], c["dh"]
    if c["op"] == "rope":
        # latent frames of 30 x 52 tokens from frame t0 on; each sequence starts a frame later
        if c["packed"]:
            s["x"] = randn(B, c["L"], 3, c["H"], dh)[:, :, 1]
        else:
            s["x"] = randn(B, c["L"], c["H"], dh)
        at = torch.arange(c["L"], device="cuda", dtype=torch.int32)
        first = torch.arange(B, device="cuda", dtype=torch.int32)[:, None] + c["t0"] + seed % 7
        thw = torch.stack([(first + at // 1560).expand(B, -1), (at // 52 % 30).expand(B, -1),
                           (at % 52).expand(B, -1)], 2)
        s["pos"] = thw[:, :, :c["axes"]].contiguous()
        s["out"] = torch.empty(B, c["L"], c["H"], dh, device="cuda", dtype=dt)
    elif c["op"] == "evict":
        L, H = c["L"], c["Hkv"]
        s["k"], s["v"] = randn(B, L, H, dh), randn(B, L, H, dh)
        # a few keys hold most of the weight; some keys were never seen (ties at zero)
        m = torch.exp(2.5 * torch.randn(B, H, L, device="cuda", generator=g))
        s["mass"] = torch.where(torch.rand(B, H, L, device="cuda", generator=g) < 0.05, torch.zeros_like(m), m)
        s["kl"] = torch.tensor(key_lens(c), device="cuda", dtype=torch.int32)
        s["lens"] = s["kl"] if c["ragged"] else None
        s["pos"] = torch.cumsum(torch.randint(1, 4, (B, H, L), device="cuda", generator=g, dtype=torch.int32), 2,
                                dtype=torch.int32) if c["meta"] else None
        n = c["budget"]
        s["k_out"], s["v_out"] = (torch.zeros(B, n, H, dh, device="cuda", dtype=dt) for _ in range(2))
        s["mass_out"] = torch.zeros(B, H, n, device="cuda")
        s["idx"] = torch.zeros(B, H, n, device="cuda", dtype=torch.int32)
        s["pos_out"] = torch.zeros(B, H, n, device="cuda", dtype=torch.int32) if c["meta"] else None
        s["lens_out"] = torch.zeros(B, device="cuda", dtype=torch.int32)
    else:
        Lq, Lk, Hq, Hkv = c["Lq"], c["Lk"], c["Hq"], c["Hkv"]
        s["q"] = randn(B, Lq, Hq, dh, scale=1.5)
        s["k"], s["v"] = randn(B, Lk, Hkv, dh), randn(B, Lk, Hkv, dh)
        kl, ql = key_lens(c), row_lens(c)

        def ints(a):
            return torch.tensor(np.ascontiguousarray(a), dtype=torch.int32, device="cuda")

        s["kl"], s["ql"] = ints(kl), ints(ql)
        s["k_lens"] = s["kl"] if c["ragged"] else None
        s["q_lens"] = s["ql"] if c["qcut"] else None
        s["k_pos"] = ints(np.broadcast_to((np.arange(Lk) + c["ring"]) % Lk, (B, Lk))) if c["ring"] else None
        s["q_pos"] = None  # default: the rows are the last of the sequence's positions
        if c["docs"]:
            kp = (np.arange(Lk) + c["ring"]) % Lk
            s["k_doc"] = ints(np.stack([doc_of(c, kp)] * B))
            s["q_doc"] = ints(np.stack([doc_of(c, np.arange(Lq) + k - q) for k, q in zip(kl, ql)]))
        else:
            s["k_doc"] = s["q_doc"] = None
        s["prefix"] = ints([c["prefix"]] * B) if c["prefix"] else None
        s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq)).float() if c["bias"] else None
        if c["op"] == "attention":
            s["o"] = torch.zeros(B, Lq, Hq, dh, device="cuda", dtype=dt)
            s["lse"] = torch.zeros(B, Hq, Lq, device="cuda")
        else:
            s["lse"] = torch.logsumexp(scores(s), 3)
            s["mass_in"] = torch.rand(B, Hkv, Lk, device="cuda", generator=g)
            s["mass_out"] = torch.zeros(B, Hkv, Lk, device="cuda")
    if own:
        s["plan"] = plan(s)
    return s


# ------------------------------------------------------------ plain forms

def angles(c, pos):
    """[B, L, pairs] in 64 bits."""
    parts = []
    for a, d in enumerate(axis_dims(c)):
        j = torch.arange(d // 2, device=pos.device, dtype=torch.float64)
        parts.append(pos[:, :, a, None].double() * torch.pow(torch.tensor(1e4, dtype=torch.float64, device=pos.device), -2.0 * j / d))
    return torch.cat(parts, 2)


def plain_rope(s):
    c, x = s["case"], s["x"].float()
    th = angles(c, s["pos"])
    cos, sin = torch.cos(th).float()[:, :, None], torch.sin(th).float()[:, :, None]
    if c["inverse"]:
        sin = -sin
    if c["halves"]:
        a, b = x.chunk(2, -1)
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return y.to(s["x"].dtype)


def seen(s):
    """[B, 1, Lq, Lk]: whether the row sees the key; and both positions."""
    c, dev = s["case"], s["q"].device
    kl, ql = s["kl"].long(), s["ql"].long()
    i, j = torch.arange(c["Lq"], device=dev), torch.arange(c["Lk"], device=dev)
    qp = (kl - ql)[:, None] + i
    kp = s["k_pos"].long() if s["k_pos"] is not None else j.expand(c["B"], -1)
    ok = (j < kl[:, None])[:, None, :] & (i < ql[:, None])[:, :, None]
    if s["k_doc"] is not None:
        ok = ok & (s["q_doc"][:, :, None] == s["k_doc"][:, None, :])
    if c["causal"]:
        ok = ok & ((kp[:, None, :] <= qp[:, :, None]) | (kp[:, None, :] < c["prefix"]))
    return ok[:, None], qp, kp


def scores(s):
    """[B, Hq, Lq, Lk] in 32 bits, -inf where the row does not see the key."""
    c = s["case"]
    B, Lq, Lk, Hq, Hkv, dh = (c[n] for n in ("B", "Lq", "Lk", "Hq", "Hkv", "dh"))
    q = s["q"].float().view(B, Lq, Hkv, Hq // Hkv, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, dh)
    x = torch.matmul(q, s["k"].float().permute(0, 2, 3, 1)).view(B, Hq, Lq, Lk)
    x *= 1.0 / math.sqrt(dh)
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    ok, qp, kp = seen(s)
    if s["slopes"] is not None:
        far = (qp[:, :, None] - kp[:, None, :]).abs().float()
        x -= s["slopes"][None, :, None, None] * far[:, None]
    return x.masked_fill_(~ok, -math.inf)


def plain_attention(s):
    c = s["case"]
    B, Lq, Lk, Hq, Hkv, dh = (c[n] for n in ("B", "Lq", "Lk", "Hq", "Hkv", "dh"))
    x = scores(s)
    m = x.amax(3, keepdim=True)
    x -= torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.exp_()
    l = x.sum(3, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, -1, Lk), s["v"].float().permute(0, 2, 1, 3)).view(B, Hq, Lq, dh)
    o = o / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + torch.log(l))[..., 0]
    there = torch.arange(Lq, device=x.device) < s["ql"][:, None]
    o = torch.where(there[:, :, None, None], o.transpose(1, 2).to(s["q"].dtype), s["o"])
    return {"o": o, "lse": torch.where(there[:, None], lse, s["lse"])}


def plain_mass(s):
    c = s["case"]
    x = scores(s)
    lse = s["lse"][..., None]
    p = torch.exp(x - torch.where(lse == -math.inf, torch.zeros_like(lse), lse))
    got = s["mass_in"] + p.view(c["B"], c["Hkv"], -1, c["Lk"]).sum(2)
    there = torch.arange(c["Lk"], device=x.device) < s["kl"][:, None]
    return torch.where(there[:, None], got, s["mass_out"])


def plain_evict(s):
    c = s["case"]
    B, H, L, n, dh = c["B"], c["Hkv"], c["L"], c["budget"], c["dh"]
    dev = s["k"].device
    lens = s["kl"].long()[:, None, None]
    j = torch.arange(L, device=dev)
    held = (j < c["sinks"]) | (j >= lens - c["recent"])
    key = torch.where(held, torch.full_like(s["mass"], math.inf), s["mass"])
    key = torch.where(j < lens, key, torch.full_like(key, -math.inf))
    first = torch.sort(key, dim=2, descending=True, stable=True).indices[:, :, :n]
    new = lens.clamp(max=n)
    used = (torch.arange(n, device=dev) < new).expand(B, H, n)
    idx = torch.sort(torch.where(used, first, torch.full_like(first, L)), dim=2).values
    at = idx.clamp(max=L - 1)
    rows = at.transpose(1, 2)[..., None].expand(B, n, H, dh)
    keep = used.transpose(1, 2)[..., None]
    out = {"k": torch.where(keep, torch.gather(s["k"], 1, rows), s["k_out"]),
           "v": torch.where(keep, torch.gather(s["v"], 1, rows), s["v_out"]),
           "mass": torch.where(used, torch.gather(s["mass"], 2, at), s["mass_out"]),
           "idx": torch.where(used, idx.int(), s["idx"]), "lens": new.view(B).int()}
    if s["pos"] is not None:
        out["pos"] = torch.where(used, torch.gather(s["pos"], 2, at), s["pos_out"])
    return out


# ------------------------------------------------------------ own calls

def plan(s):
    """The problem description and the workspace that a program keeps for its calls."""
    from autoregressive_denoising_dit_gb300 import _psv as P

    c = s["case"]
    dtype = {"bf16": P.PSV_DTYPE_BF16, "f16": P.PSV_DTYPE_F16, "f32": P.PSV_DTYPE_F32}[c["dtype"]]

    def at(t):
        return 0 if t is None else t.data_ptr()

    if c["op"] == "rope":
        return P, P.rope_problem(dtype, s["x"].shape, axis_dims(c), x_stride=s["x"].stride()[:3],
                                 out_stride=s["out"].stride()[:3], pos_stride=s["pos"].stride()[:2], theta=1e4,
                                 halves=c["halves"], inverse=c["inverse"])
    if c["op"] == "evict":
        return P, P.evict_problem(dtype, s["k"].shape, c["budget"], sinks=c["sinks"], recent=c["recent"],
                                  k_stride=s["k"].stride()[:3], v_stride=s["v"].stride()[:3],
                                  k_out_stride=s["k_out"].stride()[:3], v_out_stride=s["v_out"].stride()[:3],
                                  k_lens=at(s["lens"]), k_pos=at(s["pos"]),
                                  k_meta_stride=(c["Hkv"] * c["L"], c["L"]), pos_out=at(s["pos_out"]),
                                  lens_out=at(s["lens_out"]))
    prob = P.cache_problem(dtype, s["q"].shape, s["k"].shape, q_stride=s["q"].stride()[:3],
                           k_stride=s["k"].stride()[:3], v_stride=s["v"].stride()[:3],
                           o_stride=s["q"].stride()[:3], softcap=c["cap"], causal=c["causal"],
                           q_lens=at(s["q_lens"]), k_lens=at(s["k_lens"]), q_pos=at(s["q_pos"]), q_doc=at(s["q_doc"]),
                           q_meta_stride=c["Lq"], k_pos=at(s["k_pos"]), k_doc=at(s["k_doc"]),
                           k_meta_stride=(c["Lk"], 0), prefix=at(s["prefix"]), slopes=at(s["slopes"]))
    n = P.psv_cache_scratch_bytes(prob)
    return P, prob, torch.zeros(n, dtype=torch.uint8, device="cuda"), n


def run_own(s):
    c, stream = s["case"], torch.cuda.current_stream().cuda_stream
    P, prob = s["plan"][:2]
    if c["op"] == "rope":
        P.psv_rope(prob, s["x"].data_ptr(), s["pos"].data_ptr(), s["out"].data_ptr(), stream)
        return s["out"]
    if c["op"] == "evict":
        P.psv_cache_evict(prob, s["k"].data_ptr(), s["v"].data_ptr(), s["mass"].data_ptr(), s["k_out"].data_ptr(),
                          s["v_out"].data_ptr(), s["mass_out"].data_ptr(), s["idx"].data_ptr(), stream)
        out = {"k": s["k_out"], "v": s["v_out"], "mass": s["mass_out"], "idx": s["idx"], "lens": s["lens_out"]}
        if s["pos"] is not None:
            out["pos"] = s["pos_out"]
        return out
    scratch, n = s["plan"][2:]
    if c["op"] == "attention":
        P.psv_cache_attention(prob, s["q"].data_ptr(), s["k"].data_ptr(), s["v"].data_ptr(), s["o"].data_ptr(),
                              s["lse"].data_ptr(), scratch.data_ptr(), n, stream)
        return {"o": s["o"], "lse": s["lse"]}
    P.psv_cache_mass(prob, s["q"].data_ptr(), s["k"].data_ptr(), s["lse"].data_ptr(), s["mass_in"].data_ptr(),
                     s["mass_out"].data_ptr(), scratch.data_ptr(), n, stream)
    return s["mass_out"]


def run(s):
    if own:
        return run_own(s)
    return {"rope": plain_rope, "attention": plain_attention, "mass": plain_mass, "evict": plain_evict}[s["case"]["op"]](s)


# ------------------------------------------------------- the definition

def exact(c, seed):
    s = prepare(c, seed)
    return {"rope": exact_rope, "attention": exact_cache, "mass": exact_cache, "evict": exact_evict}[c["op"]](c, s)


def exact_rope(c, s):
    """Each pair as a complex number times exp(i angle)."""
    x = s["x"].double()
    out = torch.empty_like(x)
    dims = axis_dims(c)
    sign = -1.0 if c["inverse"] else 1.0
    first = 0
    for a, d in enumerate(dims):
        for j in range(d // 2):
            p = first + j
            lo, hi = (p, p + c["dh"] // 2) if c["halves"] else (2 * p, 2 * p + 1)
            th = sign * s["pos"][:, :, a].double() * math.exp(-math.log(1e4) * 2 * j / d)
            z = torch.complex(x[..., lo], x[..., hi]) * torch.polar(torch.ones_like(th), th)[:, :, None]
            out[..., lo], out[..., hi] = z.real, z.imag
        first += d // 2
    return out


def exact_cache(c, s):
    """Row block by row block of one sequence and head."""
    B, Lq, Lk, Hq, Hkv, dh = (c[n] for n in ("B", "Lq", "Lk", "Hq", "Hkv", "dh"))
    if B * Hq * Lq * Lk > 3e9:
        return None
    G = Hq // Hkv
    kl, ql = key_lens(c), row_lens(c)
    attn = c["op"] == "attention"
    if attn:
        o, lse = s["o"].double(), s["lse"].double()
    else:
        got = s["mass_out"].double()
    step = max(1, (1 << 26) // max(1, Lk))
    for b in range(B):
        n = kl[b]
        kp = torch.arange(n, device="cuda") if s["k_pos"] is None else s["k_pos"][b, :n].long()
        for h in range(Hq):
            k, v = s["k"][b, :n, h // G].double(), s["v"][b, :n, h // G].double()
            if not attn and h % G == 0:
                got[b, h // G, :n] = s["mass_in"][b, h // G, :n].double()
            for i0 in range(0, ql[b], step):
                i1 = min(i0 + step, ql[b])
                x = s["q"][b, i0:i1, h].double() @ k.T / dh ** 0.5
                if c["cap"]:
                    x = torch.tanh(x / c["cap"]) * c["cap"]
                qp = torch.arange(i0, i1, device="cuda")[:, None] + (n - ql[b])
                if c["bias"]:
                    x = x - float(s["slopes"][h]) * (qp - kp).abs()
                hide = torch.zeros_like(x, dtype=torch.bool)
                if c["causal"]:
                    hide |= (kp > qp) & (kp >= c["prefix"])
                if c["docs"]:
                    hide |= s["q_doc"][b, i0:i1, None] != s["k_doc"][b, None, :n]
                if attn:
                    # a large shift is taken out by the row's own largest visible score
                    top = torch.where(hide, torch.full_like(x, -math.inf), x).amax(1, keepdim=True) if n else x.new_full((i1 - i0, 1), -math.inf)
                    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
                else:
                    top = s["lse"][b, h, i0:i1, None].double()
                e = torch.exp(x - top)
                e = torch.where(hide, torch.zeros_like(e), e)
                if not attn:
                    got[b, h // G, :n] += e.sum(0)
                    continue
                z = e.sum(1, keepdim=True)
                o[b, i0:i1, h] = torch.where(z > 0, e @ v / z, torch.zeros_like(z))
                lse[b, h, i0:i1] = (torch.log(z) + top)[:, 0]
    return {"o": o, "lse": lse} if attn else got


def exact_evict(c, s):
    """Head by head: protected slots first, then by weight, the lower slot first among equals."""
    out = {"k": s["k_out"].double(), "v": s["v_out"].double(), "mass": s["mass_out"].double(), "idx": s["idx"].clone(),
           "lens": s["lens_out"].clone()}
    if s["pos"] is not None:
        out["pos"] = s["pos_out"].clone()
    weights = s["mass"].cpu().numpy().astype(np.float64)
    for b, n in enumerate(key_lens(c)):
        m = min(n, c["budget"])
        out["lens"][b] = m
        slot = np.arange(n)
        held = (slot < c["sinks"]) | (slot >= n - c["recent"])
        for h in range(c["Hkv"]):
            order = np.lexsort((slot, -weights[b, h, :n], ~held))
            idx = torch.tensor(np.sort(order[:m]), device="cuda")
            out["idx"][b, h, :m] = idx.int()
            out["k"][b, :m, h] = s["k"][b, idx, h].double()
            out["v"][b, :m, h] = s["v"][b, idx, h].double()
            out["mass"][b, h, :m] = s["mass"][b, h, idx].double()
            if s["pos"] is not None:
                out["pos"][b, h, :m] = s["pos"][b, h, idx]
    return out

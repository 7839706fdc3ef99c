"""Argument checks of the rolling-cache operators (psv_rope, psv_cache_*): every
refusal is made on the host before any device call, so these run without a GPU."""
import ctypes

import numpy as np
import pytest

from autoregressive_denoising_dit_gb300 import _psv as P


@pytest.fixture(scope="module", autouse=True)
def built():
    from autoregressive_denoising_dit_gb300 import build

    build.build()


A = 1 << 20  # an aligned address that no refused call may touch


def refused(match, call, *args):
    with pytest.raises(P.PSVError) as e:
        call(*args)
    assert e.value.code == P.PSV_EINVAL
    assert match in str(e.value), str(e.value)


def changed(make, **kw):
    p = make()
    for name, value in kw.items():
        if isinstance(value, tuple):
            value = type(getattr(p, name))(*value)
        setattr(p, name, value)
    return p


def rope():
    return P.rope_problem(P.PSV_DTYPE_BF16, (2, 5, 3, 64), (24, 20, 20))


@pytest.mark.parametrize("match,kw", [
    ("dtype", dict(dtype=7)), ("B, L, H", dict(B=0)), ("B, L, H", dict(L=0)), ("B, L, H", dict(H=-1)),
    ("dh", dict(dh=63)), ("dh", dict(dh=258)), ("n_axes", dict(n_axes=0)), ("n_axes", dict(n_axes=5)),
    ("layout", dict(layout=2)), ("axis_dims", dict(axis_dims=(24, 21, 18, 0))),
    ("axis_dims", dict(axis_dims=(24, 0, 20, 0))), ("rotate", dict(axis_dims=(24, 20, 22, 0))),
    ("theta", dict(theta=0.0)), ("theta", dict(theta=float("nan"))), ("strides", dict(x_stride=(-1, 192, 64))),
    ("overlap", dict(out_stride=(960, 192, 32))), ("overlap", dict(out_stride=(0, 192, 64))),
    ("65535", dict(B=65536)), ("2^24", dict(L=1 << 23)), ("2^24", dict(L=1 << 22, H=4)),
])
def test_rope_refuses(match, kw):
    refused(match, P.psv_rope, changed(rope, **kw), A, A, 2 * A)


def test_rope_refuses_pointers_and_frequencies():
    refused("null", P.psv_rope, rope(), 0, A, A)
    refused("null", P.psv_rope, rope(), A, 0, A)
    refused("aligned", P.psv_rope, rope(), A + 1, A, 2 * A)
    refused("aligned", P.psv_rope, rope(), A, A + 2, 2 * A)
    refused("equal strides", P.psv_rope, changed(rope, x_stride=(2000, 192, 64)), A, 2 * A, A)
    f = np.ones(32)
    f[3] = np.inf
    refused("finite", P.psv_rope, P.rope_problem(P.PSV_DTYPE_F32, (1, 1, 1, 64), (64,), freqs=f), A, A, 2 * A)
    f[3] = 1e7
    refused("1e6", P.psv_rope, P.rope_problem(P.PSV_DTYPE_F32, (1, 1, 1, 64), (64,), freqs=f), A, A, 2 * A)
    with pytest.raises(ValueError):
        P.rope_problem(P.PSV_DTYPE_F32, (1, 1, 1, 64), (64,), freqs=np.ones(31))
    with pytest.raises(ValueError):
        P.rope_problem(P.PSV_DTYPE_F32, (1, 1, 1, 64), (8,) * 5)


def cache():
    return P.cache_problem(P.PSV_DTYPE_BF16, (2, 5, 6, 64), (2, 70, 2, 64))


@pytest.mark.parametrize("match,kw", [
    ("dtype", dict(dtype=P.PSV_DTYPE_F32)), ("dtype", dict(dtype=9)), ("multiple", dict(Hq=5)), ("multiple", dict(Hkv=0)),
    ("multiple", dict(B=0)), ("multiple", dict(Hq=0)), ("dh", dict(dh=0)), ("dh", dict(dh=257)), ("Lq", dict(Lq=-1)),
    ("Lk", dict(Lk=-1)), ("Lk", dict(Lk=(1 << 28) + 1)), ("scale", dict(scale=-1.0)), ("scale", dict(scale=float("inf"))),
    ("softcap", dict(softcap=-2.0)), ("softcap", dict(softcap=float("nan"))), ("strides", dict(k_stride=(0, -8, 64))),
    ("strides", dict(q_meta_stride=-1)), ("strides", dict(k_meta_stride=(-1, 0))), ("together", dict(k_doc=A)),
    ("together", dict(q_doc=A)), ("causal", dict(prefix=A)), ("Lq", dict(Lq=(1 << 24) + 1)),
    ("2^24", dict(B=1 << 24)), ("strides", dict(v_stride=(1 << 41, 128, 64))),
])
def test_cache_refuses(match, kw):
    p = changed(cache, **kw)
    refused(match, P.psv_cache_scratch_bytes, p)
    refused(match, P.psv_cache_attention, p, A, A, A, 2 * A, 0, 3 * A, 1 << 30)
    refused(match, P.psv_cache_mass, p, A, A, A, 0, 2 * A, 3 * A, 1 << 30)


def test_cache_refuses_pointers():
    n = P.psv_cache_scratch_bytes(cache())
    assert n >= P.PSV_CACHE_SCRATCH_HEAD
    for i in (0, 1, 2, 3, 5):
        args = [A, A, A, 2 * A, 0, 3 * A, 1 << 30]
        args[i] = 0
        refused("null", P.psv_cache_attention, cache(), *args)
    refused("aligned", P.psv_cache_attention, cache(), A + 1, A, A, 2 * A, 0, 3 * A, n)
    refused("aligned", P.psv_cache_attention, cache(), A, A, A, 2 * A, A + 2, 3 * A, n)
    refused("rows overlap", P.psv_cache_attention, changed(cache, o_stride=(1920, 384, 32)), A, A, A, 2 * A, 0, 3 * A, n)
    refused("in part", P.psv_cache_mass, cache(), A, A, A, 2 * A + 4, 2 * A, 3 * A, n)
    for i in (0, 1, 2, 4, 5):
        args = [A, A, A, 0, 2 * A, 3 * A, 1 << 30]
        args[i] = 0
        refused("null", P.psv_cache_mass, cache(), *args)


def test_empty_calls_touch_nothing():
    p = changed(cache, Lq=0)
    P.psv_cache_attention(p, 0, 0, 0, 0, 0, 0, 0)
    p = changed(cache, Lk=0)
    P.psv_cache_mass(p, 0, 0, 0, 0, 0, 0, 0)


def evict():
    return P.evict_problem(P.PSV_DTYPE_BF16, (2, 50, 3, 64), 20, sinks=2, recent=8)


@pytest.mark.parametrize("match,kw", [
    ("dtype", dict(dtype=5)), ("B, Hkv", dict(B=0)), ("B, Hkv", dict(dh=0)), ("B, Hkv", dict(L=0)),
    ("budget", dict(budget=0)), ("budget", dict(budget=51)), ("sinks", dict(sinks=-1)), ("sinks", dict(recent=-1)),
    ("sinks", dict(recent=19)), ("sinks", dict(sinks=2**31 - 1)), ("strides", dict(v_stride=(-1, 192, 64))),
    ("strides", dict(k_meta_stride=(-1, 0))), ("overlap", dict(k_out_stride=(3840, 192, 32))),
    ("overlap", dict(v_out_stride=(3839, 192, 64))), ("k_doc", dict(doc_out=A)), ("lens_out", dict(k_lens=A, lens_out=A)),
    ("too many", dict(B=70000)), ("2^32", dict(L=1 << 25, budget=1 << 25, k_out_stride=(1 << 34, 192, 64),
                                              v_out_stride=(1 << 34, 192, 64))),
])
def test_evict_refuses(match, kw):
    refused(match, P.psv_cache_evict, changed(evict, **kw), A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A)


def test_evict_refuses_pointers():
    for i in range(7):
        args = [A * (k + 1) for k in range(7)]
        args[i] = 0
        refused("null", P.psv_cache_evict, evict(), *args)
    refused("aligned", P.psv_cache_evict, evict(), A + 1, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A)
    refused("overlap", P.psv_cache_evict, evict(), A, 2 * A, 3 * A, A + 64, 5 * A, 6 * A, 7 * A)
    refused("overlap", P.psv_cache_evict, evict(), A, 2 * A, 3 * A, 4 * A, 5 * A, 3 * A, 7 * A)
    refused("same buffer", P.psv_cache_evict, evict(), A, 2 * A, 3 * A, 4 * A, 4 * A, 6 * A, 7 * A)


def test_descriptions_match_the_header():
    """Field offsets of the ctypes descriptions as the C compiler lays them out."""
    import os
    import subprocess
    import tempfile

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = {"psv_rope_problem": P.RopeProblem, "psv_cache_problem": P.CacheProblem, "psv_evict_problem": P.EvictProblem}
    body = "".join(f'printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for c, s in names.items() for f, _ in s._fields_)
    body += "".join(f'printf("{c} size %zu\\n", sizeof({c}));' for c in names)
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "o.c"), os.path.join(d, "o")
        with open(src, "w") as f:
            f.write('#include <stdio.h>\n#include "psv.h"\nint main(void) {' + body + "return 0;}")
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), src, "-o", exe], check=True)
        out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    for line in out.splitlines():
        c, f, n = line.split()
        assert int(n) == (ctypes.sizeof(names[c]) if f == "size" else getattr(names[c], f).offset), line


def test_metadata_off_four_bytes_is_refused():
    """A kernel would fault on an int or a float off its alignment."""
    for name in ("q_lens", "k_lens", "q_pos", "k_pos", "prefix", "slopes"):
        p = changed(cache, causal=1, **{name: A + 2})
        refused("aligned", P.psv_cache_scratch_bytes, p)
        refused("aligned", P.psv_cache_attention, p, A, A, A, 2 * A, 0, 3 * A, 1 << 30)
        refused("aligned", P.psv_cache_mass, p, A, A, A, 0, 2 * A, 3 * A, 1 << 30)
    for kw in (dict(q_doc=A + 1, k_doc=A), dict(q_doc=A, k_doc=A + 2)):
        refused("aligned", P.psv_cache_scratch_bytes, changed(cache, **kw))
    refused("aligned", P.psv_rope, changed(rope, lens=A + 2), A, A, 2 * A)
    for name in ("k_lens", "k_pos", "pos_out", "lens_out"):
        refused("aligned", P.psv_cache_evict, changed(evict, **{name: 9 * A + 1}), *(A * k for k in range(1, 8)))
    for kw in (dict(k_doc=9 * A + 2), dict(k_doc=9 * A, doc_out=8 * A + 2)):
        refused("aligned", P.psv_cache_evict, changed(evict, **kw), *(A * k for k in range(1, 8)))


def test_evict_refuses_more_slots_than_it_can_step_over():
    """Within 1024 slots of 2^31 a 32-bit step passes the end of the numbers and never ends."""
    def make(n):
        return P.evict_problem(P.PSV_DTYPE_BF16, (1, n, 1, 1), 1)

    for n in (2**31 - 1, 2**31 - 1024, 2**30 + 1):
        refused("2^30", P.psv_cache_evict, make(n), *(k << 36 for k in range(1, 8)))


def passes_the_areas(call, *args):
    """The call gets as far as the device (which is missing, or does not hold these addresses)."""
    with pytest.raises(P.PSVError) as e:
        call(*args)
    assert "overlap" not in str(e.value) and "same buffer" not in str(e.value), str(e.value)


def test_evict_outputs_that_meet_anything_are_refused():
    k = 2 * 50 * 3 * 64 * 2  # bytes of k and of v; of k_out and v_out 15360, of mass 1200, of the lists 480
    names = ("k", "v", "mass", "k_out", "v_out", "mass_out", "idx_out")
    where = {n: A * (i + 1) for i, n in enumerate(names)}
    extra = dict(k_lens=20 * A, k_pos=21 * A, k_doc=22 * A, pos_out=23 * A, doc_out=24 * A, lens_out=25 * A)

    def call(**kw):
        at = {**where, **extra, **kw}
        return P.psv_cache_evict, changed(evict, **{n: at[n] for n in extra}), *(at[n] for n in names)

    passes_the_areas(*call())
    for out, at in (("k_out", "v"), ("v_out", "k"), ("k_out", "mass"), ("mass_out", "v"), ("idx_out", "k"), ("idx_out", "mass"),
                    ("pos_out", "k_pos"), ("doc_out", "k_doc"), ("pos_out", "mass"), ("lens_out", "k_doc"), ("mass_out", "k_lens")):
        refused("overlap", *call(**{out: {**where, **extra}[at]}))
        passes_the_areas(*call(**{out: {**where, **extra}[at] + (1 << 19)}))
    refused("overlap", *call(k_out=where["v"] + k - 2))
    passes_the_areas(*call(k_out=where["v"] + k))
    for a, b in (("v_out", "k_out"), ("mass_out", "k_out"), ("idx_out", "mass_out"), ("pos_out", "idx_out"), ("doc_out", "pos_out"),
                 ("lens_out", "doc_out")):
        refused("overlap", *call(**{a: {**where, **extra}[b] + 8}))


def test_evict_accepts_packed_buffers():
    """Keys and values side by side in one buffer, row by row or block by block."""
    H, dh, L, n = 3, 64, 50, 20
    rest = (30 * A, 31 * A)
    for st, step in (((L * H * 2 * dh, H * 2 * dh, 2 * dh), dh),      # [L][H][2][dh]
                     ((L * 2 * H * dh, 2 * H * dh, dh), H * dh),      # [L][2][H][dh]
                     ((2 * L * H * dh, H * dh, dh), L * H * dh),      # [2][L][H][dh]
                     ((2 * H * L * dh, dh, L * dh), H * L * dh)):     # [2][H][L][dh]
        p = changed(evict, k_stride=st, v_stride=st, k_out_stride=st, v_out_stride=st)
        passes_the_areas(P.psv_cache_evict, p, A, A + 2 * step, 5 * A, 3 * A, 3 * A + 2 * step, *rest)
        if step <= H * dh:  # (else k_out, of fewer rows than L, ends before)
            refused("overlap", P.psv_cache_evict, p, A, A + 2 * step, 5 * A, 3 * A, 3 * A + 2 * step - 2, *rest)
        refused("overlap", P.psv_cache_evict, p, A, A + 2 * step, 5 * A, A + 2 * step, 3 * A, *rest)
        # the same buffer's further rows
        if st[1] >= H * dh:
            long = tuple([4 * st[0], st[1], st[2]])
            p = changed(evict, k_stride=long, v_stride=long, k_out_stride=long, v_out_stride=long)
            at = A + (2 * L if step == L * H * dh else L) * st[1] * 2  # behind k's and v's rows
            passes_the_areas(P.psv_cache_evict, p, A, A + 2 * step, 5 * A, at, at + 2 * step, *rest)
            refused("overlap", P.psv_cache_evict, p, A, A + 2 * step, 5 * A, at - 2 * st[1], at + 2 * step, *rest)


def test_attention_outputs_that_meet_an_input_are_refused():
    n = 1 << 30
    passes_the_areas(P.psv_cache_attention, cache(), A, 2 * A, 3 * A, A, 0, 5 * A, n)  # in place
    refused("overlap", P.psv_cache_attention, cache(), A, 2 * A, 3 * A, A + 16, 0, 5 * A, n)
    refused("overlap", P.psv_cache_attention, changed(cache, q_stride=(5 * 400, 400, 64)), A, 2 * A, 3 * A, A, 0, 5 * A, n)
    refused("overlap", P.psv_cache_attention, cache(), A, 2 * A, 3 * A, 2 * A, 0, 5 * A, n)
    refused("overlap", P.psv_cache_attention, cache(), A, 2 * A, 3 * A, 3 * A + 35000, 0, 5 * A, n)
    passes_the_areas(P.psv_cache_attention, cache(), A, 2 * A, 3 * A, 3 * A + 35840, 0, 5 * A, n)
    for at in (A + 16, 2 * A, 3 * A + 4, 4 * A + 64):
        refused("lse overlaps", P.psv_cache_attention, cache(), A, 2 * A, 3 * A, 4 * A, at, 5 * A, n)
    # q, k, v and o of one row side by side: [B][L][6 + 2 + 2 + 6][64]
    st = (5 * 1024, 1024, 64)
    p = P.cache_problem(P.PSV_DTYPE_BF16, (2, 5, 6, 64), (2, 5, 2, 64), q_stride=st, k_stride=st, v_stride=st, o_stride=st)
    passes_the_areas(P.psv_cache_attention, p, A, A + 768, A + 1024, A + 1280, 0, 5 * A, n)
    refused("o overlaps v", P.psv_cache_attention, p, A, A + 768, A + 1024, A + 1278, 0, 5 * A, n)
    # one cache for every sequence
    p = P.cache_problem(P.PSV_DTYPE_BF16, (2, 5, 2, 64), (2, 5, 2, 64), k_stride=(0, 128, 64), v_stride=(0, 128, 64))
    passes_the_areas(P.psv_cache_attention, p, A, A + 2560, A + 3840, A + 5120, 0, 5 * A, n)
    refused("o overlaps v", P.psv_cache_attention, p, A, A + 2560, A + 3840, A + 5118, 0, 5 * A, n)


def test_mass_and_rope_outputs_that_meet_an_input_are_refused():
    n = 1 << 30
    passes_the_areas(P.psv_cache_mass, cache(), A, 2 * A, 3 * A, 4 * A, 4 * A, 5 * A, n)
    for at in (A, 2 * A, 3 * A):
        refused("mass_out overlaps", P.psv_cache_mass, cache(), A, 2 * A, 3 * A, 0, at, 5 * A, n)
    passes_the_areas(P.psv_rope, rope(), A, 2 * A, A)
    refused("out overlaps x", P.psv_rope, rope(), A, 2 * A, A + 64)
    refused("out overlaps pos", P.psv_rope, rope(), A, 2 * A, 2 * A - 512)
    st = (5 * 3 * 192, 3 * 192, 64)  # the queries of a packed projection into the place of its values
    p = changed(rope, x_stride=st, out_stride=st)
    passes_the_areas(P.psv_rope, p, A, 2 * A, A + 2 * 384)
    refused("out overlaps x", P.psv_rope, p, A, 2 * A, A + 2 * 190)


def test_areas_against_a_walk_over_all_bytes():
    """Random small layouts: what meets is refused; what does not passes where the strides agree."""
    rng = np.random.default_rng(3)
    met = 0
    for _ in range(400):
        B, L, H = (int(x) for x in rng.integers(1, 4, 3))
        dh, n = 2 * int(rng.integers(1, 3)), int(rng.integers(1, L + 1))
        order = rng.permutation(3)
        ext, st, span = (B, L, H), [0, 0, 0], dh * int(rng.integers(1, 4))
        for d in order:
            st[d] = span
            span = st[d] * ext[d] + 2 * int(rng.integers(0, 3))
        off = 2 * int(rng.integers(-span, span + 2))
        p = P.evict_problem(P.PSV_DTYPE_BF16, (B, L, H, dh), n, k_stride=st, v_stride=st, k_out_stride=st, v_out_stride=st)

        def cells(at, rows):
            return {at + b * st[0] + r * st[1] + h * st[2] + e for b in range(B) for r in range(rows) for h in range(H) for e in range(dh)}

        meets = bool(cells(0, L) & cells(off // 2, n))
        met += meets
        args = (p, A, 9 * A, 5 * A, A + off // 2 * 2, 7 * A, 30 * A, 31 * A)
        (refused if meets else passes_the_areas)(*(("k_out overlaps k",) if meets else ()), P.psv_cache_evict, *args)
    assert 50 < met < 350


def test_status_refuses():
    refused("null", P.psv_cache_status, 0)
    refused("256", P.psv_cache_status, A + 64)
    assert P.lib().psv_cache_status(A, None, None) == P.PSV_EINVAL


def test_workspace_of_shared_and_own_metadata():
    """A workspace sized for documents that the kv heads share is too small for documents of each head."""
    def size(**kw):
        return P.psv_cache_scratch_bytes(P.cache_problem(P.PSV_DTYPE_BF16, (2, 500, 8, 64), (2, 9000, 4, 64), **kw))

    docs = dict(q_doc=A, k_doc=A)
    assert size() < size(**docs, k_meta_stride=(9000, 0)) < size(**docs, k_meta_stride=(36000, 9000))


def test_in_place_with_strides_that_are_never_stepped():
    """A view's batch stride differs from a dense one's, which does not matter to a batch of one."""
    p = P.cache_problem(P.PSV_DTYPE_BF16, (1, 5, 6, 64), (1, 70, 2, 64), q_stride=(9999, 384, 64))
    passes_the_areas(P.psv_cache_attention, p, A, 2 * A, 3 * A, A, 0, 5 * A, 1 << 30)
    p = P.rope_problem(P.PSV_DTYPE_BF16, (1, 5, 3, 64), (24, 20, 20), x_stride=(7777, 192, 64))
    with pytest.raises(P.PSVError) as e:
        P.psv_rope(p, A, 2 * A, A)
    assert "strides" not in str(e.value) and "overlap" not in str(e.value)
    refused("equal strides", P.psv_rope, changed(rope, x_stride=(7777, 192, 64)), A, 2 * A, A)

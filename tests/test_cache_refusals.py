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

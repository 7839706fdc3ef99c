"""Argument checks of the paged-cache operators (psv_page_*): every refusal is made on the
host before any device call, so these run without a GPU."""
import pytest

from autoregressive_denoising_dit_gb300 import _psv as P


@pytest.fixture(scope="module", autouse=True)
def built():
    from autoregressive_denoising_dit_gb300 import build

    build.build()


A = 1 << 20  # an aligned address that no refused call may touch; the areas below are 16 MB apart
B, HKV, DH, PAGE, N, MAX = 2, 3, 64, 16, 9, 4


def at(i):
    return A + (i << 24)


def cache(form=None):
    form = P.PSV_PAGE_E4M3 if form is None else form
    scales = (at(4), at(5)) if form >= P.PSV_PAGE_E4M3 else (0, 0)
    return P.page_cache(form, (B, MAX), N, PAGE, HKV, DH, at(1), at(2), at(3), *scales)


def rows(dtype=None):
    return P.page_rows(P.PSV_DTYPE_BF16 if dtype is None else dtype, (B, 5, HKV, DH), starts=at(6), lens=at(7))


def query():
    return P.page_query(P.PSV_DTYPE_BF16, (B, 2, 6, DH), q_lens=at(6), k_lens=at(7))


def changed(p, **kw):
    for name, value in kw.items():
        setattr(p, name, type(getattr(p, name))(*value) if isinstance(value, tuple) else value)
    return p


def refused(match, call, *args):
    with pytest.raises(P.PSVError) as e:
        call(*args)
    assert e.value.code == P.PSV_EINVAL
    assert match in str(e.value), str(e.value)


def write(c=None, r=None, k=at(10), v=at(11)):
    P.psv_page_write(c or cache(), r or rows(), k, v)


def read(c=None, r=None, k=at(10), v=at(11)):
    P.psv_page_read(c or cache(), r or rows(), k, v)


def attend(c=None, q=None, x=at(10), o=at(11), lse=at(12), scratch=at(13), n=1 << 23):
    P.psv_page_attention(c or cache(), q or query(), x, o, lse, scratch, n)


@pytest.mark.parametrize("call", [write, read, attend])
@pytest.mark.parametrize("match,kw", [
    ("format", dict(format=0)), ("format", dict(format=5)), ("B of 1", dict(B=0)), ("B of 1", dict(B=65536)),
    ("B of 1", dict(Hkv=0)), ("dh", dict(dh=0)), ("dh", dict(dh=257)), ("n_pages", dict(n_pages=0)),
    ("n_pages", dict(page_size=0)), ("n_pages", dict(max_pages=0)), ("n_pages", dict(max_pages=-1)),
    ("2^30", dict(max_pages=(1 << 26) + 1)), ("2^30", dict(page_size=1 << 29)), ("2^24", dict(Hkv=1 << 24)),
    ("strides", dict(k_stride=(-1, 64, 1024))), ("strides", dict(v_stride=(3072, 64, (1 << 40) + 1))),
    ("strides", dict(scale_stride=(48, -1, 16))), ("strides", dict(table_stride=-1)),
    ("2^56", dict(k_stride=(1 << 40, 64, 1024), n_pages=1 << 20)), ("null", dict(k_pages=0)), ("null", dict(v_pages=0)),
    ("null", dict(table=0)), ("null", dict(k_scales=0)), ("null", dict(v_scales=0)), ("aligned", dict(table=at(1) + 2)),
    ("aligned", dict(k_scales=at(4) + 1)),
])
def test_caches_refused(call, match, kw):
    refused(match, call, changed(cache(), **kw))


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("match,kw", [
    ("dtype", dict(dtype=7)), ("L -1", dict(L=-1)), ("2^30", dict(L=(1 << 30) // 3 + 1)),
    ("strides", dict(k_stride=(960, -192, 64))), ("strides", dict(v_stride=(1 << 41, 192, 64))),
    ("2^56", dict(k_stride=(1 << 40, 1 << 40, 64), L=1 << 17)), ("aligned", dict(starts=at(6) + 1)),
    ("aligned", dict(lens=at(7) + 3)),
])
def test_rows_refused(call, match, kw):
    refused(match, call, None, changed(rows(), **kw))


def test_writes_and_reads_refused():
    for call in (write, read):
        refused("null", call, None, None, 0)
        refused("null", call, None, None, at(10), 0)
        refused("aligned", call, None, None, at(10) + 1)
        refused("aligned", call, None, rows(P.PSV_DTYPE_F32), at(10) + 2)
        refused("type", call, cache(P.PSV_PAGE_F16))                      # bf16 rows
        refused("type", call, cache(P.PSV_PAGE_BF16), rows(P.PSV_DTYPE_F16))
        refused("aligned", call, changed(cache(P.PSV_PAGE_BF16), k_pages=at(2) + 1))
        call(None, changed(rows(), L=0))                                   # nothing to do
    # pages whose rows overlap may be read, not written
    refused("rows overlap", write, changed(cache(), k_stride=(3072, 32, 1024)))
    refused("rows overlap", write, changed(cache(), scale_stride=(48, 0, 16)))
    refused("rows of k or v overlap", read, None, changed(rows(), k_stride=(960, 0, 64)))
    refused("rows of k or v overlap", read, None, changed(rows(), v_stride=(960, 192, 60)))
    # outputs that meet inputs or one another
    refused("k_pages overlaps k", write, None, None, at(2) + 64)
    refused("v_pages overlaps k_pages", write, changed(cache(), v_pages=at(2) + 128))
    refused("v_scales overlaps k_scales", write, changed(cache(), v_scales=at(4)))
    refused("k_scales overlaps table", write, changed(cache(), k_scales=at(1)))
    refused("k_pages overlaps starts", write, changed(cache(), k_pages=at(6) - 16))
    refused("k overlaps k_pages", read, None, None, at(2))
    refused("v overlaps k", read, None, None, at(10), at(10) + 640)
    refused("v overlaps v_scales", read, None, None, at(10), at(5))
    refused("k overlaps table", read, None, None, at(1))
    refused("k overlaps lens", read, None, None, at(7))


@pytest.mark.parametrize("match,kw", [
    ("dtype", dict(dtype=P.PSV_DTYPE_F32)), ("dtype", dict(dtype=9)), ("multiple", dict(Hq=4)), ("multiple", dict(Hq=0)),
    ("Lq", dict(Lq=-1)), ("Lq", dict(Lq=(1 << 20) + 1)), ("2^24", dict(Hq=3 << 23)), ("2^30", dict(Lq=1 << 20, Hq=516)),
    ("negative", dict(window=-1)), ("negative", dict(window=4, sinks=-1)), ("sinks need", dict(sinks=3)),
    ("scale", dict(scale=-1.0)), ("scale", dict(scale=float("nan"))), ("softcap", dict(softcap=float("inf"))),
    ("softcap", dict(softcap=-2.0)), ("strides", dict(q_stride=(-8, 384, 64))), ("strides", dict(o_stride=(768, 384, 1 << 41))),
    ("o's rows overlap", dict(o_stride=(768, 384, 32))), ("o's rows overlap", dict(o_stride=(0, 384, 64))),
    ("aligned", dict(q_lens=at(6) + 2)), ("aligned", dict(k_lens=at(7) + 1)),
    ("2^56", dict(q_stride=(1 << 40, 1 << 40, 64), Lq=1 << 16)),
])
def test_queries_refused(match, kw):
    refused(match, attend, None, changed(query(), **kw))


def test_attention_refused():
    refused("null", attend, None, None, 0)
    refused("null", attend, None, None, at(10), 0)
    refused("null", attend, None, None, at(10), at(11), at(12), 0)
    refused("aligned", attend, None, None, at(10) + 1)
    refused("aligned", attend, None, None, at(10), at(11), at(12) + 2)
    refused("256-byte", attend, None, None, at(10), at(11), at(12), at(13) + 128)
    refused("scratch of", attend, None, None, at(10), at(11), at(12), at(13), 100)
    refused("type", attend, cache(P.PSV_PAGE_F16))
    refused("type", attend, cache(P.PSV_PAGE_BF16), changed(query(), dtype=P.PSV_DTYPE_F16))
    attend(None, changed(query(), Lq=0))
    refused("o overlaps q", attend, None, None, at(10), at(10) + 128)
    refused("o overlaps q", attend, None, changed(query(), o_stride=(1024, 512, 64)), at(10), at(10))
    refused("o overlaps k_pages", attend, None, None, at(10), at(2))
    refused("o overlaps v_scales", attend, None, None, at(10), at(5))
    refused("o overlaps table", attend, None, None, at(10), at(1))
    refused("lse overlaps o", attend, None, None, at(10), at(11), at(11))
    refused("lse overlaps k_lens", attend, None, None, at(10), at(11), at(7))
    refused("scratch overlaps q", attend, None, None, at(10), at(11), at(12), at(10))
    refused("scratch overlaps k_pages", attend, None, None, at(10), at(11), at(12), at(2))
    n = P.psv_page_scratch_bytes(cache(), query())
    assert 0 < n <= 6 << 20
    refused("scratch of", attend, None, None, at(10), at(11), at(12), at(13), n - 1)


def test_workspaces_of_every_problem_are_small():
    for dh in (1, 20, 64, 128, 256):
        for dtype, form in ((P.PSV_DTYPE_BF16, P.PSV_PAGE_BF16), (P.PSV_DTYPE_F16, P.PSV_PAGE_I8)):
            for heads in (3, 24, 96):
                c = P.page_cache(form, (B, MAX), N, PAGE, HKV, dh, at(1), at(2), at(3), at(4), at(5))
                n = P.psv_page_scratch_bytes(c, P.page_query(dtype, (B, 2, heads, dh)))
                assert 0 < n <= 6 << 20


def test_descriptions_refuse_what_they_cannot_hold():
    with pytest.raises(ValueError):
        P.page_rows(P.PSV_DTYPE_BF16, (1, 2, 3))
    c = cache()
    assert tuple(c.k_stride) == (HKV * PAGE * DH, DH, PAGE * DH) and tuple(c.scale_stride) == (HKV * PAGE, 1, PAGE)
    assert c.table_stride == MAX

"""Values that are not finite behind the masks of the attention over pages, row by row: each
bad position has a column (16-bit pages) or a kv head (8-bit pages) of its own, so that every
row that does not see it is held to the definition, and every row that does shows it.  (All
rows see one of the bad positions: in one head's one column they would hide one another.)"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from test_gpu_page_ops import DT, attention_case, reference, run_attention  # noqa: E402


@pytest.fixture(scope="module")
def P():
    from autoregressive_denoising_dit_gb300 import _psv

    return _psv


WIDE = 4096  # table entries: groups are cut
NAN = float("nan")

# rows, keys and masks; the modes: clusters and cuts (width), a warp a group (many sequences)
CASES = [
    dict(B=1, Lq=6, Lk=200, Hq=8, Hkv=4, dh=128, page=32, causal=True, window=60, sinks=3),
    dict(B=1, Lq=6, Lk=200, Hq=4, Hkv=4, dh=64, page=16, causal=True, window=60, sinks=3),
    dict(B=1, Lq=6, Lk=200, Hq=8, Hkv=4, dh=80, page=7, causal=True, window=60, sinks=3),
    dict(B=1, Lq=6, Lk=200, Hq=8, Hkv=4, dh=72, page=24, causal=True, window=60, sinks=3),
    dict(B=1, Lq=6, Lk=200, Hq=4, Hkv=4, dh=256, page=64, causal=True, window=60, sinks=3),
    dict(B=1, Lq=6, Lk=200, Hq=24, Hkv=4, dh=128, page=64, causal=True, window=60, sinks=3),   # 36 rows
    dict(B=1, Lq=6, Lk=200, Hq=40, Hkv=4, dh=128, page=64, causal=True, window=100000, sinks=3),  # 60 rows, 32 at a time
    dict(B=300, Lq=6, Lk=200, Hq=4, Hkv=4, dh=128, page=16, causal=True, window=60, sinks=3),
    dict(B=300, Lq=6, Lk=200, Hq=8, Hkv=4, dh=64, page=8, causal=True, window=60, sinks=3),
    dict(B=1, Lq=6, Lk=200, Hq=8, Hkv=4, dh=100, page=16, causal=True, window=60, sinks=3),    # general kernel
    dict(B=1, Lq=6, Lk=200, Hq=8, Hkv=4, dh=128, page=32, window=60, sinks=3),                 # later keys are seen
]
# Rows stand at 194 to 199.  197: a later draft; 136: out of the window of row 196 and on; 137:
# of row 197 and on; 100: no row sees it.
BAD = [197, 136, 137, 100]


def sees(c, j, row):
    p = 194 + row
    return (not c.get("causal") or j <= p) and (j > p - c["window"] or j < c["sinks"])


@pytest.mark.parametrize("what,dtype,f", [("value", "bf16", "bf16"), ("value", "f16", "f16"), ("scale", "bf16", "e4m3"),
                                          ("scale", "f16", "i8"), ("code", "bf16", "e4m3")])
@pytest.mark.parametrize("width", [0, WIDE])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"B{c['B']}H{c['Hq']}-{c['Hkv']}dh{c['dh']}" + ("" if c.get("causal") else "all"))
def test_a_bad_value_reaches_the_rows_that_see_it_only(P, case, dtype, f, width, what):
    c = case
    cache, q, (k, v), lens, total, rows = attention_case(P, c, dtype, f, width=width)
    ref = reference(cache, c, q, k, v, total, rows)  # (without the bad ones, which are finite there)
    hit = torch.zeros(c["Lq"], c["Hq"], c["dh"], dtype=torch.bool, device="cuda")
    free = torch.zeros_like(hit)  # columns beside a code that is NaN, in rows that see it
    G = c["Hq"] // c["Hkv"]
    for i, j in enumerate(BAD):
        e, r = cache.table[:, j // c["page"]].long(), j % c["page"]  # of all sequences
        seen = [x for x in range(c["Lq"]) if sees(c, j, x)]
        if what == "value":
            cache.v[e, 1, r, 5 + 9 * i] = NAN if i % 2 else float("-inf")
            hit[seen, G:2 * G, 5 + 9 * i] = True
        elif what == "code":
            cache.v[e, i, r, 5 + 9 * i] = 0xFF if i % 2 else 0x7F
            hit[seen, i * G:(i + 1) * G, 5 + 9 * i] = True
            free[seen, i * G:(i + 1) * G] = True
        else:
            cache.v[e, i, r] = 0
            cache.vs[e, i, r] = NAN
            hit[seen, i * G:(i + 1) * G] = True
    o, lse = run_attention(P, c, cache, q, lens, rows, dtype)
    for b in range(c["B"]):
        want, tol, want_lse, ltol = ref[b]
        assert not torch.isfinite(o[b].float())[hit].any()
        assert ((o[b].double() - want).abs() <= tol)[~(hit | free)].all()
        assert ((lse[b].T.double() - want_lse).abs() <= ltol).all()


@pytest.mark.parametrize("dtype,f", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "i8")])
@pytest.mark.parametrize("width", [0, WIDE])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"B{c['B']}H{c['Hq']}-{c['Hkv']}dh{c['dh']}" + ("" if c.get("causal") else "all"))
def test_a_bad_key_reaches_the_rows_that_see_it_only(P, case, dtype, f, width):
    c = case
    cache, q, (k, v), lens, total, rows = attention_case(P, c, dtype, f, width=width)
    ref = reference(cache, c, q, k, v, total, rows)
    hit = torch.zeros(c["Lq"], c["Hq"], dtype=torch.bool, device="cuda")
    G = c["Hq"] // c["Hkv"]
    for i, j in enumerate(BAD):
        e, r = cache.table[:, j // c["page"]].long(), j % c["page"]
        if f in DT:
            cache.k[e, i, r, 3] = NAN
        elif i % 2 or f == "i8":
            cache.ks[e, i, r] = NAN
        else:
            cache.k[e, i, r, 3] = 0x7F
        hit[[x for x in range(c["Lq"]) if sees(c, j, x)], i * G:(i + 1) * G] = True
    o, lse = run_attention(P, c, cache, q, lens, rows, dtype)
    for b in range(c["B"]):
        want, tol, want_lse, ltol = ref[b]
        assert torch.isnan(o[b].float())[hit].all() and torch.isnan(lse[b].T[hit]).all()
        assert ((o[b].double() - want).abs() <= tol)[~hit].all()
        assert ((lse[b].T.double() - want_lse).abs() <= ltol)[~hit].all()

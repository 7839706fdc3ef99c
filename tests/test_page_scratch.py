"""What the header says of the paged attention's workspace, without a GPU: a program may set
aside the most that it names, once, for all its calls."""
import os
import re

import pytest

from autoregressive_denoising_dit_gb300 import _psv as P

A = 1 << 20  # an aligned address that no call here touches


@pytest.fixture(scope="module", autouse=True)
def built():
    from autoregressive_denoising_dit_gb300 import build

    build.build()


def scratch(form, dh, Lq, G, B=2, max_pages=4):
    scales = (A + (4 << 24), A + (5 << 24)) if form >= P.PSV_PAGE_E4M3 else (0, 0)
    cache = P.page_cache(form, (B, max_pages), 9, 16, 3, dh, A, A + (2 << 24), A + (3 << 24), *scales)
    dtype = P.PSV_DTYPE_F16 if form == P.PSV_PAGE_F16 else P.PSV_DTYPE_BF16
    return P.psv_page_scratch_bytes(cache, P.page_query(dtype, (B, Lq, 3 * G, dh)))


def test_the_workspace_is_no_larger_than_the_header_says():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "psv.h")
    with open(path) as f:
        most = float(re.search(r"overlap on the GPU\.\s+([\d.]+) MB", f.read()).group(1)) * 1e6
    sizes = [scratch(form, dh, Lq, G, B, n) for form in (P.PSV_PAGE_BF16, P.PSV_PAGE_F16, P.PSV_PAGE_E4M3, P.PSV_PAGE_I8)
             for dh in (8, 64, 72, 100, 128, 136, 256) for Lq, G in ((1, 1), (1, 8), (3, 3), (4, 16), (1000, 5))
             for B, n in ((1, 1), (64, 5000), (5000, 300))]
    assert max(sizes) <= most
    assert most < 1.05 * max(sizes)

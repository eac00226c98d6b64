"""fa_evict_paged refuses new weights that overlap the weights it reads (CPU only: refusals come before any CUDA call)."""

import pytest

from test_paged_fp4_host import INVALID, P, _evict, fa  # noqa: F401


@pytest.mark.parametrize("kw", [
    dict(nw=P + 4), dict(nw=P + 4 * 999),                                     # other columns that rows of 1000 do not leave free
    dict(nw=P + 4 * 3000), dict(nw=P - 4 * 3 * 128), dict(nw=P - 4 * 100),    # the last row, the first
    dict(ws=1200, nws=1200, nw=P + 4 * 999), dict(ws=1200, nws=1200, nw=P + 4 * 1100), dict(ws=1100, nws=1100, nw=P + 4 * 1000),
    dict(ws=1200, nws=1200, nw=P - 4 * 1100),
    dict(B=1, Hkv=1, nw=P + 4 * 500), dict(B=1, Hkv=1, nw=P - 4 * 127),
], ids=str)
def test_overlap_is_refused(fa, kw):  # noqa: F811
    assert _evict(fa, **kw) == INVALID
    assert b"overlaps" in fa.lib.fa_last_error_detail()

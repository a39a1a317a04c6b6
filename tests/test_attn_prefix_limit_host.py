"""The stated limit of wsw_attn_paged_prefix's list of tiles, on the host: kv heads * (requests * group / 128 + groups) *
(max_pages * page_size / 16 + 9) < 2^31 - 65536, for tables that do not end on a tile of 64 positions, too."""
import ctypes

import pytest

from test_kv_share_host import UNSUPPORTED, WORKSPACE, _attend, _cache, lib  # noqa: F401


@pytest.mark.parametrize("page,width", [(16, 1), (1, 1), (1, 17), (16, 3), (16, 4), (1, 65), (16, 5), (64, 1), (64, 100), (1, 6401)])
@pytest.mark.parametrize("requests,group", [(1, 1), (300, 5)])
def test_the_limit_is_the_stated_one(lib, page, width, requests, group):  # noqa: F811
    groups = 16384
    each = (requests * group // 128 + groups) * (page * width // 16 + 9)
    heads = ((1 << 31) - 65536 - 1) // each
    for h, want in ((heads, WORKSPACE), (heads + 1, UNSUPPORTED)):
        c = _cache(heads=h, page_size=page, head_stride=64, pos_stride=64 * h, page_stride=64 * h * page)
        assert _attend(lib, requests=requests, q_heads=h * group, cache=ctypes.byref(c), width=width, stride=width, groups=groups,
                       ws_bytes=0) == want, (h, want)

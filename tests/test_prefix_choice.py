"""Which calls read shared prefixes apart, and how much room the image of a prefix takes: the kernels' own rule on the CPU."""
import pytest

import prefix_util as u

ORDINARY = dict(tokens=128, heads=64, requests=128, groups=1, dim=512, v_dim=512, bits8=0, pages=20000, page=64, width=80)


def call(**change):
    return list({**ORDINARY, **change}.values())


def test_by_size_and_width():
    assert u.apart(*call())
    assert not u.apart(*call(tokens=5, requests=5, heads=16, width=36))       # few requests
    assert not u.apart(*call(groups=0)) and not u.apart(*call(tokens=1, requests=1, heads=4096))
    for dim, v_dim in ((64, 64), (192, 192), (576, 576), (640, 512), (520, 512), (512, 448)):
        assert not u.apart(*call(dim=dim, v_dim=v_dim)), (dim, v_dim)
    for dim, v_dim in ((576, 512), (512, 128), (448, 256), (384, 384)):
        assert u.apart(*call(dim=dim, v_dim=v_dim)), (dim, v_dim)
    assert not u.apart(*call(tokens=40000))                                    # parts of more than 4 GiB
    # 24 tiles of 64 query rows x 64 rows an SM, 64 for narrow rows, with an image or with few requests a group
    least = -(-24 * 152 // 128)
    assert u.apart(*call(width=least)) and not u.apart(*call(width=least - 1))
    for change in (dict(dim=192, v_dim=128), dict(bits8=1), dict(page=60), dict(groups=17)):
        rows = 64 * 152 // 128 * 64
        page = change.get("page", 64)
        assert u.apart(*call(width=-(-rows // page), **change)) and not u.apart(*call(width=rows // page - 2, **change)), change


@pytest.mark.parametrize("groups", [1, 3, 100, 14000])
@pytest.mark.parametrize("page", [50, 64])
def test_image_goes_by_the_cache_and_not_by_what_a_table_could_list(groups, page):
    # 8-bit rows behind tables with room for a million rows: a small cache needs a small image
    for pages in (1, 7, 300, 100000):
        rows = u.image_rows(*call(groups=groups, requests=14000, bits8=1, pages=pages, page=page, width=1 << 14))
        assert rows % 128 == 0 and rows <= -(-pages * page // 128) * 128 and rows * groups * 512 * 2 <= 1 << 30
        assert rows == min(-(-min(pages, 1 << 14) * page // 128) * 128, (1 << 30) // (groups * 1024) // 128 * 128)
    assert u.image_rows(*call(groups=groups, bits8=0, page=64)) == 0
    assert u.image_rows(*call(groups=groups, bits8=0, page=50)) == (0 if groups == 14000 else min(-(-20000 * 50 // 128), -(-80 * 50 // 128), (1 << 30) // (groups * 1024) // 128) * 128)

"""shared_attention's two ways: the sizes at which test_gpu_shared.py means the kernels for prefixes reach them, and what only those
kernels have to see to (tables that end before their requests do, prefixes longer than their image) at sizes that reach them."""
import pytest
import torch

import prefix_util
import sparse_attention_kv_csa_gb300 as csa
import test_gpu_shared as shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,v_dim", [(512, 512), (576, 512), (256, 256), (192, 128), (128, 128), (384, 384), (448, 256)])
@pytest.mark.parametrize("bits8", [False, True])
def test_the_prefix_tests_sizes(dim, v_dim, bits8):
    assert prefix_util.read_apart(shared.made(shared.TWO, 24, dim, 3, 16, bits8), v_dim)
    assert not prefix_util.read_apart(shared.made(shared.TWO, 24, dim, 3, 16, bits8, width=0), v_dim)


@pytest.mark.parametrize("page", [1, 3, 8, 50, 64, 256])
def test_the_page_tests_sizes(page):
    for bits8 in (False, True):
        assert prefix_util.read_apart(shared.made(shared.ONE, 32, 128, 1, page, bits8))


@pytest.mark.parametrize("dim,bits8", [(256, False), (512, False), (128, False), (256, True)])
def test_tables_narrower_than_the_rows(dim, bits8):
    # 32 pages of 16 rows (the first group's requests have up to 506 rows), then 31: the rows past a table's end are nobody's,
    # and a request that has such rows shares nothing
    a = shared.made([(400, [(100 + k % 7, 1) for k in range(1400)]), (300, [(k % 9, 1) for k in range(40)])], 8, dim, 1, 16, bits8, seed=23, width=0)
    assert a["block_table"].shape[1] == 32
    for b in (a, dict(a, block_table=a["block_table"][:, :31].contiguous()), dict(a, block_table=a["block_table"][:, :27].contiguous())):
        assert prefix_util.read_apart(b)
        shared.check(b)


@pytest.mark.parametrize("page", [64, 50])
@pytest.mark.parametrize("bits8", [False, True])
def test_a_prefix_that_lists_pages_twice(page, bits8):
    # its image has room for the cache's rows once; those behind are read by request
    a = shared.made([(300, [(40, 1), (9, 2), (0, 1)])], 32, 512, 1, page, bits8, True, seed=24)
    whole = 300 // page
    wide = torch.full((3, 5000), -1, dtype=torch.int32, device="cuda")
    for k in range(5):
        wide[:, k * whole:(k + 1) * whole] = a["block_table"][:, :whole]
    wide[:, 5 * whole:5 * whole + 3] = a["block_table"][:, whole:whole + 3]
    a["block_table"] = wide
    a["seq_lens"] = a["seq_lens"] + 4 * whole * page
    a["shared_rows"] = torch.tensor([5 * whole * page], dtype=torch.int32, device="cuda")
    assert prefix_util.read_apart(a)
    shared.check(a)


def test_prefixes_of_tables_far_wider_than_the_cache():
    # 8-bit rows, room for 900000 rows a table
    a = shared.made([(400, [(30, 1), (0, 1), (77, 2)]), (200, [(3, 1), (90, 1)])], 16, 512, 1, 64, True, True, seed=25, width=14000)
    assert prefix_util.read_apart(a)
    rows = prefix_util.image_rows(a["q"].shape[0], 16, 5, 2, 512, 512, True, *a["cache"].shape[:2], 14000)
    assert 400 <= rows <= a["cache"].shape[0] * 64 + 127
    shared.check(a)
    assert csa.csa_device_status() == 0

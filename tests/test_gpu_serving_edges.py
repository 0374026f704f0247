"""The serving operators where they are most likely to go wrong: totals and offsets past 32 bits, the kernels that only large
calls reach, values that are not finite, calls in place.  Each test ends with the device's status word clear."""
import pytest
import torch

import serving_util as u
import sparse_attention_kv_csa_gb300 as csa

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def status_stays_clear():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_status() == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n", [2, 3, 5, 33, 600])
def test_page_totals_past_31_bits_are_held(n):
    most = 2 ** 31 - 1
    free = i32([11, 12, 13, 14, 15, 16, 17, 18])
    table, cu, slots, counts = csa.page_tables(i32([0] * n), i32([most] * n), 1, 1, free, i32([[-1] * 4] * n), 6)
    assert table.tolist() == [[11, 12, 13, 14]] + [[-1] * 4] * (n - 1)
    assert cu.tolist() == [0] + [most] * n
    assert slots.tolist() == [11, 12, 13, 14, -1, -1]
    assert counts.tolist() == [most, 8, most - 8, most]
    # the totals pass 2^31 only with the last requests: those before are served as ever
    before, after = [0] * (n - 1) + [0], [1] * (n - 1) + [most]
    ids = i32(list(range(1000, 1000 + n + 3)))
    table, cu, slots, counts = csa.page_tables(i32(before), i32(after), 1, 1, ids, i32([[-1] * 4] * n), n + 5)
    want = [[1000 + r, -1, -1, -1] for r in range(n - 1)] + [[1000 + n - 1 + c for c in range(4)]]
    assert table.tolist() == want and cu.tolist() == list(range(n)) + [most]
    assert slots.tolist() == [1000 + i for i in range(n + 3)] + [-1, -1]
    assert counts.tolist() == [most, n + 3, most - n - 3, most]

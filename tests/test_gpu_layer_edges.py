"""The operators around attention at the ends of what their calls allow."""

import pytest
import torch

from exact_io_aware_82_b200 import attn as A
from exact_io_aware_82_b200 import build as Bld

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    Bld.build()
    A.lib()
    yield
    assert A.attn_get_device_error() == 0


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("free", [3, 1])
def test_page_update_with_the_largest_token_count(free):
    # slots and positions of 2^31 - 1 tokens (17 GB), all but a few behind the last token; enough pages, and too few
    most = 2 ** 31 - 1
    slots, positions = (torch.full((most,), 7, dtype=torch.int32, device="cuda") for _ in range(2))
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    table[1, 0] = 5
    pool = torch.tensor([4, 2, 0, -1, -1, -1], dtype=torch.int32, device="cuda")
    ring = torch.tensor([0, free, 0], device="cuda")
    out = A.attn_page_update(table, i32(0, 3, 0), i32(17, 5, 0), pool, ring, 16, most, slots=slots, positions=positions)
    torch.cuda.synchronize()
    if free == 3:
        want_s = [4 * 16 + i for i in range(16)] + [2 * 16, 5 * 16 + 3, 5 * 16 + 4]
        want_p = list(range(17)) + [3, 4]
        assert out[0].tolist() == [2, 3, 0] and out[1].tolist() == [0, 17, 19, 19]
    else:
        want_s, want_p = [], []
        assert out[0].tolist() == [0, 1, 1] and out[1].tolist() == [0, 0, 0, 0]
    n = len(want_s)
    assert slots[:n].tolist() == want_s and positions[:n].tolist() == want_p
    for t, fill in ((slots, -1), (positions, 0)):
        assert all(bool((x == fill).all()) for x in t[n:].split(1 << 28))


@pytest.mark.parametrize("bad", [-1, 6, 1 << 30])
@pytest.mark.parametrize("new", [0, 3])
def test_a_page_outside_the_pool_is_flagged_when_it_is_returned(bad, new):
    # request 1 ends or shrinks; its second page has a number that the pool of six does not have
    table = torch.tensor([[1, 2, -1, -1], [3, bad, -1, -1]], dtype=torch.int32, device="cuda")
    pool = torch.tensor([0, 4, 5, -7, -7, -7], dtype=torch.int32, device="cuda")
    ring = torch.tensor([0, 3, 0], device="cuda")
    out = A.attn_page_update(table, i32(20, 20), i32(20, new), pool, ring, 16, 4)
    assert A.attn_get_device_error() == A.ATTN_ERR_INVALID_ARG
    back = [bad] if new else [3, bad]
    assert out[0].tolist() == [0, 3 + len(back), 0] and pool.tolist() == [0, 4, 5] + back + [-7] * (3 - len(back))
    # an entry behind the last page that is kept is nobody's: it is not looked at
    table = torch.tensor([[1, 2, bad, bad], [3, 0, bad, -1]], dtype=torch.int32, device="cuda")
    A.attn_page_update(table, i32(20, 20), i32(20, new), pool, ring, 16, 4)
    assert A.attn_get_device_error() == 0


def test_a_page_outside_the_pool_is_flagged_when_it_is_taken():
    table = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    pool, ring = i32(0, 9, 2), torch.tensor([0, 3, 0], device="cuda")
    out = A.attn_page_update(table, i32(0), i32(17), pool, ring, 16, 20)
    assert A.attn_get_device_error() == A.ATTN_ERR_INVALID_ARG
    assert out[2].tolist() == list(range(16)) + [-1] * 4

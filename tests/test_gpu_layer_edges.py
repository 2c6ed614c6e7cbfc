"""The operators around attention at the ends of what their calls allow."""

import math
import threading

import numpy as np
import pytest
import torch

from exact_io_aware_82_b200 import attn as A
from exact_io_aware_82_b200 import build as Bld

from . import _layer as R

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


@pytest.mark.parametrize("B,starts,plens", [
    (65535, [3, 40000, 65000, 65001], [300, 129, 77]),     # the most sequences that a call takes
    (4000, list(range(4001)), [1 + g % 40 for g in range(4000)]),  # a prefix to every sequence
])
def test_shared_prefix_decode_with_many_sequences(B, starts, plens):
    Hq, Hkv, page, width = 8, 1, 8, 5
    g = torch.Generator(device="cuda")
    g.manual_seed(B)
    need = [-(-n // page) for n in plens]
    own_pages = B * width
    pages = own_pages + sum(need)
    kc, vc = (torch.randn(pages, page, Hkv, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, Hq, 1, 128, generator=g, device="cuda").bfloat16()
    order = torch.randperm(pages, generator=g, device="cuda").int()
    own = order[:own_pages].view(B, width)
    lens = torch.randint(0, page * width + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    prefix = torch.full((len(plens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = own_pages
    for i, n in enumerate(need):
        prefix[i, :n] = order[at:at + n]
        at += n
    o, lse = A.attn_decode_shared_prefix(q, kc, vc, prefix, i32(*plens), i32(*starts), own, lens, max(plens), page * width)
    torch.cuda.synchronize()
    assert A.attn_get_device_error() == 0

    def rows(cache, table, n):
        return cache[table[: -(-n // page)].long()].reshape(-1, Hkv, 128)[:n]

    rng = np.random.default_rng(B)
    for b in sorted(set([0, 2, 3, B - 1] + [x for x in starts if x < B] + rng.integers(0, B, 60).tolist())):
        i = int(np.searchsorted(starts, b, side="right")) - 1
        inside = 0 <= i < len(plens)
        k, v = (R.f64(torch.cat(([rows(c, prefix[i], plens[i])] if inside else []) + [rows(c, own[b], int(lens[b]))]))
                for c in (kc, vc))
        R.assert_decode(o[b, :, 0], lse[b], R.decode_reference(R.f64(q[b, :, 0]), k, v, 1 / math.sqrt(128)), "sequence %d" % b)


def test_calls_from_two_threads_on_two_streams():
    # both threads make every call at once, each on a stream of its own, and get what one alone gets
    N, Hq, Hkv = 300, 8, 2
    g = torch.Generator()
    g.manual_seed(1)
    bf = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v = bf(N, Hq, 128), bf(N, Hkv, 128), bf(N, Hkv, 128)
    w, rope = bf(128), R.rope_table(512, 128).cuda()
    dq, dk = bf(N, Hq, 128), bf(N, Hkv, 128)
    pages = 40
    new, prefix = i32(100, 57, 143), i32(7, 3)

    def step(stream):
        table = torch.full((3, 12), -1, dtype=torch.int32, device="cuda")
        pool = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda")
        kc, vc = (torch.zeros(pages, 16, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ring, cu, slots, pos = A.attn_page_update(table, i32(0, 0, 0), new, pool, torch.tensor([0, pages, 0], device="cuda"),
                                                  16, N, stream=stream)
        zq = A.attn_qk_norm_rope_paged(q, k, v, w, w, rope, pos, slots, kc, vc, stream=stream)
        grads = A.attn_qk_norm_rope_bwd(q, k, dq, dk, w, w, rope, pos, stream=stream)
        last = zq[cu[1:].long() - 1].unsqueeze(2)
        o = A.attn_decode_shared_prefix(last, kc, vc, prefix[None], i32(20), i32(0, 2), table, new, 20, 143, stream=stream)
        return (ring, cu, slots, pos, zq, kc, vc) + tuple(grads) + tuple(o)

    want = step(None)
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got[i] = [step(s) for _ in range(20)]
            s.synchronize()
        except Exception as e:  # noqa: BLE001  (reported by the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for runs in got.values():
        for out in runs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)

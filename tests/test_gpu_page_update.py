"""Page bookkeeping against a request-by-request reference: decode steps, prompts, ended and shrinking
requests, all page sizes, wrapped rings, no requests, no tokens; a pool that is short and arguments
that are not valid change nothing; a long run of steps keeps every page in one place."""

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


def make(rng, old, page, width, spare, wrap=0):
    had = [-(-n // page) for n in old]
    total = sum(had) + spare
    order = rng.permutation(total).astype(np.int32)
    table = np.full((len(old), width), -7, dtype=np.int32)
    at = 0
    for b, n in enumerate(had):
        table[b, :n] = order[at:at + n]
        at += n
    head = wrap
    free = np.full(total, -9, dtype=np.int32)
    for i in range(spare):
        free[(head + i) % total] = order[at + i]
    return table, free, np.array([head, head + spare, 123], dtype=np.int64)


def check(table, old, new, free, ring, page, max_tokens, offset=None):
    want = R.page_update(table, old, new, free, ring, page, max_tokens, offset)
    cu = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt).cuda()  # noqa: E731
    t, f = cu(table).reshape(table.shape), cu(free)
    got = A.attn_page_update(t, cu(old), cu(new), f, cu(ring, torch.int64), page, max_tokens,
                             pos_offset=None if offset is None else cu(offset))
    torch.cuda.synchronize()
    for a, b, name in zip((t, f) + tuple(got), want, ("table", "free", "ring", "cu_seqlens", "slots", "positions")):
        assert np.array_equal(a.cpu().numpy(), b), name
    return want


@pytest.mark.parametrize("B,page,wrap", [(1, 8, 0), (3, 16, 5), (64, 16, 10 ** 12), (513, 32, 77), (2049, 64, 1)])
def test_mixed_requests(B, page, wrap):
    rng = np.random.default_rng(B)
    longest = 40 * page
    old = rng.integers(0, longest, B)
    new = np.where(rng.random(B) < 0.5, old + 1, rng.integers(0, longest, B))
    new[rng.random(B) < 0.1] = 0
    old[rng.random(B) < 0.2] = 0
    grow = int(sum(max(-(-int(n) // page) - -(-int(a) // page), 0) for a, n in zip(old, new)))
    tokens = int(np.maximum(new - old, 0).sum())
    table, free, ring = make(rng, old.tolist(), page, 41, grow + 3, wrap)
    offset = rng.integers(0, 10000, B)
    check(table, old, new, free, ring, page, tokens + 11, offset)
    # exactly enough pages and tokens
    table, free, ring = make(rng, old.tolist(), page, 41, grow, wrap)
    check(table, old, new, free, ring, page, tokens)


@pytest.mark.parametrize("old,new", [([], []), ([0], [0]), ([0], [1]), ([1], [0]), ([16], [17]), ([17], [16]),
                                     ([16, 0, 32], [16, 0, 32]), ([0, 0, 0], [48, 0, 1])])
def test_small(old, new):
    rng = np.random.default_rng(0)
    table, free, ring = make(rng, old, 16, 3, 5, 2)
    check(table, np.array(old, dtype=np.int64), np.array(new, dtype=np.int64), free, ring, 16, 64)


def test_most_requests():
    rng = np.random.default_rng(1)
    B = 16384
    old = rng.integers(0, 60, B)
    table, free, ring = make(rng, old.tolist(), 16, 4, B, 3)
    check(table, old, old + 1, free, ring, 16, B)


def test_short_pool_changes_nothing():
    rng = np.random.default_rng(2)
    table, free, ring = make(rng, [16, 5, 40], 16, 8, 3)
    want = check(table, np.array([16, 5, 40]), np.array([33, 0, 80]), free, ring, 16, 100)
    assert want[2][2] == 1  # needs 2 + 2 of 3 pages: the one that the second returns is for the next call
    assert np.array_equal(want[0], table)


@pytest.mark.parametrize("what", ["negative", "too long", "tokens", "ring", "overfull"])
def test_invalid_arguments_change_nothing_and_are_flagged(what):
    rng = np.random.default_rng(3)
    table, free, ring = make(rng, [16, 5], 16, 4, 6)
    old, new, tokens = np.array([16, 5]), np.array([20, 6]), 8
    if what == "negative":
        new[1] = -1
    elif what == "too long":
        new[0] = 65
    elif what == "tokens":
        tokens = 4
    elif what == "ring":
        ring[1] = ring[0] - 1
    else:
        ring[1] = ring[0] + len(free) + 1
    want = check(table, old, new, free, ring, 16, tokens)
    assert want[2][2] == -1 and np.all(want[4] == -1)
    assert A.attn_get_device_error() == A.ATTN_ERR_INVALID_ARG


def test_extreme_lengths_do_not_overflow():
    # sums far past 32 bits are refused, not wrapped
    B, page = 4096, 1 << 20
    old, new = np.zeros(B, dtype=np.int64), np.full(B, 2 ** 31 - 1)
    table = np.full((B, 2048), -1, dtype=np.int32)
    free, ring = np.arange(7, dtype=np.int32), np.array([0, 7, 0], dtype=np.int64)
    t = torch.from_numpy(table).cuda()
    got = A.attn_page_update(t, torch.tensor(old, dtype=torch.int32).cuda(), torch.tensor(new, dtype=torch.int32).cuda(),
                             torch.from_numpy(free).cuda(), torch.from_numpy(ring).cuda(), page, 100)
    assert got[0].tolist() == [0, 7, -1] and bool((t == -1).all())
    assert A.attn_get_device_error() == A.ATTN_ERR_INVALID_ARG


def test_bad_page_in_a_table_gives_no_slot():
    rng = np.random.default_rng(4)
    table, free, ring = make(rng, [5, 5], 16, 2, 2)
    table[1, 0] = 1 << 30
    t = torch.from_numpy(table).cuda()
    lens = torch.tensor([5, 5], dtype=torch.int32).cuda()
    out = A.attn_page_update(t, lens, lens + 1, torch.from_numpy(free).cuda(), torch.from_numpy(ring).cuda(), 16, 4)
    assert out[2].tolist() == [int(table[0, 0]) * 16 + 5, -1, -1, -1]
    assert A.attn_get_device_error() == A.ATTN_ERR_INVALID_ARG


def test_many_steps_keep_every_page_in_one_place():
    rng = np.random.default_rng(5)
    B, page, pages = 40, 8, 300
    table = torch.full((B, 16), -1, dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda()
    ring = torch.tensor([0, pages, 0], dtype=torch.int64, device="cuda")
    lens = np.zeros(B, dtype=np.int64)
    for _ in range(60):
        new = np.where(rng.random(B) < 0.6, lens + rng.integers(0, 9, B), np.where(rng.random(B) < 0.3, 0, lens))
        new = np.minimum(new, 128)
        cu = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        ring, cs, slots, _ = A.attn_page_update(table, cu(lens), cu(new), free, ring, page, B * 9)
        state = ring.tolist()
        if state[2] == 0:
            lens = new
        else:
            assert state[2] > 0
            lens_end = np.where(rng.random(B) < 0.5, 0, lens)
            ring, _, _, _ = A.attn_page_update(table, cu(lens), cu(lens_end), free, ring, page, 0)
            state, lens = ring.tolist(), lens_end
        held = [table[b, : -(-int(lens[b]) // page)].tolist() for b in range(B)]
        loose = free[(torch.arange(state[0], state[1]) % pages).cuda()].tolist()
        assert sorted(sum(held, []) + loose) == list(range(pages))


def test_captured_step():
    rng = np.random.default_rng(6)
    table, free, ring = make(rng, [30, 31, 32, 1], 16, 8, 9)
    t, f = torch.from_numpy(table).cuda(), torch.from_numpy(free).cuda()
    r, r2 = torch.from_numpy(ring).cuda(), torch.zeros(3, dtype=torch.int64, device="cuda")
    old = torch.tensor([30, 31, 32, 1], dtype=torch.int32).cuda()
    A.attn_page_update(t.clone(), old, old, f.clone(), r, 16, 8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new = old + 1
        out = A.attn_page_update(t, old, new, f, r, 16, 8, ring_out=r2)
        r.copy_(r2)
        old.copy_(new)
    lens = np.array([30, 31, 32, 1])
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        table, free, ring, cu, slots, pos = R.page_update(table, lens, lens + 1, free, ring, 16, 8)
        lens = lens + 1
        assert np.array_equal(t.cpu().numpy(), table) and r.tolist() == ring.tolist()
        assert np.array_equal(out[2].cpu().numpy(), slots) and np.array_equal(out[3].cpu().numpy(), pos)

"""Decode behind shared prefixes against a 64-bit reference on each sequence's gathered keys: group
sizes and counts, every page size class, lengths from none to long, sequences without a group or
without keys, what pages hold behind the last key (NaN and infinities), wrong pages, agreement
with the paged decode, repeated, captured and concurrent calls."""

import math

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


def case(seed, B, Hq, Hkv, starts, plens, lens, page, dirty=True, q_scale=1.3):
    """Inputs; with dirty, every cache row that holds no key is NaN or infinite."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    need = [-(-n // page) for n in list(plens) + list(lens)]
    pages = sum(need) + 3
    q = (torch.randn(B, Hq, 1, 128, generator=g, device="cuda") * q_scale).bfloat16()
    kc = torch.randn(pages, page, Hkv, 128, generator=g, device="cuda").bfloat16()
    vc = torch.randn(pages, page, Hkv, 128, generator=g, device="cuda").bfloat16()
    order = torch.randperm(pages, generator=g, device="cuda").int()
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n])
        at += n
    if dirty:
        keep = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
        for r, n in zip(rows, list(plens) + list(lens)):
            keep[r.long()] = (torch.arange(len(r) * page, device="cuda") < n).view(-1, page)
        for c, bad in ((kc, float("nan")), (vc, float("inf"))):
            c[~keep] = bad
        vc[~keep, :, ::3] = float("nan")

    def table(part):
        t = torch.full((len(part), max([len(r) for r in part] + [1])), -1, dtype=torch.int32, device="cuda")
        for i, r in enumerate(part):
            t[i, : len(r)] = r
        return t

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ng = len(plens)
    return dict(q=q, k_cache=kc, v_cache=vc, prefix_table=table(rows[:ng]), prefix_lens=i32(plens),
                group_starts=i32(starts), block_table=table(rows[ng:]), seq_lens=i32(lens),
                max_prefix_len=max(plens, default=0), max_seq_len=max(lens, default=0))


def group_of(b, starts):
    for g in range(len(starts) - 1):
        if starts[g] <= b < starts[g + 1]:
            return g
    return None


def keys_of(c, b, starts, plens, lens):
    def rows(cache, table, n):
        return cache[table.long().clamp(min=0)].reshape(-1, *cache.shape[2:])[:n]

    g = group_of(b, starts)
    out = []
    for cache in (c["k_cache"], c["v_cache"]):
        part = [rows(cache, c["prefix_table"][g], plens[g])] if g is not None else []
        out.append(R.f64(torch.cat(part + [rows(cache, c["block_table"][b], lens[b])])))
    return out


def check(c, starts, plens, lens, o, lse, scale=1 / math.sqrt(128), some=None):
    assert A.attn_get_device_error() == 0  # (a wait that gave up names its test)
    for b in (some if some is not None else range(len(lens))):
        k, v = keys_of(c, b, starts, plens, lens)
        R.assert_decode(o[b, :, 0], lse[b], R.decode_reference(R.f64(c["q"][b, :, 0]), k, v, scale), "sequence %d" % b)


CASES = [
    # B, Hq, Hkv, starts, prefix lengths, own lengths, page
    (1, 1, 1, [0, 1], [1], [0], 8),
    (1, 1, 1, [0, 1], [0], [1], 8),
    (1, 8, 1, [0, 1], [129], [127], 16),
    (2, 8, 8, [0, 2], [128], [0, 0], 16),
    (3, 8, 2, [0, 3], [300], [5, 0, 700], 16),
    (5, 16, 2, [1, 3, 3, 4], [77, 500, 1], [0, 1, 128, 129, 0], 32),
    (7, 32, 4, [0, 0], [400], [3, 0, 1000, 64, 63, 65, 1], 64),
    (33, 16, 8, [0, 33], [1000], None, 8),
    (70, 8, 2, [0, 64, 70], [2049, 130], None, 128),
    (65, 4, 1, [0, 65], [600], None, 256),
    (130, 2, 2, [0, 129], [515], None, 16),
    (40, 32, 8, [0, 10, 20, 30, 40], [5000, 0, 64, 3333], None, 64),
]


def own_lens(seed, B):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 400, B)
    lens[rng.random(B) < 0.2] = 0
    return lens.tolist()


@pytest.mark.parametrize("n", range(len(CASES)))
def test_against_reference(n):
    B, Hq, Hkv, starts, plens, lens, page = CASES[n]
    lens = own_lens(n, B) if lens is None else lens
    c = case(100 + n, B, Hq, Hkv, starts, plens, lens, page)
    o, lse = A.attn_decode_shared_prefix(**c)
    torch.cuda.synchronize()
    assert A.attn_get_device_error() == 0
    check(c, starts, plens, lens, o, lse)


@pytest.mark.parametrize("scale", [-0.09, 0.0, 0.3])
def test_scales(scale):
    starts, plens, lens = [0, 3], [260], [10, 200, 0]
    c = case(120, 3, 8, 2, starts, plens, lens, 16)
    o, lse = A.attn_decode_shared_prefix(**c, scale=scale)
    torch.cuda.synchronize()
    check(c, starts, plens, lens, o, lse, scale)


def test_growing_maximum():
    # scores that rise along the keys make the running maximum move in every tile and part
    starts, plens, lens = [0, 4], [3000], [1500, 900, 10, 0]
    c = case(121, 4, 16, 4, starts, plens, lens, 64, q_scale=6.0)
    for table, n in ((c["prefix_table"][0], 3000), (c["block_table"][0], 1500)):
        rows = c["k_cache"][table.long()].float().reshape(-1, 4, 128)
        rows[:n] *= torch.linspace(0.1, 2.0, n, device="cuda")[:, None, None]
        c["k_cache"][table.long()] = rows.bfloat16().reshape(-1, 64, 4, 128)
    o, lse = A.attn_decode_shared_prefix(**c)
    torch.cuda.synchronize()
    check(c, starts, plens, lens, o, lse)


def test_no_groups_and_no_keys():
    c = case(122, 3, 8, 2, [0], [], [40, 0, 7], 16)
    assert c["prefix_table"].shape[0] == 0
    o, lse = A.attn_decode_shared_prefix(**c)
    check(c, [0], [], [40, 0, 7], o, lse)
    c = case(123, 3, 8, 2, [0, 3], [0], [0, 0, 0], 16)
    for bound in (0, 16):
        o, lse = A.attn_decode_shared_prefix(**dict(c, max_seq_len=bound, max_prefix_len=bound))
        torch.cuda.synchronize()
        assert torch.all(o == 0) and torch.all(lse == -math.inf)


def test_lengths_are_clamped_to_their_bounds():
    starts, plens, lens = [0, 2], [300], [100, 50]
    c = case(124, 2, 8, 2, starts, plens, lens, 16, dirty=False)
    c["prefix_lens"].fill_(1 << 30)
    c["seq_lens"].copy_(torch.tensor([-5, 50]))
    o, lse = A.attn_decode_shared_prefix(**dict(c, max_seq_len=48))
    torch.cuda.synchronize()
    check(c, starts, [300], [0, 48], o, lse)


def test_groups_reach_only_their_sequences():
    # entries outside [0, B] are clamped; sequences outside every group have no prefix
    starts, plens, lens = [-4, 2, 99], [70, 90], [5, 6, 7, 8]
    c = case(125, 4, 8, 2, starts, plens, lens, 16)
    o, lse = A.attn_decode_shared_prefix(**c)
    torch.cuda.synchronize()
    check(c, starts, plens, lens, o, lse)


@pytest.mark.parametrize("page", [8, 64])
def test_pages_outside_the_cache_read_as_zero_and_are_flagged(page):
    starts, plens, lens = [0, 2], [200], [100, 60]
    c = case(126, 2, 8, 2, starts, plens, lens, page)
    good = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in c.items()}
    ref_o, ref_l = A.attn_decode_shared_prefix(**good)
    assert A.attn_get_device_error() == 0
    c["block_table"][1, 0] = 1 << 30
    o, lse = A.attn_decode_shared_prefix(**c)
    assert A.attn_get_device_error() == A.ATTN_ERR_INVALID_ARG
    assert torch.equal(o[0], ref_o[0]) and torch.equal(lse[0], ref_l[0])
    k, v = keys_of(good, 1, starts, plens, lens)
    k[200:200 + min(page, 60)] = 0
    v[200:200 + min(page, 60)] = 0
    R.assert_decode(o[1, :, 0], lse[1], R.decode_reference(R.f64(c["q"][1, :, 0]), k, v, 1 / math.sqrt(128)), "zeros")


def test_agrees_with_paged_decode():
    # the prefix's pages put in front of every sequence's own: the same keys through attn_decode_paged
    page, plen = 64, 640
    lens = own_lens(3, 20)
    c = case(127, 20, 32, 8, [0, 20], [plen], lens, page, dirty=False)
    o, lse = A.attn_decode_shared_prefix(**c)
    table = torch.cat([c["prefix_table"].expand(20, -1), c["block_table"]], 1).contiguous()
    po, pl = A.attn_decode_paged(c["q"], c["k_cache"], c["v_cache"], table, c["seq_lens"] + plen, plen + max(lens))
    torch.cuda.synchronize()
    # both round their weights (2^-8) and outputs (2^-8): 2^-6 of the values' size
    assert (o.float() - po.float()).abs().max() <= 2.0 ** -6 * c["v_cache"].float().abs().max()
    assert (lse - pl).abs().max() <= 1e-4


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    # cuts of the lines at random places: wide, half-wide and thin blocks of groups beside own keys
    rng = np.random.default_rng(200 + seed)
    g = int(rng.choice([1, 2, 4, 8]))
    hkv = int(rng.choice([1, 2, 3, 5]))
    B = int(rng.integers(1, 200))
    n = int(rng.integers(0, min(B, 6) + 1))
    starts = sorted(rng.integers(0, B + 1, n + 1).tolist())
    plens = [int(x) for x in rng.choice([0, 1, 127, 128, 129, 700, 1500, 4000], n)]
    lens = [int(x) for x in np.where(rng.random(B) < 0.3, rng.integers(0, 1500, B), rng.integers(0, 150, B))]
    page = int(rng.choice([8, 16, 32, 64, 128, 256]))
    c = case(300 + seed, B, hkv * g, hkv, starts, plens, lens, page)
    o, lse = A.attn_decode_shared_prefix(**c)
    torch.cuda.synchronize()
    assert A.attn_get_device_error() == 0
    check(c, starts, plens, lens, o, lse, some=sorted(set(rng.integers(0, B, 24).tolist() + [0, B - 1])))


@pytest.mark.parametrize("B,ng,Hkv,G", [(5, 1000, 2, 4), (900, 1000, 1, 2), (1500, 3, 2, 8)])
def test_more_groups_or_sequences_than_threads(B, ng, Hkv, G):
    # several groups (most of them without a sequence) and several sequences to a thread of the walk
    rng = np.random.default_rng(B)
    starts = sorted(rng.integers(0, B + 1, ng + 1).tolist())
    plens = [int(x) for x in rng.choice([0, 1, 40, 200], ng)]
    lens = [int(x) for x in rng.integers(0, 90, B)]
    c = case(400 + B, B, Hkv * G, Hkv, starts, plens, lens, 16)
    o, lse = A.attn_decode_shared_prefix(**c)
    torch.cuda.synchronize()
    check(c, starts, plens, lens, o, lse, some=sorted(set(rng.integers(0, B, 40).tolist() + [0, B - 1])))


def test_groups_out_of_order_are_flagged_and_no_prefix_counts():
    lens = [5, 60, 7, 300]
    c = case(133, 4, 8, 2, [0, 2, 4], [70, 900], lens, 16)
    c["group_starts"].copy_(torch.tensor([0, 4, 1]))
    o, lse = A.attn_decode_shared_prefix(**c)
    assert A.attn_get_device_error() == A.ATTN_ERR_INVALID_ARG
    check(c, [0, 0, 0], [70, 900], lens, o, lse)


def test_on_another_stream_without_a_workspace():
    starts, plens, lens = [0, 30], [1000], own_lens(7, 30)
    c = case(134, 30, 16, 4, starts, plens, lens, 32)
    ref, ref_l = A.attn_decode_shared_prefix(**c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [A.attn_decode_shared_prefix(**c, stream=s, return_lse=False) for _ in range(4)]
    s.synchronize()
    for o, lse in outs:
        assert lse is None and torch.equal(o, ref)
    o, lse = torch.empty_like(ref), torch.empty_like(ref_l)
    got = A.attn_decode_shared_prefix(**c, o=o, lse=lse)
    torch.cuda.synchronize()
    assert got[0] is o and got[1] is lse and torch.equal(o, ref) and torch.equal(lse, ref_l)


def test_large_batch_and_long_prefix():
    B, plen = 256, 16384
    lens = own_lens(4, B)
    c = case(128, B, 32, 8, [0, B], [plen], lens, 32)
    o, lse = A.attn_decode_shared_prefix(**c)
    torch.cuda.synchronize()
    check(c, [0, B], [plen], lens, o, lse, some=(0, 63, 64, 200, 255))


def test_offsets_past_32_bits():
    # a cache of 9.7 GB: pages behind the first 4 GB and 2^32 elements
    pages, page, Hkv = 40000, 128, 8
    kc = torch.zeros(pages, page, Hkv, 128, dtype=torch.bfloat16, device="cuda")
    vc = kc  # the values are the keys
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    far = torch.tensor([pages - 1, pages - 9, 33000], device="cuda")
    kc[far] = torch.randn(3, page, Hkv, 128, generator=g, device="cuda").bfloat16()
    q = torch.randn(2, 8, 1, 128, generator=g, device="cuda").bfloat16()
    c = dict(q=q, k_cache=kc, v_cache=vc, prefix_table=far[None, :2].int().contiguous(),
             prefix_lens=torch.tensor([250], dtype=torch.int32, device="cuda"),
             group_starts=torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
             block_table=far[2:].int().view(1, 1).expand(2, 1).contiguous(),
             seq_lens=torch.tensor([100, 3], dtype=torch.int32, device="cuda"), max_prefix_len=250, max_seq_len=128)
    o, lse = A.attn_decode_shared_prefix(**c)
    torch.cuda.synchronize()
    check(c, [0, 2], [250], [100, 3], o, lse)


def test_calls_repeat_bitwise_and_leave_nothing_behind():
    starts, plens, lens = [0, 30, 50], [3000, 700], own_lens(6, 50)
    c = case(129, 50, 16, 4, starts, plens, lens, 16)
    nbytes = A.attn_decode_shared_prefix_workspace_bytes(50, 16, 4, 2, 3000, max(lens), 128)
    ws = torch.full((nbytes + 256,), 255, dtype=torch.uint8, device="cuda")  # NaN bits everywhere
    o1, l1 = A.attn_decode_shared_prefix(**c, workspace=ws[:nbytes])
    torch.cuda.synchronize()
    assert torch.all(ws[nbytes:] == 255)
    ws.fill_(0)
    o2, l2 = A.attn_decode_shared_prefix(**c, workspace=ws[:nbytes])
    torch.cuda.synchronize()
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    check(c, starts, plens, lens, o1, l1)


def test_two_captured_graphs_run_at_the_same_time():
    runs = []
    for seed, B in ((130, 12), (131, 40)):
        lens = own_lens(seed, B)
        c = case(seed, B, 16, 4, [0, B], [2000 + seed], lens, 16)
        ref = A.attn_decode_shared_prefix(**c)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = A.attn_decode_shared_prefix(**c)
        runs.append((graph, out, ref, torch.cuda.Stream(), c))  # a graph reads its inputs where they are
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, _, _, s, _ in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, ref, _, _ in runs:
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])


def test_short_workspace_is_refused():
    c = case(132, 4, 8, 2, [0, 4], [100], [1, 2, 3, 4], 16)
    nbytes = A.attn_decode_shared_prefix_workspace_bytes(4, 8, 2, 1, 100, 4, 128)
    with pytest.raises(A.AttnError) as e:
        A.attn_decode_shared_prefix(**c, workspace=torch.empty(nbytes - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == A.ATTN_ERR_WORKSPACE

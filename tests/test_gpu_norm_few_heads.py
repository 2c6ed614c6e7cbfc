"""Norm + rotation, its gradient and the paged form over many tokens of few heads (the share of one GPU of a
model split over several): tiles of heads that are mostly empty, and long sums of weight gradients, whose
bound follows from how the launch divides them."""

import os
import re

import pytest
import torch

from exact_io_aware_82_b200 import attn as A
from exact_io_aware_82_b200 import build as Bld

from . import _layer as R

BF, F32 = torch.bfloat16, torch.float32
CSRC = os.path.join(os.path.dirname(os.path.abspath(Bld.__file__)), "csrc")


def constant(name):
    return int(re.search(r"^constexpr int %s = (\d+);" % name, open(os.path.join(CSRC, "qk_norm_rope.cuh")).read(), re.M).group(1))


def additions(B, N, Hq, Hkv, d, size):
    """How many additions a term of a weight gradient takes part in at most, for (queries, keys).

    A tile is kTokens tokens x `heads` heads; every group of heads has the same whole number of blocks, as
    many as fit 148 x kTileBlocksBwd together.  A lane adds kUnrollBwd rows of each of its block's tiles in turn, its
    block the lanes of kTokens warps x the rows of a warp's load; of a side's blocks a thread then adds
    every kSumRows-th, eight at a time (a missing one is 0), and the rest is 2 + 5 exchanges."""
    tokens, unroll, rows = constant("kTokens"), constant("kUnrollBwd"), 512 // (d * size)
    cq, ck = (-(-h // (unroll * rows)) for h in (Hq, Hkv))
    runs = B * -(-N // tokens)
    blocks = min(runs, 148 * constant("kTileBlocksBwd") // (cq + ck))
    tiles = -(-runs // blocks)
    return [unroll * tiles + tokens * rows + 8 * -(-blocks * c // (8 * constant("kSumRows"))) + 7 for c in (cq, ck)]


def test_blocks_are_as_counted():
    # rows of partial sums that the workspace holds: 148 x kTileBlocksBwd
    Bld.build()
    A.lib()
    assert A.attn_qk_norm_rope_bwd_workspace_bytes(128) == 148 * constant("kTileBlocksBwd") * 128 * 4
    # 4 + 1 heads share the blocks evenly: 370 of 740 for each, 12 tiles each of 16384 tokens
    assert additions(1, 16384, 4, 1, 128, 2) == [24 + 8 + 8 + 7] * 2


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    Bld.build()
    A.lib()
    yield
    assert A.attn_get_device_error() == 0


CASES = [
    # dtype, B, N, Hq, Hkv, d, rot, sections, interleaved
    (BF, 1, 16384, 8, 1, 128, 128, None, False),
    (BF, 1, 16384, 4, 1, 128, 128, [16, 24, 24], False),
    (BF, 2, 5003, 16, 2, 128, 64, None, True),
    (BF, 1, 50001, 1, 1, 64, 64, None, False),
    (F32, 1, 12000, 2, 1, 128, 128, None, True),
    (F32, 3, 7001, 1, 1, 64, 32, [5, 11], False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,B,N,Hq,Hkv,d,rot,sections,inter", CASES)
def test_long_inputs_of_few_heads(gpu, dtype, B, N, Hq, Hkv, d, rot, sections, inter):
    g = torch.Generator()
    g.manual_seed(N)
    normal = lambda *s: torch.randn(s, generator=g).to(dtype).cuda()  # noqa: E731
    qkv = normal(B, N, Hq + 2 * Hkv, d)
    q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    # gradients with a mean, so that the long sums do not cancel
    dzq, dzk = normal(B, Hq, N, d) + 0.5, normal(B, Hkv, N, d) + 0.5
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2))
    rope = R.rope_table(4096, rot).cuda()
    pos = torch.randint(0, 4096, ((len(sections),) if sections else ()) + (N,), generator=g, dtype=torch.int32).cuda()
    z = A.attn_qk_norm_rope(q, k, wq, wk, rope, pos, sections=sections, interleaved=inter)
    out = A.attn_qk_norm_rope_bwd(q, k, dzq, dzk, wq, wk, rope, pos, sections=sections, interleaved=inter)
    torch.cuda.synchronize()
    count = additions(B, N, Hq, Hkv, d, dtype.itemsize)
    for i, (x, w, dz) in enumerate(((q, wq, dzq), (k, wk, dzk))):
        ref, bound = R.norm_rope(x, w, rope, pos, sections, inter)
        R.assert_within(z[i], ref, bound, dtype, "forward")
        ref, bound, rdw, mag = R.norm_rope_bwd(x, dz, w, rope, pos, sections, inter)
        R.assert_within(out[i], ref, bound, dtype, "backward")
        R.assert_within(out[2 + i], rdw, (14 + count[i]) * R.U * mag, F32, "weight gradient")


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (4, 1), (1, 1)])
def test_paged_form_of_few_heads(gpu, Hq, Hkv):
    T, pad, page = 9001, 77, 32
    g = torch.Generator()
    g.manual_seed(Hq)
    qkv = torch.randn(T, Hq + 2 * Hkv, 128, generator=g).to(BF).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    w = (1 + 0.3 * torch.randn(128, generator=g)).to(BF).cuda()
    rope = R.rope_table(512, 128).cuda()
    pos = torch.randint(0, 512, (T,), generator=g, dtype=torch.int32).cuda()
    pages = T // page + 2
    slots = torch.randperm(pages * page, generator=g)[:T].int()
    slots[torch.randperm(T, generator=g)[:pad]] = -1  # tokens left out anywhere
    slots = slots.cuda()
    live = slots >= 0
    kc, vc = (torch.full((pages, page, Hkv, 128), 3.0, dtype=BF, device="cuda") for _ in range(2))
    qo = torch.full((T, Hq, 128), 5.0, dtype=BF, device="cuda")
    A.attn_qk_norm_rope_paged(q, k, v, w, w, rope, pos, slots, kc, vc, q_out=qo)
    want_q, want_k = A.attn_qk_norm_rope(q, k, w, w, rope, pos)
    torch.cuda.synchronize()
    assert torch.equal(qo[live], want_q[live]) and torch.all(qo[~live] == 5.0)
    at = slots[live].long()
    assert torch.equal(kc.view(-1, Hkv, 128)[at], want_k[live]) and torch.equal(vc.view(-1, Hkv, 128)[at], v[live])
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.all(kc.view(-1, Hkv, 128)[rest] == 3.0) and torch.all(vc.view(-1, Hkv, 128)[rest] == 3.0)

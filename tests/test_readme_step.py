"""The serving step that the README shows, run as it stands there: on the CPU with stand-ins for the
library's calls that record what reaches the decode, and on the GPU against a 64-bit reference.
Requests grow by one token or several, stay, end and begin in one step; a pool that is short."""

import math
import os
import re

import numpy as np
import pytest
import torch

from exact_io_aware_82_b200 import attn as A
from exact_io_aware_82_b200 import build as Bld

from . import _layer as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, I32 = torch.bfloat16, torch.int32
HQ, HKV, D, PAGE, PREFIX = 8, 2, 128, 16, 21

STEPS = {
    # old lengths, new lengths, rows of padding behind the new tokens
    "a token each": ([4, 20, 6, 33, 7], [5, 21, 7, 34, 8], 0),
    "as many rows as requests": ([4, 20, 6, 33, 7], [5, 0, 7, 33, 8], 2),
    "ragged": ([4, 20, 0, 33, 7], [5, 0, 3, 33, 20], 4),
    "the first requests have none": ([4, 20, 6, 33, 7], [4, 0, 6, 36, 8], 1),
}


def snippet():
    text = open(os.path.join(ROOT, "README.md")).read()
    code = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "attn_page_update" in b]
    assert len(code) == 1
    return compile(code[0], "README.md", "exec")


def state(device, old, new, pad, spare=9):
    """What a user's program holds before the step; every cache row without a key is NaN."""
    g = torch.Generator()
    g.manual_seed(sum(new))
    B = len(old)
    had = [-(-n // PAGE) for n in [PREFIX] + list(old)]
    pages = sum(had) + spare
    order = torch.randperm(pages, generator=g).to(I32)
    caches = [torch.full((pages, PAGE, HKV, D), float("nan"), dtype=BF) for _ in range(2)]
    table, at = torch.full((B + 1, 8), -1, dtype=I32), 0
    for b, n in enumerate([PREFIX] + list(old)):
        mine = order[at:at + had[b]]
        table[b, :had[b]] = mine
        at += had[b]
        i = torch.arange(n)
        rows = mine[i // PAGE].long() * PAGE + i % PAGE
        for c in caches:
            c.view(-1, HKV, D)[rows] = torch.randn(n, HKV, D, generator=g).to(BF)
    free = torch.full((pages,), -1, dtype=I32)
    free[:spare] = order[at:]
    total = sum(max(n - o, 0) for o, n in zip(old, new)) + pad
    qkv = torch.randn(total, HQ + 2 * HKV, D, generator=g).to(BF)
    to = lambda t: t.to(device)  # noqa: E731
    qkv = to(qkv)
    i32 = lambda x: torch.tensor(x, dtype=I32, device=device)  # noqa: E731
    return dict(
        torch=torch, block_table=to(table[1:].contiguous()), old_lens=i32(old), new_lens=i32(new), free_pages=to(free),
        ring=torch.tensor([0, spare, 0], device=device), page_size=PAGE, max_tokens=total, prefix_of_each=i32([PREFIX] * B),
        q=qkv[:, :HQ], k=qkv[:, HQ:HQ + HKV], v=qkv[:, HQ + HKV:], wq=to((1 + 0.2 * torch.randn(D, generator=g)).to(BF)),
        wk=to((1 + 0.2 * torch.randn(D, generator=g)).to(BF)), rope=to(R.rope_table(128, D)), k_cache=to(caches[0]),
        v_cache=to(caches[1]), prefix_table=to(table[:1, :2].contiguous()), prefix_lens=i32([PREFIX]),
        group_starts=i32([0, B]), max_prefix_len=PREFIX, max_seq_len=64)


def newest(old, new):
    """(request, packed row of its newest token) of every request that has a new token."""
    ends = np.cumsum([max(n - o, 0) for o, n in zip(old, new)])
    return [(b, int(ends[b]) - 1) for b in range(len(old)) if new[b] > old[b]]


def stand_ins(seen):
    def page_update(table, old, new, free, ring, page, max_tokens, pos_offset=None):
        out = R.page_update(table.numpy(), old.numpy(), new.numpy(), free.numpy(), ring.numpy(), page, max_tokens,
                            pos_offset.numpy())
        table.copy_(torch.from_numpy(out[0])), free.copy_(torch.from_numpy(out[1]))
        return tuple(torch.from_numpy(x) for x in out[2:])

    def norm(q, k, v, wq, wk, rope, positions, slots, k_cache, v_cache):
        return torch.where(slots[:, None, None] >= 0, q, float("nan"))  # rows of left-out tokens: whatever was there

    def decode(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts, block_table, seq_lens, mp, ms):
        assert q.shape == (len(seq_lens), HQ, 1, D) and q.is_contiguous()
        assert seq_lens.dtype is I32 and seq_lens.is_contiguous()
        seen["q"], seen["lens"] = q, seq_lens
        return None, None

    return dict(attn_page_update=page_update, attn_qk_norm_rope_paged=norm, attn_decode_shared_prefix=decode)


@pytest.mark.parametrize("name", list(STEPS))
def test_every_request_decodes_its_own_newest_token(name):
    old, new, pad = STEPS[name]
    seen, s = {}, state("cpu", old, new, pad)
    raw = s["q"].clone()
    exec(snippet(), dict(s, **stand_ins(seen)))
    assert seen["lens"].tolist() == new
    for b, row in newest(old, new):
        assert torch.equal(seen["q"][b, :, 0], raw[row]), "request %d" % b


def test_a_pool_that_is_short_decodes_what_was_granted():
    # nothing was granted: tables keep their pages, so the lengths that go with them are the old ones
    old, new = [4, 20, 6, 33, 7], [5, 0, 90, 33, 8]
    seen, s = {}, state("cpu", old, new, 2, spare=1)
    exec(snippet(), dict(s, **stand_ins(seen)))
    assert seen["lens"].tolist() == old


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    Bld.build()
    A.lib()
    yield {n: getattr(A, n) for n in ("attn_page_update", "attn_qk_norm_rope_paged", "attn_decode_shared_prefix")}
    assert A.attn_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(STEPS))
def test_step_against_reference(gpu, name):
    old, new, pad = STEPS[name]
    s = state("cuda", old, new, pad)
    ns = dict(s, **gpu)
    exec(snippet(), ns)
    torch.cuda.synchronize()
    assert A.attn_get_device_error() == 0 and ns["ring"][2] == 0

    def rows(table, n, cache):
        i = torch.arange(n, device="cuda")
        return cache.view(-1, HKV, D)[table[i // PAGE].long() * PAGE + i % PAGE]

    for b, row in newest(old, new):
        at = torch.tensor([PREFIX + new[b] - 1], dtype=I32, device="cuda")
        q, k = A.attn_qk_norm_rope(s["q"][row:row + 1], s["k"][row:row + 1], s["wq"], s["wk"], s["rope"], at)
        keys, values = (torch.cat([rows(s["prefix_table"][0], PREFIX, c), rows(s["block_table"][b], new[b], c)])
                        for c in (s["k_cache"], s["v_cache"]))
        assert torch.equal(keys[-1], k[0]) and torch.equal(values[-1], s["v"][row])
        ref = R.decode_reference(R.f64(q[0]), R.f64(keys), R.f64(values), 1 / math.sqrt(D))
        R.assert_decode(ns["o"][b, :, 0], ns["lse"][b], ref, "request %d" % b)


@pytest.mark.gpu
def test_step_with_a_short_pool_changes_nothing(gpu):
    s = state("cuda", [4, 20, 6, 33, 7], [5, 0, 90, 33, 8], 2, spare=1)
    before = [s[n].clone() for n in ("block_table", "free_pages", "k_cache", "v_cache")]
    ns = dict(s, **gpu)
    exec(snippet(), ns)
    torch.cuda.synchronize()
    assert A.attn_get_device_error() == 0 and ns["ring"][2] > 0
    for x, n in zip(before, ("block_table", "free_pages", "k_cache", "v_cache")):
        assert torch.equal(x.view(-1).view(torch.int16 if x.dtype is BF else I32),
                           s[n].view(-1).view(torch.int16 if x.dtype is BF else I32)), n

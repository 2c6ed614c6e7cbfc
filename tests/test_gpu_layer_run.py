"""The operators around attention together, as a model's layer uses them: a serving run (pages, prompts
written into the cache, packed prefill, decode steps behind a shared prefix, ended and rejected
tokens) and a training step (norm + rotation, attention, and both backward passes), each against a
64-bit computation from the raw projections."""

import math

import numpy as np
import pytest
import torch

from exact_io_aware_82_b200 import attn as A
from exact_io_aware_82_b200 import build as Bld
from oracle import oracle as O

from . import _layer as R
from ._parity import BWD_ABS_MAX, BWD_REL, TOL_BF16, assert_close, to64

pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32
HQ, HKV, D = 16, 4, 128


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    Bld.build()
    A.lib()
    yield
    assert A.attn_get_device_error() == 0


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Layer:
    """Projections of every token ever seen, and the cache that the operators keep."""

    def __init__(self, pages, page, prefix_len, requests, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g, self.page, self.prefix_len = g, page, prefix_len
        self.wq = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(BF)
        self.wk = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(BF)
        self.rope = R.rope_table(2048, D).cuda()
        self.kc = torch.full((pages, page, HKV, D), float("nan"), dtype=BF, device="cuda")  # never initialised
        self.vc = self.kc.clone()
        self.table = torch.full((requests + 1, 64), -1, dtype=I32, device="cuda")  # the last row: the prefix
        self.free = torch.randperm(pages, generator=g, device="cuda").to(I32)
        self.ring = torch.tensor([0, pages, 0], dtype=torch.int64, device="cuda")
        self.lens = [0] * (requests + 1)
        self.seen = [torch.zeros(0, HQ + 2 * HKV, D, dtype=BF, device="cuda") for _ in range(requests + 1)]
        self.offset = i32([prefix_len] * requests + [0])

    def step(self, new_lens, pad=13):
        """Grow and shrink the requests; project, normalise, rotate and cache the new tokens."""
        counts = [max(n - o, 0) for o, n in zip(self.lens, new_lens)]
        total = sum(counts)
        self.ring, cu, slots, pos = A.attn_page_update(self.table, i32(self.lens), i32(new_lens), self.free, self.ring,
                                                       self.page, total + pad, pos_offset=self.offset)
        qkv = torch.randn(total + pad, HQ + 2 * HKV, D, generator=self.g, device="cuda").to(BF)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        qo = torch.zeros(total + pad, HQ, D, dtype=BF, device="cuda")
        A.attn_qk_norm_rope_paged(q, k, v, self.wq, self.wk, self.rope, pos, slots, self.kc, self.vc, q_out=qo)
        at = 0
        for b, (n, c) in enumerate(zip(new_lens, counts)):
            self.seen[b] = torch.cat([self.seen[b][:n], qkv[at:at + c]])
            at += c
        self.lens = list(new_lens)
        return qo, cu, counts

    def history(self, b):
        """Rotated queries, keys and values of request b behind the prefix, in 64 bits."""
        pre = self.seen[-1] if b < len(self.seen) - 1 else self.seen[-1][:0]
        x = torch.cat([pre, self.seen[b]])
        pos = torch.arange(len(x), dtype=I32)
        q, _ = R.norm_rope(x[:, :HQ].transpose(0, 1), self.wq, self.rope, pos)
        k, _ = R.norm_rope(x[:, HQ:HQ + HKV].transpose(0, 1), self.wk, self.rope, pos)
        return q, k, R.f64(x[:, HQ + HKV:].transpose(0, 1))


def check_last_row(layer, b, first, o, lse, what):
    """Output and LSE of request b's newest token over its history from position `first` on.

    The kernels see queries and keys rounded to bf16, 2^-8 of each entry, which the 64-bit history does
    not round: a score moves by at most (2^-7 + 2^-16) of the sum of its products' magnitudes, and
    LSE by no more than its scores do."""
    q, k, v = layer.history(b)
    q, k, v = q[:, -1:], k[:, first:], v[:, first:]
    ro, rl = O.attention(q[None], k[None], v[None], O.MASK_FULL, scale=1 / math.sqrt(D))
    assert_close(to64(o[b:b + 1]), None, ro, rl, TOL_BF16, what)
    mag = np.einsum("hgd,hnd->hgn", np.abs(q.reshape(HKV, HQ // HKV, D)), np.abs(k)).max(-1).reshape(HQ) / math.sqrt(D)
    bound = (2.0 ** -7 + 2.0 ** -16) * mag + TOL_BF16["lse_rel"] * np.maximum(1, np.abs(rl.reshape(HQ)))
    assert np.all(np.abs(to64(lse[b]) - rl.reshape(HQ)) <= bound), what + ": LSE"


def test_serving_run():
    requests, page, prefix_len = 6, 16, 75
    layer = Layer(200, page, prefix_len, requests, 1)
    # the shared prefix is a request of its own, then the prompts
    layer.step([0] * requests + [prefix_len])
    prompts = [33, 1, 16, 50, 5, 17]
    qo, cu, counts = layer.step(prompts + [prefix_len])
    # prefill over the prompts alone (packed), as far as the packed call covers it: causal within each
    kp = torch.cat([layer.kc.view(-1, HKV, D)[slot_rows(layer, b, prompts[b])] for b in range(requests)])
    vp = torch.cat([layer.vc.view(-1, HKV, D)[slot_rows(layer, b, prompts[b])] for b in range(requests)])
    total = sum(prompts)
    o, _ = A.attn_fwd_varlen(qo[:total].contiguous(), kp, vp, cu[:requests + 1].contiguous(),
                             cu[:requests + 1].contiguous(), max(prompts), mask_kind=A.MASK_CAUSAL)
    torch.cuda.synchronize()
    at = 0
    for b, n in enumerate(prompts):
        q, k, v = (t[:, prefix_len:] for t in layer.history(b))
        ro, rl = O.attention(q[None], k[None], v[None], O.MASK_CAUSAL, scale=1 / math.sqrt(D))
        # (queries and keys were rounded to bf16 on their way: within the tolerance of the path)
        assert_close(to64(o[at:at + n]).transpose(1, 0, 2)[None], None, ro, rl, TOL_BF16, "prompt %d" % b)
        at += n
    # decode steps: all grow by a token; one ends, one loses rejected tokens, a new one comes
    lens = list(prompts)
    for turn in range(8):
        if turn == 3:
            lens[1], lens[3] = 0, lens[3] - 2
            layer.step(lens + [prefix_len])
        if turn == 5:
            lens[1] = 40
            layer.step(lens + [prefix_len])
        live = [n > 0 for n in lens]
        lens = [n + 1 if n else 0 for n in lens]
        qo, cu, counts = layer.step(lens + [prefix_len])
        at = cu[1:requests + 1].long() - 1  # each request's new token (an ended one's: any)
        q = qo[at.clamp(min=0)].unsqueeze(2).contiguous()
        own = i32(lens)
        args = (layer.table[:requests], own)
        o, lse = A.attn_decode_shared_prefix(q, layer.kc, layer.vc, layer.table[requests:], i32([prefix_len]),
                                             i32([0, requests]), *args, prefix_len, max(lens))
        # the same through the paged decode on prefix + own pages: own keys alone here
        po, pl = A.attn_decode_paged(q, layer.kc.nan_to_num(), layer.vc.nan_to_num(), *args, max(lens))
        torch.cuda.synchronize()
        for b in range(requests):
            if not live[b]:
                continue
            check_last_row(layer, b, 0, o, lse, "turn %d request %d" % (turn, b))
            check_last_row(layer, b, prefix_len, po, pl, "own keys, turn %d request %d" % (turn, b))
    # every page is held once or free
    held = sum((layer.table[b, :-(-n // page)].tolist() for b, n in enumerate(layer.lens)), [])
    head, tail, missing = layer.ring.tolist()
    assert missing == 0
    loose = layer.free[(torch.arange(head, tail) % 200).cuda()].tolist()
    assert sorted(held + loose) == list(range(200))


def slot_rows(layer, b, n):
    i = torch.arange(n, device="cuda")
    return layer.table[b, i // layer.page].long() * layer.page + i % layer.page


def test_training_step():
    # the gradient of a fused projection through norm + rotation and attention, two position axes
    B, N = 2, 150
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    qkv = torch.randn(B, N, HQ + 2 * HKV, D, generator=g, device="cuda").to(BF)
    wq = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(BF)
    wk = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(BF)
    dout = torch.randn(B, HQ, N, D, generator=g, device="cuda").to(BF)
    rope, sections = R.rope_table(200, D).cuda(), [24, 40]
    pos = torch.randint(0, 200, (2, B, N), generator=g, device="cuda", dtype=I32)
    q, k = qkv[:, :, :HQ].transpose(1, 2), qkv[:, :, HQ:HQ + HKV].transpose(1, 2)
    v = qkv[:, :, HQ + HKV:].transpose(1, 2).contiguous()
    zq, zk = A.attn_qk_norm_rope(q, k, wq, wk, rope, pos, sections=sections)
    o, lse = A.attn_fwd(zq, zk, v, mask_kind=A.MASK_CAUSAL)
    dzq, dzk, dv = A.attn_bwd(zq, zk, v, o, lse, dout, mask_kind=A.MASK_CAUSAL)
    dqkv = torch.empty_like(qkv)
    dq, dk, dwq, dwk = A.attn_qk_norm_rope_bwd(
        q, k, dzq, dzk, wq, wk, rope, pos, sections=sections, dq=dqkv[:, :, :HQ].transpose(1, 2),
        dk=dqkv[:, :, HQ:HQ + HKV].transpose(1, 2))
    torch.cuda.synchronize()

    # 64 bits, by automatic differentiation of the plain formulas
    cos, sin = (torch.from_numpy(t)[:, None] for t in R.angles(rope, pos, sections))
    leaves = [t.detach().cpu().double().requires_grad_() for t in (q, k, v, wq, wk)]

    def turn(x, w):
        y = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w
        lo, hi = y.chunk(2, -1)
        return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)

    a, b = turn(leaves[0], leaves[3]), turn(leaves[1], leaves[4])
    s = (a @ b.repeat_interleave(HQ // HKV, 1).transpose(-1, -2)) / math.sqrt(D)
    s = s.masked_fill(~torch.ones(N, N, dtype=torch.bool).tril(), -math.inf)
    out = s.softmax(-1) @ leaves[2].repeat_interleave(HQ // HKV, 1)
    out.backward(dout.cpu().double())
    err = np.abs(to64(o) - out.detach().numpy())
    assert err.max() <= TOL_BF16["max_abs"] and err.mean() <= TOL_BF16["mean_abs"]
    # attn_bwd's tolerance (its roundings and the rounded zq, zk, dzq, dzk reach every gradient), relative to
    # the largest entry; the norm's backward pass adds one rounding of 2^-8
    for got, leaf, name in ((dq, leaves[0], "dq"), (dk, leaves[1], "dk"), (dv, leaves[2], "dv"), (dwq, leaves[3], "dwq"),
                            (dwk, leaves[4], "dwk")):
        ref = leaf.grad.numpy()
        err = np.abs(to64(got) - ref)
        assert err.max() <= (BWD_REL + 2.0 ** -8) * np.abs(ref).max() + BWD_ABS_MAX, (name, err.max(), np.abs(ref).max())

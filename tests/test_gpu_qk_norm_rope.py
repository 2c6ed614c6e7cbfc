"""Norm + rotation of queries and keys, its gradient and the paged form against 64-bit references:
types, head sizes and groups, lengths from one token up, strided views, position axes, partial and
interleaved rotation, either side without a weight, in place, extreme rows, positions and slots out
of range, padding, graph capture and other streams."""

import numpy as np
import pytest
import torch

from exact_io_aware_82_b200 import attn as A
from exact_io_aware_82_b200 import build as Bld

from . import _layer as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    Bld.build()
    A.lib()
    yield
    assert A.attn_get_device_error() == 0


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def fused(g, B, N, Hq, Hkv, d, dtype):
    """q, k as [B, H, N, d] views into one projection output."""
    qkv = normal(g, B, N, Hq + 2 * Hkv, d, dtype=dtype, scale=1.5)
    return qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)


def weight(g, d, dtype):
    return (1 + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda()


CASES = [
    # dtype, B, N, Hq, Hkv, d, rot, sections, interleaved
    (BF, 1, 1, 1, 1, 128, 128, None, False),
    (BF, 2, 7, 8, 2, 128, 128, None, False),
    (BF, 1, 131, 32, 8, 128, 64, None, True),
    (BF, 3, 33, 9, 3, 64, 64, None, False),
    (BF, 1, 65, 5, 5, 64, 32, [3, 6, 7], False),
    (BF, 2, 17, 12, 4, 128, 128, [16, 24, 24], False),
    (BF, 2, 17, 12, 4, 128, 96, [11, 0, 20, 17], True),
    (BF, 1, 40, 7, 1, 128, 0, None, False),
    (F32, 1, 1, 2, 1, 64, 64, None, False),
    (F32, 2, 50, 6, 2, 64, 48, [5, 19], True),
    (F32, 1, 77, 3, 3, 128, 128, [21, 21, 22], False),
    (F32, 2, 9, 16, 1, 128, 128, None, True),
    (BF, 1, 4097, 4, 1, 128, 128, None, False),
]


def positions_for(g, B, N, sections, max_pos, batch=True):
    shape = ((len(sections),) if sections else ()) + ((B, N) if batch else (N,))
    return torch.randint(0, max_pos, shape, generator=g, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype,B,N,Hq,Hkv,d,rot,sections,inter", CASES)
def test_forward(dtype, B, N, Hq, Hkv, d, rot, sections, inter):
    g = gen(1)
    q, k = fused(g, B, N, Hq, Hkv, d, dtype)
    wq, wk = weight(g, d, dtype), weight(g, d, dtype)
    rope = R.rope_table(999, rot).cuda()
    for batch in (False, True):
        pos = positions_for(g, B, N, sections, 999, batch)
        zq, zk = A.attn_qk_norm_rope(q, k, wq, wk, rope, pos, sections=sections, interleaved=inter)
        torch.cuda.synchronize()
        assert zq.is_contiguous() and zk.is_contiguous()
        for x, w, z, name in ((q, wq, zq, "q"), (k, wk, zk, "k")):
            ref, bound = R.norm_rope(x, w, rope, pos, sections, inter)
            R.assert_within(z, ref, bound, dtype, name)


@pytest.mark.parametrize("dtype,B,N,Hq,Hkv,d,rot,sections,inter", CASES)
def test_backward(dtype, B, N, Hq, Hkv, d, rot, sections, inter):
    g = gen(2)
    q, k = fused(g, B, N, Hq, Hkv, d, dtype)
    dzq, dzk = normal(g, B, Hq, N, d, dtype=dtype), normal(g, B, Hkv, N, d, dtype=dtype)
    wq, wk = weight(g, d, dtype), weight(g, d, dtype)
    rope = R.rope_table(500, rot).cuda()
    pos = positions_for(g, B, N, sections, 500)
    dqkv = torch.full((B, N, Hq + 2 * Hkv, d), 7.0, dtype=dtype, device="cuda")  # gradient of the projection
    dq, dk = dqkv[:, :, :Hq].transpose(1, 2), dqkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    out = A.attn_qk_norm_rope_bwd(q, k, dzq, dzk, wq, wk, rope, pos, sections=sections, interleaved=inter,
                                  dq=dq, dk=dk)
    torch.cuda.synchronize()
    assert out[0] is dq and torch.all(dqkv[:, :, Hq + Hkv:] == 7.0)
    for x, dz, w, dx, dw, H, name in ((q, dzq, wq, out[0], out[2], Hq, "q"), (k, dzk, wk, out[1], out[3], Hkv, "k")):
        ref, bound, rdw, mag = R.norm_rope_bwd(x, dz, w, rope, pos, sections, inter)
        R.assert_within(dx, ref, bound, dtype, "d" + name)
        R.assert_within(dw, rdw, R.dw_bound(mag, B * N * H), F32, "d%s_weight" % name)


def test_gradient_is_the_derivative():
    # central differences of sum(dz z) through the 64-bit forward formula
    g = gen(3)
    q, k = normal(g, 1, 2, 3, 64, dtype=F32), normal(g, 1, 1, 3, 64, dtype=F32)
    dzq, dzk = normal(g, 1, 2, 3, 64, dtype=F32), normal(g, 1, 1, 3, 64, dtype=F32)
    wq, wk = weight(g, 64, F32), weight(g, 64, F32)
    rope = R.rope_table(50, 32).cuda()
    pos = torch.tensor([3, 49, 11], dtype=torch.int32).cuda()
    dq, dk, dwq, dwk = A.attn_qk_norm_rope_bwd(q, k, dzq, dzk, wq, wk, rope, pos, eps=1e-3)

    def loss(x, w, dz):
        return (R.norm_rope(x, w, rope, pos, eps=1e-3)[0] * R.f64(dz)).sum()

    rng, h = np.random.default_rng(3), 1e-5
    for x, w, dz, dx, dw in ((q, wq, dzq, dq, dwq), (k, wk, dzk, dk, dwk)):
        step = torch.from_numpy(rng.standard_normal(tuple(x.shape)))
        diff = (loss(x.cpu().double() + h * step, w, dz) - loss(x.cpu().double() - h * step, w, dz)) / (2 * h)
        want = (R.f64(dx) * step.numpy()).sum()
        # fp32 gradients: 60 u of the summed magnitudes; the difference quotient itself h^2
        assert abs(diff - want) <= 1e-4 * np.abs(R.f64(dx) * step.numpy()).sum()
        step = torch.from_numpy(rng.standard_normal(64))
        diff = (loss(x, w.cpu().double() + h * step, dz) - loss(x, w.cpu().double() - h * step, dz)) / (2 * h)
        want = (R.f64(dw) * step.numpy()).sum()
        assert abs(diff - want) <= 1e-4 * np.abs(R.f64(dw) * step.numpy()).sum()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sides", ["q", "k", ""])
def test_sides_without_a_weight(dtype, sides):
    g = gen(4)
    q, k = fused(g, 2, 19, 6, 3, 128, dtype)
    wq = weight(g, 128, dtype) if "q" in sides else None
    wk = weight(g, 128, dtype) if "k" in sides else None
    rope = R.rope_table(40, 128).cuda()
    pos = positions_for(g, 2, 19, None, 40)
    zq, zk = A.attn_qk_norm_rope(q, k, wq, wk, rope, pos)
    dz = normal(g, 2, 6, 19, 128, dtype=dtype), normal(g, 2, 3, 19, 128, dtype=dtype)
    out = A.attn_qk_norm_rope_bwd(q, k, *dz, wq, wk, rope, pos)
    for i, (x, w, z) in enumerate(((q, wq, zq), (k, wk, zk))):
        ref, bound = R.norm_rope(x, w, rope, pos)
        R.assert_within(z, ref, bound, dtype, "forward")
        ref, bound, _, _ = R.norm_rope_bwd(x, dz[i], w, rope, pos)
        R.assert_within(out[i], ref, bound, dtype, "backward")
        assert (out[2 + i] is None) == (w is None)


def test_packed_and_dense_layouts_agree_bitwise():
    g = gen(5)
    q, k = normal(g, 37, 8, 128), normal(g, 37, 2, 128)
    wq, wk = weight(g, 128, BF), weight(g, 128, BF)
    rope = R.rope_table(64, 128).cuda()
    pos = positions_for(g, 1, 37, None, 64, batch=False)
    zq, zk = A.attn_qk_norm_rope(q, k, wq, wk, rope, pos)
    dq, dk = A.attn_qk_norm_rope(q[None].transpose(1, 2), k[None].transpose(1, 2), wq, wk, rope, pos)
    torch.cuda.synchronize()
    assert torch.equal(zq, dq[0].transpose(0, 1)) and torch.equal(zk, dk[0].transpose(0, 1))


def test_in_place_equals_out_of_place():
    g = gen(6)
    q, k = fused(g, 2, 300, 8, 2, 128, BF)
    wq, wk = weight(g, 128, BF), weight(g, 128, BF)
    rope = R.rope_table(300, 64).cuda()
    pos = torch.arange(300, dtype=torch.int32).cuda()
    zq, zk = A.attn_qk_norm_rope(q, k, wq, wk, rope, pos)
    dzq, dzk = zq.clone(), zk.clone()
    want = A.attn_qk_norm_rope_bwd(q, k, dzq, dzk, wq, wk, rope, pos)
    got = A.attn_qk_norm_rope_bwd(q, k, dzq, dzk, wq, wk, rope, pos, dq=dzq, dk=dzk)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    A.attn_qk_norm_rope(q, k, wq, wk, rope, pos, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(zq, q) and torch.equal(zk, k)


def test_gradient_in_the_place_of_its_inputs():
    g = gen(61)
    q, k = fused(g, 2, 131, 8, 2, 128, BF)
    wq, wk = weight(g, 128, BF), weight(g, 128, BF)
    rope = R.rope_table(200, 128).cuda()
    pos = torch.arange(131, dtype=torch.int32).cuda()
    dzq, dzk = (normal(g, *x.shape, dtype=BF) for x in (q, k))
    want = A.attn_qk_norm_rope_bwd(q, k, dzq, dzk, wq, wk, rope, pos)
    got = A.attn_qk_norm_rope_bwd(q, k, dzq, dzk, wq, wk, rope, pos, dq=q, dk=k)
    assert got[0] is q and got[1] is k
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_broadcast_heads_and_positions():
    # one key row shared by all heads (stride 0), positions of one sequence shared by the batch
    g = gen(7)
    q = normal(g, 3, 4, 21, 128)
    k = normal(g, 3, 1, 21, 128).expand(3, 4, 21, 128)
    wq, wk = weight(g, 128, BF), weight(g, 128, BF)
    rope = R.rope_table(64, 128).cuda()
    pos = torch.arange(21, dtype=torch.int32).cuda()[None].expand(3, 21)
    zq, zk = A.attn_qk_norm_rope(q, k, wq, wk, rope, pos)
    for x, w, z in ((q, wq, zq), (k, wk, zk)):
        ref, bound = R.norm_rope(x, w, rope, pos)
        R.assert_within(z, ref, bound, BF, "broadcast")
    # the gradient of an expanded input has a row for each of its rows
    dz = normal(g, 3, 4, 21, 128), normal(g, 3, 4, 21, 128)
    out = A.attn_qk_norm_rope_bwd(q, k, *dz, wq, wk, rope, pos)
    ref, bound, _, _ = R.norm_rope_bwd(k, dz[1], wk, rope, pos)
    R.assert_within(out[1], ref, bound, BF, "broadcast dk")


def test_extreme_rows():
    # a zero row gives zeros, tiny rows are held up by eps, a row that is not finite keeps to itself
    q = torch.zeros(1, 2, 6, 128, dtype=F32)
    q[0, :, 1] = 1e-30
    q[0, :, 2] = 1e15
    q[0, 1, 3, 5] = float("nan")
    q[0, 1, 4, 9] = float("inf")
    q[0, :, 5] = 1.0
    q = q.cuda()
    w = torch.ones(128, device="cuda")
    rope = R.rope_table(8, 64).cuda()
    pos = torch.arange(6, dtype=torch.int32).cuda()
    z, _ = A.attn_qk_norm_rope(q, q[:, :1], w, w, rope, pos)
    ok = [(0, n) for n in range(6)] + [(1, n) for n in (0, 1, 2, 5)]
    ref, bound = R.norm_rope(torch.nan_to_num(q, posinf=0.0), w, rope, pos)
    for h, n in ok:
        R.assert_within(z[0, h, n], ref[0, h, n], bound[0, h, n], F32, "row %d %d" % (h, n))
    assert torch.all(z[0, :, 0] == 0)
    assert torch.isnan(z[0, 1, 3]).all()
    assert torch.isnan(z[0, 1, 4, 9])  # inf / inf


def test_no_tokens():
    rope = R.rope_table(8, 64).cuda()
    w = torch.ones(64, device="cuda")
    q, k = torch.empty(2, 3, 0, 64, device="cuda"), torch.empty(2, 1, 0, 64, device="cuda")
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    zq, zk = A.attn_qk_norm_rope(q, k, w, w, rope, pos)
    assert zq.shape == q.shape and zk.shape == k.shape
    out = A.attn_qk_norm_rope_bwd(q, k, q, k, w, w, rope, pos)
    torch.cuda.synchronize()
    assert torch.all(out[2] == 0) and torch.all(out[3] == 0)


def test_positions_outside_the_table_are_flagged_not_followed():
    g = gen(8)
    q, k = normal(g, 1, 2, 5, 128), normal(g, 1, 1, 5, 128)
    w = weight(g, 128, BF)
    rope = R.rope_table(10, 128).cuda()
    pos = torch.tensor([[0, 9, 10, -1, 5], [1, 2, 3, 4, 1 << 30]], dtype=torch.int32).cuda()
    zq, zk = A.attn_qk_norm_rope(q, k, w, w, rope, pos, sections=[30, 34])
    assert A.attn_get_device_error() == A.ATTN_ERR_INVALID_ARG
    assert A.attn_get_device_error() == 0
    for x, z in ((q, zq), (k, zk)):
        ref, bound = R.norm_rope(x, w, rope, pos, [30, 34])
        R.assert_within(z, ref, bound, BF, "out of range")


def test_backward_is_the_same_every_time_and_on_another_stream():
    g = gen(9)
    q, k = fused(g, 2, 700, 16, 4, 128, BF)
    dz = normal(g, 2, 16, 700, 128), normal(g, 2, 4, 700, 128)
    wq, wk = weight(g, 128, BF), weight(g, 128, BF)
    rope = R.rope_table(700, 128).cuda()
    pos = torch.arange(700, dtype=torch.int32).cuda()
    first = A.attn_qk_norm_rope_bwd(q, k, *dz, wq, wk, rope, pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = A.attn_qk_norm_rope_bwd(q, k, *dz, wq, wk, rope, pos, stream=s)
    s.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,N", [(70, 1), (1, 3), (3, 2), (5, 4), (2, 5)])
def test_short_sequences_and_single_tokens(B, N):
    # one token a sequence, and fewer tokens than a tile holds; positions per sequence and shared
    g = gen(15)
    q, k = fused(g, B, N, 8, 4, 128, BF)
    wq, wk = weight(g, 128, BF), weight(g, 128, BF)
    rope = R.rope_table(64, 128).cuda()
    dz = normal(g, B, 8, N, 128), normal(g, B, 4, N, 128)
    for batch in (True, False):
        pos = positions_for(g, B, N, None, 64, batch)
        z = A.attn_qk_norm_rope(q, k, wq, wk, rope, pos)
        out = A.attn_qk_norm_rope_bwd(q, k, *dz, wq, wk, rope, pos)
        for i, (x, w) in enumerate(((q, wq), (k, wk))):
            ref, bound = R.norm_rope(x, w, rope, pos)
            R.assert_within(z[i], ref, bound, BF, "forward")
            ref, bound, rdw, mag = R.norm_rope_bwd(x, dz[i], w, rope, pos)
            R.assert_within(out[i], ref, bound, BF, "backward")
            R.assert_within(out[2 + i], rdw, R.dw_bound(mag, B * N * x.shape[1]), F32, "weight")


def test_outputs_leave_their_surroundings_alone():
    # strided outputs inside larger buffers, heads and tokens that do not fill the last tile
    g = gen(16)
    B, N, Hq, Hkv = 2, 11, 9, 3
    q, k = fused(g, B, N, Hq, Hkv, 128, BF)
    w = weight(g, 128, BF)
    rope = R.rope_table(16, 128).cuda()
    pos = torch.arange(N, dtype=torch.int32).cuda()
    buf = torch.full((B, N + 2, Hq + Hkv + 2, 192), 9.0, dtype=BF, device="cuda")
    qo = buf[:, 1:-1, 1:1 + Hq, 32:160].transpose(1, 2)
    ko = buf[:, 1:-1, 1 + Hq:-1, 32:160].transpose(1, 2)
    want = A.attn_qk_norm_rope(q, k, w, w, rope, pos)
    A.attn_qk_norm_rope(q, k, w, w, rope, pos, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    qo.fill_(9.0), ko.fill_(9.0)
    assert torch.all(buf == 9.0)


def test_offsets_past_32_bits():
    # a projection output of 6 GB: rows behind the first 4 GB
    N, H = 12000, 1000
    x = torch.zeros(1, N, 2 * H, 128, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(17)
    x[0, -5:] = torch.randn(5, 2 * H, 128, generator=g, device="cuda").to(BF)
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:].transpose(1, 2)
    w = torch.ones(128, dtype=BF, device="cuda")
    rope = R.rope_table(N, 128).cuda()
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    ref_q, bq = R.norm_rope(q[:, :, -5:], w, rope, pos[-5:])
    ref_k, bk = R.norm_rope(k[:, :, -5:], w, rope, pos[-5:])
    A.attn_qk_norm_rope(q, k, w, w, rope, pos, q_out=q, k_out=k)
    torch.cuda.synchronize()
    R.assert_within(q[:, :, -5:], ref_q, bq, BF, "q")
    R.assert_within(k[:, :, -5:], ref_k, bk, BF, "k")
    assert torch.all(x[0, :-5] == 0)


def paged_case(seed, T, pad, Hq, Hkv, page, rot=128, sections=None, inter=False):
    g = gen(seed)
    qkv = normal(g, T, Hq + 2 * Hkv, 128, scale=1.5)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    wq, wk = weight(g, 128, BF), weight(g, 128, BF)
    rope = R.rope_table(400, rot).cuda()
    pos = positions_for(g, 1, T, sections, 400, batch=False)
    pages = T // page + 3
    slots = torch.randperm(pages * page, generator=g)[:T].int()
    slots[T - pad:] = -1
    if pad > 2:
        slots[T - 2] = -(1 << 31)
    return q, k, v, wq, wk, rope, pos, slots.cuda(), pages


@pytest.mark.parametrize("T,pad,Hq,Hkv,page,rot,sections,inter", [
    (1, 0, 8, 8, 8, 128, None, False),
    (1, 1, 8, 2, 16, 128, None, False),
    (64, 0, 32, 8, 16, 128, None, False),
    (77, 13, 5, 1, 64, 96, [10, 19, 19], True),
    (2050, 5, 16, 4, 256, 64, None, False),
    (130, 0, 12, 3, 32, 0, None, False),
])
def test_paged(T, pad, Hq, Hkv, page, rot, sections, inter):
    q, k, v, wq, wk, rope, pos, slots, pages = paged_case(11, T, pad, Hq, Hkv, page, rot, sections)
    kc = torch.full((pages, page, Hkv, 128), 3.0, dtype=BF, device="cuda")
    vc = torch.full_like(kc, 4.0)
    qo = torch.full((T, Hq, 128), 5.0, dtype=BF, device="cuda")
    got = A.attn_qk_norm_rope_paged(q, k, v, wq, wk, rope, pos, slots, kc, vc, sections=sections,
                                    interleaved=inter, q_out=qo)
    torch.cuda.synchronize()
    assert got is qo
    live = T - pad
    rq, bq = R.norm_rope(q.transpose(0, 1), wq, rope, pos, sections, inter)
    rk, bk = R.norm_rope(k.transpose(0, 1), wk, rope, pos, sections, inter)
    R.assert_within(qo[:live].transpose(0, 1), rq[:, :live], bq[:, :live], BF, "q")
    assert torch.all(qo[live:] == 5.0)  # padding: left as it was
    at = slots[:live].long()
    R.assert_within(kc.view(-1, Hkv, 128)[at].transpose(0, 1), rk[:, :live], bk[:, :live], BF, "k")
    assert torch.equal(vc.view(-1, Hkv, 128)[at], v[:live])
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.all(kc.view(-1, Hkv, 128)[rest] == 3.0) and torch.all(vc.view(-1, Hkv, 128)[rest] == 4.0)


def test_paged_matches_the_packed_call_bitwise():
    q, k, v, wq, wk, rope, pos, slots, pages = paged_case(12, 90, 0, 16, 4, 16)
    kc = torch.zeros(pages, 16, 4, 128, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    zq = A.attn_qk_norm_rope_paged(q, k, v, wq, wk, rope, pos, slots, kc, vc)
    pq, pk = A.attn_qk_norm_rope(q, k, wq, wk, rope, pos)
    torch.cuda.synchronize()
    assert torch.equal(zq, pq) and torch.equal(kc.view(-1, 4, 128)[slots.long()], pk)


def test_slots_past_the_cache_are_flagged_not_followed():
    q, k, v, wq, wk, rope, pos, slots, pages = paged_case(13, 20, 0, 8, 2, 16)
    slots[7] = pages * 16
    slots[8] = 2 ** 31 - 1
    kc = torch.full((pages, 16, 2, 128), 3.0, dtype=BF, device="cuda")
    vc = torch.full_like(kc, 3.0)
    A.attn_qk_norm_rope_paged(q, k, v, wq, wk, rope, pos, slots, kc, vc)
    assert A.attn_get_device_error() == A.ATTN_ERR_INVALID_ARG
    keep = [i for i in range(20) if i not in (7, 8)]
    at = slots[keep].long()
    assert torch.equal(vc.view(-1, 2, 128)[at], v[keep])
    assert int((vc == 3.0).all(-1).all(-1).sum()) >= pages * 16 - 18


def test_captured_graph_replays_on_new_inputs():
    q, k, v, wq, wk, rope, pos, slots, pages = paged_case(14, 48, 4, 8, 2, 16)
    kc = torch.zeros(pages, 16, 2, 128, dtype=BF, device="cuda")
    vc, qo = torch.zeros_like(kc), torch.zeros(48, 8, 128, dtype=BF, device="cuda")
    dz = torch.randn(48, 8, 128, device="cuda").to(BF), torch.randn(48, 2, 128, device="cuda").to(BF)
    ws = torch.empty(A.attn_qk_norm_rope_bwd_workspace_bytes(128), dtype=torch.uint8, device="cuda")

    def step():
        A.attn_qk_norm_rope_paged(q, k, v, wq, wk, rope, pos, slots, kc, vc, q_out=qo)
        return A.attn_qk_norm_rope_bwd(q, k, *dz, wq, wk, rope, pos, workspace=ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    q.copy_(q.flip(0).clone())
    slots.copy_(slots.flip(0).clone())
    kc.zero_(), vc.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (qo, kc, vc) + out]
    kc.zero_(), vc.zero_()
    want = (qo, kc, vc) + step()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)

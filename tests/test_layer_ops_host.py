"""Refusals of the operators around attention, on the CPU: the C ABI turns bad arguments away before
it touches a device, the binding turns away tensors that do not fit the call."""

import ctypes

import pytest
import torch

from exact_io_aware_82_b200 import attn as A
from exact_io_aware_82_b200 import build as B

P = ctypes.c_void_p(16)  # non-null, aligned: refused calls never use it
Q = ctypes.c_void_p(4096)
N = ctypes.c_void_p(0)
ODD = ctypes.c_void_p(24)
E, U, W = A.ATTN_ERR_INVALID_ARG, A.ATTN_ERR_UNSUPPORTED, A.ATTN_ERR_WORKSPACE
bf16, f32, i32, i64, u8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


@pytest.fixture(scope="module")
def lib():
    B.build()
    return A.lib()


def longs(n, fill=128, **at):
    v = (ctypes.c_longlong * n)(*([fill] * n))
    for k, x in at.items():
        v[int(k[1:])] = x
    return v


def ints(*v):
    return (ctypes.c_int * len(v))(*v)


def fwd(lib, q=P, k=P, qo=P, ko=P, wq=P, wk=P, rope=P, pos=P, st=None, sec=None, dt=0, B_=2, N_=3, Hq=4, Hkv=2, d=128,
        rot=128, mp=10, axes=1, inter=0, eps=1e-6):
    return lib.attn_qk_norm_rope(q, k, qo, ko, wq, wk, rope, pos, st if st is not None else longs(14), sec, dt, B_, N_,
                                 Hq, Hkv, d, rot, mp, axes, inter, eps, N)


def bwd(lib, q=P, k=P, gq=P, gk=P, dq=P, dk=P, wq=P, wk=P, dwq=P, dwk=P, rope=P, pos=P, st=None, sec=None, dt=0, B_=2,
        N_=3, Hq=4, Hkv=2, d=128, rot=128, mp=10, axes=1, inter=0, eps=1e-6, ws=P, nb=1 << 30):
    return lib.attn_qk_norm_rope_bwd(q, k, gq, gk, dq, dk, wq, wk, dwq, dwk, rope, pos,
                                     st if st is not None else longs(20), sec, dt, B_, N_, Hq, Hkv, d, rot, mp, axes,
                                     inter, eps, ws, nb, N)


def paged(lib, q=P, k=P, v=P, qo=P, kc=P, vc=P, wq=P, wk=P, rope=P, pos=P, slots=P, st=None, sec=None, T=3, Hq=4, Hkv=2,
          pages=5, ps=16, d=128, rot=128, mp=10, axes=1, inter=0, eps=1e-6):
    return lib.attn_qk_norm_rope_paged(q, k, v, qo, kc, vc, wq, wk, rope, pos, slots,
                                       st if st is not None else longs(13), sec, T, Hq, Hkv, pages, ps, d, rot, mp, axes,
                                       inter, eps, N)


def test_norm_rope_refusals(lib):
    for call in (fwd, bwd, paged):
        for bad in ({"Hq": 0}, {"Hkv": 0}, {"rot": -16}, {"rot": 144}, {"rot": 40}, {"mp": -1}, {"axes": 0}, {"axes": 5},
                    {"axes": 2}, {"axes": 2, "sec": ints(30, 30)}, {"axes": 2, "sec": ints(65, -1)},
                    {"axes": 2, "sec": ints(2 ** 31 - 1, 2 ** 31 - 1)}, {"eps": -1.0}, {"eps": float("nan")},
                    {"eps": float("inf")}, {"rope": N}, {"pos": N}, {"q": N}, {"k": N}):
            assert call(lib, **bad) == E, (call, bad)
        assert call(lib, d=96, rot=96) == U
        assert call(lib, q=ODD) == U and call(lib, rope=ODD) == U and call(lib, wq=ODD) == U
        assert call(lib, pos=ctypes.c_void_p(18)) == U
        assert call(lib, st=longs(20, _2=132)) == U  # rows that are not 16-byte aligned
    for call in (fwd, bwd):
        assert call(lib, dt=2) == E and call(lib, dt=-1) == E and call(lib, B_=-1) == E and call(lib, N_=-1) == E
        assert call(lib, B_=70000, N_=70000) == U
    assert fwd(lib, qo=N) == E and fwd(lib, ko=N) == E
    assert lib.attn_qk_norm_rope(P, P, P, P, P, P, P, P, N, N, 0, 2, 3, 4, 2, 128, 128, 10, 1, 0, 1e-6, N) == E
    for bad in ({"gq": N}, {"gk": N}, {"dq": N}, {"dk": N}, {"dwq": N}, {"dwk": N}, {"wq": N}, {"wk": N}):
        assert bwd(lib, **bad) == E, bad
    for bad in ({"T": -1}, {"pages": -1}, {"ps": 12}, {"ps": 4}, {"v": N}, {"qo": N}, {"slots": N}, {"kc": N}, {"vc": N}):
        assert paged(lib, **bad) == E, bad
    assert paged(lib, d=64, rot=64) == U and paged(lib, pages=1 << 28, ps=16) == U
    assert A.attn_qk_norm_rope_bwd_workspace_bytes(128) == 2 * A.attn_qk_norm_rope_bwd_workspace_bytes(64) > 0
    assert A.attn_qk_norm_rope_bwd_workspace_bytes(96) == 0


def update(lib, bt=P, old=P, new=P, fr=P, ri=P, ro=Q, cu=P, sl=P, pos=P, B_=2, mp=4, ps=16, pages=9, mt=5):
    return lib.attn_page_update(bt, old, new, fr, ri, ro, cu, sl, pos, N, B_, mp, ps, pages, mt, N)


def test_page_update_refusals(lib):
    for bad in ({"B_": -1}, {"mp": -1}, {"pages": -1}, {"mt": -1}, {"ps": 0}, {"ps": 24}, {"ps": 1 << 21}, {"bt": N},
                {"old": N}, {"new": N}, {"fr": N}, {"ri": N}, {"ro": N}, {"cu": N}, {"sl": N}, {"pos": N},
                {"ro": P}, {"ro": ctypes.c_void_p(32)}):
        assert update(lib, **bad) == E, bad
    assert update(lib, B_=16385) == U
    assert update(lib, pages=1 << 28) == U
    assert update(lib, ri=ctypes.c_void_p(20)) == U


def prefix(lib, q=P, kc=P, vc=P, o=P, pt=P, pl=P, gs=P, bt=P, sl=P, B_=2, Hq=8, Hkv=2, ng=1, pages=10, ps=16, mpp=4, mpl=64,
           mp=4, ml=64, d=128, scale=0.1, ws=P, nb=1 << 40):
    return lib.attn_decode_shared_prefix(q, kc, vc, o, N, pt, pl, gs, bt, sl, B_, Hq, Hkv, ng, pages, ps, mpp, mpl, mp,
                                         ml, d, scale, ws, nb, N)


def test_shared_prefix_refusals(lib):
    for bad in ({"B_": -1}, {"Hq": 0}, {"Hkv": 0}, {"Hq": 3}, {"ng": -1}, {"pages": -1}, {"ps": 12}, {"ps": 4}, {"mpp": -1},
                {"mp": -1}, {"mpl": -1}, {"ml": -1}, {"mpl": 65}, {"ml": 65}, {"scale": float("nan")},
                {"scale": float("inf")}, {"q": N}, {"o": N}, {"kc": N}, {"vc": N}, {"pt": N}, {"pl": N}, {"gs": N},
                {"bt": N}, {"sl": N}):
        assert prefix(lib, **bad) == E, bad
    assert prefix(lib, Hq=16, Hkv=1) == U and prefix(lib, Hq=6) == U and prefix(lib, d=64) == U
    assert prefix(lib, pages=1 << 28) == U and prefix(lib, q=ODD) == U and prefix(lib, kc=ODD) == U
    # a line of steps that 32 bits cannot count
    assert prefix(lib, B_=100000, Hq=64, Hkv=64, ml=1 << 20, mp=1 << 16) == U
    need = A.attn_decode_shared_prefix_workspace_bytes
    assert need(2, 8, 3, 1, 64, 64, 128) == 0 and need(2, 8, 2, 1, 64, 64, 64) == 0 and need(-1, 8, 2, 1, 64, 64, 128) == 0
    # partial rows: 2 B Hq for wide and for thin prefix parts and for the own keys, and 256, 32 and 2 G
    # more for each of 148 CTAs; the plan
    rows = 6 * 64 * 32 + 148 * (256 + 32 + 8)
    assert need(64, 32, 8, 3, 5000, 100, 128) == -(-rows * 516 // 16) * 16 + 4 * (4 + 2 * 3 + 64)


def test_shared_prefix_longest_lengths(lib):
    # up to two tiles past a length are still counted in 32 bits
    need = A.attn_decode_shared_prefix_workspace_bytes
    most = 2 ** 31 - 1 - 512
    for args in ((most + 1, 0), (0, most + 1), (2 ** 31 - 1, 2 ** 31 - 1)):
        assert need(1, 1, 1, 1, *args, 128) == 0
        assert prefix(lib, B_=1, Hq=1, Hkv=1, mpl=args[0], ml=args[1], mp=1 << 30, mpp=1 << 30) == U
    assert need(1, 1, 1, 1, most, 0, 128) > 0 and need(1, 1, 1, 1, 0, most, 128) > 0


def t(*shape, dtype=bf16, device="cpu"):
    return torch.zeros(shape, dtype=dtype, device=device)


def raises(exc, match, fn, *args, **kw):
    with pytest.raises(exc, match=match):
        fn(*args, **kw)


def test_binding_norm_rope():
    f = A.attn_qk_norm_rope
    q, k, w, rope, pos = t(2, 8, 5, 128), t(2, 2, 5, 128), t(128), t(9, 64, dtype=f32), t(5, dtype=i32)
    raises(ValueError, "CUDA tensors", f, q, k, w, w, rope, pos)
    raises(ValueError, "CUDA tensors", f, q, k, None, w, rope, t(2, 5, dtype=i32))
    raises(ValueError, "CUDA tensors", f, q, k, w, w, rope, t(3, 5, dtype=i32), sections=[10, 11, 11])
    raises(ValueError, "CUDA tensors", f, q, k, w, w, rope, t(3, 2, 5, dtype=i32), sections=[10, 11, 11])
    raises(ValueError, "CUDA tensors", f, t(5, 8, 64), t(5, 2, 64), t(64), t(64), rope, pos)
    raises(ValueError, "CUDA tensors", f, t(2, 5, 8, 128).transpose(1, 2), k, w, w, rope, pos)
    raises(TypeError, "q must be", f, q.half(), k.half(), w, w, rope, pos)
    raises(TypeError, "k must be", f, q, k.float(), w, w, rope, pos)
    raises(ValueError, "k must have shape", f, q, t(2, 2, 4, 128), w, w, rope, pos)
    raises(ValueError, "both be", f, q, k[0], w, w, rope, pos)
    raises(ValueError, "q_weight must have shape", f, q, k, t(64), w, rope, pos)
    raises(TypeError, "k_weight must be", f, q, k, w, w.float(), rope, pos)
    raises(TypeError, "rope must be", f, q, k, w, w, rope.double(), pos)
    raises(TypeError, "positions must be", f, q, k, w, w, rope, pos.long())
    raises(ValueError, "positions must have shape", f, q, k, w, w, rope, t(4, dtype=i32))
    raises(ValueError, "positions must have shape", f, q, k, w, w, rope, pos, sections=[16, 16])
    raises(ValueError, "sections", f, q, k, w, w, rope, t(2, 5, dtype=i32), sections=[16, 15])
    raises(ValueError, "sections", f, q, k, w, w, rope, t(2, 5, dtype=i32), sections=[33, -1])
    raises(ValueError, "sections", f, q, k, w, w, rope, t(5, 5, dtype=i32), sections=[8, 8, 8, 4, 4])
    raises(ValueError, "last dimension", f, t(2, 8, 128, 5).transpose(2, 3), k, w, w, rope, pos)
    raises(ValueError, "q_out must have shape", f, q, k, w, w, rope, pos, q_out=t(2, 8, 4, 128))
    raises(ValueError, "overlaps itself", f, q, k, w, w, rope, pos, k_out=t(2, 1, 5, 128).expand(2, 2, 5, 128))
    raises(ValueError, "overlaps itself", f, q, k, w, w, rope, pos,
           k_out=t(2 * 2 * 5 * 128).as_strided((2, 2, 5, 128), (1280, 64, 128, 1)))
    raises(ValueError, "one device", f, q, k, w, w, rope, t(5, dtype=i32, device="meta"))
    g = A.attn_qk_norm_rope_bwd
    raises(ValueError, "CUDA tensors", g, q, k, q, k, w, w, rope, pos)
    raises(ValueError, "CUDA tensors", g, q, k, q, k, w, None, rope, pos, dq_weight=t(128, dtype=f32), workspace=t(8, dtype=u8))
    raises(ValueError, "dk_out must have shape", g, q, k, q, q, w, w, rope, pos)
    raises(ValueError, "weight is not", g, q, k, q, k, w, None, rope, pos, dk_weight=t(128, dtype=f32))
    raises(TypeError, "dq_weight must be", g, q, k, q, k, w, w, rope, pos, dq_weight=t(128))
    raises(ValueError, "overlaps itself", g, q, k, q, k, w, w, rope, pos, dq=t(2, 8, 1, 128).expand(2, 8, 5, 128))


def test_binding_norm_rope_paged():
    f = A.attn_qk_norm_rope_paged
    q, k, v, w = t(5, 8, 128), t(5, 2, 128), t(5, 2, 128), t(128)
    rope, pos, slots, kc = t(9, 64, dtype=f32), t(5, dtype=i32), t(5, dtype=i32), t(4, 16, 2, 128)
    raises(ValueError, "CUDA tensors", f, q, k, v, w, w, rope, pos, slots, kc, kc)
    raises(ValueError, "CUDA tensors", f, q, k, v, w, w, rope, t(2, 5, dtype=i32), slots, kc, kc, sections=[16, 16],
           q_out=t(5, 8, 128))
    raises(ValueError, "packed bf16", f, q.float(), k.float(), v, w.float(), w.float(), rope, pos, slots, kc, kc)
    raises(ValueError, "packed bf16", f, t(1, 8, 5, 128), t(1, 2, 5, 128), v, w, w, rope, pos, slots, kc, kc)
    raises(ValueError, "v must have shape", f, q, k, t(4, 2, 128), w, w, rope, pos, slots, kc, kc)
    raises(ValueError, "slots must have shape", f, q, k, v, w, w, rope, pos, t(4, dtype=i32), kc, kc)
    raises(TypeError, "slots must be", f, q, k, v, w, w, rope, pos, slots.long(), kc, kc)
    raises(ValueError, "k_cache must have shape", f, q, k, v, w, w, rope, pos, slots, t(4, 16, 1, 128), kc)
    raises(ValueError, "v_cache must have shape", f, q, k, v, w, w, rope, pos, slots, kc, t(3, 16, 2, 128))


def test_binding_page_update():
    f = A.attn_page_update
    bt, lens, free, ring = t(3, 4, dtype=i32), t(3, dtype=i32), t(12, dtype=i32), t(3, dtype=i64)
    raises(ValueError, "CUDA tensors", f, bt, lens, lens, free, ring, 16, 5)
    raises(ValueError, "CUDA tensors", f, bt, lens, lens, free, ring, 16, 0, pos_offset=lens, ring_out=t(3, dtype=i64),
           cu_seqlens=t(4, dtype=i32), slots=t(0, dtype=i32), positions=t(0, dtype=i32))
    raises(ValueError, "old_lens must have shape", f, bt, t(2, dtype=i32), lens, free, ring, 16, 5)
    raises(TypeError, "new_lens must be", f, bt, lens, lens.long(), free, ring, 16, 5)
    raises(ValueError, "ring must have shape", f, bt, lens, lens, free, t(2, dtype=i64), 16, 5)
    raises(TypeError, "ring must be", f, bt, lens, lens, free, t(3, dtype=i32), 16, 5)
    raises(ValueError, "slots must have shape", f, bt, lens, lens, free, ring, 16, 5, slots=t(4, dtype=i32))
    raises(ValueError, "pos_offset must have shape", f, bt, lens, lens, free, ring, 16, 5, pos_offset=t(2, dtype=i32))
    raises(ValueError, "max_tokens", f, bt, lens, lens, free, ring, 16, -1)


def test_binding_shared_prefix():
    f = A.attn_decode_shared_prefix
    q, kc, pt, pl = t(3, 8, 1, 128), t(9, 16, 2, 128), t(2, 4, dtype=i32), t(2, dtype=i32)
    gs, bt, sl = t(3, dtype=i32), t(3, 4, dtype=i32), t(3, dtype=i32)
    raises(ValueError, "CUDA tensors", f, q, kc, kc, pt, pl, gs, bt, sl, 64, 64)
    raises(ValueError, "one query token", f, t(3, 8, 2, 128), kc, kc, pt, pl, gs, bt, sl, 64, 64)
    raises(ValueError, "prefix_lens must have shape", f, q, kc, kc, pt, t(3, dtype=i32), gs, bt, sl, 64, 64)
    raises(ValueError, "group_starts must have shape", f, q, kc, kc, pt, pl, pl, bt, sl, 64, 64)
    raises(ValueError, "one row per sequence", f, q, kc, kc, pt, pl, gs, t(2, 4, dtype=i32), sl, 64, 64)
    raises(ValueError, "seq_lens must have shape", f, q, kc, kc, pt, pl, gs, bt, pl, 64, 64)
    raises(ValueError, "v_cache must have shape", f, q, kc, t(8, 16, 2, 128), pt, pl, gs, bt, sl, 64, 64)
    raises(TypeError, "prefix_table must be", f, q, kc, kc, pt.long(), pl, gs, bt, sl, 64, 64)
    raises(ValueError, "o must have shape", f, q, kc, kc, pt, pl, gs, bt, sl, 64, 64, o=t(3, 8, 2, 128))
    raises(TypeError, "workspace must be", f, q, kc, kc, pt, pl, gs, bt, sl, 64, 64, workspace=t(9))

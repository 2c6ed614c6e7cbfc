"""Decode behind a shared prefix beside attn_decode_paged on the same keys: each within the error that its
own arithmetic allows, and the two within the sum, element by element, so that a wrong value shows even
where outputs are small."""

import math

import numpy as np
import pytest
import torch

from exact_io_aware_82_b200 import attn as A
from exact_io_aware_82_b200 import build as Bld

from . import _layer as R
from .test_gpu_shared_prefix import case, keys_of, own_lens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    Bld.build()
    A.lib()
    yield
    assert A.attn_get_device_error() == 0


def reference(q, keys, values, scale):
    """(o [Hq, d], lse [Hq], the weights' mean of |v| [Hq, d], relative error of a weight [Hq]) in 64 bits.

    Counted in u = 2^-24 for sums in any order over n keys: a score is 128 products in fp32, 130 u of the sum
    of their magnitudes; its exponential 2^-22; a sum over the keys n u.  A weight over the sum of weights has twice
    that, and 3 holds the joining of parts (two exponentials more) as well."""
    Hq, d = q.shape
    n, Hkv, _ = keys.shape
    qh = q.reshape(Hkv, Hq // Hkv, d)
    x = np.einsum("hgd,nhd->hgn", qh, keys) * scale
    mag = np.einsum("hgd,nhd->hgn", np.abs(qh), np.abs(keys)).max(-1) * abs(scale)
    m = x.max(-1, keepdims=True)
    e = np.exp(x - m)
    z = e.sum(-1, keepdims=True)
    o = np.einsum("hgn,nhd->hgd", e / z, values)
    a = np.einsum("hgn,nhd->hgd", e / z, np.abs(values))
    delta = 130 * R.U * mag + 2.0 ** -22 + n * R.U
    lse = (m + np.log(z))[..., 0]
    return o.reshape(Hq, d), lse.reshape(Hq), a.reshape(Hq, d), delta.reshape(Hq)


@pytest.mark.parametrize("page,Hq,Hkv", [(16, 32, 8), (16, 8, 8), (32, 16, 2), (64, 32, 8), (128, 8, 4)])
def test_both_decodes_within_their_counted_errors(page, Hq, Hkv):
    plen, B = 1280 if page == 128 else 640, 20
    lens = own_lens(3, B)
    c = case(500 + page + Hkv, B, Hq, Hkv, [0, B], [plen], lens, page, dirty=False)
    o, lse = A.attn_decode_shared_prefix(**c)
    table = torch.cat([c["prefix_table"].expand(B, -1), c["block_table"]], 1).contiguous()
    po, pl = A.attn_decode_paged(c["q"], c["k_cache"], c["v_cache"], table, c["seq_lens"] + plen, plen + max(lens))
    torch.cuda.synchronize()
    half = R.half_step(torch.bfloat16)
    for b in range(B):
        k, v = keys_of(c, b, [0, B], [plen], lens)
        ref, rl, a, delta = reference(R.f64(c["q"][b, :, 0]), k, v, 1 / math.sqrt(128))
        fp32 = 3 * delta[:, None] * a
        rounded = half * a + fp32  # weights as bf16 for the product with V
        mine, paged = rounded, rounded if page >= 64 else fp32
        R.assert_within(o[b, :, 0], ref, mine, torch.bfloat16, "shared prefix, sequence %d" % b)
        R.assert_within(po[b, :, 0], ref, paged, torch.bfloat16, "paged, sequence %d" % b)
        steps = half * (2 * np.abs(ref) + mine + paged)
        assert np.all(np.abs(R.f64(o[b, :, 0]) - R.f64(po[b, :, 0])) <= mine + paged + steps)
        bound = delta + 4 * R.U * np.abs(rl)
        assert np.all(np.abs(R.f64(lse[b]) - rl) <= bound) and np.all(np.abs(R.f64(pl[b]) - rl) <= bound)
        # the bounds tell the outputs from zeros and from their neighbours'
        assert (np.abs(ref) > 4 * (mine + steps)).mean() > 0.5

"""Host sizes of the operators around attention that 32 bits do not hold: refused by name, not cut down
to whatever their low bits say (tensors on the meta device hold nothing)."""

import pytest
import torch

from exact_io_aware_82_b200 import attn as A
from exact_io_aware_82_b200 import build as B

bf16, i32, i64 = torch.bfloat16, torch.int32, torch.int64
BIG = [2 ** 31, 2 ** 32 + 64, 2 ** 63, -2 ** 31 - 1, -2 ** 32 + 64]


def t(*shape, dtype=i32):
    return torch.empty(shape, dtype=dtype, device="meta")


def refused(match, fn, *args):
    with pytest.raises(ValueError, match=match):
        fn(*args)


@pytest.mark.parametrize("big", BIG)
def test_shared_prefix(big):
    q, kc = t(3, 8, 1, 128, dtype=bf16), t(9, 16, 2, 128, dtype=bf16)
    args = (q, kc, kc, t(2, 4), t(2), t(3), t(3, 4), t(3))
    refused("CUDA tensors", A.attn_decode_shared_prefix, *args, 64, 64)
    refused("max_prefix_len", A.attn_decode_shared_prefix, *args, big, 64)
    refused("max_seq_len", A.attn_decode_shared_prefix, *args, 64, big)
    if 0 < big < 2 ** 60:
        refused("max_prefix_pages", A.attn_decode_shared_prefix, q, kc, kc, t(2, big), *args[4:], 64, 64)
        refused("max_pages_per_seq", A.attn_decode_shared_prefix, *args[:6], t(3, big), t(3), 64, 64)
    if big > 0:
        B.build()
        need = A.attn_decode_shared_prefix_workspace_bytes
        assert need(3, 8, 2, 2, 64, 64, 128) > 0
        for sizes in ((big, 8, 2, 2, 64, 64, 128), (3, 8, 2, 2, big, 64, 128), (3, 8, 2, 2, 64, big, 128)):
            assert need(*sizes) == 0


@pytest.mark.parametrize("big", BIG)
def test_page_update(big):
    lens, free, ring = t(3), t(12), t(3, dtype=i64)
    refused("CUDA tensors", A.attn_page_update, t(3, 4), lens, lens, free, ring, 16, 5)
    refused("max_tokens", A.attn_page_update, t(3, 4), lens, lens, free, ring, 16, big)
    refused("page_size", A.attn_page_update, t(3, 4), lens, lens, free, ring, big, 5)
    if 0 < big < 2 ** 60:
        refused("num_pages", A.attn_page_update, t(3, 4), lens, lens, t(big), ring, 16, 5)
        refused("max_pages_per_seq", A.attn_page_update, t(3, big), lens, lens, free, ring, 16, 5)

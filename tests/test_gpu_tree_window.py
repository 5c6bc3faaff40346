"""Tree attention over an fp16 window: many light keys beside a heavy one."""
import math

import numpy as np
import pytest
import torch

from compressed_decode_attention_zkv_b200 import build as B
from compressed_decode_attention_zkv_b200 import zkv

pytestmark = pytest.mark.gpu
D = 64
SCORES = 6 * 2.0 ** -24 * 18          # roundings of a score of 18


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.build()
    zkv.lib()


def test_light_window_keys_add_up():
    """4095 window tokens of weight 2^-25.5 each beside one of weight 1."""
    W, N, Hkv, G = 4096, 3, 2, 4
    top = 17.671875                          # (an fp16 number)
    q = torch.zeros(1, N, Hkv * G, D, dtype=torch.float16, device="cuda")
    q[..., 0] = 8
    wk = torch.zeros(1, Hkv, W, D, dtype=torch.float16, device="cuda")
    wk[:, :, 100, 0] = top
    wv = torch.full((1, Hkv, W, D), 8.0, dtype=torch.float16, device="cuda")
    wv[:, :, 100] = 1.0
    none = torch.zeros(1, N, Hkv, D, dtype=torch.float16, device="cuda")
    codes = torch.zeros(1, Hkv, 16, 1, dtype=torch.uint8, device="cuda")
    books = torch.zeros(Hkv, 1, 256, D, device="cuda")
    one = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")   # noqa: E731
    out, lse = zkv.rvq_tree_attn(q, none, none, codes, codes, one(0), books, books, wk, wv, one(W),
                                 mask=torch.zeros(N, N, dtype=torch.bool, device="cuda"))
    tail = (W - 1) * math.exp(-top)
    want = (1 + 8 * tail) / (1 + tail)
    # 64 steps of float32 sums of the weights and of the values (2^-24 each), 1 / 16 of the tail lost in
    # the one lane's sum that holds the large weight, splits of 2^-22
    assert (out.double() - want).abs().max().item() <= 130 * 2.0 ** -24 + tail / 16 + 2.0 ** -21
    assert (lse.double() - top - math.log1p(tail)).abs().max().item() <= 64 * 2.0 ** -24 + tail / 16 + SCORES

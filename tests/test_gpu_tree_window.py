"""Tree attention over an fp16 window: many light keys beside a heavy one, values that are not finite."""
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


def test_infinities_in_the_window():
    """What a visible window value holds reaches the output as the sum has it: an infinity of little weight too,
    NaN for two of opposite sign, and nothing of it in the other dimensions."""
    rng = np.random.default_rng(8)
    W, N, Hkv, G, T = 150, 5, 2, 4, 300
    new = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float16)).cuda()   # noqa: E731
    q, dk, dv = new(1, N, Hkv * G, D), new(1, N, Hkv, D), new(1, N, Hkv, D)
    wk, wv = new(1, Hkv, W, D), new(1, Hkv, W, D)
    q[..., 0] = 8
    wk[:, :, 3, 0] = -30                     # about 2^-43 of the others
    kc = torch.from_numpy(rng.integers(0, 256, (1, Hkv, 304, 2)).astype(np.uint8)).cuda()
    books = torch.from_numpy((rng.standard_normal((Hkv, 2, 256, D)) * 0.3).astype(np.float32)).cuda()
    one = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")   # noqa: E731
    plain, _ = zkv.rvq_tree_attn(q, dk, dv, kc, kc, one(T), books, books, wk, wv, one(W - 1))
    bad = wv.clone()
    bad[:, :, 3, 5], bad[:, :, 70, 9] = math.inf, -math.inf
    bad[:, :, 1, 11], bad[:, :, 140, 11] = math.inf, -math.inf
    bad[:, :, 64, 20] = math.nan
    bad[:, :, W - 1] = math.nan              # behind the window
    out, lse = zkv.rvq_tree_attn(q, dk, dv, kc, kc, one(T), books, books, wk, bad, one(W - 1))
    assert (out[..., 5] == math.inf).all() and (out[..., 9] == -math.inf).all()
    assert torch.isnan(out[..., 11]).all() and torch.isnan(out[..., 20]).all()
    rest = [i for i in range(D) if i not in (5, 9, 11, 20)]
    assert torch.equal(out[..., rest], plain[..., rest]) and torch.isfinite(lse).all()

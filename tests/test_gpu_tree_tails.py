"""Tree attention of rows where one token outweighs all others, which are many: their weight must
not be lost in the roundings of the weights.

All queries are a multiple of the first unit vector, so every score is known exactly; no draft is
visible.  Scores are float32 and reach 21: |lse error| <= 6 roundings of 2^-24 of that, 7.5e-6."""
import math

import numpy as np
import pytest
import torch

from compressed_decode_attention_zkv_b200 import build as B
from compressed_decode_attention_zkv_b200 import zkv

pytestmark = pytest.mark.gpu
D = 64
SCORES = 7.5e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.build()
    zkv.lib()


def hadamard(d):
    h = np.ones((1, 1))
    while len(h) < d:
        h = np.block([[h, h], [h, -h]])
    return h / math.sqrt(d)


def attend(T, codes, first, values, Sk, Sv, N=32, G=8, Hkv=8):
    """Rows of N G equal queries over T tokens with the given first-stage codes; codeword z of the
    first key stage scores first[z], of the first value stage is values[z]; the other stages hold
    nothing.  (256 groups of rows: a block scans tokens of one for a long while.)"""
    cap = (T + 15) // 16 * 16
    q = torch.zeros(1, N, Hkv * G, D, dtype=torch.float16, device="cuda")
    q[..., 0] = 8                        # rotated: 8 / sqrt(D) everywhere, and the scale is 1 / sqrt(D)
    Ck = torch.zeros(Hkv, Sk, 256, D, device="cuda")
    Ck[:, 0, :, 0] = torch.tensor(first, device="cuda", dtype=torch.float32) * 8
    Cv = torch.zeros(Hkv, Sv, 256, D, device="cuda")
    Cv[:, 0] = torch.tensor(values, device="cuda", dtype=torch.float32)
    kc = torch.zeros(1, Hkv, cap, Sk, dtype=torch.uint8, device="cuda")
    vc = torch.zeros(1, Hkv, cap, Sv, dtype=torch.uint8, device="cuda")
    kc[..., :T, 0] = torch.from_numpy(codes).cuda()
    vc[..., :T, 0] = torch.from_numpy(codes).cuda()
    none = torch.zeros(1, N, Hkv, D, dtype=torch.float16, device="cuda")
    win = torch.zeros(1, Hkv, 1, D, dtype=torch.float16, device="cuda")
    one = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")   # noqa: E731
    return zkv.rvq_tree_attn(q, none, none, kc, vc, one(T), Ck, Cv, win, win, one(0),
                             mask=torch.zeros(N, N, dtype=torch.bool, device="cuda"))


def expect(codes, first, values):
    count = np.bincount(codes, minlength=256).astype(np.float64)
    w = count * np.exp(np.asarray(first, np.float64))
    return (w / w.sum()) @ np.asarray(values, np.float64) @ hadamard(D), math.log(w.sum())


def tolerance(T, tile, spread):
    """Of the row's sum.  A weight is rounded to a unit of at most 2^-27 of the largest sum, at an offset
    that 8 positions x (tile / 128) warps spread evenly: 16 tokens of a tile share one, so equal
    weights are off by at most 16 units per tile.  Unequal ones: by six standard deviations of T
    independent roundings (half a unit each) more.  2^-21 for 2^x and the sums."""
    units = 16 * (T // tile + 2) + (3 * math.sqrt(T) if spread else 0)
    return units * 2.0 ** -27 + 2.0 ** -21


@pytest.mark.parametrize("at", [0, 1000, 20001])
@pytest.mark.parametrize("top", [18.0, 19.0, 19.5, 20.125, 20.75])       # 26.0 .. 29.9 in base 2
@pytest.mark.parametrize("Sk,Sv", [(1, 1), (4, 4), (2, 8)])
def test_equal_tail(top, at, Sk, Sv):
    T = 32640
    codes = np.zeros(T, np.uint8)
    codes[at] = 1
    first = [0.0, top] + [0.0] * 254
    values = np.random.default_rng(5).standard_normal((256, D))
    out, lse = attend(T, codes, first, values, Sk, Sv)
    wo, wl = expect(codes, first, values)
    tol = tolerance(T, 2048 if Sv == 8 else 1536, False)
    assert np.abs(lse.cpu().numpy() - wl).max() <= tol + SCORES
    v = np.abs(values @ hadamard(D)).max()
    # weights and their sum, and the two scores' errors on a tail of 32639 e^-top
    assert np.abs(out.cpu().numpy() - wo).max() <= 2 * v * (tol + 2 * SCORES * T * math.exp(-top) + 2.0 ** -20)


@pytest.mark.parametrize("top", [20.0, 21.0])
def test_uneven_tail(top):
    """Scores of a standard normal distribution below the large one."""
    rng = np.random.default_rng(6)
    T = 32640
    first = np.round(rng.standard_normal(256) * 64) / 64
    first[1] = top
    codes = rng.integers(2, 256, T).astype(np.uint8)
    codes[0] = 1
    values = rng.standard_normal((256, D))
    out, lse = attend(T, codes, first, values, 4, 4)
    wo, wl = expect(codes, first, values)
    tol = tolerance(T, 1536, True)
    assert np.abs(lse.cpu().numpy() - wl).max() <= tol + SCORES


def test_absent_weights_stay_zero():
    """Tokens too light for any count, and those behind the last, add nothing to their codewords."""
    T = 700
    codes = np.full(T, 2, np.uint8)
    codes[0] = 1
    first = [0.0, 0.0, -120.0] + [0.0] * 253
    values = np.zeros((256, D))
    values[0], values[1], values[2] = 5.0, 1.0, 7.0
    out, lse = attend(T, codes, first, values, 1, 1)
    wo, wl = expect(codes, first, values)
    assert np.abs(lse.cpu().numpy() - wl).max() <= 700 * 2.0 ** -27 + 2.0 ** -21
    assert np.abs(out.cpu().numpy() - wo).max() <= 8 * 7 * (700 * 2.0 ** -27 + 2.0 ** -20)

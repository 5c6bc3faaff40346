"""Captured calls of the cache class: what a graph records runs again at every replay, when the
prefix has another length than at the capture."""
import math

import numpy as np
import pytest
import torch

from compressed_decode_attention_zkv_b200 import build as B
from compressed_decode_attention_zkv_b200 import zkv

pytestmark = pytest.mark.gpu
HQ, HKV, DIM, S = 8, 2, 128, 4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    B.build()
    zkv.lib()


def twins(seed, T, W=16, capacity=1024, n=2):
    """n caches of the same contents, and a source of fp16 numbers."""
    rng = np.random.default_rng(seed)
    new = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float16)).cuda()   # noqa: E731
    books = [torch.from_numpy((rng.standard_normal((HKV, S, 256, DIM)) * 0.4).astype(np.float32)).cuda() for _ in range(2)]
    k, v = new(2, HKV, T, DIM), new(2, HKV, T, DIM)
    caches = []
    for _ in range(n):
        c = zkv.RVQKVCache(*books, batch=2, capacity=capacity, window=W)
        c.prefill(k, v)
        caches.append(c)
    return caches, new


def same_state(a, b):
    for x in ("k_codes", "v_codes", "win_k", "win_v", "comp_len", "win_len", "win_head", "error_flag"):
        assert torch.equal(getattr(a, x), getattr(b, x)), x


def close(a, b):
    """Two correct results: scores below 12 in magnitude, so float32 forms that split the tokens
    otherwise differ by less than 2 (d + 24) 2^-24 12 of the largest value."""
    assert (a.double() - b.double()).abs().max().item() <= 3e-4 * (1 + b.abs().max().item())


def captured(f):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f()
    return g


def test_replayed_rounds_see_the_tokens_that_they_commit():
    """verify, note_weights and commit in one graph, replayed until the prefix is far longer than it
    was at the capture; then eager calls, and an eager evict between replays."""
    (a, b), new = twins(81, T=100)
    N = 6
    q, dk, dv = new(2, N, HQ, DIM), new(2, N, HKV, DIM), new(2, N, HKV, DIM)
    path = torch.arange(N, dtype=torch.int32, device="cuda").repeat(2, 1)
    count = torch.tensor([N, N - 1], dtype=torch.int32, device="cuda")
    for c in (a, b):                         # makes the totals, sets the kernels' attributes
        out, lse = c.verify(q, dk, dv)
        c.note_weights(q, lse)
        c.commit(dk, dv, path, count)
    got, got_lse = torch.zeros_like(out), torch.zeros_like(lse)

    def step():
        a.verify(q, dk, dv, out=got, lse=got_lse)
        a.note_weights(q, got_lse)
        a.commit(dk, dv, path, count)
    g = captured(step)

    def rounds(n):
        for _ in range(n):
            for x in (q, dk, dv):
                x.copy_(new(*x.shape))
            g.replay()
            want, want_lse = b.verify(q, dk, dv)
            b.note_weights(q, want_lse)
            b.commit(dk, dv, path, count)
            close(got, want)
            close(got_lse, want_lse)
            close(a.acc, b.acc)
            same_state(a, b)
    rounds(60)
    assert a.comp_len.max().item() == 84 + 61 * N and a.acc[0, :, 84 + 50 * N].min().item() > 0
    close(a.verify(q, dk, dv)[0], b.verify(q, dk, dv)[0])
    close(a.attend(q[:, 0].contiguous())[0], b.attend(q[:, 0].contiguous())[0])
    for c in (a, b):
        c.evict(100, recent=20)
    rounds(10)
    close(a.verify(q, dk, dv)[0], b.verify(q, dk, dv)[0])
    close(a.attend(q[:, 0].contiguous())[0], b.attend(q[:, 0].contiguous())[0])


def test_a_captured_evict_has_not_run_yet():
    (a, b), new = twins(82, T=700)
    q, dk, dv = new(2, 4, HQ, DIM), new(2, 4, HKV, DIM), new(2, 4, HKV, DIM)
    one = q[:, 0].contiguous()
    for c in (a, b):
        c.note_weights(q, c.verify(q, dk, dv)[1])
        c.attend(one)
        c.evict(684, recent=684)             # (keeps all; sets the kernel's attributes)
    g = captured(lambda: a.evict(200, recent=50))
    for _ in range(2):
        for x, y in zip(a.verify(q, dk, dv) + a.attend(one), b.verify(q, dk, dv) + b.attend(one)):
            assert torch.equal(x, y)
        assert torch.equal(a.note_weights(q, a.verify(q, dk, dv)[1]), b.note_weights(q, b.verify(q, dk, dv)[1]))
    g.replay()
    b.evict(200, recent=50)
    same_state(a, b)
    assert torch.equal(a.acc, b.acc)
    for x, y in zip(a.verify(q, dk, dv) + a.attend(one), b.verify(q, dk, dv) + b.attend(one)):
        close(x, y)


@pytest.mark.parametrize("how", ["append and attend", "step"])
def test_replayed_decoding_sees_the_tokens_that_it_appends(how):
    (a, b), new = twins(83, T=60)
    k, v, q = new(2, HKV, DIM), new(2, HKV, DIM), new(2, HQ, DIM)
    for c in (a, b):
        c.append(k, v)
        c.attend(q)
        c.step(k, v, q)
    got = torch.zeros(2, HQ, DIM, device="cuda")

    def one_step():
        if how == "step":
            a.step(k, v, q, out=got)
        else:
            a.append(k, v)
            a.attend(q, out=got)
    g = captured(one_step)
    for i in range(200):
        for x in (k, v, q):
            x.copy_(new(*x.shape))
        g.replay()
        want, _ = b.step(k, v, q)
        if i % 20 == 19:
            close(got, want)
    same_state(a, b)
    close(a.attend(q)[0], b.attend(q)[0])


def test_a_replayed_attend_sees_what_eager_calls_append():
    (a, b), new = twins(84, T=700, capacity=4096)
    k, v, q = new(2, HKV, DIM), new(2, HKV, DIM), new(2, HQ, DIM)
    first, _ = a.attend(q)
    got = torch.zeros(2, HQ, DIM, device="cuda")
    g = captured(lambda: a.attend(q, out=got))
    g.replay()
    assert torch.equal(got, first)
    long = new(2, HKV, 3500, DIM)
    for c in (a, b):
        c.prefill(long, long)
    g.replay()
    close(got, b.attend(q)[0])
    assert math.isfinite(got.sum().item())


def test_a_captured_prefill_is_counted_at_every_replay():
    (a, b), new = twins(85, T=300)
    k, v, q = new(2, HKV, 300, DIM), new(2, HKV, 300, DIM), new(2, HQ, DIM)
    g = captured(lambda: a.prefill(k, v))
    few = new(2, HKV, 40, DIM)
    a.prefill(few, few)
    g.replay()
    b.prefill(k, v)
    same_state(a, b)
    close(a.attend(q)[0], b.attend(q)[0])


def test_a_captured_attend_outlives_more_heads():
    """A graph of attend() keeps its workspace when later calls need a larger one."""
    (a, b), new = twins(86, T=500)
    q, wide = new(2, HKV, DIM), new(2, HKV * 4, DIM)       # one head per kv head, then four
    first, _ = a.attend(q)
    got = torch.zeros_like(first)
    g = captured(lambda: a.attend(q, out=got))
    size = a._ws.numel()
    a.attend(wide)
    assert a._ws.numel() > size
    # memory of that size that the call above may have given back, filled
    fill = [torch.full((size,), 165, dtype=torch.uint8, device="cuda") for _ in range(4)]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, first)
    for f in fill:
        assert (f == 165).all()


@pytest.mark.parametrize("Sk,Sv,Hq", [(4, 4, 8), (3, 2, 2), (1, 5, 4)])
def test_any_launch_length_gives_the_same_attention(Sk, Sv, Hq):
    """Launches sized for far less and far more than the lengths that they meet."""
    rng = np.random.default_rng(87)
    Bn, T, d = 3, 9008, 64
    c = lambda a: torch.from_numpy(a).cuda()   # noqa: E731
    books = [c((rng.standard_normal((1, s, 256, d)) * 0.4).astype(np.float32)) for s in (Sk, Sv)]
    kc, vc = (c(rng.integers(0, 256, (Bn, 1, T, s)).astype(np.uint8)) for s in (Sk, Sv))
    q, wk, wv = (c(rng.standard_normal(s).astype(np.float16)) for s in ((Bn, Hq, d), (Bn, 1, 16, d), (Bn, 1, 16, d)))
    comp, win = c(np.array([9001, 0, 1025], np.int32)), c(np.array([16, 3, 0], np.int32))
    args = (q, kc, vc, comp, *books, wk, wv, win)
    want, want_lse = zkv.rvq_decode_attn(*args)
    for n in (1, 1000, 5000, 9008):
        out, lse = zkv.rvq_decode_attn(*args, launch_len=n)
        close(out, want)
        close(lse, want_lse)
        assert n < 9008 or torch.equal(out, want)
    for n in (-1, 9009):
        with pytest.raises(zkv.ZkvError):
            zkv.rvq_decode_attn(*args, launch_len=n)


def pq_twins(seed, T, capacity):
    rng = np.random.default_rng(seed)
    new = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float16)).cuda()   # noqa: E731
    books = [torch.from_numpy(rng.standard_normal((HKV, 256, 4)).astype(np.float32)).cuda() for _ in range(2)]
    caches = [zkv.PQKVCache(*books, batch=2, capacity=capacity, window=16, head_dim=DIM) for _ in range(2)]
    k, v = new(2, HKV, T, DIM), new(2, HKV, T, DIM)
    for c in caches:
        c.prefill(k, v)
    return caches, new


@pytest.mark.parametrize("what", ["attend", "append and attend"])
def test_product_vq_replays_see_the_tokens_that_are_there(what):
    (a, b), new = pq_twins(88, T=60, capacity=4096)
    k, v, q = new(2, HKV, DIM), new(2, HKV, DIM), new(2, HQ, DIM)
    for c in (a, b):
        c.step(k, v, q)
    got = torch.zeros(2, HQ, DIM, device="cuda")

    def step():
        if what != "attend":
            a.append(k, v)
        a.attend(q, out=got)
    g = captured(step)
    for i in range(40):
        for x in (k, v, q):
            x.copy_(new(*x.shape))
        if what == "attend":
            a.append(k, v)
        g.replay()
        want, _ = b.step(k, v, q)
        close(got, want)
    same_state(a, b)
    long = new(2, HKV, 4000, DIM)
    for c in (a, b):
        c.prefill(long, long)
    g.replay()
    if what != "attend":
        b.append(k, v)
    close(got, b.attend(q)[0])
    g.replay()                               # and once more than eager calls know of
    if what != "attend":
        b.append(k, v)
    same_state(a, b)
    close(a.attend(q)[0], b.attend(q)[0])


def test_a_captured_product_vq_attend_outlives_more_heads():
    (a, b), new = pq_twins(89, T=500, capacity=1024)
    q, wide = new(2, HKV, DIM), new(2, HKV * 4, DIM)
    first, _ = a.attend(q)
    got = torch.zeros_like(first)
    g = captured(lambda: a.attend(q, out=got))
    size = a._ws.numel()
    a.attend(wide)
    assert a._ws.numel() > size
    fill = [torch.full((size,), 165, dtype=torch.uint8, device="cuda") for _ in range(4)]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, first)
    for f in fill:
        assert (f == 165).all()

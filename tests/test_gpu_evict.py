"""Eviction by accumulated attention weight on the GPU: weights against float64, the choice and the copies exactly.

Bar of the weights: a weight p = 2^(k (s - m)) / sum has relative error at most e = 2^-22 (2 A + 64), A = max
|k (s - m)| over the seen scores in units of log2 (the difference, the factor k and the product are rounded to fp32:
3 * 2^-24 A ln 2 < 2^-22 A, on the weight and on the sum; 2^-22 for each of the two or three ex2.approx; under 64
roundings in any addition chain of the sum), weights under 2^-126 may be flushed; then the sum over n_q queries in
fp32, and on the old sum three roundings, 2^-24 each: decay itself, which the call takes as an fp32 argument (0.9 is
off by 2^-25.4 of itself), decay * acc, and the final addition, which also rounds the new part."""
import math

import numpy as np
import pytest
import torch

from kv_quantization_b200 import _lib as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def accumulate(scores, scale, decay, acc, row_len=None, out=None):
    G, R, T = scores.shape
    out = torch.full((G, T), 7.0, device=DEV) if out is None else out
    ws = torch.empty(max(16, L.rq_evict_accumulate_workspace_bytes(G, R, T)), dtype=torch.uint8, device=DEV)
    L.rq_evict_accumulate(scores, G, R, T, scale, decay, acc, out, ws, row_len=row_len)
    return out


def check_accumulate(got, scores, scale, decay, acc, row_len=None):
    G, R, T = scores.shape
    s = scores.double().cpu()
    n = torch.full((G, R), T) if row_len is None else row_len.cpu().long().clamp(0, T)
    seen = torch.arange(T) < n[..., None]
    a = torch.where(seen, s * scale, -math.inf)
    p = torch.softmax(a, -1).nan_to_num(0.0)
    want = p.sum(1) + (decay * acc.double().cpu() if decay else 0.0)
    span = torch.where(seen & a.isfinite(), a.amax(-1, keepdim=True) - a, 0.0).amax(-1, keepdim=True) / math.log(2)
    e = 2.0 ** -22 * (2 * span.clamp_max(140.0) + 64)
    old = (decay * acc.double().cpu()).abs() if decay else 0.0
    tol = (p * e).sum(1) + R * 2.0 ** -24 * p.sum(1) + 3 * 2.0 ** -24 * old + 2.0 ** -23 * p.sum(1) + R * 2.0 ** -120
    err = (got.double().cpu() - want).abs()
    assert (err <= tol).all(), f"worst {float((err / tol).max()):.3f} of the bar"


@pytest.mark.parametrize("G,R,T", [(1, 1, 1), (2, 3, 5), (1, 1, 1023), (3, 4, 1024), (2, 7, 1025), (5, 32, 3001),
                                   (1, 70, 20011), (2, 300, 130), (300, 2, 66), (1, 2, 100003), (2, 5, 4096)])
@pytest.mark.parametrize("ragged", [False, True])
def test_accumulate(G, R, T, ragged):
    g = torch.Generator(device=DEV)
    g.manual_seed(G * R + T)
    scores = torch.randn(G, R, T, generator=g, device=DEV) * 11
    acc = torch.rand(G, T, generator=g, device=DEV)
    row_len = None
    if ragged:
        row_len = torch.randint(-1, T + 3, (G, R), generator=g, device=DEV, dtype=torch.int32)
        row_len[0, 0] = 0
        seen = torch.arange(T, device=DEV) < row_len[..., None]
        scores = torch.where(seen, scores, math.nan)            # what a query does not see may be anything
    got = accumulate(scores, 0.25, 0.9, acc, row_len)
    check_accumulate(got, scores, 0.25, 0.9, acc, row_len)
    again = accumulate(scores, 0.25, 0.9, acc, row_len)
    assert torch.equal(got, again)


def test_accumulate_in_place_and_without_history():
    scores = torch.randn(2, 4, 777, device=DEV)
    acc = torch.rand(2, 777, device=DEV)
    want = accumulate(scores, 1.0, 0.5, acc)
    io = acc.clone()
    accumulate(scores, 1.0, 0.5, io, out=io)
    assert torch.equal(io, want)
    fresh = accumulate(scores, 1.0, 0.0, None)
    check_accumulate(fresh, scores, 1.0, 0.0, acc)
    nan = torch.full_like(acc, math.nan)                       # decay 0 does not read the old sums
    assert torch.equal(accumulate(scores, 1.0, 0.0, nan), fresh)


def test_accumulate_no_queries():
    acc = torch.rand(3, 50, device=DEV)
    out = torch.empty(3, 50, device=DEV)
    L.rq_evict_accumulate(None, 3, 0, 50, 1.0, 0.5, acc, out, None)
    assert torch.equal(out, acc * 0.5)


def test_accumulate_special_scores():
    T = 1500
    scores = torch.randn(1, 5, T, device=DEV)
    scores[0, 0] = -math.inf                                   # a row that sees nothing but -inf adds nothing
    scores[0, 1, :T - 1] = -math.inf                           # all weight on the last token
    scores[0, 2] = torch.finfo(torch.float32).min              # the type's lowest value everywhere: uniform
    scores[0, 3] = 3e38
    scores[0, 3, 7] = -3e38
    scores[0, 4] = 0.0
    zero = torch.zeros(1, T, device=DEV)
    got = accumulate(scores, 1.0, 1.0, zero).double().cpu()[0]
    want = torch.full((T,), 2.0 / T, dtype=torch.float64)
    want += 1.0 / (T - 1)
    want[7] -= 1.0 / (T - 1)
    want[-1] += 1.0
    assert ((got - want).abs() <= 2.0 ** -16 * want).all()      # sums of 1500 ones in fp32 chains of under 64


@pytest.mark.parametrize("scale", [0.0, 1e-45])
@pytest.mark.parametrize("T", [3, 1500, 4096, 9001])
@pytest.mark.parametrize("ragged", [False, True])
def test_accumulate_with_a_zero_scale(scale, T, ragged):
    """Every score that a query sees weighs the same, but for -inf, which has no weight at any scale.  The weights are
    1 / n, n a whole number: the reciprocal and the sum over 5 queries round, 2^-24 each, and 1e-45 of a score of at
    most 100 moves no weight."""
    G, R = 3, 5
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    scores = (torch.randn(G, R, T, generator=g, device=DEV) * 11).clamp(-100, 100)
    scores[:, 1, ::3] = -math.inf
    scores[:, 2] = -math.inf                                    # adds nothing
    seen = torch.ones(G, R, T, dtype=torch.bool, device=DEV)
    row_len = None
    if ragged:
        row_len = torch.randint(1, T + 1, (G, R), generator=g, device=DEV, dtype=torch.int32)
        row_len[0, 0], row_len[1, 4] = 0, T
        seen = torch.arange(T, device=DEV) < row_len[..., None]
        scores = torch.where(seen, scores, math.nan)
    live = (seen & (scores != -math.inf)).double()
    want = (live / live.sum(-1, keepdim=True).clamp_min(1.0)).sum(1)
    acc = torch.rand(G, T, generator=g, device=DEV)
    got = accumulate(scores, scale, 0.0, None, row_len)
    assert ((got.double() - want).abs() <= 8 * 2.0 ** -24 * want).all()
    io = acc.clone()                                            # in place: the old sums are not lost
    accumulate(scores, scale, 1.0, io, row_len, out=io)
    assert ((io.double() - acc.double() - want).abs() <= 2.0 ** -24 * (acc + want) + 8 * 2.0 ** -24 * want).all()


def test_accumulate_far_offsets():
    """Scores past 2^31 elements and 2^32 bytes."""
    G, R, T = 9, 8, 1 << 25
    scores = torch.zeros(G, R, T, device=DEV)
    scores[8, 7, T - 5:] = 20.0
    acc = torch.zeros(G, T, device=DEV)
    got = accumulate(scores, 1.0, 1.0, acc)
    big = math.exp(20.0)
    want = 7.0 / T + big / (5 * big + T - 5)
    assert got[8, T - 1].item() == pytest.approx(want, rel=1e-4)
    assert got[8, 0].item() == pytest.approx(7.0 / T + 1.0 / (5 * big + T - 5), rel=1e-4)
    assert got[0, T - 1].item() == pytest.approx(8.0 / T, rel=1e-4)


# ------------------------------------------------------------------ select

def select_reference(acc, n, keep, sink, recent):
    acc = acc[:n].astype(np.float64)
    acc[np.isnan(acc)] = -np.inf
    nan_last = np.isnan(acc)
    t = np.arange(n)
    forced = (t < sink) | (t >= n - recent)
    order = sorted(range(n), key=lambda i: (not forced[i], bool(nan_last[i]), -acc[i], i))
    return np.sort(np.array(order[:keep], dtype=np.int64))


def check_select(acc, keep, sink=0, recent=0, lens=None):
    G, T = acc.shape
    idx = torch.full((G, keep), 99, dtype=torch.int32, device=DEV)
    count = torch.full((G,), 99, dtype=torch.int32, device=DEV)
    L.rq_evict_select(acc, G, T, keep, idx, count, length=lens, n_sink=sink, n_recent=recent)
    assert L.rq_last_launch() == "select_kernel"
    a, i, c = acc.cpu().numpy(), idx.cpu().numpy(), count.cpu().numpy()
    for g in range(G):
        n = T if lens is None else int(min(max(int(lens[g]), 0), T))
        want = select_reference(a[g], n, keep, sink, recent)
        assert c[g] == len(want) == min(keep, n)
        assert np.array_equal(i[g, :c[g]], want), f"group {g}"
        assert (i[g, c[g]:] == -1).all()


@pytest.mark.parametrize("G,T,keep", [(1, 1, 1), (2, 5, 3), (3, 1000, 500), (2, 1024, 1), (2, 1025, 1024), (1, 4097, 4000),
                                      (3, 8192, 100), (2, 8193, 8192), (1, 20011, 7777), (1, 70001, 33333),
                                      (150, 300, 120), (1, 131072, 20001), (1, 200003, 50000), (2, 40, 64)])
@pytest.mark.parametrize("kind", ["random", "ties", "equal"])
def test_select(G, T, keep, kind):
    g = torch.Generator(device=DEV)
    g.manual_seed(T + keep)
    acc = torch.rand(G, T, generator=g, device=DEV).pow(6)
    if kind == "ties":
        acc = (acc * 8).floor()
    if kind == "equal":
        acc = torch.full_like(acc, 0.25)
    check_select(acc, keep)
    lens = torch.randint(0, T + 1, (G,), generator=g, device=DEV, dtype=torch.int32)
    if G > 1:
        lens[0], lens[1] = 0, T + 5                             # none, and more than the cache holds
    check_select(acc, keep, sink=min(4, keep // 2), recent=keep // 3, lens=lens)


def test_select_special_sums():
    T = 3001
    acc = torch.rand(4, T, device=DEV) - 0.5                   # signs
    acc[0, ::3] = math.nan
    acc[1, ::2] = math.inf
    acc[1, 1::4] = -math.inf
    acc[2] = 0.0
    acc[2, ::2] = -0.0                                          # equal to +0: ties go to the lowest index
    acc[3] = math.nan
    for keep in (1, 999, 2999):
        check_select(acc, keep)
        check_select(acc, keep, recent=1)
    check_select(torch.full((1, 50), -math.inf, device=DEV), 7)


def test_select_all_forced():
    acc = torch.rand(2, 500, device=DEV)
    check_select(acc, 20, sink=8, recent=12)
    check_select(acc, 20, sink=20)
    check_select(acc, 20, recent=20, lens=torch.tensor([30, 11], dtype=torch.int32, device=DEV))


# ------------------------------------------------------------------ gather

@pytest.mark.parametrize("G,T,keep", [(1, 1, 1), (3, 1000, 500), (2, 321, 64), (5, 77, 65), (1, 20011, 5000)])
def test_gather(G, T, keep):
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    widths = (1, 2, 3, 4, 6, 8, 16, 32, 48, 63, 64, 128, 260)
    src = [torch.randint(0, 256, (G, T, w), generator=g, device=DEV, dtype=torch.uint8) for w in widths]
    T_dst = keep + 3
    dst = [torch.full((G, T_dst, w), 9, device=DEV, dtype=torch.uint8) for w in widths]
    idx = torch.stack([torch.randperm(T, generator=g, device=DEV)[:keep].sort().values if keep <= T else
                       torch.arange(keep, device=DEV) for _ in range(G)]).int()
    count = torch.randint(0, keep + 1, (G,), generator=g, device=DEV, dtype=torch.int32)
    count[0] = keep
    idx[0, keep // 2] = T if keep > 2 else idx[0, keep // 2]    # outside: its row is left
    L.rq_evict_gather(idx, count, G, keep, T, list(zip(src, dst)), T_dst=T_dst)
    assert L.rq_last_launch() == "gather_kernel"
    for s, d, w in zip(src, dst, widths):
        want = torch.full_like(d, 9)
        for b in range(G):
            for j in range(int(count[b])):
                t = int(idx[b, j])
                if 0 <= t < T:
                    want[b, j] = s[b, t]
            if w > 3:
                break                                           # one group is enough for most widths
        assert torch.equal(d[:1] if w > 3 else d, want[:1] if w > 3 else want)


@pytest.mark.parametrize("G,T,keep", [(33, 5001, 4099), (3, 70001, 50021), (1, 131072, 131072)])
def test_gather_of_long_caches(G, T, keep):
    """keep * G of 2^17 and more (256 rows a block) with a remainder, every group, in each width of access."""
    assert keep * G >= 256 * 512
    g = torch.Generator(device=DEV)
    g.manual_seed(keep)
    widths = (1, 2, 3, 4, 8, 24, 32, 48, 64)
    src = [torch.randint(0, 256, (G, T, w), generator=g, device=DEV, dtype=torch.uint8) for w in widths]
    T_dst = keep + 5
    dst = [torch.full((G, T_dst, w), 9, device=DEV, dtype=torch.uint8) for w in widths]
    idx = torch.stack([torch.randperm(T, generator=g, device=DEV)[:keep].sort().values for _ in range(G)]).int()
    count = torch.randint(0, keep + 1, (G,), generator=g, device=DEV, dtype=torch.int32)
    count[0] = keep
    outside = torch.rand(G, keep, generator=g, device=DEV) < 0.01
    idx = torch.where(outside, torch.where(idx % 2 == 0, -idx - 1, idx + T), idx)
    L.rq_evict_gather(idx, count, G, keep, T, list(zip(src, dst)), T_dst=T_dst)
    live = (torch.arange(keep, device=DEV) < count[:, None]) & ~outside
    rows = torch.where(live, idx, 0).long()[..., None]
    for s, d, w in zip(src, dst, widths):
        want = torch.full_like(d, 9)
        want[:, :keep] = torch.where(live[..., None], torch.gather(s, 1, rows.expand(-1, -1, w)), want[:, :keep])
        assert torch.equal(d, want), f"width {w}"


def test_gather_far_offsets():
    """Records past 2^32 bytes; the same index twice."""
    T = (1 << 32) // 512 + 100
    src = torch.zeros(1, T, 512, dtype=torch.uint8, device=DEV)
    src[0, T - 1], src[0, T - 50] = 3, 5
    dst = torch.zeros(1, 4, 512, dtype=torch.uint8, device=DEV)
    idx = torch.tensor([[0, T - 50, T - 1, T - 1]], dtype=torch.int32, device=DEV)
    count = torch.tensor([4], dtype=torch.int32, device=DEV)
    L.rq_evict_gather(idx, count, 1, 4, T, [(src, dst)])
    assert dst[0, :, 0].tolist() == [0, 5, 3, 3] and (dst[0, 3] == 3).all()


def test_select_and_gather_in_a_graph_on_two_streams():
    """A captured step replayed on new sums; the same step on another stream with its own buffers."""
    G, T, keep = 4, 5000, 700
    acc = torch.rand(G, T, device=DEV)
    codes = torch.randint(0, 256, (G, T, 64), device=DEV, dtype=torch.uint8)

    def step(idx, count, dst, stream=None):
        L.rq_evict_select(acc, G, T, keep, idx, count, n_sink=2, n_recent=5, stream=stream)
        L.rq_evict_gather(idx, count, G, keep, T, [(codes, dst)], stream=stream)

    bufs = [(torch.empty(G, keep, dtype=torch.int32, device=DEV), torch.empty(G, dtype=torch.int32, device=DEV),
             torch.zeros(G, keep, 64, dtype=torch.uint8, device=DEV)) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*bufs[0])
    acc.copy_(torch.rand(G, T, device=DEV))
    torch.cuda.synchronize()
    graph.replay()
    step(*bufs[1], stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    for a, b in zip(*bufs):
        assert torch.equal(a, b)
    for g in range(G):
        assert torch.equal(bufs[0][2][g], codes[g, bufs[0][0][g].long()])

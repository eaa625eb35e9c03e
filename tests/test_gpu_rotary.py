"""rq_rotary on the GPU against a float64 rotation.

Bar, per value: |got - want| <= eps/2 |want| + 2^-20 scale (|a| + |b|) + 2^-25, eps the 16-bit type's: half a step of
the stored value (2^-25 for fp16 subnormals), and for each of the two products in fp32: the angle (the top 32 bits of
the turn rounded to 24: pi 2^-24; position * 2^-64 turns for the fixed-point frequency), 1 ulp of sincospif, the
scale's and the product's and the sum's roundings, each 2^-24 or 2^-23: together under 2^-20 of the pair's magnitude.
"""
import numpy as np
import pytest
import torch

from kv_quantization_b200 import _lib as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def reference(x, pos, freq, rot, style, scale, inverse):
    """Float64 result and the magnitude |a| + |b| of every value's pair (0 where copied)."""
    x = x.double().cpu().numpy()
    # the angle in turns, in extended precision, reduced before it is rounded to float64
    f = np.asarray(freq, np.longdouble)[: rot // 2] / (2 * np.longdouble("3.14159265358979323846264338327950288"))
    p = pos.cpu().numpy().astype(np.longdouble)[..., None]
    turn = p * f
    turn = (turn - np.rint(turn)).astype(np.float64)
    c, s = np.cos(2 * np.pi * turn)[:, :, None] * scale, np.sin(2 * np.pi * turn)[:, :, None] * scale
    if inverse:
        s = -s
    ia = np.arange(rot // 2) if style == L.RQ_ROPE_HALF else np.arange(0, rot, 2)
    ib = ia + rot // 2 if style == L.RQ_ROPE_HALF else ia + 1
    out, mag = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return out, mag


def check(got, x, pos, freq, rot, style, scale, inverse):
    want, mag = reference(x, pos, freq, rot, style, scale, inverse)
    tol = torch.finfo(x.dtype).eps / 2 * np.abs(want) + 2.0 ** -20 * abs(scale) * mag + 2.0 ** -25
    tol[..., rot:] = 0.0                                        # copied values are copied
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), f"worst {np.nanmax(err / np.maximum(tol, 1e-300)):.3f} of the bar"


def make(B, n, H, d, dtype, seed, start=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(B, n, H, d, generator=g, device=DEV).to(dtype)
    pos = start + torch.arange(n, device=DEV).expand(B, n) + torch.arange(B, device=DEV)[:, None] * 7
    return x, pos.contiguous()


@pytest.mark.parametrize("style", [L.RQ_ROPE_HALF, L.RQ_ROPE_INTERLEAVED])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,n,H,d,rot", [(1, 1, 1, 128, 128), (2, 5, 3, 128, 64), (3, 17, 8, 96, 32), (1, 33, 5, 80, 40),
                                         (2, 3, 2, 64, 20), (1, 9, 7, 10, 6), (1, 2, 1, 2, 2), (2, 4, 40, 512, 512),
                                         (1, 3, 2, 510, 510), (1, 700, 40, 128, 128), (1, 5, 2, 512, 2),
                                         (300, 1, 3, 128, 128)])
def test_against_float64(B, n, H, d, rot, dtype, style):
    x, pos = make(B, n, H, d, dtype, 3, start=1000)
    freq, _ = L.rq_rotary_frequencies(rot)
    out = torch.empty_like(x)
    L.rq_rotary(x, out, pos, freq, rot, style)
    assert L.rq_last_launch() == "rotary_kernel"
    check(out, x, pos, freq, rot, style, 1.0, False)


@pytest.mark.parametrize("start", [0, 1 << 20, (1 << 31) + 12345, 1 << 40, -5, -(1 << 33)])
def test_far_and_negative_positions(start):
    x, pos = make(2, 40, 4, 128, torch.float16, 5, start=start)
    freq, _ = L.rq_rotary_frequencies(128)
    out = torch.empty_like(x)
    L.rq_rotary(x, out, pos, freq, 128, L.RQ_ROPE_HALF)
    # the fixed-point frequency is off by at most 2^-65 turns and the float64 one by 2^-53 of itself, which the
    # reference shares: at 2^40 the former is 2^-25 turns, under the bar's share for the angle
    check(out, x, pos, freq, 128, L.RQ_ROPE_HALF, 1.0, False)


@pytest.mark.parametrize("kind,args", [(L.RQ_ROPE_YARN, (16.0, 4096.0, 32.0, 1.0)), (L.RQ_ROPE_BANDED, (8.0, 8192.0, 1.0, 4.0)),
                                       (L.RQ_ROPE_NTK, (4.0,)), (L.RQ_ROPE_LINEAR, (4.0,))])
def test_scaled_contexts(kind, args):
    x, pos = make(2, 65, 3, 128, torch.bfloat16, 6, start=100000)
    freq, scale = L.rq_rotary_frequencies(64, 10000.0, kind, *args)
    out = torch.empty_like(x)
    L.rq_rotary(x, out, pos, freq, 64, L.RQ_ROPE_INTERLEAVED, scale=scale)
    check(out, x, pos, freq, 64, L.RQ_ROPE_INTERLEAVED, scale, False)


def test_two_tensors_strides_and_batch_shared_positions():
    """Query and key heads inside one projection output, written per head ([B][H][n][d]); positions of batch stride 0."""
    B, n, H, KV, d = 3, 37, 6, 2, 128
    qkv = torch.randn(B, n, H + 2 * KV, d, device=DEV).bfloat16()
    q, k = qkv[:, :, :H], qkv[:, :, H:H + KV]
    pos = torch.randint(0, 5000, (n,), device=DEV).expand(B, n)
    freq, _ = L.rq_rotary_frequencies(d)
    qo = torch.empty(B, H, n, d, device=DEV, dtype=torch.bfloat16)
    ko = torch.empty(B, KV, n, d, device=DEV, dtype=torch.bfloat16)
    L.rq_rotary(q, qo.transpose(1, 2), pos, freq, d, L.RQ_ROPE_HALF, x2=k, out2=ko.transpose(1, 2))
    check(qo.transpose(1, 2), q, pos, freq, d, L.RQ_ROPE_HALF, 1.0, False)
    check(ko.transpose(1, 2), k, pos, freq, d, L.RQ_ROPE_HALF, 1.0, False)
    # in place in the projection output: the same bits, the value heads untouched
    keep = qkv.clone()
    L.rq_rotary(q, q, pos, freq, d, L.RQ_ROPE_HALF, x2=k, out2=k)
    assert torch.equal(q, qo.transpose(1, 2)) and torch.equal(k, ko.transpose(1, 2))
    assert torch.equal(qkv[:, :, H + KV:], keep[:, :, H + KV:])


def test_odd_strides_and_alignment():
    """Views whose strides and base suit only narrower accesses give the same bits as contiguous tensors."""
    x, pos = make(2, 9, 4, 64, torch.float16, 7)
    freq, _ = L.rq_rotary_frequencies(32)
    want = torch.empty_like(x)
    L.rq_rotary(x, want, pos, freq, 32, L.RQ_ROPE_HALF)
    for pad, off in ((4, 4), (2, 2), (1, 1), (3, 0), (8, 4), (8, 2), (8, 1)):
        buf = torch.zeros(2, 9, 4, 64 + pad, device=DEV, dtype=torch.float16)
        v = buf[..., off:off + 64]
        v.copy_(x)
        out = torch.full((2, 9, 4, 64 + pad), 7.0, device=DEV, dtype=torch.float16)
        L.rq_rotary(v, out[..., off:off + 64], pos, freq, 32, L.RQ_ROPE_HALF)
        assert torch.equal(out[..., off:off + 64], want)
        assert (out[..., :off] == 7).all() and (out[..., off + 64:] == 7).all()


def test_partly_rotated_in_place_leaves_the_rest():
    x, pos = make(1, 50, 3, 96, torch.bfloat16, 8)
    freq, _ = L.rq_rotary_frequencies(32)
    want = torch.empty_like(x)
    L.rq_rotary(x, want, pos, freq, 32, L.RQ_ROPE_INTERLEAVED)
    y = x.clone()
    L.rq_rotary(y, y, pos, freq, 32, L.RQ_ROPE_INTERLEAVED)
    assert torch.equal(y, want) and torch.equal(y[..., 32:], x[..., 32:])


@pytest.mark.parametrize("style", [L.RQ_ROPE_HALF, L.RQ_ROPE_INTERLEAVED])
def test_gradient(style):
    """The inverse call on the output's gradient is the gradient: of the formula (autograd in float64) and by
    differences of the forward formula."""
    B, n, H, d, rot = 2, 7, 3, 32, 24
    freq, scale = L.rq_rotary_frequencies(rot, 10000.0, L.RQ_ROPE_YARN, 8.0, 2048.0, 32.0, 1.0)
    x, pos = make(B, n, H, d, torch.float16, 9, start=77)
    go = torch.randn(B, n, H, d, device=DEV).half()
    got = torch.empty_like(go)
    L.rq_rotary(go, got, pos, freq, rot, style, scale=scale, inverse=True)

    def forward(v):
        ang = pos.double()[:, :, None, None] * torch.from_numpy(freq).to(DEV)
        c, s = ang.cos() * scale, ang.sin() * scale
        a, b = (v[..., :rot // 2], v[..., rot // 2:rot]) if style == L.RQ_ROPE_HALF else (v[..., 0:rot:2], v[..., 1:rot:2])
        u, w = a * c - b * s, b * c + a * s
        r = torch.cat([u, w], -1) if style == L.RQ_ROPE_HALF else torch.stack([u, w], -1).flatten(-2)
        return torch.cat([r, v[..., rot:]], -1)

    v = x.double().requires_grad_()
    (forward(v) * go.double()).sum().backward()
    tol = 2.0 ** -11 * v.grad.abs() + 2.0 ** -20 * scale * 2 * go.double().abs().amax() + 2.0 ** -25
    assert ((got.double() - v.grad).abs() <= tol).all()
    e = torch.randn_like(v)
    diff = ((forward(v.detach() + e) - forward(v.detach() - e)) * go.double()).sum() / 2
    assert torch.allclose((got.double() * e).sum(), diff, rtol=0, atol=float((tol * e.abs()).sum()))


def test_special_values_and_idle_lanes():
    x = torch.zeros(1, 4, 2, 128, device=DEV, dtype=torch.float16)
    x[0, 0, 0, 0], x[0, 1, 1, 5], x[0, 2, 0, 70] = float("inf"), float("nan"), 65504.0
    pos = torch.zeros(1, 4, device=DEV, dtype=torch.int64)
    freq, _ = L.rq_rotary_frequencies(128)
    out = torch.empty_like(x)
    L.rq_rotary(x, out, pos, freq, 128, L.RQ_ROPE_HALF)
    assert out[0, 2, 0, 70] == 65504.0 and torch.isinf(out[0, 0, 0, 0]) and torch.isnan(out[0, 1, 1, 5])
    bad = ~torch.isfinite(out)
    assert set(map(tuple, bad.nonzero().tolist())) <= {(0, 0, 0, 0), (0, 0, 0, 64), (0, 1, 1, 5), (0, 1, 1, 69)}


def test_stream_and_graph():
    x, pos = make(2, 64, 8, 128, torch.bfloat16, 11)
    freq, _ = L.rq_rotary_frequencies(128)
    want = torch.empty_like(x)
    L.rq_rotary(x, want, pos, freq, 128, L.RQ_ROPE_HALF)
    side = torch.cuda.Stream()
    out = torch.zeros_like(x)
    torch.cuda.synchronize()
    L.rq_rotary(x, out, pos, freq, 128, L.RQ_ROPE_HALF, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(graph):
        L.rq_rotary(x, out, pos, freq, 128, L.RQ_ROPE_HALF)
    x.mul_(2)
    graph.replay()
    assert torch.equal(out, want * 2)

"""qjl_tree_attention on the GPU against float64 attention over the reconstructed cache and the drafted tokens.

Bars (the arithmetic is qjl_attention's, whose tests derive them): every output within
  (2 (e^(2 e) - 1) + 2^-9) V + 2^-8 |out|,   e = 1e-3 max |scale s| over what the row sees of the cache,
V = the largest value norm that the row sees: a logit error of at most e (the estimator's 1e-3 bar) moves a convex
combination by at most twice the relative weight error times the values' spread; 2^-9 is the two fp16 roundings of a
cached product (and far above the fp32 errors of the drafted part); 2^-8 = eps(bf16) / 2, the output's rounding.
Over a whole case ||got - want|| <= (2e-3 + 2^-8) ||want||.  Rows that see nothing are exactly 0.
"""
import math

import numpy as np
import pytest
import torch

from kv_quantization_b200 import _lib as L
from tests.test_gpu_attention import compress

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 128
KERNELS = "tree_prologue_kernel,tree_attention_kernel,tree_combine_kernel"


def hadamard():
    h = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def bits_of(x):
    return np.unpackbits(x.cpu().numpy(), axis=-1, bitorder="little")


def rebuild(codes, norms, rows, bits, layout, seed, cent):
    """Float64 reconstruction of blocks (H and the diagonal restated here)."""
    if layout == L.RQ_CODES_INT8:
        c = codes.reshape(rows, D).cpu().numpy().astype(np.int64)
    else:
        c = bits_of(codes.reshape(rows, -1)).reshape(rows, D, bits).astype(np.int64) @ (1 << np.arange(bits))
    x = torch.from_numpy(np.asarray(cent, np.float64)[c]).to(DEV) @ hadamard() / D
    mask = (1 << 64) - 1
    s = []
    for w in range(2):
        z = (seed + (w + 1) * 0x9E3779B97F4A7C15) & mask
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        z ^= z >> 31
        s += [-1.0 if z >> j & 1 else 1.0 for j in range(64)]
    return x * torch.tensor(s, dtype=torch.float64, device=DEV) * norms.view(torch.float16).double().reshape(-1, 1)


def vectors(c, G, T, m, kbits, vbits):
    """Estimator vectors of the keys and reconstructed values, [G, T, D] float64."""
    sg = torch.from_numpy(bits_of(c["signs"].reshape(G * T, m // 8))).to(DEV).double() * 2 - 1
    k = sg @ c["S"].double() * (math.sqrt(math.pi / 2) / m) * c["sk"].view(torch.float16).double().reshape(-1, 1)
    if c["codes"] is not None:
        k = k + rebuild(c["codes"], c["norms"], G * T, kbits, L.RQ_CODES_PACKED, c["kseed"], c["kc"])
    v = rebuild(c["vcodes"], c["vnorms"], G * T, vbits, c["vlayout"], c["vseed"], c["vc"])
    return k.reshape(G, T, D), v.reshape(G, T, D)


def sees_of(mask, B, n):
    if mask is None:
        return torch.ones(n, n, device=DEV).tril().bool().expand(B, n, n)
    b = (mask.unsqueeze(-1) >> torch.arange(64, device=DEV)) & 1
    return b.flatten(-2)[..., :n].bool().expand(B, n, n)


def random_tree(B, n, seed, empty_row=None):
    rng = np.random.RandomState(seed)
    sees = np.zeros((B, n, -(-n // 64) * 64), np.uint8)
    for b in range(B):
        for i in range(n):
            if i:
                sees[b, i] = sees[b, rng.randint(0, i)]
            sees[b, i, i] = 1
    if empty_row is not None:
        sees[:, empty_row] = 0
    return torch.from_numpy(np.packbits(sees, axis=-1, bitorder="little").view(np.int64).copy()).to(DEV)


def run(c, q, kn, vn, mask, m, T, lens, kbits, vbits, scale, out=None, ws=None, stream=None):
    B, n, H, _ = q.shape
    KV = kn.shape[2]
    if out is None:
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    if ws is None:
        ws = torch.empty(L.qjl_tree_attention_workspace_bytes(B, KV, H // KV, n, D, m, T), dtype=torch.uint8, device=DEV)
    kw = {}
    if c["codes"] is not None:
        kw = dict(codes=c["codes"], norms=c["norms"], bits=kbits, use_signs=1, sign_seed=c["kseed"], centroids=c["kc"])
    L.qjl_tree_attention(q, kn, vn, mask, m, c["S"], c["signs"], c["sk"], T, lens, c["vcodes"], c["vnorms"], vbits,
                         c["vc"], out, ws, scale, v_layout=c["vlayout"], v_use_signs=1, v_sign_seed=c["vseed"],
                         stream=stream, **kw)
    return out


def check(got, kt, vt, q, kn, vn, mask, lens, scale):
    B, n, H, _ = q.shape
    KV = kn.shape[2]
    rep, T = H // KV, kt.shape[1]
    sees = sees_of(mask, B, n)
    num = den = 0.0
    for g in range(B * KV):
        b, kv = divmod(g, KV)
        ln = T if lens is None else int(min(max(int(lens[g]), 0), T))
        qr = q[b, :, kv * rep:(kv + 1) * rep].double()
        vis = sees[b]
        kd = torch.where(vis.any(0)[:, None], kn[b, :, kv].double(), 0.0)
        vd = torch.where(vis.any(0)[:, None], vn[b, :, kv].double(), 0.0)
        sc = torch.einsum("nrd,td->nrt", qr, kt[g, :ln]) * scale
        sd = torch.einsum("nrd,td->nrt", qr, kd) * scale
        a = torch.cat([sc, sd.masked_fill(~vis[:, None], -math.inf)], -1)
        want = torch.softmax(a, -1).nan_to_num(0.0) @ torch.cat([vt[g, :ln], vd])
        nothing = ~vis.any(-1) & (ln == 0)
        e = 1e-3 * (sc.abs().amax(-1) if ln else torch.zeros_like(sd[..., 0]))
        V = torch.cat([vt[g, :ln], vd]).norm(dim=-1).amax()
        tol = ((2 * (torch.exp(2 * e) - 1) + 2.0 ** -9) * V)[..., None] + 2.0 ** -8 * want.abs()
        have = got[b, :, kv * rep:(kv + 1) * rep].double()
        assert (have[nothing] == 0).all()
        err = (have - want).abs()
        assert (err <= tol).all(), f"group {g}: worst {float((err / tol).max()):.3f} of the bar"
        num += float((err ** 2).sum())
        den += float((want ** 2).sum())
    assert math.sqrt(num) <= (2e-3 + 2.0 ** -8) * math.sqrt(den), f"relative L2 {math.sqrt(num / max(den, 1e-300)):.2e}"


def drafted(B, n, KV, rep, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return [torch.randn(B, n, h, D, generator=g, device=DEV).bfloat16() for h in (KV * rep, KV, KV)]


CASES = [  # B, KV, rep, nodes, T, m, key bits (0: pure sketch), value bits
    (1, 1, 1, 1, 1, 128, 0, 4), (2, 2, 4, 1, 1000, 256, 0, 4), (1, 2, 4, 8, 128, 256, 0, 4), (2, 1, 3, 11, 129, 128, 2, 3),
    (1, 1, 4, 16, 777, 128, 3, 2), (1, 2, 5, 13, 513, 64, 4, 4), (1, 1, 8, 16, 1300, 256, 0, 4), (1, 1, 4, 33, 640, 256, 1, 4),
    (1, 1, 4, 65, 500, 128, 0, 8), (1, 1, 2, 130, 300, 512, 0, 3), (1, 1, 1, 7, 400, 512, 2, 4), (3, 1, 7, 5, 255, 192, 0, 1),
    (1, 1, 16, 8, 2000, 256, 4, 8), (40, 4, 2, 3, 200, 128, 0, 4), (1, 1, 2, 32, 20011, 256, 0, 4), (1, 1, 4, 70, 9000, 256, 0, 4),
]


@pytest.mark.parametrize("B,KV,rep,n,T,m,kbits,vbits", CASES)
@pytest.mark.parametrize("ragged", [False, True])
def test_against_float64(B, KV, rep, n, T, m, kbits, vbits, ragged):
    G = B * KV
    c = compress(G, T, D, m, kbits, vbits, 300 + T % 97, kbits > 0,
                 vlayout=L.RQ_CODES_INT8 if vbits == 8 else L.RQ_CODES_PACKED)
    q, kn, vn = drafted(B, n, KV, rep, T)
    mask, lens = None, None
    if ragged:
        mask = random_tree(B, n, T)
        lens = torch.tensor([(T * (i + 1) * 37 // 101) % (T + 1) for i in range(G)], dtype=torch.int32, device=DEV)
        lens[-1] = T + 9                                       # more than the capacity: all of it
        if G > 1:
            lens[0] = 0
    scale = 1 / math.sqrt(D)
    got = run(c, q, kn, vn, mask, m, T, lens, kbits, vbits, scale)
    assert L.rq_last_launch() == KERNELS
    torch.cuda.synchronize()
    assert L.rq_device_error(True) == 0
    kt, vt = vectors(c, G, T, m, kbits, vbits)
    check(got, kt, vt, q, kn, vn, mask, lens, scale)
    again = run(c, q, kn, vn, mask, m, T, lens, kbits, vbits, scale)
    assert torch.equal(got, again)


@pytest.mark.parametrize("rows,m,kbits,vbits", [(30, 256, 0, 4), (39, 128, 2, 3), (60, 192, 0, 4), (64, 512, 4, 8), (100, 256, 0, 4),
                                                (128, 256, 3, 2), (32, 512, 1, 4), (33, 64, 2, 4)])
def test_many_tiles_per_cta(rows, m, kbits, vbits):
    """Enough cached tokens that every CTA runs tens of tiles and its buffers wrap many times, in several row blocks
    and groups; sampled groups against float64."""
    B, KV, T = 24, 2, 20011
    c = compress(B * KV, T, D, m, kbits, vbits, 400 + rows, kbits > 0,
                 vlayout=L.RQ_CODES_INT8 if vbits == 8 else L.RQ_CODES_PACKED)
    q, kn, vn = drafted(B, rows, KV, 1, rows)
    lens = torch.tensor([T - 97 * i for i in range(B * KV)], dtype=torch.int32, device=DEV)
    scale = 1 / math.sqrt(D)
    got = run(c, q, kn, vn, None, m, T, lens, kbits, vbits, scale)
    torch.cuda.synchronize()
    assert L.rq_device_error(True) == 0
    for b in (0, 11, B - 1):
        part = {k: (v[b * KV * (v.shape[0] // (B * KV)):(b + 1) * KV * (v.shape[0] // (B * KV))]
                    if isinstance(v, torch.Tensor) and k not in ("k", "v", "S") else v) for k, v in c.items()}
        kt, vt = vectors(part, KV, T, m, kbits, vbits)
        check(got[b:b + 1], kt, vt, q[b:b + 1], kn[b:b + 1], vn[b:b + 1], None, lens[b * KV:(b + 1) * KV], scale)
    again = run(c, q, kn, vn, None, m, T, lens, kbits, vbits, scale)
    assert torch.equal(got, again)


@pytest.mark.parametrize("n,rep", [(5, 4), (10, 4), (20, 4), (40, 4)])
def test_scores_that_keep_growing(n, rep):
    """Keys ever longer along the query: every tile passes the running reference, by a little or by a lot."""
    T, m, KV = 2600, 256, 2
    q, kn, vn = drafted(1, n, KV, rep, 5)
    base = q[0, 0, ::rep].double()                             # [KV, D]
    grow = torch.linspace(0.0, 6.0, T, device=DEV).double() ** 2 / 6
    k = (base[:, None] * grow[None, :, None] + torch.randn(KV, T, D, device=DEV, dtype=torch.float64)).bfloat16()
    c = compress(KV, T, D, m, 0, 4, 11, False, k=k.reshape(-1))
    scale = 1 / math.sqrt(D)
    got = run(c, q, kn, vn, None, m, T, None, 0, 4, scale)
    kt, vt = vectors(c, KV, T, m, 0, 4)
    logits = torch.einsum("nhd,htd->nht", q[0].double()[:, ::rep], kt) * scale
    assert float(logits.amax() - logits[..., :128].amax()) > 20  # the references move (2^7 is 4.9)
    check(got, kt, vt, q, kn, vn, None, None, scale)


def test_agrees_with_qjl_attention():
    """With nodes that see no drafted token, the cached part is qjl_attention's."""
    G, T, m, n = 3, 1500, 256, 8
    c = compress(G, T, D, m, 2, 4, 21, True)
    q, kn, vn = drafted(G, n, 1, 4, 22)
    mask = torch.zeros(1, n, 1, dtype=torch.int64, device=DEV)
    kn.fill_(math.nan)                                         # hidden: never read into a result
    vn.fill_(math.inf)
    got = run(c, q, kn, vn, mask, m, T, None, 2, 4, 0.09)
    want = torch.empty(G, n * 4, D, device=DEV)
    ws = torch.empty(L.qjl_attention_workspace_bytes(G, n * 4, D, m, T) // 4 + 4, device=DEV)
    L.qjl_attention(q.reshape(G, n * 4, D).contiguous(), G, n * 4, D, m, c["S"], c["signs"], c["sk"], T, c["vcodes"],
                    c["vnorms"], 4, c["vc"], want, ws, 0.09, codes=c["codes"], norms=c["norms"], bits=2, use_signs=1,
                    sign_seed=c["kseed"], centroids=c["kc"], v_use_signs=1, v_sign_seed=c["vseed"])
    d = got.float().reshape(G, n * 4, D) - want
    # both within 2e-3 of float64 (their own bars) and one rounding to bf16
    assert float(d.norm()) <= (2 * 2e-3 + 2.0 ** -8) * float(want.norm())


def test_empty_cache_and_empty_rows():
    B, n, KV, rep, m = 2, 6, 2, 2, 128
    q, kn, vn = drafted(B, n, KV, rep, 31)
    c = compress(B * KV, 64, D, m, 0, 4, 32, False)
    mask = random_tree(B, n, 33, empty_row=3)
    kt, vt = vectors(c, B * KV, 64, m, 0, 4)
    lens = torch.zeros(B * KV, dtype=torch.int32, device=DEV)
    got = run(c, q, kn, vn, mask, m, 64, lens, 0, 4, 0.1)
    assert (got[:, 3] == 0).all()
    check(got, kt, vt, q, kn, vn, mask, lens, 0.1)
    # capacity 0: no cache at all
    none = {k: (None if k in ("signs", "sk", "vcodes", "vnorms") else v) for k, v in c.items()}
    got0 = run(none, q, kn, vn, mask, m, 0, None, 0, 4, 0.1)
    assert L.rq_last_launch() == "tree_combine_kernel"
    assert torch.equal(got0, got)
    lens[1] = 1                                                # a single cached token for one group, none for others
    got = run(c, q, kn, vn, mask, m, 64, lens, 0, 4, 0.1)
    check(got, kt, vt, q, kn, vn, mask, lens, 0.1)


def test_zero_scale_zero_query_and_zero_keys():
    B, n, KV, rep, m, T = 1, 3, 1, 2, 128, 200
    q, kn, vn = drafted(B, n, KV, rep, 41)
    q[:, 1] = 0
    k = torch.randn(T, D, device=DEV).bfloat16()
    k[::2] = 0
    c = compress(1, T, D, m, 2, 4, 42, True, k=k.reshape(-1))
    kt, vt = vectors(c, 1, T, m, 2, 4)
    for scale in (0.0, 0.1):
        got = run(c, q, kn, vn, None, m, T, None, 2, 4, scale)
        check(got, kt, vt, q, kn, vn, None, None, scale)


def test_a_nan_query_spoils_its_row_only():
    B, n, KV, rep, m, T = 1, 4, 1, 4, 128, 700
    q, kn, vn = drafted(B, n, KV, rep, 43)
    c = compress(1, T, D, m, 0, 4, 44, False)
    want = run(c, q, kn, vn, None, m, T, None, 0, 4, 0.1)
    q[0, 2, 1, 5] = math.nan
    got = run(c, q, kn, vn, None, m, T, None, 0, 4, 0.1)
    assert torch.isnan(got[0, 2, 1]).all()
    got[0, 2, 1] = want[0, 2, 1]
    assert torch.equal(got, want)


def test_strided_views_fp16_projection_and_shared_mask():
    """Query, key and value heads as views of one projection output, an fp16 projection matrix, one tree for all."""
    B, n, KV, rep, m, T = 3, 9, 2, 3, 128, 400
    qkv = torch.randn(B, n, KV * rep + 2 * KV, D, device=DEV).bfloat16()
    q, kn, vn = qkv[:, :, :KV * rep], qkv[:, :, KV * rep:KV * (rep + 1)], qkv[:, :, KV * (rep + 1):]
    c = compress(B * KV, T, D, m, 0, 4, 51, False)
    mask = random_tree(1, n, 52)
    big = torch.full((B, KV * rep + 2, n, D), 7.0, dtype=torch.bfloat16, device=DEV)
    out = big[:, 1:-1].transpose(1, 2)
    got = run(c, q, kn, vn, mask, m, T, None, 0, 4, 0.1, out=out)
    kt, vt = vectors(c, B * KV, T, m, 0, 4)
    check(got, kt, vt, q, kn, vn, mask, None, 0.1)
    assert (big[:, 0] == 7).all() and (big[:, -1] == 7).all()
    plain = run(c, q.contiguous(), kn.contiguous(), vn.contiguous(), mask, m, T, None, 0, 4, 0.1)
    assert torch.equal(plain, got)
    # an fp16 projection whose values bf16 does not hold
    c["S"] = (c["S"].float() * (1 + 2.0 ** -10)).half()
    got = run(c, q, kn, vn, mask, m, T, None, 0, 4, 0.1)
    kt, vt = vectors(c, B * KV, T, m, 0, 4)
    check(got, kt, vt, q, kn, vn, mask, None, 0.1)


def test_far_offsets():
    """A cache whose records lie past 2^32 bytes."""
    T, m, n = 68_000_000, 64, 4
    ln = 300
    c = compress(1, ln, D, m, 0, 4, 61, False)
    far = dict(c)
    for name, width in (("signs", 8), ("sk", 1), ("vcodes", 64), ("vnorms", 1)):
        big = torch.empty(2 * T, width, dtype=c[name].dtype, device=DEV)
        big[T:T + ln] = c[name].reshape(ln, width)
        far[name] = big
    q, kn, vn = drafted(2, n, 1, 2, 62)
    lens = torch.tensor([0, ln], dtype=torch.int32, device=DEV)
    got = run(far, q, kn, vn, None, m, T, lens, 0, 4, 0.1)
    want = run(c, q[1:], kn[1:], vn[1:], None, m, ln, None, 0, 4, 0.1)
    # the work is split over another number of CTAs: joins in another order, fp32 roundings before the last one
    assert torch.allclose(got[1:].float(), want.float(), rtol=2.0 ** -7, atol=1e-4)


def test_graph_streams_and_workspaces():
    """A captured call replayed on new queries, beside a call on another stream with its own workspace."""
    B, n, KV, rep, m, T = 2, 8, 2, 4, 256, 3000
    c = compress(B * KV, T, D, m, 0, 4, 71, False)
    q, kn, vn = drafted(B, n, KV, rep, 72)
    lens = torch.tensor([T, 5, 0, T - 1], dtype=torch.int32, device=DEV)
    ws = [torch.empty(L.qjl_tree_attention_workspace_bytes(B, KV, rep, n, D, m, T), dtype=torch.uint8, device=DEV) for _ in range(2)]
    out = [torch.zeros_like(q) for _ in range(2)]
    run(c, q, kn, vn, None, m, T, lens, 0, 4, 0.1, out=out[0], ws=ws[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c, q, kn, vn, None, m, T, lens, 0, 4, 0.1, out=out[0], ws=ws[0])
    q.copy_(torch.randn_like(q.float()))
    lens.copy_(torch.tensor([7, T, T, 0], device=DEV))
    out[0].zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph.replay()
    run(c, q, kn, vn, None, m, T, lens, 0, 4, 0.1, out=out[1], ws=ws[1], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1])
    kt, vt = vectors(c, B * KV, T, m, 0, 4)
    check(out[0], kt, vt, q, kn, vn, None, lens, 0.1)


def test_workspace_content_does_not_matter():
    B, n, KV, rep, m, T = 1, 20, 2, 4, 256, 900
    c = compress(B * KV, T, D, m, 0, 4, 81, False)
    q, kn, vn = drafted(B, n, KV, rep, 82)
    size = L.qjl_tree_attention_workspace_bytes(B, KV, rep, n, D, m, T)
    a = run(c, q, kn, vn, None, m, T, None, 0, 4, 0.1, ws=torch.full((size,), 255, dtype=torch.uint8, device=DEV))
    b = run(c, q, kn, vn, None, m, T, None, 0, 4, 0.1, ws=torch.zeros(size, dtype=torch.uint8, device=DEV))
    assert torch.equal(a, b)


@pytest.mark.parametrize("n,rep,T", [(1024, 1, 200), (300, 2, 0), (65, 16, 50)])
def test_wide_trees(n, rep, T):
    """Trees of many nodes (several mask words, shared memory beyond the default)."""
    m = 128
    c = compress(1, max(T, 1), D, m, 0, 4, 91, False)
    q, kn, vn = drafted(1, n, 1, rep, 92)
    mask = random_tree(1, n, 93, empty_row=n // 2)
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    got = run(c, q, kn, vn, mask, m, max(T, 1), lens, 0, 4, 0.09)
    kt, vt = vectors(c, 1, max(T, 1), m, 0, 4)
    check(got, kt, vt, q, kn, vn, mask, lens, 0.09)


@pytest.mark.parametrize("n", [4, 40, 80])
def test_hard_maximum(n):
    """Queries equal to cached keys and a scale so large that one key carries all the weight: its value (the weights are
    exact, so 2^-9 of the largest value and the output's rounding remain); later tiles move every reference far."""
    T, m = 900, 256
    k = torch.randn(1, T, D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(95)).bfloat16()
    picks = torch.linspace(0, T - 1, n, device=DEV).long()
    c = compress(1, T, D, m, 0, 4, 95, False, k=k.reshape(-1))
    q = k[0, picks].reshape(1, n, 1, D).contiguous()
    kn = torch.zeros(1, n, 1, D, device=DEV, dtype=torch.bfloat16)
    kt, vt = vectors(c, 1, T, m, 0, 4)
    logits = q[0, :, 0].double() @ kt[0].T
    top = logits.topk(2, -1)
    sure = (top.values[:, 0] - top.values[:, 1]) > 0.05 * top.values[:, 0]
    assert torch.equal(top.indices[sure, 0], picks[sure]) and int(sure.sum()) > n // 2
    gap = float((top.values[sure, 0] - top.values[sure, 1]).min())
    scale = 300.0 / gap                                        # 2^-400 on every other key; logits in the thousands
    got = run(c, q, kn, kn, torch.zeros(1, n, (n + 63) // 64, dtype=torch.int64, device=DEV), m, T, None, 0, 4, scale)
    want = vt[0, picks]
    tol = 2.0 ** -9 * vt.norm(dim=-1).amax() + 2.0 ** -8 * want.abs()
    assert torch.isfinite(got).all()
    assert ((got[0, :, 0].double() - want).abs() <= tol)[sure].all()


@pytest.mark.parametrize("factor", [1e-20, 1e4, 1e12, 1e20])
@pytest.mark.parametrize("n,rep,m,kbits", [(4, 4, 256, 0), (20, 2, 128, 2), (40, 2, 256, 0), (40, 2, 128, 3)])
def test_rows_of_very_different_norms(n, rep, m, kbits, factor):
    """One query row that is far longer (a drafted place that holds rubbish), or far shorter, than its neighbours: their
    outputs stay within the bar, and the long row finds its key."""
    T, at, key = 900, (0, 2, 1), 77
    k = torch.randn(1, T, D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(97)).bfloat16()
    c = compress(1, T, D, m, kbits, 4, 97, kbits > 0, k=k.reshape(-1))
    q, kn, vn = drafted(1, n, 1, rep, 98)
    q[at] = k[0, key]
    kn[:], mask = 0, torch.zeros(1, n, (n + 63) // 64, dtype=torch.int64, device=DEV)
    kt, vt = vectors(c, 1, T, m, kbits, 4)
    scale = 1 / math.sqrt(D)
    odd = q.clone()
    odd[at] = (q[at].float() * factor).bfloat16()
    got = run(c, odd, kn, vn, mask, m, T, None, kbits, 4, scale)
    torch.cuda.synchronize()
    assert L.rq_device_error(True) == 0
    assert torch.isfinite(got).all()
    if factor < 1:
        check(got, kt, vt, odd, kn, vn, mask, None, scale)
        return
    # the next key is 5 % behind at least: with the logits this large all weight is on `key`, exactly
    logits = (odd[at].double() @ kt[0].T) * scale
    top = logits.topk(2)
    assert int(top.indices[0]) == key and float(top.values[0] - top.values[1]) > max(0.05 * float(top.values[0]), 200.0)
    tol = 2.0 ** -9 * vt.norm(dim=-1).amax() + 2.0 ** -8 * vt[0, key].abs()
    assert ((got[at].double() - vt[0, key]).abs() <= tol).all()
    plain = run(c, q, kn, vn, mask, m, T, None, kbits, 4, scale)
    got[at] = plain[at]
    check(got, kt, vt, q, kn, vn, mask, None, scale)


def test_long_zero_and_nan_rows_side_by_side():
    """One chunk of rows that holds a row of 1e20, a zero one, a NaN one and one of 1e-30 times the others."""
    T, m, n, rep = 700, 256, 6, 4
    c = compress(1, T, D, m, 0, 4, 99, False)
    q, kn, vn = drafted(1, n, 1, rep, 99)
    plain = run(c, q, kn, vn, None, m, T, None, 0, 4, 0.1)
    odd = q.clone()
    odd[0, 1, 2] = 0.0
    odd[0, 4, 0] = (q[0, 4, 0].float() * 1e-30).bfloat16()
    quiet = odd.clone()
    odd[0, 2, 1] = (q[0, 2, 1].float() * 1e20).bfloat16()
    odd[0, 3, 3, 7] = math.nan
    got = run(c, odd, kn, vn, None, m, T, None, 0, 4, 0.1)
    assert torch.isfinite(got[0, 2, 1]).all() and torch.isnan(got[0, 3, 3]).all()
    got[0, 2, 1], got[0, 3, 3] = plain[0, 2, 1], plain[0, 3, 3]
    kt, vt = vectors(c, 1, T, m, 0, 4)
    check(got, kt, vt, quiet, kn, vn, None, None, 0.1)


@pytest.mark.parametrize("size,table", [(1e-4, 1.0), (1e-5, 1.0), (200.0, 2000.0), (1.0, 1e-6), (1.0, 1e3)])
@pytest.mark.parametrize("n,rep,vbits", [(4, 4, 4), (40, 2, 4), (13, 3, 3), (13, 3, 8)])
def test_values_of_every_size(n, rep, vbits, size, table):
    """Value norms (11 size) from 1e-4 to thousands, and tables of any scale.  A cached value's coordinate c 2^-e n, with
    2^e just above the largest centroid, is rounded to fp16: half a step is 2^-11 of it, or 2^-25 below 2^-14.  The
    centroids' mean square is 1 and 2^e at most 8, so at n = 1.1e-4 the latter is 2^-25 8 / 1.1e-4 / sqrt(3) = 1.3e-3 of
    the row, uncorrelated: within the 2e-3."""
    T, m = 800, 128
    v = (torch.randn(T, D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(101)) * size).bfloat16()
    c = compress(1, T, D, m, 0, vbits, 101, False, v=v.reshape(-1),
                 vlayout=L.RQ_CODES_INT8 if vbits == 8 else L.RQ_CODES_PACKED)
    c["vc"] = (c["vc"] * np.float32(table)).astype(np.float32)
    q, kn, vn = drafted(1, n, 1, rep, 102)
    vn = (vn.float() * (size * table)).bfloat16()
    got = run(c, q, kn, vn, None, m, T, None, 0, vbits, 0.3)
    kt, vt = vectors(c, 1, T, m, 0, vbits)
    check(got, kt, vt, q, kn, vn, None, None, 0.3)


@pytest.mark.parametrize("rows,m,kbits,vbits", [(128, 256, 2, 4), (64, 512, 4, 4), (32, 256, 2, 4), (16, 512, 0, 4), (48, 512, 4, 3)])
def test_single_buffers_are_used_again(rows, m, kbits, vbits):
    """Shapes whose operand and tables leave room for one weight buffer and one value buffer (or for one CTA an SM), with
    tens of tiles a CTA."""
    B, KV, T = 24, 2, 20011
    c = compress(B * KV, T, D, m, kbits, vbits, 500 + rows, kbits > 0)
    q, kn, vn = drafted(B, rows, KV, 1, 200 + rows)
    lens = torch.tensor([T - 97 * i for i in range(B * KV)], dtype=torch.int32, device=DEV)
    scale = 1 / math.sqrt(D)
    got = run(c, q, kn, vn, None, m, T, lens, kbits, vbits, scale)
    torch.cuda.synchronize()
    assert L.rq_device_error(True) == 0
    for b in (0, 11, B - 1):
        part = {k: (v[b * KV * (v.shape[0] // (B * KV)):(b + 1) * KV * (v.shape[0] // (B * KV))]
                    if isinstance(v, torch.Tensor) and k not in ("k", "v", "S") else v) for k, v in c.items()}
        kt, vt = vectors(part, KV, T, m, kbits, vbits)
        check(got[b:b + 1], kt, vt, q[b:b + 1], kn[b:b + 1], vn[b:b + 1], None, lens[b * KV:(b + 1) * KV], scale)
    assert torch.equal(got, run(c, q, kn, vn, None, m, T, lens, kbits, vbits, scale))


@pytest.mark.parametrize("kbits", [0, 2])
def test_a_row_beyond_the_range_of_logits_spoils_no_other(kbits):
    """A query of the largest finite values: its logits pass the fp32 range, its neighbours are as without it."""
    T, m, n, rep = 500, 128, 5, 4
    c = compress(1, T, D, m, kbits, 4, 111, kbits > 0)
    q, kn, vn = drafted(1, n, 1, rep, 112)
    plain = run(c, q, kn, vn, None, m, T, None, kbits, 4, 0.1)
    odd = q.clone()
    odd[0, 3, 2] = torch.finfo(torch.bfloat16).max * q[0, 3, 2].sign()
    got = run(c, odd, kn, vn, None, m, T, None, kbits, 4, 0.1)
    torch.cuda.synchronize()
    assert L.rq_device_error(True) == 0
    got[0, 3, 2] = plain[0, 3, 2]
    kt, vt = vectors(c, 1, T, m, kbits, 4)
    check(got, kt, vt, q, kn, vn, None, None, 0.1)

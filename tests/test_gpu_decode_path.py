"""The decode-side operators together, as a program runs them: positions on query and key heads, the keys compressed,
drafted tokens over the cache, the queries' weights summed, the cache cut, the next step over what is left."""
import math

import numpy as np
import pytest
import torch

from kv_quantization_b200 import _lib as L
from tests.test_gpu_attention import compress
from tests.test_gpu_tree import check, random_tree, run, vectors

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 128


def rotate(x, pos, freq):
    """Float64 rotation (half pairs), rounded to x's dtype."""
    a = pos.double()[:, :, None, None] * torch.from_numpy(freq).to(DEV)
    u, v = x[..., :D // 2].double(), x[..., D // 2:].double()
    return torch.cat([u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()], -1)


@pytest.mark.parametrize("kbits", [0, 2])
def test_decode_steps_with_eviction(kbits):
    B, KV, rep, T, n, m, keep = 2, 2, 4, 1500, 6, 256, 400
    G, scale = B * KV, 1 / math.sqrt(D)
    g = torch.Generator(device=DEV)
    g.manual_seed(7 + kbits)
    freq, _ = L.rq_rotary_frequencies(D)
    # prompt: keys at their positions, written per head, compressed with the values
    qkv = torch.randn(B, T, KV * (rep + 2), D, generator=g, device=DEV).bfloat16()
    k = qkv[:, :, KV * rep:KV * (rep + 1)]
    pos = torch.arange(T, device=DEV).expand(B, T)
    kr = torch.empty(B, KV, T, D, dtype=torch.bfloat16, device=DEV)
    L.rq_rotary(k, kr.transpose(1, 2), pos, freq, D, L.RQ_ROPE_HALF)
    want = rotate(k, pos, freq).transpose(1, 2)
    assert ((kr.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * k.double().abs().amax()).all()
    v = qkv[:, :, KV * (rep + 1):].transpose(1, 2).contiguous()
    c = compress(G, T, D, m, kbits, 4, 170, kbits > 0, k=kr.reshape(-1), v=v.reshape(-1))
    kt, vt = vectors(c, G, T, m, kbits, 4)

    # a drafted tree over the cache; query and key heads rotated in one launch inside the projection's output
    new = torch.randn(B, n, KV * (rep + 2), D, generator=g, device=DEV).bfloat16()
    depth = torch.randint(0, 4, (B, n), generator=g, device=DEV) + T
    q, kn, vn = new[:, :, :KV * rep], new[:, :, KV * rep:KV * (rep + 1)], new[:, :, KV * (rep + 1):]
    L.rq_rotary(q, q, depth, freq, D, L.RQ_ROPE_HALF, x2=kn, out2=kn)
    mask = random_tree(B, n, 8)
    lens = torch.full((G,), T, dtype=torch.int32, device=DEV)
    got = run(c, q, kn, vn, mask, m, T, lens, kbits, 4, scale)
    check(got, kt, vt, q, kn, vn, mask, lens, scale)

    # weights of the same queries from the library's scores, summed twice with decay
    nq = n * rep
    qs = q.reshape(B, n, KV, rep, D).transpose(1, 2).reshape(G, nq, D).contiguous()
    scores = torch.empty(G, nq, T, device=DEV)
    ws = torch.empty(L.qjl_score_workspace_bytes(G, nq, D, m) // 4 + 4, device=DEV)
    kw = {} if not kbits else dict(codes=c["codes"], norms=c["norms"], bits=kbits, use_signs=1, sign_seed=c["kseed"],
                                   centroids=c["kc"])
    L.qjl_score(qs, G, nq, D, m, c["S"], c["signs"], c["sk"], T, scores, ws, **kw)
    aws = torch.empty(L.rq_evict_accumulate_workspace_bytes(G, nq, T), dtype=torch.uint8, device=DEV)
    acc = torch.zeros(G, T, device=DEV)
    for _ in range(2):
        L.rq_evict_accumulate(scores, G, nq, T, scale, 0.5, acc, acc, aws)
    p = torch.softmax(torch.einsum("gqd,gtd->gqt", qs.double(), kt) * scale, -1).sum(1) * 1.5
    # the scores' bar is 1e-3 of |q| |k| scale in the exponent: e on a weight and on its sum
    e = 1e-3 * float((qs.double().norm(dim=-1).amax() * kt.norm(dim=-1).amax()) * scale)
    assert ((acc.double() - p).abs() <= (math.exp(2 * e) - 1 + 1e-4) * p + 1e-9).all()

    # keep the heaviest tokens, the first and the last ones; the records of every array move together
    idx = torch.empty(G, keep, dtype=torch.int32, device=DEV)
    count = torch.empty(G, dtype=torch.int32, device=DEV)
    L.rq_evict_select(acc, G, T, keep, idx, count, length=lens, n_sink=4, n_recent=64)
    assert (count == keep).all() and (idx[:, :4] == torch.arange(4, device=DEV)).all()
    assert (idx[:, -64:] == torch.arange(T - 64, T, device=DEV)).all()
    names = ["signs", "sk", "vcodes", "vnorms"] + (["codes", "norms"] if kbits else [])
    cut = dict(c)
    for name in names:
        cut[name] = torch.zeros(c[name].numel() // T * keep, dtype=c[name].dtype, device=DEV)
    L.rq_evict_gather(idx, count, G, keep, T, [(c[x], cut[x]) for x in names])
    rows = idx.long()[..., None].expand(-1, -1, D)
    ktc, vtc = vectors(cut, G, keep, m, kbits, 4)
    assert torch.equal(ktc, torch.gather(kt, 1, rows)) and torch.equal(vtc, torch.gather(vt, 1, rows))

    # the next step, one token, over the cache that is left
    one = [x[:, :1].contiguous() for x in (q, kn, vn)]
    got = run(cut, *one, None, m, keep, count, kbits, 4, scale)
    check(got, ktc, vtc, *one, None, count, scale)
    # and a step in which a sequence has nothing left
    count[0] = 0
    got = run(cut, *one, None, m, keep, count, kbits, 4, scale)
    check(got, ktc, vtc, *one, None, count, scale)
    assert np.isfinite(got.float().cpu().numpy()).all()

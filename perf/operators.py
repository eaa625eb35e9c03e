"""Measured cases of the decode-side cache operators, with their plain forms.

Four operators that a decoder runs beside the compressed cache:

  rotary      rotary positions of query and key heads (and the gradient, which
              is the inverse rotation), `rq_rotary`;
  tree        attention of a tree of drafted tokens (one token is the ordinary
              decode step) over a compressed cache and over the drafted tokens'
              own keys and values, `qjl_tree_attention`;
  accumulate  attention weights of a block of queries summed onto each cached
              token, `rq_evict_accumulate`;
  evict       the tokens to keep by that sum, and the cache's records moved
              together, `rq_evict_select` and `rq_evict_gather`.

`run` computes the plain form in elementary torch operations, or makes the
library's calls when `own` is true.
"""
import functools
import math

import numpy as np
import torch

own = False

DEV = "cuda"
D = 128                       # head dimension of the compressed cache
KQ = math.sqrt(math.pi / 2)   # the sketch estimator's factor


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 sequences: 32 query and 8 key heads, positions far into a long context
        dict(name="rotary_decode", op="rotary", batch=64, tokens=1, heads=32, kv_heads=8, d=128, rot=128,
             style="half", dtype="bf16", scaling="banded", start=100000, inverse=False),
        # gradient of a partly rotated, interleaved head of odd batch and length (extended context)
        dict(name="rotary_gradient", op="rotary", batch=3, tokens=4099, heads=16, kv_heads=2, d=96, rot=32,
             style="interleaved", dtype="f16", scaling="yarn", start=0, inverse=True),
        # a 32768-token prefill before its keys are compressed
        dict(name="rotary_prefill", op="rotary", batch=1, tokens=32768, heads=32, kv_heads=8, d=128, rot=128,
             style="half", dtype="bf16", scaling="plain", start=0, inverse=False),
        # the ordinary decode step of four short sequences, where latency counts
        dict(name="tree_one_token", op="tree", batch=4, kv_heads=8, rep=4, nodes=1, tokens=1000, m=256, k_bits=0,
             v_bits=4, ragged=False),
        # a small drafted tree over the long cache of the benchmark's KV line
        dict(name="tree_8_nodes", op="tree", batch=4, kv_heads=8, rep=4, nodes=8, tokens=32768, m=256, k_bits=0,
             v_bits=4, ragged=False),
        # two-stage keys, sequences of very different lengths (one of them empty), odd sizes
        dict(name="tree_two_stage_ragged", op="tree", batch=5, kv_heads=4, rep=3, nodes=13, tokens=20011, m=128,
             k_bits=2, v_bits=3, ragged=True),
        # a wide tree: 256 query rows to each key head over the long cache
        dict(name="tree_64_nodes", op="tree", batch=4, kv_heads=8, rep=4, nodes=64, tokens=32768, m=256, k_bits=0,
             v_bits=4, ragged=False),
        # weights of one decode step's queries
        dict(name="accumulate_decode", op="accumulate", groups=32, queries=4, tokens=4001, causal=False, decay=0.95),
        # weights of the last 32 queries of a long prompt, each seeing one token more than the one before
        dict(name="accumulate_window", op="accumulate", groups=32, queries=32, tokens=32768, causal=True, decay=1.0),
        # a short cache halved
        dict(name="evict_short", op="evict", groups=8, tokens=1000, keep=500, sink=4, recent=32, ragged=True),
        # the long cache cut to a quarter
        dict(name="evict_quarter", op="evict", groups=32, tokens=32768, keep=8192, sink=4, recent=64, ragged=False),
        # few, very long sequences
        dict(name="evict_long", op="evict", groups=4, tokens=131072, keep=20001, sink=16, recent=1000, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "tree", "accumulate", "evict"])
    if op == "rotary":
        d = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([d, d, d // 2, 32])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4])
        batch = _log(rng, 1, 64)
        tokens = _log(rng, 1, max(1, int(1.0e8 / (batch * (heads + kv) * d))))
        return dict(op=op, batch=batch, tokens=min(tokens, 40000), heads=heads, kv_heads=kv, d=d, rot=rot,
                    style=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bf16", "f16"]),
                    scaling=rng.choice(["plain", "linear", "ntk", "yarn", "banded"]),
                    start=rng.choice([0, _log(rng, 1, 1000000)]), inverse=rng.random() < 0.5)
    if op == "tree":
        batch, kv, rep = rng.randint(1, 6), rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
        nodes = _log(rng, 1, 70)
        most = int(2.5e8 / (batch * kv * rep * nodes))           # rows x tokens of the largest listed case
        most = min(most, 32768, int(1.0e6 / (batch * kv)))
        return dict(op=op, batch=batch, kv_heads=kv, rep=rep, nodes=nodes, tokens=_log(rng, 1, max(2, most)),
                    m=rng.choice([128, 256, 512]), k_bits=rng.choice([0, 0, 1, 2, 3, 4]),
                    v_bits=rng.choice([2, 3, 4]), ragged=rng.random() < 0.5)
    if op == "accumulate":
        groups, queries = _log(rng, 1, 64), _log(rng, 1, 70)
        return dict(op=op, groups=groups, queries=queries,
                    tokens=_log(rng, 1, max(2, min(100000, int(3.0e7 / (groups * queries))))),
                    causal=rng.random() < 0.5, decay=rng.choice([1.0, 0.9, 0.0]))
    groups = _log(rng, 1, 64)
    tokens = _log(rng, 8, min(131072, int(1.0e6 / groups)))
    keep = rng.randint(max(1, tokens // 8), tokens)
    sink = rng.randint(0, min(16, keep // 2))
    return dict(op=op, groups=groups, tokens=tokens, keep=keep, sink=sink,
                recent=rng.randint(0, min(1000, keep - sink)), ragged=rng.random() < 0.5)


def _lengths(case, n):
    """Cached tokens of each of n sequences: all of them, or spread, with an empty one."""
    T = case["tokens"]
    if not case["ragged"]:
        return [T] * n
    return [T if i == 0 else 0 if i == 2 else 1 + (T - 1) * (i * 37 % 101) // 101 for i in range(n)]


# ------------------------------------------------------------------ rotary positions

THETA = 10000.0
#: scaling -> (factor, original length, two more parameters)
SCALING = {"plain": (1.0, 1.0, 0.0, 0.0), "linear": (4.0, 1.0, 0.0, 0.0), "ntk": (4.0, 1.0, 0.0, 0.0),
           "yarn": (8.0, 4096.0, 32.0, 1.0), "banded": (8.0, 8192.0, 1.0, 4.0)}


def _frequencies(rot, scaling):
    """Angle of one position step for each pair (float64), and the factor on cosine and sine."""
    factor, length, a, b = SCALING[scaling]
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        return (THETA * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot), 1.0
    f = THETA ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        def at(turns):
            return rot * math.log(length / (turns * 2.0 * math.pi)) / (2.0 * math.log(THETA))
        low, high = max(math.floor(at(a)), 0), min(math.ceil(at(b)), rot - 1)
        ramp = np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
        return f / factor * ramp + f * (1.0 - ramp), 0.1 * math.log(factor) + 1.0
    if scaling == "banded":
        wave = 2.0 * math.pi / f
        smooth = np.clip((length / wave - a) / (b - a), 0.0, 1.0)
        return (1.0 - smooth) * f / factor + smooth * f, 1.0
    return f, 1.0


def _prepare_rotary(case, g):
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float16
    B, n, H, KV, d = (case[k] for k in ("batch", "tokens", "heads", "kv_heads", "d"))
    # query and key heads lie side by side in the projection's output, as they do in a program
    qk = torch.randn(B, n, H + KV, d, generator=g, device=DEV).to(dt)
    first = torch.randint(0, 1000, (B, 1), generator=g, device=DEV) + case["start"]
    freq, scale = _frequencies(case["rot"], case["scaling"])
    return dict(op="rotary", q=qk[:, :, :H], k=qk[:, :, H:], pos=first + torch.arange(n, device=DEV), freq=freq,
                freq_dev=torch.from_numpy(freq).to(DEV), scale=scale, rot=case["rot"], style=case["style"],
                inverse=case["inverse"])


def _rotate_plain(x, c, s, rot, style):
    r = x[..., :rot].float()
    if style == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
    else:
        a, b = r[..., 0::2], r[..., 1::2]
    u, v = a * c - b * s, b * c + a * s
    r = torch.cat([u, v], -1) if style == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([r.to(x.dtype), x[..., rot:]], -1)


def _run_rotary(st):
    if own:
        import kv_quantization_b200 as rq
        q, k = st["q"], st["k"]
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        rq.rq_rotary(q, q_out, st["pos"], st["freq"], st["rot"],
                     rq.RQ_ROPE_HALF if st["style"] == "half" else rq.RQ_ROPE_INTERLEAVED, scale=st["scale"],
                     inverse=st["inverse"], x2=k, out2=k_out)
        return q_out, k_out
    angle = st["pos"].double()[:, :, None, None] * st["freq_dev"]
    c, s = (angle.cos() * st["scale"]).float(), (angle.sin() * st["scale"]).float()
    if st["inverse"]:
        s = -s
    return (_rotate_plain(st["q"], c, s, st["rot"], st["style"]),
            _rotate_plain(st["k"], c, s, st["rot"], st["style"]))


def _exact_rotary(st):
    turn = torch.polar(torch.full_like(st["freq_dev"], st["scale"]).expand(*st["pos"].shape, -1),
                       st["pos"].double().unsqueeze(-1) * st["freq_dev"])[:, :, None]
    if st["inverse"]:
        turn = turn.conj()
    out = []
    for x in (st["q"], st["k"]):
        x, rot = x.double().clone(), st["rot"]
        first = slice(0, rot // 2) if st["style"] == "half" else slice(0, rot, 2)
        second = slice(rot // 2, rot) if st["style"] == "half" else slice(1, rot, 2)
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        out.append(x)
    return tuple(out)


# ------------------------------------------------------------------ the compressed cache

@functools.lru_cache(None)
def _levels(bits):
    """Lloyd-Max levels of N(0, 1)."""
    K = 1 << bits
    c = [4.0 * (2 * i + 1 - K) / K for i in range(K)]
    for _ in range(3000):
        t = [-math.inf] + [0.5 * (a + b) for a, b in zip(c, c[1:])] + [math.inf]
        pdf = [0.0 if math.isinf(x) else math.exp(-0.5 * x * x) / math.sqrt(2 * math.pi) for x in t]
        cdf = [0.5 * math.erfc(-x / math.sqrt(2)) for x in t]
        c = [(pdf[i] - pdf[i + 1]) / (cdf[i + 1] - cdf[i]) for i in range(K)]
    return np.array([0.5 * (c[i] - c[K - 1 - i]) for i in range(K)], dtype=np.float32)


@functools.lru_cache(None)
def _diagonal(seed):
    """The +-1 diagonal: bit j % 64 of output j // 64 of the SplitMix64 stream."""
    mask, out = (1 << 64) - 1, []
    for w in range(D // 64):
        z = (seed + (w + 1) * 0x9E3779B97F4A7C15) & mask
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        z ^= z >> 31
        out += [-1.0 if z >> j & 1 else 1.0 for j in range(64)]
    return torch.tensor(out, device=DEV)


@functools.lru_cache(None)
def _hadamard():
    h = torch.ones(1, 1, device=DEV)
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _pack(codes, bits):
    """Codes [..., n] to bytes, least significant bit first."""
    b = (codes.to(torch.uint8).unsqueeze(-1) >> torch.arange(bits, device=DEV, dtype=torch.uint8)) & 1
    b = b.flatten(-2).unflatten(-1, (-1, 8))
    return (b << torch.arange(8, device=DEV, dtype=torch.uint8)).sum(-1, dtype=torch.uint8)


def _unpack(data, bits, n):
    b = ((data.unsqueeze(-1) >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1).flatten(-2)
    if bits == 1:
        return b
    return (b.unflatten(-1, (n, bits)) << torch.arange(bits, device=DEV, dtype=torch.uint8)).sum(-1, dtype=torch.uint8)


def _quantize(x, bits, seed):
    """Packed codes, fp16 norms and the reconstruction of blocks of D values."""
    lev = torch.from_numpy(_levels(bits)).to(DEV)
    n = x.norm(dim=-1)
    y = (x * _diagonal(seed)) @ _hadamard() / n.clamp_min(1e-30).unsqueeze(-1)
    codes = torch.bucketize(y, 0.5 * (lev[1:] + lev[:-1]))
    n16 = n.half()
    back = (lev[codes] @ _hadamard()) * _diagonal(seed) * (n16.float() / D).unsqueeze(-1)
    return _pack(codes, bits), n16, back


K_SEED, V_SEED = 71, 72


def _prepare_tree(case, g):
    B, KV, rep, n, T, m = (case[k] for k in ("batch", "kv_heads", "rep", "nodes", "tokens", "m"))
    G, kb, vb = B * KV, case["k_bits"], case["v_bits"]
    lens = torch.tensor(_lengths(case, B), dtype=torch.int32, device=DEV)
    S = torch.randn(m, D, generator=g, device=DEV).bfloat16()
    channel = torch.ones(KV, 1, D, device=DEV)
    channel[:, :, torch.randperm(D, generator=g, device=DEV)[:4]] = 4.0        # outlier channels of the keys
    k = (torch.randn(B, KV, T, D, generator=g, device=DEV) * channel).reshape(G, T, D)
    st = dict(op="tree", S=S, T=T, m=m, n=n, KV=KV, rep=rep, k_bits=kb, v_bits=vb, codes=None, norms=None,
              kv_len=lens.repeat_interleave(KV), scale=1.0 / math.sqrt(D))
    # query rows: noise, and for every other row a cached key that it looks for
    q = torch.randn(G, n * rep, D, generator=g, device=DEV)
    at = torch.randint(0, T, (G, n * rep), generator=g, device=DEV)
    q[:, ::2] += 0.4 * torch.gather(k, 1, at.unsqueeze(-1).expand(-1, -1, D))[:, ::2]
    st["q"] = q.reshape(B, KV, n, rep, D).permute(0, 2, 1, 3, 4).reshape(B, n, KV * rep, D).bfloat16()
    if kb:
        st["codes"], st["norms"], back = _quantize(k, kb, K_SEED)
        k = k - back
    st["sk_norms"] = k.norm(dim=-1).half()
    st["signs"] = _pack((k @ S.float().T >= 0), 1)
    del k
    st["v_codes"], st["v_norms"], _ = _quantize(torch.randn(G, T, D, generator=g, device=DEV), vb, V_SEED)
    new = torch.randn(2, B, n, KV, D, generator=g, device=DEV).bfloat16()
    st["k_new"], st["v_new"] = new[0], new[1]
    # a random tree per sequence: each node sees itself and its ancestors
    sees = np.zeros((B, n, -(-n // 64) * 64), dtype=np.uint8)
    parent = np.random.RandomState(int(torch.randint(0, 1 << 30, (1,), generator=g, device=DEV))).rand(B, n)
    for b in range(B):
        for i in range(n):
            p = int(parent[b, i] * i)
            if i:
                sees[b, i] = sees[b, p]
            sees[b, i, i] = 1
    words = np.packbits(sees, axis=-1, bitorder="little").view(np.int64)
    st["tree_mask"] = torch.from_numpy(words.copy()).to(DEV)
    return st


def _tree_visible(st):
    """[B, n, n] truth values of the tree mask."""
    w = st["tree_mask"]
    bits = (w.unsqueeze(-1) >> torch.arange(64, device=DEV)) & 1
    return bits.flatten(-2)[..., :st["n"]].bool()


def _run_tree(st):
    q, T, m, n, KV, rep = st["q"], st["T"], st["m"], st["n"], st["KV"], st["rep"]
    B = q.shape[0]
    if own:
        import kv_quantization_b200 as rq
        if "ws" not in st:
            st["ws"] = torch.empty(rq.qjl_tree_attention_workspace_bytes(B, KV, rep, n, D, m, T), dtype=torch.uint8,
                                   device=DEV)
        out = torch.empty_like(q)
        extra = {}
        if st["k_bits"]:
            extra = dict(codes=st["codes"], norms=st["norms"], bits=st["k_bits"], use_signs=1, sign_seed=K_SEED,
                         centroids=_levels(st["k_bits"]))
        rq.qjl_tree_attention(q, st["k_new"], st["v_new"], st["tree_mask"], m, st["S"], st["signs"], st["sk_norms"],
                              T, st["kv_len"], st["v_codes"], st["v_norms"], st["v_bits"], _levels(st["v_bits"]), out,
                              st["ws"], st["scale"], v_use_signs=1, v_sign_seed=V_SEED, **extra)
        return out
    G, R = B * KV, n * rep
    qr = q.float().reshape(B, n, KV, rep, D).transpose(1, 2).reshape(G, R, D)
    sign = _unpack(st["signs"], 1, m).float().mul_(2).sub_(1)
    s = (qr @ st["S"].float().T) @ sign.transpose(1, 2) * (st["sk_norms"].float() * (KQ / m)).unsqueeze(1)
    del sign
    if st["k_bits"]:
        c = torch.from_numpy(_levels(st["k_bits"])).to(DEV)[_unpack(st["codes"], st["k_bits"], D).int()]
        s += (qr * _diagonal(K_SEED)) @ _hadamard() @ c.transpose(1, 2) * (st["norms"].float() / D).unsqueeze(1)
        del c
    s.masked_fill_(torch.arange(T, device=DEV) >= st["kv_len"][:, None, None], -math.inf)
    k_new, v_new = (st[x].float().transpose(1, 2).reshape(G, n, D) for x in ("k_new", "v_new"))
    hidden = ~_tree_visible(st)[:, None, :, None].expand(B, KV, n, rep, n).reshape(G, R, n)
    s = torch.cat([s, (qr @ k_new.transpose(1, 2)).masked_fill_(hidden, -math.inf)], -1).mul_(st["scale"])
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.from_numpy(_levels(st["v_bits"])).to(DEV)[_unpack(st["v_codes"], st["v_bits"], D).int()]
    v = (v @ _hadamard()).mul_(_diagonal(V_SEED)).mul_((st["v_norms"].float() / D).unsqueeze(-1))
    o = (p[..., :T] @ v + p[..., T:] @ v_new) / torch.where(total == 0, torch.ones_like(total), total)
    return o.reshape(B, KV, n, rep, D).transpose(1, 2).reshape(B, n, KV * rep, D).to(q.dtype)


def _fwht64(x):
    h = 1
    while h < D:
        x = x.unflatten(-1, (-1, 2, h))
        x = torch.stack([x[..., 0, :] + x[..., 1, :], x[..., 0, :] - x[..., 1, :]], -2).flatten(-3)
        h *= 2
    return x


def _exact_tree(st):
    q, T, m, n, KV, rep = st["q"].double(), st["T"], st["m"], st["n"], st["KV"], st["rep"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    sees = _tree_visible(st)
    for g in range(q.shape[0] * KV):                       # keys and values as vectors again, then softmax attention
        b, h = divmod(g, KV)
        length = int(st["kv_len"][g])
        bits = np.unpackbits(st["signs"][g, :length].cpu().numpy(), axis=-1, bitorder="little")
        k = (torch.from_numpy(bits).to(DEV).double() * 2 - 1) @ st["S"].double()
        k *= st["sk_norms"][g, :length].double().unsqueeze(-1) * math.sqrt(math.pi / 2) / m
        back = []
        for data, norm, width, seed in ((st["codes"], st["norms"], st["k_bits"], K_SEED),
                                        (st["v_codes"], st["v_norms"], st["v_bits"], V_SEED)):
            if not width:
                back.append(0.0)
                continue
            bits = np.unpackbits(data[g, :length].cpu().numpy(), axis=-1, bitorder="little")
            code = torch.from_numpy(bits.reshape(length, D, width) @ (1 << np.arange(width))).to(DEV)
            x = _fwht64(torch.from_numpy(_levels(width)).to(DEV).double()[code])
            back.append(x * _diagonal(seed).double() * norm[g, :length].double().unsqueeze(-1) / D)
        keys = torch.cat([k + back[0], st["k_new"][b, :, h].double()])
        vals = torch.cat([back[1], st["v_new"][b, :, h].double()])
        a = torch.einsum("nrd,td->nrt", q[b, :, h * rep:(h + 1) * rep], keys) * st["scale"]
        a[..., length:].masked_fill_(~sees[b][:, None], -math.inf)
        out[b, :, h * rep:(h + 1) * rep] = torch.softmax(a, -1).nan_to_num(0.0) @ vals
    return out


# ------------------------------------------------------------------ eviction

def _prepare_accumulate(case, g):
    G, R, T = case["groups"], case["queries"], case["tokens"]
    # scores of queries and keys of 128 N(0, 1) values, a few keys that every query looks for
    scores = torch.randn(G, R, T, generator=g, device=DEV) * math.sqrt(D)
    heavy = torch.rand(G, 1, T, generator=g, device=DEV) < 0.01
    scores += heavy * (4.0 * math.sqrt(D))
    row_len = None
    if case["causal"]:
        row_len = (T - R + 1 + torch.arange(R, device=DEV)).clamp_min(0).to(torch.int32).expand(G, R).contiguous()
    return dict(op="accumulate", scores=scores, row_len=row_len, scale=1.0 / math.sqrt(D), decay=case["decay"],
                acc=torch.rand(G, T, generator=g, device=DEV))


def _run_accumulate(st):
    scores = st["scores"]
    G, R, T = scores.shape
    if own:
        import kv_quantization_b200 as rq
        if "ws" not in st:
            st["ws"] = torch.empty(rq.rq_evict_accumulate_workspace_bytes(G, R, T), dtype=torch.uint8, device=DEV)
        out = torch.empty_like(st["acc"])
        rq.rq_evict_accumulate(scores, G, R, T, st["scale"], st["decay"], st["acc"], out, st["ws"],
                               row_len=st["row_len"])
        return out
    s = scores * st["scale"]
    if st["row_len"] is not None:
        s = s.masked_fill_(torch.arange(T, device=DEV) >= st["row_len"].unsqueeze(-1), -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total == 0, torch.ones_like(total), total)
    return st["acc"] * st["decay"] + p.sum(1)


def _exact_accumulate(st):
    G, R, T = st["scores"].shape
    out = st["acc"].double() * st["decay"]
    for g in range(G):
        a = st["scores"][g].double() * st["scale"]
        if st["row_len"] is not None:
            a = torch.where(torch.arange(T, device=DEV) < st["row_len"][g][:, None], a, -math.inf)
        out[g] += torch.softmax(a, -1).nan_to_num(0.0).sum(0)
    return out


#: bytes a token keeps in the evicted cache: sign bits (m = 256), fp16 norm, 4-bit value codes, fp16 norm, weight sum
RECORDS = (("signs", 32, torch.uint8), ("sk_norms", 1, torch.float16), ("v_codes", 64, torch.uint8),
           ("v_norms", 1, torch.float16), ("acc", 1, torch.float32))


def _prepare_evict(case, g):
    G, T = case["groups"], case["tokens"]
    st = dict(op="evict", T=T, keep=case["keep"], sink=case["sink"], recent=case["recent"],
              len=torch.tensor(_lengths(case, G), dtype=torch.int32, device=DEV))
    for name, width, dt in RECORDS:
        if dt == torch.uint8:
            x = torch.randint(0, 256, (G, T, width), generator=g, device=DEV, dtype=torch.uint8)
        else:
            x = torch.rand(G, T, width, generator=g, device=DEV)
            x = x.exp().to(dt)
        st[name] = x
    # sums of attention weights: most tokens next to nothing, few a lot, many equal after some steps without weight
    w = torch.rand(G, T, generator=g, device=DEV).pow(8)
    st["acc"] = torch.where(w < 1e-4, torch.full_like(w, 2.0 ** -20), w).unsqueeze(-1)
    st["kept"] = {name: torch.zeros(G, case["keep"], width, dtype=dt, device=DEV) for name, width, dt in RECORDS}
    return st


def _run_evict(st):
    acc, T, keep, length = st["acc"], st["T"], st["keep"], st["len"]
    G = acc.shape[0]
    kept = st["kept"]
    if own:
        import kv_quantization_b200 as rq
        idx = torch.empty(G, keep, dtype=torch.int32, device=DEV)
        count = torch.empty(G, dtype=torch.int32, device=DEV)
        rq.rq_evict_select(acc, G, T, keep, idx, count, length=length, n_sink=st["sink"], n_recent=st["recent"])
        rq.rq_evict_gather(idx, count, G, keep, T, [(st[name], kept[name]) for name, _, _ in RECORDS])
        return idx, count, kept
    t = torch.arange(T, device=DEV)
    n = length.unsqueeze(-1)
    a = acc.squeeze(-1)
    a = torch.where((t < st["sink"]) | (t >= n - st["recent"]), math.inf, a)
    a = torch.where(t < n, a, -math.inf)
    order = torch.sort(a, dim=-1, descending=True, stable=True).indices[:, :keep]
    order = torch.where(order < n, order, T).sort(-1).values                # tokens behind the last one go last
    count = length.clamp_max(keep)
    live = torch.arange(keep, device=DEV) < count.unsqueeze(-1)
    idx = torch.where(live, order, -1)
    row = idx.clamp_min(0)
    got = {name: torch.where(live.unsqueeze(-1),
                             torch.gather(st[name], 1, row.unsqueeze(-1).expand(-1, -1, width)), kept[name])
           for name, width, _ in RECORDS}
    return idx.int(), count, got


# ------------------------------------------------------------------ interface

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * int(seed) + 17)
    return {"rotary": _prepare_rotary, "tree": _prepare_tree, "accumulate": _prepare_accumulate,
            "evict": _prepare_evict}[case["op"]](case, g)


def run(state):
    return {"rotary": _run_rotary, "tree": _run_tree, "accumulate": _run_accumulate,
            "evict": _run_evict}[state["op"]](state)


def exact(case, seed):
    if case["op"] == "evict":
        return None                                            # whole numbers and copies: nothing is computed
    st = prepare(case, seed)
    return {"rotary": _exact_rotary, "tree": _exact_tree, "accumulate": _exact_accumulate}[case["op"]](st)


def work(case):
    if case["op"] == "rotary":
        pairs = case["batch"] * case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 4 * pairs * case["d"] + 8 * case["batch"] * case["tokens"], "flops": 3 * pairs * case["rot"]}
    if case["op"] == "tree":
        B, KV, rep, n, m, kb, vb = (case[k] for k in ("batch", "kv_heads", "rep", "nodes", "m", "k_bits", "v_bits"))
        cached = sum(_lengths(case, B)) * KV
        record = m // 8 + 2 + (kb * D // 8 + 2 if kb else 0) + vb * D // 8 + 2
        rows = B * KV * n * rep
        pairs = cached * n * rep
        return {"bytes": cached * record + 2 * m * D + 4 * rows * D + 4 * B * KV * n * D,
                "flops": 2 * pairs * (m + (D if kb else 0) + D) + 2 * rows * m * D + 4 * rows * n * D}
    if case["op"] == "accumulate":
        G, R, T = case["groups"], case["queries"], case["tokens"]
        return {"bytes": 4 * G * R * T + 8 * G * T, "flops": 5 * G * R * T}
    cached = sum(_lengths(case, case["groups"]))
    kept = sum(min(case["keep"], x) for x in _lengths(case, case["groups"]))
    return {"bytes": 4 * cached + 4 * case["groups"] * case["keep"] + 2 * kept * (32 + 2 + 64 + 2 + 4), "flops": 0}

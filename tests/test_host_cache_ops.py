"""Host side of the decode-side cache operators: refusals before anything is enqueued, and the rotary frequencies
against their formulas (no GPU)."""
import ctypes as C
import math
import os
import re

import numpy as np
import pytest
import torch

from kv_quantization_b200 import _lib as L

EINVAL, EALIGN, ESIZE, EUNSUPPORTED = -1, -2, -3, -4
ST = L.Strides(0, 0, 0)
A = 0x100000                                                   # a device address that is never dereferenced


def rotary_status(**kw):
    a = dict(x=A, xs=ST, out=A, os=ST, heads=2, x2=None, x2s=None, out2=None, o2s=None, heads2=0, dtype=L.RQ_BF16, B=1,
             n=1, d=128, rot=128, style=L.RQ_ROPE_HALF, pos=A, ps=0, freq=np.ones(256), scale=1.0, inverse=0)
    a.update(kw)
    ref = lambda s: None if s is None else C.addressof(s)  # noqa: E731
    return L.lib().rq_rotary(a["x"], ref(a["xs"]), a["out"], ref(a["os"]), a["heads"], a["x2"], ref(a["x2s"]),
                             a["out2"], ref(a["o2s"]), a["heads2"], a["dtype"], a["B"], a["n"], a["d"], a["rot"],
                             a["style"], a["pos"], a["ps"],
                             None if a["freq"] is None else a["freq"].ctypes.data, a["scale"], a["inverse"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(dtype=2), EINVAL), (dict(style=2), EINVAL), (dict(B=-1), EINVAL), (dict(n=-1), EINVAL),
    (dict(heads=0), EINVAL), (dict(heads2=-1), EINVAL), (dict(d=127), EINVAL), (dict(d=514, rot=2), EINVAL),
    (dict(rot=3), EINVAL), (dict(rot=0), EINVAL), (dict(d=64, rot=66), EINVAL), (dict(freq=None), EINVAL),
    (dict(freq=np.full(256, np.nan)), EINVAL), (dict(freq=np.full(256, 2.0 ** 20)), EINVAL),
    (dict(scale=math.inf), EINVAL), (dict(x=None), EINVAL), (dict(out=None), EINVAL), (dict(xs=None), EINVAL),
    (dict(pos=None), EINVAL), (dict(heads2=1), EINVAL), (dict(x=A + 1), EALIGN), (dict(pos=A + 4), EALIGN),
    (dict(n=1 << 31), ESIZE), (dict(B=1 << 16, n=1 << 16), ESIZE), (dict(heads=70000), ESIZE),
])
def test_rotary_refuses(kw, status):
    assert rotary_status(**kw) == status
    assert L.rq_last_launch() == ""


def test_rotary_of_no_tokens_is_a_noop():
    assert rotary_status(B=0, x=None, pos=None) == 0
    assert rotary_status(n=0, x=None, pos=None) == 0


def test_rotary_binding_checks_shapes():
    x = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    pos = torch.zeros(2, 3, dtype=torch.int64)
    f = np.ones(32)
    for bad in (lambda: L.rq_rotary(x, x[:, :2], pos, f, 64, 0), lambda: L.rq_rotary(x, x, pos.int(), f, 64, 0),
                lambda: L.rq_rotary(x, x, pos[:, :2], f, 64, 0), lambda: L.rq_rotary(x, x, pos, f[:8], 64, 0),
                lambda: L.rq_rotary(x.transpose(2, 3), x.transpose(2, 3), pos, f, 64, 0),
                lambda: L.rq_rotary(x, x, pos, f, 64, 0, x2=x[:1], out2=x[:1]),
                lambda: L.rq_rotary(x, x, pos, f, 64, 0, x2=x)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        L.rq_rotary(x, x.half(), pos, f, 64, 0)
    with pytest.raises(TypeError):
        L.rq_rotary(x.float(), x.float(), pos, f, 64, 0, stream=0)


def formula(rot, theta, kind, factor, length, p0, p1):
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if kind == L.RQ_ROPE_LINEAR:
        return f / factor
    if kind == L.RQ_ROPE_NTK:
        return np.array([(theta * factor ** (rot / (rot - 2))) ** (-2.0 * i / rot) for i in range(rot // 2)])
    if kind == L.RQ_ROPE_YARN:
        at = lambda turns: rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(at(p0)), 0), min(math.ceil(at(p1)), rot - 1)
        r = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
        return f / factor * r + f * (1 - r)
    if kind == L.RQ_ROPE_BANDED:
        s = np.clip((length / (2 * math.pi / f) - p0) / (p1 - p0), 0, 1)
        return (1 - s) * f / factor + s * f
    return f


@pytest.mark.parametrize("kind, args", [(L.RQ_ROPE_PLAIN, (1.0, 1.0, 0.0, 0.0)), (L.RQ_ROPE_LINEAR, (4.0, 1.0, 0.0, 0.0)),
                                        (L.RQ_ROPE_NTK, (8.0, 1.0, 0.0, 0.0)), (L.RQ_ROPE_YARN, (16.0, 4096.0, 32.0, 1.0)),
                                        (L.RQ_ROPE_BANDED, (8.0, 8192.0, 1.0, 4.0))])
@pytest.mark.parametrize("rot, theta", [(128, 10000.0), (64, 500000.0), (20, 10000.0), (512, 1e6), (4, 100.0)])
def test_frequencies(kind, args, rot, theta):
    f, scale = L.rq_rotary_frequencies(rot, theta, kind, *args)
    assert f.shape == (rot // 2,)
    assert np.allclose(f, formula(rot, theta, kind, *args), rtol=1e-13, atol=0)
    assert scale == pytest.approx(0.1 * math.log(args[0]) + 1.0 if kind == L.RQ_ROPE_YARN else 1.0, rel=1e-15)


def test_frequency_scaling_does_what_it_is_for():
    plain, _ = L.rq_rotary_frequencies(128)
    yarn, _ = L.rq_rotary_frequencies(128, 10000.0, L.RQ_ROPE_YARN, 8.0, 4096.0, 32.0, 1.0)
    band, _ = L.rq_rotary_frequencies(128, 10000.0, L.RQ_ROPE_BANDED, 8.0, 8192.0, 1.0, 4.0)
    ntk, _ = L.rq_rotary_frequencies(128, 10000.0, L.RQ_ROPE_NTK, 8.0)
    for f in (yarn, band):                                     # fast pairs as they were, slow ones interpolated
        assert f[0] == plain[0] and f[-1] == pytest.approx(plain[-1] / 8.0, rel=1e-12)
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(plain[-1] / 8.0, rel=1e-12)


@pytest.mark.parametrize("args", [
    (0,), (3,), (514,), (64, 1.0), (64, math.inf), (64, 1e4, 5), (64, 1e4, L.RQ_ROPE_LINEAR, 0.5),
    (64, 1e4, L.RQ_ROPE_YARN, 2.0, 0.0, 32.0, 1.0), (64, 1e4, L.RQ_ROPE_YARN, 2.0, 4096.0, 1.0, 32.0),
    (64, 1e4, L.RQ_ROPE_BANDED, 2.0, 4096.0, 4.0, 1.0), (64, 1e4, L.RQ_ROPE_BANDED, 2.0, math.nan, 1.0, 4.0),
    (2, 1e4, L.RQ_ROPE_NTK, 2.0),
])
def test_frequencies_refuse(args):
    with pytest.raises(L.RQError) as e:
        L.rq_rotary_frequencies(*args)
    assert e.value.status == EINVAL


def accumulate_status(**kw):
    a = dict(scores=A, G=2, nq=3, T=5, row_len=None, scale=1.0, decay=1.0, acc=A, out=A, ws=A, wsb=1 << 20)
    a.update(kw)
    return L.lib().rq_evict_accumulate(a["scores"], a["G"], a["nq"], a["T"], a["row_len"], a["scale"], a["decay"],
                                       a["acc"], a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(G=-1), EINVAL), (dict(nq=-1), EINVAL), (dict(T=-1), EINVAL), (dict(scale=-1.0), EINVAL),
    (dict(scale=math.nan), EINVAL), (dict(decay=math.inf), EINVAL), (dict(scores=None), EINVAL),
    (dict(acc=None), EINVAL), (dict(out=None), EINVAL), (dict(ws=None), EINVAL), (dict(wsb=0), ESIZE),
    (dict(G=65536), ESIZE), (dict(nq=4097), ESIZE), (dict(T=(1 << 31) + 1), ESIZE), (dict(scores=A + 4), EALIGN),
    (dict(row_len=A + 4), EALIGN), (dict(out=A + 8), EALIGN), (dict(ws=A + 8), EALIGN),
])
def test_accumulate_refuses(kw, status):
    assert accumulate_status(**kw) == status


def test_accumulate_of_nothing_is_a_noop():
    assert accumulate_status(G=0, scores=None, acc=None, out=None, ws=None, wsb=0) == 0
    assert accumulate_status(T=0, scores=None, acc=None, out=None, ws=None, wsb=0) == 0
    assert L.rq_evict_accumulate_workspace_bytes(0, 4, 100) == 0
    assert L.rq_evict_accumulate_workspace_bytes(2, 4, 100) > 0


@pytest.mark.parametrize("kw, status", [
    (dict(G=-1), EINVAL), (dict(T=-1), EINVAL), (dict(keep=0), EINVAL), (dict(sink=-1), EINVAL),
    (dict(recent=-1), EINVAL), (dict(sink=3, recent=6), EINVAL), (dict(acc=None), EINVAL), (dict(idx=None), EINVAL),
    (dict(count=None), EINVAL), (dict(idx=A + 4), EALIGN), (dict(acc=A + 4), EALIGN), (dict(G=65536), ESIZE),
    (dict(T=(1 << 28) + 1), ESIZE), (dict(keep=(1 << 28) + 1), ESIZE),
])
def test_select_refuses(kw, status):
    a = dict(acc=A, G=2, T=20, len=None, keep=8, sink=0, recent=0, idx=A, count=A)
    a.update(kw)
    assert L.lib().rq_evict_select(a["acc"], a["G"], a["T"], a["len"], a["keep"], a["sink"], a["recent"], a["idx"],
                                   a["count"], None) == status


@pytest.mark.parametrize("kw, status", [
    (dict(G=-1), EINVAL), (dict(keep=0), EINVAL), (dict(T_dst=7), EINVAL), (dict(n=0), EINVAL), (dict(n=17), EINVAL),
    (dict(row=0), EINVAL), (dict(row=65537), EINVAL), (dict(idx=None), EINVAL), (dict(src=None), EINVAL),
    (dict(dst=None), EINVAL), (dict(src=A + 8), EALIGN), (dict(dst=A + 0x100008), EALIGN), (dict(dst=A), EINVAL),
    (dict(dst=A + 2 * 20 * 16 - 16), EINVAL), (dict(dst=A - 2 * 8 * 16 + 16), EINVAL), (dict(G=65536), ESIZE),
])
def test_gather_refuses(kw, status):
    a = dict(idx=A, count=A, G=2, keep=8, T=20, T_dst=8, src=A, dst=A + 0x100000, row=16, n=1)
    a.update(kw)
    rows = (L.Rows * 17)()
    for r in rows:
        r.src, r.dst, r.row_bytes = a["src"], a["dst"], a["row"]
    assert L.lib().rq_evict_gather(a["idx"], a["count"], a["G"], a["keep"], a["T"], a["T_dst"], C.addressof(rows),
                                   a["n"], None) == status


def test_gather_refuses_arrays_that_share_memory():
    rows = (L.Rows * 2)()
    for r, src, dst in zip(rows, (A, A + 0x10000), (A + 0x20000, A + 0x20080)):
        r.src, r.dst, r.row_bytes = src, dst, 16
    call = lambda: L.lib().rq_evict_gather(A, A, 2, 8, 20, 8, C.addressof(rows), 2, None)  # noqa: E731
    assert call() == EINVAL                                    # two destinations
    rows[1].dst = A
    assert call() == EINVAL                                    # a destination and another array's source


def test_gather_binding_checks_sizes():
    src, dst = torch.zeros(2, 20, 3), torch.zeros(2, 7, 3)
    with pytest.raises(ValueError):
        L.rq_evict_gather(torch.zeros(2, 8, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 2, 8, 20,
                          [(src, dst)], stream=0)


def tree_status(**kw):
    a = dict(q=A, k=A, v=A, B=1, kv=1, rep=2, n=3, d=128, mask=None, mb=0, m=128, proj=A, pd=L.RQ_BF16, signs=A, sk=A,
             T=10, lens=None, codes=None, norms=None, bits=0, layout=0, cent=None, vc=A, vn=A, vb=4, vl=0,
             vcent=L.rq_lloyd_max(4), scale=1.0, out=A, ws=A, wsb=1 << 40, s=ST, os=ST)
    a.update(kw)
    ref = lambda x: None if x is None else C.addressof(x)  # noqa: E731
    tab = lambda x: None if x is None else x.ctypes.data  # noqa: E731
    return L.lib().qjl_tree_attention(
        a["q"], ref(a["s"]), a["k"], C.addressof(ST), a["v"], C.addressof(ST), a["B"], a["kv"], a["rep"], a["n"], a["d"],
        a["mask"], a["mb"], a["m"], a["proj"], a["pd"], a["signs"], a["sk"], a["T"], a["lens"], a["codes"], a["norms"],
        a["bits"], a["layout"], 0, 0, tab(a["cent"]), a["vc"], a["vn"], a["vb"], a["vl"], 0, 0, tab(a["vcent"]),
        a["scale"], a["out"], ref(a["os"]), a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(d=96), EINVAL), (dict(d=64), EUNSUPPORTED), (dict(m=12), EINVAL), (dict(m=96), EUNSUPPORTED),
    (dict(m=520), EINVAL), (dict(pd=3), EINVAL), (dict(B=-1), EINVAL), (dict(kv=0), EINVAL), (dict(rep=0), EINVAL),
    (dict(n=0), EINVAL), (dict(T=-1), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=math.nan), EINVAL),
    (dict(n=1025), ESIZE), (dict(n=1000, rep=100), ESIZE), (dict(B=70000), ESIZE), (dict(B=300, kv=300), ESIZE),
    (dict(vb=0), EINVAL), (dict(vb=9), EINVAL), (dict(vb=5), EUNSUPPORTED), (dict(vl=7), EINVAL),
    (dict(codes=A, norms=A, bits=5, cent=L.rq_lloyd_max(5)), EUNSUPPORTED), (dict(codes=A, bits=2), EINVAL),
    (dict(codes=A, norms=A, bits=2), EINVAL), (dict(proj=None), EINVAL), (dict(ws=None), EINVAL),
    (dict(signs=None), EINVAL), (dict(vn=None), EINVAL), (dict(q=None), EINVAL), (dict(out=None), EINVAL),
    (dict(s=None), EINVAL), (dict(os=None), EINVAL), (dict(q=A + 8), EALIGN), (dict(out=A + 2), EALIGN),
    (dict(signs=A + 8), EALIGN), (dict(lens=A + 4), EALIGN), (dict(mask=A + 8), EALIGN), (dict(ws=A + 8), EALIGN),
    (dict(s=L.Strides(0, 4, 0)), EALIGN), (dict(os=L.Strides(0, 0, 130)), EALIGN), (dict(vcent=None), EINVAL),
    (dict(vcent=L.rq_lloyd_max(4)[::-1].copy()), EINVAL),
])
def test_tree_refuses(kw, status):
    assert tree_status(**kw) == status
    assert L.rq_last_launch() == ""


def test_tree_of_no_sequences_is_a_noop():
    assert tree_status(B=0, q=None, ws=None) == 0


def test_tree_workspace_covers_both_kinds_of_keys():
    size = L.qjl_tree_attention_workspace_bytes
    assert size(0, 1, 1, 1, 128, 128, 10) == 0 and size(1, 1, 1, 2000, 128, 128, 10) == 0
    assert 0 < size(1, 1, 1, 1, 128, 128, 0) < size(1, 1, 1, 1, 128, 128, 5000)


def test_tree_binding_checks_shapes():
    q, k = torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 3, 2, 128, dtype=torch.bfloat16)
    ws = torch.zeros(16, dtype=torch.uint8)
    f = lambda q=q, k=k, v=k, mask=None, out=q: L.qjl_tree_attention(  # noqa: E731
        q, k, v, mask, 128, q, None, None, 0, None, None, None, 4, L.rq_lloyd_max(4), out, ws, 1.0, stream=0)
    for bad in (lambda: f(k=k[:, :2]), lambda: f(v=k[:1]), lambda: f(out=q[:, :2]), lambda: f(q=q[:, :, :3], out=q[:, :, :3]),
                lambda: f(mask=torch.zeros(2, 3, dtype=torch.int64)), lambda: f(mask=torch.zeros(3, 3, 1, dtype=torch.int64)),
                lambda: f(mask=torch.zeros(2, 3, 1, dtype=torch.int32)), lambda: f(q=q.transpose(2, 3), out=q.transpose(2, 3))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        f(q=q.half())


def test_tree_kernel_takes_the_same_way_after_an_expired_wait():
    """Every wait between the roles of the tree kernel has a limit, and none of them decides what a warp does next: a
    warp that went another way after an expired wait would leave its group's barriers, which have no limit, for good."""
    with open(os.path.join(os.path.dirname(L.LIB_PATH), "csrc", "qjl_tree.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernel = text[text.index("tree_attention_kernel("):text.index("tree_prologue_kernel(")]
    roles = kernel[kernel.index("tr_wait_previous();"):kernel.rindex("__syncthreads();")]
    assert re.search(r"void tr_wait\(uint64_t \*bar, uint32_t parity, uint32_t &limit\)", text)
    assert re.search(r"void tr_vote_wait\(", text)             # neither has an answer
    assert "break" not in roles and "__syncthreads" not in roles and "try_wait" not in roles
    # the remaining ones: the last copy and products of the issuing warps, whose answer is not looked at
    assert re.findall(r"(.*)\bmbar_wait(?:_limit)?\((.*?),", roles) == [
        ("        if (loads > 0) ", "q_full"), ("        ", "&drained[0]"), ("        ", "&drained[1]")]
    assert len(re.findall(r"\blimit\b", roles)) == len(re.findall(r", limit\)", roles)) + 3    # its start, the copies


# ------------------------------------------------------------------ arrays that a kernel would misread or leave

def zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def call_accumulate(**kw):
    a = dict(scores=zeros(2, 3, 8), acc=zeros(2, 8), out=zeros(2, 8), workspace=zeros(64, dtype=torch.uint8),
             row_len=zeros(2, 3, dtype=torch.int32))
    a.update(kw)
    L.rq_evict_accumulate(a["scores"], 2, 3, 8, 1.0, a.get("decay", 1.0), a["acc"], a["out"], a["workspace"], row_len=a["row_len"], stream=0)


def call_select(**kw):
    a = dict(acc=zeros(2, 8), idx=zeros(2, 4, dtype=torch.int32), count=zeros(2, dtype=torch.int32),
             length=zeros(2, dtype=torch.int32))
    a.update(kw)
    L.rq_evict_select(a["acc"], 2, 8, 4, a["idx"], a["count"], length=a["length"], stream=0)


def call_gather(**kw):
    a = dict(idx=zeros(2, 4, dtype=torch.int32), count=zeros(2, dtype=torch.int32), src=zeros(2, 8, 3), dst=zeros(2, 4, 3))
    a.update(kw)
    L.rq_evict_gather(a["idx"], a["count"], 2, 4, 8, [(a["src"], a["dst"])], stream=0)


def call_rotary(**kw):
    x = zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    L.rq_rotary(x, x, zeros(2, 3, dtype=torch.int64), np.ones(32), 64, 0, stream=0, **kw)


def call_tree(**kw):
    B, n, kv, rep, m, T, d = 2, 3, 2, 2, 128, 10, 128
    rows = B * kv * T
    q, k = zeros(B, n, kv * rep, d, dtype=torch.bfloat16), zeros(B, n, kv, d, dtype=torch.bfloat16)
    a = dict(proj=zeros(m, d, dtype=torch.bfloat16), signs=zeros(rows, m // 8, dtype=torch.uint8),
             sk=zeros(rows, dtype=torch.int16), kv_len=zeros(B * kv, dtype=torch.int32),
             v_codes=zeros(rows, 64, dtype=torch.uint8), v_norms=zeros(rows, dtype=torch.float16),
             codes=zeros(rows, 32, dtype=torch.uint8), norms=zeros(rows, dtype=torch.float16), mask=None,
             ws=zeros(64, dtype=torch.uint8), vc=L.rq_lloyd_max(4), kc=L.rq_lloyd_max(2))
    a.update(kw)
    L.qjl_tree_attention(q, k, k, a["mask"], m, a["proj"], a["signs"], a["sk"], T, a["kv_len"], a["v_codes"], a["v_norms"],
                         4, a["vc"], q, a["ws"], 1.0, codes=a["codes"], norms=a["norms"], bits=2, centroids=a["kc"],
                         stream=0)


def odd(t):
    """The same shape and values, in another order of memory."""
    return t.transpose(0, -1).contiguous().transpose(0, -1)


@pytest.mark.parametrize("call, name, bad, error", [
    (call_accumulate, "out", zeros(2, 8, dtype=torch.float16), TypeError), (call_accumulate, "out", zeros(2, 7), ValueError),
    (call_accumulate, "out", odd(zeros(2, 8)), ValueError),
    (call_accumulate, "scores", zeros(2, 3, 8, dtype=torch.bfloat16), TypeError),
    (call_accumulate, "scores", zeros(2, 2, 8), ValueError), (call_accumulate, "scores", odd(zeros(2, 3, 8)), ValueError),
    (call_accumulate, "acc", zeros(2, 8, dtype=torch.float16), TypeError), (call_accumulate, "acc", zeros(1, 8), ValueError),
    (call_accumulate, "row_len", zeros(2, 3, dtype=torch.int64), TypeError),
    (call_accumulate, "row_len", zeros(2, dtype=torch.int32), ValueError),
    (call_accumulate, "workspace", zeros(64, 2)[:, :1], ValueError),
    (call_select, "acc", zeros(2, 8, dtype=torch.float64), TypeError), (call_select, "acc", zeros(2, 16)[:, ::2], ValueError),
    (call_select, "idx", zeros(2, 4, dtype=torch.int64), TypeError), (call_select, "idx", zeros(2, 3, dtype=torch.int32), ValueError),
    (call_select, "count", zeros(2, dtype=torch.int64), TypeError), (call_select, "count", zeros(1, dtype=torch.int32), ValueError),
    (call_select, "length", zeros(2, dtype=torch.int64), TypeError), (call_select, "length", zeros(1, dtype=torch.int32), ValueError),
    (call_gather, "idx", zeros(2, 4, dtype=torch.int64), TypeError), (call_gather, "idx", zeros(7, dtype=torch.int32), ValueError),
    (call_gather, "count", zeros(2, dtype=torch.int64), TypeError), (call_gather, "src", odd(zeros(2, 8, 3)), ValueError),
    (call_gather, "src", zeros(2, 7, 3), ValueError), (call_gather, "dst", odd(zeros(2, 4, 3)), ValueError),
    (call_tree, "proj", zeros(128, 128), TypeError), (call_tree, "proj", zeros(64, 128, dtype=torch.bfloat16), ValueError),
    (call_tree, "signs", odd(zeros(40, 16, dtype=torch.uint8)), ValueError), (call_tree, "signs", zeros(39, 16, dtype=torch.uint8), ValueError),
    (call_tree, "sk", zeros(40), TypeError), (call_tree, "sk", zeros(39, dtype=torch.int16), ValueError),
    (call_tree, "kv_len", zeros(4, dtype=torch.int64), TypeError), (call_tree, "kv_len", zeros(2, dtype=torch.int32), ValueError),
    (call_tree, "v_codes", zeros(40, 32, dtype=torch.uint8), ValueError),
    (call_tree, "v_codes", odd(zeros(40, 64, dtype=torch.uint8)), ValueError),
    (call_tree, "v_norms", zeros(40), TypeError), (call_tree, "v_norms", zeros(20, dtype=torch.float16), ValueError),
    (call_tree, "codes", zeros(40, 16, dtype=torch.uint8), ValueError), (call_tree, "norms", zeros(40), TypeError),
    (call_tree, "norms", zeros(40, dtype=torch.bfloat16), TypeError),
    (call_tree, "mask", zeros(2, 3, 1, dtype=torch.float64), ValueError), (call_tree, "ws", zeros(64, 2)[:, :1], ValueError),
    (call_tree, "vc", L.rq_lloyd_max(3), ValueError), (call_tree, "kc", L.rq_lloyd_max(1), ValueError),
])
def test_binding_refuses_arrays_of_other_types_sizes_and_orders(call, name, bad, error):
    with pytest.raises(error, match="expected"):
        call(**{name: bad})


@pytest.mark.parametrize("call", [call_accumulate, call_select, call_gather, call_rotary, call_tree])
def test_binding_refuses_tensors_that_are_not_on_a_gpu(call):
    """Tensors that are right but for the memory they lie in: their addresses mean nothing to a kernel."""
    with pytest.raises(ValueError, match="on one GPU"):
        call()


def test_accumulate_without_history_does_not_look_at_the_old_sums():
    with pytest.raises(ValueError, match="on one GPU"):         # the only thing wrong here
        call_accumulate(decay=0.0, acc=zeros(3, dtype=torch.float16))


def test_gather_of_an_empty_cache_is_a_noop_for_the_library():
    rows = (L.Rows * 1)()
    rows[0].src, rows[0].dst, rows[0].row_bytes = A, A + 0x1000, 12
    assert L.lib().rq_evict_gather(A, A, 2, 4, 0, 4, C.addressof(rows), 1, None) == 0


@pytest.mark.parametrize("stream, raw", [(None, 77), (5, 5), (type("S", (), {"cuda_stream": 9}), 9)])
@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_the_device_of_their_tensors(monkeypatch, stream, raw, current):
    """Also when another device is current and a stream is given: the legacy stream of the current device would run the
    kernel there, on addresses of another device."""
    state, seen = dict(device=current), []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, state["device"] = state["device"], self.index

        def __exit__(self, *exc):
            state["device"] = self.before

    fake = type("Lib", (), {"rq_evict_select": staticmethod(lambda *a: seen.append((state["device"], a)) or 0)})
    monkeypatch.setattr(L, "_lib", fake)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["device"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: {1: 77}[i], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    L._call("rq_evict_select", type("T", (), {"get_device": staticmethod(lambda: 1)}), stream, ("x",))
    assert seen == [(1, ("x", raw))] and state["device"] == current

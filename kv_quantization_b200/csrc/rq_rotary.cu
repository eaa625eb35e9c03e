// rq_rotary.cu -- rotary positions of query and key heads.
//
//   (u, v) = scale (a cos t - b sin t, b cos t + a sin t),   t = position * freq_i
// for the pairs (a, b) = (x_i, x_{i + rot/2}) or (x_2i, x_2i+1), i < rot / 2; the other d - rot values of a
// head are copied.  The transpose (sin -> -sin) is the inverse rotation times scale^2: the gradient.
//
// Angles are kept in turns as 64-bit fixed point: position * F mod 2^64, F = round(freq / 2 pi * 2^64), is the
// angle modulo a full turn with no cancellation at any position (an error of |position| (1 + freq) 2^-65 turns from
// rounding F), so a far position costs one integer multiply instead of a float64 range reduction; its top 32 bits go to
// sincospif.
//
// Bound by HBM: every value is read and written once.  A CTA takes a few tokens; their cosines and sines are
// computed once into shared memory and then used for all heads (the angle does not depend on the head), each
// thread holding the factors of its V pairs in registers while it walks the heads.
#include "rq_common.cuh"
#include "rq_cache_ops.h"

namespace rq {

namespace {

constexpr int kRoThreads = 256;

template <int V> struct RoVec;                          // V 16-bit values
template <> struct RoVec<8> { uint32_t w[4]; };
template <> struct RoVec<4> { uint32_t w[2]; };
template <> struct RoVec<2> { uint32_t w[1]; };
template <> struct RoVec<1> { uint16_t w[1]; };

template <int V>
__device__ __forceinline__ RoVec<V> ro_load(const uint16_t *p)
{
    RoVec<V> r;
    if constexpr (V == 8) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else if constexpr (V == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = v.x; r.w[1] = v.y;
    } else if constexpr (V == 2) {
        r.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
        r.w[0] = *p;
    }
    return r;
}

template <int V>
__device__ __forceinline__ void ro_store(uint16_t *p, const RoVec<V> &r)
{
    if constexpr (V == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else if constexpr (V == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
    else if constexpr (V == 2) *reinterpret_cast<uint32_t *>(p) = r.w[0];
    else *p = r.w[0];
}

template <int V, bool BF16>
__device__ __forceinline__ void ro_unpack(const RoVec<V> &r, float *f)
{
    if constexpr (V == 1) {
        f[0] = BF16 ? __uint_as_float((uint32_t)r.w[0] << 16) : h16_to_f32(r.w[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) unpack2<BF16>(r.w[i], f[2 * i], f[2 * i + 1]);
    }
}

template <int V, bool BF16>
__device__ __forceinline__ RoVec<V> ro_pack(const float *f)
{
    RoVec<V> r;
    if constexpr (V == 1) {
        r.w[0] = (uint16_t)(pack2<BF16>(f[0], 0.0f) & 0xffffu);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r.w[i] = pack2<BF16>(f[2 * i], f[2 * i + 1]);
    }
    return r;
}

// Grid (token blocks, head blocks).  A thread is (item, slot): the item is one vector pair of a head (V pairs to
// rotate, or 2 V values to copy), the slot a token of the block and the first head; it walks heads in steps of hs.
template <int V, bool BF16, bool HALF>
__global__ void __launch_bounds__(kRoThreads)
rotary_kernel(const __grid_constant__ RotaryArgs a)
{
    extern __shared__ float2 cs[];                      // [TB][rot / 2] (cos, sin)
    const int half = a.rot / 2, nr = half / V, tid = threadIdx.x;
    const int64_t tok0 = (int64_t)blockIdx.x * a.tb;
    for (int i = tid; i < a.tb * half; i += kRoThreads) {
        const int tb = i / half, f = i - tb * half;
        const int64_t tok = tok0 + tb;
        if (tok >= a.B * a.n_tok) break;
        const int64_t b = tok / a.n_tok;
        const uint64_t pos = (uint64_t)__ldg(a.positions + b * a.pos_batch_stride + (tok - b * a.n_tok));
        const int32_t top = (int32_t)((pos * a.turns[f]) >> 32);       // turns, modulo 1, in [-1/2, 1/2)
        float s, c;
        sincospif((float)top * 0x1p-31f, &s, &c);
        cs[i] = make_float2(c * a.scale, (a.inverse ? -s : s) * a.scale);
    }
    __syncthreads();
    const int item = tid % a.items, slot = tid / a.items;
    const int tb = slot / a.hs, h0 = slot - tb * a.hs;
    const int64_t tok = tok0 + tb;
    if (tb >= a.tb || tok >= a.B * a.n_tok) return;
    const int64_t b = tok / a.n_tok, t = tok - b * a.n_tok;
    const bool rotate = item < nr;
    // element offsets of the item's two vectors in the head
    int o0, o1;
    if (rotate) {
        o0 = HALF ? item * V : item * 2 * V;
        o1 = HALF ? half + item * V : item * 2 * V + V;
    } else {
        o0 = a.rot + (item - nr) * 2 * V;
        o1 = o0 + V;
    }
    const bool two = o1 < a.d;                          // the last copied vector may stand alone
    float c[V], s[V];
    if (rotate) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float2 w = cs[tb * half + item * V + e];
            c[e] = w.x;
            s[e] = w.y;
        }
    }
    const int n_all = a.n_heads + a.n_heads2;
    const int h_end = min(n_all, ((int)blockIdx.y + 1) * a.heads_per_block);
    const int64_t ib = b * a.x.in_batch + t * a.x.in_token, ob = b * a.x.out_batch + t * a.x.out_token;
    const int64_t ib2 = b * a.x2.in_batch + t * a.x2.in_token, ob2 = b * a.x2.out_batch + t * a.x2.out_token;
    constexpr int U = 5;                                // heads in flight
    for (int hb = blockIdx.y * a.heads_per_block + h0; hb < h_end; hb += U * a.hs) {
        RoVec<V> v0[U], v1[U];
        uint16_t *out[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = hb + k * a.hs;
            if (h >= h_end) break;
            const bool second = h >= a.n_heads;
            const int hh = second ? h - a.n_heads : h;
            const uint16_t *in = second ? a.x2.in + ib2 + hh * a.x2.in_head : a.x.in + ib + hh * a.x.in_head;
            out[k] = second ? a.x2.out + ob2 + hh * a.x2.out_head : a.x.out + ob + hh * a.x.out_head;
            v0[k] = ro_load<V>(in + o0);
            if (two) v1[k] = ro_load<V>(in + o1);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (hb + k * a.hs >= h_end) break;
            if (!rotate) {
                ro_store<V>(out[k] + o0, v0[k]);
                if (two) ro_store<V>(out[k] + o1, v1[k]);
                continue;
            }
            float p[V], q[V], u[V], w[V];
            ro_unpack<V, BF16>(v0[k], p);
            ro_unpack<V, BF16>(v1[k], q);
            if constexpr (HALF) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    u[e] = __fmaf_rn(p[e], c[e], -(q[e] * s[e]));
                    w[e] = __fmaf_rn(q[e], c[e], p[e] * s[e]);
                }
            } else {                                    // values 2e, 2e + 1 of the 2 V in (p, q)
                float z[2 * V], y[2 * V];
#pragma unroll
                for (int e = 0; e < V; ++e) { z[e] = p[e]; z[V + e] = q[e]; }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    y[2 * e] = __fmaf_rn(z[2 * e], c[e], -(z[2 * e + 1] * s[e]));
                    y[2 * e + 1] = __fmaf_rn(z[2 * e + 1], c[e], z[2 * e] * s[e]);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) { u[e] = y[e]; w[e] = y[V + e]; }
            }
            ro_store<V>(out[k] + o0, ro_pack<V, BF16>(u));
            ro_store<V>(out[k] + o1, ro_pack<V, BF16>(w));
        }
    }
}

template <int V>
cudaError_t ro_launch(RotaryArgs a, cudaStream_t st)
{
    a.items = a.rot / 2 / V + (a.copy ? (a.d - a.rot + 2 * V - 1) / (2 * V) : 0);
    const int slots = kRoThreads / a.items, heads = a.n_heads + a.n_heads2;
    const int64_t tokens = a.B * a.n_tok;
    // Few tokens (a decode step): one head per thread, one token per CTA, heads spread over CTAs.  Many: about
    // five heads per thread, so that the cosines in its registers are used again, and several tokens per CTA.
    a.hs = tokens * heads * a.items < 4096 * kRoThreads ? heads : (heads + 4) / 5;
    if (a.hs > slots) a.hs = slots;
    a.tb = slots / a.hs;
    a.heads_per_block = heads;
    if (a.tb == 1 && a.hs == slots && tokens < 2 * a.num_sms && heads / a.hs < 65535) a.heads_per_block = a.hs;
    if (a.tb > 1 && tokens < 2 * a.num_sms) a.tb = 1;
    const int64_t gx = (tokens + a.tb - 1) / a.tb;
    if (gx > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)gx, (unsigned)((heads + a.heads_per_block - 1) / a.heads_per_block));
    const size_t smem = (size_t)a.tb * (a.rot / 2) * sizeof(float2);
    if (a.bf16) {
        if (a.half) rotary_kernel<V, true, true><<<grid, kRoThreads, smem, st>>>(a);
        else rotary_kernel<V, true, false><<<grid, kRoThreads, smem, st>>>(a);
    } else {
        if (a.half) rotary_kernel<V, false, true><<<grid, kRoThreads, smem, st>>>(a);
        else rotary_kernel<V, false, false><<<grid, kRoThreads, smem, st>>>(a);
    }
    note_launch("rotary_kernel");
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, cudaStream_t st)
{
    // the widest vector that divides the pairs, the copied tail, every stride and every base address
    int64_t all = (int64_t)(a.rot / 2) | (a.d - a.rot);
    for (const RotaryTensor *t : {&a.x, &a.x2}) {
        if (t->in == nullptr) continue;
        all |= t->in_batch | t->in_token | t->in_head | t->out_batch | t->out_token | t->out_head;
        all |= (int64_t)((reinterpret_cast<uintptr_t>(t->in) | reinterpret_cast<uintptr_t>(t->out)) / sizeof(uint16_t));
    }
    if (all % 8 == 0) return ro_launch<8>(a, st);
    if (all % 4 == 0) return ro_launch<4>(a, st);
    if (all % 2 == 0) return ro_launch<2>(a, st);
    return ro_launch<1>(a, st);
}

}  // namespace rq

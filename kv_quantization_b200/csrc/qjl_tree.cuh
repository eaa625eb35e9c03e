// qjl_tree.cuh -- attention of a tree of drafted tokens over the compressed cache (sm_100a).
//
// Query row r = (node i, head h of the key head's rep) of group g = (sequence, key head) attends to the group's
// len cached tokens (QJL / two-stage score s, values vh reconstructed from codes) and to the drafted tokens j that
// its node sees (16-bit k_j, v_j), under one softmax:
//   out = (sum_t e^(c s(r,t)) vh_t + sum_j e^(c <q,k_j>) v_j) / (sum_t e^(c s) + sum_j e^(c <q,k_j>)),   0 where it sees nothing.
// With one node it is the ordinary decode step.
//
// Three kernels:
//   tree_prologue_kernel   the score operand of every row, [H D q ; S q] / |q| in fp16, written as the image of the
//                          shared-memory operand (so that the main kernel fetches it with one bulk copy); the
//                          prefix sums of the groups' tiles;
//   tree_attention_kernel  the cached part, split evenly over the SMs whatever the lengths: (m, l, O) per segment;
//   tree_combine_kernel    joins a row's segments with its drafted part, rotates back, divides and rounds.
//
// Main kernel, per 128-token tile and block of NB query rows.  Tokens are the M dimension of the score product
// (S^T = K . Q^T, one token a TMEM lane), so that every lane works however few rows there are, and a thread's
// token-wise factors are its own registers:
//   producers (8 warps)  thread = token and half of its slices: 64 key values a slice are unpacked to fp16 and stored
//                        to TMEM, where the score product reads its A operand: unpacked keys never pass through
//                        shared memory, whose bandwidth bounds this kernel otherwise.  Then half the token's values,
//                        V' = fp16(c) * fp16(n / d), to shared memory.
//   MMA 1 (one thread)   S^T[token][row] += K slice (TMEM) . Q^T slice (shared memory).
//   softmax (8 warps)    thread = token and half of the rows: p = 2^(s g cq + (8 - ref)), fp16 P to shared memory.  The
//                        reference `ref` of a row is the maximum of the segment's first tile and moves only when a
//                        score passes it by 7 (2^15 is the most fp16 weights take): the usual tile needs one vote
//                        and no reduction over tokens.
//   MMA 2 (one thread)   O^T[d][row] += V'^T . P, accumulated in TMEM over the segment.
#pragma once
#include "rq_cache_ops.h"
#include "rq_common.cuh"
#include "sm100.cuh"

namespace rq {

constexpr int kTrTok = 128;                       // tokens a tile (M of both products' token side)
constexpr int kTrD = 128;
constexpr int kTrThreads = 18 * 32;
constexpr int kTrVBytes = kTrTok * kTrD * 2;      // one value tile, fp16
constexpr float kTrShift = 8.0f;                  // weight of the reference: 2^8
constexpr float kTrMost = 15.0f;                  // largest exponent an fp16 weight may have

__host__ __device__ inline int tr_kslots(int nb) { return nb == 128 ? 4 : 8; }
__host__ __device__ inline size_t tr_pbytes(int nb) { return (size_t)(nb > 64 ? 2 : 1) * kTrTok * 128; }
__host__ __device__ inline size_t tr_lut_bytes(int pw, int copies)
{
    return pw == 0 ? 0 : pw <= 4 ? ((size_t)1 << (2 * pw)) * copies * 4 : ((size_t)256 * copies * 2);
}
__host__ __device__ inline size_t tr_smem(int nb, int kb, int pw, int vpw, int np, int copies)
{
    return 1024 + (size_t)nb * kb * 2 + 2 * kTrVBytes + np * tr_pbytes(nb) + tr_lut_bytes(pw, copies) +
           tr_lut_bytes(vpw, copies) + (size_t)nb * 12 + (size_t)4 * nb * 4 + 8 * 40 + 16;
}
// Partial result of one (CTA, row block) segment: O [nb][128], m [nb], l [nb].
__host__ __device__ inline size_t tr_part_floats(int nb) { return (size_t)nb * (kTrD + 2); }

__device__ __forceinline__ float tr_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tr_bar(int id)
{
    asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}

__device__ __forceinline__ bool tr_bar_or(int id, bool p)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(p ? 1u : 0u), "r"(id)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void tr_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], kind::f16.
__device__ __forceinline__ void mma_f16_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
        "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
        "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint64_t tr_sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo)
{
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3ffffu) >> 4);
    d |= (uint64_t)((lbo >> 4) & 0x3fffu) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3fffu) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Reduce v[0 .. N) over the 32 lanes of a warp (N = 32 or 16): lane l returns the result of column l % N.
template <int N, typename Op>
__device__ __forceinline__ float tr_reduce_columns(float *v, int lane, Op op)
{
#pragma unroll
    for (int o = N / 2; o >= 1; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    }
    float x = v[0];
    if (N == 16) x = op(x, __shfl_xor_sync(0xffffffffu, x, 16));
    return x;
}

__device__ __forceinline__ int64_t tr_len(const TreeArgs &a, int64_t g)
{
    if (!a.kv_len) return a.T;
    const int64_t n = __ldg(a.kv_len + g);
    return n < 0 ? 0 : (n < a.T ? n : a.T);
}

// Position in the list of (group, row block, tile) items: group g's items are [off[g] rb_count, off[g+1] rb_count).
struct TreeIter {
    int64_t g, n, tile;
    int rb;
    __device__ void seek(const int64_t *off, int64_t G, int rbs, int64_t it)
    {
        int64_t lo = 0, hi = G;                   // off[lo] rbs <= it < off[hi] rbs
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (off[mid] * rbs <= it) lo = mid; else hi = mid;
        }
        g = lo;
        n = off[g + 1] - off[g];
        const int64_t rest = it - off[g] * rbs;
        rb = (int)(rest / n);
        tile = rest - rb * n;
    }
    // advance by one item (the caller knows that there is one); true when the row block changes
    __device__ bool next(const int64_t *off, int rbs)
    {
        if (++tile < n) return false;
        tile = 0;
        if (++rb == rbs) {
            rb = 0;
            do {
                ++g;
                n = off[g + 1] - off[g];
            } while (n == 0);
        }
        return true;
    }
};

// 32 sign bits to fp16 +-mag, 16 pairs.  Pair i is (bit i, bit i + 16): one shift and one masked or; the score
// product sums over all of them, so the query operand has its coordinates in the same order (tr_sign_column).
__device__ __forceinline__ void tr_signs(uint32_t w, uint32_t mag2, uint32_t *o)
{
    const uint32_t n = ~w;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = mag2 | ((n << (15 - i)) & 0x80008000u);
}
// Column, in its 64-column slice, of sketch coordinate i (0 .. 63).
__host__ __device__ inline int tr_sign_column(int i) { return (i & 32) | ((i & 15) << 1) | ((i >> 4) & 1); }

// 64 codes of PW bits (kc) to 32 pairs of fp16 centroids.
template <int PW>
__device__ __forceinline__ void tr_lookup(const uint32_t *kc, const uint32_t *lut, int copies_log2, uint32_t lane_copy, uint32_t *o)
{
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if constexpr (PW <= 4) {
            o[i] = lut[(unpack_code<32, 2 * PW>(kc, i) << copies_log2) + lane_copy];
        } else {
            const uint32_t ca = unpack_code<64, PW>(kc, 2 * i), cb = unpack_code<64, PW>(kc, 2 * i + 1);
            const uint16_t *l16 = reinterpret_cast<const uint16_t *>(lut);
            o[i] = (uint32_t)l16[(ca << copies_log2) + lane_copy] | ((uint32_t)l16[(cb << copies_log2) + lane_copy] << 16);
        }
    }
}

__device__ __forceinline__ void tr_lookup_any(int pw, const uint32_t *kc, const uint32_t *lut, int cl, uint32_t lc, uint32_t *o)
{
    switch (pw) {
    case 1: tr_lookup<1>(kc, lut, cl, lc, o); break;
    case 2: tr_lookup<2>(kc, lut, cl, lc, o); break;
    case 3: tr_lookup<3>(kc, lut, cl, lc, o); break;
    case 4: tr_lookup<4>(kc, lut, cl, lc, o); break;
    default: tr_lookup<8>(kc, lut, cl, lc, o); break;
    }
}

// 8 pw bytes (64 codes) at p, 8-byte aligned.
__device__ __forceinline__ void tr_load_codes(const uint8_t *p, int pw, bool valid, uint32_t *w)
{
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        uint2 v = make_uint2(0u, 0u);
        if (q < pw && valid) v = __ldg(reinterpret_cast<const uint2 *>(p) + q);
        w[2 * q] = v.x;
        w[2 * q + 1] = v.y;
    }
}

template <int NB>
__global__ void __launch_bounds__(kTrThreads, 1)
tree_attention_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ QuantTables TK,
                      const __grid_constant__ QuantTables TV, int np, int copies_log2)
{
    constexpr int CW = NB / 2, CH = CW < 32 ? CW : 32, NCH = CW / CH;
    constexpr int KS = NB == 128 ? 4 : 8;         // key slots in TMEM
    const bool two = a.pw != 0;
    const int kb = a.kb, nsl = kb / 64, dsl = two ? 2 : 0;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = base;
    uint8_t *sV = sQ + (size_t)NB * kb * 2;
    uint8_t *sP = sV + 2 * kTrVBytes;
    uint32_t *klut = reinterpret_cast<uint32_t *>(sP + np * tr_pbytes(NB));
    uint32_t *vlut = klut + tr_lut_bytes(a.pw, 1 << copies_log2) / 4;
    float *sF = reinterpret_cast<float *>(vlut + tr_lut_bytes(a.vpw, 1 << copies_log2) / 4);   // per pair of rows: cq, cq, 8 - ref, 8 - ref
    float *sAl = sF + 2 * NB;                     // [NB] rescale factors
    float *sX = sAl + NB;                         // [4][NB] column reductions by lane quarter
    uint64_t *k_full = reinterpret_cast<uint64_t *>(sX + 4 * NB);
    uint64_t *k_empty = k_full + KS;
    uint64_t *v_full = k_empty + KS;              // [2]
    uint64_t *s_full = v_full + 2;                // [2]
    uint64_t *s_empty = s_full + 2;               // [2]
    uint64_t *p_full = s_empty + 2;               // [2]
    uint64_t *pv_done = p_full + 2;               // [2] by tile parity: P, V free, O holds the tile
    uint64_t *o_empty = pv_done + 2;
    uint64_t *q_full = o_empty + 1;
    uint64_t *q_done = q_full + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(q_done + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t quarter = (uint32_t)(warp & 3);
    const int copies = 1 << copies_log2;
    auto fill = [&](const QuantTables &T, uint32_t *lut, int pw) {
        if (pw == 0) return;
        if (pw <= 4) {
            for (int i = tid; i < (1 << (2 * pw)) * copies; i += kTrThreads) {
                const int e = i >> copies_log2, ca = e & ((1 << pw) - 1), cb = e >> pw;
                const float fa = ca < T.levels ? T.centroid[ca] : 0.0f, fb = cb < T.levels ? T.centroid[cb] : 0.0f;
                lut[i] = (uint32_t)__half_as_ushort(__float2half_rn(fa)) |
                         ((uint32_t)__half_as_ushort(__float2half_rn(fb)) << 16);
            }
        } else {
            uint16_t *l16 = reinterpret_cast<uint16_t *>(lut);
            for (int i = tid; i < 256 * copies; i += kTrThreads) {
                const int e = i >> copies_log2;
                l16[i] = __half_as_ushort(__float2half_rn(e < T.levels ? T.centroid[e] : 0.0f));
            }
        }
    };
    fill(TK, klut, a.pw);
    fill(TV, vlut, a.vpw);
    if (tid == 0) {
        for (int b = 0; b < KS; ++b) { mbar_init(&k_full[b], 4); mbar_init(&k_empty[b], 1); }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&v_full[b], 8);
            mbar_init(&s_full[b], 1); mbar_init(&s_empty[b], 8);
            mbar_init(&p_full[b], 8); mbar_init(&pv_done[b], 1);
        }
        mbar_init(o_empty, 8);
        mbar_init(q_full, 1);
        mbar_init(q_done, 1);
        fence_barrier_init();
    }
    if (warp == 16) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem, tO = tmem + 2 * NB, tK = tmem + 3 * NB;

    const int64_t total = a.off[a.G] * a.rbs;
    const int64_t it0 = total * blockIdx.x / gridDim.x, it1 = total * (blockIdx.x + 1) / gridDim.x;
    const int64_t count = it1 - it0;
    bool ok = true;
    TreeIter it;
    if (count > 0) it.seek(a.off, a.G, a.rbs, it0);

    if (count > 0 && warp >= 8 && warp < 16) {
        // ------------------------------------------------------------ producers
        const int half = (warp - 8) >> 2;
        const int r = (int)quarter * 32 + lane;                 // token of the tile
        const uint32_t sbytes = (uint32_t)a.m / 8, cbytes = 16u * a.pw, vbytes = 16u * a.vpw;
        const float kq = 1.2533141373155002512f / (float)a.m;
        const uint32_t lc = (uint32_t)lane & (uint32_t)(copies - 1);
        const int nsig = nsl - dsl;
        uint2 sg[4];                                            // sign slices half, half + 2, ... of the sketch
        uint32_t kc[16], vc[16];
        uint16_t hn = 0, hr = 0, hv = 0;                        // first-stage, sketch and value norm
        auto load_keys = [&](const TreeIter &p) {
            const int64_t t = p.tile * kTrTok + r, kt = p.g * a.T + t;
            const bool valid = t < tr_len(a, p.g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sg[i] = make_uint2(0u, 0u);
                if (2 * i + half < nsig && valid)
                    sg[i] = __ldg(reinterpret_cast<const uint2 *>(a.signs + kt * sbytes) + 2 * i + half);
            }
            if (two) {
                tr_load_codes(a.codes + kt * cbytes + half * 8 * a.pw, a.pw, valid, kc);
                hn = valid ? __ldg(a.norms + kt) : (uint16_t)0;
                hr = valid ? __ldg(a.sk_norms + kt) : (uint16_t)0;
            }
        };
        auto load_values = [&](const TreeIter &p) {
            const int64_t t = p.tile * kTrTok + r, kt = p.g * a.T + t;
            const bool valid = t < tr_len(a, p.g);
            tr_load_codes(a.vcodes + kt * vbytes + half * 8 * a.vpw, a.vpw, valid, vc);
            hv = valid ? __ldg(a.vnorms + kt) : (uint16_t)0;
        };
        load_keys(it);
        load_values(it);
        int64_t pos0 = 0;                                       // slices before this tile
        for (int64_t c = 0; c < count && ok; ++c, pos0 += nsl) {
            uint32_t rho2 = 0x3C003C00u;
            if (two) {
                // the sketch term scaled to share the first stage's accumulator and factor n / d
                const float n1 = h16_to_f32(hn);
                float rho = 0.0f;
                if (n1 > 0.0f) rho = __fdiv_rn(__fmul_rn(__fmul_rn(kq, h16_to_f32(hr)), (float)kTrD), n1);
                const uint32_t h = (uint32_t)__half_as_ushort(__float2half_rn(rho));
                rho2 = h | (h << 16);
            }
#pragma unroll
            for (int i = 0; i < 5; ++i) {                       // slice 2 i + half: a code slice, or sign slice - dsl
                const int s = 2 * i + half;
                if (s >= nsl) break;
                const int64_t pos = pos0 + s;
                const int slot = (int)(pos % KS);
                uint32_t o[32];
                if (two && i == 0) {
                    tr_lookup_any(a.pw, kc, klut, copies_log2, lc, o);
                } else {
                    const int q = two ? i - 1 : i;
                    uint2 w = make_uint2(0u, 0u);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e == q) w = sg[e];
                    tr_signs(w.x, rho2, o);
                    tr_signs(w.y, rho2, o + 16);
                }
                if (pos >= KS && ok && !mbar_wait(&k_empty[slot], (uint32_t)((pos / KS - 1) & 1))) ok = false;
                tc_fence_after();
                const uint32_t dst = tK + (uint32_t)slot * 32u + (quarter << 21);
                tmem_st16(dst, o);
                tmem_st16(dst + 16, o + 16);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) tr_arrive(&k_full[slot]);
            }
            TreeIter nx = it;
            const bool more = c + 1 < count;
            if (more) {
                nx.next(a.off, a.rbs);
                load_keys(nx);
            }
            // half the value row: rows of tokens, two 64-wide atoms of d
            uint32_t o[32];
            tr_lookup_any(a.vpw, vc, vlut, copies_log2, lc, o);
            const float fv = __fmul_rn(h16_to_f32(hv), 1.0f / (float)kTrD);
            const __half2 f2 = __half2half2(__float2half_rn(fv));
            const int vb = (int)(c & 1);
            if (c >= 2 && ok && !mbar_wait(&pv_done[vb], (uint32_t)(((c >> 1) - 1) & 1))) ok = false;
            uint8_t *Vr = sV + (size_t)vb * kTrVBytes + (size_t)half * (kTrVBytes / 2) + (size_t)(r >> 3) * 1024 + (size_t)(r & 7) * 128;
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __half2 hv2 = __hmul2(*reinterpret_cast<const __half2 *>(&o[4 * ch + e]), f2);
                    w[e] = *reinterpret_cast<const uint32_t *>(&hv2);
                }
                *reinterpret_cast<uint4 *>(Vr + ((ch ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tr_arrive(&v_full[vb]);
            if (more) load_values(nx);
            it = nx;
        }
    } else if (count > 0 && warp == 16) {
        // ------------------------------------------------------------ MMA 1: S^T = K . Q^T
        const uint32_t sQ0 = smem_u32(sQ);
        const uint32_t idesc = idesc_f16(false, kTrTok, NB);
        const uint32_t qbytes = (uint32_t)NB * kb * 2;
        bool fresh = true;
        int64_t seg = 0, pos = 0;
        for (int64_t c = 0; c < count && ok; ++c) {
            if (fresh) {
                if (seg > 0) {
                    if (lane == 0) mma_commit(q_done);
                    if (!mbar_wait(q_done, (uint32_t)((seg - 1) & 1))) { ok = false; break; }
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, qbytes);
                    bulk_load(sQ, a.wsQ + (it.g * a.rbs + it.rb) * (int64_t)qbytes, qbytes, q_full);
                }
                if (!mbar_wait(q_full, (uint32_t)(seg & 1))) { ok = false; break; }
                ++seg;
            }
            const int sb = (int)(c & 1);
            if (c >= 2 && !mbar_wait(&s_empty[sb], (uint32_t)(((c >> 1) - 1) & 1))) { ok = false; break; }
            tc_fence_after();
            for (int s = 0; s < nsl; ++s, ++pos) {
                const int slot = (int)(pos % KS);
                if (!mbar_wait(&k_full[slot], (uint32_t)((pos / KS) & 1))) { ok = false; break; }
                tc_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f16_ta(tS + (uint32_t)sb * NB, tK + (uint32_t)slot * 32u + kk * 8u,
                                   sdesc_k_sw128(sQ0 + (uint32_t)s * (NB * 128u) + kk * 32u), idesc,
                                   (s > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(&k_empty[slot]);
                    if (s == nsl - 1) mma_commit(&s_full[sb]);
                }
                __syncwarp();
            }
            if (c + 1 < count) fresh = it.next(a.off, a.rbs);
        }
        if (seg > 0) {                                          // all products done before TMEM is freed
            if (lane == 0) mma_commit(q_done);
            if (ok) mbar_wait(q_done, (uint32_t)((seg - 1) & 1));
        }
    } else if (count > 0 && warp == 17) {
        // ------------------------------------------------------------ MMA 2: O^T += V'^T . P
        const uint32_t sP0 = smem_u32(sP), sV0 = smem_u32(sV);
        const uint32_t idesc = idesc_f16(false, kTrD, NB) | (1u << 15) | (1u << 16);    // both operands MN-major
        bool fresh = true;
        int64_t seg = 0;
        for (int64_t c = 0; c < count && ok; ++c) {
            const int b = (int)(c & 1), pb = np == 2 ? b : 0;
            if (fresh && seg++ > 0 && !mbar_wait(o_empty, (uint32_t)((seg - 2) & 1))) { ok = false; break; }
            if (!mbar_wait(&v_full[b], (uint32_t)((c >> 1) & 1))) { ok = false; break; }
            if (!mbar_wait(&p_full[b], (uint32_t)((c >> 1) & 1))) { ok = false; break; }
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_f16(tO, tr_sdesc(sV0 + (uint32_t)b * kTrVBytes + kk * 2048u, kTrVBytes / 2, 1024u),
                            tr_sdesc(sP0 + (uint32_t)pb * (uint32_t)tr_pbytes(NB) + kk * 2048u, kTrTok * 128u, 1024u), idesc,
                            (fresh && kk == 0) ? 0u : 1u);
                mma_commit(&pv_done[b]);
            }
            __syncwarp();
            fresh = c + 1 < count && it.next(a.off, a.rbs);
        }
    } else if (count > 0 && warp < 8) {
        // ------------------------------------------------------------ softmax
        const int w = warp >> 2, cb = w * CW, wt = tid & 127, bar = 1 + w;
        const int r = (int)quarter * 32 + lane;                 // token of the tile
        const uint32_t lanes = quarter << 21;
        const float kq = 1.2533141373155002512f / (float)a.m;
        const uint16_t *gsrc = two ? a.norms : a.sk_norms;
        const float gk = two ? 1.0f / (float)kTrD : kq;
        auto load_g = [&](const TreeIter &p) {
            const int64_t t = p.tile * kTrTok + r;
            return t < tr_len(a, p.g) ? h16_to_f32(__ldg(gsrc + p.g * a.T + t)) : -1.0f;   // norms are >= 0
        };
        float gn = load_g(it);
        float ref = -INFINITY;                                  // of column wt < CW
        float l[NCH == 2 ? 2 : CW];
        const float4 *F = reinterpret_cast<const float4 *>(sF) + cb / 2;
        bool fresh = true;
        for (int64_t c = 0; c < count; ++c) {                   // every item and barrier also after a wait has expired
            const int sb = (int)(c & 1);
            const int64_t pg = it.g * a.rbs + it.rb;
            const bool start = fresh;
            if (start) {
                if (wt < CW) {
                    const float cq = __ldg(a.wsC + pg * NB + cb + wt);
                    float *f = sF + ((cb + wt) >> 1) * 4 + (wt & 1);
                    f[0] = cq;
                    f[2] = 0.0f;
                }
                ref = -INFINITY;
#pragma unroll
                for (int j = 0; j < (NCH == 2 ? 2 : CW); ++j) l[j] = 0.0f;
                tr_bar(bar);
            }
            const bool valid = gn >= 0.0f;
            const float g = valid ? __fmul_rn(gn, gk) : 0.0f;
            TreeIter nx = it;
            fresh = false;
            if (c + 1 < count) {
                fresh = nx.next(a.off, a.rbs);
                gn = load_g(nx);
            }
            if (ok && !mbar_wait(&s_full[sb], (uint32_t)((c >> 1) & 1))) ok = false;
            tc_fence_after();
            uint32_t sr[CW];
            const uint32_t src = tS + (uint32_t)(sb * NB + cb) + lanes;
            auto load_s = [&]() {
                if constexpr (CW == 16) {
                    tmem_ld16(src, sr);
                } else {
#pragma unroll
                    for (int ch = 0; ch < NCH; ++ch) tmem_ld32(src + 32u * ch, sr + 32 * ch);
                }
                tmem_ld_wait();
            };
            // exponents a = s g cq + (8 - ref), in place of s; returns their maximum
            auto exponents = [&]() {
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < CW; j += 2) {
                    const float4 f = F[j >> 1];
                    const float2 x = __fmul2_rn(make_float2(__uint_as_float(sr[j]), __uint_as_float(sr[j + 1])), make_float2(g, g));
                    const float2 v = __ffma2_rn(x, make_float2(f.x, f.y), make_float2(f.z, f.w));
                    sr[j] = __float_as_uint(v.x);
                    sr[j + 1] = __float_as_uint(v.y);
                    mx = fmaxf(fmaxf(mx, v.x), v.y);
                }
                return mx;
            };
            load_s();
            const float mx = exponents();
            if (tr_bar_or(bar, start || (valid && mx > kTrMost))) {
                // new references: the maxima over the tile's tokens of s g cq
                float *X = sX + quarter * NB + cb;
#pragma unroll
                for (int ch = 0; ch < NCH; ++ch) {
                    uint32_t t32[CH];
                    if constexpr (CH == 16) tmem_ld16(src, t32);
                    else tmem_ld32(src + 32u * ch, t32);
                    tmem_ld_wait();
                    float v[CH];
#pragma unroll
                    for (int j = 0; j < CH; ++j) {
                        const float cq = sF[((cb + ch * CH + j) >> 1) * 4 + (j & 1)];
                        v[j] = valid ? __fmul_rn(__fmul_rn(__uint_as_float(t32[j]), g), cq) : -INFINITY;
                    }
                    const float x = tr_reduce_columns<CH>(v, lane, [](float p, float q) { return fmaxf(p, q); });
                    if (lane < CH) X[ch * CH + lane] = x;
                }
                tr_bar(bar);
                if (wt < CW) {
                    const float *x = sX + cb + wt;
                    const float mn = fmaxf(ref, fmaxf(fmaxf(x[0], x[NB]), fmaxf(x[2 * NB], x[3 * NB])));
                    sAl[cb + wt] = ref == -INFINITY ? 0.0f : tr_ex2(ref - mn);
                    sF[((cb + wt) >> 1) * 4 + 2 + (wt & 1)] = kTrShift - mn;
                    ref = mn;
                }
                tr_bar(bar);
                if constexpr (NCH == 2) {
                    l[0] *= sAl[cb + lane];
                    l[1] *= sAl[cb + 32 + lane];
                } else {
#pragma unroll
                    for (int j = 0; j < CW; ++j) l[j] *= sAl[cb + j];
                }
                if (!start) {                                   // O of the segment's earlier tiles
                    if (ok && !mbar_wait(&pv_done[(c - 1) & 1], (uint32_t)(((c - 1) >> 1) & 1))) ok = false;
                    tc_fence_after();
#pragma unroll
                    for (int ch = 0; ch < CW / 16; ++ch) {
                        uint32_t o[16];
                        const uint32_t at = tO + (uint32_t)(cb + 16 * ch) + lanes;
                        tmem_ld16(at, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__fmul_rn(__uint_as_float(o[j]), sAl[cb + 16 * ch + j]));
                        tmem_st16(at, o);
                    }
                    tmem_st_wait();
                }
                load_s();
                exponents();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) tr_arrive(&s_empty[sb]);
            // weights: row r of the [token][row] operand
            if (np == 2) {
                if (c >= 2 && ok && !mbar_wait(&pv_done[sb], (uint32_t)(((c >> 1) - 1) & 1))) ok = false;
            } else {
                if (c >= 1 && ok && !mbar_wait(&pv_done[(c - 1) & 1], (uint32_t)(((c - 1) >> 1) & 1))) ok = false;
            }
            uint8_t *Pr = sP + (size_t)(np == 2 ? sb : 0) * tr_pbytes(NB) + (size_t)(cb >> 6) * (kTrTok * 128) +
                          (size_t)(r >> 3) * 1024 + (size_t)(r & 7) * 128;
            const int ch0 = (cb & 63) >> 3;                     // 16-byte chunk of this half's first row
#pragma unroll
            for (int ch = 0; ch < CW / 8; ++ch) {
                uint32_t w4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 8 * ch + 2 * e;
                    const float p0 = valid ? tr_ex2(__uint_as_float(sr[j])) : 0.0f;
                    const float p1 = valid ? tr_ex2(__uint_as_float(sr[j + 1])) : 0.0f;
                    const __half2 h = __floats2half2_rn(p0, p1);
                    w4[e] = *reinterpret_cast<const uint32_t *>(&h);
                    if constexpr (NCH == 2) {
                        sr[j] = __float_as_uint(p0);
                        sr[j + 1] = __float_as_uint(p1);
                    } else {
                        l[j] += p0;
                        l[j + 1] += p1;
                    }
                }
                *reinterpret_cast<uint4 *>(Pr + (((ch0 + ch) ^ (r & 7)) << 4)) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tr_arrive(&p_full[sb]);
            if constexpr (NCH == 2) {                           // sums over the warp's tokens, column `lane` of each chunk
                auto add = [](float p, float q) { return p + q; };
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(sr[32 * ch + j]);
                    l[ch] += tr_reduce_columns<32>(v, lane, add);
                }
            }
            if (fresh || c + 1 == count) {                      // end of the segment
                if (ok && !mbar_wait(&pv_done[sb], (uint32_t)((c >> 1) & 1))) ok = false;
                tc_fence_after();
                float *part = a.part + (size_t)(blockIdx.x + pg) * tr_part_floats(NB);
#pragma unroll
                for (int ch = 0; ch < CW / 16; ++ch) {
                    uint32_t o[16];
                    tmem_ld16(tO + (uint32_t)(cb + 16 * ch) + lanes, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(size_t)(cb + 16 * ch + j) * kTrD + r] = __uint_as_float(o[j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) tr_arrive(o_empty);
                float *X = sX + quarter * NB + cb;
                if constexpr (NCH == 2) {
                    X[lane] = l[0];
                    X[32 + lane] = l[1];
                } else {
                    const float x = tr_reduce_columns<CW>(l, lane, [](float p, float q) { return p + q; });
                    if (lane < CW) X[lane] = x;
                }
                tr_bar(bar);
                if (wt < CW) {
                    const float *x = sX + cb + wt;
                    part[(size_t)NB * kTrD + cb + wt] = ref - kTrShift;
                    part[(size_t)NB * kTrD + NB + cb + wt] = (x[0] + x[NB]) + (x[2 * NB] + x[3 * NB]);
                }
                tr_bar(bar);
            }
            it = nx;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 16) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ prologue

__device__ __forceinline__ void tr_mma_bf16(float *d, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ const uint16_t *tr_row(const uint16_t *p, const rq_strides_t &s, const TreeArgs &a, int64_t g, int r)
{
    const int64_t b = g / a.kv_heads;
    const int kv = (int)(g - b * a.kv_heads), node = r / a.rep, h = r - node * a.rep;
    return p + b * s.batch + (int64_t)node * s.token + (int64_t)(kv * a.rep + h) * s.head;
}

// Grid (32-row tiles of every row block, 64-column slices); 4 warps, each 16 rows x 32 columns of
//   [q H D ; q S^T] / |q|
// as bf16 products with fp32 sums: the entries of H D are +-1, an fp16 projection is the sum of two bf16 numbers, so
// every product is exact.  A thread's 128-value rows are loaded as 64 contiguous bytes a lane of the quad; the sum
// over k runs in that order for both operands.  CTA (0, 0) also writes the prefix sums of the groups' tiles.
__global__ void __launch_bounds__(128)
tree_prologue_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ QuantTables TK)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, p = lane & 3, rr = lane >> 2;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        __shared__ int64_t sums[128];
        int64_t run = 0;
        for (int64_t g0 = 0; g0 < a.G; g0 += 128) {
            const int64_t g = g0 + tid;
            int64_t n = 0;
            if (g < a.G) {
                n = a.T;
                if (a.kv_len) {
                    n = __ldg(a.kv_len + g);
                    n = n < 0 ? 0 : (n < a.T ? n : a.T);
                }
                n = (n + 127) / 128;
            }
            sums[tid] = n;
            __syncthreads();
            for (int o = 1; o < 128; o <<= 1) {
                const int64_t x = tid >= o ? sums[tid - o] : 0;
                __syncthreads();
                sums[tid] += x;
                __syncthreads();
            }
            if (g < a.G) a.off[g + 1] = run + sums[tid];
            run += sums[127];
            __syncthreads();
        }
        if (tid == 0) a.off[0] = 0;
    }
    const int per = a.nb / 32;
    const int64_t pg = blockIdx.x / per;
    const int64_t g = pg / a.rbs;
    const int rb = (int)(pg - g * a.rbs), row0 = (int)(blockIdx.x - pg * per) * 32 + (warp & 1) * 16;
    const int s = blockIdx.y, dsl = a.pw ? 2 : 0;
    // rows row0 + rr and + 8 of the block, elements 32 p .. 32 p + 31
    uint32_t A[2][16];
    float ss[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = rb * a.nb + row0 + rr + 8 * h;
        const bool in = r < a.rows;
        const uint4 *src = in ? reinterpret_cast<const uint4 *>(tr_row(a.q, a.qs, a, g, r) + 32 * p) : nullptr;
        ss[h] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 v = in ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
            A[h][4 * i] = v.x; A[h][4 * i + 1] = v.y; A[h][4 * i + 2] = v.z; A[h][4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = bf16_lo(A[h][i]), y = bf16_hi(A[h][i]);
            ss[h] = __fmaf_rn(x, x, __fmaf_rn(y, y, ss[h]));
        }
        ss[h] += __shfl_xor_sync(0xffffffffu, ss[h], 1);
        ss[h] += __shfl_xor_sync(0xffffffffu, ss[h], 2);
    }
    const float n0 = sqrtf(ss[0]), n1 = sqrtf(ss[1]);
    const float i0 = n0 > 0.0f ? 1.0f / n0 : 0.0f, i1 = n1 > 0.0f ? 1.0f / n1 : 0.0f;
    if (s == 0 && p == 0 && (warp >> 1) == 0) {
        a.wsC[pg * a.nb + row0 + rr] = n0 * a.qscale;
        a.wsC[pg * a.nb + row0 + rr + 8] = n1 * a.qscale;
    }
    uint8_t *img = a.wsQ + pg * (int64_t)a.nb * a.kb * 2 + (int64_t)s * a.nb * 128;
#pragma unroll
    for (int n8 = 0; n8 < 4; ++n8) {
        const int c = (warp >> 1) * 32 + n8 * 8 + rr;            // this lane's operand row: column of the slice
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (s < dsl) {
            const int i = s * 64 + c;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t b[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = 32 * p + 4 * k + 2 * e;        // elements j, j + 1 of row i of H D
                    const uint32_t sw = TK.sign_words[p] >> (j & 31);
                    const uint32_t lo = ((uint32_t)__popc(i & j) ^ sw) & 1u, hi = ((uint32_t)__popc(i & (j + 1)) ^ (sw >> 1)) & 1u;
                    b[e] = 0x3F803F80u | (lo << 15) | (hi << 31);
                }
                const uint32_t af[4] = {A[0][2 * k], A[1][2 * k], A[0][2 * k + 1], A[1][2 * k + 1]};
                tr_mma_bf16(d, af, b[0], b[1]);
            }
        } else {
            const uint4 *src = reinterpret_cast<const uint4 *>(a.proj + (int64_t)((s - dsl) * 64 + c) * kTrD + 32 * p);
            uint32_t B[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = __ldg(src + i);
                B[4 * i] = v.x; B[4 * i + 1] = v.y; B[4 * i + 2] = v.z; B[4 * i + 3] = v.w;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t af[4] = {A[0][2 * k], A[1][2 * k], A[0][2 * k + 1], A[1][2 * k + 1]};
                if (a.proj_bf16) {
                    tr_mma_bf16(d, af, B[2 * k], B[2 * k + 1]);
                } else {
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x, y;
                        unpack2<false>(B[2 * k + e], x, y);
                        hi[e] = pack2<true>(x, y);
                        lo[e] = pack2<true>(x - bf16_lo(hi[e]), y - bf16_hi(hi[e]));
                    }
                    tr_mma_bf16(d, af, hi[0], hi[1]);
                    tr_mma_bf16(d, af, lo[0], lo[1]);
                }
            }
        }
        // d: rows row0 + rr (+ 8), operand rows 2 p, 2 p + 1 of this n8 group
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = row0 + rr + (e >> 1) * 8;
            int col = (warp >> 1) * 32 + n8 * 8 + 2 * p + (e & 1);
            if (s >= dsl) col = tr_sign_column(col);
            *reinterpret_cast<__half *>(img + (r >> 3) * 1024 + (r & 7) * 128 + (((col >> 3) ^ (r & 7)) << 4) + (col & 7) * 2) =
                __float2half_rn(d[e] * ((e >> 1) ? i1 : i0));
        }
    }
}

// ------------------------------------------------------------------ combine

constexpr int kTrCombineRows = 4;

// A CTA of 128 threads (thread = coordinate) joins four rows of a group: their drafted part in fp32 from the 16-bit
// keys and values, then their segments of the cached part (m, l, O), rotated back by H and D.
__global__ void __launch_bounds__(128)
tree_combine_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ QuantTables TV, int grid_main)
{
    extern __shared__ float sS[];                               // [4][n_nodes] scores, then weights
    __shared__ float sm[4], sl[4], buf[4][kTrD];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t g = blockIdx.y;
    const int r0 = blockIdx.x * kTrCombineRows, n = a.nodes;
    const int64_t b = g / a.kv_heads;
    const int kv = (int)(g - b * a.kv_heads);
    const uint64_t *mask = a.mask ? a.mask + b * a.mask_batch : nullptr;
    const int words = (n + 63) / 64;
    auto sees = [&](int r, int j) -> bool {
        if (r >= a.rows) return false;
        const int node = r / a.rep;
        return mask ? (__ldg(mask + (int64_t)node * words + (j >> 6)) >> (j & 63)) & 1u : j <= node;
    };
    // scores (in units of log2)
    {
        float q[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint2 v = make_uint2(0u, 0u);
            if (r0 + i < a.rows) v = __ldg(reinterpret_cast<const uint2 *>(tr_row(a.q, a.qs, a, g, r0 + i)) + lane);
            q[i][0] = bf16_lo(v.x); q[i][1] = bf16_hi(v.x); q[i][2] = bf16_lo(v.y); q[i][3] = bf16_hi(v.y);
        }
        for (int j = warp; j < n; j += 4) {
            bool any = false;
            bool vis[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) { vis[i] = sees(r0 + i, j); any |= vis[i]; }
            float dot[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (any) {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(a.k_new + b * a.ks.batch + (int64_t)j * a.ks.token + (int64_t)kv * a.ks.head) + lane);
                const float k0 = bf16_lo(v.x), k1 = bf16_hi(v.x), k2 = bf16_lo(v.y), k3 = bf16_hi(v.y);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x = __fmaf_rn(q[i][0], k0, __fmaf_rn(q[i][1], k1, __fmaf_rn(q[i][2], k2, q[i][3] * k3)));
                    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                    dot[i] = vis[i] ? x * a.qscale : -INFINITY;
                }
            }
            if (lane < 4) sS[lane * n + j] = lane == 0 ? dot[0] : lane == 1 ? dot[1] : lane == 2 ? dot[2] : dot[3];
        }
    }
    __syncthreads();
    {
        float m = -INFINITY, l = 0.0f;
        for (int j = lane; j < n; j += 32) m = fmaxf(m, sS[warp * n + j]);
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        for (int j = lane; j < n; j += 32) {
            const float s = sS[warp * n + j];
            const float p = s == -INFINITY ? 0.0f : tr_ex2(s - m);       // (a NaN score stays one)
            sS[warp * n + j] = p;
            l += p;
        }
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) { sm[warp] = m; sl[warp] = l; }
    }
    __syncthreads();
    float ot[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint16_t *vcol = a.v_new + b * a.vs.batch + (int64_t)kv * a.vs.head + tid;
    for (int j = 0; j < n; ++j) {
        const float p0 = sS[j], p1 = sS[n + j], p2 = sS[2 * n + j], p3 = sS[3 * n + j];
        if (p0 == 0.0f && p1 == 0.0f && p2 == 0.0f && p3 == 0.0f) continue;
        const float v = __uint_as_float((uint32_t)__ldg(vcol + (int64_t)j * a.vs.token) << 16);
        // a hidden value may be anything: it is not touched
        if (p0 != 0.0f) ot[0] = __fmaf_rn(p0, v, ot[0]);
        if (p1 != 0.0f) ot[1] = __fmaf_rn(p1, v, ot[1]);
        if (p2 != 0.0f) ot[2] = __fmaf_rn(p2, v, ot[2]);
        if (p3 != 0.0f) ot[3] = __fmaf_rn(p3, v, ot[3]);
    }
    // segments of the row block: CTAs whose ranges [total c / grid, total (c + 1) / grid) meet its items
    const int rb = r0 / a.nb;
    const int64_t pg = g * a.rbs + rb;
    float M[4], L[4], acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) { M[i] = sm[i]; L[i] = sl[i]; acc[i] = 0.0f; }
    if (grid_main > 0) {
        const int64_t total = a.off[a.G] * a.rbs, tiles = a.off[g + 1] - a.off[g];
        const int64_t lo = a.off[g] * a.rbs + rb * tiles, hi = lo + tiles;
        if (tiles > 0) {
            int c = (int)((lo * grid_main) / total);
            while (c > 0 && total * c / grid_main > lo) --c;
            while (total * (c + 1) / grid_main <= lo) ++c;
            for (; c < grid_main && total * c / grid_main < hi; ++c) {
                if (total * (c + 1) / grid_main <= total * c / grid_main) continue;     // an empty range
                const float *P = a.part + (size_t)(c + pg) * tr_part_floats(a.nb);
                const int in = r0 - rb * a.nb;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float m = P[(size_t)a.nb * kTrD + in + i], l = P[(size_t)a.nb * kTrD + a.nb + in + i];
                    const float mn = fmaxf(M[i], m);
                    const float wo = M[i] == -INFINITY ? 0.0f : tr_ex2(M[i] - mn), wn = tr_ex2(m - mn);
                    L[i] = __fmaf_rn(L[i], wo, l * wn);
                    ot[i] *= wo;
                    acc[i] = __fmaf_rn(acc[i], wo, P[(size_t)(in + i) * kTrD + tid] * wn);
                    M[i] = mn;
                }
            }
        }
    }
    // H over the 128 coordinates: stages inside the warp, then across the warps
#pragma unroll
    for (int h = 1; h < 32; h <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float o = __shfl_xor_sync(0xffffffffu, acc[i], h);
            acc[i] = (lane & h) ? o - acc[i] : acc[i] + o;
        }
    }
#pragma unroll
    for (int h = 32; h < kTrD; h <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) buf[i][tid] = acc[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float o = buf[i][tid ^ h];
            acc[i] = (tid & h) ? o - acc[i] : acc[i] + o;
        }
        __syncthreads();
    }
    const bool neg = (TV.sign_words[tid >> 5] >> (tid & 31)) & 1u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (r0 + i >= a.rows) break;
        const float x = (neg ? -acc[i] : acc[i]) + ot[i];
        const float y = L[i] == 0.0f ? 0.0f : __fdiv_rn(x, L[i]);
        uint16_t *dst = const_cast<uint16_t *>(tr_row(a.out, a.os, a, g, r0 + i));
        dst[tid] = (uint16_t)(pack2<true>(y, 0.0f) & 0xffffu);
    }
}

}  // namespace rq

// qjl_tree.cuh -- attention of a tree of drafted tokens over the compressed cache (sm_100a).
//
// Query row r = (node i, head h of the key head's rep) of group g = (sequence, key head) attends to the group's
// len cached tokens (QJL / two-stage score s, values vh reconstructed from codes) and to the drafted tokens j that
// its node sees (16-bit k_j, v_j), under one softmax:
//   out = (sum_t e^(c s(r,t)) vh_t + sum_j e^(c <q,k_j>) v_j) / (sum_t e^(c s) + sum_j e^(c <q,k_j>)),   0 where it sees nothing.
// With one node it is the ordinary decode step.
//
// Three kernels:
//   tree_prologue_kernel   the score operand of every row, [H D q ; S q] 2^-e in fp16, written as the image of the
//                          shared-memory operand (so that the main kernel fetches it with one bulk copy); the
//                          prefix sums of the groups' tiles;
//   tree_attention_kernel  the cached part, split evenly over the SMs whatever the lengths: (m, l, O) per segment;
//   tree_combine_kernel    joins a row's segments with its drafted part, rotates back, divides and rounds.
//
// Main kernel, per 128-token tile and block of NB query rows.  Tokens are the M dimension of the score product
// (S^T = K . Q^T, one token a TMEM lane), so that every lane works however few rows there are, and a thread's
// token-wise factors are its own registers:
//   producers (groups of 4 warps)  thread = token: 64 key values a slice are unpacked to fp16 and stored to TMEM, where
//                        the score product reads its A operand: unpacked keys never pass through shared memory.  Then
//                        the token's values, V' = fp16(c 2^-e) n, to shared memory (2^e above the largest centroid, so
//                        that V' fits fp16 whatever the norm; the rest of the factor, 2^e / d, is the join's).
//   MMA 1 (one thread)   S^T[token][row] += K slice (TMEM) . Q^T slice (shared memory).
//   softmax (4 warps for 32 rows)  thread = token: weights 2^((s - Q) g + 8 - ref), fp16, to shared memory.  The reference
//                        `ref` of a row is the maximum of the segment's first tile and moves only when a score passes
//                        it by 7 (2^15 is the most fp16 weights take): the usual tile needs one vote, taken while the
//                        weights are computed, and no reduction over tokens.
//   MMA 2 (one thread)   O^T[d][row] += V'^T . P and the rows' weight sums P^T . 1, in TMEM over the segment.
//
// Measured (B200): 32 rows x 32 groups x 32768 tokens, m = 256, 4-bit values: 104 us whole (105 MB: 16 us at the copy
// rate; 26 GFLOP of score and value products: 16 us); 256 rows: 414 us (206 GFLOP: 125 us).  What bounds it: neither
// memory (DRAM 10 %) nor the tensor pipe (13 and 25 %) nor the issue of instructions (0.46 and 0.40 a scheduler and
// cycle), but exposed latency: the first stall is a load (long_scoreboard: a producer's own token's records from L2, a
// softmax warp's scores from tensor memory), with too few warps to cover it.  Up to 32 rows the single weight and value
// buffer adds to it; at 256 rows the softmax warps are the critical path.
#pragma once
#include "rq_cache_ops.h"
#include "rq_common.cuh"
#include "sm100.cuh"

namespace rq {

constexpr int kTrTok = 128;                       // tokens a tile (M of both products' token side)
constexpr int kTrD = 128;
constexpr int kTrVBytes = kTrTok * kTrD * 2;      // one value tile, fp16
constexpr float kTrShift = 8.0f;                  // weight of the reference: 2^8
constexpr float kTrMost = 15.0f;                  // largest exponent an fp16 weight may have
// The score operand of a row in fp16 is [H D q ; S q] 2^-e / 16, 2^e <= max |q_i| < 2^(e + 1): at most |S_i| sqrt(2), and
// for a pure sketch times 2 .. 2^-7 (tr_bit_factor).  Rows of a chunk of 32 whose e are within kTrSpread share the
// largest: with S of N(0, 1) the coordinates of a row of N(0, 1) values that is 2^-4 of it are still 2^-13 at that
// smallest factor, where half a step of fp16, 2^-25, is as small a part as for a normal value.  In a chunk with a wider
// spread every row has its own e, and the softmax multiplies by it (32 rows x 32 x 32768 tokens: 117 us instead of 111).
constexpr int kTrSpread = 4;
constexpr float kTrRowScale = 16.0f;

constexpr int kTrAhead = 4;                       // tiles that the cache's records are prefetched into L2 ahead

// Warps of a CTA: NB / 32 groups of four softmax warps (a group has 32 rows), groups of four producer warps (with two,
// a group unpacks every second tile), two issuing warps.  Measured (32 groups x 32768 tokens, pure sketch keys): at 32
// rows one producer group in each of two CTAs an SM 111 us, two groups 115 us (spills at 72 registers); at 64 two groups
// 127 us, one 163 us; at 256 one group 420 us, two 435 us.
__host__ __device__ constexpr int tr_softmax_warps(int nb) { return nb / 8; }
__host__ __device__ constexpr int tr_producer_groups(int nb) { return nb == 64 ? 2 : 1; }
__host__ __device__ constexpr int tr_threads(int nb) { return (tr_softmax_warps(nb) + 4 * tr_producer_groups(nb) + 2) * 32; }
__host__ __device__ constexpr int tr_ctas(int nb) { return nb == 32 ? 2 : 1; }
// TMEM: score buffers, O, the weight sums (16 columns), key slots of 32 columns
__host__ __device__ constexpr int tr_sbufs(int nb) { return nb == 128 ? 1 : 2; }
__host__ __device__ constexpr int tr_kslots(int nb) { return nb == 32 ? 4 : nb == 64 ? 8 : 6; }
__host__ __device__ constexpr int tr_tmem(int nb) { return nb == 32 ? 256 : 512; }
// log2 of the copies of the value and key lookup tables: 32 copies have no bank conflicts (values with 8: 117 us, 16: 115,
// 32: 111 at 32 rows; 430, 424, 420 at 256); the keys' have fewer where shared memory is short.
__host__ __device__ constexpr int tr_vcl(int) { return 5; }
__host__ __device__ constexpr int tr_kcl(int nb) { return nb == 64 ? 5 : 3; }
__host__ __device__ inline size_t tr_pbytes(int nb) { return (size_t)(nb > 64 ? 2 : 1) * kTrTok * 128; }
__host__ __device__ inline size_t tr_lut_bytes(int pw, int cl)
{
    return pw == 0 ? 0 : pw <= 4 ? ((size_t)4 << (2 * pw + cl)) : ((size_t)512 << cl);
}
// mbarriers: key slots full and empty, values, scores full and empty, weights (2 each), P V done (4), O, the operand full
// and done, the last products of the two issuing warps, and a vote by group of softmax warps
__host__ __device__ constexpr int tr_barriers(int nb) { return 2 * tr_kslots(nb) + 4 * 2 + 4 + 3 + 2 + tr_softmax_warps(nb) / 4; }
__host__ __device__ inline size_t tr_smem(int nb, int kb, int pw, int vpw, int np, int nv)
{
    return 1024 + (size_t)nb * kb * 2 + nv * kTrVBytes + np * tr_pbytes(nb) + tr_lut_bytes(pw, tr_kcl(nb)) +
           tr_lut_bytes(vpw, tr_vcl(nb)) + 2048 + (size_t)nb * (8 + 4 + 4 + 5 * 4) + 8 * tr_barriers(nb) + 4 + tr_softmax_warps(nb) * 2;
}
// Partial result of one (CTA, row block) segment: O [nb][128], m [nb], l [nb].
__host__ __device__ inline size_t tr_part_floats(int nb) { return (size_t)nb * (kTrD + 2); }

__device__ __forceinline__ float tr_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr)
{
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
    return r;
}

__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r) : "memory");
}

// The three kernels are launched so that each may start while the one before it runs: what does not depend on it comes
// before tr_wait_previous.
__device__ __forceinline__ void tr_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void tr_wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Shared memory by 32-bit address (a lookup in a table that nothing writes any more; and accesses in program order).
__device__ __forceinline__ uint32_t tr_lds(uint32_t addr)
{
    uint32_t r;
    asm("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ uint32_t tr_lds16(uint32_t addr)
{
    uint16_t r;
    asm("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ float4 tr_lds_f4(uint32_t addr)
{
    float4 r;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(addr) : "memory");
    return r;
}
__device__ __forceinline__ void tr_sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Waits between the roles have a limit, and none of them decides what a warp does next: after an expired wait (recorded
// in the device error word) a warp goes through its remaining items like any other, with one poll for each wait.  So the
// lanes of a warp never part, as elect.sync and the instructions for tensor memory need, and every warp comes to the same
// barriers equally often.
__device__ __forceinline__ void tr_wait(uint64_t *bar, uint32_t parity, uint32_t &limit)
{
    if (!mbar_wait_limit(bar, parity, limit)) limit = 1;
}

// A barrier of the four warps of a softmax group.  They take the same way (tr_vote_wait), and no other wait is without
// limit, so all of them come to it.
__device__ __forceinline__ void tr_bar(int id)
{
    asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}

__device__ __forceinline__ void tr_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The wait for the other warps of the group to have voted.  It is never cut short, so that all of them see the same votes:
// between two places where the group meets (a vote, a barrier) a warp has at most four waits, each with the usual limit,
// so this one ends before its own limit of 16 times that.
__device__ __forceinline__ void tr_vote_wait(uint64_t *bar, uint32_t parity)
{
    mbar_wait_limit(bar, parity, 16 * kSpinLimit);
}

// True in one lane of a converged warp.  (Measured: products issued under `lane == 0` cost the issuing thread about 200
// cycles each, since their descriptors are then not warp-uniform to the compiler; under the elected lane they do not.)
__device__ __forceinline__ bool tr_elect()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)::"memory");
    return r != 0;
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

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
        "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
        "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
        "r"(r[31]), "r"(taddr)
        : "memory");
}

// Fetch [p, p + bytes) into L2 (both rounded down to 16 bytes).
__device__ __forceinline__ void tr_prefetch(const void *p, int64_t bytes)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p) & ~15ull;
    const uint32_t n = (uint32_t)((reinterpret_cast<uint64_t>(p) + bytes - a) & ~15ull);
    if (n) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"(n) : "memory");
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

// Reduce v[0 .. 32) over the 32 lanes of a warp: lane l returns the result of column l.
template <typename Op>
__device__ __forceinline__ float tr_reduce_columns(uint32_t *v, int lane, Op op)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const uint32_t send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = __float_as_uint(op(__uint_as_float(keep), __uint_as_float(__shfl_xor_sync(0xffffffffu, send, o))));
        }
    }
    return __uint_as_float(v[0]);
}

__device__ __forceinline__ int64_t tr_len(const TreeArgs &a, int64_t g)
{
    if (!a.kv_len) return a.T;
    const int64_t n = __ldg(a.kv_len + g);
    return n < 0 ? 0 : (n < a.T ? n : a.T);
}

// Position in the list of (group, row block, tile) items: group g's items are [off[g] rbs, off[g + 1] rbs).
struct TreeIter {
    int64_t g, row;                               // row: cache row of the tile's first token
    int rb, tile, n, left;                        // left: the group's tokens from the tile's first on
    __device__ void group(const TreeArgs &a)
    {
        n = (int)(a.off[g + 1] - a.off[g]);
    }
    __device__ void place(const TreeArgs &a)
    {
        row = g * a.T + (int64_t)tile * kTrTok;
        left = (int)(tr_len(a, g) - (int64_t)tile * kTrTok < 0x7fffffff ? tr_len(a, g) - (int64_t)tile * kTrTok : 0x7fffffff);
    }
    __device__ void seek(const TreeArgs &a, int64_t it)
    {
        int64_t lo = 0, hi = a.G;                 // off[lo] rbs <= it < off[hi] rbs
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (a.off[mid] * a.rbs <= it) lo = mid; else hi = mid;
        }
        g = lo;
        group(a);
        const int64_t rest = it - a.off[g] * a.rbs;
        rb = (int)(rest / n);
        tile = (int)(rest - (int64_t)rb * n);
        place(a);
    }
    // advance by one item (the caller knows that there is one); true when the row block changes
    __device__ bool next(const TreeArgs &a)
    {
        if (++tile < n) {
            row += kTrTok;
            left -= kTrTok;
            return false;
        }
        tile = 0;
        if (++rb == a.rbs) {
            rb = 0;
            do {
                ++g;
                group(a);
            } while (n == 0);
        }
        place(a);
        return true;
    }
};

// 32 sign bits to 16 pairs of fp16; pair i is (bit i, bit i + 16) in both forms.  The score product sums over all
// of them, so the query operand has its coordinates in the same order (tr_sign_column).
// +-mag: one shift and one masked or a pair.
__device__ __forceinline__ void tr_signs(uint32_t w, uint32_t mag2, uint32_t *o)
{
    const uint32_t n = ~w;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = mag2 | ((n << (15 - i)) & 0x80008000u);
}
// The bits where they lie: a set bit p (5 .. 12) of an fp16 value alone is the number c_p = 2^-19 ... 2^-11 (up to
// p = 9 a subnormal one), so a pair costs one mask, and sign = 2 bit - 1 with c_p taken into the query operand:
// sum_i sign_i q_i = 2^19 sum_i (bit_i c_p) (2^-18 q_i / c_p) - sum_i q_i.
__device__ __forceinline__ void tr_bits(uint32_t w, uint32_t *o)
{
    const uint32_t lo = w << 5, hi = w >> 3;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        o[i] = lo & (0x00200020u << i);
        o[8 + i] = hi & (0x00200020u << i);
    }
}
constexpr float kTrBitScale = 0x1p19f;
// 2^-18 / c_p of sketch coordinate i
__host__ __device__ inline float tr_bit_factor(int i)
{
    const int p = 5 + (i & 7);                    // c_p = 2^(p - 24) below 10, then 2^-14, 2^-13, 2^-11
    return p < 10 ? (float)(1 << (10 - p)) * 0.0625f : p == 10 ? 0.0625f : p == 11 ? 0.03125f : 0.0078125f;
}
// Column, in its 64-column slice, of sketch coordinate i (0 .. 63).
__host__ __device__ inline int tr_sign_column(int i) { return (i & 32) | ((i & 15) << 1) | ((i >> 4) & 1); }

// Pairs [FROM, FROM + N) of 64 codes of PW bits to fp16 centroids: the pair's 2 PW bits index a table of pairs in 2^CL
// copies.
template <int PW, int CL, int FROM, int N>
__device__ __forceinline__ void tr_lookup(const uint32_t *kc, uint32_t lut, uint32_t lane4, uint32_t *out)
{
    uint32_t *o = out - FROM;
#pragma unroll
    for (int i = FROM; i < FROM + N; ++i) {
        if constexpr (PW <= 4) {
            constexpr int B = 2 * PW;
            constexpr uint32_t mask = ((1u << B) - 1u) << (CL + 2);
            const int bit = i * B, w = bit >> 5, sh = (bit & 31) - (CL + 2);
            uint32_t x;
            if ((bit & 31) + B > 32) x = __funnelshift_r(kc[w], kc[w + 1 < 16 ? w + 1 : w], bit & 31) << (CL + 2);
            else x = sh >= 0 ? kc[w] >> (sh >= 0 ? sh : 0) : kc[w] << (sh < 0 ? -sh : 0);
            o[i] = tr_lds(lut + ((x & mask) | lane4));
        } else {
            const uint32_t l16 = lut + (lane4 >> 1);
            const uint32_t ca = unpack_code<64, PW>(kc, 2 * i), cb = unpack_code<64, PW>(kc, 2 * i + 1);
            o[i] = tr_lds16(l16 + (ca << (CL + 1))) | (tr_lds16(l16 + (cb << (CL + 1))) << 16);
        }
    }
}

template <int CL, int FROM, int N>
__device__ __forceinline__ void tr_lookup_any(int pw, const uint32_t *kc, uint32_t lut, uint32_t lane4, uint32_t *o)
{
    switch (pw) {
    case 1: tr_lookup<1, CL, FROM, N>(kc, lut, lane4, o); break;
    case 2: tr_lookup<2, CL, FROM, N>(kc, lut, lane4, o); break;
    case 3: tr_lookup<3, CL, FROM, N>(kc, lut, lane4, o); break;
    case 4: tr_lookup<4, CL, FROM, N>(kc, lut, lane4, o); break;
    default: tr_lookup<8, CL, FROM, N>(kc, lut, lane4, o); break;
    }
}

// Words [2 from, 2 to) of the 8 pw bytes (64 codes) at p, 8-byte aligned.
template <int FROM, int TO>
__device__ __forceinline__ void tr_load_codes(const uint8_t *p, int pw, bool valid, uint32_t *w)
{
#pragma unroll
    for (int q = FROM; q < TO; ++q) {
        uint2 v = make_uint2(0u, 0u);
        if (q < pw && valid) v = __ldg(reinterpret_cast<const uint2 *>(p) + q);
        w[2 * q] = v.x;
        w[2 * q + 1] = v.y;
    }
}

// V4: values of 4 bits (fewer and wider loads, no choice of width in the loop: 127 -> 111 us at 32 rows x 32 x 32768
// tokens, 143 -> 127 us at 64, 428 -> 420 us at 256).
template <int NB, bool TWO, bool V4>
__global__ void __launch_bounds__(tr_threads(NB), tr_ctas(NB))
tree_attention_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ QuantTables TK,
                      const __grid_constant__ QuantTables TV, int np, int nv)
{
    constexpr int SW = tr_softmax_warps(NB), NG = SW / 4, NPG = tr_producer_groups(NB), PW = 4 * NPG;
    constexpr int VCL = tr_vcl(NB), KCL = tr_kcl(NB), threads = tr_threads(NB), KS = tr_kslots(NB), NS = tr_sbufs(NB);
    // Every producer group has its own key slots: it may be tiles ahead of the products, but then never more than one
    // phase ahead of a slot's barrier, which is what a parity can tell.
    constexpr int SPG = KS / NPG;
    const int kb = a.kb, nsl = kb / 64, dsl = TWO ? 2 : 0;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = base;
    uint8_t *sV = sQ + (size_t)NB * kb * 2;
    uint8_t *sP = sV + (size_t)nv * kTrVBytes;
    uint8_t *ones = sP + np * tr_pbytes(NB);      // 2 KB of fp16 ones: the sums' second operand
    uint8_t *klut = ones + 2048;
    uint8_t *vlut = klut + tr_lut_bytes(a.pw, KCL);
    // per pair of rows: the operand's sums (-Q, -Q, pure sketch keys only), 8 - ref, 8 - ref
    float4 *sF = reinterpret_cast<float4 *>(vlut + tr_lut_bytes(a.vpw, VCL));
    float *sAl = reinterpret_cast<float *>(sF + NB / 2);                         // [NB] rescale factors
    float *sX = sAl + NB;                         // [4][NB] column reductions by lane quarter, [NB] moves of the exponents
    float *sR = sX + 5 * NB;                      // [NB] factors of the rows, for chunks in which they differ
    uint64_t *k_full = reinterpret_cast<uint64_t *>(sR + NB);
    uint64_t *k_empty = k_full + KS;
    uint64_t *v_full = k_empty + KS;              // [2]
    uint64_t *s_full = v_full + 2;                // [2]
    uint64_t *s_empty = s_full + 2;               // [2]
    uint64_t *p_full = s_empty + 2;               // [2]
    uint64_t *pv_done = p_full + 2;               // [4] by tile modulo 4: P, V free, O holds the tile
    uint64_t *o_empty = pv_done + 4;
    uint64_t *q_full = o_empty + 1;
    uint64_t *q_done = q_full + 1;
    uint64_t *drained = q_done + 1;               // [2] by issuing warp: all its products are done
    uint64_t *vote = drained + 2;                 // by softmax group
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(vote + NG);
    volatile uint32_t *flag = tmem_slot + 1;      // [NG][2] by softmax group and use parity

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t quarter = (uint32_t)(warp & 3);
    tr_launch_next();
    // lookup tables: one entry a thread, its copies by 16-byte stores whose order differs from lane to lane
    auto fill = [&](const QuantTables &T, uint8_t *dst, int pw, int cl, float by) {
        if (pw == 0) return;
        const int entries = pw <= 4 ? 1 << (2 * pw) : 256, bytes = (pw <= 4 ? 4 : 2) << cl, chunks = bytes / 16;
        for (int e = tid; e < entries; e += threads) {
            const int ca = pw <= 4 ? e & ((1 << pw) - 1) : e, cb = pw <= 4 ? e >> pw : e;
            const float fa = ca < T.levels ? T.centroid[ca] * by : 0.0f, fb = cb < T.levels ? T.centroid[cb] * by : 0.0f;
            const uint32_t v = (uint32_t)__half_as_ushort(__float2half_rn(fa)) |
                               ((uint32_t)__half_as_ushort(__float2half_rn(fb)) << 16);
            for (int i = 0; i < chunks; ++i)
                tr_sts128(smem_u32(dst) + (uint32_t)(e * bytes) + (uint32_t)(((i + tid) & (chunks - 1)) * 16), v, v, v, v);
        }
    };
    if (TWO) fill(TK, klut, a.pw, KCL, 1.0f);
    fill(TV, vlut, a.vpw, VCL, a.vdown);
    for (int i = tid; i < 512; i += threads) reinterpret_cast<uint32_t *>(ones)[i] = 0x3C003C00u;
    fence_proxy_async_smem();
    if (tid == 0) {
        for (int b = 0; b < 2 * NG; ++b) flag[b] = 0u;
        for (int b = 0; b < NG; ++b) mbar_init(&vote[b], 4);
        for (int b = 0; b < KS; ++b) { mbar_init(&k_full[b], 4); mbar_init(&k_empty[b], 1); }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&v_full[b], 4);
            mbar_init(&s_full[b], 1); mbar_init(&s_empty[b], SW);
            mbar_init(&p_full[b], SW);
        }
        for (int b = 0; b < 4; ++b) mbar_init(&pv_done[b], 1);
        mbar_init(o_empty, SW);
        mbar_init(q_full, 1);
        mbar_init(q_done, 1);
        for (int b = 0; b < 2; ++b) mbar_init(&drained[b], 1);
        fence_barrier_init();
    }
    if (warp == SW + PW) tmem_alloc(tmem_slot, tr_tmem(NB));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem, tO = tmem + NS * NB, tL = tO + NB, tK = tL + 16;

    tr_wait_previous();
    // the items are split over as many CTAs as have one
    const int64_t total = a.off[a.G] * a.rbs, ctas = total < gridDim.x ? total : gridDim.x;
    const int64_t it0 = blockIdx.x < ctas ? total * blockIdx.x / ctas : 0;
    const int count = blockIdx.x < ctas ? (int)(total * (blockIdx.x + 1) / ctas - it0) : 0;
    uint32_t limit = kSpinLimit;
    auto pv_wait = [&](int tile) { tr_wait(&pv_done[tile & 3], (uint32_t)((tile >> 2) & 1), limit); };
    TreeIter it;
    if (count > 0) it.seek(a, it0);

    if (count > 0 && warp >= SW && warp < SW + PW) {
        // ------------------------------------------------------------ producers
        const int group = (warp - SW) >> 2;
        const int r = (int)quarter * 32 + lane;                 // token of the tile
        const uint32_t sbytes = (uint32_t)a.m / 8, cbytes = 16u * a.pw, vbytes = 16u * a.vpw;
        const float kq = 1.2533141373155002512f / (float)a.m;
        const uint32_t lane4k = 4u * ((uint32_t)lane & ((1u << KCL) - 1u)), lane4v = 4u * ((uint32_t)lane & ((1u << VCL) - 1u));
        const uint32_t klut0 = smem_u32(klut), vlut0 = smem_u32(vlut), sV0 = smem_u32(sV);
        const int nsig = nsl - dsl;
        uint2 sg[4];                                            // four sign slices, loaded a tile ahead
        uint16_t hn = 0, hr = 0;                                // first-stage and sketch norm
        auto load_signs = [&](const TreeIter &p, int first) {
            const uint2 *src = reinterpret_cast<const uint2 *>(a.signs + (p.row + r) * sbytes) + first;
            const bool valid = r < p.left;
            if (a.m % 128 == 0) {                               // rows of whole 16 bytes
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (first + i < nsig && valid) x = __ldg(reinterpret_cast<const uint4 *>(src + i));
                    sg[i] = make_uint2(x.x, x.y);
                    sg[i + 1] = make_uint2(x.z, x.w);
                }
                return;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sg[i] = make_uint2(0u, 0u);
                if (first + i < nsig && valid) sg[i] = __ldg(src + i);
            }
        };
        auto load_norms = [&](const TreeIter &p) {
            if (TWO) {
                hn = r < p.left ? __ldg(a.norms + p.row + r) : (uint16_t)0;
                hr = r < p.left ? __ldg(a.sk_norms + p.row + r) : (uint16_t)0;
            }
        };
        // this group's next tile, `c` counting the CTA's tiles
        auto advance = [&](TreeIter &p, int c) {
#pragma unroll 1
            for (int i = 0; i < NPG && c + i + 1 < count; ++i) p.next(a);
        };
        for (int i = 0; i < group && i + 1 < count; ++i) it.next(a);
        if (group < count) {
            load_signs(it, 0);
            load_norms(it);
        }
        for (int c = group; c < count; c += NPG) {
            uint32_t rho2 = 0x3C003C00u;
            if (TWO) {
                // the sketch term scaled to share the first stage's accumulator and factor n / d
                const float n1 = h16_to_f32(hn);
                float rho = 0.0f;
                if (n1 > 0.0f) rho = __fdiv_rn(__fmul_rn(__fmul_rn(kq, h16_to_f32(hr)), (float)kTrD), n1);
                const uint32_t h = (uint32_t)__half_as_ushort(__float2half_rn(rho));
                rho2 = h | (h << 16);
            }
            const bool valid = r < it.left;
            const int64_t row = it.row + r;
#pragma unroll 1
            for (int s = 0; s < nsl; ++s) {                     // a code slice (the first two), or sign slice s - dsl
                const uint32_t n = (uint32_t)(c / NPG * nsl + s);       // slices of this group before
                const int slot = group * SPG + (int)(n % SPG);
                uint32_t o[32];
                if (TWO && s < 2) {
                    uint32_t kc[16];
                    tr_load_codes<0, 8>(a.codes + row * cbytes + s * 8 * a.pw, a.pw, valid, kc);
                    tr_lookup_any<KCL, 0, 32>(a.pw, kc, klut0, lane4k, o);
                } else {
                    if (TWO) {
                        tr_signs(sg[0].x, rho2, o);
                        tr_signs(sg[0].y, rho2, o + 16);
                    } else {
                        tr_bits(sg[0].x, o);
                        tr_bits(sg[0].y, o + 16);
                    }
                    sg[0] = sg[1];
                    sg[1] = sg[2];
                    sg[2] = sg[3];
                    if (s - dsl == 3 && nsig > 4) load_signs(it, 4);
                }
                if (n >= SPG) tr_wait(&k_empty[slot], (n / SPG - 1) & 1, limit);
                tc_fence_after();
                tmem_st32(tK + (uint32_t)slot * 32u + (quarter << 21), o);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) tr_arrive(&k_full[slot]);
            }
            uint32_t vc[16];
            const uint16_t hv = valid ? __ldg(a.vnorms + row) : (uint16_t)0;
            auto load_values = [&](int half) {
                if constexpr (V4) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.vcodes + row * 64) + 2 * half;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 x = valid ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
                        vc[4 * i] = x.x; vc[4 * i + 1] = x.y; vc[4 * i + 2] = x.z; vc[4 * i + 3] = x.w;
                    }
                } else {
                    tr_load_codes<0, 4>(a.vcodes + row * vbytes + half * 8 * a.vpw, a.vpw, valid, vc);
                }
            };
            load_values(0);
            advance(it, c);
            if (c + NPG < count) {
                load_signs(it, 0);
                load_norms(it);
            }
            // the value row: rows of tokens, two 64-wide atoms of d
            const __half2 f2 = __half2half2(__ushort_as_half(hv));
            const int vb = nv == 2 ? c & 1 : 0;
            uint32_t Vr = sV0 + (uint32_t)vb * kTrVBytes + (uint32_t)r * 128u;
#pragma unroll 1
            for (int half = 0; half < 2; ++half, Vr += kTrVBytes / 2) {
                if (!V4 && a.vpw > 4) tr_load_codes<4, 8>(a.vcodes + row * vbytes + half * 8 * a.vpw, a.vpw, valid, vc);
                if (half == 0 && c >= nv) pv_wait(c - nv);      // the tile whose values lie here.  With a
                // barrier for every fourth tile the phase before this one has been waited for (at this group's last
                // tile) and the next one needs this tile's values, so the parity tells.
                auto store = [&](int ch0, const uint32_t *o) {
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __half2 hv2 = __hmul2(*reinterpret_cast<const __half2 *>(&o[4 * ch + e]), f2);
                            w[e] = *reinterpret_cast<const uint32_t *>(&hv2);
                        }
                        tr_sts128(Vr + (uint32_t)(((ch0 + ch) ^ (r & 7)) << 4), w[0], w[1], w[2], w[3]);
                    }
                };
                uint32_t o[16];
                if constexpr (V4) tr_lookup<4, VCL, 0, 16>(vc, vlut0, lane4v, o);
                else tr_lookup_any<VCL, 0, 16>(a.vpw, vc, vlut0, lane4v, o);
                store(0, o);
                if constexpr (V4) tr_lookup<4, VCL, 16, 16>(vc, vlut0, lane4v, o);
                else tr_lookup_any<VCL, 16, 16>(a.vpw, vc, vlut0, lane4v, o);
                if (half == 0) load_values(1);
                store(4, o);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tr_arrive(&v_full[c & 1]);
        }
    } else if (count > 0 && warp == SW + PW) {
        // ------------------------------------------------------------ MMA 1: S^T = K . Q^T
        const uint32_t sQ0 = smem_u32(sQ);
        const uint32_t idesc = idesc_f16(false, kTrTok, NB);
        const uint32_t qbytes = (uint32_t)NB * kb * 2;
        bool fresh = true;
        int seg = 0, loads = 0;
        for (int c = 0; c < count; ++c) {
            if (fresh) {
                if (seg > 0) {
                    if (tr_elect()) mma_commit(q_done);
                    tr_wait(q_done, (uint32_t)((seg - 1) & 1), limit);
                }
                loads += limit > 1;                             // (lane 0's)
                if (lane == 0 && limit > 1) {
                    mbar_arrive_expect_tx(q_full, qbytes);
                    bulk_load(sQ, a.wsQ + (it.g * a.rbs + it.rb) * (int64_t)qbytes, qbytes, q_full);
                }
                tr_wait(q_full, (uint32_t)(seg & 1), limit);
                ++seg;
            }
            const int before = c - NS;                          // the tile whose scores lie in the buffer
            if (before >= 0) tr_wait(&s_empty[before & 1], (uint32_t)((before >> 1) & 1), limit);
            tc_fence_after();
            for (int s = 0; s < nsl; ++s) {
                const uint32_t n = (uint32_t)(c / NPG * nsl + s);
                const int slot = c % NPG * SPG + (int)(n % SPG);
                tr_wait(&k_full[slot], (n / SPG) & 1, limit);
                tc_fence_after();
                if (tr_elect()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f16_ta(tS + (uint32_t)(c % NS) * NB, tK + (uint32_t)slot * 32u + kk * 8u,
                                   sdesc_k_sw128(sQ0 + (uint32_t)s * (NB * 128u) + kk * 32u), idesc,
                                   (s > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(&k_empty[slot]);
                    if (s == nsl - 1) mma_commit(&s_full[c & 1]);
                }
                __syncwarp();
            }
            if (c + 1 < count) fresh = it.next(a);
        }
        // all copies and products done before shared memory and TMEM are freed, also after an expired wait
        loads = __shfl_sync(0xffffffffu, loads, 0);
        if (loads > 0) mbar_wait(q_full, (uint32_t)((loads - 1) & 1));
        if (tr_elect()) mma_commit(&drained[0]);
        mbar_wait(&drained[0], 0);
    } else if (count > 0 && warp == SW + PW + 1) {
        // ------------------------------------------------------------ MMA 2: O^T += V'^T . P; L2 prefetch
        const uint32_t sP0 = smem_u32(sP), sV0 = smem_u32(sV), ones0 = smem_u32(ones);
        const uint32_t idesc = idesc_f16(false, kTrD, NB) | (1u << 15) | (1u << 16);    // both operands MN-major
        bool fresh = true;
        int seg = 0;
        TreeIter pf = it;
        int npf = 0;
        auto fetch = [&]() {                                    // one tile of records
            const int64_t n = pf.left < kTrTok ? pf.left : kTrTok;
            if (lane == 0) {
                tr_prefetch(a.signs + pf.row * (a.m / 8), n * (a.m / 8));
                tr_prefetch(a.vcodes + pf.row * (16 * a.vpw), n * (16 * a.vpw));
                tr_prefetch(a.sk_norms + pf.row, n * 2);
                tr_prefetch(a.vnorms + pf.row, n * 2);
                if (TWO) {
                    tr_prefetch(a.codes + pf.row * (16 * a.pw), n * (16 * a.pw));
                    tr_prefetch(a.norms + pf.row, n * 2);
                }
            }
            if (++npf < count) pf.next(a);
        };
        while (npf < count && npf < kTrAhead) fetch();
        for (int c = 0; c < count; ++c) {
            if (npf < count) fetch();
            const int b = c & 1, pb = np == 2 ? b : 0;
            if (fresh && seg++ > 0) tr_wait(o_empty, (uint32_t)((seg - 2) & 1), limit);
            tr_wait(&v_full[b], (uint32_t)((c >> 1) & 1), limit);
            tr_wait(&p_full[b], (uint32_t)((c >> 1) & 1), limit);
            tc_fence_after();
            if (tr_elect()) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_f16(tO, tr_sdesc(sV0 + (uint32_t)(nv == 2 ? b : 0) * kTrVBytes + kk * 2048u, kTrVBytes / 2, 1024u),
                            tr_sdesc(sP0 + (uint32_t)pb * (uint32_t)tr_pbytes(NB) + kk * 2048u, kTrTok * 128u, 1024u), idesc,
                            (fresh && kk == 0) ? 0u : 1u);
                // sums of the weights over the tokens, [row][16 equal columns]: P^T times ones.  (Up to 64 rows the
                // second half of the operand's 128 rows is whatever lies 8 tokens further: rows that nobody reads.)
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_f16(tL, tr_sdesc(sP0 + (uint32_t)pb * (uint32_t)tr_pbytes(NB) + kk * 2048u, NB == 128 ? kTrTok * 128u : 1024u, 1024u),
                            sdesc_k_sw128(ones0), idesc_f16(false, 128, 16) | (1u << 15), (fresh && kk == 0) ? 0u : 1u);
                mma_commit(&pv_done[c & 3]);
            }
            __syncwarp();
            fresh = c + 1 < count && it.next(a);
        }
        if (tr_elect()) mma_commit(&drained[1]);
        mbar_wait(&drained[1], 0);
    } else if (count > 0 && warp < SW) {
        // ------------------------------------------------------------ softmax
        const int wg = warp >> 2, cb = wg * 32, wt = tid & 127, bar = 1 + wg;     // rows cb .. cb + 31
        const int r = (int)quarter * 32 + lane;                 // token of the tile
        const uint32_t lanes = quarter << 21, sP0 = smem_u32(sP), sF0 = smem_u32(sF) + (uint32_t)cb * 8u, sR0 = smem_u32(sR + cb);
        const uint16_t *gsrc = TWO ? a.norms : a.sk_norms;
        const float gk = kTrRowScale * (TWO ? 1.0f / (float)kTrD : 1.2533141373155002512f / (float)a.m * kTrBitScale);
        uint16_t gn = r < it.left ? __ldg(gsrc + it.row + r) : (uint16_t)0;
        float ref = -INFINITY;                                  // reference of row cb + wt (wt < 32)
        float cq = 0.0f;                                        // the chunk's factor; -1: its rows have their own
        bool fresh = true;
        uint32_t use = 0;                                       // votes so far
        for (int c = 0; c < count; ++c) {
            const bool start = fresh;
            if (start) {
                const float fr = a.wsC[(it.g * a.rbs + it.rb) * NB + cb + lane];
                cq = __shfl_sync(0xffffffffu, fr, 0);
                if (!__all_sync(0xffffffffu, fr == cq)) cq = -1.0f;
                if (wt < 32) {
                    const int row = cb + wt;
                    sR[row] = fr;
                    float sum = 0.0f;
                    if (!TWO) {
                        const float *wc = a.wsC + ((int64_t)a.G * a.rbs + it.g * a.rbs + it.rb) * NB + row;
                        for (int i = 0; i < 2 * nsl; ++i) sum += wc[(int64_t)i * a.G * a.rbs * NB];
                    }
                    float *f = reinterpret_cast<float *>(sF + (row >> 1)) + (row & 1);
                    f[0] = sum * (-1.0f / kTrBitScale) * (cq < 0.0f ? fr : 1.0f);
                    f[2] = 0.0f;
                }
                ref = -INFINITY;
                tr_bar(bar);
            }
            const bool valid = r < it.left;
            const float gg = __fmul_rn(__fmul_rn(h16_to_f32(gn), gk), fabsf(cq));
            const uint32_t vm = valid ? 0xffffffffu : 0u;
            const int64_t pg = it.g * a.rbs + it.rb;
            fresh = false;
            if (c + 1 < count) {
                fresh = it.next(a);
                gn = r < it.left ? __ldg(gsrc + it.row + r) : (uint16_t)0;
            }
            tr_wait(&s_full[c & 1], (uint32_t)((c >> 1) & 1), limit);
            tc_fence_after();
            uint32_t sr[32], w[16];                             // scores, then exponents; fp16 weights of row pairs
            // Exponents (s - Q) gg + (8 - ref) (at the start of a segment: before any reference) and their maximum.  The
            // scores stay in TMEM until the vote is known: held in registers for the unusual answer they spill (256 rows:
            // 12 % slower).
            auto exponents = [&]() {
                tmem_ld32(tS + (uint32_t)(c % NS * NB + cb) + lanes, sr);
                tmem_ld_wait();
                if (cq < 0.0f) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 x = tr_lds_f4(sR0 + (uint32_t)j * 4u);
                        const float2 lo = __fmul2_rn(make_float2(__uint_as_float(sr[j]), __uint_as_float(sr[j + 1])), make_float2(x.x, x.y));
                        const float2 hi = __fmul2_rn(make_float2(__uint_as_float(sr[j + 2]), __uint_as_float(sr[j + 3])), make_float2(x.z, x.w));
                        sr[j] = __float_as_uint(lo.x); sr[j + 1] = __float_as_uint(lo.y);
                        sr[j + 2] = __float_as_uint(hi.x); sr[j + 3] = __float_as_uint(hi.y);
                    }
                }
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float4 f = tr_lds_f4(sF0 + (uint32_t)j * 8u);
                    const float2 off = TWO ? make_float2(f.z, f.w)
                                           : __ffma2_rn(make_float2(f.x, f.y), make_float2(gg, gg), make_float2(f.z, f.w));
                    const float2 v = __ffma2_rn(make_float2(__uint_as_float(sr[j]), __uint_as_float(sr[j + 1])),
                                                make_float2(gg, gg), off);
                    sr[j] = __float_as_uint(v.x);
                    sr[j + 1] = __float_as_uint(v.y);
                    mx = fmaxf(fmaxf(mx, v.x), v.y);
                }
                return mx;
            };
            const float mx = exponents();
            auto weights = [&]() {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const __half2 h = __floats2half2_rn(tr_ex2(__uint_as_float(sr[2 * j])), tr_ex2(__uint_as_float(sr[2 * j + 1])));
                    w[j] = *reinterpret_cast<const uint32_t *>(&h) & vm;
                }
            };
            bool slow = start;
            if (!start) {
                // The group's vote, taken while the weights are computed for the usual answer.  (A flag belongs to
                // one use: written with its number, in two places in turn.)
                ++use;
                if (valid && mx > kTrMost) flag[2 * wg + (use & 1)] = use;
                __syncwarp();
                if (lane == 0) tr_arrive(&vote[wg]);
                weights();
                tr_vote_wait(&vote[wg], (use - 1) & 1);
                slow = __any_sync(0xffffffffu, flag[2 * wg + (use & 1)] == use);
            }
            if (slow) {
                // new references: the maxima over the tile's tokens
                uint32_t t[32];
                exponents();
#pragma unroll
                for (int j = 0; j < 32; ++j) t[j] = valid ? sr[j] : 0xff800000u;
                sX[quarter * NB + cb + lane] = tr_reduce_columns(t, lane, [](float p, float q) { return fmaxf(p, q); });
                tr_bar(bar);
                if (wt < 32) {
                    const float *x = sX + cb + wt;
                    float *off = reinterpret_cast<float *>(sF + ((cb + wt) >> 1)) + 2 + (wt & 1);
                    const float old = *off;                     // 8 - ref, 0 at the start
                    const float mn = fmaxf(ref, fmaxf(fmaxf(x[0], x[NB]), fmaxf(x[2 * NB], x[3 * NB])) - old);
                    sAl[cb + wt] = ref == -INFINITY ? 0.0f : tr_ex2(ref - mn);
                    sX[4 * NB + cb + wt] = (kTrShift - mn) - old;               // what the exponents move by
                    *off = kTrShift - mn;
                    ref = mn;
                }
                tr_bar(bar);
#pragma unroll
                for (int j = 0; j < 32; ++j) sr[j] = __float_as_uint(__uint_as_float(sr[j]) + sX[4 * NB + cb + j]);
                weights();
                if (!start) {                                   // O and the sums of the segment's earlier tiles
                    pv_wait(c - 1);
                    tc_fence_after();
                    const uint32_t at = tO + (uint32_t)cb + lanes;
                    tmem_ld32(at, t);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) t[j] = __float_as_uint(__fmul_rn(__uint_as_float(t[j]), sAl[cb + j]));
                    tmem_st32(at, t);
                    if (quarter == (uint32_t)(wg & 3)) {        // rows are the sums' lanes
                        const uint32_t x = tmem_ld1(tL + lanes);
                        tmem_ld_wait();
                        tmem_st1(tL + lanes, __float_as_uint(__fmul_rn(__uint_as_float(x), sAl[cb + lane])));
                    }
                    tmem_st_wait();
                    tc_fence_before();
                }
            }
            tc_fence_before();                                  // the scores are read
            __syncwarp();
            if (lane == 0) tr_arrive(&s_empty[c & 1]);
            if (c >= np) pv_wait(c - np);  // the tile whose weights lie in the buffer
            // row r of the [token][row] operand
            const uint32_t Pr = sP0 + (np == 2 ? (uint32_t)(c & 1) * (uint32_t)tr_pbytes(NB) : 0u) +
                                (uint32_t)(cb >> 6) * (kTrTok * 128u) + (uint32_t)r * 128u;
            const int ch0 = (cb & 63) >> 3;                     // 16-byte chunk of this group's first row
#pragma unroll
            for (int k = 0; k < 4; ++k)
                tr_sts128(Pr + (uint32_t)(((ch0 + k) ^ (r & 7)) << 4), w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tr_arrive(&p_full[c & 1]);
            if (fresh || c + 1 == count) {                      // end of the segment
                pv_wait(c);
                tc_fence_after();
                float *part = a.part + (size_t)(blockIdx.x + pg) * tr_part_floats(NB);
                tmem_ld32(tO + (uint32_t)cb + lanes, sr);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) part[(size_t)(cb + j) * kTrD + r] = __uint_as_float(sr[j]);
                if (quarter == (uint32_t)(wg & 3)) {
                    const uint32_t x = tmem_ld1(tL + lanes);
                    tmem_ld_wait();
                    part[(size_t)NB * kTrD + NB + cb + lane] = __uint_as_float(x);
                }
                if (wt < 32) part[(size_t)NB * kTrD + cb + wt] = ref - kTrShift;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) tr_arrive(o_empty);
                tr_bar(bar);                                    // the next segment rewrites the rows' constants
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == SW + PW) tmem_dealloc(tmem, tr_tmem(NB));
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
//   [q H D ; q S^T] 2^-e / 16
// as bf16 products with fp32 sums: the entries of H D are +-1, an fp16 projection is the sum of two bf16 numbers, so
// every product is exact.  A thread's 128-value rows are loaded as 64 contiguous bytes a lane of the quad; the sum
// over k runs in that order for both operands.  CTA (0, 0) also writes the prefix sums of the groups' tiles.
__global__ void __launch_bounds__(128)
tree_prologue_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ QuantTables TK)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, p = lane & 3, rr = lane >> 2;
    tr_launch_next();
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
    uint32_t top[2];                                            // bits of the row's largest |element|
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = rb * a.nb + row0 + rr + 8 * h;
        const bool in = r < a.rows;
        const uint4 *src = in ? reinterpret_cast<const uint4 *>(tr_row(a.q, a.qs, a, g, r) + 32 * p) : nullptr;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 v = in ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
            A[h][4 * i] = v.x; A[h][4 * i + 1] = v.y; A[h][4 * i + 2] = v.z; A[h][4 * i + 3] = v.w;
        }
        uint32_t mx = 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = __vmaxu2(mx, A[h][i] & 0x7fff7fffu);
        mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        top[h] = max(mx & 0xffffu, mx >> 16);
    }
    // exponents (biased by 127) of the chunk's rows; 0: a row of zeros, or one that is not finite, which comes out NaN by
    // itself whatever its factor
    __shared__ int exps[32];
    if (p == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            exps[(warp & 1) * 16 + rr + 8 * h] = top[h] == 0u || top[h] >= 0x7f80u ? 0 : min(max((int)(top[h] >> 7), 1), 253);
    }
    __syncthreads();
    const int ex = exps[lane];
    const int most = __reduce_max_sync(0xffffffffu, ex), least = __reduce_min_sync(0xffffffffu, ex > 0 ? ex : 255);
    const bool wide = most - least > kTrSpread;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = (warp & 1) * 16 + rr + 8 * h;
        const int own = wide ? exps[row] : most, e = own > 0 ? own : 127;
        // exact, but for elements 2^-126 of the largest
        const uint32_t down = (uint32_t)(254 - e) << 7, down2 = down | (down << 16);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&A[h][i]), *reinterpret_cast<const __nv_bfloat162 *>(&down2));
            A[h][i] = *reinterpret_cast<const uint32_t *>(&x);
        }
        if (s == 0 && warp < 2 && p == 0)
            a.wsC[pg * a.nb + row0 + rr + 8 * h] = __uint_as_float((uint32_t)e << 23) * a.qscale;
    }
    uint32_t Bs[4][16];                                         // four operand rows, loaded at once
    if (s >= dsl) {
#pragma unroll
        for (int n8 = 0; n8 < 4; ++n8) {
            const int c = (warp >> 1) * 32 + n8 * 8 + rr;
            const uint4 *src = reinterpret_cast<const uint4 *>(a.proj + (int64_t)((s - dsl) * 64 + c) * kTrD + 32 * p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = __ldg(src + i);
                Bs[n8][4 * i] = v.x; Bs[n8][4 * i + 1] = v.y; Bs[n8][4 * i + 2] = v.z; Bs[n8][4 * i + 3] = v.w;
            }
        }
    }
    float part[2] = {0.0f, 0.0f};
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
            const uint32_t *B = Bs[n8];
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
            float x = d[e] * (1.0f / kTrRowScale);
            const float f = tr_bit_factor(col);
            if (!a.pw) x *= f;                                   // by a power of two
            const __half h = __float2half_rn(x);
            if (!a.pw) part[e >> 1] += __half2float(h) / f;
            if (s >= dsl) col = tr_sign_column(col);
            *reinterpret_cast<__half *>(img + (r >> 3) * 1024 + (r & 7) * 128 + (((col >> 3) ^ (r & 7)) << 4) + (col & 7) * 2) = h;
        }
    }
    if (!a.pw) {                                                 // sums of the rounded coordinates of each row, by 32
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            part[h] += __shfl_xor_sync(0xffffffffu, part[h], 1);
            part[h] += __shfl_xor_sync(0xffffffffu, part[h], 2);
            if (p == 0)
                a.wsC[((int64_t)(1 + 2 * s + (warp >> 1)) * a.G * a.rbs + pg) * a.nb + row0 + rr + 8 * h] = part[h];
        }
    }
}

// ------------------------------------------------------------------ combine

constexpr int kTrCombineRows = 16;
constexpr int kTrCombineThreads = 256;
constexpr int kTrCombineSlots = 16;               // segments joined at a time

// A CTA joins 16 rows of a group.  Drafted part: the scores of 16 rows and 8 nodes a warp by bf16 products, a softmax
// by warps, then thread = (coordinate, 8 rows) over the values, all before the cached part has to be there.  Cached
// part: the weights of up to 16 segments at once, then the segments' rows, loads in flight together; rotated back by H
// and D, divided, rounded.
__global__ void __launch_bounds__(kTrCombineThreads)
tree_combine_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ QuantTables TV, int grid_main)
{
    extern __shared__ __align__(16) float sS[];                 // [nodes][16] scores, then weights
    __shared__ float sM[16], sL[16], sScale[16];
    __shared__ __align__(16) float sW[kTrCombineSlots][16];
    __shared__ float buf[16][kTrD];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, p = lane & 3, rr = lane >> 2;
    const int64_t g = blockIdx.y;
    const int r0 = blockIdx.x * kTrCombineRows, n = a.nodes;
    const int64_t b = g / a.kv_heads;
    const int kv = (int)(g - b * a.kv_heads);
    {
        uint32_t A[2][16];
        const uint64_t *mrow[2];
        int node[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = r0 + rr + 8 * h;
            const bool in = r < a.rows;
            node[h] = in ? r / a.rep : -1;
            mrow[h] = a.mask && in ? a.mask + b * a.mask_batch + (int64_t)node[h] * ((n + 63) / 64) : nullptr;
            const uint4 *src = in ? reinterpret_cast<const uint4 *>(tr_row(a.q, a.qs, a, g, r) + 32 * p) : nullptr;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = in ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
                A[h][4 * i] = v.x; A[h][4 * i + 1] = v.y; A[h][4 * i + 2] = v.z; A[h][4 * i + 3] = v.w;
            }
        }
        for (int j0 = 8 * warp; j0 < n; j0 += 64) {
            uint32_t B[16];
            const bool in = j0 + rr < n;
            const uint4 *src = reinterpret_cast<const uint4 *>(a.k_new + b * a.ks.batch + (int64_t)(in ? j0 + rr : 0) * a.ks.token +
                                                               (int64_t)kv * a.ks.head + 32 * p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = __ldg(src + i);
                B[4 * i] = v.x; B[4 * i + 1] = v.y; B[4 * i + 2] = v.z; B[4 * i + 3] = v.w;
            }
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t af[4] = {A[0][2 * k], A[1][2 * k], A[0][2 * k + 1], A[1][2 * k + 1]};
                tr_mma_bf16(d, af, B[2 * k], B[2 * k + 1]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t bits = mrow[h] ? (uint32_t)(__ldg(mrow[h] + (j0 >> 6)) >> (j0 & 63)) : 0u;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = j0 + 2 * p + e;
                    const bool sees = a.mask ? (bits >> (2 * p + e)) & 1u : j <= node[h];
                    if (j < n) sS[j * 16 + rr + 8 * h] = sees ? d[2 * h + e] * a.qscale : -INFINITY;
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {                               // softmax of rows 2 warp, 2 warp + 1
        const int row = 2 * warp + i;
        float m = -INFINITY, l = 0.0f;
        for (int j = lane; j < n; j += 32) m = fmaxf(m, sS[j * 16 + row]);
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        for (int j = lane; j < n; j += 32) {
            const float s = sS[j * 16 + row];
            const float w = s == -INFINITY ? 0.0f : tr_ex2(s - m);       // (a NaN score stays one)
            sS[j * 16 + row] = w;
            l += w;
        }
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) { sM[row] = m; sL[row] = l; }
    }
    __syncthreads();
    const int d = tid & (kTrD - 1), h0 = (tid >> 7) * 8;        // coordinate, first of this thread's 8 rows
    float ot[8], acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) ot[i] = acc[i] = 0.0f;
    const uint16_t *vcol = a.v_new + b * a.vs.batch + (int64_t)kv * a.vs.head + d;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
        const float v = __uint_as_float((uint32_t)__ldg(vcol + (int64_t)j * a.vs.token) << 16);
        const float4 w0 = *reinterpret_cast<const float4 *>(sS + j * 16 + h0), w1 = *reinterpret_cast<const float4 *>(sS + j * 16 + h0 + 4);
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (w[i] != 0.0f) ot[i] = __fmaf_rn(w[i], v, ot[i]);         // a hidden value may be anything: it is not used
    }
    const int rb = r0 / a.nb;
    const int64_t pg = g * a.rbs + rb;
    tr_wait_previous();
    int64_t tiles = 0;
    if (grid_main > 0) tiles = a.off[g + 1] - a.off[g];
    if (tiles > 0) {
        // the CTA of an item: the largest c with total c / ctas <= item
        const int64_t total = a.off[a.G] * a.rbs, ctas = total < grid_main ? total : grid_main;
        const int64_t lo = a.off[g] * a.rbs + rb * tiles, hi = lo + tiles - 1;
        const int c_lo = (int)(((lo + 1) * ctas - 1) / total), c_hi = (int)(((hi + 1) * ctas - 1) / total);
        const int in = r0 - rb * a.nb;
        for (int c = c_lo; c <= c_hi; c += kTrCombineSlots) {
            const int ns = c_hi - c + 1 < kTrCombineSlots ? c_hi - c + 1 : kTrCombineSlots;
            const float *P = a.part + (size_t)(c + pg) * tr_part_floats(a.nb);
            {
                const int row = tid >> 4, slot = tid & 15;
                const float *q = P + (size_t)slot * tr_part_floats(a.nb) + (size_t)a.nb * kTrD + in + row;
                const float m = slot < ns ? q[0] : -INFINITY, l = slot < ns ? q[a.nb] : 0.0f, old = sM[row];
                float mx = m;
                for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                mx = fmaxf(mx, old);
                const float w = m == -INFINITY ? 0.0f : tr_ex2(m - mx);
                float sum = w * l;
                for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                sW[slot][row] = w;
                if (slot == 0) {
                    const float sc = old == -INFINITY ? 0.0f : tr_ex2(old - mx);
                    sScale[row] = sc;
                    sL[row] = __fmaf_rn(sL[row], sc, sum);
                    sM[row] = mx;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ot[i] *= sScale[h0 + i];
                acc[i] *= sScale[h0 + i];
            }
            const float *O = P + (size_t)(in + h0) * kTrD + d;
#pragma unroll 2
            for (int s = 0; s < ns; ++s, O += tr_part_floats(a.nb)) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = O[i * kTrD];
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = __fmaf_rn(x[i], sW[s][h0 + i], acc[i]);
            }
            __syncthreads();
        }
        // H over the 128 coordinates: stages inside the warp, then across the warps
#pragma unroll
        for (int h = 1; h < 32; h <<= 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float o = __shfl_xor_sync(0xffffffffu, acc[i], h);
                acc[i] = (lane & h) ? o - acc[i] : acc[i] + o;
            }
        }
#pragma unroll
        for (int h = 32; h < kTrD; h <<= 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) buf[h0 + i][d] = acc[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float o = buf[h0 + i][d ^ h];
                acc[i] = (d & h) ? o - acc[i] : acc[i] + o;
            }
            __syncthreads();
        }
    }
    const bool neg = (TV.sign_words[d >> 5] >> (d & 31)) & 1u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + h0 + i;
        if (r >= a.rows) break;
        const float x = __fmaf_rn(neg ? -acc[i] : acc[i], a.vup, ot[i]), l = sL[h0 + i];
        const float y = l == 0.0f ? 0.0f : __fdiv_rn(x, l);
        uint16_t *dst = const_cast<uint16_t *>(tr_row(a.out, a.os, a, g, r));
        dst[d] = (uint16_t)(pack2<true>(y, 0.0f) & 0xffffu);
    }
}

}  // namespace rq

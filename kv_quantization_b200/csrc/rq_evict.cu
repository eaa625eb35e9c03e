// rq_evict.cu -- eviction from a cache by accumulated attention weight:
//   accumulate  out[t] = decay acc[t] + sum_q softmax_t(scale s(q, t))
//   select      the `keep` tokens of largest sum (first and last tokens forced, ties to the lowest index)
//   gather      the kept records of every array of the cache, moved together

#include <cooperative_groups.h>

#include "rq_common.cuh"
#include "rq_cache_ops.h"

namespace cg = cooperative_groups;

namespace rq {

namespace {

// ------------------------------------------------------------------ accumulate

constexpr int kAcThreads = 256;
constexpr int kAcChunk = 1024;                  // tokens per CTA: 4 a thread

__device__ __forceinline__ float ac_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Exponents are (s - m) k in units of log2.  k is never 0, so that a score of -inf, and the maximum of a part without
// any score, keep their weight of 0 at every scale (-inf * 0 would be NaN): at scale 0 the smallest number, which
// leaves the exponent of any finite score at 0 to within 2^-20.
__device__ __forceinline__ float ac_factor(const AccumulateArgs &a)
{
    return fmaxf(a.scale * 1.4426950408889634074f, 0x1p-149f);
}

__device__ __forceinline__ int64_t ac_row_len(const AccumulateArgs &a, int64_t row)
{
    if (!a.row_len) return a.T;
    const int64_t n = __ldg(a.row_len + row);
    return n < 0 ? 0 : (n < a.T ? n : a.T);
}

// Per (row, chunk): maximum and sum of exponentials.  A warp takes a row of the chunk; VEC: T is a multiple of 4, and a
// lane's values are 4 neighbours.  Bound by the read of the scores.
template <bool VEC>
__global__ void __launch_bounds__(kAcThreads)
accumulate_stats_kernel(const __grid_constant__ AccumulateArgs a, int n_chunks)
{
    const int64_t g = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t)blockIdx.x * kAcChunk;
    const float k = ac_factor(a);
    for (int r = warp; r < a.nq; r += kAcThreads / 32) {
        const int64_t row = g * a.nq + r;
        const int64_t left = ac_row_len(a, row) - t0;
        const int n = left < 0 ? 0 : (left < kAcChunk ? (int)left : kAcChunk);
        const float *s = a.scores + row * a.T + t0;
        float v[kAcChunk / 32], m = -INFINITY;
        if (VEC && n == kAcChunk) {
#pragma unroll
            for (int j = 0; j < kAcChunk / 32; j += 4) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(s) + (j / 4) * 32 + lane);
                v[j] = x.x; v[j + 1] = x.y; v[j + 2] = x.z; v[j + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kAcChunk / 32; ++j) {
                const int t = j * 32 + lane;
                v[j] = t < n ? __ldg(s + t) : -INFINITY;
            }
        }
#pragma unroll
        for (int j = 0; j < kAcChunk / 32; ++j) m = fmaxf(m, v[j]);
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float off = m == -INFINITY ? 0.0f : m;
        float l = 0.0f;
#pragma unroll
        for (int j = 0; j < kAcChunk / 32; ++j)          // (a whole chunk has no places behind its row's length)
            l += n == kAcChunk || j * 32 + lane < n ? ac_exp2((v[j] - off) * k) : 0.0f;
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) {
            float2 *p = reinterpret_cast<float2 *>(a.workspace) + row * n_chunks + blockIdx.x;
            *p = make_float2(m, l);
        }
    }
}

// Per (chunk, group): a thread holds 4 tokens and adds the queries' weights to them, eight queries' scores in flight.
// The second read of the scores: the groups are taken in the opposite order, so that those the first kernel read last
// are still in L2.  VEC: T is a multiple of 4 (16-byte rows); else the 4 tokens are a stride apart.
// Every CTA joins the parts of all chunks of its group's rows again: 8 bytes a query and chunk beside the 4096 bytes of
// scores that it reads, T / 1024 times, so the cost grows with T^2: 6 % of the scores' bytes at 32768 tokens, 25 % at
// 131072, as much as the scores at 524288.
template <bool VEC>
__global__ void __launch_bounds__(kAcThreads)
accumulate_columns_kernel(const __grid_constant__ AccumulateArgs a, int n_chunks)
{
    extern __shared__ float4 rows[];                     // maximum, 1 / sum, length in this chunk
    const int64_t g = gridDim.y - 1 - blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t)blockIdx.x * kAcChunk;
    const float k = ac_factor(a);
    for (int r = warp; r < a.nq; r += kAcThreads / 32) {
        const float2 *p = reinterpret_cast<const float2 *>(a.workspace) + (g * a.nq + r) * n_chunks;
        float m = -INFINITY, l = 0.0f;
        for (int c = lane; c < n_chunks; c += 32) {
            const float2 x = p[c];
            const float mn = fmaxf(m, x.x), off = mn == -INFINITY ? 0.0f : mn;
            l = l * ac_exp2((m - off) * k) + x.y * ac_exp2((x.x - off) * k);
            m = mn;
        }
        for (int o = 16; o > 0; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
            const float mn = fmaxf(m, m2), off = mn == -INFINITY ? 0.0f : mn;
            l = l * ac_exp2((m - off) * k) + l2 * ac_exp2((m2 - off) * k);
            m = mn;
        }
        if (lane == 0) {
            const int64_t left = ac_row_len(a, g * a.nq + r) - t0;
            rows[r] = make_float4(m == -INFINITY ? 0.0f : m, l == 0.0f ? 0.0f : 1.0f / l,
                                  __int_as_float(left < 0 ? 0 : (left < kAcChunk ? (int)left : kAcChunk)), 0.0f);
        }
    }
    __syncthreads();
    // the thread's tokens e = 0 .. 3: first + e step
    const int first = VEC ? 4 * threadIdx.x : threadIdx.x, step = VEC ? 1 : kAcThreads;
    const float *src = a.scores + g * a.nq * a.T + t0 + first;
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int r0 = 0; r0 < a.nq; r0 += 8) {
        float v[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int n = r0 + i < a.nq ? __float_as_int(rows[r0 + i].z) : 0;      // tokens of the chunk that it sees
            const float *p = src + (int64_t)(r0 + i) * a.T;
            if (VEC && first + 3 < n) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(p));
                v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] = first + e * step < n ? __ldg(p + e * step) : -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (r0 + i >= a.nq) break;
            const float4 x = rows[r0 + i];
            const int n = __float_as_int(x.z);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (first + e * step < n) sum[e] = __fmaf_rn(ac_exp2((v[i][e] - x.x) * k), x.y, sum[e]);
        }
    }
    const float *acc = a.acc + g * a.T + t0 + first;
    float *out = a.out + g * a.T + t0 + first;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (t0 + first + e * step >= a.T) break;
        out[e * step] = (a.decay == 0.0f ? 0.0f : a.decay * acc[e * step]) + sum[e];
    }
}

}  // namespace

size_t accumulate_workspace_bytes(int64_t G, int nq, int64_t T)
{
    return (size_t)G * nq * ((T + kAcChunk - 1) / kAcChunk) * sizeof(float2);
}

cudaError_t launch_accumulate(const AccumulateArgs &a, cudaStream_t st)
{
    const int n_chunks = (int)((a.T + kAcChunk - 1) / kAcChunk);
    const dim3 grid((unsigned)n_chunks, (unsigned)a.G);
    if (a.T % 4 == 0) accumulate_stats_kernel<true><<<grid, kAcThreads, 0, st>>>(a, n_chunks);
    else accumulate_stats_kernel<false><<<grid, kAcThreads, 0, st>>>(a, n_chunks);
    note_launch("accumulate_stats_kernel");
    const size_t smem = (size_t)a.nq * sizeof(float4);
    auto columns = a.T % 4 == 0 ? accumulate_columns_kernel<true> : accumulate_columns_kernel<false>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(columns, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    columns<<<grid, kAcThreads, smem, st>>>(a, n_chunks);
    note_launch("accumulate_columns_kernel");
    return cudaGetLastError();
}

// ------------------------------------------------------------------ select

namespace {

constexpr int kSeThreads = 1024;
constexpr int kSeMaxCluster = 8;
constexpr uint32_t kSeCandidates = 128;

// Sort key of a weight sum: larger sums have larger keys, -0 equals +0, NaN comes last (key 1); 0 is "no token".
__device__ __forceinline__ uint32_t se_key(float x)
{
    if (x != x) return 1u;
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// One cluster per group.  CTA c of the cluster holds the keys of tokens [c slice, (c + 1) slice), IT a thread in
// registers (IT = 0: read again from global memory in every pass).  The threshold (the keep-th largest key) is found
// four bits at a time: every warp counts the digits of its keys that still match by ballots, counts are summed over the
// cluster (integer sums: no order matters), and the digit in which the rank falls is appended; it ends early when
// all keys that match are wanted, or few enough match to rank them directly.  Then every CTA writes its kept indices at
// its place in index order.
// The search is bound by the latency of its (at most eight) rounds, not by the one read of the sums.
template <int IT>
__global__ void __launch_bounds__(kSeThreads, 1)
select_kernel(const __grid_constant__ SelectArgs a, int64_t slice)
{
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int64_t g = blockIdx.x / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ uint32_t local[2][16];                        // this CTA's digit counts, by round parity
    __shared__ uint32_t all[2][kSeMaxCluster][16];           // every CTA's, written by its owner
    __shared__ uint32_t above[kSeMaxCluster][2];             // every CTA's keys above / at the threshold
    __shared__ uint32_t wpre[32][2];
    __shared__ uint32_t cand[kSeCandidates];                 // the last keys that match, of all CTAs
    __shared__ uint32_t found[2], n_cand;

    int64_t len = a.T;
    if (a.len) {
        len = __ldg(a.len + g);
        len = len < 0 ? 0 : (len < a.T ? len : a.T);
    }
    const int keep = a.keep;
    int32_t *idx = a.idx + g * keep;
    const int64_t c0 = rank * slice;
    const int iters = IT > 0 ? IT : (int)(slice / kSeThreads);
    // warp w holds tokens c0 + w 32 iters ..., item j lane l: + 32 j + l
    const int64_t w0 = c0 + (int64_t)warp * 32 * iters;
    const float *acc = a.acc + g * a.T;
    auto load_key = [&](int j) -> uint32_t {
        const int64_t t = w0 + 32 * j + lane;
        if (t >= len) return 0u;
        if (t < a.n_sink || t >= len - a.n_recent) return 0xffffffffu;
        return se_key(__ldg(acc + t));
    };
    uint32_t key[IT > 0 ? IT : 1];
    if constexpr (IT > 0) {
#pragma unroll
        for (int j = 0; j < IT; ++j) key[j] = load_key(j);
    }
    auto for_keys = [&](auto &&f) {
        if constexpr (IT > 0) {
#pragma unroll
            for (int j = 0; j < IT; ++j) f(j, key[j]);
        } else {
            for (int j = 0; j < iters; ++j) f(j, load_key(j));
        }
    };
    if (tid < 32) local[tid >> 4][tid & 15] = 0u;
    if (tid == 32) n_cand = 0u;
    cl.sync();                                               // every CTA of the cluster has started

    uint32_t prefix = 0u, mask = 0u;                         // keys with (key & mask) == prefix still match
    uint32_t need = len < keep ? (uint32_t)len : (uint32_t)keep;     // of them, this many are wanted
    bool every = need == 0u || len <= keep;                  // all matching keys (not 0) are wanted
    for (int round = 0; round < 8 && !every; ++round) {
        const int shift = 28 - 4 * round, par = round & 1;
        uint32_t n = 0u;                                     // lane: the warp's keys with digit lane % 16
        for_keys([&](int, uint32_t kk) {
            const uint32_t d = kk >> shift;
            uint32_t m = __ballot_sync(0xffffffffu, kk != 0u && (kk & mask) == prefix);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint32_t set = __ballot_sync(0xffffffffu, (d >> b) & 1u);
                m &= (lane >> b) & 1 ? set : ~set;
            }
            n += __popc(m);
        });
        if (lane < 16 && n) atomicAdd(&local[par][lane], n);
        __syncthreads();
        if (tid < 16 * C) {
            uint32_t *dst = cl.map_shared_rank(&all[par][rank][tid & 15], tid >> 4);
            *dst = local[par][tid & 15];
        }
        if (tid >= kSeThreads - 16) local[par ^ 1][tid & 15] = 0u;
        if (C > 1) cl.sync();
        else __syncthreads();
        uint32_t total = 0u;                                 // lane: digit 15 - lane
        if (lane < 16)
            for (int c = 0; c < C; ++c) total += all[par][c][15 - lane];
        uint32_t run = total;                                // keys of this digit or a larger one
        for (int o = 1; o < 16; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += x;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, lane < 16 && run >= need);
        const int src = __ffs(hit) - 1;                      // the digit in which the rank falls
        const uint32_t upto = __shfl_sync(0xffffffffu, run, src), in = __shfl_sync(0xffffffffu, total, src);
        need -= upto - in;
        prefix |= (uint32_t)(15 - src) << shift;
        mask |= 15u << shift;
        every = in == need;
        if (!every && in <= kSeCandidates) {
            // few keys match: every CTA gets all of them (the places are known from the round's counts) and ranks them
            uint32_t at = 0u;
            for (int c = 0; c < rank; ++c) at += all[par][c][15 - src];
            for_keys([&](int, uint32_t kk) {
                if (kk == 0u || (kk & mask) != prefix) return;
                const uint32_t i = at + atomicAdd(&n_cand, 1u);
                for (int c = 0; c < C; ++c) *cl.map_shared_rank(&cand[i], c) = kk;
            });
            if (C > 1) cl.sync();
            else __syncthreads();
            if (tid < (int)in) {
                const uint32_t kk = cand[tid];
                uint32_t above_it = 0u, same = 0u;
                for (uint32_t i = 0; i < in; ++i) {
                    above_it += cand[i] > kk;
                    same += cand[i] == kk;
                }
                if (above_it < need && need <= above_it + same) {
                    found[0] = kk;
                    found[1] = need - above_it;
                }
            }
            __syncthreads();
            prefix = found[0];
            mask = 0xffffffffu;
            need = found[1];
            break;
        }
    }
    // keys above the threshold are kept; of those that match it, the first `need` in index order
    const uint32_t kept = len < keep ? (uint32_t)len : (uint32_t)keep;
    uint32_t gt = 0u, eq = 0u;
    auto classify = [&](uint32_t kk, bool &is_gt, bool &is_eq) {
        is_eq = kk != 0u && (kk & mask) == prefix;
        is_gt = kk != 0u && (kk & mask) > prefix;
    };
    for_keys([&](int, uint32_t kk) {
        bool ig, ie;
        classify(kk, ig, ie);
        gt += __popc(__ballot_sync(0xffffffffu, ig));
        eq += __popc(__ballot_sync(0xffffffffu, ie));
    });
    if (lane == 0) { wpre[warp][0] = gt; wpre[warp][1] = eq; }
    __syncthreads();
    uint32_t pg = wpre[lane][0], pe = wpre[lane][1];
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, pg, o), y = __shfl_up_sync(0xffffffffu, pe, o);
        if (lane >= o) { pg += x; pe += y; }
    }
    const uint32_t tot_g = __shfl_sync(0xffffffffu, pg, 31), tot_e = __shfl_sync(0xffffffffu, pe, 31);
    pg = __shfl_sync(0xffffffffu, pg, warp) - gt;            // before this warp in the CTA
    pe = __shfl_sync(0xffffffffu, pe, warp) - eq;
    if (tid < C) {
        uint32_t *dst = cl.map_shared_rank(&above[rank][0], tid);
        dst[0] = tot_g;
        dst[1] = tot_e;
    }
    cl.sync();                                               // also the last access to another CTA's memory
    for (int c = 0; c < rank; ++c) { pg += above[c][0]; pe += above[c][1]; }
    for_keys([&](int j, uint32_t kk) {
        bool ig, ie;
        classify(kk, ig, ie);
        const uint32_t bg = __ballot_sync(0xffffffffu, ig), be = __ballot_sync(0xffffffffu, ie);
        const uint32_t lower = (1u << lane) - 1u;
        const uint32_t my_g = pg + __popc(bg & lower), my_e = pe + __popc(be & lower);
        const uint32_t want = every ? 0xffffffffu : need;
        if (ig || (ie && my_e < want)) {
            const uint32_t at = my_g + (my_e < want ? my_e : want);
            idx[at] = (int32_t)(w0 + 32 * j + lane);
        }
        pg += __popc(bg);
        pe += __popc(be);
    });
    for (int64_t i = (int64_t)kept + rank * kSeThreads + tid; i < keep; i += (int64_t)C * kSeThreads) idx[i] = -1;
    if (rank == 0 && tid == 0) a.count[g] = (int32_t)kept;
}

template <int IT>
cudaError_t se_launch(const SelectArgs &a, int cluster, int64_t slice, cudaStream_t st)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.G * cluster));
    cfg.blockDim = dim3(kSeThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, select_kernel<IT>, a, slice);
    if (e != cudaSuccess) return e;
    note_launch("select_kernel");
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_select(const SelectArgs &a, cudaStream_t st)
{
    // the smallest cluster whose CTAs hold 8 keys a thread; up to 16 a thread in the largest
    int cluster = 1;
    while (cluster < kSeMaxCluster && a.T > (int64_t)cluster * 8 * kSeThreads) cluster *= 2;
    int64_t per = (a.T + cluster - 1) / cluster;
    per = (per + kSeThreads - 1) / kSeThreads;               // keys a thread
    if (per <= 1) return se_launch<1>(a, cluster, kSeThreads, st);
    if (per <= 4) return se_launch<4>(a, cluster, 4 * kSeThreads, st);
    if (per <= 8) return se_launch<8>(a, cluster, 8 * kSeThreads, st);
    if (per <= 16) return se_launch<16>(a, cluster, 16 * kSeThreads, st);
    return se_launch<0>(a, cluster, per * kSeThreads, st);
}

// ------------------------------------------------------------------ gather

namespace {

constexpr int kGaThreads = 256;

// Four units of a thread in flight.
template <typename U>
__device__ __forceinline__ void ga_copy(const uint8_t *src, uint8_t *dst, int units, const int32_t *rows, int n)
{
    const U *s = reinterpret_cast<const U *>(src);
    U *d = reinterpret_cast<U *>(dst);
    const int shift = (units & (units - 1)) == 0 ? 31 - __clz(units) : -1;
    for (int i0 = threadIdx.x; i0 < n * units; i0 += 4 * kGaThreads) {
        U v[4];
        bool take[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + e * kGaThreads;
            take[e] = i < n * units;
            if (!take[e]) continue;
            const int r = shift >= 0 ? i >> shift : i / units, u = i - r * units, t = rows[r];
            take[e] = t >= 0;
            if (take[e]) v[e] = __ldg(s + (int64_t)t * units + u);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (take[e]) d[i0 + e * kGaThreads] = v[e];
    }
}

// A CTA moves ROWS kept rows of one group in one array (blockIdx.z), in the widest unit that divides the row.
template <int ROWS>
__global__ void __launch_bounds__(kGaThreads)
gather_kernel(const __grid_constant__ GatherArgs a)
{
    __shared__ int32_t rows[ROWS];
    const int64_t g = blockIdx.y;
    const int j0 = blockIdx.x * ROWS;
    int n = __ldg(a.count + g);
    n = n < a.keep ? n : a.keep;
    n = n - j0 < ROWS ? n - j0 : ROWS;
    if (n <= 0) return;
    for (int i = threadIdx.x; i < n; i += kGaThreads) {
        const int t = __ldg(a.idx + g * a.keep + j0 + i);
        rows[i] = t >= 0 && t < a.T ? t : -1;                // an index outside the cache moves nothing
    }
    __syncthreads();
    {
        const int k = blockIdx.z;
        const int64_t rb = a.row_bytes[k];
        const uint8_t *src = a.src[k] + g * a.T * rb;
        uint8_t *dst = a.dst[k] + (g * a.T_dst + j0) * rb;
        const int64_t odd = rb | (a.T * rb) | (a.T_dst * rb);
        if (odd % 16 == 0) ga_copy<uint4>(src, dst, (int)(rb / 16), rows, n);
        else if (odd % 8 == 0) ga_copy<uint2>(src, dst, (int)(rb / 8), rows, n);
        else if (odd % 4 == 0) ga_copy<uint32_t>(src, dst, (int)(rb / 4), rows, n);
        else if (odd % 2 == 0) ga_copy<uint16_t>(src, dst, (int)(rb / 2), rows, n);
        else ga_copy<uint8_t>(src, dst, (int)rb, rows, n);
    }
}

}  // namespace

cudaError_t launch_gather(const GatherArgs &a, cudaStream_t st)
{
    // rows a CTA: enough to keep its threads' loads in flight, unless that leaves SMs without work
    const bool wide = (int64_t)a.keep * a.G >= 256 * 512;
    const int rows = wide ? 256 : 64;
    const dim3 grid((unsigned)((a.keep + rows - 1) / rows), (unsigned)a.G, (unsigned)a.n_arrays);
    if (wide) gather_kernel<256><<<grid, kGaThreads, 0, st>>>(a);
    else gather_kernel<64><<<grid, kGaThreads, 0, st>>>(a);
    note_launch("gather_kernel");
    return cudaGetLastError();
}

}  // namespace rq

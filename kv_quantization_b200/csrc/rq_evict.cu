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

__device__ __forceinline__ int64_t ac_row_len(const AccumulateArgs &a, int64_t row)
{
    if (!a.row_len) return a.T;
    const int64_t n = __ldg(a.row_len + row);
    return n < 0 ? 0 : (n < a.T ? n : a.T);
}

// Per (row, chunk): maximum and sum of exponentials.  A warp takes a row of the chunk.
__global__ void __launch_bounds__(kAcThreads)
accumulate_stats_kernel(const __grid_constant__ AccumulateArgs a, int n_chunks)
{
    const int64_t g = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t)blockIdx.x * kAcChunk;
    const float k = a.scale * 1.4426950408889634074f;
    for (int r = warp; r < a.nq; r += kAcThreads / 32) {
        const int64_t row = g * a.nq + r;
        const int64_t left = ac_row_len(a, row) - t0;
        const int n = left < 0 ? 0 : (left < kAcChunk ? (int)left : kAcChunk);
        const float *s = a.scores + row * a.T + t0;
        float v[kAcChunk / 32], m = -INFINITY;
#pragma unroll
        for (int j = 0; j < kAcChunk / 32; ++j) {
            const int t = j * 32 + lane;
            v[j] = t < n ? __ldg(s + t) : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < kAcChunk / 32; ++j) m = fmaxf(m, v[j]);
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float off = m == -INFINITY ? 0.0f : m;
        float l = 0.0f;
#pragma unroll
        for (int j = 0; j < kAcChunk / 32; ++j) l += j * 32 + lane < n ? ac_exp2((v[j] - off) * k) : 0.0f;
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) {
            float2 *p = reinterpret_cast<float2 *>(a.workspace) + row * n_chunks + blockIdx.x;
            *p = make_float2(m, l);
        }
    }
}

__global__ void __launch_bounds__(kAcThreads)
accumulate_columns_kernel(const __grid_constant__ AccumulateArgs a, int n_chunks)
{
    extern __shared__ float2 rows[];                     // (maximum, 1 / sum) of every row
    const int64_t g = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t)blockIdx.x * kAcChunk;
    const float k = a.scale * 1.4426950408889634074f;
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
        if (lane == 0) rows[r] = make_float2(m == -INFINITY ? 0.0f : m, l == 0.0f ? 0.0f : 1.0f / l);
    }
    __syncthreads();
    for (int e = 0; e < kAcChunk / kAcThreads; ++e) {
        const int64_t t = t0 + e * kAcThreads + threadIdx.x;
        if (t >= a.T) break;
        float sum = 0.0f;
        for (int r = 0; r < a.nq; ++r) {
            const int64_t row = g * a.nq + r;
            if (t < ac_row_len(a, row)) {
                const float2 x = rows[r];
                sum = __fmaf_rn(ac_exp2((__ldg(a.scores + row * a.T + t) - x.x) * k), x.y, sum);
            }
        }
        const float old = a.decay == 0.0f ? 0.0f : a.decay * a.acc[g * a.T + t];
        a.out[g * a.T + t] = old + sum;
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
    accumulate_stats_kernel<<<grid, kAcThreads, 0, st>>>(a, n_chunks);
    note_launch("accumulate_stats_kernel");
    const size_t smem = (size_t)a.nq * sizeof(float2);
    accumulate_columns_kernel<<<grid, kAcThreads, smem, st>>>(a, n_chunks);
    note_launch("accumulate_columns_kernel");
    return cudaGetLastError();
}

// ------------------------------------------------------------------ select

namespace {

constexpr int kSeThreads = 1024;
constexpr int kSeMaxCluster = 8;

// Sort key of a weight sum: larger sums have larger keys, -0 equals +0, NaN comes last (key 1); 0 is "no token".
__device__ __forceinline__ uint32_t se_key(float x)
{
    if (x != x) return 1u;
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// One cluster per group.  CTA c of the cluster holds the keys of tokens [c slice, (c + 1) slice), IT a thread in
// registers (IT = 0: read again from global memory in every pass).  The threshold (the keep-th largest key) is found
// four bits at a time: every thread counts the digits of its keys that still match, counts are summed over the
// cluster (integer sums: no order matters), and the digit in which the rank falls is appended; it ends early when
// all keys that match are wanted.  Then every CTA writes its kept indices at its place in index order.
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
    cl.sync();                                               // every CTA of the cluster has started

    uint32_t prefix = 0u, mask = 0u;                         // keys with (key & mask) == prefix still match
    uint32_t need = len < keep ? (uint32_t)len : (uint32_t)keep;     // of them, this many are wanted
    bool every = need == 0u || len <= keep;                  // all matching keys (not 0) are wanted
    for (int round = 0; round < 8 && !every; ++round) {
        const int shift = 28 - 4 * round, par = round & 1;
        uint32_t n[8];                                       // digits 2 i (low half) and 2 i + 1 (high half)
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = 0u;
        for_keys([&](int, uint32_t kk) {
            const uint32_t d = (kk >> shift) & 15u;
            const uint32_t one = (kk != 0u && (kk & mask) == prefix) ? 1u << (16 * (d & 1)) : 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] += (d >> 1) == (uint32_t)i ? one : 0u;
        });
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo = __reduce_add_sync(0xffffffffu, n[i] & 0xffffu), hi = __reduce_add_sync(0xffffffffu, n[i] >> 16);
            if (lane == 0 && lo) atomicAdd(&local[par][2 * i], lo);
            if (lane == 1 && hi) atomicAdd(&local[par][2 * i + 1], hi);
        }
        __syncthreads();
        if (tid < 16 * C) {
            uint32_t *dst = cl.map_shared_rank(&all[par][rank][tid & 15], tid >> 4);
            *dst = local[par][tid & 15];
        }
        if (tid >= kSeThreads - 16) local[par ^ 1][tid & 15] = 0u;
        cl.sync();
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
constexpr int kGaRows = 64;

template <typename U>
__device__ __forceinline__ void ga_copy(const uint8_t *src, uint8_t *dst, int units, const int32_t *rows, int n)
{
    const U *s = reinterpret_cast<const U *>(src);
    U *d = reinterpret_cast<U *>(dst);
    for (int i = threadIdx.x; i < n * units; i += kGaThreads) {
        const int r = i / units, u = i - r * units, t = rows[r];
        if (t >= 0) d[i] = __ldg(s + (int64_t)t * units + u);
    }
}

// A CTA moves kGaRows kept rows of one group in every array, in the widest unit that divides the row.
__global__ void __launch_bounds__(kGaThreads)
gather_kernel(const __grid_constant__ GatherArgs a)
{
    __shared__ int32_t rows[kGaRows];
    const int64_t g = blockIdx.y;
    const int j0 = blockIdx.x * kGaRows;
    int n = __ldg(a.count + g);
    n = n < a.keep ? n : a.keep;
    n = n - j0 < kGaRows ? n - j0 : kGaRows;
    if (n <= 0) return;
    if (threadIdx.x < n) {
        const int t = __ldg(a.idx + g * a.keep + j0 + threadIdx.x);
        rows[threadIdx.x] = t >= 0 && t < a.T ? t : -1;      // an index outside the cache moves nothing
    }
    __syncthreads();
    for (int k = 0; k < a.n_arrays; ++k) {
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
    const dim3 grid((unsigned)((a.keep + kGaRows - 1) / kGaRows), (unsigned)a.G);
    gather_kernel<<<grid, kGaThreads, 0, st>>>(a);
    note_launch("gather_kernel");
    return cudaGetLastError();
}

}  // namespace rq

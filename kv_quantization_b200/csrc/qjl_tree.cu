// qjl_tree.cu -- launcher of the attention of drafted tokens over the compressed cache (kernels in qjl_tree.cuh).
#include "qjl_tree.cuh"

#include <cmath>

namespace rq {

namespace {

int64_t up256(int64_t x) { return (x + 255) & ~(int64_t)255; }

// Query rows a block: 32 or 64 when that holds the group's rows; above, 128 (fewer passes over the cache) where the
// operand of kb columns leaves room in shared memory.  Measured over 32 x 32768 tokens: 128 rows on two-stage keys in
// blocks of 128 317 us, of 64 366 us, of 32 629 us; 256 rows on pure sketch keys 420, 416 and 672 us.
int tree_nb(int rows, int kb) { return rows <= 32 ? 32 : (rows <= 64 || kb > 384 ? 64 : 128); }

int64_t tree_grid(int64_t G, int rbs, int nb, int64_t T, int num_sms)
{
    const int64_t items = G * rbs * ((T + kTrTok - 1) / kTrTok), most = (int64_t)num_sms * tr_ctas(nb);
    return items < most ? items : most;
}

// A launch that may start before the kernel ahead of it in the stream has ended.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int NB, bool TWO, bool V4>
cudaError_t launch_main(const TreeArgs &a, const QuantTables &tk, const QuantTables &tv, int grid, cudaStream_t st)
{
    // weight and value buffers: two of each if the SM's shared memory holds them for tr_ctas CTAs (one weight buffer and
    // two value buffers, or the other way round, measured the same); else one CTA an SM
    const int cfg[][2] = {{2, 2}, {1, 2}, {1, 1}};
    const size_t limits[] = {kMaxSmemPerBlock / tr_ctas(NB) - 1024 * (tr_ctas(NB) - 1), kMaxSmemPerBlock};
    for (const size_t limit : limits) {
        for (const auto &c : cfg) {
            const size_t smem = tr_smem(NB, a.kb, a.pw, a.vpw, c[0], c[1]);
            if (smem > limit) continue;
            auto kern = tree_attention_kernel<NB, TWO, V4>;
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
            e = launch_early(kern, dim3((unsigned)grid), tr_threads(NB), smem, st, a, tk, tv, c[0], c[1]);
            if (e == cudaSuccess) note_launch("tree_attention_kernel");
            return e;
        }
    }
    return cudaErrorNotSupported;
}

template <int NB>
cudaError_t launch_nb(const TreeArgs &a, const QuantTables &tk, const QuantTables &tv, int grid, cudaStream_t st)
{
    if (a.vpw == 4) return a.pw ? launch_main<NB, true, true>(a, tk, tv, grid, st) : launch_main<NB, false, true>(a, tk, tv, grid, st);
    return a.pw ? launch_main<NB, true, false>(a, tk, tv, grid, st) : launch_main<NB, false, false>(a, tk, tv, grid, st);
}

struct Plan {
    int kb, nb, rbs;
    int64_t q, c, off, part, bytes;
};

Plan tree_plan(int64_t G, int rows, int64_t T, int m, bool two, int num_sms)
{
    Plan p;
    p.kb = m + (two ? kTrD : 0);
    p.nb = tree_nb(rows, p.kb);
    p.rbs = (rows + p.nb - 1) / p.nb;
    p.q = 0;
    p.c = up256(p.q + G * p.rbs * p.nb * (int64_t)p.kb * 2);
    p.off = up256(p.c + G * p.rbs * p.nb * (int64_t)(1 + p.kb / 32) * (int64_t)sizeof(float));
    p.part = up256(p.off + (G + 1) * (int64_t)sizeof(int64_t));
    p.bytes = p.part + (tree_grid(G, p.rbs, p.nb, T, num_sms) + G * p.rbs) * (int64_t)(tr_part_floats(p.nb) * sizeof(float));
    return p;
}

}  // namespace

bool tree_supported(int d, int m, int pw, int vpw)
{
    if (d != kTrD || m % 64 || m < 64 || m > 512) return false;
    if (!(pw == 0 || pw == 1 || pw == 2 || pw == 3 || pw == 4 || pw == 8)) return false;
    return vpw == 1 || vpw == 2 || vpw == 3 || vpw == 4 || vpw == 8;
}

size_t tree_workspace_bytes(int64_t G, int rows, int64_t T, int m, bool two, int num_sms)
{
    return (size_t)tree_plan(G, rows, T, m, two, num_sms).bytes;
}

cudaError_t launch_tree(const TreeArgs &in, const QuantTables &tk, const QuantTables &tv, void *workspace, cudaStream_t st)
{
    TreeArgs a = in;
    const Plan p = tree_plan(a.G, a.rows, a.T, a.m, a.pw != 0, a.num_sms);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.nb = p.nb; a.rbs = p.rbs; a.kb = p.kb;
    a.wsQ = ws + p.q;
    a.wsC = reinterpret_cast<float *>(ws + p.c);
    a.off = reinterpret_cast<int64_t *>(ws + p.off);
    a.part = reinterpret_cast<float *>(ws + p.part);
    // value centroids as c 2^-e, below 1: times a norm of at most 65504 they fit fp16
    float top = 0.0f;
    for (int i = 0; i < tv.levels; ++i) top = std::fmax(top, std::fabs(tv.centroid[i]));
    int e = 0;
    std::frexp(top, &e);
    e = e < -100 ? -100 : e;
    a.vdown = std::ldexp(1.0f, -e);
    a.vup = std::ldexp(1.0f / (float)kTrD, e);
    const int grid = (int)tree_grid(a.G, a.rbs, a.nb, a.T, a.num_sms);
    if (grid > 0) {
        tree_prologue_kernel<<<dim3((unsigned)(a.G * a.rbs * (a.nb / 32)), (unsigned)(a.kb / 64)), 128, 0, st>>>(a, tk);
        note_launch("tree_prologue_kernel");
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        e = a.nb == 32 ? launch_nb<32>(a, tk, tv, grid, st)
                       : a.nb == 64 ? launch_nb<64>(a, tk, tv, grid, st) : launch_nb<128>(a, tk, tv, grid, st);
        if (e != cudaSuccess) return e;
    }
    const dim3 cgrid((unsigned)((a.rows + kTrCombineRows - 1) / kTrCombineRows), (unsigned)a.G);
    const size_t smem = (size_t)kTrCombineRows * a.nodes * sizeof(float);
    if (smem > 32768) {
        const cudaError_t e = cudaFuncSetAttribute(tree_combine_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    if (grid > 0) {
        const cudaError_t e = launch_early(tree_combine_kernel, cgrid, kTrCombineThreads, smem, st, a, tv, grid);
        if (e != cudaSuccess) return e;
    } else {
        tree_combine_kernel<<<cgrid, kTrCombineThreads, smem, st>>>(a, tv, grid);
    }
    note_launch("tree_combine_kernel");
    return cudaGetLastError();
}

}  // namespace rq

// rq_cache_ops.h -- internal launch interface of the decode-side cache operators: rotary positions, tree attention
// over the compressed cache, eviction by accumulated attention weight.
#pragma once
#include "rq_kernels.h"

namespace rq {

// Rotary positions (rq_rotary.cu).
struct RotaryTensor {
    const uint16_t *in;        // nullptr: absent (n_heads2 = 0)
    uint16_t *out;
    int64_t in_batch, in_token, in_head, out_batch, out_token, out_head;   // strides in elements
};
constexpr int kMaxRot = 512;
struct RotaryArgs {
    RotaryTensor x, x2;
    int n_heads, n_heads2;
    int64_t B, n_tok;
    int d, rot;
    bool bf16, half, inverse, copy;    // copy: the d - rot unrotated values have to be written
    const int64_t *positions;
    int64_t pos_batch_stride;
    float scale;
    int num_sms;
    int items, hs, tb, heads_per_block;   // launch shape (set by launch_rotary)
    uint64_t turns[kMaxRot / 2];       // freq_i / 2 pi modulo 1, 0.64 fixed point
};
cudaError_t launch_rotary(const RotaryArgs &a, cudaStream_t st);

// Eviction from a cache by accumulated attention weight (rq_evict.cu).
struct AccumulateArgs {
    const float *scores;       // [G][nq][T]
    int64_t G, T;
    int nq;
    const int32_t *row_len;    // [G][nq] or nullptr
    float scale, decay;
    const float *acc;          // [G][T]
    float *out;
    float *workspace;
    int num_sms;
};
size_t accumulate_workspace_bytes(int64_t G, int nq, int64_t T);
cudaError_t launch_accumulate(const AccumulateArgs &a, cudaStream_t st);
struct SelectArgs {
    const float *acc;          // [G][T]
    int64_t G, T;
    const int32_t *len;        // [G] or nullptr
    int keep, n_sink, n_recent;
    int32_t *idx;              // [G][keep]
    int32_t *count;            // [G]
    int num_sms;
};
cudaError_t launch_select(const SelectArgs &a, cudaStream_t st);
constexpr int kMaxRowArrays = 16;
struct GatherArgs {
    const int32_t *idx, *count;
    int64_t G, T, T_dst;
    int keep, n_arrays;
    const uint8_t *src[kMaxRowArrays];
    uint8_t *dst[kMaxRowArrays];
    int64_t row_bytes[kMaxRowArrays];
};
cudaError_t launch_gather(const GatherArgs &a, cudaStream_t st);

// Attention of drafted tokens over the compressed cache (qjl_tree.cuh).
struct rq_strides_t { int64_t batch, token, head; };
struct TreeArgs {
    const uint16_t *q, *k_new, *v_new;     // bf16 [B][nodes][kv_heads rep or kv_heads][128]
    uint16_t *out;
    rq_strides_t qs, ks, vs, os;           // strides in elements
    int64_t B, G, T;
    int kv_heads, rep, nodes, rows;        // rows = nodes rep of a group
    const uint64_t *mask;                  // [nodes][words], batch b at mask + b mask_batch; nullptr: a chain
    int64_t mask_batch;
    int m;
    const uint16_t *proj;
    bool proj_bf16;
    const uint8_t *signs;                  // [G][T][m/8]
    const uint16_t *sk_norms;
    const int32_t *kv_len;                 // [G] or nullptr
    const uint8_t *codes;                  // first-stage codes, with norms (pw = 0: pure sketch keys)
    const uint16_t *norms;
    int pw;
    const uint8_t *vcodes;
    const uint16_t *vnorms;
    int vpw;
    float qscale;                          // softmax scale in units of log2
    int num_sms;
    // set by tree_plan / launch_tree
    int nb, rbs, kb;                       // query rows a block, row blocks a group, score operand width
    uint8_t *wsQ;                          // operand images [G rbs][kb / 64][nb][128 B]
    float *wsC;                            // [1 + kb / 32][G rbs][nb]: 2^e qscale of the rows, then sums of 32 operand coordinates
    int64_t *off;                          // [G + 1] prefix sums of the groups' tiles
    float *part;
    float vdown, vup;                      // 2^-e of the value centroids, and 2^e / d
};
constexpr int kTreeMaxNodes = 1024;
bool tree_supported(int d, int m, int pw, int vpw);
size_t tree_workspace_bytes(int64_t G, int rows, int64_t T, int m, bool two, int num_sms);
cudaError_t launch_tree(const TreeArgs &a, const QuantTables &tk, const QuantTables &tv, void *workspace, cudaStream_t st);

}  // namespace rq

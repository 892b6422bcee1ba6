// Parameters and launchers of the decoding calls' kernels (cache layout: see w4.h).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace w4 {

struct KvCache {
    void* k;
    void* v;
    const float* k_scale;    // [heads] (E4M3) or null
    const float* v_scale;
    int64_t pages;
    int layers, heads, dim, page_blocks;   // page_blocks: 16-token blocks a page
    bool e4m3;
};

struct KvAppendParams {
    const uint16_t* q;       // [T, hq, dim] rows q_stride apart, or null
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_stride, k_stride, v_stride;
    int T, hq;
    KvCache cache;
    const int32_t* slots;
    const float* rope;       // [rope_rows, rot] or null
    int64_t rope_rows;
    int rot, interleaved;
    const int32_t* positions;
    const float* q_norm;
    const float* k_norm;
    float eps;
    uint16_t* Q;
};
hipError_t launch_kv_append(const KvAppendParams& p, hipStream_t stream);

struct KvMoveParams {
    KvCache cache;
    const int32_t* page_table;
    int64_t table_pages;
    const int32_t* base;
    const int32_t* path;
    int64_t path_len;
    const int32_t* count;
    int B;
};
hipError_t launch_kv_move(const KvMoveParams& p, hipStream_t stream);

struct AttentionParams {
    const uint16_t* q;       // [T, hq, dim] rows q_stride apart
    int64_t q_stride;
    int64_t T;
    int hq;
    KvCache cache;
    const int32_t* page_table;
    int64_t table_pages;
    const int32_t* kv_len;
    const int32_t* q_start;
    int B, max_q, max_kv;
    const uint64_t* tree;
    int tree_words;
    const int32_t* positions;
    int window;              // 0: none
    float scale;
    uint16_t* O;
    float* ws;               // split partials (see attention.hip)
};
hipError_t launch_attention(const AttentionParams& p, hipStream_t stream);
size_t attention_workspace_bytes(int64_t T, int64_t B, int hq, int hk, int dim, bool e4m3, int64_t max_q,
                                 int64_t max_kv, int64_t window);

struct SampleParams {
    const void* logits;
    bool f32;
    int B, V;
    int64_t row_stride;
    const float* u;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* tokens;
    float* probs;
};
hipError_t launch_sample(const SampleParams& p, hipStream_t stream);

}  // namespace w4

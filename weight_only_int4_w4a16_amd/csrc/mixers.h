// Arguments and launchers of the token mixers: page tables, paged cache writes, paged attention, linear
// attention, the gated delta rule, and the cache with a scale for each block of tokens and head. The entry points have
// checked every argument before a launcher sees it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a16 {

struct PageTablesArgs {
    const int32_t *ctx_lens, *new_lens;
    int32_t *page_table;
    const int32_t *free_pages;
    int32_t *seq_lens, *cu_new, *slot_map, *positions, *counts;
    int64_t row_stride;
    int32_t B, max_pages, num_free, page_size, max_tokens;
};

struct KvWriteArgs {
    const void *x[2];              // keys, values
    int64_t ld[2], hs[2];          // token and head strides, elements
    void *cache[2];
    int64_t page[2], slot[2], head[2];   // cache strides, elements
    const float *scale[2];         // e4m3: float[heads] or null
    const int32_t *slot_map;
    int32_t T, heads, dim, page_size, num_pages;
    int32_t e4m3, fp16;
};

struct AttentionArgs {
    const void *q;
    const void *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *table, *lens;
    void *out;
    float *lse;
    float *work;                   // partial results
    int64_t ldq, hsq, ldo, hso, row_stride;
    int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;
    int32_t B, Hq, Hkv, dim, num_pages, page_size, max_pages, window;
    int32_t type, e4m3;
    float scale;
};

struct LinearArgs {
    const void *q, *k, *v;
    const float *g;
    const int32_t *cu;             // packed form: sequence starts, or null; step: state slots or null
    const float *state_in;
    float *state_out;
    void *out;
    float *work;
    int64_t ldq, hsq, ldk, hsk, ldv, hsv, ldg, hsg, ldo, hso;
    int32_t T, B, Hk, H, Dk, Dv, num_states;
    int32_t type;
    float scale;
};

struct DeltaArgs : LinearArgs {
    const float *beta;
    int64_t ldb, hsb;
};

// A cache of 8-bit codes and its scales (keys, values); strides of scales: page, block, head.
struct QuantizedCache {
    uint8_t *codes[2];
    int64_t page[2], slot[2], head[2];
    float *scale[2];
    int64_t scale_page[2], scale_block[2], scale_head[2];
    int32_t num_pages, page_size, heads, dim, block;
    int32_t int8;
};

struct QuantizedRowsArgs {   // rows to or from the slots of a cache
    QuantizedCache c;
    void *x[2];
    int64_t ld[2], hs[2];
    const int32_t *slot_map;
    int32_t T, fp16;
};

struct QuantizedAttentionArgs : AttentionArgs {
    int64_t k_scale_page, k_scale_block, k_scale_head, v_scale_page, v_scale_block, v_scale_head;
    int32_t block, int8;
};

hipError_t launch_page_tables(const PageTablesArgs &a, hipStream_t stream);
hipError_t launch_kv_write(const KvWriteArgs &a, int cus, hipStream_t stream);
hipError_t launch_attention(const AttentionArgs &a, int cus, hipStream_t stream);
hipError_t launch_linear(const LinearArgs &a, hipStream_t stream);
hipError_t launch_linear_step(const LinearArgs &a, hipStream_t stream);
hipError_t launch_delta(const DeltaArgs &a, hipStream_t stream);
hipError_t launch_delta_step(const DeltaArgs &a, hipStream_t stream);
hipError_t launch_quantized_write(const QuantizedRowsArgs &a, hipStream_t stream);
hipError_t launch_quantized_read(const QuantizedRowsArgs &a, int cus, hipStream_t stream);
hipError_t launch_quantized_attention(const QuantizedAttentionArgs &a, int cus, hipStream_t stream);

int64_t attention_workspace(int32_t Hq, int32_t heads, int32_t dim);
// Most units of work of one request and head.
int64_t attention_units(int32_t max_pages, int32_t page_size);
int64_t linear_workspace(int32_t T, int32_t num_seqs, int32_t H, int32_t Dk, int32_t Dv);
int64_t delta_workspace(int32_t T, int32_t num_seqs, int32_t H);

}  // namespace w4a16

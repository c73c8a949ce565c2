// C ABI of the token mixers (declared in include/w4a16.h): host-side validation and dispatch.
// Nothing here allocates device or host memory.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "device.h"
#include "mixers.h"
#include "w4a16.h"

using namespace w4a16;

namespace {

constexpr int32_t kMaxRequests = 16384;   // both running sums of a step fit in LDS
constexpr int32_t kMaxGrid = 65535;
constexpr int32_t kMaxHeads = 1 << 26;    // heads of all sequences, with a work-group for every 16 columns

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
bool strided8(int64_t a, int64_t b) { return a % 8 == 0 && b % 8 == 0; }
w4a16_status_t done(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_LAUNCH; }

// `count` int32 values from `p` share memory with rows of `width` values, `stride` apart, from `base`.
bool in_rows(const int32_t *p, int64_t count, const int32_t *base, int64_t rows, int64_t stride, int64_t width)
{
    const int64_t lo = ((int64_t)(uintptr_t)p - (int64_t)(uintptr_t)base) / 4, hi = lo + count;
    const int64_t row = lo < width ? 0 : (lo - width) / stride + 1;   // the first one that ends behind lo
    return p && count > 0 && row < rows && row * stride < hi;
}
bool shared(const int32_t *p, int64_t count, const int32_t *q, int64_t other)
{
    return q && other > 0 && in_rows(p, count, q, 1, other, other);
}

// What every call asks of a cache; `type` is that of the activations.
w4a16_status_t check_cache(const w4a16_paged_cache_t *c, int32_t type)
{
    if (!c || !c->k || !c->v)
        return W4A16_ERR_NULL_POINTER;
    if (c->type != type && c->type != W4A16_E4M3)
        return W4A16_ERR_BAD_TYPE;
    if (c->num_pages < 1 || c->page_size < 1 || c->heads < 1 || c->heads > kMaxGrid ||
        (int64_t)c->num_pages * c->page_size > 0x7FFFFFFFLL)
        return W4A16_ERR_BAD_SHAPE;
    const int64_t unit = c->type == W4A16_E4M3 ? 16 : 8;   // elements of 16 bytes
    for (int i = 0; i < 3; ++i)
        if (c->k_stride[i] % unit || c->v_stride[i] % unit)
            return W4A16_ERR_MISALIGNED;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return W4A16_ERR_MISALIGNED;
    return W4A16_OK;
}

bool known_linear(int32_t Hk, int32_t H, int32_t Dk, int32_t Dv)
{
    return H >= 1 && H <= kMaxGrid / 2 && Hk >= 1 && H % Hk == 0 && (Dk == 64 || Dk == 128) &&
           (Dv == 64 || Dv == 128);
}

w4a16_status_t check_linear(const LinearArgs &a)
{
    if (a.T > 0 && (!a.q || !a.k || !a.v || !a.g || !a.out))
        return W4A16_ERR_NULL_POINTER;
    if (a.type != W4A16_BF16 && a.type != W4A16_FP16)
        return W4A16_ERR_BAD_TYPE;
    if (!known_linear(a.Hk, a.H, a.Dk, a.Dv) || !isfinite(a.scale))
        return W4A16_ERR_BAD_SHAPE;
    for (int64_t ld : {a.ldq, a.ldk, a.ldv, a.ldg, a.ldo})   // a chunk's rows lie within 32-bit offsets
        if (ld < 0 || ld >= 1 << 24)
            return W4A16_ERR_BAD_SHAPE;
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.out, 16) ||
        !aligned(a.g, 4) || !aligned(a.cu, 4) || !aligned(a.state_in, 16) || !aligned(a.state_out, 16) ||
        !strided8(a.ldq, a.hsq) || !strided8(a.ldk, a.hsk) || !strided8(a.ldv, a.hsv) ||
        !strided8(a.ldo, a.hso))
        return W4A16_ERR_MISALIGNED;
    return W4A16_OK;
}

// What every call asks of a cache with a scale for each block.
w4a16_status_t check_quantized(const w4a16_quantized_cache_t *c)
{
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale)
        return W4A16_ERR_NULL_POINTER;
    if (c->type != W4A16_INT8 && c->type != W4A16_E4M3)
        return W4A16_ERR_BAD_TYPE;
    if (c->num_pages < 1 || c->page_size < 1 || c->heads < 1 || c->heads > kMaxGrid ||
        (int64_t)c->num_pages * c->page_size > 0x7FFFFFFFLL || c->block < 16 || c->block > 64 || c->block % 16 ||
        c->page_size % c->block || (c->dim != 64 && c->dim != 96 && c->dim != 128 && c->dim != 192 && c->dim != 256))
        return W4A16_ERR_BAD_SHAPE;
    for (int64_t slot : {c->k_stride[1], c->v_stride[1]})   // a block's rows lie within 32-bit offsets
        if (slot < 0 || slot >= 1 << 24)
            return W4A16_ERR_BAD_SHAPE;
    for (int i = 0; i < 3; ++i)
        if (c->k_stride[i] % 16 || c->v_stride[i] % 16)
            return W4A16_ERR_MISALIGNED;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return W4A16_ERR_MISALIGNED;
    return W4A16_OK;
}

QuantizedCache codes_of(const w4a16_quantized_cache_t &c)
{
    return {{(uint8_t *)c.k, (uint8_t *)c.v}, {c.k_stride[0], c.v_stride[0]}, {c.k_stride[1], c.v_stride[1]},
            {c.k_stride[2], c.v_stride[2]}, {c.k_scale, c.v_scale}, {c.k_scale_stride[0], c.v_scale_stride[0]},
            {c.k_scale_stride[1], c.v_scale_stride[1]}, {c.k_scale_stride[2], c.v_scale_stride[2]}, c.num_pages,
            c.page_size, c.heads, c.dim, c.block, c.type == W4A16_INT8};
}

// Rows that go to or come from the slots of such a cache.
w4a16_status_t check_rows(const void *k, int64_t ldk, int64_t hsk, const void *v, int64_t ldv, int64_t hsv,
                          int32_t T, int32_t type, const int32_t *slot_map, const w4a16_quantized_cache_t *cache)
{
    if (T > 0 && (!k || !v || !slot_map))
        return W4A16_ERR_NULL_POINTER;
    if (type != W4A16_BF16 && type != W4A16_FP16)
        return W4A16_ERR_BAD_TYPE;
    const w4a16_status_t st = check_quantized(cache);
    if (st != W4A16_OK)
        return st;
    if (T < 0 || (int64_t)T * cache->heads > 1LL << 35)
        return W4A16_ERR_BAD_SHAPE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 4) || !strided8(ldk, hsk) || !strided8(ldv, hsv))
        return W4A16_ERR_MISALIGNED;
    return current_device() ? W4A16_OK : W4A16_ERR_UNSUPPORTED_DEVICE;
}

w4a16_status_t check_delta(const DeltaArgs &a)
{
    if (a.T > 0 && !a.beta)
        return W4A16_ERR_NULL_POINTER;
    const w4a16_status_t st = check_linear(a);
    if (st != W4A16_OK)
        return st;
    if (a.ldb < 0 || a.ldb >= 1 << 24)
        return W4A16_ERR_BAD_SHAPE;
    return aligned(a.beta, 4) ? W4A16_OK : W4A16_ERR_MISALIGNED;
}

}  // namespace

extern "C" {

w4a16_status_t w4a16_page_tables(const int32_t *ctx_lens, const int32_t *new_lens, int32_t B,
                                 int32_t *page_table, int64_t row_stride, int32_t max_pages,
                                 const int32_t *free_pages, int32_t num_free, int32_t page_size,
                                 int32_t max_tokens, int32_t *seq_lens, int32_t *cu_new,
                                 int32_t *slot_map, int32_t *positions, int32_t *counts,
                                 hipStream_t stream)
{
    if (!ctx_lens || !new_lens || !page_table || !seq_lens || !cu_new || !counts ||
        (num_free > 0 && !free_pages) || (max_tokens > 0 && (!slot_map || !positions)))
        return W4A16_ERR_NULL_POINTER;
    if (B < 1 || B > kMaxRequests || max_pages < 1 || row_stride < max_pages || num_free < 0 ||
        page_size < 1 || page_size > 65536 || max_tokens < 0)
        return W4A16_ERR_BAD_SHAPE;
    for (const void *p : {(const void *)ctx_lens, (const void *)new_lens, (const void *)page_table,
                          (const void *)free_pages, (const void *)seq_lens, (const void *)cu_new,
                          (const void *)slot_map, (const void *)positions, (const void *)counts})
        if (!aligned(p, 4))
            return W4A16_ERR_MISALIGNED;
    if (!current_device())
        return W4A16_ERR_UNSUPPORTED_DEVICE;
    // Work-groups read the inputs while others write: nothing that is written may be read, or written twice.
    const struct { const int32_t *p; int64_t n; } own[] = {{seq_lens, B}, {cu_new, (int64_t)B + 1}, {counts, 2},
        {slot_map, max_tokens}, {positions, max_tokens}, {ctx_lens, B}, {new_lens, B}, {free_pages, num_free}};
    for (int i = 0; i < 8; ++i) {
        if (in_rows(own[i].p, own[i].n, page_table, B, row_stride, max_pages))
            return W4A16_ERR_OVERLAP;
        for (int j = i + 1; i < 5 && j < 8; ++j)
            if (shared(own[i].p, own[i].n, own[j].p, own[j].n))
                return W4A16_ERR_OVERLAP;
    }
    PageTablesArgs a{ctx_lens, new_lens, page_table, free_pages, seq_lens, cu_new, slot_map, positions,
                     counts, row_stride, B, max_pages, num_free, page_size, max_tokens};
    return done(launch_page_tables(a, stream));
}

w4a16_status_t w4a16_paged_kv_write(const void *k, int64_t ldk, int64_t hsk, const void *v,
                                    int64_t ldv, int64_t hsv, int32_t T, int32_t type,
                                    const int32_t *slot_map, const w4a16_paged_cache_t *cache,
                                    hipStream_t stream)
{
    if (T > 0 && (!k || !v || !slot_map))
        return W4A16_ERR_NULL_POINTER;
    if (type != W4A16_BF16 && type != W4A16_FP16)
        return W4A16_ERR_BAD_TYPE;
    const w4a16_status_t st = check_cache(cache, type);
    if (st != W4A16_OK)
        return st;
    if (T < 0 || cache->dim < 16 || cache->dim > 1024 || cache->dim % 16)
        return W4A16_ERR_BAD_SHAPE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 4) || !strided8(ldk, hsk) ||
        !strided8(ldv, hsv))
        return W4A16_ERR_MISALIGNED;
    const DeviceInfo *dev = current_device();
    if (!dev)
        return W4A16_ERR_UNSUPPORTED_DEVICE;
    if (T == 0)
        return W4A16_OK;
    KvWriteArgs a{{k, v}, {ldk, ldv}, {hsk, hsv}, {cache->k, cache->v},
                  {cache->k_stride[0], cache->v_stride[0]}, {cache->k_stride[1], cache->v_stride[1]},
                  {cache->k_stride[2], cache->v_stride[2]}, {cache->k_scale, cache->v_scale}, slot_map,
                  T, cache->heads, cache->dim, cache->page_size, cache->num_pages,
                  cache->type == W4A16_E4M3, type == W4A16_FP16};
    return done(launch_kv_write(a, dev->cus, stream));
}

int64_t w4a16_paged_attention_workspace(int32_t Hq, int32_t heads, int32_t dim)
{
    if (heads < 1 || Hq < 1 || Hq > kMaxGrid || Hq % heads ||
        (dim != 64 && dim != 96 && dim != 128 && dim != 192 && dim != 256))
        return 0;
    return attention_workspace(Hq, heads, dim);
}

w4a16_status_t w4a16_paged_attention(const void *q, int64_t ldq, int64_t hsq, int32_t type,
                                     const w4a16_paged_cache_t *cache, const int32_t *page_table,
                                     int64_t row_stride, int32_t max_pages,
                                     const int32_t *seq_lens, int32_t B, int32_t Hq, float scale,
                                     int32_t window, void *out, int64_t ldo, int64_t hso,
                                     float *lse, void *workspace, int64_t workspace_bytes,
                                     hipStream_t stream)
{
    if (B > 0 && (!q || !page_table || !seq_lens || !out || !workspace))
        return W4A16_ERR_NULL_POINTER;
    if (type != W4A16_BF16 && type != W4A16_FP16)
        return W4A16_ERR_BAD_TYPE;
    const w4a16_status_t st = check_cache(cache, type);
    if (st != W4A16_OK)
        return st;
    const int64_t need = w4a16_paged_attention_workspace(Hq, cache->heads, cache->dim);
    if (B < 0 || B > kMaxGrid || need == 0 || max_pages < 1 || row_stride < max_pages || window < 0 ||
        (int64_t)max_pages * cache->page_size > 0x7FFFFFFFLL || !isfinite(scale))
        return W4A16_ERR_BAD_SHAPE;
    const int64_t share = Hq / cache->heads, units = attention_units(max_pages, cache->page_size);
    if (units * B > 0x7FFFFFFFLL / (cache->heads * ((share + 15) / 16)))
        return W4A16_ERR_BAD_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(lse, 4) || !aligned(workspace, 16) || !strided8(ldq, hsq) || !strided8(ldo, hso))
        return W4A16_ERR_MISALIGNED;
    if (workspace_bytes < need && B > 0)
        return W4A16_ERR_WORKSPACE;
    const DeviceInfo *dev = current_device();
    if (!dev)
        return W4A16_ERR_UNSUPPORTED_DEVICE;
    if (B == 0)
        return W4A16_OK;
    AttentionArgs a{q, cache->k, cache->v, cache->k_scale, cache->v_scale, page_table, seq_lens, out, lse,
                    (float *)workspace, ldq, hsq, ldo, hso, row_stride, cache->k_stride[0],
                    cache->k_stride[1], cache->k_stride[2], cache->v_stride[0], cache->v_stride[1],
                    cache->v_stride[2], B, Hq, cache->heads, cache->dim, cache->num_pages,
                    cache->page_size, max_pages, window, type, cache->type == W4A16_E4M3, scale};
    return done(launch_attention(a, dev->cus, stream));
}

int64_t w4a16_linear_attention_workspace(int32_t T, int32_t num_seqs, int32_t H, int32_t Dk,
                                         int32_t Dv)
{
    if (T < 0 || T > 0x7FFFFFFF - 64 || num_seqs < 1 || num_seqs > kMaxRequests ||
        !known_linear(1, H, Dk, Dv))
        return -1;
    return linear_workspace(T, num_seqs, H, Dk, Dv);
}

w4a16_status_t w4a16_linear_attention(const void *q, int64_t ldq, int64_t hsq, const void *k,
                                      int64_t ldk, int64_t hsk, const void *v, int64_t ldv,
                                      int64_t hsv, const float *log_decay, int64_t ldg, int64_t hsg,
                                      const int32_t *cu_seqlens, int32_t num_seqs, int32_t T,
                                      int32_t Hk, int32_t H, int32_t Dk, int32_t Dv, int32_t type,
                                      float scale, const float *state_in, float *state_out,
                                      void *out, int64_t ldo, int64_t hso, void *workspace,
                                      int64_t workspace_bytes, hipStream_t stream)
{
    LinearArgs a{q, k, v, log_decay, cu_seqlens, state_in, state_out, out, (float *)workspace, ldq, hsq,
                 ldk, hsk, ldv, hsv, ldg, hsg, ldo, hso, T, num_seqs, Hk, H, Dk, Dv, num_seqs, type,
                 scale};
    const int64_t need = w4a16_linear_attention_workspace(T, num_seqs, H, Dk, Dv);
    if (need < 0 || (!cu_seqlens && num_seqs != 1))
        return W4A16_ERR_BAD_SHAPE;
    const w4a16_status_t st = state_out ? check_linear(a) : W4A16_ERR_NULL_POINTER;
    if (st != W4A16_OK)
        return st;
    if (need > 0 && !workspace)
        return W4A16_ERR_NULL_POINTER;
    if (!aligned(workspace, 16))
        return W4A16_ERR_MISALIGNED;
    if (workspace_bytes < need)
        return W4A16_ERR_WORKSPACE;
    if (!current_device())
        return W4A16_ERR_UNSUPPORTED_DEVICE;
    return done(launch_linear(a, stream));
}

w4a16_status_t w4a16_linear_attention_step(const void *q, int64_t ldq, int64_t hsq, const void *k,
                                           int64_t ldk, int64_t hsk, const void *v, int64_t ldv,
                                           int64_t hsv, const float *log_decay, int64_t ldg,
                                           int64_t hsg, const int32_t *slots, int32_t num_states,
                                           int32_t B, int32_t Hk, int32_t H, int32_t Dk, int32_t Dv,
                                           int32_t type, float scale, const float *state_in,
                                           float *state_out, void *out, int64_t ldo, int64_t hso,
                                           hipStream_t stream)
{
    LinearArgs a{q, k, v, log_decay, slots, state_in, state_out, out, nullptr, ldq, hsq, ldk, hsk, ldv,
                 hsv, ldg, hsg, ldo, hso, B, B, Hk, H, Dk, Dv, num_states, type, scale};
    const w4a16_status_t st =
        num_states > 0 && (!state_in || !state_out) ? W4A16_ERR_NULL_POINTER : check_linear(a);
    if (st != W4A16_OK)
        return st;
    if (B < 0 || B > kMaxGrid || num_states < 0 || (!slots && num_states < B))
        return W4A16_ERR_BAD_SHAPE;
    if (!current_device())
        return W4A16_ERR_UNSUPPORTED_DEVICE;
    if (B == 0)
        return W4A16_OK;
    return done(launch_linear_step(a, stream));
}

w4a16_status_t w4a16_quantized_kv_write(const void *k, int64_t ldk, int64_t hsk, const void *v, int64_t ldv,
                                        int64_t hsv, int32_t T, int32_t type, const int32_t *slot_map,
                                        const w4a16_quantized_cache_t *cache, hipStream_t stream)
{
    const w4a16_status_t st = check_rows(k, ldk, hsk, v, ldv, hsv, T, type, slot_map, cache);
    if (st != W4A16_OK || T == 0)
        return st;
    const QuantizedRowsArgs a{codes_of(*cache), {(void *)k, (void *)v}, {ldk, ldv}, {hsk, hsv}, slot_map, T,
                              type == W4A16_FP16};
    return done(launch_quantized_write(a, stream));
}

w4a16_status_t w4a16_quantized_kv_read(const w4a16_quantized_cache_t *cache, const int32_t *slot_map, int32_t T,
                                       int32_t type, void *k, int64_t ldk, int64_t hsk, void *v, int64_t ldv,
                                       int64_t hsv, hipStream_t stream)
{
    const w4a16_status_t st = check_rows(k, ldk, hsk, v, ldv, hsv, T, type, slot_map, cache);
    if (st != W4A16_OK || T == 0)
        return st;
    const QuantizedRowsArgs a{codes_of(*cache), {k, v}, {ldk, ldv}, {hsk, hsv}, slot_map, T, type == W4A16_FP16};
    return done(launch_quantized_read(a, current_device()->cus, stream));
}

int64_t w4a16_quantized_attention_workspace(int32_t Hq, int32_t heads, int32_t dim)
{
    return w4a16_paged_attention_workspace(Hq, heads, dim);
}

w4a16_status_t w4a16_quantized_attention(const void *q, int64_t ldq, int64_t hsq, int32_t type,
                                         const w4a16_quantized_cache_t *cache, const int32_t *page_table,
                                         int64_t row_stride, int32_t max_pages, const int32_t *seq_lens, int32_t B,
                                         int32_t Hq, float scale, int32_t window, void *out, int64_t ldo,
                                         int64_t hso, float *lse, void *workspace, int64_t workspace_bytes,
                                         hipStream_t stream)
{
    if (B > 0 && (!q || !page_table || !seq_lens || !out || !workspace))
        return W4A16_ERR_NULL_POINTER;
    if (type != W4A16_BF16 && type != W4A16_FP16)
        return W4A16_ERR_BAD_TYPE;
    const w4a16_status_t st = check_quantized(cache);
    if (st != W4A16_OK)
        return st;
    const int64_t need = w4a16_quantized_attention_workspace(Hq, cache->heads, cache->dim);
    if (B < 0 || B > kMaxGrid || need == 0 || max_pages < 1 || row_stride < max_pages || window < 0 ||
        (int64_t)max_pages * cache->page_size > 0x7FFFFFFFLL || !isfinite(scale))
        return W4A16_ERR_BAD_SHAPE;
    const int64_t share = Hq / cache->heads, units = attention_units(max_pages, cache->page_size);
    if (units * B > 0x7FFFFFFFLL / (cache->heads * ((share + 15) / 16)))
        return W4A16_ERR_BAD_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(lse, 4) || !aligned(workspace, 16) || !strided8(ldq, hsq) || !strided8(ldo, hso))
        return W4A16_ERR_MISALIGNED;
    if (workspace_bytes < need && B > 0)
        return W4A16_ERR_WORKSPACE;
    const DeviceInfo *dev = current_device();
    if (!dev)
        return W4A16_ERR_UNSUPPORTED_DEVICE;
    if (B == 0)
        return W4A16_OK;
    QuantizedAttentionArgs a{};
    static_cast<AttentionArgs &>(a) = {q, cache->k, cache->v, cache->k_scale, cache->v_scale, page_table, seq_lens,
                                       out, lse, (float *)workspace, ldq, hsq, ldo, hso, row_stride,
                                       cache->k_stride[0], cache->k_stride[1], cache->k_stride[2],
                                       cache->v_stride[0], cache->v_stride[1], cache->v_stride[2], B, Hq,
                                       cache->heads, cache->dim, cache->num_pages, cache->page_size, max_pages,
                                       window, type, 0, scale};
    a.k_scale_page = cache->k_scale_stride[0];
    a.k_scale_block = cache->k_scale_stride[1];
    a.k_scale_head = cache->k_scale_stride[2];
    a.v_scale_page = cache->v_scale_stride[0];
    a.v_scale_block = cache->v_scale_stride[1];
    a.v_scale_head = cache->v_scale_stride[2];
    a.block = cache->block;
    a.int8 = cache->type == W4A16_INT8;
    return done(launch_quantized_attention(a, dev->cus, stream));
}

int64_t w4a16_delta_rule_workspace(int32_t T, int32_t num_seqs, int32_t H, int32_t Dk, int32_t Dv, int32_t type)
{
    if (T < 0 || T > 0x7FFFFFFF - 64 || num_seqs < 1 || num_seqs > kMaxRequests || !known_linear(1, H, Dk, Dv) ||
        (int64_t)num_seqs * H > kMaxHeads || (type != W4A16_BF16 && type != W4A16_FP16))
        return -1;
    return delta_workspace(T, num_seqs, H);
}

w4a16_status_t w4a16_delta_rule(const void *q, int64_t ldq, int64_t hsq, const void *k, int64_t ldk, int64_t hsk,
                                const void *v, int64_t ldv, int64_t hsv, const float *log_decay, int64_t ldg,
                                int64_t hsg, const float *beta, int64_t ldb, int64_t hsb,
                                const int32_t *cu_seqlens, int32_t num_seqs, int32_t T, int32_t Hk, int32_t H,
                                int32_t Dk, int32_t Dv, int32_t type, float scale, const float *state_in,
                                float *state_out, void *out, int64_t ldo, int64_t hso, void *workspace,
                                int64_t workspace_bytes, hipStream_t stream)
{
    DeltaArgs a{{q, k, v, log_decay, cu_seqlens, state_in, state_out, out, (float *)workspace, ldq, hsq, ldk, hsk,
                 ldv, hsv, ldg, hsg, ldo, hso, T, num_seqs, Hk, H, Dk, Dv, num_seqs, type, scale}, beta, ldb, hsb};
    if (type != W4A16_BF16 && type != W4A16_FP16)
        return W4A16_ERR_BAD_TYPE;
    const int64_t need = w4a16_delta_rule_workspace(T, num_seqs, H, Dk, Dv, type);
    if (need < 0 || (!cu_seqlens && num_seqs != 1))
        return W4A16_ERR_BAD_SHAPE;
    const w4a16_status_t st = state_out ? check_delta(a) : W4A16_ERR_NULL_POINTER;
    if (st != W4A16_OK)
        return st;
    if (need > 0 && !workspace)
        return W4A16_ERR_NULL_POINTER;
    if (!aligned(workspace, 16))
        return W4A16_ERR_MISALIGNED;
    if (workspace_bytes < need)
        return W4A16_ERR_WORKSPACE;
    if (!current_device())
        return W4A16_ERR_UNSUPPORTED_DEVICE;
    return done(launch_delta(a, stream));
}

w4a16_status_t w4a16_delta_rule_step(const void *q, int64_t ldq, int64_t hsq, const void *k, int64_t ldk,
                                     int64_t hsk, const void *v, int64_t ldv, int64_t hsv, const float *log_decay,
                                     int64_t ldg, int64_t hsg, const float *beta, int64_t ldb, int64_t hsb,
                                     const int32_t *slots, int32_t num_states, int32_t B, int32_t Hk, int32_t H,
                                     int32_t Dk, int32_t Dv, int32_t type, float scale, const float *state_in,
                                     float *state_out, void *out, int64_t ldo, int64_t hso, hipStream_t stream)
{
    DeltaArgs a{{q, k, v, log_decay, slots, state_in, state_out, out, nullptr, ldq, hsq, ldk, hsk, ldv, hsv, ldg,
                 hsg, ldo, hso, B, B, Hk, H, Dk, Dv, num_states, type, scale}, beta, ldb, hsb};
    const w4a16_status_t st =
        num_states > 0 && (!state_in || !state_out) ? W4A16_ERR_NULL_POINTER : check_delta(a);
    if (st != W4A16_OK)
        return st;
    if (B < 0 || B > kMaxGrid || num_states < 0 || (!slots && num_states < B))
        return W4A16_ERR_BAD_SHAPE;
    if (!current_device())
        return W4A16_ERR_UNSUPPORTED_DEVICE;
    if (B == 0)
        return W4A16_OK;
    return done(launch_delta_step(a, stream));
}

}  // extern "C"

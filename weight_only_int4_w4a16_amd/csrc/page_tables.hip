// Page tables and slot maps of one step for gfx950. With c_b cached and n_b new tokens of request b
// and P(x) = min(ceil(x / page_size), max_pages), request b takes P(c_b + n_b) - P(c_b) pages off the
// free list, after those of the requests before it; a token's slot is its page times the page size
// plus its offset. The two running sums (tokens, pages) are the only thing that ties requests together.
//
// Every work-group makes both sums for all the requests itself, in LDS, and then serves its share of
// the tokens, pages and requests by searching them: one launch, and no work-group waits for another.
// A new page is taken from the free list by whoever needs it (the table's writer and the slot's), so
// no value written by this launch is read by it.
//
// Latency bounds it: 5.6 us for one token of each of 8 requests, 9.1 us for 500 prompts of 108 thousand
// tokens in all (0.9 MB), against about 2.5 us for an empty launch; the rest is dependent trips to memory
// (lengths; those of the request that was found, once more; table entry or free page; the stores), with the
// sums' barriers between.
#include "mixers.h"

namespace w4a16 {

namespace {

constexpr int kThreads = 256;
constexpr int kTokensPerThread = 4;
constexpr uint32_t kMost = 0x7FFFFFFFu;

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kMost); }

struct Lens {
    uint32_t c, n, p0, p1;   // cached and new tokens, first page to take and the one after the last
};

__device__ __forceinline__ Lens lens_of(const PageTablesArgs &a, int b)
{
    Lens r;
    r.c = (uint32_t)max(a.ctx_lens[b], 0);
    r.n = (uint32_t)max(a.new_lens[b], 0);
    const uint32_t ps = (uint32_t)a.page_size, most = (uint32_t)a.max_pages;
    const uint32_t end = r.c + r.n;   // below 2^32
    r.p0 = min(r.c ? (r.c - 1) / ps + 1 : 0u, most);
    r.p1 = min(end ? (end - 1) / ps + 1 : 0u, most);
    return r;
}

// The last request whose running sum before it is at most x (sums[0] = 0).
__device__ __forceinline__ int find(const uint32_t *sums, int B, uint32_t x)
{
    int lo = 0, hi = B;   // sums[lo] <= x, and sums[hi] > x where hi < B
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kThreads) void page_tables_kernel(PageTablesArgs a)
{
    extern __shared__ uint32_t lds[];
    uint32_t *tok = lds, *pag = lds + a.B + 1;   // [B + 1] running sums, the totals at the end
    __shared__ uint32_t wave_tok[kThreads / 64], wave_pag[kThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;

    // Each thread sums a run of requests, then the runs' sums are scanned (saturating addition of
    // values below 2^31 is associative).
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    uint32_t st = 0, sp = 0;
    for (int b = b0; b < b1; ++b) {
        const Lens r = lens_of(a, b);
        tok[b] = r.n;
        pag[b] = r.p1 - r.p0;
        st = sat_add(st, r.n);
        sp = sat_add(sp, r.p1 - r.p0);
    }
    uint32_t it = st, ip = sp;
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t ut = __shfl_up(it, d), up = __shfl_up(ip, d);
        if (lane >= d) {
            it = sat_add(it, ut);
            ip = sat_add(ip, up);
        }
    }
    if (lane == 63) {
        wave_tok[wave] = it;
        wave_pag[wave] = ip;
    }
    uint32_t bt = __shfl_up(it, 1), bp = __shfl_up(ip, 1);
    if (lane == 0)
        bt = bp = 0;
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        bt = sat_add(bt, wave_tok[w]);
        bp = sat_add(bp, wave_pag[w]);
    }
    for (int b = b0; b < b1; ++b) {
        const uint32_t n = tok[b], p = pag[b];
        tok[b] = bt;
        pag[b] = bp;
        bt = sat_add(bt, n);
        bp = sat_add(bp, p);
    }
    if (tid == kThreads - 1) {
        tok[a.B] = bt;
        pag[a.B] = bp;
    }
    __syncthreads();
    const uint32_t total = tok[a.B], pages = pag[a.B];
    const int64_t gid = (int64_t)blockIdx.x * kThreads + tid, step = (int64_t)gridDim.x * kThreads;
    const uint32_t ps = (uint32_t)a.page_size;

    if (gid == 0) {
        a.counts[0] = (int32_t)total;
        a.counts[1] = (int32_t)pages;
        a.cu_new[a.B] = (int32_t)total;
    }
    for (int64_t b = gid; b < a.B; b += step) {
        a.seq_lens[b] = (int32_t)min((uint32_t)max(a.ctx_lens[b], 0) + (uint32_t)max(a.new_lens[b], 0), kMost);
        a.cu_new[b] = (int32_t)tok[b];
    }

    // Pages: entry i of the free list goes to the request whose run of pages it lies in.
    for (int64_t i = gid; i < pages; i += step) {
        const int b = find(pag, a.B, (uint32_t)i);
        const Lens r = lens_of(a, b);
        const uint32_t j = r.p0 + ((uint32_t)i - pag[b]);
        if (j < r.p1)   // always, unless the sum has saturated
            a.page_table[b * a.row_stride + j] = i < a.num_free ? a.free_pages[i] : -1;
    }

    // Tokens, a run of neighbours per thread: one search, then a walk over the requests.
    for (int64_t t0 = gid * kTokensPerThread; t0 < a.max_tokens; t0 += step * kTokensPerThread) {
        int b = -1;
        Lens r{};
        uint32_t start = 0, end = 0, held = ~0u;
        int32_t page = -1;
        for (int e = 0; e < kTokensPerThread; ++e) {
            const int64_t t = t0 + e;
            if (t >= a.max_tokens)
                break;
            int32_t pos = -1, slot = -1;
            if (t < total) {
                if (b < 0 || t >= end) {
                    b = find(tok, a.B, (uint32_t)t);
                    r = lens_of(a, b);
                    start = tok[b];
                    end = tok[b + 1];
                    held = ~0u;
                }
                const uint32_t p = r.c + ((uint32_t)t - start);
                const uint32_t j = p / ps;
                pos = (int32_t)min(p, kMost);
                if (j != held && j < (uint32_t)a.max_pages) {
                    held = j;
                    if (j < r.p0) {
                        page = a.page_table[b * a.row_stride + j];
                    } else {
                        const uint32_t i = sat_add(pag[b], j - r.p0);
                        page = i < (uint32_t)a.num_free ? a.free_pages[i] : -1;
                    }
                }
                if (j < (uint32_t)a.max_pages && page >= 0) {
                    const uint64_t s = (uint64_t)(uint32_t)page * ps + (p - j * ps);
                    slot = s <= kMost ? (int32_t)s : -1;
                }
            }
            a.positions[t] = pos;
            a.slot_map[t] = slot;
        }
    }
}

}  // namespace

hipError_t launch_page_tables(const PageTablesArgs &a, hipStream_t stream)
{
    // One work-group per 1024 tokens, up to two per CU.
    const int64_t want = ((int64_t)a.max_tokens + kThreads * kTokensPerThread - 1) / (kThreads * kTokensPerThread);
    const int blocks = (int)(want < 1 ? 1 : want > 512 ? 512 : want);
    const size_t lds = 2 * ((size_t)a.B + 1) * sizeof(uint32_t);
    page_tables_kernel<<<dim3(blocks), dim3(kThreads), lds, stream>>>(a);
    return hipGetLastError();
}

}  // namespace w4a16

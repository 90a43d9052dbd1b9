// qsa_pages.cu -- qsa_page_map: page tables, slot maps, causal limits and
// length offsets from the sequences' lengths.
//
// A sequence of len cells holds ceil(len / P) pages.  Shrinking ones push the
// pages past their new length on the free stack, growing ones pop what they
// lack; both are prefix sums over (sequence, entry), so every page's place in
// the stack is known without atomics and equal inputs give equal tables.
//
// What bounds it is latency: a decode step touches a few KB.  One CTA does the
// bookkeeping (sequences in blocks of 1,024, a thread each; the freed and taken
// entries flattened over all threads, which find their sequence by bisection in
// the block's prefix sums), and the token maps too where they are few; larger
// maps go to a second, grid-wide launch, which starts as a programmatic
// dependent and waits for the first.
// Measured, roll back and grow again (two calls): 16 sequences, windows of 4, 6.8
// us; 300 sequences, windows to 2,048 and 5,000 pages each way, 19 us (1.6 of them
// the token maps' fences), with a list per sequence, 8 or 32 warps one sequence after
// another, 30 us.
#include "qsa_kv4.cuh"

namespace qsa {
namespace {

// Threads of the bookkeeping CTA: few sequences are bound by its barriers.
constexpr int kFewThreads = 256, kManyThreads = 1024;
// Token map entries up to which the bookkeeping CTA writes them itself.
constexpr int kInlineTokens = 4096;

struct PageParams {
    const int32_t *cur_len, *new_len;
    int32_t *page_table, *free_pages, *free_count, *out_len, *len_offsets;
    int32_t *positions, *slots, *q_limit;
    uint32_t *status;
    int32_t n_seq, max_new, P, table_len, pool_pages;
};

struct Lengths {
    int cur, target, held, want;
};

__device__ __forceinline__ int pages_of(int len, int P) { return P == 1 ? len : len / P + (len % P != 0); }

// Lengths and pages of sequence b; a bad length leaves the sequence as it is.
__device__ __forceinline__ Lengths lengths_of(const PageParams &p, int b, bool report)
{
    const int cap = p.table_len * p.P;
    int cur = p.cur_len[b], target = p.new_len[b];
    if (cur < 0 || cur > cap || target < 0 || target > cap || target - cur > p.max_new) {
        if (report && p.status) atomicOr(p.status, QSA_STATUS_BAD_EXTENT);
        cur = min(max(cur, 0), cap);
        target = cur;
    }
    return Lengths{cur, target, pages_of(cur, p.P), pages_of(target, p.P)};
}

// Inclusive scan over the CTA of one value per thread (fixed order).
template <int T>
__device__ __forceinline__ int block_scan(int v, int *s_warp, int *total)
{
    constexpr int kWarps = T / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads(); // the sums of the scan before have been read
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int w = lane < kWarps ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        if (lane < kWarps) s_warp[lane] = w;
    }
    __syncthreads();
    *total = s_warp[kWarps - 1];
    return v + (warp > 0 ? s_warp[warp - 1] : 0);
}

// Last i with s_pref[i] <= e: the sequence of the block that item e belongs to.
template <int T>
__device__ __forceinline__ int owner_of(const int *s_pref, int e)
{
    int lo = 0;
#pragma unroll
    for (int step = T / 2; step > 0; step >>= 1)
        if (s_pref[lo + step] <= e) lo += step;
    return lo;
}

// The entry of a freed page: is it a page of the pool?
__device__ __forceinline__ bool freed_page(const PageParams &p, int e, bool report)
{
    if (e >= 0 && e < p.pool_pages) return true;
    if (e != -1 && report && p.status) atomicOr(p.status, QSA_STATUS_BAD_SLOT);
    return false;
}

// Pushes the pages freed by at most T sequences if all of them are pages of the
// pool: then each one's place in the stack is known at once, and a thread has four
// loads in flight.  How many, or -1 if some entry is none; what has been written
// by then lies above the stack's top, where nothing is held.
template <int T>
__device__ __forceinline__ int push_pages(const PageParams &p, int count, int *s_warp, int *s_pref, int *s_seq)
{
    const int tid = threadIdx.x;
    int n = 0;
    if (tid < p.n_seq) {
        const Lengths l = lengths_of(p, tid, true);
        n = max(l.held - l.want, 0);
        s_seq[tid] = l.want;
    }
    if (!__syncthreads_or(n > 0)) return 0;
    int total;
    const int incl = block_scan<T>(n, s_warp, &total);
    s_pref[tid] = incl - n;
    __syncthreads();
    auto entry = [&](int e) {
        const int i = owner_of<T>(s_pref, e);
        return p.page_table + (size_t)i * p.table_len + s_seq[i] + (e - s_pref[i]);
    };
    bool ok = true;
    for (int e0 = tid; e0 < total; e0 += 4 * T) {
        int page[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (e0 + k * T < total) page[k] = *entry(e0 + k * T);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int e = e0 + k * T;
            if (e >= total) break;
            ok &= page[k] >= 0 && page[k] < p.pool_pages;
            const long long top = (long long)count + total - 1 - e;
            if (top < p.pool_pages) p.free_pages[top] = page[k];
        }
    }
    if (!__syncthreads_and(ok)) return -1;
    for (int e = tid; e < total; e += T) *entry(e) = -1;
    if (tid == 0 && (long long)count + total > p.pool_pages && p.status) atomicOr(p.status, QSA_STATUS_BAD_EXTENT);
    return total;
}

// The same for any number of sequences and entries of any kind: the pages are
// counted, then pushed.
template <int T>
__device__ __forceinline__ int push_checked(const PageParams &p, int count, int *s_warp, int *s_pref, int *s_seq)
{
    const int tid = threadIdx.x;
    int freed = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int rank0 = 0;
        for (int b0 = 0; b0 < p.n_seq; b0 += T) {
            const int b = b0 + tid;
            int n = 0, first = 0;
            if (b < p.n_seq) {
                const Lengths l = lengths_of(p, b, pass == 0);
                n = max(l.held - l.want, 0);
                first = l.want;
            }
            if (!__syncthreads_or(n > 0)) continue;
            int total;
            const int incl = block_scan<T>(n, s_warp, &total);
            s_pref[tid] = incl - n;
            s_seq[tid] = first;
            __syncthreads();
            for (int e0 = 0; e0 < total; e0 += T) {
                const int e = e0 + tid;
                int32_t *at = nullptr;
                int page = -1;
                if (e < total) {
                    const int i = owner_of<T>(s_pref, e);
                    at = p.page_table + (size_t)(b0 + i) * p.table_len + s_seq[i] + (e - s_pref[i]);
                    page = *at;
                }
                const bool ok = e < total && freed_page(p, page, pass == 0);
                int n_ok;
                const int rank = rank0 + block_scan<T>(ok ? 1 : 0, s_warp, &n_ok) - 1;
                rank0 += n_ok;
                if (pass == 1 && e < total) {
                    *at = -1;
                    const long long top = (long long)count + freed - 1 - rank;
                    if (ok && top < p.pool_pages) p.free_pages[top] = page;
                    if (ok && top >= p.pool_pages && p.status) atomicOr(p.status, QSA_STATUS_BAD_EXTENT);
                }
            }
            __syncthreads();
        }
        if (pass == 0) freed = rank0;
        // (entries of -1 alone leave nothing to push, but pass 1 goes over them too)
    }
    return freed;
}

// One free list: frees, then takes, in (sequence, entry) order.
template <int T>
__device__ void resize_shared(const PageParams &p, int *s_warp, int *s_pref, int *s_seq, int *s_take)
{
    const int tid = threadIdx.x;
    int count = min(max(p.free_count[0], 0), p.pool_pages);
    int freed = p.n_seq <= T ? push_pages<T>(p, count, s_warp, s_pref, s_seq) : -1;
    if (freed < 0) freed = push_checked<T>(p, count, s_warp, s_pref, s_seq);
    count = (int)min((long long)count + freed, (long long)p.pool_pages);
    __syncthreads(); // the pushed pages are visible to the CTA
    int taken = 0;     // pages taken so far
    int len_base = 0;  // cells of the sequences before this block
    long long asked = 0; // pages asked for so far, taken or not
    for (int b0 = 0; b0 < p.n_seq; b0 += T) {
        const int b = b0 + tid;
        Lengths l{0, 0, 0, 0};
        if (b < p.n_seq) l = lengths_of(p, b, false);
        const int need = max(l.want - l.held, 0);
        if (tid == 0) *s_take = 0;
        int total;
        const int incl = block_scan<T>(need, s_warp, &total);
        const bool served = need == 0 || asked + incl <= count;
        s_pref[tid] = incl - need;
        s_seq[tid] = l.held;
        if (served && need > 0) atomicMax(s_take, incl); // the served needs are the first ones
        const int len = served ? l.target : l.cur;
        if (!served && p.status) atomicOr(p.status, QSA_STATUS_NO_PAGES);
        int len_total;
        const int len_incl = block_scan<T>(len, s_warp, &len_total);
        if (b < p.n_seq) {
            p.out_len[b] = len;
            p.len_offsets[b + 1] = len_base + len_incl;
        }
        const int n_take = *s_take;
        for (int k0 = tid; k0 < n_take; k0 += 4 * T) { // (the four reads before the writes)
            int page[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k0 + e * T < n_take) page[e] = p.free_pages[count - 1 - taken - (k0 + e * T)];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = k0 + e * T;
                if (k >= n_take) break;
                const int i = owner_of<T>(s_pref, k);
                p.page_table[(size_t)(b0 + i) * p.table_len + s_seq[i] + (k - s_pref[i])] = page[e];
            }
        }
        taken += n_take;
        asked += total;
        len_base += len_total;
        __syncthreads();
    }
    if (tid == 0) {
        p.free_count[0] = count - taken;
        p.len_offsets[0] = 0;
    }
}

// A free list per sequence: a warp per sequence.
template <int T>
__device__ void resize_separate(const PageParams &p, int *s_warp)
{
    const int lane = threadIdx.x & 31;
    for (int b = threadIdx.x >> 5; b < p.n_seq; b += T / 32) {
        const Lengths l = lengths_of(p, b, lane == 0);
        int32_t *table = p.page_table + (size_t)b * p.table_len;
        int32_t *list = p.free_pages + (size_t)b * p.pool_pages;
        int count = min(max(p.free_count[b], 0), p.pool_pages);
        int freed = 0;
        for (int pass = 0; pass < 2 && l.want < l.held; ++pass) {
            int rank0 = 0;
            for (int e0 = l.want; e0 < l.held; e0 += 32) {
                const int e = e0 + lane;
                const int page = e < l.held ? table[e] : -1;
                const bool ok = freed_page(p, page, pass == 0);
                const unsigned m = __ballot_sync(0xffffffffu, ok);
                if (pass == 1 && e < l.held) {
                    table[e] = -1;
                    const long long top = (long long)count + freed - 1 - (rank0 + __popc(m & ((1u << lane) - 1u)));
                    if (ok && top < p.pool_pages) list[top] = page;
                    if (ok && top >= p.pool_pages && p.status) atomicOr(p.status, QSA_STATUS_BAD_EXTENT);
                }
                rank0 += __popc(m);
            }
            if (pass == 0) freed = rank0;
        }
        count = (int)min((long long)count + freed, (long long)p.pool_pages);
        const int need = max(l.want - l.held, 0);
        const bool served = need <= count;
        if (served) // (a sequence that grows has freed nothing: the list is as it was)
            for (int k = lane; k < need; k += 32) table[l.held + k] = list[count - 1 - k];
        if (lane == 0) {
            if (!served && p.status) atomicOr(p.status, QSA_STATUS_NO_PAGES);
            p.free_count[b] = count - (served ? need : 0);
            p.out_len[b] = served ? l.target : l.cur;
        }
    }
    __syncthreads();
    int base = 0;
    for (int b0 = 0; b0 < p.n_seq; b0 += T) {
        const int b = b0 + threadIdx.x;
        int total;
        const int incl = block_scan<T>(b < p.n_seq ? p.out_len[b] : 0, s_warp, &total);
        if (b < p.n_seq) p.len_offsets[b + 1] = base + incl;
        base += total;
    }
    if (threadIdx.x == 0) p.len_offsets[0] = 0;
}

// Maps of the W tokens i .. i + W - 1 of sequence b, whose new tokens are
// cur .. cur + n - 1 (the table by plain loads: it may have been written by this
// launch's other threads).
template <int W>
__device__ __forceinline__ void map_tokens(const PageParams &p, int b, int i, int cur, int n)
{
    int at[W], slot[W];
    int page = -1, entry = -1; // of the token before
#pragma unroll
    for (int k = 0; k < W; ++k) {
        at[k] = slot[k] = -1;
        if (i + k < n) {
            const int pos = cur + i + k, pg = p.P == 1 ? pos : pos / p.P;
            if (pg != page) {
                page = pg;
                entry = p.page_table[(size_t)b * p.table_len + pg];
            }
            at[k] = pos;
            if (entry >= 0 && entry < p.pool_pages) slot[k] = entry * p.P + (pos - pg * p.P);
        }
    }
    const size_t o = (size_t)b * p.max_new + i;
    if constexpr (W == 4) {
        *reinterpret_cast<int4 *>(p.positions + o) = make_int4(at[0], at[1], at[2], at[3]);
        *reinterpret_cast<int4 *>(p.slots + o) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        *reinterpret_cast<int4 *>(p.q_limit + o) = make_int4(at[0] + 1, at[1] + 1, at[2] + 1, at[3] + 1);
    } else {
        p.positions[o] = at[0];
        p.slots[o] = slot[0];
        p.q_limit[o] = at[0] + 1;
    }
}

__device__ __forceinline__ int held_before(const PageParams &p, int b)
{
    return min(max(p.cur_len[b], 0), p.table_len * p.P);
}

template <bool SHARED, int T>
__global__ void __launch_bounds__(T) qsa_page_map_kernel(const PageParams p, int inline_tokens)
{
    __shared__ int s_warp[32], s_pref[T], s_seq[T], s_take;
    // The map kernel of this call, if there is one, may launch; it waits for this
    // grid.  (Without one the next kernel on the stream may be another call's, which
    // reads these tables at once: no trigger.)
    if (inline_tokens < 0) cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize(); // (this one may be early too; plain loads stay behind the wait)
    if (SHARED) resize_shared<T>(p, s_warp, s_pref, s_seq, &s_take);
    else resize_separate<T>(p, s_warp);
    __syncthreads();
    for (int t = threadIdx.x; t < inline_tokens; t += T) {
        const int b = t / p.max_new, cur = held_before(p, b);
        map_tokens<1>(p, b, t - b * p.max_new, cur, p.out_len[b] - cur);
    }
    __threadfence(); // an INT8 attention launched behind this reads tables and offsets ahead of its wait
}

// A block row per sequence; W tokens per thread (16-byte stores where the rows
// allow them).
template <int W>
__global__ void __launch_bounds__(256) qsa_token_map_kernel(const PageParams p)
{
    cudaGridDependencySynchronize(); // lengths and tables
    const int b = blockIdx.y, cur = held_before(p, b), n = p.out_len[b] - cur;
    // (unsigned: the step past the last token may exceed 2^31, not 2^32)
    for (uint32_t i = (blockIdx.x * 256 + threadIdx.x) * W; i < (uint32_t)p.max_new; i += gridDim.x * 256 * W)
        map_tokens<W>(p, b, (int)i, cur, n);
    __threadfence(); // (the limits: as for the tables)
}

} // namespace
} // namespace qsa

extern "C" qsa_status qsa_page_map(int32_t n_seq, int32_t n_pools, int32_t max_new, int32_t page_cells,
                                   int32_t page_table_len, int32_t pool_pages, const int32_t *cur_len,
                                   const int32_t *new_len, int32_t *page_table, int32_t *free_pages,
                                   int32_t *free_count, int32_t *out_len, int32_t *len_offsets,
                                   int32_t *positions, int32_t *slots, int32_t *q_limit, uint32_t *status,
                                   void *stream)
{
    using namespace qsa;
    if (n_seq < 1 || max_new < 0 || page_cells < 1 || page_table_len < 1 || pool_pages < 1) return QSA_ERR_INVALID_ARG;
    if (n_pools != 1 && n_pools != n_seq) return QSA_ERR_INVALID_ARG;
    const void *arrays[] = {cur_len, new_len, page_table, free_pages, free_count, out_len, len_offsets,
                            positions, slots, q_limit};
    const int n_arrays = max_new > 0 ? 10 : 7; // without new tokens there are no maps to write
    for (int i = 0; i < n_arrays; ++i) {
        if (!arrays[i] || !kv4_aligned(arrays[i], 4)) return QSA_ERR_INVALID_ARG;
        for (int j = i < 2 ? 2 : i + 1; j < n_arrays; ++j) // (cur_len may be new_len)
            if (arrays[i] == arrays[j]) return QSA_ERR_INVALID_ARG;
    }
    if (status && !kv4_aligned(status, 4)) return QSA_ERR_INVALID_ARG;
    const long long lim = 0x7fffffffll, tokens = (long long)n_seq * max_new;
    if (n_seq > 65535 || (long long)page_table_len * page_cells > lim ||
        (long long)n_seq * page_table_len > lim / page_cells || tokens > lim ||
        (long long)pool_pages * page_cells > lim)
        return QSA_ERR_UNSUPPORTED;
    PageParams p{};
    p.cur_len = cur_len;
    p.new_len = new_len;
    p.page_table = page_table;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.out_len = out_len;
    p.len_offsets = len_offsets;
    p.positions = positions;
    p.slots = slots;
    p.q_limit = q_limit;
    p.status = status;
    p.n_seq = n_seq;
    p.max_new = max_new;
    p.P = page_cells;
    p.table_len = page_table_len;
    p.pool_pages = pool_pages;
    const bool fits = tokens <= kInlineTokens, few = n_seq <= kFewThreads && tokens <= 4 * kFewThreads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(few ? kFewThreads : kManyThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto shared = few ? qsa_page_map_kernel<true, kFewThreads> : qsa_page_map_kernel<true, kManyThreads>;
    auto separate = few ? qsa_page_map_kernel<false, kFewThreads> : qsa_page_map_kernel<false, kManyThreads>;
    if (cudaLaunchKernelEx(&cfg, n_pools == 1 ? shared : separate, (const PageParams)p, fits ? (int)tokens : -1) != cudaSuccess)
        return QSA_ERR_CUDA;
    if (fits) return QSA_OK;
    const bool four = max_new % 4 == 0 && kv4_aligned(positions, 16) && kv4_aligned(slots, 16) && kv4_aligned(q_limit, 16);
    const int per_block = 256 * (four ? 4 : 1);
    const long long blocks = ((long long)max_new + per_block - 1) / per_block;
    cfg.gridDim = dim3((unsigned)(blocks < 1024 ? blocks : 1024), (unsigned)n_seq);
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, four ? qsa_token_map_kernel<4> : qsa_token_map_kernel<1>, (const PageParams)p) == cudaSuccess
               ? QSA_OK
               : QSA_ERR_CUDA;
}

// qsa_kv4_attn.cu -- qsa_kv4_attn_batch: decode attention over 4-bit cells.
//
// Per query row q (softmax scale and log2 e folded in) and cell with codes u, v
// and scales / zeros (ks, kz, vs, vz):
//   s = ks (q . u) + kz sum(q),   p = 2^(s - m),
//   out = (sum p vs v + sum p vz) / sum p,
// a one-pass softmax with the running maximum m of the row.
//
// Both contractions (q . u over 256 dimensions, P V over cells) run on the tensor
// cores (tcgen05, f16) with exact codes: the bits 0000 0000 0000 uuuu read as f16
// are u 2^-24, those of 0000 0000 uuuu 0000 u 2^-20, so a 32-bit word of eight
// codes becomes eight f16 values with five logical operations; the factor of 16
// goes into the query.  V's take one multiply-add a pair more, which leaves
// u - 7.5 (expand_centred; the zeros' sum gets 7.5 vs back).  The other operand, a
// query row scaled by a power of two and a probability times the V scale, is one
// f16 value where queries and output are bf16 and the sum of two, about 22 bits,
// for fp32.
//
// qsa_kv4_attn.cuh: a tile's 128 cells on the MMA's M dimension, up to 32 query
// rows on N, K codes in tensor memory, V codes and P' in shared memory; of 20 warps
// four expand K, four V, eight hold the softmax (a thread: one cell, half the rows),
// one issues each contraction, two look up the cells of later tiles.
// qsa_kv4_wide.cu: 128 query rows on M, for windows of many rows.
//
// Work: the tiles of all (sequence, KV head, row block) pairs, dealt to one CTA per
// SM (see the work list).  A pair inside one range is written at once; others leave
// partial sums (at most two per CTA), which the merge kernel joins.
//
// m is a reference that moves only where a score outgrows it; V scales are divided
// by a power of two sigma not below the largest so far, so that P' = p vs / sigma
// stays inside f16.  p, sums, maxima and outputs are fp32.
//
// What bounds it, by ncu: whole contexts (8 rows a KV head, 900,000 cells, 65 us
// for 245 MB: 3.8 TB/s) keep the shared memory 87% busy with a tile's 32 KB of codes
// in and out, 64 KB of expanded V codes in and out and P' (whether that or the
// softmax's latency is the limit is not settled: halving V's share with 8-bit operands
// changed little); long selections in fp32 (24 rows, 38 us for 71 MB) that and the
// softmax; calls of a few tiles latency: a chain of list, page, cells, expansion,
// softmax, P V and merge, 9 us.  A plain gather of the cells takes 43 and 15 us.
//
// Every input is read behind the wait for the kernel before.  Lists, tables and
// cells read ahead of it would take 2.5 to 3.1 us off each call in a row (6.3 us for one
// of a few tiles), but CUDA promises them only behind it.  The figures of single
// choices, here and in the other files, are from before that: both sides lack it.
//
// Tried and slower: mma.sync (68 us whole, 64 long; its 8-bit float forms are
// carried out in f16), tcgen05 with e4m3 operands (65 us whole, but 31 against 25
// batched and 3e-3 off), codes loaded by registers rather than copied to shared
// memory (76 whole), row blocks of 48.
#include "qsa_kv4_attn.cuh"

namespace qsa {
namespace kv4 {
namespace {

constexpr int kMergeWarps = 8;
constexpr int kFewTiles = 112; // of all pairs: three quarters of the SMs
constexpr int kMaxCtas = 160; // partials in the workspace: at least one CTA per SM (152)

// Joins the partials of the pairs that several CTAs share: W warps per row, lane
// l of a warp sums dimensions 8 l .. 8 l + 7.
template <int W>
__global__ void __launch_bounds__(kMergeWarps * 32) qsa_kv4_merge_kernel(const AttnParams p, long long rows)
{
    __shared__ float s_part[W > 1 ? kMergeWarps : 1][kHeadDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = W > 1 ? blockIdx.x : (long long)blockIdx.x * kMergeWarps + warp;
    // the next call may launch: it reads and writes nothing before this grid is done
    cudaTriggerProgrammaticLaunchCompletion();
    if (row >= rows) return; // (with W > 1 the grid has a CTA per row)
    const int bg = (int)(row / p.R), r = (int)(row - (long long)bg * p.R);
    const int b = bg / p.pool.G, g = bg - b * p.pool.G, rb = r / p.rb_rows;
    const int local = r - rb * p.rb_rows;
    const size_t out_at = row_offset(p, b, g, r);
    cudaGridDependencySynchronize();
    // (the list's range and the pair's parts in one go: without cells the latter mean nothing)
    const int2 info = p.max_selected > 0 ? p.info[(long long)bg * p.n_rb + rb] : make_int2(0, 0);
    int start, n;
    list_of(p, b, start, n);
    float o[8], L = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 0.f;
    if (n > 0) {
        if (info.y == 1) return;
        auto slot = [&](int i) { return (size_t)(i == 0 ? info.x : 2 * ((info.x >> 1) + i)) * p.slot_rows + local; };
        auto part = [&](int i, float4 &x, float4 &y) {
            const float4 *src = reinterpret_cast<const float4 *>(p.part_o + slot(i) * kHeadDim + 8 * lane);
            x = src[0];
            y = src[1];
        };
        // the warp's first part is on its way while the weights are formed
        const int first = W > 1 ? warp : 0;
        float4 x, y;
        float2 mine = make_float2(0.f, 0.f);
        if (first < info.y) {
            part(first, x, y);
            mine = p.part_ml[slot(first)];
        }
        float M = -INFINITY;
        for (int i = lane; i < info.y; i += 32) M = fmaxf(M, p.part_ml[slot(i)].x);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
        // (a part without a seen cell has l = 0; NaN marks a row that is not finite)
        auto weight = [&](float m) { return m > -INFINITY ? fast_exp2(m - M) : 1.f; };
        for (int i = lane; i < info.y; i += 32) {
            const float2 ml = p.part_ml[slot(i)];
            L += weight(ml.x) * ml.y;
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) L += __shfl_xor_sync(0xffffffffu, L, k);
        for (int i = first; i < info.y; i += W) {
            const float w = weight(mine.x);
            const float4 u = x, v = y;
            if (i + W < info.y) {
                part(i + W, x, y);
                mine = p.part_ml[slot(i + W)];
            }
            o[0] = fmaf(w, u.x, o[0]); o[1] = fmaf(w, u.y, o[1]); o[2] = fmaf(w, u.z, o[2]); o[3] = fmaf(w, u.w, o[3]);
            o[4] = fmaf(w, v.x, o[4]); o[5] = fmaf(w, v.y, o[5]); o[6] = fmaf(w, v.z, o[6]); o[7] = fmaf(w, v.w, o[7]);
        }
    }
    if constexpr (W > 1) {
        float4 *mine = reinterpret_cast<float4 *>(&s_part[warp][8 * lane]);
        mine[0] = make_float4(o[0], o[1], o[2], o[3]);
        mine[1] = make_float4(o[4], o[5], o[6], o[7]);
        __syncthreads();
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kMergeWarps; ++i) v += s_part[i][threadIdx.x];
        v = L == 0.f ? 0.f : v / L;
        const size_t at = out_at + threadIdx.x;
        if (p.out_bf16) static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16(v);
        else static_cast<float *>(p.out)[at] = v;
    } else {
        const size_t at = out_at + 8 * lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = L == 0.f ? 0.f : o[i] / L;
        if (p.out_bf16) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(o[2 * i + 1]), "f"(o[2 * i]));
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at);
            dst[0] = make_float4(o[0], o[1], o[2], o[3]);
            dst[1] = make_float4(o[4], o[5], o[6], o[7]);
        }
    }
}

// How the rows of a KV head are dealt: f16 parts, row blocks.
struct Plan {
    int parts, n_rb, rb_rows, slot_rows;
    long long pairs;
    size_t off_ml, off_info, total;
};

// Whether R query rows go through the kernel with 128 of them on the MMA's M
// dimension: `tiles` tiles of cells for every block of rows.  Per tile it takes
// 2.4 us where the one of 32 rows takes 1.55, and 7 us more in all (its queries
// and partials).  Measured, bf16, 16,384 cells, 8 (sequence, KV head) pairs: 60
// rows 31.1 against 33.2 us, 72 rows 31.8 against 39.4, 384 rows 69.8 against
// 132; 8,000 cells and 2 pairs: 252 rows 24.0 against 21.8, 384 rows 27.7 against
// 29.1.  (Without rounding, so that more cells never turn it back: a workspace
// for them serves fewer cells too.)
bool is_wide(int R, long long tiles)
{
    const long long gain = 31ll * ((R + kMaxRows - 1) / kMaxRows) - 48ll * ((R + kWideRows - 1) / kWideRows); // 1/20 us
    return gain > 0 && tiles > 140ll * 152 / gain;
}

Plan plan_of(const qsa_shape *s, int n_seq, int max_selected, bool f32_out)
{
    Plan d{};
    const int R = s->q_per_kv * s->n_queries;
    d.parts = s->q_dtype == QSA_F32 || f32_out ? 2 : 1;
    // Blocks of 32 rows; of 8 or 16 where the tiles leave SMs idle all the same (48
    // fp32 rows over 2,051 cells: 9.7 us in two blocks, 8.1 in three, 7.9 in six,
    // 8.5 in eight, whose tiles come near the number of SMs).
    const long long tiles = (long long)n_seq * s->n_kv_heads * ((max_selected + kTile - 1) / kTile);
    const bool wide = d.parts == 1 && is_wide(R, tiles);
    d.slot_rows = wide ? kWideRows : kMaxRows;
    int rows = d.slot_rows;
    for (const int few : {16, 8})
        if (!wide && tiles * ((R + few - 1) / few) <= kFewTiles) rows = few;
    d.n_rb = (R + rows - 1) / rows;
    d.rb_rows = wide ? kWideRows : (R + d.n_rb - 1) / d.n_rb;
    d.pairs = (long long)n_seq * s->n_kv_heads * d.n_rb;
    if (max_selected > 0) {
        const size_t slots = (size_t)2 * kMaxCtas * d.slot_rows;
        d.off_ml = slots * kHeadDim * sizeof(float);
        d.off_info = d.off_ml + align_up(slots * sizeof(float2), 256);
        // (room for the pairs of fewer cells too, whose rows may be in more blocks)
        long long pairs = (long long)n_seq * s->n_kv_heads * ((R + kMaxRows - 1) / kMaxRows);
        if (pairs < kFewTiles) pairs = kFewTiles;
        d.total = d.off_info + align_up((size_t)pairs * sizeof(int2), 256);
    }
    return d;
}

qsa_status check_attn(const qsa_shape *s, int n_seq, int n_pools, int max_selected)
{
    const qsa_status st = kv4_check(s, n_seq, n_pools);
    if (st != QSA_OK) return st;
    if (n_seq < 1 || max_selected < 0 || s->q_per_kv < 1 || s->n_queries < 1 ||
        !(fabsf(s->softmax_scale) < 0x1p100f)) // (nor NaN; the kernels take it times powers of two)
        return QSA_ERR_INVALID_ARG;
    if (s->q_dtype != QSA_F32 && s->q_dtype != QSA_BF16) return QSA_ERR_INVALID_ARG;
    if (n_seq > 65535 || s->q_per_kv > 64 || s->n_queries > 65536 || max_selected > 0x7fffffff - 1024 ||
        (long long)s->q_per_kv * s->n_queries * s->n_kv_heads > 0x7fffffffll / n_seq)
        return QSA_ERR_UNSUPPORTED;
    return QSA_OK;
}

} // namespace
} // namespace kv4
} // namespace qsa

extern "C" qsa_status qsa_kv4_attn_workspace_bytes(const qsa_shape *shape, int32_t n_seq, int32_t max_selected,
                                                   size_t *bytes)
{
    const qsa_status st = qsa::kv4::check_attn(shape, n_seq, 1, max_selected);
    if (st != QSA_OK) return st;
    if (!bytes) return QSA_ERR_INVALID_ARG;
    // (the larger of the two output types')
    const size_t f32 = qsa::kv4::plan_of(shape, n_seq, max_selected, true).total,
                 bf16 = qsa::kv4::plan_of(shape, n_seq, max_selected, false).total;
    *bytes = f32 > bf16 ? f32 : bf16;
    return QSA_OK;
}

extern "C" qsa_status qsa_kv4_attn_batch(const qsa_shape *shape, int32_t n_seq, int32_t n_pools, const void *q,
                                         const uint8_t *kv_pool, const float *kv_scale, const int32_t *page_table,
                                         const int32_t *sel, const int32_t *sel_offsets, int32_t max_selected,
                                         const int32_t *q_limit, int32_t out_dtype, void *out, void *workspace,
                                         size_t workspace_bytes, uint32_t *status, void *stream)
{
    using namespace qsa;
    using namespace qsa::kv4;
    const qsa_status st = check_attn(shape, n_seq, n_pools, max_selected);
    if (st != QSA_OK) return st;
    if (out_dtype != QSA_F32 && out_dtype != QSA_BF16) return QSA_ERR_INVALID_ARG;
    const Plan d = plan_of(shape, n_seq, max_selected, out_dtype == QSA_F32);
    if (!q || !kv_pool || !kv_scale || !page_table || !sel_offsets || !out || (d.total > 0 && !workspace))
        return QSA_ERR_INVALID_ARG;
    if (!kv4_aligned(q, 16) || !kv4_aligned(kv_pool, 32) || !kv4_aligned(kv_scale, 16) ||
        !kv4_aligned(page_table, 4) || !kv4_aligned(sel, 4) || !kv4_aligned(sel_offsets, 4) ||
        !kv4_aligned(q_limit, 4) || !kv4_aligned(out, 16) || !kv4_aligned(workspace, 256) || !kv4_aligned(status, 4))
        return QSA_ERR_INVALID_ARG;
    for (const void *a : {(const void *)q, (const void *)kv_pool, (const void *)kv_scale})
        if (out == a || (workspace && workspace == a) || out == workspace) return QSA_ERR_INVALID_ARG;
    if (workspace_bytes < d.total) return QSA_ERR_WORKSPACE;
    // (rows of the pools are numbered in 32 bits)
    if ((long long)n_pools * shape->n_kv_heads > 0xfffffffell / shape->pool_cells) return QSA_ERR_UNSUPPORTED;

    AttnParams p{};
    p.pool = kv4_pool(shape, n_pools, page_table);
    p.q = q;
    p.codes = kv_pool;
    p.scale = reinterpret_cast<const float4 *>(kv_scale);
    p.sel = sel;
    p.sel_offsets = sel_offsets;
    p.q_limit = q_limit;
    p.out = out;
    char *ws = static_cast<char *>(workspace);
    p.part_o = reinterpret_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + d.off_ml);
    p.info = reinterpret_cast<int2 *>(ws + d.off_info);
    p.status = status;
    p.n_seq = n_seq;
    p.H = shape->q_per_kv;
    p.T = shape->n_queries;
    p.R = p.H * p.T;
    p.n_rb = d.n_rb;
    p.rb_rows = d.rb_rows;
    p.slot_rows = d.slot_rows;
    p.max_selected = max_selected;
    p.q_bf16 = shape->q_dtype == QSA_BF16;
    p.out_bf16 = out_dtype == QSA_BF16;
    p.scale_log2 = shape->softmax_scale * kLog2e;
    p.wait_cycles = wait_limit();
    const int P = p.pool.page_cells;
    p.page_shift = -1;
    p.h_mul = (uint32_t)(((1ull << 32) + p.H - 1) / p.H);
    for (int k = 0; k < 31; ++k)
        if (P == 1 << k) p.page_shift = k;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return QSA_ERR_CUDA;
    const long long tiles = d.pairs * ((max_selected + kTile - 1) / kTile);
    const int cap = sms < kMaxCtas ? sms : kMaxCtas;
    p.small = tiles < (1ll << 23);
    // (measured: a second segment costs the kernel for wide windows 14 us, 7 tiles;
    // the other one's batched decode takes 22.3 us without this, 18.1 with)
    p.seg_tiles = d.slot_rows == kWideRows ? 7 : 1;
    if (tiles / cap >= 0x7fffffffll) return QSA_ERR_UNSUPPORTED;
    const int grid = (int)(tiles < 1 ? 1 : tiles < cap ? tiles : cap);
    const cudaError_t e = d.slot_rows == kWideRows ? launch_wide(p, grid, cs)
                          : d.parts == 1 ? launch_single(p, d.rb_rows, grid, cs) : launch_split(p, d.rb_rows, grid, cs);
    if (e != cudaSuccess) return QSA_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = cs;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const long long rows = (long long)n_seq * shape->n_kv_heads * p.R;
    // Parts of a pair: the CTAs that share it, at most grid / pairs and one more
    // (when full).  A CTA per row joins more than four, a warp per row fewer, or
    // where rows enough keep the SMs busy (6,168 rows: 15 us less).
    const bool wide = grid / d.pairs + 2 > 4 && rows <= 2048;
    cfg.gridDim = dim3((unsigned)(wide ? rows : (rows + kMergeWarps - 1) / kMergeWarps));
    const cudaError_t m = wide ? cudaLaunchKernelEx(&cfg, qsa_kv4_merge_kernel<kMergeWarps>, (const AttnParams)p, rows)
                               : cudaLaunchKernelEx(&cfg, qsa_kv4_merge_kernel<1>, (const AttnParams)p, rows);
    return m == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}

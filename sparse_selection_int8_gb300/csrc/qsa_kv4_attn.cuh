// qsa_kv4_attn.cuh -- the attention kernel over 4-bit cells (see
// qsa_kv4_attn.cu for the mathematics and the launches).
#pragma once

#include <float.h>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qsa_kv4.cuh"
#include "qsa_sm100.cuh"

namespace qsa {
namespace kv4 {

using namespace sm100;

constexpr int kTile = 128;   // cells per tile (MMA M)
constexpr int kMaxRows = 32; // query rows of a row block at most
constexpr int kWideRows = 128; // the same in the kernel for wide windows (MMA M)
constexpr int kKWarps = 4, kVWarps = 4, kSoftWarps = 8;
constexpr int kSoft0 = kKWarps + kVWarps;    // first softmax warp
constexpr int kSWarp = kSoft0 + kSoftWarps;  // issues S = K.Q^T
constexpr int kPvWarp = kSWarp + 1;          // issues O += V^T.P'^T
constexpr int kRes0 = kPvWarp + 1;           // two warps look the cells up
constexpr int kThreads = (kRes0 + 2) * 32;   // 640
constexpr int kSoftThreads = kSoftWarps * 32, kSetThreads = kSoftThreads / 2;
constexpr int kPrm = 4;                      // entries of the parameter ring
constexpr int kRow = 6;                      // entries of the row ring
constexpr uint32_t kRawBytes = kTile * QSA_KV4_CODE_BYTES; // a tile's codes
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBarSet = 1, kBarSoft = 3; // named barriers: one per row set, one for both
constexpr float kSlackLog2 = 8.f;             // a new reference lies this far above the largest score
constexpr long long kDrainCycles = 1ll << 30; // bound of the waits before the CTA leaves

struct AttnParams {
    Kv4Pool pool;
    const void *q;
    const uint8_t *codes;
    const float4 *scale;
    const int32_t *sel, *sel_offsets, *q_limit;
    void *out;
    float *part_o;   // [2 * CTAs][slot_rows][256] partial sums
    float2 *part_ml; // [2 * CTAs][slot_rows] (m, l)
    int2 *info;      // [pairs] (first partial, how many): 1 means already in `out`
    uint32_t *status;
    int32_t n_seq, H, T, R;   // R = T * H rows per KV head
    int32_t n_rb, rb_rows;    // row blocks per KV head, rows of each
    int32_t slot_rows;        // rows of a partial: kMaxRows or kWideRows
    int32_t max_selected, q_bf16, out_bf16;
    float scale_log2;
    uint32_t h_mul;           // see query_of
    int32_t small;            // fewer than 2^23 tiles
    int32_t seg_tiles;        // what a segment costs besides its tiles, in tiles
    int32_t page_shift;       // log2 of the page size, -1 if it is no power of two
    long long wait_cycles;    // bound of a device-side wait, SM clock cycles
};

__device__ __forceinline__ void raise(const AttnParams &p, uint32_t bits)
{
    if (bits && p.status) atomicOr(p.status, bits);
}

// List range of sequence b (bad offsets are clamped).  (Here and below: plain loads,
// of what the kernel before may have written.)
__device__ __forceinline__ uint32_t list_of(const AttnParams &p, int b, int &start, int &n)
{
    start = p.sel_offsets[b];
    const long long len = (long long)p.sel_offsets[b + 1] - start;
    if (start < 0 || len < 0) {
        start = n = 0;
        return QSA_STATUS_BAD_OFFSETS;
    }
    n = (int)(len < p.max_selected ? len : p.max_selected);
    return len > p.max_selected ? QSA_STATUS_BAD_OFFSETS : 0u;
}

// Query of row r: r / H (h_mul = ceil(2^32 / H), exact for r < 2^22, H <= 64).
__device__ __forceinline__ int query_of(const AttnParams &p, int r)
{
    return p.H == 1 ? r : (int)__umulhi((uint32_t)r, p.h_mul);
}

// What a row's sums from the tensor cores (of codes u 2^-24 and queries scaled up from
// exponent e) are multiplied by to be scores in log2 units: 2^(e - 141) 2^24 |scale|, in
// an order that neither over- nor underflows before the result does.  Where that
// underflows (a softmax scale of 0, say) it is the smallest positive number, so that a masked
// cell's -inf stays -inf; all other scores vanish (the sums are below 2^127).
__device__ __forceinline__ float row_scale(const AttnParams &p, uint32_t e)
{
    return fmaxf(__uint_as_float((e - 2u) << 23) * (fabsf(p.scale_log2) * 0x1p12f), 0x1p-149f);
}

// Element offset of row r of (sequence b, KV head g) in q and out.
__device__ __forceinline__ size_t row_offset(const AttnParams &p, int b, int g, int r)
{
    const int t = query_of(p, r), j = r - t * p.H;
    return ((((size_t)b * p.T + t) * p.pool.G + g) * p.H + j) * kHeadDim;
}

// ---------------------------------------------------------------- work list
// A pair is a (sequence, KV head, row block); its cells are cut into tiles of
// 128.  The tiles of all pairs, in order, are dealt to the CTAs in equal
// contiguous ranges; a segment is a CTA's run of tiles of one pair.  A second
// segment costs a CTA what some tiles do (p.seg_tiles), so where a pair's tiles
// can be cut into ranges of its own that are longer by no more than that, they
// are, as many as each pair needs.

struct Walk {
    int b, g, rb, u, nu, n, start; // tile u of the pair's nu; list length and start
    int left;                      // tiles left in the CTA's range
    int parts;                     // CTAs of the pair, if its ranges are its own; else 0
    long long x;                   // index of the tile
};

// CTAs that have work: each at least one so that the CTAs of a pair are
// consecutive.
__device__ __forceinline__ int ctas_of(long long total) { return (int)min((long long)gridDim.x, total); }

// a / b for non-negative a and positive b: in 32 bits where they fit.
__device__ __forceinline__ long long quotient(long long a, long long b)
{
    return (a | b) <= 0x7fffffffll ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

__device__ __forceinline__ long long range_begin(long long total, int ncta, int cta) { return quotient(total * cta, ncta); }

// The CTA whose range holds tile x.
__device__ __forceinline__ int cta_of(long long total, int ncta, long long x)
{
    return (int)quotient((x + 1) * ncta - 1, total);
}

// How many CTAs share the pair whose first tile is the walk's.
__device__ __forceinline__ int parts_of(const Walk &w, long long total)
{
    return w.parts ? w.parts : cta_of(total, ctas_of(total), w.x + w.nu - 1) - (int)blockIdx.x + 1;
}

// First tile of this CTA, by one full warp.
__device__ inline void walk_init(const AttnParams &p, Walk &w, long long &total, int lane)
{
    if (p.small && p.n_seq <= 32) { // one look at the lists, 32-bit arithmetic
        const uint32_t per = (uint32_t)p.pool.G * p.n_rb;
        int s = 0, n = 0;
        uint32_t bad = 0;
        if (lane < p.n_seq) bad = list_of(p, lane, s, n);
        if (blockIdx.x == 0) raise(p, bad);
        const int nu = (n + kTile - 1) / kTile;
        const uint32_t mine = per * nu;
        uint32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const uint32_t sum = __shfl_sync(0xffffffffu, incl, 31), ncta = min(gridDim.x, sum);
        total = sum;
        w = Walk{};
        if (blockIdx.x >= ncta) return;
        // the shortest ranges of which there is one for every CTA at most
        const uint32_t even = (sum + ncta - 1) / ncta;
        for (uint32_t m = even; m <= even + p.seg_tiles; ++m) {
            const uint32_t k = (nu + m - 1) / m, ctas = per * k;
            if (__reduce_add_sync(0xffffffffu, ctas) > gridDim.x) continue;
            uint32_t end = ctas;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end += v;
            }
            const unsigned in = __ballot_sync(0xffffffffu, end - ctas <= blockIdx.x && blockIdx.x < end);
            if (!in) return; // (no range for this CTA)
            const int src = __ffs(in) - 1;
            const uint32_t off = blockIdx.x - __shfl_sync(0xffffffffu, end - ctas, src);
            w.b = src;
            w.n = __shfl_sync(0xffffffffu, n, src);
            w.start = __shfl_sync(0xffffffffu, s, src);
            w.nu = __shfl_sync(0xffffffffu, nu, src);
            w.parts = (int)__shfl_sync(0xffffffffu, k, src);
            const uint32_t pair = off / (uint32_t)w.parts, r = off - pair * w.parts;
            w.u = (int)((uint64_t)w.nu * r / (uint32_t)w.parts);
            w.left = (int)((uint64_t)w.nu * (r + 1) / (uint32_t)w.parts) - w.u;
            w.g = (int)(pair / (uint32_t)p.n_rb);
            w.rb = (int)(pair - (uint32_t)w.g * p.n_rb);
            return;
        }
        const uint32_t lo = sum * blockIdx.x / ncta, hi = sum * (blockIdx.x + 1) / ncta; // (< 2^31: at most 160 CTAs)
        const unsigned hit = __ballot_sync(0xffffffffu, incl - mine <= lo && lo < incl);
        const int src = __ffs(hit) - 1;
        const uint32_t off = lo - __shfl_sync(0xffffffffu, incl - mine, src);
        w.b = src;
        w.n = __shfl_sync(0xffffffffu, n, src);
        w.start = __shfl_sync(0xffffffffu, s, src);
        w.nu = __shfl_sync(0xffffffffu, nu, src);
        const uint32_t pair = off / (uint32_t)w.nu;
        w.u = (int)(off - pair * w.nu);
        w.g = (int)(pair / (uint32_t)p.n_rb);
        w.rb = (int)(pair - (uint32_t)w.g * p.n_rb);
        w.left = (int)(hi - lo);
        w.x = lo;
        return;
    }
    const long long per_tile = (long long)p.pool.G * p.n_rb;
    long long sum = 0;
    uint32_t bad = 0;
    for (int b = lane; b < p.n_seq; b += 32) {
        int s, n;
        bad |= list_of(p, b, s, n);
        sum += per_tile * ((n + kTile - 1) / kTile);
    }
    if (blockIdx.x == 0) raise(p, bad);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    total = sum;
    w = Walk{};
    if (total == 0) return;
    const int ncta = ctas_of(total);
    if ((int)blockIdx.x >= ncta) return;
    const long long lo = range_begin(total, ncta, blockIdx.x), hi = range_begin(total, ncta, blockIdx.x + 1);
    long long before = 0;
    for (int b0 = 0; b0 < p.n_seq; b0 += 32) {
        const int b = b0 + lane;
        int s = 0, n = 0;
        if (b < p.n_seq) list_of(p, b, s, n);
        const int nu = (n + kTile - 1) / kTile;
        const long long mine = per_tile * nu;
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + incl - mine <= lo && lo < before + incl);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const long long off = lo - before - __shfl_sync(0xffffffffu, incl - mine, src);
            w.b = b0 + src;
            w.n = __shfl_sync(0xffffffffu, n, src);
            w.start = __shfl_sync(0xffffffffu, s, src);
            w.nu = __shfl_sync(0xffffffffu, nu, src);
            const long long pair = quotient(off, w.nu);
            w.u = (int)(off - pair * w.nu);
            w.g = (int)quotient(pair, p.n_rb);
            w.rb = (int)(pair - (long long)w.g * p.n_rb);
            w.left = (int)(hi - lo);
            w.x = lo;
            return;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
}

// `k` tiles on, at most to the start of the next pair.
__device__ __forceinline__ void walk_next(const AttnParams &p, Walk &w, int k)
{
    w.left -= k;
    w.x += k;
    if (w.left <= 0 || (w.u += k) < w.nu) return;
    w.u = 0;
    if (++w.rb < p.n_rb) return;
    w.rb = 0;
    if (++w.g < p.pool.G) return;
    w.g = 0;
    while (++w.b < p.n_seq) { // (the range ends before the list does)
        list_of(p, w.b, w.start, w.n);
        if (w.n > 0) {
            w.nu = (w.n + kTile - 1) / kTile;
            return;
        }
    }
    w.left = 0;
}

// ------------------------------------------------------------- f16 operands

// Two values as f16 (a in the low half), and what the rounding leaves of them.
__device__ __forceinline__ uint32_t half2_of(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void rest2(uint32_t w, float &a, float &b)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    a -= f.x;
    b -= f.y;
}

// A word of eight codes as four f16 pairs, in the order of dimensions 0 4 | 1 5 |
// 2 6 | 3 7.  Bits 0-3 and 16-19 of a word read as f16 are u 2^-24, bits 4-7 and
// 20-23 are u 2^-20 (subnormal, exact): three of five operations are masks, no
// conversion, and the second and fourth pair count 16 times as much.
__device__ __forceinline__ void expand(uint32_t w, uint32_t *o)
{
    o[0] = w & 0x000f000fu;
    o[1] = w & 0x00f000f0u;
    o[2] = (w >> 8) & 0x000f000fu;
    o[3] = (w >> 8) & 0x00f000f0u;
}

// The same centred, (u - 7.5) 2^-9 in all four pairs (exact: one multiply-add of
// f16 each).  The tensor core's fp32 sums round towards zero, so a step of 16 cells
// loses about 2^-25 of the sum so far; a sum of terms of one sign is many times the
// output, which the zeros' sum takes off again (bf16, 6,000 cells a CTA: 2.3e-3
// off where rounding the output alone is 1.7e-3).  With codes of both signs
// the sum is as large as the result.
__device__ __forceinline__ void expand_centred(uint32_t w, uint32_t *o)
{
    expand(w, o);
    // times 2^15 and 2^11, less 7.5 * 2^-9
    asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(o[0]) : "r"(0x78007800u), "r"(0xa380a380u));
    asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(o[1]) : "r"(0x68006800u), "r"(0xa380a380u));
    asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(o[2]) : "r"(0x78007800u), "r"(0xa380a380u));
    asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(o[3]) : "r"(0x68006800u), "r"(0xa380a380u));
}

__device__ __forceinline__ void tmem_ld2(uint32_t taddr, float *v)
{
    uint32_t r[2];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
    v[0] = __uint_as_float(r[0]);
    v[1] = __uint_as_float(r[1]);
}

__device__ __forceinline__ void tmem_st2(uint32_t taddr, const float *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};"
                 ::"r"(taddr), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])) : "memory");
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const float *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};"
                 ::"r"(taddr), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                   "r"(__float_as_uint(v[3])) : "memory");
}

// K (even) consecutive columns of this thread's lane.
template <int K>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, float *v)
{
    constexpr int k = K >= 16 ? 16 : K >= 8 ? 8 : K >= 4 ? 4 : 2;
    if constexpr (k == 16) tmem_ld16(taddr, v);
    else if constexpr (k == 8) tmem_ld8(taddr, v);
    else if constexpr (k == 4) tmem_ld4(taddr, v);
    else tmem_ld2(taddr, v);
    if constexpr (K > k) tmem_ldn<K - k>(taddr + k, v + k);
}

template <int K>
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const float *v)
{
    constexpr int k = K >= 16 ? 16 : K >= 4 ? 4 : 2;
    if constexpr (k == 16) tmem_st16(taddr, v);
    else if constexpr (k == 4) tmem_st4(taddr, v);
    else tmem_st2(taddr, v);
    if constexpr (K > k) tmem_stn<K - k>(taddr + k, v + k);
}

// Largest over the warp (NaN left out).
__device__ __forceinline__ float warp_max(float v)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Sums over the warp of one value per row and lane, K rows (a power of two): lane
// l ends with the sum of row l % K.  After the steps among lanes of the same row,
// each step halves the rows a lane carries.
template <int K>
__device__ __forceinline__ float warp_sum_rows(float *v, int lane)
{
#pragma unroll
    for (int o = 16; o >= K; o >>= 1)
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
#pragma unroll
    for (int o = K / 2; o > 0; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0];
}

// A warp's half rows (K or V codes, 128 bytes each) of 32 cells, row of cell l in
// lane l: eight lanes per row, four rows an operation, the pieces permuted by the
// cell, so that eight neighbouring cells' reads meet no bank twice.
template <int U>
__device__ __forceinline__ void copy_rows(const uint8_t *codes, uint32_t row, uint32_t dst, int lane)
{
    const uint32_t c = lane >> 3, piece = lane & 7;
    const uint8_t *src = codes + piece * 16;
    dst += c * QSA_KV4_CODE_BYTES;
#pragma unroll(U)
    for (int i = 0; i < 8; i += 2) { // cells 4 i + c, 4 i + 4 + c
        const uint32_t r0 = __shfl_sync(0xffffffffu, row, 4 * i + c), r1 = __shfl_sync(0xffffffffu, row, 4 * i + 4 + c);
        cp_async16(dst + i * (4 * QSA_KV4_CODE_BYTES) + ((piece ^ c) << 4), src + (size_t)r0 * QSA_KV4_CODE_BYTES);
        cp_async16(dst + (i + 1) * (4 * QSA_KV4_CODE_BYTES) + ((piece ^ (c + 4)) << 4), src + (size_t)r1 * QSA_KV4_CODE_BYTES);
    }
}

// -------------------------------------------------------------------- kernel

// What two rows need at every tile: their scales and sum(q) (see the queries);
// less their references (log2 units), and 2^14 / sigma of their V scales.  A row
// that has seen no cell has reference 0 and kFresh there.
struct RowScore {
    float2 xs, qz;
};
struct RowRef {
    float2 nref, isg;
};
constexpr float kFresh = 0x1p114f;
constexpr uint64_t kLayoutSw32 = 6; // of a shared-memory matrix descriptor

struct Misc {
    float4 prm[kPrm][kTile];   // scales and zeros of the tile's cells
    int32_t pos[kRow][kTile];  // positions of the tile's cells; 2^31 - 1 where there is no cell
    uint32_t row[kRow][kTile]; // their rows in the pool
    RowScore score[kMaxRows / 2];
    RowRef ref[kMaxRows / 2];
    int32_t lim[kMaxRows];
    int32_t odd[kMaxRows]; // the row's query is not finite
    float isg_max[2];      // largest 2^14 / sigma of a set's rows
    // the rows' element offsets in q and out, by the segment's parity: a warp may stage
    // a segment's queries while a slower one still stores the outputs of the one before
    long long off[2][kMaxRows];
    float red[2][2][4][kMaxRows / 2]; // [set][what][warp][row] reductions
    float delta[kMaxRows], fac[kMaxRows], ofac[kMaxRows], fin[kMaxRows], zsum[kMaxRows];
    Walk first;
    long long total;
    uint32_t tmem;
    int abort;
    uint64_t row_full[kRow], row_empty[kRow], prm_full[kPrm], prm_empty[kPrm];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], s_empty[2], p_full[2], p_empty[2];
    uint64_t q_full, q_empty, o_full, o_empty, s_done, pv_done;
};

// PARTS: f16 parts of a query element and a probability; RS: rows of each of the
// two sets of softmax warps (2 RS rows a block).  MMA columns: a set's rows are
// consecutive, their high parts, then their low ones.
template <int RS, int PARTS>
struct Cfg {
    static constexpr int CR = PARTS * RS;           // columns of a set's rows
    static constexpr int CS = (CR + 7) / 8 * 8;     // columns of a set
    static constexpr int N = (2 * CS + 15) / 16 * 16;
    static constexpr int SL = (CR + 3) / 4 * 4;     // columns loaded at a time
    // The roles' code shares the instruction cache: with many rows, whose softmax is
    // long, the copy loops stay rolled (32 rows: 137 us against 140; 8 rows: 63.2
    // against 60.1 unrolled).
    static constexpr bool Short = RS > 8;
    // Tiles whose P.V is summed on the tensor cores at a time: an fp32 output's sums
    // of so many are added up in registers, which round to nearest (see
    // expand_centred).
    static constexpr bool Runs = PARTS > 1;
    static constexpr int Run = 8;
    // registers of the roles (warpgroups: K, V, twice softmax, the rest), where the
    // softmax holds those sums
    static constexpr int SoftRegs = 128, CodeRegs = 72, RestRegs = 80;
    static_assert(2 * SoftRegs + 2 * CodeRegs + RestRegs <= 5 * 96, "registers of the launch");
    static constexpr int ST = 3;                    // raw stages, one tile's codes each
    static constexpr int PB = N <= 48 ? 2 : 1;      // P' buffers
    static constexpr uint32_t raw = 0;
    static constexpr uint32_t v = ST * kTile * QSA_KV4_CODE_BYTES;
    static constexpr uint32_t q = v + kTile * kHeadDim * 2;
    static constexpr uint32_t p = q + N * 512u;
    static constexpr uint32_t misc = p + PB * N * 256u;
    static constexpr uint32_t total = misc + (uint32_t)sizeof(Misc);
    // tensor memory: two buffers of K (128 columns each), two of S, O in two halves
    static constexpr uint32_t colS = 256, colO = colS + 2 * N;
    static_assert(RS % 2 == 0 && 2 * RS <= kMaxRows, "rows");
    static_assert(colO + 2 * N <= kTmemCols, "columns");
    static_assert(total <= 227 * 1024, "shared memory");
    // first column of row r
    static __device__ __forceinline__ int col(int r) { return r < RS ? r : CS + r - RS; }
};

template <int RS, int PARTS>
__global__ void __launch_bounds__(kThreads, 1) qsa_kv4_attn_kernel(const AttnParams p)
{
    using C = Cfg<RS, PARTS>;
    constexpr int N = C::N, PB = C::PB, ST = C::ST;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) { // (the swizzled operand tiles need it)
        if (threadIdx.x == 0) raise(p, QSA_STATUS_LAUNCH);
        return;
    }
    Misc &ms = *reinterpret_cast<Misc *>(smem + C::misc);
    const int tid = threadIdx.x, lane = tid & 31;
    const int w = __shfl_sync(0xffffffffu, tid >> 5, 0); // provably uniform

    if (tid == 0) {
        for (int i = 0; i < kRow; ++i) {
            mbar_init(&ms.row_full[i], 64);
            mbar_init(&ms.row_empty[i], (kKWarps + kVWarps) * 32 + kSoftThreads);
        }
        for (int i = 0; i < kPrm; ++i) {
            mbar_init(&ms.prm_full[i], kKWarps * 32);
            mbar_init(&ms.prm_empty[i], kSoftThreads);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.k_full[i], kKWarps * 32);
            mbar_init(&ms.k_empty[i], 1);
            mbar_init(&ms.v_full[i], kVWarps * 16);
            mbar_init(&ms.v_empty[i], 1);
            mbar_init(&ms.s_full[i], 1);
            mbar_init(&ms.s_empty[i], kSoftThreads);
            mbar_init(&ms.p_full[i], kSoftThreads);
            mbar_init(&ms.p_empty[i], 1);
        }
        mbar_init(&ms.q_full, kSoftThreads);
        mbar_init(&ms.q_empty, 1);
        mbar_init(&ms.o_full, 1);
        mbar_init(&ms.o_empty, kSoftThreads);
        mbar_init(&ms.s_done, 1);
        mbar_init(&ms.pv_done, 1);
        ms.abort = 0;
        fence_mbar_init();
    }
    // rows of the pool from the start: a wait that runs out lets the copies read them early
    for (int i = tid; i < kRow * kTile; i += kThreads) (&ms.row[0][0])[i] = 0u;
    // All input is read behind this: the kernel before may have written any of it (the
    // merge of a call whose output is this one's query, a copy into a list or a page
    // table), and its writes are promised here only; it may also still read the
    // partials that this one writes.  Tensor memory is taken behind it too: a kernel
    // that let this one start may yet need it to end.
    cudaGridDependencySynchronize();
    if (w == kSWarp) {
        tmem_alloc(&ms.tmem, kTmemCols);
        tmem_relinquish();
    }
    if (w == kSoft0) {
        Walk f;
        long long t;
        walk_init(p, f, t, lane);
        if (lane == 0) {
            ms.first = f;
            ms.total = t;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the merge may be scheduled; it waits for this grid
    cudaTriggerProgrammaticLaunchCompletion();
    const uint32_t tmem = __shfl_sync(0xffffffffu, ms.tmem, 0);

    // A wait that runs out raises QSA_STATUS_TIMEOUT and makes all later ones of
    // the CTA return at once, so that every role reaches its end.
    volatile int *abort_flag = &ms.abort;
    // (a bound of a few cycles runs out at once: try_wait would sleep past it)
    const long long limit = p.wait_cycles < 64 ? -1 : p.wait_cycles;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_test_wait(bar, parity & 1u) || *abort_flag) return;
        const long long t0 = clock64();
        while (clock64() - t0 <= limit)
            if (mbar_try_wait(bar, parity & 1u, 0u)) return;
        *abort_flag = 1;
        raise(p, QSA_STATUS_TIMEOUT);
    };

    if (w < kKWarps) {
        // =================================================================== K
        if constexpr (C::Runs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::CodeRegs));
        // The warp's 32 cells' K codes, scales and zeros are copied two tiles ahead.
        const int cell = 32 * w + lane, tiles = ms.first.left;
        const uint8_t *src = smem + C::raw + cell * QSA_KV4_CODE_BYTES;
        const uint32_t at = (uint32_t)(cell & 7) << 4, t_lane = (uint32_t)(32 * w) << 16;
#pragma unroll 1
        for (int j = -2; j < tiles; ++j) {
            if (j + 2 < tiles) {
                const uint32_t t = j + 2, e = t % kRow, pe = t % kPrm;
                wait(&ms.row_full[e], t / kRow);
                const uint32_t row = ms.row[e][cell];
                mbar_arrive(&ms.row_empty[e]);
                copy_rows<C::Short ? 1 : 4>(p.codes, row, smem_u32(smem + C::raw) + (t % ST) * kRawBytes + w * (kRawBytes / 4), lane);
                if (t >= kPrm) wait(&ms.prm_empty[pe], t / kPrm - 1);
                cp_async16(smem_u32(&ms.prm[pe][cell]), p.scale + row);
                cp_async_mbar_arrive_noinc(&ms.prm_full[pe]);
            }
            cp_async_commit(); // (past the last tile too, so that the groups' count holds)
            if (j >= 0) {
                // K codes of the lane's cell -> tensor memory (the MMA's A operand:
                // lane = cell, two f16 per column)
                const uint32_t kb = j & 1;
                if (j >= 2) wait(&ms.k_empty[kb], (j >> 1) - 1);
                cp_async_wait_group<ST - 1>();
                __syncwarp();
                tc_fence_after();
                const uint8_t *raw = src + (j % ST) * kRawBytes;
                const uint32_t t0 = tmem + t_lane + 128u * kb;
                uint4 v = *reinterpret_cast<const uint4 *>(raw + at);
#pragma unroll(C::Short ? 1 : 2)
                for (int c = 0; c < 8; ++c) {
                    const uint4 n = *reinterpret_cast<const uint4 *>(raw + ((((c + 1) & 7) << 4) ^ at));
                    uint32_t f[16];
                    expand(v.x, f);
                    expand(v.y, f + 4);
                    expand(v.z, f + 8);
                    expand(v.w, f + 12);
                    tmem_st16u(t0 + 16u * c, f);
                    v = n;
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&ms.k_full[kb]);
                __syncwarp();
            }
        }
        cp_async_wait_all();
    } else if (w < kSoft0) {
        // =================================================================== V
        if constexpr (C::Runs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::CodeRegs));
        // Codes of the lane's cell, copied two tiles ahead -> shared memory, the
        // MMA's A operand [256 dimensions][128 cells], MN-major with the 128-byte
        // swizzle: a word of codes is one 16-byte piece.  The two halves of the
        // tile's cells are handed over (and freed) on their own.
        const int q = w - kKWarps, cell = 32 * q + lane, half = cell >> 6;
        const int tiles = ms.first.left;
        const uint8_t *src = smem + C::raw + cell * QSA_KV4_CODE_BYTES + 128;
        const uint32_t at = (uint32_t)(cell & 7) << 4;
        uint8_t *dst = smem + C::v + (cell >> 3) * 1024 + (cell & 7) * 128;
#pragma unroll 1
        for (int j = -2; j < tiles; ++j) {
            if (j + 2 < tiles) {
                const uint32_t e = (j + 2) % kRow;
                wait(&ms.row_full[e], (j + 2) / kRow);
                const uint32_t row = ms.row[e][cell];
                mbar_arrive(&ms.row_empty[e]);
                copy_rows<C::Short ? 1 : 4>(p.codes + 128, row, smem_u32(smem + C::raw) + (uint32_t)((j + 2) % ST) * kRawBytes + q * (kRawBytes / 4) + 128, lane);
            }
            cp_async_commit();
            if (j < 0) continue;
            cp_async_wait_group<ST - 1>();
            __syncwarp();
            const uint8_t *raw = src + (j % ST) * kRawBytes;
            uint4 v = *reinterpret_cast<const uint4 *>(raw + at);
            if (j >= 1) wait(&ms.v_empty[half], j - 1);
#pragma unroll 2
            for (int c = 0; c < 8; ++c) {
                const uint4 n = *reinterpret_cast<const uint4 *>(raw + ((((c + 1) & 7) << 4) ^ at));
                const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t f[4];
                    expand_centred(wd[i], f);
                    // word 4c + i: block (4c + i) / 8, piece (4c + i) % 8
                    *reinterpret_cast<uint4 *>(dst + (c >> 1) * 16384 + (((4 * (c & 1) + i) << 4) ^ at)) =
                        make_uint4(f[0], f[1], f[2], f[3]);
                }
                v = n;
            }
            fence_proxy_async_smem();
            mbar_arrive(&ms.v_full[half]);
            __syncwarp();
        }
        cp_async_wait_all();
    } else if (w < kSWarp) {
        // ============================================================= softmax
        if constexpr (C::Runs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SoftRegs));
        // Set s (warps 8-11, 12-15) holds rows s RS .. s RS + RS - 1 of the block;
        // thread: cell 32 (w % 4) + lane, the tensor-memory lane of its scores.
        const int q = w & 3, set = (w - kSoft0) >> 2, cell = 32 * q + lane, stid = tid - kSoft0 * 32;
        const int r0 = set * RS;
        const uint32_t t_lane = (uint32_t)(32 * q) << 16;
        Walk it = ms.first;
        const long long total = ms.total;
        uint32_t i = 0; // tile
        uint32_t seg = 0;
        float2 l[RS / 2], z[RS / 2]; // this thread's sums of p and of p vz, by row
#pragma unroll 1
        for (; it.left > 0; ++seg) {
            const int b = it.b, g = it.g, row0 = it.rb * p.rb_rows, n_rows = min(p.rb_rows, p.R - row0);
            const int steps = min(it.left, it.nu - it.u);

            // ----------------------------------------------------- queries
            // Row r: scaled by a power of two so that its largest magnitude lies
            // in [2^14, 2^15), as f16 parts (rows of the B operand), in the order of
            // the K codes; a warp per row, lane = word of codes.
            if (seg > 0) wait(&ms.q_empty, seg - 1);
            // (a rolled loop, the next row loaded ahead: this code runs cold)
            uint4 raw[PARTS];
            int lim = -1;
            long long at = 0;
            auto load_row = [&](int r) {
#pragma unroll
                for (int e = 0; e < PARTS; ++e) raw[e] = make_uint4(0, 0, 0, 0);
                lim = -1;
                if (r >= n_rows) return;
                at = (long long)row_offset(p, b, g, row0 + r);
                lim = p.q_limit ? p.q_limit[(size_t)b * p.T + query_of(p, row0 + r)] : 0x7fffffff;
                if (PARTS == 1 || p.q_bf16) {
                    raw[0] = load_late(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + at) + lane);
                } else {
                    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const float *>(p.q) + at) + 2 * lane;
                    raw[0] = load_late(src);
                    raw[PARTS - 1] = load_late(src + 1);
                }
            };
            load_row(w - kSoft0);
#pragma unroll 1
            for (int r = w - kSoft0; r < 2 * RS; r += kSoftWarps) {
                const uint32_t r4[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
                const uint4 u = raw[PARTS - 1];
                const int lim_r = lim;
                const long long at_r = at;
                load_row(r + kSoftWarps);
                float x[8];
                if (PARTS == 1 || p.q_bf16) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[2 * k] = bf16_bits_to_f32(r4[k] & 0xffffu);
                        x[2 * k + 1] = __uint_as_float(r4[k] & 0xffff0000u);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(r4[k]);
                    x[4] = __uint_as_float(u.x); x[5] = __uint_as_float(u.y);
                    x[6] = __uint_as_float(u.z); x[7] = __uint_as_float(u.w);
                }
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
                const uint32_t e = max(__reduce_max_sync(0xffffffffu, top) >> 23, 15u);
                float up = __uint_as_float((268u - min(e, 254u)) << 23);
                if (p.scale_log2 < 0.f) up = -up; // (the scale below is positive)
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    x[k] *= up;
                    sum += x[k];
                }
                float a[8]; // dimensions 0 4 1 5 2 6 3 7; the odd ones' codes count 16 times
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    a[4 * k] = x[2 * k];
                    a[4 * k + 1] = x[2 * k + 4];
                    a[4 * k + 2] = x[2 * k + 1] * 0.0625f;
                    a[4 * k + 3] = x[2 * k + 5] * 0.0625f;
                }
#pragma unroll
                for (int part = 0; part < PARTS; ++part) {
                    uint32_t wd[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        wd[k] = half2_of(a[2 * k], a[2 * k + 1]);
                        rest2(wd[k], a[2 * k], a[2 * k + 1]);
                    }
                    *reinterpret_cast<uint4 *>(smem + C::q + kmajor_sw128_off(C::col(r) + part * RS, 8 * lane, N)) =
                        make_uint4(wd[0], wd[1], wd[2], wd[3]);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) // the sum of what the parts hold
                    sum -= a[4 * k] + a[4 * k + 1] + 16.f * (a[4 * k + 2] + a[4 * k + 3]);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane == 0) {
                    // (sum(q) goes in 2^24 too small, as the scores come out of the MMA; a
                    // row that is not finite has no scores)
                    RowScore &c = ms.score[r >> 1];
                    RowRef &d = ms.ref[r >> 1];
                    const float xs = e < 255u ? row_scale(p, e) : __uint_as_float(0x7fffffffu);
                    (r & 1 ? c.xs.y : c.xs.x) = xs;
                    (r & 1 ? c.qz.y : c.qz.x) = sum * 0x1p-24f;
                    (r & 1 ? d.nref.y : d.nref.x) = 0.f;
                    (r & 1 ? d.isg.y : d.isg.x) = r < n_rows ? kFresh : 0.f;
                    ms.lim[r] = lim_r;
                    ms.off[seg & 1][r] = at_r;
                    ms.odd[r] = e == 255u;
                    if (r < 2) ms.isg_max[r] = r * RS < n_rows ? kFresh : 0.f;
                }
            }
            fence_proxy_async_smem();
            named_bar(kBarSoft, kSoftThreads);
            mbar_arrive(&ms.q_full);
            // the rows' smallest and largest limit
            int lim_min = 0x7fffffff, lim_max = -1;
            for (int r = lane; r < n_rows; r += 32) {
                const int v = ms.lim[r];
                lim_min = min(lim_min, ms.odd[r] ? -1 : v); // (rows that are not finite: row by row)
                lim_max = max(lim_max, v);
            }
            lim_min = __reduce_min_sync(0xffffffffu, lim_min);
            lim_max = __reduce_max_sync(0xffffffffu, lim_max);
#pragma unroll
            for (int r = 0; r < RS / 2; ++r) l[r] = z[r] = make_float2(0.f, 0.f);
            float acc[2][C::Runs ? RS : 1]; // this thread's dimensions of earlier runs, by half and row
            if constexpr (C::Runs) {
#pragma unroll
                for (int r = 0; r < RS; ++r) acc[0][r] = acc[1][r] = 0.f;
            }

#pragma unroll 1
            for (int step = 0; step < steps; ++step, ++i) {
                const uint32_t pe = i % kPrm, par = i & 1, pb = i % PB;
                wait(&ms.row_full[i % kRow], i / kRow);
                const int pos = ms.pos[i % kRow][cell];
                mbar_arrive(&ms.row_empty[i % kRow]);
                wait(&ms.prm_full[pe], i / kPrm);
                float4 f = ms.prm[pe][cell];
                mbar_arrive(&ms.prm_empty[pe]);
                // a cell that no row sees counts nothing, whatever it holds
                const bool none = pos >= lim_max;
                if (none) f = make_float4(0.f, 0.f, 0.f, 0.f);
                // limits between the rows: row by row
                const bool by_row = lim_min < 0 || __any_sync(0xffffffffu, !none && pos >= lim_min);
                f.w = fmaf(7.5f, f.z, f.w); // (V's codes go in less 7.5)
                // with care where an unseen cell's V scale (as P' takes it) or zero is not
                // finite: a row's sigma may be far below a scale that it does not see
                const bool care = by_row && __any_sync(0xffffffffu, !(fabsf(f.z) * ms.isg_max[set] < INFINITY && fabsf(f.w) < INFINITY));
                const float avs = none ? 0.f : fmaxf(fabsf(f.z), 0x1p-98f);
                const float2 ks = make_float2(f.x, f.x), kz = make_float2(f.y, f.y), vs = make_float2(f.z, f.z),
                             vz = make_float2(f.w, f.w);
                const float bias1 = none ? -INFINITY : 0.f;
                const float2 bias = make_float2(bias1, bias1);
                wait(&ms.s_full[par], i >> 1);
                tc_fence_after();
                {
                    // x: log2 of the probability against the row's reference
                    float2 xl[C::SL / 2]; // the high parts' scores, then the low ones'
                    tmem_ldn<C::SL>(tmem + t_lane + C::colS + par * N + set * C::CS, &xl[0].x);
                    tmem_wait_ld();
                    regs_after_wait<C::SL>(&xl[0].x);
                    tc_fence_before();
                    mbar_arrive(&ms.s_empty[par]);
                    float2 x[RS / 2];
#pragma unroll
                    for (int r = 0; r < RS / 2; ++r) x[r] = PARTS == 2 ? add2(xl[r], xl[(PARTS - 1) * (RS / 2) + r]) : xl[r];
                    float top = -INFINITY;
#pragma unroll
                    for (int r = 0; r < RS / 2; ++r) {
                        const RowScore c = ms.score[(r0 >> 1) + r];
                        const float2 nref = ms.ref[(r0 >> 1) + r].nref;
                        x[r] = fma2(fma2(x[r], ks, fma2(kz, c.qz, bias)), c.xs, nref);
                        top = fmaxf(top, fmaxf(x[r].x, x[r].y));
                    }
                    bool need = avs * ms.isg_max[set] > 0x1p15f || top > 0.f;
                    if (by_row) {
                        need = false;
#pragma unroll
                        for (int r = 0; r < RS; ++r) {
                            float &xr = r & 1 ? x[r >> 1].y : x[r >> 1].x;
                            const RowRef c = ms.ref[(r0 + r) >> 1];
                            const bool see = pos < ms.lim[r0 + r];
                            if (!see) xr = -INFINITY;
                            need |= xr > 0.f || (see && avs * (r & 1 ? c.isg.y : c.isg.x) > 0x1p15f);
                        }
                    }
                    if (named_bar_or(kBarSet + set, kSetThreads, need)) {
                        // --------------------------------- move the references
                        // (a row's first cell, a score above its reference, a V
                        // scale above twice sigma): the tile's true maxima
                        {
                            float m1 = -INFINITY, v1 = 0.f;
                            // (V's scale over the cells that the row sees)
                            const float v_all = by_row ? 0.f : warp_max(none ? 0.f : fabsf(f.z));
#pragma unroll
                            for (int r = 0; r < RS; ++r) {
                                const float xr = r & 1 ? x[r >> 1].y : x[r >> 1].x;
                                const float top_r = warp_max(xr);
                                float v_r = v_all;
                                if (by_row) v_r = warp_max(xr != -INFINITY ? fabsf(f.z) : 0.f);
                                if (lane == r) {
                                    m1 = top_r;
                                    v1 = v_r;
                                }
                            }
                            if (lane < RS) {
                                ms.red[set][0][q][lane] = m1;
                                ms.red[set][1][q][lane] = v1;
                            }
                        }
                        named_bar(kBarSet + set, kSetThreads);
                        bool moved = false;
                        if (q == 0) { // a lane per row
                            float isg_new = 0.f;
                            if (lane < RS) {
                                float m1 = ms.red[set][0][0][lane], v1 = ms.red[set][1][0][lane];
#pragma unroll
                                for (int k = 1; k < 4; ++k) {
                                    m1 = fmaxf(m1, ms.red[set][0][k][lane]);
                                    v1 = fmaxf(v1, ms.red[set][1][k][lane]);
                                }
                                const int r = r0 + lane;
                                RowRef &c = ms.ref[r >> 1];
                                float &nref = r & 1 ? c.nref.y : c.nref.x, &isg = r & 1 ? c.isg.y : c.isg.x;
                                float delta = 0.f, fac = 1.f, ofac = 1.f;
                                isg_new = isg;
                                if (m1 > -INFINITY && isg > 0.f) {
                                    const bool fresh = isg == kFresh;
                                    if (fresh || m1 > 0.f) delta = -m1 - kSlackLog2;
                                    if (!fresh) fac = fast_exp2(delta);
                                    // sigma: a power of two not below the largest scale so far
                                    const uint32_t up = (__float_as_uint(fmaxf(v1, 0x1p-99f)) + 0x7fffffu) & 0x7f800000u;
                                    isg_new = fminf(isg, __uint_as_float((268u << 23) - up));
                                    if (!fresh) ofac = fac * (isg_new / isg);
                                    nref += delta;
                                    isg = isg_new;
                                }
                                ms.delta[r] = delta;
                                ms.fac[r] = fac;
                                ms.ofac[r] = ofac;
                                moved = ofac != 1.f;
                            }
                            isg_new = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(isg_new)));
                            if (lane == 0) ms.isg_max[set] = isg_new;
                        }
                        moved = named_bar_or(kBarSet + set, kSetThreads, moved);
#pragma unroll
                        for (int r = 0; r < RS / 2; ++r) {
                            const float2 fac = *reinterpret_cast<const float2 *>(&ms.fac[r0 + 2 * r]);
                            x[r] = add2(x[r], *reinterpret_cast<const float2 *>(&ms.delta[r0 + 2 * r]));
                            l[r] = mul2(l[r], fac);
                            z[r] = mul2(z[r], fac);
                        }
                        if (moved && step > 0) {
                            // the sums so far, once P.V of the tile before is done
                            wait(&ms.p_empty[(i - 1) % PB], (i - 1) / PB);
                            tc_fence_after();
#pragma unroll 1
                            for (int k = 0; k < 2 * PARTS; ++k) {
                                const uint32_t ta = tmem + t_lane + C::colO + (k & 1) * N + set * C::CS + (k >> 1) * RS;
                                float v[RS];
                                tmem_ldn<RS>(ta, v);
                                tmem_wait_ld();
                                regs_after_wait<RS>(v);
#pragma unroll
                                for (int r = 0; r < RS; ++r) v[r] *= ms.ofac[r0 + r];
                                tmem_stn<RS>(ta, v);
                            }
                            tmem_wait_st();
                            if constexpr (C::Runs) {
#pragma unroll
                                for (int r = 0; r < RS; ++r) {
                                    acc[0][r] *= ms.ofac[r0 + r];
                                    acc[1][r] *= ms.ofac[r0 + r];
                                }
                            }
                        }
                    }
                    if constexpr (C::Runs) {
                        if (step > 0 && step % C::Run == 0) { // a run's sums, once its last P.V is done
                            wait(&ms.p_empty[(i - 1) % PB], (i - 1) / PB);
                            tc_fence_after();
#pragma unroll
                            for (int k = 0; k < 2 * PARTS; ++k) {
                                float v[RS];
                                tmem_ldn<RS>(tmem + t_lane + C::colO + (k & 1) * N + set * C::CS + (k >> 1) * RS, v);
                                tmem_wait_ld();
                                regs_after_wait<RS>(v);
#pragma unroll
                                for (int r = 0; r < RS; ++r) acc[k & 1][r] += v[r];
                            }
                        }
                    }
                    if (i >= PB) wait(&ms.p_empty[pb], i / PB - 1);
                    // ---- P' = p vs 2^14 / sigma, as f16 parts, into the B operand of
                    // the P.V MMA, rows contiguous (MN-major with the 32-byte
                    // swizzle): the cell's rows of the set are whole 16-byte pieces;
                    // this thread's sums
                    uint32_t h[C::CS / 2];
#pragma unroll
                    for (int r = C::CR / 2; r < C::CS / 2; ++r) h[r] = 0u;
#pragma unroll
                    for (int r = 0; r < RS / 2; ++r) {
                        const float2 isg = ms.ref[(r0 >> 1) + r].isg;
                        const float2 pe2 = make_float2(fast_exp2(x[r].x), fast_exp2(x[r].y));
                        float2 pv;
                        l[r] = add2(l[r], pe2);
                        if (!care) {
                            z[r] = fma2(pe2, vz, z[r]);
                            pv = mul2(pe2, mul2(vs, isg));
                        } else { // (what an unseen cell holds must not reach the row)
                            float2 &zr = z[r];
                            pv.x = x[r].x != -INFINITY ? pe2.x * (f.z * isg.x) : 0.f;
                            pv.y = x[r].y != -INFINITY ? pe2.y * (f.z * isg.y) : 0.f;
                            if (x[r].x != -INFINITY) zr.x = fmaf(pe2.x, f.w, zr.x);
                            if (x[r].y != -INFINITY) zr.y = fmaf(pe2.y, f.w, zr.y);
                        }
                        h[r] = half2_of(pv.x, pv.y);
                        if (PARTS == 2) {
                            rest2(h[r], pv.x, pv.y);
                            h[(PARTS - 1) * (RS / 2) + r] = half2_of(pv.x, pv.y);
                        }
                    }
                    uint8_t *dst = smem + C::p + pb * (N * 256u) + (cell >> 3) * 256 + (cell & 7) * 32;
#pragma unroll
                    for (int c = 0; c < C::CS / 8; ++c) {
                        const uint32_t n8 = set * (C::CS / 8) + c; // 16-byte piece of the cell's columns
                        *reinterpret_cast<uint4 *>(dst + (n8 >> 1) * 4096u + (((n8 & 1u) ^ ((cell >> 2) & 1u)) << 4)) =
                            make_uint4(h[4 * c], h[4 * c + 1], h[4 * c + 2], h[4 * c + 3]);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&ms.p_full[pb]);
            }

            // --------------------------------------------- the segment's sums
            {
                // (eight rows at a time)
#pragma unroll
                for (int c = 0; c < RS; c += 8) {
                    float lx[8], zx[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const bool in = c + r < RS;
                        const float2 l2 = l[in ? (c + r) >> 1 : 0], z2 = z[in ? (c + r) >> 1 : 0];
                        lx[r] = in ? (r & 1 ? l2.y : l2.x) : 0.f;
                        zx[r] = in ? (r & 1 ? z2.y : z2.x) : 0.f;
                    }
                    const float ls = warp_sum_rows<8>(lx, lane), zs = warp_sum_rows<8>(zx, lane);
                    if (lane < 8 && c + lane < RS) {
                        ms.red[set][0][q][c + lane] = ls;
                        ms.red[set][1][q][c + lane] = zs;
                    }
                }
            }
            named_bar(kBarSet + set, kSetThreads);
            const bool direct = it.u == 0 && steps == it.nu;
            const int slot = 2 * (int)blockIdx.x + (seg == 0 ? 0 : 1);
            if (cell < RS) {
                float L = 0.f, Z = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    L += ms.red[set][0][k][cell];
                    Z += ms.red[set][1][k][cell];
                }
                const int r = r0 + cell;
                const RowRef &c = ms.ref[r >> 1];
                const float isg = r & 1 ? c.isg.y : c.isg.x, ref = -(r & 1 ? c.nref.y : c.nref.x);
                const float inv = direct ? (L == 0.f ? 0.f : 1.f / L) : 1.f; // (NaN: a row that is not finite)
                ms.fin[r] = 0x1p9f / isg * inv;
                ms.zsum[r] = Z * inv;
                if (!direct && r < n_rows) p.part_ml[(size_t)slot * kMaxRows + r] = make_float2(L == 0.f ? -INFINITY : ref, L);
            }
            if (it.u == 0 && stid == 0) {
                const long long pair = ((long long)b * p.pool.G + g) * p.n_rb + it.rb;
                p.info[pair] = make_int2(slot, direct ? 1 : parts_of(it, total));
            }
            named_bar(kBarSoft, kSoftThreads);
            // O: tensor-memory lane = dimension of half `set` (in the codes' order),
            // columns = rows
            wait(&ms.o_full, seg);
            tc_fence_after();
            if constexpr (C::Runs) {
                if (steps > C::Run) { // earlier runs' sums to the last one's
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float v[RS];
                        const uint32_t ta = tmem + t_lane + C::colO + k * N + set * C::CS;
                        tmem_ldn<RS>(ta, v);
                        tmem_wait_ld();
                        regs_after_wait<RS>(v);
#pragma unroll
                        for (int r = 0; r < RS; ++r) v[r] += acc[k][r];
                        tmem_stn<RS>(ta, v);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    named_bar(kBarSoft, kSoftThreads);
                    tc_fence_after();
                }
            }
            const int dim = 128 * set + (cell & ~7) + ((cell & 7) >> 1) + 4 * (cell & 1);
            constexpr int RC = RS % 8 == 0 ? 8 : RS % 4 == 0 ? 4 : 2; // rows at a time
#pragma unroll 1
            for (int c0 = 0; c0 < 2 * RS && c0 < n_rows; c0 += RC) {
                float v[RC];
                const uint32_t ta = tmem + t_lane + C::colO + set * N + C::col(c0);
                tmem_ldn<RC>(ta, v);
                if constexpr (PARTS == 2) {
                    float lo[RC];
                    tmem_ldn<RC>(ta + RS, lo);
                    tmem_wait_ld();
                    regs_after_wait<RC>(v);
                    regs_after_wait<RC>(lo);
#pragma unroll
                    for (int r = 0; r < RC; ++r) v[r] += lo[r];
                } else {
                    tmem_wait_ld();
                    regs_after_wait<RC>(v);
                }
#pragma unroll
                for (int r = 0; r < RC; ++r) {
                    if (c0 + r >= n_rows) break;
                    const float o = fmaf(v[r], ms.fin[c0 + r], ms.zsum[c0 + r]);
                    if (direct) {
                        const long long at = ms.off[seg & 1][c0 + r] + dim;
                        if (p.out_bf16) static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16(o);
                        else static_cast<float *>(p.out)[at] = o;
                    } else {
                        p.part_o[((size_t)slot * kMaxRows + c0 + r) * kHeadDim + dim] = o;
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(&ms.o_empty);
            walk_next(p, it, steps);
        }
    } else {
        if constexpr (C::Runs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::RestRegs));
        if (w == kSWarp) {
            // ============================================================ S = K.Q^T
            // All lanes run the loop (every value is uniform), one issues.
            const bool leader = elect_one();
            const uint32_t idesc = idesc_f16(128, N, false, false, false, false);
            Walk it = ms.first;
            uint32_t i = 0;
#pragma unroll 1
            for (uint32_t seg = 0; it.left > 0; ++seg) {
                const int steps = min(it.left, it.nu - it.u);
                wait(&ms.q_full, seg);
#pragma unroll 1
                for (int step = 0; step < steps; ++step, ++i) {
                    const uint32_t kb = i & 1;
                    wait(&ms.k_full[kb], i >> 1);
                    if (i >= 2) wait(&ms.s_empty[kb], (i >> 1) - 1);
                    tc_fence_after();
                    const uint64_t qd = smem_desc(smem_u32(smem + C::q), 16, 1024);
                    const uint32_t sd = tmem + C::colS + kb * N;
                    if (leader) {
#pragma unroll 4
                        for (int kk = 0; kk < kHeadDim / 16; ++kk)
                            mma_f16_ts(sd, tmem + 128u * kb + 8u * kk,
                                       qd + (uint64_t)(((uint32_t)(kk >> 2) * N * 128u + (uint32_t)(kk & 3) * 32u) >> 4), idesc, kk > 0);
                        mma_commit(&ms.k_empty[kb]);
                        mma_commit(&ms.s_full[kb]);
                    }
                    __syncwarp();
                }
                if (leader) mma_commit(&ms.q_empty);
                __syncwarp();
                walk_next(p, it, steps);
            }
            // before the CTA leaves (also after a time-out): every MMA complete
            if (leader) mma_commit(&ms.s_done);
            __syncwarp();
            mbar_wait(&ms.s_done, 0, kDrainCycles);
        } else if (w == kPvWarp) {
            // ======================================================= O += V^T.P'^T
            const bool leader = elect_one();
            const uint32_t idesc = idesc_f16(128, N, false, false, true, true);
            Walk it = ms.first;
            uint32_t i = 0;
#pragma unroll 1
            for (uint32_t seg = 0; it.left > 0; ++seg) {
                const int steps = min(it.left, it.nu - it.u);
                if (seg > 0) wait(&ms.o_empty, seg - 1);
#pragma unroll 1
                for (int step = 0; step < steps; ++step, ++i) {
                    const uint32_t pb = i % PB;
                    wait(&ms.p_full[pb], i / PB);
                    const uint64_t ad0 = smem_desc(smem_u32(smem + C::v), 16384, 1024);
                    // 16 columns 4096 bytes apart, 8 cells 256
                    const uint64_t bd0 = smem_desc(smem_u32(smem + C::p) + pb * (N * 256u), 4096, 256, kLayoutSw32);
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        wait(&ms.v_full[half], i);
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int kk = 4 * half; kk < 4 * half + 4; ++kk) {
                                const uint64_t bd = bd0 + (uint64_t)((512u * kk) >> 4);
#pragma unroll
                                for (int hh = 0; hh < 2; ++hh)
                                    mma_f16_ss(tmem + C::colO + hh * N, ad0 + (uint64_t)((32768u * hh + 2048u * kk) >> 4), bd, idesc,
                                               ((C::Runs ? step % C::Run : step) > 0 || kk > 0) ? 1u : 0u);
                            }
                            mma_commit(&ms.v_empty[half]);
                        }
                        __syncwarp();
                    }
                    if (leader) {
                        mma_commit(&ms.p_empty[pb]);
                        if (step == steps - 1) mma_commit(&ms.o_full);
                    }
                    __syncwarp();
                }
                walk_next(p, it, steps);
            }
            if (leader) mma_commit(&ms.pv_done);
            __syncwarp();
            mbar_wait(&ms.pv_done, 0, kDrainCycles);
        } else {
            // ============================================================== lookup
            // Lane l of warp k resolves cells 64 k + l and + 32 of every tile, one
            // stage per tile: the list entry two tiles, the page entry one tile before
            // the row in the pool, which goes to the ring.
            const int c0 = 64 * (w - kRes0) + lane;
            Walk head = ms.first;
            const int tiles = head.left;
            const int cap = p.pool.page_table_len * p.pool.page_cells;
            int a_pos[2] = {0, 0}, c_pos[2] = {0, 0}, c_entry[2] = {0, 0}, c_off[2] = {0, 0};
            int a_b = 0, a_g = 0, c_b = 0, c_g = 0;
            bool a_in[2] = {false, false}, c_in[2] = {false, false};
#pragma unroll 1
            for (int t = -2; t < tiles; ++t) {
                if (t >= 0) { // row
                    const uint32_t e = (uint32_t)t % kRow;
                    if (t >= kRow) wait(&ms.row_empty[e], (uint32_t)t / kRow - 1);
                    const size_t base = kv4_row(p.pool, c_b, c_g, 0);
                    uint32_t bad = 0;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        int slot = -1;
                        if (c_in[k]) {
                            uint32_t why = 0;
                            slot = kv4_slot(p.pool, c_entry[k], c_off[k], why);
                            bad |= why;
                        }
                        // (where there is no cell, the row of slot 0: any does)
                        ms.row[e][c0 + 32 * k] = (uint32_t)(base + max(slot, 0));
                        ms.pos[e][c0 + 32 * k] = slot >= 0 ? c_pos[k] : 0x7fffffff;
                    }
                    raise(p, bad & ~QSA_STATUS_NOT_RESIDENT);
                    mbar_arrive(&ms.row_full[e]);
                }
                c_b = a_b;
                c_g = a_g;
#pragma unroll
                for (int k = 0; k < 2; ++k) { // page entry
                    c_in[k] = a_in[k];
                    c_pos[k] = a_pos[k];
                    if (c_in[k] && (a_pos[k] < 0 || a_pos[k] >= cap)) {
                        raise(p, QSA_STATUS_BAD_POSITION);
                        c_in[k] = false;
                    }
                    if (c_in[k]) {
                        const int page = p.page_shift >= 0 ? a_pos[k] >> p.page_shift : a_pos[k] / p.pool.page_cells;
                        c_off[k] = a_pos[k] - page * p.pool.page_cells;
                        c_entry[k] = p.pool.page_table[(size_t)a_b * p.pool.page_table_len + page];
                    }
                    a_in[k] = false;
                }
                if (head.left > 0) { // list entry
                    const int i0 = head.u * kTile + c0;
                    a_b = head.b;
                    a_g = head.g;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int i = i0 + 32 * k;
                        a_in[k] = i < head.n;
                        if (a_in[k]) a_pos[k] = p.sel ? p.sel[(long long)head.start + i] : i;
                    }
                    walk_next(p, head, 1);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == kSWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int RS, int PARTS>
cudaError_t launch(const AttnParams &p, int grid, cudaStream_t stream)
{
    auto kernel = qsa_kv4_attn_kernel<RS, PARTS>;
    constexpr int bytes = (int)Cfg<RS, PARTS>::total;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// By rows of a block; each number of parts in a translation unit of its own.
cudaError_t launch_single(const AttnParams &p, int rows, int grid, cudaStream_t stream);
cudaError_t launch_split(const AttnParams &p, int rows, int grid, cudaStream_t stream);
// Blocks of 128 rows, bf16 queries and output.
cudaError_t launch_wide(const AttnParams &p, int grid, cudaStream_t stream);

} // namespace kv4
} // namespace qsa

// qsa_kv4.cu -- qsa_kv4_append and qsa_kv4_read: K and V rows into 4-bit cells
// and back.
//
// Append, per row of 256 values x (K and V each): zero z = min x, scale
// s = (max x - z) * (1/15), code u = (x - z) / s rounded to nearest, ties to even.
// Read: s u + z.
//
// Both are bound by HBM (append: 2 KB of fp32 or 1 KB of bf16 in, 272 bytes
// out per cell and KV head; read the reverse).  A warp takes one (cell, KV head)
// at a time, the next one's rows loaded before the current one's are worked on
// (two in flight per warp): lane l holds elements 8l..8l+7 of a row, so a row is
// one 16- or 32-byte load per lane and its codes one 4-byte word per lane (128
// contiguous bytes per warp store), and minimum and maximum are two warp
// reductions.  65,536 (cell, KV head) rows: append of fp32 25.6 us (5.9 TB/s), of
// bf16 20.2 us (4.2 TB/s; bound by its instructions, a third of them for quotients
// on a border between codes, which bf16 values often give); read to fp32 29 us (5.2
// TB/s, writes mostly), to bf16 16.9 us (5.0 TB/s; 12.9 where the output fits the L2).
#include "qsa_kv4.cuh"
#include "qsa_sm100.cuh"

namespace qsa {
namespace {

constexpr int kKv4Warps = 8;
constexpr int kKv4Blocks = 4; // resident per SM (64 registers)

struct Kv4RowsParams {
    Kv4Pool pool;
    const void *k_new, *v_new; // append: [n_seq][n_new][G][D]
    void *k_out, *v_out;       // read: the same shape
    const int32_t *positions;  // [n_seq][n_new]
    uint8_t *codes;
    float4 *scale;
    uint32_t *status;
    uint32_t items, n_new; // (cell, KV head) rows; new cells per sequence
};

// Elements 8*lane .. 8*lane + 7 of a row of 256, as they are stored.
template <bool BF16>
struct Row8 {
    uint32_t w[BF16 ? 4 : 8];

    __device__ __forceinline__ void load(const void *base, size_t row, int lane)
    {
        if constexpr (BF16) {
            const uint4 a = load_late(static_cast<const uint4 *>(base) + row * (kHeadDim / 8) + lane);
            w[0] = a.x;
            w[1] = a.y;
            w[2] = a.z;
            w[3] = a.w;
        } else {
            load_late256(static_cast<const uint8_t *>(base) + row * kHeadDim * 4 + 32 * lane, w);
        }
    }

    __device__ __forceinline__ void values(float *x) const
    {
        if constexpr (BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16_bits_to_f32(w[i] & 0xffffu);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        }
    }
};

// Code of x whose quotient lies about halfway between u and u + 1; d = fl(x - z).
__device__ __forceinline__ uint32_t at_border(float x, float z, float d, float s, float u)
{
    // x - z = d + e exactly (two-sum), (u + 1/2) s = a + b exactly (fused
    // multiply-add); d and a nearly agree, so their difference is exact too
    const float v = __fsub_rn(d, x);
    const float e = __fsub_rn(__fsub_rn(x, __fsub_rn(d, v)), __fadd_rn(z, v));
    const float t = u + 0.5f, a = __fmul_rn(t, s), b = __fmaf_rn(t, s, -a);
    const float r = __fadd_rn(__fsub_rn(d, a), __fsub_rn(e, b));
    const uint32_t c = (uint32_t)u;
    return c + (r > 0.f || (r == 0.f && (c & 1u)) ? 1u : 0u); // a tie goes to the even code
}

// Code of x by a division in 64 bits, for the scales that the fast way cannot take.
__device__ __noinline__ uint32_t code_f64(float x, float z, float s)
{
    const double u = rint(((double)x - (double)z) / (double)s);
    return (uint32_t)fmin(fmax(u, 0.0), 15.0);
}

// x[i], by selects: registers cannot be indexed, and an array that is would live
// in local memory.
__device__ __forceinline__ float pick8(const float *x, int i)
{
    float r;
    asm("{\n\t.reg .pred a, b, c;\n\t.reg .f32 s, t, u, v;\n\t.reg .b32 m;\n\t"
        "and.b32 m, %1, 1;\n\tsetp.ne.u32 a, m, 0;\n\tand.b32 m, %1, 2;\n\tsetp.ne.u32 b, m, 0;\n\t"
        "and.b32 m, %1, 4;\n\tsetp.ne.u32 c, m, 0;\n\t"
        "selp.f32 s, %3, %2, a;\n\tselp.f32 t, %5, %4, a;\n\tselp.f32 u, %7, %6, a;\n\tselp.f32 v, %9, %8, a;\n\t"
        "selp.f32 s, t, s, b;\n\tselp.f32 u, v, u, b;\n\tselp.f32 %0, u, s, c;\n\t}"
        : "=f"(r)
        : "r"(i), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// The lane's 8 codes as one word (element 2i in the low, 2i + 1 in the high
// bits of byte i), and the row's scale and zero.
__device__ __forceinline__ uint32_t quantise8(const float *x, float &scale, float &zero)
{
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
    asm volatile("redux.sync.min.f32 %0, %0, 0xffffffff;" : "+f"(lo));
    asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(hi));
    zero = lo;
    scale = __fmul_rn(__fsub_rn(hi, lo), 1.f / 15.f);
    if (!(scale > 0.f)) {
        scale = 0.f;
        return 0u;
    }
    uint32_t w = 0;
    if (scale > 0x1p-90f && scale < 0x1p120f) { // the same for the whole warp
        // The fp32 quotient is within 2^-19 of the exact one (at most 15: a rounding of
        // x - z, one of the product, the reciprocal's 1 ulp), so it rounds the same way (here by adding 1.5 * 2^23, whose unit in the last
        // place is 1) unless it lies within 1e-4 of a border: one element in a
        // hundred of bf16 rows lies on one.
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
        const float2 lo2 = make_float2(-lo, -lo), inv2 = make_float2(inv, inv), magic = make_float2(12582912.f, 12582912.f),
                     less = make_float2(-12582912.f, -12582912.f), neg = make_float2(-1.f, -1.f);
        // The codes c are put together as floats while that is exact (FMAs where
        // shifts and masks would take twice as many instructions):
        // c0 + 16 c1 + 256 (c2 + 16 c3) + 1.5 * 2^23 has them in its low 16 bits.
        uint32_t half[2], near = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 q0 = mul2(add2(make_float2(x[4 * h], x[4 * h + 1]), lo2), inv2);
            const float2 q1 = mul2(add2(make_float2(x[4 * h + 2], x[4 * h + 3]), lo2), inv2);
            const float2 m0 = add2(q0, magic), m1 = add2(q1, magic);
            const float2 c0 = add2(m0, less), c1 = add2(m1, less);
            const float2 r0 = fma2(c0, neg, q0), r1 = fma2(c1, neg, q1);
            half[h] = __float_as_uint(fmaf(256.f, fmaf(16.f, c1.y, c1.x), fmaf(16.f, c0.y, m0.x)));
            const float off = fmaxf(fmaxf(fabsf(r0.x), fabsf(r0.y)), fmaxf(fabsf(r1.x), fabsf(r1.y)));
            if (off > 0.4999f)
                near |= ((fabsf(r0.x) > 0.4999f ? 1u : 0u) | (fabsf(r0.y) > 0.4999f ? 2u : 0u) |
                         (fabsf(r1.x) > 0.4999f ? 4u : 0u) | (fabsf(r1.y) > 0.4999f ? 8u : 0u))
                        << (4 * h);
        }
        w = __byte_perm(half[0], half[1], 0x5410);
        while (near) { // elements near a border, seldom two in a lane
            const int i = __ffs(near) - 1;
            near &= near - 1;
            const float xi = pick8(x, i), d = __fsub_rn(xi, lo), v = __fmul_rn(d, inv);
            const uint32_t c = at_border(xi, lo, d, scale, rintf(v - 0.5f));
            w = (w & ~(15u << (4 * i))) | c << (4 * i);
        }
        return w;
    }
    // a scale for which the reciprocal or the terms of the test could leave the fp32 range
#pragma unroll 1
    for (int i = 0; i < 8; ++i) w |= code_f64(pick8(x, i), lo, scale) << (4 * i);
    return w;
}

// The rows in the pools of a warp's next 32 items (one item = one cell and KV
// head): lane l looks up item first + l * stride, so that the divisions and the
// dependent loads of positions and page tables are paid once in 32 items.  -1
// where the cell has no row; status bits outside `quiet` are raised.
struct ItemRows {
    long long row;
    int at;

    __device__ __forceinline__ long long next(const Kv4RowsParams &p, uint32_t i, uint32_t stride, int lane, uint32_t quiet)
    {
        if (at == 32) { // the same for the whole warp
            at = 0;
            row = -1;
            const uint32_t mine = i + (uint32_t)lane * stride; // below 2^31 + 31 * stride
            if (mine < p.items) {
                const uint32_t cell = mine / (uint32_t)p.pool.G;
                const int b = (int)(cell / p.n_new);
                uint32_t bad = 0;
                const int slot = kv4_resolve(p.pool, b, p.positions[cell], bad);
                bad &= ~quiet;
                if (bad && p.status) atomicOr(p.status, bad);
                if (slot >= 0) row = (long long)kv4_row(p.pool, b, (int)(mine - cell * (uint32_t)p.pool.G), slot);
            }
            __syncwarp();
        }
        return __shfl_sync(0xffffffffu, row, at++);
    }
};

template <bool BF16>
__global__ void __launch_bounds__(kKv4Warps * 32, kKv4Blocks) qsa_kv4_append_kernel(const Kv4RowsParams p)
{
    const int lane = threadIdx.x & 31;
    const uint32_t stride = gridDim.x * kKv4Warps;
    // (Launched early behind a kernel that allows it; whatever that kernel wrote is read
    // behind the wait, by loads that stay there.)
    cudaGridDependencySynchronize();
    uint32_t i = blockIdx.x * kKv4Warps + (threadIdx.x >> 5);
    Row8<BF16> k, v;
    if (i < p.items) {
        k.load(p.k_new, i, lane);
        v.load(p.v_new, i, lane);
    }
    ItemRows rows{-1, 32};
    while (i < p.items) {
        const long long row = rows.next(p, i, stride, lane, 0u);
        const uint32_t next = i + stride;
        Row8<BF16> kn, vn;
        if (next < p.items) {
            kn.load(p.k_new, next, lane);
            vn.load(p.v_new, next, lane);
        }
        if (row >= 0) { // the whole warp agrees
            float4 s;
            float x[8];
            k.values(x);
            const uint32_t kc = quantise8(x, s.x, s.y);
            v.values(x);
            const uint32_t vc = quantise8(x, s.z, s.w);
            uint32_t *dst = reinterpret_cast<uint32_t *>(p.codes + (size_t)row * QSA_KV4_CODE_BYTES);
            dst[lane] = kc;
            dst[32 + lane] = vc;
            if (lane == 0) p.scale[row] = s;
        }
        k = kn;
        v = vn;
        i = next;
    }
}

// The lane's 8 values of a word of codes.
template <bool BF16>
__device__ __forceinline__ void store8(void *base, size_t row, int lane, uint32_t w, float scale, float zero)
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(scale, (float)((w >> (4 * i)) & 15u), zero);
    if (BF16) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(base) + row * kHeadDim * 2 + 16 * lane) =
            make_uint4(o[0], o[1], o[2], o[3]);
    } else {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                     ::"l"(static_cast<uint8_t *>(base) + row * kHeadDim * 4 + 32 * lane), "r"(__float_as_uint(x[0])),
                       "r"(__float_as_uint(x[1])), "r"(__float_as_uint(x[2])), "r"(__float_as_uint(x[3])),
                       "r"(__float_as_uint(x[4])), "r"(__float_as_uint(x[5])), "r"(__float_as_uint(x[6])),
                       "r"(__float_as_uint(x[7]))
                     : "memory");
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kKv4Warps * 32, kKv4Blocks) qsa_kv4_read_kernel(const Kv4RowsParams p)
{
    const int lane = threadIdx.x & 31;
    const uint32_t stride = gridDim.x * kKv4Warps;
    cudaGridDependencySynchronize();
    uint32_t i = blockIdx.x * kKv4Warps + (threadIdx.x >> 5);
    uint32_t kc = 0, vc = 0;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    ItemRows rows{-1, 32};
    auto load = [&](uint32_t at) {
        const long long row = rows.next(p, at, stride, lane, QSA_STATUS_NOT_RESIDENT); // a masked cell reads as zeros
        kc = vc = 0u;
        s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row >= 0) {
            const uint32_t *src = reinterpret_cast<const uint32_t *>(p.codes + (size_t)row * QSA_KV4_CODE_BYTES);
            kc = src[lane];
            vc = src[32 + lane];
            s = p.scale[row];
        }
    };
    if (i < p.items) load(i);
    while (i < p.items) {
        const uint32_t k0 = kc, v0 = vc;
        const float4 s0 = s;
        const uint32_t next = i + stride;
        if (next < p.items) load(next);
        store8<BF16>(p.k_out, i, lane, k0, s0.x, s0.y);
        store8<BF16>(p.v_out, i, lane, v0, s0.z, s0.w);
        i = next;
    }
}

qsa_status run_rows(Kv4RowsParams &p, const qsa_shape *shape, int n_seq, int n_new, int dtype,
                    void (*f32)(Kv4RowsParams), void (*bf16)(Kv4RowsParams), void *stream)
{
    const long long cells = (long long)n_seq * n_new;
    if (cells == 0) return QSA_OK;
    if (cells >= (1ll << 31) || cells * shape->n_kv_heads >= (1ll << 31)) return QSA_ERR_UNSUPPORTED;
    const long long items = cells * shape->n_kv_heads;
    p.items = (uint32_t)items;
    p.n_new = (uint32_t)n_new;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return QSA_ERR_CUDA;
    // as many blocks as are resident at once (every warp strides over the rows)
    const long long need = (items + kKv4Warps - 1) / kKv4Warps, cap = (long long)sms * kKv4Blocks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(need < cap ? need : cap));
    cfg.blockDim = dim3(kKv4Warps * 32);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dtype == QSA_BF16 ? bf16 : f32, p) == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}

qsa_status check_rows(const qsa_shape *shape, int n_seq, int n_pools, int n_new, int dtype, const void *k,
                      const void *v, const int32_t *positions, const int32_t *page_table, const void *kv_pool,
                      const void *kv_scale, const uint32_t *status)
{
    const qsa_status st = kv4_check(shape, n_seq, n_pools);
    if (st != QSA_OK) return st;
    if (n_new < 0 || (dtype != QSA_F32 && dtype != QSA_BF16)) return QSA_ERR_INVALID_ARG;
    if (n_seq == 0 || n_new == 0) return QSA_OK; // nothing to do, no buffers needed
    if (!k || !v || !positions || !page_table || !kv_pool || !kv_scale) return QSA_ERR_INVALID_ARG;
    if (!kv4_aligned(k, 32) || !kv4_aligned(v, 32) || !kv4_aligned(positions, 4) || !kv4_aligned(page_table, 4) ||
        !kv4_aligned(kv_pool, 32) || !kv4_aligned(kv_scale, 16) || (status && !kv4_aligned(status, 4)))
        return QSA_ERR_INVALID_ARG;
    if (k == kv_pool || v == kv_pool || k == kv_scale || v == kv_scale || kv_pool == kv_scale)
        return QSA_ERR_INVALID_ARG;
    return QSA_OK;
}

} // namespace
} // namespace qsa

extern "C" qsa_status qsa_kv4_append(const qsa_shape *shape, int32_t n_seq, int32_t n_pools, int32_t n_new,
                                     int32_t kv_dtype, const void *k_new, const void *v_new,
                                     const int32_t *positions, const int32_t *page_table, uint8_t *kv_pool,
                                     float *kv_scale, uint32_t *status, void *stream)
{
    const qsa_status st = qsa::check_rows(shape, n_seq, n_pools, n_new, kv_dtype, k_new, v_new, positions,
                                          page_table, kv_pool, kv_scale, status);
    if (st != QSA_OK) return st;
    qsa::Kv4RowsParams p{};
    p.pool = qsa::kv4_pool(shape, n_pools, page_table);
    p.k_new = k_new;
    p.v_new = v_new;
    p.positions = positions;
    p.codes = kv_pool;
    p.scale = reinterpret_cast<float4 *>(kv_scale);
    p.status = status;
    return qsa::run_rows(p, shape, n_seq, n_new, kv_dtype, qsa::qsa_kv4_append_kernel<false>,
                         qsa::qsa_kv4_append_kernel<true>, stream);
}

extern "C" qsa_status qsa_kv4_read(const qsa_shape *shape, int32_t n_seq, int32_t n_pools, int32_t n_cells,
                                   int32_t out_dtype, const int32_t *positions, const int32_t *page_table,
                                   const uint8_t *kv_pool, const float *kv_scale, void *k_out, void *v_out,
                                   uint32_t *status, void *stream)
{
    const qsa_status st = qsa::check_rows(shape, n_seq, n_pools, n_cells, out_dtype, k_out, v_out, positions,
                                          page_table, kv_pool, kv_scale, status);
    if (st != QSA_OK) return st;
    if (k_out && k_out == v_out) return QSA_ERR_INVALID_ARG;
    qsa::Kv4RowsParams p{};
    p.pool = qsa::kv4_pool(shape, n_pools, page_table);
    p.k_out = k_out;
    p.v_out = v_out;
    p.positions = positions;
    p.codes = const_cast<uint8_t *>(kv_pool);
    p.scale = reinterpret_cast<float4 *>(const_cast<float *>(kv_scale));
    p.status = status;
    return qsa::run_rows(p, shape, n_seq, n_cells, out_dtype, qsa::qsa_kv4_read_kernel<false>,
                         qsa::qsa_kv4_read_kernel<true>, stream);
}

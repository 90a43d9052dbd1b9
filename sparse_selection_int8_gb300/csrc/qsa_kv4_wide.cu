// qsa_kv4_wide.cu -- the attention kernel over 4-bit cells for wide windows
// (many query rows per KV head, bf16 queries and output).
//
// The mathematics, the work list and the partials are those of
// qsa_kv4_attn.cu; here the MMA's M dimension holds 128 query rows instead of
// 128 cells:
//   S [rows][cells] = Q . K^T   Q (f16, scaled by row) resident, K codes
//   O [rows][dims] += P' . V    P' = p vs / sigma in tensor memory, V codes
// so a tile's codes are expanded once for 128 rows (the other kernel's for 32),
// and a warp holds half the scores of 32 rows.  Scores and P' share two
// tensor-memory buffers, so S of the next tile runs while the softmax works on
// this one.  A tile's exponentials are formed with the references that the rows
// have; only where a score or a V scale outgrows one (the first tiles, mostly) are
// they formed again behind the maxima of both halves.
//
// A tile takes 2.1 us, twice what the tensor cores need: 3.8 K cycles of shared
// memory, of which the operands' reads (192 KB) are 1.5 K, the expanded codes'
// stores 1 K and the softmax's reads of scales and zeros most of the rest (ncu),
// behind the softmax's own latency.  3,084 rows of two heads over 8,000 cells: 64 us
// (50.5 GFLOP, 41% of the measured tensor rate), where blocks of 32 rows take 137.
// A softmax thread per half row, which reads four times as many scales, took 68.
#include "qsa_kv4_attn.cuh"

namespace qsa {
namespace kv4 {
namespace {

constexpr int kWSoft = 8, kWCodes = 8; // softmax warps, expanding warps (four for K, four for V)
constexpr int kWMma = kWSoft + kWCodes, kWRes = kWMma + 1; // issues the MMAs; two look the cells up
constexpr int kWideThreads = (kWRes + 3) * 32; // 640, the last warp idle: five warpgroups of 128 threads,
// launched with 96 registers a thread and split by what the roles hold.
constexpr int kSoftRegs = 152, kCodeRegs = 64, kRestRegs = 48;
static_assert(2 * kSoftRegs + 2 * kCodeRegs + kRestRegs <= 5 * 96, "registers of the launch");
constexpr int kWRow = 4, kWPrm = 3;                                  // ring entries
constexpr uint32_t kOperand = kTile * kHeadDim * 2;                  // 64 KB: Q, K, V

struct WideMisc {
    float4 k[kWPrm][kTile / 2];  // scales, then zeros, of two neighbouring cells
    float4 v[kWPrm][kTile / 2];
    int32_t pos[kWPrm][kTile];   // 2^31 - 1 where there is no cell
    int32_t pos_max[kWPrm][2];   // of a lookup warp's 64 cells
    float vs_max[kWPrm][2];      // largest |vs| of them
    uint32_t row[kWRow][kTile];  // the cells' rows in the pool
    float2 score[kTile];         // the rows' scales and sum(q)
    float2 fin[kTile];           // what their sums are scaled by and get added in the end
    int32_t lim[kTile];
    float2 half[2][2][kTile];    // [tile parity][column half][row]: (max, |vs|), in the end (l, z)
    Walk first;
    long long total;
    uint32_t tmem;
    int abort;
    uint64_t row_full[kWRow], row_empty[kWRow], prm_full[kWPrm], prm_empty[kWPrm];
    uint64_t k_full, k_done, v_full, o_done, q_full, p_full, s_full[2], mma_done;
};
constexpr uint32_t kWideBytes = 3 * kOperand + (uint32_t)sizeof(WideMisc);
static_assert(kWideBytes <= 227 * 1024, "shared memory");

// Power of two 2^6 / sigma, sigma a power of two not below v.
__device__ __forceinline__ float sigma_inverse(float v)
{
    const uint32_t up = (__float_as_uint(fmaxf(v, 0x1p-99f)) + 0x7fffffu) & 0x7f800000u;
    return __uint_as_float((260u << 23) - up);
}

__global__ void __launch_bounds__(kWideThreads, 1) qsa_kv4_wide_kernel(const AttnParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) { // (the swizzled operand tiles need it)
        if (threadIdx.x == 0) raise(p, QSA_STATUS_LAUNCH);
        return;
    }
    WideMisc &ms = *reinterpret_cast<WideMisc *>(smem + 3 * kOperand);
    const int tid = threadIdx.x, lane = tid & 31;
    const int w = __shfl_sync(0xffffffffu, tid >> 5, 0);

    if (tid == 0) {
        for (int i = 0; i < kWRow; ++i) {
            mbar_init(&ms.row_full[i], 64);
            mbar_init(&ms.row_empty[i], 256);
        }
        for (int i = 0; i < kWPrm; ++i) {
            mbar_init(&ms.prm_full[i], 64);
            mbar_init(&ms.prm_empty[i], 256);
        }
        mbar_init(&ms.k_full, 128);
        mbar_init(&ms.k_done, 1);
        mbar_init(&ms.v_full, 128);
        mbar_init(&ms.o_done, 1);
        mbar_init(&ms.q_full, 256);
        mbar_init(&ms.p_full, 256);
        mbar_init(&ms.s_full[0], 1);
        mbar_init(&ms.s_full[1], 1);
        mbar_init(&ms.mma_done, 1);
        ms.abort = 0;
        fence_mbar_init();
    }
    // rows of the pool from the start: a wait that runs out lets the loads read them early
    for (int i = tid; i < kWRow * kTile; i += kWideThreads) (&ms.row[0][0])[i] = 0u;
    // All input is read, and tensor memory taken, behind this (see qsa_kv4_attn_kernel).
    cudaGridDependencySynchronize();
    if (w == kWMma) {
        tmem_alloc(&ms.tmem, 512);
        tmem_relinquish();
    }
    if (w == 0) {
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
    const uint32_t tmem = __shfl_sync(0xffffffffu, ms.tmem, 0), t_o = tmem + 2 * kTile; // S at columns 0 and 128
    const int tiles = ms.first.left;

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

    if (w < kWSoft) {
        // ============================================================= softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // Warp: query rows 32 (w % 4) .. + 31, its tensor-memory lanes, and column half
        // w / 4 of S (cells) and O (dimensions).  Thread: rows 8 j + lane / 4, j = 0..3,
        // of them and the cells 8 k + 2 (lane % 4), + 1, so that it reads the scales and
        // zeros of 16 cells a tile, not of 64; a row's reference is kept by one of its
        // four threads, that of row 8 (lane % 4) + lane / 4.
        const int hc = w >> 2, quad = lane & 3, rows0 = 32 * (w & 3), mine = rows0 + 8 * quad + (lane >> 2);
        const uint32_t t_lane = (uint32_t)(32 * (w & 3)) << 16;
        const uint32_t pair_bar = 1 + (w & 3); // the warps of the two halves
        Walk it = ms.first;
        const long long total = ms.total;
        uint32_t i = 0; // tile
#pragma unroll 1
        for (uint32_t seg = 0; it.left > 0; ++seg) {
            const int b = it.b, g = it.g, row0 = it.rb * p.rb_rows, n_rows = min(p.rb_rows, p.R - row0);
            const int steps = min(it.left, it.nu - it.u);

            // ----------------------------------------------------- queries
            // A warp per row, lane = eight dimensions: scaled by a power of two so
            // that the row's largest magnitude lies in [2^14, 2^15), in the order of
            // the codes (dimensions 0 4 1 5 2 6 3 7, the odd ones' codes counting 16
            // times).
#pragma unroll 1
            for (int r0 = w; r0 < kTile; r0 += 4 * kWSoft) {
                uint4 raw[4]; // four rows in flight
                int lims[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = r0 + k * kWSoft;
                    raw[k] = make_uint4(0, 0, 0, 0);
                    lims[k] = 0x7fffffff; // (rows past the last one are zeros, and not written)
                    if (r < n_rows) {
                        lims[k] = p.q_limit ? p.q_limit[(size_t)b * p.T + query_of(p, row0 + r)] : 0x7fffffff;
                        raw[k] = load_late(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + row_offset(p, b, g, row0 + r)) + lane);
                    }
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int r = r0 + m * kWSoft, lim = lims[m];
                    const uint32_t r4[4] = {raw[m].x, raw[m].y, raw[m].z, raw[m].w};
                    float x[8];
                    uint32_t top = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[2 * k] = bf16_bits_to_f32(r4[k] & 0xffffu);
                        x[2 * k + 1] = __uint_as_float(r4[k] & 0xffff0000u);
                        top = max(top, max(__float_as_uint(x[2 * k]) & 0x7fffffffu, __float_as_uint(x[2 * k + 1]) & 0x7fffffffu));
                    }
                    const uint32_t e = max(__reduce_max_sync(0xffffffffu, top) >> 23, 15u);
                    float up = __uint_as_float((268u - min(e, 254u)) << 23);
                    if (p.scale_log2 < 0.f) up = -up; // (the scale below is positive)
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] *= up;
                    const float a[8] = {x[0], x[4], x[1] * 0.0625f, x[5] * 0.0625f, x[2], x[6], x[3] * 0.0625f, x[7] * 0.0625f};
                    float sum = 0.f; // of what the f16 values hold
                    uint32_t wd[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        wd[k] = half2_of(a[2 * k], a[2 * k + 1]);
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&wd[k]));
                        sum += (k & 1 ? 16.f : 1.f) * (f.x + f.y);
                    }
                    *reinterpret_cast<uint4 *>(smem + kmajor_sw128_off(r, 8 * lane, kTile)) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane == 0) {
                        // (sum(q) goes in 2^24 too small, as the scores come out of the
                        // MMA; a row that is not finite has NaN for the scores that it sees)
                        ms.score[r] = make_float2(e == 255u ? 1.f : row_scale(p, e),
                                                  e == 255u ? __uint_as_float(0x7fffffffu) : sum * 0x1p-24f);
                        ms.lim[r] = lim;
                    }
                }
            }
            fence_proxy_async_smem();
            named_bar(5, kWSoft * 32);
            mbar_arrive(&ms.q_full);
            const int lim_min = __reduce_min_sync(0xffffffffu, ms.lim[rows0 + lane]); // of the warp's rows
            float m_ref = -INFINITY, isg = 1.f; // of row `mine`: reference (log2 units), 2^6 / sigma
            // by row: scale and sum(q) of the scores, -reference and 2^6 / sigma, this
            // thread's sums of p and of p vz
            float2 sc[4], nm[4], sg[4], l[4], z[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sc[j] = ms.score[rows0 + 8 * j + (lane >> 2)];
                nm[j] = sg[j] = l[j] = z[j] = make_float2(0.f, 0.f);
            }

#pragma unroll 1
            for (int step = 0; step < steps; ++step, ++i) {
                const uint32_t pe = i % kWPrm, par = i & 1;
                wait(&ms.prm_full[pe], i / kWPrm);
                // cells that some row of the warp does not see: row by row
                const bool by_row = max(ms.pos_max[pe][0], ms.pos_max[pe][1]) >= lim_min;
                const float v_all = fmaxf(ms.vs_max[pe][0], ms.vs_max[pe][1]);
                wait(&ms.s_full[par], i >> 1);
                tc_fence_after();
                const uint32_t t_s = tmem + par * kTile + t_lane + hc * 64;
                uint32_t hw[2][16]; // P', two cells a word: rows 0 and 1, 2 and 3
                float of = 1.f;
                auto raw_scores = [&](float2 (&t)[4][8]) {
                    float u[2][32];
                    tmem_ld_16x256b<8>(t_s, u[0]);
                    tmem_ld_16x256b<8>(t_s + (16u << 16), u[1]);
                    tmem_wait_ld();
                    regs_after_wait<32>(u[0]);
                    regs_after_wait<32>(u[1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int k = 0; k < 8; ++k) t[j][k] = make_float2(u[j >> 1][4 * k + 2 * (j & 1)], u[j >> 1][4 * k + 2 * (j & 1) + 1]);
                };
                auto score = [&](float2 t, const float4 &f, int j) { // / xs
                    return fma2(t, make_float2(f.x, f.y), mul2(make_float2(f.z, f.w), make_float2(sc[j].y, sc[j].y)));
                };
                // P' of row j and cells k, and their part of the sums
                auto probability = [&](float2 t, float2 vs, float2 vz, int j, int k, float2 &ls, float2 &zs) {
                    float2 e = fma2(t, make_float2(sc[j].x, sc[j].x), nm[j]);
                    e.x = fast_exp2(e.x);
                    e.y = fast_exp2(e.y);
                    ls = add2(ls, e);
                    zs = fma2(e, vz, zs);
                    e = mul2(e, mul2(vs, sg[j]));
                    // one rounding of P', 2^-11; the cells' order is that of V's rows
                    hw[j >> 1][4 * (k >> 1) + 2 * (j & 1) + (k & 1)] = half2_of(e.x, e.y);
                };
                // With the references that the rows have, as if they held: they do for all
                // but the first tiles, and nothing waits for the other threads' maxima.
                bool need = true;
                if (!by_row && __all_sync(0xffffffffu, m_ref > -INFINITY)) {
                    float2 t[4][8], ls[4], zs[4];
                    float mx[4];
                    raw_scores(t);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        ls[j] = zs[j] = make_float2(0.f, 0.f);
                        mx[j] = -INFINITY;
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 f = ms.k[pe][32 * hc + 4 * k + quad], v = ms.v[pe][32 * hc + 4 * k + quad];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 x = score(t[j][k], f, j);
                            mx[j] = fmaxf(mx[j], fmaxf(x.x, x.y));
                            probability(x, make_float2(v.x, v.y), make_float2(v.z, v.w), j, k, ls[j], zs[j]);
                        }
                    }
                    need = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) need |= fmaf(mx[j], sc[j].x, nm[j].x) > 8.f || v_all * sg[j].x > 0x1p7f;
                    need = named_bar_or(pair_bar, 64, need);
                    if (!need) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            l[j] = add2(l[j], ls[j]);
                            z[j] = add2(z[j], zs[j]);
                        }
                    }
                } else {
                    named_bar_or(pair_bar, 64, true);
                }
                if (need) { // both halves: the maxima first
                    float2 t[4][8];
                    raw_scores(t);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 f = ms.k[pe][32 * hc + 4 * k + quad];
#pragma unroll
                        for (int j = 0; j < 4; ++j) t[j][k] = score(t[j][k], f, j);
                    }
                    float v1 = v_all;
                    if (by_row) {
                        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int2 at = *reinterpret_cast<const int2 *>(&ms.pos[pe][64 * hc + 8 * k + 2 * quad]);
                            const float4 f = ms.v[pe][32 * hc + 4 * k + quad];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int lim = ms.lim[rows0 + 8 * j + (lane >> 2)];
                                if (at.x >= lim) t[j][k].x = -INFINITY; else v[j] = fmaxf(v[j], fabsf(f.x));
                                if (at.y >= lim) t[j][k].y = -INFINITY; else v[j] = fmaxf(v[j], fabsf(f.y));
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[j] = fmaxf(v[j], __shfl_xor_sync(0xffffffffu, v[j], 1));
                            v[j] = fmaxf(v[j], __shfl_xor_sync(0xffffffffu, v[j], 2));
                        }
                        v1 = quad == 0 ? v[0] : quad == 1 ? v[1] : quad == 2 ? v[2] : v[3];
                    }
                    float mx;
                    {
                        float m[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            m[j] = fmaxf(t[j][0].x, t[j][0].y);
#pragma unroll
                            for (int k = 1; k < 8; ++k) m[j] = fmaxf(m[j], fmaxf(t[j][k].x, t[j][k].y));
                            m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 1));
                            m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 2));
                            m[j] = m[j] > -INFINITY ? m[j] * sc[j].x : -INFINITY; // (NaN counts for nothing)
                        }
                        mx = quad == 0 ? m[0] : quad == 1 ? m[1] : quad == 2 ? m[2] : m[3];
                    }
                    // the row's other half (the buffer's last readers passed a barrier since)
                    ms.half[par][hc][mine] = make_float2(mx, v1);
                    named_bar(pair_bar, 64);
                    {
                        const float2 a = ms.half[par][0][mine], o = ms.half[par][1][mine];
                        mx = fmaxf(a.x, o.x);
                        v1 = fmaxf(a.y, o.y);
                    }
                    // The reference is the maximum at its last move, sigma at least the
                    // largest V scale then: P' = p vs 2^6 / sigma stays below 2^8 * 2 * 2^6.
                    float fac = 1.f;
                    if (mx > -INFINITY) {
                        if (m_ref == -INFINITY) {
                            m_ref = mx;
                            isg = sigma_inverse(v1);
                        } else {
                            if (mx > m_ref + 8.f) {
                                fac = fast_exp2(m_ref - mx);
                                m_ref = mx;
                            }
                            of = fac;
                            if (v1 * isg > 0x1p7f) {
                                const float s = fminf(isg, sigma_inverse(v1));
                                of *= s / isg;
                                isg = s;
                            }
                        }
                    }
                    const float m_sub = m_ref > -INFINITY ? -m_ref : 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a = __shfl_sync(0xffffffffu, m_sub, j, 4), c = __shfl_sync(0xffffffffu, isg, j, 4),
                                    f = __shfl_sync(0xffffffffu, fac, j, 4);
                        nm[j] = make_float2(a, a);
                        sg[j] = make_float2(c, c);
                        l[j] = mul2(l[j], make_float2(f, f));
                        z[j] = mul2(z[j], make_float2(f, f));
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 f = ms.v[pe][32 * hc + 4 * k + quad];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float2 vs = make_float2(f.x, f.y), vz = make_float2(f.z, f.w);
                            if (by_row) { // (what an unseen cell holds must not reach the row, finite or not)
                                if (t[j][k].x == -INFINITY) vs.x = vz.x = 0.f;
                                if (t[j][k].y == -INFINITY) vs.y = vz.y = 0.f;
                            }
                            probability(t[j][k], vs, vz, j, k, l[j], z[j]);
                        }
                    }
                }
                // over this warp's half of S
                tmem_st_16x256b_x4(t_s, hw[0]);
                tmem_st_16x256b_x4(t_s + (16u << 16), hw[1]);
                mbar_arrive(&ms.prm_empty[pe]);
                // P.V of the tile before, for whoever reads O next.  (Phases are told
                // apart by parity, so a wait must not come two of them late: S of this
                // tile was issued after P.V of the one two before, and this tile's P.V
                // waits for this thread.)
                const bool moved = __any_sync(0xffffffffu, of != 1.f) && step > 0;
                if (i >= 1 && (moved || step == steps - 1)) wait(&ms.o_done, i - 1);
                if (moved) { // O so far
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) { // 32 dimensions of 16 rows
                        const uint32_t ta = t_o + t_lane + ((uint32_t)(16 * (c & 1)) << 16) + hc * 128 + (c >> 1) * 32;
                        const float f0 = __shfl_sync(0xffffffffu, of, 2 * (c & 1), 4), f1 = __shfl_sync(0xffffffffu, of, 2 * (c & 1) + 1, 4);
                        float v[16];
                        uint32_t u[16];
                        tmem_ld_16x256b_x4(ta, v);
                        tmem_wait_ld();
                        regs_after_wait<16>(v);
#pragma unroll
                        for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(v[k] * (k & 2 ? f1 : f0));
                        tmem_st_16x256b_x4(ta, u);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&ms.p_full);
            }

            // --------------------------------------------- the segment's sums
            float L, Z;
            {
                float x[4], y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = l[j].x + l[j].y;
                    y[j] = z[j].x + z[j].y;
                    x[j] += __shfl_xor_sync(0xffffffffu, x[j], 1);
                    y[j] += __shfl_xor_sync(0xffffffffu, y[j], 1);
                    x[j] += __shfl_xor_sync(0xffffffffu, x[j], 2);
                    y[j] += __shfl_xor_sync(0xffffffffu, y[j], 2);
                }
                ms.half[i & 1][hc][mine] = make_float2(quad == 0 ? x[0] : quad == 1 ? x[1] : quad == 2 ? x[2] : x[3],
                                                       quad == 0 ? y[0] : quad == 1 ? y[1] : quad == 2 ? y[2] : y[3]);
                named_bar(pair_bar, 64);
                const float2 a = ms.half[i & 1][0][mine], o = ms.half[i & 1][1][mine];
                L = a.x + o.x;
                Z = a.y + o.y;
            }
            const bool direct = it.u == 0 && steps == it.nu;
            const int slot = 2 * (int)blockIdx.x + (seg == 0 ? 0 : 1);
            if (hc == 0) {
                const float inv = direct ? (L == 0.f ? 0.f : 1.f / L) : 1.f; // (NaN: a row that is not finite)
                ms.fin[mine] = make_float2(0x1p9f / isg * inv, Z * inv);
                if (!direct && mine < n_rows)
                    p.part_ml[(size_t)slot * p.slot_rows + mine] = make_float2(L == 0.f ? -INFINITY : m_ref, L);
            }
            if (it.u == 0 && tid == 0) {
                const long long pair = ((long long)b * p.pool.G + g) * p.n_rb + it.rb;
                p.info[pair] = make_int2(slot, direct ? 1 : parts_of(it, total));
            }
            named_bar(pair_bar, 64);
            // O by rows: thread = row rows0 + lane
            const int row = rows0 + lane;
            const float fin = ms.fin[row].x, zs = ms.fin[row].y;
            const size_t at = row < n_rows ? row_offset(p, b, g, row0 + row) + 128 * hc : 0;
            float *part = p.part_o + ((size_t)slot * p.slot_rows + row) * kHeadDim + 128 * hc;
            wait(&ms.o_done, i - 1);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
                float v[16], d[16];
                tmem_ld16(t_o + t_lane + hc * 128 + c * 16, v);
                tmem_wait_ld();
                regs_after_wait<16>(v);
                // (the order of the codes)
#pragma unroll
                for (int k = 0; k < 16; ++k) d[(k & 8) + ((k & 7) >> 1) + 4 * (k & 1)] = fmaf(v[k], fin, zs);
                if (row >= n_rows) continue;
                if (direct) {
                    uint32_t o2[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o2[k]) : "f"(d[2 * k + 1]), "f"(d[2 * k]));
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at + 16 * c);
                    dst[0] = make_uint4(o2[0], o2[1], o2[2], o2[3]);
                    dst[1] = make_uint4(o2[4], o2[5], o2[6], o2[7]);
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(part + 16 * c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) dst[k] = make_float4(d[4 * k], d[4 * k + 1], d[4 * k + 2], d[4 * k + 3]);
                }
            }
            tc_fence_before(); // (the next P.V follows this thread's next p_full)
            walk_next(p, it, steps);
        }
    } else if (w < kWMma) {
        // ============================================================== K and V
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCodeRegs));
        // Thread: one cell's 128 bytes of K (or V) codes, loaded a tile ahead,
        // expanded into the operand tile (K-major for K, MN-major for V: the same
        // places): a word of codes is one 16-byte piece.  V's cells stand in the order
        // in which the softmax threads hold P: row 16 a + 4 q + 2 j + b is cell
        // 16 a + 8 j + 2 q + b.
        const bool is_v = w >= kWSoft + kWCodes / 2;
        const int place = 32 * (w & 3) + lane;
        const int cell = is_v ? (place & ~15) | ((place >> 1) & 1) << 3 | ((place >> 2) & 3) << 1 | (place & 1) : place;
        const uint32_t at = (uint32_t)(place & 7) << 4;
        uint8_t *dst = smem + (is_v ? 2 : 1) * kOperand + (place >> 3) * 1024 + (place & 7) * 128;
        uint64_t *full = is_v ? &ms.v_full : &ms.k_full, *done = is_v ? &ms.o_done : &ms.k_done;
        uint32_t raw[32];
        auto fetch = [&](uint32_t j) {
            const uint32_t e = j % kWRow;
            wait(&ms.row_full[e], j / kWRow);
            const uint8_t *src = p.codes + (size_t)ms.row[e][cell] * QSA_KV4_CODE_BYTES + (is_v ? 128 : 0);
            mbar_arrive(&ms.row_empty[e]);
#pragma unroll
            for (int c = 0; c < 4; ++c) load_late256(src + 32 * c, raw + 8 * c);
        };
        if (tiles > 0) fetch(0);
#pragma unroll 1
        for (int j = 0; j < tiles; ++j) {
            if (j >= 1) wait(done, j - 1);
            if (is_v) {
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    uint32_t f[4];
                    expand_centred(raw[c], f);
                    *reinterpret_cast<uint4 *>(dst + (c >> 3) * 16384 + (((uint32_t)(c & 7) << 4) ^ at)) = make_uint4(f[0], f[1], f[2], f[3]);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    uint32_t f[4];
                    expand(raw[c], f);
                    *reinterpret_cast<uint4 *>(dst + (c >> 3) * 16384 + (((uint32_t)(c & 7) << 4) ^ at)) = make_uint4(f[0], f[1], f[2], f[3]);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(full);
            if (j + 1 < tiles) fetch(j + 1);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
        if (w == kWMma) {
            // ================================================================= MMA
            // All lanes run the loop (every value is uniform), one issues.  The tensor
            // pipe runs one thread's MMAs in order: S of tile i + 1 goes ahead of P.V of
            // tile i (but for a new segment's, whose queries follow that P.V), into the
            // buffer whose P the P.V before has read.
            const bool leader = elect_one();
            const uint32_t idesc_s = idesc_f16(kTile, kTile, false, false, false, false);
            const uint32_t idesc_o = idesc_f16(kTile, kHeadDim, false, false, false, true);
            const uint64_t qd = smem_desc(smem_u32(smem), 16, 1024), kd = smem_desc(smem_u32(smem + kOperand), 16, 1024);
            const uint64_t vd = smem_desc(smem_u32(smem + 2 * kOperand), 16384, 1024);
            auto issue_s = [&](uint32_t i) {
                wait(&ms.k_full, i);
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kHeadDim / 16; ++kk) {
                        const uint64_t at = (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
                        mma_f16_ss(tmem + (i & 1) * kTile, qd + at, kd + at, idesc_s, kk > 0);
                    }
                    mma_commit(&ms.k_done);
                    mma_commit(&ms.s_full[i & 1]);
                }
                __syncwarp();
            };
            Walk it = ms.first;
            uint32_t i = 0;
#pragma unroll 1
            for (uint32_t seg = 0; it.left > 0; ++seg) {
                const int steps = min(it.left, it.nu - it.u);
                wait(&ms.q_full, seg);
                issue_s(i);
#pragma unroll 1
                for (int step = 0; step < steps; ++step, ++i) {
                    if (step + 1 < steps) issue_s(i + 1);
                    wait(&ms.p_full, i);
                    wait(&ms.v_full, i);
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk) // (P of cells 64.. begins at column 64)
                            mma_f16_ts(t_o, tmem + (i & 1) * kTile + 8 * kk + (kk < 4 ? 0 : 32), vd + (uint64_t)((2048 * kk) >> 4),
                                       idesc_o, (step > 0 || kk > 0) ? 1u : 0u);
                        mma_commit(&ms.o_done);
                    }
                    __syncwarp();
                }
                walk_next(p, it, steps);
            }
            // before the CTA leaves (also after a time-out): every MMA complete
            if (leader) mma_commit(&ms.mma_done);
            __syncwarp();
            mbar_wait(&ms.mma_done, 0, kDrainCycles);
        } else if (w < kWRes + 2) {
            // ============================================================== lookup
            // Lane l of warp k resolves cells 64 k + l and + 32 of every tile, one stage
            // per tile: the list entry two tiles, the page entry one tile before the row
            // in the pool, its scales and zeros one tile after that.
            const int half = w - kWRes, c0 = 64 * half + lane;
            Walk head = ms.first;
            const int cap = p.pool.page_table_len * p.pool.page_cells;
            int a_pos[2] = {0, 0}, c_pos[2] = {0, 0}, c_entry[2] = {0, 0}, c_off[2] = {0, 0}, d_pos[2] = {0, 0};
            int a_b = 0, a_g = 0, c_b = 0, c_g = 0;
            bool a_in[2] = {false, false}, c_in[2] = {false, false};
            float4 f[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 1
            for (int t = -2; t <= tiles; ++t) {
                if (t >= 1) { // scales and zeros of tile t - 1
                    const uint32_t j = t - 1, e = j % kWPrm;
                    if (j >= kWPrm) wait(&ms.prm_empty[e], j / kWPrm - 1);
                    int top = -1;
                    float v = 0.f;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int c = c0 + 32 * k;
                        f[k].w = fmaf(7.5f, f[k].z, f[k].w); // (V's codes go in less 7.5)
                        float *const kp = &ms.k[e][c >> 1].x + (c & 1), *const vp = &ms.v[e][c >> 1].x + (c & 1);
                        kp[0] = f[k].x;
                        kp[2] = f[k].y;
                        vp[0] = f[k].z;
                        vp[2] = f[k].w;
                        ms.pos[e][c] = d_pos[k];
                        top = max(top, d_pos[k]);
                        v = fmaxf(v, fabsf(f[k].z));
                    }
                    top = __reduce_max_sync(0xffffffffu, top);
                    v = warp_max(v);
                    if (lane == 0) {
                        ms.pos_max[e][half] = top;
                        ms.vs_max[e][half] = v;
                    }
                    mbar_arrive(&ms.prm_full[e]);
                }
                if (t >= 0 && t < tiles) { // row
                    const uint32_t e = (uint32_t)t % kWRow;
                    if (t >= kWRow) wait(&ms.row_empty[e], (uint32_t)t / kWRow - 1);
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
                        // (where there is no cell, the row of slot 0, any does, and zeros)
                        const uint32_t r = (uint32_t)(base + max(slot, 0));
                        ms.row[e][c0 + 32 * k] = r;
                        d_pos[k] = slot >= 0 ? c_pos[k] : 0x7fffffff;
                        f[k] = slot >= 0 ? p.scale[r] : make_float4(0.f, 0.f, 0.f, 0.f);
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
    if (w == kWMma) tmem_dealloc(tmem, 512);
}

} // namespace

cudaError_t launch_wide(const AttnParams &p, int grid, cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(qsa_kv4_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWideBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kWideThreads);
    cfg.dynamicSmemBytes = kWideBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qsa_kv4_wide_kernel, p);
}

} // namespace kv4
} // namespace qsa

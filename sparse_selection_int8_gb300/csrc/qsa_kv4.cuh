// qsa_kv4.cuh -- shared by the kernels of the 4-bit cells (see include/qsa.h
// for the format: 256 code bytes and four fp32 values per cell and KV head).
#pragma once

#include "qsa_internal.cuh"

namespace qsa {

// Where the cells of one call lie.
struct Kv4Pool {
    const int32_t *page_table; // [n_seq][page_table_len]
    int32_t G, n_pools;        // pools: one shared by the sequences, or one each
    int32_t pool_cells, page_table_len;
    int32_t page_cells, pool_pages; // P cells per page; valid entries 0 .. pool_pages - 1
};

// Row of (sequence b, KV head g, slot) in kv_pool and kv_scale.
__device__ __forceinline__ size_t kv4_row(const Kv4Pool &p, int b, int g, int slot)
{
    return ((size_t)(p.n_pools == 1 ? 0 : b) * p.G + g) * p.pool_cells + slot;
}

// Pool slot of page entry e for the position at offset `off` of its page; -1
// (and the reason) if the entry is not in the pool.
__device__ __forceinline__ int kv4_slot(const Kv4Pool &p, int e, int off, uint32_t &bad)
{
    if (e == -1) {
        bad = QSA_STATUS_NOT_RESIDENT;
        return -1;
    }
    if (e < 0 || e >= p.pool_pages) {
        bad = QSA_STATUS_BAD_SLOT;
        return -1;
    }
    return e * p.page_cells + off; // < pool_cells
}

// Pool slot of position pos of sequence b; -1 (and the reason) if it has none.
// Position -1 is a padding row, without a reason.
__device__ __forceinline__ int kv4_resolve(const Kv4Pool &p, int b, int pos, uint32_t &bad)
{
    if (pos == -1) return -1;
    const int P = p.page_cells;
    if (pos < 0 || (long long)pos >= (long long)p.page_table_len * P) {
        bad = QSA_STATUS_BAD_POSITION;
        return -1;
    }
    const int page = P == 1 ? pos : pos / P;
    return kv4_slot(p, p.page_table[(size_t)b * p.page_table_len + page], pos - page * P, bad);
}

// Loads that stay behind cudaGridDependencySynchronize(), of data that the kernel
// before may have written while this one was being launched (no read-only path, no
// L1).
__device__ __forceinline__ uint4 load_late(const uint4 *ptr)
{
    uint4 v;
    asm volatile("ld.global.cg.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(ptr) : "memory");
    return v;
}

__device__ __forceinline__ void load_late256(const void *ptr, uint32_t *r) // 32-byte aligned
{
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(ptr) : "memory");
}

// Two fp32 values in one operation.
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t &>(d)) : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t &>(d)) : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}

inline bool kv4_aligned(const void *ptr, size_t a) { return ((uintptr_t)ptr % a) == 0; }

// The shape fields that every call on 4-bit cells reads.
inline qsa_status kv4_check(const qsa_shape *s, int n_seq, int n_pools)
{
    if (!s) return QSA_ERR_INVALID_ARG;
    if (s->n_kv_heads < 1 || s->pool_cells < 1 || s->page_table_len < 1 || s->page_cells < 0)
        return QSA_ERR_INVALID_ARG;
    const int P = s->page_cells > 0 ? s->page_cells : 1;
    if (s->pool_cells % P != 0 || (long long)s->page_table_len * P > 0x7fffffffll) return QSA_ERR_INVALID_ARG;
    if (n_seq < 0 || (n_pools != 1 && n_pools != n_seq)) return QSA_ERR_INVALID_ARG;
    if (s->head_dim != kHeadDim || s->n_kv_heads > 65535) return QSA_ERR_UNSUPPORTED;
    return QSA_OK;
}

inline Kv4Pool kv4_pool(const qsa_shape *s, int n_pools, const int32_t *page_table)
{
    Kv4Pool p{};
    p.page_table = page_table;
    p.G = s->n_kv_heads;
    p.n_pools = n_pools;
    p.pool_cells = s->pool_cells;
    p.page_table_len = s->page_table_len;
    p.page_cells = s->page_cells > 0 ? s->page_cells : 1;
    p.pool_pages = s->pool_cells / p.page_cells;
    return p;
}

} // namespace qsa

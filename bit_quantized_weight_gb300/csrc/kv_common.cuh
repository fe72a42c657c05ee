// kv_common.cuh -- what the cache kernels (kv_cache.cu) and the attention over
// the cache (tree_attention.cu) share: a call's sequences, the place of a
// token in the pages, and the sizes of the three storage formats.
#pragma once

#include "common.cuh"
#include "kv_internal.h"

namespace qg {

// Bytes of one token's codes and scales of one head.
__host__ __device__ constexpr int kv_row_bytes(int fmt, int dim)
{
    return fmt == QG_KV_BF16 ? 2 * dim : fmt == QG_KV_FP8 ? dim : dim / 2;
}

__host__ __device__ constexpr int kv_scale_bytes(int fmt, int dim)
{
    return fmt == QG_KV_BF16 ? 0 : fmt == QG_KV_FP8 ? 1 : dim / 16;
}

// Four E4M3 codes of a register as two f16x2, in order.
__device__ __forceinline__ void e4m3x4_to_f16x2x2(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Sequence b of a call: its rows [row0, row0 + rows) and the tokens the cache
// held before. rows = 0 for a sequence whose entries do not fit (recorded).
struct KvSeq {
    int row0;
    int rows;
    int len;
};

__device__ __forceinline__ KvSeq kv_seq_of(const KvArgs& a, int row0, int end, int len, int max_rows)
{
    KvSeq s;
    s.row0 = row0;
    s.len = len;
    s.rows = static_cast<int>(static_cast<unsigned>(end) - static_cast<unsigned>(row0));
    const bool ok = s.row0 >= 0 && end >= s.row0 && end <= a.n_tokens && s.len >= 0 && s.rows <= max_rows &&
                    static_cast<int64_t>(s.len) + s.rows <=
                        min(static_cast<int64_t>(a.max_pages) * a.page_size, static_cast<int64_t>(kKvMaxPositions));
    if (!ok) {
        set_device_status(a.status, QG_ERR_INVALID_ARG);
        s.rows = 0;
    }
    return s;
}

// p / page_size without a division: with k = page_size / 16 <= 64 groups of 16
// positions per page and x = p / 16 < 2^27, x * ceil(2^36 / k) exceeds
// x * 2^36 / k by less than x < 2^36 / k, so the high part is x / k exactly.
__device__ __forceinline__ int kv_page_index(const KvArgs& a, int p)
{
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(p) >> 4) * a.page_magic) >> 36);
}

__device__ __forceinline__ KvSeq kv_seq(const KvArgs& a, int b, int max_rows)
{
    return kv_seq_of(a, a.start[b], a.start[b + 1], a.lens[b], max_rows);
}

// The table's entry for position p of sequence b, which kv_valid then checks:
// apart, so that several entries can be on their way at a time.
__device__ __forceinline__ int kv_entry(const KvArgs& a, int b, int p)
{
    return a.table[static_cast<int64_t>(b) * a.max_pages + kv_page_index(a, p)];
}

// The page that an entry names, or -1 (recorded) if it lies outside the cache.
__device__ __forceinline__ int kv_valid(const KvArgs& a, int entry)
{
    if (static_cast<unsigned>(entry) < static_cast<unsigned>(a.num_pages)) return entry;
    set_device_status(a.status, QG_ERR_INVALID_ARG);
    return -1;
}

__device__ __forceinline__ int kv_page(const KvArgs& a, int b, int p) { return kv_valid(a, kv_entry(a, b, p)); }

// Index of (page, head, position) among the cache's rows: rows * row bytes is
// the offset of its codes (64 bits: a pool may pass 2^31 rows' bytes).
__device__ __forceinline__ int64_t kv_row(const KvArgs& a, int page, int head, int p)
{
    return (static_cast<int64_t>(page) * a.heads + head) * a.page_size + (p - kv_page_index(a, p) * a.page_size);
}

}  // namespace qg

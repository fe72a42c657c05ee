// tree_common.cuh -- how tree_attention splits its work, shared by the kernels
// that read the cache and the one that joins their parts.
//
// A unit is (sequence, key/value head, tile of query rows): the rows of a
// sequence's tokens that share a head, G per token, in tiles of R. A unit's
// keys are cut into steps. All steps of a call, in order, are dealt out evenly:
// CTA c of the n that get work takes [c * total / n, (c + 1) * total / n), whatever sequence they
// belong to, so ragged lengths balance by themselves and lengths stay device
// data. A CTA
// that holds only a piece of a unit writes it to the workspace: a unit's first
// piece to slot 2c + 1 (it ends at the CTA's end), any other to slot 2c (it
// starts at the CTA's start).
#pragma once

#include "kv_common.cuh"

namespace qg {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct TreeArgs {
    KvArgs a;
    const uint16_t* q;
    int64_t q_stride;
    int q_heads;
    int group;                // query heads per key/value head
    int max_tree;
    const uint64_t* mask;
    float scale;              // softmax scale
    uint16_t* out;
    float* lse;
    float* part_o;            // [slots][R][dim], relative to part_ml's maximum
    float2* part_ml;          // [slots][R]: (log2 of the unit weight, sum of weights)
    int rows;                 // R
    int step;                 // keys per step
    int grid;                 // CTAs of the reading kernel
    int run;                  // keys of a page that the tensor-core kernel copies at a time
    uint64_t wait_ns;         // limit of the tensor-core kernel's waits
    int starve;               // fault injection: its key tiles are never announced
};

struct TreeSeq {
    KvSeq s;
    int keys;                 // positions in the cache
    int steps;                // per unit
    int tiles;                // row tiles per head
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& t, int b)
{
    TreeSeq u;
    u.s = kv_seq(t.a, b, t.max_tree);
    u.keys = u.s.rows ? u.s.len + u.s.rows : 0;
    u.steps = (u.keys - 1 + t.step) / t.step;
    u.tiles = (u.s.rows * t.group + t.rows - 1) / t.rows;
    return u;
}

// Exclusive prefix sums of the sequences' steps into `prefix`
// [n_seqs + 1] (shared), by the first warp; the caller synchronises.
__device__ __forceinline__ void tree_prefix(const TreeArgs& t, int64_t* prefix)
{
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    int64_t total = 0;
    for (int j = 0; j < t.a.n_seqs; j += 32) {
        int64_t w = 0;
        if (j + lane < t.a.n_seqs) {
            const TreeSeq u = tree_seq(t, j + lane);
            w = static_cast<int64_t>(u.steps) * u.tiles * t.a.heads;
        }
        int64_t sum = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += up;
        }
        if (j + lane < t.a.n_seqs) prefix[j + lane] = total + sum - w;
        total += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) prefix[t.a.n_seqs] = total;
}

// The last sequence whose first step is at or before `step`.
__device__ __forceinline__ int tree_find(const int64_t* prefix, int n, int64_t step)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= step)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The CTAs that get work: no more than there are steps, so that each of them
// holds at least one. The first step of CTA c, and the CTA that holds a step:
// the last c with c * total / n <= step.
__device__ __forceinline__ int64_t tree_ctas(int64_t total, int grid) { return min(total, static_cast<int64_t>(grid)); }
__device__ __forceinline__ int64_t tree_first(int64_t total, int grid, int64_t c)
{
    const int64_t n = tree_ctas(total, grid);
    return c < n ? c * total / n : total;
}
__device__ __forceinline__ int64_t tree_owner(int64_t total, int grid, int64_t step)
{
    return ((step + 1) * tree_ctas(total, grid) - 1) / total;
}

// 1 / L with 0 for an empty row.
__device__ __forceinline__ float tree_inverse(float l) { return l > 0.f || l != l ? 1.f / l : 0.f; }

__device__ __forceinline__ float tree_lse(float m, float l)
{
    return l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY;
}

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A stored value, one at a time (rare paths).
__device__ __forceinline__ float kv_value(const KvArgs& a, int kv, int64_t row, int d)
{
    const uint8_t* c = a.codes[kv] + row * kv_row_bytes(a.fmt, a.dim);
    if (a.fmt == QG_KV_BF16) return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(c)[d]);
    const int sb = kv_scale_bytes(a.fmt, a.dim);
    uint32_t h, s;
    if (a.fmt == QG_KV_FP8) {
        h = e4m3x2_to_f16x2(c[d]);
        s = static_cast<uint32_t>(a.scales[kv][row]) << 10;
    } else {
        h = e2m1x2_to_f16x2((c[d / 2] >> (4 * (d & 1))) & 15u);
        s = e4m3x2_to_f16x2(a.scales[kv][row * sb + d / 16]);
    }
    return half_bits_to_f32(hmul2(h, s & 0xFFFFu) & 0xFFFFu);
}

cudaError_t launch_tree_tc(const TreeArgs& t, cudaStream_t stream);
cudaError_t launch_tree_join(const TreeArgs& t, cudaStream_t stream);

}  // namespace qg

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

#include <atomic>

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

// (step, rows: t.step and t.rows, or the constants that they are to a kernel)
__device__ __forceinline__ TreeSeq tree_seq_of(const TreeArgs& t, const KvSeq& s, uint32_t step, uint32_t rows)
{
    TreeSeq u;
    u.s = s;
    u.keys = s.rows ? s.len + s.rows : 0;
    u.steps = (static_cast<uint32_t>(u.keys) + step - 1) / step;
    u.tiles = (static_cast<uint32_t>(s.rows) * t.group + rows - 1) / rows;
    return u;
}

__device__ __forceinline__ TreeSeq tree_seq_of(const TreeArgs& t, const KvSeq& s)
{
    return tree_seq_of(t, s, t.step, t.rows);
}

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& t, int b)
{
    return tree_seq_of(t, kv_seq(t.a, b, t.max_tree));
}

__device__ __forceinline__ int64_t tree_steps(const TreeArgs& t, const TreeSeq& u)
{
    return static_cast<int64_t>(u.steps) * u.tiles * t.a.heads;
}

// The call's steps, scanned by one warp with its sequences' entries in its
// lanes: 32 sequences at a time, and the first 32 (mostly all) read only once.
struct TreeScan {
    KvSeq mine;                  // sequence `first + lane`, the last chunk looked at
    int first;
    int64_t before, steps;       // steps ahead of it, and its own
    int64_t total;

    __device__ __forceinline__ void load(const TreeArgs& t, int chunk, int64_t ahead)
    {
        const int lane = threadIdx.x & 31;
        first = chunk;
        mine = KvSeq{0, 0, 0};
        steps = 0;
        if (chunk + lane < t.a.n_seqs) {
            mine = kv_seq(t.a, chunk + lane, t.max_tree);
            steps = tree_steps(t, tree_seq_of(t, mine));
        }
        int64_t sum = steps;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += up;
        }
        before = ahead + sum - steps;
    }

    __device__ __forceinline__ int64_t end() const { return __shfl_sync(0xffffffffu, before + steps, 31); }

    __device__ __forceinline__ void run(const TreeArgs& t)
    {
        load(t, 0, 0);
        total = end();
        for (int c = 32; c < t.a.n_seqs; c += 32) {
            load(t, c, total);
            total = end();
        }
    }

    // The sequence that holds a step (< total): its index, entries and first step.
    __device__ __forceinline__ int find(const TreeArgs& t, int64_t step, KvSeq& s, int64_t& base)
    {
        if (first != 0) load(t, 0, 0);
        while (step >= end()) load(t, first + 32, end());
        const uint32_t hit = __ballot_sync(0xffffffffu, steps > 0 && before <= step && step < before + steps);
        return pick(__ffs(hit) - 1, s, base);
    }

    // The sequence that row i belongs to, -1 for a row of none.
    __device__ __forceinline__ int find_row(const TreeArgs& t, int i, KvSeq& s, int64_t& base)
    {
        if (first != 0) load(t, 0, 0);
        for (;;) {
            const uint32_t hit = __ballot_sync(0xffffffffu, mine.rows > 0 && i >= mine.row0 && i - mine.row0 < mine.rows);
            if (hit) return pick(__ffs(hit) - 1, s, base);
            if (first + 32 >= t.a.n_seqs) return -1;
            load(t, first + 32, end());
        }
    }

    __device__ __forceinline__ int pick(int from, KvSeq& s, int64_t& base) const
    {
        s.row0 = __shfl_sync(0xffffffffu, mine.row0, from);
        s.rows = __shfl_sync(0xffffffffu, mine.rows, from);
        s.len = __shfl_sync(0xffffffffu, mine.len, from);
        base = __shfl_sync(0xffffffffu, before, from);
        return first + from;
    }
};

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

// Lets a kernel have its dynamic shared memory, once per device (a bit of
// `done` each; other devices than the first 64 set it every time).
template <typename K>
cudaError_t allow_smem(K kern, int bytes, std::atomic<uint64_t>& done)
{
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return e;
    const uint64_t bit = d < 64 ? 1ull << d : 0;
    if (done.load() & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

cudaError_t launch_tree_tc(const TreeArgs& t, cudaStream_t stream);
cudaError_t launch_tree_join(const TreeArgs& t, cudaStream_t stream);

}  // namespace qg

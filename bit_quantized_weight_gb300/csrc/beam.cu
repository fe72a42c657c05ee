// beam.cu -- beam search's selection: the best continuations of a lane over
// its beams and the vocabulary (beam_select).
//
// score(r, t) = scores[r] + logits[r][t] - ln sum_t' exp(logits[r][t']): the
// order of a row's tokens is that of its logits, so one pass over a row gives
// both its sum of exponentials (a running maximum and the sum scaled to it)
// and its n_out best tokens; a lane's best are among those of its rows. Rows
// are cut into parts, a block each; a second kernel joins the parts of a lane.
#include "kv_common.cuh"

namespace qg {
namespace {

constexpr int kScanWarps = 8, kScanThreads = 32 * kScanWarps;
constexpr int kVec = 8;                              // values a thread takes at a time
constexpr int kUnroll = 4;
constexpr int kTile = 32 * kVec * kUnroll;           // values a warp takes at a time
constexpr int kList = 128;                           // keys a warp holds
constexpr int kMaxOut = 64;
constexpr int kJoinThreads = 256;
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// One whole number that orders a row's tokens: by the logit, then the lower
// token first. -0 counts as 0. 0 stands for no token.
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t b = __float_as_uint(v + 0.f);
    return b ^ (b & 0x80000000u ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ uint64_t make_key(float v, uint32_t token)
{
    return static_cast<uint64_t>(ordered(v)) << 32 | ~token;
}

__device__ __forceinline__ float key_value(uint64_t key)
{
    const uint32_t o = static_cast<uint32_t>(key >> 32);
    return __uint_as_float(o ^ (o & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ uint32_t key_token(uint64_t key) { return ~static_cast<uint32_t>(key); }

// Whether a row's logits are looked at: its score is a number and it goes on.
__device__ __forceinline__ bool row_live(const BeamArgs& a, int row)
{
    const float s = a.scores[row];
    return s > -INFINITY && s < INFINITY && !(a.finished && a.finished[row]);
}

// The words of 16-byte pieces from byte `skip` on.
template <int N>
__device__ __forceinline__ void shift_words(uint32_t (&w)[N], int skip)
{
    if (skip & 8) {
#pragma unroll
        for (int i = 0; i + 2 < N; ++i) w[i] = w[i + 2];
    }
    if (skip & 4) {
#pragma unroll
        for (int i = 0; i + 1 < N; ++i) w[i] = w[i + 1];
    }
    if (skip & 2) {
#pragma unroll
        for (int i = 0; i + 1 < N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
}

// Values e .. e + 7 of a row of `vocab`, -infinity behind its end. The same
// values go to the same thread whatever the row's alignment; a row that does
// not start at 16 bytes is read in the aligned pieces around it, but for the
// last values, which are read one by one. (Plain loads: the kernel before may
// have written them while this one had started already.)
template <bool F32>
__device__ __forceinline__ void load8(const uint8_t* row, int vocab, int e, float (&v)[kVec])
{
    constexpr int kSize = F32 ? 4 : 2, kPieces = F32 ? 2 : 1;
    const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
    const uint8_t* at = row + static_cast<int64_t>(e) * kSize;
    if (e + kVec + (skip ? 16 / kSize : 0) <= vocab) {
        uint32_t w[4 * (kPieces + 1)];
#pragma unroll
        for (int i = 0; i <= kPieces; ++i)
            if (i < kPieces || skip) {
                const uint4 x = *reinterpret_cast<const uint4*>(at - skip + 16 * i);
                w[4 * i] = x.x;
                w[4 * i + 1] = x.y;
                w[4 * i + 2] = x.z;
                w[4 * i + 3] = x.w;
            }
        if (skip) shift_words(w, skip);
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            v[i] = F32 ? __uint_as_float(w[i]) : __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            v[i] = -INFINITY;
            if (e + i < vocab)
                v[i] = F32 ? reinterpret_cast<const float*>(at)[i]
                           : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(at)[i]);
        }
    }
}

// A warp's best tokens so far: up to kList keys, and a bound below which none
// is among its n best.
struct Best {
    uint64_t* keys;
    int count;
    int n;
    uint64_t bound;
};

// Keep the n best, in order: each key's place is the number of greater ones.
__device__ __forceinline__ void keep_best(Best& b, int lane)
{
    uint64_t mine[kList / 32];
    int place[kList / 32];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kList / 32; ++i) {
        mine[i] = lane + 32 * i < b.count ? b.keys[lane + 32 * i] : 0;
        place[i] = 0;
    }
    for (int j = 0; j < b.count; ++j) {
        const uint64_t k = b.keys[j];
#pragma unroll
        for (int i = 0; i < kList / 32; ++i) place[i] += k > mine[i];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kList / 32; ++i)
        if (mine[i] && place[i] < b.n) b.keys[place[i]] = mine[i];
    __syncwarp();
    b.count = min(b.count, b.n);
    if (b.count == b.n) b.bound = b.keys[b.n - 1];
}

template <bool F32>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const __grid_constant__ BeamArgs a, int parts, int span,
                                                                 float2* sums, uint64_t* out)
{
    __shared__ uint64_t lists[kScanWarps][kList];
    __shared__ uint64_t merged[kScanWarps * kMaxOut];
    __shared__ int counts[kScanWarps];
    __shared__ float2 warp_sums[kScanWarps];
    pdl_enter();
    const int row_i = blockIdx.x / parts, part = blockIdx.x % parts;
    if (!row_live(a, row_i)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint8_t* row = static_cast<const uint8_t*>(a.logits) + row_i * a.stride * (F32 ? 4 : 2);
    const int begin = part * span, end = min(begin + span, a.vocab);
    Best best{lists[warp], 0, a.n_out, make_key(-INFINITY, 0)};
    float top = kLowest, sum = 0.f;
    for (int base = begin + warp * kTile; base < end; base += kScanWarps * kTile) {
        float v[kUnroll][kVec];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) load8<F32>(row, a.vocab, base + u * 32 * kVec + lane * kVec, v[u]);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float m = v[u][0];
#pragma unroll
            for (int i = 1; i < kVec; ++i) m = fmaxf(m, v[u][i]);
            if (m > top) {
                sum *= ex2((top - m) * kLog2e);
                top = m;
            }
#pragma unroll
            for (int i = 0; i < kVec; ++i) sum += ex2((v[u][i] - top) * kLog2e);
            if (!__any_sync(0xffffffffu, m >= key_value(best.bound))) continue;
#pragma unroll 1
            for (int i = 0; i < kVec; ++i) {
                float x = v[u][0];
#pragma unroll
                for (int j = 1; j < kVec; ++j) x = i == j ? v[u][j] : x;
                const uint64_t key = make_key(x, static_cast<uint32_t>(base + u * 32 * kVec + lane * kVec + i));
                uint32_t with = __ballot_sync(0xffffffffu, x == x && key > best.bound);
                if (!with) continue;
                if (best.count + __popc(with) > kList) {
                    keep_best(best, lane);
                    with = __ballot_sync(0xffffffffu, x == x && key > best.bound);
                }
                if (with >> lane & 1u) best.keys[best.count + __popc(with & ((1u << lane) - 1u))] = key;
                best.count += __popc(with);
            }
        }
    }
    if (best.count > best.n) keep_best(best, lane);
    // the warp's sum, then the block's, in a fixed order
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float t = __shfl_xor_sync(0xffffffffu, top, o), s = __shfl_xor_sync(0xffffffffu, sum, o);
        const float m = fmaxf(top, t);
        // lanes that swap have to round alike: the two products are added, whichever is whose
        sum = __fadd_rn(__fmul_rn(sum, ex2((top - m) * kLog2e)), __fmul_rn(s, ex2((t - m) * kLog2e)));
        top = m;
    }
    if (lane == 0) {
        warp_sums[warp] = make_float2(top, sum);
        counts[warp] = best.count;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float m = kLowest, s = 0.f;
        for (int w = 0; w < kScanWarps; ++w) m = fmaxf(m, warp_sums[w].x);
        for (int w = 0; w < kScanWarps; ++w) s += warp_sums[w].y * ex2((warp_sums[w].x - m) * kLog2e);
        sums[blockIdx.x] = make_float2(m, s);
    }
    int total = 0, before = 0;
    for (int w = 0; w < kScanWarps; ++w) {
        if (w < warp) before += counts[w];
        total += counts[w];
    }
    for (int i = lane; i < best.count; i += 32) merged[before + i] = best.keys[i];
    __syncthreads();
    uint64_t* to = out + static_cast<int64_t>(blockIdx.x) * a.n_out;
    for (int i = threadIdx.x; i < total; i += kScanThreads) {
        const uint64_t k = merged[i];
        int place = 0;
        for (int j = 0; j < total; ++j) place += merged[j] > k;
        if (place < a.n_out) to[place] = k;
    }
    for (int i = total + threadIdx.x; i < a.n_out; i += kScanThreads) to[i] = 0;
}

// A candidate of a lane: its score, and its row and token in one number, the
// lower the better.
struct Candidate {
    double score;
    uint64_t id;
};

__device__ __forceinline__ bool better(const Candidate& x, const Candidate& y)
{
    return x.score > y.score || (x.score == y.score && x.id < y.id);
}

// A block per lane.
__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const __grid_constant__ BeamArgs a, int parts, const float2* sums,
                                                                 const uint64_t* keys)
{
    enum { kNone, kGoesOn, kFinished };
    __shared__ double scores[64], z[64];
    __shared__ int state[64];
    __shared__ Candidate warps[kJoinThreads / 32];
    pdl_enter();
    const int lane = blockIdx.x, tid = threadIdx.x, row0 = lane * a.beams;
    if (tid < a.beams) {
        const int row = row0 + tid;
        const float s = a.scores[row];
        int st = kNone;
        double zr = 0.0;
        if (s != s || s == INFINITY) {
            set_device_status(a.status, QG_ERR_INVALID_ARG);
        } else if (s > -INFINITY) {
            if (a.finished && a.finished[row]) {
                st = kFinished;
            } else {
                float top = kLowest;
                for (int p = 0; p < parts; ++p) top = fmaxf(top, sums[static_cast<int64_t>(row) * parts + p].x);
                double sum = 0.0;
                for (int p = 0; p < parts; ++p) {
                    const float2 x = sums[static_cast<int64_t>(row) * parts + p];
                    sum += x.y * exp(static_cast<double>(x.x) - top);
                }
                if (!(sum >= 0.0 && sum < INFINITY))
                    set_device_status(a.status, QG_ERR_INVALID_ARG);
                else if (sum > 0.0) {
                    st = kGoesOn;
                    zr = top + log(sum);
                }
            }
        }
        scores[tid] = s;
        z[tid] = zr;
        state[tid] = st;
    }
    __syncthreads();
    const int per_row = parts * a.n_out, all = a.beams * per_row;
    const Candidate none{-INFINITY, ~0ull};
    Candidate last{INFINITY, 0};
    for (int o = 0; o < a.n_out; ++o) {
        Candidate best = none;
        for (int i = tid; i < all; i += kJoinThreads) {
            const int beam = i / per_row, place = i % per_row;
            const int row = row0 + beam;
            Candidate c = none;
            if (state[beam] == kFinished) {
                if (place == 0) c = Candidate{scores[beam], static_cast<uint64_t>(row) << 24 | static_cast<uint32_t>(a.pad)};
            } else if (state[beam] == kGoesOn) {
                const uint64_t key = keys[static_cast<int64_t>(row) * per_row + place];
                if (key)
                    c = Candidate{scores[beam] + (static_cast<double>(key_value(key)) - z[beam]),
                                  static_cast<uint64_t>(row) << 24 | key_token(key)};
            }
            if (better(last, c) && better(c, best)) best = c;
        }
#pragma unroll
        for (int s = 16; s; s >>= 1) {
            const Candidate c{__shfl_xor_sync(0xffffffffu, best.score, s), __shfl_xor_sync(0xffffffffu, best.id, s)};
            if (better(c, best)) best = c;
        }
        if ((tid & 31) == 0) warps[tid >> 5] = best;
        __syncthreads();
        best = warps[0];
        for (int w = 1; w < kJoinThreads / 32; ++w)
            if (better(warps[w], best)) best = warps[w];
        __syncthreads();
        last = best;
        if (tid == 0) {
            const int64_t at = static_cast<int64_t>(lane) * a.n_out + o;
            const bool some = best.id != ~0ull;
            const int row = some ? static_cast<int>(best.id >> 24) : row0;
            const int token = some ? static_cast<int>(best.id & 0xFFFFFFu) : a.pad;
            a.out_scores[at] = static_cast<float>(best.score);
            a.out_tokens[at] = token;
            a.out_parents[at] = row;
            if (a.out_finished) a.out_finished[at] = some && (state[row - row0] == kFinished || token == a.eos);
        }
    }
}

// How a call's rows are cut: parts of whole block tiles.
struct Cut {
    int parts;
    int span;
};

Cut cut_rows(int lanes, int beams, int vocab)
{
    const int tile = kScanWarps * kTile, rows = lanes * beams > 0 ? lanes * beams : 1;
    const int most = (vocab + tile - 1) / tile, want = (4 * sm_count(-1) + rows - 1) / rows;
    Cut c;
    c.span = ((most + min(most, want) - 1) / min(most, want)) * tile;
    c.parts = (vocab + c.span - 1) / c.span;
    return c;
}

size_t sums_bytes(int lanes, int beams, int parts)
{
    return (static_cast<size_t>(lanes) * beams * parts * sizeof(float2) + 255) / 256 * 256;
}

}  // namespace

size_t beam_select_workspace_bytes(int lanes, int beams, int vocab, int n_out)
{
    const Cut c = cut_rows(lanes, beams, vocab);
    return sums_bytes(lanes, beams, c.parts) + static_cast<size_t>(lanes) * beams * c.parts * n_out * sizeof(uint64_t) + 256;
}

qg_status launch_beam_select(const BeamArgs& in, void* workspace, cudaStream_t stream)
{
    BeamArgs a = in;
    a.status = device_status_ptr();
    if (!a.status) return QG_ERR_CUDA;
    const Cut c = cut_rows(a.lanes, a.beams, a.vocab);
    float2* sums = static_cast<float2*>(workspace);
    uint64_t* keys = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + sums_bytes(a.lanes, a.beams, c.parts));
    auto scan = a.f32 ? beam_scan_kernel<true> : beam_scan_kernel<false>;
    cudaError_t e = launch_pdl(scan, dim3(static_cast<unsigned>(a.lanes * a.beams * c.parts)), dim3(kScanThreads), 0, stream,
                               a, c.parts, c.span, sums, keys);
    if (e == cudaSuccess)
        e = launch_pdl(beam_join_kernel, dim3(static_cast<unsigned>(a.lanes)), dim3(kJoinThreads), 0, stream, a, c.parts,
                       static_cast<const float2*>(sums), static_cast<const uint64_t*>(keys));
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

}  // namespace qg

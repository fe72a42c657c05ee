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
constexpr int kList = 1024;                          // tokens a block can hold
constexpr int kJoinThreads = 1024, kJoinWarps = kJoinThreads / 32;
constexpr int kJoinKeys = 8;                         // candidates a thread of the join takes at a time
constexpr int kGroups = 128;                         // candidates' groups, by whose best one is bounded
constexpr int kPairs = 1024;                         // parts of a lane's rows, at most
constexpr int kPicked = 512;                         // candidates of a lane that are looked at in 64 bits
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

__device__ __forceinline__ float warp_max(float v)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// The n-th largest of the warp's values, n <= 32.
__device__ __forceinline__ float nth_of_warp(float v, int n)
{
    for (;;) {
        const float most = warp_max(v);
        if (--n == 0) return most;
        if (__ffs(__ballot_sync(0xffffffffu, v == most)) - 1 == static_cast<int>(threadIdx.x & 31)) v = -INFINITY;
    }
}

// A part of a row: the maximum and the scaled sum of its exponentials, and how
// many of its tokens are handed on.
struct PartSum {
    float top;
    float sum;
    int count;
    int pad;
};

// A block's tokens that may be among its n best: those above `bound`, a key
// that n of the block's tokens reach.
struct ScanSmem {
    uint64_t list[kList];
    uint64_t bound;
    int count;
    float tops[kScanWarps];
    float2 sums[kScanWarps];
};

// Keep the n best of the first k keys, in order: a key's place is the number
// of greater ones.
__device__ __forceinline__ void keep_best(ScanSmem& s, int k, int n)
{
    constexpr int kMine = kList / kScanThreads;
    uint64_t mine[kMine];
    int place[kMine];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int at = threadIdx.x + i * kScanThreads;
        mine[i] = at < k ? s.list[at] : 0;
        place[i] = 0;
    }
    if (k <= kScanThreads) {
        for (int j = 0; j < k; ++j) place[0] += s.list[j] > mine[0];
    } else {
        for (int j = 0; j < k; ++j) {
            const uint64_t x = s.list[j];
#pragma unroll
            for (int i = 0; i < kMine; ++i) place[i] += x > mine[i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i)
        if (mine[i] && place[i] < n) {
            s.list[place[i]] = mine[i];
            if (place[i] == n - 1) s.bound = mine[i];
        }
    if (threadIdx.x == 0) s.count = min(k, n);
    __syncthreads();
}

// A block takes a part of a row, U * 8 values per thread at a time. Its bound
// starts from the first of these: the m-th largest of a warp's threads'
// maxima, the least over w warps, with m w >= n, is reached by n tokens. Few
// tokens reach it (about n H(w) of independent ones for m = 1), and the list
// that these fill is cut to its n best when it is long, which raises the bound.
template <bool F32, int U>
__global__ void __launch_bounds__(kScanThreads, 4) beam_scan_kernel(const __grid_constant__ BeamArgs a, int parts, int span, int slots,
                                                                 PartSum* sums, uint64_t* out)
{
    __shared__ ScanSmem s;
    constexpr int kTile = kScanThreads * kVec * U;
    pdl_enter();
    const int row_i = blockIdx.x / parts, part = blockIdx.x % parts;
    if (!row_live(a, row_i)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.n_out;
    const uint8_t* row = static_cast<const uint8_t*>(a.logits) + row_i * a.stride * (F32 ? 4 : 2);
    const int begin = part * span, end = min(begin + span, a.vocab);
    if (tid == 0) {
        s.count = 0;
        s.bound = make_key(-INFINITY, 0);
    }
    uint64_t bound = make_key(-INFINITY, 0);
    float top = kLowest, sum = 0.f;
    for (int base = begin; base < end; base += kTile) {
        float v[U][kVec];
#pragma unroll
        for (int u = 0; u < U; ++u) load8<F32>(row, a.vocab, base + (u * kScanThreads + tid) * kVec, v[u]);
        float tops[U], most = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            tops[u] = -INFINITY;
#pragma unroll
            for (int i = 0; i < kVec; ++i) tops[u] = fmaxf(tops[u], v[u][i]);
            most = fmaxf(most, tops[u]);
        }
        if (most > top) {
            sum *= ex2((top - most) * kLog2e);
            top = most;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < kVec; ++i) sum += ex2((v[u][i] - top) * kLog2e);
        if (base == begin) {
            const int warps = max(1, min(kScanWarps, (end - begin) / (32 * kVec)));    // whose threads all have values
            const int m = (n + warps - 1) / warps;
            if (m <= 32) {
                const float t = nth_of_warp(most, m);
                if (lane == 0) s.tops[warp] = t;
                __syncthreads();
                float least = s.tops[0];
                for (int w = 1; w < warps; ++w) least = fminf(least, s.tops[w]);
                if (least > -INFINITY) bound = make_key(least, 0xFFFFFFFFu) - 1;
            } else {
                __syncthreads();
            }
        }
        for (;;) {
            const float least = key_value(bound);
            int seen = 0;
            if (__any_sync(0xffffffffu, most >= least)) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (U > 1 && !__any_sync(0xffffffffu, tops[u] >= least)) continue;
                    uint32_t hits = 0;
#pragma unroll
                    for (int i = 0; i < kVec; ++i) hits |= static_cast<uint32_t>(v[u][i] >= least) << i;
                    while (__any_sync(0xffffffffu, hits != 0)) {
                        const int at = __ffs(hits) - 1;
                        float x = v[u][0];
#pragma unroll
                        for (int i = 1; i < kVec; ++i) x = i == at ? v[u][i] : x;
                        const uint64_t key = make_key(x, static_cast<uint32_t>(base + (u * kScanThreads + tid) * kVec + at));
                        const uint32_t with = __ballot_sync(0xffffffffu, hits && key > bound);
                        int place = 0;
                        if (lane == 0 && with) place = atomicAdd(&s.count, __popc(with));
                        place = __shfl_sync(0xffffffffu, place, 0);
                        seen = max(seen, place + __popc(with));
                        place += __popc(with & ((1u << lane) - 1u));
                        if ((with >> lane & 1u) && place < kList) s.list[place] = key;
                        hits &= hits - 1;
                    }
                }
            }
            if (!__syncthreads_or(seen > 2 * slots)) break;
            // a long list: cut, which raises the bound
            const int k = s.count;
            keep_best(s, min(k, kList), n);
            bound = s.bound;
            if (k <= kList) break;
            // some found no place: those of this tile are taken again, above the new bound (each turn at least
            // kList - n fewer)
            __syncthreads();
            if (warp == 0) {
                const uint64_t k0 = lane < n ? s.list[lane] : 0, k1 = lane + 32 < n ? s.list[lane + 32] : 0;
                const bool old0 = k0 && key_token(k0) < static_cast<uint32_t>(base);
                const bool old1 = k1 && key_token(k1) < static_cast<uint32_t>(base);
                const uint32_t b0 = __ballot_sync(0xffffffffu, old0), b1 = __ballot_sync(0xffffffffu, old1);
                __syncwarp();
                if (old0) s.list[__popc(b0 & ((1u << lane) - 1u))] = k0;
                if (old1) s.list[__popc(b0) + __popc(b1 & ((1u << lane) - 1u))] = k1;
                if (lane == 0) s.count = __popc(b0) + __popc(b1);
            }
            bound -= 1;
            __syncthreads();
        }
    }
    // the warp's sum, then the block's, in a fixed order
    const float warp_top = warp_max(top);
    sum *= ex2((top - warp_top) * kLog2e);
    top = warp_top;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s.sums[warp] = make_float2(top, sum);
    __syncthreads();
    int k = s.count;
    if (k > slots) {
        keep_best(s, k, n);
        k = n;
    }
    if (tid == 0) {
        float m = kLowest, x = 0.f;
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) m = fmaxf(m, s.sums[w].x);
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) x += s.sums[w].y * ex2((s.sums[w].x - m) * kLog2e);
        sums[blockIdx.x] = PartSum{m, x, k, 0};
    }
    for (int i = tid; i < k; i += kScanThreads) out[static_cast<int64_t>(blockIdx.x) * slots + i] = s.list[i];
}

// A candidate of a lane: its score as a whole number of the same order, and
// its row and token in one number, the lower the better. {0, ~0}: none.
struct Candidate {
    uint64_t score;
    uint64_t id;
};

__device__ __forceinline__ bool better(const Candidate& x, const Candidate& y)
{
    return x.score > y.score || (x.score == y.score && x.id < y.id);
}

__device__ __forceinline__ uint64_t ordered64(double v)
{
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return b ^ (b >> 63 ? ~0ull : 1ull << 63);
}

__device__ __forceinline__ double value64(uint64_t o)
{
    return __longlong_as_double(static_cast<long long>(o ^ (o >> 63 ? 1ull << 63 : ~0ull)));
}

enum RowState { kNone, kGoesOn, kFinished };

struct JoinSmem {
    double z[64];                // ln of the row's sum
    float score[64];
    float base[64];              // score - z, rounded
    int state[64];
    int parts[kPairs];           // handed-on tokens of a part, and its beam from bit 16 on
    float4 best[kGroups / 4];
    uint64_t keys[kPicked];
    int beams[kPicked];          // of the keys picked; -1 - beam: its finished row's one candidate
    Candidate picked[kPicked];
    Candidate warps[kJoinWarps];
    float bound;
    int count;
};

// ln x of a normal x >= 1, within 6e-8: with x = 2^k m, m in [sqrt(1/2),
// sqrt(2)), and t = (m - 1) / (m + 1), ln m = 2 (t + t^3/3 + t^5/5 + ...), |t| <
// 0.172; six terms leave less than 1e-10, t is off by 2^-23 of it.
__device__ __forceinline__ float split_log(float x, int& k)
{
    const uint32_t b = __float_as_uint(x);
    k = static_cast<int>((b - 0x3F3504F3u) >> 23);
    const float m = __uint_as_float(b - (static_cast<uint32_t>(k) << 23));
    const float d = m + 1.f;
    float t = __fdividef(m - 1.f, d);
    t = fmaf(fmaf(-t, d, m - 1.f), 0.5f, t);             // what the quotient misses, over a rough d
    const float q = t * t;
    float p = 1.f / 11.f;
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    return fmaf(p * q, 2.f * t, 2.f * t);
}

// Candidate `i` of a beam's part from its key, in 64 bits.
__device__ __forceinline__ Candidate candidate(const JoinSmem& s, int row0, int beam, uint64_t key)
{
    return Candidate{ordered64(static_cast<double>(s.score[beam]) + (static_cast<double>(key_value(key)) - s.z[beam])),
                     static_cast<uint64_t>(row0 + beam) << 24 | key_token(key)};
}

__device__ __forceinline__ Candidate finished_candidate(const BeamArgs& a, const JoinSmem& s, int row0, int beam)
{
    return Candidate{ordered64(s.score[beam]), static_cast<uint64_t>(row0 + beam) << 24 | static_cast<uint32_t>(a.pad)};
}

__device__ __forceinline__ void write_out(const BeamArgs& a, const JoinSmem& s, int row0, int place, const Candidate& c)
{
    const int64_t at = static_cast<int64_t>(blockIdx.x) * a.n_out + place;
    const bool some = c.id != ~0ull;
    const int row = some ? static_cast<int>(c.id >> 24) : row0;
    const int token = some ? static_cast<int>(c.id & 0xFFFFFFu) : a.pad;
    a.out_scores[at] = some ? static_cast<float>(value64(c.score)) : -INFINITY;
    a.out_tokens[at] = token;
    a.out_parents[at] = row;
    if (a.out_finished) a.out_finished[at] = some && (s.state[row - row0] == kFinished || token == a.eos);
}

// A block per lane. A candidate's score in 32 bits, f, is off by less than e =
// 2^-21 (|score - z| + |logit|): score - z is rounded once and the sum with the
// logit once, 2^-24 of each. The n-th largest of the groups' best f - e is
// reached by n candidates, so only those with f + e at or above it are looked
// at in 64 bits (which this GPU adds and compares slowly).
__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const __grid_constant__ BeamArgs a, int parts, int slots_log2,
                                                                 const PartSum* sums, const uint64_t* keys)
{
    __shared__ JoinSmem s;
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.n_out;
    const int row0 = static_cast<int>(blockIdx.x) * a.beams;
    const int all = a.beams * parts << slots_log2, mask = (1 << slots_log2) - 1;
    const uint64_t* mine = keys + (static_cast<int64_t>(row0) * parts << slots_log2);
    // the first keys are on their way while the sums are joined; whether they are any is known then
    uint64_t key[kJoinKeys];
#pragma unroll
    for (int r = 0; r < kJoinKeys; ++r) {
        const int i = r * kJoinThreads + tid;
        key[r] = i < all ? mine[i] : 0;
    }
    for (int beam = warp; beam < a.beams; beam += kJoinWarps) {
        const int row = row0 + beam;
        const float score = a.scores[row];
        const bool done = a.finished && a.finished[row];
        int state = kNone;
        double z = 0.0;
        if (!(score > -INFINITY && score < INFINITY)) {
            if (lane == 0 && score != -INFINITY) set_device_status(a.status, QG_ERR_INVALID_ARG);
        } else if (done) {
            state = kFinished;
        } else {
            const PartSum* p = sums + static_cast<int64_t>(row) * parts;
            float top = kLowest, sum = 0.f;
            for (int i = lane; i < parts; i += 32) {
                const PartSum x = p[i];
                s.parts[beam * parts + i] = x.count | beam << 16;
                const float m = fmaxf(top, x.top);
                sum = sum * ex2((top - m) * kLog2e) + x.sum * ex2((x.top - m) * kLog2e);
                top = m;
            }
            const float most = warp_max(top);
            sum *= ex2((top - most) * kLog2e);
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (!(sum >= 0.f && sum < INFINITY)) {
                if (lane == 0) set_device_status(a.status, QG_ERR_INVALID_ARG);
            } else if (sum > 0.f) {
                int k;
                const float l = split_log(sum, k);
                state = kGoesOn;
                z = fma(static_cast<double>(k), 0.69314718055994531, static_cast<double>(most)) + l;
            }
        }
        if (state != kGoesOn)
            for (int i = lane; i < parts; i += 32) s.parts[beam * parts + i] = beam << 16;
        if (lane == 0) {
            s.score[beam] = score;
            s.z[beam] = z;
            s.base[beam] = static_cast<float>(score - z);
            s.state[beam] = state;
        }
    }
    if (tid == 0) {
        s.bound = -INFINITY;
        s.count = 0;
    }
    __syncthreads();

    const float kOff = 4.76837158e-7f;                  // 2^-21
    float best = -INFINITY;
    for (int i0 = 0; i0 < all; i0 += kJoinKeys * kJoinThreads) {
#pragma unroll
        for (int r = 0; r < kJoinKeys; ++r) {
            const int i = i0 + r * kJoinThreads + tid;
            if (i0 && i < all) key[r] = mine[i];
            if (i >= all) continue;
            const int p = s.parts[i >> slots_log2];
            const float x = key_value(key[r]), base = s.base[p >> 16];
            if ((i & mask) < (p & 0xFFFF)) best = fmaxf(best, base + x - kOff * (fabsf(base) + fabsf(x)));
        }
    }
    if (tid < a.beams && s.state[tid] == kFinished) best = fmaxf(best, s.score[tid]);
#pragma unroll
    for (int o = 1; o < kJoinThreads / kGroups; o <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
    float* bests = reinterpret_cast<float*>(s.best);
    if (tid % (kJoinThreads / kGroups) == 0) bests[tid / (kJoinThreads / kGroups)] = best;
    __syncthreads();
    if (tid < kGroups) {
        const float x = bests[tid];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < kGroups / 4; ++j) {
            const float4 y = s.best[j];
            place += (y.x > x || (y.x == x && 4 * j < tid)) + (y.y > x || (y.y == x && 4 * j + 1 < tid)) +
                     (y.z > x || (y.z == x && 4 * j + 2 < tid)) + (y.w > x || (y.w == x && 4 * j + 3 < tid));
        }
        if (place == n - 1) s.bound = x;
    }
    __syncthreads();
    const float bound = s.bound;
    auto pick = [&](uint64_t k, int beam) {
        const int at = atomicAdd(&s.count, 1);
        if (at < kPicked) {
            s.keys[at] = k;
            s.beams[at] = beam;
        }
    };
    for (int i0 = 0; i0 < all; i0 += kJoinKeys * kJoinThreads) {
#pragma unroll
        for (int r = 0; r < kJoinKeys; ++r) {
            const int i = i0 + r * kJoinThreads + tid;
            if (all > kJoinKeys * kJoinThreads && i < all) key[r] = mine[i];
            if (i >= all) continue;
            const int p = s.parts[i >> slots_log2];
            const float x = key_value(key[r]), base = s.base[p >> 16];
            if ((i & mask) < (p & 0xFFFF) && !(base + x + kOff * (fabsf(base) + fabsf(x)) < bound)) pick(key[r], p >> 16);
        }
    }
    if (tid < a.beams && s.state[tid] == kFinished && s.score[tid] >= bound) pick(0, -1 - tid);
    __syncthreads();
    const int count = s.count;
    if (count <= kPicked) {
        // a candidate's place is the number of better ones
        Candidate c{0, ~0ull};
        if (tid < count) {
            const int beam = s.beams[tid];
            c = beam < 0 ? finished_candidate(a, s, row0, -1 - beam) : candidate(s, row0, beam, s.keys[tid]);
            s.picked[tid] = c;
        }
        __syncthreads();
        int place = 0;
        if (tid < count)
            for (int j = 0; j < count; ++j) place += better(s.picked[j], c);
        if (tid >= count) place = tid;
        if (place < n) write_out(a, s, row0, place, c);
        return;
    }
    // more candidates within the rounding of each other than are held: the best of what is left, one after another
    Candidate last{~0ull, 0};
    for (int o = 0; o < n; ++o) {
        Candidate c{0, ~0ull};
        for (int i = tid; i < all; i += kJoinThreads) {
            const int p = s.parts[i >> slots_log2];
            if ((i & mask) >= (p & 0xFFFF)) continue;
            const Candidate x = candidate(s, row0, p >> 16, mine[i]);
            if (better(last, x) && better(x, c)) c = x;
        }
        if (tid < a.beams && s.state[tid] == kFinished) {
            const Candidate x = finished_candidate(a, s, row0, tid);
            if (better(last, x) && better(x, c)) c = x;
        }
#pragma unroll
        for (int h = 16; h; h >>= 1) {
            const Candidate x{__shfl_xor_sync(0xffffffffu, c.score, h), __shfl_xor_sync(0xffffffffu, c.id, h)};
            if (better(x, c)) c = x;
        }
        if (lane == 0) s.warps[warp] = c;
        __syncthreads();
        c = s.warps[0];
        for (int w = 1; w < kJoinWarps; ++w)
            if (better(s.warps[w], c)) c = s.warps[w];
        __syncthreads();
        last = c;
        if (tid == 0) write_out(a, s, row0, o, c);
    }
}

// How a call's rows are cut: parts of whole tiles, and the tokens that each may
// hand on.
struct Cut {
    int unroll;
    int parts;
    int span;
    int slots_log2;
};

Cut cut_rows(int lanes, int beams, int vocab, int n_out)
{
    const int rows = lanes * beams > 0 ? lanes * beams : 1, sms = sm_count(-1);
    const int64_t values = static_cast<int64_t>(rows) * vocab;
    Cut c;
    c.unroll = values <= static_cast<int64_t>(sms) * 2 * 4096 ? 1 : values <= static_cast<int64_t>(sms) * 4 * 8192 ? 2 : 4;
    const int tile = kScanThreads * kVec * c.unroll;
    const int most = (vocab + tile - 1) / tile, want = min((4 * sms + rows - 1) / rows, kPairs / beams);
    c.span = ((most + min(most, want) - 1) / min(most, want)) * tile;
    c.parts = (vocab + c.span - 1) / c.span;
    c.slots_log2 = n_out <= 8 ? 5 : n_out <= 24 ? 6 : n_out <= 48 ? 7 : 8;
    return c;
}

size_t sums_bytes(int lanes, int beams, int parts)
{
    return (static_cast<size_t>(lanes) * beams * parts * sizeof(PartSum) + 255) / 256 * 256;
}

}  // namespace

size_t beam_select_workspace_bytes(int lanes, int beams, int vocab, int n_out)
{
    const Cut c = cut_rows(lanes, beams, vocab, n_out);
    return sums_bytes(lanes, beams, c.parts) + (static_cast<size_t>(lanes) * beams * c.parts << c.slots_log2) * sizeof(uint64_t) + 256;
}

qg_status launch_beam_select(const BeamArgs& in, void* workspace, cudaStream_t stream)
{
    BeamArgs a = in;
    a.status = device_status_ptr();
    if (!a.status) return QG_ERR_CUDA;
    const Cut c = cut_rows(a.lanes, a.beams, a.vocab, a.n_out);
    PartSum* sums = static_cast<PartSum*>(workspace);
    uint64_t* keys = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + sums_bytes(a.lanes, a.beams, c.parts));
    auto pick = [&](auto u1, auto u2, auto u4) { return c.unroll == 1 ? u1 : c.unroll == 2 ? u2 : u4; };
    auto scan = a.f32 ? pick(beam_scan_kernel<true, 1>, beam_scan_kernel<true, 2>, beam_scan_kernel<true, 4>)
                      : pick(beam_scan_kernel<false, 1>, beam_scan_kernel<false, 2>, beam_scan_kernel<false, 4>);
    cudaError_t e = launch_pdl(scan, dim3(static_cast<unsigned>(a.lanes * a.beams * c.parts)), dim3(kScanThreads), 0, stream,
                               a, c.parts, c.span, 1 << c.slots_log2, sums, keys);
    if (e == cudaSuccess)
        e = launch_pdl(beam_join_kernel, dim3(static_cast<unsigned>(a.lanes)), dim3(kJoinThreads), 0, stream, a, c.parts,
                       c.slots_log2, static_cast<const PartSum*>(sums), static_cast<const uint64_t*>(keys));
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

}  // namespace qg

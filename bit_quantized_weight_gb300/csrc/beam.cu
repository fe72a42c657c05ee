// beam.cu -- beam search's selection: the best continuations of a lane over
// its beams and the vocabulary (beam_select).
//
// score(r, t) = scores[r] + logits[r][t] - ln sum_t' exp(logits[r][t']): a
// row's sum is needed before its tokens can be compared with another row's, so
// one kernel reads all logits and leaves, of every piece of 1,024, the maximum
// and the sum of the exponentials scaled to it; a second joins a lane's sums.
// The n_out best tokens lie in the n_out pieces whose maxima have the best
// scores (a token of any other piece is worse than those maxima, or equal and
// behind them), so it reads just these again.
#include "kv_common.cuh"

namespace qg {
namespace {

constexpr int kPiece = 1024;                         // values, 32 of a lane
constexpr int kScanWarps = 8;                        // of a block, at most
constexpr int kGroups = 128;                         // candidates' groups, by whose best one is bounded
constexpr int kPieces = 128;                         // pieces of a lane that are read again, if more than n_out
constexpr int kPicked = 512;                         // candidates of a lane that are looked at in 64 bits,
constexpr int kFew = 96;                             // if their number was not bounded twice
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

// N values of each lane from `base` on of a row of `vocab`, -infinity behind
// its end: pieces of 16 bytes, one lane's after the other. The same values go
// to the same lane whatever the row's alignment: fp32 rows that do not start at
// 16 bytes, and the last values of a row, are read one by one, bf16 rows in the
// aligned pieces around a lane's. (Plain loads: the kernel before may have
// written them while this one had started already.)
template <bool F32, int N>
__device__ __forceinline__ void load_values(const uint8_t* row, int vocab, int base, float (&v)[N])
{
    constexpr int kSize = F32 ? 4 : 2, kN = 16 / kSize;
    const int lane = threadIdx.x & 31, skip = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
    const uint8_t* at = row + static_cast<int64_t>(base + lane * kN) * kSize - skip;
    if (base + 32 * N <= vocab && skip == 0) {
#pragma unroll
        for (int u = 0; u < N / kN; ++u) {
            const uint4 x = *reinterpret_cast<const uint4*>(at + 512 * u);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < kN; ++i)
                v[u * kN + i] = F32 ? __uint_as_float(w[i]) : __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        }
    } else if (!F32 && base + 32 * N + kN <= vocab) {
#pragma unroll
        for (int u = 0; u < N / kN; ++u) {
            const uint4 x = *reinterpret_cast<const uint4*>(at + 512 * u), y = *reinterpret_cast<const uint4*>(at + 512 * u + 16);
            uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            shift_words(w, skip);
#pragma unroll
            for (int i = 0; i < kN; ++i) v[u * kN + i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        }
    } else {
        at += skip;
        const int left = vocab - base - lane * kN;
#pragma unroll
        for (int u = 0; u < N / kN; ++u)
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                v[u * kN + i] = -INFINITY;
                if (32 * kN * u + i < left)
                    v[u * kN + i] = F32 ? reinterpret_cast<const float*>(at + 512 * u)[i]
                                        : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(at + 512 * u)[i]);
            }
    }
}

// Which token the i-th of these values is.
template <bool F32>
__device__ __forceinline__ int token_of(int base, int i)
{
    constexpr int kN = F32 ? 4 : 8;
    return base + (i / kN * 32 + static_cast<int>(threadIdx.x & 31)) * kN + i % kN;
}

__device__ __forceinline__ float warp_max(float v)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Of some of a row's logits: the maximum and the sum of the exponentials,
// scaled to it.
struct ScaledSum {
    float top;
    float sum;
};

__device__ __forceinline__ void join_sums(ScaledSum& x, float top, float sum)
{
    const float m = fmaxf(x.top, top);
    x.sum = x.sum * ex2((x.top - m) * kLog2e) + sum * ex2((top - m) * kLog2e);
    x.top = m;
}

// Over the warp, in a fixed order.
__device__ __forceinline__ void warp_sum(ScaledSum& x)
{
    const float top = warp_max(x.top);
    x.sum *= ex2((x.top - top) * kLog2e);
    x.top = top;
#pragma unroll
    for (int o = 16; o; o >>= 1) x.sum += __shfl_xor_sync(0xffffffffu, x.sum, o);
}

__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

// sum of 2^((v - top) log2 e), two values an instruction but for 2^x.
template <int N>
__device__ __forceinline__ float exp_sum(const float (&v)[N], float top)
{
    const uint64_t off = pair(-top, -top), scale = pair(kLog2e, kLog2e);
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        uint64_t x;
        float lo, hi;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(pair(v[i], v[i + 1])), "l"(off));
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(x), "l"(scale));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(sum) : "l"(sum), "l"(pair(ex2(lo), ex2(hi))));
    }
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(sum));
    return lo + hi;
}

// A warp per piece. Nothing is kept from one to the next, and blocks need no
// order: as many loads are on their way as registers hold. Bound by the
// logits' bytes: 512 rows of 131,072 fp32 logits in 43 us, 6.2 TB/s. (Passes
// that kept a list of the best tokens as they went, over rings of bulk copies,
// took 66 us and more: the lists' branches and the registers for them left too
// few warps to cover each other's waits.)
template <bool F32>
__global__ void __launch_bounds__(32 * kScanWarps, 4) beam_scan_kernel(const __grid_constant__ BeamArgs a, int pieces, ScaledSum* sums)
{
    pdl_enter();
    const int at = static_cast<int>(blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32);
    const int row = at / pieces;
    if (row >= a.lanes * a.beams || !row_live(a, row)) return;
    float v[kPiece / 32];
    load_values<F32>(static_cast<const uint8_t*>(a.logits) + row * a.stride * (F32 ? 4 : 2), a.vocab, at % pieces * kPiece, v);
    float top = kLowest;
#pragma unroll
    for (int i = 0; i < kPiece / 32; ++i) top = fmaxf(top, v[i]);
    top = warp_max(top);
    float sum = exp_sum(v, top);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) sums[at] = ScaledSum{top, sum};
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

template <int kThreads>
struct JoinSmem {
    double z[64];                // ln of the row's sum
    float score[64];
    float base[64];              // score - z, rounded
    int state[64];
    float4 best[kGroups / 4];
    float mine[kThreads];
    int pieces[kPieces];
    uint64_t keys[kPicked];
    int beams[kPicked];          // of the keys picked; -1 - beam: its finished row's one candidate
    Candidate picked[kPicked];
    Candidate warps[kThreads / 32];
    float bound;
    int n_pieces;
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

// A block per lane, bound by its chain of loads and barriers: 8 beams of 65,536
// tokens in 4.5 us (sums 1.5, pieces 1.4, tokens 1.2, order and outputs 0.4) of
// 6.9 with the scan. A candidate's score in 32 bits, f, is off by less than e =
// 2^-21 (|score - z| + |logit|): score - z is rounded once and the sum with the
// logit once, 2^-24 of each. The n-th largest of the groups' best f - e is
// reached by n candidates, so only those with f + e at or above it are looked
// at in 64 bits (which this GPU adds and compares slowly).
template <bool F32, int kThreads>
__global__ void __launch_bounds__(kThreads) beam_join_kernel(const __grid_constant__ BeamArgs a, int pieces, const ScaledSum* sums)
{
    __shared__ JoinSmem<kThreads> s;
    constexpr int kWarps = kThreads / 32;
    constexpr float kOff = 4.76837158e-7f;             // 2^-21
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.n_out;
    const int row0 = static_cast<int>(blockIdx.x) * a.beams, all = a.beams * pieces;
    const ScaledSum* mine = sums + static_cast<int64_t>(row0) * pieces;
    for (int beam = warp; beam < a.beams; beam += kWarps) {
        // the first sums are on their way before it is known whether they are any
        const ScaledSum* p = mine + beam * pieces;
        ScaledSum x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = i * 32 + lane < pieces ? p[i * 32 + lane] : ScaledSum{kLowest, 0.f};
        const float score = a.scores[row0 + beam];
        const bool done = a.finished && a.finished[row0 + beam];
        int state = kNone;
        double z = 0.0;
        if (!(score > -INFINITY && score < INFINITY)) {
            if (lane == 0 && score != -INFINITY) set_device_status(a.status, QG_ERR_INVALID_ARG);
        } else if (done) {
            state = kFinished;
        } else {
            ScaledSum r{fmaxf(fmaxf(x[0].top, x[1].top), fmaxf(x[2].top, x[3].top)), 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i) r.sum += x[i].sum * ex2((x[i].top - r.top) * kLog2e);
            for (int i = 128 + lane; i < pieces; i += 32) join_sums(r, p[i].top, p[i].sum);
            warp_sum(r);
            if (!(r.sum >= 0.f && r.sum < INFINITY)) {
                if (lane == 0) set_device_status(a.status, QG_ERR_INVALID_ARG);
            } else if (r.sum > 0.f) {
                int k;
                const float l = split_log(r.sum, k);
                state = kGoesOn;
                z = fma(static_cast<double>(k), 0.69314718055994531, static_cast<double>(r.top)) + l;
            }
        }
        if (lane == 0) {
            s.score[beam] = score;
            s.z[beam] = z;
            s.base[beam] = static_cast<float>(score - z);
            s.state[beam] = state;
        }
    }
    if (tid == 0) s.n_pieces = s.count = 0;
    __syncthreads();

    const bool finished = tid < a.beams && s.state[tid] == kFinished;
    auto lower = [&](int beam, float x) { return s.base[beam] + x - kOff * (fabsf(s.base[beam]) + fabsf(x)); };
    auto may_be = [&](int beam, float x, float bound) { return !(s.base[beam] + x + kOff * (fabsf(s.base[beam]) + fabsf(x)) < bound); };
    auto exact = [&](int beam, float x, int which) {
        return Candidate{ordered64(static_cast<double>(s.score[beam]) + (static_cast<double>(x) - s.z[beam])),
                         static_cast<uint64_t>(row0 + beam) << 24 | static_cast<uint32_t>(which)};
    };
    auto of_finished = [&](int beam) {
        return Candidate{ordered64(s.score[beam]), static_cast<uint64_t>(row0 + beam) << 24 | static_cast<uint32_t>(a.pad)};
    };
    // the n-th largest of the groups' best; -infinity if there are not as many
    auto nth_best = [&](float best) {
        if (finished) best = fmaxf(best, s.score[tid]);
        s.mine[tid] = best;
        __syncthreads();
        float* bests = reinterpret_cast<float*>(s.best);
        if (tid < kGroups) {
#pragma unroll
            for (int k = 1; k < kThreads / kGroups; ++k) best = fmaxf(best, s.mine[tid + k * kGroups]);
            bests[tid] = best;
        }
        __syncthreads();
        // some threads for each group, each with a share of the others
        constexpr int kEach = kThreads / kGroups;
        best = bests[tid / kEach];
        int above = 0, level = 0;
#pragma unroll
        for (int j = 0; j < kGroups / 4 / kEach; ++j) {
            const float4 y = s.best[j * kEach + tid % kEach];
            above += (y.x > best) + (y.y > best) + (y.z > best) + (y.w > best);
            level += (y.x == best) + (y.y == best) + (y.z == best) + (y.w == best);
        }
#pragma unroll
        for (int o = 1; o < kEach; o <<= 1) {
            above += __shfl_xor_sync(0xffffffffu, above, o);
            level += __shfl_xor_sync(0xffffffffu, level, o);
        }
        if (above < n && n <= above + level) s.bound = best;
        __syncthreads();
        return s.bound;
    };
    // the best of all threads' candidates, known to all
    auto best_of_block = [&](Candidate c) {
#pragma unroll
        for (int h = 16; h; h >>= 1) {
            const Candidate x{__shfl_xor_sync(0xffffffffu, c.score, h), __shfl_xor_sync(0xffffffffu, c.id, h)};
            if (better(x, c)) c = x;
        }
        if (lane == 0) s.warps[warp] = c;
        __syncthreads();
        c = s.warps[0];
        for (int w = 1; w < kWarps; ++w)
            if (better(s.warps[w], c)) c = s.warps[w];
        __syncthreads();
        return c;
    };

    // the pieces whose maxima may be among the n best
    auto each_piece = [&](auto&& f) {
        for (int i = tid; i < all; i += kThreads) {
            const int beam = i / pieces;
            if (s.state[beam] != kGoesOn) continue;
            const ScaledSum x = mine[i];
            if (x.sum > 0.f) f(i, beam, x.top);
        }
    };
    float best = -INFINITY;
    each_piece([&](int, int beam, float top) { best = fmaxf(best, lower(beam, top)); });
    float bound = nth_best(best);
    each_piece([&](int i, int beam, float top) {
        if (!may_be(beam, top, bound)) return;
        const int at = atomicAdd(&s.n_pieces, 1);
        if (at < kPieces) s.pieces[at] = i;
    });
    __syncthreads();
    int chosen = s.n_pieces;
    if (chosen > kPieces) {
        // too many within the rounding of each other: the best of what is left, one after another
        Candidate last{~0ull, 0};
        for (chosen = 0; chosen < n; ++chosen) {
            Candidate c{0, ~0ull};
            each_piece([&](int i, int beam, float top) {
                const Candidate x = exact(beam, top, i - beam * pieces);
                if (better(last, x) && better(x, c)) c = x;
            });
            c = last = best_of_block(c);
            if (c.id == ~0ull) break;
            if (tid == 0) s.pieces[chosen] = (static_cast<int>(c.id >> 24) - row0) * pieces + static_cast<int>(c.id & 0xFFFFFFu);
        }
        __syncthreads();
    }

    // their tokens that may be
    constexpr int kEach = kPiece / 32;
    auto logits_of = [&](int beam) { return static_cast<const uint8_t*>(a.logits) + (row0 + beam) * a.stride * (F32 ? 4 : 2); };
    auto each_chosen = [&](auto&& f) {                 // a warp for each
        for (int u = warp; u < chosen; u += kWarps) {
            const int i = s.pieces[u], beam = i / pieces, base = (i - beam * pieces) * kPiece;
            float v[kEach];
            load_values<F32>(logits_of(beam), a.vocab, base, v);
            f(beam, base, v);
        }
    };
    // Tokens whose f + e may reach the bound, while f(...) is true. With |x| <= 2 (|base| + |bound|) e is at most 3 2^-21 of that sum, and 2^-21
    // more of it is above what is rounded here; a lower x is too low by far.
    auto each_token = [&](auto&& f) {
        each_chosen([&](int beam, int base, const float (&v)[kEach]) {
            const float least = bound - s.base[beam] - 4.f * kOff * (fabsf(s.base[beam]) + fabsf(bound));
            uint32_t hits = 0;
#pragma unroll
            for (int k = 0; k < kEach; ++k) hits |= static_cast<uint32_t>(!(v[k] < least) && v[k] > -INFINITY) << k;
            const uint8_t* row = logits_of(beam);
            for (; hits; hits &= hits - 1) {           // few: read again, which spares a copy of this code for each
                const int token = token_of<F32>(base, __ffs(hits) - 1);
                const float x = F32 ? reinterpret_cast<const float*>(row)[token]
                                    : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(row)[token]);
                if (!f(beam, x, token)) break;
            }
        });
    };
    auto pick = [&](uint64_t key, int beam) {
        const int at = atomicAdd(&s.count, 1);
        if (at < kPicked) {
            s.keys[at] = key;
            s.beams[at] = beam;
        }
        return at < kPicked;
    };
    bool closer = bound == -INFINITY && chosen * kPiece > kFew;
    for (;;) {
        if (closer) {                                  // bounded by the tokens' groups too; either bound holds
            best = -INFINITY;
            each_chosen([&](int beam, int, const float (&v)[kEach]) {
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < kEach; ++k) top = fmaxf(top, v[k]);
                if (top > -INFINITY) best = fmaxf(best, lower(beam, top));
            });
            bound = fmaxf(bound, nth_best(best));
        }
        each_token([&](int beam, float x, int token) { return pick(make_key(x, token), beam); });
        if (finished && s.score[tid] >= bound) pick(0, -1 - tid);
        __syncthreads();
        if (s.count <= kFew || closer) break;
        closer = true;
        __syncthreads();
        if (tid == 0) s.count = 0;
    }
    const int count = s.count;
    auto write_out = [&](int place, const Candidate& c) {
        const int64_t at = static_cast<int64_t>(blockIdx.x) * n + place;
        const bool some = c.id != ~0ull;
        const int row = some ? static_cast<int>(c.id >> 24) : row0;
        const int token = some ? static_cast<int>(c.id & 0xFFFFFFu) : a.pad;
        a.out_scores[at] = some ? static_cast<float>(value64(c.score)) : -INFINITY;
        a.out_tokens[at] = token;
        a.out_parents[at] = row;
        if (a.out_finished) a.out_finished[at] = some && (s.state[row - row0] == kFinished || token == a.eos);
    };
    if (count <= kPicked) {
        // a candidate's place is the number of better ones
        for (int i = tid; i < count; i += kThreads) {
            const int beam = s.beams[i];
            s.picked[i] = beam < 0 ? of_finished(-1 - beam) : exact(beam, key_value(s.keys[i]), key_token(s.keys[i]));
        }
        __syncthreads();
        constexpr int kShare = 8;                      // threads for each
        for (int i0 = 0; i0 < max(count, n); i0 += kThreads / kShare) {
            const int i = i0 + tid / kShare;
            const Candidate c = i < count ? s.picked[i] : Candidate{0, ~0ull};
            int place = 0;
            for (int j = tid % kShare; j < count; j += kShare) place += better(s.picked[j], c);
#pragma unroll
            for (int o = 1; o < kShare; o <<= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
            if (i >= count) place = i;
            if (tid % kShare == 0 && place < n) write_out(place, c);
        }
        return;
    }
    // too many within the rounding of each other: the best of what is left, one after another
    Candidate last{~0ull, 0};
    for (int o = 0; o < n; ++o) {
        Candidate c{0, ~0ull};
        each_token([&](int beam, float x, int token) {
            const Candidate y = exact(beam, x, token);
            if (better(last, y) && better(y, c)) c = y;
            return true;
        });
        if (finished) {
            const Candidate y = of_finished(tid);
            if (better(last, y) && better(y, c)) c = y;
        }
        last = best_of_block(c);
        if (tid == 0) write_out(o, last);
    }
}

template <bool F32>
cudaError_t launch(const BeamArgs& a, ScaledSum* sums, cudaStream_t stream)
{
    const int pieces = (a.vocab + kPiece - 1) / kPiece, sms = sm_count(-1);
    const int64_t all = static_cast<int64_t>(a.lanes) * a.beams * pieces;
    const int warps = static_cast<int>(max(static_cast<int64_t>(1), min(all / sms, static_cast<int64_t>(kScanWarps))));
    const cudaError_t e = launch_pdl(beam_scan_kernel<F32>, dim3(static_cast<unsigned>((all + warps - 1) / warps)),
                                     dim3(static_cast<unsigned>(32 * warps)), 0, stream, a, pieces, sums);
    if (e != cudaSuccess) return e;
    // One block of 1,024 threads, two of 512 or four of 256 are on an SM at a time: the fastest that all lanes find room in
    // (bf16 rows of 4,096, 8 of them for 1,024 / 512 / 256 threads: 150 lanes 8.7 / 9.0 / 11.2 us, 304 lanes 14.5 / 9.3 /
    // 11.7, 400 lanes 19.7 / 14.2 / 11.9).
    const int threads = a.lanes <= sms ? 1024 : a.lanes <= 2 * sms ? 512 : 256;
    return launch_pdl(threads == 1024 ? beam_join_kernel<F32, 1024> : threads == 512 ? beam_join_kernel<F32, 512> : beam_join_kernel<F32, 256>,
                      dim3(static_cast<unsigned>(a.lanes)), dim3(static_cast<unsigned>(threads)), 0, stream, a, pieces,
                      static_cast<const ScaledSum*>(sums));
}

}  // namespace

size_t beam_select_workspace_bytes(int lanes, int beams, int vocab)
{
    return static_cast<size_t>(lanes) * beams * ((vocab + kPiece - 1) / kPiece) * sizeof(ScaledSum) + 256;
}

qg_status launch_beam_select(const BeamArgs& in, void* workspace, cudaStream_t stream)
{
    BeamArgs a = in;
    a.status = device_status_ptr();
    if (!a.status) return QG_ERR_CUDA;
    ScaledSum* sums = static_cast<ScaledSum*>(workspace);
    const cudaError_t e = a.f32 ? launch<true>(a, sums, stream) : launch<false>(a, sums, stream);
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

}  // namespace qg

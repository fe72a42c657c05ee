// tree_attention.cu -- attention of drafted tokens over the paged cache on
// warp-level MMA, and the kernel that joins a unit's parts.
//
// out = softmax(scale q K^T) V over a cache that is read once: what bounds it
// is the cache's bytes. Each warp walks its own blocks of keys with its own
// running maximum and sum (no barrier between warps until a unit ends), its
// keys and values arriving through a ring of cp.async copies in which every
// lane fetches exactly the bytes that it will feed to its MMA fragments:
//   * m16n8k16 wants, for the keys (B operand of q K^T), two pairs of values
//     along head_dim per lane and key, and sums do not care in which order
//     head_dim is walked: lane (g, c) takes 16 bytes at 16 c (+ 64 u) of key g
//     and uses them in order, q being laid out to match;
//   * for the values (B operand of P V), pairs of keys per lane and column:
//     lane (g, c) takes 16 bytes at 16 g (+ 128 p) of the keys 2c, 2c + 1,
//     2c + 8, 2c + 9, so that its columns are bytes of its own registers, and
//     pairs up two keys' bytes with byte permutes before the conversion.
// Nothing is transposed through shared memory and no lane reads another's copy
// (block scales apart). FP8 keys keep their codes' values in the MMA, their
// scale is a factor of the score's column; FP8 values too, their scale is added
// to the score (2^(s - 15) times a weight 2^x is 2^(x + s - 15)) and taken out of
// the sum of weights again.
//
// Bound: the cache's bytes at long contexts, 5.2 TB/s (77 % of the measured copy
// rate) from one context length to the next; before that about 12 us of launch,
// first loads, join of the warps and join of the parts. Measured on a GB300 (48
// query, 4 key/value heads of 128, one token per lane): 8 x 16,384 tokens in bf16
// 63 us, FP8 42, NVFP4 34; 8 x 65,536 FP8 119 us; one lane of 1,000 tokens 8 us
// on the device. Three CTAs of four warps per SM at 168 registers; two at 255
// took 3 % longer. A unit of more rows than a tile has its cache read once per
// tile: at head_dim 256, where every tile has 16 rows, trees of 7 on 12 query heads
// per key/value head read it 6 times (8 x 16,384 in bf16 301 us, one token 65).
#include <atomic>
#include <type_traits>

#include "tree_common.cuh"

namespace qg {
namespace {

constexpr int kMmaWarps = 4;
constexpr int kMmaThreads = 32 * kMmaWarps;
// Weights are 2^(s - (m - 7)), m the row's largest score at some time: f16 keeps 11
// bits down to 2^-21 of the largest. m is replaced only once a weight passes 2^15
// (< 65504). That is asked of s - (m - 7) as the weights have it: from 2^24 on,
// m - 7 is not exact, and s > m + 8 would let weights of 2^16 pass.
constexpr float kOffset = 7.f;
constexpr float kMost = 15.f;

template <int V>
using Int = std::integral_constant<int, V>;

// Sizes of a format's rows as the lanes fetch them.
template <int FMT, int D>
struct Lay {
    static constexpr int kRow = kv_row_bytes(FMT, D);
    static constexpr int kScale = kv_scale_bytes(FMT, D);
    static constexpr int kPerByteX2 = FMT == QG_KV_BF16 ? 1 : FMT == QG_KV_FP8 ? 2 : 4;  // values per 2 bytes
    static constexpr int kKB = kRow / 4 < 16 ? kRow / 4 : 16;    // bytes of a key piece
    static constexpr int kKP = kRow / 4 / kKB;                   // pieces per lane and key
    static constexpr int kKE = kKB * kPerByteX2 / 2;             // values of a key piece
    static constexpr int kVB = kRow / 8 < 16 ? kRow / 8 : 16;    // the same for values
    static constexpr int kVP = kRow / 8 / kVB;
    static constexpr int kVE = kVB * kPerByteX2 / 2;
    // keys per block (16 or 32): a block's bytes stay within 8 KB
    static constexpr int kGroups = kRow <= 128 ? 2 : 1;
    static constexpr int kKeys = 16 * kGroups;
    static constexpr int kKBytes = kKeys * kRow;
    static constexpr int kSBytes = kKeys * kScale;
    static constexpr int kStage = 2 * (kKBytes + kSBytes);
};

template <int FMT, int D, int RT>
struct MmaPlan {
    using L = Lay<FMT, D>;
    static constexpr int kRows = 16 * RT;
    static constexpr int kStep = kMmaWarps * L::kKeys;
    static constexpr int kQ = RT * D * 32;                       // bytes of q fragments
    static constexpr int kHead = kQ + kRows * 16;                // + masks, exponents
    // three CTAs per SM where the accumulators leave the registers for it, else
    // two, one where two blocks per warp do not fit beside each other
    static constexpr int kCtas = RT == 1 && D <= 128 ? 3 : kHead + 2 * kMmaWarps * L::kStage <= 112 * 1024 ? 2 : 1;
    static constexpr int kBudget = (kCtas == 3 ? 74 : kCtas == 2 ? 112 : 224) * 1024 - kHead;
    static constexpr int kFit = kBudget / (kMmaWarps * L::kStage);
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kRing = kMmaWarps * kStages * L::kStage;
    static constexpr int kJoin = kMmaWarps * kRows * (D + 4) * 4 + kMmaWarps * kRows * 8;
    static constexpr int kBody = kRing > kJoin ? kRing : kJoin;
    static constexpr int kSmem = kHead + kBody;
    static_assert(kStages >= 2, "ring too short");
    static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "too much shared memory");
};

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool on)
{
    const int n = on ? BYTES : 0;                                // 0: zeros, nothing is read
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n)
                     : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// `BYTES` of this lane's copy as words.
template <int BYTES>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[BYTES / 4])
{
    if constexpr (BYTES == 16) {
        const uint4 v = lds128(addr);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else if constexpr (BYTES == 8) {
        const uint2 v = lds64(addr);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = lds32(addr);
    }
}

template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    uint32_t r;
    if constexpr (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Values of a key piece: the pairs that k-step w of the piece feeds to the MMA.
template <int FMT, int WORDS>
__device__ __forceinline__ void key_pair(const uint32_t (&r)[WORDS], int w, const uint32_t (&sc)[2], uint32_t& b0,
                                         uint32_t& b1)
{
    if constexpr (FMT == QG_KV_BF16) {
        b0 = r[2 * w];
        b1 = r[2 * w + 1];
    } else if constexpr (FMT == QG_KV_FP8) {
        e4m3x4_to_f16x2x2(r[w], b0, b1);
    } else {
        const uint32_t x = r[w / 2] >> (16 * (w & 1));
        b0 = hmul2(e2m1x2_to_f16x2(x & 0xFFu), sc[w / 4]);
        b1 = hmul2(e2m1x2_to_f16x2((x >> 8) & 0xFFu), sc[w / 4]);
    }
}

// Values of two keys' pieces side by side: word i holds elements of both; out
// gets one f16x2 / bf16x2 (key 0 low, key 1 high) per element, in order. (FP8:
// the codes' own values, their scales are in the weights.)
template <int FMT>
__device__ __forceinline__ void value_pairs(uint32_t w0, uint32_t w1, uint32_t sc,
                                            uint32_t (&out)[FMT == QG_KV_BF16 ? 2 : FMT == QG_KV_FP8 ? 4 : 8])
{
    if constexpr (FMT == QG_KV_BF16) {
        out[0] = __byte_perm(w0, w1, 0x5410);
        out[1] = __byte_perm(w0, w1, 0x7632);
    } else if constexpr (FMT == QG_KV_FP8) {
        e4m3x4_to_f16x2x2(__byte_perm(w0, w1, 0x5140), out[0], out[1]);
        e4m3x4_to_f16x2x2(__byte_perm(w0, w1, 0x7362), out[2], out[3]);
    } else {
        const uint32_t even = (w0 & 0x0F0F0F0Fu) | ((w1 & 0x0F0F0F0Fu) << 4);
        const uint32_t odd = ((w0 >> 4) & 0x0F0F0F0Fu) | (w1 & 0xF0F0F0F0u);
        uint32_t e[4], o[4];
        e2m1x8_to_f16x2x4(even, e);
        e2m1x8_to_f16x2x4(odd, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            out[2 * i] = hmul2(e[i], sc);
            out[2 * i + 1] = hmul2(o[i], sc);
        }
    }
}

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts8(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "h"(static_cast<uint16_t>(v)) : "memory");
}

// The values of a block with drafts, or with places behind the last key, made
// harmless where it lies: from key `context` on, what is not finite becomes zero
// (0 times it would reach rows that do not see the draft), and so do scales
// behind the last key, whose codes are zeros already. The keys before it are the
// context's: every row sees them, and what is not finite there reaches them all.
// True if a draft's value was not finite.
template <int FMT, int D>
__device__ __noinline__ bool clean_values(uint32_t values, uint32_t scales, int context, int keys, int lane)
{
    using L = Lay<FMT, D>;
    bool odd = false;
    if constexpr (FMT == QG_KV_NVFP4) {
        if (lane < L::kKeys && lane >= min(context, keys))
            for (int i = 0; i < L::kScale; ++i) {
                const uint32_t at = scales + lane * L::kScale + i;
                const bool nan = (lds8(at) & 0x7Fu) == 0x7Fu;
                odd = odd || (nan && lane < keys);
                if (nan || lane >= keys) sts8(at, 0);
            }
    } else {
        for (int i = 0; i < L::kKBytes / 128; ++i) {          // this lane's words of its own pieces
            const int piece = i / (L::kVB / 4), y = piece / L::kVP;
            const int key = 16 * (y >> 2) + 2 * (lane & 3) + (y & 1) + 8 * (y >> 1 & 1);
            const uint32_t at = values + piece * (32 * L::kVB) + lane * L::kVB + i % (L::kVB / 4) * 4;
            const uint32_t w = lds32(at);
            const uint32_t bad = FMT == QG_KV_BF16 ? __vcmpeq2(w & 0x7F807F80u, 0x7F807F80u)
                                                   : __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            const uint32_t e = key < context ? 0u : bad;      // (no branch before the load: the loads overlap)
            odd = odd || e;
            if (e) sts32(at, w & ~e);
        }
    }
    __syncwarp();
    return __any_sync(0xffffffffu, odd);
}

// One warp's side of a unit: where its keys stand and what its ring holds.
struct Walk {
    int b, head;
    int first, end;              // the segment's keys
    int len, keys;               // context and all keys of the sequence
    int n;                       // this warp's blocks
};

// Adds to four outputs of a row the drafts' values that are not finite and were
// left out of the products, for the drafts that the row sees: whatever their
// weights, they make it infinite or NaN. Rare.
template <int D>
__device__ __noinline__ float4 odd_values(const KvArgs& a, const Walk& k, uint64_t mask, int d, float4 v)
{
    float* o = reinterpret_cast<float*>(&v);
    for (int p = max(k.first, k.len); p < k.end; ++p) {
        if (!((mask >> (p - k.len)) & 1ull)) continue;
        const int page = kv_page(a, k.b, p);
        if (page < 0) continue;
        const int64_t row = kv_row(a, page, k.head, p);
        for (int i = 0; i < 4; ++i) {
            const float x = kv_value(a, 1, row, d + i);
            if (!(fabsf(x) < INFINITY)) o[i] += x;
        }
    }
    return v;
}

// The copies of 16 keys of which only `left` are in the sequence: zeros behind
// them (nothing is read there).
template <int FMT, int D>
__device__ __noinline__ void copy_partly(uint32_t kd, uint32_t vd, const uint8_t* kl, const uint8_t* vl, int left, int g,
                                         int c)
{
    using L = Lay<FMT, D>;
    for (int j = 0; j < 2; ++j)
        for (int x = 0; x < L::kKP; ++x)
            cp_async<L::kKB>(kd + (j * L::kKP + x) * 32 * L::kKB, kl + 8 * j * L::kRow + x * 4 * L::kKB,
                             8 * j + g < left);
    for (int y = 0; y < 4; ++y)
        for (int x = 0; x < L::kVP; ++x) {
            const int key = (y & 1) + 8 * (y >> 1);
            cp_async<L::kVB>(vd + (y * L::kVP + x) * 32 * L::kVB, vl + key * L::kRow + x * 8 * L::kVB,
                             2 * c + key < left);
        }
}

template <int FMT, int D, int RT>
__global__ void __launch_bounds__(kMmaThreads, MmaPlan<FMT, D, RT>::kCtas) tree_mma_kernel(const __grid_constant__ TreeArgs t)
{
    using L = Lay<FMT, D>;
    using P = MmaPlan<FMT, D, RT>;
    constexpr bool kBf16 = FMT == QG_KV_BF16;
    constexpr int kNT = 2 * L::kGroups;              // key tiles of 8 per block
    constexpr int kOT = D / 8;                       // output tiles of 8 columns
    constexpr int kSteps = L::kKE / 4;               // k-steps per key piece
    extern __shared__ __align__(128) uint8_t smem[];
    uint4* q_frag = reinterpret_cast<uint4*>(smem);
    uint64_t* row_mask = reinterpret_cast<uint64_t*>(smem + P::kQ);
    int* row_exp = reinterpret_cast<int*>(smem + P::kQ + P::kRows * 8);
    uint8_t* body = smem + P::kHead;
    const KvArgs& a = t.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;

    // Predecessors are complete after the wait, so the joining kernel, which
    // starts early, may read the batch as soon as it is launched.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    TreeScan scan;
    scan.run(t);
    const int64_t total = scan.total;
    const int64_t cta_first = tree_first(total, t.grid, blockIdx.x);
    const int64_t cta_end = tree_first(total, t.grid, blockIdx.x + 1);
    if (cta_first >= cta_end) return;
    int64_t base;                                    // first step of sequence b
    KvSeq seq;
    int b = scan.find(t, cta_first, seq, base);
    TreeSeq u = tree_seq_of(t, seq);

    const uint32_t ring = smem_u32(body) + warp * (P::kStages * L::kStage);
    int64_t at = cta_first;
    while (at < cta_end) {
        while (at >= base + tree_steps(t, u)) {
            base += tree_steps(t, u);
            u = tree_seq(t, ++b);
        }
        const int unit = static_cast<int>((at - base) / u.steps);
        const int s0 = static_cast<int>((at - base) % u.steps);
        const int s1 = static_cast<int>(min(static_cast<int64_t>(u.steps), s0 + (cta_end - at)));
        const int head = unit / u.tiles, tile = unit % u.tiles;
        Walk k;
        k.b = b;
        k.head = head;
        k.first = s0 * P::kStep;
        k.end = min(u.keys, s1 * P::kStep);
        k.len = u.s.len;
        k.keys = u.keys;
        const int blocks = (k.end - k.first + L::kKeys - 1) / L::kKeys;
        k.n = blocks > warp ? (blocks - warp - 1) / kMmaWarps + 1 : 0;
        const int row0 = tile * P::kRows;
        const int n_rows = min(P::kRows, u.s.rows * t.group - row0);

        // ---- the ring
        uint32_t bad = 0;                            // per ring place: groups whose page lies outside the cache
        int entry[L::kGroups], off[L::kGroups];      // the next block's page table entries, places in their pages
        const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;
        auto look_up = [&](int i) {
#pragma unroll
            for (int s = 0; s < L::kGroups; ++s) {
                const int p = k.first + (warp + i * kMmaWarps) * L::kKeys + 16 * s;
                const int x = kv_page_index(a, p);
                off[s] = p - x * a.page_size;
                entry[s] = p < k.end ? table[x] : 0;
            }
        };
        const uint32_t page_rows = a.heads * a.page_size;
        const uint32_t head_rows = head * a.page_size;
        const uint8_t* k_lane = a.codes[0] + g * L::kRow + c * L::kKB;
        const uint8_t* v_lane = a.codes[1] + 2 * c * L::kRow + g * L::kVB;
        auto issue = [&](int i) {
            const int place = i % P::kStages;
            const uint32_t dst = ring + place * L::kStage;
            bad &= ~(3u << (2 * place));
            if (i < k.n) {
#pragma unroll
                for (int s = 0; s < L::kGroups; ++s) {
                    const int p = k.first + (warp + i * kMmaWarps) * L::kKeys + 16 * s;
                    int left = k.end - p;                        // keys of this group
                    const bool in = static_cast<uint32_t>(entry[s]) < static_cast<uint32_t>(a.num_pages);
                    if (!in) {
                        set_device_status(a.status, QG_ERR_INVALID_ARG);
                        bad |= 1u << (2 * place + s);
                        left = 0;
                    }
                    const int64_t row = static_cast<int64_t>(in ? entry[s] : 0) * page_rows + (head_rows + off[s]);
                    const uint8_t* kl = k_lane + row * L::kRow;
                    const uint8_t* vl = v_lane + row * L::kRow;
                    const uint32_t kd = dst + 2 * s * L::kKP * 32 * L::kKB + lane * L::kKB;
                    const uint32_t vd = dst + L::kKBytes + 4 * s * L::kVP * 32 * L::kVB + lane * L::kVB;
                    if (left >= 16) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int x = 0; x < L::kKP; ++x)
                                cp_async<L::kKB>(kd + (j * L::kKP + x) * 32 * L::kKB,
                                                 kl + 8 * j * L::kRow + x * 4 * L::kKB);
#pragma unroll
                        for (int y = 0; y < 4; ++y)
#pragma unroll
                            for (int x = 0; x < L::kVP; ++x)
                                cp_async<L::kVB>(vd + (y * L::kVP + x) * 32 * L::kVB,
                                                 vl + ((y & 1) + 8 * (y >> 1)) * L::kRow + x * 8 * L::kVB);
                    } else {
                        copy_partly<FMT, D>(kd, vd, kl, vl, left, g, c);
                    }
                    if constexpr (L::kScale > 0) {
                        // 16 keys' scales are kScale pieces of 16 bytes
                        const uint32_t sd = dst + 2 * L::kKBytes + 16 * s * L::kScale;
                        if (lane < 2 * L::kScale) {
                            const int kv = lane >= L::kScale, x = lane - kv * L::kScale;
                            cp_async<16>(sd + kv * L::kSBytes + x * 16, a.scales[kv] + row * L::kScale + x * 16,
                                         left > 0);
                        }
                    }
                }
            }
            cp_commit();
        };
        look_up(0);
#pragma unroll
        for (int i = 0; i < P::kStages - 1; ++i) {
            issue(i);
            look_up(i + 1);
        }

        // ---- q as MMA fragments, scaled to f16's range by a power of two per row
        for (int r = warp; r < P::kRows; r += kMmaWarps) {
            const int tok = (row0 + r) / t.group, qh = head * t.group + (row0 + r) % t.group;
            constexpr int kPer = D / 32 < 4 ? 4 : D / 32;      // values per lane
            uint32_t w2[kPer / 2] = {};
            const bool on = r < n_rows && lane * kPer < D;
            if (on) {
                const uint16_t* src = t.q + (u.s.row0 + tok) * t.q_stride + qh * D + lane * kPer;
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i) w2[i] = reinterpret_cast<const uint32_t*>(src)[i];
            }
            int pe = 0;
            if constexpr (!kBf16) {
                uint32_t mag = 0;
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i) {
                    const uint32_t m = w2[i] & 0x7FFF7FFFu;
                    mag = max(mag, max(m & 0xFFFFu, m >> 16));
                }
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, off));
                pe = mag < 0x7F80u ? prescale_exponent(mag) : 0;
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i)
                    w2[i] = pack_f16x2(ldexp_exact(__uint_as_float(w2[i] << 16), pe),
                                       ldexp_exact(__uint_as_float(w2[i] & 0xFFFF0000u), pe));
            }
            if (lane == 0) {
                row_exp[r] = pe;
                row_mask[r] = r >= n_rows ? 0 : t.mask ? t.mask[u.s.row0 + tok] : (2ull << tok) - 1;
            }
            if (lane * kPer < D) {
#pragma unroll
                for (int i = 0; i < kPer / 4; ++i) {
                    const int d = lane * kPer + 4 * i;         // four values: one lane's share of one k-step
                    const int piece = d / (4 * L::kKE), in = d % (4 * L::kKE);
                    const int kk = piece * kSteps + in % L::kKE / 4;
                    const int to = (r % 8) * 4 + in / L::kKE;
                    uint32_t* f = reinterpret_cast<uint32_t*>(q_frag + (r / 16 * (D / 16) + kk) * 32 + to);
                    f[(r % 16) / 8] = w2[2 * i];
                    f[(r % 16) / 8 + 2] = w2[2 * i + 1];
                }
            }
        }
        __syncthreads();

        float o[RT][kOT][4], m[RT][2], l[RT][2], rowf[RT][2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
            for (int j = 0; j < kOT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[rt][j][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[rt][e] = -INFINITY;
                l[rt][e] = 0.f;
                rowf[rt][e] = ldexp_exact(t.scale * kLog2e * a.g[0], -row_exp[16 * rt + 8 * e + g]);
            }
        }

        bool odd = false;                            // a draft's value was not finite
#pragma unroll 1
        for (int i = 0; i < k.n; ++i) {
            cp_wait<P::kStages - 2>();
            __syncwarp();
            issue(i + P::kStages - 1);
            look_up(i + P::kStages);
            const int place = i % P::kStages;
            const uint32_t src = ring + place * L::kStage;
            const uint32_t k_sc = src + 2 * L::kKBytes, v_sc = k_sc + L::kSBytes;
            const int p0 = k.first + (warp + i * kMmaWarps) * L::kKeys;
            const uint32_t gone = (bad >> (2 * place)) & 3u;
            const bool special = p0 + L::kKeys > k.len || gone;
            if (special) odd = clean_values<FMT, D>(src + L::kKBytes, v_sc, k.len - p0, k.end - p0, lane) || odd;

            // ---- scores
            float s[RT][kNT][4];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int j = 0; j < kNT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[rt][j][e] = 0.f;
#pragma unroll
            for (int x = 0; x < L::kKP; ++x) {
                uint32_t raw[kNT][L::kKB / 4], sc[kNT][2];
#pragma unroll
                for (int j = 0; j < kNT; ++j) {
                    lds_words<L::kKB>(src + ((j * L::kKP + x) * 32 + lane) * L::kKB, raw[j]);
                    if constexpr (FMT == QG_KV_NVFP4) {
                        // the piece's one or two blocks of 16
                        const uint32_t at8 = k_sc + (8 * j + g) * L::kScale + (x * 4 + c) * L::kKE / 16;
                        const uint32_t two = L::kKE == 32 ? lds16(at8) : lds8(at8);
                        const uint32_t f = e4m3x2_to_f16x2(two);
                        sc[j][0] = __byte_perm(f, f, 0x1010);
                        sc[j][1] = __byte_perm(f, f, 0x3232);
                    }
                }
#pragma unroll
                for (int w4 = 0; w4 < kSteps; ++w4) {
                    uint4 af[RT];
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        af[rt] = q_frag[(rt * (D / 16) + x * kSteps + w4) * 32 + lane];
#pragma unroll
                    for (int j = 0; j < kNT; ++j) {
                        uint32_t b0, b1;
                        key_pair<FMT>(raw[j], w4, sc[j], b0, b1);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) mma_16816<kBf16>(s[rt][j], af[rt], b0, b1);
                    }
                }
            }

            // ---- base-2 scores, masks, running maxima
            float inv[kNT][2];                       // FP8: 2^-(exponent of the value's scale) ...
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
                float cf[2], add[2];
                if constexpr (FMT == QG_KV_FP8) {
                    const uint32_t two = lds16(k_sc + 8 * j + 2 * c), vs = lds16(v_sc + 8 * j + 2 * c) & 0x1F1Fu;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        cf[e] = __uint_as_float((((two >> (8 * e)) & 0xFFu) + 112u) << 23);
                        const int b = (vs >> (8 * e)) & 0xFFu;
                        add[e] = static_cast<float>(b - 15);
                        inv[j][e] = __int_as_float((142 - b) << 23);
                    }
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // ... which the weights take in, as an addition to the score
                        if constexpr (FMT == QG_KV_FP8)
                            s[rt][j][e] = fmaf(s[rt][j][e] * cf[e & 1], rowf[rt][e >> 1], add[e & 1]);
                        else
                            s[rt][j][e] = __fmul_rn(s[rt][j][e], rowf[rt][e >> 1]);   // the score that m is of too
                    }
            }
            if (special) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const uint64_t mk[2] = {row_mask[16 * rt + g], row_mask[16 * rt + 8 + g]};
#pragma unroll
                    for (int j = 0; j < kNT; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int p = p0 + 8 * j + 2 * c + (e & 1);
                            const bool seen = p < k.end && !((gone >> (j >> 1)) & 1u) &&
                                              (p < k.len || ((mk[e >> 1] >> (p - k.len)) & 1ull));
                            if (!seen) s[rt][j][e] = -INFINITY;
                        }
                }
            }
            bool raise = false;
            float top[RT][2];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = -INFINITY;
#pragma unroll
                    for (int j = 0; j < kNT; ++j) x = fmaxf(x, fmaxf(s[rt][j][2 * e], s[rt][j][2 * e + 1]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    top[rt][e] = x;
                    raise = raise || x - (m[rt][e] - kOffset) > kMost;
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mn = fmaxf(m[rt][e], top[rt][e]);
                        const float f = mn == -INFINITY ? 1.f : ex2(m[rt][e] - mn);
                        m[rt][e] = mn;
                        l[rt][e] *= f;
#pragma unroll
                        for (int j = 0; j < kOT; ++j) {
                            o[rt][j][2 * e] *= f;
                            o[rt][j][2 * e + 1] *= f;
                        }
                    }
            }
            // ---- weights
            uint4 pf[RT][L::kGroups];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const float z0 = (m[rt][0] == -INFINITY ? 0.f : m[rt][0]) - kOffset;
                const float z1 = (m[rt][1] == -INFINITY ? 0.f : m[rt][1]) - kOffset;
#pragma unroll
                for (int j = 0; j < kNT; ++j) {
                    s[rt][j][0] = ex2(s[rt][j][0] - z0);
                    s[rt][j][1] = ex2(s[rt][j][1] - z0);
                    s[rt][j][2] = ex2(s[rt][j][2] - z1);
                    s[rt][j][3] = ex2(s[rt][j][3] - z1);
                    if constexpr (FMT == QG_KV_FP8) {
                        l[rt][0] = fmaf(s[rt][j][0], inv[j][0], fmaf(s[rt][j][1], inv[j][1], l[rt][0]));
                        l[rt][1] = fmaf(s[rt][j][2], inv[j][0], fmaf(s[rt][j][3], inv[j][1], l[rt][1]));
                    } else {
                        l[rt][0] += s[rt][j][0] + s[rt][j][1];
                        l[rt][1] += s[rt][j][2] + s[rt][j][3];
                    }
                }
#pragma unroll
                for (int x = 0; x < L::kGroups; ++x) {
                    pf[rt][x].x = pack16<kBf16>(s[rt][2 * x][0], s[rt][2 * x][1]);
                    pf[rt][x].y = pack16<kBf16>(s[rt][2 * x][2], s[rt][2 * x][3]);
                    pf[rt][x].z = pack16<kBf16>(s[rt][2 * x + 1][0], s[rt][2 * x + 1][1]);
                    pf[rt][x].w = pack16<kBf16>(s[rt][2 * x + 1][2], s[rt][2 * x + 1][3]);
                }
            }

            // ---- values
#pragma unroll
            for (int x = 0; x < L::kGroups; ++x) {
#pragma unroll
                for (int y = 0; y < L::kVP; ++y) {
                    uint32_t raw[4][L::kVB / 4];
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        lds_words<L::kVB>(src + L::kKBytes + (((4 * x + z) * L::kVP + y) * 32 + lane) * L::kVB,
                                          raw[z]);
                    constexpr int kPer = kBf16 ? 2 : FMT == QG_KV_FP8 ? 4 : 8;   // values of a word
                    uint32_t sc[2] = {0, 0};         // NVFP4: scales of keys (2c, 2c + 1) and (2c + 8, 2c + 9)
#pragma unroll
                    for (int i4 = 0; i4 < L::kVB / 4; ++i4) {
                        if constexpr (FMT == QG_KV_NVFP4) {
                            if (i4 % 2 == 0) {       // a block of 16 is two words
                                const int blk = (y * 8 * L::kVE + g * L::kVE + i4 * 8) / 16;
#pragma unroll
                                for (int z = 0; z < 2; ++z) {
                                    const uint32_t at8 = v_sc + (16 * x + 8 * z + 2 * c) * L::kScale + blk;
                                    sc[z] = e4m3x2_to_f16x2(lds8(at8) | lds8(at8 + L::kScale) << 8);
                                }
                            }
                        }
                        uint32_t b0[kPer], b1[kPer];
                        value_pairs<FMT>(raw[0][i4], raw[1][i4], sc[0], b0);
                        value_pairs<FMT>(raw[2][i4], raw[3][i4], sc[1], b1);
#pragma unroll
                        for (int e = 0; e < kPer; ++e)
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt)
                                mma_16816<kBf16>(o[rt][y * L::kVE + i4 * kPer + e], pf[rt][x], b0[e], b1[e]);
                    }
                }
            }
        }

        // ---- join the warps and write
        cp_wait<0>();
        odd = __syncthreads_or(odd);
        float* jo = reinterpret_cast<float*>(body);
        float2* jm = reinterpret_cast<float2*>(body + kMmaWarps * P::kRows * (D + 4) * 4);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[rt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                const int r = 16 * rt + 8 * e + g;
                if (c == 0) jm[warp * P::kRows + r] = make_float2(m[rt][e] - kOffset, x);
                float* dst = jo + (warp * P::kRows + r) * (D + 4);
#pragma unroll
                for (int j = 0; j < kOT; j += 4)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int d = j / L::kVE * (8 * L::kVE) + (2 * c + n) * L::kVE + j % L::kVE;
                        *reinterpret_cast<float4*>(dst + d) =
                            make_float4(o[rt][j][2 * e + n], o[rt][j + 1][2 * e + n], o[rt][j + 2][2 * e + n],
                                        o[rt][j + 3][2 * e + n]);
                    }
            }
        __syncthreads();
        const bool whole = s0 == 0 && s1 == u.steps;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (s0 == 0);
        for (int x = threadIdx.x; x < n_rows * (D / 4); x += kMmaThreads) {
            const int r = x / (D / 4), d = x % (D / 4) * 4;
            float mt = -INFINITY;
#pragma unroll
            for (int y = 0; y < kMmaWarps; ++y) mt = fmaxf(mt, jm[y * P::kRows + r].x);
            float lt = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int y = 0; y < kMmaWarps; ++y) {
                const float2 ml = jm[y * P::kRows + r];
                const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mt);
                const float4 z = *reinterpret_cast<const float4*>(jo + (y * P::kRows + r) * (D + 4) + d);
                lt += f * ml.y;
                v.x += f * z.x;
                v.y += f * z.y;
                v.z += f * z.z;
                v.w += f * z.w;
            }
            if (odd) v = odd_values<D>(a, k, row_mask[r], d, v);
            if (whole) {
                const int tok = u.s.row0 + (row0 + r) / t.group;
                const int64_t h = static_cast<int64_t>(tok) * t.q_heads + head * t.group + (row0 + r) % t.group;
                const float f = tree_inverse(lt) * a.g[1];
                uint2 y;
                y.x = pack16<true>(v.x * f, v.y * f);
                y.y = pack16<true>(v.z * f, v.w * f);
                *reinterpret_cast<uint2*>(t.out + h * D + d) = y;
                if (t.lse && d == 0) t.lse[h] = tree_lse(mt, lt);
            } else {
                *reinterpret_cast<float4*>(t.part_o + (slot * P::kRows + r) * D + d) = v;
                if (d == 0) t.part_ml[slot * P::kRows + r] = make_float2(mt, lt);
            }
        }
        __syncthreads();
        at += s1 - s0;
    }
}

// ------------------------------------------------------------------ join
// The rows (token, query head) whose unit was read in several parts. Bound by
// two chained loads (the batch's entries, before the wait; then the parts with
// their maxima and sums). W warps share a row, taking every W-th part: four for
// a decode step, whose few rows have many parts, one where there are rows enough
// to fill the GPU (16,384 rows of four parts: 36 us with four warps each).
constexpr int kJoinWarps = 4;

template <int D, int W>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const __grid_constant__ TreeArgs t)
{
    constexpr int kPer = D / 32;
    constexpr int kAhead = 4;                        // parts on their way per warp
    __shared__ float part[kJoinWarps][D];
    __shared__ float2 part_ml[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row_at = static_cast<int64_t>(blockIdx.x) * (kJoinWarps / W) + warp / W;
    const int i = static_cast<int>(row_at / t.q_heads), h = static_cast<int>(row_at % t.q_heads);
    TreeScan scan;
    scan.run(t);
    int64_t base, c0 = 0, c1 = 0;
    KvSeq seq;
    int r = 0;
    if (scan.total > 0 && scan.find_row(t, i, seq, base) >= 0) {
        const TreeSeq u = tree_seq_of(t, seq);
        const int row = (i - seq.row0) * t.group + h % t.group;
        const int64_t first = base + static_cast<int64_t>(h / t.group * u.tiles + row / t.rows) * u.steps;
        c0 = tree_owner(scan.total, t.grid, first);
        c1 = tree_owner(scan.total, t.grid, first + u.steps - 1);
        r = row % t.rows;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (c0 == c1) return;                            // written whole, or nobody's row
    float m = -INFINITY, l = 0.f, acc[kPer] = {};
    for (int64_t y0 = c0 + warp % W; y0 <= c1; y0 += kAhead * W) {
        float2 ml[kAhead];
        float v[kAhead][kPer];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int64_t y = y0 + x * W;
            ml[x] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int z = 0; z < kPer; ++z) v[x][z] = 0.f;
            if (y <= c1) {
                const int64_t at = (2 * y + (y == c0)) * t.rows + r;   // a unit's first part is its CTA's last
                ml[x] = t.part_ml[at];
                const float* src = t.part_o + at * D + lane * kPer;
                if constexpr (kPer == 2) {
                    const float2 w = *reinterpret_cast<const float2*>(src);
                    v[x][0] = w.x;
                    v[x][1] = w.y;
                } else {
#pragma unroll
                    for (int z = 0; z < kPer; z += 4) {
                        const float4 w = *reinterpret_cast<const float4*>(src + z);
                        v[x][z] = w.x;
                        v[x][z + 1] = w.y;
                        v[x][z + 2] = w.z;
                        v[x][z + 3] = w.w;
                    }
                }
            }
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            // a part whose row saw nothing (not one whose scores are all NaN: they raise no maximum, and its NaN
            // sums make the row's NaN)
            if (ml[x].x == -INFINITY && ml[x].y == 0.f) continue;
            const float mn = fmaxf(m, ml[x].x), f = ex2(m - mn), g = ex2(ml[x].x - mn);
            m = mn;
            l = l * f + ml[x].y * g;
#pragma unroll
            for (int z = 0; z < kPer; ++z) acc[z] = acc[z] * f + v[x][z] * g;
        }
    }
    const int64_t to = static_cast<int64_t>(i) * t.q_heads + h;
    if constexpr (W == 1) {
        const float scale = tree_inverse(l) * t.a.g[1];
        uint32_t* out = reinterpret_cast<uint32_t*>(t.out + to * D) + lane * (kPer / 2);
#pragma unroll
        for (int z = 0; z < kPer / 2; ++z) out[z] = pack16<true>(acc[2 * z] * scale, acc[2 * z + 1] * scale);
        if (t.lse && lane == 0) t.lse[to] = tree_lse(m, l);
    } else {
#pragma unroll
        for (int z = 0; z < kPer; ++z) part[warp][lane * kPer + z] = acc[z];
        if (lane == 0) part_ml[warp] = make_float2(m, l);
        __syncthreads();
        m = -INFINITY;
        for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, part_ml[w].x);
        l = 0.f;
        float f[kJoinWarps];
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            f[w] = part_ml[w].x == -INFINITY ? 0.f : ex2(part_ml[w].x - m);
            l += f[w] * part_ml[w].y;
        }
        const float scale = tree_inverse(l) * t.a.g[1];
        for (int d = 2 * threadIdx.x; d < D; d += 64 * kJoinWarps) {
            float x0 = 0.f, x1 = 0.f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) {
                // with a factor of 0 too: a warp without parts holds zeros, and sums that are not finite arrive
                x0 += f[w] * part[w][d];
                x1 += f[w] * part[w][d + 1];
            }
            *reinterpret_cast<uint32_t*>(t.out + to * D + d) = pack16<true>(x0 * scale, x1 * scale);
        }
        if (t.lse && threadIdx.x == 0) t.lse[to] = tree_lse(m, l);
    }
}

// ------------------------------------------------------------------ plans
template <int FMT, int D, int RT>
cudaError_t run_mma(TreeArgs t, cudaStream_t stream)
{
    using P = MmaPlan<FMT, D, RT>;
    t.step = P::kStep;
    t.grid = P::kCtas * sm_count(-1);
    auto kern = tree_mma_kernel<FMT, D, RT>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, P::kSmem, done);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(static_cast<unsigned>(t.grid)), dim3(kMmaThreads), P::kSmem, stream, t);
    if (e != cudaSuccess) return e;
    return launch_tree_join(t, stream);
}

template <int FMT, int D>
cudaError_t run_dim(const TreeArgs& t, cudaStream_t stream)
{
    if constexpr (D <= 128)
        if (t.rows == 32) return run_mma<FMT, D, 2>(t, stream);
    return run_mma<FMT, D, 1>(t, stream);
}

template <int FMT>
cudaError_t run_format(const TreeArgs& t, cudaStream_t stream)
{
    if (t.a.dim == 64) return run_dim<FMT, 64>(t, stream);
    if (t.a.dim == 128) return run_dim<FMT, 128>(t, stream);
    return run_dim<FMT, 256>(t, stream);
}

// Rows per unit R, which also says which kernel runs, and the workspace's two
// parts, for the most CTAs (slots: two per CTA) that a format's kernel takes.
// Up to 16 rows one row tile of the warp-MMA kernel, up to 32 two; more go to
// the tensor-core kernel, in one or two tiles of 128, but for head_dim 256: that
// kernel runs two streams, whose accumulators (256 columns each) leave no tensor
// memory for scores; it has no form with one. Measured at 24 rows, 8 lanes of 2,048 /
// 16,384 / 65,536 tokens, warp-MMA against tensor-core kernel (us): FP8 19 / 57 /
// 162 against 28 / 73 / 213, NVFP4 18 / 49 / 137 against 28 / 68 / 185, bf16 21 / 68 /
// 217 against 29 / 67 / 178. So long bf16 contexts lose up to 22 % by the rule: the
// lengths are device data, and max_pages * page_size, which bounds them, may lie far
// above them. At 84 rows (8 x 16,384, NVFP4) three passes of 32 took 107 us, the
// tensor-core kernel takes 74.
struct TreePlan {
    int rows;
    size_t o_bytes, ml_bytes;
};

TreePlan plan_tree(int head_dim, int group, int max_tree)
{
    const int rows = group * max_tree;
    TreePlan p;
    p.rows = rows <= 16 || head_dim == 256 ? 16 : rows <= 32 ? 32 : rows <= 128 ? 128 : 256;
    const size_t ctas = (p.rows == 256 ? 1 : p.rows == 16 ? 3 : 2) * static_cast<size_t>(sm_count(-1));
    const size_t rows_held = 2 * ctas * p.rows;
    p.o_bytes = rows_held * head_dim * sizeof(float);
    p.ml_bytes = rows_held * sizeof(float2);
    return p;
}

}  // namespace

cudaError_t launch_tree_join(const TreeArgs& t, cudaStream_t stream)
{
    const int64_t rows = static_cast<int64_t>(t.a.n_tokens) * t.q_heads;
    const bool many = rows >= 16LL * sm_count(-1);
    const dim3 grid(static_cast<unsigned>(many ? (rows + kJoinWarps - 1) / kJoinWarps : rows)), block(32 * kJoinWarps);
    auto run = [&](auto d) {
        constexpr int D = decltype(d)::value;
        return launch_pdl(many ? tree_join_kernel<D, 1> : tree_join_kernel<D, kJoinWarps>, grid, block, 0, stream, t);
    };
    return t.a.dim == 64 ? run(Int<64>{}) : t.a.dim == 128 ? run(Int<128>{}) : run(Int<256>{});
}

// A TMA coordinate has 31 bits, and the tensor-core kernel copies bf16 rows by one
// that counts all the cache's rows (2^31 of them are 256 GB or more).
bool tree_attention_serves(const KvArgs& a, int group, int max_tree)
{
    const bool tc = group * max_tree > 32 && a.dim != 256;
    return !tc || a.fmt != QG_KV_BF16 || static_cast<int64_t>(a.num_pages) * a.heads * a.page_size <= 0x7FFFFFFF;
}

size_t tree_attention_workspace_bytes(int head_dim, int group, int max_tree)
{
    const TreePlan p = plan_tree(head_dim, group, max_tree);
    return p.o_bytes + p.ml_bytes;
}

qg_status launch_tree_attention(const KvArgs& in, const uint16_t* q, int64_t q_stride, int q_heads, int max_tree,
                                const uint64_t* mask, float scale, uint16_t* out, float* lse, void* workspace,
                                cudaStream_t stream)
{
    TreeArgs t{};
    t.a = in;
    t.a.status = device_status_ptr();
    if (!t.a.status) return QG_ERR_CUDA;
    t.q = q;
    t.q_stride = q_stride;
    t.q_heads = q_heads;
    t.group = q_heads / in.heads;
    t.max_tree = max_tree;
    t.mask = mask;
    t.scale = scale;
    t.out = out;
    t.lse = lse;
    const TreePlan p = plan_tree(in.dim, t.group, max_tree);
    t.rows = p.rows;
    t.part_o = static_cast<float*>(workspace);
    t.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.o_bytes);
    const DebugState dbg = debug_state();
    t.wait_ns = dbg.wait_ns;
    t.starve = dbg.starve;
    const cudaError_t e = t.rows >= 128           ? launch_tree_tc(t, stream)
                          : in.fmt == QG_KV_BF16  ? run_format<QG_KV_BF16>(t, stream)
                          : in.fmt == QG_KV_FP8 ? run_format<QG_KV_FP8>(t, stream)
                                                : run_format<QG_KV_NVFP4>(t, stream);
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

}  // namespace qg

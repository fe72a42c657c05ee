// tree_tc.cu -- attention of drafted tokens over the paged cache on the
// 5th-generation tensor cores, for units of many query rows.
//
// With R query rows per key/value head, a cached value of b bytes takes
// 2 R / b multiplications: at 6.8 TB/s a tree of 8 tokens with 12 query heads
// per head already asks for 650 (bf16) to 2,300 TFLOP/s (NVFP4). So the keys
// and values are brought into shared memory once per CTA as exact f16 (bf16)
// tiles and multiplied by tcgen05.mma:
//   S = Q K^T   both operands in shared memory, 128 rows x 64 keys -> TMEM
//   O += P V    P in TMEM (written over S by the softmax warps), V in shared
//               memory as it is stored (head_dim contiguous: N-major)
// A CTA (one per SM) runs two streams of row tiles, so that one's softmax
// overlaps the other's products: either the two halves of a unit of 256 rows
// over the same tiles of keys, or two ranges of steps with up to 128 rows each
// (two "virtual CTAs"). Each stream has two buffers of S and one of O: 512
// columns of TMEM for both at head_dim 128.
// Warps: 0-3 and 4-7 softmax of streams 0 and 1 (a thread per row); 8-11 convert
// coded tiles, two of keys and two of values (bf16: 8 and 9 copy keys and
// values); 12 and 13 issue the streams' MMAs; 14 and 15 start the copies of
// coded keys and values.
//
// Bound: at 256 rows the tensor core, by how fast it is fed: an MMA of 128 x 64 x
// 16 with both operands in shared memory takes about 85 cycles for 32 of
// arithmetic, P V 71 for 64, so that a tile of 64 keys takes about 2,230 cycles
// for both streams where the arithmetic alone is 1,020. Measured on a GB300: 8
// lanes of 16,384 tokens, trees of 64, 32 query and 4 key/value heads of 128,
// bf16: 141 us (975 TFLOP/s of 1,946 measured); one lane of 260,096 tokens, 16
// drafts, 48 heads, FP8: 139 us (735 TFLOP/s). At up to 128 rows the bytes
// (bf16, 8 x 65,536 tokens, trees of 7: 188 us, 5.7 TB/s) or the conversion (FP8,
// NVFP4: 8 x 16,384 tokens, trees of 7: 81 and 74 us). S for 128 keys at a time
// halves the tensor core's work on S, but waits for both halves of P: no faster.
#include <atomic>
#include <type_traits>

#include "tcgen05.cuh"
#include "tree_common.cuh"

namespace qg {
namespace {

constexpr int kTcKeys = 64;                  // keys per tile
constexpr int kTcRows = 128;                 // rows per stream
constexpr int kTcThreads = 512;               // four warpgroups, 128 registers per thread at launch ...
constexpr int kMmaWarp = 12;                  // of stream 0; the next warp is stream 1's
constexpr int kCopyWarp = 14;                 // starts the copies of coded keys, the next of values
constexpr int kLaunchRegs = 128;
constexpr int kSoftmaxRegs = 144;            // ... dealt out anew: 2 * 144 + 104 + 120 = 4 * 128
constexpr int kLoadRegs = 104;
constexpr int kIssueRegs = 120;
static_assert(2 * kSoftmaxRegs + kLoadRegs + kIssueRegs <= 4 * kLaunchRegs, "more registers than the block has");
constexpr int kStages = 4;                   // tiles of keys and of values (SHARED; else two per stream)
constexpr int kMaxRaw = 3;                   // tiles of keys, and of values, as they are stored: see convert()
// Weights are 2^(s - z) with z = m - 8, replaced only once a score passes z by 15:
// a weight is at most 2^15, within f16, the largest at least 2^7. m is the row's
// largest score; for f16 weights rounded up to a whole number, so that a change of
// z scales what was summed by a power of two, without rounding. Not for bf16 ones:
// they have 8 bits, so the largest is 2^8 itself there, which they hold exactly (a
// row with one key gets its value as it is, where 2^-9 of it would show). The sum
// that divides has the weights before that rounding: lse is made of it. The
// exponent takes the product of score and factor unrounded, which is off from the
// rounded one in m by half a last place: too much from 2^24 on. Rows with a z of
// 2^23 or more ("far") round every product first, so that the largest is m itself,
// and take z = m, since m - 8 may round to anything between m - 16 and m there.
constexpr float kTcOffset = 8.f;
constexpr float kTcMost = 15.f;
constexpr float kTcFar = 8388608.f;
constexpr int kStagePitch = 20;              // floats per row of 16 columns on their way out: no bank twice

enum Bar : int {
    kKFull = 0,                              // [stage]
    kKEmpty = kKFull + kStages,
    kVFull = kKEmpty + kStages,
    kVEmpty = kVFull + kStages,
    kQFull = kVEmpty + kStages,              // [stream]
    kSFull = kQFull + 2,                     // [2 * stream + buffer]
    kPFull = kSFull + 4,
    kPvDone = kPFull + 4,
    kRawFull = kPvDone + 4,                  // [2 * raw stage + (0: keys, 1: values)]
    kRawEmpty = kRawFull + 2 * kMaxRaw,
    kVLand = kRawEmpty + 2 * kMaxRaw,
    kDrain = kVLand + 1,                     // [stream]
    kBars = kDrain + 2
};

template <int FMT, int D>
struct TcPlan {
    static constexpr int kQTile = kTcRows * D * 2;
    static constexpr int kTile = kTcKeys * D * 2;        // of keys or values, as f16 or bf16
    static constexpr int kHead = 1024;                   // barriers and what the warps tell each other
    static constexpr int kQ = kHead;
    static constexpr int kK = kQ + 2 * kQTile;
    static constexpr int kV = kK + kStages * kTile;
    static constexpr int kRaw = kV + kStages * kTile;
    static constexpr int kCodes = kTcKeys * kv_row_bytes(FMT, D);
    static constexpr int kRawStage = FMT == QG_KV_BF16 ? 0 : kCodes + kTcKeys * kv_scale_bytes(FMT, D);
    static constexpr int kFit = kRawStage ? (227 * 1024 - 1024 - kRaw) / (2 * (kRawStage ? kRawStage : 1)) : 0;
    static constexpr int kNRaw = kFit < kMaxRaw ? kFit : kMaxRaw;
    static constexpr int kSmem = kRaw + 2 * kNRaw * kRawStage + 1024;    // + alignment
    static_assert(kSmem <= 227 * 1024 && (FMT == QG_KV_BF16 || kNRaw >= 2), "too much shared memory");
    static_assert(kBars * 8 <= 512, "barriers");
};

// Operand tiles lie as blocks of 64 columns (128 bytes) by ROWS rows, the
// 16-byte pieces of a row permuted by the row's low three bits (the 128-byte
// swizzle). Byte offset of piece `ch` (of 8 values) of `row`.
template <int ROWS>
__device__ __forceinline__ uint32_t tile_at(int row, int ch)
{
    return (ch >> 3) * (ROWS * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
}

// Descriptors of such a tile. K-major (Q, K): eight rows are 1024 bytes apart.
// N-major (V): 64-column blocks are `lbo` apart, eight keys 1024 bytes.
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr, uint32_t lbo)
{
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
           static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}

// The n-th tile of a ring: its stage, and the parity of the phase in which it
// is filled. SHARED, one ring for both streams; else each stream has half.
template <bool SHARED>
struct Stage {
    uint32_t at, parity;
    __device__ __forceinline__ Stage(int stream, uint32_t n)
        : at(SHARED ? n % kStages : 2 * stream + n % 2), parity(SHARED ? n / kStages & 1u : n / 2 & 1u)
    {
    }
};

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

template <int N>
__device__ __forceinline__ void regs_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A bounded wait of a whole warp: all of its lanes go on, or none. It sleeps
// while it waits, so that it costs the other warps no issue slots.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const TreeArgs& t)
{
    bool ok = mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        const uint64_t t0 = global_timer_ns();
        while (!ok) {
            ok = mbar_try_wait_sleep(bar, parity, 10000);
            if (!ok && global_timer_ns() - t0 > t.wait_ns) {
                set_device_status(t.a.status, QG_ERR_DEVICE_TIMEOUT);
                break;
            }
        }
        ok = __all_sync(0xffffffffu, ok);
    }
    return ok;
}

// A piece of a unit: what one stream does between two epilogues.
struct Segment {
    int b, head;
    int row0, n_rows;            // query rows of the unit
    int first, end;              // keys
    int len, tok0, n_tok;        // context, the sequence's rows
    int tiles;
    int slot;                    // -1: the whole unit
};

// The segments of one virtual CTA's range of steps, in order: where the next
// begins, and the steps that are left.
struct Cursor {
    int64_t left;
    int b, head, tile, step;
    int vc;

    // by a whole warp
    __device__ __forceinline__ void locate(const TreeArgs& t, TreeScan& scan, int vcta)
    {
        vc = vcta;
        const int64_t at = tree_first(scan.total, t.grid, vcta);
        left = tree_first(scan.total, t.grid, vcta + 1) - at;
        b = head = tile = step = 0;
        if (left <= 0) return;
        KvSeq s;
        int64_t base;
        b = scan.find(t, at, s, base);
        const TreeSeq u = tree_seq_of(t, s);
        const int64_t unit = (at - base) / u.steps;
        step = static_cast<int>((at - base) % u.steps);
        head = static_cast<int>(unit / u.tiles);
        tile = static_cast<int>(unit % u.tiles);
    }

    template <int ROWS>
    __device__ __forceinline__ bool next(const TreeArgs& t, Segment& g)
    {
        if (left <= 0) return false;
        TreeSeq u = tree_seq_of(t, kv_seq(t.a, b, t.max_tree), kTcKeys, ROWS);
        while (u.steps == 0) u = tree_seq_of(t, kv_seq(t.a, ++b, t.max_tree), kTcKeys, ROWS);
        const int n = static_cast<int>(min(static_cast<int64_t>(u.steps - step), left));
        g.b = b;
        g.head = head;
        g.row0 = tile * ROWS;
        g.n_rows = min(ROWS, u.s.rows * t.group - g.row0);
        g.first = step * kTcKeys;
        g.end = min(u.keys, (step + n) * kTcKeys);
        g.len = u.s.len;
        g.tok0 = u.s.row0;
        g.n_tok = u.s.rows;
        g.tiles = n;
        g.slot = n == u.steps ? -1 : 2 * vc + (step == 0);
        left -= n;
        step += n;
        if (step == u.steps) {
            step = 0;
            if (++tile == u.tiles) {
                tile = 0;
                if (++head == t.a.heads) {
                    head = 0;
                    ++b;
                }
            }
        }
        return true;
    }
};

// The tiles of a CTA in the order in which they are brought and multiplied:
// SHARED, one cursor and every tile for both streams; else the two streams'
// tiles in turn while both have some.
template <int ROWS>
struct Side {
    Cursor cur;
    Segment seg;
    int tile;
    bool live;

    __device__ __forceinline__ void start(const TreeArgs& t, const Cursor& from)
    {
        cur = from;
        live = cur.template next<ROWS>(t, seg);
        tile = 0;
    }

    __device__ __forceinline__ void take(const TreeArgs& t, Segment& g, int& j)
    {
        g = seg;
        j = tile;
        if (++tile == g.tiles) {
            live = cur.template next<ROWS>(t, seg);
            tile = 0;
        }
    }
};

template <bool SHARED>
struct Items {
    Side<SHARED ? 2 * kTcRows : kTcRows> x, y;
    int turn;

    __device__ __forceinline__ void start(const TreeArgs& t, const Cursor* from)
    {
        turn = 0;
        x.start(t, from[0]);
        if (!SHARED) y.start(t, from[1]);
    }

    // The next tile: its stream (0 when SHARED), or -1 after the last.
    __device__ __forceinline__ int next(const TreeArgs& t, Segment& g, int& j)
    {
        if (SHARED) {
            if (!x.live) return -1;
            x.take(t, g, j);
            return 0;
        }
        if (!x.live && !y.live) return -1;
        if (y.live && (turn == 1 || !x.live)) {
            y.take(t, g, j);
            turn = 0;
            return 1;
        }
        x.take(t, g, j);
        turn = 1;
        return 0;
    }
};

// ------------------------------------------------------------------ loads
// What the warp that starts a tile's copies tells those that convert it.
struct RawInfo {
    int left;                    // keys of the tile, -1: there are no more tiles
    int drafts;                  // its keys from here on are drafts
    uint32_t groups;             // groups of 16 keys whose page lies in the cache
    uint32_t stage;              // where it goes, and the parity of its phase there
    uint32_t parity;
    uint32_t seq;                // which tile it is
    int pad[2];
};

// The runs of a tile: consecutive keys of one page, t.run of them (the largest
// of 16, 32 and 64 that divides the page size), one lane each. The page table
// is read 32 runs at a time, a lane each, and 32 runs ahead, so that a tile
// waits for none of it but at a segment's start.
template <bool SHARED>
struct Runs {
    Items<SHARED> items;
    int64_t row;                 // first row of this lane's run in the cache
    int keys;                    // its keys in the tile, up to a multiple of 16
    bool on;                     // it is copied
    RawInfo info;
    bool more;
    Segment g;
    int j, owner;
    int now[2], then[2];         // by stream: this lane's entries of the 32 runs at hand, and of the next 32
    uint32_t n[2];               // tiles of each ring so far

    __device__ __forceinline__ int key() const { return (threadIdx.x & 31); }

    __device__ __forceinline__ int entry(const TreeArgs& t, int q) const
    {
        const int p = g.first + (q + key()) * t.run;
        return p < g.end ? kv_entry(t.a, g.b, p) : 0;
    }

    // What the tile at hand needs of the page table is on its way.
    template <int S>
    __device__ __forceinline__ void look_up(const TreeArgs& t)
    {
        const int q = j * (kTcKeys / t.run);                 // its first run in the segment
        if (q % 32) return;
        now[S] = j ? then[S] : entry(t, 0);
        then[S] = entry(t, q + 32);
    }

    __device__ __forceinline__ void look_up(const TreeArgs& t)
    {
        if (owner == 0)
            look_up<0>(t);
        else if (!SHARED && owner == 1)
            look_up<SHARED ? 0 : 1>(t);
    }

    __device__ __forceinline__ void start(const TreeArgs& t, const Cursor* from)
    {
        items.start(t, from);
        n[0] = n[1] = 0;
        now[0] = now[1] = then[0] = then[1] = 0;
        owner = items.next(t, g, j);
        look_up(t);
        step(t);
    }

    __device__ __forceinline__ void step(const TreeArgs& t)
    {
        more = owner >= 0;
        if (!more) return;
        const Stage<SHARED> st(owner, owner ? n[1]++ : n[0]++);
        info.stage = st.at;
        info.parity = st.parity;
        const int p0 = g.first + j * kTcKeys, k0 = key() * t.run;
        info.left = min(kTcKeys, g.end - p0);
        info.drafts = g.len - p0;
        const int at = j * (kTcKeys / t.run) % 32 + key();
        const int found = __shfl_sync(0xffffffffu, !SHARED && owner ? now[1] : now[0], at & 31);
        const int page = k0 < info.left ? kv_valid(t.a, found) : -1;
        on = page >= 0;
        row = on ? kv_row(t.a, page, g.head, p0 + k0) : 0;
        keys = on ? min(t.run, (info.left - k0 + 15) & ~15) : 0;
        info.groups = __reduce_or_sync(0xffffffffu, on ? ((1u << (keys >> 4)) - 1u) << (k0 >> 4) : 0u);
        owner = items.next(t, g, j);
        look_up(t);
    }

    // Some of the tile's places get no key of the context.
    __device__ __forceinline__ static bool special(const RawInfo& i)
    {
        return i.left < kTcKeys || i.drafts < kTcKeys || i.groups != (1u << (kTcKeys / 16)) - 1u;
    }
};

// One 16-byte piece of a stored row as f16 values, eight to an element of `out`.
template <int FMT>
__device__ __forceinline__ void piece_values(const uint4 raw, uint32_t sc, uint4* out)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (FMT == QG_KV_FP8) {
        const uint32_t s2 = sc * 0x04000400u;                // 2^(s-15) as f16, twice
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo, hi;
            e4m3x4_to_f16x2x2(w[i], lo, hi);
            h[2 * i] = hmul2(lo, s2);
            h[2 * i + 1] = hmul2(hi, s2);
        }
        out[0] = make_uint4(h[0], h[1], h[2], h[3]);
        out[1] = make_uint4(h[4], h[5], h[6], h[7]);
    } else {
        const uint32_t f = e4m3x2_to_f16x2(sc);              // the scales of the piece's two blocks
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t s2 = __byte_perm(f, f, i < 2 ? 0x1010 : 0x3232);
            uint32_t h[4];
            e2m1x8_to_f16x2x4(w[i], h);
            out[i] = make_uint4(hmul2(h[0], s2), hmul2(h[1], s2), hmul2(h[2], s2), hmul2(h[3], s2));
        }
    }
}

// Zeroes each 16-bit value that is infinite or NaN.
template <bool BF16>
__device__ __forceinline__ void drop_odd(uint4& v, bool& odd)
{
    constexpr uint32_t e = BF16 ? 0x7F80u : 0x7C00u;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & e) == e) {
            w[i] &= 0xFFFF0000u;
            odd = true;
        }
        if (((w[i] >> 16) & e) == e) {
            w[i] &= 0x0000FFFFu;
            odd = true;
        }
    }
}

// What a warp wrote of a tile is in place: visible to the tensor core, then counted.
__device__ __forceinline__ void announce(uint64_t* bar)
{
    fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A tile of values with drafts, or with places that no key fills, by one warp:
// the places become zeros, and so does what is not finite of a draft (0 times it
// would reach rows that do not see the draft; it is flagged for the epilogue).
// Rare, so small rather than fast.
template <int D, bool BF16>
__device__ __noinline__ void clear_places(uint8_t* tile, int left, int drafts, uint32_t groups, volatile int* odd_flag,
                                          int lane)
{
    bool odd = false;
#pragma unroll 1
    for (int x = lane; x < kTcKeys * D / 8; x += 32) {
        const int key = x / (D / 8);
        const bool on = key < left && ((groups >> (key >> 4)) & 1u);
        if (on && key < drafts) continue;
        uint4* at = reinterpret_cast<uint4*>(tile + tile_at<kTcKeys>(key, x % (D / 8)));
        uint4 y = on ? *at : make_uint4(0, 0, 0, 0);
        drop_odd<BF16>(y, odd);
        *at = y;
    }
    if (odd) *odd_flag = 1;
    __syncwarp();
}

// Coded keys (kv = 0) or values (1): one warp each starts the copies of the
// tiles as they are stored, into a ring of raw stages. On a timeout it waits
// for the copies that are on their way.
template <int FMT, int D, bool SHARED>
__device__ __forceinline__ void copy_coded(const TreeArgs& t, const Cursor* from, uint8_t* smem, uint64_t* bar,
                                           RawInfo* infos, int kv)
{
    using P = TcPlan<FMT, D>;
    constexpr int kRow = kv_row_bytes(FMT, D), kScale = kv_scale_bytes(FMT, D);
    const int lane = threadIdx.x & 31;
    const uint8_t* codes = t.a.codes[kv];
    const uint8_t* scales = t.a.scales[kv];
    const bool go = kv == 1 || !t.starve;
    Runs<SHARED> runs;
    runs.start(t, from);
    uint32_t r = 0, phase = 0, n = 0;                        // raw stage, its phase's parity, tiles
    auto advance = [&]() {
        ++n;
        if (++r == P::kNRaw) {
            r = 0;
            phase ^= 1u;
        }
    };
    for (; runs.more; advance()) {
        const uint32_t x = 2 * r + kv;
        if (!warp_wait(&bar[kRawEmpty + x], phase ^ 1u, t)) {
            for (uint32_t y = go && n > P::kNRaw ? n - P::kNRaw : 0; go && y < n; ++y)
                warp_wait(&bar[kRawFull + 2 * (y % P::kNRaw) + kv], y / P::kNRaw & 1u, t);
            return;
        }
        uint8_t* dst = smem + P::kRaw + x * P::kRawStage;
        if (lane == 0) {
            runs.info.seq = n;
            infos[x] = runs.info;
            if (go) mbar_arrive_expect_tx(&bar[kRawFull + x], __popc(runs.info.groups) * 16 * (kRow + kScale));
        }
        __syncwarp();
        if (runs.on && go) {
            const int k0 = lane * t.run;
            bulk_load(dst + k0 * kRow, codes + runs.row * kRow, runs.keys * kRow, &bar[kRawFull + x]);
            bulk_load(dst + P::kCodes + k0 * kScale, scales + runs.row * kScale, runs.keys * kScale,
                      &bar[kRawFull + x]);
        }
        runs.step(t);
    }
    for (int y = 0; y < 2; ++y, advance()) {                 // no more: to both converting warps
        const uint32_t x = 2 * r + kv;
        if (!warp_wait(&bar[kRawEmpty + x], phase ^ 1u, t)) return;
        if (lane == 0) {
            infos[x].left = -1;
            infos[x].seq = n;
            mbar_arrive(&bar[kRawFull + x]);
        }
        __syncwarp();
    }
}

// ... and two warps convert keys, two values, every second tile each, to f16
// tiles. The two meet in a stage by turns, and a stage's parity alone would let
// a warp pass that comes too early (while the tile one round before its own has
// not landed): it looks at the tile's number too, and then at the parity again.
// Of the tiles before the one that a warp converts, all but the last are in
// place then: its own last one, and those whose raw stages were filled anew. So
// no tile before it can still wait for the same stage of the ring (the last has
// another), and the parity it waits for there is that of its own phase. That
// holds for up to three raw stages: with four, and one stream at its end, a warp
// could find its tile while the other still waits for that stage.
template <int FMT, int D>
__device__ __forceinline__ void convert(const TreeArgs& t, uint8_t* smem, uint64_t* bar, const RawInfo* infos,
                                        volatile int* odd_flag, int w)
{
    using P = TcPlan<FMT, D>;
    constexpr int kRow = kv_row_bytes(FMT, D), kScale = kv_scale_bytes(FMT, D);
    constexpr int kPerKey = kRow / 16;                       // pieces of a row
    constexpr int kN = kTcKeys * kPerKey / 32;               // pieces per lane
    constexpr int kChunks = FMT == QG_KV_FP8 ? 2 : 4;        // pieces of eight f16 from one of codes
    constexpr int kBatch = 4;
    const int lane = threadIdx.x & 31, kv = w & 1;
    // Piece x of this lane. At head_dim 128 eight neighbouring lanes take keys
    // of all residues (mod 2 for FP8, mod 4 for NVFP4) and, by residue, one or
    // the other half of the row: their reads and their swizzled writes then
    // fall into eight different groups of banks.
    auto key_of = [&](int x) {
        if constexpr (D == 128 && FMT == QG_KV_FP8) return 2 * ((x * 4 + (lane >> 3)) >> 1) + (lane >> 2 & 1);
        else if constexpr (D == 128) return 4 * ((x * 4 + (lane >> 3)) >> 1) + (lane >> 1 & 3);
        else return (x * 32 + lane) / kPerKey;
    };
    // its place in the row (the same for every x: x * 4 is even)
    const int half = lane >> 3 & 1;
    const int c = D != 128 ? lane % kPerKey
                  : FMT == QG_KV_FP8 ? (lane & 3) + 4 * ((lane >> 2 & 1) ^ half)
                                     : (lane & 1) + 2 * ((lane >> 2 & 1) ^ half);
    for (uint32_t n = w >> 1;; n += 2) {
        const uint32_t x = 2 * (n % P::kNRaw) + kv, phase = n / P::kNRaw & 1u;
        const volatile RawInfo* v = &infos[x];
        const uint64_t t0 = global_timer_ns();
        for (;;) {
            if (!warp_wait(&bar[kRawFull + x], phase, t)) return;
            if (__all_sync(0xffffffffu, v->seq == n)) break;
            if (__any_sync(0xffffffffu, global_timer_ns() - t0 > t.wait_ns)) {
                set_device_status(t.a.status, QG_ERR_DEVICE_TIMEOUT);
                return;
            }
        }
        if (!warp_wait(&bar[kRawFull + x], phase, t)) return;
        const RawInfo info = infos[x];
        if (info.left < 0) return;
        if (!warp_wait(&bar[(kv ? kVEmpty : kKEmpty) + info.stage], info.parity ^ 1u, t)) return;
        const uint32_t src = smem_u32(smem + P::kRaw + x * P::kRawStage);
        uint8_t* tile = smem + (kv ? P::kV : P::kK) + info.stage * P::kTile;
#pragma unroll 1
        for (int y0 = 0; y0 < kN; y0 += kBatch) {
            // a batch of pieces is read before any is converted, so that one latency covers them all
            uint4 raw[kBatch];
            uint32_t sc[kBatch];
#pragma unroll
            for (int y = 0; y < kBatch; ++y) {
                const int key = key_of(y0 + y);
                const uint32_t at = src + P::kCodes + key * kScale;
                raw[y] = lds128(src + key * kRow + c * 16);
                sc[y] = FMT == QG_KV_FP8 ? lds8(at) : lds16(at + 2 * c);
            }
#pragma unroll
            for (int y = 0; y < kBatch; ++y) {
                uint4 out[kChunks];
                piece_values<FMT>(raw[y], sc[y], out);
                const int key = key_of(y0 + y);
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
                    *reinterpret_cast<uint4*>(tile + tile_at<kTcKeys>(key, c * kChunks + i)) = out[i];
            }
        }
        // The raw stage can be filled again: only now, when every lane has stored what it made of it. (Once the
        // reads are merely issued is too early: the arrival does not wait for them, the next copy could come first.)
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kRawEmpty + x]);
        if (kv == 1 && Runs<false>::special(info)) {
            __syncwarp();
            clear_places<D, false>(tile, info.left, info.drafts, info.groups, odd_flag, lane);
        }
        announce(&bar[(kv ? kVFull : kKFull) + info.stage]);
    }
}

// bf16 keys (kv = 0) or values (1): copied straight into the tiles, swizzled on
// the way, by one warp each. A tile of values with places to clear is announced
// by this warp once it has done so. On a timeout it waits for the copies that
// are on their way.
template <int D, bool SHARED>
__device__ __forceinline__ void copy_plain(const TreeArgs& t, const CUtensorMap* map, const Cursor* from,
                                           uint8_t* tiles, uint64_t* full, uint64_t* empty, uint64_t* land,
                                           volatile int* odd_flag, int kv)
{
    constexpr int kTile = TcPlan<QG_KV_BF16, D>::kTile;
    const int lane = threadIdx.x & 31;
    Runs<SHARED> runs;
    runs.start(t, from);
    uint32_t landed = 0, filled = 0, parities = 0;               // stages ever filled, the parity of their last phase
    const bool go = kv == 1 || !t.starve;
    for (; runs.more; runs.step(t)) {
        const uint32_t st = runs.info.stage;
        if (!warp_wait(&empty[st], runs.info.parity ^ 1u, t)) {
            if (go)
                for (uint32_t x = 0; x < kStages; ++x)
                    if (filled >> x & 1u) warp_wait(&full[x], parities >> x & 1u, t);
            return;
        }
        filled |= 1u << st;
        parities = (parities & ~(1u << st)) | runs.info.parity << st;
        const bool clear = kv == 1 && Runs<SHARED>::special(runs.info);
        uint64_t* done = clear ? land : &full[st];
        // boxes are whole runs: what lies behind the last key is cleared or masked
        const uint32_t n_runs = __popc(__ballot_sync(0xffffffffu, runs.on));
        if (lane == 0 && go) mbar_arrive_expect_tx(done, n_runs * t.run * D * 2);
        __syncwarp();
        if (runs.on && go)
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
                tma_load_2d(tiles + st * kTile + x * (kTcKeys * 128) + lane * t.run * 128, map, 64 * x,
                            static_cast<int32_t>(runs.row), done);
        if (clear) {
            if (!warp_wait(land, landed++ & 1u, t)) return;
            clear_places<D, true>(tiles + st * kTile, runs.info.left, runs.info.drafts, runs.info.groups, odd_flag,
                                  lane);
            announce(&full[st]);
        }
    }
}

// ------------------------------------------------------------------ softmax
using f2 = unsigned long long;               // two floats, low half first
__device__ __forceinline__ f2 f2_pack(float lo, float hi)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_unpack(f2 v, float& lo, float& hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b)
{
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The weights of a tile for a warp with far rows, 32 keys at a time: their sum.
// Rare, and out of line: 64 products with a factor in the way of every tile cost up
// to 8 % (4-bit, 260,096 keys: 131 -> 141 us).
template <bool BF16>
__device__ __noinline__ float far_weights(uint32_t ts, float rowf, float z, uint32_t seen0, uint32_t seen1)
{
    const bool far = fabsf(z) >= kTcFar;
    const float first = far ? rowf : 1.f, then = far ? 1.f : rowf;
    const float zs = z == -INFINITY ? 0.f : -z;
    float sum = 0.f;
#pragma unroll 1
    for (int y = 0; y < 2; ++y) {
        const uint32_t seen = y ? seen1 : seen0;
        uint32_t x[32], h[16];
        tc_ld<32>(ts + 32 * y, x);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float s = __fmul_rn(__uint_as_float(tc_after_wait(x[i + e])), first);
                w[e] = (seen >> (i + e)) & 1u ? ex2(fmaf(s, then, zs)) : 0.f;
                sum += w[e];
            }
            h[i / 2] = pack16<BF16>(w[0], w[1]);
        }
        tc_st_x16(ts + 16 * y, h);
        tc_wait_st();
    }
    return sum;
}

// One tile's 64 scores of this thread's row to weights, in place: the weights
// of 32 keys take the columns of 16 scores that were read before. A row whose
// scores became too large for its z has z raised, and what was summed with the
// old one is scaled: l and the row of O, once the products of the tile before
// are complete (those before it are: they came ahead of these scores). That is
// rare, so small rather than fast.
template <bool BF16, bool SPECIAL, int D>
__device__ __forceinline__ bool weights(const TreeArgs& t, uint32_t ts, uint32_t to, uint64_t* before, uint32_t parity,
                                        float rowf, const uint32_t (&seen)[2], float& z, float& l, bool& far)
{
    uint32_t x[64];
    tc_ld<32>(ts, x);
    tc_ld<32>(ts + 32, x + 32);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 64; ++i) x[i] = tc_after_wait(x[i]);
    if constexpr (SPECIAL) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
            if (!((seen[i / 32] >> (i & 31)) & 1u)) x[i] = 0xFF800000u;
    }
    float mx[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) mx[i] = fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 4]));
#pragma unroll
    for (int i = 8; i < 64; i += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(x[i + e])), __uint_as_float(x[i + e + 4]));
    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * rowf;
    if (__any_sync(0xffffffffu, top - z > kTcMost)) {
        const float m = BF16 ? top : ceilf(top);
        const float zn = fmaxf(z, fabsf(m) < kTcFar ? m - kTcOffset : m);   // fmaxf: z where m is NaN
        const float f = zn == -INFINITY ? 1.f : ex2(z - zn);
        z = zn;
        far = __any_sync(0xffffffffu, fabsf(z) >= kTcFar && fabsf(z) < INFINITY);
        l *= f;
        if (before) {
            if (!warp_wait(before, parity, t)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
                uint32_t v[16];
                tc_ld<16>(to + 16 * c, v);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(tc_after_wait(v[i])) * f);
                tc_st_x16(to + 16 * c, v);
            }
        }
    }
    if (far) {
        l += far_weights<BF16>(ts, rowf, z, SPECIAL ? seen[0] : ~0u, SPECIAL ? seen[1] : ~0u);
        return true;
    }
    const float zs = z == -INFINITY ? 0.f : -z;
    const f2 rowf2 = f2_pack(rowf, rowf), z2 = f2_pack(zs, zs);
    f2 sum[2] = {0, 0};
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        uint32_t h[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[32 * y + i]), __uint_as_float(x[32 * y + i + 1])), rowf2, z2),
                      x0, x1);
            x0 = ex2(x0);
            x1 = ex2(x1);
            if constexpr (SPECIAL) {         // also where z is still -infinity, or the scale is 0
                x0 = (seen[y] >> i) & 1u ? x0 : 0.f;
                x1 = (seen[y] >> (i + 1)) & 1u ? x1 : 0.f;
            }
            sum[(i >> 1) & 1] = f2_add(sum[(i >> 1) & 1], f2_pack(x0, x1));
            h[i / 2] = pack16<BF16>(x0, x1);
        }
        tc_st_x16(ts + 16 * y, h);
    }
    float a, b, a1, b1;
    f2_unpack(sum[0], a, a1);
    f2_unpack(sum[1], b, b1);
    l += (a + a1) + (b + b1);
    tc_wait_st();
    return true;
}

// ------------------------------------------------------------------ products
// One MMA with both operands in shared memory.
template <bool ACCUMULATE>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(ACCUMULATE ? 1 : 0)
        : "memory");
}

// One warp per stream issues its products: S of a tile into one of two
// buffers, and O += P V once the weights have taken its place; S runs two tiles
// ahead of P V, so that scores are ready when the softmax warps want them. S of a
// tile overwrites the weights that the P V two tiles before reads, and waits for
// its end: products with different accumulators are not promised to run in the
// order in which they were issued. (Without the wait nothing was ever seen to go
// wrong; when it came it cost 133 -> 141 us over 260,096 keys in FP8 with 16 drafts, 156 ->
// 162 us for 8 x 16,384 with trees of 64, and 1 us in most others.) The whole
// warp walks the tiles, so that what addresses them stays in uniform registers;
// one lane issues.
template <int FMT, int D, bool SHARED>
__device__ __forceinline__ bool multiply(const TreeArgs& t, const Cursor* from, uint8_t* smem, uint64_t* bar,
                                         uint32_t tmem, int s, bool leader)
{
    using P = TcPlan<FMT, D>;
    constexpr bool kBf16 = FMT == QG_KV_BF16;
    constexpr uint32_t id_s = tc_idesc_f16(128, kTcKeys, kBf16);
    constexpr uint32_t id_o = tc_idesc_f16(128, D, kBf16) | 1u << 16;   // B is N-major
    const uint64_t dq = tile_desc(smem_u32(smem + P::kQ) + s * P::kQTile, 16);
    const uint64_t dk = tile_desc(smem_u32(smem + P::kK), 16);
    const uint64_t dv = tile_desc(smem_u32(smem + P::kV), kTcKeys * 128);
    const uint32_t ts = tmem + 256 * s, to = ts + 128;
    auto wait = [&](int b, uint32_t parity) { return warp_wait(&bar[b], parity, t); };
    uint32_t n = 0, x = 0, y = 0, nq = 0;            // ring position; tiles with S and with P V issued; segments
    uint32_t starts = 0;                             // bit x % 32: tile x is its segment's first
    uint32_t rings[2] = {0, 0};                      // ring positions of the tiles between y and x
    auto product_v = [&]() {
        const uint32_t buf = y & 1u;
        const Stage<SHARED> st(s, buf ? rings[1] : rings[0]);
        if (!wait(kVFull + st.at, st.parity) || !wait(kPFull + 2 * s + buf, y / 2 & 1u)) return false;
        tc_fence_after();
        const uint64_t d = dv + st.at * (P::kTile >> 4);
        const uint32_t tp = ts + 64 * buf;
        const bool keep = !(starts >> (y & 31u) & 1u);
        if (leader) {
            tc_mma_f16_ts(to, tp, d, id_o, keep);
#pragma unroll
            for (int i = 1; i < kTcKeys / 16; ++i) tc_mma_f16_ts(to, tp + 8 * i, d + i * (2048 >> 4), id_o, true);
            tc_commit(&bar[kPvDone + 2 * s + buf]);
            tc_commit(&bar[kVEmpty + st.at]);
        }
        __syncwarp();
        ++y;
        return true;
    };
    Items<SHARED> items;
    items.start(t, from);
    Segment g;
    int j, owner;
    while ((owner = items.next(t, g, j)) >= 0) {
        if (!SHARED && owner != s) continue;
        // before a segment's first S everything of the one before is issued: its Q is replaced after its epilogue
        const bool idle = SHARED && s == 1 && g.n_rows <= kTcRows;      // the other stream's tile alone
        while (y < x && (j == 0 || idle || x - y == 2))
            if (!product_v()) return false;
        const Stage<SHARED> st(s, n);
        if (!wait(kKFull + st.at, st.parity)) return false;
        if (idle) {                                  // only counted
            if (leader) mbar_arrive(&bar[kKEmpty + st.at]);
            if (!wait(kVFull + st.at, st.parity)) return false;
            if (leader) mbar_arrive(&bar[kVEmpty + st.at]);
            ++n;
            continue;
        }
        if (j == 0 && !wait(kQFull + s, nq++ & 1u)) return false;
        const uint32_t buf = x & 1u;
        // these scores take the place of weights that P V of two tiles before reads
        if (x >= 2 && !wait(kPvDone + 2 * s + buf, (x / 2 - 1) & 1u)) return false;
        tc_fence_after();
        if (leader) {
            const uint64_t d = dk + st.at * (P::kTile >> 4);
            mma_ss<false>(ts + 64 * buf, dq, d, id_s);
#pragma unroll
            for (int i = 1; i < D / 16; ++i)
                mma_ss<true>(ts + 64 * buf, dq + (((i >> 2) * (kTcRows * 128) + (i & 3) * 32) >> 4),
                             d + (((i >> 2) * (kTcKeys * 128) + (i & 3) * 32) >> 4), id_s);
            tc_commit(&bar[kSFull + 2 * s + buf]);
            tc_commit(&bar[kKEmpty + st.at]);
        }
        __syncwarp();
        starts = (starts & ~(1u << (x & 31u))) | static_cast<uint32_t>(j == 0) << (x & 31u);
        if (buf)
            rings[1] = n;
        else
            rings[0] = n;
        ++n;
        ++x;
    }
    while (y < x)
        if (!product_v()) return false;
    return true;
}

// The sum of the values at column d that are not finite, of the drafts that a
// row sees (they were left out of the tiles; whatever their weights, they make
// the output infinite or NaN). Rare.
__device__ __noinline__ float odd_sum(const KvArgs& a, int b, int head, int first, int end, int len, uint64_t mask,
                                      int d)
{
    float sum = 0.f;
    for (int p = max(first, len); p < end; ++p) {
        if (!((mask >> (p - len)) & 1ull)) continue;
        const int page = kv_page(a, b, p);
        if (page < 0) continue;
        const float x = kv_value(a, 1, kv_row(a, page, head, p), d);
        if (!(fabsf(x) < INFINITY)) sum += x;
    }
    return sum;
}

template <int FMT, int D, bool SHARED>
__global__ void __launch_bounds__(kTcThreads, 1) tree_tc_kernel(const __grid_constant__ TreeArgs t,
                                                                const __grid_constant__ CUtensorMap k_map,
                                                                const __grid_constant__ CUtensorMap v_map)
{
    using P = TcPlan<FMT, D>;
    constexpr bool kBf16 = FMT == QG_KV_BF16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 512);
    volatile int* odd_flag = reinterpret_cast<volatile int*>(smem + 520);   // a draft's value was not finite
    const KvArgs& a = t.a;
    const int lane = threadIdx.x & 31, warp = warp_index_uniform();

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // what earlier kernels wrote is read by bulk copies too
    asm volatile("fence.proxy.async;" ::: "memory");
    Cursor* from = reinterpret_cast<Cursor*>(smem + 576);    // where the CTA's one or two ranges begin
    RawInfo* infos = reinterpret_cast<RawInfo*>(smem + 640);
    if (warp < 2) {
        TreeScan scan;
        scan.run(t);
        Cursor c;
        c.locate(t, scan, warp * gridDim.x + blockIdx.x);
        if (lane == 0) from[warp] = c;
    }
    if (threadIdx.x == 64) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bar[kKFull + s], 1);
            mbar_init(&bar[kKEmpty + s], SHARED ? 2 : 1);
            mbar_init(&bar[kVFull + s], 1);
            mbar_init(&bar[kVEmpty + s], SHARED ? 2 : 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar[kQFull + s], 4);
            mbar_init(&bar[kDrain + s], 1);
        }
        for (int x = 0; x < 4; ++x) {
            mbar_init(&bar[kSFull + x], 1);
            mbar_init(&bar[kPFull + x], 4);
            mbar_init(&bar[kPvDone + x], 1);
        }
        for (int x = 0; x < 2 * kMaxRaw; ++x) {
            mbar_init(&bar[kRawFull + x], 1);
            mbar_init(&bar[kRawEmpty + x], 1);
        }
        mbar_init(&bar[kVLand], 1);
        for (int x = 0; x < 2 * kMaxRaw; ++x) infos[x].seq = ~0u;
        *odd_flag = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tc_alloc(tmem_slot, 512);
        tc_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;                // stream s: S and P at 256 s (two buffers), O at 256 s + 128

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        regs_up<kSoftmaxRegs>();
        const int s = warp >> 2;
        const int r = threadIdx.x & 127;             // row of the stream's tile = TMEM lane
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + 256 * s, to = ts + 128;
        uint32_t x = 0;                              // tiles so far
        bool ok = true;
        Cursor mine = from[SHARED ? 0 : s];
        Segment g;
        while (ok && mine.template next<SHARED ? 2 * kTcRows : kTcRows>(t, g)) {
            const int base = SHARED ? 128 * s : 0;
            const int n_rows = g.n_rows - base;      // of this stream
            if (n_rows <= 0) continue;
            const bool on = r < n_rows;
            const bool busy = 32 * (warp & 3) < n_rows;
            const int row = g.row0 + base + (on ? r : 0);
            const int tok = row / t.group, qh = g.head * t.group + row % t.group;
            // on their way together with the row of Q
            const uint64_t mask_word = t.mask ? t.mask[g.tok0 + tok] : (2ull << tok) - 1;
            int p_check = g.first - g.first % a.page_size + lane * a.page_size;
            const int entry = p_check < g.end ? kv_entry(a, g.b, p_check) : 0;
            // ---- this row of Q, times a power of two that brings its largest value to f16's upper range
            float rowf = 0.f;
            {
                uint32_t w[D / 2];
                const uint4* src = reinterpret_cast<const uint4*>(t.q + (g.tok0 + tok) * t.q_stride + qh * D);
                uint32_t mag = 0;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 v = on ? src[i] : make_uint4(0, 0, 0, 0);
                    w[4 * i] = v.x;
                    w[4 * i + 1] = v.y;
                    w[4 * i + 2] = v.z;
                    w[4 * i + 3] = v.w;
                }
                int pe = 0;
                if constexpr (!kBf16) {
#pragma unroll
                    for (int i = 0; i < D / 2; ++i) {
                        const uint32_t m = w[i] & 0x7FFF7FFFu;
                        mag = max(mag, max(m & 0xFFFFu, m >> 16));
                    }
                    pe = mag < 0x7F80u ? prescale_exponent(mag) : 0;
                }
                // a negative scale turns q round, so that larger products are always larger scores
                const uint32_t flip = t.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    uint32_t h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x = w[4 * i + e];
                        if constexpr (kBf16)
                            h[e] = x ^ flip;
                        else
                            h[e] = pack_f16x2(ldexp_exact(__uint_as_float(x << 16), pe),
                                              ldexp_exact(__uint_as_float(x & 0xFFFF0000u), pe)) ^
                                   flip;
                    }
                    *reinterpret_cast<uint4*>(smem + P::kQ + s * P::kQTile + tile_at<kTcRows>(r, i)) =
                        make_uint4(h[0], h[1], h[2], h[3]);
                }
                rowf = ldexp_exact(fabsf(t.scale) * kLog2e * a.g[0], -pe);
            }
            const uint64_t own = g.n_tok < 64 ? (1ull << g.n_tok) - 1 : ~0ull;
            const uint64_t mask = mask_word & own;
            bool bad = kv_valid(a, entry) < 0 && p_check < g.end;   // a page of these keys lies outside the cache
            for (p_check += 32 * a.page_size; p_check < g.end; p_check += 32 * a.page_size)
                bad = kv_page(a, g.b, p_check) < 0 || bad;
            bad = __any_sync(0xffffffffu, bad);
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kQFull + s]);

            float z = -INFINITY, l = 0.f;
            bool far = false;
            for (int j = 0; j < g.tiles; ++j, ++x) {
                const uint32_t buf = x & 1u;
                ok = warp_wait(&bar[kSFull + 2 * s + buf], x / 2 & 1u, t);
                if (!ok) break;
                tc_fence_after();
                if (busy) {
                    const int p0 = g.first + j * kTcKeys;
                    uint64_t* before = j > 0 ? &bar[kPvDone + 2 * s + (buf ^ 1u)] : nullptr;
                    const uint32_t parity = (x - 1) / 2 & 1u;
                    uint32_t seen[2] = {~0u, ~0u};
                    if (p0 + kTcKeys > g.len || bad) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int off = p0 + 32 * c - g.len;
                            seen[c] = off <= -32 ? ~0u
                                      : off < 0  ? ((1u << -off) - 1u) | static_cast<uint32_t>(mask << -off)
                                      : off < 64 ? static_cast<uint32_t>(mask >> off)
                                                 : 0u;
                            if (bad)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const int p = p0 + 32 * c + 16 * y;
                                    if (p < g.end && kv_page(a, g.b, p) < 0) seen[c] &= ~(0xFFFFu << (16 * y));
                                }
                        }
                        ok = weights<kBf16, true, D>(t, ts + 64 * buf, to, before, parity, rowf, seen, z, l, far);
                    } else {
                        ok = weights<kBf16, false, D>(t, ts + 64 * buf, to, before, parity, rowf, seen, z, l, far);
                    }
                    if (!ok) break;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kPFull + 2 * s + buf]);
            }
            if (!ok) break;
            ok = warp_wait(&bar[kPvDone + 2 * s + ((x - 1) & 1u)], (x - 1) / 2 & 1u, t);
            if (!ok) break;
            tc_fence_after();
            if (!busy) continue;
            const int64_t h = static_cast<int64_t>(g.tok0 + tok) * t.q_heads + qh;
            const bool some = l > 0.f || l != l;     // the row saw a key
            const float scale = g.slot < 0 ? tree_inverse(l) * a.g[1] : 1.f;
            const int64_t at = static_cast<int64_t>(g.slot) * t.rows + base + r;
            const bool fix = g.end > g.len && *odd_flag;
            // Rows are stored 16 columns at a time through shared memory, where this warp's rows of Q were, so
            // that a store's lanes write whole runs of a few rows rather than 16 bytes of each.
            uint8_t* row_out = !on         ? nullptr
                               : g.slot < 0 ? reinterpret_cast<uint8_t*>(t.out + h * D)
                                            : reinterpret_cast<uint8_t*>(t.part_o + at * D);
            float* stage = reinterpret_cast<float*>(smem + P::kQ + s * P::kQTile + (warp & 3) * 4096);
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
                uint32_t v[16];
                __syncwarp();
                tc_ld<16>(to + 16 * c, v);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = tc_after_wait(v[i]);
                if (fix && on) {
#pragma unroll 1
                    for (int i = 0; i < 16; ++i) {
                        const float x = odd_sum(a, g.b, g.head, g.first, g.end, g.len, mask, 16 * c + i);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (e == i) v[e] = __float_as_uint(__uint_as_float(v[e]) + x);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = some ? __uint_as_float(v[4 * i + e]) * scale : 0.f;
                    *reinterpret_cast<float4*>(stage + lane * kStagePitch + 4 * i) = make_float4(y[0], y[1], y[2], y[3]);
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {        // eight rows at a time, four lanes each
                    const int from = 8 * i + lane / 4;
                    const float4 y = *reinterpret_cast<const float4*>(stage + from * kStagePitch + lane % 4 * 4);
                    uint8_t* dst = reinterpret_cast<uint8_t*>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row_out), from));
                    if (!dst) continue;
                    if (g.slot < 0)
                        *reinterpret_cast<uint2*>(dst + c * 32 + lane % 4 * 8) =
                            make_uint2(pack16<true>(y.x, y.y), pack16<true>(y.z, y.w));
                    else
                        *reinterpret_cast<float4*>(dst + c * 64 + lane % 4 * 16) = y;
                }
            }
            __syncwarp();                            // before the next row of Q takes the place
            if (on) {
                if (g.slot >= 0)
                    t.part_ml[at] = make_float2(z, l);
                else if (t.lse)
                    t.lse[h] = tree_lse(z, l);
            }
        }
    } else if (warp < kMmaWarp) {
        regs_down<kLoadRegs>();
        if constexpr (kBf16) {
            const int kv = warp - 8;
            if (kv < 2)
                copy_plain<D, SHARED>(t, kv ? &v_map : &k_map, from, smem + (kv ? P::kV : P::kK),
                                      &bar[kv ? kVFull : kKFull], &bar[kv ? kVEmpty : kKEmpty], &bar[kVLand], odd_flag,
                                      kv);
        } else {
            convert<FMT, D>(t, smem, bar, infos, odd_flag, warp - 8);
        }
    } else {
        regs_down<kIssueRegs>();
        if (warp < kMmaWarp + 2) {
            const int s = warp - kMmaWarp;
            const bool leader = elect_one();
            if (!multiply<FMT, D, SHARED>(t, from, smem, bar, tmem, s, leader)) {
                if (leader) tc_commit(&bar[kDrain + s]);     // given up: products on their way still end
                warp_wait(&bar[kDrain + s], 0, t);
            }
        } else if constexpr (!kBf16) {
            copy_coded<FMT, D, SHARED>(t, from, smem, bar, infos, warp - kCopyWarp);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

template <int FMT, int D, bool SHARED>
cudaError_t run_tc(TreeArgs t, cudaStream_t stream)
{
    using P = TcPlan<FMT, D>;
    auto kern = tree_tc_kernel<FMT, D, SHARED>;
    // The warpgroups' registers are dealt out anew inside the kernel, which
    // would wait for ever for more than the block was launched with.
    static const bool fits = [&] {
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, kern) == cudaSuccess && f.numRegs >= kLaunchRegs;
    }();
    if (!fits) return cudaErrorInvalidConfiguration;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, P::kSmem, done);
    if (e != cudaSuccess) return e;
    const int sms = sm_count(-1);
    t.step = kTcKeys;
    t.grid = SHARED ? sms : 2 * sms;
    t.run = 16;
    while (t.run < kTcKeys && t.a.page_size % (2 * t.run) == 0) t.run *= 2;
    CUtensorMap maps[2] = {};
    const uint64_t rows = static_cast<uint64_t>(t.a.num_pages) * t.a.heads * t.a.page_size;
    if (FMT == QG_KV_BF16)
        for (int kv = 0; kv < 2; ++kv)
            // (rows fit a coordinate: tree_attention_serves)
            if (!encode_tmap_2d(&maps[kv], t.a.codes[kv], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, D, rows, 64, t.run,
                                true))
                return cudaErrorInvalidValue;
    e = launch_pdl(kern, dim3(static_cast<unsigned>(sms)), dim3(kTcThreads), P::kSmem, stream, t, maps[0], maps[1]);
    if (e != cudaSuccess) return e;
    return launch_tree_join(t, stream);
}

template <int FMT>
cudaError_t run_tc_format(const TreeArgs& t, cudaStream_t stream)
{
    if (t.a.dim == 64)
        return t.rows == 256 ? run_tc<FMT, 64, true>(t, stream) : run_tc<FMT, 64, false>(t, stream);
    return t.rows == 256 ? run_tc<FMT, 128, true>(t, stream) : run_tc<FMT, 128, false>(t, stream);
}

}  // namespace

cudaError_t launch_tree_tc(const TreeArgs& t, cudaStream_t stream)
{
    return t.a.fmt == QG_KV_BF16  ? run_tc_format<QG_KV_BF16>(t, stream)
           : t.a.fmt == QG_KV_FP8 ? run_tc_format<QG_KV_FP8>(t, stream)
                                  : run_tc_format<QG_KV_NVFP4>(t, stream);
}

}  // namespace qg

// kv_pages.cu -- the pages that sequences of a cache share: rows of a page
// table go on from others (kv_pages_fork), get pages for what they write next
// (kv_pages_reserve), are moved to the front of the pool (kv_pages_compact),
// and the moves that these ask for are carried out in a layer's cache
// (kv_pages_copy). refs[p] counts the holders of page p; a free page is one
// that nobody holds, and the lowest free ones are handed out first, so that no
// list of free pages, and no order of its entries, has to be kept.
#include "kv_common.cuh"

namespace qg {
namespace {

constexpr int kForkThreads = 256, kForkCols = 32;
constexpr int kPlanThreads = 1024;
constexpr int kTableThreads = 256;
constexpr int kHash = 2048;
constexpr int kCopyWarps = 8, kCopyPieces = 4;
constexpr int kScaleChunk = 4096;

// ------------------------------------------------------------------ rows
// Row b of a page record: its tokens and entries, none if they do not fit.
struct PageRow {
    int len;
    int held;
    bool ok;
};

__device__ __forceinline__ PageRow page_row(const PageArgs& a, int b)
{
    PageRow r;
    r.len = a.lens[b];
    r.held = a.held[b];
    r.ok = r.len >= 0 && r.len <= kKvMaxPositions && r.held >= 0 && r.held <= a.max_pages &&
           (r.len + a.page_size - 1) / a.page_size <= r.held;
    if (!r.ok) r.len = r.held = 0;
    return r;
}

__device__ __forceinline__ bool in_pool(const PageArgs& a, int page)
{
    return static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages);
}

__device__ __forceinline__ int parent_of(const PageArgs& a, const int32_t* parent, int i, bool& bad)
{
    const int p = parent[i];
    bad = p < -1 || p >= a.n_seqs;
    return bad ? i : p;
}

// ------------------------------------------------------------------ fork
// A block takes kForkCols columns of the whole table: every row's entries go
// to shared memory first, so that rows may be permuted in place. An entry of
// old row j is held by kids[j] rows afterwards (by none behind the page of the
// row's last token) and was held once: refs changes by the difference.
__global__ void __launch_bounds__(kForkThreads) pages_fork_kernel(const __grid_constant__ PageArgs a, const int32_t* parent)
{
    extern __shared__ int smem[];
    pdl_enter();
    const int n = a.n_seqs, tid = threadIdx.x;
    int* par = smem;
    int* keep = par + n;
    int* held = keep + n;
    int* kids = held + n;
    int* slab = kids + n;
    for (int i = tid; i < n; i += kForkThreads) kids[i] = 0;
    __syncthreads();
    int most = 0;
    for (int i = tid; i < n; i += kForkThreads) {
        bool bad;
        const PageRow r = page_row(a, i);
        const int p = parent_of(a, parent, i, bad);
        if (blockIdx.x == 0 && (bad || !r.ok)) set_device_status(a.status, QG_ERR_INVALID_ARG);
        par[i] = p;
        keep[i] = (r.len + a.page_size - 1) / a.page_size;
        held[i] = r.held;
        most = max(most, r.held);
        if (p >= 0) atomicAdd(&kids[p], 1);
    }
    const int c = static_cast<int>(blockIdx.x) * kForkCols + (tid & 31);
    if (__syncthreads_or(most > static_cast<int>(blockIdx.x) * kForkCols) == 0) return;
    for (int j = tid >> 5; j < n; j += kForkThreads / 32) {
        if (c >= held[j]) continue;
        const int e = a.table[static_cast<int64_t>(j) * a.max_pages + c];
        slab[j * kForkCols + (tid & 31)] = e;
        const int change = (c < keep[j] ? kids[j] : 0) - 1;
        if (!in_pool(a, e))
            set_device_status(a.status, QG_ERR_INVALID_ARG);
        else if (change)
            atomicAdd(&a.refs[e], change);
    }
    __syncthreads();
    for (int i = tid >> 5; i < n; i += kForkThreads / 32) {
        const int p = par[i];
        if (p < 0 || p == i || c >= keep[p]) continue;
        a.table[static_cast<int64_t>(i) * a.max_pages + c] = slab[p * kForkCols + (tid & 31)];
    }
}

// The lengths and counts of entries, after the table: one block, which reads
// all of them before it writes any.
__global__ void __launch_bounds__(kPlanThreads) pages_fork_rows_kernel(const __grid_constant__ PageArgs a, const int32_t* parent)
{
    pdl_enter();
    const int i = threadIdx.x;
    int len = 0;
    if (i < a.n_seqs) {
        bool bad;
        const int p = parent_of(a, parent, i, bad);
        len = p < 0 ? 0 : page_row(a, p).len;
    }
    __syncthreads();
    if (i < a.n_seqs) {
        a.lens[i] = len;
        a.held[i] = (len + a.page_size - 1) / a.page_size;
    }
}

// ------------------------------------------------------------------ scans over the pool
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Every thread of the cluster arrives and waits; what was written before, to
// shared or global memory, is seen after.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// The word at `p` of this block's shared memory in block `rank` of the cluster.
__device__ __forceinline__ int cluster_word(const int* p, uint32_t rank)
{
    uint32_t at;
    int v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// Sum over the block of v, and what the threads before this one have.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    T s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    const T before = __shfl_sync(0xffffffffu, s, warp ? warp - 1 : 0);
    return x - v + (warp ? before : T(0));
}

// A block's share of the pool, `words` words of 32 pages from word `word0` on:
// bit i of a word is set for a page that is held (free_bits: that is free).
// Pages behind the pool have bit 0.
__device__ __forceinline__ void scan_refs(const PageArgs& a, int word0, int words, bool free_bits, uint32_t* bits)
{
    const int lane = threadIdx.x & 31;
    const int64_t first = static_cast<int64_t>(word0) * 32;
    for (int base = 0; base < words * 32; base += 4 * kPlanThreads) {
        const int at = base + 4 * static_cast<int>(threadIdx.x);
        const int64_t p = first + at;
        uint32_t nib = 0;
        if (at < words * 32) {
            if (p + 4 <= a.num_pages) {
                const int4 r = *reinterpret_cast<const int4*>(a.refs + p);
                nib = (r.x != 0) | (r.y != 0) << 1 | (r.z != 0) << 2 | (r.w != 0) << 3;
                if (free_bits) nib ^= 15u;
            } else {
                for (int i = 0; i < 4; ++i)
                    if (p + i < a.num_pages) nib |= static_cast<uint32_t>((a.refs[p + i] != 0) != free_bits) << i;
            }
        }
        uint32_t w = nib << (4 * (lane & 7));
        w |= __shfl_xor_sync(0xffffffffu, w, 1);
        w |= __shfl_xor_sync(0xffffffffu, w, 2);
        w |= __shfl_xor_sync(0xffffffffu, w, 4);
        if ((lane & 7) == 0 && at < words * 32) bits[at / 32] = w;
    }
    __syncthreads();
}

// The words of this block of the cluster, and of each of its threads.
struct Share {
    int word0;
    int words;
    int per;
    int from;
    int to;
};

__device__ __forceinline__ Share share_of(const PageArgs& a)
{
    Share s;
    const int all = (a.num_pages + 31) / 32, size = static_cast<int>(cluster_size());
    const int each = (all + size - 1) / size;
    s.word0 = min(static_cast<int>(cluster_rank()) * each, all);
    s.words = min(each, all - s.word0);
    s.per = (s.words + kPlanThreads - 1) / kPlanThreads;
    s.from = min(static_cast<int>(threadIdx.x) * s.per, s.words);
    s.to = min(s.from + s.per, s.words);
    return s;
}

// ------------------------------------------------------------------ reserve
struct ReserveSmem {
    int off[kKvMaxSeqs + 1];     // new pages before row b
    int first[kKvMaxSeqs];       // the table column of a page that is replaced, -1: none
    int held[kKvMaxSeqs];
    int tail[kKvMaxSeqs];        // the page that is replaced
    int tokens[kKvMaxSeqs];      // its tokens
    int move[kKvMaxSeqs];        // its place among the moves
    int page[kHash];             // part-filled pages that rows of the call write,
    int writers[kHash];          // how many do,
    int lowest[kHash];           // and the lowest of them
    int64_t sums[32];
    int count;
};

// One cluster. Each block looks at every row (thread b at row b) and at its
// share of the pool; with the free pages of the blocks before it, it knows the
// number that each of its free pages has among all, and so the row and the
// column that each is for. Nothing is written before every block has read.
__global__ void __launch_bounds__(kPlanThreads) pages_reserve_kernel(const __grid_constant__ PageArgs a, const int32_t* n_new,
                                                                     const MoveArgs m, int32_t* n_free)
{
    extern __shared__ int smem[];
    ReserveSmem& s = *reinterpret_cast<ReserveSmem*>(smem);
    uint32_t* bits = reinterpret_cast<uint32_t*>(smem + (sizeof(ReserveSmem) + 3) / 4);
    pdl_enter();
    const int b = threadIdx.x, rank = static_cast<int>(cluster_rank());
    for (int i = b; i < kHash; i += kPlanThreads) {
        s.page[i] = -1;
        s.writers[i] = 0;
        s.lowest[i] = kKvMaxSeqs;
    }
    __syncthreads();

    // this thread's row
    bool writes = false, bad = false;
    int first = 0, last = 0, tail = -1, count = 0, slot = -1;
    PageRow r{0, 0, true};
    if (b < a.n_seqs) {
        r = page_row(a, b);
        const int add = n_new[b];
        const int64_t end = static_cast<int64_t>(r.len) + add;
        bad = !r.ok || add < 0 ||
              end > min(static_cast<int64_t>(a.max_pages) * a.page_size, static_cast<int64_t>(kKvMaxPositions));
        writes = !bad && add > 0;
        if (writes) {
            const int32_t* row = a.table + static_cast<int64_t>(b) * a.max_pages;
            first = r.len / a.page_size;
            last = static_cast<int>((end + a.page_size - 1) / a.page_size);
            int c = first;
            if (r.len % a.page_size) {
                tail = row[c++];
                if (in_pool(a, tail)) count = a.refs[tail];
                bad = count < 1;
            }
            for (; c < min(r.held, last); ++c) {       // held ahead: has to be its own
                const int e = row[c];
                bad = bad || !in_pool(a, e) || a.refs[e] != 1;
            }
            writes = !bad;
        }
    }
    if (bad && rank == 0) set_device_status(a.status, QG_ERR_INVALID_ARG);
    if (writes && count > 1) {
        slot = (tail * 0x9E3779B1u) >> 21;             // the upper 11 bits of the product
        for (;;) {
            const int was = atomicCAS(&s.page[slot], -1, tail);
            if (was == -1 || was == tail) break;
            slot = (slot + 1) & (kHash - 1);
        }
        atomicAdd(&s.writers[slot], 1);
        atomicMin(&s.lowest[slot], b);
    }
    __syncthreads();
    const bool replaced = slot >= 0 && !(s.writers[slot] == count && s.lowest[slot] == b);
    const int fresh = writes ? max(0, last - r.held) : 0;
    int64_t total, moves;
    const int64_t before = block_scan<int64_t>(static_cast<int64_t>(fresh) + replaced, s.sums, total);
    const int64_t at = block_scan<int64_t>(replaced, s.sums, moves);
    s.off[b] = static_cast<int>(before);               // exact where it is used: total <= the pool's pages
    s.first[b] = replaced ? first : -1;
    s.held[b] = r.held;
    s.tail[b] = tail;
    s.tokens[b] = writes ? r.len % a.page_size : 0;
    s.move[b] = static_cast<int>(at);
    if (b == 0) s.off[kKvMaxSeqs] = static_cast<int>(total);

    // this block's share of the pool
    const Share sh = share_of(a);
    scan_refs(a, sh.word0, sh.words, true, bits);
    int mine = 0;
    for (int w = sh.from; w < sh.to; ++w) mine += __popc(bits[w]);
    int64_t block_free;
    int k = static_cast<int>(block_scan<int64_t>(mine, s.sums, block_free));
    if (b == 0) s.count = static_cast<int>(block_free);
    cluster_sync();
    int64_t free_pages = 0;
    for (int x = 0; x < static_cast<int>(cluster_size()); ++x) {
        const int v = cluster_word(&s.count, x);
        if (x < rank) k += v;
        free_pages += v;
    }
    const bool enough = total <= free_pages;
    if (rank == 0) {
        if (b == 0) {
            *m.count = enough ? static_cast<int>(moves) : 0;
            if (n_free) *n_free = static_cast<int>(max(free_pages - total, static_cast<int64_t>(-0x7FFFFFFF)));
        }
        if (enough && writes) a.held[b] = max(r.held, last);
        if (enough && replaced) atomicSub(&a.refs[tail], 1);
    }
    if (enough) {
        for (int w = sh.from; w < sh.to && k < total; ++w)
            for (uint32_t x = bits[w]; x && k < total; x &= x - 1, ++k) {
                const int page = (sh.word0 + w) * 32 + __ffs(x) - 1;
                int lo = 0, hi = kKvMaxSeqs;           // the last row with off <= k has the page
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (s.off[mid] <= k) lo = mid;
                    else hi = mid;
                }
                const int local = k - s.off[lo], c = s.first[lo];
                const bool copy = c >= 0 && local == 0;
                const int col = copy ? c : s.held[lo] + local - (c >= 0);
                a.table[static_cast<int64_t>(lo) * a.max_pages + col] = page;
                a.refs[page] = 1;
                if (copy) m.list[s.move[lo]] = make_int4(s.tail[lo], page, s.tokens[lo], 0);
            }
    }
    cluster_sync();                                    // no block leaves while another reads its count
}

// ------------------------------------------------------------------ compact
struct CompactSmem {
    int64_t sums[32];
    int live;
    int holes;
    int movers;
};

// One cluster. Of L pages in use, those at L and above move into the free
// places below L: as many of one as of the other. A block counts the holes of
// the blocks before it and the movers of those behind it.
__global__ void __launch_bounds__(kPlanThreads) pages_compact_kernel(const __grid_constant__ PageArgs a, const MoveArgs m,
                                                                     int32_t* page_map, int32_t* n_live)
{
    extern __shared__ int smem[];
    CompactSmem& s = *reinterpret_cast<CompactSmem*>(smem);
    uint32_t* bits = reinterpret_cast<uint32_t*>(smem + (sizeof(CompactSmem) + 3) / 4);
    pdl_enter();
    const int tid = threadIdx.x, rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
    const Share sh = share_of(a);
    scan_refs(a, sh.word0, sh.words, false, bits);
    int mine = 0;
    for (int w = sh.from; w < sh.to; ++w) mine += __popc(bits[w]);
    int64_t all;
    block_scan<int64_t>(mine, s.sums, all);
    if (tid == 0) s.live = static_cast<int>(all);
    cluster_sync();
    int live = 0;
    for (int x = 0; x < size; ++x) live += cluster_word(&s.live, x);
    // bits of a word for pages below L
    auto below = [&](int w) {
        const int64_t n = live - static_cast<int64_t>(sh.word0 + w) * 32;
        return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
    };
    int holes = 0, movers = 0;
    for (int w = sh.from; w < sh.to; ++w) {
        holes += __popc(~bits[w] & below(w));
        movers += __popc(bits[w] & ~below(w));
    }
    int64_t block_holes, block_movers;
    int hole = static_cast<int>(block_scan<int64_t>(holes, s.sums, block_holes));
    const int64_t movers_before = block_scan<int64_t>(movers, s.sums, block_movers);
    int mover = static_cast<int>(block_movers - movers_before) - movers;    // movers of the threads behind
    if (tid == 0) {
        s.holes = static_cast<int>(block_holes);
        s.movers = static_cast<int>(block_movers);
    }
    cluster_sync();
    int n = 0;
    for (int x = 0; x < size; ++x) {
        const int h = cluster_word(&s.holes, x);
        if (x < rank) hole += h;
        if (x > rank) mover += cluster_word(&s.movers, x);
        n += h;
    }
    n = min(n, m.capacity);
    if (rank == 0 && tid == 0) {
        *m.count = n;
        if (n_live) *n_live = live;
    }
    for (int i = tid; i < sh.words * 32; i += kPlanThreads) {
        const int page = sh.word0 * 32 + i;
        if (page < a.num_pages) page_map[page] = bits[i / 32] >> (i & 31) & 1u ? page : -1;
    }
    for (int w = sh.from; w < sh.to && hole < n; ++w)
        for (uint32_t x = ~bits[w] & below(w); x && hole < n; x &= x - 1, ++hole)
            m.list[hole].y = (sh.word0 + w) * 32 + __ffs(x) - 1;
    cluster_sync();
    for (int w = sh.to - 1; w >= sh.from && mover < n; --w)
        for (uint32_t x = bits[w] & ~below(w); x && mover < n; ++mover) {
            const int bit = 31 - __clz(x);
            x ^= 1u << bit;
            const int page = (sh.word0 + w) * 32 + bit, to = __ldcg(&m.list[mover].y);
            m.list[mover] = make_int4(page, to, a.page_size, 0);
            a.refs[to] = a.refs[page];
            a.refs[page] = 0;
            page_map[page] = to;
        }
}

// The entries in use, through the map.
__global__ void __launch_bounds__(kTableThreads) pages_table_kernel(const __grid_constant__ PageArgs a, const int32_t* page_map)
{
    pdl_enter();
    const int b = blockIdx.y;
    const PageRow r = page_row(a, b);
    if (!r.ok && blockIdx.x == 0 && threadIdx.x == 0) set_device_status(a.status, QG_ERR_INVALID_ARG);
    for (int c = blockIdx.x * kTableThreads + threadIdx.x; c < r.held; c += gridDim.x * kTableThreads) {
        int32_t* e = a.table + static_cast<int64_t>(b) * a.max_pages + c;
        const int was = *e, to = in_pool(a, was) ? page_map[was] : -1;
        if (to < 0)
            set_device_status(a.status, QG_ERR_INVALID_ARG);
        else if (to != was)
            *e = to;
    }
}

// ------------------------------------------------------------------ copy
// n consecutive bytes of each head (heads `stride` bytes apart) from one page
// to another, pieces of sizeof(T); this warp's pieces are first + lane, 32 on
// at a time, up to `end`.
template <typename T, int U>
__device__ __forceinline__ void copy_pieces(const uint8_t* src, uint8_t* dst, int64_t stride, int64_t n, int64_t first, int64_t end)
{
    const uint32_t per = static_cast<uint32_t>(n / static_cast<int64_t>(sizeof(T)));
    for (int64_t x0 = first + (threadIdx.x & 31); x0 < end; x0 += 32 * U) {
        T v[U];
        int64_t at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t x = x0 + 32 * u;
            if (x < end) {
                const uint32_t head = static_cast<uint32_t>(x) / per, off = static_cast<uint32_t>(x) % per;
                at[u] = head * stride + off * static_cast<int64_t>(sizeof(T));
                v[u] = *reinterpret_cast<const T*>(src + at[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (x0 + 32 * u < end) *reinterpret_cast<T*>(dst + at[u]) = v[u];
    }
}

// A warp takes an item: a run of a move's codes, or of its scales, of one side.
__global__ void __launch_bounds__(32 * kCopyWarps) pages_copy_kernel(const __grid_constant__ KvArgs a, const MoveArgs m,
                                                                     int code_items, int scale_items)
{
    pdl_enter();
    const int count = *m.count;
    if (count < 0 || count > m.capacity) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_device_status(a.status, QG_ERR_INVALID_ARG);
        return;
    }
    const int per_side = code_items + scale_items, per_move = 2 * per_side;
    const int rb = kv_row_bytes(a.fmt, a.dim), sb = kv_scale_bytes(a.fmt, a.dim);
    const int64_t total = static_cast<int64_t>(count) * per_move;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kCopyWarps;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5); i < total; i += step) {
        const int move = static_cast<int>(i / per_move);
        int item = static_cast<int>(i % per_move);
        const int kv = item >= per_side;
        item -= kv * per_side;
        const int4 e = m.list[move];
        if (static_cast<unsigned>(e.x) >= static_cast<unsigned>(a.num_pages) ||
            static_cast<unsigned>(e.y) >= static_cast<unsigned>(a.num_pages) || e.z < 0 || e.z > a.page_size) {
            set_device_status(a.status, QG_ERR_INVALID_ARG);
            continue;
        }
        if (e.z == 0) continue;
        const bool scales = item >= code_items;
        const int unit = scales ? sb : rb;
        uint8_t* base = scales ? a.scales[kv] : a.codes[kv];
        const int64_t stride = static_cast<int64_t>(a.page_size) * unit, page = stride * a.heads;
        const int64_t n = static_cast<int64_t>(e.z) * unit, all = n * a.heads;
        const uint8_t* src = base + e.x * page;
        uint8_t* dst = base + e.y * page;
        const int64_t chunk = scales ? kScaleChunk : 32 * 16 * kCopyPieces;
        const int64_t first = (scales ? item - code_items : item) * chunk, end = min(first + chunk, all);
        if (first >= end) continue;
        if (n % 16 == 0)
            copy_pieces<uint4, kCopyPieces>(src, dst, stride, n, first / 16, end / 16);
        else if (n % 4 == 0)
            copy_pieces<uint32_t, kCopyPieces>(src, dst, stride, n, first / 4, end / 4);
        else
            copy_pieces<uint8_t, kCopyPieces>(src, dst, stride, n, first, end);
    }
}

// ------------------------------------------------------------------ launches
constexpr int kPlanSmemMax = 160 << 10;

// One block scans a small pool, a cluster of eight a large one.
int plan_blocks(const PageArgs& a) { return a.num_pages > 8192 ? 8 : 1; }

size_t plan_smem(const PageArgs& a, size_t fixed)
{
    const int words = (a.num_pages + 31) / 32, blocks = plan_blocks(a);
    return (fixed + 3) / 4 * 4 + static_cast<size_t>((words + blocks - 1) / blocks) * 4;
}

bool allow_smem(const void* kern, bool (&set)[64])
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanSmemMax) != cudaSuccess) return false;
        set[dev] = true;
    }
    return true;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), int blocks, size_t smem, cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(blocks);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

bool with_status(const PageArgs& in, PageArgs& a)
{
    a = in;
    a.status = device_status_ptr();
    return a.status != nullptr;
}

}  // namespace

qg_status launch_pages_fork(const PageArgs& in, const int32_t* parent, cudaStream_t stream)
{
    static bool set[64] = {};
    PageArgs a;
    if (!with_status(in, a) || !allow_smem(reinterpret_cast<const void*>(pages_fork_kernel), set)) return QG_ERR_CUDA;
    const size_t smem = static_cast<size_t>(a.n_seqs) * (4 + kForkCols) * 4;
    cudaError_t e = launch_pdl(pages_fork_kernel, dim3(static_cast<unsigned>((a.max_pages - 1) / kForkCols + 1)),
                               dim3(kForkThreads), smem, stream, a, parent);
    if (e == cudaSuccess) e = launch_pdl(pages_fork_rows_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a, parent);
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

qg_status launch_pages_reserve(const PageArgs& in, const int32_t* n_new, const MoveArgs& m, int32_t* n_free,
                               cudaStream_t stream)
{
    static bool set[64] = {};
    PageArgs a;
    if (!with_status(in, a) || !allow_smem(reinterpret_cast<const void*>(pages_reserve_kernel), set)) return QG_ERR_CUDA;
    const cudaError_t e = launch_cluster(pages_reserve_kernel, plan_blocks(a), plan_smem(a, sizeof(ReserveSmem)), stream,
                                         a, n_new, m, n_free);
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

qg_status launch_pages_compact(const PageArgs& in, const MoveArgs& m, int32_t* page_map, int32_t* n_live,
                               cudaStream_t stream)
{
    static bool set[64] = {};
    PageArgs a;
    if (!with_status(in, a) || !allow_smem(reinterpret_cast<const void*>(pages_compact_kernel), set)) return QG_ERR_CUDA;
    cudaError_t e = launch_cluster(pages_compact_kernel, plan_blocks(a), plan_smem(a, sizeof(CompactSmem)), stream, a, m,
                                   page_map, n_live);
    if (e == cudaSuccess && a.n_seqs) {
        const int blocks = min((a.max_pages - 1) / kTableThreads + 1, 64);
        e = launch_pdl(pages_table_kernel, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(a.n_seqs)),
                       dim3(kTableThreads), 0, stream, a, static_cast<const int32_t*>(page_map));
    }
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

qg_status launch_pages_copy(const KvArgs& in, const MoveArgs& m, cudaStream_t stream)
{
    KvArgs a = in;
    a.status = device_status_ptr();
    if (!a.status) return QG_ERR_CUDA;
    const int64_t rows = static_cast<int64_t>(a.heads) * a.page_size;
    const int64_t code = 32 * 16 * kCopyPieces;
    const int code_items = static_cast<int>((rows * kv_row_bytes(a.fmt, a.dim) + code - 1) / code);
    const int scale_items = static_cast<int>((rows * kv_scale_bytes(a.fmt, a.dim) + kScaleChunk - 1) / kScaleChunk);
    const int64_t warps = static_cast<int64_t>(m.capacity) * 2 * (code_items + scale_items);
    const int64_t blocks = min((warps + kCopyWarps - 1) / kCopyWarps, static_cast<int64_t>(sm_count(-1)) * 8);
    const cudaError_t e = launch_pdl(pages_copy_kernel, dim3(static_cast<unsigned>(blocks)), dim3(32 * kCopyWarps), 0,
                                     stream, a, m, code_items, scale_items);
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

}  // namespace qg

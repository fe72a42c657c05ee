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

constexpr int kForkThreads = 1024, kForkCols = 8, kForkAhead = 4;
constexpr int kFewThreads = 512, kFewRows = 16, kFewCols = 64;
constexpr int kPlanThreads = 1024;
constexpr int kTableThreads = 256;
constexpr int kHash = 2048;
constexpr int kCopyWarps = 8, kCopyParts = 16;
constexpr int kBulkChunk = 16 << 10, kBulkStages = 4, kBulkAhead = 2, kBulkBlocks = 2, kBulkLeast = 4 << 10;

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

// ------------------------------------------------------------------ clusters
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
    if (cluster_size() == 1) __syncthreads();
    else asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// ------------------------------------------------------------------ fork
// A block takes kForkCols columns of the whole table: every row's entries go
// to shared memory first, so that rows may be permuted in place. An entry of
// old row j is held by kids[j] rows afterwards (by none behind the page of the
// row's last token) and was held once: refs changes by the difference. A page
// that the rows of a prompt share stands in one column of rows next to each
// other: what it changes by is added up over a warp's four rows first, which
// for beams that go on from each other is often nothing. Bound by chained
// loads (lengths, then entries, 32 bytes of a row) and the second launch: 1,024
// rows of 2,048 entries in 12.3 us where two of every four rows go on and in
// 12.5 where the best few of 16 have most children (blocks of 32 columns with
// an atomic for each entry: 50).
__global__ void __launch_bounds__(kForkThreads, 2) pages_fork_kernel(const __grid_constant__ PageArgs a, const int32_t* parent)
{
    extern __shared__ int smem[];
    pdl_enter();
    const int n = a.n_seqs, tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * kForkCols;
    int* par = smem;
    int* keep = par + n;
    int* held = keep + n;
    int* kids = held + n;
    int* slab = kids + n;
    for (int i = tid; i < n; i += threads) kids[i] = 0;
    __syncthreads();
    int most = 0;
    for (int i = tid; i < n; i += threads) {
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
    if (__syncthreads_or(most > col0) == 0) return;
    const int64_t c = col0 + tid % kForkCols;
    const int row0 = tid / kForkCols, step = threads / kForkCols;
    for (int j0 = row0; j0 - lane / 8 < n; j0 += kForkAhead * step) {        // the same for a whole warp
        int e[kForkAhead];
#pragma unroll
        for (int u = 0; u < kForkAhead; ++u) {
            const int j = j0 + u * step;
            if (j < n && c < held[j]) e[u] = a.table[static_cast<int64_t>(j) * a.max_pages + c];
        }
#pragma unroll
        for (int u = 0; u < kForkAhead; ++u) {
            const int j = j0 + u * step;
            int page = -1, change = 0;
            if (j < n && c < held[j]) {
                slab[j * kForkCols + tid % kForkCols] = e[u];
                if (in_pool(a, e[u])) {
                    page = e[u];
                    change = (c < keep[j] ? kids[j] : 0) - 1;
                } else {
                    set_device_status(a.status, QG_ERR_INVALID_ARG);
                }
            }
            // the sum over a run goes to its first row's lane
            const int up = __shfl_up_sync(0xffffffffu, page, 8), next = __shfl_down_sync(0xffffffffu, page, 8);
            const int after = __shfl_down_sync(0xffffffffu, page, 16), more = __shfl_down_sync(0xffffffffu, change, 8);
            if (lane < 24 && next == page) change += more;
            const int rest = __shfl_down_sync(0xffffffffu, change, 16);
            if (lane < 16 && next == page && after == page) change += rest;
            if (page >= 0 && (lane < 8 || up != page) && change) atomicAdd(&a.refs[page], change);
        }
    }
    __syncthreads();
    for (int i = row0; i < n; i += step) {
        const int p = par[i];
        if (p < 0 || p == i || c >= keep[p]) continue;
        a.table[static_cast<int64_t>(i) * a.max_pages + c] = slab[p * kForkCols + tid % kForkCols];
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

// Few rows: one launch, of a cluster whose blocks have all read the lengths
// before one of them writes any. 8 rows of 257 entries in 2.3 us, 16 in 2.8 (by
// the two launches above 3.5 and 3.6); for 32 rows both take 3.7. Beyond 512
// columns a block has several runs of them: 8 rows of 1,028 entries 3.0 us (by
// the two launches 3.6), 16 rows 3.9 (3.7), 8 rows of 2,052 4.4 (3.6).
__global__ void __launch_bounds__(kFewThreads) pages_fork_few_kernel(const __grid_constant__ PageArgs a, const int32_t* parent)
{
    __shared__ int par[kFewRows], keep[kFewRows], held[kFewRows], kids[kFewRows], lens[kFewRows];
    __shared__ int slab[kFewRows][kFewCols];
    __shared__ int most;
    pdl_enter();
    const int n = a.n_seqs, tid = threadIdx.x, rank = static_cast<int>(cluster_rank());
    if (tid < n) kids[tid] = 0;
    if (tid == 0) most = 0;
    __syncthreads();
    if (tid < n) {
        bool bad;
        const PageRow r = page_row(a, tid);
        const int p = parent_of(a, parent, tid, bad);
        if (rank == 0 && (bad || !r.ok)) set_device_status(a.status, QG_ERR_INVALID_ARG);
        par[tid] = p;
        keep[tid] = (r.len + a.page_size - 1) / a.page_size;
        held[tid] = r.held;
        lens[tid] = r.len;
        atomicMax(&most, r.held);
        if (p >= 0) atomicAdd(&kids[p], 1);
    }
    cluster_sync();
    if (rank == 0 && tid < n) {
        const int p = par[tid];
        a.lens[tid] = p < 0 ? 0 : lens[p];
        a.held[tid] = p < 0 ? 0 : keep[p];
    }
    const int col = tid % kFewCols, step = kFewThreads / kFewCols;
    for (int c = rank * kFewCols + col; c - col < most; c += static_cast<int>(cluster_size()) * kFewCols) {
#pragma unroll 4
        for (int j = tid / kFewCols; j < n; j += step) {
            if (c >= held[j]) continue;
            const int e = a.table[static_cast<int64_t>(j) * a.max_pages + c];
            slab[j][col] = e;
            const int change = (c < keep[j] ? kids[j] : 0) - 1;
            if (!in_pool(a, e)) set_device_status(a.status, QG_ERR_INVALID_ARG);
            else if (change) atomicAdd(&a.refs[e], change);
        }
        __syncthreads();
        for (int i = tid / kFewCols; i < n; i += step) {
            const int p = par[i];
            if (p < 0 || p == i || c >= keep[p]) continue;
            a.table[static_cast<int64_t>(i) * a.max_pages + c] = slab[p][col];
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ scans over the pool
// The word at `p` of this block's shared memory in block `rank` of the cluster.
__device__ __forceinline__ int cluster_word(const int* p, uint32_t rank)
{
    uint32_t at;
    int v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// Sums over a warp up to each lane, and of the warps before this one: a barrier
// lies between the two, which several numbers share. Each scan of a kernel has
// its own warp_sums.
template <typename T>
__device__ __forceinline__ T warp_scan(T v)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

template <typename T>
__device__ __forceinline__ T before_warp(const T* warp_sums, T& total)
{
    const int warp = threadIdx.x >> 5;
    const T s = warp_scan(warp_sums[threadIdx.x & 31]);
    total = __shfl_sync(0xffffffffu, s, 31);
    const T before = __shfl_sync(0xffffffffu, s, warp ? warp - 1 : 0);
    return warp ? before : T(0);
}

// Sum over the block of v, and what the threads before this one have.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total)
{
    const int x = warp_scan(v);
    if ((threadIdx.x & 31) == 31) warp_sums[threadIdx.x >> 5] = x;
    __syncthreads();
    return x - v + before_warp(warp_sums, total);
}

// The counts of four pages of a thread, 0 behind the pool.
struct RefsLoad {
    int4 r;

    __device__ __forceinline__ RefsLoad(const PageArgs& a, int word0, int words, int base)
    {
        const int at = base + 4 * static_cast<int>(threadIdx.x);
        const int64_t p = static_cast<int64_t>(word0) * 32 + at;
        r = int4{};
        if (at >= words * 32) return;
        if (p + 4 <= a.num_pages) {
            r = *reinterpret_cast<const int4*>(a.refs + p);
        } else {
            if (p < a.num_pages) r.x = a.refs[p];
            if (p + 1 < a.num_pages) r.y = a.refs[p + 1];
            if (p + 2 < a.num_pages) r.z = a.refs[p + 2];
        }
    }
};

// A block's share of the pool, `words` words of 32 pages from word `word0` on:
// bit i of a word is set for a page that is held (free_bits: that is free).
// Pages behind the pool have bit 0. `ahead`: the first counts, loaded before.
__device__ __forceinline__ void scan_refs(const PageArgs& a, int word0, int words, bool free_bits, uint32_t* bits, RefsLoad ahead)
{
    const int lane = threadIdx.x & 31;
    const int64_t first = static_cast<int64_t>(word0) * 32;
    for (int base = 0; base < words * 32; base += 4 * kPlanThreads) {
        const int at = base + 4 * static_cast<int>(threadIdx.x);
        const int4 r = ahead.r;
        if (base + 4 * kPlanThreads < words * 32) ahead = RefsLoad(a, word0, words, base + 4 * kPlanThreads);
        uint32_t nib = (r.x != 0) | (r.y != 0) << 1 | (r.z != 0) << 2 | (r.w != 0) << 3;
        if (free_bits) {
            const int64_t left = a.num_pages - first - at;
            nib = ~nib & (left >= 4 ? 15u : left <= 0 ? 0u : (1u << left) - 1u);
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

__device__ __forceinline__ int share_words(const PageArgs& a)
{
    return ((a.num_pages + 31) / 32 + static_cast<int>(cluster_size()) - 1) / static_cast<int>(cluster_size());
}

__device__ __forceinline__ Share share_of(const PageArgs& a)
{
    Share s;
    const int all = (a.num_pages + 31) / 32, each = share_words(a);
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
    int64_t row_sums[32];
    int page_sums[32];
    int count;
};

// One cluster. Each block looks at every row (thread b at row b) and at its
// share of the pool; with the free pages of the blocks before it, it knows the
// number that each of its free pages has among all, and so the row and the
// column that each is for. Nothing is written before every block has read.
// Bound by chained loads and barriers (a row's length, last entry and count of
// that page; two scans; the cluster's sum): 8 rows of a step in 5.0 us, 10.2 for
// 64 rows and 21,000 pages of a pool of 100,000. Of some 18,000 cycles of the
// latter the pool's bits and the rows take 4,800, the scans 2,200, the cluster's
// barrier 1,400, its blocks' counts, read one after another, 3,100, and the
// pages handed out 6,300. 32 pages held ahead by each row cost 1.9 us: a row's
// thread looks at one after another.
__global__ void __launch_bounds__(kPlanThreads, 1) pages_reserve_kernel(const __grid_constant__ PageArgs a, const int32_t* n_new,
                                                                     const MoveArgs m, int32_t* n_free)
{
    extern __shared__ int smem[];
    ReserveSmem& s = *reinterpret_cast<ReserveSmem*>(smem);
    uint32_t* bits = reinterpret_cast<uint32_t*>(smem + (sizeof(ReserveSmem) + 3) / 4);
    int* before_word = reinterpret_cast<int*>(bits) + share_words(a);
    pdl_enter();
    const int b = threadIdx.x, rank = static_cast<int>(cluster_rank());
    const Share sh = share_of(a);
    const RefsLoad ahead(a, sh.word0, sh.words, 0);
    // this thread's row, on its way while the free pages are looked for
    PageRow r{0, 0, true};
    int add = 0;
    if (b < a.n_seqs) {
        r = page_row(a, b);
        add = n_new[b];
    }
    for (int i = b; i < kHash; i += kPlanThreads) {
        s.page[i] = -1;
        s.writers[i] = 0;
        s.lowest[i] = kKvMaxSeqs;
    }
    scan_refs(a, sh.word0, sh.words, true, bits, ahead);
    int mine = 0;
    for (int w = sh.from; w < sh.to; ++w) mine += __popc(bits[w]);

    bool writes = false, bad = false;
    int first = 0, last = 0, tail = -1, count = 0, slot = -1;
    if (b < a.n_seqs) {
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
    // new pages (at most 2^26 + 1 of a row), and in the lower 11 bits replaced ones (at most 2^10)
    const int64_t want = (static_cast<int64_t>(fresh) + replaced) << 11 | replaced;
    const int64_t rows_to = warp_scan(want);
    const int pages_to = warp_scan(mine);
    if ((b & 31) == 31) {
        s.row_sums[b >> 5] = rows_to;
        s.page_sums[b >> 5] = pages_to;
    }
    __syncthreads();
    int64_t both;
    int block_free;
    const int64_t before = rows_to - want + before_warp(s.row_sums, both);
    int k = pages_to - mine + before_warp(s.page_sums, block_free);
    const int64_t total = both >> 11;
    const int moves = static_cast<int>(both & 2047);
    s.off[b] = static_cast<int>(before >> 11);         // exact where it is used: total <= the pool's pages
    s.first[b] = replaced ? first : -1;
    s.held[b] = r.held;
    s.tail[b] = tail;
    s.tokens[b] = writes ? r.len % a.page_size : 0;
    s.move[b] = static_cast<int>(before & 2047);
    if (b == 0) s.off[kKvMaxSeqs] = static_cast<int>(total);

    if (b == 0) s.count = block_free;
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
            *m.count = enough ? moves : 0;
            if (n_free) *n_free = static_cast<int>(max(free_pages - total, static_cast<int64_t>(-0x7FFFFFFF)));
            else if (!enough) set_device_status(a.status, QG_ERR_INVALID_ARG);       // nobody would hear of it
        }
        if (enough && writes) a.held[b] = max(r.held, last);
        if (enough && replaced) atomicSub(&a.refs[tail], 1);
    }
    if (enough) {
        for (int w = sh.from; w < sh.to; ++w) {
            before_word[w] = k;
            k += __popc(bits[w]);
        }
        __syncthreads();
        // a thread per four pages, a warp per 128: the row of its first one is looked for by all lanes, the lanes' own
        // follow soon
        const int lane = b & 31;
        for (int i0 = b - lane; i0 < 8 * sh.words; i0 += kPlanThreads) {
            const int i = i0 + lane;
            const bool in = i < 8 * sh.words;
            const uint32_t word = in ? bits[i / 8] : 0u, low = 4 * (i % 8);
            k = in ? before_word[i / 8] + __popc(word & ((1u << low) - 1u)) : INT32_MAX;
            const int k0 = __shfl_sync(0xffffffffu, k, 0);
            if (k0 >= total) break;
            const int part = __popc(__ballot_sync(0xffffffffu, s.off[32 * lane] <= k0)) - 1;
            int lo = 32 * part + __popc(__ballot_sync(0xffffffffu, s.off[32 * part + lane] <= k0)) - 1;
            int next = s.off[lo + 1], col = 0;
            int32_t* row = nullptr;
            for (uint32_t x = word & 15u << low; x && k < total; x &= x - 1, ++k) {
                const int page = (sh.word0 + i / 8) * 32 + __ffs(x) - 1;
                if (!row || k >= next) {               // the last row with off <= k; off[kKvMaxSeqs] = total
                    while (k >= next) next = s.off[++lo + 1];
                    row = a.table + static_cast<int64_t>(lo) * a.max_pages;
                    const int local = k - s.off[lo], c = s.first[lo];
                    col = s.held[lo] + local - (c >= 0);
                    if (c >= 0 && local == 0) {        // the one that is replaced comes before new ones
                        row[c] = page;
                        m.list[s.move[lo]] = make_int4(s.tail[lo], page, s.tokens[lo], 0);
                        a.refs[page] = 1;
                        ++col;
                        continue;
                    }
                }
                row[col++] = page;
                a.refs[page] = 1;
            }
        }
    }
    cluster_sync();                                    // no block leaves while another reads its count
}

// ------------------------------------------------------------------ compact
struct CompactSmem {
    int sums[32];
    int live;
    int holes;
};

// One cluster. Of L pages in use, those at L and above move into the free
// places below L: as many of one as of the other. With S(p) pages in use below
// page p, a free one below L is hole number p - S(p), and one in use from L on
// is number L - 1 - S(p) of those that move, counted from the highest: 46,000
// pages in use of 92,000, half of them moved, in 14.5 us with the table. Of some
// 22,000 cycles before the table, bits and scan take 2,800, the first barrier
// 1,700, the blocks' counts, read one after another, twice 3,100, the map and
// the list with the barrier that waits for them 8,500, and the moves 1,100 to
// 3,000.
__global__ void __launch_bounds__(kPlanThreads) pages_compact_kernel(const __grid_constant__ PageArgs a, const MoveArgs m,
                                                                     int32_t* page_map, int32_t* n_live)
{
    extern __shared__ int smem[];
    CompactSmem& s = *reinterpret_cast<CompactSmem*>(smem);
    uint32_t* bits = reinterpret_cast<uint32_t*>(smem + (sizeof(CompactSmem) + 3) / 4);
    int* before_word = reinterpret_cast<int*>(bits) + share_words(a);
    pdl_enter();
    const int tid = threadIdx.x, rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
    const Share sh = share_of(a);
    scan_refs(a, sh.word0, sh.words, false, bits, RefsLoad(a, sh.word0, sh.words, 0));
    int mine = 0;
    for (int w = sh.from; w < sh.to; ++w) mine += __popc(bits[w]);
    int all, below = block_scan(mine, s.sums, all);
    if (tid == 0) {
        s.live = all;
        s.holes = 0;
    }
    cluster_sync();
    int live = 0;
    for (int x = 0; x < size; ++x) {
        const int v = cluster_word(&s.live, x);
        if (x < rank) below += v;
        live += v;
    }
    for (int w = sh.from; w < sh.to; ++w) {
        before_word[w] = below;
        below += __popc(bits[w]);
    }
    __syncthreads();
    // a thread per four pages: the map, places and pages of the list
    for (int i = tid; i < 8 * sh.words; i += kPlanThreads) {
        const uint32_t word = bits[i / 8], low = 4 * (i % 8);
        const int page0 = (sh.word0 + i / 8) * 32 + static_cast<int>(low);
        int under = before_word[i / 8] + __popc(word & ((1u << low) - 1u)), map[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int page = page0 + k;
            const bool used = word >> (low + k) & 1u;
            map[k] = used ? page : -1;
            if (page == live) s.holes = live - under;
            if (!used && page < live && page - under < m.capacity) m.list[page - under].y = page;
            if (used && page >= live && live - 1 - under < m.capacity) m.list[live - 1 - under].x = page;
            under += used;
        }
        if (page0 + 4 <= a.num_pages)
            *reinterpret_cast<int4*>(page_map + page0) = make_int4(map[0], map[1], map[2], map[3]);
        else
            for (int k = 0; page0 + k < a.num_pages; ++k) page_map[page0 + k] = map[k];
    }
    cluster_sync();
    int n = 0;                                         // known to the block that has page L; none if all pages are in use
    for (int x = 0; x < size; ++x) n = max(n, cluster_word(&s.holes, x));
    n = min(n, m.capacity);
    if (rank == 0 && tid == 0) {
        *m.count = n;
        if (n_live) *n_live = live;
    }
    // then the moves side by side
    constexpr int kAhead = 4;
    const int step = kPlanThreads * size;
    for (int i0 = rank * kPlanThreads + tid; i0 < n; i0 += kAhead * step) {
        int4 e[kAhead];
        int held[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (i0 + u * step < n) e[u] = __ldcg(&m.list[i0 + u * step]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (i0 + u * step < n) held[u] = __ldcg(&a.refs[e[u].x]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (i0 + u * step < n) {
                m.list[i0 + u * step] = make_int4(e[u].x, e[u].y, a.page_size, 0);
                a.refs[e[u].y] = held[u];
                a.refs[e[u].x] = 0;
                page_map[e[u].x] = e[u].y;
            }
    }
    cluster_sync();                                    // no block leaves while another reads its count
}

// The entries in use, through the map.
__global__ void __launch_bounds__(kTableThreads) pages_table_kernel(const __grid_constant__ PageArgs a, const int32_t* page_map)
{
    pdl_enter();
    const int b = blockIdx.y;
    const PageRow r = page_row(a, b);
    if (!r.ok && blockIdx.x == 0 && threadIdx.x == 0) set_device_status(a.status, QG_ERR_INVALID_ARG);
    for (int64_t c = blockIdx.x * kTableThreads + threadIdx.x; c < r.held; c += gridDim.x * kTableThreads) {
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
// to another in pieces of sizeof(T), those from `first` up to `end` by a warp.
template <typename T, int U>
__device__ __forceinline__ void copy_pieces(const uint8_t* src, uint8_t* dst, int64_t stride, int64_t n, uint32_t first, uint32_t end)
{
    const uint32_t per = static_cast<uint32_t>(n / static_cast<int64_t>(sizeof(T)));
    for (uint32_t x0 = first + (threadIdx.x & 31); x0 < end; x0 += 32 * U) {
        T v[U];
        int64_t at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t x = x0 + 32 * u;
            if (x < end) {
                at[u] = x / per * stride + x % per * static_cast<int64_t>(sizeof(T));
                v[u] = *reinterpret_cast<const T*>(src + at[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (x0 + 32 * u < end) *reinterpret_cast<T*>(dst + at[u]) = v[u];
    }
}

// Share `part` of `parts` of what a move copies of one side's codes or
// scales, `unit` bytes a token and head.
__device__ __noinline__ void copy_part(const KvArgs& a, uint8_t* base, int unit, const int4& e, int part, int parts)
{
    const int64_t stride = static_cast<int64_t>(a.page_size) * unit, page = stride * a.heads;
    const int64_t n = static_cast<int64_t>(e.z) * unit;
    const uint8_t* src = base + e.x * page;
    uint8_t* dst = base + e.y * page;
    auto share = [&](uint32_t size, uint32_t& first, uint32_t& end) {          // in whole warps' pieces
        const uint32_t all = static_cast<uint32_t>(n * a.heads / size), each = (all + 32 * parts - 1) / (32 * parts) * 32;
        first = min(part * each, all);
        end = min(first + each, all);
    };
    uint32_t first, end;
    if (n % 16 == 0) {
        share(16, first, end);
        copy_pieces<uint4, 4>(src, dst, stride, n, first, end);
    } else if (n % 4 == 0) {
        share(4, first, end);
        copy_pieces<uint32_t, 4>(src, dst, stride, n, first, end);
    } else {
        share(1, first, end);
        copy_pieces<uint8_t, 4>(src, dst, stride, n, first, end);
    }
}

// Entry `move` of the list, checked; without tokens where it does not fit.
__device__ __forceinline__ int4 move_at(const KvArgs& a, const MoveArgs& m, int move)
{
    int4 e = m.list[move];
    if (static_cast<unsigned>(e.x) >= static_cast<unsigned>(a.num_pages) ||
        static_cast<unsigned>(e.y) >= static_cast<unsigned>(a.num_pages) || e.z < 0 || e.z > a.page_size) {
        set_device_status(a.status, QG_ERR_INVALID_ARG);
        e = make_int4(0, 0, 0, 0);
    }
    return e;
}

// One warp of a block keeps kBulkAhead chunks on their way into shared memory
// and stores them from there, all with bulk copies: codes of whole pages, which
// lie next to each other, and of a head's tokens. The other warps take scales
// and what is too short for that, several to a side of a move where there are
// more warps than sides. Bound by bytes: 2,048 pages of 2 x 128 KB in 165 us,
// 6.5 TB/s read and written (with 16-byte loads and stores of all warps 192); 8
// moves of 37 fp8 tokens of 4 heads in 2.3 us. In bulk and by the warps: pages
// of 4 KB (8,192 moves of nvfp4) 39.9 and 47.5 us, 1 KB (fp8) 32.4 and 19.2;
// heads' tokens of 8 KB (1,000 moves of bf16) 27.7 and 36.8, 4.6 KB (1,000 of
// fp8) 28.8 and 32.7, 1.6 KB (2,048 of fp8) 68 and 18. Where every warp has at
// most one of the shares, tokens of 4.6 KB (8 moves of fp8) 2.8 and 2.3, 8 KB
// (64 of bf16) 4.0 and 3.7, 16 KB (8 of bf16) 2.7 and 4.4.
struct BulkChunk {
    const uint8_t* src;
    uint8_t* dst;
    uint32_t bytes;
};

__global__ void __launch_bounds__(32 * kCopyWarps, kBulkBlocks) pages_copy_kernel(const __grid_constant__ KvArgs a, const MoveArgs m, const DebugState dbg)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kBulkStages];
    const int tid = threadIdx.x;
    if (tid == 0) {
        for (int i = 0; i < kBulkStages; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
    }
    pdl_enter();
    const int count = *m.count;
    if (count < 0 || count > m.capacity) {
        if (blockIdx.x == 0 && tid == 0) set_device_status(a.status, QG_ERR_INVALID_ARG);
        return;
    }
    const int rb = kv_row_bytes(a.fmt, a.dim), sb = kv_scale_bytes(a.fmt, a.dim), sides = 2 * count;
    const int64_t stride = static_cast<int64_t>(a.page_size) * rb, page = stride * a.heads;
    const int warps = gridDim.x * (kCopyWarps - 1), least = (sides * kCopyParts > warps ? 1 : 3) * kBulkLeast;
    if (tid >= 32) {
        const int kinds = sb ? 2 : 1;
        const int parts = max(1, min(kCopyParts, warps / max(1, sides * kinds)));
        const int64_t items = static_cast<int64_t>(sides) * kinds * parts;
        for (int64_t i = blockIdx.x * (kCopyWarps - 1) + (tid >> 5) - 1; i < items; i += warps) {
            const int part = static_cast<int>(i % parts), x = static_cast<int>(i / parts), side = x / kinds;
            const int4 e = move_at(a, m, side >> 1);
            if (x % kinds) {
                if (e.z) copy_part(a, a.scales[side & 1], sb, e, part, parts);
            } else if (e.z && !(e.z == a.page_size ? page >= kBulkLeast : e.z * rb >= least)) {
                copy_part(a, a.codes[side & 1], rb, e, part, parts);
            }
        }
        return;
    }
    const int slots = static_cast<int>((page + kBulkChunk - 1) / kBulkChunk), heads = (a.heads + slots - 1) / slots;
    // A slot is a chunk of a whole page, or some heads' tokens of another. Of the block's slots, gridDim.x from each other,
    // each lane looks at one: `left` chunks of it are still to be copied, in runs of `run` bytes, `stride` from each other.
    // Lane i also has the chunk on its way that is i-th of kBulkAhead.
    const int64_t total = static_cast<int64_t>(sides) * slots;
    int64_t batch = blockIdx.x;
    uint32_t some = 0;
    BulkChunk mine{}, waiting{};
    int left = 0, run = 0, per_run = 1, sub = 0;
    int loaded = 0, stored = 0;
    uint32_t round = 0;
    for (int put = 0, got = 0;; ++stored) {
        while (loaded - stored < kBulkAhead) {
            while (!some && batch < total) {
                const int64_t at = batch + static_cast<int64_t>(tid) * gridDim.x;
                left = sub = 0;
                if (at < total) {
                    const int side = static_cast<int>(at / slots), kv = side & 1, slot = static_cast<int>(at - static_cast<int64_t>(side) * slots);
                    const int4 e = move_at(a, m, side >> 1);
                    int64_t from = static_cast<int64_t>(slot) * kBulkChunk;
                    if (e.z == a.page_size && page >= kBulkLeast) {
                        left = per_run = 1;
                        run = static_cast<int>(min(page - from, static_cast<int64_t>(kBulkChunk)));
                    } else if (e.z < a.page_size && e.z * rb >= least) {
                        run = e.z * rb;
                        per_run = (run + kBulkChunk - 1) / kBulkChunk;
                        left = max(0, min(heads, a.heads - slot * heads)) * per_run;
                        from = slot * heads * stride;
                    }
                    mine = BulkChunk{a.codes[kv] + e.x * page + from, a.codes[kv] + e.y * page + from, 0};
                }
                some = __ballot_sync(0xffffffffu, left > 0);
                batch += 32 * static_cast<int64_t>(gridDim.x);
            }
            if (!some) break;
            const int of_lane = __ffs(some) - 1;
            const int64_t off = sub / per_run * stride + sub % per_run * kBulkChunk;
            const BulkChunk c{reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine.src + off), of_lane)),
                              reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine.dst + off), of_lane)),
                              static_cast<uint32_t>(__shfl_sync(0xffffffffu, min(run - sub % per_run * kBulkChunk, kBulkChunk), of_lane))};
            if (tid == of_lane) ++sub;
            if (__shfl_sync(0xffffffffu, left - sub, of_lane) == 0) some &= some - 1;
            if (tid == 0 && !dbg.starve) {
                // the stage's last store is at least kBulkStages - kBulkAhead + 1 stores back
                if (loaded >= kBulkStages) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kBulkStages - kBulkAhead) : "memory");
                mbar_arrive_expect_tx(&full[put], c.bytes);
                bulk_load(ring + put * kBulkChunk, c.src, c.bytes, &full[put]);
            }
            if (tid == loaded % kBulkAhead) waiting = c;
            put = put + 1 == kBulkStages ? 0 : put + 1;
            ++loaded;
        }
        if (stored == loaded) break;
        const int of = stored % kBulkAhead;
        const uint64_t dst = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(waiting.dst), of);
        const uint32_t bytes = __shfl_sync(0xffffffffu, waiting.bytes, of);
        if (!__all_sync(0xffffffffu, tid || mbar_wait_bounded(&full[got], round, dbg.wait_ns, a.status))) {
            // no more is asked for; what is on its way into this block is waited for as long once more
            for (; tid == 0 && stored < loaded; ++stored) {
                mbar_wait_bounded(&full[got], round, dbg.wait_ns, a.status);
                got = got + 1 == kBulkStages ? 0 : got + 1;
                round ^= got == 0;
            }
            break;
        }
        if (tid == 0)
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\ncp.async.bulk.commit_group;" ::"l"(dst),
                         "r"(smem_u32(ring + got * kBulkChunk)), "r"(bytes)
                         : "memory");
        got = got + 1 == kBulkStages ? 0 : got + 1;
        round ^= got == 0;
    }
    if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------------ launches
constexpr int kPlanSmemMax = 192 << 10;

bool allow_smem(const void* kern, bool (&set)[64], int bytes = kPlanSmemMax)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
        set[dev] = true;
    }
    return true;
}

// One block scans a small pool, a cluster of 16 a large one, or of eight where
// the device has no room for such; 0 on an error. One block and a cluster of 16
// take, with the copy that restores the record, 8.2 and 8.9 us to reserve from
// 13,000 pages, 9.3 and 9.3 from 24,500 and 11.9 and 9.5 from 49,000; to
// compact these 10.5 and 11.1, 13.4 and 12.0, 20.4 and 12.6. 21,000 pages of
// 100,000 are handed out in 12.2 us by 16 blocks and in 14.4 by eight.
int plan_blocks(const PageArgs& a, const void* kern, int (&most)[64])
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!most[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanSmemMax) != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 16;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(kPlanThreads);
        cfg.dynamicSmemBytes = kPlanSmemMax;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int room = 0;
        const bool asked = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                           cudaOccupancyMaxActiveClusters(&room, kern, &cfg) == cudaSuccess;
        if (!asked) cudaGetLastError();
        most[dev] = asked && room > 0 ? 16 : 8;
    }
    return a.num_pages > 16384 ? most[dev] : 1;
}

size_t plan_smem(const PageArgs& a, size_t fixed, int blocks)
{
    const int words = (a.num_pages + 31) / 32;
    return (fixed + 3) / 4 * 4 + static_cast<size_t>((words + blocks - 1) / blocks) * 8;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), int blocks, size_t smem, cudaStream_t stream, int threads, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
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
    if (!with_status(in, a)) return QG_ERR_CUDA;
    if (a.n_seqs <= kFewRows && a.max_pages <= 8 * kFewCols) {
        const cudaError_t e = launch_cluster(pages_fork_few_kernel, min((a.max_pages - 1) / kFewCols + 1, 8), 0, stream, kFewThreads,
                                             a, parent);
        return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
    }
    if (!allow_smem(reinterpret_cast<const void*>(pages_fork_kernel), set)) return QG_ERR_CUDA;
    const size_t smem = static_cast<size_t>(a.n_seqs) * (4 + kForkCols) * 4;
    const int threads = min(kForkThreads, max(64, (a.n_seqs * kForkCols + 31) / 32 * 32));
    cudaError_t e = launch_pdl(pages_fork_kernel, dim3(static_cast<unsigned>((a.max_pages - 1) / kForkCols + 1)),
                               dim3(static_cast<unsigned>(threads)), smem, stream, a, parent);
    if (e == cudaSuccess) e = launch_pdl(pages_fork_rows_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a, parent);
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

qg_status launch_pages_reserve(const PageArgs& in, const int32_t* n_new, const MoveArgs& m, int32_t* n_free,
                               cudaStream_t stream)
{
    static int most[64] = {};
    PageArgs a;
    const int blocks = plan_blocks(in, reinterpret_cast<const void*>(pages_reserve_kernel), most);
    if (!blocks || !with_status(in, a)) return QG_ERR_CUDA;
    const cudaError_t e = launch_cluster(pages_reserve_kernel, blocks, plan_smem(a, sizeof(ReserveSmem), blocks), stream,
                                         kPlanThreads, a, n_new, m, n_free);
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

qg_status launch_pages_compact(const PageArgs& in, const MoveArgs& m, int32_t* page_map, int32_t* n_live,
                               cudaStream_t stream)
{
    static int most[64] = {};
    PageArgs a;
    const int blocks = plan_blocks(in, reinterpret_cast<const void*>(pages_compact_kernel), most);
    if (!blocks || !with_status(in, a)) return QG_ERR_CUDA;
    cudaError_t e = launch_cluster(pages_compact_kernel, blocks, plan_smem(a, sizeof(CompactSmem), blocks), stream,
                                   kPlanThreads, a, m, page_map, n_live);
    if (e == cudaSuccess && a.n_seqs) {
        const int wide = min((a.max_pages - 1) / kTableThreads + 1, 64);
        e = launch_pdl(pages_table_kernel, dim3(static_cast<unsigned>(wide), static_cast<unsigned>(a.n_seqs)),
                       dim3(kTableThreads), 0, stream, a, static_cast<const int32_t*>(page_map));
    }
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

qg_status launch_pages_copy(const KvArgs& in, const MoveArgs& m, cudaStream_t stream)
{
    static bool set[64] = {};
    constexpr int kSmem = kBulkStages * kBulkChunk;
    KvArgs a = in;
    a.status = device_status_ptr();
    if (!a.status || !allow_smem(reinterpret_cast<const void*>(pages_copy_kernel), set, kSmem)) return QG_ERR_CUDA;
    const cudaError_t e = launch_pdl(pages_copy_kernel, dim3(static_cast<unsigned>(kBulkBlocks * sm_count(-1))),
                                     dim3(32 * kCopyWarps), kSmem, stream, a, m, debug_state());
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

}  // namespace qg

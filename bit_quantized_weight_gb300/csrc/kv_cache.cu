// kv_cache.cu -- the paged low-precision cache of a decode step: quantise as
// it is written (kv_cache_append), read it back (kv_cache_read), keep the
// accepted path of a drafted tree (kv_cache_accept). The pages name the
// formats (NInfer article, section 4: BF16, FP8-E4M3 and NVFP4 in pages of 64
// tokens; Decapybara README, decode_ops.cu); the layouts are include/qgemv.h's.
//
// All three are bound by bytes (large calls) or by one chain of dependent
// loads (a decode step: token_start -> page table -> the row). A lane holds
// eight consecutive values of a head, 16 bytes as bf16, so that a row's lanes
// are neighbours and an amax is a few shuffles. Measured on a GB300, 4 heads of
// 128: 32,256 tokens appended in bf16 in 20 us (6.4 TB/s, 94 % of the measured
// copy rate), FP8 24 us and NVFP4 28 us (4.0 and 2.9 TB/s: instructions, mostly
// conversions), read back as bf16 in 20, 19 and 18 us (6.2, 4.9, 4.5 TB/s); a
// step of 8 lanes with 4 tokens appended in 1.9 us, a path of 4 accepted in 8
// lanes in 5 us.
#include <type_traits>

#include "kv_common.cuh"

namespace qg {
namespace {

constexpr int kWarps = 8;
constexpr int kAcceptThreads = 512;

template <int V>
using Int = std::integral_constant<int, V>;

__device__ __forceinline__ void unpack8(const uint4 r, float (&f)[8])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Nearest E4M3 / E2M1 codes, ties to even, saturating; the first argument in
// the low bits.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n cvt.u32.u8 %0, b;\n}\n"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// x / d to nearest, for eight x: with r = 1 / d to nearest and q = x r, one
// residual x - q d (exact in an fma) corrects q to the nearest quotient
// (Markstein, IBM J. Res. Dev. 34, 1990). The residual is taken as q d - x and
// given its sign in the correction: for a zero x that adds a zero of x's sign,
// so that -0 stays -0. That holds while nothing leaves the normal range: the
// largest |x|, `top`, and d lie within 2^+-60, and an x so much smaller that its
// residual is not exact is a zero code whatever its last bit. Else the division
// itself.
__device__ __forceinline__ void divide8(float (&x)[8], float d, float top)
{
    const uint32_t e = __float_as_uint(top) >> 23, ed = __float_as_uint(d) >> 23;
    if (e > 67u && e < 187u && ed > 67u && ed < 187u) {
        const float r = __frcp_rn(d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = x[i] * r;
            x[i] = fmaf(-fmaf(q, d, -x[i]), r, q);
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            // x[i] = x[i] / d without indexing registers
            float v = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) v = i == j ? x[j] : v;
            v = __fdiv_rn(v, d);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = i == j ? v : x[j];
        }
    }
}

// The largest |y|, NaN left out; and with a NaN if there is one.
__device__ __forceinline__ float max8(const float (&y)[8])
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
    return m;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The places of T consecutive rows: their pages and positions, page -2 for a
// row that has none, -1 for one whose page lies outside the cache. A row's
// sequence is the number of sequences that end at or before it, by ballots over
// 32 sequences at a time whose entries the lanes hold; two chained loads in all
// (the sequences' entries, the page table), shared by the T rows.
template <int T>
__device__ __forceinline__ void places(const KvArgs& a, int i0, int lane, int (&page)[T], int (&pos)[T])
{
    KvSeq s[T];
    int b[T];
#pragma unroll
    for (int x = 0; x < T; ++x) {
        b[x] = -1;
        s[x] = KvSeq{0, 0, 0};
    }
    for (int j = 0; j < a.n_seqs; j += 32) {
        const bool on = j + lane < a.n_seqs;
        const int row0 = on ? a.start[j + lane] : 0, end = on ? a.start[j + lane + 1] : 0x7FFFFFFF;
        const int len = on ? a.lens[j + lane] : 0;
        bool more = false;
#pragma unroll
        for (int x = 0; x < T; ++x) {
            const int n = __popc(__ballot_sync(0xffffffffu, end <= i0 + x));
            more = more || n == 32;
            const int r0 = __shfl_sync(0xffffffffu, row0, n & 31), e = __shfl_sync(0xffffffffu, end, n & 31);
            const int l = __shfl_sync(0xffffffffu, len, n & 31);
            if (b[x] >= 0 || n == 32 || j + n >= a.n_seqs) continue;
            b[x] = j + n;
            s[x] = kv_seq_of(a, r0, e, l, a.n_tokens);
        }
        if (!more) break;
    }
    int entry[T];
#pragma unroll
    for (int x = 0; x < T; ++x) {
        const int at = i0 + x - s[x].row0;
        const bool on = b[x] >= 0 && at >= 0 && at < s[x].rows;
        pos[x] = on ? s[x].len + at : -1;
        entry[x] = on ? kv_entry(a, b[x], pos[x]) : 0;
    }
#pragma unroll
    for (int x = 0; x < T; ++x) page[x] = pos[x] < 0 ? -2 : kv_valid(a, entry[x]);
}

// Every sequence's entries are looked at once per call, so that one that no
// row finds is recorded too: by a block of its own behind those that have rows,
// where nothing waits for it.
__device__ __forceinline__ bool checks_all(const KvArgs& a)
{
    if (blockIdx.x + 1 != gridDim.x) return false;
    for (int b = threadIdx.x; b < a.n_seqs; b += blockDim.x) kv_seq(a, b, a.n_tokens);
    return true;
}

// ------------------------------------------------------------------ append
// One lane's eight values of a row: quantise and store. The row's DIM / 8
// lanes (FP8) or the block's two lanes (NVFP4) share the scale.
template <int FMT, int DIM>
__device__ __forceinline__ void store8(const KvArgs& a, int kv, int64_t row, int c, const uint4 raw, int lane)
{
    if constexpr (FMT == QG_KV_BF16) {
        if (row >= 0) *reinterpret_cast<uint4*>(a.codes[kv] + row * (2 * DIM) + c * 16) = raw;
    } else {
        float y[8];
        unpack8(raw, y);
        const float g = a.g[kv];
        if (g != 1.f) divide8(y, g, max8(y));
        if constexpr (FMT == QG_KV_FP8) {
            float top = max8(y);
#pragma unroll
            for (int off = 1; off < DIM / 8; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            // 448 = 1.75 * 2^8, so top <= 448 * 2^e first at e = exponent - 8, one more above 1.75
            const uint32_t m = __float_as_uint(top);
            const int e = max(-14, min(7, static_cast<int>(m >> 23) - 135 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0)));
            const float up = __int_as_float((127 - e) << 23);
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = to_e4m3x2(y[4 * i] * up, y[4 * i + 1] * up) |
                       to_e4m3x2(y[4 * i + 2] * up, y[4 * i + 3] * up) << 16;
            if (row >= 0) {
                *reinterpret_cast<uint2*>(a.codes[kv] + row * DIM + c * 8) = make_uint2(w[0], w[1]);
                if (c == 0) a.scales[kv][row] = static_cast<uint8_t>(e + 15);
            }
        } else {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(y[i]));
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
            uint32_t sc, w = 0;
            if (top != top) {
                sc = 0x7F;  // NaN
            } else {
                sc = to_e4m3x2(__fdiv_rn(top, 6.f), 0.f) & 0xFFu;
                if (sc) {
                    divide8(y, half_bits_to_f32(e4m3x2_to_f16x2(sc) & 0xFFFFu), top);
#pragma unroll
                    for (int i = 0; i < 4; ++i) w |= to_e2m1x2(y[2 * i], y[2 * i + 1]) << (8 * i);
                }
            }
            if (row >= 0) {
                *reinterpret_cast<uint32_t*>(a.codes[kv] + row * (DIM / 2) + c * 4) = w;
                if ((lane & 1) == 0) a.scales[kv][row * (DIM / 16) + c / 2] = static_cast<uint8_t>(sc);
            }
        }
    }
}

// A warp takes U * 32 lanes' worth of the rows (keys of every head, then
// values) of T consecutive tokens.
template <int FMT, int DIM, int T, int U>
__global__ void __launch_bounds__(32 * kWarps) kv_append_kernel(const __grid_constant__ KvArgs a, const uint16_t* k, int64_t k_stride,
                                                                const uint16_t* v, int64_t v_stride, int parts)
{
    pdl_enter();
    if (checks_all(a)) return;
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int i0 = static_cast<int>(unit / parts) * T;
    if (i0 >= a.n_tokens) return;
    constexpr int kLanes = DIM / 8;                 // lanes of a row
    const int per_side = a.heads * kLanes;
    const int first = static_cast<int>(unit % parts) * 32 * U + lane;
    uint4 raw[T][U];
#pragma unroll
    for (int y = 0; y < T; ++y)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = first + 32 * u;
            raw[y][u] = make_uint4(0, 0, 0, 0);
            if (x < 2 * per_side && i0 + y < a.n_tokens) {
                const int64_t i = i0 + y;
                const uint16_t* src = x < per_side ? k + i * k_stride + x * 8 : v + i * v_stride + (x - per_side) * 8;
                raw[y][u] = ldg_cg_128(src);
            }
        }
    int page[T], pos[T];
    places<T>(a, i0, lane, page, pos);
#pragma unroll
    for (int y = 0; y < T; ++y) {
        if (page[y] < 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = first + 32 * u;
            const int kv = x >= per_side;
            const int z = x - kv * per_side;
            const int64_t row = x < 2 * per_side ? kv_row(a, page[y], z / kLanes, pos[y]) : -1;
            store8<FMT, DIM>(a, kv, row, z % kLanes, raw[y][u], lane);
        }
    }
}

// ------------------------------------------------------------------ read
// One lane's eight values as they are stored. All zeros read as zeros. (Plain
// loads: the kernel before, which may run on while this one starts, may be what
// wrote them, and the read-only path is for what nothing writes meanwhile.)
template <int FMT>
struct Stored {
    uint4 codes;                 // FP8: two words, NVFP4: one
    uint32_t scale;

    __device__ __forceinline__ void load(const uint8_t* c, const uint8_t* s, int64_t row, int piece, int dim)
    {
        if constexpr (FMT == QG_KV_BF16) {
            codes = ldg_cg_128(c + row * (2 * dim) + piece * 16);
        } else if constexpr (FMT == QG_KV_FP8) {
            const uint2 w = *reinterpret_cast<const uint2*>(c + row * dim + piece * 8);
            codes.x = w.x;
            codes.y = w.y;
            scale = s[row];
        } else {
            codes.x = *reinterpret_cast<const uint32_t*>(c + row * (dim / 2) + piece * 4);
            scale = s[row * (dim / 16) + piece / 2];
        }
    }

    // code * scale is an f16 number; times g in 32 bits
    __device__ __forceinline__ void values(float g, float (&f)[8]) const
    {
        if constexpr (FMT == QG_KV_BF16) {
            unpack8(codes, f);
        } else {
            uint32_t h[4], s2;
            if constexpr (FMT == QG_KV_FP8) {
                e4m3x4_to_f16x2x2(codes.x, h[0], h[1]);
                e4m3x4_to_f16x2x2(codes.y, h[2], h[3]);
                s2 = scale * 0x04000400u;                        // 2^(s-15) as f16, twice
            } else {
                e2m1x8_to_f16x2x4(codes.x, h);
                const uint32_t e = e4m3x2_to_f16x2(scale);
                s2 = __byte_perm(e, e, 0x1010);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t p = hmul2(h[i], s2);
                f[2 * i] = half_bits_to_f32(p & 0xFFFFu) * g;
                f[2 * i + 1] = half_bits_to_f32(p >> 16) * g;
            }
        }
    }
};

template <int FMT, int DIM, int T, int U>
__global__ void __launch_bounds__(32 * kWarps) kv_read_kernel(const __grid_constant__ KvArgs a, void* k_out, void* v_out, int f32, int parts)
{
    pdl_enter();
    if (checks_all(a)) return;
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int i0 = static_cast<int>(unit / parts) * T;
    if (i0 >= a.n_tokens) return;
    constexpr int kLanes = DIM / 8;
    const int per_side = a.heads * kLanes;
    const int first = static_cast<int>(unit % parts) * 32 * U + lane;
    int page[T], pos[T];
    places<T>(a, i0, lane, page, pos);
    Stored<FMT> raw[T][U];
#pragma unroll
    for (int y = 0; y < T; ++y)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = first + 32 * u;
            raw[y][u] = Stored<FMT>{};
            if (x < 2 * per_side && page[y] >= 0) {
                const int kv = x >= per_side;
                const int z = x - kv * per_side;
                raw[y][u].load(a.codes[kv], a.scales[kv], kv_row(a, page[y], z / kLanes, pos[y]), z % kLanes, DIM);
            }
        }
#pragma unroll
    for (int y = 0; y < T; ++y) {
        if (page[y] < -1) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = first + 32 * u;
            if (x >= 2 * per_side) continue;
            const int kv = x >= per_side;
            float f[8];
            raw[y][u].values(a.g[kv], f);
            const int64_t at = (static_cast<int64_t>(i0 + y) * per_side + (x - kv * per_side)) * 8;
            void* out = kv ? v_out : k_out;
            if (f32) {
                float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
                o[0] = make_float4(f[0], f[1], f[2], f[3]);
                o[1] = make_float4(f[4], f[5], f[6], f[7]);
            } else {
                uint4 o;
                o.x = pack_bf16x2(f[0], f[1]);
                o.y = pack_bf16x2(f[2], f[3]);
                o.z = pack_bf16x2(f[4], f[5]);
                o.w = pack_bf16x2(f[6], f[7]);
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = o;
            }
        }
    }
}

// ------------------------------------------------------------------ accept
// Moves one column (a 16-byte piece of a head's codes, or a piece of its
// scales) of a sequence's accepted tokens, in path order. path[i] >= i and
// ascending: position i is written only after everything that path sends to
// positions up to i was read, so batches that load first and store then are
// safe in place.
template <typename T>
__device__ __forceinline__ void move_column(const KvArgs& a, const KvSeq& s, int b, int head, uint8_t* base,
                                            int64_t row_bytes, int col, const int32_t* path, int n)
{
    constexpr int kBatch = 16;
    for (int i0 = 0; i0 < n; i0 += kBatch) {
        T v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (i0 + u < n) {
                const int p = s.len + path[s.row0 + i0 + u];
                const int page = a.table[static_cast<int64_t>(b) * a.max_pages + kv_page_index(a, p)];
                v[u] = *reinterpret_cast<const T*>(base + kv_row(a, page, head, p) * row_bytes + col);
            }
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (i0 + u < n) {
                const int p = s.len + i0 + u;
                const int page = a.table[static_cast<int64_t>(b) * a.max_pages + kv_page_index(a, p)];
                *reinterpret_cast<T*>(base + kv_row(a, page, head, p) * row_bytes + col) = v[u];
            }
    }
}

// One block per sequence. It checks the path and the pages first (a sequence
// is moved as a whole or not at all), and only then writes, new_lens last, so
// that new_lens may be seq_lens.
__global__ void __launch_bounds__(kAcceptThreads) kv_accept_kernel(const __grid_constant__ KvArgs a, const int32_t* path,
                                                                   const int32_t* n_accept, int32_t* new_lens)
{
    pdl_enter();
    const int b = blockIdx.x;
    const KvSeq s = kv_seq(a, b, a.n_tokens);
    int n = n_accept[b];
    bool bad = n < 0 || n > s.rows;
    if (!bad)
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const int p = path[s.row0 + i];
            if (p < i || p >= s.rows || (i > 0 && path[s.row0 + i - 1] >= p))
                bad = true;
            else
                bad = kv_page(a, b, s.len + p) < 0 || kv_page(a, b, s.len + i) < 0 || bad;
        }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) set_device_status(a.status, QG_ERR_INVALID_ARG);
        n = 0;
    }
    const int rb = kv_row_bytes(a.fmt, a.dim), sb = kv_scale_bytes(a.fmt, a.dim);
    const int code_cols = rb / 16, scale_cols = sb >= 4 ? sb / 4 : sb;
    const int cols = code_cols + scale_cols;
    for (int x = threadIdx.x; x < 2 * a.heads * cols; x += blockDim.x) {
        const int kv = x / (a.heads * cols);
        const int head = x / cols % a.heads, c = x % cols;
        if (c < code_cols)
            move_column<uint4>(a, s, b, head, a.codes[kv], rb, c * 16, path, n);
        else if (sb >= 4)
            move_column<uint32_t>(a, s, b, head, a.scales[kv], sb, (c - code_cols) * 4, path, n);
        else
            move_column<uint8_t>(a, s, b, head, a.scales[kv], sb, 0, path, n);
    }
    if (new_lens && threadIdx.x == 0) new_lens[b] = s.len + n;
}

// How a call's rows are dealt to warps: one token and 32 lanes each, so that a
// decode step's few rows spread over many SMs, or 128 lanes of one token
// (append) or two (read) once that still makes four warps per scheduler.
// Measured on 32,256 tokens of 4 heads of 128, append in FP8 and read of NVFP4
// (us): 1 x 128 lanes 26.2 and 20.2, 2 x 128 28.0 and 18.1, 2 x 64 29.3 and
// 21.9, 4 x 64 30.4 and 20.3, 2 x 32 34.4 and 27.5.
constexpr int kPieces = 4, kAppendTokens = 1, kReadTokens = 2;

struct RowPlan {
    bool wide;
    int parts;
    unsigned blocks;
};

RowPlan plan_rows(const KvArgs& a, int wide_tokens)
{
    const int64_t lanes = 2LL * a.heads * (a.dim / 8);
    RowPlan p;
    p.wide = a.n_tokens * lanes >= 32LL * wide_tokens * kPieces * 16 * sm_count(-1);
    const int per = 32 * (p.wide ? kPieces : 1), tokens = p.wide ? wide_tokens : 1;
    p.parts = static_cast<int>((lanes + per - 1) / per);
    const int64_t warps = (static_cast<int64_t>(a.n_tokens) + tokens - 1) / tokens * p.parts;
    p.blocks = static_cast<unsigned>((warps + kWarps - 1) / kWarps) + 1;
    return p;
}

template <int FMT, int DIM>
cudaError_t append_dim(const KvArgs& a, const uint16_t* k, int64_t ks, const uint16_t* v, int64_t vs,
                       cudaStream_t stream)
{
    const RowPlan p = plan_rows(a, kAppendTokens);
    auto kern = p.wide ? kv_append_kernel<FMT, DIM, kAppendTokens, kPieces> : kv_append_kernel<FMT, DIM, 1, 1>;
    return launch_pdl(kern, dim3(p.blocks), dim3(32 * kWarps), 0, stream, a, k, ks, v, vs, p.parts);
}

template <int FMT, int DIM>
cudaError_t read_dim(const KvArgs& a, void* k, void* v, int f32, cudaStream_t stream)
{
    const RowPlan p = plan_rows(a, kReadTokens);
    auto kern = p.wide ? kv_read_kernel<FMT, DIM, kReadTokens, kPieces> : kv_read_kernel<FMT, DIM, 1, 1>;
    return launch_pdl(kern, dim3(p.blocks), dim3(32 * kWarps), 0, stream, a, k, v, f32, p.parts);
}

// fn(std::integral_constant fmt, std::integral_constant dim)
template <typename Fn>
cudaError_t by_format(const KvArgs& a, Fn fn)
{
    auto with = [&](auto f) {
        if (a.dim == 64) return fn(f, Int<64>{});
        if (a.dim == 128) return fn(f, Int<128>{});
        return fn(f, Int<256>{});
    };
    if (a.fmt == QG_KV_BF16) return with(Int<QG_KV_BF16>{});
    if (a.fmt == QG_KV_FP8) return with(Int<QG_KV_FP8>{});
    return with(Int<QG_KV_NVFP4>{});
}

bool with_status(const KvArgs& in, KvArgs& a)
{
    a = in;
    a.status = device_status_ptr();
    return a.status != nullptr;
}

}  // namespace

qg_status launch_kv_append(const KvArgs& in, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           cudaStream_t stream)
{
    KvArgs a;
    if (!with_status(in, a)) return QG_ERR_CUDA;
    const cudaError_t e = by_format(a, [&](auto f, auto d) {
        return append_dim<decltype(f)::value, decltype(d)::value>(a, static_cast<const uint16_t*>(k), k_stride,
                                                                  static_cast<const uint16_t*>(v), v_stride, stream);
    });
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

qg_status launch_kv_read(const KvArgs& in, void* k_out, void* v_out, int f32, cudaStream_t stream)
{
    KvArgs a;
    if (!with_status(in, a)) return QG_ERR_CUDA;
    const cudaError_t e = by_format(a, [&](auto f, auto d) {
        return read_dim<decltype(f)::value, decltype(d)::value>(a, k_out, v_out, f32, stream);
    });
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

qg_status launch_kv_accept(const KvArgs& in, const int32_t* path, const int32_t* n_accept, int32_t* new_lens,
                           cudaStream_t stream)
{
    KvArgs a;
    if (!with_status(in, a)) return QG_ERR_CUDA;
    const cudaError_t e = launch_pdl(kv_accept_kernel, dim3(static_cast<unsigned>(a.n_seqs)), dim3(kAcceptThreads), 0,
                                     stream, a, path, n_accept, new_lens);
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

}  // namespace qg

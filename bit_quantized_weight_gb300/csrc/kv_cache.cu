// kv_cache.cu -- the paged low-precision cache of a decode step: quantise as
// it is written (kv_cache_append), read it back (kv_cache_read), keep the
// accepted path of a drafted tree (kv_cache_accept). The pages name the
// formats (NInfer article, section 4: BF16, FP8-E4M3 and NVFP4 in pages of 64
// tokens; Decapybara README, decode_ops.cu); the layouts are include/qgemv.h's.
//
// All three are bound by bytes (large calls) or by one chain of dependent
// loads (a decode step: token_start -> page table -> the row). A lane holds
// eight consecutive values of a head, 16 bytes as bf16, so that a row's lanes
// are neighbours and an amax is a few shuffles.
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

__device__ __forceinline__ uint32_t max8_bits(const float (&y)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    return m;
}

// The sequence that row i belongs to: the number of sequences that end at or
// before it, by ballots over 32 sequences at a time (one load latency for up
// to 32). n_seqs for a row behind the last sequence.
__device__ __forceinline__ int seq_of_row(const KvArgs& a, int i, int lane)
{
    int b = 0;
    for (int j = 0; j < a.n_seqs; j += 32) {
        const bool before = j + lane < a.n_seqs && a.start[j + lane + 1] <= i;
        const int n = __popc(__ballot_sync(0xffffffffu, before));
        b += n;
        if (n < 32) break;
    }
    return b;
}

// The place of row i: its page and position, or false if it has none.
__device__ __forceinline__ bool place_of_row(const KvArgs& a, int i, int lane, int& page, int& pos)
{
    const int b = seq_of_row(a, i, lane);
    if (b >= a.n_seqs) return false;
    const KvSeq s = kv_seq(a, b, a.n_tokens);
    if (i < s.row0 || i - s.row0 >= s.rows) return false;
    pos = s.len + (i - s.row0);
    page = kv_page(a, b, pos);
    return true;
}

// Every sequence's entries are looked at once per call, so that one that no
// row finds is recorded too.
__device__ __forceinline__ void check_all(const KvArgs& a)
{
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.n_seqs; b += blockDim.x) kv_seq(a, b, a.n_tokens);
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
        if (g != 1.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(y[i], g);
        }
        if constexpr (FMT == QG_KV_FP8) {
            // a NaN (bits above infinity's) does not count for the maximum
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t v = __float_as_uint(y[i]) & 0x7FFFFFFFu;
                m = max(m, v > 0x7F800000u ? 0u : v);
            }
#pragma unroll
            for (int off = 1; off < DIM / 8; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
            // 448 = 1.75 * 2^8, so m <= 448 * 2^e first at e = exponent - 8, one more above 1.75
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
            uint32_t m = max8_bits(y);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            uint32_t sc, w = 0;
            if (m > 0x7F800000u) {
                sc = 0x7F;  // NaN
            } else {
                sc = to_e4m3x2(__fdiv_rn(__uint_as_float(m), 6.f), 0.f) & 0xFFu;
                if (sc) {
                    const float f = half_bits_to_f32(e4m3x2_to_f16x2(sc) & 0xFFFFu);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w |= to_e2m1x2(__fdiv_rn(y[2 * i], f), __fdiv_rn(y[2 * i + 1], f)) << (8 * i);
                }
            }
            if (row >= 0) {
                *reinterpret_cast<uint32_t*>(a.codes[kv] + row * (DIM / 2) + c * 4) = w;
                if ((lane & 1) == 0) a.scales[kv][row * (DIM / 16) + c / 2] = static_cast<uint8_t>(sc);
            }
        }
    }
}

// A warp takes U * 32 lanes' worth of one token's rows (keys of every head,
// then values).
template <int FMT, int DIM, int U>
__global__ void __launch_bounds__(32 * kWarps) kv_append_kernel(KvArgs a, const uint16_t* k, int64_t k_stride,
                                                                const uint16_t* v, int64_t v_stride, int parts)
{
    pdl_enter();
    check_all(a);
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int i = static_cast<int>(unit / parts);
    if (i >= a.n_tokens) return;
    constexpr int kLanes = DIM / 8;                 // lanes of a row
    const int per_side = a.heads * kLanes;
    const int first = static_cast<int>(unit % parts) * 32 * U + lane;
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int x = first + 32 * u;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (x < 2 * per_side) {
            const uint16_t* src = x < per_side ? k + i * k_stride + x * 8 : v + i * v_stride + (x - per_side) * 8;
            raw[u] = *reinterpret_cast<const uint4*>(src);
        }
    }
    int page, pos;
    if (!place_of_row(a, i, lane, page, pos) || page < 0) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int x = first + 32 * u;
        const int kv = x >= per_side;
        const int y = x - kv * per_side;
        const int64_t row = x < 2 * per_side ? kv_row(a, page, y / kLanes, pos) : -1;
        store8<FMT, DIM>(a, kv, row, y % kLanes, raw[u], lane);
    }
}

// ------------------------------------------------------------------ read
// The f16 values (code * scale, exact) of one lane's eight codes.
template <int FMT>
__device__ __forceinline__ void load8(const uint8_t* codes, const uint8_t* scales, int64_t row, int c, int dim,
                                      float g, float (&f)[8])
{
    if constexpr (FMT == QG_KV_BF16) {
        unpack8(ldg_nc_128(codes + row * (2 * dim) + c * 16), f);
    } else {
        uint32_t h[4], s;
        if constexpr (FMT == QG_KV_FP8) {
            const uint2 w = *reinterpret_cast<const uint2*>(codes + row * dim + c * 8);
            h[0] = e4m3x2_to_f16x2(w.x & 0xFFFFu);
            h[1] = e4m3x2_to_f16x2(w.x >> 16);
            h[2] = e4m3x2_to_f16x2(w.y & 0xFFFFu);
            h[3] = e4m3x2_to_f16x2(w.y >> 16);
            s = static_cast<uint32_t>(scales[row]) << 10;   // 2^(s-15) as f16
        } else {
            e2m1x8_to_f16x2x4(*reinterpret_cast<const uint32_t*>(codes + row * (dim / 2) + c * 4), h);
            s = e4m3x2_to_f16x2(scales[row * (dim / 16) + c / 2]) & 0xFFFFu;
        }
        s |= s << 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t p = hmul2(h[i], s);
            f[2 * i] = half_bits_to_f32(p & 0xFFFFu) * g;
            f[2 * i + 1] = half_bits_to_f32(p >> 16) * g;
        }
    }
}

template <int FMT, int DIM, int U>
__global__ void __launch_bounds__(32 * kWarps) kv_read_kernel(KvArgs a, void* k_out, void* v_out, int f32, int parts)
{
    pdl_enter();
    check_all(a);
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int i = static_cast<int>(unit / parts);
    if (i >= a.n_tokens) return;
    constexpr int kLanes = DIM / 8;
    const int per_side = a.heads * kLanes;
    const int first = static_cast<int>(unit % parts) * 32 * U + lane;
    int page, pos;
    if (!place_of_row(a, i, lane, page, pos)) return;
    float f[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int x = first + 32 * u;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[u][j] = 0.f;
        if (x < 2 * per_side && page >= 0) {
            const int kv = x >= per_side;
            const int y = x - kv * per_side;
            load8<FMT>(a.codes[kv], a.scales[kv], kv_row(a, page, y / kLanes, pos), y % kLanes, DIM, a.g[kv], f[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int x = first + 32 * u;
        if (x >= 2 * per_side) continue;
        const int kv = x >= per_side;
        const int64_t at = (static_cast<int64_t>(i) * per_side + (x - kv * per_side)) * 8;
        void* out = kv ? v_out : k_out;
        if (f32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
            o[0] = make_float4(f[u][0], f[u][1], f[u][2], f[u][3]);
            o[1] = make_float4(f[u][4], f[u][5], f[u][6], f[u][7]);
        } else {
            uint4 o;
            o.x = pack_bf16x2(f[u][0], f[u][1]);
            o.y = pack_bf16x2(f[u][2], f[u][3]);
            o.z = pack_bf16x2(f[u][4], f[u][5]);
            o.w = pack_bf16x2(f[u][6], f[u][7]);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = o;
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
    constexpr int kBatch = 8;
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
__global__ void __launch_bounds__(kAcceptThreads) kv_accept_kernel(KvArgs a, const int32_t* path,
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

// Warps of a call over every token's rows: U * 32 lanes each. Four pieces per
// lane once that still fills the GPU several times over, else one, so that a
// decode step's few rows spread over more SMs.
struct RowPlan {
    int u, parts;
    unsigned blocks;
};

RowPlan plan_rows(const KvArgs& a)
{
    const int64_t lanes = 2LL * a.heads * (a.dim / 8);
    RowPlan p;
    p.u = a.n_tokens * lanes >= 4LL * 32 * 64 * sm_count(-1) ? 4 : 1;
    p.parts = static_cast<int>((lanes + 32 * p.u - 1) / (32 * p.u));
    p.blocks = static_cast<unsigned>((static_cast<int64_t>(a.n_tokens) * p.parts + kWarps - 1) / kWarps);
    return p;
}

template <int FMT, int DIM>
cudaError_t append_dim(const KvArgs& a, const uint16_t* k, int64_t ks, const uint16_t* v, int64_t vs,
                       cudaStream_t stream)
{
    const RowPlan p = plan_rows(a);
    if (p.u == 4)
        return launch_pdl(kv_append_kernel<FMT, DIM, 4>, dim3(p.blocks), dim3(32 * kWarps), 0, stream, a, k, ks, v,
                          vs, p.parts);
    return launch_pdl(kv_append_kernel<FMT, DIM, 1>, dim3(p.blocks), dim3(32 * kWarps), 0, stream, a, k, ks, v, vs,
                      p.parts);
}

template <int FMT, int DIM>
cudaError_t read_dim(const KvArgs& a, void* k, void* v, int f32, cudaStream_t stream)
{
    const RowPlan p = plan_rows(a);
    if (p.u == 4)
        return launch_pdl(kv_read_kernel<FMT, DIM, 4>, dim3(p.blocks), dim3(32 * kWarps), 0, stream, a, k, v, f32,
                          p.parts);
    return launch_pdl(kv_read_kernel<FMT, DIM, 1>, dim3(p.blocks), dim3(32 * kWarps), 0, stream, a, k, v, f32,
                      p.parts);
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

// The call's grid may pass 2^31 - 1 blocks only for more than 10^9 rows.
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

// tree_attention.cu -- attention of drafted tokens over the paged cache.
#include "kv_common.cuh"

namespace qg {
namespace {

// One warp per (row, query head): the running maximum and sum of a softmax,
// one key at a time.
__global__ void __launch_bounds__(256) tree_simple_kernel(KvArgs a, const uint16_t* q, int64_t q_stride, int q_heads,
                                                          int max_tree, const uint64_t* mask, float scale,
                                                          uint16_t* out, float* lse)
{
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int row = static_cast<int>(unit / q_heads), h = static_cast<int>(unit % q_heads);
    if (row >= a.n_tokens) return;
    int b = 0;
    KvSeq s{};
    for (; b < a.n_seqs; ++b) {
        s = kv_seq(a, b, max_tree);
        if (row >= s.row0 && row - s.row0 < s.rows) break;
    }
    if (b == a.n_seqs) return;
    const int n = a.dim / 32;
    float qf[8], acc[8];
    for (int i = 0; i < n; ++i) {
        qf[i] = bf16_bits_to_f32(q[row * q_stride + h * a.dim + lane * n + i]);
        acc[i] = 0.f;
    }
    const int j = row - s.row0, head = h / (q_heads / a.heads);
    const uint64_t bits = mask ? mask[row] : (2ull << j) - 1;
    float m = -INFINITY, l = 0.f;
    const int rb = kv_row_bytes(a.fmt, a.dim), sb = kv_scale_bytes(a.fmt, a.dim);
    for (int p = 0; p < s.len + s.rows; ++p) {
        if (p >= s.len && !((bits >> (p - s.len)) & 1)) continue;
        const int page = kv_page(a, b, p);
        if (page < 0) continue;
        const int64_t r = kv_row(a, page, head, p);
        float kf[2][8];
        for (int kv = 0; kv < 2; ++kv)
            for (int i = 0; i < n; ++i) {
                const int d = lane * n + i;
                const uint8_t* c = a.codes[kv] + r * rb;
                float v;
                if (a.fmt == QG_KV_BF16) {
                    v = bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(c)[d]);
                } else if (a.fmt == QG_KV_FP8) {
                    v = half_bits_to_f32(e4m3x2_to_f16x2(c[d]) & 0xFFFFu) *
                        half_bits_to_f32(static_cast<uint32_t>(a.scales[kv][r]) << 10) * a.g[kv];
                } else {
                    v = half_bits_to_f32(e2m1x2_to_f16x2(c[d / 2] >> (4 * (d & 1)) & 15) & 0xFFFFu) *
                        half_bits_to_f32(e4m3x2_to_f16x2(a.scales[kv][r * sb + d / 16]) & 0xFFFFu) * a.g[kv];
                }
                kf[kv][i] = v;
            }
        float dot = 0.f;
        for (int i = 0; i < n; ++i) dot += qf[i] * kf[0][i];
        for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        dot *= scale;
        const float mn = fmaxf(m, dot), f = expf(m - mn), w = expf(dot - mn);
        l = l * f + w;
        for (int i = 0; i < n; ++i) acc[i] = acc[i] * f + w * kf[1][i];
        m = mn;
    }
    for (int i = 0; i < n; ++i)
        out[(static_cast<int64_t>(row) * q_heads + h) * a.dim + lane * n + i] =
            f32_to_bf16_bits_rn(l > 0.f ? acc[i] / l : 0.f);
    if (lse && lane == 0) lse[static_cast<int64_t>(row) * q_heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t tree_attention_workspace_bytes(int head_dim, int group, int max_tree)
{
    (void)head_dim;
    (void)group;
    (void)max_tree;
    return 256;
}

qg_status launch_tree_attention(const KvArgs& in, const uint16_t* q, int64_t q_stride, int q_heads, int max_tree,
                                const uint64_t* mask, float scale, uint16_t* out, float* lse, void*,
                                cudaStream_t stream)
{
    KvArgs a = in;
    a.status = device_status_ptr();
    if (!a.status) return QG_ERR_CUDA;
    const int64_t units = static_cast<int64_t>(a.n_tokens) * q_heads;
    const cudaError_t e = launch_pdl(tree_simple_kernel, dim3(static_cast<unsigned>((units + 7) / 8)), dim3(256), 0,
                                     stream, a, q, q_stride, q_heads, max_tree, mask, scale, out, lse);
    return e == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

}  // namespace qg

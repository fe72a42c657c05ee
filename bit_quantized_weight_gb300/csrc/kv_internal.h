// kv_internal.h -- types shared by the host launchers and the kernels of the
// paged cache, the attention over it, the pages that sequences share and the
// selection of beam search.
#pragma once

#include "qgemv_internal.h"

namespace qg {

constexpr int kKvMaxSeqs = 1024;                      // sequences of a cache call
constexpr int kKvMaxTokens = 1 << 24;                 // rows of a cache call
constexpr int kKvMaxPositions = 1 << 30;              // of a sequence

// A paged cache and a call's batch of sequences as the kernels read them
// (qg_kv_cache and qg_kv_batch after validation).
struct KvArgs {
    int fmt;                    // qg_kv_format
    int num_pages;
    int page_size;
    int heads;                  // key/value heads
    int dim;
    uint8_t* codes[2];          // keys, values
    uint8_t* scales[2];
    float g[2];
    const int32_t* table;
    const int32_t* lens;
    const int32_t* start;
    int n_seqs;
    int max_pages;
    int n_tokens;
    uint64_t page_magic;        // ceil(2^36 / (page_size / 16)), see kv_page_index
    int* status;
};

constexpr int kKvMaxPoolPages = 1 << 22;              // of a page record

// A page record as the kernels read and change it (qg_kv_pages after
// validation), and a list of moves.
struct PageArgs {
    int32_t* table;
    int32_t* lens;
    int32_t* held;
    int32_t* refs;
    int n_seqs;
    int max_pages;
    int num_pages;
    int page_size;
    int* status;
};

struct MoveArgs {
    int4* list;
    int32_t* count;
    int capacity;
};

qg_status launch_pages_fork(const PageArgs& a, const int32_t* parent, cudaStream_t stream);
qg_status launch_pages_reserve(const PageArgs& a, const int32_t* n_new, const MoveArgs& m, int32_t* n_free,
                               cudaStream_t stream);
qg_status launch_pages_compact(const PageArgs& a, const MoveArgs& m, int32_t* page_map, int32_t* n_live,
                               cudaStream_t stream);
qg_status launch_pages_copy(const KvArgs& a, const MoveArgs& m, cudaStream_t stream);

// Beam search's selection (beam_select after validation).
struct BeamArgs {
    const void* logits;
    int f32;
    int64_t stride;
    int lanes;
    int beams;
    int vocab;
    const float* scores;
    const uint8_t* finished;
    int eos;
    int pad;
    int n_out;
    float* out_scores;
    int32_t* out_tokens;
    int32_t* out_parents;
    uint8_t* out_finished;
    int* status;
};

size_t beam_select_workspace_bytes(int lanes, int beams, int vocab);
qg_status launch_beam_select(const BeamArgs& a, void* workspace, cudaStream_t stream);

qg_status launch_kv_append(const KvArgs& a, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           cudaStream_t stream);
qg_status launch_kv_read(const KvArgs& a, void* k_out, void* v_out, int f32, cudaStream_t stream);
qg_status launch_kv_accept(const KvArgs& a, const int32_t* path, const int32_t* n_accept, int32_t* new_lens,
                           cudaStream_t stream);
bool tree_attention_serves(const KvArgs& a, int group, int max_tree);
size_t tree_attention_workspace_bytes(int head_dim, int group, int max_tree);
qg_status launch_tree_attention(const KvArgs& a, const uint16_t* q, int64_t q_stride, int q_heads, int max_tree,
                                const uint64_t* mask, float scale, uint16_t* out, float* lse, void* workspace,
                                cudaStream_t stream);

}  // namespace qg

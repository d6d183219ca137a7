// Host-side launch interface between the C-ABI layer (pkv_api.cu) and the
// kernel translation units.  Internal to libpkv.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

namespace pkv {

// Launch `kern` with programmatic stream serialisation: its CTAs may be scheduled
// while the previous kernel on the stream drains; every libpkv kernel starts with
// griddep_wait(), so no input is read before the predecessor has completed.
// With pdl false the launch is ordinary: no CTA is placed before the predecessor ends.
template <typename... KArgs, typename... Args>
cudaError_t launch_maybe_pdl(bool pdl, void (*kern)(KArgs...), dim3 grid, dim3 block,
                             size_t smem, cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args&&... args) {
    return launch_maybe_pdl(true, kern, grid, block, smem, stream, std::forward<Args>(args)...);
}

// Upper bound on split-KV partitions of one sequence (combine kernel's smem).
constexpr int kMaxParts = 1024;

struct DecodeArgs {
    void* out;
    const void* q;
    const void* k_pool;
    const void* v_pool;
    const int32_t* block_tables;
    const int32_t* context_lens;
    float* o_part;   // [S][Hq][max_parts][D]
    float* m_part;   // [S][Hq][max_parts]  (log2 domain)
    float* l_part;   // [S][Hq][max_parts]
    int* status;
    int64_t num_blocks;
    int max_blocks_per_seq;   // block-table row stride, in pool blocks
    int num_seqs;
    int num_q_heads;
    int num_kv_heads;
    // The kernels walk a sequence in 16-token chunks: chunk c is rows
    // 16 (c & (2^chunk_shift - 1)) .. + 15 of the block in table entry c >> chunk_shift
    // (chunk_shift = log2(block_size / 16): 0 for 16-token blocks, 1 for 32).
    int chunk_shift;
    int partition_chunks;   // 16-token chunks per split-KV partition
    int max_parts;          // partitions of the decoded chunk range per sequence
    float scale_log2;       // softmax scale * log2(e)
    // Cascade decode: chunks [0, chunk_offset) of every sequence were handled by a
    // separate shared-prefix pass whose partial sits at partition 0; the split kernel
    // covers chunks [chunk_offset, nchunks) into partitions extra_parts.. and the combine
    // merges extra_parts + max_parts partials per row.
    int chunk_offset;
    int extra_parts;
    int defer_combine;   // nonzero: the launcher leaves the combine to the caller
    // nonzero: the split kernel is launched without programmatic dependent launch, so its
    // CTAs take no SM before the stream's previous kernel has ended (the cascade decode:
    // the prefix pass on the side stream is placed first).
    int no_pdl;
    // Test hook (both decode kernels): nonzero makes warp 0 of CTA (0, 0, 0) arm its first
    // stage for 16 bytes more than the stage's copies deliver, so that wait runs out of
    // time (PKV_ERR_TIMEOUT) while every copy still lands.  Zero in normal use.
    int test_stall;
    // Fused append (decode only): non-null k_new / v_new ([num_seqs][Hkv][D], pool
    // dtype) are the K / V of each sequence's newest token, position context_lens[s] - 1.
    // The CTA whose chunk holds that position stores them into the pool slot the block
    // table gives for it and uses them in place of the row it staged from the pool (which
    // the append has not reached yet).
    const void* k_new;
    const void* v_new;
    // Accumulated attention weights (pkv_paged_decode_weights): non-null `scores` makes
    // the split kernels keep every score, scale * log2(e) * q.k, in
    // scores[S][Hkv][score_tokens][G].  From them and the partitions' m / l the finishing
    // launch adds each cached token's weight to weights[row][kvh][token]; where there is one
    // partition, its CTA does so itself and no second launch follows.
    float* scores;
    int score_tokens;         // tokens per (sequence, kv head) in `scores`
    float* weights;
    const int32_t* row_ids;   // weight row of each sequence (null: its index)
    int64_t weights_stride;   // floats between the rows of two kv heads
    int num_rows;
    float decay;
};

#ifdef __CUDACC__
// Zeros of the G output rows (kv head kvh's query heads) of sequence `seq`, elem_bytes
// per element, stored 16 bytes at a time by the threads of the calling CTA; for a
// sequence the decode kernels reject (context length below 1), so that its rows hold no
// stale memory.
__device__ __forceinline__ void zero_invalid_rows(const DecodeArgs& a, int seq, int kvh, int G,
                                                  int D, int elem_bytes) {
    const size_t row0 = static_cast<size_t>(seq) * a.num_q_heads + static_cast<size_t>(kvh) * G;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(a.out) + row0 * D * elem_bytes);
    const int n16 = G * D * elem_bytes / 16;
    for (int i = threadIdx.x; i < n16; i += blockDim.x) dst[i] = make_uint4(0, 0, 0, 0);
}
#endif

// CUDA-core decode (fp32 and bf16 pools): split kernel + combine.
cudaError_t launch_paged_decode(const DecodeArgs& a, int dtype, int head_dim, int group,
                                cudaStream_t stream);
// Tensor-core decode for bf16 pools (warp-level MMA): split kernel + combine.
cudaError_t launch_paged_decode_tc(const DecodeArgs& a, int head_dim, int group,
                                   cudaStream_t stream);
// Log-sum-exp merge of the split-KV partials into `out`, and, beside it in the same
// launch, the accumulated attention weights (a.scores set).
cudaError_t launch_decode_finish(const DecodeArgs& a, int dtype, int head_dim, int group,
                                 cudaStream_t stream);
// Log-sum-exp merge of the split-KV partials into `out`.
cudaError_t launch_decode_combine(const DecodeArgs& a, int dtype, int head_dim,
                                  cudaStream_t stream);

// Tensor maps (host): a pool viewed as rows [num_blocks * Hkv * 16] x head_dim bf16,
// box 64 columns x 16 rows, 128-byte swizzle.
bool make_pool_map(CUtensorMap* m, const void* pool, int64_t rows, int head_dim);
// The same pool (head_dim 128) as one box per 16-row block: dims {64 columns, 8 rows,
// 2 column halves, rows / 8 row groups}, box {64, 8, 2, 2} = 4 KB, landing in shared
// memory as [row group][half][8 rows][128 B] with the 128-byte swizzle.
bool make_pool_block_map(CUtensorMap* m, const void* pool, int64_t rows);
// cudaFuncSetAttribute(kern, MaxDynamicSharedMemorySize, bytes), made once per kernel and
// device (later calls with no more bytes return at once).
cudaError_t set_smem_once(const void* kern, int bytes);
// q [tokens][Hq][head_dim] bf16 read as boxes of 64 columns x G heads x tok tokens.
bool make_q_group_map(CUtensorMap* m, const void* q, int tokens, int hq, int head_dim, int G,
                      int tok);

cudaError_t launch_kv_append(void* k_pool, void* v_pool, const int64_t* slot_mapping,
                             const void* k, const void* v, int64_t num_tokens, int num_kv_heads,
                             int row_bytes, int block_size, int64_t num_blocks, int* status,
                             cudaStream_t stream);

cudaError_t launch_copy_blocks(void* k_pool, void* v_pool, const int32_t* pairs, int num_pairs,
                               int64_t block_bytes, int64_t num_blocks, int* status,
                               cudaStream_t stream);

struct PrefillArgs {
    int head_dim;     // 64 or 128
    int block_size;   // tokens per pool block: 16 or 32
    void* out;
    const void* q;
    const void* k_pool;
    const void* v_pool;
    const int32_t* block_tables;
    const int32_t* cached_lens;
    const int32_t* new_lens;
    const int32_t* q_offsets;
    int* status;
    int64_t num_blocks;
    int max_blocks_per_seq;
    int num_reqs;
    int total_new;
    int max_new;
    int num_q_heads;
    int num_kv_heads;
    float scale_log2;
    // Cascade mode (shared-prefix decode): one "request" whose cascade_keys keys are the
    // shared prefix and whose cascade_rows query rows are the sequences (one token each);
    // every row attends all prefix keys (no causal mask), the grid's z dimension splits
    // the prefix's tiles (cascade_tiles_per_split each) and split z writes its partial to
    // slot z of the split-KV partials (max_parts_total slots per row) instead of `out`.
    int cascade;
    int cascade_keys;   // cascade: prefix length (keys); rows come from cascade_rows
    int cascade_rows;   // cascade: number of sequences (query rows per head)
    int cascade_tiles_per_split;   // cascade: 128-key tiles per split (grid z = splits)
    int max_parts_total;
    float* o_part;
    float* m_part;
    float* l_part;
    // A CTA whose rows all attend at least this many keys stores P as one bf16 value
    // (round to nearest); otherwise as bf16 hi + lo (see the prefill kernel).
    int p_single_min_keys;
};

cudaError_t launch_paged_prefill(const PrefillArgs& a, int group, cudaStream_t stream);

// Rotary positions of q rows (k_pool null), or of q and k rows with k and v stored into
// their pool slots.  Strides are elements per token.
struct RopeArgs {
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    void* k_pool;
    void* v_pool;
    const int64_t* slot_mapping;
    const int32_t* positions;
    const double* inv_freq;   // [rotary_dim / 2], radians per position
    int* status;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    int64_t num_tokens;
    int64_t num_slots;
    int num_q_heads;
    int num_kv_heads;
    int rotary_dim;    // a multiple of 16, at most the head dim
    int block_shift;   // log2(block_size)
    int interleaved;
    int inverse;
    float attn_scale;
};
cudaError_t launch_rope(const RopeArgs& a, int dtype, int head_dim, cudaStream_t stream);

// Accumulated attention weights of the requests' last `window` new tokens.
struct PrefillWeightsArgs {
    const void* q;
    const void* k_pool;
    const int32_t* block_tables;
    const int32_t* cached_lens;
    const int32_t* new_lens;
    const int32_t* q_offsets;
    const int32_t* row_ids;   // weight row of each request (null: its index)
    float* weights;           // [num_rows][Hkv][weights_stride]
    float2* stats;            // workspace: (reference, sum) [R][Hkv][splits][rows_pad];
                              // tensor cores: two of them, [..][splits][2][rows_pad]
    int* next_item;           // workspace (tensor cores): pass 1's counter of items taken
    float* neg_lse;           // workspace (tensor cores): -log2(sum 2^s) [R][Hkv][rows_pad]
    int* status;
    int64_t num_blocks;
    int64_t weights_stride;
    int num_rows;
    int max_blocks_per_seq;
    int block_shift;
    int num_reqs;
    int total_new;
    int max_new;
    int max_rows;      // tokens that count per request at most: max_new, or the window
    int max_context;
    int num_q_heads;
    int num_kv_heads;
    int window;        // 0: every new token
    int splits;        // parts the keys of a query tile are split into in pass 1
    int chunk_tiles;   // tensor cores: 128-key tiles per split
    int rows_pad;      // rows of one (request, kv head, split) in `stats`: a multiple of 128
    int group_shift;   // log2(G)
    // Pass 2 splits a key tile's rows into row_parts of rows_per_part (a multiple of 128) where
    // there are few key tiles; with more than one, each part's sums go to `parts`
    // ([R][Hkv][row_parts][max_context], workspace) and a last launch adds them up.
    int row_parts;
    int rows_per_part;
    float* parts;
    // fp32: a launch takes heads_per_launch (request, kv head) pairs; pass 1 keeps their scores,
    // [heads_per_launch][rows_pad][key_pad], for pass 2, or, null, pass 2 computes them again.
    float* scores;
    int64_t key_pad;
    int heads_per_launch;
    float scale_log2;
    float decay;
    // Tensor cores, tests only: 1 or 2 makes the first wait of CTA 0 for that pass's A tiles run
    // out of time (its barrier waits for 16 bytes more than the copies deliver).
    int test_stall;
};
// fp32 pools, on the CUDA cores.
cudaError_t launch_prefill_weights(const PrefillWeightsArgs& a, int head_dim, int group,
                                   cudaStream_t stream);
// The last launch of either where row_parts > 1: weights = decay * weights + the parts' sums.
// key_unit, row_unit: keys per pass-2 item and rows per tile, which say what parts a key has.
cudaError_t launch_add_parts(const PrefillWeightsArgs& a, int key_unit, int row_unit,
                             cudaStream_t stream);
// bf16 pools, on the tensor cores.
cudaError_t launch_prefill_weights_tc(const PrefillWeightsArgs& a, int head_dim, int group,
                                      cudaStream_t stream);

// Eviction by accumulated weight.  A row's bits have to fit in the shared memory of a cluster.
constexpr int kEvictMaxContext = 1 << 20;
struct EvictArgs {
    void* k_pool;
    void* v_pool;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* budgets;
    const int32_t* seen_lens;      // null: context_lens
    const int32_t* tracked_lens;   // null: zeros
    const int32_t* row_ids;        // null: the sequence's index
    const float* weights;
    float* weights_out;
    const int32_t* positions;
    int32_t* positions_out;
    int32_t* new_lens;
    int32_t* moves;   // workspace: [S][Hkv][5][max_context / 2]
    int* status;
    int64_t num_blocks;
    int64_t weights_stride;
    int num_rows;
    int max_blocks_per_seq;
    int block_shift;
    int max_context;
    int num_seqs;
    int num_kv_heads;
    int row_shift;   // log2 of a row's 16-byte chunks
    int sinks;
    int recent;
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

}  // namespace pkv

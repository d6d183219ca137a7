// C-ABI entry points of libpkv: argument validation, workspace carving and
// kernel launches.  Declarations and contracts are in include/pkv.h.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <algorithm>
#include <climits>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include <nvtx3/nvToolsExt.h>

#include "../../include/pkv.h"
#include "kernels.h"
#include "prefill_f32.h"

namespace {

constexpr int kChunk = 16;   // the kernels walk sequences in 16-token chunks
constexpr int kMaxDevices = 64;
constexpr double kLog2e = 1.4426950408889634;

// log2(block_size / 16) for the supported block sizes 16 and 32, else -1.
int chunk_shift(int block_size) { return block_size == 16 ? 0 : block_size == 32 ? 1 : -1; }

// Library device status word: first error code raised by a kernel (0 = none).
__device__ int g_pkv_status = 0;

std::mutex g_status_mu;
int* g_status_addr[kMaxDevices] = {nullptr};

// Device address of g_pkv_status on the current device, looked up once per device
// (a __device__ symbol's host-side name is not a device address).
int* status_word() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lk(g_status_mu);
    if (!g_status_addr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_pkv_status) != cudaSuccess) return nullptr;
        g_status_addr[dev] = static_cast<int*>(p);
    }
    return g_status_addr[dev];
}

std::mutex g_side_mu;
cudaStream_t g_side_stream[kMaxDevices] = {nullptr};

// A library-owned non-blocking stream per device, for work that runs beside the
// caller's stream inside one call (joined back before the call's last launch).  It has
// the greatest priority, so that its CTAs -- which need a whole SM's shared memory --
// are placed before the caller stream's kernel fills every SM.
cudaStream_t side_stream() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lk(g_side_mu);
    int least = 0, greatest = 0;
    if (!g_side_stream[dev] &&
        (cudaDeviceGetStreamPriorityRange(&least, &greatest) != cudaSuccess ||
         cudaStreamCreateWithPriority(&g_side_stream[dev], cudaStreamNonBlocking, greatest) !=
             cudaSuccess))
        g_side_stream[dev] = nullptr;
    return g_side_stream[dev];
}

cudaStream_t g_copy_stream[kMaxDevices][2] = {{nullptr, nullptr}};

// Two more library-owned non-blocking streams per device, for the copies of a host-buffer
// step that overlap its kernels on the caller's stream: 0 carries host-to-device copies,
// 1 device-to-host copies, so that both copy directions and the kernels run at once.
cudaStream_t copy_stream(int which) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lk(g_side_mu);
    cudaStream_t& s = g_copy_stream[dev][which];
    if (!s && cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) != cudaSuccess) s = nullptr;
    return s;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// An NVTX range around each call that enqueues GPU work, named after the call, so that
// a profiler's timeline groups the call's kernels under it and ncu can select them
// (--nvtx --nvtx-include "pkv_paged_decode/").  With no tool attached a push and a pop
// cost a few nanoseconds.
struct CallRange {
    explicit CallRange(const char* name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};

int elem_bytes(int dtype) { return dtype == PKV_BF16 ? 2 : 4; }

pkv_status check_pool(const pkv_pool_desc* pool) {
    if (!pool) return PKV_ERR_INVALID;
    if (pool->num_blocks <= 0 || pool->num_kv_heads <= 0 || pool->head_dim <= 0 ||
        pool->block_size <= 0)
        return PKV_ERR_INVALID;
    if (pool->dtype != PKV_F32 && pool->dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (chunk_shift(pool->block_size) < 0) return PKV_ERR_UNSUPPORTED;
    if (pool->head_dim != 64 && pool->head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (pool->num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
    if (pool->num_blocks > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

pkv_status from_cuda(cudaError_t e) { return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA; }

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// Partition policy for split-KV decode, in 16-token chunks: at least 64 chunks (1024
// tokens) per partition -- each CTA pays a fixed start-up (block ids, first copies
// in flight, merge), and on the Llama-3-8B-shaped batch 64 chunks measured best (16:
// 81 %, 32: 89 %, 64: 90 % of the copy bandwidth) -- and at most 64 partitions per
// sequence to bound the workspace; shrink partitions (down to 8 chunks) while fewer
// than 2 x 152 CTAs would be busy.  The result is a multiple of 4 chunks (one per warp
// per step) and so of 2 (a whole number of 32-token blocks): each halving rounds up to
// a multiple of 4.
// The CTA estimate counts ceil(Hq / 8) kv heads per sequence (a lower bound: a
// GQA group is at most 8 query heads) so that the choice, and with it the
// workspace size, depends only on (num_seqs, num_q_heads, max_context).
int auto_partition_chunks(int num_seqs, int num_q_heads, int max_context) {
    const int max_chunks = ceil_div(max_context, kChunk);
    const int64_t kv_heads_min = ceil_div(num_q_heads, 8);
    int pc = ceil_div(max_chunks, 64);
    if (pc < 64) pc = 64;
    pc = (pc + 3) / 4 * 4;
    while (pc > 8 && static_cast<int64_t>(num_seqs) * kv_heads_min * ceil_div(max_chunks, pc) <
                         304)
        pc = (pc / 2 + 3) / 4 * 4;
    return pc;
}

// The same in pool blocks.
int auto_partition(int num_seqs, int num_q_heads, int max_context, int block_size) {
    return auto_partition_chunks(num_seqs, num_q_heads, max_context) >> chunk_shift(block_size);
}

// bf16 decode runs on the tensor-core kernel; PKV_DECODE_KERNEL=simt selects the
// CUDA-core kernel instead (read at each call; used to test and compare the two).
bool decode_use_simt() {
    const char* v = std::getenv("PKV_DECODE_KERNEL");
    return v != nullptr && std::strcmp(v, "simt") == 0;
}

// Prefill probabilities: one bf16 value per weight for query tiles whose rows all
// attend at least kPSingleMinKeys keys, the exact hi + lo split below that;
// PKV_PREFILL_P=split forces the split everywhere (read at each call; used to test and
// compare the two).
constexpr int kPSingleMinKeys = 1024;
int prefill_p_single_min_keys() {
    const char* v = std::getenv("PKV_PREFILL_P");
    return (v != nullptr && std::strcmp(v, "split") == 0) ? INT_MAX : kPSingleMinKeys;
}

// PKV_TEST_DECODE_STALL=1 arms the decode kernels' timeout test hook (one wait of one
// warp runs out of time; read at each call; tests only).
int decode_test_stall() {
    const char* v = std::getenv("PKV_TEST_DECODE_STALL");
    return v != nullptr && std::strcmp(v, "1") == 0;
}

// PKV_TEST_PREFILL_WEIGHTS_STALL=1 or 2 does the same in that pass of the bf16 prompt weights
// (read at each call; tests only).
int prefill_weights_test_stall() {
    const char* v = std::getenv("PKV_TEST_PREFILL_WEIGHTS_STALL");
    return v == nullptr ? 0 : std::strcmp(v, "1") == 0 ? 1 : std::strcmp(v, "2") == 0 ? 2 : 0;
}

// PKV_TEST_CASCADE_SUFFIX_FAIL=1 makes the cascade decode report a failed suffix launch
// (without launching it) after its prefix pass was forked onto the side stream, so that
// tests reach that error path (read at each call; tests only).
bool cascade_test_fail_suffix() {
    const char* v = std::getenv("PKV_TEST_CASCADE_SUFFIX_FAIL");
    return v != nullptr && std::strcmp(v, "1") == 0;
}

size_t decode_workspace(int num_seqs, int num_q_heads, int head_dim, int max_parts) {
    if (max_parts <= 1) return 0;
    const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * max_parts;
    const size_t o = rows * head_dim * sizeof(float);
    const size_t ml = (rows * sizeof(float) + 15) / 16 * 16;
    return o + 2 * ml;
}

// Built-in decode scratch for pkv_paged_decode_noalloc: callers that cannot
// allocate device memory get the split-KV partials here.  The array is reserved on
// every GPU that loads this library's device code and held until the process exits.
constexpr size_t kNoAllocScratchBytes = 64u << 20;  // 64 MiB
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

std::mutex g_scratch_mu;
void* g_scratch_addr[kMaxDevices] = {nullptr};

// Device address of g_noalloc_scratch on the current device.  The host-side name
// of a __device__ array is only a stand-in, so the address is looked up once per
// device, with that device current, and cached; nullptr if the lookup fails.
void* noalloc_scratch() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lk(g_scratch_mu);
    if (!g_scratch_addr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess) return nullptr;
        g_scratch_addr[dev] = p;
    }
    return g_scratch_addr[dev];
}

}  // namespace

extern "C" {

const char* pkv_status_string(int status) {
    switch (status) {
        case PKV_OK: return "ok";
        case PKV_ERR_INVALID: return "invalid argument";
        case PKV_ERR_UNSUPPORTED: return "unsupported configuration";
        case PKV_ERR_CUDA: return "CUDA error";
        case PKV_ERR_TIMEOUT: return "device pipeline wait timed out";
        case PKV_ERR_OOB: return "slot or block id outside the pool";
        case PKV_ERR_NOMEM: return "out of blocks or workspace too small";
        case PKV_ERR_NOT_FOUND: return "unknown or duplicate sequence id";
        default: return "unknown status";
    }
}

int pkv_version(void) { return 100; }

uint64_t pkv_pool_bytes(const pkv_pool_desc* pool) {
    if (!pool || pool->num_blocks <= 0 || pool->block_size <= 0 || pool->num_kv_heads <= 0 ||
        pool->head_dim <= 0 || (pool->dtype != PKV_F32 && pool->dtype != PKV_BF16))
        return 0;
    return static_cast<uint64_t>(pool->num_blocks) * pool->num_kv_heads * pool->block_size *
           pool->head_dim * elem_bytes(pool->dtype);
}

pkv_status pkv_kv_append(const pkv_pool_desc* pool, void* k_pool, void* v_pool,
                         const int64_t* slot_mapping, const void* k, const void* v,
                         int64_t num_tokens, void* stream) {
    CallRange range("pkv_kv_append");
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (num_tokens < 0) return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (!k_pool || !v_pool || !slot_mapping || !k || !v) return PKV_ERR_INVALID;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k) || !aligned16(v))
        return PKV_ERR_INVALID;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;
    const int row_bytes = pool->head_dim * elem_bytes(pool->dtype);
    return from_cuda(pkv::launch_kv_append(k_pool, v_pool, slot_mapping, k, v, num_tokens,
                                           pool->num_kv_heads, row_bytes, pool->block_size,
                                           pool->num_blocks, status,
                                           static_cast<cudaStream_t>(stream)));
}

int pkv_paged_decode_auto_partition(int num_seqs, int num_q_heads, int max_context,
                                    int block_size) {
    if (num_seqs <= 0 || num_q_heads <= 0 || max_context <= 0 || chunk_shift(block_size) < 0)
        return 0;
    return auto_partition(num_seqs, num_q_heads, max_context, block_size);
}

size_t pkv_paged_decode_workspace_bytes(int num_seqs, int num_q_heads, int head_dim,
                                        int max_context, int block_size, int partition_blocks) {
    if (num_seqs <= 0 || num_q_heads <= 0 || head_dim <= 0 || max_context <= 0 ||
        chunk_shift(block_size) < 0 || partition_blocks < 0)
        return 0;
    const int pb = partition_blocks ? partition_blocks
                                    : auto_partition(num_seqs, num_q_heads, max_context, block_size);
    const int max_parts = ceil_div(ceil_div(max_context, block_size), pb);
    return decode_workspace(num_seqs, num_q_heads, head_dim, max_parts);
}

namespace {

// Where accumulated attention weights go (see pkv_paged_decode_weights).
struct WeightsOut {
    float* weights;
    int64_t stride;
    const int32_t* row_ids;
    int num_rows;
    float decay;
};

bool weights_ok(const WeightsOut& w, int num_seqs, int max_context) {
    return w.weights && w.stride >= max_context && w.num_rows > 0 &&
           (w.row_ids || w.num_rows >= num_seqs) && w.decay >= 0.f && w.decay <= 1.f &&
           aligned4(w.weights) && aligned4(w.row_ids);
}

// The scores are kept for whole partitions: none is longer than the context.
int weights_partition(int partition_blocks, int max_context, int block_size) {
    return std::min(partition_blocks, ceil_div(max_context, block_size));
}

size_t round16(size_t x) { return (x + 15) / 16 * 16; }

// Workspace of a decode with accumulated weights: the partials' outputs, m and l (none for
// one partition), and every score of the partitions' span.
struct WeightsWorkspace {
    size_t ml_at, scores_at, bytes;
    int score_tokens;
};
bool weights_workspace(int num_seqs, int num_q_heads, int head_dim, int max_parts,
                       int partition_chunks, WeightsWorkspace* w) {
    const int64_t span = static_cast<int64_t>(max_parts) * partition_chunks * kChunk;
    if (span > INT32_MAX) return false;
    const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads;
    w->score_tokens = static_cast<int>(span);
    w->ml_at = max_parts > 1 ? rows * max_parts * head_dim * sizeof(float) : 0;
    w->scores_at = w->ml_at + (max_parts > 1 ? 2 * round16(rows * max_parts * sizeof(float)) : 0);
    w->bytes = w->scores_at + rows * static_cast<size_t>(span) * sizeof(float);
    return true;
}

// pkv_paged_decode; with k_new / v_new set pkv_paged_decode_append; with `wo` set
// pkv_paged_decode_weights.
pkv_status decode_impl(const pkv_pool_desc* pool, void* out, const void* q, const void* k_pool,
                       const void* v_pool, const int32_t* block_tables, int max_blocks_per_seq,
                       const int32_t* context_lens, int max_context, int num_seqs,
                       int num_q_heads, float scale, int partition_blocks, void* workspace,
                       size_t workspace_bytes, const void* k_new, const void* v_new,
                       void* stream, const WeightsOut* wo = nullptr) {
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (num_seqs < 0 || num_q_heads <= 0 || partition_blocks < 0) return PKV_ERR_INVALID;
    if (num_seqs == 0) return PKV_OK;
    if (wo && !weights_ok(*wo, num_seqs, max_context)) return PKV_ERR_INVALID;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !context_lens)
        return PKV_ERR_INVALID;
    const int B = pool->block_size;
    if (max_blocks_per_seq <= 0 || max_context <= 0 ||
        static_cast<int64_t>(max_context) > static_cast<int64_t>(max_blocks_per_seq) * B)
        return PKV_ERR_INVALID;
    if (num_q_heads % pool->num_kv_heads != 0) return PKV_ERR_INVALID;
    const int group = num_q_heads / pool->num_kv_heads;
    if (group != 1 && group != 2 && group != 4 && group != 8) return PKV_ERR_UNSUPPORTED;
    if (num_seqs > 65535) return PKV_ERR_UNSUPPORTED;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool))
        return PKV_ERR_INVALID;

    int pb = partition_blocks ? partition_blocks
                              : auto_partition(num_seqs, num_q_heads, max_context, B);
    if (wo) pb = weights_partition(pb, max_context, B);
    const int max_parts = ceil_div(ceil_div(max_context, B), pb);
    if (max_parts > pkv::kMaxParts) return PKV_ERR_UNSUPPORTED;
    size_t need = decode_workspace(num_seqs, num_q_heads, pool->head_dim, max_parts);
    WeightsWorkspace ww{};
    if (wo) {
        if (!weights_workspace(num_seqs, num_q_heads, pool->head_dim, max_parts,
                               pb << chunk_shift(B), &ww))
            return PKV_ERR_UNSUPPORTED;
        need = ww.bytes;
    }
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
        return PKV_ERR_NOMEM;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;

    pkv::DecodeArgs a{};
    a.out = out;
    a.q = q;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.status = status;
    a.num_blocks = pool->num_blocks;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_seqs = num_seqs;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = pool->num_kv_heads;
    a.chunk_shift = chunk_shift(B);
    a.partition_chunks = pb << a.chunk_shift;
    a.max_parts = max_parts;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * kLog2e);
    a.k_new = k_new;
    a.v_new = v_new;
    if (need > 0) {
        const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * max_parts;
        const size_t ml = (rows * sizeof(float) + 15) / 16 * 16;
        char* w = static_cast<char*>(workspace);
        a.o_part = reinterpret_cast<float*>(w);
        a.m_part = reinterpret_cast<float*>(w + rows * pool->head_dim * sizeof(float));
        a.l_part = reinterpret_cast<float*>(w + rows * pool->head_dim * sizeof(float) + ml);
    }
    if (wo) {
        const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * max_parts;
        char* w = static_cast<char*>(workspace);
        a.m_part = reinterpret_cast<float*>(w + ww.ml_at);
        a.l_part = reinterpret_cast<float*>(w + ww.ml_at + round16(rows * sizeof(float)));
        a.scores = reinterpret_cast<float*>(w + ww.scores_at);
        a.score_tokens = ww.score_tokens;
        a.weights = wo->weights;
        a.row_ids = wo->row_ids;
        a.weights_stride = wo->stride;
        a.num_rows = wo->num_rows;
        a.decay = wo->decay;
    }
    const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
    a.test_stall = decode_test_stall();
    if (pool->dtype == PKV_BF16 && !decode_use_simt())
        return from_cuda(pkv::launch_paged_decode_tc(a, pool->head_dim, group, st_));
    return from_cuda(pkv::launch_paged_decode(a, pool->dtype, pool->head_dim, group, st_));
}

}  // namespace

pkv_status pkv_paged_decode(const pkv_pool_desc* pool, void* out, const void* q,
                            const void* k_pool, const void* v_pool,
                            const int32_t* block_tables, int max_blocks_per_seq,
                            const int32_t* context_lens, int max_context, int num_seqs,
                            int num_q_heads, float scale, int partition_blocks,
                            void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("pkv_paged_decode");
    return decode_impl(pool, out, q, k_pool, v_pool, block_tables, max_blocks_per_seq,
                       context_lens, max_context, num_seqs, num_q_heads, scale,
                       partition_blocks, workspace, workspace_bytes, nullptr, nullptr, stream);
}

pkv_status pkv_paged_decode_append(const pkv_pool_desc* pool, void* out, const void* q,
                                   void* k_pool, void* v_pool, const void* k_new,
                                   const void* v_new, const int32_t* block_tables,
                                   int max_blocks_per_seq, const int32_t* context_lens,
                                   int max_context, int num_seqs, int num_q_heads, float scale,
                                   int partition_blocks, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    CallRange range("pkv_paged_decode_append");
    if (num_seqs > 0 && (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)))
        return PKV_ERR_INVALID;
    return decode_impl(pool, out, q, k_pool, v_pool, block_tables, max_blocks_per_seq,
                       context_lens, max_context, num_seqs, num_q_heads, scale,
                       partition_blocks, workspace, workspace_bytes, k_new, v_new, stream);
}

namespace {

uint64_t round256(uint64_t x) { return (x + 255) / 256 * 256; }

// The address through which kernels reach host memory `p` in place, or nullptr.
// Page-locked memory from cudaHostAlloc / cudaMallocHost / cudaHostRegister is mapped
// into the device address space under unified addressing (on a Grace-Blackwell node
// the GPU then reads and writes it over NVLink-C2C); pageable memory is not.
void* mapped_host_ptr(const void* p) {
    cudaPointerAttributes a{};
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();   // a failed query is left as the last error: clear it
        return nullptr;
    }
    return a.type == cudaMemoryTypeHost ? a.devicePointer : nullptr;
}

}  // namespace

pkv_status pkv_decode_step_layout(const pkv_pool_desc* pool, int num_seqs, int num_q_heads,
                                  int max_blocks_per_seq, pkv_step_layout* layout) {
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (!layout || num_seqs < 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0)
        return PKV_ERR_INVALID;
    const uint64_t row = static_cast<uint64_t>(pool->head_dim) * elem_bytes(pool->dtype);
    const uint64_t S = static_cast<uint64_t>(num_seqs);
    uint64_t off = 0;
    layout->q = off;
    off = round256(off + S * num_q_heads * row);
    layout->k_new = off;
    off = round256(off + S * pool->num_kv_heads * row);
    layout->v_new = off;
    off = round256(off + S * pool->num_kv_heads * row);
    layout->block_tables = off;
    off = round256(off + S * max_blocks_per_seq * sizeof(int32_t));
    layout->context_lens = off;
    off = round256(off + S * sizeof(int32_t));
    layout->bytes = off;
    return PKV_OK;
}

size_t pkv_paged_decode_append_host_staging_bytes(const pkv_pool_desc* pool, int num_seqs,
                                                  int num_q_heads, int max_blocks_per_seq,
                                                  int max_context, int partition_blocks) {
    pkv_step_layout l;
    if (pkv_decode_step_layout(pool, num_seqs, num_q_heads, max_blocks_per_seq, &l) != PKV_OK ||
        num_seqs <= 0 || max_context <= 0 || partition_blocks < 0)
        return 0;
    const uint64_t out = round256(static_cast<uint64_t>(num_seqs) * num_q_heads *
                                  pool->head_dim * elem_bytes(pool->dtype));
    return l.bytes + out +
           pkv_paged_decode_workspace_bytes(num_seqs, num_q_heads, pool->head_dim, max_context,
                                            pool->block_size, partition_blocks);
}

pkv_status pkv_paged_decode_append_host(const pkv_pool_desc* pool, void* k_pool, void* v_pool,
                                        const void* host_in, void* host_out,
                                        int max_blocks_per_seq, int max_context, int num_seqs,
                                        int num_q_heads, float scale, int partition_blocks,
                                        void* staging, size_t staging_bytes, void* stream) {
    CallRange range("pkv_paged_decode_append_host");
    pkv_step_layout l;
    pkv_status st = pkv_decode_step_layout(pool, num_seqs, num_q_heads, max_blocks_per_seq, &l);
    if (st != PKV_OK) return st;
    if (num_seqs == 0) return PKV_OK;
    if (!host_in || !host_out || !staging || (reinterpret_cast<uintptr_t>(staging) & 255u))
        return PKV_ERR_INVALID;
    if (max_context <= 0 || partition_blocks < 0) return PKV_ERR_INVALID;
    const size_t need = pkv_paged_decode_append_host_staging_bytes(
        pool, num_seqs, num_q_heads, max_blocks_per_seq, max_context, partition_blocks);
    if (need == 0) return PKV_ERR_INVALID;
    if (staging_bytes < need) return PKV_ERR_NOMEM;
    const uint64_t out_bytes = static_cast<uint64_t>(num_seqs) * num_q_heads * pool->head_dim *
                               elem_bytes(pool->dtype);
    char* dev = static_cast<char*>(staging);
    char* out = dev + l.bytes;
    char* ws = out + round256(out_bytes);
    const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
    // Mapped (page-locked) host buffers are read and written by the kernels in place;
    // any other host memory, or a buffer not 16-byte aligned (the kernels' vector
    // accesses need that), goes through the staging buffer with one copy each way.
    const char* in = static_cast<const char*>(mapped_host_ptr(host_in));
    char* out_map = static_cast<char*>(mapped_host_ptr(host_out));
    if (!aligned16(in)) in = nullptr;
    if (!aligned16(out_map)) out_map = nullptr;
    if (!in) {
        if (cudaMemcpyAsync(dev, host_in, l.bytes, cudaMemcpyHostToDevice, st_) != cudaSuccess)
            return PKV_ERR_CUDA;
        in = dev;
    }
    st = pkv_paged_decode_append(pool, out_map ? out_map : out, in + l.q, k_pool, v_pool,
                                 in + l.k_new, in + l.v_new,
                                 reinterpret_cast<const int32_t*>(in + l.block_tables),
                                 max_blocks_per_seq,
                                 reinterpret_cast<const int32_t*>(in + l.context_lens),
                                 max_context, num_seqs, num_q_heads, scale, partition_blocks, ws,
                                 need - (ws - dev), stream);
    if (st != PKV_OK || out_map) return st;
    return from_cuda(cudaMemcpyAsync(host_out, out, out_bytes, cudaMemcpyDeviceToHost, st_));
}

pkv_status pkv_paged_decode_noalloc(const pkv_pool_desc* pool, void* out, const void* q,
                                    const void* k_pool, const void* v_pool,
                                    const int32_t* block_tables, int max_blocks_per_seq,
                                    const int32_t* context_lens, int max_context, int num_seqs,
                                    int num_q_heads, float scale, int partition_blocks,
                                    void* stream) {
    CallRange range("pkv_paged_decode_noalloc");
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (num_seqs < 0 || num_q_heads <= 0 || partition_blocks < 0 || max_context <= 0)
        return PKV_ERR_INVALID;
    if (num_seqs == 0) return PKV_OK;
    const size_t need = pkv_paged_decode_workspace_bytes(
        num_seqs, num_q_heads, pool->head_dim, max_context, pool->block_size, partition_blocks);
    if (need > kNoAllocScratchBytes) return PKV_ERR_NOMEM;
    void* scratch = nullptr;
    if (need > 0) {
        scratch = noalloc_scratch();
        if (!scratch) return PKV_ERR_CUDA;
    }
    return pkv_paged_decode(pool, out, q, k_pool, v_pool, block_tables, max_blocks_per_seq,
                            context_lens, max_context, num_seqs, num_q_heads, scale,
                            partition_blocks, scratch, need, stream);
}

namespace {

// Splits of the cascade decode's prefix pass over its 128-key tiles.  The pass has about
// ceil(S * Hq / 128) CTAs (query tiles times kv heads), each needing a whole SM, and runs
// beside the suffix decode, which is HBM-bound and wants the other SMs: its tiles are
// divided among as many CTAs per query tile (up to 8, none empty) as keep the pass within
// half the SMs (76).  On the shared-prefix batch (64 query tiles) 1, 2, 3 and 4 splits
// measured 113, 121, 125 and 128 us.  Depends only on (num_seqs, num_q_heads, prefix_len).
int cascade_splits(int num_seqs, int num_q_heads, int prefix_len, int* tiles_per_split) {
    const int tiles = ceil_div(prefix_len, 128);
    const int ctas = ceil_div(static_cast<int64_t>(num_seqs) * num_q_heads, 128);
    int ns = 76 / ctas;
    ns = std::max(1, std::min(ns, std::min(8, tiles)));
    const int tps = ceil_div(tiles, ns);
    *tiles_per_split = tps;
    return ceil_div(tiles, tps);
}

}  // namespace

size_t pkv_paged_decode_cascade_workspace_bytes(int num_seqs, int num_q_heads, int head_dim,
                                                int prefix_len, int max_context, int block_size,
                                                int partition_blocks) {
    if (num_seqs <= 0 || num_q_heads <= 0 || head_dim <= 0 || prefix_len <= 0 ||
        max_context < prefix_len || chunk_shift(block_size) < 0 || partition_blocks < 0)
        return 0;
    const int suffix = max_context - prefix_len;
    const int pb = partition_blocks
                       ? partition_blocks
                       : (suffix > 0 ? auto_partition(num_seqs, num_q_heads, suffix, block_size) : 1);
    const int parts = suffix > 0 ? ceil_div(ceil_div(suffix, block_size), pb) : 0;
    int tps = 0;
    const int ns = cascade_splits(num_seqs, num_q_heads, prefix_len, &tps);
    const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * (parts + ns);
    const size_t ml = (rows * sizeof(float) + 15) / 16 * 16;
    return rows * head_dim * sizeof(float) + 2 * ml;
}

namespace {

// pkv_paged_decode_cascade, and with k_new / v_new set pkv_paged_decode_cascade_append
// (the suffix decode stores and attends each sequence's newest token).
pkv_status cascade_impl(const pkv_pool_desc* pool, void* out, const void* q, const void* k_pool,
                        const void* v_pool, const int32_t* prefix_blocks, int prefix_len,
                        const int32_t* block_tables, int max_blocks_per_seq,
                        const int32_t* context_lens, int max_context, int num_seqs,
                        int num_q_heads, float scale, int partition_blocks, void* workspace,
                        size_t workspace_bytes, const void* k_new, const void* v_new,
                        void* stream) {
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (num_seqs < 0 || num_q_heads <= 0 || partition_blocks < 0 || !(scale > 0.f))
        return PKV_ERR_INVALID;
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !k_pool || !v_pool || !prefix_blocks || !block_tables || !context_lens)
        return PKV_ERR_INVALID;
    const int B = pool->block_size;
    if (prefix_len <= 0 || prefix_len % B != 0 || max_context < prefix_len ||
        max_blocks_per_seq <= 0 ||
        static_cast<int64_t>(max_context) > static_cast<int64_t>(max_blocks_per_seq) * B)
        return PKV_ERR_INVALID;
    if (num_q_heads % pool->num_kv_heads != 0) return PKV_ERR_INVALID;
    const int group = num_q_heads / pool->num_kv_heads;
    if (pool->dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (group != 1 && group != 2 && group != 4 && group != 8) return PKV_ERR_UNSUPPORTED;
    if (num_seqs > 65535) return PKV_ERR_UNSUPPORTED;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool))
        return PKV_ERR_INVALID;
    const int suffix = max_context - prefix_len;
    const int pb = partition_blocks
                       ? partition_blocks
                       : (suffix > 0 ? auto_partition(num_seqs, num_q_heads, suffix, B) : 1);
    const int parts = suffix > 0 ? ceil_div(ceil_div(suffix, B), pb) : 0;
    int tps = 0;
    const int ns = cascade_splits(num_seqs, num_q_heads, prefix_len, &tps);
    if (parts + ns > pkv::kMaxParts) return PKV_ERR_UNSUPPORTED;
    const size_t need = pkv_paged_decode_cascade_workspace_bytes(
        num_seqs, num_q_heads, pool->head_dim, prefix_len, max_context, B, partition_blocks);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return PKV_ERR_NOMEM;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;
    const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * (parts + ns);
    const size_t ml = (rows * sizeof(float) + 15) / 16 * 16;
    char* w = static_cast<char*>(workspace);
    float* o_part = reinterpret_cast<float*>(w);
    float* m_part = reinterpret_cast<float*>(w + rows * pool->head_dim * sizeof(float));
    float* l_part = reinterpret_cast<float*>(w + rows * pool->head_dim * sizeof(float) + ml);
    const float sl2 = static_cast<float>(static_cast<double>(scale) * kLog2e);
    const cudaStream_t st_ = static_cast<cudaStream_t>(stream);

    // 1. every sequence's query heads against the shared prefix, on the tensor cores
    pkv::PrefillArgs pa{};
    pa.head_dim = pool->head_dim;
    pa.block_size = B;
    pa.q = q;
    pa.k_pool = k_pool;
    pa.v_pool = v_pool;
    pa.block_tables = prefix_blocks;
    pa.status = status;
    pa.num_blocks = pool->num_blocks;
    pa.max_blocks_per_seq = prefix_len / B;
    pa.num_reqs = ns;   // grid z: one per split of the prefix's tiles
    pa.total_new = num_seqs;
    pa.max_new = num_seqs;
    pa.num_q_heads = num_q_heads;
    pa.num_kv_heads = pool->num_kv_heads;
    pa.scale_log2 = sl2;
    pa.cascade = 1;
    pa.cascade_keys = prefix_len;
    pa.cascade_rows = num_seqs;
    pa.cascade_tiles_per_split = tps;
    pa.max_parts_total = parts + ns;
    pa.p_single_min_keys = prefill_p_single_min_keys();
    pa.o_part = o_part;
    pa.m_part = m_part;
    pa.l_part = l_part;
    // The prefix pass (tensor-bound, its K/V L2-resident) runs on a side stream beside
    // the suffix decode (HBM-bound); the combine waits for both.
    cudaStream_t side = side_stream();
    if (!side) return PKV_ERR_CUDA;
    cudaEvent_t fork = nullptr, join = nullptr;
    if (cudaEventCreateWithFlags(&fork, cudaEventDisableTiming) != cudaSuccess)
        return PKV_ERR_CUDA;
    if (cudaEventCreateWithFlags(&join, cudaEventDisableTiming) != cudaSuccess) {
        cudaEventDestroy(fork);
        return PKV_ERR_CUDA;
    }
    struct Events {   // released once their work completes
        cudaEvent_t a, b;
        ~Events() { cudaEventDestroy(a); cudaEventDestroy(b); }
    } ev{fork, join};
    if (cudaEventRecord(fork, st_) != cudaSuccess || cudaStreamWaitEvent(side, fork, 0) != cudaSuccess)
        return PKV_ERR_CUDA;
    // From here on the side stream carries this call's work: every exit, the error
    // returns included, makes the caller's stream wait for it, so that no work of the call
    // runs on past its return unordered with the caller's stream, and a stream capture
    // ends with the side stream joined back.
    struct Rejoin {
        cudaStream_t side, st;
        cudaEvent_t ev;
        bool recorded = false, waited = false;
        cudaError_t record() {
            recorded = true;
            return cudaEventRecord(ev, side);
        }
        cudaError_t wait() {
            cudaError_t e = recorded ? cudaSuccess : record();
            waited = true;
            const cudaError_t w = cudaStreamWaitEvent(st, ev, 0);
            return e != cudaSuccess ? e : w;
        }
        ~Rejoin() {
            if (!waited) wait();
        }
    } rejoin{side, st_, join};
    cudaError_t e = pkv::launch_paged_prefill(pa, group, side);
    if (e != cudaSuccess) return e == cudaErrorNotSupported ? PKV_ERR_UNSUPPORTED : PKV_ERR_CUDA;
    if (rejoin.record() != cudaSuccess) return PKV_ERR_CUDA;

    // 2. private suffixes (blocks from prefix_len / B on) + 3. log-sum-exp merge
    pkv::DecodeArgs a{};
    a.out = out;
    a.q = q;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.status = status;
    a.num_blocks = pool->num_blocks;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_seqs = num_seqs;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = pool->num_kv_heads;
    a.chunk_shift = chunk_shift(B);
    a.partition_chunks = pb << a.chunk_shift;
    a.max_parts = parts;
    a.scale_log2 = sl2;
    a.o_part = o_part;
    a.m_part = m_part;
    a.l_part = l_part;
    a.chunk_offset = prefix_len / kChunk;
    a.extra_parts = ns;
    a.defer_combine = 1;
    a.no_pdl = 1;
    a.k_new = k_new;
    a.v_new = v_new;
    if (cascade_test_fail_suffix()) return PKV_ERR_CUDA;   // test hook: the rejoin still runs
    e = decode_use_simt() ? pkv::launch_paged_decode(a, pool->dtype, pool->head_dim, group, st_)
                          : pkv::launch_paged_decode_tc(a, pool->head_dim, group, st_);
    if (e != cudaSuccess) return e == cudaErrorNotSupported ? PKV_ERR_UNSUPPORTED : PKV_ERR_CUDA;
    if (rejoin.wait() != cudaSuccess) return PKV_ERR_CUDA;
    return from_cuda(pkv::launch_decode_combine(a, pool->dtype, pool->head_dim, st_));
}

}  // namespace

pkv_status pkv_paged_decode_cascade(const pkv_pool_desc* pool, void* out, const void* q,
                                    const void* k_pool, const void* v_pool,
                                    const int32_t* prefix_blocks, int prefix_len,
                                    const int32_t* block_tables, int max_blocks_per_seq,
                                    const int32_t* context_lens, int max_context, int num_seqs,
                                    int num_q_heads, float scale, int partition_blocks,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("pkv_paged_decode_cascade");
    return cascade_impl(pool, out, q, k_pool, v_pool, prefix_blocks, prefix_len, block_tables,
                        max_blocks_per_seq, context_lens, max_context, num_seqs, num_q_heads,
                        scale, partition_blocks, workspace, workspace_bytes, nullptr, nullptr,
                        stream);
}

pkv_status pkv_paged_decode_cascade_append(const pkv_pool_desc* pool, void* out, const void* q,
                                           void* k_pool, void* v_pool, const void* k_new,
                                           const void* v_new, const int32_t* prefix_blocks,
                                           int prefix_len, const int32_t* block_tables,
                                           int max_blocks_per_seq, const int32_t* context_lens,
                                           int max_context, int num_seqs, int num_q_heads,
                                           float scale, int partition_blocks, void* workspace,
                                           size_t workspace_bytes, void* stream) {
    CallRange range("pkv_paged_decode_cascade_append");
    if (num_seqs > 0 && (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)))
        return PKV_ERR_INVALID;
    return cascade_impl(pool, out, q, k_pool, v_pool, prefix_blocks, prefix_len, block_tables,
                        max_blocks_per_seq, context_lens, max_context, num_seqs, num_q_heads,
                        scale, partition_blocks, workspace, workspace_bytes, k_new, v_new,
                        stream);
}

pkv_status pkv_paged_prefill(const pkv_pool_desc* pool, void* out, const void* q,
                             const void* k_pool, const void* v_pool,
                             const int32_t* block_tables, int max_blocks_per_seq,
                             const int32_t* cached_lens, const int32_t* new_lens,
                             const int32_t* q_offsets, int num_reqs, int total_new, int max_new,
                             int num_q_heads, float scale, void* stream) {
    CallRange range("pkv_paged_prefill");
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (num_reqs < 0 || total_new < 0 || max_new < 0 || num_q_heads <= 0 || !(scale > 0.f))
        return PKV_ERR_INVALID;
    if (num_reqs == 0 || total_new == 0 || max_new == 0) return PKV_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !cached_lens || !new_lens ||
        !q_offsets || max_blocks_per_seq <= 0)
        return PKV_ERR_INVALID;
    if (num_q_heads % pool->num_kv_heads != 0) return PKV_ERR_INVALID;
    const int group = num_q_heads / pool->num_kv_heads;
    if (group != 1 && group != 2 && group != 4 && group != 8) return PKV_ERR_UNSUPPORTED;
    if (num_reqs > 65535) return PKV_ERR_UNSUPPORTED;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool))
        return PKV_ERR_INVALID;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;
    pkv::PrefillArgs a{};
    a.head_dim = pool->head_dim;
    a.block_size = pool->block_size;
    a.out = out;
    a.q = q;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.block_tables = block_tables;
    a.cached_lens = cached_lens;
    a.new_lens = new_lens;
    a.q_offsets = q_offsets;
    a.status = status;
    a.num_blocks = pool->num_blocks;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_reqs = num_reqs;
    a.total_new = total_new;
    a.max_new = max_new;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = pool->num_kv_heads;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * kLog2e);
    a.p_single_min_keys = prefill_p_single_min_keys();
    // fp32 pools run on the CUDA cores: the tensor cores would round fp32 operands to tf32.
    const cudaError_t e =
        pool->dtype == PKV_F32
            ? pkv::launch_paged_prefill_f32(a, group, static_cast<cudaStream_t>(stream))
            : pkv::launch_paged_prefill(a, group, static_cast<cudaStream_t>(stream));
    if (e == cudaErrorNotSupported) return PKV_ERR_UNSUPPORTED;
    return from_cuda(e);
}

pkv_status pkv_prefill_step_layout(const pkv_pool_desc* pool, int num_reqs, int total_new,
                                   int num_q_heads, int max_blocks_per_seq,
                                   pkv_prefill_layout* layout) {
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (!layout || num_reqs < 0 || total_new < 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0)
        return PKV_ERR_INVALID;
    const uint64_t row = static_cast<uint64_t>(pool->head_dim) * elem_bytes(pool->dtype);
    const uint64_t R = static_cast<uint64_t>(num_reqs);
    const uint64_t T = static_cast<uint64_t>(total_new);
    uint64_t off = 0;
    layout->q = off;
    off = round256(off + T * num_q_heads * row);
    layout->block_tables = off;
    off = round256(off + R * max_blocks_per_seq * sizeof(int32_t));
    layout->cached_lens = off;
    off = round256(off + R * sizeof(int32_t));
    layout->new_lens = off;
    off = round256(off + R * sizeof(int32_t));
    layout->q_offsets = off;
    off = round256(off + (R + 1) * sizeof(int32_t));
    layout->copied_bytes = off;
    layout->k_new = off;
    off = round256(off + T * pool->num_kv_heads * row);
    layout->v_new = off;
    off = round256(off + T * pool->num_kv_heads * row);
    layout->slot_mapping = off;
    off = round256(off + T * sizeof(int64_t));
    layout->bytes = off;
    return PKV_OK;
}

size_t pkv_paged_prefill_append_host_staging_bytes(const pkv_pool_desc* pool, int num_reqs,
                                                   int total_new, int num_q_heads,
                                                   int max_blocks_per_seq) {
    pkv_prefill_layout l;
    if (pkv_prefill_step_layout(pool, num_reqs, total_new, num_q_heads, max_blocks_per_seq,
                                &l) != PKV_OK)
        return 0;
    const uint64_t out = round256(static_cast<uint64_t>(total_new) * num_q_heads *
                                  pool->head_dim * elem_bytes(pool->dtype));
    return l.bytes + out;
}

pkv_status pkv_paged_prefill_append_host(const pkv_pool_desc* pool, void* k_pool, void* v_pool,
                                         const void* host_in, void* host_out, int num_reqs,
                                         int total_new, int max_new, int num_q_heads,
                                         int max_blocks_per_seq, float scale, void* staging,
                                         size_t staging_bytes, void* stream) {
    CallRange range("pkv_paged_prefill_append_host");
    pkv_prefill_layout l;
    pkv_status st =
        pkv_prefill_step_layout(pool, num_reqs, total_new, num_q_heads, max_blocks_per_seq, &l);
    if (st != PKV_OK) return st;
    if (num_reqs == 0 || total_new == 0) return PKV_OK;
    if (!host_in || !host_out || !staging || (reinterpret_cast<uintptr_t>(staging) & 255u))
        return PKV_ERR_INVALID;
    const size_t need = pkv_paged_prefill_append_host_staging_bytes(
        pool, num_reqs, total_new, num_q_heads, max_blocks_per_seq);
    if (need == 0) return PKV_ERR_INVALID;
    if (staging_bytes < need) return PKV_ERR_NOMEM;
    const char* hin = static_cast<const char*>(host_in);
    const int32_t* qoff = reinterpret_cast<const int32_t*>(hin + l.q_offsets);
    if (qoff[0] != 0 || qoff[num_reqs] != total_new) return PKV_ERR_INVALID;
    for (int r = 0; r < num_reqs; ++r)
        if (qoff[r + 1] < qoff[r]) return PKV_ERR_INVALID;
    char* dev = static_cast<char*>(staging);
    char* out = dev + l.bytes;
    const uint64_t esz = elem_bytes(pool->dtype);
    const uint64_t qrow = static_cast<uint64_t>(num_q_heads) * pool->head_dim * esz;
    const uint64_t kvrow = static_cast<uint64_t>(pool->num_kv_heads) * pool->head_dim * esz;
    const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
    // Every input goes to the device by copy (the prefill loads q by TMA) and the output
    // comes back by copy, chunk by chunk, on two library streams beside the kernels.  On
    // the 16 x 512-token batch the link moves about 200 GB/s each way, whether copy
    // engines or SMs drive it; read in place by the append kernel, the new rows cost
    // more on the kernels' stream than their copy does beside it, and stored in place the
    // prefill's output tiles held the kernel up (1.23 -> 1.87 ms a step unchunked).
    // Requests in up to kChunks chunks of about equal new rows: chunk c's query rows are
    // copied in on one copy stream while chunk c - 1's append and prefill run on `stream`
    // and chunk c - 2's output is copied back on the other.
    constexpr int kChunks = 4;
    int bounds[kChunks + 1];
    int nch = 0;
    bounds[0] = 0;
    for (int c = 1; c <= kChunks && bounds[nch] < num_reqs; ++c) {
        const int64_t target = static_cast<int64_t>(total_new) * c / kChunks;
        int r = bounds[nch] + 1;
        while (r < num_reqs && qoff[r] < target) ++r;
        if (c == kChunks) r = num_reqs;
        bounds[++nch] = r;
    }
    cudaStream_t cin = copy_stream(0), cout = copy_stream(1);
    if (!cin || !cout) return PKV_ERR_CUDA;
    struct Events {   // the fork, two per chunk and the two joins
        cudaEvent_t e[2 * kChunks + 3] = {};
        int n = 0;
        cudaEvent_t make() {
            cudaEvent_t ev = nullptr;
            if (n < 2 * kChunks + 3 &&
                cudaEventCreateWithFlags(&ev, cudaEventDisableTiming) == cudaSuccess)
                e[n++] = ev;
            return ev;
        }
        ~Events() {   // released once their work completes
            for (int i = 0; i < n; ++i) cudaEventDestroy(e[i]);
        }
    } ev;
    cudaEvent_t fork = ev.make();
    if (!fork || cudaEventRecord(fork, st_) != cudaSuccess ||
        cudaStreamWaitEvent(cin, fork, 0) != cudaSuccess ||
        cudaStreamWaitEvent(cout, fork, 0) != cudaSuccess)
        return PKV_ERR_CUDA;
    // From here on the copy streams carry this call's work: every exit makes `stream` wait
    // for both, so that nothing of the call runs on past it unordered and a stream capture
    // ends with them joined.
    struct Rejoin {
        cudaStream_t a, b, st;
        Events* ev;
        ~Rejoin() {
            for (cudaStream_t s : {a, b}) {
                cudaEvent_t j = ev->make();
                if (j && cudaEventRecord(j, s) == cudaSuccess) cudaStreamWaitEvent(st, j, 0);
            }
        }
    } rejoin{cin, cout, st_, &ev};
    // the control arrays, then chunk by chunk q, the new rows and their slots
    if (cudaMemcpyAsync(dev + l.block_tables, hin + l.block_tables,
                        l.copied_bytes - l.block_tables, cudaMemcpyHostToDevice, cin) != cudaSuccess)
        return PKV_ERR_CUDA;
    cudaEvent_t in_done[kChunks];
    for (int c = 0; c < nch; ++c) {
        const uint64_t t0 = qoff[bounds[c]], t1 = qoff[bounds[c + 1]];
        const struct { uint64_t off, row; } parts[4] = {
            {l.q, qrow}, {l.k_new, kvrow}, {l.v_new, kvrow}, {l.slot_mapping, sizeof(int64_t)}};
        for (const auto& pt : parts)
            if (t1 > t0 && cudaMemcpyAsync(dev + pt.off + t0 * pt.row, hin + pt.off + t0 * pt.row,
                                           (t1 - t0) * pt.row, cudaMemcpyHostToDevice,
                                           cin) != cudaSuccess)
                return PKV_ERR_CUDA;
        in_done[c] = ev.make();
        if (!in_done[c] || cudaEventRecord(in_done[c], cin) != cudaSuccess) return PKV_ERR_CUDA;
    }
    const int32_t* dbt = reinterpret_cast<const int32_t*>(dev + l.block_tables);
    const int32_t* dcl = reinterpret_cast<const int32_t*>(dev + l.cached_lens);
    const int32_t* dnl = reinterpret_cast<const int32_t*>(dev + l.new_lens);
    const int32_t* dqo = reinterpret_cast<const int32_t*>(dev + l.q_offsets);
    const char* rows = dev;
    const int64_t* slots = reinterpret_cast<const int64_t*>(rows + l.slot_mapping);
    for (int c = 0; c < nch; ++c) {
        const int r0 = bounds[c], r1 = bounds[c + 1];
        const int64_t t0 = qoff[r0], t1 = qoff[r1];
        if (cudaStreamWaitEvent(st_, in_done[c], 0) != cudaSuccess) return PKV_ERR_CUDA;
        st = pkv_kv_append(pool, k_pool, v_pool, slots + t0, rows + l.k_new + t0 * kvrow,
                           rows + l.v_new + t0 * kvrow, t1 - t0, stream);
        if (st != PKV_OK) return st;
        // the chunk's requests; q_offsets stay absolute rows of the whole q and out
        st = pkv_paged_prefill(pool, out, dev + l.q, k_pool, v_pool,
                               dbt + static_cast<size_t>(r0) * max_blocks_per_seq,
                               max_blocks_per_seq, dcl + r0, dnl + r0, dqo + r0, r1 - r0,
                               total_new, max_new, num_q_heads, scale, stream);
        if (st != PKV_OK) return st;
        cudaEvent_t done = ev.make();
        if (!done || cudaEventRecord(done, st_) != cudaSuccess ||
            cudaStreamWaitEvent(cout, done, 0) != cudaSuccess)
            return PKV_ERR_CUDA;
        if (t1 > t0 && cudaMemcpyAsync(static_cast<char*>(host_out) + t0 * qrow, out + t0 * qrow,
                                       (t1 - t0) * qrow, cudaMemcpyDeviceToHost, cout) != cudaSuccess)
            return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

size_t pkv_paged_decode_weights_workspace_bytes(const pkv_pool_desc* pool, int num_seqs,
                                                int num_q_heads, int max_context,
                                                int partition_blocks) {
    if (check_pool(pool) != PKV_OK || num_seqs <= 0 || num_q_heads <= 0 || max_context <= 0 ||
        partition_blocks < 0)
        return 0;
    const int B = pool->block_size;
    const int pb = weights_partition(partition_blocks
                                         ? partition_blocks
                                         : auto_partition(num_seqs, num_q_heads, max_context, B),
                                     max_context, B);
    WeightsWorkspace w;
    return weights_workspace(num_seqs, num_q_heads, pool->head_dim,
                             ceil_div(ceil_div(max_context, B), pb), pb << chunk_shift(B), &w)
               ? w.bytes
               : 0;
}

pkv_status pkv_paged_decode_weights(const pkv_pool_desc* pool, void* out, const void* q,
                                    void* k_pool, void* v_pool, const void* k_new,
                                    const void* v_new, const int32_t* block_tables,
                                    int max_blocks_per_seq, const int32_t* context_lens,
                                    int max_context, int num_seqs, int num_q_heads, float scale,
                                    int partition_blocks, float* weights, int64_t weights_stride,
                                    const int32_t* row_ids, int num_rows, float decay,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("pkv_paged_decode_weights");
    if (num_seqs > 0 && (!k_new != !v_new || !aligned16(k_new) || !aligned16(v_new)))
        return PKV_ERR_INVALID;
    const WeightsOut wo{weights, weights_stride, row_ids, num_rows, decay};
    return decode_impl(pool, out, q, k_pool, v_pool, block_tables, max_blocks_per_seq,
                       context_lens, max_context, num_seqs, num_q_heads, scale,
                       partition_blocks, workspace, workspace_bytes, k_new, v_new, stream, &wo);
}

namespace {

int block_shift(int block_size) { return 4 + chunk_shift(block_size); }

// Token stride of a row array: whole 16-byte chunks.
bool stride_ok(int64_t stride, int64_t least, int es) {
    return stride >= least && (stride * es) % 16 == 0;
}

// n rows of `bytes` each, `step` bytes apart (0: the same row n times).
struct Rows {
    const void* at;
    int64_t step, bytes;
};
// Whether n rows `out` have no byte in common with n rows `in`: a kernel's CTAs read and write
// them in any order.  Rows of one step may lie between one another (slices of one projection).
bool rows_apart(const Rows& out, const Rows& in, int64_t n) {
    const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(in.at) -
                                           reinterpret_cast<uintptr_t>(out.at));
    if (d >= (n - 1) * out.step + out.bytes || -d >= (n - 1) * in.step + in.bytes) return true;
    // The first row of `out`, from row `first` on, that ends behind a row of `in` which begins e
    // bytes from out's row 0: apart where it is none of them or begins behind that row.
    const int64_t step = std::max<int64_t>(out.step, 1);
    auto apart_from = [&](int64_t e, int64_t first) {
        const int64_t gap = e - out.bytes;
        const int64_t below = gap >= 0 ? gap / step : -((-gap + step - 1) / step);   // rounded down
        const int64_t u = std::max(below + 1, first);
        return u >= n || u * step >= e + in.bytes;
    };
    if (in.step == out.step) return apart_from(d, 1 - n);   // by the difference of the rows' numbers
    for (int64_t t = 0; t < (in.step ? n : 1); ++t)
        if (!apart_from(d + t * in.step, 0)) return false;
    return true;
}
// The same rows, turned in place, or apart.
bool same_or_rows_apart(const Rows& out, const Rows& in, int64_t n) {
    return (out.at == in.at && (out.step == in.step || n == 1)) || rows_apart(out, in, n);
}

}  // namespace

pkv_status pkv_rope(int dtype, void* out, int64_t out_stride, const void* x, int64_t x_stride,
                    const int32_t* positions, const double* inv_freq, int rotary_dim,
                    int interleaved, int inverse, float attn_scale, int64_t num_tokens,
                    int num_heads, int head_dim, void* stream) {
    CallRange range("pkv_rope");
    if (num_tokens < 0 || num_heads <= 0 || head_dim <= 0 || rotary_dim <= 0)
        return PKV_ERR_INVALID;
    if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if ((head_dim != 64 && head_dim != 128) || rotary_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
    if (rotary_dim > head_dim) return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (num_tokens > INT32_MAX || num_heads > 1 << 20) return PKV_ERR_UNSUPPORTED;
    if (!out || !x || !positions || !inv_freq || !aligned16(out) || !aligned16(x) ||
        !aligned4(positions) || !aligned8(inv_freq))
        return PKV_ERR_INVALID;
    const int es = elem_bytes(dtype);
    if (!stride_ok(out_stride, static_cast<int64_t>(num_heads) * head_dim, es) ||
        !stride_ok(x_stride, 0, es))
        return PKV_ERR_INVALID;
    const int64_t row = static_cast<int64_t>(num_heads) * head_dim * es;
    if (!same_or_rows_apart({out, out_stride * es, row}, {x, x_stride * es, row}, num_tokens))
        return PKV_ERR_INVALID;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;
    pkv::RopeArgs a{};
    a.q = x;
    a.k = x;
    a.v = x;
    a.q_out = out;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.status = status;
    a.q_stride = x_stride;
    a.q_out_stride = out_stride;
    a.num_tokens = num_tokens;
    a.num_q_heads = num_heads;
    a.rotary_dim = rotary_dim;
    a.interleaved = interleaved != 0;
    a.inverse = inverse != 0;
    a.attn_scale = attn_scale;
    return from_cuda(
        pkv::launch_rope(a, dtype, head_dim, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_rope_append(const pkv_pool_desc* pool, void* k_pool, void* v_pool,
                           const int64_t* slot_mapping, void* q_out, int64_t q_out_stride,
                           const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, const int32_t* positions,
                           const double* inv_freq, int rotary_dim, int interleaved,
                           float attn_scale, int64_t num_tokens, int num_q_heads, void* stream) {
    CallRange range("pkv_rope_append");
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (num_tokens < 0 || num_q_heads <= 0 || rotary_dim <= 0) return PKV_ERR_INVALID;
    if (rotary_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
    if (rotary_dim > pool->head_dim) return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (num_tokens > INT32_MAX || num_q_heads > 1 << 20) return PKV_ERR_UNSUPPORTED;
    if (!k_pool || !v_pool || !slot_mapping || !q_out || !q || !k || !v || !positions || !inv_freq)
        return PKV_ERR_INVALID;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(q_out) || !aligned16(q) ||
        !aligned16(k) || !aligned16(v) || !aligned8(slot_mapping) || !aligned4(positions) ||
        !aligned8(inv_freq))
        return PKV_ERR_INVALID;
    const int es = elem_bytes(pool->dtype);
    if (!stride_ok(q_out_stride, static_cast<int64_t>(num_q_heads) * pool->head_dim, es) ||
        !stride_ok(q_stride, 0, es) || !stride_ok(k_stride, 0, es) || !stride_ok(v_stride, 0, es))
        return PKV_ERR_INVALID;
    const int64_t head = static_cast<int64_t>(pool->head_dim) * es;
    const int64_t q_row = num_q_heads * head, kv_row = pool->num_kv_heads * head;
    const Rows turned = {q_out, q_out_stride * es, q_row};
    if (!same_or_rows_apart(turned, {q, q_stride * es, q_row}, num_tokens) ||
        !rows_apart(turned, {k, k_stride * es, kv_row}, num_tokens) ||
        !rows_apart(turned, {v, v_stride * es, kv_row}, num_tokens))
        return PKV_ERR_INVALID;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;
    pkv::RopeArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.slot_mapping = slot_mapping;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.status = status;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.num_tokens = num_tokens;
    a.num_slots = pool->num_blocks * pool->block_size;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = pool->num_kv_heads;
    a.rotary_dim = rotary_dim;
    a.block_shift = block_shift(pool->block_size);
    a.interleaved = interleaved != 0;
    a.attn_scale = attn_scale;
    return from_cuda(pkv::launch_rope(a, pool->dtype, pool->head_dim,
                                      static_cast<cudaStream_t>(stream)));
}

namespace {

// Query tokens of a request that count, at most.
int window_rows(int max_new, int window) {
    return window > 0 && window < max_new ? window : max_new;
}

// How pass 1 cuts the keys of a query tile, and the workspace that gives.
struct PrefillWeightsPlan {
    int rows_pad, splits, chunk_tiles, row_parts, rows_per_part, heads_per_launch;
    int64_t key_pad;
    size_t stats_bytes, lse_bytes, score_bytes, bytes;
};
// What the kept scores of one launch may take (fp32): as many (request, kv head) pairs as fit
// kScoreBytes, or one alone that fits kScoreMost.  A larger one has its scores computed twice.
// Both bound a caller's workspace rather than the time.  16 pairs of 32 MB, D 64: 839 us for the
// call with a share of 64 MB, 783 with 256, 727 with 1 GB; 16 pairs of 128 MB, D 128: 5.13, 5.23
// and 4.85 ms; computed twice 1071 us and 7.61 ms, and one pair of 512 MB 2.11 ms for 1.30.
constexpr int64_t kScoreBytes = int64_t{256} << 20, kScoreMost = int64_t{1} << 30;
constexpr size_t kCounterBytes = 16;   // at the start of the workspace
bool prefill_weights_plan(const pkv_pool_desc* pool, int num_reqs, int num_q_heads, int max_new,
                          int max_context, int window, PrefillWeightsPlan* p) {
    const int64_t rows = static_cast<int64_t>(window_rows(max_new, window)) *
                         (num_q_heads / pool->num_kv_heads);
    if (rows > INT32_MAX - 128) return false;
    p->rows_pad = static_cast<int>((rows + 127) / 128 * 128);
    const int64_t heads = static_cast<int64_t>(num_reqs) * pool->num_kv_heads;
    if (heads > INT32_MAX) return false;
    p->heads_per_launch = static_cast<int>(heads);
    p->key_pad = 0;
    p->score_bytes = 0;
    const bool f32 = pool->dtype == PKV_F32;
    const int tiles = ceil_div(max_context, 128);
    const int row_tiles = p->rows_pad / 128;
    if (f32) {
        // CUDA cores: 64-row by 64-key tiles; parts of the keys up to two CTAs of a launch per SM,
        // which is what fits (a few more would be a second wave).  512 new tokens after 32k, 32
        // heads on 8, D 64, a launch per kv head: 3.34 ms, 18.8 with parts for all heads' CTAs.
        p->chunk_tiles = 0;
        p->key_pad = (static_cast<int64_t>(max_context) + 63) / 64 * 64;
        int64_t fit = 65535;   // a grid's second dimension
        if (p->key_pad <= kScoreMost / 4 / p->rows_pad) {
            const int64_t one = p->rows_pad * p->key_pad * 4;
            fit = std::max<int64_t>(std::min(fit, kScoreBytes / one), 1);
            p->score_bytes = static_cast<size_t>(std::min(fit, heads) * one);
        }
        p->heads_per_launch = static_cast<int>(std::min(fit, heads));
        const int64_t ctas = static_cast<int64_t>(p->heads_per_launch) * (p->rows_pad / 64);
        p->splits = static_cast<int>(std::min<int64_t>(
            std::min<int64_t>(std::max<int64_t>(304 / ctas, 1), ceil_div(max_context, 64)), 32));
    } else {
        // Tensor cores: parts of 24 tiles of 128 keys, shorter, down to 4, where there would be
        // fewer than one item per SM, and at most 32 of them: an item's own first tiles and
        // statistics count for more than evener CTAs.  The call with parts of
        //                                            32     24     16     12      8      6
        // 16 x 512 tokens, 32 heads, to 8k: us      559    553    562    567    583    599
        // their last 64 tokens                    128.0  115.1  119.1  119.6  120.5  123.6
        // 4 x 512 tokens                          220.9  199.9  202.7  200.9  205.7  214.7
        // The lengths are not known here, only their bound.
        const int64_t items = heads * ((row_tiles + 1) / 2);
        p->chunk_tiles = static_cast<int>(
            std::max<int64_t>(4, std::min<int64_t>(24, (items * tiles + 151) / 152)));
        p->chunk_tiles = std::max(p->chunk_tiles, ceil_div(tiles, 32));
        p->splits = ceil_div(tiles, p->chunk_tiles);
    }
    // Pass 2: parts of the rows, of two tiles of 128 at least, up to two items per SM.  500 tokens
    // after 2k, 8 heads on 1, fp32: 126 us with up to one item per SM, 108 with two, 103 with four;
    // bf16 26.9, 30.4 and 30.3.
    const int64_t items2 = static_cast<int64_t>(p->heads_per_launch) *
                           (f32 ? ceil_div(max_context, 64) : (tiles + 1) / 2);
    const int most = std::min(16, std::max(1, row_tiles / 2));
    p->row_parts = static_cast<int>(std::min<int64_t>(std::max<int64_t>(304 / items2, 1), most));
    p->rows_per_part = ceil_div(row_tiles, p->row_parts) * 128;
    p->row_parts = ceil_div(p->rows_pad, p->rows_per_part);
    p->stats_bytes = static_cast<size_t>(heads) * p->splits * (f32 ? 1 : 2) * p->rows_pad *
                     sizeof(float2);
    p->lse_bytes = f32 ? 0 : static_cast<size_t>(heads) * p->rows_pad * sizeof(float);
    p->bytes = kCounterBytes + p->stats_bytes + p->lse_bytes + p->score_bytes +
               (p->row_parts > 1 ? static_cast<size_t>(heads) * p->row_parts *
                                       static_cast<size_t>(max_context) * sizeof(float)
                                 : 0);
    return true;
}

}  // namespace

size_t pkv_paged_prefill_weights_workspace_bytes(const pkv_pool_desc* pool, int num_reqs,
                                                 int num_q_heads, int max_new, int max_context,
                                                 int window) {
    if (check_pool(pool) != PKV_OK || num_reqs <= 0 || num_q_heads <= 0 || max_new <= 0 ||
        max_context <= 0 || window < 0 || num_q_heads % pool->num_kv_heads != 0)
        return 0;
    PrefillWeightsPlan p;
    return prefill_weights_plan(pool, num_reqs, num_q_heads, max_new, max_context, window, &p)
               ? p.bytes
               : 0;
}

pkv_status pkv_paged_prefill_weights(const pkv_pool_desc* pool, const void* q, const void* k_pool,
                                     const int32_t* block_tables, int max_blocks_per_seq,
                                     const int32_t* cached_lens, const int32_t* new_lens,
                                     const int32_t* q_offsets, int num_reqs, int total_new,
                                     int max_new, int max_context, int num_q_heads, float scale,
                                     int window, float* weights, int64_t weights_stride,
                                     const int32_t* row_ids, int num_rows, float decay,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("pkv_paged_prefill_weights");
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (num_reqs < 0 || total_new < 0 || max_new < 0 || num_q_heads <= 0 || window < 0 ||
        !(scale > 0.f))
        return PKV_ERR_INVALID;
    if (num_reqs == 0 || total_new == 0 || max_new == 0) return PKV_OK;
    if (!q || !k_pool || !block_tables || !cached_lens || !new_lens || !q_offsets ||
        max_blocks_per_seq <= 0 || max_context <= 0 || !aligned16(q) || !aligned16(k_pool))
        return PKV_ERR_INVALID;
    if (static_cast<int64_t>(max_context) >
        static_cast<int64_t>(max_blocks_per_seq) * pool->block_size)
        return PKV_ERR_INVALID;
    const WeightsOut wo{weights, weights_stride, row_ids, num_rows, decay};
    if (!weights_ok(wo, num_reqs, max_context)) return PKV_ERR_INVALID;
    if (num_q_heads % pool->num_kv_heads != 0) return PKV_ERR_INVALID;
    const int group = num_q_heads / pool->num_kv_heads;
    if (group != 1 && group != 2 && group != 4 && group != 8) return PKV_ERR_UNSUPPORTED;
    if (num_reqs > 65535) return PKV_ERR_UNSUPPORTED;
    PrefillWeightsPlan plan;
    if (!prefill_weights_plan(pool, num_reqs, num_q_heads, max_new, max_context, window, &plan))
        return PKV_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < plan.bytes || !aligned16(workspace)) return PKV_ERR_NOMEM;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;
    pkv::PrefillWeightsArgs a{};
    a.q = q;
    a.k_pool = k_pool;
    a.block_tables = block_tables;
    a.cached_lens = cached_lens;
    a.new_lens = new_lens;
    a.q_offsets = q_offsets;
    a.row_ids = row_ids;
    a.weights = weights;
    char* base = static_cast<char*>(workspace) + kCounterBytes;
    a.next_item = static_cast<int*>(workspace);
    a.stats = reinterpret_cast<float2*>(base);
    a.neg_lse = reinterpret_cast<float*>(base + plan.stats_bytes);
    char* after = base + plan.stats_bytes + plan.lse_bytes;
    a.scores = plan.score_bytes ? reinterpret_cast<float*>(after) : nullptr;
    a.parts = reinterpret_cast<float*>(after + plan.score_bytes);
    a.key_pad = plan.key_pad;
    a.heads_per_launch = plan.heads_per_launch;
    a.row_parts = plan.row_parts;
    a.rows_per_part = plan.rows_per_part;
    a.group_shift = group == 1 ? 0 : group == 2 ? 1 : group == 4 ? 2 : 3;
    a.status = status;
    a.num_blocks = pool->num_blocks;
    a.weights_stride = weights_stride;
    a.num_rows = num_rows;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.block_shift = block_shift(pool->block_size);
    a.num_reqs = num_reqs;
    a.total_new = total_new;
    a.max_new = max_new;
    a.max_rows = window_rows(max_new, window);
    a.max_context = max_context;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = pool->num_kv_heads;
    a.window = window;
    a.splits = plan.splits;
    a.chunk_tiles = plan.chunk_tiles;
    a.rows_pad = plan.rows_pad;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * kLog2e);
    a.decay = decay;
    a.test_stall = prefill_weights_test_stall();
    const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
    const cudaError_t e = pool->dtype == PKV_BF16
                              ? pkv::launch_prefill_weights_tc(a, pool->head_dim, group, st_)
                              : pkv::launch_prefill_weights(a, pool->head_dim, group, st_);
    if (e == cudaErrorNotSupported) return PKV_ERR_UNSUPPORTED;
    return from_cuda(e);
}

namespace {

// No byte in common (`b` null: not given); or the same array.
bool apart(const void* a, const void* b, uint64_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return !b || x + bytes <= y || y + bytes <= x;
}
bool same_or_apart(const void* a, const void* b, uint64_t bytes) {
    return a == b || apart(a, b, bytes);
}

}  // namespace

size_t pkv_evict_workspace_bytes(const pkv_pool_desc* pool, int num_seqs, int max_context) {
    if (check_pool(pool) != PKV_OK || num_seqs <= 0 || max_context <= 0) return 0;
    return static_cast<size_t>(num_seqs) * pool->num_kv_heads * 5 *
           static_cast<size_t>(std::max(max_context / 2, 1)) * sizeof(int32_t);
}

pkv_status pkv_evict(const pkv_pool_desc* pool, void* k_pool, void* v_pool,
                     const int32_t* block_tables, int max_blocks_per_seq,
                     const int32_t* context_lens, int max_context, int num_seqs,
                     const int32_t* budgets, int sinks, int recent, const int32_t* seen_lens,
                     const int32_t* tracked_lens, const float* weights, float* weights_out,
                     const int32_t* positions, int32_t* positions_out, int64_t weights_stride,
                     const int32_t* row_ids, int num_rows, int32_t* new_lens, void* workspace,
                     size_t workspace_bytes, void* stream) {
    CallRange range("pkv_evict");
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (num_seqs < 0 || sinks < 0 || recent < 0) return PKV_ERR_INVALID;
    if (num_seqs == 0) return PKV_OK;
    if (!k_pool || !v_pool || !block_tables || !context_lens || !budgets || !weights_out ||
        !positions || !positions_out || !new_lens || max_blocks_per_seq <= 0 || max_context <= 0)
        return PKV_ERR_INVALID;
    if (!aligned16(k_pool) || !aligned16(v_pool)) return PKV_ERR_INVALID;
    if (static_cast<int64_t>(max_context) >
        static_cast<int64_t>(max_blocks_per_seq) * pool->block_size)
        return PKV_ERR_INVALID;
    const WeightsOut wo{const_cast<float*>(weights), weights_stride, row_ids, num_rows, 1.f};
    if (!weights_ok(wo, num_seqs, max_context)) return PKV_ERR_INVALID;
    const uint64_t extent = static_cast<uint64_t>(num_rows) * pool->num_kv_heads *
                            static_cast<uint64_t>(weights_stride) * 4;
    if (!same_or_apart(weights, weights_out, extent) ||
        !same_or_apart(positions, positions_out, extent))
        return PKV_ERR_INVALID;
    // the CTAs of a sequence run at different times: nothing they read may change meanwhile
    const uint64_t lens = static_cast<uint64_t>(num_seqs) * sizeof(int32_t);
    if (!apart(new_lens, context_lens, lens) || !apart(new_lens, budgets, lens) ||
        !apart(new_lens, seen_lens, lens) || !apart(new_lens, tracked_lens, lens) ||
        !apart(new_lens, row_ids, lens))
        return PKV_ERR_INVALID;
    if (!aligned4(context_lens) || !aligned4(budgets) || !aligned4(seen_lens) ||
        !aligned4(tracked_lens) || !aligned4(row_ids) || !aligned4(new_lens) ||
        !aligned4(positions) || !aligned4(positions_out) || !aligned4(weights_out) ||
        !aligned4(block_tables))
        return PKV_ERR_INVALID;
    if (num_seqs > 65535 || max_context > pkv::kEvictMaxContext) return PKV_ERR_UNSUPPORTED;
    const size_t need = pkv_evict_workspace_bytes(pool, num_seqs, max_context);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return PKV_ERR_NOMEM;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;
    pkv::EvictArgs a{};
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.budgets = budgets;
    a.seen_lens = seen_lens;
    a.tracked_lens = tracked_lens;
    a.row_ids = row_ids;
    a.weights = weights;
    a.weights_out = weights_out;
    a.positions = positions;
    a.positions_out = positions_out;
    a.new_lens = new_lens;
    a.moves = static_cast<int32_t*>(workspace);
    a.status = status;
    a.num_blocks = pool->num_blocks;
    a.weights_stride = weights_stride;
    a.num_rows = num_rows;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.block_shift = block_shift(pool->block_size);
    a.max_context = max_context;
    a.num_seqs = num_seqs;
    a.num_kv_heads = pool->num_kv_heads;
    const int chunks = pool->head_dim * elem_bytes(pool->dtype) / 16;   // 8, 16 or 32
    a.row_shift = chunks == 8 ? 3 : chunks == 16 ? 4 : 5;
    a.sinks = sinks;
    a.recent = recent;
    return from_cuda(pkv::launch_evict(a, static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- quantised cache

namespace {

pkv_status check_quant(const pkv_quant_cache* c) {
    if (!c || c->num_blocks <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0 || c->block_size <= 0)
        return PKV_ERR_INVALID;
    if (c->format != PKV_FP8 && c->format != PKV_FP4) return PKV_ERR_UNSUPPORTED;
    if (chunk_shift(c->block_size) < 0) return PKV_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (c->num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
    // the kernels count rows in 32 bits
    if (c->num_blocks > INT32_MAX / (static_cast<int64_t>(c->num_kv_heads) * c->block_size))
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

// Bytes of a block's codes (K or V, all kv heads), and of what lies beside them.
int64_t quant_code_bytes(const pkv_quant_cache* c) {
    const int64_t rows = static_cast<int64_t>(c->num_kv_heads) * c->block_size;
    return rows * (c->format == PKV_FP8 ? c->head_dim : c->head_dim / 2);
}
int64_t quant_side_bytes(const pkv_quant_cache* c) {
    const int64_t runs = static_cast<int64_t>(c->num_kv_heads) * (c->block_size / 16);
    return runs * (c->format == PKV_FP8 ? 16 : c->head_dim + 16);
}

// The four arrays, present and aligned.
bool quant_arrays_ok(const pkv_quant_cache* c) {
    return c->k_codes && c->v_codes && c->k_scales && c->v_scales && aligned16(c->k_codes) &&
           aligned16(c->v_codes) && aligned16(c->k_scales) && aligned16(c->v_scales);
}

// Runs of bytes, one after another in no order: whether none shares a byte with another.
struct Run {
    const void* at;
    uint64_t bytes;
};
bool runs_apart(std::initializer_list<Run> runs) {
    for (const Run* x = runs.begin(); x != runs.end(); ++x)
        for (const Run* y = runs.begin(); y != x; ++y) {
            const uintptr_t p = reinterpret_cast<uintptr_t>(x->at);
            const uintptr_t q = reinterpret_cast<uintptr_t>(y->at);
            if (p < q + y->bytes && q < p + x->bytes) return false;
        }
    return true;
}

// The four arrays apart from one another, and from each of two runs beside them: kernels store to
// any of them in any order.
bool quant_arrays_apart(const pkv_quant_cache* c, Run a = {nullptr, 0}, Run b = {nullptr, 0}) {
    const uint64_t codes = static_cast<uint64_t>(c->num_blocks) * quant_code_bytes(c);
    const uint64_t side = static_cast<uint64_t>(c->num_blocks) * quant_side_bytes(c);
    return runs_apart({{c->k_codes, codes}, {c->v_codes, codes}, {c->k_scales, side},
                       {c->v_scales, side}, a}) &&
           (!b.bytes || runs_apart({{c->k_codes, codes}, {c->v_codes, codes}, {c->k_scales, side},
                                    {c->v_scales, side}, b}));
}

pkv::QuantArgs quant_args(const pkv_quant_cache* c, int* status) {
    pkv::QuantArgs a{};
    a.k_codes = static_cast<uint8_t*>(c->k_codes);
    a.v_codes = static_cast<uint8_t*>(c->v_codes);
    a.k_scales = static_cast<uint8_t*>(c->k_scales);
    a.v_scales = static_cast<uint8_t*>(c->v_scales);
    a.status = status;
    a.num_blocks = c->num_blocks;
    a.num_slots = c->num_blocks * c->block_size;
    a.num_kv_heads = c->num_kv_heads;
    a.block_shift = block_shift(c->block_size);
    return a;
}

// pkv_kv_append_quant, and with `read` pkv_kv_read_quant.
pkv_status quant_rows(const pkv_quant_cache* cache, const int64_t* slot_mapping, int dtype,
                      const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                      int64_t num_tokens, bool read, void* stream) {
    pkv_status st = check_quant(cache);
    if (st != PKV_OK) return st;
    if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (num_tokens < 0) return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (num_tokens > INT32_MAX / cache->num_kv_heads) return PKV_ERR_UNSUPPORTED;
    if (!quant_arrays_ok(cache) || !slot_mapping || !k || !v || !aligned16(k) || !aligned16(v) ||
        !aligned8(slot_mapping))
        return PKV_ERR_INVALID;
    const int es = elem_bytes(dtype);
    const int64_t row = static_cast<int64_t>(cache->num_kv_heads) * cache->head_dim;
    if (!stride_ok(k_stride, read ? row : 0, es) || !stride_ok(v_stride, read ? row : 0, es))
        return PKV_ERR_INVALID;
    if (read && !rows_apart({k, k_stride * es, row * es}, {v, v_stride * es, row * es}, num_tokens))
        return PKV_ERR_INVALID;
    if (!quant_arrays_apart(cache)) return PKV_ERR_INVALID;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;
    pkv::QuantArgs a = quant_args(cache, status);
    a.k = k;
    a.v = v;
    a.k_out = const_cast<void*>(k);
    a.v_out = const_cast<void*>(v);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slots = slot_mapping;
    a.num_rows = static_cast<uint32_t>(num_tokens * cache->num_kv_heads);
    a.wide = aligned32(k) && aligned32(v) && (k_stride * es) % 32 == 0 && (v_stride * es) % 32 == 0;
    return from_cuda(pkv::launch_quant_move(a, cache->format, cache->head_dim, dtype, false, read,
                                            static_cast<cudaStream_t>(stream)));
}

// pkv_quantize_blocks, and with `read` pkv_dequantize_blocks.
pkv_status quant_blocks(const pkv_quant_cache* cache, const pkv_pool_desc* pool, const void* k,
                        const void* v, const int32_t* pairs, int num_pairs, bool read,
                        void* stream) {
    pkv_status st = check_quant(cache);
    if (st == PKV_OK) st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (pool->block_size != cache->block_size || pool->num_kv_heads != cache->num_kv_heads ||
        pool->head_dim != cache->head_dim || num_pairs < 0)
        return PKV_ERR_INVALID;
    if (num_pairs == 0) return PKV_OK;
    const int64_t per = static_cast<int64_t>(cache->num_kv_heads) * cache->block_size;
    if (num_pairs > INT32_MAX / per) return PKV_ERR_UNSUPPORTED;
    if (!quant_arrays_ok(cache) || !k || !v || !pairs || !aligned16(k) || !aligned16(v) ||
        !aligned4(pairs))
        return PKV_ERR_INVALID;
    const uint64_t bytes = pkv_pool_bytes(pool);
    if (!quant_arrays_apart(cache, {k, bytes}, {v, bytes}) ||
        (read && !runs_apart({{k, bytes}, {v, bytes}})))
        return PKV_ERR_INVALID;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;
    pkv::QuantArgs a = quant_args(cache, status);
    a.k = k;
    a.v = v;
    a.k_out = const_cast<void*>(k);
    a.v_out = const_cast<void*>(v);
    a.pairs = pairs;
    a.pool_blocks = pool->num_blocks;
    a.num_rows = static_cast<uint32_t>(num_pairs * per);
    a.wide = aligned32(k) && aligned32(v);
    return from_cuda(pkv::launch_quant_move(a, cache->format, cache->head_dim, pool->dtype, true,
                                            read, static_cast<cudaStream_t>(stream)));
}

// Partition of a decode over a quantised cache, in pool blocks.  A CTA's start and its merge cost
// about as much as 16 chunks a warp, so 256 chunks (4096 tokens), or 128, where that leaves 12
// CTAs an SM, four (three) for each that is resident; with fewer the last ones leave SMs idle.  us
// with 256 / 128 / 64 chunks, 8 kv heads of 128:
//   12 sequences of 16k .. 128k     fp8 321 / 325 / 348   fp4 279 / 290 / 322
//   16                                  398 / 401 / 434       346 / 361 / 405   (256: 4096 CTAs)
//   6                                   162 / 155 / 163       147 / 141 / 156   (1536)
//   100 of 1024 .. 8192                 155 / 150 / 151       138 / 135 / 147   (1600)
//   32 of 2048 .. 16384                 100 /  91 /  91        93 /  82 /  86   (1024)
//   64 of 512 .. 4096                  53.8 / 55.0 / 53.0    53.2 / 54.8 / 53.6 (512)
// Else 64 chunks, where more, shorter ones cost more than they balance (the last row with 32: 55.7 and
// 60.2), and below that only while there would be fewer than 456 CTAs, three an SM.  A multiple of 8
// chunks (a pair for each warp), and at most 512 partitions.
int quant_partition(const pkv_quant_cache* cache, int num_seqs, int max_context,
                    int partition_blocks) {
    if (partition_blocks) return partition_blocks;
    const int64_t rows = static_cast<int64_t>(num_seqs) * cache->num_kv_heads;
    const int chunks = ceil_div(max_context, kChunk);
    const int least = ceil_div(ceil_div(chunks, 512), 8) * 8;
    auto halved = [](int pc) { return (pc / 2 + 7) / 8 * 8; };
    int pc = std::max(256, least);
    while (pc > 64 && halved(pc) >= least && rows * ceil_div(chunks, pc) < 12 * 152) pc = halved(pc);
    while (pc > 8 && halved(pc) >= least && rows * ceil_div(chunks, pc) < 3 * 152) pc = halved(pc);
    return pc >> chunk_shift(cache->block_size);
}

}  // namespace

uint64_t pkv_quant_codes_bytes(const pkv_quant_cache* cache) {
    if (check_quant(cache) != PKV_OK) return 0;
    return static_cast<uint64_t>(cache->num_blocks) * quant_code_bytes(cache);
}

uint64_t pkv_quant_scales_bytes(const pkv_quant_cache* cache) {
    if (check_quant(cache) != PKV_OK) return 0;
    return static_cast<uint64_t>(cache->num_blocks) * quant_side_bytes(cache);
}

pkv_status pkv_kv_append_quant(const pkv_quant_cache* cache, const int64_t* slot_mapping,
                               int dtype, const void* k, int64_t k_stride, const void* v,
                               int64_t v_stride, int64_t num_tokens, void* stream) {
    CallRange range("pkv_kv_append_quant");
    return quant_rows(cache, slot_mapping, dtype, k, k_stride, v, v_stride, num_tokens, false,
                      stream);
}

pkv_status pkv_kv_read_quant(const pkv_quant_cache* cache, const int64_t* slot_mapping, int dtype,
                             void* k_out, int64_t k_stride, void* v_out, int64_t v_stride,
                             int64_t num_tokens, void* stream) {
    CallRange range("pkv_kv_read_quant");
    return quant_rows(cache, slot_mapping, dtype, k_out, k_stride, v_out, v_stride, num_tokens,
                      true, stream);
}

pkv_status pkv_quantize_blocks(const pkv_quant_cache* cache, const pkv_pool_desc* pool,
                               const void* k_pool, const void* v_pool, const int32_t* pairs,
                               int num_pairs, void* stream) {
    CallRange range("pkv_quantize_blocks");
    return quant_blocks(cache, pool, k_pool, v_pool, pairs, num_pairs, false, stream);
}

pkv_status pkv_dequantize_blocks(const pkv_quant_cache* cache, const pkv_pool_desc* pool,
                                 void* k_pool, void* v_pool, const int32_t* pairs, int num_pairs,
                                 void* stream) {
    CallRange range("pkv_dequantize_blocks");
    return quant_blocks(cache, pool, k_pool, v_pool, pairs, num_pairs, true, stream);
}

pkv_status pkv_copy_blocks_quant(const pkv_quant_cache* cache, const int32_t* pairs,
                                 int num_pairs, void* stream) {
    CallRange range("pkv_copy_blocks_quant");
    pkv_status st = check_quant(cache);
    if (st != PKV_OK) return st;
    if (num_pairs < 0) return PKV_ERR_INVALID;
    if (num_pairs == 0) return PKV_OK;
    if (!quant_arrays_ok(cache) || !pairs || !aligned4(pairs) || !quant_arrays_apart(cache))
        return PKV_ERR_INVALID;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;
    pkv::QuantArgs a = quant_args(cache, status);
    a.pairs = pairs;
    return from_cuda(pkv::launch_quant_copy(a, num_pairs, quant_code_bytes(cache),
                                            quant_side_bytes(cache),
                                            static_cast<cudaStream_t>(stream)));
}

size_t pkv_paged_decode_quant_workspace_bytes(const pkv_quant_cache* cache, int num_seqs,
                                              int num_q_heads, int max_context,
                                              int partition_blocks) {
    if (check_quant(cache) != PKV_OK || num_seqs <= 0 || num_q_heads <= 0 || max_context <= 0 ||
        partition_blocks < 0)
        return 0;
    const int pb = quant_partition(cache, num_seqs, max_context, partition_blocks);
    return decode_workspace(num_seqs, num_q_heads, cache->head_dim,
                            ceil_div(ceil_div(max_context, cache->block_size), pb));
}

pkv_status pkv_paged_decode_quant(const pkv_quant_cache* cache, int dtype, void* out, const void* q,
                                  const void* k_new, const void* v_new,
                                  const int32_t* block_tables, int max_blocks_per_seq,
                                  const int32_t* context_lens, int max_context, int num_seqs,
                                  int num_q_heads, float scale, int partition_blocks,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("pkv_paged_decode_quant");
    pkv_status st = check_quant(cache);
    if (st != PKV_OK) return st;
    if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_q_heads <= 0 || partition_blocks < 0) return PKV_ERR_INVALID;
    if (num_seqs == 0) return PKV_OK;
    if (!quant_arrays_ok(cache) || !out || !q || !block_tables || !context_lens ||
        !k_new != !v_new)
        return PKV_ERR_INVALID;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_new) || !aligned16(v_new) ||
        !aligned4(block_tables) || !aligned4(context_lens))
        return PKV_ERR_INVALID;
    const int B = cache->block_size;
    if (max_blocks_per_seq <= 0 || max_context <= 0 ||
        static_cast<int64_t>(max_context) > static_cast<int64_t>(max_blocks_per_seq) * B)
        return PKV_ERR_INVALID;
    if (num_q_heads % cache->num_kv_heads != 0) return PKV_ERR_INVALID;
    const int group = num_q_heads / cache->num_kv_heads;
    if (group != 1 && group != 2 && group != 4 && group != 8) return PKV_ERR_UNSUPPORTED;
    if (num_seqs > 65535 || max_blocks_per_seq > INT32_MAX / 64) return PKV_ERR_UNSUPPORTED;
    const int pb = quant_partition(cache, num_seqs, max_context, partition_blocks);
    if (pb > INT32_MAX / 64) return PKV_ERR_UNSUPPORTED;
    const int max_parts = ceil_div(ceil_div(max_context, B), pb);
    if (max_parts > pkv::kMaxParts) return PKV_ERR_UNSUPPORTED;
    const size_t need = decode_workspace(num_seqs, num_q_heads, cache->head_dim, max_parts);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
        return PKV_ERR_NOMEM;
    if (!quant_arrays_apart(cache)) return PKV_ERR_INVALID;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;

    pkv::DecodeArgs a{};
    a.out = out;
    a.q = q;
    a.k_pool = cache->k_codes;
    a.v_pool = cache->v_codes;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.status = status;
    a.num_blocks = cache->num_blocks;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_seqs = num_seqs;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = cache->num_kv_heads;
    a.chunk_shift = chunk_shift(B);
    a.partition_chunks = pb << a.chunk_shift;
    a.max_parts = max_parts;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * kLog2e);
    a.k_new = k_new;
    a.v_new = v_new;
    a.test_stall = decode_test_stall();
    if (need > 0) {
        const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * max_parts;
        char* w = static_cast<char*>(workspace);
        a.o_part = reinterpret_cast<float*>(w);
        w += rows * cache->head_dim * sizeof(float);
        a.m_part = reinterpret_cast<float*>(w);
        a.l_part = reinterpret_cast<float*>(w + round16(rows * sizeof(float)));
    }
    const pkv::QuantSides sides = {static_cast<uint8_t*>(cache->k_scales),
                                   static_cast<uint8_t*>(cache->v_scales)};
    return from_cuda(pkv::launch_quant_decode(a, sides, cache->format, dtype, cache->head_dim,
                                              group, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_copy_blocks(const pkv_pool_desc* pool, void* k_pool, void* v_pool,
                           const int32_t* pairs, int num_pairs, void* stream) {
    CallRange range("pkv_copy_blocks");
    pkv_status st = check_pool(pool);
    if (st != PKV_OK) return st;
    if (num_pairs < 0) return PKV_ERR_INVALID;
    if (num_pairs == 0) return PKV_OK;
    if (!k_pool || !v_pool || !pairs) return PKV_ERR_INVALID;
    if (!aligned16(k_pool) || !aligned16(v_pool)) return PKV_ERR_INVALID;
    if (num_pairs > 65535 * 1024) return PKV_ERR_UNSUPPORTED;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;
    const int64_t block_bytes = static_cast<int64_t>(pool->num_kv_heads) * pool->block_size *
                                pool->head_dim * elem_bytes(pool->dtype);
    return from_cuda(pkv::launch_copy_blocks(k_pool, v_pool, pairs, num_pairs, block_bytes,
                                             pool->num_blocks, status,
                                             static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_read_device_status(int* status_out, void* stream) {
    if (!status_out) return PKV_ERR_INVALID;
    int* status = status_word();
    if (!status) return PKV_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int v = 0;
    if (cudaMemcpyAsync(&v, status, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return PKV_ERR_CUDA;
    if (cudaMemsetAsync(status, 0, sizeof(int), s) != cudaSuccess) return PKV_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return PKV_ERR_CUDA;
    *status_out = v;
    return PKV_OK;
}

}  // extern "C"

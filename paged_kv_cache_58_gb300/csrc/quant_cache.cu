// Rows and blocks in and out of a quantised cache.
//
// kv_append_quant writes new tokens' rows into their slots, kv_read_quant reads rows back;
// quantize_blocks and dequantize_blocks move whole blocks between a pool and the cache.  All
// four are one pass over the rows: D / 16 lanes share a row, 16 elements (32 or 64 bytes of a
// pool's row, 16 or 8 of codes) each.  Bound: HBM.
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;

// A row of the cache: block, kv head, token of the block.
template <int FMT, int D>
struct RowAt {
    using R = QuantRow<FMT, D>;
    size_t row;    // row of codes
    size_t side;   // what lies beside its 16 rows, in bytes
    int t;         // token of the 16
    PKV_DEVINL RowAt(int64_t blk, int head, int num_kv_heads, int off, int block_shift) {
        const size_t bh = static_cast<size_t>(blk) * num_kv_heads + head;
        row = (bh << block_shift) + off;
        side = ((bh << (block_shift - 4)) + (off >> 4)) * R::kSide;
        t = off & 15;
    }
};

template <int FMT, int D>
PKV_DEVINL void store_row(const QuantArgs& a, bool is_v, const RowAt<FMT, D>& at, int lane,
                          const Quantised& q) {
    using R = QuantRow<FMT, D>;
    uint8_t* codes = is_v ? a.v_codes : a.k_codes;
    uint8_t* side = (is_v ? a.v_scales : a.k_scales) + at.side;
    uint8_t* dst = codes + at.row * R::kCodes + lane * R::kLaneBytes;
    if constexpr (FMT == PKV_FP8) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(q.codes[0], q.codes[1], q.codes[2], q.codes[3]);
    } else {
        *reinterpret_cast<uint2*>(dst) = make_uint2(q.codes[0], q.codes[1]);
        side[scale_at<D>(is_v, at.t, lane)] = static_cast<uint8_t>(q.scale);
    }
    if (lane == 0) side[R::kScales + at.t] = static_cast<uint8_t>(q.exp);
}

template <int FMT, int D>
PKV_DEVINL void load_row(const QuantArgs& a, bool is_v, const RowAt<FMT, D>& at, int lane,
                         float (&x)[16]) {
    using R = QuantRow<FMT, D>;
    const uint8_t* codes = is_v ? a.v_codes : a.k_codes;
    const uint8_t* side = (is_v ? a.v_scales : a.k_scales) + at.side;
    const uint8_t* src = codes + at.row * R::kCodes + lane * R::kLaneBytes;
    uint32_t c[4] = {0, 0, 0, 0};
    uint32_t scale = 0;
    if constexpr (FMT == PKV_FP8) {
        const uint4 w = *reinterpret_cast<const uint4*>(src);
        c[0] = w.x; c[1] = w.y; c[2] = w.z; c[3] = w.w;
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(src);
        c[0] = w.x; c[1] = w.y;
        scale = side[scale_at<D>(is_v, at.t, lane)];
    }
    dequantise<FMT>(c, scale, side[R::kScales + at.t], x);
}

// Rows by slot.  grid (rows, 2): y selects K or V.  READ: cache to rows, else rows to cache.
template <int FMT, int D, typename T, bool READ>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(const QuantArgs a) {
    using R = QuantRow<FMT, D>;
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t row = blockIdx.x * (kThreads / R::kLanes) + threadIdx.x / R::kLanes;
    const int lane = threadIdx.x % R::kLanes;
    const bool is_v = blockIdx.y != 0;
    const bool there = row < a.num_rows;
    const uint32_t tok = there ? row / static_cast<uint32_t>(a.num_kv_heads) : 0;
    const int head = there ? static_cast<int>(row - tok * a.num_kv_heads) : 0;
    int64_t slot = there ? __ldg(a.slots + tok) : -1;
    const int64_t at_elem = static_cast<int64_t>(tok) * (is_v ? a.v_stride : a.k_stride) +
                            static_cast<int64_t>(head) * D + 16 * lane;
    if (slot >= a.num_slots) {
        raise_status(a.status, PKV_ERR_OOB);
        slot = -1;
    }
    const RowAt<FMT, D> at(slot >= 0 ? slot >> a.block_shift : 0, head, a.num_kv_heads,
                           static_cast<int>(slot & ((1 << a.block_shift) - 1)), a.block_shift);
    if constexpr (READ) {
        if (!there) return;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
        if (slot >= 0) load_row<FMT, D>(a, is_v, at, lane, x);
        Elems16<T>::store(static_cast<T*>(is_v ? a.v_out : a.k_out) + at_elem, x);
    } else {
        Elems16<T> in;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
        if (slot >= 0) {
            in.load(static_cast<const T*>(is_v ? a.v : a.k) + at_elem);
            in.values(x);
        }
        const Quantised q = quantise<FMT, D, sizeof(T) == 4>(x);
        if (slot >= 0) store_row<FMT, D>(a, is_v, at, lane, q);
    }
}

// Whole blocks by pairs (source, destination).  grid (rows of all pairs, 2).
template <int FMT, int D, typename T, bool READ>
__global__ void __launch_bounds__(kThreads) quant_blocks_kernel(const QuantArgs a) {
    using R = QuantRow<FMT, D>;
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t row = blockIdx.x * (kThreads / R::kLanes) + threadIdx.x / R::kLanes;
    const int lane = threadIdx.x % R::kLanes;
    const bool is_v = blockIdx.y != 0;
    const bool there = row < a.num_rows;
    const uint32_t per = static_cast<uint32_t>(a.num_kv_heads) << a.block_shift;
    const uint32_t pair = there ? row / per : 0;
    const uint32_t in = there ? row - pair * per : 0;
    const int head = static_cast<int>(in >> a.block_shift);
    const int off = static_cast<int>(in & ((1u << a.block_shift) - 1));
    const int src = __ldg(a.pairs + 2 * static_cast<size_t>(pair));
    const int dst = __ldg(a.pairs + 2 * static_cast<size_t>(pair) + 1);
    const int kept = READ ? src : dst, plain = READ ? dst : src;
    const bool ok = kept >= 0 && kept < a.num_blocks && plain >= 0 && plain < a.pool_blocks;
    if (!ok && there) raise_status(a.status, PKV_ERR_OOB);
    const bool go = ok && there;
    const RowAt<FMT, D> at(go ? kept : 0, head, a.num_kv_heads, off, a.block_shift);
    const size_t elem = (static_cast<size_t>(go ? plain : 0) * per + in) * D + 16 * lane;
    if constexpr (READ) {
        if (!go) return;
        float x[16];
        load_row<FMT, D>(a, is_v, at, lane, x);
        Elems16<T>::store(static_cast<T*>(is_v ? a.v_out : a.k_out) + elem, x);
    } else {
        Elems16<T> in16;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
        if (go) {
            in16.load(static_cast<const T*>(is_v ? a.v : a.k) + elem);
            in16.values(x);
        }
        const Quantised q = quantise<FMT, D, sizeof(T) == 4>(x);
        if (go) store_row<FMT, D>(a, is_v, at, lane, q);
    }
}

// pool[dst] = pool[src] of the codes and of what lies beside them.  grid (pairs, 2).
__global__ void __launch_bounds__(kThreads)
quant_copy_kernel(const QuantArgs a, const int code_units, const int side_units) {
    griddep_wait();
    griddep_launch_dependents();
    const int src = __ldg(a.pairs + 2 * static_cast<size_t>(blockIdx.x));
    const int dst = __ldg(a.pairs + 2 * static_cast<size_t>(blockIdx.x) + 1);
    if (src < 0 || src >= a.num_blocks || dst < 0 || dst >= a.num_blocks) {
        if (threadIdx.x == 0) raise_status(a.status, PKV_ERR_OOB);
        return;
    }
    uint4* codes = reinterpret_cast<uint4*>(blockIdx.y ? a.v_codes : a.k_codes);
    uint4* side = reinterpret_cast<uint4*>(blockIdx.y ? a.v_scales : a.k_scales);
    for (int i = threadIdx.x; i < code_units; i += kThreads)
        codes[static_cast<size_t>(dst) * code_units + i] =
            codes[static_cast<size_t>(src) * code_units + i];
    for (int i = threadIdx.x; i < side_units; i += kThreads)
        side[static_cast<size_t>(dst) * side_units + i] =
            side[static_cast<size_t>(src) * side_units + i];
}

template <int FMT, int D, typename T>
cudaError_t launch_typed(const QuantArgs& a, bool blocks, bool read, cudaStream_t stream) {
    constexpr uint32_t per = kThreads / QuantRow<FMT, D>::kLanes;
    auto kern = blocks ? (read ? quant_blocks_kernel<FMT, D, T, true>
                               : quant_blocks_kernel<FMT, D, T, false>)
                       : (read ? quant_rows_kernel<FMT, D, T, true>
                               : quant_rows_kernel<FMT, D, T, false>);
    return launch_pdl(kern, dim3((a.num_rows + per - 1) / per, 2), dim3(kThreads), 0, stream, a);
}

template <int FMT, int D>
cudaError_t launch_dtype(const QuantArgs& a, int dtype, bool blocks, bool read,
                         cudaStream_t stream) {
    return dtype == PKV_BF16 ? launch_typed<FMT, D, uint16_t>(a, blocks, read, stream)
                             : launch_typed<FMT, D, float>(a, blocks, read, stream);
}

}  // namespace

cudaError_t launch_quant_move(const QuantArgs& a, int format, int head_dim, int dtype, bool blocks,
                              bool read, cudaStream_t stream) {
    if (format == PKV_FP8)
        return head_dim == 128 ? launch_dtype<PKV_FP8, 128>(a, dtype, blocks, read, stream)
                               : launch_dtype<PKV_FP8, 64>(a, dtype, blocks, read, stream);
    return head_dim == 128 ? launch_dtype<PKV_FP4, 128>(a, dtype, blocks, read, stream)
                           : launch_dtype<PKV_FP4, 64>(a, dtype, blocks, read, stream);
}

cudaError_t launch_quant_copy(const QuantArgs& a, int num_pairs, int64_t code_bytes,
                              int64_t side_bytes, cudaStream_t stream) {
    return launch_pdl(quant_copy_kernel, dim3(num_pairs, 2), dim3(kThreads), 0, stream, a,
                      static_cast<int>(code_bytes / 16), static_cast<int>(side_bytes / 16));
}

}  // namespace pkv

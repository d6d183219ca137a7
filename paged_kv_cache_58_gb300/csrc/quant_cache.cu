// Rows and blocks in and out of a quantised cache.
//
// kv_append_quant writes new tokens' rows into their slots, kv_read_quant reads rows back;
// quantize_blocks and dequantize_blocks move whole blocks between a pool and the cache.  All
// four are one pass over the rows: D / 16 lanes share a row, 16 elements (32 or 64 bytes of a
// pool's row, 16 or 8 of codes) each, and take the row of K and that of V, whose places are found
// once.
//
// Bound: HBM for large ones (4608 blocks of 16 tokens and 8 heads of 128 from fp8 to bf16: 69 us, 6.6
// TB/s); fp4 and its way back 62 us for 2048 blocks, 5.5 TB/s, the instructions of the codes beside
// the bytes.  K's and V's rows by CTAs of their own took 76 and 74 us.
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
    size_t codes;   // of the lane, in bytes
    size_t side;    // what lies beside its 16 rows, in bytes
    int t;          // token of the 16
    PKV_DEVINL RowAt(uint32_t blk, uint32_t head, const QuantArgs& a, uint32_t off, int lane) {
        const uint32_t bh = blk * a.num_kv_heads + head;   // the cache's rows number below 2^31
        codes = static_cast<size_t>((bh << a.block_shift) + off) * R::kCodes + lane * R::kLaneBytes;
        side = static_cast<size_t>((bh << (a.block_shift - 4)) + (off >> 4)) * R::kSide;
        t = static_cast<int>(off & 15);
    }
};

// n / d for n < 2^31, d's mul and shift from the host.
PKV_DEVINL uint32_t divide(uint32_t n, const QuantArgs& a) {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * a.div_mul) >> a.div_shift);
}

template <int FMT, int D>
PKV_DEVINL void store_row(const QuantArgs& a, bool is_v, const RowAt<FMT, D>& at, int lane,
                          const Quantised& q) {
    using R = QuantRow<FMT, D>;
    uint8_t* side = (is_v ? a.v_scales : a.k_scales) + at.side;
    uint8_t* dst = (is_v ? a.v_codes : a.k_codes) + at.codes;
    if constexpr (FMT == PKV_FP8) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(q.codes[0], q.codes[1], q.codes[2], q.codes[3]);
    } else {
        *reinterpret_cast<uint2*>(dst) = make_uint2(q.codes[0], q.codes[1]);
        side[scale_at<D>(is_v, at.t, lane)] = static_cast<uint8_t>(q.scale);
    }
    if (lane == 0) side[R::kScales + at.t] = static_cast<uint8_t>(q.exp);
}

// A lane's codes, scale and exponent.
template <int FMT, int D>
PKV_DEVINL Quantised load_row(const QuantArgs& a, bool is_v, const RowAt<FMT, D>& at, int lane) {
    using R = QuantRow<FMT, D>;
    const uint8_t* side = (is_v ? a.v_scales : a.k_scales) + at.side;
    const uint8_t* src = (is_v ? a.v_codes : a.k_codes) + at.codes;
    Quantised q;
    if constexpr (FMT == PKV_FP8) {
        const uint4 w = *reinterpret_cast<const uint4*>(src);
        q.codes[0] = w.x; q.codes[1] = w.y; q.codes[2] = w.z; q.codes[3] = w.w;
        q.scale = 0;
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(src);
        q.codes[0] = w.x; q.codes[1] = w.y;
        q.codes[2] = q.codes[3] = 0;
        q.scale = side[scale_at<D>(is_v, at.t, lane)];
    }
    q.exp = side[R::kScales + at.t];
    return q;
}

// Moves a lane's elements of K's and of V's row: READ from the cache, else into it (all lanes of the
// warp call; `go`: this one has a row).
template <int FMT, int D, typename T, bool READ>
PKV_DEVINL void move_rows(const QuantArgs& a, const RowAt<FMT, D>& at, bool go, int64_t k_at,
                          int64_t v_at, int lane) {
    if constexpr (READ) {
        if (!go) return;
        const Quantised k = load_row(a, false, at, lane), v = load_row(a, true, at, lane);
        float x[16];
        dequantise<FMT>(k.codes, k.scale, k.exp, x);
        Elems16<T>::store(static_cast<T*>(a.k_out) + k_at, a.wide, x);
        dequantise<FMT>(v.codes, v.scale, v.exp, x);
        Elems16<T>::store(static_cast<T*>(a.v_out) + v_at, a.wide, x);
    } else {
        Elems16<T> k, v;
        k.clear();
        v.clear();
        if (go) {
            k.load(static_cast<const T*>(a.k) + k_at, a.wide);
            v.load(static_cast<const T*>(a.v) + v_at, a.wide);
        }
        const Quantised qk = quantise<FMT, D>(k);
        if (go) store_row<FMT, D>(a, false, at, lane, qk);
        const Quantised qv = quantise<FMT, D>(v);
        if (go) store_row<FMT, D>(a, true, at, lane, qv);
    }
}

// Rows by slot.  READ: cache to rows, else rows to cache.
template <int FMT, int D, typename T, bool READ>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(const QuantArgs a) {
    constexpr int L = QuantRow<FMT, D>::kLanes;
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t row = blockIdx.x * (kThreads / L) + threadIdx.x / L;   // (token, head)
    const int lane = threadIdx.x % L;
    const bool there = row < a.num_rows;
    const uint32_t tok = there ? divide(row, a) : 0;
    const uint32_t head = there ? row - tok * a.num_kv_heads : 0;
    const int64_t slot = there ? __ldg(a.slots + tok) : -1;
    const int64_t in_row = static_cast<int64_t>(head) * D + 16 * lane;
    const int64_t k_at = tok * a.k_stride + in_row, v_at = tok * a.v_stride + in_row;
    const bool go = slot >= 0 && slot < a.num_slots;
    if (slot >= a.num_slots) raise_status(a.status, PKV_ERR_OOB);
    const uint32_t s = go ? static_cast<uint32_t>(slot) : 0;
    const RowAt<FMT, D> at(s >> a.block_shift, head, a, s & ((1u << a.block_shift) - 1), lane);
    move_rows<FMT, D, T, READ>(a, at, go, k_at, v_at, lane);
    if constexpr (READ) {
        if (!there || go) return;
        const float zeros[16] = {};   // padding, and slots past the cache
        Elems16<T>::store(static_cast<T*>(a.k_out) + k_at, a.wide, zeros);
        Elems16<T>::store(static_cast<T*>(a.v_out) + v_at, a.wide, zeros);
    }
}

// Whole blocks by pairs (source, destination).
template <int FMT, int D, typename T, bool READ>
__global__ void __launch_bounds__(kThreads) quant_blocks_kernel(const QuantArgs a) {
    constexpr int L = QuantRow<FMT, D>::kLanes;
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t row = blockIdx.x * (kThreads / L) + threadIdx.x / L;   // (pair, head, token)
    const int lane = threadIdx.x % L;
    const bool there = row < a.num_rows;
    const uint32_t pair = there ? divide(row, a) : 0;
    const uint32_t per = static_cast<uint32_t>(a.num_kv_heads) << a.block_shift;
    const uint32_t in = there ? row - pair * per : 0;
    const int src = __ldg(a.pairs + 2 * static_cast<size_t>(pair));
    const int dst = __ldg(a.pairs + 2 * static_cast<size_t>(pair) + 1);
    const int kept = READ ? src : dst, plain = READ ? dst : src;
    const bool ok = kept >= 0 && kept < a.num_blocks && plain >= 0 && plain < a.pool_blocks;
    if (!ok && there) raise_status(a.status, PKV_ERR_OOB);
    const bool go = ok && there;
    const RowAt<FMT, D> at(go ? kept : 0, in >> a.block_shift, a, in & ((1u << a.block_shift) - 1),
                           lane);
    const int64_t elem = (static_cast<int64_t>(go ? plain : 0) * per + in) * D + 16 * lane;
    move_rows<FMT, D, T, READ>(a, at, go, elem, elem, lane);
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
    return launch_pdl(kern, dim3((a.num_rows + per - 1) / per), dim3(kThreads), 0, stream, a);
}

template <int FMT, int D>
cudaError_t launch_dtype(const QuantArgs& a, int dtype, bool blocks, bool read,
                         cudaStream_t stream) {
    return dtype == PKV_BF16 ? launch_typed<FMT, D, uint16_t>(a, blocks, read, stream)
                             : launch_typed<FMT, D, float>(a, blocks, read, stream);
}

cudaError_t launch_format(const QuantArgs& a, int format, int head_dim, int dtype, bool blocks,
                          bool read, cudaStream_t stream) {
    if (format == PKV_FP8)
        return head_dim == 128 ? launch_dtype<PKV_FP8, 128>(a, dtype, blocks, read, stream)
                               : launch_dtype<PKV_FP8, 64>(a, dtype, blocks, read, stream);
    return head_dim == 128 ? launch_dtype<PKV_FP4, 128>(a, dtype, blocks, read, stream)
                           : launch_dtype<PKV_FP4, 64>(a, dtype, blocks, read, stream);
}

}  // namespace

cudaError_t launch_quant_move(const QuantArgs& a, int format, int head_dim, int dtype, bool blocks,
                              bool read, cudaStream_t stream) {
    // n / d = n mul >> shift for n < 2^31: mul is 2^shift / d rounded up, by less than 2^s / d of it
    // (2^s the power of two from d on), and n of that is less than 1 / d.
    QuantArgs b = a;
    const uint32_t d = blocks ? static_cast<uint32_t>(a.num_kv_heads) << a.block_shift
                              : static_cast<uint32_t>(a.num_kv_heads);
    int s = 0;
    while ((uint32_t{1} << s) < d) ++s;
    b.div_shift = 31 + s;
    b.div_mul = static_cast<uint32_t>(((uint64_t{1} << b.div_shift) + d - 1) / d);
    return launch_format(b, format, head_dim, dtype, blocks, read, stream);
}

cudaError_t launch_quant_copy(const QuantArgs& a, int num_pairs, int64_t code_bytes,
                              int64_t side_bytes, cudaStream_t stream) {
    return launch_pdl(quant_copy_kernel, dim3(num_pairs, 2), dim3(kThreads), 0, stream, a,
                      static_cast<int>(code_bytes / 16), static_cast<int>(side_bytes / 16));
}

}  // namespace pkv

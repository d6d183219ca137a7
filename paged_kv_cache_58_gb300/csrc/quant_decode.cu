// Paged decode over a quantised cache (fp8 or fp4 rows), on the tensor cores.
//
// One CTA per (partition, kv head, sequence), as over bf16 pools (paged_decode_tc.cu): warp w of four
// takes the pairs of 16-token chunks w, w + 4, ... of the partition through a ring of stages of its
// own and keeps its own online softmax, one step for the 32 tokens of a pair; the four states
// merge at the end, and partitions merge in the combine kernel.  (Chunk by chunk instead of in pairs:
// 4 % more time in fp8 and 20 % in fp4, before the weights had two parts.)  A chunk is
//   S^T[16 tokens x 8 heads] = K[16 x D] . q^T,   O^T[D x 8 heads] += V^T[D x 16] . P^T
// as fp16 MMAs m16n8k16 with fp32 sums.  fp16, because every e4m3 value is one of fp16, and so is
// every product of an e2m1 value and its e4m3 scale (6 digits, 2^-10 or more): what the MMAs
// multiply is the stored row over its power of two, exactly.  The powers of two go where they
// are exact too:
//   K's 2^e scales the token's scores (fp32);
//   V's 2^e goes into the weight: token j adds 2^((s_j - a) + (e_j - b)) code_j to O and 2^(s_j - a)
//     to the denominator, s the scores in powers of two.  a + b follows the largest s_j + e_j, the
//     size of what the token adds, so that the fp16 weights keep their digits where V's rows
//     differ in size by any power of two; a alone follows the largest score, so that s_j - a loses
//     nothing beside an exponent, and an exponent nothing beside a score of any size.
// a and b are whole numbers, raised only where a score would pass 2^8 or a weight 2^15 (the weights
// stay in fp16's range, the largest at 2^6 or more): one vote a pair, and the maxima over lanes only
// then.
// q is scaled by a power of two into fp16's range, for fp32 in two fp16 parts.  A weight is two
// fp16 parts (22 digits; in one it was off by up to 2^-12, and V's of one sign add that up).  The
// low parts take MMAs of their own for groups of 8 heads, and for smaller ones the idle columns 4 ..
// 7, whose sums join at the end.
//
// Copies.  A pair's 4 to 8 KB come 16 bytes a lane (cp.async, swizzled by the lane, counted on an
// mbarrier), 512 bytes an instruction.  As eight bulk and tensor copies a pair, each lane's own and
// so issued one after the other, they took 30 instructions more (1 % of the time in fp8, 3 in fp4) and
// tensor maps for every call's arrays.
//
// Bound.  fp8: HBM (16 x 16k .. 128k tokens, 8 query heads to a kv head: 407 us a call, 6.9 TB/s; 64 x
// 512 .. 4096: 53 us, 5.8 TB/s, a sixth of it the first copies, the ends of CTAs and the combine).
// fp4: its bytes would take 236 us where the long batch takes 346, with 352 warp instructions a chunk,
// 128 of them to make fp16 of 4096 codes (two values each for cvt.f16x2.e2m1x2 and for the product with
// the scale), issued at 2.5 of 4 a clock by 12 warps an SM: instructions and their latency both.
//
// Fragments.  The index that an MMA sums over may be in any order, if both sides share it.  So
// lane (g, j) = (lane / 4, lane % 4) takes elements j D / 4 .. of K's row as they lie, and the
// same of q; V^T comes out of ldmatrix .m16n16.trans.b8 with 4 tokens of one dimension (fp4: of
// two) in a register, tokens 4 j .. 4 j + 3; row g of S^T is token 4 (g / 2) + g % 2 and row
// g + 8 the token two further, which is the order in which movmatrix hands the weights on.
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kBlk = 16;
constexpr float kTop = 15.f;     // weights are at most 2^kTop
constexpr float kStart = 7.f;    // and the largest one is put at about 2^kStart
constexpr float kFar = 8.f;      // scores are at most this far above their reference

template <int FMT, int D, int G>
struct QuantSmem {
    using R = QuantRow<FMT, D>;
    static constexpr int kSlab = kBlk * R::kCodes;
    // A stage: K and V of two chunks.  The loop is unrolled over the stages, and past two its code
    // costs more than copies further ahead bring (head_dim 64, 64 x 512 .. 4096 and 16 x 16k .. 128k
    // tokens, fp8: 33.8 and 216 us, four stages 38.9 and 222, six 50.5 and 262; fp4 36.2 and 216, 43.1
    // and 249, 48.9 and 289).
    static constexpr int kStages = 2;
    static constexpr int kCodeRing = kWarps * kStages * 4 * kSlab;
    static constexpr int kSideRing = kWarps * kStages * 4 * R::kSide;
    static constexpr int kBars = kWarps * kStages * 8;
    // merge scratch reuses the rings once every warp is done
    static constexpr int kMerge = kWarps * G * D * 4 + 3 * kWarps * G * 4;
    static constexpr int kBody = kCodeRing + kSideRing > kMerge ? kCodeRing + kSideRing : kMerge;
    static constexpr int kTotal = kBody + kBars + 1024;   // + alignment slack
    static_assert(kBody % 8 == 0 && R::kSide % 16 == 0, "alignment");
};

PKV_DEVINL void ldsm_t_b8(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                          uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}
// 16 bytes from global to shared memory, or 16 zeros (bytes == 0: src is not read).
PKV_DEVINL void copy16(uint32_t dst, const uint8_t* src, uint32_t bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
                 "l"(src), "r"(bytes), "l"(policy)
                 : "memory");
}
// This thread arrives at `bar` once its copies so far have landed.
PKV_DEVINL void arrive_with_copies(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
PKV_DEVINL uint4 lds128(uint32_t addr) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(addr));
    return r;
}
PKV_DEVINL uint2 lds64(uint32_t addr) {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr));
    return r;
}
PKV_DEVINL uint32_t lds16(uint32_t addr) {
    uint32_t r;
    asm volatile("{\n\t.reg .b16 h;\n\tld.shared.b16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}"
                 : "=r"(r)
                 : "r"(addr));
    return r;
}
PKV_DEVINL uint32_t lds8(uint32_t addr) {
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(addr));
    return r;
}
PKV_DEVINL uint32_t movm_t(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
PKV_DEVINL uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// D = A (16x16 fp16, row) * B (16x8 fp16, col) + D, fp32 accumulate.
PKV_DEVINL void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Where the 16-byte piece c of row t of a slab lies: swizzled so that eight rows' pieces c, and four
// pieces of two rows, lie in banks of their own.
template <int ROW>
PKV_DEVINL uint32_t piece_at(uint32_t base, int t, int c) {
    const int f = ROW == 128 ? t & 7 : ROW == 64 ? (t >> 1) & 3 : (t >> 2) & 1;
    return base + t * ROW + ((c ^ f) << 4);
}

// Four tokens' bytes of two fp4 codes (dimensions d, d + 1): the codes in pairs of tokens, of d and of
// d + 1 in turn (a swap of the middle two codes of each half).
PKV_DEVINL uint32_t pair_tokens(uint32_t r) {
    const uint32_t t = (r ^ (r >> 4)) & 0x00f000f0u;
    return r ^ (t * 17u);
}

PKV_DEVINL void store_out(uint16_t* p, float x) {
    *p = static_cast<uint16_t>(pack_bf16x2(x, 0.f) & 0xffffu);
}
PKV_DEVINL void store_out(float* p, float x) { *p = x; }

// The new token's rows, quantised: into the stage (row t of the slabs and of what lies beside
// them) and into the cache.  K's by lanes 0 .. D / 16 - 1, V's by as many after them.
template <int FMT, int D, typename T>
__device__ __noinline__ void append_row(const DecodeArgs& a, const QuantSides& qs, int seq, int kvh,
                                        int blk, int t, const int32_t* bt, int lane, uint8_t* kst,
                                        uint8_t* vst, uint8_t* ksd, uint8_t* vsd) {
    using R = QuantRow<FMT, D>;
    const int which = lane / R::kLanes, ln = lane % R::kLanes;
    const bool mine = which < 2, v = which == 1;
    Elems16<T> in;
    in.clear();
    if (mine)
        in.load(static_cast<const T*>(v ? a.v_new : a.k_new) +
                    (static_cast<size_t>(seq) * a.num_kv_heads + kvh) * D + 16 * ln, false);
    const Quantised q = quantise<FMT, D>(in);
    if (!mine) return;
    const int phys = __ldg(bt + (blk >> a.chunk_shift));
    const bool there = phys >= 0 && phys < a.num_blocks;
    const size_t chunk = ((static_cast<size_t>(there ? phys : 0) * a.num_kv_heads + kvh)
                          << a.chunk_shift) + (blk & ((1 << a.chunk_shift) - 1));
    uint8_t* pool = static_cast<uint8_t*>(const_cast<void*>(v ? a.v_pool : a.k_pool)) +
                    (chunk * kBlk + t) * R::kCodes + ln * R::kLaneBytes;
    uint8_t* pside = (v ? qs.v : qs.k) + chunk * R::kSide;
    uint8_t* slab = v ? vst : kst;
    uint8_t* side = v ? vsd : ksd;
    if constexpr (FMT == PKV_FP8) {
        const uint4 w = make_uint4(q.codes[0], q.codes[1], q.codes[2], q.codes[3]);
        *reinterpret_cast<uint4*>(slab + piece_at<R::kCodes>(0, t, ln)) = w;
        if (there) *reinterpret_cast<uint4*>(pool) = w;
    } else {
        const uint2 w = make_uint2(q.codes[0], q.codes[1]);
        *reinterpret_cast<uint2*>(slab + piece_at<R::kCodes>(0, t, ln >> 1) + 8 * (ln & 1)) = w;
        const int at = scale_at<D>(v, t, ln);
        side[at] = static_cast<uint8_t>(q.scale);
        if (there) {
            *reinterpret_cast<uint2*>(pool) = w;
            pside[at] = static_cast<uint8_t>(q.scale);
        }
    }
    if (ln == 0) {
        side[R::kScales + t] = static_cast<uint8_t>(q.exp);
        if (there) pside[R::kScales + t] = static_cast<uint8_t>(q.exp);
    }
}

// q of one head: E elements from p on, scaled by the power of two that puts the head's largest
// element into [2^14, 2^15), as fp16 pairs (and what they leave, for fp32).  Returns the scale's
// inverse.  The four lanes of a head call together.
template <typename T, int E, bool SPLIT>
PKV_DEVINL float load_q(const T* p, bool there, uint32_t (&hi)[E / 4][2],
                        uint32_t (&lo)[SPLIT ? E / 4 : 1][2]) {
    float x[E];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < E / 16; ++i) {
        float v[16];
        Elems16<T> in;
        in.clear();
        if (there) in.load(p + 16 * i, false);
        in.values(v);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            x[16 * i + k] = v[k];
            top = fmaxf(top, fabsf(v[k]));
        }
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int up = min(126, 14 + 127 - (__float_as_int(top) >> 23));   // -114 .. 126
    const float f = pow2f(up);
#pragma unroll
    for (int ks = 0; ks < E / 4; ++ks)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float u = x[4 * ks + 2 * h] * f, v = x[4 * ks + 2 * h + 1] * f;
            hi[ks][h] = pack_f16x2(u, v);
            if constexpr (SPLIT)
                lo[ks][h] = pack_f16x2(u - f16lo_to_f32(hi[ks][h]), v - f16hi_to_f32(hi[ks][h]));
        }
    return pow2f(max(-126, -up));
}

// CTAs that share an SM: four for bf16 rows of 64, three of 168 registers a thread for the others (us
// with three / four / five, of 168, 128 and 96 registers, 64 x 512 .. 4096 and 16 x 16k .. 128k tokens:
// head_dim 64 fp8 34.7 / 33.8 / 34.9 and 218 / 216 / 216, fp4 37.4 / 36.2 / 41.1 and 230 / 216 / 249;
// head_dim 128 fp4, where 128 registers spill, 53.3 / 56.4 / 68.3 and 345 / 359 / 450; fp8 rows of 128
// have 66 KB of rings a CTA).
template <int D, typename T>
constexpr int kCtas = sizeof(T) == 2 && D == 64 ? 4 : 3;

template <int FMT, int D, int G, typename T>
__global__ void __launch_bounds__(kThreads, kCtas<D, T>)
quant_decode_kernel(const DecodeArgs a, const QuantSides qs) {
    using SM = QuantSmem<FMT, D, G>;
    using R = QuantRow<FMT, D>;
    constexpr int KS = D / 16;            // k-steps of the scores, m-tiles of P.V
    constexpr int kStages = SM::kStages;
    constexpr bool kSplit = sizeof(T) == 4;   // fp32: q in two fp16 parts
    constexpr bool kBeside = G <= 4;      // a weight's low part: in column g + 4, or in MMAs of its own
    constexpr int E = D / 4;              // elements of a K row in one lane
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));

    griddep_wait();
    griddep_launch_dependents();
    // Partitions before sequences: with the first partitions of all sequences first, as the pools'
    // decode has them, the CTAs of a wave are equally long, end together, and leave HBM idle
    // while the next ones start (64 sequences of 512 .. 4096 tokens, fp8: 59.2 us; 56.0 so).
    const int kvh = blockIdx.x;
    const int part = blockIdx.y;
    const int seq = blockIdx.z;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    const int32_t* bt = a.block_tables + static_cast<size_t>(seq) * a.max_blocks_per_seq;
    const int b0 = part * a.partition_chunks;
    // Warp w takes the pairs of chunks w, w + 4, ...; lane l keeps the block id of chunk l % 2 of
    // pair l / 2 of 16 pairs.  The first ones do not wait for the length.
    const int my_first = b0 + 2 * warp + 2 * kWarps * (lane >> 1) + (lane & 1);
    int ids0;
    {
        const int e = my_first >> a.chunk_shift;
        ids0 = e < a.max_blocks_per_seq ? __ldg(bt + e) : -1;
    }
    int L = a.context_lens[seq];
    const int span = a.max_parts * a.partition_chunks;
    const int max_chunks = a.max_blocks_per_seq << a.chunk_shift;
    bool append = a.k_new != nullptr;
    if (L > min(max_chunks, span) * static_cast<int64_t>(kBlk)) {
        if (part == 0 && threadIdx.x == 0) raise_status(a.status, PKV_ERR_OOB);
        L = static_cast<int>(min(min(max_chunks, span) * static_cast<int64_t>(kBlk),
                                 static_cast<int64_t>(0x7ffffff0)));
        append = false;   // the clamped end is not the new token
    }
    const int nblk = (L + kBlk - 1) / kBlk;
    if (L <= 0 || b0 >= nblk) {   // uniform over the CTA, before any barrier
        if (L <= 0 && part == 0) {
            if (threadIdx.x == 0) raise_status(a.status, PKV_ERR_INVALID);
            zero_invalid_rows(a, seq, kvh, G, D, sizeof(T));
        }
        return;
    }
    const int b1 = min(nblk, b0 + a.partition_chunks);
    const int my_count = max(0, (b1 - b0 - 2 * warp + 2 * kWarps - 1) / (2 * kWarps));   // pairs

    uint8_t* ring = smem + warp * kStages * 4 * SM::kSlab;
    uint8_t* sides = smem + SM::kCodeRing + warp * kStages * 4 * R::kSide;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::kBody) + warp * kStages;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) mbar_init(&bars[i], 32);
        fence_mbar_init();
    }
    __syncwarp();

    // A sequence reads each byte once.  (A block that many tables name is read by each of them, and
    // under the same policy.)
    const uint64_t stream_policy = l2_policy_evict_first();
    int ids = my_first < b1 ? ids0 : -1;
    auto fetch_ids = [&](int base) {
        const int c = my_first + 2 * kWarps * base;
        ids = c < b1 ? __ldg(bt + (c >> a.chunk_shift)) : -1;
    };
    // Pair i into stage st, 16 bytes a lane and copy: 512 bytes of codes lie in 4, 8 or 16 rows.
    constexpr int kPieces = R::kCodes / 16;    // of a row
    const int lane_row = lane / kPieces, lane_pc = lane % kPieces;
    const uint8_t* codes[2] = {static_cast<const uint8_t*>(a.k_pool) + 16 * lane,
                               static_cast<const uint8_t*>(a.v_pool) + 16 * lane};
    const uint32_t lane_dst = smem_u32(ring) + piece_at<R::kCodes>(0, lane_row, lane_pc);
    // What lies beside a chunk's K and V: lanes 0 .. and as many after them.
    constexpr int kSidePieces = R::kSide / 16;
    const int side_v = lane / kSidePieces, side_pc = lane % kSidePieces;
    const bool lane_side = side_v < 2;
    const uint8_t* side_src = (side_v == 1 ? qs.v : qs.k) + 16 * side_pc;
    const uint32_t side_dst = smem_u32(sides) + (side_v & 1) * R::kSide + 16 * side_pc;
    const int block_step = a.num_kv_heads << a.chunk_shift;
    const int block_at = kvh << a.chunk_shift;
    bool lost = false;   // a block id outside the pool
    int next = b0 + 2 * warp;   // the next pair's first chunk
    auto issue = [&](int st, int i, bool arrive) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int phys = __shfl_sync(0xffffffffu, ids, 2 * (i & 15) + u);
            const bool there = u == 0 || next + 1 < b1;
            const bool ok = static_cast<uint32_t>(phys) < static_cast<uint32_t>(a.num_blocks);
            lost |= there && !ok;
            const uint32_t bytes = there && ok ? 16u : 0u;
            // (blocks of two chunks: b0 is even there)
            const int chunk = (ok ? phys : 0) * block_step + block_at + (a.chunk_shift & u);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint8_t* src = codes[kv] + static_cast<int64_t>(chunk) * SM::kSlab;
                const uint32_t dst = lane_dst + (4 * st + 2 * u + kv) * SM::kSlab;
#pragma unroll
                for (int p = 0; p < SM::kSlab / 512; ++p)   // rows of 128: four on turn the swizzle
                    copy16((R::kCodes == 128 && (p & 1) ? dst ^ 64 : dst) + 512 * p, src + 512 * p,
                           bytes, stream_policy);
            }
            if (lane_side)
                copy16(side_dst + (4 * st + 2 * u) * R::kSide,
                       side_src + static_cast<int64_t>(chunk) * R::kSide, bytes, stream_policy);
        }
        if (arrive) arrive_with_copies(&bars[st]);
        next += 2 * kWarps;
    };
    const bool stall = a.test_stall && warp == 0 && blockIdx.x == 0 && blockIdx.y == 0 &&
                       blockIdx.z == 0;
#pragma unroll
    for (int i = 0; i < kStages; ++i)
        if (i < my_count) issue(i, i, !(stall && i == 0 && lane == 0));

    // q: head g, elements j E ..  (kBeside: columns 4 .. 7 take the heads of 0 .. 3 again)
    const int g8 = lane >> 2;
    const int j4 = lane & 3;
    const int head = kBeside ? g8 & 3 : g8;
    uint32_t qb[KS][2], ql[kSplit ? KS : 1][2];
    const float q_unit = load_q<T, E, kSplit>(
        static_cast<const T*>(a.q) +
            (static_cast<size_t>(seq) * a.num_q_heads + kvh * G + (head < G ? head : 0)) * D + j4 * E,
        head < G, qb, ql);
    // Scores are held for heads 2 j, 2 j + 1 of tokens t_lo and t_lo + 2.
    const int t_lo = 4 * (g8 >> 1) + (g8 & 1);
    float hs[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        hs[h] = a.scale_log2 * __shfl_sync(0xffffffffu, q_unit, (2 * j4 + h) * 4);

    float acc[KS][4];
#pragma unroll
    for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mt][e] = 0.f;
    // Finite (a chunk of -inf scores adds zeros), and so low that any other score raises them.
    float a_ref[2] = {-3.4028235e38f, -3.4028235e38f}, b_ref[2] = {-200.f, -200.f};
    float l_part[2] = {0.f, 0.f};   // this lane's share of the denominators, over 2^a_ref

    // ldmatrix row of this lane: token lane % 16, piece 2 i + lane / 16
    const int v_tok = lane & 15;
    const int v_pc = lane >> 4;

    const int full_end = min(b1, L / kBlk);
    // Pairs that reach past this have rows to clear, or the new token.
    const int plain_end = append && b1 == nblk ? min(full_end, nblk - 1) : full_end;
    int failed_at = -1;
    uint32_t phase = 0;
    int c0 = b0 + 2 * warp;
    for (int i0 = 0; i0 < my_count && failed_at < 0; i0 += kStages, phase ^= 1) {
#pragma unroll
    for (int st_i = 0; st_i < kStages; ++st_i, c0 += 2 * kWarps) {
        const int i = i0 + st_i;
        if (i >= my_count) break;
        if (!mbar_wait_warp(&bars[st_i], phase, a.status)) {
            failed_at = i;
            break;
        }
        uint8_t* slabs = ring + 4 * st_i * SM::kSlab;     // K, V of the first chunk, of the second
        uint8_t* besides = sides + 4 * st_i * R::kSide;
        const uint32_t slab0 = smem_u32(slabs), side0 = smem_u32(besides);
        const bool full = c0 + 2 <= full_end;

        if (c0 + 2 > plain_end) {
            for (int u = 0; u < 2; ++u) {
                const int blk = c0 + u;
                const int valid = blk < b1 ? min(kBlk, L - blk * kBlk) : 0;
                uint8_t* kst = slabs + 2 * u * SM::kSlab;
                uint8_t* vst = kst + SM::kSlab;
                uint8_t* ksd = besides + 2 * u * R::kSide;
                uint8_t* vsd = ksd + R::kSide;
                // Rows past the context may hold anything (an fp8 NaN, an fp4 scale that is
                // one): zero V's, so that a weight of zero adds zero.
                for (int idx = lane; idx < (kBlk - valid) * kPieces; idx += 32)
                    *reinterpret_cast<uint4*>(vst + piece_at<R::kCodes>(0, valid + idx / kPieces,
                                                                        idx % kPieces)) =
                        make_uint4(0, 0, 0, 0);
                if constexpr (FMT == PKV_FP4) {
                    for (int idx = lane; idx < (kBlk - valid) * KS; idx += 32)
                        vsd[scale_at<D>(true, valid + idx / KS, idx % KS)] = 0;
                }
                if (append && blk == nblk - 1 && blk < b1)   // holds the new token, row valid - 1
                    append_row<FMT, D, T>(a, qs, seq, kvh, blk, valid - 1, bt, lane, kst, vst, ksd,
                                          vsd);
            }
            __syncwarp();
        }

        // S^T = K . q^T
        float s[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][e] = 0.f;
        if constexpr (FMT == PKV_FP8) {
#pragma unroll
            for (int p = 0; p < E / 16; ++p) {
                uint32_t va[2][4], vb[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t kb = slab0 + 2 * u * SM::kSlab;
                    const uint4 wa = lds128(piece_at<R::kCodes>(kb, t_lo, j4 * (E / 16) + p));
                    const uint4 wb = lds128(piece_at<R::kCodes>(kb, t_lo + 2, j4 * (E / 16) + p));
                    va[u][0] = wa.x; va[u][1] = wa.y; va[u][2] = wa.z; va[u][3] = wa.w;
                    vb[u][0] = wb.x; vb[u][1] = wb.y; vb[u][2] = wb.z; vb[u][3] = wb.w;
                }
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_to_f16x4(va[u][w], a0, a2);
                        e4m3x4_to_f16x4(vb[u][w], a1, a3);
                        const int ks = 4 * p + w;
                        mma_f16(s[u], a0, a1, a2, a3, qb[ks][0], qb[ks][1]);
                        if constexpr (kSplit) mma_f16(s[u], a0, a1, a2, a3, ql[ks][0], ql[ks][1]);
                    }
            }
        } else {
            uint32_t va[2][E / 8], vb[2][E / 8], sa[2], sb[2];   // scales: of a group, or two
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t kb = slab0 + 2 * u * SM::kSlab, ksb = side0 + 2 * u * R::kSide;
                if constexpr (D == 128) {
                    const uint4 wa = lds128(piece_at<R::kCodes>(kb, t_lo, j4));
                    const uint4 wb = lds128(piece_at<R::kCodes>(kb, t_lo + 2, j4));
                    va[u][0] = wa.x; va[u][1] = wa.y; va[u][2] = wa.z; va[u][3] = wa.w;
                    vb[u][0] = wb.x; vb[u][1] = wb.y; vb[u][2] = wb.z; vb[u][3] = wb.w;
                    sa[u] = e4m3x2_to_f16x2(lds16(ksb + t_lo * 8 + 2 * j4));
                    sb[u] = e4m3x2_to_f16x2(lds16(ksb + (t_lo + 2) * 8 + 2 * j4));
                } else {
                    const uint2 wa =
                        lds64(piece_at<R::kCodes>(kb, t_lo, j4 >> 1) + 8 * (j4 & 1));
                    const uint2 wb =
                        lds64(piece_at<R::kCodes>(kb, t_lo + 2, j4 >> 1) + 8 * (j4 & 1));
                    va[u][0] = wa.x; va[u][1] = wa.y;
                    vb[u][0] = wb.x; vb[u][1] = wb.y;
                    sa[u] = e4m3x2_to_f16x2(lds8(ksb + t_lo * 4 + j4));
                    sb[u] = e4m3x2_to_f16x2(lds8(ksb + (t_lo + 2) * 4 + j4));
                }
            }
#pragma unroll
            for (int w = 0; w < E / 8; ++w)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t xa[4], xb[4];
                    e2m1x8_to_f16x8(va[u][w], xa);
                    e2m1x8_to_f16x8(vb[u][w], xb);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        xa[e] = w < 2 ? hmul2_lo(xa[e], sa[u]) : hmul2_hi(xa[e], sa[u]);
                        xb[e] = w < 2 ? hmul2_lo(xb[e], sb[u]) : hmul2_hi(xb[e], sb[u]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int ks = 2 * w + h;
                        mma_f16(s[u], xa[2 * h], xb[2 * h], xa[2 * h + 1], xb[2 * h + 1],
                                qb[ks][0], qb[ks][1]);
                        if constexpr (kSplit)
                            mma_f16(s[u], xa[2 * h], xb[2 * h], xa[2 * h + 1], xb[2 * h + 1],
                                    ql[ks][0], ql[ks][1]);
                    }
                }
        }
        // scores in powers of two, and the exponents of V's rows: their bytes as the low digits of
        // 2^23, from which one subtraction takes kBias and b
        constexpr float kBias = 8388608.f + 127.f;
        float ve[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = side0 + 2 * u * R::kSide + R::kScales + t_lo + 2 * h;
                const float unit = __int_as_float(lds8(at) << 23);
                ve[u][h] = __int_as_float(lds8(at + R::kSide) | 0x4b000000);
#pragma unroll
                for (int e = 0; e < 2; ++e)   // (in this order: unit * hs may pass fp32's range)
                    s[u][2 * h + e] = s[u][2 * h + e] * unit * hs[e];
                if (!full) {
                    const int blk = c0 + u;
                    if (t_lo + 2 * h >= (blk < b1 ? L - blk * kBlk : 0)) {
                        s[u][2 * h] = s[u][2 * h + 1] = -INFINITY;
                        ve[u][h] = kBias;
                    }
                }
            }
        // Over the references: t = (s - a) + (e - b), the first difference and the second each exact
        // where it counts, and s - a.
        float d[2][4], t[2][4];
        float most_d = -INFINITY, most_t = -INFINITY;
        auto refer = [&] {
            const float bias[2] = {kBias + b_ref[0], kBias + b_ref[1]};
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        d[u][2 * h + e] = s[u][2 * h + e] - a_ref[e];
                        t[u][2 * h + e] = d[u][2 * h + e] + (ve[u][h] - bias[e]);
                    }
                    most_d = fmax3(most_d, d[u][2 * h], d[u][2 * h + 1]);
                    most_t = fmax3(most_t, t[u][2 * h], t[u][2 * h + 1]);
                }
        };
        refer();
        if (__any_sync(0xffffffffu, most_d > kFar || most_t > kTop)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float ms = fmaxf(fmaxf(s[0][h], s[0][2 + h]), fmaxf(s[1][h], s[1][2 + h]));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, o));
                const float a_new = ms > a_ref[h] + kFar ? ceilf(ms) : a_ref[h];
                const float shift = a_ref[h] - a_new;
                const float b_same = b_ref[h] + shift;   // a + b as it was
                float mt = -INFINITY;
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    mt = fmax3(mt, (s[u][h] - a_new) + (ve[u][0] - kBias),
                               (s[u][2 + h] - a_new) + (ve[u][1] - kBias));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
                const float b_new = mt > b_same + kTop ? ceilf(mt) - kStart : b_same;
                a_ref[h] = a_new;
                b_ref[h] = b_new;
                l_part[h] *= fast_exp2(shift);
                const float al = b_same == b_new ? 1.f : fast_exp2(b_same - b_new);
#pragma unroll
                for (int m = 0; m < KS; ++m) {
                    acc[m][h] *= al;
                    acc[m][2 + h] *= al;
                }
            }
            refer();
        }
        // P^T fragments: [token][head] 8x8 tiles transposed in registers, (4 j, 4 j + 1) and the two
        // tokens after them of head g.  A weight is two fp16 parts, 22 digits.
        uint32_t ph[2][2], pl[kBeside ? 1 : 2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[e] = fast_exp2(t[u][e]);
                l_part[e & 1] += fast_exp2(d[u][e]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t hi = pack_f16x2(p[2 * h], p[2 * h + 1]);
                const uint32_t lo = pack_f16x2(p[2 * h] - f16lo_to_f32(hi),
                                               p[2 * h + 1] - f16hi_to_f32(hi));
                if constexpr (kBeside) {
                    ph[u][h] = movm_t(j4 < 2 ? hi : lo);
                } else {
                    ph[u][h] = movm_t(hi);
                    pl[u][h] = movm_t(lo);
                }
            }
        }
        // O^T += V^T . P^T
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t vbase = slab0 + (2 * u + 1) * SM::kSlab;
            if constexpr (FMT == PKV_FP8) {
#pragma unroll
                for (int p2 = 0; p2 < KS / 2; ++p2) {   // 32 dimensions
                    uint32_t r[4];
                    ldsm_t_b8(piece_at<R::kCodes>(vbase, v_tok, 2 * p2 + v_pc), r[0], r[1], r[2],
                              r[3]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_to_f16x4(r[2 * h], a0, a2);
                        e4m3x4_to_f16x4(r[2 * h + 1], a1, a3);
                        mma_f16(acc[2 * p2 + h], a0, a1, a2, a3, ph[u][0], ph[u][1]);
                        if constexpr (!kBeside)
                            mma_f16(acc[2 * p2 + h], a0, a1, a2, a3, pl[u][0], pl[u][1]);
                    }
                }
            } else {
                const uint32_t vsb = side0 + (2 * u + 1) * R::kSide;
                uint32_t sc[KS];
#pragma unroll
                for (int q4 = 0; q4 < KS / 4; ++q4) {
                    const uint4 w = lds128(vsb + j4 * (D / 4) + 16 * q4);
                    sc[4 * q4] = w.x; sc[4 * q4 + 1] = w.y;
                    sc[4 * q4 + 2] = w.z; sc[4 * q4 + 3] = w.w;
                }
#pragma unroll
                for (int p2 = 0; p2 < KS / 4; ++p2) {   // 64 dimensions
                    uint32_t r[4];
                    ldsm_t_b8(piece_at<R::kCodes>(vbase, v_tok, 2 * p2 + v_pc), r[0], r[1], r[2],
                              r[3]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {       // 32 dimensions: two groups
                        // Dimensions d and d + 1 of four tokens, d + 16 and d + 17: as pairs of
                        // tokens, of d and of d + 1 in turn.
                        uint32_t x[4], y[4], s01, s23, z01, z23;
                        e2m1x8_to_f16x8(pair_tokens(r[2 * h]), x);
                        e2m1x8_to_f16x8(pair_tokens(r[2 * h + 1]), y);
                        const int g0 = 4 * p2 + 2 * h;      // scales of those tokens
                        e4m3x4_to_f16x4(sc[g0], s01, s23);
                        e4m3x4_to_f16x4(sc[g0 + 1], z01, z23);
#pragma unroll
                        for (int odd = 0; odd < 2; ++odd) {
                            const uint32_t a0 = hmul2(x[odd], s01), a2 = hmul2(x[2 + odd], s23);
                            const uint32_t a1 = hmul2(y[odd], z01), a3 = hmul2(y[2 + odd], z23);
                            mma_f16(acc[g0 + odd], a0, a1, a2, a3, ph[u][0], ph[u][1]);
                            if constexpr (!kBeside)
                                mma_f16(acc[g0 + odd], a0, a1, a2, a3, pl[u][0], pl[u][1]);
                        }
                    }
                }
            }
        }
        __syncwarp();
        const int nxt = i + kStages;
        if (nxt < my_count) {
            if ((nxt & 15) == 0) fetch_ids(nxt);
            issue(st_i, nxt, true);
        }
    }
    }
    if (lost && lane == 0) raise_status(a.status, PKV_ERR_OOB);
    if (failed_at >= 0) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (int k = failed_at + 1; k < my_count && k < failed_at + kStages; ++k)
            mbar_wait_warp(&bars[k % kStages], (k / kStages) & 1, a.status);
    }

    if constexpr (kBeside) {   // what the low parts summed, two lanes further
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][e] += __shfl_xor_sync(0xffffffffu, acc[mt][e], 2);
    }
    // This warp's output over its denominators, and over 1.  b is 91 at most (a score 8 above a, an
    // exponent of 90, less 7) and -106 at least (no weight passes 2^15) once anything counts.
    float inv[2], unit[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
            l_part[h] += __shfl_xor_sync(0xffffffffu, l_part[h], o);
        inv[h] = l_part[h] == 0.f ? 0.f : 1.f / l_part[h];   // zero: no tokens, or none with weight
        unit[h] = pow2f(static_cast<int>(fmaxf(-126.f, fminf(126.f, b_ref[h]))));
    }
    __syncthreads();  // every warp is done with its ring: reuse it as merge scratch
    float* macc = reinterpret_cast<float*>(smem);            // [W][G][D], over the denominator
    float* mm = macc + kWarps * G * D;                       // [W][G]
    float* ml = mm + kWarps * G;                             // [W][G]
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int h = 2 * j4 + hh;
        if (h < G) {
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
                float* row = macc + (warp * G + h) * D;
                // fp8: dimensions 16 mt + g and + 8.  fp4: the even or the odd ones of 32, + 16
                const int d0 = FMT == PKV_FP8 ? 16 * mt + g8
                                              : 32 * (mt >> 1) + 2 * g8 + (mt & 1);
                row[d0] = acc[mt][hh] * inv[hh] * unit[hh];
                row[d0 + (FMT == PKV_FP8 ? 8 : 16)] = acc[mt][2 + hh] * inv[hh] * unit[hh];
            }
            if (g8 == 0) {
                mm[warp * G + h] = my_count > 0 ? a_ref[hh] : -INFINITY;
                ml[warp * G + h] = my_count > 0 ? l_part[hh] : 0.f;
            }
        }
    }
    __syncthreads();
    // What each warp's output counts, of all four denominators.
    const size_t row0 = static_cast<size_t>(seq) * a.num_q_heads + kvh * G;
    const bool whole = a.max_parts == 1;
    float* share = ml + kWarps * G;                          // [W][G]
    if (threadIdx.x < G) {
        const int g = threadIdx.x;
        float M = -INFINITY, l = 0.f, f[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mm[w * G + g]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            f[w] = fast_exp2(mm[w * G + g] - M) * ml[w * G + g];
            l += f[w];
        }
        // no weight at all: 0 / 0, as the softmax has it, but in a part of a row zeros
        const float inv_l = !whole && l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) share[w * G + g] = f[w] * inv_l;
        if (!whole) {
            // The denominator's power of two joins M where that is exact, so that the combine's
            // products of l and outputs stay in range; beyond, scores differ by 1 / 2 or not at all.
            if (fabsf(M) < 0x1p22f && l > 0.f && l < INFINITY) {
                const int e = (__float_as_int(l) >> 23) - 127;
                M += static_cast<float>(e);
                l *= pow2f(max(-126, min(126, -e)));
            }
            a.m_part[(row0 + g) * a.max_parts + part] = M;
            a.l_part[(row0 + g) * a.max_parts + part] = l;
        }
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < G * D; idx += kThreads) {
        const int g = idx / D;
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) o = fmaf(share[w * G + g], macc[w * G * D + idx], o);
        if (whole)
            store_out(static_cast<T*>(a.out) + row0 * D + idx, o);
        else
            a.o_part[((row0 + g) * a.max_parts + part) * D + idx % D] = o;
    }
}

template <int FMT, int D, int G, typename T>
cudaError_t launch_quant(const DecodeArgs& a, const QuantSides& qs, cudaStream_t stream) {
    using SM = QuantSmem<FMT, D, G>;
    auto kern = quant_decode_kernel<FMT, D, G, T>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), SM::kTotal);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(a.num_kv_heads, a.max_parts, a.num_seqs), dim3(kThreads), SM::kTotal,
                   stream, a, qs);
    if (e != cudaSuccess || a.max_parts == 1) return e;
    return launch_decode_combine(a, sizeof(T) == 4 ? PKV_F32 : PKV_BF16, D, stream);
}

template <int FMT, int D, typename T>
cudaError_t launch_group(const DecodeArgs& a, const QuantSides& qs, int G, cudaStream_t stream) {
    switch (G) {
        case 1: return launch_quant<FMT, D, 1, T>(a, qs, stream);
        case 2: return launch_quant<FMT, D, 2, T>(a, qs, stream);
        case 4: return launch_quant<FMT, D, 4, T>(a, qs, stream);
        case 8: return launch_quant<FMT, D, 8, T>(a, qs, stream);
        default: return cudaErrorInvalidValue;
    }
}

template <int FMT, typename T>
cudaError_t launch_dim(const DecodeArgs& a, const QuantSides& qs, int D, int G,
                       cudaStream_t stream) {
    return D == 128 ? launch_group<FMT, 128, T>(a, qs, G, stream)
                    : launch_group<FMT, 64, T>(a, qs, G, stream);
}

}  // namespace

cudaError_t launch_quant_decode(const DecodeArgs& a, const QuantSides& qs, int format, int dtype,
                                int head_dim, int group, cudaStream_t stream) {
    if (format == PKV_FP8)
        return dtype == PKV_BF16 ? launch_dim<PKV_FP8, uint16_t>(a, qs, head_dim, group, stream)
                                 : launch_dim<PKV_FP8, float>(a, qs, head_dim, group, stream);
    return dtype == PKV_BF16 ? launch_dim<PKV_FP4, uint16_t>(a, qs, head_dim, group, stream)
                             : launch_dim<PKV_FP4, float>(a, qs, head_dim, group, stream);
}

}  // namespace pkv

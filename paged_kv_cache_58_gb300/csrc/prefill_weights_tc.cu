// Accumulated attention weights of a prompt chunk for bf16 pools, on the tcgen05 tensor
// cores.  The mathematics, and why there are two passes over Q K^T, is in
// prefill_weights.cu; here both passes are one kernel skeleton:
//
//   pass 1 (row statistics)  S[128 query rows x 128 keys]  = Q K^T    A = Q, B = K
//   pass 2 (column sums)     S[128 keys x 128 query rows]  = K Q^T    A = K, B = Q
//
// The side whose sums are wanted sits on the M side of the product, so it lies along the
// TMEM lanes: a thread owns a query row (pass 1) or a key (pass 2) and reduces over its
// own registers.  An item holds up to two A tiles (256 rows or keys) and streams B tiles
// past them; every B tile staged serves both, which halves the copies per product.  Each A
// tile has two TMEM buffers of 128 columns (all 512 columns) and two consumer warpgroups,
// one per half of the columns: with 16 consumer warps a scheduler has four to switch
// between while loads from TMEM, exponentials and barriers are under way (8 warps took 1.2
// times as long).
//
// What bounds it: a product of 128 x 128 x 128 takes the tensor pipe 512 cycles, its 16384
// exponentials 512 cycles at 32 a cycle, and its operands are read from shared memory at 128
// bytes a cycle, all there is, so that the copies' writes (32 KB per B tile) and pass 2's
// reads of -lse slow the products down.  On the 16 x 512-token batch (every new token, 3.2e11
// flop a pass) the two passes take 260 and 287 us; pass 1 took 285 before its items were
// balanced, 250 without exponentials and 240 with its products alone.  Measured there and not
// kept, when the call took 596 us: four A tiles per B tile with one TMEM buffer each (half the
// copies): 653 us; B tiles of 256, whose products read 96 bytes a cycle, with one TMEM buffer
// per A tile: 638 us (425 us without exponentials: a tile's product and its exponentials take
// turns); TMEM loads a step ahead: 639 us; equal contiguous stretches of A tiles per CTA
// instead of every n-th item: 620 us.  A tiles in TMEM took pass 1 from 285 to 267 us, but leave
// three score buffers for two groups of consumers: a group that sat out an item could pass
// the wait for a buffer's next phase before the other group's phase was over.
//
// Pass 1 keeps the maximum of a row's first tile of the item (the first with a score above
// -inf) as its reference and adds
// 2^(s - m) from there on without looking for a larger one: there is no accumulator to
// keep in range, only a sum in fp32, whose relative precision does not depend on the
// reference.  Only a sum past 2^96 (later scores beyond the first tile's maximum by that
// much) takes the tile again with a new reference.  The keys of a row tile are cut into
// chunks that different CTAs take; a small launch merges the chunks' (m, sum) into
// -log2(sum 2^s) per row, which is all that pass 2 needs:
//   p = 2^(scale_log2 s - lse).
//
// Persistent CTAs, one per SM: producers run ahead into the next item's tiles while the
// consumers finish the current one.  Pass 1's items differ in length (the last chunk of keys,
// the causal edge), and every gridDim.x-th item to a CTA left the longest with a quarter more
// than the mean; taken from a shared counter, the call went from 590 to 552 us.  Pass 2's are
// many and alike: every gridDim.x-th.  Roles: warps 0-15 consumers, warp 16 A tiles, warp 17 B
// tiles, warp 18 MMA and TMEM, warp 19 the B rows' -lse (pass 2).
#include <atomic>

#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "prefill_weights.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kTile = 128;
constexpr int kChunk = 16;          // tokens per TMA box of K
constexpr int kBoxes = kTile / kChunk;
constexpr int kHalf = kTile * 128;  // a 64-column half of a Q tile: 16 KB
constexpr int kThreads = 640;
constexpr int kConsumers = 16;      // warps
constexpr int kWarpA = 16, kWarpB = 17, kWarpMma = 18, kWarpL = 19;
constexpr int kMaxReqs = 256;       // requests per launch (the item offsets in shared memory)
constexpr int kRing = 4;            // items announced (pass 1)
constexpr int kReaders = kConsumers + 2;   // warps that read them: consumers, B tiles, MMA
constexpr int kStagesL = 3;         // tiles of -lse staged (pass 2), 512 B each
constexpr float kSumLimit = 7.9e28f;   // 2^96

template <int D>
struct Geom {
    static constexpr int kHalves = D / 64;
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kChunkBytes = kChunk * D * 2;
    static constexpr int kGroupBytes = 8 * D * 2;    // 8 key rows, every half
    static constexpr int kStagesB = D == 128 ? 3 : 6;
    static constexpr int kOffA = 0;                   // two pairs of tiles
    static constexpr int kOffB = 4 * kTileBytes;
    static constexpr int kOffBar = kOffB + kStagesB * kTileBytes;
    // barriers
    static constexpr int A_FULL = 0, A_EMPTY = 2, B_FULL = 4, B_EMPTY = 4 + kStagesB,
                         S_FULL = 4 + 2 * kStagesB, S_FREE = S_FULL + 4, L_FULL = S_FREE + 4,
                         L_EMPTY = L_FULL + kStagesL, X_FULL = L_EMPTY + kStagesL,
                         DRAIN = X_FULL + 16;
    static constexpr int R_FULL = DRAIN + 1;
    static constexpr int R_EMPTY = R_FULL + kRing;
    static constexpr int kBars = R_EMPTY + kRing;
    static constexpr int kOffL = kOffBar + (kBars * 8 + 15) / 16 * 16;
    static constexpr int kOffCtl = kOffL + kStagesL * kTile * 4;   // TMEM address, abort flag
    static constexpr int kOffRing = kOffCtl + 16;
    static constexpr int kOffItems = kOffRing + kRing * 4;
    static constexpr int kBytes = kOffItems + (kMaxReqs + 1) * 4;
};
// One CTA fills an SM; there is no room for slack to align by, so the kernel relies on the
// dynamic shared memory starting on a 1 KB boundary (there is no static) and checks it.
static_assert(Geom<128>::kBytes <= 232448, "shared memory of one SM");

struct Ctl {
    uint64_t* bars;
    volatile int* abort_flag;
    int* status;
};

// Bounded wait of a converged warp; gives up when another role did, or out of time.
PKV_DEVINL bool wait_bar(const Ctl& c, int idx, uint32_t parity) {
    uint64_t* bar = &c.bars[idx];
    if (__any_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (;;) {
        if (__any_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *c.abort_flag != 0)) return false;
        if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitBudgetNs)) {
            if ((threadIdx.x & 31) == 0) {
                raise_status(c.status, PKV_ERR_TIMEOUT);
                *c.abort_flag = 1;
            }
            __syncwarp();
            return false;
        }
    }
}

PKV_DEVINL int ceil_div(int x, int y) { return (x + y - 1) / y; }

// One item: A tiles a0, a0 + 1 (na of them) against B tiles [b0, b0 + nb), which are those of
// one chunk of keys (pass 1) or of one part of the rows (pass 2).
struct Item {
    int r, kvh, chunk, a0, na, b0, nb;
    int base;   // last key that the window's first token sees
    Request q;
};

// The walk over a CTA's items: item k of request r (off[r] <= k < off[r + 1]).  Pass 2, whose
// items are many and alike, and launches with an item per CTA at most, take every gridDim.x-th.
// Otherwise the A role takes the next one from a counter that all CTAs share whenever it is
// ready for one, and announces it to the CTA's other roles in a ring; a place of the ring is
// written again when all of them have read it.  Indices only grow, so the search for the
// request goes on where it was.
template <int PASS>
struct Walk {
    const PrefillWeightsArgs& a;
    const int* off;
    const Ctl& ctl;
    int* ring;
    int ring_bar;
    int k, r = 0, n = 0;
    bool shared;
    PKV_DEVINL Walk(const PrefillWeightsArgs& args, const int* offsets, const Ctl& c, int* entries,
                    int first_bar)
        : a(args), off(offsets), ctl(c), ring(entries), ring_bar(first_bar), k(blockIdx.x),
          shared(PASS == 1 && args.next_item != nullptr) {}
    // The whole warp calls, for the next item or the end of them.
    PKV_DEVINL bool next(Item& it, bool announces = false) {
        if (!shared) return decode(it, gridDim.x);
        const int e = n % kRing;
        if (announces) {
            const int lane = threadIdx.x & 31;
            bool found;
            do {   // one item at a time: those without a tile to do are passed over
                if (lane == 0) k = atomicAdd(a.next_item, 1);
                k = __shfl_sync(0xffffffffu, k, 0);
                found = k < off[a.num_reqs] && decode(it, 0);
            } while (!found && k < off[a.num_reqs]);
            if (n >= kRing && !wait_bar(ctl, ring_bar + kRing + e, (n / kRing - 1) & 1))
                return false;
            if (lane == 0) {
                ring[e] = found ? k : -1;
                mbar_arrive(&ctl.bars[ring_bar + e]);
            }
            __syncwarp();
            ++n;
            return found;
        }
        if (!wait_bar(ctl, ring_bar + e, (n / kRing) & 1)) return false;
        k = *static_cast<volatile int*>(ring + e);
        __syncwarp();
        mbar_arrive_if((threadIdx.x & 31) == 0, &ctl.bars[ring_bar + kRing + e]);
        ++n;
        return k >= 0 && decode(it, 0);
    }
    // Item k; or, where it has nothing to do and `step` is not 0, the first of the items `step`
    // apart from there on that has.
    PKV_DEVINL bool decode(Item& it, int step) {
        for (;; k += step) {
            if (k >= off[a.num_reqs]) return false;
            while (off[r + 1] <= k) ++r;
            it.r = r;
            it.q = request_of(a, r, 1 << a.group_shift, false);
            it.base = it.q.c + it.q.n - it.q.m;
            const int keys = it.q.c + it.q.n;
            int rem = k - off[r];
            if (PASS == 1) {   // query-tile pair fastest: neighbours read the same keys
                const int tiles = ceil_div(it.q.rows, kTile), pairs = (tiles + 1) / 2;
                const int chunks = ceil_div(ceil_div(keys, kTile), a.chunk_tiles);
                it.a0 = 2 * (rem % pairs);
                rem /= pairs;
                it.chunk = rem % chunks;
                it.kvh = rem / chunks;
                it.na = min(2, tiles - it.a0);
                const int last_row = min((it.a0 + it.na) * kTile, it.q.rows) - 1;
                const int last_key = it.base + (last_row >> a.group_shift);
                it.b0 = it.chunk * a.chunk_tiles;
                it.nb = min(a.chunk_tiles, last_key / kTile + 1 - it.b0);
            } else {
                const int tiles = ceil_div(keys, kTile), pairs = (tiles + 1) / 2;
                it.a0 = 2 * (rem % pairs);
                rem /= pairs;
                it.chunk = rem % a.row_parts;
                it.kvh = rem / a.row_parts;
                it.na = min(2, tiles - it.a0);
                // rows from the first that sees the item's first key, of the item's part
                const int first = max(0, it.a0 * kTile - it.base) << a.group_shift;
                const int part = a.rows_per_part / kTile;
                it.b0 = max(first / kTile, it.chunk * part);
                it.nb = min(ceil_div(it.q.rows, kTile), (it.chunk + 1) * part) - it.b0;
            }
            if (it.nb > 0) {
                k += step;
                return true;
            }
            if (step == 0) return false;
        }
    }
};

// Sum of 2^(x * sl2 + off) over 32 values, into four pairs of accumulators.
PKV_DEVINL void add_exp(const float (&x)[32], float sl2, float off, float (&acc)[8]) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float a0, a1;
        ffma2(a0, a1, x[e], x[e + 1], sl2, sl2, off, off);
        const int u = e & 6;
        fadd2(acc[u], acc[u + 1], acc[u], acc[u + 1], fast_exp2(a0), fast_exp2(a1));
    }
}
PKV_DEVINL float sum8(const float (&v)[8]) {
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// The K boxes of one tile: lane b < nb copies 16-token chunk `chunk`, in block `phys`.  `bar` waits
// for more_bytes more than they are (see PrefillWeightsArgs::test_stall).
template <int D>
PKV_DEVINL void copy_k_boxes(const PrefillWeightsArgs& a, const void* tm_k, const Item& it,
                             int chunk, int phys, int nb, uint8_t* dst, uint64_t* bar, int lane,
                             int more_bytes = 0) {
    using GM = Geom<D>;
    const int csh = a.block_shift - 4;
    const int row = ((phys * a.num_kv_heads + it.kvh) << a.block_shift) +
                    (chunk & ((1 << csh) - 1)) * kChunk;
    mbar_arrive_expect_tx_if(lane == 0, bar, nb * GM::kChunkBytes + more_bytes);
    __syncwarp();
    if constexpr (D == 128)
        tma_load_4d_if(lane < nb, dst + lane * GM::kChunkBytes, tm_k, 0, 0, 0, row / 8, bar);
    else
        tma_load_2d_if(lane < nb, dst + lane * GM::kChunkBytes, tm_k, 0, row, bar);
}

// The block of the request's 16-token chunk `chunk`, or 0 past its end; a bad id is reported
// and replaced by 0, which keeps the byte counts (the request's weights are then not valid).
PKV_DEVINL int block_of(const PrefillWeightsArgs& a, const Item& it, int chunk, int chunks) {
    int phys = 0;
    if (chunk < chunks) {
        phys = __ldg(a.block_tables + static_cast<size_t>(it.r) * a.max_blocks_per_seq +
                     (chunk >> (a.block_shift - 4)));
        if (phys < 0 || phys >= a.num_blocks) {
            raise_status(a.status, PKV_ERR_OOB);
            phys = 0;
        }
    }
    __syncwarp();
    return phys;
}

// The Q tile `tile` of the window's rows.
template <int D>
PKV_DEVINL void copy_q_tile(const PrefillWeightsArgs& a, const void* tm_q, const Item& it, int tile,
                            uint8_t* dst, uint64_t* bar, int lane) {
    using GM = Geom<D>;
    const int token = it.q.qoff + it.q.n - it.q.m + ((tile * kTile) >> a.group_shift);
    if (lane == 0) {
        mbar_arrive_expect_tx(bar, GM::kTileBytes);
#pragma unroll
        for (int h = 0; h < GM::kHalves; ++h)
            tma_load_3d(dst + h * kHalf, tm_q, 64 * h, it.kvh << a.group_shift, token, bar);
    }
    __syncwarp();
}

template <int D, int PASS>
__global__ void __launch_bounds__(kThreads, 1)
prefill_weights_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k, const PrefillWeightsArgs a) {
    using GM = Geom<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + GM::kOffBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + GM::kOffCtl);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* off = reinterpret_cast<int*>(smem + GM::kOffItems);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    griddep_wait();
    griddep_launch_dependents();
    if (smem_u32(smem) & 1023u) {   // the swizzled tiles would not lie as their copies assume
        if (threadIdx.x == 0) raise_status(a.status, PKV_ERR_UNSUPPORTED);
        return;
    }
    if (warp == kWarpA) {
        if (lane == 0) {
            for (int i = 0; i < GM::kBars; ++i)   // arrivals: an A tile's consumers, all of them, 1
                mbar_init(&bars[i],
                          i >= GM::S_FREE && i < GM::S_FREE + 4 ? kConsumers / 2
                          : i >= GM::L_EMPTY && i < GM::L_EMPTY + kStagesL ? kConsumers
                          : i >= GM::R_EMPTY                               ? kReaders
                                                                           : 1);
            *abort_flag = 0;
            fence_mbar_init();
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
        }
    } else if (warp == kWarpMma) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    } else if (warp == 0) {
        // Items per request, and their running total, 32 requests at a time.
        int run = 0;
        for (int r0 = 0; r0 < a.num_reqs; r0 += 32) {
            int n = 0;
            if (r0 + lane < a.num_reqs) {
                const Request q = request_of(a, r0 + lane, 1 << a.group_shift,
                                             PASS == 1 && blockIdx.x == 0);
                if (q.rows > 0) {
                    const int key_tiles = ceil_div(q.c + q.n, kTile);
                    n = PASS == 1 ? (ceil_div(q.rows, kTile) + 1) / 2 *
                                        ceil_div(key_tiles, a.chunk_tiles)
                                  : (key_tiles + 1) / 2 * a.row_parts;
                    n *= a.num_kv_heads;
                }
            }
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            if (r0 + lane < a.num_reqs) off[r0 + lane] = run + incl - n;
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) off[a.num_reqs] = run;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Ctl ctl{bars, abort_flag, a.status};
    Walk<PASS> walk(a, off, ctl, reinterpret_cast<int*>(smem + GM::kOffRing), GM::R_FULL);
    Item it;

    if (warp == kWarpA) {
        // ------------------------------------------------------------ A tiles
        int i = 0, issued = 0;
        for (; walk.next(it, true); ++i) {
            const int s = i & 1;
            if (i >= 2 && !wait_bar(ctl, GM::A_EMPTY + s, ((i >> 1) - 1) & 1)) break;
            uint8_t* dst = smem + GM::kOffA + s * 2 * GM::kTileBytes;
            uint64_t* bar = &bars[GM::A_FULL + s];
            // test hook: the first item's tiles are waited for in vain
            const int stall = a.test_stall == PASS && i == 0 && blockIdx.x == 0 ? 16 : 0;
            if (PASS == 1) {
                const int token = it.q.qoff + it.q.n - it.q.m + ((it.a0 * kTile) >> a.group_shift);
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, it.na * GM::kTileBytes + stall);
                    for (int t = 0; t < it.na; ++t)
#pragma unroll
                        for (int h = 0; h < GM::kHalves; ++h)
                            tma_load_3d(dst + t * GM::kTileBytes + h * kHalf, &tm_q, 64 * h,
                                        it.kvh << a.group_shift,
                                        token + t * (kTile >> a.group_shift), bar);
                }
                __syncwarp();
            } else {
                // both tiles' chunks, one lane each
                const int chunks = ceil_div(it.q.c + it.q.n, kChunk);
                const int first = it.a0 * kBoxes;
                const int n = min(2 * kBoxes, chunks - first);
                const int phys = block_of(a, it, lane < n ? first + lane : chunks, chunks);
                copy_k_boxes<D>(a, &tm_k, it, first + lane, phys, n, dst, bar, lane, stall);
            }
            ++issued;
        }
        // every copy has landed before the CTA goes
        for (int s = 0; s < 2; ++s)
            if (issued > s)
                mbar_wait_warp(&bars[GM::A_FULL + s], ((issued - 1 - s) >> 1) & 1, a.status);
    } else if (warp == kWarpB) {
        // ------------------------------------------------------------ B tiles
        int g = 0;
        bool ok = true;
        while (ok && walk.next(it)) {
            const int chunks = ceil_div(it.q.c + it.q.n, kChunk);
            int ids = 0;   // pass 1: the blocks of the next four tiles' chunks, one per lane
            for (int j = 0; j < it.nb; ++j) {
                if (PASS == 1 && (j & 3) == 0)
                    ids = block_of(a, it, (it.b0 + j) * kBoxes + lane, chunks);
                const int s = g % GM::kStagesB;
                if (g >= GM::kStagesB &&
                    !wait_bar(ctl, GM::B_EMPTY + s, (g / GM::kStagesB - 1) & 1)) {
                    ok = false;
                    break;
                }
                uint8_t* dst = smem + GM::kOffB + s * GM::kTileBytes;
                uint64_t* bar = &bars[GM::B_FULL + s];
                if (PASS == 1) {
                    const int first = (it.b0 + j) * kBoxes;
                    const int id = __shfl_sync(0xffffffffu, ids, (j & 3) * kBoxes + (lane & 7));
                    copy_k_boxes<D>(a, &tm_k, it, first + (lane & 7), id,
                                    min(kBoxes, chunks - first), dst, bar, lane);
                } else {
                    copy_q_tile<D>(a, &tm_q, it, it.b0 + j, dst, bar, lane);
                }
                ++g;
            }
        }
        for (int s = 0; s < GM::kStagesB; ++s)
            if (g > s)
                mbar_wait_warp(&bars[GM::B_FULL + s], ((g - 1 - s) / GM::kStagesB) & 1, a.status);
    } else if (warp == kWarpMma) {
        // ------------------------------------------------------------ MMA issuer
        // Q tiles: 8-row atoms 1 KB apart, column halves 16 KB apart; K tiles: 8-row
        // groups every 8 D * 2 bytes, column halves 1 KB apart.
        constexpr uint32_t idesc = idesc_bf16_f32(kTile, kTile, false, false);
        constexpr uint32_t hi_q = smem_desc_sw128_hi(1024);
        constexpr uint32_t hi_k = smem_desc_sw128_hi(GM::kGroupBytes);
        constexpr uint32_t step_q = kHalf >> 4, step_k = 1024 >> 4;
        constexpr uint32_t hi_a = PASS == 1 ? hi_q : hi_k, hi_b = PASS == 1 ? hi_k : hi_q;
        constexpr uint32_t step_a = PASS == 1 ? step_q : step_k;
        constexpr uint32_t step_b = PASS == 1 ? step_k : step_q;
        const uint32_t lo_a = smem_desc_sw128_lo(smem_u32(smem + GM::kOffA), 16);
        const uint32_t lo_b = smem_desc_sw128_lo(smem_u32(smem + GM::kOffB), 16);
        const bool leader = elect_one();
        int i = 0, g = 0, used[2] = {0, 0};   // items, B tiles, tiles given to warpgroup w
        bool ok = true;
        while (ok && walk.next(it)) {
            const int sa = i & 1;
            ok = wait_bar(ctl, GM::A_FULL + sa, (i >> 1) & 1);
            for (int j = 0; ok && j < it.nb; ++j, ++g) {
                const int sb = g % GM::kStagesB;
                ok = wait_bar(ctl, GM::B_FULL + sb, (g / GM::kStagesB) & 1);
                if (!ok) break;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (w >= it.na) continue;
                    const int buf = w + 2 * (used[w] & 1);
                    if (used[w] >= 2 &&
                        !wait_bar(ctl, GM::S_FREE + buf, ((used[w] >> 1) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t la = lo_a + (((sa * 2 + w) * GM::kTileBytes) >> 4);
                    const uint32_t lb = lo_b + ((sb * GM::kTileBytes) >> 4);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t kc = ((ks & 3) * 32) >> 4;
                        umma_bf16_if(leader, tmem + buf * 128,
                                     desc_join(la + (ks >> 2) * step_a + kc, hi_a),
                                     desc_join(lb + (ks >> 2) * step_b + kc, hi_b), idesc, ks > 0);
                    }
                    umma_commit_if(leader, &bars[GM::S_FULL + buf]);
                    ++used[w];
                }
                umma_commit_if(leader, &bars[GM::B_EMPTY + sb]);
            }
            // not after a wait that ran out: the place's copies may still be on their way
            if (ok) umma_commit_if(leader, &bars[GM::A_EMPTY + sa]);
            ++i;
        }
        // every product has completed before the TMEM goes
        umma_commit_if(leader, &bars[GM::DRAIN]);
        mbar_wait_warp(&bars[GM::DRAIN], 0, a.status);
    } else if (warp == kWarpL) {
        // ------------------------------------------------------------ -lse of the B rows
        if (PASS == 2) {
            int g = 0;
            bool ok = true;
            while (ok && walk.next(it)) {
                const float* lse = a.neg_lse +
                                   (static_cast<size_t>(it.r) * a.num_kv_heads + it.kvh) *
                                       a.rows_pad;
                for (int j = 0; j < it.nb; ++j) {
                    const int s = g % kStagesL;
                    if (g >= kStagesL && !wait_bar(ctl, GM::L_EMPTY + s, (g / kStagesL - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bars[GM::L_FULL + s], kTile * 4);
                        bulk_g2s(smem + GM::kOffL + s * kTile * 4, lse + (it.b0 + j) * kTile,
                                 kTile * 4, &bars[GM::L_FULL + s]);
                    }
                    __syncwarp();
                    ++g;
                }
            }
            for (int s = 0; s < kStagesL; ++s)
                if (g > s)
                    mbar_wait_warp(&bars[GM::L_FULL + s], ((g - 1 - s) / kStagesL) & 1, a.status);
        }
    } else if (warp < kConsumers) {
        // ------------------------------------------------------------ consumers
        const int wg = (warp >> 2) & 1;           // A tile of the item
        const int half = warp >> 3;               // columns 64 half .. 64 half + 63
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;      // TMEM lane: query row or key of the tile
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const float sl2 = a.scale_log2;
        int used = 0, gl = 0;   // tiles of this A tile's consumers; tiles of -lse
        uint32_t met_phase[2] = {0, 0};
        bool ok = true;
        while (ok && walk.next(it)) {
            const int tile = it.a0 + wg;
            const bool mine = wg < it.na;
            const size_t head = static_cast<size_t>(it.r) * a.num_kv_heads + it.kvh;
            if (PASS == 1) {
                if (!mine) continue;
                const int rho = tile * kTile + row;
                // Rows that pad the request's last tile have a say in no vote (their sum is NaN from
                // the start): what they look at is other requests' queries and whatever the last
                // key tile's shared memory held, and a vote moves the references of its warp's rows.
                const bool there = rho < it.q.rows;
                const int lim = it.base + (rho >> a.group_shift);        // last key seen
                const int least = it.base + ((tile * kTile) >> a.group_shift);
                float m = 0.f, l = there ? 0.f : NAN;
                for (int j = 0; j < it.nb; ++j, ++used) {
                    const int buf = wg + 2 * (used & 1);
                    if (!wait_bar(ctl, GM::S_FULL + buf, (used >> 1) & 1)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t tS = tmem + lanes + buf * 128 + 64 * half;
                    const int key0 = (it.b0 + j) * kTile + 64 * half;
                    const int seen = lim - key0 + 1;   // the columns that the row sees
                    const bool whole = key0 + 63 <= least;
                    auto load = [&](int q, float (&x)[32]) {
                        tmem_ld32(tS + q * 32, x);
                        tmem_wait_ld32(x);
                        if (!whole) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                x[e] = q * 32 + e < seen ? x[e] : -INFINITY;
                        }
                    };
                    auto tile_max = [&]() {
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                        for (int q = 0; q < 2; ++q) {
                            float x[32];
                            load(q, x);
#pragma unroll
                            for (int e = 0; e < 32; e += 2)
                                mx[(e >> 1) & 3] = fmax3(mx[(e >> 1) & 3], x[e], x[e + 1]);
                        }
                        return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
                    };
                    auto tile_sum = [&](float ref) {
                        float t[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) t[u] = 0.f;
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float x[32];
                            load(q, x);
                            add_exp(x, sl2, -ref, t);
                        }
                        return sum8(t);
                    };
                    if (j == 0 || __any_sync(0xffffffffu, l == 0.f)) {
                        // no reference yet; a tile of which the row sees nothing, or -inf
                        // scores alone, leaves any
                        const float mt = tile_max();
                        if (l == 0.f) m = mt == -INFINITY ? 0.f : mt;
                    }
                    const float t = tile_sum(m);
                    if (__any_sync(0xffffffffu, l + t > kSumLimit)) {
                        // far above the reference: take the tile again from its own maximum
                        const float mt = fmaxf(m, tile_max());
                        if (mt > m) {
                            l *= fast_exp2(m - mt);
                            m = mt;
                        }
                        l += tile_sum(m);
                    } else {
                        l += t;
                    }
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_if(lane == 0, &bars[GM::S_FREE + buf]);
                }
                if (ok && there)
                    a.stats[((head * a.splits + it.chunk) * 2 + half) * a.rows_pad + rho] =
                        make_float2(m, l);
            } else {
                const int key = tile * kTile + row;
                const int last = tile * kTile + kTile - 1;
                // rows that see the key: rho >= from
                const int from = max(0, key - it.base) << a.group_shift;
                const int from_last = max(0, last - it.base) << a.group_shift;
                const bool there = mine && half == 0 && key < it.q.c + it.q.n;
                // added to the weights, or kept for the launch that adds the parts up
                const bool whole_sum = a.row_parts == 1;
                float* w = whole_sum
                               ? a.weights + (static_cast<size_t>(it.q.wrow) * a.num_kv_heads +
                                              it.kvh) * static_cast<size_t>(a.weights_stride) + key
                               : a.parts + (head * a.row_parts + it.chunk) * a.max_context + key;
                const float decay = whole_sum ? a.decay : 0.f;
                const float before = there && decay != 0.f ? *w : 0.f;
                float acc[8], total = 0.f;
#pragma unroll
                for (int u = 0; u < 8; ++u) acc[u] = 0.f;
                for (int j = 0; j < it.nb; ++j, ++gl) {
                    const int sl = gl % kStagesL;
                    if (!wait_bar(ctl, GM::L_FULL + sl, (gl / kStagesL) & 1)) { ok = false; break; }
                    if (mine) {
                        const int buf = wg + 2 * (used & 1);
                        const uint32_t phase = (used >> 1) & 1;
                        if (!wait_bar(ctl, GM::S_FULL + buf, phase)) { ok = false; break; }
                        ++used;
                        tc_fence_after();
                        const uint32_t tS = tmem + lanes + buf * 128;
                        const int row0 = (it.b0 + j) * kTile + 64 * half;
                        const bool whole = row0 >= from_last && row0 + 64 <= it.q.rows;
                        // the rows' -lse, the same address in every lane
                        const float4* n4 = reinterpret_cast<const float4*>(
                            smem + GM::kOffL + sl * kTile * 4 + 256 * half);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float x[32];
                            tmem_ld32(tS + 64 * half + q * 32, x);
                            tmem_wait_ld32(x);
                            if (whole) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const float4 n = n4[q * 8 + e];
                                    float a0, a1, a2, a3;
                                    ffma2(a0, a1, x[4 * e], x[4 * e + 1], sl2, sl2, n.x, n.y);
                                    ffma2(a2, a3, x[4 * e + 2], x[4 * e + 3], sl2, sl2, n.z, n.w);
                                    const int u = 4 * (e & 1);
                                    fadd2(acc[u], acc[u + 1], acc[u], acc[u + 1], fast_exp2(a0),
                                          fast_exp2(a1));
                                    fadd2(acc[u + 2], acc[u + 3], acc[u + 2], acc[u + 3],
                                          fast_exp2(a2), fast_exp2(a3));
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const float4 n = n4[q * 8 + e];
                                    const float nn[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
                                    for (int f = 0; f < 4; ++f) {
                                        const int rho = row0 + q * 32 + 4 * e + f;
                                        const bool on = rho >= from && rho < it.q.rows;
                                        acc[f] +=
                                            on ? fast_exp2(fmaf(x[4 * e + f], sl2, nn[f])) : 0.f;
                                    }
                                }
                            }
                        }
                        if (j + 1 == it.nb) {
                            // The two halves' sums of a key meet: half 1 leaves its own in a
                            // column of the tile's buffer that it has read, half 0 takes it
                            // from there before the buffer is given back.
                            uint64_t* met = &bars[GM::X_FULL + buf * 4 + quarter];
                            total = sum8(acc);
                            if (half == 1) {
                                tmem_st1(tS + 127, total);
                                tmem_wait_st();
                                tc_fence_before();
                                __syncwarp();
                                mbar_arrive_if(lane == 0, met);
                            } else {
                                if (!wait_bar(ctl, GM::X_FULL + buf * 4 + quarter,
                                              met_phase[(buf >> 1)])) {
                                    ok = false;
                                    break;
                                }
                                met_phase[(buf >> 1)] ^= 1;
                                tc_fence_after();
                                total += tmem_ld1(tS + 127);
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        mbar_arrive_if(lane == 0, &bars[GM::S_FREE + buf]);
                    }
                    __syncwarp();
                    mbar_arrive_if(lane == 0, &bars[GM::L_EMPTY + sl]);
                }
                if (ok && there) *w = decay != 0.f ? fmaf(decay, before, total) : total;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Pass 1's counter of items taken.
__global__ void reset_items_kernel(const PrefillWeightsArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    if (threadIdx.x == 0) *a.next_item = 0;
}

// -log2 of a row's sum over its chunks, and -inf for the rows that pad the last tile.
// Grid (row blocks, kv head, request).
__global__ void __launch_bounds__(128)
merge_stats_kernel(const PrefillWeightsArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int rho = blockIdx.x * 128 + threadIdx.x;
    const Request q = request_of(a, blockIdx.z, 1 << a.group_shift, false);
    if (q.rows == 0 || blockIdx.x * 128 >= q.rows) return;
    const size_t head = static_cast<size_t>(blockIdx.z) * a.num_kv_heads + blockIdx.y;
    float neg = -INFINITY;
    if (rho < q.rows) {
        // the chunks of the row's tile pair: those up to the last key that the pair sees
        const int pair_last = min((rho / 256 + 1) * 256, q.rows) - 1;
        const int last_key = q.c + q.n - q.m + (pair_last >> a.group_shift);
        const int chunks = 2 * (last_key / kTile / a.chunk_tiles + 1);   // two halves each
        const float2* st = a.stats + head * a.splits * 2 * a.rows_pad + rho;
        float M = -INFINITY;
        for (int z = 0; z < chunks; ++z) {
            const float2 f = st[static_cast<size_t>(z) * a.rows_pad];
            if (f.y != 0.f) M = fmaxf(M, f.x);   // 0: a chunk the row sees nothing of
        }
        float l = 0.f;
        for (int z = 0; z < chunks; ++z) {
            const float2 f = st[static_cast<size_t>(z) * a.rows_pad];
            if (f.y != 0.f) l += f.y * fast_exp2(f.x - M);
        }
        neg = -(M + log2f(l));
    }
    a.neg_lse[head * a.rows_pad + rho] = neg;
}

// Streaming multiprocessors of the current device.
int sm_count() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    int v = cached[dev].load(std::memory_order_relaxed);
    if (v <= 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
            return 1;
        cached[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

template <int D>
cudaError_t launch_d(const PrefillWeightsArgs& a, int group, cudaStream_t stream) {
    using GM = Geom<D>;
    CUtensorMap mq, mk;
    const int64_t rows = (a.num_blocks * a.num_kv_heads) << a.block_shift;
    const bool ok = D == 128 ? make_pool_block_map(&mk, a.k_pool, rows)
                             : make_pool_map(&mk, a.k_pool, rows, D);
    if (!ok || !make_q_group_map(&mq, a.q, a.total_new, a.num_q_heads, D, group, kTile / group))
        return cudaErrorInvalidValue;
    auto pass1 = prefill_weights_kernel<D, 1>;
    auto pass2 = prefill_weights_kernel<D, 2>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(pass1), GM::kBytes);
    if (e == cudaSuccess) e = set_smem_once(reinterpret_cast<const void*>(pass2), GM::kBytes);
    if (e != cudaSuccess) return e;
    const int64_t row_tiles = (static_cast<int64_t>(a.max_rows) * group + kTile - 1) / kTile;
    const int64_t key_pairs = (static_cast<int64_t>(a.max_context) + 2 * kTile - 1) / (2 * kTile);
    // Up to kMaxReqs requests per round of launches (their item offsets sit in shared memory).
    const int total = a.num_reqs;
    for (int r0 = 0; r0 < total; r0 += kMaxReqs) {
        PrefillWeightsArgs g = a;
        g.num_reqs = total - r0 < kMaxReqs ? total - r0 : kMaxReqs;
        g.block_tables += static_cast<size_t>(r0) * a.max_blocks_per_seq;
        g.cached_lens += r0;
        g.new_lens += r0;
        g.q_offsets += r0;
        if (a.row_ids) {
            g.row_ids += r0;
        } else {
            g.weights += static_cast<size_t>(r0) * a.num_kv_heads * a.weights_stride;
            g.num_rows -= r0;
        }
        const int64_t heads = static_cast<int64_t>(g.num_reqs) * a.num_kv_heads;
        const int64_t items1 = heads * ((row_tiles + 1) / 2) * a.splits;
        const int64_t items2 = heads * key_pairs * a.row_parts;
        if (items1 > INT32_MAX - 65536 || items2 > INT32_MAX) return cudaErrorNotSupported;
        const int sms = sm_count();
        if (items1 > sms) {   // the counter passes their number by one a CTA at most
            e = launch_pdl(reset_items_kernel, dim3(1), dim3(32), 0, stream, g);
            if (e != cudaSuccess) return e;
        } else {
            g.next_item = nullptr;
        }
        e = launch_pdl(pass1, dim3(static_cast<unsigned>(items1 < sms ? items1 : sms)),
                       dim3(kThreads), GM::kBytes, stream, mq, mk, g);
        if (e != cudaSuccess) return e;
        e = launch_pdl(merge_stats_kernel,
                       dim3(static_cast<unsigned>(row_tiles), a.num_kv_heads, g.num_reqs),
                       dim3(128), 0, stream, g);
        if (e != cudaSuccess) return e;
        e = launch_pdl(pass2, dim3(static_cast<unsigned>(items2 < sms ? items2 : sms)),
                       dim3(kThreads), GM::kBytes, stream, mq, mk, g);
        if (e != cudaSuccess) return e;
        if (a.row_parts > 1) {
            e = launch_add_parts(g, 2 * kTile, kTile, stream);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_prefill_weights_tc(const PrefillWeightsArgs& a, int head_dim, int group,
                                      cudaStream_t stream) {
    return head_dim == 128 ? launch_d<128>(a, group, stream) : launch_d<64>(a, group, stream);
}

}  // namespace pkv

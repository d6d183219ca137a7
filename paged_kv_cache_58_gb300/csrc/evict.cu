// Eviction by accumulated attention weight: each (sequence, kv head) keeps `budget` of
// its L cached entries and closes up.
//
// Which: the protected entries (original position below `sinks`, or among the last
// `recent` positions seen) rank above the others; within a class the larger weight ranks
// higher, and the lower index among equal weights.  The budget's worth of that order is
// kept.  Where: kept entries below the budget stay; the k-th kept entry past it moves
// into the k-th freed place below it (both ascending).  Attention does not depend on the
// order of keys, so nothing else has to move: the K/V traffic is the moved rows alone,
// and sources (past the budget) and destinations (below it) never overlap.
//
// Selecting the budget-th value is a radix select over the weights' bit patterns, mapped
// so that unsigned order is their order: four passes of 8 bits narrow the prefix shared
// with the threshold, each a histogram of the entries that still match it.
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace pkv {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Unsigned order of the result = order of the weights; -0 equals +0, NaN ranks last.
PKV_DEVINL uint32_t order_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of `flag` over the CTA's threads in index order; `total` gets the sum.
PKV_DEVINL int block_rank(bool flag, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t ball = __ballot_sync(0xffffffffu, flag);
    if (lane == 0) warp_sums[warp] = __popc(ball);
    __syncthreads();
    const int v = lane < kWarps ? warp_sums[lane] : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    const int before = __shfl_sync(0xffffffffu, incl - v, warp);
    __syncthreads();   // warp_sums may be reused
    return before + __popc(ball & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(kThreads)
evict_kernel(const EvictArgs a) {
    __shared__ int hist[256];
    __shared__ int warp_sums[kWarps];
    __shared__ int pick[3];   // digit, entries above it, entries in it
    griddep_wait();
    griddep_launch_dependents();
    const int kvh = blockIdx.x, seq = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    const int row = a.row_ids ? __ldg(a.row_ids + seq) : seq;
    const int L = __ldg(a.context_lens + seq);
    const int b = __ldg(a.budgets + seq);
    const bool reports = kvh == 0 && tid == 0;
    const int64_t cap = static_cast<int64_t>(a.max_blocks_per_seq) << a.block_shift;
    if (row < 0 || L <= 0) {   // a padding row, or nothing cached
        if (reports) {
            a.new_lens[seq] = max(L, 0);
            if (L < 0) raise_status(a.status, PKV_ERR_INVALID);
        }
        return;
    }
    if (row >= a.num_rows || L > a.max_context || L > cap) {   // left as it is
        if (reports) {
            a.new_lens[seq] = L;
            raise_status(a.status, PKV_ERR_OOB);
        }
        return;
    }
    const bool shrinks = b >= 0 && L > b;
    if (reports) a.new_lens[seq] = shrinks ? b : L;

    const size_t at = (static_cast<size_t>(row) * a.num_kv_heads + kvh) *
                      static_cast<size_t>(a.weights_stride);
    const float* w = a.weights + at;
    float* wo = a.weights_out + at;
    const int32_t* pos = a.positions + at;
    int32_t* po = a.positions_out + at;
    const int tracked = a.tracked_lens ? min(max(__ldg(a.tracked_lens + seq), 0), L) : 0;
    const int seen = a.seen_lens ? __ldg(a.seen_lens + seq) : L;
    auto position = [&](int j) { return j < tracked ? pos[j] : seen - L + j; };
    const int recent_from = seen - a.recent;
    auto safe = [&](int j) {
        const int p = position(j);
        return p < a.sinks || p >= recent_from;
    };

    if (!shrinks) {
        for (int j = tid; j < L; j += kThreads) {
            wo[j] = w[j];
            po[j] = position(j);
        }
        return;
    }

    // The protected entries: all are kept and the rest of the budget goes to the others,
    // unless they alone exceed it; then it is theirs.
    int mine = 0;
    for (int j = tid; j < L; j += kThreads) mine += safe(j);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) warp_sums[warp] = mine;
    __syncthreads();
    int nsafe = 0;
    for (int i = 0; i < kWarps; ++i) nsafe += warp_sums[i];
    __syncthreads();
    const bool among_safe = nsafe >= b;
    int need = among_safe ? b : b - nsafe;   // entries to pick among the contested class

    uint32_t prefix = 0, mask = 0;   // digits of the threshold found so far
    if (need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int j = tid; j < L; j += kThreads) {
                const uint32_t key = order_key(w[j]);
                if (safe(j) == among_safe && (key & mask) == prefix)
                    atomicAdd(&hist[(key >> shift) & 255], 1);
            }
            __syncthreads();
            if (warp == 0) {   // the digit at which the count from above reaches `need`
                int cnt[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    cnt[i] = hist[255 - (lane * 8 + i)];
                    sum += cnt[i];
                }
                int incl = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                int above = incl - sum;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (above < need && above + cnt[i] >= need) {
                        pick[0] = 255 - (lane * 8 + i);
                        pick[1] = above;
                    }
                    above += cnt[i];
                }
            }
            __syncthreads();
            prefix |= static_cast<uint32_t>(pick[0]) << shift;
            mask |= 255u << shift;
            need -= pick[1];
            __syncthreads();
        }
    }
    // Kept of the contested class: keys above `prefix`, and the first `need` equal to it.
    const bool none = need == 0;

    // Emission in index order: freed places below the budget, kept entries past it.
    int32_t* list = a.moves + (static_cast<size_t>(seq) * a.num_kv_heads + kvh) *
                                  static_cast<size_t>(a.max_context);
    int32_t* holes = list;                          // at most min(b, L - b) of each:
    int32_t* movers = list + (a.max_context >> 1);  // both halves suffice
    int ties = 0, nholes = 0, nmovers = 0;
    for (int j0 = 0; j0 < L; j0 += kThreads) {
        const int j = j0 + tid;
        bool keep = false, tie = false;
        if (j < L) {
            const bool s = safe(j);
            const uint32_t key = order_key(w[j]);
            if (s != among_safe) {
                keep = s;
            } else if (!none) {
                keep = key > prefix;
                tie = key == prefix;
            }
        }
        int n;
        const int rank = ties + block_rank(tie, warp_sums, n);
        ties += n;
        keep |= tie && rank < need;
        const bool hole = j < b && !keep, mover = j >= b && j < L && keep;
        const int h = nholes + block_rank(hole, warp_sums, n);
        nholes += n;
        const int m = nmovers + block_rank(mover, warp_sums, n);
        nmovers += n;
        if (hole) holes[h] = j;
        if (mover) movers[m] = j;
        if (j < b && keep) {
            wo[j] = w[j];
            po[j] = position(j);
        }
    }
    __syncthreads();
    for (int k = tid; k < nmovers; k += kThreads) {
        const int from = movers[k], to = holes[k];
        wo[to] = w[from];
        po[to] = position(from);
    }
    __syncthreads();
    for (int j = b + tid; j < L; j += kThreads) wo[j] = 0.f;   // free places start at zero

    // The rows themselves, 16 bytes per lane.
    const int32_t* bt = a.block_tables + static_cast<size_t>(seq) * a.max_blocks_per_seq;
    const int cpr = a.row_bytes >> 4;   // chunks per row: 8, 16 or 32
    for (int64_t t = tid; t < static_cast<int64_t>(nmovers) * cpr; t += kThreads) {
        const int k = static_cast<int>(t / cpr), ch = static_cast<int>(t % cpr);
        const int from = movers[k], to = holes[k];
        const int pf = __ldg(bt + (from >> a.block_shift));
        const int pt = __ldg(bt + (to >> a.block_shift));
        if (pf < 0 || pf >= a.num_blocks || pt < 0 || pt >= a.num_blocks) {
            raise_status(a.status, PKV_ERR_OOB);
            continue;
        }
        const int low = (1 << a.block_shift) - 1;
        const size_t src = ((((static_cast<size_t>(pf) * a.num_kv_heads + kvh) << a.block_shift) +
                             (from & low)) * cpr) + ch;
        const size_t dst = ((((static_cast<size_t>(pt) * a.num_kv_heads + kvh) << a.block_shift) +
                             (to & low)) * cpr) + ch;
        static_cast<uint4*>(a.k_pool)[dst] = static_cast<const uint4*>(a.k_pool)[src];
        static_cast<uint4*>(a.v_pool)[dst] = static_cast<const uint4*>(a.v_pool)[src];
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
    return launch_pdl(evict_kernel, dim3(a.num_kv_heads, a.num_seqs), dim3(kThreads), 0, stream,
                      a);
}

}  // namespace pkv

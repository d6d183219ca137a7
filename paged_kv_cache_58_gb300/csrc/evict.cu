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
// A row (sequence, kv head) is one cluster of C CTAs, each with a slice of its entries:
//   1. weights -> 32-bit keys whose unsigned order is theirs, into shared memory, with a
//      bit per entry for its class; the protected are counted.  Either all of them are
//      kept and the others compete for what is left of the budget, or they alone do.
//   2. radix select of the threshold among the competing class, 11 + 11 + 10 bits: a
//      histogram of the entries that match the digits found so far, equal digits of a
//      warp added at once (weights crowd into few exponents: one atomic per entry spent
//      most of a pass waiting on the same counter); it ends early when a bin is kept whole.
//   3. places: freed ones below the budget and kept ones past it are numbered by scans
//      over the threads' contiguous segments and written to two lists, a mover with its
//      weight and position, so that its old entry can be cleared at once.
//   4. after one cluster barrier all threads copy the listed rows, 16 bytes of K and of V
//      per lane, four rows in flight per lane.
// With C = 1 there are no cluster barriers.  Entries past the shared-memory capacity of a
// slice are looked at in global memory again in each step.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace pkv {

namespace {

namespace cg = cooperative_groups;

constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kCapEntries = 32768;   // entries of a slice held in shared memory, at most

// Unsigned order of the result = order of the weights; -0 equals +0, NaN ranks last.
PKV_DEVINL uint32_t order_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One spare word in 32, so that threads walking contiguous segments of 2^n entries do not
// meet in one bank.
PKV_DEVINL int padded(int i) { return i + (i >> 5); }

struct Shared {                       // after it: keys, class bits, cluster histograms
    int hist[kBins];
    unsigned long long warp_sums[32];
    unsigned long long cluster_sums[2][kMaxCluster];
    int pick[3];                      // bin, entries above it, entries in it
};

// Exclusive prefix of v over the CTA's threads; `total` gets the sum.
template <int NT>
PKV_DEVINL unsigned long long block_scan(unsigned long long v, unsigned long long* warp_sums,
                                         unsigned long long& total) {
    constexpr int W = NT / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    unsigned long long s = lane < W ? warp_sums[lane] : 0, t = s;
#pragma unroll
    for (int o = 1; o < W; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += y;
    }
    total = __shfl_sync(0xffffffffu, t, W - 1);
    const unsigned long long before = __shfl_sync(0xffffffffu, t - s, warp);
    __syncthreads();   // warp_sums may be written again
    return before + incl - v;
}

template <int NT>
__global__ void __launch_bounds__(NT)
evict_kernel(const EvictArgs a, const int C, const int cap) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& sm = *reinterpret_cast<Shared*>(raw);
    uint32_t* keys = reinterpret_cast<uint32_t*>(raw + sizeof(Shared));   // [padded(cap)]
    uint32_t* bits = keys + padded(cap) + 1;                               // [cap / 32 + 1]
    int* ghist = reinterpret_cast<int*>(bits + cap / 32 + 1);              // [3][kBins], C > 1
    griddep_wait();
    griddep_launch_dependents();
    const int kvh = blockIdx.x / C, rank = blockIdx.x % C, seq = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31;

    const int row = a.row_ids ? __ldg(a.row_ids + seq) : seq;
    const int L = __ldg(a.context_lens + seq);
    const int b = __ldg(a.budgets + seq);
    const int tracked_in = a.tracked_lens ? __ldg(a.tracked_lens + seq) : 0;
    const int seen = a.seen_lens ? __ldg(a.seen_lens + seq) : L;
    const bool reports = blockIdx.x == 0 && tid == 0;
    const int64_t table = static_cast<int64_t>(a.max_blocks_per_seq) << a.block_shift;
    if (row < 0 || L <= 0) {   // a padding row, or nothing cached (the same in every CTA)
        if (reports) {
            a.new_lens[seq] = max(L, 0);
            if (L < 0) raise_status(a.status, PKV_ERR_INVALID);
        }
        return;
    }
    if (row >= a.num_rows || L > a.max_context || L > table) {   // left as it is
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
    const int tracked = min(max(tracked_in, 0), L);
    auto position = [&](int j) { return j < tracked ? pos[j] : seen - L + j; };

    // this CTA's slice [i0, i0 + n)
    const int per = ((L + C - 1) / C + 31) & ~31;
    const int i0 = min(rank * per, L);
    const int n = min(per, L - i0);
    // What stays where it is, entry by entry (freed places are filled in step 4).
    auto copy_through = [&](int end) {
        const int m = min(n, end - i0);
        const bool ws = w != wo, ps = pos != po;
        for (int i = tid; i < m; i += NT) {
            const int j = i0 + i;
            if (ws) wo[j] = w[j];
            if (ps || j >= tracked) po[j] = position(j);
        }
    };
    if (!shrinks) {
        copy_through(L);
        return;
    }

    // ---------------------------------------------------------------- 1. keys and classes
    const int recent_from = seen - a.recent;
    auto is_safe = [&](int j) {
        const int p = position(j);
        return p < a.sinks || p >= recent_from;
    };
    for (int i = tid; i < kBins; i += NT) sm.hist[i] = 0;
    if (C > 1)
        for (int i = tid; i < 3 * kBins; i += NT) ghist[i] = 0;
    int mine = 0;
    for (int i = tid; i - lane < n; i += NT) {   // whole warps
        bool s = false;
        if (i < n) {
            s = is_safe(i0 + i);
            if (i < cap) keys[padded(i)] = order_key(w[i0 + i]);
        }
        const uint32_t ball = __ballot_sync(0xffffffffu, s);
        if (lane == 0 && i < cap) bits[i >> 5] = ball;
        mine += s;
    }
    unsigned long long total;
    block_scan<NT>(static_cast<unsigned long long>(mine), sm.warp_sums, total);
    cg::cluster_group cluster = cg::this_cluster();
    // Totals of the CTAs before this one, and of all, in `slot` of the exchange array.
    auto gather = [&](unsigned long long v, int slot, unsigned long long& before,
                      unsigned long long& all) {
        before = 0;
        all = v;
        if (C == 1) return;
        if (tid < C) *cluster.map_shared_rank(&sm.cluster_sums[slot][rank], tid) = v;
        cluster.sync();
        all = 0;
        for (int r = 0; r < C; ++r) {
            if (r == rank) before = all;
            all += sm.cluster_sums[slot][r];
        }
    };
    unsigned long long before, all;
    gather(total, 0, before, all);
    const int nsafe = static_cast<int>(all);
    const bool among_safe = nsafe >= b;
    int need = among_safe ? b : b - nsafe;   // entries to pick among the competing class

    // Key and class of entry i of the slice.
    auto entry = [&](int i, uint32_t& key) {
        if (i < cap) {
            key = keys[padded(i)];
            return ((bits[i >> 5] >> (i & 31)) & 1u) != 0;
        }
        key = order_key(w[i0 + i]);
        return is_safe(i0 + i);
    };

    // ---------------------------------------------------------------- 2. threshold
    uint32_t prefix = 0, mask = 0;   // digits of the threshold found so far
    int in_bin = need > 0 ? 0 : -1;
    for (int pass = 0; need > 0 && pass < 3 && in_bin != need; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digit_mask = pass == 2 ? 1023u : 2047u;
        if (pass > 0) {
            for (int i = tid; i < kBins; i += NT) sm.hist[i] = 0;
            __syncthreads();
        }
        for (int i = tid; i - lane < n; i += NT) {
            uint32_t key = 0;
            const bool on = i < n && entry(i, key) == among_safe && (key & mask) == prefix;
            const uint32_t active = __ballot_sync(0xffffffffu, on);
            if (on) {
                const uint32_t digit = (key >> shift) & digit_mask;
                const uint32_t same = __match_any_sync(active, digit);
                if (lane == __ffs(same) - 1) atomicAdd(&sm.hist[digit], __popc(same));
            }
        }
        __syncthreads();
        int* g = sm.hist;
        if (C > 1) {   // the cluster's histogram, in its first CTA
            g = ghist + pass * kBins;
            int* first = cluster.map_shared_rank(g, 0);
            for (int i = tid; i < kBins; i += NT)
                if (sm.hist[i]) atomicAdd(first + i, sm.hist[i]);
            cluster.sync();
        }
        if (rank == 0) {   // the bin at which the count from above reaches `need`
            constexpr int PER = kBins / NT;
            int cnt[PER], sum = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                cnt[i] = g[kBins - 1 - (tid * PER + i)];
                sum += cnt[i];
            }
            unsigned long long t;
            int above = static_cast<int>(
                block_scan<NT>(static_cast<unsigned long long>(sum), sm.warp_sums, t));
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (above < need && above + cnt[i] >= need)
                    for (int r = 0; r < C; ++r) {
                        int* p = C > 1 ? cluster.map_shared_rank(sm.pick, r) : sm.pick;
                        p[0] = kBins - 1 - (tid * PER + i);
                        p[1] = above;
                        p[2] = cnt[i];
                    }
                above += cnt[i];
            }
        }
        if (C > 1)
            cluster.sync();
        else
            __syncthreads();
        prefix |= static_cast<uint32_t>(sm.pick[0]) << shift;
        mask |= digit_mask << shift;
        need -= sm.pick[1];
        in_bin = sm.pick[2];
    }
    // Kept of the competing class: (key & mask) above `prefix`, and the first `need` equal
    // to it (all of them where the bin was kept whole).

    // ---------------------------------------------------------------- 3. places
    const int E = (n + NT - 1) / NT;
    const int s0 = min(tid * E, n), s1 = min(s0 + E, n);   // this thread's segment
    // -1: not kept, 0: in the threshold's bin, 1: kept
    auto verdict = [&](int i) {
        uint32_t key;
        const bool s = entry(i, key);
        if (s != among_safe) return s ? 1 : -1;
        if (need <= 0) return -1;   // nothing of the competing class is kept
        const uint32_t k = key & mask;
        return k > prefix ? 1 : k == prefix ? 0 : -1;
    };
    int ties = 0;
    for (int i = s0; i < s1; ++i) ties += verdict(i) == 0;
    int tie_rank = static_cast<int>(
        block_scan<NT>(static_cast<unsigned long long>(ties), sm.warp_sums, total));
    gather(total, 1, before, all);
    tie_rank += static_cast<int>(before);

    unsigned long long moved = 0;   // freed places, and kept entries past the budget << 32
    int t = tie_rank;
    for (int i = s0; i < s1; ++i) {
        const int v = verdict(i);
        const bool keep = v > 0 || (v == 0 && t < need);
        t += v == 0;
        if (i0 + i < b)
            moved += keep ? 0ull : 1ull;
        else
            moved += keep ? 1ull << 32 : 0ull;
    }
    unsigned long long first = block_scan<NT>(moved, sm.warp_sums, total);
    gather(total, 0, before, all);
    first += before;
    const int nmoves = static_cast<int>(all >> 32);
    // lists of at most min(b, L - b) <= max_context / 2 moves
    const int most = a.max_context >> 1;
    int32_t* holes = a.moves + (static_cast<size_t>(seq) * a.num_kv_heads + kvh) *
                                   (4 * static_cast<size_t>(most));
    int32_t* movers = holes + most;
    float* mover_w = reinterpret_cast<float*>(movers + most);
    int32_t* mover_pos = movers + 2 * static_cast<size_t>(most);
    int h = static_cast<int>(first & 0xffffffffu), m = static_cast<int>(first >> 32);
    t = tie_rank;
    if (moved)
        for (int i = s0; i < s1; ++i) {
            const int v = verdict(i);
            const bool keep = v > 0 || (v == 0 && t < need);
            t += v == 0;
            const int j = i0 + i;
            if (j < b) {
                if (!keep) holes[h++] = j;
            } else if (keep) {
                movers[m] = j;
                mover_w[m] = w[j];
                mover_pos[m] = position(j);
                ++m;
            }
        }
    __syncthreads();
    copy_through(b);
    for (int i = max(0, b - i0) + tid; i < n; i += NT) wo[i0 + i] = 0.f;   // free places
    if (C > 1)
        cluster.sync();
    else
        __syncthreads();

    // ---------------------------------------------------------------- 4. moves
    const int worker = rank * NT + tid, workers = C * NT;
    for (int k = worker; k < nmoves; k += workers) {
        const int to = holes[k];
        wo[to] = mover_w[k];
        po[to] = mover_pos[k];
    }
    const int32_t* bt = a.block_tables + static_cast<size_t>(seq) * a.max_blocks_per_seq;
    const int csh = a.row_shift;            // log2 of 16-byte chunks per row
    const int ch = worker & ((1 << csh) - 1);
    const int step = workers >> csh;        // rows per sweep
    const int low = (1 << a.block_shift) - 1;
    uint4* kp = static_cast<uint4*>(a.k_pool);
    uint4* vp = static_cast<uint4*>(a.v_pool);
    constexpr int U = 4;
    for (int k0 = worker >> csh; k0 < nmoves; k0 += U * step) {
        int from[U], to[U], pf[U], pt[U];
        bool ok[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * step;
            ok[u] = k < nmoves;
            from[u] = ok[u] ? movers[k] : 0;
            to[u] = ok[u] ? holes[k] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            pf[u] = ok[u] ? __ldg(bt + (from[u] >> a.block_shift)) : 0;
            pt[u] = ok[u] ? __ldg(bt + (to[u] >> a.block_shift)) : 0;
        }
        uint4 xk[U], xv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!ok[u]) continue;
            if (pf[u] < 0 || pf[u] >= a.num_blocks || pt[u] < 0 || pt[u] >= a.num_blocks) {
                raise_status(a.status, PKV_ERR_OOB);
                ok[u] = false;
                continue;
            }
            const size_t src = (((((static_cast<size_t>(pf[u]) * a.num_kv_heads + kvh)
                                   << a.block_shift) + (from[u] & low))) << csh) + ch;
            xk[u] = kp[src];
            xv[u] = vp[src];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!ok[u]) continue;
            const size_t dst = (((((static_cast<size_t>(pt[u]) * a.num_kv_heads + kvh)
                                   << a.block_shift) + (to[u] & low))) << csh) + ch;
            kp[dst] = xk[u];
            vp[dst] = xv[u];
        }
    }
}

template <int NT>
cudaError_t launch_nt(const EvictArgs& a, int C, cudaStream_t stream) {
    const int slice = ((a.max_context + C - 1) / C + 31) & ~31;
    const int cap = slice < kCapEntries ? slice : kCapEntries;
    const int words = cap + (cap >> 5) + 1 + cap / 32 + 1 + (C > 1 ? 3 * kBins : 0);
    const int smem = static_cast<int>(sizeof(Shared)) + 4 * words;
    auto kern = evict_kernel<NT>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.num_kv_heads * C, a.num_seqs);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a, C, cap);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
    // CTAs per row: enough that a slice fits in shared memory beside others, and that about
    // two CTAs per SM exist where there are few rows.
    const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
    int C = 1;
    while (C < kMaxCluster &&
           (a.max_context > 16384 * C || (rows * C < 304 && a.max_context > 1024 * C)))
        C *= 2;
    // Short rows: CTAs of 256 threads, so that more of them share an SM.
    return C == 1 ? launch_nt<256>(a, C, stream) : launch_nt<512>(a, C, stream);
}

}  // namespace pkv

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
//   1. one scan over the weights: a bit per entry for its class, the protected counted, and
//      a histogram of the others' first digit.  Weights become 32-bit keys whose unsigned
//      order is theirs; a radix select narrows the threshold by 11 + 11 + 10 bits.  Either
//      all protected entries are kept and the others compete for what is left of the
//      budget, or (rarely: then the histogram is made again) the protected alone do.
//   2. a second scan decides every entry outside the threshold's first bin, and lists the
//      few inside it; the other digits and the rest of the decisions come from that list.
//      (Where it overflows, as with many equal weights, from scans of the slice.)  The
//      select ends early when a bin is kept whole.
//   3. freed places below the budget and kept entries past it are counted and numbered 32 at
//      a time, a thread per word of the bits, and written to two lists, a mover with its
//      weight and position, so that its old entry is cleared in the same scan.  Short lists
//      of a CTA with its row alone stay in shared memory.
//   4. after one cluster barrier all threads copy the listed rows, 16 bytes of K and of V
//      per lane, three or four rows in flight per lane and the places of the next ones looked
//      up meanwhile.  (A cluster looks the sources' up when it lists them: 239 us against 254
//      for 16 x 128k; one CTA as it moves them, a chain of loads less: 64.4 us against 66.3 for
//      64 x 4k.)
// Measured (one call of many, from a graph): 64 x 8 rows of 1040 entries, 16 over budget, 10.3
// us, a chain of dependent steps; 512 to 4096 down to 1024, 62.7 us, about 44 of them the
// moves at 5.7 TB/s; 16 x 8 rows of 16k to 128k down to 8192, 240 us, 133 of them the moves at
// 7.3 TB/s, the rest three scans of 10.9 M entries at about 90 issue slots per 32.  Four CTAs
// per SM: with three and the registers that leaves, 320 rows take 52.7 us for 54.9 (3000 entries
// down to 1024), but 512 rows a second wave, 14.4 us for 10.3 and 89.8 for 76.0.
// With C = 1 there are no cluster barriers.  The scans read the weights where they are, in
// L2 after the first: keys kept in shared memory left two CTAs on an SM and a row's
// latencies uncovered.  Weights crowd into few exponents (and many may be zero), but counting
// the lanes that share a digit at once, with votes, was slower than one shared-memory atomic
// per entry (16 x 128k tokens: 256 against 245 us; with all weights zero 230 against 204).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace pkv {

namespace {

namespace cg = cooperative_groups;

constexpr int NT = 256;              // threads
constexpr int kWarps = NT / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kList = 1024;          // entries of the threshold's bin listed per CTA

// Unsigned order of the result = order of the weights; -0 equals +0, NaN ranks last.
PKV_DEVINL uint32_t order_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One spare word in 8: a thread walks 8 neighbouring bins, and the threads of a warp should
// not meet in one bank.
PKV_DEVINL int spread(int bin) { return bin + (bin >> 3); }
constexpr int kHist = kBins + kBins / 8;

struct Shared {   // after it: three bits per entry
    int hist[kHist];
    int cluster_hist[kHist];          // the cluster's, in its first CTA
    unsigned long long list[kList];   // key << 32 | ~index: a larger one ranks higher
    unsigned long long warp_sums[kWarps];
    unsigned long long cluster_sums[3][kMaxCluster];
    int pick[3];                      // bin, entries above it, entries in it
    int listed;
};

// Exclusive prefix of v over the CTA's threads; `total` gets the sum.
template <typename V>
PKV_DEVINL V block_scan(V v, unsigned long long* warp_sums, V& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    V incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[warp] = static_cast<unsigned long long>(incl);
    __syncthreads();
    V before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const V s = static_cast<V>(warp_sums[i]);
        if (i < warp) before += s;
        total += s;
    }
    __syncthreads();   // warp_sums may be written again
    return before + incl - v;
}

// F: entries in flight per thread in a scan.  ONE: a CTA has its row alone (C = 1).
template <int F, bool ONE>
__global__ void __launch_bounds__(NT, 4)
evict_kernel(const EvictArgs a, const int cluster_ctas, const int words) {
    const int C = ONE ? 1 : cluster_ctas;
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& sm = *reinterpret_cast<Shared*>(raw);
    uint32_t* safe_bits = reinterpret_cast<uint32_t*>(raw + sizeof(Shared));   // protected
    uint32_t* keep_bits = safe_bits + words;
    uint32_t* tie_bits = keep_bits + words;      // equal to the threshold
    const int kvh = blockIdx.x / C, rank = blockIdx.x % C, seq = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31;
    for (int i = tid; i < kHist; i += NT) sm.hist[i] = sm.cluster_hist[i] = 0;
    if (tid == 0) sm.listed = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();

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

    // this CTA's slice [i0, i0 + n): whole words but for the row's end
    const int per = ((L + C - 1) / C + 31) & ~31;
    const int i0 = min(rank * per, L);
    const int n = min(per, L - i0);
    const bool move_w = w != wo, move_p = pos != po;
    if (!shrinks) {
        for (int i = tid; i < n; i += NT) {
            const int j = i0 + i;
            if (move_w) wo[j] = w[j];
            if (move_p || j >= tracked) po[j] = position(j);
        }
        return;
    }
    cg::cluster_group cluster = cg::this_cluster();
    // No CTA touches another's shared memory before all of the cluster are known to run: they
    // arrive here (the returns above are taken by all of a cluster or by none) and wait ahead
    // of the first remote access, behind the first scan.
    if (!ONE) cluster.barrier_arrive();

    // ---------------------------------------------------------------- 1. classes, first digit
    const int recent_from = seen - a.recent;
    int mine = 0;
    for (int ib = tid; ib - lane < n; ib += F * NT) {   // whole warps
        float x[F];
        int p[F];
#pragma unroll
        for (int u = 0; u < F; ++u) {
            const int i = ib + u * NT;
            if (i < n) {
                x[u] = w[i0 + i];
                p[u] = position(i0 + i);
            }
        }
#pragma unroll
        for (int u = 0; u < F; ++u) {
            const int i = ib + u * NT;
            if (i - lane >= n) break;
            const bool in = i < n;
            if (in && i0 + i < b) {   // most of these stay: step 4 overwrites the freed places
                if (move_w) wo[i0 + i] = x[u];
                if (move_p || i0 + i >= tracked) po[i0 + i] = p[u];
            }
            const bool s = in && (p[u] < a.sinks || p[u] >= recent_from);
            const uint32_t ball = __ballot_sync(0xffffffffu, s);
            if (lane == 0) {
                safe_bits[i >> 5] = ball;
                mine += __popc(ball);
            }
            if (in && !s) atomicAdd(&sm.hist[spread(order_key(x[u]) >> 21)], 1);
        }
    }
    int cta_safe;
    block_scan(mine, sm.warp_sums, cta_safe);
    if (!ONE) cluster.barrier_wait();
    // Totals of the CTAs before this one, and of all, through `slot` of the exchange array.
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
    unsigned long long before, all, total;
    gather(static_cast<unsigned long long>(cta_safe), 0, before, all);
    const int nsafe = static_cast<int>(all);
    const bool among_safe = nsafe >= b;
    int need = among_safe ? b : b - nsafe;   // entries to pick among the competing class
    // Entry i's class bit: 1 where it competes.
    const uint32_t flip = among_safe ? 0u : 0xffffffffu;
    auto competes = [&](int i) {
        return (((safe_bits[i >> 5] ^ flip) >> (i & 31)) & 1u) != 0;
    };
    // f(i, in, weight) for the slice's entries, whole warps at a time, one by one: for the
    // rare cases (a batch of entries unrolled in every one of them would be mostly code, which
    // a CTA that runs each line once has to fetch).
    auto scan = [&](auto f) {
#pragma unroll 1
        for (int i = tid; i - lane < n; i += NT) f(i, i < n, i < n ? w[i0 + i] : 0.f);
    };
    if (among_safe) {   // the counted class does not compete after all
        for (int i = tid; i < kHist; i += NT) sm.hist[i] = 0;
        __syncthreads();
        scan([&](int i, bool in, float x) {
            if (in && competes(i)) atomicAdd(&sm.hist[spread(order_key(x) >> 21)], 1);
        });
        __syncthreads();
    }

    // ---------------------------------------------------------------- 2. threshold
    uint32_t prefix = 0, mask = 0;   // digits of the threshold found so far
    int in_bin = -1;
    // The histogram's bin at which the count from above reaches `need`; leaves hist zeroed.
    auto narrow = [&](int shift, uint32_t digit_mask) {
        int* g = sm.hist;
        if (C > 1) {   // the cluster's histogram, in its first CTA
            g = sm.cluster_hist;
            int* first = cluster.map_shared_rank(g, 0);
            for (int i = tid; i < kHist; i += NT)
                if (sm.hist[i]) {
                    atomicAdd(first + i, sm.hist[i]);
                    sm.hist[i] = 0;
                }
            cluster.sync();
        }
        if (rank == 0) {
            constexpr int PER = kBins / NT;
            int cnt[PER], sum = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                int& bin = g[spread(kBins - 1 - (tid * PER + i))];
                cnt[i] = bin;
                bin = 0;
                sum += cnt[i];
            }
            int t;
            int above = block_scan(sum, sm.warp_sums, t);
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
    };
    if (need > 0) narrow(21, 2047u);
    // Second scan: kept for sure above the bin (the whole bin, if it is kept whole); what is
    // in it is listed and its next digit counted.
    const bool open = need > 0 && in_bin != need;
    for (int ib = tid; ib - lane < n; ib += F * NT) {
        float x[F];
#pragma unroll
        for (int u = 0; u < F; ++u) {
            const int i = ib + u * NT;
            x[u] = i < n ? w[i0 + i] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < F; ++u) {
            const int i = ib + u * NT;
            if (i - lane >= n) break;
            const bool rival = i < n && competes(i);
            const uint32_t key = order_key(x[u]), k = key & mask;
            const bool keep = i < n && (rival ? need > 0 && (k > prefix || (!open && k == prefix))
                                              : !among_safe);
            const bool inside = rival && open && k == prefix;
            const uint32_t kept = __ballot_sync(0xffffffffu, keep);
            if (lane == 0) {
                keep_bits[i >> 5] = kept;
                tie_bits[i >> 5] = 0;
            }
            if (inside) {
                atomicAdd(&sm.hist[spread((key >> 10) & 2047u)], 1);
                const int slot = atomicAdd(&sm.listed, 1);
                if (slot < kList)
                    sm.list[slot] = static_cast<unsigned long long>(key) << 32 |
                                    ~static_cast<uint32_t>(i);
            }
        }
    }
    __syncthreads();
    const int listed = open ? sm.listed : 0;
    // A short list of one CTA is ranked outright, each entry against all.
    const bool ranked = open && C == 1 && listed <= NT;
    if (ranked && tid < listed) {
        const unsigned long long entry = sm.list[tid];
        const int i = static_cast<int>(~static_cast<uint32_t>(entry));
        int better = 0;
#pragma unroll 8
        for (int q = 0; q < listed; ++q) better += sm.list[q] > entry;
        if (better < need) atomicOr(&keep_bits[i >> 5], 1u << (i & 31));
    }
    if (ranked) __syncthreads();
    if (open && !ranked) {
        const bool by_list = listed <= kList;
        // f(i, on, key) for the entries in the first bin, whole warps at a time
        const uint32_t bin_mask = mask, bin = prefix;
        auto candidates = [&](auto f) {
            if (by_list) {
                for (int q = tid; q - lane < listed; q += NT) {
                    const bool on = q < listed;
                    const unsigned long long entry = on ? sm.list[q] : 0xffffffffull;
                    f(static_cast<int>(~static_cast<uint32_t>(entry)), on,
                      static_cast<uint32_t>(entry >> 32));
                }
            } else {
                scan([&](int i, bool in, float x) {
                    const uint32_t key = order_key(x);
                    f(i, in && competes(i) && (key & bin_mask) == bin, key);
                });
            }
        };
        narrow(10, 2047u);
        if (in_bin != need) {   // the last ten bits
            candidates([&](int, bool on, uint32_t key) {
                if (on && (key & mask) == prefix) atomicAdd(&sm.hist[spread(key & 1023u)], 1);
            });
            __syncthreads();
            narrow(0, 1023u);
        }
        const bool whole = in_bin == need;
        candidates([&](int i, bool on, uint32_t key) {
            const uint32_t k = key & mask;
            if (on && (k > prefix || (whole && k == prefix)))
                atomicOr(&keep_bits[i >> 5], 1u << (i & 31));
            else if (on && k == prefix)
                atomicOr(&tie_bits[i >> 5], 1u << (i & 31));
        });
        __syncthreads();
    }

    // ---------------------------------------------------------------- 3. places
    const int nw = (n + 31) >> 5;
    const int E = (nw + NT - 1) / NT;
    const int w0 = min(tid * E, nw), w1 = min(w0 + E, nw);   // this thread's words
    if (open && !ranked && in_bin != need) {   // equal weights: the first `need` of them, by index
        int ties = 0, cta_ties;
        for (int x = w0; x < w1; ++x) ties += __popc(tie_bits[x]);
        int no = block_scan(ties, sm.warp_sums, cta_ties);
        gather(static_cast<unsigned long long>(cta_ties), 1, before, all);
        no += static_cast<int>(before);
        for (int x = w0; x < w1; ++x) {
            uint32_t tied = tie_bits[x];
            const int cnt = __popc(tied);
            for (int drop = no + cnt - need; drop > 0 && tied; --drop)   // the last ones go
                tied &= ~(0x80000000u >> __clz(tied));
            keep_bits[x] |= tied;
            no += cnt;
        }
    }
    // Entries of word x that are freed places, and that move.
    auto hole_mask = [&](int x) {
        const int left = b - i0 - 32 * x;   // entries below the budget
        return left <= 0 ? 0u : ~keep_bits[x] & (left >= 32 ? 0xffffffffu : (1u << left) - 1u);
    };
    auto mover_mask = [&](int x) {
        const int left = b - i0 - 32 * x;
        return left >= 32 ? 0u : keep_bits[x] & (left <= 0 ? 0xffffffffu : ~((1u << left) - 1u));
    };
    unsigned long long moved = 0;   // freed places, and movers << 32
    for (int x = w0; x < w1; ++x)
        moved += static_cast<unsigned long long>(__popc(hole_mask(x))) |
                 static_cast<unsigned long long>(__popc(mover_mask(x))) << 32;
    unsigned long long first = block_scan(moved, sm.warp_sums, total);
    gather(total, 2, before, all);
    first += before;
    // Equal counts, unless the weights change while they are read (a row used by two sequences
    // at once): then no more moves than both lists hold.
    const int most = a.max_context >> 1;
    const int nmoves = min(min(static_cast<int>(all >> 32), static_cast<int>(all & 0xffffffffu)),
                           most);
    // lists of at most min(b, L - b) <= max_context / 2 = most moves
    int32_t* holes = a.moves + (static_cast<size_t>(seq) * a.num_kv_heads + kvh) *
                                   (5 * static_cast<size_t>(most));
    int32_t* movers = holes + most;
    uint32_t* mover_slot = reinterpret_cast<uint32_t*>(movers + most);   // clusters
    float* mover_w = reinterpret_cast<float*>(mover_slot + most);
    int32_t* mover_pos = holes + 4 * static_cast<size_t>(most);
    int room = most;
    if (C == 1 && max(static_cast<int>(all >> 32), static_cast<int>(all & 0xffffffffu)) <= kList) {
        // short lists of one CTA: where the threshold's bin and the histograms were
        static_assert(kHist >= kList, "a list in a histogram's place");
        holes = reinterpret_cast<int32_t*>(sm.list);
        movers = holes + kList;
        mover_w = reinterpret_cast<float*>(sm.hist);
        mover_pos = sm.cluster_hist;
        room = kList;
    }
    // Pool slots fit 32 bits: 2^32 rows of the least 128 bytes are more than this GPU holds.
    const int32_t* bt = a.block_tables + static_cast<size_t>(seq) * a.max_blocks_per_seq;
    const uint32_t low = (1u << a.block_shift) - 1u;
    constexpr uint32_t kNoSlot = 0xffffffffu;
    auto slot_of = [&](int j) {
        const int phys = __ldg(bt + (j >> a.block_shift));
        if (phys < 0 || phys >= a.num_blocks) {
            raise_status(a.status, PKV_ERR_OOB);
            return kNoSlot;
        }
        return (static_cast<uint32_t>(phys) << a.block_shift) + (static_cast<uint32_t>(j) & low);
    };
    // The listed entries' indices, word by word, then what goes with them, entry by entry with
    // every lane at work (one entry in ten is listed where 128k tokens shrink to 8k).
    int h = static_cast<int>(first & 0xffffffffu), m = static_cast<int>(first >> 32);
    for (int x = w0; x < w1; ++x) {
        for (uint32_t bits = hole_mask(x); bits; bits &= bits - 1, ++h)
            if (h < room) holes[h] = i0 + 32 * x + __ffs(bits) - 1;
        for (uint32_t bits = mover_mask(x); bits; bits &= bits - 1, ++m)
            if (m < room) movers[m] = i0 + 32 * x + __ffs(bits) - 1;
    }
    __syncthreads();
    const int m0 = static_cast<int>(before >> 32);
    const int m1 = min(m0 + static_cast<int>(total >> 32), room);
    for (int kb = m0 + tid; kb < m1; kb += F * NT) {
        int j[F], p[F];
        uint32_t slot[F];
        float x[F];
#pragma unroll
        for (int u = 0; u < F; ++u) {
            const int k = kb + u * NT;
            j[u] = k < m1 ? movers[k] : -1;
        }
#pragma unroll
        for (int u = 0; u < F; ++u) {
            if (j[u] < 0) continue;
            if (!ONE) slot[u] = slot_of(j[u]);
            x[u] = w[j[u]];
            p[u] = position(j[u]);
        }
#pragma unroll
        for (int u = 0; u < F; ++u) {
            const int k = kb + u * NT;
            if (j[u] < 0) continue;
            if (!ONE) mover_slot[k] = slot[u];
            mover_w[k] = x[u];
            mover_pos[k] = p[u];
        }
    }
    __syncthreads();
    // The places past the budget start at zero.
    const int under = min(max(b - i0, 0), n);   // entries of the slice below the budget
    for (int i = under + tid; i < n; i += NT) wo[i0 + i] = 0.f;
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
    const int csh = a.row_shift;            // log2 of 16-byte chunks per row
    const int ch = worker & ((1 << csh) - 1);
    const int step = workers >> csh;        // rows per sweep
    uint4* kp = static_cast<uint4*>(a.k_pool);
    uint4* vp = static_cast<uint4*>(a.v_pool);
    auto chunk = [&](uint32_t slot) {       // 16-byte chunk of the slot's row of this head
        const size_t blk = slot >> a.block_shift;
        return ((((blk * a.num_kv_heads + kvh) << a.block_shift) + (slot & low)) << csh) + ch;
    };
    constexpr int U = ONE ? 3 : 4;   // rows in flight: four cost registers that spill with ONE
    uint32_t from[U], to[U];
    auto look_up = [&](int k0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * step;
            from[u] = k >= nmoves ? kNoSlot : ONE ? static_cast<uint32_t>(movers[k]) : mover_slot[k];
            to[u] = k < nmoves ? static_cast<uint32_t>(holes[k]) : kNoSlot;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (to[u] != kNoSlot) {
                if (ONE) from[u] = slot_of(static_cast<int>(from[u]));
                to[u] = slot_of(static_cast<int>(to[u]));
            }
    };
    int k0 = worker >> csh;
    look_up(k0);
    while (k0 < nmoves) {
        uint4 xk[U], xv[U];
        size_t dst[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            on[u] = from[u] != kNoSlot && to[u] != kNoSlot;
            if (!on[u]) continue;
            const size_t src = chunk(from[u]);
            xk[u] = kp[src];
            xv[u] = vp[src];
            dst[u] = chunk(to[u]);
        }
        k0 += U * step;
        look_up(k0);   // the next rows' places, while these rows are on their way
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!on[u]) continue;
            kp[dst[u]] = xk[u];
            vp[dst[u]] = xv[u];
        }
    }
}

template <int F, bool ONE>
cudaError_t launch_f(const EvictArgs& a, int C, cudaStream_t stream) {
    auto kern = evict_kernel<F, ONE>;
    const int words = ((a.max_context + C - 1) / C + 31) / 32;
    const int smem = static_cast<int>(sizeof(Shared)) + 3 * 4 * words;
    // allowed for the longest slice at once: host threads that raised the limit to what each
    // needs could lower it for one another
    constexpr int kMost = sizeof(Shared) + 3 * 4 * (kEvictMaxContext / kMaxCluster / 32);
    static_assert(kMost <= 232448, "the bits of the longest slice fit");
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), kMost);
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
    cfg.numAttrs = C > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, C, words);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
    // CTAs per row: enough that a slice has at most 16384 entries (128 rows of 16k to 128k: 241 us,
    // 247 with slices of 32768, 241 with 8192; 512 rows of 16k to 20k: 364, 375 and 361), and that
    // about two CTAs per SM exist where there are few rows.  More where rows fill the SMs only adds cluster barriers (512 rows with two each: a
    // block of 64 took 39 us against 15.6, 512 to 4096 entries 76 against 72).
    // Entries in flight per thread: four in a CTA that has its row alone (eight: 12.2 and 67.2 us
    // against 11.4 and 66.3), eight where clusters scan long rows (four 243.5 us, sixteen 258,
    // against 241).
    const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
    int C = 1;
    while (C < kMaxCluster &&
           (a.max_context > 16384 * C || (rows * C < 304 && a.max_context > 1024 * C)))
        C *= 2;
    return C == 1 ? launch_f<4, true>(a, C, stream) : launch_f<8, false>(a, C, stream);
}

}  // namespace pkv

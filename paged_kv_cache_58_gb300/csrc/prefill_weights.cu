// Accumulated attention weights of a prompt chunk: how much attention each cached key
// receives from a request's last `window` new tokens, summed over them and over the
// query heads of its kv head,
//   weights[j] = decay * weights[j] + sum_{rows r that see j} 2^(s_rj - M_r) / sum_r,
// s = scale * log2(e) * q.k.  A row's statistics (M_r, sum_r) need every key before any
// of its weights is known, so there are two passes:
//   pass 1  per 64-row query tile, online (max, sum) of each row over its keys,
//   pass 2  per 64-key tile, the column sums over all the query tiles that see it.
// A key tile of a request and kv head belongs to one CTA, which walks its query tiles in
// order; where there are too few key tiles for the SMs, to one CTA per part of its rows, and
// a last launch adds the parts in order.  No atomics, and the same bits every time.
//
// This is the CUDA-core form, for fp32 pools (the tensor cores would round the operands to
// tf32; bf16 pools have a tensor-core form in prefill_weights_tc.cu, which computes Q K^T
// twice): a product is dear here, 2 D operations per score against 8 bytes to write a score
// and read it back, so pass 1 keeps the scores in the workspace and pass 2 streams them.  One
// request of 500 tokens after 1 to 2k, 8 heads on 1, D 128: 106 us against 173 with the
// products computed twice; 4 x 300 tokens, 16 heads on 4, D 64: 166 against 288; three requests
// of some 70 tokens 13.4 against 19.7.  The launches take as many (request, kv head) pairs at
// a time as the workspace's share for scores holds; a pair with more than that (a gigabyte)
// has its products computed twice.
//
// Products: a 64 x 64 tile of scores per step, 256 threads of 4 x 4 scores each, both operand
// tiles in shared memory, the next tile on its way into registers meanwhile; the even and the
// odd elements of a row pair are summed by packed multiply-adds (one request: 184 us then with
// single ones, 173 with packed; the small one 24.6 and 19.7).  Bound by the reads from shared
// memory: 8 of 512 bytes per warp and 32 packed multiply-adds.  Pass 1 splits a row tile's keys
// over CTAs where there are few; pass 2 merges the parts' statistics as it reads them.
#include <algorithm>

#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "prefill_weights.cuh"

namespace pkv {

namespace {

constexpr int kTile = 64;       // rows, and keys, of a score tile
constexpr int kThreads = 256;   // 16 x 16 threads, 4 x 4 scores each

template <int D>
struct Smem {
    static constexpr int kStride = D + 4;   // 16-byte rows, shifted 4 banks per row
    float q[kTile][kStride];
    float k[kTile][kStride];
    float red[2][kTile][17];
};

// A tile on its way from global memory: each thread holds its pieces in registers while the
// tile before it is worked on, then puts them into shared memory.
template <int D>
struct Fetch {
    static constexpr int kPieces = kTile * (D / 4) / kThreads;   // 16-byte pieces per thread
    float4 v[kPieces];
    PKV_DEVINL void put(float (*dst)[Smem<D>::kStride]) const {
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            const int t = threadIdx.x + u * kThreads;
            *reinterpret_cast<float4*>(&dst[t / (D / 4)][t % (D / 4) * 4]) = v[u];
        }
    }
    // Rows (i, g) of the window, token-major: row rho is token n - m + rho / G of the
    // request's new tokens, head kvh * G + rho % G.
    PKV_DEVINL void rows(const PrefillWeightsArgs& a, const Request& rq, int group, int kvh,
                         int row0) {
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            const int t = threadIdx.x + u * kThreads;
            const int rho = row0 + t / (D / 4);
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (rho < rq.rows) {
                const int64_t tok = static_cast<int64_t>(rq.qoff) + rq.n - rq.m + rho / group;
                const float* src = static_cast<const float*>(a.q) +
                                   (tok * a.num_q_heads + kvh * group + rho % group) * D +
                                   t % (D / 4) * 4;
                v[u] = __ldg(reinterpret_cast<const float4*>(src));
            }
        }
    }
    // Keys key0 .. of the request, those from `keys` on as zeros.
    PKV_DEVINL void keys(const PrefillWeightsArgs& a, int req, int kvh, int key0, int keys) {
        const int32_t* bt = a.block_tables + static_cast<size_t>(req) * a.max_blocks_per_seq;
        int phys[kPieces];
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            const int key = key0 + (threadIdx.x + u * kThreads) / (D / 4);
            phys[u] = key < keys ? __ldg(bt + (key >> a.block_shift)) : -1;
            if (key < keys && (phys[u] < 0 || phys[u] >= a.num_blocks)) {
                raise_status(a.status, PKV_ERR_OOB);
                phys[u] = -1;
            }
        }
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            const int t = threadIdx.x + u * kThreads;
            const int key = key0 + t / (D / 4);
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (phys[u] >= 0) {
                const float* src = static_cast<const float*>(a.k_pool) +
                                   (((static_cast<int64_t>(phys[u]) * a.num_kv_heads + kvh)
                                     << a.block_shift) +
                                    (key & ((1 << a.block_shift) - 1))) * D + t % (D / 4) * 4;
                v[u] = __ldg(reinterpret_cast<const float4*>(src));
            }
        }
    }
};

// The thread's place in the 16 x 16 grid: a warp covers 4 rows by 8 keys, so that each of its
// 16-byte shared-memory reads is one pass (2 by 16 needs two for the keys; the times were alike).
PKV_DEVINL int thread_x() { return (threadIdx.x & 7) + ((threadIdx.x >> 5) & 1) * 8; }
PKV_DEVINL int thread_y() { return ((threadIdx.x >> 3) & 3) + (threadIdx.x >> 6) * 4; }

// s[i][j] = q row (ty + 16 i) . k row (tx + 16 j), scaled; 4 x 4 per thread.
template <int D>
PKV_DEVINL void scores(const Smem<D>& sm, float scale, float (&s)[4][4]) {
    const int tx = thread_x(), ty = thread_y();
    float even[4][4], odd[4][4];   // the sums over even and odd d, one packed product for both
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) even[i][j] = odd[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = *reinterpret_cast<const float4*>(&sm.q[ty + 16 * i][d]);
            y[i] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * i][d]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ffma2(even[i][j], odd[i][j], x[i].x, x[i].y, y[j].x, y[j].y, even[i][j], odd[i][j]);
                ffma2(even[i][j], odd[i][j], x[i].z, x[i].w, y[j].z, y[j].w, even[i][j], odd[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = (even[i][j] + odd[i][j]) * scale;
}

// The (request, kv head) of a CTA: launches take a.heads_per_launch of them, from head0 on.
struct Head {
    int req, kvh;
};
PKV_DEVINL Head head_of(const PrefillWeightsArgs& a, int head0) {
    const int head = head0 + static_cast<int>(blockIdx.y);
    return {head / a.num_kv_heads, head % a.num_kv_heads};
}

// Pass 1.  Grid (query tile x splits, (request, kv head)); split z of the keys.  KEEP: the
// scores are kept for pass 2.
template <int D, bool KEEP>
__global__ void __launch_bounds__(kThreads, 2)
row_stats_kernel(const PrefillWeightsArgs a, const int group, const int head0) {
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
    griddep_wait();
    griddep_launch_dependents();
    const int tile = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
    const auto [req, kvh] = head_of(a, head0);
    const Request rq = request_of(a, req, group, threadIdx.x == 0 && blockIdx.x == 0);
    const int row0 = tile * kTile;
    if (row0 >= rq.rows) return;
    const int tx = thread_x(), ty = thread_y();
    // keys any row of the tile sees
    const int last = rq.c + rq.n - rq.m + (min(row0 + kTile, rq.rows) - 1) / group;
    const int key_tiles = last / kTile + 1;
    const int per = (key_tiles + a.splits - 1) / a.splits;
    const int t0 = split * per, t1 = min(key_tiles, t0 + per);
    Fetch<D> f;
    f.rows(a, rq, group, kvh, row0);
    f.put(sm.q);
    if (t0 < t1) f.keys(a, req, kvh, t0 * kTile, last + 1);
    float m[4], l[4];
    int lim[4];   // last key of each of the thread's rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        lim[i] = rq.c + rq.n - rq.m + (row0 + ty + 16 * i) / group;
    }
    for (int t = t0; t < t1; ++t) {
        f.put(sm.k);
        __syncthreads();
        if (t + 1 < t1) f.keys(a, req, kvh, (t + 1) * kTile, last + 1);
        float s[4][4];
        scores<D>(sm, a.scale_log2, s);
        if constexpr (KEEP) {
            float* sp = a.scores +
                        (static_cast<size_t>(blockIdx.y) * a.rows_pad + row0 + ty) * a.key_pad +
                        t * kTile + tx;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sp[static_cast<size_t>(16 * i) * a.key_pad + 16 * j] = s[i][j];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (t * kTile + tx + 16 * j > lim[i]) s[i][j] = -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
            if (mx > -INFINITY) {   // this thread has seen a key of the row
                float add = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) add += fast_exp2(s[i][j] - mx);
                l[i] = l[i] * fast_exp2(m[i] - mx) + add;
                m[i] = mx;
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sm.red[0][ty + 16 * i][tx] = m[i];
        sm.red[1][ty + 16 * i][tx] = l[i];
    }
    __syncthreads();
    if (threadIdx.x < kTile) {
        const int row = threadIdx.x;
        float M = -INFINITY, l_all = 0.f;
        for (int x = 0; x < 16; ++x) M = fmaxf(M, sm.red[0][row][x]);
        if (M > -INFINITY)
            for (int x = 0; x < 16; ++x)
                l_all += sm.red[1][row][x] * fast_exp2(sm.red[0][row][x] - M);
        float2* st = a.stats + ((static_cast<size_t>(req) * a.num_kv_heads + kvh) * a.splits +
                                split) * a.rows_pad;
        if (row0 + row < rq.rows) st[row0 + row] = make_float2(M, l_all);
    }
}

// The reference and 1 / sum of row rho, from the splits' statistics of its head; 0 sums (no
// score above -inf) and NaN stay what they are.
PKV_DEVINL float2 row_stat(const PrefillWeightsArgs& a, size_t head, int rho) {
    const float2* st = a.stats + head * a.splits * a.rows_pad + rho;
    float M = -INFINITY, l = 0.f;
    for (int z = 0; z < a.splits; ++z) M = fmaxf(M, st[static_cast<size_t>(z) * a.rows_pad].x);
    for (int z = 0; z < a.splits; ++z) {
        const float2 f = st[static_cast<size_t>(z) * a.rows_pad];
        l += f.y * fast_exp2(f.x - M);
    }
    return make_float2(M, l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l));
}

// A key's sum over the rows of one part, to where it belongs.
PKV_DEVINL void put_sum(const PrefillWeightsArgs& a, const Request& rq, int req, int kvh, int part,
                        int key, float t) {
    if (a.row_parts > 1) {
        a.parts[((static_cast<size_t>(req) * a.num_kv_heads + kvh) * a.row_parts + part) *
                    a.max_context + key] = t;
    } else {
        float* w = a.weights + (static_cast<size_t>(rq.wrow) * a.num_kv_heads + kvh) *
                                   static_cast<size_t>(a.weights_stride) + key;
        *w = a.decay != 0.f ? fmaf(a.decay, *w, t) : t;
    }
}

// Pass 2 from the scores that pass 1 kept.  Grid (key tile x row parts, (request, kv head)).  A
// thread takes four neighbouring keys of every 16th row, four rows in flight.
__global__ void __launch_bounds__(kThreads, 3)
column_sums_kept_kernel(const PrefillWeightsArgs a, const int group, const int head0) {
    constexpr int kLanes = kTile / 4;            // threads per row
    constexpr int kRows = kThreads / kLanes;     // rows at a time
    __shared__ float2 stat[2][kTile];
    __shared__ float4 red[kRows][kLanes];
    griddep_wait();
    griddep_launch_dependents();
    const auto [req, kvh] = head_of(a, head0);
    const Request rq = request_of(a, req, group, false);
    const int part = blockIdx.x % a.row_parts;
    const int key0 = blockIdx.x / a.row_parts * kTile;
    const int keys = rq.c + rq.n;
    if (rq.rows == 0 || key0 >= keys) return;
    const int base = rq.c + rq.n - rq.m;
    const int first = max(0, key0 - base) * group;
    const int start = max(first / kTile * kTile, part * a.rows_per_part);
    const int stop = min(rq.rows, (part + 1) * a.rows_per_part);
    if (start >= stop) return;
    const size_t head = static_cast<size_t>(req) * a.num_kv_heads + kvh;
    const int kx = threadIdx.x % kLanes, ry = threadIdx.x / kLanes;
    const int key = key0 + 4 * kx;
    const float* sp = a.scores + static_cast<size_t>(blockIdx.y) * a.rows_pad * a.key_pad + key;
    constexpr int kIn = kTile / kRows;           // rows in flight
    float4 x[kIn];
    auto load = [&](int row0) {   // all of the tile's rows are there: rows_pad is whole tiles
#pragma unroll
        for (int u = 0; u < kIn; ++u)
            x[u] = *reinterpret_cast<const float4*>(
                sp + static_cast<size_t>(row0 + ry + kRows * u) * a.key_pad);
    };
    auto load_stat = [&](int row0, int buf) {
        const int rho = row0 + static_cast<int>(threadIdx.x);
        if (threadIdx.x < kTile)
            stat[buf][threadIdx.x] = rho < rq.rows ? row_stat(a, head, rho) : make_float2(0.f, 0.f);
    };
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    load(start);
    load_stat(start, 0);
    __syncthreads();
    int buf = 0;
    for (int row0 = start; row0 < stop; row0 += kTile, buf ^= 1) {
        float s[kIn][4];
#pragma unroll
        for (int u = 0; u < kIn; ++u) {
            s[u][0] = x[u].x; s[u][1] = x[u].y; s[u][2] = x[u].z; s[u][3] = x[u].w;
        }
        if (row0 + kTile < stop) {
            load(row0 + kTile);
            load_stat(row0 + kTile, buf ^ 1);
        }
#pragma unroll
        for (int u = 0; u < kIn; ++u) {
            const int rho = row0 + ry + kRows * u;
            const float2 f = stat[buf][ry + kRows * u];
            const int seen = rho < rq.rows ? base + rho / group - key : -1;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= seen) sum[j] = fmaf(fast_exp2(s[u][j] - f.x), f.y, sum[j]);
        }
        __syncthreads();
    }
    red[ry][kx] = make_float4(sum[0], sum[1], sum[2], sum[3]);
    __syncthreads();
    if (threadIdx.x < kTile && key0 + static_cast<int>(threadIdx.x) < keys) {
        float t = 0.f;
        for (int y = 0; y < kRows; ++y)
            t += reinterpret_cast<const float*>(&red[y][0])[threadIdx.x];
        put_sum(a, rq, req, kvh, part, key0 + threadIdx.x, t);
    }
}

// Pass 2 with the products computed again.  Grid (key tile x row parts, (request, kv head)).
template <int D>
__global__ void __launch_bounds__(kThreads)
column_sums_kernel(const PrefillWeightsArgs a, const int group, const int head0) {
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
    griddep_wait();
    griddep_launch_dependents();
    const auto [req, kvh] = head_of(a, head0);
    const size_t head = static_cast<size_t>(req) * a.num_kv_heads + kvh;
    const Request rq = request_of(a, req, group, false);
    const int part = blockIdx.x % a.row_parts;
    const int key0 = blockIdx.x / a.row_parts * kTile;
    const int keys = rq.c + rq.n;
    if (rq.rows == 0 || key0 >= keys) return;
    const int tx = thread_x(), ty = thread_y();
    Fetch<D> f;
    f.keys(a, req, kvh, key0, keys);
    f.put(sm.k);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    const int base = rq.c + rq.n - rq.m;   // last key of the window's first token
    const int first = max(0, key0 - base) * group;   // earlier rows see no key of the tile
    const int start = max(first / kTile * kTile, part * a.rows_per_part);
    const int stop = min(rq.rows, (part + 1) * a.rows_per_part);
    if (start >= stop) return;   // nothing of the part sees the tile
    f.rows(a, rq, group, kvh, start);
    for (int row0 = start; row0 < stop; row0 += kTile) {
        f.put(sm.q);
        if (threadIdx.x < kTile) {   // merge the splits' statistics of the tile's rows
            const int rho = row0 + static_cast<int>(threadIdx.x);
            const float2 st = rho < rq.rows ? row_stat(a, head, rho) : make_float2(0.f, 0.f);
            sm.red[0][threadIdx.x][0] = st.x;
            sm.red[1][threadIdx.x][0] = st.y;
        }
        __syncthreads();
        if (row0 + kTile < stop) f.rows(a, rq, group, kvh, row0 + kTile);
        float s[4][4];
        scores<D>(sm, a.scale_log2, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rho = row0 + ty + 16 * i;
            const int lim = base + rho / group;
            const float M = sm.red[0][ty + 16 * i][0], inv = sm.red[1][ty + 16 * i][0];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (rho < rq.rows && key0 + tx + 16 * j <= lim)
                    sum[j] = fmaf(fast_exp2(s[i][j] - M), inv, sum[j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sm.red[0][tx + 16 * j][ty] = sum[j];
    __syncthreads();
    if (threadIdx.x < kTile) {
        const int key = key0 + threadIdx.x;
        if (key < keys) {
            float t = 0.f;
            for (int y = 0; y < 16; ++y) t += sm.red[0][threadIdx.x][y];
            put_sum(a, rq, req, kvh, part, key, t);
        }
    }
}

// Grid (256 keys, kv head, request).
__global__ void __launch_bounds__(256)
add_parts_kernel(const PrefillWeightsArgs a, const int key_unit, const int row_unit) {
    griddep_wait();
    griddep_launch_dependents();
    const int req = blockIdx.z, kvh = blockIdx.y;
    const Request rq = request_of(a, req, 1 << a.group_shift, false);
    const int key = blockIdx.x * 256 + threadIdx.x;
    if (rq.rows == 0 || key >= rq.c + rq.n) return;
    // first row of the key's pass-2 item
    const int base = rq.c + rq.n - rq.m;
    const int first = (max(0, key / key_unit * key_unit - base) << a.group_shift) / row_unit *
                      row_unit;
    const float* s = a.parts + (static_cast<size_t>(req) * a.num_kv_heads + kvh) * a.row_parts *
                                   a.max_context + key;
    float t = 0.f;
    for (int p = 0; p < a.row_parts && p * a.rows_per_part < rq.rows; ++p)
        if ((p + 1) * a.rows_per_part > first) t += s[static_cast<size_t>(p) * a.max_context];
    float* w = a.weights + (static_cast<size_t>(rq.wrow) * a.num_kv_heads + kvh) *
                               static_cast<size_t>(a.weights_stride) + key;
    *w = a.decay != 0.f ? fmaf(a.decay, *w, t) : t;
}

template <int D>
cudaError_t launch_typed(const PrefillWeightsArgs& a, int group, cudaStream_t stream) {
    const int smem = sizeof(Smem<D>);
    const bool keep = a.scores != nullptr;
    auto pass1 = keep ? row_stats_kernel<D, true> : row_stats_kernel<D, false>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(pass1), smem);
    if (e != cudaSuccess) return e;
    if (!keep) e = set_smem_once(reinterpret_cast<const void*>(column_sums_kernel<D>), smem);
    if (e != cudaSuccess) return e;
    const int64_t row_tiles = (static_cast<int64_t>(a.max_rows) * group + kTile - 1) / kTile;
    const int64_t key_tiles = (static_cast<int64_t>(a.max_context) + kTile - 1) / kTile;
    const int64_t grid1 = row_tiles * a.splits, grid2 = key_tiles * a.row_parts;
    if (grid1 > INT32_MAX || grid2 > INT32_MAX) return cudaErrorInvalidValue;
    const int heads = a.num_reqs * a.num_kv_heads;
    for (int h = 0; h < heads; h += a.heads_per_launch) {
        const unsigned n = static_cast<unsigned>(std::min(a.heads_per_launch, heads - h));
        e = launch_pdl(pass1, dim3(static_cast<unsigned>(grid1), n), dim3(kThreads), smem, stream, a,
                       group, h);
        if (e != cudaSuccess) return e;
        e = keep ? launch_pdl(column_sums_kept_kernel, dim3(static_cast<unsigned>(grid2), n),
                              dim3(kThreads), 0, stream, a, group, h)
                 : launch_pdl(column_sums_kernel<D>, dim3(static_cast<unsigned>(grid2), n),
                              dim3(kThreads), smem, stream, a, group, h);
        if (e != cudaSuccess) return e;
    }
    return a.row_parts > 1 ? launch_add_parts(a, kTile, kTile, stream) : cudaSuccess;
}

}  // namespace

cudaError_t launch_add_parts(const PrefillWeightsArgs& a, int key_unit, int row_unit,
                             cudaStream_t stream) {
    return launch_pdl(add_parts_kernel,
                      dim3((a.max_context + 255) / 256, a.num_kv_heads, a.num_reqs), dim3(256), 0,
                      stream, a, key_unit, row_unit);
}

cudaError_t launch_prefill_weights(const PrefillWeightsArgs& a, int head_dim, int group,
                                   cudaStream_t stream) {
    return head_dim == 128 ? launch_typed<128>(a, group, stream)
                           : launch_typed<64>(a, group, stream);
}

}  // namespace pkv

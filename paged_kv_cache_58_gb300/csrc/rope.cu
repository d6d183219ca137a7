// Rotary positions, alone and with the append of the rotated keys.
//
// A row's first rotary_dim elements are pairs (x_a, x_b) turned by the angle
// pos * inv_freq[i] of their pair i:
//   y_a = x_a cos - x_b sin,   y_b = x_b cos + x_a sin,
// with a = i, b = i + rotary_dim / 2 (half layout) or a = 2i, b = 2i + 1 (interleaved);
// the elements past rotary_dim pass unchanged.
//
// Angles without rounding trouble at far positions: only the angle modulo one turn
// matters, and positions are integers.  inv_freq[i] / (2 pi) becomes a 64-bit binary
// fraction of a turn; its product with the position modulo 2^64 is the angle's fraction
// of a turn, exactly, whatever the position.  The fraction's own rounding, at most 2^-54 of
// a turn for frequencies up to one radian a position and in proportion above that, times a
// position below 2^31 stays under 2^-23 of a turn at the very end of that range and under
// 2^-33 at 2^20.  The top two bits after rounding are the quadrant; the rest, within an
// eighth of a turn, goes through sincospif.  The fraction is made anew for each (token,
// pair): five operations in fp64, which this GPU runs at 1/60 of fp32.  At 8192 tokens of 64
// pairs they keep the fp64 pipes busy for some 4 us of the 37 that the rows take (6.5 % of an
// fp32 call's 65 us); the sine, the cosine and the reduction of the angle need none.
//
// Work split: a CTA takes TT consecutive tokens.  It computes each (token, pair) angle
// once, into shared memory, and a thread then keeps the cosines and sines of its
// (token, 32-byte unit) in registers for all the rows (heads) it walks.  A unit is two
// 16-byte chunks: the chunks holding x_a and x_b (half layout), or two neighbouring
// ones (interleaved, and everywhere past rotary_dim), so that each thread loads and
// stores whole 16-byte chunks and every pair lies in one thread.  A thread's first
// rows are loaded before the angles are computed, so the two overlap.
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 2;   // rows in flight per thread (8192 tokens of 48 rows: 1, 3 and 6
                            // took 38.8, 39.1 and 37.7 us, 2 takes 36.9)

// Fraction of a turn per position, in units of 2^-64 turns.
PKV_DEVINL uint64_t turn_fraction(double inv_freq) {
    double f = inv_freq * 0.15915494309189533577;   // 1 / (2 pi)
    f -= floor(f);
    return __double2ull_rz(f * 18446744073709551616.0);
}

// cos and sin of `angle` (2^-64 turns).
PKV_DEVINL void turn_sincos(uint64_t angle, float& c, float& s) {
    const uint64_t quadrant = (angle + (uint64_t{1} << 61)) >> 62;
    const int64_t rest = static_cast<int64_t>(angle - (quadrant << 62));
    // high word: 2^-32 turns = 2^-31 half turns, within [-1/4, 1/4] half turns
    const float x = static_cast<float>(static_cast<int32_t>(rest >> 32)) * 4.656612873077393e-10f;
    float sn, cs;
    sincospif(x, &sn, &cs);
    const bool odd = quadrant & 1;
    c = odd ? sn : cs;
    s = odd ? cs : sn;
    if (quadrant == 1 || quadrant == 2) c = -c;
    if (quadrant >= 2) s = -s;
}

template <typename T>
struct Chunk;   // one 16-byte chunk as floats
template <>
struct Chunk<float> {
    static constexpr int E = 4;
    PKV_DEVINL static void get(const uint4& u, float (&f)[4]) {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    }
    PKV_DEVINL static uint4 put(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};
template <>
struct Chunk<uint16_t> {
    static constexpr int E = 8;
    PKV_DEVINL static void get(const uint4& u, float (&f)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16lo_to_f32(w[i]);
            f[2 * i + 1] = bf16hi_to_f32(w[i]);
        }
    }
    // rounded once, to nearest even
    PKV_DEVINL static uint4 put(const float (&f)[8]) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                          pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};

template <typename T, int D, bool INTERLEAVED, int TT>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const RopeArgs a) {
    using C = Chunk<T>;
    constexpr int E = C::E;
    constexpr int UPR = D / (2 * E);              // units per row
    constexpr int RL = kThreads / (UPR * TT);     // row lanes per token
    static_assert(RL >= 1, "a token's units must fit the CTA");
    __shared__ __align__(16) float cs_s[TT][D / 2];
    __shared__ __align__(16) float sn_s[TT][D / 2];

    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int unit = tid % UPR;
    const int rl = (tid / UPR) % RL;
    const int tt = tid / (UPR * RL);
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * TT;
    const int64_t tok = tok0 + tt;
    const bool live = tok < a.num_tokens;
    const int half = a.rotary_dim >> 1;
    const int turned_units = half / E;            // rotary_dim is a multiple of 2 E
    const bool turned = unit < turned_units;
    // the unit's two chunks
    const int ca = (!INTERLEAVED && turned) ? unit : 2 * unit;
    const int cb = (!INTERLEAVED && turned) ? unit + turned_units : 2 * unit + 1;

    const bool append = a.k_pool != nullptr;
    const int rows = a.num_q_heads + (append ? 2 * a.num_kv_heads : 0);
    int64_t slot = -1;
    if (append && live) {
        slot = __ldg(a.slot_mapping + tok);
        if (slot >= a.num_slots) {
            if (unit == 0 && rl == 0) raise_status(a.status, PKV_ERR_OOB);
            slot = -1;
        }
    }
    const T* q = static_cast<const T*>(a.q) + (live ? tok : 0) * a.q_stride;
    const T* k = static_cast<const T*>(a.k) + (live ? tok : 0) * a.k_stride;
    const T* v = static_cast<const T*>(a.v) + (live ? tok : 0) * a.v_stride;
    const int kv0 = a.num_q_heads;
    const int v0 = kv0 + a.num_kv_heads;

    auto load = [&](int r, uint4& xa, uint4& xb) {
        const T* src = r < kv0 ? q + static_cast<int64_t>(r) * D
                       : r < v0 ? k + static_cast<int64_t>(r - kv0) * D
                                : v + static_cast<int64_t>(r - v0) * D;
        const uint4* s = reinterpret_cast<const uint4*>(src);
        xa = s[ca];
        xb = s[cb];
    };
    // A row to move: live token, existing row, and for k and v a slot to go to.
    auto wanted = [&](int r) { return live && r < rows && (r < kv0 || slot >= 0); };

    uint4 xa[kBatch], xb[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
        if (wanted(rl + u * RL)) load(rl + u * RL, xa[u], xb[u]);

    for (int t = tid; t < TT * half; t += kThreads) {
        const int at = t / half;
        const int i = t - at * half;
        if (tok0 + at < a.num_tokens) {
            const int64_t pos = __ldg(a.positions + tok0 + at);
            uint64_t angle = turn_fraction(__ldg(a.inv_freq + i)) * static_cast<uint64_t>(pos);
            if (a.inverse) angle = 0 - angle;
            float c, s;
            turn_sincos(angle, c, s);
            cs_s[at][i] = c * a.attn_scale;
            sn_s[at][i] = s * a.attn_scale;
        }
    }
    __syncthreads();
    float cs[E], sn[E];
    if (turned) {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const float4 c4 = *reinterpret_cast<const float4*>(&cs_s[tt][unit * E + e]);
            const float4 s4 = *reinterpret_cast<const float4*>(&sn_s[tt][unit * E + e]);
            cs[e] = c4.x; cs[e + 1] = c4.y; cs[e + 2] = c4.z; cs[e + 3] = c4.w;
            sn[e] = s4.x; sn[e + 1] = s4.y; sn[e + 2] = s4.z; sn[e + 3] = s4.w;
        }
    }

    const int64_t blk = slot >= 0 ? slot >> a.block_shift : 0;
    const int64_t off = slot >= 0 ? slot & ((int64_t{1} << a.block_shift) - 1) : 0;
    for (int r0 = rl; r0 < rows; r0 += kBatch * RL) {
        if (r0 != rl) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (wanted(r0 + u * RL)) load(r0 + u * RL, xa[u], xb[u]);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int r = r0 + u * RL;
            if (!wanted(r)) continue;
            uint4 ya = xa[u], yb = xb[u];
            if (turned && r < v0) {
                float fa[E], fb[E];
                C::get(ya, fa);
                C::get(yb, fb);
                if constexpr (INTERLEAVED) {
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float a0 = fa[e], a1 = fa[e + 1], b0 = fb[e], b1 = fb[e + 1];
                        const int i = e / 2, j = E / 2 + e / 2;
                        fa[e] = a0 * cs[i] - a1 * sn[i];
                        fa[e + 1] = a1 * cs[i] + a0 * sn[i];
                        fb[e] = b0 * cs[j] - b1 * sn[j];
                        fb[e + 1] = b1 * cs[j] + b0 * sn[j];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float x = fa[e], y = fb[e];
                        fa[e] = x * cs[e] - y * sn[e];
                        fb[e] = y * cs[e] + x * sn[e];
                    }
                }
                ya = C::put(fa);
                yb = C::put(fb);
            }
            T* dst;
            if (r < kv0) {
                dst = static_cast<T*>(a.q_out) + tok * a.q_out_stride + static_cast<int64_t>(r) * D;
            } else {
                const int h = r < v0 ? r - kv0 : r - v0;
                T* pool = static_cast<T*>(r < v0 ? a.k_pool : a.v_pool);
                dst = pool + (((blk * a.num_kv_heads + h) << a.block_shift) + off) * D;
            }
            uint4* d = reinterpret_cast<uint4*>(dst);
            d[ca] = ya;
            d[cb] = yb;
        }
    }
}

template <typename T, int D, int TT>
cudaError_t launch_tt(const RopeArgs& a, cudaStream_t stream) {
    const int64_t grid = (a.num_tokens + TT - 1) / TT;
    auto kern = a.interleaved ? rope_kernel<T, D, true, TT> : rope_kernel<T, D, false, TT>;
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, a);
}

template <typename T, int D>
cudaError_t launch_d(const RopeArgs& a, cudaStream_t stream) {
    // Few tokens: one per CTA, so that as many SMs as there are tokens work; many: four, so
    // that the angles of a CTA fill its threads and a thread has more rows to walk.  At 64 tokens
    // of 48 rows one takes 2.4 us; at 8192 of them (three rows in flight) one took 42.8 us, two
    // 37.6 and four 39.1; at 4097 fp32 tokens of 16 rows 12.3, 8.4 and 7.35 us.
    return a.num_tokens >= 2048 ? launch_tt<T, D, 4>(a, stream) : launch_tt<T, D, 1>(a, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, int head_dim, cudaStream_t stream) {
    if (dtype == PKV_BF16)
        return head_dim == 128 ? launch_d<uint16_t, 128>(a, stream)
                               : launch_d<uint16_t, 64>(a, stream);
    return head_dim == 128 ? launch_d<float, 128>(a, stream) : launch_d<float, 64>(a, stream);
}

}  // namespace pkv

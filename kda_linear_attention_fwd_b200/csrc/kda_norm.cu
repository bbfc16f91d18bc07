// The norms before and after a block, fused with the block's gate and the
// scaled residual, and their gradient (kda_block_norm, kda_block_norm_bwd):
//
//   yn = y * iy,  iy = rsqrt(mean(y^2) + eps)        (post norm; else yn = y)
//   u  = act(gate) * yn * w_post
//   r  = x + c u                                     (no residual: r = c u)
//   h  = r * ir * w_pre,  ir = rsqrt(mean(r^2) + eps)  (pre norm of the next block)
//
// and for given dr, dh, with m = dh w_pre, rn = r ir:
//   dR = dr + ir (m - rn mean(m rn)),   dx = dR,   du = c dR
//   dgate = du yn w_post act'(gate),    dn = du act(gate) w_post
//   dy = iy (dn - yn mean(dn yn))                    (no post norm: dy = dn)
//   dw_post = sum_rows du act(gate) yn, dw_pre = sum_rows dh rn
//
// Everything is one pass over the rows: each input is read once in its own
// type, the row statistics are fp32, h is taken from the unrounded r, and the
// outputs are rounded once.  The floor is that traffic.  Measured on one B200
// (6531 GB/s copied): the per-head norm with its gate over 262144 rows of 128
// (201 MB) 37 us, 83% of that; its gradient over 131072 rows (168 MB) 42 us, 61%;
// the gradient of the norms around a block over 8192 rows of 4096 (537 MB) 150 us,
// 55%, bound by the instructions per element and the two rounds of row sums.
//
// A row belongs to TPR threads (a power of two; up to 32 of them inside a
// warp, more as whole warps), each holding NV vectors of VEC elements; a CTA
// of 256 threads (or of TPR, when a row takes more) holds 256 / TPR rows.
// VEC is 16 bytes when D, the strides and the addresses allow it and one
// element otherwise.  A fixed number of CTAs runs over the rows; in the
// gradient each thread thereby keeps the sums of its columns of dw in
// registers, and the CTAs' partial sums are added in a second, small launch in
// a fixed order.
#include <algorithm>
#include <type_traits>

#include "../../include/kda.h"
#include "kda_args.h"
#include "kda_common.cuh"
#include "kda_lin.h"
#include "kda_sm100.cuh"

namespace kda {
namespace norm {

constexpr int kThreads = 256;
constexpr int kMaxD = 16384;

struct Params {
    const void *y, *gate, *x, *w_post, *w_pre;
    long y_ld, gate_ld, x_ld;
    void *out, *normed;
    // gradient
    const void *dr, *dh;
    void *dy, *dgate, *dx;
    float *part;      // [gridDim][2][D]
    int want_post, want_pre;
    long rows;
    int D, tpr, flags;
    float c, eps;
};

template <typename T, int VEC> struct Vec { T e[VEC]; };
template <typename T, int VEC> struct alignas(16) Vec16 { T e[VEC]; };
template <typename T, int VEC>
using VecT = typename std::conditional<VEC == 1, Vec<T, 1>, Vec16<T, VEC>>::type;

template <typename T, int VEC>
KDA_DEVICE VecT<T, VEC> load_vec(const void *base, long at) {
    return *reinterpret_cast<const VecT<T, VEC> *>((const T *)base + at);
}
// The arithmetic runs on pairs (one fp32 instruction for two elements); a
// single element is a pair whose second half is zero.
using sm100::f2fma;
using sm100::f2mul;
KDA_DEVICE float2 pair(float x) { return make_float2(x, x); }
KDA_DEVICE float2 f2add(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}
template <int VEC> constexpr int kPairs = VEC == 1 ? 1 : VEC / 2;
template <typename T, int VEC>
KDA_DEVICE float2 get(const VecT<T, VEC> &v, int i) {
    if constexpr (VEC == 1) return make_float2(ld(&v.e[0]), 0.f);
    else if constexpr (VEC == 8) return sm100::unpack_bf16(reinterpret_cast<const uint32_t *>(v.e)[i]);
    else return make_float2(ld(&v.e[2 * i]), ld(&v.e[2 * i + 1]));
}
template <typename T, int VEC>
KDA_DEVICE void store_vec(void *base, long at, const float2 (&v)[kPairs<VEC>]) {
    VecT<T, VEC> o;
    if constexpr (VEC == 1) {
        st(&o.e[0], v[0].x);
    } else if constexpr (VEC == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t *>(o.e)[i] = sm100::pack_bf16(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kPairs<VEC>; ++i) {
            st(&o.e[2 * i], v[i].x);
            st(&o.e[2 * i + 1], v[i].y);
        }
    }
    *reinterpret_cast<VecT<T, VEC> *>((T *)base + at) = o;
}

// Sum of N values over the TPR threads of a row (every thread gets it).  red
// is not written again before another barrier of the CTA.  Two or three sums
// over several warps go through one tree of four: a step halves the values
// that a lane still carries, 6 shuffles instead of 5 for each.
template <int N>
KDA_DEVICE void row_sum(float (&v)[N], int tpr, float (*red)[4]) {
    const unsigned all = 0xffffffffu;
    if (tpr <= 32) {
        for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(all, v[i], o);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = tpr >> 5, first = warp / nw * nw;
    if constexpr (N == 1) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[0] += __shfl_xor_sync(all, v[0], o);
        if (lane == 0) red[warp][0] = v[0];
        __syncthreads();
        v[0] = lane < nw ? red[first + lane][0] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[0] += __shfl_xor_sync(all, v[0], o);
    } else {
        float x[4] = {v[0], v[1], N > 2 ? v[N > 2 ? 2 : 0] : 0.f, 0.f};
        const bool hi = lane & 16, mid = lane & 8;  // value 2 hi + mid stays in this lane
        const float y0 = (hi ? x[2] : x[0]) + __shfl_xor_sync(all, hi ? x[0] : x[2], 16);
        const float y1 = (hi ? x[3] : x[1]) + __shfl_xor_sync(all, hi ? x[1] : x[3], 16);
        float z = (mid ? y1 : y0) + __shfl_xor_sync(all, mid ? y0 : y1, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) z += __shfl_xor_sync(all, z, o);
        if ((lane & 7) == 0) red[warp][(hi ? 2 : 0) + (mid ? 1 : 0)] = z;
        __syncthreads();
        z = 0.f;  // lane: value lane % 4 of warps lane / 4, + 8, ...
#pragma unroll
        for (int w = 0; w < 32; w += 8)
            if (w + (lane >> 2) < nw) z += red[first + w + (lane >> 2)][lane & 3];
#pragma unroll
        for (int o = 16; o > 2; o >>= 1) z += __shfl_xor_sync(all, z, o);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(all, z, i);
    }
}

// The gate: none, as given, its logistic function, z times that.  GATE_ANY:
// decided at run time (the single-element kernels, which are not worth four
// instances each).
enum Gate { GATE_NONE, GATE_GIVEN, GATE_SIGMOID, GATE_SILU, GATE_ANY };
template <int G>
KDA_DEVICE int gate_of(const Params &p) {
    if (G != GATE_ANY) return G;
    if (!p.gate) return GATE_NONE;
    return (p.flags & KDA_NORM_GATE_SIGMOID) ? GATE_SIGMOID : (p.flags & KDA_NORM_GATE_SILU) ? GATE_SILU : GATE_GIVEN;
}
// 1 / (1 + exp(-z)) of a pair, with the approximate reciprocal (an ulp; 0 below
// 2^-126): IEEE division would be a third of the gated kernels' instructions.  The
// exponential is that of the rounded z log2 e, off by up to 2^-18.  bf16 rows, whose
// results keep 8 bits, take it as it is; fp32 rows multiply it by 2 to the power of
// what was rounded away, 1 + lo ln 2, which costs them nothing (6553 rows of 5120,
// norm, gate, residual and norm: 130 us; expf 165, and IEEE division too 145 with
// rows of 2304 at 229 instead of 127).
constexpr float kLog2e = 1.4426950408889634f, kLog2eLo = (float)(1.4426950408889634 - (double)kLog2e);
template <typename T>
KDA_DEVICE float2 logistic(float2 z) {
    const float2 t = f2mul(z, pair(-kLog2e));
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    if constexpr (std::is_same<T, float>::value) {
        // (where z is so large that lo is no such rounding, e is 0 or infinity and has to stay that)
        float2 lo = f2fma(z, pair(-kLog2eLo), f2fma(z, pair(-kLog2e), make_float2(-t.x, -t.y)));
        lo = make_float2(fminf(fmaxf(lo.x, -1.f), 1.f), fminf(fmaxf(lo.y, -1.f), 1.f));
        e = f2mul(e, f2fma(lo, pair(0.6931471805599453f), pair(1.f)));
    }
    e = f2add(e, pair(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
    return r;
}
// act(z) and its slope, s being logistic(z) where the gate has one
KDA_DEVICE float2 act_of(int g, float2 z, float2 s) {
    return g == GATE_GIVEN ? z : g == GATE_SIGMOID ? s : f2mul(z, s);
}
KDA_DEVICE float2 slope_of(int g, float2 z, float2 s) {
    if (g == GATE_GIVEN) return pair(1.f);
    const float2 rest = f2fma(s, pair(-1.f), pair(1.f));  // 1 - s
    return g == GATE_SIGMOID ? f2mul(s, rest) : f2fma(f2mul(z, s), rest, s);
}

// The thread's part of a weight, or ones
template <typename T, int VEC, int NV>
KDA_DEVICE void load_weight(float2 (&w)[NV][kPairs<VEC>], const void *base, int tpr, int t, int D) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * VEC;
        VecT<T, VEC> v;
        if (base && c < D) v = load_vec<T, VEC>(base, c);
#pragma unroll
        for (int e = 0; e < kPairs<VEC>; ++e) w[i][e] = base && c < D ? get<T, VEC>(v, e) : pair(1.f);
    }
}

// A fixed number of CTAs runs over the rows; the weights stay in registers
// (rows of one vector per thread) and the vectors of the next row are
// requested before this row's arithmetic ends.
template <typename T, int VEC, int NV, int MT, int G, bool RES, bool PRE>
__global__ void __launch_bounds__(MT) fwd_kernel(const __grid_constant__ Params p) {
    constexpr int NP = kPairs<VEC>;
    __shared__ float red[2][2][32][4];
    const int tpr = p.tpr, t = threadIdx.x & (tpr - 1), g = gate_of<G>(p);
    const int per = blockDim.x / tpr;
    const bool post = p.flags & KDA_NORM_POST;
    const float inv_d = 1.f / p.D;
    VecT<T, VEC> y[NV], z[NV], x[NV];
    auto load = [&](long row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            if (row < p.rows && c < p.D) {
                y[i] = load_vec<T, VEC>(p.y, row * p.y_ld + c);
                if (g != GATE_NONE) z[i] = load_vec<T, VEC>(p.gate, row * p.gate_ld + c);
                if (RES) x[i] = load_vec<T, VEC>(p.x, row * p.x_ld + c);
            }
        }
    };
    const long step = (long)gridDim.x * per;
    long row = (long)blockIdx.x * per + threadIdx.x / tpr;
    load(row);
    float2 wa[NV][NP], wb[PRE ? NV : 1][NP];
    if (NV == 1) {
        load_weight<T, VEC, NV>(wa, p.w_post, tpr, t, p.D);
        if constexpr (PRE) load_weight<T, VEC, NV>(wb, p.w_pre, tpr, t, p.D);
    }
    int par = 0;
    for (long row0 = (long)blockIdx.x * per; row0 < p.rows; row0 += step, row += step, par ^= 1) {
        if (NV > 1) load_weight<T, VEC, NV>(wa, p.w_post, tpr, t, p.D);
        float2 u[NV][NP];
        float f = p.c;  // iy c
        float2 ss = pair(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = row < p.rows && (i * tpr + t) * VEC < p.D;
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                u[i][e] = in ? get<T, VEC>(y[i], e) : pair(0.f);
                ss = f2fma(u[i][e], u[i][e], ss);
            }
        }
        if (post) {
            float s1[1] = {ss.x + ss.y};
            row_sum(s1, tpr, red[par][0]);
            f *= rsqrtf(fmaf(s1[0], inv_d, p.eps));
        }
        float2 rr = pair(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            if (row < p.rows && c < p.D) {
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    float2 a = wa[i][e];
                    if (g != GATE_NONE) {
                        const float2 zz = get<T, VEC>(z[i], e);
                        a = f2mul(a, act_of(g, zz, g >= GATE_SIGMOID ? logistic<T>(zz) : pair(0.f)));
                    }
                    a = f2mul(a, u[i][e]);
                    u[i][e] = RES ? f2fma(a, pair(f), get<T, VEC>(x[i], e)) : f2mul(a, pair(f));
                    if (PRE) rr = f2fma(u[i][e], u[i][e], rr);
                }
                store_vec<T, VEC>(p.out, row * p.D + c, u[i]);
            }
        }
        load(row + step);
        if constexpr (PRE) {
            if (NV > 1) load_weight<T, VEC, NV>(wb, p.w_pre, tpr, t, p.D);
            float s1[1] = {rr.x + rr.y};
            row_sum(s1, tpr, red[par][1]);
            const float2 ir = pair(rsqrtf(fmaf(s1[0], inv_d, p.eps)));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * tpr + t) * VEC;
                if (row < p.rows && c < p.D) {
#pragma unroll
                    for (int e = 0; e < NP; ++e) u[i][e] = f2mul(u[i][e], f2mul(ir, wb[i][e]));
                    store_vec<T, VEC>(p.normed, row * p.D + c, u[i]);
                }
            }
        }
    }
}

// RES: a residual that the norm of `out` needs.  PRE: that norm is there and
// has a gradient.  A row's vectors stay in registers in their own type.  The
// row sums are what a row waits for, so there are as few as the algebra allows:
// mean(dn yn) is taken apart into sums over a = w_post act(gate) y that are
// known before dn is, one round of sums without PRE and two with it.
// Rows that bwd_kernel requests ahead through shared memory, and its CTAs per
// SM.  One row's vectors of 512 threads are 40 KB: without rows ahead a CTA
// waited for memory once per row (8192 x 4096: 198 us, 155 us with them).
template <int MT> constexpr int kBwdCtas = MT == 256 ? 3 : 1;
template <int VEC, int NV, int MT>
constexpr int kStages = VEC == 1 || 5 * NV * MT * 16 * 2 * kBwdCtas<MT> > 200 * 1024 ? 0
                        : 5 * NV * MT * 16 * 3 * kBwdCtas<MT> > 200 * 1024 ? 2 : 3;

template <typename T, int VEC, int NV, int MT, int G, bool PRE, bool RES>
__global__ void __launch_bounds__(MT, kBwdCtas<MT>) bwd_kernel(const __grid_constant__ Params p) {
    constexpr int NP = kPairs<VEC>, ST = kStages<VEC, NV, MT>;
    using V = VecT<T, VEC>;
    __shared__ float red[2][2][32][4];
    extern __shared__ __align__(16) unsigned char dyn[];
    float *colsum = reinterpret_cast<float *>(dyn);  // [2][D], when a CTA holds more than one row (at the end)
    const int tpr = p.tpr, t = threadIdx.x & (tpr - 1), g = gate_of<G>(p);
    const int per = blockDim.x / tpr, sub = threadIdx.x / tpr;
    const bool post = p.flags & KDA_NORM_POST;
    const float inv_d = 1.f / p.D;
    float2 gpost[NV][NP], gpre[PRE ? NV : 1][NP];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            gpost[i][e] = pair(0.f);
            if (PRE) gpre[i][e] = pair(0.f);
        }
    // The vectors of a row, y, gate, residual, dr, dh: with stages they wait in
    // shared memory, each thread reading back only what it has copied
    V reg[ST ? 1 : 5][ST ? 1 : NV] = {};
    V *stage = reinterpret_cast<V *>(dyn) + threadIdx.x;
    int slot = 0;
    auto at = [&](int kind, int i) -> V { return ST ? stage[((slot * 5 + kind) * NV + i) * MT] : reg[ST ? 0 : kind][ST ? 0 : i]; };
    auto load = [&](long row, int to) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            if (row < p.rows && c < p.D) {
                auto one = [&](int kind, const void *base, long off) {
                    if constexpr (ST > 0)
                        sm100::cp_async16(&stage[((to * 5 + kind) * NV + i) * MT], (const T *)base + off, true);
                    else
                        reg[ST ? 0 : kind][ST ? 0 : i] = load_vec<T, VEC>(base, off);
                };
                one(0, p.y, row * p.y_ld + c);
                if (g != GATE_NONE) one(1, p.gate, row * p.gate_ld + c);
                if (RES) one(2, p.x, row * p.x_ld + c);
                if (p.dr) one(3, p.dr, row * p.D + c);
                if (PRE) one(4, p.dh, row * p.D + c);
            }
        }
        if (ST > 0) sm100::cp_async_commit();
    };
    const long step = (long)gridDim.x * per;
    long row = (long)blockIdx.x * per + sub;
    if (ST == 0) load(row, 0);
#pragma unroll
    for (int i = 0; i + 1 < ST; ++i) load(row + i * step, i);
    float2 wa[NV][NP], wb[PRE ? NV : 1][NP];
    if (NV == 1) {
        load_weight<T, VEC, NV>(wa, p.w_post, tpr, t, p.D);
        if constexpr (PRE) load_weight<T, VEC, NV>(wb, p.w_pre, tpr, t, p.D);
    }
    int par = 0;
    for (long row0 = (long)blockIdx.x * per; row0 < p.rows; row0 += step, row += step, par ^= 1) {
        const bool live = row < p.rows;
        if constexpr (ST > 0) {
            load(row + (ST - 1) * step, slot == 0 ? ST - 1 : slot - 1);
            sm100::cp_async_wait<ST - 1>();
        }
        if (NV > 1) {
            load_weight<T, VEC, NV>(wa, p.w_post, tpr, t, p.D);
            if constexpr (PRE) load_weight<T, VEC, NV>(wb, p.w_pre, tpr, t, p.D);
        }
        float2 sg[NV][NP];                                  // logistic(gate)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (g >= GATE_SIGMOID && live && (i * tpr + t) * VEC < p.D)
#pragma unroll
                for (int e = 0; e < NP; ++e) sg[i][e] = logistic<T>(get<T, VEC>(at(1, i), e));
        auto weighted_act = [&](int i, int e) {             // w_post act(gate)
            return g == GATE_NONE ? wa[i][e] : f2mul(wa[i][e], act_of(g, get<T, VEC>(at(1, i), e), sg[i][e]));
        };
        // with a = w_post act(gate) y: sum y^2, sum dr a, sum dh w_pre a
        float iy = 1.f, s_dra = 0.f, s_ma = 0.f;
        if (post || PRE) {
            float2 q[3] = {pair(0.f), pair(0.f), pair(0.f)};
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live && (i * tpr + t) * VEC < p.D)
#pragma unroll
                    for (int e = 0; e < NP; ++e) {
                        const float2 v = get<T, VEC>(at(0, i), e), a = f2mul(weighted_act(i, e), v);
                        q[0] = f2fma(v, v, q[0]);
                        if (p.dr) q[1] = f2fma(get<T, VEC>(at(3, i), e), a, q[1]);
                        if constexpr (PRE) q[2] = f2fma(f2mul(get<T, VEC>(at(4, i), e), wb[i][e]), a, q[2]);
                    }
            float s1[PRE ? 3 : 2] = {q[0].x + q[0].y, q[1].x + q[1].y};
            if constexpr (PRE) s1[2] = q[2].x + q[2].y;
            row_sum(s1, tpr, red[par][0]);
            if (post) iy = rsqrtf(fmaf(s1[0], inv_d, p.eps));
            s_dra = s1[1];
            if constexpr (PRE) s_ma = s1[2];
        }
        // sum r^2, sum dh w_pre r, sum r a
        const float f = iy * p.c;
        float ir = 0.f, k2 = 0.f;                           // dR = dr + ir dh w_pre - k2 r
        float k3 = f * s_dra;                               // sum dn yn, then dy = iy dn - k3 y
        float2 r[PRE ? NV : 1][NP];                         // out, unrounded
        if constexpr (PRE) {
            float2 q[3] = {pair(0.f), pair(0.f), pair(0.f)};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (live && (i * tpr + t) * VEC < p.D) {
#pragma unroll
                    for (int e = 0; e < NP; ++e) {
                        const float2 a = f2mul(weighted_act(i, e), get<T, VEC>(at(0, i), e));
                        const float2 v = RES ? f2fma(a, pair(f), get<T, VEC>(at(2, i), e)) : f2mul(a, pair(f));
                        r[i][e] = v;
                        q[0] = f2fma(v, v, q[0]);
                        q[1] = f2fma(f2mul(get<T, VEC>(at(4, i), e), wb[i][e]), v, q[1]);
                        q[2] = f2fma(v, a, q[2]);
                    }
                }
            }
            float s[3] = {q[0].x + q[0].y, q[1].x + q[1].y, q[2].x + q[2].y};
            row_sum(s, tpr, red[par][1]);
            ir = rsqrtf(fmaf(s[0], inv_d, p.eps));
            k2 = s[1] * ir * ir * ir * inv_d;
            k3 = f * (s_dra + ir * s_ma - k2 * s[2]);
        }
        k3 = post ? k3 * iy * iy * inv_d : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + t) * VEC;
            if (live && c < p.D) {
                float2 dR[NP], dz[NP], dy[NP];
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    const float2 yv = get<T, VEC>(at(0, i), e), yn = f2mul(yv, pair(iy));
                    float2 d = p.dr ? get<T, VEC>(at(3, i), e) : pair(0.f);
                    if constexpr (PRE) {
                        const float2 dhe = get<T, VEC>(at(4, i), e);
                        d = f2fma(r[i][e], pair(-k2), f2fma(f2mul(dhe, wb[i][e]), pair(ir), d));
                        gpre[i][e] = f2fma(dhe, f2mul(r[i][e], pair(ir)), gpre[i][e]);
                    }
                    dR[e] = d;
                    const float2 du = f2mul(d, pair(p.c));
                    const float2 q = f2mul(du, yn);
                    if (g != GATE_NONE) {
                        const float2 zz = get<T, VEC>(at(1, i), e);
                        dz[e] = f2mul(f2mul(q, wa[i][e]), slope_of(g, zz, sg[i][e]));
                        gpost[i][e] = f2fma(q, act_of(g, zz, sg[i][e]), gpost[i][e]);
                    } else {
                        gpost[i][e] = f2add(gpost[i][e], q);
                    }
                    dy[e] = f2fma(yv, pair(-k3), f2mul(f2mul(du, weighted_act(i, e)), pair(iy)));
                }
                if (p.dx) store_vec<T, VEC>(p.dx, row * p.D + c, dR);
                if (g != GATE_NONE && p.dgate) store_vec<T, VEC>(p.dgate, row * p.D + c, dz);
                store_vec<T, VEC>(p.dy, row * p.D + c, dy);
            }
        }
        if (ST == 0) load(row + step, 0);
        slot = slot + 1 == ST ? 0 : slot + 1;
    }
    if (ST > 0) __syncthreads();  // the stages become the column sums
    if (!p.want_post && !p.want_pre) return;
    // this CTA's column sums: over its row groups in order, then to the workspace
    float *dst = p.part + (size_t)blockIdx.x * 2 * p.D;
    for (int s = 0; s < per; ++s) {
        if (per > 1) __syncthreads();
        if (sub == s) {
            float *to = per > 1 ? colsum : dst;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * tpr + t) * VEC;
                if (c < p.D)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float a = e & 1 ? gpost[i][e / 2].y : gpost[i][e / 2].x;
                        to[c + e] = (s ? to[c + e] : 0.f) + a;
                        if (PRE) {
                            const float b = e & 1 ? gpre[i][e / 2].y : gpre[i][e / 2].x;
                            to[p.D + c + e] = (s ? to[p.D + c + e] : 0.f) + b;
                        } else {
                            to[p.D + c + e] = 0.f;
                        }
                    }
            }
        }
    }
    if (per > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * p.D; c += blockDim.x) dst[c] = colsum[c];
    }
}

// dw[c] = sum over the CTAs' partial sums in a fixed order: 32 columns x 32
// parts at a time per CTA, four of each thread's loads in flight.
__global__ void __launch_bounds__(1024) weight_sum_kernel(const float *part, int parts, int D, float *dpost, float *dpre) {
    __shared__ float s[32][33];
    lin::after_previous();
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5, c = blockIdx.x * 32 + cx;
    float *out = blockIdx.y ? dpre : dpost;
    if (!out) return;
    const float *src = part + (size_t)blockIdx.y * D + c;
    float a = 0.f;
    if (c < D) {
        int i = ry;
        for (; i + 96 < parts; i += 128) {
            const float x0 = src[(size_t)i * 2 * D], x1 = src[(size_t)(i + 32) * 2 * D], x2 = src[(size_t)(i + 64) * 2 * D],
                        x3 = src[(size_t)(i + 96) * 2 * D];
            a += (x0 + x1) + (x2 + x3);
        }
        for (; i < parts; i += 32) a += src[(size_t)i * 2 * D];
    }
    s[ry][cx] = a;
    __syncthreads();
    a = s[cx][ry];  // column ry, part cx
    a = warp_sum(a);
    if (cx == 0 && blockIdx.x * 32 + ry < D) out[blockIdx.x * 32 + ry] = a;
}

struct Shape {
    int vec, nv, tpr, threads, per;
};
// Threads per row: one vector each while 512 threads are enough, so that all
// of a row's loads are in flight at once and the row's values take few
// registers; 2, 4 or, for single elements, 16 behind that.
Shape choose_shape(int D, int vec) {
    static constexpr int most[5][2] = {{1, 512}, {2, 512}, {2, 1024}, {4, 1024}, {16, 1024}};
    const int vecs = (D + vec - 1) / vec;
    int i = 0;
    while (i < 4 && most[i][0] * most[i][1] < vecs) ++i;
    Shape s;
    s.vec = vec;
    s.nv = most[i][0];
    s.tpr = 1;
    while (s.tpr * s.nv < vecs) s.tpr *= 2;
    s.threads = std::max(kThreads, s.tpr);
    s.per = s.threads / s.tpr;
    return s;
}

template <typename T, int VEC, int NV, int MT, int G, bool PRE, bool RES>
cudaError_t launch_k(const Params &p, const Shape &s, bool bwd, unsigned grid, cudaStream_t st) {
    if (bwd) {
        constexpr int stages = 5 * kStages<VEC, NV, MT> * NV * MT * 16;
        if (stages > 48 * 1024) {
            static std::atomic<uint64_t> done;
            const cudaError_t e = lin::allow_smem(done, (const void *)bwd_kernel<T, VEC, NV, MT, G, PRE, RES>, stages);
            if (e != cudaSuccess) return e;
        }
        const int sums = s.per > 1 ? 2 * p.D * (int)sizeof(float) : 0;
        bwd_kernel<T, VEC, NV, MT, G, PRE, RES><<<grid, s.threads, std::max(stages, sums), st>>>(p);
    } else {
        fwd_kernel<T, VEC, NV, MT, G, RES, PRE><<<grid, s.threads, 0, st>>>(p);
    }
    return cudaGetLastError();
}
template <typename T, int VEC, int NV, int MT, int G>
cudaError_t launch_g(const Params &p, const Shape &s, bool bwd, unsigned grid, cudaStream_t st) {
    const bool pre = (p.flags & KDA_NORM_PRE) && (!bwd || p.dh);
    if (pre && p.x) return launch_k<T, VEC, NV, MT, G, true, true>(p, s, bwd, grid, st);
    if (pre) return launch_k<T, VEC, NV, MT, G, true, false>(p, s, bwd, grid, st);
    if (bwd || !p.x) return launch_k<T, VEC, NV, MT, G, false, false>(p, s, bwd, grid, st);
    fwd_kernel<T, VEC, NV, MT, G, true, false><<<grid, s.threads, 0, st>>>(p);
    return cudaGetLastError();
}
template <typename T, int VEC, int NV, int MT>
cudaError_t launch_nv(const Params &p, const Shape &s, bool bwd, unsigned grid, cudaStream_t st) {
    if constexpr (VEC == 1) {
        return launch_g<T, VEC, NV, MT, GATE_ANY>(p, s, bwd, grid, st);
    } else {
        if (!p.gate) return launch_g<T, VEC, NV, MT, GATE_NONE>(p, s, bwd, grid, st);
        if (p.flags & KDA_NORM_GATE_SIGMOID) return launch_g<T, VEC, NV, MT, GATE_SIGMOID>(p, s, bwd, grid, st);
        if (p.flags & KDA_NORM_GATE_SILU) return launch_g<T, VEC, NV, MT, GATE_SILU>(p, s, bwd, grid, st);
        return launch_g<T, VEC, NV, MT, GATE_GIVEN>(p, s, bwd, grid, st);
    }
}
template <typename T, int VEC>
cudaError_t launch_vec(const Params &p, const Shape &s, bool bwd, unsigned grid, cudaStream_t st) {
    if (s.nv == 1 && s.threads == 256) return launch_nv<T, VEC, 1, 256>(p, s, bwd, grid, st);
    if (s.nv == 1) return launch_nv<T, VEC, 1, 512>(p, s, bwd, grid, st);
    if (s.nv == 2 && s.threads == 512) return launch_nv<T, VEC, 2, 512>(p, s, bwd, grid, st);
    if (s.nv == 2) return launch_nv<T, VEC, 2, 1024>(p, s, bwd, grid, st);
    // 8 elements x 2 x 1024 = kMaxD: longer rows are fp32 or single elements
    if constexpr (VEC <= 4) {
        if (s.nv == 4) return launch_nv<T, VEC, 4, 1024>(p, s, bwd, grid, st);
    }
    if constexpr (VEC == 1) return launch_nv<T, 1, 16, 1024>(p, s, bwd, grid, st);
    return cudaErrorInvalidValue;
}
template <typename T>
cudaError_t launch_t(const Params &p, const Shape &s, bool bwd, unsigned grid, cudaStream_t st) {
    if (s.vec == 1) return launch_vec<T, 1>(p, s, bwd, grid, st);
    return launch_vec<T, 16 / (int)sizeof(T)>(p, s, bwd, grid, st);
}

}  // namespace norm
}  // namespace kda

namespace {

using kda::is_aligned;
using kda::norm::Params;
using kda::norm::Shape;

int sm_count() { return kda::lin::sm_count(); }

int check_shape(int64_t rows, int32_t D, kda_dtype dtype, int32_t flags, float eps) {
    const int all = KDA_NORM_POST | KDA_NORM_PRE | KDA_NORM_GATE_SIGMOID | KDA_NORM_GATE_SILU;
    const int acts = KDA_NORM_GATE_SIGMOID | KDA_NORM_GATE_SILU;
    if (rows < 0 || D < 1 || (flags & ~all) || (flags & acts) == acts || !(eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
    if (D > kda::norm::kMaxD || rows > (1LL << 40) / D) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// 16-byte vectors when every row of every buffer allows them
int vec_of(const Params &p, const void *const *ptrs, int n, size_t esz) {
    const int vec = (int)(16 / esz);
    if (p.D % vec || p.y_ld % vec || (p.gate && p.gate_ld % vec) || (p.x && p.x_ld % vec)) return 1;
    for (int i = 0; i < n; ++i)
        if (ptrs[i] && !is_aligned(ptrs[i], 16)) return 1;
    return vec;
}
int check_elems(const void *const *ptrs, int n, size_t esz) {
    for (int i = 0; i < n; ++i)
        if (ptrs[i] && !is_aligned(ptrs[i], esz)) return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}

int bwd_parts(int64_t rows, const Shape &s) {
    const int64_t batches = (rows + s.per - 1) / s.per;
    return (int)std::max<int64_t>(1, std::min<int64_t>(batches, (int64_t)sm_count() * (s.threads == 256 ? kda::norm::kBwdCtas<256> : 1)));
}

}  // namespace

extern "C" {

int kda_block_norm(const void *y, int64_t y_stride, const void *post_weight, const void *gate, int64_t gate_stride,
                   const void *residual, int64_t residual_stride, const void *pre_weight, void *out, void *normed,
                   int64_t rows, int32_t D, kda_dtype dtype, float res_scale, float eps, int32_t flags,
                   kda_stream_t stream) {
    int rc = check_shape(rows, D, dtype, flags, eps);
    if (rc != KDA_OK) return rc;
    if ((post_weight && !(flags & KDA_NORM_POST)) || (pre_weight && !(flags & KDA_NORM_PRE))) return KDA_ERR_INVALID_ARG;
    if (rows == 0) return KDA_OK;
    if ((normed != nullptr) != ((flags & KDA_NORM_PRE) != 0)) return KDA_ERR_INVALID_ARG;
    if (!y || !out || y_stride < D || (gate && gate_stride < D) || (residual && residual_stride < D))
        return KDA_ERR_INVALID_ARG;
    const bool bf16 = dtype == KDA_DTYPE_BF16;
    const void *ptrs[] = {y, gate, residual, post_weight, pre_weight, out, normed};
    rc = check_elems(ptrs, 7, bf16 ? 2 : 4);
    if (rc != KDA_OK) return rc;
    Params p{};
    p.y = y; p.gate = gate; p.x = residual; p.w_post = post_weight; p.w_pre = pre_weight;
    p.y_ld = y_stride; p.gate_ld = gate_stride; p.x_ld = residual_stride;
    p.out = out; p.normed = normed;
    p.rows = rows; p.D = D; p.flags = flags; p.c = res_scale; p.eps = eps;
    const Shape s = kda::norm::choose_shape(D, vec_of(p, ptrs, 7, bf16 ? 2 : 4));
    p.tpr = s.tpr;
    // as many CTAs as an SM holds at 64 (with the pre norm) or 40 registers a thread
    const int64_t grid = std::min<int64_t>((rows + s.per - 1) / s.per, (int64_t)sm_count() * std::max(1, (flags & KDA_NORM_PRE ? 1024 : 1536) / s.threads));
    const cudaError_t e = bf16 ? kda::norm::launch_t<__nv_bfloat16>(p, s, false, (unsigned)grid, (cudaStream_t)stream)
                               : kda::norm::launch_t<float>(p, s, false, (unsigned)grid, (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_block_norm_bwd_workspace_size(int64_t rows, int32_t D, kda_dtype dtype) {
    if (check_shape(rows, D, dtype, 0, 0.f) != KDA_OK) return 0;
    // the most partial sums either vector width makes
    const int wide = bwd_parts(rows, kda::norm::choose_shape(D, dtype == KDA_DTYPE_BF16 ? 8 : 4));
    const int one = bwd_parts(rows, kda::norm::choose_shape(D, 1));
    return (size_t)std::max(wide, one) * 2 * D * sizeof(float);
}

int kda_block_norm_bwd(const void *dout, const void *dnormed, const void *y, int64_t y_stride, const void *post_weight,
                       const void *gate, int64_t gate_stride, const void *residual, int64_t residual_stride,
                       const void *pre_weight, void *dy, void *dgate, void *dresidual, float *dpost_weight,
                       float *dpre_weight, int64_t rows, int32_t D, kda_dtype dtype, float res_scale, float eps,
                       int32_t flags, void *workspace, size_t workspace_bytes, kda_stream_t stream) {
    cudaStream_t st = (cudaStream_t)stream;
    int rc = check_shape(rows, D, dtype, flags, eps);
    if (rc != KDA_OK) return rc;
    if ((post_weight && !(flags & KDA_NORM_POST)) || (pre_weight && !(flags & KDA_NORM_PRE)) ||
        (dpost_weight && !post_weight) || (dpre_weight && !pre_weight) || (dnormed && !(flags & KDA_NORM_PRE)) ||
        (dgate && !gate) || (dresidual && !residual))
        return KDA_ERR_INVALID_ARG;
    const bool weights = dpost_weight || dpre_weight;
    if (rows > 0 && (!y || !dy || (!dout && !dnormed) || y_stride < D || (gate && gate_stride < D) ||
                     (residual && residual_stride < D)))
        return KDA_ERR_INVALID_ARG;
    const bool bf16 = dtype == KDA_DTYPE_BF16;
    const void *ptrs[] = {y, gate, residual, post_weight, pre_weight, dout, dnormed, dy, dgate, dresidual};
    rc = check_elems(ptrs, 10, bf16 ? 2 : 4);
    if (rc != KDA_OK) return rc;
    if (!is_aligned(dpost_weight, 4) || !is_aligned(dpre_weight, 4) || !is_aligned(workspace, 16)) return KDA_ERR_ALIGNMENT;
    Params p{};
    p.y = y; p.gate = gate; p.x = residual; p.w_post = post_weight; p.w_pre = pre_weight;
    p.y_ld = y_stride; p.gate_ld = gate_stride; p.x_ld = residual_stride;
    p.dr = dout; p.dh = dnormed; p.dy = dy; p.dgate = dgate; p.dx = dresidual;
    p.rows = rows; p.D = D; p.flags = flags; p.c = res_scale; p.eps = eps;
    p.want_post = dpost_weight != nullptr;
    p.want_pre = dpre_weight != nullptr;
    const Shape s = kda::norm::choose_shape(D, vec_of(p, ptrs, 10, bf16 ? 2 : 4));
    p.tpr = s.tpr;
    const int parts = bwd_parts(rows, s);
    if (weights && (!workspace || workspace_bytes < (size_t)parts * 2 * D * sizeof(float))) return KDA_ERR_WORKSPACE;
    p.part = (float *)workspace;
    if (rows > 0) {
        const cudaError_t e = bf16 ? kda::norm::launch_t<__nv_bfloat16>(p, s, true, (unsigned)parts, st)
                                   : kda::norm::launch_t<float>(p, s, true, (unsigned)parts, st);
        if (e != cudaSuccess) return KDA_ERR_CUDA;
    }
    if (weights) {
        if (kda::lin::launch(kda::norm::weight_sum_kernel, dim3((D + 31) / 32, 2), 1024, 0, st, rows > 0, p.part,
                             rows > 0 ? parts : 0, D, dpost_weight, dpre_weight) != cudaSuccess)
            return KDA_ERR_CUDA;
    }
    return KDA_OK;
}

}  // extern "C"

// Linear attention with one decay per head, token by token in fp32: the
// forward, its window summaries and the gradient's three passes.
//
// The recurrence itself (kda_lin.h) costs two FMAs per state element and
// token, so fp32 inputs, which the tensor cores could only take split into
// several products, run it directly: the whole state of one head sits in the
// registers of one CTA of 128 threads and every product is a plain fp32 FMA
// (the paired instruction has the same rate, and its operands would have to be
// put together first).  Three things keep it near two FMAs:
//   * the decay is one number, so it is kept outside the state: the registers
//     hold S / e^G with G the log-decay summed since the last renormalisation;
//     a write adds k (v e^-G)^T and a read is scaled by e^G.  The state is
//     renormalised (one multiply per element) every 16 tokens, and at every
//     token of a group of four over which G falls below -40, so e^-G stays in
//     range and G is always a short sum (its rounding is what limits the
//     decay's accuracy);
//   * a warp's 32 lanes are RG row groups x CGW column groups, each thread
//     holding RT rows x 4 columns, so the vectors come from shared memory as
//     broadcast 16-byte reads (17 reads for 256 FMAs at 128 x 128);
//   * four tokens at a time: their partial outputs are summed over the row
//     groups together (12 shuffles, after which a lane holds one token's four
//     columns), so that the sums of one token do not hold up the next.
// Tokens arrive 16 at a time by cp.async, up to three blocks ahead.
//
// The gradient in the same form (B_t = dL/dS_t, L = sum o . do + <dS_T, S_T>):
//   B_t = exp(g_{t+1}) B_{t+1} + scale q_t do_t^T
//   dq_t = scale S_t do_t,  dk_t = B_t v_t,  dv_t = B_t^T k_t,
//   dS_0 = exp(g_1) B_1,    dg_t = <exp(g_t) S_{t-1}, B_t>.
// dq is this recurrence with the roles (read do, write v, value k), dk the
// reversed one with (read v, write do, value q), dv with (read k, write q,
// value do), so one kernel makes all three.  dg uses
//   <exp(g_t) S_{t-1}, B_t> = <S_e, exp(g_{e+1}) B_{e+1}>
//                             + sum_{t<=s<=e} (q_s . dq'_s - k_s . dk'_s),
// e being the last token of t's 64-token chunk, and dq', dk' being without the
// term of the token itself, (q_s . k_s)(do_s . v_s), which both have: they read
// the state before the write, so that for strong decays both are as small as dg
// and nothing cancels.  The dq pass leaves S_e of every chunk in the workspace
// and the dk pass takes the product with its own state there, so the sums that
// cancel are at most 64 tokens long.
//
// What bounds it: short calls (2345 tokens of 5 sequences x 8 heads, 64 x 128,
// gradient 179 us; 256 tokens x 2 heads of 64 x 64 forward 26 us; the floors of
// their bytes 7 and 0.1 us) the latency of a token group's chain: read, sum over
// the lanes, store; long ones the FMAs, two per state element and token.
#include "kda_common.cuh"
#include "kda_lin.h"
#include "kda_sm100.cuh"

namespace kda {
namespace lin {

using namespace sm100;

constexpr int kThreads = 128;
constexpr int kSub = 16;    // tokens per staged block
constexpr int kCkpt = 64;   // tokens per chunk of the gradient's dg sums

enum Mode { FWD, SUM, SUMR, DQ, DK, DV };  // SUMR: the reversed summary

template <int M> struct ModeOf {
    static constexpr bool rev = M == SUMR || M == DK || M == DV;
    static constexpr bool sum = M == SUM || M == SUMR;
    static constexpr bool out = !sum;
    static constexpr bool xd = M == DQ || M == DK;
};

template <int DA, int DB, int M>
struct Stage {  // one block of 16 tokens
    float wr[kSub][DA];
    float val[kSub][DB];
    float rd[ModeOf<M>::out ? kSub : 1][ModeOf<M>::out ? DA : 8];
    float ext[ModeOf<M>::xd ? kSub : 1][ModeOf<M>::xd ? DB : 8];
};
// CTAs per SM (by registers: the state takes DA DB / 128 of each thread's) and
// blocks in flight: what their shared memory has room for, up to four.
template <int DA, int DB> constexpr int kCtas = DA * DB > 128 * 64 ? 2 : 3;
template <int DA, int DB, int M>
struct Smem {
    static constexpr int room = 216 * 1024 / kCtas<DA, DB> / (int)sizeof(Stage<DA, DB, M>);
    static constexpr int stages = room < 4 ? room : 4;
    static_assert(stages >= 2, "blocks in flight");
    alignas(16) Stage<DA, DB, M> st[stages];
    float g[stages][kSub];
    float xp[kCkpt][4];  // per token and warp: partial out . ext
    float xq[kCkpt];
    float fdot[4];
};

KDA_DEVICE float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

template <int DA, int DB, int M>
KDA_DEVICE void rec_body(const Params &p, unsigned char *smem_raw) {
    using T = float;
    using MO = ModeOf<M>;
    constexpr int CGW = DB / 16;        // column groups (of 4) per warp
    constexpr int RG = 32 / CGW;        // row groups
    constexpr int RT = DA / RG;         // rows per thread
    constexpr int NQ = RT / 4;          // in quads: quad i is rows 4 (i RG + rg) .. + 3
    static_assert(NQ >= 1 && CGW * 4 * 4 == DB, "tile shape");
    Smem<DA, DB, M> &sm = *reinterpret_cast<Smem<DA, DB, M> *>(smem_raw);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rg = lane / CGW;
    const int col0 = (warp * CGW + lane % CGW) * 4;
    const int h = blockIdx.x, w = blockIdx.y;
    const int H = p.H;
    if (h == 0 && w == 0 && tid < 3 && p.clear_err) p.err[tid] = 0;  // no wait here can give up
    const Window wd = window_of(p, w, reinterpret_cast<int *>(&sm.fdot[0]));
    const int t0 = wd.t0, t1 = wd.t1, lo = wd.lo;
    let_next_start();
    after_previous();
    const int hr = MO::out ? h / p.rd_div : 0, Hr = MO::out ? H / p.rd_div : 1;
    const int hw = h / p.wr_div, Hw = H / p.wr_div;
    const int hv = h / p.val_div, Hv = H / p.val_div;
    const int he = MO::xd ? h / p.ext_div : 0, He = MO::xd ? H / p.ext_div : 1;
    const T *rd = (const T *)p.rd, *wr = (const T *)p.wr, *val = (const T *)p.val, *ext = (const T *)p.ext;

    float s[NQ][4][4];  // quad, row, column: S / e^G

    auto row_of = [&](int i, int r) { return 4 * (i * RG + rg) + r; };
    // state element access of a [DA][DB] matrix, or its transpose
    auto load_state = [&](const float *base, bool transposed) {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                if (base && !transposed) {
                    const float4 v4 = *reinterpret_cast<const float4 *>(base + (size_t)row_of(i, r) * DB + col0);
                    x[0] = v4.x; x[1] = v4.y; x[2] = v4.z; x[3] = v4.w;
                } else if (base) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) x[c] = base[(size_t)(col0 + c) * DA + row_of(i, r)];
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) s[i][r][c] = x[c];
            }
    };
    auto store_state = [&](float *base, bool transposed, float f) {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float x[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) x[c] = f * s[i][r][c];
                if (!transposed) {
                    *reinterpret_cast<float4 *>(base + (size_t)row_of(i, r) * DB + col0) = make_float4(x[0], x[1], x[2], x[3]);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) base[(size_t)(col0 + c) * DA + row_of(i, r)] = x[c];
                }
            }
    };
    auto scale_state = [&](float f) {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[i][r][c] *= f;
    };
    auto load_g = [&](int t) -> float {
        return clamp_g(((const float *)p.g)[p.g_per_head ? (size_t)h : (size_t)t * H + h]);
    };

    // tokens [a, b) of sequence n, whose true range is [qa, qb)
    float gamma = 1.f;
    auto run_segment = [&](int n, int a, int b, int qa, int qb) {
        const int len = b - a;
        const int nsub = (len + kSub - 1) / kSub;
        auto stage = [&](int sb, int buf) {
            const int base = a + sb * kSub, rows = min(kSub, b - base);
            Stage<DA, DB, M> &S = sm.st[buf];
            auto copy = [&](T *dst, const T *src, int D, int Hx, int hx) {
                const int per = D * (int)sizeof(T) / 16;
                for (int x = tid; x < rows * per; x += kThreads) {
                    const int r = x / per, c = x % per;
                    cp_async16((char *)(dst + r * D) + c * 16,
                               (const char *)(src + ((size_t)(base + r) * Hx + hx) * D) + c * 16, true);
                }
            };
            copy(&S.wr[0][0], wr, DA, Hw, hw);
            copy(&S.val[0][0], val, DB, Hv, hv);
            if constexpr (MO::out) copy(&S.rd[0][0], rd, DA, Hr, hr);
            if constexpr (MO::xd) copy(&S.ext[0][0], ext, DB, He, he);
            if (tid < kSub) {  // (clamped when used)
                const int t = base + tid + (MO::rev ? 1 : 0);
                const bool on = tid < rows && (!MO::rev || t < qb);
                const float *src = (const float *)p.g + (!on ? 0 : p.g_per_head ? (size_t)h : (size_t)t * H + h);
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem_u32(&sm.g[buf][tid])), "l"(src),
                             "r"(on ? 4 : 0)
                             : "memory");
            }
            cp_async_commit();
        };
        constexpr int NS = Smem<DA, DB, M>::stages;
        // a group per block, empty behind the last, so that the wait counts alike
        auto ahead = [&](int it) {
            if (it < nsub) stage(MO::rev ? nsub - 1 - it : it, it % NS);
            else cp_async_commit();
        };
        for (int it = 0; it < NS - 1; ++it) ahead(it);
        for (int it = 0; it < nsub; ++it) {
            const int sb = MO::rev ? nsub - 1 - it : it, buf = it % NS;
            ahead(it + NS - 1);
            cp_async_wait<NS - 1>();
            __syncthreads();
            const Stage<DA, DB, M> &S = sm.st[buf];
            const int base = a + sb * kSub, rows = min(kSub, b - base);
            const int chunk = sb / (kCkpt / kSub);
            const int in_chunk = (sb % (kCkpt / kSub)) * kSub;
            const int chunk_len = min(kCkpt, len - chunk * kCkpt);
            const size_t slot = (size_t)((a + chunk * kCkpt) / kCkpt + n) * H + h;
            if constexpr (M == DK) {
                if (in_chunk + rows == chunk_len) {  // the chunk's last token comes first
                    const float *ck = (const float *)p.ckpt + slot * (DA * DB);
                    float d = 0.f;
#pragma unroll
                    for (int i = 0; i < NQ; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float4 v4 = *reinterpret_cast<const float4 *>(ck + (size_t)row_of(i, r) * DB + col0);
                            const float x[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                            for (int c = 0; c < 4; ++c) d = fmaf(x[c], s[i][r][c], d);
                        }
                    d = warp_sum(d) * expf(clamp_g(sm.g[buf][rows - 1]));
                    if (lane == 0) sm.fdot[warp] = d;
                    if (tid < chunk_len) sm.xq[tid] = p.xdot[(size_t)(a + chunk * kCkpt + tid) * H + h];
                }
            }
            float G = 0.f;
            const bool hi = lane & 16, mid = lane & 8;
            const int mine = 2 * hi + mid;  // the token of a group whose output this lane ends up with
#pragma unroll 1
            for (int j0 = MO::rev ? (rows - 1) & ~3 : 0; j0 >= 0 && j0 < rows; j0 += MO::rev ? -4 : 4) {
                // in the order of the pass: token e of the group is j0 + e, or j0 + 3 - e
                float gs[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) gs[e] = clamp_g(sm.g[buf][MO::rev ? j0 + 3 - e : j0 + e]);
                const bool slow = G + ((gs[0] + gs[1]) + (gs[2] + gs[3])) < -40.f;  // the same in every thread
#pragma unroll 1
                for (int only = slow ? 0 : 3; only < 4; ++only) {  // slow: one token per round, renormalised at each
                    // (expf: exp2 of a rounded G log2 e, up to 58, would be off by 1e-6, and a write and the
                    // renormalisation behind it not by the same; 2345 tokens' gradient 176 -> 179 us)
                    float wf[4], rf[4];
                    if (slow) {
                        const float f = expf(G + (only == 0 ? gs[0] : only == 1 ? gs[1] : only == 2 ? gs[2] : gs[3]));
                        scale_state(f);
                        gamma *= f;
                        G = 0.f;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = MO::rev ? j0 + 3 - e : j0 + e;
                        const bool on = j < rows && (!slow || e == only);
                        if (!slow) G += gs[e];
                        wf[e] = on ? (slow ? 1.f : expf(-G)) * p.wr_scale : 0.f;
                        rf[e] = (slow ? 1.f : expf(G)) * p.rd_scale;
                    }
                    float o[4][4], dd[4] = {0.f, 0.f, 0.f, 0.f};  // dd: rd . wr of the token (gradient passes)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = MO::rev ? j0 + 3 - e : j0 + e;
                        const bool on = j < rows;  // (rows behind the end are not staged)
                        const float4 v4 = on ? ld4(&S.val[j][col0]) : make_float4(0.f, 0.f, 0.f, 0.f);
                        const float vs[4] = {v4.x * wf[e], v4.y * wf[e], v4.z * wf[e], v4.w * wf[e]};
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[e][c] = 0.f;
                        if (on) {
#pragma unroll
                            for (int i = 0; i < NQ; ++i) {
                                const float4 k4 = ld4(&S.wr[j][row_of(i, 0)]);
                                const float k[4] = {k4.x, k4.y, k4.z, k4.w};
                                const float4 q4 = MO::out ? ld4(&S.rd[j][row_of(i, 0)]) : k4;
                                const float q[4] = {q4.x, q4.y, q4.z, q4.w};
                                if constexpr (MO::xd) {  // read before the write
#pragma unroll
                                    for (int r = 0; r < 4; ++r) {
                                        dd[e] = fmaf(q[r], k[r], dd[e]);
#pragma unroll
                                        for (int c = 0; c < 4; ++c) o[e][c] = fmaf(q[r], s[i][r][c], o[e][c]);
                                    }
                                }
#pragma unroll
                                for (int r = 0; r < 4; ++r)
#pragma unroll
                                    for (int c = 0; c < 4; ++c) s[i][r][c] = fmaf(k[r], vs[c], s[i][r][c]);
                                if constexpr (MO::out && !MO::xd) {
#pragma unroll
                                    for (int r = 0; r < 4; ++r)
#pragma unroll
                                        for (int c = 0; c < 4; ++c) o[e][c] = fmaf(q[r], s[i][r][c], o[e][c]);
                                }
                            }
                        }
                    }
                    if constexpr (MO::out) {
                        // sums over the row groups: tokens 2 hi, 2 hi + 1, then the one of them with mid
                        float y[2][4], z[4];
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                y[e][c] = (hi ? o[2 + e][c] : o[e][c]) +
                                          __shfl_xor_sync(0xffffffffu, hi ? o[e][c] : o[2 + e][c], 16);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            z[c] = (mid ? y[1][c] : y[0][c]) + __shfl_xor_sync(0xffffffffu, mid ? y[0][c] : y[1][c], 8);
                        const float r = hi ? (mid ? rf[3] : rf[2]) : (mid ? rf[1] : rf[0]);
                        const int j = MO::rev ? j0 + 3 - mine : j0 + mine;
                        const bool on = j < rows && (!slow || mine == only);
                        const size_t at = ((size_t)(base + j) * H + h) * DB + col0;
                        float x1 = 0.f, own = 0.f;  // own: the token's write as it reads it
                        if constexpr (MO::xd) {
                            const float d0 = (hi ? dd[2] : dd[0]) + __shfl_xor_sync(0xffffffffu, hi ? dd[0] : dd[2], 16);
                            const float d1 = (hi ? dd[3] : dd[1]) + __shfl_xor_sync(0xffffffffu, hi ? dd[1] : dd[3], 16);
                            own = (mid ? d1 : d0) + __shfl_xor_sync(0xffffffffu, mid ? d0 : d1, 8);
                            if constexpr (RG == 8) own += __shfl_xor_sync(0xffffffffu, own, 4);
                            own *= p.rd_scale * p.wr_scale;
                        }
                        if constexpr (RG == 8) {
                            const bool up = lane & 4;
                            const float a0 = ((up ? z[2] : z[0]) + __shfl_xor_sync(0xffffffffu, up ? z[0] : z[2], 4)) * r;
                            const float a1 = ((up ? z[3] : z[1]) + __shfl_xor_sync(0xffffffffu, up ? z[1] : z[3], 4)) * r;
                            const int c = up ? 2 : 0;
                            if (on) {
                                float2 a = make_float2(a0, a1);
                                if constexpr (MO::xd) {
                                    const float2 e2 = *reinterpret_cast<const float2 *>(&S.ext[j][col0 + c]);
                                    const float2 v2 = *reinterpret_cast<const float2 *>(&S.val[j][col0 + c]);
                                    x1 = a.x * e2.x + a.y * e2.y;
                                    a = make_float2(fmaf(own, v2.x, a.x), fmaf(own, v2.y, a.y));
                                }
                                *reinterpret_cast<float2 *>((float *)p.out + at + c) = a;
                            }
                        } else if (on) {
                            float4 a = make_float4(z[0] * r, z[1] * r, z[2] * r, z[3] * r);
                            if constexpr (MO::xd) {
                                const float4 e4 = ld4(&S.ext[j][col0]), v4 = ld4(&S.val[j][col0]);
                                x1 = (a.x * e4.x + a.y * e4.y) + (a.z * e4.z + a.w * e4.w);
                                a = make_float4(fmaf(own, v4.x, a.x), fmaf(own, v4.y, a.y), fmaf(own, v4.z, a.z), fmaf(own, v4.w, a.w));
                            }
                            *reinterpret_cast<float4 *>((float *)p.out + at) = a;
                        }
                        if constexpr (MO::xd) {
#pragma unroll
                            for (int m = 4; m > 0; m >>= 1) x1 += __shfl_xor_sync(0xffffffffu, x1, m);
                            if (on && (lane & 7) == 0) sm.xp[in_chunk + j][warp] = x1;
                        }
                    }
                }
            }
            if (G != 0.f) {  // renormalise
                const float f = expf(G);
                scale_state(f);
                gamma *= f;
            }
            if constexpr (M == DQ) {
                if (in_chunk + rows == chunk_len) store_state((float *)p.ckpt + slot * (DA * DB), false, 1.f);
            }
            __syncthreads();
            if constexpr (M == DQ) {
                if (tid < rows) {
                    const float *x = sm.xp[in_chunk + tid];
                    p.xdot[(size_t)(base + tid) * H + h] = (x[0] + x[1]) + (x[2] + x[3]);
                }
            }
            if constexpr (M == DK) {
                if (in_chunk == 0 && warp == 0) {  // the chunk is done: suffix sums of its 64 tokens
                    const float F = (sm.fdot[0] + sm.fdot[1]) + (sm.fdot[2] + sm.fdot[3]);
                    float d[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = 2 * lane + e;
                        const float *x = sm.xp[j];
                        d[e] = j < chunk_len ? sm.xq[j] - ((x[0] + x[1]) + (x[2] + x[3])) : 0.f;
                    }
                    float tot = d[0] + d[1];  // inclusive suffix scan over the lanes
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const float y = __shfl_down_sync(0xffffffffu, tot, o);
                        if (lane + o < 32) tot += y;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = 2 * lane + e, t = a + chunk * kCkpt + j;
                        float dg = F + (e ? tot - d[0] : tot);
                        if (p.zero_first_dg && t == qa) dg = 0.f;
                        if (j < chunk_len) {
                            ((float *)p.dg)[(size_t)t * H + h] = dg;
                        }
                    }
                }
            }
        }
        __syncthreads();
    };

    auto seq_state = [&](int n) -> size_t { return ((size_t)n * H + h) * (DA * DB); };
    const size_t win_at = ((size_t)w * H + h) * (DA * DB);

    // sequence n's tokens inside the window
    auto seg_a = [&](int n) { return min(max(p.cu[n], t0), t1); };
    auto seg_b = [&](int n, int a) { return max(a, min(p.cu[n + 1], t1)); };

    if constexpr (MO::sum) {
        const int n = crossing(p, wd, MO::rev);
        if (n < 0) {
            if (tid == 0) p.gamma[(size_t)w * H + h] = kNoCarry;
            return;
        }
        const int a = seg_a(n), b = seg_b(n, a);
        const bool whole = M == SUM ? p.cu[n] >= t0 : p.cu[n + 1] <= t1;  // starts (ends) in this window
        load_state(whole && p.init ? p.init + seq_state(n) : nullptr, p.init_t);
        if (whole && p.start_copy) store_state(p.start_copy + win_at, false, 1.f);
        run_segment(n, a, b, p.cu[n], min(p.cu[n + 1], p.T));
        store_state(p.win_state + win_at, false, 1.f);
        if (tid == 0) p.gamma[(size_t)w * H + h] = whole ? kBegins : gamma;
    } else {
        const int first = wd.first, end = wd.end;
        for (int i = first; i < end; ++i) {
            const int n = MO::rev ? end - 1 - (i - first) : i;
            const int a = seg_a(n), b = seg_b(n, a);
            const bool from_win = !p.by_seq && (MO::rev ? p.cu[n + 1] > t1 : n < lo);
            const bool ends = MO::rev ? n >= lo : p.cu[n + 1] <= t1;
            if (from_win)
                load_state(p.win_state + win_at, p.win_t);
            else if (p.start_copy && p.cu[n + 1] > t1)  // its final state may replace its initial one by now
                load_state(p.start_copy + win_at, false);
            else
                load_state(p.init ? p.init + seq_state(n) : nullptr, p.init_t);
            run_segment(n, a, b, p.cu[n], min(p.cu[n + 1], p.T));
            if (ends && p.final_state) {
                const float f = MO::rev && b > a ? expf(load_g(a)) : 1.f;
                store_state(p.final_state + seq_state(n), p.init_t, f);
            }
        }
    }
}

// One pass per CTA layer, or two at once (independent ones, blockIdx.z).
template <int DA, int DB, int M>
__global__ void __launch_bounds__(kThreads, kCtas<DA, DB>) rec_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    rec_body<DA, DB, M>(p, smem_raw);
}
template <int DA, int DB, int M, int DA2, int DB2, int M2>
__global__ void __launch_bounds__(kThreads, kCtas<DA, DB>) rec_pair_kernel(const __grid_constant__ Params p, const __grid_constant__ Params p2) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    if (blockIdx.z == 0) rec_body<DA, DB, M>(p, smem_raw);
    else rec_body<DA2, DB2, M2>(p2, smem_raw);
}

// The states entering the windows, in place of the windows' Z:
// S_in(w + 1) = gamma_w S_in(w) + Z_w (reversed: S_in(w - 1)).  One thread per
// four state elements; the next kAhead windows' Z are requested before these
// are folded.
constexpr int kAhead = 8;
struct ScanSide {
    float4 *z;
    const float *gamma;
    int rev;
};
__global__ void __launch_bounds__(128) scan_kernel(const ScanSide a, const ScanSide b, int W, int H, int quads) {
    const ScanSide sd = blockIdx.z == 0 ? a : b;
    const int e = blockIdx.x * 128 + threadIdx.x, h = blockIdx.y;  // quads is a multiple of 128
    let_next_start();
    after_previous();
    float4 carry = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 zz[kAhead], nz[kAhead];
    float gm[kAhead], ng[kAhead];
    auto window = [&](int w) { return (size_t)(sd.rev ? W - 1 - w : w) * H + h; };
    auto load = [&](int w0, float4(&z)[kAhead], float(&g)[kAhead]) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (w0 + i < W) {
                g[i] = sd.gamma[window(w0 + i)];
                z[i] = sd.z[window(w0 + i) * quads + e];
            }
    };
    load(0, zz, gm);
    for (int w0 = 0; w0 < W; w0 += kAhead) {
        load(w0 + kAhead, nz, ng);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (w0 + i < W) {
                sd.z[window(w0 + i) * quads + e] = carry;
                if (gm[i] < 0.f) {
                    carry = gm[i] == kBegins ? zz[i] : make_float4(0.f, 0.f, 0.f, 0.f);
                } else {
                    carry.x = fmaf(gm[i], carry.x, zz[i].x);
                    carry.y = fmaf(gm[i], carry.y, zz[i].y);
                    carry.z = fmaf(gm[i], carry.z, zz[i].z);
                    carry.w = fmaf(gm[i], carry.w, zz[i].w);
                }
            }
            zz[i] = nz[i];
            gm[i] = ng[i];
        }
    }
}

// The forward's states, and with `rev` also the reversed pass's.
cudaError_t launch_scan(const Params &p, const Params *rev, int elems, cudaStream_t st) {
    const int quads = elems / 4;
    const ScanSide a{(float4 *)p.win_state, p.gamma, 0};
    const ScanSide b = rev ? ScanSide{(float4 *)rev->win_state, rev->gamma, 1} : a;
    return launch(scan_kernel, dim3(quads / 128, p.H, rev ? 2 : 1), 128, 0, st, true, a, b, p.W, p.H, quads);
}

template <int DA, int DB, int M>
static cudaError_t launch_one(const Params &p, cudaStream_t st, bool follows) {
    constexpr int bytes = (int)sizeof(Smem<DA, DB, M>);
    static std::atomic<uint64_t> done;
    cudaError_t e = allow_smem(done, (const void *)rec_kernel<DA, DB, M>, bytes);
    if (e != cudaSuccess) return e;
    Params q = p;
    q.clear_err = !follows;
    return launch(rec_kernel<DA, DB, M>, dim3(p.H, p.W), kThreads, bytes, st, follows, q);
}
template <int DA, int DB, int M, int DA2, int DB2, int M2>
static cudaError_t launch_two(const Params &p, const Params &p2, cudaStream_t st, bool follows) {
    constexpr int b1 = (int)sizeof(Smem<DA, DB, M>), b2 = (int)sizeof(Smem<DA2, DB2, M2>), bytes = b1 > b2 ? b1 : b2;
    static std::atomic<uint64_t> done;
    cudaError_t e = allow_smem(done, (const void *)rec_pair_kernel<DA, DB, M, DA2, DB2, M2>, bytes);
    if (e != cudaSuccess) return e;
    Params q = p;
    q.clear_err = !follows;
    return launch(rec_pair_kernel<DA, DB, M, DA2, DB2, M2>, dim3(p.H, p.W, 2), kThreads, bytes, st, follows, q, p2);
}

template <int DK_, int DV_>
static cudaError_t fwd_t(const Params &p, cudaStream_t st) {
    const bool split = p.W > 1 && !p.by_seq;
    if (split) {
        cudaError_t e = launch_one<DK_, DV_, SUM>(p, st, false);
        if (e == cudaSuccess) e = launch_scan(p, nullptr, DK_ * DV_, st);
        if (e != cudaSuccess) return e;
    }
    return launch_one<DK_, DV_, FWD>(p, st, split);
}
template <int DK_, int DV_>
static cudaError_t bwd_t(const Params &a, const Params &b, const Params &d, cudaStream_t st) {
    const bool split = a.W > 1 && !a.by_seq;
    if (split) {
        cudaError_t e = launch_two<DV_, DK_, SUM, DV_, DK_, SUMR>(a, b, st, false);
        if (e == cudaSuccess) e = launch_scan(a, &b, DK_ * DV_, st);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = launch_two<DV_, DK_, DQ, DK_, DV_, DV>(a, d, st, split);
    return e == cudaSuccess ? launch_one<DV_, DK_, DK>(b, st, true) : e;
}

// fp32: the forward (summary, scan, output), and the gradient's passes (dq, dk and dg, dv and dS0).
cudaError_t rec_forward(const Params &p, int dk, int dv, cudaStream_t st) {
    if (dk == 128) return dv == 128 ? fwd_t<128, 128>(p, st) : fwd_t<128, 64>(p, st);
    return dv == 128 ? fwd_t<64, 128>(p, st) : fwd_t<64, 64>(p, st);
}
cudaError_t rec_backward(const Params &q, const Params &k, const Params &v, int dk, int dv, cudaStream_t st) {
    if (dk == 128) return dv == 128 ? bwd_t<128, 128>(q, k, v, st) : bwd_t<128, 64>(q, k, v, st);
    return dv == 128 ? bwd_t<64, 128>(q, k, v, st) : bwd_t<64, 64>(q, k, v, st);
}

}  // namespace lin
}  // namespace kda

// Linear attention with one decay per head on the 5th-generation tensor
// cores: bf16 inputs, chunks of 128 tokens.
//
// One CTA runs the tokens of one (window, head) (kda_lin.h), chunk after
// chunk.  With c_t the log-decay summed from the chunk's first token to t,
// D[t][s] = exp(c_t - c_s) for s <= t and w_s = exp(c_last - c_s), a chunk is
//   A   = R W^T                  R: the read vectors (q), W: the write vectors (k)
//   P   = scale D (.) A          fp32 from TMEM, rounded to bf16 once, back to TMEM
//   O   = R S                    S: bf16 copy of the state entering the chunk
//   O   = scale exp(c_t) O + P V (scaled in TMEM, then added to)
//   S   = exp(c_last) S + W^T (w V)      (the decay kept aside, see carried)
// The state stays in TMEM in fp32 for the whole window.  w V is split into two
// bf16 parts (hi + lo, 2^-16 of the value), so the state that is carried and
// returned has fp32-like accuracy, but that the tensor core truncates where it
// accumulates: up to 16 x 2^-23 of the state for every chunk that it remembers
// (measured 9e-7).  P and the copy of the state that R reads are one bf16, as two
// parts would double their products (R S and P V) and the copy's 32 KB; the
// outputs, bf16 themselves, are 2.3e-3 from exact with it and 1.7e-3 by their own
// rounding alone.
// Reversed passes (the gradient) keep the tokens in their rows and flip the
// triangle: c_t is then summed from the chunk's last token back to t.
//
// The decays are never formed as exp(-c): between two 32-token blocks they
// factor into exp(c_t - c_block end) * exp(c_block end - c_s), both at most 1,
// one exponential per row and block; only the diagonal blocks need one per
// element.
//
// What bounds it: at 128 x 128 a chunk moves 128 KB through HBM, 3.0 us of one
// SM's share at 6.5 TB/s, against five 128^3 products (about 2600 tensor-pipe
// cycles, 1.4 us).  So the chunk's serial chains have to stay hidden: every
// step has its own warpgroup, one chunk apart at most, joined by mbarriers:
//   warps  0- 3  P    the decayed products           (TMEM lane = token)
//   warps  4- 7  S    the state: bf16 copy to shared memory, scaled in TMEM now and then
//   warps  8-15  V    w V as hi and lo parts, 32 tokens at a time, every group into a buffer of
//                     its own (with fewer groups this is what a chunk waits for; a summary,
//                     which has no P and O, takes their warps for it too: four groups)
//   warps 16-19  O    the outputs                    (TMEM lane = token)
//   warp  20     TMA  tiles of 128 tokens x 64 channels, 128-byte swizzle
//   warp  21     MMA  issues A and the state's products
//   warp  22     MMA  issues R S and P V, whose waits are other ones than the state's
// Shared memory (128 x 128): a ring of five tiles of 32 KB (R, W, V of the
// chunks in turn), two hi/lo buffers of 16 KB (four in a summary, with the
// place of the state's copy) and the copy of the state (32 KB).  TMEM: the state 128
// columns, A (P in its place) two buffers of 128, O 128.
//
// Measured on one B200 (6531 GB/s copied, 1653 TFLOP/s): 131072 x 32 heads of
// 128 x 128 in 1450 to 1525 us (floor 658; summary 345, scan 10, outputs 970) at
// the 1000 W cap (1.75 GHz); 30202 tokens in 8 ragged sequences x 32 heads 300 us
// (floor 119).  A chunk of the outputs' pass takes 4.3 us (its products 1.4, its
// bytes 3.0), one of a summary 2.4; on the ragged batch the tensor pipe is active
// 27% of the time and DRAM 41%.  What is
// left is the chain of a chunk: w V -> state -> its copy -> R S -> scaling ->
// P V -> O, with the waits and the code of each step.
//
// The gradient (kda_lin_rec.cu has the formulas) is three such passes: dq
// (read do, write v, value k), dk and dv reversed.  Its dg_t is the sum of
// d(log weight) over all pairs u < t <= s of an earlier and a later token.
// Summing q . dq - k . dk would cancel to nothing for short memories, at
// bf16 accuracy, so the pairs are added up as they are, without differences
// of rounded numbers:
//   both in the chunk          the dq pass has X = (q k^T) (.) P in fp32 (Q K^T is
//                              one more product) and takes row sums less column sums
//   u before the chunk         q . (the state's part of dq)      (dq pass)
//   s behind the chunk         k . (the state's part of dk)      (dk pass)
//   u before and s behind      exp(chunk) <S_in, B_in>, in fp32: the dq pass leaves the
//                              state that enters every chunk in the workspace.  (This part
//                              is the same for a chunk's 128 tokens, so a bf16 copy would
//                              not average out in the sum over the tokens.)
//
// The kernel's code is long for what an SM holds of it close by, and a warp that
// runs each instruction once per chunk (the MMA warps above all) waits for its
// code longer than for anything else; so the products are loops, the slow part of
// a wait is a call, and what a chunk does not need is kept out of its loop (with
// these three 131072 x 32 went from 1904 to 1736 us).
//
// Every wait is bounded (2 s): one that gives up marks the workspace's error
// word and the CTA, whose remaining waits then return at once; the loads and
// products in flight are waited for before TMEM is released.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "kda_common.cuh"
#include "kda_lin.h"
#include "kda_sm100.cuh"

namespace kda {
namespace lin {

cudaError_t launch_scan(const Params &p, const Params *rev, int elems, cudaStream_t st);

namespace tc {

using namespace sm100;

constexpr int kC = 128;             // tokens per chunk
constexpr int kBox = 64 * kC * 2;   // bytes of one TMA box: 64 channels x 128 tokens
constexpr int kWarps = 23;
constexpr int kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;

constexpr float kForgotten = -280.f;  // 2^-280 times the largest fp32 number is under half the smallest
constexpr int kSkipFrom = 16;         // a summary of fewer takes all (8 chunks: 79.2 us as such a call, 79.9 us with the look at the decays)

enum Mode { FWD, SUM, SUMR, DQ, DK, DV };

struct Maps {
    CUtensorMap rd, wr, val, ext;
};

constexpr int kMaxSlots = 8;  // of the ring; more would let a chunk's V arrive too early (see clean)
constexpr int kVBars = 4;     // a summary's ring of eight slots holds the V of four chunks

// A wait by parity is right only while its barrier is in the phase waited for or
// the next.  The waits on a slot's `full` are: the tile before it in the slot has
// been waited for by then (R and W by the MMA warps, which take part in every
// tile's release), and none behind it can come before the waiter has released it.
// The groups that make w V have neither: they take no part in the release, and
// where a chunk has fewer quarters than there are groups some run ahead through
// it without waiting for anything else.  So V has barriers by chunk instead,
// whose every phase each group sees, and v_seen holds back the load that would
// begin the next phase until all of them have.  (The V's slot then counts as full
// as soon as it is asked for, so that its phases go on as the ring does.)

template <bool DQ>
struct Ctl {
    unsigned long long full[kMaxSlots], free[kMaxSlots];  // the ring's slots
    unsigned long long v_full[kVBars], v_seen[kVBars];    // V of chunk c in c % kVBars
    unsigned long long a_full[2];         // A is in TMEM (two buffers)
    unsigned long long p_full[2];         // P is in TMEM, in A's place
    unsigned long long a_free[2];         // P V has read it
    unsigned long long s_full;            // the scaled state and its copy are in place
    unsigned long long vb_full[4], vb_free[4];  // the hi/lo quarters, in turn
    unsigned long long kv_done;           // the state has this chunk's writes
    unsigned long long qs_done;           // R S is in O
    unsigned long long o_scaled;          // and multiplied by its rows' decays
    unsigned long long pv_done;           // O is complete
    unsigned long long o_free;            // O has been read
    unsigned long long clean[2];          // rows behind a short chunk's end are zero (even, odd chunks)
    unsigned long long end;
    int dead;
    uint32_t tmem;
    // P: c within the 32-token block, exp(to the block's far end), block sums.  In two
    // buffers where no barrier of the warpgroup follows their last use
    alignas(16) float pc[DQ ? 1 : 2][kC], pe[DQ ? 1 : 2][kC];
    float pt[2][4];
    float ot[2][4];                        // O: block sums
    float sd[2][4];                        // DK, S: partial products with the checkpoint
    float xs[2][4];                        // DK, O: block sums
};

template <int DA, int DB, int M>
struct Cfg {
    static constexpr bool rev = M == SUMR || M == DK || M == DV;
    static constexpr bool sum = M == SUM || M == SUMR;
    static constexpr bool out = !sum;
    // Shared memory: a ring of tiles in the order in which their products are
    // done with them -- [E,] R, W, V of each chunk (W, V in a summary) -- then
    // the hi/lo buffers and the state copy
    static constexpr int tiles = sum ? 2 : M == DQ ? 4 : 3;
    static constexpr int tE = 0, tR = M == DQ ? 1 : 0, tW = sum ? 0 : tR + 1, tV = tW + 1;
    static constexpr int a_bytes = DA / 64 * kBox, b_bytes = DB / 64 * kBox;  // tiles of R, W and of V, E
    static constexpr int slot_bytes = a_bytes > b_bytes ? a_bytes : b_bytes;
    static constexpr int vb_part = DB / 64 * (32 * 128);  // 32 tokens of hi or lo
    static constexpr int vb_bytes = 2 * vb_part;
    static constexpr int groups = sum ? 4 : 2;            // warpgroups making them, a buffer each
    static constexpr int sb_bytes = out ? DB / 64 * (DA * 128) : 0;
    static constexpr int xc_bytes = M == DQ ? 10 * 32 * 4 : 0;  // DQ: column sums of X, per warp and block
    static constexpr int fit = (232448 - groups * vb_bytes - sb_bytes - xc_bytes - (int)sizeof(Ctl<M == DQ>)) / slot_bytes;
    static constexpr int slots = fit < kMaxSlots ? fit : kMaxSlots;
    // the state's products still hold W(c) when A(c + 1), issued in their middle, waits for V(c + 1)'s cleared rows
    static_assert(slots >= (M == DQ ? tiles + 1 : tiles + 2), "ring");
    static constexpr int off_vb = slots * slot_bytes;
    static constexpr int off_sb = off_vb + groups * vb_bytes;
    static constexpr int off_xc = off_sb + sb_bytes;
    static constexpr int off_ctl = off_xc + xc_bytes;
    static constexpr int bytes = off_ctl + (int)sizeof(Ctl<M == DQ>);
    // TMEM columns
    static constexpr uint32_t col_s = 0, col_a = 128, col_o = 384;  // A twice (DQ: A and Q K^T)
    static constexpr uint32_t cols = out ? 512 : 128;
};

// 32 bytes of one row: one whole sector when the address allows it
KDA_DEVICE void st_global32(void *p, const uint32_t (&r)[8], bool aligned32) {
    if (!aligned32) {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
KDA_DEVICE void ld_global32(uint4 (&r)[2], const void *p, bool aligned32) {
    if (!aligned32) {
        r[0] = reinterpret_cast<const uint4 *>(p)[0];
        r[1] = reinterpret_cast<const uint4 *>(p)[1];
        return;
    }
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0].x), "=r"(r[0].y), "=r"(r[0].z), "=r"(r[0].w), "=r"(r[1].x), "=r"(r[1].y), "=r"(r[1].z),
                   "=r"(r[1].w)
                 : "l"(p));
}
KDA_DEVICE float exp2_fast(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// inclusive scans over the lanes of a warp
KDA_DEVICE float scan_up(float x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}
KDA_DEVICE float scan_down(float x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, x, o);
        if (lane + o < 32) x += y;
    }
    return x;
}

// A wait whose first try failed: bounded, see the file comment.  Out of line, as
// the kernel's code is what its single warps wait for most (see there).
__device__ __noinline__ void slow_wait(uint32_t bar, uint32_t parity, volatile int *dead, int32_t *err) {
    if (*dead || mbar_wait(bar, parity)) return;
    *dead = 1;
    if (err) atomicOr(err + 2, 1);
}

// `n` products of K = 16 each, kept as a loop: A and B advance by the given
// bytes, and A (B) by `jump` instead after every fourth when it is K-major in
// 64-channel boxes.
struct Operand {
    uint64_t desc;
    uint32_t step;
    int32_t jump;  // 0: none
};
KDA_DEVICE Operand kmajor(uint32_t at) { return {sdesc_sw128(at, 16, 1024), 32, kBox - 96}; }
KDA_DEVICE Operand mnmajor(uint32_t at, uint32_t block) { return {sdesc_sw128(at, block, 1024), 2048, 0}; }
KDA_DEVICE void advance(Operand &o, int kk) { o.desc += (uint64_t)((o.jump && (kk & 3) == 3 ? (uint32_t)o.jump : o.step) >> 4); }
KDA_DEVICE void products(uint32_t d, Operand a, Operand b, uint32_t idesc, int n, uint32_t accumulate) {
#pragma unroll 1
    for (int kk = 0; kk < n; ++kk) {
        tc_mma_ss(d, a.desc, b.desc, idesc, accumulate);
        accumulate = 1u;
        advance(a, kk);
        advance(b, kk);
    }
}

template <int DA, int DB, int M>
__global__ void __launch_bounds__(kThreads, 1) tc_kernel(const __grid_constant__ Params p,
                                                         const __grid_constant__ Maps maps) {
    using C = Cfg<DA, DB, M>;
    extern __shared__ __align__(1024) unsigned char sm[];  // the swizzle's period
    Ctl<M == DQ> &ctl = *reinterpret_cast<Ctl<M == DQ> *>(sm + C::off_ctl);
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, role = warp >> 2;
    const int h = blockIdx.x, w = blockIdx.y, H = p.H;
    const Window wd = window_of(p, w, &ctl.dead);
    const int t0 = wd.t0, t1 = wd.t1, lo = wd.lo;
    volatile int *dead = &ctl.dead;
    if (p.by_seq) __syncthreads();  // every thread has read the shared word

    // (the first kernel of a call clears the error words, long before a wait can give up)
    if (h == 0 && w == 0 && tid < 3 && p.err && p.clear_err) p.err[tid] = 0;
    if (warp == 20 && elect_one_sync()) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.wr) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.val) : "memory");
        if (C::out) asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.rd) : "memory");
    }

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem)),
                     "r"(C::cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 32) {
        for (int i = 0; i < C::slots; ++i) {
            mbar_init(smem_u32(&ctl.full[i]), 1);
            mbar_init(smem_u32(&ctl.free[i]), 2);  // both MMA warps, or one twice
        }
        for (int i = 0; i < kVBars; ++i) {
            mbar_init(smem_u32(&ctl.v_full[i]), 1);
            mbar_init(smem_u32(&ctl.v_seen[i]), 4 * C::groups);  // their warps
        }
        for (int i = 0; i < C::groups; ++i) {
            mbar_init(smem_u32(&ctl.vb_full[i]), 128);
            mbar_init(smem_u32(&ctl.vb_free[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl.a_free[i]), 1);
            mbar_init(smem_u32(&ctl.a_full[i]), 1);
            mbar_init(smem_u32(&ctl.p_full[i]), 128);
        }
        unsigned long long *one[] = {&ctl.qs_done, &ctl.kv_done, &ctl.pv_done};
        mbar_init(smem_u32(&ctl.end), 2);
        unsigned long long *wg[] = {&ctl.s_full, &ctl.o_scaled, &ctl.o_free, &ctl.clean[0], &ctl.clean[1]};
        for (auto *b : one) mbar_init(smem_u32(b), 1);
        for (auto *b : wg) mbar_init(smem_u32(b), 128);
        ctl.dead = (sbase & 1023u) != 0;  // never: the tiles would be read wrongly
        if (ctl.dead && p.err) atomicOr(p.err + 2, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    let_next_start();
    after_previous();

    auto wait = [&](unsigned long long &bar, uint32_t parity) {
        if (!mbar_try_wait(smem_u32(&bar), parity)) slow_wait(smem_u32(&bar), parity, dead, p.err);
    };
    auto arrive = [&](unsigned long long &bar) { mbar_arrive(smem_u32(&bar)); };
    // tile j of chunk c in the ring
    auto slot = [&](int c, int j) { return (c * C::tiles + j) % C::slots; };
    auto phase = [&](int c, int j) -> uint32_t { return (uint32_t)((c * C::tiles + j) / C::slots) & 1u; };
    auto wait_v = [&](int c) { wait(ctl.v_full[c % kVBars], (uint32_t)(c / kVBars) & 1u); };
    const bf16 *gp = (const bf16 *)p.g + h;
    const uint32_t gs = p.g_per_head ? 0u : (uint32_t)H;
    auto load_g = [&](int t) -> float {  // in powers of two
        return clamp_g(__bfloat162float(gp[(size_t)(uint32_t)t * gs])) * kLog2e;
    };
    // the decay that row `row` of the chunk of `rows` tokens at `base` multiplies the running state with
    auto row_g = [&](int base, int rows, int row, int qb) -> float {
        const int t = base + row + (C::rev ? 1 : 0);
        return row < rows && (!C::rev || t < qb) ? load_g(t) : 0.f;
    };

    int first = wd.first, end = wd.end;
    if (C::sum) {
        const int n = crossing(p, wd, C::rev);
        first = n < 0 ? 0 : n;
        end = n < 0 ? 0 : n + 1;
        if (n < 0 && tid == 0) p.gamma[(size_t)w * H + h] = kNoCarry;
    }

    // A summary leaves out the tokens that the decays behind them have multiplied by less than 2^kForgotten,
    // which takes any finite fp32 state to 0: whole chunks at the pass's beginning, `last` of them staying.
    int last = 1 << 30;
    if (C::sum && first < end) {
        const int qa = p.cu[first], qb = min(p.cu[first + 1], p.T);
        const int a = min(max(qa, t0), t1), b = max(a, min(qb, t1)), nch = (b - a + kC - 1) / kC;
        constexpr int kRound = 2 * kC;  // chunks at a time; their decays in pc
        float *tot = &ctl.pc[0][0], sum = 0.f;
        for (int r0 = 0; nch >= kSkipFrom && r0 < nch && last > nch; r0 += kRound) {
            const int here = min(kRound, nch - r0);
#pragma unroll 4
            for (int x = warp; x < here; x += kWarps) {
                const int base = a + (C::rev ? r0 + x : nch - 1 - r0 - x) * kC, rows = min(kC, b - base);
                float g[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] = row_g(base, rows, 32 * e + lane, qb);
                const float t = warp_sum((g[0] + g[1]) + (g[2] + g[3]));
                if (lane == 0) tot[x] = t;
            }
            __syncthreads();
            for (int x0 = 0; x0 < here; x0 += 32) {
                const float run = sum + scan_up(x0 + lane < here ? tot[x0 + lane] : 0.f, lane);
                const unsigned gone = __ballot_sync(0xffffffffu, run < kForgotten);
                if (gone) {
                    last = r0 + x0 + __ffs(gone);
                    break;
                }
                sum = __shfl_sync(0xffffffffu, run, 31);
            }
            __syncthreads();
        }
        last = min(last, nch);
    }
    auto leave_out = [&](int &a, int &b) {
        if (C::sum && C::rev) b = min(b, a + last * kC);
        if (C::sum && !C::rev) a += ((b - a + kC - 1) / kC - last) * kC;
    };

    // f(n, a, b, qb): tokens [a, b) of sequence n, which ends at qb, in the order of the pass
    auto segments = [&](auto f) {
        for (int i = first; i < end; ++i) {
            const int n = C::rev ? end - 1 - (i - first) : i;
            const int qa = p.cu[n], qb = min(p.cu[n + 1], p.T);
            int a = min(max(qa, t0), t1), b = max(a, min(qb, t1));
            leave_out(a, b);
            f(n, a, b, qa, qb);
        }
    };
    // f(base, rows): its chunks
    auto chunks = [&](int a, int b, auto f) {
        const int nch = (b - a + kC - 1) / kC;
        for (int i = 0; i < nch; ++i) {
            const int base = a + (C::rev ? nch - 1 - i : i) * kC;
            f(base, min(kC, b - base), i, nch);
        }
    };
    auto next_base = [&](int base) { return C::rev ? base - kC : base + kC; };

    // The state in TMEM is S / 2^G: its decay is kept in G (every role that needs it computes the same) and
    // multiplied in only when G would fall below -24, so most chunks leave the accumulator where it is.
    // carried: G behind a chunk with the decays gx (row 32 x + lane in gx[x]); 0 when it is multiplied in.
    auto chunk_sum = [&](const float(&gx)[4]) { return warp_sum((gx[0] + gx[1]) + (gx[2] + gx[3])); };
    auto carried = [&](float G, const float(&gx)[4]) {
        const float g = G + chunk_sum(gx);
        return g < -24.f ? 0.f : g;
    };

    int it = 0;  // chunks done by this role
    if (C::out && role == 0) {
        // --------------------------------------------------------------- P
        {
            const int row = tid;  // 32 * warp + lane
            const uint32_t ta0 = tmem + ((uint32_t)(32 * warp) << 16) + C::col_a;
            const float sc = p.rd_scale * p.wr_scale;
            segments([&](int n, int a, int b, int qa, int qb) {
                float gx = 0.f;
                chunks(a, b, [&](int base, int rows, int i, int nch) {
                    if (i == 0) gx = row_g(base, rows, row, qb);
                    const int pb = M == DQ ? 0 : it & 1;
                    const float c = C::rev ? scan_down(gx, lane) : scan_up(gx, lane);
                    const float tot = __shfl_sync(0xffffffffu, c, C::rev ? 0 : 31);
                    ctl.pc[pb][row] = c;
                    ctl.pe[pb][row] = exp2f(tot - c);
                    if (lane == 0) ctl.pt[pb][warp] = tot;
                    if (i + 1 < nch) gx = row_g(next_base(base), min(kC, b - next_base(base)), row, qb);
                    bar_sync(1, 128);
                    const int ab = M == DQ ? 0 : it & 1;
                    const uint32_t ta = ta0 + 128 * ab;
                    wait(ctl.a_full[ab], (M == DQ ? it : it >> 1) & 1);
                    tc_fence_after();
                    float xr = 0.f;  // DQ: this row's sum of X over earlier tokens
                    float *xc = reinterpret_cast<float *>(sm + C::off_xc) + 16 * warp * (warp + 1);  // blocks 0 .. warp
                    // block by block upwards: P's block lies in columns 16 blk .. + 15, which hold products of
                    // block blk / 2, read by then or not needed by this warp
#pragma unroll 1
                    for (int blk = 0; blk < 4; ++blk) {
                        uint32_t pk[16];
                        if (C::rev ? blk < warp : blk > warp) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) pk[e] = 0u;
                        } else {
                            uint32_t r[32];
                            uint32_t y[M == DQ ? 32 : 1];
                            if constexpr (M == DQ) tmem_ld32(ta + 128 + 32 * blk, y);
                            tmem_ld32_wait(ta + 32 * blk, r);
                            if (blk == warp) {
#pragma unroll
                                for (int e4 = 0; e4 < 8; ++e4) {
                                    const float4 cs = *reinterpret_cast<const float4 *>(&ctl.pc[pb][32 * blk + 4 * e4]);
                                    const float cc[4] = {cs.x, cs.y, cs.z, cs.w};
                                    float v[4];
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const int s = 4 * e4 + e;
                                        const bool on = C::rev ? s >= lane : s <= lane;
                                        v[e] = on ? __uint_as_float(r[s]) * (exp2_fast(c - cc[e]) * sc) : 0.f;
                                    }
                                    pk[2 * e4] = pack_bf16(v[0], v[1]);
                                    pk[2 * e4 + 1] = pack_bf16(v[2], v[3]);
                                    if constexpr (M == DQ) {
#pragma unroll
                                        for (int e = 0; e < 4; ++e) {
                                            const int s = 4 * e4 + e;
                                            y[s] = __float_as_uint(s < lane ? v[e] * __uint_as_float(y[s]) : 0.f);
                                        }
                                    }
                                }
                            } else {
                                float far = c;  // + the blocks between
                                for (int j = min(blk, warp) + 1; j < max(blk, warp); ++j) far += ctl.pt[pb][j];
                                const float f = exp2f(far) * sc;
                                const float2 f2 = make_float2(f, f);
#pragma unroll
                                for (int e4 = 0; e4 < 8; ++e4) {
                                    const float4 es = *reinterpret_cast<const float4 *>(&ctl.pe[pb][32 * blk + 4 * e4]);
                                    const float2 v0 = f2mul(f2mul(make_float2(es.x, es.y), f2),
                                                            make_float2(__uint_as_float(r[4 * e4]), __uint_as_float(r[4 * e4 + 1])));
                                    const float2 v1 = f2mul(f2mul(make_float2(es.z, es.w), f2),
                                                            make_float2(__uint_as_float(r[4 * e4 + 2]), __uint_as_float(r[4 * e4 + 3])));
                                    pk[2 * e4] = pack_bf16(v0);
                                    pk[2 * e4 + 1] = pack_bf16(v1);
                                    if constexpr (M == DQ) {
                                        y[4 * e4] = __float_as_uint(v0.x * __uint_as_float(y[4 * e4]));
                                        y[4 * e4 + 1] = __float_as_uint(v0.y * __uint_as_float(y[4 * e4 + 1]));
                                        y[4 * e4 + 2] = __float_as_uint(v1.x * __uint_as_float(y[4 * e4 + 2]));
                                        y[4 * e4 + 3] = __float_as_uint(v1.y * __uint_as_float(y[4 * e4 + 3]));
                                    }
                                }
                            }
                            if constexpr (M == DQ) {
                                // rows behind the end hold other tokens
#pragma unroll
                                for (int half = 0; half < 2; ++half) {
                                    float v[16];
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        v[e] = row < rows ? __uint_as_float(y[16 * half + e]) : 0.f;
                                        xr += v[e];
                                    }
                                    const float cs = warp_sum16_scatter(v, lane);
                                    if (!(lane & 1)) xc[32 * blk + 16 * half + row_of_lane(lane)] = cs;
                                }
                            }
                        }
                        tmem_st16(ta + 16 * blk, pk);
                    }
                    tc_wait_st();
                    tc_fence_before();
                    arrive(ctl.p_full[ab]);
                    if constexpr (M == DQ) {
                        // pairs (s, u), u < s, whose later token is this row less those whose earlier one is
                        bar_sync(1, 128);
                        const float *all = reinterpret_cast<const float *>(sm + C::off_xc);
                        for (int j = warp; j < 4; ++j) xr -= all[16 * j * (j + 1) + row];
                        if (row < rows) p.xdot[(size_t)(base + row) * H + h] = xr;
                    }
                    ++it;
                });
            });
        }
    } else if (role == 1) {
        // --------------------------------------------------------------- S
        const int row = tid - 128, wl = warp & 3;
        const uint32_t ts = tmem + ((uint32_t)(32 * wl) << 16) + C::col_s;
        const bool mine = row < DA;
        float gamma = 1.f;
        segments([&](int n, int a, int b, int qa, int qb) {
            const bool from_win = !p.by_seq && (C::rev ? p.cu[n + 1] > t1 : n < lo);
            const bool ends = C::rev ? n >= lo : p.cu[n + 1] <= t1;
            const size_t win_at = ((size_t)w * H + h) * (DA * DB), seq_at = ((size_t)n * H + h) * (DA * DB);
            const float *src;
            bool src_t = false;
            if (C::sum) {
                src = from_win ? nullptr : p.init ? p.init + seq_at : nullptr;
                src_t = p.init_t;
            } else if (from_win) {
                src = p.win_state + win_at;
                src_t = p.win_t;
            } else if (p.start_copy && p.cu[n + 1] > t1) {
                src = p.start_copy + win_at;
            } else {
                src = p.init ? p.init + seq_at : nullptr;
                src_t = p.init_t;
            }
            // the state's start to TMEM (the previous segment's products are complete)
            if (mine) {
#pragma unroll 1
                for (int cb = 0; cb < DB / 32; ++cb) {
                    uint32_t r[32];
                    if (!src) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = 0u;
                    } else if (!src_t) {
#pragma unroll
                        for (int e4 = 0; e4 < 8; ++e4) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(src + (size_t)row * DB + 32 * cb + 4 * e4);
                            r[4 * e4] = v.x; r[4 * e4 + 1] = v.y; r[4 * e4 + 2] = v.z; r[4 * e4 + 3] = v.w;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(src[(size_t)(32 * cb + e) * DA + row]);
                    }
                    tmem_st32(ts + 32 * cb, r);
                    if (C::sum && p.start_copy && !from_win) {
                        float *dst = p.start_copy + win_at + (size_t)row * DB + 32 * cb;
#pragma unroll
                        for (int e4 = 0; e4 < 8; ++e4)
                            reinterpret_cast<uint4 *>(dst)[e4] = make_uint4(r[4 * e4], r[4 * e4 + 1], r[4 * e4 + 2], r[4 * e4 + 3]);
                    }
                }
                tc_wait_st();
            }
            float gx[4] = {0.f, 0.f, 0.f, 0.f}, G = 0.f;
            chunks(a, b, [&](int base, int rows, int i, int nch) {
                if (i == 0)
#pragma unroll
                    for (int x = 0; x < 4; ++x) gx[x] = row_g(base, rows, 32 * x + lane, qb);
                const float total = chunk_sum(gx), f = exp2f(total), before = exp2f(G);
                G = carried(G, gx);
                const bool fold = G == 0.f && total < 0.f;  // multiply the decays so far and this chunk's in
                gamma *= f;
                if (i + 1 < nch)
#pragma unroll
                    for (int x = 0; x < 4; ++x) gx[x] = row_g(next_base(base), min(kC, b - next_base(base)), 32 * x + lane, qb);
                float *ck = nullptr;
                // four columns of all rows, then the next four: a warp's 16-byte accesses are 512 bytes in a row
                if (M == DQ || M == DK) ck = (float *)p.ckpt + (((size_t)(base / kC + n)) * H + h) * (DA * DB) + 4 * row;
                float4 cv[M == DK ? 4 : 1];  // DK: 16 columns of the checkpoint, requested one round ahead
                if (M == DK && mine)
#pragma unroll
                    for (int e = 0; e < (M == DK ? 4 : 0); ++e) cv[e] = *reinterpret_cast<const float4 *>(ck + 4 * DA * e);
                if (i > 0) {
                    wait(ctl.kv_done, (it - 1) & 1);
                    if (C::out) wait(ctl.qs_done, (it - 1) & 1);  // the copy has been read
                    tc_fence_after();
                }
                float dot = 0.f;
                if (mine && (C::out || fold)) {
                    auto scale = [](uint32_t(&r)[32], float x) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 v = f2mul(make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), make_float2(x, x));
                            r[2 * e] = __float_as_uint(v.x);
                            r[2 * e + 1] = __float_as_uint(v.y);
                        }
                    };
#pragma unroll 1
                    for (int cb = 0; cb < DB / 32; ++cb) {
                        uint32_t r[32];
                        tmem_ld32_wait(ts + 32 * cb, r);
                        scale(r, before);
                        if (C::out) {  // the copy that R reads: [DA rows][64 channels] boxes, 128-byte swizzle
                            unsigned char *box = sm + C::off_sb + (cb >> 1) * (DA * 128) + row * 128;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint4 v;
                                v.x = pack_bf16(__uint_as_float(r[8 * e]), __uint_as_float(r[8 * e + 1]));
                                v.y = pack_bf16(__uint_as_float(r[8 * e + 2]), __uint_as_float(r[8 * e + 3]));
                                v.z = pack_bf16(__uint_as_float(r[8 * e + 4]), __uint_as_float(r[8 * e + 5]));
                                v.w = pack_bf16(__uint_as_float(r[8 * e + 6]), __uint_as_float(r[8 * e + 7]));
                                *reinterpret_cast<uint4 *>(box + ((((cb & 1) * 4 + e) ^ (row & 7)) << 4)) = v;
                            }
                        }
                        if constexpr (M == DQ) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint4 *>(ck + DA * (32 * cb + 4 * e)) =
                                    make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
                        }
                        if constexpr (M == DK) {
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const int at = 32 * cb + 16 * half;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float4 v = cv[e];
                                    if (at + 16 < DB) cv[e] = *reinterpret_cast<const float4 *>(ck + DA * (at + 16 + 4 * e));
                                    dot = fmaf(v.x, __uint_as_float(r[16 * half + 4 * e]), dot);
                                    dot = fmaf(v.y, __uint_as_float(r[16 * half + 4 * e + 1]), dot);
                                    dot = fmaf(v.z, __uint_as_float(r[16 * half + 4 * e + 2]), dot);
                                    dot = fmaf(v.w, __uint_as_float(r[16 * half + 4 * e + 3]), dot);
                                }
                            }
                        }
                        if (fold) {
                            scale(r, f);
                            tmem_st32(ts + 32 * cb, r);
                        }
                    }
                    tc_wait_st();
                }
                if (C::out) fence_async_smem();
                tc_fence_before();
                arrive(ctl.s_full);
                if constexpr (M == DK) {
                    // pairs whose tokens lie on either side of the chunk: the same for its every token
                    dot = warp_sum(dot);
                    if (lane == 0) ctl.sd[it & 1][wl] = dot;
                    bar_sync(3, 128);
                    if (row < rows) {
                        const float *d = ctl.sd[it & 1];
                        p.across[(size_t)(base + row) * H + h] = ((d[0] + d[1]) + (d[2] + d[3])) * f * exp2f(load_g(base));
                    }
                }
                ++it;
            });
            // the state behind the segment
            float *dst = C::sum ? p.win_state + win_at : ends && p.final_state ? p.final_state + seq_at : nullptr;
            const bool dst_t = !C::sum && p.init_t;
            if (b > a) {
                wait(ctl.kv_done, (it - 1) & 1);
                if (C::out) wait(ctl.qs_done, (it - 1) & 1);
                tc_fence_after();
            }
            if (dst && mine) {
                const float f = exp2f(!C::sum && C::rev && b > a ? G + load_g(a) : G);
#pragma unroll 1
                for (int cb = 0; cb < DB / 32; ++cb) {
                    uint32_t r[32];
                    tmem_ld32_wait(ts + 32 * cb, r);
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                    if (!dst_t) {
#pragma unroll
                        for (int e4 = 0; e4 < 8; ++e4)
                            *reinterpret_cast<uint4 *>(dst + (size_t)row * DB + 32 * cb + 4 * e4) =
                                make_uint4(r[4 * e4], r[4 * e4 + 1], r[4 * e4 + 2], r[4 * e4 + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) dst[(size_t)(32 * cb + e) * DA + row] = __uint_as_float(r[e]);
                    }
                }
            }
            if (C::sum && row == 0) p.gamma[(size_t)w * H + h] = from_win ? gamma : kBegins;
        });
        tc_fence_before();
    } else if (role == 2 || role == 3 || (C::sum && role < 5)) {
        // --------------------------------------------------------------- V (each group every NG-th quarter)
        constexpr int NG = C::groups;
        const int grp = NG == 2 ? role - 2 : role == 0 ? 0 : role - 1, wl = warp & 3;
        int quarters = 0;
        float G = 0.f;
        segments([&](int n, int a, int b, int qa, int qb) {
            float gx[4] = {0.f, 0.f, 0.f, 0.f};
            chunks(a, b, [&](int base, int rows, int i, int nch) {
                if (i == 0)
#pragma unroll
                    for (int x = 0; x < 4; ++x) gx[x] = row_g(base, rows, 32 * x + lane, qb);
                const int nq = (rows + 31) / 32;
                if (i == 0) G = 0.f;
                G = carried(G, gx);
                // this group's quarters: f0, f0 + NG; the decays behind their rows, in the order of the pass
                const int f0 = (grp - quarters) & (NG - 1);
                float wq[4 / NG];
                {
                    float tot[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) tot[x] = warp_sum(gx[x]);
#pragma unroll
                    for (int e = 0; e < 4 / NG; ++e) {
                        const float g1 = NG == 2 ? (f0 ? gx[2 * e + 1] : gx[2 * e])
                                                 : f0 == 0 ? gx[0] : f0 == 1 ? gx[1] : f0 == 2 ? gx[2] : gx[3];
                        const float inc = C::rev ? scan_up(g1, lane) : scan_down(g1, lane);
                        float exc = C::rev ? __shfl_up_sync(0xffffffffu, inc, 1) : __shfl_down_sync(0xffffffffu, inc, 1);
                        if (lane == (C::rev ? 0 : 31)) exc = 0.f;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (C::rev ? j < f0 + NG * e : j > f0 + NG * e) exc += tot[j];
                        wq[e] = exp2f(exc - G) * p.wr_scale;
                    }
                }
                if (i + 1 < nch)
#pragma unroll
                    for (int x = 0; x < 4; ++x) gx[x] = row_g(next_base(base), min(kC, b - next_base(base)), 32 * x + lane, qb);
                unsigned char *tw = sm + slot(it, C::tW) * C::slot_bytes, *tv = sm + slot(it, C::tV) * C::slot_bytes;
                wait_v(it);
                __syncwarp();
                if (lane == 0) arrive(ctl.v_seen[it % kVBars]);
                if (rows < kC && ((quarters + nq - 1) & (NG - 1)) == grp) {
                    // The last quarter's rows behind the end hold other tokens: zero, whatever they are (the
                    // quarters behind it are not read); each thread the channels that it reads below.  Both MMA
                    // warps have passed their wait for the short chunk two before this one, if that was one:
                    // this chunk's V lies in a slot (of kMaxSlots at most) whose last tile they released behind it.
                    wait(ctl.full[slot(it, C::tW)], phase(it, C::tW));
                    const int r = 32 * (nq - 1) + lane;
                    if (r >= rows) {
                        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                        for (int c0 = 0; c0 < DA / 32; ++c0) {
                            const int c = wl * (DA / 32) + c0;
                            *reinterpret_cast<uint4 *>(tw + (c >> 3) * kBox + r * 128 + (c & 7) * 16) = z;
                        }
#pragma unroll
                        for (int c0 = 0; c0 < DB / 32; ++c0) {
                            const int c = wl * (DB / 32) + c0;
                            *reinterpret_cast<uint4 *>(tv + (c >> 3) * kBox + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = z;
                        }
                    }
                    fence_async_smem();
                    arrive(ctl.clean[it & 1]);
                }
                // 32 tokens at a time: lane = token, warp = quarter of the channels
                for (int qq = 0; qq < nq; ++qq, ++quarters) {
                    const int vb = quarters & (NG - 1);
                    if (vb != grp) continue;
                    if (quarters >= NG) wait(ctl.vb_free[vb], (quarters / NG - 1) & 1);
                    const int r = 32 * qq + lane;
                    const float f = qq < NG ? wq[0] : wq[4 / NG - 1];
                    const float2 f2 = make_float2(f, f);
                    constexpr int CH = DB / 32;  // 16-byte pieces
#pragma unroll
                    for (int c0 = 0; c0 < CH; ++c0) {
                        const int c = wl * CH + c0, box = c >> 3, off = ((c & 7) ^ (lane & 7)) << 4;
                        const uint4 x = *reinterpret_cast<const uint4 *>(tv + box * kBox + r * 128 + off);
                        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                        uint32_t hi[4], lw[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 v = f2mul(unpack_bf16(xs[e]), f2);
                            hi[e] = pack_bf16(v);
                            const float2 k2 = unpack_bf16(hi[e]);
                            lw[e] = pack_bf16(f2fma(k2, make_float2(-1.f, -1.f), v));
                        }
                        unsigned char *dst = sm + C::off_vb + vb * C::vb_bytes + box * 4096 + lane * 128 + off;
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4 *>(dst + C::vb_part) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
                    }
                    fence_async_smem();
                    arrive(ctl.vb_full[vb]);
                }
                ++it;
            });
        });
    } else if (role == 4) {
        // --------------------------------------------------------------- O
        if (C::out) {
            const int row = tid - 512, wl = warp & 3;
            const uint32_t lane_off = (uint32_t)(32 * wl) << 16;
            const bool al32 = ((uintptr_t)p.out & 31) == 0;
            const uint32_t to = tmem + lane_off + C::col_o;
            segments([&](int n, int a, int b, int qa, int qb) {
                float gx = 0.f;
                chunks(a, b, [&](int base, int rows, int i, int nch) {
                    if (i == 0) gx = row_g(base, rows, row, qb);
                    const int pb = it & 1;
                    float c = C::rev ? scan_down(gx, lane) : scan_up(gx, lane);
                    if (lane == (C::rev ? 0 : 31)) ctl.ot[pb][wl] = c;
                    if (i + 1 < nch) gx = row_g(next_base(base), min(kC, b - next_base(base)), row, qb);
                    bar_sync(2, 128);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (C::rev ? j > wl : j < wl) c += ctl.ot[pb][j];
                    const float f = exp2f(c) * p.rd_scale;
                    // the state's part, scaled by its rows' decays before P V is added to it
                    const size_t at = ((size_t)(base + row) * H + h) * DB;
                    const float2 f2 = make_float2(f, f);
                    float xi = 0.f;  // gradient passes: the state's part of out . ext
                    constexpr bool XD = M == DQ || M == DK;
                    const bool ext32 = ((uintptr_t)p.ext & 31) == 0;
                    uint4 e4[XD ? 2 : 1][2];  // 32 channels of ext, requested one round ahead
                    auto load_ext = [&](int cb) {
                        const bf16 *src =
                            (const bf16 *)p.ext + ((size_t)(base + row) * (H / p.ext_div) + h / p.ext_div) * DB + 32 * cb;
                        if (XD && row < rows)
#pragma unroll
                            for (int e = 0; e < (XD ? 2 : 0); ++e) ld_global32(e4[e], src + 16 * e, ext32);
                    };
                    if (XD) {
#pragma unroll
                        for (int e = 0; e < (XD ? 4 : 0); ++e) e4[e >> 1][e & 1] = make_uint4(0u, 0u, 0u, 0u);
                        load_ext(0);
                    }
                    wait(ctl.qs_done, it & 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int cb = 0; cb < DB / 32; ++cb) {
                        uint32_t x[32];
                        tmem_ld32_wait(to + 32 * cb, x);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 v = f2mul(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), f2);
                            x[2 * e] = __float_as_uint(v.x);
                            x[2 * e + 1] = __float_as_uint(v.y);
                        }
                        tmem_st32(to + 32 * cb, x);
                        if constexpr (XD) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint4 u4 = e4[e >> 1][e & 1];
                                const uint32_t es[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const float2 u = unpack_bf16(es[k]);
                                    xi = fmaf(u.x, __uint_as_float(x[8 * e + 2 * k]), xi);
                                    xi = fmaf(u.y, __uint_as_float(x[8 * e + 2 * k + 1]), xi);
                                }
                            }
                            if (cb + 1 < DB / 32) load_ext(cb + 1);
                        }
                    }
                    tc_wait_st();
                    tc_fence_before();
                    arrive(ctl.o_scaled);
                    wait(ctl.pv_done, it & 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int cb = 0; cb < DB / 32; ++cb) {
                        uint32_t x[32];
                        tmem_ld32_wait(to + 32 * cb, x);
                        if (cb == DB / 32 - 1) {
                            tc_fence_before();
                            arrive(ctl.o_free);
                        }
                        if (row < rows) {
                            if ((M == DQ || M == DK) && p.out_f32) {
                                float *dst = (float *)p.out + at + 32 * cb;
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const uint32_t v[8] = {x[8 * q], x[8 * q + 1], x[8 * q + 2], x[8 * q + 3],
                                                           x[8 * q + 4], x[8 * q + 5], x[8 * q + 6], x[8 * q + 7]};
                                    st_global32(dst + 8 * q, v, al32);
                                }
                            } else {
                                bf16 *dst = (bf16 *)p.out + at + 32 * cb;
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    uint32_t v[8];
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        v[e] = pack_bf16(__uint_as_float(x[16 * q + 2 * e]), __uint_as_float(x[16 * q + 2 * e + 1]));
                                    st_global32(dst + 16 * q, v, al32);
                                }
                            }
                        }
                    }
                    if constexpr (M == DQ) {
                        if (row < rows) p.xstate[(size_t)(base + row) * H + h] = xi;
                    }
                    if constexpr (M == DK) {
                        // dg but for the pairs across the chunk: the pairs inside it and those with an
                        // earlier state from this token on, those with a later state before it
                        float u = 0.f;
                        const size_t th = (size_t)(base + row) * H + h;
                        if (row < rows) u = p.xdot[th] + p.xstate[th];
                        const float ik = row < rows ? xi : 0.f;
                        float suf = scan_down(u, lane), pre = scan_up(ik, lane) - ik;
                        if (lane == 0) ctl.xs[0][wl] = suf;
                        if (lane == 31) ctl.xs[1][wl] = pre + ik;
                        bar_sync(2, 128);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (j > wl) suf += ctl.xs[0][j];
                            if (j < wl) pre += ctl.xs[1][j];
                        }
                        if (row < rows) p.xstate[th] = p.zero_first_dg && base + row == qa ? 0.f : suf + pre;
                    }
                    ++it;
                });
            });
        }
    } else if (warp == 20) {
        // --------------------------------------------------------------- TMA
        const int hr = C::out ? h / p.rd_div : 0, hw = h / p.wr_div, hv = h / p.val_div, he = M == DQ ? h / p.ext_div : 0;
        segments([&](int n, int a, int b, int qa, int qb) {
            chunks(a, b, [&](int base, int rows, int i, int nch) {
                auto load = [&](int j, const CUtensorMap &map, int head, int boxes) {
                    const int sl = slot(it, j), vb = it % kVBars;
                    if (it * C::tiles + j >= C::slots) wait(ctl.free[sl], phase(it, j) ^ 1u);
                    if (j == C::tV && it >= kVBars) wait(ctl.v_seen[vb], (uint32_t)(it / kVBars - 1) & 1u);
                    if (elect_one_sync() && !*dead) {
                        const uint32_t bar = smem_u32(j == C::tV ? &ctl.v_full[vb] : &ctl.full[sl]), dst = sbase + sl * C::slot_bytes;
                        mbar_arrive_expect_tx(bar, boxes * kBox);
                        if (j == C::tV) arrive(ctl.full[sl]);
                        for (int x = 0; x < boxes; ++x) {
                            tma_load_3d(dst + x * kBox, &map, 64 * x, head, base, bar);
                            if (i + 1 < nch) tma_prefetch_3d(&map, 64 * x, head, next_base(base));
                        }
                    }
                    __syncwarp();
                };
                if (M == DQ) load(C::tE, maps.ext, he, DB / 64);
                if (C::out) load(C::tR, maps.rd, hr, DA / 64);
                load(C::tW, maps.wr, hw, DA / 64);
                load(C::tV, maps.val, hv, DB / 64);
                if (M == DK && i + 1 < nch && elect_one_sync()) {  // the next chunk's ext and checkpoint to L2
#pragma unroll
                    for (int x = 0; x < DB / 64; ++x) tma_prefetch_3d(&maps.ext, 64 * x, h / p.ext_div, next_base(base));
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"((const float *)p.ckpt +
                                     ((size_t)(next_base(base) / kC + n) * H + h) * (DA * DB)),
                                 "r"((uint32_t)(DA * DB * 4))
                                 : "memory");
                }
                __syncwarp();
                ++it;
            });
        });
        // nothing in flight arrives behind the CTA's end: the last products' arrivals, the last of which are
        // their tiles' releases, and, when a wait gave up, the loads (bounded)
        for (int x = max(0, it * C::tiles - C::slots); x < it * C::tiles; ++x)
            wait(ctl.free[x % C::slots], (uint32_t)(x / C::slots) & 1u);
        if (*dead)
            for (int x = max(0, it * C::tiles - C::slots); x < it * C::tiles; ++x) {
                const int c = x / C::tiles;
                if (x % C::tiles == C::tV) mbar_wait(smem_u32(&ctl.v_full[c % kVBars]), (uint32_t)(c / kVBars) & 1u);
                else mbar_wait(smem_u32(&ctl.full[x % C::slots]), (uint32_t)(x / C::slots) & 1u);
            }
    } else {
        // --------------------------------------------------------------- MMA
        constexpr uint32_t ID_A = idesc_bf16(128, 128, 0, 0);  // R (K-major) x W (K-major)
        constexpr uint32_t ID_O = idesc_bf16(128, DB, 0, 1);   // R (K-major) x S (MN-major)
        constexpr uint32_t ID_KV = idesc_bf16(128, DB, 1, 1);  // W^T (MN-major) x w V (MN-major)
        constexpr uint32_t ID_PV = idesc_bf16(128, DB, 0, 1);  // P (TMEM) x V (MN-major)
        auto tile = [&](int c, int j) -> uint32_t { return sbase + (uint32_t)slot(c, j) * C::slot_bytes; };
        auto release = [&](int c, int j) { tc_commit(smem_u32(&ctl.free[slot(c, j)])); };
        // a walk over the chunks that can run one ahead of another
        struct Cursor {
            int seg, ci, nch, a, b, base, rows;
        };
        auto next = [&](Cursor &c) -> bool {
            ++c.ci;
            while (c.ci >= c.nch) {
                if (++c.seg >= end - first) return false;
                const int n = C::rev ? end - 1 - c.seg : first + c.seg;
                c.a = min(max(p.cu[n], t0), t1);
                c.b = max(c.a, min(min(p.cu[n + 1], p.T), t1));
                leave_out(c.a, c.b);
                c.nch = (c.b - c.a + kC - 1) / kC;
                c.ci = 0;
            }
            c.base = c.a + (C::rev ? c.nch - 1 - c.ci : c.ci) * kC;
            c.rows = min(kC, c.b - c.base);
            return true;
        };
        Cursor cur{-1, 0, 0, 0, 0, 0, 0};
        if (warp == 21) {
            // A, one chunk ahead of the state's products where it has two buffers (P's warps then
            // never wait for it), and the state's products
            Cursor ahead = cur;
            int quarters = 0, k = 0;  // k: chunks whose A has been issued
            uint32_t cleans[2] = {0u, 0u};
            auto begin = [&]() {
                if (!next(ahead)) return;
                if (C::out) wait(ctl.full[slot(k, C::tR)], phase(k, C::tR));
                wait(ctl.full[slot(k, C::tW)], phase(k, C::tW));
                if (M == DQ) {
                    wait(ctl.full[slot(k, C::tE)], phase(k, C::tE));
                    wait_v(k);
                }
                if (ahead.rows < kC) {
                    const uint32_t seen = k & 1 ? cleans[1] : cleans[0];
                    wait(ctl.clean[k & 1], seen & 1);
                    (k & 1 ? cleans[1] : cleans[0]) = seen + 1;
                }
                if (C::out) {
                    const uint32_t ab = M == DQ ? 0u : (uint32_t)(k & 1);
                    const int use = M == DQ ? k : k >> 1;  // of this buffer
                    if (use > 0) wait(ctl.a_free[ab], (use - 1) & 1);
                    tc_fence_after();
                    const uint32_t tr = tile(k, C::tR), tw = tile(k, C::tW);
                    const uint32_t te = M == DQ ? tile(k, C::tE) : 0u, tv = M == DQ ? tile(k, C::tV) : 0u;
                    if (elect_one_sync()) {
                        products(tmem + C::col_a + 128 * ab, kmajor(tr), kmajor(tw), ID_A, DA / 16, 0u);
                        if constexpr (M == DQ) {  // Q K^T beside it
                            products(tmem + C::col_a + 128, kmajor(te), kmajor(tv), ID_A, DB / 16, 0u);
                            release(k, C::tE);
                            release(k, C::tE);
                        }
                        tc_commit(smem_u32(&ctl.a_full[ab]));
                        release(k, C::tR);
                    }
                    __syncwarp();
                }
                ++k;
            };
            if (M != DQ) begin();
            while (next(cur)) {
                if (M == DQ) begin();
                const int nq = (cur.rows + 31) / 32;
                const uint32_t tw = tile(it, C::tW);
                wait(ctl.s_full, it & 1);
                auto quarter = [&](int qq) {
                    const int vbuf = quarters & (C::groups - 1);
                    wait(ctl.vb_full[vbuf], (quarters / C::groups) & 1);
                    tc_fence_after();
                    const uint32_t vb = sbase + C::off_vb + vbuf * C::vb_bytes;
                    if (elect_one_sync()) {
#pragma unroll 1
                        for (int part = 0; part < 2; ++part)
                            products(tmem + C::col_s, mnmajor(tw + 4096 * qq, kBox), mnmajor(vb + part * C::vb_part, 4096), ID_KV, 2, 1u);
                        tc_commit(smem_u32(&ctl.vb_free[vbuf]));
                        if (qq == nq - 1) {
                            tc_commit(smem_u32(&ctl.kv_done));
                            release(it, C::tW);
                            release(it, C::tW);
                            release(it, C::tV);
                            if (C::sum) release(it, C::tV);
                        }
                    }
                    __syncwarp();
                    ++quarters;
                };
                const int before = M == DQ ? nq : min(nq, 2);
                for (int qq = 0; qq < before; ++qq) quarter(qq);
                if (M != DQ) begin();  // the next chunk's
                for (int qq = before; qq < nq; ++qq) quarter(qq);
                ++it;
            }
        } else if (C::out) {
            uint32_t cleans[2] = {0u, 0u};
            while (next(cur)) {
                if (cur.rows < kC) {
                    const uint32_t seen = it & 1 ? cleans[1] : cleans[0];
                    wait(ctl.clean[it & 1], seen & 1);
                    (it & 1 ? cleans[1] : cleans[0]) = seen + 1;
                }
                wait(ctl.full[slot(it, C::tR)], phase(it, C::tR));
                wait(ctl.s_full, it & 1);
                if (it > 0) wait(ctl.o_free, (it - 1) & 1);
                tc_fence_after();
                const uint32_t tr = tile(it, C::tR);
                if (elect_one_sync()) {
                    products(tmem + C::col_o, kmajor(tr), mnmajor(sbase + C::off_sb, DA * 128), ID_O, DA / 16, 0u);
                    tc_commit(smem_u32(&ctl.qs_done));
                    release(it, C::tR);
                }
                __syncwarp();
                const uint32_t ab = M == DQ ? 0u : (uint32_t)(it & 1), tv = tile(it, C::tV);
                wait_v(it);
                wait(ctl.p_full[ab], (M == DQ ? it : it >> 1) & 1);
                wait(ctl.o_scaled, it & 1);
                tc_fence_after();
                if (elect_one_sync()) {
                    Operand v = mnmajor(tv, kBox);
#pragma unroll 1
                    for (int kk = 0; kk < (cur.rows + 15) / 16; ++kk) {
                        tc_mma_ts(tmem + C::col_o, tmem + C::col_a + 128 * ab + 8 * kk, v.desc, ID_PV, 1u);
                        advance(v, kk);
                    }
                    tc_commit(smem_u32(&ctl.pv_done));
                    tc_commit(smem_u32(&ctl.a_free[ab]));
                    release(it, C::tV);
                }
                __syncwarp();
                ++it;
            }
        }
        if (*dead) {  // the products in flight end before TMEM is released (bounded)
            if (elect_one_sync()) tc_commit(smem_u32(&ctl.end));
            __syncwarp();
            mbar_wait(smem_u32(&ctl.end), 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::cols) : "memory");
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return (PFN_cuTensorMapEncodeTiled_v12000) nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// [T][Hx][D] bf16 as (channel, head, token); box 64 x 1 x 128.
bool encode(CUtensorMap *m, const void *base, int T, int Hx, int D) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hx, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)Hx * D * 2};
    const cuuint32_t box[3] = {64, 1, kC};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DA, int DB, int M>
cudaError_t launch_t(const Params &p, cudaStream_t st, bool follows) {
    using C = Cfg<DA, DB, M>;
    constexpr int bytes = C::bytes;
    static_assert(bytes <= 232448 && C::off_ctl % 16 == 0, "shared memory");
    Maps maps;
    if (!encode(&maps.wr, p.wr, p.T, p.H / p.wr_div, DA) || !encode(&maps.val, p.val, p.T, p.H / p.val_div, DB) ||
        !encode(&maps.rd, C::out ? p.rd : p.wr, p.T, C::out ? p.H / p.rd_div : p.H / p.wr_div, DA) ||
        !encode(&maps.ext, M == DQ || M == DK ? p.ext : p.val, p.T, M == DQ || M == DK ? p.H / p.ext_div : p.H / p.val_div, DB))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done;
    cudaError_t e = allow_smem(done, (const void *)tc_kernel<DA, DB, M>, bytes);
    if (e != cudaSuccess) return e;
    Params q = p;
    q.clear_err = !follows;
    return launch(tc_kernel<DA, DB, M>, dim3(p.H, p.W), kThreads, bytes, st, follows, q, maps);
}
template <int DK_, int DV_>
cudaError_t fwd_t(const Params &p, cudaStream_t st) {
    const bool split = p.W > 1 && !p.by_seq;
    if (split) {
        cudaError_t e = launch_t<DK_, DV_, SUM>(p, st, false);
        if (e == cudaSuccess) e = launch_scan(p, nullptr, DK_ * DV_, st);
        if (e != cudaSuccess) return e;
    }
    return launch_t<DK_, DV_, FWD>(p, st, split);
}
template <int DK_, int DV_>
cudaError_t bwd_t(const Params &a, const Params &b, const Params &d, cudaStream_t st) {
    const bool split = a.W > 1 && !a.by_seq;
    cudaError_t e = cudaSuccess;
    if (split) {
        e = launch_t<DV_, DK_, SUM>(a, st, false);
        if (e == cudaSuccess) e = launch_t<DV_, DK_, SUMR>(b, st, true);
        if (e == cudaSuccess) e = launch_scan(a, &b, DK_ * DV_, st);
    }
    if (e == cudaSuccess) e = launch_t<DV_, DK_, DQ>(a, st, split);
    if (e == cudaSuccess) e = launch_t<DV_, DK_, DK>(b, st, true);
    if (e == cudaSuccess) e = launch_t<DK_, DV_, DV>(d, st, true);
    return e;
}

}  // namespace tc

// bf16 (T > 0): the same as rec_forward and rec_backward.
cudaError_t tc_forward(const Params &p, int dk, int dv, cudaStream_t st) {
    if (dk == 128) return dv == 128 ? tc::fwd_t<128, 128>(p, st) : tc::fwd_t<128, 64>(p, st);
    return dv == 128 ? tc::fwd_t<64, 128>(p, st) : tc::fwd_t<64, 64>(p, st);
}
cudaError_t tc_backward(const Params &q, const Params &k, const Params &v, int dk, int dv, cudaStream_t st) {
    if (dk == 128) return dv == 128 ? tc::bwd_t<128, 128>(q, k, v, st) : tc::bwd_t<128, 64>(q, k, v, st);
    return dv == 128 ? tc::bwd_t<64, 128>(q, k, v, st) : tc::bwd_t<64, 64>(q, k, v, st);
}

}  // namespace lin
}  // namespace kda

// Linear attention with one decay per head: shared definitions.
//
// Per (sequence n, head h), S in R^{dk x dv} (fp32):
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = S_t^T (scale q_t),
// g_t <= 0 one number per token and head (or per head).  q and k have Hk
// heads, head h reads head h / (H / Hk).
//
// Windows: the packed token axis is cut into W equal windows of `win` tokens,
// and one CTA runs the tokens of one (window, head), sequence after sequence,
// so the load is even whatever the sequence lengths are and no table has to be
// made on the device.  The state that enters a window in the middle of a
// sequence comes from the windows before it: a window maps it as
// S -> gamma S + Z (the decay is one number per head, so the transition is
// one number), every window's (gamma, Z) is made in parallel by a summary
// pass, and a scan over the windows turns Z into the incoming states.
//
// When the host knows the sequence lengths and there are enough sequences and
// heads to fill the SMs evenly, a window is a whole sequence instead
// (by_seq), the longest first, and neither summary nor scan is needed.
//
// Reverse passes (the gradient) run the same recurrence from the last token
// to the first: the state is dL/dS_t, which step t reaches with the decay of
// token t + 1.  There "init" is dL/d(final state) and "final" dL/d(initial
// state), which also takes the decay of the sequence's first token.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace kda {
namespace lin {

// Log-decays below this leave nothing of an fp32 state (exp(-104) is 0 in
// fp32), so clamping there changes no result; it keeps sums of -inf finite.
constexpr float kMinG = -110.f;
// (NaN stays NaN, as it is in the single-token step, which does not clamp)
__device__ __forceinline__ float clamp_g(float g) {
    float x;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(g), "f"(kMinG));
    return x;
}

// In place of a window's gamma: nobody reads its outgoing state (no sequence
// crosses its end), and that state begins in the window, so that nothing of what
// enters it may reach it (not even times 0, which inf would survive as NaN).
constexpr float kNoCarry = -1.f, kBegins = -2.f;

struct Params {
    // one pass of the recurrence: state [DA][DB] += wr (x) val, out = state^T rd
    const void *rd, *wr;    // [T][H / rd_div][DA], [T][H / wr_div][DA]
    const void *val;        // [T][H / val_div][DB]
    const void *ext;        // [T][H / ext_div][DB]: xdot_t = out_t . ext_t (gradient passes)
    int rd_div, wr_div, val_div, ext_div;
    float rd_scale, wr_scale;
    const void *g;          // [T][H], or [H] when g_per_head
    int g_per_head;
    void *out;              // [T][H][DB], input type (or fp32 when out_f32)
    int out_f32;
    const int32_t *cu;
    int num_seqs, T, H, W, win;
    int by_seq;             // window w is the sequence with w longer ones (kSortSeqs at most; behind that, sequence w)
    const float *init;      // [num_seqs][H] states or null; transposed ([DB][DA]) when init_t
    float *final_state;     // same layout, or null
    int init_t;
    float *win_state;       // [W][H] states [DA][DB]: Z out of the summary, incoming states after the scan (with
                            // by_seq not one per window, and not to be read whatever the offsets say)
    int win_t;              // the pass reads them transposed
    float *gamma;           // [W][H]
    float *start_copy;      // [W][H] states or null.  When final_state is init, the summary keeps here the
                            // initial state of the sequence that starts in the window and crosses its end:
                            // its last window overwrites that state in the same launch
    int32_t *err;           // [3] words of the workspace's header: [2] bit 0 = a bounded wait gave up
    int clear_err;          // this kernel clears them
    // gradient passes
    float *xdot;            // [T][H]: q . dq, written by the dq pass, read by the dk pass
    void *ckpt;             // [slots][H][DA][DB]: fp32: in fp32 passes the state after each 64-token chunk, in
                            // bf16 passes, before each 128-token chunk, as [DB / 4][DA][4]
    float *xstate, *across;  // bf16 passes, [T][H]: see kda_lin_tc.cu
    void *dg;               // [T][H], input type, or fp32 when g_per_head
    int zero_first_dg;      // no initial state: d(first log-decay) is exactly 0
};

constexpr int kSortSeqs = 128;

// The tokens [t0, t1) of window w, and its sequences first .. end - 1, of
// which those from `lo` on start in it.
struct Window {
    int t0, t1, lo, first, end;
};
__device__ __forceinline__ int first_at_or_behind(const Params &p, int x) {
    int lo = 0, hi = p.num_seqs;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid] < x) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}
// Called by all threads of the CTA (at least kSortSeqs); ends with a barrier
// when by_seq.  `slot`: a shared word.
__device__ __forceinline__ Window window_of(const Params &p, int w, int *slot) {
    Window v;
    if (p.by_seq) {
        if (p.num_seqs <= kSortSeqs) {
            const int n = threadIdx.x;
            if (n < p.num_seqs) {
                const int len = p.cu[n + 1] - p.cu[n];
                int rank = 0;
                for (int m = 0; m < p.num_seqs; ++m) {
                    const int other = p.cu[m + 1] - p.cu[m];
                    rank += other > len || (other == len && m < n);
                }
                if (rank == w) *slot = n;
            }
            __syncthreads();
            v.first = *slot;
        } else {
            v.first = w;
        }
        v.lo = v.first;
        v.end = v.first + 1;
        v.t0 = min(max(p.cu[v.first], 0), p.T);
        v.t1 = min(max(p.cu[v.end], v.t0), p.T);
        return v;
    }
    v.t0 = w * p.win;
    v.t1 = min(p.T, v.t0 + p.win);
    v.lo = first_at_or_behind(p, v.t0);
    // the sequence that continues into the window, then those that start in it (the last window also
    // takes the empty ones at the very end)
    v.first = v.lo > 0 && p.cu[v.lo] > v.t0 ? v.lo - 1 : v.lo;
    v.end = w == p.W - 1 ? p.num_seqs : first_at_or_behind(p, v.t1);
    return v;
}
// The sequence whose state a summary carries over the window's outgoing edge, or -1.
__device__ __forceinline__ int crossing(const Params &p, const Window &v, bool rev) {
    int n;
    if (!rev) {
        n = v.t1 < p.T ? first_at_or_behind(p, v.t1) - 1 : -1;
        if (n >= 0 && p.cu[n + 1] <= v.t1) n = -1;
    } else {
        n = v.t0 > 0 ? v.lo - 1 : -1;
        if (n >= 0 && p.cu[n + 1] <= v.t0) n = -1;
    }
    return n;
}

// Launches of one call follow each other early: a kernel is started while the
// one before it drains, does what depends on the call's inputs only (offsets,
// barriers, tensor memory) and waits in after_previous() until that one's
// results are there.  The first launch of a call is an ordinary one.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... K, typename... A>
cudaError_t launch(void (*kernel)(K...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, bool follows, A... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = follows ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, K(args)...);
}

// SMs of the current device (148 when there is none).
int sm_count();
// Lets `kernel` use `bytes` of dynamic shared memory on the current device;
// `done` remembers the devices where it has been said.
cudaError_t allow_smem(std::atomic<uint64_t> &done, const void *kernel, int bytes);

}  // namespace lin
}  // namespace kda

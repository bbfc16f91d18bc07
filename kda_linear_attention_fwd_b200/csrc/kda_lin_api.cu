// C-ABI entry points of linear attention with one decay per head (declared in
// include/kda.h): argument checks, the window plan and the launch sequences.
// No allocation, no host synchronisation, no exceptions across the boundary.
#include <algorithm>
#include <atomic>

#include "../../include/kda.h"
#include "kda_args.h"
#include "kda_common.cuh"
#include "kda_lin.h"

namespace kda {
namespace lin {

cudaError_t rec_forward(const Params &p, int dk, int dv, cudaStream_t st);
cudaError_t rec_backward(const Params &q, const Params &k, const Params &v, int dk, int dv, cudaStream_t st);
cudaError_t tc_forward(const Params &p, int dk, int dv, cudaStream_t st);
cudaError_t tc_backward(const Params &q, const Params &k, const Params &v, int dk, int dv, cudaStream_t st);
cudaError_t launch_decode(bool bf16, int dk, int dv, const void *q, const void *k, const void *v, const void *g,
                          void *out, float *state, long nh, int H, int rep, int g_per_head, float scale, int sms,
                          cudaStream_t st);

int sm_count() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return 148;
    }
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            return 148;
        }
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

cudaError_t allow_smem(std::atomic<uint64_t> &done, const void *kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (bit & done.load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// The tokens of a packed call that lie in a sequence: [cu[0], cu[num_seqs]).
struct Tokens {
    const int32_t *cu;
    int num_seqs, T;
    KDA_DEVICE long first() const { return min(max(cu[0], 0), T); }
    KDA_DEVICE long last() const { return min(max(cu[num_seqs], 0), T); }
};

// out[t][hk][i] = sum over r of in[t][hk * rep + r][i]: the gradient of a head
// shared by rep heads, rounded once.  D a multiple of 4.
template <typename T>
__global__ void __launch_bounds__(256) head_sum_kernel(const float4 *in0, T *out0, const float4 *in1, T *out1, const Tokens tk,
                                                       int Hk, int rep, int d4) {
    let_next_start();
    after_previous();
    const float4 *in = blockIdx.y ? in1 : in0;
    T *out = blockIdx.y ? out1 : out0;
    const long row4 = (long)Hk * d4;
    for (long i = tk.first() * row4 + (long)blockIdx.x * 256 + threadIdx.x; i < tk.last() * row4; i += (long)gridDim.x * 256) {
        const long th = i / d4, c = i % d4;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < rep; ++r) {
            const float4 x = __ldcs(in + (th * rep + r) * d4 + c);
            a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
        }
        st(out + 4 * i, a.x); st(out + 4 * i + 1, a.y); st(out + 4 * i + 2, a.z); st(out + 4 * i + 3, a.w);
    }
}

// out = x + y, rounded
template <typename T>
__global__ void __launch_bounds__(256) add_kernel(const float *x, const float *y, T *out, const Tokens tk, int H) {
    let_next_start();
    after_previous();
    for (long i = tk.first() * H + (long)blockIdx.x * 256 + threadIdx.x; i < tk.last() * H; i += (long)gridDim.x * 256)
        st(out + i, x[i] + y[i]);
}

// Column sums of x (+ y) [T][H] in two steps whose order is fixed: per block of
// kSumRows rows, then over the blocks.
constexpr int kSumRows = 512;
__global__ void __launch_bounds__(256) token_sum_kernel(const float *x, const float *y, float *part, const Tokens tk, int H) {
    let_next_start();
    after_previous();
    __shared__ float s[8][33];
    const int hx = threadIdx.x & 31, ry = threadIdx.x >> 5, h = blockIdx.y * 32 + hx;
    const long b0 = (long)blockIdx.x * kSumRows, t0 = max(b0, tk.first()), t1 = min(b0 + kSumRows, tk.last());
    float a = 0.f;
    if (h < H)
        for (long t = t0 + ry; t < t1; t += 8) a += x[t * H + h] + (y ? y[t * H + h] : 0.f);
    s[ry][hx] = a;
    __syncthreads();
    if (ry == 0 && h < H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) a += s[i][hx];
        part[(size_t)blockIdx.x * H + h] = a;
    }
}
template <typename T>
__global__ void __launch_bounds__(256) part_sum_kernel(const float *part, T *out, int parts, int H) {
    let_next_start();
    after_previous();
    __shared__ float s[8][33];
    const int hx = threadIdx.x & 31, ry = threadIdx.x >> 5, h = blockIdx.x * 32 + hx;
    float a = 0.f;
    if (h < H)
        for (int i = ry; i < parts; i += 8) a += part[(size_t)i * H + h];
    s[ry][hx] = a;
    __syncthreads();
    if (ry == 0 && h < H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) a += s[i][hx];
        st(out + h, a);
    }
}

}  // namespace lin
}  // namespace kda

namespace {

using kda::is_aligned;
using kda::lin::Params;

using kda::lin::sm_count;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Windows {
    int win, W;
};
// How the tokens are divided over CTAs.  Each pass runs in rounds of as many
// CTAs as the device holds (tensor cores: one per SM; token by token: two or
// three), so its time is about rounds x steps of the longest window (128
// tokens on the tensor cores, one otherwise) + a start-up per round; more than
// one window also costs the summary pass, about 0.6 of the main one, and the
// scan.  The gradient's token-by-token passes keep whole 64-token chunks.
enum class Pass { tc, rec_fwd, rec_bwd };
struct Model {
    long slots, step, unit, start, scan;  // CTAs at once; window granularity; tokens per step; steps per round, per scan
};
Model model_of(int dk, int dv, Pass pass) {
    const long sms = sm_count();
    if (pass == Pass::tc) return {sms, 128, 128, 1, 2};
    return {(dk * dv > 128 * 64 ? 2 : 3) * sms, pass == Pass::rec_bwd ? 64 : 32, 1, 15, 25};
}
long div_up(long a, long b) { return (a + b - 1) / b; }
double windows_cost(const Model &m, long T, int H, long W) {
    const double main = (double)div_up(W * H, m.slots) * (div_up(div_up(T, W), m.unit) + m.start);
    return W > 1 ? 1.6 * main + m.scan : main;
}
Windows choose_windows(int T, int H, int dk, int dv, Pass pass) {
    const Model m = model_of(dk, dv, pass);
    // one window, or as many as fill the slots once, twice, three or four times
    long best = 1;
    for (long k = 1; k <= 4; ++k) {
        const long W = std::min(std::max(1L, k * m.slots / H), div_up(std::max(T, 1), m.step));
        const long win = div_up(div_up(T, W), m.step) * m.step;
        if (W > 1 && windows_cost(m, T, H, div_up(T, win)) < windows_cost(m, T, H, best)) best = div_up(T, win);
    }
    const long win = std::max(m.step, div_up(div_up(T, best), m.step) * m.step);
    return {(int)win, std::max(1, (int)div_up(T, win))};
}
// Whole sequences as windows: no summary, but a CTA per (sequence, head), the
// longest first, which takes about max(longest, work / slots).
bool choose_by_seq(int T, int N, int H, int dk, int dv, Pass pass, const int32_t *cu_host, const Windows &wd) {
    if (!cu_host || N > 65535) return false;
    const Model m = model_of(dk, dv, pass);
    long total = 0, longest = 0;
    for (int n = 0; n < N; ++n) {
        const long c = div_up(cu_host[n + 1] - cu_host[n], m.unit) + m.start;
        total += c;
        longest = std::max(longest, c);
    }
    const double cost = std::max((double)longest, (double)total * H / m.slots + (N > kda::lin::kSortSeqs ? longest : 0));
    return cost < windows_cost(m, T, H, wd.W);
}

// bf16 on the tensor cores, fp32 (and calls with no tokens at all) token by token
bool use_tc(kda_dtype dtype, int T) { return dtype == KDA_DTYPE_BF16 && T > 0; }

struct FwdLayout {
    size_t header, gamma, z, start, total;
};
FwdLayout fwd_layout(const Windows &wd, int H, int dk, int dv) {
    FwdLayout L;
    const size_t states = (size_t)wd.W * H * dk * dv * sizeof(float);
    size_t o = 0;
    L.header = o; o = align256(o + 64 * sizeof(int32_t));
    L.gamma = o; o = align256(o + (size_t)wd.W * H * sizeof(float));
    L.z = o;     o = align256(o + states);
    L.start = o; o = align256(o + states);
    L.total = o;
    return L;
}

struct BwdLayout {
    size_t header, gamma_f, gamma_r, zf, zr, xdot, xstate, across, ckpt, part, dq, dk, total;
};
BwdLayout bwd_layout(const Windows &wd, bool tc, int T, int N, int H, int Hk, int dk, int dv) {
    BwdLayout L;
    const size_t states = (size_t)wd.W * H * dk * dv * sizeof(float), th = (size_t)T * H * sizeof(float);
    const size_t ckpt = ((size_t)T / (tc ? 128 : 64) + N + 1) * sizeof(float);
    size_t o = 0;
    L.header = o;  o = align256(o + 64 * sizeof(int32_t));
    L.gamma_f = o; o = align256(o + (size_t)wd.W * H * sizeof(float));
    L.gamma_r = o; o = align256(o + (size_t)wd.W * H * sizeof(float));
    L.zf = o;      o = align256(o + states);
    L.zr = o;      o = align256(o + states);
    L.xdot = o;    o = align256(o + th);
    L.xstate = o;  o = align256(o + th);
    L.across = o;  o = align256(o + (tc ? th : 0));
    L.ckpt = o;    o = align256(o + ckpt * H * dk * dv);
    L.part = o;    o = align256(o + ((size_t)T / kda::lin::kSumRows + 1) * H * sizeof(float));
    L.dq = o;      o = align256(o + (H == Hk ? 0 : th * dk));
    L.dk = o;      o = align256(o + (H == Hk ? 0 : th * dk));
    L.total = o;
    return L;
}

int check_sizes(int32_t num_seqs, int32_t T, int32_t H, int32_t Hk, int32_t dk, int32_t dv, kda_dtype dtype,
                int32_t flags) {
    const int rc = kda::check_prefill_sizes(num_seqs, T, H, dk, dv, dtype);
    if (rc != KDA_OK) return rc;
    if (Hk < 1 || H % Hk != 0 || (flags & ~KDA_LIN_DECAY_PER_HEAD)) return KDA_ERR_INVALID_ARG;
    if (H > (1 << 20)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

bool overlap(const void *a, const void *b, size_t bytes) {
    return a && b && (const char *)a < (const char *)b + bytes && (const char *)b < (const char *)a + bytes;
}

// the checks that the packed calls share; `a16` must be 16-byte aligned
int check_packed(const int32_t *cu, const int32_t *cu_host, int32_t num_seqs, int32_t T, const void *g, size_t esz,
                 const void *const *a16, int n16) {
    if (!cu) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < n16; ++i)
        if (a16[i] && !is_aligned(a16[i], 16)) return KDA_ERR_ALIGNMENT;
    if (!is_aligned(g, esz) || !is_aligned(cu, 4)) return KDA_ERR_ALIGNMENT;
    if (cu_host) {
        if (cu_host[0] != 0 || cu_host[num_seqs] != T) return KDA_ERR_INVALID_ARG;
        for (int n = 0; n < num_seqs; ++n)
            if (cu_host[n + 1] < cu_host[n]) return KDA_ERR_INVALID_ARG;
    }
    return KDA_OK;
}

template <typename F> bool ok(F e) { return e == cudaSuccess; }

}  // namespace

extern "C" {

size_t kda_lin_chunk_fwd_workspace_size(int32_t total_tokens, int32_t num_seqs, int32_t H, int32_t Hk, int32_t dk,
                                        int32_t dv, kda_dtype dtype) {
    if (check_sizes(num_seqs, total_tokens, H, Hk, dk, dv, dtype, 0) != KDA_OK) return 0;
    return fwd_layout(choose_windows(total_tokens, H, dk, dv, use_tc(dtype, total_tokens) ? Pass::tc : Pass::rec_fwd), H, dk, dv).total;
}

int kda_lin_chunk_fwd(const void *q, const void *k, const void *v, const void *g, void *out, const int32_t *cu_seqlens,
                      const int32_t *cu_seqlens_host, int32_t num_seqs, int32_t total_tokens, int32_t H, int32_t Hk,
                      int32_t dk, int32_t dv, kda_dtype dtype, float scale, int32_t flags, const float *initial_state,
                      float *final_state, void *workspace, size_t workspace_bytes, kda_stream_t stream) {
    cudaStream_t st = (cudaStream_t)stream;
    int rc = check_sizes(num_seqs, total_tokens, H, Hk, dk, dv, dtype, flags);
    if (rc != KDA_OK) return rc;
    if (num_seqs == 0) return total_tokens == 0 ? KDA_OK : KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!q || !k || !v || !g || !out)) return KDA_ERR_INVALID_ARG;
    const bool bf16 = dtype == KDA_DTYPE_BF16;
    const void *a16[] = {q, k, v, out, initial_state, final_state, workspace};
    rc = check_packed(cu_seqlens, cu_seqlens_host, num_seqs, total_tokens, g, bf16 ? 2 : 4, a16, 7);
    if (rc != KDA_OK) return rc;
    const bool in_place = initial_state && initial_state == final_state;
    if (!in_place && overlap(initial_state, final_state, (size_t)num_seqs * H * dk * dv * sizeof(float)))
        return KDA_ERR_INVALID_ARG;
    const bool tc = use_tc(dtype, total_tokens);
    const Windows wd = choose_windows(total_tokens, H, dk, dv, tc ? Pass::tc : Pass::rec_fwd);
    const FwdLayout L = fwd_layout(wd, H, dk, dv);
    if (!workspace || workspace_bytes < L.total) return KDA_ERR_WORKSPACE;
    char *ws = (char *)workspace;

    Params p{};
    p.rd = q; p.wr = k; p.val = v; p.g = g; p.out = out;
    p.rd_div = p.wr_div = H / Hk;
    p.val_div = p.ext_div = 1;
    p.rd_scale = scale;
    p.wr_scale = 1.f;
    p.g_per_head = flags & KDA_LIN_DECAY_PER_HEAD;
    p.cu = cu_seqlens;
    p.num_seqs = num_seqs; p.T = total_tokens; p.H = H; p.W = wd.W; p.win = wd.win;
    p.by_seq = choose_by_seq(total_tokens, num_seqs, H, dk, dv, tc ? Pass::tc : Pass::rec_fwd, cu_seqlens_host, wd);
    if (p.by_seq) p.W = num_seqs;
    p.init = initial_state;
    p.final_state = final_state;
    p.gamma = (float *)(ws + L.gamma);
    p.win_state = (float *)(ws + L.z);
    p.start_copy = in_place && wd.W > 1 && !p.by_seq ? (float *)(ws + L.start) : nullptr;
    p.err = (int32_t *)(ws + L.header);
    return ok(tc ? kda::lin::tc_forward(p, dk, dv, st) : kda::lin::rec_forward(p, dk, dv, st)) ? KDA_OK : KDA_ERR_CUDA;
}

int kda_lin_decode_step(const void *q, const void *k, const void *v, const void *g, void *out, float *state,
                        int32_t num_seqs, int32_t H, int32_t Hk, int32_t dk, int32_t dv, kda_dtype dtype, float scale,
                        int32_t flags, kda_stream_t stream) {
    const int rc = check_sizes(num_seqs, 0, H, Hk, dk, dv, dtype, flags);
    if (rc != KDA_OK) return rc;
    if (num_seqs == 0) return KDA_OK;
    if (!q || !k || !v || !g || !out || !state) return KDA_ERR_INVALID_ARG;
    const bool bf16 = dtype == KDA_DTYPE_BF16;
    const void *a16[] = {q, k, v, out, state};
    for (const void *p : a16)
        if (!is_aligned(p, 16)) return KDA_ERR_ALIGNMENT;
    if (!is_aligned(g, bf16 ? 2 : 4)) return KDA_ERR_ALIGNMENT;
    const long nh = (long)num_seqs * H;
    if (nh > 0x7fffffffL) return KDA_ERR_UNSUPPORTED;
    return ok(kda::lin::launch_decode(bf16, dk, dv, q, k, v, g, out, state, nh, H, H / Hk,
                                      flags & KDA_LIN_DECAY_PER_HEAD, scale, sm_count(), (cudaStream_t)stream))
               ? KDA_OK
               : KDA_ERR_CUDA;
}

size_t kda_lin_bwd_workspace_size(int32_t total_tokens, int32_t num_seqs, int32_t H, int32_t Hk, int32_t dk,
                                  int32_t dv) {
    if (check_sizes(num_seqs, total_tokens, H, Hk, dk, dv, KDA_DTYPE_F32, 0) != KDA_OK) return 0;
    // enough for either element type
    size_t total = 0;
    for (bool tc : {false, true})
        total = std::max(total, bwd_layout(choose_windows(total_tokens, H, dk, dv, tc ? Pass::tc : Pass::rec_bwd), tc, total_tokens, num_seqs, H, Hk, dk, dv).total);
    return total;
}

int kda_lin_bwd(const void *q, const void *k, const void *v, const void *g, const void *dy, const int32_t *cu_seqlens,
                const int32_t *cu_seqlens_host, int32_t num_seqs, int32_t total_tokens, int32_t H, int32_t Hk,
                int32_t dk, int32_t dv, kda_dtype dtype, float scale, int32_t flags, const float *initial_state,
                const float *d_final_state, void *dq, void *dk_out, void *dv_out, void *dg, float *d_initial_state,
                void *workspace, size_t workspace_bytes, kda_stream_t stream) {
    using namespace kda::lin;
    cudaStream_t st = (cudaStream_t)stream;
    int rc = check_sizes(num_seqs, total_tokens, H, Hk, dk, dv, dtype, flags);
    if (rc != KDA_OK) return rc;
    if (num_seqs == 0) {
        if (total_tokens != 0) return KDA_ERR_INVALID_ARG;
        if (!(flags & KDA_LIN_DECAY_PER_HEAD) || !dg) return KDA_OK;
        return ok(cudaMemsetAsync(dg, 0, (size_t)H * (dtype == KDA_DTYPE_BF16 ? 2 : 4), st)) ? KDA_OK : KDA_ERR_CUDA;
    }
    if (total_tokens > 0 && (!q || !k || !v || !g || !dy || !dq || !dk_out || !dv_out || !dg)) return KDA_ERR_INVALID_ARG;
    const bool bf16 = dtype == KDA_DTYPE_BF16;
    const size_t esz = bf16 ? 2 : 4;
    const void *a16[] = {q, k, v, dy, initial_state, d_final_state, dq, dk_out, dv_out, d_initial_state, workspace};
    rc = check_packed(cu_seqlens, cu_seqlens_host, num_seqs, total_tokens, g, esz, a16, 11);
    if (rc != KDA_OK) return rc;
    if (!is_aligned(dg, esz)) return KDA_ERR_ALIGNMENT;
    const size_t state_bytes = (size_t)num_seqs * H * dk * dv * sizeof(float);
    if (overlap(initial_state, d_initial_state, state_bytes) || overlap(d_final_state, d_initial_state, state_bytes))
        return KDA_ERR_INVALID_ARG;
    const bool tc = use_tc(dtype, total_tokens);
    const Windows wd = choose_windows(total_tokens, H, dk, dv, tc ? Pass::tc : Pass::rec_bwd);
    const BwdLayout L = bwd_layout(wd, tc, total_tokens, num_seqs, H, Hk, dk, dv);
    if (!workspace || workspace_bytes < kda_lin_bwd_workspace_size(total_tokens, num_seqs, H, Hk, dk, dv))
        return KDA_ERR_WORKSPACE;
    char *ws = (char *)workspace;
    const int rep = H / Hk, per_head = flags & KDA_LIN_DECAY_PER_HEAD;

    Params c{};
    c.g = g;
    c.g_per_head = per_head;
    c.cu = cu_seqlens;
    c.num_seqs = num_seqs; c.T = total_tokens; c.H = H; c.W = wd.W; c.win = wd.win;
    c.by_seq = choose_by_seq(total_tokens, num_seqs, H, dk, dv, tc ? Pass::tc : Pass::rec_bwd, cu_seqlens_host, wd);
    if (c.by_seq) c.W = num_seqs;
    c.xdot = (float *)(ws + L.xdot);
    c.xstate = (float *)(ws + L.xstate);
    c.across = (float *)(ws + L.across);
    c.err = (int32_t *)(ws + L.header);
    c.ckpt = ws + L.ckpt;
    c.dg = per_head ? (void *)(ws + L.xstate) : dg;
    c.zero_first_dg = initial_state == nullptr;
    c.out_f32 = rep > 1;

    // dq: read dy, write v, value k; state [dv][dk]
    Params a = c;
    a.rd = dy; a.wr = v; a.val = k; a.ext = q;
    a.rd_div = a.wr_div = 1;
    a.val_div = a.ext_div = rep;
    a.rd_scale = scale;
    a.wr_scale = 1.f;
    a.out = rep > 1 ? (void *)(ws + L.dq) : dq;
    a.init = initial_state;
    a.init_t = 1;
    a.win_state = (float *)(ws + L.zf);
    a.gamma = (float *)(ws + L.gamma_f);
    // dk, reversed: read v, write dy, value q; state [dv][dk]
    Params b = c;
    b.rd = v; b.wr = dy; b.val = q; b.ext = k;
    b.rd_div = b.wr_div = 1;
    b.val_div = b.ext_div = rep;
    b.rd_scale = 1.f;
    b.wr_scale = scale;
    b.out = rep > 1 ? (void *)(ws + L.dk) : dk_out;
    b.init = d_final_state;
    b.init_t = 1;
    b.win_state = (float *)(ws + L.zr);
    b.gamma = (float *)(ws + L.gamma_r);
    // dv, reversed: read k, write q, value dy; state [dk][dv]
    Params d = c;
    d.rd = k; d.wr = q; d.val = dy;
    d.rd_div = d.wr_div = rep;
    d.val_div = d.ext_div = 1;
    d.rd_scale = 1.f;
    d.wr_scale = scale;
    d.out = dv_out;
    d.out_f32 = 0;
    d.init = d_final_state;
    d.final_state = d_initial_state;
    d.win_state = b.win_state;
    d.win_t = 1;
    d.gamma = b.gamma;

    if (!ok(tc ? tc_backward(a, b, d, dk, dv, st) : rec_backward(a, b, d, dk, dv, st))) return KDA_ERR_CUDA;
    if (total_tokens == 0) {
        if (per_head && dg && !ok(cudaMemsetAsync(dg, 0, (size_t)H * esz, st))) return KDA_ERR_CUDA;
        return KDA_OK;
    }
    const Tokens tk{cu_seqlens, num_seqs, total_tokens};
    if (rep > 1) {
        const long n4 = (long)total_tokens * Hk * dk / 4;
        const dim3 grid((unsigned)std::min<long>((n4 + 255) / 256, 4L * 148), 2);
        const float4 *in0 = (const float4 *)(ws + L.dq), *in1 = (const float4 *)(ws + L.dk);
        const cudaError_t e =
            bf16 ? launch(head_sum_kernel<__nv_bfloat16>, grid, 256, 0, st, true, in0, (__nv_bfloat16 *)dq, in1,
                          (__nv_bfloat16 *)dk_out, tk, Hk, rep, dk / 4)
                 : launch(head_sum_kernel<float>, grid, 256, 0, st, true, in0, (float *)dq, in1, (float *)dk_out, tk, Hk, rep,
                          dk / 4);
        if (!ok(e)) return KDA_ERR_CUDA;
    }
    if (per_head) {
        const int parts = (total_tokens + kSumRows - 1) / kSumRows, hb = (H + 31) / 32;
        float *part = (float *)(ws + L.part);
        if (!ok(launch(token_sum_kernel, dim3(parts, hb), 256, 0, st, true, c.xstate, tc ? c.across : nullptr, part, tk, H)))
            return KDA_ERR_CUDA;
        if (!ok(bf16 ? launch(part_sum_kernel<__nv_bfloat16>, dim3(hb), 256, 0, st, true, part, (__nv_bfloat16 *)dg, parts, H)
                     : launch(part_sum_kernel<float>, dim3(hb), 256, 0, st, true, part, (float *)dg, parts, H)))
            return KDA_ERR_CUDA;
    }
    if (tc && !per_head) {
        const long n = (long)total_tokens * H;
        if (!ok(launch(add_kernel<__nv_bfloat16>, dim3((unsigned)std::min<long>((n + 255) / 256, 8L * 148)), 256, 0, st, true,
                       c.xstate, c.across, (__nv_bfloat16 *)dg, tk, H)))
            return KDA_ERR_CUDA;
    }
    return ok(cudaGetLastError()) ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"

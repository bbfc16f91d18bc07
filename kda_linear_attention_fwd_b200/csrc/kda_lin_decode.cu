// Linear attention with one decay per head, one token per sequence:
//   S' = exp(g) S + k v^T,   o = S'^T (scale q),   S in place.
//
// A read-modify-write of the state (64 KiB per head at 128 x 128) bound by
// HBM bandwidth: one CTA of 256 threads owns DVS columns of one head, every
// thread keeps its part of the state in registers between the read and the
// write, and rows are read as 16-byte vectors.  The read of the state starts
// before anything else.  All DV columns in one CTA give the longest rows
// (512 bytes); with few heads the columns are split over DV / DVS CTAs so
// that more SMs load at once (launch_decode below).  Measured on one B200
// (6531 GB/s copied): 256 sequences x 32 heads of 128 x 128 (1.07 GB) 160 us;
// one sequence x 16 heads 3.6 us, bound by the latency of one round trip.
#include "kda_common.cuh"

namespace kda {
namespace lin {

template <int DK, int DVS, typename T>
__global__ void __launch_bounds__(256, 2)
    decode_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, const T *__restrict__ g,
                  T *__restrict__ out, float *state, int H, int rep, int dv, int g_per_head, float scale) {
    constexpr int NT = 256;
    constexpr int COLG = DVS / 4;
    constexpr int RPP = NT / COLG;              // rows covered by one pass of the CTA
    constexpr int PASSES = DK / RPP;
    constexpr int RW = COLG < 32 ? 32 / COLG : 1;  // rows of one warp
    static_assert(NT % COLG == 0 && DK % RPP == 0 && COLG <= 32, "tile shape");
    __shared__ float sk[DK], sq[DK];
    __shared__ __align__(16) float red[NT / 32][DVS];

    const unsigned nh = blockIdx.x;             // flattened (n, h)
    const int h = nh % H;
    const size_t nk = (size_t)(nh / H) * (H / rep) + h / rep;
    const int tid = threadIdx.x, cg = tid % COLG, r0 = tid / COLG, c0 = blockIdx.y * DVS;
    float4 *S = reinterpret_cast<float4 *>(state + (size_t)nh * DK * dv + c0);
    const int ld4 = dv / 4;

    float4 s[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) s[p] = ld_stream(S + (r0 + p * RPP) * ld4 + cg);

    for (int i = tid; i < DK; i += NT) {
        sk[i] = ld(k + nk * DK + i);
        sq[i] = ld(q + nk * DK + i);
    }
    const float a = expf(ld(g + (g_per_head ? (size_t)h : (size_t)nh)));
    float vv[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) vv[c] = ld(v + (size_t)nh * dv + c0 + cg * 4 + c);
    __syncthreads();

    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int i = r0 + p * RPP;
        const float ki = sk[i], qi = sq[i];
        s[p].x = fmaf(s[p].x, a, ki * vv[0]); s[p].y = fmaf(s[p].y, a, ki * vv[1]);
        s[p].z = fmaf(s[p].z, a, ki * vv[2]); s[p].w = fmaf(s[p].w, a, ki * vv[3]);
        st_stream(S + i * ld4 + cg, s[p]);
        o[0] = fmaf(qi, s[p].x, o[0]); o[1] = fmaf(qi, s[p].y, o[1]);
        o[2] = fmaf(qi, s[p].z, o[2]); o[3] = fmaf(qi, s[p].w, o[3]);
    }
#pragma unroll
    for (int m = COLG; m < 32; m <<= 1)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] += __shfl_xor_sync(0xffffffffu, o[c], m);
    if ((tid & 31) < COLG) *reinterpret_cast<float4 *>(&red[tid / 32][cg * 4]) = make_float4(o[0], o[1], o[2], o[3]);
    __syncthreads();
    for (int j = tid; j < DVS; j += NT) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) x += red[w][j];
        st(out + (size_t)nh * dv + c0 + j, scale * x);
    }
}

template <int DK, int DVS, typename T>
static cudaError_t launch_decode_t(const void *q, const void *k, const void *v, const void *g, void *out, float *state,
                                   long nh, int H, int rep, int dv, int g_per_head, float scale, cudaStream_t st) {
    decode_kernel<DK, DVS, T><<<dim3((unsigned)nh, dv / DVS), 256, 0, st>>>(
        (const T *)q, (const T *)k, (const T *)v, (const T *)g, (T *)out, state, H, rep, dv, g_per_head, scale);
    return cudaGetLastError();
}

template <typename T>
static cudaError_t launch_decode_dt(int dk, int dv, int dvs, const void *q, const void *k, const void *v,
                                    const void *g, void *out, float *state, long nh, int H, int rep, int g_per_head,
                                    float scale, cudaStream_t st) {
#define KDA_LIN_DECODE(DK, DVS) \
    return launch_decode_t<DK, DVS, T>(q, k, v, g, out, state, nh, H, rep, dv, g_per_head, scale, st)
    if (dk == 128) {
        if (dvs == 128) KDA_LIN_DECODE(128, 128);
        if (dvs == 64) KDA_LIN_DECODE(128, 64);
        KDA_LIN_DECODE(128, 32);
    }
    if (dvs == 128) KDA_LIN_DECODE(64, 128);
    if (dvs == 64) KDA_LIN_DECODE(64, 64);
    KDA_LIN_DECODE(64, 32);
#undef KDA_LIN_DECODE
}

cudaError_t launch_decode(bool bf16, int dk, int dv, const void *q, const void *k, const void *v, const void *g,
                          void *out, float *state, long nh, int H, int rep, int g_per_head, float scale, int sms,
                          cudaStream_t st) {
    // columns split only while the heads alone leave SMs without work
    const int dvs = nh < sms ? 32 : dv;
    if (bf16)
        return launch_decode_dt<__nv_bfloat16>(dk, dv, dvs, q, k, v, g, out, state, nh, H, rep, g_per_head, scale, st);
    return launch_decode_dt<float>(dk, dv, dvs, q, k, v, g, out, state, nh, H, rep, g_per_head, scale, st);
}

}  // namespace lin
}  // namespace kda

// lindecode.hip -- S new tokens of each request through the linear-attention
// recurrence, the state kept in registers between its load from the pool and
// its store:
//   S <- e^{g} S + v k^T,   o = scale S q     (per token)
//
// The rows of the state (one per value column, K floats) are independent, so
// a block takes RPT passes of NT/(K/4) rows of one (request, value head): K/4
// lanes of 16 bytes hold a row, and every wave-wide access covers whole rows.
// The step is bound by moving the state, read and written once: 107 us for 256
// requests of 16 heads of 128 x 128 (529 MB, 4.9 TB/s, a large copy reaching
// 5.1).  One request of 16 heads takes 3.3 us, less than the host needs.
#include "gdp_common.h"
#include "gdp_internal.h"
#include "linattn.h"

namespace gdp {

namespace {
template <typename T> __device__ __forceinline__ f32x4 get4(const T *p);
template <> __device__ __forceinline__ f32x4 get4<float>(const float *p) { return *(const f32x4 *)p; }
template <> __device__ __forceinline__ f32x4 get4<bf16>(const bf16 *p) {
    const uint2 u = *(const uint2 *)p;
    return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                 __uint_as_float(u.y & 0xffff0000u)};
}
}  // namespace

template <typename T, int KD, int RPT>
__global__ void __launch_bounds__(256) gdp_lin_decode_k(gdp_linattn_decode_args a) {
    constexpr int NT = 256, TPR = KD / 4, RSTEP = NT / TPR, ROWS = RSTEP * RPT;
    const int parts = a.V / ROWS;
    const int64_t req = blockIdx.x / (uint32_t)parts;
    const int hv = blockIdx.y, hk = hv / (a.HV / a.H);
    const int tid = threadIdx.x, p = tid % TPR, r0 = (int)(blockIdx.x % (uint32_t)parts) * ROWS + tid / TPR;
    const int64_t slot = a.slots ? (int64_t)a.slots[req] : req;
    T *o = (T *)a.o + ((req * a.S) * a.HV + hv) * (int64_t)a.V + r0;
    const int64_t os = (int64_t)a.HV * a.V;

    if (slot < 0 || slot >= a.pool) {  // padding entry: its rows are zero
        if (p == 0)
            for (int64_t t = 0; t < a.S; ++t)
#pragma unroll
                for (int j = 0; j < RPT; ++j) o[t * os + j * RSTEP] = from_f32<T>(0.f);
        return;
    }
    float *st = a.state + ((slot * a.HV + hv) * (int64_t)a.V + r0) * KD + 4 * p;
    f32x4 s[RPT];
#pragma unroll
    for (int j = 0; j < RPT; ++j) s[j] = *(const f32x4 *)(st + j * RSTEP * KD);

    for (int64_t t = 0; t < a.S; ++t) {
        const f32x4 k = get4<T>((const T *)a.k + req * a.k_n_stride + t * a.k_t_stride + (int64_t)hk * KD + 4 * p);
        const f32x4 q = get4<T>((const T *)a.q + req * a.q_n_stride + t * a.q_t_stride + (int64_t)hk * KD + 4 * p) * a.scale;
        const T *vp = (const T *)a.v + req * a.v_n_stride + t * a.v_t_stride + (int64_t)hv * a.V + r0;
        const float *gp = a.g ? a.g + req * a.g_n_stride + t * a.g_t_stride + hv : a.g_head ? a.g_head + hv : nullptr;
        const float alpha = gp ? expf(*gp) : 1.0f;
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            s[j] = alpha * s[j] + to_f32(vp[j * RSTEP]) * k;
            const f32x4 x = s[j] * q;
            const float sum = group_sum<TPR>((x[0] + x[1]) + (x[2] + x[3]));
            if (p == 0) o[t * os + j * RSTEP] = from_f32<T>(sum);
        }
    }
#pragma unroll
    for (int j = 0; j < RPT; ++j) *(f32x4 *)(st + j * RSTEP * KD) = s[j];
}

template <typename T, int KD>
static hipError_t launch_lin_decode_k(const gdp_linattn_decode_args &a, hipStream_t stream) {
    constexpr int RSTEP = 256 / (KD / 4);
    // 8 rows of 16 bytes in flight a thread; a step too small to fill the
    // card with those takes one, for more blocks
    const bool wide = a.n * a.HV * (a.V / (8 * RSTEP)) >= 1024 && a.V % (8 * RSTEP) == 0;
    const int rows = wide ? 8 * RSTEP : RSTEP;
    const int64_t x = a.n * (a.V / rows);
    if (x > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 grid((unsigned)x, (unsigned)a.HV);
    if (wide) hipLaunchKernelGGL((gdp_lin_decode_k<T, KD, 8>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((gdp_lin_decode_k<T, KD, 1>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_lin_decode(const gdp_linattn_decode_args &a, hipStream_t stream) {
    if (a.n == 0 || a.S == 0) return hipSuccess;
    if (a.dtype == GDP_BF16)
        return a.K == 64 ? launch_lin_decode_k<bf16, 64>(a, stream) : launch_lin_decode_k<bf16, 128>(a, stream);
    return a.K == 64 ? launch_lin_decode_k<float, 64>(a, stream) : launch_lin_decode_k<float, 128>(a, stream);
}

}  // namespace gdp

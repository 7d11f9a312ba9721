// rotary.hip -- rotary positions of queries and keys: the pair (u, v) of
// frequency i turns by the angle position * freq[i],
//   (u, v) -> scale (u cos - v sin, u sin + v cos)
// pairs (i, i + R/2) or (2i, 2i + 1) of the first R elements of every head; the
// inverse turns back, which is what the gradients take.
//
// Angles are formed in 64 bits, reduced to a part of a turn and only then
// rounded: at position 10^6 a float product would be off by 0.06.  The cosines
// and sines of a block's tokens are computed once, into LDS, for all heads of
// both tensors.
#include "rows.h"

namespace gdp {

namespace {
constexpr int RNT = 256;
constexpr int MAX_TOK = 64;
constexpr int MAX_CS = 4096;  // cosine and sine pairs in LDS: 32 KB
}  // namespace

template <typename T, int E>
__global__ void __launch_bounds__(RNT) gdp_rotary_k(Rotary p, int ntok) {
    __shared__ uint8_t code[MAX_TOK];
    __shared__ int seq[MAX_TOK];
    __shared__ double pos[MAX_TOK];
    __shared__ float2 cs[MAX_CS];
    const uint32_t r0 = blockIdx.x * (uint32_t)ntok;
    const int half = p.R / 2;
    find_rows<RNT>(p.m, r0, ntok, code, seq);
    __syncthreads();
    for (int i = threadIdx.x; i < ntok; i += RNT) {
        if (!(code[i] & ROW_IN)) continue;
        const uint32_t r = r0 + i, b = p.m.cu ? 0 : (uint32_t)seq[i], t = r - b * (p.m.cu ? 0 : p.m.T);
        if (p.positions) {
            pos[i] = (double)p.positions[b * p.pos_bs + t * p.pos_ts];
        } else {
            const int64_t first = p.m.cu ? (p.m.cu[seq[i]] < 0 ? 0 : p.m.cu[seq[i]]) : 0;
            pos[i] = (double)((int64_t)t - first + (p.offsets ? p.offsets[seq[i]] : 0));
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ntok * half; i += RNT) {
        const int tok = i / half, f = i - tok * half;
        if (!(code[tok] & ROW_IN)) continue;
        const double turns = pos[tok] * p.freq[f] * 0.15915494309189535;
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        cs[i] = make_float2(c * p.scale, (p.inverse ? -s : s) * p.scale);
    }
    __syncthreads();
    // units of a head: E elements of each of the two halves, or E elements of
    // pairs; then what is not rotated
    const int turn = p.interleaved ? p.R / E : half / E, rest = (p.D - p.R) / E, per = turn + rest;
    const int heads = p.H[0] + p.H[1], items = heads * per;
    for (int it = threadIdx.x; it < ntok * items; it += RNT) {
        const int tok = it / items, w = it - tok * items, head = w / per, u = w - head * per;
        if (!(code[tok] & ROW_IN)) continue;
        const int which = head >= p.H[0];
        const int64_t col = (int64_t)(head - (which ? p.H[0] : 0)) * p.D;
        const uint32_t r = r0 + tok, b = p.m.cu ? 0 : (uint32_t)seq[tok], t = r - b * (p.m.cu ? 0 : p.m.T);
        const Strided &si = p.in[which], &so = p.out[which];
        const T *in = (const T *)si.p + b * si.bs + t * si.ts + col;
        T *out = (T *)so.p + b * so.bs + t * so.ts + col;
        Chans<T, E> a, c;
        if (u >= turn) {
            a.load(in + p.R + (u - turn) * E);
            a.store(out + p.R + (u - turn) * E);
            continue;
        }
        float x[E], y[E];
        if (!p.interleaved) {
            a.load(in + u * E);
            c.load(in + half + u * E);
            a.to(x);
            c.to(y);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float2 z = cs[tok * half + u * E + e];
                const float v = x[e];
                x[e] = v * z.x - y[e] * z.y;
                y[e] = v * z.y + y[e] * z.x;
            }
            a.from(x);
            c.from(y);
            a.store(out + u * E);
            c.store(out + half + u * E);
        } else if constexpr (E > 1) {
            a.load(in + u * E);
            a.to(x);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 z = cs[tok * half + (u * E + e) / 2];
                const float v = x[e];
                x[e] = v * z.x - x[e + 1] * z.y;
                x[e + 1] = v * z.y + x[e + 1] * z.x;
            }
            a.from(x);
            a.store(out + u * E);
        } else if (u % 2 == 0) {  // a pair by its first element
            a.load(in + u);
            c.load(in + u + 1);
            a.to(x);
            c.to(y);
            const float2 z = cs[tok * half + u / 2];
            const float v = x[0];
            x[0] = v * z.x - y[0] * z.y;
            y[0] = v * z.y + y[0] * z.x;
            a.from(x);
            c.from(y);
            a.store(out + u);
            c.store(out + u + 1);
        }
    }
}

hipError_t launch_rotary(const Rotary &p, gdp_dtype dtype, hipStream_t stream) {
    const int half = p.R / 2;
    int ntok = half > 0 ? MAX_CS / half : MAX_TOK;
    ntok = ntok > 8 ? 8 : ntok;
    const int64_t blocks = ((int64_t)p.m.rows + ntok - 1) / ntok;
    if (blocks == 0) return hipSuccess;
    if (blocks * RNT > 0xffffffffll) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks);
    if (dtype == GDP_BF16) {
        if (p.vec) hipLaunchKernelGGL((gdp_rotary_k<bf16, 8>), grid, dim3(RNT), 0, stream, p, ntok);
        else hipLaunchKernelGGL((gdp_rotary_k<bf16, 1>), grid, dim3(RNT), 0, stream, p, ntok);
    } else {
        if (p.vec) hipLaunchKernelGGL((gdp_rotary_k<float, 4>), grid, dim3(RNT), 0, stream, p, ntok);
        else hipLaunchKernelGGL((gdp_rotary_k<float, 1>), grid, dim3(RNT), 0, stream, p, ntok);
    }
    return hipGetLastError();
}

}  // namespace gdp

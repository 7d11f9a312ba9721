// rotary.hip -- rotary positions of queries and keys: the pair (u, v) of
// frequency i turns by the angle position * freq[i],
//   (u, v) -> scale (u cos - v sin, u sin + v cos)
// pairs (i, i + R/2) or (2i, 2i + 1) of the first R elements of every head; the
// inverse turns back, which is what the gradients take.
//
// Angles are formed in 64 bits, reduced to a part of a turn and only then
// rounded: at position 10^6 a float product would be off by 0.06.  The cosines
// and sines of a block's tokens are computed once, into LDS, for all heads of
// both tensors.  What is left is to move them: 32768 tokens of 16 + 16 heads of
// 128, half of each turned, 101 us (537 MB, 5.3 TB/s; a large copy reaches 5.1);
// 15151 packed tokens of 16 + 4 heads 32; a single token 3, and the host 10.
#include "rows.h"

namespace gdp {

namespace {

constexpr int RNT = 256;
constexpr int MAX_TOK = 64;
constexpr int MAX_CS = 4096;  // cosine and sine pairs of a block: 32 KB of LDS

// What a thread turns of a head: E elements of both halves, or E elements of
// neighbouring pairs (a pair where E is 1); or it copies E that are not turned.
template <typename T, int E, bool INTER>
struct Piece {
    Chans<T, E> a, c;
    __device__ __forceinline__ void load(const T *p, int second) {
        a.load(p);
        if (second) c.load(p + second);
    }
    __device__ __forceinline__ void store(T *p, int second) const {
        a.store(p);
        if (second) c.store(p + second);
    }
    __device__ __forceinline__ void turn(const float2 *cs) {
        float x[E], y[E];
        a.to(x);
        if constexpr (INTER && E > 1) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 z = cs[e / 2];
                const float v = x[e];
                x[e] = v * z.x - x[e + 1] * z.y;
                x[e + 1] = v * z.y + x[e + 1] * z.x;
            }
            a.from(x);
        } else {
            c.to(y);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float2 z = cs[e];
                const float v = x[e];
                x[e] = v * z.x - y[e] * z.y;
                y[e] = v * z.y + y[e] * z.x;
            }
            a.from(x);
            c.from(y);
        }
    }
};

}  // namespace

// lanes: threads side by side on the pieces of a token (a power of two)
template <typename T, int E, bool INTER>
__global__ void __launch_bounds__(RNT) gdp_rotary_k(Rotary p, int ntok, int lanes_log) {
    __shared__ uint8_t code[MAX_TOK];
    __shared__ int seq[MAX_TOK];
    __shared__ double pos[MAX_TOK];
    extern __shared__ float2 cs[];  // [ntok][R / 2]
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
    constexpr int STEP = INTER && E == 1 ? 2 : E;  // elements from one turned piece to the next
    const int turned = INTER ? p.R / STEP : half / E, per = turned + (p.D - p.R) / E;
    const int pieces = (p.H[0] + p.H[1]) * per, lanes = 1 << lanes_log, rows = RNT >> lanes_log;
    for (int w = threadIdx.x & (lanes - 1); w < pieces; w += lanes) {
        const int head = w / per, u = w - head * per, which = head >= p.H[0];
        const bool turn = u < turned;
        const int at = turn ? u * STEP : p.R + (u - turned) * E, second = !turn || (INTER && E > 1) ? 0 : INTER ? 1 : half;
        const int64_t col = (int64_t)(head - (which ? p.H[0] : 0)) * p.D + at;
        const int f = INTER ? at / 2 : at;  // first frequency of the piece
        const Strided &si = p.in[which], &so = p.out[which];
        if (!turn && si.p == so.p) continue;  // already there
        const auto place = [&](const Strided &s, int tok) {
            const uint32_t r = r0 + tok, b = p.m.cu ? 0 : (uint32_t)seq[tok], t = r - b * (p.m.cu ? 0 : p.m.T);
            return (T *)s.p + b * s.bs + t * s.ts + col;
        };
        // a few tokens' loads under way together (32768 x 32 heads interleaved, of 2 / 4 / 8 tokens 100 / 98 / 114 us;
        // halves are two loads: 15151 x 20 heads, 1 / 2 / 4 pairs of loads 29 / 27 / 31)
        constexpr int N = INTER && E > 1 ? 4 : 2;
        for (int t0 = threadIdx.x >> lanes_log; t0 < ntok; t0 += N * rows) {
            Piece<T, E, INTER> x[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int tok = t0 + j * rows;
                if (tok < ntok && (code[tok] & ROW_IN)) x[j].load(place(si, tok), second);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int tok = t0 + j * rows;
                if (tok < ntok && (code[tok] & ROW_IN)) {
                    if (turn) x[j].turn(cs + tok * half + f);
                    x[j].store(place(so, tok), second);
                }
            }
        }
    }
}

namespace {
template <typename T, int E>
hipError_t run_rotary(const Rotary &p, int ntok, int lanes_log, hipStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)p.m.rows + ntok - 1) / ntok));
    const size_t lds = (size_t)ntok * (p.R / 2) * sizeof(float2);
    if (p.interleaved) hipLaunchKernelGGL((gdp_rotary_k<T, E, true>), grid, dim3(RNT), lds, stream, p, ntok, lanes_log);
    else hipLaunchKernelGGL((gdp_rotary_k<T, E, false>), grid, dim3(RNT), lds, stream, p, ntok, lanes_log);
    return hipGetLastError();
}
// Elements of a piece, threads side by side on a token's, and tokens of a block:
// four or eight for every thread, few enough for 1024 blocks (one alone: a step
// of a few tokens is all latency) and for LDS.
struct Shape {
    int E, lanes_log, ntok;
    Shape(const Rotary &p, gdp_dtype dtype) : E(!p.vec ? 1 : dtype == GDP_BF16 ? 8 : 4), lanes_log(0) {
        const int half = p.R / 2, turned = p.interleaved ? p.R / (E == 1 ? 2 : E) : half / E;
        const int64_t pieces = (int64_t)(p.H[0] + p.H[1]) * (turned + (p.D - p.R) / E);
        while (lanes_log < 8 && (1 << lanes_log) < pieces) ++lanes_log;
        ntok = 8 * (RNT >> lanes_log);
        while (ntok > 1 && p.m.rows / ntok < 1024) ntok /= 2;
        ntok = ntok > MAX_TOK ? MAX_TOK : ntok;
        ntok = ntok > MAX_CS / half ? MAX_CS / half : ntok;
    }
};
}  // namespace

bool rotary_fits(const Rotary &p, gdp_dtype dtype) {
    const int ntok = Shape(p, dtype).ntok;
    return ((int64_t)p.m.rows + ntok - 1) / ntok * RNT <= 0xffffffffll;
}
hipError_t launch_rotary(const Rotary &p, gdp_dtype dtype, hipStream_t stream) {
    if (p.m.rows == 0) return hipSuccess;
    const Shape s(p, dtype);
    if (dtype == GDP_BF16)
        return s.E == 8 ? run_rotary<bf16, 8>(p, s.ntok, s.lanes_log, stream) : run_rotary<bf16, 1>(p, s.ntok, s.lanes_log, stream);
    return s.E == 4 ? run_rotary<float, 4>(p, s.ntok, s.lanes_log, stream) : run_rotary<float, 1>(p, s.ntok, s.lanes_log, stream);
}

}  // namespace gdp

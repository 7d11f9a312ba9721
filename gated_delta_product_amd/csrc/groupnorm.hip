// groupnorm.hip -- group norm with an activation, channels last, every token a
// sample of its own (the norm per head that follows a token mixer).
//
//   xh = (x - mean) rstd  over the D channels of a group (or x rstd),  u = xh w + b
//   y  = u act(z)  or  act(u)
// and with du the gradient of u (dy act(z), or dy act'(u)) and dxh = du w:
//   dx = rstd (dxh - mean(dxh) - xh mean(dxh xh)),  dz = dy u act'(z)
//   dw = sum over tokens of du xh,  db = sum over tokens of du
//
// LPG neighbouring lanes hold a group, NU units of 16 bytes each (of one
// element where a row is not made of aligned units), so a group is read once
// and reduced inside a wave; neighbouring groups of a token sit in
// neighbouring lanes.  Both directions move each tensor once and are bound by
// that: 32768 rows of 16 x 128 bf16 with a gate, forwards 82 us (403 MB, 4.9
// TB/s, a large copy reaching 5.1), backwards 140 us (671 MB, 4.8 TB/s;
// three inputs, the next row's too, and two sums a channel take 111 registers).
// 256 such rows take 5 us, 2048 x 1024 backwards 14 and 5 for the sums.
// Slower: gradients where the groups do not divide a block's row sets (any but
// a power of two), whose partial sums are not joined (5.5 M elements, gated: 3 x 40
// channels 164 us, 4 x 40 34; 3 x 128 67, 4 x 128 25; 24 x 128 28, 16 x 128 26), and
// groups of over 1024 channels, which one wave holds: from 2049 on the gradients
// spill (8192 rows of one group of 4096: 69 us forwards, 378 backwards, where 32
// groups of 128 take 38 and 83).
#include "gdp_common.h"
#include "gdp_internal.h"
#include "groupnorm.h"

namespace gdp {

namespace {

constexpr int GNT = 256;

template <typename T, int E> struct Unit;
template <> struct Unit<bf16, 8> { typedef uint4 type; };
template <> struct Unit<float, 4> { typedef uint4 type; };
template <> struct Unit<bf16, 1> { typedef bf16 type; };
template <> struct Unit<float, 1> { typedef float type; };

// The units of a lane, as they lie in memory; lanes past the group hold zeros.
template <typename T, int E, int LPG, int NU>
struct Raw {
    typedef typename Unit<T, E>::type U;
    U u[NU];
    __device__ __forceinline__ void load(const T *p, int l, int D) {
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int d = (l + k * LPG) * E;
            u[k] = U{};
            if (d < D) u[k] = *(const U *)(p + d);
        }
    }
    __device__ __forceinline__ void floats(float *f) const {
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const U v = u[k];
            const T *e = (const T *)&v;
#pragma unroll
            for (int i = 0; i < E; ++i) f[k * E + i] = to_f32(e[i]);
        }
    }
};
template <typename T, int E>
__device__ __forceinline__ void put(T *p, const float *f) {
    typedef typename Unit<T, E>::type U;
    U u;
    T *e = (T *)&u;
#pragma unroll
    for (int i = 0; i < E; ++i) e[i] = from_f32<T>(f[i]);
    *(U *)p = u;
}

__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }
__device__ __forceinline__ float act(int kind, float x) {
    if (kind == GDP_ACT_NONE) return x;
    const float s = sigmoid(x);
    return kind == GDP_ACT_SILU ? x * s : s;
}
__device__ __forceinline__ float act_slope(int kind, float x) {
    if (kind == GDP_ACT_NONE) return 1.0f;
    const float s = sigmoid(x);
    return kind == GDP_ACT_SILU ? s * (1.0f + x * (1.0f - s)) : s * (1.0f - s);
}

__device__ __forceinline__ int64_t row_at(uint32_t row, uint32_t T, int64_t ns, int64_t ts) {
    const uint32_t n = row / T;
    return (int64_t)n * ns + (int64_t)(row - n * T) * ts;
}

// x of one group into xh (normalised) and its rstd
template <int N, int LPG>
__device__ __forceinline__ float normalise(float (&x)[N], const bool (&in)[N], int D, float eps, bool centered) {
    const float inv = 1.0f / (float)D;
    if (centered) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) s += x[i];  // lanes past the group hold zeros
        const float mean = group_sum<LPG>(s) * inv;
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = in[i] ? x[i] - mean : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) q += x[i] * x[i];
    const float rstd = 1.0f / sqrtf(group_sum<LPG>(q) * inv + eps);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= rstd;
    return rstd;
}

}  // namespace

template <typename T, int E, int LPG, int NU, bool GATE>
__global__ void __launch_bounds__(GNT) gdp_group_norm_k(GroupNorm p) {
    constexpr int N = E * NU;
    const int64_t set = ((int64_t)blockIdx.x * GNT + threadIdx.x) / LPG;
    const int l = threadIdx.x % LPG;
    const uint32_t gi = (uint32_t)(set % p.groups);
    const int64_t r0 = set / p.groups;
    if (r0 >= p.split) return;
    const int col = (int)gi * p.D;
    bool in[N];
    float w[N], b[N];
#pragma unroll
    for (int k = 0; k < NU; ++k) {
        const int d = (l + k * LPG) * E;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            in[k * E + i] = d < p.D;
            w[k * E + i] = p.w && d < p.D ? p.w[col + d + i] : 1.f;
            b[k * E + i] = p.b && d < p.D ? p.b[col + d + i] : 0.f;
        }
    }
    // the next row's loads are in flight while a row is worked on (wide groups
    // have no registers for it)
    constexpr bool AHEAD = N <= 16;
    Raw<T, E, LPG, NU> rx, rz;
    auto load = [&](int64_t row) {
        rx.load((const T *)p.x + row_at((uint32_t)row, p.T, p.x_ns, p.x_ts) + col, l, p.D);
        if constexpr (GATE) rz.load((const T *)p.z + row_at((uint32_t)row, p.T, p.z_ns, p.z_ts) + col, l, p.D);
    };
    if constexpr (AHEAD) load(r0);
    for (int64_t row = r0; row < p.rows; row += p.split) {
        if constexpr (!AHEAD) load(row);
        float v[N], zv[GATE ? N : 1];
        rx.floats(v);
        if constexpr (GATE) rz.floats(zv);
        if (AHEAD && row + p.split < p.rows) load(row + p.split);
        normalise<N, LPG>(v, in, p.D, p.eps, p.centered);
        T *y = (T *)p.y + row * ((int64_t)p.groups * p.D) + col;
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int d = (l + k * LPG) * E;
            if (d >= p.D) continue;
            float o[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float u = v[k * E + i] * w[k * E + i] + b[k * E + i];
                o[i] = GATE ? u * act(p.act, zv[GATE ? k * E + i : 0]) : act(p.act, u);
            }
            put<T, E>(y + d, o);
        }
    }
}

// Threads of a block backwards: with few elements a thread, large blocks hold
// the same channels of several rows (p.join) and add those up in LDS before
// they write partial sums.
constexpr int bwd_threads(int n) { return n <= 8 ? 512 : 256; }

template <typename T, int E, int LPG, int NU, bool GATE>
__global__ void __launch_bounds__(bwd_threads(E * NU)) gdp_group_norm_bwd_k(GroupNorm p) {
    constexpr int N = E * NU, NT = bwd_threads(N);
    const int64_t set = ((int64_t)blockIdx.x * NT + threadIdx.x) / LPG;
    const int l = threadIdx.x % LPG;
    const uint32_t gi = (uint32_t)(set % p.groups);
    const int64_t r0 = set / p.groups;
    const bool any = r0 < p.split;
    if (!any && p.join == 1) return;
    const int col = (int)gi * p.D;
    const int64_t C = (int64_t)p.groups * p.D;
    const float inv = 1.0f / (float)p.D;
    bool in[N];
    float w[N], b[N], dw[N], db[N];
#pragma unroll
    for (int k = 0; k < NU; ++k) {
        const int d = (l + k * LPG) * E;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            in[k * E + i] = d < p.D;
            w[k * E + i] = p.w && d < p.D ? p.w[col + d + i] : 1.f;
            b[k * E + i] = p.b && d < p.D ? p.b[col + d + i] : 0.f;
            dw[k * E + i] = db[k * E + i] = 0.f;
        }
    }
    constexpr bool AHEAD = N <= 16;
    Raw<T, E, LPG, NU> rx, rz, ry;
    auto load = [&](int64_t row) {
        rx.load((const T *)p.x + row_at((uint32_t)row, p.T, p.x_ns, p.x_ts) + col, l, p.D);
        ry.load((const T *)p.dy + row_at((uint32_t)row, p.T, p.dy_ns, p.dy_ts) + col, l, p.D);
        if constexpr (GATE) rz.load((const T *)p.z + row_at((uint32_t)row, p.T, p.z_ns, p.z_ts) + col, l, p.D);
    };
    if (AHEAD && any) load(r0);
    for (int64_t row = any ? r0 : p.rows; row < p.rows; row += p.split) {
        if constexpr (!AHEAD) load(row);
        float v[N], dv[N], zv[GATE ? N : 1];
        rx.floats(v);
        ry.floats(dv);
        if constexpr (GATE) rz.floats(zv);
        if (AHEAD && row + p.split < p.rows) load(row + p.split);
        const float rstd = normalise<N, LPG>(v, in, p.D, p.eps, p.centered);
        const int64_t at = row * C + col;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int d = (l + k * LPG) * E;
            float dz[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int j = k * E + i;
                const float u = v[j] * w[j] + b[j], g = dv[j];
                float du;
                if constexpr (GATE) {
                    du = g * act(p.act, zv[j]);
                    dz[i] = g * u * act_slope(p.act, zv[j]);
                } else {
                    du = g * act_slope(p.act, u);
                }
                dw[j] += du * v[j];
                db[j] += du;
                dv[j] = du * w[j];  // dxh
                s1 += dv[j];
                s2 += dv[j] * v[j];
            }
            if constexpr (GATE)
                if (d < p.D) put<T, E>((T *)p.dz + at + d, dz);
        }
        const float m1 = p.centered ? group_sum<LPG>(s1) * inv : 0.f, m2 = group_sum<LPG>(s2) * inv;
#pragma unroll
        for (int k = 0; k < NU; ++k) {
            const int d = (l + k * LPG) * E;
            if (d >= p.D) continue;
            float o[E];
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = rstd * (dv[k * E + i] - m1 - v[k * E + i] * m2);
            put<T, E>((T *)p.dx + at + d, o);
        }
    }
    if (!p.part) return;
    if constexpr (NT > GNT) {
        if (p.join > 1) {
            // the block's p.join row sets, one after the other in lanes, for each of dw and db
            __shared__ float red[NT * N];
            const int per = p.groups * LPG;
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                float *v = which ? db : dw;
                if (which) __syncthreads();
#pragma unroll
                for (int i = 0; i < N; ++i) red[i * NT + threadIdx.x] = v[i];
                __syncthreads();
                if ((int)threadIdx.x < per)
                    for (int j = 1; j < p.join; ++j)
#pragma unroll
                        for (int i = 0; i < N; ++i) v[i] += red[i * NT + threadIdx.x + j * per];
            }
            if ((int)threadIdx.x >= per) return;
        }
    }
    // these rows, for the thread's channels: [split / join][2][C]
    float *part = p.part + r0 / p.join * 2 * C + col;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
        const int d = (l + k * LPG) * E;
        if (d >= p.D) continue;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            part[d + i] = dw[k * E + i];
            part[C + d + i] = db[k * E + i];
        }
    }
}

// dw and db: the partial sums of every split, in a fixed order.  64 channels
// a block, its 16 waves every 16th split each, 16 of them in flight.
constexpr int GSW = 16;
__global__ void __launch_bounds__(64 * GSW) gdp_group_norm_sum_k(const float *part, int64_t split, int64_t C, float *dw,
                                                                 float *db) {
    __shared__ double s[GSW][64];
    const int64_t c = (int64_t)blockIdx.x * 64 + lane_id();
    const int which = blockIdx.y;
    float *out = which ? db : dw;
    if (!out) return;
    const float *q = part + which * C + c;
    double x = 0.0;
    if (c < C)
        for (int64_t i = wave_id(); i < split; i += 16 * GSW) {
            float f[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = i + j * GSW < split ? q[(i + j * GSW) * 2 * C] : 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) x += f[j];
        }
    s[wave_id()][lane_id()] = x;
    __syncthreads();
    if (wave_id() == 0 && c < C) {
        double t = 0.0;
        for (int w = 0; w < GSW; ++w) t += s[w][lane_id()];
        out[c] = (float)t;
    }
}

namespace {

struct Shape {
    bool vec;
    int units, lpg, nu;
};
Shape shape_of(const GroupNorm &p, gdp_dtype dtype) {
    Shape s;
    const int e = dtype == GDP_BF16 ? 8 : 4;
    s.vec = p.vec && p.D % e == 0;
    s.units = s.vec ? p.D / e : p.D;
    s.lpg = 1;
    while (s.lpg < 64 && s.lpg < s.units) s.lpg *= 2;
    s.nu = 1;
    while (s.nu * s.lpg < s.units) s.nu *= 2;
    return s;
}

template <typename T, int E, int LPG, int NU>
hipError_t launch(GroupNorm &p, hipStream_t stream) {
    const int nt = p.bwd ? bwd_threads(E * NU) : GNT, sets = nt / LPG;
    p.join = p.bwd && nt > GNT && sets % p.groups == 0 ? sets / p.groups : 1;
    const int64_t blocks = (p.split * p.groups * LPG + nt - 1) / nt;
    if (blocks * nt > 0xffffffffll) return hipErrorInvalidValue;
    if (blocks == 0) return hipSuccess;
    const dim3 grid((unsigned)blocks);
    if (!p.bwd) {
        if (p.z) hipLaunchKernelGGL((gdp_group_norm_k<T, E, LPG, NU, true>), grid, dim3(GNT), 0, stream, p);
        else hipLaunchKernelGGL((gdp_group_norm_k<T, E, LPG, NU, false>), grid, dim3(GNT), 0, stream, p);
    } else {
        if (p.z) hipLaunchKernelGGL((gdp_group_norm_bwd_k<T, E, LPG, NU, true>), grid, dim3(nt), 0, stream, p);
        else hipLaunchKernelGGL((gdp_group_norm_bwd_k<T, E, LPG, NU, false>), grid, dim3(nt), 0, stream, p);
    }
    return hipGetLastError();
}

template <typename T, int E>
hipError_t launch_shape(GroupNorm &p, const Shape &s, hipStream_t stream) {
    if (s.nu == 1) {
        switch (s.lpg) {
        case 1: return launch<T, E, 1, 1>(p, stream);
        case 2: return launch<T, E, 2, 1>(p, stream);
        case 4: return launch<T, E, 4, 1>(p, stream);
        case 8: return launch<T, E, 8, 1>(p, stream);
        case 16: return launch<T, E, 16, 1>(p, stream);
        case 32: return launch<T, E, 32, 1>(p, stream);
        case 64: return launch<T, E, 64, 1>(p, stream);
        }
    }
    switch (s.nu) {
    case 2: return launch<T, E, 64, 2>(p, stream);
    case 4: return launch<T, E, 64, 4>(p, stream);
    case 8: return launch<T, E, 64, 8>(p, stream);
    case 16: if constexpr (E != 8) return launch<T, E, 64, 16>(p, stream); break;
    case 32: if constexpr (E == 1) return launch<T, E, 64, 32>(p, stream); break;
    case 64: if constexpr (E == 1) return launch<T, E, 64, 64>(p, stream); break;
    }
    return hipErrorInvalidValue;
}

}  // namespace

// Row sets that run side by side: threads of one set walk rows r0, r0 + split, ...
int64_t group_norm_split(int64_t rows, int groups, int D, bool bwd) {
    // about 16 rows a thread forwards once the card is full (32768 x 2048: 4 / 8
    // / 16 / 32 rows 107 / 95 / 90 / 91 us).  Backwards no more threads than two
    // waves a SIMD (each set of rows costs 8 bytes a channel of partial sums;
    // one, two or three times as many 154, 163, 166 us, and 173 with one block
    // too many, that runs alone at the end) and at least 4 rows.  Both rules count
    // 8 elements a thread, which holds for aligned bf16 groups of at most 512
    // channels; float32 runs twice as many threads, single elements (rows that do
    // not start on 16 bytes) up to eight times, wider groups fewer.
    const int64_t fill = (bwd ? 131072 : 262144) * 8 / ((int64_t)groups * D);
    const int64_t few = (rows + (bwd ? 3 : 15)) / (bwd ? 4 : 16);
    int64_t s = bwd ? (few < fill ? few : fill) : (few > fill ? few : fill);
    s = s < 1 ? 1 : s;
    if (s >= rows) return rows;
    const int64_t each = (rows + s - 1) / s;  // as many rows for every thread
    return (rows + each - 1) / each;
}

hipError_t launch_group_norm(GroupNorm p, gdp_dtype dtype, hipStream_t stream) {
    const Shape s = shape_of(p, dtype);
    hipError_t e;
    if (dtype == GDP_BF16) e = s.vec ? launch_shape<bf16, 8>(p, s, stream) : launch_shape<bf16, 1>(p, s, stream);
    else e = s.vec ? launch_shape<float, 4>(p, s, stream) : launch_shape<float, 1>(p, s, stream);
    if (e != hipSuccess || !(p.dw || p.db)) return e;
    const int64_t C = (int64_t)p.groups * p.D;
    hipLaunchKernelGGL(gdp_group_norm_sum_k, dim3((unsigned)((C + 63) / 64), 2), dim3(64 * GSW), 0, stream, p.part,
                       (p.split + p.join - 1) / p.join, C, p.dw, p.db);
    return hipGetLastError();
}

}  // namespace gdp

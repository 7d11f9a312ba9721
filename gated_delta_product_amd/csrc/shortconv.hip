// shortconv.hip -- short causal convolution, channels last, W taps a channel:
//   u_t = b + sum_j w_j x_{t-W+1+j},  y_t = act(u_t)
// where the rows before a sequence come from its state, the W - 1 inputs
// before it (oldest first), and with du = dy act'(u):
//   dx_s = sum_j w_j du_{s+W-1-j},  dw_j = sum_t du_t x_{t-W+1+j},  db = sum du
//
// A thread walks TT rows of E channels with the last W - 1 rows in registers.
#include "rows.h"

namespace gdp {

namespace {

constexpr int CNT = 256;
constexpr int CTT = 16;

// A thread's place: channels col .. col + E of the rows row0 .. row0 + TT;
// 2^lognx threads side by side hold a row of the block.
template <int NT, int E, int TT>
struct Spot {
    int nx, ny, tx, ty, col;
    uint32_t tile0, row0;
    bool live;
    __device__ __forceinline__ Spot(int lognx, int C, uint32_t tile, uint32_t strip) {
        nx = 1 << lognx;
        ny = NT >> lognx;
        tx = threadIdx.x & (nx - 1);
        ty = threadIdx.x >> lognx;
        col = (int)((strip << lognx) + tx) * E;
        live = col < C;
        tile0 = tile * (uint32_t)(ny * TT);
        row0 = tile0 + ty * TT;
    }
};

// The W - 1 inputs before a row, oldest first.
template <typename T, int E, int W>
struct Window {
    float v[W - 1][E];
    // of the row with this code, in sequence seq (anything where it is in none)
    __device__ __forceinline__ void start(const ShortConv &p, uint32_t row, uint32_t code, int seq, int col) {
        const int before = (int)rows_before(code);
#pragma unroll
        for (int k = 1; k < W; ++k) {
            Chans<T, E> r;
            r.zero();
            if (!(code & ROW_IN)) {
            } else if (k <= before) {
                const RowWalk<T> at(p.x, p.m, row - k, col);
                r.load(at.p);
            } else if (p.h0) {
                r.load((const T *)p.h0 + ((int64_t)seq * (W - 1) + (W - 1 - k + before)) * p.C + col);
            }
            r.to(v[W - 1 - k]);
        }
    }
    __device__ __forceinline__ void push(const float (&x)[E]) {
#pragma unroll
        for (int k = 0; k + 2 < W; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) v[k][e] = v[k + 1][e];
#pragma unroll
        for (int e = 0; e < E; ++e) v[W - 2][e] = x[e];
    }
};

template <int E, int W>
struct Taps {
    float w[E][W], b[E];
    __device__ __forceinline__ void load(const float *pw, const float *pb, int col) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[e][j] = pw[(int64_t)(col + e) * W + j];
            b[e] = pb ? pb[col + e] : 0.f;
        }
    }
    template <typename T>
    __device__ __forceinline__ float at(const Window<T, E, W> &win, const float (&x)[E], int e) const {
        float u = b[e];
#pragma unroll
        for (int j = 0; j + 1 < W; ++j) u = fmaf(w[e][j], win.v[j][e], u);
        return fmaf(w[e][W - 1], x[e], u);
    }
};

// Final states (or dh0 from dht) of the empty sequences: those before them.
template <typename T, int E, int W>
__device__ __forceinline__ void empty_states(const RowMap &m, const void *from, void *to, int C, int col) {
    for (int q = blockIdx.x; q < m.nseq; q += gridDim.x)
        if (seq_empty(m, q))
            for (int k = 0; k < W - 1; ++k) {
                Chans<T, E> r;
                r.zero();
                const int64_t at = ((int64_t)q * (W - 1) + k) * C + col;
                if (from) r.load((const T *)from + at);
                r.store((T *)to + at);
            }
}

}  // namespace

template <typename T, int E, int W>
__global__ void __launch_bounds__(CNT) gdp_conv_k(ShortConv p) {
    constexpr int TT = CTT;
    __shared__ uint8_t code[CNT * TT];
    __shared__ int seq[CNT * TT];
    const Spot<CNT, E, TT> at(p.lognx, p.C, blockIdx.x, blockIdx.y);
    find_rows<CNT>(p.m, at.tile0, at.ny * TT, code, seq);
    __syncthreads();
    if (!at.live) return;
    Taps<E, W> f;
    f.load(p.w, p.b, at.col);
    const int k0 = at.ty * TT;
    Window<T, E, W> win;
    win.start(p, at.row0, code[k0], seq[k0], at.col);
    RowWalk<T> in(p.x, p.m, at.row0, at.col);
    for (int i = 0; i < TT; ++i, in.next()) {
        const uint32_t c = code[k0 + i];
        if (!(c & ROW_IN)) continue;
        if (row_first(c)) win.start(p, at.row0 + i, c, seq[k0 + i], at.col);
        Chans<T, E> r;
        float x[E], y[E];
        r.load(in.p);
        r.to(x);
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = act_exact(p.act, f.at(win, x, e));
        win.push(x);
        r.from(y);
        r.store((T *)p.y + (int64_t)(at.row0 + i) * p.C + at.col);
        if (p.ht && row_last(c))
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                r.from(win.v[k]);
                r.store((T *)p.ht + ((int64_t)seq[k0 + i] * (W - 1) + k) * p.C + at.col);
            }
    }
    if (p.ht && at.ty == 0) empty_states<T, E, W>(p.m, p.h0, p.ht, p.C, at.col);
}

template <typename T, int E, int W>
__global__ void __launch_bounds__(CNT) gdp_conv_bwd_k(ShortConv p) {
    constexpr int TT = CTT, X = W - 1;
    __shared__ uint8_t code[CNT * TT + X];
    __shared__ int seq[CNT * TT + X];
    __shared__ float red[CNT * E];
    const Spot<CNT, E, TT> at(p.lognx, p.C, blockIdx.x, blockIdx.y);
    find_rows<CNT>(p.m, at.tile0, at.ny * TT + X, code, seq);
    __syncthreads();
    float dw[W][E], db[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
    }
    if (at.live) {
        Taps<E, W> f;
        f.load(p.w, p.b, at.col);
        const int k0 = at.ty * TT;
        Window<T, E, W> win;
        win.start(p, at.row0, code[k0], seq[k0], at.col);
        RowWalk<T> in(p.x, p.m, at.row0, at.col), dn(p.dy, p.m, at.row0, at.col);
        float du[W][E];  // of the rows r - X .. r
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < E; ++e) du[j][e] = 0.f;
        for (int i = 0; i < TT + X; ++i, in.next(), dn.next()) {
            const uint32_t c = code[k0 + i];
#pragma unroll
            for (int j = 0; j < X; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) du[j][e] = du[j + 1][e];
            if (c & ROW_IN) {
                if (row_first(c)) win.start(p, at.row0 + i, c, seq[k0 + i], at.col);
                Chans<T, E> r;
                float x[E], d[E];
                r.load(in.p);
                r.to(x);
                r.load(dn.p);
                r.to(d);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float u = d[e] * act_slope_exact(p.act, f.at(win, x, e));
                    du[X][e] = u;
                    if (i < TT) {
                        db[e] += u;
#pragma unroll
                        for (int j = 0; j < X; ++j) dw[j][e] = fmaf(u, win.v[j][e], dw[j][e]);
                        dw[X][e] = fmaf(u, x[e], dw[X][e]);
                    }
                }
                win.push(x);
            }
            if (i < X) continue;
            // row s = r - X: its du and those of the rows behind it are du[0 .. X]
            const uint32_t s = at.row0 + i - X, cs = code[k0 + i - X];
            if (s >= p.m.rows) continue;
            const int behind = (int)rows_behind(cs), q = seq[k0 + i - X];
            Chans<T, E> r;
            float dx[E];
#pragma unroll
            for (int e = 0; e < E; ++e) dx[e] = 0.f;
            if (cs & ROW_IN) {
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (j <= behind)
#pragma unroll
                        for (int e = 0; e < E; ++e) dx[e] = fmaf(f.w[e][X - j], du[j][e], dx[e]);
                if (p.dht && behind < X) {
                    float z[E];
                    r.load((const T *)p.dht + ((int64_t)q * X + X - 1 - behind) * p.C + at.col);
                    r.to(z);
#pragma unroll
                    for (int e = 0; e < E; ++e) dx[e] += z[e];
                }
                if (p.dh0 && row_first(cs))
#pragma unroll
                    for (int k = 0; k < X; ++k) {  // state row k: read by the taps k - d of the rows d behind the first
                        float z[E];
#pragma unroll
                        for (int e = 0; e < E; ++e) z[e] = 0.f;
                        if (p.dht && k > behind) {  // a sequence so short that its final state still holds the row
                            r.load((const T *)p.dht + ((int64_t)q * X + k - 1 - behind) * p.C + at.col);
                            r.to(z);
                        }
#pragma unroll
                        for (int d = 0; d <= k; ++d)
                            if (d <= behind)
#pragma unroll
                                for (int e = 0; e < E; ++e) z[e] = fmaf(f.w[e][k - d], du[d][e], z[e]);
                        r.from(z);
                        r.store((T *)p.dh0 + ((int64_t)q * X + k) * p.C + at.col);
                    }
            }
            r.from(dx);
            r.store((T *)p.dx + (int64_t)s * p.C + at.col);
        }
        if (p.dh0 && at.ty == 0) empty_states<T, E, W>(p.m, p.dht, p.dh0, p.C, at.col);
    }
    if (!p.part) return;
    // the block's rows: [tiles][W + 1][C]
    const int w = at.nx * E, c = (int)(blockIdx.y * w) + (int)threadIdx.x;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) red[at.ty * w + at.tx * E + e] = j < W ? dw[j < W ? j : 0][e] : db[e];
        __syncthreads();
        for (int k = threadIdx.x; k < w; k += CNT) {
            float t = 0.f;
            for (int y = 0; y < at.ny; ++y) t += red[y * w + k];
            if (c - (int)threadIdx.x + k < p.C)
                p.part[((int64_t)blockIdx.x * (W + 1) + j) * p.C + c - threadIdx.x + k] = t;
        }
    }
}

// dw [C, W] and db [C]: the partial sums of every tile, in a fixed order.  64
// channels of a tap a block, its 16 waves every 16th tile each.
constexpr int CSW = 16;
__global__ void __launch_bounds__(64 * CSW) gdp_conv_sum_k(const float *part, int64_t tiles, int64_t C, int W, float *dw,
                                                          float *db) {
    __shared__ double s[CSW][64];
    const int64_t c = (int64_t)blockIdx.x * 64 + lane_id();
    const int j = blockIdx.y;
    if (j < W ? !dw : !db) return;
    const float *q = part + j * C + c;
    const int64_t n = (W + 1) * C;
    double x = 0.0;
    if (c < C)
        for (int64_t i = wave_id(); i < tiles; i += 8 * CSW) {
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = i + k * CSW < tiles ? q[(i + k * CSW) * n] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) x += f[k];
        }
    s[wave_id()][lane_id()] = x;
    __syncthreads();
    if (wave_id() == 0 && c < C) {
        double t = 0.0;
        for (int w = 0; w < CSW; ++w) t += s[w][lane_id()];
        if (j < W) dw[c * W + j] = (float)t;
        else db[c] = (float)t;
    }
}

// S new tokens of a request; its W - 1 inputs are read from its slot once and
// written once.
template <typename T, int E, int W>
__global__ void __launch_bounds__(CNT) gdp_conv_decode_k(gdp_conv_decode_args a) {
    const int per = (a.C + E - 1) / E;
    const int64_t id = (int64_t)blockIdx.x * CNT + threadIdx.x;
    const int64_t req = id / per;
    if (req >= a.n) return;
    const int col = (int)(id - req * per) * E;
    const int64_t slot = a.slots ? (int64_t)a.slots[req] : req;
    T *y = (T *)a.y + req * a.S * (int64_t)a.C + col;
    Chans<T, E> r;
    if (slot < 0 || slot >= a.pool) {
        r.zero();
        for (int64_t t = 0; t < a.S; ++t) r.store(y + t * a.C);
        return;
    }
    Taps<E, W> f;
    f.load(a.w, a.b, col);
    T *state = (T *)a.state + slot * (W - 1) * (int64_t)a.C + col;
    Window<T, E, W> win;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        r.load(state + (int64_t)k * a.C);
        r.to(win.v[k]);
    }
    const T *xp = (const T *)a.x + req * a.x_n_stride + col;
    for (int64_t t = 0; t < a.S; ++t) {
        float x[E], u[E];
        r.load(xp + t * a.x_t_stride);
        r.to(x);
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] = act_exact(a.activation, f.at(win, x, e));
        win.push(x);
        r.from(u);
        r.store(y + t * a.C);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        r.from(win.v[k]);
        r.store(state + (int64_t)k * a.C);
    }
}

namespace {

int elems_of(const ShortConv &p, gdp_dtype dtype) { return !p.vec ? 1 : dtype == GDP_BF16 ? 8 : 4; }
int lanes_log(const ShortConv &p, gdp_dtype dtype) {
    const int E = elems_of(p, dtype);
    int l = 0;
    while (l < 6 && (E << l) < p.C) ++l;
    return l;
}
int64_t tiles_of(const ShortConv &p, gdp_dtype dtype) {
    const int64_t per = (int64_t)(CNT >> lanes_log(p, dtype)) * CTT;
    return (p.m.rows + per - 1) / per;
}

template <typename T, int E, int W>
hipError_t run_conv(const ShortConv &p, bool back, hipStream_t stream) {
    const int w = E << p.lognx;
    const dim3 grid((unsigned)(p.tiles > 0 ? p.tiles : 1), (unsigned)((p.C + w - 1) / w));
    if (back) hipLaunchKernelGGL((gdp_conv_bwd_k<T, E, W>), grid, dim3(CNT), 0, stream, p);
    else hipLaunchKernelGGL((gdp_conv_k<T, E, W>), grid, dim3(CNT), 0, stream, p);
    return hipGetLastError();
}
template <typename T, int E>
hipError_t run_width(const ShortConv &p, bool back, hipStream_t stream) {
    switch (p.W) {
    case 2: return run_conv<T, E, 2>(p, back, stream);
    case 3: return run_conv<T, E, 3>(p, back, stream);
    case 4: return run_conv<T, E, 4>(p, back, stream);
    }
    return hipErrorInvalidValue;
}
hipError_t run_types(ShortConv p, gdp_dtype dtype, bool back, hipStream_t stream) {
    p.lognx = lanes_log(p, dtype);
    p.tiles = (int)tiles_of(p, dtype);
    if (dtype == GDP_BF16) return p.vec ? run_width<bf16, 8>(p, back, stream) : run_width<bf16, 1>(p, back, stream);
    return p.vec ? run_width<float, 4>(p, back, stream) : run_width<float, 1>(p, back, stream);
}

template <typename T, int E>
hipError_t run_decode(const gdp_conv_decode_args &a, hipStream_t stream) {
    const int64_t threads = a.n * ((a.C + E - 1) / E);
    const dim3 grid((unsigned)((threads + CNT - 1) / CNT));
    switch (a.W) {
    case 2: hipLaunchKernelGGL((gdp_conv_decode_k<T, E, 2>), grid, dim3(CNT), 0, stream, a); break;
    case 3: hipLaunchKernelGGL((gdp_conv_decode_k<T, E, 3>), grid, dim3(CNT), 0, stream, a); break;
    case 4: hipLaunchKernelGGL((gdp_conv_decode_k<T, E, 4>), grid, dim3(CNT), 0, stream, a); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

bool conv_fits(const ShortConv &p, gdp_dtype dtype, bool) { return tiles_of(p, dtype) * CNT <= 0xffffffffll; }
int64_t conv_space(const ShortConv &p, gdp_dtype dtype) {
    const int64_t tiles = tiles_of(p, dtype);
    return (tiles > 0 ? tiles : 1) * (p.W + 1) * p.C * (int64_t)sizeof(float);
}
hipError_t launch_conv(ShortConv p, gdp_dtype dtype, hipStream_t stream) { return run_types(p, dtype, false, stream); }
hipError_t launch_conv_bwd(ShortConv p, gdp_dtype dtype, hipStream_t stream) {
    const hipError_t e = run_types(p, dtype, true, stream);
    if (e != hipSuccess || !p.part) return e;
    const int64_t tiles = tiles_of(p, dtype);
    hipLaunchKernelGGL(gdp_conv_sum_k, dim3((unsigned)((p.C + 63) / 64), (unsigned)(p.W + 1)), dim3(64 * CSW), 0, stream,
                       p.part, tiles > 0 ? tiles : 1, (int64_t)p.C, p.W, p.dw, p.db);
    return hipGetLastError();
}
hipError_t launch_conv_decode(const gdp_conv_decode_args &a, bool vec, hipStream_t stream) {
    if (a.dtype == GDP_BF16) return vec ? run_decode<bf16, 8>(a, stream) : run_decode<bf16, 1>(a, stream);
    return vec ? run_decode<float, 4>(a, stream) : run_decode<float, 1>(a, stream);
}

}  // namespace gdp

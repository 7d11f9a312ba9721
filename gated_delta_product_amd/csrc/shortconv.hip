// shortconv.hip -- short causal convolution, channels last, W taps a channel:
//   u_t = b + sum_j w_j x_{t-W+1+j},  y_t = act(u_t)
// where the rows before a sequence come from its state, the W - 1 inputs
// before it (oldest first), and with du = dy act'(u):
//   dx_s = sum_j w_j du_{s+W-1-j},  dw_j = sum_t du_t x_{t-W+1+j},  db = sum du
//
// A thread walks a run of rows of E channels with the last W - 1 rows (and
// backwards the last W du) in registers, a few rows' loads ahead.  Every tensor
// is moved once but for the rows around a run's ends, which come from the
// caches, and that bounds the forward pass: 32768 x 10240 bfloat16, W = 4, 244 us
// (1342 MB, 5.5 TB/s; a large copy reaches 5.1).  The gradients form 36
// instructions an element, which take as long as two thirds of the time and are
// not all hidden, and before them a thread asks what its 64 rows are, one after
// the other (plain_rows): 15151 x 5632 125 us (513 MB, 4.1 TB/s), 6 of them the
// sums of the runs' partial dw and db.  256 steps of 10240 channels take 11 us (the
// floor is 8): a thread's taps come first, then its state and its rows, and five
// waves a SIMD (94 registers) hide little of the one round that they are.
// Rows that do not start on 16 bytes go by single elements (16384 x 4999
// bfloat16: 107 and 173 us, 16384 x 5000: 71 and 140).
#include "rows.h"

namespace gdp {

namespace {

constexpr int CNT = 256;
constexpr int CHUNK = 4;  // rows whose loads are under way together, the next ones' meanwhile
// Rows of a thread: forwards 16; backwards so many that with the W - 1 rows
// behind them, whose du it forms too, they are whole chunks (runs of 29 / 45 / 61
// / 125 rows: 141 / 133 / 130 / 137 us; chunks of 2 / 4 / 8: 142 / 130 / 150).
constexpr int run_of(bool back, int W) { return back ? 16 * CHUNK - (W - 1) : 4 * CHUNK; }

// 1 / (1 + e^-u).  bfloat16: to (2 + |u|) 2^-24, far within the rows' own 2^-9; the
// float32 dw and db sum such terms, and their own roundings hide it (15151 x 512:
// both 1.6e-7 off, as with an exact power, which takes 7 us more at 5632).
template <typename T> __device__ __forceinline__ float sigmoid_of(float u) {
    if constexpr (std::is_same<T, float>::value) return sigmoid_exact(u);
    else return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u * -1.44269502f));
}
template <typename T> __device__ __forceinline__ float act_of(int kind, float u) {
    if (kind == GDP_ACT_NONE) return u;
    const float s = sigmoid_of<T>(u);
    return kind == GDP_ACT_SILU ? u * s : s;
}
template <typename T> __device__ __forceinline__ float act_slope_of(int kind, float u) {
    if (kind == GDP_ACT_NONE) return 1.0f;
    const float s = sigmoid_of<T>(u), r = fmaf(-s, s, s);  // s (1 - s)
    return kind == GDP_ACT_SILU ? fmaf(u, r, s) : r;
}

// Rows of a strided tensor by their distance from a thread's first one, also
// in front of it and behind its tile; zeros past the ends of the tensor.  FLAT:
// they lie at even distances.
template <typename T, int E, bool FLAT>
struct Reader {
    TileRows<T> rows;
    const Strided &x;
    const RowMap &m;
    bool live;
    uint32_t row0;
    int col;
    template <typename P>
    __device__ __forceinline__ Reader(const Strided &x, const RowMap &m, const P &at, int run, int tile_rows, int C)
        : rows(start(x, m, at, run, tile_rows, C)), x(x), m(m), live(at.live), row0(at.row0), col(at.col) {}
    // the tile with three rows in front of it and three behind, as far as there are
    template <typename P>
    static __device__ __forceinline__ TileRows<T> start(const Strided &x, const RowMap &m, const P &at, int run, int tile_rows, int C) {
        const uint32_t front = at.tile0 < 3 ? at.tile0 : 3, first = at.tile0 - front;
        const uint32_t n = FLAT && first < m.rows ? min(m.rows - first, front + tile_rows + 3) : 0;
        return TileRows<T>((const T *)x.p + (int64_t)first * x.ts, x.ts, n, C, (int)front + at.ty * run, at.col, at.live);
    }
    __device__ __forceinline__ void load(Chans<T, E> &u, int i) const {
        if constexpr (FLAT) {
            u.load(rows.r, rows.off + (uint32_t)i * rows.step);
        } else {
            const int64_t r = (int64_t)row0 + i;
            u.zero();
            if (live && r >= 0 && r < m.rows) u.load(RowWalk<T>(x, m, (uint32_t)r, col).p);
        }
    }
};

// The W - 1 inputs before a row, oldest first.
template <typename T, int E, int W>
struct Window {
    float v[W - 1][E];
    // of a sequence's first row
    __device__ __forceinline__ void start(const ShortConv &p, int seq, int col) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            Chans<T, E> r;
            r.zero();
            if (p.h0) r.load((const T *)p.h0 + ((int64_t)seq * (W - 1) + k) * p.C + col);
            r.to(v[k]);
        }
    }
    // of a thread's first row, with this code, in sequence seq (anything where it is in none)
    template <bool FLAT>
    __device__ __forceinline__ void start(const ShortConv &p, const Reader<T, E, FLAT> &in, uint32_t code, int seq, int col) {
        const int before = (int)rows_before(code);
#pragma unroll
        for (int k = 1; k < W; ++k) {
            Chans<T, E> r;
            if (!(code & ROW_IN)) r.zero();
            else if (k <= before) in.load(r, -k);
            else {
                r.zero();
                if (p.h0) r.load((const T *)p.h0 + ((int64_t)seq * (W - 1) + (W - 1 - k + before)) * p.C + col);
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
        const float *q = pw + (int64_t)col * W;
        if (E > 1 && !((uintptr_t)pw & 15)) {  // E W of them in a row: a thread's first is on 16 bytes, as E is 4 or 8
#pragma unroll
            for (int i = 0; i < E * W / 4; ++i) {
                const f32x4 v = ((const f32x4 *)q)[i];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[(4 * i + k) / W][(4 * i + k) % W] = v[k];
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int j = 0; j < W; ++j) w[e][j] = q[e * W + j];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) b[e] = 0.f;
        if (pb) {
            if (E > 1 && !((uintptr_t)pb & 15)) {
#pragma unroll
                for (int i = 0; i < E / 4; ++i) {
                    const f32x4 v = ((const f32x4 *)(pb + col))[i];
#pragma unroll
                    for (int k = 0; k < 4; ++k) b[4 * i + k] = v[k];
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) b[e] = pb[col + e];
            }
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
__device__ __forceinline__ void empty_states(const RowMap &m, const void *from, void *to, int C, int col, int tile, int tiles) {
    for (int q = tile; q < m.nseq; q += tiles)
        if (seq_empty(m, q))
            for (int k = 0; k < W - 1; ++k) {
                Chans<T, E> r;
                r.zero();
                const int64_t at = ((int64_t)q * (W - 1) + k) * C + col;
                if (from) r.load((const T *)from + at);
                r.store((T *)to + at);
            }
}

// Whether none of the wave's rows is outside the sequences or within three of
// an end: nothing has to be asked row by row then.
__device__ __forceinline__ bool plain_rows(const uint8_t *code, int n) {
    bool odd = false;
    for (int i = 0; i < n; ++i) odd = odd || code[i] != (ROW_IN | 3 << 1 | 3 << 3);
    return !__any(odd);
}

}  // namespace

template <typename T, int E, int W, int NX, bool FLAT>
__global__ void __launch_bounds__(CNT) gdp_conv_k(ShortConv p, int strips, int tiles) {
    constexpr int NY = CNT / NX, TT = run_of(false, W);
    __shared__ uint8_t code[NY * TT];
    __shared__ int seq[NY * TT];
    const uint32_t tile = blockIdx.x / (uint32_t)strips, strip = blockIdx.x - tile * strips;
    const Place<NX, NY, E, TT> at(p.C, tile, strip);
    const Reader<T, E, FLAT> in(p.x, p.m, at, TT, NY * TT, p.C);
    Chans<T, E> next[CHUNK];
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) in.load(next[i], i);
    find_rows<CNT>(p.m, at.tile0, NY * TT, code, seq);
    __syncthreads();
    if (!at.live) return;
    const int k0 = at.ty * TT;
    Taps<E, W> f;
    f.load(p.w, p.b, at.col);
    Window<T, E, W> win;
    win.start(p, in, code[k0], seq[k0], at.col);
    const bool plain = plain_rows(code + k0, TT);
    const uint32_t n = at.tile0 < p.m.rows ? min(p.m.rows - at.tile0, (uint32_t)(NY * TT)) : 0;
    const TileRows<T> y((T *)p.y + (int64_t)at.tile0 * p.C, p.C, n, p.C, k0, at.col, true);
    const auto row = [&](auto is_plain, Chans<T, E> &raw, int i) {
        constexpr bool PLAIN = decltype(is_plain)::value;
        const int k = k0 + i;
        const uint32_t c = PLAIN ? 0u : code[k];
        if (!PLAIN && !(c & ROW_IN)) return;
        if (!PLAIN && row_first(c)) win.start(p, seq[k], at.col);
        float x[E], o[E];
        raw.to(x);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = act_of<T>(p.act, f.at(win, x, e));
        win.push(x);
        raw.from(o);
        raw.store(y.r, y.off + i * y.step);
        if (!PLAIN && row_last(c) && p.ht)
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                raw.from(win.v[j]);
                raw.store((T *)p.ht + ((int64_t)seq[k] * (W - 1) + j) * p.C + at.col);
            }
    };
#pragma unroll
    for (int i0 = 0; i0 < TT; i0 += CHUNK) {
        Chans<T, E> raw[CHUNK];
#pragma unroll
        for (int i = 0; i < CHUNK; ++i) raw[i] = next[i];
        if (i0 + CHUNK < TT)
#pragma unroll
            for (int i = 0; i < CHUNK; ++i) in.load(next[i], i0 + CHUNK + i);
        // one block of code for the chunk where nothing has to be asked
        if (plain) {
#pragma unroll
            for (int i = 0; i < CHUNK; ++i) row(std::true_type{}, raw[i], i0 + i);
        } else {
#pragma unroll
            for (int i = 0; i < CHUNK; ++i) row(std::false_type{}, raw[i], i0 + i);
        }
    }
    if (p.ht && at.ty == 0) empty_states<T, E, W>(p.m, p.h0, p.ht, p.C, at.col, tile, tiles);
}

template <typename T, int E, int W, int NX, bool FLAT>
__global__ void __launch_bounds__(CNT) gdp_conv_bwd_k(ShortConv p, int strips, int tiles) {
    constexpr int NY = CNT / NX, TT = run_of(true, W), X = W - 1, CW = NX * E;
    __shared__ uint8_t code[NY * TT + X];
    __shared__ int seq[NY * TT + X];
    __shared__ float red[CNT * E];
    const uint32_t tile = blockIdx.x / (uint32_t)strips, strip = blockIdx.x - tile * strips;
    const Place<NX, NY, E, TT> at(p.C, tile, strip);
    const Reader<T, E, FLAT> in(p.x, p.m, at, TT, NY * TT, p.C), dn(p.dy, p.m, at, TT, NY * TT, p.C);
    Chans<T, E> nx[CHUNK], nd[CHUNK];
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) {
        in.load(nx[i], i);
        dn.load(nd[i], i);
    }
    find_rows<CNT>(p.m, at.tile0, NY * TT + X, code, seq);
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
        win.start(p, in, code[k0], seq[k0], at.col);
        const bool plain = plain_rows(code + k0, TT + X);
        const uint32_t n = at.tile0 < p.m.rows ? min(p.m.rows - at.tile0, (uint32_t)(NY * TT)) : 0;
        const TileRows<T> out((T *)p.dx + (int64_t)at.tile0 * p.C, p.C, n, p.C, k0, at.col, true);
        float du[W][E];  // of the rows i - X .. i
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < E; ++e) du[j][e] = 0.f;
        // (asking row by row: code of their own for plain chunks takes 182 registers for 128, 135 us for 130)
        const auto row = [&](const Chans<T, E> &rx, const Chans<T, E> &rd, int k) {
            const uint32_t c = plain ? ROW_IN : code[k0 + k];
#pragma unroll
            for (int j = 0; j < X; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) du[j][e] = du[j + 1][e];
            if (plain || (c & ROW_IN)) {
                if (!plain && row_first(c)) win.start(p, seq[k0 + k], at.col);
                float x[E], d[E];
                rx.to(x);
                rd.to(d);
                const bool own = k < TT;  // the rows behind are another thread's for the sums
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float u = d[e] * act_slope_of<T>(p.act, f.at(win, x, e)), s = own ? u : 0.f;
                    du[X][e] = u;
                    db[e] += s;
                    if (own) {
#pragma unroll
                        for (int j = 0; j < X; ++j) dw[j][e] = fmaf(s, win.v[j][e], dw[j][e]);
                        dw[X][e] = fmaf(s, x[e], dw[X][e]);
                    }
                }
                win.push(x);
            }
            if (k < X) return;
            // row s = k - X: its du and those of the rows behind it are du[0 .. X]
            const int s = k - X;
            Chans<T, E> r;
            float dx[E];
#pragma unroll
            for (int e = 0; e < E; ++e) dx[e] = 0.f;
            if (plain) {
#pragma unroll
                for (int j = 0; j < W; ++j)
#pragma unroll
                    for (int e = 0; e < E; ++e) dx[e] = fmaf(f.w[e][X - j], du[j][e], dx[e]);
            } else if (const uint32_t cs = code[k0 + s]; cs & ROW_IN) {
                const int behind = (int)rows_behind(cs), q = seq[k0 + s];
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
                    for (int t = 0; t < X; ++t) {  // state row t: read by the taps t - d of the rows d behind the first
                        float z[E];
#pragma unroll
                        for (int e = 0; e < E; ++e) z[e] = 0.f;
                        if (p.dht && t > behind) {  // a sequence so short that its final state still holds the row
                            r.load((const T *)p.dht + ((int64_t)q * X + t - 1 - behind) * p.C + at.col);
                            r.to(z);
                        }
#pragma unroll
                        for (int d = 0; d <= t; ++d)
                            if (d <= behind)
#pragma unroll
                                for (int e = 0; e < E; ++e) z[e] = fmaf(f.w[e][t - d], du[d][e], z[e]);
                        r.from(z);
                        r.store((T *)p.dh0 + ((int64_t)q * X + t) * p.C + at.col);
                    }
            }
            r.from(dx);
            r.store(out.r, out.off + s * out.step);
        };
#pragma unroll 1
        for (int i0 = 0; i0 < TT + X; i0 += CHUNK) {
            Chans<T, E> rx[CHUNK], rd[CHUNK];
#pragma unroll
            for (int i = 0; i < CHUNK; ++i) {
                rx[i] = nx[i];
                rd[i] = nd[i];
            }
            if (i0 + CHUNK < TT + X)
#pragma unroll
                for (int i = 0; i < CHUNK; ++i) {
                    in.load(nx[i], i0 + CHUNK + i);
                    dn.load(nd[i], i0 + CHUNK + i);
                }
#pragma unroll
            for (int i = 0; i < CHUNK; ++i) row(rx[i], rd[i], i0 + i);
        }
        if (p.dh0 && at.ty == 0) empty_states<T, E, W>(p.m, p.dht, p.dh0, p.C, at.col, tile, tiles);
    }
    if (!p.part) return;
    // the block's rows: [tiles][W + 1][C]
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) red[at.ty * CW + at.tx * E + e] = j < W ? dw[j < W ? j : 0][e] : db[e];
        __syncthreads();
        for (int k = threadIdx.x; k < CW; k += CNT) {
            float t = 0.f;
#pragma unroll
            for (int y = 0; y < NY; ++y) t += red[y * CW + k];
            const int c = (int)strip * CW + k;
            if (c < p.C) p.part[((int64_t)tile * (W + 1) + j) * p.C + c] = t;
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
        for (int e = 0; e < E; ++e) u[e] = act_of<T>(a.activation, f.at(win, x, e));
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

// Channels of a thread: units of 16 bytes, backwards of 8 in bfloat16 (its
// sums take the registers).  Narrow rows are walked by fewer threads side by
// side.
int elems_of(const ShortConv &p, gdp_dtype dtype, bool back) { return !p.vec ? 1 : dtype == GDP_BF16 && !back ? 8 : 4; }
int lanes_of(const ShortConv &p, gdp_dtype dtype, bool back) { return p.C > 16 * elems_of(p, dtype, back) ? 64 : 16; }
int64_t tile_rows(const ShortConv &p, gdp_dtype dtype, bool back) {
    return (int64_t)(CNT / lanes_of(p, dtype, back)) * run_of(back, p.W);
}
int64_t tiles_of(const ShortConv &p, gdp_dtype dtype, bool back) {
    const int64_t per = tile_rows(p, dtype, back), n = (p.m.rows + per - 1) / per;
    return n > 0 ? n : 1;
}

template <typename T, int E, int W, int NX>
hipError_t run_lanes(const ShortConv &p, int64_t tiles, bool back, hipStream_t stream) {
    const int strips = (p.C + NX * E - 1) / (NX * E);
    const dim3 grid((unsigned)(tiles * strips));  // a tile's strips side by side: whole rows are under way at once
    // forwards and backwards differ in E: each is built for its own
    if constexpr (E != 8) {
        if (back && p.flat) hipLaunchKernelGGL((gdp_conv_bwd_k<T, E, W, NX, true>), grid, dim3(CNT), 0, stream, p, strips, (int)tiles);
        else if (back) hipLaunchKernelGGL((gdp_conv_bwd_k<T, E, W, NX, false>), grid, dim3(CNT), 0, stream, p, strips, (int)tiles);
    }
    if constexpr (!(E == 4 && std::is_same<T, bf16>::value)) {
        if (!back && p.flat) hipLaunchKernelGGL((gdp_conv_k<T, E, W, NX, true>), grid, dim3(CNT), 0, stream, p, strips, (int)tiles);
        else if (!back) hipLaunchKernelGGL((gdp_conv_k<T, E, W, NX, false>), grid, dim3(CNT), 0, stream, p, strips, (int)tiles);
    }
    return hipGetLastError();
}
template <typename T, int E>
hipError_t run_width(const ShortConv &p, gdp_dtype dtype, bool back, hipStream_t stream) {
    const int64_t tiles = tiles_of(p, dtype, back);
    const bool wide = lanes_of(p, dtype, back) == 64;
    switch (p.W) {
    case 2: return wide ? run_lanes<T, E, 2, 64>(p, tiles, back, stream) : run_lanes<T, E, 2, 16>(p, tiles, back, stream);
    case 3: return wide ? run_lanes<T, E, 3, 64>(p, tiles, back, stream) : run_lanes<T, E, 3, 16>(p, tiles, back, stream);
    case 4: return wide ? run_lanes<T, E, 4, 64>(p, tiles, back, stream) : run_lanes<T, E, 4, 16>(p, tiles, back, stream);
    }
    return hipErrorInvalidValue;
}
hipError_t run_types(ShortConv p, gdp_dtype dtype, bool back, hipStream_t stream) {
    const int64_t rows = tile_rows(p, dtype, back) + 6;  // and three on either side
    p.flat = even_rows(p.x, p.m, rows) && (!back || even_rows(p.dy, p.m, rows));
    switch (elems_of(p, dtype, back)) {
    case 8: return run_width<bf16, 8>(p, dtype, back, stream);
    case 4: return dtype == GDP_BF16 ? run_width<bf16, 4>(p, dtype, back, stream) : run_width<float, 4>(p, dtype, back, stream);
    default: return dtype == GDP_BF16 ? run_width<bf16, 1>(p, dtype, back, stream) : run_width<float, 1>(p, dtype, back, stream);
    }
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

bool conv_fits(const ShortConv &p, gdp_dtype dtype, bool backward) {
    const int64_t w = lanes_of(p, dtype, backward) * elems_of(p, dtype, backward);
    return tiles_of(p, dtype, backward) * ((p.C + w - 1) / w) * CNT <= 0xffffffffll;
}
int64_t conv_space(const ShortConv &p, gdp_dtype dtype) {
    return tiles_of(p, dtype, true) * (p.W + 1) * p.C * (int64_t)sizeof(float);
}
hipError_t launch_conv(const ShortConv &p, gdp_dtype dtype, hipStream_t stream) { return run_types(p, dtype, false, stream); }
hipError_t launch_conv_bwd(const ShortConv &p, gdp_dtype dtype, hipStream_t stream) {
    const hipError_t e = run_types(p, dtype, true, stream);
    if (e != hipSuccess || !p.part) return e;
    hipLaunchKernelGGL(gdp_conv_sum_k, dim3((unsigned)((p.C + 63) / 64), (unsigned)(p.W + 1)), dim3(64 * CSW), 0, stream,
                       p.part, tiles_of(p, dtype, true), (int64_t)p.C, p.W, p.dw, p.db);
    return hipGetLastError();
}
hipError_t launch_conv_decode(const gdp_conv_decode_args &a, bool vec, hipStream_t stream) {
    if (a.dtype == GDP_BF16) return vec ? run_decode<bf16, 8>(a, stream) : run_decode<bf16, 1>(a, stream);
    return vec ? run_decode<float, 4>(a, stream) : run_decode<float, 1>(a, stream);
}

}  // namespace gdp

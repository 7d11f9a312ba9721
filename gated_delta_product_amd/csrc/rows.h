// rows.h -- which sequence the rows of a tile belong to, and loads of the
// channels of a row.  Device helpers of the kernels that walk rows [B*T, C]
// in tiles of their own (linrec.hip, shortconv.hip, rotary.hip): sequences may
// begin and end anywhere inside a tile.
#pragma once
#include "gdp_common.h"
#include "mixops.h"

namespace gdp {

// A row's code: whether it is inside a sequence, and how far that one's first
// and last rows are (at most 3 counted: 3 stands for 3 or more).
constexpr uint32_t ROW_IN = 1;
__device__ __forceinline__ uint32_t row_code(uint32_t before, uint32_t behind) {
    return ROW_IN | (before < 3 ? before : 3) << 1 | (behind < 3 ? behind : 3) << 3;
}
__device__ __forceinline__ uint32_t rows_before(uint32_t code) { return code >> 1 & 3; }
__device__ __forceinline__ uint32_t rows_behind(uint32_t code) { return code >> 3 & 3; }
__device__ __forceinline__ bool row_first(uint32_t code) { return (code & 7) == ROW_IN; }
__device__ __forceinline__ bool row_last(uint32_t code) { return (code & 25) == ROW_IN; }

// The last i in [0, n) with cu[i] <= r, or -1: 64 probes at a time by the
// lanes of a wave (r uniform).  Any contents of cu end it, inside the array.
__device__ __forceinline__ int last_at_or_before(const int32_t *cu, int n, int r) {
    int lo = -1, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 62) / 64, p = lo + 1 + lane_id() * step;
        const uint64_t below = __ballot(p < hi && cu[p < hi ? p : lo + 1] <= r);
        const int k = below == ~0ull ? 64 : __builtin_ctzll(~below);
        const int next = lo + 1 + k * step;
        hi = k < 64 && next < hi ? next : hi;
        lo = k ? lo + 1 + (k - 1) * step : lo;
    }
    return lo;
}

// Codes and sequences of rows [r0, r0 + n), n <= the arrays' size; by the
// whole block (NT threads), which synchronises afterwards.
template <int NT>
__device__ __forceinline__ void find_rows(const RowMap &m, uint32_t r0, int n, uint8_t *code, int *seq) {
    for (int base = wave_id() * 64; base < n; base += NT) {
        const int i = base + lane_id();
        const uint32_t r = r0 + i;
        uint32_t c = 0;
        int s = 0;
        if (!m.cu) {
            if (r < m.rows) {
                const uint32_t q = r / m.T, d = r - q * m.T;
                s = (int)q;
                c = row_code(d, m.T - 1 - d);
            }
        } else if (r0 + base < m.rows) {
            const uint32_t last = r0 + base + 63 < m.rows ? r0 + base + 63 : m.rows - 1;
            int lo = last_at_or_before(m.cu, m.nseq, (int)(r0 + base));
            int hi = lo + 1 < m.nseq && m.cu[lo + 1] <= (int)last ? last_at_or_before(m.cu, m.nseq, (int)last) : lo;
            while (lo < hi) {  // cu[lo] <= r (or lo == -1), and the answer is at most hi
                const int mid = (lo + hi + 1) / 2;
                if (m.cu[mid] <= (int)r) lo = mid;
                else hi = mid - 1;
            }
            if (lo >= 0 && r < m.rows) {
                const int64_t b = m.cu[lo] < 0 ? 0 : m.cu[lo], e = m.cu[lo + 1] < (int)m.rows ? m.cu[lo + 1] : (int)m.rows;
                s = lo;
                if ((int64_t)r < e) c = row_code(r - (uint32_t)b, (uint32_t)e - 1 - r);
            }
        }
        if (i < n) {
            code[i] = (uint8_t)c;
            seq[i] = s;
        }
    }
}
__device__ __forceinline__ bool seq_empty(const RowMap &m, int i) {
    if (!m.cu) return m.T == 0;
    int64_t b, e;
    seq_bounds(m.cu, m.rows, i, b, e);
    return b == e;
}

// E neighbouring channels as they lie in memory (8 or 16 bytes, or one element;
// 8 float32 are two units).
template <typename T, int E>
struct Chans {
    static constexpr int N = (int)(E * sizeof(T) + 15) / 16;
    typedef typename std::conditional<E == 1, T, typename std::conditional<E * sizeof(T) == 8, uint2, uint4>::type>::type U;
    U u[N];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = U{};
    }
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = ((const U *)p)[i];
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < N; ++i) ((U *)p)[i] = u[i];
    }
    __device__ __forceinline__ void load(rsrc_t r, uint32_t off) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(U) == 16) u[i] = buf_load16(r, off + 16 * i);
            else if constexpr (sizeof(U) == 8) u[i] = buf_load8(r, off);
            else if constexpr (sizeof(U) == 4) u[i] = buf_load_f32(r, off);
            else u[i] = __builtin_bit_cast(U, (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0));
        }
    }
    __device__ __forceinline__ void store(rsrc_t r, uint32_t off) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(U) == 16) buf_store16(r, off + 16 * i, u[i]);
            else if constexpr (sizeof(U) == 8) buf_store8(r, off, u[i]);
            else if constexpr (sizeof(U) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, u[i]), r, (int)off, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, u[i]), r, (int)off, 0, 0);
        }
    }
    // Makes the compiler forget what it has formed from the contents, which it
    // would otherwise keep in registers for a second walk over them.
    __device__ __forceinline__ void forget() {
        if constexpr (E * sizeof(T) == 8) {
            asm volatile("" : "+v"(u[0].x), "+v"(u[0].y));
        } else if constexpr (E > 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) asm volatile("" : "+v"(u[i].x), "+v"(u[i].y), "+v"(u[i].z), "+v"(u[i].w));
        }
    }
    __device__ __forceinline__ void to(float *f) const {
        if constexpr (E == 1) {
            f[0] = to_f32(u[0]);
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const f32x4 v = __builtin_bit_cast(f32x4, u[i]);
#pragma unroll
                for (int k = 0; k < 4; ++k) f[4 * i + k] = v[k];
            }
        } else {
            typedef uint32_t words __attribute__((ext_vector_type(E / 2)));
            const words v = __builtin_bit_cast(words, u[0]);
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                f[2 * k] = __uint_as_float(v[k] << 16);
                f[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ void from(const float *f) {
        if constexpr (E == 1) {
            u[0] = from_f32<T>(f[0]);
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) u[i] = __builtin_bit_cast(U, f32x4{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]});
        } else {
            typedef __bf16 vec __attribute__((ext_vector_type(E)));
            vec v;
#pragma unroll
            for (int k = 0; k < E; ++k) v[k] = (bf16)f[k];
            u[0] = __builtin_bit_cast(U, v);
        }
    }
};

// A thread's place in a block of NX threads side by side and NY one behind the
// other: channels col .. col + E of the rows row0 .. row0 + TT.
template <int NX, int NY, int E, int TT>
struct Place {
    int tx, ty, col;
    uint32_t tile0, row0;
    bool live;
    __device__ __forceinline__ Place(int C, uint32_t tile, uint32_t strip)
        : tx(threadIdx.x % NX), ty(threadIdx.x / NX), col((int)(strip * NX + tx) * E), tile0(tile * (NY * TT)),
          row0(tile0 + ty * TT), live(col < C) {}
};

// Walks the rows of a strided [B, T, C] one after the other.
template <typename T>
struct RowWalk {
    const T *p;
    const Strided &x;
    uint32_t b, t, T_;
    int col;
    __device__ __forceinline__ RowWalk(const Strided &x, const RowMap &m, uint32_t row, int col) : x(x), T_(m.T), col(col) {
        b = m.T ? row / m.T : 0;
        t = row - b * m.T;
        p = (const T *)x.p + (int64_t)b * x.bs + (int64_t)t * x.ts + col;
    }
    __device__ __forceinline__ void next() {
        p += x.ts;
        if (++t == T_) {
            t = 0;
            ++b;
            p = (const T *)x.p + (int64_t)b * x.bs + col;
        }
    }
};

template <int E>
__device__ __forceinline__ void forget(float (&f)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) asm volatile("" : "+v"(f[e]));
}

// The rows of a tile, n of them, ts elements apart, as a buffer: a row past the
// last one, or a thread without channels, reads zeros and writes nothing.  The
// tile's rows lie within 2^31 bytes.
template <typename T>
struct TileRows {
    rsrc_t r;
    uint32_t off, step;  // of the thread's first row, and from row to row
    __device__ __forceinline__ TileRows(const T *tile, int64_t ts, uint32_t n, int C, int row, int col, bool live) {
        step = (uint32_t)ts * sizeof(T);
        r = make_rsrc((const void *)uniform_i64((int64_t)tile), __builtin_amdgcn_readfirstlane(n ? (n - 1) * step + C * (uint32_t)sizeof(T) : 0));
        off = live ? row * step + col * sizeof(T) : 0x80000000u;
    }
};
// TT raw rows of a thread; past the last row, or the last channel, zeros.
// flat: every row ts behind the one before, and a tile's within 2^31 bytes
template <typename T, int E, int TT, typename P>
__device__ __forceinline__ void load_rows(Chans<T, E> (&u)[TT], const Strided &x, const RowMap &m, bool flat, const P &at,
                                          uint32_t n, int C) {
    if (flat) {
        const TileRows<T> rows((const T *)x.p + (int64_t)at.tile0 * x.ts, x.ts, n, C, at.ty * TT, at.col, at.live);
#pragma unroll
        for (int i = 0; i < TT; ++i) u[i].load(rows.r, rows.off + i * rows.step);
    } else {
        RowWalk<T> row(x, m, at.row0, at.col);
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            u[i].zero();
            if (at.live && at.row0 + i < m.rows) u[i].load(row.p);
            row.next();
        }
    }
}

// E channels of a sequence's float state [nseq, C] (zeros without one).
template <int E>
__device__ __forceinline__ void load_state(float (&h)[E], const float *s, int64_t seq, int C, int col) {
    if (s) {
        const float *q = s + seq * C + col;
        if (E > 1 && !((uintptr_t)s & 15)) {  // C and col are whole units of four
#pragma unroll
            for (int i = 0; i < E / 4; ++i) {
                const f32x4 v = ((const f32x4 *)q)[i];
#pragma unroll
                for (int k = 0; k < 4; ++k) h[4 * i + k] = v[k];
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) h[e] = q[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = 0.f;
    }
}
template <int E>
__device__ __forceinline__ void store_state(float *s, int64_t seq, int C, int col, const float (&h)[E]) {
    float *q = s + seq * C + col;
    if (E > 1 && !((uintptr_t)s & 15)) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) ((f32x4 *)q)[i] = f32x4{h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]};
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] = h[e];
    }
}

// e^g to about an ulp: 2^(g log2 e) with the product's rounding put back
__device__ __forceinline__ float exp_exact(float g) {
    const float L = 1.44269502f, t = g * L, l = fmaf(g, 1.92596299e-8f, fmaf(g, L, -t)), v = __builtin_amdgcn_exp2f(t);
    return fabsf(g) < 88.0f ? fmaf(v, l * 0.693147182f, v) : v;
}
__device__ __forceinline__ float sigmoid_exact(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_exact(-x)); }

}  // namespace gdp

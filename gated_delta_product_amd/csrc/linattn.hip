// linattn.hip -- linear attention with a decay for each head, chunked.
//
//   S_t = e^{g_t} S_{t-1} + v_t k_t^T   (V x K),     o_t = scale S_t q_t
//
// Unrolled over pairs, with D(i,j) = exp(sum of g over (j, i]):
//   o_i  = scale [ D(i,start) S_0 q_i + sum_{j<=i} D(i,j) (q_i.k_j) v_j ]
// and its gradients are the same sum with the roles of the tensors changed:
//   dq_i = scale [ D(i,start) S_0^T do_i + sum_{j<=i} D(i,j) (do_i.v_j) k_j ]
//   dk_j = D(end,j) dht^T v_j + scale sum_{i>=j} D(i,j) (v_j.do_i) q_i
//   dv_j = D(end,j) dht k_j   + scale sum_{i>=j} D(i,j) (k_j.q_i) do_i
// so one kernel, the walk below, runs them all: it takes tensors a, b (DA
// columns) and c (DC columns), walks the rows forwards or backwards in time
// and gives y_i = sum_j D(i,j) (a_i.b_j) c_j, keeping the state
// S = sum D c_j b_j^T of the rows it has passed.
//
// A walk takes chunks of CT rows.  Per chunk, with G the inclusive cumulative
// log decay inside it (a prefix sum in 64 bits, kept as two floats, so that
// differences hold their bits behind a strong decay; chunks lie alike in every
// walk, counted from the segment's first row in time):
//   P[i][j] = (a_i.b_j) 2^(G_i - G_j), j <= i      the masked in-chunk scores
//   y_i     = 2^G_i S a_i + sum_j P[i][j] c_j
//   S      <- 2^G_end S + sum_j 2^(G_end - G_j) c_j b_j^T
// The waves (one to 16 columns of c) share the score tiles through LDS and
// then own their columns: S^T stays in registers as result tiles of the
// matrix core, whose lanes hold 4 consecutive rows a of a column c; the
// columns of b are taken in the order 8g + i, 8g + 4 + i for the two tiles
// of 32 columns, so those tiles are the operand of S a as they stand.
//
// What bounds it: not the bytes but the chain of a chunk (scores, barrier,
// decayed products, barrier) in 8 to 16 waves a compute unit, with matrix and
// vector instructions sharing the issue.  Kernel times in microseconds in an
// unbroken run of calls (clock 2.1 to 2.5 GHz; a call takes 3 to 16% more there
// than in a short run), bf16, K = V = 128, [what the bytes alone take] at 5.1 TB/s
// and the share of time that the matrix cores are busy:
//   32768 tokens, 16 heads, forwards: segment pass 83 [53 for k, v] 28%, scan 18,
//     rows 164 [105] 33%
//   8 requests of 821 to 3562 tokens, H 4, HV 16: 46 (18%) + 14 + 90 (24%)
//   the same backwards: segment pass 72 (20%), scan 25, 3 walks in one launch 264
//     (27%, 24-bit states), head sums 61, dg 18, zeros 5
//   8192 tokens, 32 heads, V = 256 backwards, decay per head: segment pass 127
//     (24%), scan 11, walks 477 (29%; 256 rows of S^T a wave leave two waves a
//     SIMD), dg 41 + 5
// A third of the LDS cycles of every walk are bank conflicts.
#include "gdp_common.h"
#include "gdp_internal.h"
#include "linattn.h"

namespace gdp {

// ---------------------------------------------------------------- LDS tiles
// Rows of D elements without padding; the 16-byte unit u of row r sits at
// u ^ swz(r).  16 rows at one unit (operand rows) then fall on 16 units
// (8 with 8 units a row, two rows to a span of all banks), and 4 rows at 4
// neighbouring units (the transposed reads) on all banks once.
// The low bits run 0, 2, 3, 1 over the blocks of 4 rows: a 16-byte read takes
// lanes 0-3 with 20-23, 4-7 with 16-19 and so on at once, and those then sit
// on different units too.
template <int UPR>
__device__ __forceinline__ int swz(int row) {
    const int low = (0x78 >> (2 * ((row >> 2) & 3))) & 3;
    if constexpr (UPR == 8) return (((row >> 1) & 1) << 2) | low;
    else return ((row & 3) << 2) | low;
}
template <typename T, int D>
struct Tile {
    static constexpr int E = 16 / sizeof(T);  // elements of a unit
    static constexpr int UPR = D / E;
    typedef typename Frag<T>::type frag;
    typedef typename Frag<T>::half half;
    static __device__ __forceinline__ int at(int row, int col) {
        return row * D + (((col / E) ^ swz<UPR>(row)) * E) + col % E;
    }

    // Operand rows: 8 elements [16 ib + m][32 kb + 8 g .. + 7] for lane 16 g + m.
    // swz looks at the row's low 4 bits and 32 kb at the unit's bits above
    // g's, so one offset per lane serves every ib (added) and kb (xor).
    static __device__ __forceinline__ int row_base(int lane) { return at(lane & 15, 8 * (lane >> 4)); }
    static __device__ __forceinline__ frag row8(const T *t, int base, int ib, int kb) {
        const T *p = t + ((base ^ (32 * kb)) + 16 * ib * D);
        if constexpr (sizeof(T) == 2) return *(const frag *)p;
        else return join<T>(*(const f32x4 *)p, *(const f32x4 *)(t + ((base ^ (32 * kb) ^ 4) + 16 * ib * D)));
    }

    // Operand columns: rows 32 tb + 8 g + 0 .. 7 of one column per lane, the
    // transposed read (a 16-lane group: source lane s points at row s / 4;
    // output lane 4 i + j receives slot j of the sources 4 r + i).  The column
    // of lane m is col0 + STEP * (m / 4) + m % 4: 16 neighbours (STEP 4), or
    // with STEP 8 every other four of 32.  bf16: two offsets per lane (rows
    // + 0 and + 4); 32-column groups come in by xor, rows and a step of 4
    // columns (STEP 8) by addition.
    struct Cols {
        int o[2];
    };
    template <int STEP>
    static __device__ __forceinline__ Cols col_base(int lane, int col0) {
        const int q = lane & 15, r = 8 * (lane >> 4) + (q >> 2);
        return Cols{{at(r, col0 + STEP * (q & 3)), at(r + 4, col0 + STEP * (q & 3))}};
    }
    template <int STEP>
    static __device__ __forceinline__ frag col8(const T *t, const Cols &c, int lane, int tb, int kb, int add) {
        if constexpr (sizeof(T) == 2) {
            half h[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const T *p = t + ((c.o[k] ^ (32 * kb)) + 32 * tb * D + add);
                h[k] = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                      (lds_i16x4 *)((__attribute__((address_space(3))) const char *)p)));
            }
            return join<T>(h[0], h[1]);
        } else {
            // o[0] holds the plain column
            const int m = lane & 15, col = c.o[0] + 32 * kb + add + STEP * (m >> 2) + (m & 3), r = 32 * tb + 8 * (lane >> 4);
            frag f;
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = t[at(r + i, col)];
            return f;
        }
    }
    template <int STEP>
    static __device__ __forceinline__ Cols cols(int lane, int col0) {
        if constexpr (sizeof(T) == 2) return col_base<STEP>(lane, col0);
        else return Cols{{col0, 0}};
    }
};

// The scores P of a chunk as operands: 16 x 32 tiles (rows i, 32 rows j) at
// and below the diagonal, each value in two bf16 parts (all first parts, then
// all second ones); in float32, rows as above.  The tiles (0, 0) and (2, 1)
// hold 16 columns, the lanes of the other 16 read the zeros behind them: two
// parts then take 10 KB, and two blocks of the widest walk fit a compute unit.
template <typename T, int CT>
struct Scores {
    typedef Tile<T, CT> TP;
    typedef typename Frag<T>::type frag;
    typedef typename Frag<T>::half half;
    static constexpr int PARTS = 1, SIZE = CT * CT;
    struct Lane {
        int full;
    };
    static __device__ __forceinline__ Lane lane_of(int m, int g4) { return Lane{TP::at(m, 8 * g4)}; }
    static __device__ __forceinline__ void clear(T *p, int tid, int nt) {
        for (int i = tid; i < SIZE; i += nt) p[i] = 0.f;
    }
    // columns 16 jb + 4 g4 .. + 3 of row 16 ib + m
    static __device__ __forceinline__ void put(T *p, int ib, int jb, int m, int g4, f32x4 x) {
        *(half *)(p + TP::at(16 * ib + m, 16 * jb + 4 * g4)) = x;
    }
    static __device__ __forceinline__ frag get(const T *p, Lane l, int ib, int tb, int) { return TP::row8(p, l.full, ib, tb); }
};
template <>
struct Scores<bf16, 64> {
    static constexpr int PARTS = 2, HALF = 16 * 16 + 8, FULL = 16 * 32, PART = 2 * HALF + 4 * FULL, SIZE = PARTS * PART;
    struct Lane {
        int full, half;
    };
    // (0, 0), (2, 1); (1, 0), (2, 0), (3, 0), (3, 1)
    static constexpr __device__ __forceinline__ bool is_half(int ib, int tb) { return ib == 2 * tb; }
    static constexpr __device__ __forceinline__ int at(int ib, int tb) {
        return is_half(ib, tb) ? HALF * tb : 2 * HALF + FULL * (ib - 1 + tb);
    }
    static __device__ __forceinline__ Lane lane_of(int m, int g4) {
        return Lane{32 * m + 8 * g4, g4 < 2 ? 16 * m + 8 * g4 : 16 * 16};
    }
    static __device__ __forceinline__ void clear(bf16 *p, int tid, int) {
        if (tid < 4 * 8) p[(tid >> 4) * PART + (tid >> 3 & 1) * HALF + 16 * 16 + (tid & 7)] = (bf16)0.f;
    }
    static __device__ __forceinline__ void put(bf16 *p, int ib, int jb, int m, int g4, f32x4 x) {
        const int tb = jb >> 1, at0 = at(ib, tb) + (is_half(ib, tb) ? 16 * m : 32 * m + 16 * (jb & 1)) + 4 * g4;
        bf16x4 hi, lo;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            hi[r] = (bf16)x[r];
            lo[r] = (bf16)(x[r] - (float)hi[r]);
        }
        *(bf16x4 *)(p + at0) = hi;
        *(bf16x4 *)(p + at0 + PART) = lo;
    }
    static __device__ __forceinline__ bf16x8 get(const bf16 *p, Lane l, int ib, int tb, int part) {
        return *(const bf16x8 *)(p + part * PART + at(ib, tb) + (is_half(ib, tb) ? l.half : l.full));
    }
};

// Values x[0..7] as NS parts of the storage type whose sum carries 8 NS
// bits (bf16); for float storage one part is the value.
template <typename T, int NS>
__device__ __forceinline__ void split8(const float *x, typename Frag<T>::type *part) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int p = 0; p < NS; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const T h = from_f32<T>(r[i]);
            part[p][i] = h;
            if (p + 1 < NS) r[i] -= to_f32(h);
        }
}

// Inclusive prefix sum of a double over the 64 lanes of a wave, on DPP moves.
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ double dpp_or_zero_f64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROW_MASK, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROW_MASK, 0xF, false);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_inclusive_sum_f64(double x) {
    x += dpp_or_zero_f64<0x111>(x);
    x += dpp_or_zero_f64<0x112>(x);
    x += dpp_or_zero_f64<0x114>(x);
    x += dpp_or_zero_f64<0x118>(x);
    x += dpp_or_zero_f64<0x142, 0xA>(x);
    x += dpp_or_zero_f64<0x143, 0xC>(x);
    return x;
}

__device__ __forceinline__ double lane63_f64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// A log decay in log2 units.  Anything below -160 empties the state as far
// as a float can tell (2^-160 is zero), and is held there so that the
// cumulative sums stay finite (g = -inf is a reset).
__device__ __forceinline__ double decay_log2(float g) {
    const double x = (double)g * 1.4426950408889634;
    return x < -160.0 ? -160.0 : x;
}

// ---------------------------------------------------------------- items
// Sequence i owns max(1, ceil(len / seg_tok)) items (segments); an empty one
// owns an item with no rows, which hands its state through.  Every thread of
// the block calls it (barriers inside).
struct LinItem {
    int64_t seq, seg, slot0, bos, eos;  // slot0: the sequence's first item
};
__device__ __forceinline__ int64_t lin_segs(int64_t len, int64_t seg_tok) {
    return len <= seg_tok ? 1 : ceil_div64(len, seg_tok);
}
__device__ __forceinline__ LinItem lin_item(const int32_t *cu, int64_t nseq, int64_t T, int64_t seg_tok, int64_t id) {
    LinItem r;
    if (cu == nullptr) {
        const uint32_t per = (uint32_t)lin_segs(T, seg_tok);
        const uint32_t q = (uint32_t)id / per;
        r.seq = q;
        r.seg = (uint32_t)id - q * per;
        r.slot0 = (int64_t)q * per;
        seq_bounds(nullptr, T, r.seq, r.bos, r.eos);
        return r;
    }
    __shared__ int64_t s_item[3];
    if (wave_id() == 0) {
        const int lane = lane_id();
        if (lane == 0) s_item[0] = -1;
        int64_t carry = 0;
        for (int64_t i0 = 0; i0 < nseq && carry <= id; i0 += 64) {
            const int64_t i = i0 + lane;
            int64_t n = 0;
            if (i < nseq) {
                int64_t b, e;
                seq_bounds(cu, T, i, b, e);
                n = lin_segs(e - b, seg_tok);
            }
            const int64_t incl = carry + wave_inclusive_sum_i64(n);
            const int64_t excl = incl - n;
            if (i < nseq && id >= excl && id < incl) {  // at most one lane
                s_item[0] = i;
                s_item[1] = id - excl;
                s_item[2] = excl;
            }
            carry = __shfl(incl, 63, 64);
        }
    }
    __syncthreads();
    r.seq = uniform_i64(s_item[0]);
    r.seg = uniform_i64(s_item[1]);
    r.slot0 = uniform_i64(s_item[2]);
    r.bos = r.eos = 0;
    if (r.seq >= 0) seq_bounds(cu, T, r.seq, r.bos, r.eos);
    __syncthreads();
    return r;
}

// ---------------------------------------------------------------- the walk
// OUT: rows y are computed (else only the state: the segment pass).
// DOT: also rho_i = x_i . (y_i without its own row's term), from unrounded
//      values: the part of the row that the decays scale.
// NS:  bf16 parts of the decayed c in the state update (16 or 24 bits).
// NQ:  parts of the state in S a (1 in float32, 2 for bf16 rows, 3 for dg).
//      The segment pass has no such product; with 3, states that dg is formed
//      from, it rounds a chunk's parts into its state together (that state is
//      never scaled, and each part by itself rounds relative to all of it:
//      5.5e-7 -> 2.1e-7 off after 2048 rows, for 10% of the pass).
template <typename T> constexpr bool F32_Y = sizeof(T) == 4;
template <typename T> constexpr int ROW_PARTS = sizeof(T) == 4 ? 1 : 2;

template <typename T, int DA, int DC, int NS, int NQ, bool OUT, bool DOT>
struct Walk {
    static constexpr bool F32 = sizeof(T) == 4;
    static constexpr int CT = F32 ? 32 : 64;     // rows of a chunk
    static constexpr int NB = CT / 16;           // 16-row blocks
    static constexpr int NP = NB * (NB + 1) / 2;  // score tiles at and below the diagonal
    static constexpr int TB = CT / 32;           // 32-row blocks
    static constexpr int KT = DA / 16;           // 16-row tiles of S^T
    static constexpr int WV = DC / 16;           // waves
    // chunks whose decays are formed together, by a wave each (fewer where
    // their tables would cost a compute unit a block)
    static constexpr int GD = F32 ? 4 : DOT ? 3 : DA == 128 && WV == 4 ? 2 : 4;
    static constexpr int NT = 64 * WV;
    // waves a SIMD: two blocks to a compute unit where their LDS fits (and
    // with 256 rows of S^T a wave needs the registers of two)
    static constexpr int OCC = DA == 256 ? (WV == 8 ? 2 : 1) : WV / 2;
    // tiles whose operands are loaded together: fewer where registers are
    // short (a spill's reload would wait for every row in flight)
    static constexpr bool TOGETHER = !OUT && NQ == 3;
    static constexpr int KG = TOGETHER || (DOT && OCC >= 4) ? 2 : 4, IG = DOT && OCC >= 4 ? 2 : NB;
    static constexpr int UA = CT * DA * (int)sizeof(T) / 16 / NT, UC = CT * DC * (int)sizeof(T) / 16 / NT;
    typedef Tile<T, DA> TA;
    typedef Tile<T, DC> TC;
    typedef Scores<T, CT> TP;
    typedef typename Frag<T>::type frag;

    struct Lds {
        T b[CT * DA];
        T c[CT * DC];
        T a[OUT ? CT * DA : 8];
        T x[DOT ? CT * DC : 8];
        T p[OUT ? TP::SIZE : 8];
        // decays of GD chunks: G as two floats, 2^G_i, sb 2^(G_end - G_i), G_end
        float gh[OUT ? GD : 1][CT], gl[OUT ? GD : 1][CT], eg[OUT ? GD : 1][CT], wg[GD][CT];
        double gend[GD];
        float rho[DOT ? WV * CT : 4];  // rows' shares: of the columns of a wave,
        float rho_p[DOT ? 16 * NP : 4];  // and of a score tile
    };
};

// A chunk's rows of one tensor into registers, 16 bytes a thread and step, and
// from there into a tile.  Row r of the walk is row r of the buffer, or going
// backwards row n - 1 - r; rows past n lie outside the buffer's range (there
// below its start, as a large unsigned offset) and come as zeros.
template <typename T, int D, int NT, int UNITS>
struct Rows {
    static constexpr int E = 16 / sizeof(T), UPR = D / E, STEP = NT / UPR;
    uint4 r[UNITS];
    template <bool REV>
    __device__ __forceinline__ void fetch(const T *base, uint32_t ts_elems, int n, int tid) {
        const uint32_t ts = ts_elems * sizeof(T);  // bytes of a row
        const rsrc_t rs = make_rsrc(base, (uint32_t)(n - 1) * ts + D * sizeof(T));
        const int row = tid / UPR;
        const uint32_t off = (uint32_t)(REV ? n - 1 - row : row) * ts + tid % UPR * 16;
        const uint32_t step = REV ? 0u - STEP * ts : STEP * ts;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) r[i] = buf_load16(rs, off + i * step);
    }
    // The same rows straight into a tile (no registers): lane 16-byte slots of
    // LDS lie in a row, so each lane asks for the unit that belongs in its slot.
    template <bool REV>
    static __device__ __forceinline__ void dma(T *t, const T *base, uint32_t ts_elems, int n, int wave, int lane) {
        const uint32_t ts = ts_elems * sizeof(T);
        const rsrc_t rs = make_rsrc(base, (uint32_t)(n - 1) * ts + D * sizeof(T));
        const uint32_t lds = lds_addr(t) + wave * 1024;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            const int slot = NT * i + wave * 64 + lane, row = slot / UPR;
            const uint32_t unit = (uint32_t)(slot % UPR) ^ swz<UPR>(row);
            dma16(rs, (uint32_t)(REV ? n - 1 - row : row) * ts + unit * 16, lds + NT * 16 * i);
        }
    }
    __device__ __forceinline__ void stage(T *t, int tid) const {
        if constexpr (STEP % 16 == 0) {  // whole periods of the swizzle
            T *p = t + Tile<T, D>::at(tid / UPR, tid % UPR * E);
#pragma unroll
            for (int i = 0; i < UNITS; ++i) *(uint4 *)(p + i * STEP * D) = r[i];
        } else {
#pragma unroll
            for (int i = 0; i < UNITS; ++i) *(uint4 *)(t + Tile<T, D>::at(tid / UPR + i * STEP, tid % UPR * E)) = r[i];
        }
    }
};

template <typename T, int DA, int DC, int NS, int NQ, bool OUT, bool DOT, bool REV>
__device__ __forceinline__ void lin_walk(const LinWalk &w, int64_t id, int hv, int slice,
                                         typename Walk<T, DA, DC, NS, NQ, OUT, DOT>::Lds &sm) {
    typedef Walk<T, DA, DC, NS, NQ, OUT, DOT> W;
    typedef typename W::frag frag;
    typedef typename W::TA TA;
    typedef typename W::TC TC;
    typedef typename W::TP TP;
    constexpr int CT = W::CT, NT = W::NT;
    int lane = lane_id();
    const int wave = wave_id();

    const LinItem it = lin_item(w.cu, w.nseq, w.T, w.seg_tok, id);
    if (it.seq < 0) return;
    const int64_t t0 = it.bos + it.seg * w.seg_tok;
    const int64_t t1 = t0 + w.seg_tok < it.eos ? t0 + w.seg_tok : it.eos;
    const bool at_end = REV ? it.seg == 0 : t1 == it.eos;  // the walk's last segment of the sequence
    if (!OUT && at_end) return;  // no segment is entered from it
    const int len = (int)(t1 - t0);
    // batch row and the token offset inside it (packed rows are one batch row)
    const int64_t bi = w.cu ? 0 : it.seq, tb0 = w.cu ? t0 : t0 - it.bos;
    const int64_t eos_in = w.cu ? it.eos : w.T;

    // the segment's lowest row of each tensor, and row r from there
    auto base_of = [&](const LinRows &r, int d, int first) {
        return (const T *)r.p + bi * r.bs + tb0 * r.ts + (int64_t)(hv / r.div) * d + first;
    };
    const T *pa = OUT ? base_of(w.a, DA, 0) : nullptr, *pb = base_of(w.b, DA, 0), *pc = base_of(w.c, w.dc, slice * DC);
    const T *px = DOT ? base_of(w.x, w.dc, slice * DC) : nullptr;
    const uint32_t sa = (uint32_t)w.a.ts, sb = (uint32_t)w.b.ts, sc = (uint32_t)w.c.ts, sx = (uint32_t)w.x.ts;
    auto row = [](const T *p, uint32_t ts, int r) { return p + (uint64_t)(uint32_t)r * ts; };
    const float *pg = w.g ? w.g + bi * w.g_bs + hv : nullptr;

    // The segment pass takes its chunks from the last to the first (each row's
    // weight then reaches to the segment's end and the sum is never scaled):
    // the rows walk that follows starts on the rows that were read last, which
    // the last level of cache still holds.
    const int nch = (int)(((uint32_t)len + (CT - 1)) / CT);
    // Chunks lie on multiples of CT from the segment's first row in time, in
    // every walk: low(ch) is the lowest row of the ch-th that is taken.
    auto low = [&](int ch) { return (REV == OUT ? nch - 1 - ch : ch) * CT; };
    auto count = [&](int lo) { return len - lo < CT ? len - lo : CT; };

    typedef Rows<T, DA, NT, W::UA> RA;
    typedef Rows<T, DC, NT, W::UC> RC;
    // a chunk's rows of b and c on their way; the segment pass, which has the registers, keeps two chunks' under way
    struct Set {
        RA b;
        RC c;
    };
    constexpr int AHEAD = OUT ? 1 : 2;
    Set set[AHEAD];
    // the chunk at row lo into registers
    auto fetch = [&](int lo, Set &r) {
        const int n = count(lo), tid = wave * 64 + lane;
        r.b.template fetch<REV>(row(pb, sb, lo), sb, n, tid);
        r.c.template fetch<REV>(row(pc, sc, lo), sc, n, tid);
    };
    // a and x are done with halfway through a chunk: the next rows then go into
    // their tiles directly (b and c, needed to its end, wait in registers)
    auto fetch_ax = [&](int lo) {
        const int n = count(lo);
        RA::template dma<REV>(sm.a, row(pa, sa, lo), sa, n, wave, lane);
        if constexpr (DOT) RC::template dma<REV>(sm.x, row(px, sx, lo), sx, n, wave, lane);
    };
    // The decays of GD chunks at once, one chunk to each of the last GD waves;
    // their log decays (one row a lane) are asked for a group ahead.
    float rg = 0.f;
    auto fetch_g = [&](int group) {
        const int k = group * W::GD + wave - (W::WV - W::GD);
        rg = 0.f;
        if (!pg || wave < W::WV - W::GD || k >= nch) return;
        const int lo = low(k), n = count(lo);
        // backwards, a row is entered through the decay of the row after it
        const int64_t t = tb0 + lo + (REV ? n - lane : lane);
        if (lane < n && t < eos_in) rg = pg[t * w.g_ts];
    };
    auto decays = [&]() {  // rows past the chunk's end have none, nor have chunks past the walk's
        const int k = wave - (W::WV - W::GD);
        if (k < 0) return;
        const double G = wave_inclusive_sum_f64(decay_log2(rg)), Gend = lane63_f64(G);
        if (lane < CT) {
            if constexpr (OUT) {
                const float hi = (float)G;
                sm.gh[k][lane] = hi;
                sm.gl[k][lane] = (float)(G - (double)hi);
                sm.eg[k][lane] = __builtin_amdgcn_exp2f((float)G);
            }
            sm.wg[k][lane] = w.sb * __builtin_amdgcn_exp2f((float)(Gend - G));
        }
        if (lane == 0) sm.gend[k] = Gend;
    };
    double tot = 0.0;  // segment pass: log2 decay of the chunks taken
    fetch_g(0);
    if (nch > 0) {
        fetch(low(0), set[0]);
        if (AHEAD == 2 && nch > 1) fetch(low(1), set[AHEAD - 1]);
        if constexpr (OUT) fetch_ax(low(0));
    }

    // entering state: S^T tiles [kt], rows a = 32 (kt/2) + 8 g4 + 4 (kt%2) + i, column c
    f32x4 s[W::KT];
    const int cw = wave * 16;  // first column of this wave in the slice
    const uint32_t yrow = (uint32_t)w.HV * w.dc;  // elements of a row of y, and its first one of this wave
    const int64_t y0 = ((bi * w.T + tb0) * w.HV + hv) * (int64_t)w.dc + slice * DC + cw;
    {
        const int m = lane & 15, g4 = lane >> 4, col = slice * DC + cw + m;
        const float *s0 = nullptr;
        if (w.seg_in) s0 = w.seg_in + ((it.slot0 + it.seg) * w.HV + hv) * (int64_t)w.dc * DA;
        else if (OUT && w.s0) s0 = w.s0 + (it.seq * w.HV + hv) * (int64_t)w.dc * DA;
        if (!s0) {
#pragma unroll
            for (int kt = 0; kt < W::KT; ++kt) s[kt] = zero4();
        } else if (w.trans) {
            const float *q = s0 + 8 * g4 * w.dc + col;
#pragma unroll
            for (int kt = 0; kt < W::KT; ++kt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[kt][i] = q[(32 * (kt / 2) + 4 * (kt % 2) + i) * w.dc];
        } else {
            const float *q = s0 + col * DA + 8 * g4;
#pragma unroll
            for (int kt = 0; kt < W::KT; ++kt) s[kt] = *(const f32x4 *)(q + 32 * (kt / 2) + 4 * (kt % 2));
        }
    }
    // what is read of P above the diagonal stays zero (a 32-row contraction of an even block reads 16 rows)
    if constexpr (OUT) TP::clear(sm.p, threadIdx.x, NT);

    // The barriers order LDS only: the next chunk's rows stay in flight over
    // them, and so do the stores of y.
    auto chunk = [&](int ch, Set &cur) __attribute__((always_inline)) {
        const int lo = low(ch), n = count(lo), buf = ch % W::GD;
        // rho of a decay per head: pairs inside a chunk weighed by their distance, see gdp_lin_dg_spans_k
        const bool apart = DOT && w.rho_in_chunk;
        // LDS addresses are formed anew in each chunk: held over it they would
        // not fit the registers
        asm volatile("" : "+v"(lane));
        const int m = lane & 15, g4 = lane >> 4, tid = wave * 64 + lane;
        cur.b.stage(sm.b, tid);
        cur.c.stage(sm.c, tid);
        if (buf == 0) decays();
        if constexpr (OUT) wait_vmcnt<0>();  // a and x
        lds_barrier();
        if (buf == 0) fetch_g(ch / W::GD + 1);
        if (ch + AHEAD < nch) fetch(low(ch + AHEAD), cur);
        const int arow = TA::row_base(lane);

        f32x4 y[W::NB];
        if constexpr (OUT) {
            // score tiles at and below the diagonal: P^T (rows j, columns i)
#pragma unroll
            for (int k = 0; k < (W::NP + W::WV - 1) / W::WV; ++k) {
                const int t = W::WV * k + wave;
                if (t >= W::NP) break;
                const int ib = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3, jb = t - ib * (ib + 1) / 2;
                f32x4 acc[2] = {zero4(), zero4()}, e = zero4();
#pragma unroll
                for (int kb = 0; kb < DA / 32; ++kb)
                    acc[kb & 1] = mma(TA::row8(sm.b, arow, jb, kb), TA::row8(sm.a, arow, ib, kb), acc[kb & 1]);
                if constexpr (DOT) {
                    const int crow = TC::row_base(lane);
#pragma unroll
                    for (int kb = 0; kb < DC / 32; ++kb)
                        e = mma(TC::row8(sm.c, crow, jb, kb), TC::row8(sm.x, crow, ib, kb), e);
                }
                const int i = 16 * ib + m, j0 = 16 * jb + 4 * g4;
                const float sbsy = w.sb * w.sy;
                const float ghi = sm.gh[buf][i], gli = sm.gl[buf][i];
                const f32x4 ghj = *(const f32x4 *)&sm.gh[buf][j0], glj = *(const f32x4 *)&sm.gl[buf][j0];
                f32x4 pv;
                float q = 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float d = __builtin_amdgcn_exp2f((ghi - ghj[r]) + (gli - glj[r])) * sbsy;
                    const float sc = j0 + r <= i ? (acc[0][r] + acc[1][r]) * d : 0.f;
                    pv[r] = sc;
                    if constexpr (DOT) q += j0 + r < i ? sc * e[r] * (apart ? (float)(i - j0 - r) : 1.f) : 0.f;
                }
                TP::put(sm.p, ib, jb, m, g4, pv);
                if constexpr (DOT) {
                    q = xor32_sum(xor16_sum(q));
                    if (g4 == 0) sm.rho_p[16 * t + m] = q;
                }
            }
            // S a: S^T tiles as the operand, rounded to NQ parts.  For dg the
            // smaller parts have a sum of their own: a row of rho is then off by
            // the roundings of the first parts only (2.0e-7 -> 1.4e-7).
            f32x4 yl[W::NB];
#pragma unroll
            for (int ib = 0; ib < W::NB; ++ib) y[ib] = yl[ib] = zero4();
#pragma unroll
            for (int kb = 0; kb < DA / 32; ++kb) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = s[2 * kb + i / 4][i % 4];
                frag sp[NQ];
                split8<T, NQ>(v, sp);
#pragma unroll
                for (int i0 = 0; i0 < W::NB; i0 += W::IG) {
                    frag fa[W::IG];
#pragma unroll
                    for (int i = 0; i < W::IG; ++i) fa[i] = TA::row8(sm.a, arow, i0 + i, kb);
#pragma unroll
                    for (int p = NQ - 1; p >= 0; --p)
#pragma unroll
                        for (int i = 0; i < W::IG; ++i)
                            if (DOT && p) yl[i0 + i] = mma(sp[p], fa[i], yl[i0 + i]);
                            else y[i0 + i] = mma(sp[p], fa[i], y[i0 + i]);
                }
            }
#pragma unroll
            for (int ib = 0; ib < W::NB; ++ib) {
                if constexpr (DOT) y[ib] += yl[ib];
                y[ib] *= sm.eg[buf][16 * ib + m] * w.sy;
                if constexpr (DOT) {
                    const auto xv = *(const typename Frag<T>::half *)(sm.x + TC::at(16 * ib + m, cw + 4 * g4));
                    float q = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) q += to_f32(xv[i]) * y[ib][i];
                    q = xor32_sum(xor16_sum(q));
                    if (g4 == 0) sm.rho[wave * CT + 16 * ib + m] = q;
                }
            }
            lds_barrier();
            if (ch + 1 < nch) fetch_ax(low(ch + 1));
        }

        // the rows c as operands, once for P c and (decayed) for the state
        const auto ccol = TC::template cols<4>(lane, cw);
        const auto bcol = TA::template cols<8>(lane, 0);
        const auto prow = TP::lane_of(m, g4);
        if constexpr (OUT) {
            const float dec = sm.eg[buf][CT - 1];
#pragma unroll
            for (int kt = 0; kt < W::KT; ++kt) s[kt] *= dec;
        }
        const float later = OUT ? 1.f : __builtin_amdgcn_exp2f((float)tot);  // the chunks taken before come after it
        if constexpr (!OUT) tot += sm.gend[buf];
#pragma unroll
        for (int tb = 0; tb < W::TB; ++tb) {
            const frag fc = TC::template col8<4>(sm.c, ccol, lane, tb, 0, 0);
            frag fw[NS];
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = to_f32(fc[i]) * (sm.wg[buf][32 * tb + 8 * g4 + i] * later);
            split8<T, NS>(v, fw);
            if constexpr (OUT) {
#pragma unroll
                for (int part = TP::PARTS - 1; part >= 0; --part)
#pragma unroll
                    for (int ib = 2 * tb; ib < W::NB; ++ib) y[ib] = mma(fc, TP::get(sm.p, prow, ib, tb, part), y[ib]);
            }
            // KG tiles at a time, so that a tile's parts are not back to back
#pragma unroll
            for (int k0 = 0; k0 < W::KT; k0 += W::KG) {
                frag fb[W::KG];
#pragma unroll
                for (int k = 0; k < W::KG; ++k)
                    fb[k] = TA::template col8<8>(sm.b, bcol, lane, tb, (k0 + k) / 2, 4 * (k % 2));
                if constexpr (!W::TOGETHER) {
#pragma unroll
                    for (int p = NS - 1; p >= 0; --p)
#pragma unroll
                        for (int k = 0; k < W::KG; ++k) s[k0 + k] = mma(fb[k], fw[p], s[k0 + k]);
                } else {
                    f32x4 e[W::KG];
#pragma unroll
                    for (int k = 0; k < W::KG; ++k) e[k] = zero4();
#pragma unroll
                    for (int p = NS - 1; p >= 0; --p)
#pragma unroll
                        for (int k = 0; k < W::KG; ++k) e[k] = mma(fb[k], fw[p], e[k]);
#pragma unroll
                    for (int k = 0; k < W::KG; ++k) s[k0 + k] += e[k];
                }
            }
        }
        if constexpr (OUT) {
            // rows of y as a buffer that ends with the chunk, like the inputs' (stores past it are dropped)
            const uint32_t es = w.y32 ? 4 : sizeof(T), ys = yrow * es;
            const char *yp = (const char *)w.y + (y0 + (uint64_t)(uint32_t)lo * yrow) * es;
            const rsrc_t rs = make_rsrc(yp, (uint32_t)(n - 1) * ys + 16 * es);
            const uint32_t off = (uint32_t)(REV ? n - 1 - m : m) * ys + 4 * g4 * es, step = REV ? 0u - 16 * ys : 16 * ys;
            if (F32_Y<T> || w.y32) {
#pragma unroll
                for (int ib = 0; ib < W::NB; ++ib) {
                    const f32x4 v = y[ib];
                    buf_store16(rs, off + ib * step, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                                __float_as_uint(v[2]), __float_as_uint(v[3])));
                }
            } else {
#pragma unroll
                for (int ib = 0; ib < W::NB; ++ib) {
                    const f32x4 v = y[ib];
                    const bf16x4 o = {(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
                    buf_store8(rs, off + ib * step, __builtin_bit_cast(uint2, o));
                }
            }
        }
        if constexpr (DOT) {
            // the state that crosses a span's border
            const int at = REV ? lo : lo + CT;
            if (w.mid && at % LIN_SPAN == 0 && at > 0 && at < len) {
                float *so = w.mid + ((uint64_t)(bi * w.T + tb0 + at) / LIN_SPAN * w.HV + hv) * ((uint64_t)w.dc * DA) +
                            (slice * DC + cw + m) * DA + 8 * g4;
#pragma unroll
                for (int kt = 0; kt < W::KT; ++kt) *(f32x4 *)(so + 32 * (kt / 2) + 4 * (kt % 2)) = s[kt];
            }
        }
        lds_barrier();
        if constexpr (DOT) {
            if (wave == 0 && lane < n) {
                float q = 0.f, qp = 0.f;
#pragma unroll
                for (int i = 0; i < W::WV; ++i) q += sm.rho[i * CT + lane];
                const int ib = lane / 16;
                for (int jb = 0; jb <= ib; ++jb) qp += sm.rho_p[16 * (ib * (ib + 1) / 2 + jb) + lane % 16];
                const int64_t r0 = ((int64_t)slice * w.HV + hv) * (w.B * w.T) + bi * w.T + tb0;
                const int64_t at = r0 + lo + (REV ? n - 1 - lane : lane);
                w.rho[at] = apart ? q : q + qp;
                if (!REV && apart) w.rho_in_chunk[at] = qp;
            }
        }
    };
    for (int ch = 0; ch < nch; ch += AHEAD) {
        chunk(ch, set[0]);
        if (AHEAD == 2 && ch + 1 < nch) chunk(ch + 1, set[AHEAD - 1]);
    }

    // the state after the walk: the segment's own (segment pass), or the sequence's
    float *so = nullptr;
    float f = 1.f;
    if constexpr (!OUT) {
        so = w.seg_out + ((it.slot0 + it.seg) * w.HV + hv) * (int64_t)w.dc * DA;
        if (threadIdx.x == 0 && slice == 0) w.seg_tot[(it.slot0 + it.seg) * w.HV + hv] = (float)tot;
    } else if (at_end && w.s_out) {
        so = w.s_out + (it.seq * w.HV + hv) * (int64_t)w.dc * DA;
        if (REV && pg && it.eos > it.bos)  // through the first row's decay too
            f = __builtin_amdgcn_exp2f((float)decay_log2(pg[(w.cu ? it.bos : 0) * w.g_ts]));
    }
    if (!so) return;
    const int col = slice * DC + cw + (lane & 15), g4 = lane >> 4;
#pragma unroll
    for (int kt = 0; kt < W::KT; ++kt)
        *(f32x4 *)(so + col * DA + 32 * (kt / 2) + 8 * g4 + 4 * (kt % 2)) = s[kt] * f;
}

// The block's item, value head and column slice.
template <typename T, int DA, int DC, int NS, int NQ, bool OUT, bool DOT, bool REV>
__device__ __forceinline__ void lin_block(const LinWalk &w, void *lds) {
    const uint32_t b = blockIdx.x, slices = w.dc / DC, per = (uint32_t)w.HV * slices;
    const uint32_t id = b / per, r = b - id * per;
    if (id >= w.items) return;
    lin_walk<T, DA, DC, NS, NQ, OUT, DOT, REV>(w, id, (int)(r / slices), (int)(r % slices),
                                               *(typename Walk<T, DA, DC, NS, NQ, OUT, DOT>::Lds *)lds);
}

template <typename T, int DA, int DC, int NS, int NQ, bool OUT>
__global__ void __launch_bounds__((Walk<T, DA, DC, NS, NQ, OUT, false>::NT), (Walk<T, DA, DC, NS, NQ, OUT, false>::OCC))
gdp_lin_walk_k(LinWalks p) {
    __shared__ __align__(16) char lds[sizeof(typename Walk<T, DA, DC, NS, NQ, OUT, false>::Lds)];
    if (blockIdx.y == 0) lin_block<T, DA, DC, NS, NQ, OUT, false, false>(p.w[0], lds);
    else if constexpr (!OUT) lin_block<T, DA, DC, NS, NQ, OUT, false, true>(p.w[1], lds);
}

// The three walks of the gradients in one launch: dq and dk (DA = V, slices of
// K columns) and dv (DA = K, slices of V columns), all in slices of SL.
// ND: parts of dv's state, which also leaves as dh0.
template <typename T, int K, int V, int SL, int NS, int NQ, int ND, bool DOT>
struct Grads {
    typedef Walk<T, V, SL, NS, NQ, true, DOT> QK;
    typedef Walk<T, K, SL, ND, ROW_PARTS<T>, true, false> D;
    static constexpr int OCC = QK::OCC < D::OCC ? QK::OCC : D::OCC;
    static constexpr int BYTES = sizeof(typename QK::Lds) > sizeof(typename D::Lds) ? sizeof(typename QK::Lds)
                                                                                   : sizeof(typename D::Lds);
};
template <typename T, int K, int V, int SL, int NS, int NQ, int ND, bool DOT>
__global__ void __launch_bounds__(SL * 4, (Grads<T, K, V, SL, NS, NQ, ND, DOT>::OCC)) gdp_lin_grads_k(LinWalks p) {
    __shared__ __align__(16) char lds[Grads<T, K, V, SL, NS, NQ, ND, DOT>::BYTES];
    if (blockIdx.y == 0) lin_block<T, V, SL, NS, NQ, true, DOT, false>(p.w[0], lds);
    else if (blockIdx.y == 1) lin_block<T, V, SL, NS, NQ, true, DOT, true>(p.w[1], lds);
    else lin_block<T, K, SL, ND, ROW_PARTS<T>, true, false, true>(p.w[2], lds);
}

// ---------------------------------------------------------------- the scan over segments
// Each sequence's segments in walk order: entering state of the first is h0
// (or zero), then S <- 2^tot S + E.  The E of a segment is replaced by the
// state entering it.  One thread per 4 state elements: the states go in and
// out once.  With 16 heads and more the chain over the segments is short (16 to
// 32) and the bytes bound it: 18 us for 32 segments of 16 heads (34 MB, 3.8 TB/s
// both ways).  With one or two heads a row has up to 256 segments and more, and
// the chain, 8 loads at a time, bounds it: 79 us at 32768 tokens of one head,
// beside 11 and 18 us of walks.
__global__ void __launch_bounds__(256) gdp_lin_scan_k(LinScan p) {
    const int64_t seq = blockIdx.x / p.HV;
    const int hv = (int)(blockIdx.x % p.HV);
    int64_t bos, eos, slot0;
    seq_bounds(p.cu, p.T, seq, bos, eos);
    if (p.cu == nullptr) {
        slot0 = seq * lin_segs(p.T, p.seg_tok);
    } else {
        __shared__ int64_t s_part[4];
        int64_t acc = 0;
        for (int64_t j = threadIdx.x; j < seq; j += 256) {
            int64_t b, e;
            seq_bounds(p.cu, p.T, j, b, e);
            acc += lin_segs(e - b, p.seg_tok);
        }
        acc = wave_sum_i64(acc);
        if (lane_id() == 0) s_part[threadIdx.x >> 6] = acc;
        __syncthreads();
        slot0 = s_part[0] + s_part[1] + s_part[2] + s_part[3];
    }
    const int64_t nseg = lin_segs(eos - bos, p.seg_tok);
    if (slot0 + nseg > p.items) return;  // overlapping requests: out of slots
    const int64_t i = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4;
    if (i >= p.elems) return;
    const auto &sc = p.s[blockIdx.z];
    const bool rev = sc.rev;
    const int64_t step = p.HV * p.elems;
    f32x4 cur = zero4();
    if (sc.s0) cur = *(const f32x4 *)(sc.s0 + (seq * p.HV + hv) * p.elems + i);
    const int64_t last = nseg - 1;
    float *base = sc.seg + (slot0 * p.HV + hv) * p.elems + i;
    const float *tot = sc.tot + slot0 * p.HV + hv;
    constexpr int U = 8;  // segments in flight
    for (int64_t k0 = 0; k0 < nseg; k0 += U) {
        f32x4 e[U];
        float f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = k0 + u, sg = rev ? nseg - 1 - k : k;
            e[u] = zero4();
            f[u] = 1.f;
            if (k < last) {
                e[u] = *(const f32x4 *)(base + sg * step);
                f[u] = __builtin_amdgcn_exp2f(tot[sg * p.HV]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = k0 + u, sg = rev ? nseg - 1 - k : k;
            if (k >= nseg) break;
            *(f32x4 *)(base + sg * step) = cur;
            cur = cur * f[u] + e[u];
        }
    }
}

// ---------------------------------------------------------------- gradient of the decays
// dg_t is the sum of D(i,j) scale (q_i.k_j)(do_i.v_j) over the pairs i >= t > j
// (the initial state an earlier row, the final state's gradient a later one),
// so  dg_t - dg_{t+1} = rho_q[t] - rho_k[t]:  what row t takes from earlier rows
// less what it gives to later ones.  Each segment is anchored at one border,
// where the sum is the product of the state and the gradient that meet there,
// so the running sums (64 bits) stay as short as a segment.  A block per
// segment and head: the product <S, R> (2 K V floats) and rho move once; 18 us
// for 20 segments of 16 heads and 128 x 128 states.
constexpr int DGT = 512;

// <S, R> of one head, for thread 0 (red: a double for each wave; every thread of the block calls it)
__device__ __forceinline__ double state_product(const float *S, const float *R, int64_t elems, double *red) {
    // 4 elements a thread and step, four steps' loads in flight (elems: 4096 to 32768)
    float acc = 0.f;
    for (int64_t i0 = (int64_t)threadIdx.x * 4; i0 < elems; i0 += 16 * DGT) {
        f32x4 u[4], v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t i = i0 + k * 4 * DGT;
            u[k] = v[k] = zero4();
            if (i < elems) {
                u[k] = *(const f32x4 *)(S + i);
                v[k] = *(const f32x4 *)(R + i);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            acc += (u[k][0] * v[k][0] + u[k][1] * v[k][1]) + (u[k][2] * v[k][2] + u[k][3] * v[k][3]);
    }
    double x = acc;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d, 64);
    if (lane_id() == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    double c = 0.0;
    if (threadIdx.x == 0)
#pragma unroll 1
        for (int i = 0; i < DGT / 64; ++i) c += red[i];
    return c;
}
// What row t's decay scales a border's product by.
__device__ __forceinline__ double row_decay(const LinDg &p, int64_t bi, int64_t t, int hv) {
    return p.g ? (double)__builtin_amdgcn_exp2f((float)decay_log2(p.g[bi * p.g_bs + t * p.g_ts + hv])) : 1.0;
}

__global__ void __launch_bounds__(DGT) gdp_lin_dg_k(LinDg p) {
    const uint32_t b = blockIdx.x;
    const int64_t id = b / (uint32_t)p.HV;
    const int hv = (int)(b % (uint32_t)p.HV);
    __shared__ double s_red[DGT / 64];
    __shared__ double s_carry;
    const LinItem it = lin_item(p.cu, p.nseq, p.T, p.seg_tok, id);
    if (it.seq < 0) return;
    const int64_t t0 = it.bos + it.seg * p.seg_tok;
    const int64_t t1 = t0 + p.seg_tok < it.eos ? t0 + p.seg_tok : it.eos;
    const int64_t bi = p.cu ? 0 : it.seq, tb0 = p.cu ? t0 : t0 - it.bos, tb1 = tb0 + (t1 - t0);
    // the anchor: at the segment's end (the state after it is the one entering
    // the next segment), for the last segment at its start unless nothing
    // comes in behind it
    const bool last = t1 == it.eos, fwd = last && !p.end_zero;
    const int64_t own = ((it.slot0 + it.seg) * p.HV + hv) * p.elems, step = p.HV * p.elems;
    const float *S = nullptr, *R = nullptr;
    int64_t through = -1;  // the row whose decay lies on the border
    if (!last && id + 1 < p.items) {
        S = p.s_in + own + step;
        R = p.r_in + own;
        through = tb1;
    } else if (fwd && it.seg > 0) {
        S = p.s_in + own;
        R = p.r_in + own - step;
        through = tb0;
    } else if (fwd && p.h0) {  // dh0 has the first row's decay in it
        S = p.h0 + (it.seq * p.HV + hv) * p.elems;
        R = p.dh0 + (it.seq * p.HV + hv) * p.elems;
    }
    const double c = S ? state_product(S, R, p.elems, s_red) : 0.0;
    if (threadIdx.x == 0) s_carry = through >= 0 ? c * row_decay(p, bi, through, hv) : c;
    __syncthreads();
    // the rows from the anchored border, DGT at a time
    const int64_t BT = p.B * p.T;
    for (int64_t k0 = 0; k0 < tb1 - tb0; k0 += DGT) {
        const int64_t k = k0 + threadIdx.x, t = fwd ? tb0 + k : tb1 - 1 - k;
        const bool in = k < tb1 - tb0;
        double d = 0.0;
        if (in) {
            const int64_t at = (int64_t)hv * BT + bi * p.T + t;
            for (int i = 0; i < p.nq; ++i) d += (double)p.rho_q[at + (int64_t)i * p.HV * BT];
            for (int i = 0; i < p.nk; ++i) d -= (double)p.rho_k[at + (int64_t)i * p.HV * BT];
            if (fwd) d = -d;
        }
        const double incl = wave_inclusive_sum_f64(d);
        const double tot = __shfl(incl, 63, 64);
        if (lane_id() == 0) s_red[threadIdx.x >> 6] = tot;
        __syncthreads();
        double upto = s_carry + incl;
#pragma unroll 1
        for (int i = 0; i < (int)(threadIdx.x >> 6); ++i) upto += s_red[i];
        const double v = fwd ? upto - d : upto;
        if (in) p.dg[(bi * p.T + t) * p.HV + hv] = (float)v;
        __syncthreads();
        if (threadIdx.x == DGT - 1) s_carry = upto;
        __syncthreads();
    }
}

// A decay per head wants the sum of dg over the rows: every pair, i - j times.
// Pairs inside a chunk are weighed and summed by themselves (rho_in_chunk);
// rho holds the pairs that cross a chunk's border.  For those, a span of n rows
// between borders whose products B, B' are known gives, with d = rho_q - rho_k of
// its s-th row, sum dg_t = (n+1)/2 B + (n-1)/2 B' + sum (s - (n+1)/2) d_s: the running
// sum from B', with its mismatch at B spread evenly over the rows.  An error of d
// thus counts n/2 times at most, so spans are short (LIN_SPAN rows, the walks
// leave the states at their borders).  Where nothing is known of one border
// (h0 without dh0, dht), the sum runs from the other.  A decay that takes a
// whole chunk below 2^-24 leaves no pairs over it: then rows weigh by their
// distance to their own chunk's ends, sum s rho_q + (n - s) rho_k, and no
// difference is taken at all.
// 8192 rows of 32 heads, 128 x 256: 1.3 to 3.3e-6 off with one anchor to 2048
// rows, 3 to 6e-7 now, for 5% of the call (the walks' 100 MB of states).  A block a
// segment and head, its spans one after the other (a block to each was 33 us for
// 34 here, but 596 for 177 with 1000 requests of 20 rows); bound by the borders'
// states, 134 MB here (33 us, 41 in an unbroken run of calls).
__global__ void __launch_bounds__(DGT) gdp_lin_dg_spans_k(LinDg p) {
    const uint32_t b = blockIdx.x;
    const int64_t id = b / (uint32_t)p.HV;
    const int hv = (int)(b % (uint32_t)p.HV);
    __shared__ double s_red[DGT / 64];
    const LinItem it = lin_item(p.cu, p.nseq, p.T, p.seg_tok, id);
    const int64_t t0 = it.bos + it.seg * p.seg_tok;
    const int64_t t1 = it.seq < 0 ? t0 : t0 + p.seg_tok < it.eos ? t0 + p.seg_tok : it.eos;
    const int64_t bi = p.cu ? 0 : it.seq, BT = p.B * p.T;
    const bool start_known = !p.h0 || p.dh0;  // of a sequence
    const bool none_over = decay_log2(p.g[hv]) * p.chunk < -24.0;

    double sum = 0.0;
    for (int sp = 0; sp < p.spans; ++sp) {
        const int64_t a0 = t0 + (int64_t)sp * LIN_SPAN, a1 = a0 + LIN_SPAN < t1 ? a0 + LIN_SPAN : t1;
        if (a0 >= a1) break;
        const int n = (int)(a1 - a0);
        const bool first = a0 == it.bos, end_known = a1 < it.eos || p.end_zero, apart = none_over && end_known;
        const int64_t tb0 = p.cu ? a0 : a0 - it.bos;

        // the product at the span's first row: its weight in this span and in the one before
        double wb = 0.0;
        if (!apart && (!first || start_known)) wb = end_known ? 0.5 * (n + 1) : (double)n;
        if (!first && !none_over) {
            const int before = sp > 0 ? LIN_SPAN : (int)(p.seg_tok - (int64_t)(p.spans - 1) * LIN_SPAN);
            wb += a0 - before > it.bos || start_known ? 0.5 * (before - 1) : (double)before;
        }
        const float *S = nullptr, *R = nullptr;
        if (wb != 0.0) {
            const int64_t slot = it.slot0 + it.seg;
            if (sp > 0) {
                const int64_t at = ((bi * p.T + tb0) / LIN_SPAN * p.HV + hv) * p.elems;
                S = p.s_mid + at;
                R = p.r_mid + at;
            } else if (!first) {
                S = p.s_in + (slot * p.HV + hv) * p.elems;
                R = p.r_in + ((slot - 1) * p.HV + hv) * p.elems;
            } else if (p.h0) {  // dh0 has the first row's decay in it
                S = p.h0 + (it.seq * p.HV + hv) * p.elems;
                R = p.dh0 + (it.seq * p.HV + hv) * p.elems;
            }
        }
        for (int k = threadIdx.x; k < n; k += DGT) {
            const int64_t at = (int64_t)hv * BT + bi * p.T + tb0 + k;
            double q = 0.0, r = 0.0;
            for (int i = 0; i < p.nq; ++i) q += (double)p.rho_q[at + (int64_t)i * p.HV * BT];
            for (int i = 0; i < p.nk; ++i) r += (double)p.rho_k[at + (int64_t)i * p.HV * BT];
            for (int i = 0; i < p.nq; ++i) sum += (double)p.rho_in_chunk[at + (int64_t)i * p.HV * BT];
            if (apart) {
                const int lo = k / p.chunk * p.chunk, rows = n - lo < p.chunk ? n - lo : p.chunk;
                sum += (k - lo + 1) * q + (rows - 1 - (k - lo)) * r;
            } else {
                const double w = !end_known ? k + 1 - n : first && !start_known ? k + 1 : k + 1 - 0.5 * (n + 1);
                sum += w * (q - r);
            }
        }
        if (S) {
            const double c = state_product(S, R, p.elems, s_red);
            if (threadIdx.x == 0) sum += wb * (first ? c : c * row_decay(p, bi, tb0, hv));
            __syncthreads();
        }
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
    if (lane_id() == 0) s_red[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int i = 0; i < DGT / 64; ++i) t += s_red[i];
        p.part[id * p.HV + hv] = t;
    }
}

// dg of a decay per head: the sum over every segment, in a fixed order
__global__ void __launch_bounds__(256) gdp_lin_dg_head_k(const double *part, int64_t items, int HV, float *out) {
    __shared__ double s_red[4];
    const int hv = blockIdx.x;
    double x = 0.0;
    for (int64_t i = threadIdx.x; i < items; i += 256) x += part[i * HV + hv];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d, 64);
    if (lane_id() == 0) s_red[threadIdx.x >> 6] = x;
    __syncthreads();
    if (threadIdx.x == 0) out[hv] = (float)((s_red[0] + s_red[1]) + (s_red[2] + s_red[3]));
}

// Gradients of shared key heads: the sum of r neighbouring heads' float rows,
// rounded once.  One thread per 4 elements; tokens outside every request are
// left alone (requests follow each other, so those lie before the first
// offset or behind the last).  Bound by the float rows that the walks have just
// written (60 us for 248 MB of them).
template <typename T>
__global__ void __launch_bounds__(256) gdp_lin_group_k(LinGroup p) {
    const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (u >= p.units) return;
    const int64_t row = u / p.upr;  // (token, key head)
    if (p.cu) {
        const int64_t t = row / p.H;
        if (t < p.cu[0] || t >= p.cu[p.nseq]) return;
    }
    const float *x = p.x[blockIdx.y] + (row * p.r * p.upr + u % p.upr) * 4;
    f32x4 s = *(const f32x4 *)x;
    for (int i = 1; i < p.r; ++i) s += *(const f32x4 *)(x + (int64_t)i * p.upr * 4);
    typename Frag<T>::half o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = from_f32<T>(s[i]);
    *(typename Frag<T>::half *)((T *)p.y[blockIdx.y] + u * 4) = o;
}

// Gradients of tokens outside every request: zero.  A block looks after 64
// tokens and mostly finds them inside.
__global__ void __launch_bounds__(256) gdp_lin_outside_k(LinOutside p) {
    const int64_t t0 = (int64_t)blockIdx.x * 64, t1 = t0 + 64 < p.T ? t0 + 64 : p.T;
    // requests follow each other from the first offset to the last
    int64_t lo = 0, hi = 0;
    if (p.nseq > 0) {
        lo = p.cu[0] < 0 ? 0 : p.cu[0];
        hi = p.cu[p.nseq];
    }
    if (t0 >= lo && t1 <= hi) return;
    for (int64_t t = t0; t < t1; ++t) {
        if (t >= lo && t < hi) continue;
        for (int i = 0; i < 4; ++i) {
            uint32_t *y = (uint32_t *)p.y[i];
            if (!y) continue;
            for (int64_t w = threadIdx.x; w < p.words[i]; w += 256) y[t * p.words[i] + w] = 0;
        }
    }
}

// ---------------------------------------------------------------- launches
template <typename T, int DA, int DC, int NS, int NQ, bool OUT>
static hipError_t launch_walk_t(const LinWalks &w, hipStream_t stream) {
    const int64_t blocks = w.w[0].items * w.w[0].HV * (w.w[0].dc / DC);
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((gdp_lin_walk_k<T, DA, DC, NS, NQ, OUT>), dim3((unsigned)blocks, w.n), dim3(4 * DC), 0, stream, w);
    return hipGetLastError();
}

template <typename T, int NS, int NQ, bool OUT>
static hipError_t launch_walk_dims(const LinWalks &w, hipStream_t stream) {
    const int da = w.w[0].da, dc = w.w[0].dc;
    if (da == 64)
        return dc == 64 ? launch_walk_t<T, 64, 64, NS, NQ, OUT>(w, stream) : launch_walk_t<T, 64, 128, NS, NQ, OUT>(w, stream);
    return dc == 64 ? launch_walk_t<T, 128, 64, NS, NQ, OUT>(w, stream) : launch_walk_t<T, 128, 128, NS, NQ, OUT>(w, stream);
}

hipError_t launch_lin_rows(const LinWalks &w, gdp_dtype dtype, bool exact, hipStream_t stream) {
    if (w.w[0].items == 0) return hipSuccess;
    if (dtype == GDP_F32) return launch_walk_dims<float, 1, 1, true>(w, stream);
    return exact ? launch_walk_dims<bf16, 3, 2, true>(w, stream) : launch_walk_dims<bf16, 2, 2, true>(w, stream);
}

hipError_t launch_lin_segments(const LinWalks &w, gdp_dtype dtype, bool exact, bool dg, hipStream_t stream) {
    if (w.w[0].items == 0) return hipSuccess;
    if (dtype == GDP_F32) return dg ? launch_walk_dims<float, 1, 3, false>(w, stream) : launch_walk_dims<float, 1, 1, false>(w, stream);
    if (dg) return launch_walk_dims<bf16, 3, 3, false>(w, stream);
    return exact ? launch_walk_dims<bf16, 3, 2, false>(w, stream) : launch_walk_dims<bf16, 2, 2, false>(w, stream);
}

// Columns of c that one walk of the gradients takes: as many waves in each of the three.
int lin_grads_slice(int K, int V) { return K == 64 || V == 64 ? 64 : 128; }

template <typename T, int K, int V, int NS, int NQ, int ND, bool DOT>
static hipError_t launch_grads_t(const LinWalks &w, hipStream_t stream) {
    constexpr int SL = K == 64 || V == 64 ? 64 : 128;
    const int64_t most = w.w[0].items * w.w[0].HV * ((K > V ? K : V) / SL);
    if (most > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((gdp_lin_grads_k<T, K, V, SL, NS, NQ, ND, DOT>), dim3((unsigned)most, 3), dim3(4 * SL), 0, stream, w);
    return hipGetLastError();
}
template <typename T, int NS, int NQ, int ND, bool DOT>
static hipError_t launch_grads_dims(const LinWalks &w, hipStream_t stream) {
    switch (w.w[2].da * 1000 + w.w[2].dc) {
    case 64064: return launch_grads_t<T, 64, 64, NS, NQ, ND, DOT>(w, stream);
    case 64128: return launch_grads_t<T, 64, 128, NS, NQ, ND, DOT>(w, stream);
    case 64256: return launch_grads_t<T, 64, 256, NS, NQ, ND, DOT>(w, stream);
    case 128064: return launch_grads_t<T, 128, 64, NS, NQ, ND, DOT>(w, stream);
    case 128128: return launch_grads_t<T, 128, 128, NS, NQ, ND, DOT>(w, stream);
    case 128256: return launch_grads_t<T, 128, 256, NS, NQ, ND, DOT>(w, stream);
    default: return hipErrorInvalidValue;
    }
}
// Parts of bf16 in the state's products.  What leaves in float32 (ht, dh0, and
// dg through rho) takes three, 24 bits: with two, dg was 1e-5 off and ht 2e-6
// (relative to 64 bits; with three 1e-6 and 2e-7, as float32 sums are).  What
// only reaches bf16 rows takes two, 16 bits: the scores, the decayed rows and
// the state as the operand of S a.  A row is then off by its own rounding,
// 1.65e-3; with scores and operand in one part it was 2.3e-3, and elements
// whose terms cancel were off by many times their rounding.  The second parts
// cost 3 to 10% of a call (packed prompts 119 to 129 us, 32768 tokens 210 to 230).
hipError_t launch_lin_grads(const LinWalks &w, gdp_dtype dtype, bool dot, hipStream_t stream) {
    if (w.w[0].items == 0) return hipSuccess;
    if (dtype == GDP_F32)
        return dot ? launch_grads_dims<float, 1, 1, 1, true>(w, stream) : launch_grads_dims<float, 1, 1, 1, false>(w, stream);
    if (w.w[2].s_out)
        return dot ? launch_grads_dims<bf16, 3, 3, 3, true>(w, stream) : launch_grads_dims<bf16, 2, 2, 3, false>(w, stream);
    return dot ? launch_grads_dims<bf16, 3, 3, 2, true>(w, stream) : launch_grads_dims<bf16, 2, 2, 2, false>(w, stream);
}

hipError_t launch_lin_scan(const LinScan &p, hipStream_t stream) {
    if (p.nseq == 0) return hipSuccess;
    hipLaunchKernelGGL(gdp_lin_scan_k, dim3((unsigned)(p.nseq * p.HV), (unsigned)(p.elems / 1024), p.n), dim3(256), 0,
                       stream, p);
    return hipGetLastError();
}

hipError_t launch_lin_dg(const LinDg &p, float *dg_head, hipStream_t stream) {
    if (p.items > 0) {
        const dim3 grid((unsigned)(p.items * p.HV));
        if (p.dg) hipLaunchKernelGGL(gdp_lin_dg_k, grid, dim3(DGT), 0, stream, p);
        else hipLaunchKernelGGL(gdp_lin_dg_spans_k, grid, dim3(DGT), 0, stream, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!dg_head) return hipSuccess;
    hipLaunchKernelGGL(gdp_lin_dg_head_k, dim3((unsigned)p.HV), dim3(256), 0, stream, p.part, p.items, p.HV, dg_head);
    return hipGetLastError();
}

hipError_t launch_lin_outside(const LinOutside &p, hipStream_t stream) {
    hipLaunchKernelGGL(gdp_lin_outside_k, dim3((unsigned)((p.T + 63) / 64)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_lin_group(const LinGroup &p, gdp_dtype dtype, hipStream_t stream) {
    if (p.units == 0) return hipSuccess;
    const dim3 grid((unsigned)((p.units + 255) / 256), 2);
    if (dtype == GDP_BF16) hipLaunchKernelGGL(gdp_lin_group_k<bf16>, grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(gdp_lin_group_k<float>, grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace gdp

// linrec.hip -- gated linear recurrence, a state of one number per channel:
//   h_t = a_t h_{t-1} + c_t x_t,  y_t = h_t,   c = 1 or 1 - a
// and its gradients, with l_t that of h_t:
//   l_t = dy_t + a_{t+1} l_{t+1},  dx = c l,  da = l (h_{t-1} - [c = 1 - a] x),
//   dg = a da  (a = e^g)  or  a (1 - a) da  (a = 1 / (1 + e^-g))
//
// A run of rows takes the state h to A h + B, and runs compose, so a tile of
// rows is cut over the threads of a block: each walks TT rows of E channels
// from a zero state, the block joins the runs of every channel in order, and
// the threads walk their rows again from the state that enters them.
#include "rows.h"

namespace gdp {

namespace {

constexpr int LNT = 256;

// The decay a of a row in one number d, a = 1 + d where d < 0, else a = d:
// close to one its distance from one is kept, which a rounding of a itself
// would lose and compound over the rows that a slow channel remembers; a fast
// channel keeps a.
__device__ __forceinline__ float decay_log(float g) {
    // e^g - 1 by its series near zero, where the difference would cancel
    float p = fmaf(g, 1.0f / 5040.0f, 1.0f / 720.0f);
    p = fmaf(g, p, 1.0f / 120.0f);
    p = fmaf(g, p, 1.0f / 24.0f);
    p = fmaf(g, p, 1.0f / 6.0f);
    p = fmaf(g, p, 0.5f);
    p = fmaf(g * g, p, g);
    return g < 0.f && g >= -0.35f ? p : exp_exact(g);
}
__device__ __forceinline__ float decay_sigmoid(float g) {
    const float r = __builtin_amdgcn_rcpf(1.0f + exp_exact(fabsf(g)));
    return g > 0.f ? -fmaxf(r, 1.17549435e-38f) : r;  // never -0, which would be a = 0
}
template <int N>
__device__ __forceinline__ void decays(float (&d)[N], bool sigmoid) {
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = decay_sigmoid(d[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = decay_log(d[i]);
    }
}
__device__ __forceinline__ float keep(float d, float h) { return fmaf(d, h, d < 0.f ? h : 0.f); }  // a h
__device__ __forceinline__ float rest(float d) { return d < 0.f ? -d : 1.0f - d; }                 // 1 - a

template <bool COMP>
__device__ __forceinline__ float step(float h, float d, float x) {
    return COMP ? fmaf(rest(d), x, keep(d, h)) : keep(d, h) + x;
}

// What a run of rows does to the state; A < 0: it ends with B whatever came in
// (a sequence begins inside), so that nothing of another one is multiplied.
struct Run {
    float A, B;
};
__device__ __forceinline__ float enter(Run r, float h) { return r.A < 0.f ? r.B : fmaf(r.A, h, r.B); }

}  // namespace

// PHASE 0: what each tile does to the state -> space [tiles][2][C];
// PHASE 1: the rows.
template <typename T, typename G, int E, int TT, bool COMP, int PHASE>
__global__ void __launch_bounds__(LNT) gdp_linrec_k(LinRec p) {
    __shared__ uint8_t code[LNT * TT];
    __shared__ int seq[LNT * TT];
    __shared__ float ra[LNT * E], rb[LNT * E];
    const Place<LNT, E, TT> at(p.lognx, p.C, blockIdx.x, blockIdx.y);
    const int w = at.nx * E;  // channels of the block

    Chans<T, E> xr[TT];
    Chans<G, E> gr[TT];
    load_rows<T, E, TT>(xr, p.x, p.m, at.row0, at.col, at.live);
    load_rows<G, E, TT>(gr, p.g, p.m, at.row0, at.col, at.live);
    find_rows<LNT>(p.m, at.tile0, at.ny * TT, code, seq);
    __syncthreads();

    float d[TT][E];
    uint32_t in = 0, first = 0, last = 0;
    const int k0 = at.ty * TT;
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        gr[i].to(d[i]);
        decays<E>(d[i], p.sigmoid);
        const uint32_t c = code[k0 + i];
        in |= (c & ROW_IN) << i;
        first |= (uint32_t)row_first(c) << i;
        last |= (uint32_t)row_last(c) << i;
    }

    Run run[E];
#pragma unroll
    for (int e = 0; e < E; ++e) run[e] = {1.f, 0.f};
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        float x[E];
        xr[i].to(x);
        if (first >> i & 1) {
            float h[E];
            load_state<E>(h, at.live ? p.h0 : nullptr, seq[k0 + i], p.C, at.col);
#pragma unroll
            for (int e = 0; e < E; ++e) run[e] = {-1.f, h[e]};
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            run[e].B = step<COMP>(run[e].B, d[i][e], x[e]);
            if (run[e].A >= 0.f) run[e].A = keep(d[i][e], run[e].A);
        }
        if (!(in >> i & 1))
#pragma unroll
            for (int e = 0; e < E; ++e) run[e] = {-1.f, 0.f};
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        ra[at.ty * w + at.tx * E + e] = run[e].A;
        rb[at.ty * w + at.tx * E + e] = run[e].B;
    }
    __syncthreads();

    // one thread a channel: its runs in order
    const int c = (int)(blockIdx.y * w) + (int)threadIdx.x;
    float *agg = (float *)p.space;
    if ((int)threadIdx.x < w && c < p.C) {
        if constexpr (PHASE == 0) {
            Run all{1.f, 0.f};
            for (int y = 0; y < at.ny; ++y) {
                const float A = ra[y * w + threadIdx.x], B = rb[y * w + threadIdx.x];
                all = {A < 0.f ? -1.f : all.A < 0.f ? -1.f : A * all.A, A < 0.f ? B : fmaf(A, all.B, B)};
            }
            agg[(int64_t)blockIdx.x * 2 * p.C + c] = all.A;
            agg[(int64_t)blockIdx.x * 2 * p.C + p.C + c] = all.B;
        } else {
            float h = 0.f;
            for (int64_t t = 0; t < (int64_t)blockIdx.x; ++t) h = enter({agg[t * 2 * p.C + c], agg[t * 2 * p.C + p.C + c]}, h);
            for (int y = 0; y < at.ny; ++y) {
                const Run r{ra[y * w + threadIdx.x], rb[y * w + threadIdx.x]};
                rb[y * w + threadIdx.x] = h;
                h = enter(r, h);
            }
        }
    }
    if constexpr (PHASE == 1) {
        __syncthreads();
        if (!at.live) return;
        float h[E];
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = rb[at.ty * w + at.tx * E + e];
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (!(in >> i & 1)) continue;
            float x[E];
            xr[i].to(x);
            if (first >> i & 1) load_state<E>(h, p.h0, seq[k0 + i], p.C, at.col);
#pragma unroll
            for (int e = 0; e < E; ++e) h[e] = step<COMP>(h[e], d[i][e], x[e]);
            Chans<T, E> o;
            o.from(h);
            o.store((T *)p.y + (int64_t)(at.row0 + i) * p.C + at.col);
            if (p.ht && (last >> i & 1)) store_state<E>(p.ht, seq[k0 + i], p.C, at.col, h);
        }
        if (p.ht && at.ty == 0)
            for (int q = blockIdx.x; q < p.m.nseq; q += gridDim.x)
                if (seq_empty(p.m, q)) {
                    float z[E];
                    load_state<E>(z, p.h0, q, p.C, at.col);
                    store_state<E>(p.ht, q, p.C, at.col, z);
                }
    }
}

// Backwards.  PHASE 0: what each tile does to the state (forwards) and to a l
// (from its last row to its first) -> space [tiles][4][C]; PHASE 1: the rows.
template <typename T, typename G, int E, int TT, bool COMP, int PHASE>
__global__ void __launch_bounds__(LNT) gdp_linrec_bwd_k(LinRec p) {
    __shared__ uint8_t code[LNT * TT];
    __shared__ int seq[LNT * TT];
    __shared__ float ra[2][LNT * E], rb[2][LNT * E];
    const Place<LNT, E, TT> at(p.lognx, p.C, blockIdx.x, blockIdx.y);
    const int w = at.nx * E;

    Chans<T, E> xr[TT], dr[TT];
    Chans<G, E> gr[TT];
    load_rows<T, E, TT>(xr, p.x, p.m, at.row0, at.col, at.live);
    load_rows<G, E, TT>(gr, p.g, p.m, at.row0, at.col, at.live);
    load_rows<T, E, TT>(dr, p.dy, p.m, at.row0, at.col, at.live);
    find_rows<LNT>(p.m, at.tile0, at.ny * TT, code, seq);
    __syncthreads();

    float d[TT][E];
    uint32_t in = 0, first = 0, last = 0;
    const int k0 = at.ty * TT;
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        gr[i].to(d[i]);
        decays<E>(d[i], p.sigmoid);
        const uint32_t c = code[k0 + i];
        in |= (c & ROW_IN) << i;
        first |= (uint32_t)row_first(c) << i;
        last |= (uint32_t)row_last(c) << i;
    }
    Run run[E], back[E];
#pragma unroll
    for (int e = 0; e < E; ++e) run[e] = back[e] = {1.f, 0.f};
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        float x[E];
        xr[i].to(x);
        if (first >> i & 1) {
            float h[E];
            load_state<E>(h, at.live ? p.h0 : nullptr, seq[k0 + i], p.C, at.col);
#pragma unroll
            for (int e = 0; e < E; ++e) run[e] = {-1.f, h[e]};
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            run[e].B = step<COMP>(run[e].B, d[i][e], x[e]);
            if (run[e].A >= 0.f) run[e].A = keep(d[i][e], run[e].A);
        }
        if (!(in >> i & 1))
#pragma unroll
            for (int e = 0; e < E; ++e) run[e] = {-1.f, 0.f};
    }
#pragma unroll
    for (int i = TT - 1; i >= 0; --i) {
        float dy[E];
        dr[i].to(dy);
        if (last >> i & 1) {
            float z[E];
            load_state<E>(z, at.live ? p.dht : nullptr, seq[k0 + i], p.C, at.col);
#pragma unroll
            for (int e = 0; e < E; ++e) back[e] = {-1.f, z[e]};
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float l = dy[e] + back[e].B;
            back[e].B = keep(d[i][e], l);
            if (back[e].A >= 0.f) back[e].A = keep(d[i][e], back[e].A);
        }
        if (!(in >> i & 1))
#pragma unroll
            for (int e = 0; e < E; ++e) back[e] = {-1.f, 0.f};
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int k = at.ty * w + at.tx * E + e;
        ra[0][k] = run[e].A;
        rb[0][k] = run[e].B;
        ra[1][k] = back[e].A;
        rb[1][k] = back[e].B;
    }
    __syncthreads();
    const int c = (int)(blockIdx.y * w) + (int)threadIdx.x;
    float *agg = (float *)p.space;
    const int64_t C = p.C;
    if ((int)threadIdx.x < w && c < p.C) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            if constexpr (PHASE == 0) {
                Run all{1.f, 0.f};
                for (int j = 0; j < at.ny; ++j) {
                    const int y = z ? at.ny - 1 - j : j;
                    const float A = ra[z][y * w + threadIdx.x], B = rb[z][y * w + threadIdx.x];
                    all = {A < 0.f ? -1.f : all.A < 0.f ? -1.f : A * all.A, A < 0.f ? B : fmaf(A, all.B, B)};
                }
                agg[((int64_t)blockIdx.x * 4 + 2 * z) * C + c] = all.A;
                agg[((int64_t)blockIdx.x * 4 + 2 * z + 1) * C + c] = all.B;
            } else {
                float h = 0.f;
                if (z == 0)
                    for (int64_t t = 0; t < (int64_t)blockIdx.x; ++t) h = enter({agg[t * 4 * C + c], agg[(t * 4 + 1) * C + c]}, h);
                else
                    for (int64_t t = (int64_t)gridDim.x - 1; t > (int64_t)blockIdx.x; --t)
                        h = enter({agg[(t * 4 + 2) * C + c], agg[(t * 4 + 3) * C + c]}, h);
                for (int j = 0; j < at.ny; ++j) {
                    const int y = z ? at.ny - 1 - j : j;
                    const Run r{ra[z][y * w + threadIdx.x], rb[z][y * w + threadIdx.x]};
                    rb[z][y * w + threadIdx.x] = h;
                    h = enter(r, h);
                }
            }
        }
    }
    if constexpr (PHASE == 1) {
        __syncthreads();
        if (!at.live) return;
        float h[E], m[E], hp[TT][E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            h[e] = rb[0][at.ty * w + at.tx * E + e];
            m[e] = rb[1][at.ty * w + at.tx * E + e];
        }
#pragma unroll
        for (int i = 0; i < TT; ++i) {  // hp: what da is l times
            float x[E];
            xr[i].to(x);
            if (first >> i & 1) load_state<E>(h, p.h0, seq[k0 + i], p.C, at.col);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                hp[i][e] = COMP ? h[e] - x[e] : h[e];
                h[e] = step<COMP>(h[e], d[i][e], x[e]);
            }
        }
#pragma unroll
        for (int i = TT - 1; i >= 0; --i) {
            if (at.row0 + i >= p.m.rows) continue;
            float dy[E], dx[E], dg[E];
            dr[i].to(dy);
            if (last >> i & 1) load_state<E>(m, p.dht, seq[k0 + i], p.C, at.col);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float l = dy[e] + m[e], al = keep(d[i][e], l), c = rest(d[i][e]);
                dx[e] = COMP ? c * l : l;
                dg[e] = hp[i][e] * (p.sigmoid ? c * al : al);
                m[e] = al;
            }
            if (!(in >> i & 1))
#pragma unroll
                for (int e = 0; e < E; ++e) dx[e] = dg[e] = 0.f;
            Chans<T, E> ox;
            Chans<G, E> og;
            ox.from(dx);
            og.from(dg);
            ox.store((T *)p.dx + (int64_t)(at.row0 + i) * p.C + at.col);
            og.store((G *)p.dg + (int64_t)(at.row0 + i) * p.C + at.col);
            if (p.dh0 && (first >> i & 1)) store_state<E>(p.dh0, seq[k0 + i], p.C, at.col, m);
        }
        if (p.dh0 && at.ty == 0)
            for (int q = blockIdx.x; q < p.m.nseq; q += gridDim.x)
                if (seq_empty(p.m, q)) {
                    float z[E];
                    load_state<E>(z, p.dht, q, p.C, at.col);
                    store_state<E>(p.dh0, q, p.C, at.col, z);
                }
    }
}

// S new tokens of a request, its state in registers between the load from its
// slot and the store.
template <typename T, typename G, int E>
__global__ void __launch_bounds__(LNT) gdp_linrec_decode_k(gdp_linrec_decode_args a) {
    const int per = (a.C + E - 1) / E;
    const int64_t id = (int64_t)blockIdx.x * LNT + threadIdx.x;
    const int64_t req = id / per;
    if (req >= a.n) return;
    const int col = (int)(id - req * per) * E;
    const int64_t slot = a.slots ? (int64_t)a.slots[req] : req;
    T *y = (T *)a.y + req * a.S * (int64_t)a.C + col;
    if (slot < 0 || slot >= a.pool) {
        Chans<T, E> z;
        z.zero();
        for (int64_t t = 0; t < a.S; ++t) z.store(y + t * a.C);
        return;
    }
    float h[E];
    load_state<E>(h, a.state + slot * a.C, 0, a.C, col);
    const T *xp = (const T *)a.x + req * a.x_n_stride + col;
    const G *gp = (const G *)a.g + req * a.g_n_stride + col;
    for (int64_t t = 0; t < a.S; ++t) {
        Chans<T, E> xr;
        Chans<G, E> gr;
        xr.load(xp + t * a.x_t_stride);
        gr.load(gp + t * a.g_t_stride);
        float x[E], d[E];
        xr.to(x);
        gr.to(d);
        decays<E>(d, a.decay == GDP_DECAY_SIGMOID);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = a.complement ? step<true>(h[e], d[e], x[e]) : step<false>(h[e], d[e], x[e]);
        xr.from(h);
        xr.store(y + t * a.C);
    }
    store_state<E>(a.state + slot * a.C, 0, a.C, col, h);
}

namespace {

// Rows a thread holds: 8 of 16 bytes, 16 single elements; half of it backwards,
// where three tensors and two states are held.
constexpr int rows_of(int E, bool back) { return (E == 1 ? 16 : 8) / (back ? 2 : 1); }

int lanes_log(const LinRec &p, gdp_dtype dtype) {
    const int E = !p.vec ? 1 : dtype == GDP_BF16 ? 8 : 4;
    int l = 0;
    while (l < (E == 1 ? 6 : 4) && (E << l) < p.C) ++l;
    return l;
}
int elems_of(const LinRec &p, gdp_dtype dtype) { return !p.vec ? 1 : dtype == GDP_BF16 ? 8 : 4; }
int64_t tiles_of(const LinRec &p, gdp_dtype dtype, bool back) {
    const int64_t per = (int64_t)(LNT >> lanes_log(p, dtype)) * rows_of(elems_of(p, dtype), back);
    return (p.m.rows + per - 1) / per;
}

template <typename T, typename G, int E, bool COMP>
hipError_t run_linrec(const LinRec &p, bool back, hipStream_t stream) {
    const int w = E << p.lognx;
    const dim3 grid((unsigned)(p.tiles > 0 ? p.tiles : 1), (unsigned)((p.C + w - 1) / w));
    constexpr int TF = rows_of(E, false), TB = rows_of(E, true);
    if (back) {
        if (p.tiles > 1) hipLaunchKernelGGL((gdp_linrec_bwd_k<T, G, E, TB, COMP, 0>), grid, dim3(LNT), 0, stream, p);
        hipLaunchKernelGGL((gdp_linrec_bwd_k<T, G, E, TB, COMP, 1>), grid, dim3(LNT), 0, stream, p);
    } else {
        if (p.tiles > 1) hipLaunchKernelGGL((gdp_linrec_k<T, G, E, TF, COMP, 0>), grid, dim3(LNT), 0, stream, p);
        hipLaunchKernelGGL((gdp_linrec_k<T, G, E, TF, COMP, 1>), grid, dim3(LNT), 0, stream, p);
    }
    return hipGetLastError();
}
template <typename T, typename G, int E>
hipError_t run_kind(const LinRec &p, bool back, hipStream_t stream) {
    return p.complement ? run_linrec<T, G, E, true>(p, back, stream) : run_linrec<T, G, E, false>(p, back, stream);
}
hipError_t run_types(LinRec p, gdp_dtype dtype, bool back, hipStream_t stream) {
    p.lognx = lanes_log(p, dtype);
    p.tiles = (int)tiles_of(p, dtype, back);
    if (dtype == GDP_F32) return p.vec ? run_kind<float, float, 4>(p, back, stream) : run_kind<float, float, 1>(p, back, stream);
    if (p.g32) return p.vec ? run_kind<bf16, float, 8>(p, back, stream) : run_kind<bf16, float, 1>(p, back, stream);
    return p.vec ? run_kind<bf16, bf16, 8>(p, back, stream) : run_kind<bf16, bf16, 1>(p, back, stream);
}

template <typename T, typename G, int E>
hipError_t run_decode(const gdp_linrec_decode_args &a, hipStream_t stream) {
    const int64_t threads = a.n * ((a.C + E - 1) / E);
    hipLaunchKernelGGL((gdp_linrec_decode_k<T, G, E>), dim3((unsigned)((threads + LNT - 1) / LNT)), dim3(LNT), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

bool linrec_fits(const LinRec &p, gdp_dtype dtype, bool backward) {
    return tiles_of(p, dtype, backward) * LNT <= 0xffffffffll;
}
int64_t linrec_space(const LinRec &p, gdp_dtype dtype, bool backward) {
    const int64_t tiles = tiles_of(p, dtype, backward);
    return tiles > 1 ? tiles * (backward ? 4 : 2) * p.C * (int64_t)sizeof(float) : 0;
}
hipError_t launch_linrec(LinRec p, gdp_dtype dtype, hipStream_t stream) { return run_types(p, dtype, false, stream); }
hipError_t launch_linrec_bwd(LinRec p, gdp_dtype dtype, hipStream_t stream) { return run_types(p, dtype, true, stream); }

hipError_t launch_linrec_decode(const gdp_linrec_decode_args &a, bool vec, hipStream_t stream) {
    if (a.dtype == GDP_F32) return vec ? run_decode<float, float, 4>(a, stream) : run_decode<float, float, 1>(a, stream);
    if (a.g_dtype == GDP_F32) return vec ? run_decode<bf16, float, 8>(a, stream) : run_decode<bf16, float, 1>(a, stream);
    return vec ? run_decode<bf16, bf16, 8>(a, stream) : run_decode<bf16, bf16, 1>(a, stream);
}

}  // namespace gdp

// linrec.hip -- gated linear recurrence, a state of one number per channel:
//   h_t = a_t h_{t-1} + c_t x_t,  y_t = h_t,   c = 1 or 1 - a
// and its gradients, with l_t that of h_t:
//   l_t = dy_t + a_{t+1} l_{t+1},  dx = c l,  da = l (h_{t-1} - [c = 1 - a] x),
//   dg = a da  (a = e^g)  or  a (1 - a) da  (a = 1 / (1 + e^-g))
//
// A run of rows takes the state h to A h + B, and runs compose, so a tile of
// rows is cut over the threads of a block: each walks TT rows of E channels
// from a zero state, the block joins the runs of every channel in order, and
// the threads walk their rows again from the state that enters them.  Tiles are
// all under way at once and hand the state on while they run (below), so that
// forwards every tensor is moved once.  Backwards a first pass over x and g
// leaves the states at the tiles' borders, since a tile cannot wait for both
// its neighbours.
//
// Measured, with inputs that are not in the caches: 32768 x 2048 rows in
// bfloat16 with float32 log decays 120 us (537 MB, 4.5 TB/s, a large copy
// reaching 5.1), a ragged pack of 15151 x 2048 gates 65 (186 MB); gradients of
// 32768 x 2048 gates 233: 6 for clearing the words, 64 for the states (268 MB),
// 163 for the rows (671 MB).  Left over is what a block waits: for its number,
// its rows, and the state, some 12 us of which the other two or three blocks of
// its compute unit hide the most.  float32 rows of 16384 x 2000 take 99 and 207
// us (floors 78 and 129).  Rows that do not start on 16 bytes go by single
// elements (16384 x 1999 bfloat16: 101 and 221 us, 16384 x 2000: 62 and 137).
#include "rows.h"

namespace gdp {

namespace {

constexpr int LNT = 256;
constexpr int W = 64;  // channels of a block: those that a wave joins, a lane each

// The decay a of a row and channel in one number.  Near one it is the distance
// a - 1, whose rounding a slow channel does not compound over the rows that it
// remembers as it would one of a; elsewhere a, so that what little a fast
// channel keeps is as exact.  The number's last bit says which: both a and 1 - a
// are known to a few 2^-24 of themselves for every a, above one too.  Rows in
// bfloat16 take the hardware's power of a rounded product, (2 + |g|) 2^-24 off.
namespace decay {
constexpr float LOG2E = 1.44269502f;
template <typename T> __device__ __forceinline__ float log(float g) {
    // e^g - 1 by its series near zero, where the difference would cancel
    constexpr bool LONG = std::is_same<T, float>::value;
    float p = LONG ? fmaf(g, 1.0f / 5040.0f, 1.0f / 720.0f) : 1.0f / 720.0f;
    p = fmaf(g, p, 1.0f / 120.0f);
    p = fmaf(g, p, 1.0f / 24.0f);
    p = fmaf(g, p, 1.0f / 6.0f);
    p = fmaf(g, p, 0.5f);
    p = fmaf(g * g, p, g);
    const bool near = fabsf(g) <= (LONG ? 0.35f : 0.25f);
    const float v = near ? p : LONG ? exp_exact(g) : __builtin_amdgcn_exp2f(g * LOG2E);
    return __uint_as_float((__float_as_uint(v) & ~1u) | (near ? 1u : 0u));
}
template <typename T> __device__ __forceinline__ float sigmoid(float g) {
    // r: the smaller one of a and 1 - a, which are kept as r, and as -r with the last bit set: where q is negative
    const float q = g * -LOG2E;
    const float e = std::is_same<T, float>::value ? exp_exact(fabsf(g)) : __builtin_amdgcn_exp2f(fabsf(q));
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    const uint32_t n = (uint32_t)((int)__float_as_uint(q) >> 31), m = 0x80000001u;
    return __uint_as_float((n & m) | (__float_as_uint(r) & ~m));
}
// Whether d is a - 1: all bits or none
__device__ __forceinline__ uint32_t is_near(float d) {
    return (uint32_t)__builtin_amdgcn_sbfe((int)__float_as_uint(d), 0, 1);
}
// a h
__device__ __forceinline__ float keep(float d, uint32_t n, float h) {
    return fmaf(d, h, __uint_as_float(n & __float_as_uint(h)));
}
// 1 - a
__device__ __forceinline__ float rest(float d, uint32_t n) { return __uint_as_float(~n & 0x3f800000u) - d; }
// a h + (1 - a) x as h + (a - 1) (h - x) or x + a (h - x): exact at a = 0, and no product is larger than what it decays
template <bool COMP> __device__ __forceinline__ float step(float h, float d, uint32_t n, float x) {
    return COMP ? fmaf(d, h - x, __uint_as_float((n & __float_as_uint(h)) | (~n & __float_as_uint(x)))) : keep(d, n, h) + x;
}
}  // namespace decay
template <typename T, int N>
__device__ __forceinline__ void decays(float (&d)[N], bool sigmoid) {
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = decay::sigmoid<T>(d[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = decay::log<T>(d[i]);
    }
}

// What a run of rows does to the state; A < 0: it ends with B whatever came in
// (a sequence begins inside), so that nothing of another one is multiplied.
struct Run {
    float A, B;
    // Makes the compiler form A here.  Put off to where the walk ends, which it would do, it takes the kinds of all the
    // decays there, two scalar registers each: 113 spilled (15151 x 2048 55.6 -> 52.7 us with this and the sign of q).
    __device__ __forceinline__ void A_now() { asm volatile("" : "+v"(A)); }
};
// Zeros come out as +0.
__device__ __forceinline__ float enter(Run r, float h) { return (r.A < 0.f ? r.B : fmaf(r.A, h, r.B)) + 0.f; }
// What r does after all
__device__ __forceinline__ Run after(Run all, Run r) {
    return {r.A < 0.f || all.A < 0.f ? -1.f : r.A * all.A, enter(r, all.B)};
}

// ---------------------------------------------------------------- tiles in order
//
// The tiles of a strip of channels, in the order of their chain, hand the state
// on through words in the workspace, cleared before the launch.  A tile
// publishes its Run P as soon as its rows are joined.  A few tiles in a row are
// a group: its last tile publishes the Run G of them all, and, entering G from
// the state H after the group before, the state after the group.  The state
// that enters a tile is the H before its group with the P of the group's
// earlier tiles entered one by one; that H is the nearest one there is with the
// G since then entered.  So the same products and sums are formed in the same
// order whatever is found, and the bits do not depend on timing.
//
// A value and its being there are one word, so nothing else has to be ordered:
// a word of zeros is not there yet, and a zero is kept as -0.  What has been
// published is noted in flags too, so that one load of a wave looks at all that
// a tile may wait for; they only tell where to look, and come in any order.
//
// The tiles of a strip are numbered by a counter in the order in which its
// blocks start, so every tile before one that waits belongs to a block that runs
// already.  (One counter for all strips takes 4 ns a block: 64 of 311 us of the
// gradients of 32768 x 2048.)
typedef unsigned long long u64;
struct Chain {
    uint32_t *count;  // [strips], COUNT_STEP apart: blocks that have started
    uint32_t *flag;   // [strips][tiles] 1: P
    uint32_t *gflag;  // [strips][groups] 1: G, 2: H
    u64 *P, *G;       // [tiles][C], [groups][C]
    uint32_t *H;      // [groups][C]
    int tiles, group, groups;
};
// Tiles of a group.  Entered one by one from the nearest state, with some 24
// tiles of a strip under way, the words a tile reads hold up the rest (states of
// 32768 x 2048: 84 us, in groups of 4 64, of 8 62).  A short chain goes without:
// a step less to wait for (2 x 1024 x 1024 backwards 25 -> 19 us).
__host__ __device__ inline int group_of(int64_t tiles) { return tiles <= 16 ? 16 : 8; }
constexpr int COUNT_STEP = 64;     // counters in lines of their own
constexpr int PATIENCE = 1 << 22;  // looks (seconds) before a tile gives up, with NaN

template <typename T> __device__ __forceinline__ T look(const T *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T> __device__ __forceinline__ void show(T *p, T x) {
    __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t not_zero(float x) { return x == 0.f ? 0x80000000u : __float_as_uint(x); }
__device__ __forceinline__ u64 word(Run r) { return (u64)__float_as_uint(r.B) << 32 | not_zero(r.A); }
__device__ __forceinline__ Run run_of(u64 w) {  // of no word: NaN
    return w ? Run{__uint_as_float((uint32_t)w) + 0.f, __uint_as_float((uint32_t)(w >> 32))} : Run{-1.f, __builtin_nanf("")};
}

// Enters the n Runs at `at` (one every C words) into h, the first eight as they
// were asked for before; one that is not there yet is asked for again.
__device__ __forceinline__ float enter_words(const u64 *at, int64_t C, int n, u64 (&w)[8], float h, bool mine, int &patience) {
    for (int k = 0; k < n; k += 8) {
        if (k)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = k + i < n && mine ? look(at + (k + i) * C) : 1;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < n) {
                while (!w[i] && --patience > 0) w[i] = look(at + (k + i) * C);
                h = enter(run_of(w[i]), h);
            }
    }
    return h;
}
__device__ __forceinline__ void ask(const u64 *at, int64_t C, int n, u64 (&w)[8], bool mine) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < n && mine ? look(at + i * C) : 1;
}

// Publishes the Run of tile pos and returns the state that enters it, for the
// channel c of every lane (mine: it has one), by one wave.  Where that is not
// wanted, or nothing enters the tile whatever comes before (alone), only the
// last tile of a group waits.  `meanwhile` is done once P is out.
template <typename F>
__device__ __forceinline__ float hand_on(Run own, const Chain &ch, int64_t C, int strip, int pos, int c, bool mine, bool alone,
                                         bool wanted, F meanwhile) {
    const int lane = lane_id(), g = pos / ch.group, r = pos - g * ch.group;
    u64 *P = ch.P + (int64_t)(pos - r) * C + c, *G = ch.G + (int64_t)g * C + c;
    uint32_t *H = ch.H + (int64_t)g * C + c, *flag = ch.flag + (int64_t)strip * ch.tiles + pos - r,
             *gflag = ch.gflag + (int64_t)strip * ch.groups + g;
    const bool more = pos + 1 < ch.tiles, ends = more && r == ch.group - 1;
    if (more && !ends) {
        if (mine) show(P + r * C, word(own));
        if (lane == 0) show(flag + r, 1u);
    }
    meanwhile();
    if ((alone || !wanted) && !ends) return 0.f;
    int patience = PATIENCE, near = -1;
    bool have = false;
    u64 w[8], q[8];
    Run all{1.f, 0.f};
    do {
        // lanes 0 to 47: the groups before, nearest first (before the first one the state is there, and zero); from 48 on:
        // the group's earlier tiles
        const uint32_t f = lane < 48 ? (lane < g ? look(gflag - 1 - lane) : 2u) : lane - 48 < r ? look(flag + lane - 48) : 1u;
        const uint64_t some = __ballot(f >= 1), done = __ballot(f == 2) & ((1ull << 48) - 1);
        if (!have && some >> 48 == 0xffff) {
            have = true;
            if (ends) {
                for (int k = 0; k < r; k += 8) {
                    ask(P + k * C, C, r - k, q, mine);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (k + i < r) {
                            while (!q[i] && --patience > 0) q[i] = look(P + (k + i) * C);
                            all = after(all, run_of(q[i]));
                        }
                }
                all = after(all, own);
                const bool cut = __all(!mine || all.A < 0.f);  // nothing gets past the group
                if (mine) {
                    if (cut) show(H, not_zero(all.B));
                    else show(G, word(all));
                }
                if (lane == 0) show(gflag, cut ? 2u : 1u);
                if (cut && (alone || !wanted)) return 0.f;
            }
        }
        if (have && done) {
            const int k = __builtin_ctzll(done);
            if (!(~some & ((1ull << k) - 1))) near = k;
        }
        if (near < 0) __builtin_amdgcn_s_sleep(1);
    } while (near < 0 && --patience > 0);
    float h = 0.f;
    if (near < 0) {
        near = 0;
        patience = 1;
        h = __builtin_nanf("");
    } else {
        // all asked for at once
        uint32_t first = near < g && mine ? look(H - (near + 1) * C) : 1u;
        ask(G - near * C, C, near, w, mine);
        ask(P, C, r, q, mine);
        while (!first && --patience > 0) first = look(H - (near + 1) * C);
        h = near == g ? 0.f : first ? __uint_as_float(first) + 0.f : __builtin_nanf("");
        h = enter_words(G - near * C, C, near, w, h, mine, patience);
    }
    if (ends) {
        if (mine) show(H, not_zero(enter(all, h)));
        if (lane == 0) show(gflag, 2u);
    }
    return wanted && have ? enter_words(P, C, r, q, h, mine, patience) : h;
}
// The state that enters tile pos of a chain that has ended, for a channel.
__device__ __forceinline__ float handed_on(const Chain &ch, int64_t C, int pos, int c) {
    const int g = pos / ch.group, r = pos - g * ch.group;
    const u64 *P = ch.P + (int64_t)(pos - r) * C + c;
    float h = g > 0 ? __uint_as_float(ch.H[(int64_t)(g - 1) * C + c]) + 0.f : 0.f;
    for (int k = 0; k < r; k += 8) {
        u64 q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = k + i < r ? P[(k + i) * C] : 1;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < r) h = enter(run_of(q[i]), h);
    }
    return h;
}

// A block's tile and strip of channels, and the tile's place in its chain: the
// tiles from the first one on, or from the last one back.
struct Turn {
    int tile, strip, pos;
};
template <bool BACK>
__device__ __forceinline__ Turn next_turn(const LinRec &p, uint32_t *count, int strips) {
    __shared__ uint32_t id;
    Turn t;
    t.strip = (int)(blockIdx.x % (uint32_t)strips);
    t.pos = 0;
    if (p.tiles > 1) {
        if (threadIdx.x == 0) id = atomicAdd(count + t.strip * COUNT_STEP, 1u);
        __syncthreads();
        t.pos = (int)__builtin_amdgcn_readfirstlane(id);
    }
    t.tile = BACK ? p.tiles - 1 - t.pos : t.pos;
    return t;
}

// What the rows of a thread are: bit i for its i-th.
template <int TT>
struct Kinds {
    uint32_t in = 0, first = 0, last = 0;
    bool plain;  // all rows of the wave inside a sequence, none its first or last
    __device__ __forceinline__ Kinds(const uint8_t *code) {
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const uint32_t c = code[i];
            in |= (c & ROW_IN) << i;
            first |= (uint32_t)row_first(c) << i;
            last |= (uint32_t)row_last(c) << i;
        }
        plain = !__any(in != (1u << TT) - 1 || first || last);
    }
    __device__ __forceinline__ bool inside(int i) const { return plain || (in >> i & 1); }
    __device__ __forceinline__ bool is_first(int i) const { return !plain && (first >> i & 1); }
    __device__ __forceinline__ bool is_last(int i) const { return !plain && (last >> i & 1); }
    // nothing from before (or behind) them gets past these rows
    __device__ __forceinline__ bool cut() const { return in != (1u << TT) - 1 || first; }
    __device__ __forceinline__ bool cut_back() const { return in != (1u << TT) - 1 || last; }
};

// A thread's rows from the first to the last: h <- a h + c x
template <bool COMP, typename T, int E, int TT, typename F>
__device__ __forceinline__ void walk(Run (&run)[E], const Chans<T, E> (&xr)[TT], F decay, const Kinds<TT> &is, const int *seq,
                                     const float *h0, int C, int col) {
#pragma unroll
    for (int e = 0; e < E; ++e) run[e] = {1.f, 0.f};
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        float x[E], d[E];
        xr[i].to(x);
        decay(d, i);
        if (is.is_first(i)) {
            float h[E];
            load_state<E>(h, h0, seq[i], C, col);
#pragma unroll
            for (int e = 0; e < E; ++e) run[e].B = h[e];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t near = decay::is_near(d[e]);
            run[e].B = decay::step<COMP>(run[e].B, d[e], near, x[e]);
            run[e].A = decay::keep(d[e], near, run[e].A);
            run[e].A_now();
        }
        if (!is.inside(i))
#pragma unroll
            for (int e = 0; e < E; ++e) run[e].B = 0.f;
    }
    if (!is.plain && is.cut())
#pragma unroll
        for (int e = 0; e < E; ++e) run[e].A = -1.f;
}
// From the last to the first: m <- a (dy + m), the gradient of the state before the row
template <typename T, int E, int TT>
__device__ __forceinline__ void walk_back(Run (&run)[E], const Chans<T, E> (&dr)[TT], const float (&d)[TT][E],
                                          const Kinds<TT> &is, const int *seq, const float *dht, int C, int col) {
#pragma unroll
    for (int e = 0; e < E; ++e) run[e] = {1.f, 0.f};
#pragma unroll
    for (int i = TT - 1; i >= 0; --i) {
        float dy[E];
        dr[i].to(dy);
        if (is.is_last(i)) {
            float h[E];
            load_state<E>(h, dht, seq[i], C, col);
#pragma unroll
            for (int e = 0; e < E; ++e) run[e].B = h[e];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t near = decay::is_near(d[i][e]);
            run[e].B = decay::keep(d[i][e], near, dy[e] + run[e].B);
            run[e].A = decay::keep(d[i][e], near, run[e].A);
            run[e].A_now();
        }
        if (!is.inside(i))
#pragma unroll
            for (int e = 0; e < E; ++e) run[e].B = 0.f;
    }
    if (!is.plain && is.cut_back())
#pragma unroll
        for (int e = 0; e < E; ++e) run[e].A = -1.f;
}

// The block's runs of every channel, joined in order, a channel a lane: every
// wave its own runs, then the waves.
constexpr int LNW = LNT / 64;
template <int NY, bool BACK>
struct Joint {
    static constexpr int PER = NY / LNW;
    float *ra, *rb;  // [NY][W], the runs; rb becomes the state that enters each
    Run *part;       // [LNW][W], the waves' runs
    __device__ __forceinline__ Joint(float *ra, float *rb, Run *part) : ra(ra), rb(rb), part(part) {}
    __device__ __forceinline__ int row(int i) const { return (wave_id() * PER + (BACK ? PER - 1 - i : i)) * W + lane_id(); }
    __device__ __forceinline__ void own() const {
        Run all{1.f, 0.f};
        for (int i = 0; i < PER; ++i) all = after(all, {ra[row(i)], rb[row(i)]});
        part[wave_id() * W + lane_id()] = all;
    }
    // From the state that enters the tile
    __device__ __forceinline__ void enter_own(float h) const {
#pragma unroll
        for (int v = 0; v < LNW - 1; ++v) {
            const int u = BACK ? LNW - 1 - v : v;
            if (BACK ? u > wave_id() : u < wave_id()) h = enter(part[u * W + lane_id()], h);
        }
        for (int i = 0; i < PER; ++i) {
            const Run r{ra[row(i)], rb[row(i)]};
            rb[row(i)] = h;
            h = enter(r, h);
        }
        __builtin_amdgcn_wave_barrier();  // rb is read by other lanes of the wave that wrote it
    }
    __device__ __forceinline__ Run all() const {
        Run r{1.f, 0.f};
#pragma unroll
        for (int v = 0; v < LNW; ++v) r = after(r, part[(BACK ? LNW - 1 - v : v) * W + lane_id()]);
        return r;
    }
};

}  // namespace

// ROWS: y and the final states; without: only the chain, for the gradients.
// Three blocks to a compute unit with rows in bfloat16 (165 registers).
template <typename T, typename G, int E, int TT, bool COMP, bool ROWS>
__global__ void __launch_bounds__(LNT, ROWS ? 3 : 1) gdp_linrec_k(LinRec p, Chain ch, int strips) {
    __shared__ uint8_t code[LNT / (W / E) * TT];
    __shared__ int seq[LNT / (W / E) * TT];
    __shared__ float ra[LNT * E], rb[LNT * E], enters[W];
    __shared__ Run part[LNW * W];
    const Turn t = next_turn<false>(p, ch.count, strips);
    constexpr int NX = W / E, NY = LNT / NX;  // threads side by side, and one behind the other
    const Place<NX, NY, E, TT> at(p.C, t.tile, t.strip);
    const int k0 = at.ty * TT;  // the thread's rows in the tile
    const uint32_t n = at.tile0 < p.m.rows ? min(p.m.rows - at.tile0, (uint32_t)(NY * TT)) : 0;

    Chans<T, E> xr[TT];
    Chans<G, E> gr[TT];
    load_rows(xr, p.x, p.m, p.flat, at, n, p.C);
    load_rows(gr, p.g, p.m, p.flat, at, n, p.C);
    find_rows<LNT>(p.m, at.tile0, NY * TT, code, seq);
    __syncthreads();

    const Kinds<TT> is(code + k0);
    float d[ROWS ? TT : 1][E];
    Run run[E];
    const auto decay = [&](float (&s)[E], int i) {  // kept for the rows, or formed as they are walked
        gr[i].to(s);
        decays<T>(s, p.sigmoid);
        if constexpr (ROWS)
#pragma unroll
            for (int e = 0; e < E; ++e) d[i][e] = s[e];
    };
    walk<COMP>(run, xr, decay, is, seq + k0, at.live ? p.h0 : nullptr, p.C, at.col);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        ra[at.ty * W + at.tx * E + e] = run[e].A;
        rb[at.ty * W + at.tx * E + e] = run[e].B;
    }
    __syncthreads();
    const Joint<NY, false> join(ra, rb, part);
    join.own();
    __syncthreads();
    const int c = t.strip * W + lane_id();
    if (wave_id() == 0) {
        const bool alone = row_first(code[0]) || !(code[0] & ROW_IN);
        enters[lane_id()] = p.tiles > 1 ? hand_on(join.all(), ch, p.C, t.strip, t.pos, c, c < p.C, alone, ROWS, [] {}) : 0.f;
    }
    if constexpr (ROWS) {
        __syncthreads();
        join.enter_own(enters[lane_id()]);
        if (!at.live) return;
        const TileRows<T> y((T *)p.y + (int64_t)at.tile0 * p.C, p.C, n, p.C, k0, at.col, true);
        float h[E];
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = rb[at.ty * W + at.tx * E + e];
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            xr[i].forget();
            forget(d[i]);
        }
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (!is.inside(i)) continue;
            float x[E];
            xr[i].to(x);
            if (is.is_first(i)) load_state<E>(h, p.h0, seq[k0 + i], p.C, at.col);
#pragma unroll
            for (int e = 0; e < E; ++e) h[e] = decay::step<COMP>(h[e], d[i][e], decay::is_near(d[i][e]), x[e]);
            Chans<T, E> o;
            o.from(h);
            o.store(y.r, y.off + i * y.step);
            if (is.is_last(i) && p.ht) store_state<E>(p.ht, seq[k0 + i], p.C, at.col, h);
        }
        if (p.ht && at.ty == 0)
            for (int q = t.tile; q < p.m.nseq; q += p.tiles)
                if (seq_empty(p.m, q)) {
                    float z[E];
                    load_state<E>(z, p.h0, q, p.C, at.col);
                    store_state<E>(p.ht, q, p.C, at.col, z);
                }
    }
}

// The gradients, tiles from the last to the first; fwd is the chain that
// gdp_linrec_k without ROWS leaves, of the same tiles.  Four blocks to a compute
// unit with rows in bfloat16 (128 registers, two or three more spill) instead of
// three (136): 235 -> 226 us for 32768 x 2048.  float32 rows take 165.
template <typename T, typename G, int E, int TT, bool COMP>
__global__ void __launch_bounds__(LNT, E == 8 ? 4 : 1) gdp_linrec_bwd_k(LinRec p, Chain fwd, Chain ch, int strips) {
    __shared__ uint8_t code[LNT / (W / E) * TT];
    __shared__ int seq[LNT / (W / E) * TT];
    __shared__ float ra[2][LNT * E], rb[2][LNT * E], enters[W];
    __shared__ Run part[2][LNW * W];
    const Turn t = next_turn<true>(p, ch.count, strips);
    constexpr int NX = W / E, NY = LNT / NX;
    const Place<NX, NY, E, TT> at(p.C, t.tile, t.strip);
    const int k0 = at.ty * TT;
    const uint32_t n = at.tile0 < p.m.rows ? min(p.m.rows - at.tile0, (uint32_t)(NY * TT)) : 0;

    Chans<T, E> xr[TT], dr[TT];
    Chans<G, E> gr[TT];
    load_rows(xr, p.x, p.m, p.flat, at, n, p.C);
    load_rows(gr, p.g, p.m, p.flat, at, n, p.C);
    load_rows(dr, p.dy, p.m, p.flat, at, n, p.C);
    find_rows<LNT>(p.m, at.tile0, NY * TT, code, seq);
    __syncthreads();

    const Kinds<TT> is(code + k0);
    float d[TT][E];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        gr[i].to(d[i]);
        decays<T>(d[i], p.sigmoid);
    }
    Run run[E];
    const auto kept = [&](float (&s)[E], int i) {
#pragma unroll
        for (int e = 0; e < E; ++e) s[e] = d[i][e];
    };
#pragma unroll
    for (int z = 0; z < 2; ++z) {
#pragma unroll
        for (int i = 0; i < TT; ++i) forget(d[i]);
        if (z) walk_back(run, dr, d, is, seq + k0, at.live ? p.dht : nullptr, p.C, at.col);
        else walk<COMP>(run, xr, kept, is, seq + k0, at.live ? p.h0 : nullptr, p.C, at.col);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            ra[z][at.ty * W + at.tx * E + e] = run[e].A;
            rb[z][at.ty * W + at.tx * E + e] = run[e].B;
        }
    }
    __syncthreads();
    const Joint<NY, false> to(ra[0], rb[0], part[0]);
    const Joint<NY, true> back(ra[1], rb[1], part[1]);
    to.own();
    back.own();
    __syncthreads();
    const int c = t.strip * W + lane_id(), end = NY * TT - 1;
    const bool mine = c < p.C;
    const auto forwards = [&] { to.enter_own(p.tiles > 1 && mine ? handed_on(fwd, p.C, t.tile, c) : 0.f); };
    if (wave_id() == 0 && p.tiles > 1) {
        const bool alone = row_last(code[end]) || !(code[end] & ROW_IN);
        enters[lane_id()] = hand_on(back.all(), ch, p.C, t.strip, t.pos, c, mine, alone, true, forwards);
    } else {
        forwards();
        if (wave_id() == 0) enters[lane_id()] = 0.f;
    }
    __syncthreads();
    back.enter_own(enters[lane_id()]);
    if (!at.live) return;
    const TileRows<T> rx((T *)p.dx + (int64_t)at.tile0 * p.C, p.C, n, p.C, k0, at.col, true);
    const TileRows<G> rg((G *)p.dg + (int64_t)at.tile0 * p.C, p.C, n, p.C, k0, at.col, true);
    float h[E], m[E], hp[TT][E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        h[e] = rb[0][at.ty * W + at.tx * E + e];
        m[e] = rb[1][at.ty * W + at.tx * E + e];
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        xr[i].forget();
        dr[i].forget();
        forget(d[i]);
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {  // hp: what da is l times
        float x[E];
        xr[i].to(x);
        if (is.is_first(i)) load_state<E>(h, p.h0, seq[k0 + i], p.C, at.col);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            hp[i][e] = COMP ? h[e] - x[e] : h[e];
            h[e] = decay::step<COMP>(h[e], d[i][e], decay::is_near(d[i][e]), x[e]);
        }
        forget(h);  // row by row (the complement's gradients of 32768 x 2048: 230 us without, 227)
    }
#pragma unroll
    for (int i = TT - 1; i >= 0; --i) {
        float dy[E], dx[E], dg[E];
        dr[i].to(dy);
        if (is.is_last(i)) load_state<E>(m, p.dht, seq[k0 + i], p.C, at.col);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t near = decay::is_near(d[i][e]);
            const float l = dy[e] + m[e], al = decay::keep(d[i][e], near, l), cl = decay::rest(d[i][e], near);
            dx[e] = COMP ? cl * l : l;
            dg[e] = hp[i][e] * (p.sigmoid ? cl * al : al);
            m[e] = al;
        }
        if (!is.inside(i))
#pragma unroll
            for (int e = 0; e < E; ++e) dx[e] = dg[e] = 0.f;
        Chans<T, E> ox;
        Chans<G, E> og;
        ox.from(dx);
        og.from(dg);
        ox.store(rx.r, rx.off + i * rx.step);
        og.store(rg.r, rg.off + i * rg.step);
        if (is.is_first(i) && p.dh0) store_state<E>(p.dh0, seq[k0 + i], p.C, at.col, m);
    }
    if (p.dh0 && at.ty == 0)
        for (int q = t.tile; q < p.m.nseq; q += p.tiles)
            if (seq_empty(p.m, q)) {
                float z[E];
                load_state<E>(z, p.dht, q, p.C, at.col);
                store_state<E>(p.dh0, q, p.C, at.col, z);
            }
}

// The workspace's words before a launch: none there yet.
__global__ void __launch_bounds__(LNT) gdp_linrec_clear_k(uint4 *p, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * LNT + threadIdx.x;
    if (i < n) p[i] = uint4{};
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
        decays<T>(d, a.decay == GDP_DECAY_SIGMOID);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = a.complement ? decay::step<true>(h[e], d[e], decay::is_near(d[e]), x[e])
                                                       : decay::step<false>(h[e], d[e], decay::is_near(d[e]), x[e]);
        xr.from(h);
        xr.store(y + t * a.C);
    }
    store_state<E>(a.state + slot * a.C, 0, a.C, col, h);
}

namespace {

// Channels and rows that a thread holds: 16 bytes of a row, and about as many
// registers of rows as let three or four blocks share a compute unit
// (bfloat16, inputs in the caches, 4 / 8 rows forwards: 15151 x 2048 56 / 53 us,
// 32768 x 2048 127 / 120.  Backwards 4 / 8: 226 / 254, 2 x 1024 x 1024 20 / 25).
int elems_of(const LinRec &p) { return !p.vec ? 1 : p.f32 ? 4 : 8; }
constexpr int rows_of(int E, bool back) { return E == 1 ? (back ? 8 : 16) : E == 4 || !back ? 8 : 4; }
int strips_of(const LinRec &p) { return (p.C + W - 1) / W; }
int64_t tile_rows(const LinRec &p, bool back) { return (int64_t)(LNT / (W / elems_of(p))) * rows_of(elems_of(p), back); }
int64_t tiles_of(const LinRec &p, bool back) { return (p.m.rows + tile_rows(p, back) - 1) / tile_rows(p, back); }

// The words of a chain, in whole units of 256 bytes: counters and flags, P, G, H.
int64_t units(int64_t bytes) { return (bytes + 255) / 256 * 256; }
int64_t chain_bytes(int64_t tiles, int64_t strips, int64_t C, char *q = nullptr, Chain *ch = nullptr) {
    const int64_t group = group_of(tiles), groups = (tiles + group - 1) / group, marks = units(4 * strips * (COUNT_STEP + tiles + groups));
    if (ch) {
        ch->count = (uint32_t *)q;
        ch->flag = ch->count + strips * COUNT_STEP;
        ch->gflag = ch->flag + strips * tiles;
        ch->P = (u64 *)(q + marks);
        ch->G = ch->P + tiles * C;
        ch->H = (uint32_t *)(ch->G + groups * C);
        ch->tiles = (int)tiles;
        ch->group = (int)group;
        ch->groups = (int)groups;
    }
    return marks + units((tiles * 8 + groups * 12) * C);
}

template <typename T, typename G, int E, bool COMP>
hipError_t run_linrec(const LinRec &p, bool back, hipStream_t stream) {
    const int strips = strips_of(p);
    const int64_t tiles = p.tiles, words = chain_bytes(tiles, strips, p.C);
    const dim3 grid((unsigned)(tiles * strips));
    constexpr int TF = rows_of(E, false), TB = rows_of(E, true);
    Chain one{}, two{};
    if (tiles > 1) {
        chain_bytes(tiles, strips, p.C, (char *)p.space, &one);
        if (back) chain_bytes(tiles, strips, p.C, (char *)p.space + words, &two);
        const int64_t n = (back ? 2 : 1) * words / 16;
        hipLaunchKernelGGL(gdp_linrec_clear_k, dim3((unsigned)((n + LNT - 1) / LNT)), dim3(LNT), 0, stream, (uint4 *)p.space, n);
    }
    if (back) {
        if (tiles > 1) hipLaunchKernelGGL((gdp_linrec_k<T, G, E, TB, COMP, false>), grid, dim3(LNT), 0, stream, p, one, strips);
        hipLaunchKernelGGL((gdp_linrec_bwd_k<T, G, E, TB, COMP>), grid, dim3(LNT), 0, stream, p, one, two, strips);
    } else {
        hipLaunchKernelGGL((gdp_linrec_k<T, G, E, TF, COMP, true>), grid, dim3(LNT), 0, stream, p, one, strips);
    }
    return hipGetLastError();
}
template <typename T, typename G, int E>
hipError_t run_kind(const LinRec &p, bool back, hipStream_t stream) {
    return p.complement ? run_linrec<T, G, E, true>(p, back, stream) : run_linrec<T, G, E, false>(p, back, stream);
}
hipError_t run_types(LinRec p, bool back, hipStream_t stream) {
    const int64_t rows = tile_rows(p, back);
    p.flat = even_rows(p.x, p.m, rows) && even_rows(p.g, p.m, rows) && (!back || even_rows(p.dy, p.m, rows));
    const int64_t tiles = tiles_of(p, back);
    p.tiles = tiles > 1 ? (int)tiles : 1;
    if (p.f32) return p.vec ? run_kind<float, float, 4>(p, back, stream) : run_kind<float, float, 1>(p, back, stream);
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

bool linrec_fits(const LinRec &p, bool backward) {
    const int64_t tiles = tiles_of(p, backward), strips = strips_of(p);
    return tiles * strips * LNT <= 0xffffffffll && 2 * chain_bytes(tiles, strips, p.C) / 16 <= 0xffffff00ll;
}
int64_t linrec_space(const LinRec &p, bool backward) {
    const int64_t tiles = tiles_of(p, backward);
    return tiles > 1 ? (backward ? 2 : 1) * chain_bytes(tiles, strips_of(p), p.C) : 0;
}
hipError_t launch_linrec(const LinRec &p, bool backward, hipStream_t stream) { return run_types(p, backward, stream); }

hipError_t launch_linrec_decode(const gdp_linrec_decode_args &a, bool vec, hipStream_t stream) {
    if (a.dtype == GDP_F32) return vec ? run_decode<float, float, 4>(a, stream) : run_decode<float, float, 1>(a, stream);
    if (a.g_dtype == GDP_F32) return vec ? run_decode<bf16, float, 8>(a, stream) : run_decode<bf16, float, 1>(a, stream);
    return vec ? run_decode<bf16, bf16, 8>(a, stream) : run_decode<bf16, bf16, 1>(a, stream);
}

}  // namespace gdp

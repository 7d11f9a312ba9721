// linattn.h -- launcher interface of linattn.hip (host side).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gdp.h"

namespace gdp {

// A tensor [B, T, heads, D]: element (b, t, h, d) at p + b*bs + t*ts + h*D + d;
// value head hv reads head hv / div.
struct LinRows {
    const void *p = nullptr;
    int64_t bs = 0, ts = 0;
    int div = 1;
};

// Rows of a span: a segment's states are kept at every border between two of
// its spans (the one before its t-th token in slot t / LIN_SPAN, which no two
// borders share: they lie a span apart).
constexpr int LIN_SPAN = 512;

// One walk (linattn.hip): y_i = sum D(i,j) (a_i.b_j) c_j over every sequence,
// cut into segments of seg_tok rows.
struct LinWalk {
    LinRows a, b, c, x;
    int da, dc;        // columns of a and b, of c (and x, y)
    int HV;
    float sb, sy;      // factors of the products a_i.b_j (and c_j b_j^T), and of y
    int64_t B, T, nseq, seg_tok, items;
    const int32_t *cu;
    const float *g;    // log decay of (b, t, hv) at g + b*g_bs + t*g_ts + hv, or NULL
    int64_t g_bs, g_ts;
    bool trans;        // states that are read hold element (c, a) at [a][c]
    bool y32;          // y is float
    void *y;           // [B, T, HV, dc]
    float *rho;        // [slices, HV, B*T]
    const float *s0;   // [nseq, HV, dc, da] or NULL: state before the first row of the walk
    const float *seg_in;  // [slots, HV, dc, da] or NULL: state entering each segment (then s0 is not read)
    float *s_out;      // [nseq, HV, dc, da] or NULL: state after the walk
    float *seg_out;    // segment pass: [slots, HV, dc, da] and [slots, HV]
    float *seg_tot;
    float *rho_in_chunk;  // as rho, or NULL: then rho holds every pair, else those of two chunks (the walk
                          // forwards writes the others here, weighed by their distance)
    float *mid;        // [B T / LIN_SPAN + 1, HV, dc, da] or NULL: states at the borders of spans
};

// The walks of a launch: one forwards, with a second one of its shape backwards
// (segment passes), or the gradients' three (dq's forwards, the others back).
struct LinWalks {
    LinWalk w[3];
    int n;
};

struct LinScan {
    const int32_t *cu;
    int64_t T, nseq, seg_tok, elems, items;
    int HV, n;         // states that are scanned
    struct {
        bool rev;
        const float *s0;
        float *seg;
        const float *tot;
    } s[2];
};

struct LinDg {
    const int32_t *cu;
    int64_t B, T, nseq, seg_tok, elems, items;
    int HV, nq, nk;    // slices of rho_q and rho_k
    int spans, chunk;  // of a segment, and rows of a chunk (a decay per head)
    const float *g;
    int64_t g_bs, g_ts;
    const float *rho_q, *rho_k;
    const float *rho_in_chunk;        // a decay per head
    const float *s_in, *r_in;         // states entering each segment, forwards and backwards
    const float *s_mid, *r_mid;       // and its spans after the first (a decay per head)
    const float *h0, *dh0;            // [nseq, HV, V, K] or NULL
    bool end_zero;                    // no gradient enters behind the last row
    float *dg;         // [B, T, HV], or NULL for a decay per head
    double *part;      // [items, HV]: sums over each segment (a decay per head)
};

// y[i] [B*T, H, D] = sums over r neighbouring heads of x[i] [B*T, H*r, D]
// (units: 4 elements of y); with cu only the tokens of its requests
struct LinGroup {
    const float *x[2];
    void *y[2];
    int64_t units, nseq;
    int H, r, upr;     // upr: units of a head
    const int32_t *cu;
};

// Zeros in the rows outside every request: y[i] [T, words[i]] of 4 bytes (or NULL).
struct LinOutside {
    void *y[4];
    int64_t words[4];
    int64_t T, nseq;
    const int32_t *cu;
};
hipError_t launch_lin_outside(const LinOutside &p, hipStream_t stream);

// the rows y; exact: states to 24 bits
hipError_t launch_lin_rows(const LinWalks &w, gdp_dtype dtype, bool exact, hipStream_t stream);
// each segment's own state; dg: it is to serve dg too
hipError_t launch_lin_segments(const LinWalks &w, gdp_dtype dtype, bool exact, bool dg, hipStream_t stream);
// w[0] dq, w[1] dk, w[2] dv; dot: rho of dq and dk too
int lin_grads_slice(int K, int V);
hipError_t launch_lin_grads(const LinWalks &w, gdp_dtype dtype, bool dot, hipStream_t stream);
hipError_t launch_lin_scan(const LinScan &p, hipStream_t stream);
hipError_t launch_lin_dg(const LinDg &p, float *dg_head, hipStream_t stream);
hipError_t launch_lin_group(const LinGroup &p, gdp_dtype dtype, hipStream_t stream);
hipError_t launch_lin_decode(const gdp_linattn_decode_args &a, hipStream_t stream);

}  // namespace gdp

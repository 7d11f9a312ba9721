// mixops.h -- launcher interface of linrec.hip, shortconv.hip and rotary.hip
// (host side, and the parameters their kernels take).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gdp.h"

namespace gdp {

// The sequences of rows [B*T]: B of T rows each, or with cu (B == 1, T = rows)
// the nseq packed requests.
struct RowMap {
    const int32_t *cu;
    uint32_t T, rows;
    int nseq;
};

// [B, T, C]: element (b, t, c) at p + b*bs + t*ts + c
struct Strided {
    const void *p;
    int64_t bs, ts;
};

// Whether the rows [B*T] of a tensor lie at even distances, those of a tile of
// `rows` within 2^30 bytes of 4-byte elements.
inline bool even_rows(const Strided &s, const RowMap &m, int64_t rows) {
    return (m.T == m.rows || s.bs == (int64_t)m.T * s.ts) && s.ts <= (1 << 28) / rows;
}

struct LinRec {
    RowMap m;
    Strided x, g, dy;
    int C;
    bool vec;  // every row of every tensor starts on 16 bytes, C in whole units
    bool f32, g32, sigmoid, complement;  // f32: x, y, dy, dx
    int tiles;  // set at launch, as is flat: the rows of x, g, dy lie at even distances
    bool flat;
    const float *h0, *dht;
    void *y, *dx, *dg;
    float *ht, *dh0;
    void *space;
};
int64_t linrec_space(const LinRec &p, bool backward);
bool linrec_fits(const LinRec &p, bool backward);
hipError_t launch_linrec(const LinRec &p, bool backward, hipStream_t stream);
hipError_t launch_linrec_decode(const gdp_linrec_decode_args &a, bool vec, hipStream_t stream);

struct ShortConv {
    RowMap m;
    Strided x, dy;
    int C, W, act;
    bool vec, flat;  // flat: the rows of x and dy lie at even distances (set at launch)
    const float *w, *b;
    const void *h0, *dht;  // [nseq, W - 1, C]
    void *y, *ht, *dx, *dh0;
    float *dw, *db, *part;
};
int64_t conv_space(const ShortConv &p, gdp_dtype dtype);
bool conv_fits(const ShortConv &p, gdp_dtype dtype, bool backward);
hipError_t launch_conv(const ShortConv &p, gdp_dtype dtype, hipStream_t stream);
hipError_t launch_conv_bwd(const ShortConv &p, gdp_dtype dtype, hipStream_t stream);
hipError_t launch_conv_decode(const gdp_conv_decode_args &a, bool vec, hipStream_t stream);

struct Rotary {
    RowMap m;
    Strided in[2], out[2];
    int H[2], D, R;
    bool interleaved, inverse, vec;
    float scale;
    const int32_t *positions, *offsets;
    int64_t pos_bs, pos_ts;
    const double *freq;
};
bool rotary_fits(const Rotary &p, gdp_dtype dtype);
hipError_t launch_rotary(const Rotary &p, gdp_dtype dtype, hipStream_t stream);

}  // namespace gdp

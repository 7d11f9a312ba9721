// groupnorm.h -- launcher interface of groupnorm.hip (host side).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gdp.h"

namespace gdp {

struct GroupNorm {
    const void *x, *z, *dy;
    int64_t x_ns, x_ts, z_ns, z_ts, dy_ns, dy_ts;
    int64_t rows, split;  // rows = n * T; split: row sets side by side
    uint32_t T;
    int groups, D, act;
    int join;             // row sets of a block whose partial sums it joins (set at launch)
    bool centered, vec, bwd;  // vec: every row of every tensor starts on 16 bytes
    float eps;
    const float *w, *b;
    void *y, *dx, *dz;
    float *part, *dw, *db;
};

int64_t group_norm_split(int64_t rows, int groups, int D, bool bwd);
hipError_t launch_group_norm(GroupNorm p, gdp_dtype dtype, hipStream_t stream);

}  // namespace gdp

// api_mixops.cpp -- the C ABI of the gated linear recurrence, the short causal
// convolution and rotary positions (include/gdp.h): argument validation and
// launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <cmath>

#include "api_common.h"
#include "mixops.h"

using namespace gdp::api;

namespace {

constexpr int64_t kMaxC = 1 << 20;

bool known(gdp_dtype d) { return d == GDP_F32 || d == GDP_BF16; }

// B rows of T tokens, or packed requests.
gdp_status check_map(const char *name, int64_t B, int64_t T, const int32_t *cu, int64_t num_seqs, gdp::RowMap *m) {
    if (B < 0 || T < 0) return fail(GDP_ERR_INVALID, "%s: B and T must be >= 0", name);
    if (cu && B != 1) return fail(GDP_ERR_INVALID, "%s: cu_seqlens requires B == 1", name);
    if (cu && num_seqs < 0) return fail(GDP_ERR_INVALID, "%s: num_seqs < 0", name);
    if ((uintptr_t)cu & 3) return fail(GDP_ERR_INVALID, "%s: cu_seqlens is not 4-byte aligned", name);
    const int64_t nseq = cu ? num_seqs : B;
    // row numbers of a tile past the last row stay within 32 bits
    if (B > 0x7fffffff || T > 0x7fffffff || B * T > 0x7fffffff || nseq > (1 << 30))
        return fail(GDP_ERR_UNSUPPORTED, "%s: problem too large for one launch", name);
    *m = gdp::RowMap{cu, (uint32_t)T, (uint32_t)(B * T), (int)nseq};
    return ok();
}

// A strided [B, T, C] input of whole elements; *vec is cleared where its rows do not start on units of so many elements.
// The stride of a dimension of one element does not matter.
gdp_status check_input(const char *name, const char *what, const void *p, int64_t bs, int64_t ts, int64_t B, int64_t T,
                       gdp_dtype dtype, bool *vec, gdp::Strided *out, int64_t unit) {
    if (!p) return fail(GDP_ERR_INVALID, "%s: %s is NULL", name, what);
    if ((B > 1 && bs < 0) || (T > 1 && ts < 0)) return fail(GDP_ERR_INVALID, "%s: strides of %s must be >= 0", name, what);
    if ((uintptr_t)p % dsize(dtype)) return fail(GDP_ERR_INVALID, "%s: %s is not aligned to its type", name, what);
    if ((uintptr_t)p % (unit * dsize(dtype)) || (B > 1 && bs % unit) || (T > 1 && ts % unit)) *vec = false;
    // rows of one token lie a batch stride apart
    *out = gdp::Strided{p, B > 1 ? bs : 0, T > 1 ? ts : B > 1 ? bs : 0};
    return ok();
}
// A contiguous array of states, or NULL.
gdp_status check_states(const char *name, const char *what, const void *p, gdp_dtype dtype, bool *vec, int64_t unit) {
    if ((uintptr_t)p % dsize(dtype)) return fail(GDP_ERR_INVALID, "%s: %s is not aligned to its type", name, what);
    if ((uintptr_t)p % (unit * dsize(dtype))) *vec = false;
    return ok();
}
gdp_status check_output(const char *name, const char *what, const void *p, gdp_dtype dtype, bool *vec, int64_t unit) {
    if (!p) return fail(GDP_ERR_INVALID, "%s: %s is NULL", name, what);
    return check_states(name, what, p, dtype, vec, unit);
}
// An output of contiguous [B, T, C] on top of an input: only where that one's elements are the output's.
gdp_status check_on_top(const char *name, const char *what, const void *y, gdp_dtype dtype, const void *x, gdp_dtype x_dtype,
                        int64_t bs, int64_t ts, int64_t B, int64_t T, int64_t C) {
    if (y == x && (dtype != x_dtype || (B > 1 && bs != T * C) || (T > 1 && ts != C)))
        return fail(GDP_ERR_INVALID, "%s: y is %s, of other strides or another type", name, what);
    return ok();
}
// Whether two of the rows of `width` elements at b*bs + t*ts share one.
bool rows_overlap(int64_t B, int64_t T, int64_t bs, int64_t ts, int64_t width) {
    if (B > T) {
        const int64_t n = B, s = bs;
        B = T, bs = ts, T = n, ts = s;
    }
    if ((B > 1 && bs < width) || (T > 1 && ts < width)) return true;
    const auto reach = [&](int64_t n, int64_t s) { return (__int128)(n - 1) * s + width; };
    if (B <= 1 || bs >= reach(T, ts) || ts >= reach(B, bs)) return false;
    for (int64_t b = 1; b < B; ++b) {  // the rows next to row (b, 0); B^2 <= B*T < 2^31
        const __int128 at = (__int128)b * bs, t = at / ts, r = at % ts;
        if (t >= T) break;
        if (r < width || (t + 1 < T && ts - r < width)) return true;
    }
    return false;
}
// Elements of 16 bytes
int64_t unit_of(gdp_dtype d) { return 16 / (int64_t)dsize(d); }

gdp_status check_decode(const char *name, int64_t n, int64_t S, int32_t C, int64_t pool, const int32_t *slots) {
    if (n < 0 || S < 0) return fail(GDP_ERR_INVALID, "%s: n and S must be >= 0", name);
    if (C < 1) return fail(GDP_ERR_INVALID, "%s: C must be >= 1", name);
    if (C > kMaxC || S > 4096 || n > 0xffffff00ll / C) return fail(GDP_ERR_UNSUPPORTED, "%s: step too large (n, S or C)", name);
    if (pool < 0 || (!slots && pool < n)) return fail(GDP_ERR_INVALID, "%s: state pool too small", name);
    if ((uintptr_t)slots & 3) return fail(GDP_ERR_INVALID, "%s: slots is not 4-byte aligned", name);
    return ok();
}

gdp_status check_linrec(const char *name, const gdp_linrec_args *a, gdp::LinRec *p) {
    if (!a) return fail(GDP_ERR_INVALID, "%s: args is NULL", name);
    if (!known(a->dtype) || !(a->g_dtype == a->dtype || a->g_dtype == GDP_F32))
        return fail(GDP_ERR_INVALID, "%s: dtypes %d of x, %d of g", name, (int)a->dtype, (int)a->g_dtype);
    if (a->decay != GDP_DECAY_LOG && a->decay != GDP_DECAY_SIGMOID)
        return fail(GDP_ERR_INVALID, "%s: unknown decay %d", name, (int)a->decay);
    if (a->C < 1) return fail(GDP_ERR_INVALID, "%s: C must be >= 1", name);
    if (a->C > kMaxC) return fail(GDP_ERR_UNSUPPORTED, "%s: C=%d over 2^20", name, a->C);
    *p = gdp::LinRec{};
    const gdp_status st = check_map(name, a->B, a->T, a->cu_seqlens, a->num_seqs, &p->m);
    if (st != GDP_OK) return st;
    p->C = a->C;
    p->f32 = a->dtype == GDP_F32;
    p->g32 = a->g_dtype == GDP_F32;
    p->sigmoid = a->decay == GDP_DECAY_SIGMOID;
    p->complement = a->complement != 0;
    p->vec = a->C % unit_of(a->dtype) == 0;
    return ok();
}
// What the tensors' alignment leaves open: the larger workspace of both.
int64_t largest_space(gdp::LinRec p, bool backward) {
    const int64_t n = gdp::linrec_space(p, backward);
    p.vec = false;
    const int64_t m = gdp::linrec_space(p, backward);
    return n > m ? n : m;
}

gdp_status check_conv(const char *name, const gdp_conv_args *a, gdp::ShortConv *p) {
    if (!a) return fail(GDP_ERR_INVALID, "%s: args is NULL", name);
    if (!known(a->dtype)) return fail(GDP_ERR_INVALID, "%s: unknown dtype %d", name, (int)a->dtype);
    if (a->activation != GDP_ACT_NONE && a->activation != GDP_ACT_SILU && a->activation != GDP_ACT_SIGMOID)
        return fail(GDP_ERR_INVALID, "%s: unknown activation %d", name, (int)a->activation);
    if (a->C < 1 || a->W < 1) return fail(GDP_ERR_INVALID, "%s: C and W must be >= 1", name);
    if (a->W < 2 || a->W > 4) return fail(GDP_ERR_UNSUPPORTED, "%s: W=%d not built (2, 3, 4)", name, a->W);
    if (a->C > kMaxC) return fail(GDP_ERR_UNSUPPORTED, "%s: C=%d over 2^20", name, a->C);
    *p = gdp::ShortConv{};
    const gdp_status st = check_map(name, a->B, a->T, a->cu_seqlens, a->num_seqs, &p->m);
    if (st != GDP_OK) return st;
    p->C = a->C;
    p->W = a->W;
    p->act = a->activation;
    p->vec = a->C % unit_of(a->dtype) == 0;
    return ok();
}
int64_t largest_space(gdp::ShortConv p, gdp_dtype dtype) {
    const int64_t n = gdp::conv_space(p, dtype);
    p.vec = false;
    const int64_t m = gdp::conv_space(p, dtype);
    return n > m ? n : m;
}
gdp_status check_taps(const char *name, const float *w, const float *b) {
    if (!w) return fail(GDP_ERR_INVALID, "%s: w is NULL", name);
    if (((uintptr_t)w | (uintptr_t)b) & 3) return fail(GDP_ERR_INVALID, "%s: w or b is not 4-byte aligned", name);
    return ok();
}

#define TRY(call)                          \
    do {                                   \
        const gdp_status st_ = (call);     \
        if (st_ != GDP_OK) return st_;     \
    } while (0)

gdp_status too_large(const char *name) { return fail(GDP_ERR_UNSUPPORTED, "%s: problem too large for one launch", name); }

}  // namespace

extern "C" {

int64_t gdp_linrec_workspace_bytes(const gdp_linrec_args *a, int32_t backward) {
    gdp::LinRec p;
    if (check_linrec("gdp_linrec_workspace_bytes", a, &p) != GDP_OK) return -1;
    return largest_space(p, backward != 0);
}

gdp_status gdp_linrec_fwd(const gdp_linrec_args *a, void *workspace, int64_t workspace_bytes, void *stream) {
    const char *name = "gdp_linrec_fwd";
    gdp::LinRec p;
    TRY(check_linrec(name, a, &p));
    const int64_t unit = unit_of(a->dtype), gunit = unit_of(a->g_dtype);
    if (p.m.rows > 0) {
        TRY(check_input(name, "x", a->x, a->x_b_stride, a->x_t_stride, a->B, a->T, a->dtype, &p.vec, &p.x, unit));
        TRY(check_input(name, "g", a->g, a->g_b_stride, a->g_t_stride, a->B, a->T, a->g_dtype, &p.vec, &p.g, gunit));
        TRY(check_output(name, "y", a->y, a->dtype, &p.vec, unit));
        TRY(check_on_top(name, "x", a->y, a->dtype, a->x, a->dtype, a->x_b_stride, a->x_t_stride, a->B, a->T, a->C));
        TRY(check_on_top(name, "g", a->y, a->dtype, a->g, a->g_dtype, a->g_b_stride, a->g_t_stride, a->B, a->T, a->C));
    }
    TRY(check_states(name, "h0", a->h0, GDP_F32, &p.vec, 1));
    TRY(check_states(name, "ht", a->ht, GDP_F32, &p.vec, 1));
    // a first row reads its h0 again where the last row of its sequence may have left ht already
    if (a->ht && a->ht == a->h0) return fail(GDP_ERR_INVALID, "%s: ht may not be h0", name);
    p.h0 = a->h0;
    p.y = a->y;
    p.ht = a->ht;
    if (!gdp::linrec_fits(p, false)) return too_large(name);
    TRY(check_space(name, workspace, workspace_bytes, largest_space(p, false)));
    p.space = workspace;
    if (p.m.nseq == 0 || (p.m.rows == 0 && !p.ht)) return ok();
    return hip_status(gdp::launch_linrec(p, false, (hipStream_t)stream), name);
}

gdp_status gdp_linrec_bwd(const gdp_linrec_args *a, const gdp_linrec_grads *d, void *workspace, int64_t workspace_bytes,
                          void *stream) {
    const char *name = "gdp_linrec_bwd";
    gdp::LinRec p;
    TRY(check_linrec(name, a, &p));
    const int64_t unit = unit_of(a->dtype), gunit = unit_of(a->g_dtype);
    if (!d) return fail(GDP_ERR_INVALID, "%s: grads is NULL", name);
    if (p.m.rows > 0) {
        TRY(check_input(name, "x", a->x, a->x_b_stride, a->x_t_stride, a->B, a->T, a->dtype, &p.vec, &p.x, unit));
        TRY(check_input(name, "g", a->g, a->g_b_stride, a->g_t_stride, a->B, a->T, a->g_dtype, &p.vec, &p.g, gunit));
        TRY(check_input(name, "dy", d->dy, d->dy_b_stride, d->dy_t_stride, a->B, a->T, a->dtype, &p.vec, &p.dy, unit));
        TRY(check_output(name, "dx", d->dx, a->dtype, &p.vec, unit));
        TRY(check_output(name, "dg", d->dg, a->g_dtype, &p.vec, gunit));
    }
    TRY(check_states(name, "h0", a->h0, GDP_F32, &p.vec, 1));
    TRY(check_states(name, "dht", d->dht, GDP_F32, &p.vec, 1));
    TRY(check_states(name, "dh0", d->dh0, GDP_F32, &p.vec, 1));
    if (d->dh0 && (d->dh0 == d->dht || d->dh0 == a->h0))
        return fail(GDP_ERR_INVALID, "%s: dh0 may not be dht or h0", name);
    p.h0 = a->h0;
    p.dht = d->dht;
    p.dx = d->dx;
    p.dg = d->dg;
    p.dh0 = d->dh0;
    if (!gdp::linrec_fits(p, true)) return too_large(name);
    TRY(check_space(name, workspace, workspace_bytes, largest_space(p, true)));
    p.space = workspace;
    if (p.m.rows == 0 && !p.dh0) return ok();
    return hip_status(gdp::launch_linrec(p, true, (hipStream_t)stream), name);
}

gdp_status gdp_linrec_decode(const gdp_linrec_decode_args *a, void *stream) {
    const char *name = "gdp_linrec_decode";
    if (!a) return fail(GDP_ERR_INVALID, "%s: args is NULL", name);
    if (!known(a->dtype) || !(a->g_dtype == a->dtype || a->g_dtype == GDP_F32))
        return fail(GDP_ERR_INVALID, "%s: dtypes %d of x, %d of g", name, (int)a->dtype, (int)a->g_dtype);
    if (a->decay != GDP_DECAY_LOG && a->decay != GDP_DECAY_SIGMOID)
        return fail(GDP_ERR_INVALID, "%s: unknown decay %d", name, (int)a->decay);
    TRY(check_decode(name, a->n, a->S, a->C, a->pool, a->slots));
    if (a->n == 0 || a->S == 0) return ok();
    const int64_t unit = unit_of(a->dtype);
    bool vec = a->C % unit == 0;
    gdp::Strided x, g;
    TRY(check_input(name, "x", a->x, a->x_n_stride, a->x_t_stride, a->n, a->S, a->dtype, &vec, &x, unit));
    TRY(check_input(name, "g", a->g, a->g_n_stride, a->g_t_stride, a->n, a->S, a->g_dtype, &vec, &g, unit_of(a->g_dtype)));
    TRY(check_output(name, "y", a->y, a->dtype, &vec, unit));
    TRY(check_on_top(name, "x", a->y, a->dtype, a->x, a->dtype, a->x_n_stride, a->x_t_stride, a->n, a->S, a->C));
    TRY(check_on_top(name, "g", a->y, a->dtype, a->g, a->g_dtype, a->g_n_stride, a->g_t_stride, a->n, a->S, a->C));
    if (!a->state && a->pool > 0) return fail(GDP_ERR_INVALID, "%s: state is NULL", name);
    TRY(check_states(name, "state", a->state, GDP_F32, &vec, 1));
    return hip_status(gdp::launch_linrec_decode(*a, vec, (hipStream_t)stream), name);
}

gdp_status gdp_conv_fwd(const gdp_conv_args *a, void *stream) {
    const char *name = "gdp_conv_fwd";
    gdp::ShortConv p;
    TRY(check_conv(name, a, &p));
    TRY(check_taps(name, a->w, a->b));
    const int64_t unit = unit_of(a->dtype);
    if (p.m.rows > 0) {
        TRY(check_input(name, "x", a->x, a->x_b_stride, a->x_t_stride, a->B, a->T, a->dtype, &p.vec, &p.x, unit));
        TRY(check_output(name, "y", a->y, a->dtype, &p.vec, unit));
        if (a->x == a->y) return fail(GDP_ERR_INVALID, "%s: y may not be x", name);
    }
    TRY(check_states(name, "h0", a->h0, a->dtype, &p.vec, unit));
    TRY(check_states(name, "ht", a->ht, a->dtype, &p.vec, unit));
    if (a->ht && a->ht == a->h0) return fail(GDP_ERR_INVALID, "%s: ht may not be h0", name);
    p.w = a->w;
    p.b = a->b;
    p.h0 = a->h0;
    p.y = a->y;
    p.ht = a->ht;
    if (!gdp::conv_fits(p, a->dtype, false)) return too_large(name);
    if (p.m.nseq == 0 || (p.m.rows == 0 && !p.ht)) return ok();
    return hip_status(gdp::launch_conv(p, a->dtype, (hipStream_t)stream), name);
}

int64_t gdp_conv_workspace_bytes(const gdp_conv_args *a) {
    gdp::ShortConv p;
    if (check_conv("gdp_conv_workspace_bytes", a, &p) != GDP_OK) return -1;
    return largest_space(p, a->dtype);
}

gdp_status gdp_conv_bwd(const gdp_conv_args *a, const gdp_conv_grads *d, void *workspace, int64_t workspace_bytes,
                        void *stream) {
    const char *name = "gdp_conv_bwd";
    gdp::ShortConv p;
    TRY(check_conv(name, a, &p));
    if (!d) return fail(GDP_ERR_INVALID, "%s: grads is NULL", name);
    TRY(check_taps(name, a->w, a->b));
    const int64_t unit = unit_of(a->dtype);
    if (p.m.rows > 0) {
        TRY(check_input(name, "x", a->x, a->x_b_stride, a->x_t_stride, a->B, a->T, a->dtype, &p.vec, &p.x, unit));
        TRY(check_input(name, "dy", d->dy, d->dy_b_stride, d->dy_t_stride, a->B, a->T, a->dtype, &p.vec, &p.dy, unit));
        TRY(check_output(name, "dx", d->dx, a->dtype, &p.vec, unit));
        if (d->dx == a->x || d->dx == d->dy) return fail(GDP_ERR_INVALID, "%s: dx may not be x or dy", name);
    }
    TRY(check_states(name, "h0", a->h0, a->dtype, &p.vec, unit));
    TRY(check_states(name, "dht", d->dht, a->dtype, &p.vec, unit));
    TRY(check_states(name, "dh0", d->dh0, a->dtype, &p.vec, unit));
    if (d->dh0 && (d->dh0 == d->dht || d->dh0 == a->h0))
        return fail(GDP_ERR_INVALID, "%s: dh0 may not be dht or h0", name);
    if (((uintptr_t)d->dw | (uintptr_t)d->db) & 3)
        return fail(GDP_ERR_INVALID, "%s: dw or db is not 4-byte aligned", name);
    p.w = a->w;
    p.b = a->b;
    p.h0 = a->h0;
    p.dht = d->dht;
    p.dx = d->dx;
    p.dw = d->dw;
    p.db = d->db;
    p.dh0 = d->dh0;
    if (!gdp::conv_fits(p, a->dtype, true)) return too_large(name);
    if (d->dw || d->db) {
        TRY(check_space(name, workspace, workspace_bytes, largest_space(p, a->dtype)));
        p.part = (float *)workspace;
    }
    if (p.m.rows == 0 && !p.part && !p.dh0) return ok();
    return hip_status(gdp::launch_conv_bwd(p, a->dtype, (hipStream_t)stream), name);
}

gdp_status gdp_conv_decode(const gdp_conv_decode_args *a, void *stream) {
    const char *name = "gdp_conv_decode";
    if (!a) return fail(GDP_ERR_INVALID, "%s: args is NULL", name);
    gdp_conv_args sizes{};
    sizes.B = sizes.T = 1;
    sizes.C = a->C;
    sizes.W = a->W;
    sizes.dtype = a->dtype;
    sizes.activation = a->activation;
    gdp::ShortConv p;
    TRY(check_conv(name, &sizes, &p));
    TRY(check_decode(name, a->n, a->S, a->C, a->pool, a->slots));
    if (a->n == 0 || a->S == 0) return ok();
    TRY(check_taps(name, a->w, a->b));
    const int64_t unit = unit_of(a->dtype);
    TRY(check_input(name, "x", a->x, a->x_n_stride, a->x_t_stride, a->n, a->S, a->dtype, &p.vec, &p.x, unit));
    TRY(check_output(name, "y", a->y, a->dtype, &p.vec, unit));
    TRY(check_on_top(name, "x", a->y, a->dtype, a->x, a->dtype, a->x_n_stride, a->x_t_stride, a->n, a->S, a->C));
    if (!a->state && a->pool > 0) return fail(GDP_ERR_INVALID, "%s: state is NULL", name);
    TRY(check_states(name, "state", a->state, a->dtype, &p.vec, unit));
    return hip_status(gdp::launch_conv_decode(*a, p.vec, (hipStream_t)stream), name);
}

gdp_status gdp_rotary(const gdp_rotary_args *a, void *stream) {
    const char *name = "gdp_rotary";
    if (!a) return fail(GDP_ERR_INVALID, "%s: args is NULL", name);
    if (!known(a->dtype)) return fail(GDP_ERR_INVALID, "%s: unknown dtype %d", name, (int)a->dtype);
    if (a->H < 0 || a->HK < 0 || (int64_t)a->H + a->HK < 1 || a->D < 1)
        return fail(GDP_ERR_INVALID, "%s: H + HK and D must be >= 1", name);
    if (a->R < 2 || a->R % 2 || a->R > a->D) return fail(GDP_ERR_INVALID, "%s: R=%d must be even, 2 to D", name, a->R);
    if (a->D > 4096 || ((int64_t)a->H + a->HK) * a->D > (1 << 24))
        return fail(GDP_ERR_UNSUPPORTED, "%s: D over 4096 or rows of over 2^24 elements", name);
    if (!std::isfinite(a->scale)) return fail(GDP_ERR_INVALID, "%s: scale is not finite", name);
    gdp::Rotary p{};
    TRY(check_map(name, a->B, a->T, a->cu_seqlens, a->num_seqs, &p.m));
    if (a->positions && a->offsets) return fail(GDP_ERR_INVALID, "%s: at most one of positions and offsets", name);
    if (((uintptr_t)a->positions | (uintptr_t)a->offsets) & 3)
        return fail(GDP_ERR_INVALID, "%s: positions or offsets is not 4-byte aligned", name);
    if (a->positions && ((a->B > 1 && a->pos_b_stride < 0) || (a->T > 1 && a->pos_t_stride < 0)))
        return fail(GDP_ERR_INVALID, "%s: strides of positions must be >= 0", name);
    if (!a->freq || ((uintptr_t)a->freq & 7)) return fail(GDP_ERR_INVALID, "%s: freq is NULL or not 8-byte aligned", name);
    if (p.m.rows == 0 || p.m.nseq == 0) return ok();
    const int64_t unit = unit_of(a->dtype);
    p.vec = a->D % unit == 0 && (a->interleaved ? a->R : a->R / 2) % unit == 0;
    const struct {
        const char *in, *out;
        int32_t heads;
        const void *x;
        int64_t bs, ts;
        void *y;
        int64_t ybs, yts;
    } t[2] = {{"q", "qo", a->H, a->q, a->q_b_stride, a->q_t_stride, a->qo, a->qo_b_stride, a->qo_t_stride},
              {"k", "ko", a->HK, a->k, a->k_b_stride, a->k_t_stride, a->ko, a->ko_b_stride, a->ko_t_stride}};
    for (int i = 0; i < 2; ++i) {
        p.H[i] = t[i].heads;
        if (!t[i].heads) continue;
        TRY(check_input(name, t[i].in, t[i].x, t[i].bs, t[i].ts, a->B, a->T, a->dtype, &p.vec, &p.in[i], unit));
        TRY(check_input(name, t[i].out, t[i].y, t[i].ybs, t[i].yts, a->B, a->T, a->dtype, &p.vec, &p.out[i], unit));
        const int64_t width = (int64_t)t[i].heads * a->D;
        if (rows_overlap(a->B, a->T, t[i].ybs, t[i].yts, width))
            return fail(GDP_ERR_INVALID, "%s: rows of %s overlap", name, t[i].out);
        if (t[i].x == t[i].y && (p.in[i].bs != p.out[i].bs || p.in[i].ts != p.out[i].ts))
            return fail(GDP_ERR_INVALID, "%s: %s is %s with other strides", name, t[i].out, t[i].in);
    }
    if (a->H && a->HK && (a->qo == a->ko || a->qo == a->k || a->ko == a->q))
        return fail(GDP_ERR_INVALID, "%s: an output lies on another tensor", name);
    p.D = a->D;
    p.R = a->R;
    p.interleaved = a->interleaved != 0;
    p.inverse = a->inverse != 0;
    p.scale = a->scale;
    p.positions = a->positions;
    p.pos_bs = a->pos_b_stride;
    p.pos_ts = a->pos_t_stride;
    p.offsets = a->offsets;
    p.freq = a->freq;
    if (!gdp::rotary_fits(p, a->dtype)) return too_large(name);
    return hip_status(gdp::launch_rotary(p, a->dtype, (hipStream_t)stream), name);
}

}  // extern "C"

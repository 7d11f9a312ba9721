// api_linattn.cpp -- the C ABI of the linear-attention and group-norm entry
// points (include/gdp.h): argument validation, the segment plan, workspace
// layout and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <cmath>

#include "api_common.h"
#include "gdp_internal.h"
#include "groupnorm.h"
#include "linattn.h"

using namespace gdp::api;

namespace {

int64_t round_up(int64_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// Consecutive arrays of a workspace.
struct Arena {
    char *base;
    int64_t used = 0;
    template <typename T> T *take(int64_t n) {
        T *p = base ? (T *)(base + used) : nullptr;
        used += round_up(n * (int64_t)sizeof(T));
        return p;
    }
};

// The cut of every sequence into segments of seg_tok tokens (seg_tok >= T: none).
struct Plan {
    int64_t nseq, seg_tok, items;
    bool segments;
};

// Segments of all sequences together that fill the card: as many walks as its
// 256 compute units hold at once (by registers and LDS two blocks of eight
// waves or three of four to a unit; one where a walk keeps 256 rows of S^T).
int64_t segments_to_fill(const gdp_linattn_args &a, bool backward) {
    const int sl = backward ? gdp::lin_grads_slice(a.K, a.V) : (a.V < 128 ? a.V : 128);
    const int da = backward ? a.V : a.K;
    const int64_t walks = da == 256 ? 256 : sl == 64 ? 768 : 512;
    return walks / ((int64_t)a.HV * (backward ? 2 * a.K / sl : a.V / sl));  // backward: dq and dk first
}

Plan plan_of(const gdp_linattn_args &a, bool backward) {
    Plan p;
    p.nseq = a.cu_seqlens ? a.num_seqs : a.B;
    p.seg_tok = a.T > 0 ? a.T : 1;
    p.segments = false;
    p.items = p.nseq;
    // eight chunks one after the other take as long as the two launches more
    if (p.nseq == 0 || a.T <= 512) return p;
    const int64_t fill = segments_to_fill(a, backward);
    int64_t seg = a.T;
    if (a.cu_seqlens) {
        // The lengths lie on the device.  With as many requests as fill the
        // card none is cut (backwards only at 2048 rows): 64 requests of 500
        // tokens, 16 heads, take 150 us, 187 cut as below.  The price is a long
        // request among them, which one walk a head then takes alone: 30000
        // tokens and 31 requests of 200 take 1867 us, 272 cut (backwards 868
        // and 810).
        // Fewer requests are ragged: last segments are half full on average, and the long
        // walks of the gradients are cut finer, so that none ends alone (8
        // requests of 821 to 3562 tokens, 16 heads: once / twice / three / four
        // times the card 451 / 441 / 466 / 493 us)
        const int64_t n = (backward ? 2 : 1) * fill - p.nseq / 2;
        if (p.nseq < fill) seg = cdiv(a.T, n > 1 ? n : 1);
    } else if (fill >= 2 * a.B) {
        seg = cdiv(a.T, fill / a.B);
    }
    // backward: the running sums of dg are as long as a segment
    if (backward && seg > 2048) seg = 2048;
    seg = (seg + 63) / 64 * 64;
    if (seg < 128) seg = 128;  // a state costs as much traffic as 128 rows
    if (seg >= a.T) return p;
    p.segments = true;
    p.seg_tok = seg;
    p.items = a.cu_seqlens ? cdiv(a.T, seg) + p.nseq : a.B * cdiv(a.T, seg);
    return p;
}

// Whether every launch of a call fits: the walks (4 max(K, V) threads a head and item), dg (512), the scan (256 a head
// and sequence), and backwards the passes over the tokens of packed requests and of shared heads.
bool launches_fit(const gdp_linattn_args &a, const Plan &p, bool backward) {
    const int64_t wide = 4 * (int64_t)(a.K > a.V ? a.K : a.V), n = p.items > p.nseq ? p.items : p.nseq;
    if (!fits_launch(n * a.HV * (wide > 512 ? wide : 512))) return false;
    return !backward || (fits_launch((a.T + 63) / 64 * 256) &&
                         (a.H == a.HV || fits_launch(a.B * a.T * a.H * (a.K / 4) + 255)));
}

struct FwdSpace {
    float *seg, *tot;
};
int64_t lay_fwd(const gdp_linattn_args &a, const Plan &p, void *ws, FwdSpace *s) {
    Arena m{(char *)ws};
    const int64_t heads = p.segments ? p.items * a.HV : 0;
    s->seg = m.take<float>(heads * a.K * a.V);
    s->tot = m.take<float>(heads);
    return m.used;
}

struct BwdSpace {
    float *s, *s_tot, *r, *r_tot, *rho_q, *rho_k, *rho_in, *s_mid, *r_mid, *dq, *dk, *dh0;
    double *part;
    int nq, nk, spans;
};
int64_t lay_bwd(const gdp_linattn_args &a, const Plan &p, void *ws, BwdSpace *s) {
    Arena m{(char *)ws};
    const int64_t heads = p.segments ? p.items * a.HV : 0, E = (int64_t)a.K * a.V, BTH = a.B * a.T * a.HV;
    s->s = m.take<float>(heads * E);
    s->s_tot = m.take<float>(heads);
    s->r = m.take<float>(heads * E);
    s->r_tot = m.take<float>(heads);
    s->nq = s->nk = a.K / gdp::lin_grads_slice(a.K, a.V);
    s->rho_q = m.take<float>(s->nq * BTH);
    s->rho_k = m.take<float>(s->nk * BTH);
    // a decay per head (or none yet): the pairs of a chunk apart, and the states at the borders of spans
    s->spans = (int)cdiv(p.seg_tok, gdp::LIN_SPAN);
    const int64_t mids = a.g || s->spans == 1 ? 0 : a.B * a.T / gdp::LIN_SPAN + 1;
    s->rho_in = m.take<float>(a.g ? 0 : s->nq * BTH);
    s->s_mid = m.take<float>(mids * a.HV * E);
    s->r_mid = m.take<float>(mids * a.HV * E);
    s->part = m.take<double>(a.g ? 0 : p.items * a.HV);
    const bool shared = a.HV != a.H;
    s->dq = m.take<float>(shared ? BTH * a.K : 0);
    s->dk = m.take<float>(shared ? BTH * a.K : 0);
    s->dh0 = m.take<float>(a.h0 ? p.nseq * a.HV * E : 0);
    return m.used;
}

gdp_status check_dims(const char *name, int32_t H, int32_t HV, int32_t K, int32_t V, float scale, gdp_dtype dtype) {
    if (dtype != GDP_F32 && dtype != GDP_BF16) return fail(GDP_ERR_INVALID, "%s: unknown dtype %d", name, (int)dtype);
    if (H < 1 || HV < 1 || HV % H) return fail(GDP_ERR_INVALID, "%s: HV must be a positive multiple of H", name);
    if ((int64_t)HV * (K > V ? K : V) > (1 << 22))
        return fail(GDP_ERR_UNSUPPORTED, "%s: rows of over 2^22 elements (HV=%d)", name, HV);
    if (!(K == 64 || K == 128) || !(V == 64 || V == 128 || V == 256))
        return fail(GDP_ERR_UNSUPPORTED, "%s: head dims K=%d, V=%d not built (K in {64, 128}, V in {64, 128, 256})", name,
                    K, V);
    if (!std::isfinite(scale)) return fail(GDP_ERR_INVALID, "%s: scale is not finite", name);
    return ok();
}

// Rows of a strided [B, T, width] input: base and strides on 16 bytes, no overlap, and a chunk of rows within 32-bit
// offsets.  The stride of a dimension of one element does not matter.
gdp_status check_rows(const char *name, const char *what, const void *p, int64_t bs, int64_t ts, int64_t B, int64_t T,
                      int64_t width, gdp_dtype dtype) {
    const int64_t unit = 16 / (int64_t)dsize(dtype);
    if (!p) return fail(GDP_ERR_INVALID, "%s: %s is NULL", name, what);
    if (bs < 0 || ts < 0) return fail(GDP_ERR_INVALID, "%s: strides of %s must be >= 0", name, what);
    if (!aligned16(p) || (B > 1 && bs % unit) || (T > 1 && ts % unit))
        return fail(GDP_ERR_INVALID, "%s: rows of %s are not 16-byte aligned", name, what);
    if (T > 1 && ts < width)
        return fail(GDP_ERR_INVALID, "%s: rows of %s overlap (stride %lld < width %lld)", name, what, (long long)ts,
                    (long long)width);
    if (T > 1 && ts > (1 << 23)) return fail(GDP_ERR_UNSUPPORTED, "%s: token stride of %s over 2^23 elements", name, what);
    return ok();
}

gdp_status check_sizes(const char *name, const gdp_linattn_args *a) {
    if (!a) return fail(GDP_ERR_INVALID, "%s: args is NULL", name);
    const gdp_status st = check_dims(name, a->H, a->HV, a->K, a->V, a->scale, a->dtype);
    if (st != GDP_OK) return st;
    if (a->B < 0 || a->T < 0) return fail(GDP_ERR_INVALID, "%s: B and T must be >= 0", name);
    if (a->cu_seqlens && a->B != 1) return fail(GDP_ERR_INVALID, "%s: cu_seqlens requires B == 1", name);
    if (a->cu_seqlens && a->num_seqs < 0) return fail(GDP_ERR_INVALID, "%s: num_seqs < 0", name);
    const int64_t nseq = a->cu_seqlens ? a->num_seqs : a->B;
    // launches and 32-bit item ids: every item count below is under T B / 64 + nseq
    if (a->T > 0x7fffffff || a->B > 0x7fffffff || nseq > 0x7fffffff || a->B * a->T > ((int64_t)1 << 36) ||
        (a->B * cdiv(a->T, 64) + nseq) * a->HV * 4 > 0x7fffffff)
        return fail(GDP_ERR_UNSUPPORTED, "%s: problem too large for one launch", name);
    return ok();
}

gdp_status check_linattn(const char *name, const gdp_linattn_args *a, bool forward) {
    gdp_status st = check_sizes(name, a);
    if (st != GDP_OK) return st;
    const int64_t nseq = a->cu_seqlens ? a->num_seqs : a->B;
    if (a->g && a->g_head) return fail(GDP_ERR_INVALID, "%s: at most one of g and g_head", name);
    if (a->g && (a->g_b_stride < 0 || a->g_t_stride < 0))
        return fail(GDP_ERR_INVALID, "%s: strides of g must be >= 0", name);
    if (((uintptr_t)a->g | (uintptr_t)a->g_head | (uintptr_t)a->cu_seqlens) & 3)
        return fail(GDP_ERR_INVALID, "%s: g, g_head or cu_seqlens is not 4-byte aligned", name);
    if (!aligned16(a->h0) || !aligned16(a->ht)) return fail(GDP_ERR_INVALID, "%s: h0 or ht is not 16-byte aligned", name);
    if (a->T == 0 || (forward ? nseq : a->B) == 0) return ok();
    if ((st = check_rows(name, "q", a->q, a->q_b_stride, a->q_t_stride, a->B, a->T, (int64_t)a->H * a->K, a->dtype)) != GDP_OK) return st;
    if ((st = check_rows(name, "k", a->k, a->k_b_stride, a->k_t_stride, a->B, a->T, (int64_t)a->H * a->K, a->dtype)) != GDP_OK) return st;
    if ((st = check_rows(name, "v", a->v, a->v_b_stride, a->v_t_stride, a->B, a->T, (int64_t)a->HV * a->V, a->dtype)) != GDP_OK) return st;
    if (forward && (!a->o || !aligned16(a->o))) return fail(GDP_ERR_INVALID, "%s: o is NULL or not 16-byte aligned", name);
    return ok();
}

// A tensor of a walk; the stride of a single token does not matter and is made that of a plain row.
gdp::LinRows rows_of(const void *p, int64_t bs, int64_t ts, int64_t T, int64_t width, int div) {
    return gdp::LinRows{p, bs, T > 1 ? ts : width, div};
}

// What every walk of a call shares.
gdp::LinWalk walk_base(const gdp_linattn_args &a, const Plan &p) {
    gdp::LinWalk w{};
    w.HV = a.HV;
    w.B = a.B;
    w.T = a.T;
    w.nseq = p.nseq;
    w.seg_tok = p.seg_tok;
    w.items = p.items;
    w.cu = a.cu_seqlens;
    w.g = a.g ? a.g : a.g_head;
    w.g_bs = a.g ? a.g_b_stride : 0;
    w.g_ts = a.g ? a.g_t_stride : 0;
    w.sb = w.sy = 1.0f;
    return w;
}
gdp::LinScan scan_base(const gdp_linattn_args &a, const Plan &p) {
    gdp::LinScan s{};
    s.cu = a.cu_seqlens;
    s.T = a.T;
    s.nseq = p.nseq;
    s.seg_tok = p.seg_tok;
    s.elems = (int64_t)a.K * a.V;
    s.items = p.items;
    s.HV = a.HV;
    return s;
}

}  // namespace

extern "C" {

int64_t gdp_linattn_workspace_bytes(const gdp_linattn_args *a, int32_t backward) {
    if (check_sizes("gdp_linattn_workspace_bytes", a) != GDP_OK) return -1;
    const Plan p = plan_of(*a, backward != 0);
    if (!launches_fit(*a, p, backward != 0)) {
        fail(GDP_ERR_UNSUPPORTED, "gdp_linattn_workspace_bytes: problem too large for one launch");
        return -1;
    }
    FwdSpace f;
    BwdSpace b;
    return backward ? lay_bwd(*a, p, nullptr, &b) : lay_fwd(*a, p, nullptr, &f);
}

gdp_status gdp_linattn_fwd(const gdp_linattn_args *args, void *workspace, int64_t workspace_bytes, void *stream) {
    const char *name = "gdp_linattn_fwd";
    gdp_status st = check_linattn(name, args, true);
    if (st != GDP_OK) return st;
    gdp_linattn_args a = *args;
    if (!(a.scale > 0.f)) a.scale = 1.0f / std::sqrt((float)a.K);
    const Plan p = plan_of(a, false);
    if (!launches_fit(a, p, false)) return fail(GDP_ERR_UNSUPPORTED, "%s: problem too large for one launch", name);
    FwdSpace ws;
    if ((st = check_space(name, workspace, workspace_bytes, lay_fwd(a, p, workspace, &ws))) != GDP_OK) return st;
    if (p.nseq == 0 || (a.T == 0 && !a.ht)) return ok();
    hipStream_t s = (hipStream_t)stream;

    gdp::LinWalk w = walk_base(a, p);
    const int r = a.HV / a.H;
    w.a = rows_of(a.q, a.q_b_stride, a.q_t_stride, a.T, (int64_t)a.H * a.K, r);
    w.b = rows_of(a.k, a.k_b_stride, a.k_t_stride, a.T, (int64_t)a.H * a.K, r);
    w.c = rows_of(a.v, a.v_b_stride, a.v_t_stride, a.T, (int64_t)a.HV * a.V, 1);
    w.da = a.K;
    w.dc = a.V;
    w.s0 = a.h0;
    if (p.segments) {
        gdp::LinWalks e{{w, {}, {}}, 1};
        e.w[0].seg_out = ws.seg;
        e.w[0].seg_tot = ws.tot;
        if ((st = hip_status(gdp::launch_lin_segments(e, a.dtype, a.ht != nullptr, false, s), name)) != GDP_OK) return st;
        gdp::LinScan c = scan_base(a, p);
        c.n = 1;
        c.s[0] = {false, a.h0, ws.seg, ws.tot};
        if ((st = hip_status(gdp::launch_lin_scan(c, s), name)) != GDP_OK) return st;
        w.seg_in = ws.seg;
    }
    w.sy = a.scale;
    w.y = a.o;
    w.s_out = a.ht;
    return hip_status(gdp::launch_lin_rows({{w, {}, {}}, 1}, a.dtype, a.ht != nullptr, s), name);
}

gdp_status gdp_linattn_bwd(const gdp_linattn_args *args, const gdp_linattn_grads *d, void *workspace,
                           int64_t workspace_bytes, void *stream) {
    const char *name = "gdp_linattn_bwd";
    gdp_status st = check_linattn(name, args, false);
    if (st != GDP_OK) return st;
    if (!d) return fail(GDP_ERR_INVALID, "%s: grads is NULL", name);
    gdp_linattn_args a = *args;
    if (d->dg && !a.g) return fail(GDP_ERR_INVALID, "%s: dg without g", name);
    if (d->dg_head && !a.g_head) return fail(GDP_ERR_INVALID, "%s: dg_head without g_head", name);
    if (d->dh0 && !a.h0) return fail(GDP_ERR_INVALID, "%s: dh0 without h0", name);
    if (((uintptr_t)d->dg | (uintptr_t)d->dg_head) & 3)
        return fail(GDP_ERR_INVALID, "%s: dg or dg_head is not 4-byte aligned", name);
    if (!aligned16(d->dht) || !aligned16(d->dh0))
        return fail(GDP_ERR_INVALID, "%s: dht or dh0 is not 16-byte aligned", name);
    if (d->dh0 && (d->dh0 == d->dht || d->dh0 == a.h0))
        return fail(GDP_ERR_INVALID, "%s: dh0 may not be dht or h0", name);
    if (!(a.scale > 0.f)) a.scale = 1.0f / std::sqrt((float)a.K);
    const Plan p = plan_of(a, true);
    if (!launches_fit(a, p, true)) return fail(GDP_ERR_UNSUPPORTED, "%s: problem too large for one launch", name);
    if (a.B > 0 && a.T > 0) {
        if ((st = check_rows(name, "dout", d->dout, d->do_b_stride, d->do_t_stride, a.B, a.T, (int64_t)a.HV * a.V,
                             a.dtype)) != GDP_OK) return st;
        if (!d->dq || !d->dk || !d->dv || !aligned16(d->dq) || !aligned16(d->dk) || !aligned16(d->dv))
            return fail(GDP_ERR_INVALID, "%s: dq, dk or dv is NULL or not 16-byte aligned", name);
    }
    BwdSpace ws;
    if ((st = check_space(name, workspace, workspace_bytes, lay_bwd(a, p, workspace, &ws))) != GDP_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    const bool want_g = d->dg || d->dg_head;
    gdp::LinDg g{};
    g.cu = a.cu_seqlens;
    g.B = a.B;
    g.T = a.T;
    g.nseq = p.nseq;
    g.seg_tok = p.seg_tok;
    g.elems = (int64_t)a.K * a.V;
    g.items = p.items;  // 0 without sequences: dg_head is zero then
    g.HV = a.HV;
    g.spans = ws.spans;
    g.chunk = a.dtype == GDP_F32 ? 32 : 64;

    const int r = a.HV / a.H;
    const int64_t wk = (int64_t)a.H * a.K, wv = (int64_t)a.HV * a.V;
    if (p.nseq == 0 && a.T == 0) return hip_status(gdp::launch_lin_dg(g, d->dg_head, s), name);
    const gdp::LinRows q = rows_of(a.q, a.q_b_stride, a.q_t_stride, a.T, wk, r),
                       k = rows_of(a.k, a.k_b_stride, a.k_t_stride, a.T, wk, r),
                       v = rows_of(a.v, a.v_b_stride, a.v_t_stride, a.T, wv, 1),
                       o = rows_of(d->dout, d->do_b_stride, d->do_t_stride, a.T, wv, 1);
    const gdp::LinWalk base = walk_base(a, p);
    const bool shared = r > 1;
    // the states S entering every segment, and their gradients entering it from behind
    if (p.segments) {
        gdp::LinWalk f = base;
        f.da = a.K;
        f.dc = a.V;
        f.b = k;
        f.c = v;
        f.seg_out = ws.s;
        f.seg_tot = ws.s_tot;
        gdp::LinWalk b = f;
        b.b = q;
        b.c = o;
        b.sb = a.scale;
        b.seg_out = ws.r;
        b.seg_tot = ws.r_tot;
        if ((st = hip_status(gdp::launch_lin_segments({{f, b, {}}, 2}, a.dtype, d->dh0 != nullptr, want_g, s), name)) != GDP_OK)
            return st;
        gdp::LinScan c = scan_base(a, p);
        c.n = 2;
        c.s[0] = {false, a.h0, ws.s, ws.s_tot};
        c.s[1] = {true, d->dht, ws.r, ws.r_tot};
        if ((st = hip_status(gdp::launch_lin_scan(c, s), name)) != GDP_OK) return st;
    }
    // dq: (do, v, k) forwards from S^T; dk: (v, do, q) backwards from the gradient's transpose
    gdp::LinWalk f = base;
    f.a = o;
    f.b = v;
    f.c = k;
    f.x = q;
    f.da = a.V;
    f.dc = a.K;
    f.trans = true;
    f.s0 = a.h0;
    f.seg_in = p.segments ? ws.s : nullptr;
    f.sy = a.scale;
    f.y = shared ? (void *)ws.dq : d->dq;
    f.y32 = shared;
    f.rho = ws.rho_q;
    f.rho_in_chunk = d->dg_head ? ws.rho_in : nullptr;
    f.mid = d->dg_head && ws.spans > 1 ? ws.s_mid : nullptr;
    gdp::LinWalk w = f;
    w.a = v;
    w.b = o;
    w.c = q;
    w.x = k;
    w.s0 = d->dht;
    w.seg_in = p.segments ? ws.r : nullptr;
    w.sb = a.scale;
    w.sy = 1.0f;
    w.y = shared ? (void *)ws.dk : d->dk;
    w.rho = ws.rho_k;
    w.mid = f.mid ? ws.r_mid : nullptr;
    // dv: (k, q, do) backwards
    gdp::LinWalk x = w;
    x.a = k;
    x.b = q;
    x.c = o;
    x.x = gdp::LinRows{};
    x.da = a.K;
    x.dc = a.V;
    x.trans = false;
    x.y = d->dv;
    x.y32 = false;
    x.rho = x.mid = nullptr;
    // <h0, dh0> anchors dg where one segment has a state before it and a gradient behind it
    x.s_out = d->dh0 ? d->dh0 : want_g && d->dht && a.h0 ? ws.dh0 : nullptr;
    if ((st = hip_status(gdp::launch_lin_grads({{f, w, x}, 3}, a.dtype, want_g, s), name)) != GDP_OK) return st;
    if (a.cu_seqlens && a.T > 0) {
        const int64_t es = (int64_t)dsize(a.dtype);
        const gdp::LinOutside c{{d->dq, d->dk, d->dv, d->dg}, {wk * es / 4, wk * es / 4, wv * es / 4, a.HV}, a.T, p.nseq,
                                a.cu_seqlens};
        if ((st = hip_status(gdp::launch_lin_outside(c, s), name)) != GDP_OK) return st;
    }
    if (shared) {
        const gdp::LinGroup c{{ws.dq, ws.dk}, {d->dq, d->dk}, a.B * a.T * a.H * (a.K / 4), p.nseq, a.H, r, a.K / 4,
                              a.cu_seqlens};
        if ((st = hip_status(gdp::launch_lin_group(c, a.dtype, s), name)) != GDP_OK) return st;
    }
    if (!want_g) return ok();
    g.nq = ws.nq;
    g.nk = ws.nk;
    g.g = base.g;
    g.g_bs = base.g_bs;
    g.g_ts = base.g_ts;
    g.rho_q = ws.rho_q;
    g.rho_k = ws.rho_k;
    g.rho_in_chunk = ws.rho_in;
    g.s_in = ws.s;
    g.r_in = ws.r;
    g.s_mid = ws.s_mid;
    g.r_mid = ws.r_mid;
    g.h0 = a.h0;
    g.dh0 = x.s_out;
    g.end_zero = !d->dht;
    g.dg = d->dg;
    g.part = ws.part;
    return hip_status(gdp::launch_lin_dg(g, d->dg_head, s), name);
}

gdp_status gdp_linattn_decode(const gdp_linattn_decode_args *args, void *stream) {
    const char *name = "gdp_linattn_decode";
    if (!args) return fail(GDP_ERR_INVALID, "%s: args is NULL", name);
    gdp_linattn_decode_args a = *args;
    gdp_status st = check_dims(name, a.H, a.HV, a.K, a.V, a.scale, a.dtype);
    if (st != GDP_OK) return st;
    if (a.n < 0 || a.S < 0) return fail(GDP_ERR_INVALID, "%s: n and S must be >= 0", name);
    // up to K/4 threads for each state row
    if (a.S > 4096 || a.n > 0xffffffffll / ((int64_t)a.V * (a.K / 4))) return fail(GDP_ERR_UNSUPPORTED, "%s: step too large (n or S)", name);
    if (a.pool < 0 || (!a.slots && a.pool < a.n)) return fail(GDP_ERR_INVALID, "%s: state pool too small", name);
    if (a.g && a.g_head) return fail(GDP_ERR_INVALID, "%s: at most one of g and g_head", name);
    if (a.g && (a.g_n_stride < 0 || a.g_t_stride < 0))
        return fail(GDP_ERR_INVALID, "%s: strides of g must be >= 0", name);
    if (((uintptr_t)a.g | (uintptr_t)a.g_head | (uintptr_t)a.slots) & 3)
        return fail(GDP_ERR_INVALID, "%s: g, g_head or slots is not 4-byte aligned", name);
    if (a.n == 0 || a.S == 0) return ok();
    if ((st = check_rows(name, "q", a.q, a.q_n_stride, a.q_t_stride, a.n, a.S, (int64_t)a.H * a.K, a.dtype)) != GDP_OK) return st;
    if ((st = check_rows(name, "k", a.k, a.k_n_stride, a.k_t_stride, a.n, a.S, (int64_t)a.H * a.K, a.dtype)) != GDP_OK) return st;
    if ((st = check_rows(name, "v", a.v, a.v_n_stride, a.v_t_stride, a.n, a.S, (int64_t)a.HV * a.V, a.dtype)) != GDP_OK) return st;
    if ((!a.state && a.pool > 0) || !aligned16(a.state))
        return fail(GDP_ERR_INVALID, "%s: state is NULL or not 16-byte aligned", name);
    if (!a.o || !aligned16(a.o)) return fail(GDP_ERR_INVALID, "%s: o is NULL or not 16-byte aligned", name);
    if (!(a.scale > 0.f)) a.scale = 1.0f / std::sqrt((float)a.K);
    return hip_status(gdp::launch_lin_decode(a, (hipStream_t)stream), name);
}

}  // extern "C"

namespace {

gdp_status check_norm(const char *name, const gdp_group_norm_args *a) {
    if (!a) return fail(GDP_ERR_INVALID, "%s: args is NULL", name);
    if (a->dtype != GDP_F32 && a->dtype != GDP_BF16)
        return fail(GDP_ERR_INVALID, "%s: unknown dtype %d", name, (int)a->dtype);
    if (a->activation != GDP_ACT_NONE && a->activation != GDP_ACT_SILU && a->activation != GDP_ACT_SIGMOID)
        return fail(GDP_ERR_INVALID, "%s: unknown activation %d", name, (int)a->activation);
    if (a->n < 0 || a->T < 0 || a->groups < 1 || a->D < 1)
        return fail(GDP_ERR_INVALID, "%s: n, T must be >= 0 and groups, D >= 1", name);
    if (!(a->eps >= 0.f) || std::isinf(a->eps)) return fail(GDP_ERR_INVALID, "%s: eps must be finite and >= 0", name);
    if (a->D > 4096) return fail(GDP_ERR_UNSUPPORTED, "%s: D=%d over 4096", name, a->D);
    if (a->n > 0x7fffffff || a->T > 0x7fffffff || (a->T > 0 && a->n * a->T > 0x7fffffff) ||
        (int64_t)a->groups * a->D > (1 << 27))
        return fail(GDP_ERR_UNSUPPORTED, "%s: problem too large for one launch", name);
    return ok();
}

// A strided [n, T, C] tensor of whole elements; *vec is cleared where its rows do not start on 16 bytes.
gdp_status check_strided(const char *name, const char *what, const void *p, int64_t ns, int64_t ts, gdp_dtype dtype,
                         bool *vec) {
    if (!p) return fail(GDP_ERR_INVALID, "%s: %s is NULL", name, what);
    if (ns < 0 || ts < 0) return fail(GDP_ERR_INVALID, "%s: strides of %s must be >= 0", name, what);
    if ((uintptr_t)p % dsize(dtype)) return fail(GDP_ERR_INVALID, "%s: %s is not aligned to its type", name, what);
    const int64_t unit = 16 / (int64_t)dsize(dtype);
    if (!aligned16(p) || ns % unit || ts % unit) *vec = false;
    return ok();
}

gdp::GroupNorm norm_base(const gdp_group_norm_args &a, bool bwd) {
    gdp::GroupNorm p{};
    p.x = a.x;
    p.x_ns = a.x_n_stride;
    p.x_ts = a.x_t_stride;
    p.z = a.z;
    p.z_ns = a.z_n_stride;
    p.z_ts = a.z_t_stride;
    p.rows = a.n * a.T;
    p.T = (uint32_t)a.T;
    p.groups = a.groups;
    p.D = a.D;
    p.act = a.activation;
    p.centered = a.centered != 0;
    p.vec = true;
    p.bwd = bwd;
    p.eps = a.eps;
    p.w = a.w;
    p.b = a.b;
    p.split = gdp::group_norm_split(p.rows, a.groups, a.D, bwd);
    return p;
}

}  // namespace

extern "C" {

gdp_status gdp_group_norm_fwd(const gdp_group_norm_args *a, void *stream) {
    const char *name = "gdp_group_norm_fwd";
    gdp_status st = check_norm(name, a);
    if (st != GDP_OK || a->n * a->T == 0) return st;
    gdp::GroupNorm p = norm_base(*a, false);
    const int64_t C = (int64_t)a->groups * a->D;
    if ((st = check_strided(name, "x", a->x, a->x_n_stride, a->x_t_stride, a->dtype, &p.vec)) != GDP_OK) return st;
    if (a->z && (st = check_strided(name, "z", a->z, a->z_n_stride, a->z_t_stride, a->dtype, &p.vec)) != GDP_OK)
        return st;
    if ((st = check_strided(name, "y", a->y, a->T * C, C, a->dtype, &p.vec)) != GDP_OK) return st;
    if (((uintptr_t)a->w | (uintptr_t)a->b) & 3) return fail(GDP_ERR_INVALID, "%s: w or b is not 4-byte aligned", name);
    p.y = a->y;
    return hip_status(gdp::launch_group_norm(p, a->dtype, (hipStream_t)stream), name);
}

int64_t gdp_group_norm_workspace_bytes(const gdp_group_norm_args *a) {
    if (check_norm("gdp_group_norm_workspace_bytes", a) != GDP_OK) return -1;
    const int64_t rows = a->n * a->T, C = (int64_t)a->groups * a->D;
    return gdp::group_norm_split(rows, a->groups, a->D, true) * 2 * C * (int64_t)sizeof(float);
}

gdp_status gdp_group_norm_bwd(const gdp_group_norm_args *a, const gdp_group_norm_grads *d, void *workspace,
                              int64_t workspace_bytes, void *stream) {
    const char *name = "gdp_group_norm_bwd";
    gdp_status st = check_norm(name, a);
    if (st != GDP_OK) return st;
    if (!d) return fail(GDP_ERR_INVALID, "%s: grads is NULL", name);
    gdp::GroupNorm p = norm_base(*a, true);
    const int64_t C = (int64_t)a->groups * a->D;
    if (((uintptr_t)a->w | (uintptr_t)a->b | (uintptr_t)d->dw | (uintptr_t)d->db) & 3)
        return fail(GDP_ERR_INVALID, "%s: w, b, dw or db is not 4-byte aligned", name);
    if (p.rows > 0) {
        if ((st = check_strided(name, "x", a->x, a->x_n_stride, a->x_t_stride, a->dtype, &p.vec)) != GDP_OK) return st;
        if (a->z && (st = check_strided(name, "z", a->z, a->z_n_stride, a->z_t_stride, a->dtype, &p.vec)) != GDP_OK)
            return st;
        if ((st = check_strided(name, "dy", d->dy, d->dy_n_stride, d->dy_t_stride, a->dtype, &p.vec)) != GDP_OK)
            return st;
        if ((st = check_strided(name, "dx", d->dx, a->T * C, C, a->dtype, &p.vec)) != GDP_OK) return st;
        if (a->z && (st = check_strided(name, "dz", d->dz, a->T * C, C, a->dtype, &p.vec)) != GDP_OK) return st;
    }
    p.dy = d->dy;
    p.dy_ns = d->dy_n_stride;
    p.dy_ts = d->dy_t_stride;
    p.dx = d->dx;
    p.dz = d->dz;
    p.dw = d->dw;
    p.db = d->db;
    if (d->dw || d->db) {
        if ((st = check_space(name, workspace, workspace_bytes, gdp_group_norm_workspace_bytes(a))) != GDP_OK) return st;
        p.part = (float *)workspace;
    }
    if (p.rows == 0 && !d->dw && !d->db) return ok();
    return hip_status(gdp::launch_group_norm(p, a->dtype, (hipStream_t)stream), name);
}

}  // extern "C"

// layer_api.cu -- the extern "C" entry points of the linear-attention layer and
// of the norms around it: host-side argument checks, workspaces and launches.
// The operations are described in include/mambascan.h.

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "mambascan.h"
#include "ms_internal.h"

namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
int elem_bytes(int32_t dt) { return dt == MS_BF16 ? 2 : 4; }
bool dtype_ok(int32_t dt) { return dt == MS_F32 || dt == MS_BF16; }

// Whether the largest element offset of an array of these extents and strides
// stays within int64 (extents >= 1, strides >= 0).
bool offsets_ok(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t n3) {
    const __int128 o = (__int128)(n0 - 1) * s0 + (__int128)(n1 - 1) * s1 + (__int128)(n2 - 1) * s2 + (n3 - 1);
    return o <= (__int128)INT64_MAX / 8;
}

// Whether an array of these extents and strides, rows of n3 dense elements at the
// end, holds no element twice: each dimension steps over all that the smaller steps span.
bool distinct(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t n3) {
    struct Dim {
        int64_t s, n;
    } d[3] = {{s0, n0}, {s1, n1}, {s2, n2}};
    std::sort(d, d + 3, [](const Dim &x, const Dim &y) { return x.s < y.s; });
    __int128 span = n3;
    for (const Dim &x : d) {
        if (x.n <= 1) continue;
        if (x.s < span) return false;
        span += (__int128)(x.n - 1) * x.s;
    }
    return true;
}

int num_sms_current() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms > 0 ? sms : 148;
}

int cuda_rc(cudaError_t e) {
    if (e == cudaSuccess) return MS_OK;
    cudaGetLastError();
    return MS_ERR_CUDA;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Sizes, strides and types of a linear-attention call, with its token arrays
// as pointers (q, k, v, o or dout, and the gradients). Arrays that are written
// must not hold an element twice: o, or (bwd) what has the strides of q, k and v.
int check_linattn(const ms_linattn_dims *d, bool packed, bool bwd, const void *const *tok, int ntok, const float *const *f32,
                  int nf32, const int32_t *seq_start) {
    if (!d) return MS_ERR_NULL;
    if (!dtype_ok(d->dtype)) return MS_ERR_DTYPE;
    if (d->batch < 0 || d->nheads < 1 || d->kv_heads < 1 || d->nheads % d->kv_heads != 0 || d->dk < 1 || d->dk > 128 ||
        d->dv < 1 || d->dv > 128 || d->nheads > INT32_MAX || (packed ? d->total : d->seqlen) < 0)
        return MS_ERR_SHAPE;
    if (d->q_sb < 0 || d->q_sl < 0 || d->q_sh < 0 || d->k_sb < 0 || d->k_sl < 0 || d->k_sh < 0 || d->v_sb < 0 ||
        d->v_sl < 0 || d->v_sh < 0 || d->o_sb < 0 || d->o_sl < 0 || d->o_sh < 0)
        return MS_ERR_STRIDE;
    const int64_t rows = packed ? d->total : d->seqlen, nb = packed ? 1 : (d->batch < 1 ? 1 : d->batch);
    if (rows > INT32_MAX - 1024 || d->batch > INT32_MAX) return MS_ERR_SHAPE;
    if (rows > 0) {
        const int64_t H = d->nheads, G = d->kv_heads;
        if (!offsets_ok(nb, d->q_sb, rows, d->q_sl, H, d->q_sh, d->dk) ||
            !offsets_ok(nb, d->k_sb, rows, d->k_sl, G, d->k_sh, d->dk) ||
            !offsets_ok(nb, d->v_sb, rows, d->v_sl, G, d->v_sh, d->dv) ||
            !offsets_ok(nb, d->o_sb, rows, d->o_sl, H, d->o_sh, d->dv) ||
            (__int128)nb * rows * H * 128 > (__int128)INT64_MAX / 8 ||
            (__int128)d->batch * d->nheads * d->dk * d->dv > (__int128)INT64_MAX / 8)
            return MS_ERR_SHAPE;
    }
    if ((__int128)d->batch * d->nheads > INT32_MAX) return MS_ERR_SHAPE;
    if (rows > 0) {
        const int64_t H = d->nheads, G = d->kv_heads;
        if (!bwd && !distinct(nb, d->o_sb, rows, d->o_sl, H, d->o_sh, d->dv)) return MS_ERR_STRIDE;
        if (bwd && (!distinct(nb, d->q_sb, rows, d->q_sl, H, d->q_sh, d->dk) ||
                    !distinct(nb, d->k_sb, rows, d->k_sl, G, d->k_sh, d->dk) ||
                    !distinct(nb, d->v_sb, rows, d->v_sl, G, d->v_sh, d->dv)))
            return MS_ERR_STRIDE;
    }
    if (d->batch == 0) return MS_OK;
    if (!f32[0]) return MS_ERR_NULL;  // log_decay
    if (rows > 0)
        for (int i = 0; i < ntok; ++i)
            if (!tok[i]) return MS_ERR_NULL;
    for (int i = 0; i < ntok; ++i)
        if (tok[i] && !aligned(tok[i], elem_bytes(d->dtype))) return MS_ERR_ALIGN;
    for (int i = 0; i < nf32; ++i)
        if (f32[i] && !aligned(f32[i], 4)) return MS_ERR_ALIGN;
    if (seq_start && !aligned(seq_start, 4)) return MS_ERR_ALIGN;
    return MS_OK;
}

ms::LaArgs la_args(const ms_linattn_dims *d, const float *log_decay, const int32_t *seq_start, int *status) {
    ms::LaArgs a{};
    a.log_decay = log_decay;
    a.seq_start = seq_start;
    a.status = status;
    a.batch = d->batch;
    a.seqlen = d->seqlen;
    a.total = d->total;
    a.H = d->nheads;
    return a;
}

// A token array in a role of a problem.
struct Tok {
    const void *p;
    int64_t sb, sl, sh;
    int share;  // heads per head of the array
    int d;
};

ms::LaProblem la_problem(const Tok &x, const Tok &y, const Tok &z, const Tok &o, const float *s0, bool s0_turned,
                         float *fin, bool rev, float scale) {
    ms::LaProblem p{};
    p.x = x.p; p.x_sb = x.sb; p.x_sl = x.sl; p.x_sh = x.sh; p.xg = x.share;
    p.y = y.p; p.y_sb = y.sb; p.y_sl = y.sl; p.y_sh = y.sh; p.yg = y.share;
    p.z = z.p; p.z_sb = z.sb; p.z_sl = z.sl; p.z_sh = z.sh; p.zg = z.share;
    p.o = const_cast<void *>(o.p); p.o_sb = o.sb; p.o_sl = o.sl; p.o_sh = o.sh;
    p.dx = x.d;
    p.dz = z.d;
    p.s0 = s0;
    p.s0_sr = s0_turned ? 1 : z.d;
    p.s0_sc = s0_turned ? x.d : 1;
    p.fin = fin;
    p.rev = rev ? 1 : 0;
    p.ws = rev ? scale : 1.0f;
    p.ro = rev ? 1.0f : scale;
    return p;
}

// fp32 gradients per query head of shared keys and values, before their sum.
size_t shared_bytes(const ms_linattn_dims *d, int64_t width, bool packed) {
    if (d->nheads == d->kv_heads) return 0;
    const size_t rows = packed ? (size_t)d->total : (size_t)d->batch * (size_t)d->seqlen;
    return round256(rows * (size_t)d->nheads * (size_t)width * sizeof(float));
}

// States between segments on the tensor-core path (needed by any bf16 call of
// these sizes, so that the size does not depend on pointers and strides).
size_t state_bytes(const ms_linattn_dims *d, bool packed, bool bwd) {
    if (!d || d->dtype != MS_BF16 || d->batch < 1 || d->nheads < 1 || d->seqlen < 0 || d->total < 0 || d->dk < 1 ||
        d->dk > 128 || d->dv < 1 || d->dv > 128)
        return 0;
    return round256(ms::linattn_tc_workspace(d->batch, packed ? d->total : d->seqlen, packed, d->nheads, (int)d->dk,
                                             (int)d->dv, bwd, num_sms_current()));
}

cudaError_t launch_linattn(const ms::LaArgs &a, bool bf16, void *states, cudaStream_t st) {
    return ms::linattn_tc_applies(a, bf16) ? ms::launch_linattn_tc(a, states, num_sms_current(), st)
                                           : ms::launch_linattn_plain(a, bf16, st);
}

}  // namespace

extern "C" {

size_t mamba_linattn_workspace_size(const ms_linattn_dims *d, int packed) {
    return state_bytes(d, packed != 0, false);
}

int mamba_linattn_fwd(const void *q, const void *k, const void *v, const float *log_decay, float scale,
                      const int32_t *seq_start, const float *initial_state, void *o, float *final_state,
                      const ms_linattn_dims *d, void *workspace, size_t workspace_bytes, int *dev_status,
                      ms_stream_t stream) {
    const void *tok[] = {q, k, v, o};
    const float *f32[] = {log_decay, initial_state, final_state};
    const bool packed = seq_start != nullptr;
    int rc = check_linattn(d, packed, false, tok, 4, f32, 3, seq_start);
    if (rc != MS_OK) return rc;
    if (d->batch == 0) return MS_OK;
    const size_t need = mamba_linattn_workspace_size(d, packed);
    if (workspace_bytes < need || (need > 0 && !workspace)) return MS_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 16)) return MS_ERR_ALIGN;
    if (o && (o == q || o == k || o == v)) return MS_ERR_SHAPE;
    const int share = (int)(d->nheads / d->kv_heads), dk = (int)d->dk, dv = (int)d->dv;
    ms::LaArgs a = la_args(d, log_decay, seq_start, dev_status);
    a.np = 1;
    a.p[0] = la_problem(Tok{q, d->q_sb, d->q_sl, d->q_sh, 1, dk}, Tok{k, d->k_sb, d->k_sl, d->k_sh, share, dk},
                        Tok{v, d->v_sb, d->v_sl, d->v_sh, share, dv}, Tok{o, d->o_sb, d->o_sl, d->o_sh, 1, dv},
                        initial_state, false, final_state, false, scale);
    return cuda_rc(launch_linattn(a, d->dtype == MS_BF16, workspace, (cudaStream_t)stream));
}

size_t mamba_linattn_bwd_workspace_size(const ms_linattn_dims *d, int packed) {
    if (!d || d->batch < 1 || d->nheads < 1 || d->kv_heads < 1 || d->seqlen < 0 || d->total < 0) return 0;
    return shared_bytes(d, d->dk, packed != 0) + shared_bytes(d, d->dv, packed != 0) + state_bytes(d, packed != 0, true);
}

int mamba_linattn_bwd(const void *q, const void *k, const void *v, const float *log_decay, float scale,
                      const int32_t *seq_start, const float *initial_state, const void *dout, const float *dfinal,
                      void *dq, void *dk_, void *dv_, float *dinitial_state, const ms_linattn_dims *d, void *workspace,
                      size_t workspace_bytes, int *dev_status, ms_stream_t stream) {
    const void *tok[] = {q, k, v, dout, dq, dk_, dv_};
    const float *f32[] = {log_decay, initial_state, dfinal, dinitial_state};
    const bool packed = seq_start != nullptr;
    int rc = check_linattn(d, packed, true, tok, 7, f32, 4, seq_start);
    if (rc != MS_OK) return rc;
    if (d->batch == 0) return MS_OK;
    if (dinitial_state && (dinitial_state == dfinal || dinitial_state == initial_state)) return MS_ERR_SHAPE;
    const size_t need = mamba_linattn_bwd_workspace_size(d, packed);
    if (workspace_bytes < need || (need > 0 && !workspace)) return MS_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 16)) return MS_ERR_ALIGN;
    for (const void *g : {dq, dk_, dv_})
        for (const void *in : {q, k, v, dout})
            if (g && g == in) return MS_ERR_SHAPE;
    if (dq && (dq == dk_ || dq == dv_ || dk_ == dv_)) return MS_ERR_SHAPE;
    const int share = (int)(d->nheads / d->kv_heads), dk = (int)d->dk, dv = (int)d->dv;
    const bool bf16 = d->dtype == MS_BF16;
    const cudaStream_t st = (cudaStream_t)stream;
    const Tok tq{q, d->q_sb, d->q_sl, d->q_sh, 1, dk}, tk{k, d->k_sb, d->k_sl, d->k_sh, share, dk};
    const Tok tv{v, d->v_sb, d->v_sl, d->v_sh, share, dv}, to{dout, d->o_sb, d->o_sl, d->o_sh, 1, dv};
    const Tok gq{dq, d->q_sb, d->q_sl, d->q_sh, 1, dk};
    Tok gk{dk_, d->k_sb, d->k_sl, d->k_sh, 1, dk}, gv{dv_, d->v_sb, d->v_sl, d->v_sh, 1, dv};
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const size_t pk = shared_bytes(d, dk, packed), pv = shared_bytes(d, dv, packed);
    if (share > 1) {
        const int64_t H = d->nheads;
        gk = Tok{ws, d->seqlen * H * dk, H * dk, dk, 1, dk};
        gv = Tok{ws + pk, d->seqlen * H * dv, H * dv, dv, 1, dv};
    }
    ms::LaArgs a = la_args(d, log_decay, seq_start, dev_status);
    a.np = 3;
    a.p[0] = la_problem(to, tv, tk, gq, initial_state, true, nullptr, false, scale);
    a.p[1] = la_problem(tv, to, tq, gk, dfinal, true, nullptr, true, scale);
    a.p[2] = la_problem(tk, tq, to, gv, dfinal, false, dinitial_state, true, scale);
    a.p[1].o_f32 = a.p[2].o_f32 = share > 1 ? 1 : 0;
    cudaError_t e = launch_linattn(a, bf16, ws + pk + pv, st);
    if (e == cudaSuccess && share > 1) {
        ms::LaReduceArgs r{};
        r.seq_start = seq_start;
        r.status = dev_status;
        r.batch = d->batch; r.seqlen = d->seqlen; r.total = d->total; r.H = d->nheads; r.kv = d->kv_heads;
        r.part = reinterpret_cast<const float *>(ws);
        r.out = dk_; r.d = dk; r.o_sb = d->k_sb; r.o_sl = d->k_sl; r.o_sh = d->k_sh;
        ms::LaReduceArgs r2 = r;
        r2.part = reinterpret_cast<const float *>(ws + pk);
        r2.out = dv_; r2.d = dv; r2.o_sb = d->v_sb; r2.o_sl = d->v_sl; r2.o_sh = d->v_sh;
        e = ms::launch_linattn_reduce(r, r2, bf16, st);
    }
    return cuda_rc(e);
}

int mamba_linattn_state_update(float *state, const void *q, const void *k, const void *v, const float *log_decay,
                               float scale, void *o, const ms_linattn_update_dims *d, int *dev_status,
                               ms_stream_t stream) {
    if (!d) return MS_ERR_NULL;
    if (!dtype_ok(d->dtype)) return MS_ERR_DTYPE;
    if (d->batch < 0 || d->nheads < 1 || d->kv_heads < 1 || d->nheads % d->kv_heads != 0 || d->dk < 1 ||
        d->dk > INT32_MAX || d->dv < 1 || d->dv > 256 || (__int128)d->batch * d->nheads > INT32_MAX)
        return MS_ERR_SHAPE;
    if (d->q_sb < 0 || d->q_sh < 0 || d->k_sb < 0 || d->k_sh < 0 || d->v_sb < 0 || d->v_sh < 0 || d->o_sb < 0 ||
        d->o_sh < 0 || d->state_sb < 0 || d->state_sh < 0)
        return MS_ERR_STRIDE;
    if (d->batch == 0) return MS_OK;
    if (!state || !q || !k || !v || !log_decay || !o) return MS_ERR_NULL;
    const int es = elem_bytes(d->dtype);
    if (!aligned(state, 4) || !aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(o, es) ||
        !aligned(log_decay, 4))
        return MS_ERR_ALIGN;
    const int64_t H = d->nheads, G = d->kv_heads;
    if (!offsets_ok(d->batch, d->state_sb, H, d->state_sh, d->dk, d->dv, d->dv) ||
        !offsets_ok(d->batch, d->q_sb, H, d->q_sh, 1, 0, d->dk) || !offsets_ok(d->batch, d->k_sb, G, d->k_sh, 1, 0, d->dk) ||
        !offsets_ok(d->batch, d->v_sb, G, d->v_sh, 1, 0, d->dv) || !offsets_ok(d->batch, d->o_sb, H, d->o_sh, 1, 0, d->dv))
        return MS_ERR_SHAPE;
    // two heads' (or rows') states in the same memory would be updated twice, in no order
    if (!distinct(d->batch, d->state_sb, H, d->state_sh, 1, 0, d->dk * d->dv) ||
        !distinct(d->batch, d->o_sb, H, d->o_sh, 1, 0, d->dv))
        return MS_ERR_STRIDE;
    ms::LaUpdateArgs a{};
    a.state = state; a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.o = o; a.status = dev_status;
    a.batch = d->batch; a.H = H; a.kv = G; a.dk = (int)d->dk; a.dv = (int)d->dv;
    a.q_sb = d->q_sb; a.q_sh = d->q_sh; a.k_sb = d->k_sb; a.k_sh = d->k_sh; a.v_sb = d->v_sb; a.v_sh = d->v_sh;
    a.o_sb = d->o_sb; a.o_sh = d->o_sh; a.st_sb = d->state_sb; a.st_sh = d->state_sh;
    a.scale = scale;
    return cuda_rc(ms::launch_linattn_update(a, d->dtype == MS_BF16, (cudaStream_t)stream));
}

// ----------------------------------------------------------------- norms ----

static int check_gated(const ms_gated_norm_dims *d) {
    if (!d) return MS_ERR_NULL;
    if (!dtype_ok(d->dtype)) return MS_ERR_DTYPE;
    if (d->rows < 0 || d->width < 1 || d->groups < 1 || d->width % d->groups != 0 ||
        d->width / d->groups > ms::kNormMaxWidth || d->groups > 65535 || !(d->eps >= 0.0f) || std::isinf(d->eps))
        return MS_ERR_SHAPE;
    if (d->x_sr < 0 || d->z_sr < 0 || d->y_sr < 0) return MS_ERR_STRIDE;
    if (d->rows > 0 &&
        (!offsets_ok(d->rows, d->x_sr, 1, 0, 1, 0, d->width) || !offsets_ok(d->rows, d->z_sr, 1, 0, 1, 0, d->width) ||
         !offsets_ok(d->rows, d->y_sr, 1, 0, 1, 0, d->width) || !offsets_ok(d->rows, d->width, 1, 0, 1, 0, d->width)))
        return MS_ERR_SHAPE;
    return MS_OK;
}

static ms::GatedNormArgs gated_args(const ms_gated_norm_dims *d, const void *x, const void *z, const float *w,
                                    int *status) {
    ms::GatedNormArgs a{};
    a.x = x; a.z = z; a.w = w; a.status = status;
    a.rows = d->rows; a.width = d->width; a.groups = d->groups;
    a.x_sr = d->x_sr; a.z_sr = d->z_sr; a.y_sr = d->y_sr;
    a.eps = d->eps;
    a.gate_first = d->gate_first ? 1 : 0;
    return a;
}

int mamba_gated_norm_fwd(const void *x, const void *z, const float *weight, void *y, const ms_gated_norm_dims *d,
                         int *dev_status, ms_stream_t stream) {
    const int rc = check_gated(d);
    if (rc != MS_OK) return rc;
    if (d->rows == 0) return MS_OK;
    if (!x || !y) return MS_ERR_NULL;
    const int es = elem_bytes(d->dtype);
    if (!aligned(x, es) || !aligned(z, es) || !aligned(y, es) || !aligned(weight, 4)) return MS_ERR_ALIGN;
    if (!distinct(d->rows, d->y_sr, 1, 0, 1, 0, d->width)) return MS_ERR_STRIDE;
    ms::GatedNormArgs a = gated_args(d, x, z, weight, dev_status);
    a.y = y;
    return cuda_rc(ms::launch_gated_norm(a, d->dtype == MS_BF16, false, num_sms_current(), (cudaStream_t)stream));
}

size_t mamba_gated_norm_bwd_workspace_size(const ms_gated_norm_dims *d) {
    if (check_gated(d) != MS_OK || d->rows == 0) return 0;
    return ms::norm_parts(d->rows, d->width, d->groups, num_sms_current()) * (size_t)d->width * sizeof(float);
}

int mamba_gated_norm_bwd(const void *x, const void *z, const float *weight, const void *dy, void *dx, void *dz,
                         float *dweight, const ms_gated_norm_dims *d, void *workspace, size_t workspace_bytes,
                         int *dev_status, ms_stream_t stream) {
    const int rc = check_gated(d);
    if (rc != MS_OK) return rc;
    const cudaStream_t st = (cudaStream_t)stream;
    if (!aligned(dweight, 4)) return MS_ERR_ALIGN;
    if (d->rows == 0)  // a sum over no rows
        return dweight ? cuda_rc(cudaMemsetAsync(dweight, 0, (size_t)d->width * sizeof(float), st)) : MS_OK;
    if (!x || !dy || !dx || (z != nullptr) != (dz != nullptr)) return MS_ERR_NULL;
    const int es = elem_bytes(d->dtype);
    if (!aligned(x, es) || !aligned(z, es) || !aligned(dy, es) || !aligned(dx, es) || !aligned(dz, es) ||
        !aligned(weight, 4))
        return MS_ERR_ALIGN;
    if (dweight) {
        if (!workspace || workspace_bytes < mamba_gated_norm_bwd_workspace_size(d)) return MS_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return MS_ERR_ALIGN;
    }
    ms::GatedNormArgs a = gated_args(d, x, z, weight, dev_status);
    a.dy = dy; a.dx = dx; a.dz = dz; a.dw = dweight;
    a.part = static_cast<float *>(workspace);
    return cuda_rc(ms::launch_gated_norm(a, d->dtype == MS_BF16, true, num_sms_current(), st));
}

static int check_residual(const ms_residual_norm_dims *d) {
    if (!d) return MS_ERR_NULL;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->res_dtype)) return MS_ERR_DTYPE;
    if (d->rows < 0 || d->width < 1 || d->width > ms::kNormMaxWidth || !(d->eps >= 0.0f) || std::isinf(d->eps))
        return MS_ERR_SHAPE;
    if (d->x_sr < 0 || d->res_sr < 0 || d->y_sr < 0 || d->resout_sr < 0) return MS_ERR_STRIDE;
    if (d->rows > 0)
        for (int64_t sr : {d->x_sr, d->res_sr, d->y_sr, d->resout_sr, d->width})
            if (!offsets_ok(d->rows, sr, 1, 0, 1, 0, d->width)) return MS_ERR_SHAPE;
    return MS_OK;
}

static ms::ResidualNormArgs residual_args(const ms_residual_norm_dims *d, const float *w, const float *cs, int *status) {
    ms::ResidualNormArgs a{};
    a.w = w; a.cs = cs; a.status = status;
    a.rows = d->rows; a.width = d->width;
    a.x_sr = d->x_sr; a.res_sr = d->res_sr; a.y_sr = d->y_sr; a.ro_sr = d->resout_sr;
    a.eps = d->eps; a.scale = d->res_scale;
    return a;
}

int mamba_residual_norm_fwd(const void *x, const void *residual, const float *weight, const float *channel_scale,
                            void *y, void *residual_out, const ms_residual_norm_dims *d, int *dev_status,
                            ms_stream_t stream) {
    const int rc = check_residual(d);
    if (rc != MS_OK) return rc;
    if (d->rows == 0) return MS_OK;
    if (!x || !y) return MS_ERR_NULL;
    const int es = elem_bytes(d->dtype), rs = elem_bytes(d->res_dtype);
    if (!aligned(x, es) || !aligned(y, es) || !aligned(residual, rs) || !aligned(residual_out, rs) ||
        !aligned(weight, 4) || !aligned(channel_scale, 4))
        return MS_ERR_ALIGN;
    // rows written twice; or, in place, one row's sum over another row that is still to be read
    if (!distinct(d->rows, d->y_sr, 1, 0, 1, 0, d->width) ||
        (residual_out && !distinct(d->rows, d->resout_sr, 1, 0, 1, 0, d->width)) ||
        (residual_out && residual_out == residual && d->rows > 1 && d->res_sr != d->resout_sr))
        return MS_ERR_STRIDE;
    ms::ResidualNormArgs a = residual_args(d, weight, channel_scale, dev_status);
    a.x = x; a.res = residual; a.y = y; a.res_out = residual_out;
    return cuda_rc(ms::launch_residual_norm(a, d->dtype == MS_BF16, d->res_dtype == MS_BF16, false, num_sms_current(),
                                            (cudaStream_t)stream));
}

size_t mamba_residual_norm_bwd_workspace_size(const ms_residual_norm_dims *d) {
    if (check_residual(d) != MS_OK || d->rows == 0) return 0;
    return 2 * ms::norm_parts(d->rows, d->width, 1, num_sms_current()) * (size_t)d->width * sizeof(float);
}

int mamba_residual_norm_bwd(const void *residual_out, const float *weight, const void *dy, const void *dresidual_out,
                            const void *x, const float *channel_scale, void *dx, void *dresidual, float *dweight,
                            float *dchannel_scale, const ms_residual_norm_dims *d, void *workspace,
                            size_t workspace_bytes, int *dev_status, ms_stream_t stream) {
    const int rc = check_residual(d);
    if (rc != MS_OK) return rc;
    const cudaStream_t st = (cudaStream_t)stream;
    if (!aligned(dweight, 4) || !aligned(dchannel_scale, 4)) return MS_ERR_ALIGN;
    if (dchannel_scale && !channel_scale) return MS_ERR_NULL;
    if (d->rows == 0) {
        cudaError_t e = cudaSuccess;
        for (float *p : {dweight, dchannel_scale})
            if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, (size_t)d->width * sizeof(float), st);
        return cuda_rc(e);
    }
    if (!residual_out || !dy || (dchannel_scale && !x)) return MS_ERR_NULL;
    const int es = elem_bytes(d->dtype), rs = elem_bytes(d->res_dtype);
    if (!aligned(residual_out, rs) || !aligned(dy, es) || !aligned(dresidual_out, rs) || !aligned(x, es) ||
        !aligned(dx, es) || !aligned(dresidual, rs) || !aligned(weight, 4) || !aligned(channel_scale, 4))
        return MS_ERR_ALIGN;
    if (dweight || dchannel_scale) {
        if (!workspace || workspace_bytes < mamba_residual_norm_bwd_workspace_size(d)) return MS_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return MS_ERR_ALIGN;
    }
    ms::ResidualNormArgs a = residual_args(d, weight, channel_scale, dev_status);
    a.res_out = const_cast<void *>(residual_out);
    a.dy = dy; a.dres_out = dresidual_out; a.x = x; a.dx = dx; a.dres = dresidual; a.dw = dweight; a.dcs = dchannel_scale;
    a.part = static_cast<float *>(workspace);
    return cuda_rc(ms::launch_residual_norm(a, d->dtype == MS_BF16, d->res_dtype == MS_BF16, true, num_sms_current(), st));
}

}  // extern "C"

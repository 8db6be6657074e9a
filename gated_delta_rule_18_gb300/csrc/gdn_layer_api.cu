// gdn_layer_api.cu -- the C entry points of the state-space layer's operators
// (include/gdn.h): host-side checks, workspace layout and dispatch.
#include "gdn_checks.cuh"
#include "gdn_launch.cuh"
#include "gdn_layer.cuh"
#include "gdn_ssm.cuh"

namespace {

using namespace gdn;

// the forward: the error word, and the chunks' sums where a line is cut
struct SsmWs {
    int nchunk, clen0, clen;
    size_t sums, dsum, total;
};
SsmWs ssm_ws(int lines, int T, int D, int N) {
    SsmWs L;
    ssm_split(lines, T, D, N, &L.nchunk, &L.clen0, &L.clen);
    const size_t items = (size_t)lines * (L.nchunk - 1);
    L.sums = kAlign;
    L.dsum = align_up(L.sums + items * D * ssm_np(N) * 4);
    L.total = align_up(L.dsum + items * D * 4);
    return L;
}
struct SsmBwdWs {
    int nrun, rlen, ngroup;
    size_t sums, dsum, gsum, gs, bc, a, d, total;
};
bool ssm_shape_ok(int B, int T, int D, int N, int n_seq, int varlen) {
    if (!dense_ok(B, T, D) || N < 1 || N > kSsmMaxN) return false;
    return varlen ? B == 1 && n_seq >= 1 : n_seq == B;
}
SsmBwdWs ssm_bwd_ws(int B, int T, int D, int N, int varlen) {
    SsmBwdWs L;
    const int lines = varlen ? 1 : B;
    L.rlen = ssm_bwd_run(lines, T, D, N);
    L.nrun = (T + L.rlen - 1) / L.rlen;
    L.ngroup = (T + kSsmGroup - 1) / kSsmGroup;
    const size_t groups = (size_t)lines * L.ngroup, runs = (size_t)lines * L.nrun, dnp = (size_t)D * ssm_np(N);
    size_t off = kAlign;
    auto take = [&](size_t floats) {
        const size_t at = off;
        off = align_up(off + floats * 4);
        return at;
    };
    L.sums = take(groups * dnp);
    L.dsum = take(groups * D);
    L.gsum = take(runs * D);
    L.gs = take(runs * dnp);
    L.bc = take((size_t)ssm_bwd_tiles(D, N) * B * T * 2 * N);
    L.a = take(runs * D * N);
    L.d = take(runs * 2 * D);
    L.total = off;
    return L;
}

}  // namespace

extern "C" {

gdn_status gdn_rmsnorm_fwd(const void *x, int64_t x_st, int x_dtype, const void *residual, int64_t res_st,
                           int res_dtype, const float *weight, void *out, int64_t out_st, int out_dtype,
                           void *res_out, int64_t res_out_st, float *scale, int R, int D, int group, float eps,
                           cudaStream_t stream) {
    if (R > 0 && (!x || !weight || !out)) return GDN_ERR_NULL;
    if (!norm_shape_ok(R, D) || !(eps >= 0.f)) return GDN_ERR_SHAPE;
    if (!dtype_ok(x_dtype) || (residual && !dtype_ok(res_dtype))) return GDN_ERR_DTYPE;
    if (out_dtype != GDN_E4M3 && out_dtype != x_dtype) return GDN_ERR_DTYPE;
    if (R > 0 && ((residual != nullptr) != (res_out != nullptr) || (out_dtype == GDN_E4M3) != (scale != nullptr)))
        return GDN_ERR_NULL;
    if (out_dtype == GDN_E4M3 && group != 0 && group != 32 && group != 64 && group != 128 && group != 256)
        return GDN_ERR_SHAPE;
    Rows r;
    r.add(x, x_dtype, 0, x_st);
    r.add(residual, res_dtype, 0, res_st);
    r.add(res_out, res_dtype, 0, res_out_st);
    r.add(out, out_dtype, 0, out_st, out_dtype == GDN_E4M3 ? 8 : 16);
    r.add(weight, GDN_F32, 0, 0);
    if (!r.ok || !f32_ok(scale)) return GDN_ERR_LAYOUT;
    if (R == 0) return GDN_OK;
    const int64_t groups = group > 0 ? ((int64_t)D + group - 1) / group : 1;
    const gdn_status a = areas_ok({Area(out, out_dtype, 0, out_st, 1, R, D), Area(res_out, res_dtype, 0, res_out_st, 1, R, D)},
                                  {Area(scale, GDN_F32, R * groups)},
                                  {Area(x, x_dtype, 0, x_st, 1, R, D), Area(residual, res_dtype, 0, res_st, 1, R, D)}, {});
    if (a != GDN_OK) return a;
    NormParams p{};
    p.x = x, p.res = residual, p.x_st = x_st, p.res_st = res_st;
    p.x_bf16 = x_dtype == GDN_BF16, p.res_bf16 = res_dtype == GDN_BF16;
    p.weight = weight, p.out = out, p.res_out = res_out, p.o_st = out_st, p.ro_st = res_out_st;
    p.scale = scale, p.R = R, p.D = D, p.group = group, p.eps = eps;
    p.vec = r.wide && D % 8 == 0;
    return cuda_status(launch(KNorm, stream, [&] { return launch_rmsnorm(p, stream); }));
}

size_t gdn_rmsnorm_bwd_workspace_size(int R, int D) {
    if (!norm_shape_ok(R, D)) return 0;
    return align_up((size_t)norm_bwd_parts(R, D) * D * 4) + kAlign;
}

gdn_status gdn_rmsnorm_bwd(const void *s, int64_t s_st, int s_dtype, const void *dy, int64_t dy_st, int dy_dtype,
                           const void *dres, int64_t dres_st, const float *weight, void *dx, int64_t dx_st,
                           float *dweight, int R, int D, float eps, void *workspace, size_t ws_bytes,
                           cudaStream_t stream) {
    if (!dweight || (R > 0 && (!s || !dy || !weight || !dx))) return GDN_ERR_NULL;
    if (!norm_shape_ok(R, D) || !(eps >= 0.f)) return GDN_ERR_SHAPE;
    if (!dtype_ok(s_dtype) || !dtype_ok(dy_dtype)) return GDN_ERR_DTYPE;
    Rows r;
    r.add(s, s_dtype, 0, s_st);
    r.add(dy, dy_dtype, 0, dy_st);
    r.add(dres, s_dtype, 0, dres_st);
    r.add(dx, s_dtype, 0, dx_st);
    r.add(weight, GDN_F32, 0, 0);
    if (!r.ok || !f32_ok(dweight)) return GDN_ERR_LAYOUT;
    const gdn_status a = areas_ok({Area(dx, s_dtype, 0, dx_st, 1, R, D)}, {Area(dweight, GDN_F32, D)},
                                  {Area(s, s_dtype, 0, s_st, 1, R, D), Area(dy, dy_dtype, 0, dy_st, 1, R, D),
                                   Area(dres, s_dtype, 0, dres_st, 1, R, D)}, {});
    if (a != GDN_OK) return a;
    if (!ws_ok(workspace, ws_bytes, gdn_rmsnorm_bwd_workspace_size(R, D))) return GDN_ERR_WORKSPACE;
    NormBwdParams p{};
    p.s = s, p.dy = dy, p.dres = dres, p.s_st = s_st, p.dy_st = dy_st, p.dr_st = dres_st;
    p.s_bf16 = s_dtype == GDN_BF16, p.dy_bf16 = dy_dtype == GDN_BF16;
    p.weight = weight, p.dx = dx, p.dx_st = dx_st, p.dweight = dweight;
    p.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + kAlign);
    p.R = R, p.D = D, p.eps = eps;
    p.vec = r.wide && D % 8 == 0;
    cudaError_t e = cudaSuccess;
    if (R > 0) e = launch(KNormBwd, stream, [&] { return launch_rmsnorm_bwd(p, stream); });
    if (e == cudaSuccess)
        e = launch(KColSum, stream, [&] {
            return launch_col_sum(p.part, D, R > 0 ? norm_bwd_parts(R, D) : 0, D, dweight, 0, nullptr, stream);
        });
    return cuda_status(e);
}

gdn_status gdn_conv_fwd(const void *x, int64_t x_sb, int64_t x_st, const float *weight, int W, const float *bias,
                        const void *initial_state, const int32_t *cu_seqlens, int n_seq, void *out, int64_t out_sb,
                        int64_t out_st, void *final_state, int B, int T, int D, int dtype, int flags,
                        void *workspace, size_t ws_bytes, cudaStream_t stream) {
    if (!weight || (T > 0 && (!x || !out))) return GDN_ERR_NULL;
    if (!batch_ok(B, T, D, cu_seqlens, n_seq) || W < 2 || W > kConvMaxW) return GDN_ERR_SHAPE;
    if (!dtype_ok(dtype)) return GDN_ERR_DTYPE;
    if (flags & ~GDN_SILU) return GDN_ERR_UNSUPPORTED;
    Rows r;
    r.add(x, dtype, x_sb, x_st);
    r.add(out, dtype, out_sb, out_st);
    r.add(initial_state, dtype, 0, D);
    r.add(final_state, dtype, 0, D);
    r.add(weight, GDN_F32, 0, 0);
    r.add(bias, GDN_F32, 0, 0);
    if (!r.ok || !f32_ok(cu_seqlens)) return GDN_ERR_LAYOUT;
    // (the inputs before a run of tokens are read by other threads than write there)
    const int64_t window = (int64_t)n_seq * (W - 1) * D;
    const gdn_status a = areas_ok({}, {Area(out, dtype, out_sb, out_st, B, T, D), Area(final_state, dtype, window)}, {},
                                  {Area(x, dtype, x_sb, x_st, B, T, D), Area(initial_state, dtype, window)});
    if (a != GDN_OK) return a;
    if (cu_seqlens && !ws_ok(workspace, ws_bytes, kAlign)) return GDN_ERR_WORKSPACE;
    if (T == 0 && !final_state && !cu_seqlens) return GDN_OK;
    ConvParams p{};
    p.x = x, p.x_sb = x_sb, p.x_st = x_st, p.weight = weight, p.bias = bias, p.init = initial_state;
    p.cu = cu_seqlens, p.n_seq = n_seq, p.out = out, p.o_sb = out_sb, p.o_st = out_st, p.final_state = final_state;
    p.B = B, p.T = T, p.D = D, p.W = W, p.silu = flags & GDN_SILU, p.bf16 = dtype == GDN_BF16;
    p.vec = r.wide && D % 8 == 0;
    p.err = cu_seqlens ? static_cast<int *>(workspace) : nullptr;
    return cuda_status(launch(KConv, stream, [&] { return launch_conv(p, stream); }));
}

size_t gdn_conv_bwd_workspace_size(int B, int T, int D, int W) {
    if (!dense_ok(B, T, D) || W < 2 || W > kConvMaxW) return 0;
    return align_up((size_t)conv_bwd_parts(B, T, conv_bwd_run(B, T, D)) * D * (W + 1) * 4) + kAlign;
}

gdn_status gdn_conv_bwd(const void *x, int64_t x_sb, int64_t x_st, const float *weight, int W, const float *bias,
                        const void *initial_state, const int32_t *cu_seqlens, int n_seq, const void *dout,
                        int64_t dout_sb, int64_t dout_st, const void *dfinal_state, void *dx, float *dweight,
                        float *dbias, void *dinitial_state, int B, int T, int D, int dtype, int flags,
                        void *workspace, size_t ws_bytes, cudaStream_t stream) {
    if (!weight || !dweight || (T > 0 && (!x || !dout || !dx))) return GDN_ERR_NULL;
    if (!batch_ok(B, T, D, cu_seqlens, n_seq) || W < 2 || W > kConvMaxW) return GDN_ERR_SHAPE;
    if (!dtype_ok(dtype)) return GDN_ERR_DTYPE;
    if (flags & ~GDN_SILU) return GDN_ERR_UNSUPPORTED;
    Rows r;
    r.add(x, dtype, x_sb, x_st);
    r.add(dout, dtype, dout_sb, dout_st);
    r.add(dx, dtype, 0, D);
    r.add(initial_state, dtype, 0, D);
    r.add(dfinal_state, dtype, 0, D);
    r.add(dinitial_state, dtype, 0, D);
    r.add(weight, GDN_F32, 0, 0);
    r.add(bias, GDN_F32, 0, 0);
    if (!r.ok || !f32_ok(cu_seqlens) || !f32_ok(dweight) || !f32_ok(dbias)) return GDN_ERR_LAYOUT;
    const int64_t window = (int64_t)n_seq * (W - 1) * D;
    const gdn_status a =
        areas_ok({}, {Area(dx, dtype, (int64_t)B * T * D), Area(dinitial_state, dtype, window),
                      Area(dweight, GDN_F32, (int64_t)D * W), Area(dbias, GDN_F32, D)}, {},
                 {Area(x, dtype, x_sb, x_st, B, T, D), Area(dout, dtype, dout_sb, dout_st, B, T, D),
                  Area(initial_state, dtype, window), Area(dfinal_state, dtype, window)});
    if (a != GDN_OK) return a;
    if (!ws_ok(workspace, ws_bytes, gdn_conv_bwd_workspace_size(B, T, D, W))) return GDN_ERR_WORKSPACE;
    ConvParams p{};
    p.x = x, p.x_sb = x_sb, p.x_st = x_st, p.weight = weight, p.bias = bias, p.init = initial_state;
    p.cu = cu_seqlens, p.n_seq = n_seq, p.dout = dout, p.do_sb = dout_sb, p.do_st = dout_st;
    p.dfinal = dfinal_state, p.dx = dx, p.dinit = dinitial_state, p.dweight = dweight, p.dbias = dbias;
    p.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + kAlign);
    p.B = B, p.T = T, p.D = D, p.W = W, p.silu = flags & GDN_SILU, p.bf16 = dtype == GDN_BF16;
    p.vec = r.wide && D % 8 == 0;
    p.err = cu_seqlens ? static_cast<int *>(workspace) : nullptr;
    cudaError_t e = cudaSuccess;
    if (T > 0 || cu_seqlens || dinitial_state)
        e = launch(KConvBwd, stream, [&] { return launch_conv_bwd(p, stream); });
    if (e == cudaSuccess)
        e = launch(KColSum, stream, [&] {
            return launch_col_sum(p.part, (int64_t)D * (W + 1), conv_bwd_parts(B, T, conv_bwd_run(B, T, D)),
                                  (int64_t)D * W, dweight,
                                  dbias ? D : 0, dbias, stream);
        });
    return cuda_status(e);
}

gdn_status gdn_conv_step(const void *x, int64_t x_st, const float *weight, int W, const float *bias, void *state,
                         const int32_t *slots, int n_slots, void *out, int64_t out_st, int n, int D, int dtype,
                         int flags, cudaStream_t stream) {
    if (n > 0 && (!x || !weight || !out || (n_slots > 0 && !state))) return GDN_ERR_NULL;
    if (n < 0 || n > 65535 || D < 1 || D > (1 << 20) || W < 2 || W > kConvMaxW || n_slots < 0 ||
        (!slots && n > n_slots))
        return GDN_ERR_SHAPE;
    if (!dtype_ok(dtype)) return GDN_ERR_DTYPE;
    if (flags & ~GDN_SILU) return GDN_ERR_UNSUPPORTED;
    Rows r;
    r.add(x, dtype, 0, x_st);
    r.add(out, dtype, 0, out_st);
    r.add(state, dtype, 0, D);
    r.add(weight, GDN_F32, 0, 0);
    r.add(bias, GDN_F32, 0, 0);
    if (!r.ok || !f32_ok(slots)) return GDN_ERR_LAYOUT;
    if (n == 0) return GDN_OK;
    const gdn_status a = areas_ok({Area(out, dtype, 0, out_st, 1, n, D)}, {Area(state, dtype, (int64_t)n_slots * (W - 1) * D)},
                                  {Area(x, dtype, 0, x_st, 1, n, D)}, {});
    if (a != GDN_OK) return a;
    ConvStepParams p{};
    p.x = x, p.x_st = x_st, p.weight = weight, p.bias = bias, p.state = state, p.slots = slots;
    p.out = out, p.o_st = out_st, p.n = n, p.n_slots = n_slots, p.D = D, p.W = W;
    p.silu = flags & GDN_SILU, p.bf16 = dtype == GDN_BF16;
    p.vec = r.wide && D % 8 == 0;
    return cuda_status(launch(KConvStep, stream, [&] { return launch_conv_step(p, stream); }));
}

}  // extern "C"

namespace {
// The checks and the parameter block gdn_ssm_fwd and gdn_ssm_bwd share.
gdn_status ssm_setup(const void *x, int64_t x_sb, int64_t x_st, const void *dt, int64_t dt_sb, int64_t dt_st,
                     const float *A, const void *bm, int64_t bm_sb, int64_t bm_st, const void *cm, int64_t cm_sb,
                     int64_t cm_st, const float *Dv, const void *z, int64_t z_sb, int64_t z_st,
                     const float *dt_bias, const float *h0, const int32_t *cu, int n_seq, int B, int T, int D, int N,
                     int dtype, int flags, Rows &r, SsmParams &p) {
    if (!A || (T > 0 && (!x || !dt || !bm || !cm))) return GDN_ERR_NULL;
    if (!ssm_shape_ok(B, T, D, N, n_seq, cu != nullptr)) return GDN_ERR_SHAPE;
    if (!dtype_ok(dtype)) return GDN_ERR_DTYPE;
    if (flags & ~GDN_SOFTPLUS) return GDN_ERR_UNSUPPORTED;
    r.add(x, dtype, x_sb, x_st);
    r.add(dt, dtype, dt_sb, dt_st);
    r.add(z, dtype, z_sb, z_st);
    Rows bc;  // (B, T, N) rows are staged by element where they are not wide
    bc.add(bm, dtype, bm_sb, bm_st, 4 * elem_size(dtype));
    bc.add(cm, dtype, cm_sb, cm_st, 4 * elem_size(dtype));
    if (!r.ok || !bc.ok) return GDN_ERR_LAYOUT;
    for (const void *f : {(const void *)A, (const void *)Dv, (const void *)dt_bias, (const void *)h0, (const void *)cu})
        if (!f32_ok(f)) return GDN_ERR_LAYOUT;
    p = SsmParams{};
    p.x = x, p.x_sb = x_sb, p.x_st = x_st, p.dt = dt, p.dt_sb = dt_sb, p.dt_st = dt_st;
    p.bm = bm, p.bm_sb = bm_sb, p.bm_st = bm_st, p.cm = cm, p.cm_sb = cm_sb, p.cm_st = cm_st;
    p.z = z, p.z_sb = z_sb, p.z_st = z_st, p.A = A, p.Dv = Dv, p.dt_bias = dt_bias, p.h0 = h0;
    p.cu = cu, p.n_seq = n_seq, p.B = B, p.T = T, p.D = D, p.N = N;
    p.softplus = flags & GDN_SOFTPLUS, p.bf16 = dtype == GDN_BF16;
    p.bc_vec = bc.wide && N % 4 == 0;
    p.n_wide = N % 4 == 0 && addr(A) % 16 == 0 && addr(h0) % 16 == 0;
    return GDN_OK;
}
}  // namespace

extern "C" {

size_t gdn_ssm_workspace_size(int B, int T, int D, int N, int n_seq, int varlen) {
    return ssm_shape_ok(B, T, D, N, n_seq, varlen) ? ssm_ws(varlen ? 1 : B, T, D, N).total : 0;
}

gdn_status gdn_ssm_fwd(const void *x, int64_t x_sb, int64_t x_st, const void *dt, int64_t dt_sb, int64_t dt_st,
                       const float *A, const void *bm, int64_t bm_sb, int64_t bm_st, const void *cm, int64_t cm_sb,
                       int64_t cm_st, const float *Dv, const void *z, int64_t z_sb, int64_t z_st,
                       const float *dt_bias, const float *h0, const int32_t *cu_seqlens, int n_seq, void *out,
                       int64_t out_sb, int64_t out_st, float *h_final, int B, int T, int D, int N, int dtype,
                       int flags, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    Rows r;
    SsmParams p;
    if (T > 0 && !out) return GDN_ERR_NULL;
    r.add(out, dtype, out_sb, out_st);
    const gdn_status s = ssm_setup(x, x_sb, x_st, dt, dt_sb, dt_st, A, bm, bm_sb, bm_st, cm, cm_sb, cm_st, Dv, z, z_sb,
                                   z_st, dt_bias, h0, cu_seqlens, n_seq, B, T, D, N, dtype, flags, r, p);
    if (s != GDN_OK) return s;
    if (!f32_ok(h_final)) return GDN_ERR_LAYOUT;
    const int64_t states = (int64_t)n_seq * D * N;
    const gdn_status a =
        areas_ok({Area(out, dtype, out_sb, out_st, B, T, D)}, {Area(h_final, GDN_F32, states)},
                 {Area(x, dtype, x_sb, x_st, B, T, D), Area(dt, dtype, dt_sb, dt_st, B, T, D), Area(z, dtype, z_sb, z_st, B, T, D)},
                 {Area(bm, dtype, bm_sb, bm_st, B, T, N), Area(cm, dtype, cm_sb, cm_st, B, T, N), Area(h0, GDN_F32, states)});
    if (a != GDN_OK) return a;
    const SsmWs L = ssm_ws(cu_seqlens ? 1 : B, T, D, N);
    if (!ws_ok(workspace, ws_bytes, L.total)) return GDN_ERR_WORKSPACE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    p.out = out, p.o_sb = out_sb, p.o_st = out_st, p.h_final = h_final;
    p.nchunk = L.nchunk, p.clen0 = L.clen0, p.clen = L.clen;
    p.sums = reinterpret_cast<float *>(ws + L.sums), p.dsum = reinterpret_cast<float *>(ws + L.dsum);
    p.err = cu_seqlens ? reinterpret_cast<int *>(ws) : nullptr;
    p.vec = r.wide && D % 8 == 0;
    p.n_wide = p.n_wide && addr(h_final) % 16 == 0;
    cudaError_t e = cudaSuccess;
    if (p.nchunk > 1) {
        e = launch(KSsmSum, stream, [&] { return launch_ssm_sum(p, stream); });
        if (e == cudaSuccess) e = launch(KSsmChain, stream, [&] { return launch_ssm_chain(p, stream); });
    }
    if (e == cudaSuccess) e = launch(KSsmScan, stream, [&] { return launch_ssm_scan(p, stream); });
    return cuda_status(e);
}

size_t gdn_ssm_bwd_workspace_size(int B, int T, int D, int N, int n_seq, int varlen) {
    if (!ssm_shape_ok(B, T, D, N, n_seq, varlen)) return 0;
    return ssm_bwd_ws(B, T, D, N, varlen).total;
}

gdn_status gdn_ssm_bwd(const void *x, int64_t x_sb, int64_t x_st, const void *dt, int64_t dt_sb, int64_t dt_st,
                       const float *A, const void *bm, int64_t bm_sb, int64_t bm_st, const void *cm, int64_t cm_sb,
                       int64_t cm_st, const float *Dv, const void *z, int64_t z_sb, int64_t z_st,
                       const float *dt_bias, const float *h0, const int32_t *cu_seqlens, int n_seq, const void *dout,
                       int64_t dout_sb, int64_t dout_st, const float *dh_final, void *dx, void *ddt, float *dA,
                       void *dbm, void *dcm, float *dD, void *dz, float *ddt_bias, float *dh0, int B, int T, int D,
                       int N, int dtype, int flags, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    Rows r;
    SsmParams p;
    if (!dA || (T > 0 && (!dout || !dx || !ddt || !dbm || !dcm))) return GDN_ERR_NULL;
    if (dz && !z) return GDN_ERR_NULL;
    r.add(dout, dtype, dout_sb, dout_st);
    r.add(dx, dtype, 0, D);
    r.add(ddt, dtype, 0, D);
    r.add(dz, dtype, 0, D);
    const gdn_status s = ssm_setup(x, x_sb, x_st, dt, dt_sb, dt_st, A, bm, bm_sb, bm_st, cm, cm_sb, cm_st, Dv, z, z_sb,
                                   z_st, dt_bias, h0, cu_seqlens, n_seq, B, T, D, N, dtype, flags, r, p);
    if (s != GDN_OK) return s;
    Rows g;
    g.add(dbm, dtype, 0, N);
    g.add(dcm, dtype, 0, N);
    if (!g.ok) return GDN_ERR_LAYOUT;
    for (const void *f : {(const void *)dh_final, (const void *)dA, (const void *)dD, (const void *)ddt_bias,
                          (const void *)dh0})
        if (!f32_ok(f)) return GDN_ERR_LAYOUT;
    const int64_t states = (int64_t)n_seq * D * N, rows = (int64_t)B * T;
    const gdn_status a =
        areas_ok({Area(dx, dtype, 0, D, 1, rows, D), Area(ddt, dtype, 0, D, 1, rows, D), Area(dz, dtype, 0, D, 1, rows, D)},
                 {Area(dbm, dtype, rows * N), Area(dcm, dtype, rows * N), Area(dA, GDN_F32, (int64_t)D * N),
                  Area(dD, GDN_F32, D), Area(ddt_bias, GDN_F32, D), Area(dh0, GDN_F32, states)},
                 {Area(x, dtype, x_sb, x_st, B, T, D), Area(dt, dtype, dt_sb, dt_st, B, T, D),
                  Area(z, dtype, z_sb, z_st, B, T, D), Area(dout, dtype, dout_sb, dout_st, B, T, D)},
                 {Area(bm, dtype, bm_sb, bm_st, B, T, N), Area(cm, dtype, cm_sb, cm_st, B, T, N),
                  Area(h0, GDN_F32, states), Area(dh_final, GDN_F32, states)});
    if (a != GDN_OK) return a;
    const SsmBwdWs L = ssm_bwd_ws(B, T, D, N, cu_seqlens != nullptr);
    if (!ws_ok(workspace, ws_bytes, L.total)) return GDN_ERR_WORKSPACE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    p.dout = dout, p.do_sb = dout_sb, p.do_st = dout_st, p.dh_final = dh_final;
    p.dx = dx, p.ddt = ddt, p.dbm = dbm, p.dcm = dcm, p.dz = dz;
    p.dA = dA, p.dD = dD, p.ddt_bias = ddt_bias, p.dh0 = dh0;
    auto at = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
    p.nrun = L.nrun, p.rlen = L.rlen, p.ngroup = L.ngroup;
    p.sums = at(L.sums), p.dsum = at(L.dsum), p.gsum = at(L.gsum), p.gs = at(L.gs);
    p.part_bc = at(L.bc), p.part_a = at(L.a), p.part_d = at(L.d);
    p.err = cu_seqlens ? reinterpret_cast<int *>(ws) : nullptr;
    p.vec = r.wide && D % 8 == 0;
    p.n_wide = p.n_wide && addr(dh_final) % 16 == 0 && addr(dh0) % 16 == 0;
    cudaError_t e = cudaSuccess;
    auto run = [&](int kind, cudaError_t (*f)(const SsmParams &, cudaStream_t)) {
        if (e == cudaSuccess) e = launch(kind, stream, [&] { return f(p, stream); });
    };
    if (L.ngroup > 1) {  // one group's entering state and gradient are h0 and dh_final
        run(KSsmBwdSum, launch_ssm_bwd_sum);
        run(KSsmBwdChain, launch_ssm_bwd_chain);
    }
    if (T > 0) run(KSsmBwd, launch_ssm_bwd);
    run(KSsmBwdReduce, launch_ssm_bwd_reduce);
    return cuda_status(e);
}

gdn_status gdn_ssm_step(const void *x, int64_t x_st, const void *dt, int64_t dt_st, const float *A, const void *bm,
                        int64_t bm_st, const void *cm, int64_t cm_st, const float *Dv, const void *z, int64_t z_st,
                        const float *dt_bias, float *state, const int32_t *slots, int n_slots, void *out,
                        int64_t out_st, int n, int D, int N, int dtype, int flags, cudaStream_t stream) {
    if (n > 0 && (!x || !dt || !A || !bm || !cm || !out || (n_slots > 0 && !state))) return GDN_ERR_NULL;
    if (n < 0 || n > 65535 || D < 1 || D > (1 << 20) || N < 1 || N > kSsmMaxN || n_slots < 0 ||
        (!slots && n > n_slots))
        return GDN_ERR_SHAPE;
    if (!dtype_ok(dtype)) return GDN_ERR_DTYPE;
    if (flags & ~GDN_SOFTPLUS) return GDN_ERR_UNSUPPORTED;
    Rows r;
    r.add(x, dtype, 0, x_st);
    r.add(dt, dtype, 0, dt_st);
    r.add(z, dtype, 0, z_st);
    r.add(out, dtype, 0, out_st);
    Rows bc;
    bc.add(bm, dtype, 0, bm_st, 4 * elem_size(dtype));
    bc.add(cm, dtype, 0, cm_st, 4 * elem_size(dtype));
    if (!r.ok || !bc.ok || !f32_ok(A) || !f32_ok(Dv) || !f32_ok(dt_bias) || !f32_ok(state) || !f32_ok(slots))
        return GDN_ERR_LAYOUT;
    if (n == 0) return GDN_OK;
    const gdn_status a =
        areas_ok({Area(out, dtype, 0, out_st, 1, n, D)}, {Area(state, GDN_F32, (int64_t)n_slots * D * N)},
                 {Area(x, dtype, 0, x_st, 1, n, D), Area(dt, dtype, 0, dt_st, 1, n, D), Area(z, dtype, 0, z_st, 1, n, D)},
                 {Area(bm, dtype, 0, bm_st, 1, n, N), Area(cm, dtype, 0, cm_st, 1, n, N)});
    if (a != GDN_OK) return a;
    SsmStepParams p{};
    p.x = x, p.dt = dt, p.bm = bm, p.cm = cm, p.z = z;
    p.x_st = x_st, p.dt_st = dt_st, p.bm_st = bm_st, p.cm_st = cm_st, p.z_st = z_st;
    p.A = A, p.Dv = Dv, p.dt_bias = dt_bias, p.state = state, p.slots = slots, p.out = out, p.o_st = out_st;
    p.n_wide = N % 4 == 0 && addr(A) % 16 == 0 && addr(state) % 16 == 0;
    p.bc_vec = bc.wide && N % 4 == 0;
    p.n = n, p.n_slots = n_slots, p.D = D, p.N = N, p.softplus = flags & GDN_SOFTPLUS, p.bf16 = dtype == GDN_BF16;
    return cuda_status(launch(KSsmStep, stream, [&] { return launch_ssm_step(p, stream); }));
}

}  // extern "C"

// gdn_block_api.cu -- the C entry points of the operators around a mixer and
// of the gated recurrence (include/gdn.h): host-side checks, workspace layout
// and dispatch.
#include <cfloat>
#include <utility>

#include "gdn_block.cuh"
#include "gdn_checks.cuh"
#include "gdn_launch.cuh"

namespace {

using namespace gdn;

// A (B, T, H, D) tensor: its bytes as rows of lines where its dimensions merge
// into two and a row, else the range that holds them (`hull`).
struct Heads {
    Area area;
    bool hull = false, apart = true;  // apart: no two rows share a byte
    static Heads of(const void *p, int dtype, int64_t sb, int64_t st, int64_t sh, int64_t B, int64_t T, int64_t H, int64_t D) {
        struct Dim {
            int64_t n, s;
        } d[3];
        int k = 0;
        if (B * T * H == 0) p = nullptr;
        for (const Dim &x : {Dim{B, sb}, Dim{T, st}, Dim{H, sh}})
            if (x.n > 1) d[k++] = x;
        for (int i = 0; i < k; ++i)
            for (int j = i + 1; j < k; ++j)
                if (d[j].s > d[i].s) std::swap(d[i], d[j]);
        int64_t row = D;
        while (k > 0 && d[k - 1].s == row) row *= d[--k].n;
        for (int i = 0; i + 1 < k;) {
            if (d[i].s == d[i + 1].n * d[i + 1].s) {
                d[i].n *= d[i + 1].n, d[i].s = d[i + 1].s;
                for (int j = i + 1; j + 1 < k; ++j) d[j] = d[j + 1];
                --k;
            } else {
                ++i;
            }
        }
        if (k <= 2) {
            const Dim one{1, 0};
            const Dim outer = k == 2 ? d[0] : one, inner = k ? d[k - 1] : one;
            Heads h{Area(p, dtype, outer.s, inner.s, outer.n, inner.n, row)};
            h.apart = rows_apart(h.area);
            return h;
        }
        int64_t span = row;
        bool nest = true;
        for (int i = k - 1; i >= 0; --i) nest = nest && d[i].s >= span, span += (d[i].n - 1) * d[i].s;
        Heads h{Area(p, dtype, 0, 0, 1, 1, span)};
        h.hull = true, h.apart = nest;
        return h;
    }
};

// rows that lie on 16 bytes, on words in pairs, or anywhere (LruParams::how)
struct LruLayout {
    Rows wide, words;
    void add(const void *p, int dtype, int64_t sb, int64_t st) { wide.add(p, dtype, sb, st), words.add(p, dtype, sb, st, 4); }
    bool ok() const { return wide.ok; }
    int how(int C, int dtype) const {
        if (wide.wide && C % 8 == 0) return 0;
        return words.wide && (dtype == GDN_F32 || C % 2 == 0) ? 1 : 2;
    }
};
struct LruWs {
    size_t ck, part, total;
};
LruWs lru_bwd_ws(int B, int T, int C, bool saved) {
    LruWs L;
    L.ck = kAlign;
    L.part = align_up(L.ck + (saved ? 0 : (size_t)B * ((T + kLruTile - 1) / kLruTile) * C * 4));
    L.total = align_up(L.part + (size_t)B * lru_bwd_ranks(B, T, C) * C * 4);
    return L;
}

bool gate_ok(const void *gate, int gate_rows, int act, int R) {
    if (act < GDN_GATE_NONE || act > GDN_GATE_SILU || (R > 0 && (act != GDN_GATE_NONE) != (gate != nullptr))) return false;
    if (gate_rows == 1) return true;
    return act != GDN_GATE_NONE && gate_rows > 1 && R % gate_rows == 0 && R / gate_rows <= 65535;
}

}  // namespace

extern "C" {

gdn_status gdn_rotary(const void *q, int64_t q_sb, int64_t q_st, int64_t q_sh, int Hq, void *q_out, int64_t qo_sb,
                      int64_t qo_st, int64_t qo_sh, const void *k, int64_t k_sb, int64_t k_st, int64_t k_sh, int Hk,
                      void *k_out, int64_t ko_sb, int64_t ko_st, int64_t ko_sh, const double *inv_freq,
                      const void *positions, int pos_bits, int64_t pos_sb, int64_t pos_st, int64_t offset, int B, int T,
                      int D, int rot, float scale, int dtype, int flags, cudaStream_t stream) {
    const bool with_k = k != nullptr || k_out != nullptr;
    const bool some = B > 0 && T > 0;
    if (some && (!q || !q_out || !inv_freq || (with_k && (!k || !k_out)))) return GDN_ERR_NULL;
    if (B < 0 || T < 0 || (int64_t)B * T > INT32_MAX - 65535 || Hq < 1 || (with_k ? Hk < 1 : Hk != 0)) return GDN_ERR_SHAPE;
    if (D < 1 || D > kRotaryMaxD || rot < 2 || rot % 2 || rot > D || Hq > 65535 || Hk > 65535) return GDN_ERR_SHAPE;
    if (!dtype_ok(dtype)) return GDN_ERR_DTYPE;
    if (positions && pos_bits != 32 && pos_bits != 64) return GDN_ERR_DTYPE;
    if (flags & ~(GDN_INTERLEAVED | GDN_INVERSE)) return GDN_ERR_UNSUPPORTED;
    Rows r;
    r.add(q, dtype, q_sb, q_st), r.add(q, dtype, q_sh, 0);
    r.add(q_out, dtype, qo_sb, qo_st), r.add(q_out, dtype, qo_sh, 0);
    r.add(k, dtype, k_sb, k_st), r.add(k, dtype, k_sh, 0);
    r.add(k_out, dtype, ko_sb, ko_st), r.add(k_out, dtype, ko_sh, 0);
    if (!r.ok || addr(inv_freq) % 8 || pos_sb < 0 || pos_st < 0) return GDN_ERR_LAYOUT;
    if (positions && addr(positions) % (pos_bits / 8)) return GDN_ERR_LAYOUT;
    if (!some) return GDN_OK;
    const Heads in[2] = {Heads::of(q, dtype, q_sb, q_st, q_sh, B, T, Hq, D), Heads::of(k, dtype, k_sb, k_st, k_sh, B, T, Hk, D)};
    const Heads out[2] = {Heads::of(q_out, dtype, qo_sb, qo_st, qo_sh, B, T, Hq, D),
                          Heads::of(k_out, dtype, ko_sb, ko_st, ko_sh, B, T, Hk, D)};
    const auto same = [&](int64_t a, int64_t b, int n) { return a == b || n == 1; };
    const bool at[2] = {q == q_out && same(q_sb, qo_sb, B) && same(q_st, qo_st, T) && same(q_sh, qo_sh, Hq),
                        k == k_out && same(k_sb, ko_sb, B) && same(k_st, ko_st, T) && same(k_sh, ko_sh, Hk)};
    for (int i = 0; i < 2; ++i) {
        if (!out[i].apart) return GDN_ERR_LAYOUT;
        for (int j = 0; j < 2; ++j)
            if (!(i == j && at[i]) && meet(out[i].area, in[j].area)) return GDN_ERR_UNSUPPORTED;
    }
    if (meet(out[0].area, out[1].area)) return GDN_ERR_UNSUPPORTED;
    RotaryParams p{};
    p.x[0] = RotaryTensor{q, q_out, q_sb, q_st, q_sh, qo_sb, qo_st, qo_sh, Hq, rot < D && !at[0]};
    if (with_k) p.x[1] = RotaryTensor{k, k_out, k_sb, k_st, k_sh, ko_sb, ko_st, ko_sh, Hk, rot < D && !at[1]};
    p.inv_freq = inv_freq, p.pos = positions, p.pos64 = pos_bits == 64, p.p_sb = pos_sb, p.p_st = pos_st, p.offset = offset;
    p.B = B, p.T = T, p.D = D, p.rot = rot, p.interleaved = flags & GDN_INTERLEAVED, p.bf16 = dtype == GDN_BF16;
    p.scale = scale, p.sign = flags & GDN_INVERSE ? -1.f : 1.f;
    const int v = 16 / elem_size(dtype);
    p.vec = r.wide && D % v == 0 && (p.interleaved ? rot : rot / 2) % v == 0;
    return cuda_status(launch(KRotary, stream, [&] { return launch_rotary(p, stream); }));
}

gdn_status gdn_block_norm_fwd(const void *y, int64_t y_st, int y_dtype, const void *residual, int64_t res_st,
                              int res_dtype, const void *gate, int64_t gate_st, int gate_rows, int act,
                              const float *post_weight, const float *pre_weight, const float *scale, float alpha,
                              void *res_out, int64_t res_out_st, void *out, int64_t out_st, int R, int D, float eps,
                              cudaStream_t stream) {
    if (R > 0 && (!y || !residual || !res_out || (!post_weight && !pre_weight) || (out != nullptr) != (pre_weight != nullptr)))
        return GDN_ERR_NULL;
    if (!norm_shape_ok(R, D) || !(eps >= 0.f) || !gate_ok(gate, gate_rows, act, R)) return GDN_ERR_SHAPE;
    if (!dtype_ok(y_dtype) || !dtype_ok(res_dtype)) return GDN_ERR_DTYPE;
    Rows r;
    r.add(y, y_dtype, 0, y_st);
    r.add(residual, res_dtype, 0, res_st);
    r.add(gate, y_dtype, 0, gate_st);
    r.add(res_out, res_dtype, 0, res_out_st);
    r.add(out, y_dtype, 0, out_st);
    for (const float *w : {post_weight, pre_weight, scale}) r.add(w, GDN_F32, 0, 0);
    if (!r.ok) return GDN_ERR_LAYOUT;
    if (R == 0) return GDN_OK;
    const Area ga(gate, y_dtype, 0, gate_st, 1, R / gate_rows, D), none(nullptr, y_dtype, 0);
    const gdn_status a =
        areas_ok({Area(res_out, res_dtype, 0, res_out_st, 1, R, D), Area(out, y_dtype, 0, out_st, 1, R, D)}, {},
                 {Area(y, y_dtype, 0, y_st, 1, R, D), Area(residual, res_dtype, 0, res_st, 1, R, D), gate_rows == 1 ? ga : none},
                 {gate_rows == 1 ? none : ga});
    if (a != GDN_OK) return a;
    BlockNormParams p{};
    p.y = y, p.res = residual, p.gate = gate, p.y_st = y_st, p.r_st = res_st, p.g_st = gate_st;
    p.post = post_weight, p.pre = pre_weight, p.scale = scale, p.res_out = res_out, p.out = out;
    p.ro_st = res_out_st, p.o_st = out_st, p.R = R, p.D = D, p.gate_rows = gate_rows, p.act = act;
    p.y_bf16 = y_dtype == GDN_BF16, p.r_bf16 = res_dtype == GDN_BF16, p.alpha = alpha, p.eps = eps;
    p.shared = gate_rows > 1;
    p.vec = r.wide && D % 8 == 0;
    return cuda_status(launch(KBlockNorm, stream, [&] { return launch_block_norm(p, stream); }));
}

size_t gdn_block_norm_bwd_workspace_size(int R, int D, int gate_rows) {
    if (!norm_shape_ok(R, D) || gate_rows < 1 || (gate_rows > 1 && (R % gate_rows || R / gate_rows > 65535))) return 0;
    const size_t row = (size_t)2 * D * 4;
    return align_up((size_t)block_norm_parts(R, D, gate_rows) * row) + (gate_rows > 1 ? align_up((size_t)(R / gate_rows) * row) : 0) + kAlign;
}

gdn_status gdn_block_norm_bwd(const void *y, int64_t y_st, int y_dtype, const void *s, int64_t s_st, int s_dtype,
                              const void *gate, int64_t gate_st, int gate_rows, int act, const void *dout,
                              int64_t dout_st, const void *dres, int64_t dres_st, const float *post_weight,
                              const float *pre_weight, const float *scale, float alpha, void *dy, int64_t dy_st,
                              void *dresidual, int64_t dresidual_st, void *dgate, int64_t dgate_st,
                              float *dpost_weight, float *dpre_weight, float *dscale, int R, int D, float eps,
                              void *workspace, size_t ws_bytes, cudaStream_t stream) {
    if (!post_weight && !pre_weight) return GDN_ERR_NULL;
    if (R > 0 && (!y || !dy || !dresidual || (gate && !dgate) || (pre_weight ? !s || !dout : !dres))) return GDN_ERR_NULL;
    if ((dpost_weight && !post_weight) || (dpre_weight && !pre_weight) || (dscale && !scale) || (dgate && !gate)) return GDN_ERR_NULL;
    if (!norm_shape_ok(R, D) || !(eps >= 0.f) || !gate_ok(gate, gate_rows, act, R)) return GDN_ERR_SHAPE;
    if (!dtype_ok(y_dtype) || !dtype_ok(s_dtype)) return GDN_ERR_DTYPE;
    const int64_t g_rows = R / gate_rows;
    if (!pre_weight) s = dout = nullptr;
    Rows r;
    r.add(y, y_dtype, 0, y_st);
    r.add(s, s_dtype, 0, s_st);
    r.add(gate, y_dtype, 0, gate_st);
    r.add(dout, y_dtype, 0, dout_st);
    r.add(dres, s_dtype, 0, dres_st);
    r.add(dy, y_dtype, 0, dy_st);
    r.add(dresidual, s_dtype, 0, dresidual_st);
    r.add(dgate, y_dtype, 0, dgate_st);
    for (const float *w : {post_weight, pre_weight, scale}) r.add(w, GDN_F32, 0, 0);
    if (!r.ok || !f32_ok(dpost_weight) || !f32_ok(dpre_weight) || !f32_ok(dscale)) return GDN_ERR_LAYOUT;
    const gdn_status a =
        areas_ok({}, {Area(dy, y_dtype, 0, dy_st, 1, R, D), Area(dresidual, s_dtype, 0, dresidual_st, 1, R, D),
                      Area(dgate, y_dtype, 0, dgate_st, 1, g_rows, D), Area(dpost_weight, GDN_F32, D),
                      Area(dpre_weight, GDN_F32, D), Area(dscale, GDN_F32, D)}, {},
                 {Area(y, y_dtype, 0, y_st, 1, R, D), Area(s, s_dtype, 0, s_st, 1, R, D),
                  Area(gate, y_dtype, 0, gate_st, 1, g_rows, D), Area(dout, y_dtype, 0, dout_st, 1, R, D),
                  Area(dres, s_dtype, 0, dres_st, 1, R, D), Area(post_weight, GDN_F32, D), Area(pre_weight, GDN_F32, D),
                  Area(scale, GDN_F32, D)});
    if (a != GDN_OK) return a;
    if (!ws_ok(workspace, ws_bytes, gdn_block_norm_bwd_workspace_size(R, D, gate_rows))) return GDN_ERR_WORKSPACE;
    BlockNormBwdParams p{};
    p.y = y, p.s = s, p.gate = gate, p.dout = dout, p.dres = dres;
    p.y_st = y_st, p.s_st = s_st, p.g_st = gate_st, p.do_st = dout_st, p.dr_st = dres_st;
    p.post = post_weight, p.pre = pre_weight, p.scale = scale, p.dy = dy, p.ds = dresidual, p.dgate = dgate;
    p.dy_st = dy_st, p.ds_st = dresidual_st, p.dg_st = dgate_st;
    p.dpost = dpost_weight, p.dpre = dpre_weight, p.dscale = dscale;
    p.R = R, p.D = D, p.gate_rows = gate_rows, p.act = act, p.y_bf16 = y_dtype == GDN_BF16, p.r_bf16 = s_dtype == GDN_BF16;
    p.shared = gate && gate_rows > 1 && R > 0, p.alpha = alpha, p.eps = eps;
    p.vec = r.wide && D % 8 == 0;
    unsigned char *ws = static_cast<unsigned char *>(workspace) + kAlign;
    p.part = reinterpret_cast<float *>(ws);
    p.part2 = reinterpret_cast<float *>(ws + align_up((size_t)block_norm_parts(R, D, gate_rows) * 2 * D * 4));
    cudaError_t e = cudaSuccess;
    if (R > 0) e = launch(KBlockNormBwd, stream, [&] { return launch_block_norm_bwd(p, stream); });
    if (e == cudaSuccess && R > 0 && block_norm_by_sequence(p))
        e = launch(KBlockNormSeq, stream, [&] { return launch_block_norm_sequences(p, stream); });
    if (e == cudaSuccess && (dpost_weight || dpre_weight || dscale || p.shared))
        e = launch(KBlockNormReduce, stream, [&] { return launch_block_norm_reduce(p, stream); });
    return cuda_status(e);
}

}  // extern "C"

namespace {
// The checks and the parameter block gdn_lru_fwd and gdn_lru_bwd share.
gdn_status lru_setup(const void *x, int64_t x_sb, int64_t x_st, const void *r, int64_t r_sb, int64_t r_st, const void *i,
                     int64_t i_sb, int64_t i_st, const float *lam, const void *z, int64_t z_sb, int64_t z_st, float c,
                     const float *h0, const int32_t *cu, int n_seq, int B, int T, int C, int dtype, LruLayout &rows, LruParams &p) {
    if (!lam || (T > 0 && (!x || !r || !i))) return GDN_ERR_NULL;
    if (!batch_ok(B, T, C, cu, n_seq) || !(c >= 0.f && c <= FLT_MAX)) return GDN_ERR_SHAPE;
    if (!dtype_ok(dtype)) return GDN_ERR_DTYPE;
    rows.add(x, dtype, x_sb, x_st);
    rows.add(r, dtype, r_sb, r_st);
    rows.add(i, dtype, i_sb, i_st);
    rows.add(z, dtype, z_sb, z_st);
    if (!rows.ok() || !f32_ok(lam) || !f32_ok(h0) || !f32_ok(cu)) return GDN_ERR_LAYOUT;
    p = LruParams{};
    p.x = x, p.x_sb = x_sb, p.x_st = x_st, p.r = r, p.r_sb = r_sb, p.r_st = r_st, p.i = i, p.i_sb = i_sb, p.i_st = i_st;
    p.lam = lam, p.z = z, p.z_sb = z_sb, p.z_st = z_st, p.c = c, p.h0 = h0, p.cu = cu, p.n_seq = n_seq;
    p.B = B, p.T = T, p.C = C, p.bf16 = dtype == GDN_BF16;
    p.first = 1, p.stall_cta = stall_test_set().cta.load();
    p.wait_us = p.stall_cta >= 0 ? stall_test_set().us.load() : 500000;
    return GDN_OK;
}
}  // namespace

extern "C" {

gdn_status gdn_lru_fwd(const void *x, int64_t x_sb, int64_t x_st, const void *r, int64_t r_sb, int64_t r_st,
                       const void *i, int64_t i_sb, int64_t i_st, const float *lam, const void *z, int64_t z_sb,
                       int64_t z_st, float c, const float *h0, const int32_t *cu_seqlens, int n_seq, void *out,
                       int64_t out_sb, int64_t out_st, float *h_final, float *checkpoints, int B, int T, int C,
                       int dtype, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    LruLayout rows;
    LruParams p;
    if (T > 0 && !out) return GDN_ERR_NULL;
    rows.add(out, dtype, out_sb, out_st);
    const gdn_status s = lru_setup(x, x_sb, x_st, r, r_sb, r_st, i, i_sb, i_st, lam, z, z_sb, z_st, c, h0, cu_seqlens, n_seq,
                                   B, T, C, dtype, rows, p);
    if (s != GDN_OK) return s;
    if (!f32_ok(h_final) || !f32_ok(checkpoints)) return GDN_ERR_LAYOUT;
    const int64_t states = (int64_t)n_seq * C, tiles = (T + kLruTile - 1) / kLruTile;
    const gdn_status a =
        areas_ok({Area(out, dtype, out_sb, out_st, B, T, C)}, {Area(h_final, GDN_F32, states), Area(checkpoints, GDN_F32, B * tiles * C)},
                 {Area(x, dtype, x_sb, x_st, B, T, C), Area(r, dtype, r_sb, r_st, B, T, C), Area(i, dtype, i_sb, i_st, B, T, C),
                  Area(z, dtype, z_sb, z_st, B, T, C)},
                 {Area(lam, GDN_F32, C), Area(h0, GDN_F32, states)});
    if (a != GDN_OK) return a;
    if (cu_seqlens && !ws_ok(workspace, ws_bytes, kAlign)) return GDN_ERR_WORKSPACE;
    if (T == 0 && !h_final && !cu_seqlens) return GDN_OK;
    p.out = out, p.o_sb = out_sb, p.o_st = out_st, p.h_final = h_final, p.ck = checkpoints;
    p.how = rows.how(C, dtype);
    const LruShape shape = lru_shape(B, T, C, p.bf16, p.how == 0);
    p.ranks = shape.ranks, p.warps = shape.warps;
    p.err = ws_ok(workspace, ws_bytes, kAlign) ? static_cast<int *>(workspace) : nullptr;
    return cuda_status(launch(KLru, stream, [&] { return launch_lru(p, stream); }));
}

size_t gdn_lru_bwd_workspace_size(int B, int T, int C, int with_checkpoints) {
    return dense_ok(B, T, C) ? lru_bwd_ws(B, T, C, with_checkpoints != 0).total : 0;
}

gdn_status gdn_lru_bwd(const void *x, int64_t x_sb, int64_t x_st, const void *r, int64_t r_sb, int64_t r_st,
                       const void *i, int64_t i_sb, int64_t i_st, const float *lam, const void *z, int64_t z_sb,
                       int64_t z_st, float c, const float *h0, const int32_t *cu_seqlens, int n_seq, const void *dout,
                       int64_t dout_sb, int64_t dout_st, const float *dh_final, const float *checkpoints, void *dx,
                       void *dr, void *di, float *dlam, void *dz, float *dh0, int B, int T, int C, int dtype,
                       void *workspace, size_t ws_bytes, cudaStream_t stream) {
    LruLayout rows;
    LruParams p;
    if (!dlam || (T > 0 && (!dout || !dx || !dr || !di || (z && !dz)))) return GDN_ERR_NULL;
    if ((dz && !z) || (dh0 && !h0)) return GDN_ERR_NULL;
    rows.add(dout, dtype, dout_sb, dout_st);
    for (const void *d : {dx, dr, di, dz}) rows.add(d, dtype, 0, C);
    const gdn_status s = lru_setup(x, x_sb, x_st, r, r_sb, r_st, i, i_sb, i_st, lam, z, z_sb, z_st, c, h0, cu_seqlens, n_seq,
                                   B, T, C, dtype, rows, p);
    if (s != GDN_OK) return s;
    if (!f32_ok(dh_final) || !f32_ok(checkpoints) || !f32_ok(dlam) || !f32_ok(dh0)) return GDN_ERR_LAYOUT;
    const int64_t states = (int64_t)n_seq * C, n = (int64_t)B * T * C, tiles = (T + kLruTile - 1) / kLruTile;
    const gdn_status a =
        areas_ok({}, {Area(dx, dtype, n), Area(dr, dtype, n), Area(di, dtype, n), Area(dz, dtype, n), Area(dlam, GDN_F32, C),
                      Area(dh0, GDN_F32, states)}, {},
                 {Area(x, dtype, x_sb, x_st, B, T, C), Area(r, dtype, r_sb, r_st, B, T, C), Area(i, dtype, i_sb, i_st, B, T, C),
                  Area(z, dtype, z_sb, z_st, B, T, C), Area(dout, dtype, dout_sb, dout_st, B, T, C), Area(lam, GDN_F32, C),
                  Area(h0, GDN_F32, states), Area(dh_final, GDN_F32, states), Area(checkpoints, GDN_F32, B * tiles * C)});
    if (a != GDN_OK) return a;
    const LruWs L = lru_bwd_ws(B, T, C, checkpoints != nullptr);
    if (!ws_ok(workspace, ws_bytes, L.total)) return GDN_ERR_WORKSPACE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    p.err = reinterpret_cast<int *>(ws);
    p.how = rows.how(C, dtype);
    cudaError_t e = cudaSuccess;
    p.ck = const_cast<float *>(checkpoints);
    if (!checkpoints && T > 0) {  // the states that enter the tiles, by a forward pass without outputs
        p.ck = reinterpret_cast<float *>(ws + L.ck);
        LruParams f = p;
        f.z = nullptr;
        const LruShape shape = lru_shape(B, T, C, p.bf16, p.how == 0);
        f.ranks = shape.ranks, f.warps = shape.warps;
        e = launch(KLru, stream, [&] { return launch_lru(f, stream); });
        p.first = 0;
    }
    p.dout = dout, p.do_sb = dout_sb, p.do_st = dout_st, p.dh_final = dh_final;
    p.dx = dx, p.dr = dr, p.di = di, p.dz = dz, p.dlam = dlam, p.dh0 = dh0;
    p.part = reinterpret_cast<float *>(ws + L.part);
    p.ranks = lru_bwd_ranks(B, T, C);
    if (e == cudaSuccess) e = launch(KLruBwd, stream, [&] { return launch_lru_bwd(p, stream); });
    if (e == cudaSuccess)
        e = launch(KColSum, stream, [&] { return launch_col_sum(p.part, C, B * p.ranks, C, dlam, 0, nullptr, stream); });
    return cuda_status(e);
}

void gdn_set_lru_cluster(int most) { set_lru_cluster(most); }

gdn_status gdn_lru_step(const void *x, int64_t x_st, const void *r, int64_t r_st, const void *i, int64_t i_st,
                        const float *lam, const void *z, int64_t z_st, float c, float *state, const int32_t *slots,
                        int n_slots, void *out, int64_t out_st, int n, int C, int dtype, cudaStream_t stream) {
    if (n > 0 && (!x || !r || !i || !lam || !out || (n_slots > 0 && !state))) return GDN_ERR_NULL;
    if (n < 0 || n > 65535 || C < 1 || C > (1 << 20) || n_slots < 0 || (!slots && n > n_slots) || !(c >= 0.f && c <= FLT_MAX))
        return GDN_ERR_SHAPE;
    if (!dtype_ok(dtype)) return GDN_ERR_DTYPE;
    Rows rows;  // four channels a thread
    const int bytes = 4 * elem_size(dtype);
    rows.add(x, dtype, 0, x_st, bytes);
    rows.add(r, dtype, 0, r_st, bytes);
    rows.add(i, dtype, 0, i_st, bytes);
    rows.add(z, dtype, 0, z_st, bytes);
    rows.add(out, dtype, 0, out_st, bytes);
    rows.add(state, GDN_F32, 0, C);
    rows.add(lam, GDN_F32, 0, 0);
    if (!rows.ok || !f32_ok(slots)) return GDN_ERR_LAYOUT;
    if (n == 0) return GDN_OK;
    const gdn_status a =
        areas_ok({Area(out, dtype, 0, out_st, 1, n, C)}, {Area(state, GDN_F32, (int64_t)n_slots * C)},
                 {Area(x, dtype, 0, x_st, 1, n, C), Area(r, dtype, 0, r_st, 1, n, C), Area(i, dtype, 0, i_st, 1, n, C),
                  Area(z, dtype, 0, z_st, 1, n, C)}, {Area(lam, GDN_F32, C)});
    if (a != GDN_OK) return a;
    LruStepParams p{};
    p.x = x, p.x_st = x_st, p.r = r, p.r_st = r_st, p.i = i, p.i_st = i_st, p.lam = lam, p.z = z, p.z_st = z_st, p.c = c;
    p.state = state, p.slots = slots, p.out = out, p.o_st = out_st, p.n = n, p.n_slots = n_slots, p.C = C;
    p.bf16 = dtype == GDN_BF16, p.vec = rows.wide && C % 4 == 0;
    return cuda_status(launch(KLruStep, stream, [&] { return launch_lru_step(p, stream); }));
}

}  // extern "C"

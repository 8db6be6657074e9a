// gdn_lru_bwd.cu -- the gradient of the gated linear recurrence. With s =
// silu(z) (1 without z) and q = 1 - a^2, backwards along each sequence:
//   g_t = dout_t s_t + a_{t+1} g_{t+1}          (+ dh_final at its end)
//   dx = g sqrt(q) sigmoid(i),   di = g b (1 - sigmoid(i)),  b = sqrt(q) sigmoid(i) x
//   w  = u g (a^2 b / q - a h_{t-1})            (u times the gradient of u)
//   dr = w (1 - sigmoid(r)),     dlam = sum w . sigmoid(lam) / softplus(lam)
//   dz = dout h silu'(z),        dh0 = a_0 g_0.
// b / q = sigmoid(i) x / sqrt(q) grows without bound as u -> 0, and u times it
// goes to 0 with sqrt(u): both are formed with 1 / sqrt(q) and meet no 0 / 0.
//
// The same tiles, clusters and joins as the forward, from the line's end. The
// states inside a tile are formed again from the state that enters it, which
// the forward saved (one in 64 tokens), so the line is read once here too.
#include "gdn_lru.cuh"

namespace gdn {
namespace {

constexpr int kRanks = 8;

struct Exchange {
    LruRun fwd[2][kLruWarps][32];  // A, H of a warp's tokens
    f32x2 back[2][kLruWarps][32];  // what they add to the gradient before them
    LruRun ranks[2][kRanks][32];
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kLruWarps, 2) lru_bwd_kernel(const LruParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Exchange ex;
    constexpr int KW = RowVec<T, 2>::kWords, kRow = kLruCh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int K = p.ranks, rank = K > 1 ? blockIdx.x % K : 0, line = blockIdx.y;
    const int c0 = (blockIdx.x / K) * kLruCh, c = c0 + 2 * lane, nc = p.C - c;
    if (p.err && blockIdx.x == 0 && blockIdx.y == 0) ssm_check_cu(p.cu, p.n_seq, p.T, p.err);
    auto ld_state = [&](const float *s, int64_t row) {
        float2 f = make_float2(0.f, 0.f);
        if (s && nc > 0) f.x = s[row * p.C + c];
        if (s && nc > 1) f.y = s[row * p.C + c + 1];
        return pack2(f.x, f.y);
    };
    auto st_state = [&](float *s, int64_t row, f32x2 v) {
        const float2 f = unpack2(v);
        if (nc > 0) s[row * p.C + c] = f.x;
        if (nc > 1) s[row * p.C + c + 1] = f.y;
    };
    if (p.dh0 && rank == 0) {  // of sequences without tokens
        if (!p.cu) {
            if (p.T == 0 && warp == 0) st_state(p.dh0, line, ld_state(p.dh_final, line));
        } else {
            for (int s = warp; s < p.n_seq; s += kLruWarps)
                if (p.cu[s + 1] <= p.cu[s]) st_state(p.dh0, s, ld_state(p.dh_final, s));
        }
    }
    const int steps = (p.T + K * kLruTile - 1) / (K * kLruTile), tiles = (p.T + kLruTile - 1) / kLruTile;
    const T *x = (const T *)p.x + line * p.x_sb, *r = (const T *)p.r + line * p.r_sb, *in = (const T *)p.i + line * p.i_sb;
    const T *z = p.z ? (const T *)p.z + line * p.z_sb : nullptr, *dout = (const T *)p.dout + line * p.do_sb;
    constexpr int kTensor = kLruLen * kRow;
    T *stage = (T *)smem + warp * 5 * kTensor;
    constexpr int kStage = kLruWarps * 5 * kTensor;  // elements of a stage
    auto first = [&](int n) { return ((steps - 1 - n) * K + rank) * kLruTile + warp * kLruLen; };
    auto fetch = [&](int n) {
        if constexpr (VEC) {
            if (n < steps) {
                const int t = first(n), rows = min(max(p.T - t, 0), kLruLen);
                T *s = stage + (n & 1) * kStage;
                if (rows > 0) {
                    lru_copy(s, x + t * p.x_st, p.x_st, rows, c0, p.C);
                    lru_copy(s + kTensor, r + t * p.r_st, p.r_st, rows, c0, p.C);
                    lru_copy(s + 2 * kTensor, in + t * p.i_st, p.i_st, rows, c0, p.C);
                    lru_copy(s + 3 * kTensor, dout + t * p.do_st, p.do_st, rows, c0, p.C);
                    if (z) lru_copy(s + 4 * kTensor, z + t * p.z_st, p.z_st, rows, c0, p.C);
                }
            }
            cp_async_commit();
        }
    };
    fetch(0);
    float cl[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (k < nc) cl[k] = lru_decay(p.lam[c + k], p.c);
    const f32x2 cl2 = pack2(cl[0], cl[1]), one = pack2(1.f, 1.f), zero = pack2(0.f, 0.f);
    f32x2 carry = zero;  // a g of the token behind the cluster's tiles
    f32x2 dlam = zero;
    if (K > 1) cluster_arrive(), cluster_wait();
    for (int n = 0; n < steps; ++n) {
        const int t0 = first(n), len = min(max(p.T - t0, 0), kLruLen), flip = n & 1, tile = (steps - 1 - n) * K + rank;
        const LruMarks m = lru_marks(p.cu, p.n_seq, p.T, t0);
        f32x2 h = tile < tiles ? ld_state(p.ck, (int64_t)line * tiles + tile) : zero;
        __syncwarp();  // every lane has read what the next copies overwrite
        fetch(n + 1);
        if constexpr (VEC) {
            cp_async_wait<1>();
            __syncwarp();
        }
        const T *staged = stage + flip * kStage;
        // a pair of tensor k (x, r, i, dout, z) at token j of the warp
        auto get = [&](int k, int j) -> f32x2 {
            uint32_t w[KW] = {};
            if constexpr (VEC) {
                ld_words(w, staged + k * kTensor + j * kRow + 2 * lane);
            } else if (nc > 0) {
                const int64_t t = t0 + j;
                const T *at = k == 0 ? x + t * p.x_st : k == 1 ? r + t * p.r_st : k == 2 ? in + t * p.i_st
                              : k == 3 ? dout + t * p.do_st : z + t * p.z_st;
                ld_row<T, 2, false>(w, at + c, nc);
            }
            return lru_pair<T>(w);
        };
        f32x2 a[kLruLen], b[kLruLen], gd[kLruLen];
        LruRun run{one, zero};
#pragma unroll
        for (int j = 0; j < kLruLen; ++j) {
            a[j] = one, b[j] = gd[j] = zero;
            if (j >= len) continue;
            const LruGate g(get(1, j), get(2, j), cl2);
            a[j] = g.a, b[j] = mul2(mul2(g.beta(), g.gi), get(0, j));
            gd[j] = get(3, j);
            if (z) {
                const float2 v = unpack2(get(4, j)), s = sigmoid2(v);
                gd[j] = mul2(gd[j], pack2(v.x * s.x, v.y * s.y));
            }
            if (m.fin >> j & 1 && p.dh_final)
                gd[j] = add2(gd[j], ld_state(p.dh_final, lru_seq(p.cu, p.n_seq, p.T, line, t0 + j)));
            if (m.cut >> j & 1) {
                if (p.h0) b[j] = fma2(a[j], ld_state(p.h0, lru_seq(p.cu, p.n_seq, p.T, line, t0 + j)), b[j]);
                run.A = pack2(-0.f, -0.f), run.H = b[j];
            } else {
                run.A = mul2(run.A, a[j]), run.H = fma2(a[j], run.H, b[j]);
            }
        }
        f32x2 back = zero;
#pragma unroll
        for (int j = kLruLen - 1; j >= 0; --j) {
            if (j < len) back = m.cut >> j & 1 ? zero : mul2(a[j], add2(gd[j], back));
        }
        ex.fwd[flip][warp][lane] = run, ex.back[flip][warp][lane] = back;
        __syncthreads();
        // the state before this warp's tokens; the CTA's run backwards and the part behind this warp
        LruRun all{one, zero}, behind = all;
#pragma unroll
        for (int w = 0; w < kLruWarps; ++w) {
            if (w < warp) {
                const LruRun v = ex.fwd[flip][w][lane];
                h = lru_apply2(v.A, v.H, h);
            }
        }
#pragma unroll
        for (int w = kLruWarps - 1; w >= 0; --w) {
            if (w == warp) behind = all;
            const f32x2 A = ex.fwd[flip][w][lane].A;
            all.H = lru_apply2(A, ex.back[flip][w][lane], all.H), all.A = lru_join(all.A, A);
        }
        f32x2 gm = carry;  // a g of the token behind this one
        if (K > 1) {
            if (warp < K) st_cluster(&ex.ranks[flip][rank][lane], warp, all);
            cluster_arrive(), cluster_wait();
            for (int k = K - 1; k >= 0; --k) {
                const LruRun v = ex.ranks[flip][k][lane];
                if (k == rank) gm = carry;
                carry = lru_apply2(v.A, v.H, carry);
            }
        } else {
            carry = lru_apply2(all.A, all.H, carry);
        }
        gm = lru_apply2(behind.A, behind.H, gm);
        const f32x2 h_in = h;
#pragma unroll
        for (int j = 0; j < kLruLen; ++j) {  // b becomes h
            if (j >= len) break;
            h = b[j] = m.cut >> j & 1 ? b[j] : fma2(a[j], h, b[j]);
        }
        const int64_t at0 = ((int64_t)line * p.T + t0) * p.C + c;
#pragma unroll
        for (int j = kLruLen - 1; j >= 0; --j) {
            if (j >= len) continue;
            const f32x2 xv = get(0, j), g = add2(gd[j], gm);
            const LruGate gt(get(1, j), get(2, j), cl2);
            f32x2 prev = j > 0 ? b[j > 0 ? j - 1 : 0] : h_in;
            const f32x2 ag = mul2(a[j], g);
            gm = ag;
            if (m.cut >> j & 1) {
                const int seq = lru_seq(p.cu, p.n_seq, p.T, line, t0 + j);
                prev = ld_state(p.h0, seq);
                if (p.dh0) st_state(p.dh0, seq, ag);
                gm = zero;
            }
            const float2 q = unpack2(gt.q);
            const f32x2 rs = pack2(rsqrt_approx(fmaxf(q.x, 1e-37f)), rsqrt_approx(fmaxf(q.y, 1e-37f)));
            const f32x2 beta = mul2(gt.q, rs), gbi = mul2(mul2(g, beta), gt.gi), ix = mul2(gt.gi, xv);
            const f32x2 di = mul2(mul2(gbi, xv), fma2(gt.gi, pack2(-1.f, -1.f), one));
            // u g (a^2 i x / sqrt(q) - a prev)
            const f32x2 in_term = mul2(mul2(gt.u, rs), mul2(a[j], ix));
            const f32x2 w = mul2(ag, fma2(mul2(gt.u, pack2(-1.f, -1.f)), prev, in_term));
            const f32x2 dr = mul2(w, fma2(gt.gr, pack2(-1.f, -1.f), one));
            dlam = add2(dlam, w);
            if (nc <= 0) continue;
            const int64_t at = at0 + (int64_t)j * p.C;
            auto put = [&](void *to, f32x2 v) {
                const float2 f = unpack2(v);
                const float o[2] = {f.x, f.y};
                st_row_f<T, 2, VEC>((T *)to + at, o, nc);
            };
            put(p.dx, gbi), put(p.di, di), put(p.dr, dr);
            if (z) {
                const float2 v = unpack2(get(4, j)), s = sigmoid2(v), d = unpack2(mul2(get(3, j), b[j]));
                put(p.dz, pack2(d.x * (s.x + v.x * s.x * (1.f - s.x)), d.y * (s.y + v.y * s.y * (1.f - s.y))));
            }
        }
    }
    // the channels' sums over the warps, in one order
    __syncthreads();
    f32x2 *sums = &ex.back[0][0][0];
    sums[warp * 32 + lane] = dlam;
    __syncthreads();
    if (warp == 0 && nc > 0) {
#pragma unroll
        for (int w = 1; w < kLruWarps; ++w) dlam = add2(dlam, sums[w * 32 + lane]);
        const float2 f = unpack2(dlam);
        float o[2] = {f.x, f.y};
        for (int k = 0; k < 2; ++k) {
            if (k >= nc) break;
            const float lam = p.lam[c + k];  // sigmoid / softplus goes to 1
            if (lam > -15.f || lam != lam) o[k] *= sigmoid2(make_float2(lam, lam)).x / softplus2(make_float2(lam, lam)).x;
            p.part[((int64_t)line * K + rank) * p.C + c + k] = o[k];
        }
    }
}

}  // namespace

cudaError_t launch_lru_bwd(const LruParams &p, cudaStream_t st) {
    using bf = __nv_bfloat16;
    const void *k = p.bf16 ? (p.vec ? (const void *)lru_bwd_kernel<bf, true> : (const void *)lru_bwd_kernel<bf, false>)
                           : (p.vec ? (const void *)lru_bwd_kernel<float, true> : (const void *)lru_bwd_kernel<float, false>);
    const int smem = p.vec ? 2 * 5 * kLruTile * kLruCh * (p.bf16 ? 2 : 4) : 0;
    return lru_launch(k, p.B, p.C, p.ranks, smem, p, st);
}

}  // namespace gdn

// gdn_block_norm.cu -- what stands between two blocks: the norm behind a
// block, its gate and residual scale, the residual's addition and the norm in
// front of the next block, in one pass over the rows, and its gradient. Per row
// of D channels, with k = alpha scale and f = act(gate):
//   u = y inv_y post  (y without post),  inv_y = 1 / sqrt(mean(y^2) + eps)
//   s = residual + k f u,  out = s inv_s pre.
// Gradient, for dout and the stream's own gradient dres, at s as stored:
//   ds = dres + N'(s; pre) dout,  dy = N'(y; post) (k f ds)
//   dgate = k u act'(gate) ds,    dpre = sum dout s inv_s
//   dpost = k sum ds f y inv_y,   dscale = alpha post sum ds f y inv_y:
// the last two are one sum. A gate row that the tokens of a sequence share
// takes sum ds y inv_y by sequence, of which the other sum is made too.
//
// Bound by HBM: every tensor is read once and written once; a row belongs to
// tpr threads of one CTA, 8 channels a vector, and both of its reductions
// cross warps through shared memory. Sums and norms are fp32.
#include "gdn_block.cuh"
#include "gdn_ssm.cuh"

namespace gdn {
namespace {

constexpr int kVecN = 8, kPairs = kVecN / 2;

struct RowShape {
    int tpr, nv, rpb;  // threads a row, vectors a thread, rows a CTA
};
RowShape row_shape(int D) {
    const int vecs = (D + kVecN - 1) / kVecN;
    RowShape s;
    s.tpr = 32;
    while (s.tpr < 512 && s.tpr < vecs) s.tpr *= 2;
    s.nv = 1;
    while (s.nv * s.tpr < vecs) s.nv *= 2;
    s.rpb = s.tpr >= 128 ? 1 : 128 / s.tpr;
    return s;
}

template <typename T>
__device__ __forceinline__ void to_pairs(f32x2 (&v)[kPairs], const uint32_t (&w)[RowVec<T, kVecN>::kWords]) {
    float f[kVecN];
    words_to_f<T, kVecN>(f, w);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) v[i] = pack2(f[2 * i], f[2 * i + 1]);
}
template <typename T, bool VEC>
__device__ __forceinline__ void put(T *p, const f32x2 (&v)[kPairs], int n) {
    float f[kVecN];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const float2 x = unpack2(v[i]);
        f[2 * i] = x.x, f[2 * i + 1] = x.y;
    }
    st_row_f<T, kVecN, VEC>(p, f, n);
}
// n > 0 channels of a row; `other` without one
template <typename T, bool VEC>
__device__ __forceinline__ void get(f32x2 (&v)[kPairs], const T *p, int n, float other = 0.f) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) v[i] = pack2(other, other);
        return;
    }
    uint32_t w[RowVec<T, kVecN>::kWords];
    ld_row<T, kVecN, VEC>(w, p, n);
    to_pairs<T>(v, w);
}
// alpha scale post, what multiplies y inv_y f
template <bool VEC>
__device__ __forceinline__ void get_factor(f32x2 (&k)[kPairs], const float *scale, const float *post, float alpha, int c, int n) {
    f32x2 s[kPairs];
    get<float, VEC>(s, scale ? scale + c : nullptr, n, 1.f);
    get<float, VEC>(k, post ? post + c : nullptr, n, 1.f);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) k[j] = mul2(mul2(pack2(alpha, alpha), s[j]), k[j]);
}

__device__ __forceinline__ float2 sigmoid_nan(float2 x) {  // sigmoid2 passes a NaN over
    const float2 g = sigmoid2(x);
    return make_float2(x.x != x.x ? x.x : g.x, x.y != x.y ? x.y : g.y);
}
__device__ __forceinline__ f32x2 gate_of(f32x2 g, int act) {
    if (act == kGateLinear) return g;
    const float2 x = unpack2(g), s = sigmoid_nan(x);
    if (act == kGateSigmoid) return pack2(s.x, s.y);
    return pack2(x.x * s.x, x.y * s.y);
}
// the factor and its derivative
__device__ __forceinline__ f32x2 gate_of(f32x2 g, int act, f32x2 &d) {
    d = pack2(1.f, 1.f);
    if (act == kGateLinear) return g;
    const float2 x = unpack2(g), s = sigmoid_nan(x);
    if (act == kGateSigmoid) {
        d = pack2(s.x * (1.f - s.x), s.y * (1.f - s.y));
        return pack2(s.x, s.y);
    }
    const float2 f = make_float2(x.x * s.x, x.y * s.y);
    d = pack2(s.x + f.x * (1.f - s.x), s.y + f.y * (1.f - s.y));
    return pack2(f.x, f.y);
}

// sums of N values over a row's warps; red: N rows of 16 floats, one a warp
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[16], int tpr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (tpr == 32) return;
    const int warp = threadIdx.x >> 5, wpr = tpr >> 5, w0 = warp & ~(wpr - 1);
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) red[k][warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (wpr == 2) {
            v[k] = red[k][w0] + red[k][w0 + 1];
        } else {
            v[k] = 0.f;
            for (int i = 0; i < wpr; i += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(red[k] + w0 + i);
                v[k] += (f.x + f.y) + (f.z + f.w);
            }
        }
    }
}

// One CTA walks rows blockIdx, blockIdx + grid, ...; PRE: the next row's loads
// are issued before this row's sums are known, and the weights stay in
// registers. Above 8192 channels they do not fit and are read again a row.
template <typename TX, typename TR, int NV, bool VEC>
__global__ void __launch_bounds__(512) block_norm_kernel(const BlockNormParams p, int tpr) {
    __shared__ __align__(16) float red[2][2][1][16];
    constexpr int WX = RowVec<TX, kVecN>::kWords, WR = RowVec<TR, kVecN>::kWords;
    constexpr bool PRE = NV <= 2;
    const int rpb = blockDim.x / tpr, lr = threadIdx.x / tpr, tid = threadIdx.x - lr * tpr;
    const int64_t step = (int64_t)gridDim.x * rpb;
    int64_t row = (int64_t)blockIdx.x * rpb + lr;
    uint32_t ny[NV][WX], ng[NV][WX], nr[NV][WR];
    auto fetch = [&](int64_t r) {
        const int64_t gr = p.gate_rows > 1 ? r / p.gate_rows : r;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
#pragma unroll
            for (int j = 0; j < WX; ++j) ny[i][j] = ng[i][j] = 0u;
#pragma unroll
            for (int j = 0; j < WR; ++j) nr[i][j] = 0u;
            if (r < p.R && c < p.D) {
                ld_row<TX, kVecN, VEC>(ny[i], (const TX *)p.y + r * p.y_st + c, p.D - c);
                ld_row<TR, kVecN, VEC>(nr[i], (const TR *)p.res + r * p.r_st + c, p.D - c);
                if (p.act) ld_row<TX, kVecN, VEC>(ng[i], (const TX *)p.gate + gr * p.g_st + c, p.D - c);
            }
        }
    };
    fetch(row);
    f32x2 w1[PRE ? NV : 1][kPairs], w2[PRE ? NV : 1][kPairs];
    auto weights = [&](int i, int at) {
        const int c = (i * tpr + tid) * kVecN;
        if (c < p.D) {
            get_factor<VEC>(w1[at], p.scale, p.post, p.alpha, c, p.D - c);
            get<float, VEC>(w2[at], p.pre ? p.pre + c : nullptr, p.D - c);
        }
    };
    if (PRE) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) w1[i][j] = w2[i][j] = pack2(0.f, 0.f);
            weights(i, i);
        }
    }
    const float rd = 1.f / (float)p.D;
    int flip = 0;
    // every thread of the CTA makes the same number of turns
    for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < p.R; r0 += step, row += step, flip ^= 1) {
        const bool live = row < p.R;
        f32x2 s[NV][kPairs];
        float inv = 1.f;
        if (p.post) {
            f32x2 sum2 = pack2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                to_pairs<TX>(s[i], ny[i]);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) sum2 = fma2(s[i][j], s[i][j], sum2);
            }
            const float2 su = unpack2(sum2);
            float v[1] = {su.x + su.y};
            row_sums<1>(v, red[flip][0], tpr);
            inv = rsqrtf(v[0] * rd + p.eps);
        }
        const f32x2 inv2 = pack2(inv, inv);
        f32x2 sum2 = pack2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
            f32x2 g[kPairs], r[kPairs];
            const int at = PRE ? i : 0;
            if (!PRE) weights(i, 0);
            to_pairs<TX>(s[i], ny[i]);
            to_pairs<TX>(g, ng[i]);
            to_pairs<TR>(r, nr[i]);
            if (!(live && c < p.D)) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) s[i][j] = pack2(0.f, 0.f);
                continue;
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                f32x2 v = mul2(mul2(s[i][j], inv2), w1[at][j]);
                if (p.act) v = mul2(v, gate_of(g[j], p.act));
                s[i][j] = add2(r[j], v);
            }
            put<TR, VEC>((TR *)p.res_out + row * p.ro_st + c, s[i], p.D - c);
            // (channels past D hold zeros: their factors and residuals are loaded as zeros)
#pragma unroll
            for (int j = 0; j < kPairs; ++j) sum2 = fma2(s[i][j], s[i][j], sum2);
        }
        if (PRE) fetch(row + step);
        if (p.pre) {
            const float2 su = unpack2(sum2);
            float v[1] = {su.x + su.y};
            row_sums<1>(v, red[flip][1], tpr);
            const float q = rsqrtf(v[0] * rd + p.eps);
            const f32x2 q2 = pack2(q, q);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * tpr + tid) * kVecN;
                if (!(live && c < p.D)) continue;
                if (!PRE) weights(i, 0);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) s[i][j] = mul2(mul2(s[i][j], q2), w2[PRE ? i : 0][j]);
                put<TX, VEC>((TX *)p.out + row * p.o_st + c, s[i], p.D - c);
            }
        }
        if (!PRE) fetch(row + step);
    }
}

// The gradient of a norm at channel pair x for the weighted gradient gw = w dy,
// with S = sum x^2, G = sum gw x, inv: both sums lose the channel's own terms
// first, which cancel exactly (they are all there is when one channel
// dominates its row).
struct NormGrad {
    float S, G, k, ke, inv;
    __device__ __forceinline__ NormGrad(float S_, float G_, float rd, float eps) : S(S_), G(G_) {
        inv = rsqrtf(S * rd + eps);
        k = inv * inv * rd, ke = eps * inv * inv;
    }
    __device__ __forceinline__ f32x2 at(f32x2 x, f32x2 gw) const {
        const float2 f = unpack2(x), g = unpack2(gw);
        const f32x2 so = pack2(__fsub_rn(S, __fmul_rn(f.x, f.x)), __fsub_rn(S, __fmul_rn(f.y, f.y)));
        const f32x2 go = pack2(__fsub_rn(__fmul_rn(g.x, f.x), G), __fsub_rn(__fmul_rn(g.y, f.y), G));
        const f32x2 rest = fma2(gw, so, mul2(x, go));
        return mul2(pack2(inv, inv), fma2(pack2(k, k), rest, mul2(pack2(ke, ke), gw)));
    }
};

// A CTA walks a run of one sequence's rows (blockIdx.y; all rows are one where
// no gate is shared). A thread keeps its channels' sums, in registers with one
// vector a thread (rows of up to 4096 channels), else in its own slots of
// shared memory, where it also reads its row again instead of holding it.
template <typename TX, typename TR, int NV, bool VEC>
__global__ void __launch_bounds__(512) block_norm_bwd_kernel(const BlockNormBwdParams p, int tpr) {
    __shared__ __align__(16) float red[2][4][16];
    extern __shared__ __align__(16) f32x2 kept[];  // [NV][2][kPairs][threads]
    constexpr bool HOLD = NV == 1;
    const int rpb = blockDim.x / tpr, lr = threadIdx.x / tpr, tid = threadIdx.x - lr * tpr;
    const int64_t rows = p.shared ? p.gate_rows : p.R, first = (int64_t)blockIdx.y * rows;
    const int64_t r_end = first + rows, run0 = first + (int64_t)blockIdx.x * p.run;
    const int64_t run1 = run0 + p.run < r_end ? run0 + p.run : r_end;
    f32x2 hy[kPairs], hs[kPairs], hd[kPairs], hg[kPairs], hr[kPairs], w1[kPairs], w2[kPairs], sa[kPairs], sr[kPairs];
    auto slot = [&](int i, int q, int j) -> f32x2 & { return kept[((i * 2 + q) * kPairs + j) * blockDim.x + threadIdx.x]; };
    auto zero = [&](f32x2 (&v)[kPairs]) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) v[j] = pack2(0.f, 0.f);
    };
    auto weights = [&](int c) {
        get_factor<VEC>(w1, p.scale, p.post, p.alpha, c, p.D - c);
        get<float, VEC>(w2, p.pre ? p.pre + c : nullptr, p.D - c);
    };
    zero(w1), zero(w2), zero(sa), zero(sr);
    if constexpr (HOLD) {
        if (tid * kVecN < p.D) weights(tid * kVecN);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < kPairs; ++j) slot(i, 0, j) = slot(i, 1, j) = pack2(0.f, 0.f);
    }
    auto take = [&](int64_t row, int c) {  // a vector of every input
        const int n = p.D - c;
        const int64_t gr = p.gate_rows > 1 ? row / p.gate_rows : row;
        get<TX, VEC>(hy, (const TX *)p.y + row * p.y_st + c, n);
        get<TX, VEC>(hg, p.act ? (const TX *)p.gate + gr * p.g_st + c : nullptr, n);
        get<TR, VEC>(hr, p.dres ? (const TR *)p.dres + row * p.dr_st + c : nullptr, n);
        if (p.pre) {
            get<TR, VEC>(hs, (const TR *)p.s + row * p.s_st + c, n);
            get<TX, VEC>(hd, (const TX *)p.dout + row * p.do_st + c, n);
        }
    };
    const float rd = 1.f / (float)p.D;
    int flip = 0;
    for (int64_t r0 = run0; r0 < run1; r0 += rpb, flip ^= 1) {
        const int64_t row = r0 + lr;
        const bool live = row < run1;
        float v[3] = {0.f, 0.f, 0.f};  // of s^2, pre dout s, y^2
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
            if (!(live && c < p.D)) continue;
            take(row, c);
            if (!HOLD) weights(c);
            f32x2 a = pack2(0.f, 0.f), b = a, d = a;
            if (p.pre) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j)
                    a = fma2(hs[j], hs[j], a), b = fma2(mul2(hd[j], w2[j]), hs[j], b);
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j) d = fma2(hy[j], hy[j], d);
            const float2 fa = unpack2(a), fb = unpack2(b), fd = unpack2(d);
            v[0] += fa.x + fa.y, v[1] += fb.x + fb.y, v[2] += fd.x + fd.y;
        }
        row_sums<3>(v, red[flip], tpr);
        const NormGrad ns(v[0], v[1], rd, p.eps);
        const float inv_y = p.post ? rsqrtf(v[2] * rd + p.eps) : 1.f;
        const f32x2 iy2 = pack2(inv_y, inv_y), is2 = pack2(ns.inv, ns.inv);
        f32x2 ds[kPairs], e[kPairs];
        auto stream = [&](int j) {  // ds, and e = k post f ds
            ds[j] = hr[j];
            if (p.pre) ds[j] = add2(ns.at(hs[j], mul2(hd[j], w2[j])), hr[j]);
        };
        float ge[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
            if (!(live && c < p.D)) continue;
            if (!HOLD) take(row, c), weights(c);
            f32x2 g2 = pack2(0.f, 0.f), dg[kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                stream(j);
                const f32x2 yn = mul2(hy[j], iy2);
                f32x2 f = pack2(1.f, 1.f), df = f;
                if (p.act) f = gate_of(hg[j], p.act, df);
                const f32x2 dsf = mul2(ds[j], f);
                e[j] = mul2(dsf, w1[j]);
                dg[j] = mul2(mul2(mul2(ds[j], w1[j]), yn), df);
                g2 = fma2(e[j], hy[j], g2);
                const f32x2 add = mul2(p.shared ? ds[j] : dsf, yn);
                if constexpr (HOLD) {
                    sa[j] = add2(sa[j], add);
                    if (p.pre) sr[j] = fma2(hd[j], mul2(hs[j], is2), sr[j]);
                } else {
                    slot(i, 0, j) = add2(slot(i, 0, j), add);
                    if (p.pre) slot(i, 1, j) = fma2(hd[j], mul2(hs[j], is2), slot(i, 1, j));
                }
            }
            const float2 fg = unpack2(g2);
            ge[0] += fg.x + fg.y;
            put<TR, VEC>((TR *)p.ds + row * p.ds_st + c, ds, p.D - c);
            if (p.act && !p.shared) put<TX, VEC>((TX *)p.dgate + row * p.dg_st + c, dg, p.D - c);
        }
        if (p.post) row_sums<1>(ge, red[flip] + 3, tpr);
        const NormGrad ny(v[2], ge[0], rd, p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
            if (!(live && c < p.D)) continue;
            if constexpr (!HOLD) {
                take(row, c), weights(c);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    stream(j);
                    e[j] = mul2(p.act ? mul2(ds[j], gate_of(hg[j], p.act)) : ds[j], w1[j]);
                }
            }
            if (p.post) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) e[j] = ny.at(hy[j], e[j]);
            }
            put<TX, VEC>((TX *)p.dy + row * p.dy_st + c, e, p.D - c);
        }
    }
    float *part = p.part + (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * rpb + lr) * 2 * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + tid) * kVecN;
        if (c >= p.D) continue;
        if constexpr (!HOLD) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) sa[j] = slot(i, 0, j), sr[j] = slot(i, 1, j);
        }
        put<float, VEC>(part + c, sa, p.D - c);
        put<float, VEC>(part + p.D + c, sr, p.D - c);
    }
}

// Sums over the runs, 32 columns a CTA, Y threads a column, in a fixed order.
template <int Y>
__device__ __forceinline__ float2 column_sums(const float *in, int64_t parts, int D, int c, float (*red)[33][2]) {
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    float a = 0.f, b = 0.f;
    if (c < D) {
#pragma unroll 4
        for (int64_t q = y; q < parts; q += Y) a += in[q * 2 * D + c], b += in[q * 2 * D + D + c];
    }
    red[y][x][0] = a, red[y][x][1] = b;
    __syncthreads();
    if (y == 0) {
#pragma unroll
        for (int i = 1; i < Y; ++i) a += red[i][x][0], b += red[i][x][1];
    }
    return make_float2(a, b);
}
constexpr int kSumY = 16;
// of one sequence (blockIdx.y): its gate row's gradient, and its share of the sums
template <typename TX>
__global__ void __launch_bounds__(32 * kSumY) block_norm_sequences_kernel(const BlockNormBwdParams p, int parts) {
    __shared__ float red[kSumY][33][2];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31);
    const int64_t q = blockIdx.y;
    const float2 v = column_sums<kSumY>(p.part + q * parts * 2 * p.D, parts, p.D, c, red);
    if (threadIdx.x >= 32 || c >= p.D) return;
    const float g = (float)((const TX *)p.gate)[q * p.g_st + c];
    f32x2 df2;
    const float2 f = unpack2(gate_of(pack2(g, g), p.act, df2));
    const float w = p.alpha * (p.scale ? p.scale[c] : 1.f) * (p.post ? p.post[c] : 1.f);
    ((TX *)p.dgate)[q * p.dg_st + c] = to_type<TX>(v.x * w * unpack2(df2).x);
    p.part2[q * 2 * p.D + c] = v.x * f.x;
    p.part2[q * 2 * p.D + p.D + c] = v.y;
}
__global__ void __launch_bounds__(32 * kSumY) block_norm_reduce_kernel(const BlockNormBwdParams p, const float *in, int64_t parts) {
    __shared__ float red[kSumY][33][2];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31);
    const float2 v = column_sums<kSumY>(in, parts, p.D, c, red);
    if (threadIdx.x >= 32 || c >= p.D) return;
    if (p.dpost) p.dpost[c] = v.x * (p.alpha * (p.scale ? p.scale[c] : 1.f));
    if (p.dscale) p.dscale[c] = v.x * (p.alpha * (p.post ? p.post[c] : 1.f));
    if (p.dpre) p.dpre[c] = v.y;
}

template <typename TX, typename TR>
cudaError_t norm_nv(const BlockNormParams &p, cudaStream_t st) {
    const RowShape s = row_shape(p.D);
    const unsigned nt = s.tpr * s.rpb, need = (unsigned)((p.R + s.rpb - 1) / s.rpb);
    const unsigned most = 152 * (1024 / nt), grid = need < most ? need : most;
    auto run = [&](auto vec) {
        constexpr bool V = decltype(vec)::value;
        if (s.nv == 1) block_norm_kernel<TX, TR, 1, V><<<grid, nt, 0, st>>>(p, s.tpr);
        else if (s.nv == 2) block_norm_kernel<TX, TR, 2, V><<<grid, nt, 0, st>>>(p, s.tpr);
        else block_norm_kernel<TX, TR, 4, V><<<grid, nt, 0, st>>>(p, s.tpr);
    };
    if (p.vec) run(std::true_type());
    else run(std::false_type());
    return cudaGetLastError();
}
template <typename TX, typename TR>
cudaError_t norm_bwd_nv(const BlockNormBwdParams &p, cudaStream_t st) {
    const RowShape s = row_shape(p.D);
    const unsigned nt = s.tpr * s.rpb;
    const dim3 grid(p.runs, p.shared ? p.R / p.gate_rows : 1);
    auto run = [&](auto nv, auto vec) -> cudaError_t {
        auto *k = block_norm_bwd_kernel<TX, TR, nv(), vec()>;
        const int smem = nv() > 1 ? nv() * 2 * kPairs * 8 * nt : 0;
        if (smem > 40 * 1024) {  // 48 KB with the static part
            const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
        }
        k<<<grid, nt, smem, st>>>(p, s.tpr);
        return cudaGetLastError();
    };
    auto by_vectors = [&](auto vec) {
        if (s.nv == 1) return run(std::integral_constant<int, 1>(), vec);
        if (s.nv == 2) return run(std::integral_constant<int, 2>(), vec);
        return run(std::integral_constant<int, 4>(), vec);
    };
    return p.vec ? by_vectors(std::true_type()) : by_vectors(std::false_type());
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormParams &p, cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (p.y_bf16) return p.r_bf16 ? norm_nv<bf, bf>(p, st) : norm_nv<bf, float>(p, st);
    return p.r_bf16 ? norm_nv<float, bf>(p, st) : norm_nv<float, float>(p, st);
}

// Runs of a sequence's rows: about 608 CTAs in all (four a SM where they fit).
void block_norm_runs(int R, int D, int gate_rows, int *runs, int *run, int64_t *parts) {
    const RowShape s = row_shape(D);
    const int rows = gate_rows > 1 ? gate_rows : R, n = gate_rows > 1 ? R / gate_rows : 1;
    const int most = n < 608 ? 608 / n : 1, need = (int)(((int64_t)rows + s.rpb - 1) / s.rpb);
    const int want = need < most ? need : most;
    *run = want > 0 ? (need + want - 1) / want * s.rpb : s.rpb;
    *runs = (int)(((int64_t)rows + *run - 1) / *run);
    *parts = (int64_t)n * *runs * s.rpb;
}

cudaError_t launch_block_norm_bwd(const BlockNormBwdParams &p, cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (p.y_bf16) return p.r_bf16 ? norm_bwd_nv<bf, bf>(p, st) : norm_bwd_nv<bf, float>(p, st);
    return p.r_bf16 ? norm_bwd_nv<float, bf>(p, st) : norm_bwd_nv<float, float>(p, st);
}

cudaError_t launch_block_norm_sequences(const BlockNormBwdParams &p, cudaStream_t st) {
    const RowShape s = row_shape(p.D);
    const dim3 grid((p.D + 31) / 32, p.R / p.gate_rows);
    if (p.y_bf16) block_norm_sequences_kernel<__nv_bfloat16><<<grid, 32 * kSumY, 0, st>>>(p, p.runs * s.rpb);
    else block_norm_sequences_kernel<float><<<grid, 32 * kSumY, 0, st>>>(p, p.runs * s.rpb);
    return cudaGetLastError();
}

cudaError_t launch_block_norm_reduce(const BlockNormBwdParams &p, cudaStream_t st) {
    const RowShape s = row_shape(p.D);
    const int64_t parts = p.R == 0 ? 0 : p.shared ? p.R / p.gate_rows : (int64_t)p.runs * s.rpb;
    block_norm_reduce_kernel<<<(p.D + 31) / 32, 32 * kSumY, 0, st>>>(p, p.shared ? p.part2 : p.part, parts);
    return cudaGetLastError();
}

}  // namespace gdn

// gdn_norm.cu -- root-mean-square norm over rows of D channels, with the
// residual's addition in front and an optional 8-bit output, and its
// gradient. With s = x + residual (fp32):
//   inv = 1 / sqrt(mean(s^2) + eps),  y = s inv w,  residual_out = s
//   8 bits: per group of channels (or per row) scale = max|y| / 448 and
//   q = e4m3(y / scale), q = 0 where scale = 0.
// Gradient, for dy and the residual stream's own gradient dres:
//   ds = inv w dy - s inv^3 mean(w dy s) + dres,  dw = sum over rows dy s inv.
//
// Both are bound by HBM: every input is read once and held in registers
// (a row belongs to tpr threads of one CTA, 8 channels a vector, nv vectors
// a thread), the row's sum crosses warps once through shared memory, and the
// result is written once. Sums, the norm and the scales are fp32.
#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr int kVecN = 8;

// maximum that keeps NaN, as the comparison with a NaN has to show in the scale
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// two fp32 to two e4m3 (round to nearest even, finite values saturate)
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// y / scale for one scale. An IEEE division costs some ten instructions a
// value; one reciprocal and a correction of the quotient by its remainder
// round the same (|y| <= 448 scale (1 + 2^-24), no intermediate overflows
// unless the scale itself is out of range, where the plain quotient is taken).
__device__ __forceinline__ void quantise(float (&y)[kVecN], float scale) {
    const float dv = scale == 0.f ? 1.f : scale, r = 1.f / dv;
    const bool safe = dv > 1e-30f && dv < 1e30f;
#pragma unroll
    for (int j = 0; j < kVecN; ++j) {
        const float q = y[j] * r;
        y[j] = safe ? fmaf(fmaf(-q, dv, y[j]), r, q) : y[j] / dv;
    }
}

// Threads a row and vectors a thread: one vector a thread up to 512 threads.
struct RowShape {
    int tpr, nv, rpb;
};
RowShape row_shape(int D, int max_tpr) {
    const int vecs = (D + kVecN - 1) / kVecN;
    RowShape s;
    s.tpr = 32;
    while (s.tpr < max_tpr && s.tpr < vecs) s.tpr *= 2;
    s.nv = 1;
    while (s.nv * s.tpr < vecs) s.nv *= 2;
    s.rpb = s.tpr >= 128 ? 1 : 128 / s.tpr;
    return s;
}

// the row's sum (or NaN-keeping maximum) over its warps; red: a float a warp
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float *red, int tpr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? max_nan(v, u) : v + u;
    }
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, wpr = tpr >> 5, w0 = warp & ~(wpr - 1);
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    v = red[w0];
    for (int i = 1; i < wpr; ++i) v = MAX ? max_nan(v, red[w0 + i]) : v + red[w0 + i];
    return v;
}

// One CTA walks rows blockIdx, blockIdx + grid, ..., the weights in registers.
// PRE: the next row's loads are issued before this row's sum is known.
template <typename TX, typename TR, bool Q8, int NV, bool VEC, bool PRE>
__global__ void __launch_bounds__(512) rmsnorm_kernel(const NormParams p, int tpr) {
    __shared__ float red[2][2][16];
    constexpr int WX = RowVec<TX, kVecN>::kWords, WR = RowVec<TR, kVecN>::kWords;
    const int rpb = blockDim.x / tpr, lr = threadIdx.x / tpr, tid = threadIdx.x - lr * tpr;
    const int64_t step = (int64_t)gridDim.x * rpb;
    int64_t row = (int64_t)blockIdx.x * rpb + lr;
    uint32_t nx[NV][WX], nr[NV][WR];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
#pragma unroll
            for (int j = 0; j < WX; ++j) nx[i][j] = 0u;
#pragma unroll
            for (int j = 0; j < WR; ++j) nr[i][j] = 0u;
            if (r < p.R && c < p.D) {
                ld_row<TX, kVecN, VEC>(nx[i], (const TX *)p.x + r * p.x_st + c, p.D - c);
                if (p.res) ld_row<TR, kVecN, VEC>(nr[i], (const TR *)p.res + r * p.res_st + c, p.D - c);
            }
        }
    };
    fetch(row);
    float w[NV][kVecN];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + tid) * kVecN;
#pragma unroll
        for (int j = 0; j < kVecN; ++j) w[i][j] = 0.f;
        if (c < p.D) ld_row_f<float, kVecN, VEC>(w[i], p.weight + c, p.D - c);
    }
    const int groups = p.group > 0 ? (p.D + p.group - 1) / p.group : 1;
    int flip = 0;
    // every thread of the CTA makes the same number of turns
    for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < p.R; r0 += step, row += step, flip ^= 1) {
        const bool live = row < p.R;
        float s[NV][kVecN];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
            words_to_f<TX, kVecN>(s[i], nx[i]);
            if (p.res) {
                float r[kVecN];
                words_to_f<TR, kVecN>(r, nr[i]);
#pragma unroll
                for (int j = 0; j < kVecN; ++j) s[i][j] += r[j];
                if (live && c < p.D) st_row_f<TR, kVecN, VEC>((TR *)p.res_out + row * p.ro_st + c, s[i], p.D - c);
            }
        }
        if (PRE) fetch(row + step);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < kVecN; ++j) sum = fmaf(s[i][j], s[i][j], sum);
        sum = row_reduce<false>(sum, red[flip][0], tpr);
        const float inv = rsqrtf(sum / (float)p.D + p.eps);
        float row_max = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
            const bool in = live && c < p.D;
#pragma unroll
            for (int j = 0; j < kVecN; ++j) s[i][j] = s[i][j] * inv * w[i][j];
            if constexpr (!Q8) {
                if (in) st_row_f<TX, kVecN, VEC>((TX *)p.out + row * p.o_st + c, s[i], p.D - c);
            } else {
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < kVecN; ++j) m = max_nan(m, fabsf(s[i][j]));
                row_max = max_nan(row_max, m);
                if (p.group > 0) {
                    // a group's vectors sit in group / 8 neighbouring lanes
                    for (int o = p.group / kVecN / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const float sc = m / 448.f;
                    if (in && c % p.group == 0) p.scale[row * groups + c / p.group] = sc;
                    quantise(s[i], sc);
                }
            }
        }
        if constexpr (Q8) {
            if (p.group == 0) {
                const float sc = row_reduce<true>(row_max, red[flip][1], tpr) / 448.f;
                if (live && tid == 0) p.scale[row] = sc;
#pragma unroll
                for (int i = 0; i < NV; ++i) quantise(s[i], sc);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * tpr + tid) * kVecN;
                if (!(live && c < p.D)) continue;
                uint32_t q[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    q[j] = pack_e4m3(s[i][4 * j], s[i][4 * j + 1]) | pack_e4m3(s[i][4 * j + 2], s[i][4 * j + 3]) << 16;
                uint8_t *o = (uint8_t *)p.out + row * p.o_st + c;
                if constexpr (VEC) {
                    st_words(o, q);
                } else {
#pragma unroll
                    for (int j = 0; j < kVecN; ++j)
                        if (c + j < p.D) o[j] = (uint8_t)(q[j >> 2] >> (8 * (j & 3)));
                }
            }
        }
        if (!PRE) fetch(row + step);
    }
}

// One CTA walks rows blockIdx, blockIdx + grid, ...; a thread keeps its
// channels' share of dw and writes it once, so dw is summed in a fixed order.
// A channel's own terms cancel exactly between the two parts of ds (they are
// all there is when one channel dominates its row), so both sums lose them
// first: with S = sum s^2, G = sum w dy s,
//   ds_i = inv [ inv^2 / D (w dy_i (S - s_i^2) - s_i (G - w dy_i s_i)) + eps inv^2 w dy_i ].
// PRE: the next row's loads are issued before this row's sum is known.
template <typename TS, typename TY, int NV, bool VEC, bool PRE>
__global__ void __launch_bounds__(512) rmsnorm_bwd_kernel(const NormBwdParams p, int tpr) {
    __shared__ float red[2][2][16];
    constexpr int WS = RowVec<TS, kVecN>::kWords, WY = RowVec<TY, kVecN>::kWords;
    const int rpb = blockDim.x / tpr;
    const int lr = threadIdx.x / tpr, tid = threadIdx.x - lr * tpr;
    float dw[NV][kVecN], w[NV][kVecN];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + tid) * kVecN;
#pragma unroll
        for (int j = 0; j < kVecN; ++j) dw[i][j] = 0.f, w[i][j] = 0.f;
        if (c < p.D) ld_row_f<float, kVecN, VEC>(w[i], p.weight + c, p.D - c);
    }
    const int64_t step = (int64_t)gridDim.x * rpb;
    int64_t row = (int64_t)blockIdx.x * rpb + lr;
    uint32_t ns[NV][WS], ny[NV][WY], nr[NV][WS];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
            if (r < p.R && c < p.D) {
                ld_row<TS, kVecN, VEC>(ns[i], (const TS *)p.s + r * p.s_st + c, p.D - c);
                ld_row<TY, kVecN, VEC>(ny[i], (const TY *)p.dy + r * p.dy_st + c, p.D - c);
                if (p.dres) ld_row<TS, kVecN, VEC>(nr[i], (const TS *)p.dres + r * p.dr_st + c, p.D - c);
            } else {
#pragma unroll
                for (int j = 0; j < WS; ++j) ns[i][j] = 0u;
#pragma unroll
                for (int j = 0; j < WY; ++j) ny[i][j] = 0u;
            }
        }
    };
    if (PRE) fetch(row);
    const float rd = 1.f / (float)p.D;
    int flip = 0;
    // every thread of the CTA makes the same number of turns
    for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < p.R; r0 += step, row += step, flip ^= 1) {
        if (!PRE) fetch(row);
        uint32_t rs[NV][WS], ry[NV][WY], rr[NV][WS];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < WS; ++j) rs[i][j] = ns[i][j], rr[i][j] = nr[i][j];
#pragma unroll
            for (int j = 0; j < WY; ++j) ry[i][j] = ny[i][j];
        }
        if (PRE) fetch(row + step);
        float ss = 0.f, gs = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float s[kVecN], g[kVecN];
            words_to_f<TS, kVecN>(s, rs[i]);
            words_to_f<TY, kVecN>(g, ry[i]);
#pragma unroll
            for (int j = 0; j < kVecN; ++j) {
                ss += __fmul_rn(s[j], s[j]);
                gs += __fmul_rn(g[j] * w[i][j], s[j]);
            }
        }
        ss = warp_sum(ss), gs = warp_sum(gs);
        if (tpr > 32) {
            const int warp = threadIdx.x >> 5, wpr = tpr >> 5, w0 = warp & ~(wpr - 1);
            if ((threadIdx.x & 31) == 0) red[flip][0][warp] = ss, red[flip][1][warp] = gs;
            __syncthreads();
            ss = red[flip][0][w0], gs = red[flip][1][w0];
            for (int i = 1; i < wpr; ++i) ss += red[flip][0][w0 + i], gs += red[flip][1][w0 + i];
        }
        const float inv = rsqrtf(ss * rd + p.eps);
        const float k = inv * inv * rd, ke = p.eps * inv * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
            if (!(row < p.R && c < p.D)) continue;
            float s[kVecN], g[kVecN], o[kVecN];
            words_to_f<TS, kVecN>(s, rs[i]);
            words_to_f<TY, kVecN>(g, ry[i]);
            if (p.dres) {
                words_to_f<TS, kVecN>(o, rr[i]);
            } else {
#pragma unroll
                for (int j = 0; j < kVecN; ++j) o[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < kVecN; ++j) {
                const float gw = g[j] * w[i][j];
                const float rest = gw * (ss - __fmul_rn(s[j], s[j])) - s[j] * (gs - __fmul_rn(gw, s[j]));
                o[j] += inv * fmaf(k, rest, ke * gw);
                dw[i][j] = fmaf(g[j], s[j] * inv, dw[i][j]);
            }
            st_row_f<TS, kVecN, VEC>((TS *)p.dx + row * p.dx_st + c, o, p.D - c);
        }
    }
    float *part = p.part + ((int64_t)blockIdx.x * rpb + lr) * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + tid) * kVecN;
        if (c < p.D) st_row_f<float, kVecN, VEC>(part + c, dw[i], p.D - c);
    }
}

// 32 columns a CTA, 8 threads a column.
__global__ void __launch_bounds__(256) col_sum_kernel(const float *in, int64_t ld, int parts, int64_t n, float *out,
                                                      int64_t n2, float *out2) {
    __shared__ float red[8][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + x;
    float a = 0.f;
    if (c < n + n2)
        for (int p = y; p < parts; p += 8) a += in[p * ld + c];
    red[y][x] = a;
    __syncthreads();
    if (y == 0 && c < n + n2) {
#pragma unroll
        for (int i = 1; i < 8; ++i) a += red[i][x];
        float *o = c < n ? out + c : out2 + (c - n);
        *o = a;
    }
}

template <typename TX, typename TR, bool Q8>
cudaError_t norm_nv(const NormParams &p, cudaStream_t st) {
    const RowShape s = row_shape(p.D, 512);
    const unsigned nt = s.tpr * s.rpb, need = (unsigned)((p.R + s.rpb - 1) / s.rpb);
    const unsigned most = 152 * (1024 / nt), grid = need < most ? need : most;
    if (!p.vec) {
        rmsnorm_kernel<TX, TR, Q8, 4, false, false><<<grid, nt, 0, st>>>(p, s.tpr);
    } else if (s.nv == 1) {
        rmsnorm_kernel<TX, TR, Q8, 1, true, true><<<grid, nt, 0, st>>>(p, s.tpr);
    } else if (s.nv == 2) {
        rmsnorm_kernel<TX, TR, Q8, 2, true, true><<<grid, nt, 0, st>>>(p, s.tpr);
    } else {
        rmsnorm_kernel<TX, TR, Q8, 4, true, false><<<grid, nt, 0, st>>>(p, s.tpr);
    }
    return cudaGetLastError();
}
template <typename TS, typename TY>
cudaError_t norm_bwd_nv(const NormBwdParams &p, cudaStream_t st) {
    const RowShape s = row_shape(p.D, 512);
    const unsigned grid = norm_bwd_parts(p.R, p.D) / s.rpb, nt = s.tpr * s.rpb;
    if (!p.vec) {
        rmsnorm_bwd_kernel<TS, TY, 4, false, false><<<grid, nt, 0, st>>>(p, s.tpr);
    } else if (s.nv == 1) {
        rmsnorm_bwd_kernel<TS, TY, 1, true, true><<<grid, nt, 0, st>>>(p, s.tpr);
    } else if (s.nv == 2) {
        rmsnorm_bwd_kernel<TS, TY, 2, true, false><<<grid, nt, 0, st>>>(p, s.tpr);
    } else {
        rmsnorm_bwd_kernel<TS, TY, 4, true, false><<<grid, nt, 0, st>>>(p, s.tpr);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rmsnorm(const NormParams &p, cudaStream_t st) {
    using bf = __nv_bfloat16;
    const bool rb = p.res ? p.res_bf16 : p.x_bf16;
    if (p.scale) {
        if (p.x_bf16) return rb ? norm_nv<bf, bf, true>(p, st) : norm_nv<bf, float, true>(p, st);
        return rb ? norm_nv<float, bf, true>(p, st) : norm_nv<float, float, true>(p, st);
    }
    if (p.x_bf16) return rb ? norm_nv<bf, bf, false>(p, st) : norm_nv<bf, float, false>(p, st);
    return rb ? norm_nv<float, bf, false>(p, st) : norm_nv<float, float, false>(p, st);
}

// Rows of partial sums: at most four CTAs a SM, each rpb rows at a time.
int norm_bwd_parts(int R, int D) {
    const RowShape s = row_shape(D, 512);
    const int need = (int)(((int64_t)R + s.rpb - 1) / s.rpb);
    return (need < 608 ? need : 608) * s.rpb;
}

cudaError_t launch_rmsnorm_bwd(const NormBwdParams &p, cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (p.s_bf16) return p.dy_bf16 ? norm_bwd_nv<bf, bf>(p, st) : norm_bwd_nv<bf, float>(p, st);
    return p.dy_bf16 ? norm_bwd_nv<float, bf>(p, st) : norm_bwd_nv<float, float>(p, st);
}

cudaError_t launch_col_sum(const float *in, int64_t ld, int parts, int64_t n, float *out, int64_t n2, float *out2,
                           cudaStream_t st) {
    if (n + n2 <= 0) return cudaSuccess;
    col_sum_kernel<<<(unsigned)((n + n2 + 31) / 32), 256, 0, st>>>(in, ld, parts, n, out, n2, out2);
    return cudaGetLastError();
}

}  // namespace gdn

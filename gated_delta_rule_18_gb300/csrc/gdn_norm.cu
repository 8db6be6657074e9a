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
// result is written once. Sums, the norm and the scales are fp32. 16384 rows
// of 4096 bf16 channels with an fp32 residual to 8 bits: 115 us, 6.5 TB/s or
// 95% of the measured copy rate. 16384 rows of 2048, bf16, the gradient: 48 us
// for 268 MB (82%) and 5 more for the sum of dw's parts; 8192 rows of 8192,
// fp32: 183 us for 1.07 GB (86%). With the next row in registers instead of
// shared memory: 49 and 244. Above 8192 channels a thread's 32 channels do not
// fit its registers and no row is under way: 4096 rows of 16384 take 169 us in
// bf16 and 298 in fp32 (47 and 53%).
#include "gdn_ssm.cuh"

namespace gdn {
namespace {

constexpr int kVecN = 8, kPairs = kVecN / 2;

// two fp32 to two e4m3 (round to nearest even, finite values saturate)
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// y / scale for one scale, rounded to nearest, by Markstein's theorem (IBM J.
// Res. Dev. 34, 1990): with r the nearest to 1 / scale and q = y r, the
// remainder y - q scale is exact in a fused multiply-add and q + r (y - q scale)
// rounds to the nearest quotient. It needs the remainder's bits above 2^-149
// for every y that is not 0 in e4m3 (y >= 2^-10 scale, remainder >= 2^-47 y) and
// a normal r: scales out of that range are divided by. One reciprocal serves
// the eight values of a vector.
__device__ __forceinline__ void quantise(f32x2 (&y)[kPairs], float scale) {
    const float dv = scale == 0.f ? 1.f : scale;
    if (dv > 1e-27f && dv < 1e30f) {
        const float r = 1.f / dv;
        const f32x2 r2 = pack2(r, r), n2 = pack2(-dv, -dv);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const f32x2 q = mul2(y[j], r2);
            y[j] = fma2(fma2(q, n2, y[j]), r2, q);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const float2 f = unpack2(y[j]);
            y[j] = pack2(f.x / dv, f.y / dv);
        }
    }
}

// Threads a row (32 to 512) for so many vectors a thread, and rows a CTA.
struct RowShape {
    int tpr, nv, rpb;
};
RowShape row_shape(int D, int vectors) {
    const int vecs = (D + kVecN - 1) / kVecN;
    RowShape s;
    s.tpr = 32;
    while (s.tpr < 512 && s.tpr * vectors < vecs) s.tpr *= 2;
    s.nv = 1;
    while (s.nv * s.tpr < vecs) s.nv *= 2;
    s.rpb = s.tpr >= 128 ? 1 : 128 / s.tpr;
    return s;
}

template <typename T>
__device__ __forceinline__ void words_to_pairs(f32x2 (&v)[kPairs], const uint32_t (&w)[RowVec<T, kVecN>::kWords]) {
    float f[kVecN];
    words_to_f<T, kVecN>(f, w);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) v[i] = pack2(f[2 * i], f[2 * i + 1]);
}
template <typename T, bool VEC>
__device__ __forceinline__ void st_pairs(T *p, const f32x2 (&v)[kPairs], int n) {
    float f[kVecN];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const float2 x = unpack2(v[i]);
        f[2 * i] = x.x, f[2 * i + 1] = x.y;
    }
    st_row_f<T, kVecN, VEC>(p, f, n);
}
// the weights of a thread's vectors
template <int NV, bool VEC>
__device__ __forceinline__ void ld_weights(f32x2 (&w)[NV][kPairs], const float *weight, int tpr, int tid, int D) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + tid) * kVecN;
        uint32_t u[kVecN] = {};
        if (c < D) ld_row<float, kVecN, VEC>(u, weight + c, D - c);
        words_to_pairs<float>(w[i], u);
    }
}

// the row's sum (or NaN-keeping maximum) over its warps; red: 16 floats, one a warp
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
    if (wpr == 2) return MAX ? max_nan(red[w0], red[w0 + 1]) : red[w0] + red[w0 + 1];
    v = MAX ? 0.f : 0.f;
    for (int i = 0; i < wpr; i += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(red + w0 + i);
        v = MAX ? max_nan(v, max_nan(max_nan(f.x, f.y), max_nan(f.z, f.w))) : v + ((f.x + f.y) + (f.z + f.w));
    }
    return v;
}

// One CTA walks rows blockIdx, blockIdx + grid, ..., the weights in registers.
// PRE: the next row's loads are issued before this row's sum is known. Pairs
// of channels in packed instructions and few warps a row: the instructions,
// not the bytes, were the limit before (138 us where this takes 115).
template <typename TX, typename TR, bool Q8, int NV, bool VEC, bool PRE>
__global__ void __launch_bounds__(512) rmsnorm_kernel(const NormParams p, int tpr) {
    __shared__ __align__(16) float red[2][2][16];
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
    f32x2 w[NV][kPairs];
    ld_weights<NV, VEC>(w, p.weight, tpr, tid, p.D);
    const int groups = p.group > 0 ? (p.D + p.group - 1) / p.group : 1;
    const float rd = 1.f / (float)p.D;
    int flip = 0;
    // every thread of the CTA makes the same number of turns
    for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < p.R; r0 += step, row += step, flip ^= 1) {
        const bool live = row < p.R;
        f32x2 s[NV][kPairs], sum2 = pack2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
            words_to_pairs<TX>(s[i], nx[i]);
            if (p.res) {
                f32x2 r[kPairs];
                words_to_pairs<TR>(r, nr[i]);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) s[i][j] = add2(s[i][j], r[j]);
                if (live && c < p.D) st_pairs<TR, VEC>((TR *)p.res_out + row * p.ro_st + c, s[i], p.D - c);
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j) sum2 = fma2(s[i][j], s[i][j], sum2);
        }
        if (PRE) fetch(row + step);
        const float2 su = unpack2(sum2);
        const float sum = row_reduce<false>(su.x + su.y, red[flip][0], tpr);
        const float inv = rsqrtf(sum * rd + p.eps);
        const f32x2 inv2 = pack2(inv, inv);
        float row_max = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
            const bool in = live && c < p.D;
#pragma unroll
            for (int j = 0; j < kPairs; ++j) s[i][j] = mul2(mul2(s[i][j], inv2), w[i][j]);
            if constexpr (!Q8) {
                if (in) st_pairs<TX, VEC>((TX *)p.out + row * p.o_st + c, s[i], p.D - c);
            } else {
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const float2 f = unpack2(s[i][j]);
                    m = max_nan(m, max_nan(fabsf(f.x), fabsf(f.y)));
                }
                row_max = max_nan(row_max, m);
                if (p.group > 0) {
                    // a group's vectors sit in group / 8 neighbouring lanes
                    for (int o = p.group / kVecN / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const float sc = m / 448.f;
                    if (in && (c & (p.group - 1)) == 0) p.scale[row * groups + c / p.group] = sc;
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
                for (int j = 0; j < 2; ++j) {
                    const float2 a = unpack2(s[i][2 * j]), b = unpack2(s[i][2 * j + 1]);
                    q[j] = pack_e4m3(a.x, a.y) | pack_e4m3(b.x, b.y) << 16;
                }
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
// Rows in shared memory: of three, four CTAs a SM keep theirs (2048 channels, bf16: 51, 48
// and 60 us with two, three and four); two of fp32 take as much.
template <typename TS, typename TY>
constexpr int kRowsAhead = sizeof(TS) + sizeof(TY) == 4 ? 3 : 2;
template <typename TS, typename TY, int NV, bool VEC, bool AHEAD>
__global__ void __launch_bounds__(512) rmsnorm_bwd_kernel(const NormBwdParams p, int tpr) {
    __shared__ __align__(16) float red[2][2][16];
    constexpr int WS = RowVec<TS, kVecN>::kWords, WY = RowVec<TY, kVecN>::kWords;
    const int rpb = blockDim.x / tpr;
    const int lr = threadIdx.x / tpr, tid = threadIdx.x - lr * tpr;
    f32x2 dw[NV][kPairs], w[NV][kPairs];
    ld_weights<NV, VEC>(w, p.weight, tpr, tid, p.D);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < kPairs; ++j) dw[i][j] = pack2(0.f, 0.f);
    const int64_t step = (int64_t)gridDim.x * rpb;
    int64_t row = (int64_t)blockIdx.x * rpb + lr;
    // Rows on their way: asynchronous copies to this thread's own slots of
    // shared memory, S - 1 rows ahead, where rows are wide (AHEAD); else loaded
    // where they are used.
    constexpr int S = kRowsAhead<TS, TY>, P = NV * (2 * WS + WY) / 4;
    extern __shared__ __align__(16) uint4 slots[];
    auto slot = [&](int g, int k) { return slots + ((g % S) * P + k) * blockDim.x + threadIdx.x; };
    uint32_t rs[NV][WS], ry[NV][WY], rr[NV][WS];
    int got = 0;
    auto fetch = [&](int64_t r, int g) {
        if (r < p.R) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * tpr + tid) * kVecN;
                if (c >= p.D) continue;
                const TS *s = (const TS *)p.s + r * p.s_st + c, *q = (const TS *)p.dres + r * p.dr_st + c;
                const TY *y = (const TY *)p.dy + r * p.dy_st + c;
#pragma unroll
                for (int k = 0; k < WS / 4; ++k) copy_async<16>(slot(g, i * (WS / 4) + k), s + k * 16 / sizeof(TS));
#pragma unroll
                for (int k = 0; k < WY / 4; ++k)
                    copy_async<16>(slot(g, NV * WS / 4 + i * (WY / 4) + k), y + k * 16 / sizeof(TY));
                if (p.dres) {
#pragma unroll
                    for (int k = 0; k < WS / 4; ++k)
                        copy_async<16>(slot(g, NV * (WS + WY) / 4 + i * (WS / 4) + k), q + k * 16 / sizeof(TS));
                }
            }
        }
        cp_async_commit();
    };
    auto take = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
            if (r < p.R && c < p.D) {
                if constexpr (AHEAD) {
                    auto read = [&](auto &w, int k0) {
                        constexpr int N = sizeof(w) / 16;
#pragma unroll
                        for (int k = 0; k < N; ++k) {
                            const uint4 u = *slot(got, k0 + i * N + k);
                            w[4 * k] = u.x, w[4 * k + 1] = u.y, w[4 * k + 2] = u.z, w[4 * k + 3] = u.w;
                        }
                    };
                    read(rs[i], 0), read(ry[i], NV * WS / 4);
                    if (p.dres) read(rr[i], NV * (WS + WY) / 4);
                } else {
                    ld_row<TS, kVecN, VEC>(rs[i], (const TS *)p.s + r * p.s_st + c, p.D - c);
                    ld_row<TY, kVecN, VEC>(ry[i], (const TY *)p.dy + r * p.dy_st + c, p.D - c);
                    if (p.dres) ld_row<TS, kVecN, VEC>(rr[i], (const TS *)p.dres + r * p.dr_st + c, p.D - c);
                }
            } else {
#pragma unroll
                for (int j = 0; j < WS; ++j) rs[i][j] = 0u;
#pragma unroll
                for (int j = 0; j < WY; ++j) ry[i][j] = 0u;
            }
        }
    };
    if constexpr (AHEAD) {
#pragma unroll
        for (int g = 0; g + 1 < S; ++g) fetch(row + g * step, g);
    }
    const float rd = 1.f / (float)p.D;
    int flip = 0;
    // every thread of the CTA makes the same number of turns
    for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < p.R; r0 += step, row += step, flip ^= 1, ++got) {
        if constexpr (AHEAD) copies_arrived<S - 2>();
        take(row);
        if constexpr (AHEAD) fetch(row + (S - 1) * step, got + S - 1);
        f32x2 ss2 = pack2(0.f, 0.f), gs2 = ss2;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            f32x2 s[kPairs], g[kPairs];
            words_to_pairs<TS>(s, rs[i]);
            words_to_pairs<TY>(g, ry[i]);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                ss2 = fma2(s[j], s[j], ss2);
                gs2 = fma2(mul2(g[j], w[i][j]), s[j], gs2);
            }
        }
        const float2 sa = unpack2(ss2), ga = unpack2(gs2);
        float ss = warp_sum(sa.x + sa.y), gs = warp_sum(ga.x + ga.y);
        if (tpr > 32) {
            const int warp = threadIdx.x >> 5, wpr = tpr >> 5, w0 = warp & ~(wpr - 1);
            if ((threadIdx.x & 31) == 0) red[flip][0][warp] = ss, red[flip][1][warp] = gs;
            __syncthreads();
            if (wpr == 2) {
                ss = red[flip][0][w0] + red[flip][0][w0 + 1], gs = red[flip][1][w0] + red[flip][1][w0 + 1];
            } else {
                ss = gs = 0.f;
                for (int i = 0; i < wpr; i += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(red[flip][0] + w0 + i);
                    const float4 b = *reinterpret_cast<const float4 *>(red[flip][1] + w0 + i);
                    ss += (a.x + a.y) + (a.z + a.w), gs += (b.x + b.y) + (b.z + b.w);
                }
            }
        }
        const float inv = rsqrtf(ss * rd + p.eps);
        const float k = inv * inv * rd, ke = p.eps * inv * inv;
        const f32x2 k2 = pack2(k, k), ke2 = pack2(ke, ke), inv2 = pack2(inv, inv);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + tid) * kVecN;
            if (!(row < p.R && c < p.D)) continue;
            f32x2 s[kPairs], g[kPairs], o[kPairs];
            words_to_pairs<TS>(s, rs[i]);
            words_to_pairs<TY>(g, ry[i]);
            if (p.dres) {
                words_to_pairs<TS>(o, rr[i]);
            } else {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) o[j] = pack2(0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                // products rounded as in the sums and not fused, as packed ones may be: a lone
                // channel's cancel to zero
                const f32x2 gw = mul2(g[j], w[i][j]);
                const float2 sf = unpack2(s[j]), gf = unpack2(gw);
                const f32x2 so = pack2(__fsub_rn(ss, __fmul_rn(sf.x, sf.x)), __fsub_rn(ss, __fmul_rn(sf.y, sf.y)));
                const f32x2 go = pack2(__fsub_rn(__fmul_rn(gf.x, sf.x), gs), __fsub_rn(__fmul_rn(gf.y, sf.y), gs));
                const f32x2 rest = fma2(gw, so, mul2(s[j], go));
                o[j] = fma2(inv2, fma2(k2, rest, mul2(ke2, gw)), o[j]);
                dw[i][j] = fma2(g[j], mul2(s[j], inv2), dw[i][j]);
            }
            st_pairs<TS, VEC>((TS *)p.dx + row * p.dx_st + c, o, p.D - c);
        }
    }
    float *part = p.part + ((int64_t)blockIdx.x * rpb + lr) * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + tid) * kVecN;
        if (c < p.D) st_pairs<float, VEC>(part + c, dw[i], p.D - c);
    }
}

// 32 columns a CTA, Y threads a column.
template <int Y>
__global__ void __launch_bounds__(32 * Y) col_sum_kernel(const float *in, int64_t ld, int parts, int64_t n, float *out,
                                                         int64_t n2, float *out2) {
    __shared__ float red[Y][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + x;
    float a = 0.f;
    if (c < n + n2) {
#pragma unroll 4
        for (int p = y; p < parts; p += Y) a += in[p * ld + c];
    }
    red[y][x] = a;
    __syncthreads();
    if (y == 0 && c < n + n2) {
#pragma unroll
        for (int i = 1; i < Y; ++i) a += red[i][x];
        *(c < n ? out + c : out2 + (c - n)) = a;
    }
}

template <typename TX, typename TR, bool Q8>
cudaError_t norm_nv(const NormParams &p, cudaStream_t st) {
    const RowShape s = row_shape(p.D, 1);
    const unsigned nt = s.tpr * s.rpb, need = (unsigned)((p.R + s.rpb - 1) / s.rpb);
    const unsigned most = 152 * (1024 / nt), grid = need < most ? need : most;
    auto run = [&](auto vec) {
        constexpr bool V = decltype(vec)::value;
        if (s.nv == 1) rmsnorm_kernel<TX, TR, Q8, 1, V, true><<<grid, nt, 0, st>>>(p, s.tpr);
        else if (s.nv == 2) rmsnorm_kernel<TX, TR, Q8, 2, V, true><<<grid, nt, 0, st>>>(p, s.tpr);
        else rmsnorm_kernel<TX, TR, Q8, 4, V, false><<<grid, nt, 0, st>>>(p, s.tpr);
    };
    if (p.vec) run(std::true_type());
    else run(std::false_type());
    return cudaGetLastError();
}
template <typename TS, typename TY>
cudaError_t norm_bwd_nv(const NormBwdParams &p, cudaStream_t st) {
    const RowShape s = row_shape(p.D, 2);
    const unsigned grid = norm_bwd_parts(p.R, p.D) / s.rpb, nt = s.tpr * s.rpb;
    auto run = [&](auto nv, auto vec, auto ahead) -> cudaError_t {
        auto *k = rmsnorm_bwd_kernel<TS, TY, nv(), vec(), ahead()>;
        constexpr int each = ahead() ? kRowsAhead<TS, TY> * nv() * (2 * sizeof(TS) + sizeof(TY)) * kVecN : 0;
        const int smem = each * nt;
        if (smem > 40 * 1024) {  // 48 KB with the static part
            // (of 512 threads: a smaller call's own size would lower the kernel's limit under another thread's launch)
            const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, each * 512);
            if (e != cudaSuccess) return e;
        }
        k<<<grid, nt, smem, st>>>(p, s.tpr);
        return cudaGetLastError();
    };
    auto by_vectors = [&](auto vec) {
        if (s.nv == 1) return run(std::integral_constant<int, 1>(), vec, vec);
        if (s.nv == 2) return run(std::integral_constant<int, 2>(), vec, vec);
        return run(std::integral_constant<int, 4>(), vec, std::false_type());
    };
    return p.vec ? by_vectors(std::true_type()) : by_vectors(std::false_type());
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
    const RowShape s = row_shape(D, 2);
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
    // few columns over hundreds of parts are bound by the loads' latency: more threads a column
    const unsigned grid = (unsigned)((n + n2 + 31) / 32);
    if (grid < 152) col_sum_kernel<32><<<grid, 1024, 0, st>>>(in, ld, parts, n, out, n2, out2);
    else col_sum_kernel<8><<<grid, 256, 0, st>>>(in, ld, parts, n, out, n2, out2);
    return cudaGetLastError();
}

}  // namespace gdn

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

#include <type_traits>

namespace gdn {
namespace {

constexpr int kVecN = 8, kPairs = kVecN / 2;

struct RowShape {
    int tpr, nv, rpb;  // threads a row, vectors a thread, rows a CTA
};
// Whole warps, as few as cover the row (1792 channels: 7, not 8), up to 512
// threads; rows of up to two warps share a CTA.
RowShape row_shape(int D) {
    const int vecs = (D + kVecN - 1) / kVecN;
    RowShape s;
    s.nv = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4;
    s.tpr = ((vecs + s.nv - 1) / s.nv + 31) / 32 * 32;
    s.rpb = s.tpr > 64 ? 1 : 128 / s.tpr;
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

__device__ __forceinline__ f32x2 gate_of(f32x2 x, int act) {
    if (act == kGateLinear) return x;
    const f32x2 s = sigmoid_2(x);
    return act == kGateSigmoid ? s : mul2(x, s);
}
// the factor and its derivative
__device__ __forceinline__ f32x2 gate_of(f32x2 x, int act, f32x2 &d) {
    const f32x2 one = pack2(1.f, 1.f), minus = pack2(-1.f, -1.f);
    d = one;
    if (act == kGateLinear) return x;
    const f32x2 s = sigmoid_2(x), rest = fma2(s, minus, one);
    if (act == kGateSigmoid) {
        d = mul2(s, rest);
        return s;
    }
    const f32x2 f = mul2(x, s);
    d = fma2(f, rest, s);
    return f;
}

// sums of N values over a row's warps; red: N rows of 16 floats, one a warp,
// zeros past the CTA's
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[16], int tpr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (tpr == 32) return;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) red[k][warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (tpr == 64) {
            v[k] = red[k][warp & ~1] + red[k][warp | 1];
        } else {
            v[k] = 0.f;
            for (int i = 0; i < tpr >> 5; i += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(red[k] + i);
                v[k] += (f.x + f.y) + (f.z + f.w);
            }
        }
    }
}

// The rows of a run on their way: asynchronous copies of 16 bytes to a thread's
// own slots of shared memory, which no other thread reads, `stages` - 1 rows
// ahead. A tensor's vector is N = 16 or 32 bytes of a thread's channels.
struct Slots {
    uint4 *base;     // this thread's first
    int pieces, stages;
    __device__ __forceinline__ uint4 *at(int stage, int piece) const { return base + (stage * pieces + piece) * blockDim.x; }
    template <typename T>
    __device__ __forceinline__ void copy(int stage, int piece, const T *src) const {
#pragma unroll
        for (int k = 0; k < kVecN * (int)sizeof(T) / 16; ++k) copy_async<16>(at(stage, piece + k), src + k * 16 / sizeof(T));
    }
    template <typename T>
    __device__ __forceinline__ void get(f32x2 (&v)[kPairs], int stage, int piece) const {
        uint32_t w[RowVec<T, kVecN>::kWords];
#pragma unroll
        for (int k = 0; k < kVecN * (int)sizeof(T) / 16; ++k) {
            const uint4 u = *at(stage, piece + k);
            w[4 * k] = u.x, w[4 * k + 1] = u.y, w[4 * k + 2] = u.z, w[4 * k + 3] = u.w;
        }
        to_pairs<T>(v, w);
    }
};
__device__ __forceinline__ void slots_arrived(int ahead) {  // all but the last `ahead` rows
    if (ahead == 1) copies_arrived<1>();
    else copies_arrived<0>();
}

// A CTA walks a run of one sequence's rows (blockIdx.y; all rows are one where
// no gate is shared). AHEAD: rows come by asynchronous copies; else (rows that
// are not wide, or of more than 8192 channels) loads where they are used, and
// the weights, which do not fit the registers there, too.
template <typename TX, typename TR, int NV, bool VEC, bool AHEAD>
__global__ void __launch_bounds__(512) block_norm_kernel(const BlockNormParams p, int tpr, int stages) {
    __shared__ __align__(16) float red[2][2][16];
    extern __shared__ __align__(16) uint4 staged[];
    constexpr int NX = kVecN * sizeof(TX) / 16, NR = kVecN * sizeof(TR) / 16;
    constexpr bool HOLD = NV <= 2;  // weights in registers
    const int rpb = blockDim.x / tpr, lr = threadIdx.x / tpr, tid = threadIdx.x - lr * tpr;
    const int64_t rows = p.shared ? p.gate_rows : p.R, first = (int64_t)blockIdx.y * rows;
    const int64_t run0 = first + (int64_t)blockIdx.x * p.run, run1 = min(run0 + p.run, first + rows);
    const bool token = p.act && !p.shared;
    const Slots slots{staged + threadIdx.x, NV * (NX * (token ? 2 : 1) + NR), stages};
    auto piece = [&](int i, int k) { return i * (NX * (token ? 2 : 1) + NR) + (k == 0 ? 0 : k == 1 ? NX : NX + NR); };
    auto channel = [&](int i) { return (i * tpr + tid) * kVecN; };
    if (threadIdx.x < 64) (&red[0][0][0])[threadIdx.x] = 0.f;
    auto fetch = [&](int64_t row, int stage) {
        if (row < run1) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = channel(i);
                if (c >= p.D) continue;
                slots.copy(stage, piece(i, 0), (const TX *)p.y + row * p.y_st + c);
                slots.copy(stage, piece(i, 1), (const TR *)p.res + row * p.r_st + c);
                if (token) slots.copy(stage, piece(i, 2), (const TX *)p.gate + row * p.g_st + c);
            }
        }
        cp_async_commit();
    };
    if (AHEAD)
        for (int g = 0; g + 1 < stages; ++g) fetch(run0 + lr + (int64_t)g * rpb, g);
    // alpha scale post, with the gate's factor where the run shares it; pre
    f32x2 w1[HOLD ? NV : 1][kPairs], w2[HOLD ? NV : 1][kPairs];
    auto weights = [&](int c, int at) {
        const int n = p.D - c;
        get_factor<VEC>(w1[at], p.scale, p.post, p.alpha, c, n);
        get<float, VEC>(w2[at], p.pre ? p.pre + c : nullptr, n);
        if (p.shared) {
            f32x2 g[kPairs];
            get<TX, VEC>(g, (const TX *)p.gate + (int64_t)blockIdx.y * p.g_st + c, n);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) w1[at][j] = mul2(w1[at][j], gate_of(g[j], p.act));
        }
    };
    if (HOLD) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (channel(i) < p.D) weights(channel(i), i);
    }
    const float rd = 1.f / (float)p.D;
    int flip = 0, stage = 0;
    __syncthreads();
    for (int64_t r0 = run0; r0 < run1; r0 += rpb, flip ^= 1) {
        const int64_t row = r0 + lr;
        const bool live = row < run1;
        int ahead = stage + stages - 1;
        if (ahead >= stages) ahead -= stages;
        if (AHEAD) slots_arrived(stages - 2), fetch(row + (int64_t)(stages - 1) * rpb, ahead);
        auto take_y = [&](f32x2 (&v)[kPairs], int i, int c) {
            if (AHEAD) slots.get<TX>(v, stage, piece(i, 0));
            else get<TX, VEC>(v, (const TX *)p.y + row * p.y_st + c, p.D - c);
        };
        f32x2 s[NV][kPairs];
        float inv = 1.f;
        if (p.post) {
            f32x2 sum2 = pack2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = channel(i);
                if (!(live && c < p.D)) continue;
                take_y(s[i], i, c);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) sum2 = fma2(s[i][j], s[i][j], sum2);
            }
            const float2 su = unpack2(sum2);
            float v[1] = {su.x + su.y};
            row_sums<1>(v, red[flip], tpr);
            inv = rsqrtf(v[0] * rd + p.eps);
        }
        const f32x2 inv2 = pack2(inv, inv);
        f32x2 sum2 = pack2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = channel(i), at = HOLD ? i : 0;
            if (!(live && c < p.D)) continue;
            if (!HOLD) weights(c, 0);
            f32x2 g[kPairs], r[kPairs];
            if (!p.post) take_y(s[i], i, c);
            if (AHEAD) slots.get<TR>(r, stage, piece(i, 1));
            else get<TR, VEC>(r, (const TR *)p.res + row * p.r_st + c, p.D - c);
            if (token) {
                if (AHEAD) slots.get<TX>(g, stage, piece(i, 2));
                else get<TX, VEC>(g, (const TX *)p.gate + row * p.g_st + c, p.D - c);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) s[i][j] = mul2(mul2(s[i][j], inv2), gate_of(g[j], p.act));
            } else {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) s[i][j] = mul2(s[i][j], inv2);
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j) s[i][j] = fma2(s[i][j], w1[at][j], r[j]);
            put<TR, VEC>((TR *)p.res_out + row * p.ro_st + c, s[i], p.D - c);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) sum2 = fma2(s[i][j], s[i][j], sum2);
        }
        if (p.pre) {
            // (channels past D are zeros: y, residual and weights are loaded so)
            const float2 su = unpack2(sum2);
            float v[1] = {su.x + su.y};
            row_sums<1>(v, red[flip] + 1, tpr);
            const float q = rsqrtf(v[0] * rd + p.eps);
            const f32x2 q2 = pack2(q, q);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = channel(i);
                if (!(live && c < p.D)) continue;
                if (!HOLD) weights(c, 0);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) s[i][j] = mul2(mul2(s[i][j], q2), w2[HOLD ? i : 0][j]);
                put<TX, VEC>((TX *)p.out + row * p.o_st + c, s[i], p.D - c);
            }
        }
        if (++stage == stages) stage = 0;
    }
}

// The gradient of a norm at channel pair x for the weighted gradient gw = w dy,
// with S = sum x^2, G = sum gw x, inv, added to `more`: both sums lose the
// channel's own terms first, rounded as the sums have them, which cancel
// exactly (they are all there is when one channel dominates its row; scalar
// subtractions, as packed ones may be fused with the products).
struct NormGrad {
    f32x2 k, ke;
    float S, G, inv;
    __device__ __forceinline__ NormGrad(float S_, float G_, float rd, float eps) : S(S_), G(G_) {
        inv = rsqrtf(S * rd + eps);
        const float a = inv * (inv * inv * rd), b = inv * (eps * inv * inv);
        k = pack2(a, a), ke = pack2(b, b);
    }
    __device__ __forceinline__ f32x2 at(f32x2 x, f32x2 gw, f32x2 more) const {
        const float2 xx = unpack2(mul2(x, x)), gx = unpack2(mul2(gw, x));
        const f32x2 so = pack2(__fsub_rn(S, xx.x), __fsub_rn(S, xx.y)), go = pack2(__fsub_rn(gx.x, G), __fsub_rn(gx.y, G));
        return fma2(k, fma2(gw, so, mul2(x, go)), fma2(ke, gw, more));
    }
};

// Runs as in the forward. A thread keeps its channels' sums, in registers with
// one vector a thread (rows of up to 4096 channels), else in its own slots of
// shared memory. A row is read from its slots once a phase rather than held.
template <typename TX, typename TR, int NV, bool VEC, bool AHEAD, bool TOKEN>
__global__ void __launch_bounds__(512) block_norm_bwd_kernel(const BlockNormBwdParams p, int tpr, int stages) {
    __shared__ __align__(16) float red[2][4][16];
    extern __shared__ __align__(16) uint4 staged[];
    constexpr int NX = kVecN * sizeof(TX) / 16, NR = kVecN * sizeof(TR) / 16;
    constexpr bool HOLD = NV == 1;  // sums and weights in registers
    constexpr int kKept = HOLD ? 0 : NV * 2 * kPairs / 2;  // 16-byte slots a thread of sums
    const int rpb = blockDim.x / tpr, lr = threadIdx.x / tpr, tid = threadIdx.x - lr * tpr;
    const int64_t rows = p.shared ? p.gate_rows : p.R, first = (int64_t)blockIdx.y * rows;
    const int64_t run0 = first + (int64_t)blockIdx.x * p.run, run1 = min(run0 + p.run, first + rows);
    // y, dres, then s and dout with pre, then the gate
    const int n_dres = p.dres ? NR : 0, n_pre = p.pre ? NR + NX : 0, vec_pieces = NX + n_dres + n_pre + (TOKEN ? NX : 0);
    const Slots slots{staged + kKept * blockDim.x + threadIdx.x, NV * vec_pieces, stages};
    auto sums = [&](int i, int q, int j) -> f32x2 & {
        return reinterpret_cast<f32x2 *>(staged)[((i * 2 + q) * kPairs + j) * blockDim.x + threadIdx.x];
    };
    auto channel = [&](int i) { return (i * tpr + tid) * kVecN; };
    const f32x2 zero = pack2(0.f, 0.f);
    for (int e = threadIdx.x; e < 128; e += blockDim.x) (&red[0][0][0])[e] = 0.f;
    auto fetch = [&](int64_t row, int stage) {
        if (row < run1) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = channel(i), o = i * vec_pieces;
                if (c >= p.D) continue;
                slots.copy(stage, o, (const TX *)p.y + row * p.y_st + c);
                if (p.dres) slots.copy(stage, o + NX, (const TR *)p.dres + row * p.dr_st + c);
                if (p.pre) {
                    slots.copy(stage, o + NX + n_dres, (const TR *)p.s + row * p.s_st + c);
                    slots.copy(stage, o + NX + n_dres + NR, (const TX *)p.dout + row * p.do_st + c);
                }
                if (TOKEN) slots.copy(stage, o + NX + n_dres + n_pre, (const TX *)p.gate + row * p.g_st + c);
            }
        }
        cp_async_commit();
    };
    if (AHEAD)
        for (int g = 0; g + 1 < stages; ++g) fetch(run0 + lr + (int64_t)g * rpb, g);
    f32x2 w1[kPairs], w2[kPairs], sa[kPairs], sr[kPairs];  // as in the forward; the sums
    auto weights = [&](int c) {
        const int n = p.D - c;
        get_factor<VEC>(w1, p.scale, p.post, p.alpha, c, n);
        get<float, VEC>(w2, p.pre ? p.pre + c : nullptr, n);
        if (!TOKEN && p.shared) {
            f32x2 g[kPairs];
            get<TX, VEC>(g, (const TX *)p.gate + (int64_t)blockIdx.y * p.g_st + c, n);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) w1[j] = mul2(w1[j], gate_of(g[j], p.act));
        }
    };
#pragma unroll
    for (int j = 0; j < kPairs; ++j) w1[j] = w2[j] = sa[j] = sr[j] = zero;
    if constexpr (HOLD) {
        if (tid * kVecN < p.D) weights(tid * kVecN);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < kPairs; ++j) sums(i, 0, j) = sums(i, 1, j) = zero;
    }
    const float rd = 1.f / (float)p.D;
    int flip = 0, stage = 0;
    __syncthreads();
    for (int64_t r0 = run0; r0 < run1; r0 += rpb, flip ^= 1) {
        const int64_t row = r0 + lr;
        const bool live = row < run1;
        int ahead = stage + stages - 1;
        if (ahead >= stages) ahead -= stages;
        if (AHEAD) slots_arrived(stages - 2), fetch(row + (int64_t)(stages - 1) * rpb, ahead);
        auto take_y = [&](f32x2 (&v)[kPairs], int i, int c) {
            if (AHEAD) slots.get<TX>(v, stage, i * vec_pieces);
            else get<TX, VEC>(v, (const TX *)p.y + row * p.y_st + c, p.D - c);
        };
        auto take_s = [&](f32x2 (&s)[kPairs], f32x2 (&d)[kPairs], int i, int c) {  // and dout
            const int o = i * vec_pieces + NX + n_dres;
            if (AHEAD) slots.get<TR>(s, stage, o), slots.get<TX>(d, stage, o + NR);
            else get<TR, VEC>(s, (const TR *)p.s + row * p.s_st + c, p.D - c), get<TX, VEC>(d, (const TX *)p.dout + row * p.do_st + c, p.D - c);
        };
        float v[3] = {0.f, 0.f, 0.f};  // of s^2, pre dout s, y^2
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = channel(i);
            if (!(live && c < p.D)) continue;
            if (!HOLD) weights(c);
            f32x2 a = zero, b = zero, d = zero, hs[kPairs], hd[kPairs], hy[kPairs];
            if (p.pre) {
                take_s(hs, hd, i, c);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) a = fma2(hs[j], hs[j], a), b = fma2(mul2(hd[j], w2[j]), hs[j], b);
            }
            if (p.post) {
                take_y(hy, i, c);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) d = fma2(hy[j], hy[j], d);
            }
            const float2 fa = unpack2(a), fb = unpack2(b), fd = unpack2(d);
            v[0] += fa.x + fa.y, v[1] += fb.x + fb.y, v[2] += fd.x + fd.y;
        }
        row_sums<3>(v, red[flip], tpr);
        const NormGrad ns(v[0], v[1], rd, p.eps);
        const float inv_y = p.post ? rsqrtf(v[2] * rd + p.eps) : 1.f;
        const f32x2 iy2 = pack2(inv_y, inv_y), is2 = pack2(ns.inv, ns.inv);
        f32x2 e[kPairs];  // k post f ds, the gradient behind y's norm
        float ge[1] = {0.f};
        // The stream's gradient and what follows from it. again: e alone (rows
        // whose e is not held).
        auto stream = [&](int i, int c, auto form) {
            constexpr bool again = decltype(form)::value;
            f32x2 ds[kPairs], hy[kPairs];
            if (p.dres) {
                if (AHEAD) slots.get<TR>(ds, stage, i * vec_pieces + NX);
                else get<TR, VEC>(ds, (const TR *)p.dres + row * p.dr_st + c, p.D - c);
            } else {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) ds[j] = zero;
            }
            if (p.pre) {
                f32x2 hs[kPairs], hd[kPairs];
                take_s(hs, hd, i, c);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    ds[j] = ns.at(hs[j], mul2(hd[j], w2[j]), ds[j]);
                    if (!again) {
                        const f32x2 sn = mul2(hs[j], is2);
                        if constexpr (HOLD) sr[j] = fma2(hd[j], sn, sr[j]);
                        else sums(i, 1, j) = fma2(hd[j], sn, sums(i, 1, j));
                    }
                }
            }
            if (!again) {
                put<TR, VEC>((TR *)p.ds + row * p.ds_st + c, ds, p.D - c);
                take_y(hy, i, c);
            }
            f32x2 hg[kPairs];
            if (TOKEN) {
                if (AHEAD) slots.get<TX>(hg, stage, i * vec_pieces + NX + n_dres + n_pre);
                else get<TX, VEC>(hg, (const TX *)p.gate + row * p.g_st + c, p.D - c);
            }
            f32x2 g2 = zero;
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                f32x2 dsf = ds[j], df;
                if (TOKEN) dsf = mul2(ds[j], gate_of(hg[j], p.act, df));
                e[j] = mul2(dsf, w1[j]);
                if (!again) {
                    const f32x2 yn = mul2(hy[j], iy2);
                    if (TOKEN) hg[j] = mul2(mul2(mul2(ds[j], w1[j]), yn), df);
                    g2 = fma2(e[j], hy[j], g2);
                    if constexpr (HOLD) sa[j] = fma2(dsf, yn, sa[j]);
                    else sums(i, 0, j) = fma2(dsf, yn, sums(i, 0, j));
                }
            }
            if (!again) {
                const float2 fg = unpack2(g2);
                ge[0] += fg.x + fg.y;
                if (TOKEN) put<TX, VEC>((TX *)p.dgate + row * p.dg_st + c, hg, p.D - c);
            }
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = channel(i);
            if (!(live && c < p.D)) continue;
            if (!HOLD) weights(c);
            stream(i, c, std::false_type());
        }
        if (p.post) row_sums<1>(ge, red[flip] + 3, tpr);
        const NormGrad ny(v[2], ge[0], rd, p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = channel(i);
            if (!(live && c < p.D)) continue;
            if (!HOLD) weights(c), stream(i, c, std::true_type());
            if (p.post) {
                f32x2 hy[kPairs];
                take_y(hy, i, c);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) e[j] = ny.at(hy[j], e[j], zero);
            }
            put<TX, VEC>((TX *)p.dy + row * p.dy_st + c, e, p.D - c);
        }
        if (++stage == stages) stage = 0;
    }
    float *part = p.part + (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * rpb + lr) * 2 * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = channel(i);
        if (c >= p.D) continue;
        if constexpr (!HOLD) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) sa[j] = sums(i, 0, j), sr[j] = sums(i, 1, j);
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

// Stages of `row` bytes that leave `ctas` CTAs a SM: two or three.
int stages_for(int row, int kept, int ctas) { return (3 * row + kept) * ctas <= 216 * 1024 ? 3 : 2; }
template <class K>
cudaError_t with_smem(K *k, int smem) {
    if (smem <= 40 * 1024) return cudaSuccess;  // 48 KB with the static part
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}
template <typename TX, typename TR>
cudaError_t norm_nv(const BlockNormParams &p, cudaStream_t st) {
    const RowShape s = row_shape(p.D);
    const int nt = s.tpr * s.rpb, token = p.act && !p.shared;
    const dim3 grid(p.runs, p.shared ? p.R / p.gate_rows : 1);
    auto run = [&](auto nv, auto vec, auto ahead) -> cudaError_t {
        auto *k = block_norm_kernel<TX, TR, nv(), vec(), ahead()>;
        const int row = ahead() ? nv() * kVecN * ((int)sizeof(TX) * (1 + token) + (int)sizeof(TR)) * nt : 0;
        const int stages = stages_for(row, 0, 1024 / nt < 4 ? 1024 / nt : 4), smem = ahead() ? stages * row : 0;
        const cudaError_t e = with_smem(k, smem);
        if (e != cudaSuccess) return e;
        k<<<grid, nt, smem, st>>>(p, s.tpr, stages);
        return cudaGetLastError();
    };
    auto by_vectors = [&](auto vec) {
        if (s.nv == 1) return run(std::integral_constant<int, 1>(), vec, vec);
        if (s.nv == 2) return run(std::integral_constant<int, 2>(), vec, vec);
        return run(std::integral_constant<int, 4>(), vec, std::false_type());
    };
    return p.vec ? by_vectors(std::true_type()) : by_vectors(std::false_type());
}
template <typename TX, typename TR>
cudaError_t norm_bwd_nv(const BlockNormBwdParams &p, cudaStream_t st) {
    const RowShape s = row_shape(p.D);
    const int nt = s.tpr * s.rpb;
    const bool token = p.act && !p.shared;
    const dim3 grid(p.runs, p.shared ? p.R / p.gate_rows : 1);
    auto run = [&](auto nv, auto vec, auto ahead, auto tok) -> cudaError_t {
        auto *k = block_norm_bwd_kernel<TX, TR, nv(), vec(), ahead(), tok()>;
        const int kept = nv() > 1 ? nv() * 2 * kPairs * 8 * nt : 0, x = sizeof(TX), r = sizeof(TR);
        const int row = ahead() ? nv() * kVecN * (x * (1 + tok() + (p.pre ? 1 : 0)) + r * ((p.dres ? 1 : 0) + (p.pre ? 1 : 0))) * nt : 0;
        const int stages = stages_for(row, kept, nv() > 1 ? 1 : nt > 256 ? 1 : 2), smem = kept + (ahead() ? stages * row : 0);
        const cudaError_t e = with_smem(k, smem);
        if (e != cudaSuccess) return e;
        k<<<grid, nt, smem, st>>>(p, s.tpr, stages);
        return cudaGetLastError();
    };
    auto by_gate = [&](auto nv, auto vec, auto ahead) {
        return token ? run(nv, vec, ahead, std::true_type()) : run(nv, vec, ahead, std::false_type());
    };
    auto by_vectors = [&](auto vec) {
        if (s.nv == 1) return by_gate(std::integral_constant<int, 1>(), vec, vec);
        if (s.nv == 2) return by_gate(std::integral_constant<int, 2>(), vec, std::false_type());
        return by_gate(std::integral_constant<int, 4>(), vec, std::false_type());
    };
    return p.vec ? by_vectors(std::true_type()) : by_vectors(std::false_type());
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormParams &p, cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (p.y_bf16) return p.r_bf16 ? norm_nv<bf, bf>(p, st) : norm_nv<bf, float>(p, st);
    return p.r_bf16 ? norm_nv<float, bf>(p, st) : norm_nv<float, float>(p, st);
}

// Runs of a sequence's rows: as many CTAs as make 1024 threads a SM, two at least.
void block_norm_runs(int R, int D, int gate_rows, int *runs, int *run, int64_t *parts) {
    const RowShape s = row_shape(D);
    const int rows = gate_rows > 1 ? gate_rows : R, n = gate_rows > 1 ? R / gate_rows : 1;
    const int nt = s.tpr * s.rpb, ctas = 152 * (nt <= 128 ? 8 : nt <= 256 ? 4 : 2), most = n < ctas ? ctas / n : 1;
    const int need = (int)(((int64_t)rows + s.rpb - 1) / s.rpb);
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

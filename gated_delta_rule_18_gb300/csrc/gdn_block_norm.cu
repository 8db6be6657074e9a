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
// HBM is the bound: every tensor is read once and written once; a row belongs to
// tpr threads of one CTA, 8 channels a vector, and both of its reductions
// cross warps through shared memory. Sums and norms are fp32.
//
// Measured (copy rate 6.78 TB/s): forward, 4 x 4096 rows of 4096 channels with a
// gate a token, fp32 residual 152 us (91 %), bf16 113 (87 %), all fp32 214 (93 %);
// gradient 300 (72 %), 289 (55 %) and 361 (88 %). 2 x 8192 rows of 1792 channels, bf16, gate shared: 48, and 111
// in three launches (98, 10, 5). In bf16 the gradient's instructions come before
// its bytes: 140 a warp and channel pair (two norms' sums and gradients), at 0.56
// a cycle from the 16 warps a SM that 128 registers leave.
#include "gdn_block.cuh"
#include "gdn_ssm.cuh"

#include <cfloat>
#include <type_traits>

namespace gdn {
namespace {

constexpr int kVecN = 8, kPairs = kVecN / 2;

struct RowShape {
    int tpr, nv, rpb;  // threads a row, vectors a thread, rows a CTA
};
// `two`: two vectors a thread where that leaves a row two warps, as what a row
// costs each warp (its two sums, pointers, barriers) is as much as four pairs
// of channels. Not for the gradient with a gate value a token, whose two
// vectors do not fit the registers (4 x 4096 x 4096, bf16, fp32 stream: 366 us
// for 323), nor for rows that are not wide. Whole warps, as few as cover the
// row, up to 512 threads; rows of up to two warps share a CTA.
RowShape row_shape(int D, bool two) {
    const int vecs = (D + kVecN - 1) / kVecN;
    RowShape s;
    s.nv = vecs <= (two ? 64 : 512) ? 1 : vecs <= 1024 ? 2 : 4;
    s.tpr = ((vecs + s.nv - 1) / s.nv + 31) / 32 * 32;
    s.rpb = s.tpr > 64 ? 1 : 128 / s.tpr;
    return s;
}
RowShape row_shape(const BlockNormParams &p) { return row_shape(p.D, p.vec); }
RowShape row_shape(const BlockNormBwdParams &p) { return row_shape(p.D, p.vec && !(p.act && !p.shared)); }
// Runs of a sequence's rows: as many CTAs as make 1024 threads a SM, two at least.
struct Runs {
    int n, len;
    int64_t parts;
};
Runs runs_of(int R, int gate_rows, const RowShape &s) {
    const bool shared = gate_rows > 1 && R > 0;
    const int rows = shared ? gate_rows : R, n = shared ? R / gate_rows : 1;
    const int nt = s.tpr * s.rpb, ctas = 152 * (nt <= 128 ? 8 : nt <= 256 ? 4 : 2), most = n < ctas ? ctas / n : 1;
    const int need = (int)(((int64_t)rows + s.rpb - 1) / s.rpb), want = need < most ? need : most;
    Runs r;
    r.len = want > 0 ? (need + want - 1) / want * s.rpb : s.rpb;
    r.n = (int)(((int64_t)rows + r.len - 1) / r.len);
    r.parts = (int64_t)n * r.n * s.rpb;
    return r;
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

// 1 / sqrt(v), the approximation made as good as a rounding by one step of
// Newton's: it is a factor of the whole row, and each sum of a bf16 stream that
// it moves over a tie counts 2^-8 in what comes after. (The forward's; it costs
// the gradient 3 %, which has no sums to round.)
__device__ __forceinline__ float inv_root(float v) {
    const float r = rsqrtf(v), e = fmaf(-v * r, r, 1.f);
    return fabsf(e) < 1.f ? fmaf(0.5f * r, e, r) : r;  // (0 and infinity as they are)
}

// The warps of a thread's row: `n` from `w0` on, whose sums lie side by side.
struct RowWarps {
    int w0, n;
    __device__ __forceinline__ RowWarps(int tpr) : w0(tpr == 64 ? (threadIdx.x >> 5) & ~1 : 0), n(tpr >> 5) {}
};
// The row's sum of v; red: 16 floats, one a warp, zeros past the CTA's.
__device__ __forceinline__ float row_sum(float v, float *red, RowWarps r) {
    v = warp_sum(v);
    if (r.n == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    if (r.n == 2) return red[r.w0] + red[r.w0 + 1];
    v = 0.f;
#pragma unroll 1
    for (int i = 0; i < r.n; i += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(red + i);
        v += (f.x + f.y) + (f.z + f.w);
    }
    return v;
}
// The row's sums of three values: lanes halve what they carry as they halve
// the lanes (6 shuffles where one value at a time takes 15). red as above, of
// four values a warp.
__device__ __forceinline__ void row_sums3(float (&v)[3], float4 *red, RowWarps r) {
    const int lane = threadIdx.x & 31;
    const bool up = lane & 16, half = lane & 8;
    float a = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
    const float b = (up ? 0.f : v[1]) + __shfl_xor_sync(0xffffffffu, up ? v[1] : 0.f, 16);
    a = (half ? b : a) + __shfl_xor_sync(0xffffffffu, half ? a : b, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (r.n == 1) {
#pragma unroll
        for (int k = 0; k < 3; ++k) v[k] = __shfl_sync(0xffffffffu, a, 8 * k);
        return;
    }
    if ((lane & 7) == 0) reinterpret_cast<float *>(red + (threadIdx.x >> 5))[lane >> 3] = a;
    __syncthreads();
    f32x2 xy = pack2(0.f, 0.f);
    v[2] = 0.f;
#pragma unroll 1
    for (int i = 0; i < r.n; i += 2) {
        const float4 f = red[r.w0 + i], g = red[r.w0 + i + 1];
        xy = add2(xy, add2(pack2(f.x, f.y), pack2(g.x, g.y))), v[2] += f.z + g.z;
    }
    const float2 f = unpack2(xy);
    v[0] = f.x, v[1] = f.y;
}

// The rows of a run on their way: asynchronous copies of 16 bytes to a thread's
// own slots of shared memory, which no other thread reads, `stages` - 1 rows
// ahead.
struct Slots {
    uint4 *base;  // this thread's first
    int pieces;   // of 16 bytes a row
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
    // n pieces of values times a power of two, which every type holds; zeros for 0. (Few rows need it: as
    // loops, for the registers.)
    template <typename T>
    __device__ __forceinline__ void scale(int stage, int piece, int n, float power) const {
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
            uint32_t *w = reinterpret_cast<uint32_t *>(at(stage, piece + k));
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4) {
                    w[j] = power == 0.f ? 0u : __float_as_uint(__uint_as_float(w[j]) * power);
                } else {
                    const float lo = __uint_as_float(w[j] << 16) * power, hi = __uint_as_float(w[j] & 0xffff0000u) * power;
                    w[j] = power == 0.f ? 0u : __float_as_uint(lo) >> 16 | (__float_as_uint(hi) & 0xffff0000u);
                }
            }
        }
    }
};
__device__ __forceinline__ void slots_arrived(int ahead) {  // all but the last `ahead` rows
    if (ahead == 1) copies_arrived<1>();
    else copies_arrived<0>();
}
// A tensor's row pointer of this thread. The elements from one of its rows to
// the next, stride times rows a CTA, come with the parameters: in registers
// they would be two more a tensor.
struct Steps {
    int64_t y, res, gate, out, res_out;               // forward
    int64_t s, dout, dres, dy, ds, dgate;             // gradient (and y, gate)
};
template <typename T>
__device__ __forceinline__ T *row_of(T *p, int64_t st, int64_t row, int c) { return p + row * st + c; }

// A CTA walks a run of one sequence's rows (blockIdx.y; all rows are one where
// no gate is shared). AHEAD: rows come by asynchronous copies; else (rows that
// are not wide, or of more than 8192 channels) they are loaded where the row
// begins. Weights stay in registers for up to two vectors a thread.
template <typename TX, typename TR, int NV, bool VEC, bool AHEAD>
__global__ void __launch_bounds__(NV == 1 && VEC ? 128 : 512, NV == 1 && VEC ? 8 : 1) block_norm_kernel(const BlockNormParams p, const Steps step, int tpr, int stages) {
    __shared__ __align__(16) float red[2][2][16];
    extern __shared__ __align__(16) uint4 staged[];
    constexpr int NX = kVecN * sizeof(TX) / 16, NR = kVecN * sizeof(TR) / 16;
    constexpr bool HOLD = NV <= 2;
    const int rpb = blockDim.x / tpr, lr = threadIdx.x / tpr, tid = threadIdx.x - lr * tpr, c0 = tid * kVecN, cs = tpr * kVecN;
    const int rows = p.shared ? p.gate_rows : p.R;
    const int64_t run0 = (int64_t)blockIdx.y * rows + (int64_t)blockIdx.x * p.run;
    const int n_rows = min(p.run, rows - (int)blockIdx.x * p.run);
    const bool token = p.act && !p.shared;
    const RowWarps warps(tpr);
    const int vec_pieces = NX * (token ? 2 : 1) + NR;
    const Slots slots{staged + threadIdx.x, NV * vec_pieces};
    if (threadIdx.x < 64) (&red[0][0][0])[threadIdx.x] = 0.f;
    const TX *y = row_of((const TX *)p.y, p.y_st, run0 + lr, c0);
    const TX *gate = token ? row_of((const TX *)p.gate, p.g_st, run0 + lr, c0) : nullptr;
    const TR *res = row_of((const TR *)p.res, p.r_st, run0 + lr, c0);
    TR *res_out = row_of((TR *)p.res_out, p.ro_st, run0 + lr, c0);
    TX *out = row_of((TX *)p.out, p.o_st, run0 + lr, c0);
    auto next_in = [&]() {
        y += step.y, res += step.res;
        if (token) gate += step.gate;
    };
    int left = n_rows - lr;  // the copies' row exists
    auto fetch = [&](int stage) {
        if (left > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (c0 + i * cs >= p.D) continue;
                slots.copy(stage, i * vec_pieces, y + i * cs);
                slots.copy(stage, i * vec_pieces + NX, res + i * cs);
                if (token) slots.copy(stage, i * vec_pieces + NX + NR, gate + i * cs);
            }
        }
        cp_async_commit();
        left -= rpb;
        next_in();
    };
    if (AHEAD)
        for (int g = 0; g + 1 < stages; ++g) fetch(g);
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
            if (c0 + i * cs < p.D) weights(c0 + i * cs, i);
    }
    const float rd = 1.f / (float)p.D;
    int flip = 0, stage = 0;
    __syncthreads();
#pragma unroll 1
    for (int k = lr; k - lr < n_rows; k += rpb, flip ^= 1) {
        const bool live = k < n_rows;
        if (AHEAD) {
            const int ahead = stage == 0 ? stages - 1 : stage - 1;
            slots_arrived(stages - 2), fetch(ahead);
        }
        // (not ahead: the whole row is asked for before its first use)
        uint32_t ny[NV][RowVec<TX, kVecN>::kWords], ng[NV][RowVec<TX, kVecN>::kWords], nr[NV][RowVec<TR, kVecN>::kWords];
        if (!AHEAD) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int o = i * cs, n = p.D - c0 - o;
                if (!(live && n > 0)) continue;
                ld_row<TX, kVecN, VEC>(ny[i], y + o, n);
                ld_row<TR, kVecN, VEC>(nr[i], res + o, n);
                if (token) ld_row<TX, kVecN, VEC>(ng[i], gate + o, n);
            }
            next_in();
        }
        auto take_y = [&](f32x2 (&v)[kPairs], int i) {
            if (AHEAD) slots.get<TX>(v, stage, i * vec_pieces);
            else to_pairs<TX>(v, ny[i]);
        };
        f32x2 s[NV][kPairs];
        float inv = 1.f;
        if (p.post) {
            f32x2 sum2 = pack2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!(live && c0 + i * cs < p.D)) continue;
                take_y(s[i], i);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) sum2 = fma2(s[i][j], s[i][j], sum2);
            }
            const float2 su = unpack2(sum2);
            inv = inv_root(row_sum(su.x + su.y, red[flip][0], warps) * rd + p.eps);
        }
        const f32x2 inv2 = pack2(inv, inv);
        f32x2 sum2 = pack2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = HOLD ? i : 0, o = i * cs, n = p.D - c0 - o;
            if (!(live && n > 0)) continue;
            if (!HOLD) weights(c0 + o, 0);
            f32x2 g[kPairs], r[kPairs];
            if (NV > 2 || !p.post) take_y(s[i], i);  // (four vectors: as stored until here, for the registers)
            if (AHEAD) slots.get<TR>(r, stage, i * vec_pieces + NX);
            else to_pairs<TR>(r, nr[i]);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) s[i][j] = mul2(s[i][j], inv2);
            if (token) {
                if (AHEAD) slots.get<TX>(g, stage, i * vec_pieces + NX + NR);
                else to_pairs<TX>(g, ng[i]);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) s[i][j] = mul2(s[i][j], gate_of(g[j], p.act));
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j) s[i][j] = fma2(s[i][j], w1[at][j], r[j]);
            put<TR, VEC>(res_out + o, s[i], n);
            // (channels past D are zeros: y, residual and weights are loaded so)
#pragma unroll
            for (int j = 0; j < kPairs; ++j) sum2 = fma2(s[i][j], s[i][j], sum2);
        }
        if (p.pre) {
            const float2 su = unpack2(sum2);
            const float q = inv_root(row_sum(su.x + su.y, red[flip][1], warps) * rd + p.eps);
            const f32x2 q2 = pack2(q, q);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int o = i * cs, n = p.D - c0 - o;
                if (!(live && n > 0)) continue;
                if (!HOLD) weights(c0 + o, 0);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) s[i][j] = mul2(mul2(s[i][j], q2), w2[HOLD ? i : 0][j]);
                put<TX, VEC>(out + o, s[i], n);
            }
            out += step.out;
        }
        res_out += step.res_out;
        if (++stage == stages) stage = 0;
    }
}

// A row as a norm's gradient takes it: its values times `power`, a power of two
// that brings their root mean square into fp32's middle where it is far out
// (2^30 either way: past that inv^3 / D becomes a denormal, from 1e13 on, or
// gw S overflows, and gradients that are finite come out as zeros or NaN). The
// norm does not see the factor, and no rounding does. A row whose S passes
// fp32's range is normed to zeros: its power is 0.
struct NormRow {
    float S, inv;  // of the row times its power
    __device__ __forceinline__ NormRow(float S_, float rd, float eps) : S(S_), inv(rsqrtf(S_ * rd + eps)) {}
    __device__ __forceinline__ bool far() const { return inv < 0x1p-30f || inv > 0x1p30f; }
    __device__ __forceinline__ float bring_near() {  // the row's power
        if (!far()) return 1.f;
        const int bits = __float_as_int(inv);
        const bool none = S > FLT_MAX;
        const float power = none ? 0.f : __int_as_float(bits & 0x7f800000);
        inv = none ? 0.f : __int_as_float((bits & 0x7fffff) | 0x3f800000), S = none ? 0.f : S * power * power;
        return power;
    }
};
// The gradient of a norm at channel pair x for the weighted gradient gw = w dy,
// with S = sum x^2, G = sum gw x, inv, added to `more`: both sums lose the
// channel's own terms first, rounded as the sums have them, which cancel
// exactly (they are all there is when one channel dominates its row; scalar
// subtractions, as packed ones may be fused with the products).
struct NormGrad {
    f32x2 k, ke;
    float S, G;
    __device__ __forceinline__ NormGrad(const NormRow &r, float power, float G_, float rd, float eps) : S(r.S), G(G_) {
        const float inv = r.inv * power, a = inv * (r.inv * r.inv * rd), b = inv * (eps * inv * inv);
        k = pack2(a, a), ke = pack2(b, b);
    }
    __device__ __forceinline__ f32x2 at(f32x2 x, f32x2 gw, f32x2 more) const {
        const float2 xx = unpack2(mul2(x, x)), gx = unpack2(mul2(gw, x));
        const f32x2 so = pack2(__fsub_rn(S, xx.x), __fsub_rn(S, xx.y)), go = pack2(__fsub_rn(gx.x, G), __fsub_rn(gx.y, G));
        return fma2(k, fma2(gw, so, mul2(x, go)), fma2(ke, gw, more));
    }
};
// times a row's power; what is not finite goes with a row of zeros
__device__ __forceinline__ void scale_row(f32x2 (&v)[kPairs], float power) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) v[j] = power == 0.f ? pack2(0.f, 0.f) : mul2(v[j], pack2(power, power));
}

// Runs as in the forward. A thread keeps its channels' sums, in registers with
// up to two vectors a thread, else in its own slots of shared memory. A row is
// read from its slots once a phase rather than held.
template <typename TX, typename TR, int NV, bool VEC, bool AHEAD, bool TOKEN>
__global__ void __launch_bounds__(NV == 1 && VEC && !TOKEN ? 128 : 512, NV == 1 && VEC && !TOKEN ? 5 : 1) block_norm_bwd_kernel(const BlockNormBwdParams p, const Steps step, int tpr, int stages) {
    __shared__ __align__(16) float4 red3[2][16];
    __shared__ __align__(16) float red1[2][16];
    extern __shared__ __align__(16) uint4 staged[];
    constexpr int NX = kVecN * sizeof(TX) / 16, NR = kVecN * sizeof(TR) / 16;
    constexpr bool HOLD = NV <= 2;  // sums and weights in registers
    constexpr int kKept = HOLD ? 0 : NV * 2 * kPairs / 2, kHeld = HOLD ? NV : 1;  // 16-byte slots a thread of sums
    const int rpb = blockDim.x / tpr, lr = threadIdx.x / tpr, tid = threadIdx.x - lr * tpr, c0 = tid * kVecN, cs = tpr * kVecN;
    const int rows = p.shared ? p.gate_rows : p.R;
    const int64_t run0 = (int64_t)blockIdx.y * rows + (int64_t)blockIdx.x * p.run, row0 = run0 + lr;
    const int n_rows = min(p.run, rows - (int)blockIdx.x * p.run);
    const RowWarps warps(tpr);
    // y, dres, then s and dout with pre, then the gate
    const int n_dres = p.dres ? NR : 0, n_pre = p.pre ? NR + NX : 0, vec_pieces = NX + n_dres + n_pre + (TOKEN ? NX : 0);
    const Slots slots{staged + kKept * blockDim.x + threadIdx.x, NV * vec_pieces};
    auto kept = [&](int i, int q, int j) -> f32x2 & {
        return reinterpret_cast<f32x2 *>(staged)[((i * 2 + q) * kPairs + j) * blockDim.x + threadIdx.x];
    };
    const f32x2 zero = pack2(0.f, 0.f);
    for (int e = threadIdx.x; e < 32; e += blockDim.x) (&red3[0][0])[e] = make_float4(0.f, 0.f, 0.f, 0.f), (&red1[0][0])[e] = 0.f;
    const TX *y = row_of((const TX *)p.y, p.y_st, row0, c0), *dout = row_of((const TX *)p.dout, p.do_st, row0, c0);
    const TX *gate = TOKEN ? row_of((const TX *)p.gate, p.g_st, row0, c0) : nullptr;
    const TR *s = row_of((const TR *)p.s, p.s_st, row0, c0), *dres = row_of((const TR *)p.dres, p.dr_st, row0, c0);
    TX *dy = row_of((TX *)p.dy, p.dy_st, row0, c0), *dgate = TOKEN ? row_of((TX *)p.dgate, p.dg_st, row0, c0) : nullptr;
    TR *ds_out = row_of((TR *)p.ds, p.ds_st, row0, c0);
    auto next_in = [&]() {
        y += step.y, dres += step.dres;
        if (p.pre) s += step.s, dout += step.dout;
        if (TOKEN) gate += step.gate;
    };
    int left = n_rows - lr;  // the copies' row exists
    auto fetch = [&](int stage) {
        if (left > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = i * cs, o = i * vec_pieces;
                if (c0 + c >= p.D) continue;
                slots.copy(stage, o, y + c);
                if (p.dres) slots.copy(stage, o + NX, dres + c);
                if (p.pre) slots.copy(stage, o + NX + n_dres, s + c), slots.copy(stage, o + NX + n_dres + NR, dout + c);
                if (TOKEN) slots.copy(stage, o + NX + n_dres + n_pre, gate + c);
            }
        }
        cp_async_commit();
        left -= rpb;
        next_in();
    };
    if (AHEAD)
        for (int g = 0; g + 1 < stages; ++g) fetch(g);
    f32x2 w1[kHeld][kPairs], w2[kHeld][kPairs], sa[kHeld][kPairs], sr[kHeld][kPairs];  // as in the forward; the sums
    auto weights = [&](int c, int at) {
        const int n = p.D - c;
        get_factor<VEC>(w1[at], p.scale, p.post, p.alpha, c, n);
        get<float, VEC>(w2[at], p.pre ? p.pre + c : nullptr, n);
        if (!TOKEN && p.shared) {
            f32x2 g[kPairs];
            get<TX, VEC>(g, (const TX *)p.gate + (int64_t)blockIdx.y * p.g_st + c, n);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) w1[at][j] = mul2(w1[at][j], gate_of(g[j], p.act));
        }
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (HOLD) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) w1[i % kHeld][j] = w2[i % kHeld][j] = sa[i % kHeld][j] = sr[i % kHeld][j] = zero;
            if (c0 + i * cs < p.D) weights(c0 + i * cs, i % kHeld);
        } else {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) kept(i, 0, j) = kept(i, 1, j) = zero;
        }
    }
    const float rd = 1.f / (float)p.D;
    int flip = 0, stage = 0;
    __syncthreads();
#pragma unroll 1
    for (int k = lr; k - lr < n_rows; k += rpb, flip ^= 1) {
        const bool live = k < n_rows;
        if (AHEAD) {
            const int ahead = stage == 0 ? stages - 1 : stage - 1;
            slots_arrived(stages - 2), fetch(ahead);
        }
        bool far = false;  // the row's powers (NormRow) are not one
        float of_s = 1.f, of_y = 1.f;
        auto take_y = [&](f32x2 (&v)[kPairs], int i, int n) {
            if (AHEAD) slots.get<TX>(v, stage, i * vec_pieces);
            else get<TX, VEC>(v, y + i * cs, n);
            if (!AHEAD && far) scale_row(v, of_y);
        };
        auto take_s = [&](f32x2 (&vs)[kPairs], f32x2 (&vd)[kPairs], int i, int n) {  // and dout
            const int o = i * vec_pieces + NX + n_dres;
            if (AHEAD) slots.get<TR>(vs, stage, o), slots.get<TX>(vd, stage, o + NR);
            else get<TR, VEC>(vs, s + i * cs, n), get<TX, VEC>(vd, dout + i * cs, n);
            if (!AHEAD && far) scale_row(vs, of_s);
        };
        f32x2 a = zero, b = zero, d = zero;  // of s^2, pre dout s, y^2
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * cs, at = HOLD ? i : 0;
            if (!(live && c < p.D)) continue;
            if (!HOLD) weights(c, 0);
            f32x2 hs[kPairs], hd[kPairs], hy[kPairs];
            if (p.pre) {
                take_s(hs, hd, i, p.D - c);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) a = fma2(hs[j], hs[j], a), b = fma2(mul2(hd[j], w2[at][j]), hs[j], b);
            }
            if (p.post) {
                take_y(hy, i, p.D - c);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) d = fma2(hy[j], hy[j], d);
            }
        }
        const float2 fa = unpack2(a), fb = unpack2(b), fd = unpack2(d);
        float v[3] = {fa.x + fa.y, fb.x + fb.y, fd.x + fd.y};
        row_sums3(v, red3[flip], warps);
        NormRow row_s(v[0], rd, p.eps), row_y(v[2], rd, p.eps);
        far = (p.pre && row_s.far()) || (p.post && row_y.far());
        if (far) {
            if (p.pre) of_s = row_s.bring_near();
            if (p.post) of_y = row_y.bring_near();
            v[1] = of_s == 0.f ? 0.f : v[1] * of_s;
            if (AHEAD) {
#pragma unroll 1
                for (int i = 0; i < NV; ++i) {
                    const int o = i * vec_pieces;
                    if (p.pre) slots.scale<TR>(stage, o + NX + n_dres, NR, of_s);
                    slots.scale<TX>(stage, o, NX, of_y);
                }
            }
        }
        const NormGrad ns(row_s, of_s, v[1], rd, p.eps);
        const float inv_y = p.post ? row_y.inv : 1.f;
        const f32x2 iy2 = pack2(inv_y, inv_y), is2 = pack2(row_s.inv, row_s.inv);
        f32x2 e[kHeld][kPairs], g2 = zero;  // k post f ds, the gradient behind y's norm; of e y
        // The stream's gradient and what follows from it. again: e alone (rows
        // whose e is not held).
        auto stream = [&](int i, int n, auto form) {
            constexpr bool again = decltype(form)::value;
            const int at = HOLD ? i : 0;
            f32x2 ds[kPairs], hy[kPairs], hg[kPairs];
            if (p.dres) {
                if (AHEAD) slots.get<TR>(ds, stage, i * vec_pieces + NX);
                else get<TR, VEC>(ds, dres + i * cs, n);
            } else {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) ds[j] = zero;
            }
            if (p.pre) {
                f32x2 hs[kPairs], hd[kPairs];
                take_s(hs, hd, i, n);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    ds[j] = ns.at(hs[j], mul2(hd[j], w2[at][j]), ds[j]);
                    if (!again) {
                        const f32x2 sn = mul2(hs[j], is2);
                        if constexpr (HOLD) sr[at][j] = fma2(hd[j], sn, sr[at][j]);
                        else kept(i, 1, j) = fma2(hd[j], sn, kept(i, 1, j));
                    }
                }
            }
            if (!again) {
                put<TR, VEC>(ds_out + i * cs, ds, n);
                take_y(hy, i, n);
            }
            if (TOKEN) {
                if (AHEAD) slots.get<TX>(hg, stage, i * vec_pieces + NX + n_dres + n_pre);
                else get<TX, VEC>(hg, gate + i * cs, n);
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                f32x2 dsf = ds[j], df;
                if (TOKEN) dsf = mul2(ds[j], gate_of(hg[j], p.act, df));
                e[at][j] = mul2(dsf, w1[at][j]);
                if (!again) {
                    const f32x2 yn = mul2(hy[j], iy2);
                    if (TOKEN) hg[j] = mul2(mul2(mul2(ds[j], w1[at][j]), yn), df);
                    g2 = fma2(e[at][j], hy[j], g2);
                    if constexpr (HOLD) sa[at][j] = fma2(dsf, yn, sa[at][j]);
                    else kept(i, 0, j) = fma2(dsf, yn, kept(i, 0, j));
                }
            }
            if (TOKEN && !again) put<TX, VEC>(dgate + i * cs, hg, n);
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * cs;
            if (!(live && c < p.D)) continue;
            if (!HOLD) weights(c, 0);
            stream(i, p.D - c, std::false_type());
        }
        float ge = 0.f;
        if (p.post) {
            const float2 fg = unpack2(g2);
            ge = row_sum(fg.x + fg.y, red1[flip], warps);
        }
        const NormGrad ny(row_y, of_y, ge, rd, p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * cs, at = HOLD ? i : 0;
            if (!(live && c < p.D)) continue;
            if (!HOLD) weights(c, 0), stream(i, p.D - c, std::true_type());
            if (p.post) {
                f32x2 hy[kPairs];
                take_y(hy, i, p.D - c);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) e[at][j] = ny.at(hy[j], e[at][j], zero);
            }
            put<TX, VEC>(dy + i * cs, e[at], p.D - c);
        }
        if (!AHEAD) next_in();
        dy += step.dy, ds_out += step.ds;
        if (TOKEN) dgate += step.dgate;
        if (++stage == stages) stage = 0;
    }
    float *part = p.part + (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * rpb + lr) * 2 * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * cs, at = HOLD ? i : 0;
        if (c >= p.D) continue;
        if constexpr (!HOLD) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) sa[0][j] = kept(i, 0, j), sr[0][j] = kept(i, 1, j);
        }
        put<float, VEC>(part + c, sa[at], p.D - c);
        put<float, VEC>(part + p.D + c, sr[at], p.D - c);
    }
}

// Sums over the runs in a fixed order: 8 columns a CTA (a row's 32 bytes), 32
// threads a column.
constexpr int kSumX = 8, kSumY = 32;
__device__ __forceinline__ float2 column_sums(const float *in, int64_t parts, int D, int c) {
    __shared__ float red[kSumY][kSumX][2];
    const int x = threadIdx.x % kSumX, y = threadIdx.x / kSumX;
    float a = 0.f, b = 0.f;
    if (c < D) {
#pragma unroll 8
        for (int64_t q = y; q < parts; q += kSumY) a += in[q * 2 * D + c], b += in[q * 2 * D + D + c];
    }
    red[y][x][0] = a, red[y][x][1] = b;
    __syncthreads();
    if (y == 0) {
#pragma unroll
        for (int i = 1; i < kSumY; ++i) a += red[i][x][0], b += red[i][x][1];
    }
    return make_float2(a, b);
}
// the gradient of sequence q's gate row at channel c from its sum of ds y
// inv_y; returns the factor of the sum that the weights' gradients take
template <typename TX>
__device__ __forceinline__ float gate_gradient(const BlockNormBwdParams &p, int64_t q, int c, float sum) {
    const float g = (float)((const TX *)p.gate)[q * p.g_st + c];
    f32x2 df2;
    const float2 f = unpack2(gate_of(pack2(g, g), p.act, df2));
    const float w = p.alpha * (p.scale ? p.scale[c] : 1.f) * (p.post ? p.post[c] : 1.f);
    ((TX *)p.dgate)[q * p.dg_st + c] = to_type<TX>(sum * w * unpack2(df2).x);
    return f.x;
}
// of one sequence (blockIdx.y): its gate row's gradient, and its share of the sums
template <typename TX>
__global__ void __launch_bounds__(kSumX *kSumY) block_norm_sequences_kernel(const BlockNormBwdParams p, int parts) {
    const int c = blockIdx.x * kSumX + threadIdx.x % kSumX;
    const int64_t q = blockIdx.y;
    const float2 v = column_sums(p.part + q * parts * 2 * p.D, parts, p.D, c);
    if (threadIdx.x >= kSumX || c >= p.D) return;
    p.part2[q * 2 * p.D + c] = v.x * gate_gradient<TX>(p, q, c, v.x);
    p.part2[q * 2 * p.D + p.D + c] = v.y;
}
// of all of them; a single sequence's shared gate row gets its gradient here
template <typename TX>
__global__ void __launch_bounds__(kSumX *kSumY) block_norm_reduce_kernel(const BlockNormBwdParams p, const float *in, int64_t parts) {
    const int c = blockIdx.x * kSumX + threadIdx.x % kSumX;
    float2 v = column_sums(in, parts, p.D, c);
    if (threadIdx.x >= kSumX || c >= p.D) return;
    if (p.shared && in == p.part) v.x *= gate_gradient<TX>(p, 0, c, v.x);
    if (p.dpost) p.dpost[c] = v.x * (p.alpha * (p.scale ? p.scale[c] : 1.f));
    if (p.dscale) p.dscale[c] = v.x * (p.alpha * (p.post ? p.post[c] : 1.f));
    if (p.dpre) p.dpre[c] = v.y;
}

// Stages of `row` bytes that leave `ctas` CTAs a SM: two or three.
constexpr int kMostSmem = 216 * 1024;
int stages_for(int row, int kept, int ctas) { return (3 * row + kept) * ctas <= kMostSmem ? 3 : 2; }
// (the limit is the kernel's, not the call's: a smaller call's own size would lower it under another thread's launch)
template <class K>
cudaError_t with_smem(K *k, int smem) {
    if (smem <= 40 * 1024) return cudaSuccess;  // 48 KB with the static part
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
}
template <typename TX, typename TR>
cudaError_t norm_nv(BlockNormParams p, cudaStream_t st) {
    const RowShape s = row_shape(p);
    const Runs r = runs_of(p.R, p.gate_rows, s);
    p.runs = r.n, p.run = r.len;
    const int nt = s.tpr * s.rpb, token = p.act && !p.shared;
    const dim3 grid(p.runs, p.shared ? p.R / p.gate_rows : 1);
    auto run = [&](auto nv, auto vec, auto ahead) -> cudaError_t {
        auto *k = block_norm_kernel<TX, TR, nv(), vec(), ahead()>;
        const int row = ahead() ? nv() * kVecN * ((int)sizeof(TX) * (1 + token) + (int)sizeof(TR)) * nt : 0;
        const int stages = stages_for(row, 0, 1024 / nt < 4 ? 1024 / nt : 4), smem = ahead() ? stages * row : 0;
        const cudaError_t e = with_smem(k, smem);
        if (e != cudaSuccess) return e;
        const Steps step{p.y_st * s.rpb, p.r_st * s.rpb, p.g_st * s.rpb, p.o_st * s.rpb, p.ro_st * s.rpb};
        k<<<grid, nt, smem, st>>>(p, step, s.tpr, stages);
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
cudaError_t norm_bwd_nv(BlockNormBwdParams p, cudaStream_t st) {
    const RowShape s = row_shape(p);
    const Runs runs = runs_of(p.R, p.gate_rows, s);
    p.runs = runs.n, p.run = runs.len;
    const int nt = s.tpr * s.rpb;
    const bool token = p.act && !p.shared;
    const dim3 grid(p.runs, p.shared ? p.R / p.gate_rows : 1);
    auto run = [&](auto nv, auto vec, auto ahead, auto tok) -> cudaError_t {
        auto *k = block_norm_bwd_kernel<TX, TR, nv(), vec(), ahead(), tok()>;
        const int kept = nv() > 2 ? nv() * 2 * kPairs * 8 * nt : 0, x = sizeof(TX), r = sizeof(TR);
        const int row = ahead() ? nv() * kVecN * (x * (1 + tok() + (p.pre ? 1 : 0)) + r * ((p.dres ? 1 : 0) + (p.pre ? 1 : 0))) * nt : 0;
        const int stages = stages_for(row, kept, nt > 256 ? 1 : nt > 128 ? 2 : 4), smem = kept + (ahead() ? stages * row : 0);
        const cudaError_t e = with_smem(k, smem);
        if (e != cudaSuccess) return e;
        Steps step{};
        step.y = p.y_st * s.rpb, step.gate = p.g_st * s.rpb, step.s = p.s_st * s.rpb, step.dout = p.do_st * s.rpb;
        step.dres = p.dr_st * s.rpb, step.dy = p.dy_st * s.rpb, step.ds = p.ds_st * s.rpb, step.dgate = p.dg_st * s.rpb;
        k<<<grid, nt, smem, st>>>(p, step, s.tpr, stages);
        return cudaGetLastError();
    };
    auto by_gate = [&](auto nv, auto vec, auto ahead) {
        return token ? run(nv, vec, ahead, std::true_type()) : run(nv, vec, ahead, std::false_type());
    };
    auto by_vectors = [&](auto vec) {
        if (s.nv == 1) return by_gate(std::integral_constant<int, 1>(), vec, vec);
        // (two rows of five tensors have to fit: not those of 8192 fp32 channels)
        const int x = sizeof(TX), r = sizeof(TR), row = kVecN * 2 * nt * (x * (1 + token + (p.pre ? 1 : 0)) + r * ((p.dres ? 1 : 0) + (p.pre ? 1 : 0)));
        if (s.nv == 2 && 2 * row > kMostSmem) return by_gate(std::integral_constant<int, 2>(), vec, std::false_type());
        if (s.nv == 2) return by_gate(std::integral_constant<int, 2>(), vec, vec);
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

int64_t block_norm_parts(int R, int D, int gate_rows) {
    const int64_t a = runs_of(R, gate_rows, row_shape(D, false)).parts, b = runs_of(R, gate_rows, row_shape(D, true)).parts;
    return a > b ? a : b;
}

cudaError_t launch_block_norm_bwd(const BlockNormBwdParams &p, cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (p.y_bf16) return p.r_bf16 ? norm_bwd_nv<bf, bf>(p, st) : norm_bwd_nv<bf, float>(p, st);
    return p.r_bf16 ? norm_bwd_nv<float, bf>(p, st) : norm_bwd_nv<float, float>(p, st);
}

cudaError_t launch_block_norm_sequences(const BlockNormBwdParams &p, cudaStream_t st) {
    const RowShape s = row_shape(p);
    const int parts = runs_of(p.R, p.gate_rows, s).n * s.rpb;
    const dim3 grid((p.D + kSumX - 1) / kSumX, p.R / p.gate_rows);
    if (p.y_bf16) block_norm_sequences_kernel<__nv_bfloat16><<<grid, kSumX * kSumY, 0, st>>>(p, parts);
    else block_norm_sequences_kernel<float><<<grid, kSumX * kSumY, 0, st>>>(p, parts);
    return cudaGetLastError();
}

bool block_norm_by_sequence(const BlockNormBwdParams &p) { return p.shared && p.R > p.gate_rows; }

cudaError_t launch_block_norm_reduce(const BlockNormBwdParams &p, cudaStream_t st) {
    const bool joined = block_norm_by_sequence(p);
    const int64_t parts = p.R == 0 ? 0 : joined ? p.R / p.gate_rows : runs_of(p.R, p.gate_rows, row_shape(p)).parts;
    const float *in = joined ? p.part2 : p.part;
    const unsigned grid = (p.D + kSumX - 1) / kSumX;
    if (p.y_bf16) block_norm_reduce_kernel<__nv_bfloat16><<<grid, kSumX * kSumY, 0, st>>>(p, in, parts);
    else block_norm_reduce_kernel<float><<<grid, kSumX * kSumY, 0, st>>>(p, in, parts);
    return cudaGetLastError();
}

}  // namespace gdn

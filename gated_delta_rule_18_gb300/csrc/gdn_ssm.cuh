// gdn_ssm.cuh -- what the selective scan's kernels share: packed fp32
// arithmetic, the token functions and sequence bounds.
#pragma once

#include "gdn_layer.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------- packed fp32 pairs --------
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float ex2f(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcpf(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 a) {
    const float2 v = unpack2(a);
    return pack2(ex2f(v.x), ex2f(v.y));
}
// ---------------------------------------------------- token functions -------
// The functions below take the two halves of a pair in scalar instructions:
// their constants are then immediates, where a packed instruction would need
// each in a register pair of its own.
//
// 1 / a and 1 / b from one reciprocal (its rate is half the exponential's);
// |a b| has to stay finite.
__device__ __forceinline__ float2 rcp2(float a, float b) {
    const float r = rcpf(a * b);
    return make_float2(r * b, r * a);
}
// maximum that keeps NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// softplus(v) = max(v, 0) + log1p(e), e = exp(-|v|) <= 1, by
//   log1p(e) = 2 artanh(s), s = e / (2 + e) <= 1/3, artanh(s) = s P(s^2).
// P interpolates artanh(sqrt t) / sqrt t on [0, 1/9] at five Chebyshev points
// (relative error of log1p 8e-9); no cancellation for small e, as log(1 + e) has.
constexpr float SP1 = 0.333331608f, SP2 = 0.200122976f, SP3 = 0.139825789f, SP4 = 0.140788892f;
__device__ __forceinline__ float log1p_of(float e, float r) {  // r = 1 / (2 + e)
    const float s = e * r, t = s * s;
    float p = fmaf(SP4, t, SP3);
    p = fmaf(p, t, SP2);
    p = fmaf(p, t, SP1);
    p = fmaf(p, t, 1.f);
    return (s + s) * p;
}
__device__ __forceinline__ float2 softplus2(float2 v) {
    // (a NaN of one half must reach its own result and not the shared reciprocal)
    const float e0 = ex2f(fmaxf(-fabsf(v.x) * kLog2e, -200.f)), e1 = ex2f(fmaxf(-fabsf(v.y) * kLog2e, -200.f));
    const float2 r = rcp2(e0 + 2.f, e1 + 2.f);
    return make_float2(log1p_of(e0, r.x) + max_nan(v.x, 0.f), log1p_of(e1, r.y) + max_nan(v.y, 0.f));
}
// sigmoid of a pair by e = exp(-|x|) <= 1: 1 / (1 + e), and e times that for
// x < 0, so that it goes to 0 with e and x sigmoid(x) to -0 for the lowest x
// (a NaN takes no part in e, nor so in the shared reciprocal, and comes back
// where the caller multiplies by x).
__device__ __forceinline__ float2 sigmoid2(float2 x) {
    const float e0 = ex2f(fmaxf(-fabsf(x.x) * kLog2e, -200.f)), e1 = ex2f(fmaxf(-fabsf(x.y) * kLog2e, -200.f));
    const float2 r = rcp2(e0 + 1.f, e1 + 1.f);
    return make_float2(x.x < 0.f ? e0 * r.x : r.x, x.y < 0.f ? e1 * r.y : r.y);
}

// ------------------------------------------------------------ sequences -----
// The line of tokens a chunk lies on, and the sequence it is in: `end` is the
// first token past the sequence. Bounds are clamped to the line, so a
// malformed cu cannot send an access out of range.
struct SsmSeq {
    int seg, end;
    bool starts;  // the token is the sequence's first
};
__device__ __forceinline__ SsmSeq ssm_find(const int32_t *cu, int n_seq, int T, int line, int t) {
    SsmSeq q;
    if (!cu) {
        q.seg = line, q.end = T, q.starts = t == 0;
        return q;
    }
    int lo = 0, hi = n_seq - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (__ldg(cu + m) <= t) lo = m;
        else hi = m - 1;
    }
    q.seg = lo;
    q.starts = __ldg(cu + lo) == t;
    q.end = min(max(__ldg(cu + lo + 1), t + 1), T);
    return q;
}
// the sequence that begins at t = q.end
__device__ __forceinline__ void ssm_next(SsmSeq &q, const int32_t *cu, int n_seq, int T, int t) {
    if (!cu) return;
    while (q.seg + 1 < n_seq && __ldg(cu + q.seg + 1) <= t) ++q.seg;
    q.end = min(max(__ldg(cu + q.seg + 1), t + 1), T);
}
__device__ __forceinline__ void ssm_check_cu(const int32_t *cu, int n_seq, int T, int *err) {
    int bad = 0;
    for (int s = threadIdx.x; s < n_seq; s += blockDim.x) bad |= cu[s + 1] < cu[s];
    if (threadIdx.x == 0) bad |= cu[0] != 0 || cu[n_seq] != T;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *err = bad ? 1 : 0;
}

// ------------------------------------------------------------ staging -------
// `rows` rows of CH channels from channel c0 on into shared memory (row
// stride CH), by 16-byte asynchronous copies. Channels past D and rows past
// `rows` are zeros (a pair's halves share a reciprocal, a warp's channels the
// sums of dB and dC). NT threads take part.
template <typename T, int CH, int TS, int NT>
__device__ __forceinline__ void ssm_copy_tile(T *dst, const T *src, int64_t stride, int rows, int c0, int D) {
    constexpr int VE = 16 / sizeof(T), kCopies = TS * CH / VE;
#pragma unroll
    for (int i = 0; i < (kCopies + NT - 1) / NT; ++i) {
        const int e = threadIdx.x + i * NT, r = e / (CH / VE), c = e % (CH / VE) * VE;
        const bool in = r < rows && c0 + c < D;
        if (kCopies % NT == 0 || e < kCopies) cp_async16(dst + r * CH + c, in ? src + r * stride + c0 + c : src, in ? 16 : 0);
    }
}
// The same for rows that start on any element: loaded into registers, by
// pairs of channels, and stored when their place is free.
template <typename T, int CH, int TS, int NT>
struct SsmTile {
    static constexpr int kPairs = TS * CH / 2, kLoads = (kPairs + NT - 1) / NT, KW = RowVec<T, 2>::kWords;
    uint32_t w[kLoads][KW];
    __device__ __forceinline__ void load(const T *src, int64_t stride, int rows, int c0, int D) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int e = threadIdx.x + i * NT, r = e / (CH / 2), c = c0 + e % (CH / 2) * 2;
#pragma unroll
            for (int k = 0; k < KW; ++k) w[i][k] = 0u;
            if ((kPairs % NT == 0 || e < kPairs) && r < rows && c < D) ld_row<T, 2, false>(w[i], src + r * stride + c, D - c);
        }
    }
    __device__ __forceinline__ void store(T *dst) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int e = threadIdx.x + i * NT;
            if (kPairs % NT == 0 || e < kPairs) st_row<T, 2, true>(dst + 2 * e, w[i], 2);
        }
    }
};
// The (B, C) rows of TS tokens, [TS][2][NP] fp32 in shared memory: loaded as
// stored into registers by fetch, converted where they are staged.
template <typename T, int NP, int TS, int NT>
struct SsmBc {
    static constexpr int kVals = TS * 2 * NP, V = kVals / NT < 4 ? kVals / NT : 4, kLoads = kVals / (NT * V);
    uint32_t w[kLoads][RowVec<T, V>::kWords];
    template <bool WITH_C>
    __device__ __forceinline__ void fetch(const T *bg, int64_t b_st, const T *cg, int64_t c_st, int rows, int N, bool vec) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int e = (threadIdx.x + i * NT) * V, r = e / (2 * NP), k = e % (2 * NP), n = k % NP;
#pragma unroll
            for (int j = 0; j < RowVec<T, V>::kWords; ++j) w[i][j] = 0u;
            if (r < rows && n < N && (WITH_C || k < NP)) {
                const T *at = k < NP ? bg + r * b_st + n : cg + r * c_st + n;
                if (vec) ld_row<T, V, true>(w[i], at, N - n);
                else ld_row<T, V, false>(w[i], at, N - n);
            }
        }
    }
    __device__ __forceinline__ void stage(float *dst) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            float f[V];
            words_to_f<T, V>(f, w[i]);
#pragma unroll
            for (int k = 0; k < V; ++k) dst[(threadIdx.x + i * NT) * V + k] = f[k];
        }
    }
};

// ------------------------------------------------------------- states -------
// Q neighbouring states of a channel, in pairs; swap = 1: neighbouring quads
// change places
template <int Q>
__device__ __forceinline__ void ld_states(f32x2 (&v)[Q / 2], const float *p, int n, bool wide, int swap = 0) {
#pragma unroll
    for (int j = 0; j < Q / 4; ++j) {
        const int k = 4 * (j ^ swap);
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (wide) {
            if (k < n) f = *reinterpret_cast<const float4 *>(p + k);
        } else {
            if (k < n) f.x = p[k];
            if (k + 1 < n) f.y = p[k + 1];
            if (k + 2 < n) f.z = p[k + 2];
            if (k + 3 < n) f.w = p[k + 3];
        }
        v[2 * j] = pack2(f.x, f.y), v[2 * j + 1] = pack2(f.z, f.w);
    }
}
template <int Q>
__device__ __forceinline__ void st_states(float *p, const f32x2 (&v)[Q / 2], int n, bool wide, int swap = 0) {
#pragma unroll
    for (int j = 0; j < Q / 4; ++j) {
        const int k = 4 * (j ^ swap);
        const float2 a = unpack2(v[2 * j]), b = unpack2(v[2 * j + 1]);
        if (wide) {
            if (k < n) *reinterpret_cast<float4 *>(p + k) = make_float4(a.x, a.y, b.x, b.y);
        } else {
            if (k < n) p[k] = a.x;
            if (k + 1 < n) p[k + 1] = a.y;
            if (k + 2 < n) p[k + 2] = b.x;
            if (k + 3 < n) p[k + 3] = b.y;
        }
    }
}
// of the two channels at p and p + ld; on: which of them exist
template <int Q>
__device__ __forceinline__ void ld_pair(f32x2 (&v)[2][Q / 2], const float *p, int ld, int n, bool wide,
                                        const bool (&on)[2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) ld_states<Q>(v[k], p + k * ld, on[k] ? n : 0, wide);
}
template <int Q>
__device__ __forceinline__ void st_pair(float *p, const f32x2 (&v)[2][Q / 2], int ld, int n, bool wide,
                                        const bool (&on)[2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) st_states<Q>(p + k * ld, v[k], on[k] ? n : 0, wide);
}

// States a lane and lanes a channel: NP = Q LN >= N.
template <class F>
cudaError_t ssm_by_states(int N, F &&f) {
    if (N <= 8) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
    if (N <= 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
    if (N <= 32) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 2>());
    if (N <= 64) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 4>());
    return f(std::integral_constant<int, 16>(), std::integral_constant<int, 8>());
}
inline int ssm_np(int N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : N <= 64 ? 64 : 128; }
inline int ssm_lanes(int N) { return N <= 16 ? 1 : N <= 32 ? 2 : N <= 64 ? 4 : 8; }

}  // namespace gdn

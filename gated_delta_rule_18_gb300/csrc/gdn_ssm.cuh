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
// (relative error 4e-9); no cancellation for small e, as log(1 + e) has.
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
// sigmoid of a pair: 1 / (1 + exp(-x)); exp(-x) is held under 2^60 for rcp2,
// where the sigmoid is under 2^-60.
__device__ __forceinline__ float2 sigmoid2(float2 x) {
    return rcp2(ex2f(fminf(x.x * -kLog2e, 60.f)) + 1.f, ex2f(fminf(x.y * -kLog2e, 60.f)) + 1.f);
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

// gdn_ssm.cu -- the selective state-space scan. Per channel d and state n,
//   delta = softplus(dt + bias),  a = exp(delta A),
//   h <- a h + delta x B_n,  y = sum_n C_n h + D x,  out = y silu(z),
// for whole sequences (dense or packed) and for single tokens with the
// states in a pool. h is fp32 throughout.
//
// A group of LN lanes holds a channel's states, four a lane; y crosses the
// group by shuffles.
#include "gdn_layer.cuh"

namespace gdn {
namespace {

__device__ __forceinline__ float softplus_f(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

constexpr float kLog2e = 1.4426950408889634f;

// One CTA: 128 / LN channels of one sequence, token by token.
template <typename T, int LN>
__global__ void __launch_bounds__(128) ssm_scan_kernel(const SsmParams p) {
    const int seq = blockIdx.y;
    const int d = blockIdx.x * (128 / LN) + threadIdx.x / LN, n0 = threadIdx.x % LN * 4;
    const bool in = d < p.D;
    if (p.err && blockIdx.x == 0 && seq == 0) {
        int bad = 0;
        for (int s = threadIdx.x; s < p.n_seq; s += 128) bad |= p.cu[s + 1] < p.cu[s];
        if (threadIdx.x == 0) bad |= p.cu[0] != 0 || p.cu[p.n_seq] != p.T;
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *p.err = bad;
    }
    const int row = p.cu ? 0 : seq;
    const int t0 = p.cu ? min(max(p.cu[seq], 0), p.T) : 0, t1 = p.cu ? min(p.cu[seq + 1], p.T) : p.T;
    float a2[4], h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool on = in && n0 + j < p.N;
        a2[j] = on ? p.A[(int64_t)d * p.N + n0 + j] * kLog2e : 0.f;
        h[j] = on && p.h0 ? p.h0[((int64_t)seq * p.D + d) * p.N + n0 + j] : 0.f;
    }
    const float dv = in && p.Dv ? p.Dv[d] : 0.f, bias = in && p.dt_bias ? p.dt_bias[d] : 0.f;
    for (int t = t0; t < t1; ++t) {
        const float x = in ? ldf((const T *)p.x + row * p.x_sb + t * p.x_st + d) : 0.f;
        float dl = in ? ldf((const T *)p.dt + row * p.dt_sb + t * p.dt_st + d) + bias : 0.f;
        if (p.softplus) dl = softplus_f(dl);
        const float u = dl * x;
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool on = n0 + j < p.N;
            const float b = on ? ldf((const T *)p.bm + row * p.bm_sb + t * p.bm_st + n0 + j) : 0.f;
            const float c = on ? ldf((const T *)p.cm + row * p.cm_sb + t * p.cm_st + n0 + j) : 0.f;
            h[j] = fmaf(exp2f(dl * a2[j]), h[j], u * b);
            y = fmaf(h[j], c, y);
        }
#pragma unroll
        for (int o = LN / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (in && threadIdx.x % LN == 0) {
            y = fmaf(dv, x, y);
            if (p.z) {
                const float z = ldf((const T *)p.z + row * p.z_sb + t * p.z_st + d);
                y *= z * sigmoid_f(z);
            }
            ((T *)p.out)[row * p.o_sb + t * p.o_st + d] = to_type<T>(y);
        }
    }
    if (p.h_final) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (in && n0 + j < p.N) p.h_final[((int64_t)seq * p.D + d) * p.N + n0 + j] = h[j];
    }
}

// One token of each request: the state is read, updated and written back.
template <typename T, int LN>
__global__ void __launch_bounds__(128) ssm_step_kernel(const SsmStepParams p) {
    const int i = blockIdx.y;
    const int d = blockIdx.x * (128 / LN) + threadIdx.x / LN, n0 = threadIdx.x % LN * 4;
    const bool in = d < p.D;
    const int slot = p.slots ? p.slots[i] : i;
    if (slot < 0 || slot >= p.n_slots) {  // a padding row
        if (in && n0 == 0) ((T *)p.out)[i * p.o_st + d] = to_type<T>(0.f);
        return;
    }
    float *state = p.state + ((int64_t)slot * p.D + d) * p.N + n0;
    const float x = in ? ldf((const T *)p.x + i * p.x_st + d) : 0.f;
    float dl = in ? ldf((const T *)p.dt + i * p.dt_st + d) + (p.dt_bias ? p.dt_bias[d] : 0.f) : 0.f;
    if (p.softplus) dl = softplus_f(dl);
    const float u = dl * x;
    float y = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (!in || n0 + j >= p.N) continue;
        const float b = ldf((const T *)p.bm + i * p.bm_st + n0 + j), c = ldf((const T *)p.cm + i * p.cm_st + n0 + j);
        const float h = fmaf(exp2f(dl * (p.A[(int64_t)d * p.N + n0 + j] * kLog2e)), state[j], u * b);
        state[j] = h;
        y = fmaf(h, c, y);
    }
#pragma unroll
    for (int o = LN / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (in && n0 == 0) {
        if (p.Dv) y = fmaf(p.Dv[d], x, y);
        if (p.z) {
            const float z = ldf((const T *)p.z + i * p.z_st + d);
            y *= z * sigmoid_f(z);
        }
        ((T *)p.out)[i * p.o_st + d] = to_type<T>(y);
    }
}

// calls f with the lanes a channel as a constant
template <class F>
cudaError_t by_lanes(int N, F &&f) {
    if (N <= 16) return f(std::integral_constant<int, 4>());
    if (N <= 32) return f(std::integral_constant<int, 8>());
    if (N <= 64) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

}  // namespace

cudaError_t launch_ssm_scan(const SsmParams &p, cudaStream_t st) {
    return by_lanes(p.N, [&](auto ln) {
        const dim3 grid((p.D + 128 / ln() - 1) / (128 / ln()), p.n_seq);
        if (p.bf16) ssm_scan_kernel<__nv_bfloat16, ln()><<<grid, 128, 0, st>>>(p);
        else ssm_scan_kernel<float, ln()><<<grid, 128, 0, st>>>(p);
        return cudaGetLastError();
    });
}
cudaError_t launch_ssm_step(const SsmStepParams &p, cudaStream_t st) {
    return by_lanes(p.N, [&](auto ln) {
        const dim3 grid((p.D + 128 / ln() - 1) / (128 / ln()), p.n);
        if (p.bf16) ssm_step_kernel<__nv_bfloat16, ln()><<<grid, 128, 0, st>>>(p);
        else ssm_step_kernel<float, ln()><<<grid, 128, 0, st>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace gdn

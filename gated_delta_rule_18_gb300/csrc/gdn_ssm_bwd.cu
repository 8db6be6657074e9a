// gdn_ssm_bwd.cu -- the gradient of the selective scan. With dy = dout
// silu(z) and g the gradient of h, walked back in time,
//   g_t = C_t dy_t + a_{t+1} g_{t+1},
//   dC_n = sum_d dy h,  dB_n = sum_d delta x g,  dx = D dy + delta sum_n B g,
//   ddelta = sum_n A a h_{t-1} g + x sum_n B g,  dA = sum_t delta a h_{t-1} g,
//   ddt = ddelta sigmoid(dt + bias),  dz = dout y silu'(z),  dh0 = a_0 g_0.
//
// One CTA walks a sequence's channels forward, keeping the state every 16
// tokens, then back, recomputing 16 tokens' states at a time in registers.
// Sums over channels (dB, dC) and over sequences (dA, dD, dbias) leave
// partial sums that a second kernel adds in a fixed order.
#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float softplus_f(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

template <typename T, int LN>
__global__ void __launch_bounds__(128) ssm_bwd_kernel(const SsmParams p) {
    constexpr int CH = 128 / LN, L = kSsmCkpt;
    __shared__ float red[4][2 * 4 * LN];
    const int seq = blockIdx.y;
    const int d = blockIdx.x * CH + threadIdx.x / LN, n0 = threadIdx.x % LN * 4;
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
    // checkpoints of a sequence start at (its first token / L + sequence): one more than its whole groups fits
    const int64_t ck0 = p.cu ? t0 / L + seq : (int64_t)seq * (p.T / L + 1);
    float a1[4], a2[4], h[4], g[4], dA[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool on = in && n0 + j < p.N;
        a1[j] = on ? p.A[(int64_t)d * p.N + n0 + j] : 0.f;
        a2[j] = a1[j] * kLog2e;
        h[j] = on && p.h0 ? p.h0[((int64_t)seq * p.D + d) * p.N + n0 + j] : 0.f;
        g[j] = on && p.dh_final ? p.dh_final[((int64_t)seq * p.D + d) * p.N + n0 + j] : 0.f;
        dA[j] = 0.f;
    }
    const float dv = in && p.Dv ? p.Dv[d] : 0.f, bias = in && p.dt_bias ? p.dt_bias[d] : 0.f;
    auto token = [&](int t, float &x, float &v, float &dl, float (&b)[4], float (&c)[4]) {
        x = in ? ldf((const T *)p.x + row * p.x_sb + t * p.x_st + d) : 0.f;
        v = in ? ldf((const T *)p.dt + row * p.dt_sb + t * p.dt_st + d) + bias : 0.f;
        dl = p.softplus ? softplus_f(v) : v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            b[j] = n0 + j < p.N ? ldf((const T *)p.bm + row * p.bm_sb + t * p.bm_st + n0 + j) : 0.f;
            c[j] = n0 + j < p.N ? ldf((const T *)p.cm + row * p.cm_sb + t * p.cm_st + n0 + j) : 0.f;
        }
    };
    float x, v, dl, b[4], c[4];
    for (int t = t0; t < t1; ++t) {
        if ((t - t0) % L == 0 && in) {
            float *ck = p.ckpt + ((ck0 + (t - t0) / L) * p.D + d) * (LN * 4) + n0;
            *reinterpret_cast<float4 *>(ck) = make_float4(h[0], h[1], h[2], h[3]);
        }
        token(t, x, v, dl, b, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = fmaf(exp2f(dl * a2[j]), h[j], dl * x * b[j]);
    }
    float dD = 0.f, dbias = 0.f;
    for (int q = (t1 - t0 + L - 1) / L - 1; q >= 0; --q) {
        const int s = t0 + q * L, e = min(s + L, t1);
        float hs[L + 1][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) hs[0][j] = 0.f;
        if (in) {
            const float4 k = *reinterpret_cast<const float4 *>(p.ckpt + ((ck0 + q) * p.D + d) * (LN * 4) + n0);
            hs[0][0] = k.x, hs[0][1] = k.y, hs[0][2] = k.z, hs[0][3] = k.w;
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (s + i < e) token(s + i, x, v, dl, b, c);
            else x = v = dl = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) hs[i + 1][j] = fmaf(exp2f(dl * a2[j]), hs[i][j], dl * x * b[j]);
        }
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            const int t = s + i;
            if (t >= e) continue;
            token(t, x, v, dl, b, c);
            const float go = in ? ldf((const T *)p.dout + row * p.do_sb + t * p.do_st + d) : 0.f;
            const float z = in && p.z ? ldf((const T *)p.z + row * p.z_sb + t * p.z_st + d) : 0.f;
            const float sz = sigmoid_f(z);
            const float dy = p.z ? go * z * sz : go;
            float y = 0.f, gb = 0.f, gd = 0.f, rb[4], rc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y = fmaf(hs[i + 1][j], c[j], y);
                g[j] = fmaf(c[j], dy, g[j]);
                gb = fmaf(g[j], b[j], gb);
                rb[j] = dl * x * g[j];
                rc[j] = dy * hs[i + 1][j];
                g[j] *= exp2f(dl * a2[j]);
                const float k = g[j] * hs[i][j];
                gd = fmaf(k, a1[j], gd);
                dA[j] = fmaf(k, dl, dA[j]);
            }
#pragma unroll
            for (int o = LN / 2; o > 0; o >>= 1) {
                y += __shfl_xor_sync(0xffffffffu, y, o);
                gb += __shfl_xor_sync(0xffffffffu, gb, o);
                gd += __shfl_xor_sync(0xffffffffu, gd, o);
            }
            if (in && n0 == 0) {
                const int64_t at = ((int64_t)row * p.T + t) * p.D + d;
                y = fmaf(dv, x, y);
                if (p.dz) ((T *)p.dz)[at] = to_type<T>(go * y * sz * fmaf(z, 1.f - sz, 1.f));
                ((T *)p.dx)[at] = to_type<T>(fmaf(dv, dy, dl * gb));
                float ddl = fmaf(x, gb, gd);
                if (p.softplus) ddl *= sigmoid_f(v);
                ((T *)p.ddt)[at] = to_type<T>(ddl);
                dD = fmaf(dy, x, dD);
                dbias += ddl;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int o = 16; o >= LN; o >>= 1) {
                    rb[j] += __shfl_xor_sync(0xffffffffu, rb[j], o);
                    rc[j] += __shfl_xor_sync(0xffffffffu, rc[j], o);
                }
                if ((threadIdx.x & 31) < LN) {
                    red[threadIdx.x >> 5][n0 + j] = rb[j];
                    red[threadIdx.x >> 5][4 * LN + n0 + j] = rc[j];
                }
            }
            __syncthreads();
            for (int n = threadIdx.x; n < 2 * p.N; n += 128) {
                const int k = n < p.N ? n : 4 * LN + n - p.N;
                p.part_bc[((int64_t)blockIdx.x * p.B * p.T + (int64_t)row * p.T + t) * (2 * p.N) + n] =
                    red[0][k] + red[1][k] + red[2][k] + red[3][k];
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (in && n0 + j < p.N) {
            const int64_t at = ((int64_t)seq * p.D + d) * p.N + n0 + j;
            p.part_a[at] = dA[j];
            if (p.dh0) p.dh0[at] = g[j];
        }
    if (in && n0 == 0) {
        p.part_d[(int64_t)seq * 2 * p.D + d] = dD;
        p.part_d[(int64_t)seq * 2 * p.D + p.D + d] = dbias;
    }
}

// dB and dC: the channel tiles' partial sums, rounded once
template <typename T>
__global__ void __launch_bounds__(256) ssm_bwd_reduce_kernel(const SsmParams p, int tiles) {
    const int64_t rows = (int64_t)p.B * p.T, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * 2 * p.N) return;
    float a = 0.f;
    for (int k = 0; k < tiles; ++k) a += p.part_bc[k * rows * 2 * p.N + i];
    const int64_t r = i / (2 * p.N);
    const int n = (int)(i - r * 2 * p.N);
    if (n < p.N) ((T *)p.dbm)[r * p.N + n] = to_type<T>(a);
    else ((T *)p.dcm)[r * p.N + n - p.N] = to_type<T>(a);
}

template <class F>
cudaError_t by_lanes(int N, F &&f) {
    if (N <= 16) return f(std::integral_constant<int, 4>());
    if (N <= 32) return f(std::integral_constant<int, 8>());
    if (N <= 64) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}
int lanes(int N) { return N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32; }

}  // namespace

int ssm_bwd_tiles(int D, int N) { return (D + 128 / lanes(N) - 1) / (128 / lanes(N)); }

cudaError_t launch_ssm_bwd(const SsmParams &p, cudaStream_t st) {
    return by_lanes(p.N, [&](auto ln) {
        const dim3 grid(ssm_bwd_tiles(p.D, p.N), p.n_seq);
        if (p.bf16) ssm_bwd_kernel<__nv_bfloat16, ln()><<<grid, 128, 0, st>>>(p);
        else ssm_bwd_kernel<float, ln()><<<grid, 128, 0, st>>>(p);
        return cudaGetLastError();
    });
}
cudaError_t launch_ssm_bwd_reduce(const SsmParams &p, cudaStream_t st) {
    const int64_t n = (int64_t)p.B * p.T * 2 * p.N;
    if (n == 0) return cudaSuccess;
    const unsigned grid = (unsigned)((n + 255) / 256);
    const int tiles = ssm_bwd_tiles(p.D, p.N);
    if (p.bf16) ssm_bwd_reduce_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p, tiles);
    else ssm_bwd_reduce_kernel<float><<<grid, 256, 0, st>>>(p, tiles);
    return cudaGetLastError();
}

}  // namespace gdn

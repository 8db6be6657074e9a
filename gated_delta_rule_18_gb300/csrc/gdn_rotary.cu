// gdn_rotary.cu -- rotary positions: the first `rot` channels of every head of
// q and k are turned in pairs, pair j of a token at position p by the angle
// p f_j,
//   (a, b) -> scale (a cos - b sin, b cos + a sin),
// where the pairs are channels (2 j, 2 j + 1) (interleaved) or (j, j + rot / 2)
// (half); the other channels pass. The gradient is the same map with the
// opposite angle.
//
// The angle is formed in turns as a 64-bit fixed-point fraction: f_j / 2 pi to
// 2^-64 of a turn, times the position modulo one turn, which the integer
// product's overflow is. Positions up to 2^31 lose 2^-34 of a turn, where an
// fp32 product of a far position has none of the angle left.
//
// Bound by HBM: a head's row is read and written once. A CTA turns a few
// tokens; their cosines and sines are formed once, in shared memory, and serve
// all heads of q and k.
#include "gdn_block.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// f / 2 pi as a fraction of a turn in units of 2^-64
__device__ __forceinline__ unsigned long long turns_of(double f) {
    double t = f * 0.15915494309189533577;
    t -= rint(t);
    return (unsigned long long)__double2ll_rn(t * 18446744073709551616.0);
}

template <typename T, bool VEC, bool HALF>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p, int tokens_cta) {
    extern __shared__ __align__(16) float table[];  // cosines, sines: [token][rot / 2]
    const int pairs = p.rot >> 1;
    float *cs = table, *sn = table + tokens_cta * ((pairs + 3) & ~3);
    const int ld = (pairs + 3) & ~3;
    const int64_t n_tok = (int64_t)p.B * p.T, tok0 = (int64_t)blockIdx.x * tokens_cta;
    const int toks = (int)(n_tok - tok0 < tokens_cta ? n_tok - tok0 : tokens_cta);
    for (int e = threadIdx.x; e < toks * pairs; e += kThreads) {
        const int k = e / pairs, j = e - k * pairs;
        const int64_t b = (tok0 + k) / p.T, t = tok0 + k - b * p.T, at = b * p.p_sb + t * p.p_st;
        const long long pos = !p.pos ? p.offset + t : p.pos64 ? ((const long long *)p.pos)[at] : ((const int *)p.pos)[at];
        const unsigned long long a = (unsigned long long)pos * turns_of(p.inv_freq[j]);
        float s, c;
        sincospif((float)(int)(a >> 32) * 0x1p-31f, &s, &c);
        cs[k * ld + j] = c * p.scale, sn[k * ld + j] = s * p.scale * p.sign;
    }
    __syncthreads();
    // units of a head: V pairs (interleaved: V / 2), then V channels that pass
    constexpr int V = VEC ? 16 / (int)sizeof(T) : 1, W = VEC ? 4 : 1;
    constexpr int P = HALF || !VEC ? V : V / 2;  // pairs a unit
    const int turn = pairs / P, units = turn + (p.x[0].copy | p.x[1].copy ? (p.D - p.rot) / V : 0);
    const int items = (p.x[0].H + p.x[1].H) * units;
    for (int e = threadIdx.x; e < toks * items; e += kThreads) {
        const int k = e / items, r = e - k * items;
        int h = r / units;
        const int u = r - h * units, which = h >= p.x[0].H;
        h -= which ? p.x[0].H : 0;
        const RotaryTensor &x = p.x[which];
        const int64_t b = (tok0 + k) / p.T, t = tok0 + k - b * p.T;
        const T *in = (const T *)x.in + b * x.in_sb + t * x.in_st + h * x.in_sh;
        T *out = (T *)x.out + b * x.out_sb + t * x.out_st + h * x.out_sh;
        if (u >= turn) {
            if (!x.copy) continue;
            const int c = p.rot + (u - turn) * V;
            if constexpr (VEC) *(uint4 *)(out + c) = *(const uint4 *)(in + c);
            else out[c] = in[c];
            continue;
        }
        const float *c = cs + k * ld + u * P, *s = sn + k * ld + u * P;
        if constexpr (!VEC) {
            const int ia = HALF ? u : 2 * u, ib = HALF ? u + pairs : 2 * u + 1;
            const float a = (float)in[ia], d = (float)in[ib];
            out[ia] = to_type<T>(a * c[0] - d * s[0]), out[ib] = to_type<T>(d * c[0] + a * s[0]);
        } else if constexpr (HALF) {
            uint32_t wa[W], wb[W];
            float a[V], d[V];
            ld_words(wa, in + u * V), ld_words(wb, in + pairs + u * V);
            words_to_f<T, V>(a, wa), words_to_f<T, V>(d, wb);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float y = a[j] * c[j] - d[j] * s[j];
                d[j] = d[j] * c[j] + a[j] * s[j], a[j] = y;
            }
            f_to_words<T, V>(wa, a), f_to_words<T, V>(wb, d);
            st_words(out + u * V, wa), st_words(out + pairs + u * V, wb);
        } else {
            uint32_t wa[W];
            float a[V];
            ld_words(wa, in + u * V);
            words_to_f<T, V>(a, wa);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const float y = a[2 * j] * c[j] - a[2 * j + 1] * s[j];
                a[2 * j + 1] = a[2 * j + 1] * c[j] + a[2 * j] * s[j], a[2 * j] = y;
            }
            f_to_words<T, V>(wa, a);
            st_words(out + u * V, wa);
        }
    }
}

template <typename T>
cudaError_t rotary(const RotaryParams &p, cudaStream_t st) {
    const int64_t tokens = (int64_t)p.B * p.T;
    const int v = p.vec ? 16 / (int)sizeof(T) : 1, items = (p.x[0].H + p.x[1].H) * (p.D / v);
    int n = 1;
    while (n < 16 && n * items < 4 * kThreads && tokens > 608 * n) n *= 2;
    const int64_t grid = (tokens + n - 1) / n;
    const int smem = n * ((p.rot / 2 + 3) & ~3) * 8;
    auto run = [&](auto vec, auto half) {
        rotary_kernel<T, vec(), half()><<<(unsigned)grid, kThreads, smem, st>>>(p, n);
        return cudaGetLastError();
    };
    const std::true_type yes;
    const std::false_type no;
    if (p.interleaved) return p.vec ? run(yes, no) : run(no, no);
    return p.vec ? run(yes, yes) : run(no, yes);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams &p, cudaStream_t st) {
    return p.bf16 ? rotary<__nv_bfloat16>(p, st) : rotary<float>(p, st);
}

}  // namespace gdn

// gdn_conv.cu -- the short causal convolution in front of the scan: W taps a
// channel over the last W tokens of the same sequence, bias and SiLU,
//   p_t = b + sum_j w_j x_{t-W+1+j},  y = silu(p),
// where the inputs before a sequence's first token are its carried window
// (n_seq, W - 1, D), oldest first, or zero; its gradient
//   dp = dy silu'(p),  dx_t = sum_j w_j dp_{t+W-1-j},
//   dw_j = sum_t dp_t x_{t-W+1+j},  db = sum_t dp_t;
// and the single-token form that shifts the window in place.
//
// All are bound by HBM (2 W + 5 operations per 4 bytes). A thread keeps a few
// channels (one vector access a token), walks a run of tokens and holds the
// window in registers, so each input is read from HBM once; the W - 1 tokens
// before its run come from L1 or L2. Packed batches need no second form: a
// thread finds the sequence of its first token by bisection and swaps the
// window for the next sequence's carried one where that begins.
#include "gdn_layer.cuh"

namespace gdn {
namespace {

constexpr int kTokL = 16;     // tokens a thread, forward
constexpr int kTokLBwd = 32;  // tokens a thread, gradient
constexpr int kConvY = 4, kConvYBwd = 8;

__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// The sequence of a token: the last s with cu[s] <= t, its bounds clamped so
// that a malformed cu cannot send an access out of range.
struct Seq {
    int seg, s0, s1;
};
__device__ __forceinline__ Seq find_seq(const int32_t *cu, int n_seq, int T, int b, int t) {
    Seq q;
    if (!cu) {
        q.seg = b, q.s0 = 0, q.s1 = T;
        return q;
    }
    int lo = 0, hi = n_seq - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (__ldg(cu + m) <= t) lo = m;
        else hi = m - 1;
    }
    q.seg = lo;
    q.s0 = min(max(__ldg(cu + lo), 0), t);
    q.s1 = max(__ldg(cu + lo + 1), t + 1);
    return q;
}
// the sequence that begins at t, after q
__device__ __forceinline__ void next_seq(Seq &q, const int32_t *cu, int n_seq, int t) {
    while (q.seg + 1 < n_seq && __ldg(cu + q.seg + 1) <= t) ++q.seg;
    q.s0 = t;
    q.s1 = max(__ldg(cu + q.seg + 1), t + 1);
}

template <typename T, int NC, int W, bool VEC>
__device__ __forceinline__ void load_taps(float (&w)[W][NC], const float *weight, int c, int n) {
    if constexpr (VEC) {
        uint32_t u[NC * W];
        ld_words(u, weight + (int64_t)c * W);
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = __uint_as_float(u[i * W + j]);
    } else {
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = i < n ? weight[(int64_t)(c + i) * W + j] : 0.f;
    }
}

// win[k] = the input k + 1 tokens before t
template <typename T, int NC, int W, bool VEC>
__device__ __forceinline__ void load_window(uint32_t (&win)[W - 1][RowVec<T, NC>::kWords], const ConvParams &p,
                                            const T *x, int t, const Seq &q, int c, int n) {
#pragma unroll
    for (int k = 1; k < W; ++k) {
        const int back = t - k;
        if (back >= q.s0) {
            ld_row<T, NC, VEC>(win[k - 1], x + (int64_t)back * p.x_st, n);
        } else if (p.init) {
            const int row = W - 1 - k + (t - q.s0);
            ld_row<T, NC, VEC>(win[k - 1], (const T *)p.init + ((int64_t)q.seg * (W - 1) + row) * p.D + c, n);
        } else {
#pragma unroll
            for (int i = 0; i < RowVec<T, NC>::kWords; ++i) win[k - 1][i] = 0u;
        }
    }
}

__device__ __forceinline__ void check_cu(const int32_t *cu, int n_seq, int T, int *err) {
    int bad = 0;
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, nt = blockDim.x * blockDim.y;
    for (int s = tid; s < n_seq; s += nt) bad |= cu[s + 1] < cu[s];
    if (tid == 0) bad |= cu[0] != 0 || cu[n_seq] != T;
    bad = __syncthreads_or(bad);
    if (tid == 0) *err = bad ? 1 : 0;
}

template <typename T, int NC, int W, bool VEC>
__global__ void __launch_bounds__(32 * kConvY) conv_kernel(const ConvParams p, int nblk) {
    constexpr int NW = RowVec<T, NC>::kWords, U = 4;
    const int c = (blockIdx.y * 32 + threadIdx.x) * NC, n = p.D - c, b = blockIdx.z;
    if (blockIdx.x == nblk) {  // checks, and the windows of empty sequences
        if (p.err && blockIdx.y == 0 && b == 0) check_cu(p.cu, p.n_seq, p.T, p.err);
        if (!p.final_state || c >= p.D || b > 0) return;
        for (int s = threadIdx.y; s < p.n_seq; s += kConvY) {
            if (p.cu ? p.cu[s + 1] > p.cu[s] : p.T > 0) continue;
            for (int r = 0; r < W - 1; ++r) {
                const int64_t at = ((int64_t)s * (W - 1) + r) * p.D + c;
                uint32_t v[NW] = {};
                if (p.init) ld_row<T, NC, VEC>(v, (const T *)p.init + at, n);
                st_row<T, NC, VEC>((T *)p.final_state + at, v, n);
            }
        }
        return;
    }
    const int64_t first = ((int64_t)blockIdx.x * kConvY + threadIdx.y) * kTokL;
    if (c >= p.D || first >= p.T) return;
    const int t0 = (int)first, t1 = min(p.T - t0, kTokL) + t0;
    const T *x = (const T *)p.x + b * p.x_sb + c;
    T *out = (T *)p.out + b * p.o_sb + c;
    float w[W][NC], bias[NC];
    load_taps<T, NC, W, VEC>(w, p.weight, c, n);
#pragma unroll
    for (int i = 0; i < NC; ++i) bias[i] = 0.f;
    if (p.bias) ld_row_f<float, NC, VEC>(bias, p.bias + c, n);
    Seq q = find_seq(p.cu, p.n_seq, p.T, b, t0);
    uint32_t win[W - 1][NW];
    load_window<T, NC, W, VEC>(win, p, x, t0, q, c, n);
    for (int t = t0; t < t1; t += U) {
        uint32_t raw[U][NW];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < t1) ld_row<T, NC, VEC>(raw[u], x + (int64_t)(t + u) * p.x_st, n);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= t1) break;
            if (t + u == q.s1) {
                next_seq(q, p.cu, p.n_seq, t + u);
                load_window<T, NC, W, VEC>(win, p, x, t + u, q, c, n);
            }
            float a[NC], v[NC];
            words_to_f<T, NC>(v, raw[u]);
#pragma unroll
            for (int i = 0; i < NC; ++i) a[i] = fmaf(w[W - 1][i], v[i], bias[i]);
#pragma unroll
            for (int k = 1; k < W; ++k) {
                words_to_f<T, NC>(v, win[k - 1]);
#pragma unroll
                for (int i = 0; i < NC; ++i) a[i] = fmaf(w[W - 1 - k][i], v[i], a[i]);
            }
            if (p.silu) {
#pragma unroll
                for (int i = 0; i < NC; ++i) a[i] *= sigmoid_f(a[i]);
            }
            st_row_f<T, NC, VEC>(out + (int64_t)(t + u) * p.o_st, a, n);
#pragma unroll
            for (int k = W - 2; k > 0; --k)
#pragma unroll
                for (int i = 0; i < NW; ++i) win[k][i] = win[k - 1][i];
#pragma unroll
            for (int i = 0; i < NW; ++i) win[0][i] = raw[u][i];
            if (p.final_state && t + u + 1 == q.s1) {
#pragma unroll
                for (int k = 1; k < W; ++k)
                    st_row<T, NC, VEC>((T *)p.final_state + ((int64_t)q.seg * (W - 1) + W - 1 - k) * p.D + c,
                                       win[k - 1], n);
            }
        }
    }
}

// dp at token t from the window before it (win), the token's own input and dout
template <typename T, int NC, int W>
__device__ __forceinline__ void dpre(float (&dp)[NC], const float (&w)[W][NC], const float (&bias)[NC],
                                     const uint32_t (&win)[W - 1][RowVec<T, NC>::kWords], const float (&x)[NC],
                                     const float (&dout)[NC], int silu) {
    float v[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) dp[i] = dout[i];
    if (!silu) return;
    float a[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) a[i] = fmaf(w[W - 1][i], x[i], bias[i]);
#pragma unroll
    for (int k = 1; k < W; ++k) {
        words_to_f<T, NC>(v, win[k - 1]);
#pragma unroll
        for (int i = 0; i < NC; ++i) a[i] = fmaf(w[W - 1 - k][i], v[i], a[i]);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const float s = sigmoid_f(a[i]);
        dp[i] *= s * fmaf(a[i], 1.f - s, 1.f);
    }
}
template <typename T, int NC, int W>
__device__ __forceinline__ void push(uint32_t (&win)[W - 1][RowVec<T, NC>::kWords],
                                     const uint32_t (&raw)[RowVec<T, NC>::kWords]) {
#pragma unroll
    for (int k = W - 2; k > 0; --k)
#pragma unroll
        for (int i = 0; i < RowVec<T, NC>::kWords; ++i) win[k][i] = win[k - 1][i];
#pragma unroll
    for (int i = 0; i < RowVec<T, NC>::kWords; ++i) win[0][i] = raw[i];
}

// pend[k] holds the part of dx of the token k + 1 back that later tokens have
// already given; a token's dx is complete W - 1 tokens later, so a run of
// tokens is followed by W - 1 more that only add to the run's own.
template <typename T, int NC, int W, bool VEC>
__global__ void __launch_bounds__(32 * kConvYBwd) conv_bwd_kernel(const ConvParams p, int nblk) {
    constexpr int NW = RowVec<T, NC>::kWords;
    extern __shared__ float red[];  // [kConvYBwd][NC * (W + 1)][32]
    const int c = (blockIdx.y * 32 + threadIdx.x) * NC, n = p.D - c, b = blockIdx.z;
    const bool extra = blockIdx.x == nblk;
    if (extra && p.err && blockIdx.y == 0 && b == 0) check_cu(p.cu, p.n_seq, p.T, p.err);
    if (extra && (!p.dinit || c >= p.D || b > 0)) return;
    float w[W][NC], bias[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) bias[i] = 0.f;
    if (c < p.D) {
        load_taps<T, NC, W, VEC>(w, p.weight, c, n);
        if (p.bias) ld_row_f<float, NC, VEC>(bias, p.bias + c, n);
    }
    uint32_t win[W - 1][NW], raw[NW];
    float x[NC], go[NC], dp[NC];
    if (extra) {  // the gradient of each carried window: its sequence's first W - 1 tokens
        for (int s = threadIdx.y; s < p.n_seq; s += kConvYBwd) {
            Seq q;
            q.seg = s;
            q.s0 = p.cu ? min(max(p.cu[s], 0), p.T) : 0;
            q.s1 = p.cu ? min(max(p.cu[s + 1], q.s0), p.T) : p.T;
            const int len = q.s1 - q.s0, row_b = p.cu ? 0 : s;
            const T *xs = (const T *)p.x + row_b * p.x_sb + c;
            const T *ds = (const T *)p.dout + row_b * p.do_sb + c;
            float acc[W - 1][NC];
#pragma unroll
            for (int r = 0; r < W - 1; ++r) {
#pragma unroll
                for (int i = 0; i < NC; ++i) acc[r][i] = 0.f;
                if (p.dfinal && r >= len)
                    ld_row_f<T, NC, VEC>(acc[r], (const T *)p.dfinal + ((int64_t)s * (W - 1) + r - len) * p.D + c, n);
            }
            load_window<T, NC, W, VEC>(win, p, xs, q.s0, q, c, n);
#pragma unroll
            for (int u = 0; u < W - 1; ++u) {
                if (u < len) {
                    ld_row<T, NC, VEC>(raw, xs + (int64_t)(q.s0 + u) * p.x_st, n);
                    words_to_f<T, NC>(x, raw);
                    ld_row_f<T, NC, VEC>(go, ds + (int64_t)(q.s0 + u) * p.do_st, n);
                    dpre<T, NC, W>(dp, w, bias, win, x, go, p.silu);
                    // token u reads window row r through tap r - u
#pragma unroll
                    for (int r = u; r < W - 1; ++r)
#pragma unroll
                        for (int i = 0; i < NC; ++i) acc[r][i] = fmaf(w[r - u][i], dp[i], acc[r][i]);
                    push<T, NC, W>(win, raw);
                }
            }
#pragma unroll
            for (int r = 0; r < W - 1; ++r)
                st_row_f<T, NC, VEC>((T *)p.dinit + ((int64_t)s * (W - 1) + r) * p.D + c, acc[r], n);
        }
        return;
    }
    float dw[W][NC], db[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
    }
    const int64_t first = ((int64_t)blockIdx.x * kConvYBwd + threadIdx.y) * kTokLBwd;
    if (c < p.D && first < p.T) {
        const int t0 = (int)first, t1 = min(p.T - t0, kTokLBwd) + t0;
        const T *xs = (const T *)p.x + b * p.x_sb + c;
        const T *ds = (const T *)p.dout + b * p.do_sb + c;
        T *dx = (T *)p.dx + (int64_t)b * p.T * p.D + c;
        Seq q = find_seq(p.cu, p.n_seq, p.T, b, t0);
        load_window<T, NC, W, VEC>(win, p, xs, t0, q, c, n);
        float pend[W][NC];
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int i = 0; i < NC; ++i) pend[k][i] = 0.f;
        for (int t = t0; t < t1 + W - 1; ++t) {
#pragma unroll
            for (int k = W - 1; k > 0; --k)
#pragma unroll
                for (int i = 0; i < NC; ++i) pend[k][i] = pend[k - 1][i];
#pragma unroll
            for (int i = 0; i < NC; ++i) pend[0][i] = 0.f;
            if (t < p.T) {
                if (t == q.s1) {
                    next_seq(q, p.cu, p.n_seq, t);
                    load_window<T, NC, W, VEC>(win, p, xs, t, q, c, n);
                }
                ld_row<T, NC, VEC>(raw, xs + (int64_t)t * p.x_st, n);
                words_to_f<T, NC>(x, raw);
                ld_row_f<T, NC, VEC>(go, ds + (int64_t)t * p.do_st, n);
                dpre<T, NC, W>(dp, w, bias, win, x, go, p.silu);
                if (t < t1) {
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        db[i] += dp[i];
                        dw[W - 1][i] = fmaf(dp[i], x[i], dw[W - 1][i]);
                    }
#pragma unroll
                    for (int k = 1; k < W; ++k) {
                        float v[NC];
                        words_to_f<T, NC>(v, win[k - 1]);
#pragma unroll
                        for (int i = 0; i < NC; ++i) dw[W - 1 - k][i] = fmaf(dp[i], v[i], dw[W - 1 - k][i]);
                    }
                    if (p.dfinal && t >= q.s1 - (W - 1))
                        ld_row_f<T, NC, VEC>(
                            pend[0],
                            (const T *)p.dfinal + ((int64_t)q.seg * (W - 1) + t - (q.s1 - (W - 1))) * p.D + c, n);
                }
#pragma unroll
                for (int k = 0; k < W; ++k)
                    if (t - k >= q.s0) {
#pragma unroll
                        for (int i = 0; i < NC; ++i) pend[k][i] = fmaf(w[W - 1 - k][i], dp[i], pend[k][i]);
                    }
                push<T, NC, W>(win, raw);
            }
            const int done = t - (W - 1);
            if (done >= t0 && done < t1) st_row_f<T, NC, VEC>(dx + (int64_t)done * p.D, pend[W - 1], n);
        }
    }
    // the CTA's share of dw and db
    constexpr int Q = NC * (W + 1);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) red[(threadIdx.y * Q + i * W + j) * 32 + threadIdx.x] = dw[j][i];
        red[(threadIdx.y * Q + NC * W + i) * 32 + threadIdx.x] = db[i];
    }
    __syncthreads();
    float *part = p.part + ((int64_t)b * nblk + blockIdx.x) * ((int64_t)p.D * (W + 1));
    for (int r = threadIdx.y; r < Q; r += kConvYBwd) {
        float a = 0.f;
#pragma unroll
        for (int y = 0; y < kConvYBwd; ++y) a += red[(y * Q + r) * 32 + threadIdx.x];
        const int i = r < NC * W ? r / W : r - NC * W;
        if (c + i >= p.D) continue;
        if (r < NC * W) part[(int64_t)(c + i) * W + (r - i * W)] = a;
        else part[(int64_t)p.D * W + c + i] = a;
    }
}

template <typename T, int NC, int W, bool VEC>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvStepParams p) {
    constexpr int NW = RowVec<T, NC>::kWords;
    const int c = (blockIdx.x * 128 + threadIdx.x) * NC, n = p.D - c, i0 = blockIdx.y;
    if (c >= p.D) return;
    const int slot = p.slots ? p.slots[i0] : i0;
    T *out = (T *)p.out + (int64_t)i0 * p.o_st + c;
    float a[NC], v[NC], w[W][NC];
    uint32_t raw[W][NW];
#pragma unroll
    for (int i = 0; i < NC; ++i) a[i] = 0.f;
    if (slot < 0 || slot >= p.n_slots) {  // a padding row
        st_row_f<T, NC, VEC>(out, a, n);
        return;
    }
    T *state = (T *)p.state + (int64_t)slot * (W - 1) * p.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) ld_row<T, NC, VEC>(raw[j], state + (int64_t)j * p.D, n);
    ld_row<T, NC, VEC>(raw[W - 1], (const T *)p.x + (int64_t)i0 * p.x_st + c, n);
    load_taps<T, NC, W, VEC>(w, p.weight, c, n);
    if (p.bias) ld_row_f<float, NC, VEC>(a, p.bias + c, n);
#pragma unroll
    for (int j = W - 1; j >= 0; --j) {
        words_to_f<T, NC>(v, raw[j]);
#pragma unroll
        for (int i = 0; i < NC; ++i) a[i] = fmaf(w[j][i], v[i], a[i]);
        if (j > 0) st_row<T, NC, VEC>(state + (int64_t)(j - 1) * p.D, raw[j], n);
    }
    if (p.silu) {
#pragma unroll
        for (int i = 0; i < NC; ++i) a[i] *= sigmoid_f(a[i]);
    }
    st_row_f<T, NC, VEC>(out, a, n);
}

// calls f with the tap count as a constant
template <class F>
cudaError_t by_taps(int W, F &&f) {
    switch (W) {
        case 2: return f(std::integral_constant<int, 2>());
        case 3: return f(std::integral_constant<int, 3>());
        case 4: return f(std::integral_constant<int, 4>());
        case 5: return f(std::integral_constant<int, 5>());
        case 6: return f(std::integral_constant<int, 6>());
        case 7: return f(std::integral_constant<int, 7>());
        case 8: return f(std::integral_constant<int, 8>());
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t conv_t(const ConvParams &p, cudaStream_t st) {
    constexpr int NC = 16 / sizeof(T);
    const int nblk = (int)(((int64_t)p.T + kConvY * kTokL - 1) / (kConvY * kTokL));
    const bool extra = p.cu != nullptr || p.T == 0;
    const dim3 grid(nblk + (extra ? 1 : 0), (p.D + 32 * NC - 1) / (32 * NC), p.T == 0 ? 1 : p.B), block(32, kConvY);
    return by_taps(p.W, [&](auto w) {
        if (p.vec) conv_kernel<T, NC, w(), true><<<grid, block, 0, st>>>(p, nblk);
        else conv_kernel<T, NC, w(), false><<<grid, block, 0, st>>>(p, nblk);
        return cudaGetLastError();
    });
}
template <typename T>
cudaError_t conv_bwd_t(const ConvParams &p, cudaStream_t st) {
    constexpr int NC = 4;
    const int nblk = conv_bwd_parts(1, p.T);
    const bool extra = p.cu != nullptr || p.dinit;
    const dim3 grid(nblk + (extra ? 1 : 0), (p.D + 32 * NC - 1) / (32 * NC), p.T == 0 ? 1 : p.B),
        block(32, kConvYBwd);
    return by_taps(p.W, [&](auto w) {
        const size_t smem = sizeof(float) * 32 * kConvYBwd * NC * (w() + 1);
        if (p.vec) conv_bwd_kernel<T, NC, w(), true><<<grid, block, smem, st>>>(p, nblk);
        else conv_bwd_kernel<T, NC, w(), false><<<grid, block, smem, st>>>(p, nblk);
        return cudaGetLastError();
    });
}
template <typename T>
cudaError_t conv_step_t(const ConvStepParams &p, cudaStream_t st) {
    constexpr int NC = 16 / sizeof(T);
    const dim3 grid((p.D + 128 * NC - 1) / (128 * NC), p.n);
    return by_taps(p.W, [&](auto w) {
        if (p.vec) conv_step_kernel<T, NC, w(), true><<<grid, 128, 0, st>>>(p);
        else conv_step_kernel<T, NC, w(), false><<<grid, 128, 0, st>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace

cudaError_t launch_conv(const ConvParams &p, cudaStream_t st) {
    return p.bf16 ? conv_t<__nv_bfloat16>(p, st) : conv_t<float>(p, st);
}
// CTAs along the tokens of all rows: each leaves one row of partial sums
int conv_bwd_parts(int B, int T) {
    return B * (int)(((int64_t)T + kConvYBwd * kTokLBwd - 1) / (kConvYBwd * kTokLBwd));
}
cudaError_t launch_conv_bwd(const ConvParams &p, cudaStream_t st) {
    return p.bf16 ? conv_bwd_t<__nv_bfloat16>(p, st) : conv_bwd_t<float>(p, st);
}
cudaError_t launch_conv_step(const ConvStepParams &p, cudaStream_t st) {
    return p.bf16 ? conv_step_t<__nv_bfloat16>(p, st) : conv_step_t<float>(p, st);
}

}  // namespace gdn

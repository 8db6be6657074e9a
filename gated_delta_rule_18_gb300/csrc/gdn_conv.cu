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
// before its run come from L1 or L2. The next twelve tokens' rows are under
// way to shared memory while four are computed, in packed pairs of channels;
// four tokens of one sequence run without a branch. Packed batches need no
// second form: a thread finds the sequence of its first token by bisection and
// swaps the window for the next sequence's carried one where that begins.
// 16384 tokens of 4096 channels, 4 taps: bf16 54.5 us for 268 MB (73% of the
// measured copy rate), fp32 90.5 (87%); the gradient 90 us for 403 MB (66%)
// and 144 (82%). With the rows held in registers, four tokens ahead: 59, 95,
// 95 and 171. In bf16 neither limit is reached (issue slots 55 to 58 % used, DRAM
// 56 to 58 % by the profiler): at 21 warps a SM, in the gradient 15 (128
// registers), the latencies of loads and of dependent instructions are left.
#include "gdn_ssm.cuh"

namespace gdn {
namespace {

constexpr int kConvY = 4, kConvYBwd = 8;
// Groups of four tokens in shared memory. Gradient, 4 x 4096 tokens of 4096
// channels: bf16 89, 86, 90 us for 4, 3, 2 (two CTAs a SM), fp32 138, 144, 167.
constexpr int kAhead = 4;
template <typename T>
constexpr int kAheadBwd = sizeof(T) == 4 ? 4 : 3;

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

// the taps and biases of NC channels, in pairs of channels
template <typename T, int NC, int W, bool VEC>
__device__ __forceinline__ void load_taps(f32x2 (&w)[W][NC / 2], f32x2 (&bias)[NC / 2], const float *weight,
                                          const float *b, int c, int n) {
    float f[NC * W], g[NC];
    if constexpr (VEC) {
        uint32_t u[NC * W];
        ld_words(u, weight + (int64_t)c * W);
#pragma unroll
        for (int i = 0; i < NC * W; ++i) f[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < NC * W; ++i) f[i] = i / W < n ? weight[(int64_t)c * W + i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) g[i] = 0.f;
    if (b) ld_row_f<float, NC, VEC>(g, b + c, n);
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
        bias[i] = pack2(g[2 * i], g[2 * i + 1]);
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = pack2(f[2 * i * W + j], f[(2 * i + 1) * W + j]);
    }
}
template <typename T, int NC>
__device__ __forceinline__ void words_to_pairs(f32x2 (&v)[NC / 2], const uint32_t (&w)[RowVec<T, NC>::kWords]) {
    float f[NC];
    words_to_f<T, NC>(f, w);
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) v[i] = pack2(f[2 * i], f[2 * i + 1]);
}
template <typename T, int NC, bool VEC>
__device__ __forceinline__ void st_pairs(T *p, const f32x2 (&v)[NC / 2], int n) {
    float f[NC];
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
        const float2 x = unpack2(v[i]);
        f[2 * i] = x.x, f[2 * i + 1] = x.y;
    }
    st_row_f<T, NC, VEC>(p, f, n);
}

// win[k] = the input k + 1 tokens before t
template <typename T, int NC, int W, bool VEC>
__device__ __forceinline__ void load_window(f32x2 (&win)[W - 1][NC / 2], const ConvParams &p, const T *x, int t,
                                            const Seq &q, int c, int n) {
#pragma unroll
    for (int k = 1; k < W; ++k) {
        const int back = t - k;
        uint32_t v[RowVec<T, NC>::kWords] = {};
        if (back >= q.s0) {
            ld_row<T, NC, VEC>(v, x + (int64_t)back * p.x_st, n);
        } else if (p.init) {
            const int row = W - 1 - k + (t - q.s0);
            ld_row<T, NC, VEC>(v, (const T *)p.init + ((int64_t)q.seg * (W - 1) + row) * p.D + c, n);
        }
        words_to_pairs<T, NC>(win[k - 1], v);
    }
}
template <int NC, int W>
__device__ __forceinline__ void push(f32x2 (&win)[W - 1][NC / 2], const f32x2 (&v)[NC / 2]) {
#pragma unroll
    for (int k = W - 2; k > 0; --k)
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) win[k][i] = win[k - 1][i];
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) win[0][i] = v[i];
}
// sigmoid of a pair; exp(-x) = inf gives 0
__device__ __forceinline__ f32x2 sigmoid_pair(f32x2 x) {
    const f32x2 e = add2(ex2_2(mul2(x, pack2(-kLog2e, -kLog2e))), pack2(1.f, 1.f));
    const float2 f = unpack2(e);
    return pack2(rcpf(f.x), rcpf(f.y));
}
// the convolution at the token whose input is v
template <int NC, int W>
__device__ __forceinline__ void convolve(f32x2 (&a)[NC / 2], const f32x2 (&w)[W][NC / 2], const f32x2 (&bias)[NC / 2],
                                         const f32x2 (&win)[W - 1][NC / 2], const f32x2 (&v)[NC / 2]) {
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
        a[i] = fma2(w[W - 1][i], v[i], bias[i]);
#pragma unroll
        for (int k = 1; k < W; ++k) a[i] = fma2(w[W - 1 - k][i], win[k - 1][i], a[i]);
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

// A thread's own rows on their way: groups of U tokens of one tensor, S - 1 of
// them under way while one is used. Wide rows go by asynchronous copies to
// slots of shared memory that only this thread touches (so nothing is waited
// for but its own copies, and no registers hold what is under way); others
// through registers, one group ahead.
template <typename T, int NC, int U, bool VEC, int NT, int GROUPS>
struct Ahead {
    static constexpr int NW = RowVec<T, NC>::kWords, S = VEC ? GROUPS : 2;
    static constexpr __host__ __device__ int words() { return VEC ? S * U * NT * NW : 0; }  // of all threads
    uint32_t *slots;                                              // this thread's first one
    uint32_t next[VEC ? 1 : U][NW];
    __device__ __forceinline__ uint32_t *slot(int g, int u) { return slots + ((g % S) * U + u) * NT * NW; }
    // row u of group g; on: it exists
    __device__ __forceinline__ void fetch(int g, int u, const T *row, int n, bool on) {
        if (!on) return;
        if constexpr (VEC) copy_async<NW * 4>(slot(g, u), row);
        else ld_row<T, NC, false>(next[u], row, n);
    }
    // this thread's copies but those of the last S - 2 groups have arrived
    static __device__ __forceinline__ void arrived() {
        if (VEC) copies_arrived<S - 2>();
    }
    __device__ __forceinline__ void take(uint32_t (&raw)[U][NW], int g) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (VEC) {
                ld_words(raw[u], slot(g, u));
            } else {
#pragma unroll
                for (int i = 0; i < NW; ++i) raw[u][i] = next[u][i];
            }
        }
    }
};

template <typename T, int NC, int W, bool VEC>
__global__ void __launch_bounds__(32 * kConvY, sizeof(T) == 2 && W <= 4 ? 6 : 3) conv_kernel(const ConvParams p, int nblk, int run) {
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
    const int64_t first = ((int64_t)blockIdx.x * kConvY + threadIdx.y) * run;
    if (c >= p.D || first >= p.T) return;
    const int t0 = (int)first, t1 = min(p.T - t0, run) + t0;
    const T *x = (const T *)p.x + b * p.x_sb + c;
    T *out = (T *)p.out + b * p.o_sb + c;
    f32x2 w[W][NC / 2], bias[NC / 2], win[W - 1][NC / 2];
    load_taps<T, NC, W, VEC>(w, bias, p.weight, p.bias, c, n);
    Seq q = find_seq(p.cu, p.n_seq, p.T, b, t0);
    load_window<T, NC, W, VEC>(win, p, x, t0, q, c, n);
    using Rows = Ahead<T, NC, U, VEC, 32 * kConvY, kAhead>;
    extern __shared__ __align__(16) uint32_t ring[];
    Rows in;
    in.slots = ring + (threadIdx.y * 32 + threadIdx.x) * NW;
    const T *xp = x + (int64_t)t0 * p.x_st;  // the next load's and store's rows
    T *op = out + (int64_t)t0 * p.o_st;
    int put = 0, got = 0;
    auto fetch = [&] {
        const int t = t0 + put * U;
        if (t + U <= t1) {
#pragma unroll
            for (int u = 0; u < U; ++u, xp += p.x_st) in.fetch(put, u, xp, n, true);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u, xp += p.x_st) in.fetch(put, u, xp, n, t + u < t1);
        }
        if (VEC) cp_async_commit();
        ++put;
    };
    for (int i = 0; i + 1 < Rows::S; ++i) fetch();
    auto window_out = [&](int seg) {
#pragma unroll
        for (int k = 1; k < W; ++k)
            st_pairs<T, NC, VEC>((T *)p.final_state + ((int64_t)seg * (W - 1) + W - 1 - k) * p.D + c, win[k - 1], n);
    };
    auto token = [&](const uint32_t (&raw)[NW]) {
        f32x2 a[NC / 2], v[NC / 2];
        words_to_pairs<T, NC>(v, raw);
        convolve<NC, W>(a, w, bias, win, v);
        if (p.silu) {
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) a[i] = mul2(a[i], sigmoid_pair(a[i]));
        }
        st_pairs<T, NC, VEC>(op, a, n);
        op += p.o_st;
        push<NC, W>(win, v);
    };
    for (int t = t0; t < t1; t += U) {
        uint32_t raw[U][NW];
        Rows::arrived();
        in.take(raw, got++);
        fetch();
        if (t == q.s1) {
            next_seq(q, p.cu, p.n_seq, t);
            load_window<T, NC, W, VEC>(win, p, x, t, q, c, n);
        }
        if (t + U <= t1 && t + U <= q.s1) {  // four tokens of one sequence, without a branch
#pragma unroll
            for (int u = 0; u < U; ++u) token(raw[u]);
            if (p.final_state && t + U == q.s1) window_out(q.seg);
        } else {
#pragma unroll 1
            for (int u = 0; u < U && t + u < t1; ++u) {
                if (t + u == q.s1) {
                    next_seq(q, p.cu, p.n_seq, t + u);
                    load_window<T, NC, W, VEC>(win, p, x, t + u, q, c, n);
                }
                uint32_t cur[NW];
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    cur[i] = u == 0 ? raw[0][i] : u == 1 ? raw[1][i] : u == 2 ? raw[2][i] : raw[3][i];
                token(cur);
                if (p.final_state && t + u + 1 == q.s1) window_out(q.seg);
            }
        }
    }
}

// dp at the token whose input is v
template <int NC, int W>
__device__ __forceinline__ void dpre(f32x2 (&dp)[NC / 2], const f32x2 (&w)[W][NC / 2], const f32x2 (&bias)[NC / 2],
                                     const f32x2 (&win)[W - 1][NC / 2], const f32x2 (&v)[NC / 2],
                                     const f32x2 (&dout)[NC / 2], int silu) {
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) dp[i] = dout[i];
    if (!silu) return;
    f32x2 a[NC / 2];
    convolve<NC, W>(a, w, bias, win, v);
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
            // silu' = s + a s (1 - s)
        const f32x2 s = sigmoid_pair(a[i]), as = mul2(a[i], s);
        const f32x2 r = fma2(mul2(as, pack2(-1.f, -1.f)), s, as);
        dp[i] = mul2(dp[i], add2(s, r));
    }
}

// pend[k] holds the part of dx of the token k + 1 back that later tokens have
// already given; a token's dx is complete W - 1 tokens later, so a run of
// tokens is followed by W - 1 more that only add to the run's own.
template <typename T, int NC, int W, bool VEC>
__global__ void __launch_bounds__(32 * kConvYBwd, sizeof(T) == 2 && W <= 4 ? 2 : 1) conv_bwd_kernel(const ConvParams p, int nblk, int run) {
    constexpr int NW = RowVec<T, NC>::kWords;
    extern __shared__ float red[];  // [kConvYBwd][NC * (W + 1)][32]
    const int c = (blockIdx.y * 32 + threadIdx.x) * NC, n = p.D - c, b = blockIdx.z;
    const bool extra = blockIdx.x == nblk;
    if (extra && p.err && blockIdx.y == 0 && b == 0) check_cu(p.cu, p.n_seq, p.T, p.err);
    if (extra && (!p.dinit || c >= p.D || b > 0)) return;
    f32x2 w[W][NC / 2], bias[NC / 2], win[W - 1][NC / 2];
    if (c < p.D) load_taps<T, NC, W, VEC>(w, bias, p.weight, p.bias, c, n);
    if (extra) {  // the gradient of each carried window: its sequence's first W - 1 tokens
        for (int s = threadIdx.y; s < p.n_seq; s += kConvYBwd) {
            Seq q;
            q.seg = s;
            q.s0 = p.cu ? min(max(p.cu[s], 0), p.T) : 0;
            q.s1 = p.cu ? min(max(p.cu[s + 1], q.s0), p.T) : p.T;
            const int len = q.s1 - q.s0, row_b = p.cu ? 0 : s;
            const T *xs = (const T *)p.x + row_b * p.x_sb + c;
            const T *ds = (const T *)p.dout + row_b * p.do_sb + c;
            f32x2 acc[W - 1][NC / 2];
            uint32_t raw[NW];
#pragma unroll
            for (int r = 0; r < W - 1; ++r) {
#pragma unroll
                for (int i = 0; i < NW; ++i) raw[i] = 0u;
                if (p.dfinal && r >= len)
                    ld_row<T, NC, VEC>(raw, (const T *)p.dfinal + ((int64_t)s * (W - 1) + r - len) * p.D + c, n);
                words_to_pairs<T, NC>(acc[r], raw);
            }
            load_window<T, NC, W, VEC>(win, p, xs, q.s0, q, c, n);
#pragma unroll
            for (int u = 0; u < W - 1; ++u) {
                if (u < len) {
                    f32x2 x[NC / 2], go[NC / 2], dp[NC / 2];
                    ld_row<T, NC, VEC>(raw, xs + (int64_t)(q.s0 + u) * p.x_st, n);
                    words_to_pairs<T, NC>(x, raw);
                    ld_row<T, NC, VEC>(raw, ds + (int64_t)(q.s0 + u) * p.do_st, n);
                    words_to_pairs<T, NC>(go, raw);
                    dpre<NC, W>(dp, w, bias, win, x, go, p.silu);
                    // token u reads window row r through tap r - u
#pragma unroll
                    for (int r = u; r < W - 1; ++r)
#pragma unroll
                        for (int i = 0; i < NC / 2; ++i) acc[r][i] = fma2(w[r - u][i], dp[i], acc[r][i]);
                    push<NC, W>(win, x);
                }
            }
#pragma unroll
            for (int r = 0; r < W - 1; ++r)
                st_pairs<T, NC, VEC>((T *)p.dinit + ((int64_t)s * (W - 1) + r) * p.D + c, acc[r], n);
        }
        return;
    }
    f32x2 dw[W][NC / 2], db[NC / 2];
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
        db[i] = pack2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = pack2(0.f, 0.f);
    }
    const int64_t first = ((int64_t)blockIdx.x * kConvYBwd + threadIdx.y) * run;
    if (c < p.D && first < p.T) {
        constexpr int U = VEC ? 4 : 2;
        const int t0 = (int)first, t1 = min(p.T - t0, run) + t0, t2 = min(p.T - t1, W - 1) + t1;
        const T *xs = (const T *)p.x + b * p.x_sb + c;
        const T *ds = (const T *)p.dout + b * p.do_sb + c;
        T *dx = (T *)p.dx + (int64_t)b * p.T * p.D + c;
        Seq q = find_seq(p.cu, p.n_seq, p.T, b, t0);
        load_window<T, NC, W, VEC>(win, p, xs, t0, q, c, n);
        f32x2 pend[W][NC / 2];
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) pend[k][i] = pack2(0.f, 0.f);
        using Rows = Ahead<T, NC, U, VEC, 32 * kConvYBwd, kAheadBwd<T>>;
        Rows in_x, in_d;
        in_x.slots = reinterpret_cast<uint32_t *>(red + 32 * kConvYBwd * NC * (W + 1)) + (threadIdx.y * 32 + threadIdx.x) * NW;
        in_d.slots = in_x.slots + Rows::words();
        const T *xp = xs + (int64_t)t0 * p.x_st, *dp_ = ds + (int64_t)t0 * p.do_st;  // the next loads' rows
        T *op = dx + (int64_t)(t0 - (W - 1)) * p.D;                                   // of the next dx
        int put = 0, got = 0;
        auto fetch = [&] {
            const int t = t0 + put * U;
            if (t + U <= t2) {
#pragma unroll
                for (int u = 0; u < U; ++u, xp += p.x_st, dp_ += p.do_st) {
                    in_x.fetch(put, u, xp, n, true);
                    in_d.fetch(put, u, dp_, n, true);
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u, xp += p.x_st, dp_ += p.do_st) {
                    in_x.fetch(put, u, xp, n, t + u < t2);
                    in_d.fetch(put, u, dp_, n, t + u < t2);
                }
            }
            if (VEC) cp_async_commit();
            ++put;
        };
        for (int i = 0; i + 1 < Rows::S; ++i) fetch();
        // one token: own, its dw and db count; s0, its sequence's first token
        auto token = [&](int t, const uint32_t (&rx)[NW], const uint32_t (&rd)[NW], bool own, bool whole) {
            f32x2 x[NC / 2], go[NC / 2], dp[NC / 2];
            words_to_pairs<T, NC>(x, rx);
            words_to_pairs<T, NC>(go, rd);
            dpre<NC, W>(dp, w, bias, win, x, go, p.silu);
            if (own) {
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) {
                    db[i] = add2(db[i], dp[i]);
                    dw[W - 1][i] = fma2(dp[i], x[i], dw[W - 1][i]);
#pragma unroll
                    for (int k = 1; k < W; ++k) dw[W - 1 - k][i] = fma2(dp[i], win[k - 1][i], dw[W - 1 - k][i]);
                }
            }
#pragma unroll
            for (int k = 0; k < W; ++k)
                if (whole || t - k >= q.s0) {
#pragma unroll
                    for (int i = 0; i < NC / 2; ++i) pend[k][i] = fma2(w[W - 1 - k][i], dp[i], pend[k][i]);
                }
            push<NC, W>(win, x);
        };
        auto shift = [&] {
#pragma unroll
            for (int k = W - 1; k > 0; --k)
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) pend[k][i] = pend[k - 1][i];
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) pend[0][i] = pack2(0.f, 0.f);
        };
        // slow: a few tokens from tb on, of any sequences
        auto slow = [&](int tb, const uint32_t (&rx)[U][NW], const uint32_t (&rd)[U][NW]) {
#pragma unroll 1
            for (int u = 0; u < U; ++u) {
                const int t = tb + u;
                uint32_t cx[NW], cd[NW];
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    cx[i] = rx[0][i], cd[i] = rd[0][i];
#pragma unroll
                    for (int k = 1; k < U; ++k)
                        if (u == k) cx[i] = rx[k][i], cd[i] = rd[k][i];
                }
                shift();
                if (t < t2) {
                    if (t == q.s1) {
                        next_seq(q, p.cu, p.n_seq, t);
                        load_window<T, NC, W, VEC>(win, p, xs, t, q, c, n);
                    }
                    if (p.dfinal && t < t1 && t >= q.s1 - (W - 1)) {
                        uint32_t raw[NW];
                        ld_row<T, NC, VEC>(
                            raw, (const T *)p.dfinal + ((int64_t)q.seg * (W - 1) + t - (q.s1 - (W - 1))) * p.D + c, n);
                        words_to_pairs<T, NC>(pend[0], raw);
                    }
                    token(t, cx, cd, t < t1, false);
                }
                const int done = t - (W - 1);
                if (done >= t0 && done < t1) st_pairs<T, NC, VEC>(op, pend[W - 1], n);
                op += p.D;
            }
        };
        for (int tb = t0; tb < t1 + W - 1; tb += U) {
            uint32_t rx[U][NW], rd[U][NW];
            Rows::arrived();
            in_x.take(rx, got), in_d.take(rd, got++);
            fetch();
            // without a branch: tokens that, with the W - 1 before and after them, are one sequence's
            const bool inside = tb - (W - 1) >= q.s0;
            if (inside && tb + U <= t1 && tb + U <= q.s1 - (W - 1)) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    shift();
                    token(tb + u, rx[u], rd[u], true, true);
                    if (u >= W - 1 || tb + u - (W - 1) >= t0) st_pairs<T, NC, VEC>(op, pend[W - 1], n);
                    op += p.D;
                }
            } else if (W - 1 <= U && inside && tb == t1 && t2 == t1 + W - 1 && t2 <= q.s1) {  // the run's last
#pragma unroll
                for (int u = 0; u < (W - 1 < U ? W - 1 : U); ++u) {
                    shift();
                    token(tb + u, rx[u], rd[u], false, true);
                    st_pairs<T, NC, VEC>(op, pend[W - 1], n);
                    op += p.D;
                }
            } else {
                slow(tb, rx, rd);
            }
        }
    }
    // the CTA's share of dw and db
    constexpr int Q = NC * (W + 1);
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
#pragma unroll
        for (int j = 0; j <= W; ++j) {
            const float2 f = unpack2(j < W ? dw[j < W ? j : 0][i] : db[i]);
            const int r0 = j < W ? 2 * i * W + j : NC * W + 2 * i, r1 = j < W ? r0 + W : r0 + 1;
            red[(threadIdx.y * Q + r0) * 32 + threadIdx.x] = f.x;
            red[(threadIdx.y * Q + r1) * 32 + threadIdx.x] = f.y;
        }
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
    f32x2 a[NC / 2], v[NC / 2], w[W][NC / 2];
    uint32_t raw[W][NW];
    if (slot < 0 || slot >= p.n_slots) {  // a padding row
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) a[i] = pack2(0.f, 0.f);
        st_pairs<T, NC, VEC>(out, a, n);
        return;
    }
    T *state = (T *)p.state + (int64_t)slot * (W - 1) * p.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) ld_row<T, NC, VEC>(raw[j], state + (int64_t)j * p.D, n);
    ld_row<T, NC, VEC>(raw[W - 1], (const T *)p.x + (int64_t)i0 * p.x_st + c, n);
    load_taps<T, NC, W, VEC>(w, a, p.weight, p.bias, c, n);
#pragma unroll
    for (int j = W - 1; j >= 0; --j) {
        words_to_pairs<T, NC>(v, raw[j]);
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) a[i] = fma2(w[j][i], v[i], a[i]);
        if (j > 0) st_row<T, NC, VEC>(state + (int64_t)(j - 1) * p.D, raw[j], n);
    }
    if (p.silu) {
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) {
            a[i] = mul2(a[i], sigmoid_pair(a[i]));
        }
    }
    st_pairs<T, NC, VEC>(out, a, n);
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
    constexpr int NC = 4;
    // Tokens a thread: 32, where W - 1 more inputs are read for each run, or down
    // to 8 while that leaves SMs without a CTA.
    int run = 32;
    auto blocks = [&] { return (int)(((int64_t)p.T + kConvY * run - 1) / (kConvY * run)); };
    while (run > 8 && (int64_t)blocks() * ((p.D + 32 * NC - 1) / (32 * NC)) * p.B < 608) run /= 2;
    const int nblk = blocks();
    const bool extra = p.cu != nullptr || p.T == 0;
    const dim3 grid(nblk + (extra ? 1 : 0), (p.D + 32 * NC - 1) / (32 * NC), p.T == 0 ? 1 : p.B), block(32, kConvY);
    return by_taps(p.W, [&](auto w) {
        if (p.vec) conv_kernel<T, NC, w(), true><<<grid, block, 4 * Ahead<T, NC, 4, true, 32 * kConvY, kAhead>::words(), st>>>(p, nblk, run);
        else conv_kernel<T, NC, w(), false><<<grid, block, 0, st>>>(p, nblk, run);
        return cudaGetLastError();
    });
}
template <typename T>
cudaError_t conv_bwd_t(const ConvParams &p, cudaStream_t st) {
    constexpr int NC = 4;
    const int run = conv_bwd_run(p.B, p.T, p.D), nblk = conv_bwd_parts(1, p.T, run);
    const bool extra = p.cu != nullptr || p.dinit;
    const dim3 grid(nblk + (extra ? 1 : 0), (p.D + 32 * NC - 1) / (32 * NC), p.T == 0 ? 1 : p.B),
        block(32, kConvYBwd);
    return by_taps(p.W, [&](auto w) {
        constexpr int smem = (int)sizeof(float) * 32 * kConvYBwd * NC * (w() + 1);
        if (p.vec) {
            constexpr int all = smem + 8 * Ahead<T, NC, 4, true, 32 * kConvYBwd, kAheadBwd<T>>::words();
            const cudaError_t e =
                cudaFuncSetAttribute(conv_bwd_kernel<T, NC, w(), true>, cudaFuncAttributeMaxDynamicSharedMemorySize, all);
            if (e != cudaSuccess) return e;
            conv_bwd_kernel<T, NC, w(), true><<<grid, block, all, st>>>(p, nblk, run);
            return cudaGetLastError();
        }
        conv_bwd_kernel<T, NC, w(), false><<<grid, block, smem, st>>>(p, nblk, run);
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
// Tokens a thread of the gradient: 64, whose W - 1 tokens on either side cost
// little, or down to 16 while that leaves SMs without a CTA.
int conv_bwd_run(int B, int T, int D) {
    int run = 64;
    while (run > 16 && (int64_t)conv_bwd_parts(B, T, run) * ((D + 127) / 128) < 304) run /= 2;
    return run;
}
// CTAs along the tokens of all rows: each leaves one row of partial sums
int conv_bwd_parts(int B, int T, int run) {
    return B * (int)(((int64_t)T + kConvYBwd * run - 1) / (kConvYBwd * run));
}
cudaError_t launch_conv_bwd(const ConvParams &p, cudaStream_t st) {
    return p.bf16 ? conv_bwd_t<__nv_bfloat16>(p, st) : conv_bwd_t<float>(p, st);
}
cudaError_t launch_conv_step(const ConvStepParams &p, cudaStream_t st) {
    return p.bf16 ? conv_step_t<__nv_bfloat16>(p, st) : conv_step_t<float>(p, st);
}

}  // namespace gdn

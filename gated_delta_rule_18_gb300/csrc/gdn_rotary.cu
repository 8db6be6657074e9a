// gdn_rotary.cu -- rotary positions: the first `rot` channels of every head of
// q and k are turned in pairs, pair j of a token at position p by the angle
// p f_j,
//   (a, b) -> scale (a cos - b sin, b cos + a sin),
// where the pairs are channels (2 j, 2 j + 1) (interleaved) or (j, j + rot / 2)
// (half); the other channels pass. The gradient is the same map with the
// opposite angle.
//
// The angle is formed in turns, in fixed point: f_j / 2 pi to 2^-128 of a turn,
// times the position modulo one turn, which the integer product's overflow is.
// An fp32 product of a far position has none of the angle left.
//
// Bound by HBM: a head's row is read and written once. A CTA turns a few
// tokens, whose cosines and sines are formed once, in shared memory, and serve
// all heads of q and k. A thread keeps one piece of a head (8 pairs in bf16 as
// two vectors of the halves, 4 as one interleaved) of one token, its cosines
// and sines in registers, and walks the token's heads with several heads'
// loads under way.
//
// Measured, bf16 (copy rate 6.78 TB/s): 4 x 4096 tokens, 32 + 8 heads of 128
// channels, halves, 56 us (49.5 at the copy rate); 2 x 8192, 16 + 16 heads of 112
// with 64 turning, interleaved, 44, out of wider rows (34.6). Loads on their way
// are the largest stall (20 warps a SM, 80 registers). In fp32 103 (96 %) and 73 (95 %).
// With cosines read again for every head and fp64 angles it took 66 and 68. Parts whose
// half is not whole vectors (interleaved: the part) and rows off 16 bytes go by
// single elements, two heads under way: 4 x 4096 tokens, 32 + 8 heads of 96 channels
// with 24 turning in halves, bf16, 177 us (37 at the copy rate; interleaved, by vectors,
// 46), of 80 with 20 or 40 turning 157 (31).
#include "gdn_ssm.cuh"
#include "gdn_block.cuh"

#include <type_traits>

namespace gdn {
namespace {

constexpr int kThreads = 256;

// The angle pos f as a fraction of a turn in units of 2^-64, in integers (a
// GB300 SM takes 16 cycles for a warp's fp64 instruction): f = m 2^e with 53
// bits of m, times 2^66 / 2 pi in 64 (rounded: 1.3e-21 of itself off), shifted to units
// of 2^-128, times the position; whole turns fall off. What is left of it is as
// good as f is, whose own half step is 2^-53: pos f 1.3e-21 radians off for an exact
// f, 6e-3 at position 2^62 of f = 1.
__device__ __forceinline__ unsigned long long turn_of(long long pos, double f) {
    const unsigned long long bits = (unsigned long long)__double_as_longlong(f), kTurn = 0xA2F9836E4E44152Aull;
    const int field = (int)(bits >> 52 & 0x7ff);
    const unsigned long long m = (bits & 0xfffffffffffffull) | (field ? 1ull << 52 : 0ull);
    unsigned long long hi = __umul64hi(m, kTurn), lo = m * kTurn;
    int s = 1013 - (field ? field : 1);  // f / 2 pi = (hi, lo) 2^-(s + 128)
    if (s >= 64) lo = hi, hi = 0, s -= 64;
    if (s <= -64) hi = lo, lo = 0, s += 64;
    if (s >= 64 || s <= -64) hi = lo = 0;
    else if (s > 0) lo = hi << (64 - s) | lo >> s, hi >>= s;
    else if (s < 0) hi = hi << -s | lo >> (64 + s), lo <<= -s;
    const unsigned long long at = pos < 0 ? 0ull - (unsigned long long)pos : (unsigned long long)pos;
    const unsigned long long t = at * hi + __umul64hi(at, lo);
    return (pos < 0) != (bool)(bits >> 63) ? 0ull - t : t;
}

// Pieces of a head: those that turn, then those that pass (as many vectors).
template <typename T, bool VEC, bool HALF>
struct Piece {
    static constexpr bool kTwo = HALF || !VEC;           // two vectors, else one of whole pairs
    static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;  // channels of a vector
    static constexpr int P = kTwo ? V : V / 2;               // pairs
    static constexpr int kHeads = VEC ? HALF ? 4 : 8 : 2;    // heads under way
};

template <typename T, bool VEC, bool HALF>
__global__ void __launch_bounds__(kThreads, 3) rotary_kernel(const RotaryParams p, int pieces, int head_lanes, int tokens) {
    using X = Piece<T, VEC, HALF>;
    constexpr int V = X::V, P = X::P, N = X::kHeads, K = X::kTwo ? 2 : 1, W = VEC ? 4 : 1;
    extern __shared__ __align__(16) float table[];  // cosines, sines: [token][rot / 2]
    const int pairs = p.rot >> 1, ld = (pairs + 3) & ~3, turn = pairs / P;
    float *cs = table, *sn = table + tokens * ld;
    const unsigned n_tok = (unsigned)p.B * (unsigned)p.T, tok0 = blockIdx.x * (unsigned)tokens;  // (below 2^31)
    const int toks = min((int)(n_tok - tok0), tokens);
    const int lanes = pieces < kThreads ? pieces : kThreads, g = threadIdx.x / lanes, k = g / head_lanes;
    const int h0 = g - k * head_lanes;
    const bool live = k < toks;
    const unsigned b = (tok0 + k) / (unsigned)p.T, t = tok0 + k - b * p.T;
    int u = threadIdx.x - g * lanes;
    // the piece's vectors: their first channels
    int ca, cb;
    bool turns, two;
    auto piece = [&]() {
        turns = u < turn;
        ca = turns ? (X::kTwo && !HALF ? 2 * u : u * V) : p.rot + (u - turn) * V * K;
        cb = turns ? (HALF ? ca + pairs : ca + 1) : ca + V;
        two = K == 2 && (turns || cb < p.D);  // a passing piece may end with its first vector
    };
    // N heads from h on, `in` pointing at the first of them
    uint32_t w[N][K][W];
    auto load = [&](const RotaryTensor &x, const T *in, int h) {
        const int64_t step = head_lanes * x.in_sh;
#pragma unroll
        for (int i = 0; i < N; ++i, in += step) {
            if (h + i * head_lanes >= x.H) break;
            if constexpr (VEC) {
                ld_words(w[i][0], in + ca);
                if (two) ld_words(w[i][K - 1], in + cb);
            } else {
                w[i][0][0] = __float_as_uint((float)in[ca]);
                if (two) w[i][K - 1][0] = __float_as_uint((float)in[cb]);
            }
        }
    };
    const T *const q0 = (const T *)p.x[0].in + b * p.x[0].in_sb + t * p.x[0].in_st + h0 * p.x[0].in_sh;
    piece();
    // the first heads' loads are under way while the cosines are formed
    bool loaded = live && u < pieces && (turns || p.x[0].copy);
    if (loaded) load(p.x[0], q0, h0);
    for (int e = threadIdx.x; e < toks * pairs; e += kThreads) {
        const int q = e / pairs, j = e - q * pairs;
        const unsigned bq = (tok0 + q) / (unsigned)p.T, tq = tok0 + q - bq * p.T;
        const int64_t at = bq * p.p_sb + tq * p.p_st;
        const long long pos = !p.pos ? p.offset + (long long)tq : p.pos64 ? ((const long long *)p.pos)[at] : ((const int *)p.pos)[at];
        const unsigned long long a = turn_of(pos, p.inv_freq[j]);
        float s, c;
        sincospif((float)(int)(a >> 32) * 0x1p-31f, &s, &c);
        cs[q * ld + j] = c * p.scale, sn[q * ld + j] = s * p.scale * p.sign;
    }
    __syncthreads();
    if (!live) return;
    for (; u < pieces; u += lanes, loaded = false) {
        piece();
        float c[P], s[P];
        if (turns) {
            const float *c_at = cs + k * ld + u * P, *s_at = sn + k * ld + u * P;
            if constexpr (P % 4 == 0) {
                uint32_t cw[P], sw[P];
                ld_words(cw, c_at), ld_words(sw, s_at);
                words_to_f<float, P>(c, cw), words_to_f<float, P>(s, sw);
            } else {
#pragma unroll
                for (int j = 0; j < P; ++j) c[j] = c_at[j], s[j] = s_at[j];
            }
        }
        auto heads = [&](const RotaryTensor &x, const T *in, bool have) {
            if (!turns && !x.copy) return;
            T *out = (T *)x.out + b * x.out_sb + t * x.out_st + h0 * x.out_sh;
            const int64_t step = head_lanes * x.out_sh;
#pragma unroll 1
            for (int h = h0; h < x.H; h += N * head_lanes, have = false) {
                if (!have) load(x, in, h);
                in += N * head_lanes * x.in_sh;
#pragma unroll
                for (int i = 0; i < N; ++i, out += step) {
                    if (h + i * head_lanes >= x.H) continue;
                    if constexpr (!VEC) {
                        const float a = __uint_as_float(w[i][0][0]), d = __uint_as_float(w[i][1][0]);
                        out[ca] = to_type<T>(turns ? a * c[0] - d * s[0] : a);
                        if (two) out[cb] = to_type<T>(turns ? d * c[0] + a * s[0] : d);
                    } else {
                        if (turns) {
                            float a[V], d[V];
                            words_to_f<T, V>(a, w[i][0]);
                            if constexpr (HALF) {
                                words_to_f<T, V>(d, w[i][1]);
#pragma unroll
                                for (int j = 0; j < V; ++j) {
                                    const float y = a[j] * c[j] - d[j] * s[j];
                                    d[j] = d[j] * c[j] + a[j] * s[j], a[j] = y;
                                }
                                f_to_words<T, V>(w[i][1], d);
                            } else {
#pragma unroll
                                for (int j = 0; j < P; ++j) {
                                    const float y = a[2 * j] * c[j] - a[2 * j + 1] * s[j];
                                    a[2 * j + 1] = a[2 * j + 1] * c[j] + a[2 * j] * s[j], a[2 * j] = y;
                                }
                            }
                            f_to_words<T, V>(w[i][0], a);
                        }
                        st_words(out + ca, w[i][0]);
                        if (two) st_words(out + cb, w[i][K - 1]);
                    }
                }
            }
        };
        heads(p.x[0], q0, loaded);
        if (p.x[1].H) heads(p.x[1], (const T *)p.x[1].in + b * p.x[1].in_sb + t * p.x[1].in_st + h0 * p.x[1].in_sh, false);
    }
}

template <typename T, bool VEC, bool HALF>
cudaError_t rotary(const RotaryParams &p, cudaStream_t st) {
    using X = Piece<T, VEC, HALF>;
    const int64_t n_tok = (int64_t)p.B * p.T;
    const int vecs = X::V * (X::kTwo ? 2 : 1);
    const int pieces = p.rot / 2 / X::P + (p.x[0].copy | p.x[1].copy ? (p.D - p.rot + vecs - 1) / vecs : 0);
    const int groups = kThreads / (pieces < kThreads ? pieces : kThreads), heads = p.x[0].H > p.x[1].H ? p.x[0].H : p.x[1].H;
    // A thread's heads: as many as are under way, fewer where the tokens alone would not fill the
    // GPU; what the CTA's groups leave takes tokens.
    int lanes = 1;
    while (lanes < groups && lanes < heads && (lanes * (VEC ? X::kHeads : 4) < heads || n_tok * lanes < (int64_t)groups * 608)) lanes *= 2;
    if (lanes > groups) lanes = groups;
    int tokens = groups / lanes;
    const int most = 32 * 1024 / (((p.rot / 2 + 3) & ~3) * 8);  // of shared memory
    if (tokens > most) tokens = most;
    const int smem = tokens * ((p.rot / 2 + 3) & ~3) * 8;
    const int64_t grid = (n_tok + tokens - 1) / tokens;
    rotary_kernel<T, VEC, HALF><<<(unsigned)grid, kThreads, smem, st>>>(p, pieces, lanes, tokens);
    return cudaGetLastError();
}
template <typename T>
cudaError_t rotary_form(const RotaryParams &p, cudaStream_t st) {
    if (p.interleaved) return p.vec ? rotary<T, true, false>(p, st) : rotary<T, false, false>(p, st);
    return p.vec ? rotary<T, true, true>(p, st) : rotary<T, false, true>(p, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams &p, cudaStream_t st) {
    return p.bf16 ? rotary_form<__nv_bfloat16>(p, st) : rotary_form<float>(p, st);
}

}  // namespace gdn

// gdn_lru.cuh -- what the gated recurrence's kernels share: the gates of a
// channel pair, the marks of a warp's tokens, the joining of runs.
#pragma once

#include "gdn_block.cuh"
#include "gdn_ssm.cuh"

#include <type_traits>

namespace gdn {

constexpr int kLruWarps = 8, kLruLen = 8;  // a tile: eight warps of eight tokens
constexpr int kLruCh = 64;                 // channels a CTA, two a lane
static_assert(kLruWarps * kLruLen == kLruTile, "a CTA's tile");

// 1 - exp(-y) for y >= 0 and a2 = exp(-y): by the series where the difference
// cancels (y < 1/8: the first term left out is y^5 / 720 of the value, 4e-8)
__device__ __forceinline__ f32x2 one_minus_exp(f32x2 y, f32x2 a2) {
    f32x2 s = fma2(y, pack2(1.f / 120.f, 1.f / 120.f), pack2(-1.f / 24.f, -1.f / 24.f));
    s = fma2(s, y, pack2(1.f / 6.f, 1.f / 6.f));
    s = fma2(s, y, pack2(-0.5f, -0.5f));
    s = fma2(s, y, pack2(1.f, 1.f));
    const float2 t = unpack2(mul2(s, y)), v = unpack2(y), f = unpack2(fma2(a2, pack2(-1.f, -1.f), pack2(1.f, 1.f)));
    return pack2(v.x < 0.125f ? t.x : f.x, v.y < 0.125f ? t.y : f.y);
}
__device__ __forceinline__ f32x2 sqrt_2(f32x2 x) {
    float2 v = unpack2(x);
    asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(v.x));
    asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(v.y));
    return pack2(v.x, v.y);
}
// 1 / sqrt(x), 1e18 or more where x is 0
__device__ __forceinline__ f32x2 rsqrt_2(f32x2 x) {
    float2 v = unpack2(x);
    v.x = fmaxf(v.x, 1e-37f), v.y = fmaxf(v.y, 1e-37f);
    asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(v.x));
    asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(v.y));
    return pack2(v.x, v.y);
}
// Sigmoids of a pair, 1 / (1 + exp(-v)): exactly 0 where exp(-v) overflows, and
// a NaN stays a NaN and its own. A reciprocal each: one for two values would
// have to keep their product finite (comparisons and selections, which cost
// more than the reciprocal does).
__device__ __forceinline__ f32x2 sigmoid_2(f32x2 v) {
    const float2 d = unpack2(add2(ex2_2(mul2(v, pack2(-kLog2e, -kLog2e))), pack2(1.f, 1.f)));
    return pack2(rcpf(d.x), rcpf(d.y));
}
// u = c softplus(lam) sigmoid(r): a = exp(-u), q = 1 - a^2. cl: c softplus(lam).
struct LruGate {
    f32x2 u, a, q, gr, gi;
    __device__ __forceinline__ LruGate(f32x2 r, f32x2 i, f32x2 cl) {
        gr = sigmoid_2(r), gi = sigmoid_2(i);
        u = mul2(cl, gr);
        a = ex2_2(mul2(u, pack2(-kLog2e, -kLog2e)));
        q = one_minus_exp(add2(u, u), mul2(a, a));
    }
};
// c softplus(lam) of a channel
__device__ __forceinline__ float lru_decay(float lam, float c) {
    return c * softplus2(make_float2(lam, lam)).x;
}

// Which of a warp's tokens t0 .. t0 + kLruLen - 1 of a packed batch begin a
// sequence (cut) and which end one (fin); nothing past the line. A dense
// line has none: its state and gradient go in and out as the carries.
struct LruMarks {
    unsigned cut, fin;
};
__device__ __forceinline__ LruMarks lru_marks(const int32_t *cu, int n_seq, int T, int t0) {
    LruMarks m{0u, 0u};
    if (t0 >= T) return m;
    SsmSeq q = ssm_find(cu, n_seq, T, 0, t0);
    m.cut = q.starts;
    while (q.end - t0 <= kLruLen) {
        m.fin |= 1u << (q.end - 1 - t0);
        const int t = q.end;
        if (t >= T || t - t0 >= kLruLen) break;
        m.cut |= 1u << (t - t0);
        ssm_next(q, cu, n_seq, T, t);
    }
    return m;
}
__device__ __forceinline__ int lru_seq(const int32_t *cu, int n_seq, int T, int t) { return ssm_find(cu, n_seq, T, 0, t).seg; }

// A run of tokens maps the value before it to A v + H. A run in which a
// sequence begins passes nothing: its A is -0 (others are not negative), and
// what a product would make of a non-finite v stays out.
__device__ __forceinline__ float lru_apply(float A, float H, float v) { return __float_as_int(A) < 0 ? H : fmaf(A, v, H); }
template <bool CUTS>
__device__ __forceinline__ f32x2 lru_apply2(f32x2 A, f32x2 H, f32x2 v) {
    if (!CUTS) return fma2(A, v, H);
    const float2 a = unpack2(A), h = unpack2(H), x = unpack2(v);
    return pack2(lru_apply(a.x, h.x, x.x), lru_apply(a.y, h.y, x.y));
}
// the product of two runs' A
template <bool CUTS>
__device__ __forceinline__ f32x2 lru_join(f32x2 a, f32x2 b) {
    if (!CUTS) return mul2(a, b);
    const float2 x = unpack2(a), y = unpack2(b);
    return pack2((__float_as_int(x.x) | __float_as_int(y.x)) < 0 ? -0.f : x.x * y.x,
                 (__float_as_int(x.y) | __float_as_int(y.y)) < 0 ? -0.f : x.y * y.y);
}
struct alignas(16) LruRun {
    f32x2 A, H;
};

// --------------------------------------------------------- clusters ---------
constexpr int kLruRanks = 8;  // most CTAs of a cluster
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The runs of a step's tiles, of the warps here and of the cluster's CTAs. The
// ranks' are sent by asynchronous stores that count their bytes on the
// receiver's barrier: no fence, and no wait for a CTA's outputs on their way
// to memory, as a barrier of the cluster has it. Two steps' places: a CTA
// sends step n + 2 after it has step n + 1 of all others, and they send that
// after they have read step n.
struct LruRanks {
    LruRun runs[2][kLruRanks][32];
    unsigned long long bar[2];
    __device__ __forceinline__ void init() {  // one thread; then a sync of the cluster
        mbar_init(smem_u32(&bar[0]), 1), mbar_init(smem_u32(&bar[1]), 1);
        fence_mbar_init();
    }
    // one warp: this CTA's run of step n to every CTA of the cluster
    __device__ __forceinline__ void send(int n, int K, int rank, const LruRun &v) {
        const int flip = n & 1, lane = threadIdx.x & 31;
        if (lane == 0) arrive_expect_tx(smem_u32(&bar[flip]), K * 32 * (int)sizeof(LruRun));
        __syncwarp();
        const float2 A = unpack2(v.A), H = unpack2(v.H);
        const uint32_t to = smem_u32(&runs[flip][rank][lane]), on = smem_u32(&bar[flip]);
        for (int k = 0; k < K; ++k)
            asm volatile(
                "{\n .reg .b32 a, b;\n mapa.shared::cluster.u32 a, %0, %2;\n mapa.shared::cluster.u32 b, %1, %2;\n"
                " st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [a], {%3, %4, %5, %6}, [b];\n}" ::"r"(to),
                "r"(on), "r"(k), "r"(__float_as_uint(A.x)), "r"(__float_as_uint(A.y)), "r"(__float_as_uint(H.x)),
                "r"(__float_as_uint(H.y))
                : "memory");
    }
    // false after about half a second
    __device__ __forceinline__ bool wait(int n) const {
        const uint32_t at = smem_u32(&bar[n & 1]), parity = n >> 1 & 1;
        uint64_t t0 = 0;
        for (uint32_t it = 0;; ++it) {
            uint32_t ok;
            asm volatile(
                "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
                " selp.u32 %0, 1, 0, p;\n}"
                : "=r"(ok)
                : "r"(at), "r"(parity)
                : "memory");
            if (ok) return true;
            if ((it & 255) == 255) {
                const uint64_t t = now_ns();
                if (t0 == 0) t0 = t;
                else if (t - t0 > 500000000ull) return false;
            }
        }
    }
};

// --------------------------------------------------------- staging ----------
// A warp's rows of one tensor (kLruLen tokens x kLruCh channels) into shared
// memory by 16-byte asynchronous copies; rows from `rows` on and channels from n
// on are zeros. Only the warp itself reads them.
template <typename T>
__device__ __forceinline__ void lru_copy(T *dst, const T *src, int64_t st, int rows, int n) {
    constexpr int VE = 16 / (int)sizeof(T), kRow = kLruCh / VE, kCopies = kLruLen * kRow;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < kCopies / 32; ++k) {
        const int e = lane + 32 * k, r = e / kRow, c = e % kRow * VE;
        const bool in = r < rows && c < n;
        cp_async16(dst + r * kLruCh + c, in ? src + r * st + c : src, in ? 16 : 0);
    }
}
template <typename T>
__device__ __forceinline__ f32x2 lru_pair(const T *p) {  // of a staged row
    uint32_t w[RowVec<T, 2>::kWords];
    ld_words(w, p);
    float f[2];
    words_to_f<T, 2>(f, w);
    return pack2(f[0], f[1]);
}
template <typename T, bool VEC>
__device__ __forceinline__ void lru_put(T *p, f32x2 v, int nc) {
    const float2 f = unpack2(v);
    const float o[2] = {f.x, f.y};
    st_row_f<T, 2, VEC>(p, o, nc);
}
// two channels of a row of states, of which nc exist; zeros without a tensor
__device__ __forceinline__ f32x2 lru_ld_state(const float *s, int64_t row, int C, int c, int nc) {
    float2 f = make_float2(0.f, 0.f);
    if (s && nc > 0) f.x = s[row * C + c];
    if (s && nc > 1) f.y = s[row * C + c + 1];
    return pack2(f.x, f.y);
}
__device__ __forceinline__ void lru_st_state(float *s, int64_t row, int C, int c, int nc, f32x2 v) {
    const float2 f = unpack2(v);
    if (nc > 0) s[row * C + c] = f.x;
    if (nc > 1) s[row * C + c + 1] = f.y;
}

// f(element, wide rows, packed batch, with z) for a call's form
template <class F>
cudaError_t lru_by_form(const LruParams &p, bool with_z, F &&f) {
    const std::true_type yes;
    const std::false_type no;
    auto by_z = [&](auto t, auto v, auto k) { return with_z ? f(t, v, k, yes) : f(t, v, k, no); };
    auto by_cu = [&](auto t, auto v) { return p.cu ? by_z(t, v, yes) : by_z(t, v, no); };
    auto by_vec = [&](auto t) { return p.vec ? by_cu(t, yes) : by_cu(t, no); };
    return p.bf16 ? by_vec(__nv_bfloat16()) : by_vec(float());
}
cudaError_t lru_launch(const void *kernel, int lines, int C, int ranks, int smem, const LruParams &p, cudaStream_t st);

}  // namespace gdn

// gdn_lru.cuh -- what the gated recurrence's kernels share: the gates of a
// channel pair, the marks of a warp's tokens, the joining of runs.
#pragma once

#include "gdn_block.cuh"
#include "gdn_ssm.cuh"

namespace gdn {

constexpr int kLruWarps = 8, kLruLen = 8;  // a tile: eight warps of eight tokens
constexpr int kLruCh = 64;                 // channels a CTA, two a lane
static_assert(kLruWarps * kLruLen == kLruTile, "a CTA's tile");

__device__ __forceinline__ f32x2 max2(f32x2 a, float b) {
    const float2 v = unpack2(a);
    return pack2(fmaxf(v.x, b), fmaxf(v.y, b));
}
// 1 - exp(-y) for y >= 0 and a2 = exp(-y): by the series where the difference
// cancels (y < 1/4: the first term left out is y^6 / 5040 of the value, 5e-8)
__device__ __forceinline__ f32x2 one_minus_exp(f32x2 y, f32x2 a2) {
    f32x2 s = fma2(y, pack2(-1.f / 720.f, -1.f / 720.f), pack2(1.f / 120.f, 1.f / 120.f));
    s = fma2(s, y, pack2(-1.f / 24.f, -1.f / 24.f));
    s = fma2(s, y, pack2(1.f / 6.f, 1.f / 6.f));
    s = fma2(s, y, pack2(-0.5f, -0.5f));
    s = fma2(s, y, pack2(1.f, 1.f));
    const float2 t = unpack2(mul2(s, y)), f = unpack2(a2), v = unpack2(y);
    return pack2(v.x < 0.25f ? t.x : 1.f - f.x, v.y < 0.25f ? t.y : 1.f - f.y);
}
__device__ __forceinline__ float sqrt_approx(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// The sigmoids of a channel pair's two gates, by e = exp(-|v|) <= 1 as
// sigmoid2; one reciprocal serves both gates of a channel (a NaN of one reaches
// the other, and both make the same state).
__device__ __forceinline__ void sigmoids(f32x2 r, f32x2 i, f32x2 &gr, f32x2 &gi) {
    const float2 a = unpack2(r), b = unpack2(i);
    const f32x2 one = pack2(1.f, 1.f);
    const f32x2 ea = pack2(ex2f(-fabsf(a.x) * kLog2e), ex2f(-fabsf(a.y) * kLog2e));
    const f32x2 eb = pack2(ex2f(-fabsf(b.x) * kLog2e), ex2f(-fabsf(b.y) * kLog2e));
    const f32x2 da = add2(ea, one), db = add2(eb, one);
    const float2 d = unpack2(mul2(da, db));
    const f32x2 q = pack2(rcpf(d.x), rcpf(d.y));
    const f32x2 ra = mul2(q, db), rb = mul2(q, da);
    const float2 pa = unpack2(ra), na = unpack2(mul2(ra, ea)), pb = unpack2(rb), nb = unpack2(mul2(rb, eb));
    gr = pack2(a.x < 0.f ? na.x : pa.x, a.y < 0.f ? na.y : pa.y);
    gi = pack2(b.x < 0.f ? nb.x : pb.x, b.y < 0.f ? nb.y : pb.y);
}
// u = c softplus(lam) sigmoid(r): a = exp(-u), q = 1 - a^2
struct LruGate {
    f32x2 u, a, q, gr, gi;
    __device__ __forceinline__ LruGate(f32x2 r, f32x2 i, f32x2 cl) {
        sigmoids(r, i, gr, gi);
        u = mul2(cl, gr);
        a = ex2_2(mul2(u, pack2(-kLog2e, -kLog2e)));
        q = one_minus_exp(add2(u, u), mul2(a, a));
    }
    __device__ __forceinline__ f32x2 beta() const {
        const float2 f = unpack2(q);
        return pack2(sqrt_approx(f.x), sqrt_approx(f.y));
    }
};
// c softplus(lam) of a channel
__device__ __forceinline__ float lru_decay(float lam, float c) {
    return c * softplus2(make_float2(lam, lam)).x;
}

// Which of a warp's tokens t0 .. t0 + kLruLen - 1 begin a sequence (cut) and
// which end one (fin); nothing past the line.
struct LruMarks {
    unsigned cut, fin;
};
__device__ __forceinline__ LruMarks lru_marks(const int32_t *cu, int n_seq, int T, int t0) {
    LruMarks m{0u, 0u};
    if (t0 >= T) return m;
    if (!cu) {
        m.cut = t0 == 0;
        m.fin = T - 1 - t0 < kLruLen ? 1u << (T - 1 - t0) : 0u;
        return m;
    }
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
__device__ __forceinline__ int lru_seq(const int32_t *cu, int n_seq, int T, int line, int t) {
    return ssm_find(cu, n_seq, T, line, t).seg;
}

// A run of tokens maps the value before it to A v + H. A run in which a
// sequence begins passes nothing: its A is -0 (others are not negative), and
// what a product would make of a non-finite v stays out.
__device__ __forceinline__ float lru_apply(float A, float H, float v) { return __float_as_int(A) < 0 ? H : fmaf(A, v, H); }
__device__ __forceinline__ f32x2 lru_apply2(f32x2 A, f32x2 H, f32x2 v) {
    const float2 a = unpack2(A), h = unpack2(H), x = unpack2(v);
    return pack2(lru_apply(a.x, h.x, x.x), lru_apply(a.y, h.y, x.y));
}
// the product of two runs' A
__device__ __forceinline__ f32x2 lru_join(f32x2 a, f32x2 b) {
    const float2 x = unpack2(a), y = unpack2(b);
    return pack2((__float_as_int(x.x) | __float_as_int(y.x)) < 0 ? -0.f : x.x * y.x,
                 (__float_as_int(x.y) | __float_as_int(y.y)) < 0 ? -0.f : x.y * y.y);
}
struct alignas(16) LruRun {
    f32x2 A, H;
};

// --------------------------------------------------------- clusters ---------
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// stores 16 bytes to the same place of another CTA's shared memory
__device__ __forceinline__ void st_cluster(void *mine, int rank, const LruRun &v) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(at), "l"(v.A), "l"(v.H) : "memory");
}

// --------------------------------------------------------- staging ----------
// A warp's rows of one tensor (kLruLen tokens x kLruCh channels) into shared
// memory by 16-byte asynchronous copies; rows from `rows` on and channels past
// C are zeros. Only the warp itself reads them.
template <typename T>
__device__ __forceinline__ void lru_copy(T *dst, const T *src, int64_t st, int rows, int c0, int C) {
    constexpr int VE = 16 / (int)sizeof(T), kRow = kLruCh / VE, kCopies = kLruLen * kRow;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < kCopies / 32; ++k) {
        const int e = lane + 32 * k, r = e / kRow, c = e % kRow * VE;
        const bool in = r < rows && c0 + c < C;
        cp_async16(dst + r * kLruCh + c, in ? src + r * st + c0 + c : src, in ? 16 : 0);
    }
}
template <typename T>
__device__ __forceinline__ f32x2 lru_pair(const uint32_t (&w)[RowVec<T, 2>::kWords]) {
    float f[2];
    words_to_f<T, 2>(f, w);
    return pack2(f[0], f[1]);
}

cudaError_t lru_launch(const void *kernel, int lines, int C, int ranks, int smem, const LruParams &p, cudaStream_t st);

}  // namespace gdn

// gdn_lru.cuh -- what the gated recurrence's kernels share: the gates of a
// channel pair, the marks of a warp's tokens, the joining of runs.
#pragma once

#include <cuda.h>

#include "gdn_block.cuh"
#include "gdn_ssm.cuh"

#include <type_traits>

namespace gdn {

// A CTA's tile: W warps of L tokens, 64 channels, two a lane; saved states lie
// where warps begin.
constexpr int kLruCh = 64;

// a = exp(-u) (as the unit forms it) and q = 1 - a^2 = (1 - a)(1 + a), for u >=
// 0. Where u < 1/8, both from 1 - a by its series (the first term left out is
// u^5 / 720 of the value, 4e-8): q would cancel, and a product of many a near
// one keeps the unit's error of each (2^-22, of one sign), not a rounding's:
// dlam was 2.5e-6 off after 348 tokens. In scalar instructions: their constants
// are immediates.
// NEAR: all u are below 1/8.
constexpr float kLruNear = 0.125f;
template <bool NEAR>
__device__ __forceinline__ void lru_decay(float &a, float &q, float u) {
    float t = fmaf(u, 1.f / 120.f, -1.f / 24.f);
    t = fmaf(t, u, 1.f / 6.f);
    t = fmaf(t, u, -0.5f);
    t = fmaf(t, u, 1.f);
    const bool near = NEAR || u < kLruNear;
    const float near_a = fmaf(-t, u, 1.f);
    t = near ? __fmul_rn(t, u) : 1.f - a;
    a = near ? near_a : a;
    q = fmaf(t, a, t);
}
template <bool NEAR>
__device__ __forceinline__ void lru_decay2(f32x2 &a, f32x2 &q, f32x2 u) {
    float2 f = unpack2(a), r, v = unpack2(u);
    lru_decay<NEAR>(f.x, r.x, v.x), lru_decay<NEAR>(f.y, r.y, v.y);
    a = pack2(f.x, f.y), q = pack2(r.x, r.y);
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
// What a channel pair's gates are made with: -c softplus(lam) log2(e), c softplus(lam).
struct LruDecay {
    f32x2 base, rate;
    __device__ __forceinline__ LruDecay(const float *lam, float c, int nc) {
        // (each by itself: halves of a pair would share a reciprocal, and its rounding)
        const float x = nc > 0 ? lam[0] : 0.f, y = nc > 1 ? lam[1] : 0.f;
        const float2 s = make_float2(softplus2(make_float2(x, x)).x, softplus2(make_float2(y, y)).x);
        base = pack2(-kLog2e * (c * s.x), -kLog2e * (c * s.y)), rate = pack2(c * s.x, c * s.y);
    }
    // No gate takes any of the warp's channels to u = 1/8: a needs no exponential
    // (4 x 4096 tokens of 4096 channels, bf16: 125 us, with it 133; the same bits).
    __device__ __forceinline__ bool near(int nc) const {
        const float2 f = unpack2(rate);
        return __all_sync(0xffffffffu, (nc < 1 || f.x < kLruNear) && (nc < 2 || f.y < kLruNear));
    }
};
// u = c softplus(lam) sigmoid(r): a = exp(-u), q = 1 - a^2
template <bool NEAR>
struct LruGate {
    f32x2 a, q, gr, gi;
    __device__ __forceinline__ LruGate(f32x2 r, f32x2 i, const LruDecay &d) {
        gr = sigmoid_2(r), gi = sigmoid_2(i);
        a = NEAR ? d.rate : ex2_2(mul2(d.base, gr));
        lru_decay2<NEAR>(a, q, mul2(d.rate, gr));
    }
};
// Which of a warp's tokens t0 .. t0 + L - 1 of a packed batch begin a
// sequence (cut) and which end one (fin); nothing past the line. A dense
// line has none: its state and gradient go in and out as the carries.
struct LruMarks {
    unsigned cut, fin;
};
template <int L>
__device__ __forceinline__ LruMarks lru_marks(const int32_t *cu, int n_seq, int T, int t0) {
    LruMarks m{0u, 0u};
    if (t0 >= T) return m;
    SsmSeq q = ssm_find(cu, n_seq, T, 0, t0);
    m.cut = q.starts;
    while (q.end - t0 <= L) {
        m.fin |= 1u << (q.end - 1 - t0);
        const int t = q.end;
        if (t >= T || t - t0 >= L) break;
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
constexpr int kLruRanks = 16;  // most CTAs of a cluster
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Waits for a phase of a barrier of this CTA; false after the limit.
__device__ __forceinline__ bool lru_wait(uint32_t bar, uint32_t parity, int limit_us) {
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((it & 255) == 0) {
            const uint64_t t = now_ns();
            if (t0 == 0) t0 = t;
            else if (t - t0 > (uint64_t)limit_us * 1000u) return false;
        }
    }
}
// What a warp has given up waiting for. The CTA agrees at the next barrier of the
// walk, before anything that follows from what did not come is passed on, and
// leaves the walk: the warp's tokens of the step in which it gave up, the rest of
// the CTA's tokens and its states become NaN. It sends no more runs, so that the
// other CTAs of the cluster, whose places it may not write any longer, run into
// their own limits. A CTA gives up once and waits (once more, at most) for its
// copies in flight.
enum { kLostRows = 1, kLostRuns = 2, kLostZ = 4 };
// the error word: cleared, with a packed batch's bounds checked, by the call's first kernel
template <bool PACKED>
__device__ __forceinline__ void lru_begin(const LruParams &p) {
    if (!p.err || !p.first || blockIdx.x != 0 || blockIdx.y != 0) return;
    if (PACKED) ssm_check_cu(p.cu, p.n_seq, p.T, p.err);
    else if (threadIdx.x == 0) *p.err = 0;
}
__device__ __forceinline__ bool lru_stalled(const LruParams &p) {
    return p.stall_cta >= 0 && (int64_t)blockIdx.y * gridDim.x + blockIdx.x == p.stall_cta;
}
// The runs of the cluster's CTAs in a step. They are sent by asynchronous
// stores that count their bytes on the receiver's barrier: no fence, and no
// wait for a CTA's outputs on their way to memory, as a barrier of the cluster
// has it. Two steps' places: a CTA sends step n + 2 after it has step n + 1 of
// all others, and they send that after they have read step n.
struct LruRanks {
    LruRun *runs;  // [2][places][32]
    unsigned long long *bar;
    int K, places;  // ranks that are not there change nothing
    static __host__ __device__ constexpr int places_of(int K) { return K == 1 ? 0 : K <= 8 ? 8 : 16; }
    __device__ __forceinline__ LruRun &at(int n, int rank) const { return runs[((n & 1) * places + rank) * 32 + (threadIdx.x & 31)]; }
    // all threads; then a sync of the cluster
    __device__ __forceinline__ void init() const {
        for (int e = threadIdx.x; e < 2 * places * 32; e += blockDim.x)
            if (e / 32 % places >= K) runs[e] = LruRun{pack2(1.f, 1.f), pack2(0.f, 0.f)};
        if (threadIdx.x == 0) {
            mbar_init(smem_u32(&bar[0]), 1), mbar_init(smem_u32(&bar[1]), 1);
            fence_mbar_init();
        }
    }
    // one warp: this CTA's run of step n to every CTA of the cluster
    __device__ __forceinline__ void send(int n, int rank, const LruRun &v) const {
        const uint32_t on = smem_u32(&bar[n & 1]), to = smem_u32(&at(n, rank));
        if ((threadIdx.x & 31) == 0) arrive_expect_tx(on, K * 32 * (int)sizeof(LruRun));
        __syncwarp();
        const float2 A = unpack2(v.A), H = unpack2(v.H);
        for (int k = 0; k < K; ++k)
            asm volatile(
                "{\n .reg .b32 a, b;\n mapa.shared::cluster.u32 a, %0, %2;\n mapa.shared::cluster.u32 b, %1, %2;\n"
                " st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [a], {%3, %4, %5, %6}, [b];\n}" ::"r"(to),
                "r"(on), "r"(k), "r"(__float_as_uint(A.x)), "r"(__float_as_uint(A.y)), "r"(__float_as_uint(H.x)),
                "r"(__float_as_uint(H.y))
                : "memory");
    }
    __device__ __forceinline__ bool wait(int n, int limit_us) const { return lru_wait(smem_u32(&bar[n & 1]), n >> 1 & 1, limit_us); }
};

// --------------------------------------------------------- staging ----------
// How a warp's rows of its tensors (L tokens x kLruCh channels each) get
// into its part of shared memory, which only the warp itself reads: by tensor
// copies, one lane's (rows on 16 bytes; 16-byte copies by all lanes took a
// quarter of the forward's instructions, and a bulk copy a row, which a warp's
// lanes issue one by one, 236 us where all together take 171); by asynchronous
// copies of a word of each lane's pair (rows on any word); or through registers
// (bf16 rows on odd elements).
enum { kLruWide, kLruWords, kLruElements };
// x, r, i, then z, or dout and z: (B, T, C), boxes of a warp's rows
struct LruMaps {
    CUtensorMap m[5];
};
__device__ __forceinline__ void lru_tensor_copy(uint32_t dst, const CUtensorMap *m, int c, int t, int line, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(c), "r"(t), "r"(line), "r"(bar)
        : "memory");
}
// N tensors whose rows are copied together. Rows past the line and channels
// past C hold anything: no lane that exists reads them.
template <typename T, int HOW, int N, int L>
struct LruFetch {
    static constexpr int kRows = L * kLruCh;  // elements of a warp's rows of a tensor
    static constexpr int kHeld = HOW == kLruWide ? 1 : N;
    const T *at[kHeld];
    int64_t st[kHeld];
    const CUtensorMap *maps;  // the tensors', one after another
    int c0, line, n;          // n: channels that exist from the tile's first, c0
    // base[k]: tensor k's line at c0
    __device__ __forceinline__ LruFetch(const T *const (&base)[N], const int64_t (&stride)[N], const CUtensorMap *m, int c, int l, int C)
        : maps(m), c0(c), line(l), n(C - c) {
#pragma unroll
        for (int q = 0; q < kHeld; ++q)
            if (HOW != kLruWide) at[q] = base[q] + 2 * (threadIdx.x & 31), st[q] = stride[q];
    }
    // rows t .. t + rows - 1 (none for rows <= 0) into dst[tensor][kRows];
    // `bar` counts them (one phase a call), or the lane's next group of copies
    __device__ __forceinline__ void copy(T *dst, int t, int rows, uint32_t bar) const {
        const int lane = threadIdx.x & 31;
        if constexpr (HOW == kLruWide) {
            if (lane == 0) {
                if (rows > 0) {
                    arrive_expect_tx(bar, N * kRows * (int)sizeof(T));  // (whole boxes, zeros outside the tensor)
#pragma unroll
                    for (int k = 0; k < N; ++k) lru_tensor_copy(smem_u32(dst + k * kRows), maps + k, c0, t, line, bar);
                } else {
                    arrive(bar);
                }
            }
        } else if constexpr (HOW == kLruWords) {
            constexpr int kWords = 2 * (int)sizeof(T) / 4;
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int j = 0; j < L; ++j)
#pragma unroll
                    for (int w = 0; w < kWords; ++w)
                        if (j < rows && 2 * lane + (kWords == 2 ? w : 1) < n)
                            copy_async<4>(reinterpret_cast<uint32_t *>(dst + k * kRows + j * kLruCh + 2 * lane) + w,
                                          reinterpret_cast<const uint32_t *>(at[k] + (t + j) * st[k]) + w);
            cp_async_commit();
        } else {
            // (with a branch an element the loads wait for one another, 328 us for 226
            // with 4 x 17498 tokens of 167 channels: rows and channels that are not
            // there take the last that are)
            const int d0 = min(2 * lane, n - 1) - 2 * lane, d1 = min(2 * lane + 1, n - 1) - 2 * lane;
            if (rows > 0) {
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    unsigned short lo[L], hi[L];
#pragma unroll
                    for (int j = 0; j < L; ++j) {
                        const unsigned short *e = reinterpret_cast<const unsigned short *>(at[k] + (int64_t)(t + min(j, rows - 1)) * st[k]);
                        lo[j] = e[d0], hi[j] = e[d1];
                    }
#pragma unroll
                    for (int j = 0; j < L; ++j)
                        *reinterpret_cast<uint32_t *>(dst + k * kRows + j * kLruCh + 2 * lane) = lo[j] | (uint32_t)hi[j] << 16;
                }
            }
            cp_async_commit();
        }
    }
    // the copy that is followed by LATER others has arrived
    template <int LATER>
    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, int limit_us) const {
        bool ok = true;
        if constexpr (HOW == kLruWide) ok = lru_wait(bar, parity, limit_us);
        else cp_async_wait<LATER>();
        __syncwarp();
        return ok;
    }
};
// the barriers of a warp's stages: one thread of it; then a sync of the CTA
__device__ __forceinline__ void lru_init_bars(unsigned long long *bars, int n) {
    for (int k = 0; k < n; ++k) mbar_init(smem_u32(bars + k), 1);
    fence_mbar_init();
}
template <typename T>
__device__ __forceinline__ f32x2 lru_pair(const T *p) {  // of a staged row
    uint32_t w[RowVec<T, 2>::kWords];
    ld_words(w, p);
    float f[2];
    words_to_f<T, 2>(f, w);
    return pack2(f[0], f[1]);
}
// pairs on a boundary of their own size are stored whole
template <typename T, int HOW>
__device__ __forceinline__ void lru_put(T *p, f32x2 v, int nc) {
    const float2 f = unpack2(v);
    const float o[2] = {f.x, f.y};
    st_row_f<T, 2, HOW == kLruWide || (HOW == kLruWords && sizeof(T) == 2)>(p, o, nc);
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

// f(element, how rows are copied, packed batch, with z) for a call's form
template <class F>
cudaError_t lru_by_form(const LruParams &p, int how, bool with_z, F &&f) {
    const std::true_type yes;
    const std::false_type no;
    auto by_z = [&](auto t, auto h, auto k) { return with_z ? f(t, h, k, yes) : f(t, h, k, no); };
    auto by_cu = [&](auto t, auto h) { return p.cu ? by_z(t, h, yes) : by_z(t, h, no); };
    if (!p.bf16) {
        if (how == kLruWide) return by_cu(float(), std::integral_constant<int, kLruWide>());
        return by_cu(float(), std::integral_constant<int, kLruWords>());
    }
    const __nv_bfloat16 t{};
    if (how == kLruWide) return by_cu(t, std::integral_constant<int, kLruWide>());
    if (how == kLruWords) return by_cu(t, std::integral_constant<int, kLruWords>());
    return by_cu(t, std::integral_constant<int, kLruElements>());
}
// the maps of a call's tensors, boxes of len tokens, into m; false where they have none (a stride
// of zero): its rows are then copied by words
bool lru_maps(const LruParams &p, bool gradient, int len, LruMaps *m);
// smem: the shared memory of a CTA in a cluster of so many
cudaError_t lru_launch(const void *kernel, int warps, int (*smem)(int ranks), LruParams &p, const LruMaps &m, cudaStream_t st);

}  // namespace gdn

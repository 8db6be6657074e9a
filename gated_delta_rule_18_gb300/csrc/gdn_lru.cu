// gdn_lru.cu -- the gated linear recurrence, per channel and sequence:
//   u = c softplus(lam) sigmoid(r),  a = exp(-u),
//   h <- a h + sqrt(1 - a^2) sigmoid(i) x,  out = h silu(z)  (h without z),
// for whole sequences (dense or packed) and for single tokens with the states
// in a pool. h is fp32 throughout.
//
// Bound by HBM on paper (10 bytes a token and channel in bf16). A line of
// tokens is cut in tiles of 64 tokens by 64 channels; a cluster of CTAs takes
// consecutive tiles of the same channels at once and walks the line so. A warp
// has eight tokens of 64 channels: it forms a and the input of each in
// registers and what its run does to the state before it (A v + H); the runs
// are joined over the CTA's warps through shared memory, over the cluster
// through distributed shared memory, in one order, and each warp then walks its
// tokens from its entering state. Inputs are read once, by asynchronous copies
// one tile ahead, and results repeat bit for bit.
#include "gdn_lru.cuh"

namespace gdn {
namespace {

constexpr int kRanks = 8;  // most CTAs of a cluster

struct Exchange {
    LruRun warps[2][kLruWarps][32];
    LruRun ranks[2][kRanks][32];
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kLruWarps, 2) lru_kernel(const LruParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Exchange ex;
    constexpr int KW = RowVec<T, 2>::kWords, kRow = kLruCh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int K = p.ranks, rank = K > 1 ? blockIdx.x % K : 0, line = blockIdx.y;
    const int c0 = (blockIdx.x / K) * kLruCh, c = c0 + 2 * lane, nc = p.C - c;  // nc: channels of the pair that exist
    if (p.err && blockIdx.x == 0 && blockIdx.y == 0) ssm_check_cu(p.cu, p.n_seq, p.T, p.err);
    auto ld_state = [&](const float *s, int64_t row) {
        float2 f = make_float2(0.f, 0.f);
        if (s && nc > 0) f.x = s[row * p.C + c];
        if (s && nc > 1) f.y = s[row * p.C + c + 1];
        return pack2(f.x, f.y);
    };
    auto st_state = [&](float *s, int64_t row, f32x2 v) {
        const float2 f = unpack2(v);
        if (nc > 0) s[row * p.C + c] = f.x;
        if (nc > 1) s[row * p.C + c + 1] = f.y;
    };
    // sequences without tokens keep their states
    if (p.h_final && rank == 0) {
        if (!p.cu) {
            if (p.T == 0 && warp == 0) st_state(p.h_final, line, ld_state(p.h0, line));
        } else {
            for (int s = warp; s < p.n_seq; s += kLruWarps)
                if (p.cu[s + 1] <= p.cu[s]) st_state(p.h_final, s, ld_state(p.h0, s));
        }
    }
    const int steps = (p.T + K * kLruTile - 1) / (K * kLruTile);
    const T *x = (const T *)p.x + line * p.x_sb, *r = (const T *)p.r + line * p.r_sb, *in = (const T *)p.i + line * p.i_sb;
    const T *z = p.z ? (const T *)p.z + line * p.z_sb : nullptr;
    T *out = p.out ? (T *)p.out + line * p.o_sb : nullptr;
    constexpr int kTensor = kLruLen * kRow;  // elements of a warp's rows of one tensor
    T *stage = (T *)smem + warp * 4 * kTensor;
    auto first = [&](int n) { return (n * K + rank) * kLruTile + warp * kLruLen; };  // token of step n
    auto fetch = [&](int n) {
        if constexpr (VEC) {
            const int t = first(n), rows = n < steps ? min(max(p.T - t, 0), kLruLen) : 0;
            if (rows > 0) {
                lru_copy(stage, x + t * p.x_st, p.x_st, rows, c0, p.C);
                lru_copy(stage + kTensor, r + t * p.r_st, p.r_st, rows, c0, p.C);
                lru_copy(stage + 2 * kTensor, in + t * p.i_st, p.i_st, rows, c0, p.C);
                if (z) lru_copy(stage + 3 * kTensor, z + t * p.z_st, p.z_st, rows, c0, p.C);
            }
            cp_async_commit();
        }
    };
    fetch(0);
    float cl[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (k < nc) cl[k] = lru_decay(p.lam[c + k], p.c);
    const f32x2 cl2 = pack2(cl[0], cl[1]);
    f32x2 carry = pack2(0.f, 0.f);  // the state before the cluster's tiles
    if (K > 1) cluster_arrive(), cluster_wait();  // every CTA's shared memory is there
    for (int n = 0; n < steps; ++n) {
        const int t0 = first(n), len = min(max(p.T - t0, 0), kLruLen), flip = n & 1;
        const LruMarks m = lru_marks(p.cu, p.n_seq, p.T, t0);
        if constexpr (VEC) {
            cp_async_wait<0>();
            __syncwarp();
        }
        f32x2 a[kLruLen], b[kLruLen];
        uint32_t zw[kLruLen][KW];
        LruRun run{pack2(1.f, 1.f), pack2(0.f, 0.f)};
#pragma unroll
        for (int j = 0; j < kLruLen; ++j) {
            uint32_t wx[KW] = {}, wr[KW] = {}, wi[KW] = {};
#pragma unroll
            for (int k = 0; k < KW; ++k) zw[j][k] = 0u;
            a[j] = pack2(1.f, 1.f), b[j] = pack2(0.f, 0.f);
            if (j >= len) continue;
            if constexpr (VEC) {
                const T *s = stage + j * kRow + 2 * lane;
                ld_words(wx, s), ld_words(wr, s + kTensor), ld_words(wi, s + 2 * kTensor);
                if (z) ld_words(zw[j], s + 3 * kTensor);
            } else if (nc > 0) {
                const int64_t t = t0 + j;
                ld_row<T, 2, false>(wx, x + t * p.x_st + c, nc), ld_row<T, 2, false>(wr, r + t * p.r_st + c, nc);
                ld_row<T, 2, false>(wi, in + t * p.i_st + c, nc);
                if (z) ld_row<T, 2, false>(zw[j], z + t * p.z_st + c, nc);
            }
            const LruGate g(lru_pair<T>(wr), lru_pair<T>(wi), cl2);
            a[j] = g.a, b[j] = mul2(mul2(g.beta(), g.gi), lru_pair<T>(wx));
            if (m.cut >> j & 1) {
                if (p.h0) b[j] = fma2(g.a, ld_state(p.h0, lru_seq(p.cu, p.n_seq, p.T, line, t0 + j)), b[j]);
                a[j] = pack2(-0.f, -0.f);
                run.A = a[j], run.H = b[j];
            } else {
                run.A = mul2(run.A, a[j]), run.H = fma2(a[j], run.H, b[j]);
            }
        }
        if constexpr (VEC) __syncwarp();
        fetch(n + 1);
        ex.warps[flip][warp][lane] = run;
        __syncthreads();
        // the CTA's run, and the part of it before this warp
        LruRun all{pack2(1.f, 1.f), pack2(0.f, 0.f)}, before = all;
#pragma unroll
        for (int w = 0; w < kLruWarps; ++w) {
            const LruRun v = ex.warps[flip][w][lane];
            if (w == warp) before = all;
            all.H = lru_apply2(v.A, v.H, all.H), all.A = lru_join(all.A, v.A);
        }
        f32x2 h = carry;
        if (K > 1) {
            if (warp < K) st_cluster(&ex.ranks[flip][rank][lane], warp, all);
            cluster_arrive(), cluster_wait();
            for (int k = 0; k < K; ++k) {
                const LruRun v = ex.ranks[flip][k][lane];
                if (k == rank) h = carry;
                carry = lru_apply2(v.A, v.H, carry);
            }
        } else {
            carry = lru_apply2(all.A, all.H, carry);
        }
        h = lru_apply2(before.A, before.H, h);
        if (p.ck && warp * kLruLen % kLruTile == 0 && t0 < p.T)
            st_state(p.ck, (int64_t)line * ((p.T + kLruTile - 1) / kLruTile) + t0 / kLruTile, h);
        if (!p.out && !m.fin) continue;
#pragma unroll
        for (int j = 0; j < kLruLen; ++j) {
            if (j >= len) break;
            h = m.cut >> j & 1 ? b[j] : fma2(a[j], h, b[j]);
            if (p.out && nc > 0) {
                float o[2];
                float2 f = unpack2(h);
                if (z) {
                    const float2 v = unpack2(lru_pair<T>(zw[j])), s = sigmoid2(v);
                    f.x *= v.x * s.x, f.y *= v.y * s.y;
                }
                o[0] = f.x, o[1] = f.y;
                st_row_f<T, 2, VEC>(out + (int64_t)(t0 + j) * p.o_st + c, o, nc);
            }
            if (p.h_final && m.fin >> j & 1) st_state(p.h_final, lru_seq(p.cu, p.n_seq, p.T, line, t0 + j), h);
        }
    }
}

// One token of n requests: four channels a thread.
template <typename T, bool VEC>
__global__ void __launch_bounds__(128) lru_step_kernel(const LruStepParams p) {
    const int c = (blockIdx.x * 128 + threadIdx.x) * 4, n = p.C - c;
    if (n <= 0) return;
    const int64_t req = blockIdx.y;
    const int slot = p.slots ? p.slots[req] : (int)req;
    const bool live = slot >= 0 && slot < p.n_slots;
    float x[4] = {}, r[4] = {}, i[4] = {}, z[4] = {}, lam[4] = {}, h[4] = {};
    float *state = p.state + (int64_t)slot * p.C + c;
    if (live) {
        ld_row_f<float, 4, VEC>(h, state, n), ld_row_f<float, 4, VEC>(lam, p.lam + c, n);
        ld_row_f<T, 4, VEC>(x, (const T *)p.x + req * p.x_st + c, n), ld_row_f<T, 4, VEC>(r, (const T *)p.r + req * p.r_st + c, n);
        ld_row_f<T, 4, VEC>(i, (const T *)p.i + req * p.i_st + c, n);
        if (p.z) ld_row_f<T, 4, VEC>(z, (const T *)p.z + req * p.z_st + c, n);
    }
    float o[4];
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
        const float2 sp = softplus2(make_float2(lam[k], lam[k + 1]));
        const LruGate g(pack2(r[k], r[k + 1]), pack2(i[k], i[k + 1]), pack2(p.c * sp.x, p.c * sp.y));
        const float2 v = unpack2(fma2(g.a, pack2(h[k], h[k + 1]), mul2(mul2(g.beta(), g.gi), pack2(x[k], x[k + 1]))));
        h[k] = o[k] = v.x, h[k + 1] = o[k + 1] = v.y;
        if (p.z) {
            const float2 s = sigmoid2(make_float2(z[k], z[k + 1]));
            o[k] *= z[k] * s.x, o[k + 1] *= z[k + 1] * s.y;
        }
        if (!live) o[k] = o[k + 1] = 0.f;
    }
    if (live) st_row_f<float, 4, VEC>(state, h, n);
    st_row_f<T, 4, VEC>((T *)p.out + req * p.o_st + c, o, n);
}

}  // namespace

// CTAs of a cluster: a line's tiles side by side, up to eight, while the
// channels alone do not fill the GPU and the line is long enough.
int lru_ranks(int lines, int T, int C) {
    const int64_t ctas = (int64_t)lines * ((C + kLruCh - 1) / kLruCh);
    const int tiles = (T + kLruTile - 1) / kLruTile;
    int k = 1;
    while (k < kRanks && k < tiles && ctas * k < 8 * 152) k *= 2;
    return k;
}

cudaError_t lru_launch(const void *kernel, int lines, int C, int ranks, int smem, const LruParams &p, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((C + kLruCh - 1) / kLruCh * ranks, lines);
    cfg.blockDim = dim3(32 * kLruWarps);
    cfg.dynamicSmemBytes = smem, cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ranks, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
    cfg.attrs = &at, cfg.numAttrs = 1;
    void *args[] = {const_cast<LruParams *>(&p)};
    e = cudaLaunchKernelExC(&cfg, kernel, args);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_lru(const LruParams &p, cudaStream_t st) {
    using bf = __nv_bfloat16;
    const void *k = p.bf16 ? (p.vec ? (const void *)lru_kernel<bf, true> : (const void *)lru_kernel<bf, false>)
                           : (p.vec ? (const void *)lru_kernel<float, true> : (const void *)lru_kernel<float, false>);
    const int smem = p.vec ? 4 * kLruTile * kLruCh * (p.bf16 ? 2 : 4) : 0;
    return lru_launch(k, p.B, p.C, p.ranks, smem, p, st);
}

cudaError_t launch_lru_step(const LruStepParams &p, cudaStream_t st) {
    const dim3 grid((p.C + 511) / 512, p.n);
    using bf = __nv_bfloat16;
    if (p.bf16) {
        if (p.vec) lru_step_kernel<bf, true><<<grid, 128, 0, st>>>(p);
        else lru_step_kernel<bf, false><<<grid, 128, 0, st>>>(p);
    } else {
        if (p.vec) lru_step_kernel<float, true><<<grid, 128, 0, st>>>(p);
        else lru_step_kernel<float, false><<<grid, 128, 0, st>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace gdn

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

template <typename T, int HOW, bool PACKED, bool Z>
__global__ void __launch_bounds__(32 * kLruWarps, 3) lru_kernel(const LruParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ LruRun runs[2][kLruWarps][32];
    __shared__ LruRanks ranks;
    constexpr int kRow = kLruCh, kTensor = kLruLen * kRow;  // elements of a warp's rows of one tensor
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int K = p.ranks, rank = blockIdx.x % K, line = blockIdx.y;
    const int c0 = (blockIdx.x / K) * kLruCh, c = c0 + 2 * lane, nc = p.C - c;  // nc: channels of the pair that exist
    const f32x2 one = pack2(1.f, 1.f), zero = pack2(0.f, 0.f);
    if (PACKED) {
        if (p.err && blockIdx.x == 0) ssm_check_cu(p.cu, p.n_seq, p.T, p.err);
        if (p.h_final && rank == 0) {  // sequences without tokens keep their states
            for (int s = warp; s < p.n_seq; s += kLruWarps)
                if (p.cu[s + 1] <= p.cu[s]) lru_st_state(p.h_final, s, p.C, c, nc, lru_ld_state(p.h0, s, p.C, c, nc));
        }
    }
    const int steps = (p.T + K * kLruTile - 1) / (K * kLruTile);
    const LruRows<T, HOW> x((const T *)p.x + line * p.x_sb + c0, p.x_st), r((const T *)p.r + line * p.r_sb + c0, p.r_st),
        in((const T *)p.i + line * p.i_sb + c0, p.i_st), z((const T *)p.z + (Z ? line * p.z_sb + c0 : 0), p.z_st);
    T *out = (T *)p.out + (p.out ? line * p.o_sb + c : 0);
    T *const stage = (T *)smem + warp * (Z ? 4 : 3) * kTensor, *const staged = stage + 2 * lane;
    auto first = [&](int n) { return (n * K + rank) * kLruTile + warp * kLruLen; };  // token of step n
    // two groups of copies a step: x, r and i are free for the next step's once
    // a and b are formed, z once the outputs are
    auto fetch = [&](int n) {
        const int t = first(n), rows = p.T - t;
        if (n < steps && rows > 0) {
            x.copy(stage, t, rows, p.C - c0), r.copy(stage + kTensor, t, rows, p.C - c0);
            in.copy(stage + 2 * kTensor, t, rows, p.C - c0);
        }
        cp_async_commit();
    };
    auto fetch_z = [&](int n) {
        const int t = first(n), rows = p.T - t;
        if (Z && n < steps && rows > 0) z.copy(stage + 3 * kTensor, t, rows, p.C - c0);
        cp_async_commit();
    };
    auto get = [&](int k, int j) { return lru_pair(staged + k * kTensor + j * kRow); };  // a pair of x, r, i or z
    fetch(0), fetch_z(0);
    const LruDecay decay(p.lam + c, p.c, nc);
    f32x2 carry = PACKED ? zero : lru_ld_state(p.h0, line, p.C, c, nc);  // the state before the cluster's tiles
    bool lost = false;
    if (K > 1) {
        ranks.init(K);
        cluster_sync();
    }
    for (int n = 0; n < steps; ++n) {
        const int t0 = first(n), len = min(max(p.T - t0, 0), kLruLen), flip = n & 1;
        LruMarks m{0u, 0u};
        if (PACKED) m = lru_marks(p.cu, p.n_seq, p.T, t0);
        cp_async_wait<1>();
        __syncwarp();
        f32x2 a[kLruLen], b[kLruLen];
        LruRun run{one, zero};
        auto gates = [&](auto form) {  // whole: eight tokens, none of which begins a sequence
            constexpr bool whole = decltype(form)::value;
#pragma unroll
            for (int j = 0; j < kLruLen; ++j) {
                if (!whole && j >= len) {
                    a[j] = one, b[j] = zero;
                    continue;
                }
                const LruGate g(get(1, j), get(2, j), decay);
                a[j] = g.a, b[j] = mul2(mul2(sqrt_2(g.q), g.gi), get(0, j));
                if (PACKED && !whole && m.cut >> j & 1) {
                    if (p.h0) b[j] = fma2(g.a, lru_ld_state(p.h0, lru_seq(p.cu, p.n_seq, p.T, t0 + j), p.C, c, nc), b[j]);
                    run.A = pack2(-0.f, -0.f), run.H = b[j];
                } else {
                    run.A = mul2(run.A, a[j]), run.H = fma2(a[j], run.H, b[j]);
                }
            }
        };
        if (len == kLruLen && !m.cut) gates(std::true_type());
        else gates(std::false_type());
        __syncwarp();  // every lane has read what the next copies overwrite
        fetch(n + 1);
        runs[flip][warp][lane] = run;
        __syncthreads();
        f32x2 h = carry;
        if (K > 1) {
            if (warp == 0) {
                LruRun all = run;
#pragma unroll
                for (int w = 1; w < kLruWarps; ++w) {
                    const LruRun v = runs[flip][w][lane];
                    all.H = lru_apply2<PACKED>(v.A, v.H, all.H), all.A = lru_join<PACKED>(all.A, v.A);
                }
                ranks.send(n, K, rank, all);
            }
            if (!lost) lost = !ranks.wait(n);
#pragma unroll 8
            for (int k = 0; k < (K > 8 ? 16 : 8); ++k) {
                const LruRun v = ranks.runs[flip][k][lane];
                if (k == rank) h = carry;
                carry = lru_apply2<PACKED>(v.A, v.H, carry);
            }
#pragma unroll
            for (int w = 0; w < kLruWarps - 1; ++w) {
                if (w >= warp) break;
                const LruRun v = runs[flip][w][lane];
                h = lru_apply2<PACKED>(v.A, v.H, h);
            }
        } else {
#pragma unroll
            for (int w = 0; w < kLruWarps; ++w) {
                const LruRun v = runs[flip][w][lane];
                if (w == warp) h = carry;
                carry = lru_apply2<PACKED>(v.A, v.H, carry);
            }
        }
        if (lost) h = carry = pack2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
        if (p.ck && warp == 0 && t0 < p.T)
            lru_st_state(p.ck, (int64_t)line * ((p.T + kLruTile - 1) / kLruTile) + t0 / kLruTile, p.C, c, nc, h);
        cp_async_wait<1>();
        __syncwarp();
        T *o = out + (int64_t)t0 * p.o_st;
        auto walk = [&](auto form) {
            constexpr bool whole = decltype(form)::value;
#pragma unroll
            for (int j = 0; j < kLruLen; ++j, o += p.o_st) {
                if (!whole && j >= len) break;
                h = PACKED && !whole && m.cut >> j & 1 ? b[j] : fma2(a[j], h, b[j]);
                f32x2 y = h;
                if (Z) {
                    const f32x2 v = get(3, j);
                    y = mul2(h, mul2(v, sigmoid_2(v)));
                }
                if (nc > 0) lru_put<T, HOW>(o, y, nc);
                if (PACKED && !whole && p.h_final && m.fin >> j & 1)
                    lru_st_state(p.h_final, lru_seq(p.cu, p.n_seq, p.T, t0 + j), p.C, c, nc, h);
            }
        };
        if (p.out) {
            if (len == kLruLen && !(m.cut | m.fin)) walk(std::true_type());
            else walk(std::false_type());
        }
        __syncwarp();
        fetch_z(n + 1);
    }
    if (!PACKED && p.h_final && rank == 0 && warp == 0) lru_st_state(p.h_final, line, p.C, c, nc, carry);
    if (K > 1) cluster_sync();  // no CTA leaves before all have what it sent
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
        const LruGate g(pack2(r[k], r[k + 1]), pack2(i[k], i[k + 1]), LruDecay(lam + k, p.c, 2));
        const float2 v = unpack2(fma2(g.a, pack2(h[k], h[k + 1]), mul2(mul2(sqrt_2(g.q), g.gi), pack2(x[k], x[k + 1]))));
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

// CTAs of a cluster: a line's tiles side by side, up to eight, while all lines
// have fewer than four CTAs a SM and are long enough; sixteen only where that
// leaves two a SM (clusters of sixteen fit an SM group badly). Forward, bf16,
// with z: 4 x 4096 tokens of 4096 channels 180, 191, 171, 187, 246 us for 1, 2,
// 4, 8, 16; 32768 tokens of 1024 channels 885, 543, 277, 200, 152; fp32, 5003
// tokens of 1792 channels 148, 93, 56, 42, 50.
int lru_ranks(int lines, int T, int C) {
    const int64_t ctas = (int64_t)lines * ((C + kLruCh - 1) / kLruCh);
    const int tiles = (T + kLruTile - 1) / kLruTile;
    int k = 1;
    while (k < 8 && k < tiles && ctas * k < 608) k *= 2;
    return k == 8 && k < tiles && ctas * 16 <= 304 ? 16 : k;
}

cudaError_t lru_launch(const void *kernel, int lines, int C, int ranks, int smem, const LruParams &p, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (ranks > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
    return lru_by_form(p, p.z != nullptr, [&](auto type, auto how, auto packed, auto z) {
        using T = decltype(type);
        const int smem = (z() ? 4 : 3) * kLruTile * kLruCh * (int)sizeof(T);
        return lru_launch((const void *)lru_kernel<T, how(), packed(), z()>, p.B, p.C, p.ranks, smem, p, st);
    });
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

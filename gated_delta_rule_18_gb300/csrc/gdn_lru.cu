// gdn_lru.cu -- the gated linear recurrence, per channel and sequence:
//   u = c softplus(lam) sigmoid(r),  a = exp(-u),
//   h <- a h + sqrt(1 - a^2) sigmoid(i) x,  out = h silu(z)  (h without z),
// for whole sequences (dense or packed) and for single tokens with the states
// in a pool. h is fp32 throughout.
//
// HBM would be its bound (10 bytes a token and channel with z in bf16). A CTA
// has 64 channels and 64 or 128 consecutive tokens, sixteen to a warp; a cluster
// of CTAs takes consecutive tiles of the same channels at once and walks the
// line so. A warp forms a and the input of each token in registers and what its
// run does to the state before it (A v + H); the runs are joined over the CTA's
// warps through shared memory, over the cluster by asynchronous stores to the
// other CTAs', in one order, and each warp then walks its tokens from its
// entering state. Inputs are read once: the next tile's x, r, i by tensor
// copies as soon as the gates are formed, z after the walk. Results repeat bit
// for bit.
//
// Measured (calls among others, copy rate 6.78 TB/s): 4 x 4096 tokens of 4096
// channels with z in bf16 125 us (79 % of the copy rate) where all of a tile's
// channels decay slowly (c softplus(lam) < 1/8) and 133 (74 %) where one does not, in
// fp32 194 and 198 (all of it); 8 x 1024 of 4096 channels, bf16, 68 and 73: 75
// instructions a warp and channel pair at 0.56 a cycle from 14 warps a SM, 14 of
// them for the exponential unit (16 where a channel decays fast), whose queue is
// a large stall. 32768 tokens of 1024 channels 106 and 113 (47 %): with 16 tiles of
// channels only, 10 warps a SM, and an exchange over the cluster every 1536
// tokens.
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "gdn_lru.cuh"

namespace gdn {
namespace {

// A warp's tokens. With eight what a warp does once a tile (waits, joins,
// addresses) was a fifth of its instructions: 165 us for 138 (4 x 4096 tokens of
// 4096 channels, bf16).
constexpr int L = 16;

// shared memory: a stage of x, r, i and one of z by warp, the warps' runs, the ranks'
template <typename T, bool Z, int W>
struct LruSmem {
    static constexpr int kRows = L * kLruCh, kWarp = (Z ? 4 : 3) * kRows;
    static constexpr int kRuns = W * kWarp * (int)sizeof(T), kRanks = kRuns + 2 * W * 32 * (int)sizeof(LruRun);
    static constexpr int bytes(int K) { return kRanks + 2 * LruRanks::places_of(K) * 32 * (int)sizeof(LruRun); }
};

template <typename T, int HOW, bool PACKED, bool Z, int W>
__global__ void __launch_bounds__(32 * W, 16 / W) lru_kernel(const LruParams p, const __grid_constant__ LruMaps maps) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ unsigned long long bars[W][2], rank_bars[2];
    using M = LruSmem<T, Z, W>;
    constexpr int kTile = W * L;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int K = p.ranks, rank = blockIdx.x % K, line = blockIdx.y;
    const int c0 = (blockIdx.x / K) * kLruCh, c = c0 + 2 * lane, nc = p.C - c;  // nc: channels of the pair that exist
    const f32x2 one = pack2(1.f, 1.f), zero = pack2(0.f, 0.f);
    lru_begin<PACKED>(p);
    if (PACKED) {
        if (p.h_final && rank == 0) {  // sequences without tokens keep their states
            for (int s = warp; s < p.n_seq; s += W)
                if (p.cu[s + 1] <= p.cu[s]) lru_st_state(p.h_final, s, p.C, c, nc, lru_ld_state(p.h0, s, p.C, c, nc));
        }
    }
    const int steps = (p.T + K * kTile - 1) / (K * kTile);
    const LruFetch<T, HOW, 3, L> xri({(const T *)p.x + line * p.x_sb + c0, (const T *)p.r + line * p.r_sb + c0,
                                   (const T *)p.i + line * p.i_sb + c0}, {p.x_st, p.r_st, p.i_st}, maps.m, c0, line, p.C);
    const LruFetch<T, HOW, 1, L> zs({(const T *)p.z + (Z ? line * p.z_sb + c0 : 0)}, {p.z_st}, maps.m + 3, c0, line, p.C);
    T *out = (T *)p.out + (p.out ? line * p.o_sb + c : 0);
    T *const stage = (T *)smem + warp * M::kWarp, *const z_stage = stage + 3 * M::kRows;
    auto runs = reinterpret_cast<LruRun(*)[W][32]>(smem + M::kRuns);
    const LruRanks ranks{reinterpret_cast<LruRun *>(smem + M::kRanks), rank_bars, K, LruRanks::places_of(K)};
    if (lane == 0) lru_init_bars(bars[warp], 2);
    __syncwarp();
    auto first = [&](int n) { return (n * K + rank) * kTile + warp * L; };  // token of step n
    auto fetch = [&](int n) {
        if (n < steps) xri.copy(stage, first(n), p.T - first(n), smem_u32(&bars[warp][0]));
        else cp_async_commit();
    };
    auto fetch_z = [&](int n) {
        if (Z && n < steps) zs.copy(z_stage, first(n), p.T - first(n), smem_u32(&bars[warp][1]));
        else cp_async_commit();
    };
    const bool stalled = lru_stalled(p);
    if (!stalled) fetch(0);
    fetch_z(0);
    const LruDecay decay(p.lam + c, p.c, nc);
    const bool near = decay.near(nc);
    f32x2 carry = PACKED ? zero : lru_ld_state(p.h0, line, p.C, c, nc);  // the state before the cluster's tiles
    int lost = 0, n = 0;
    const f32x2 nan = pack2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
    auto lose = [&](int n) {  // this warp's tokens of step n
        const int t0 = first(n), len = min(max(p.T - t0, 0), L);
        LruMarks m{0u, 0u};
        if (PACKED) m = lru_marks<L>(p.cu, p.n_seq, p.T, t0);
        if (p.ck && warp * L % kLruTile == 0 && t0 < p.T)
            lru_st_state(p.ck, (int64_t)line * ((p.T + kLruTile - 1) / kLruTile) + t0 / kLruTile, p.C, c, nc, nan);
#pragma unroll 1
        for (int j = 0; j < len; ++j) {
            if (p.out && nc > 0) lru_put<T, HOW>(out + (int64_t)(t0 + j) * p.o_st, nan, nc);
            if (PACKED && p.h_final && m.fin >> j & 1)
                lru_st_state(p.h_final, lru_seq(p.cu, p.n_seq, p.T, t0 + j), p.C, c, nc, nan);
        }
    };
    if (K > 1) {
        ranks.init();
        cluster_sync();
    }
#pragma unroll 1
    for (; n < steps; ++n) {
        const int t0 = first(n), len = min(max(p.T - t0, 0), L), flip = n & 1;
        LruMarks m{0u, 0u};
        if (PACKED) m = lru_marks<L>(p.cu, p.n_seq, p.T, t0);
        if (!xri.template wait<1>(smem_u32(&bars[warp][0]), n & 1, p.wait_us)) lost |= kLostRows;
        if (HOW != kLruWide && stalled) lost |= kLostRuns;
        auto get = [&](int k, int j) { return lru_pair(stage + 2 * lane + k * M::kRows + j * kLruCh); };  // a pair of x, r or i
        f32x2 a[L], b[L];
        LruRun run{one, zero};
        auto gates = [&](auto form, auto close) {  // whole: all tokens are there, none begins a sequence
            constexpr bool whole = decltype(form)::value;
#pragma unroll
            for (int j = 0; j < L; ++j) {
                if (!whole && j >= len) {
                    a[j] = one, b[j] = zero;
                    continue;
                }
                const LruGate<decltype(close)::value> g(get(1, j), get(2, j), decay);
                a[j] = g.a, b[j] = mul2(mul2(sqrt_2(g.q), g.gi), get(0, j));
                if (PACKED && !whole && m.cut >> j & 1) {
                    if (p.h0) b[j] = fma2(g.a, lru_ld_state(p.h0, lru_seq(p.cu, p.n_seq, p.T, t0 + j), p.C, c, nc), b[j]);
                    run.A = pack2(-0.f, -0.f), run.H = b[j];
                } else {
                    run.A = mul2(run.A, a[j]), run.H = fma2(a[j], run.H, b[j]);
                }
            }
        };
        if (HOW == kLruWide && near && len == L && !m.cut) gates(std::true_type(), std::bool_constant<HOW == kLruWide>());
        else if (len == L && !m.cut) gates(std::true_type(), std::false_type());
        else gates(std::false_type(), std::false_type());
        runs[flip][warp][lane] = run;
        __syncwarp();  // every lane has read what the next copies overwrite
        if (!(lost & kLostRows)) fetch(n + 1);
        if (__syncthreads_or(lost)) break;
        f32x2 h = carry;
        if (K > 1) {
            if (warp == 0) {
                LruRun all = run;
#pragma unroll
                for (int w = 1; w < W; ++w) {
                    const LruRun v = runs[flip][w][lane];
                    all.H = lru_apply2<PACKED>(v.A, v.H, all.H), all.A = lru_join<PACKED>(all.A, v.A);
                }
                ranks.send(n, rank, all);
            }
            if (!ranks.wait(n, p.wait_us)) lost |= kLostRuns;
#pragma unroll 8
            for (int k = 0; k < ranks.places; ++k) {
                const LruRun v = ranks.at(n, k);
                if (k == rank) h = carry;
                carry = lru_apply2<PACKED>(v.A, v.H, carry);
            }
#pragma unroll
            for (int w = 0; w < W - 1; ++w) {
                if (w >= warp) break;
                const LruRun v = runs[flip][w][lane];
                h = lru_apply2<PACKED>(v.A, v.H, h);
            }
        } else {
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const LruRun v = runs[flip][w][lane];
                if (w == warp) h = carry;
                carry = lru_apply2<PACKED>(v.A, v.H, carry);
            }
        }
        if (p.ck && warp * L % kLruTile == 0 && t0 < p.T)
            lru_st_state(p.ck, (int64_t)line * ((p.T + kLruTile - 1) / kLruTile) + t0 / kLruTile, p.C, c, nc, h);
        if (Z && !zs.template wait<1>(smem_u32(&bars[warp][1]), n & 1, p.wait_us)) lost |= kLostZ;
        T *o = out + (int64_t)t0 * p.o_st;
        auto walk = [&](auto form) {
            constexpr bool whole = decltype(form)::value;
#pragma unroll
            for (int j = 0; j < L; ++j, o += p.o_st) {
                if (!whole && j >= len) break;
                h = PACKED && !whole && m.cut >> j & 1 ? b[j] : fma2(a[j], h, b[j]);
                f32x2 y = h;
                if (Z) {
                    const f32x2 v = lru_pair(z_stage + 2 * lane + j * kLruCh);
                    y = mul2(h, mul2(v, sigmoid_2(v)));
                }
                if (nc > 0) lru_put<T, HOW>(o, y, nc);
                if (PACKED && !whole && p.h_final && m.fin >> j & 1)
                    lru_st_state(p.h_final, lru_seq(p.cu, p.n_seq, p.T, t0 + j), p.C, c, nc, h);
            }
        };
        if (p.out) {
            if (len == L && !(m.cut | m.fin)) walk(std::true_type());
            else walk(std::false_type());
        }
        __syncwarp();  // every lane is through with the stages
        if (!(lost & kLostZ)) fetch_z(n + 1);
    }
    if (n < steps || __any_sync(0xffffffffu, lost)) {
        if (lost && p.err) atomicOr(p.err, kDevErrTimeout);
        carry = nan;
        const int from = lost & (kLostRuns | kLostZ) ? max(n - 1, 0) : n;
        if (HOW != kLruWide) {
            cp_async_wait<0>();
        } else if (lane == 0) {  // (of the last copies that were asked for)
            const int left = n < steps ? n : steps - 1, rows = n < steps && !(lost & kLostRows) ? min(n + 1, steps - 1) : left;
            lru_wait(smem_u32(&bars[warp][0]), rows & 1, p.wait_us);
            if (Z) lru_wait(smem_u32(&bars[warp][1]), (n < steps && lost & kLostZ ? n - 1 : left) & 1, p.wait_us);
        }
#pragma unroll 1
        for (n = from; n < steps; ++n) lose(n);
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
        const LruGate<false> g(pack2(r[k], r[k + 1]), pack2(i[k], i[k + 1]), LruDecay(lam + k, p.c, 2));
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

// Whether `tiles` CTAs fill what waves they take of `slots` at a time to so many percent.
static bool lru_fills(int64_t tiles, int slots, int percent) {
    return tiles * 100 >= (tiles + slots - 1) / slots * slots * percent;
}
// CTAs of a cluster, which take a line's tiles side by side, and warps of a CTA.
// In bf16 a cluster pays for its exchange at every step, and a line of one CTA
// for the SMs that stand idle at the end. So a line's channel tile goes to one
// CTA of eight warps where those fill the SMs to three quarters and lines are
// short (4096 channels, one CTA and four: 24 x 512 tokens 93 us and 125, 16 x 1024
// 116 and 136, 8 x 1700 111 and 113), and for longer lines only where they fill
// them to nine tenths (9 x 4096: 251 and 268) or are many (16 x 8192: 854 and 887);
// else to four (8 x 2048: 128.3 and 127.7, 12 x 4096: 365 and 348, 4 x 8192: 251
// and 239). Rows by words are the same (four warps; 4098 channels, 8 x 1024: 107 and
// 109, 8 x 4096: 407 and 390, 16 x 4000: 689 and 735), and so are channels that
// decay fast. In fp32, which HBM bounds, one CTA of four warps is best (8 x 1024
// tokens of 2048 channels: 62, with eight warps 64, four CTAs 72). With few tiles,
// eight warps and as many CTAs as make 256, up to twelve a line (32768 tokens of
// 1024 channels with 8, 12, 16: 148, 109, 130 us; sixteen warps with 6, 8, 12: 113,
// 163, 124).
LruShape lru_shape(int lines, int T, int C, bool bf16, bool wide) {
    const int64_t tiles = (int64_t)lines * ((C + kLruCh - 1) / kLruCh);
    LruShape s{1, 4};
    if (tiles >= 192) {
        const int slots = wide ? 304 : 608;
        const bool whole = lru_fills(tiles, slots, T < 2048 || tiles >= 1024 ? 75 : 90);
        s.ranks = !bf16 || whole ? 1 : 4, s.warps = bf16 && whole && wide ? 8 : 4;
    } else {
        const int most = wide ? 12 : 16, all = wide ? 256 : 512;
        s.warps = wide && T > 64 ? 8 : 4;
        s.ranks = (int)(tiles * most <= all ? most : all / tiles);
        if (wide && s.ranks > 8 && s.ranks < most) s.ranks = 8;  // (larger clusters fit an SM group badly)
    }
    const int steps = (T + s.warps * L - 1) / (s.warps * L);
    if (s.ranks > steps) s.ranks = steps > 0 ? steps : 1;
    return s;
}
// Of the gradient: eight warps of eight tokens, by the same rules in both types
// (16 x 1024 tokens of 4096 channels, bf16, one CTA a line 294 us, four 339;
// 8 x 2048 of 2560 channels 262 and 217, fp32 349 and 265).
int lru_bwd_ranks(int lines, int T, int C) {
    const int64_t tiles = (int64_t)lines * ((C + kLruCh - 1) / kLruCh);
    int k = tiles >= 192 ? lru_fills(tiles, 304, 75) ? 1 : 4 : (int)(tiles * 12 <= 256 ? 12 : 256 / tiles);
    const int steps = (T + kLruTile - 1) / kLruTile;
    return k > steps ? steps > 0 ? steps : 1 : k;
}

bool lru_maps(const LruParams &p, bool gradient, int len, LruMaps *m) {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    if (!fn || p.T < 1) return false;
    const int e = p.bf16 ? 2 : 4;
    int n = 0;
    auto add = [&](const void *at, int64_t sb, int64_t st) {
        if (!at) return true;
        cuuint64_t dims[3] = {(cuuint64_t)p.C, (cuuint64_t)p.T, (cuuint64_t)p.B};
        // (the stride of a dimension of one is free)
        cuuint64_t strides[2] = {(cuuint64_t)((p.T > 1 ? st : p.C) * e), (cuuint64_t)((p.B > 1 ? sb : p.C) * e)};
        for (const cuuint64_t s : strides)
            if (s == 0 || s % 16 != 0 || s >= 1ull << 40) return false;
        cuuint32_t box[3] = {kLruCh, (cuuint32_t)len, 1}, es[3] = {1, 1, 1};
        return fn(&m->m[n++], p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(at),
                  dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    return add(p.x, p.x_sb, p.x_st) && add(p.r, p.r_sb, p.r_st) && add(p.i, p.i_sb, p.i_st) &&
           (!gradient || add(p.dout, p.do_sb, p.do_st)) && add(p.z, p.z_sb, p.z_st);
}

static std::atomic<int> g_most{0};
void set_lru_cluster(int most) { g_most.store(most > 0 ? most : 0); }

cudaError_t lru_launch(const void *kernel, int warps, int (*smem)(int ranks), LruParams &p, const LruMaps &m, cudaStream_t st) {
    // (the limit is the kernel's, not the call's: a smaller call's own size would lower it under another thread's launch)
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem(kLruRanks));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
    cfg.blockDim = dim3(32 * warps), cfg.stream = st, cfg.attrs = &at, cfg.numAttrs = 1;
    const auto of = [&](int ranks) {
        cfg.gridDim = dim3((p.C + kLruCh - 1) / kLruCh * ranks, p.B), cfg.dynamicSmemBytes = smem(ranks), at.val.clusterDim.x = ranks;
    };
    const int most = g_most.load(std::memory_order_relaxed);
    if (most && p.ranks > most) p.ranks = most;
    of(p.ranks);
    if (p.ranks > 8) {  // eight are portable; more need a group of SMs that holds them, which not every GPU (or part of one) has
        int n = 0;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess) cudaGetLastError();  // (not the call's)
        if (e != cudaSuccess || n < 1) p.ranks = 8, of(8);
    }
    void *args[] = {&p, const_cast<LruMaps *>(&m)};
    e = cudaLaunchKernelExC(&cfg, kernel, args);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_lru(LruParams &p, cudaStream_t st) {
    LruMaps m{};
    const int how = p.how == kLruWide && !lru_maps(p, false, L, &m) ? (int)kLruWords : p.how;
    return lru_by_form(p, how, p.z != nullptr, [&](auto type, auto how, auto packed, auto z) {
        using T = decltype(type);
        auto run = [&](auto w) {
            return lru_launch((const void *)lru_kernel<T, how(), packed(), z(), w()>, w(), LruSmem<T, z(), w()>::bytes, p, m, st);
        };
        if constexpr (how() == kLruWide) {
            if (p.warps == 8) return run(std::integral_constant<int, 8>());
        }
        return run(std::integral_constant<int, 4>());
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

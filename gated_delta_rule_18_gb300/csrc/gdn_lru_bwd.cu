// gdn_lru_bwd.cu -- the gradient of the gated linear recurrence. With s =
// silu(z) (1 without z) and q = 1 - a^2, backwards along each sequence:
//   g_t = dout_t s_t + a_{t+1} g_{t+1}          (+ dh_final at its end)
//   dx = g sqrt(q) sigmoid(i),   di = g b (1 - sigmoid(i)),  b = sqrt(q) sigmoid(i) x
//   w  = u g (a^2 b / q - a h_{t-1})            (u times the gradient of u)
//   dr = w (1 - sigmoid(r)),     dlam = sum w . sigmoid(lam) / softplus(lam)
//   dz = dout h silu'(z),        dh0 = a_0 g_0.
// b / q = sigmoid(i) x / sqrt(q) grows without bound as u -> 0, and u times it
// goes to 0 with sqrt(u): both are formed with 1 / sqrt(q) and meet no 0 / 0.
//
// The clusters and joins of the forward, from the line's end, with eight warps
// of eight tokens (sixteen: 396 us where these took 321). The states inside a tile are formed
// again from the one saved for its 64 tokens, so the line is read once here
// too. The walk back takes the gates and roots as the sweep before it left them:
// in shared memory, and in the places of r and i, which only the sweep reads.
//
// Measured: 4 x 4096 tokens of 4096 channels, bf16, 314 us (57 % of the copy
// rate, where the bytes take 178; 317 where channels decay fast), fp32 351 (all of
// it); out of wider rows 320 and 381. 174 instructions a warp and channel pair at
// 0.53 a cycle, 14 warps a SM (128 registers, 86 KB a CTA). Next rows in two halves,
// the first asked for amid the walk: 332 for 321; sigmoid(z) kept as well: 327.
#include "gdn_lru.cuh"

namespace gdn {
namespace {

// L tokens a warp, W warps.
// shared memory: the stage of the tensors by warp, the warps' runs both ways, the ranks'
template <typename T, bool Z, int L, int W>
struct LruBwdSmem {
    static constexpr int kTensors = Z ? 5 : 4, kRows = L * kLruCh, kWarp = kTensors * kRows;
    static constexpr bool kInPlace = sizeof(T) == 4;  // the gates take the places of r and i
    static constexpr int kGates = W * kWarp * (int)sizeof(T);
    static constexpr int kRuns = kGates + (kInPlace ? 0 : W * L * 32 * (int)sizeof(uint4)), kBacks = kRuns + 2 * W * 32 * (int)sizeof(LruRun);
    static constexpr int kRanks = kBacks + 2 * W * 32 * 8;
    static constexpr int bytes(int K) { return kRanks + 2 * LruRanks::places_of(K) * 32 * (int)sizeof(LruRun); }
};

template <typename T, int HOW, bool PACKED, bool Z, int L, int W>
__global__ void __launch_bounds__(32 * W, 16 / W) lru_bwd_kernel(const LruParams p, const __grid_constant__ LruMaps maps) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ unsigned long long bars[W], rank_bars[2];
    using M = LruBwdSmem<T, Z, L, W>;
    constexpr int N = M::kTensors, kTile = W * L;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int K = p.ranks, rank = blockIdx.x % K, line = blockIdx.y;
    const int c0 = (blockIdx.x / K) * kLruCh, c = c0 + 2 * lane, nc = p.C - c;
    auto runs = reinterpret_cast<LruRun(*)[W][32]>(smem + M::kRuns);   // A, H of a warp's tokens
    auto backs = reinterpret_cast<f32x2(*)[W][32]>(smem + M::kBacks);  // what they add to the gradient before them
    const LruRanks ranks{reinterpret_cast<LruRun *>(smem + M::kRanks), rank_bars, K, LruRanks::places_of(K)};
    const f32x2 one = pack2(1.f, 1.f), zero = pack2(0.f, 0.f), minus = pack2(-1.f, -1.f);
    lru_begin<PACKED>(p);
    if (PACKED) {
        if (p.dh0 && rank == 0) {  // of sequences without tokens
            for (int s = warp; s < p.n_seq; s += W)
                if (p.cu[s + 1] <= p.cu[s]) lru_st_state(p.dh0, s, p.C, c, nc, lru_ld_state(p.dh_final, s, p.C, c, nc));
        }
    }
    const int steps = (p.T + K * kTile - 1) / (K * kTile), tiles = (p.T + kLruTile - 1) / kLruTile;
    const T *bases[5] = {(const T *)p.x + line * p.x_sb + c0, (const T *)p.r + line * p.r_sb + c0, (const T *)p.i + line * p.i_sb + c0,
                         (const T *)p.dout + line * p.do_sb + c0, (const T *)p.z + (Z ? line * p.z_sb + c0 : 0)};
    const T *base[N];
    int64_t stride[N];
    const int64_t strides[5] = {p.x_st, p.r_st, p.i_st, p.do_st, p.z_st};
#pragma unroll
    for (int k = 0; k < N; ++k) base[k] = bases[k], stride[k] = strides[k];
    const LruFetch<T, HOW, N, L> rows(base, stride, maps.m, c0, line, p.C);
    T *const stage = (T *)smem + warp * M::kWarp;
    uint4 *const gates_at = reinterpret_cast<uint4 *>(smem + M::kGates) + warp * L * 32 + lane;
    if (lane == 0) lru_init_bars(&bars[warp], 1);
    __syncwarp();
    auto first = [&](int n) { return ((steps - 1 - n) * K + rank) * kTile + warp * L; };
    auto fetch = [&](int n) {
        if (n < steps) rows.copy(stage, first(n), p.T - first(n), smem_u32(&bars[warp]));
        else cp_async_commit();
    };
    const bool stalled = lru_stalled(p);
    if (!stalled) fetch(0);
    const LruDecay decay(p.lam + c, p.c, nc);
    const bool near = decay.near(nc);
    // a g of the token behind the cluster's tiles
    f32x2 carry = PACKED ? zero : lru_ld_state(p.dh_final, line, p.C, c, nc), dlam = zero;
    int lost = 0, n = 0;
    const f32x2 nan = pack2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
    auto lose = [&](int n) {  // this warp's tokens of step n
        const int t0 = first(n), len = min(max(p.T - t0, 0), L);
        LruMarks m{0u, 0u};
        if (PACKED) m = lru_marks<L>(p.cu, p.n_seq, p.T, t0);
#pragma unroll 1
        for (int j = 0; j < len; ++j) {
            const int64_t at = ((int64_t)line * p.T + t0 + j) * p.C + c;
            if (nc > 0) {
                lru_put<T, HOW>((T *)p.dx + at, nan, nc), lru_put<T, HOW>((T *)p.dr + at, nan, nc);
                lru_put<T, HOW>((T *)p.di + at, nan, nc);
                if (Z) lru_put<T, HOW>((T *)p.dz + at, nan, nc);
            }
            if (PACKED && p.dh0 && m.cut >> j & 1) lru_st_state(p.dh0, lru_seq(p.cu, p.n_seq, p.T, t0 + j), p.C, c, nc, nan);
        }
    };
    if (K > 1) {
        ranks.init();
        cluster_sync();
    }
#pragma unroll 1
    for (; n < steps; ++n) {
        const int t0 = first(n), len = min(max(p.T - t0, 0), L), flip = n & 1, tile = t0 / kLruTile;
        LruMarks m{0u, 0u};
        if (PACKED) m = lru_marks<L>(p.cu, p.n_seq, p.T, t0);
        f32x2 h = tile < tiles ? lru_ld_state(p.ck, (int64_t)line * tiles + tile, p.C, c, nc) : zero;
        if (!rows.template wait<0>(smem_u32(&bars[warp]), n & 1, p.wait_us)) lost |= kLostRows;
        if (HOW != kLruWide && stalled) lost |= kLostRuns;
        T *const staged = stage + 2 * lane;
        auto get = [&](int k, int j) { return lru_pair(staged + k * M::kRows + j * kLruCh); };  // of x, r, i, dout, z
        const bool all_inside = len == L && !(m.cut | m.fin);
        f32x2 a[L], b[L], back = zero;
        LruRun run{one, zero};
        auto gates = [&](auto form, auto close) {  // whole: all tokens are there, within a sequence
            constexpr bool whole = decltype(form)::value;
            bool open = true;  // no sequence has begun in the run
#pragma unroll
            for (int j = 0; j < L; ++j) {
                if (!whole && j >= len) {
                    a[j] = one, b[j] = zero;
                    continue;
                }
                const LruGate<decltype(close)::value> g(get(1, j), get(2, j), decay);
                const f32x2 root = sqrt_2(g.q);
                a[j] = g.a, b[j] = mul2(mul2(root, g.gi), get(0, j));
                if constexpr (M::kInPlace) {
                    *reinterpret_cast<f32x2 *>(staged + M::kRows + j * kLruCh) = g.gr;
                    *reinterpret_cast<f32x2 *>(staged + 2 * M::kRows + j * kLruCh) = g.gi;
                } else {
                    const float2 gr = unpack2(g.gr), gi = unpack2(g.gi);
                    gates_at[j * 32] = make_uint4(__float_as_uint(gr.x), __float_as_uint(gr.y), __float_as_uint(gi.x), __float_as_uint(gi.y));
                    const float2 q = unpack2(root);
                    *reinterpret_cast<float *>(staged + M::kRows + j * kLruCh) = q.x;
                    *reinterpret_cast<float *>(staged + 2 * M::kRows + j * kLruCh) = q.y;
                }
                f32x2 gd = get(3, j);
                if (Z) {
                    const f32x2 v = get(4, j);
                    gd = mul2(gd, mul2(v, sigmoid_2(v)));
                }
                if (PACKED && !whole) {
                    if (m.fin >> j & 1 && p.dh_final)
                        gd = add2(gd, lru_ld_state(p.dh_final, lru_seq(p.cu, p.n_seq, p.T, t0 + j), p.C, c, nc));
                    if (m.cut >> j & 1) {
                        if (p.h0) b[j] = fma2(a[j], lru_ld_state(p.h0, lru_seq(p.cu, p.n_seq, p.T, t0 + j), p.C, c, nc), b[j]);
                        run.A = pack2(-0.f, -0.f), run.H = b[j];
                        open = false;
                        continue;
                    }
                }
                run.H = fma2(a[j], run.H, b[j]);
                // (behind a cut A stays -0: a decay that is NaN would take the mark off)
                if (whole || open) run.A = mul2(run.A, a[j]), back = fma2(run.A, gd, back);
            }
        };
        if (HOW == kLruWide && near && all_inside) gates(std::true_type(), std::bool_constant<HOW == kLruWide>());
        else if (all_inside) gates(std::true_type(), std::false_type());
        else gates(std::false_type(), std::false_type());
        runs[flip][warp][lane] = run, backs[flip][warp][lane] = back;
        if (__syncthreads_or(lost)) break;
        f32x2 gm = carry;  // a g of the token behind this one
        if (K > 1) {
            if (warp == 0) {
                LruRun all{runs[flip][W - 1][lane].A, backs[flip][W - 1][lane]};
#pragma unroll
                for (int w = W - 2; w >= 0; --w) {
                    const f32x2 A = runs[flip][w][lane].A;
                    all.H = lru_apply2<PACKED>(A, backs[flip][w][lane], all.H), all.A = lru_join<PACKED>(all.A, A);
                }
                ranks.send(n, rank, all);
            }
        }
        // the state before this warp's tokens, from the one saved for its 64
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w / (kLruTile / L) != warp / (kLruTile / L)) continue;
            if (w >= warp) break;
            const LruRun v = runs[flip][w][lane];
            h = lru_apply2<PACKED>(v.A, v.H, h);
        }
        const f32x2 h_in = h;
#pragma unroll
        for (int j = 0; j < L; ++j)  // b becomes h (it stays where tokens end)
            h = b[j] = PACKED && m.cut >> j & 1 ? b[j] : fma2(a[j], h, b[j]);
        if (K > 1) {
            if (!ranks.wait(n, p.wait_us)) lost |= kLostRuns;
#pragma unroll 8
            for (int k = ranks.places - 1; k >= 0; --k) {
                const LruRun v = ranks.at(n, k);
                if (k == rank) gm = carry;
                carry = lru_apply2<PACKED>(v.A, v.H, carry);
            }
#pragma unroll
            for (int w = W - 1; w > 0; --w) {
                if (w <= warp) break;
                gm = lru_apply2<PACKED>(runs[flip][w][lane].A, backs[flip][w][lane], gm);
            }
        } else {
#pragma unroll
            for (int w = W - 1; w >= 0; --w) {
                if (w == warp) gm = carry;
                carry = lru_apply2<PACKED>(runs[flip][w][lane].A, backs[flip][w][lane], carry);
            }
        }
        const int64_t at0 = ((int64_t)line * p.T + t0) * p.C + c;
        auto walk = [&](auto form) {
            constexpr bool whole = decltype(form)::value;
#pragma unroll
            for (int j = L - 1; j >= 0; --j) {
                if (!whole && j >= len) continue;
                const int64_t at = at0 + (int64_t)j * p.C;
                f32x2 g = get(3, j);
                if (Z) {
                    // silu' = s + v s (1 - s)
                    const f32x2 v = get(4, j), s = sigmoid_2(v), vs = mul2(v, s);
                    const f32x2 ds = fma2(vs, fma2(s, minus, one), s);
                    if (nc > 0) lru_put<T, HOW>((T *)p.dz + at, mul2(mul2(g, b[j]), ds), nc);
                    g = mul2(g, vs);
                }
                f32x2 prev = j > 0 ? b[j > 0 ? j - 1 : 0] : h_in;
                if (PACKED && !whole && m.fin >> j & 1 && p.dh_final)
                    g = add2(g, lru_ld_state(p.dh_final, lru_seq(p.cu, p.n_seq, p.T, t0 + j), p.C, c, nc));
                g = add2(g, gm);
                gm = mul2(a[j], g);
                const f32x2 ag = gm;
                if (PACKED && !whole && m.cut >> j & 1) {
                    const int seq = lru_seq(p.cu, p.n_seq, p.T, t0 + j);
                    prev = lru_ld_state(p.h0, seq, p.C, c, nc);
                    if (p.dh0) lru_st_state(p.dh0, seq, p.C, c, nc, ag);
                    gm = zero;
                }
                f32x2 gr, gi, root, rs;  // sqrt(q) and its reciprocal
                if constexpr (M::kInPlace) {
                    gr = get(1, j), gi = get(2, j);
                    f32x2 av = a[j], q;  // (1 - a itself is not in a as exactly)
                    lru_decay2<false>(av, q, mul2(decay.rate, gr));
                    rs = rsqrt_2(q), root = mul2(q, rs);
                } else {
                    const uint4 v = gates_at[j * 32];
                    gr = pack2(__uint_as_float(v.x), __uint_as_float(v.y)), gi = pack2(__uint_as_float(v.z), __uint_as_float(v.w));
                    root = pack2(*reinterpret_cast<const float *>(staged + M::kRows + j * kLruCh),
                                 *reinterpret_cast<const float *>(staged + 2 * M::kRows + j * kLruCh));
                    const float2 q = unpack2(root);
                    rs = pack2(rcpf(fmaxf(q.x, 1e-18f)), rcpf(fmaxf(q.y, 1e-18f)));
                }
                const f32x2 u = mul2(decay.rate, gr);
                const f32x2 xv = get(0, j), ix = mul2(gi, xv);
                const f32x2 dx = mul2(mul2(g, root), gi), di = mul2(mul2(dx, xv), fma2(gi, minus, one));
                // u g (a^2 i x / sqrt(q) - a prev); u goes with 1 / sqrt(q) first, which
                // a masked token's x, however large, then meets as a zero
                const f32x2 w = mul2(ag, fma2(mul2(u, prev), minus, mul2(mul2(mul2(u, rs), a[j]), ix)));
                dlam = add2(dlam, w);
                if (nc > 0) {
                    lru_put<T, HOW>((T *)p.dx + at, dx, nc), lru_put<T, HOW>((T *)p.di + at, di, nc);
                    lru_put<T, HOW>((T *)p.dr + at, mul2(w, fma2(gr, minus, one)), nc);
                }
            }
        };
        if (all_inside) walk(std::true_type());
        else walk(std::false_type());
        if (HOW == kLruWide) fence_async_smem();  // (what was kept in their places, before the copies)
        __syncwarp();  // every lane is through with the stage
        fetch(n + 1);
    }
    if (n < steps || __any_sync(0xffffffffu, lost)) {
        if (lost && p.err) atomicOr(p.err, kDevErrTimeout);
        carry = dlam = nan;
        // (rows that did arrive have none behind them)
        if (HOW == kLruWide && lane == 0 && lost & kLostRows) lru_wait(smem_u32(&bars[warp]), n & 1, p.wait_us);
#pragma unroll 1
        for (n = lost & kLostRuns ? max(n - 1, 0) : n; n < steps; ++n) lose(n);
    }
    if (!PACKED && p.dh0 && rank == 0 && warp == 0) lru_st_state(p.dh0, line, p.C, c, nc, carry);
    // the channels' sums over the warps, in one order
    __syncthreads();
    f32x2 *sums = &backs[0][0][0];
    sums[warp * 32 + lane] = dlam;
    __syncthreads();
    if (warp == 0 && nc > 0) {
#pragma unroll
        for (int w = 1; w < W; ++w) dlam = add2(dlam, sums[w * 32 + lane]);
        const float2 f = unpack2(dlam);
        float o[2] = {f.x, f.y};
        for (int k = 0; k < 2; ++k) {
            if (k >= nc) break;
            const float lam = p.lam[c + k];  // sigmoid / softplus goes to 1
            if (lam > -15.f || lam != lam) o[k] *= sigmoid2(make_float2(lam, lam)).x / softplus2(make_float2(lam, lam)).x;
            p.part[((int64_t)line * K + rank) * p.C + c + k] = o[k];
        }
    }
    if (K > 1) cluster_sync();  // no CTA leaves before all have what it sent
}

}  // namespace

cudaError_t launch_lru_bwd(LruParams &p, cudaStream_t st) {
    LruMaps m{};
    constexpr int L = 8, W = 8;
    const int how = p.how == kLruWide && !lru_maps(p, true, L, &m) ? (int)kLruWords : p.how;
    return lru_by_form(p, how, p.z != nullptr, [&](auto type, auto how, auto packed, auto z) {
        using T = decltype(type);
        return lru_launch((const void *)lru_bwd_kernel<T, how(), packed(), z(), L, W>, W, LruBwdSmem<T, z(), L, W>::bytes, p, m, st);
    });
}

}  // namespace gdn

// gdn_ssm_bwd.cu -- the gradient of the selective scan. With dy = dout
// silu(z) and g the gradient of h, walked back in time,
//   g_t = C_t dy_t + a_{t+1} g_{t+1},
//   dC_n = sum_d dy h,  dB_n = sum_d delta x g,  dx = D dy + delta sum_n B g,
//   ddelta = sum_n A a h_{t-1} g + x sum_n B g,  dA = sum_t delta a h_{t-1} g,
//   ddt = ddelta sigmoid(dt + bias),  dz = dout y silu'(z),  dh0 = a_0 g_0.
//
// The line of tokens is cut into runs, a run into groups of 32 tokens:
//   ssm_bwd_sum   per group the state from zero and the sum of delta, per run
//                 the gradient that reaches its start from its own tokens
//                 (sum over t of prod_{s <= t} a_s C_t dy_t);
//   ssm_bwd_chain both chained: the state entering every group, the gradient
//                 leaving every run;
//   ssm_bwd       one CTA walks a run back group by group: states forward
//                 with a checkpoint every four tokens, then back four at a
//                 time, the four tokens' entering states and decays in
//                 registers;
//   ssm_bwd_reduce  dB and dC over the channel tiles; dA, dD and dbias over
//                 the runs. Every sum has one order.
// Bound by the latencies between dependent instructions at 11 to 13 warps a
// SM (issue slots 57 to 63 % used, DRAM 10 to 19 %) and by the number of
// instructions: the states' decays are formed three times (12 cycles a warp for
// 32 elements on the exponential unit) and the walk back has ten packed
// operations an element pair. 4 x 4096 tokens of 4096 channels, 16 states,
// bf16: sums 409 us, chain 61, walk 1403 (fp32 1726), sums of parts 35.
#include "gdn_ssm.cuh"

namespace gdn {
namespace {

constexpr int kNT = 64;      // threads of every CTA here
constexpr int kGroup = kSsmGroup;
constexpr int kStage = 8;    // tokens a stage of the sums

// ------------------------------------------------------------ sums ----------
// A lane has eight states of two neighbouring channels: their state, the
// run's gradient and the decay since the run's start. What a token's channels
// need once is formed by the warp for a stage of tokens and handed over in
// shared memory, as in the scan.
template <typename T, int LN, bool USUAL>
__global__ void __launch_bounds__(kNT, 8) ssm_bwd_sum_kernel(const SsmParams p, int ntile) {
    constexpr int Q = 8, CH = 2 * kNT / LN, NP = Q * LN, TS = kStage, NA = 4;  // x, dt, z, dout
    constexpr int kTile = TS * CH * (int)sizeof(T), kBuf = NA * kTile, kBc = TS * 2 * NP, PW = 32 / LN;
    extern __shared__ __align__(16) unsigned char smem[];
    float4 *dus = reinterpret_cast<float4 *>(smem + 2 * kBuf);            // [TS][CH / 2] delta, delta x
    float2 *dys = reinterpret_cast<float2 *>(dus + TS * CH / 2);          // [TS][CH / 2] dy
    float *bcs = reinterpret_cast<float *>(dys + TS * CH / 2);            // [2][TS][2][NP]
    const int tid = threadIdx.x, lane = tid & 31, pr = tid / LN, ch = 2 * pr, ln = tid % LN;
    const int tile = blockIdx.x % ntile, item = blockIdx.x / ntile;
    const int line = item / p.nrun, run = item - line * p.nrun;
    const int t0 = run * p.rlen, t1 = min(p.T - t0, p.rlen) + t0;
    const int c0 = tile * CH, d = c0 + ch, n0 = ln * Q, nn = p.N - n0;
    const bool on[2] = {d < p.D && nn > 0, d + 1 < p.D && nn > 0};
    const int64_t hrow = (int64_t)p.D * p.N, dnp = (int64_t)p.D * NP;
    const int64_t own = (int64_t)d * p.N + n0, own_p = (int64_t)d * NP + n0;
    const bool softplus = USUAL || p.softplus, gate = USUAL || p.z, vec = USUAL || p.vec;

    f32x2 a2[2][Q / 2], h[2][Q / 2], g[2][Q / 2], w[2][Q / 2];  // w: the decay since the run's start
    ld_pair<Q>(a2, p.A + own, p.N, nn, p.n_wide, on);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < Q / 2; ++j) {
            a2[k][j] = mul2(a2[k][j], pack2(kLog2e, kLog2e));
            g[k][j] = pack2(0.f, 0.f), w[k][j] = pack2(1.f, 1.f);
        }
    auto first_h = [&](int seg, bool zero) {
        if (p.h0 && !zero) {
            ld_pair<Q>(h, p.h0 + seg * hrow + own, p.N, nn, p.n_wide, on);
        } else {
#pragma unroll
            for (int j = 0; j < Q / 2; ++j) h[0][j] = h[1][j] = pack2(0.f, 0.f);
        }
    };
    SsmSeq q = ssm_find(p.cu, p.n_seq, p.T, line, t0);
    bool reset = q.starts, alive = true;
    first_h(q.seg, !q.starts);

    const T *src[4] = {(const T *)p.x + line * p.x_sb, (const T *)p.dt + line * p.dt_sb,
                       (const T *)p.z + line * p.z_sb, (const T *)p.dout + line * p.do_sb};
    const int64_t str[4] = {p.x_st, p.dt_st, p.z_st, p.do_st};
    // as in the scan
    auto tile_at = [&](int b, int a) { return reinterpret_cast<T *>(smem + b * kBuf + a * kTile); };
    auto copy = [&](int s, int b) {
        if (s < t1) {
#pragma unroll
            for (int a = 0; a < NA; ++a)
                if (a != 2 || gate)
                    ssm_copy_tile<T, CH, TS, kNT>(tile_at(b, a), src[a] + s * str[a], str[a], t1 - s, c0, p.D);
        }
        cp_async_commit();
    };
    SsmTile<T, CH, TS, kNT> held[USUAL ? 1 : NA];
    auto hold = [&](int s) {
#pragma unroll
        for (int a = 0; a < (USUAL ? 0 : NA); ++a)
            if (a != 2 || gate) held[a].load(src[a] + s * str[a], str[a], t1 - s, c0, p.D);
    };
    auto release = [&](int b) {
#pragma unroll
        for (int a = 0; a < (USUAL ? 0 : NA); ++a)
            if (a != 2 || gate) held[a].store(tile_at(b, a));
    };
    const T *bg = (const T *)p.bm + line * p.bm_sb, *cg = (const T *)p.cm + line * p.cm_sb;
    SsmBc<T, NP, TS, kNT> nbc;
    auto fetch_bc = [&](int s) {
        nbc.template fetch<true>(bg + s * p.bm_st, p.bm_st, cg + s * p.cm_st, p.cm_st, t1 - s, p.N, p.bc_vec);
    };
    if (vec) {
        copy(t0, 0);
        copy(t0 + TS, 1);
    } else {
        hold(t0);
        release(0);
    }
    fetch_bc(t0);
    float *gs = p.gs + ((int64_t)line * p.nrun + run) * dnp + own_p;
    float2 dsum = make_float2(0.f, 0.f), rsum = dsum;  // of the group, of the run
    int buf = 0;
    for (int s = t0; s < t1; s += TS, buf ^= 1) {
        float *bc = bcs + buf * kBc;
        nbc.stage(bc);
        if (s + TS < t1) fetch_bc(s + TS);
        if (vec) cp_async_wait<1>();
        else if (s + TS < t1) hold(s + TS);
        __syncthreads();
        const int m = min(t1 - s, TS);
        // this warp's pairs of the stage
#pragma unroll 2
        for (int e = lane; e < TS * PW; e += 32) {
            const int t = e / PW, k = tid / 32 * PW + e % PW, c = c0 + 2 * k;
            const T *xs = reinterpret_cast<const T *>(smem + buf * kBuf) + t * CH + 2 * k;
            float x[2], v[2], o[2];
            ld_row_f<T, 2, true>(x, xs, 2);
            ld_row_f<T, 2, true>(v, xs + TS * CH, 2);
            ld_row_f<T, 2, true>(o, xs + 3 * TS * CH, 2);
            float2 dl = make_float2(v[0], v[1]);
            if (p.dt_bias) {
                if (c < p.D) dl.x += p.dt_bias[c];
                if (c + 1 < p.D) dl.y += p.dt_bias[c + 1];
            }
            if (softplus) dl = softplus2(dl);
            if (gate) {
                float z[2];
                ld_row_f<T, 2, true>(z, xs + 2 * TS * CH, 2);
                const float2 sg = sigmoid2(make_float2(z[0], z[1]));
                o[0] *= z[0] * sg.x, o[1] *= z[1] * sg.y;
            }
            dus[t * (CH / 2) + k] = make_float4(dl.x, dl.y, dl.x * x[0], dl.y * x[1]);
            dys[t * (CH / 2) + k] = make_float2(o[0], o[1]);
        }
        __syncwarp();
        auto token = [&](int t) {
            const float4 du = dus[t * (CH / 2) + pr];
            const float2 dy = dys[t * (CH / 2) + pr];
            dsum.x += du.x, dsum.y += du.y;
            const float4 *b4 = reinterpret_cast<const float4 *>(bc + t * 2 * NP + n0);
            const f32x2 d2[2] = {pack2(du.x, du.x), pack2(du.y, du.y)}, u2[2] = {pack2(du.z, du.z), pack2(du.w, du.w)};
            const f32x2 y2[2] = {pack2(dy.x, dy.x), pack2(dy.y, dy.y)};
#pragma unroll
            for (int j = 0; j < Q / 4; ++j) {
                const float4 b = b4[j], c = b4[NP / 4 + j];
                const f32x2 b2[2] = {pack2(b.x, b.y), pack2(b.z, b.w)}, c2[2] = {pack2(c.x, c.y), pack2(c.z, c.w)};
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int l = 2 * j + i;
                        const f32x2 a = ex2_2(mul2(d2[k], a2[k][l]));
                        h[k][l] = fma2(a, h[k][l], mul2(u2[k], b2[i]));
                        // the run's start lies before this token's decay
                        w[k][l] = mul2(w[k][l], a);
                        g[k][l] = fma2(w[k][l], mul2(c2[i], y2[k]), g[k][l]);
                    }
            }
        };
        // a group's state, and zero for the next
        auto cut = [&](int last) {
            const int64_t at = (int64_t)line * p.ngroup + last / kGroup;
            st_pair<Q>(p.sums + at * dnp + own_p, h, NP, Q, true, on);
            float *o = p.dsum + at * p.D + d;
            if (ln == 0 && d < p.D) o[0] = reset ? __int_as_float(0x7fffffff) : dsum.x;
            if (ln == 0 && d + 1 < p.D) o[1] = reset ? __int_as_float(0x7fffffff) : dsum.y;
            rsum.x += dsum.x, rsum.y += dsum.y;
            dsum = make_float2(0.f, 0.f);
            reset = false;
            first_h(0, true);
        };
        if (m == TS && q.end > s + TS) {  // no sequence ends in the stage; groups end with stages
#pragma unroll 4
            for (int t = 0; t < TS; ++t) token(t);
            if ((s + TS) % kGroup == 0 || s + TS == t1) cut(s + TS - 1);
        } else {
#pragma unroll 1
            for (int t = 0; t < m; ++t) {
                token(t);
                const int tt = s + t + 1;
                if (tt == t1 || tt % kGroup == 0) cut(tt - 1);
                if (tt == q.end) {
                    if (alive) {
                        if (p.dh_final) {
                            f32x2 e[2][Q / 2];
                            ld_pair<Q>(e, p.dh_final + q.seg * hrow + own, p.N, nn, p.n_wide, on);
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int j = 0; j < Q / 2; ++j) g[k][j] = fma2(w[k][j], e[k][j], g[k][j]);
                        }
                        // what follows belongs to other sequences
                        st_pair<Q>(gs, g, NP, Q, true, on);
                        alive = false;
                    }
                    if (tt < p.T) {
                        ssm_next(q, p.cu, p.n_seq, p.T, tt);
                        first_h(q.seg, false);
                        reset = true;
                    }
                }
            }
        }
        __syncthreads();  // the buffer has been read
        if (vec) copy(s + 2 * TS, buf);
        else if (s + TS < t1) release(buf ^ 1);
    }
    if (alive) st_pair<Q>(gs, g, NP, Q, true, on);
    if (ln == 0) {  // where nothing crosses the run: marked by NaN
        float *r = p.gsum + ((int64_t)line * p.nrun + run) * p.D + d;
        if (d < p.D) r[0] = alive ? rsum.x : __int_as_float(0x7fffffff);
        if (d + 1 < p.D) r[1] = alive ? rsum.y : __int_as_float(0x7fffffff);
    }
}

// Blocks with y = 0: the state entering group c + 1 replaces group c's, h <-
// exp(A sum delta) h + S. With y = 1: the gradient at the start of each run,
// G <- G + exp(A sum delta over the run) (G of the next run), from the last. Four
// loads ahead of their stores: 61 us for 4 x 4096 tokens of 4096 channels, 16
// states (eight 72, sixteen 109).
__global__ void __launch_bounds__(256) ssm_bwd_chain_kernel(const SsmParams p, int np) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, dnp = (int64_t)p.D * np;
    const int lines = p.cu ? 1 : p.B;
    if (i >= lines * dnp) return;
    const int line = (int)(i / dnp), d = (int)(i % dnp / np), n = (int)(i % np);
    const float a = n < p.N ? p.A[(int64_t)d * p.N + n] * kLog2e : 0.f;
    if (blockIdx.y == 0) {
        float *s = p.sums + (int64_t)line * p.ngroup * dnp + i % dnp;
        const float *q = p.dsum + (int64_t)line * p.ngroup * p.D + d;
        float h = 0.f;
        for (int c = 0; c + 1 < p.ngroup; c += 4) {
            float v[4], e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = c + k + 1 < p.ngroup;
                v[k] = in ? q[(int64_t)(c + k) * p.D] : 0.f, e[k] = in ? s[(c + k) * dnp] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h = isnan(v[k]) || h == 0.f ? e[k] : fmaf(ex2f(a * v[k]), h, e[k]);  // (A > 0 may overflow)
                if (c + k + 1 < p.ngroup) s[(c + k) * dnp] = h;
            }
        }
    } else {
        float *s = p.gs + (int64_t)line * p.nrun * dnp + i % dnp;
        const float *q = p.gsum + (int64_t)line * p.nrun * p.D + d;
        float g = 0.f;
        for (int r = p.nrun - 1; r >= 0; r -= 4) {
            float v[4], e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = r >= k ? q[(int64_t)(r - k) * p.D] : 0.f, e[k] = r >= k ? s[(r - k) * dnp] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                g = isnan(v[k]) || g == 0.f ? e[k] : fmaf(ex2f(a * v[k]), g, e[k]);
                if (r >= k) s[(r - k) * dnp] = g;
            }
        }
    }
}

// -------------------------------------------------------------- walk back ---
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

constexpr int kWalk = 128;  // threads of the walk's CTA

// Lanes: lane = ln * CL + lc has channel lc of its warp and states ln Q ..
// ln Q + Q - 1, eight of them up to N = 64. More states a lane would spare
// work that is repeated by a channel's lanes, but the four tokens' states and
// decays then fill the register file (16 states a lane: 255 registers, two
// warps a scheduler, 1.9 to 2.3 ms for 16384 tokens of 4096 channels).
//
// dB and dC are sums over channels, i.e. over lanes: 2 Q values a lane and
// token, in fp32 and apart for every state, so that a rounding or a value that
// is not finite stays in its own sum. Eight states at a time: at each step two
// lanes, one bit of the channel apart, exchange the half of the values that
// the other one goes on with: quads of states, dB or dC, pairs, elements
// (8 + 4 + 2 + 1 shuffles of 16 values for 16 lanes). Lanes of odd channels hold
// their quads in swapped order, so that the first exchange, of half of all
// shuffles, selects nothing. (By tensor-core products against ones: in tf32,
// 1476 us for 1403 here, in two parts for fp32 tensors 2053 for 1726, and a
// value that is not finite spread over eight states of both sums.)
__device__ __forceinline__ f32x2 shfl_xor2(f32x2 v, int lanes) {
    const float2 f = unpack2(v);
    return pack2(__shfl_xor_sync(0xffffffffu, f.x, lanes), __shfl_xor_sync(0xffffffffu, f.y, lanes));
}
// rb, rc: eight states of a channel, own quad first. Adds the sums over CL
// neighbouring lanes to to[0 .. 7] (dB) and to[np .. np + 7] (dC), where two
// warps add to zeros: either order gives the same sum.
template <int CL>
__device__ __forceinline__ void channel_sums(const f32x2 *rb, const f32x2 *rc, float *to, int np, int lane) {
    const bool u1 = lane & 2;
    f32x2 k[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2 b = add2(rb[i], shfl_xor2(rb[2 + i], 1)), c = add2(rc[i], shfl_xor2(rc[2 + i], 1));
        k[i] = add2(u1 ? c : b, shfl_xor2(u1 ? b : c, 2));
    }
    to += (u1 ? np : 0) + (lane & 1) * 4;
    if constexpr (CL == 4) {
        const float2 f0 = unpack2(k[0]), f1 = unpack2(k[1]);
        atomicAdd(to, f0.x), atomicAdd(to + 1, f0.y), atomicAdd(to + 2, f1.x), atomicAdd(to + 3, f1.y);
    } else {
        const bool u2 = lane & 4;
        const float2 f = unpack2(add2(u2 ? k[1] : k[0], shfl_xor2(u2 ? k[0] : k[1], 4)));
        to += u2 ? 2 : 0;
        if constexpr (CL == 8) {
            atomicAdd(to, f.x), atomicAdd(to + 1, f.y);
        } else {
            const bool u3 = lane & 8;
            float s = (u3 ? f.y : f.x) + __shfl_xor_sync(0xffffffffu, u3 ? f.x : f.y, 8);
            if (CL == 32) s += __shfl_xor_sync(0xffffffffu, s, 16);
            if (CL == 16 || !(lane & 16)) atomicAdd(to + (u3 ? 1 : 0), s);
        }
    }
}

template <typename T, int Q, int LN, bool USUAL>
__global__ void __launch_bounds__(kWalk, Q == 8 ? 3 : 2) ssm_bwd_kernel(const SsmParams p, int ntile) {
    constexpr int NP = Q * LN, CL = 32 / LN, CH = 4 * CL, TG = kGroup, SUB = 4, H = Q / 2;
    constexpr int kTile = TG * CH, kPart = TG * 2 * NP;
    extern __shared__ __align__(16) unsigned char smem[];
    T *tiles = reinterpret_cast<T *>(smem);                     // x, dt, z, dout: [4][TG][CH]
    float *dls = reinterpret_cast<float *>(tiles + 4 * kTile);  // delta: [TG][CH]
    float *dys = dls + kTile;                                   // dy: [TG][CH]
    float *bcs = dys + kTile;                                   // [TG][2][NP]
    float *part = bcs + kPart;                                  // [2][TG][2][NP], two warps' sums each
    float4 *ckpt = reinterpret_cast<float4 *>(part + 2 * kPart);  // [TG / SUB - 2][Q / 4][kWalk]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ln = lane / CL, lc = lane % CL, fk = ln & 1, sw = lc & 1;  // sw: quads of states swapped
    const int tile = blockIdx.x % ntile, item = blockIdx.x / ntile;
    const int line = item / p.nrun, run = item - line * p.nrun;
    const int r0 = run * p.rlen, r1 = min(p.T - r0, p.rlen) + r0;
    const int c0 = tile * CH, ch = warp * CL + lc, d = c0 + ch, n0 = ln * Q, nn = p.N - n0;
    const bool on = d < p.D && nn > 0, fin = d < p.D && ln < 2;
    const int ns = on ? nn : 0, qs = on ? Q : 0;
    const int64_t hrow = (int64_t)p.D * p.N, dnp = (int64_t)p.D * NP;
    const int64_t own = (int64_t)d * p.N + n0, own_p = (int64_t)d * NP + n0;
    const bool softplus = USUAL || p.softplus, gate = USUAL || p.z, vec = USUAL || p.vec;

    f32x2 a2[H], g[H], dA[H], h[H], w[SUB][H], a[SUB][H];
    ld_states<Q>(a2, p.A + own, ns, p.n_wide, sw);
#pragma unroll
    for (int j = 0; j < H; ++j) {
        a2[j] = mul2(a2[j], pack2(kLog2e, kLog2e));
        g[j] = dA[j] = pack2(0.f, 0.f);
    }
    // from the run's end on
    if (run + 1 < p.nrun) ld_states<Q>(g, p.gs + ((int64_t)line * p.nrun + run + 1) * dnp + own_p, qs, true, sw);
    float dD = 0.f, dbias = 0.f;
    const float dv = p.Dv && d < p.D ? p.Dv[d] : 0.f, bias = p.dt_bias && d < p.D ? p.dt_bias[d] : 0.f;
    const T *src[4] = {(const T *)p.x + line * p.x_sb, (const T *)p.dt + line * p.dt_sb,
                       (const T *)p.z + line * p.z_sb, (const T *)p.dout + line * p.do_sb};
    const int64_t str[4] = {p.x_st, p.dt_st, p.z_st, p.do_st};

    // the pair of channels whose delta and dy this thread forms
    static_assert(kWalk % (CH / 2) == 0, "a thread keeps its pair");
    const int pc = tid % (CH / 2);
    const float2 pbias = make_float2(p.dt_bias && c0 + 2 * pc < p.D ? p.dt_bias[c0 + 2 * pc] : 0.f,
                                     p.dt_bias && c0 + 2 * pc + 1 < p.D ? p.dt_bias[c0 + 2 * pc + 1] : 0.f);
    auto boundary = [&](const float *from, int seg, f32x2 (&v)[H]) {  // a sequence's h0 or dh_final, or zero
        if (from) {
            ld_states<Q>(v, from + seg * hrow + own, ns, p.n_wide, sw);
        } else {
#pragma unroll
            for (int j = 0; j < H; ++j) v[j] = pack2(0.f, 0.f);
        }
    };
    for (int grp = (r1 - 1) / TG; grp * TG >= r0; --grp) {
        const int t0 = grp * TG, m = min(p.T - t0, TG);
        __syncthreads();  // the group before has been read
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k == 2 && !gate) continue;
            if (vec) {
                ssm_copy_tile<T, CH, TG, kWalk>(tiles + k * kTile, src[k] + t0 * str[k], str[k], m, c0, p.D);
            } else {
                SsmTile<T, CH, TG, kWalk> tile;
                tile.load(src[k] + t0 * str[k], str[k], m, c0, p.D);
                tile.store(tiles + k * kTile);
            }
        }
        cp_async_commit();
        {
            SsmBc<T, NP, TG, kWalk> bc;
            bc.template fetch<true>((const T *)p.bm + line * p.bm_sb + t0 * p.bm_st, p.bm_st,
                                    (const T *)p.cm + line * p.cm_sb + t0 * p.cm_st, p.cm_st, m, p.N, p.bc_vec);
            bc.stage(bcs);
        }
        // tokens at which a sequence begins, and those that end one
        uint32_t starts;
        {
            bool s = false;
            if (lane < m) s = ssm_find(p.cu, p.n_seq, p.T, line, t0 + lane).starts;
            starts = __ballot_sync(0xffffffffu, s);
        }
        bool end_last = t0 + m == p.T;
        if (!end_last && p.cu) end_last = ssm_find(p.cu, p.n_seq, p.T, line, t0 + m).starts;
        const uint32_t ends = starts >> 1 | (end_last ? 1u << (m - 1) : 0u);
        for (int e = tid; e < 2 * kPart; e += kWalk) part[e] = 0.f;
        cp_async_wait<0>();
        __syncthreads();
        // delta and dy of the tile, by pairs of channels (each thread's own)
#pragma unroll 2
        for (int r = tid / (CH / 2); r < TG; r += kWalk / (CH / 2)) {
            const int c = 2 * pc;
            float f[2];
            ld_row_f<T, 2, true>(f, tiles + kTile + r * CH + c, 2);
            float2 v = make_float2(f[0] + pbias.x, f[1] + pbias.y);
            if (softplus) v = softplus2(v);
            *reinterpret_cast<float2 *>(dls + r * CH + c) = v;
            ld_row_f<T, 2, true>(f, tiles + 3 * kTile + r * CH + c, 2);
            if (gate) {
                float z[2];
                ld_row_f<T, 2, true>(z, tiles + 2 * kTile + r * CH + c, 2);
                const float2 sg = sigmoid2(make_float2(z[0], z[1]));
                f[0] *= z[0] * sg.x, f[1] *= z[1] * sg.y;
            }
            *reinterpret_cast<float2 *>(dys + r * CH + c) = make_float2(f[0], f[1]);
        }
        __syncthreads();
        if (grp * TG > r0) {  // the next group's rows and states towards L2
            constexpr int kLine = 128 / (int)sizeof(T), kPer = (CH + kLine - 1) / kLine;
            for (int e = tid; e < 4 * TG * kPer; e += kWalk) {
                const int k = e / (TG * kPer), r = e / kPer % TG, c = c0 + e % kPer * kLine;
                if ((k != 2 || gate) && c < p.D) prefetch_l2(src[k] + (t0 - TG + r) * str[k] + c);
            }
            if (grp > 1 && fin) prefetch_l2(p.sums + ((int64_t)line * p.ngroup + grp - 2) * dnp + own_p);
        }
        const T *xs = tiles + ch;
        const int64_t o0 = ((int64_t)line * p.T + t0) * p.D + d;
        T *dxp = (T *)p.dx + o0, *dtp = (T *)p.ddt + o0, *dzp = (T *)p.dz + o0;
        // Edge groups, in which a sequence begins or ends or which are not
        // whole, ask at every token; the others run without a branch.
        auto group = [&](auto edge_c) {
            constexpr bool EDGE = decltype(edge_c)::value;
            const int nsub = EDGE ? (m + SUB - 1) / SUB : TG / SUB;
            auto seg_of = [&](int t) { return ssm_find(p.cu, p.n_seq, p.T, line, t0 + t).seg; };
            // one token forward: wd = a h, h <- wd + u B
            auto forward = [&](f32x2 (&wd)[H], f32x2 (&ad)[H], int i) {
                const float dl = dls[i * CH + ch], u = dl * ldf(xs + i * CH);
                const f32x2 d2 = pack2(dl, dl), u2 = pack2(u, u);
                const float4 *b4 = reinterpret_cast<const float4 *>(bcs + i * 2 * NP + n0);
#pragma unroll
                for (int j = 0; j < Q / 4; ++j) {
                    const float4 b = b4[j ^ sw];
                    const f32x2 b2[2] = {pack2(b.x, b.y), pack2(b.z, b.w)};
#pragma unroll
                    for (int l = 2 * j; l < 2 * j + 2; ++l) {
                        ad[l] = ex2_2(mul2(d2, a2[l]));
                        wd[l] = mul2(ad[l], h[l]);
                        h[l] = fma2(u2, b2[l & 1], wd[l]);
                    }
                }
            };
            // the state entering the group; the first sub-block's is read again
            // where the walk reaches it, the last one's stays in registers
            auto enter = [&] {
                if (grp > 0 && !(EDGE && (starts & 1u)))
                    ld_states<Q>(h, p.sums + ((int64_t)line * p.ngroup + grp - 1) * dnp + own_p, qs, true, sw);
                else
                    boundary(nullptr, 0, h);
            };
            // what a channel's outputs need of token t: its sums over the states
            auto finish = [&](int t, float y, float s1, float s2, bool here) {
                const float dl = dls[t * CH + ch], dy = dys[t * CH + ch], x = ldf(xs + t * CH);
                y = fmaf(dv, x, y);
                float dd = fmaf(x, s1, s2 * 0.6931471805599453f);
                // sigmoid(v) = exp(v - softplus(v))
                if (softplus) dd *= ex2f((ldf(xs + kTile + t * CH) + bias - dl) * kLog2e);
                if (fin && here) {
                    const int at = t * p.D;
                    dxp[at] = to_type<T>(fmaf(dv, dy, dl * s1));
                    dtp[at] = to_type<T>(dd);
                    if (gate && (USUAL || p.dz)) {
                        const float z = ldf(xs + 2 * kTile + t * CH), go = ldf(xs + 3 * kTile + t * CH);
                        const float sg = rcpf(1.f + ex2f(z * -kLog2e));
                        dzp[at] = to_type<T>(go * y * sg * fmaf(z, 1.f - sg, 1.f));
                    }
                    dD = fmaf(dy, x, dD);
                    dbias += dd;
                }
            };
            enter();
#pragma unroll 1
            for (int sb = 0; sb + 1 < nsub; ++sb) {
                if (sb > 0) {
#pragma unroll
                    for (int k = 0; k < Q / 4; ++k) {
                        const float2 u = unpack2(h[2 * k]), v = unpack2(h[2 * k + 1]);
                        ckpt[((sb - 1) * (Q / 4) + k) * kWalk + tid] = make_float4(u.x, u.y, v.x, v.y);
                    }
                }
#pragma unroll
                for (int i = 0; i < SUB; ++i) {
                    const int t = sb * SUB + i;
                    if (EDGE && (starts >> t & 1u)) boundary(p.h0, seg_of(t), h);
                    forward(w[0], a[0], t);
                }
            }
#pragma unroll 1
            for (int sb = nsub - 1; sb >= 0; --sb) {
                if (sb == 0 && nsub > 1) {
                    enter();
                } else if (sb + 1 < nsub) {
#pragma unroll
                    for (int k = 0; k < Q / 4; ++k) {
                        const float4 f = ckpt[((sb - 1) * (Q / 4) + k) * kWalk + tid];
                        h[2 * k] = pack2(f.x, f.y), h[2 * k + 1] = pack2(f.z, f.w);
                    }
                }
#pragma unroll
                for (int i = 0; i < SUB; ++i) {
                    const int t = sb * SUB + i;
                    if (EDGE && t >= m) continue;
                    if (EDGE && (starts >> t & 1u)) boundary(p.h0, seg_of(t), h);
                    forward(w[i], a[i], t);
                }
                float r[2][3];  // y, sum B g, sum A a h g of two tokens
#pragma unroll
                for (int i = SUB - 1; i >= 0; --i) {
                    const int t = sb * SUB + i;
                    if (EDGE && t >= m) {
                        r[i & 1][0] = r[i & 1][1] = r[i & 1][2] = 0.f;
                    } else {
                        if (EDGE && (ends >> t & 1u)) boundary(p.dh_final, seg_of(t), g);
                        const float dl = dls[t * CH + ch], u = dl * ldf(xs + t * CH), dy = dys[t * CH + ch];
                        const f32x2 d2 = pack2(dl, dl), u2 = pack2(u, u), y2 = pack2(dy, dy);
                        const float4 *b4 = reinterpret_cast<const float4 *>(bcs + t * 2 * NP + n0);
                        f32x2 ys, gb, gd, rb[H], rc[H];
#pragma unroll
                        for (int j = 0; j < Q / 4; ++j) {
                            const float4 b = b4[j ^ sw], c = b4[NP / 4 + (j ^ sw)];
                            const f32x2 b2[2] = {pack2(b.x, b.y), pack2(b.z, b.w)};
                            const f32x2 c2[2] = {pack2(c.x, c.y), pack2(c.z, c.w)};
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int l = 2 * j + k;
                                const f32x2 hn = fma2(u2, b2[k], w[i][l]);  // h_t
                                const f32x2 gn = fma2(c2[k], y2, g[l]);
                                const f32x2 e = mul2(gn, w[i][l]);          // g a h_{t-1}
                                ys = l ? fma2(hn, c2[k], ys) : mul2(hn, c2[k]);
                                gb = l ? fma2(gn, b2[k], gb) : mul2(gn, b2[k]);
                                gd = l ? fma2(e, a2[l], gd) : mul2(e, a2[l]);
                                rb[l] = mul2(u2, gn), rc[l] = mul2(y2, hn);
                                dA[l] = fma2(e, d2, dA[l]);
                                g[l] = mul2(gn, a[i][l]);
                            }
                        }
                        if (EDGE && (starts >> t & 1u) && p.dh0)
                            st_states<Q>(p.dh0 + seg_of(t) * hrow + own, g, ns, p.n_wide, sw);
                        const float2 v0 = unpack2(ys), v1 = unpack2(gb), v2 = unpack2(gd);
                        r[i & 1][0] = v0.x + v0.y, r[i & 1][1] = v1.x + v1.y, r[i & 1][2] = v2.x + v2.y;
                        // over the channels: dB and dC. Two warps add to zeros: either order gives
                        // the same sum.
                        float *pw = part + (warp >> 1) * kPart + t * 2 * NP + n0;
#pragma unroll
                        for (int o = 0; o < Q / 8; ++o)
                            channel_sums<CL>(rb + 4 * o, rc + 4 * o, pw + 8 * o, NP, lane);
                    }
                    if (i & 1) continue;
                    // two tokens are done: lanes ln = 0 and 1 finish one each
                    if constexpr (LN == 1) {
                        finish(t + 1, r[1][0], r[1][1], r[1][2], !EDGE || t + 1 < m);
                        finish(t, r[0][0], r[0][1], r[0][2], !EDGE || t < m);
                    } else {
                        float s[3];
#pragma unroll
                        for (int q = 0; q < 3; ++q) {
#pragma unroll
                            for (int o = 2 * CL; o < 32; o <<= 1) {
                                r[0][q] += __shfl_xor_sync(0xffffffffu, r[0][q], o);
                                r[1][q] += __shfl_xor_sync(0xffffffffu, r[1][q], o);
                            }
                            const float give = fk ? r[0][q] : r[1][q], keep = fk ? r[1][q] : r[0][q];
                            s[q] = keep + __shfl_xor_sync(0xffffffffu, give, CL);
                        }
                        finish(t + fk, s[0], s[1], s[2], !EDGE || t + fk < m);
                    }
                }
            }
        };
        if (m < TG || (starts | ends)) group(std::true_type());
        else group(std::false_type());
        __syncthreads();
        // the tile's dB and dC of the group
        for (int e = tid; e < m * 2 * p.N; e += kWalk) {
            const int r = e / (2 * p.N), k = e % (2 * p.N), n = r * 2 * NP + (k < p.N ? k : NP + k - p.N);
            p.part_bc[((int64_t)tile * p.B * p.T + (int64_t)line * p.T + t0 + r) * (2 * p.N) + k] = part[n] + part[kPart + n];
        }
    }
    st_states<Q>(p.part_a + ((int64_t)line * p.nrun + run) * hrow + own, dA, ns, p.n_wide, sw);
    // dD and dbias: each of the two lanes has half of the tokens
    if (LN > 1) {
        dD += __shfl_xor_sync(0xffffffffu, dD, CL);
        dbias += __shfl_xor_sync(0xffffffffu, dbias, CL);
    }
    if (d < p.D && ln == 0) {
        float *pd = p.part_d + ((int64_t)line * p.nrun + run) * 2 * p.D + d;
        pd[0] = dD, pd[p.D] = dbias;
    }
}

// What the walk left in parts, in one launch. The first nbc blocks: dB and dC
// over the channel tiles, rounded once. The next nd: dA, dD and dbias over the
// runs, 32 columns a block. The rest: without a token in a sequence its
// state's gradient passes through.
template <typename T>
__global__ void __launch_bounds__(256) ssm_bwd_reduce_kernel(const SsmParams p, int tiles, unsigned nbc, unsigned nd) {
    __shared__ float red[8][33];
    const int64_t dn = (int64_t)p.D * p.N;
    if (p.err && blockIdx.x == 0) ssm_check_cu(p.cu, p.n_seq, p.T, p.err);
    if (blockIdx.x < nbc) {
        const int64_t rows = (int64_t)p.B * p.T, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        if (i >= rows * 2 * p.N) return;
        float a = 0.f;
#pragma unroll 8
        for (int k = 0; k < tiles; ++k) a += p.part_bc[k * rows * 2 * p.N + i];
        const int64_t r = i / (2 * p.N);
        const int n = (int)(i - r * 2 * p.N);
        if (n < p.N) ((T *)p.dbm)[r * p.N + n] = to_type<T>(a);
        else ((T *)p.dcm)[r * p.N + n - p.N] = to_type<T>(a);
    } else if (blockIdx.x < nbc + nd) {
        const int x = threadIdx.x & 31, y = threadIdx.x >> 5, parts = (p.cu ? 1 : p.B) * p.nrun;
        const int64_t c = (int64_t)(blockIdx.x - nbc) * 32 + x;  // a column of dA, then of dD, then of dbias
        const bool in = c < dn + 2 * p.D;
        const float *from = c < dn ? p.part_a + c : p.part_d + (c - dn);
        const int64_t ld = c < dn ? dn : 2 * p.D;
        float a = 0.f;
        if (in) {
#pragma unroll 4
            for (int k = y; k < parts; k += 8) a += from[k * ld];
        }
        red[y][x] = a;
        __syncthreads();
        if (y > 0 || !in) return;
#pragma unroll
        for (int i = 1; i < 8; ++i) a += red[i][x];
        if (c < dn) p.dA[c] = a;
        else if (c < dn + p.D) {
            if (p.dD) p.dD[c - dn] = a;
        } else if (p.ddt_bias) {
            p.ddt_bias[c - dn - p.D] = a;
        }
    } else {
        const unsigned nb = gridDim.x - nbc - nd;
        for (int64_t i = (int64_t)(blockIdx.x - nbc - nd) * 256 + threadIdx.x; i < dn; i += (int64_t)nb * 256)
            for (int s = 0; s < p.n_seq; ++s)
                if (p.cu ? p.cu[s + 1] <= p.cu[s] : p.T == 0)
                    p.dh0[s * dn + i] = p.dh_final ? p.dh_final[s * dn + i] : 0.f;
    }
}

template <typename T, int LN>
cudaError_t sum_t(const SsmParams &p, cudaStream_t st) {
    constexpr int CH = 2 * kNT / LN;
    constexpr int smem = 2 * 4 * kStage * CH * (int)sizeof(T) + kStage * CH / 2 * 24 + 2 * kStage * 2 * 8 * LN * 4;
    const bool usual = p.vec && p.softplus && p.z;
    auto *k = usual ? ssm_bwd_sum_kernel<T, LN, true> : ssm_bwd_sum_kernel<T, LN, false>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    const int ntile = (p.D + CH - 1) / CH;
    const int64_t items = (int64_t)(p.cu ? 1 : p.B) * p.nrun;
    if (items * ntile > INT32_MAX) return cudaErrorInvalidValue;
    k<<<(unsigned)(items * ntile), kNT, smem, st>>>(p, ntile);
    return cudaGetLastError();
}
template <typename T, int Q, int LN>
cudaError_t walk_t(const SsmParams &p, cudaStream_t st) {
    constexpr int CH = kWalk / LN, NP = Q * LN;
    constexpr int smem = 4 * kGroup * CH * (int)sizeof(T) + 2 * kGroup * CH * 4 + 3 * kGroup * 2 * NP * 4 +
                         (kGroup / 4 - 2) * (Q / 4) * kWalk * 16;
    const bool usual = p.vec && p.softplus && p.z && p.dz;
    auto *k = usual ? ssm_bwd_kernel<T, Q, LN, true> : ssm_bwd_kernel<T, Q, LN, false>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int ntile = ssm_bwd_tiles(p.D, p.N);
    const int64_t items = (int64_t)(p.cu ? 1 : p.B) * p.nrun;
    if (items * ntile > INT32_MAX) return cudaErrorInvalidValue;
    k<<<(unsigned)(items * ntile), kWalk, smem, st>>>(p, ntile);
    return cudaGetLastError();
}
// lanes a channel of the walk back: eight states a lane, sixteen above N = 64
int walk_lanes(int N) { return N <= 8 ? 1 : N <= 16 ? 2 : N <= 32 ? 4 : 8; }

}  // namespace

int ssm_bwd_tiles(int D, int N) {
    const int ch = kWalk / walk_lanes(N);
    return (D + ch - 1) / ch;
}
// Tokens a run: 256, less while that leaves under eight CTAs a SM. 4 x 4096
// tokens of 4096 channels: runs of 512 make the walk 1.55 ms for 1.48 (a last
// wave of long CTAs), runs of 128 store and chain twice as many gradients.
int ssm_bwd_run(int lines, int T, int D, int N) {
    int len = 256;
    while (len > kGroup && (int64_t)lines * ssm_bwd_tiles(D, N) * ((T + len - 1) / len) < 1216) len /= 2;
    return len;
}

cudaError_t launch_ssm_bwd_sum(const SsmParams &p, cudaStream_t st) {
    auto f = [&](auto ln) { return p.bf16 ? sum_t<__nv_bfloat16, ln()>(p, st) : sum_t<float, ln()>(p, st); };
    switch (ssm_np(p.N) / 8) {
        case 1: return f(std::integral_constant<int, 1>());
        case 2: return f(std::integral_constant<int, 2>());
        case 4: return f(std::integral_constant<int, 4>());
        case 8: return f(std::integral_constant<int, 8>());
    }
    return f(std::integral_constant<int, 16>());
}
cudaError_t launch_ssm_bwd_chain(const SsmParams &p, cudaStream_t st) {
    const int np = ssm_np(p.N);
    const int64_t n = (int64_t)(p.cu ? 1 : p.B) * p.D * np;
    ssm_bwd_chain_kernel<<<dim3((unsigned)((n + 255) / 256), 2), 256, 0, st>>>(p, np);
    return cudaGetLastError();
}
cudaError_t launch_ssm_bwd(const SsmParams &p, cudaStream_t st) {
    auto f = [&](auto q, auto ln) {
        return p.bf16 ? walk_t<__nv_bfloat16, q(), ln()>(p, st) : walk_t<float, q(), ln()>(p, st);
    };
    using I8 = std::integral_constant<int, 8>;
    if (p.N > 64) return f(std::integral_constant<int, 16>(), I8());
    switch (walk_lanes(p.N)) {
        case 1: return f(I8(), std::integral_constant<int, 1>());
        case 2: return f(I8(), std::integral_constant<int, 2>());
        case 4: return f(I8(), std::integral_constant<int, 4>());
    }
    return f(I8(), I8());
}
cudaError_t launch_ssm_bwd_reduce(const SsmParams &p, cudaStream_t st) {
    const int64_t n = (int64_t)p.B * p.T * 2 * p.N, dn = (int64_t)p.D * p.N;
    if (n / 256 > INT32_MAX / 2) return cudaErrorInvalidValue;
    const unsigned nbc = (unsigned)((n + 255) / 256), nd = (unsigned)((dn + 2 * p.D + 31) / 32);
    const bool empty = p.dh0 && (p.cu || p.T == 0);
    const unsigned ne = empty ? (unsigned)((dn + 255) / 256 < 608 ? (dn + 255) / 256 : 608) : 0;
    const int tiles = ssm_bwd_tiles(p.D, p.N);
    if (p.bf16) ssm_bwd_reduce_kernel<__nv_bfloat16><<<nbc + nd + ne, 256, 0, st>>>(p, tiles, nbc, nd);
    else ssm_bwd_reduce_kernel<float><<<nbc + nd + ne, 256, 0, st>>>(p, tiles, nbc, nd);
    return cudaGetLastError();
}

}  // namespace gdn

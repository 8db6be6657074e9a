// gdn_ssm.cu -- the selective state-space scan. Per channel d and state n,
//   delta = softplus(dt + bias),  a = exp(delta A),
//   h <- a h + delta x B_n,  y = sum_n C_n h + D x,  out = y silu(z),
// for whole sequences (dense or packed) and for single tokens with the
// states in a pool. h is fp32 throughout.
//
// What bounds the scan: a (token, channel, state) costs one exponential and
// four multiply-adds; both pipes take 4 cycles a warp for them (32 ex2 and 128
// fp32 operations a clock and SM, measured), so 16 states of a token and
// channel cost 64 cycles a warp, more than the 8 bytes it moves.
// The main loop is written in packed pairs to leave issue slots for the rest.
// What is left idle is latency: with 10 to 11 warps a SM (164 registers) the
// issue slots are 56 to 61 % used, the exponential unit 42 to 51 %, DRAM 14 to 19.
//
// A line of tokens is one CTA's from end to end while channels alone fill the
// GPU. Where they do not, the line is cut into chunks: a first pass scans the
// first chunk and forms the others' states from zero and sums of delta (the
// decay of a chunk is exp(A sum delta), so it needs no product of its own), a
// short pass chains them, and a second scan runs the chunks from their
// entering states. 4 x 4096 tokens of 4096 channels, 16 states, bf16: 206, 10
// and 270 us (8.6 and 11.2 cycles a warp for 32 (token, channel, state); the
// bare loops take 5.0 and 6.2, the rest is what a token and channel needs
// once: softplus, gate and the conversions). Whole lines: 1018 us (128 CTAs).
#include "gdn_ssm.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 64;  // a CTA: 2 * 64 / LN channels
constexpr int kStage = 8;     // tokens a stage

// The states of two channels as pairs of one state each: v[j] = (channel 0's
// state j, channel 1's).
template <int Q>
__device__ __forceinline__ void ld_across(f32x2 (&v)[Q], const float *p, int ld, int n, bool wide, const bool (&on)[2]) {
    f32x2 a[2][Q / 2];
    ld_pair<Q>(a, p, ld, n, wide, on);
#pragma unroll
    for (int j = 0; j < Q / 2; ++j) {
        const float2 x = unpack2(a[0][j]), y = unpack2(a[1][j]);
        v[2 * j] = pack2(x.x, y.x), v[2 * j + 1] = pack2(x.y, y.y);
    }
}
template <int Q>
__device__ __forceinline__ void st_across(float *p, const f32x2 (&v)[Q], int ld, int n, bool wide, const bool (&on)[2]) {
    f32x2 a[2][Q / 2];
#pragma unroll
    for (int j = 0; j < Q / 2; ++j) {
        const float2 x = unpack2(v[2 * j]), y = unpack2(v[2 * j + 1]);
        a[0][j] = pack2(x.x, y.x), a[1][j] = pack2(x.y, y.y);
    }
    st_pair<Q>(p, a, ld, n, wide, on);
}

// One chunk of a line. A lane has Q states of two neighbouring channels, which
// are the halves of its packed pairs; LN lanes a channel (LN = 1 up to 16
// states, so nothing crosses lanes there). x, dt and z come through two shared-memory buffers, a stage ahead of their use; B and
// C, the same for every channel, are staged as fp32 and read by broadcast, 4
// bytes a (channel, state). A stage has three loops: delta and delta x of its
// tokens (the chain of a softplus is some 150 cycles: four tokens' side by
// side hide it), the states, whose only chain is one multiply-add a token, and
// the outputs; between them a thread's own slots of shared memory. One loop
// that did all three took 0.33 ms where this takes 0.29 for 32768 tokens of
// 2048 channels. USUAL: softplus, a gate and rows for wide accesses, known
// beforehand.
template <typename T, int Q, int LN, bool SUM, bool USUAL>
__device__ __forceinline__ void ssm_walk(const SsmParams &p, int line, int chunk, int tile) {
    constexpr int CH = 2 * kThreads / LN, NP = Q * LN, TS = kStage;
    constexpr int NA = SUM ? 2 : 3;  // x, dt, z
    constexpr int kTile = TS * CH * (int)sizeof(T), kBuf = NA * kTile, kBc = TS * 2 * NP;
    extern __shared__ __align__(16) unsigned char smem[];
    float4 *slot = reinterpret_cast<float4 *>(smem + 2 * kBuf) + threadIdx.x;  // [TS][kThreads], delta, delta x or y
    float *bcs = reinterpret_cast<float *>(smem + 2 * kBuf + TS * kThreads * 16);  // [2][TS][2][NP]
    const int tid = threadIdx.x, ch = tid / LN * 2, ln = tid % LN;
    const int t0 = chunk ? p.clen0 + (chunk - 1) * p.clen : 0, t1 = min(p.T - t0, chunk ? p.clen : p.clen0) + t0;
    const int c0 = tile * CH, d = c0 + ch, n0 = ln * Q, nn = p.N - n0;
    const bool on[2] = {d < p.D && nn > 0, d + 1 < p.D && nn > 0}, out = d < p.D && ln == 0;
    const int64_t hrow = (int64_t)p.D * p.N, dnp = (int64_t)p.D * NP;
    const int64_t own = (int64_t)d * p.N + n0, own_p = (int64_t)d * NP + n0;

    f32x2 a2[Q], h[Q];
    ld_across<Q>(a2, p.A + own, p.N, nn, p.n_wide, on);
#pragma unroll
    for (int j = 0; j < Q; ++j) a2[j] = mul2(a2[j], pack2(kLog2e, kLog2e));
    auto pair_of = [&](const float *v) {
        return make_float2(v && d < p.D ? v[d] : 0.f, v && d + 1 < p.D ? v[d + 1] : 0.f);
    };
    const bool softplus = USUAL || p.softplus, gate = USUAL || p.z, vec = USUAL || p.vec;
    const float2 bias = pair_of(p.dt_bias), dv = pair_of(SUM ? nullptr : p.Dv);
    auto zero_h = [&] {
#pragma unroll
        for (int j = 0; j < Q; ++j) h[j] = pack2(0.f, 0.f);
    };
    auto first_h = [&](int seg) {
        if (p.h0) ld_across<Q>(h, p.h0 + seg * hrow + own, p.N, nn, p.n_wide, on);
        else zero_h();
    };
    SsmSeq q{0, 0, false};
    if (t0 < t1) q = ssm_find(p.cu, p.n_seq, p.T, line, t0);
    bool reset = q.starts;
    if (q.starts) first_h(q.seg);
    else if (!SUM && chunk > 0) ld_across<Q>(h, p.sums + ((int64_t)line * (p.nchunk - 1) + chunk - 1) * dnp + own_p, NP, Q, true, on);
    else zero_h();

    const T *src[3] = {(const T *)p.x + line * p.x_sb, (const T *)p.dt + line * p.dt_sb, (const T *)p.z + line * p.z_sb};
    const int64_t str[3] = {p.x_st, p.dt_st, p.z_st};
    // The stage that begins at token s into buffer b: by asynchronous copies two
    // stages ahead, or through registers one stage ahead.
    auto tile_at = [&](int b, int a) { return reinterpret_cast<T *>(smem + b * kBuf + a * kTile); };
    auto copy = [&](int s, int b) {
        if (s < t1) {
#pragma unroll
            for (int a = 0; a < NA; ++a)
                if (a < 2 || gate)
                    ssm_copy_tile<T, CH, TS, kThreads>(tile_at(b, a), src[a] + s * str[a], str[a], t1 - s, c0, p.D);
        }
        cp_async_commit();
    };
    SsmTile<T, CH, TS, kThreads> held[USUAL ? 1 : NA];
    auto hold = [&](int s) {
#pragma unroll
        for (int a = 0; a < (USUAL ? 0 : NA); ++a)
            if (a < 2 || gate) held[a].load(src[a] + s * str[a], str[a], t1 - s, c0, p.D);
    };
    auto release = [&](int b) {
#pragma unroll
        for (int a = 0; a < (USUAL ? 0 : NA); ++a)
            if (a < 2 || gate) held[a].store(tile_at(b, a));
    };
    const T *bg = (const T *)p.bm + line * p.bm_sb, *cg = (const T *)p.cm + line * p.cm_sb;
    SsmBc<T, NP, TS, kThreads> nbc;
    auto fetch_bc = [&](int s) {
        nbc.template fetch<!SUM>(bg + s * p.bm_st, p.bm_st, cg + s * p.cm_st, p.cm_st, t1 - s, p.N, p.bc_vec);
    };
    if (t0 < t1) {
        if (vec) {
            copy(t0, 0);
            copy(t0 + TS, 1);
        } else {
            hold(t0);
            release(0);
        }
        fetch_bc(t0);
    }
    f32x2 dsum = pack2(0.f, 0.f);
    int buf = 0;
    for (int s = t0; s < t1; s += TS, buf ^= 1) {
        float *bc = bcs + buf * kBc;
        nbc.stage(bc);
        if (s + TS < t1) fetch_bc(s + TS);
        if (vec) cp_async_wait<1>();
        else if (s + TS < t1) hold(s + TS);
        __syncthreads();
        const int m = min(t1 - s, TS);
        const T *xs = reinterpret_cast<const T *>(smem + buf * kBuf) + ch;
        auto pair_at = [&](int i, int a) {  // the pair's x, dt or z
            float f[2];
            ld_row_f<T, 2, true>(f, xs + (a * TS + i) * CH, 2);
            return make_float2(f[0], f[1]);
        };
#pragma unroll 4
        for (int t = 0; t < TS; ++t) {
            const float2 v = pair_at(t, 1), x = pair_at(t, 0);
            float2 dl = make_float2(v.x + bias.x, v.y + bias.y);
            if (softplus) dl = softplus2(dl);
            slot[t * kThreads] = make_float4(dl.x, dl.y, dl.x * x.x, dl.y * x.y);
        }
        auto states = [&](int i) {
            const ulonglong2 du = *reinterpret_cast<const ulonglong2 *>(slot + i * kThreads);
            const float4 *b4 = reinterpret_cast<const float4 *>(bc + i * 2 * NP + n0);
            f32x2 ya, yb;
#pragma unroll
            for (int j = 0; j < Q / 4; ++j) {
                const float4 b = b4[j];
                const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    h[4 * j + k] = fma2(ex2_2(mul2(du.x, a2[4 * j + k])), h[4 * j + k], mul2(du.y, pack2(bv[k], bv[k])));
                if (!SUM) {
                    const float4 c = b4[NP / 4 + j];
                    ya = j ? fma2(h[4 * j], pack2(c.x, c.x), ya) : mul2(h[0], pack2(c.x, c.x));
                    yb = j ? fma2(h[4 * j + 1], pack2(c.y, c.y), yb) : mul2(h[1], pack2(c.y, c.y));
                    ya = fma2(h[4 * j + 2], pack2(c.z, c.z), ya);
                    yb = fma2(h[4 * j + 3], pack2(c.w, c.w), yb);
                }
            }
            if (SUM) dsum = add2(dsum, du.x);
            else *reinterpret_cast<f32x2 *>(slot + i * kThreads) = add2(ya, yb);
        };
        if (m == TS && q.end > s + TS) {  // no sequence ends in the stage
#pragma unroll 4
            for (int t = 0; t < TS; ++t) states(t);
        } else {
#pragma unroll 1
            for (int t = 0; t < m; ++t) {
                states(t);
                if (s + t + 1 == q.end) {
                    if (!SUM && p.h_final) st_across<Q>(p.h_final + q.seg * hrow + own, h, p.N, nn, p.n_wide, on);
                    if (q.end < p.T) {
                        ssm_next(q, p.cu, p.n_seq, p.T, q.end);
                        first_h(q.seg);
                        if (s + t + 1 < t1) reset = true;
                    }
                }
            }
        }
        if (!SUM) {
            T *os = (T *)p.out + line * p.o_sb + s * p.o_st + d;
#pragma unroll 4
            for (int t = 0; t < TS; ++t, os += p.o_st) {
                float2 y = *reinterpret_cast<const float2 *>(slot + t * kThreads);
#pragma unroll
                for (int o = LN / 2; o > 0; o >>= 1) {
                    y.x += __shfl_xor_sync(0xffffffffu, y.x, o);
                    y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
                }
                const float2 x = pair_at(t, 0);
                float f[2] = {fmaf(dv.x, x.x, y.x), fmaf(dv.y, x.y, y.y)};
                if (gate) {
                    const float2 z = pair_at(t, 2), g = sigmoid2(z);
                    f[0] *= z.x * g.x, f[1] *= z.y * g.y;
                }
                if (out && t < m) {
                    if (vec) st_row_f<T, 2, true>(os, f, 2);
                    else st_row_f<T, 2, false>(os, f, p.D - d);
                }
            }
        }
        __syncthreads();  // the buffer has been read
        if (vec) copy(s + 2 * TS, buf);
        else if (s + TS < t1) release(buf ^ 1);
    }
    if (SUM || (chunk == 0 && p.nchunk > 1)) {
        const int64_t at = (int64_t)line * (p.nchunk - 1) + chunk;
        st_across<Q>(p.sums + at * dnp + own_p, h, NP, Q, true, on);
        // a chunk in which a sequence begins passes nothing on: marked by NaN
        const float2 ds = unpack2(dsum);
        float *o = p.dsum + at * p.D + d;
        if (ln == 0 && d < p.D) o[0] = reset ? __int_as_float(0x7fffffff) : ds.x;
        if (ln == 0 && d + 1 < p.D) o[1] = reset ? __int_as_float(0x7fffffff) : ds.y;
    }
    if (!SUM && p.h_final && chunk == 0 && (p.cu || p.T == 0)) {
        // sequences without a token pass their state on
        for (int s = 0; s < p.n_seq; ++s) {
            if (p.cu ? p.cu[s + 1] > p.cu[s] : s != line) continue;
            first_h(s);
            st_across<Q>(p.h_final + s * hrow + own, h, p.N, nn, p.n_wide, on);
        }
    }
}

// Every chunk but the first, or whole lines. Six CTAs a SM: eight have to do
// with 128 registers and took 0.31 ms for 0.30.
template <typename T, int Q, int LN, bool USUAL>
__global__ void __launch_bounds__(kThreads, 6) ssm_scan_kernel(const SsmParams p, int ntile) {
    if (p.err && blockIdx.x == 0) ssm_check_cu(p.cu, p.n_seq, p.T, p.err);
    const int item = blockIdx.x / ntile, nch = max(p.nchunk - 1, 1), line = item / nch;
    ssm_walk<T, Q, LN, false, USUAL>(p, line, item - line * nch + (p.nchunk > 1), blockIdx.x % ntile);
}
// The first launch over a line in chunks: the first chunk's scan, whose state
// is its sum, beside the sums of the others but the last.
template <typename T, int Q, int LN, bool USUAL>
__global__ void __launch_bounds__(kThreads, 6) ssm_sum_kernel(const SsmParams p, int ntile) {
    const int item = blockIdx.x / ntile, nch = p.nchunk - 1, line = item / nch, chunk = item - line * nch;
    if (chunk > 0) return ssm_walk<T, Q, LN, true, USUAL>(p, line, chunk, blockIdx.x % ntile);
    ssm_walk<T, Q, LN, false, USUAL>(p, line, 0, blockIdx.x % ntile);
}

// The state entering chunk c + 1 replaces chunk c's sum: h <- exp(A sum
// delta) h + S. One thread a (line, channel, state).
__global__ void __launch_bounds__(256) ssm_chain_kernel(const SsmParams p, int np) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, dnp = (int64_t)p.D * np;
    const int lines = p.cu ? 1 : p.B, nch = p.nchunk - 1;
    if (i >= lines * dnp) return;
    const int line = (int)(i / dnp), d = (int)(i % dnp / np), n = (int)(i % np);
    const float a = n < p.N ? p.A[(int64_t)d * p.N + n] * kLog2e : 0.f;
    float *s = p.sums + line * nch * dnp + i % dnp;
    const float *q = p.dsum + (int64_t)line * nch * p.D + d;
    float h = 0.f;
    for (int c = 0; c < nch; c += 8) {
        float v[8], e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const bool in = c + k < nch;
            v[k] = in ? q[(int64_t)(c + k) * p.D] : 0.f, e[k] = in ? s[(c + k) * dnp] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            h = isnan(v[k]) || h == 0.f ? e[k] : fmaf(ex2f(a * v[k]), h, e[k]);  // (A > 0 may overflow)
            if (c + k < nch) s[(c + k) * dnp] = h;
        }
    }
}

// One token of each request: the state is read, updated and written back, all
// that counts. LN lanes a channel with four states each, four channels a lane
// (8 states' loads under way); of a lane's four channels lane ln forms delta
// and the gate of channel ln % 4 and finishes it. Channel 8 k + lc of the
// warp's is a lane's k-th where LN = 4, so that every access runs over
// neighbouring channels. 256 requests of 4096 channels, 16 states: 26.5 us for
// 142 MB (79% of the measured copy rate; with one channel a lane 41 us); one
// request is bound by the launch.
template <typename T, int LN>
__global__ void __launch_bounds__(128) ssm_step_kernel(const SsmStepParams p) {
    constexpr int CL = 32 / LN, CW = 4 * CL;
    const int i = blockIdx.y, lane = threadIdx.x & 31, ln = lane % LN, lc = lane / LN, n0 = ln * 4;
    const int64_t slot = p.slots ? p.slots[i] : i;
    const int c0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * CW + lc, dm = c0 + (ln & 3) * CL;
    T *out = (T *)p.out + i * p.o_st;
    if (slot < 0 || slot >= p.n_slots) {  // a padding row
        if (ln < 4 && dm < p.D) out[dm] = to_type<T>(0.f);
        return;
    }
    float *state = p.state + slot * p.D * p.N;
    float h[4][4], a[4][4], b[4], c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int d = c0 + k * CL;
        const bool on = d < p.D && n0 < p.N;
        const int64_t own = (int64_t)d * p.N + n0;
        if (p.n_wide) {
            const float4 u = on ? *reinterpret_cast<const float4 *>(state + own) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 v = on ? __ldg(reinterpret_cast<const float4 *>(p.A + own)) : make_float4(0.f, 0.f, 0.f, 0.f);
            h[k][0] = u.x, h[k][1] = u.y, h[k][2] = u.z, h[k][3] = u.w;
            a[k][0] = v.x, a[k][1] = v.y, a[k][2] = v.z, a[k][3] = v.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[k][j] = on && n0 + j < p.N ? state[own + j] : 0.f;
                a[k][j] = on && n0 + j < p.N ? p.A[own + j] : 0.f;
            }
        }
    }
    const T *bm = (const T *)p.bm + i * p.bm_st + n0, *cm = (const T *)p.cm + i * p.cm_st + n0;
    if (p.bc_vec && n0 < p.N) {
        ld_row_f<T, 4, true>(b, bm, 4);
        ld_row_f<T, 4, true>(c, cm, 4);
    } else {
        ld_row_f<T, 4, false>(b, bm, p.N - n0);
        ld_row_f<T, 4, false>(c, cm, p.N - n0);
    }
    float x = 0.f, dl = 0.f, z = 0.f, dv = 0.f;
    if (dm < p.D) {
        x = ldf((const T *)p.x + i * p.x_st + dm);
        dl = ldf((const T *)p.dt + i * p.dt_st + dm);
        if (p.z) z = ldf((const T *)p.z + i * p.z_st + dm);
        if (p.dt_bias) dl += p.dt_bias[dm];
        if (p.Dv) dv = p.Dv[dm];
    }
    if (p.softplus) dl = softplus2(make_float2(dl, dl)).x;
    const float u = dl * x, dk = dl * kLog2e;
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int from = lane - (ln & 3) + k;  // the lane of this group of four that has channel k
        const float dks = __shfl_sync(0xffffffffu, dk, from), us = __shfl_sync(0xffffffffu, u, from);
        y[k] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[k][j] = fmaf(ex2f(dks * a[k][j]), h[k][j], us * b[j]);
            y[k] = fmaf(h[k][j], c[j], y[k]);
        }
        const int d = c0 + k * CL;
        const int64_t own = (int64_t)d * p.N + n0;
        if (d < p.D && n0 < p.N) {
            if (p.n_wide) {
                *reinterpret_cast<float4 *>(state + own) = make_float4(h[k][0], h[k][1], h[k][2], h[k][3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n0 + j < p.N) state[own + j] = h[k][j];
            }
        }
    }
    // the four sums over the lanes of a channel, one to each of four lanes
#pragma unroll
    for (int o = LN / 2; o >= 4; o >>= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] += __shfl_xor_sync(0xffffffffu, y[k], o);
    const bool l1 = ln & 1, l2 = ln & 2;
    const float g0 = l2 ? y[0] : y[2], g1 = l2 ? y[1] : y[3];
    float k0 = l2 ? y[2] : y[0], k1 = l2 ? y[3] : y[1];
    k0 += __shfl_xor_sync(0xffffffffu, g0, 2), k1 += __shfl_xor_sync(0xffffffffu, g1, 2);
    const float g2 = l1 ? k0 : k1;
    float r = (l1 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, g2, 1);
    r = fmaf(dv, x, r);
    if (p.z) r *= z * rcpf(1.f + ex2f(z * -kLog2e));
    if (ln < 4 && dm < p.D) out[dm] = to_type<T>(r);
}

template <typename T, int Q, int LN, bool SUM>
cudaError_t scan_t(const SsmParams &p, cudaStream_t st) {
    constexpr int CH = 2 * kThreads / LN;
    constexpr int smem = 2 * 3 * kStage * CH * (int)sizeof(T) + kStage * kThreads * 16 + 2 * kStage * 2 * Q * LN * 4;
    const bool usual = p.vec && p.softplus && p.z;
    auto *k = SUM ? (usual ? ssm_sum_kernel<T, Q, LN, true> : ssm_sum_kernel<T, Q, LN, false>)
                  : (usual ? ssm_scan_kernel<T, Q, LN, true> : ssm_scan_kernel<T, Q, LN, false>);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    const int ntile = (p.D + CH - 1) / CH;
    const int64_t items = (int64_t)(p.cu ? 1 : p.B) * (p.nchunk > 1 ? p.nchunk - 1 : 1);
    if (items * ntile > INT32_MAX) return cudaErrorInvalidValue;
    k<<<(unsigned)(items * ntile), kThreads, smem, st>>>(p, ntile);
    return cudaGetLastError();
}

// lanes a channel at four states a lane
template <class F>
cudaError_t by_lanes(int N, F &&f) {
    if (N <= 16) return f(std::integral_constant<int, 4>());
    if (N <= 32) return f(std::integral_constant<int, 8>());
    if (N <= 64) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

}  // namespace

// Chunks of a line, by the number of CTAs that whole lines give.
void ssm_split(int lines, int T, int D, int N, int *nchunk, int *clen0, int *clen) {
    const int ch = 2 * kThreads / ssm_lanes(N);
    const int64_t ctas = (int64_t)lines * ((D + ch - 1) / ch);
    // Each launch takes n chunks of a line, with six CTAs a SM (three warps a
    // scheduler), one chunk more than n of at least 64 tokens to a line (so 48
    // and 40 for the shortest cut line, 129 tokens); whole lines where n would be
    // one. 4096 channels: 10 x 3000 tokens (320 CTAs) 1067 us whole, 969 cut;
    // 16 x 2048 (512 CTAs) 736 whole.
    int64_t n = 912 / ctas;
    if (n > (T + 63) / 64 - 1) n = (T + 63) / 64 - 1;
    if (n < 2) {
        *clen0 = *clen = T > 0 ? T : 1, *nchunk = 1;
        return;
    }
    // a token's scan takes 1.3 times its sum: so much shorter is the first chunk
    auto stages = [](int64_t v) { return (int)((v + kStage - 1) / kStage * kStage); };
    *clen = stages((int64_t)T * 4 / (4 * n + 3));
    *clen0 = stages((int64_t)*clen * 3 / 4);
    *nchunk = 1 + (int)(((int64_t)T - *clen0 + *clen - 1) / *clen);
}

cudaError_t launch_ssm_sum(const SsmParams &p, cudaStream_t st) {
    return ssm_by_states(p.N, [&](auto q, auto ln) {
        return p.bf16 ? scan_t<__nv_bfloat16, q(), ln(), true>(p, st) : scan_t<float, q(), ln(), true>(p, st);
    });
}
cudaError_t launch_ssm_chain(const SsmParams &p, cudaStream_t st) {
    const int np = ssm_np(p.N);
    const int64_t n = (int64_t)(p.cu ? 1 : p.B) * p.D * np;
    ssm_chain_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(p, np);
    return cudaGetLastError();
}
cudaError_t launch_ssm_scan(const SsmParams &p, cudaStream_t st) {
    return ssm_by_states(p.N, [&](auto q, auto ln) {
        return p.bf16 ? scan_t<__nv_bfloat16, q(), ln(), false>(p, st) : scan_t<float, q(), ln(), false>(p, st);
    });
}
cudaError_t launch_ssm_step(const SsmStepParams &p, cudaStream_t st) {
    return by_lanes(p.N, [&](auto ln) {
        const int cw = 4 * (32 / ln()) * 4;  // channels a CTA
        const dim3 grid((p.D + cw - 1) / cw, p.n);
        if (p.bf16) ssm_step_kernel<__nv_bfloat16, ln()><<<grid, 128, 0, st>>>(p);
        else ssm_step_kernel<float, ln()><<<grid, 128, 0, st>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace gdn

// gdn_layer.cuh -- the state-space layer's operators beside the scan of the
// gated delta rule: residual RMS norm (gdn_norm.cu), short causal
// convolution (gdn_conv.cu), selective scan (gdn_ssm.cu, gdn_ssm_bwd.cu).
// Launch parameter blocks and the row-vector accesses they share. All
// strides are in elements.
#pragma once

#include "gdn_common.cuh"

namespace gdn {

// ------------------------------------------------------ row vectors ---------
// N consecutive channels of a row as fp32. VEC: the row starts on a boundary
// of the vector's size and n >= N holds for every full vector, so one wide
// access; otherwise element accesses, of which only the first n are made
// (rows of any length and alignment).
template <typename T, int N>
struct RowVec {  // in 32-bit words
    static constexpr int kBytes = N * (int)sizeof(T);
    static constexpr int kWords = kBytes / 4;
    static_assert(kBytes == 4 || kBytes == 8 || kBytes % 16 == 0, "vector size");
};
template <int WORDS>
__device__ __forceinline__ void ld_words(uint32_t (&w)[WORDS], const void *p) {
    if constexpr (WORDS == 1) {
        w[0] = *static_cast<const uint32_t *>(p);
    } else if constexpr (WORDS == 2) {
        const uint2 u = *static_cast<const uint2 *>(p);
        w[0] = u.x, w[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) {
            const uint4 u = static_cast<const uint4 *>(p)[i];
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
    }
}
template <int WORDS>
__device__ __forceinline__ void st_words(void *p, const uint32_t (&w)[WORDS]) {
    if constexpr (WORDS == 1) {
        *static_cast<uint32_t *>(p) = w[0];
    } else if constexpr (WORDS == 2) {
        *static_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i)
            static_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}
// Asynchronous copies that only the issuing thread waits for and reads
// (ordered against its other accesses, hence the clobbers).
template <int BYTES>
__device__ __forceinline__ void copy_async(void *smem, const void *gmem) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(smem_u32(smem)), "l"(gmem), "n"(BYTES) : "memory");
}
template <int LEFT>  // all but the last LEFT groups
__device__ __forceinline__ void copies_arrived() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(LEFT) : "memory");
}
template <typename T>
__device__ __forceinline__ T to_type(float x);
template <>
__device__ __forceinline__ float to_type<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_type<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// words of a vector to fp32
template <typename T, int N>
__device__ __forceinline__ void words_to_f(float (&f)[N], const uint32_t (&w)[RowVec<T, N>::kWords]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <typename T, int N>
__device__ __forceinline__ void f_to_words(uint32_t (&w)[RowVec<T, N>::kWords], const float (&f)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    }
}
// Whole vectors of 16-bit elements that start on any element: words where the
// address allows, else an element, N / 2 - 1 words and an element.
template <int N>
__device__ __forceinline__ void ld_half_row(uint32_t (&w)[N / 2], const unsigned short *e) {
    if ((reinterpret_cast<uintptr_t>(e) & 3) == 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = reinterpret_cast<const uint32_t *>(e)[i];
    } else {
        uint32_t m[N / 2 + 1];
        m[0] = (uint32_t)e[0] << 16;
#pragma unroll
        for (int i = 0; i < N / 2 - 1; ++i) m[i + 1] = reinterpret_cast<const uint32_t *>(e + 1)[i];
        m[N / 2] = e[N - 1];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = __funnelshift_l(m[i], m[i + 1], 16);
    }
}
template <int N>
__device__ __forceinline__ void st_half_row(unsigned short *e, const uint32_t (&w)[N / 2]) {
    if ((reinterpret_cast<uintptr_t>(e) & 3) == 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) reinterpret_cast<uint32_t *>(e)[i] = w[i];
    } else {
        e[0] = (unsigned short)w[0];
#pragma unroll
        for (int i = 0; i < N / 2 - 1; ++i) reinterpret_cast<uint32_t *>(e + 1)[i] = __funnelshift_l(w[i], w[i + 1], 16);
        e[N - 1] = (unsigned short)(w[N / 2 - 1] >> 16);
    }
}
// raw load: zeros past n in the element form
template <typename T, int N, bool VEC>
__device__ __forceinline__ void ld_row(uint32_t (&w)[RowVec<T, N>::kWords], const T *p, int n) {
    if constexpr (VEC) {
        ld_words(w, p);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = i < n ? __float_as_uint(static_cast<const float *>(p)[i]) : 0u;
    } else {
        const unsigned short *e = reinterpret_cast<const unsigned short *>(p);
        if (n >= N) {
            ld_half_row<N>(w, e);
            return;
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = 0u;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) w[i >> 1] |= (uint32_t)e[i] << (16 * (i & 1));
    }
}
template <typename T, int N, bool VEC>
__device__ __forceinline__ void ld_row_f(float (&f)[N], const T *p, int n) {
    uint32_t w[RowVec<T, N>::kWords];
    ld_row<T, N, VEC>(w, p, n);
    words_to_f<T, N>(f, w);
}
template <typename T, int N, bool VEC>
__device__ __forceinline__ void st_row(T *p, const uint32_t (&w)[RowVec<T, N>::kWords], int n) {
    if constexpr (VEC) {
        st_words(p, w);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) reinterpret_cast<uint32_t *>(p)[i] = w[i];
    } else {
        unsigned short *e = reinterpret_cast<unsigned short *>(p);
        if (n >= N) {
            st_half_row<N>(e, w);
            return;
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) e[i] = (unsigned short)(w[i >> 1] >> (16 * (i & 1)));
    }
}
template <typename T, int N, bool VEC>
__device__ __forceinline__ void st_row_f(T *p, const float (&f)[N], int n) {
    uint32_t w[RowVec<T, N>::kWords];
    f_to_words<T, N>(w, f);
    st_row<T, N, VEC>(p, w, n);
}

// ------------------------------------------------------------- norm ---------
constexpr int kNormMaxD = 16384;
struct NormParams {
    const void *x, *res;  // (R, D); res or null
    int64_t x_st, res_st;
    int x_bf16, res_bf16;
    const float *weight;  // (D)
    void *out, *res_out;  // out: x's type, or e4m3 with scale
    int64_t o_st, ro_st;
    float *scale;         // (R, groups) or null: out in x's type
    int R, D, group;      // group: channels a scale, 0: the row
    float eps;
    int vec;              // every row is 16-byte aligned (8 for the e4m3 output)
};
cudaError_t launch_rmsnorm(const NormParams &p, cudaStream_t st);
struct NormBwdParams {
    const void *s, *dy, *dres;  // (R, D); dres (s's type) or null
    int64_t s_st, dy_st, dr_st;
    int s_bf16, dy_bf16;
    const float *weight;
    void *dx;  // s's type
    int64_t dx_st;
    float *part;  // workspace: partial sums of dweight, (norm_bwd_parts, D)
    float *dweight;
    int R, D;
    float eps;
    int vec;
};
int norm_bwd_parts(int R, int D);
cudaError_t launch_rmsnorm_bwd(const NormBwdParams &p, cudaStream_t st);
// out[c] = sum over p < parts of in[p * ld + c], c < n, in a fixed order;
// columns n .. n + n2 - 1 go to out2
cudaError_t launch_col_sum(const float *in, int64_t ld, int parts, int64_t n, float *out, int64_t n2, float *out2,
                           cudaStream_t st);

// ----------------------------------------------------- convolution ----------
constexpr int kConvMaxW = 8;
struct ConvParams {
    const void *x;  // (B, T, D)
    int64_t x_sb, x_st;
    const float *weight, *bias;  // (D, W); (D) or null
    const void *init;            // (n_seq, W - 1, D) or null
    const int32_t *cu;           // (n_seq + 1) or null
    int n_seq;
    void *out;
    int64_t o_sb, o_st;
    void *final_state;  // (n_seq, W - 1, D) or null
    // gradient
    const void *dout, *dfinal;
    int64_t do_sb, do_st;
    void *dx, *dinit;  // (B, T, D) contiguous; (n_seq, W - 1, D)
    float *part;       // workspace: partial sums of dweight and dbias
    float *dweight, *dbias;
    int B, T, D, W, silu, bf16, vec;
    int *err;  // device error word or null
};
int conv_bwd_run(int B, int T, int D);
int conv_bwd_parts(int B, int T, int run);
cudaError_t launch_conv(const ConvParams &p, cudaStream_t st);
cudaError_t launch_conv_bwd(const ConvParams &p, cudaStream_t st);
struct ConvStepParams {
    const void *x;  // (n, D)
    int64_t x_st;
    const float *weight, *bias;
    void *state;           // (n_slots, W - 1, D)
    const int32_t *slots;  // (n) or null
    void *out;
    int64_t o_st;
    int n, n_slots, D, W, silu, bf16, vec;
};
cudaError_t launch_conv_step(const ConvStepParams &p, cudaStream_t st);

// ------------------------------------------------------ selective scan ------
constexpr int kSsmMaxN = 128;
constexpr int kSsmGroup = 32;  // the gradient keeps the state entering every group of so many tokens
struct SsmParams {
    const void *x, *dt, *bm, *cm, *z;  // (B, T, D); bm, cm (B, T, N); z or null
    int64_t x_sb, x_st, dt_sb, dt_st, bm_sb, bm_st, cm_sb, cm_st, z_sb, z_st;
    const float *A, *Dv, *dt_bias;  // (D, N); (D) or null
    const float *h0;                // (n_seq, D, N) or null
    const int32_t *cu;              // (n_seq + 1) or null
    int n_seq;
    void *out;
    int64_t o_sb, o_st;
    float *h_final;  // (n_seq, D, N) or null
    int B, T, D, N, softplus, bf16;
    int vec;             // rows of x, dt, z, out (and the gradients) are 16-byte aligned
    int n_wide;          // rows of A and of the states are
    int bc_vec;          // rows of B and C are, in whole vectors of four
    int nchunk, clen0, clen;  // chunks of a line, tokens of the first and of the others
    float *sums, *dsum;  // workspace: (lines, nchunk - 1, D, padded N), (lines, nchunk - 1, D)
    int *err;
    // gradient; activations' gradients contiguous in x's type
    const void *dout;
    int64_t do_sb, do_st;
    const float *dh_final;
    void *dx, *ddt, *dbm, *dcm, *dz;
    float *dA, *dD, *ddt_bias, *dh0;
    // runs of a line, tokens a run, groups of a line; workspace: sums and dsum
    // by group, the sums of delta by run (gsum), the runs' gradients (lines,
    // nrun, D, padded N), partial sums by channel tile and by run
    int nrun, rlen, ngroup;
    float *gsum, *gs, *part_bc, *part_a, *part_d;
};
void ssm_split(int lines, int T, int D, int N, int *nchunk, int *clen0, int *clen);
cudaError_t launch_ssm_sum(const SsmParams &p, cudaStream_t st);
cudaError_t launch_ssm_chain(const SsmParams &p, cudaStream_t st);
cudaError_t launch_ssm_scan(const SsmParams &p, cudaStream_t st);
int ssm_bwd_tiles(int D, int N);
int ssm_bwd_run(int lines, int T, int D, int N);
cudaError_t launch_ssm_bwd_sum(const SsmParams &p, cudaStream_t st);
cudaError_t launch_ssm_bwd_chain(const SsmParams &p, cudaStream_t st);
cudaError_t launch_ssm_bwd(const SsmParams &p, cudaStream_t st);
cudaError_t launch_ssm_bwd_reduce(const SsmParams &p, cudaStream_t st);
struct SsmStepParams {
    const void *x, *dt, *bm, *cm, *z;  // (n, D); bm, cm (n, N); z or null
    int64_t x_st, dt_st, bm_st, cm_st, z_st;
    const float *A, *Dv, *dt_bias;
    float *state;          // (n_slots, D, N)
    const int32_t *slots;  // (n) or null
    void *out;
    int64_t o_st;
    int n, n_slots, D, N, softplus, bf16;
    int n_wide;  // rows of A and of the states are 16-byte aligned
    int bc_vec;  // rows of B and C are, in whole vectors of four
};
cudaError_t launch_ssm_step(const SsmStepParams &p, cudaStream_t st);

}  // namespace gdn

// gdn_block.cuh -- the operators around a mixer and the recurrence that can
// stand in its place: rotary positions (gdn_rotary.cu), the norms behind and
// in front of a block with its gate and residual scale (gdn_block_norm.cu),
// the gated linear recurrence (gdn_lru.cu, gdn_lru_bwd.cu). Launch parameter
// blocks. All strides are in elements.
#pragma once

#include "gdn_layer.cuh"

namespace gdn {

// ----------------------------------------------------------- rotary ---------
constexpr int kRotaryMaxD = 512;
struct RotaryTensor {
    const void *in;  // (B, T, H, D)
    void *out;
    int64_t in_sb, in_st, in_sh, out_sb, out_st, out_sh;
    int H;
    int copy;  // the channels past rot are copied (out is not in)
};
struct RotaryParams {
    RotaryTensor x[2];       // q, and k or no heads
    const double *inv_freq;  // (rot / 2), radians a position
    const void *pos;         // (B, T) int32 or int64, or null: offset + t
    int64_t p_sb, p_st, offset;
    int B, T, D, rot, pos64, interleaved, bf16;
    float scale, sign;
    int vec;  // rows and their turning parts are whole 16-byte vectors
};
cudaError_t launch_rotary(const RotaryParams &p, cudaStream_t st);

// ------------------------------------------------------- block norm ---------
enum { kGateNone = 0, kGateLinear, kGateSigmoid, kGateSilu };
struct BlockNormParams {
    const void *y, *res, *gate;  // (R, D); gate (R / gate_rows, D) or null
    int64_t y_st, r_st, g_st;
    const float *post, *pre, *scale;  // (D) or null
    void *res_out, *out;              // out: y's type, with pre only
    int64_t ro_st, o_st;
    int R, D, gate_rows, act;  // gate_rows: rows that share one of the gate
    int y_bf16, r_bf16;
    int shared;     // gate_rows > 1 rows share one of the gate: runs keep to one sequence
    int runs, run;  // of a sequence's rows (of all rows, where nothing is shared): set by the launch
    float alpha, eps;
    int vec;
};
cudaError_t launch_block_norm(const BlockNormParams &p, cudaStream_t st);
struct BlockNormBwdParams {
    const void *y, *s, *gate, *dout, *dres;  // s, dres (or null): the stream's type
    int64_t y_st, s_st, g_st, do_st, dr_st;
    const float *post, *pre, *scale;
    void *dy, *ds, *dgate;  // dgate: (R, D), or (R / gate_rows, D)
    int64_t dy_st, ds_st, dg_st;
    float *dpost, *dpre, *dscale;
    float *part, *part2;  // workspace: sums by run of rows (parts, 2, D), by sequence (sequences, 2, D)
    int R, D, gate_rows, act, y_bf16, r_bf16;
    int shared, runs, run;
    float alpha, eps;
    int vec;
};
int64_t block_norm_parts(int R, int D, int gate_rows);  // most rows of partial sums
cudaError_t launch_block_norm_bwd(const BlockNormBwdParams &p, cudaStream_t st);
bool block_norm_by_sequence(const BlockNormBwdParams &p);  // needs the launch below before the last
cudaError_t launch_block_norm_sequences(const BlockNormBwdParams &p, cudaStream_t st);
cudaError_t launch_block_norm_reduce(const BlockNormBwdParams &p, cudaStream_t st);

// ------------------------------------------------ gated recurrence ----------
constexpr int kLruTile = 64;  // tokens a saved state stands for
struct LruParams {
    const void *x, *r, *i, *z;  // (B, T, C); z or null
    int64_t x_sb, x_st, r_sb, r_st, i_sb, i_st, z_sb, z_st;
    const float *lam;  // (C)
    float c;
    const float *h0;    // (n_seq, C) or null
    const int32_t *cu;  // (n_seq + 1) or null
    int n_seq;
    void *out;  // or null: the states alone
    int64_t o_sb, o_st;
    float *h_final;  // (n_seq, C) or null
    float *ck;       // (B, ceil(T / 64), C) or null: the states entering the tiles
    int B, T, C, bf16;
    int how;    // rows of all activations lie on 16 bytes (0), on words in pairs (1) or anywhere (2)
    int ranks;  // CTAs of a cluster, which take a line's tiles in turn
    int warps;  // of a CTA (the forward over wide rows): 4 or 8
    int *err;   // or null: the call's error word
    int first;  // the call's first kernel: it clears the word and checks cu
    int wait_us, stall_cta;  // limit of a wait; testing aid: a CTA whose waits run out (-1: none)
    // gradient; activations' gradients contiguous in x's type
    const void *dout;
    int64_t do_sb, do_st;
    const float *dh_final;
    void *dx, *dr, *di, *dz;
    float *part;  // workspace: partial sums of dlam, (B ranks, C)
    float *dlam, *dh0;
};
struct LruShape {
    int ranks, warps;
};
LruShape lru_shape(int lines, int T, int C, bool bf16, bool wide);
int lru_bwd_ranks(int lines, int T, int C);
// p.ranks may come back smaller: as many as fit
cudaError_t launch_lru(LruParams &p, cudaStream_t st);
cudaError_t launch_lru_bwd(LruParams &p, cudaStream_t st);
void set_lru_cluster(int most);
struct LruStepParams {
    const void *x, *r, *i, *z;  // (n, C); z or null
    int64_t x_st, r_st, i_st, z_st;
    const float *lam;
    float c;
    float *state;          // (n_slots, C)
    const int32_t *slots;  // (n) or null
    void *out;
    int64_t o_st;
    int n, n_slots, C, bf16, vec;
};
cudaError_t launch_lru_step(const LruStepParams &p, cudaStream_t st);

}  // namespace gdn

// Host-side launchers of the operators around the layer in a training step
// (internal to libtwell.so): 8-bit activation checkpoints and the backward pass
// from one, the token embedding, log probabilities, the norms around the layer.
// Every launcher only enqueues on `s` and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace twell {

// 8-bit activation checkpoints: int8 codes [n_rows][act8_pitch(d)] and one
// float32 scale per row and block of kAct8Block columns.
constexpr int kAct8Block = 128;
inline int act8_blocks(int d) { return (d - 1) / kAct8Block + 1; }
inline int act8_pitch(int d) { return ((d - 1) / 16 + 1) * 16; }
hipError_t launch_act8_pack(int64_t n_rows, int d, int elem_bytes, const void* x, int8_t* codes,
                            float* scales, hipStream_t s);
hipError_t launch_act8_unpack(int64_t n_rows, int d, int elem_bytes, const int8_t* codes,
                              const float* scales, void* x, hipStream_t s);

// launch_backward from x as an 8-bit checkpoint, dz held in float32.
struct BwdAct8 {
  const int8_t* codes;
  const float* scales;
};
bool bwd_act8_supported(const Geometry& g);
size_t bwd_act8_bytes(const Geometry& g, int64_t dense_cap);
hipError_t launch_backward_act8(const Geometry& g, int elem_bytes, const BwdHybrid& hy,
                                const BwdAct8& x8, const void* w_up_t, const void* w_down,
                                const void* dy, void* ws, void* dx, float* dw_up_t, float* db,
                                float* dw_down, hipStream_t s);

// Token embedding: out = scale * table[tokens], and the table's gradient.
// tokens are int32 or int64 (index_bytes 4 or 8).
constexpr int kEmbedGradStep = 1024;  // most tokens that a loop over an id's steps by
struct EmbedGradBufs {
  int32_t* counters;   // [4] places, short, medium and long ids handed out (cleared)
  int32_t* count;      // [vocab] tokens of each id (cleared)
  int64_t clear_ints;  // ints of counters + count, cleared together
  int32_t* base;       // [vocab] first place of each used id
  int32_t* pos;        // [n + 512] a token's place within its id, then the long ids' tokens in
                       // order (the sort: where its segments start)
  int32_t* perm;       // [n] token numbers, by id
  // used ids as {id, first place, tokens, 0}
  int4* short_segs;    // [min(n, vocab)] of at most 8 tokens
  int4* medium_segs;   // [n / 9 + 1] of at most 64
  int4* long_segs;     // [n / 65 + 1] of more
  size_t bytes;        // total workspace bytes
};
EmbedGradBufs embed_grad_carve(int64_t n_tokens, int vocab, void* ws);
hipError_t launch_embed_forward(int64_t n, int vocab, int d, int elem_bytes, int index_bytes,
                                float scale, const void* table, const void* tokens, void* out,
                                hipStream_t s);
hipError_t launch_embed_backward(int64_t n, int vocab, int d, int elem_bytes, int index_bytes,
                                 float scale, const void* dout, const void* tokens,
                                 const EmbedGradBufs& b, float* dtable, hipStream_t s);

// Log probabilities of targets [n_rows], entropy and log-sum-exp per row, and
// the `top` best columns; logits rows `stride` elements apart.
constexpr int kLogprobMaxTop = 32;
struct LogprobArgs {
  const void* logits;
  const void* targets;
  int64_t n_rows, stride;
  int vocab, top;
  float scale;
  float *logp, *entropy, *lse;  // [n_rows]
  int32_t* top_ids;             // [n_rows][top]
  float* top_logp;              // [n_rows][top]
  float4* parts;                // workspace: {m, s, t, 0} per part of a row
  float* part_top;              // workspace: [parts][top] values, best first
  int32_t* part_ids;            // workspace: [parts][top] columns
};
// Parts a row is split in, each taken by one wave (1: no workspace).
int logprob_splits(int64_t n_rows, int vocab, int elem_bytes);
// Sets the workspace parts of `a` (ws nullptr: sizes only); returns its bytes.
size_t logprob_carve(LogprobArgs* a, int elem_bytes, void* ws);
hipError_t launch_logprob_forward(const LogprobArgs& a, int elem_bytes, int index_bytes,
                                  hipStream_t s);
struct LogprobGradArgs {
  const void* logits;
  const void* targets;
  int64_t n_rows, stride, out_stride;
  int vocab;
  float scale;
  const float *lse, *entropy;     // [n_rows]; entropy is read with dentropy only
  const float *dlogp, *dentropy;  // [n_rows]; dentropy nullptr: none
  void* dlogits;
};
hipError_t launch_logprob_backward(const LogprobGradArgs& a, int elem_bytes, int index_bytes,
                                   hipStream_t s);

// Norms around the layer: residual_out = alpha residual + gate * norm(y) * w_post,
// x = norm(residual_out) * w_pre.  Weights are float32 [d], each may be null.
constexpr int kNormMaxWidth = 16384;
struct NormArgs {
  int64_t n_rows;
  int d;
  float alpha, eps;
  const float *w_post, *gate, *w_pre;
};
hipError_t launch_norm_forward(const NormArgs& a, int elem_bytes, const void* residual,
                               const void* y, void* residual_out, void* x, hipStream_t s);
template <typename E>
struct NormGradPtrs {
  const E *residual_out, *y, *d_residual_out, *dx;
  E *d_residual, *dy;
};
struct NormGradArgs {
  const void *residual_out, *y, *d_residual_out, *dx;
  void *d_residual, *dy;
  float *dw_post, *dgate, *dw_pre;
  float* sums;  // workspace: [2][groups][d]
};
// Groups of lanes the rows are dealt to, each with column sums of its own.
int norm_grad_groups(int64_t n_rows, int d);
hipError_t launch_norm_backward(const NormArgs& a, int elem_bytes, const NormGradArgs& p,
                                hipStream_t s);

// Log probabilities of targets [n_rows] under softmax(scale * x w^T) without the
// logits, and their gradient.  x [n_rows][d], w [vocab][d].
struct HeadArgs {
  const void *x, *w, *targets;
  int64_t n_rows;
  int vocab, d, index_bytes;
  float scale;
};
size_t head_forward_bytes(const HeadArgs& a, int elem_bytes);
size_t head_backward_bytes(const HeadArgs& a, int elem_bytes);
// stats [n_rows][2]: each row's largest z and its sum of exp(z - that)
hipError_t launch_head_forward(const HeadArgs& a, int elem_bytes, void* ws, float* logp,
                               float* lse, float* stats, hipStream_t s);
hipError_t launch_head_backward(const HeadArgs& a, int elem_bytes, const float* stats,
                                const float* dlogp, void* ws, void* dx, void* dw, hipStream_t s);

// The orthogonalised update of in [rows][cols] by `steps` Newton-Schulz steps with
// coefficients a, b, c; out may be in.
struct OrthArgs {
  const void* in;
  void* out;
  int rows, cols, steps;
  float a, b, c, eps, scale;
};
size_t orth_bytes(const OrthArgs& a, int elem_bytes);
hipError_t launch_orthogonalize(const OrthArgs& a, int elem_bytes, void* ws, hipStream_t s);

}  // namespace twell

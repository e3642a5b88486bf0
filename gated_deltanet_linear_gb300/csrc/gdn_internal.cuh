// Internal declarations shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

constexpr int kDim = 128;  // kd == vd: the only head size the kernels serve

// Launch modes of launch_steps.
//   kOverlapNone: an ordinary launch.
//   kOverlapPrologue: a programmatic dependent of the previous kernel on the
//     stream, which must not write S_in (the kernel starts loading the
//     state before it waits for that kernel): the layer prologue.
//   kOverlapAny: a programmatic dependent of whatever kernel came before;
//     the kernel reads nothing before that kernel has ended, so it only
//     takes over the launch and the start of its CTAs.  Applied to grids
//     that fill every CTA slot; smaller grids launch ordinarily.
constexpr int kOverlapNone = 0, kOverlapPrologue = 1, kOverlapAny = 2;
// Launches of more tokens than this start ordinarily: a long launch gains
// nothing from an earlier start, and its CTAs would wait on SM slots beside
// the previous launch's last CTAs.
constexpr int kOverlapMaxTokens = 16;

// Token-serial update of every head over M tokens (gdn_step, gdn_step_m and
// the fp32 prefill path).  Pointers and layouts as in gdn.h; S_out may equal
// S_in.  ckpt may be nullptr.  overlap: one of the modes above.
// host_inputs: some token input is in mapped host memory (single-token
// launches then use larger CTAs, whose warps share the inputs in L1).
cudaError_t launch_steps(const float *S_in, float *S_out, float *ckpt,
                         const float *q, const float *k, const float *v,
                         const float *g, const float *beta, float *o, int B,
                         int kh, int vh, int M, cudaStream_t stream,
                         int overlap = kOverlapNone, bool host_inputs = false);

// Layer prologue (conv1d + SiLU with a width-4 history, q/k normalisation,
// gates) writing the token inputs q, k, v, g, beta of M tokens.  hist_in and
// hist_out must not overlap.  overlap: launch as a programmatic dependent of
// the kernel before it; the prologue reads and writes nothing before that
// kernel has ended, and only then lets its own dependents start.
cudaError_t launch_layer_prologue(const float *hist_in, float *hist_out,
                                  const float *x, const float *conv_w,
                                  const float *a, const float *b,
                                  const float *A_log, const float *dt_bias,
                                  float eps, float *q, float *k, float *v,
                                  float *g, float *beta, int B, int kh, int vh,
                                  int M, cudaStream_t stream,
                                  bool overlap = false);

// Gated RMSNorm of `rows` rows of 128 channels (see gdn_gated_rmsnorm_m);
// y may equal o.
cudaError_t launch_gate_norm(const float *o, const float *z, const float *w,
                             float *y, float eps, size_t rows,
                             cudaStream_t stream);

// Per-sequence conv-history rollback (see gdn_layer_hist_rollback).
cudaError_t launch_hist_rollback(float *hist, const float *hist_snap,
                                 const float *x, const int *m_dev, int *err_dev,
                                 int B, int M, int conv_dim,
                                 cudaStream_t stream);

// dst[i] = src[i] for n floats (n % 4 == 0, both 16-byte aligned).
cudaError_t launch_copy(float *dst, const float *src, size_t n,
                        cudaStream_t stream);

// Per-sequence rollback copy (see gdn_rollback_seq).
cudaError_t launch_rollback_seq(float *S, const float *snap, const float *ckpt,
                                const int *m_dev, int *err_dev, int B, int vh,
                                int M, cudaStream_t stream);

// Linear attention with a decay for each head (gdn_linattn_step_m): token
// rows q, k, v, o in fp32 or bf16, states and g in fp32.  S_out may equal
// S_in, ckpt may be null.  lens (device, or null): sequence b has its first
// lens[b] of the M tokens; a value outside 0..M leaves the sequence alone
// and raises *err (may be null); the prompts alone take lens and err.
struct LinattnArgs {
  const float *S_in;
  float *S_out, *ckpt;
  const void *q, *k, *v;
  const float *g;
  void *o;
  const int *lens;
  int *err;
  float scale;
  int g_head;  // g is [vh] rather than [B][M][vh]
  int B, kh, vh, rep, M;
};
cudaError_t launch_linattn_steps(const LinattnArgs &P, bool bf16,
                                 cudaStream_t stream);
// The same over whole prompts (gdn_linattn_prefill), in place.
size_t linattn_prefill_workspace_bytes(int B, int vh, int T);
cudaError_t launch_linattn_prefill(const LinattnArgs &P, bool bf16,
                                   void *workspace, cudaStream_t stream);
// CTAs of it that gave up a wait.
cudaError_t linattn_timeouts(unsigned int *count);

// y = x W^T, W in 4 bits with fp16 group scales (gdn_quant_linear).
cudaError_t launch_quant_linear(const void *x, const unsigned char *qw,
                                const void *scales, void *y, int rows, int N,
                                int K, int group, bool bf16,
                                cudaStream_t stream);
// The form for many rows of x (called by launch_quant_linear).
cudaError_t launch_quant_linear_wide(const void *x, const unsigned char *qw, const void *scales,
                                     void *y, int rows, int N, int K, int group, bool bf16,
                                     cudaStream_t stream);
// Threads of it that gave up a wait for their products.
cudaError_t quant_timeouts(unsigned int *count);

// A paged key-value cache (gdn_kv_cache, checked): rows of hd channels at
// ((page * kvh + head) << page_shift) + row of the page, and their scales.
constexpr int kKvBf16 = 0, kKvInt8 = 1, kKvE4m3 = 2;
struct KvCache {
  void *k, *v;
  float *k_scale, *v_scale;  // null for bf16
  int kind, pages, kvh, page_shift;
};

// Rows to turn, to write into a cache or to read from one.  pos given: rope
// alone, `tokens` rows of qh heads; otherwise B sequences of M tokens at
// positions start[b] + m of their pages.  Strides in elements from token to
// token.  Reading: k goes to q_out, v to v_out.
struct KvRows {
  KvCache c;
  const void *q, *k, *v;
  void *q_out, *v_out;
  long long q_stride, k_stride, v_stride, tokens;
  const int *pos, *start, *counts, *table;
  int *err;
  const double *freq;
  float amp;
  int half, pairs;  // rot / 2; pairs side by side
  int M, cols, qh;
  int run;  // heads of a token side by side (set by the launch)
};
cudaError_t launch_kv_rows(const KvRows &P, int hd, bool bf16, bool read,
                           cudaStream_t stream);

// New tokens against a paged cache (gdn_attn_step_m).
struct AttnArgs {
  KvCache c;
  const void *q;
  void *o;
  float *lse;
  const int *table, *start, *counts;
  int *err;
  float scale;  // times log2 e
  int B, M, cols, qh, group;
  float *part;  // the workspace
};
size_t attn_workspace_bytes(int kind, int M, int group, int hd);
cudaError_t launch_attn(const AttnArgs &P, int hd, bool bf16, cudaStream_t stream);

// Chunked tensor-core prefill (defined in gdn_prefill.cu).
size_t prefill_workspace_bytes(int B, int kh, int vh, int T, int chunk,
                               int precision);
// precision: 1 = split-bf16 (three products), 2 = bf16 (one product).
cudaError_t launch_prefill_chunked(float *S, const float *q, const float *k,
                                   const float *v, const float *g,
                                   const float *beta, float *o, int B, int kh,
                                   int vh, int T, int precision,
                                   void *workspace, cudaStream_t stream);
cudaError_t prefill_timeouts(unsigned int *count);
// Ring waits of the multi-token kernel that ran out (gdn_decode.cu).
cudaError_t steps_timeouts(unsigned int *count);

}  // namespace gdn

struct gdn_shape;

namespace gdn {

// The checks gdn_layer_step_m makes of every argument except its workspace
// (a gdn.h status; GDN_OK also for B == 0).  Defined in gdn_api.cu.
int layer_step_check(const gdn_shape *s, int M, int ck, float eps,
                     const float *S_in, float *S_out, float *ckpt,
                     const float *hist_in, float *hist_out, const float *x,
                     const float *conv_w, const float *a, const float *b,
                     const float *A_log, const float *dt_bias, float *o);

}  // namespace gdn

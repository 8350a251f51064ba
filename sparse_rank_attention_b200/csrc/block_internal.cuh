// Internal declarations of the operators around RoLA (plan-less calls of the C ABI).
#pragma once

#include "rola_internal.cuh"

namespace rola {

struct RotArgs {
  int pos;                     // rola_pos
  int gt, gh, gw, st, sh, sw;
  int batched;                 // positions are [B, N, 3]
  int pt, ph;                  // pairs of the t and h axes (w takes the rest)
  const int32_t* positions;
  double turns[64];            // turns of pair c per unit of its axis: base^(-c'/P_axis) / 2 pi
};

struct NormRopeArgs {
  int B, N, H, d;
  int head_shift;              // log2(d)
  float eps;
  rola_strides q, k, qo, ko;   // inputs; outputs (forward) or upstream gradients (backward)
  RotArgs rot;
};

// Partial rows of dw that a launch over rows of C channels of one or two tensors writes.
int norm_rope_parts(int B, int N, int C, int tensors);
cudaError_t launch_norm_rope(const NormRopeArgs& a, rola_dtype dt, rola_qk_norm norm, const void* q, const void* k,
                             const float* wq, const float* wk, void* qo, void* ko, cudaStream_t st);
cudaError_t launch_norm_rope_backward(const NormRopeArgs& a, rola_dtype dt, rola_dtype gdt, rola_qk_norm norm,
                                      const void* dqo, const void* dko, const void* q, const void* k, const float* wq,
                                      const float* wk, void* dq, void* dk, float* dwq, float* dwk, float* part,
                                      cudaStream_t st);

struct GatedNormArgs {
  int B, N, C, T;
  int per;                     // tokens of a modulation row, N / T
  int chunks, chunk;           // backward: chunks of a modulation row's tokens, tokens of a chunk
  float eps;
  int64_t gate_b, gate_t, scale_b, scale_t, shift_b, shift_t;
};

void gated_norm_chunks(const rola_gated_norm_params& p, bool back, int* chunks, int* chunk);
size_t gated_norm_workspace(const rola_gated_norm_params& p);
cudaError_t launch_gated_norm(const GatedNormArgs& a, rola_dtype xt, rola_dtype yt, rola_norm_kind kind, const void* x,
                              const void* branch, const float* gate, const float* scale, const float* shift,
                              const float* weight, const float* bias, void* r, void* y, cudaStream_t st);
cudaError_t launch_gated_norm_backward(const GatedNormArgs& a, rola_dtype xt, rola_dtype yt, rola_norm_kind kind,
                                       const void* dy, const void* dr, const void* r, const void* branch,
                                       const float* gate, const float* scale, const float* weight, void* dx,
                                       void* dbranch, float* dgate, float* dscale, float* dshift, float* dweight,
                                       float* dbias, float* part, cudaStream_t st);

struct CrossArgs {
  int B, Nq, Nk, H, d;
  float scale;
  rola_strides q, k, v, dout;
  const int32_t* kv_len;
  const uint8_t* key_mask;
};

bool make_heads_map(CUtensorMap* m, const void* ptr, int B, int N, int H, int d, const rola_strides& s,
                    uint32_t rows);
// The bf16 forward on the tensor cores; `splits` blocks share a query tile's keys as below.
cudaError_t launch_cross_sm100(const CrossArgs& a, int splits, const void* q, const void* k, const void* v, void* out,
                               float* lse, float* part, cudaStream_t st);
// Its gradients: rows of softmax statistics first, then dq, then dk and dv.  stats: 2 * B * H *
// cross_padded_rows(Nq) floats.  splits_k as in the forward; splits_q blocks share a key tile's
// queries.
inline size_t cross_padded_rows(int Nq) { return ((size_t)Nq + 255) / 256 * 256; }
cudaError_t launch_cross_sm100_backward(const CrossArgs& a, int splits_q, int splits_k, const void* dout,
                                        const void* q, const void* k, const void* v, const void* out,
                                        const float* lse, void* dq, void* dk, void* dv, float* stats, float* part,
                                        cudaStream_t st);
// Read and clear this device's status word of those kernels.
cudaError_t cross_sm100_status(int* word, cudaStream_t st);
cudaError_t cross_sm100_backward_status(int* word, cudaStream_t st);

// Joins `splits` parts of the forward (each with its own softmax: [splits][B, Nq, H, d] fp32 and
// [splits][B, H, Nq]); sums `parts` parts of a gradient, `stride` floats apart.
cudaError_t launch_cross_join(const CrossArgs& a, rola_dtype dt, int splits, const float* part, const float* plse,
                              void* out, float* lse, cudaStream_t st);
cudaError_t launch_cross_sum(rola_dtype dt, int parts, size_t n, size_t stride, const float* part, void* out,
                             cudaStream_t st);
// splits_k: blocks that share a query tile's keys; splits_q: blocks that share a key tile's queries.
cudaError_t launch_cross_simt(const CrossArgs& a, int splits_k, const float* q, const float* k, const float* v,
                              float* out, float* lse, float* part, cudaStream_t st);
cudaError_t launch_cross_simt_backward(const CrossArgs& a, int splits_q, int splits_k, const float* dout,
                                       const float* q, const float* k, const float* v, const float* out,
                                       const float* lse, float* dq, float* dk, float* dv, float* drow, float* part,
                                       cudaStream_t st);

}  // namespace rola

// RMS norm of q and k with rotary positions on three axes, and its gradients.
//
//   u = x * w * rstd,  rstd = 1 / sqrt(mean(x^2) + eps);   y = R(p) u
//   g = R(p)^T dy;  dw = sum over tokens of g * x * rstd;  h = g * w;
//   dx = rstd * (h - x * rstd^2 * mean(h * x))
//
// Bound by memory: every element is read once and written once, so a token's row stays in
// registers between the statistics and the rotation.  A group of warps owns a token, a thread
// the same 8 channels (four rotary pairs) of every token it meets: the gains stay in registers,
// q and k go side by side under the same angles, and the next token's loads are issued before
// the present one is worked on.  A token's d/2 angles are formed once, by the first threads of
// its group, and shared through shared memory: the angle in fp64 turns, reduced to one turn
// (exact to 2^-53 of the position), then sincospi in fp32.
#include <cmath>

#include "block_internal.cuh"
#include "row_ops.cuh"

namespace rola {
namespace {

constexpr int kMaxGroups = 8;
constexpr int kThreadsPerSM = 1536;   // resident threads that the grid is sized for

struct Shared {
  float2 cs[2][kMaxGroups][64];
  float red[2][kMaxRowWarps * 4 + kMaxGroups * 4];   // groups side by side, [warp][values]
};

// cos and sin of token n's pairs into cs[0 .. d/2).
__device__ __forceinline__ void token_turns(const NormRopeArgs& a, int b, int n, int t, int threads, float2* cs) {
  const RotArgs& r = a.rot;
  const int P = a.d >> 1;
  for (int c = t; c < P; c += threads) {
    const int axis = c < r.pt ? 0 : c < r.pt + r.ph ? 1 : 2;
    long long p;
    if (r.pos == ROLA_POS_GIVEN) {
      p = __ldg(r.positions + ((size_t)(r.batched ? b : 0) * a.N + n) * 3 + axis);
    } else {
      const int hw = r.gh * r.gw;
      const int tt = n / hw, rem = n - tt * hw, y = rem / r.gw;
      p = axis == 0 ? (long long)tt + r.st : axis == 1 ? (long long)y + r.sh : (long long)(rem - y * r.gw) + r.sw;
      if (tt >= r.gt) p = 0;   // past the grid: not turned
    }
    double turn = (double)p * r.turns[c];
    turn -= rint(turn);
    float2 v;
    sincospif(2.f * (float)turn, &v.y, &v.x);
    cs[c] = v;
  }
}

// y = R u (kBack: R^T u) on a thread's four pairs.
template <bool kBack>
__device__ __forceinline__ void turn8(const float2* cs, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c = cs[i].x, s = kBack ? -cs[i].y : cs[i].y;
    const float a = v[2 * i], b = v[2 * i + 1];
    v[2 * i] = fmaf(a, c, -b * s);
    v[2 * i + 1] = fmaf(a, s, b * c);
  }
}

// Sum over the threads that hold one head's channels (d/8 neighbouring lanes: 8 or 16).
__device__ __forceinline__ float head_sum(float v, int d) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  if (d == 128) v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v;
}

template <typename T, int NORM, bool ROT>
__global__ void __launch_bounds__(1024) norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int W,
                                                         const T* q, const T* k,
                                                         const float* __restrict__ wq, const float* __restrict__ wk,
                                                         T* qo, T* ko) {
  __shared__ Shared sh;
  const RowGroup rg(W);
  const int G = blockDim.x / (32 * W);
  const int c0 = kVec * rg.t, h = c0 >> a.head_shift, c = c0 & (a.d - 1);
  const bool on = h < a.H, two = k != nullptr;
  const long long rows = (long long)a.B * a.N, step = (long long)gridDim.x * G;
  float gq[kVec], gk[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int at = NORM == ROLA_NORM_TOKEN ? c0 + i : c + i;
    gq[i] = NORM != ROLA_NORM_NONE && on ? __ldg(wq + at) : 1.f;
    gk[i] = NORM != ROLA_NORM_NONE && on && two ? __ldg(wk + at) : 1.f;
  }
  float* red = sh.red[0] + rg.g * (W + 1) * 2;
  const float inv = 1.f / (NORM == ROLA_NORM_TOKEN ? a.H * a.d : a.d);
  Raw8<T> nq, nk;
  nq.zero();
  nk.zero();
  auto fetch = [&](long long row) {
    if (row < rows && on) {
      const int b = (int)(row / a.N), n = (int)(row - (long long)b * a.N);
      nq.load(q + b * a.q.b + n * a.q.n + h * a.q.h + c);
      if (two) nk.load(k + b * a.k.b + n * a.k.n + h * a.k.h + c);
    }
  };
  long long row = (long long)blockIdx.x * G + rg.g;
  fetch(row);
  for (int it = 0; row < rows; row += step, ++it) {
    const int b = (int)(row / a.N), n = (int)(row - (long long)b * a.N);
    float x[kVec], y[kVec];
    nq.get(x);
    nk.get(y);
    fetch(row + step);
    float2* cs = sh.cs[it & 1][rg.g];
    if (ROT) token_turns(a, b, n, rg.t, 32 * W, cs);
    float s[2] = {0.f, 0.f};
    if (NORM != ROLA_NORM_NONE) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        s[0] = fmaf(x[i], x[i], s[0]);
        s[1] = fmaf(y[i], y[i], s[1]);
      }
    }
    if (NORM == ROLA_NORM_TOKEN) {
      group_sum<2>(rg, s, red + (it & 1) * (kMaxRowWarps * 4 + kMaxGroups * 4));
    } else {
      if (NORM == ROLA_NORM_HEAD) {
        s[0] = head_sum(s[0], a.d);
        s[1] = head_sum(s[1], a.d);
      }
      if (ROT) rg.sync();
    }
    if (NORM != ROLA_NORM_NONE) {
      const float rq = rsqrtf(fmaf(s[0], inv, a.eps)), rk = rsqrtf(fmaf(s[1], inv, a.eps));
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        x[i] = x[i] * rq * gq[i];
        y[i] = y[i] * rk * gk[i];
      }
    }
    if (on) {
      if (ROT) {
        turn8<false>(cs + (c >> 1), x);
        turn8<false>(cs + (c >> 1), y);
      }
      store8(qo + b * a.qo.b + n * a.qo.n + h * a.qo.h + c, x);
      if (two) store8(ko + b * a.ko.b + n * a.ko.n + h * a.ko.h + c, y);
    }
  }
}

// Backward.  dq, dk are contiguous.  part: [gridDim.x * G][2][H * d] partial sums of dw.
template <typename T, typename TG, int NORM, bool ROT>
__global__ void __launch_bounds__(1024) norm_rope_backward_kernel(
    const __grid_constant__ NormRopeArgs a, int W, const TG* dqo, const TG* dko,
    const T* __restrict__ q, const T* __restrict__ k, const float* __restrict__ wq, const float* __restrict__ wk,
    T* dq, T* dk, float* __restrict__ part) {
  __shared__ Shared sh;
  const RowGroup rg(W);
  const int G = blockDim.x / (32 * W);
  const int C = a.H * a.d;
  const int c0 = kVec * rg.t, h = c0 >> a.head_shift, c = c0 & (a.d - 1);
  const bool on = h < a.H, two = dko != nullptr;
  const long long rows = (long long)a.B * a.N, step = (long long)gridDim.x * G;
  float aq[kVec], ak[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) aq[i] = ak[i] = 0.f;
  const float* wqt = wq + (NORM == ROLA_NORM_TOKEN ? c0 : c);
  const float* wkt = wk + (NORM == ROLA_NORM_TOKEN ? c0 : c);
  float* red = sh.red[0] + rg.g * (W + 1) * 4;
  const float inv = 1.f / (NORM == ROLA_NORM_TOKEN ? C : a.d);
  int it = 0;
  for (long long row = (long long)blockIdx.x * G + rg.g; row < rows; row += step, ++it) {
    const int b = (int)(row / a.N), n = (int)(row - (long long)b * a.N);
    Raw8<T> xq, xk;
    Raw8<TG> rq, rk;
    xq.zero(); xk.zero(); rq.zero(); rk.zero();
    if (on) {
      rq.load(dqo + b * a.qo.b + n * a.qo.n + h * a.qo.h + c);
      if (two) rk.load(dko + b * a.ko.b + n * a.ko.n + h * a.ko.h + c);
      if (NORM != ROLA_NORM_NONE) {
        xq.load(q + b * a.q.b + n * a.q.n + h * a.q.h + c);
        if (two) xk.load(k + b * a.k.b + n * a.k.n + h * a.k.h + c);
      }
    }
    float2* cs = sh.cs[it & 1][rg.g];
    if (ROT) {
      token_turns(a, b, n, rg.t, 32 * W, cs);
      rg.sync();
    }
    float gq[kVec], gk[kVec];
    rq.get(gq);
    rk.get(gk);
    if (ROT && on) {
      turn8<true>(cs + (c >> 1), gq);
      turn8<true>(cs + (c >> 1), gk);
    }
    if (NORM != ROLA_NORM_NONE) {
      float x[kVec], y[kVec];
      xq.get(x);
      xk.get(y);
      float w[kVec], u[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        w[i] = on ? __ldg(wqt + i) : 0.f;
        u[i] = on && two ? __ldg(wkt + i) : 0.f;
      }
      float s[4] = {0.f, 0.f, 0.f, 0.f};   // sum x^2 and sum h x, of q and of k
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        s[0] = fmaf(x[i], x[i], s[0]);
        s[1] = fmaf(gq[i] * w[i], x[i], s[1]);
        s[2] = fmaf(y[i], y[i], s[2]);
        s[3] = fmaf(gk[i] * u[i], y[i], s[3]);
      }
      if (NORM == ROLA_NORM_TOKEN) {
        group_sum<4>(rg, s, red + (it & 1) * (kMaxRowWarps * 4 + kMaxGroups * 4));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = head_sum(s[i], a.d);
      }
      const float iq = rsqrtf(fmaf(s[0], inv, a.eps)), ik = rsqrtf(fmaf(s[2], inv, a.eps));
      const float mq = s[1] * inv * iq * iq, mk = s[3] * inv * ik * ik;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        aq[i] = fmaf(gq[i], x[i] * iq, aq[i]);
        ak[i] = fmaf(gk[i], y[i] * ik, ak[i]);
        gq[i] = iq * (gq[i] * w[i] - x[i] * mq);
        gk[i] = ik * (gk[i] * u[i] - y[i] * mk);
      }
    }
    if (on) {
      const size_t at = ((size_t)row * a.H + h) * a.d + c;
      store8(dq + at, gq);
      if (two) store8(dk + at, gk);
    }
  }
  if (NORM != ROLA_NORM_NONE && on) {
    float* p = part + ((size_t)blockIdx.x * G + rg.g) * 2 * C + c0;
    store8(p, aq);
    if (two) store8(p + C, ak);
  }
}

// dw[c] = sum over parts (and, per head, over heads) in a fixed order: 8 threads take every
// eighth part, then their sums in order.
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const float* __restrict__ part, int parts, int C, int cols,
                                                           float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float sum[8][32];
  const int col = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
  const float* p = part + (size_t)blockIdx.y * C;
  float s = 0.f;
  if (col < cols)
    for (int i = y; i < parts; i += 8)
      for (int c = col; c < C; c += cols) s += p[(size_t)i * 2 * C + c];
  sum[y][threadIdx.x] = s;
  __syncthreads();
  if (y == 0 && col < cols) {
    for (int i = 1; i < 8; ++i) s += sum[i][threadIdx.x];
    (blockIdx.y ? dwk : dwq)[col] = s;
  }
}

template <typename T, int NORM>
cudaError_t forward(const NormRopeArgs& a, const void* q, const void* k, const float* wq, const float* wk, void* qo,
                    void* ko, cudaStream_t st) {
  const RowShape s = row_shape((long long)a.B * a.N, a.H * a.d, kThreadsPerSM);
  if (a.rot.pos == ROLA_POS_NONE)
    norm_rope_kernel<T, NORM, false><<<s.blocks, s.threads, 0, st>>>(a, s.W, (const T*)q, (const T*)k, wq, wk, (T*)qo,
                                                                     (T*)ko);
  else
    norm_rope_kernel<T, NORM, true><<<s.blocks, s.threads, 0, st>>>(a, s.W, (const T*)q, (const T*)k, wq, wk, (T*)qo,
                                                                    (T*)ko);
  return cudaGetLastError();
}

template <typename T, typename TG, int NORM>
cudaError_t backward(const NormRopeArgs& a, const void* dqo, const void* dko, const void* q, const void* k,
                     const float* wq, const float* wk, void* dq, void* dk, float* dwq, float* dwk, float* part,
                     cudaStream_t st) {
  const int C = a.H * a.d;
  const RowShape s = row_shape((long long)a.B * a.N, C, kThreadsPerSM);
  if (a.rot.pos == ROLA_POS_NONE)
    norm_rope_backward_kernel<T, TG, NORM, false><<<s.blocks, s.threads, 0, st>>>(
        a, s.W, (const TG*)dqo, (const TG*)dko, (const T*)q, (const T*)k, wq, wk, (T*)dq, (T*)dk, part);
  else
    norm_rope_backward_kernel<T, TG, NORM, true><<<s.blocks, s.threads, 0, st>>>(
        a, s.W, (const TG*)dqo, (const TG*)dko, (const T*)q, (const T*)k, wq, wk, (T*)dq, (T*)dk, part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || NORM == ROLA_NORM_NONE) return e;
  const int cols = NORM == ROLA_NORM_HEAD ? a.d : C;
  norm_rope_dw_kernel<<<dim3((cols + 31) / 32, dko ? 2 : 1), dim3(32, 8), 0, st>>>(part, s.blocks * s.G, C, cols, dwq,
                                                                                 dwk);
  return cudaGetLastError();
}

template <typename T, typename TG, typename... A>
cudaError_t backward_norm(rola_qk_norm norm, const A&... x) {
  if (norm == ROLA_NORM_NONE) return backward<T, TG, ROLA_NORM_NONE>(x...);
  if (norm == ROLA_NORM_TOKEN) return backward<T, TG, ROLA_NORM_TOKEN>(x...);
  return backward<T, TG, ROLA_NORM_HEAD>(x...);
}
template <typename T, typename... A>
cudaError_t forward_norm(rola_qk_norm norm, const A&... x) {
  if (norm == ROLA_NORM_NONE) return forward<T, ROLA_NORM_NONE>(x...);
  if (norm == ROLA_NORM_TOKEN) return forward<T, ROLA_NORM_TOKEN>(x...);
  return forward<T, ROLA_NORM_HEAD>(x...);
}

}  // namespace

int norm_rope_parts(long long rows, int C) {
  const RowShape s = row_shape(rows, C, kThreadsPerSM);
  return s.blocks * s.G;
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, rola_dtype dt, rola_qk_norm norm, const void* q, const void* k,
                             const float* wq, const float* wk, void* qo, void* ko, cudaStream_t st) {
  if (dt == ROLA_F32) return forward_norm<float>(norm, a, q, k, wq, wk, qo, ko, st);
  return forward_norm<__nv_bfloat16>(norm, a, q, k, wq, wk, qo, ko, st);
}

cudaError_t launch_norm_rope_backward(const NormRopeArgs& a, rola_dtype dt, rola_dtype gdt, rola_qk_norm norm,
                                      const void* dqo, const void* dko, const void* q, const void* k, const float* wq,
                                      const float* wk, void* dq, void* dk, float* dwq, float* dwk, float* part,
                                      cudaStream_t st) {
  if (dt == ROLA_F32) return backward_norm<float, float>(norm, a, dqo, dko, q, k, wq, wk, dq, dk, dwq, dwk, part, st);
  if (gdt == ROLA_F32)
    return backward_norm<__nv_bfloat16, float>(norm, a, dqo, dko, q, k, wq, wk, dq, dk, dwq, dwk, part, st);
  return backward_norm<__nv_bfloat16, __nv_bfloat16>(norm, a, dqo, dko, q, k, wq, wk, dq, dk, dwq, dwk, part, st);
}

}  // namespace rola

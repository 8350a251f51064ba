// RMS norm of q and k with rotary positions on three axes, and its gradients.
//
//   u = x * w * rstd,  rstd = 1 / sqrt(mean(x^2) + eps);   y = R(p) u
//   g = R(p)^T dy;  dw = sum over tokens of g * x * rstd;  h = g * w;
//   dx = rstd * (h - x * rstd^2 * mean(h * x))
//
// Bound by memory: every element is read once and written once, so a token's row stays in
// registers between the statistics and the rotation.  A group of warps owns the rows of one
// tensor (q or k); a thread has up to four vectors of 8 channels, at the same channels of their
// heads (a group's width is a multiple of the head), so that one set of four angles serves them
// all and 1/rms is folded into it.  A token's d/2 angles are formed one token ahead by the first
// threads of the group: the angle in fp64 turns, reduced to one turn (exact to 2^-53 of the
// position), then sincospi in fp32.
#include <cmath>
#include <type_traits>

#include "block_internal.cuh"
#include "row_ops.cuh"

namespace rola {
namespace {

constexpr int kAhead = 3;       // token rows in flight per thread
constexpr int kMaxGroups = 4;
constexpr int kThreadsPerSM = 1024;

struct Shared {
  alignas(16) float2 cs[3][kMaxGroups][64];   // written one token ahead: three in turn
  alignas(16) float red[2][kMaxGroups][2 * kMaxRowWarps];
};

// The angles of a thread: pairs t and t + threads of the group.
struct Turner {
  double turns[2];
  int axis[2], pair[2];
  __device__ __forceinline__ Turner(const NormRopeArgs& a, int t, int threads) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = t + i * threads;
      pair[i] = c < (a.d >> 1) ? c : -1;
      axis[i] = c < a.rot.pt ? 0 : c < a.rot.pt + a.rot.ph ? 1 : 2;
      turns[i] = pair[i] >= 0 ? a.rot.turns[c] : 0.0;
    }
  }
  // cos and sin of token n's pairs into cs[0 .. d/2)
  __device__ __forceinline__ void write(const NormRopeArgs& a, int b, int n, float2* cs) const {
    if (pair[0] < 0) return;
    const RotArgs& r = a.rot;
    int tt = 0, y = 0, x = 0;
    if (r.pos == ROLA_POS_GRID) {
      const unsigned hw = r.gh * r.gw;
      tt = (unsigned)n / hw;
      const unsigned rem = n - tt * hw;
      y = rem / (unsigned)r.gw;
      x = rem - y * r.gw;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (pair[i] < 0) return;
      long long p;
      if (r.pos == ROLA_POS_GIVEN)
        p = __ldg(r.positions + ((size_t)(r.batched ? b : 0) * a.N + n) * 3 + axis[i]);
      else if (tt >= r.gt)
        p = 0;                         // past the grid: not turned
      else
        p = axis[i] == 0 ? (long long)tt + r.st : axis[i] == 1 ? (long long)y + r.sh : (long long)x + r.sw;
      double turn = (double)p * turns[i];
      turn -= rint(turn);
      float2 v;
      sincospif(2.f * (float)turn, &v.y, &v.x);
      cs[pair[i]] = v;
    }
  }
};

// v = R u (kBack: R^T u) on four pairs.
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
__device__ __forceinline__ void load_turns(const float2* p, float2* cs) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 2);
  cs[0] = make_float2(a.x, a.y);
  cs[1] = make_float2(a.z, a.w);
  cs[2] = make_float2(b.x, b.y);
  cs[3] = make_float2(b.z, b.w);
}

// Sum over the threads that hold one head's channels (d/8 neighbouring lanes: 8 or 16).
__device__ __forceinline__ float head_sum(float v, int d) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  if (d == 128) v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v;
}

// grid (token groups, B, q | k).
template <typename T, int NORM, bool ROT, int V>
__global__ void __launch_bounds__(256) norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int W, const T* q,
                                                        const T* k, const float* __restrict__ wq,
                                                        const float* __restrict__ wk, T* qo, T* ko) {
  constexpr int kPieces = V * Raw8<T>::kPieces;
  __shared__ Shared sh;
  extern __shared__ uint4 ring[];      // [kAhead][pieces][threads]
  const RowGroup rg(W);
  const int G = blockDim.x / (32 * W), b = blockIdx.y, nt = blockDim.x;
  const bool is_k = blockIdx.z;
  const rola_strides si = is_k ? a.k : a.q, so = is_k ? a.ko : a.qo;
  const float* w = is_k ? wk : wq;
  const int h0 = (kVec * rg.t) >> a.head_shift, c = (kVec * rg.t) & (a.d - 1), hs = (kVec * 32 * W) >> a.head_shift;
  const T* src = (is_k ? k : q) + b * si.b + h0 * si.h + c;
  T* dst = (is_k ? ko : qo) + b * so.b + h0 * so.h + c;
  float gain[V][kVec];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const bool on = h0 + j * hs < a.H;
      gain[j][i] = NORM == ROLA_NORM_NONE || !on ? 1.f
                   : NORM == ROLA_NORM_HEAD      ? __ldg(w + c + i)
                                                 : __ldg(w + (size_t)(h0 + j * hs) * a.d + c + i);
    }
  const Turner turner(a, rg.t, 32 * W);
  const float inv = 1.f / (NORM == ROLA_NORM_TOKEN ? a.H * a.d : a.d);
  const int first = blockIdx.x * G + rg.g, step = gridDim.x * G;
  uint4* mine = ring + threadIdx.x;
  auto fetch = [&](long long n, int s) {
    if (n < a.N) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (h0 + j * hs < a.H)
          copy_vec(mine + (s * kPieces + j * Raw8<T>::kPieces) * nt, nt, src + n * si.n + j * hs * si.h);
    }
    copy_commit();
  };
#pragma unroll
  for (int s = 0; s < kAhead - 1; ++s) fetch(first + (long long)s * step, s);
  if (ROT && first < a.N) turner.write(a, b, first, sh.cs[0][rg.g]);
  int slot = 0, turn = 0, it = 0;
  for (long long n = first; n < a.N; n += step, ++it) {
    fetch(n + (long long)(kAhead - 1) * step, slot == 0 ? kAhead - 1 : slot - 1);
    copy_wait<kAhead - 1>();
    float x[V][kVec];
    float sum = 0.f, rms[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool on = h0 + j * hs < a.H;
      Raw8<T> raw;
      raw.slot(mine + (slot * kPieces + j * Raw8<T>::kPieces) * nt, nt);
      raw.get(x[j]);
      float s = 0.f;
      if (NORM != ROLA_NORM_NONE && on) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) s = fmaf(x[j][i], x[j][i], s);
      }
      sum += s;
      if (NORM == ROLA_NORM_HEAD) rms[j] = rsqrtf(fmaf(head_sum(s, a.d), inv, a.eps));
    }
    const int next = turn == 2 ? 0 : turn + 1;
    if (ROT && n + step < a.N) turner.write(a, b, (int)(n + step), sh.cs[next][rg.g]);
    float unit = 1.f;
    if (NORM == ROLA_NORM_TOKEN)
      unit = rsqrtf(fmaf(group_sum(rg, sum, sh.red[it & 1][rg.g]), inv, a.eps));
    else if (ROT)
      rg.sync();
    float2 cs[4];
    if (ROT) {
      load_turns(sh.cs[turn][rg.g] + (c >> 1), cs);
#pragma unroll
      for (int i = 0; i < 4; ++i) cs[i] = make_float2(cs[i].x * unit, cs[i].y * unit);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (h0 + j * hs >= a.H) continue;
      const float f = (NORM == ROLA_NORM_HEAD ? rms[j] : 1.f) * (ROT ? 1.f : unit);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        if (NORM != ROLA_NORM_NONE) x[j][i] *= gain[j][i];
        if (NORM == ROLA_NORM_HEAD || (NORM == ROLA_NORM_TOKEN && !ROT)) x[j][i] *= f;
      }
      if (ROT) turn8<false>(cs, x[j]);
      store8(dst + n * so.n + j * hs * so.h, x[j]);
    }
    slot = slot == kAhead - 1 ? 0 : slot + 1;
    turn = next;
  }
  copy_wait<0>();
}

// Backward.  dq, dk are contiguous.  part: [gridDim.x * B * G][2][H * d] partial sums of dw.
template <typename T, typename TG, int NORM, bool ROT, int V>
__global__ void __launch_bounds__(256, V == 4 ? 1 : 2) norm_rope_backward_kernel(
    const __grid_constant__ NormRopeArgs a, int W, const TG* dqo, const TG* dko, const T* __restrict__ q,
    const T* __restrict__ k, const float* __restrict__ wq, const float* __restrict__ wk, T* dq, T* dk,
    float* __restrict__ part) {
  constexpr int kPg = Raw8<TG>::kPieces, kPx = NORM == ROLA_NORM_NONE ? 0 : Raw8<T>::kPieces;
  constexpr int kPieces = V * (kPg + kPx);
  __shared__ Shared sh;
  extern __shared__ uint4 ring[];      // [kAhead][pieces][threads]
  const RowGroup rg(W);
  const int G = blockDim.x / (32 * W), b = blockIdx.y, nt = blockDim.x, C = a.H * a.d;
  const bool is_k = blockIdx.z;
  const rola_strides si = is_k ? a.k : a.q, su = is_k ? a.ko : a.qo;
  const float* w = is_k ? wk : wq;
  const int h0 = (kVec * rg.t) >> a.head_shift, c = (kVec * rg.t) & (a.d - 1), hs = (kVec * 32 * W) >> a.head_shift;
  const T* src = NORM == ROLA_NORM_NONE ? nullptr : (is_k ? k : q) + b * si.b + h0 * si.h + c;
  const TG* up = (is_k ? dko : dqo) + b * su.b + h0 * su.h + c;
  T* dst = (is_k ? dk : dq) + ((size_t)b * a.N * a.H + h0) * a.d + c;
  float gain[V][kVec], acc[V][kVec];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const bool on = h0 + j * hs < a.H;
      gain[j][i] = NORM == ROLA_NORM_NONE || !on ? 0.f
                   : NORM == ROLA_NORM_HEAD      ? __ldg(w + c + i)
                                                 : __ldg(w + (size_t)(h0 + j * hs) * a.d + c + i);
      acc[j][i] = 0.f;
    }
  const Turner turner(a, rg.t, 32 * W);
  const float inv = 1.f / (NORM == ROLA_NORM_TOKEN ? C : a.d);
  const int first = blockIdx.x * G + rg.g, step = gridDim.x * G;
  uint4* mine = ring + threadIdx.x;
  auto fetch = [&](long long n, int s) {
    if (n < a.N) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (h0 + j * hs < a.H) {
          uint4* at = mine + (s * kPieces + j * (kPg + kPx)) * nt;
          copy_vec(at, nt, up + n * su.n + j * hs * su.h);
          if (NORM != ROLA_NORM_NONE) copy_vec(at + kPg * nt, nt, src + n * si.n + j * hs * si.h);
        }
    }
    copy_commit();
  };
#pragma unroll
  for (int s = 0; s < kAhead - 1; ++s) fetch(first + (long long)s * step, s);
  if (ROT && first < a.N) turner.write(a, b, first, sh.cs[0][rg.g]);
  if (ROT) rg.sync();
  int slot = 0, turn = 0, it = 0;
  for (long long n = first; n < a.N; n += step, ++it) {
    fetch(n + (long long)(kAhead - 1) * step, slot == 0 ? kAhead - 1 : slot - 1);
    copy_wait<kAhead - 1>();
    float2 cs[4];
    if (ROT) load_turns(sh.cs[turn][rg.g] + (c >> 1), cs);
    float g[V][kVec];
    float s0 = 0.f, s1 = 0.f, r[V], m[V];   // sums of x^2 and of h x;  1/rms and r^2 mean(h x)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const bool on = h0 + j * hs < a.H;
      const uint4* at = mine + (slot * kPieces + j * (kPg + kPx)) * nt;
      Raw8<TG> raw;
      raw.slot(at, nt);
      raw.get(g[j]);
      if (ROT) turn8<true>(cs, g[j]);
      if (NORM != ROLA_NORM_NONE) {
        Raw8<T> raw_x;                 // read again below: cheaper than V x 8 more registers
        float x[kVec];
        raw_x.slot(at + kPg * nt, nt);
        raw_x.get(x);
        float t0 = 0.f, t1 = 0.f;
        if (on) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            t0 = fmaf(x[i], x[i], t0);
            t1 = fmaf(g[j][i] * gain[j][i], x[i], t1);
          }
        }
        s0 += t0;
        s1 += t1;
        if (NORM == ROLA_NORM_HEAD) {
          r[j] = rsqrtf(fmaf(head_sum(t0, a.d), inv, a.eps));
          m[j] = head_sum(t1, a.d) * inv * r[j] * r[j];
        }
      }
    }
    const int next = turn == 2 ? 0 : turn + 1;
    if (ROT && n + step < a.N) turner.write(a, b, (int)(n + step), sh.cs[next][rg.g]);
    if (NORM == ROLA_NORM_TOKEN) {
      const float2 s = group_sum(rg, s0, s1, sh.red[it & 1][rg.g]);
      if (ROT && W == 1) __syncwarp();
      r[0] = rsqrtf(fmaf(s.x, inv, a.eps));
      m[0] = s.y * inv * r[0] * r[0];
#pragma unroll
      for (int j = 1; j < V; ++j) r[j] = r[0], m[j] = m[0];
    } else if (ROT) {
      rg.sync();
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (h0 + j * hs >= a.H) continue;
      if (NORM != ROLA_NORM_NONE) {
        Raw8<T> raw_x;
        float x[kVec];
        raw_x.slot(mine + (slot * kPieces + j * (kPg + kPx) + kPg) * nt, nt);
        raw_x.get(x);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          acc[j][i] = fmaf(g[j][i], x[i] * r[j], acc[j][i]);
          g[j][i] = r[j] * (g[j][i] * gain[j][i] - x[i] * m[j]);
        }
      }
      store8(dst + ((size_t)n * a.H + j * hs) * a.d, g[j]);
    }
    slot = slot == kAhead - 1 ? 0 : slot + 1;
    turn = next;
  }
  copy_wait<0>();
  if (NORM != ROLA_NORM_NONE) {
    const size_t group = ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * G + rg.g;
    float* p = part + (group * 2 + is_k) * C + (size_t)h0 * a.d + c;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (h0 + j * hs < a.H) store8(p + (size_t)j * hs * a.d, acc[j]);
  }
}

// dw of q and k (blockIdx.y) from the partial sums; per head, over the heads too.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* __restrict__ part, int parts, int C, int cols,
                                                            float* __restrict__ dwq, float* __restrict__ dwk) {
  column_sum(part + (size_t)blockIdx.y * C, parts, 2 * (size_t)C, cols, C / cols, blockIdx.y ? dwk : dwq);
}

// Blocks of token groups: the SMs full with the rows of both tensors and all samples.
int token_blocks(const RowShape& s, int B, int N, int tensors) {
  const long long fill = (long long)kRowSMs * (kThreadsPerSM / s.threads);
  long long x = (fill + (long long)B * tensors - 1) / ((long long)B * tensors);
  const long long most = (N + s.G - 1) / s.G;
  return (int)(x < most ? x : most);
}

template <typename K>
cudaError_t opt_in(K kern, size_t smem) {
  return smem <= 40 * 1024 ? cudaSuccess
                           : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

template <typename T, int NORM, bool ROT, int V>
cudaError_t forward_v(const NormRopeArgs& a, const RowShape& s, const void* q, const void* k, const float* wq,
                      const float* wk, void* qo, void* ko, cudaStream_t st) {
  const size_t smem = 16 * (size_t)kAhead * V * Raw8<T>::kPieces * s.threads;
  const int tensors = k ? 2 : 1;
  cudaError_t e = opt_in(norm_rope_kernel<T, NORM, ROT, V>, smem);
  if (e != cudaSuccess) return e;
  norm_rope_kernel<T, NORM, ROT, V><<<dim3(token_blocks(s, a.B, a.N, tensors), a.B, tensors), s.threads, smem, st>>>(
      a, s.W, (const T*)q, (const T*)k, wq, wk, (T*)qo, (T*)ko);
  return cudaGetLastError();
}

template <typename T, int NORM>
cudaError_t forward(const NormRopeArgs& a, const void* q, const void* k, const float* wq, const float* wk, void* qo,
                    void* ko, cudaStream_t st) {
  const RowShape s = row_shape(a.H * a.d, 4);
  auto go = [&](auto rot) {
    constexpr bool R = decltype(rot)::value;
    return s.V == 1   ? forward_v<T, NORM, R, 1>(a, s, q, k, wq, wk, qo, ko, st)
           : s.V == 2 ? forward_v<T, NORM, R, 2>(a, s, q, k, wq, wk, qo, ko, st)
                      : forward_v<T, NORM, R, 4>(a, s, q, k, wq, wk, qo, ko, st);
  };
  return a.rot.pos == ROLA_POS_NONE ? go(std::false_type{}) : go(std::true_type{});
}

template <typename T, typename TG, int NORM, bool ROT, int V>
cudaError_t backward_v(const NormRopeArgs& a, const RowShape& s, const void* dqo, const void* dko, const void* q,
                       const void* k, const float* wq, const float* wk, void* dq, void* dk, float* dwq, float* dwk,
                       float* part, cudaStream_t st) {
  const size_t smem = 16 * (size_t)kAhead * V * (Raw8<TG>::kPieces + (NORM ? Raw8<T>::kPieces : 0)) * s.threads;
  const int tensors = dko ? 2 : 1, C = a.H * a.d, blocks = token_blocks(s, a.B, a.N, tensors);
  cudaError_t e = opt_in(norm_rope_backward_kernel<T, TG, NORM, ROT, V>, smem);
  if (e != cudaSuccess) return e;
  norm_rope_backward_kernel<T, TG, NORM, ROT, V><<<dim3(blocks, a.B, tensors), s.threads, smem, st>>>(
      a, s.W, (const TG*)dqo, (const TG*)dko, (const T*)q, (const T*)k, wq, wk, (T*)dq, (T*)dk, part);
  e = cudaGetLastError();
  if (e != cudaSuccess || NORM == ROLA_NORM_NONE) return e;
  const int cols = NORM == ROLA_NORM_HEAD ? a.d : C;
  norm_rope_dw_kernel<<<dim3((cols + 31) / 32, tensors), dim3(32, 32), 0, st>>>(part, blocks * a.B * s.G, C, cols, dwq,
                                                                              dwk);
  return cudaGetLastError();
}

template <typename T, typename TG, int NORM>
cudaError_t backward(const NormRopeArgs& a, const void* dqo, const void* dko, const void* q, const void* k,
                     const float* wq, const float* wk, void* dq, void* dk, float* dwq, float* dwk, float* part,
                     cudaStream_t st) {
  const RowShape s = row_shape(a.H * a.d, 4);
  auto go = [&](auto rot) {
    constexpr bool R = decltype(rot)::value;
    return s.V == 1   ? backward_v<T, TG, NORM, R, 1>(a, s, dqo, dko, q, k, wq, wk, dq, dk, dwq, dwk, part, st)
           : s.V == 2 ? backward_v<T, TG, NORM, R, 2>(a, s, dqo, dko, q, k, wq, wk, dq, dk, dwq, dwk, part, st)
                      : backward_v<T, TG, NORM, R, 4>(a, s, dqo, dko, q, k, wq, wk, dq, dk, dwq, dwk, part, st);
  };
  return a.rot.pos == ROLA_POS_NONE ? go(std::false_type{}) : go(std::true_type{});
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

int norm_rope_parts(int B, int N, int C, int tensors) {
  const RowShape s = row_shape(C, 4);
  return token_blocks(s, B, N, tensors) * B * s.G;
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

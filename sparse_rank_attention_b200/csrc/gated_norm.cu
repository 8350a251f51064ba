// Gated residual with the modulated norm of the sum, and its gradients.
//
//   r = x + gate * branch;  xhat = (r - mean) * rstd  (or r * rstd);  y = xhat * A + B
//   with A, B = 1 + scale, shift  or  weight, bias.
//   g = dy * A;  dx = dr + rstd * (g - mean(g) - xhat * mean(g * xhat))  (rms: no mean(g))
//   dbranch = gate * dx;  dgate = sum dx * branch;  dA = sum dy * xhat;  dB = sum dy,
//   the sums over the tokens that share a row of the modulation (all tokens for weight, bias).
//
// Bound by memory: each tensor is read or written once.  A group of warps owns a token; a thread
// has the same pieces of E channels of every token it meets, so that the modulation stays in
// registers while the tokens share it and the column sums of the backward are private to a
// thread.  The variance is taken about the mean of the values held in registers (a second sum,
// not E[x^2] - E[x]^2, which loses everything when the mean is large).
//
// Measured with x in fp32, branch and y in bf16, 5120 channels: 75600 tokens 820 to 870 us for
// 4.64 GB (5.3 to 5.7 TB/s, 0.82 to 0.87 of a plain copy); the backward of 32760 tokens 530 to 580 us
// for 3.02 GB (0.80 to 0.87).  Reads and writes mixed over five streams, as here, do not reach a copy's
// rate.  The backward of 2331 rows of 1000 fp32 channels: 9 us and 6 for the sums of the weight.
#include <type_traits>

#include "block_internal.cuh"
#include "row_ops.cuh"

namespace rola {
namespace {

constexpr int kThreadsPerSM = 1024;   // resident threads that a grid is sized for
constexpr size_t kRing = 192 * 1024;  // shared memory for the rows in flight of a block
constexpr int kMaxGroups = 4;
constexpr int kMaxThreads = 512;      // 8192 channels
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kDeep = 3;              // rows in flight of a group, where so many fit into the ring

struct Shared {
  alignas(16) float red[2][kMaxGroups][2 * kMaxWarps];
};

// Channels of a piece; pieces of 8 go by two, pieces of 4 by four.
constexpr int piece_of(rola_dtype x, rola_dtype y) { return x == ROLA_F32 || y == ROLA_F32 ? 4 : 8; }
RowShape shape_of(int C, int E) { return row_shape(C, E, 16 / E, kMaxWarps); }
// The most threads of a block of that shape: with fewer pieces a thread than may be, rows of 8 warps
// and more would have taken twice as many.
constexpr int widest(int E, int V) { return V * E == 16 ? kMaxThreads : 256; }

// A group's walk over its rows: the tokens of segment `seg`, then of seg + groups, ...; a segment
// is a chunk of the tokens that share a modulation row.
struct Cursor {
  long long seg;
  int b, t, n, n1;
  __device__ __forceinline__ void open(const GatedNormArgs& a, long long segs) {
    if (seg >= segs) return;
    const unsigned mod = (unsigned)(seg / a.chunks), ch = (unsigned)(seg - (long long)mod * a.chunks);
    b = mod / (unsigned)a.T;
    t = mod - b * a.T;
    n = t * a.per + ch * a.chunk;
    const int end = (t + 1) * a.per;   // at most 2^31 - 1, which n + a.chunk may pass
    n1 = end - n > a.chunk ? n + a.chunk : end;
  }
  // the next row; true where it opens a segment
  __device__ __forceinline__ bool next(const GatedNormArgs& a, long long segs, long long groups) {
    if (++n < n1) return false;
    seg += groups;
    open(a, segs);
    return true;
  }
};

template <typename TX, typename TY, int E, bool LAYER, bool BRANCH, int V>
__global__ void __launch_bounds__(kMaxThreads) gated_norm_kernel(
    const __grid_constant__ GatedNormArgs a, int W, const TX* x, const TY* __restrict__ branch,
    const float* __restrict__ gate, const float* __restrict__ scale, const float* __restrict__ shift,
    const float* __restrict__ weight, const float* __restrict__ bias, TX* r, TY* __restrict__ y) {
  constexpr int kBx = piece_bytes<E, TX>(), kBb = BRANCH ? piece_bytes<E, TY>() : 0, kRow = V * (kBx + kBb);
  constexpr int kAhead = kDeep;
  __shared__ Shared sh;
  extern __shared__ __align__(16) uint8_t ring[];   // [kAhead][V][x, branch][threads] pieces
  const RowGroup rg(W);
  const int G = blockDim.x / (32 * W), nt = blockDim.x, c0 = E * rg.t, cs = E * 32 * W;
  const float inv = 1.f / a.C;
  const long long segs = (long long)a.B * a.T * a.chunks, groups = (long long)gridDim.x * G;
  float mg[V][E], ma[V][E], mb[V][E];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = c0 + j * cs + i;
      mg[j][i] = 1.f;
      ma[j][i] = weight && c < a.C ? __ldg(weight + c) : 1.f;
      mb[j][i] = bias && c < a.C ? __ldg(bias + c) : 0.f;
    }
  Cursor ahead{(long long)blockIdx.x * G + rg.g, 0, 0, 0, 0};
  ahead.open(a, segs);
  Cursor now = ahead;
  auto fetch = [&](int s) {
    if (ahead.seg < segs) {
      const size_t row = (size_t)ahead.b * a.N + ahead.n;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = c0 + j * cs;
        if (c < a.C) {
          uint8_t* at = ring + (s * kRow + j * (kBx + kBb)) * nt;
          fetch_piece<E>(at, x + row * a.C + c);
          if (BRANCH) fetch_piece<E>(at + kBx * nt, branch + row * a.C + c);
        }
      }
      ahead.next(a, segs, groups);
    }
    copy_commit();
  };
#pragma unroll
  for (int s = 0; s < kAhead - 1; ++s) fetch(s);
  bool open = true;
  for (int it = 0, slot = 0; now.seg < segs; ++it) {
    {
      const size_t row = (size_t)now.b * a.N + now.n;
      if (open) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = c0 + j * cs;
          if (c < a.C) {
            if (gate) load_floats<E>(gate + now.b * a.gate_b + now.t * a.gate_t + c, mg[j]);
            if (scale) {
              load_floats<E>(scale + now.b * a.scale_b + now.t * a.scale_t + c, ma[j]);
              load_floats<E>(shift + now.b * a.shift_b + now.t * a.shift_t + c, mb[j]);
#pragma unroll
              for (int i = 0; i < E; ++i) ma[j][i] += 1.f;
            }
          }
        }
      }
      fetch(slot == 0 ? kAhead - 1 : slot - 1);
      copy_wait<kAhead - 1>();
      float v[V][E];
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = c0 + j * cs;
        const uint8_t* at = ring + (slot * kRow + j * (kBx + kBb)) * nt;
        if (c < a.C) {
          read_piece<E, TX>(at, v[j]);
          if (BRANCH) {
            float u[E];
            read_piece<E, TY>(at + kBx * nt, u);
#pragma unroll
            for (int i = 0; i < E; ++i) v[j][i] = fmaf(mg[j][i], u[i], v[j][i]);
            store_piece<E>(r + row * a.C + c, v[j]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i) v[j][i] = 0.f;
        }
        if (LAYER) {
#pragma unroll
          for (int i = 0; i < E; ++i) sum += v[j][i];
        }
      }
      if (LAYER) {
        const float mean = group_sum(rg, sum, sh.red[0][rg.g]) * inv;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int i = 0; i < E; ++i) v[j][i] = c0 + j * cs < a.C ? v[j][i] - mean : 0.f;
      }
      float sq = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) sq = fmaf(v[j][i], v[j][i], sq);
      const float rstd = rsqrtf(fmaf(group_sum(rg, sq, sh.red[LAYER ? 1 : it & 1][rg.g]), inv, a.eps));
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = c0 + j * cs;
        if (c < a.C) {
#pragma unroll
          for (int i = 0; i < E; ++i) v[j][i] = fmaf(v[j][i] * rstd, ma[j][i], mb[j][i]);
          store_piece<E>(y + row * a.C + c, v[j]);
        }
      }
    }
    slot = slot == kAhead - 1 ? 0 : slot + 1;
    open = now.next(a, segs, groups);
  }
  copy_wait<0>();
}

// A group takes one segment after the other: a chunk of the tokens that share a modulation
// row.  A segment's column sums go to msum, [segments][3][C] (dgate, dscale, dshift): the
// gradients themselves where a modulation row is one segment (outputs given), else partial
// sums.  The sums of weight and bias run over all segments of the group: wsum [groups][2][C].
template <typename TX, typename TY, int E, bool LAYER, bool DR, bool BRANCH, int V, int kAhead, int kMost>
__global__ void __launch_bounds__(kMost) gated_norm_backward_kernel(
    const __grid_constant__ GatedNormArgs a, int W, const TY* __restrict__ dy, const TX* dr,
    const TX* __restrict__ r, const TY* __restrict__ branch, const float* __restrict__ gate,
    const float* __restrict__ scale, const float* __restrict__ weight, TX* dx, TY* __restrict__ dbranch,
    float* __restrict__ dgate, float* __restrict__ dscale, float* __restrict__ dshift, int64_t sum_stride,
    float* __restrict__ wsum) {
  constexpr int kBx = piece_bytes<E, TX>(), kBy = piece_bytes<E, TY>();
  constexpr int kD = kBx + kBy, kB = kD + (DR ? kBx : 0), kEach = kB + (BRANCH ? kBy : 0), kRow = V * kEach;
  __shared__ Shared sh;
  extern __shared__ __align__(16) uint8_t ring[];   // [kAhead][V][r, dy, dr, branch][threads] pieces
  const RowGroup rg(W);
  const int G = blockDim.x / (32 * W), nt = blockDim.x, c0 = E * rg.t, cs = E * 32 * W;
  const float inv = 1.f / a.C;
  const long long segs = (long long)a.B * a.T * a.chunks, groups = (long long)gridDim.x * G;
  const long long group = (long long)blockIdx.x * G + rg.g;
  float mg[V][E], ma[V][E], sg[V][E], sa[V][E], sb[V][E];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = c0 + j * cs + i;
      mg[j][i] = 1.f;
      ma[j][i] = weight && c < a.C ? __ldg(weight + c) : 1.f;
      sg[j][i] = sa[j][i] = sb[j][i] = 0.f;
    }
  Cursor ahead{group, 0, 0, 0, 0};
  ahead.open(a, segs);
  Cursor now = ahead;
  auto fetch = [&](int s) {
    if (ahead.seg < segs) {
      const size_t row = (size_t)ahead.b * a.N + ahead.n;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = c0 + j * cs;
        if (c < a.C) {
          uint8_t* at = ring + (s * kRow + j * kEach) * nt;
          fetch_piece<E>(at, r + row * a.C + c);
          fetch_piece<E>(at + kBx * nt, dy + row * a.C + c);
          if (DR) fetch_piece<E>(at + kD * nt, dr + row * a.C + c);
          if (BRANCH) fetch_piece<E>(at + kB * nt, branch + row * a.C + c);
        }
      }
      ahead.next(a, segs, groups);
    }
    copy_commit();
  };
#pragma unroll
  for (int s = 0; s < kAhead - 1; ++s) fetch(s);
  bool open = true;
  for (int it = 0, slot = 0; now.seg < segs; ++it) {
    const long long seg = now.seg;
    {
      const size_t row = (size_t)now.b * a.N + now.n;
      if (open) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = c0 + j * cs;
          if (c < a.C) {
            if (BRANCH && gate) load_floats<E>(gate + now.b * a.gate_b + now.t * a.gate_t + c, mg[j]);
            if (scale) {
              load_floats<E>(scale + now.b * a.scale_b + now.t * a.scale_t + c, ma[j]);
#pragma unroll
              for (int i = 0; i < E; ++i) ma[j][i] += 1.f;
            }
          }
        }
      }
      fetch(slot == 0 ? kAhead - 1 : slot - 1);
      copy_wait<kAhead - 1>();
      const uint8_t* at = ring + slot * kRow * nt;
      float v[V][E], d[V][E];
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (c0 + j * cs < a.C) {
          read_piece<E, TX>(at + j * kEach * nt, v[j]);
          read_piece<E, TY>(at + (j * kEach + kBx) * nt, d[j]);
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i) v[j][i] = d[j][i] = 0.f;
        }
        if (LAYER) {
#pragma unroll
          for (int i = 0; i < E; ++i) {
            s0 += v[j][i];
            s1 = fmaf(d[j][i], ma[j][i], s1);
          }
        }
      }
      float gm = 0.f;
      if (LAYER) {
        const float2 s = group_sum(rg, s0, s1, sh.red[0][rg.g]);
        const float mean = s.x * inv;
        gm = s.y * inv;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int i = 0; i < E; ++i) v[j][i] = c0 + j * cs < a.C ? v[j][i] - mean : 0.f;
      }
      float q0 = 0.f, q1 = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          q0 = fmaf(v[j][i], v[j][i], q0);
          q1 = fmaf(d[j][i] * ma[j][i], v[j][i], q1);
        }
      const float2 q = group_sum(rg, q0, q1, sh.red[LAYER ? 1 : it & 1][rg.g]);
      const float rstd = rsqrtf(fmaf(q.x, inv, a.eps));
      const float proj = q.y * inv * rstd;           // mean(g * xhat)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = c0 + j * cs;
        if (c >= a.C) continue;
        float o[E], e[E];
        if (DR) read_piece<E, TX>(at + (j * kEach + kD) * nt, o);
        if (BRANCH) read_piece<E, TY>(at + (j * kEach + kB) * nt, e);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float xh = v[j][i] * rstd;
          sa[j][i] = fmaf(d[j][i], xh, sa[j][i]);
          sb[j][i] += d[j][i];
          const float in = fmaf(d[j][i], ma[j][i], -gm) - xh * proj;
          o[i] = DR ? fmaf(rstd, in, o[i]) : rstd * in;
          if (BRANCH) sg[j][i] = fmaf(o[i], e[i], sg[j][i]);
        }
        store_piece<E>(dx + row * a.C + c, o);
        if (BRANCH) {
#pragma unroll
          for (int i = 0; i < E; ++i) o[i] *= mg[j][i];
          store_piece<E>(dbranch + row * a.C + c, o);
        }
      }
    }
    slot = slot == kAhead - 1 ? 0 : slot + 1;
    open = now.next(a, segs, groups);
    if (!open) continue;
#pragma unroll
    for (int j = 0; j < V; ++j) {      // the segment's sums
      const int c = c0 + j * cs;
      if (c >= a.C) continue;
      if (BRANCH && gate) {
        store_floats<E>(dgate + seg * sum_stride + c, sg[j]);
#pragma unroll
        for (int i = 0; i < E; ++i) sg[j][i] = 0.f;
      }
      if (scale) {
        store_floats<E>(dscale + seg * sum_stride + c, sa[j]);
        store_floats<E>(dshift + seg * sum_stride + c, sb[j]);
#pragma unroll
        for (int i = 0; i < E; ++i) sa[j][i] = sb[j][i] = 0.f;
      }
    }
  }
  copy_wait<0>();
  if (weight)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = c0 + j * cs;
      if (c < a.C) {
        store_floats<E>(wsum + group * 2 * a.C + c, sa[j]);
        store_floats<E>(wsum + (group * 2 + 1) * a.C + c, sb[j]);
      }
    }
}

// Sums `parts` consecutive partial rows of `sums` vectors of C for each of gridDim.z outputs
// rows; blockIdx.y picks the vector and its output.
__global__ void __launch_bounds__(1024) gated_norm_reduce_kernel(const float* __restrict__ part, int parts,
                                                                 int sums, int C, float* o0, float* o1, float* o2) {
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  column_sum(part + ((size_t)blockIdx.z * parts * sums + blockIdx.y) * C, (unsigned)parts, (size_t)sums * C, C, 1,
             out + (size_t)blockIdx.z * C);
}

// Groups of a full grid, at most one per segment.
int blocks_for(const RowShape& s, long long segs) {
  const int per = kThreadsPerSM / s.threads;
  const long long most = (long long)kRowSMs * (per < 1 ? 1 : per), want = (segs + s.G - 1) / s.G;
  return (int)(want < most ? want : most);
}

static_assert(kRing + sizeof(Shared) <= kMostSharedMemory, "the ring and the sums fit");

template <typename TX, typename TY, int E, bool LAYER, bool BRANCH, int V>
cudaError_t forward_v(const GatedNormArgs& a, const RowShape& s, const void* x, const void* branch, const float* gate,
                      const float* scale, const float* shift, const float* weight, const float* bias, void* r, void* y,
                      cudaStream_t st) {
  auto* kern = gated_norm_kernel<TX, TY, E, LAYER, BRANCH, V>;
  constexpr int kRow = V * (piece_bytes<E, TX>() + (BRANCH ? piece_bytes<E, TY>() : 0));
  static_assert((size_t)kDeep * kRow * widest(E, V) <= kRing, "the forward's rows always fit three times");
  const size_t smem = (size_t)kDeep * kRow * s.threads;
  const cudaError_t e = allow_shared_memory<kRing>(kern, smem);
  if (e != cudaSuccess) return e;
  kern<<<blocks_for(s, (long long)a.B * a.T * a.chunks), s.threads, smem, st>>>(
      a, s.W, (const TX*)x, (const TY*)branch, gate, scale, shift, weight, bias, (TX*)r, (TY*)y);
  return cudaGetLastError();
}

// Calls go with the shape's V as a constant.
template <int E, typename F>
cudaError_t with_shape(const RowShape& s, const F& go) {
  if constexpr (E == 4)
    if (s.V == 4) return go(std::integral_constant<int, 4>{});
  return s.V == 2 ? go(std::integral_constant<int, 2>{}) : go(std::integral_constant<int, 1>{});
}

template <typename TX, typename TY, typename... A>
cudaError_t forward(const GatedNormArgs& a, rola_norm_kind kind, const void* x, const void* branch, A... rest) {
  constexpr int E = sizeof(TX) == 4 ? 4 : 8;
  const RowShape s = shape_of(a.C, E);
  auto go = [&](auto layer, auto with) {
    constexpr bool L = decltype(layer)::value, B = decltype(with)::value;
    return with_shape<E>(s, [&](auto v) {
      return forward_v<TX, TY, E, L, B, decltype(v)::value>(a, s, x, branch, rest...);
    });
  };
  using Y = std::true_type;
  using N = std::false_type;
  if (kind == ROLA_LAYER) return branch ? go(Y{}, Y{}) : go(Y{}, N{});
  return branch ? go(N{}, Y{}) : go(N{}, N{});
}

template <typename TX, typename TY, int E, bool LAYER, bool DR, bool BRANCH, int V, int kAhead, int kMost>
cudaError_t backward_v(const GatedNormArgs& a, const RowShape& s, const void* dy, const void* dr, const void* r,
                       const void* branch, const float* gate, const float* scale, const float* weight, void* dx,
                       void* dbranch, float* dgate, float* dscale, float* dshift, float* dweight, float* dbias,
                       float* part, cudaStream_t st) {
  auto* kern = gated_norm_backward_kernel<TX, TY, E, LAYER, DR, BRANCH, V, kAhead, kMost>;
  constexpr int kBx = piece_bytes<E, TX>(), kBy = piece_bytes<E, TY>();
  const size_t smem = (size_t)kAhead * V * (kBx * (DR ? 2 : 1) + kBy * (BRANCH ? 2 : 1)) * s.threads;
  cudaError_t e = allow_shared_memory<kRing>(kern, smem);
  if (e != cudaSuccess) return e;
  const long long mods = (long long)a.B * a.T;
  const int blocks = blocks_for(s, mods * a.chunks);
  const bool direct = a.chunks == 1;   // a segment's sums are the gradients
  float* msum = part;
  float* wsum = part + (direct || !(gate || scale) ? 0 : mods * a.chunks * 3 * a.C);
  kern<<<blocks, s.threads, smem, st>>>(a, s.W, (const TY*)dy, (const TX*)dr, (const TX*)r, (const TY*)branch, gate,
                                        scale, weight, (TX*)dx, (TY*)dbranch, direct ? dgate : msum,
                                        direct ? dscale : msum + a.C, direct ? dshift : msum + 2 * a.C,
                                        (direct ? 1 : 3) * (int64_t)a.C, wsum);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned cols = (a.C + kSumCols - 1) / kSumCols;
  const dim3 sums(kSumCols, kSumRows);
  if (!direct && (gate || scale))      // more than one chunk: fewer modulation rows than groups
    gated_norm_reduce_kernel<<<dim3(cols, 3, (unsigned)mods), sums, 0, st>>>(msum, a.chunks, 3, a.C, dgate, dscale,
                                                                             dshift);
  if (weight)
    gated_norm_reduce_kernel<<<dim3(cols, 2, 1), sums, 0, st>>>(wsum, blocks * s.G, 2, a.C, dweight, dbias, nullptr);
  return cudaGetLastError();
}

// A block is compiled for up to 320, 384 or 512 threads.  384 leave a thread 168 registers and 512 leave
// 128, at which the wide rows spill: 27300 rows of 6144 channels with dr and branch, 384 threads, take
// 639 us (x fp32, branch bf16) and 403 (bf16) compiled for 384, 1020 and 750 for 512.  320 leave 168 as
// well, but give other code: compiled for 384 instead, 2048 bf16 channels take 369 us, not 352, and
// 2048 of fp32 and bf16 without dr and branch 366, not 337.
// Three rows in flight where they fit into the ring, else one (with one throughout, the backward of
// 32760 x 5120 takes 741 us, not 571; only rows of more than 4096 fp32 channels or so do not fit).
template <typename TX, typename TY, typename... A>
cudaError_t backward(const GatedNormArgs& a, rola_norm_kind kind, const void* dy, const void* dr, const void* r,
                     const void* branch, A... rest) {
  constexpr int E = sizeof(TX) == 4 ? 4 : 8, kBx = piece_bytes<E, TX>(), kBy = piece_bytes<E, TY>();
  const RowShape s = shape_of(a.C, E);
  using Y = std::true_type;
  using N = std::false_type;
  auto go = [&](auto layer, auto add, auto with) {
    constexpr bool L = decltype(layer)::value, D = decltype(add)::value, B = decltype(with)::value;
    return with_shape<E>(s, [&](auto v) {
      constexpr int V = decltype(v)::value, kMost = widest(E, V);
      constexpr size_t kRows = (size_t)kDeep * V * (kBx * (D ? 2 : 1) + kBy * (B ? 2 : 1));   // bytes of a thread
      const bool deep = kRows * s.threads <= kRing;
      // blocks of kLeast to kBound threads: with three rows in flight, or one, where some width takes it
      auto most = [&](auto least, auto bound) {
        constexpr int kLeast = decltype(least)::value, kBound = decltype(bound)::value;
        constexpr int kWidest = kBound < kMost ? kBound : kMost;
        if constexpr (kRows * kWidest > kRing)
          if (!deep) return backward_v<TX, TY, E, L, D, B, V, 1, kBound>(a, s, dy, dr, r, branch, rest...);
        if constexpr (kRows * kLeast <= kRing)
          return backward_v<TX, TY, E, L, D, B, V, kDeep, kBound>(a, s, dy, dr, r, branch, rest...);
        else
          return cudaErrorInvalidValue;
      };
      if constexpr (kMost > 320) {
        if (s.threads > 384) return most(std::integral_constant<int, 416>{}, std::integral_constant<int, kMost>{});
        if (s.threads > 320) return most(std::integral_constant<int, 352>{}, std::integral_constant<int, 384>{});
      }
      return most(std::integral_constant<int, 32>{}, std::integral_constant<int, 320>{});
    });
  };
  auto pick = [&](auto layer) {
    if (dr) return branch ? go(layer, Y{}, Y{}) : go(layer, Y{}, N{});
    return branch ? go(layer, N{}, Y{}) : go(layer, N{}, N{});
  };
  return kind == ROLA_LAYER ? pick(Y{}) : pick(N{});
}

}  // namespace

// Rows that a partial sum of the backward is worth: with a group per row the sums of 2331 rows of
// 1000 channels were as large as the rows (fp32: 13 + 11 us; with four rows a group 9 + 6), while
// four groups an SM keep loads enough in flight.
constexpr int kRowsPerSum = 4;

// Chunks of the tokens that share a modulation row: a segment for every group of a full grid,
// and no more (each costs a row of partial sums).
void gated_norm_chunks(const rola_gated_norm_params& p, bool back, int* chunks, int* chunk) {
  const RowShape s = shape_of(p.C, piece_of(p.x_dtype, p.y_dtype));
  const int per = p.N / p.T;
  const long long mods = (long long)p.B * p.T;
  const long long rows = (long long)p.B * p.N, sums = rows / kRowsPerSum;
  const long long few = sums > 4 * kRowSMs ? sums : 4 * kRowSMs;
  long long groups = (long long)blocks_for(s, rows) * s.G;
  if (back && groups > few) groups = few;
  long long want = (groups + mods - 1) / mods;
  if (want > per) want = per;
  *chunk = (int)((per + want - 1) / want);
  *chunks = (per - 1) / *chunk + 1;
}

size_t gated_norm_workspace(const rola_gated_norm_params& p) {
  int chunks, chunk;
  gated_norm_chunks(p, true, &chunks, &chunk);
  const long long segs = (long long)p.B * p.T * chunks;
  const RowShape s = shape_of(p.C, piece_of(p.x_dtype, p.y_dtype));
  return sizeof(float) * (size_t)p.C * ((chunks > 1 ? 3 * segs : 0) + 2 * (long long)blocks_for(s, segs) * s.G);
}

cudaError_t launch_gated_norm(const GatedNormArgs& a, rola_dtype xt, rola_dtype yt, rola_norm_kind kind, const void* x,
                              const void* branch, const float* gate, const float* scale, const float* shift,
                              const float* weight, const float* bias, void* r, void* y, cudaStream_t st) {
  if (xt == ROLA_BF16)
    return forward<__nv_bfloat16, __nv_bfloat16>(a, kind, x, branch, gate, scale, shift, weight, bias, r, y, st);
  if (yt == ROLA_BF16)
    return forward<float, __nv_bfloat16>(a, kind, x, branch, gate, scale, shift, weight, bias, r, y, st);
  return forward<float, float>(a, kind, x, branch, gate, scale, shift, weight, bias, r, y, st);
}

cudaError_t launch_gated_norm_backward(const GatedNormArgs& a, rola_dtype xt, rola_dtype yt, rola_norm_kind kind,
                                       const void* dy, const void* dr, const void* r, const void* branch,
                                       const float* gate, const float* scale, const float* weight, void* dx,
                                       void* dbranch, float* dgate, float* dscale, float* dshift, float* dweight,
                                       float* dbias, float* part, cudaStream_t st) {
  if (xt == ROLA_BF16)
    return backward<__nv_bfloat16, __nv_bfloat16>(a, kind, dy, dr, r, branch, gate, scale, weight, dx, dbranch, dgate,
                                                  dscale, dshift, dweight, dbias, part, st);
  if (yt == ROLA_BF16)
    return backward<float, __nv_bfloat16>(a, kind, dy, dr, r, branch, gate, scale, weight, dx, dbranch, dgate, dscale,
                                          dshift, dweight, dbias, part, st);
  return backward<float, float>(a, kind, dy, dr, r, branch, gate, scale, weight, dx, dbranch, dgate, dscale, dshift,
                                dweight, dbias, part, st);
}

}  // namespace rola

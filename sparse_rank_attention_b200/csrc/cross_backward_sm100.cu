// Gradients of the cross attention on the sm_100a tensor cores (tcgen05 + TMEM + TMA), bf16,
// head dim 64 or 128.
//
//   P = 2^(S scale log2 e - lse log2 e);  dP = dO v^T;  dS = P (dP - D),  D = rowsum(dO * O)
//   dq = scale dS k;   dk = scale dS^T q;   dv = P^T dO
//
// P and dS are rounded to bf16 where they enter a product (the type of its other operand); S, dP
// and all sums are fp32.  Three kernels:
//
//   statistics   lse log2 e (+inf where a row has no valid key or lies past Nq, so that P = 0) and
//                D per row, in rows padded to 256; bound by the reads of dO and O.
//   dq           a block holds two query tiles of 128, A and B, and walks the key tiles: S, dP and
//                dQ += dS K, 3 products.  S and then dP take the same 128 columns of tensor memory
//                (P waits in registers), so that both tiles fit beside their dQ.  Eight warps per
//                query tile; with the statistics given no row needs an exchange between threads.
//   dk, dv       a block holds a key tile and walks a run of query tiles, on the transposed scores:
//                S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q, 4 products; P^T and dS^T
//                go over S^T and dP^T in tensor memory as A operands.  Queries are split over
//                blocks, the parts summed in a fixed order (no atomics: results repeat bit by bit).
//
// dq recomputes S and dP, two products of seven: the sums over key tiles for dq and over query
// tiles for dk, dv cannot both stay in one block's tensor memory, and adding dq up in global
// memory would need atomics.
//
// Measured: 32760 queries x 512 keys, 40 heads of 128, kv_len between half and all of the keys:
// 1600 to 1770 us: statistics 141 (0.67 GB, 4.8 TB/s), dq 720 (3 products), dk and dv 737 (4
// products), the sums of the parts 2 x 14.  As in the forward the chain of one tile bounds dq; in
// dk, dv two of the four products wait for P^T and dS^T of the tile that they belong to.
//
// Every mbarrier wait is bounded, as in the forward.
#include <climits>
#include <cuda.h>

#include "cross_sm100.cuh"
#include "row_ops.cuh"

namespace rola {
namespace {

using namespace sm100;

__device__ int g_status[1];

constexpr unsigned long long kLimitCycles = 2000000000ull;   // 1 s at 2 GHz

// ------------------------------------------------------------------ statistics

// zl = lse log2 e (infinity for rows without keys and rows past Nq: P = 0), zd = D = rowsum(dO * O),
// both [B, H, padded].  d / 8 threads per row, one row each, in 32-bit indices of a sample (with
// 64-bit divisions it was bound by them: 147 us at 32760 x 40 x 128, now 141; four rows per thread
// take 180).
template <int D>
__global__ void __launch_bounds__(256) cross_stats_kernel(const __grid_constant__ CrossArgs a, unsigned padded,
                                                          const __nv_bfloat16* __restrict__ dout,
                                                          const __nv_bfloat16* __restrict__ out,
                                                          const float* __restrict__ lse, float* __restrict__ zl,
                                                          float* __restrict__ zd) {
  constexpr int kPer = D / kVec;
  const unsigned row = blockIdx.x * (256 / kPer) + threadIdx.x / kPer, n = row / (unsigned)a.H, h = row - n * a.H;
  const int c = (threadIdx.x % kPer) * kVec, b = blockIdx.y;
  float s = 0.f;
  const bool on = n < (unsigned)a.Nq;
  if (on) {
    float u[kVec], v[kVec];
    load8(dout + b * a.dout.b + (int64_t)n * a.dout.n + (int64_t)h * a.dout.h + c, u);
    load8(out + ((size_t)b * a.Nq * a.H + row) * D + c, v);
#pragma unroll
    for (int i = 0; i < kVec; ++i) s = fmaf(u[i], v[i], s);
  }
#pragma unroll
  for (int o = kPer / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (c != 0 || n >= padded) return;
  const size_t head = (size_t)b * a.H + h, at = head * padded + n;
  const float z = on ? __ldg(lse + head * a.Nq + n) : -INFINITY;
  zl[at] = z == -INFINITY ? INFINITY : z * 1.4426950408889634f;
  zd[at] = s;
}

// Ring index arithmetic of a role: the n'th use of an S-deep ring.
template <int S>
struct Ring {
  static __device__ __forceinline__ int slot(int n) { return n % S; }
  static __device__ __forceinline__ uint32_t full(int n) { return (n / S) & 1; }
  static __device__ __forceinline__ uint32_t empty(int n) { return ((n / S) - 1) & 1; }   // n >= S
};

// ------------------------------------------------------------------ dq

constexpr int kDqThreads = 640;

template <int D>
struct DqGeo {
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kTileBytes = kBoxes * kBox;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr uint32_t kOffQ = 0;                 // Q of A, B
  static constexpr uint32_t kOffDo = 2 * kTileBytes;   // dO of A, B
  static constexpr uint32_t kOffKV = 4 * kTileBytes;
  static constexpr uint32_t kOffCtl = kOffKV + kStages * kTileBytes;
  static constexpr uint32_t kColS = 0;                 // S, dP, dS of A, B
  static constexpr uint32_t kColO = 256;               // dQ of A, B
};
struct DqCtl {
  uint64_t q_full[2], q_empty[2], do_full[2], do_empty[2], k_full[6], v_full[6], k_ready[6], kv_empty[6];
  uint64_t s_full[2], p_read[2], dp_full[2], ds_full[2], dq_done[2], o_free[2], drain;
  uint32_t tmem;
  int abort;
};
template <int D>
constexpr size_t dq_smem() { return DqGeo<D>::kOffCtl + sizeof(DqCtl) + 1024; }

template <int D>
__global__ void __launch_bounds__(kDqThreads, 1) cross_dq_sm100_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const __grid_constant__ CrossArgs a, const __grid_constant__ Work w, const float* __restrict__ zl,
    const float* __restrict__ zd, __nv_bfloat16* __restrict__ dq, float* __restrict__ part) {
  using G = DqGeo<D>;
  using R = Ring<G::kStages>;
  constexpr int kStages = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  DqCtl* ctl = reinterpret_cast<DqCtl*>(base + G::kOffCtl);
  const uint32_t sbase = smem_addr(base);
  // uniform for the compiler too
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto bar = [&](uint64_t& m) { return smem_addr(&m); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(ctl->q_full[s]), 1);
      mbar_init(bar(ctl->q_empty[s]), 1);
      mbar_init(bar(ctl->do_full[s]), 1);
      mbar_init(bar(ctl->do_empty[s]), 1);
      mbar_init(bar(ctl->s_full[s]), 1);
      mbar_init(bar(ctl->p_read[s]), 8);     // one arrive per warp of the query tile
      mbar_init(bar(ctl->dp_full[s]), 1);
      mbar_init(bar(ctl->ds_full[s]), 8);
      mbar_init(bar(ctl->dq_done[s]), 1);
      mbar_init(bar(ctl->o_free[s]), 8);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(ctl->k_full[s]), 1);
      mbar_init(bar(ctl->v_full[s]), 1);
      mbar_init(bar(ctl->k_ready[s]), 1);
      mbar_init(bar(ctl->kv_empty[s]), 1);
    }
    mbar_init(bar(ctl->drain), 1);
    ctl->abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&ctl->tmem), 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);
  const WaitCtl wc{&ctl->abort, g_status, kLimitCycles};

  if (warp == 0) {
    // ------------------------------------------------------------ loads: Q, dO; K, V, K, V, ...
    if (lane == 0) {
      int nq[2] = {0, 0}, nkv = 0, nk = 0, nv = 0;   // items of A, B; K and V tiles; K; V
      bool ok = true;
      Item x{};
      auto load = [&](uint32_t dst, const CUtensorMap* tm, int n, uint32_t full) {
        mbar_expect_tx(full, G::kTileBytes);
        for (int c = 0; c < G::kBoxes; ++c) tma_load_4d(dst + c * kBox, tm, 64 * c, x.h, n, x.b, full);
      };
      // K and V tiles share the slots in turn; each kind has its own full barriers, as in the forward
      auto load_kv = [&](const CUtensorMap* tm, uint64_t* full, int& n, int t) {
        const int s = R::slot(nkv);
        if (nkv >= kStages && !mbar_wait(bar(ctl->kv_empty[s]), R::empty(nkv), wc)) return false;
        load(sbase + G::kOffKV + s * G::kTileBytes, tm, t * kTile, bar(full[R::slot(n)]));
        ++nkv;
        ++n;
        return true;
      };
      for (int i = next_item(a, w, blockIdx.x, &x); ok && i < w.items; i = next_item(a, w, i + gridDim.x, &x)) {
        for (int s = 0; ok && s < x.streams; ++s) {
          if (nq[s] >= 1 && !mbar_wait(bar(ctl->q_empty[s]), (nq[s] - 1) & 1, wc)) { ok = false; break; }
          load(sbase + G::kOffQ + s * G::kTileBytes, &tm_q, x.q0 + s * kTile, bar(ctl->q_full[s]));
          if (s == 0) ok = load_kv(&tm_k, ctl->k_full, nk, x.t0);
        }
        for (int s = 0; ok && s < x.streams; ++s) {
          if (nq[s] >= 1 && !mbar_wait(bar(ctl->do_empty[s]), (nq[s] - 1) & 1, wc)) { ok = false; break; }
          load(sbase + G::kOffDo + s * G::kTileBytes, &tm_do, x.q0 + s * kTile, bar(ctl->do_full[s]));
          ++nq[s];
        }
        for (int t = x.t0; ok && t < x.t1; ++t) {
          ok = load_kv(&tm_v, ctl->v_full, nv, t);
          if (ok && t + 1 < x.t1) ok = load_kv(&tm_k, ctl->k_full, nk, t + 1);
        }
        if (!ok) {   // a Q whose dO was not issued: it too lands before the block leaves
          for (int s = 0; s < 2; ++s) mbar_wait(bar(ctl->q_full[s]), nq[s] & 1, wc, false);
        }
      }
      for (int s = 0; s < 2; ++s)
        if (nq[s] > 0) {
          mbar_wait(bar(ctl->q_full[s]), (nq[s] - 1) & 1, wc, false);
          mbar_wait(bar(ctl->do_full[s]), (nq[s] - 1) & 1, wc, false);
        }
      for (int y = nk > kStages ? nk - kStages : 0; y < nk; ++y)
        mbar_wait(bar(ctl->k_full[R::slot(y)]), R::full(y), wc, false);
      for (int y = nv > kStages ? nv - kStages : 0; y < nv; ++y)
        mbar_wait(bar(ctl->v_full[R::slot(y)]), R::full(y), wc, false);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    int steps[2] = {0, 0}, nq[2] = {0, 0}, no[2] = {0, 0};   // tiles, items of a query tile
    int nkv = 0, nkt = 0;                                     // K and V tiles, K tiles alone
    bool ok = true;
    auto wait = [&](uint64_t& m, uint32_t parity) { return warp_wait(m, parity, wc); };
    auto slot = [&](int n) { return sbase + G::kOffKV + R::slot(n) * G::kTileBytes; };
    auto commit = [&](uint64_t& m) {
      if (elect_leader()) mma_commit(bar(m));
      __syncwarp();
    };
    // S of the next tile takes the columns of dS: dQ of the previous tile must be done
    auto issue_s = [&](int s, int n, int kt, bool first, bool last) {
      if (first && !wait(ctl->q_full[s], nq[s] & 1)) return false;
      if (!wait(ctl->k_ready[R::slot(kt)], R::full(kt))) return false;
      if (steps[s] > 0 && !wait(ctl->dq_done[s], (steps[s] - 1) & 1)) return false;
      tc_fence_after();
      if (elect_leader()) {
        product_ss<D>(tmem + G::kColS + 128 * s, sbase + G::kOffQ + s * G::kTileBytes, slot(n));
        mma_commit(bar(ctl->s_full[s]));
        if (last) mma_commit(bar(ctl->q_empty[s]));
      }
      __syncwarp();
      return true;
    };
    Item x{}, y{};
    int i = next_item(a, w, blockIdx.x, &x);
    if (i < w.items)
      for (int s = 0; ok && s < x.streams; ++s) ok = issue_s(s, 0, 0, true, x.t1 == x.t0 + 1);
    while (ok && i < w.items) {
      const int i2 = next_item(a, w, i + gridDim.x, &y);
      for (int t = x.t0; ok && t < x.t1; ++t) {
        const bool first = t == x.t0, more = t + 1 < x.t1;
        const int next_streams = more ? x.streams : i2 < w.items ? y.streams : 0;
        const int n_k = nkv, n_v = nkv + 1, n_next = nkv + 2;
#pragma unroll
        for (int s = 0; s < 2; ++s) {                         // dP = dO V^T once S has been read
          if (!ok || s >= x.streams) break;
          if (first) ok = wait(ctl->do_full[s], nq[s] & 1);
          ok = ok && wait(ctl->v_full[R::slot(nkt)], R::full(nkt)) &&   // V tile as many as K tile
               wait(ctl->p_read[s], steps[s] & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_leader()) {
            product_ss<D>(tmem + G::kColS + 128 * s, sbase + G::kOffDo + s * G::kTileBytes, slot(n_v));
            mma_commit(bar(ctl->dp_full[s]));
            if (!more) mma_commit(bar(ctl->do_empty[s]));
          }
          __syncwarp();
          nq[s] += !more;
        }
        if (!ok) break;
        commit(ctl->kv_empty[R::slot(n_v)]);
#pragma unroll
        for (int s = 0; s < 2; ++s) {                         // dQ += dS K
          if (!ok || s >= x.streams) break;
          if (first && no[s]++ > 0) ok = wait(ctl->o_free[s], (no[s] - 2) & 1);
          ok = ok && wait(ctl->ds_full[s], steps[s] & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_leader()) {
            product_ts<D>(tmem + G::kColO + D * s, tmem + G::kColS + 128 * s, 64, slot(n_k), !first);
            mma_commit(bar(ctl->dq_done[s]));
          }
          __syncwarp();
          ++steps[s];
        }
        if (!ok) break;
        commit(ctl->kv_empty[R::slot(n_k)]);
        nkv += 2;
        ++nkt;
#pragma unroll
        for (int s = 0; s < 2; ++s)
          if (ok && s < next_streams) ok = issue_s(s, n_next, nkt, !more, more ? t + 2 == x.t1 : y.t1 == y.t0 + 1);
      }
      x = y;
      i = i2;
    }
    commit(ctl->drain);
    mbar_wait(bar(ctl->drain), 0, wc, false);
  } else if (warp == 2) {
    // ------------------------------------------------------------ K rows that do not count (0 * NaN in dS K)
    int nkt = 0;
    bool ok = true;
    Item x{};
    for (int i = next_item(a, w, blockIdx.x, &x); ok && i < w.items; i = next_item(a, w, i + gridDim.x, &x)) {
      const int len = key_count(a, x.b);
      for (int t = x.t0; t < x.t1; ++t, ++nkt) {
        const int n = 2 * nkt, s = R::slot(n);
        uint32_t bits[4];
        tile_bits(a, x.b, len, t, lane, bits);
        ok = __all_sync(0xffffffffu, mbar_wait(bar(ctl->k_full[R::slot(nkt)]), R::full(nkt), wc));
        if (!ok) break;
        if (!all_set(bits)) {
          clear_rows<G::kBoxes>(base + G::kOffKV + s * G::kTileBytes, bits, lane);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ctl->k_ready[R::slot(nkt)]));
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ P, dS and results
    // Eight warps per query tile: thread (row, half) has the row's keys 64 half .. 64 half + 63.
    const int s = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, wq = warp & 3, row = 32 * wq + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * wq) << 16);
    const uint32_t t_s = lane_addr + G::kColS + 128 * s + 64 * half, gbar = 1 + s;
    const uint32_t t_o = lane_addr + G::kColO + D * s + (D / 2) * half;
    const float sl2 = a.scale * 1.4426950408889634f;
    int step = 0;
    bool fail = false;
    for (int i = blockIdx.x; i < w.items; i += gridDim.x) {
      const Item x = item_at(a, w, i);
      if (s >= x.streams) continue;
      const int len = key_count(a, x.b), n = x.q0 + s * kTile + row;
      const size_t zat = ((size_t)x.b * a.H + x.h) * w.padded + n;
      const float zn = -__ldg(zl + zat), dn = -__ldg(zd + zat);
      for (int t = x.t0; t < x.t1; ++t, ++step) {
        uint32_t bits[4];
        const bool partial = a.key_mask || (t + 1) * kTile > len;
        if (partial) tile_bits(a, x.b, len, t, lane, bits);
        const uint32_t b0 = partial ? (half ? bits[2] : bits[0]) : 0xffffffffu;
        const uint32_t b1 = partial ? (half ? bits[3] : bits[1]) : 0xffffffffu;
        fail |= !mbar_wait(bar(ctl->s_full[s]), step & 1, wc);
        if (__any_sync(0xffffffffu, fail)) break;
        tc_fence_after();
        float p[64];
        tmem_ld32(t_s, p);
        tmem_ld32(t_s + 32, p + 32);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ctl->p_read[s]));      // S is in registers
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          fma2(p[c], p[c + 1], p[c], p[c + 1], sl2, sl2, zn, zn);
          p[c] = ex2_approx(p[c]);
          p[c + 1] = ex2_approx(p[c + 1]);
        }
        fail |= !mbar_wait(bar(ctl->dp_full[s]), step & 1, wc);
        if (__any_sync(0xffffffffu, fail)) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          float d[32], pk[16];
          tmem_ld32(t_s + c, d);
          tmem_wait_ld();
          const uint32_t valid = c ? b1 : b0;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            add2(d[e], d[e + 1], dn, dn);
            mul2(d[e], d[e + 1], p[c + e], p[c + e + 1]);
            if (partial) {
              if (!((valid >> e) & 1u)) d[e] = 0.f;
              if (!((valid >> (e + 1)) & 1u)) d[e + 1] = 0.f;
            }
            pk[e >> 1] = __uint_as_float(pack_bf16(d[e], d[e + 1]));
          }
          tmem_st16(t_s + (c >> 1), pk);   // columns that this thread has read
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ctl->ds_full[s]));
      }
      if (named_vote_or(gbar, 256, fail)) break;
      const bool none = x.t1 == x.t0;
      if (!none) fail |= !mbar_wait(bar(ctl->dq_done[s]), (step - 1) & 1, wc);
      if (named_vote_or(gbar, 256, fail)) break;
      tc_fence_after();
      const size_t at = (((size_t)x.b * a.Nq + n) * a.H + x.h) * D + (D / 2) * half;
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 32) {
        float o[32];
        if (none) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        } else {
          tmem_ld32(t_o + c, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= a.scale;
        if (n < a.Nq) {
#pragma unroll
          for (int e = 0; e < 32; e += kVec) {
            if (w.splits == 1)
              store8(dq + at + c + e, o + e);
            else
              store8(part + (size_t)x.split * a.B * a.Nq * a.H * D + at + c + e, o + e);
          }
        }
      }
      if (!none) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ctl->o_free[s]));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dk, dv

constexpr int kDkvThreads = 384;
constexpr int kQStages = 2;   // Q and dO tiles in flight

template <int D>
struct DkvGeo {
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kTileBytes = kBoxes * kBox;
  static constexpr uint32_t kOffK = 0, kOffV = kTileBytes;
  static constexpr uint32_t kOffQ = 2 * kTileBytes;                         // [stage]
  static constexpr uint32_t kOffDo = kOffQ + kQStages * kTileBytes;         // [stage]
  static constexpr uint32_t kOffZ = kOffDo + kQStages * kTileBytes;         // [stage][lse | D][128]
  static constexpr uint32_t kOffCtl = kOffZ + kQStages * 1024;
  static constexpr uint32_t kColS = 0, kColP = 128;                         // S^T, dP^T
  static constexpr uint32_t kColV = 256, kColK = 384;                       // dV, dK
};
struct DkvCtl {
  uint64_t k_full, k_empty, q_full[kQStages], q_empty[kQStages], do_full[kQStages], do_empty[kQStages];
  uint64_t s_full, p_full, dp_full, ds_full, dv_done, dk_done, o_free, drain;
  uint32_t tmem;
  int abort;
};
template <int D>
constexpr size_t dkv_smem() { return DkvGeo<D>::kOffCtl + sizeof(DkvCtl) + 1024; }

// One work item: a key tile of a head over a run of query tiles.
struct KeyItem {
  int b, h, m0, split, t0, t1;
};
struct KeyWork {
  int ktiles, splits, run, qtiles, padded, items;
};
__device__ __forceinline__ KeyItem key_item_at(const CrossArgs& a, const KeyWork& w, int i) {
  KeyItem x;
  const int bh = i / (w.ktiles * w.splits), rest = i - bh * w.ktiles * w.splits;
  // key tiles innermost: the blocks at work share the query tiles of a run
  x.split = rest / w.ktiles;
  x.m0 = (rest - x.split * w.ktiles) * kTile;
  x.b = bh / a.H;
  x.h = bh - x.b * a.H;
  x.t0 = x.split * w.run;
  x.t1 = x.m0 < key_count(a, x.b) ? max(x.t0, min(w.qtiles, x.t0 + w.run)) : x.t0;
  return x;
}
__device__ __forceinline__ int next_key_item(const CrossArgs& a, const KeyWork& w, int i, KeyItem* x) {
  for (; i < w.items; i += gridDim.x) {
    *x = key_item_at(a, w, i);
    if (x->t1 > x->t0) return i;
  }
  return w.items;
}

template <int D>
__global__ void __launch_bounds__(kDkvThreads, 1) cross_dkv_sm100_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const __grid_constant__ CrossArgs a, const __grid_constant__ KeyWork w, const float* __restrict__ zl,
    const float* __restrict__ zd, __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv,
    float* __restrict__ part) {
  using G = DkvGeo<D>;
  using R = Ring<kQStages>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  DkvCtl* ctl = reinterpret_cast<DkvCtl*>(base + G::kOffCtl);
  const uint32_t sbase = smem_addr(base);
  // uniform for the compiler too
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto bar = [&](uint64_t& m) { return smem_addr(&m); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kQStages; ++s) {
      mbar_init(bar(ctl->q_full[s]), 1);
      mbar_init(bar(ctl->q_empty[s]), 1);
      mbar_init(bar(ctl->do_full[s]), 1);
      mbar_init(bar(ctl->do_empty[s]), 1);
    }
    mbar_init(bar(ctl->k_full), 1);
    mbar_init(bar(ctl->k_empty), 1);
    mbar_init(bar(ctl->s_full), 1);
    mbar_init(bar(ctl->p_full), 8);          // one arrive per warp
    mbar_init(bar(ctl->dp_full), 1);
    mbar_init(bar(ctl->ds_full), 8);
    mbar_init(bar(ctl->dv_done), 1);
    mbar_init(bar(ctl->dk_done), 1);
    mbar_init(bar(ctl->o_free), 8);
    mbar_init(bar(ctl->drain), 1);
    ctl->abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&ctl->tmem), 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem, 0);
  const WaitCtl wc{&ctl->abort, g_status, kLimitCycles};

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    // Q comes with the rows' lse and D (bulk copies of 512 bytes): its slot is free after dK,
    // when both have been read.
    if (lane == 0) {
      int nk = 0, nq = 0, ndo = 0;
      bool ok = true;
      KeyItem x{};
      auto load = [&](uint32_t dst, const CUtensorMap* tm, int n, uint32_t full, int tiles, uint32_t more) {
        mbar_expect_tx(full, tiles * G::kTileBytes + more);
        for (int c = 0; c < G::kBoxes; ++c) tma_load_4d(dst + c * kBox, tm, 64 * c, x.h, n, x.b, full);
      };
      for (int i = next_key_item(a, w, blockIdx.x, &x); ok && i < w.items; i = next_key_item(a, w, i + gridDim.x, &x)) {
        if (nk >= 1 && !mbar_wait(bar(ctl->k_empty), (nk - 1) & 1, wc)) break;
        load(sbase + G::kOffK, &tm_k, x.m0, bar(ctl->k_full), 2, 0);
        for (int c = 0; c < G::kBoxes; ++c)
          tma_load_4d(sbase + G::kOffV + c * kBox, &tm_v, 64 * c, x.h, x.m0, x.b, bar(ctl->k_full));
        ++nk;
        const size_t zrow = ((size_t)x.b * a.H + x.h) * w.padded;
        for (int t = x.t0; t < x.t1; ++t) {
          const int s = R::slot(nq);
          const uint32_t z = sbase + G::kOffZ + s * 1024;
          if (nq >= kQStages && !mbar_wait(bar(ctl->q_empty[s]), R::empty(nq), wc)) { ok = false; break; }
          load(sbase + G::kOffQ + s * G::kTileBytes, &tm_q, t * kTile, bar(ctl->q_full[s]), 1, 1024);
          bulk_load(z, zl + zrow + t * kTile, 512, bar(ctl->q_full[s]));
          bulk_load(z + 512, zd + zrow + t * kTile, 512, bar(ctl->q_full[s]));
          ++nq;
          if (ndo >= kQStages && !mbar_wait(bar(ctl->do_empty[s]), R::empty(ndo), wc)) { ok = false; break; }
          load(sbase + G::kOffDo + s * G::kTileBytes, &tm_do, t * kTile, bar(ctl->do_full[s]), 1, 0);
          ++ndo;
        }
      }
      if (nk > 0) mbar_wait(bar(ctl->k_full), (nk - 1) & 1, wc, false);
      for (int y = nq > kQStages ? nq - kQStages : 0; y < nq; ++y)
        mbar_wait(bar(ctl->q_full[R::slot(y)]), R::full(y), wc, false);
      for (int y = ndo > kQStages ? ndo - kQStages : 0; y < ndo; ++y)
        mbar_wait(bar(ctl->do_full[R::slot(y)]), R::full(y), wc, false);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    int step = 0, items = 0;   // query tiles and items begun
    bool ok = true;
    auto wait = [&](uint64_t& m, uint32_t parity) { return warp_wait(m, parity, wc); };
    auto q_tile = [&](int n) { return sbase + G::kOffQ + R::slot(n) * G::kTileBytes; };
    auto do_tile = [&](int n) { return sbase + G::kOffDo + R::slot(n) * G::kTileBytes; };
    // S^T of tile n of the sequence; its columns held P^T of the tile before
    auto issue_s = [&](int n) {
      if (!wait(ctl->q_full[R::slot(n)], R::full(n))) return false;
      if (n > 0 && !wait(ctl->dv_done, (n - 1) & 1)) return false;
      tc_fence_after();
      if (elect_leader()) {
        product_ss<D>(tmem + G::kColS, sbase + G::kOffK, q_tile(n));
        mma_commit(bar(ctl->s_full));
      }
      __syncwarp();
      return true;
    };
    auto issue_dp = [&](int n) {
      if (!wait(ctl->do_full[R::slot(n)], R::full(n))) return false;
      if (n > 0 && !wait(ctl->dk_done, (n - 1) & 1)) return false;
      tc_fence_after();
      if (elect_leader()) {
        product_ss<D>(tmem + G::kColP, sbase + G::kOffV, do_tile(n));
        mma_commit(bar(ctl->dp_full));
      }
      __syncwarp();
      return true;
    };
    KeyItem x{};
    for (int i = next_key_item(a, w, blockIdx.x, &x); ok && i < w.items; i = next_key_item(a, w, i + gridDim.x, &x)) {
      ok = wait(ctl->k_full, items & 1) && issue_s(step) && issue_dp(step);
      if (ok && items > 0) ok = wait(ctl->o_free, (items - 1) & 1);
      ++items;
      for (int t = x.t0; ok && t < x.t1; ++t, ++step) {
        const bool more = t + 1 < x.t1;
        ok = wait(ctl->p_full, step & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_leader()) {
          product_ts<D>(tmem + G::kColV, tmem + G::kColS, 64, do_tile(step), t > x.t0);
          mma_commit(bar(ctl->dv_done));
          mma_commit(bar(ctl->do_empty[R::slot(step)]));   // dP of this tile was issued before
        }
        __syncwarp();
        ok = (!more || issue_s(step + 1)) && wait(ctl->ds_full, step & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_leader()) {
          product_ts<D>(tmem + G::kColK, tmem + G::kColP, 64, q_tile(step), t > x.t0);
          mma_commit(bar(ctl->dk_done));
          mma_commit(bar(ctl->q_empty[R::slot(step)]));
          if (!more) mma_commit(bar(ctl->k_empty));
        }
        __syncwarp();
        if (more) ok = issue_dp(step + 1);
      }
    }
    if (elect_leader()) mma_commit(bar(ctl->drain));
    __syncwarp();
    mbar_wait(bar(ctl->drain), 0, wc, false);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ P^T, dS^T and results
    // Thread (row, half) has key m0 + row and the queries 64 half .. 64 half + 63 of each tile.
    const int half = (warp - 4) >> 2, wq = warp & 3, row = 32 * wq + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * wq) << 16);
    const uint32_t t_s = lane_addr + G::kColS + 64 * half, t_p = lane_addr + G::kColP + 64 * half;
    const float sl2 = a.scale * 1.4426950408889634f;
    int step = 0, items = 0;
    bool fail = false;
    for (int i = blockIdx.x; i < w.items; i += gridDim.x) {
      const KeyItem x = key_item_at(a, w, i);
      const int m = x.m0 + row;
      bool valid = m < key_count(a, x.b);
      if (valid && a.key_mask) valid = __ldg(a.key_mask + (size_t)x.b * a.Nk + m) != 0;
      for (int t = x.t0; t < x.t1; ++t, ++step) {
        const int st = R::slot(step);
        const float* z = reinterpret_cast<const float*>(base + G::kOffZ + st * 1024) + 64 * half;
        fail |= !mbar_wait(bar(ctl->q_full[st]), R::full(step), wc);      // the rows' lse and D
        fail |= !mbar_wait(bar(ctl->s_full), step & 1, wc);
        if (__any_sync(0xffffffffu, fail)) break;
        tc_fence_after();
        float p[64];
        tmem_ld32(t_s, p);
        tmem_ld32(t_s + 32, p + 32);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          float pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(z + c + e);
            float* q = p + c + e;
            fma2(q[0], q[1], q[0], q[1], sl2, sl2, -l4.x, -l4.y);
            fma2(q[2], q[3], q[2], q[3], sl2, sl2, -l4.z, -l4.w);
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = valid ? ex2_approx(q[j]) : 0.f;
            pk[e >> 1] = __uint_as_float(pack_bf16(q[0], q[1]));
            pk[(e >> 1) + 1] = __uint_as_float(pack_bf16(q[2], q[3]));
          }
          tmem_st16(t_s + (c >> 1), pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ctl->p_full));
        fail |= !mbar_wait(bar(ctl->dp_full), step & 1, wc);
        if (__any_sync(0xffffffffu, fail)) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          float d[32], pk[16];
          tmem_ld32(t_p + c, d);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 d4 = *reinterpret_cast<const float4*>(z + 128 + c + e);
            float* q = d + e;
            const float* pp = p + c + e;
            add2(q[0], q[1], -d4.x, -d4.y);
            add2(q[2], q[3], -d4.z, -d4.w);
            mul2(q[0], q[1], pp[0], pp[1]);
            mul2(q[2], q[3], pp[2], pp[3]);
            if (!valid) q[0] = q[1] = q[2] = q[3] = 0.f;
            pk[e >> 1] = __uint_as_float(pack_bf16(q[0], q[1]));
            pk[(e >> 1) + 1] = __uint_as_float(pack_bf16(q[2], q[3]));
          }
          tmem_st16(t_p + (c >> 1), pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ctl->ds_full));
      }
      if (named_vote_or(1, 256, fail)) break;
      const bool none = x.t1 == x.t0;
      if (!none) {
        fail |= !mbar_wait(bar(ctl->dv_done), (step - 1) & 1, wc);
        fail |= !mbar_wait(bar(ctl->dk_done), (step - 1) & 1, wc);
        ++items;
      }
      if (named_vote_or(1, 256, fail)) break;
      tc_fence_after();
      // the first half of the warps writes dV, the second dK
      const size_t at = (((size_t)x.b * a.Nk + m) * a.H + x.h) * D, total = (size_t)a.B * a.Nk * a.H * D;
      const float f = half ? a.scale : 1.f;
      __nv_bfloat16* dst = half ? dk : dv;
      float* pdst = part + (2 * (size_t)x.split + (half ? 0 : 1)) * total;
      const uint32_t t_o = lane_addr + (half ? G::kColK : G::kColV);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        if (!none) {
          tmem_ld32(t_o + c, o);
          tmem_wait_ld();
        }
        // a key that does not count has sums of 0 * dO and 0 * q, which may be NaN
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = valid && !none ? o[e] * f : 0.f;
        if (m < a.Nk) {
#pragma unroll
          for (int e = 0; e < 32; e += kVec) {
            if (w.splits == 1)
              store8(dst + at + c + e, o + e);
            else
              store8(pdst + at + c + e, o + e);
          }
        }
      }
      if (!none) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ctl->o_free));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t backward(const CrossArgs& a, int splits_q, int splits_k, const void* dout, const void* q, const void* k,
                     const void* v, const void* out, const float* lse, void* dq, void* dk, void* dv, float* stats,
                     float* part, cudaStream_t st) {
  CUtensorMap tq, td, tk, tv;
  if (!make_heads_map(&tq, q, a.B, a.Nq, a.H, D, a.q, kTile) ||
      !make_heads_map(&td, dout, a.B, a.Nq, a.H, D, a.dout, kTile) ||
      !make_heads_map(&tk, k, a.B, a.Nk, a.H, D, a.k, kTile) || !make_heads_map(&tv, v, a.B, a.Nk, a.H, D, a.v, kTile))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(cross_dq_sm100_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)dq_smem<D>());
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(cross_dkv_sm100_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)dkv_smem<D>());
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int padded = (int)cross_padded_rows(a.Nq), ktiles = (a.Nk + kTile - 1) / kTile;
  float *zl = stats, *zd = stats + (size_t)a.B * a.H * padded;
  const long long rows = (long long)padded * a.H;   // of a sample: below 2^31 + 2^17
  cross_stats_kernel<D><<<dim3((unsigned)((rows * (D / kVec) + 255) / 256), a.B), 256, 0, st>>>(
      a, (unsigned)padded, (const __nv_bfloat16*)dout, (const __nv_bfloat16*)out, lse, zl, zd);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;

  Work w;
  w.pairs = padded / (2 * kTile);
  w.splits = splits_k;
  w.run = (ktiles + splits_k - 1) / splits_k;
  w.padded = padded;
  set_divisors(&w, a.H);
  const long long items = (long long)a.B * a.H * w.pairs * splits_k;
  if (items > INT_MAX - 4096) return cudaErrorInvalidValue;
  w.items = (int)items;
  cross_dq_sm100_kernel<D><<<(unsigned)(items < sms ? items : sms), kDqThreads, dq_smem<D>(), st>>>(
      tq, td, tk, tv, a, w, zl, zd, (__nv_bfloat16*)dq, part);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const size_t nq = (size_t)a.B * a.Nq * a.H * D, nk = (size_t)a.B * a.Nk * a.H * D;
  if (splits_k > 1 && (e = launch_cross_sum(ROLA_BF16, splits_k, nq, nq, part, dq, st)) != cudaSuccess) return e;

  KeyWork kw;
  kw.ktiles = ktiles;
  kw.splits = splits_q;
  kw.qtiles = (a.Nq + kTile - 1) / kTile;
  kw.run = (kw.qtiles + splits_q - 1) / splits_q;
  kw.padded = padded;
  const long long kitems = (long long)a.B * a.H * ktiles * splits_q;
  if (kitems > INT_MAX - 4096) return cudaErrorInvalidValue;
  kw.items = (int)kitems;
  cross_dkv_sm100_kernel<D><<<(unsigned)(kitems < sms ? kitems : sms), kDkvThreads, dkv_smem<D>(), st>>>(
      tq, td, tk, tv, a, kw, zl, zd, (__nv_bfloat16*)dk, (__nv_bfloat16*)dv, part);
  e = cudaGetLastError();
  if (e != cudaSuccess || splits_q == 1) return e;
  e = launch_cross_sum(ROLA_BF16, splits_q, nk, 2 * nk, part, dk, st);
  return e != cudaSuccess ? e : launch_cross_sum(ROLA_BF16, splits_q, nk, 2 * nk, part + nk, dv, st);
}

}  // namespace

cudaError_t launch_cross_sm100_backward(const CrossArgs& a, int splits_q, int splits_k, const void* dout,
                                        const void* q, const void* k, const void* v, const void* out,
                                        const float* lse, void* dq, void* dk, void* dv, float* stats, float* part,
                                        cudaStream_t st) {
  return a.d == 64 ? backward<64>(a, splits_q, splits_k, dout, q, k, v, out, lse, dq, dk, dv, stats, part, st)
                   : backward<128>(a, splits_q, splits_k, dout, q, k, v, out, lse, dq, dk, dv, stats, part, st);
}

cudaError_t cross_sm100_backward_status(int* word, cudaStream_t st) { return take_status(g_status, word, st); }

}  // namespace rola

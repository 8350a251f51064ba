// Dense attention to an encoder's states on the sm_100a tensor cores (tcgen05 + TMEM + TMA),
// bf16, head dim 64 or 128.
//
//   S = q k^T  (bf16 products, fp32 sums);  P = 2^(S * scale * log2 e - m);  O = P v;  out = O / l
//
// One block works on two query tiles of 128 at a time, A and B, over the same key tiles of 128:
// a K or V tile then serves 256 queries (32 bytes of L2 reads a clock and SM at the full product
// rate), and while one tile's scores are in the exponentials the other's products run.  Thread t
// of a softmax group owns query row t: row sums and maxima need no exchange.  P is rounded to
// bf16 (V's type; the sum l takes the unrounded values) and goes back into tensor memory over S,
// from where it is the A operand of the second product.
//
// The offset m of a row moves only when a score exceeds it by more than 8 (log2 units): P stays
// within [0, 256], O and l are rescaled rarely.  That needs no wait: S of a tile is issued after
// the previous P v is done.
//
// Roles (384 threads): warp 0 loads Q, K, V; warp 1 issues the products; warp 2 clears the rows
// of a V tile whose keys do not count (0 * NaN would not vanish); warps 4-7 and 8-11 are the
// softmax groups, which also write the results (staged in shared memory, TMA stores that clip
// rows past Nq).  Blocks are persistent and walk (head, query pair) items head by head, so that
// the blocks at work share K and V in L2.
//
// Measured: 75600 queries x 512 keys, 40 heads of 128 (0.79 TFLOP) 962 to 998 us back to back (795
// to 825 TFLOP/s, 0.57 to 0.59 of the sustained library rate; the power limit holds the clock down)
// and 820 us in a burst.  Neither the tensor pipe (44 % of its cycles) nor the issue slots (36 %) nor
// L2 is full: what bounds it is one query tile's chain S, softmax, P v (by the clock in a copy made
// to read it about 1000, 2300 and 900 clocks) and the handovers between, of which two run side by
// side.  Tried and slower: 64-key scores in two buffers (946 us in a burst), P
// through shared memory (1000), Q an item ahead with result warps of their own (1026), spinning
// waits (1107 up), results stored from registers (1090).
//
// Every mbarrier wait is bounded; when one runs out, all roles leave, copies in flight are waited
// for and tensor memory is freed (ROLA_ERR_DEVICE_TIMEOUT in the device's status word).
#include <climits>
#include <cuda.h>

#include "cross_sm100.cuh"

namespace rola {
namespace {

using namespace sm100;

__device__ int g_status[1];

constexpr int kThreads = 384;
constexpr float kSlack = 8.f;                 // log2 units a score may exceed its row's offset by

template <int D>
struct Geo {
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kTileBytes = kBoxes * kBox;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr uint32_t kOffQ = 0;                               // Q of A, B
  static constexpr uint32_t kOffOut = 2 * kTileBytes;                // output staging of A, B
  static constexpr uint32_t kOffKV = 4 * kTileBytes;
  static constexpr uint32_t kOffCtl = kOffKV + kStages * kTileBytes;
  static constexpr uint32_t kColS = 0;                               // S of A, B (P over it)
  static constexpr uint32_t kColO = 256;                             // O of A, B
};

struct Ctl {
  uint64_t q_full[2], q_empty[2], k_full[6], v_full[6], v_ready[6], kv_empty[6];
  uint64_t s_full[2], p_full[2], pv_done[2], o_free[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

template <int D>
constexpr size_t smem_bytes() { return Geo<D>::kOffCtl + sizeof(Ctl) + 1024; }

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cross_sm100_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_out,
    const __grid_constant__ CrossArgs a, const __grid_constant__ Work w, float* __restrict__ lse,
    float* __restrict__ part, float* __restrict__ plse, unsigned long long limit_cycles) {
  using G = Geo<D>;
  constexpr int kStages = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl* ctl = reinterpret_cast<Ctl*>(base + G::kOffCtl);
  const uint32_t sbase = smem_addr(base);
  // uniform for the compiler too
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto bar = [&](uint64_t& m) { return smem_addr(&m); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(ctl->q_full[s]), 1);
      mbar_init(bar(ctl->q_empty[s]), 1);
      mbar_init(bar(ctl->s_full[s]), 1);
      mbar_init(bar(ctl->p_full[s]), 4);     // one arrive per warp of the group
      mbar_init(bar(ctl->pv_done[s]), 1);
      mbar_init(bar(ctl->o_free[s]), 4);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(ctl->k_full[s]), 1);
      mbar_init(bar(ctl->v_full[s]), 1);
      mbar_init(bar(ctl->v_ready[s]), 1);
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
  const WaitCtl wc{&ctl->abort, g_status, limit_cycles};

  if (warp == 0) {
    // ------------------------------------------------------------ loads of Q, K, V
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      int nq[2] = {0, 0}, nkv = 0, nk = 0, nv = 0;   // tiles loaded: Q of A, B; K and V; K; V
      bool ok = true;
      Item x{};
      auto load = [&](uint32_t dst, const CUtensorMap* tm, int h, int n, int b, uint32_t full) {
        mbar_expect_tx(full, G::kTileBytes);
        for (int c = 0; c < G::kBoxes; ++c) tma_load_4d(dst + c * kBox, tm, 64 * c, h, n, b, full);
      };
      // K and V tiles share the ring's slots in turn, but each kind has its own full barriers: who
      // waits for one kind alone then sees every phase of its barriers.
      auto load_kv = [&](const CUtensorMap* tm, uint64_t* full, int& n, int t) {
        const int s = nkv % kStages;
        if (nkv >= kStages && !mbar_wait(bar(ctl->kv_empty[s]), ((nkv / kStages) - 1) & 1, wc)) return false;
        load(sbase + G::kOffKV + s * G::kTileBytes, tm, x.h, t * kTile, x.b, bar(full[n % kStages]));
        ++nkv;
        ++n;
        return true;
      };
      for (int i = next_item(a, w, blockIdx.x, &x); ok && i < w.items; i = next_item(a, w, i + gridDim.x, &x)) {
        for (int s = 0; ok && s < x.streams; ++s) {
          if (nq[s] >= 1 && !mbar_wait(bar(ctl->q_empty[s]), (nq[s] - 1) & 1, wc)) { ok = false; break; }
          load(sbase + G::kOffQ + s * G::kTileBytes, &tm_q, x.h, x.q0 + s * kTile, x.b, bar(ctl->q_full[s]));
          ++nq[s];
          if (s == 0) ok = load_kv(&tm_k, ctl->k_full, nk, x.t0);   // the first K right behind the first Q
        }
        for (int t = x.t0; ok && t < x.t1; ++t) {
          ok = load_kv(&tm_v, ctl->v_full, nv, t);
          if (ok && t + 1 < x.t1) ok = load_kv(&tm_k, ctl->k_full, nk, t + 1);
        }
      }
      // every issued copy lands before the block leaves
      for (int s = 0; s < 2; ++s)
        if (nq[s] > 0) mbar_wait(bar(ctl->q_full[s]), (nq[s] - 1) & 1, wc, false);
      for (int y = nk > kStages ? nk - kStages : 0; y < nk; ++y)
        mbar_wait(bar(ctl->k_full[y % kStages]), (y / kStages) & 1, wc, false);
      for (int y = nv > kStages ? nv - kStages : 0; y < nv; ++y)
        mbar_wait(bar(ctl->v_full[y % kStages]), (y / kStages) & 1, wc, false);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    {
      int steps[2] = {0, 0}, nq[2] = {0, 0}, no[2] = {0, 0};   // tiles, items of a stream
      int nkv = 0, nkt = 0, nvt = 0;                            // K and V tiles, of each kind alone
      bool ok = true;
      auto wait = [&](uint64_t& m, uint32_t parity) { return warp_wait(m, parity, wc); };
      auto kv_wait = [&](uint64_t* full, int n) { return wait(full[n % kStages], (n / kStages) & 1); };
      auto slot = [&](int n) { return sbase + G::kOffKV + (n % kStages) * G::kTileBytes; };
      auto commit = [&](uint64_t& m) {
        if (elect_leader()) mma_commit(bar(m));
        __syncwarp();
      };
      // S_s = Q_s K^T; K is the nkt'th K tile, in the slot of the n'th tile.  P of the stream's
      // previous tile lies where S goes, so its product with V must be done.
      auto issue_s = [&](int s, int n, bool first, bool last) {
        if (first && !wait(ctl->q_full[s], nq[s] & 1)) return false;
        if (!kv_wait(ctl->k_full, nkt)) return false;
        if (steps[s] > 0 && !wait(ctl->pv_done[s], (steps[s] - 1) & 1)) return false;
        tc_fence_after();
        if (elect_leader()) {
          product_ss<D>(tmem + G::kColS + 128 * s, sbase + G::kOffQ + s * G::kTileBytes, slot(n));
          mma_commit(bar(ctl->s_full[s]));
          if (last) mma_commit(bar(ctl->q_empty[s]));   // Q may be replaced
        }
        __syncwarp();
        nq[s] += last;
        return true;
      };
      Item x{}, y{};
      int i = next_item(a, w, blockIdx.x, &x);
      if (i < w.items) {
        for (int s = 0; ok && s < x.streams; ++s) ok = issue_s(s, nkv, true, x.t1 == x.t0 + 1);
        if (ok) commit(ctl->kv_empty[nkv % kStages]);
        ++nkv;
        ++nkt;
      }
      while (ok && i < w.items) {
        const int i2 = next_item(a, w, i + gridDim.x, &y);
        for (int t = x.t0; ok && t < x.t1; ++t) {
          const bool more = t + 1 < x.t1, any = more || i2 < w.items;
          const int next_streams = more ? x.streams : i2 < w.items ? y.streams : 0;
          const int nv = nkv, nk = nkv + 1;       // V of this tile, K of the next
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (ok && s < x.streams) {
              // the previous item's O has been read
              if (t == x.t0 && no[s]++ > 0) ok = wait(ctl->o_free[s], (no[s] - 2) & 1);
              ok = ok && kv_wait(ctl->v_ready, nvt) && wait(ctl->p_full[s], steps[s] & 1);
              if (!ok) break;
              tc_fence_after();
              if (elect_leader()) {
                product_ts<D>(tmem + G::kColO + D * s, tmem + G::kColS + 128 * s, 32, slot(nv), t > x.t0);
                mma_commit(bar(ctl->pv_done[s]));
                if (s == x.streams - 1) mma_commit(bar(ctl->kv_empty[nv % kStages]));
              }
              __syncwarp();
              ++steps[s];
            }
            if (ok && s < next_streams) ok = issue_s(s, nk, !more, more ? t + 2 == x.t1 : y.t1 == y.t0 + 1);
          }
          if (ok && any) commit(ctl->kv_empty[nk % kStages]);
          nkv += 1 + any;
          nkt += any;
          ++nvt;
        }
        x = y;
        i = i2;
      }
      commit(ctl->drain);                        // no product may run when tensor memory is freed
      mbar_wait(bar(ctl->drain), 0, wc, false);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ V rows that do not count
    int nkv = 0, nvt = 0;
    bool ok = true;
    Item x{};
    for (int i = next_item(a, w, blockIdx.x, &x); ok && i < w.items; i = next_item(a, w, i + gridDim.x, &x)) {
      const int len = key_count(a, x.b);
      for (int t = x.t0; t < x.t1; ++t, ++nvt) {  // tiles are loaded K, V, K, V, ... in each item
        const int n = nkv + 2 * (t - x.t0) + 1, s = n % kStages;
        uint32_t bits[4];
        tile_bits(a, x.b, len, t, lane, bits);
        ok = __all_sync(0xffffffffu, mbar_wait(bar(ctl->v_full[nvt % kStages]), (nvt / kStages) & 1, wc));
        if (!ok) break;
        if (!all_set(bits)) {
          clear_rows<G::kBoxes>(base + G::kOffKV + s * G::kTileBytes, bits, lane);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ctl->v_ready[nvt % kStages]));
      }
      nkv += 2 * (x.t1 - x.t0);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax and results
    const int s = (warp - 4) >> 2, wq = warp & 3, row = 32 * wq + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * wq) << 16);
    const uint32_t t_s = lane_addr + G::kColS + 128 * s, t_o = lane_addr + G::kColO + D * s, gbar = 1 + s;
    const float sl2 = a.scale * 1.4426950408889634f;
    int step = 0, stores = 0;
    bool fail = false;
    for (int i = blockIdx.x; i < w.items; i += gridDim.x) {
      const Item x = item_at(a, w, i);
      if (s >= x.streams) continue;
      const int len = key_count(a, x.b), n = x.q0 + s * kTile + row;
      float m = -INFINITY, l = 0.f;
      for (int t = x.t0; t < x.t1; ++t, ++step) {
        uint32_t bits[4];
        const bool partial = a.key_mask || (t + 1) * kTile > len;
        if (partial) tile_bits(a, x.b, len, t, lane, bits);
        fail |= !mbar_wait(bar(ctl->s_full[s]), step & 1, wc);
        if (__any_sync(0xffffffffu, fail)) break;
        tc_fence_after();
        // The scores stay in registers from the maximum to the exponentials.
        float v[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, v + 32 * c);
        tmem_wait_ld();
        if (partial) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (!((bits[c >> 5] >> (c & 31)) & 1u)) v[c] = -INFINITY;
        }
        float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int c = 4; c < 128; c += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top[e] = c + 4 + e < 128 ? max3f(top[e], v[c + e], v[c + 4 + e]) : fmaxf(top[e], v[c + e]);
        }
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * sl2;   // sl2 > 0
        // rows whose offset moves: from nothing (O and l hold nothing yet), or by more than kSlack
        const bool move = mx > m + kSlack;                    // m = -inf: true for any finite score
        if (__any_sync(0xffffffffu, move)) {
          const float keep = move ? ex2_approx(m - mx) : 1.f;   // 2^-inf = 0
          if (move) m = mx;
          l *= keep;
          if (t > x.t0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tmem_ld16(t_o + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= keep;
              tmem_st16(t_o + c, o);
            }
          }
        }
        const float off = m == -INFINITY ? 0.f : -m;          // no score yet: P = 2^-inf = 0
        const float2 s2 = make_float2(sl2, sl2), o2 = make_float2(off, off);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          float pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float2 p = __ffma2_rn(make_float2(v[c + e], v[c + e + 1]), s2, o2);
            p.x = ex2_approx(p.x);
            p.y = ex2_approx(p.y);
            sum[(e >> 1) & 1] = __fadd2_rn(sum[(e >> 1) & 1], p);
            pk[e >> 1] = __uint_as_float(pack_bf16(p.x, p.y));
          }
          tmem_st16(t_s + (c >> 1), pk);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ctl->p_full[s]));
      }
      if (named_vote_or(gbar, 128, fail)) break;
      // ---------------------------------------------------------- results of the item
      const bool none = x.t1 == x.t0;
      const float inv = l == 0.f ? 0.f : 1.f / l;             // a row without a valid key: zeros
      const float z = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      if (!none) fail |= !mbar_wait(bar(ctl->pv_done[s]), (step - 1) & 1, wc);
      if (named_vote_or(gbar, 128, fail)) break;
      tc_fence_after();
      uint8_t* stage = base + G::kOffOut + s * G::kTileBytes;
      if (w.splits == 1 && stores > 0) {                      // the staging has been read
        if (row == 0) tma_store_wait_read0();
        named_sync(gbar, 128);
      }
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        if (none) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        } else {
          tmem_ld32(t_o + c, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= inv;
        if (w.splits == 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4 u = make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                       pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
            const int chunk = ((c & 32) >> 3) + e;            // of the row's 8 in its box
            *reinterpret_cast<uint4*>(stage + (c >> 6) * kBox + row * 128 + ((chunk ^ (row & 7)) << 4)) = u;
          }
        } else if (n < a.Nq) {
          float* p = part + (((size_t)x.split * a.B + x.b) * a.Nq + n) * a.H * D + (size_t)x.h * D + c;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(p + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (!none) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ctl->o_free[s]));
      }
      if (n < a.Nq) {
        const size_t at = ((size_t)x.b * a.H + x.h) * a.Nq + n;
        if (w.splits > 1)
          plse[(size_t)x.split * a.B * a.H * a.Nq + at] = z;
        else if (lse)
          lse[at] = z;
      }
      if (w.splits == 1) {
        fence_proxy_async_smem();
        named_sync(gbar, 128);
        if (row == 0) {
          for (int c = 0; c < G::kBoxes; ++c)
            tma_store_4d(&tm_out, 64 * c, x.h, x.q0 + s * kTile, x.b,
                         sbase + G::kOffOut + s * G::kTileBytes + c * kBox);
          tma_store_commit();
        }
        ++stores;
      }
    }
    if (row == 0 && stores > 0) tma_store_wait_all();
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
cudaError_t launch(const CrossArgs& a, int splits, const void* q, const void* k, const void* v, void* out, float* lse,
                   float* part, cudaStream_t st) {
  CUtensorMap tq, tk, tv, to;
  const rola_strides so{(int64_t)a.Nq * a.H * D, (int64_t)a.H * D, D};
  if (!make_heads_map(&tq, q, a.B, a.Nq, a.H, D, a.q, kTile) ||
      !make_heads_map(&tk, k, a.B, a.Nk, a.H, D, a.k, kTile) ||
      !make_heads_map(&tv, v, a.B, a.Nk, a.H, D, a.v, kTile) || !make_heads_map(&to, out, a.B, a.Nq, a.H, D, so, kTile))
    return cudaErrorInvalidValue;
  constexpr size_t smem = smem_bytes<D>();
  cudaError_t e = cudaFuncSetAttribute(cross_sm100_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  Work w;
  const int tiles = (a.Nk + kTile - 1) / kTile;
  w.pairs = (a.Nq + 2 * kTile - 1) / (2 * kTile);
  w.splits = splits;
  w.run = (tiles + splits - 1) / splits;
  const long long items = (long long)a.B * a.H * w.pairs * splits;
  if (items > INT_MAX - 4096) return cudaErrorInvalidValue;
  w.items = (int)items;
  w.padded = 0;
  set_divisors(&w, a.H);
  float* plse = part + (size_t)splits * a.B * a.Nq * a.H * D;
  const unsigned long long limit_cycles = 2000000000ull;   // 1 s at 2 GHz
  cross_sm100_kernel<D><<<(unsigned)(items < sms ? items : sms), kThreads, smem, st>>>(tq, tk, tv, to, a, w, lse, part,
                                                                                     plse, limit_cycles);
  e = cudaGetLastError();
  if (e != cudaSuccess || splits == 1) return e;
  return launch_cross_join(a, ROLA_BF16, splits, part, plse, out, lse, st);
}

}  // namespace

cudaError_t launch_cross_sm100(const CrossArgs& a, int splits, const void* q, const void* k, const void* v, void* out,
                               float* lse, float* part, cudaStream_t st) {
  return a.d == 64 ? launch<64>(a, splits, q, k, v, out, lse, part, st)
                   : launch<128>(a, splits, q, k, v, out, lse, part, st);
}

cudaError_t cross_sm100_status(int* word, cudaStream_t st) { return take_status(g_status, word, st); }

}  // namespace rola

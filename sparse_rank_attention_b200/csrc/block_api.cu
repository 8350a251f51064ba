// C ABI of the operators around RoLA: argument checks, workspace layout, launch order.  The
// operators, layouts and error rules are stated in include/rola.h.
#include <cmath>
#include <cstring>

#include "block_internal.cuh"
#include "row_ops.cuh"

namespace {

using rola::CrossArgs;
using rola::GatedNormArgs;
using rola::NormRopeArgs;

constexpr long long kMaxRows = (1ll << 31) - 1;   // tokens of a call: kernels index them in 32 bits
constexpr int kMaxGrid = 65535;                   // blocks on the y and z axes of a grid

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool given(const void* p) { return p && aligned16(p); }
bool optional(const void* p) { return !p || aligned16(p); }
bool words(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }   // read one by one
size_t elem_size(rola_dtype t) { return t == ROLA_F32 ? 4 : 2; }
bool known(rola_dtype t) { return t == ROLA_F32 || t == ROLA_BF16 || t == ROLA_FP8_E4M3; }
rola_status cuda_status(cudaError_t e) { return e == cudaSuccess ? ROLA_OK : ROLA_ERR_CUDA; }

// Whether so many elements lie within an address space; the spans below then fit 64 bits.
bool reachable(double elements, size_t el) { return elements * el < (double)(1ll << 48); }

// A strided [B, N, H, d] tensor; the strides of axes of size one take those of a contiguous one.
struct View {
  const char* p;
  int B, N, H, d;
  size_t el;
  rola_strides s;
  View(const void* ptr, int B, int N, int H, int d, rola_dtype t, const rola_strides& st)
      : p(static_cast<const char*>(ptr)), B(B), N(N), H(H), d(d), el(elem_size(t)), s(st) {
    if (H == 1) s.h = d;
    if (N == 1) s.n = (int64_t)H * d;
    if (B == 1) s.b = (int64_t)N * H * d;
  }
  static View contiguous(const void* ptr, int B, int N, int H, int d, rola_dtype t) {
    return View(ptr, B, N, H, d, t, rola_strides{(int64_t)N * H * d, (int64_t)H * d, d});
  }
  bool strides_ok() const {
    const int64_t unit = (int64_t)(16 / el);
    for (int64_t x : {s.b, s.n, s.h})
      if (x < d || x % unit != 0 || x > (1ll << 36)) return false;   // 2^36: in reach of a tensor map
    return reachable((double)(B - 1) * s.b + (double)(N - 1) * s.n + (double)(H - 1) * s.h + d, el);
  }
  size_t span() const { return el * (size_t)((B - 1) * s.b + (int64_t)(N - 1) * s.n + (int64_t)(H - 1) * s.h + d); }
  // no two of its elements share memory (for tensors that are written in place)
  bool distinct() const {
    const int64_t h = (int64_t)(H - 1) * s.h, n = (int64_t)(N - 1) * s.n;
    const bool token_major = (N == 1 || s.n >= h + d) && (B == 1 || s.b >= n + h + d);
    const bool head_major = (H == 1 || s.h >= n + d) && (B == 1 || s.b >= n + h + d);
    return token_major || head_major;
  }
  bool same_as(const View& o) const { return p == o.p && el == o.el && s.b == o.s.b && s.n == o.s.n && s.h == o.s.h; }
};

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

struct Axis {
  int64_t stride;
  int n;
};

// Whether a distance of `gap` elements is less than d away from some i s0 + j s1 + l s2, each index
// within one axis' length of zero: two views that far apart then share an element.  Axes from the
// longest stride on; where one does not reach past the axes inside it, the answer is yes.
bool meets(int64_t gap, const Axis* axis, int axes, int d) {
  if (axes == 0) return gap < d && gap > -d;
  int64_t reach = d;                   // the rest has to come closer than this
  for (int i = 1; i < axes; ++i) reach += (axis[i].n - 1) * axis[i].stride;
  if (axis->stride < reach) return true;
  const int64_t low = gap / axis->stride - (gap % axis->stride < 0);
  for (int64_t i = low; i <= low + 1; ++i)
    if (i < axis->n && i > -axis->n && meets(gap - i * axis->stride, axis + 1, axes - 1, d)) return true;
  return false;
}

// Whether two views may share memory.  Views of equal strides may lie inside one another's gaps (the
// parts of a fused projection: side by side in a token, in a head, between the heads).
bool overlaps(const View& a, const View& b) {
  if (!overlaps(a.p, a.span(), b.p, b.span())) return false;
  if (a.el != b.el || a.s.b != b.s.b || a.s.n != b.s.n || a.s.h != b.s.h) return true;
  Axis axis[3];
  int axes = 0;
  for (const Axis& x : {Axis{a.s.b, a.B}, Axis{a.s.n, a.N}, Axis{a.s.h, a.H}}) {
    if (x.n == 1) continue;
    int at = axes++;
    for (; at > 0 && axis[at - 1].stride < x.stride; --at) axis[at] = axis[at - 1];
    axis[at] = x;
  }
  return meets((a.p - b.p) / (int64_t)a.el, axis, axes, a.d);
}
bool overlaps(const View& a, const void* b, size_t nb) { return overlaps(a.p, a.span(), b, nb); }

// ------------------------------------------------------------------ qk_norm_rope

rola_status check(const rola_norm_rope_params* p) {
  if (!p || p->B < 1 || p->N < 1 || p->H < 1) return ROLA_ERR_INVALID_ARG;
  if (!known(p->dtype) || !known(p->grad_dtype)) return ROLA_ERR_INVALID_ARG;
  if (p->norm < ROLA_NORM_NONE || p->norm > ROLA_NORM_HEAD) return ROLA_ERR_INVALID_ARG;
  if (p->pos < ROLA_POS_NONE || p->pos > ROLA_POS_GIVEN) return ROLA_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || std::isinf(p->eps)) return ROLA_ERR_INVALID_ARG;
  if (p->dtype == ROLA_FP8_E4M3 || p->grad_dtype == ROLA_FP8_E4M3) return ROLA_ERR_UNSUPPORTED;
  if (p->grad_dtype != p->dtype && p->grad_dtype != ROLA_F32) return ROLA_ERR_UNSUPPORTED;
  if (p->d != 64 && p->d != 128) return ROLA_ERR_UNSUPPORTED;
  if ((long long)p->H * p->d > rola::kMaxRowChannels) return ROLA_ERR_UNSUPPORTED;
  if ((long long)p->B * p->N > kMaxRows || p->B > kMaxGrid) return ROLA_ERR_UNSUPPORTED;
  if (p->pos == ROLA_POS_NONE) return ROLA_OK;
  if (!(p->rope_base > 1.0) || std::isinf(p->rope_base)) return ROLA_ERR_INVALID_ARG;
  if (p->rope_pairs_t < 0 || p->rope_pairs_h < 0 || p->rope_pairs_w < 0) return ROLA_ERR_INVALID_ARG;
  const long long pairs = (long long)p->rope_pairs_t + p->rope_pairs_h + p->rope_pairs_w;
  if (pairs != 0 && pairs != p->d / 2) return ROLA_ERR_INVALID_ARG;
  if (p->pos == ROLA_POS_GRID) {
    if (p->grid_t < 1 || p->grid_h < 1 || p->grid_w < 1) return ROLA_ERR_INVALID_ARG;
    const long long hw = (long long)p->grid_h * p->grid_w;
    if (hw > p->N || hw * p->grid_t > p->N) return ROLA_ERR_INVALID_ARG;
  } else if (p->positions_batched != 0 && p->positions_batched != 1) {
    return ROLA_ERR_INVALID_ARG;
  }
  return ROLA_OK;
}

NormRopeArgs args_of(const rola_norm_rope_params& p, const int32_t* positions) {
  NormRopeArgs a{};
  a.B = p.B; a.N = p.N; a.H = p.H; a.d = p.d;
  a.head_shift = p.d == 64 ? 6 : 7;
  a.eps = p.eps;
  a.rot.pos = p.pos;
  if (p.pos == ROLA_POS_NONE) return a;
  a.rot.gt = p.grid_t; a.rot.gh = p.grid_h; a.rot.gw = p.grid_w;
  a.rot.st = p.start_t; a.rot.sh = p.start_h; a.rot.sw = p.start_w;
  a.rot.batched = p.positions_batched;
  a.rot.positions = positions;
  int n[3] = {p.rope_pairs_t, p.rope_pairs_h, p.rope_pairs_w};
  const int P = p.d / 2;
  if (n[0] + n[1] + n[2] == 0) {
    if (p.pos == ROLA_POS_GRID && p.grid_t == 1 && p.grid_h == 1) {
      n[2] = P;
    } else {
      n[1] = n[2] = P / 3;
      n[0] = P - 2 * (P / 3);
    }
  }
  a.rot.pt = n[0];
  a.rot.ph = n[1];
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  for (int axis = 0, c = 0; axis < 3; ++axis)
    for (int i = 0; i < n[axis]; ++i, ++c) a.rot.turns[c] = std::pow(p.rope_base, -(double)i / n[axis]) / kTwoPi;
  return a;
}

size_t weight_bytes(const rola_norm_rope_params& p) {
  return p.norm == ROLA_NORM_NONE ? 0 : 4 * (size_t)(p.norm == ROLA_NORM_TOKEN ? p.H * p.d : p.d);
}

// ------------------------------------------------------------------ gated_norm

rola_status check(const rola_gated_norm_params* p) {
  if (!p || p->B < 1 || p->N < 1 || p->C < 1 || p->T < 1) return ROLA_ERR_INVALID_ARG;
  if (!known(p->x_dtype) || !known(p->y_dtype)) return ROLA_ERR_INVALID_ARG;
  if (p->norm != ROLA_LAYER && p->norm != ROLA_RMS) return ROLA_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || std::isinf(p->eps)) return ROLA_ERR_INVALID_ARG;
  if (p->N % p->T != 0) return ROLA_ERR_INVALID_ARG;
  if (p->x_dtype == ROLA_FP8_E4M3 || p->y_dtype == ROLA_FP8_E4M3) return ROLA_ERR_UNSUPPORTED;
  if (p->x_dtype != p->y_dtype && !(p->x_dtype == ROLA_F32 && p->y_dtype == ROLA_BF16)) return ROLA_ERR_UNSUPPORTED;
  if (p->C % rola::kVec != 0 || p->C > rola::kMaxRowChannels) return ROLA_ERR_UNSUPPORTED;
  if ((long long)p->B * p->N > kMaxRows) return ROLA_ERR_UNSUPPORTED;
  return ROLA_OK;
}

// Bytes from the first to past the last element of a modulation [B, T, C], 0 for bad strides.
size_t mod_span(const rola_gated_norm_params& p, int64_t sb, int64_t st) {
  if (p.B == 1) sb = 0;
  if (p.T == 1) st = 0;
  if (sb < 0 || st < 0 || sb % 4 != 0 || st % 4 != 0) return 0;
  if (!reachable((double)(p.B - 1) * sb + (double)(p.T - 1) * st + p.C, 4)) return 0;
  return 4 * (size_t)((p.B - 1) * sb + (p.T - 1) * st + p.C);
}

GatedNormArgs args_of(const rola_gated_norm_params& p, bool back) {
  GatedNormArgs a{};
  a.B = p.B; a.N = p.N; a.C = p.C; a.T = p.T;
  a.per = p.N / p.T;
  a.eps = p.eps;
  a.gate_b = p.gate_b; a.gate_t = p.gate_t;
  a.scale_b = p.scale_b; a.scale_t = p.scale_t;
  a.shift_b = p.shift_b; a.shift_t = p.shift_t;
  rola::gated_norm_chunks(p, back, &a.chunks, &a.chunk);
  return a;
}

// ------------------------------------------------------------------ cross_attend

rola_status check(const rola_cross_params* p) {
  if (!p || p->B < 1 || p->Nq < 1 || p->Nk < 1 || p->H < 1) return ROLA_ERR_INVALID_ARG;
  if (!known(p->dtype)) return ROLA_ERR_INVALID_ARG;
  if (!(p->softmax_scale >= 0.f) || std::isinf(p->softmax_scale)) return ROLA_ERR_INVALID_ARG;
  if (p->dtype == ROLA_FP8_E4M3) return ROLA_ERR_UNSUPPORTED;
  if (p->d != 64 && p->d != 128) return ROLA_ERR_UNSUPPORTED;
  if (p->B > kMaxGrid || p->H > 512) return ROLA_ERR_UNSUPPORTED;
  // tiles end up to a pair of query tiles behind the last token
  const long long most = kMaxRows - 255;
  if ((long long)p->B * p->Nq * p->H > most || (long long)p->B * p->Nk * p->H > most) return ROLA_ERR_UNSUPPORTED;
  return ROLA_OK;
}

CrossArgs args_of(const rola_cross_params& p, const int32_t* kv_len, const uint8_t* key_mask) {
  CrossArgs a{};
  a.B = p.B; a.Nq = p.Nq; a.Nk = p.Nk; a.H = p.H; a.d = p.d;
  a.scale = p.softmax_scale > 0.f ? p.softmax_scale : (float)(1.0 / std::sqrt((double)p.d));
  a.q = View(nullptr, p.B, p.Nq, p.H, p.d, p.dtype, p.q).s;
  a.k = View(nullptr, p.B, p.Nk, p.H, p.d, p.dtype, p.k).s;
  a.v = View(nullptr, p.B, p.Nk, p.H, p.d, p.dtype, p.v).s;
  a.dout = View(nullptr, p.B, p.Nq, p.H, p.d, p.dtype, p.dout).s;
  a.kv_len = kv_len;
  a.key_mask = key_mask;
  return a;
}

// Blocks that share the long axis (`tiles` tiles) of one of `rows` independent tiles: `want`
// blocks in all, each with `least` tiles at least (joining the parts costs a launch and the
// parts' traffic).  Forward of 12 heads of 128, in one part, as chosen, in more: one query
// to 2000 keys 36, 16 and 15 us, to 8192 keys 130, 24 and 35; 200 queries to 8192 keys 139, 35 and
// 64, at 40 heads 141, 70 and 98.  Under 8 tiles (2 x 1 query, 512 keys) one part takes 12 us, four 11.
int split_of(long long rows, int tiles, long long want, int least) {
  long long s = want / rows;
  if (s > tiles / least) s = tiles / least;
  if (s > 64) s = 64;
  if (s < 2) return 1;
  const int run = (int)((tiles + s - 1) / s);
  return (tiles + run - 1) / run;
}

// The same for fp32, whose tiles take long enough that the last round of blocks counts: of all
// splits the one with the least rounds * (tiles of a block + its start and end) + joining, in
// tiles' times (dq of 1000 x 257 at 12 heads of 128: 192 blocks of 5 tiles on 148 SMs 131 us, 576
// of 1 or 2 with the sum 106; dk, dv: 240 blocks of 4 as long as 120 of 8).  Forward in one part, as
// chosen, in more: 2 x 777 x 333 at 3 heads of 64 34, 27 and 30 us, 1000 x 257 at 12 of 128
// 97, 83 and 89, 64 x 8192 at 8 of 128 1184, 87 and 97, 2 x 1 x 512 at 12 of 128 76, 25 and 27.
int even_split(long long rows, int tiles, int slots) {
  int best = 1;
  double least = 0;
  for (int want = 1; want <= tiles && want <= 64; ++want) {
    const int run = (tiles + want - 1) / want, s = (tiles + run - 1) / run;
    const double rounds = (double)((rows * s + slots - 1) / slots);
    const double cost = rounds * ((double)tiles / s + 0.4) + (s > 1 ? 0.4 + 0.1 * s : 0.0);
    if (want == 1 || cost < least) least = cost, best = s;
  }
  return best;
}
// Resident blocks of an fp32 kernel.
int simt_slots(int d) { return (d == 64 ? 2 : 1) * rola::kRowSMs; }

struct CrossSplits {
  int keys, queries;
};
int tiles_of(int n, int tile) { return (n - 1) / tile + 1; }
// Forward: blocks that share a query tile's keys (fp32: tiles of 64 x 64; bf16: of 256 queries x
// 128 keys, one block an SM).
int forward_splits(const rola_cross_params& p) {
  const long long bh = (long long)p.B * p.H;
  if (p.dtype == ROLA_F32) return even_split(bh * tiles_of(p.Nq, 64), tiles_of(p.Nk, 64), simt_slots(p.d));
  return split_of(bh * tiles_of(p.Nq, 256), tiles_of(p.Nk, 128), rola::kRowSMs, 4);
}
// Backward: the same for dq, and blocks that share a key tile's queries for dk, dv (bf16: tiles
// of 128 keys x 128 queries; several items per SM even out the last round of blocks: 32760 x 512
// keys of 40 heads, 160 key tiles, 1677 us for the call in 7 parts, 2086 in one).
CrossSplits backward_splits(const rola_cross_params& p) {
  const long long bh = (long long)p.B * p.H;
  if (p.dtype == ROLA_F32) {
    const int tq = tiles_of(p.Nq, 64), tk = tiles_of(p.Nk, 64);
    return {even_split(bh * tq, tk, simt_slots(p.d)), even_split(bh * tk, tq, simt_slots(p.d))};
  }
  return {forward_splits(p), split_of(bh * tiles_of(p.Nk, 128), tiles_of(p.Nq, 128), 8 * rola::kRowSMs, 8)};
}

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

size_t forward_bytes(const rola_cross_params& p) {
  const int s = forward_splits(p);
  return s == 1 ? 0 : 4 * (size_t)s * p.B * p.Nq * p.H * (p.d + 1);
}

// Statistics per row: D (fp32), or lse and D in padded rows (bf16).
size_t stats_bytes(const rola_cross_params& p) {
  if (p.dtype == ROLA_F32) return align16(4 * (size_t)p.B * p.H * p.Nq);
  return 8 * (size_t)p.B * p.H * rola::cross_padded_rows(p.Nq);
}

size_t backward_bytes(const rola_cross_params& p) {
  const CrossSplits s = backward_splits(p);
  const size_t q = s.keys == 1 ? 0 : 4 * (size_t)s.keys * p.B * p.Nq * p.H * p.d;
  const size_t k = s.queries == 1 ? 0 : 8 * (size_t)s.queries * p.B * p.Nk * p.H * p.d;
  return stats_bytes(p) + (q > k ? q : k);
}

}  // namespace

extern "C" {

rola_status rola_norm_rope_params_default(rola_norm_rope_params* p) {
  if (!p) return ROLA_ERR_INVALID_ARG;
  std::memset(p, 0, sizeof(*p));
  p->B = p->N = p->H = 1;
  p->d = 128;
  p->dtype = p->grad_dtype = ROLA_BF16;
  p->norm = ROLA_NORM_TOKEN;
  p->eps = 1e-6f;
  p->pos = ROLA_POS_GRID;
  p->grid_t = p->grid_h = p->grid_w = 1;
  p->rope_base = 10000.0;
  return ROLA_OK;
}

rola_status rola_qk_norm_rope(const rola_norm_rope_params* p, const void* q, const void* k, const float* wq,
                              const float* wk, const int32_t* positions, void* q_out, void* k_out,
                              rola_stream_t stream) {
  const rola_status s = check(p);
  if (s != ROLA_OK) return s;
  const bool norm = p->norm != ROLA_NORM_NONE, table = p->pos == ROLA_POS_GIVEN;
  if (!given(q) || !given(q_out) || !optional(k) || !optional(k_out) || (k == nullptr) != (k_out == nullptr))
    return ROLA_ERR_INVALID_ARG;
  if (norm != (wq != nullptr) || (norm && k) != (wk != nullptr) || table != (positions != nullptr))
    return ROLA_ERR_INVALID_ARG;
  if (!optional(wq) || !optional(wk) || !words(positions)) return ROLA_ERR_INVALID_ARG;
  const int n = k ? 2 : 1;
  const View in[2] = {View(q, p->B, p->N, p->H, p->d, p->dtype, p->q), View(k, p->B, p->N, p->H, p->d, p->dtype, p->k)};
  View out[2] = {View::contiguous(q_out, p->B, p->N, p->H, p->d, p->dtype),
                 View::contiguous(k_out, p->B, p->N, p->H, p->d, p->dtype)};
  const size_t wb = weight_bytes(*p), pb = table ? 12 * (size_t)(p->positions_batched ? p->B : 1) * p->N : 0;
  for (int i = 0; i < n; ++i) {
    if (!in[i].strides_ok()) return ROLA_ERR_INVALID_ARG;
    if (out[i].p == in[i].p) out[i] = in[i];   // in place
  }
  for (int i = 0; i < n; ++i) {
    if (!out[i].distinct()) return ROLA_ERR_INVALID_ARG;
    for (int j = 0; j < n; ++j) {
      if (!(i == j && out[i].same_as(in[i])) && overlaps(out[i], in[j])) return ROLA_ERR_INVALID_ARG;
      if (j != i && overlaps(out[i], out[j])) return ROLA_ERR_INVALID_ARG;
    }
    if (norm && (overlaps(out[i], wq, wb) || (k && overlaps(out[i], wk, wb)))) return ROLA_ERR_INVALID_ARG;
    if (table && overlaps(out[i], positions, pb)) return ROLA_ERR_INVALID_ARG;
  }
  NormRopeArgs a = args_of(*p, positions);
  a.q = in[0].s; a.k = in[1].s; a.qo = out[0].s; a.ko = out[1].s;
  return cuda_status(rola::launch_norm_rope(a, p->dtype, p->norm, q, k, wq, wk, q_out, k_out,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

rola_status rola_qk_norm_rope_workspace_size(const rola_norm_rope_params* p, size_t* bytes) {
  if (!bytes) return ROLA_ERR_INVALID_ARG;
  const rola_status s = check(p);
  if (s != ROLA_OK) return s;
  const int C = p->H * p->d;
  if (p->norm == ROLA_NORM_NONE) {
    *bytes = 0;
    return ROLA_OK;
  }
  const int one = rola::norm_rope_parts(p->B, p->N, C, 1), two = rola::norm_rope_parts(p->B, p->N, C, 2);
  *bytes = 8 * (size_t)C * (one > two ? one : two);
  return ROLA_OK;
}

rola_status rola_qk_norm_rope_backward(const rola_norm_rope_params* p, const void* dq_out, const void* dk_out,
                                       const void* q, const void* k, const float* wq, const float* wk,
                                       const int32_t* positions, void* dq, void* dk, float* dwq, float* dwk,
                                       void* workspace, size_t workspace_bytes, rola_stream_t stream) {
  size_t need = 0;
  const rola_status s = rola_qk_norm_rope_workspace_size(p, &need);
  if (s != ROLA_OK) return s;
  const bool norm = p->norm != ROLA_NORM_NONE, table = p->pos == ROLA_POS_GIVEN, two = dk_out != nullptr;
  if (!given(dq_out) || !given(dq) || !optional(dk_out) || !optional(dk) || two != (dk != nullptr))
    return ROLA_ERR_INVALID_ARG;
  if (norm && (!given(q) || !given(wq) || !given(dwq))) return ROLA_ERR_INVALID_ARG;
  if (norm && two && (!given(k) || !given(wk) || !given(dwk))) return ROLA_ERR_INVALID_ARG;
  if (!norm && (wq || wk || dwq || dwk)) return ROLA_ERR_INVALID_ARG;
  if (table != (positions != nullptr) || !words(positions)) return ROLA_ERR_INVALID_ARG;
  if (need && (!given(workspace) || workspace_bytes < need)) return ROLA_ERR_WORKSPACE;
  const int n = two ? 2 : 1;
  const View up[2] = {View(dq_out, p->B, p->N, p->H, p->d, p->grad_dtype, p->dq_out),
                      View(dk_out, p->B, p->N, p->H, p->d, p->grad_dtype, p->dk_out)};
  const View in[2] = {View(q, p->B, p->N, p->H, p->d, p->dtype, p->q), View(k, p->B, p->N, p->H, p->d, p->dtype, p->k)};
  const View out[2] = {View::contiguous(dq, p->B, p->N, p->H, p->d, p->dtype),
                       View::contiguous(dk, p->B, p->N, p->H, p->d, p->dtype)};
  const float* w[2] = {wq, wk};
  float* dw[2] = {dwq, dwk};
  const size_t wb = weight_bytes(*p), pb = table ? 12 * (size_t)(p->positions_batched ? p->B : 1) * p->N : 0;
  for (int i = 0; i < n; ++i)
    if (!up[i].strides_ok() || (norm && !in[i].strides_ok())) return ROLA_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    for (int j = 0; j < n; ++j) {
      if (!(i == j && out[i].same_as(up[i])) && overlaps(out[i], up[j])) return ROLA_ERR_INVALID_ARG;
      if (j != i && overlaps(out[i], out[j])) return ROLA_ERR_INVALID_ARG;
      if (!norm) continue;
      if (overlaps(out[i], in[j]) || overlaps(out[i], w[j], wb) || overlaps(out[i], dw[j], wb))
        return ROLA_ERR_INVALID_ARG;
      if (overlaps(up[j], dw[i], wb) || overlaps(in[j], dw[i], wb) || overlaps(w[j], wb, dw[i], wb) ||
          (j != i && overlaps(dw[j], wb, dw[i], wb)))
        return ROLA_ERR_INVALID_ARG;
      if (overlaps(workspace, need, w[j], wb) || overlaps(workspace, need, dw[j], wb) ||
          overlaps(in[j], workspace, need))
        return ROLA_ERR_INVALID_ARG;
    }
    if (need && (overlaps(out[i], workspace, need) || overlaps(up[i], workspace, need))) return ROLA_ERR_INVALID_ARG;
    if (table && (overlaps(out[i], positions, pb) || (norm && overlaps(positions, pb, dw[i], wb)) ||
                  overlaps(positions, pb, workspace, need)))
      return ROLA_ERR_INVALID_ARG;
  }
  NormRopeArgs a = args_of(*p, positions);
  a.q = in[0].s; a.k = in[1].s; a.qo = up[0].s; a.ko = up[1].s;
  return cuda_status(rola::launch_norm_rope_backward(a, p->dtype, p->grad_dtype, p->norm, dq_out, dk_out, q, k, wq, wk,
                                                     dq, dk, dwq, dwk, static_cast<float*>(workspace),
                                                     reinterpret_cast<cudaStream_t>(stream)));
}

rola_status rola_gated_norm(const rola_gated_norm_params* p, const void* x, const void* branch, const float* gate,
                            const float* scale, const float* shift, const float* weight, const float* bias, void* r,
                            void* y, rola_stream_t stream) {
  const rola_status s = check(p);
  if (s != ROLA_OK) return s;
  if (!given(x) || !given(y) || !optional(branch) || !optional(gate) || !optional(scale) || !optional(shift) ||
      !optional(weight) || !optional(bias) || !optional(r))
    return ROLA_ERR_INVALID_ARG;
  if ((branch == nullptr) != (r == nullptr) || (gate && !branch) || (scale == nullptr) != (shift == nullptr) ||
      (bias && !weight) || (scale && weight))
    return ROLA_ERR_INVALID_ARG;
  const size_t n = (size_t)p->B * p->N * p->C, xb = n * elem_size(p->x_dtype), yb = n * elem_size(p->y_dtype);
  const struct { const void* p; size_t n; } in[] = {
      {branch, yb}, {gate, mod_span(*p, p->gate_b, p->gate_t)}, {scale, mod_span(*p, p->scale_b, p->scale_t)},
      {shift, mod_span(*p, p->shift_b, p->shift_t)}, {weight, 4 * (size_t)p->C}, {bias, 4 * (size_t)p->C}};
  for (const auto& i : in) {
    if (!i.p) continue;
    if (!i.n || overlaps(y, yb, i.p, i.n) || (r && overlaps(r, xb, i.p, i.n))) return ROLA_ERR_INVALID_ARG;
  }
  if (overlaps(y, yb, x, xb) || (r && (overlaps(y, yb, r, xb) || (r != x && overlaps(r, xb, x, xb)))))
    return ROLA_ERR_INVALID_ARG;
  return cuda_status(rola::launch_gated_norm(args_of(*p, false), p->x_dtype, p->y_dtype, p->norm, x, branch, gate,
                                             scale, shift, weight, bias, r, y,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

rola_status rola_gated_norm_workspace_size(const rola_gated_norm_params* p, size_t* bytes) {
  if (!bytes) return ROLA_ERR_INVALID_ARG;
  const rola_status s = check(p);
  if (s != ROLA_OK) return s;
  *bytes = rola::gated_norm_workspace(*p);
  return ROLA_OK;
}

rola_status rola_gated_norm_backward(const rola_gated_norm_params* p, const void* dy, const void* dr, const void* r,
                                     const void* branch, const float* gate, const float* scale, const float* weight,
                                     void* dx, void* dbranch, float* dgate, float* dscale, float* dshift,
                                     float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                                     rola_stream_t stream) {
  size_t need = 0;
  const rola_status s = rola_gated_norm_workspace_size(p, &need);
  if (s != ROLA_OK) return s;
  if (!given(dy) || !given(r) || !given(dx)) return ROLA_ERR_INVALID_ARG;
  for (const void* x : {dr, branch, (const void*)gate, (const void*)scale, (const void*)weight, (const void*)dbranch,
                        (const void*)dgate, (const void*)dscale, (const void*)dshift, (const void*)dweight,
                        (const void*)dbias})
    if (!optional(x)) return ROLA_ERR_INVALID_ARG;
  if ((branch == nullptr) != (dbranch == nullptr) || (gate && !branch) || (gate == nullptr) != (dgate == nullptr) ||
      (scale == nullptr) != (dscale == nullptr) || (scale == nullptr) != (dshift == nullptr) ||
      (weight == nullptr) != (dweight == nullptr) || (dbias && !weight) || (scale && weight))
    return ROLA_ERR_INVALID_ARG;
  if (!given(workspace) || workspace_bytes < need) return ROLA_ERR_WORKSPACE;
  const size_t n = (size_t)p->B * p->N * p->C, xb = n * elem_size(p->x_dtype), yb = n * elem_size(p->y_dtype);
  const size_t mb = 4 * (size_t)p->B * p->T * p->C, cb = 4 * (size_t)p->C;
  struct Span { const void* p; size_t n; };
  const Span in[] = {{dy, yb}, {r, xb}, {branch, yb}, {gate, mod_span(*p, p->gate_b, p->gate_t)},
                     {scale, mod_span(*p, p->scale_b, p->scale_t)}, {weight, cb}, {dr, xb}};
  const Span out[] = {{dx, xb}, {dbranch, yb}, {dgate, mb}, {dscale, mb}, {dshift, mb}, {dweight, cb}, {dbias, cb},
                      {workspace, need}};
  for (const Span& i : in)
    if (i.p && !i.n) return ROLA_ERR_INVALID_ARG;
  for (int a = 0; a < 8; ++a) {
    if (!out[a].p) continue;
    for (int c = 0; c < 7; ++c) {
      if (!in[c].p || (a == 0 && c == 6 && dx == dr)) continue;
      if (overlaps(out[a].p, out[a].n, in[c].p, in[c].n)) return ROLA_ERR_INVALID_ARG;
    }
    for (int c = a + 1; c < 8; ++c)
      if (out[c].p && overlaps(out[a].p, out[a].n, out[c].p, out[c].n)) return ROLA_ERR_INVALID_ARG;
  }
  return cuda_status(rola::launch_gated_norm_backward(
      args_of(*p, true), p->x_dtype, p->y_dtype, p->norm, dy, dr, r, branch, gate, scale, weight, dx, dbranch, dgate,
      dscale, dshift, dweight, dbias, static_cast<float*>(workspace), reinterpret_cast<cudaStream_t>(stream)));
}

rola_status rola_cross_workspace_size(const rola_cross_params* p, size_t* bytes) {
  if (!bytes) return ROLA_ERR_INVALID_ARG;
  const rola_status s = check(p);
  if (s != ROLA_OK) return s;
  *bytes = forward_bytes(*p);
  return ROLA_OK;
}

rola_status rola_cross_attend(const rola_cross_params* p, const void* q, const void* k, const void* v,
                              const int32_t* kv_len, const uint8_t* key_mask, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, rola_stream_t stream) {
  const rola_status s = check(p);
  if (s != ROLA_OK) return s;
  if (!given(q) || !given(k) || !given(v) || !given(out) || !words(lse) || !words(kv_len))
    return ROLA_ERR_INVALID_ARG;
  const size_t need = forward_bytes(*p);
  if (need && (!given(workspace) || workspace_bytes < need)) return ROLA_ERR_WORKSPACE;
  const View in[] = {View(q, p->B, p->Nq, p->H, p->d, p->dtype, p->q), View(k, p->B, p->Nk, p->H, p->d, p->dtype, p->k),
                     View(v, p->B, p->Nk, p->H, p->d, p->dtype, p->v)};
  const size_t rows = (size_t)p->B * p->Nq * p->H;
  const struct { const void* p; size_t n; } outs[] = {
      {out, rows * p->d * elem_size(p->dtype)}, {lse, lse ? 4 * rows : 0}, {need ? workspace : nullptr, need}};
  for (const View& i : in)
    if (!i.strides_ok()) return ROLA_ERR_INVALID_ARG;
  for (int a = 0; a < 3; ++a) {
    if (!outs[a].p) continue;
    for (const View& i : in)
      if (overlaps(i, outs[a].p, outs[a].n)) return ROLA_ERR_INVALID_ARG;
    for (int c = a + 1; c < 3; ++c)
      if (outs[c].p && overlaps(outs[a].p, outs[a].n, outs[c].p, outs[c].n)) return ROLA_ERR_INVALID_ARG;
    if (kv_len && overlaps(outs[a].p, outs[a].n, kv_len, 4 * (size_t)p->B)) return ROLA_ERR_INVALID_ARG;
    if (key_mask && overlaps(outs[a].p, outs[a].n, key_mask, (size_t)p->B * p->Nk)) return ROLA_ERR_INVALID_ARG;
  }
  const CrossArgs a = args_of(*p, kv_len, key_mask);
  const int splits = forward_splits(*p);
  float* part = static_cast<float*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p->dtype == ROLA_F32)
    return cuda_status(rola::launch_cross_simt(a, splits, static_cast<const float*>(q), static_cast<const float*>(k),
                                               static_cast<const float*>(v), static_cast<float*>(out), lse, part, st));
  return cuda_status(rola::launch_cross_sm100(a, splits, q, k, v, out, lse, part, st));
}

rola_status rola_cross_backward_workspace_size(const rola_cross_params* p, size_t* bytes) {
  if (!bytes) return ROLA_ERR_INVALID_ARG;
  const rola_status s = check(p);
  if (s != ROLA_OK) return s;
  *bytes = backward_bytes(*p);
  return ROLA_OK;
}

rola_status rola_cross_attend_backward(const rola_cross_params* p, const void* dout, const void* q, const void* k,
                                       const void* v, const void* out, const float* lse, const int32_t* kv_len,
                                       const uint8_t* key_mask, void* dq, void* dk, void* dv, void* workspace,
                                       size_t workspace_bytes, rola_stream_t stream) {
  const rola_status s = check(p);
  if (s != ROLA_OK) return s;
  for (const void* x : {dout, q, k, v, out, (const void*)dq, (const void*)dk, (const void*)dv})
    if (!given(x)) return ROLA_ERR_INVALID_ARG;
  if (!lse || !words(lse) || !words(kv_len)) return ROLA_ERR_INVALID_ARG;
  const size_t need = backward_bytes(*p);
  if (!given(workspace) || workspace_bytes < need) return ROLA_ERR_WORKSPACE;
  const View in[] = {View(dout, p->B, p->Nq, p->H, p->d, p->dtype, p->dout),
                     View(q, p->B, p->Nq, p->H, p->d, p->dtype, p->q), View(k, p->B, p->Nk, p->H, p->d, p->dtype, p->k),
                     View(v, p->B, p->Nk, p->H, p->d, p->dtype, p->v),
                     View::contiguous(out, p->B, p->Nq, p->H, p->d, p->dtype)};
  const size_t el = elem_size(p->dtype), rows = (size_t)p->B * p->Nq * p->H, nk = (size_t)p->B * p->Nk * p->H * p->d;
  const struct { const void* p; size_t n; } outs[] = {
      {dq, rows * p->d * el}, {dk, nk * el}, {dv, nk * el}, {workspace, need}};
  for (const View& i : in)
    if (!i.strides_ok()) return ROLA_ERR_INVALID_ARG;
  for (int a = 0; a < 4; ++a) {
    for (const View& i : in)
      if (overlaps(i, outs[a].p, outs[a].n)) return ROLA_ERR_INVALID_ARG;
    for (int c = a + 1; c < 4; ++c)
      if (overlaps(outs[a].p, outs[a].n, outs[c].p, outs[c].n)) return ROLA_ERR_INVALID_ARG;
    if (overlaps(outs[a].p, outs[a].n, lse, 4 * rows)) return ROLA_ERR_INVALID_ARG;
    if (kv_len && overlaps(outs[a].p, outs[a].n, kv_len, 4 * (size_t)p->B)) return ROLA_ERR_INVALID_ARG;
    if (key_mask && overlaps(outs[a].p, outs[a].n, key_mask, (size_t)p->B * p->Nk)) return ROLA_ERR_INVALID_ARG;
  }
  const CrossSplits sp = backward_splits(*p);
  float* stats = static_cast<float*>(workspace);
  float* part = stats + stats_bytes(*p) / 4;
  const CrossArgs a = args_of(*p, kv_len, key_mask);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p->dtype == ROLA_F32)
    return cuda_status(rola::launch_cross_simt_backward(
        a, sp.queries, sp.keys, static_cast<const float*>(dout), static_cast<const float*>(q),
        static_cast<const float*>(k), static_cast<const float*>(v), static_cast<const float*>(out), lse,
        static_cast<float*>(dq), static_cast<float*>(dk), static_cast<float*>(dv), stats, part, st));
  return cuda_status(rola::launch_cross_sm100_backward(a, sp.queries, sp.keys, dout, q, k, v, out, lse, dq, dk, dv,
                                                       stats, part, st));
}

rola_status rola_block_poll_status(rola_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int word = 0;
  int back = 0;
  if (cudaStreamSynchronize(st) != cudaSuccess || rola::cross_sm100_status(&word, st) != cudaSuccess ||
      rola::cross_sm100_backward_status(&back, st) != cudaSuccess)
    return ROLA_ERR_CUDA;
  return static_cast<rola_status>(word ? word : back);
}

}  // extern "C"

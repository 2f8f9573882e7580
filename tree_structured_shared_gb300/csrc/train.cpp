// Host side of the operators around the tree attention of a training step: rotation
// of packed rows and its tables, the cross entropy of a large vocabulary, 8-bit
// checkpoints.  Checks of arguments, then one of the launchers; nothing here allocates.
#include "../../include/padoc.h"
#include "padoc_internal.h"

#include <algorithm>
#include <cmath>
#include <string>

using namespace padoc;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// n rows of `row` bytes, `step` bytes apart.
struct Rows {
  const void* p;
  int64_t row, step, n;
};
__int128 floor_div(__int128 a, __int128 b) { return a >= 0 ? a / b : -((-a + b - 1) / b); }
// Whether two lists of rows share a byte.  Exact for equal steps and where one list is
// dense; otherwise lists whose ranges meet count as sharing one.
bool overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.n <= 0 || b.n <= 0 || a.row <= 0 || b.row <= 0) return false;
  const __int128 x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const __int128 xe = x + static_cast<__int128>(a.n - 1) * a.step + a.row;
  const __int128 ye = y + static_cast<__int128>(b.n - 1) * b.step + b.row;
  if (xe <= y || ye <= x) return false;
  if (a.step == b.step) {
    // row i of b begins at y + i step; relative to a row of a it lies m steps and y - x on
    const __int128 s = a.step, delta = y - x;
    const __int128 m = std::max<__int128>(floor_div(-static_cast<__int128>(b.row) - delta, s) + 1, -(b.n > a.n ? b.n : a.n) + 1);
    return m < std::max(a.n, b.n) && delta + m * s < a.row;
  }
  const bool a_dense = a.row == a.step || a.n == 1;
  if (!a_dense && b.row != b.step && b.n != 1) return true;
  const Rows& r = a_dense ? b : a;  // rows against the other's one range
  const __int128 lo = a_dense ? x : y, hi = a_dense ? xe : ye, p = a_dense ? y : x;
  const __int128 i = lo < p + r.row ? 0 : (lo - p - r.row) / r.step + 1;  // the first row that ends behind lo
  return i < r.n && p + i * r.step < hi;
}
Rows range(const void* p, int64_t bytes) { return Rows{p, bytes, bytes, bytes > 0 ? 1 : 0}; }

}  // namespace

// ============================================================== rotation

extern "C" int padoc_rope_table(const padoc_rope_scaling* sc, int64_t first, int32_t n_pos, float* cos_sin,
                                padoc_stream_t stream) {
  if (!sc) return set_error(PADOC_ERR_INVALID, "rope_table: null scaling");
  if (sc->rot_dim < 32 || sc->rot_dim > 128 || sc->rot_dim % 32)
    return set_error(PADOC_ERR_INVALID, "rope_table: rot_dim must be a multiple of 32 in [32, 128]");
  if (!(sc->base > 1.0) || !std::isfinite(sc->base))
    return set_error(PADOC_ERR_INVALID, "rope_table: base must be a finite number above 1");
  if (sc->kind < PADOC_ROPE_PLAIN || sc->kind > PADOC_ROPE_RAMP)
    return set_error(PADOC_ERR_INVALID, "rope_table: unknown kind %d", sc->kind);
  if (sc->kind != PADOC_ROPE_PLAIN && (!(sc->factor >= 1.0) || !std::isfinite(sc->factor)))
    return set_error(PADOC_ERR_INVALID, "rope_table: factor must be a finite number of at least 1");
  if (sc->kind == PADOC_ROPE_BANDS || sc->kind == PADOC_ROPE_RAMP) {
    if (!(sc->context > 0.0) || !std::isfinite(sc->context))
      return set_error(PADOC_ERR_INVALID, "rope_table: context must be positive");
    if (!(sc->turns_lo > 0.0) || !(sc->turns_hi > sc->turns_lo) || !std::isfinite(sc->turns_hi))
      return set_error(PADOC_ERR_INVALID, "rope_table: turns must satisfy 0 < turns_lo < turns_hi");
  }
  if (!(sc->amplitude >= 0.0) || !std::isfinite(static_cast<float>(sc->amplitude)))
    return set_error(PADOC_ERR_INVALID, "rope_table: amplitude must be a finite number of at least 0 (0 means 1)");
  if (first < 0 || n_pos < 0 || first > (1ll << 31) - n_pos)
    return set_error(PADOC_ERR_INVALID, "rope_table: positions must lie in [0, 2^31)");
  if (n_pos == 0) return PADOC_OK;
  if (!cos_sin || !aligned16(cos_sin))
    return set_error(PADOC_ERR_INVALID, "rope_table: cos_sin must be a 16-byte aligned device pointer");
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  RopeTableArgs a{};
  a.cos_sin = cos_sin;
  a.first = first;
  a.n_pos = n_pos;
  a.rot_dim = sc->rot_dim;
  a.amplitude = sc->amplitude > 0.0 ? static_cast<float>(sc->amplitude) : 1.f;
  const double rot = sc->rot_dim;
  const double base = sc->kind == PADOC_ROPE_BASE ? sc->base * std::pow(sc->factor, rot / (rot - 2.0)) : sc->base;
  if (!std::isfinite(base)) return set_error(PADOC_ERR_INVALID, "rope_table: base and factor are too large");
  double lo = 0.0, hi = 0.0;
  if (sc->kind == PADOC_ROPE_RAMP) {
    // the pair (as a real number) that makes r turns over the context
    auto pair = [&](double r) { return rot * std::log(sc->context / (r * kTwoPi)) / (2.0 * std::log(base)); };
    lo = std::max(std::floor(pair(sc->turns_hi)), 0.0);
    hi = std::min(std::ceil(pair(sc->turns_lo)), rot - 1.0);
  }
  for (int i = 0; i < sc->rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (sc->kind == PADOC_ROPE_LINEAR) f /= sc->factor;
    if (sc->kind == PADOC_ROPE_BANDS || sc->kind == PADOC_ROPE_RAMP) {
      double keep;
      if (sc->kind == PADOC_ROPE_BANDS)
        keep = (sc->context * f / kTwoPi - sc->turns_lo) / (sc->turns_hi - sc->turns_lo);
      else
        keep = 1.0 - (i - lo) / std::max(hi - lo, 0.001);
      keep = std::min(1.0, std::max(0.0, keep));
      f *= keep + (1.0 - keep) / sc->factor;
    }
    a.turns[i] = static_cast<uint64_t>(std::ldexp(f / kTwoPi, 64));  // f <= 1, so below 2^62
  }
  std::string err;
  const int rc = launch_rope_table(a, reinterpret_cast<cudaStream_t>(stream), &err);
  return rc ? set_error(rc, "rope_table: %s", err.c_str()) : PADOC_OK;
}

extern "C" int padoc_rope_apply(const padoc_rope* rope, int32_t n_parts, const padoc_rope_part* parts, int32_t dtype,
                                int32_t d, int64_t n, const int32_t* positions, int32_t backward,
                                padoc_stream_t stream) {
  if (!rope) return set_error(PADOC_ERR_INVALID, "rope_apply: null rope");
  if (n_parts < 1 || n_parts > kRopeParts || !parts)
    return set_error(PADOC_ERR_INVALID, "rope_apply: between 1 and %d parts are needed", kRopeParts);
  if (dtype != PADOC_BF16 && dtype != PADOC_F32) return set_error(PADOC_ERR_INVALID, "rope_apply: unknown dtype %d", dtype);
  if (d != 64 && d != 128) return set_error(PADOC_ERR_UNSUPPORTED, "rope_apply: d must be 64 or 128");
  if (rope->rot_dim < 0 || rope->rot_dim > d || rope->rot_dim % 32)
    return set_error(PADOC_ERR_INVALID, "rope_apply: rot_dim must be a multiple of 32 in [0, d]");
  if (n < 0) return set_error(PADOC_ERR_INVALID, "rope_apply: negative row count");
  if (!aligned4(positions)) return set_error(PADOC_ERR_INVALID, "rope_apply: positions must be aligned to 4 bytes");
  const int size = dtype == PADOC_BF16 ? 2 : 4, vec = 16 / size;
  RopeArgs a{};
  int64_t heads = 0;
  for (int i = 0; i < n_parts; ++i) {
    const padoc_rope_part& p = parts[i];
    if (p.heads < 0) return set_error(PADOC_ERR_INVALID, "rope_apply: negative head count");
    const int64_t row = static_cast<int64_t>(p.heads) * d;
    if (n > 0 && p.heads > 0) {
      if (!p.x || !p.out || !aligned16(p.x) || !aligned16(p.out))
        return set_error(PADOC_ERR_INVALID, "rope_apply: x and out must be 16-byte aligned device pointers");
      if (p.stride < row || p.out_stride < row || p.stride % vec || p.out_stride % vec)
        return set_error(PADOC_ERR_INVALID, "rope_apply: row strides must be multiples of 16 bytes of at least heads * d");
    }
    a.first[i] = static_cast<int32_t>(heads);
    a.x[i] = p.x;
    a.out[i] = p.out;
    a.stride[i] = p.stride;
    a.out_stride[i] = p.out_stride;
    heads += p.heads;
    if (heads > (1 << 20)) return set_error(PADOC_ERR_UNSUPPORTED, "rope_apply: too many heads");
  }
  for (int i = n_parts; i < kRopeParts; ++i) a.first[i] = static_cast<int32_t>(heads);
  if (n == 0 || heads == 0) return PADOC_OK;
  if (rope->rot_dim > 0) {
    if (!rope->cos_sin || !aligned16(rope->cos_sin))
      return set_error(PADOC_ERR_INVALID, "rope_apply: cos_sin must be a 16-byte aligned device pointer");
    if (rope->n_pos < 0) return set_error(PADOC_ERR_INVALID, "rope_apply: negative table length");
    if (!positions && n > rope->n_pos)
      return set_error(PADOC_ERR_INVALID, "rope_apply: %lld rows without positions need a table as long, not of %d",
                       static_cast<long long>(n), rope->n_pos);
  }
  // Rows are turned in no order: an output may lie on its own input, row on row, and on
  // nothing else that the call reads or writes.
  const Rows table = range(rope->cos_sin, static_cast<int64_t>(rope->n_pos) * rope->rot_dim * 4);
  const Rows pos = range(positions, n * 4);
  for (int i = 0; i < n_parts; ++i) {
    const int64_t row = static_cast<int64_t>(parts[i].heads) * d * size;
    const Rows out{parts[i].out, row, parts[i].out_stride * size, n};
    for (int j = 0; j < n_parts; ++j) {
      const int64_t row_j = static_cast<int64_t>(parts[j].heads) * d * size;
      const Rows in{parts[j].x, row_j, parts[j].stride * size, n}, other{parts[j].out, row_j, parts[j].out_stride * size, n};
      const bool same = i == j && out.p == in.p && (n == 1 || out.step == in.step);
      if ((!same && overlap(out, in)) || (i != j && overlap(out, other)))
        return set_error(PADOC_ERR_INVALID, "rope_apply: an output overlaps rows that the call reads or writes elsewhere");
    }
    if (overlap(out, table) || overlap(out, pos))
      return set_error(PADOC_ERR_INVALID, "rope_apply: an output overlaps the table or the positions");
  }
  a.cos_sin = rope->cos_sin;
  a.positions = positions;
  a.n = n;
  a.n_pos = rope->n_pos;
  a.rot_dim = rope->rot_dim;
  a.interleaved = rope->interleaved;
  a.backward = backward;
  a.heads = static_cast<int32_t>(heads);
  std::string err;
  const int rc = launch_rope_apply(a, dtype, d, reinterpret_cast<cudaStream_t>(stream), &err);
  return rc ? set_error(rc, "rope_apply: %s", err.c_str()) : PADOC_OK;
}

// ============================================================== 8-bit checkpoints

extern "C" int padoc_act_bytes(int64_t n, int32_t width, size_t* bytes) {
  if (!bytes) return set_error(PADOC_ERR_INVALID, "act_bytes: null argument");
  if (n < 0 || width <= 0 || width % 32)
    return set_error(PADOC_ERR_INVALID, "act_bytes: width must be a positive multiple of 32, and n not negative");
  *bytes = static_cast<size_t>(n) * width + static_cast<size_t>(n) * (width / 32);
  return PADOC_OK;
}

static int act_call(int32_t n_tensors, const padoc_act* t, bool keep, const char* what, padoc_stream_t stream) {
  if (n_tensors < 0 || n_tensors > kActTensors || (n_tensors > 0 && !t))
    return set_error(PADOC_ERR_INVALID, "%s: between 0 and %d tensors are allowed", what, kActTensors);
  ActArgs a{};
  a.n = n_tensors;
  a.sums = -1;
  for (int i = 0; i < n_tensors; ++i) {
    if (t[i].n < 0 || t[i].width <= 0 || t[i].width % 32)
      return set_error(PADOC_ERR_INVALID, "%s: width must be a positive multiple of 32, and n not negative", what);
    if (t[i].n == 0) continue;
    if (!t[i].rows || !t[i].kept || !aligned16(t[i].rows) || !aligned16(t[i].kept))
      return set_error(PADOC_ERR_INVALID, "%s: rows and kept must be 16-byte aligned device pointers", what);
    if (t[i].stride < t[i].width || t[i].stride % 8)
      return set_error(PADOC_ERR_INVALID, "%s: the row stride must be a multiple of 8 of at least the width", what);
    if (t[i].n > (static_cast<int64_t>(UINT32_MAX) * 16) / t[i].width)
      return set_error(PADOC_ERR_UNSUPPORTED, "%s: too many values in one tensor", what);
    a.t[i].rows = t[i].rows;
    a.t[i].stride = t[i].stride;
    a.t[i].kept = static_cast<uint8_t*>(t[i].kept);
    a.t[i].pieces = t[i].n * (t[i].width / 16);
    a.t[i].per_row = static_cast<uint32_t>(t[i].width / 16);
    a.t[i].dense = t[i].stride == t[i].width || t[i].n == 1;
  }
  for (int i = 0; i < n_tensors; ++i) {
    const int64_t width = t[i].width;
    const Rows rows{t[i].rows, width * 2, t[i].stride * 2, t[i].n};
    const Rows kept = range(t[i].kept, t[i].n * width + t[i].n * (width / 32));
    for (int j = 0; j < n_tensors; ++j) {
      const int64_t w = t[j].width;
      const Rows rows_j{t[j].rows, w * 2, t[j].stride * 2, t[j].n};
      const Rows kept_j = range(t[j].kept, t[j].n * w + t[j].n * (w / 32));
      const Rows& out = keep ? kept : rows;
      if (overlap(out, keep ? rows_j : kept_j) || (i != j && overlap(out, keep ? kept_j : rows_j)))
        return set_error(PADOC_ERR_INVALID, "%s: an output overlaps what the call reads or writes elsewhere", what);
    }
  }
  std::string err;
  const int rc = launch_act(a, keep, reinterpret_cast<cudaStream_t>(stream), &err);
  return rc ? set_error(rc, "%s: %s", what, err.c_str()) : PADOC_OK;
}

extern "C" int padoc_act_keep(int32_t n_tensors, const padoc_act* tensors, padoc_stream_t stream) {
  return act_call(n_tensors, tensors, true, "act_keep", stream);
}
extern "C" int padoc_act_restore(int32_t n_tensors, const padoc_act* tensors, padoc_stream_t stream) {
  return act_call(n_tensors, tensors, false, "act_restore", stream);
}

// ============================================================== cross entropy

static int lm_shape(int32_t n, int32_t D, int32_t V, const char* what) {
  if (n < 0 || D <= 0 || V <= 0 || D % 8)
    return set_error(PADOC_ERR_INVALID, "%s: n must not be negative, V positive, and D a positive multiple of 8", what);
  const int64_t tiles = ((static_cast<int64_t>(n) + 255) / 256) * ((static_cast<int64_t>(V) + 255) / 256);
  if (n > (1 << 25) || D > (1 << 20) || V > (1 << 28) || tiles > (1 << 28))
    return set_error(PADOC_ERR_UNSUPPORTED, "%s: n, D, V or n * V is too large", what);
  return PADOC_OK;
}

extern "C" int padoc_lm_loss_ws_size(int32_t n, int32_t D, int32_t V, int32_t backward, size_t* bytes) {
  if (!bytes) return set_error(PADOC_ERR_INVALID, "lm_loss_ws_size: null argument");
  const int rc = lm_shape(n, D, V, "lm_loss_ws_size");
  if (rc) return rc;
  *bytes = n == 0 ? 0 : lm_plan(n, D, V, false).bytes;
  if (backward && n > 0) *bytes = std::max(*bytes, lm_plan(n, D, V, true).bytes);
  return PADOC_OK;
}

static int lm_check(const padoc_lm_head* head, const void* ws, size_t ws_bytes, bool backward, LmCall* l, const char* what) {
  if (!head) return set_error(PADOC_ERR_INVALID, "%s: null head", what);
  const int rc = lm_shape(head->n, head->D, head->V, what);
  if (rc) return rc;
  if (head->n == 0) return PADOC_OK;
  if (!head->h || !head->w || !head->targets || !aligned16(head->h) || !aligned16(head->w) || !aligned4(head->targets))
    return set_error(PADOC_ERR_INVALID, "%s: h and w must be 16-byte aligned device pointers, and targets a 4-byte aligned one", what);
  if (head->h_stride < head->D || head->w_stride < head->D || head->h_stride % 8 || head->w_stride % 8)
    return set_error(PADOC_ERR_INVALID, "%s: row strides must be multiples of 8 of at least D", what);
  const size_t need = lm_plan(head->n, head->D, head->V, backward).bytes;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || ws_bytes < need)
    return set_error(PADOC_ERR_INVALID, "%s: ws must be 256-byte aligned and hold %zu bytes", what, need);
  l->h = head->h;
  l->h_stride = head->h_stride;
  l->w = head->w;
  l->w_stride = head->w_stride;
  l->targets = head->targets;
  l->n = head->n;
  l->D = head->D;
  l->V = head->V;
  return PADOC_OK;
}

// Outputs (and the workspace) apart from each other and from what is read.
static int lm_apart(const padoc_lm_head* h, const Rows* in, int n_in, const Rows* out, int n_out, const char* what) {
  const Rows read[3] = {Rows{h->h, static_cast<int64_t>(h->D) * 2, h->h_stride * 2, h->n},
                        Rows{h->w, static_cast<int64_t>(h->D) * 2, h->w_stride * 2, h->V},
                        range(h->targets, static_cast<int64_t>(h->n) * 4)};
  for (int i = 0; i < n_out; ++i) {
    bool bad = false;
    for (const Rows& r : read) bad = bad || overlap(out[i], r);
    for (int j = 0; j < n_in; ++j) bad = bad || overlap(out[i], in[j]);
    for (int j = 0; j < n_out; ++j) bad = bad || (j != i && overlap(out[i], out[j]));
    if (bad) return set_error(PADOC_ERR_INVALID, "%s: an output or the workspace overlaps what the call reads or writes elsewhere", what);
  }
  return PADOC_OK;
}

extern "C" int padoc_lm_loss(const padoc_lm_head* head, float* loss, float* lse, void* ws, size_t ws_bytes,
                             padoc_stream_t stream) {
  LmCall l{};
  int rc = lm_check(head, ws, ws_bytes, false, &l, "lm_loss");
  if (rc || head->n == 0) return rc;
  if (!loss || !lse || !aligned4(loss) || !aligned4(lse))
    return set_error(PADOC_ERR_INVALID, "lm_loss: loss and lse must be 4-byte aligned device pointers");
  const int64_t n4 = static_cast<int64_t>(l.n) * 4;
  const Rows out[3] = {range(loss, n4), range(lse, n4), range(ws, static_cast<int64_t>(lm_plan(l.n, l.D, l.V, false).bytes))};
  rc = lm_apart(head, nullptr, 0, out, 3, "lm_loss");
  if (rc) return rc;
  l.loss = loss;
  l.lse = lse;
  std::string err;
  rc = launch_lm_loss(l, ws, reinterpret_cast<cudaStream_t>(stream), &err);
  return rc ? set_error(rc, "lm_loss: %s", err.c_str()) : PADOC_OK;
}

extern "C" int padoc_lm_loss_bwd(const padoc_lm_head* head, const float* lse, const float* d_loss, void* dh, void* dw,
                                 void* ws, size_t ws_bytes, padoc_stream_t stream) {
  LmCall l{};
  int rc = lm_check(head, ws, ws_bytes, true, &l, "lm_loss_bwd");
  if (rc) return rc;
  if ((dh && !aligned16(dh)) || (dw && !aligned16(dw)))
    return set_error(PADOC_ERR_INVALID, "lm_loss_bwd: dh and dw must be 16-byte aligned");
  const int64_t w_bytes = static_cast<int64_t>(head->V) * head->D * 2;
  if (head->n == 0) {  // no row: the weights' gradient is zero
    if (!dw) return PADOC_OK;
    const cudaError_t e = cudaMemsetAsync(dw, 0, static_cast<size_t>(w_bytes), reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PADOC_OK : set_error(PADOC_ERR_CUDA, "lm_loss_bwd: cudaMemsetAsync: %s", cudaGetErrorString(e));
  }
  if (!lse || !d_loss || !aligned4(lse) || !aligned4(d_loss))
    return set_error(PADOC_ERR_INVALID, "lm_loss_bwd: lse and d_loss must be 4-byte aligned device pointers");
  if (!dh && !dw) return PADOC_OK;
  const int64_t n4 = static_cast<int64_t>(l.n) * 4;
  const Rows in[2] = {range(lse, n4), range(d_loss, n4)};
  const Rows out[3] = {range(dh, dh ? static_cast<int64_t>(l.n) * l.D * 2 : 0), range(dw, dw ? w_bytes : 0),
                       range(ws, static_cast<int64_t>(lm_plan(l.n, l.D, l.V, true).bytes))};
  rc = lm_apart(head, in, 2, out, 3, "lm_loss_bwd");
  if (rc) return rc;
  l.lse = const_cast<float*>(lse);
  l.d_loss = d_loss;
  l.dh = dh;
  l.dw = dw;
  std::string err;
  rc = launch_lm_loss_bwd(l, ws, reinterpret_cast<cudaStream_t>(stream), &err);
  return rc ? set_error(rc, "lm_loss_bwd: %s", err.c_str()) : PADOC_OK;
}

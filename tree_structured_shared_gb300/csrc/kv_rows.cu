// Rows in and out of the paged KV pool.
//
//   kv_write_kernel   rows of K and V into pool slots, K turned by its
//                     position on the way (and, in the same launch, Q), into a
//                     bf16 or a 4-bit pool
//   kv_gather_kernel  cached rows of a bf16 or 4-bit pool as dense bf16 K, V
//
// Rotation of a pair (a, b) by the angle of its position, cosine and sine from
// an f32 table: (a c - b s, b c + a s), in f32, each product and sum rounded
// on its own (so the result does not depend on how a compiler contracts it).
//
// Both kernels are streams, bound by HBM once the rows fill the GPU and by the
// launch below that.  A record names up to 16 consecutive rows of one block
// and is one CTA.  To write, a warp takes eight (token, head) at a time, K and V of
// them together: four lanes a head, each with two whole groups of 16 dims.  Where pairs
// are half a rotation apart, the two groups are partners, elsewhere neighbours, so
// neither the rotation nor a group's scale needs an exchange between lanes.  To read
// back, a warp takes a token, lanes 0-15 K's 128 dims and lanes 16-31 V's.
// Small record lists ride in the kernel's parameters: no upload is needed.
//
// Measured (16 query heads, 8 kv heads, all dims turned): 16 x 4809 rows into a bf16
// pool in 225 us, 6.3 TB/s; 64 x 4809 rows into a 4-bit pool and back out in 1030 us
// (941 at HBM rate), the way back at HBM rate (64 pages of 4000-6144 tokens in 260 us,
// 6.6 TB/s); 1-16 rows of 1490 sequences and back in 74 us.  384 rows of one token take
// 4 us.  Before, with sixteen lanes a head and 8 dims a lane, a group spread over four
// lanes, a token cost twice the instructions (1190 and 82 us).  Eight heads of a token
// instead of eight tokens of a head to a 4-bit pool: 1102 us (its bytes are scattered
// over the unit, 44 sectors written become 176); to a bf16 pool the other way round:
// 255 us.  The write holds three CTAs an SM; two, or four (which spills), take 9 and
// 7 % longer, two query heads on their way at once (which spills) 7 %, rows prefetched
// to L2 by the CTA nothing.
#include <cuda_bf16.h>

#include <string>

#include "../../include/padoc.h"
#include "kv_i4.cuh"
#include "padoc_internal.h"
#include "ptx_sm103.cuh"

namespace padoc {
namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWriteCtas = 3;

struct InlineRecs {
  RowRec r[kInlineRecs];
};
struct NoRecs {};

// A lane's two groups of 16 dims of a row, bf16.
struct Raw {
  uint4 a[2], b[2];
};
__device__ __forceinline__ Raw load_raw(const __nv_bfloat16* row, int ga, int gb) {
  const uint4 *a = reinterpret_cast<const uint4*>(row + 16 * ga), *b = reinterpret_cast<const uint4*>(row + 16 * gb);
  return Raw{{__ldcs(a), __ldcs(a + 1)}, {__ldcs(b), __ldcs(b + 1)}};
}
__device__ __forceinline__ void store_raw(__nv_bfloat16* row, int ga, int gb, const Raw& r) {
  uint4 *a = reinterpret_cast<uint4*>(row + 16 * ga), *b = reinterpret_cast<uint4*>(row + 16 * gb);
  a[0] = r.a[0];
  a[1] = r.a[1];
  b[0] = r.b[0];
  b[1] = r.b[1];
}
__device__ __forceinline__ void unpack(const uint4 (&u)[2], float (&x)[16]) {
  const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void pack(const float (&x)[16], uint4 (&u)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    u[h] = make_uint4(pack_bf16x2(x[8 * h], x[8 * h + 1]), pack_bf16x2(x[8 * h + 2], x[8 * h + 3]),
                      pack_bf16x2(x[8 * h + 4], x[8 * h + 5]), pack_bf16x2(x[8 * h + 6], x[8 * h + 7]));
}

__device__ __forceinline__ RowRec get_rec(const RowsArgs& a, const InlineRecs& in, int r) { return in.r[r]; }
__device__ __forceinline__ RowRec get_rec(const RowsArgs& a, const NoRecs&, int r) {
  if (a.recs) return a.recs[r];
  // rows of one sequence, through its row of the block table
  const int b = a.seq_first / 16 + r;
  const int lo = max(a.seq_first, b * 16), hi = min(a.seq_first + static_cast<int>(a.n_rows), (b + 1) * 16);
  return RowRec{lo - a.seq_first, a.table_row[b], (lo & 15) | ((hi - lo) << 8), 0};
}

// RN(x / b) from y = RN(1 / b), by Markstein's theorem: q = x y, r = x - q b
// exact, q + r y.
__device__ __forceinline__ float quotient(float x, float b, float y) {
  const float q = __fmul_rn(x, y);
  return fmaf(fmaf(-q, b, x), y, q);
}

// RN(1 / s) of an s with a four-bit significand: one Newton step on an estimate
// good to 2^-22.  1 - s y is exact (28 bits), so the step leaves (1 - e^2) / s
// with e below 2^-22, and no 1 / m, m = 9 .. 15, lies as near as 2^-44 to a
// midpoint between floats.
__device__ __forceinline__ float short_reciprocal(float s) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  return fmaf(fmaf(-s, y, 1.f), y, y);
}

// The codes of a quad as a word has them when the quad is its lower one (shifted
// up by 8 for the upper one): codes 0..3 at nibbles 0, 4, 1, 5.  A quotient is
// rounded to the nearest integer, ties to even, by adding 1.5 * 2^23 + 8, which
// leaves n + 8 in the low bits.  Only a scale below 2^-14 or at its limit lets a
// quotient pass 7.5 (elsewhere it is at most 7 * 17 / 16), so only those clamp.
template <bool CLAMP>
__device__ __forceinline__ uint32_t i4_quad(const float* x, float s, float y) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float n = quotient(x[i], s, y);
    if (CLAMP) n = fminf(fmaxf(n, -7.f), 7.f);
    b[i] = __float_as_uint(n + 12582920.f);  // 0x4B400000 + 8 + n
  }
  return (b[0] + b[1] * 65536u) + (b[2] + b[3] * 65536u) * 16u - 0x4B400000u * 0x110011u;
}

// A group's two words of codes and its scale byte.
struct Group {
  uint32_t w0, w1, scale;
};
template <bool CLAMP>
__device__ __forceinline__ void i4_codes(const float (&x)[16], float s, float y, Group* g) {
  g->w0 = i4_quad<CLAMP>(x, s, y) | i4_quad<CLAMP>(x + 4, s, y) << 8;
  g->w1 = i4_quad<CLAMP>(x + 8, s, y) | i4_quad<CLAMP>(x + 12, s, y) << 8;
}
// The largest magnitude; a NaN if there is one.
__device__ __forceinline__ float largest(const float (&x)[16]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 16; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(x[i])));
  return m;
}
// A lane's two groups; whether one holds a NaN or an infinity (its codes are then of no
// use).  The whole warp calls it.
__device__ __forceinline__ bool quantise(const float (&xa)[16], const float (&xb)[16], Group* a, Group* b) {
  constexpr float kSeventh = 1.f / 7.f;
  const float la = largest(xa), lb = largest(xb);
  const bool bad = !(la < INFINITY) || !(lb < INFINITY);
  const float ma = quotient(la, 7.f, kSeventh), mb = quotient(lb, 7.f, kSeventh);
  if (__any_sync(0xffffffffu, !i4_plain(ma) || !i4_plain(mb))) {
    a->scale = i4_scale_byte(bad ? 0.f : ma);
    b->scale = i4_scale_byte(bad ? 0.f : mb);
    const float sa = i4_scale_value(a->scale), sb = i4_scale_value(b->scale);
    // a scale of zero: every code is that of zero
    i4_codes<true>(xa, sa, a->scale ? __frcp_rn(sa) : 0.f, a);
    i4_codes<true>(xb, sb, b->scale ? __frcp_rn(sb) : 0.f, b);
  } else {
    const float sa = i4_plain_scale(ma, &a->scale), sb = i4_plain_scale(mb, &b->scale);
    i4_codes<false>(xa, sa, short_reciprocal(sa), a);
    i4_codes<false>(xb, sb, short_reciprocal(sb), b);
  }
  return bad;
}

template <bool I4, class RECS>
__global__ void __launch_bounds__(kThreads, kWriteCtas) kv_write_kernel(const __grid_constant__ RowsArgs a,
                                                                        const __grid_constant__ RECS in) {
  const RowRec rec = get_rec(a, in, blockIdx.x);
  const int n = rec.slot_n >> 8, slot0 = rec.slot_n & 255;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane & 3, sub = lane >> 2;
  // the lane's two groups of dims: half a rotation apart where they turn so
  const int hr = a.rot_dim / 2;
  const bool turns = 32 * l < a.rot_dim, split = turns && !a.interleaved;
  const int ga = split ? l : 2 * l, gb = split ? l + hr / 16 : 2 * l + 1;
  auto rotate = [&](float (&xa)[16], float (&xb)[16], int64_t row, int t) {
    if (!turns) return;
    const int pos = a.positions ? a.positions[row] : rec.pos + t;
    const float* tab = a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim + 16 * l;
    auto turn = [](float& p, float& q, float c, float s) {
      const float u = __fsub_rn(__fmul_rn(p, c), __fmul_rn(q, s));
      q = __fadd_rn(__fmul_rn(q, c), __fmul_rn(p, s));
      p = u;
    };
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      float cs[4], sn[4];
      *reinterpret_cast<float4*>(cs) = *reinterpret_cast<const float4*>(tab + i);
      *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(tab + hr + i);
      if (a.interleaved) {
        // the lane's pair i + j: dims 2 (i + j), + 1 of its 32
#pragma unroll
        for (int j = 0; j < 4; ++j)
          turn(i < 8 ? xa[2 * (i + j)] : xb[2 * (i + j) - 16], i < 8 ? xa[2 * (i + j) + 1] : xb[2 * (i + j) - 15], cs[j], sn[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) turn(xa[i + j], xb[i + j], cs[j], sn[j]);
      }
    }
  };
  // passes of eight (token, head): K and V together, then Q
  const int n_kv = n * a.Hkv, n_q = a.q ? n * a.Hq : 0;
  const int kv_passes = (n_kv + 7) / 8, passes = kv_passes + (n_q + 7) / 8;
  for (int pass = warp; pass < passes; pass += kWarps) {
    const bool is_q = pass >= kv_passes;
    const int last = (is_q ? n_q : n_kv) - 1;
    const int p = (is_q ? pass - kv_passes : pass) * 8 + sub;
    const bool ok = p <= last;
    const int at = min(p, last);
    int t, u;
    if (I4 && !is_q) {
      // eight slots of a head fill whole sectors of its unit
      u = at / n;
      t = at - u * n;
    } else {
      // a token's heads lie side by side and share its angles
      const int H = is_q ? a.Hq : a.Hkv;
      t = at / H;
      u = at - t * H;
    }
    const int64_t row = static_cast<int64_t>(rec.row) + t;
    float xa[16], xb[16];
    Raw r;
    if (is_q) {
      r = load_raw(a.q + row * a.q_stride + u * kHeadDim, ga, gb);
      unpack(r.a, xa);
      unpack(r.b, xb);
      rotate(xa, xb, row, t);
      pack(xa, r.a);
      pack(xb, r.b);
      if (ok) store_raw(a.q_rot + (row * a.Hq + u) * kHeadDim, ga, gb, r);
      continue;
    }
    r = load_raw(a.k + row * a.k_stride + u * kHeadDim, ga, gb);
    const Raw rv = load_raw(a.v + row * a.v_stride + u * kHeadDim, ga, gb);
    const int64_t unit = static_cast<int64_t>(rec.block) * a.Hkv + u;
    const int slot = slot0 + t;
    unpack(r.a, xa);
    unpack(r.b, xb);
    rotate(xa, xb, row, t);
    if (a.k_rot || !I4) {
      pack(xa, r.a);
      pack(xb, r.b);
      if (ok && a.k_rot) store_raw(a.k_rot + (row * a.Hkv + u) * kHeadDim, ga, gb, r);
    }
    if (!I4) {
      const int64_t dst = (unit * 16 + slot) * kHeadDim;
      if (ok) {
        store_raw(static_cast<__nv_bfloat16*>(a.k_pool) + dst, ga, gb, r);
        store_raw(static_cast<__nv_bfloat16*>(a.v_pool) + dst, ga, gb, rv);
      }
    } else {
      Group k0, k1, v0, v1;
      bool bad = quantise(xa, xb, &k0, &k1);
      unpack(rv.a, xa);
      unpack(rv.b, xb);
      bad |= quantise(xa, xb, &v0, &v1);
      // a NaN or an infinity in this token's K or V of this head (its four lanes): K
      // becomes NaN (through its first group) and V zero, so every query that sees the
      // token gets NaN and no other does
      if (__ballot_sync(0xffffffffu, bad) & (15u << (lane & 28))) {
        k0 = Group{0x88888888u, 0x88888888u, ga == 0 ? kI4Nan : 0u};
        k1 = v0 = v1 = Group{0x88888888u, 0x88888888u, 0u};
      }
      if (ok) {
        uint8_t *k = static_cast<uint8_t*>(a.k_pool) + unit * kI4Unit, *v = static_cast<uint8_t*>(a.v_pool) + unit * kI4Unit;
        auto put_k = [&](int g, const Group& x) {
          *reinterpret_cast<uint2*>(k + (g >> 1) * 256 + slot * 16 + (g & 1) * 8) = make_uint2(x.w0, x.w1);
          k[kI4Scales + slot * 8 + g] = static_cast<uint8_t>(x.scale);
        };
        auto put_v = [&](int g, const Group& x) {
          *reinterpret_cast<uint2*>(v + g * 128 + slot * 8) = make_uint2(x.w0, x.w1);
          v[kI4Scales + g * 16 + slot] = static_cast<uint8_t>(x.scale);
        };
        put_k(ga, k0);
        put_k(gb, k1);
        put_v(ga, v0);
        put_v(gb, v1);
      }
    }
  }
}

// Lane l of a half warp takes a row's dims 8 l .. 8 l + 7, of K or of V.
template <bool I4, class RECS>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const __grid_constant__ RowsArgs a,
                                                             const __grid_constant__ RECS in) {
  const RowRec rec = get_rec(a, in, blockIdx.x);
  const int n = rec.slot_n >> 8, slot0 = rec.slot_n & 255;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane & 15, half = lane >> 4;
  const int hg_n = n == 1 ? 8 : n == 2 ? 4 : n <= 4 ? 2 : 1;  // warps that share a token's heads
  constexpr int kUnroll = 4;
  for (int item = warp; item < n * hg_n; item += kWarps) {
    const int t = item / hg_n, hg = item - t * hg_n;
    const int slot = slot0 + t;
    const uint8_t* pool = static_cast<const uint8_t*>(half ? a.v_pool : a.k_pool);
    const int64_t bh = static_cast<int64_t>(rec.block) * a.Hkv;
    const int word_at = half ? (l >> 1) * 128 + slot * 8 + (l & 1) * 4 : (l >> 2) * 256 + slot * 16 + (l & 3) * 4;
    const int scale_at = kI4Scales + (half ? (l >> 1) * 16 + slot : slot * 8 + (l >> 1));
    const uint8_t* src = I4 ? pool + bh * kI4Unit : pool + ((bh * 16 + slot) * kHeadDim + 8 * l) * 2;
    __nv_bfloat16* dst = (half ? a.v_out : a.k_out) + (static_cast<int64_t>(rec.row) + t) * a.Hkv * kHeadDim + 8 * l;
    for (int u0 = hg; u0 < a.Hkv; u0 += hg_n * kUnroll) {
      uint4 w[kUnroll];
      uint32_t b[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int u = u0 + i * hg_n;
        if (u >= a.Hkv) break;
        if (I4) {
          w[i].x = *reinterpret_cast<const uint32_t*>(src + u * kI4Unit + word_at);
          b[i] = src[u * kI4Unit + scale_at];
        } else {
          w[i] = __ldcs(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(u) * 16 * kHeadDim * 2));
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int u = u0 + i * hg_n;
        if (u >= a.Hkv) break;
        uint4 out = w[i];
        if (I4) {
          // a code or-ed under 128 in bf16 makes 136 + n; n and n s are exact
          const float s = i4_scale_value(b[i]);
          const uint32_t s2 = pack_bf16x2(s, s), x = w[i].x;
          auto pair = [&](uint32_t v) {
            uint32_t d;
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(mask_or(v, 0x000F000Fu, 0x43004300u)), "r"(0x43084308u));
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(d) : "r"(s2));
            return d;
          };
          out = make_uint4(pair(x), pair(x >> 4), pair(x >> 8), pair(x >> 12));
        }
        __stcs(reinterpret_cast<uint4*>(dst + u * kHeadDim), out);
      }
    }
  }
}

int launch_error(const char* what, std::string* err) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return PADOC_OK;
  *err = std::string(what) + ": " + cudaGetErrorString(e);
  return PADOC_ERR_CUDA;
}

InlineRecs inline_recs(const RowsArgs& a) {
  InlineRecs in{};
  for (int i = 0; i < a.n_recs; ++i) in.r[i] = a.host_recs[i];
  return in;
}

}  // namespace

int launch_kv_write(const RowsArgs& a, cudaStream_t s, std::string* err) {
  if (a.n_recs == 0) return PADOC_OK;
  if (a.host_recs) {
    const InlineRecs in = inline_recs(a);
    if (a.i4)
      kv_write_kernel<true, InlineRecs><<<a.n_recs, kThreads, 0, s>>>(a, in);
    else
      kv_write_kernel<false, InlineRecs><<<a.n_recs, kThreads, 0, s>>>(a, in);
  } else if (a.i4) {
    kv_write_kernel<true, NoRecs><<<a.n_recs, kThreads, 0, s>>>(a, NoRecs{});
  } else {
    kv_write_kernel<false, NoRecs><<<a.n_recs, kThreads, 0, s>>>(a, NoRecs{});
  }
  return launch_error("kv write launch", err);
}

int launch_kv_gather(const RowsArgs& a, cudaStream_t s, std::string* err) {
  if (a.n_recs == 0) return PADOC_OK;
  if (a.host_recs) {
    const InlineRecs in = inline_recs(a);
    if (a.i4)
      kv_gather_kernel<true, InlineRecs><<<a.n_recs, kThreads, 0, s>>>(a, in);
    else
      kv_gather_kernel<false, InlineRecs><<<a.n_recs, kThreads, 0, s>>>(a, in);
  } else if (a.i4) {
    kv_gather_kernel<true, NoRecs><<<a.n_recs, kThreads, 0, s>>>(a, NoRecs{});
  } else {
    kv_gather_kernel<false, NoRecs><<<a.n_recs, kThreads, 0, s>>>(a, NoRecs{});
  }
  return launch_error("kv gather launch", err);
}

}  // namespace padoc

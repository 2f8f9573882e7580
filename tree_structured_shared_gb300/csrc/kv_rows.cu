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
// and is one CTA; a warp takes a token and walks its heads, lanes 0-15 holding
// the 128 dims of K (or of one query head), lanes 16-31 those of V (or of the
// next query head), so the table is read once a token.  A lane holds two quads
// of dims, A and B.  Where pairs are half a rotation apart, quad A of the lanes
// that turn is the pairs' first dims and B their second, so a rotation needs no
// exchange between lanes; elsewhere A and B are neighbours.
// Small record lists ride in the kernel's parameters: no upload is needed.
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

struct InlineRecs {
  RowRec r[kInlineRecs];
};
struct NoRecs {};

struct Quads {
  uint2 a, b;  // bf16
};
__device__ __forceinline__ void unpack(const Quads& u, float (&x)[8]) {
  const uint32_t w[4] = {u.a.x, u.a.y, u.b.x, u.b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store(__nv_bfloat16* row, int da, int db, const float (&x)[8]) {
  *reinterpret_cast<uint2*>(row + da) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  *reinterpret_cast<uint2*>(row + db) = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ RowRec get_rec(const RowsArgs& a, const InlineRecs& in, int r) { return in.r[r]; }
__device__ __forceinline__ RowRec get_rec(const RowsArgs& a, const NoRecs&, int r) {
  if (a.recs) return a.recs[r];
  // rows of one sequence, through its row of the block table
  const int b = a.seq_first / 16 + r;
  const int lo = max(a.seq_first, b * 16), hi = min(a.seq_first + static_cast<int>(a.n_rows), (b + 1) * 16);
  return RowRec{lo - a.seq_first, a.table_row[b], (lo & 15) | ((hi - lo) << 8), 0};
}

// The codes of a quad as a word has them when the quad is its lower one (shifted
// up by 8 for the upper one): codes 0..3 at nibbles 0, 4, 1, 5.
//
// n = x / s rounded to the nearest integer, ties to even.  The quotient is
// correctly rounded by Markstein's theorem (q = x y, r = x - q s exact,
// q' = q + r y, with y the correctly rounded reciprocal of s), so that a tie is
// a tie; adding 1.5 * 2^23 + 8 leaves n + 8 in the low bits of the sum.
__device__ __forceinline__ uint32_t i4_quad(const float* x, float s, float y) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q = __fmul_rn(x[i], y);
    const float n = fminf(fmaxf(fmaf(fmaf(-q, s, x[i]), y, q), -7.f), 7.f);
    const uint32_t bits = __float_as_uint(n + 12582920.f) - 0x4B400000u;
    w += bits << (4 * (i >> 1) + 16 * (i & 1));
  }
  return w;
}

template <bool I4, class RECS>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const __grid_constant__ RowsArgs a,
                                                            const __grid_constant__ RECS in) {
  const RowRec rec = get_rec(a, in, blockIdx.x);
  const int n = rec.slot_n >> 8, slot0 = rec.slot_n & 255;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane & 15, half = lane >> 4;  // K (half 0) or V (half 1)
  // few tokens: several warps share a token's heads
  const int hg_n = n == 1 ? 8 : n == 2 ? 4 : n <= 4 ? 2 : 1;
  const int n_units = a.Hkv + (a.q ? (a.Hq + 1) / 2 : 0);
  const int hr = a.rot_dim / 2;
  const bool split = !a.interleaved && 8 * l < a.rot_dim;  // quads a half rotation apart
  const bool turns = 8 * l < a.rot_dim;
  const int da = split ? 4 * l : 8 * l, db = split ? hr + 4 * l : 8 * l + 4;
  for (int item = warp; item < n * hg_n; item += kWarps) {
    const int t = item / hg_n, hg = item - t * hg_n;
    const int64_t src = static_cast<int64_t>(rec.row) + t;
    const int slot = slot0 + t;
    // the lane's four angles
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (turns) {
      const int pos = a.positions ? a.positions[src] : rec.pos + t;
      const float* tab = a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim + 4 * l;
      *reinterpret_cast<float4*>(cs) = *reinterpret_cast<const float4*>(tab);
      *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(tab + hr);
    }
    constexpr int kUnroll = 4;
    for (int u0 = hg; u0 < n_units; u0 += hg_n * kUnroll) {
      Quads ld[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int u = u0 + i * hg_n;
        const __nv_bfloat16* p = nullptr;
        if (u < a.Hkv) {
          p = (half ? a.v + src * a.v_stride : a.k + src * a.k_stride) + u * kHeadDim;
        } else {
          const int h = 2 * (u - a.Hkv) + half;
          if (u < n_units && h < a.Hq) p = a.q + src * a.q_stride + h * kHeadDim;
        }
        ld[i].a = p ? __ldcs(reinterpret_cast<const uint2*>(p + da)) : make_uint2(0, 0);
        ld[i].b = p ? __ldcs(reinterpret_cast<const uint2*>(p + db)) : make_uint2(0, 0);
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int u = u0 + i * hg_n;
        if (u >= n_units) break;
        const bool kv = u < a.Hkv;
        float x[8];
        unpack(ld[i], x);
        if (turns && !(kv && half)) {
          float y[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // pair j: quads' dims j, or dims 2j, 2j + 1
            const float p = split ? x[j] : x[2 * j], q = split ? x[4 + j] : x[2 * j + 1];
            const float r0 = __fsub_rn(__fmul_rn(p, cs[j]), __fmul_rn(q, sn[j]));
            const float r1 = __fadd_rn(__fmul_rn(q, cs[j]), __fmul_rn(p, sn[j]));
            y[j] = r0;
            y[4 + j] = r1;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = split ? y[j] : y[(j >> 1) + 4 * (j & 1)];
        }
        if (!kv) {
          const int h = 2 * (u - a.Hkv) + half;
          if (h < a.Hq) store(a.q_rot + (src * a.Hq + h) * kHeadDim, da, db, x);
          continue;
        }
        if (a.k_rot && !half) store(a.k_rot + (src * a.Hkv + u) * kHeadDim, da, db, x);
        const int64_t bh = static_cast<int64_t>(rec.block) * a.Hkv + u;
        if (!I4) {
          store(static_cast<__nv_bfloat16*>(half ? a.v_pool : a.k_pool) + (bh * 16 + slot) * kHeadDim, da, db, x);
        } else {
          // the largest magnitude of each quad's group: of four neighbouring lanes
          // where the quads lie apart, of two lanes' both quads elsewhere
          float ma = fmaxf(max3f(fabsf(x[0]), fabsf(x[1]), fabsf(x[2])), fabsf(x[3]));
          float mb = fmaxf(max3f(fabsf(x[4]), fabsf(x[5]), fabsf(x[6])), fabsf(x[7]));
          // 0 unless one is NaN or infinite
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) sum = fmaf(x[j], 0.f, sum);
          if (!split) ma = mb = fmaxf(ma, mb);
          ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, 1));
          mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
          const float ma2 = __shfl_xor_sync(0xffffffffu, ma, 2), mb2 = __shfl_xor_sync(0xffffffffu, mb, 2);
          if (split) {
            ma = fmaxf(ma, ma2);
            mb = fmaxf(mb, mb2);
          }
          uint32_t ba = i4_scale_byte(__fdiv_rn(ma, 7.f)), bb = i4_scale_byte(__fdiv_rn(mb, 7.f));
          const float sa = i4_scale_value(ba), sb = i4_scale_value(bb);
          // a scale of zero: every code is that of zero
          uint32_t wa = i4_quad(x, sa, ba ? __frcp_rn(sa) : 0.f);
          uint32_t wb = i4_quad(x + 4, sb, bb ? __frcp_rn(sb) : 0.f);
          // a NaN or an infinity in this token's K or V of this head: K becomes
          // NaN (through its first group) and V zero, so every query that sees
          // the token gets NaN and no other does
          if (__any_sync(0xffffffffu, !(sum == 0.f))) {
            wa = wb = 0x00880088u;
            ba = !half && da < 16 ? kI4Nan : 0u;
            bb = !half && db < 16 ? kI4Nan : 0u;
          }
          // one word a lane: of its own two quads, or of two neighbours' A (even lane) or B (odd lane)
          const uint32_t other = __shfl_xor_sync(0xffffffffu, (l & 1) ? wa : wb, 1);
          const uint32_t word = !split ? wa | wb << 8 : (l & 1) ? other | wb << 8 : wa | other << 8;
          const int at = !split ? l : ((l & 1) ? hr / 8 : 0) + (l >> 1);  // word of the row
          // and one scale: of a group's first lane
          const bool has = split ? (l & 2) == 0 : (l & 1) == 0;
          const uint32_t b = split && (l & 1) ? bb : ba;
          const int grp = at >> 1;
          uint8_t* dst = static_cast<uint8_t*>(half ? a.v_pool : a.k_pool) + bh * kI4Unit;
          if (!half) {
            *reinterpret_cast<uint32_t*>(dst + (at >> 2) * 256 + slot * 16 + (at & 3) * 4) = word;
            if (has) dst[kI4Scales + slot * 8 + grp] = static_cast<uint8_t>(b);
          } else {
            *reinterpret_cast<uint32_t*>(dst + grp * 128 + slot * 8 + (at & 1) * 4) = word;
            if (has) dst[kI4Scales + grp * 16 + slot] = static_cast<uint8_t>(b);
          }
        }
      }
    }
  }
}

template <bool I4, class RECS>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const __grid_constant__ RowsArgs a,
                                                             const __grid_constant__ RECS in) {
  const RowRec rec = get_rec(a, in, blockIdx.x);
  const int n = rec.slot_n >> 8, slot0 = rec.slot_n & 255;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane & 15, half = lane >> 4;
  for (int item = warp; item < n * a.Hkv; item += kWarps) {
    const int t = item / a.Hkv, h = item - t * a.Hkv;
    const int64_t dst = ((static_cast<int64_t>(rec.row) + t) * a.Hkv + h) * kHeadDim + 8 * l;
    const int slot = slot0 + t;
    const int64_t bh = static_cast<int64_t>(rec.block) * a.Hkv + h;
    uint4 out;
    if (!I4) {
      const __nv_bfloat16* pool = static_cast<const __nv_bfloat16*>(half ? a.v_pool : a.k_pool);
      out = *reinterpret_cast<const uint4*>(pool + (bh * 16 + slot) * kHeadDim + 8 * l);
    } else {
      const uint8_t* s = static_cast<const uint8_t*>(half ? a.v_pool : a.k_pool) + bh * kI4Unit;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(
          half ? s + (l >> 1) * 128 + slot * 8 + (l & 1) * 4 : s + (l >> 2) * 256 + slot * 16 + (l & 3) * 4);
      const uint32_t b = half ? s[kI4Scales + (l >> 1) * 16 + slot] : s[kI4Scales + slot * 8 + (l >> 1)];
      const I4Scale sc = i4_scale(b | b << 16);
      const uint32_t p[4] = {i4_pair<0>(w, w >> 8, sc), i4_pair<1>(w, w >> 8, sc), i4_pair<2>(w, w >> 8, sc),
                             i4_pair<3>(w, w >> 8, sc)};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
        o[i] = pack_bf16x2(f.x * kI4Unscale, f.y * kI4Unscale);  // exact: a value has at most 7 significant bits
      }
      out = make_uint4(o[0], o[1], o[2], o[3]);
    }
    __stcs(reinterpret_cast<uint4*>((half ? a.v_out : a.k_out) + dst), out);
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

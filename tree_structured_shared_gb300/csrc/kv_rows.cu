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
//
// Measured (16 query heads, 8 kv heads, all dims turned): 16 x 4809 rows into a bf16
// pool in 225 us, 6.3 TB/s; 64 x 4809 rows into a 4-bit pool and back out in 1190 us
// (941 at HBM rate): the write, about 200 warp instructions a (token, kv head) to
// scale and round, is bound by instruction issue, the way back by HBM (64 pages of
// 4000-6144 tokens in 260 us, 6.6 TB/s).  384 rows of one token take 4 us.  Finer or
// coarser splits of a token's heads over the warps: the same or slower (1-16 rows of
// 1490 sequences, write and way back: 82 us; two warps a token 84, eight 121).
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

// A lane's two quads of a row whose quad A starts at p, quad B db elements on.
struct Quads {
  uint2 a, b;  // bf16
};
__device__ __forceinline__ Quads load_quads(const __nv_bfloat16* p, int db) {
  return Quads{__ldcs(reinterpret_cast<const uint2*>(p)), __ldcs(reinterpret_cast<const uint2*>(p + db))};
}
__device__ __forceinline__ void unpack(const Quads& u, float (&x)[8]) {
  const uint32_t w[4] = {u.a.x, u.a.y, u.b.x, u.b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store(__nv_bfloat16* p, int db, const float (&x)[8]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  *reinterpret_cast<uint2*>(p + db) = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
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

template <bool I4, class RECS>
__global__ void __launch_bounds__(kThreads, 3) kv_write_kernel(const __grid_constant__ RowsArgs a,
                                                            const __grid_constant__ RECS in) {
  const RowRec rec = get_rec(a, in, blockIdx.x);
  const int n = rec.slot_n >> 8, slot0 = rec.slot_n & 255;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane & 15, half = lane >> 4;  // K (half 0) or V (half 1)
  // few tokens: several warps share a token's heads
  const int hg_n = n == 1 ? 8 : n == 2 ? 4 : n <= 4 ? 2 : 1;
  const int hr = a.rot_dim / 2;
  const bool turns = 8 * l < a.rot_dim;
  const bool split = turns && !a.interleaved;  // quads a half rotation apart
  const int da = split ? 4 * l : 8 * l, db = split ? hr : 4;
  const int n_q = a.q ? (a.Hq + 1) / 2 : 0;  // pairs of query heads
  // where the lane's word of codes and, if it has one, its scale go (I4)
  const int word_at = !split ? l : ((l & 1) ? hr / 8 : 0) + (l >> 1);
  const int grp = word_at >> 1;
  const bool has_scale = split ? (l & 2) == 0 : (l & 1) == 0;
  constexpr int kUnroll = 4;
  for (int item = warp; item < n * hg_n; item += kWarps) {
    const int t = item / hg_n, hg = item - t * hg_n;
    const int64_t src = static_cast<int64_t>(rec.row) + t;
    const int slot = slot0 + t;
    // the lane's four angles
    float cs[4], sn[4];
    if (turns) {
      const int pos = a.positions ? a.positions[src] : rec.pos + t;
      const float* tab = a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim + 4 * l;
      *reinterpret_cast<float4*>(cs) = *reinterpret_cast<const float4*>(tab);
      *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(tab + hr);
    }
    auto rotate = [&](float (&x)[8]) {
      // pair j: dims j of the two quads, or dims 2j, 2j + 1
      auto turn = [&](float& p, float& q, int j) {
        const float u = __fsub_rn(__fmul_rn(p, cs[j]), __fmul_rn(q, sn[j]));
        q = __fadd_rn(__fmul_rn(q, cs[j]), __fmul_rn(p, sn[j]));
        p = u;
      };
      if (!turns) return;
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) turn(x[2 * j], x[2 * j + 1], j);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) turn(x[j], x[4 + j], j);
      }
    };
    {
      const __nv_bfloat16* in = (half ? a.v + src * a.v_stride : a.k + src * a.k_stride) + da;
      __nv_bfloat16* rot = a.k_rot && !half ? a.k_rot + src * a.Hkv * kHeadDim + da : nullptr;
      const int64_t bh = static_cast<int64_t>(rec.block) * a.Hkv;
      uint8_t* pool = static_cast<uint8_t*>(half ? a.v_pool : a.k_pool);
      // I4: the word's place, the scale's; bf16: the row's
      uint8_t* dst = I4 ? pool + bh * kI4Unit + (half ? grp * 128 + slot * 8 + (word_at & 1) * 4
                                                      : (word_at >> 2) * 256 + slot * 16 + (word_at & 3) * 4)
                        : pool + ((bh * 16 + slot) * kHeadDim + da) * 2;
      const int scale_at = kI4Scales + (half ? grp * 16 + slot : slot * 8 + grp) -
                           (half ? grp * 128 + slot * 8 + (word_at & 1) * 4 : (word_at >> 2) * 256 + slot * 16 + (word_at & 3) * 4);
      for (int u0 = hg; u0 < a.Hkv; u0 += hg_n * kUnroll) {
        Quads ld[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
          if (u0 + i * hg_n < a.Hkv) ld[i] = load_quads(in + (u0 + i * hg_n) * kHeadDim, db);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          const int u = u0 + i * hg_n;
          if (u >= a.Hkv) break;
          float x[8];
          unpack(ld[i], x);
          if (!half) rotate(x);
          if (rot) store(rot + u * kHeadDim, db, x);
          if (!I4) {
            store(reinterpret_cast<__nv_bfloat16*>(dst) + u * 16 * kHeadDim, db, x);
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
            constexpr float kSeventh = 1.f / 7.f;
            ma = quotient(ma, 7.f, kSeventh);
            mb = quotient(mb, 7.f, kSeventh);
            uint32_t wa, wb, ba, bb;
            if (__any_sync(0xffffffffu, !(sum == 0.f) || !i4_plain(ma) || !i4_plain(mb))) {
              ba = i4_scale_byte(ma);
              bb = i4_scale_byte(mb);
              const float sa = i4_scale_value(ba), sb = i4_scale_value(bb);
              // a scale of zero: every code is that of zero
              wa = i4_quad<true>(x, sa, ba ? __frcp_rn(sa) : 0.f);
              wb = i4_quad<true>(x + 4, sb, bb ? __frcp_rn(sb) : 0.f);
              // a NaN or an infinity in this token's K or V of this head: K becomes
              // NaN (through its first group) and V zero, so every query that sees
              // the token gets NaN and no other does
              if (__any_sync(0xffffffffu, !(sum == 0.f))) {
                wa = wb = 0x00880088u;
                ba = !half && da < 16 ? kI4Nan : 0u;
                bb = !half && da + db < 16 ? kI4Nan : 0u;
              }
            } else {
              const float sa = i4_plain_scale(ma, &ba), sb = i4_plain_scale(mb, &bb);
              wa = i4_quad<false>(x, sa, short_reciprocal(sa));
              wb = i4_quad<false>(x + 4, sb, short_reciprocal(sb));
            }
            // one word a lane: of its own two quads, or of two neighbours' A (even lane) or B (odd lane)
            const uint32_t other = __shfl_xor_sync(0xffffffffu, (l & 1) ? wa : wb, 1);
            uint8_t* p = dst + u * kI4Unit;
            *reinterpret_cast<uint32_t*>(p) = !split ? wa | wb << 8 : (l & 1) ? other | wb << 8 : wa | other << 8;
            if (has_scale) p[scale_at] = static_cast<uint8_t>(split && (l & 1) ? bb : ba);
          }
        }
      }
    }
    if (n_q) {
      const __nv_bfloat16* in = a.q + src * a.q_stride + half * kHeadDim + da;
      __nv_bfloat16* rot = a.q_rot + (src * a.Hq + half) * kHeadDim + da;
      for (int u0 = hg; u0 < n_q; u0 += hg_n * kUnroll) {
        Quads ld[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          const int h = 2 * (u0 + i * hg_n);
          if (h + half < a.Hq) ld[i] = load_quads(in + h * kHeadDim, db);
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          const int h = 2 * (u0 + i * hg_n);
          if (h + half >= a.Hq) continue;
          float x[8];
          unpack(ld[i], x);
          rotate(x);
          store(rot + h * kHeadDim, db, x);
        }
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

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
// the 128 dims of K (or of one query head) in 16-byte pieces, lanes 16-31
// those of V (or of the next query head), so the table is read once a token.
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

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ RowRec get_rec(const RowsArgs& a, const InlineRecs& in, int r) { return in.r[r]; }
__device__ __forceinline__ RowRec get_rec(const RowsArgs& a, const NoRecs&, int r) {
  if (a.recs) return a.recs[r];
  // rows of one sequence, through its row of the block table
  const int b = a.seq_first / 16 + r;
  const int lo = max(a.seq_first, b * 16), hi = min(a.seq_first + static_cast<int>(a.n_rows), (b + 1) * 16);
  return RowRec{lo - a.seq_first, a.table_row[b], (lo & 15) | ((hi - lo) << 8), 0};
}

// Codes and scale of a lane's 8 dims, half of a group of 16 (the lane pair
// l, l ^ 1 holds the group): the word of codes and the group's scale byte.
__device__ __forceinline__ void i4_encode(const float (&x)[8], uint32_t* word, uint32_t* scale) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const uint32_t b = i4_scale_byte(__fdiv_rn(m, 7.f));
  const float s = i4_scale_value(b);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float n = b ? fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -7.f), 7.f) : 0.f;
    const uint32_t code = static_cast<uint32_t>(static_cast<int>(n) + 8);
    w |= code << (4 * ((i >> 1) + 4 * (i & 1)));
  }
  *word = w;
  *scale = b;
}

template <bool I4, class RECS>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const __grid_constant__ RowsArgs a,
                                                            const __grid_constant__ RECS in) {
  const RowRec rec = get_rec(a, in, blockIdx.x);
  const int n = rec.slot_n >> 8, slot0 = rec.slot_n & 255;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane & 15, half = lane >> 4;  // dims 8 l .. 8 l + 7 of K (half 0) or V (half 1)
  // few tokens: several warps share a token's heads
  const int hg_n = n == 1 ? 8 : n == 2 ? 4 : n <= 4 ? 2 : 1;
  const int n_units = a.Hkv + (a.q ? (a.Hq + 1) / 2 : 0);
  const int d0 = 8 * l, hr = a.rot_dim / 2;
  for (int item = warp; item < n * hg_n; item += kWarps) {
    const int t = item / hg_n, hg = item - t * hg_n;
    const int64_t src = static_cast<int64_t>(rec.row) + t;
    const int slot = slot0 + t;
    // the lane's angles: for half-split pairs (i, i + hr) eight, for interleaved pairs four
    float cs[8], sn[8];
    if (d0 < a.rot_dim) {
      const int pos = a.positions ? a.positions[src] : rec.pos + t;
      const float* tab = a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim;
      if (a.interleaved) {
        *reinterpret_cast<float4*>(cs) = *reinterpret_cast<const float4*>(tab + d0 / 2);
        *reinterpret_cast<float4*>(sn) = *reinterpret_cast<const float4*>(tab + hr + d0 / 2);
      } else {
        const float* p = tab + (d0 < hr ? d0 : d0 - hr);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          reinterpret_cast<float4*>(cs)[i] = reinterpret_cast<const float4*>(p)[i];
          reinterpret_cast<float4*>(sn)[i] = reinterpret_cast<const float4*>(p + hr)[i];
        }
      }
    }
    const int partner = (lane & 16) | (d0 < hr ? l + (hr >> 3) : l - (hr >> 3));
    constexpr int kUnroll = 4;
    for (int u0 = hg; u0 < n_units; u0 += hg_n * kUnroll) {
      uint4 ld[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int u = u0 + i * hg_n;
        ld[i] = make_uint4(0, 0, 0, 0);
        if (u < a.Hkv) {
          const __nv_bfloat16* p = half ? a.v + src * a.v_stride : a.k + src * a.k_stride;
          ld[i] = __ldcs(reinterpret_cast<const uint4*>(p + u * kHeadDim + d0));
        } else if (u < n_units) {
          const int h = 2 * (u - a.Hkv) + half;
          if (h < a.Hq) ld[i] = __ldcs(reinterpret_cast<const uint4*>(a.q + src * a.q_stride + h * kHeadDim + d0));
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int u = u0 + i * hg_n;
        if (u >= n_units) break;
        const bool kv = u < a.Hkv;
        float x[8];
        unpack8(ld[i], x);
        if (a.rot_dim) {
          float y[8];
          if (a.interleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              y[2 * j] = __fsub_rn(__fmul_rn(x[2 * j], cs[j]), __fmul_rn(x[2 * j + 1], sn[j]));
              y[2 * j + 1] = __fadd_rn(__fmul_rn(x[2 * j + 1], cs[j]), __fmul_rn(x[2 * j], sn[j]));
            }
          } else {
            const bool low = d0 < hr;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float p = __shfl_sync(0xffffffffu, x[j], partner & 31);
              const float xc = __fmul_rn(x[j], cs[j]), ps = __fmul_rn(p, sn[j]);
              y[j] = low ? __fsub_rn(xc, ps) : __fadd_rn(xc, ps);
            }
          }
          if (d0 < a.rot_dim && !(kv && half)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = y[j];
          }
        }
        if (!kv) {
          const int h = 2 * (u - a.Hkv) + half;
          if (h < a.Hq) *reinterpret_cast<uint4*>(a.q_rot + (src * a.Hq + h) * kHeadDim + d0) = pack8(x);
          continue;
        }
        if (a.k_rot && !half) *reinterpret_cast<uint4*>(a.k_rot + (src * a.Hkv + u) * kHeadDim + d0) = pack8(x);
        const int64_t bh = static_cast<int64_t>(rec.block) * a.Hkv + u;
        if (!I4) {
          __nv_bfloat16* pool = static_cast<__nv_bfloat16*>(half ? a.v_pool : a.k_pool);
          *reinterpret_cast<uint4*>(pool + (bh * 16 + slot) * kHeadDim + d0) = pack8(x);
        } else {
          bool bad = false;
#pragma unroll
          for (int j = 0; j < 8; ++j) bad |= !(fabsf(x[j]) <= 3.4028235e38f);
          uint32_t w, s;
          // a NaN or an infinity in this token's K or V of this head: K becomes
          // NaN (through its first group) and V zero, so every query that sees
          // the token gets NaN and no other does
          if (__any_sync(0xffffffffu, bad)) {
            w = 0x88888888u;
            s = (!half && l < 2) ? kI4Nan : 0u;
          } else {
            i4_encode(x, &w, &s);
          }
          uint8_t* dst = static_cast<uint8_t*>(half ? a.v_pool : a.k_pool) + bh * kI4Unit;
          if (!half) {
            *reinterpret_cast<uint32_t*>(dst + (l >> 2) * 256 + slot * 16 + (l & 3) * 4) = w;
            if (!(l & 1)) dst[kI4Scales + slot * 8 + (l >> 1)] = static_cast<uint8_t>(s);
          } else {
            *reinterpret_cast<uint32_t*>(dst + (l >> 1) * 128 + slot * 8 + (l & 1) * 4) = w;
            if (!(l & 1)) dst[kI4Scales + (l >> 1) * 16 + slot] = static_cast<uint8_t>(s);
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

// Activations kept in 8 bits between a forward and its backward pass.
//
//   keep_kernel     bf16 rows -> codes and scales
//   restore_kernel  codes and scales -> bf16 rows; for the attention's backward pass
//                   also the row sums D = dO . O straight from O's codes
//
// 32 neighbours of a row share a scale, a power of two: the smallest (at least 2^-126
// and at most 2^121) of which 127 reach the group's largest magnitude; a code is the
// nearest integer (ties to even) in [-127, 127].  code * scale has seven significant
// bits at most, so it is exact in bf16 and nothing is rounded on the way back.  (A scale
// with bits of its own would lie a third nearer on average, but its products would be
// rounded to bf16 when they are restored.)  An infinity or a NaN gives its group the
// scale byte 255, and all of the group reads back as NaN.
//
// Streams, bound by HBM: 2 bytes a value in and 1 + 1/32 out, or the reverse.  Two lanes
// share a group, so its largest magnitude takes one exchange, and a lane moves 32 bytes
// of values and 16 of codes.  Magnitudes are compared as integers, two at a time: bf16
// bits without the sign are in the order of the values, infinities and NaNs on top.
//
// 131072 rows of 6144 values in four tensors: kept in 360 us, restored in 364, 6.7 TB/s (360
// each at the copy rate).  462 rows of 1536: 4 us each, a launch.
#include <cuda_bf16.h>

#include <algorithm>
#include <string>

#include "../../include/padoc.h"
#include "padoc_internal.h"
#include "ptx_sm103.cuh"

namespace padoc {
namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kUnroll = 2;  // pieces of 16 values a thread, kThreads apart
constexpr int64_t kPiecesRound = kThreads * kUnroll;
// A CTA costs its launch: long tensors take kRounds of them one after another (131072 rows
// of 6144 values 360 and 364 us; with one round 379 and 404, with 16 5 us more than with
// four); short ones
// spread over the GPU (462 rows of 1536 4.3 us, with four rounds 6.3).
constexpr int kRounds = 4, kManyRounds = 16 * 152;

// 16 values from a place that is 16-byte aligned.
struct Piece {
  uint32_t w[8];
};
__device__ __forceinline__ Piece load_piece(const __nv_bfloat16* p) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p)), b = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
  return Piece{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// The value index of piece i of a tensor whose rows are `per_row` pieces long.
__device__ __forceinline__ int64_t piece_at(const ActTensor& x, uint32_t i) {
  if (x.dense) return static_cast<int64_t>(i) * 16;
  const uint32_t row = i / x.per_row;
  return static_cast<int64_t>(row) * x.stride + static_cast<int64_t>(i - row * x.per_row) * 16;
}

__device__ __forceinline__ int find(const ActArgs& a, int block) {
  int t = 0;
#pragma unroll
  for (int i = 1; i < kActTensors; ++i) t += block >= a.first_block[i];
  return t;
}

__global__ void __launch_bounds__(kThreads) keep_kernel(const __grid_constant__ ActArgs a) {
  const int ti = find(a, blockIdx.x);
  const ActTensor& x = a.t[ti];
  const int64_t begin = static_cast<int64_t>(blockIdx.x - a.first_block[ti]) * a.pieces_cta;
  const int64_t end = min(x.pieces, begin + a.pieces_cta);
  for (int64_t i0 = begin + threadIdx.x; i0 - threadIdx.x < end; i0 += kPiecesRound) {
    Piece p[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i0 + u * kThreads < x.pieces)
        p[u] = load_piece(static_cast<const __nv_bfloat16*>(x.rows) + piece_at(x, static_cast<uint32_t>(i0 + u * kThreads)));
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = i0 + u * kThreads;
      const bool in = i < x.pieces;  // both lanes of a pair or neither: pieces are even
      uint32_t m = 0;
      if (in) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m = __vmaxu2(m, p[u].w[j] & 0x7fff7fffu);
      }
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m & 0xffffu, m >> 16);
      if (!in) continue;
      const bool bad = m >= 0x7f80u;
      // of bf16's largest value 127 steps of 2^121 fall short, but 64 of 2^122 are infinite
      const uint32_t e = min(max(static_cast<int>(m >> 7) - 6 + ((m & 0x7f) == 0x7f), 1), 248);
      const float inv = __uint_as_float((254u - e) << 23);
      uint32_t code[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t b[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t w = p[u].w[2 * j + k];
          if (m == 0x7f7fu) w -= __vcmpeq2(w & 0x7fff7fffu, 0x7f7f7f7fu) & 0x00010001u;  // the value below it is 127 steps
          // the product is exact; the sum rounds it to an integer, whose low byte is the code
          b[2 * k] = __float_as_uint(fmaf(__uint_as_float(w << 16), inv, 12582912.f));
          b[2 * k + 1] = __float_as_uint(fmaf(__uint_as_float(w & 0xffff0000u), inv, 12582912.f));
        }
        code[j] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        if (bad) code[j] = 0;
      }
      *reinterpret_cast<uint4*>(x.kept + i * 16) = make_uint4(code[0], code[1], code[2], code[3]);
      if (!(i & 1)) x.kept[x.pieces * 16 + i / 2] = static_cast<uint8_t>(bad ? 255u : e);
    }
  }
}

__device__ __forceinline__ float scale_of(uint8_t b) {
  return __uint_as_float(b == 255 ? 0x7fffffffu : static_cast<uint32_t>(b) << 23);
}
// Four codes as floats: a byte plus 128 in the low bits of 2^23, less 2^23 + 128.
__device__ __forceinline__ void codes_up(uint32_t c, float* x) {
  c ^= 0x80808080u;
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(__byte_perm(c, 0x4b000000u, 0x7440 + k)) - 8388736.f;
}

__global__ void __launch_bounds__(kThreads) restore_kernel(const __grid_constant__ ActArgs a) {
  const int ti = find(a, blockIdx.x);
  const ActTensor& x = a.t[ti];
  const int64_t begin = static_cast<int64_t>(blockIdx.x - a.first_block[ti]) * a.pieces_cta;
  const int64_t end = min(x.pieces, begin + a.pieces_cta);
  if (a.zero && blockIdx.x == 0 && threadIdx.x < 2) a.zero[threadIdx.x] = 0;
  const bool sums = ti == a.sums;  // rows is dO, and the row sums of dO * value are wanted
  for (int64_t i0 = begin + threadIdx.x; i0 - threadIdx.x < end; i0 += kPiecesRound) {
    uint4 c[kUnroll];
    uint8_t e[kUnroll];
    Piece d[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = i0 + u * kThreads;
      if (i >= x.pieces) continue;
      c[u] = __ldcs(reinterpret_cast<const uint4*>(x.kept + i * 16));
      e[u] = x.kept[x.pieces * 16 + i / 2];
      if (sums) d[u] = load_piece(static_cast<const __nv_bfloat16*>(x.rows) + i * 16);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = i0 + u * kThreads;
      const bool in = i < x.pieces;
      float v[16];
      if (in) {
        const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
        const float s = scale_of(e[u]);
#pragma unroll
        for (int j = 0; j < 4; ++j) codes_up(w[j], v + 4 * j);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= s;
      }
      if (!sums) {
        if (!in) continue;
        uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(x.rows) + piece_at(x, static_cast<uint32_t>(i)));
#pragma unroll
        for (int h = 0; h < 2; ++h)
          out[h] = make_uint4(pack_bf16x2(v[8 * h], v[8 * h + 1]), pack_bf16x2(v[8 * h + 2], v[8 * h + 3]),
                              pack_bf16x2(v[8 * h + 4], v[8 * h + 5]), pack_bf16x2(v[8 * h + 6], v[8 * h + 7]));
        continue;
      }
      float sum = 0.f;
      if (in) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sum = fmaf(__uint_as_float(d[u].w[j] << 16), v[2 * j], sum);
          sum = fmaf(__uint_as_float(d[u].w[j] & 0xffff0000u), v[2 * j + 1], sum);
        }
      }
      // a head's lanes lie side by side, and its pieces begin at a multiple of their number
      for (int k = 1; k < a.head_pieces; k *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      const uint32_t place = static_cast<uint32_t>(i), th = place / a.head_pieces;
      if (in && place % a.head_pieces == 0) a.delta[static_cast<int64_t>(th % a.heads) * a.T + th / a.heads] = sum;
    }
  }
}

int launched(const char* what, std::string* err) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return PADOC_OK;
  *err = std::string(what) + " launch: " + cudaGetErrorString(e);
  return PADOC_ERR_CUDA;
}

// Deals the tensors out to CTAs; false when there are too many.
bool deal(ActArgs* a, int64_t* blocks) {
  int64_t b = 0;
  for (int i = 0; i < a->n; ++i) b += (a->t[i].pieces + kPiecesRound - 1) / kPiecesRound;
  a->pieces_cta = kPiecesRound * (b > kManyRounds ? kRounds : 1);
  b = 0;
  for (int i = 0; i < kActTensors; ++i) {
    a->first_block[i] = static_cast<int32_t>(b);
    if (i < a->n) b += (a->t[i].pieces + a->pieces_cta - 1) / a->pieces_cta;
    if (b > INT32_MAX) return false;
  }
  // tensors without CTAs (an empty one, or none) are stepped over: the next one's first
  // block is theirs too
  *blocks = b;
  return true;
}

}  // namespace

int launch_act(ActArgs a, bool keep, cudaStream_t s, std::string* err) {
  int64_t blocks = 0;
  if (!deal(&a, &blocks)) {
    *err = "too many values for one launch";
    return PADOC_ERR_UNSUPPORTED;
  }
  if (!blocks) return PADOC_OK;
  if (keep)
    keep_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
  else
    restore_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
  return launched(keep ? "keep_kernel" : "restore_kernel", err);
}

}  // namespace padoc

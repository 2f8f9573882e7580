// Rotation of packed rows by position, its gradient, and the tables of cosines and
// sines for contexts of any length.
//
//   rope_table_kernel  cosines and sines of p * f_i for positions p and pairs i
//   rope_apply_kernel  rows of q, k (or any heads) turned, or their gradients turned back
//
// A pair (a, b) becomes (a c - b s, b c + a s), in f32, each product and sum rounded on
// its own, as in kv_write_kernel: a row turned here and one turned on its way into the
// cache are the same bits.  The map is linear, so the gradient goes through its
// transpose (a c + b s, b c - a s); that is the rotation back times the amplitude's
// square where the table holds an amplitude other than 1.
//
// Both are streams.  A warp takes a row: eight lanes a head of 128 dims (four of 64),
// each with 16 dims that hold both partners of its eight pairs, so no lane needs
// another's values, and cosines and sines are read once for the heads that follow one
// another through the warp.
//
// Angles: a position and an angle a step are an integer and a fraction of a turn, so a
// position's fraction is their product modulo 2^64 with the step as a 64-bit binary
// fraction.  That is exact but for the step's own rounding (2^-53 of it), at any
// position, without a 64-bit floating operation; the remainder within half a turn goes
// to sincospif.
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
constexpr int kWarps = kThreads / 32;

// 16 dims of a row: 8 from each of two places.
template <class T>
struct Item;
template <>
struct Item<__nv_bfloat16> {
  uint4 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* pa, const __nv_bfloat16* pb) {
    a = __ldcs(reinterpret_cast<const uint4*>(pa));
    b = __ldcs(reinterpret_cast<const uint4*>(pb));
  }
  __device__ __forceinline__ void store(__nv_bfloat16* pa, __nv_bfloat16* pb) const {
    *reinterpret_cast<uint4*>(pa) = a;
    *reinterpret_cast<uint4*>(pb) = b;
  }
  static __device__ __forceinline__ void up(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 down(const float* x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
  __device__ __forceinline__ void get(float (&x)[16]) const {
    up(a, x);
    up(b, x + 8);
  }
  __device__ __forceinline__ void put(const float (&x)[16]) {
    a = down(x);
    b = down(x + 8);
  }
};
template <>
struct Item<float> {
  float4 v[4];
  __device__ __forceinline__ void load(const float* pa, const float* pb) {
    v[0] = __ldcs(reinterpret_cast<const float4*>(pa));
    v[1] = __ldcs(reinterpret_cast<const float4*>(pa) + 1);
    v[2] = __ldcs(reinterpret_cast<const float4*>(pb));
    v[3] = __ldcs(reinterpret_cast<const float4*>(pb) + 1);
  }
  __device__ __forceinline__ void store(float* pa, float* pb) const {
    reinterpret_cast<float4*>(pa)[0] = v[0];
    reinterpret_cast<float4*>(pa)[1] = v[1];
    reinterpret_cast<float4*>(pb)[0] = v[2];
    reinterpret_cast<float4*>(pb)[1] = v[3];
  }
  __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = v[i].x;
      x[4 * i + 1] = v[i].y;
      x[4 * i + 2] = v[i].z;
      x[4 * i + 3] = v[i].w;
    }
  }
  __device__ __forceinline__ void put(const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
};

// (a, b) in place; sn is negated by the caller for the gradient.
__device__ __forceinline__ void turn(float& a, float& b, float c, float sn) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, sn));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, sn));
  a = x;
}

template <class T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_apply_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int ITEMS = D / 16, SLOTS = 32 / ITEMS;  // lanes a head, heads a warp
  constexpr int U = sizeof(T) == 2 ? 4 : 2;          // heads of a lane on their way at once
  const int lane = threadIdx.x & 31, item = lane % ITEMS, slot = lane / ITEMS;
  const int half = a.rot_dim / 2, turning = a.rot_dim / 16;
  // places of the lane's dims in a head
  const bool turns = item < turning;
  int pa = 16 * item, pb = pa + 8;
  if (turns && !INTERLEAVED) {
    pa = 8 * item;
    pb = half + 8 * item;
  }
  const int64_t rows = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < a.n; t += rows) {
    float c[8], s[8];
    if (turns) {
      const int64_t p = a.positions ? a.positions[t] : t;
      if (p >= 0 && p < a.n_pos) {
        const float4* w = reinterpret_cast<const float4*>(a.cos_sin + p * a.rot_dim + 8 * item);
        const float4* z = reinterpret_cast<const float4*>(a.cos_sin + p * a.rot_dim + half + 8 * item);
        const float4 w0 = __ldg(w), w1 = __ldg(w + 1), z0 = __ldg(z), z1 = __ldg(z + 1);
        c[0] = w0.x, c[1] = w0.y, c[2] = w0.z, c[3] = w0.w, c[4] = w1.x, c[5] = w1.y, c[6] = w1.z, c[7] = w1.w;
        s[0] = z0.x, s[1] = z0.y, s[2] = z0.z, s[3] = z0.w, s[4] = z1.x, s[5] = z1.y, s[6] = z1.z, s[7] = z1.w;
        if (a.backward) {
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = -s[i];
        }
      } else {  // a position outside the table is no position: the row says so
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = s[i] = __uint_as_float(0x7fffffffu);
      }
    }
    for (int h0 = slot; h0 < a.heads; h0 += SLOTS * U) {
      Item<T> x[U];
      T* out[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * SLOTS;
        out[u] = nullptr;
        if (h >= a.heads) continue;
        int p = 0;
#pragma unroll
        for (int i = 1; i < kRopeParts; ++i) p += h >= a.first[i];
        const int64_t at = static_cast<int64_t>(h - a.first[p]) * D;
        const T* row = static_cast<const T*>(a.x[p]) + t * a.stride[p] + at;
        out[u] = static_cast<T*>(a.out[p]) + t * a.out_stride[p] + at;
        x[u].load(row + pa, row + pb);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!out[u]) continue;
        if (turns) {
          float v[16];
          x[u].get(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (INTERLEAVED)
              turn(v[2 * i], v[2 * i + 1], c[i], s[i]);
            else
              turn(v[i], v[8 + i], c[i], s[i]);
          }
          x[u].put(v);
        }
        x[u].store(out[u] + pa, out[u] + pb);
      }
    }
  }
}

// A thread: four neighbouring pairs of a position, and kTableRows positions one after
// another (the steps stay in registers).
constexpr int kTableRows = 4;
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ RopeTableArgs a) {
  const int per_row = a.rot_dim / 8;  // threads a position
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int q = static_cast<int>(id % per_row);
  int64_t t = id / per_row;
  const int64_t step = (static_cast<int64_t>(gridDim.x) * kThreads) / per_row;  // the grid is whole rows
  uint64_t f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = a.turns[4 * q + i];
  for (; t < a.n_pos; t += step) {
    const uint64_t p = static_cast<uint64_t>(a.first + t);
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t part = static_cast<int64_t>(p * f[i]);  // of a turn, in [-2^63, 2^63)
      sincospif(__ll2float_rn(part) * 1.0842021724855044e-19f /* 2^-63: half turns */, &s[i], &c[i]);
      c[i] *= a.amplitude;
      s[i] *= a.amplitude;
    }
    float* row = a.cos_sin + t * a.rot_dim + 4 * q;
    *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(row + a.rot_dim / 2) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

template <class T, int D>
void apply(const RopeArgs& a, int grid, cudaStream_t s) {
  if (a.interleaved)
    rope_apply_kernel<T, D, true><<<grid, kThreads, 0, s>>>(a);
  else
    rope_apply_kernel<T, D, false><<<grid, kThreads, 0, s>>>(a);
}

int launched(const char* what, std::string* err) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return PADOC_OK;
  *err = std::string(what) + " launch: " + cudaGetErrorString(e);
  return PADOC_ERR_CUDA;
}

}  // namespace

int launch_rope_apply(const RopeArgs& a, int32_t dtype, int32_t d, cudaStream_t s, std::string* err) {
  const int64_t want = (a.n + kWarps - 1) / kWarps;
  const int grid = static_cast<int>(std::min<int64_t>(want, static_cast<int64_t>(num_sms()) * 32));
  if (dtype == PADOC_BF16) {
    if (d == 128)
      apply<__nv_bfloat16, 128>(a, grid, s);
    else
      apply<__nv_bfloat16, 64>(a, grid, s);
  } else {
    if (d == 128)
      apply<float, 128>(a, grid, s);
    else
      apply<float, 64>(a, grid, s);
  }
  return launched("rope_apply_kernel", err);
}

int launch_rope_table(const RopeTableArgs& a, cudaStream_t s, std::string* err) {
  // whole positions a grid: per_row divides kThreads * 3 for every rot_dim
  const int64_t per_row = a.rot_dim / 8;
  int64_t grid = (a.n_pos * per_row + kThreads * kTableRows - 1) / (kThreads * kTableRows);
  grid = (grid + 2) / 3 * 3;
  rope_table_kernel<<<static_cast<int>(std::min<int64_t>(grid, 1 << 20) / 3 * 3), kThreads, 0, s>>>(a);
  return launched("rope_table_kernel", err);
}

}  // namespace padoc

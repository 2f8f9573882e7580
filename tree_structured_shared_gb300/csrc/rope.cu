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
// Both are streams.  A warp takes a row (or more, of few heads): a lane holds two chunks
// of 16 bytes of a head with both partners of its pairs, so no lane needs another's
// values, and cosines and sines are read once for the heads that follow one another
// through the warp.
//
// Angles: a position and an angle a step are an integer and a fraction of a turn, so a
// position's fraction is their product modulo 2^64 with the step as a 64-bit binary
// fraction.  That is exact but for the step's own rounding (2^-53 of it), at any
// position, without a 64-bit floating operation; its upper 32 bits are used, which cut it
// off at 2^-32 of a turn, 1.5e-9 (the step is cut off at 2^-64).
//
// Bound by HBM, and by launches below some 10 MB.  131072 rows of 24 heads of 128 in bf16:
// 246 us, 6.6 TB/s of reads and writes (240 at the copy rate).  50003 rows of 6 heads of 64
// in f32: 30 us (23.4): rows of 1.5 KB are short for a warp, and a GPU of CTAs takes 2.7
// rounds of them; with each lane's 16 dims side by side, which spreads a load over twice
// the lines, 37.  384 rows: 6 us, the host's call.  A table of 131072 positions of 128: 14.3 us
// for 67 MB (a fill of them takes 12.5); with sincospif on the remainder of a 64-bit
// product 20.6.
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

// Values of 16 bytes, and their arithmetic in f32.
template <class T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int V = 8;
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void put(const float* x) {
    u = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
};
template <>
struct Chunk<float> {
  static constexpr int V = 4;
  float4 u;
  __device__ __forceinline__ void load(const float* p) { u = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = u; }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = u.x;
    x[1] = u.y;
    x[2] = u.z;
    x[3] = u.w;
  }
  __device__ __forceinline__ void put(const float* x) { u = make_float4(x[0], x[1], x[2], x[3]); }
};

// (a, b) in place; sn is negated by the caller for the gradient.
__device__ __forceinline__ void turn(float& a, float& b, float c, float sn) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, sn));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, sn));
  a = x;
}

// N consecutive f32 of the table, 8-byte aligned at least.
template <int N>
__device__ __forceinline__ void table(const float* p, float* x) {
  if (N == 2) {
    const float2 v = __ldg(reinterpret_cast<const float2*>(p));
    x[0] = v.x;
    x[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
      x[4 * i] = v.x;
      x[4 * i + 1] = v.y;
      x[4 * i + 2] = v.z;
      x[4 * i + 3] = v.w;
    }
  }
}

template <class T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_apply_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int V = Chunk<T>::V, ITEMS = D / (2 * V);  // lanes a head
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // heads of a lane on their way at once
  const int lane = threadIdx.x & 31, item = lane % ITEMS;
  // A warp takes one row, or as many as it has heads for.
  const int slots = a.slots, sub = lane / ITEMS / slots, slot = lane / ITEMS % slots;
  const int half = a.rot_dim / 2;
  // The lane's two chunks of a head, neighbours' chunks beside them.  Partners half the
  // rotation apart: the same place of both halves; else any two.
  int ca = item, cb = item + ITEMS;
  bool ta = ca * V < a.rot_dim, tb = cb * V < a.rot_dim;
  if (!INTERLEAVED) {
    const int turning = half / V;
    if (item < turning) {
      cb = item + turning;
      ta = tb = true;
    } else {
      ca = 2 * turning + (item - turning);
      cb = ca + (ITEMS - turning);
      ta = tb = false;
    }
  }
  const int pa = ca * V, pb = cb * V;
  const int64_t rows = static_cast<int64_t>(gridDim.x) * kWarps * a.rows_warp;
  for (int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * a.rows_warp + sub; t < a.n; t += rows) {
    Chunk<T> x[U], y[U];
    T* out[U];
    auto load = [&](int h0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * slots;
        out[u] = nullptr;
        if (h >= a.heads) continue;
        int p = 0;
#pragma unroll
        for (int i = 1; i < kRopeParts; ++i) p += h >= a.first[i];
        const int64_t at = static_cast<int64_t>(h - a.first[p]) * D;
        const T* row = static_cast<const T*>(a.x[p]) + t * a.stride[p] + at;
        out[u] = static_cast<T*>(a.out[p]) + t * a.out_stride[p] + at;
        x[u].load(row + pa);
        y[u].load(row + pb);
      }
    };
    load(slot);  // on its way while the position and then the table are
    float c[V], s[V];  // half a rotation apart: of the pairs; else of a's pairs, then b's
    if (ta || tb) {
      const int64_t p = a.positions ? a.positions[t] : t;
      if (p >= 0 && p < a.n_pos) {
        const float* w = a.cos_sin + p * a.rot_dim;
        if (!INTERLEAVED) {
          table<V>(w + pa, c);
          table<V>(w + half + pa, s);
        } else {
          if (ta) {
            table<V / 2>(w + pa / 2, c);
            table<V / 2>(w + half + pa / 2, s);
          }
          if (tb) {
            table<V / 2>(w + pb / 2, c + V / 2);
            table<V / 2>(w + half + pb / 2, s + V / 2);
          }
        }
        if (a.backward) {
#pragma unroll
          for (int i = 0; i < V; ++i) s[i] = -s[i];
        }
      } else {  // a position outside the table is no position: the row says so
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = s[i] = __uint_as_float(0x7fffffffu);
      }
    }
    for (int h0 = slot; h0 < a.heads;) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!out[u]) continue;
        if (ta || tb) {
          float v[V], w[V];
          x[u].get(v);
          y[u].get(w);
          if (!INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < V; ++i) turn(v[i], w[i], c[i], s[i]);
          } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
              if (ta) turn(v[2 * i], v[2 * i + 1], c[i], s[i]);
              if (tb) turn(w[2 * i], w[2 * i + 1], c[V / 2 + i], s[V / 2 + i]);
            }
          }
          x[u].put(v);
          y[u].put(w);
        }
        x[u].store(out[u] + pa);
        y[u].store(out[u] + pb);
      }
      h0 += slots * U;
      if (h0 < a.heads) load(h0);
    }
  }
}

// Cosines and sines of two angles given as fractions of 2^32 of a turn: the nearest
// quarter turn, and the Taylor polynomials of what is left, x <= pi / 4.  The first terms
// left out are x^11 / 11! < 2^-29 of the sine and x^12 / 12! < 2^-32 of the cosine.  In f32 x
// is off by three half steps (the integer, 2 pi 2^-32, their product), 3 2^-24 x, which moves
// either by 3 2^-24 x sin x or x cos x < 1.7 2^-24; x^2 and the sum before the last by 0.7 2^-24,
// the last sum by 0.5 and the amplitude's product by 0.8 (results of pi / 4): 4 2^-24 in all.
__device__ __forceinline__ void turns_of(uint32_t p0, uint32_t p1, float amplitude, float* c, float* s) {
  const uint32_t q0 = (p0 + (1u << 29)) >> 30, q1 = (p1 + (1u << 29)) >> 30;
  const auto both = [](float v) { return f2pack(v, v); };
  const uint64_t x = mul2(f2pack(__int2float_rn(static_cast<int32_t>(p0 - (q0 << 30))),
                                 __int2float_rn(static_cast<int32_t>(p1 - (q1 << 30)))),
                          both(1.4629180792671596e-9f) /* 2 pi 2^-32 */);
  const uint64_t z = mul2(x, x);
  uint64_t si = fma2(z, both(2.7557319e-6f), both(-1.9841270e-4f));
  si = fma2(z, si, both(8.3333333e-3f));
  si = fma2(z, si, both(-1.6666667e-1f));
  si = fma2(mul2(x, z), si, x);
  uint64_t co = fma2(z, both(-2.7557319e-7f), both(2.4801587e-5f));
  co = fma2(z, co, both(-1.3888889e-3f));
  co = fma2(z, co, both(4.1666667e-2f));
  co = fma2(z, co, both(-0.5f));
  co = fma2(z, co, both(1.f));
  float s0, s1, c0, c1;
  f2unpack(mul2(si, both(amplitude)), s0, s1);
  f2unpack(mul2(co, both(amplitude)), c0, c1);
  // quarter turns: (c, s), (-s, c), (-c, -s), (s, -c)
  const auto sign = [](float v, uint32_t bit) { return __uint_as_float(__float_as_uint(v) ^ (bit << 31)); };
  c[0] = sign(q0 & 1 ? s0 : c0, (q0 + 1) >> 1 & 1);
  s[0] = sign(q0 & 1 ? c0 : s0, q0 >> 1 & 1);
  c[1] = sign(q1 & 1 ? s1 : c1, (q1 + 1) >> 1 & 1);
  s[1] = sign(q1 & 1 ? c1 : s1, q1 >> 1 & 1);
}

// A thread: four neighbouring pairs, and every so many positions of its CTA's run (the
// steps stay in registers).
constexpr int kTableRun = 128;  // positions of a CTA
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ RopeTableArgs a) {
  const int per_row = a.rot_dim / 8, rows = kThreads / per_row;  // threads a position, positions at once
  const int q = threadIdx.x % per_row, r = threadIdx.x / per_row;
  if (r >= rows) return;
  uint64_t f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = a.turns[4 * q + i];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTableRun;
  const int n = static_cast<int>(min(static_cast<int64_t>(kTableRun), a.n_pos - t0));
  const uint32_t first = static_cast<uint32_t>(a.first + t0);
  float* out = a.cos_sin + t0 * a.rot_dim + 4 * q;
#pragma unroll 4
  for (int t = r; t < n; t += rows) {
    const uint64_t p = first + static_cast<uint32_t>(t);
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2)
      turns_of(static_cast<uint32_t>((p * f[i]) >> 32), static_cast<uint32_t>((p * f[i + 1]) >> 32), a.amplitude, c + i, s + i);
    float* row = out + t * a.rot_dim;
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

int launch_rope_apply(RopeArgs a, int32_t dtype, int32_t d, cudaStream_t s, std::string* err) {
  const int slots = 32 / (d / (dtype == PADOC_BF16 ? 16 : 8));
  a.slots = 1;
  while (a.slots < slots && a.slots < a.heads) a.slots *= 2;
  a.rows_warp = slots / a.slots;
  // A CTA costs its launch: short rows are taken several a warp, as many as come to the
  // 6 KB of 24 heads of 128 (50003 rows of 1.5 KB: 28 us, with a row a warp 37), unless
  // that leaves SMs without work.
  const int64_t row_bytes = static_cast<int64_t>(a.heads) * d * (dtype == PADOC_BF16 ? 2 : 4);
  const int64_t cta = static_cast<int64_t>(kWarps) * a.rows_warp, want = (a.n + cta - 1) / cta;
  const int64_t each = std::max<int64_t>(1, 6144 / (row_bytes * a.rows_warp));
  const int grid = static_cast<int>(std::min<int64_t>(std::max<int64_t>((want + each - 1) / each, std::min<int64_t>(want, 4 * num_sms())), 1 << 20));
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
  rope_table_kernel<<<static_cast<unsigned>((a.n_pos + kTableRun - 1) / kTableRun), kThreads, 0, s>>>(a);
  return launched("rope_table_kernel", err);
}

}  // namespace padoc

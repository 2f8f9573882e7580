// Branch decode / verify over a 4-bit pool, warp-level matrix instructions.
//
// A unit is one kv head, up to 8 NT query rows (tokens times the query heads of
// the group, row R = token R / G, head R % G) and a run of cached keys: a chunk
// of a page's shared prefix with the rows of all its branches (each prefix
// token is read from HBM once a page), or a branch's own suffix with its own
// rows and query block.  Four warps share a unit: each takes every fourth
// 16-token block with a running softmax of its own, and the partial results
// meet in shared memory.
//
// Keys go on the matrix instruction's M side, so one query token (G <= 8 rows)
// fills its N side and a key costs one instruction of each product a row tile:
//     S^T[key][row]  = K  Q^T   m16n8k16, M = 16 keys, K = 16 dims
//     O^T[dim][row] += V^T P^T  m16n8k16, M = 16 dims, K = 16 keys
// Codes become fp16 operands in registers (n s is exact in fp16), never a
// wider copy in memory.  Which dims and keys a lane holds is free as long as
// both operands agree, so lane (i, c) = (lane / 4, lane % 4) reads chunk c of
// its two keys and group i of its four keys, 16 bytes at a time.
//
// Q is scaled by a power of two, one for the unit's rows, so that its largest
// magnitude lies in [2^14, 2^15): values down to 2^-28 of that keep every bit
// of their bf16 form, and the scale joins the softmax's.  P is formed as
// 2^(x - m + 10) with m a running maximum that moves only when exceeded by
// 2^4: at most 2^14, and what falls below fp16's smallest step is less than
// 2^-35 of the row's largest weight.  Sums, maxima and O are f32.
//
// The query block (bf16 rows that are not in the cache yet) has its scores from
// bf16 matrix instructions and its values added in f32 by key, only for rows
// that see the key, so a NaN in a hidden draft token stays there.
#include <cuda_bf16.h>

#include <string>

#include "../../include/padoc.h"
#include "kv_i4.cuh"
#include "padoc_internal.h"
#include "ptx_sm103.cuh"

namespace padoc {
namespace {

using namespace ptx;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kPShift = 10.f;  // log2 of P's weight at the running maximum
constexpr float kPSlack = 4.f;   // how far (log2) a score may exceed it
constexpr float kNoMax = -3.0e38f;  // reference of a row that has seen no key: any score exceeds it

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 tile of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// One 16-token block of a kv head as a lane holds it.
struct BlockRegs {
  uint4 ka, kb;      // chunk c of the keys 4 (i / 2) + i % 2 and + 2
  uint32_t sa, sb;   // their scales of groups 2c, 2c + 1
  uint4 v0, v1;      // group i of the keys 4c, 4c + 1 and 4c + 2, 4c + 3
  uint32_t sv;       // the four keys' scales of group i
};

__device__ __forceinline__ BlockRegs load_block(const uint8_t* kp, const uint8_t* vp, int key_a, int i, int c) {
  BlockRegs b;
  b.ka = ld_stream(kp + c * 256 + key_a * 16);
  b.kb = ld_stream(kp + c * 256 + key_a * 16 + 32);
  b.sa = *reinterpret_cast<const uint16_t*>(kp + kI4Scales + key_a * 8 + 2 * c);
  b.sb = *reinterpret_cast<const uint16_t*>(kp + kI4Scales + key_a * 8 + 16 + 2 * c);
  b.v0 = ld_stream(vp + i * 128 + c * 32);
  b.v1 = ld_stream(vp + i * 128 + c * 32 + 16);
  b.sv = *reinterpret_cast<const uint32_t*>(vp + kI4Scales + i * 16 + c * 4);
  return b;
}

template <int NT>
struct Smem {
  float o[kWarps][8 * NT][kHeadDim];
  float m[kWarps][8 * NT], l[kWarps][8 * NT];
};

template <int NT>
__global__ void __launch_bounds__(kThreads) decode_i4_kernel(const I4Args a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<NT>& sm = *reinterpret_cast<Smem<NT>*>(smem_raw);
  const int u = a.unit0 + blockIdx.x / a.Hkv, g = blockIdx.x % a.Hkv;
  const I4Unit un = a.units[u];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = lane >> 2, c = lane & 3;
  const int G = a.group;
  const int key_a = 4 * (i >> 1) + (i & 1);
  const int32_t* ids = a.table + static_cast<int64_t>(un.seq) * a.max_bps + un.blk0;
  const int n_keys = un.n_keys, n_steps = (n_keys + 15) >> 4;

  // the first block's bytes are on their way while Q is laid out
  auto block_ptr = [&](const void* pool, int step) {
    return static_cast<const uint8_t*>(pool) + (static_cast<int64_t>(ids[step]) * a.Hkv + g) * kI4Unit;
  };
  BlockRegs nx{};
  if (warp < n_steps) nx = load_block(block_ptr(a.k_pool, warp), block_ptr(a.v_pool, warp), key_a, i, c);

  // Q^T fragments: row nt * 8 + i, dims 32 c .. 32 c + 31
  auto q_row = [&](int nt) -> const __nv_bfloat16* {
    const int R = un.row0 + nt * 8 + i;
    return nt * 8 + i < un.rows
               ? a.q + (static_cast<int64_t>(un.q_first + R / G) * a.Hq + g * G + R % G) * kHeadDim + 32 * c
               : nullptr;
  };
  uint32_t q[NT][16];
  float amax = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const __nv_bfloat16* p = q_row(nt);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint4 v = p ? reinterpret_cast<const uint4*>(p)[x] : make_uint4(0, 0, 0, 0);
      q[nt][4 * x] = v.x;
      q[nt][4 * x + 1] = v.y;
      q[nt][4 * x + 2] = v.z;
      q[nt][4 * x + 3] = v.w;
    }
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const float lo = fabsf(__uint_as_float(q[nt][x] << 16)), hi = fabsf(__uint_as_float(q[nt][x] & 0xffff0000u));
      amax = fmaxf(amax, lo <= 3.4028235e38f ? lo : 0.f);
      amax = fmaxf(amax, hi <= 3.4028235e38f ? hi : 0.f);
    }
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
  const int kexp = amax > 0.f ? min(100, 14 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127)) : 0;
  const float qf = __uint_as_float(static_cast<uint32_t>(127 + kexp) << 23);
  const float sl2q = a.sl2 * __uint_as_float(static_cast<uint32_t>(127 - kexp) << 23);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 16; ++x)
      q[nt][x] = pack_f16x2(__uint_as_float(q[nt][x] << 16) * qf, __uint_as_float(q[nt][x] & 0xffff0000u) * qf);

  // rows 2c, 2c + 1 of each tile: keys they may see, running reference (log2, less kPShift), sums
  int lim[NT][2];
  float mo[NT][2], l[NT][2];
  float o[NT][8][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = nt * 8 + 2 * c + e;
      lim[nt][e] = n_keys;
      if (un.branch < 0 && r < un.rows)
        lim[nt][e] = min(n_keys, a.q_plen[un.q_first + (un.row0 + r) / G] - un.key0);
      mo[nt][e] = kNoMax;
      l[nt][e] = 0.f;
    }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][x][e] = 0.f;
  int lim_min = n_keys;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) lim_min = min(lim_min, min(lim[nt][0], lim[nt][1]));
  lim_min = __reduce_min_sync(0xffffffffu, lim_min);

  // P of one tile of scores (log2 units) against the running references, which
  // move first where a score exceeds them by more than kPSlack
  auto softmax = [&](float (&s)[NT][4]) {
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) grow |= s[nt][e] - mo[nt][e & 1] > kPShift + kPSlack;
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float al[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(s[nt][e], s[nt][2 + e]);
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, k));
          al[e] = 1.f;
          if (t - mo[nt][e] > kPShift + kPSlack) {
            al[e] = fast_exp2(mo[nt][e] - (t - kPShift));
            mo[nt][e] = t - kPShift;
          }
          l[nt][e] *= al[e];
        }
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][x][e] *= al[e & 1];
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[nt][e] = fast_exp2(s[nt][e] - mo[nt][e & 1]);
        l[nt][e & 1] += s[nt][e];
      }
  };

  for (int step = warp; step < n_steps; step += kWarps) {
    const BlockRegs b = nx;
    if (step + kWarps < n_steps)
      nx = load_block(block_ptr(a.k_pool, step + kWarps), block_ptr(a.v_pool, step + kWarps), key_a, i, c);
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
    {
      const uint32_t wa[4] = {b.ka.x, b.ka.y, b.ka.z, b.ka.w}, wb[4] = {b.kb.x, b.kb.y, b.kb.z, b.kb.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        // words 0, 1 of the chunk are its first group, 2, 3 its second
        const uint32_t ba = w < 2 ? b.sa & 0xffu : b.sa >> 8, bb = w < 2 ? b.sb & 0xffu : b.sb >> 8;
        const uint32_t sa = i4_scale_pair(ba, ba), sb = i4_scale_pair(bb, bb);
        const uint32_t fa = i4_offset(sa), fb = i4_offset(sb);
        const uint32_t f0[4] = {i4_pair<0>(wa[w], sa, fa), i4_pair<0>(wb[w], sb, fb), i4_pair<1>(wa[w], sa, fa),
                                i4_pair<1>(wb[w], sb, fb)};
        const uint32_t f1[4] = {i4_pair<2>(wa[w], sa, fa), i4_pair<2>(wb[w], sb, fb), i4_pair<3>(wa[w], sa, fa),
                                i4_pair<3>(wb[w], sb, fb)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(s[nt], f0, q[nt][4 * w], q[nt][4 * w + 1]);
          mma_f16(s[nt], f1, q[nt][4 * w + 2], q[nt][4 * w + 3]);
        }
      }
    }
    const int key0 = step * 16 + key_a;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] *= sl2q;
    if (step * 16 + 16 > lim_min) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key0 + (e >> 1) * 2 >= lim[nt][e & 1]) s[nt][e] = -INFINITY;
    }
    softmax(s);
    uint32_t p[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      p[nt][0] = transpose8(pack_f16x2(s[nt][0], s[nt][1]));
      p[nt][1] = transpose8(pack_f16x2(s[nt][2], s[nt][3]));
    }
    const uint32_t s01 = i4_scale_pair(b.sv & 0xffu, (b.sv >> 8) & 0xffu);
    const uint32_t s23 = i4_scale_pair((b.sv >> 16) & 0xffu, b.sv >> 24);
    const uint32_t f01 = i4_offset(s01), f23 = i4_offset(s23);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      // low halves: even dims of two keys side by side; high halves: odd dims
      const uint32_t k0 = w ? b.v0.y : b.v0.x, k1 = w ? b.v0.w : b.v0.z;
      const uint32_t k2 = w ? b.v1.y : b.v1.x, k3 = w ? b.v1.w : b.v1.z;
      const uint32_t e01 = __byte_perm(k0, k1, 0x5410), d01 = __byte_perm(k0, k1, 0x7632);
      const uint32_t e23 = __byte_perm(k2, k3, 0x5410), d23 = __byte_perm(k2, k3, 0x7632);
      auto pv = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
        const uint32_t f[4] = {a0, a1, a2, a3};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][mt], f, p[nt][0], p[nt][1]);
      };
      pv(4 * w + 0, i4_pair<0>(e01, s01, f01), i4_pair<0>(d01, s01, f01), i4_pair<0>(e23, s23, f23), i4_pair<0>(d23, s23, f23));
      pv(4 * w + 1, i4_pair<1>(e01, s01, f01), i4_pair<1>(d01, s01, f01), i4_pair<1>(e23, s23, f23), i4_pair<1>(d23, s23, f23));
      pv(4 * w + 2, i4_pair<2>(e01, s01, f01), i4_pair<2>(d01, s01, f01), i4_pair<2>(e23, s23, f23), i4_pair<2>(d23, s23, f23));
      pv(4 * w + 3, i4_pair<3>(e01, s01, f01), i4_pair<3>(d01, s01, f01), i4_pair<3>(e23, s23, f23), i4_pair<3>(d23, s23, f23));
    }
  }

  // ---------------------------------------------------------------- query block
  // scores of all 16 keys by every warp; warp w then takes the keys j % 4 == w
  if (un.branch >= 0 && un.q_len > 0) {
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
    const int64_t krow = static_cast<int64_t>(a.Hkv) * kHeadDim;
    const __nv_bfloat16* kn = a.k_new + un.qb_first * krow + g * kHeadDim + 32 * c;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint4 z = make_uint4(0, 0, 0, 0);
      const uint4 va = key_a < un.q_len ? *reinterpret_cast<const uint4*>(kn + key_a * krow + 8 * x) : z;
      const uint4 vb = key_a + 2 < un.q_len ? *reinterpret_cast<const uint4*>(kn + (key_a + 2) * krow + 8 * x) : z;
      const uint32_t f0[4] = {va.x, vb.x, va.y, vb.y}, f1[4] = {va.z, vb.z, va.w, vb.w};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const __nv_bfloat16* p = q_row(nt);
        const uint4 qv = p ? reinterpret_cast<const uint4*>(p)[x] : z;
        mma_bf16(s[nt], f0, qv.x, qv.y);
        mma_bf16(s[nt], f1, qv.z, qv.w);
      }
    }
    uint32_t vis[NT][2];  // bit j: the row sees key j, one of this warp's
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * c + e;
        uint32_t bits = 0;
        if (r < un.rows) {
          const int qi = (un.row0 + r) / G;
          bits = a.tree_bits ? static_cast<uint32_t>(a.tree_bits[un.qb_first + qi]) : (2u << qi) - 1u;
        }
        vis[nt][e] = bits & ((1u << un.q_len) - 1u) & (0x1111u << warp);
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[nt][e] = ((vis[nt][e & 1] >> (key_a + (e >> 1) * 2)) & 1u) ? s[nt][e] * a.sl2 : -INFINITY;
    softmax(s);
    const __nv_bfloat16* vn = a.v_new + un.qb_first * krow + g * kHeadDim + 16 * i;
    for (int j = warp; j < un.q_len; j += 4) {
      // key j's P sits in lane row 2 (j / 4) + j % 2, first or second register pair
      const int from = ((2 * (j >> 2) + (warp & 1)) << 2) | c;
      const uint4 x0 = *reinterpret_cast<const uint4*>(vn + j * krow), x1 = *reinterpret_cast<const uint4*>(vn + j * krow + 8);
      const uint32_t xv[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float pj = __shfl_sync(0xffffffffu, warp < 2 ? s[nt][e] : s[nt][2 + e], from);
          if ((vis[nt][e] >> j) & 1u) {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              o[nt][x][e] = fmaf(pj, __uint_as_float(xv[x] << 16), o[nt][x][e]);
              o[nt][x][2 + e] = fmaf(pj, __uint_as_float(xv[x] & 0xffff0000u), o[nt][x][2 + e]);
            }
          }
        }
    }
  }

  // ---------------------------------------------------------------- the four warps' results
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], k);
      const int r = nt * 8 + 2 * c + e;
      if (i == 0) {
        sm.m[warp][r] = mo[nt][e];
        sm.l[warp][r] = l[nt][e];
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        *reinterpret_cast<float4*>(&sm.o[warp][r][16 * i + 4 * x]) =
            make_float4(o[nt][2 * x][e], o[nt][2 * x][2 + e], o[nt][2 * x + 1][e], o[nt][2 * x + 1][2 + e]);
    }
  __syncthreads();
  // thread t is head dim t
  const int t = threadIdx.x;
  for (int r = 0; r < un.rows; ++r) {
    const int R = un.row0 + r;
    const int64_t qh = static_cast<int64_t>(R / G) * a.Hq + g * G + R % G;  // (token, head) from q_first
    float M = kNoMax, L = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (!(sm.l[w][r] == 0.f)) M = fmaxf(M, sm.m[w][r]);
    const int n_pre = un.n_pre;
    for (int k = 0; k < n_pre; ++k) M = fmaxf(M, a.part_lse[un.pre + k * un.pre_stride + qh]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (!(sm.l[w][r] == 0.f)) {
        const float e = fast_exp2(sm.m[w][r] - M);
        L = fmaf(sm.l[w][r], e, L);
        acc = fmaf(sm.o[w][r][t], e, acc);
      }
    for (int k = 0; k < n_pre; ++k) {
      const int64_t row = un.pre + k * un.pre_stride + qh;
      const float e = fast_exp2(a.part_lse[row] - M);
      if (e > 0.f || !(e == e)) {
        L += e;
        acc = fmaf(a.part_o[row * kHeadDim + t], e, acc);
      }
    }
    const bool any = !(L == 0.f);
    const float out = any ? acc / L : 0.f;
    if (un.part >= 0) {
      a.part_o[(un.part + qh) * kHeadDim + t] = out;
      if (t == 0) a.part_lse[un.part + qh] = any ? M + __log2f(L) : -INFINITY;
    } else {
      const int64_t row = static_cast<int64_t>(un.q_first) * a.Hq + qh;
      a.o[row * kHeadDim + t] = __float2bfloat16_rn(out);
      if (t == 0) a.lse[row] = any ? (M + __log2f(L)) * kLn2 : -INFINITY;
    }
  }
}

// Rows of branches whose partial results are many: one CTA a (token, head),
// thread t is head dim t.
__global__ void __launch_bounds__(kHeadDim) merge_i4_kernel(const I4Args a) {
  const I4Merge mg = a.merges[blockIdx.x / a.Hq];
  const int h = blockIdx.x % a.Hq, t = threadIdx.x;
  __shared__ float red[2][4];
  const int n = mg.n_pre + mg.n_own;
  auto row_of = [&](int k) -> int64_t {
    return k < mg.n_pre ? mg.pre + static_cast<int64_t>(k) * mg.pre_stride + h
                        : mg.own + static_cast<int64_t>(k - mg.n_pre) * mg.own_stride + h;
  };
  float M = kNoMax;
  for (int k = t; k < n; k += kHeadDim) M = fmaxf(M, a.part_lse[row_of(k)]);
#pragma unroll
  for (int s = 16; s; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
  if ((t & 31) == 0) red[0][t >> 5] = M;
  __syncthreads();
  M = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  float L = 0.f, acc = 0.f;
#pragma unroll 8
  for (int k = 0; k < n; ++k) {
    const int64_t row = row_of(k);
    const float e = fast_exp2(a.part_lse[row] - M);
    L += e;
    const float v = a.part_o[row * kHeadDim + t];
    acc = e == 0.f ? acc : fmaf(v, e, acc);
  }
  const bool any = !(L == 0.f);
  const int64_t out = static_cast<int64_t>(mg.token) * a.Hq + h;
  a.o[out * kHeadDim + t] = __float2bfloat16_rn(any ? acc / L : 0.f);
  if (t == 0) a.lse[out] = any ? (M + __log2f(L)) * kLn2 : -INFINITY;
}

int launch_error(const char* what, std::string* err) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return PADOC_OK;
  *err = std::string(what) + ": " + cudaGetErrorString(e);
  return PADOC_ERR_CUDA;
}

template <int NT>
int launch_units(I4Args a, int32_t unit0, int32_t n, cudaStream_t s, std::string* err) {
  if (n == 0) return PADOC_OK;
  const int bytes = sizeof(Smem<NT>);
  if (bytes > 48 * 1024) {
    // per device, so set at each launch (a host call of well under a microsecond)
    const cudaError_t e = cudaFuncSetAttribute(decode_i4_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) {
      *err = std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e);
      return PADOC_ERR_CUDA;
    }
  }
  a.unit0 = unit0;
  decode_i4_kernel<NT><<<static_cast<unsigned>(n) * a.Hkv, kThreads, bytes, s>>>(a);
  return launch_error("i4 decode launch", err);
}

}  // namespace

int launch_i4_units(const I4Args& a, const int32_t (&first)[4], cudaStream_t s, std::string* err) {
  int rc = launch_units<1>(a, first[0], first[1] - first[0], s, err);
  if (!rc) rc = launch_units<2>(a, first[1], first[2] - first[1], s, err);
  if (!rc) rc = launch_units<4>(a, first[2], first[3] - first[2], s, err);
  return rc;
}

int launch_i4_merge(const I4Args& a, int32_t n_merges, cudaStream_t s, std::string* err) {
  if (n_merges == 0) return PADOC_OK;
  merge_i4_kernel<<<static_cast<unsigned>(n_merges) * a.Hq, kHeadDim, 0, s>>>(a);
  return launch_error("i4 merge launch", err);
}

}  // namespace padoc

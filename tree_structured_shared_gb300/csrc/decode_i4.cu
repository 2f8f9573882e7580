// Branch decode / verify over a 4-bit pool, warp-level matrix instructions.
//
// A unit is one kv head, up to 8 query rows (tokens times the query heads of the
// group, row R = token R / G, head R % G) and a run of cached keys: a chunk of a
// page's shared prefix with rows of its branches, or a branch's own suffix with
// its own rows and, once, the query block.  W warps share a unit and are a CTA:
// each takes every W-th 16-token block with a running softmax of its own, and
// the others' results reach the first as register images in shared memory.  One
// warp a unit costs least where there are units enough to fill the GPU.
//
// Keys go on the matrix instruction's M side, so one query token (G <= 8 rows)
// fills its N side and a key costs one instruction of the two products together:
//     S^T[key][row]  = K  Q^T   m16n8k16, M = 16 keys, K = 16 dims
//     O^T[dim][row] += V^T P^T  m16n8k16, M = 16 dims, K = 16 keys
// More rows are more units: tiles of 16 and 32 rows a warp decode a key for more
// rows at once, but their 64 and 128 accumulators leave too few warps an SM
// (verify's own pass on 64 pages: 341, 369 and 401 us with tiles of 8, 16, 32).
//
// Codes become fp16 operands in registers (n s is exact in fp16), never a
// wider copy in memory.  Which dims and keys a lane holds is free as long as
// both operands agree, so lane (i, c) = (lane / 4, lane % 4) reads chunk c of
// its two keys and group i of its four keys, 16 bytes at a time.
//
// Each row of Q is scaled by a power of two of its own, so that its largest
// magnitude lies in [2^14, 2^15): values down to 2^-28 of that keep every bit
// of their bf16 form, and the scale joins the softmax's.  P is formed as
// 2^(x - m + 10) with m a running maximum that moves only when exceeded by
// 2^4: at most 2^14, and what falls below fp16's smallest step is less than
// 2^-35 of the row's largest weight.  Sums, maxima and O are f32.
//
// What bounds it: a key costs a warp about 25 instructions for a head's 8 rows, and
// four warps a scheduler (128 registers) issue one every other cycle.  Suffixes of 4500
// branches (0-1024 tokens, 8 kv heads): 562 us, of which the copies alone take 449 (404
// at HBM rate) and the arithmetic alone 490; 1500 branches with up to 16 query tokens:
// 300 us (237 at HBM rate).  Neither more independent products (two blocks' score
// chains interleaved, accumulators split) nor shorter loops nor the query block and
// the partial results fetched ahead change that by more than 1 %.
//
// The query block (bf16 rows that are not in the cache yet) has its scores and, with P
// as the sum of two bf16 numbers, its values from bf16 matrix instructions.  Where a
// value of the block is not finite (or there are few keys), the values are added in f32
// by key, only for rows that see the key, so a NaN in a hidden draft token stays there.  (Doing so always cost
// 130 instructions a key: 335 us instead of 300 on the second case above.)
#include <cuda_bf16.h>

#include <algorithm>
#include <string>

#include "../../include/padoc.h"
#include "kv_i4.cuh"
#include "padoc_internal.h"
#include "ptx_sm103.cuh"

namespace padoc {
namespace {

using namespace ptx;

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kPShift = 10.f;  // log2 of P's weight at the running maximum
constexpr float kPSlack = 4.f;   // how far (log2) a score may exceed it
// Query blocks up to this long have their values added key by key (one token a branch,
// 128 pages: 566 us, 568 to 572 by matrix instructions; up to 3 and 4 tokens: 136 and
// 140 us key by key, 133 and 134 by matrix instructions).
constexpr int kFewKeys = 2;
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
// One 16-token block of a kv head as a lane holds it.
struct KRegs {
  uint4 ka, kb;      // chunk c of the keys 4 (i / 2) + i % 2 and + 2
  uint32_t sa, sb;   // their scales of groups 2c, 2c + 1
};
struct VRegs {
  uint4 v0, v1;      // group i of the keys 4c, 4c + 1 and 4c + 2, 4c + 3
  uint32_t sv;       // the four keys' scales of group i
};

// A block in a warp's ring in shared memory: K codes with 32 bytes between the
// 256-byte chunks, K scales, V codes with the halves of the odd groups' 32-byte
// pieces swapped, V scales.  Eight neighbouring lanes of a 16-byte read then
// touch every bank once.
constexpr int kRing = 4;  // blocks of a warp's ring: a pair is worked on, a pair is on its way
constexpr int kRingKS = 4 * 288, kRingV = kRingKS + 128, kRingVS = kRingV + 1024, kRingBlock = kRingVS + 128;

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// A lane's share of a block's 144 16-byte pieces (72 of K, then 72 of V): pieces
// lane, 32 + lane of K; a third that is K's for lanes 0-7, V's for the rest; and
// two of V.  What depends on the lane alone is kept: three source addresses of the
// unit's kv head, four offsets within a stage.
struct CopyLane {
  const uint8_t *k, *m, *v;
  uint32_t dk, dm, dv, dw;
};
__device__ __forceinline__ CopyLane copy_lane(int lane) {
  auto v_at = [](int p) { return static_cast<uint32_t>(kRingV + (p < 64 ? (p * 16) ^ (((p >> 3) & 1) << 4) : p * 16)); };
  CopyLane l;
  l.dk = lane * 16 + (lane >> 4) * 32;
  l.dm = lane < 8 ? kRingKS + lane * 16 : v_at(lane - 8);
  l.dv = v_at(lane + 24);
  l.dw = v_at(lane + 56);
  return l;
}
__device__ __forceinline__ void copy_unit(CopyLane& l, const void* k_pool, const void* v_pool, int g, int lane) {
  const uint8_t* k = static_cast<const uint8_t*>(k_pool) + g * kI4Unit;
  const uint8_t* v = static_cast<const uint8_t*>(v_pool) + g * kI4Unit;
  l.k = k + lane * 16;
  l.m = lane < 8 ? k + (64 + lane) * 16 : v + (lane - 8) * 16;
  l.v = v + (24 + lane) * 16;
}
// Starts the copy of a block (at = its number * the pool's block stride).
__device__ __forceinline__ void copy_block(const CopyLane& l, uint32_t dst, int64_t at, int lane) {
  copy16(dst + l.dk, l.k + at);
  copy16(dst + l.dk + 576, l.k + at + 512);
  copy16(dst + l.dm, l.m + at);
  copy16(dst + l.dv, l.v + at);
  if (lane < 16) copy16(dst + l.dw, l.v + at + 512);
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ KRegs read_k(uint32_t src, int key_a, int c) {
  KRegs b;
  b.ka = lds128(src + c * 288 + key_a * 16);
  b.kb = lds128(src + c * 288 + key_a * 16 + 32);
  b.sa = lds16(src + kRingKS + key_a * 8 + 2 * c);
  b.sb = lds16(src + kRingKS + key_a * 8 + 16 + 2 * c);
  return b;
}
__device__ __forceinline__ VRegs read_v(uint32_t src, int i, int c) {
  VRegs b;
  const uint32_t v = src + kRingV + i * 128 + c * 32 + ((i & 1) << 4);
  b.v0 = lds128(v);
  b.v1 = lds128(v ^ 16);
  b.sv = lds32(src + kRingVS + i * 16 + c * 4);
  return b;
}

template <int W>
struct Smem {
  uint4 ring[W][kRing * kRingBlock / 16];
  // what warps 1 .. W - 1 leave for warp 0: the lane's 32 sums of O and, of its
  // two rows, the reference and the sum
  float4 o[W > 1 ? W - 1 : 1][W > 1 ? 8 : 1][32];
  float4 ml[W > 1 ? W - 1 : 1][32];
};

// A persistent CTA's k-th unit: units come longest first and are dealt back and
// forth, so that every CTA gets about the same number of keys.
__device__ __forceinline__ int nth_work(int k) {
  return k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

template <int W>
__global__ void __launch_bounds__(32 * W, 16 / W) decode_i4_kernel(const I4Args a, const int n_work) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<W>& sm = *reinterpret_cast<Smem<W>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = lane >> 2, c = lane & 3;
  const int G = a.group;
  const int key_a = 4 * (i >> 1) + (i & 1);

  // The copies' own walk over the warp's blocks, a pair ahead of the work: unit
  // number, its step, its ids (lane l: step l of the current 32), and the next
  // unit's record and first ids, read while this one's blocks are copied.
  const uint32_t ring = smem_u32(&sm.ring[warp][0]);
  int ck = 0, cstep = 0, csteps = 0, cid = 0;
  CopyLane cl = copy_lane(lane);
  const int64_t block_stride = static_cast<int64_t>(a.Hkv) * kI4Unit;
  const int32_t* cids = nullptr;
  int nsteps = 0, nid = 0;
  const int32_t* nids = nullptr;
  auto read_next = [&](int k) {  // the record and the ids of the warp's k-th unit
    const int w = nth_work(k);
    nsteps = 0;
    if (w >= n_work) return;
    const I4Unit& un = a.units[a.unit0 + w / a.Hkv];
    nids = a.table + static_cast<int64_t>(un.seq) * a.max_bps + un.blk0 + warp;
    const int n = (un.n_keys + 15) >> 4;
    nsteps = n > warp ? (n - warp + W - 1) / W : 0;
    nid = lane < nsteps ? nids[W * lane] : 0;
  };
  auto open_next = [&]() {  // to the next unit that has a block for this warp
    do {
      cids = nids;
      cid = nid;
      csteps = nsteps;
      cstep = 0;
      const int w = nth_work(ck);
      if (w >= n_work) return;
      copy_unit(cl, a.k_pool, a.v_pool, w % a.Hkv, lane);
      ++ck;
      read_next(ck);
    } while (csteps == 0);
  };
  auto copy_pair = [&](uint32_t dst) {
    if (cstep < csteps) {
      copy_block(cl, dst, __shfl_sync(0xffffffffu, cid, cstep & 31) * block_stride, lane);
      if (cstep + 1 < csteps)
        copy_block(cl, dst + kRingBlock, __shfl_sync(0xffffffffu, cid, (cstep & 31) + 1) * block_stride, lane);
      cstep += 2;
      if (cstep >= csteps)
        open_next();
      else if ((cstep & 31) == 0)
        cid = cstep + lane < csteps ? cids[W * (cstep + lane)] : 0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  read_next(0);
  open_next();
  copy_pair(ring);
  copy_pair(ring + 2 * kRingBlock);
  uint32_t stage = ring;

  for (int wk = 0, w0 = nth_work(0); w0 < n_work; w0 = nth_work(++wk)) {
    const int g = w0 % a.Hkv;
    const I4Unit& un = a.units[a.unit0 + w0 / a.Hkv];
    const int n_keys = un.n_keys, n_steps = (n_keys + 15) >> 4;
    const int rows = un.rows, row0 = un.row0, q_first = un.q_first, branch = un.branch;

    // Q^T fragments: row i, dims 32 c .. 32 c + 31
    const uint4* q_row = nullptr;
    if (i < rows) {
      const int t = div_g(row0 + i, a.g_inv);
      q_row = reinterpret_cast<const uint4*>(
          a.q + (static_cast<int64_t>(q_first + t) * a.Hq + g * G + row0 + i - t * G) * kHeadDim + 32 * c);
    }
    uint32_t q[16];
    // the largest magnitude as its bf16 bits, which order as the magnitudes do
    uint32_t most2 = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint4 v = q_row ? q_row[x] : make_uint4(0, 0, 0, 0);
      q[4 * x] = v.x;
      q[4 * x + 1] = v.y;
      q[4 * x + 2] = v.z;
      q[4 * x + 3] = v.w;
    }
#pragma unroll
    for (int x = 0; x < 16; ++x) most2 = __vmaxu2(most2, q[x] & 0x7fff7fffu);
    // of row i: a row's factor is its own, whatever the rows beside it hold
    auto row_max = [](uint32_t m) {
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    };
    uint32_t mx = row_max(max(most2 & 0xffffu, most2 >> 16));
    // an infinity or a NaN: every score is infinite or NaN, and so the softmax NaN, of
    // scores that are all -inf too, which would pass for keys that the row does not see
    const bool infinite = mx >= 0x7f80u;
    if (__any_sync(0xffffffffu, infinite)) {
      // the row's largest finite one sets the factor
      uint32_t m = 0;
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const uint32_t lo = q[x] & 0x7fffu, hi = (q[x] >> 16) & 0x7fffu;
        m = max(m, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
      }
      mx = row_max(m);
    }
    const int kexp = mx ? min(100, 14 - (static_cast<int>(mx >> 7) - 127)) : 0;
    const float qf = __uint_as_float(static_cast<uint32_t>(127 + kexp) << 23);
#pragma unroll
    for (int x = 0; x < 16; ++x)
      q[x] = pack_f16x2(__uint_as_float(q[x] << 16) * qf, __uint_as_float(q[x] & 0xffff0000u) * qf);
    // the scores' factors, of the rows 2c and 2c + 1 that the lane's scores are of
    const uint32_t back = infinite ? 0x7fc00000u : static_cast<uint32_t>(127 - kexp) << 23;
    float sl2q[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      sl2q[e] = a.sl2 * kI4Unscale * __uint_as_float(__shfl_sync(0xffffffffu, back, (2 * c + e) * 4));

    // rows 2c, 2c + 1: running reference (log2, less kPShift), sums, O of dims 16 i + 2 x + {0, 1}
    float mo[2] = {kNoMax, kNoMax}, l[2] = {0.f, 0.f};
    float o[8][4];
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[x][e] = 0.f;
    // keys a row of a page's prefix may see; a branch's own keys are seen by all its rows
    auto limit_of = [&](int r) {
      return branch < 0 && r < rows ? min(n_keys, a.q_plen[q_first + div_g(row0 + r, a.g_inv)] - un.key0) : n_keys;
    };
    int lim_min = n_keys;
    if (branch < 0) lim_min = __reduce_min_sync(0xffffffffu, limit_of(lane & 7));

    // P of H blocks' scores (log2 units) against the running references, which move
    // first where a score exceeds them by more than kPSlack
    auto softmax = [&](auto& s) {
      constexpr int H = sizeof(s) / sizeof(s[0]);
      float top[2] = {fmaxf(s[0][0], s[0][2]), fmaxf(s[0][1], s[0][3])};
#pragma unroll
      for (int h = 1; h < H; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) top[e] = max3f(top[e], s[h][e], s[h][2 + e]);
      if (__any_sync(0xffffffffu, fmaxf(top[0] - mo[0], top[1] - mo[1]) > kPShift + kPSlack)) {
        float al[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = top[e];
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, k));
          al[e] = 1.f;
          if (t - mo[e] > kPShift + kPSlack) {
            const float m = __fadd_ru(t, -kPShift);  // up: where floats are 16 apart, down would make P 2^16
            al[e] = fast_exp2(mo[e] - m);
            mo[e] = m;
          }
          l[e] *= al[e];
        }
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[x][e] *= al[e & 1];
      }
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[h][e] = fast_exp2(s[h][e] - mo[e & 1]);
          l[e & 1] += s[h][e];
        }
    };
    // S^T of a block, and O^T += V^T P^T of one
    auto scores = [&](uint32_t src, float (&s)[4]) {
      const KRegs b = read_k(src, key_a, c);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = 0.f;
      const I4Scale sa0 = i4_scale_both<0>(b.sa), sa1 = i4_scale_both<1>(b.sa);
      const I4Scale sb0 = i4_scale_both<0>(b.sb), sb1 = i4_scale_both<1>(b.sb);
      const uint32_t wa[4] = {b.ka.x, b.ka.y, b.ka.z, b.ka.w}, wb[4] = {b.kb.x, b.kb.y, b.kb.z, b.kb.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        // words 0, 1 of the chunk are its first group, 2, 3 its second
        const I4Scale &sa = w < 2 ? sa0 : sa1, &sb = w < 2 ? sb0 : sb1;
        const uint32_t va = wa[w] >> 8, vb = wb[w] >> 8;
        const uint32_t f0[4] = {i4_pair<0>(wa[w], va, sa), i4_pair<0>(wb[w], vb, sb), i4_pair<1>(wa[w], va, sa),
                                i4_pair<1>(wb[w], vb, sb)};
        const uint32_t f1[4] = {i4_pair<2>(wa[w], va, sa), i4_pair<2>(wb[w], vb, sb), i4_pair<3>(wa[w], va, sa),
                                i4_pair<3>(wb[w], vb, sb)};
        mma_f16(s, f0, q[4 * w], q[4 * w + 1]);
        mma_f16(s, f1, q[4 * w + 2], q[4 * w + 3]);
      }
    };
    auto add_values = [&](uint32_t src, const float (&s)[4]) {
      const VRegs b = read_v(src, i, c);
      const uint32_t p0 = transpose8(pack_f16x2(s[0], s[1])), p1 = transpose8(pack_f16x2(s[2], s[3]));
      const I4Scale s01 = i4_scale_two<0>(b.sv), s23 = i4_scale_two<2>(b.sv);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        // low halves: even dims of two keys side by side; high halves: odd dims
        const uint32_t k0 = w ? b.v0.y : b.v0.x, k1 = w ? b.v0.w : b.v0.z;
        const uint32_t k2 = w ? b.v1.y : b.v1.x, k3 = w ? b.v1.w : b.v1.z;
        const uint32_t e01 = __byte_perm(k0, k1, 0x5410), d01 = __byte_perm(k0, k1, 0x7632);
        const uint32_t e23 = __byte_perm(k2, k3, 0x5410), d23 = __byte_perm(k2, k3, 0x7632);
        const uint32_t e01v = e01 >> 8, d01v = d01 >> 8, e23v = e23 >> 8, d23v = d23 >> 8;
        const uint32_t f0[4] = {i4_pair<0>(e01, e01v, s01), i4_pair<0>(d01, d01v, s01), i4_pair<0>(e23, e23v, s23),
                                i4_pair<0>(d23, d23v, s23)};
        mma_f16(o[4 * w + 0], f0, p0, p1);
        const uint32_t f1[4] = {i4_pair<1>(e01, e01v, s01), i4_pair<1>(d01, d01v, s01), i4_pair<1>(e23, e23v, s23),
                                i4_pair<1>(d23, d23v, s23)};
        mma_f16(o[4 * w + 1], f1, p0, p1);
        const uint32_t f2[4] = {i4_pair<2>(e01, e01v, s01), i4_pair<2>(d01, d01v, s01), i4_pair<2>(e23, e23v, s23),
                                i4_pair<2>(d23, d23v, s23)};
        mma_f16(o[4 * w + 2], f2, p0, p1);
        const uint32_t f3[4] = {i4_pair<3>(e01, e01v, s01), i4_pair<3>(d01, d01v, s01), i4_pair<3>(e23, e23v, s23),
                                i4_pair<3>(d23, d23v, s23)};
        mma_f16(o[4 * w + 3], f3, p0, p1);
      }
    };

#pragma unroll 1
    for (int step = warp; step < n_steps; step += 2 * W) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      const bool two = step + W < n_steps;  // an odd count's last pair has one block
      float s[2][4];
      scores(stage, s[0]);
      if (two) {
        scores(stage + kRingBlock, s[1]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[1][e] = -INFINITY;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[h][e] *= sl2q[e & 1];
      if ((step + W) * 16 + 16 > lim_min) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int lim = limit_of(2 * c + e);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key0 = (step + h * W) * 16 + key_a;
            if (key0 >= lim) s[h][e] = -INFINITY;
            if (key0 + 2 >= lim) s[h][2 + e] = -INFINITY;
          }
        }
      }
      softmax(s);
      add_values(stage, s[0]);
      if (two) add_values(stage + kRingBlock, s[1]);
      __syncwarp();
      copy_pair(stage);
      stage = stage == ring ? ring + 2 * kRingBlock : ring;
    }

    // -------------------------------------------------------------- query block
    // scores of all 16 keys by every warp; warp w then takes the keys j % W == w
    const int q_len = un.q_len;
    if (q_len > 0) {
      float s1[1][4] = {{0.f, 0.f, 0.f, 0.f}};
      float(&s)[4] = s1[0];
      const int64_t krow = static_cast<int64_t>(a.Hkv) * kHeadDim;
      const int64_t at = un.qb_first * krow + g * kHeadDim;
      const __nv_bfloat16* kn = a.k_new + at + 32 * c;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint4 z = make_uint4(0, 0, 0, 0);
        const uint4 va = key_a < q_len ? *reinterpret_cast<const uint4*>(kn + key_a * krow + 8 * x) : z;
        const uint4 vb = key_a + 2 < q_len ? *reinterpret_cast<const uint4*>(kn + (key_a + 2) * krow + 8 * x) : z;
        const uint32_t f0[4] = {va.x, vb.x, va.y, vb.y}, f1[4] = {va.z, vb.z, va.w, vb.w};
        const uint4 qv = q_row ? q_row[x] : z;
        mma_bf16(s, f0, qv.x, qv.y);
        mma_bf16(s, f1, qv.z, qv.w);
      }
      constexpr uint32_t kMine = W == 1 ? 0xffffu : W == 2 ? 0x5555u : W == 4 ? 0x1111u : 0x0101u;
      uint32_t vis[2];  // bit j: the row sees key j, one of this warp's
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * c + e;
        uint32_t bits = 0;
        if (r < rows) {
          const int qi = div_g(row0 + r, a.g_inv);
          bits = a.tree_bits ? static_cast<uint32_t>(a.tree_bits[un.qb_first + qi]) : (2u << qi) - 1u;
        }
        vis[e] = bits & ((1u << q_len) - 1u) & (kMine << warp);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)  // plus zero, or NaN, times the row's factor
        s[e] = ((vis[e & 1] >> (key_a + (e >> 1) * 2)) & 1u) ? fmaf(0.f, sl2q[e & 1], s[e] * a.sl2) : -INFINITY;
      softmax(s1);
      const __nv_bfloat16* vn = a.v_new + at + 16 * i;
      bool added = false;
      if (q_len > kFewKeys) {
        // group i of the keys 4c .. 4c + 3, this warp's; any that is not finite?
        uint32_t x[4][8], special = 0;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int j = 4 * c + y;
          const bool mine = j < q_len && (((kMine << warp) >> j) & 1u);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 v = mine ? *reinterpret_cast<const uint4*>(vn + j * krow + 8 * h) : make_uint4(0, 0, 0, 0);
            x[y][4 * h] = v.x;
            x[y][4 * h + 1] = v.y;
            x[y][4 * h + 2] = v.z;
            x[y][4 * h + 3] = v.w;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(special) : "r"(x[y][k]), "r"(0u));
        }
        added = !__any_sync(0xffffffffu, (special & 0x7fff7fffu) != 0u);
        if (added) {
          // P as the sum of two bf16 numbers (16 bits of it); O of cached keys lacks the factor kI4Unscale
          uint32_t ph[2], pl[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = s[2 * h] * (1.f / kI4Unscale), p1 = s[2 * h + 1] * (1.f / kI4Unscale);
            const uint32_t hi = pack_bf16x2(p0, p1);
            ph[h] = transpose8(hi);
            pl[h] = transpose8(pack_bf16x2(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u)));
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            // even dims of two keys side by side, then odd dims
            const uint32_t f[4] = {__byte_perm(x[0][k], x[1][k], 0x5410), __byte_perm(x[0][k], x[1][k], 0x7632),
                                   __byte_perm(x[2][k], x[3][k], 0x5410), __byte_perm(x[2][k], x[3][k], 0x7632)};
            mma_bf16(o[k], f, ph[0], ph[1]);
            mma_bf16(o[k], f, pl[0], pl[1]);
          }
        }
      }
      // a few, or one is not: each is added in f32 to the rows that see it, and to no other
#pragma unroll 1
      for (int j = added ? q_len : warp; j < q_len; j += W) {
        // key j's P sits in lane row 2 (j / 4) + j % 2, first or second register
        // pair; O of cached keys lacks the factor kI4Unscale
        const int from = ((2 * (j >> 2) + (j & 1)) << 2) | c;
        const uint4 x0 = *reinterpret_cast<const uint4*>(vn + j * krow), x1 = *reinterpret_cast<const uint4*>(vn + j * krow + 8);
        const uint32_t xv[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float pj = __shfl_sync(0xffffffffu, (j & 2) ? s[2 + e] : s[e], from) * (1.f / kI4Unscale);
          if ((vis[e] >> j) & 1u) {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              o[x][e] = fmaf(pj, __uint_as_float(xv[x] << 16), o[x][e]);
              o[x][2 + e] = fmaf(pj, __uint_as_float(xv[x] & 0xffff0000u), o[x][2 + e]);
            }
          }
        }
      }
    }

    // -------------------------------------------------------------- results
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], k);
    if constexpr (W > 1) {
      if (warp > 0) {
#pragma unroll
        for (int x = 0; x < 8; ++x) sm.o[warp - 1][x][lane] = make_float4(o[x][0], o[x][1], o[x][2], o[x][3]);
        sm.ml[warp - 1][lane] = make_float4(mo[0], mo[1], l[0], l[1]);
      }
      __syncthreads();
      if (warp == 0) {
#pragma unroll 1
        for (int w = 0; w < W - 1; ++w) {
          const float4 ml = sm.ml[w][lane];
          const float m2[2] = {ml.x, ml.y}, l2[2] = {ml.z, ml.w};
          float f1[2], f2[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // a side that has seen nothing has kNoMax and zero sums
            const float M = fmaxf(mo[e], m2[e]);
            f1[e] = fast_exp2(mo[e] - M);
            f2[e] = fast_exp2(m2[e] - M);
            mo[e] = M;
            l[e] = l[e] * f1[e] + l2[e] * f2[e];
          }
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float4 v = sm.o[w][x][lane];
            o[x][0] = fmaf(v.x, f2[0], o[x][0] * f1[0]);
            o[x][1] = fmaf(v.y, f2[1], o[x][1] * f1[1]);
            o[x][2] = fmaf(v.z, f2[0], o[x][2] * f1[0]);
            o[x][3] = fmaf(v.w, f2[1], o[x][3] * f1[1]);
          }
        }
      }
    }
    if (warp == 0) {
      const int n_pre = un.n_pre;
      const int64_t pre = un.pre, pre_stride = un.pre_stride, part = un.part;
      // the lane's two rows: dims 16 i .. 16 i + 15 of each
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * c + e;
        if (r >= rows) continue;
        const int t = div_g(row0 + r, a.g_inv);
        const int64_t qh = static_cast<int64_t>(t) * a.Hq + g * G + row0 + r - t * G;  // (token, head) from q_first
        float M = mo[e], L = l[e];
        float acc[16];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          acc[2 * x] = o[x][e] * kI4Unscale;
          acc[2 * x + 1] = o[x][2 + e] * kI4Unscale;
        }
#pragma unroll 1
        for (int k = 0; k < n_pre; k += 2) {
          // two results on their way at a time; a missing second one is empty
          float m2[2];
          float4 v[2][4];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int64_t row = pre + min(k + y, n_pre - 1) * pre_stride + qh;
            const float4* src = reinterpret_cast<const float4*>(a.part_o + row * kHeadDim + 16 * i);
            m2[y] = a.part_lse[row];
#pragma unroll
            for (int x = 0; x < 4; ++x) v[y][x] = src[x];
          }
          if (k + 1 == n_pre) m2[1] = -INFINITY;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if (m2[y] == -INFINITY) continue;  // the row saw nothing there
            const float Mn = fmaxf(M, m2[y]);
            const float f1 = fast_exp2(M - Mn), f2 = fast_exp2(m2[y] - Mn);
            M = Mn;
            L = fmaf(L, f1, f2);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              acc[4 * x] = fmaf(v[y][x].x, f2, acc[4 * x] * f1);
              acc[4 * x + 1] = fmaf(v[y][x].y, f2, acc[4 * x + 1] * f1);
              acc[4 * x + 2] = fmaf(v[y][x].z, f2, acc[4 * x + 2] * f1);
              acc[4 * x + 3] = fmaf(v[y][x].w, f2, acc[4 * x + 3] * f1);
            }
          }
        }
        const bool any = !(L == 0.f);  // NaN counts
        const float inv = any ? 1.f / L : 0.f;
#pragma unroll
        for (int x = 0; x < 16; ++x) acc[x] *= inv;
        if (part >= 0) {
          float4* dst = reinterpret_cast<float4*>(a.part_o + (part + qh) * kHeadDim + 16 * i);
#pragma unroll
          for (int x = 0; x < 4; ++x) dst[x] = make_float4(acc[4 * x], acc[4 * x + 1], acc[4 * x + 2], acc[4 * x + 3]);
          if (i == 0) a.part_lse[part + qh] = any ? M + __log2f(L) : -INFINITY;
        } else {
          const int64_t row = static_cast<int64_t>(q_first) * a.Hq + qh;
          uint4* dst = reinterpret_cast<uint4*>(a.o + row * kHeadDim + 16 * i);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            dst[x] = make_uint4(pack_bf16x2(acc[8 * x], acc[8 * x + 1]), pack_bf16x2(acc[8 * x + 2], acc[8 * x + 3]),
                                pack_bf16x2(acc[8 * x + 4], acc[8 * x + 5]), pack_bf16x2(acc[8 * x + 6], acc[8 * x + 7]));
          if (i == 0) a.lse[row] = any ? (M + __log2f(L)) * kLn2 : -INFINITY;
        }
      }
    }
    if (W > 1) __syncthreads();  // the exchange area is free for the next unit
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Rows of branches whose partial results are many: one CTA a (token, head), its
// warps taking every sixteenth result, four of them on their way at a time; lane l
// sums dims 4 l .. 4 l + 3.
constexpr int kMergeWarps = 16;
__global__ void __launch_bounds__(kMergeWarps * 32) merge_i4_kernel(const I4Args a) {
  const I4Merge mg = a.merges[blockIdx.x / a.Hq];
  const int h = blockIdx.x % a.Hq, t = threadIdx.x, warp = t >> 5, lane = t & 31;
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps];
  __shared__ float4 s_o[kMergeWarps][32];
  const int n = mg.n_pre + mg.n_own;
  auto row_of = [&](int k) -> int64_t {
    return k < mg.n_pre ? mg.pre + static_cast<int64_t>(k) * mg.pre_stride + h
                        : mg.own + static_cast<int64_t>(k - mg.n_pre) * mg.own_stride + h;
  };
  float M = kNoMax, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kU = 4;
  for (int k0 = warp; k0 < n; k0 += kMergeWarps * kU) {
    float m[kU];
    float4 v[kU];
#pragma unroll
    for (int x = 0; x < kU; ++x) {
      const int k = k0 + x * kMergeWarps;
      m[x] = -INFINITY;
      v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < n) {
        const int64_t row = row_of(k);
        m[x] = a.part_lse[row];
        v[x] = *reinterpret_cast<const float4*>(a.part_o + row * kHeadDim + 4 * lane);
      }
    }
#pragma unroll
    for (int x = 0; x < kU; ++x) {
      if (m[x] == -INFINITY) continue;  // the row saw nothing there
      const float Mn = fmaxf(M, m[x]);
      const float f1 = fast_exp2(M - Mn), f2 = fast_exp2(m[x] - Mn);
      M = Mn;
      L = fmaf(L, f1, f2);
      acc = make_float4(fmaf(v[x].x, f2, acc.x * f1), fmaf(v[x].y, f2, acc.y * f1), fmaf(v[x].z, f2, acc.z * f1),
                        fmaf(v[x].w, f2, acc.w * f1));
    }
  }
  s_o[warp][lane] = acc;
  if (lane == 0) {
    s_m[warp] = M;
    s_l[warp] = L;
  }
  __syncthreads();
  if (warp) return;
  for (int w = 1; w < kMergeWarps; ++w) {
    const float m2 = s_m[w], Mn = fmaxf(M, m2);
    const float f1 = fast_exp2(M - Mn), f2 = fast_exp2(m2 - Mn);
    const float4 v = s_o[w][lane];
    M = Mn;
    L = L * f1 + s_l[w] * f2;
    acc = make_float4(fmaf(v.x, f2, acc.x * f1), fmaf(v.y, f2, acc.y * f1), fmaf(v.z, f2, acc.z * f1),
                      fmaf(v.w, f2, acc.w * f1));
  }
  const bool any = !(L == 0.f);  // NaN counts
  const float inv = any ? 1.f / L : 0.f;
  const int64_t out = static_cast<int64_t>(mg.token) * a.Hq + h;
  *reinterpret_cast<uint2*>(a.o + out * kHeadDim + 4 * lane) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0) a.lse[out] = any ? (M + __log2f(L)) * kLn2 : -INFINITY;
}

int launch_error(const char* what, std::string* err) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return PADOC_OK;
  *err = std::string(what) + ": " + cudaGetErrorString(e);
  return PADOC_ERR_CUDA;
}

template <int W>
int launch_units(I4Args a, int32_t unit0, int32_t n, cudaStream_t s, std::string* err) {
  const int bytes = sizeof(Smem<W>);
  int per_sm = 0;
  // per device, so asked at each launch (host calls of about a microsecond)
  cudaError_t e = cudaFuncSetAttribute(decode_i4_kernel<W>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, decode_i4_kernel<W>, 32 * W, bytes);
  if (e != cudaSuccess || per_sm < 1) {
    *err = std::string("i4 decode occupancy: ") + cudaGetErrorString(e);
    return PADOC_ERR_CUDA;
  }
  a.unit0 = unit0;
  const int n_work = n * a.Hkv;
  decode_i4_kernel<W><<<std::min(n_work, per_sm * num_sms()), 32 * W, bytes, s>>>(a, n_work);
  return launch_error("i4 decode launch", err);
}

}  // namespace

int launch_i4_units(const I4Args& a, int32_t unit0, int32_t n, int warps, cudaStream_t s, std::string* err) {
  if (n == 0) return PADOC_OK;
  if (warps == 1) return launch_units<1>(a, unit0, n, s, err);
  if (warps == 2) return launch_units<2>(a, unit0, n, s, err);
  if (warps == 4) return launch_units<4>(a, unit0, n, s, err);
  return launch_units<8>(a, unit0, n, s, err);
}

int launch_i4_merge(const I4Args& a, int32_t n_merges, cudaStream_t s, std::string* err) {
  if (n_merges == 0) return PADOC_OK;
  merge_i4_kernel<<<static_cast<unsigned>(n_merges) * a.Hq, kMergeWarps * 32, 0, s>>>(a);
  return launch_error("i4 merge launch", err);
}

}  // namespace padoc

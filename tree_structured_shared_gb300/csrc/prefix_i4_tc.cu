// Prefix pass of branch decode / verify over a 4-bit pool on the tensor cores
// (sm_103a: tcgen05 + TMEM), for pages with many query rows.
//
// A unit is 128 query rows (the rows of every branch of a page, token R / G,
// head R % G of the group) of one kv head against a chunk of the page's shared
// prefix in tiles of 128 keys.  The cache's codes become fp16 operands on the
// way to shared memory: one warpgroup decodes K, one V, each thread taking its
// 72 bytes of a tile straight from global memory into registers a tile ahead,
// so the codes are read once a row tile and no wider copy exists outside the
// SM.  fp16 holds every decoded value exactly; Q's rows are scaled by a power
// of two each (largest magnitude in [2^14, 2^15)), and the scale joins the
// row's softmax.
//
// Roles (512 threads, one persistent CTA per SM):
//   warps 0-3   softmax: thread r owns TMEM lane r = query row r; it also lays
//               out its row of Q, the next unit's before this unit's epilogue
//   warps 4-7   K: thread t decodes key t of the tile (128 dims)
//   warps 8-11  V: thread t decodes 8 keys of one group of 16 dims
//   warp 12     MMA issuer (one thread): S = Q K^T two tiles ahead of O += P V
//   warps 13-15 idle (they complete the warpgroup that gives its registers to
//               the softmax)
// TMEM: three S tiles (P in fp16 written over each) and O, 512 columns.
// Shared memory (128-byte swizzle, two 64-column halves a tile):
//   Q 2 x 32 KB | K 2 x 32 KB | V 2 x 32 KB | barriers
//
// Softmax: P = 2^(x - m + 10) against a running maximum m that moves only when
// exceeded by 2^4 (then O is rescaled in TMEM), so P stays in fp16's range and
// what rounds to zero is below 2^-34 of the row's largest weight.
// Every wait is bounded; a role that gives up raises the CTA's abort flag and
// the device error word, and all roles leave their loops.
#include <cuda_bf16.h>

#include <algorithm>
#include <string>

#include "../../include/padoc.h"
#include "kv_i4.cuh"
#include "padoc_internal.h"
#include "ptx_sm103.cuh"

namespace padoc {

__device__ unsigned int g_i4_err;

namespace {

using namespace ptx;

constexpr int kThreads = 512;
constexpr int kHalf = 16384;  // one 64-column half of a 128-row tile
constexpr int kTileBytes = 2 * kHalf;
constexpr int kQBufs = 2, kKStages = 2, kVStages = 2, kSBufs = 3;
constexpr int SM_Q = 0;
constexpr int SM_K = SM_Q + kQBufs * kTileBytes;
constexpr int SM_V = SM_K + kKStages * kTileBytes;
constexpr int SM_BAR = SM_V + kVStages * kTileBytes;
enum {
  B_Q_FULL = 0,    // +buffer (2), count 4: the unit's Q rows are laid out
  B_K_FULL = 2,    // +stage (2), count 4
  B_K_EMPTY = 4,   // +stage
  B_V_FULL = 6,    // +stage (2), count 4
  B_V_EMPTY = 8,   // +stage: P V of the tile has run
  B_S_FULL = 10,   // +buffer (3): S of the tile is in TMEM
  B_P_FULL = 13,   // +buffer (3), count 4: P of the tile is in TMEM
  B_DRAIN = 16,
  N_BARS = 17
};
constexpr int SM_MISC = SM_BAR + N_BARS * 8;
constexpr int kSmemBytes = SM_MISC + 16 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr uint32_t kTmemO = 384;
constexpr float kPShift = 10.f, kPSlack = 4.f;

// kind::f16 with fp16 A and B and f32 accumulation; b_mn selects an MN-major B.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

template <int R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 ld_cached(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

__device__ __forceinline__ void raise_abort(volatile int* abort, unsigned site) {
  *abort = 1;
  atomicOr(&g_i4_err, site);
}

// Eight dims of a word as one 16-byte piece of a swizzled tile row.
__device__ __forceinline__ void put_word(uint32_t row_addr, int piece, int sw, uint32_t w, uint32_t s2, uint32_t off) {
  // piece 0..15: 16-byte piece of the row's 256 bytes; sw = row & 7
  st_shared_v4(row_addr + (piece >> 3) * kHalf + (((piece & 7) ^ sw) << 4), i4_pair<0>(w, s2, off), i4_pair<1>(w, s2, off),
               i4_pair<2>(w, s2, off), i4_pair<3>(w, s2, off));
}

struct KRegs {
  uint4 c[4];
  uint2 s;
};
struct VRegs {
  uint4 c[4];
  uint2 s;
};

__global__ void __launch_bounds__(kThreads, 1) prefix_i4_kernel(const I4Args a, const int n_work) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + SM_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  if (threadIdx.x == 0) {
    for (int i = 0; i < N_BARS; ++i) {
      uint32_t cnt = 1;
      if (i < B_K_EMPTY || (i >= B_V_FULL && i < B_V_EMPTY) || (i >= B_P_FULL && i < B_DRAIN)) cnt = 4;
      mbar_init(bar(i), cnt);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int G = a.group;

  auto unit_of = [&](int w) -> const I4Unit& { return a.units[a.unit0 + w / a.Hkv]; };

  if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ decoders of K (warps 4-7) and V (8-11)
    regs_dec<104>();
    const bool is_k = warp < 8;
    const int t = threadIdx.x & 127;
    // V: thread t takes block t >> 4, group (t >> 1) & 7, slots 8 (t & 1) .. + 7
    const int tb = t >> 4;  // block of the tile, K and V alike
    const int vg = (t >> 1) & 7, vh = t & 1;
    const uint8_t* pool = static_cast<const uint8_t*>(is_k ? a.k_pool : a.v_pool);
    const int b_full = is_k ? B_K_FULL : B_V_FULL, b_empty = is_k ? B_K_EMPTY : B_V_EMPTY;
    const uint32_t ring = sbase + (is_k ? SM_K : SM_V);
    uint32_t kt = 0;
    bool failed = false;
    for (int w = blockIdx.x; w < n_work && !failed; w += gridDim.x) {
      const I4Unit& un = unit_of(w);
      const int g = w % a.Hkv, n_keys = un.n_keys;
      const int32_t* ids = a.table + static_cast<int64_t>(un.seq) * a.max_bps + un.blk0;
      const int n_tiles = (n_keys + kTileKeys - 1) / kTileKeys, n_blocks = (n_keys + 15) >> 4;
      // the thread's bytes of tile j; blocks past the end read as zero codes of zero scale
      auto load = [&](int j, uint4 (&c)[4], uint2& s, int id) {
        if (j * 8 + tb >= n_blocks || j >= n_tiles) {
#pragma unroll
          for (int x = 0; x < 4; ++x) c[x] = make_uint4(0, 0, 0, 0);
          s = make_uint2(0, 0);
          return;
        }
        const uint8_t* p = pool + (static_cast<int64_t>(id) * a.Hkv + g) * kI4Unit;
        if (is_k) {
          const int slot = t & 15;
#pragma unroll
          for (int x = 0; x < 4; ++x) c[x] = ld_cached(p + x * 256 + slot * 16);
          s = __ldg(reinterpret_cast<const uint2*>(p + kI4Scales + slot * 8));
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) c[x] = ld_cached(p + vg * 128 + vh * 64 + x * 16);
          s = __ldg(reinterpret_cast<const uint2*>(p + kI4Scales + vg * 16 + vh * 8));
        }
      };
      auto id_of = [&](int j) { return j * 8 + tb < n_blocks ? __ldg(ids + j * 8 + tb) : 0; };
      // write tile j's operands into the ring from the thread's registers
      auto emit = [&](int j, const uint4 (&c)[4], const uint2& s) -> bool {
        const int st = kt % 2;
        if (!__all_sync(0xffffffffu, mbar_wait(bar(b_empty + st), ((kt >> 1) & 1) ^ 1, abort))) return false;
        const uint32_t base = ring + st * kTileBytes;
        if (is_k) {
          const uint32_t row = base + t * 128;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t wd[4] = {c[x].x, c[x].y, c[x].z, c[x].w};
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t b = ((x < 2 ? s.x : s.y) >> (8 * ((2 * x + y) & 3))) & 0xffu;
              const uint32_t s2 = i4_scale_pair(b, b), off = i4_offset(s2);
              put_word(row, 4 * x + 2 * y, t & 7, wd[2 * y], s2, off);
              put_word(row, 4 * x + 2 * y + 1, t & 7, wd[2 * y + 1], s2, off);
            }
          }
        } else {
          // keys past the end may hold old bytes: their rows become zero
          const int valid = n_keys - j * kTileKeys - tb * 16 - vh * 8;  // of the thread's 8 slots
          const int swap = vh;  // odd threads take the two slots of a load the other way round: no bank twice
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t lo[2] = {swap ? c[x].z : c[x].x, swap ? c[x].w : c[x].y};
            const uint32_t hi[2] = {swap ? c[x].x : c[x].z, swap ? c[x].y : c[x].w};
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int slot = 2 * x + (y ^ swap);  // of the thread's 8
              const int key = tb * 16 + vh * 8 + slot;
              uint32_t b = ((x < 2 ? s.x : s.y) >> (8 * (slot & 3))) & 0xffu;
              if (slot >= valid) b = 0;
              const uint32_t s2 = i4_scale_pair(b, b), off = i4_offset(s2);
              const uint32_t row = base + key * 128;
              put_word(row, 2 * vg, key & 7, y ? hi[0] : lo[0], s2, off);
              put_word(row, 2 * vg + 1, key & 7, y ? hi[1] : lo[1], s2, off);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b_full + st));
        ++kt;
        return true;
      };
      // two tiles in registers: a tile's loads have two tiles' time to land
      uint4 c0[4], c1[4];
      uint2 s0, s1;
      load(0, c0, s0, id_of(0));
      load(1, c1, s1, id_of(1));
      int id2 = id_of(2), id3 = id_of(3);
      for (int j = 0; j < n_tiles; j += 2) {
        if (!emit(j, c0, s0)) { failed = true; break; }
        load(j + 2, c0, s0, id2);
        id2 = id_of(j + 4);
        if (j + 1 < n_tiles) {
          if (!emit(j + 1, c1, s1)) { failed = true; break; }
          load(j + 3, c1, s1, id3);
          id3 = id_of(j + 5);
        }
      }
    }
    if (failed && lane == 0) raise_abort(abort, is_k ? 0x10000 : 0x20000);
  } else if (warp >= 12) {
    // ------------------------------------------------------------ MMA issuer
    regs_dec<56>();
    if (warp == 12 && lane == 0) {
      constexpr uint32_t id_qk = idesc_f16(128, 128, false), id_pv = idesc_f16(128, 128, true);
      uint32_t ks = 0, kp = 0;  // tiles whose S / P V are issued
      int iu = 0;
      bool failed = false;
      for (int w = blockIdx.x; w < n_work && !failed; w += gridDim.x, ++iu) {
        const int n = (unit_of(w).n_keys + kTileKeys - 1) / kTileKeys;
        if (!mbar_wait_relaxed(bar(B_Q_FULL + (iu & 1)), (iu >> 1) & 1, abort)) { failed = true; break; }
        const uint64_t d_q = sdesc_sw128(sbase + SM_Q + (iu & 1) * kTileBytes, 16, 1024);
        auto issue_s = [&]() -> bool {
          const int st = ks % 2, sb = ks % kSBufs;
          if (!mbar_wait_relaxed(bar(B_K_FULL + st), (ks >> 1) & 1, abort)) return false;
          tc_fence_after();
          const uint64_t d_k = sdesc_sw128(sbase + SM_K + st * kTileBytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t off = static_cast<uint64_t>(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
            mma_bf16_ss(tmem + sb * 128, d_q + off, d_k + off, id_qk, kk > 0);
          }
          mma_commit(bar(B_S_FULL + sb));
          mma_commit(bar(B_K_EMPTY + st));
          ++ks;
          return true;
        };
        if (!issue_s() || (n > 1 && !issue_s())) { failed = true; break; }
        for (int j = 0; j < n; ++j) {
          const int pb = kp % kSBufs, st = kp % 2;
          if (!mbar_wait_relaxed(bar(B_P_FULL + pb), (kp / kSBufs) & 1, abort)) { failed = true; break; }
          tc_fence_after();
          // the S buffer of tile j + 2 last held P of tile j - 1, whose P V was issued before
          if (j + 2 < n && !issue_s()) { failed = true; break; }
          if (!mbar_wait_relaxed(bar(B_V_FULL + st), (kp >> 1) & 1, abort)) { failed = true; break; }
          tc_fence_after();
          const uint64_t d_v = sdesc_sw128(sbase + SM_V + st * kTileBytes, kHalf, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts(tmem + kTmemO, tmem + pb * 128 + kk * 8, d_v + static_cast<uint64_t>(kk * (2048 >> 4)), id_pv,
                        (j > 0 || kk > 0) ? 1u : 0u);
          mma_commit(bar(B_V_EMPTY + st));
          ++kp;
        }
      }
      if (failed) raise_abort(abort, 0x40000);
      // every product issued has completed before TMEM is released
      mma_commit(bar(B_DRAIN));
      int never = 0;
      mbar_wait(bar(B_DRAIN), 0, &never);
    }
  } else {
    // ------------------------------------------------------------ softmax (warps 0-3)
    regs_inc<232>();
    const int r = threadIdx.x;
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    uint32_t kt = 0;
    bool failed = false;
    // lays out row r of a unit's Q in buffer qb; returns the row's softmax factor
    auto lay_q = [&](int w, int qb) -> float {
      const I4Unit& un = unit_of(w);
      const int g = w % a.Hkv, R = un.row0 + r;
      float sl2 = a.sl2;
      if (r < un.rows) {
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + (static_cast<int64_t>(un.q_first + R / G) * a.Hq + g * G + R % G) * kHeadDim);
        uint4 v[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) v[x] = src[x];
        float amax = 0.f;
        auto most = [&](uint32_t u) {
          const float lo = fabsf(__uint_as_float(u << 16)), hi = fabsf(__uint_as_float(u & 0xffff0000u));
          amax = fmaxf(amax, lo <= 3.4028235e38f ? lo : 0.f);
          amax = fmaxf(amax, hi <= 3.4028235e38f ? hi : 0.f);
        };
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          most(v[x].x);
          most(v[x].y);
          most(v[x].z);
          most(v[x].w);
        }
        const int kexp = amax > 0.f ? min(100, 14 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127)) : 0;
        const float qf = __uint_as_float(static_cast<uint32_t>(127 + kexp) << 23);
        sl2 = a.sl2 * __uint_as_float(static_cast<uint32_t>(127 - kexp) << 23);
        auto h = [&](uint32_t u) { return pack_f16x2(__uint_as_float(u << 16) * qf, __uint_as_float(u & 0xffff0000u) * qf); };
        const uint32_t row = sbase + SM_Q + qb * kTileBytes + r * 128;
#pragma unroll
        for (int x = 0; x < 16; ++x)
          st_shared_v4(row + (x >> 3) * kHalf + (((x & 7) ^ (r & 7)) << 4), h(v[x].x), h(v[x].y), h(v[x].z), h(v[x].w));
      }
      // rows past the unit's keep what the buffer held: their results are not read
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_Q_FULL + qb));
      return sl2;
    };
    float sl2_next = blockIdx.x < n_work ? lay_q(blockIdx.x, 0) : 0.f;
    int iu = 0;
    for (int w = blockIdx.x; w < n_work && !failed; w += gridDim.x, ++iu) {
      const I4Unit un = unit_of(w);
      const int g = w % a.Hkv;
      const int n = (un.n_keys + kTileKeys - 1) / kTileKeys;
      const float sl2 = sl2_next;
      const bool valid = r < un.rows, warp_valid = warp * 32 < un.rows;
      const int R = un.row0 + r;
      const int limit = valid ? min(un.n_keys, a.q_plen[un.q_first + R / G] - un.key0) : un.n_keys;
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < n; ++j, ++kt) {
        const int sb = kt % kSBufs;
        if (!__all_sync(0xffffffffu, mbar_wait_relaxed(bar(B_S_FULL + sb), (kt / kSBufs) & 1, abort))) {
          failed = true;
          break;
        }
        tc_fence_after();
        if (warp_valid) {
          float s[128];
          {
            uint32_t v0[32], v1[32], v2[32], v3[32];
            tmem_ld32(tmem + lane_base + sb * 128 + 0, v0);
            tmem_ld32(tmem + lane_base + sb * 128 + 32, v1);
            tmem_ld32(tmem + lane_base + sb * 128 + 64, v2);
            tmem_ld32(tmem + lane_base + sb * 128 + 96, v3);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              s[i] = __uint_as_float(v0[i]);
              s[32 + i] = __uint_as_float(v1[i]);
              s[64 + i] = __uint_as_float(v2[i]);
              s[96 + i] = __uint_as_float(v3[i]);
            }
          }
          const int vis = limit - j * kTileKeys;
          if (vis < kTileKeys) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c >= vis) s[c] = -INFINITY;
          }
          float m8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) m8[i] = s[i];
#pragma unroll
          for (int c = 8; c < 120; c += 16)
#pragma unroll
            for (int i = 0; i < 8; ++i) m8[i] = max3f(m8[i], s[c + i], s[c + 8 + i]);
#pragma unroll
          for (int i = 0; i < 8; ++i) m8[i] = fmaxf(m8[i], s[120 + i]);
          const float tmax = max3f(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
          const float mt = tmax * sl2;
          const bool grow = mt > m_run + kPSlack;
          const float alpha = grow ? fast_exp2(m_run - mt) : 1.f;  // 0 while m_run is -inf
          if (grow) {
            l_run *= alpha;
            m_run = mt;
          }
          const float m_use = (m_run == -INFINITY ? 0.f : m_run) - kPShift;
          {
            const uint64_t sl2x2 = f2pack(sl2, sl2), negm = f2pack(-m_use, -m_use);
            uint64_t l2[4] = {0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < 128; c += 2) {
              float x0, x1;
              f2unpack(fma2(f2pack(s[c], s[c + 1]), sl2x2, negm), x0, x1);
              s[c] = fast_exp2(x0);
              s[c + 1] = fast_exp2(x1);
              l2[(c >> 1) & 3] = add2(l2[(c >> 1) & 3], f2pack(s[c], s[c + 1]));
            }
            float l8[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) f2unpack(l2[k], l8[2 * k], l8[2 * k + 1]);
            l_run += ((l8[0] + l8[1]) + (l8[2] + l8[3])) + ((l8[4] + l8[5]) + (l8[6] + l8[7]));
          }
          if (j > 0 && __any_sync(0xffffffffu, grow)) {
            // O holds sums against the old maximum: rescale once P V of the previous tile has run
            const uint32_t q = kt - 1;
            if (!__all_sync(0xffffffffu, mbar_wait_relaxed(bar(B_V_EMPTY + (q & 1)), (q >> 1) & 1, abort))) {
              failed = true;
              break;
            }
            tc_fence_after();
            uint32_t v[32];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              tmem_ld32(tmem + kTmemO + lane_base + c * 32, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
              tmem_st32(tmem + kTmemO + lane_base + c * 32, v);
            }
            tmem_wait_st();
          }
          uint32_t pk[64];
#pragma unroll
          for (int c = 0; c < 64; ++c) pk[c] = pack_f16x2(s[2 * c], s[2 * c + 1]);
          tmem_st64(tmem + lane_base + sb * 128, pk);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P_FULL + sb));
      }
      if (failed) break;
      // the next unit's Q goes out first, so its S runs while O is read here
      if (w + static_cast<int>(gridDim.x) < n_work) sl2_next = lay_q(w + gridDim.x, (iu + 1) & 1);
      const uint32_t q = kt - 1;
      if (!__all_sync(0xffffffffu, mbar_wait_relaxed(bar(B_V_EMPTY + (q & 1)), (q >> 1) & 1, abort))) {
        failed = true;
        break;
      }
      tc_fence_after();
      if (warp_valid) {
        const bool any = !(l_run == 0.f);
        const float inv = any ? 1.f / l_run : 0.f;
        const int64_t row = un.part + static_cast<int64_t>(R / G) * a.Hq + g * G + R % G;
        float* dst = a.part_o + row * kHeadDim;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(tmem + kTmemO + lane_base + c * 32, v);
          tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t x[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = __float_as_uint(__uint_as_float(v[8 * h + i]) * inv);
              st_global_v8(dst + c * 32 + h * 8, x);
            }
          }
        }
        if (valid) a.part_lse[row] = any ? m_run - kPShift + __log2f(l_run) : -INFINITY;
      }
      // O is read: this warp's next P_FULL arrival (after its
      // tcgen05.fence::before_thread_sync) lets P V overwrite it
    }
    if (failed && lane == 0) raise_abort(abort, 0x80000);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace

int launch_i4_prefix_tc(I4Args a, int32_t unit0, int32_t n_units, cudaStream_t s, std::string* err) {
  if (n_units == 0) return PADOC_OK;
  cudaError_t e = cudaFuncSetAttribute(prefix_i4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) {
    *err = std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e);
    return PADOC_ERR_CUDA;
  }
  a.unit0 = unit0;
  const int n_work = n_units * a.Hkv;
  prefix_i4_kernel<<<std::min(n_work, num_sms()), kThreads, kSmemBytes, s>>>(a, n_work);
  e = cudaGetLastError();
  if (e != cudaSuccess) {
    *err = std::string("i4 prefix launch: ") + cudaGetErrorString(e);
    return PADOC_ERR_CUDA;
  }
  return PADOC_OK;
}

int read_and_clear_i4_error(cudaStream_t s, unsigned* word) {
  unsigned zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_i4_err, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_i4_err, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? PADOC_OK : PADOC_ERR_CUDA;
}

}  // namespace padoc

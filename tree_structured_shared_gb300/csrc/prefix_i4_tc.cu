// Prefix pass of branch decode / verify over a 4-bit pool on the tensor cores
// (sm_103a: tcgen05 + TMEM), for pages with many query rows.
//
// A unit is 128 query rows (the rows of every branch of a page, token R / G,
// head R % G of the group) of one kv head against a chunk of the page's shared
// prefix in tiles of 128 keys.  Two warpgroups turn a tile's codes into fp16
// operand tiles in shared memory, each thread from the 72 bytes it copied there
// itself three tiles ahead; no wider copy exists outside the SM.  fp16 holds
// every decoded value exactly (kv_i4.cuh); Q's rows are scaled by a power of two each
// (largest magnitude in [2^14, 2^15)), and the scale joins the row's softmax.
//
// Roles (544 threads, one persistent CTA per SM):
//   warps 0-3    softmax of the even tiles (numbered across all units of the
//                CTA): thread r owns TMEM lane r = query row r; epilogue
//   warps 4-7    softmax of the odd tiles; lays out the next unit's Q
//   warps 8-11   K: thread t decodes key t of the tile (128 dims)
//   warps 12-15  V: thread t decodes two slots of a block, four groups of 16 dims
//   warp 16      MMA issuer (one thread)
// Even and odd tiles have a running maximum, a sum and an O of their own, joined
// at the unit's end, so neither softmax waits for the other; both halves of TMEM
// hold an S tile (P in fp16 is written over it) and an O.
// Shared memory (operand tiles in two 64-column halves, 128-byte swizzle):
//   Q 32 KB | K 2 x 32 KB | V 2 x 32 KB | codes 3 x 18 KB | row data | barriers
// The decoders and the softmax walk their tiles in short loops: long straight-
// line streams, three a scheduler, starved on instruction fetches (3300 cycles a
// tile at 0.4 instructions a cycle).
//
// Softmax: P = 2^(x - m + 10) against a running maximum m that moves only when
// exceeded by 2^4: at most 2^14, so P stays in fp16's range, and what rounds to
// zero is below 2^-34 of the row's largest weight.
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

constexpr int kThreads = 544;
constexpr int kHalf = 16384;  // one 64-column half of a 128-row tile
constexpr int kTileBytes = 2 * kHalf;
constexpr int kCStages = 3;          // ring of codes
constexpr int kCodes = 4 * 128 * 16;  // a tile's codes, K or V: [4 pieces][thread][16 bytes]
constexpr int kCStage = kCodes + 8 * 128;  // and its scales
constexpr int SM_Q = 0;
constexpr int SM_K = SM_Q + kTileBytes;
constexpr int SM_V = SM_K + 2 * kTileBytes;
constexpr int SM_CK = SM_V + 2 * kTileBytes;
constexpr int SM_CV = SM_CK + kCStages * kCStage;
constexpr int SM_ROW = SM_CV + kCStages * kCStage;  // per unit parity: sl2, m and l of the odd tiles [128] f32
constexpr int kRowBuf = 3 * 128 * 4;
constexpr int SM_BAR = SM_ROW + 2 * kRowBuf;
enum {
  B_Q_FULL = 0,   // count 4: the unit's Q rows are laid out
  B_ML_FULL = 1,  // count 4: the odd tiles' m and l are in shared memory
  B_O_FREE = 2,   // count 4: the epilogue has read both O
  B_K_FULL = 3,   // +tile (2), count 4: K of the CTA's first two tiles
  B_T_FULL = 5,   // +half (2), count 12: P and V of the tile, and K of the tile two on
  B_S_FULL = 7,   // +half (2): S of the tile is in TMEM, its K stage free
  B_PV_DONE = 9,  // +half (2): P V of the tile has run, its V stage free
  B_DRAIN = 11,
  N_BARS = 12
};
// Everything the MMA thread needs for P V of a tile and S of the tile two on
// completes one barrier: tcgen05.mma issue stalls while the pipe is full, so each
// wait and commit between two groups is pipe idle time (with three waits and three
// commits a tile took 2500 cycles).
constexpr int SM_MISC = SM_BAR + N_BARS * 8;
constexpr int kSmemBytes = SM_MISC + 16 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr uint32_t kTmemO = 256;  // S / P of half h at 128 h, O at 256 + 128 h
constexpr float kPShift = 10.f, kPSlack = 4.f;

// kind::f16 with fp16 A and B and f32 accumulation; b_mn selects an MN-major B.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// N bytes from global to shared memory; with ok false the N bytes become zero.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool ok) {
  const uint32_t n = ok ? N : 0;
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ void raise_abort(volatile int* abort, unsigned site) {
  *abort = 1;
  atomicOr(&g_i4_err, site);
}

// The eight dims of a word of codes as one 16-byte piece of an operand tile.
__device__ __forceinline__ void put_word(uint32_t addr, uint32_t w, const I4Scale& s) {
  const uint32_t v = w >> 8;
  st_shared_v4(addr, i4_pair<0>(w, v, s), i4_pair<1>(w, v, s), i4_pair<2>(w, v, s), i4_pair<3>(w, v, s));
}

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
      if (i < B_T_FULL) cnt = 4;
      if (i == B_T_FULL || i == B_T_FULL + 1) cnt = 12;
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

  if (warp >= 8 && warp < 16) {
    // ------------------------------------------------------------ decoders of K (warps 8-11) and V (12-15)
    const bool is_k = warp < 12;
    const int t = threadIdx.x & 127;
    const int b_empty = is_k ? B_S_FULL : B_PV_DONE;
    const uint32_t stage0 = sbase + (is_k ? SM_CK : SM_CV);
    // Half a warp takes a block of the tile, thread s = t & 15 of it the 16-byte
    // pieces s, 16 + s, 32 + s, 48 + s: of K the four chunks of slot s; of V the
    // slots 2 (s & 7), + 1 of the groups 2 x + (s >> 3).  And 8 bytes of scales: K's
    // of slot s; V's of group s >> 1, which its half warp shares.
    const int tb = t >> 4, s16 = t & 15;
    // the copies' own walk over the CTA's tiles, three ahead of the decoding
    int lw = blockIdx.x, lk0 = 0, l_keys = 0;
    const int32_t* l_ids = nullptr;
    const uint8_t* l_pool = nullptr;
    int32_t id = 0;
    const int64_t stride = static_cast<int64_t>(a.Hkv) * kI4Unit;
    auto open_unit = [&]() {
      if (lw >= n_work) return;
      const I4Unit& un = unit_of(lw);
      l_keys = un.n_keys;
      l_ids = a.table + static_cast<int64_t>(un.seq) * a.max_bps + un.blk0 + tb;
      l_pool = static_cast<const uint8_t*>(is_k ? a.k_pool : a.v_pool) + (lw % a.Hkv) * kI4Unit + s16 * 16;
    };
    auto read_id = [&]() { id = lw < n_work && lk0 + tb * 16 < l_keys ? __ldg(l_ids + (lk0 >> 4)) : 0; };
    auto copy_tile = [&](uint32_t dst) {
      if (lw < n_work) {
        const uint8_t* p = l_pool + id * stride;
        const bool ok = lk0 + tb * 16 < l_keys;
#pragma unroll
        for (int x = 0; x < 4; ++x) copy_async<16>(dst + x * 2048 + t * 16, p + x * 256, ok);
        copy_async<8>(dst + kCodes + t * 8, p + kI4Scales - s16 * 8, ok);
        lk0 += kTileKeys;
        if (lk0 >= l_keys) {
          lk0 = 0;
          lw += gridDim.x;
          open_unit();
        }
        read_id();
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    open_unit();
    read_id();
    for (int cs = 0; cs < kCStages; ++cs) copy_tile(stage0 + cs * kCStage);
    // where the thread's pieces of an operand tile go: K, row t; V, the rows of its
    // two slots, the upper four pairs of slots the other way round, so that eight
    // neighbours write eight different banks' pieces
    const int hi = s16 >> 3, swap = (s16 >> 2) & 1;
    const int ka = is_k ? t : tb * 16 + 2 * (s16 & 7) + swap, kb = is_k ? t : ka ^ 1;
    const int first = is_k ? 0 : 2 * hi;
    uint32_t to[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = is_k || k < 2 ? ka : kb, piece = first + (is_k ? k : k & 1);
      to[k] = row * 128 + ((piece ^ (row & 7)) << 4);
    }
    const uint32_t tiles = sbase + (is_k ? SM_K : SM_V);
    uint32_t kt = 0, codes = stage0;
    bool failed = false;
    for (int w = blockIdx.x; w < n_work && !failed; w += gridDim.x) {
      const int n_keys = unit_of(w).n_keys;
      for (int k0 = 0; k0 < n_keys; k0 += kTileKeys, ++kt) {
        const int st = kt & 1;
        asm volatile("cp.async.wait_group %0;" ::"n"(kCStages - 1) : "memory");
        __syncwarp();
        if (!__all_sync(0xffffffffu, mbar_wait(bar(b_empty + st), ((kt >> 1) & 1) ^ 1, abort))) {
          failed = true;
          break;
        }
        const uint32_t tile = tiles + st * kTileBytes;
        if (is_k) {
          // keys past the end are zero or old bytes: their scores are masked
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            const uint32_t src = codes + x * 4096 + t * 16, dst = tile + x * kHalf;
            const uint32_t sc = ld_shared_u32(codes + kCodes + t * 8 + x * 4);
            const uint4 c0 = ld_shared_v4(src), c1 = ld_shared_v4(src + 2048);
            const I4Scale s0 = i4_scale_both<0>(sc), s1 = i4_scale_both<1>(sc);
            put_word(dst + to[0], c0.x, s0);
            put_word(dst + to[1], c0.y, s0);
            put_word(dst + to[2], c0.z, s1);
            put_word(dst + to[3], c0.w, s1);
            const I4Scale s2 = i4_scale_both<2>(sc), s3 = i4_scale_both<3>(sc);
            put_word(dst + (to[0] ^ 64), c1.x, s2);
            put_word(dst + (to[1] ^ 64), c1.y, s2);
            put_word(dst + (to[2] ^ 64), c1.z, s3);
            put_word(dst + (to[3] ^ 64), c1.w, s3);
          }
        } else {
          // keys past the end may hold old bytes and must not be NaN: scales of zero
          const int left = n_keys - k0 - tb * 16 - 2 * (s16 & 7);
          const uint32_t keep = left >= 2 ? 0xffffu : left == 1 ? 0xffu : 0u;
          const uint32_t sel = swap ? 0x4401u : 0x4410u;  // the slots' scales in the order they are written
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            const uint32_t src = codes + x * 4096 + t * 16, dst = tile + x * kHalf;
            // groups 4 x + hi and 4 x + 2 + hi
            const uint32_t sc = codes + kCodes + tb * 128 + (4 * x + hi) * 16 + 2 * (s16 & 7);
            const uint32_t b0 = __byte_perm(ld_shared_u16(sc) & keep, 0u, sel), b1 = __byte_perm(ld_shared_u16(sc + 32) & keep, 0u, sel);
            const uint4 c0 = ld_shared_v4(src), c1 = ld_shared_v4(src + 2048);
            const I4Scale s0 = i4_scale_both<0>(b0), s1 = i4_scale_both<1>(b0);
            put_word(dst + to[0], swap ? c0.z : c0.x, s0);
            put_word(dst + to[1], swap ? c0.w : c0.y, s0);
            put_word(dst + to[2], swap ? c0.x : c0.z, s1);
            put_word(dst + to[3], swap ? c0.y : c0.w, s1);
            const I4Scale s2 = i4_scale_both<0>(b1), s3 = i4_scale_both<1>(b1);
            put_word(dst + (to[0] ^ 64), swap ? c1.z : c1.x, s2);
            put_word(dst + (to[1] ^ 64), swap ? c1.w : c1.y, s2);
            put_word(dst + (to[2] ^ 64), swap ? c1.x : c1.z, s3);
            put_word(dst + (to[3] ^ 64), swap ? c1.y : c1.w, s3);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(is_k && kt < 2 ? B_K_FULL + st : B_T_FULL + st));
        copy_tile(codes);  // the warp has read its bytes of this stage
        codes = codes == stage0 + (kCStages - 1) * kCStage ? stage0 : codes + kCStage;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // the CTA's last two tiles have no K two on
    for (uint32_t v = kt; is_k && v < kt + 2 && !failed; ++v) {
      if (v < 2) continue;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(B_S_FULL + (v & 1)), ((v >> 1) & 1) ^ 1, abort)))
        failed = true;
      else if (lane == 0)
        mbar_arrive(bar(B_T_FULL + (v & 1)));
    }
    if (failed && lane == 0) raise_abort(abort, is_k ? 0x10000 : 0x20000);
  } else if (warp == 16) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_qk = idesc_f16(128, 128, false), id_pv = idesc_f16(128, 128, true);
      uint32_t kt = 0;  // the unit's first tile
      int iu = 0;
      bool failed = false;
      const uint64_t d_q = sdesc_sw128(sbase + SM_Q, 16, 1024);
      // S of tile k.  Its half of TMEM last held P of the tile two back, whose P V
      // this thread has issued before (tcgen05.mma runs in issue order).
      auto issue_s = [&](uint32_t k) {
        const int st = k & 1;
        const uint64_t d_k = sdesc_sw128(sbase + SM_K + st * kTileBytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t off = static_cast<uint64_t>(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
          mma_bf16_ss(tmem + st * 128, d_q + off, d_k + off, id_qk, kk > 0);
        }
        mma_commit(bar(B_S_FULL + st));
      };
      for (int w = blockIdx.x; w < n_work; w += gridDim.x, ++iu) {
        const int n = (unit_of(w).n_keys + kTileKeys - 1) / kTileKeys;
        if (!mbar_wait_relaxed(bar(B_Q_FULL), iu & 1, abort) ||
            (kt == 0 && !mbar_wait_relaxed(bar(B_K_FULL), 0, abort)) ||
            (kt < 2 && kt + n > 1 && !mbar_wait_relaxed(bar(B_K_FULL + 1), 0, abort))) {
          failed = true;
          break;
        }
        tc_fence_after();
        issue_s(kt);
        if (n > 1) issue_s(kt + 1);
        for (int j = 0; j < n; ++j) {
          const uint32_t k = kt + j;
          const int st = k & 1;
          if (!mbar_wait_relaxed(bar(B_T_FULL + st), (k >> 1) & 1, abort)) { failed = true; break; }
          tc_fence_after();
          const uint64_t d_v = sdesc_sw128(sbase + SM_V + st * kTileBytes, kHalf, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts(tmem + kTmemO + st * 128, tmem + st * 128 + kk * 8, d_v + static_cast<uint64_t>(kk * (2048 >> 4)), id_pv,
                        (j > 1 || kk > 0) ? 1u : 0u);
          mma_commit(bar(B_PV_DONE + st));
          if (j + 2 < n) issue_s(k + 2);
        }
        if (failed) break;
        kt += n;
      }
      if (failed) raise_abort(abort, 0x40000);
      // every product issued has completed before TMEM is released
      mma_commit(bar(B_DRAIN));
      int never = 0;
      mbar_wait(bar(B_DRAIN), 0, &never);
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int odd = warp >> 2;  // this warpgroup's tiles, its half of TMEM
    const int r = threadIdx.x & 127, wq = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t t_s = tmem + lane_base + odd * 128, t_o = tmem + kTmemO + lane_base;
    uint32_t kt0 = 0;  // number of the unit's first tile
    bool failed = false;
    auto row_buf = [&](int iu) { return reinterpret_cast<float*>(smem + SM_ROW + (iu & 1) * kRowBuf); };
    // Odd tiles' threads: row r of the next unit's Q.  Its scaling is found after the
    // unit's first odd tile, while the thread would wait for its next S (which also
    // brings the row near); once every S of the unit has run, the row goes to shared
    // memory.
    int q_for = -1;                 // the unit that the following is of
    const uint4* q_src = nullptr;   // its row, if it has one
    float q_scale = 1.f, q_sl2 = a.sl2 * kI4Unscale;
    auto prepare_q = [&](int w) {
      if (w >= n_work) return;
      const I4Unit& un = unit_of(w);
      q_for = w;
      q_src = nullptr;
      if (r >= un.rows) return;
      const int R = un.row0 + r, t = div_g(R, a.g_inv);
      q_src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<int64_t>(un.q_first + t) * a.Hq + (w % a.Hkv) * G + R - t * G) * kHeadDim);
      // the largest magnitude as its bf16 bits, which order as the magnitudes do
      uint32_t most2 = 0, fin = 0;
#pragma unroll
      for (int x0 = 0; x0 < 16; x0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = __ldg(q_src + x0 + x);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const uint32_t u[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) most2 = __vmaxu2(most2, u[k] & 0x7fff7fffu);
        }
      }
      uint32_t mx = max(most2 & 0xffffu, most2 >> 16);
      if (mx >= 0x7f80u) {
        // an infinity or a NaN: the largest finite one sets the factor
        for (int x = 0; x < 64; ++x) {
          const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(q_src) + x), lo = u & 0x7fffu, hi = (u >> 16) & 0x7fffu;
          fin = max(fin, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
        mx = fin;
      }
      const int kexp = mx ? min(100, 14 - (static_cast<int>(mx >> 7) - 127)) : 0;
      q_scale = __uint_as_float(static_cast<uint32_t>(127 + kexp) << 23);
      q_sl2 = a.sl2 * kI4Unscale * __uint_as_float(static_cast<uint32_t>(127 - kexp) << 23);
    };
    auto put_q = [&](int w, int iu) {
      if (q_for != w) prepare_q(w);
      if (q_src) {
        auto h = [&](uint32_t u) {
          return pack_f16x2(__uint_as_float(u << 16) * q_scale, __uint_as_float(u & 0xffff0000u) * q_scale);
        };
        const uint32_t row = sbase + SM_Q + r * 128;
#pragma unroll
        for (int x0 = 0; x0 < 16; x0 += 8) {
          uint4 v[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) v[x] = __ldg(q_src + x0 + x);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            st_shared_v4(row + (x0 >> 3) * kHalf + ((x ^ (r & 7)) << 4), h(v[x].x), h(v[x].y), h(v[x].z), h(v[x].w));
        }
      }
      // rows past the unit's keep what the buffer held: their results are not read
      row_buf(iu)[r] = q_sl2;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_Q_FULL));
    };
    if (odd && blockIdx.x < n_work) put_q(blockIdx.x, 0);
    int iu = 0;
    for (int w = blockIdx.x; w < n_work && !failed; w += gridDim.x, ++iu) {
      const I4Unit& un = unit_of(w);
      const int rows = un.rows, n_keys = un.n_keys;
      const int n = (n_keys + kTileKeys - 1) / kTileKeys;
      const bool valid = r < rows, warp_valid = wq * 32 < rows;
      const int R = un.row0 + r, tok = div_g(R, a.g_inv);
      const int limit = valid ? min(n_keys, a.q_plen[un.q_first + tok] - un.key0) : n_keys;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(B_Q_FULL), iu & 1, abort))) {
        failed = true;
        break;
      }
      const float sl2 = row_buf(iu)[r];
      const int j0 = (kt0 & 1) == odd ? 0 : 1;  // the unit's first tile of this parity
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = j0; j < n; j += 2) {
        const uint32_t kt = kt0 + j;
        if (!__all_sync(0xffffffffu, mbar_wait_relaxed(bar(B_S_FULL + odd), (kt >> 1) & 1, abort))) {
          failed = true;
          break;
        }
        tc_fence_after();
        if (warp_valid) {
          const int vis = limit - j * kTileKeys;  // keys [0, vis) of the tile are visible
          auto mask32 = [&](int c, uint32_t (&v)[32]) {
            const int left = vis - c * 32;
            if (left < 32) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i >= left) v[i] = 0xff800000u;
            }
          };
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            uint32_t v0[32], v1[32];
            tmem_ld32(t_s + c * 32, v0);
            tmem_ld32(t_s + c * 32 + 32, v1);
            tmem_wait_ld();
            mask32(c, v0);
            mask32(c + 1, v1);
            float m4[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; i += 4)
#pragma unroll
              for (int k = 0; k < 4; ++k) m4[k] = max3f(m4[k], __uint_as_float(v0[i + k]), __uint_as_float(v1[i + k]));
            mx = fmaxf(max3f(m4[0], m4[1], m4[2]), m4[3]);
          }
          const float mt = mx * sl2;
          const bool grow = mt > m_run + kPSlack;
          const float alpha = grow ? fast_exp2(m_run - mt) : 1.f;  // 0 while m_run is -inf
          if (grow) {
            l_run *= alpha;
            m_run = mt;
          }
          if (j > j0 && __any_sync(0xffffffffu, grow)) {
            // O holds sums against the old maximum: rescale once P V of the previous tile has run
            if (!__all_sync(0xffffffffu, mbar_wait_relaxed(bar(B_PV_DONE + odd), ((kt - 2) >> 1) & 1, abort))) {
              failed = true;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t v[32];
              tmem_ld32(t_o + odd * 128 + c * 32, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
              tmem_st32(t_o + odd * 128 + c * 32, v);
            }
            tmem_wait_st();
          }
          const float m_use = (m_run == -INFINITY ? 0.f : m_run) - kPShift;
          const uint64_t sl2x2 = f2pack(sl2, sl2), negm = f2pack(-m_use, -m_use);
          uint64_t l2[2] = {0, 0};
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32], pk[16];
            tmem_ld32(t_s + c * 32, v);
            tmem_wait_ld();
            mask32(c, v);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float x0, x1;
              f2unpack(fma2(f2pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sl2x2, negm), x0, x1);
              x0 = fast_exp2(x0);
              x1 = fast_exp2(x1);
              l2[(i >> 1) & 1] = add2(l2[(i >> 1) & 1], f2pack(x0, x1));
              pk[i >> 1] = pack_f16x2(x0, x1);
            }
            // over columns of S that this loop has read
            tmem_st16(t_s + c * 16, pk);
          }
          float l4[4];
          f2unpack(l2[0], l4[0], l4[1]);
          f2unpack(l2[1], l4[2], l4[3]);
          l_run += (l4[0] + l4[1]) + (l4[2] + l4[3]);
          tmem_wait_st();
        }
        if (odd && j == j0 && iu > 0 &&
            !__all_sync(0xffffffffu, mbar_wait(bar(B_O_FREE), (iu - 1) & 1, abort))) {
          failed = true;  // P V may overwrite the odd tiles' O once the last epilogue has read it
          break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_T_FULL + odd));
        if (odd && j == j0) prepare_q(w + gridDim.x);
      }
      if (failed) break;
      // the unit's last tile, and the last of the other parity (if it has one)
      const uint32_t last = kt0 + n - 1;
      kt0 += n;
      if (odd) {
        row_buf(iu)[128 + r] = m_run;
        row_buf(iu)[256 + r] = l_run;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_ML_FULL));
        if (w + static_cast<int>(gridDim.x) < n_work) {
          // Q is free once every S of this unit has run; the even tiles' last one
          // is waited for here (its barrier cannot move on before the next Q is out)
          const uint32_t k = (last & 1) ? last - 1 : last;
          if ((n > 1 || !(last & 1)) &&
              !__all_sync(0xffffffffu, mbar_wait_relaxed(bar(B_S_FULL), (k >> 1) & 1, abort))) {
            failed = true;
            break;
          }
          put_q(w + gridDim.x, iu + 1);
        }
        continue;
      }
      const uint32_t ke = (last & 1) ? last - 1 : last, ko = (last & 1) ? last : last - 1;  // last even, last odd tile
      const bool has_e = n > 1 || !(last & 1), has_o = n > 1 || (last & 1);
      if ((has_e && !__all_sync(0xffffffffu, mbar_wait_relaxed(bar(B_PV_DONE), (ke >> 1) & 1, abort))) ||
          (has_o && !__all_sync(0xffffffffu, mbar_wait_relaxed(bar(B_PV_DONE + 1), (ko >> 1) & 1, abort))) ||
          !__all_sync(0xffffffffu, mbar_wait(bar(B_ML_FULL), iu & 1, abort))) {
        failed = true;
        break;
      }
      tc_fence_after();
      if (warp_valid) {
        const float m_o = row_buf(iu)[128 + r], l_o = row_buf(iu)[256 + r];
        const bool any_e = !(l_run == 0.f), any_o = !(l_o == 0.f);  // NaN counts
        const float M = fmaxf(any_e ? m_run : -INFINITY, any_o ? m_o : -INFINITY);
        const float we = any_e ? fast_exp2(m_run - M) : 0.f, wo = any_o ? fast_exp2(m_o - M) : 0.f;
        const float L = (any_e ? l_run * we : 0.f) + (any_o ? l_o * wo : 0.f);
        const float fe = any_e ? we * kI4Unscale / L : 0.f, fo = any_o ? wo * kI4Unscale / L : 0.f;
        const int64_t row = un.part + static_cast<int64_t>(tok) * a.Hq + (w % a.Hkv) * G + R - tok * G;
        float* dst = a.part_o + row * kHeadDim;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t ve[32], vo[32];
          tmem_ld32(t_o + c * 32, ve);
          tmem_ld32(t_o + 128 + c * 32, vo);
          tmem_wait_ld();
          if (valid) {
            // an O that no tile of this unit wrote holds old values: its factor is 0 and it is left out
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t x[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                x[i] = __float_as_uint((any_e ? __uint_as_float(ve[8 * h + i]) * fe : 0.f) +
                                       (any_o ? __uint_as_float(vo[8 * h + i]) * fo : 0.f));
              st_global_v8(dst + c * 32 + h * 8, x);
            }
          }
        }
        if (valid) a.part_lse[row] = any_e || any_o ? M - kPShift + __log2f(L) : -INFINITY;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_O_FREE));
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

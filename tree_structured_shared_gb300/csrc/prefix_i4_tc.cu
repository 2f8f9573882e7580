// Prefix pass of branch decode / verify over a 4-bit pool on the tensor cores
// (sm_103a: tcgen05 + TMEM), for pages with many query rows.
//
// A unit is 128 query rows (the rows of every branch of a page, token R / G,
// head R % G of the group) of one kv head against a run of the page's shared
// prefix in tiles of 128 keys.  Two warpgroups turn a tile's codes into fp16
// operand tiles in shared memory, each thread from the 72 bytes it copied there
// itself three tiles ahead; no wider copy exists outside the SM.  fp16 holds
// every decoded value exactly (kv_i4.cuh); Q's rows are scaled by a power of two each
// (largest magnitude in [2^14, 2^15)), and the scale joins the row's softmax.
//
// Roles (768 threads, one persistent CTA per SM; a kv head's CTAs walk runs of
// units that the plan made equally long):
//   warps 0-11   softmax, three groups of four: group b takes the tiles b, b + 3, ...
//                (numbered across all units of the CTA), thread r TMEM lane r = query
//                row r; group 0 also stores the results, group 2 lays out the next Q
//   warps 12-15  K: thread t decodes key t of the tile (128 dims)
//   warps 16-19  V: thread t decodes two slots of a block, four groups of 16 dims
//   warps 20, 21 issue S = Q K^T and O += P V (one thread each)
// TMEM: an S tile for each group (P in fp16 is written over it) and O, 512 columns.
// The groups keep a sum of their own but share each row's reference: a tile takes
// over the one of the tile before it (published in shared memory once that tile's
// maximum is known) and moves it only where it must.
// Shared memory (operand tiles in two 64-column halves, 128-byte swizzle):
//   Q 32 KB | K 2 x 32 KB | V 2 x 32 KB | codes 3 x 18 KB | row data | barriers
//
// What bounds it: a tile goes round its S buffer in some 6000 cycles, three tiles at a
// time (S issued in 900, first softmax pass 1000, second 1700, P V issued in 800, some
// 450 between any two), so 1950 cycles a tile, of which the products need 1024 of the
// tensor pipe.  (These are from before the second pass took the difference of two scores
// ahead of the factor, see below; the whole pass takes 3 to 4 % longer since.)  The
// products run slower than that because shared memory's data pipe is 73 % busy: a tile's
// products read 96 KB, the decoders write 64 KB, and the codes pass twice, 72 KB.  Schedulers
// issue every other cycle.
//   128 pages of 4000-6144 tokens with 8-60 branches: 326 us (112 at HBM rate)
//   64 pages of 4809 tokens, 8-40 branches of up to 16 query tokens: 588 us (the
//   products alone: 336)
// What was measured on the way there (the two cases in us):
//   - two softmax groups instead of three: 640 on the second; one thread issuing both
//     products spends 2240 cycles a tile on issue and waits;
//   - loops: six warps a scheduler run different code and starve on instruction
//     fetches.  First pass of 32 columns a round instead of 64, masked scores put back
//     instead of masked again by the second pass, K and V decoded by the same
//     instructions: 380 -> 343, 601 -> 572.  Half the columns a round in the second
//     pass, or half the words in the decoders', costs 3 %, twice the columns 10 %;
//   - P handed over in two halves, the reference waited for ahead of S: 336, 564;
//   - lanes past a unit's rows, whose Q is what the buffer held, no longer ask for
//     rescalings of O: 324; decoders' reads without bank conflicts: 316, 566;
//   - scores less the reference before the factor, below: 326, 588;
//   - issue code with constant stages and buffers, or more registers for it: 2 to 6 %
//     slower.
//
// A wait names a phase by its parity, so every waiter knows the phase before to be
// over: from the barriers that it waited for, or from what the phase's arrivals
// themselves waited for.
//
// Softmax: P = 2^(x - m + 10) against a running maximum m that moves only when
// exceeded by 2^4: at most 2^14, so P stays in fp16's range, and what rounds to
// zero is below 2^-34 of the row's largest weight.  References are scores as they come
// out of S, and x - m is their difference times the factor: the product of each, rounded
// on its own, would be off by whole powers of two from scores of 2^24 on, and P infinite
// or zero.  (One fma an element and no subtraction: 12 us less on the first case, 22 on
// the second, own pass included.  Finding such rows by their factor and multiplying their
// scores ahead of that fma cost 10 to 33 us, though no row took it.)
// Every wait is bounded; a role that gives up raises the CTA's abort flag and
// the device error word, and all roles leave their loops: no warp arrives twice on a
// barrier's phase, since it first waits for what that phase's completion implies; the
// decoders wait for their copies, and each issuer commits once more and waits for that,
// before the CTA's threads meet and TMEM is released.
#include <cuda_bf16.h>

#include <algorithm>
#include <string>

#include "../../include/padoc.h"
#include "kv_i4.cuh"
#include "padoc_internal.h"
#include "ptx_sm103.cuh"

namespace padoc {

__device__ unsigned int g_i4_err;
// Longest time one wait of the prefix kernel may take before it gives up (nanoseconds of
// the global timer); settable for tests, read at launch.
__device__ unsigned long long g_i4_wait_limit_ns = ptx::kWaitLimitNs;

namespace {

using namespace ptx;

constexpr int kThreads = 768;
// registers a thread of each role, dealt from the 80 a thread that 768 threads start with
constexpr int kRegsSoft = 104, kRegsDec = 64, kRegsMma = 40;
constexpr int kRegsLaunch = 80;
static_assert(384 * kRegsSoft + 256 * kRegsDec + 128 * kRegsMma <= kRegsLaunch * kThreads, "register budget");
static_assert(kRegsSoft >= kRegsLaunch && kRegsDec <= kRegsLaunch && kRegsMma <= kRegsLaunch,
              "a role may only grow by the increasing form and shrink by the other");
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
constexpr int SM_ROW = SM_CV + kCStages * kCStage;  // per unit parity: sl2, groups 1's and 2's references and sums [128] f32
constexpr int kRowBuf = 5 * 128 * 4;
constexpr int SM_M = SM_ROW + 2 * kRowBuf;  // per group: the rows' references [128] f32
constexpr int SM_BAR = SM_M + 3 * 128 * 4;
enum {
  B_Q_FULL = 0,   // count 4: the unit's Q rows are laid out
  B_O_FREE = 1,   // count 4: the epilogue has read O
  B_K_FULL = 2,   // +stage (2), count 4
  B_V_FULL = 4,   // +stage (2), count 4
  B_M_FULL = 6,   // +group (3), count 4: the tile's references are in shared memory
  B_P_FULL = 9,   // +group (3), count 4: and of the others
  B_P_HALF = 12,  // +group (3), count 4: P of the tile's first 64 keys
  B_ML_FULL = 15, // count 8: groups 1's and 2's references and sums are in shared memory
  B_E_IN = 16,    // count 8: groups 0 and 1 have entered the unit
  B_PV_DONE = 17, // +group (3): P V of the tile has run, its V stage and S buffer free
  B_S_FULL = 20,  // +group (3): S of the tile is in TMEM, its K stage free
  B_DRAIN = 23,   // count 2: the issuers' last commits
  N_BARS = 24
};
// The commits of S and P V free the stages that they read too: each wait and commit
// between two groups of products is time in which the issuing thread stands still.
constexpr int SM_MISC = SM_BAR + N_BARS * 8;  // TMEM address, abort flag, limit of a wait (64 bits)
static_assert(SM_MISC % 8 == 0, "the limit's alignment");
constexpr int kSmemBytes = SM_MISC + 16 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr uint32_t kTmemO = 384;  // S / P of buffer b at 128 b
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
template <int N, bool Up>
__device__ __forceinline__ void set_max_regs() {
  if (Up)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
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

// As mbar_wait and mbar_wait_relaxed, with the limit that lies behind the abort flag.
template <bool RELAXED>
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort) {
  auto done = [&]() { return RELAXED ? mbar_try_wait_relaxed(bar, parity) : mbar_try_wait(bar, parity); };
  if (done()) return true;
  const uint64_t t0 = global_timer();
  while (true) {
    for (int i = 0; i < 32; ++i)
      if (done()) return true;
    if (*abort) return false;
    if (global_timer() - t0 > *reinterpret_cast<volatile uint64_t*>(abort + 1)) return false;
  }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  return wait_phase<false>(bar, parity, abort);
}
__device__ __forceinline__ bool wait_relaxed(uint32_t bar, uint32_t parity, volatile int* abort) {
  return wait_phase<true>(bar, parity, abort);
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

__global__ void __launch_bounds__(kThreads, 1) prefix_i4_kernel(const I4Args a) {
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
      // one arrival a warp, one a commit
      const uint32_t cnt = i < B_ML_FULL ? 4 : i < B_PV_DONE ? 8 : i == B_DRAIN ? 2 : 1;
      mbar_init(bar(i), cnt);
    }
    *abort = 0;
    *reinterpret_cast<volatile uint64_t*>(abort + 1) = kWaitLimitNs;
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
  // a group of CTAs takes a run of units, each CTA one kv head of them
  const int g = blockIdx.x % a.Hkv, u0 = a.tc_first[blockIdx.x / a.Hkv], u1 = a.tc_first[blockIdx.x / a.Hkv + 1];

  if (warp >= 12 && warp < 20) {
    // ------------------------------------------------------------ decoders of K (warps 12-15) and V (16-19)
    set_max_regs<kRegsDec, false>();
    const bool is_k = warp < 16;
    const int t = threadIdx.x & 127;
    const uint32_t stage0 = sbase + (is_k ? SM_CK : SM_CV);
    // Half a warp takes a block of the tile, thread s = t & 15 of it the 16-byte
    // pieces s, 16 + s, 32 + s, 48 + s: of K the four chunks of slot s; of V the
    // slots 2 (s & 7), + 1 of the groups 2 x + (s >> 3).  And 8 bytes of scales: K's
    // of slot s; V's of group s >> 1, which its half warp shares.
    const int tb = t >> 4, s16 = t & 15;
    // the copies' own walk over the CTA's tiles, three ahead of the decoding
    int lu = u0, lk0 = 0, l_keys = 0;
    const int32_t* l_ids = nullptr;
    const uint8_t* l_pool = nullptr;
    int32_t id = 0;
    const int64_t stride = static_cast<int64_t>(a.Hkv) * kI4Unit;
    auto open_unit = [&]() {
      if (lu >= u1) return;
      const I4Unit& un = a.units[lu];
      l_keys = un.n_keys;
      l_ids = a.table + static_cast<int64_t>(un.seq) * a.max_bps + un.blk0 + tb;
      l_pool = static_cast<const uint8_t*>(is_k ? a.k_pool : a.v_pool) + (g) * kI4Unit + s16 * 16;
    };
    auto read_id = [&]() { id = lu < u1 && lk0 + tb * 16 < l_keys ? __ldg(l_ids + (lk0 >> 4)) : 0; };
    auto copy_tile = [&](uint32_t dst) {
      if (lu < u1) {
        const uint8_t* p = l_pool + id * stride;
        const bool ok = lk0 + tb * 16 < l_keys;
#pragma unroll
        for (int x = 0; x < 4; ++x) copy_async<16>(dst + x * 2048 + t * 16, p + x * 256, ok);
        copy_async<8>(dst + kCodes + t * 8, p + kI4Scales - s16 * 8, ok);
        lk0 += kTileKeys;
        if (lk0 >= l_keys) {
          lk0 = 0;
          ++lu;
          open_unit();
        }
        read_id();
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    open_unit();
    read_id();
    for (int cs = 0; cs < kCStages; ++cs) copy_tile(stage0 + cs * kCStage);
    // Where the thread's pieces of an operand tile go: K, row t; V, the rows of its two
    // slots.  A thread reads its 16 bytes of codes in two halves, some the upper one
    // first (swap), so that sixteen neighbours read every bank once (thread s and s + 8
    // start with different halves) and eight neighbours write eight different banks'
    // pieces.  K's halves are two groups of dims, V's the two slots.
    const int hi = s16 >> 3, swap = is_k ? hi : hi ^ ((s16 >> 2) & 1), sw = swap * 8;
    uint32_t to[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = is_k ? t : tb * 16 + 2 * (s16 & 7) + ((k >> 1) ^ swap);
      const int piece = is_k ? k ^ (2 * swap) : 2 * hi + (k & 1);
      to[k] = row * 128 + ((piece ^ (row & 7)) << 4);
    }
    const uint32_t tiles = sbase + (is_k ? SM_K : SM_V);
    uint32_t kt = 0, codes = stage0;
    bool failed = false;
    for (int u = u0; u < u1 && !failed; ++u) {
      const int n_keys = a.units[u].n_keys;
      for (int k0 = 0; k0 < n_keys; k0 += kTileKeys, ++kt) {
        const int st = kt & 1;
        asm volatile("cp.async.wait_group %0;" ::"n"(kCStages - 1) : "memory");
        __syncwarp();
        // the stage's last tile, two back: S (K) or P V (V) has run
        const uint32_t old = kt - 2;
        if (kt >= 2 &&
            !__all_sync(0xffffffffu, wait(bar((is_k ? B_S_FULL : B_PV_DONE) + old % 3), (old / 3) & 1, abort))) {
          failed = true;
          break;
        }
        const uint32_t tile = tiles + st * kTileBytes;
        // Keys past the end may hold old bytes: K's scores are masked, V's scales become
        // zero.  K and V run the same instructions (see the top) but for their scales:
        // K's groups 4 x .. 4 x + 3 of its slot, V's of its two slots in the groups 4 x + hi
        // and 4 x + 2 + hi, in the order in which they are used.
        const int left = n_keys - k0 - tb * 16 - 2 * (s16 & 7);
        const uint32_t keep = left >= 2 ? 0xffffu : left == 1 ? 0xffu : 0u;
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          const uint32_t src = codes + x * 4096 + t * 16, dst = tile + x * kHalf;
          uint32_t sc;
          if (is_k) {
            sc = __byte_perm(ld_shared_u32(codes + kCodes + t * 8 + x * 4), 0u, swap ? 0x2301u : 0x3210u);
          } else {
            const uint32_t at = codes + kCodes + tb * 128 + (4 * x + hi) * 16 + 2 * (s16 & 7);
            sc = __byte_perm(ld_shared_u16(at) & keep, ld_shared_u16(at + 32) & keep, swap ? 0x4501u : 0x5410u);
          }
          const uint2 c0 = ld_shared_v2(src + sw), c1 = ld_shared_v2(src + (sw ^ 8));
          const uint2 c2 = ld_shared_v2(src + 2048 + sw), c3 = ld_shared_v2(src + 2048 + (sw ^ 8));
          const I4Scale s0 = i4_scale_both<0>(sc), s1 = i4_scale_both<1>(sc);
          put_word(dst + to[0], c0.x, s0);
          put_word(dst + to[1], c0.y, s0);
          put_word(dst + to[2], c1.x, s1);
          put_word(dst + to[3], c1.y, s1);
          const I4Scale s2 = i4_scale_both<2>(sc), s3 = i4_scale_both<3>(sc);
          put_word(dst + (to[0] ^ 64), c2.x, s2);
          put_word(dst + (to[1] ^ 64), c2.y, s2);
          put_word(dst + (to[2] ^ 64), c3.x, s3);
          put_word(dst + (to[3] ^ 64), c3.y, s3);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar((is_k ? B_K_FULL : B_V_FULL) + st));
        copy_tile(codes);  // the warp has read its bytes of this stage
        codes = codes == stage0 + (kCStages - 1) * kCStage ? stage0 : codes + kCStage;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (failed && lane == 0) raise_abort(abort, is_k ? 0x10000 : 0x20000);
  } else if (warp >= 20) {
    // ------------------------------------------------------------ issuers
    set_max_regs<kRegsMma, false>();
    if (warp == 20 && lane == 0) {
      // S = Q K^T
      constexpr uint32_t id_qk = idesc_f16(128, 128, false);
      const uint64_t d_q = sdesc_sw128(sbase + SM_Q, 16, 1024);
      uint32_t k = 0, sb = 0, round = 0;  // tile, its buffer k % 3, k / 3
      int iu = 0;
      bool failed = false;
      for (int u = u0; u < u1 && !failed; ++u, ++iu) {
        const int n = (a.units[u].n_keys + kTileKeys - 1) / kTileKeys;
        if (!wait_relaxed(bar(B_Q_FULL), iu & 1, abort)) failed = true;
        for (int j = 0; j < n && !failed; ++j, ++k) {
          // the buffer last held P of the tile three back
          if ((round > 0 && !wait_relaxed(bar(B_PV_DONE + sb), (round - 1) & 1, abort)) ||
              !wait_relaxed(bar(B_K_FULL + (k & 1)), (k >> 1) & 1, abort)) {
            failed = true;
            break;
          }
          tc_fence_after();
          const uint64_t d_k = sdesc_sw128(sbase + SM_K + (k & 1) * kTileBytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t off = static_cast<uint64_t>(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
            mma_bf16_ss(tmem + sb * 128, d_q + off, d_k + off, id_qk, kk > 0);
          }
          mma_commit(bar(B_S_FULL + sb));
          if (++sb == 3) {
            sb = 0;
            ++round;
          }
        }
      }
      if (failed) raise_abort(abort, 0x40000);
      // every product issued has completed before TMEM is released
      mma_commit(bar(B_DRAIN));
      int never = 0;
      mbar_wait(bar(B_DRAIN), 0, &never);
    } else if (warp == 21 && lane == 0) {
      // O += P V
      constexpr uint32_t id_pv = idesc_f16(128, 128, true);
      uint32_t k = 0, pb = 0, round = 0;  // tile, its buffer k % 3, k / 3
      bool failed = false;
      for (int u = u0; u < u1 && !failed; ++u) {
        const int n = (a.units[u].n_keys + kTileKeys - 1) / kTileKeys;
        for (int j = 0; j < n; ++j, ++k) {
          const int st = k & 1;
          if (!wait_relaxed(bar(B_V_FULL + st), (k >> 1) & 1, abort) ||
              !wait_relaxed(bar(B_P_HALF + pb), round & 1, abort)) {
            failed = true;
            break;
          }
          tc_fence_after();
          const uint64_t d_v = sdesc_sw128(sbase + SM_V + st * kTileBytes, kHalf, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ts(tmem + kTmemO, tmem + pb * 128 + kk * 8, d_v + static_cast<uint64_t>(kk * (2048 >> 4)), id_pv,
                        (j > 0 || kk > 0) ? 1u : 0u);
          if (!wait_relaxed(bar(B_P_FULL + pb), round & 1, abort)) {
            failed = true;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 4; kk < 8; ++kk)
            mma_bf16_ts(tmem + kTmemO, tmem + pb * 128 + kk * 8, d_v + static_cast<uint64_t>(kk * (2048 >> 4)), id_pv, 1u);
          mma_commit(bar(B_PV_DONE + pb));
          if (++pb == 3) {
            pb = 0;
            ++round;
          }
        }
      }
      if (failed) raise_abort(abort, 0x100000);
      mma_commit(bar(B_DRAIN));
      int never = 0;
      mbar_wait(bar(B_DRAIN), 0, &never);
    } else if (warp == 22 && lane == 0) {
      // here, by a warp without work: ahead of the roles, the load would add its latency to
      // every launch (decode of one page 28.6 us instead of 27.4)
      *reinterpret_cast<volatile uint64_t*>(abort + 1) = g_i4_wait_limit_ns;
    }
  } else {
    // ------------------------------------------------------------ softmax
    set_max_regs<kRegsSoft, true>();
    const int wg = warp >> 2;  // its tiles are wg, wg + 3, ...: buffer wg
    const int r = threadIdx.x & 127, wq = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t t_o = tmem + kTmemO + lane_base, t_s = tmem + wg * 128 + lane_base;
    float* m_sh = reinterpret_cast<float*>(smem + SM_M);
    const int before = wg ? wg - 1 : 2;  // group of the tile before
    uint32_t kt0 = 0;     // number of the unit's first tile
    uint32_t round = 0;   // of the group's tiles
    int j = wg;           // the group's next tile, from the unit's first
    bool failed = false;
    auto row_buf = [&](int iu) { return reinterpret_cast<float*>(smem + SM_ROW + (iu & 1) * kRowBuf); };
    // Group 2's threads: row r of the next unit's Q.  Its scaling is found after the
    // group's first tile of the unit, while the thread would wait for its next S (which
    // also brings the row near); once every S of the unit has run, the row goes to
    // shared memory.
    int q_for = -1;                 // the unit that the following is of
    const uint4* q_src = nullptr;   // its row, if it has one
    float q_scale = 1.f, q_sl2 = a.sl2 * kI4Unscale;
    auto prepare_q = [&](int u) {
      if (u >= u1) return;
      const I4Unit& un = a.units[u];
      q_for = u;
      q_src = nullptr;
      if (r >= un.rows) return;
      const int R = un.row0 + r, t = div_g(R, a.g_inv);
      q_src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<int64_t>(un.q_first + t) * a.Hq + (g) * G + R - t * G) * kHeadDim);
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
      // never zero: it multiplies infinite references
      q_sl2 = fmaxf(a.sl2 * kI4Unscale * __uint_as_float(static_cast<uint32_t>(127 - kexp) << 23), 1.2e-38f);
    };
    auto put_q = [&](int u, int iu) {
      if (q_for != u) prepare_q(u);
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
    if (wg == 2 && u0 < u1) put_q(u0, 0);
    int iu = 0;
    for (int u = u0; u < u1 && !failed; ++u, ++iu) {
      const I4Unit& un = a.units[u];
      const int rows = un.rows, n_keys = un.n_keys;
      const int n = (n_keys + kTileKeys - 1) / kTileKeys;
      const bool valid = r < rows, warp_valid = wq * 32 < rows;
      const int R = un.row0 + r, tok = div_g(R, a.g_inv);
      const int limit = valid ? min(n_keys, a.q_plen[un.q_first + tok] - un.key0) : n_keys;
      const int limit_min = __reduce_min_sync(0xffffffffu, limit);
      if (!__all_sync(0xffffffffu, wait(bar(B_Q_FULL), iu & 1, abort))) {
        failed = true;
        break;
      }
      const float sl2 = row_buf(iu)[r];
      if (wg < 2) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_E_IN));
      }
      const int j0 = j;
      float m_run = -INFINITY, l_run = 0.f;     // the reference last used here, the sum against it
      for (; j < n; j += 3, ++round) {
        // A tile that opens a unit: the last epilogue must have read O before P V
        // overwrites it, and the references before this tile's take their place.
        if (j == 0 && wg > 0 && iu > 0 && !__all_sync(0xffffffffu, wait(bar(B_O_FREE), (iu - 1) & 1, abort))) {
          failed = true;
          break;
        }
        // the reference of the tile before, long there when S of this one is
        float m_old = -INFINITY;
        const uint32_t kt_before = kt0 + j - 1;
        if (j > 0) {
          if (!__all_sync(0xffffffffu, wait(bar(B_M_FULL + before), (kt_before / 3) & 1, abort))) {
            failed = true;
            break;
          }
          m_old = m_sh[before * 128 + r];
        }
        if (!__all_sync(0xffffffffu, wait_relaxed(bar(B_S_FULL + wg), round & 1, abort))) {
          failed = true;
          break;
        }
        tc_fence_after();
        // keys [0, vis) of the tile are visible to the row, [0, vis_min) to the warp's rows
        const int vis = limit - j * kTileKeys, vis_min = limit_min - j * kTileKeys;
        auto mask32 = [&](int c, uint32_t (&v)[32]) {
          const int left = vis - c * 32;
          if (left < 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i >= left) v[i] = 0xff800000u;
          }
        };
        float mx = -INFINITY;
        if (warp_valid) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v0[32];
            tmem_ld32(t_s + c * 32, v0);
            tmem_wait_ld();
            if (vis_min < c * 32 + 32) {
              // masked scores go back, for the second pass (the whole warp stores)
              mask32(c, v0);
              __syncwarp();
              tmem_st32(t_s + c * 32, v0);
              tmem_wait_st();
            }
            float m4[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; i += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) m4[k] = max3f(m4[k], __uint_as_float(v0[i + k]), __uint_as_float(v0[i + 4 + k]));
            mx = fmaxf(max3f(m4[0], m4[1], m4[2]), m4[3]);
          }
        }
        const bool grow = valid && (mx - m_old) * sl2 > kPSlack;  // what Q's buffer held in other rows asks for no rescaling
        const float m_new = grow ? mx : m_old;
        m_sh[wg * 128 + r] = m_new;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_M_FULL + wg));
        if (warp_valid) {
          if (m_new != m_run) {
            l_run *= m_run == -INFINITY ? 0.f : fast_exp2((m_run - m_new) * sl2);
            m_run = m_new;
          }
          if (j > 0 && __any_sync(0xffffffffu, grow)) {
            // O holds sums against the old reference: rescale once P V of the tile before
            // has run (the one before it on that barrier had when S of that tile was issued)
            const float alpha = grow ? fast_exp2((m_old - mx) * sl2) : 1.f;  // 0 while m_old is -inf
            if (!__all_sync(0xffffffffu, wait_relaxed(bar(B_PV_DONE + before), (kt_before / 3) & 1, abort))) {
              failed = true;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t v[32];
              tmem_ld32(t_o + c * 32, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
              tmem_st32(t_o + c * 32, v);
            }
            tmem_wait_st();
          }
          const float m_use = m_run == -INFINITY ? 0.f : m_run;
          const uint64_t sl2x2 = f2pack(sl2, sl2), negm = f2pack(-m_use, -m_use), shift = f2pack(kPShift, kPShift);
          uint64_t l2[2] = {0, 0};
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32], pk[16];
            tmem_ld32(t_s + c * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float x0, x1;
              f2unpack(fma2(add2(f2pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), negm), sl2x2, shift), x0, x1);
              x0 = fast_exp2(x0);
              x1 = fast_exp2(x1);
              l2[(i >> 1) & 1] = add2(l2[(i >> 1) & 1], f2pack(x0, x1));
              pk[i >> 1] = pack_f16x2(x0, x1);
            }
            // over columns of S that this loop has read
            tmem_st16(t_s + c * 16, pk);
            if (c == 1) {
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(B_P_HALF + wg));
              __syncwarp();
            }
          }
          float l4[4];
          f2unpack(l2[0], l4[0], l4[1]);
          f2unpack(l2[1], l4[2], l4[3]);
          l_run += (l4[0] + l4[1]) + (l4[2] + l4[3]);
          tmem_wait_st();
        } else if (lane == 0) {
          mbar_arrive(bar(B_P_HALF + wg));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P_FULL + wg));
        if (wg == 2 && j == j0) prepare_q(u + 1);
      }
      if (failed) break;
      const uint32_t last = kt0 + n - 1;
      kt0 += n;
      j -= n;
      if (wg > 0) {
        // not before group 0 is through with the unit before: it follows these
        // barriers one phase at a time
        if (iu > 0 && !__all_sync(0xffffffffu, wait(bar(B_O_FREE), (iu - 1) & 1, abort))) {
          failed = true;
          break;
        }
        float* ml = row_buf(iu) + (2 * wg - 1) * 128 + r;
        ml[0] = m_run;
        ml[128] = l_run;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_ML_FULL));
        if (wg == 2 && u + 1 < u1) {
          // Q is free once the unit's last S has run (its barrier cannot move on before
          // the next Q is out), and Q_FULL once the other groups have seen it
          if (!__all_sync(0xffffffffu, wait(bar(B_E_IN), iu & 1, abort)) ||
              !__all_sync(0xffffffffu, wait_relaxed(bar(B_S_FULL + last % 3), (last / 3) & 1, abort))) {
            failed = true;
            break;
          }
          put_q(u + 1, iu + 1);
        }
        continue;
      }
      // The other groups have handed over all their P; the last P V's commit covers all
      // before it (the one before it on that barrier had run when the last S was issued).
      if (!__all_sync(0xffffffffu, wait(bar(B_ML_FULL), iu & 1, abort)) ||
          !__all_sync(0xffffffffu, wait_relaxed(bar(B_PV_DONE + last % 3), (last / 3) & 1, abort))) {
        failed = true;
        break;
      }
      tc_fence_after();
      if (warp_valid) {
        // O is against the last tile's reference, the largest one
        const float* ml = row_buf(iu) + 128 + r;
        const float m1 = ml[0], l1 = ml[128], m2 = ml[256], l2 = ml[384];
        const float M = max3f(m_run, m1, m2);
        // Without a reference the sum is zero, or NaN where all that the group's rows saw
        // were NaN scores, which no maximum shows: it has to reach L.
        auto part = [&](float m, float l) { return m == -INFINITY ? l : l * fast_exp2((m - M) * sl2); };
        const float L = part(m_run, l_run) + part(m1, l1) + part(m2, l2);
        const bool any = !(L == 0.f);  // NaN counts
        const float inv = any ? kI4Unscale / L : 0.f;
        const int64_t row = un.part + static_cast<int64_t>(tok) * a.Hq + (g) * G + R - tok * G;
        float* dst = a.part_o + row * kHeadDim;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(t_o + c * 32, v);
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
        if (valid) {
          a.part_lse[row] = any ? fmaf(M, sl2, -kPShift) + __log2f(L) : -INFINITY;
          for (int k = 1; k <= un.n_pre; ++k) a.part_lse[row + k * un.pre_stride] = -INFINITY;
        }
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

int launch_i4_prefix_tc(const I4Args& a, int32_t n_groups, cudaStream_t s, std::string* err) {
  if (n_groups <= 0) return PADOC_OK;
  cudaError_t e = cudaFuncSetAttribute(prefix_i4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) {
    *err = std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e);
    return PADOC_ERR_CUDA;
  }
  // the roles draw on the registers that the block starts with
  static const int regs = [] {
    cudaFuncAttributes f{};
    return cudaFuncGetAttributes(&f, prefix_i4_kernel) == cudaSuccess ? f.numRegs : 0;
  }();
  if (regs < kRegsLaunch) {
    *err = "the i4 prefix kernel was built for " + std::to_string(regs) + " registers a thread";
    return PADOC_ERR_CUDA;
  }
  prefix_i4_kernel<<<n_groups * a.Hkv, kThreads, kSmemBytes, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) {
    *err = std::string("i4 prefix launch: ") + cudaGetErrorString(e);
    return PADOC_ERR_CUDA;
  }
  return PADOC_OK;
}

int set_i4_wait_limit(uint64_t ns) {
  const unsigned long long v = ns;
  return cudaMemcpyToSymbol(g_i4_wait_limit_ns, &v, sizeof(v)) == cudaSuccess ? PADOC_OK : PADOC_ERR_CUDA;
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

// Cross entropy of a large vocabulary and its gradient, without the logits in memory
// (sm_103a: tcgen05 on pairs of CTAs, TMEM, TMA).
//
// Rows h [n, D], weights w [V, D] (bf16), a target t a row:
//   x = h w^T,  lse = log sum_v exp(x_v),  loss = lse - x_t
//   G = d_loss (exp(x - lse) - onehot(t)),  dh = G w,  dw = G^T h
// Products accumulate in f32; maxima, sums, lse and loss are f32.  G is rounded to bf16
// once, since the products that follow take bf16 operands: with the rounding of the
// gradients themselves that is 2^-8 relative twice (up to 128 rows G has two bf16 parts).
// dh is summed over pieces in f32.
//
// Rows without a target take no part: the others are gathered first (lm_rows_kernel), and
// the number of them stays on the device, where every kernel here reads it.  A page's
// prefix has no targets, so that is most of the work saved, and whatever padded rows hold
// cannot reach a gradient.
//
// lm_kernel: persistent pairs of CTAs (two SMs share an MMA of 256 x 256 x 16: each holds
// half of A's rows, half of B's, and its half of the accumulator's rows).  A 128 x 256
// tile of one CTA would read 96 bytes a cycle of operands from L2, more than an SM
// gets; a pair's tile takes 64.  Units are drawn from a counter.  Kinds of unit:
//   REC  x of 256 rows and R tiles of 256 words.  Forward: running maximum and sum of a
//        row, written once a unit.  Backward: G in bf16 for a piece of the vocabulary.
//   DH   dh (256 rows x 256 dims) += G w over a piece, or a part of it when rows are few
//   DW   dw (256 words x 256 dims) = G^T h over all rows
// A backward launch runs DH and DW of one piece and REC of the next side by side: long
// units first, the short ones fill what is left, so no launch ends in a half-empty wave.
// G lives in two buffers of a piece each.
//
// Roles of a CTA (352 threads): warps 0-7 epilogue (TMEM lanes 32 (w % 4), columns
// 128 (w / 4) of the tile), warp 8 TMA producer; of the pair's first CTA, warp 9 issues
// the products and warp 10 draws the units (of the second, it passes on that they were
// read).  Shared memory: a ring of six
// stages of 64 k (A 128 rows, B 128 rows, 16 KB each).  TMEM: two accumulators.
// Barriers that both CTAs use live in the first: a stage is full when both CTAs' copies
// are in; an accumulator is free when both have read it.  The commit of a stage's
// products frees it in both.
//
// Every wait is bounded.  A role that gives up raises its CTA's abort flag and the device
// error word; the others leave their loops, the issuer commits once more and waits for
// that, copies in flight get a thousand times their latency to land, and the CTAs meet
// before TMEM is released.
//
// What bounds it.  Many rows: the tensor cores.  16384 rows, 14746 of them with a target,
// 151936 words, D = 1024: lm_kernel<forward> 2.30 ms, 2.0 PFLOP/s; a backward launch, three
// products of a piece of 19200 words, 0.92 ms, 1.9 PFLOP/s (tensor pipe 92 % busy on 4096
// rows); back to back the power limit makes that 2.5 and 8.4 ms.  Copies then run at 54
// bytes a cycle and SM, which is what they reach without products too.  Few rows: reading
// the weights, and latency.  One row, 151936 words: 54 to 57 us for 311 MB of weights (a plain
// read of them takes 57).  397 rows, 32003 words, D = 896: forward 33 us, of which 15 are
// products (four rounds of tiles, the last a third full), 4 the gathering of rows, 3 until
// the first stage is there, 3 from the last one to the end and 3 the join; backward 90.
// Steps on the way, 16384 rows and 397 rows, forward and backward together (ms, us):
//   first right kernel 11.3, 169
//   a tile leaves TMEM at once, before it is worked on, packed arithmetic 11.0, 137
//   units worked out by the thread that draws them, which is a warp of its own 10.7, 132
//   "read" signalled by an arrival that does not wait for the thread's stores 10.6, 120
//   (as a release at cluster scope, which does: one row's forward 71 us instead of 63)
// Tried without gain: copies of a row tile's rows that exist in boxes of 32 (10 % slower),
// another k to start with for each tile, waits without acquire in the issuer, a ring of
// eleven smaller stages for few rows, the first words asked for ahead of the rows, dw stored
// from registers by lines instead of by TMA, the next unit taken ahead by the producer.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <string>

#include "../../include/padoc.h"
#include "padoc_internal.h"
#include "ptx_sm103.cuh"

namespace padoc {

__device__ unsigned int g_lm_err;
// Longest time one wait of lm_kernel may take before it gives up (nanoseconds of the global
// timer); settable for tests, and part of each launch's arguments.
static std::atomic<uint64_t> g_wait_limit_ns{ptx::kWaitLimitNs};

namespace {

using namespace ptx;

constexpr int kThreads = 352;
constexpr int kEpiWarps = 8;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kDrawWarp = 10;
constexpr int kLongUnit = 32;  // stages; see the drawing warp
constexpr int kOperand = 16384;  // 128 rows of 64 k, or 64 k of 128, bf16
constexpr int kStages = 6;
constexpr int kStage = 2 * kOperand;  // A, then B
constexpr int kURing = 4;
constexpr int kOut = 4096;  // an epilogue warp's 32 rows of 64 values on their way out
constexpr int SM_OUT = kStages * kStage;
constexpr int SM_BAR = SM_OUT + kEpiWarps * kOut;
enum {
  B_FULL = 0,                   // +stage: both CTAs' copies have landed (first CTA)
  B_EMPTY = B_FULL + kStages,   // +stage: the stage's products have run
  B_ACC_FULL = B_EMPTY + kStages,   // +accumulator (2)
  B_ACC_FREE = B_ACC_FULL + 2,      // +accumulator (2), count 16: both CTAs' epilogues (first CTA)
  B_U_FULL = B_ACC_FREE + 2,        // +slot: the ring's slot holds a unit
  B_U_FREE = B_U_FULL + kURing,     // +slot, count 11: all readers have it (first CTA)
  B_U_READ = B_U_FREE + kURing,     // +slot, count 9: the second CTA's readers have it (there)
  B_DRAIN = B_U_READ + kURing,
  N_BARS
};
constexpr int SM_UNIT = (SM_BAR + N_BARS * 8 + 15) / 16 * 16;  // unit ring
constexpr int SM_MISC = SM_UNIT + kURing * 32;   // TMEM address, abort flag, units that the producer has begun
constexpr int kSmemBytes = SM_MISC + 16 + 1024;   // and room to align the ring
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kUReaders = 1 + kEpiWarps;  // of a CTA, but for the issuer: its producer and epilogue

// ---------------------------------------------------------------- pairs of CTAs
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrivals at a shared::cluster address.  The first says that an accumulator has been read,
// by loads that the caller has waited for.  It does not wait for the caller's stores to
// global memory (which a release at cluster scope does, about a microsecond a time).
__device__ __forceinline__ void arrive_read(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// What the caller read from or wrote to either CTA's shared memory comes before it, and what
// others of its CTA did before they arrived at a barrier that the caller waited for.
__device__ __forceinline__ void arrive_released(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, int a, int b, int c, int d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ int4 ld_shared_v4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for a phase; false when `limit` nanoseconds ran out or another role of the CTA gave
// up.  CLUSTER: what the other CTA did before it arrived comes before what follows.
template <bool CLUSTER>
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  const auto is_over = [&] { return CLUSTER ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
  if (is_over()) return true;
  const uint64_t t0 = global_timer();
  while (true) {
    for (int i = 0; i < 32; ++i)
      if (is_over()) return true;
    if (*abort) return false;
    if (global_timer() - t0 > limit) return false;
  }
}
// A copy into this CTA that counts on a barrier of the pair's first.
__device__ __forceinline__ void tma_pair_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the products issued so far have run.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  const uint16_t both = 3;
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(both)
      : "memory");
}

// Kernels of a call follow one another without a gap: each lets the next one's CTAs
// start where there is room and waits, past its own set-up, for the one before to end.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// A tile of 32 rows of 64 values (128 bytes, swizzled) out of shared memory; what lies
// outside the tensor is not written.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ---------------------------------------------------------------- units
enum { END = -1, REC = 0, DH = 1, DW = 2 };
struct Unit {
  int kind, m, n, tiles, k0, nkb, part;  // tile row, first tile column and their number; k blocks from k0
};

// Roundings of G average out over many rows; of a few, each shows in dw.  Up to kTwice rows
// with a target G is held in two bf16 parts: they fill half of a row tile, so its other
// half takes the same rows and what the first rounding left over, at no further product's
// cost but a step of dw's sum.  (dw of one row: 2^-8 of its values off by two roundings at
// worst, now by its own.)
constexpr int kTwice = 128;

struct Counts {
  bool twice;
  int rows, mt, dh, dw, rec_groups, all;
};
template <bool FWD>
__device__ __forceinline__ Counts counts(const LmArgs& a) {
  Counts c;
  c.rows = *a.n_rows;
  c.twice = !FWD && c.rows <= kTwice;
  c.mt = (c.rows + 255) / 256;
  c.dh = a.dh ? c.mt * a.d_tiles * a.splits : 0;
  c.dw = a.dw ? ((a.g_cols + 255) / 256) * a.d_tiles : 0;
  c.rec_groups = (((a.rec_cols + 255) / 256) + a.run - 1) / a.run;
  c.all = c.dh + c.dw + c.mt * c.rec_groups;
  return c;
}
__device__ __forceinline__ Unit unit_of(const LmArgs& a, const Counts& c, int u) {
  Unit x;
  x.tiles = 1;
  x.k0 = 0;
  x.part = 0;
  if (u >= c.all) {
    x.kind = END;
    return x;
  }
  if (u < c.dh) {  // the dims of a row tile side by side: they share G
    x.kind = DH;
    x.n = u % a.d_tiles;
    u /= a.d_tiles;
    x.part = u % a.splits;
    x.m = u / a.splits;
    const int kb = (a.g_cols + 63) / 64, each = (kb + a.splits - 1) / a.splits;
    x.k0 = min(x.part * each, kb);
    x.nkb = min(each, kb - x.k0);
    return x;
  }
  u -= c.dh;
  if (u < c.dw) {
    x.kind = DW;
    x.n = u % a.d_tiles;
    x.m = u / a.d_tiles;
    x.nkb = (c.rows + 63) / 64 * (c.twice ? 2 : 1);
    return x;
  }
  u -= c.dw;  // all rows of a few words, then the next words: the weights are read once
  x.kind = REC;
  x.m = u % c.mt;
  const int g = u / c.mt;
  x.n = g * a.run;
  x.tiles = min(a.run, (a.rec_cols + 255) / 256 - x.n);
  x.nkb = a.k_blocks;
  return x;
}

// A unit goes to the roles worked out: its divisions would stall each of them.
__device__ __forceinline__ void publish(uint32_t slot, const Unit& x) {  // a shared::cluster address
  st_cluster_v4(slot, x.kind, x.m, x.n, x.tiles);
  st_cluster_v4(slot + 16, x.k0, x.nkb, x.part, 0);
}
__device__ __forceinline__ Unit taken(uint32_t slot) {
  const int4 a = ld_shared_v4(slot), b = ld_shared_v4(slot + 16);
  return Unit{a.x, a.y, a.z, a.w, b.x, b.y, b.z};
}

__device__ __forceinline__ void give_up(volatile int* abort, unsigned site) {
  *abort = 1;
  atomicOr(&g_lm_err, site);
}

__device__ __forceinline__ uint4 pack8(const uint32_t* w) {
  return make_uint4(pack_bf16x2(__uint_as_float(w[0]), __uint_as_float(w[1])),
                    pack_bf16x2(__uint_as_float(w[2]), __uint_as_float(w[3])),
                    pack_bf16x2(__uint_as_float(w[4]), __uint_as_float(w[5])),
                    pack_bf16x2(__uint_as_float(w[6]), __uint_as_float(w[7])));
}

// A row's 128 logits of words from `word` into its running maximum and sum; its target's
// into *picked.  The maximum comes off before log2(e) multiplies: its own exponential is 1
// and a sum whose maximum stays is kept as it is, so the sum is that of exp(x - maximum) at
// any size of the logits.  (Taken off as the rounded product m log2(e), in one fma, the sum
// is a factor of up to 2^(|m| 2^-24) off, once more each tile.)
__device__ __forceinline__ void reduce_tile(uint32_t (&v)[2][64], int word, int V, int target, float& top, float& sum,
                                            float* picked) {
  if (word + 128 > V) {
#pragma unroll
    for (int i = 0; i < 128; ++i)
      if (word + i >= V) v[i >> 6][i & 63] = 0xff800000u;
  }
  float m[4] = {top, top, top, top};
#pragma unroll
  for (int i = 0; i < 64; ++i)
    m[i & 3] = max3f(m[i & 3], __uint_as_float(v[i >> 5][2 * (i & 31)]), __uint_as_float(v[i >> 5][2 * (i & 31) + 1]));
  const float t = fmaxf(max3f(m[0], m[1], m[2]), m[3]);
  // all -inf so far: any finite reference keeps the exponentials at zero
  const float ref = t == -INFINITY ? 0.f : t;
  const uint64_t scale = f2pack(kLog2e, kLog2e), less = f2pack(-ref, -ref);
  uint64_t s[4];
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const uint64_t y = mul2(
        add2(f2pack(__uint_as_float(v[i >> 5][2 * (i & 31)]), __uint_as_float(v[i >> 5][2 * (i & 31) + 1])), less), scale);
    float lo, hi;
    f2unpack(y, lo, hi);
    const uint64_t e = f2pack(fast_exp2(lo), fast_exp2(hi));
    s[i & 3] = i < 4 ? e : add2(s[i & 3], e);
  }
  float lo, hi;
  f2unpack(add2(add2(s[0], s[1]), add2(s[2], s[3])), lo, hi);
  sum = fmaf(sum, fast_exp2((top - ref) * kLog2e), lo + hi);
  top = t;
  // last, so that the target has arrived
  const int hit = target - word;
  if (hit >= 0 && hit < 128) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < 128; ++i)
      if (hit == i) x = __uint_as_float(v[i >> 6][i & 63]);
    *picked = x;
  }
}

// G of a row's 128 words from `word`, bf16 (or what that rounding leaves of it), to `out`,
// the second 64 `block` on; zero from word V on.  As above, lse comes off first: of a sure
// target, whose logit is nearly lse, the difference is exact.
__device__ __forceinline__ void gradient_tile(const uint32_t (&v)[2][64], int word, int V, int target, float lse,
                                              float d_loss, bool rest, __nv_bfloat16* out, int64_t block) {
  const uint64_t scale = f2pack(kLog2e, kLog2e), less = f2pack(-lse, -lse), by = f2pack(d_loss, d_loss);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int hit = target - word - 32 * q;
    uint32_t g[16];
    if (rest || __any_sync(0xffffffffu, (hit >= 0 && hit < 32) || word + 32 * q + 32 > V)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float p[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          p[k] = fast_exp2((__uint_as_float(v[q >> 1][32 * (q & 1) + 2 * i + k]) - lse) * kLog2e);
          if (hit == 2 * i + k) p[k] -= 1.f;
          p[k] = word + 32 * q + 2 * i + k < V ? p[k] * d_loss : 0.f;
        }
        g[i] = pack_bf16x2(p[0], p[1]);
        if (rest)
          g[i] = pack_bf16x2(p[0] - __uint_as_float(g[i] << 16), p[1] - __uint_as_float(g[i] & 0xffff0000u));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float lo, hi;
        f2unpack(mul2(add2(f2pack(__uint_as_float(v[q >> 1][32 * (q & 1) + 2 * i]),
                                  __uint_as_float(v[q >> 1][32 * (q & 1) + 2 * i + 1])),
                           less),
                      scale),
                 lo, hi);
        f2unpack(mul2(f2pack(fast_exp2(lo), fast_exp2(hi)), by), lo, hi);
        g[i] = pack_bf16x2(lo, hi);
      }
    }
    __nv_bfloat16* to = out + (q >> 1) * block + 32 * (q & 1);
    st_global_v8(to, g);
    st_global_v8(to + 16, g + 8);
  }
}

template <bool FWD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    lm_kernel(const __grid_constant__ LmArgs a, const __grid_constant__ CUtensorMap m_hk,
              const __grid_constant__ CUtensorMap m_wk, const __grid_constant__ CUtensorMap m_hm,
              const __grid_constant__ CUtensorMap m_wm, const __grid_constant__ CUtensorMap m_gk,
              const __grid_constant__ CUtensorMap m_gm, const __grid_constant__ CUtensorMap m_wo) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* sptr = smem_raw + (sbase - smem_u32(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  auto bar = [&](int i) { return sbase + SM_BAR + 8u * i; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sptr + SM_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(sptr + SM_MISC + 4);
  volatile uint32_t* begun = reinterpret_cast<volatile uint32_t*>(sptr + SM_MISC + 8);

  if (threadIdx.x == 0) {
    for (int i = 0; i < N_BARS; ++i) {
      const int count = (i >= B_ACC_FREE && i < B_ACC_FREE + 2)       ? 2 * kEpiWarps
                        : (i >= B_U_FREE && i < B_U_FREE + kURing) ? kUReaders + 2
                        : (i >= B_U_READ && i < B_U_READ + kURing) ? kUReaders
                                                                   : 1;
      mbar_init(bar(i), count);
    }
    *abort = 0;
    *begun = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp)
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + SM_MISC), "r"(512)
                 : "memory");
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_previous();
  const Counts c = counts<FWD>(a);

  // A unit has been read: said within the CTA; the second CTA's draw warp passes it on.
  const int unit_read = rank == 0 ? B_U_FREE : B_U_READ;

  if (warp == kProducerWarp) {
    if (lane == 0) {
      const uint32_t full0 = in_cta(bar(B_FULL), 0);
      uint32_t k = 0, uk = 0;  // stages and units so far
      while (true) {
        const int slot = uk % kURing;
        if (!wait<true>(bar(B_U_FULL + slot), (uk / kURing) & 1, abort, a.wait_limit)) {
          give_up(abort, 2u);
          break;
        }
        const Unit x = taken(sbase + SM_UNIT + 32 * slot);
        mbar_arrive(bar(unit_read + slot));
        *begun = ++uk;
        if (x.kind == END) break;
        bool ok = true;
        for (int t = 0; t < x.tiles && ok; ++t) {
          for (int j = 0; j < x.nkb; ++j, ++k) {
            const int s = k % kStages;
            if (!wait<false>(bar(B_EMPTY + s), ((k / kStages) & 1) ^ 1, abort, a.wait_limit)) {
              give_up(abort, 4u);
              ok = false;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(bar(B_FULL + s), 2 * kStage);
            const uint32_t sa = sbase + s * kStage, sb = sa + kOperand, full = full0 + 8u * s;
            int kk = (x.k0 + j) * 64;
            if (x.kind == REC) {
              tma_pair_2d(sa, &m_hk, full, kk, x.m * 256 + 128 * rank);
              tma_pair_2d(sb, &m_wk, full, kk, a.rec_v0 + (x.n + t) * 256 + 128 * rank);
            } else if (!FWD && x.kind == DH) {
              tma_pair_2d(sa, &m_gk, full, 0, (x.k0 + j) * a.g_rows + x.m * 256 + 128 * rank);
              tma_pair_2d(sb, &m_wm, full, x.n * 256 + 128 * rank, a.g_v0 + kk);
              tma_pair_2d(sb + kOperand / 2, &m_wm, full, x.n * 256 + 128 * rank + 64, a.g_v0 + kk);
            } else if (!FWD) {
              const int block = 4 * x.m + 2 * rank;  // of 64 words
              // the second parts' rows
              if (c.twice && j >= x.nkb / 2) kk += kTwice - 64 * (x.nkb / 2);
              tma_pair_2d(sa, &m_gm, full, 0, block * a.g_rows + kk);
              tma_pair_2d(sa + kOperand / 2, &m_gm, full, 0, (block + 1) * a.g_rows + kk);
              tma_pair_2d(sb, &m_hm, full, x.n * 256 + 128 * rank, kk);
              tma_pair_2d(sb + kOperand / 2, &m_hm, full, x.n * 256 + 128 * rank + 64, kk);
            }
          }
        }
        if (!ok) break;
      }
    }
    __syncwarp();
  } else if (warp == kDrawWarp) {
    // Draws units, works them out and publishes them to both CTAs, as far ahead as the ring
    // goes: a draw takes about as long as four stages.  Behind a long unit it waits until
    // the producer has begun that one, so that what is left at the end goes to whoever is free.
    if (lane == 0 && rank == 0) {
      int next = blockIdx.x / 2;  // the first without a draw
      for (uint32_t uk = 0;; ++uk) {
        const int slot = uk % kURing;
        const Unit x = unit_of(a, c, next);
        if (!wait<true>(bar(B_U_FREE + slot), ((uk / kURing) & 1) ^ 1, abort, a.wait_limit)) {
          give_up(abort, 1u);
          break;
        }
        for (uint32_t r = 0; r < 2; ++r) {
          publish(in_cta(sbase + SM_UNIT + 32 * slot, r), x);
          arrive_released(in_cta(bar(B_U_FULL + slot), r));
        }
        if (x.kind == END) break;
        if (x.nkb * x.tiles > kLongUnit) {
          const uint64_t t0 = global_timer();
          while (*begun <= uk && !*abort && global_timer() - t0 < a.wait_limit) __nanosleep(100);
        }
        next = gridDim.x / 2 + atomicAdd(a.counter, 1);
      }
    } else if (lane == 0) {
      for (uint32_t uk = 0;; ++uk) {
        const int slot = uk % kURing;
        const uint32_t phase = (uk / kURing) & 1;
        if (!wait<true>(bar(B_U_FULL + slot), phase, abort, a.wait_limit)) {
          give_up(abort, 256u);
          break;
        }
        if (taken(sbase + SM_UNIT + 32 * slot).kind == END) break;  // its slot is not written again
        if (!wait<false>(bar(B_U_READ + slot), phase, abort, a.wait_limit)) {
          give_up(abort, 512u);
          break;
        }
        arrive_released(in_cta(bar(B_U_FREE + slot), 0));
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (lane == 0 && rank == 0) {
      uint32_t k = 0, uk = 0, tile = 0;
      bool ok = true;
      while (ok) {
        const int slot = uk % kURing;
        if (!wait<true>(bar(B_U_FULL + slot), (uk / kURing) & 1, abort, a.wait_limit)) {
          give_up(abort, 8u);
          break;
        }
        const Unit x = taken(sbase + SM_UNIT + 32 * slot);
        mbar_arrive(bar(unit_read + slot));
        ++uk;
        if (x.kind == END) break;
        const bool a_mn = x.kind == DW, b_mn = x.kind != REC;
        const uint32_t idesc = idesc_bf16_f32(256, 256, a_mn, b_mn);
        // K-major steps 16 k by 32 bytes of a row; MN-major by 16 rows of 128 bytes, with
        // the operand's second 64 columns 8 KB further on
        const uint64_t da = sdesc_sw128(sbase, a_mn ? kOperand / 2 : 16, 1024);
        const uint64_t db = sdesc_sw128(sbase + kOperand, b_mn ? kOperand / 2 : 16, 1024);
        const uint32_t step_a = (a_mn ? 2048 : 32) >> 4, step_b = (b_mn ? 2048 : 32) >> 4;
        for (int t = 0; t < x.tiles && ok; ++t, ++tile) {
          const int acc = tile & 1;
          if (!wait<false>(bar(B_ACC_FREE + acc), ((tile >> 1) & 1) ^ 1, abort, a.wait_limit)) {
            give_up(abort, 16u);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + 256 * acc;
          for (int j = 0; j < x.nkb; ++j, ++k) {
            const int s = k % kStages;
            if (!wait<false>(bar(B_FULL + s), (k / kStages) & 1, abort, a.wait_limit)) {
              give_up(abort, 32u);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t off = static_cast<uint64_t>((s * kStage) >> 4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_pair(d, da + off + i * step_a, db + off + i * step_b, idesc, (j | i) != 0);
            commit_pair(bar(B_EMPTY + s));
          }
          if (ok) commit_pair(bar(B_ACC_FULL + acc));
        }
      }
      if (!ok || *abort) {  // nothing may still run when TMEM is released
        commit_pair(bar(B_DRAIN));
        const uint64_t t0 = global_timer();
        while (!mbar_try_wait(bar(B_DRAIN), 0) && global_timer() - t0 < kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + 128 * half;
    const int r_in = 128 * rank + 32 * quarter + lane;  // the thread's row of the tile
    uint32_t uk = 0, tile = 0;
    bool ok = true;
    while (ok) {
      const int slot = uk % kURing;
      if (!__all_sync(0xffffffffu, wait<true>(bar(B_U_FULL + slot), (uk / kURing) & 1, abort, a.wait_limit))) {
        give_up(abort, 64u);
        break;
      }
      const Unit x = taken(sbase + SM_UNIT + 32 * slot);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(unit_read + slot));
      ++uk;
      if (x.kind == END) break;
      const int row = x.m * 256 + r_in;
      const int place = c.twice ? row & (kTwice - 1) : row;  // among the rows with a target
      const bool has_row = place < c.rows;
      int target = -1;
      float lse = 0.f, d_loss = 0.f;
      if (x.kind == REC && has_row) {
        target = a.targets[place];
        if (!FWD) {
          lse = a.lse[place];
          d_loss = a.d_loss[place];
        }
      }
      float top = -INFINITY, sum = 0.f;  // forward: the row's running maximum and sum
      for (int t = 0; t < x.tiles; ++t, ++tile) {
        const int acc = tile & 1;
        if (!__all_sync(0xffffffffu, wait<false>(bar(B_ACC_FULL + acc), (tile >> 1) & 1, abort, a.wait_limit))) {
          give_up(abort, 128u);
          ok = false;
          break;
        }
        tc_fence_after();
        // all of the warp's values, so that the accumulator is free before they are worked on
        uint32_t v[2][64];
        tmem_ld64(t_lane + 256 * acc, v[0]);
        tmem_ld64(t_lane + 256 * acc + 64, v[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_read(in_cta(bar(B_ACC_FREE + acc), 0));
        const int col = (x.n + t) * 256 + 128 * half;  // of the piece, or of dims
        if (FWD) {
          reduce_tile(v, col, a.V, target, top, sum, a.picked + row);
        } else if (x.kind == REC) {
          gradient_tile(v, a.rec_v0 + col, has_row ? a.V : 0, target, lse, d_loss,
                        c.twice && rank == 1, a.g_out + (static_cast<int64_t>(col / 64) * a.g_rows + row) * 64, static_cast<int64_t>(a.g_rows) * 64);
        } else if (x.kind == DH) {
          if (!has_row) continue;
          if (x.nkb == 0) {
#pragma unroll
            for (int i = 0; i < 128; ++i) v[i >> 6][i & 63] = 0u;
          }
          float* sums = a.acc + (static_cast<int64_t>(x.part) * a.acc_rows + row) * a.acc_ld + col;
          const bool finish = a.finish && !c.twice;
          __nv_bfloat16* out = a.dh + (finish ? static_cast<int64_t>(a.rows[row]) * a.D + col : 0);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint32_t* w = &v[i >> 3][8 * (i & 7)];
            if (a.add) {
              const float4 o = reinterpret_cast<const float4*>(sums)[2 * i], z = reinterpret_cast<const float4*>(sums)[2 * i + 1];
              w[0] = __float_as_uint(__uint_as_float(w[0]) + o.x);
              w[1] = __float_as_uint(__uint_as_float(w[1]) + o.y);
              w[2] = __float_as_uint(__uint_as_float(w[2]) + o.z);
              w[3] = __float_as_uint(__uint_as_float(w[3]) + o.w);
              w[4] = __float_as_uint(__uint_as_float(w[4]) + z.x);
              w[5] = __float_as_uint(__uint_as_float(w[5]) + z.y);
              w[6] = __float_as_uint(__uint_as_float(w[6]) + z.z);
              w[7] = __float_as_uint(__uint_as_float(w[7]) + z.w);
            }
            if (!finish)
              st_global_v8(sums + 8 * i, w);
            else if (col + 8 * i < a.D)
              reinterpret_cast<uint4*>(out)[i] = pack8(w);
          }
        } else {
          // 32 words of 64 dims at a time, through shared memory
          const uint32_t out = sbase + SM_OUT + warp * kOut;
          const int first = a.g_v0 + x.m * 256 + 128 * rank + 32 * quarter;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (lane == 0) store_read();  // the copy before has left the buffer
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 w = x.nkb ? pack8(&v[h][8 * i]) : make_uint4(0, 0, 0, 0);
              st_shared_v4(out + lane * 128 + ((i ^ (lane & 7)) << 4), w.x, w.y, w.z, w.w);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && col + 64 * h < a.D && first < a.V) tma_store_2d(&m_wo, out, col + 64 * h, first);
          }
        }
      }
      if (FWD && ok && has_row)
        a.part[static_cast<int64_t>(row) * a.part_ld + 2 * (x.n / a.run) + half] = make_float2(top, sum);
    }
    if (!FWD && lane == 0) store_done();
    __syncwarp();
  }

  if (*abort) {  // copies in flight: they take microseconds
    const uint64_t t0 = global_timer();
    while (global_timer() - t0 < 5000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  cluster_sync();
}

// ---------------------------------------------------------------- rows with a target
// The rows with a target side by side, in order, with what the epilogues ask of them, and
// zeros up to the next multiple of 64 (dw sums over rows in steps of 64).  The others get
// their zeros here.  A target of V or more is no word: its row's loss is NaN and it takes
// no part.
//
// A CTA takes a run of rows, a warp K of them at a time (one where rows are few, so that
// they spread over the GPU).  Where they go depends on all targets before them, which every
// CTA counts for itself: n / 256 reads a thread, which take less time than a launch of
// their own would up to some 10^5 rows, and the CTAs are at most kRowCtas to bound them.
constexpr int kRowThreads = 256, kRowCtas = 512;
template <int K>
__global__ void __launch_bounds__(kRowThreads) lm_rows_kernel(const LmRows a) {
  __shared__ int s_all[kRowThreads / 32], s_before[kRowThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * a.rows_cta;
  auto word = [&](int32_t t) { return static_cast<uint32_t>(t) < static_cast<uint32_t>(a.V); };
  int all = 0, before = 0;
#pragma unroll 8
  for (int i = threadIdx.x; i < a.n; i += kRowThreads) {
    const int is = word(a.targets[i]);
    all += is;
    before += i < first ? is : 0;
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) {
    s_all[warp] = all;
    s_before[warp] = before;
  }
  __syncthreads();
  all = before = 0;
#pragma unroll
  for (int i = 0; i < kRowThreads / 32; ++i) {
    all += s_all[i];
    before += s_before[i];
  }
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.heads; i += kRowThreads) a.head[i] = i == 0 ? all : 0;
  constexpr int kGroup = 8 * K;
  for (int64_t g = first; g < first + a.rows_cta && g < a.n; g += kGroup) {
    const int t = lane < kGroup && g + lane < a.n ? a.targets[g + lane] : -1;
    const uint32_t who = __ballot_sync(0xffffffffu, word(t));
    if (warp == 0 && lane < kGroup && g + lane < a.n) {
      if (word(t)) {
        const int at = before + __popc(who & ((1u << lane) - 1));
        a.rows[at] = static_cast<int32_t>(g) + lane;
        a.t_out[at] = t;
        if (a.lse_out) {
          a.lse_out[at] = a.lse[g + lane];
          a.d_out[at] = a.d_loss[g + lane];
        }
      } else if (!a.lse_out) {
        a.loss[g + lane] = t < 0 ? 0.f : __uint_as_float(0x7fffffffu);
        a.lse[g + lane] = 0.f;
      }
    }
    const uint4* src[K];
    uint4* dst[K];
    const int64_t again = a.lse_out && all <= kTwice ? static_cast<int64_t>(kTwice) * a.vecs : 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int r = K * warp + k;
      const int64_t i = g + r;
      src[k] = nullptr;
      dst[k] = a.dh && i < a.n ? a.dh + i * a.vecs : nullptr;
      if (who >> r & 1) {
        src[k] = a.h + i * a.h_vecs;
        dst[k] = a.out + static_cast<int64_t>(before + __popc(who & ((1u << r) - 1))) * a.vecs;
      }
    }
#pragma unroll 2
    for (int j = lane; j < a.vecs; j += 32) {
      uint4 v[K];
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = src[k] ? src[k][j] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (dst[k]) {
          dst[k][j] = v[k];
          if (again && src[k]) dst[k][again + j] = v[k];
        }
    }
    before += __popc(who);
  }
  const int64_t pad = static_cast<int64_t>(-all & 63) * a.vecs;
  for (int64_t j = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; j < pad; j += static_cast<int64_t>(gridDim.x) * kRowThreads)
    for (int k = 0; k < (a.lse_out && all <= kTwice ? 2 : 1); ++k)
      a.out[(static_cast<int64_t>(all) + k * kTwice) * a.vecs + j] = make_uint4(0, 0, 0, 0);
}

// lse and loss of a row from its partial maxima and sums, which lie side by side.
// THREADS a row: a warp, or, of many partial results (few rows), four.
constexpr int kJoinThreads = 128;
template <int THREADS>
__global__ void __launch_bounds__(kJoinThreads) lm_join_kernel(const float2* __restrict__ part, int32_t parts,
                                                               const float* __restrict__ picked,
                                                               const int32_t* __restrict__ rows,
                                                               const int32_t* __restrict__ head, float* __restrict__ loss,
                                                               float* __restrict__ lse) {
  __shared__ float s_max[kJoinThreads / 32], s_sum[kJoinThreads / 32];
  wait_for_previous();
  constexpr bool kOne = THREADS == 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = threadIdx.x % THREADS;
  const int row = blockIdx.x * (kJoinThreads / THREADS) + threadIdx.x / THREADS;
  if (row >= *head) return;
  part += static_cast<int64_t>(row) * parts;
  constexpr int kAhead = 4;
  float m = -INFINITY, l = 0.f;
  for (int p0 = me; p0 < parts; p0 += kAhead * THREADS) {
    float2 x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      x[i] = p0 + i * THREADS < parts ? part[p0 + i * THREADS] : make_float2(-INFINITY, 0.f);
    float t = m;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) t = fmaxf(t, x[i].x);
    const float ref = t == -INFINITY ? 0.f : t;
    // a NaN logit is in its sum: fmaxf drops it from the maximum
    l *= fast_exp2((m - ref) * kLog2e);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) l += x[i].y * fast_exp2((x[i].x - ref) * kLog2e);
    m = t;
  }
  float t = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
  if (!kOne) {
    if (lane == 0) s_max[warp] = t;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) t = fmaxf(t, s_max[i]);
  }
  const float ref = t == -INFINITY ? 0.f : t;
  l *= fast_exp2((m - ref) * kLog2e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (!kOne) {
    if (lane == 0) s_sum[warp] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) l += s_sum[i];
  }
  if (me == 0) {
    const float over = logf(l);  // of lse over the largest logit
    const int32_t at = rows[row];
    lse[at] = t + over;
    // not lse - picked: where the target is the largest, and the loss small, this cancels nothing
    loss[at] = (t - picked[row]) + over;
  }
}

// dh of few rows: the parts of the vocabulary added up, in their order, and both parts of
// G.  `done`: dh is there already, but where G has two parts.
// GROUPS of 256 threads share a row's parts.
template <int GROUPS>
__global__ void __launch_bounds__(256 * GROUPS) lm_finish_kernel(const float* __restrict__ acc, int64_t acc_rows,
                                                                   int32_t acc_ld, int32_t splits,
                                                                   const int32_t* __restrict__ rows,
                                                                   const int32_t* __restrict__ head, int32_t D, bool done,
                                                                   __nv_bfloat16* __restrict__ dh) {
  __shared__ float4 s_sum[GROUPS][256];
  wait_for_previous();
  const int row = blockIdx.x, count = *head, lane = threadIdx.x & 255, group = threadIdx.x >> 8;
  const bool twice = count <= kTwice;
  if (row >= count || (done && !twice)) return;
  const int64_t at = rows[row];
  for (int c0 = 0; c0 < D; c0 += 1024) {
    const int col = c0 + 4 * lane;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < D) {
      const float* x = acc + static_cast<int64_t>(row) * acc_ld + col;
#pragma unroll 8
      for (int p = group; p < splits; p += GROUPS) {
        const float4 y = *reinterpret_cast<const float4*>(x + p * acc_rows * acc_ld);
        const float4 z = twice ? *reinterpret_cast<const float4*>(x + (p * acc_rows + kTwice) * acc_ld)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
        s = make_float4(s.x + (y.x + z.x), s.y + (y.y + z.y), s.z + (y.z + z.z), s.w + (y.w + z.w));
      }
    }
    if (group) s_sum[group][lane] = s;
    __syncthreads();
    if (!group && col < D) {
#pragma unroll
      for (int i = 1; i < GROUPS; ++i) {
        const float4 y = s_sum[i][lane];
        s = make_float4(s.x + y.x, s.y + y.y, s.z + y.z, s.w + y.w);
      }
      *reinterpret_cast<uint2*>(dh + at * D + col) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    }
    __syncthreads();
  }
}

int make_map(EncodeTiledFn enc, CUtensorMap* m, const void* ptr, int64_t cols, int64_t rows, int64_t ld, int box_rows,
             std::string* err) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, one[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r == CUDA_SUCCESS) return PADOC_OK;
  *err = "cuTensorMapEncodeTiled failed (" + std::to_string(static_cast<int>(r)) + ")";
  return PADOC_ERR_CUDA;
}

// A launch that may begin its set-up while the kernel before it on the stream, which is
// one of this file's, still runs.
template <class... P, class... A>
int launch_after(void (*kernel)(P...), unsigned grid, int threads, int smem, cudaStream_t s, const char* what,
                 std::string* err, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  if (e == cudaSuccess) return PADOC_OK;
  *err = std::string(what) + " launch: " + cudaGetErrorString(e);
  return PADOC_ERR_CUDA;
}

enum { M_HK, M_WK, M_HM, M_WM, M_GK, M_GM, M_WO, N_MAPS };

template <bool FWD>
int launch_gemm(const LmArgs& args, const CUtensorMap* m, cudaStream_t s, std::string* err) {
  LmArgs a = args;
  a.wait_limit = g_wait_limit_ns.load(std::memory_order_relaxed);
  // an attribute of the current device's copy of the kernel
  const cudaError_t e = cudaFuncSetAttribute(lm_kernel<FWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) {
    *err = std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e);
    return PADOC_ERR_CUDA;
  }
  return launch_after(lm_kernel<FWD>, num_sms() / 2 * 2, kThreads, kSmemBytes, s, "lm_kernel", err, a, m[M_HK], m[M_WK],
                      m[M_HM], m[M_WM], m[M_GK], m[M_GM], m[M_WO]);
}

int launch_rows(const LmCall& l, const LmPlan& p, uint8_t* ws, bool backward, cudaStream_t s, std::string* err) {
  LmRows a{};
  a.h = static_cast<const uint4*>(l.h);
  a.h_vecs = l.h_stride / 8;
  a.targets = l.targets;
  a.n = l.n;
  a.V = l.V;
  a.vecs = l.D / 8;
  a.heads = p.heads;
  a.head = reinterpret_cast<int32_t*>(ws + p.head);
  a.rows = reinterpret_cast<int32_t*>(ws + p.rows);
  a.t_out = reinterpret_cast<int32_t*>(ws + p.t);
  a.out = reinterpret_cast<uint4*>(ws + p.hc);
  a.loss = l.loss;
  a.lse = l.lse;
  if (backward) {
    a.lse_out = reinterpret_cast<float*>(ws + p.lse);
    a.d_loss = l.d_loss;
    a.d_out = reinterpret_cast<float*>(ws + p.d);
    a.dh = static_cast<uint4*>(l.dh);
  }
  const bool few = l.n <= 8 * kRowCtas;
  const int64_t group = few ? 8 : 32, groups = (static_cast<int64_t>(l.n) + group - 1) / group;
  a.rows_cta = (groups + kRowCtas - 1) / kRowCtas * group;
  const unsigned grid = static_cast<unsigned>((l.n + a.rows_cta - 1) / a.rows_cta);
  if (few)
    lm_rows_kernel<1><<<grid, kRowThreads, 0, s>>>(a);
  else
    lm_rows_kernel<4><<<grid, kRowThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return PADOC_OK;
  *err = std::string("lm_rows_kernel launch: ") + cudaGetErrorString(e);
  return PADOC_ERR_CUDA;
}

}  // namespace

// Sizes of a call, from its shape alone.  The number of rows with a target is not known
// here, so everything is laid out for all of them.
LmPlan lm_plan(int32_t n, int32_t D, int32_t V, bool backward) {
  constexpr int pairs = 76;  // of a GB300
  LmPlan p{};
  const int64_t word_tiles = (static_cast<int64_t>(V) + 255) / 256, row_tiles = (static_cast<int64_t>(n) + 255) / 256;
  const int64_t d_tiles = (D + 255) / 256;
  p.n_pad = row_tiles * 256;
  // Tiles of words one after another in a REC unit: as many as leave each pair eight units
  // to draw, so that drawing and (forward) partial results cost little, and the units end
  // together.
  p.run = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(16, word_tiles * row_tiles / (8 * pairs))));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += (bytes + 255) / 256 * 256;
    return r;
  };
  if (!backward) {
    p.heads = 2;
    p.head = take(p.heads * sizeof(int32_t));
    p.rows = take(n * sizeof(int32_t));
    p.t = take(n * sizeof(int32_t));
    p.hc = take(static_cast<size_t>(p.n_pad) * D * 2);
    p.parts = static_cast<int32_t>(2 * ((word_tiles + p.run - 1) / p.run));
    p.part = take(static_cast<size_t>(p.parts) * p.n_pad * sizeof(float2));
    p.picked = take(static_cast<size_t>(p.n_pad) * sizeof(float));
    p.bytes = at;
    return p;
  }
  // A piece of the vocabulary is what 640 MB of G hold, or 4096 words where rows are many:
  // long enough that a piece's products dwarf the f32 sums of dh which go through memory
  // once a piece.
  const int64_t cap = std::max<int64_t>(16, (640ll << 20) / (2 * 256 * p.n_pad));
  p.pieces = static_cast<int32_t>((word_tiles + cap - 1) / cap);
  p.piece_tiles = static_cast<int32_t>((word_tiles + p.pieces - 1) / p.pieces);
  p.pieces = static_cast<int32_t>((word_tiles + p.piece_tiles - 1) / p.piece_tiles);
  // Few rows leave few dh tiles with a long sum each: the sum is cut until every pair has
  // a part of one.
  p.splits = static_cast<int32_t>(
      std::max<int64_t>(1, std::min<int64_t>(pairs / (row_tiles * d_tiles), p.piece_tiles)));
  p.heads = 2 + p.pieces;
  p.head = take(p.heads * sizeof(int32_t));
  p.rows = take(n * sizeof(int32_t));
  p.t = take(n * sizeof(int32_t));
  p.lse = take(n * sizeof(float));
  p.d = take(n * sizeof(float));
  p.hc = take(static_cast<size_t>(p.n_pad) * D * 2);
  p.acc_ld = static_cast<int32_t>(d_tiles * 256);
  p.acc = take(static_cast<size_t>(p.pieces > 1 || p.splits > 1 ? p.splits * p.n_pad : 2 * kTwice) * p.acc_ld * sizeof(float));
  p.g_bytes = static_cast<size_t>(p.n_pad) * p.piece_tiles * 512;
  p.g = take(p.g_bytes * (p.pieces > 1 ? 2 : 1));
  p.bytes = at;
  return p;
}

int launch_lm_loss(const LmCall& l, void* ws_, cudaStream_t s, std::string* err) {
  const LmPlan p = lm_plan(l.n, l.D, l.V, false);
  uint8_t* ws = static_cast<uint8_t*>(ws_);
  EncodeTiledFn enc = get_encode_fn(err);
  if (!enc) return PADOC_ERR_CUDA;
  CUtensorMap m[N_MAPS]{};
  int rc = make_map(enc, &m[M_HK], ws + p.hc, l.D, p.n_pad, l.D, 128, err);
  if (!rc) rc = make_map(enc, &m[M_WK], l.w, l.D, l.V, l.w_stride, 128, err);
  if (rc) return rc;
  rc = launch_rows(l, p, ws, false, s, err);
  if (rc) return rc;
  int32_t* head = reinterpret_cast<int32_t*>(ws + p.head);
  LmArgs a{};
  a.n_rows = head;
  a.counter = head + 1;
  a.rows = reinterpret_cast<int32_t*>(ws + p.rows);
  a.targets = reinterpret_cast<int32_t*>(ws + p.t);
  a.D = l.D;
  a.V = l.V;
  a.k_blocks = (l.D + 63) / 64;
  a.d_tiles = (l.D + 255) / 256;
  a.run = p.run;
  a.splits = 1;
  a.rec_cols = l.V;
  a.part = reinterpret_cast<float2*>(ws + p.part);
  a.part_ld = p.parts;
  a.picked = reinterpret_cast<float*>(ws + p.picked);
  rc = launch_gemm<true>(a, m, s, err);
  if (rc) return rc;
  const bool many = p.parts > 256;
  return launch_after(many ? lm_join_kernel<kJoinThreads> : lm_join_kernel<32>,
                      many ? static_cast<unsigned>(l.n) : static_cast<unsigned>((l.n + 3) / 4), kJoinThreads, 0, s,
                      "lm_join_kernel", err, a.part, p.parts, a.picked, a.rows, head, l.loss, l.lse);
}

int launch_lm_loss_bwd(const LmCall& l, void* ws_, cudaStream_t s, std::string* err) {
  const LmPlan p = lm_plan(l.n, l.D, l.V, true);
  uint8_t* ws = static_cast<uint8_t*>(ws_);
  EncodeTiledFn enc = get_encode_fn(err);
  if (!enc) return PADOC_ERR_CUDA;
  const int32_t g_ld = p.piece_tiles * 256;
  CUtensorMap m[N_MAPS]{}, gk[2], gm[2];
  int rc = make_map(enc, &m[M_HK], ws + p.hc, l.D, p.n_pad, l.D, 128, err);
  if (!rc) rc = make_map(enc, &m[M_WK], l.w, l.D, l.V, l.w_stride, 128, err);
  if (!rc) rc = make_map(enc, &m[M_HM], ws + p.hc, l.D, p.n_pad, l.D, 64, err);
  if (!rc) rc = make_map(enc, &m[M_WM], l.w, l.D, l.V, l.w_stride, 64, err);
  if (!rc && l.dw) rc = make_map(enc, &m[M_WO], l.dw, l.D, l.V, l.D, 32, err);
  for (int i = 0; i < (p.pieces > 1 ? 2 : 1) && !rc; ++i) {
    // G lies in blocks of 64 words, all rows of a block together: what a copy takes of it,
    // for either product, is then one run of bytes
    rc = make_map(enc, &gk[i], ws + p.g + i * p.g_bytes, 64, p.n_pad * (g_ld / 64), 64, 128, err);
    if (!rc) rc = make_map(enc, &gm[i], ws + p.g + i * p.g_bytes, 64, p.n_pad * (g_ld / 64), 64, 64, err);
  }
  if (rc) return rc;
  rc = launch_rows(l, p, ws, true, s, err);
  if (rc) return rc;
  int32_t* head = reinterpret_cast<int32_t*>(ws + p.head);
  LmArgs a{};
  a.n_rows = head;
  a.rows = reinterpret_cast<int32_t*>(ws + p.rows);
  a.targets = reinterpret_cast<int32_t*>(ws + p.t);
  a.D = l.D;
  a.V = l.V;
  a.k_blocks = (l.D + 63) / 64;
  a.d_tiles = (l.D + 255) / 256;
  a.run = p.run;
  a.splits = p.splits;
  a.lse = reinterpret_cast<float*>(ws + p.lse);
  a.d_loss = reinterpret_cast<float*>(ws + p.d);
  a.acc = reinterpret_cast<float*>(ws + p.acc);
  a.acc_rows = p.n_pad;
  a.acc_ld = p.acc_ld;
  a.g_rows = static_cast<int32_t>(p.n_pad);
  // launch i: the gradients of piece i - 1 and G of piece i
  for (int i = 0; i <= p.pieces; ++i) {
    const int done = i - 1;
    a.counter = head + 1 + i;
    a.dh = nullptr;
    a.dw = nullptr;
    if (done >= 0) {
      a.dh = static_cast<__nv_bfloat16*>(l.dh);
      a.dw = static_cast<__nv_bfloat16*>(l.dw);
      a.g_v0 = done * g_ld;
      a.g_cols = static_cast<int32_t>(std::min<int64_t>(g_ld, static_cast<int64_t>(l.V) - a.g_v0));
      a.add = done > 0;
      a.finish = i == p.pieces && p.splits == 1;
    }
    a.rec_v0 = i * g_ld;
    a.rec_cols = i < p.pieces ? static_cast<int32_t>(std::min<int64_t>(g_ld, static_cast<int64_t>(l.V) - a.rec_v0)) : 0;
    const int from = done > 0 ? done & 1 : 0;
    a.g_out = reinterpret_cast<__nv_bfloat16*>(ws + p.g + (i < p.pieces && i & 1 ? p.g_bytes : 0));
    m[M_GK] = gk[from];
    m[M_GM] = gm[from];
    rc = launch_gemm<false>(a, m, s, err);
    if (rc) return rc;
  }
  if (l.dh) {
    const bool done = p.splits == 1;
    const bool few = l.n <= kTwice;
    return launch_after(few ? lm_finish_kernel<4> : lm_finish_kernel<1>,
                        static_cast<unsigned>(done ? std::min(l.n, kTwice) : l.n), few ? 1024 : 256, 0, s, "lm_finish_kernel", err, a.acc, a.acc_rows,
                        static_cast<int32_t>(a.acc_ld), p.splits, a.rows, head, l.D, done, static_cast<__nv_bfloat16*>(l.dh));
  }
  return PADOC_OK;
}

void set_lm_wait_limit(uint64_t ns) { g_wait_limit_ns.store(ns ? ns : ptx::kWaitLimitNs); }

int read_and_clear_lm_error(cudaStream_t s, unsigned* word) {
  const unsigned zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_lm_err, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && *word) e = cudaMemcpyToSymbolAsync(g_lm_err, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? PADOC_OK : PADOC_ERR_CUDA;
}

}  // namespace padoc

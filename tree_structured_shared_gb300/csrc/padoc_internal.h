// Structures shared by the host library and the kernel launchers.
#pragma once
#include <cstdint>
#include <string>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace padoc {

// ---------------------------------------------------------------- forward
// A query segment: packed positions [q_start, q_start + q_len) that share one
// ordered list of key/value segments kvsegs[kv_first .. kv_first + kv_count).
struct QSeg {
  int32_t q_start, q_len, kv_first, kv_count;
};
// Keys [start, start + len); when causal, a query at packed position t sees
// only keys <= t (all keys of the segment before the query are visible).
struct KVSeg {
  int32_t start, len, causal, pad;
};
// One query tile: tile_tokens consecutive tokens of one query segment.
struct FwdItem {
  int32_t qseg, tile_start;
  int32_t n_tiles;  // key tiles the tile's walk visits (every kernel role counts on it)
  // the query segment's fields and its first key segment, copied so a
  // kernel reads one record per unit
  int32_t q_end, kv_first, kv_count, tile_last, pad;
  KVSeg kv0;
};

constexpr int kTileKeys = 128;  // keys per K/V tile
constexpr int kTileRows = 128;  // MMA M: query rows (tokens x heads of a GQA group)
constexpr int kMaxChunkTiles = 40;  // prefix pass: key tiles in one chunk of a page's prefix, at most
constexpr int kHeadDim = 128;   // d of the tensor-core path
constexpr int kI4UnitBytes = 1152;  // one (block, kv head) of a 4-bit pool, K or V (kv_i4.cuh)

struct FwdPlan {
  const QSeg* qsegs;
  const KVSeg* kvsegs;
  const FwdItem* items;
  int32_t n_items;
  int32_t group;        // Hq / Hkv
  int32_t tile_tokens;  // kTileRows / group
};

struct FwdArgs {
  FwdPlan plan;
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  int64_t T;
  int32_t Hq, Hkv, d;
  float scale;
};

// ---------------------------------------------------------------- backward
// Key-stationary work of the backward: keys are cut into tiles on a global
// kTileKeys grid; an entry lists queries [q_lo, q_hi) of one query segment
// that see keys [k_lo, k_hi) of the tile through one key segment (when
// causal, a query at t sees only keys <= t).  Entries of one tile cover
// disjoint (query, key) pairs, so their contributions simply add.
struct BwdEntry {
  int32_t k_lo, k_hi, causal, q_lo, q_hi, pad[3];
};
struct BwdItem {
  int32_t k_start, k_len, e_first, e_count;
};
struct BwdPlan {
  const BwdItem* items;
  const BwdEntry* entries;
  int32_t n_items;
};

struct BwdArgs {
  FwdPlan fwd;  // query-stationary work (dQ), as in the forward
  BwdPlan bwd;  // key-stationary work (dK, dV)
  const void* q;
  const void* k;
  const void* v;
  const void* o;
  const float* lse;   // [Hq, T]
  const void* dout;   // [T, Hq, d]
  void* dq;
  void* dk;
  void* dv;
  float* delta;       // workspace [Hq, T]: rowsum(dO * O)
  int32_t* work;      // workspace: unit counter of the dK/dV pass (zeroed by its launcher)
  bool have_delta = false;  // the row sums are in delta already, and the unit counters are zero
  // parts of the key tiles' queries, the first part of each tile (and the end), and room
  // for their sums: null where the tiles are not cut
  BwdPlan split{};
  const int32_t* split_first = nullptr;
  float* parts = nullptr;
  int64_t T;
  int32_t Hq, Hkv, d;
  float scale;
};

// ---------------------------------------------------------------- decode
struct DecPage {
  int32_t seq;           // block-table row holding the shared prefix
  int32_t P;             // prefix tokens any branch of the page sees
  int32_t q_first;       // first query row of the page
  int32_t nq;            // query rows of the page
  int32_t item_base;     // first prefix item of the page
  int32_t n_chunks;      // prefix chunks
  int32_t chunk_tokens;  // tokens per chunk (multiple of kTileKeys)
  int32_t row_tiles;     // ceil(nq * group / kTileRows)
};
struct DecItem {
  int32_t page, tile, chunk;
  int32_t rows;      // valid rows of this row tile
  int32_t row_base;  // partial row index of head 0; head g adds g * rows
  // fused verify: the branches whose query rows the tile holds, and the
  // first query token of the first of them
  int32_t b_first, b_count, tok_lo;
  int32_t n_tiles;  // key tiles of the unit (prefix chunk; fused verify: + own suffixes + query block)
  int32_t pad[3];
};
struct DecBranch {
  int32_t page, seq;
  int32_t prefix_len;  // shared prefix tokens this branch sees
  int32_t own_len;     // own cached tokens
  int32_t n_shared;    // leading blocks of seq that belong to the prefix
  int32_t q_first, q_len;
  int32_t q_in_page;   // index of its first query among its page's queries
};

struct DecodeArgs {
  const DecPage* pages;
  const DecItem* items;
  const DecBranch* branches;
  const int32_t* q_plen;  // [nq] prefix tokens visible to each query row
  const int32_t* q_branch;  // [nq] branch of each query row
  const int32_t* table;   // device block table [max_seqs][max_bps]
  int32_t max_bps;
  int32_t n_pages, n_items, n_branches, nq;
  int32_t Hq, Hkv, group, d;
  float scale;
  const void* q;
  const void* k_new;
  const void* v_new;
  const uint16_t* tree_bits;
  void* o;
  float* lse;
  float* part_o;    // [rows][d] f32 normalised partial outputs of the prefix pass
  float* part_lse;  // [rows] f32
  int32_t* work;    // unit counter of the tensor-core passes (zeroed by their launchers)
  const void* k_pool;
  const void* v_pool;
  int64_t num_blocks;
};

// ---------------------------------------------------------------- decode over a 4-bit pool
// One kv head's work of a CTA: query rows against a run of cached keys.  Rows
// are (token, head of the group): row R is token q_first + R / G.
struct I4Unit {
  int32_t seq, blk0;       // block-table row and the place in it of the first key's block
  int32_t key0, n_keys;    // first key (prefix: its position in the page's prefix) and keys
  int32_t q_first, row0, rows;
  int32_t branch;          // own keys of this branch; -1: keys of a page's prefix
  int32_t q_len, qb_first; // query tokens of the branch when the unit takes its query block, else 0
  // own keys: prefix partial results merged here, one each pre_stride from pre; a page's
  // prefix: results behind its own, pre_stride apart, that it marks as empty
  int32_t n_pre, pad;
  int64_t pre, pre_stride; // partial rows, counted from (q_first, head 0)
  int64_t part;            // where the unit's partial rows go (as pre), or -1: write o and lse
};
// A query token whose partial results the merge kernel joins.
struct I4Merge {
  int32_t token, n_pre, n_own, pad;
  int64_t pre, pre_stride, own, own_stride;
};
struct I4Args {
  const I4Unit* units;
  const I4Merge* merges;
  const int32_t* tc_first;  // first unit of each group of CTAs of the tcgen05 kernel, and the end
  const int32_t* q_plen;  // [nq] prefix tokens visible to each query token
  const int32_t* table;
  int32_t max_bps, unit0;
  int32_t Hq, Hkv, group;
  uint32_t g_inv;  // 2^32 / group rounded up, 0 when group is 1
  float sl2;       // scale * log2(e)
  const __nv_bfloat16* q;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  const uint16_t* tree_bits;
  __nv_bfloat16* o;
  float* lse;
  float* part_o;    // [rows][d] normalised
  float* part_lse;  // [rows] log2 units
  const void* k_pool;
  const void* v_pool;
};

// ---------------------------------------------------------------- cache rows
// Up to 16 consecutive rows of one pool block: source / destination rows
// [row, row + n) are its slots [slot, slot + n).  slot_n = slot | n << 8; pos
// is the first row's position when the rows have no position array.
struct RowRec {
  int32_t row, block, slot_n, pos;
};
// Records of a list up to this long ride in the kernel's parameters (with the
// arguments below 4 KB).
constexpr int kInlineRecs = 224;

struct RowsArgs {
  const RowRec* recs;       // device, or null
  const RowRec* host_recs;  // host, at most kInlineRecs, or null
  // neither: the rows [seq_first, seq_first + n_rows) of one sequence's own
  // tokens, through its row of the block table (from its first own block)
  const int32_t* table_row;
  int32_t seq_first;
  int32_t n_recs;
  int64_t n_rows;
  bool i4;
  void* k_pool;
  void* v_pool;
  int32_t Hkv, Hq;
  // write
  const int32_t* positions;  // device [n_rows], or null: RowRec::pos
  const float* cos_sin;      // [position][cosines, then sines]
  int32_t rot_dim, interleaved;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t q_stride, k_stride, v_stride;  // elements between rows
  __nv_bfloat16* q_rot;
  __nv_bfloat16* k_rot;
  // gather
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
};

// ---------------------------------------------------------------- rotation of packed rows
constexpr int kRopeParts = 4;
struct RopeArgs {
  const float* cos_sin;  // [n_pos][cosines, then sines]
  const int32_t* positions;  // [n], or null: the row's index
  int64_t n;
  int32_t n_pos, rot_dim, interleaved, backward;
  int32_t heads;              // of all parts together
  int32_t slots, rows_warp;   // heads of a row that a warp holds at once, and rows (the launcher's)
  int32_t first[kRopeParts];  // first head of each part (heads: no such part)
  const void* x[kRopeParts];
  void* out[kRopeParts];
  int64_t stride[kRopeParts], out_stride[kRopeParts];  // elements between rows
};
struct RopeTableArgs {
  float* cos_sin;
  int64_t first, n_pos;
  int32_t rot_dim;
  float amplitude;
  uint64_t turns[64];  // of a pair a position, as a fraction of 2^64
};

// ---------------------------------------------------------------- 8-bit checkpoints
constexpr int kActTensors = 8;
struct ActTensor {
  void* rows;      // bf16
  int64_t stride;  // elements between rows
  uint8_t* kept;   // codes, then scales
  int64_t pieces;  // of 16 values
  uint32_t per_row;
  int32_t dense;   // rows follow one another
};
struct ActArgs {
  ActTensor t[kActTensors];
  int32_t n;
  int32_t first_block[kActTensors];
  int64_t pieces_cta;  // the launcher's
  // the tensor whose row sums with `rows` are wanted instead of its values, or -1
  int32_t sums;
  float* delta;  // [heads][T]
  int64_t T;
  uint32_t heads, head_pieces;
  int32_t* zero;  // two counters that restore_kernel zeroes, or null
};

// ---------------------------------------------------------------- cross entropy
struct LmCall {
  const void* h;
  int64_t h_stride;
  const void* w;
  int64_t w_stride;
  const int32_t* targets;
  int32_t n, D, V;
  float* loss;
  float* lse;
  const float* d_loss;
  void* dh;
  void* dw;
};
// Where things lie in a call's workspace (bytes), and how its work is cut.
struct LmPlan {
  int64_t n_pad;
  int32_t run, parts, pieces, piece_tiles, splits, heads, acc_ld;
  size_t head, rows, t, lse, d, hc, part, picked, acc, g, g_bytes, bytes;
};
struct LmRows {
  const uint4* h;
  int64_t h_vecs;  // 16-byte vectors between rows
  const int32_t* targets;
  int32_t n, V, vecs, heads;
  int64_t rows_cta;
  int32_t* head;   // number of rows with a target, then unit counters
  int32_t* rows;   // their indices
  int32_t* t_out;  // their targets
  uint4* out;      // their h
  float* loss;     // forward
  float* lse;      // forward: out, backward: in
  const float* d_loss;
  float* lse_out;  // backward: theirs
  float* d_out;
  uint4* dh;       // backward, may be null
};
struct LmArgs {
  uint64_t wait_limit;  // the launcher's
  const int32_t* n_rows;
  int32_t* counter;  // of units, zero at launch
  const int32_t* rows;     // of the rows with a target: index, target (and lse, d_loss below)
  const int32_t* targets;
  int32_t D, V;
  int32_t k_blocks, d_tiles, run, splits;
  int32_t rec_v0, rec_cols;  // words of the REC units
  int32_t g_v0, g_cols;      // words of the piece whose gradients are taken
  int32_t add, finish;       // dh: sums so far in acc; this launch writes it in bf16
  // forward
  float2* part;
  int64_t part_ld;
  float* picked;
  // backward
  const float* lse;
  const float* d_loss;
  __nv_bfloat16* g_out;  // [64 words][row][word]
  int32_t g_rows;
  float* acc;
  int64_t acc_rows, acc_ld;
  __nv_bfloat16* dh;
  __nv_bfloat16* dw;
};

// Launchers (return 0 or a PADOC_ERR_* code, message in *err).
int launch_rope_apply(RopeArgs a, int32_t dtype, int32_t d, cudaStream_t s, std::string* err);
int launch_rope_table(const RopeTableArgs& a, cudaStream_t s, std::string* err);
int launch_act(ActArgs a, bool keep, cudaStream_t s, std::string* err);
LmPlan lm_plan(int32_t n, int32_t D, int32_t V, bool backward);
int launch_lm_loss(const LmCall& l, void* ws, cudaStream_t s, std::string* err);
int launch_lm_loss_bwd(const LmCall& l, void* ws, cudaStream_t s, std::string* err);
void set_lm_wait_limit(uint64_t ns);
int read_and_clear_lm_error(cudaStream_t s, unsigned* word);
int launch_fwd_bf16(const FwdArgs& a, cudaStream_t s, std::string* err);
int launch_fwd_f32(const FwdArgs& a, cudaStream_t s, std::string* err);
int launch_decode_prefix(const DecodeArgs& a, cudaStream_t s, std::string* err);
int launch_decode_own(const DecodeArgs& a, cudaStream_t s, std::string* err);
int launch_decode_own_tc(const DecodeArgs& a, cudaStream_t s, std::string* err);
// Verify own pass with keys on the MMA's M side (Hq / Hkv of 1 or 2).
int launch_decode_own_kmajor(const DecodeArgs& a, cudaStream_t s, std::string* err);
// Verify step in one pass (plans marked fused): each (page, row tile, kv
// head) walks the prefix, the own suffixes of the branches it holds and
// their query block, and writes the final O and LSE.
int launch_decode_verify_fused(const DecodeArgs& a, cudaStream_t s, std::string* err);
int launch_kv_append(void* k_pool, void* v_pool, const int32_t* table_row, int32_t first_own,
                     int32_t n, int32_t Hkv, int32_t d, const void* k, const void* v,
                     cudaStream_t s, std::string* err);

int launch_accept(const void* logits, int64_t V, int32_t nq, const int32_t* tokens, const int32_t* parents,
                  const int32_t* q_offsets, int32_t n_branches, int32_t max_nodes, float log_tau,
                  int32_t* n_acc, int32_t* path, int32_t* free_token, cudaStream_t s, std::string* err);
// plan: device int4 per row {source row, block, slot, 0}
int launch_commit(void* k_pool, void* v_pool, const void* plan, int64_t n_rows, int32_t Hkv, const void* k,
                  const void* v, cudaStream_t s, std::string* err);

// n units of up to 8 rows from units[unit0]; warps (1, 2, 4 or 8) share each.
int launch_i4_units(const I4Args& a, int32_t unit0, int32_t n, int warps, cudaStream_t s, std::string* err);
// The same for a page's prefix and units of up to 128 rows.
int launch_i4_prefix_tc(const I4Args& a, int32_t n_groups, cudaStream_t s, std::string* err);
int read_and_clear_i4_error(cudaStream_t s, unsigned* word);
int set_i4_wait_limit(uint64_t ns);
int launch_i4_merge(const I4Args& a, int32_t n_merges, cudaStream_t s, std::string* err);
int launch_kv_write(const RowsArgs& a, cudaStream_t s, std::string* err);
int launch_kv_gather(const RowsArgs& a, cudaStream_t s, std::string* err);

int launch_bwd_core(const BwdArgs& a, int32_t dtype, cudaStream_t s, std::string* err);
int launch_bwd_delta(const BwdArgs& a, int32_t dtype, cudaStream_t s, std::string* err);
int launch_bwd_tc(const BwdArgs& a, cudaStream_t s, std::string* err);
int read_and_clear_bwd_error(cudaStream_t s, unsigned* word);

// Device error words (set by kernels that give up a bounded wait).
int read_and_clear_tc_error(cudaStream_t s, unsigned* word);
int read_and_clear_own_error(cudaStream_t s, unsigned* word);

// Driver entry point for tensor-map encoding (resolved through the runtime).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode_fn(std::string* err);
int num_sms();

// Records an error message for padoc_last_error() and returns code.
int set_error(int code, const char* fmt, ...);
int32_t pool_num_blocks(const padoc_kv_pool* pool);
// True once the pool's device block table exists (padoc_kv_pool_sync ran).
bool pool_has_device_table(const padoc_kv_pool* pool);
// PADOC_OK when the pool has no device table yet or its device is current;
// else PADOC_ERR_INVALID (message names the call).
int pool_check_device(const padoc_kv_pool* pool, const char* what);

}  // namespace padoc

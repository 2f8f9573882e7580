// Checks of the plan over a 4-bit pool, on the host: random batches are planned
// and every unit and merge record is followed.  Built by test_i4_plan.py together
// with the library's own translation unit, whose internals it reads.
//   - the units of a page's prefix cover each key once for each of its rows, and a
//     branch's own units its keys; each row's query block is taken once
//   - every partial-result row is written once, or marked as empty once, and read
//     once, by the own unit that joins it or by the merge record of its token
//   - blocks and keys stay inside the sequences, groups of CTAs inside the GPU
#include "../tree_structured_shared_gb300/csrc/host.cpp"

#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>

#define REQ(x)                                                        \
  do {                                                                \
    if (!(x)) {                                                       \
      std::printf("batch %d, line %d: %s\n", batch_no, __LINE__, #x); \
      return 1;                                                       \
    }                                                                 \
  } while (0)

namespace {

using Row = std::pair<int, int>;  // token, head of the group
using Runs = std::map<Row, std::vector<std::pair<int, int>>>;

bool covers(std::vector<std::pair<int, int>> runs, int n) {
  std::sort(runs.begin(), runs.end());
  int at = 0;
  for (const auto& r : runs) {
    if (r.first != at) return false;
    at += r.second;
  }
  return at == n;
}

int check_one(std::mt19937& rng, int batch_no, long* seen) {
  auto pick = [&](int a, int b) { return a + static_cast<int>(rng() % static_cast<unsigned>(b - a + 1)); };
  const int Hkv = pick(1, 4) * (batch_no % 7 == 0 ? 3 : 1), G = pick(1, 8), Hq = Hkv * G, n_sms = batch_no % 11 ? 152 : 7;
  padoc_kv_pool* pool = nullptr;
  REQ(padoc_kv_pool_create(&pool, nullptr, nullptr, 60000, 16, Hkv, 128, PADOC_I4, 400, 2000) == 0);
  std::unique_ptr<padoc_kv_pool, int (*)(padoc_kv_pool*)> owner(pool, padoc_kv_pool_destroy);
  const int n_pages = pick(0, batch_no % 5 == 0 ? 12 : 3);
  std::vector<int32_t> pages, branch_off{0}, branches, q_off{0};
  for (int p = 0; p < n_pages; ++p) {
    const int P = batch_no % 3 ? pick(0, 700) : pick(0, 9000);
    int32_t s;
    REQ(padoc_kv_alloc(pool, P, &s) == 0 && padoc_kv_advance(pool, s, P) == 0);
    pages.push_back(s);
    for (int b = pick(0, batch_no % 4 == 0 ? 20 : 4); b > 0; --b) {
      int32_t c;
      const int own = pick(0, 3) ? pick(0, 40) : pick(0, 3000);
      REQ(padoc_kv_fork(pool, s, pick(0, 2) ? std::max(0, P - pick(0, 20)) : pick(0, P), &c) == 0);
      REQ(padoc_kv_reserve(pool, c, own) == 0 && padoc_kv_advance(pool, c, own) == 0);
      branches.push_back(c);
      q_off.push_back(q_off.back() + (batch_no % 2 ? 1 : pick(1, 16)));
    }
    branch_off.push_back(static_cast<int32_t>(branches.size()));
  }
  padoc_decode_batch b{};
  b.n_pages = n_pages;
  b.page_seq = pages.data();
  b.branch_offsets = branch_off.data();
  b.n_branches = static_cast<int32_t>(branches.size());
  b.branch_seq = branches.data();
  b.q_offsets = q_off.data();
  DecodePlan pl;
  REQ(plan_decode(pool, &b, Hq, n_sms, &pl) == 0);
  if (b.n_branches == 0) return 0;
  const int nq = q_off.back(), first_own = pl.n_tc + pl.n_pre;
  REQ(static_cast<int>(pl.units.size()) == first_own + pl.n_own);
  if (pl.n_tc) {
    REQ(pl.tc_first.front() == 0 && pl.tc_first.back() == pl.n_tc);
    for (size_t i = 1; i < pl.tc_first.size(); ++i) REQ(pl.tc_first[i] > pl.tc_first[i - 1]);
    REQ(static_cast<int>(pl.tc_first.size()) - 1 <= std::max(1, n_sms / Hkv));
  } else {
    REQ(pl.tc_first.empty());
  }
  std::vector<int> page_of(nq), branch_of(nq), reach(n_pages, 0);
  for (int p = 0; p < n_pages; ++p)
    for (int i = branch_off[p]; i < branch_off[p + 1]; ++i)
      for (int t = q_off[i]; t < q_off[i + 1]; ++t) {
        page_of[t] = p;
        branch_of[t] = i;
        reach[p] = std::max(reach[p], pool->seqs[branches[i]].fork_len);
      }

  std::vector<int> written(pl.part_rows, 0), read(pl.part_rows, 0);
  auto mark = [&](std::vector<int>* v, int64_t base, int t, int h) {  // row (t from the base's token, h) of every kv head
    for (int g = 0; g < Hkv; ++g) {
      const int64_t r = base + static_cast<int64_t>(t) * Hq + g * G + h;
      if (r < 0 || r >= pl.part_rows) return false;
      ++(*v)[r];
    }
    return true;
  };
  Runs pre, own;
  std::map<Row, int> query_blocks;
  std::map<int, const I4Merge*> merge_of;
  for (const I4Merge& m : pl.merges) {
    REQ(!merge_of.count(m.token));
    merge_of[m.token] = &m;
  }
  int before = 1 << 30;
  for (int i = 0; i < static_cast<int>(pl.units.size()); ++i) {
    const I4Unit& u = pl.units[i];
    const Seq& s = pool->seqs[u.seq];
    const bool tc = i < pl.n_tc, is_own = i >= first_own;
    REQ((u.branch >= 0) == is_own && u.rows > 0 && u.rows <= (tc ? kTileRows : 8));
    REQ(is_own || u.n_keys > 0);
    REQ(u.key0 % (tc ? kTileKeys : 16) == 0);
    if (i == pl.n_tc || i == first_own) before = 1 << 30;
    if (!tc) {  // dealt out longest first
      REQ((u.n_keys + 15) / 16 <= before);
      before = (u.n_keys + 15) / 16;
    }
    if (u.n_keys) {
      REQ(u.blk0 == (is_own ? s.n_shared : 0) + u.key0 / 16);
      REQ(u.blk0 + (u.n_keys + 15) / 16 <= static_cast<int>(s.blocks.size()));
      REQ(u.key0 + u.n_keys <= (is_own ? s.len - s.fork_len : s.len));
    }
    if (is_own) REQ((u.part >= 0) == (merge_of.count(u.q_first) > 0));
    for (int r = u.row0; r < u.row0 + u.rows; ++r) {
      const int t = u.q_first + r / G, h = r % G;
      REQ(t < nq);
      (is_own ? own : pre)[{t, h}].push_back({u.key0, u.n_keys});
      if (is_own) {
        REQ(branch_of[t] == u.branch && branches[u.branch] == u.seq);
        if (u.q_len) {
          ++query_blocks[{t, h}];
          REQ(u.q_len == q_off[u.branch + 1] - q_off[u.branch] && u.qb_first == q_off[u.branch]);
        }
      } else {
        REQ(pages[page_of[t]] == u.seq && u.part >= 0);
      }
      if (u.part >= 0) {
        REQ(mark(&written, u.part, r / G, h));
        for (int k = 1; tc && k <= u.n_pre; ++k) REQ(mark(&written, u.part + k * u.pre_stride, r / G, h));
      } else {
        for (int k = 0; k < u.n_pre; ++k) REQ(mark(&read, u.pre + k * u.pre_stride, r / G, h));
      }
    }
    seen[tc ? 0 : is_own ? 2 : 1] += 1;
    seen[3] += tc && u.key0 > 0;
  }
  for (const I4Merge& m : pl.merges)
    for (int h = 0; h < G; ++h) {
      for (int k = 0; k < m.n_pre; ++k) REQ(mark(&read, m.pre + k * m.pre_stride, 0, h));
      for (int k = 0; k < m.n_own; ++k) REQ(mark(&read, m.own + k * m.own_stride, 0, h));
    }
  seen[4] += static_cast<long>(pl.merges.size());
  for (int64_t r = 0; r < pl.part_rows; ++r) REQ(written[r] == 1 && read[r] == 1);
  for (int t = 0; t < nq; ++t) {
    const Seq& s = pool->seqs[branches[branch_of[t]]];
    REQ(pl.q_plen[t] == s.fork_len);
    for (int h = 0; h < G; ++h) {
      REQ(covers(pre[{t, h}], reach[page_of[t]]));
      REQ(covers(own[{t, h}], s.len - s.fork_len));
      REQ((query_blocks[{t, h}] == 1));
    }
  }
  return 0;
}

}  // namespace

int main(int argc, char** argv) {
  const int n = argc > 1 ? std::atoi(argv[1]) : 1000;
  std::mt19937 rng(1);
  long seen[5] = {};
  for (int i = 0; i < n; ++i)
    if (check_one(rng, i, seen)) return 1;
  std::printf("tcgen05 %ld warp-level %ld own %ld cut %ld merges %ld\n", seen[0], seen[1], seen[2], seen[3], seen[4]);
  return 0;
}

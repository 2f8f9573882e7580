// Checks of what a tree descriptor uploads, on the host: random pages are uploaded to a device
// that is made up here, and what arrived is read back.  Built by test_tree_desc_upload.py
// together with the library's own translation unit, whose internals it reads.
//   - one allocation and one copy a device and group; a failure of either leaves nothing behind
//   - the parts of the key tiles' queries: every query of every entry once, in order, cut where
//     a query tile ends; no part empty, none above the limit; as many as sized the workspace
#include <cuda_runtime.h>

#include <cstdlib>
#include <set>

namespace made_up {
long allocs = 0, copies = 0, fail_alloc = 0, fail_copy = 0;
std::set<void*> live;
cudaError_t get_device(int* d) {
  *d = 0;
  return cudaSuccess;
}
cudaError_t set_device(int) { return cudaSuccess; }
template <class T>
cudaError_t alloc(T** p, size_t n) {
  ++allocs;
  if (fail_alloc) return cudaErrorMemoryAllocation;
  *p = static_cast<T*>(std::aligned_alloc(256, (n + 255) / 256 * 256));
  live.insert(*p);
  return cudaSuccess;
}
cudaError_t copy(void* to, const void* from, size_t n, cudaMemcpyKind) {
  ++copies;
  if (fail_copy) return cudaErrorUnknown;
  __builtin_memcpy(to, from, n);
  return cudaSuccess;
}
cudaError_t release(void* p) {
  if (!p) return cudaSuccess;
  if (!live.erase(p)) std::abort();
  std::free(p);
  return cudaSuccess;
}
}  // namespace made_up
#define cudaGetDevice made_up::get_device
#define cudaSetDevice made_up::set_device
#define cudaMalloc made_up::alloc
#define cudaMemcpy made_up::copy
#define cudaFree made_up::release
#include "../tree_structured_shared_gb300/csrc/host.cpp"

#include <cstdio>
#include <random>

#define REQ(x)                                                         \
  do {                                                                 \
    if (!(x)) {                                                        \
      std::printf("pages no. %d, line %d: %s\n", no, __LINE__, #x);    \
      return 1;                                                        \
    }                                                                  \
  } while (0)

namespace {

long cut = 0, whole = 0;  // descriptors with parts, and without

int check_parts(const padoc_tree_desc* desc, const DevPlan& p, int no) {
  REQ(p.n_sitems == count_parts(desc, p.tile_tokens));
  const int32_t most = part_tiles(desc, p.tile_tokens);
  int32_t entry = 0;  // of all parts
  REQ(p.sfirst[0] == 0 && p.sfirst[desc->bitems.size()] == p.n_sitems);
  for (size_t x = 0; x < desc->bitems.size(); ++x) {
    const BwdItem& it = desc->bitems[x];
    REQ(p.sfirst[x] < p.sfirst[x + 1]);
    int32_t e = it.e_first, q = desc->bentries[e].q_lo;
    for (int32_t i = p.sfirst[x]; i < p.sfirst[x + 1]; ++i) {
      REQ(p.sitems[i].k_start == it.k_start && p.sitems[i].k_len == it.k_len);
      REQ(p.sitems[i].e_first == entry && p.sitems[i].e_count > 0);
      int32_t tiles = 0;
      for (int32_t j = 0; j < p.sitems[i].e_count; ++j, ++entry) {
        const BwdEntry &got = p.sentries[entry], &of = desc->bentries[e];
        REQ(e < it.e_first + it.e_count);
        REQ(got.k_lo == of.k_lo && got.k_hi == of.k_hi && got.causal == of.causal);
        REQ(got.q_lo == q && got.q_hi > q && got.q_hi <= of.q_hi);
        REQ(got.q_hi == of.q_hi || (got.q_hi - of.q_lo) % p.tile_tokens == 0);
        tiles += entry_tiles(got, p.tile_tokens);
        q = got.q_hi;
        if (q == of.q_hi && ++e < it.e_first + it.e_count) q = desc->bentries[e].q_lo;
      }
      REQ(tiles > 0 && tiles <= most);
    }
    REQ(e == it.e_first + it.e_count);
  }
  return 0;
}

int check_one(std::mt19937& rng, int no) {
  auto pick = [&](int a, int b) { return a + static_cast<int>(rng() % static_cast<unsigned>(b - a + 1)); };
  const int n_pages = pick(0, no % 9 ? 3 : 8);
  std::vector<int32_t> prefix, regions, lay, con;
  for (int i = 0; i < n_pages; ++i) {
    prefix.push_back(pick(0, 3) ? pick(0, 500) : pick(0, 4000));
    regions.push_back(pick(0, no % 4 ? 6 : 40));
    for (int r = 0; r < regions.back(); ++r) {
      lay.push_back(pick(0, 12));
      con.push_back(pick(0, 3) ? pick(0, 60) : pick(0, 700));
    }
  }
  prefix.push_back(0), regions.push_back(0), lay.push_back(0), con.push_back(0);
  padoc_tree_spec spec{};
  spec.n_pages = n_pages;
  spec.prefix_len = prefix.data();
  spec.n_regions = regions.data();
  spec.layout_len = lay.data();
  spec.content_len = con.data();
  spec.order = no % 2 ? PADOC_PACK_DOCUMENT : PADOC_PACK_CANONICAL;
  padoc_tree_desc* desc = nullptr;
  REQ(padoc_tree_desc_build(&spec, &desc) == 0);
  std::unique_ptr<padoc_tree_desc, int (*)(padoc_tree_desc*)> owner(desc, padoc_tree_desc_free);
  const bool few = few_units(desc, 1);
  ++(few ? cut : whole);
  for (int i = 0; i < 5; ++i) {
    const int group = 1 << i;
    made_up::fail_alloc = no % 5 == 1;
    made_up::fail_copy = no % 5 == 2;
    if (made_up::fail_alloc || (made_up::fail_copy && desc->T > 0)) {
      const size_t had = made_up::live.size();
      REQ(padoc_tree_desc_upload(desc, group) == PADOC_ERR_CUDA);
      REQ(made_up::live.size() == had);
    }
    made_up::fail_alloc = made_up::fail_copy = 0;
    size_t before = 0, after = 0;
    const int Hkv = pick(1, 8);
    REQ(padoc_tree_attn_varlen_bwd_kept_ws_size(desc, Hkv * group, Hkv, 128, &before) == 0);
    made_up::allocs = made_up::copies = 0;
    REQ(padoc_tree_desc_upload(desc, group) == 0 && padoc_tree_desc_upload(desc, group) == 0);
    REQ(made_up::allocs == 1 && made_up::copies <= 1);
    REQ(padoc_tree_attn_varlen_bwd_kept_ws_size(desc, Hkv * group, Hkv, 128, &after) == 0 && before == after);
    DevPlan* p = nullptr;
    REQ(upload_desc(desc, group, &p) == 0 && made_up::allocs == 1);
    const auto items = build_items(desc, p->tile_tokens);
    auto same = [](const void* a, const void* b, size_t n) { return n == 0 || std::memcmp(a, b, n) == 0; };
    REQ(same(p->qsegs, desc->qsegs.data(), desc->qsegs.size() * sizeof(QSeg)));
    REQ(same(p->kvsegs, desc->kvsegs.data(), desc->kvsegs.size() * sizeof(KVSeg)));
    REQ(same(p->items, items.data(), items.size() * sizeof(FwdItem)));
    REQ(same(p->bitems, desc->bitems.data(), desc->bitems.size() * sizeof(BwdItem)));
    REQ(same(p->bentries, desc->bentries.data(), desc->bentries.size() * sizeof(BwdEntry)));
    REQ(few || p->n_sitems == 0);
    if (few && check_parts(desc, *p, no)) return 1;
    // the workspace holds every part's sums of both gradients where the parts are taken
    const bool taken = few_units(desc, Hkv) && !desc->bitems.empty();
    const size_t sums = taken ? 2 * sizeof(float) * static_cast<size_t>(p->n_sitems) * kTileKeys * Hkv * 128 : 0;
    REQ(bwd_parts_bytes(desc, Hkv * group, Hkv, 128) == sums);
    REQ(bwd_parts_bytes(desc, Hkv * group, Hkv, 64) == 0);
  }
  return 0;
}

}  // namespace

int main(int argc, char** argv) {
  std::mt19937 rng(7);
  const int n = argc > 1 ? std::atoi(argv[1]) : 500;
  for (int no = 0; no < n; ++no)
    if (check_one(rng, no)) return 1;
  if (!made_up::live.empty()) {
    std::printf("%zu allocations left\n", made_up::live.size());
    return 1;
  }
  std::printf("cut %ld whole %ld\n", cut, whole);
  return 0;
}

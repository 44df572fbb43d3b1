// Host run of the paged kernels' plans (no kernel is launched): see test_paged_host.py.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <vector>

#include "fa_paged_decode.cuh"

#define REQUIRE(x)                                                      \
  do {                                                                  \
    if (!(x)) {                                                         \
      std::printf("failed: %s (line %d)\n", #x, __LINE__);              \
      std::exit(1);                                                     \
    }                                                                   \
  } while (0)

using namespace fa;

static void bad_indices() {
  int table[6] = {0, 5, 9, 10, -1, 0x7fffffff}, status = 0;
  PagedBatch p{};
  p.table = table;
  p.num_pages = 10;
  p.max_pages = 3;
  p.page_shift = 4;
  p.B = 2;
  p.T = 20;
  p.max_q = 8;
  p.Hkv = 2;
  p.status = &status;
  REQUIRE(load_page(p, 0, 0) == 0 && load_page(p, 0, 1) == 5 && load_page(p, 0, 2) == 9 && status == 0);
  for (int i = 0; i < 3; ++i) {
    status = 0;
    REQUIRE(load_page(p, 1, i) == -1 && status == kBadPage);
  }
  struct {
    int r0, r1, len, rows, got_len, what;
  } cases[] = {{0, 3, 10, 3, 10, 0},          {0, 8, 48, 8, 48, 0},           {0, 9, 48, 0, 48, kBadRows},
               {5, 4, 48, 0, 48, kBadRows},   {-1, 2, 48, 0, 48, kBadRows},   {15, 21, 48, 0, 48, kBadRows},
               {12, 20, 49, 8, 48, kBadLength}, {0, 2, -1, 2, 0, kBadLength}, {0, 2, 0x7fffffff, 2, 48, kBadLength},
               {0, 0, 0, 0, 0, 0},            {-2147483647, 2147483647, 5, 0, 5, kBadRows}};
  for (const auto& c : cases) {
    int cu[3] = {c.r0, c.r1, 0}, lens[2] = {c.len, 0};
    p.cu_q = cu;
    p.lens = lens;
    status = 0;
    const SeqInfo s = load_seq(p, 0);
    REQUIRE(s.rows == c.rows && s.len == c.got_len && status == c.what);
    REQUIRE(s.rows == 0 || (s.row0 >= 0 && s.row0 + s.rows <= p.T));
  }
}

static void shares(std::mt19937& rng, bool whole) {
  auto pick = [&](int lo, int hi) { return lo + static_cast<int>(rng() % static_cast<unsigned>(hi - lo + 1)); };
  const int B = pick(1, 12), n_cta = pick(1, 40);
  std::vector<int> cu{0}, lens;
  for (int b = 0; b < B; ++b) {
    cu.push_back(cu.back() + pick(0, 40));
    lens.push_back(pick(0, 3) == 0 ? pick(0, 3) : pick(0, whole ? 250 : 6000));
  }
  int status = 0;
  DecodeParams p{};
  p.b.cu_q = cu.data();
  p.b.lens = lens.data();
  p.b.B = B;
  p.b.T = cu.back();
  p.b.max_q = 40;
  p.b.max_pages = 1000;
  p.b.page_shift = 4;
  p.b.num_pages = 1;
  p.b.Hkv = pick(1, 4);
  p.b.status = &status;
  p.G = pick(1, 5);
  p.tile = pick(0, 1) ? 64 : 128;
  p.rows = pick(0, 1) ? 8 : 16;
  p.max_rows = pick(0, 2) ? 1 << 30 : 48;
  p.whole = whole;
  long long total = 0;
  for (int b = 0; b < B; ++b) total += decode_units(p, decode_seq(p, b));
  const long long per = decode_per(p, total, n_cta);
  REQUIRE(per * n_cta >= total);
  auto locate = [&](int c) {
    DecodeShare s{total, per, B, 0};
    long long at = 0;
    for (int b = 0; b < B; ++b) {
      const long long u = decode_units(p, decode_seq(p, b));
      if (per * c >= at && per * c < at + u) s.b = b, s.off = per * c - at;
      at += u;
    }
    return s;
  };
  std::map<std::pair<int, int>, std::vector<int>> seen;               // (b, item): times each tile was taken
  std::map<std::pair<int, int>, std::vector<int>> parts;              // slots that hold parts of it
  std::map<int, int> slots;
  for (int c = 0; c < n_cta; ++c) {
    const DecodeShare s = locate(c);
    if (s.b >= B) continue;
    DecodeWalk w;
    w.start(p, s, c);
    do {
      REQUIRE(w.item >= 0 && w.item < w.d.items && w.t0 >= 0 && w.t0 < w.t1 && w.t1 <= w.d.tiles);
      auto& v = seen[{w.b, w.item}];
      v.resize(w.d.tiles);
      for (int t = w.t0; t < w.t1; ++t) ++v[t];
      REQUIRE(w.whole == (w.t0 == 0 && w.t1 == w.d.tiles));
      if (!w.whole) {
        const int slot = decode_slot(c, w.t0);
        REQUIRE(slot >= 0 && slot < 2 * n_cta && slots[slot]++ == 0);
        parts[{w.b, w.item}].push_back(slot);
      }
    } while (w.next(p));
  }
  long long items = 0;
  for (int b = 0; b < B; ++b) items += decode_seq(p, b).items;
  REQUIRE(static_cast<long long>(seen.size()) == items);
  for (auto& kv : seen)
    for (int n : kv.second) REQUIRE(n == 1);
  if (whole) {
    REQUIRE(parts.empty());
    return;
  }
  for (int c = 1; c < n_cta; ++c) {
    const DecodeShare s = locate(c);
    if (s.b >= B) continue;
    const DecodeCut cut = decode_cut(per, c, s.off, decode_seq(p, s.b).tiles);
    if (cut.last < c || cut.first != c - 1) continue;
    auto it = parts.find({s.b, cut.item});
    REQUIRE(it != parts.end());
    std::vector<int> want;
    for (int k = c - 1; k <= cut.last; ++k) want.push_back(decode_slot(k, k - (c - 1)));
    REQUIRE(it->second == want);
    parts.erase(it);
  }
  REQUIRE(parts.empty());  // everything that was left is joined
  REQUIRE(status == 0);
}

int main() {
  bad_indices();
  std::mt19937 rng(1);
  for (int i = 0; i < 20000; ++i) shares(rng, i % 4 == 0);
  std::printf("ok\n");
  return 0;
}

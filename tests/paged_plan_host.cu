// Host run of the paged kernels' plans (no kernel is launched): see test_paged_host.py.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <vector>

#include "fa_paged_decode.cuh"
#include "fa_paged_prefill.cuh"

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
    if (w.start(p, s, c)) do {
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
    DecodeWalk w;
    if (!w.start(p, s, c) || w.t0 == 0) continue;
    const Cut cut = cut_of(per, c, w.t0, w.d.tiles);
    REQUIRE(cut.last >= c && cut.first < c);
    if (cut.first != c - 1) continue;
    auto it = parts.find({s.b, w.item});
    REQUIRE(it != parts.end());
    std::vector<int> want;
    for (int k = c - 1; k <= cut.last; ++k) want.push_back(decode_slot(k, k - (c - 1)));
    REQUIRE(it->second == want);
    parts.erase(it);
  }
  REQUIRE(parts.empty());  // everything that was left is joined
  REQUIRE(status == 0);
}

static void many_rows(std::mt19937& rng) {
  auto pick = [&](int lo, int hi) { return lo + static_cast<int>(rng() % static_cast<unsigned>(hi - lo + 1)); };
  const int B = pick(1, 6);
  std::vector<int> cu{0}, lens;
  for (int b = 0; b < B; ++b) {
    const int q = pick(0, 3) == 0 ? pick(0, 3) : pick(0, 900);
    cu.push_back(cu.back() + q);
    lens.push_back(pick(0, 4) == 0 ? pick(0, 900) : q + pick(0, 3000));
  }
  int status = 0;
  PrefillParams p{};
  p.b.cu_q = cu.data();
  p.b.lens = lens.data();
  p.b.B = B;
  p.b.T = cu.back();
  p.b.max_q = 900;
  p.b.max_pages = 1000;
  p.b.page_shift = 4;
  p.b.num_pages = 1;
  p.b.Hkv = pick(1, 4);
  p.b.status = &status;
  p.G = pick(1, 9);
  p.min_rows = pick(0, 1) ? 32 : 200;
  p.causal = pick(0, 3) != 0;
  long long total = 0;
  std::vector<long long> units;
  for (int b = 0; b < B; ++b) {
    const PrefillSeq d = prefill_seq(p, b);
    REQUIRE((d.pairs == 0) == (static_cast<long long>(d.s.rows) * p.G <= p.min_rows));
    long long sum = 0;
    for (int k = 0; k < d.pairs; ++k) {
      REQUIRE(d.before(k) == sum);
      sum += d.count(k) + kPreItemCost;
      // a pair's rows see none but its own tiles
      const int last_row = std::min((k + 1) * kPreRows, d.s.rows * p.G) - 1;
      const int last = p.causal ? d.s.len - d.s.rows + last_row / p.G : d.s.len - 1;
      const int seen = last < 0 ? 0 : std::min(last, d.s.len - 1) / 128 + 1;
      const bool half = k == d.pairs - 1 && d.s.rows * p.G - k * kPreRows <= 128;
      REQUIRE((k == d.pairs - 1 && d.half) == half);
      REQUIRE(d.count(k) * (half ? 2 : 1) >= std::max(seen, 1));
      if (d.linear && seen > 0) REQUIRE(d.count(k) == (half ? (seen + 1) / 2 : seen));
    }
    REQUIRE(d.head_units() == sum);
    units.push_back(sum * p.b.Hkv);
    total += units.back();
  }
  const long long per = prefill_per(total);
  REQUIRE(per * kPreCtas >= total);
  auto locate = [&](int c) {
    PrefillShare s{total, per, 0, B};
    long long at = 0;
    for (int b = 0; b < B; ++b) {
      if (per * c >= at && per * c < at + units[b]) s.b = b, s.off = per * c - at;
      at += units[b];
    }
    return s;
  };
  using Item = std::vector<int>;
  std::map<Item, std::vector<int>> seen, parts;
  std::map<int, int> slots;
  for (int c = 0; c < kPreCtas; ++c) {
    const PrefillShare s = locate(c);
    if (s.b >= B) continue;
    PrefillWalk w;
    if (w.start(p, s, c, FindPairAlone{})) do {
      REQUIRE(w.p >= 0 && w.p < w.d.pairs && w.h < p.b.Hkv && w.t0 >= 0 && w.t0 < w.t1 && w.t1 <= w.n);
      for (int t = 0; t < 2; ++t) {
        const int f = w.split() ? 2 : 1, key0 = w.t0 * f, key1 = w.t1 * f;
        const int end = w.end(p, t), first = w.p * kPreRows + (w.split() ? 0 : t * kTile);
        REQUIRE(w.first() == key0 && end >= key0 && end <= key1 && (end == key0 || end * 128 < w.d.s.len + 128));
        if (first >= w.d.s.rows * p.G) REQUIRE(end == key0);
        if (w.split()) REQUIRE(w.end(p, 0) == w.end(p, 1) && w.d.s.rows * p.G - w.p * kPreRows <= 128);
        // every visible key of every row of the tile is in a tile below `end`, or in another segment
        for (int r = first; r < std::min(first + kTile, w.d.s.rows * p.G); ++r) {
          const int last = std::min(w.d.s.len - 1, p.causal ? w.d.s.len - w.d.s.rows + r / p.G : w.d.s.len - 1);
          if (last >= key0 * 128) REQUIRE(end >= std::min(key1, last / 128 + 1));
        }
      }
      auto& v = seen[{w.b, w.h, w.p}];
      v.resize(w.n);
      for (int t = w.t0; t < w.t1; ++t) ++v[t];
      if (!w.whole) {
        const int slot = decode_slot(c, w.t0);
        REQUIRE(slot >= 0 && slot < 2 * kPreCtas && slots[slot]++ == 0);
        parts[{w.b, w.h, w.p}].push_back(slot);
      }
    } while (w.next(p));
  }
  long long items = 0;
  for (int b = 0; b < B; ++b) items += static_cast<long long>(prefill_seq(p, b).pairs) * p.b.Hkv;
  REQUIRE(static_cast<long long>(seen.size()) == items);
  for (auto& kv : seen)
    for (int n : kv.second) REQUIRE(n == 1);
  for (int c = 1; c < kPreCtas; ++c) {
    const PrefillShare s = locate(c);
    if (s.b >= B) continue;
    PrefillWalk w;
    if (!w.start(p, s, c, FindPairAlone{}) || w.t0 == 0) continue;
    const Cut cut = cut_of(per, c, w.t0, w.n);
    REQUIRE(cut.last >= c && cut.first < c);
    if (cut.first != c - 1) continue;
    auto it = parts.find({s.b, w.h, w.p});
    REQUIRE(it != parts.end());
    std::vector<int> want;
    for (int k = c - 1; k <= cut.last; ++k) want.push_back(decode_slot(k, k - (c - 1)));
    REQUIRE(it->second == want);
    parts.erase(it);
  }
  REQUIRE(parts.empty());
}

static void sums() {
  for (long long m = 1; m < 12; ++m)
    for (long long a = 0; a < 9; ++a)
      for (long long b = 0; b < 60; b += 7)
        for (long long n = 0, s = 0; n < 40; ++n) {
          REQUIRE(floor_sum(n, m, a, b) == s);
          s += (a * n + b) / m;
        }
}

int main() {
  sums();
  bad_indices();
  std::mt19937 rng(1);
  for (int i = 0; i < 20000; ++i) shares(rng, i % 4 == 0);
  for (int i = 0; i < 3000; ++i) many_rows(rng);
  std::printf("ok\n");
  return 0;
}

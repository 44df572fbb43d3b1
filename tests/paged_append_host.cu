// Host run of the append's index checks (no kernel is launched): see test_paged_host.py.
#include <cstdio>
#include <cstdlib>

#include "fa_append.cuh"

#define REQUIRE(x)                                                      \
  do {                                                                  \
    if (!(x)) {                                                         \
      std::printf("failed: %s (line %d)\n", #x, __LINE__);              \
      std::exit(1);                                                     \
    }                                                                   \
  } while (0)

using namespace fa;

int main() {
  int table[3] = {0, 5, 9}, status = 0;
  PagedBatch p{};
  p.table = table;
  p.num_pages = 10;
  p.max_pages = 3;  // 48 tokens
  p.page_shift = 4;
  p.B = 1;
  p.T = 60;
  p.max_q = 50;
  p.Hkv = 2;
  p.status = &status;
  struct {
    int rows, len, got_rows, what;
  } cases[] = {{1, 1, 1, 0},           {8, 48, 8, 0},          {48, 48, 48, 0},        {1, 49, 0, kBadLength},
               {8, 49, 0, kBadLength}, {49, 49, 0, kBadLength}, {3, 0x7fffffff, 0, kBadLength}, {3, 2, 0, kBadLength},
               {1, 0, 0, kBadLength},  {1, -1, 0, kBadLength}, {2, -0x7fffffff - 1, 0, kBadLength}, {51, 48, 0, kBadRows},
               {0, 0, 0, 0},           {0, 48, 0, 0},          {0, 49, 0, kBadLength}, {0, -1, 0, kBadLength}};
  for (const auto& c : cases) {
    int cu[2] = {4, 4 + c.rows}, lens[1] = {c.len};
    p.cu_q = cu;
    p.lens = lens;
    status = 0;
    const SeqInfo s = append_seq(p, 0);
    REQUIRE(s.rows == c.got_rows && status == c.what);
    if (s.rows > 0) REQUIRE(s.row0 == 4 && s.len == c.len && s.len >= s.rows && s.len <= 48);
  }
  std::printf("ok\n");
  return 0;
}

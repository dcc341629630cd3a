// Host unit test of the cut of a batch between the row-streaming and the tiled
// base products (built with g++ under AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_base_plan.py).
#include <algorithm>
#include <cstdint>
#include <cstdio>

#include "base_plan.hpp"

#define CHECK(c)                                                        \
  do {                                                                  \
    if (!(c)) {                                                         \
      std::fprintf(stderr, "CHECK failed line %d: %s\n", __LINE__, #c); \
      return 1;                                                         \
    }                                                                   \
  } while (0)

using namespace lora;

static BatchCut cut(WKind kind, int n_proj, int32_t h_in, int32_t h_out, int32_t adapters, int32_t max_rank, int32_t n) {
  return cut_batch(BaseShape{kind, n_proj, h_in, h_out, adapters, max_rank}, n);
}

int main() {
  // ---- every token goes one way, whatever the shape; a short batch streams rows
  for (WKind kind : {WKind::kBf16, WKind::kFp8, WKind::kInt4, WKind::kTable4})
    for (int n_proj : {1, 2})
      for (int32_t h_in : {64, 768, 4096, 1 << 20})
        for (int32_t h_out : {64, 2304, 12288, 1 << 20})
          for (int32_t adapters : {0, 1, 64, 8192})
            for (int32_t rank : {1, 64})
              for (int64_t n = 0; n <= INT32_MAX; n = n * 2 + 1)
                for (int64_t m : {n, n / 256 * 256, n / 256 * 256 + 63}) {
                  if (m > INT32_MAX) continue;
                  const BatchCut c = cut(kind, n_proj, h_in, h_out, adapters, rank, static_cast<int32_t>(m));
                  CHECK(c.tiles >= 0 && c.rows >= 0 && static_cast<int64_t>(c.tiles) + c.rows == m);
                  CHECK(m > kRowsTokens || c.tiles == 0);
                  CHECK(c.rows <= kRowsMaxTokens);
                  CHECK(c.rows == 0 || c.tiles % 256 == 0);
                }

  // ---- a call without ids has no adapters: the rank that the pool's adapters may have is nothing to it
  for (WKind kind : {WKind::kBf16, WKind::kFp8, WKind::kInt4, WKind::kTable4})
    for (int n_proj : {1, 2})
      for (int32_t h_in : {256, 768, 2048, 4096, 8192})
        for (int32_t h_out : {512, 2304, 4096, 8192, 12288})
          for (int32_t n : {65, 100, 128, 200, 256, 300, 512, 777, 1000, 1500, 2048, 2111, 4096}) {
            const BatchCut a = cut(kind, n_proj, h_in, h_out, 0, 1, n), b = cut(kind, n_proj, h_in, h_out, 0, 64, n);
            CHECK(a.tiles == b.tiles && a.rows == b.rows);
          }

  // ---- the faster way of measured calls without ids (us a call on rows / on tiles)
  struct Measured {
    WKind kind;
    int n_proj;
    int32_t h_in, h_out, n;
    int rows_us, tiles_us;
  };
  const Measured m[] = {
      {WKind::kTable4, 2, 768, 2304, 256, 20, 41},    {WKind::kTable4, 2, 768, 2304, 512, 19, 42},
      {WKind::kTable4, 2, 768, 2304, 1000, 35, 44},   {WKind::kInt4, 1, 4096, 4096, 256, 24, 135},
      {WKind::kInt4, 1, 4096, 4096, 512, 36, 138},    {WKind::kInt4, 1, 4096, 4096, 1000, 50, 141},
      {WKind::kInt4, 1, 4096, 4096, 2048, 100, 149},  {WKind::kFp8, 2, 2048, 8192, 256, 31, 65},
      {WKind::kFp8, 2, 2048, 8192, 512, 60, 70},      {WKind::kFp8, 2, 2048, 8192, 1000, 115, 72},
      {WKind::kFp8, 2, 2048, 8192, 2048, 241, 143},   {WKind::kBf16, 2, 4096, 12288, 256, 172, 98},
      {WKind::kBf16, 2, 4096, 12288, 512, 260, 105},  {WKind::kBf16, 2, 4096, 12288, 1000, 505, 207},
      {WKind::kBf16, 2, 4096, 12288, 2048, 1046, 360}, {WKind::kInt4, 1, 2048, 5120, 512, 31, 78},
      {WKind::kInt4, 1, 2048, 5120, 1000, 58, 81},    {WKind::kInt4, 1, 2048, 5120, 2048, 91, 84},
      {WKind::kTable4, 2, 768, 2304, 2048, 54, 47},
  };
  for (const Measured& s : m)
    for (int32_t rank : {16, 64}) {
      const BatchCut c = cut(s.kind, s.n_proj, s.h_in, s.h_out, 0, rank, s.n);
      CHECK(s.rows_us < s.tiles_us ? c.rows == s.n : c.tiles >= s.n / 256 * 256);
    }

  // ---- with ids: measured us a call, a batch in runs on rows / on tiles and one of unlike neighbours on rows / on
  // tiles.  The host does not know which batch it has: the way taken costs at most a quarter more than the better one
  // when one batch in sixteen is of unlike neighbours.
  struct WithIds {
    WKind kind;
    int n_proj;
    int32_t h_in, h_out, adapters, max_rank, n;
    int runs_rows, runs_tiles, unlike_rows, unlike_tiles;
  };
  const WithIds w[] = {
      {WKind::kTable4, 2, 768, 2304, 64, 16, 512, 42, 60, 64, 555},
      {WKind::kTable4, 2, 768, 2304, 64, 64, 512, 51, 103, 72, 1057},
      {WKind::kTable4, 2, 768, 2304, 8, 16, 512, 41, 60, 40, 117},
      {WKind::kTable4, 2, 768, 2304, 64, 16, 1000, 69, 64, 98, 553},
      {WKind::kTable4, 2, 768, 2304, 64, 64, 1000, 78, 110, 109, 1037},
      {WKind::kTable4, 2, 768, 2304, 8, 16, 1000, 67, 63, 63, 121},
      {WKind::kTable4, 2, 768, 2304, 64, 16, 2048, 117, 67, 180, 546},
      {WKind::kTable4, 2, 768, 2304, 64, 64, 2048, 133, 112, 201, 1028},
      {WKind::kTable4, 2, 768, 2304, 8, 16, 2048, 114, 67, 109, 124},
      {WKind::kInt4, 1, 4096, 4096, 64, 16, 512, 58, 156, 66, 447},
      {WKind::kInt4, 1, 4096, 4096, 64, 64, 512, 64, 177, 86, 721},
      {WKind::kInt4, 1, 4096, 4096, 8, 16, 512, 50, 154, 50, 188},
      {WKind::kInt4, 1, 4096, 4096, 64, 16, 1000, 97, 157, 108, 442},
      {WKind::kInt4, 1, 4096, 4096, 64, 64, 1000, 97, 170, 133, 731},
      {WKind::kInt4, 1, 4096, 4096, 8, 16, 1000, 93, 157, 81, 188},
      {WKind::kInt4, 1, 4096, 4096, 64, 16, 2048, 177, 159, 193, 448},
      {WKind::kInt4, 1, 4096, 4096, 64, 64, 2048, 173, 172, 241, 748},
      {WKind::kInt4, 1, 4096, 4096, 8, 16, 2048, 148, 158, 143, 188},
      {WKind::kFp8, 2, 2048, 8192, 64, 16, 512, 116, 96, 124, 628},
      {WKind::kFp8, 2, 2048, 8192, 64, 64, 512, 140, 145, 158, 1165},
      {WKind::kFp8, 2, 2048, 8192, 8, 16, 512, 115, 97, 101, 159},
      {WKind::kFp8, 2, 2048, 8192, 64, 16, 1000, 204, 100, 229, 625},
      {WKind::kFp8, 2, 2048, 8192, 64, 64, 1000, 238, 148, 277, 1153},
      {WKind::kFp8, 2, 2048, 8192, 8, 16, 1000, 201, 100, 179, 161},
      {WKind::kFp8, 2, 2048, 8192, 64, 16, 2048, 403, 185, 471, 1094},
      {WKind::kFp8, 2, 2048, 8192, 64, 64, 2048, 428, 238, 534, 2046},
      {WKind::kFp8, 2, 2048, 8192, 8, 16, 2048, 395, 183, 385, 283},
      {WKind::kBf16, 2, 4096, 12288, 64, 16, 256, 204, 127, 209, 697},
      {WKind::kBf16, 2, 4096, 12288, 64, 64, 256, 229, 174, 225, 1276},
      {WKind::kBf16, 2, 4096, 12288, 8, 16, 256, 207, 127, 205, 195},
      {WKind::kBf16, 2, 4096, 12288, 64, 16, 512, 338, 133, 385, 686},
      {WKind::kBf16, 2, 4096, 12288, 64, 64, 512, 367, 176, 426, 1243},
      {WKind::kBf16, 2, 4096, 12288, 8, 16, 512, 335, 135, 321, 198},
      {WKind::kBf16, 2, 4096, 12288, 64, 16, 1000, 630, 258, 694, 1148},
      {WKind::kBf16, 2, 4096, 12288, 64, 64, 1000, 647, 312, 807, 2091},
      {WKind::kBf16, 2, 4096, 12288, 8, 16, 1000, 628, 255, 613, 359},
      {WKind::kBf16, 2, 4096, 12288, 64, 16, 2048, 1306, 426, 1468, 1620},
      {WKind::kBf16, 2, 4096, 12288, 64, 64, 2048, 1341, 484, 1593, 2899},
      {WKind::kBf16, 2, 4096, 12288, 8, 16, 2048, 1310, 421, 1284, 549},
      {WKind::kInt4, 1, 2048, 5120, 64, 16, 512, 60, 90, 68, 361},
      {WKind::kInt4, 1, 2048, 5120, 64, 64, 512, 67, 111, 74, 617},
      {WKind::kInt4, 1, 2048, 5120, 8, 16, 512, 44, 90, 43, 122},
      {WKind::kInt4, 1, 2048, 5120, 64, 16, 1000, 97, 96, 103, 358},
      {WKind::kInt4, 1, 2048, 5120, 64, 64, 1000, 104, 116, 124, 613},
      {WKind::kInt4, 1, 2048, 5120, 8, 16, 1000, 79, 94, 76, 125},
      {WKind::kInt4, 1, 2048, 5120, 64, 16, 2048, 160, 99, 175, 359},
      {WKind::kInt4, 1, 2048, 5120, 64, 64, 2048, 159, 111, 217, 621},
      {WKind::kInt4, 1, 2048, 5120, 8, 16, 2048, 141, 97, 131, 126},
  };
  for (const WithIds& s : w) {
    const BatchCut c = cut(s.kind, s.n_proj, s.h_in, s.h_out, s.adapters, s.max_rank, s.n);
    const double rows = 15 * s.runs_rows + s.unlike_rows, tiles = 15 * s.runs_tiles + s.unlike_tiles;
    CHECK((c.rows == s.n ? rows : tiles) <= 1.25 * std::min(rows, tiles));
  }
  std::puts("base plan ok");
  return 0;
}

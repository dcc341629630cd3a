// Host unit test of the cut of a batch between the row-streaming and the tiled
// base products (built with g++ under AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_base_plan.py).
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
  std::puts("base plan ok");
  return 0;
}

// How attention calls are split, on the host: whatever the sizes, a call that has places for partial results is given a workspace
// for them, a joining launch, and no more items than both can take.
#include <stdio.h>
#include <stdlib.h>

#include "hc_attend.h"

#define CHECK(cond)                                                                                              \
  do {                                                                                                           \
    if (!(cond)) {                                                                                               \
      fprintf(stderr, "check failed at line %d: %s (seqs %lld, q_rows %lld, max_q %lld, max_kv %lld, heads %d of %d, R %d)\n", \
              __LINE__, #cond, (long long)a.num_seqs, (long long)a.q_rows, (long long)a.max_q, (long long)a.max_kv, \
              a.q_heads, a.kv_heads, R);                                                                         \
      exit(1);                                                                                                   \
    }                                                                                                            \
  } while (0)

int main() {
  uint64_t seed = 1;
  auto below = [&](int64_t n) {
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    return (int64_t)((seed >> 33) % (uint64_t)n);
  };
  auto size = [&](int bits) { return below((int64_t)1 << (1 + below(bits))); };
  int split = 0, few_places = 0, none = 0, no_rows = 0;
  for (int round = 0; round < 2000000; round++) {
    hc::AttendArgs a = {};
    a.num_seqs = 1 + size(14);
    a.q_rows = 1 + size(16);
    a.max_q = below(4) ? size(12) : 0;
    if (a.max_q > a.q_rows) a.max_q = a.q_rows;
    a.max_kv = size(20);
    const int32_t dim = below(3) == 0 ? hc::kLatDim : below(2) ? 64 : 128;
    a.kv_heads = dim == hc::kLatDim ? 1 : 1 + (int32_t)below(12);
    a.group = 1 + (int32_t)below(20);
    a.q_heads = a.group * a.kv_heads;
    const int R = below(2) ? hc::kRowTile : dim == hc::kLatDim ? hc::kLatRows : hc::kTileRows;
    // of elements, and of 4-bit rows of few rows, whose items are of several KV heads
    const int heads = below(2) || R != hc::kRowTile ? 0 : a.kv_heads % 4 == 0 ? 4 : a.kv_heads % 2 == 0 ? 2 : 1;
    if (heads) a.kv_heads /= heads;
    const hc::Plan p = hc::plan(&a, R, dim, 256, heads, heads ? dim == hc::kLatDim ? 2 : 4 : 0, heads ? 32 + (int)size(8) : 0);
    const int64_t tiles = hc::most_tiles(a, R) * a.kv_heads;
    CHECK(p.items >= tiles && tiles > 0);
    CHECK((a.slots > 0) == (a.join_parts > 0) && (a.slots > 0) == (p.joins > 0));
    CHECK(p.joins == a.slots * a.join_parts);
    CHECK(!p.few_places || a.slots > 0);
    CHECK(a.slots == 0 || a.slots == (p.few_places ? 2 * a.target : p.items));
    CHECK(a.slots <= p.items);
    if (a.slots == 0) CHECK(a.min_split > a.max_kv);  // no tile is split
    split += a.slots > 0;
    few_places += p.few_places;
    none += a.slots == 0;
    no_rows += a.max_q == 0 && a.max_kv > 1000 && tiles > 2 * a.target;
  }
  if (split < 100000 || few_places < 10000 || none < 10000 || no_rows < 1000) {
    fprintf(stderr, "not all was met: %d %d %d %d\n", split, few_places, none, no_rows);
    return 1;
  }
  printf("attend_plan ok: %d split, %d of them with few places, %d not\n", split, few_places, none);
  return 0;
}

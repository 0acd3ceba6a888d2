// Host-side arithmetic of the forward-pass calls, under AddressSanitizer + UBSan.
//
// Extents (hc_extent.h): sizes and strides whose products pass 64 bits are told apart from small
// tensors, small ones are counted element by element.
//
// Overlap of two strided tensors, against every element of both: never missed, and told apart exactly
// where both step alike.
//
// Reports (hc_wrong.h): two reports made between any two steps of a hc_pool_sync that takes others;
// each is in what this sync or the next one takes, with its position.
#include <stdio.h>
#include <stdlib.h>

#include <functional>
#include <set>
#include <vector>

#include "hc_extent.h"
#include "hc_wrong.h"

#define CHECK(cond)                                                              \
  do {                                                                           \
    if (!(cond)) {                                                               \
      fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond);         \
      exit(1);                                                                   \
    }                                                                            \
  } while (0)

static void extents_that_wrap() {
  const int64_t far = (int64_t)1 << 40;
  // (2^23 rows - 1) of stride 2^40 are 2^63 elements: in 64 bits that left 2 * dim bytes
  for (int64_t n : {((int64_t)1 << 22) + 1, ((int64_t)1 << 23) + 1, ((int64_t)1 << 24) + 1, (int64_t)1 << 31}) {
    const int64_t rows[2] = {far, 128}, heads[2] = {128, far};
    CHECK(hc::tensor_bytes(rows, n, 1, 128) == hc::kTooFar);
    CHECK(hc::tensor_bytes(heads, 1, n, 128) == hc::kTooFar);
    CHECK(hc::rows_apart(rows, n, 8, 128));
  }
  const int64_t both[2] = {far, far};
  CHECK(hc::tensor_bytes(both, 1 << 22, 1 << 22, 128) == hc::kTooFar);
  CHECK(!hc::rows_apart(both, 1 << 24, 1 << 24, 128));  // its heads take 2^64 elements of a stride of 2^40
  for (int64_t rows : {((int64_t)1 << 20) + 1, ((int64_t)1 << 21) + 1, ((int64_t)1 << 30), ((int64_t)1 << 31) - 1})
    CHECK(hc::table_bytes(rows, 4, far) == hc::kTooFar);
  // the largest that fit
  CHECK(hc::table_bytes(2, 1, ((int64_t)1 << 60) - 2) == 8 * (((int64_t)1 << 60) - 1));
  CHECK(hc::table_bytes(2, 1, ((int64_t)1 << 60) - 1) == hc::kTooFar);
  const int64_t last[2] = {((int64_t)1 << 62) - 8, 8};
  CHECK(hc::tensor_bytes(last, 2, 1, 7) == INT64_MAX - 1);
  CHECK(hc::tensor_bytes(last, 2, 1, 8) == hc::kTooFar);
}

static void small_extents_and_overlaps() {
  for (int64_t s0 = 0; s0 <= 40; s0 += 4)
    for (int64_t s1 = 0; s1 <= 40; s1 += 4)
      for (int64_t n = 0; n <= 4; n++)
        for (int64_t heads = 0; heads <= 4; heads++)
          for (int64_t dim : {4, 8, 12}) {
            const int64_t stride[2] = {s0, s1};
            std::set<int64_t> seen;
            int64_t last = -1;
            bool apart = true;
            for (int64_t i = 0; i < n; i++)
              for (int64_t h = 0; h < heads; h++)
                for (int64_t d = 0; d < dim; d++) {
                  const int64_t at = i * s0 + h * s1 + d;
                  apart &= seen.insert(at).second;
                  if (at > last) last = at;
                }
            CHECK(hc::tensor_bytes(stride, n, heads, dim) == 2 * (last + 1));
            if (n > 0 && heads > 0 && hc::rows_apart(stride, n, heads, dim)) CHECK(apart);
            // nested layouts are recognised
            const bool rows_outside = s1 >= dim && s0 >= s1 * (heads - 1) + dim;
            const bool heads_outside = s0 >= dim && s1 >= s0 * (n - 1) + dim;
            if (n > 0 && heads > 0 && (rows_outside || heads_outside)) CHECK(hc::rows_apart(stride, n, heads, dim));
            CHECK(hc::table_bytes(n, dim, s0) == (n > 0 ? 8 * ((n - 1) * s0 + dim) : 0));
          }
  CHECK(hc::table_bytes(5, 0, 10) == 0);
}

static void tensors_that_share() {
  uint64_t seed = 1;
  auto below = [&](int n) {
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    return (int64_t)((seed >> 33) % n);
  };
  static int16_t memory[4096];
  int alike = 0, apart = 0, enclosed = 0;
  for (int round = 0; round < 300000; round++) {
    hc::Tensor t[2];
    std::set<int64_t> at[2];
    const int64_t token = below(30), head = below(12);
    for (int i = 0; i < 2; i++) {
      const bool own = below(3) == 0;
      const int64_t base = below(120);
      t[i] = {memory + base, {own ? below(30) : token, own ? below(12) : head}, below(5), below(4), 1 + below(5)};
      for (int64_t n = 0; n < t[i].n; n++)
        for (int64_t h = 0; h < t[i].heads; h++)
          for (int64_t d = 0; d < t[i].dim; d++) at[i].insert(base + n * t[i].stride[0] + h * t[i].stride[1] + d);
    }
    bool want = false;
    for (int64_t x : at[0]) want |= at[1].count(x) > 0;
    const bool got = hc::share(t[0], t[1]);
    CHECK(got == hc::share(t[1], t[0]));
    CHECK(got || !want);
    const bool tokens = t[0].n <= 1 || t[1].n <= 1 || t[0].stride[0] == t[1].stride[0];
    const bool heads = t[0].heads <= 1 || t[1].heads <= 1 || t[0].stride[1] == t[1].stride[1];
    if (tokens && heads) CHECK(got == want);
    alike += tokens && heads && want;
    apart += tokens && heads && !want && !at[0].empty() && !at[1].empty() &&
             hc::overlap(t[0].at, t[0].bytes(), t[1].at, t[1].bytes());
    enclosed += got && !want;
  }
  CHECK(alike > 10000 && apart > 1000 && enclosed > 100);  // all of it was met
  // tables side by side in one buffer of rows of 8 entries
  static int64_t rows[64];
  CHECK(!hc::share(hc::table_tensor(rows, 8, 4, 8), hc::table_tensor(rows + 4, 8, 4, 8)));
  CHECK(hc::share(hc::table_tensor(rows, 8, 5, 8), hc::table_tensor(rows + 4, 7, 4, 8)));
  CHECK(hc::share(hc::table_tensor(rows, 8, 4, 8), hc::table_tensor(rows, 8, 4, 8)));
}

// Atomics that let something else happen before each of them.
struct Stepped {
  static std::function<void()> between;
  static void minimum(hc::WrongWord* word, hc::WrongWord x) {
    if (x < *word) *word = x;
  }
  static hc::WrongWord exchange(hc::WrongWord* word, hc::WrongWord x) {
    between();
    const hc::WrongWord old = *word;
    *word = x;
    return old;
  }
};
std::function<void()> Stepped::between;

// The reports of one hc_pool_sync: a look at the words, and if there is something, all of it taken.
static std::vector<hc::WrongWord> sync_takes(hc::WrongWord* words) {
  std::vector<hc::WrongWord> taken(hc::kWrongKinds, hc::kNothing);
  Stepped::between();
  std::vector<hc::WrongWord> seen(words, words + hc::kWrongKinds);
  hc::WrongWord first = hc::kNothing;
  if (hc::wrong_code(seen.data(), &first)) hc::take_wrong<Stepped>(words, taken.data());
  Stepped::between();
  return taken;
}

static void reports_beside_a_sync() {
  struct Report {
    hc::Wrong kind;
    int64_t position;
    int step;  // made before this step
  };
  for (int before = 0; before < 2; before++)  // something to take at the start
    for (int i = 0; i < 4; i++)
      for (int j = 0; j < 4; j++)
        for (int kinds = 0; kinds < 4; kinds++)
          for (int order = 0; order < 2; order++) {
            hc::WrongWord words[hc::kWrongKinds] = {hc::kNothing, hc::kNothing};
            if (before) hc::report_wrong<Stepped>(words, hc::kWrongIndex, 50);
            Report r[2] = {{(kinds & 1) ? hc::kWrongLengths : hc::kWrongIndex, order ? 7 : 90, i},
                           {(kinds & 2) ? hc::kWrongLengths : hc::kWrongIndex, order ? 90 : 7, j}};
            int step = 0;
            bool made[2] = {false, false};
            Stepped::between = [&] {
              for (int k = 0; k < 2; k++)
                if (r[k].step == step) {
                  hc::report_wrong<Stepped>(words, r[k].kind, r[k].position);
                  made[k] = true;
                }
              step++;
            };
            std::vector<std::vector<hc::WrongWord>> takes = {sync_takes(words)};
            while (step < 4) Stepped::between();
            Stepped::between = [] {};
            takes.push_back(sync_takes(words));
            takes.push_back(sync_takes(words));
            for (int k = 0; k < 2; k++) {
              CHECK(made[k]);
              bool found = false;
              for (auto& t : takes) found |= t[r[k].kind] <= (hc::WrongWord)r[k].position;
              CHECK(found);
            }
            if (before) CHECK(takes[0][hc::kWrongIndex] <= 50);
            CHECK(takes[2][0] == hc::kNothing && takes[2][1] == hc::kNothing);  // and nothing twice
          }
  hc::WrongWord words[hc::kWrongKinds] = {hc::kNothing, hc::kNothing}, first = hc::kNothing;
  CHECK(hc::wrong_code(words, &first) == 0 && first == hc::kNothing);
  words[hc::kWrongLengths] = 9;
  CHECK(hc::wrong_code(words, &first) == 4 && first == 9);
  words[hc::kWrongIndex] = 3;
  first = 12;  // what the transfers reported
  CHECK(hc::wrong_code(words, &first) == 5 && first == 3);
}

int main() {
  reports_beside_a_sync();
  extents_that_wrap();
  small_extents_and_overlaps();
  tensors_that_share();
  printf("forward_host ok\n");
  return 0;
}

// Every sum of the balance loss is found where the forward pass left it: the tokens'
// values are added as its blocks and waves add them, in whole numbers, then looked up
// with the functions that the kernel uses.  Starts of sequences: argv[1] of them drawn
// for every number of tokens.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <vector>

#include "balance_places.hpp"

using namespace qmoe;

static uint32_t state = 1;
static uint32_t draw() { return state = state * 1664525u + 1013904223u, state >> 8; }

// The last sequence that begins at or before t (-1, S: none).
static int sequence_of(const std::vector<int>& starts, int t) {
  return (int)(std::upper_bound(starts.begin(), starts.end(), t) - starts.begin()) - 1;
}

static int check(int T, const std::vector<int>& starts) {
  const int S = (int)starts.size() - 1, run = run_of(T), per = ROW_WAVES * run;
  std::vector<int64_t> value(T), q(T, -1);  // -1: no sum there
  for (int t = 0; t < T; t++) value[t] = 1 + draw() % 1000;
  for (int b = 0; b * per < T; b++) {
    const int block_s = sequence_of(starts, b * per);
    int64_t of_block = 0;
    for (int first = b * per; first < std::min((b + 1) * per, T); first += run) {
      int s = -2, from = 0;
      int64_t total = 0;
      auto put = [&] {
        if (s == block_s)
          of_block += total;
        else if (s >= 0 && s < S)
          q.at(from) = total;
      };
      for (int t = first; t < std::min(first + run, T); t++) {
        if (sequence_of(starts, t) != s) {
          if (t > first) put();
          s = sequence_of(starts, t), from = t, total = 0;
        }
        total += value[t];
      }
      put();
    }
    q.at(b * per) = of_block;
  }
  for (int s = 0; s < S; s++) {
    const int first = starts[s], end = starts[s + 1];
    int64_t want = 0, sum = 0;
    for (int t = first; t < end; t++) want += value[t];
    bool missing = false;
    auto get = [&](int at) {
      if (at >= T || q[at] < 0)
        missing = true;
      else
        sum += q[at];
    };
    for (int wave = 0; wave < ROW_WAVES; wave++) {
      const int at = wave_place(first, end, wave, run);
      if (at >= 0) get(at);
    }
    for (int b = block_from(first, run); b * per < end; b++) get(b * per);
    if (missing || sum != want) {
      printf("T %d, sequence %d of %d [%d, %d): sum %lld, not %lld%s\n", T, s, S, first, end, (long long)sum, (long long)want,
             missing ? ", a place without a sum" : "");
      return 1;
    }
  }
  return 0;
}

int main(int argc, char** argv) {
  const int draws = argc > 1 ? atoi(argv[1]) : 10;
  int bad = 0;
  for (int T : {0, 1, 2, 15, 16, 17, 129, 255, 256, 257, 4096, 8191, 8192, 8193, 8195, 16449, 40000, 65529, 65536})
    for (int i = 0; i < draws && bad < 20; i++) {
      const int S = i == 0 ? 1 : 1 + draw() % (i % 2 ? 5 : 300);
      std::vector<int> starts(S + 1);
      const int range = i % 3 ? T : std::min(T, 40);  // (short ones next to each other, all others empty)
      const int from = i % 3 == 2 ? std::max(0, T - 40) : 0;
      for (int& v : starts) v = i == 0 ? 0 : std::min(T, from + (int)(draw() % (range + 1)));
      std::sort(starts.begin(), starts.end());
      if (i % 4 == 0) starts[S] = T;
      bad += check(T, starts);
    }
  if (!bad) printf("OK\n");
  return bad != 0;
}

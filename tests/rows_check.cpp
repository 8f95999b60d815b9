// rows_overlap against every byte, over drawn sets of rows.
#include <stdio.h>

#include <random>
#include <vector>

#include "rows.h"

int main() {
  std::mt19937 rng(7);
  auto upto = [&](int n) { return (int)(rng() % n); };
  int together = 0;
  for (int i = 0; i < 400000; ++i) {
    pkv::Rows r[2];
    for (int k = 0; k < 2; ++k) {
      r[k].n = 1 + upto(5);
      r[k].bytes = 1 + upto(9);
      r[k].stride = r[k].bytes + (upto(3) ? upto(14) : 0);
      r[k].at = 1000 + upto(60);
    }
    if (upto(2)) {                                    // parts of the same rows
      r[1].stride = r[0].stride;
      if (r[1].bytes > r[1].stride) r[1].bytes = r[1].stride;
    }
    for (int k = 0; k < 2; ++k)
      if (r[k].n == 1 && upto(2)) r[k].stride = upto(4);             // one row's stride says nothing
    std::vector<char> used(400, 0);
    bool want = false;
    for (int k = 0; k < 2; ++k)
      for (int j = 0; j < r[k].n; ++j)
        for (int b = 0; b < r[k].bytes; ++b) {
          char& u = used[r[k].at - 1000 + j * r[k].stride + b];
          if (k == 1 && u) want = true;
          if (k == 0) u = 1;
        }
    together += want;
    if (pkv::rows_overlap(r[0], r[1]) != want || pkv::rows_overlap(r[1], r[0]) != want) {
      printf("n %d %d, stride %d %d, bytes %d %d, at %d %d: %d\n", (int)r[0].n, (int)r[1].n, (int)r[0].stride, (int)r[1].stride,
             (int)r[0].bytes, (int)r[1].bytes, (int)r[0].at, (int)r[1].at, want);
      return 1;
    }
  }
  return together < 40000 || together > 360000;
}

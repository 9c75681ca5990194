// The rule that maps a call's rows to requests (csrc/requests.h), on the host:
// whatever the offsets hold, a row that request_of gives to a request is one
// of that request's rows, and no request has rows outside the call.  Offsets in
// order give every row between the first and the last one its owner.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <vector>

#include "requests.h"

int main() {
  srand(1);
  int64_t cases = 0, owned = 0;
  for (int run = 0; run < 20000; ++run) {
    const int B = 1 + rand() % 9, T = rand() % 40;
    std::vector<int32_t> off(B + 1);
    const int kind = run % 4;                  // in order and inside, in order, any, with extremes
    for (auto& o : off) o = kind == 0 ? rand() % (T + 1) : rand() % 120 - 40;
    if (kind < 2) std::sort(off.begin(), off.end());
    if (kind == 3) off[rand() % (B + 1)] = rand() & 1 ? 2147483647 : -2147483647 - 1;
    mxq::CacheArgs c = {};
    c.q_offsets = off.data();
    c.B = B;
    for (int b = 0; b < B; ++b) {
      const mxq::RequestRows r = mxq::request_rows(c, b, T);
      if (r.len < 0 || (r.len && (r.begin < 0 || (int64_t)r.begin + r.len > T))) {
        printf("run %d request %d: rows %d + %d of %d\n", run, b, r.begin, r.len, T);
        return 1;
      }
    }
    for (int t = 0; t < T; ++t, ++cases) {
      mxq::RequestRows own;
      const int64_t b = mxq::request_of(c, t, T, own);
      if (b >= 0) {
        const mxq::RequestRows r = mxq::request_rows(c, b, T);
        if (b >= B || own.begin != r.begin || own.len != r.len || t < r.begin || t >= r.begin + r.len) {
          printf("run %d row %d: owner %d has rows %d + %d\n", run, t, (int)b, r.begin, r.len);
          return 1;
        }
        ++owned;
      }
      const bool inside = t >= off[0] && t < off[B];
      if (kind == 0 && (b >= 0) != inside) {
        printf("run %d row %d: owner %d\n", run, t, (int)b);
        return 1;
      }
    }
  }
  printf("ok %lld rows, %lld owned\n", (long long)cases, (long long)owned);
  return 0;
}

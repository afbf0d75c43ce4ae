// Prints which kernel the 4-bit products' planner chooses, one line of input after another (host code only):
//   M K N act experts  ->  "refused", or the kernel, its launch's tiles and its parts of K as `name=value` words.
// Built and run by tests/test_mx4_plans.py.
#include "mx4_api.hip"

#include <stdio.h>

int main() {
  long long M, K, N;
  int act, experts;
  while (scanf("%lld %lld %lld %d %d", &M, &K, &N, &act, &experts) == 5) {
    linear_desc d{M, K, N, act, MLP_BF16, experts};
    MxPlan p;
    if (make_plan(&d, p) != MLP_OK) printf("refused\n");
    else if (p.skinny) printf("form=stream tiles=%d splits=1\n", p.tiles);
    else printf("form=%dx%d tiles=%d splits=%d\n", p.bm, p.bn, p.tiles, p.splits);
  }
  return 0;
}

// Prints which kernels the mixture-of-experts planner chooses, one line of input after another (host code only):
//   fwd|bwd M K N act dtype experts [dx dw]  ->  the tiles, splits and schedule as `name=value` words.
// Built and run by tests/test_moe_plans.py.
#include "moe_api.hip"

#include <stdio.h>
#include <string.h>

static const char* tile_name(TileShape t) {
  switch (t) {
    case TILE_256x256: return "256x256";
    case TILE_256x128: return "256x128";
    case TILE_128x128: return "128x128";
    case TILE_256x256_W8: return "256x256w8";
    case TILE_256x128_W8: return "256x128w8";
    case TILE_128x128_RING: return "128x128";
    case TILE_64x64: return "64x64";
    default: return "none";
  }
}

int main() {
  char phase[8];
  long long M, K, N;
  int act, dtype, experts, dx, dw;
  while (scanf("%7s %lld %lld %lld %d %d %d %d %d", phase, &M, &K, &N, &act, &dtype, &experts, &dx, &dw) == 9) {
    linear_desc d{M, K, N, act, dtype, experts};
    if (check_linear(&d) != MLP_OK) {
      printf("refused\n");
    } else if (!strcmp(phase, "fwd") && experts) {
      const ExpertPlan p = plan_experts(&d, true);
      if (p.form == EXPERT_SKINNY) printf("form=stream\n");
      else printf("form=tiles tile=%s\n", tile_name(p.tile));
    } else if (!strcmp(phase, "fwd")) {
      const LinearFwd f = plan_linear(&d);
      if (f.skinny) printf("form=stream\n");
      else printf("form=tiles tile=%s splits=%d\n", tile_name(f.plan.tile), f.plan.splits);
    } else {
      const LinearBwd b = experts || M == 0 ? LinearBwd{} : plan_linear_bwd(&d, dx != 0, dw != 0);
      if (experts || M == 0 || b.small) {
        const ExpertPlan p = plan_experts(&d, false);
        printf("form=%s tile=%s splits=%d pieces=%d dw_first=%d\n", p.strip_parts ? "strips" : "experts", tile_name(p.tile),
               p.dx_splits, p.piece_rows, (int)p.dw_first);
      } else if (b.group) {
        printf("form=group\n");
      } else {
        printf("form=apart dx=%s dx_splits=%d dx_tail=%d dw=%s dw_splits=%d\n", tile_name(b.dx.main.tile), b.dx.main.splits,
               (int)(b.dx.m1 > 0), tile_name(b.dw.tile), b.dw.splits);
      }
    }
  }
  return 0;
}

// Prints which kernel takes a 4-bit product, for lines of "rows n k matrices" on the input.
#include <stdio.h>

#include "../lossless_draft_verification_spec_amd/csrc/w4_plan.h"

int main() {
  int rows, n, k, mats;
  while (scanf("%d %d %d %d", &rows, &n, &k, &mats) == 4) {
    const psispec::ManyPlan m = psispec::many_plan(rows, n, k, mats, PSISPEC_W4_INT);
    const psispec::FewPlan f = psispec::few_plan(rows, (n + 15) / 16, (k + 127) / 128, mats);
    if (m.use)
      printf("many %d %d\n", m.nb, m.parts > 1);
    else
      printf("few %d %d %d\n", 4 * f.r4, f.nt, f.kw);
  }
  return 0;
}

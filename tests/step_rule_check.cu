// Checks on the host when single tokens get a cluster of CTAs for each segment: never more clusters
// than the device holds at once.
#include <cstdio>
#include <vector>

#include "pa_window.cu"

int main() {
  int bad = 0;
  struct Case {
    int seqs, keys, heads;
    StepFit fit;
    int want;
  };
  const StepFit some = {{304, 152, 74, 36}}, none = {{304, 0, 0, 0}}, all = {{304, 152, 76, 40}};
  const Case cases[] = {
      {16, 1024, 4, some, 4}, {18, 1024, 4, some, 4}, {19, 1024, 4, some, 0}, {19, 1024, 4, all, 4}, {74, 4096, 1, some, 4}, {75, 4096, 1, some, 0},
      {8, 4096, 4, some, 8}, {9, 4096, 4, some, 0}, {9, 4096, 4, all, 8}, {34, 2048, 1, some, 8}, {35, 2048, 1, some, 0},
      {38, 1024, 4, some, 2}, {38, 1024, 4, none, 0}, {16, 1024, 4, none, 0}, {64, 1024, 4, none, 1}, {76, 1024, 4, some, 1}, {128, 1024, 4, some, 1}};
  for (const Case& c : cases) {
    std::vector<int32_t> lens(c.seqs, c.keys), n_new(c.seqs, 1);
    Batch b{lens.data(), n_new.data(), (uint32_t)c.seqs, kAllKeys, 0, c.heads};
    pa_pool_desc d = {};
    d.n_kv_heads = (uint32_t)c.heads;
    if (check_batch(d, ~0u, &b) != PA_OK || step_cluster(b, 152, &c.fit) != c.want)
      ++bad, std::printf("%d sequences of %d keys, %d heads: %d, not %d\n", c.seqs, c.keys, c.heads, step_cluster(b, 152, &c.fit), c.want);
  }
  std::printf("mismatches %d\n", bad);
  return bad != 0;
}

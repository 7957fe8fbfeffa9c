// Checks on the host that the scratch of the windowed attention never shrinks when a token, a key, a
// sequence, a longer window or more first keys are added, and that it holds what the call puts there.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "pa_window.cu"

static long long bad = 0;
#define CHECK(x)                                                          \
  do {                                                                    \
    if (!(x) && ++bad <= 20) std::printf("line %d: %s (batch %d)\n", __LINE__, #x, batch); \
  } while (0)

struct Call {
  std::vector<int32_t> lens, fresh;
  uint32_t window, sinks;
  int heads;

  Batch batch_of() const {
    pa_pool_desc d = {};
    d.n_kv_heads = (uint32_t)heads;
    Batch b{lens.data(), fresh.data(), (uint32_t)lens.size(), clamp_keys(window ? window : ~0u), clamp_keys(sinks), heads};
    if (check_batch(d, ~0u, &b) != PA_OK) ++bad, std::printf("a batch was refused\n");
    return b;
  }
  size_t bytes() const { return layout_of(152, batch_of()).total; }
};

int main(int argc, char** argv) {
  const int batches = argc > 1 ? std::atoi(argv[1]) : 300;
  std::mt19937 rng(5);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int batch = 0; batch < batches; ++batch) {
    Call c;
    c.heads = pick(1, 8);
    const uint32_t windows[] = {1, 15, 16, 17, 64, (uint32_t)pick(1, 400)};
    c.window = windows[pick(0, 5)];
    c.sinks = (uint32_t)(pick(0, 1) ? pick(0, 40) : 0);
    const int n_seq = pick(1, 4);
    for (int i = 0; i < n_seq; ++i) {
      c.fresh.push_back(pick(0, 2) ? pick(55, 70) : pick(0, 3) ? pick(0, 12) : pick(60, 400));
      c.lens.push_back(c.fresh[i] + pick(0, 600));
    }
    size_t last = c.bytes();
    for (int step = 0; step < 60; ++step) {
      const int i = pick(0, (int)c.lens.size() - 1);
      switch (pick(0, 9)) {
        case 0: ++c.window; break;
        case 1: c.window += (uint32_t)pick(1, 40); break;
        case 2: ++c.sinks; break;
        case 3: c.lens.push_back(pick(0, 200)), c.fresh.push_back(pick(0, c.lens.back())); break;
        case 4: case 5: case 6: ++c.lens[i]; break;
        case 7: c.lens[i] += pick(1, 40); break;
        default:
          ++c.fresh[i];
          if (c.lens[i] < c.fresh[i]) c.lens[i] = c.fresh[i];
      }
      const size_t bytes = c.bytes();
      CHECK(bytes >= last);
      last = bytes;
    }
    CHECK((c.window = 0, c.bytes()) >= last);  // all keys
    // what a call of this batch uses: the prompts' row groups one sequence's after the other's, the kernels' slots
    for (const uint32_t window : {c.window, 1u, 33u}) {
      c.window = window;
      const Batch b = c.batch_of();
      const WsLayout l = layout_of(152, b);
      long long groups = 0;
      int most = 0;
      bool prompts = false;
      for (uint32_t i = 0; i < b.n_seq; ++i) {
        if (b.many(i)) groups += seq_span(b.lens[i], b.n_new[i], b.window, b.sinks).groups, prompts = true;
        else if (b.n_new[i] > most) most = b.n_new[i];
      }
      CHECK((long long)(l.v - l.k) >= groups * b.heads * kGroupBytes && (long long)(l.wide - l.v) >= groups * b.heads * kGroupBytes);
      CHECK((long long)(l.total - l.wide) >= groups * b.heads * 2);
      const size_t few = (size_t)2 * 152 * slot_rows_of((uint32_t)most), many = prompts ? (size_t)2 * 76 * kPromptRows : 0;
      const size_t rows = std::max(few, many);
      CHECK(l.o >= rows * sizeof(float2) && l.o + rows * kD * sizeof(float) <= l.k);
    }
  }
  std::printf("mismatches %lld\n", bad);
  return bad != 0;
}

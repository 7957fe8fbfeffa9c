// Checks on the host that batches of more units than a launch of the windowed attention takes go over
// several launches, each unit's rows once and in order.
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

template <class P>
static void check(int batches, bool many, int max_ctas) {
  std::mt19937 rng(3);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  static P p;
  static MergeParams m;
  for (int batch = 0; batch < batches; ++batch) {
    std::vector<int32_t> lens, fresh;
    long long rows = 0, units = 0, tokens = 0;
    while (units <= 2 * P::kMaxUnits + pick(0, P::kMaxUnits)) {
      const int n = pick(0, 5) == 0 ? 0 : pick(0, 9) == 0 ? (many ? pick(1, 63) : pick(64, 300)) : many ? pick(64, 900) : pick(1, 63);
      fresh.push_back(n);
      lens.push_back(n + pick(0, 300));
      if (Batch::is_many(n) == many) rows += kGqa * n, units += (kGqa * n + P::kUnitRows - 1) / P::kUnitRows;
    }
    p.window = pick(0, 1) ? kAllKeys : pick(1, 200);
    p.sinks = pick(0, 20);
    p.n_kv_heads = pick(1, 4);
    p.slot_rows = m.slot_rows = P::kUnitRows;
    const Batch b{lens.data(), fresh.data(), (uint32_t)lens.size(), p.window, p.sinks, p.n_kv_heads};
    int launches = 0;
    long long seen = 0, seen_units = 0, next_token = 0;
    uint32_t seq = 0;
    for (Cursor at{0, 0, 0}; at.seq < b.n_seq;) {
      const Plan plan = plan_chunk(p, m, b, many, max_ctas, &at);
      if (p.n_units == 0) break;
      ++launches;
      CHECK(p.n_units <= P::kMaxUnits && plan.cuts <= p.n_ctas);
      int places = 0;
      for (int i = 0; i < p.n_units; ++i) {
        const Unit& u = p.unit[i];
        for (; seq < (uint32_t)u.seq; ++seq) next_token += fresh[seq], seen = 0;
        CHECK(Batch::is_many(fresh[u.seq]) == many);
        CHECK(u.token == next_token + seen / kGqa && unit_row0(u) == seen % kGqa);  // where the unit before ended
        CHECK(u.pos == lens[u.seq] - fresh[u.seq] + seen / kGqa && u.len == lens[u.seq]);
        CHECK(unit_rows(u) == std::min<long long>(P::kUnitRows, (long long)kGqa * fresh[u.seq] - seen));
        CHECK(u.at >= places);
        places = u.at;
        seen += unit_rows(u);
        tokens += unit_rows(u);
        ++seen_units;
      }
    }
    CHECK(launches > 2 && seen_units == units && tokens == rows);
  }
}

int main() {
  check<WindowParams>(12, false, 152);
  check<PromptParams>(12, true, 76);
  std::printf("mismatches %lld\n", bad);
  return bad != 0;
}

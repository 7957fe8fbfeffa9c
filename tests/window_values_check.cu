// Checks on the host which values the prompts' kernel multiplies: every unit has the values of the keys
// that its tokens see, and none of a key that lies more than 64 places from what one of its tokens sees.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "pa_window.cu"

static long long bad = 0, edges = 0;
#define CHECK(x)                                                          \
  do {                                                                    \
    if (!(x) && ++bad <= 20) std::printf("line %d: %s (batch %d)\n", __LINE__, #x, batch); \
  } while (0)

int main(int argc, char** argv) {
  const int batches = argc > 1 ? std::atoi(argv[1]) : 300;
  std::mt19937 rng(9);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  static PromptParams p;
  static MergeParams m;
  for (int batch = 0; batch < batches; ++batch) {
    const int win[] = {1, 15, 16, 17, pick(1, 100), pick(1, 600), kAllKeys}, snk[] = {0, 1, 4, 15, 16, 17, 31, pick(0, 300), kAllKeys};
    p.window = win[pick(0, 6)];
    p.sinks = snk[pick(0, 8)];
    p.n_kv_heads = pick(1, 4);
    std::vector<int32_t> lens, fresh;
    for (int i = pick(1, 4); i > 0; --i) {
      fresh.push_back(pick(0, 4) ? pick(64, 900) : pick(0, 63));
      lens.push_back(fresh.back() + (pick(0, 1) ? 0 : pick(0, 400)));
    }
    const Batch b{lens.data(), fresh.data(), (uint32_t)lens.size(), p.window, p.sinks, p.n_kv_heads};
    p.slot_rows = m.slot_rows = kPromptRows;
    std::vector<PromptSeq> seqs(lens.size());  // as prepare_prompts has them
    int group0 = 0;
    for (uint32_t i = 0; i < b.n_seq; ++i) {
      if (!b.many(i)) continue;
      const SeqSpan s = seq_span(lens[i], fresh[i], p.window, p.sinks);
      seqs[i] = PromptSeq{(int32_t)i, lens[i], s.lo, s.s16, s.shift, s.groups, group0, s.edge, 0};
      group0 += s.groups;
      edges += s.edge >= 0;
      CHECK(s.edge < s.groups && s.groups == ceil_div(s.end, kGroup) + (s.edge >= 0));
    }
    uint32_t seq = 0;
    group0 = 0;
    for (Cursor at{0, 0, 0}; at.seq < b.n_seq;) {
      plan_chunk(p, m, b, true, 76, &at);
      if (p.n_units == 0) break;
      place_prompts(p, b, &seq, &group0);
      for (int i = 0; i < p.n_units; ++i) {
        const PromptUnit& u = p.unit[i];
        const PromptSeq& s = seqs[u.seq];
        const Span sp = span_of(u, p.window, p.sinks);
        CHECK(u.group0 == s.group0 && u.groups == s.groups);
        const int last = u.pos + (unit_row0(u) + unit_rows(u) - 1) / kGqa;
        const int whole = (sp.end + 15) & ~15, from = 16 * pick(0, 3);  // copies begin at any row group
        Run run{0, 0};
        for (int v = std::min(from, whole); v < whole; ++v) {
          if (v % 16 == 0 && (v == from || v == run.stop)) {
            run = run_of(u, sp, u.edge, v, whole);
            CHECK(run.stop > v && run.stop <= whole && run.stop % 16 == 0);
            run.group -= v >> 4;
          }
          const int key = v < sp.s16 ? v : v + sp.shift, group = run.group + (v >> 4);
          CHECK(v < run.stop && group >= 0 && group < u.groups && first_key(s, group) + (v & 15) == key);
          const Run keys = run_of(u, sp, -1, v & ~15, whole);
          CHECK(keys.group == group_of(u, sp, v) && keys.group != s.edge);
          const bool has = has_value(s, group, key, p.sinks);
          if (has) CHECK(key < u.len);
          for (int pos = u.pos; pos <= last; ++pos) {
            const int lo = pos >= p.window ? pos - p.window + 1 : 0;
            if (key <= pos && (key >= lo || key < p.sinks)) CHECK(has);
            else if (has) CHECK(key > pos ? key - pos <= 64 : lo - key <= 64);
          }
        }
      }
    }
  }
  std::printf("mismatches %lld, %lld sequences with a group of their own\n", bad, edges);
  return bad != 0 || edges < batches / 20;
}

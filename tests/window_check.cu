// Checks the plan of the windowed attention on the host: the units, the ranges and the cuts
// that pa_window.cu makes, and what pa_window_impl.cuh derives from them for a tile (key
// order, masks, live keys, slots), against the definition, over random batches.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <tuple>

#include "pa_window.cu"

static long long bad = 0, listed = 0;
#define CHECK(x)                                         \
  do {                                                   \
    if (!(x)) {                                          \
      if (++bad <= 20) std::printf("line %d: %s (batch %d)\n", __LINE__, #x, batch); \
    }                                                    \
  } while (0)

template <class P>
constexpr bool kPrompt = false;
template <>
constexpr bool kPrompt<PromptParams> = true;

static bool sees(const Unit& u, int row, int key, int window, int sinks) {
  const long long pos = u.pos + (unit_row0(u) + row) / kGqa;
  return key <= pos && (key > pos - window || key < sinks);
}

// A tile of the kernel for few tokens: its masks, live keys.
static void masks(const WindowParams& p, const Unit& u, const Span& s, int key0, int last_pos, int batch) {
  const int last_lo = last_pos >= p.window ? last_pos - p.window + 1 : 0;
  const bool inner = sees_all(s, key0, u.pos, last_lo, p.sinks);
  Tile tl{};
  tl.open = u.pos;
  tl.row0 = unit_row0(u);
  tl.pad[0] = key0;
  tl.pad[1] = s.shift;
  const WindowKeys live = live_keys(p, live_of(s, key0, p.sinks), 0);
  for (int k = 0; k < kKeys; ++k) {
    const int v = key0 + k, key = v < s.s16 ? v : v + s.shift;
    const int2 see = rows_that_see(p, tl, k);
    bool any = false, all = true;
    for (int r = 0; r < unit_rows(u); ++r) {
      const bool yes = v < s.end && sees(u, r, key, p.window, p.sinks);
      CHECK(yes == (r >= see.x && r < see.y));
      any |= yes;
      all &= yes;
    }
    CHECK(live.has(k) == any || (live.has(k) && v < s.end && key <= last_pos));
    if (any) CHECK(live.has(k));
    if (inner) CHECK(all);
    if (live.has(k)) CHECK(key < u.len);
  }
  for (int h = 0; h < 2; ++h) {
    const WindowKeys half = live_keys(p, live_of(s, key0, p.sinks), kStageKeys * h);
    bool every = true;
    for (int k = 0; k < kStageKeys; ++k) {
      every &= half.has(k);
      CHECK(half.has(k) == live.has(kStageKeys * h + k));
    }
    CHECK(!half.all() || every);
  }
}

// A tile of the prompts' kernel: its masks, and where its keys lie among the sequence's.
static void masks(const PromptParams& p, const PromptUnit& u, const Span& s, int key0, int last_pos, int batch) {
  const int last_lo = last_pos >= p.window ? last_pos - p.window + 1 : 0;
  const bool inner = sees_all(s, key0, u.pos, last_lo, p.sinks);
  const int n = std::min(kKeys, s.end - key0);
  for (int k = 0; k < kKeys; ++k) {
    const int v = key0 + k, key = v < s.s16 ? v : v + s.shift;
    for (int r = 0; r < kPromptRows; r += 1 + r % 5) {
      const bool yes = row_keys(u, s, r, p.window).has(v, p.sinks);
      if (r >= unit_rows(u)) {
        CHECK(!yes);
        continue;
      }
      CHECK(yes == (v < s.end && sees(u, r, key, p.window, p.sinks)));
      CHECK(yes == (row_keys(u, s, r, p.window).bits(v & ~63, p.sinks) >> (v & 63) & 1));
      if (inner) CHECK(yes);
    }
    if (k >= ((n + 15) & ~15)) continue;  // not copied
    const int g = group_of(u, s, v), at = 16 * g, s16 = s.s16;
    CHECK(g >= 0 && g < u.groups);
    CHECK((at < s16 ? at : at + u.shift0) == (key & ~15));
  }
}

template <class P>
static int check(int batches, bool many) {
  std::mt19937 rng(7);
  auto pick = [&](long long lo, long long hi) { return (int)(lo + (long long)(rng() % (unsigned long long)(hi - lo + 1))); };
  static P p;
  static MergeParams m;
  for (int batch = 0; batch < batches; ++batch) {
    const bool big = batch % 50 == 49;  // more units than one launch takes
    const int n_seq = big ? (many ? pick(70, 150) : pick(300, 700)) : pick(1, 12), max_ctas = pick(1, 3) == 1 ? pick(1, 7) : many ? 76 : 152;
    const int win[] = {1, 2, 15, 16, 17, pick(1, 300), pick(1, 3000), kAllKeys}, snk[] = {0, 0, 1, 4, 16, 17, pick(0, 300), kAllKeys};
    p.window = win[pick(0, 7)];
    p.sinks = snk[pick(0, 7)];
    p.n_kv_heads = pick(1, 4);
    std::vector<int32_t> lens(n_seq), fresh(n_seq);
    uint32_t most = 0;
    long long tokens = 0;
    for (int i = 0; i < n_seq; ++i) {
      fresh[i] = pick(0, 3) == 0 ? 0 : pick(0, 2) == 0 && !big ? pick(1, 120) : many && pick(0, 5) ? pick(64, 700) : pick(1, 8);
      lens[i] = fresh[i] + (pick(0, 2) == 0 ? pick(0, 5) : pick(0, big ? 300 : 4000));
      most = std::max(most, (uint32_t)fresh[i]);
      tokens += fresh[i];
    }
    for (int32_t& n : fresh) tokens -= Batch::is_many(n) != many ? n : 0;  // the other kernel's
    const Batch b{lens.data(), fresh.data(), (uint32_t)n_seq, p.window, p.sinks, p.n_kv_heads};
    p.slot_rows = m.slot_rows = many ? kPromptRows : slot_rows_of(most);
    uint32_t prompt_seq = 0;
    int group0 = 0;
    std::map<std::tuple<int, int, int>, int> rows_seen;  // (sequence, head, query row) -> times
    Cursor at{0, 0, 0};
    int launches = 0;
    while (at.seq < (uint32_t)n_seq) {
      const Cursor before = at;
      const Plan plan = plan_chunk(p, m, b, many, max_ctas, &at);
      CHECK(at.seq > before.seq || at.rt > before.rt);
      if (at.seq == before.seq && at.rt == before.rt) return 1;
      if (p.n_units == 0) break;
      ++launches;
      if constexpr (kPrompt<P>) {
        place_prompts(p, b, &prompt_seq, &group0);
        if (list_segments(p, plan)) {  // every segment once, some for every pair
          std::set<int> once;
          CHECK(p.first[0] == 0 && p.first[p.n_ctas] == p.n_units * p.n_kv_heads);
          for (int i = 0; i < p.n_ctas; ++i) CHECK(p.first[i] < p.first[i + 1]);
          for (int i = 0; i < p.first[p.n_ctas]; ++i) CHECK(p.list[i] < p.n_units * p.n_kv_heads && once.insert(p.list[i]).second);
          ++listed;
        }
      }
      CHECK(p.n_units <= P::kMaxUnits && p.n_ctas >= 1 && p.n_ctas <= max_ctas && plan.cuts < kMaxCtas);
      std::map<std::pair<int, int>, std::pair<int, int>> pieces;  // (unit, head) -> (first CTA, pieces) where cut
      int tile = 0;
      std::set<int> slots;
      std::vector<int> next_j((size_t)p.n_units * p.n_kv_heads, 0);
      for (int cta = 0; cta < p.n_ctas; ++cta) {
        const int x0 = (int)((long long)cta * p.total_len / p.n_ctas), x1 = (int)((long long)(cta + 1) * p.total_len / p.n_ctas);
        Pos t = locate(p, x0);
        const int end = x1 < p.total_len ? locate(p, x1).tile : p.total_tiles;
        CHECK(t.tile == tile && end > tile);
        CHECK(p.start[cta].tile == t.tile && p.start[cta].j == t.j && p.start[cta].unit_head == (t.unit | t.head << 16) &&
              p.start[cta + 1].tile == end);
        for (bool fresh_seg = t.j == 0; tile < end; ++tile) {
          CHECK(t.unit < p.n_units && t.head < p.n_kv_heads);
          const auto& u = p.unit[t.unit];
          CHECK(next_j[(size_t)t.unit * p.n_kv_heads + t.head]++ == t.j);
          const Span s = span_of(u, p.window, p.sinks);
          const int key0 = t.j * kKeys, last_pos = u.pos + (unit_row0(u) + unit_rows(u) - 1) / kGqa;
          const bool ends = t.j + 1 == t.nt, last = ends || tile + 1 == end;
          if (last) {
            const int slot = slot_of(fresh_seg, ends, cta, p.slot_rows);
            CHECK((slot < 0) == (fresh_seg && ends));
            if (slot >= 0) {
              CHECK(slots.insert(slot).second && slot + unit_rows(u) <= 2 * p.n_ctas * p.slot_rows && slot % p.slot_rows == 0);
              auto& pc = pieces[{t.unit, t.head}];
              if (pc.second == 0) pc.first = cta;
              CHECK(pc.first + pc.second == cta && slot == (2 * cta + (pc.second == 0 ? 1 : 0)) * p.slot_rows);
              ++pc.second;
            }
          }
          // the masks of a head's tiles
          if (t.head == 0 && (big ? pick(0, 30) == 0 : true)) masks(p, u, s, key0, last_pos, batch);
          if (t.j == 0) {
            for (int r = 0; r < unit_rows(u); ++r) {
              const int tok = u.token + (unit_row0(u) + r) / kGqa;
              ++rows_seen[{u.seq, t.head, tok * kGqa + (unit_row0(u) + r) % kGqa}];
            }
            // a row's visible keys are all in the order, and its first one in the first tile of any piece with one
            for (int r = 0; r < unit_rows(u); r += 7) {
              const int pos = u.pos + (unit_row0(u) + r) / kGqa, lo = pos >= p.window ? pos - p.window + 1 : 0;
              CHECK(lo >= s.lo && pos - s.shift < s.end && (s.shift == 0 || lo >= s.s16 + s.shift));
              CHECK(lo - s.shift - (s.lo - s.shift) < kKeys - kGroup);
            }
          }
          if (tile + 1 < end) {
            const int unit = t.unit, head = t.head;
            advance(p, t);
            if (t.unit != unit || t.head != head) fresh_seg = true;
          }
        }
      }
      CHECK(tile == p.total_tiles);
      for (size_t i = 0; i < next_j.size(); ++i)
        CHECK(next_j[i] == tiles_of(p.unit[i / p.n_kv_heads], p.window, p.sinks));
      CHECK((int)pieces.size() == plan.cuts);
      for (int i = 0; i < plan.cuts; ++i) {
        const Cut& c = m.cut[i];
        bool found = false;
        for (const auto& [key, pc] : pieces) {
          const Unit& u = p.unit[key.first];
          if (u.seq == c.seq && u.token == c.token && u.rows_row0 == c.rows_row0 && key.second == c.head) {
            found = true;
            CHECK(pc.first == c.cta && pc.second == c.n && u.len == c.len && unit_rows(u) <= plan.rows);
          }
        }
        CHECK(found);
      }
    }
    long long rows = 0;
    for (const auto& r : rows_seen) {
      CHECK(r.second == 1);
      ++rows;
    }
    CHECK(rows == tokens * kGqa * p.n_kv_heads);
    if (big) CHECK(launches >= 1);
  }
  return 0;
}

// The rule for pa_step_kernel: a cluster that its launch may have, the device well filled, never for other batches.
int check_steps() {
  struct Step {
    int n_seq, keys, want;
  };
  const Step steps[] = {{64, 1, 1}, {64, 1024, 1}, {76, 64, 1}, {77, 4096, 0}, {60, 64, 0}, {33, 512, 2}, {33, 255, 0}, {16, 512, 4}, {16, 511, 0},
                        {8, 1024, 8}, {8, 1023, 0}, {7, 4096, 0}, {1, 30000, 0}, {128, 256, 1}, {128, 255, 0}, {300, 512, 1}};
  int batch = 0;
  for (const Step& t : steps) {
    ++batch;
    std::vector<int32_t> lens(t.n_seq + 2, t.keys), n_new(t.n_seq + 2, 1);
    lens[0] = 9, n_new[0] = 0;
    n_new[t.n_seq + 1] = 0;
    auto cluster = [&](int window) {
      Batch b{lens.data(), n_new.data(), (uint32_t)lens.size(), clamp_keys(window ? window : ~0u), 0, 4};
      pa_pool_desc d = {};
      d.n_kv_heads = 4;
      CHECK(check_batch(d, ~0u, &b) == PA_OK);
      return step_cluster(b, 152);
    };
    CHECK(cluster(0) == t.want);
    for (int i = 1; i <= t.n_seq; ++i) lens[i] += 7000 + i;  // a window makes sequences of different lengths equal
    CHECK(cluster(t.keys) == t.want);
    if (t.n_seq > 1) {
      lens[1] += 20000;
      CHECK(cluster(0) == 0);
      lens[1] -= 20000;
    }
    n_new[t.n_seq + 1] = kPromptTokens;  // whatever else the batch holds for other kernels
    lens[t.n_seq + 1] = 30000;
    CHECK(cluster(t.keys) == t.want);
    n_new[1] = 2;
    CHECK(cluster(t.keys) == 0);
  }
  return 0;
}

int main(int argc, char** argv) {
  const int batches = argc > 1 ? std::atoi(argv[1]) : 300;
  if (check_steps() || check<WindowParams>(batches, false) || check<PromptParams>(batches, true)) return 1;
  std::printf("mismatches %lld, %lld launches of whole segments\n", bad, listed);
  return bad != 0 || listed == 0;
}

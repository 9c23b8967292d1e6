// Work lists of the chunk attention planner, worked out by its own source on the
// CPU.  Plans on stdin, one after another in one process (each finds the shared
// memory of the one before):
//   order num_seqs num_tokens num_kv_heads group rows causal cap ctas max_tiles max_merges max_slots
//   q_starts[num_seqs + 1] context_lens[num_seqs]
// Out: "error n_entries n_merges", then the entries and the merges, a line each.
// A write outside the arrays ends the program with exit code 3, a dead wait with 4.
#include "block.h"

#include "plan_source.h"

int main() {
  int order, S, T, heads, group, rows, causal, cap, ctas, max_tiles, max_merges, max_slots;
  while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d %d", &order, &S, &T, &heads, &group, &rows, &causal, &cap, &ctas,
                    &max_tiles, &max_merges, &max_slots) == 12) {
    std::vector<int> starts(S + 1), lens(S);
    for (int& x : starts)
      if (std::scanf("%d", &x) != 1) return 2;
    for (int& x : lens)
      if (std::scanf("%d", &x) != 1) return 2;
    constexpr int kGuard = 4096;
    const int max_entries = max_tiles + max_slots;
    std::vector<pa::PrefillEntry> entries(max_entries + kGuard);
    std::vector<pa::PrefillMerge> merges(max_merges + kGuard);
    std::vector<int> ends(S + kGuard, -7), steps(max_tiles + kGuard, -7);
    std::memset(static_cast<void*>(entries.data()), 0x7f, sizeof(pa::PrefillEntry) * entries.size());
    std::memset(static_cast<void*>(merges.data()), 0x7f, sizeof(pa::PrefillMerge) * merges.size());
    pa::PrefillHeader header{-1, -1};
    pa::PrefillPlanParams p{};
    p.q_starts = starts.data();
    p.context_lens = lens.data();
    p.header = &header;
    p.tile_ends = ends.data();
    p.entries = entries.data();
    p.merges = merges.data();
    p.num_seqs = S;
    p.num_tokens = T;
    p.num_kv_heads = heads;
    p.group = group;
    p.rows = rows;
    p.causal = causal;
    p.cap = cap;
    p.ctas = ctas;
    p.max_tiles = max_tiles;
    p.max_merges = max_merges;
    p.max_slots = max_slots;
    p.tile_steps = steps.data();
    p.cost = rows == pa::kPrefillRows16 ? pa::kPlanCost16 : pa::kPlanCost32;
    emu::device_error = 0;
    if (!emu::run(pa::kPrefillPlanThreads, emu::order_of(pa::kPrefillPlanThreads, order),
                  [&] { pa::prefill_plan_kernel(p); }))
      return 4;
    auto untouched = [](const void* b, size_t n, unsigned char v) {
      const unsigned char* c = static_cast<const unsigned char*>(b);
      return std::all_of(c, c + n, [&](unsigned char x) { return x == v; });
    };
    const bool fine = untouched(&entries[max_entries], kGuard * sizeof(entries[0]), 0x7f) &&
                      untouched(&merges[max_merges], kGuard * sizeof(merges[0]), 0x7f) &&
                      std::all_of(ends.begin() + S, ends.end(), [](int x) { return x == -7; }) &&
                      std::all_of(steps.begin() + max_tiles, steps.end(), [](int x) { return x == -7; }) &&
                      header.num_entries >= 0 && header.num_entries <= max_entries && header.num_merges >= 0 &&
                      header.num_merges <= max_merges;
    if (!fine) return 3;
    std::printf("%d %d %d\n", emu::device_error, header.num_entries, header.num_merges);
    for (int i = 0; i < header.num_entries; ++i) {
      const pa::PrefillEntry& e = entries[i];
      std::printf("%d %d %d %d %d %d %d %d\n", e.seq, e.tok0, e.ntok, e.step0, e.step1, e.ctx, e.lim0, e.slot);
    }
    for (int i = 0; i < header.num_merges; ++i)
      std::printf("%d %d %d %d\n", merges[i].tok0, merges[i].ntok, merges[i].slot0, merges[i].pieces);
    std::fflush(stdout);
  }
  return 0;
}

// Walks through every interleaving of the four warps of a group over the ring of key
// stages (csrc/kv4_ring.cuh, the code that the kernel runs) and of the copies' arrivals.
// The steps of a warp do not depend on the interleaving, so they are recorded once; a
// state is where each warp stands and what the slots and barriers hold.
//
//   ring_walk D KEYS BASE [skip]   prints "states N" or the first fault, exit code 1
//
// skip leaves out the wait for a stage that the warp does not read (a planted mistake).
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>
#include <unordered_set>
#include <vector>

#include "kv4_ring.cuh"

namespace {
enum Kind { kFull, kRead, kRelease, kRefill };
struct Step {
  Kind kind;
  int stage, slot;
  uint32_t parity;
};

// The group's slots: stage held (copied or on its way), phases completed.
struct Slot {
  int8_t stage;     // -1 none
  int8_t copying;   // 1: `full` of the stage has not completed
  int8_t full;      // completed phases of the two barriers
  int8_t empty;
  int8_t arrivals;  // in the current phase of `empty`
};
constexpr int kMaxSlots = 4, kWarps = fc::kRingWarps;
struct State {
  int16_t at[kWarps];
  Slot slot[kMaxSlots];
};

template <int S>
int walk(int keys, int base, int group, bool skip, size_t& states) {
  constexpr int kOwn = S / fc::kRingGroups;
  static_assert(kOwn <= kMaxSlots, "slots");
  const int n_stages = (keys + kWarps * fc::kRingKeys - 1) / (kWarps * fc::kRingKeys);
  int i0 = 0;  // the group's first stage: slots stay with their group
  while ((base + i0) % fc::kRingGroups != group) ++i0;
  std::vector<Step> steps[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    std::vector<Step>& s = steps[w];
    const int own = fc::ring_own_stages(keys, w);
    int last = 0, before = 0;  // stages whose logits, values come
    fc::ring_walk<S>(
        base, i0, own, n_stages,
        [&](int i, int slot, uint32_t parity) {
          if (!(skip && i >= own)) s.push_back({kFull, i, slot, parity});
          before = last;
          last = i;
          return true;
        },
        [&](int slot) { s.push_back({kRead, last, slot, 0}); },
        [&](int, int) {},
        [&](int slot) {
          s.push_back({kRead, (base + last) % S == slot ? last : before, slot, 0});
        },
        [&](int slot) { s.push_back({kRelease, 0, slot, 0}); },
        [&](int i, int slot, uint32_t parity) {
          if (fc::ring_refills<S>(i, w, n_stages)) s.push_back({kRefill, i + S, slot, parity});
        },
        [] { return true; });
  }
  State first;
  memset(&first, 0, sizeof first);
  for (int k = 0; k < kMaxSlots; ++k) first.slot[k].stage = -1;
  auto own_slot = [&](int slot) { return slot / fc::kRingGroups; };
  for (int x = 0; x < base; ++x)
    if (x % fc::kRingGroups == group) {
      ++first.slot[own_slot(x % S)].full;
      ++first.slot[own_slot(x % S)].empty;
    }
  State last = first;
  for (int i = i0; i < n_stages; i += fc::kRingGroups) {
    Slot& l = last.slot[own_slot((base + i) % S)];
    ++l.full, ++l.empty;
    if (i < S) {
      Slot& f = first.slot[own_slot((base + i) % S)];
      f.stage = (int8_t)i, f.copying = 1;
    }
  }
  auto done = [](int completed, uint32_t parity) {  // mbarrier.try_wait.parity
    return ((uint32_t)completed & 1u) != parity;
  };
  std::unordered_set<std::string> seen;
  std::vector<State> todo{first};
  auto key = [](const State& s) { return std::string((const char*)&s, sizeof s); };
  seen.insert(key(first));
  auto push = [&](const State& s) {
    if (seen.insert(key(s)).second) todo.push_back(s);
  };
  auto fault = [&](const char* what, int w, const Step& s) {
    printf("%s: warp %d, stage %d, slot %d\n", what, w, s.stage, s.slot);
    return 1;
  };
  bool ended = false;
  while (!todo.empty()) {
    const State st = todo.back();
    todo.pop_back();
    bool moved = false, over = true;
    for (int k = 0; k < kOwn; ++k)  // a copy arrives
      if (st.slot[k].copying) {
        State n = st;
        n.slot[k].copying = 0;
        ++n.slot[k].full;
        push(n);
        moved = true, over = false;
      }
    for (int w = 0; w < kWarps; ++w) {
      if (st.at[w] == (int)steps[w].size()) continue;
      over = false;
      const Step& s = steps[w][st.at[w]];
      const Slot& at = st.slot[own_slot(s.slot)];
      State n = st;
      Slot& to = n.slot[own_slot(s.slot)];
      ++n.at[w];
      if (s.kind == kFull) {
        if (!done(at.full, s.parity)) continue;
        if (at.stage != s.stage || at.copying) return fault("early answer", w, s);
      } else if (s.kind == kRead) {
        if (at.stage != s.stage || at.copying) return fault("overwritten", w, s);
      } else if (s.kind == kRelease) {
        if (++to.arrivals == kWarps) to.arrivals = 0, ++to.empty;
      } else {
        if (!done(at.empty, s.parity)) continue;
        if (at.copying) return fault("two copies", w, s);
        to.stage = (int8_t)s.stage;
        to.copying = 1;
      }
      push(n);
      moved = true;
    }
    if (over) {
      ended = true;
      for (int k = 0; k < kOwn; ++k)
        if (st.slot[k].full != last.slot[k].full || st.slot[k].empty != last.slot[k].empty ||
            st.slot[k].arrivals != 0)
          return fault("phases at the end", -1, Step{kFull, 0, k, 0});
    } else if (!moved) {
      return fault("nobody can go on", -1, Step{kFull, 0, 0, 0});
    }
  }
  states += seen.size();
  return ended ? 0 : 1;
}
}  // namespace

int main(int argc, char** argv) {
  if (argc < 4) return 2;
  const int d = atoi(argv[1]), keys = atoi(argv[2]), base = atoi(argv[3]);
  const bool skip = argc > 4 && strcmp(argv[4], "skip") == 0;
  size_t states = 0;
  for (int group = 0; group < fc::kRingGroups; ++group) {
    const int r = d == 128 ? walk<fc::ring_slots(128)>(keys, base, group, skip, states)
                           : walk<fc::ring_slots(64)>(keys, base, group, skip, states);
    if (r != 0) return r;
  }
  printf("states %zu\n", states);
  return 0;
}

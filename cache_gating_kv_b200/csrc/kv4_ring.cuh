// The ring of key stages of the attention for few rows: which warp waits, reads,
// releases and refills in which order.  Apart from the kernel so that a host program
// can walk through all interleavings of a group of warps (no CUDA header is needed).
//
// Stage i of a piece lies in slot (base + i) % S, in phase (base + i) / S of the
// slot's two barriers: `full` completes with the bytes of the copies, `empty` with one
// arrival of each warp of the group that the slot belongs to.  `empty` counts arrivals,
// not warps, and a wait for a parity is answered by the phase two before it as well.
// So every warp of the group waits for `full` of every stage of the group, in order,
// and releases it once, behind that wait, whether it has keys there or not: stage i is
// copied only after `empty` of stage i - S has completed, so no arrival can fall into
// an earlier phase, and no wait can start two phases early.  (A warp that released the
// last stage, in which it has no keys, without the wait could arrive twice in the
// phase of stage last - S, and the copy overwrote what a slower warp still read.)
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FC_RING_FN __device__ __forceinline__
#else
#define FC_RING_FN inline
#endif

namespace fc {

constexpr int kRingGroups = 2;  // groups of warps, taking stages in turn
constexpr int kRingWarps = 4;   // warps of a group, 32 keys of a stage to each
constexpr int kRingKeys = 32;   // of a warp
// Slots: a multiple of the groups, so that a slot always belongs to one of them.
constexpr int ring_slots(int d) { return d == 128 ? 6 : 8; }

// Stages of a piece of `keys` keys in which a warp (of the group) has keys.
FC_RING_FN int ring_own_stages(int keys, int warp) {
  constexpr int kStage = kRingWarps * kRingKeys;
  const int off = warp * kRingKeys;
  return keys > off ? (keys - off + kStage - 1) / kStage : 0;
}
// The warp that refills the slot of stage i, if there is a stage to come.
template <int S>
FC_RING_FN bool ring_refills(int i, int warp, int n_stages) {
  return i + S < n_stages && (i / kRingGroups) % kRingWarps == warp;
}

// A warp's way through the stages i, i + 2, .. of a piece of n_stages, with keys of its
// own in those below n_own.  The values of a stage and the logits of the next are
// independent work for one instruction stream; the slot is refilled a softmax after
// the warp's own release, when the others have released it too.
//   full(i, slot, parity)    waits for a stage; false when the wait gave up
//   logits(slot), softmax(i, slot), values(slot)
//   release(slot)            the warp's arrival on `empty`
//   refill(i, slot, parity)  behind the release of stage i
//   sound()                  whether no wait of the warp has given up
template <int S, class Full, class Logits, class Softmax, class Values, class Release,
          class Refill, class Sound>
FC_RING_FN void ring_walk(int base, int i, int n_own, int n_stages, Full&& full, Logits&& logits,
                          Softmax&& softmax, Values&& values, Release&& release, Refill&& refill,
                          Sound&& sound) {
  static_assert(S % kRingGroups == 0, "a slot belongs to one group");
  int slot = (base + i) % S;
  uint32_t parity = ((base + i) / S) & 1;
  if (i < n_own && full(i, slot, parity)) {
    logits(slot);
    softmax(i, slot);
    for (int nx = i + kRingGroups; nx < n_own; nx += kRingGroups) {
      int to = slot + kRingGroups;
      uint32_t to_parity = parity;
      if (to >= S) {
        to -= S;
        to_parity ^= 1;
      }
      if (!full(nx, to, to_parity)) break;
      logits(to);
      values(slot);
      release(slot);
      softmax(nx, to);
      refill(i, slot, parity);
      i = nx;
      slot = to;
      parity = to_parity;
    }
    if (sound()) values(slot);
  }
  // The last stage of its own, and one in which it has no keys: the wait is the order
  // in which arrivals reach `empty` (see above).  Behind a wait that gave up, releases
  // only: every phase has its arrivals.
  for (; i < n_stages; i += kRingGroups) {
    const int at = (base + i) % S;
    if (sound()) full(i, at, ((base + i) / S) & 1);
    release(at);
  }
}

}  // namespace fc

// How many slots and barriers take turns in the pipelines of the tensor-core cross-attention kernels:
// plain C++, so that a host test can walk the kernels' barrier protocols with the numbers that the
// kernels are compiled with (tests/test_barrier_protocols.py).
//
// A wait names a phase by its parity, so it is sound only while the phase before it has completed and
// the phase after it cannot: whoever waits has to follow every phase of the barrier, and whoever
// completes the next phase has to depend on the waiter.
#pragma once

namespace p3d {
namespace xa {

constexpr int kTile = 128;              // rows or states of a tile
constexpr int kSmemLimit = 232448;      // shared memory of a CTA
constexpr int kSmemLimitOfTwo = 116736;  // and of each of two CTAs on an SM, 1 KB of which is the system's
constexpr int row_bytes(int rows, int d) { return rows * d * 2; }  // bf16
constexpr int at_most(int n, int most) { return n < most ? n : most; }

// ---- k_cross_fwd (o, lse)
constexpr int kFwdTile = 64;  // states of a tile
// sums and references of the rows, two buffers of two row tiles, then the ring; barriers behind it
constexpr int fwd_ring_at(int d) { return 4096 + 4 * row_bytes(kTile, d); }
// Slots of the ring in which K and V tiles take turns (item 2 j is K of the j-th tile, 2 j + 1 its V).
// An even number: K and V then have slots of their own, and the warps that wait for K alone (or V
// alone) follow every phase of those slots' barriers. At head_dim 128 five would fit.
constexpr int fwd_slots(int d) {
  return at_most((kSmemLimit - 1024 - 512 - fwd_ring_at(d)) / row_bytes(kFwdTile, d), 8) & ~1;
}
constexpr int fwd_bufs(int d) { return d <= 96 ? 2 : 1; }  // of S
// Barriers of V tiles whose masked rows are cleared: more than the V tiles of the ring
constexpr int kFwdReady = 8;

// ---- k_cross_dq (dq)
constexpr int dq_ring_at(int d) { return 2 * row_bytes(kTile, d); }
// Slots in which V and K tiles of 64 states take turns. An odd number is sound here: the warps that
// wait see both items of every step.
constexpr int dq_slots(int d) {
  return at_most((kSmemLimitOfTwo - 1024 - 512 - dq_ring_at(d)) / row_bytes(64, d), 6);
}
constexpr bool dq_own(int d) { return d <= 96; }  // dS has tensor memory of its own
constexpr int kDqReady = 8;

// ---- k_cross_dkv (dk, dv), head_dim d
// stages of 64 rows; even: a group of elementwise warps, which takes every second step, then sees the
// same slots and all of their phases
constexpr int dkv_stages(int d) { return d <= 96 ? 6 : 4; }
// five slots of S, dP, P and dS in tensor memory, or four
constexpr bool dkv_five(int d) { return d <= 96; }
// Barriers that "P and dS written" and "products done" of consecutive steps take turns on. With two,
// step i + 2 would share step i's: with five slots its scores wait for the products of step i - 1
// alone, so a warp two steps ahead could arrive for a slower one of its group, and the phase of step
// i + 2 could complete while the warp that issues the products still waits for step i's (or the
// warp that issues the scores for that of step i - 3 while step i - 1's completes). Step i + 4's
// scores wait for the products of step i + 1.
constexpr int kDkvTurns = 4;

// ---- k_cross_fwd_short (o, lse of at most 128 states)
// Barriers of staged output rows, in turn as the two buffers of rows are. With one, the rows of tile
// n + 1, which wait for the store of tile n - 1 alone, could complete the next phase while the
// storing warp still waits for those of tile n.
constexpr int kShortTurns = 2;

}  // namespace xa
}  // namespace p3d

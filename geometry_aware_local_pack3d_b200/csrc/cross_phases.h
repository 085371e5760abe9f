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

}  // namespace xa
}  // namespace p3d

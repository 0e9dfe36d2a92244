// Addresses of the 8-bit integer products that depend on the end of K. Plain C++
// (constexpr functions run on the device too), so that a program on the host can
// check them.
#pragma once

namespace moe {

// Values of K that a step of a wave of the few-rows kernel covers.
constexpr int kI8Step = 128;

// A lane's load of weights in the few-rows kernel: 16 values of its weight row, of
// the 64 of half h (0, 1) of the step that begins at k those of its group of lanes
// (0 to 3).  They begin at a multiple of 16 below K, as K does, or count for
// nothing.
constexpr int i8_weights_at(int k, int h, int grp) { return k + 64 * h + 16 * grp; }
constexpr bool i8_weights_count(int k, int h, int grp, int K) { return i8_weights_at(k, h, grp) < K; }
// The value of the row at which the load begins: where it counts for nothing the
// first, from which 16 lie in the row whatever K (at least 16).
constexpr int i8_weights_load(int k, int h, int grp, int K) {
    return i8_weights_count(k, h, grp, K) ? i8_weights_at(k, h, grp) : 0;
}

}  // namespace moe

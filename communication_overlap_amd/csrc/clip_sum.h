// What wavefronts and workgroups of the gradient norm hand on: one float64,
// the sum of squares of their gradients, which is 0 or more, infinite or NaN
// whatever the gradients hold, or kClipForeign where they met a table entry
// that is not their plan's.  The verdict is read off every term before it is
// added: in the total it would be lost beside an infinity or a NaN.
#pragma once

namespace ovl {

constexpr double kClipForeign = -1.0;

struct ClipTotal {
  double sum = 0;
  bool foreign = false;

  constexpr void add(double v) {
    foreign |= v < 0;
    sum += v;  // means nothing once there is a foreign term
  }
  constexpr double word() const { return foreign ? kClipForeign : sum; }
};

}  // namespace ovl

// The columns that one of a row's threads takes (not part of the ABI). Plain
// C++, which a host program can walk too.
#pragma once

namespace dgw4 {

// f(k) for k = first, first + STEP, ... below end. The position is unsigned:
// end may be any int, and the step that leaves the loop may pass 2^31 (first
// and STEP are below 2^16).
template <unsigned STEP, class F>
constexpr void each_column(int first, int end, F &&f)
{
    for (unsigned k = (unsigned)first; k < (unsigned)end; k += STEP)
        f((int)k);
}

}  // namespace dgw4

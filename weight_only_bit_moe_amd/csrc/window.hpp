// The part of an operand's memory that one copy of a few rows may read.
#pragma once

#include <stdint.h>

#ifndef __HIPCC__
#define __host__
#define __device__
#endif

namespace wna16 {

struct Window {
    long long start;        // bytes behind the operand's first row
    uint32_t bytes;
};

// Rows [first, first + n) of `rows` that lie ld bytes apart and hold K each (K <= ld), for
// lanes that read row r of the n at r * ld + column + k, column and k of a piece inside the row.
// A buffer's range check compares the lane's own offset with its size; whether it adds the wave's
// offset k, and what it makes of one past the size, is not relied on:
//   - rows past the end are outside by r * ld alone, at least (their number) * ld >= bytes;
//   - rows inside are inside with column + k;
//   - k < K <= bytes always: without a row left, the window is the last row's.
__host__ __device__ constexpr Window window_of(int first, int n, int rows, uint32_t ld, uint32_t K)
{
    const int at = first < rows ? first : rows - 1;
    const int left = rows - at < n ? rows - at : n;
    return Window{(long long)at * ld, (uint32_t)(left - 1) * ld + K};
}

}  // namespace wna16

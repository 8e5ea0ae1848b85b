// What one launch can hold.
#pragma once

#include <cstddef>

namespace specv {

// A launch has fewer than 2^32 work-items.  A call whose grid would have more
// is refused before anything is enqueued.
inline bool grid_fits(size_t blocks, size_t threads) { return blocks <= 0xffffffffu / threads; }

}  // namespace specv

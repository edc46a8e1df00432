// expert_access.h -- where the experts' kernels may take whole 16-byte pieces of a row: address
// arithmetic alone, the same in kernels, launchers and host programs (constexpr functions are
// both host and device code).
#pragma once

#include <stdint.h>

namespace ctr {

// Whether rows of `width` elements of `size` bytes, `stride` elements apart from address `p` on,
// are whole aligned pieces.  The width counts also where there are no rows (p is 0 then): what is
// written for them, as the bias gradient of no rows, has the same width.
constexpr bool whole_pieces(uintptr_t p, int64_t stride, int64_t width, int size) {
  return p % 16 == 0 && stride * size % 16 == 0 && width * size % 16 == 0;
}

// A piece of `count` elements that begins at column `first` of a row of `width`, count <= width:
// the column where it is read whole, inside the row, and by how many elements what belongs at
// `first` then comes later in it.  A piece that is wholly past the row holds any of its elements.
struct PieceAt {
  int64_t column;
  int down;
};
constexpr PieceAt piece_at(int64_t first, int64_t width, int count) {
  return first + count <= width ? PieceAt{first, 0}
         : first < width        ? PieceAt{width - count, (int)(first + count - width)}
                                : PieceAt{width - count, 0};
}

}  // namespace ctr

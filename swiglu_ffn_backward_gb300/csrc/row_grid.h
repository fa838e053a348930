// Grid sizes of the persistent row-wise kernels (host arithmetic only).
#pragma once

#include <stdint.h>

namespace swg {

// Blocks (or clusters) of a kernel whose groups take row after row, `fit` of which run at once and `need` of
// which give every group at most one row. multiple: a group's rows have to lie so many rows (or a multiple)
// apart, because it keeps what belongs to one offset within 16 bytes; so where groups take several rows, the
// number of blocks is a multiple of it. 0 where too few fit for that (a small part of a device): the kernel
// cannot take these rows.
inline int64_t persistent_blocks(int64_t fit, int64_t need, int64_t multiple) {
  return need <= fit ? need : fit - fit % multiple;
}

}  // namespace swg

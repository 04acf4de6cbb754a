// row_pieces.cuh -- which of the 16-byte pieces of memory that cover a row of a dense tensor [rows, D] hold nothing but
// the tensor. Arithmetic on elements alone, without anything of CUDA's, so that a host compiler can check it too.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

// kShort: rows may be shorter than a piece, so that one next to the first or last row can reach past the tensor's end
// too. Otherwise D >= piece - 1, a neighbour on either side holds what a row's pieces have beside it, and only the first and
// last row are looked at: with the products for every row 16384 x 7001 bf16 took 209 us forward and 395 backward instead
// of 197 and 364.

// Whether all pieces (of `piece` elements) that cover a row with neighbours hold nothing but the tensor.
template <bool kShort>
MOE_HOST_DEVICE bool neighbours_cover(int32_t D, int piece) {
    return !kShort || D >= piece - 1;
}

// Whether the piece from the row's element `first` (negative: before the row) to its element `last` does.
template <bool kShort>
MOE_HOST_DEVICE bool piece_inside(int64_t row, int64_t rows, int32_t D, int first, int last) {
    if (kShort) return row * D + first >= 0 && row * D + last < rows * D;
    return (row > 0 || first >= 0) && (row < rows - 1 || last < D);
}

}  // namespace moe

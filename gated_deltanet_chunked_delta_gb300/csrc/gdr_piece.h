// gdr_piece.h -- which eight-element pieces of a row may be read whole
// (gdr_norm.cu).  Plain C++, so that the index arithmetic can be run on the
// host.  Not part of the ABI.
#pragma once

#ifdef __CUDACC__
#define GDR_BOTH __host__ __device__ __forceinline__
#else
#define GDR_BOTH inline
#endif

namespace gdr {

// Whether elements c .. c + 7, counted from the start of row `row`, lie between
// the first and the last element of M rows of D, `stride` elements apart.  c is
// negative for a piece that begins in the row before.
GDR_BOTH bool piece_inside(long long row, int c, long long M, int D, long long stride) {
    return stride >= D && row * stride + c >= 0 && c + 8 <= (M - 1 - row) * stride + D;
}

}  // namespace gdr

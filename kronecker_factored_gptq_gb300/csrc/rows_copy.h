// Which bytes of a 16-byte piece a copy of a row may read (plain C++, so that it
// can be checked without a GPU).
#pragma once

#ifdef __CUDACC__
#define BAKRON_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define BAKRON_HOST_DEVICE inline
#endif

namespace bakron {

struct PieceBytes {
  int from, to;      // bytes [from, to) of the piece, none when from >= to
};

// A row's columns lie in aligned 16-byte pieces, the first of which begins
// `shift` bytes in front of them.  `at`: the piece's place behind the first
// one's; `left`: bytes from the first piece on to the row's end; `before`: bytes of
// the array in front of the columns (16 stands for more).  What lies in front of them inside the
// first piece is read along with them where it belongs to the array, and left
// out where the array begins later (not in its first row alone: of rows shorter than
// 16 bytes several begin inside the array's first piece).
BAKRON_HOST_DEVICE PieceBytes piece_bytes(int before, int shift, int left, int at) {
  PieceBytes p;
  p.from = at == 0 && before < shift ? shift : 0;
  p.to = left - at < 16 ? left - at : 16;
  if (p.to < 0) p.to = 0;
  return p;
}

}  // namespace bakron

// Where the bytes of a matrix's rows lie, which operands share any, and when a
// team of threads leaves its loop over rows: arithmetic of the operators'
// kernels and host checks in plain C++, so that it can be tested without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>

#ifdef __CUDACC__
#define VRCCL_HD __host__ __device__ __forceinline__
#else
#define VRCCL_HD inline
#endif

namespace vrccl {

// What a call reads or writes: rows of `width` bytes, `pitch` apart (0: one run); nothing where p is NULL. bytes: from the
// first to the last.
struct Span {
  const void* p;
  size_t bytes, pitch, width;
};
inline Span vectorSpan(const void* p, size_t bytes) { return {p, bytes, 0, bytes}; }
inline Span matrixSpan(const void* p, size_t ld, size_t rows, size_t cols, size_t elemSize) {
  if (rows == 0 || cols == 0) return vectorSpan(p, 0);
  return {p, ((rows - 1) * ld + cols) * elemSize, rows > 1 ? ld * elemSize : 0, cols * elemSize};
}
// Whether two of them share a byte. Operands of one pitch may lie side by side
// (column slices of a wider buffer), a run between the rows of a matrix; of two
// pitches the whole ranges count.
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
  if (!a.p || !b.p || !a.bytes || !b.bytes || pa >= pb + b.bytes || pb >= pa + a.bytes) return false;
  const size_t pitch = a.pitch ? a.pitch : b.pitch;
  if (pitch == 0 || (a.pitch && b.pitch && a.pitch != b.pitch)) return true;
  const size_t from = pb >= pa ? (pb - pa) % pitch : (pitch - (pa - pb) % pitch) % pitch;  // where b's rows start in a's pitch
  return from < a.width || from + b.width > pitch;
}

// Where a row's bytes lie and which of them a bulk copy may take: the 16-byte
// blocks it touches that lie inside the matrix's own bytes, first row's start
// to last row's end. A row on no 16-byte boundary shares its first and last
// block with what is before and after it, which is copied and ignored. Its
// elements in blocks that the matrix's ends cut, [row, headEnd) and
// [tailBegin, end), are copied one by one.
struct Window {
  uintptr_t row, end, lo, hi;  // the row's elements; the blocks a bulk copy takes (lo == hi: none)
  VRCCL_HD uintptr_t headEnd() const { return lo < end ? lo : end; }
  VRCCL_HD uintptr_t tailBegin() const { return hi > row ? hi : row; }
};
// Rows at either end of the matrix that may touch a block which that end cuts: one, and more where rows are shorter than
// a block. (Told by their number, so that the rows between need no comparison of addresses: with it for every row
// backward passes over odd rows took 15 % longer.)
VRCCL_HD unsigned cutRows(size_t ld, unsigned elemSize) { return ld * elemSize > 14 ? 1 : 14 / ((unsigned)ld * elemSize) + 1; }
VRCCL_HD bool maybeCut(size_t row, size_t rows, unsigned cutAtEnds) { return row < cutAtEnds || row + cutAtEnds >= rows; }
VRCCL_HD Window rowWindow(uintptr_t base, size_t ld, size_t row, size_t rows, unsigned cols, unsigned elemSize,
                          unsigned cutAtEnds) {
  Window w;
  w.row = base + row * ld * elemSize;
  w.end = w.row + cols * elemSize;
  w.lo = w.row & ~(uintptr_t)15;
  w.hi = (w.end + 15) & ~(uintptr_t)15;
  if (maybeCut(row, rows, cutAtEnds)) {
    if (w.lo < base) w.lo += 16;
    if (w.hi > w.end + (rows - 1 - row) * ld * elemSize) w.hi -= 16;
    if (w.hi < w.lo) w.hi = w.lo;
  }
  return w;
}

// A team's word for a wait that was given up says in which turn it was, by the
// turn's parity (0 or 1). A turn has one barrier, after which every thread
// reads the word: it finds what was written before the barrier, or what a
// faster thread has already written in the next turn (not in a later one: that
// is another barrier on). The latter is the next turn's to act on, or the
// threads of a team would leave their loop at different barriers.
VRCCL_HD int givenUpWord(int turn) { return turn + 1; }
VRCCL_HD bool givenUp(int word, int turn) { return word == givenUpWord(turn); }

}  // namespace vrccl

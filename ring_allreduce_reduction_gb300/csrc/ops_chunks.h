// Rows in chunks of eight elements, one a lane, on whatever byte they start,
// and the generator of the dropout: arithmetic of the operators' kernels in
// plain C++, so that it can be tested without a GPU.
#pragma once

#include "ops_rows.h"

namespace vrccl {

constexpr int kChunk = 8;  // elements: 16 bytes of a 2-byte type, 32 of binary32

// Lanes of a warp hold consecutive chunks of a row: all 32, or 16 or 8 of them
// the whole of a short one.
struct Place {
  int lane, lanes;  // this one among those of its row
  int chunk, step;  // its chunk's number in the row; chunks that the lanes take at a time
};
// A row starts `skew` bytes (a multiple of the element's size E) after a
// 16-byte boundary. With skew > 0 a chunk's memory is the end of one 16-byte
// block, its head, and the beginnings of those after it: block i of a chunk is
// the 16 bytes from its byte 16 (i + 1) - skew on, the last one's end being the
// next lane's head. A block is stored at once if the row has all its elements
// (`left`: from the chunk's first to the row's end) and the lanes hold them;
// what lies in other blocks in pieces of 8, 4 and 2 bytes: a head ends, a rest
// begins on a boundary. (A head that the row ends in goes by elements.)
// The last lane's last block is never held. So a warp may take 31 chunks and
// hold the next one's first (step = lanes - 1): its last lane stores nothing,
// and pieces are left at the row's two ends alone. In place that is sound where
// the row starts on the same skew as what it overwrites: no other lane stores
// that head.
VRCCL_HD int headOf(unsigned skew) { return 16 - (int)skew; }
VRCCL_HD bool wholeBlock(int i, unsigned skew, int E, int left, const Place& at) {
  const int end = headOf(skew) + 16 * (i + 1);  // in bytes from the chunk's first
  return left * E >= end && (end <= kChunk * E || at.lane < at.lanes - 1);
}
// Whether the lane before stores this one's head.
VRCCL_HD bool headStored(unsigned skew, int E, int left, const Place& at) {
  return (at.step < at.lanes ? at.chunk : at.lane) > 0 && left * E >= headOf(skew);
}
// Bytes of the chunk in its block i, which is not whole.
VRCCL_HD int restOf(int i, unsigned skew, int E, int left) {
  return (left < kChunk ? left : kChunk) * E - headOf(skew) - 16 * i;
}
// Where the pieces of a head and of a rest of n bytes begin (of size 2, 4, 8: those whose bit n has).
VRCCL_HD int headPiece(int n, int size) { return n & (size - 1); }
VRCCL_HD int restPiece(int n, int size) { return n & (16 - 2 * size); }
// Chunks that a warp takes at a time of rows of `per` > 32: the pieces of 32 cost it a seventh of its time.
inline int stepOf(int per) { return (per + 30) / 31 * 7 <= (per + 31) / 32 * 8 ? 31 : 32; }
// Loading, a lane asks for the blocks that its row touches and that lie inside the matrix's own bytes [begin, end) ...
VRCCL_HD bool blockLoaded(uintptr_t block, uintptr_t rowEnd, uintptr_t begin, uintptr_t end) {
  return block < rowEnd && block >= begin && block + 16 <= end;
}
// ... and puts its chunk (from byte p, `left` elements to the row's end) together from them if they are all there; else it
// asks for the elements one by one.
VRCCL_HD bool fromBlocks(uintptr_t p, int E, int left, uintptr_t begin, uintptr_t end) {
  const uintptr_t last = p + (uintptr_t)((left < kChunk ? left : kChunk) * E);
  return (p & ~(uintptr_t)15) >= begin && ((last + 15) & ~(uintptr_t)15) <= end;
}

// Philox4x32-10: 128 random bits for a counter under a key (Salmon, Moraes,
// Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011). Ten rounds
// of two 32 x 32-bit products whose halves are crossed and mixed with the key,
// which grows by a constant a round.
struct Random128 {
  uint32_t w[4];
};
VRCCL_HD Random128 philox(uint64_t key, uint64_t counter, uint64_t stream) {
  uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
  uint32_t a = (uint32_t)counter, b = (uint32_t)(counter >> 32), c = (uint32_t)stream, d = (uint32_t)(stream >> 32);
#ifdef __CUDA_ARCH__
#pragma unroll
#endif
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = (uint64_t)0xD2511F53u * a, q = (uint64_t)0xCD9E8D57u * c;
    a = (uint32_t)(q >> 32) ^ b ^ k0;
    b = (uint32_t)q;
    c = (uint32_t)(p >> 32) ^ d ^ k1;
    d = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{a, b, c, d}};
}
// Element e of a chunk is decided by 16 of its 128 bits: it is kept if they are not below the threshold, `drop` of 65536.
// That is one comparison with last = 65536 drop - 1 for every drop but 0, where `all` are kept.
VRCCL_HD bool keeps(const Random128& r, int e, uint32_t last, bool all) {
  const uint32_t w = r.w[e >> 1];
  return (e & 1 ? w : w << 16) > last || all;  // (the lower half of w is below the threshold's one)
}
inline int dropThreshold(float p) { return (int)((double)p * 65536 + 0.5); }

// n / d for n below 2^31 by a 32-bit product: the upper half of n mul, shifted (d >= 2). mul is 2^(32 + shift) / d rounded up, too
// large by less than d / 2^(32 + shift) of 1; shift is the least with 2^(shift + 1) >= d, so that n times that stays below 1 / d,
// the least by which n / d misses the next integer.
struct Division {
  uint32_t mul, shift;
};
inline Division divisionOf(uint32_t d) {
  uint32_t shift = 0;
  while (((uint64_t)2 << shift) < d) ++shift;
  return {(uint32_t)((((uint64_t)1 << (32 + shift)) + d - 1) / d), shift};
}
VRCCL_HD uint32_t quotient(uint32_t n, const Division& by) { return (uint32_t)(((uint64_t)n * by.mul) >> 32) >> by.shift; }

}  // namespace vrccl

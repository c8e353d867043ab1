// Rows in chunks of eight elements, one a lane, on whatever byte they start,
// and the generator of the dropout: arithmetic of the operators' kernels in
// plain C++, so that it can be tested without a GPU.
#pragma once

#include "ops_rows.h"

namespace vrccl {

constexpr int kChunk = 8;  // elements: 16 bytes of a 2-byte type, 32 of binary32

// A warp's lanes hold consecutive chunks of a row that starts `skew` bytes
// (a multiple of the element's size E) after a 16-byte boundary. With skew > 0
// a chunk's memory is the end of one 16-byte block, and the beginnings of those
// after it: block i of a chunk is the 16 bytes from its byte 16 (i + 1) - skew
// on, the last one's end being the next lane's first bytes. A block is stored
// at once if the row has all its elements (`left`: from the chunk's first to
// the row's end) and the warp holds them; every other element by itself.
VRCCL_HD bool wholeBlock(int i, unsigned skew, int E, int left, int lane) {
  const int end = 16 * (i + 2) - (int)skew;  // in bytes from the chunk's first
  return left * E >= end && (end <= kChunk * E || lane < 31);
}
// What a chunk has before its first block lies in the last block of the lane before: whether that one is stored whole.
VRCCL_HD bool headStored(unsigned skew, int E, int left, int lane) { return lane > 0 && left * E >= 16 - (int)skew; }
VRCCL_HD bool storedSingly(int e, unsigned skew, int E, int left, int lane) {
  if (e >= left) return false;
  return e * E < 16 - (int)skew ? !headStored(skew, E, left, lane)
                                : !wholeBlock((e * E + (int)skew) / 16 - 1, skew, E, left, lane);
}
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

// n / d for n below 2^64 / d by the high half of one product: magicOf(d) is the least integer not below 2^64 / d (0 where
// the quotients need not be exact or fit: the caller then divides).
inline uint64_t magicOf(uint64_t d, uint64_t most) {
  if (d < 2 || most > ~(uint64_t)0 / d) return 0;
  return ~(uint64_t)0 / d + 1;
}

}  // namespace vrccl

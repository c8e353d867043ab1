// Chunks of eight elements as packed words: loaded from and stored to rows on
// any element (ops_chunks.h has the arithmetic).
#pragma once

#include "ops_chunks.h"
#include "ops_common.cuh"

namespace vrccl {

template <int DT>
struct Chunk {
  static constexpr int E = floatTypeSize(DT), NB = kChunk * E / 16, NW = 4 * NB;
  uint32_t w[NW];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void set(int b, const uint4& v) { w[4 * b] = v.x, w[4 * b + 1] = v.y, w[4 * b + 2] = v.z, w[4 * b + 3] = v.w; }
  __device__ __forceinline__ uint4 block(int b) const { return make_uint4(w[4 * b], w[4 * b + 1], w[4 * b + 2], w[4 * b + 3]); }
  __device__ __forceinline__ void expand(float (&f)[kChunk]) const {
    if constexpr (E == 4) {
#pragma unroll
      for (int e = 0; e < kChunk; ++e) f[e] = __uint_as_float(w[e]);
    } else {
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const float2 p = unpack2<DT>(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
      }
    }
  }
  __device__ __forceinline__ void pack(const float (&f)[kChunk]) {
    if constexpr (E == 4) {
#pragma unroll
      for (int e = 0; e < kChunk; ++e) w[e] = __float_as_uint(f[e]);
    } else {
#pragma unroll
      for (int i = 0; i < NW; ++i) w[i] = pack2<DT>(f[2 * i], f[2 * i + 1]);
    }
  }
  // Elements from `left` on become zero.
  __device__ __forceinline__ void cut(int left) {
    if (left >= kChunk) return;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      if constexpr (E == 4)
        w[i] = i < left ? w[i] : 0;
      else
        w[i] = 2 * i + 1 < left ? w[i] : 2 * i < left ? w[i] & 0xffffu : 0;
    }
  }
  __device__ __forceinline__ uint32_t bits(int e) const { return E == 4 ? w[E == 4 ? e : 0] : (w[e / 2] >> (e % 2 * 16)) & 0xffffu; }
  __device__ __forceinline__ void storeOne(char* p, int e) const {
    if constexpr (E == 4)
      reinterpret_cast<uint32_t*>(p)[e] = w[e];
    else
      reinterpret_cast<unsigned short*>(p)[e] = (unsigned short)bits(e);
  }
};

// out[i] = word i of the bytes that begin `skew` bytes into v (16 <= the bytes of v beyond out's). skew is the same for a
// row, so that the switch does not diverge.
template <int N, int M>
__device__ __forceinline__ void shiftedWords(const uint32_t (&v)[M], unsigned skew, uint32_t (&out)[N]) {
  static_assert(M >= N + 4, "a block more");
  const unsigned sh = skew % 4 * 8;
  switch (skew / 4) {
    case 0:
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = __funnelshift_r(v[i], v[i + 1], sh);
      break;
    case 1:
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = __funnelshift_r(v[i + 1], v[i + 2], sh);
      break;
    case 2:
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = __funnelshift_r(v[i + 2], v[i + 3], sh);
      break;
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = __funnelshift_r(v[i + 3], v[i + 4 < M ? i + 4 : M - 1], sh);  // (the last: sh > 0 only)
  }
}

// A warp loads 32 consecutive chunks of a row, this lane the one at p with
// `left` elements to the row's end (none: left <= 0); [begin, end) are the
// matrix's bytes. All lanes call it.
template <int DT>
__device__ __forceinline__ Chunk<DT> loadChunk(const char* p, int left, uintptr_t begin, uintptr_t end) {
  using C = Chunk<DT>;
  constexpr int E = C::E, NB = C::NB;
  C c;
  c.clear();
  const uintptr_t at = (uintptr_t)p, rowEnd = at + (intptr_t)left * E, first = at & ~(uintptr_t)15;
  const unsigned skew = at & 15;
  const bool whole = left > 0 && fromBlocks(at, E, left, begin, end);
  if (skew == 0) {
    if (whole) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
        if (blockLoaded(first + 16 * b, rowEnd, begin, end)) c.set(b, __ldcs(reinterpret_cast<const uint4*>(first) + b));
    }
  } else {
    uint32_t v[4 * NB + 4];
    auto block = [&](int b) {
      return blockLoaded(first + 16 * b, rowEnd, begin, end) ? __ldcs(reinterpret_cast<const uint4*>(first) + b) : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint4 q = block(b);
      v[4 * b] = q.x, v[4 * b + 1] = q.y, v[4 * b + 2] = q.z, v[4 * b + 3] = q.w;
    }
    uint4 after = make_uint4(0, 0, 0, 0);
    if ((threadIdx.x & 31) == 31) after = block(NB);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * NB + i] = __shfl_down_sync(0xffffffffu, v[i], 1);
    if ((threadIdx.x & 31) == 31) v[4 * NB] = after.x, v[4 * NB + 1] = after.y, v[4 * NB + 2] = after.z, v[4 * NB + 3] = after.w;
    if (whole) shiftedWords(v, skew, c.w);
  }
  if (left > 0 && !whole) {
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
      if (e >= left) continue;
      if constexpr (E == 4)
        c.w[e] = reinterpret_cast<const uint32_t*>(p)[e];
      else
        c.w[e / 2] |= (uint32_t) reinterpret_cast<const unsigned short*>(p)[e] << (e % 2 * 16);
    }
  }
  return c;
}

// A warp stores 32 consecutive chunks of a row (p, left as above). All lanes call it.
template <int DT>
__device__ __forceinline__ void storeChunk(char* p, const Chunk<DT>& c, int left) {
  using C = Chunk<DT>;
  constexpr int E = C::E, NB = C::NB;
  const unsigned skew = (uintptr_t)p & 15;
  if (skew == 0) {
    if (left >= kChunk) {
#pragma unroll
      for (int b = 0; b < NB; ++b) __stcs(reinterpret_cast<uint4*>(p) + b, c.block(b));
    } else {
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (e < left) c.storeOne(p, e);
    }
    return;
  }
  const int lane = threadIdx.x & 31;
  left = min(left, 64);  // (more says nothing more, and its bytes might pass 31 bits)
  uint32_t v[4 * NB + 4], out[4 * NB];
#pragma unroll
  for (int i = 0; i < 4 * NB; ++i) v[i] = c.w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[4 * NB + i] = __shfl_down_sync(0xffffffffu, c.w[i], 1);
  if (left <= 0) return;
  shiftedWords(v, 16 - skew, out);
  bool all = headStored(skew, E, left, lane);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const bool whole = wholeBlock(b, skew, E, left, lane);
    if (whole) __stcs(reinterpret_cast<uint4*>(p + 16 - skew) + b, make_uint4(out[4 * b], out[4 * b + 1], out[4 * b + 2], out[4 * b + 3]));
    all &= whole;
  }
  if (all) return;
#pragma unroll
  for (int e = 0; e < kChunk; ++e)
    if (storedSingly(e, skew, E, left, lane)) c.storeOne(p, e);
}

}  // namespace vrccl

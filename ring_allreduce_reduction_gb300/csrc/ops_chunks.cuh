// Chunks of eight elements as packed words: loaded from and stored to rows on
// any element (ops_chunks.h has the arithmetic).
#pragma once

#include "ops_chunks.h"
#include "ops_common.cuh"

namespace vrccl {

// Whether rows of the same number lie on the same skew in two matrices.
inline bool sameSkew(const void* p, size_t ldp, const void* q, size_t ldq, int elem) {
  return ((uintptr_t)p - (uintptr_t)q) % 16 == 0 && (ldp - ldq) * elem % 16 == 0;
}

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
  // Elements before number n become zero (n < 8).
  __device__ __forceinline__ void cutHead(int n) {
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      if constexpr (E == 4)
        w[i] = i < n ? 0 : w[i];
      else
        w[i] = 2 * i + 1 < n ? 0 : 2 * i < n ? w[i] & 0xffff0000u : w[i];
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

// out[i] = word i of the bytes that begin `skew` bytes (at most 16) into v. skew is the same for a row, so that the switch
// does not diverge where a warp has one (selections instead took as long or 3 % longer).
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

// Whether 32 lanes whose first has chunk `chunk` hold whole chunks of a row, another one follows, and the row has others
// before and after it: then every block that a chunk touches lies inside the matrix.
__device__ __forceinline__ bool innerChunks(size_t row, size_t rows, int chunk, int cols) {
  return row > 0 && row + 1 < rows && chunk <= cols / kChunk - 33;
}

// `lanes` lanes load consecutive chunks of a row, this one (its place among
// them: lane) the one at p with `left` elements to the row's end (none: left <=
// 0); [begin, end) are the matrix's bytes. All lanes of a warp call it.
template <int DT>
__device__ __forceinline__ Chunk<DT> loadChunk(const char* p, int left, uintptr_t begin, uintptr_t end, int lane, int lanes, bool inner) {
  using C = Chunk<DT>;
  constexpr int E = C::E, NB = C::NB;
  const bool last = lane == lanes - 1;
  if (inner) {
    C c;
    const unsigned skew = (uintptr_t)p & 15;
    const uint4* q = reinterpret_cast<const uint4*>(p - skew);
    if (skew == 0) {
#pragma unroll
      for (int b = 0; b < NB; ++b) c.set(b, __ldcs(q + b));
      return c;
    }
    uint32_t v[4 * NB + 4];
    uint4 after = make_uint4(0, 0, 0, 0);
    if (last) after = __ldcs(q + NB);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint4 w = __ldcs(q + b);
      v[4 * b] = w.x, v[4 * b + 1] = w.y, v[4 * b + 2] = w.z, v[4 * b + 3] = w.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * NB + i] = __shfl_down_sync(0xffffffffu, v[i], 1);
    if (last) v[4 * NB] = after.x, v[4 * NB + 1] = after.y, v[4 * NB + 2] = after.z, v[4 * NB + 3] = after.w;
    shiftedWords(v, skew, c.w);
    return c;
  }
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
    if (last) after = block(NB);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * NB + i] = __shfl_down_sync(0xffffffffu, v[i], 1, lanes);
    if (last) v[4 * NB] = after.x, v[4 * NB + 1] = after.y, v[4 * NB + 2] = after.z, v[4 * NB + 3] = after.w;
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

// A head of n bytes, the first of w, at p, and a rest of n bytes at a boundary p.
__device__ __forceinline__ void storeHead(char* p, int n, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
  const unsigned sh = (n & 2) * 8;
  const uint32_t s0 = __funnelshift_r(w0, w1, sh), s1 = __funnelshift_r(w1, w2, sh), s2 = __funnelshift_r(w2, w3, sh);
  if (n & 2) *reinterpret_cast<unsigned short*>(p) = (unsigned short)w0;
  if (n & 4) *reinterpret_cast<uint32_t*>(p + headPiece(n, 4)) = s0;
  if (n & 8) *reinterpret_cast<uint2*>(p + headPiece(n, 8)) = n & 4 ? make_uint2(s1, s2) : make_uint2(s0, s1);
}
__device__ __forceinline__ void storeRest(char* p, int n, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
  if (n & 8) *reinterpret_cast<uint2*>(p) = make_uint2(w0, w1);
  const uint32_t a = n & 8 ? w2 : w0, b = n & 8 ? w3 : w1;
  if (n & 4) *reinterpret_cast<uint32_t*>(p + restPiece(n, 4)) = a;
  if (n & 2) *reinterpret_cast<unsigned short*>(p + restPiece(n, 2)) = (unsigned short)(n & 4 ? b : a);
}

// Bytes [from, to) of the 16-byte block at p.
template <int E>
__device__ __forceinline__ void storePart(char* p, int from, int to, const uint4& v) {
  if (from == 0 && to == 16) {
    __stcs(reinterpret_cast<uint4*>(p), v);
  } else if (from == 0) {
    storeRest(p, to, v.x, v.y, v.z, v.w);
  } else if (to == 16) {
    const int n = 16 - from;
    if (n & 8) *reinterpret_cast<uint2*>(p + 8) = make_uint2(v.z, v.w);
    const uint32_t a = n & 8 ? v.y : v.w, b = n & 8 ? v.x : v.z;
    if (n & 4) *reinterpret_cast<uint32_t*>(p + 12 - (n & 8)) = a;
    if (n & 2) *reinterpret_cast<unsigned short*>(p + from) = (unsigned short)((n & 4 ? b : a) >> 16);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int at = 0; at < 16; at += E) {
      if (at < from || at >= to) continue;
      if constexpr (E == 4)
        *reinterpret_cast<uint32_t*>(p + at) = w[at / 4];
      else
        *reinterpret_cast<unsigned short*>(p + at) = (unsigned short)(w[at / 4] >> (at % 4 * 8));
    }
  }
}
// Of a chunk at a boundary p its elements from number `from` on and before number `to`.
template <int DT>
__device__ __forceinline__ void storeElements(char* p, const Chunk<DT>& c, int from, int to) {
  constexpr int E = Chunk<DT>::E, NB = Chunk<DT>::NB;
  from = max(0, from) * E;
  to = min(kChunk, to) * E;
  if (from == 0 && to == kChunk * E) {
#pragma unroll
    for (int b = 0; b < NB; ++b) __stcs(reinterpret_cast<uint4*>(p) + b, c.block(b));
  } else {
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (max(from - 16 * b, 0) < min(to - 16 * b, 16)) storePart<E>(p + 16 * b, max(from - 16 * b, 0), min(to - 16 * b, 16), c.block(b));
  }
}
// And the same loaded, from a matrix of bytes [begin, end): what lies beside them is anything.
template <int DT>
__device__ __forceinline__ Chunk<DT> loadElements(const char* p, int from, int to, uintptr_t begin, uintptr_t end) {
  constexpr int E = Chunk<DT>::E, NB = Chunk<DT>::NB;
  Chunk<DT> c;
  if (from <= 0 && to >= kChunk) {
#pragma unroll
    for (int b = 0; b < NB; ++b) c.set(b, __ldcs(reinterpret_cast<const uint4*>(p) + b));
    return c;
  }
  c.clear();
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int first = max(from, 16 / E * b), last = min(to, 16 / E * (b + 1));
    if (first >= last) continue;
    if ((uintptr_t)p + 16 * b >= begin && (uintptr_t)p + 16 * (b + 1) <= end) {
      c.set(b, __ldcs(reinterpret_cast<const uint4*>(p) + b));
      continue;
    }
#pragma unroll
    for (int e = 16 / E * b; e < 16 / E * (b + 1); ++e) {
      if (e < first || e >= last) continue;
      if constexpr (E == 4)
        c.w[e] = reinterpret_cast<const uint32_t*>(p)[e];
      else
        c.w[e / 2] |= (uint32_t) reinterpret_cast<const unsigned short*>(p)[e] << (e % 2 * 16);
    }
  }
  return c;
}

// Lanes store consecutive chunks of a row (p, left as above). All lanes of a warp call it.
template <int DT>
__device__ __forceinline__ void storeChunk(char* p, const Chunk<DT>& c, int left, const Place& at, bool inner) {
  using C = Chunk<DT>;
  constexpr int E = C::E, NB = C::NB;
  const unsigned skew = (uintptr_t)p & 15;
  if (inner) {
    if (skew == 0) {
      if (at.lane < at.step)
#pragma unroll
        for (int b = 0; b < NB; ++b) __stcs(reinterpret_cast<uint4*>(p) + b, c.block(b));
      return;
    }
    uint32_t v[4 * NB + 4], out[4 * NB];
#pragma unroll
    for (int i = 0; i < 4 * NB; ++i) v[i] = c.w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * NB + i] = __shfl_down_sync(0xffffffffu, c.w[i], 1);
    const int head = headOf(skew);
    shiftedWords(v, head, out);
    if (at.lane >= at.step) return;
    if (!headStored(skew, E, kChunk, at)) storeHead(p, head, c.w[0], c.w[1], c.w[2], c.w[3]);
    p += head;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b == NB - 1 && at.lane == 31)
        storeRest(p + 16 * b, skew, out[4 * b], out[4 * b + 1], out[4 * b + 2], out[4 * b + 3]);
      else
        __stcs(reinterpret_cast<uint4*>(p) + b, make_uint4(out[4 * b], out[4 * b + 1], out[4 * b + 2], out[4 * b + 3]));
    }
    return;
  }
  left = min(left, 64);  // (more says nothing more, and its bytes might pass 31 bits)
  if (skew == 0 && left >= kChunk && at.lane < at.step) {
#pragma unroll
    for (int b = 0; b < NB; ++b) __stcs(reinterpret_cast<uint4*>(p) + b, c.block(b));
  }
  uint32_t v[4 * NB + 4], out[4 * NB];
#pragma unroll
  for (int i = 0; i < 4 * NB; ++i) v[i] = c.w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[4 * NB + i] = __shfl_down_sync(0xffffffffu, c.w[i], 1, at.lanes);
  if (left <= 0 || at.lane >= at.step) return;
  if (skew == 0) {
    if (left < kChunk) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int n = left * E - 16 * b;
        if (n >= 16)
          __stcs(reinterpret_cast<uint4*>(p) + b, c.block(b));
        else if (n > 0)
          storeRest(p + 16 * b, n, c.w[4 * b], c.w[4 * b + 1], c.w[4 * b + 2], c.w[4 * b + 3]);
      }
    }
    return;
  }
  const int head = headOf(skew);
  if (!headStored(skew, E, left, at)) {
    if (left * E < head) {
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (e < left) c.storeOne(p, e);
      return;
    }
    storeHead(p, head, c.w[0], c.w[1], c.w[2], c.w[3]);
  }
  shiftedWords(v, head, out);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    char* q = p + head + 16 * b;
    if (wholeBlock(b, skew, E, left, at)) {
      __stcs(reinterpret_cast<uint4*>(q), make_uint4(out[4 * b], out[4 * b + 1], out[4 * b + 2], out[4 * b + 3]));
    } else {
      const int n = restOf(b, skew, E, left);
      if (n > 0) storeRest(q, n, out[4 * b], out[4 * b + 1], out[4 * b + 2], out[4 * b + 3]);
    }
  }
}

}  // namespace vrccl

// Dropout from a counter-based generator, with the residual's addition.
//
//   y  = residual + (kept ? x scale : 0)
//   dx = kept ? dy scale : 0,   scale = 65536 / (65536 - drop), drop = round(65536 p)
//
// Nothing is stored of the mask: both directions draw it anew. Columns go in
// chunks of eight; chunk number (firstRow + row) ceil(cols / 8) + col / 8 and
// the call's offset are the counter of Philox4x32-10 under the seed, whose 128
// bits give each element of the chunk 16. An element is kept if its 16 bits are
// not below `drop`. The mask depends on seed, offset, row number and column
// alone: not on strides, alignment, type or how the rows are split over calls.
//
// Sixteen bits an element, not 32: the probability is then a multiple of 2^-16
// (and the scale that of the rounded one, so that the expectation is exact),
// and the generator takes 2.5 products an element instead of 5.
//
// Bound by memory. A thread takes chunks of its own. Where all rows start on
// 16-byte boundaries and are whole chunks long, the matrix is one run of chunks
// (the row by a multiplication); else a warp takes chunks of one row, or
// several short ones: whole blocks where rows lie on the same skew in every
// matrix, else put together from blocks and the neighbouring lanes'.
#include "ops_chunks.cuh"

namespace vrccl {
namespace {

struct DropoutArgs {
  const char* x;
  const char* r;  // NULL: none
  char* y;
  uintptr_t xEnd, rEnd;  // behind the matrices' last elements
  const uint64_t* seed;
  uint64_t offset, firstChunk;  // the counter of chunk 0
  Division division;            // by `per` or `segments`, for fewer than 2^31 chunks or shares
  size_t ldx, ldr, ldy, rows, chunks;  // chunks: in all rows (one run), or warps' shares of them (split rows)
  int cols;
  unsigned per;       // chunks a row
  unsigned segments;  // shares a row
  int lanes, step;    // Place
  float scale;
  uint32_t last;  // what 32 bits with an element's in the upper half exceed if it is kept ...
  bool all;       // ... or all are
};

constexpr int kThreads = 256;

template <int DT, bool RES>
__device__ __forceinline__ void dropChunk(const DropoutArgs& a, const Random128& bits, const Chunk<DT>& x, const Chunk<DT>& r,
                                          Chunk<DT>& y) {
  float f[kChunk], g[kChunk];
  x.expand(f);
  if constexpr (RES) r.expand(g);
  const F2 scale = pair(a.scale, a.scale);
#pragma unroll
  for (int e = 0; e < kChunk; e += 2) {
    float2 v;
    if constexpr (RES)
      v = split(fma2(pair(f[e], f[e + 1]), scale, pair(g[e], g[e + 1])));
    else
      v = split(mul2(pair(f[e], f[e + 1]), scale));
    // (chosen, not multiplied by zero: what is dropped may hold anything)
    f[e] = keeps(bits, e, a.last, a.all) ? v.x : RES ? g[e] : 0.f;
    f[e + 1] = keeps(bits, e + 1, a.last, a.all) ? v.y : RES ? g[e + 1] : 0.f;
  }
  y.pack(f);
}

// How rows of whole chunks on 16-byte boundaries lie: with no gaps between them; with the same stride in every matrix, which
// ends less than 4 GB from its beginning (16384 x 4096 + 8 bf16 52 us, by 64-bit addresses 58); anyhow.
enum Gaps { kNone, kAlike, kAny };
// One run of chunks; U a thread, asked for before the bits are drawn.
template <int DT, bool RES, int U, Gaps GAPS>
__global__ void __launch_bounds__(kThreads) dropoutRun(const __grid_constant__ DropoutArgs a) {
  using C = Chunk<DT>;
  constexpr int E = C::E, NB = C::NB;
  const size_t block = (size_t)blockIdx.x * (kThreads * U);
  C x[U], r[U];
  size_t row[U];
  unsigned col[U];  // kAlike: the chunk's place in bytes
  auto place = [&](const char* p, size_t ld, int u) {
    return GAPS == kNone    ? reinterpret_cast<const uint4*>(p) + (block + threadIdx.x) * NB + u * (kThreads * NB)
           : GAPS == kAlike ? reinterpret_cast<const uint4*>(p + col[u])
                            : reinterpret_cast<const uint4*>(p + row[u] * ld * E) + (size_t)col[u] * NB;
  };
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const size_t n = block + threadIdx.x + u * kThreads;
    if (n >= a.chunks) continue;
    if constexpr (GAPS == kAlike) {
      const uint32_t r = a.per == 1 ? (uint32_t)n : quotient((uint32_t)n, a.division);
      col[u] = r * (uint32_t)(a.ldx * E) + ((uint32_t)n - r * a.per) * (16 * NB);
    } else if constexpr (GAPS == kAny) {
      row[u] = a.chunks >> 31 || a.per == 1 ? n / a.per : quotient((uint32_t)n, a.division);
      col[u] = (unsigned)n - (unsigned)row[u] * a.per;
    }
    const uint4 *p = place(a.x, a.ldx, u), *q = place(a.r, a.ldr, u);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      x[u].set(b, __ldcs(p + b));
      if constexpr (RES) r[u].set(b, __ldcs(q + b));
    }
  }
  const uint64_t seed = *a.seed, counter = a.firstChunk + block;
  // Where a block's counters share their upper half, a thread's chunks share the half of the first two rounds that comes of
  // it and of the offset.
  auto draw = [&](auto shared) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (block + threadIdx.x + u * kThreads >= a.chunks) continue;
      const unsigned n = threadIdx.x + u * kThreads;
      const uint64_t number = decltype(shared)::value ? (counter & ~(uint64_t)0xffffffffu) | ((uint32_t)counter + n) : counter + n;
      C y;
      dropChunk<DT, RES>(a, philox(seed, number, a.offset), x[u], r[u], y);
      uint4* p = const_cast<uint4*>(place(a.y, a.ldy, u));
#pragma unroll
      for (int b = 0; b < NB; ++b) __stcs(p + b, y.block(b));
    }
  };
  if ((uint32_t)counter <= ~0u - kThreads * U)
    draw(std::true_type{});
  else
    draw(std::false_type{});
}

// Rows each on the same skew in every matrix. Chunks are counted from the boundary before the row's first element, column
// -shift, and are whole blocks in every matrix (parts of them at the row's ends); a lane draws the bits of the columns' chunk
// of that number and takes the other part of its own from the lane before. In rows of more than 32 chunks a warp takes 31,
// its first lane drawing for the second alone.
template <int DT, bool RES>
__global__ void __launch_bounds__(kThreads) dropoutSame(const __grid_constant__ DropoutArgs a) {
  using C = Chunk<DT>;
  constexpr int E = C::E;
  const size_t warp = (size_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (warp >= a.chunks) return;
  int lane = threadIdx.x & 31, ci;
  size_t row = warp;
  if (a.segments > 1) {
    row = a.chunks >> 31 ? warp / a.segments : quotient((uint32_t)warp, a.division);
    ci = (int)((unsigned)warp - (unsigned)row * a.segments) * 31 + lane - 1;
  } else {
    row = warp * (32 / a.lanes) + lane / a.lanes;
    ci = lane &= a.lanes - 1;
  }
  const char* px = a.x + row * a.ldx * E;
  const int shift = (int)((uintptr_t)px & 15) / E, from = shift - ci * kChunk, to = a.cols + from;
  const bool own = row < a.rows && to > 0 && ci >= 0 && (a.segments == 1 || lane > 0);
  const ptrdiff_t at = ((ptrdiff_t)ci * kChunk - shift) * E;
  C x, r, y;
  if (own) {
    x = loadElements<DT>(px + at, from, to, (uintptr_t)a.x, a.xEnd);
    if constexpr (RES) r = loadElements<DT>(a.r + row * a.ldr * E + at, from, to, (uintptr_t)a.r, a.rEnd);
  }
  Random128 bits = philox(*a.seed, a.firstChunk + row * a.per + ci, a.offset);
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __shfl_up_sync(0xffffffffu, bits.w[i], 1, a.lanes), v[4 + i] = bits.w[i];
  if (!own) return;
  if (shift) shiftedWords(v, 16 - 2 * shift, bits.w);  // two bytes an element
  dropChunk<DT, RES>(a, bits, x, r, y);
  storeElements<DT>(a.y + row * a.ldy * E + at, y, from, to);
}

// Rows on any element: a warp takes `step` chunks of one, or short ones whole.
template <int DT, bool RES>
__global__ void __launch_bounds__(kThreads) dropoutRows(const __grid_constant__ DropoutArgs a) {
  using C = Chunk<DT>;
  constexpr int E = C::E;
  const size_t warp = (size_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (warp >= a.chunks) return;
  Place at = {(int)(threadIdx.x & 31), a.lanes, 0, a.step};
  size_t row = warp;
  int first = 0;  // the warp's first chunk
  if (a.lanes < 32) {
    row = warp * (32 / a.lanes) + at.lane / a.lanes;
    at.lane &= a.lanes - 1;
  } else if (a.segments > 1) {
    row = a.chunks >> 31 ? warp / a.segments : quotient((uint32_t)warp, a.division);
    first = (int)((unsigned)warp - (unsigned)row * a.segments) * a.step;
  }
  at.chunk = first + at.lane;
  const int left = row < a.rows ? a.cols - at.chunk * kChunk : 0;
  const bool inner = a.segments > 1 && innerChunks(row, a.rows, first, a.cols);
  auto place = [&](const char* p, size_t ld) { return p + row * ld * E + (size_t)at.chunk * (kChunk * E); };
  const C x = loadChunk<DT>(place(a.x, a.ldx), left, (uintptr_t)a.x, a.xEnd, at.lane, at.lanes, inner);
  C r, y;
  if constexpr (RES) r = loadChunk<DT>(place(a.r, a.ldr), left, (uintptr_t)a.r, a.rEnd, at.lane, at.lanes, inner);
  dropChunk<DT, RES>(a, philox(*a.seed, a.firstChunk + row * a.per + at.chunk, a.offset), x, r, y);
  storeChunk<DT>(const_cast<char*>(place(a.y, a.ldy)), y, left, at, inner);
}

template <int DT, bool RES>
vrcclResult_t launchDropout(DropoutArgs& a, bool run, bool same, cudaStream_t st) {
  const bool one = a.rows == 1;
  if (!run) {
    // Lanes of a row, shares of longer ones, and the warps that are made of them, on any skew of the rows.
    auto deal = [&](unsigned most, int step) {
      a.lanes = most <= 8 ? 8 : most <= 16 ? 16 : 32;
      a.step = a.lanes < 32 ? a.lanes : step;
      a.segments = (most + a.step - 1) / a.step;
      return a.segments > 1 ? a.rows * a.segments : (a.rows + 32 / a.lanes - 1) / (32 / a.lanes);
    };
    const unsigned most = (unsigned)(((size_t)a.cols + 16 / Chunk<DT>::E - 1 + kChunk - 1) / kChunk);
    const size_t sameWarps = deal(most, most > 32 ? 31 : 32), warps = deal(a.per, a.per > 32 ? stepOf((int)a.per) : 32);
    // A warp of rows on the same skew takes nine tenths of the other's time, three quarters with a residual (16384 x 4097 bf16 with
    // it 114 -> 82 us, 16384 x 4096 without 86 -> 77, 262144 x 65 77 -> 49), but there may be more of them (262144 x 255: 98, 157).
    same = same && (RES ? sameWarps * 3 <= warps * 4 : sameWarps * 9 <= warps * 10);
    a.chunks = same ? deal(most, most > 32 ? 31 : 32) : warps;
    a.division = divisionOf(a.segments);
    const size_t blocks = (a.chunks + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks >= (size_t(1) << 31)) return vrcclInvalidArgument;
    return launchShaped(same ? dropoutSame<DT, RES> : dropoutRows<DT, RES>, {dim3((unsigned)blocks), kThreads, 0, 0, false}, st, a);
  }
  a.chunks = a.rows * a.per;
  a.division = divisionOf(a.per);
  const size_t cols = a.cols;
  const bool alike = a.ldx == a.ldy && (!RES || a.ldr == a.ldy), none = one || (alike && a.ldx == cols);
  const bool near = alike && a.chunks >> 31 == 0 && ((a.rows - 1) * a.ldx + cols) * Chunk<DT>::E < (size_t(1) << 32);
  const bool many = a.chunks >= (size_t)smCount() * kThreads * 8;
  constexpr int U = DT == vrcclFloat32 ? 2 : 4;
  const int u = many ? U : 1;
  const size_t blocks = (a.chunks + kThreads * u - 1) / (kThreads * u);
  if (blocks >= (size_t(1) << 31)) return vrcclInvalidArgument;
  const LaunchShape s = {dim3((unsigned)blocks), kThreads, 0, 0, false};
  auto launch = [&](auto gaps) {
    constexpr Gaps G = decltype(gaps)::value;
    return many ? launchShaped(dropoutRun<DT, RES, U, G>, s, st, a) : launchShaped(dropoutRun<DT, RES, 1, G>, s, st, a);
  };
  return none   ? launch(std::integral_constant<Gaps, kNone>{})
         : near ? launch(std::integral_constant<Gaps, kAlike>{})
                : launch(std::integral_constant<Gaps, kAny>{});
}

vrcclResult_t dropout(const void* x, size_t ldx, const void* r, size_t ldr, void* y, size_t ldy, size_t rows, size_t cols,
                      int dtype, float p, const uint64_t* seed, uint64_t offset, size_t firstRow,
                      vrcclStream_t stream) {
  if (rows >= kMaxExtent || cols >= (size_t(1) << 31) - 65536 || !isOperatorType(dtype) || !(p >= 0.f && p <= 1.f) ||
      firstRow >= kMaxExtent)
    return vrcclInvalidArgument;
  if (rows == 0 || cols == 0) return vrcclSuccess;
  const int E = floatTypeSize(dtype);
  if (!goodMatrix(x, ldx, rows, cols, E) || !goodMatrix(y, ldy, rows, cols, E) || !goodVector(seed, 8) ||
      (r && !goodMatrix(r, ldr, rows, cols, E)))
    return vrcclInvalidArgument;
  const size_t per = (cols + kChunk - 1) / kChunk;
  if (firstRow + rows > (~size_t(0) >> 1) / per) return vrcclInvalidArgument;  // chunks are numbered in 63 bits
  const Span out[] = {matrixSpan(y, ldy, rows, cols, E)};
  const Span in[] = {unlessInPlace(matrixSpan(x, ldx, rows, cols, E), ldx, y, ldy),
                     r ? unlessInPlace(matrixSpan(r, ldr, rows, cols, E), ldr, y, ldy) : vectorSpan(nullptr, 0),
                     vectorSpan(seed, 8)};
  if (!apart(out, in)) return vrcclInvalidArgument;
  cudaStream_t st = (cudaStream_t)stream;
  const int drop = dropThreshold(p);
  DropoutArgs a = {};
  a.x = static_cast<const char*>(x);
  a.r = static_cast<const char*>(r);
  a.y = static_cast<char*>(y);
  a.xEnd = (uintptr_t)x + ((rows - 1) * ldx + cols) * E;
  a.rEnd = (uintptr_t)r + ((rows - 1) * ldr + cols) * E;
  a.seed = seed;
  a.offset = offset;
  a.firstChunk = firstRow * per;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldy;
  a.rows = rows;
  a.cols = (int)cols;
  a.per = (unsigned)per;
  a.scale = drop < 65536 ? 65536.f / (float)(65536 - drop) : 0.f;
  a.last = (uint32_t)drop * 65536u - 1;
  a.all = drop == 0;
  const bool run = cols % kChunk == 0 && rowsAligned(x, ldx, E) && rowsAligned(y, ldy, E) && (!r || rowsAligned(r, ldr, E));
  const bool same = sameSkew(x, ldx, y, ldy, E) && (!r || sameSkew(r, ldr, y, ldy, E));
  auto go = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    return r ? launchDropout<DT, true>(a, run, same, st) : launchDropout<DT, false>(a, run, same, st);
  };
  return dtype == vrcclFloat32    ? go(std::integral_constant<int, vrcclFloat32>{})
         : dtype == vrcclBfloat16 ? go(std::integral_constant<int, vrcclBfloat16>{})
                                  : go(std::integral_constant<int, vrcclFloat16>{});
}

}  // namespace
}  // namespace vrccl

using namespace vrccl;

extern "C" vrcclResult_t vrcclDropoutForward(const void* x, size_t ldx, const void* residual, size_t ldr, void* y, size_t ldy,
                                             size_t rows, size_t cols, vrcclDataType_t dtype, float p,
                                             const uint64_t* seed, uint64_t offset, size_t firstRow,
                                             vrcclStream_t stream) {
  return dropout(x, ldx, residual, ldr, y, ldy, rows, cols, dtype, p, seed, offset, firstRow, stream);
}

extern "C" vrcclResult_t vrcclDropoutBackward(const void* dy, size_t lddy, void* dx, size_t lddx, size_t rows, size_t cols,
                                              vrcclDataType_t dtype, float p, const uint64_t* seed,
                                              uint64_t offset, size_t firstRow, vrcclStream_t stream) {
  return dropout(dy, lddy, nullptr, 0, dx, lddx, rows, cols, dtype, p, seed, offset, firstRow, stream);
}

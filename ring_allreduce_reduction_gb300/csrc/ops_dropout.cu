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
// and the generator takes 5 products an element instead of 10.
//
// Bound by memory. A thread takes chunks of its own. Where all rows start on
// 16-byte boundaries and are whole chunks long, the matrix is one run of chunks
// (the row by a multiplication); else a warp takes 32 chunks of one row, and
// lanes put theirs together from 16-byte blocks and their neighbours'.
#include "ops_chunks.cuh"

namespace vrccl {
namespace {

struct DropoutArgs {
  const char* x;
  const char* r;  // NULL: none
  char* y;
  const uint64_t* seed;
  uint64_t offset, firstChunk;  // the counter of chunk 0
  uint64_t magic;               // of `per` (0: divide)
  size_t ldx, ldr, ldy, rows, chunks;     // chunks: in all rows, or a warp's share of them (split rows)
  size_t cols;
  unsigned per;  // chunks a row
  unsigned segments;  // runs of 32 chunks a row
  float scale;
  uint32_t last;  // what 32 bits with an element's in the upper half exceed if it is kept ...
  bool all;       // ... or all are
};

constexpr int kThreads = 256;

template <int DT, bool RES>
__device__ __forceinline__ void dropChunk(const DropoutArgs& a, uint64_t seed, uint64_t number, const Chunk<DT>& x,
                                          const Chunk<DT>& r, Chunk<DT>& y) {
  const Random128 bits = philox(seed, a.firstChunk + number, a.offset);
  float f[kChunk], g[kChunk];
  x.expand(f);
  if constexpr (RES) r.expand(g);
#pragma unroll
  for (int e = 0; e < kChunk; ++e) {
    // (chosen, not multiplied by zero: what is dropped may hold anything)
    if constexpr (RES)
      f[e] = keeps(bits, e, a.last, a.all) ? fmaf(f[e], a.scale, g[e]) : g[e];
    else
      f[e] = keeps(bits, e, a.last, a.all) ? f[e] * a.scale : 0.f;
  }
  y.pack(f);
}

// One run of chunks; U a thread, asked for before the bits are drawn.
template <int DT, bool RES, int U>
__global__ void __launch_bounds__(kThreads) dropoutRun(const __grid_constant__ DropoutArgs a) {
  using C = Chunk<DT>;
  constexpr int E = C::E, NB = C::NB;
  const size_t first = (size_t)blockIdx.x * (kThreads * U) + threadIdx.x;
  C x[U], r[U];
  size_t row[U];
  unsigned col[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const size_t n = first + u * kThreads;
    if (n >= a.chunks) continue;
    row[u] = a.magic ? __umul64hi(n, a.magic) : n / a.per;
    col[u] = (unsigned)(n - row[u] * a.per);
    const uint4* p = reinterpret_cast<const uint4*>(a.x + row[u] * a.ldx * E) + (size_t)col[u] * NB;
    const uint4* q = reinterpret_cast<const uint4*>(a.r + row[u] * a.ldr * E) + (size_t)col[u] * NB;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      x[u].set(b, __ldcs(p + b));
      if constexpr (RES) r[u].set(b, __ldcs(q + b));
    }
  }
  const uint64_t seed = *a.seed;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const size_t n = first + u * kThreads;
    if (n >= a.chunks) continue;
    C y;
    dropChunk<DT, RES>(a, seed, n, x[u], r[u], y);
    uint4* p = reinterpret_cast<uint4*>(a.y + row[u] * a.ldy * E) + (size_t)col[u] * NB;
#pragma unroll
    for (int b = 0; b < NB; ++b) __stcs(p + b, y.block(b));
  }
}

// A warp a run of 32 chunks of one row, on any element.
template <int DT, bool RES>
__global__ void __launch_bounds__(kThreads) dropoutRows(const __grid_constant__ DropoutArgs a) {
  using C = Chunk<DT>;
  constexpr int E = C::E;
  const size_t warp = ((size_t)blockIdx.x * kThreads + threadIdx.x) / 32;
  if (warp >= a.chunks) return;
  const size_t row = warp / a.segments;
  const unsigned chunk = (unsigned)(warp - row * a.segments) * 32 + (threadIdx.x & 31);
  const size_t col = (size_t)chunk * kChunk;
  const int left = (int)min((long long)a.cols - (long long)col, (long long)(1 << 20));
  auto span = [&](const char* p, size_t ld) { return (uintptr_t)p + ((a.rows - 1) * ld + a.cols) * E; };
  const C x = loadChunk<DT>(a.x + (row * a.ldx + col) * E, left, (uintptr_t)a.x, span(a.x, a.ldx));
  C r, y;
  if constexpr (RES) r = loadChunk<DT>(a.r + (row * a.ldr + col) * E, left, (uintptr_t)a.r, span(a.r, a.ldr));
  dropChunk<DT, RES>(a, *a.seed, row * a.per + chunk, x, r, y);
  storeChunk<DT>(a.y + (row * a.ldy + col) * E, y, left);
}

template <int DT, bool RES>
vrcclResult_t launchDropout(DropoutArgs& a, bool run, cudaStream_t st) {
  if (!run) {
    a.segments = (a.per + 31) / 32;
    a.chunks = a.rows * a.segments;
    const size_t blocks = (a.chunks + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks >= (size_t(1) << 31)) return vrcclInvalidArgument;
    return launchShaped(dropoutRows<DT, RES>, {dim3((unsigned)blocks), kThreads, 0, 0, false}, st, a);
  }
  a.chunks = a.rows * a.per;
  a.magic = magicOf(a.per, a.chunks);
  const bool many = a.chunks >= (size_t)smCount() * kThreads * 8;
  const int u = many ? 4 : 1;
  const size_t blocks = (a.chunks + kThreads * u - 1) / (kThreads * u);
  if (blocks >= (size_t(1) << 31)) return vrcclInvalidArgument;
  const LaunchShape s = {dim3((unsigned)blocks), kThreads, 0, 0, false};
  return many ? launchShaped(dropoutRun<DT, RES, 4>, s, st, a) : launchShaped(dropoutRun<DT, RES, 1>, s, st, a);
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
  a.seed = seed;
  a.offset = offset;
  a.firstChunk = firstRow * per;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldy;
  a.rows = rows;
  a.cols = cols;
  a.per = (unsigned)per;
  a.scale = drop < 65536 ? 65536.f / (float)(65536 - drop) : 0.f;
  a.last = (uint32_t)drop * 65536u - 1;
  a.all = drop == 0;
  const bool run = cols % kChunk == 0 && rowsAligned(x, ldx, E) && rowsAligned(y, ldy, E) && (!r || rowsAligned(r, ldr, E));
  auto go = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    return r ? launchDropout<DT, true>(a, run, st) : launchDropout<DT, false>(a, run, st);
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

// RMS norm, backward (ops_rmsnorm.cu has the mathematics).
#include "ops_rmsnorm.cuh"

namespace vrccl {
namespace {

template <int DT, bool DSUM, Lie LIE, bool HOLD, bool WIDE>
__global__ void __launch_bounds__(32 * backwardWarps(HOLD, WIDE)) rmsBackward(const __grid_constant__ RmsArgs a) {
  using C = Chunk<DT>;
  constexpr int E = C::E, NP = kChunk / 2;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ unsigned long long full[kMaxTeams * kMaxStages];
  __shared__ float red[2][32];
  __shared__ int deadWord[kMaxTeams];
  Ring<E, DSUM ? 3 : 2, !HOLD> ring(a, smem, full, deadWord);
  const int shift = shiftOf<DT, LIE>(a, ring.first);
  const int t = ring.t, T = a.threads, lane = t & 31, warps = T / 32;
  F2 g[kHeld][NP], dg[kHeld][NP];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    gammaOf<DT>(a, chunkOf<LIE>(a, j, warps, t), g[j], shift);
#pragma unroll
    for (int i = 0; i < NP; ++i) dg[j][i] = 0;
  }
  const float inv = 1.f / (float)a.cols;
  letNextIn();
  float nextRstd = ring.first < a.rows ? a.rstd[ring.first] : 0.f;
  teamSync(ring.team, T);
  for (size_t row = ring.first; row < a.rows; row += ring.stride, ring.next()) {
    const float rstd = nextRstd;
    const unsigned char* stage = ring.wait();
    C s[kHeld], d[kHeld], r[kHeld];  // (HOLD)
    const F2 scale = pair(rstd, rstd);
    F2 dot = 0;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int ci = chunkOf<LIE>(a, j, warps, t);
      C sj = taken<DT, LIE>(a, stage, 0, row, ci, shift), dj = taken<DT, LIE>(a, stage, 1, row, ci, shift);
      if constexpr (HOLD) {
        s[j] = sj, d[j] = dj;
        if constexpr (DSUM) r[j] = taken<DT, LIE>(a, stage, 2, row, ci, shift);
      }
      if (!ownChunk<LIE>(a, t)) continue;
      F2 xh[NP], dy[NP];
      pairsOf(sj, xh);
      pairsOf(dj, dy);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        xh[i] = mul2(xh[i], scale);
        dot = fma2(mul2(dy[i], g[j][i]), xh[i], dot);
        dg[j][i] = fma2(dy[i], xh[i], dg[j][i]);
      }
    }
    float w = warpSum(sumOf(dot));
    if (lane == 0) red[ring.turn][threadIdx.x >> 5] = w;
    if (ring.sync(row)) break;
    if (row + ring.stride < a.rows) nextRstd = a.rstd[row + ring.stride];
    if (warps > 1) w = sumOfLanes<32>(lane < warps ? red[ring.turn][ring.team * warps + lane] : 0.f);
    const F2 minus = pair(-w * inv, -w * inv);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int ci = chunkOf<LIE>(a, j, warps, t);
      F2 xh[NP], dy[NP], add[NP];
      pairsOf(HOLD ? s[j] : taken<DT, LIE>(a, stage, 0, row, ci, shift), xh);
      pairsOf(HOLD ? d[j] : taken<DT, LIE>(a, stage, 1, row, ci, shift), dy);
      if constexpr (DSUM) pairsOf(HOLD ? r[j] : taken<DT, LIE>(a, stage, 2, row, ci, shift), add);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const F2 v = fma2(mul2(xh[i], scale), minus, mul2(dy[i], g[j][i]));
        dy[i] = DSUM ? fma2(v, scale, add[i]) : mul2(v, scale);
      }
      putChunk<DT, LIE>(a, a.y, a.ldy, row, packed<DT>(dy), ci, shift);
    }
  }
  if (!a.partial) return;
  // the teams own the same columns: every team lays its sums out, and the block adds them in the teams' order
  float* sum = reinterpret_cast<float*>(smem);
  __syncthreads();  // no team reads its ring any more
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    if (ownChunk<LIE>(a, t)) layOut(sum + (size_t)ring.team * a.cols, dg[j], chunkOf<LIE>(a, j, warps, t), a.cols, shift);
  __syncthreads();
  float* p = a.partial + (size_t)blockIdx.x * a.cols;
  for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
    float x = sum[c];
    for (int w = 1; w < a.teams; ++w) x += sum[(size_t)w * a.cols + c];
    p[c] = x;
  }
}

template <int DT, int G, bool DSUM>
__global__ void __launch_bounds__(kNarrowThreads) rmsBackwardNarrow(const __grid_constant__ RmsArgs a) {
  using C = Chunk<DT>;
  constexpr int NP = kChunk / 2, R = 32 / G, U = kNarrowTurn;
  __shared__ float sum[kNarrowThreads / 32][kNarrowCols];
  const int lane = threadIdx.x & 31, own = lane % G, w = threadIdx.x >> 5;
  const bool held = own < a.chunks;
  const size_t warps = (size_t)gridDim.x * (kNarrowThreads / 32);
  const float inv = 1.f / (float)a.cols;
  F2 g[NP], dg[NP];
  gammaOf<DT>(a, own, g);
#pragma unroll
  for (int i = 0; i < NP; ++i) dg[i] = 0;
  letNextIn();
  for (size_t r0 = ((size_t)blockIdx.x * (kNarrowThreads / 32) + w) * R * U; r0 < a.rows; r0 += warps * R * U) {
    C s[U], d[U], r[U];
    float rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t row = r0 + u * R + lane / G;
      const bool there = held && row < a.rows;
      s[u] = narrowChunk<DT>(a.src[0], row, own, there);
      d[u] = narrowChunk<DT>(a.src[1], row, own, there);
      if constexpr (DSUM) r[u] = narrowChunk<DT>(a.src[2], row, own, there);
      rstd[u] = row < a.rows ? a.rstd[row] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t row = r0 + u * R + lane / G;
      const F2 scale = pair(rstd[u], rstd[u]);
      F2 xh[NP], dy[NP], add[NP], dot = 0;
      pairsOf(s[u], xh);
      pairsOf(d[u], dy);
      if constexpr (DSUM) pairsOf(r[u], add);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        xh[i] = mul2(xh[i], scale);
        dg[i] = fma2(dy[i], xh[i], dg[i]);
        dy[i] = mul2(dy[i], g[i]);
        dot = fma2(dy[i], xh[i], dot);
      }
      const float m = -sumOfLanes<G>(sumOf(dot)) * inv;
      if (held && row < a.rows) {
        const F2 minus = pair(m, m);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const F2 v = fma2(xh[i], minus, dy[i]);
          dy[i] = DSUM ? fma2(v, scale, add[i]) : mul2(v, scale);
        }
        storeNarrow<DT>(a.y, row, a.ldy, own, packed<DT>(dy));
      }
    }
  }
  if (!a.partial) return;
  // the warp's groups of lanes hold the same columns, then the block's warps do
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int o = G; o < 32; o *= 2) dg[i] = add2(dg[i], __shfl_xor_sync(0xffffffffu, dg[i], o));
  if (lane < G && held) layOut(sum[w], dg, own, a.cols);
  __syncthreads();
  float* p = a.partial + (size_t)blockIdx.x * a.cols;
  for (int c = threadIdx.x; c < a.cols; c += kNarrowThreads) {
    float x = sum[0][c];
#pragma unroll
    for (int k = 1; k < kNarrowThreads / 32; ++k) x += sum[k][c];
    p[c] = x;
  }
}

// HOLD: the columns' sums in registers, for rows of up to kLongHeld; else rmsColumns makes them first.
template <int DT, bool DSUM, bool HOLD>
__global__ void __launch_bounds__(kLongThreads) rmsBackwardLong(const __grid_constant__ RmsArgs a) {
  using C = Chunk<DT>;
  constexpr int NP = kChunk / 2;
  __shared__ float red[2][32];
  const float inv = 1.f / (float)a.cols;
  const int lane = threadIdx.x & 31;
  F2 dg[kHeld][NP];
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
#pragma unroll
    for (int i = 0; i < NP; ++i) dg[j][i] = 0;
  if (HOLD) letNextIn();
  int turn = 0;
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const float rstd = a.rstd[row];
    const F2 scale = pair(rstd, rstd);
    F2 dot = 0;
    auto sums = [&](int ci, F2 (&sum)[NP]) {
      C s = longChunk<DT>(a, 0, row, ci), d = longChunk<DT>(a, 1, row, ci);
      s.cut(a.cols - ci * kChunk);
      d.cut(a.cols - ci * kChunk);
      F2 xh[NP], dy[NP], g[NP];
      pairsOf(s, xh);
      pairsOf(d, dy);
      gammaOf<DT>(a, ci, g);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        xh[i] = mul2(xh[i], scale);
        dot = fma2(mul2(dy[i], g[i]), xh[i], dot);
        if (HOLD) sum[i] = fma2(dy[i], xh[i], sum[i]);
      }
    };
    if constexpr (HOLD) {
#pragma unroll
      for (int j = 0; j < kHeld; ++j) sums(j * kLongThreads + threadIdx.x, dg[j]);
    } else {
      for (int ci = threadIdx.x; ci - lane < a.chunks; ci += kLongThreads) sums(ci, dg[0]);
    }
    float w = warpSum(sumOf(dot));
    if (lane == 0) red[turn][threadIdx.x >> 5] = w;
    __syncthreads();
    w = warpSum(red[turn][lane]);
    const F2 minus = pair(-w * inv, -w * inv);
    for (int ci = threadIdx.x; ci - lane < a.chunks; ci += kLongThreads) {
      C s = longChunk<DT>(a, 0, row, ci), d = longChunk<DT>(a, 1, row, ci);
      F2 xh[NP], dy[NP], g[NP], add[NP];
      pairsOf(s, xh);
      pairsOf(d, dy);
      gammaOf<DT>(a, ci, g);
      if constexpr (DSUM) pairsOf(longChunk<DT>(a, 2, row, ci), add);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const F2 v = fma2(mul2(xh[i], scale), minus, mul2(dy[i], g[i]));
        dy[i] = DSUM ? fma2(v, scale, add[i]) : mul2(v, scale);
      }
      putChunk<DT, kAny>(a, a.y, a.ldy, row, packed<DT>(dy), ci, 0);
    }
  }
  if constexpr (HOLD) {
    if (!a.partial) return;
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      layOut(a.partial + (size_t)blockIdx.x * a.cols, dg[j], j * kLongThreads + threadIdx.x, a.cols);
  }
}
// Partial column sums of rows beyond kLongHeld: block (i, p) takes 256 chunks and every gridDim.y-th row. It runs before
// rmsBackwardLong, which may overwrite what it reads.
template <int DT>
__global__ void __launch_bounds__(256) rmsColumns(const __grid_constant__ RmsArgs a) {
  constexpr int NP = kChunk / 2;
  const int ci = blockIdx.x * 256 + threadIdx.x;
  F2 dg[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) dg[i] = 0;
  for (size_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float rstd = a.rstd[row];
    F2 xh[NP], dy[NP];
    pairsOf(longChunk<DT>(a, 0, row, ci), xh);
    pairsOf(longChunk<DT>(a, 1, row, ci), dy);
#pragma unroll
    for (int i = 0; i < NP; ++i) dg[i] = fma2(dy[i], mul2(xh[i], pair(rstd, rstd)), dg[i]);
  }
  if (ci < a.chunks) layOut(a.partial + (size_t)blockIdx.y * a.cols, dg, ci, a.cols);
}

// dgamma from the blocks' partial sums: 32 columns a block, the partial rows split over its 32 warps and joined in warp order.
__global__ void __launch_bounds__(1024) rmsJoin(const float* partial, int blocks, int cols, void* dgamma, int ptype) {
  const int c = blockIdx.x * 32 + (threadIdx.x & 31);
  waitForPrevious();
  const float s = columnSum(partial + c, blocks, (size_t)cols, c < cols);
  if (threadIdx.x < 32 && c < cols) storeParam(dgamma, ptype, c, s);
}

template <int DT, bool DSUM, Lie LIE>
RmsFn pickRing(const Shape& s) {
  return s.hold ? rmsBackward<DT, DSUM, LIE, true, false> : s.wide ? rmsBackward<DT, DSUM, LIE, false, true> : rmsBackward<DT, DSUM, LIE, false, false>;
}
template <int DT, bool DSUM>
RmsFn pickBackward(const Shape& s, int cols) {
  if (s.walk == kRing)
    return s.lie == kAny ? rmsBackward<DT, DSUM, kAny, false, false> : s.lie == kSame ? pickRing<DT, DSUM, kSame>(s) : pickRing<DT, DSUM, kWhole>(s);
  if (s.walk == kLong) return cols <= kLongHeld ? rmsBackwardLong<DT, DSUM, true> : rmsBackwardLong<DT, DSUM, false>;
  return s.lanes == 4 ? rmsBackwardNarrow<DT, 4, DSUM> : s.lanes == 8 ? rmsBackwardNarrow<DT, 8, DSUM> : rmsBackwardNarrow<DT, 16, DSUM>;
}

}  // namespace

int rmsBackwardStatus(int* code) { return cudaMemcpyFromSymbol(code, gRingStatus, sizeof(*code)); }

}  // namespace vrccl

using namespace vrccl;

extern "C" vrcclResult_t vrcclRmsNormWorkspace(size_t rows, size_t cols, size_t* bytes) {
  if (!bytes || !goodSizes(rows, cols, vrcclFloat32, vrcclFloat32)) return vrcclInvalidArgument;
  *bytes = rows && cols ? size_t(mostBlocks(rows, (int)cols)) * cols * sizeof(float) : 0;  // (rmsShape divides by what fits)
  return vrcclSuccess;
}

extern "C" vrcclResult_t vrcclRmsNormBackward(const void* dy, size_t lddy, const void* dsum, size_t ldds, const void* s,
                                              size_t lds, const void* gamma, const float* rstd, void* dx, size_t lddx,
                                              void* dgamma, size_t rows, size_t cols, vrcclDataType_t dtype,
                                              vrcclDataType_t paramType, void* workspace, size_t workspaceBytes,
                                              vrcclStream_t stream) {
  if (!goodSizes(rows, cols, dtype, paramType)) return vrcclInvalidArgument;
  if (cols == 0) return vrcclSuccess;
  const int E = floatTypeSize(dtype), PE = floatTypeSize(paramType);
  if ((gamma && !goodVector(gamma, PE)) || (dgamma && !goodVector(dgamma, PE))) return vrcclInvalidArgument;
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) {  // a sum over no rows
    if (dgamma && cudaMemsetAsync(dgamma, 0, cols * PE, st) != cudaSuccess) {
      cudaGetLastError();
      return vrcclCudaError;
    }
    return vrcclSuccess;
  }
  if (!goodMatrix(dy, lddy, rows, cols, E) || (dsum && !goodMatrix(dsum, ldds, rows, cols, E)) ||
      !goodMatrix(s, lds, rows, cols, E) || !goodMatrix(dx, lddx, rows, cols, E) || !goodVector(rstd, 4))
    return vrcclInvalidArgument;
  const size_t need = dgamma ? size_t(mostBlocks(rows, (int)cols)) * cols * sizeof(float) : 0;  // what the query says
  if (dgamma && (!goodVector(workspace, 16) || workspaceBytes < need)) return vrcclInvalidArgument;
  const Span none = vectorSpan(nullptr, 0), spanDy = matrixSpan(dy, lddy, rows, cols, E), spanS = matrixSpan(s, lds, rows, cols, E);
  const Span spanDsum = dsum ? matrixSpan(dsum, ldds, rows, cols, E) : none;
  const Span other[] = {vectorSpan(dgamma, cols * PE), vectorSpan(workspace, need)};
  const Span all[] = {matrixSpan(dx, lddx, rows, cols, E), other[0], other[1]};
  const Span in[] = {vectorSpan(gamma, cols * PE), vectorSpan(rstd, rows * 4), unlessInPlace(spanDy, lddy, dx, lddx),
                     unlessInPlace(spanS, lds, dx, lddx), unlessInPlace(spanDsum, ldds, dx, lddx)};
  const Span matrices[] = {spanDy, spanS, spanDsum};
  if (!apart(all, in) || !apart(other, matrices)) return vrcclInvalidArgument;
  const bool sources = rowsAligned(dy, lddy, E) && rowsAligned(s, lds, E) && (!dsum || rowsAligned(dsum, ldds, E));
  const Lie lie = lieOf({{s, lds}, {dy, lddy}, {dsum, ldds}, {dx, lddx}}, cols, E);
  const Shape shape = rmsShape(rows, (int)cols, E, dsum ? 3 : 2, lie, false, false);
  const int blocks = rmsBlocks(rows, shape);
  RmsArgs a = {};
  a.src[0] = sourceOf(s, lds, E);
  a.src[1] = sourceOf(dy, lddy, E);
  a.src[2] = sourceOf(dsum, ldds, E);
  a.gamma = gamma;
  a.y = static_cast<char*>(dx);
  a.rstd = const_cast<float*>(rstd);
  a.partial = dgamma ? static_cast<float*>(workspace) : nullptr;
  a.ldy = lddx;
  a.rows = rows;
  a.cols = (int)cols;
  a.chunks = (int)((cols + kChunk - 1) / kChunk);
  a.ptype = paramType;
  a.wideParams = ((uintptr_t)gamma & 15) == 0;
  a.aligned = sources && cols * E % 16 == 0;
  if (shape.walk == kLong && dgamma && cols > (size_t)kLongHeld) {
    const dim3 grid((unsigned)((a.chunks + 255) / 256), (unsigned)blocks);
    const RmsFn columns = forType(dtype, [](auto dt) { return (RmsFn)rmsColumns<decltype(dt)::value>; });
    const vrcclResult_t r = launchShaped(columns, {grid, 256, 0, 0, false}, st, a);
    if (r != vrcclSuccess) return r;
  }
  const RmsFn fn = forType(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    return dsum ? pickBackward<DT, true>(shape, (int)cols) : pickBackward<DT, false>(shape, (int)cols);
  });
  const vrcclResult_t r = launchRms(fn, shape, (unsigned)blocks, a, E, st);
  if (r != vrcclSuccess || !dgamma) return r;
  return launchShaped(rmsJoin, {dim3((unsigned)((cols + 31) / 32)), 1024, 0, 0, true}, st, static_cast<const float*>(workspace), blocks,
                      (int)cols, dgamma, (int)paramType);
}

// RMS norm over the columns of a [rows, cols] matrix with the residual's
// addition, forward (to the element type, to 8 bits with scales, or both) and backward.
//
//   s  = x + residual, rounded to the element type (what is stored is what is normed)
//   y  = s rstd gamma,  rstd = 1 / sqrt(mean(s^2) + eps)
//   code = round(y / scale),  scale = max |y| over a group of columns / largest code
//   g  = dy gamma,  xh = s rstd
//   dx = dsum + rstd (g - xh mean(g xh))      (of x and of the residual alike)
//   dgamma = sum over rows of dy xh
//
// Both directions are bound by memory. A row is handled in chunks of eight
// columns, a thread holding two; it arrives in shared memory by bulk copies,
// several rows ahead, whatever element it starts on (the copy takes the
// 16-byte blocks that it touches). The barrier inside a row's reduction is also the point
// where every thread has taken its chunks, and the row's stage is filled anew
// (or, where registers do not hold the row, the stage of the one before it).
// Teams of warps walk rows of their own, so that one team's reduction runs
// under the others' loads and stores.
//
// Rows on no 16-byte boundary: where each row lies on the same skew in every
// matrix of a call, as it does in matrices of one stride, a team takes rows of
// one skew only, and its chunks are counted from the boundary before the row's
// first element. They are whole blocks in every matrix then, parts of them at a
// row's two ends, and what is shifted is gamma, once, in its registers. (16384 x
// 4097 bf16 forward 118 -> 93 us, backward 178 -> 133; 32768 x 1001 fp16 backward
// 126 -> 65.) Else a thread shifts its chunk out of two neighbouring blocks, and
// a warp takes 31 chunks and looks at the next one (ops_chunks.h); so where
// groups of columns share a scale, with 32.
//
// The weight's gradient is summed down the columns in the registers of the
// threads that own them, over all the rows that a team walks; a block joins its
// teams and writes one row of partial sums, and a second kernel adds those in
// order. No atomics: the same call gives the same bits.
//
// Short rows that start on boundaries go several to a warp (narrow); rows beyond
// a block's threads or shared memory are read twice, the second time through L2
// (long): 2048 x 16384 fp32 backward 144 us.
#include "ops_rmsnorm.cuh"

namespace vrccl {
namespace {

template <int DT, bool RES, bool Q, Lie LIE, bool WIDE>
__global__ void __launch_bounds__(32 * forwardWarps(LIE, WIDE)) rmsForward(const __grid_constant__ RmsArgs a) {
  using C = Chunk<DT>;
  constexpr int E = C::E, NP = kChunk / 2;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ unsigned long long full[kMaxTeams * kMaxStages];
  __shared__ float2 red[2][32];  // turn, warp: (sum of squares, largest)
  __shared__ int deadWord[kMaxTeams];
  Ring<E, RES ? 2 : 1, false> ring(a, smem, full, deadWord);
  const int shift = shiftOf<DT, LIE>(a, ring.first);
  const int t = ring.t, T = a.threads, lane = t & 31, warps = T / 32;
  F2 g[kHeld][NP];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) gammaOf<DT>(a, chunkOf<LIE>(a, j, warps, t), g[j], shift);
  const float inv = 1.f / (float)a.cols;
  teamSync(ring.team, T);
  for (size_t row = ring.first; row < a.rows; row += ring.stride, ring.next()) {
    const unsigned char* stage = ring.wait();
    C s[kHeld];
    F2 squares = 0;
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int ci = chunkOf<LIE>(a, j, warps, t);
      s[j] = taken<DT, LIE>(a, stage, 0, row, ci, shift);
      if constexpr (RES) addTo(s[j], taken<DT, LIE>(a, stage, 1, row, ci, shift));
      F2 x[NP];
      pairsOf(s[j], x);
      if (ownChunk<LIE>(a, t))
#pragma unroll
        for (int i = 0; i < NP; ++i) squares = fma2(x[i], x[i], squares);
      if constexpr (Q)
        if (a.group == 0) {
#pragma unroll
          for (int i = 0; i < NP; ++i) x[i] = mul2(x[i], g[j][i]);
          most = maxOrNan(most, largest(x));
        }
      // (in place: the row is in shared memory)
      if (RES && a.sum) putChunk<DT, LIE>(a, a.sum, a.lds, row, s[j], ci, shift);
    }
    float2 w = make_float2(warpSum(sumOf(squares)), most);
    if constexpr (Q)
      if (a.group == 0) w.y = largestOfLanes<32>(most);
    if (lane == 0) red[ring.turn][threadIdx.x >> 5] = w;
    if (ring.sync(row)) break;
    if (warps > 1) {
      w = lane < warps ? red[ring.turn][ring.team * warps + lane] : make_float2(0.f, 0.f);
      w.x = sumOfLanes<32>(w.x);
      if constexpr (Q)
        if (a.group == 0) w.y = largestOfLanes<32>(w.y);
    }
    const float rstd = rsqrtf(w.x * inv + a.eps);
    if (t == 0 && a.rstd) a.rstd[row] = rstd;
    const F2 scale = pair(rstd, rstd);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int ci = chunkOf<LIE>(a, j, warps, t);
      F2 x[NP];
      pairsOf(s[j], x);
#pragma unroll
      for (int i = 0; i < NP; ++i) x[i] = mul2(mul2(x[i], scale), g[j][i]);
      if (!RES && a.sum) putChunk<DT, LIE>(a, a.sum, a.lds, row, s[j], ci, shift);
      if (!Q || a.y) putChunk<DT, LIE>(a, a.y, a.ldy, row, packed<DT>(x), ci, shift);
      if constexpr (Q) storeGroup(a, row, ci, x, w.y * rstd, ownChunk<LIE>(a, t), shift);
    }
  }
}

template <int DT, int G, bool RES, bool Q>
__global__ void __launch_bounds__(kNarrowThreads, RES || DT == vrcclFloat32 ? 2 : 4) rmsForwardNarrow(const __grid_constant__ RmsArgs a) {
  using C = Chunk<DT>;
  constexpr int NP = kChunk / 2, R = 32 / G, U = kNarrowTurn;
  const int lane = threadIdx.x & 31, own = lane % G;
  const bool held = own < a.chunks;
  const size_t warps = (size_t)gridDim.x * (kNarrowThreads / 32);
  const float inv = 1.f / (float)a.cols;
  F2 g[NP];
  gammaOf<DT>(a, own, g);
  for (size_t r0 = ((size_t)blockIdx.x * (kNarrowThreads / 32) + (threadIdx.x >> 5)) * R * U; r0 < a.rows; r0 += warps * R * U) {
    C s[U], r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t row = r0 + u * R + lane / G;
      s[u] = narrowChunk<DT>(a.src[0], row, own, held && row < a.rows);
      if constexpr (RES) r[u] = narrowChunk<DT>(a.src[1], row, own, held && row < a.rows);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t row = r0 + u * R + lane / G;
      if constexpr (RES) addTo(s[u], r[u]);
      F2 x[NP], squares = 0;
      pairsOf(s[u], x);
#pragma unroll
      for (int i = 0; i < NP; ++i) squares = fma2(x[i], x[i], squares);
      const float rstd = rsqrtf(sumOfLanes<G>(sumOf(squares)) * inv + a.eps);
      const F2 scale = pair(rstd, rstd);
#pragma unroll
      for (int i = 0; i < NP; ++i) x[i] = mul2(mul2(x[i], scale), g[i]);
      const bool there = held && row < a.rows;
      if (there) {
        if (own == 0 && a.rstd) a.rstd[row] = rstd;
        if (a.sum) storeNarrow<DT>(a.sum, row, a.lds, own, s[u]);
        if (!Q || a.y) storeNarrow<DT>(a.y, row, a.ldy, own, packed<DT>(x));
      }
      if constexpr (Q) {
        const int lanes = a.group ? min(G, a.group / kChunk) : G;
        float most = largest(x);
#pragma unroll
        for (int o = 1; o < G; o *= 2) {
          const float other = __shfl_xor_sync(0xffffffffu, most, o);
          if (o < lanes) most = maxOrNan(most, other);
        }
        if (there) {
          const float q = scaleOf(most, a.quant);
          if (own % lanes == 0) a.scales[row * a.ldsc + own / lanes] = q;
          storeCodes(a.codes + row * a.ldc + own * kChunk, x, q, a.quant, 0, kChunk);
        }
      }
    }
  }
}

template <int DT, bool RES, bool Q>
__global__ void __launch_bounds__(kLongThreads) rmsForwardLong(const __grid_constant__ RmsArgs a) {
  using C = Chunk<DT>;
  constexpr int NP = kChunk / 2;
  __shared__ float2 red[2][32];
  const float inv = 1.f / (float)a.cols;
  const int lane = threadIdx.x & 31;
  int turn = 0;
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    F2 squares = 0;
    float most = 0.f;
    auto sumAt = [&](int ci) {
      C s = longChunk<DT>(a, 0, row, ci);
      if constexpr (RES) addTo(s, longChunk<DT>(a, 1, row, ci));
      s.cut(a.cols - ci * kChunk);
      return s;
    };
    for (int ci = threadIdx.x; ci - lane < a.chunks; ci += kLongThreads) {
      const C s = sumAt(ci);
      F2 x[NP], g[NP];
      pairsOf(s, x);
#pragma unroll
      for (int i = 0; i < NP; ++i) squares = fma2(x[i], x[i], squares);
      if constexpr (Q)
        if (a.group == 0) {
          gammaOf<DT>(a, ci, g);
#pragma unroll
          for (int i = 0; i < NP; ++i) x[i] = mul2(x[i], g[i]);
          most = maxOrNan(most, largest(x));
        }
    }
    float2 w = make_float2(warpSum(sumOf(squares)), Q ? largestOfLanes<32>(most) : 0.f);
    if (lane == 0) red[turn][threadIdx.x >> 5] = w;
    __syncthreads();
    w = red[turn][lane];
    w.x = warpSum(w.x);
    if constexpr (Q) w.y = largestOfLanes<32>(w.y);
    const float rstd = rsqrtf(w.x * inv + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
    const F2 scale = pair(rstd, rstd);
    for (int ci = threadIdx.x; ci - lane < a.chunks; ci += kLongThreads) {
      const C s = sumAt(ci);
      F2 x[NP], g[NP];
      pairsOf(s, x);
      gammaOf<DT>(a, ci, g);
#pragma unroll
      for (int i = 0; i < NP; ++i) x[i] = mul2(mul2(x[i], scale), g[i]);
      // (in place: a chunk's elements are read by its own lane alone, before this)
      if (a.sum) putChunk<DT, kAny>(a, a.sum, a.lds, row, s, ci, 0);
      if (!Q || a.y) putChunk<DT, kAny>(a, a.y, a.ldy, row, packed<DT>(x), ci, 0);
      if constexpr (Q) storeGroup(a, row, ci, x, w.y * rstd, true);
    }
  }
}

template <int DT, bool RES, bool Q>
RmsFn pickForward(const Shape& s) {
  if (s.walk == kRing) {
    if (s.wide)
      return s.lie == kWhole ? rmsForward<DT, RES, Q, kWhole, true> : s.lie == kSame ? rmsForward<DT, RES, Q, kSame, true> : rmsForward<DT, RES, Q, kAny, true>;
    return s.lie == kWhole ? rmsForward<DT, RES, Q, kWhole, false> : s.lie == kSame ? rmsForward<DT, RES, Q, kSame, false> : rmsForward<DT, RES, Q, kAny, false>;
  }
  if (s.walk == kLong) return rmsForwardLong<DT, RES, Q>;
  return s.lanes == 4 ? rmsForwardNarrow<DT, 4, RES, Q> : s.lanes == 8 ? rmsForwardNarrow<DT, 8, RES, Q> : rmsForwardNarrow<DT, 16, RES, Q>;
}

}  // namespace

int rmsStatus(int* code) { return cudaMemcpyFromSymbol(code, gRingStatus, sizeof(*code)); }

}  // namespace vrccl

using namespace vrccl;

extern "C" vrcclResult_t vrcclRmsNormForward(const void* x, size_t ldx, const void* residual, size_t ldr, const void* gamma,
                                             void* sum, size_t lds, void* y, size_t ldy, void* codes, size_t ldc,
                                             float* scales, size_t ldsc, float* rstd, size_t rows, size_t cols,
                                             vrcclDataType_t dtype, vrcclDataType_t paramType, vrcclQuant_t quant,
                                             size_t group, float eps, vrcclStream_t stream) {
  if (!goodSizes(rows, cols, dtype, paramType) || !(eps >= 0.f)) return vrcclInvalidArgument;
  if (rows == 0 || cols == 0) return vrcclSuccess;
  const int E = floatTypeSize(dtype), PE = floatTypeSize(paramType);
  if (!goodMatrix(x, ldx, rows, cols, E) || (residual && !goodMatrix(residual, ldr, rows, cols, E)) ||
      (sum && !goodMatrix(sum, lds, rows, cols, E)) || (y && !goodMatrix(y, ldy, rows, cols, E)) || (!y && !codes))
    return vrcclInvalidArgument;
  if ((gamma && !goodVector(gamma, PE)) || (rstd && !goodVector(rstd, 4))) return vrcclInvalidArgument;
  size_t groups = 0;
  if (codes) {
    if ((quant != vrcclQuantInt8 && quant != vrcclQuantE4M3) || (group != 0 && group != 32 && group != 64 && group != 128))
      return vrcclInvalidArgument;
    groups = group ? (cols + group - 1) / group : 1;
    if (!goodMatrix(codes, ldc, rows, cols, 1) || !goodMatrix(scales, ldsc, rows, groups, 4)) return vrcclInvalidArgument;
  }
  const Span spanX = matrixSpan(x, ldx, rows, cols, E), none = vectorSpan(nullptr, 0);
  const Span spanR = residual ? matrixSpan(residual, ldr, rows, cols, E) : none;
  const Span rest[] = {codes ? matrixSpan(codes, ldc, rows, cols, 1) : none, codes ? matrixSpan(scales, ldsc, rows, groups, 4) : none,
                       vectorSpan(rstd, rows * 4)};
  const Span in[] = {spanX, spanR, vectorSpan(gamma, cols * PE)};
  const Span spanSum = sum ? matrixSpan(sum, lds, rows, cols, E) : none, spanY = y ? matrixSpan(y, ldy, rows, cols, E) : none;
  const Span matrices[] = {spanSum, spanY};
  const Span besideSum[] = {unlessInPlace(spanX, ldx, sum, lds), unlessInPlace(spanR, ldr, sum, lds), in[2]};
  const Span besideY[] = {unlessInPlace(spanX, ldx, y, ldy), unlessInPlace(spanR, ldr, y, ldy), in[2], spanSum};
  if (!apart(rest, in) || !apart(rest, matrices) || !apart({spanSum}, besideSum) || !apart({spanY}, besideY))
    return vrcclInvalidArgument;
  const Lie lie = lieOf({{x, ldx}, {residual, ldr}, {sum, lds}, {y, ldy}}, cols, E);
  const Shape s = rmsShape(rows, (int)cols, E, residual ? 2 : 1, lie, true, codes && group);
  RmsArgs a = {};
  a.src[0] = sourceOf(x, ldx, E);
  a.src[1] = sourceOf(residual, ldr, E);
  a.gamma = gamma;
  a.y = static_cast<char*>(y);
  a.sum = static_cast<char*>(sum);
  a.codes = static_cast<unsigned char*>(codes);
  a.scales = scales;
  a.rstd = rstd;
  a.ldy = ldy;
  a.lds = lds;
  a.ldc = ldc;
  a.ldsc = ldsc;
  a.rows = rows;
  a.cols = (int)cols;
  a.chunks = (int)((cols + kChunk - 1) / kChunk);
  a.ptype = paramType;
  a.wideParams = ((uintptr_t)gamma & 15) == 0;
  a.aligned = rowsAligned(x, ldx, E) && (!residual || rowsAligned(residual, ldr, E)) && cols * E % 16 == 0;
  a.quant = quant;
  a.group = (int)group;
  a.eps = eps;
  const RmsFn fn = forType(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    return residual ? (codes ? pickForward<DT, true, true>(s) : pickForward<DT, true, false>(s))
                    : (codes ? pickForward<DT, false, true>(s) : pickForward<DT, false, false>(s));
  });
  return launchRms(fn, s, (unsigned)rmsBlocks(rows, s), a, E, (cudaStream_t)stream);
}

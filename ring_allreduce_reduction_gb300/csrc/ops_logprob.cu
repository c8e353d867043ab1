// Log probabilities of given tokens, entropy and the likeliest alternatives,
// forward, and the gradient of the first two.
//
// Over a row's logits s with temperature T, m their largest:
//
//   x_v      = (s_v - m) / T,   L = log sum_v exp(x_v),   log q_v = x_v - L
//   logprob  = log q_token,     H = -sum_v q_v log q_v = L - sum_v exp(x_v) x_v / sum_v exp(x_v)
//   d logprob / d s_v = (1[v = token] - q_v) / T
//   d H / d s_v       = -q_v (log q_v + H) / T
//
// Forward reads the logits once. A thread keeps its largest logit m, the sum l
// of 2^x and the sum w of 2^x x over what it has seen, where x = s c - M, c =
// log2(e) / T and M is m c rounded: one operation for x, rounded once, and M's
// own rounding is taken back exactly at the end (M - m c is one more). When m
// grows by d (in units of x), w' = (w + l d) 2^d and l' = l 2^d. The passes are
// bound by issue slots nearly as much as by memory, so that the loop looks at
// nothing else: a product of 0 and -inf (a masked entry, of -inf or the type's lowest
// value), an M beyond binary32
// or a NaN leave w not finite, and the thread then takes the step back and goes
// on with care: x = (s - m) c, held above -1000, where 2^x and 2^x x are 0. A
// NaN stays NaN through that bound. So do rows whose M is no longer small
// beside 2^24.
//
// The k likeliest entries, in the order (larger logit, lower index). A warp's
// load reads 512 bytes of the row, and the largest logit of such a segment (or
// of a few after one another) costs one reduction over the lanes. Of the
// segments in the order (larger largest logit, lower index) the first k hold
// all the k entries wanted: fewer than k have a larger logit than the k-th
// one's, and an entry equal to that has as many of lower index before it. Those
// segments are read once more by the whole block, and what reaches the k-th
// one's largest (k entries do) is collected; places, of segments and of
// entries, are counts of what is above. Of ties there may be too many to
// collect (a row of one value): each warp then keeps its best in order, one a
// lane, and the warps' lists are merged two and two. Many short rows go a warp
// each, whose steps need no barrier.
//
// Backward reads the logits and writes the gradient; the statistics are saved,
// so that a row may be cut into independent slices.
//
// Rows whose token lies outside the vocabulary (padding) read no logits forward and have results
// of zero; rows of nothing but -inf have no distribution: logprob -inf, entropy
// 0, gradient 0.
#include <cooperative_groups.h>

#include <type_traits>

#include "ops_common.cuh"

namespace vrccl {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;  // of a block, at most
constexpr int kUnroll = 4;     // vectors a thread asks for at once
constexpr int kPass = 32 * kUnroll;  // vectors of a warp's pass
constexpr int kSegments = 512;       // of a block's part of a row, at most
constexpr int kCollected = 512;      // entries, at most
constexpr float kFloor = -1000.f;  // 2^-1000 is 0 in binary32, and its product with -1000 too
constexpr float kLn2 = 0.6931471805599453f;

struct LogProbArgs {
  const void* logits;
  const void* token;
  float* logprob;
  float* entropy;
  float2* stats;
  float* top;
  int* topIndex;
  const float* dlogprob;
  const float* dentropy;
  void* dlogits;
  size_t ldl, ldt, ldi, ldd, lstride, hstride, vocab, rows;
  size_t slice;  // backward: elements of a row one block takes
  int k, span, shift;  // span: loads of a segment, 2^shift
  bool wide;  // 64-bit tokens
  float invT;
};

// The row's token; -1: none given (no list), -2: one outside the vocabulary.
__device__ __forceinline__ long long tokenOf(const LogProbArgs& a, size_t row) {
  if (!a.token) return -1;
  const long long t = a.wide ? static_cast<const long long*>(a.token)[row] : static_cast<const int*>(a.token)[row];
  return t >= 0 && (unsigned long long)t < a.vocab ? t : -2;
}

// A key orders entries as the list does: the logit's bits made ascending (zeros of either sign alike, a NaN above
// everything) over the inverted index. 0: no entry.
using Key = unsigned long long;
__device__ __forceinline__ uint32_t ascending(float s) {
  const uint32_t b = s == s ? __float_as_uint(s + 0.f) : 0x7fffffffu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float fromAscending(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u); }

// m, the sum l of 2^x and the sum w of 2^x x, x = (s - m) c.
struct Sums {
  float m, l, w;
};
// (s - m) c, no lower than kFloor; NaN stays.
__device__ __forceinline__ float scaled(float d, float c) { return maxOrNan(d * c, kFloor); }
// Of a warp's lanes, in every lane: relative to the largest m, then added up.
__device__ __forceinline__ Sums warpJoin(Sums r, float c) {
  const float m = fromAscending(__reduce_max_sync(0xffffffffu, ascending(r.m)));
  if (m != -INFINITY) {
    const float d = r.m == m ? 0.f : scaled(r.m - m, c), e = fastExp2(d);
    r.w = (r.w + r.l * d) * e;
    r.l *= e;
  }
  const float2 s = warpSum2(make_float2(r.l, r.w));
  return {m, s.x, s.y};
}

// The largest of a warp's lanes, NaN if one is.
__device__ __forceinline__ float largestOfWarp(float x) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));  // (not to be moved under a lane's condition)
  return r;
}
template <int DT>
__device__ __forceinline__ float largestOf(const uint4& v) {
  if constexpr (DT == vrcclFloat32) {
    return maxOrNan(maxOrNan(__uint_as_float(v.x), __uint_as_float(v.y)), maxOrNan(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else {  // two at a time
    const uint32_t p = maxPackedOrNan<DT>(maxPackedOrNan<DT>(v.x, v.y), maxPackedOrNan<DT>(v.z, v.w));
    const float2 f = unpack2<DT>(p);
    return maxOrNan(f.x, f.y);
  }
}

// With care: any values. Of the sums relative to m.
template <int N>
__device__ __forceinline__ void runOver(Sums& r, const float (&f)[N], float c) {
  float top = f[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, f[i]);
  if (top > r.m) {
    const float d = scaled(r.m - top, c), e = fastExp2(d);  // l and w are 0 while m is -inf
    r.w = (r.w + r.l * d) * e;
    r.l *= e;
    r.m = top;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (r.m == -INFINITY) {  // nothing above -inf so far
      r.l += f[i] == f[i] ? 0.f : NAN;
    } else {
      const float x = scaled(f[i] - r.m, c), e = fastExp2(x);
      r.l += e;
      r.w = fmaf(e, x, r.w);
    }
  }
}

template <int DT>
__device__ __noinline__ Sums withCare(Sums r, uint4 v, float c) {
  float f[Vec16<DT>::N];
  Vec16<DT>::expand(v, f);
  runOver<Vec16<DT>::N>(r, f, c);
  return r;
}

// A thread's running sums: relative to M (or to m, with care).
struct Stream {
  Sums s;
  float M;
  bool careful;
};
__device__ __forceinline__ Sums settled(const Stream& a, float c) {  // relative to m
  if (a.careful || a.s.m == -INFINITY) return a.s;
  const float d = fmaf(-a.s.m, c, a.M), e = exp2f(d);  // what M was rounded by
  return {a.s.m, a.s.l * e, (a.s.w + a.s.l * d) * e};
}
template <int DT, int N>
__device__ __forceinline__ float largestOf(const uint4 (&v)[N]) {  // NaN if one is
  if constexpr (DT == vrcclFloat32) {
    float top = largestOf<DT>(v[0]);
#pragma unroll
    for (int n = 1; n < N; ++n) top = maxOrNan(top, largestOf<DT>(v[n]));
    return top;
  } else {
    uint4 p = v[0];
#pragma unroll
    for (int n = 1; n < N; ++n)
      p = make_uint4(maxPackedOrNan<DT>(p.x, v[n].x), maxPackedOrNan<DT>(p.y, v[n].y), maxPackedOrNan<DT>(p.z, v[n].z), maxPackedOrNan<DT>(p.w, v[n].w));
    return largestOf<DT>(p);
  }
}
template <int DT, int N>
__device__ __forceinline__ void runOver(Stream& a, const uint4 (&v)[N], float top, float c) {
  constexpr int V = Vec16<DT>::N;
  if (!a.careful) {
    Sums r = a.s;
    float M = a.M;
    if (top > r.m) {
      const float next = top * c, d = maxOrNan(M - next, kFloor), e = fastExp2(d);  // l and w are 0 while M is -inf
      r.w = (r.w + r.l * d) * e;
      r.l *= e;
      r.m = top;
      M = next;
    }
    const F2 cc = pair(c, c), minus = pair(-M, -M);
    F2 l = 0, w = 0;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float f[V];
      Vec16<DT>::expand(v[n], f);
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const F2 x = fma2(pair(f[i], f[i + 1]), cc, minus);
        const float2 y = split(x);
        const F2 e = pair(fastExp2(y.x), fastExp2(y.y));
        l = add2(l, e);
        w = fma2(e, x, w);
      }
    }
    const float2 p = split(l), q = split(w);
    r.l += p.x + p.y;
    r.w += q.x + q.y;
    if (fabsf(r.w) < INFINITY && fabsf(M) < 0x1p24f) {  // (beyond, M's rounding is no small part of x)
      a.s = r;
      a.M = M;
      return;
    }
    a.s = settled(a, c);  // as it was before these vectors
    a.careful = true;
  }
#pragma unroll
  for (int n = 0; n < N; ++n) a.s = withCare<DT>(a.s, v[n], c);
}

// ------------------------------------------------------------ the likeliest entries
__device__ __forceinline__ Key keyOf(uint32_t value, size_t index) { return (Key)value << 32 | (uint32_t)~(uint32_t)index; }

// Lists of 32, one entry a lane, the largest in lane 0: the 32 largest of two.
__device__ __forceinline__ Key merged(Key a, const Key* other) {
  const int lane = threadIdx.x & 31;
  a = max(a, other[31 - lane]);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const Key b = __shfl_xor_sync(0xffffffffu, a, o);
    a = (lane & o) == 0 ? max(a, b) : min(a, b);
  }
  return a;
}
// The block's warps' lists into warp 0's: each step the upper half hands its lists to the lower. All threads call it; `s`
// holds 32 entries for each of WARPS / 2 warps.
template <int WARPS>
__device__ __forceinline__ Key mergedOverWarps(Key a, Key* s) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int half = WARPS / 2; half; half /= 2) {
    if (w >= half && w < 2 * half) s[(w - half) * 32 + lane] = a;
    __syncthreads();
    if (w < half) a = merged(a, s + w * 32);
    __syncthreads();
  }
  return a;
}
// Puts the lanes' candidates above `bound` into the warp's list and raises the bound to its k-th.
__device__ __forceinline__ void insert(Key& list, Key& bound, Key candidate, int k) {
  const int lane = threadIdx.x & 31;
  unsigned who;
  while ((who = __ballot_sync(0xffffffffu, candidate > bound)) != 0) {
    const int from = __ffs(who) - 1;
    const Key x = __shfl_sync(0xffffffffu, candidate, from);
    if (lane == from) candidate = 0;
    const int at = __popc(__ballot_sync(0xffffffffu, list > x));
    const Key up = __shfl_up_sync(0xffffffffu, list, 1);
    list = lane < at ? list : lane == at ? x : up;
    const Key last = __shfl_sync(0xffffffffu, list, k - 1);
    bound = last > bound ? last : bound;
  }
}
// How many of n entries are above one.
__device__ __forceinline__ int above(const Key* v, int n, Key own) {
  int count = 0;
#pragma unroll 4
  for (int j = 0; j < n; ++j) count += v[j] > own;
  return count;
}
// How many of v[0 .. n) come before number i in the order (larger, lower number). n: a multiple of 4, v aligned.
__device__ __forceinline__ int before(const uint32_t* v, int n, int i) {
  const uint32_t own = v[i];
  int count = 0;
#pragma unroll 2
  for (int j = 0; j < n; j += 4) {
    const uint4 q = *reinterpret_cast<const uint4*>(v + j);
    count += q.x > own || (q.x == own && j < i);
    count += q.y > own || (q.y == own && j + 1 < i);
    count += q.z > own || (q.z == own && j + 2 < i);
    count += q.w > own || (q.w == own && j + 3 < i);
  }
  return count;
}

// A row's elements before its first 16-byte boundary, whole vectors, and the rest.
template <int DT>
struct Row {
  using S = typename Ty<DT>::S;
  static constexpr int V = Vec16<DT>::N;
  const S* p;
  const uint4* vec;
  size_t head, nvec, vocab;

  __device__ __forceinline__ Row(const LogProbArgs& a, size_t row) : vocab(a.vocab) {
    p = reinterpret_cast<const S*>(a.logits) + row * a.ldl;
    head = min(vocab, ((16 - (uintptr_t)p % 16) % 16) / sizeof(S));
    nvec = (vocab - head) / V;
    vec = reinterpret_cast<const uint4*>(p + head);
  }
  __device__ __forceinline__ int odd() const { return (int)(vocab - nvec * V); }  // single elements
  __device__ __forceinline__ size_t oddIndex(int i) const { return (size_t)i < head ? (size_t)i : i + nvec * V; }
  __device__ __forceinline__ float at(size_t i) const { return Ty<DT>::toF(p[i]); }
};

// A thread's pass (vectors i, i + 32, ... of a row, i - lane a multiple of kPass) into its sums; own: the largest of each vector.
// AGAIN: they will soon be read once more.
template <int DT, bool AGAIN = false>
__device__ __forceinline__ void runPass(Stream& stream, const Row<DT>& in, size_t i, float (&own)[kUnroll], float c) {
  constexpr int U = kUnroll;
  if (i - (threadIdx.x & 31) + kPass <= in.nvec) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = (AGAIN ? __ldca(in.vec + i + u * 32) : __ldcs(in.vec + i + u * 32));
#pragma unroll
    for (int u = 0; u < U; ++u) own[u] = largestOf<DT>(v[u]);
    runOver<DT, U>(stream, v, maxOrNan(maxOrNan(own[0], own[1]), maxOrNan(own[2], own[3])), c);
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      own[u] = -INFINITY;
      if (i + u * 32 < in.nvec) {
        const uint4 v[1] = {(AGAIN ? __ldca(in.vec + i + u * 32) : __ldcs(in.vec + i + u * 32))};
        own[u] = largestOf<DT>(v[0]);
        runOver<DT, 1>(stream, v, own[u], c);
      }
    }
  }
}
__device__ __forceinline__ void sayPadding(const LogProbArgs& a, size_t row) {  // a warp
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    if (a.logprob) a.logprob[row] = 0.f;
    if (a.entropy) a.entropy[row] = 0.f;
    if (a.stats) a.stats[row] = make_float2(0.f, 0.f);
  }
  if (lane < a.k) {
    a.top[row * a.ldt + lane] = -INFINITY;
    a.topIndex[row * a.ldi + lane] = -1;
  }
}
// A row's results from its sums, the token's logit and the likeliest entries' keys: a warp.
template <bool TOP>
__device__ __forceinline__ void sayRow(const LogProbArgs& a, size_t row, const Sums& r, float given, const Key* best) {
  const int lane = threadIdx.x & 31;
  const bool nothing = r.m == -INFINITY && r.l == 0.f;
  const float ll = nothing ? 0.f : logf(r.l);
  auto logOf = [&](float s) { return nothing ? -INFINITY : (s - r.m) * a.invT - ll; };
  if (lane == 0) {
    if (a.logprob) a.logprob[row] = logOf(given);
    if (a.entropy) a.entropy[row] = nothing ? 0.f : ll - r.w / r.l * kLn2;
    if (a.stats) a.stats[row] = make_float2(r.m, ll);
  }
  if constexpr (TOP) {
    if (lane < a.k) {
      const Key entry = best[lane];
      a.top[row * a.ldt + lane] = entry ? logOf(fromAscending((uint32_t)(entry >> 32))) : -INFINITY;
      a.topIndex[row * a.ldi + lane] = entry ? (int)~(uint32_t)entry : -1;
    }
  }
}
template <int DT>
__device__ __forceinline__ void prefetchPass(const Row<DT>& in, size_t i) {  // into L2
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if ((threadIdx.x & 7) == 0 && i + u * 32 < in.nvec) asm volatile("prefetch.global.L2 [%0];" ::"l"(in.vec + i + u * 32));
}
// Sums of the first threads' single elements too; the warp's, joined.
template <int DT>
__device__ __forceinline__ Sums endRow(const Stream& stream, const Row<DT>& in, bool singles, float c) {
  Sums r = settled(stream, c);
  if (singles && (int)threadIdx.x < in.odd()) {
    const float f[1] = {in.at(in.oddIndex(threadIdx.x))};
    runOver<1>(r, f, c);
  }
  return warpJoin(r, c);
}

// What a block needs for the likeliest entries.
template <int T>
struct Finder {
  uint32_t tops[(kSegments > T ? kSegments : T) + 4];  // of segments, by number, or of the threads; ascending()
  uint32_t groups[kSegments];
  int segment[32];
  Key collected[kCollected];  // (or the warps' lists: T / 64 of 32)
  Key best[32];
  uint32_t least;
  int entries, candidates;
};
struct NoFinder {};

// ------------------------------------------------------------ short rows
// A warp a row: nothing but shuffles between its lanes. Each lane has the largest of either half of its vectors, and the k-th
// of those 64 bounds the k-th entry from below; what reaches it (64 log 2 = 44 entries are to be expected for k = 32, however
// long the row) is collected in a second reading.
constexpr int kShortThreads = 128, kShortCollected = 128, kShortVectors = 1024;  // (a lane has the largest logit of 32 vectors)
struct ShortFinder {
  Key collected[kShortCollected];
  Key best[32];
  int entries;
};
// The lanes' values in order, the largest in lane 0 ; of two values a lane, the 32 largest.
__device__ __forceinline__ uint32_t sortedOverLanes(uint32_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int o = size / 2; o; o /= 2) {
      const uint32_t y = __shfl_xor_sync(0xffffffffu, x, o);
      x = ((lane & o) == 0) == ((lane & size) == 0 || size == 32) ? max(x, y) : min(x, y);
    }
  return x;
}
__device__ __forceinline__ uint32_t sortedOverLanes(uint32_t x, uint32_t y) {
  const int lane = threadIdx.x & 31;
  x = max(sortedOverLanes(x), __shfl_sync(0xffffffffu, sortedOverLanes(y), 31 - lane));
#pragma unroll
  for (int o = 16; o; o /= 2) {
    const uint32_t b = __shfl_xor_sync(0xffffffffu, x, o);
    x = (lane & o) == 0 ? max(x, b) : min(x, b);
  }
  return x;
}
template <int DT, bool TOP>
__global__ void __launch_bounds__(kShortThreads, 8) logProbForwardShort(const __grid_constant__ LogProbArgs a) {
  constexpr int V = Vec16<DT>::N, U = kUnroll;
  __shared__ __align__(16) std::conditional_t<TOP, ShortFinder, NoFinder> finders[kShortThreads / 32];
  const int lane = threadIdx.x & 31;
  const size_t row = (size_t)blockIdx.x * (kShortThreads / 32) + threadIdx.x / 32;
  if (row >= a.rows) return;
  const Row<DT> in(a, row);
  const float c = a.invT * kLog2e;
  const long long token = tokenOf(a, row);
  if (token == -2) {
    sayPadding(a, row);
    return;
  }
  const float given = token >= 0 ? in.at(token) : 0.f;
  const bool single = lane < in.odd();
  const size_t singleAt = single ? in.oddIndex(lane) : 0;
  const float singleLogit = single ? in.at(singleAt) : 0.f;
  Stream stream = {{-INFINITY, 0.f, 0.f}, -INFINITY, false};
  float half[2] = {-INFINITY, -INFINITY}, top = -INFINITY;  // the lane's, and of vectors 32 lane ..
  for (size_t i = lane; i < in.nvec + lane; i += kPass) {  // (the warp's lanes together)
    float own[U];
    runPass<DT, TOP>(stream, in, i, own, c);
    if constexpr (TOP) {
      half[0] = maxOrNan(half[0], maxOrNan(own[0], own[1]));
      half[1] = maxOrNan(half[1], maxOrNan(own[2], own[3]));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float x = largestOfWarp(own[u]);
        if (lane == (int)(i / 32) + u) top = x;
      }
    }
  }
  Sums r = settled(stream, c);
  if (single) {
    const float f[1] = {singleLogit};
    runOver<1>(r, f, c);
  }
  r = warpJoin(r, c);
  if constexpr (TOP) {
    ShortFinder& find = finders[threadIdx.x / 32];
    const uint32_t first = (size_t)lane < in.nvec ? ascending(half[0]) : 0, second = (size_t)lane + 64 < in.nvec ? ascending(half[1]) : 0;
    const uint32_t enough = __shfl_sync(0xffffffffu, sortedOverLanes(first, second), a.k - 1);
    const float bound = enough ? fromAscending(enough) : -INFINITY;  // (a NaN: all are taken)
    find.best[lane] = 0;
    if (lane == 0) find.entries = 0;
    __syncwarp();
    auto push = [&](float f, size_t index) {
      const int to = atomicAdd(&find.entries, 1);
      if (to < kShortCollected) find.collected[to] = keyOf(ascending(f), index);
    };
    // the warp's loads with such entries, U at a time, to fn(a vector, whether it is one, its first element)
    const unsigned loads = __ballot_sync(0xffffffffu, !(top < bound));
    auto forAll = [&](auto fn) {
      for (unsigned rest = loads; rest;) {
        uint4 v[U];
        int i[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          i[u] = rest ? (__ffs(rest) - 1) * 32 + lane : kShortVectors;
          rest &= rest - 1;
          v[u] = i[u] < (int)in.nvec ? __ldca(in.vec + i[u]) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) fn(v[u], i[u] < (int)in.nvec, in.head + i[u] * V);
      }
    };
    forAll([&](const uint4& v, bool there, size_t first) {
      if (!there || largestOf<DT>(v) < bound) return;  // (a NaN is the largest, and not below)
      float f[V];
      Vec16<DT>::expand(v, f);
      unsigned who = 0;
#pragma unroll
      for (int e = 0; e < V; ++e) who |= f[e] < bound ? 0 : 1u << e;
      for (; who; who &= who - 1) push(in.at(first + __ffs(who) - 1), first + __ffs(who) - 1);
    });
    if (single && !(singleLogit < bound)) push(singleLogit, singleAt);
    __syncwarp();
    const int n = find.entries;
    if (n <= kShortCollected) {
      for (int j = lane; j < n; j += 32) {
        const int place = above(find.collected, n, find.collected[j]);
        if (place < a.k) find.best[place] = find.collected[j];
      }
    } else {
      Key list = 0, last = 0;
      forAll([&](const uint4& v, bool there, size_t first) {
        float f[V];
        Vec16<DT>::expand(v, f);
#pragma unroll
        for (int e = 0; e < V; ++e) insert(list, last, there ? keyOf(ascending(f[e]), first + e) : 0, a.k);
      });
      insert(list, last, single ? keyOf(ascending(singleLogit), singleAt) : 0, a.k);
      find.best[lane] = list;
    }
    __syncwarp();
    sayRow<TOP>(a, row, r, given, find.best);
  } else {
    sayRow<TOP>(a, row, r, given, nullptr);
  }
}

// A row over the blocks of a cluster, T threads each. TOP: with the likeliest entries.
template <int DT, int T, bool TOP>
__global__ void __launch_bounds__(T, T == 128 ? 8 : 3 * kThreads / T) logProbForward(const __grid_constant__ LogProbArgs a) {
  constexpr int V = Vec16<DT>::N, U = kUnroll, warps = T / 32;
  __shared__ Sums part[32];
  __shared__ Sums mine;
  __shared__ __align__(16) std::conditional_t<TOP, Finder<T>, NoFinder> find;
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned parts = cluster.num_blocks(), block = cluster.block_rank();
  const size_t row = blockIdx.x / parts;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Row<DT> in(a, row);
  const int odd = block == 0 ? in.odd() : 0;  // single elements, the first threads'
  const float c = a.invT * kLog2e;
  // runs of passes over the row, a segment each where one is longer than a pass; a block has [firstRun, lastRun), its warps in turn
  const unsigned perRun = TOP ? max(1, a.span / U) : 1, passes = (unsigned)((in.nvec + kPass - 1) / kPass), runs = (passes + perRun - 1) / perRun;
  const unsigned runsEach = (runs + parts - 1) / parts, firstRun = min(runs, runsEach * block), lastRun = min(runs, firstRun + runsEach);
  prefetchPass(in, (size_t)(firstRun + warp) * perRun * kPass + lane);  // (before it is known whether the row is read)
  const long long token = tokenOf(a, row);
  if (token == -2) {  // the whole cluster takes this way
    if (block == 0 && warp == 0) sayPadding(a, row);
    return;
  }
  Stream stream = {{-INFINITY, 0.f, 0.f}, -INFINITY, false};
  for (unsigned run = firstRun + warp; run < lastRun; run += warps) {
    float top = -INFINITY;
    for (unsigned n = 0; n < perRun; ++n) {
      const unsigned pass = run * perRun + n;
      float own[U];
      runPass<DT>(stream, in, (size_t)pass * kPass + lane, own, c);
      if constexpr (TOP) {
        auto keep = [&](float x, unsigned segment) {
          x = largestOfWarp(x);
          if (lane == 0) find.tops[segment] = ascending(x);
        };
        if (a.span == 1) {
#pragma unroll
          for (int u = 0; u < U; ++u) keep(own[u], (pass - firstRun) * U + u);
        } else if (a.span == 2) {
          keep(maxOrNan(own[0], own[1]), (pass - firstRun) * 2);
          keep(maxOrNan(own[2], own[3]), (pass - firstRun) * 2 + 1);
        } else {
          top = maxOrNan(top, maxOrNan(maxOrNan(own[0], own[1]), maxOrNan(own[2], own[3])));
          if (n == perRun - 1) keep(top, run - firstRun);
        }
      }
    }
  }
  const float given = warp == 0 && block == 0 && token >= 0 ? in.at(token) : 0.f;
  Sums r = endRow(stream, in, block == 0, c);
  if (lane == 0) part[warp] = r;
  if constexpr (TOP) {
    const int segments = (int)(lastRun - firstRun) * (a.span < U ? U / a.span : 1);
    // groups of segments, 2 k at least where there are as many: the k-th of their largest is a bound for the k-th segment's
    const int size = segments >= 8 * a.k ? 4 : segments >= 4 * a.k ? 2 : 1, groups = (segments + size - 1) / size, padded = (groups + 3) & ~3;
    if (warp == 0) {
      find.best[lane] = 0;
      find.segment[lane] = -1;
      if (lane < 4) find.tops[segments + lane] = 0;
    }
    if (threadIdx.x == 0) find.entries = find.least = find.candidates = 0;
    __syncthreads();
    for (int g = threadIdx.x; g < padded; g += T) {
      uint32_t top = 0;
      for (int j = 0; j < size; ++j) top = max(top, g < groups ? find.tops[g * size + j] : 0);
      find.groups[g] = top;
    }
    __syncthreads();
    for (int g = threadIdx.x; g < groups; g += T)
      if (before(find.groups, padded, g) == a.k - 1) find.least = find.groups[g];
    __syncthreads();
    for (int s = threadIdx.x; s < segments; s += T)
      if (find.tops[s] >= find.least) find.collected[atomicAdd(&find.candidates, 1)] = keyOf(find.tops[s], s);
    __syncthreads();
    for (int j = threadIdx.x; j < find.candidates; j += T) {
      const int place = above(find.collected, find.candidates, find.collected[j]);
      if (place < a.k) find.segment[place] = (int)~(uint32_t)find.collected[j];
      if (place == a.k - 1) find.least = (uint32_t)(find.collected[j] >> 32);
    }
    __syncthreads();
    const size_t firstVector = (size_t)firstRun * perRun * kPass, lastVector = min((size_t)lastRun * perRun * kPass, in.nvec);
    if (firstVector + (size_t)(a.k - 1) * a.span * 32 >= lastVector) {
      // too few segments hold anything for a bound: the k-th of the threads' largest is one (fewer threads: none)
      const bool some = (firstRun + warp < lastRun && (firstRun + warp) * (size_t)kPass + lane < in.nvec) || (int)threadIdx.x < odd;
      find.tops[threadIdx.x] = some ? ascending(stream.s.l == stream.s.l ? stream.s.m : INFINITY) : 0;
      __syncthreads();
      if (before(find.tops, T, threadIdx.x) == a.k - 1) find.least = find.tops[threadIdx.x];
      __syncthreads();
    }
    const uint32_t enough = max(1u, find.least);
    // the k segments' vectors, to fn(a vector, whether it is one, its first element); warps stay together
    const int number = min(segments, a.k) * a.span * 32;
    auto forAll = [&](auto fn) {
      for (int q0 = 0; q0 < number; q0 += U * T) {
        uint4 v[U];
        size_t i[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int q = q0 + u * T + threadIdx.x, load = q >> 5;
          i[u] = in.nvec;
          if (q < number) i[u] = ((size_t)firstRun * perRun * U + ((size_t)find.segment[load >> a.shift] << a.shift) + (load & (a.span - 1))) * 32 + lane;
          v[u] = i[u] < in.nvec ? __ldcg(in.vec + i[u]) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) fn(v[u], i[u] < in.nvec, in.head + i[u] * V);
      }
    };
    auto push = [&](uint32_t value, size_t index) {
      const int to = atomicAdd(&find.entries, 1);
      if (to < kCollected) find.collected[to] = keyOf(value, index);
    };
    forAll([&](const uint4& v, bool there, size_t first) {
      if (!there || ascending(largestOf<DT>(v)) < enough) return;
      float f[V];
      Vec16<DT>::expand(v, f);
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (ascending(f[e]) >= enough) push(ascending(f[e]), first + e);
    });
    const bool single = (int)threadIdx.x < odd;
    const size_t singleAt = single ? in.oddIndex(threadIdx.x) : 0;
    const uint32_t singleValue = single ? ascending(in.at(singleAt)) : 0;
    if (singleValue >= enough) push(singleValue, singleAt);
    __syncthreads();
    const int n = find.entries;
    if (n <= kCollected) {
      for (int j = threadIdx.x; j < n; j += T) {
        const int place = above(find.collected, n, find.collected[j]);
        if (place < a.k) find.best[place] = find.collected[j];
      }
    } else {
      __syncthreads();  // (all have seen the number)
      Key list = 0, bound = ((Key)enough << 32) - 1;
      forAll([&](const uint4& v, bool there, size_t first) {
        float f[V];
        Vec16<DT>::expand(v, f);
#pragma unroll
        for (int e = 0; e < V; ++e) insert(list, bound, there ? keyOf(ascending(f[e]), first + e) : 0, a.k);
      });
      insert(list, bound, single ? keyOf(singleValue, singleAt) : 0, a.k);
      list = mergedOverWarps<warps>(list, find.collected);
      if (warp == 0) find.best[lane] = list;
    }
  }
  __syncthreads();
  if (parts > 1) {
    if (warp == 0) {
      r = warpJoin(lane < warps ? part[lane] : Sums{-INFINITY, 0.f, 0.f}, c);
      if (lane == 0) mine = r;
    }
    cluster.sync();
    Key list = 0;
    if (block == 0) {
      if (warp == 0) part[lane] = lane < (int)parts ? *cluster.map_shared_rank(&mine, lane) : Sums{-INFINITY, 0.f, 0.f};
      if constexpr (TOP)
        if (warp < (int)parts) list = cluster.map_shared_rank(find.best, warp)[lane];
    }
    cluster.sync();
    if (block != 0) return;
    if constexpr (TOP) {  // (a block has as many warps as the cluster has blocks, at least)
      list = mergedOverWarps<warps>(list, find.collected);
      if (warp == 0) find.best[lane] = list;
    }
  }
  if (warp != 0) return;
  __syncwarp();
  r = warpJoin(lane < (parts > 1 ? (int)parts : warps) ? part[lane] : Sums{-INFINITY, 0.f, 0.f}, c);
  if constexpr (TOP)
    sayRow<TOP>(a, row, r, given, find.best);
  else
    sayRow<TOP>(a, row, r, given, nullptr);
}

// T threads a slice of a row: a block, or a warp (T = 32) a short row.
template <int DT, int T>
__global__ void __launch_bounds__(T == 32 ? kShortThreads : T, T == 32 ? 8 : 2 * kThreads / T) logProbBackward(const __grid_constant__ LogProbArgs a) {
  using S = typename Ty<DT>::S;
  constexpr int E = floatTypeSize(DT), V = 16 / E, U = kUnroll;
  const size_t slices = (a.vocab + a.slice - 1) / a.slice;
  const size_t row = T == 32 ? (size_t)blockIdx.x * (kShortThreads / 32) + threadIdx.x / 32 : blockIdx.x / slices, part = T == 32 ? 0 : blockIdx.x % slices;
  const unsigned thread = T == 32 ? threadIdx.x & 31 : threadIdx.x;
  if (T == 32 && row >= a.rows) return;
  const S* logits = reinterpret_cast<const S*>(a.logits) + row * a.ldl;
  S* out = reinterpret_cast<S*>(a.dlogits) + row * a.ldd;
  // A block's elements: slices are whole vectors of the output counted from its row's first boundary, and the first one
  // takes the head before it; vectors are loaded whole where the logits share the output's boundaries.
  const size_t head = min(a.vocab, ((16 - (uintptr_t)out % 16) % 16) / E);
  const bool together = ((uintptr_t)logits - (uintptr_t)out) % 16 == 0;
  const size_t from = part * a.slice, to = min(a.vocab, from + a.slice);
  const size_t begin = part == 0 ? 0 : min(a.vocab, from + head), end = to == a.vocab ? a.vocab : min(a.vocab, to + head);
  const size_t first = part == 0 ? head : begin;  // the first vector's element
  const size_t nvec = end > first ? (end - first) / V : 0, tail = first + nvec * V, edge = part == 0 ? min(head, end) : 0;
  const uint4* src = reinterpret_cast<const uint4*>(logits + first);
  uint4* dst = reinterpret_cast<uint4*>(out + first);
  size_t i = thread;
  uint4 v[U];
  if (together)
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + (size_t)u * T < nvec) v[u] = __ldcs(src + i + (size_t)u * T);
  const float2 st = a.stats[row];
  const long long token = tokenOf(a, row);
  if (token == -2 || (st.x == -INFINITY && st.y == 0.f)) {
    for (; i < nvec; i += T) __stcs(dst + i, make_uint4(0, 0, 0, 0));
    if (thread < edge) out[thread] = S(0);
    if (tail + thread < end) out[tail + thread] = S(0);
    return;
  }
  // With x = log2 q: gradient = 2^x (A + B x), and dlogprob / T more at the token.
  const float dl = a.dlogprob ? a.dlogprob[row * a.lstride] * a.invT : 0.f, dh = a.dentropy ? a.dentropy[row * a.hstride] * a.invT : 0.f;
  const float A = -(dl + (a.dentropy ? dh * a.entropy[row] : 0.f)), B = -dh * kLn2;
  const float c = a.invT * kLog2e, shift = st.y * kLog2e;
  auto at = [&](float s) {
    const float x = maxOrNan(fmaf(s - st.x, c, -shift), kFloor);
    return fastExp2(x) * fmaf(B, x, A);
  };
  const F2 minus2 = pair(-st.x, -st.x), c2 = pair(c, c), shift2 = pair(-shift, -shift), A2 = pair(A, A), B2 = pair(B, B);
  auto at2 = [&](float& a, float& b) {
    float2 x = split(fma2(add2(pair(a, b), minus2), c2, shift2));
    x.x = maxOrNan(x.x, kFloor);
    x.y = maxOrNan(x.y, kFloor);
    const float2 y = split(mul2(pair(fastExp2(x.x), fastExp2(x.y)), fma2(B2, pair(x.x, x.y), A2)));
    a = y.x;
    b = y.y;
  };
  // the vector that holds the token, and where in it
  const size_t hit = token >= 0 && (size_t)token >= first && (size_t)token < tail ? ((size_t)token - first) / V : ~size_t(0);
  const int within = (int)(((size_t)token - first) % V);
  if (together) {
    while (i < nvec) {
      uint4 w[U];
      const size_t next = i + (size_t)U * T;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (next + (size_t)u * T < nvec) w[u] = __ldcs(src + next + (size_t)u * T);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i + (size_t)u * T < nvec) {
          float f[V];
          Vec16<DT>::expand(v[u], f);
#pragma unroll
          for (int e = 0; e < V; e += 2) at2(f[e], f[e + 1]);
          if (i + (size_t)u * T == hit)
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] += e == within ? dl : 0.f;
          __stcs(dst + i + (size_t)u * T, Vec16<DT>::pack(f));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = w[u];
      i = next;
    }
  } else {
    for (; i < nvec; i += T) {
      float f[V];
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = at(Ty<DT>::toF(logits[first + i * V + e])) + (i == hit && e == within ? dl : 0.f);
      __stcs(dst + i, Vec16<DT>::pack(f));
    }
  }
  auto single = [&](size_t j) { out[j] = Ty<DT>::fromF(at(Ty<DT>::toF(logits[j])) + ((long long)j == token ? dl : 0.f)); };
  if (thread < edge) single(thread);
  if (tail + thread < end) single(tail + thread);
}

// Threads of a block: with a row in 16 vectors a thread or fewer, so that several short rows share a multiprocessor and
// one's reductions run under another's loads; more where blocks are few. `most`: at most, where there are many.
int blockThreads(size_t bytes, size_t blocks, int most) {
  const bool few = blocks < (size_t)smCount() * 2;
  int t = 128;
  while (t < (few ? kThreads : most) && bytes > t * size_t(few ? 64 : 256)) t *= 2;
  return t;
}

using LogProbFn = void (*)(LogProbArgs);
template <int DT, bool TOP>
LogProbFn pickForward(int threads) {
  return threads == 128 ? logProbForward<DT, 128, TOP> : threads == 256 ? logProbForward<DT, 256, TOP> : logProbForward<DT, 512, TOP>;
}
template <int DT>
LogProbFn pickBackward(int threads) {
  return threads == 32 ? logProbBackward<DT, 32> : threads == 128 ? logProbBackward<DT, 128> : threads == 256 ? logProbBackward<DT, 256> : logProbBackward<DT, 512>;
}

bool goodTypes(size_t rows, size_t vocab, int dtype, int ttype, float temperature) {
  return rows < (size_t(1) << 31) && vocab < (size_t(1) << 31) && isOperatorType(dtype) &&
         (ttype == vrcclInt32 || ttype == vrcclInt64) && temperature >= 1e-18f && temperature <= 1e18f;
}
LogProbArgs logProbArgs(const void* logits, size_t ldl, const void* token, int ttype, size_t vocab, float temperature) {
  LogProbArgs a = {};
  a.logits = logits;
  a.token = token;
  a.ldl = ldl;
  a.vocab = vocab;
  a.wide = ttype == vrcclInt64;
  a.invT = 1.f / temperature;
  return a;
}

}  // namespace
}  // namespace vrccl

using namespace vrccl;

extern "C" vrcclResult_t vrcclLogProbForward(const void* logits, size_t ldl, const void* token, float* logprob,
                                             float* entropy, float* stats, float* top, size_t ldt, int32_t* topIndex,
                                             size_t ldi, size_t rows, size_t vocab, size_t k, vrcclDataType_t dtype,
                                             vrcclDataType_t tokenType, float temperature, vrcclStream_t stream) {
  if (!goodTypes(rows, vocab, dtype, tokenType, temperature) || k > VRCCL_LOGPROB_MAX_K) return vrcclInvalidArgument;
  if (rows == 0) return vrcclSuccess;
  const int E = floatTypeSize(dtype), TE = tokenType == vrcclInt64 ? 8 : 4;
  if (vocab > 0 && !goodMatrix(logits, ldl, rows, vocab, E)) return vrcclInvalidArgument;
  if ((token && !goodVector(token, TE)) || (logprob && (!goodVector(logprob, 4) || !token)) ||
      (entropy && !goodVector(entropy, 4)) || (stats && !goodVector(stats, 8)))
    return vrcclInvalidArgument;
  if (k > 0 && (!goodMatrix(top, ldt, rows, k, 4) || !goodMatrix(topIndex, ldi, rows, k, 4))) return vrcclInvalidArgument;
  const Span out[] = {vectorSpan(logprob, rows * 4), vectorSpan(entropy, rows * 4), vectorSpan(stats, rows * 8),
                      k ? matrixSpan(top, ldt, rows, k, 4) : vectorSpan(nullptr, 0),
                      k ? matrixSpan(topIndex, ldi, rows, k, 4) : vectorSpan(nullptr, 0)};
  const Span in[] = {matrixSpan(logits, ldl, rows, vocab, E), vectorSpan(token, rows * TE)};
  if (!apart(out, in)) return vrcclInvalidArgument;
  LogProbArgs a = logProbArgs(logits, ldl, token, tokenType, vocab, temperature);
  a.logprob = logprob;
  a.entropy = entropy;
  a.stats = reinterpret_cast<float2*>(stats);
  a.top = top;
  a.topIndex = topIndex;
  a.ldt = ldt;
  a.ldi = ldi;
  a.k = (int)k;
  a.rows = rows;
  // split a row over a cluster until there are more than two blocks an SM (91 x 70133 fp32 13.1 us, with one 15.4; with
  // thirteen 1000 x 100000 bf16 70 for 61) or a block has less than two vectors a thread
  unsigned parts = 1;
  const size_t bytes = vocab * E;
  while (parts < 8 && rows * parts * 2 <= (size_t)smCount() * 4 && bytes / (parts * 2) >= size_t(kThreads) * 32) parts *= 2;
  const int threads = std::max(blockThreads(bytes / parts, rows * parts, 256), (int)parts * 32);
  // a segment: as few loads as make no more than kSegments of a block's part
  const size_t passes = (bytes / 16 / kPass + 1 + parts - 1) / parts + 1;
  a.span = 1;
  while (a.span < kUnroll ? passes * (kUnroll / a.span) > kSegments : passes / (a.span / kUnroll) + 1 > kSegments) a.span *= 2;
  while ((1 << a.shift) < a.span) ++a.shift;
  // a warp a row, where rows are short and many, or very short. bf16, k = 8, a warp against a block a row: 1024 columns 4 rows 3.8 / 5.3 us,
  // 400: 4.6 / 7.7, 20000: 28 / 152; 4096 columns 400 rows 8.7 / 6.5, 2000: 9.2 / 14.8, 20000: 52 / 122; 8192 columns 1000 rows 12.0 / 10.2, 5000:
  // 29 / 40; 20000: 78 / 144; 16384 columns 10000 rows (with longer segments) 118 / 98. Without a list 20000 x 4096 31 / 48.
  const bool brief = bytes <= kShortVectors * 16 && (bytes <= 4096 || rows >= bytes / 8);
  auto pick = [&](auto dt) -> LogProbFn {
    constexpr int DT = decltype(dt)::value;
    if (brief) return k ? logProbForwardShort<DT, true> : logProbForwardShort<DT, false>;
    return k ? pickForward<DT, true>(threads) : pickForward<DT, false>(threads);
  };

  const LogProbFn fn = dtype == vrcclFloat32    ? pick(std::integral_constant<int, vrcclFloat32>{})
                       : dtype == vrcclBfloat16 ? pick(std::integral_constant<int, vrcclBfloat16>{})
                                                : pick(std::integral_constant<int, vrcclFloat16>{});
  if (brief) return launchShaped(fn, {dim3((unsigned)((rows + kShortThreads / 32 - 1) / (kShortThreads / 32))), kShortThreads, 0, 0, false}, (cudaStream_t)stream, a);
  return launchShaped(fn, {dim3((unsigned)(rows * parts)), threads, 0, (int)parts, false}, (cudaStream_t)stream, a);
}

extern "C" vrcclResult_t vrcclLogProbBackward(const void* logits, size_t ldl, const void* token, const float* stats,
                                              const float* entropy, const float* dlogprob, size_t dlogprobStride,
                                              const float* dentropy, size_t dentropyStride, void* dlogits, size_t ldd,
                                              size_t rows, size_t vocab, vrcclDataType_t dtype, vrcclDataType_t tokenType,
                                              float temperature, vrcclStream_t stream) {
  if (!goodTypes(rows, vocab, dtype, tokenType, temperature)) return vrcclInvalidArgument;
  if (rows == 0 || vocab == 0) return vrcclSuccess;
  const int E = floatTypeSize(dtype), TE = tokenType == vrcclInt64 ? 8 : 4;
  if (!goodMatrix(logits, ldl, rows, vocab, E) || !goodMatrix(dlogits, ldd, rows, vocab, E) || !goodVector(stats, 8))
    return vrcclInvalidArgument;
  if ((token && !goodVector(token, TE)) || (dlogprob && (!goodVector(dlogprob, 4) || !token)) ||
      (dentropy && (!goodVector(dentropy, 4) || !goodVector(entropy, 4))) || (!dlogprob && !dentropy))
    return vrcclInvalidArgument;
  for (size_t stride : {dlogprobStride, dentropyStride})
    if (stride >= kMaxExtent || rows - 1 > (size_t(1) << 46) / std::max<size_t>(1, stride)) return vrcclInvalidArgument;
  const Span out[] = {matrixSpan(dlogits, ldd, rows, vocab, E)};
  const Span in[] = {unlessInPlace(matrixSpan(logits, ldl, rows, vocab, E), ldl, dlogits, ldd),
                     vectorSpan(token, rows * TE),
                     vectorSpan(stats, rows * 8),
                     vectorSpan(dentropy ? entropy : nullptr, rows * 4),
                     dlogprob ? matrixSpan(dlogprob, dlogprobStride, rows, 1, 4) : vectorSpan(nullptr, 0),
                     dentropy ? matrixSpan(dentropy, dentropyStride, rows, 1, 4) : vectorSpan(nullptr, 0)};
  if (!apart(out, in)) return vrcclInvalidArgument;
  LogProbArgs a = logProbArgs(logits, ldl, token, tokenType, vocab, temperature);
  a.stats = const_cast<float2*>(reinterpret_cast<const float2*>(stats));
  a.entropy = const_cast<float*>(entropy);
  a.dlogprob = dlogprob;
  a.dentropy = dentropy;
  a.lstride = dlogprobStride;
  a.hstride = dentropyStride;
  a.dlogits = dlogits;
  a.rows = rows;
  a.ldd = ldd;
  // even pieces, until there are four blocks a multiprocessor or a piece has 32 KB. (In place too: an element is read by the
  // thread that writes it, and by no other.)
  const size_t unit = size_t(kThreads) * (16 / E);
  const size_t pieces = std::max<size_t>(1, std::min((size_t)smCount() * 4 / rows, vocab * E / 32768));
  a.slice = std::min(vocab, ((vocab + pieces - 1) / pieces + unit - 1) / unit * unit);
  const size_t slices = (vocab + a.slice - 1) / a.slice;
  if (rows * slices >= (size_t(1) << 31)) return vrcclInvalidArgument;
  // as many blocks as four a multiprocessor are all at work at once with 256 threads each
  // a warp a row: 1467 x 1269 bf16 4.0 us for 4.9, 20000 x 1024 17 for 38, 20000 x 4096 52 for 54 (8192 columns 104 for 95)
  const bool brief = vocab * E <= 8192 && rows >= (size_t)smCount() * 8;
  const int threads = brief ? 32 : rows * slices <= (size_t)smCount() * 4 ? 256 : blockThreads(a.slice * E, rows * slices, kThreads);
  const LogProbFn fn = dtype == vrcclFloat32    ? pickBackward<vrcclFloat32>(threads)
                       : dtype == vrcclBfloat16 ? pickBackward<vrcclBfloat16>(threads)
                                                : pickBackward<vrcclFloat16>(threads);
  const size_t blocks = brief ? (rows + kShortThreads / 32 - 1) / (kShortThreads / 32) : rows * slices;
  return launchShaped(fn, {dim3((unsigned)blocks), brief ? kShortThreads : threads, 0, 0, false}, (cudaStream_t)stream, a);
}

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
// Forward reads the logits once: each thread keeps its largest logit m, the
// sum l of exp(x) and the sum w of exp(x) x, rescaled when m grows:
// with d = (m - m') / T, w' = (w + l d) exp(d), l' = l exp(d). Terms of
// masked entries (-inf or the type's lowest value) are exp(-inf) x = 0: x is
// held above -1000 (base 2), where its power is 0 in binary32. A NaN stays NaN
// through that bound.
//
// The k likeliest entries, in the order (larger logit, lower index), are found
// from the largest logits m_t that the threads hold anyway: the k-th largest
// of them is a bound that k entries reach, and so do all of the k wanted. The
// few threads whose m_t reaches it have their elements read once more (about
// k of 512 threads' shares, mostly from L2), a warp a share, each warp keeping its best in order, one a
// lane; the warps' lists (and the blocks') are merged two and two. Whatever
// the logits hold, the lists are right: ties only mean more shares to read.
//
// Backward reads the logits and writes the gradient; the statistics are saved,
// so that a row may be cut into independent slices.
//
// Rows whose token lies outside the vocabulary (padding) read no logits forward and have results
// of zero; rows of nothing but -inf have no distribution: logprob -inf, entropy
// 0, gradient 0.
#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace vrccl {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;  // of a block, at most
constexpr int kUnroll = 4;     // vectors a thread asks for at once
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
  size_t ldl, ldt, ldi, ldd, lstride, hstride, vocab;
  size_t slice;  // backward: elements of a row one block takes
  int k;
  bool wide;  // 64-bit tokens
  float temperature, invT;
};

// The row's token; -1: none given (no list), -2: one outside the vocabulary.
__device__ __forceinline__ long long tokenOf(const LogProbArgs& a, size_t row) {
  if (!a.token) return -1;
  const long long t = a.wide ? static_cast<const long long*>(a.token)[row] : static_cast<const int*>(a.token)[row];
  return t >= 0 && (unsigned long long)t < a.vocab ? t : -2;
}

// m, the sum l of 2^x and the sum w of 2^x x, x = (s - m) c.
struct Sums {
  float m, l, w;
};
// (s - m) c, no lower than kFloor; NaN stays.
__device__ __forceinline__ float scaled(float d, float c) { return maxOrNan(d * c, kFloor); }
__device__ __forceinline__ Sums joined(const Sums& a, const Sums& b, float c) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  if (r.m == -INFINITY) return {r.m, a.l + b.l, a.w + b.w};  // nothing above -inf: both zero, or NaN
  const float da = a.m == r.m ? 0.f : scaled(a.m - r.m, c), db = b.m == r.m ? 0.f : scaled(b.m - r.m, c);
  const float ea = exp2f(da), eb = exp2f(db);
  r.l = a.l * ea + b.l * eb;
  r.w = (a.w + a.l * da) * ea + (b.w + b.l * db) * eb;
  return r;
}
__device__ __forceinline__ Sums warpJoin(Sums r, float c) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Sums b;
    b.m = __shfl_xor_sync(0xffffffffu, r.m, o);
    b.l = __shfl_xor_sync(0xffffffffu, r.l, o);
    b.w = __shfl_xor_sync(0xffffffffu, r.w, o);
    // the same order on both sides: every lane has the same bits
    r = (threadIdx.x & o) ? joined(b, r, c) : joined(r, b, c);
  }
  return r;
}

template <int DT>
__device__ __forceinline__ float largestOf(const uint4& v) {
  if constexpr (DT == vrcclFloat32) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else {  // two at a time; a NaN loses
    const uint32_t p = maxPacked<DT>(maxPacked<DT>(v.x, v.y), maxPacked<DT>(v.z, v.w));
    const float2 f = unpack2<DT>(p);
    return fmaxf(f.x, f.y);
  }
}

template <int N>
__device__ __forceinline__ void runOver(Sums& r, const float (&f)[N], float top, float c) {
  if (top > r.m) {
    const float d = scaled(r.m - top, c), e = fastExp2(d);  // l and w are 0 while m is -inf
    r.w = (r.w + r.l * d) * e;
    r.l *= e;
    r.m = top;
  }
  if (r.m == -INFINITY) {  // nothing above -inf so far
#pragma unroll
    for (int i = 0; i < N; ++i) r.l += f[i] == f[i] ? 0.f : NAN;
  } else if constexpr (N % 2 == 0) {
    const F2 minus = pair(-r.m, -r.m), cc = pair(c, c);
    F2 l = 0, w = 0;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float2 x = split(mul2(add2(pair(f[i], f[i + 1]), minus), cc));
      x.x = maxOrNan(x.x, kFloor);
      x.y = maxOrNan(x.y, kFloor);
      const F2 e = pair(fastExp2(x.x), fastExp2(x.y));
      l = add2(l, e);
      w = fma2(e, pair(x.x, x.y), w);
    }
    const float2 a = split(l), b = split(w);
    r.l += a.x + a.y;
    r.w += b.x + b.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = scaled(f[i] - r.m, c), e = fastExp2(x);
      r.l += e;
      r.w = fmaf(e, x, r.w);
    }
  }
}

// ------------------------------------------------------------ the likeliest entries
// A key orders entries as the list does: the logit's bits made ascending (zeros of either sign alike, a NaN above
// everything) over the inverted index. 0: no entry.
using Key = unsigned long long;
__device__ __forceinline__ uint32_t ascending(float s) {
  const uint32_t b = s == s ? __float_as_uint(s + 0.f) : 0x7fffffffu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float fromAscending(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u); }
__device__ __forceinline__ Key keyOf(uint32_t value, size_t index) { return (Key)value << 32 | (uint32_t)~(uint32_t)index; }

// Lists of 32, one entry a lane, the largest in lane 0.
template <typename K>
__device__ __forceinline__ K tidied(K a) {  // a bitonic list into order
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const K b = __shfl_xor_sync(0xffffffffu, a, o);
    a = ((lane & o) == 0) == (a > b) ? a : b;
  }
  return a;
}
template <typename K>
__device__ __forceinline__ K sorted(K a) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll
    for (int o = n / 2; o; o >>= 1) {
      const K b = __shfl_xor_sync(0xffffffffu, a, o);
      a = (((lane & o) == 0) == ((lane & n) == 0)) == (a > b) ? a : b;
    }
  return a;
}
// The 32 largest of two lists in order, in order.
template <typename K>
__device__ __forceinline__ K merged(K a, const K* other) {
  const K b = other[31 - (threadIdx.x & 31)];
  return tidied(a > b ? a : b);
}
// The block's warps' lists into warp 0's: each step the upper half hands its lists to the lower. All threads call it; `s`
// holds 32 entries for each of warps / 2 warps.
template <typename K, int WARPS>
__device__ __forceinline__ K mergedOverWarps(K a, K* s) {
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

// T threads a block, a compile-time stride.
template <int DT, int T>
__global__ void __launch_bounds__(T, 3 * kThreads / T) logProbForward(const __grid_constant__ LogProbArgs a) {
  using S = typename Ty<DT>::S;
  constexpr int E = floatTypeSize(DT), V = 16 / E, U = kUnroll, warps = T / 32;
  __shared__ Sums part[32];
  __shared__ Sums mine;
  __shared__ Key best[warps / 2 * 32];
  __shared__ int flagged[T];
  __shared__ int flags;
  __shared__ uint32_t least;
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned parts = cluster.num_blocks(), rank = cluster.block_rank();
  const size_t row = blockIdx.x / parts;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const S* logits = reinterpret_cast<const S*>(a.logits) + row * a.ldl;
  // [head | whole 16-byte vectors | tail] of the row; the vectors are dealt to the blocks in runs
  const size_t head = min(a.vocab, ((16 - (uintptr_t)logits % 16) % 16) / E);
  const size_t nvec = (a.vocab - head) / V, tail = head + nvec * V;
  const size_t per = (nvec + parts - 1) / parts;
  const size_t lo = min(nvec, per * rank), hi = min(nvec, lo + per);
  const uint4* vec = reinterpret_cast<const uint4*>(logits + head);
  const int odd = rank == 0 ? (int)(head + (a.vocab - tail)) : 0;  // single elements, the first threads'
  auto oddIndex = [&](int i) { return (size_t)i < head ? (size_t)i : i - head + tail; };
  const float c = a.invT * kLog2e;
  size_t i = lo + threadIdx.x;
  // until it is known whether the row is read, its first vectors come into L2
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (threadIdx.x % 8 == 0 && i + (size_t)u * T < hi)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(vec + i + (size_t)u * T));
  const long long token = tokenOf(a, row);
  if (token == -2) {  // the whole cluster takes this way
    if (rank == 0 && threadIdx.x == 0) {
      if (a.logprob) a.logprob[row] = 0.f;
      if (a.entropy) a.entropy[row] = 0.f;
      if (a.stats) a.stats[row] = make_float2(0.f, 0.f);
    }
    if (rank == 0 && threadIdx.x < a.k) {
      a.top[row * a.ldt + threadIdx.x] = -INFINITY;
      a.topIndex[row * a.ldi + threadIdx.x] = -1;
    }
    return;
  }
  Sums r = {-INFINITY, 0.f, 0.f};
  for (; i + (size_t)(U - 1) * T < hi; i += (size_t)U * T) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = __ldcs(vec + i + (size_t)u * T);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[V];
      Vec16<DT>::expand(v[u], f);
      runOver<V>(r, f, largestOf<DT>(v[u]), c);
    }
  }
  for (; i < hi; i += T) {
    const uint4 v = __ldcs(vec + i);
    float f[V];
    Vec16<DT>::expand(v, f);
    runOver<V>(r, f, largestOf<DT>(v), c);
  }
  if ((int)threadIdx.x < odd) {
    const float f[1] = {Ty<DT>::toF(logits[oddIndex(threadIdx.x)])};
    runOver<1>(r, f, f[0], c);
  }
  Key list = 0;
  if (a.k > 0) {
    // what this thread's largest is at least (a sum of NaN: +inf or a NaN is among its elements); 0: it has none
    const uint32_t own = lo + threadIdx.x < hi || (int)threadIdx.x < odd ? ascending(r.l == r.l ? r.m : INFINITY) : 0;
    const uint32_t order = mergedOverWarps<uint32_t, warps>(sorted(own), reinterpret_cast<uint32_t*>(best));
    if (threadIdx.x == a.k - 1) least = order;
    if (threadIdx.x == 0) flags = 0;
    __syncthreads();
    const uint32_t enough = least;
    if (own && own >= enough) flagged[atomicAdd(&flags, 1)] = threadIdx.x;  // (in any order: the list does not depend on it)
    __syncthreads();
    Key bound = enough ? ((Key)enough << 32) - 1 : 0;
    for (int n = warp; n < flags; n += warps) {
      const int share = flagged[n];
      for (size_t j = lo + share; j < hi; j += (size_t)32 * T) {
        const size_t at = j + (size_t)lane * T;
        float f[V];
        Vec16<DT>::expand(at < hi ? __ldcs(vec + at) : make_uint4(0, 0, 0, 0), f);
        bool any = false;
        Key key[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          key[e] = at < hi ? keyOf(ascending(f[e]), head + at * V + e) : 0;
          any |= key[e] > bound;
        }
        if (__any_sync(0xffffffffu, any))
#pragma unroll
          for (int e = 0; e < V; ++e) insert(list, bound, key[e], a.k);
      }
      if (share < odd)
        insert(list, bound, lane == 0 ? keyOf(ascending(Ty<DT>::toF(logits[oddIndex(share)])), oddIndex(share)) : 0, a.k);
    }
    list = mergedOverWarps<Key, warps>(list, best);
  }
  r = warpJoin(r, c);
  if (lane == 0) part[warp] = r;
  __syncthreads();
  if (parts > 1) {
    if (threadIdx.x < 32) {
      r = warpJoin(lane < warps ? part[lane] : Sums{-INFINITY, 0.f, 0.f}, c);
      if (lane == 0) mine = r;
      best[lane] = list;
    }
    cluster.sync();
    if (rank == 0 && threadIdx.x < 32) {
      Sums o = {-INFINITY, 0.f, 0.f};
      if (lane < (int)parts) o = *cluster.map_shared_rank(&mine, lane);
      part[lane] = o;
      for (unsigned p = 1; a.k > 0 && p < parts; ++p) list = merged(list, cluster.map_shared_rank(best, p));
    }
    cluster.sync();
    if (rank != 0) return;
  }
  if (threadIdx.x >= 32) return;
  r = warpJoin(lane < (parts > 1 ? (int)parts : warps) ? part[lane] : Sums{-INFINITY, 0.f, 0.f}, c);
  const bool nothing = r.m == -INFINITY && r.l == 0.f;
  const float ll = nothing ? 0.f : logf(r.l);
  auto logOf = [&](float s) { return nothing ? -INFINITY : (s - r.m) * a.invT - ll; };
  if (lane == 0) {
    if (a.logprob) a.logprob[row] = logOf(Ty<DT>::toF(logits[token]));
    if (a.entropy) a.entropy[row] = nothing ? 0.f : ll - r.w / r.l * kLn2;
    if (a.stats) a.stats[row] = make_float2(r.m, ll);
  }
  if (lane < a.k) {
    a.top[row * a.ldt + lane] = list ? logOf(fromAscending((uint32_t)(list >> 32))) : -INFINITY;
    a.topIndex[row * a.ldi + lane] = list ? (int)~(uint32_t)list : -1;
  }
}

template <int DT, int T>
__global__ void __launch_bounds__(T, 2 * kThreads / T) logProbBackward(const __grid_constant__ LogProbArgs a) {
  using S = typename Ty<DT>::S;
  constexpr int E = floatTypeSize(DT), V = 16 / E, U = kUnroll;
  const size_t slices = (a.vocab + a.slice - 1) / a.slice;
  const size_t row = blockIdx.x / slices, part = blockIdx.x % slices;
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
  size_t i = threadIdx.x;
  uint4 v[U];
  if (together)
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + (size_t)u * T < nvec) v[u] = __ldcs(src + i + (size_t)u * T);
  const float2 st = a.stats[row];
  const long long token = tokenOf(a, row);
  if (token == -2 || (st.x == -INFINITY && st.y == 0.f)) {
    for (; i < nvec; i += T) __stcs(dst + i, make_uint4(0, 0, 0, 0));
    if (threadIdx.x < edge) out[threadIdx.x] = S(0);
    if (tail + threadIdx.x < end) out[tail + threadIdx.x] = S(0);
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
  if (threadIdx.x < edge) single(threadIdx.x);
  if (tail + threadIdx.x < end) single(tail + threadIdx.x);
}

// Threads of a block: with a row in 16 vectors a thread or fewer, so that several short rows share a multiprocessor and
// one's reductions run under another's loads; more where blocks are few.
int blockThreads(size_t bytes, size_t blocks) {
  int t = 128;
  const size_t most = blocks < (size_t)smCount() * 2 ? 64 : 256;  // bytes a thread
  while (t < kThreads && bytes > t * most) t *= 2;
  return t;
}

using LogProbFn = void (*)(LogProbArgs);
template <int DT>
LogProbFn pickForward(int threads) {
  return threads == 128 ? logProbForward<DT, 128> : threads == 256 ? logProbForward<DT, 256> : logProbForward<DT, 512>;
}
template <int DT>
LogProbFn pickBackward(int threads) {
  return threads == 128 ? logProbBackward<DT, 128> : threads == 256 ? logProbBackward<DT, 256> : logProbBackward<DT, 512>;
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
  a.temperature = temperature;
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
  // split a row over a cluster until the grid fills the GPU or a block has less than two vectors a thread
  unsigned parts = 1;
  const size_t bytes = vocab * E;
  while (parts < 8 && rows * parts * 2 <= (size_t)smCount() * 2 && bytes / (parts * 2) >= size_t(kThreads) * 32) parts *= 2;
  const int threads = blockThreads(bytes / parts, rows * parts);
  const LogProbFn fn = dtype == vrcclFloat32    ? pickForward<vrcclFloat32>(threads)
                       : dtype == vrcclBfloat16 ? pickForward<vrcclBfloat16>(threads)
                                                : pickForward<vrcclFloat16>(threads);
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
  a.ldd = ldd;
  // even pieces, until there are four blocks a multiprocessor or a piece has 32 KB. (In place too: an element is read by the
  // thread that writes it, and by no other.)
  const size_t unit = size_t(kThreads) * (16 / E);
  const size_t pieces = std::max<size_t>(1, std::min((size_t)smCount() * 4 / rows, vocab * E / 32768));
  a.slice = std::min(vocab, ((vocab + pieces - 1) / pieces + unit - 1) / unit * unit);
  const size_t slices = (vocab + a.slice - 1) / a.slice;
  if (rows * slices >= (size_t(1) << 31)) return vrcclInvalidArgument;
  // as many blocks as four a multiprocessor are all at work at once with 256 threads each
  const int threads = rows * slices <= (size_t)smCount() * 4 ? 256 : blockThreads(a.slice * E, rows * slices);
  const LogProbFn fn = dtype == vrcclFloat32    ? pickBackward<vrcclFloat32>(threads)
                       : dtype == vrcclBfloat16 ? pickBackward<vrcclBfloat16>(threads)
                                                : pickBackward<vrcclFloat16>(threads);
  return launchShaped(fn, {dim3((unsigned)(rows * slices)), threads, 0, 0, false}, (cudaStream_t)stream, a);
}

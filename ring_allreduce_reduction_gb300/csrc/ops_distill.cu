// Distillation from a teacher's top logits, forward and backward.
//
// A row holds the student's logits s over the whole vocabulary and the
// teacher's logits t at k of its entries. With temperature T, over the kept
// entries j (index inside the vocabulary, t_j not -inf; a NaN is kept, and shows):
//
//   p_j  = exp(t_j / T) / sum_i exp(t_i / T)
//   q_v  = exp(s_v / T) / sum_u exp(s_u / T)
//   loss = T^2 sum_j p_j (log p_j - log q_{idx_j})
//   d loss / d s_v = T (q_v - sum of p_j over the j with idx_j = v)
//
// Everything is taken relative to the row's largest logit, (s - max) / T, so
// masked entries (-inf or the type's lowest value) contribute exp(-inf) = 0
// without overflowing on the way. Forward saves max and log sum exp apart:
// their sum would round away the fraction of a large logit. An entry whose
// p_j is 0 in binary32 adds nothing, whatever q is there. A row without a kept
// entry (a padding position) has loss 0 and gradient 0 whatever its logits
// hold; forward reads none of them, backward the first few, which it asks for
// before it knows.
//
// Both directions are bound by memory: forward reads the logits once (each
// thread keeps a running maximum and a sum rescaled when the maximum grows,
// joined at the end), backward reads them and writes the gradient. Where there
// are fewer rows than multiprocessors a row is split: forward over the blocks
// of a cluster, which join their (max, sum) through distributed shared memory;
// backward over independent blocks, since the saved statistics are all an
// element needs.
//
// Measured, of a copy's 6.7 TB/s: 4096 x 131072 bf16 forward 168 us (6.4 TB/s),
// backward 337 us (6.4); fp32 forward 7.0. With 2-byte logits the passes run
// near their issue slots, hence the packed arithmetic and the constant strides.
// Shorter rows leave the reductions between loads in sight: 8192 x 32000 bf16
// forward 96 us (5.4 TB/s), backward 179 us (5.9).
#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace vrccl {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;  // of a block, at most
constexpr int kUnroll = 4;     // vectors a thread asks for at once
constexpr int kSeen = 2 * VRCCL_DISTILL_MAX_K;  // hash table slots; 2^11, which the hash is shifted to

struct DistillArgs {
  const void* logits;
  const void* teacher;
  const void* index;
  float* loss;
  float2* stats;
  const float* dloss;
  void* dlogits;
  size_t ldl, ldt, ldi, ldd, dstride, rows, vocab;
  size_t slice;  // backward: elements of a row one block takes
  int k, ttype;
  bool wide;  // 64-bit indices
  float temperature, invT;
};

__device__ __forceinline__ float warpMax(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// A thread's entries: number j of the row is thread j mod blockDim's. They are
// asked for before the row's logits and used after them.
constexpr int kOwnEntries = 2;  // blocks have at least k / 2 threads
struct Entries {
  int at[kOwnEntries];   // the index, -1 where the entry is not kept
  float t[kOwnEntries];  // the teacher's logit
  float s[kOwnEntries];  // the student's logit there
};
// true: this thread has a kept one
template <int DT>
__device__ __forceinline__ bool loadEntries(const DistillArgs& a, size_t row, Entries& en) {
  const char* logits = static_cast<const char*>(a.logits) + row * a.ldl * floatTypeSize(DT);
  const char* teacher = static_cast<const char*>(a.teacher) + row * a.ldt * (a.ttype == vrcclFloat32 ? 4 : 2);
  bool any = false;
#pragma unroll
  for (int i = 0; i < kOwnEntries; ++i) {
    const int j = threadIdx.x + i * blockDim.x;
    en.at[i] = -1;
    en.t[i] = en.s[i] = 0.f;
    if (j < a.k) {
      const long long at = a.wide ? static_cast<const long long*>(a.index)[row * a.ldi + j]
                                  : static_cast<const int*>(a.index)[row * a.ldi + j];
      en.t[i] = loadParam(teacher, a.ttype, j);
      if (at >= 0 && (unsigned long long)at < a.vocab && en.t[i] != -INFINITY) {  // a NaN is kept, and shows
        en.at[i] = (int)at;
        en.s[i] = loadOne<DT>(logits, at);
        any = true;
      }
    }
  }
  return any;
}
// The largest of this thread's kept teacher logits.
__device__ __forceinline__ float ownTop(const Entries& en) {
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kOwnEntries; ++i)
    if (en.at[i] >= 0) top = fmaxf(top, en.t[i]);
  return top;
}

// A running maximum m and the sum l of exp((x - m) invT) over what was seen.
struct Running {
  float m, l;
};
__device__ __forceinline__ float shifted(float x, float m, float invT) {
  // -inf while nothing above -inf was seen: every term is then 0
  return m == -INFINITY ? -INFINITY : (x - m) * invT;
}
__device__ __forceinline__ Running joined(Running a, Running b, float invT) {
  Running r;
  r.m = fmaxf(a.m, b.m);
  r.l = a.l * expf(shifted(a.m, r.m, invT)) + b.l * expf(shifted(b.m, r.m, invT));
  if (a.l != a.l || b.l != b.l) r.l = NAN;
  return r;
}
__device__ __forceinline__ Running warpJoin(Running r, float invT) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Running b;
    b.m = __shfl_xor_sync(0xffffffffu, r.m, o);
    b.l = __shfl_xor_sync(0xffffffffu, r.l, o);
    r = joined(r, b, invT);
  }
  return r;
}

// exp for the long sums: 2^x on the special function unit, relative error about
// 2^-22 of its own; the rounding of its argument adds |x| 2^-24, so that a
// term of 2^-100 is off by 2^-17 of itself. The terms that make up a sum have
// small arguments, and their errors average out.
__device__ __forceinline__ float fastExp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

template <int N>
__device__ __forceinline__ void runOver(Running& r, const float (&f)[N], float c) {  // c = invT log2(e)
  float top = f[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, f[i]);
  if (top > r.m) {
    r.l *= fastExp2((r.m - top) * c);  // r.l is 0 while r.m is -inf
    r.m = top;
  }
  if (r.m == -INFINITY) {  // nothing above -inf so far
#pragma unroll
    for (int i = 0; i < N; ++i) r.l += f[i] == f[i] ? 0.f : NAN;
  } else if constexpr (N % 4 == 0) {
    const F2 minus = pair(-r.m, -r.m), cc = pair(c, c);
    F2 sum = 0;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 x = split(mul2(add2(pair(f[i], f[i + 1]), minus), cc));
      sum = add2(sum, pair(fastExp2(x.x), fastExp2(x.y)));
    }
    const float2 s = split(sum);
    r.l += s.x + s.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r.l += fastExp2((f[i] - r.m) * c);
  }
}

// T threads a block: a compile-time stride saves the long loops their address arithmetic (162 us against 174 at
// 4096 x 131072 bf16).
template <int DT, int T>
__global__ void __launch_bounds__(T, 4 * kThreads / T) distillForward(const __grid_constant__ DistillArgs a) {
  using S = typename Ty<DT>::S;
  constexpr int E = floatTypeSize(DT), V = 16 / E, U = kUnroll;
  __shared__ float top[32];
  __shared__ float2 red[32];
  __shared__ Running part[32];
  __shared__ Running mine;
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned parts = cluster.num_blocks(), rank = cluster.block_rank();
  const size_t row = blockIdx.x / parts;
  const int lane = threadIdx.x & 31;
  constexpr int warps = T / 32;
  const S* logits = reinterpret_cast<const S*>(a.logits) + row * a.ldl;
  // [head | whole 16-byte vectors | tail] of the row; the vectors are dealt to the blocks in runs
  const size_t head = min(a.vocab, ((16 - (uintptr_t)logits % 16) % 16) / E);
  const size_t nvec = (a.vocab - head) / V, tail = head + nvec * V;
  const size_t per = (nvec + parts - 1) / parts;
  const size_t lo = min(nvec, per * rank), hi = min(nvec, lo + per);
  const uint4* vec = reinterpret_cast<const uint4*>(logits + head);
  const float c = a.invT * kLog2e;
  size_t i = lo + threadIdx.x;
  // every block of a cluster loads the entries: whether there are any decides if the row is read; until that is known its
  // first vectors come into L2
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (threadIdx.x % 8 == 0 && i + (size_t)u * T < hi)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(vec + i + (size_t)u * T));
  // (kept in shared memory over the long loop, which needs the registers: 162 us against 167 at 4096 x 131072)
  __shared__ Entries kept[T];
  bool any;
  {
    Entries en;
    any = loadEntries<DT>(a, row, en);
    kept[threadIdx.x] = en;
  }
  if (!__syncthreads_or(any)) {
    if (rank == 0 && threadIdx.x == 0) {
      a.loss[row] = 0.f;
      if (a.stats) a.stats[row] = make_float2(0.f, 0.f);
    }
    return;  // the whole cluster takes this way
  }
  Running r = {-INFINITY, 0.f};
  for (; i + (size_t)(U - 1) * T < hi; i += (size_t)U * T) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = __ldcs(vec + i + (size_t)u * T);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[V];
      Vec16<DT>::expand(v[u], f);
      runOver<V>(r, f, c);
    }
  }
  for (; i < hi; i += T) {
    float f[V];
    Vec16<DT>::expand(__ldcs(vec + i), f);
    runOver<V>(r, f, c);
  }
  if (rank == 0 && threadIdx.x < head + (a.vocab - tail)) {
    float f[1] = {Ty<DT>::toF(logits[threadIdx.x < head ? threadIdx.x : threadIdx.x - head + tail])};
    runOver<1>(r, f, c);
  }
  r = warpJoin(r, a.invT);
  const Entries en = kept[threadIdx.x];
  const float ownMax = warpMax(ownTop(en));
  if (lane == 0) {
    part[threadIdx.x >> 5] = r;
    top[threadIdx.x >> 5] = ownMax;
  }
  __syncthreads();
  if (parts > 1) {
    if (threadIdx.x < 32) {
      r = warpJoin(lane < warps ? part[lane] : Running{-INFINITY, 0.f}, a.invT);
      if (lane == 0) mine = r;
    }
    cluster.sync();
    if (rank == 0 && threadIdx.x < 32) {
      Running o = {-INFINITY, 0.f};
      if (lane < (int)parts) o = *cluster.map_shared_rank(&mine, lane);
      part[lane] = o;
    }
    cluster.sync();
    if (rank != 0) return;
  }
  r = warpJoin(lane < (parts > 1 ? (int)parts : warps) ? part[lane] : Running{-INFINITY, 0.f}, a.invT);
  const float m = r.m, ll = logf(r.l);
  // With e_j = exp((t_j - top) / T) and sum e = Z, p_j = e_j / Z and sum p = 1:
  //   sum p (log p - log q) = sum e_j ((t_j - top) / T - (s_j - m) / T) / Z - log Z + ll
  const float teacherTop = warpMax(lane < warps ? top[lane] : -INFINITY);
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kOwnEntries; ++i) {
    if (en.at[i] < 0) continue;
    const float d = (en.t[i] - teacherTop) * a.invT, e = expf(d);
    sum.x += e;
    if (e != 0.f) sum.y += e * (d - (en.s[i] - m) * a.invT);
  }
  sum = blockSum2(sum, red);
  if (threadIdx.x == 0) {
    a.loss[row] = (sum.y / sum.x - logf(sum.x) + ll) * a.temperature * a.temperature;
    if (a.stats) a.stats[row] = make_float2(m, ll);
  }
}

template <int DT, int T>
__global__ void __launch_bounds__(T, 2 * kThreads / T) distillBackward(const __grid_constant__ DistillArgs a) {
  using S = typename Ty<DT>::S;
  constexpr int E = floatTypeSize(DT), V = 16 / E, U = kUnroll;
  __shared__ float top[32];
  __shared__ float red[32];
  __shared__ __align__(16) int at[VRCCL_DISTILL_MAX_K];
  __shared__ __align__(16) float prob[VRCCL_DISTILL_MAX_K];
  const size_t slices = (a.vocab + a.slice - 1) / a.slice;
  const size_t row = blockIdx.x / slices, part = blockIdx.x % slices;
  const int lane = threadIdx.x & 31;
  constexpr int warps = T / 32;
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
  const float scale = a.dloss[row * a.dstride] * a.temperature;
  Entries en;
  const bool any = loadEntries<DT>(a, row, en);
  const float ownMax = warpMax(ownTop(en));
  if (lane == 0) top[threadIdx.x >> 5] = ownMax;
  // (in place: from here on the entries' logits may be overwritten)
  if (!__syncthreads_or(any)) {
    for (; i < nvec; i += T) __stcs(dst + i, make_uint4(0, 0, 0, 0));
    if (threadIdx.x < edge) out[threadIdx.x] = S(0);
    if (tail + threadIdx.x < end) out[tail + threadIdx.x] = S(0);
    return;
  }
  // q_v dloss T = exp2((s - max) c - shift) scale
  const float c = a.invT * kLog2e, shift = st.y * kLog2e;
  auto dense = [&](float s) { return fastExp2(fmaf(s - st.x, c, -shift)) * scale; };
  const F2 minus2 = pair(-st.x, -st.x), c2 = pair(c, c), shift2 = pair(-shift, -shift), scale2 = pair(scale, scale);
  auto dense2 = [&](float& a, float& b) {
    const float2 x = split(fma2(add2(pair(a, b), minus2), c2, shift2));
    const float2 y = split(mul2(pair(fastExp2(x.x), fastExp2(x.y)), scale2));
    a = y.x;
    b = y.y;
  };
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
          for (int e = 0; e < V; e += 2) dense2(f[e], f[e + 1]);
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
      for (int e = 0; e < V; ++e) f[e] = dense(Ty<DT>::toF(logits[first + i * V + e]));
      __stcs(dst + i, Vec16<DT>::pack(f));
    }
  }
  if (threadIdx.x < edge) out[threadIdx.x] = Ty<DT>::fromF(dense(Ty<DT>::toF(logits[threadIdx.x])));
  if (tail + threadIdx.x < end) out[tail + threadIdx.x] = Ty<DT>::fromF(dense(Ty<DT>::toF(logits[tail + threadIdx.x])));
  // the teacher's entries
  const float teacherTop = warpMax(lane < warps ? top[lane] : -INFINITY);
  float e[kOwnEntries], sum = 0.f;
#pragma unroll
  for (int i = 0; i < kOwnEntries; ++i) {
    e[i] = en.at[i] < 0 ? 0.f : expf((en.t[i] - teacherTop) * a.invT);
    sum += e[i];
  }
  const float inv = 1.f / blockSum(sum, red);
  const int padded = (a.k + 3) / 4 * 4;
#pragma unroll
  for (int i = 0; i < kOwnEntries; ++i) {
    const int j = threadIdx.x + i * T;
    if (j < padded) {
      at[j] = en.at[i];
      prob[j] = e[i] * inv;
    }
  }
  __syncthreads();  // also: every element of the slice is written
  // Entries that share an index all write the same sum. They are looked for where there can be any: up to 64 entries
  // always, more only if a hash table of the indices says that some are met twice.
  bool shared = true;
  if (a.k > 64) {
    __shared__ int seen[kSeen];
    for (int j = threadIdx.x; j < kSeen; j += T) seen[j] = -1;
    __syncthreads();
    bool twice = false;
#pragma unroll
    for (int i = 0; i < kOwnEntries; ++i) {
      if (en.at[i] < 0) continue;
      for (unsigned h = (unsigned)en.at[i] * 2654435761u >> 21;; h = (h + 1) % kSeen) {
        const int met = atomicCAS(&seen[h], -1, en.at[i]);
        twice |= met == en.at[i];
        if (met == -1 || met == en.at[i]) break;
      }
    }
    shared = __syncthreads_or(twice);
  }
#pragma unroll
  for (int i = 0; i < kOwnEntries; ++i) {
    const int own = en.at[i];
    if (own < 0 || (size_t)own < begin || (size_t)own >= end) continue;
    float p = shared ? 0.f : e[i] * inv;
    for (int j = 0; shared && j < padded; j += 4) {
      const int4 q = *reinterpret_cast<const int4*>(at + j);
      if (q.x == own) p += prob[j];
      if (q.y == own) p += prob[j + 1];
      if (q.z == own) p += prob[j + 2];
      if (q.w == own) p += prob[j + 3];
    }
    out[own] = Ty<DT>::fromF((expf((en.s[i] - st.x) * a.invT - st.y) - p) * scale);
  }
}

// Threads of a block: with a row in 16 vectors a thread or fewer, so that several short rows share a multiprocessor and
// one's reductions run under another's loads; more where blocks are few; and enough for the row's entries.
int blockThreads(size_t bytes, size_t blocks, size_t k) {
  int t = 128;
  const size_t most = blocks < (size_t)smCount() * 2 ? 64 : 256;  // bytes a thread
  while (t < kThreads && (bytes > t * most || k > (size_t)t * kOwnEntries)) t *= 2;
  return t;
}

using DistillFn = void (*)(DistillArgs);
template <int DT>
DistillFn pickForward(int threads) {
  return threads == 128 ? distillForward<DT, 128> : threads == 256 ? distillForward<DT, 256> : distillForward<DT, 512>;
}
template <int DT>
DistillFn pickBackward(int threads) {
  return threads == 128 ? distillBackward<DT, 128> : threads == 256 ? distillBackward<DT, 256> : distillBackward<DT, 512>;
}

bool goodDistill(const void* logits, size_t ldl, const void* teacher, size_t ldt, const void* index, size_t ldi,
                 size_t rows, size_t vocab, size_t k, int dtype, int ttype, int itype) {
  const int is = itype == vrcclInt64 ? 8 : 4;
  return goodMatrix(logits, ldl, rows, vocab, floatTypeSize(dtype)) && goodMatrix(teacher, ldt, rows, k, floatTypeSize(ttype)) &&
         goodMatrix(index, ldi, rows, k, is);
}
bool goodTypes(size_t rows, size_t vocab, size_t k, int dtype, int ttype, int itype, float temperature) {
  return rows < (size_t(1) << 31) && vocab < (size_t(1) << 31) && k <= VRCCL_DISTILL_MAX_K && isOperatorType(dtype) &&
         isOperatorType(ttype) && (itype == vrcclInt32 || itype == vrcclInt64) && temperature >= 1e-18f &&
         temperature <= 1e18f;  // its square and its reciprocal are then normal numbers
}
DistillArgs distillArgs(const void* logits, size_t ldl, const void* teacher, size_t ldt, const void* index, size_t ldi,
                        size_t rows, size_t vocab, size_t k, int ttype, int itype, float temperature) {
  DistillArgs a = {};
  a.logits = logits;
  a.teacher = teacher;
  a.index = index;
  a.ldl = ldl;
  a.ldt = ldt;
  a.ldi = ldi;
  a.rows = rows;
  a.vocab = vocab;
  a.k = (int)k;
  a.ttype = ttype;
  a.wide = itype == vrcclInt64;
  a.temperature = temperature;
  a.invT = 1.f / temperature;
  return a;
}

}  // namespace
}  // namespace vrccl

using namespace vrccl;

extern "C" vrcclResult_t vrcclDistillForward(const void* logits, size_t ldl, const void* teacher, size_t ldt,
                                             const void* index, size_t ldi, float* loss, float* stats, size_t rows,
                                             size_t vocab, size_t k, vrcclDataType_t dtype, vrcclDataType_t teacherType,
                                             vrcclDataType_t indexType, float temperature, vrcclStream_t stream) {
  if (!goodTypes(rows, vocab, k, dtype, teacherType, indexType, temperature)) return vrcclInvalidArgument;
  if (rows == 0) return vrcclSuccess;
  cudaStream_t st = (cudaStream_t)stream;
  if (!goodVector(loss, 4) || (stats && !goodVector(stats, 8))) return vrcclInvalidArgument;
  if (vocab == 0 || k == 0) {  // no row has an entry
    if (cudaMemsetAsync(loss, 0, rows * 4, st) != cudaSuccess ||
        (stats && cudaMemsetAsync(stats, 0, rows * 8, st) != cudaSuccess)) {
      cudaGetLastError();
      return vrcclCudaError;
    }
    return vrcclSuccess;
  }
  if (!goodDistill(logits, ldl, teacher, ldt, index, ldi, rows, vocab, k, dtype, teacherType, indexType))
    return vrcclInvalidArgument;
  const Span out[] = {vectorSpan(loss, rows * 4), vectorSpan(stats, rows * 8)};
  const Span in[] = {matrixSpan(logits, ldl, rows, vocab, floatTypeSize(dtype)),
                     matrixSpan(teacher, ldt, rows, k, floatTypeSize(teacherType)),
                     matrixSpan(index, ldi, rows, k, indexType == vrcclInt64 ? 8 : 4)};
  if (!apart(out, in)) return vrcclInvalidArgument;
  DistillArgs a = distillArgs(logits, ldl, teacher, ldt, index, ldi, rows, vocab, k, teacherType, indexType, temperature);
  a.loss = loss;
  a.stats = reinterpret_cast<float2*>(stats);
  // split a row over a cluster until the grid fills the GPU or a block has less than two vectors a thread
  unsigned parts = 1;
  const size_t bytes = vocab * floatTypeSize(dtype);
  while (parts < 8 && rows * parts * 2 <= (size_t)smCount() * 2 && bytes / (parts * 2) >= size_t(kThreads) * 32) parts *= 2;
  const int threads = blockThreads(bytes / parts, rows * parts, k);
  const DistillFn fn = dtype == vrcclFloat32    ? pickForward<vrcclFloat32>(threads)
                       : dtype == vrcclBfloat16 ? pickForward<vrcclBfloat16>(threads)
                                                : pickForward<vrcclFloat16>(threads);
  return launchShaped(fn, {dim3((unsigned)(rows * parts)), threads, 0, (int)parts, false}, st, a);
}

extern "C" vrcclResult_t vrcclDistillBackward(const void* logits, size_t ldl, const void* teacher, size_t ldt,
                                              const void* index, size_t ldi, const float* stats, const float* dloss,
                                              size_t dlossStride, void* dlogits, size_t ldd, size_t rows, size_t vocab,
                                              size_t k, vrcclDataType_t dtype, vrcclDataType_t teacherType,
                                              vrcclDataType_t indexType, float temperature, vrcclStream_t stream) {
  if (!goodTypes(rows, vocab, k, dtype, teacherType, indexType, temperature)) return vrcclInvalidArgument;
  if (rows == 0 || vocab == 0) return vrcclSuccess;
  const int E = floatTypeSize(dtype);
  cudaStream_t st = (cudaStream_t)stream;
  if (!goodMatrix(dlogits, ldd, rows, vocab, E)) return vrcclInvalidArgument;
  if (k == 0) {  // no row has an entry
    if (cudaMemset2DAsync(dlogits, ldd * E, 0, vocab * E, rows, st) != cudaSuccess) {
      cudaGetLastError();
      return vrcclCudaError;
    }
    return vrcclSuccess;
  }
  if (!goodDistill(logits, ldl, teacher, ldt, index, ldi, rows, vocab, k, dtype, teacherType, indexType) ||
      !goodVector(stats, 8) || !goodVector(dloss, 4) || dlossStride >= kMaxExtent)
    return vrcclInvalidArgument;
  if (rows - 1 > (size_t(1) << 46) / std::max<size_t>(1, dlossStride)) return vrcclInvalidArgument;
  const Span out[] = {matrixSpan(dlogits, ldd, rows, vocab, E)};
  const Span in[] = {unlessInPlace(matrixSpan(logits, ldl, rows, vocab, E), ldl, dlogits, ldd),
                     matrixSpan(teacher, ldt, rows, k, floatTypeSize(teacherType)),
                     matrixSpan(index, ldi, rows, k, indexType == vrcclInt64 ? 8 : 4),
                     vectorSpan(stats, rows * 8),
                     matrixSpan(dloss, dlossStride, rows, 1, 4)};
  if (!apart(out, in)) return vrcclInvalidArgument;
  DistillArgs a = distillArgs(logits, ldl, teacher, ldt, index, ldi, rows, vocab, k, teacherType, indexType, temperature);
  a.stats = const_cast<float2*>(reinterpret_cast<const float2*>(stats));
  a.dloss = dloss;
  a.dstride = dlossStride;
  a.dlogits = dlogits;
  a.ldd = ldd;
  // In place a row stays with one block: another slice's entries could be overwritten before they are read.
  const size_t unit = size_t(kThreads) * (16 / E);
  size_t pieces = 1;
  if (dlogits != logits)  // even pieces, until there are four blocks a multiprocessor or a piece has 32 KB
    pieces = std::max<size_t>(1, std::min((size_t)smCount() * 4 / rows, vocab * E / 32768));
  a.slice = std::min(vocab, ((vocab + pieces - 1) / pieces + unit - 1) / unit * unit);
  const size_t slices = (vocab + a.slice - 1) / a.slice;
  if (rows * slices >= (size_t(1) << 31)) return vrcclInvalidArgument;
  // As many blocks as four a multiprocessor are all at work at once with 256 threads each (301 x 50001 fp32: 19.6 us; with
  // 512, two rounds of them, 23.2); more do better with 512 (3000 x 50001: 190 against 198).
  const int threads = rows * slices <= (size_t)smCount() * 4 && k <= 256 * kOwnEntries ? 256 : blockThreads(a.slice * E, rows * slices, k);
  const DistillFn fn = dtype == vrcclFloat32    ? pickBackward<vrcclFloat32>(threads)
                       : dtype == vrcclBfloat16 ? pickBackward<vrcclBfloat16>(threads)
                                                : pickBackward<vrcclFloat16>(threads);
  return launchShaped(fn, {dim3((unsigned)(rows * slices)), threads, 0, 0, false}, st, a);
}

// Distillation from a teacher's top logits, forward and backward.
//
// A row holds the student's logits s over the whole vocabulary and the
// teacher's logits t at k of its entries. With temperature T, over the kept
// entries j (index inside the vocabulary, t_j above -inf):
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
// hold, and they are not read.
//
// Both directions are bound by memory: forward reads the logits once (each
// thread keeps a running maximum and a sum rescaled when the maximum grows,
// joined at the end), backward reads them and writes the gradient. Where there
// are fewer rows than multiprocessors a row is split: forward over the blocks
// of a cluster, which join their (max, sum) through distributed shared memory;
// backward over independent blocks, since the saved statistics are all an
// element needs.
#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace vrccl {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;

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

// The row's kept teacher entries in shared memory.
struct Entries {
  float p[VRCCL_DISTILL_MAX_K];     // p_j, 0 where not kept
  float logp[VRCCL_DISTILL_MAX_K];
  float s[VRCCL_DISTILL_MAX_K];     // the student's logit there
  int at[VRCCL_DISTILL_MAX_K];      // the entry's index, -1 where not kept
};

__device__ __forceinline__ float warpMax(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float blockMax(float x, float* s) {
  x = warpMax(x);
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  return warpMax(lane < warps ? s[lane] : -INFINITY);
}

// Loads the entries and forms the teacher's distribution; false (in every
// thread) where none is kept. Entry j belongs to thread j mod blockDim.
template <int DT>
__device__ __forceinline__ bool loadEntries(const DistillArgs& a, size_t row, Entries& en, float* r0, float* r1) {
  constexpr int E = floatTypeSize(DT);
  const char* logits = static_cast<const char*>(a.logits) + row * a.ldl * E;
  const int te = a.ttype == vrcclFloat32 ? 4 : 2;
  const char* teacher = static_cast<const char*>(a.teacher) + row * a.ldt * te;
  float top = -INFINITY;
  bool any = false, nan = false;
  for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
    const long long at = a.wide ? static_cast<const long long*>(a.index)[row * a.ldi + j]
                                : static_cast<const int*>(a.index)[row * a.ldi + j];
    const float t = loadParam(teacher, a.ttype, j);
    const bool in = at >= 0 && (unsigned long long)at < a.vocab;
    const bool kept = in && t != -INFINITY;  // a NaN is kept, and shows
    en.at[j] = kept ? (int)at : -1;
    en.logp[j] = t;
    en.s[j] = kept ? loadOne<DT>(logits, at) : 0.f;
    if (kept) {
      any = true;
      nan |= t != t;
      top = fmaxf(top, t);
    }
  }
  top = blockMax(top, r0);
  if (!__syncthreads_or(any)) return false;
  float sum = 0.f;
  for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
    if (en.at[j] < 0) continue;
    const float d = (en.logp[j] - top) * a.invT;
    en.logp[j] = d;
    sum += expf(d);
  }
  if (nan) sum = NAN;
  sum = blockSum(sum, r1);
  const float ls = logf(sum);
  for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
    if (en.at[j] < 0) {
      en.p[j] = 0.f;
      continue;
    }
    en.logp[j] -= ls;
    en.p[j] = expf(en.logp[j]);
  }
  return true;
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

// exp for the long sums: 2^(x log2 e) on the special function unit, relative
// error below 2^-21 for the arguments that matter (x <= 0); the statistics it
// feeds are sums of many terms whose errors average out.
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
  if (r.m != -INFINITY) {
#pragma unroll
    for (int i = 0; i < N; ++i) r.l += fastExp2((f[i] - r.m) * c);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r.l += f[i] == f[i] ? 0.f : NAN;
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) distillForward(const __grid_constant__ DistillArgs a) {
  using S = typename Ty<DT>::S;
  constexpr int E = floatTypeSize(DT), V = 16 / E, U = 4;
  __shared__ Entries en;
  __shared__ float red[2][32];
  __shared__ Running part[32];
  __shared__ Running mine;
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned parts = cluster.num_blocks(), rank = cluster.block_rank();
  const size_t row = blockIdx.x / parts;
  const S* logits = reinterpret_cast<const S*>(a.logits) + row * a.ldl;
  // every block of a cluster loads the entries: whether there are any decides
  // if the row is read at all
  if (!loadEntries<DT>(a, row, en, red[0], red[1])) {
    if (rank == 0 && threadIdx.x == 0) {
      a.loss[row] = 0.f;
      if (a.stats) a.stats[row] = make_float2(0.f, 0.f);
    }
    return;  // the whole cluster takes this way
  }
  // [head | whole 16-byte vectors | tail] of the row; the vectors are dealt to the blocks in runs
  const size_t head = min(a.vocab, ((16 - (uintptr_t)logits % 16) % 16) / E);
  const size_t nvec = (a.vocab - head) / V, tail = head + nvec * V;
  const size_t per = (nvec + parts - 1) / parts;
  const size_t lo = min(nvec, per * rank), hi = min(nvec, lo + per);
  const uint4* vec = reinterpret_cast<const uint4*>(logits + head);
  const float c = a.invT * kLog2e;
  Running r = {-INFINITY, 0.f};
  size_t i = lo + threadIdx.x;
  for (; i + (U - 1) * kThreads < hi; i += U * kThreads) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = __ldcs(vec + i + u * kThreads);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[V];
      Vec16<DT>::expand(v[u], f);
      runOver<V>(r, f, c);
    }
  }
  for (; i < hi; i += kThreads) {
    float f[V];
    Vec16<DT>::expand(__ldcs(vec + i), f);
    runOver<V>(r, f, c);
  }
  if (rank == 0) {
    const size_t extra = threadIdx.x < head ? threadIdx.x : threadIdx.x - head + tail;
    if (threadIdx.x < head + (a.vocab - tail)) {
      float f[1] = {Ty<DT>::toF(logits[extra])};
      runOver<1>(r, f, c);
    }
  }
  r = warpJoin(r, a.invT);
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.x >> 5] = r;
  __syncthreads();
  if (threadIdx.x < 32) {
    r = warpJoin(lane < kThreads / 32 ? part[lane] : Running{-INFINITY, 0.f}, a.invT);
    if (lane == 0) mine = r;
  }
  if (parts > 1) {
    cluster.sync();
    if (rank == 0 && threadIdx.x < 32) {
      Running o = {-INFINITY, 0.f};
      if (lane < (int)parts) o = *cluster.map_shared_rank(&mine, lane);
      r = warpJoin(o, a.invT);
      if (lane == 0) mine = r;
    }
    cluster.sync();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }
  const float m = mine.m, ll = logf(mine.l);
  float loss = 0.f;
  for (int j = threadIdx.x; j < a.k; j += kThreads) {
    const float p = en.p[j];
    if (p != 0.f) loss += p * (en.logp[j] - ((en.s[j] - m) * a.invT - ll));
  }
  loss = blockSum(loss, red[0]);
  if (threadIdx.x == 0) {
    a.loss[row] = loss * a.temperature * a.temperature;
    if (a.stats) a.stats[row] = make_float2(m, ll);
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) distillBackward(const __grid_constant__ DistillArgs a) {
  using S = typename Ty<DT>::S;
  constexpr int E = floatTypeSize(DT), V = 16 / E, U = 4;
  __shared__ Entries en;
  __shared__ float red[2][32];
  const size_t slices = (a.vocab + a.slice - 1) / a.slice;
  const size_t row = blockIdx.x / slices, part = blockIdx.x % slices;
  const S* logits = reinterpret_cast<const S*>(a.logits) + row * a.ldl;
  S* out = reinterpret_cast<S*>(a.dlogits) + row * a.ldd;
  const size_t from = part * a.slice, to = min(a.vocab, from + a.slice);
  const bool some = loadEntries<DT>(a, row, en, red[0], red[1]);
  // slices are whole vectors of the output counted from its row's first boundary, where the logits share it
  const size_t head = min(a.vocab, ((16 - (uintptr_t)out % 16) % 16) / E);
  const bool together = ((uintptr_t)logits - (uintptr_t)out) % 16 == 0;
  const size_t begin = part == 0 ? 0 : min(a.vocab, from + head);
  const size_t end = to == a.vocab ? a.vocab : min(a.vocab, to + head);
  const float2 st = some ? a.stats[row] : make_float2(0.f, 0.f);
  const float scale = some ? a.dloss[row * a.dstride] * a.temperature : 0.f;
  const float c = a.invT * kLog2e, shift = st.y * kLog2e;
  // q_v scale = exp2((s - max) c - shift) scale
  const size_t first = part == 0 ? head : begin;  // the first vector's element
  const size_t nvec = end > first ? (end - first) / V : 0, tail = first + nvec * V;
  uint4* dst = reinterpret_cast<uint4*>(out + first);
  if (!some) {
    for (size_t i = threadIdx.x; i < nvec; i += kThreads) __stcs(dst + i, make_uint4(0, 0, 0, 0));
    const size_t edge = (part == 0 ? min(head, end) : 0);
    if (threadIdx.x < edge) out[threadIdx.x] = S(0);
    if (tail + threadIdx.x < end) out[tail + threadIdx.x] = S(0);
    return;
  }
  __syncthreads();  // the entries' logits are read (in place: before they are overwritten)
  size_t i = threadIdx.x;
  if (together) {
    const uint4* src = reinterpret_cast<const uint4*>(logits + first);
    for (; i + (U - 1) * kThreads < nvec; i += U * kThreads) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = __ldcs(src + i + u * kThreads);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[V];
        Vec16<DT>::expand(v[u], f);
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = fastExp2((f[e] - st.x) * c - shift) * scale;
        __stcs(dst + i + u * kThreads, Vec16<DT>::pack(f));
      }
    }
  }
  for (; i < nvec; i += kThreads) {
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = fastExp2((Ty<DT>::toF(logits[first + i * V + e]) - st.x) * c - shift) * scale;
    __stcs(dst + i, Vec16<DT>::pack(f));
  }
  const size_t edge = part == 0 ? min(head, end) : 0;
  if (threadIdx.x < edge)
    out[threadIdx.x] = Ty<DT>::fromF(fastExp2((Ty<DT>::toF(logits[threadIdx.x]) - st.x) * c - shift) * scale);
  if (tail + threadIdx.x < end)
    out[tail + threadIdx.x] =
        Ty<DT>::fromF(fastExp2((Ty<DT>::toF(logits[tail + threadIdx.x]) - st.x) * c - shift) * scale);
  __syncthreads();
  // the teacher's entries of this slice; entries that share an index all write the same sum
  for (int j = threadIdx.x; j < a.k; j += kThreads) {
    const int at = en.at[j];
    if (at < 0 || (size_t)at < begin || (size_t)at >= end) continue;
    float p = 0.f;
    for (int i = 0; i < a.k; ++i)
      if (en.at[i] == at) p += en.p[i];
    out[at] = Ty<DT>::fromF((expf((en.s[j] - st.x) * a.invT - st.y) - p) * scale);
  }
}

bool goodDistill(const void* logits, size_t ldl, const void* teacher, size_t ldt, const void* index, size_t ldi,
                 size_t rows, size_t vocab, size_t k, int dtype, int ttype, int itype) {
  const int is = itype == vrcclInt64 ? 8 : 4;
  return goodMatrix(logits, ldl, vocab, floatTypeSize(dtype)) && goodMatrix(teacher, ldt, k, floatTypeSize(ttype)) &&
         goodMatrix(index, ldi, k, is);
}
bool goodTypes(size_t rows, size_t vocab, size_t k, int dtype, int ttype, int itype, float temperature) {
  return rows < (size_t(1) << 31) && vocab < (size_t(1) << 31) && k <= VRCCL_DISTILL_MAX_K && isOperatorType(dtype) &&
         isOperatorType(ttype) && (itype == vrcclInt32 || itype == vrcclInt64) && temperature > 0.f &&
         temperature <= 3.0e38f && 1.f / temperature <= 3.0e38f;
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
  DistillArgs a = distillArgs(logits, ldl, teacher, ldt, index, ldi, rows, vocab, k, teacherType, indexType, temperature);
  a.loss = loss;
  a.stats = reinterpret_cast<float2*>(stats);
  // split a row over a cluster until the grid fills the GPU or a block has less than two vectors a thread
  unsigned parts = 1;
  const size_t bytes = vocab * floatTypeSize(dtype);
  while (parts < 8 && rows * parts * 2 <= (size_t)smCount() * 2 && bytes / (parts * 2) >= size_t(kThreads) * 32) parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto fn = dtype == vrcclFloat32    ? distillForward<vrcclFloat32>
            : dtype == vrcclBfloat16 ? distillForward<vrcclBfloat16>
                                     : distillForward<vrcclFloat16>;
  if (cudaLaunchKernelEx(&cfg, fn, a) != cudaSuccess) {
    cudaGetLastError();
    return vrcclCudaError;
  }
  return vrcclSuccess;
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
  if (!goodMatrix(dlogits, ldd, vocab, E)) return vrcclInvalidArgument;
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
  if (!(dlogits == logits && ldd == ldl) &&
      overlap(dlogits, spanBytes(ldd, rows, vocab, E), logits, spanBytes(ldl, rows, vocab, E)))
    return vrcclInvalidArgument;
  DistillArgs a = distillArgs(logits, ldl, teacher, ldt, index, ldi, rows, vocab, k, teacherType, indexType, temperature);
  a.stats = const_cast<float2*>(reinterpret_cast<const float2*>(stats));
  a.dloss = dloss;
  a.dstride = dlossStride;
  a.dlogits = dlogits;
  a.ldd = ldd;
  // In place a row stays with one block: another slice's entries could be overwritten before they are read.
  a.slice = vocab;
  if (dlogits != logits) {
    const size_t unit = size_t(kThreads) * 4 * (16 / E);
    const size_t want = std::max<size_t>(1, (size_t)smCount() * 4 / rows);
    a.slice = std::min(vocab, (vocab / want + unit) / unit * unit);
  }
  const size_t slices = (vocab + a.slice - 1) / a.slice;
  if (rows * slices >= (size_t(1) << 31)) return vrcclInvalidArgument;
  auto fn = dtype == vrcclFloat32    ? distillBackward<vrcclFloat32>
            : dtype == vrcclBfloat16 ? distillBackward<vrcclBfloat16>
                                     : distillBackward<vrcclFloat16>;
  fn<<<(unsigned)(rows * slices), kThreads, 0, st>>>(a);
  return launchResult();
}

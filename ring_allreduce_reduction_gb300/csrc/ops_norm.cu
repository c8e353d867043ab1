// Layer norm over the columns of a [rows, cols] matrix, forward and backward.
//
//   xh = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   y  = xh gamma + beta
//   g  = dy gamma
//   dx = rstd (g - mean(g) - xh mean(g xh))
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Both directions are bound by memory: forward reads x and writes y, backward
// reads dy and x and writes dx. A row is read once; its sums are formed from
// registers, so that the mean is known before the squares are taken:
// sum((x - mean)^2) loses nothing to cancellation where sum(x^2) - mean^2
// would. Where several warps share a row each takes its elements' squares about
// its own mean, and these are joined about the row's with one barrier. All sums
// are binary32.
//
// The weight's gradient is a sum down the columns. A thread owns the same
// columns in every row that its block walks and keeps the two sums in
// registers; a block writes them once, as one row of a [blocks, 2, cols]
// workspace, and a second kernel adds those rows in order. No atomics: the
// same call gives the same bits.
//
// By row length: several rows a warp (narrow), several teams of warps a block
// (to 8192 columns), a block a row (to 16384), passes through L2 beyond. What
// they measured, of a copy's 6.7 TB/s: bf16 forward 32768 x 4096 84 us (6.4
// TB/s), 2 M x 64 89 us (6.0), 8192 x 16384 96 us (5.6); backward
// 16384 x 8192 139 us (5.8, the joining of 152 blocks' sums among them),
// 8192 x 16384 165 us (4.9). Rows on no 16-byte boundary pay for one-element
// accesses: 5003 x 1001 fp16 backward 19 us, 19157 x 3503 bf16 forward 85 us
// (3.1 TB/s), bound by issue slots.
#include <mutex>

#include "ops_ring.cuh"

namespace vrccl {
namespace {

struct NormArgs {
  const void* x;
  const void* dy;
  const void* gamma;
  const void* beta;
  void* y;  // forward: y, backward: dx
  float* mean;
  float* rstd;
  float* partial;  // [blocks][2][cols], NULL: no weight gradient
  size_t ldx, lddy, ldy, rows;
  int cols;
  int ptype;
  bool wideParams;  // gamma and beta start on 16-byte boundaries
  int stages, teams;
  unsigned cutX, cutDy;  // cutRows of x and dy
  float eps;
};

constexpr int kMaxHeldCols = 32768;  // 1024 threads x 32 elements; longer rows are re-read (through L2)

// NV accesses of V elements each: element e of access j of thread t is column
// (j T + t) V + e. V is a whole 16-byte vector where every row of every
// operand starts on a 16-byte boundary and cols is a multiple of V, else 1.
template <int DT, bool VEC, int EPT>
struct Held {
  static constexpr int V = VEC ? 16 / floatTypeSize(DT) : 1;
  static constexpr int NV = EPT / V;
  using S = typename Ty<DT>::S;
  using Raw = std::conditional_t<VEC, uint4, S>;
  Raw raw[NV];

  __device__ __forceinline__ void load(const void* row, int t, int T, int cols) {
    const Raw* p = reinterpret_cast<const Raw*>(row);
    const int n = cols / V;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = j * T + t;
      if (i < n)
        raw[j] = __ldcs(p + i);
      else
        raw[j] = Raw{};
    }
  }
  __device__ __forceinline__ void get(int j, float (&f)[V]) const {
    if constexpr (VEC)
      Vec16<DT>::expand(raw[j], f);
    else
      f[0] = Ty<DT>::toF(raw[j]);
  }
  static __device__ __forceinline__ void put(void* row, int i, const float (&f)[V]) {
    if constexpr (VEC)
      __stcs(reinterpret_cast<uint4*>(row) + i, Vec16<DT>::pack(f));
    else
      reinterpret_cast<S*>(row)[i] = Ty<DT>::fromF(f[0]);
  }
};

// ------------------------------------------------------------ teams
// Rows of up to 8192 elements. A block of up to 512 threads is cut into teams
// of a few warps, 16 elements of a row a thread; every team walks rows of its
// own with the grid's stride and keeps its columns' parameters in registers.
// Rows arrive in shared memory by bulk copies, several rows ahead, so the
// copies run under the sums and the stores; the barrier inside a row's
// reduction is also the point where every thread has taken its elements out of
// the stage, and the team's first thread refills it.
constexpr int kTeamElems = 16;
constexpr int kTeamCols = 512 * kTeamElems;
constexpr int kTeamSmem = 192 * 1024, kWideSmem = 224 * 1024;  // of the 227 KB a block may have

__host__ __device__ constexpr int slotBytes(int cols, int E) { return ((cols * E + 15) / 16 + 1) * 16; }

// The 16 elements of thread t of a team of T: element q is column
// ((q / V) T + t) V + q % V, V a whole 16-byte vector (VEC) or 1. T is a
// constant: offsets are then part of the instructions (with a T of any multiple
// of 32 an element of a row on no boundary took 120 of them).
template <int DT, bool VEC, int T>
struct Team {
  static constexpr int E = floatTypeSize(DT), V = VEC ? 16 / E : 1, NV = kTeamElems / V;
  using S = typename Ty<DT>::S;

  static __device__ __forceinline__ void fetch(unsigned char* slot, const void* p, size_t ld, size_t row, size_t rows,
                                               int cols, unsigned cut, unsigned long long* bar, unsigned long long policy) {
    if constexpr (VEC) {
      bulkLoadOnce(slot, static_cast<const char*>(p) + row * ld * E, cols * E, bar, policy);
      return;
    }
    const Window w = rowWindow((uintptr_t)p, ld, row, rows, cols, E, cut);
    if (w.hi > w.lo) bulkLoadOnce(slot + (w.lo - (w.row & ~(uintptr_t)15)), (const void*)w.lo, w.hi - w.lo, bar, policy);
  }
  // What a bulk copy may not take of a row (Window), copied by the thread that is about to announce it: its arrival
  // at the row's barrier makes them visible with the rest.
  static __device__ __forceinline__ void edges(unsigned char* slot, const void* p, size_t ld, size_t row, size_t rows,
                                               int cols, unsigned cut) {
    if constexpr (!VEC) {
      if (!maybeCut(row, rows, cut)) return;
      const Window w = rowWindow((uintptr_t)p, ld, row, rows, cols, E, cut);
      S* v = reinterpret_cast<S*>(slot + (w.row & 15));
      for (uintptr_t at = w.row; at < w.headEnd(); at += E) v[(at - w.row) / E] = *(const S*)at;
      for (uintptr_t at = w.tailBegin(); at < w.end; at += E) v[(at - w.row) / E] = *(const S*)at;
      fenceProxyAsync();  // a later row's copy into this slot comes after these writes
    }
  }
  static __device__ __forceinline__ unsigned fetchBytes(const void* p, size_t ld, size_t row, size_t rows, int cols,
                                                    unsigned cut) {
    if constexpr (VEC) return cols * E;
    const Window w = rowWindow((uintptr_t)p, ld, row, rows, cols, E, cut);
    return w.hi - w.lo;
  }
  // Elements FROM .. FROM + N of the thread's 16 (whole vectors).
  template <int FROM, int N>
  static __device__ __forceinline__ void takeSome(const unsigned char* slot, const void* p, size_t ld, size_t row,
                                                  size_t rows, int cols, int t, float (&f)[N]) {
    if constexpr (VEC) {
      const uint4* v = reinterpret_cast<const uint4*>(slot);
#pragma unroll
      for (int j = 0; j < N / V; ++j) {
        const int i = (FROM / V + j) * T + t;
        float g[V];
        Vec16<DT>::expand(i * V < cols ? v[i] : make_uint4(0, 0, 0, 0), g);
#pragma unroll
        for (int e = 0; e < V; ++e) f[j * V + e] = g[e];
      }
    } else {
      const S* v = reinterpret_cast<const S*>(slot + (((unsigned)(uintptr_t)p + (unsigned)row * (unsigned)ld * E) & 15)) + t;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        f[j] = 0.f;
        if ((FROM + j) * T + t < cols) f[j] = Ty<DT>::toF(v[(FROM + j) * T]);
      }
    }
  }
  static __device__ __forceinline__ void take(const unsigned char* slot, const void* p, size_t ld, size_t row,
                                              size_t rows, int cols, int t, float (&f)[kTeamElems]) {
    takeSome<0, kTeamElems>(slot, p, ld, row, rows, cols, t, f);
  }
  static __device__ __forceinline__ void storeSome(void* row, int cols, int t, int from, const float* f, int n) {
#pragma unroll
    for (int j = 0; j < n / V; ++j) {
      const int i = (from / V + j) * T + t;
      if (i * V >= cols) break;
      if constexpr (VEC) {
        float g[V];
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] = f[j * V + e];
        __stcs(reinterpret_cast<uint4*>(row) + i, Vec16<DT>::pack(g));
      } else {
        reinterpret_cast<S*>(row)[i] = Ty<DT>::fromF(f[j]);
      }
    }
  }
  static __device__ __forceinline__ void store(void* row, int cols, int t, const float (&f)[kTeamElems]) {
    storeSome(row, cols, t, 0, f, kTeamElems);
  }
  static __device__ __forceinline__ void params(const void* p, int ptype, bool wide, float dflt, int cols, int t,
                                                float (&f)[kTeamElems]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * T + t) * V;
      float g[V];
#pragma unroll
      for (int e = 0; e < V; ++e) g[e] = 0.f;
      if (c < cols) loadParams<V>(p, ptype, wide, c, dflt, g);
#pragma unroll
      for (int e = 0; e < V; ++e) f[j * V + e] = g[e];
    }
  }
  // The thread's two sums of its columns to p[0 .. cols) and p[cols .. 2 cols).
  static __device__ __forceinline__ void layOut(float* p, const F2 (&dg)[kTeamElems / 2], const F2 (&db)[kTeamElems / 2],
                                                int cols, int t) {
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < kTeamElems; q += 4) {
        if (!held(q, cols, t)) continue;
        float* at = p + (q / V * T + t) * V + q % V;
        const float2 a = split(dg[q / 2]), b = split(dg[q / 2 + 1]), c = split(db[q / 2]), d = split(db[q / 2 + 1]);
        *reinterpret_cast<float4*>(at) = make_float4(a.x, a.y, b.x, b.y);
        *reinterpret_cast<float4*>(at + cols) = make_float4(c.x, c.y, d.x, d.y);
      }
    } else {
#pragma unroll
      for (int q = 0; q < kTeamElems; ++q) {
        if (!held(q, cols, t)) continue;
        const float2 a = split(dg[q / 2]), c = split(db[q / 2]);
        p[q * T + t] = q & 1 ? a.y : a.x;
        p[cols + q * T + t] = q & 1 ? c.y : c.x;
      }
    }
  }
  static __device__ __forceinline__ bool held(int q, int cols, int t) { return (q / V * T + t) * V < cols; }
};

template <int T>
__device__ __forceinline__ void teamSync(int team) {
  if constexpr (T == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(T) : "memory");
}

// Two rows a turn, so that one row's reduction hides the other's latency and
// one shuffle moves both rows' values (lanes 0-15 end up with row 0's sum,
// lanes 16-31 with row 1's).
__device__ __forceinline__ float sumTwo(float a, float b, bool high) {
  float x = (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, 16);
#pragma unroll
  for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float sumHalf(float x) {
#pragma unroll
  for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int DT, bool VEC, int T>
__global__ void __launch_bounds__(512) normForwardTeams(const __grid_constant__ NormArgs a) {
  using M = Team<DT, VEC, T>;
  constexpr int E = M::E, NP = kTeamElems / 2;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ unsigned long long full[16 * kMaxStages];
  __shared__ float2 red[16][2][2][16];  // team, turn, row, warp: (sum, squares about the warp's mean)
  __shared__ int deadWord[16];
  const int team = threadIdx.x / T, t = threadIdx.x % T, lane = t & 31;
  const int cols = a.cols, stages = a.stages, slot = slotBytes(cols, E);
  constexpr int warps = T / 32;
  unsigned char* mine = ring + (size_t)team * stages * slot;
  unsigned long long* bar = full + team * kMaxStages;
  int* dead = &deadWord[team];
  const size_t stride = (size_t)gridDim.x * a.teams, first = (size_t)blockIdx.x * a.teams + team;
  unsigned long long policy = 0;
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbarInit(&bar[s], 1);
    *dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    policy = evictFirstPolicy();
  }
  auto refill = [&](int s, size_t row) {
    if (row >= a.rows) return;
    M::edges(mine + (size_t)s * slot, a.x, a.ldx, row, a.rows, cols, a.cutX);
    expectBytes(&bar[s], M::fetchBytes(a.x, a.ldx, row, a.rows, cols, a.cutX));
    M::fetch(mine + (size_t)s * slot, a.x, a.ldx, row, a.rows, cols, a.cutX, &bar[s], policy);
  };
  if (t == 0)
    for (int s = 0; s < stages; ++s) refill(s, first + s * stride);
  F2 g[NP], b[NP];
  {
    float p[kTeamElems];
    M::params(a.gamma, a.ptype, a.wideParams, 1.f, cols, t, p);
#pragma unroll
    for (int i = 0; i < NP; ++i) g[i] = pair(p[2 * i], p[2 * i + 1]);
    M::params(a.beta, a.ptype, a.wideParams, 0.f, cols, t, p);
#pragma unroll
    for (int i = 0; i < NP; ++i) b[i] = pair(p[2 * i], p[2 * i + 1]);
  }
  const float inv = 1.f / (float)cols;
  const bool high = lane >= 16;
  // elements of warp w of the team: of this thread's own, and of the one its lane joins
  auto warpCount = [&](int w) {
    int n = 0;
    for (int j = 0; j < M::NV; ++j) n += min(32, max(0, (cols + M::V - 1) / M::V - j * T - w * 32)) * M::V;
    return (float)n;
  };
  const float ownCount = warpCount(t >> 5), ownInv = ownCount > 0.f ? 1.f / ownCount : 0.f;
  const float joinCount = (lane & 15) < warps ? warpCount(lane & 15) : 0.f, joinInv = joinCount > 0.f ? 1.f / joinCount : 0.f;
  teamSync<T>(team);
  int stage = 0, round = 0, turn = 0;
  for (size_t row = first; row < a.rows; row += 2 * stride, turn ^= 1) {
    const bool two = row + stride < a.rows;
    float f[2][kTeamElems];
    waitRow(&bar[stage], round & 1, dead, turn);
    M::take(mine + (size_t)stage * slot, a.x, a.ldx, row, a.rows, cols, t, f[0]);
    if (two) {
      waitRow(&bar[stage + 1], round & 1, dead, turn);
      M::take(mine + (size_t)(stage + 1) * slot, a.x, a.ldx, row + stride, a.rows, cols, t, f[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kTeamElems; ++i) f[1][i] = 0.f;
    }
    F2 x[2][NP];
    float s[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      F2 acc = 0;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        x[r][i] = pair(f[r][2 * i], f[r][2 * i + 1]);
        acc = add2(acc, x[r][i]);
      }
      const float2 q = split(acc);
      s[r] = q.x + q.y;
    }
    const float both = sumTwo(s[0], s[1], high);
    const float m0 = __shfl_sync(0xffffffffu, both, 0) * ownInv, m1 = __shfl_sync(0xffffffffu, both, 16) * ownInv;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const F2 minus = pair(r ? -m1 : -m0, r ? -m1 : -m0);
      F2 acc = 0;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const F2 d = add2(x[r][i], minus);
        if constexpr (VEC) {
          if (M::held(2 * i, cols, t)) acc = fma2(d, d, acc);
        } else {
          const float2 q = split(d);
          acc = fma2(d, pair(M::held(2 * i, cols, t) ? q.x : 0.f, M::held(2 * i + 1, cols, t) ? q.y : 0.f), acc);
        }
      }
      const float2 q = split(acc);
      s[r] = q.x + q.y;
    }
    const float squares = sumTwo(s[0], s[1], high);
    if ((lane & 15) == 0) red[team][turn][high][t >> 5] = make_float2(both, squares);
    teamSync<T>(team);
    if (givenUp(*reinterpret_cast<volatile int*>(dead), turn)) {
      abandon(bar, stages, stage, round, t == 0, dead, turn);
      break;
    }
    if (t == 0) {
      refill(stage, row + stages * stride);
      refill(stage + 1, row + (stages + 1) * stride);
    }
    // squares = sum over warps of squares_w + count_w (mean_w - mean)^2
    const float2 w = (lane & 15) < warps ? red[team][turn][high][lane & 15] : make_float2(0.f, 0.f);
    const float mean = sumHalf(w.x) * inv, d = w.x * joinInv - mean;
    const float rstd = rsqrtf(sumHalf(w.y + joinCount * d * d) * inv + a.eps);
    if (t == 0 || (t == 16 && two)) {
      const size_t at = t ? row + stride : row;
      if (a.mean) a.mean[at] = mean;
      if (a.rstd) a.rstd[at] = rstd;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float rs = __shfl_sync(0xffffffffu, rstd, r * 16), mn = __shfl_sync(0xffffffffu, mean, r * 16);
      if (r && !two) break;
      const F2 scale = pair(rs, rs), shift = pair(-mn, -mn);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float2 q = split(fma2(mul2(add2(x[r][i], shift), scale), g[i], b[i]));
        f[r][2 * i] = q.x;
        f[r][2 * i + 1] = q.y;
      }
      M::store(static_cast<char*>(a.y) + (row + r * stride) * a.ldy * E, cols, t, f[r]);
    }
    if ((stage += 2) == stages) {
      stage = 0;
      ++round;
    }
  }
}

// Backward: x and dy rows arrive together, a row a turn; the columns' two sums
// stay in registers to the end, where the block's teams add them up. 8192
// columns of bf16 are one team a multiprocessor: a row's 48 KB take 2100 cycles
// at the memory's rate, its reduction's latency about 1500, most of it under
// the next rows' copies.
template <int DT, bool VEC, int T>
__global__ void __launch_bounds__(512) normBackwardTeams(const __grid_constant__ NormArgs a) {
  using M = Team<DT, VEC, T>;
  constexpr int E = M::E, NP = kTeamElems / 2;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ unsigned long long full[16 * kMaxStages];
  __shared__ float2 red[16][2][16];
  __shared__ int deadWord[16];
  const int team = threadIdx.x / T, t = threadIdx.x % T, lane = t & 31;
  const int cols = a.cols, stages = a.stages, slot = slotBytes(cols, E);
  constexpr int warps = T / 32;
  unsigned char* mine = ring + (size_t)team * stages * 2 * slot;
  unsigned long long* bar = full + team * kMaxStages;
  int* dead = &deadWord[team];
  const size_t stride = (size_t)gridDim.x * a.teams, first = (size_t)blockIdx.x * a.teams + team;
  unsigned long long policy = 0;
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbarInit(&bar[s], 1);
    *dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    policy = evictFirstPolicy();
  }
  auto refill = [&](int s, size_t row) {
    if (row >= a.rows) return;
    unsigned char* q = mine + (size_t)s * 2 * slot;
    M::edges(q, a.x, a.ldx, row, a.rows, cols, a.cutX);
    M::edges(q + slot, a.dy, a.lddy, row, a.rows, cols, a.cutDy);
    expectBytes(&bar[s], M::fetchBytes(a.x, a.ldx, row, a.rows, cols, a.cutX) + M::fetchBytes(a.dy, a.lddy, row, a.rows, cols, a.cutDy));
    M::fetch(q, a.x, a.ldx, row, a.rows, cols, a.cutX, &bar[s], policy);
    M::fetch(q + slot, a.dy, a.lddy, row, a.rows, cols, a.cutDy, &bar[s], policy);
  };
  if (t == 0)
    for (int s = 0; s < stages; ++s) refill(s, first + s * stride);
  F2 g[NP], dg[NP], db[NP];
  {
    float p[kTeamElems];
    M::params(a.gamma, a.ptype, a.wideParams, 1.f, cols, t, p);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      g[i] = pair(p[2 * i], p[2 * i + 1]);
      dg[i] = db[i] = 0;
    }
  }
  const float inv = 1.f / (float)cols;
  letNextIn();
  float nextMean = 0.f, nextRstd = 0.f;
  if (first < a.rows) {
    nextMean = a.mean[first];
    nextRstd = a.rstd[first];
  }
  teamSync<T>(team);
  int stage = 0, round = 0, turn = 0;
  for (size_t row = first; row < a.rows; row += stride, turn ^= 1) {
    const float mean = nextMean, rstd = nextRstd;
    waitRow(&bar[stage], round & 1, dead, turn);
    const unsigned char* q = mine + (size_t)stage * 2 * slot;
    F2 xh[NP], gd[NP];
    float2 s;
    {
      float f[kTeamElems];
      const F2 scale = pair(rstd, rstd), shift = pair(-mean, -mean);
      M::take(q, a.x, a.ldx, row, a.rows, cols, t, f);
#pragma unroll
      for (int i = 0; i < NP; ++i) xh[i] = mul2(add2(pair(f[2 * i], f[2 * i + 1]), shift), scale);
      M::take(q + slot, a.dy, a.lddy, row, a.rows, cols, t, f);
      F2 sg = 0, sx = 0;  // dy is zero in columns that do not exist
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const F2 d = pair(f[2 * i], f[2 * i + 1]);
        gd[i] = mul2(d, g[i]);
        sg = add2(sg, gd[i]);
        sx = fma2(gd[i], xh[i], sx);
        dg[i] = fma2(d, xh[i], dg[i]);
        db[i] = add2(db[i], d);
      }
      const float2 u = split(sg), w = split(sx);
      s = make_float2(u.x + u.y, w.x + w.y);
    }
    const float part = sumTwo(s.x, s.y, lane >= 16);
    if ((lane & 15) == 0) reinterpret_cast<float*>(&red[team][turn][t >> 5])[lane >> 4] = part;
    teamSync<T>(team);
    if (givenUp(*reinterpret_cast<volatile int*>(dead), turn)) {
      abandon(bar, stages, stage, round, t == 0, dead, turn);
      break;
    }
    if (t == 0) refill(stage, row + stages * stride);
    if (row + stride < a.rows) {
      nextMean = a.mean[row + stride];
      nextRstd = a.rstd[row + stride];
    }
    const float joined = sumHalf((lane & 15) < warps ? reinterpret_cast<float*>(&red[team][turn][lane & 15])[lane >> 4] : 0.f);
    const float m1 = __shfl_sync(0xffffffffu, joined, 0) * inv, m2 = __shfl_sync(0xffffffffu, joined, 16) * inv;
    const F2 n1 = pair(-m1, -m1), n2 = pair(-m2, -m2), scale = pair(rstd, rstd);
    float f[kTeamElems];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 u = split(mul2(scale, fma2(xh[i], n2, add2(gd[i], n1))));
      f[2 * i] = u.x;
      f[2 * i + 1] = u.y;
    }
    M::store(static_cast<char*>(a.y) + row * a.ldy * E, cols, t, f);
    if (++stage == stages) {
      stage = 0;
      ++round;
    }
  }
  if (!a.partial) return;
  // the teams own the same columns: every team lays its sums out, and the block adds them in the teams' order
  float* sum = reinterpret_cast<float*>(ring);
  __syncthreads();  // no team reads its ring any more
  M::layOut(sum + (size_t)team * 2 * cols, dg, db, cols, t);
  __syncthreads();
  float* p = a.partial + (size_t)blockIdx.x * 2 * cols;
  for (int c = threadIdx.x; c < 2 * cols; c += blockDim.x) {
    float x = sum[c];
    for (int w = 1; w < a.teams; ++w) x += sum[(size_t)w * 2 * cols + c];
    p[c] = x;
  }
}

// ------------------------------------------------------------ narrow rows
// Rows of at most 32 whole vectors (heads, and their like): G lanes a row, one
// vector each, 32 / G rows a warp at a time and kNarrowTurn such steps in
// flight. Such rows reduce within a warp; there is nothing to wait for.
constexpr int kNarrowTurn = 4, kNarrowThreads = 256;

template <int G>
__device__ __forceinline__ float sumLanes(float x) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int DT, int G>
__global__ void __launch_bounds__(kNarrowThreads) normForwardNarrow(const __grid_constant__ NormArgs a) {
  constexpr int E = floatTypeSize(DT), V = 16 / E, R = 32 / G, U = kNarrowTurn;
  const int lane = threadIdx.x & 31, own = lane % G;
  const bool held = own * V < a.cols;
  const size_t warps = (size_t)gridDim.x * (kNarrowThreads / 32);
  const float inv = 1.f / (float)a.cols;
  F2 g[V / 2], b[V / 2];
  {
    float p[V];
    if (held) {
      loadParams<V>(a.gamma, a.ptype, a.wideParams, own * V, 1.f, p);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) g[e] = pair(p[2 * e], p[2 * e + 1]);
      loadParams<V>(a.beta, a.ptype, a.wideParams, own * V, 0.f, p);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) b[e] = pair(p[2 * e], p[2 * e + 1]);
    }
  }
  for (size_t r0 = ((size_t)blockIdx.x * (kNarrowThreads / 32) + (threadIdx.x >> 5)) * R * U; r0 < a.rows; r0 += warps * R * U) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t row = r0 + u * R + lane / G;
      raw[u] = held && row < a.rows ? __ldcs(reinterpret_cast<const uint4*>(static_cast<const char*>(a.x) + row * a.ldx * E) + own)
                                    : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t row = r0 + u * R + lane / G;
      float f[V];
      Vec16<DT>::expand(raw[u], f);
      F2 x[V / 2], acc = 0;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        x[e] = pair(f[2 * e], f[2 * e + 1]);
        acc = add2(acc, x[e]);
      }
      float2 q = split(acc);
      const float mean = sumLanes<G>(q.x + q.y) * inv;
      const F2 shift = pair(-mean, -mean);
      acc = 0;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        x[e] = add2(x[e], shift);
        acc = fma2(x[e], x[e], acc);
      }
      q = split(acc);
      const float rstd = rsqrtf(sumLanes<G>(held ? q.x + q.y : 0.f) * inv + a.eps);
      if (row >= a.rows) continue;
      if (own == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
      if (held) {
        const F2 scale = pair(rstd, rstd);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          const float2 y = split(fma2(mul2(x[e], scale), g[e], b[e]));
          f[2 * e] = y.x;
          f[2 * e + 1] = y.y;
        }
        __stcs(reinterpret_cast<uint4*>(static_cast<char*>(a.y) + row * a.ldy * E) + own, Vec16<DT>::pack(f));
      }
    }
  }
}

template <int DT, int G>
__global__ void __launch_bounds__(kNarrowThreads) normBackwardNarrow(const __grid_constant__ NormArgs a) {
  constexpr int E = floatTypeSize(DT), V = 16 / E, R = 32 / G, U = kNarrowTurn;
  __shared__ float sum[kNarrowThreads / 32][2][32 * V];
  const int lane = threadIdx.x & 31, own = lane % G, w = threadIdx.x >> 5;
  const bool held = own * V < a.cols;
  const size_t warps = (size_t)gridDim.x * (kNarrowThreads / 32);
  const float inv = 1.f / (float)a.cols;
  F2 g[V / 2], dg[V / 2], db[V / 2];
  {
    float p[V] = {};
    if (held) loadParams<V>(a.gamma, a.ptype, a.wideParams, own * V, 1.f, p);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      g[e] = pair(p[2 * e], p[2 * e + 1]);
      dg[e] = db[e] = 0;
    }
  }
  letNextIn();
  for (size_t r0 = ((size_t)blockIdx.x * (kNarrowThreads / 32) + w) * R * U; r0 < a.rows; r0 += warps * R * U) {
    uint4 rx[U], rd[U];
    float mean[U], rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t row = r0 + u * R + lane / G;
      const bool there = held && row < a.rows;
      rx[u] = there ? __ldcs(reinterpret_cast<const uint4*>(static_cast<const char*>(a.x) + row * a.ldx * E) + own) : make_uint4(0, 0, 0, 0);
      rd[u] = there ? __ldcs(reinterpret_cast<const uint4*>(static_cast<const char*>(a.dy) + row * a.lddy * E) + own) : make_uint4(0, 0, 0, 0);
      mean[u] = row < a.rows ? a.mean[row] : 0.f;
      rstd[u] = row < a.rows ? a.rstd[row] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t row = r0 + u * R + lane / G;
      float fx[V], fd[V];
      Vec16<DT>::expand(rx[u], fx);
      Vec16<DT>::expand(rd[u], fd);  // zero where nothing is held: such lanes add nothing to any sum
      const F2 shift = pair(-mean[u], -mean[u]), scale = pair(rstd[u], rstd[u]);
      F2 xh[V / 2], gd[V / 2], sg = 0, sx = 0;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const F2 d = pair(fd[2 * e], fd[2 * e + 1]);
        xh[e] = mul2(add2(pair(fx[2 * e], fx[2 * e + 1]), shift), scale);
        gd[e] = mul2(d, g[e]);
        sg = add2(sg, gd[e]);
        sx = fma2(gd[e], xh[e], sx);
        dg[e] = fma2(d, xh[e], dg[e]);
        db[e] = add2(db[e], d);
      }
      const float2 q = split(sg), r = split(sx);
      const float m1 = sumLanes<G>(q.x + q.y) * inv, m2 = sumLanes<G>(r.x + r.y) * inv;
      if (held && row < a.rows) {
        const F2 n1 = pair(-m1, -m1), n2 = pair(-m2, -m2);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          const float2 v = split(mul2(scale, fma2(xh[e], n2, add2(gd[e], n1))));
          fx[2 * e] = v.x;
          fx[2 * e + 1] = v.y;
        }
        __stcs(reinterpret_cast<uint4*>(static_cast<char*>(a.y) + row * a.ldy * E) + own, Vec16<DT>::pack(fx));
      }
    }
  }
  if (!a.partial) return;
  // the warp's row groups hold the same columns, then the block's warps do
#pragma unroll
  for (int e = 0; e < V / 2; ++e) {
#pragma unroll
    for (int o = G; o < 32; o *= 2) {
      dg[e] = add2(dg[e], __shfl_xor_sync(0xffffffffu, dg[e], o));
      db[e] = add2(db[e], __shfl_xor_sync(0xffffffffu, db[e], o));
    }
    if (lane < G) {
      *reinterpret_cast<F2*>(&sum[w][0][own * V + 2 * e]) = dg[e];
      *reinterpret_cast<F2*>(&sum[w][1][own * V + 2 * e]) = db[e];
    }
  }
  __syncthreads();
  float* p = a.partial + (size_t)blockIdx.x * 2 * a.cols;
  for (int i = threadIdx.x; i < 2 * a.cols; i += kNarrowThreads) {
    const int which = i >= a.cols, c = i - which * a.cols;
    float x = sum[0][which][c];
#pragma unroll
    for (int k = 1; k < kNarrowThreads / 32; ++k) x += sum[k][which][c];
    p[i] = x;
  }
}

// ------------------------------------------------------------ a whole block for a row
// Rows of up to 16384 elements: a team of up to 1024 threads, which leaves each
// 64 registers. What the smaller teams keep in registers is divided: forward
// holds the row and reads the parameters from shared memory, backward holds the
// columns' sums and passes over the row's stage twice (so that a stage is
// refilled a row later, when the next barrier shows that all are through).
constexpr int kWideCols = 1024 * kTeamElems;

// A thread's own parameters in shared memory, pair i at [i T + t]: laid out so
// that a warp reads its pairs side by side (by column, vectors of eight would
// put its lanes 32 bytes apart and a read would take eight turns).
template <int DT, bool VEC, int T>
__device__ __forceinline__ void keepParams(F2* own, const void* p, int ptype, bool wide, float dflt, int cols, int t) {
  float f[kTeamElems];
  Team<DT, VEC, T>::params(p, ptype, wide, dflt, cols, t, f);
#pragma unroll
  for (int i = 0; i < kTeamElems / 2; ++i) own[i * T + t] = pair(f[2 * i], f[2 * i + 1]);
}

template <int DT, bool VEC, int T>
__global__ void __launch_bounds__(T, 1) normForwardWide(const __grid_constant__ NormArgs a) {
  using M = Team<DT, VEC, T>;
  constexpr int E = M::E, NP = kTeamElems / 2;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ unsigned long long full[kMaxStages];
  __shared__ float2 red[2][32];
  __shared__ int dead;
  constexpr int warps = T / 32;
  const int t = threadIdx.x, lane = t & 31;
  const int cols = a.cols, stages = a.stages, slot = slotBytes(cols, E);
  F2* gamma = reinterpret_cast<F2*>(ring + (size_t)stages * slot);
  F2* beta = gamma + NP * T;
  const size_t stride = gridDim.x;
  unsigned long long policy = 0;
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbarInit(&full[s], 1);
    dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    policy = evictFirstPolicy();
  }
  auto refill = [&](int s, size_t row) {
    if (row >= a.rows) return;
    M::edges(ring + (size_t)s * slot, a.x, a.ldx, row, a.rows, cols, a.cutX);
    expectBytes(&full[s], M::fetchBytes(a.x, a.ldx, row, a.rows, cols, a.cutX));
    M::fetch(ring + (size_t)s * slot, a.x, a.ldx, row, a.rows, cols, a.cutX, &full[s], policy);
  };
  if (t == 0)
    for (int s = 0; s < stages; ++s) refill(s, blockIdx.x + s * stride);
  keepParams<DT, VEC, T>(gamma, a.gamma, a.ptype, a.wideParams, 1.f, cols, t);
  keepParams<DT, VEC, T>(beta, a.beta, a.ptype, a.wideParams, 0.f, cols, t);
  const float inv = 1.f / (float)cols;
  auto warpCount = [&](int w) {
    int n = 0;
    for (int j = 0; j < M::NV; ++j) n += min(32, max(0, (cols + M::V - 1) / M::V - j * T - w * 32)) * M::V;
    return (float)n;
  };
  const float ownCount = warpCount(t >> 5), ownInv = ownCount > 0.f ? 1.f / ownCount : 0.f;
  const float joinCount = lane < warps ? warpCount(lane) : 0.f, joinInv = joinCount > 0.f ? 1.f / joinCount : 0.f;
  __syncthreads();
  int stage = 0, round = 0, turn = 0;
  for (size_t row = blockIdx.x; row < a.rows; row += stride, turn ^= 1) {
    waitRow(&full[stage], round & 1, &dead, turn);
    F2 x[NP];
    float s;
    {
      float f[kTeamElems];
      M::take(ring + (size_t)stage * slot, a.x, a.ldx, row, a.rows, cols, t, f);
      F2 acc = 0;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        x[i] = pair(f[2 * i], f[2 * i + 1]);
        acc = add2(acc, x[i]);
      }
      const float2 q = split(acc);
      s = warpSum(q.x + q.y);
    }
    float squares;
    {
      const F2 minus = pair(-s * ownInv, -s * ownInv);
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float2 d = split(add2(x[i], minus));
        q += M::held(2 * i, cols, t) ? d.x * d.x : 0.f;
        q += M::held(2 * i + 1, cols, t) ? d.y * d.y : 0.f;
      }
      squares = warpSum(q);
    }
    if (lane == 0) red[turn][t >> 5] = make_float2(s, squares);
    __syncthreads();
    if (givenUp(*reinterpret_cast<volatile int*>(&dead), turn)) {
      abandon(full, stages, stage, round, t == 0, &dead, turn);
      break;
    }
    if (t == 0) refill(stage, row + stages * stride);
    const float2 w = lane < warps ? red[turn][lane] : make_float2(0.f, 0.f);
    const float mean = warpSum(w.x) * inv, d = w.x * joinInv - mean;
    const float rstd = rsqrtf(warpSum(w.y + joinCount * d * d) * inv + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    float f[kTeamElems];
    const F2 scale = pair(rstd, rstd), shift = pair(-mean, -mean);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 q = split(fma2(mul2(add2(x[i], shift), scale), gamma[i * T + t], beta[i * T + t]));
      f[2 * i] = q.x;
      f[2 * i + 1] = q.y;
    }
    M::store(static_cast<char*>(a.y) + row * a.ldy * E, cols, t, f);
    if (++stage == stages) {
      stage = 0;
      ++round;
    }
  }
}

// fn(0), fn(N), ... over a thread's elements, the argument a constant.
template <int N, int FROM = 0, typename Fn>
__device__ __forceinline__ void chunks(Fn& fn) {
  if constexpr (FROM < kTeamElems) {
    fn(std::integral_constant<int, FROM>{});
    chunks<N, FROM + N>(fn);
  }
}

template <int DT, bool VEC, int T>
__global__ void __launch_bounds__(T, 1) normBackwardWide(const __grid_constant__ NormArgs a) {
  using M = Team<DT, VEC, T>;
  constexpr int E = M::E, NP = kTeamElems / 2, kChunk = VEC ? 8 : 4;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ unsigned long long full[kMaxStages];
  __shared__ float2 red[2][32];
  __shared__ int dead;
  constexpr int warps = T / 32;
  const int t = threadIdx.x, lane = t & 31;
  const int cols = a.cols, stages = a.stages, slot = slotBytes(cols, E);
  F2* gamma = reinterpret_cast<F2*>(ring + (size_t)stages * 2 * slot);
  const size_t stride = gridDim.x;
  unsigned long long policy = 0;
  if (t == 0) {
    for (int s = 0; s < stages; ++s) mbarInit(&full[s], 1);
    dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    policy = evictFirstPolicy();
  }
  auto refill = [&](int s, size_t row) {
    if (row >= a.rows) return;
    unsigned char* q = ring + (size_t)s * 2 * slot;
    M::edges(q, a.x, a.ldx, row, a.rows, cols, a.cutX);
    M::edges(q + slot, a.dy, a.lddy, row, a.rows, cols, a.cutDy);
    expectBytes(&full[s], M::fetchBytes(a.x, a.ldx, row, a.rows, cols, a.cutX) + M::fetchBytes(a.dy, a.lddy, row, a.rows, cols, a.cutDy));
    M::fetch(q, a.x, a.ldx, row, a.rows, cols, a.cutX, &full[s], policy);
    M::fetch(q + slot, a.dy, a.lddy, row, a.rows, cols, a.cutDy, &full[s], policy);
  };
  if (t == 0)
    for (int s = 0; s < stages; ++s) refill(s, blockIdx.x + s * stride);
  keepParams<DT, VEC, T>(gamma, a.gamma, a.ptype, a.wideParams, 1.f, cols, t);
  F2 dg[NP], db[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) dg[i] = db[i] = 0;
  const float inv = 1.f / (float)cols;
  letNextIn();
  __syncthreads();
  int stage = 0, round = 0, turn = 0, behind = 0;
  for (size_t row = blockIdx.x; row < a.rows; row += stride, turn ^= 1) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    waitRow(&full[stage], round & 1, &dead, turn);
    const unsigned char* q = ring + (size_t)stage * 2 * slot;
    const F2 scale = pair(rstd, rstd), shift = pair(-mean, -mean);
    F2 sg = 0, sx = 0;
    // a few elements at a time: more at once would not fit beside the sums, and what spills finds no L1 (shared memory
    // has it)
    auto sums = [&](auto from) {
      constexpr int kFrom = decltype(from)::value;
      float fx[kChunk], fd[kChunk];
      M::template takeSome<kFrom, kChunk>(q, a.x, a.ldx, row, a.rows, cols, t, fx);
      M::template takeSome<kFrom, kChunk>(q + slot, a.dy, a.lddy, row, a.rows, cols, t, fd);
#pragma unroll
      for (int i = 0; i < kChunk / 2; ++i) {
        const int p = kFrom / 2 + i;
        const F2 xh = mul2(add2(pair(fx[2 * i], fx[2 * i + 1]), shift), scale), d = pair(fd[2 * i], fd[2 * i + 1]);
        const F2 gd = mul2(d, gamma[p * T + t]);
        sg = add2(sg, gd);
        sx = fma2(gd, xh, sx);
        dg[p] = fma2(d, xh, dg[p]);
        db[p] = add2(db[p], d);
      }
      asm volatile("" ::: "memory");
    };
    chunks<kChunk>(sums);
    const float2 u = split(sg), w = split(sx);
    const float2 s = warpSum2(make_float2(u.x + u.y, w.x + w.y));
    if (lane == 0) red[turn][t >> 5] = s;
    __syncthreads();
    if (givenUp(*reinterpret_cast<volatile int*>(&dead), turn)) {
      abandon(full, stages, stage, round, t == 0, &dead, turn);
      break;
    }
    // all are through with the row before this one: its stage takes the row `stages` after it
    if (t == 0 && stages > 1 && row != blockIdx.x) refill(behind, row + (stages - 1) * stride);
    behind = stage;
    const float2 m = warpSum2(lane < warps ? red[turn][lane] : make_float2(0.f, 0.f));
    const F2 n1 = pair(-m.x * inv, -m.x * inv), n2 = pair(-m.y * inv, -m.y * inv);
    auto outputs = [&](auto from) {
      constexpr int kFrom = decltype(from)::value;
      float fx[kChunk], fd[kChunk];
      M::template takeSome<kFrom, kChunk>(q, a.x, a.ldx, row, a.rows, cols, t, fx);
      M::template takeSome<kFrom, kChunk>(q + slot, a.dy, a.lddy, row, a.rows, cols, t, fd);
#pragma unroll
      for (int i = 0; i < kChunk / 2; ++i) {
        const F2 xh = mul2(add2(pair(fx[2 * i], fx[2 * i + 1]), shift), scale), g = gamma[(kFrom / 2 + i) * T + t];
        const float2 v = split(mul2(scale, fma2(xh, n2, fma2(pair(fd[2 * i], fd[2 * i + 1]), g, n1))));
        fx[2 * i] = v.x;
        fx[2 * i + 1] = v.y;
      }
      M::storeSome(static_cast<char*>(a.y) + row * a.ldy * E, cols, t, kFrom, fx, kChunk);
      asm volatile("" ::: "memory");
    };
    chunks<kChunk>(outputs);
    if (stages == 1) {  // (binary32 rows of 11261 elements and more: there is room for one)
      __syncthreads();
      if (t == 0) refill(0, row + stride);
    }
    if (++stage == stages) {
      stage = 0;
      ++round;
    }
  }
  if (!a.partial) return;
  M::layOut(a.partial + (size_t)blockIdx.x * 2 * cols, dg, db, cols, t);
}

// ------------------------------------------------------------ longer rows
// Rows of up to 32768 elements forward, one a block, EPT elements a thread, the parameters read where they are used.
template <int DT, bool VEC, int EPT>
__global__ void __launch_bounds__(1024) normForward(const __grid_constant__ NormArgs a) {
  using H = Held<DT, VEC, EPT>;
  constexpr int V = H::V, NV = H::NV, E = floatTypeSize(DT);
  __shared__ float red[2][32];
  const int T = blockDim.x, t = threadIdx.x;
  const float inv = 1.f / (float)a.cols;
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    H h;
    h.load(static_cast<const char*>(a.x) + row * a.ldx * E, t, T, a.cols);
    float f[V], s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      h.get(j, f);
#pragma unroll
      for (int e = 0; e < V; ++e) s += f[e];
    }
    const float mean = blockSum(s, red[0]) * inv;
    s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if ((j * T + t) * V < a.cols) {
        h.get(j, f);
#pragma unroll
        for (int e = 0; e < V; ++e) s += (f[e] - mean) * (f[e] - mean);
      }
    }
    const float rstd = 1.f / sqrtf(blockSum(s, red[1]) * inv + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    void* out = static_cast<char*>(a.y) + row * a.ldy * E;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = j * T + t;
      if (i * V < a.cols) {
        float g[V], b[V];
        loadParams<V>(a.gamma, a.ptype, a.wideParams, i * V, 1.f, g);
        loadParams<V>(a.beta, a.ptype, a.wideParams, i * V, 0.f, b);
        h.get(j, f);
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = (f[e] - mean) * rstd * g[e] + b[e];
        H::put(out, i, f);
      }
    }
  }
}

// Rows longer than a block holds: three passes over the row, the later ones
// through L2.
template <int DT>
__global__ void __launch_bounds__(1024) normForwardLong(const __grid_constant__ NormArgs a) {
  constexpr int E = floatTypeSize(DT);
  __shared__ float red[2][32];
  const float inv = 1.f / (float)a.cols;
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char* x = static_cast<const char*>(a.x) + row * a.ldx * E;
    float s = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) s += loadOne<DT>(x, c);
    const float mean = blockSum(s, red[0]) * inv;
    s = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float d = loadOne<DT>(x, c) - mean;
      s += d * d;
    }
    const float rstd = 1.f / sqrtf(blockSum(s, red[1]) * inv + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    using S = typename Ty<DT>::S;
    S* y = reinterpret_cast<S*>(static_cast<char*>(a.y) + row * a.ldy * E);
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = a.gamma ? loadParam(a.gamma, a.ptype, c) : 1.f, b = a.beta ? loadParam(a.beta, a.ptype, c) : 0.f;
      y[c] = Ty<DT>::fromF((loadOne<DT>(x, c) - mean) * rstd * g + b);
    }
  }
}

// Rows longer than a block holds: the row's two sums, then dx, each a pass
// over the row; the weight's gradient by normColumns.
template <int DT>
__global__ void __launch_bounds__(1024) normBackwardLong(const __grid_constant__ NormArgs a) {
  constexpr int E = floatTypeSize(DT);
  __shared__ float2 red[2][32];
  const float inv = 1.f / (float)a.cols;
  int turn = 0;
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char* x = static_cast<const char*>(a.x) + row * a.ldx * E;
    const char* dy = static_cast<const char*>(a.dy) + row * a.lddy * E;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float2 s = make_float2(0.f, 0.f);
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = loadOne<DT>(dy, c) * (a.gamma ? loadParam(a.gamma, a.ptype, c) : 1.f);
      s.x += g;
      s.y += g * (loadOne<DT>(x, c) - mean) * rstd;
    }
    s = blockSum2(s, red[turn ^= 1]);
    using S = typename Ty<DT>::S;
    S* dx = reinterpret_cast<S*>(static_cast<char*>(a.y) + row * a.ldy * E);
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = loadOne<DT>(dy, c) * (a.gamma ? loadParam(a.gamma, a.ptype, c) : 1.f);
      dx[c] = Ty<DT>::fromF(rstd * (g - s.x * inv - (loadOne<DT>(x, c) - mean) * rstd * s.y * inv));
    }
  }
}
// Partial column sums of long rows: block (i, p) takes 256 columns and every
// gridDim.y-th row. It runs before normBackwardLong, which may overwrite dy.
template <int DT>
__global__ void __launch_bounds__(256) normColumns(const __grid_constant__ NormArgs a) {
  constexpr int E = floatTypeSize(DT);
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float dg = 0.f, db = 0.f;
  for (size_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float d = loadOne<DT>(static_cast<const char*>(a.dy) + row * a.lddy * E, c);
    dg += d * (loadOne<DT>(static_cast<const char*>(a.x) + row * a.ldx * E, c) - a.mean[row]) * a.rstd[row];
    db += d;
  }
  float* p = a.partial + (size_t)blockIdx.y * 2 * a.cols;
  p[c] = dg;
  p[a.cols + c] = db;
}

// dgamma and dbeta from the blocks' partial sums: 32 columns a block, the
// partial rows split over its 32 warps (a handful each, all asked for at once)
// and joined in warp order.
__global__ void __launch_bounds__(1024) normJoin(const float* partial, int blocks, int cols, void* dgamma, void* dbeta,
                                                 int ptype) {
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), which = blockIdx.y;
  waitForPrevious();
  const float s = columnSum(partial + (size_t)which * cols + c, blocks, (size_t)2 * cols, c < cols);
  void* out = which ? dbeta : dgamma;
  if (threadIdx.x < 32 && c < cols && out) storeParam(out, ptype, c, s);
}

// ------------------------------------------------------------ host

enum Walk { kNarrow, kTeams, kWide, kBlockRow, kLongRow };
struct Shape {
  Walk walk;
  bool vec;
  int threads;   // of a block
  int teams, teamThreads, stages, smem;
  int resident;  // blocks a multiprocessor
};
// The thread counts that kernels are made for.
constexpr int kTeamSizes[] = {32, 64, 96, 128, 192, 256, 320, 384, 512, 640, 768, 1024};
int teamThreads(int cols) {
  for (int t : kTeamSizes)
    if (t * kTeamElems >= cols) return t;
  return 0;
}
Shape normShape(size_t rows, int cols, int elem, bool aligned, bool forward) {
  Shape s = {};
  s.vec = aligned && cols % (16 / elem) == 0;
  s.teams = 1;
  auto up = [](int n, int per) { return std::max(32, (n + per * 32 - 1) / (per * 32) * 32); };
  if (s.vec && cols <= 32 * (16 / elem)) {
    s.walk = kNarrow;
    s.threads = kNarrowThreads;
    int lanes = 4;
    while (lanes * (16 / elem) < cols) lanes *= 2;
    s.teamThreads = lanes;
    s.teams = kNarrowThreads / lanes * kNarrowTurn;  // rows a block takes at a time
    s.resident = 4;
  } else if (cols <= kTeamCols) {
    // one block of up to 512 threads a multiprocessor: 128 registers each. With few rows, fewer teams to a block.
    s.walk = kTeams;
    s.teamThreads = teamThreads(cols);
    s.teams = (int)std::min<size_t>(512 / s.teamThreads, std::max<size_t>(1, (rows + smCount() - 1) / smCount()));
    s.threads = s.teams * s.teamThreads;
    const int row = slotBytes(cols, elem) * (forward ? 1 : 2);
    // no more stages than a team has rows (and two: forward takes two rows at a time)
    const size_t turns = (rows + (size_t)smCount() * s.teams - 1) / ((size_t)smCount() * s.teams);
    s.stages = std::min(kMaxStages, kTeamSmem / (s.teams * row)) & (forward ? ~1 : ~0);
    s.stages = (int)std::min<size_t>(s.stages, std::max<size_t>(2, (turns + 1) & ~size_t(1)));
    s.smem = s.teams * s.stages * row;
    s.resident = 1;
  } else if (cols <= kWideCols) {
    s.walk = kWide;
    s.threads = teamThreads(cols);
    const int row = slotBytes(cols, elem) * (forward ? 1 : 2), params = s.threads * kTeamElems * 4 * (forward ? 2 : 1);
    s.stages = std::min(4, (kWideSmem - params) / row);
    s.smem = s.stages * row + params;
    s.resident = 1;
  } else if (forward && cols <= kMaxHeldCols) {
    s.walk = kBlockRow;
    s.threads = up(cols, 32);
    s.resident = 1 << 20;
  } else {
    s.walk = kLongRow;
    s.threads = 1024;
    s.resident = forward ? 1 << 20 : 2;
  }
  return s;
}
int normBlocks(size_t rows, const Shape& s) {
  return (int)std::min<size_t>((rows + s.teams - 1) / s.teams, (size_t)smCount() * s.resident);
}
// Row blocks of the partial sums, whatever the strides and the type of a call.
int mostBlocks(size_t rows, int cols) {
  int most = 0;
  for (int elem : {2, 4})
    for (bool aligned : {false, true}) most = std::max(most, normBlocks(rows, normShape(rows, cols, elem, aligned, false)));
  return most;
}

using NormFn = void (*)(NormArgs);
template <int DT, bool VEC, bool FWD, int I = 0>
NormFn pickTeams(int threads) {
  constexpr int T = kTeamSizes[I];
  if constexpr (T < 1024)
    if (threads > T) return pickTeams<DT, VEC, FWD, I + 1>(threads);
  if constexpr (FWD && T <= 512)
    return normForwardTeams<DT, VEC, T>;
  else if constexpr (FWD)
    return normForwardWide<DT, VEC, T>;
  else if constexpr (T <= 512)
    return normBackwardTeams<DT, VEC, T>;
  else
    return normBackwardWide<DT, VEC, T>;
}
template <int DT, bool FWD, int G = 4>
NormFn pickNarrow(int lanes) {
  if constexpr (G < 32)
    if (lanes > G) return pickNarrow<DT, FWD, 2 * G>(lanes);
  if constexpr (FWD)
    return normForwardNarrow<DT, G>;
  else
    return normBackwardNarrow<DT, G>;
}
template <int DT, bool FWD>
NormFn pickKernel(const Shape& s) {
  if (s.walk == kLongRow) {
    if constexpr (FWD) return normForwardLong<DT>;
    else return normBackwardLong<DT>;
  }
  if constexpr (FWD)
    if (s.walk == kBlockRow) return s.vec ? normForward<DT, true, 32> : normForward<DT, false, 32>;
  if (s.walk == kNarrow) return pickNarrow<DT, FWD>(s.teamThreads);
  const int threads = s.walk == kTeams ? s.teamThreads : s.threads;
  return s.vec ? pickTeams<DT, true, FWD>(threads) : pickTeams<DT, false, FWD>(threads);
}
template <bool FWD>
vrcclResult_t launchNorm(int dt, const Shape& s, unsigned blocks, NormArgs& a, cudaStream_t st) {
  const NormFn fn = dt == vrcclFloat32    ? pickKernel<vrcclFloat32, FWD>(s)
                    : dt == vrcclBfloat16 ? pickKernel<vrcclBfloat16, FWD>(s)
                                          : pickKernel<vrcclFloat16, FWD>(s);
  if (s.smem > 32 * 1024) {  // (beside static shared memory, 48 KB come without asking)
    const vrcclResult_t r = allowSharedMemory((const void*)fn);
    if (r != vrcclSuccess) return r;
  }
  a.stages = s.stages;
  a.teams = s.teams;
  return launchShaped(fn, {dim3(blocks), s.threads, s.smem, 0, false}, st, a);
}

bool goodSizes(size_t rows, size_t cols, int dtype, int ptype) {
  return rows < kMaxExtent && cols < (size_t(1) << 31) - 65536 && isOperatorType(dtype) && isOperatorType(ptype);
}

}  // namespace

int normStatus(int* code) { return cudaMemcpyFromSymbol(code, gRingStatus, sizeof(*code)); }

vrcclResult_t allowSharedMemory(const void* fn) {
  static std::mutex mu;
  static struct {
    const void* fn;
    int dev;
  } done[256];
  static int count = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return vrcclCudaError;
  }
  std::lock_guard<std::mutex> lk(mu);
  for (int i = 0; i < count; ++i)
    if (done[i].fn == fn && done[i].dev == dev) return vrcclSuccess;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, maxDynamicSmem(fn, dev)) != cudaSuccess) {
    cudaGetLastError();
    return vrcclCudaError;
  }
  if (count < 256) done[count++] = {fn, dev};
  return vrcclSuccess;
}

int smCount() {
  static int count[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 152;
  }
  if (!count[dev]) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    count[dev] = n > 0 ? n : 152;
  }
  return count[dev];
}

}  // namespace vrccl

using namespace vrccl;

extern "C" vrcclResult_t vrcclLayerNormForward(const void* x, size_t ldx, const void* gamma, const void* beta, void* y,
                                               size_t ldy, float* mean, float* rstd, size_t rows, size_t cols,
                                               vrcclDataType_t dtype, vrcclDataType_t paramType, float eps,
                                               vrcclStream_t stream) {
  if (!goodSizes(rows, cols, dtype, paramType) || !(eps >= 0.f)) return vrcclInvalidArgument;
  if (rows == 0 || cols == 0) return vrcclSuccess;
  const int E = floatTypeSize(dtype), PE = floatTypeSize(paramType);
  if (!goodMatrix(x, ldx, rows, cols, E) || !goodMatrix(y, ldy, rows, cols, E)) return vrcclInvalidArgument;
  if ((gamma && !goodVector(gamma, PE)) || (beta && !goodVector(beta, PE)) || (mean && !goodVector(mean, 4)) ||
      (rstd && !goodVector(rstd, 4)))
    return vrcclInvalidArgument;
  const Span out[] = {matrixSpan(y, ldy, rows, cols, E), vectorSpan(mean, rows * 4), vectorSpan(rstd, rows * 4)};
  const Span spanX = matrixSpan(x, ldx, rows, cols, E);
  const Span in[] = {unlessInPlace(spanX, ldx, y, ldy), vectorSpan(gamma, cols * PE), vectorSpan(beta, cols * PE)};
  if (!apart(out, in) || overlap(out[1], spanX) || overlap(out[2], spanX))
    return vrcclInvalidArgument;
  const Shape s = normShape(rows, (int)cols, E, rowsAligned(x, ldx, E) && rowsAligned(y, ldy, E), true);
  NormArgs a = {};
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.ldx = ldx;
  a.cutX = cutRows(ldx, E);
  a.ldy = ldy;
  a.rows = rows;
  a.cols = (int)cols;
  a.ptype = paramType;
  a.eps = eps;
  a.wideParams = (((uintptr_t)gamma | (uintptr_t)beta) & 15) == 0;
  return launchNorm<true>(dtype, s, (unsigned)normBlocks(rows, s), a, (cudaStream_t)stream);
}

extern "C" vrcclResult_t vrcclLayerNormWorkspace(size_t rows, size_t cols, size_t* bytes) {
  if (!bytes || !goodSizes(rows, cols, vrcclFloat32, vrcclFloat32)) return vrcclInvalidArgument;
  *bytes = size_t(mostBlocks(rows, (int)cols)) * 2 * cols * sizeof(float);
  return vrcclSuccess;
}

extern "C" vrcclResult_t vrcclLayerNormBackward(const void* dy, size_t lddy, const void* x, size_t ldx,
                                                const void* gamma, const float* mean, const float* rstd, void* dx,
                                                size_t lddx, void* dgamma, void* dbeta, size_t rows, size_t cols,
                                                vrcclDataType_t dtype, vrcclDataType_t paramType, void* workspace,
                                                size_t workspaceBytes, vrcclStream_t stream) {
  if (!goodSizes(rows, cols, dtype, paramType)) return vrcclInvalidArgument;
  if (cols == 0) return vrcclSuccess;
  const int E = floatTypeSize(dtype), PE = floatTypeSize(paramType);
  if ((gamma && !goodVector(gamma, PE)) || (dgamma && !goodVector(dgamma, PE)) || (dbeta && !goodVector(dbeta, PE)))
    return vrcclInvalidArgument;
  const bool weights = dgamma || dbeta;
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) {  // a sum over no rows
    if ((dgamma && cudaMemsetAsync(dgamma, 0, cols * PE, st) != cudaSuccess) ||
        (dbeta && cudaMemsetAsync(dbeta, 0, cols * PE, st) != cudaSuccess)) {
      cudaGetLastError();
      return vrcclCudaError;
    }
    return vrcclSuccess;
  }
  if (!goodMatrix(dy, lddy, rows, cols, E) || !goodMatrix(x, ldx, rows, cols, E) || !goodMatrix(dx, lddx, rows, cols, E) ||
      !goodVector(mean, 4) || !goodVector(rstd, 4))
    return vrcclInvalidArgument;
  const Shape s =
      normShape(rows, (int)cols, E, rowsAligned(dy, lddy, E) && rowsAligned(x, ldx, E) && rowsAligned(dx, lddx, E), false);
  const int blocks = normBlocks(rows, s);
  const size_t need = weights ? size_t(mostBlocks(rows, (int)cols)) * 2 * cols * sizeof(float) : 0;  // what the query says
  if (weights && (!goodVector(workspace, 16) || workspaceBytes < need)) return vrcclInvalidArgument;
  const Span spanDy = matrixSpan(dy, lddy, rows, cols, E), spanX = matrixSpan(x, ldx, rows, cols, E);
  const Span other[] = {vectorSpan(dgamma, cols * PE), vectorSpan(dbeta, cols * PE), vectorSpan(workspace, need)};
  const Span all[] = {matrixSpan(dx, lddx, rows, cols, E), other[0], other[1], other[2]};
  const Span in[] = {vectorSpan(gamma, cols * PE), vectorSpan(mean, rows * 4), vectorSpan(rstd, rows * 4),
                     unlessInPlace(spanDy, lddy, dx, lddx), unlessInPlace(spanX, ldx, dx, lddx)};
  const Span matrices[] = {spanDy, spanX};
  if (!apart(all, in) || !apart(other, matrices)) return vrcclInvalidArgument;
  NormArgs a = {};
  a.x = x;
  a.dy = dy;
  a.gamma = gamma;
  a.y = dx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.partial = weights ? static_cast<float*>(workspace) : nullptr;
  a.ldx = ldx;
  a.cutX = cutRows(ldx, E);
  a.lddy = lddy;
  a.cutDy = cutRows(lddy, E);
  a.ldy = lddx;
  a.rows = rows;
  a.cols = (int)cols;
  a.ptype = paramType;
  a.wideParams = ((uintptr_t)gamma & 15) == 0;
  if (s.walk == kLongRow && weights) {
    const dim3 grid((unsigned)((cols + 255) / 256), (unsigned)blocks);
    const NormFn columns = dtype == vrcclFloat32    ? normColumns<vrcclFloat32>
                           : dtype == vrcclBfloat16 ? normColumns<vrcclBfloat16>
                                                    : normColumns<vrcclFloat16>;
    const vrcclResult_t r = launchShaped(columns, {grid, 256, 0, 0, false}, st, a);
    if (r != vrcclSuccess) return r;
  }
  const vrcclResult_t r = launchNorm<false>(dtype, s, (unsigned)blocks, a, st);
  if (r != vrcclSuccess) return r;
  if (weights)
    return launchShaped(normJoin, {dim3((unsigned)((cols + 31) / 32), 2), 1024, 0, 0, true}, st,
                        static_cast<const float*>(workspace), blocks, (int)cols, dgamma, dbeta, (int)paramType);
  return vrcclSuccess;
}

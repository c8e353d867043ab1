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
// 16-byte blocks that it touches, and a thread shifts its chunk out of two
// neighbouring blocks). The barrier inside a row's reduction is also the point
// where every thread has taken its chunks, and the row's stage is filled anew
// (or, where registers do not hold the row, the stage of the one before it).
// Teams of warps walk rows of their own, so that one team's reduction runs
// under the others' loads and stores. On rows that do not start on 16-byte
// boundaries a warp takes 31 chunks and looks at the next one (ops_chunks.h).
//
// The weight's gradient is summed down the columns in the registers of the
// threads that own them, over all the rows that a team walks; a block joins its
// teams and writes one row of partial sums, and a second kernel adds those in
// order. No atomics: the same call gives the same bits.
//
// Short rows that start on boundaries go several to a warp (narrow); rows beyond
// a block's threads or shared memory are read twice, the second time through L2
// (long): 2048 x 16384 fp32 backward 142 us.
#include <cfloat>

#include "ops_chunks.cuh"
#include "ops_ring.cuh"

namespace vrccl {
namespace {

// Rows that a kernel reads.
struct Source {
  const char* p;
  size_t ld;
  unsigned cut;  // cutRows
};
struct RmsArgs {
  Source src[3];  // forward: x, residual; backward: s, dy, dsum
  const void* gamma;
  char* y;    // forward: y; backward: dx
  char* sum;  // forward: s
  unsigned char* codes;
  float* scales;
  float* rstd;
  float* partial;  // [blocks][cols], NULL: no weight gradient
  size_t ldy, lds, ldc, ldsc, rows;
  int cols, chunks, ptype;
  bool wideParams;  // gamma starts on a 16-byte boundary
  bool aligned;     // every source's rows are whole 16-byte blocks
  int stages, teams, threads, slot;
  int step;  // chunks of its own that a warp takes
  int quant, group;  // group: columns of a scale (then step is 32), 0 for the row
  float eps;
};

constexpr int kHeld = 2;  // chunks a thread holds
// Warps of a block (one an SM), and so the registers of a thread: what is left of 65536, in steps of four warps. Measured
// with 32768 x 4096 bf16 and residual: 16 warps 175 us, 20: 179, 24: 170, 28: 175, 32: 182; 16384 x 5120 to e4m3 20: 118.5,
// 24: 120, 28: 140, 32: 117; 16384 x 4097 (three teams of nine from 27 on) 20: 136, 24: 142, 28: 118, 32: 132. Rows that
// need more warps have 32 (wide).
constexpr int forwardWarps(bool vec, bool q, bool wide) { return wide || q ? 32 : vec ? 24 : 28; }
// Backward keeps a row's chunks in registers (hold) where 16 warps do: 16384 x 8192 bf16 159 us (20 warps: 205). Else it reads
// them from the stage once more: 16384 x 4097 20 warps 178 us (16 and held: 246, 24: 222, 28: 201), 4096 x 16384 with 32: 110.
constexpr int backwardWarps(bool vec, bool hold) { return hold ? 16 : vec ? 32 : 20; }
constexpr int kMaxTeams = 15;  // (as many named barriers, and the block's)
constexpr int kRingSmem = 208 * 1024;  // of the 227 KB a block may have

template <int DT>
__device__ __forceinline__ void gammaOf(const RmsArgs& a, int ci, F2 (&g)[kChunk / 2]) {
  float f[kChunk];
  const int left = a.cols - ci * kChunk;
  if (left >= kChunk) {
    loadParams<kChunk>(a.gamma, a.ptype, a.wideParams, ci * kChunk, 1.f, f);
  } else {
#pragma unroll
    for (int e = 0; e < kChunk; ++e) f[e] = e >= left ? 0.f : a.gamma ? loadParam(a.gamma, a.ptype, ci * kChunk + e) : 1.f;
  }
#pragma unroll
  for (int i = 0; i < kChunk / 2; ++i) g[i] = pair(f[2 * i], f[2 * i + 1]);
}
template <int DT>
__device__ __forceinline__ void pairsOf(const Chunk<DT>& c, F2 (&x)[kChunk / 2]) {
  float f[kChunk];
  c.expand(f);
#pragma unroll
  for (int i = 0; i < kChunk / 2; ++i) x[i] = pair(f[2 * i], f[2 * i + 1]);
}
template <int DT>
__device__ __forceinline__ Chunk<DT> packed(const F2 (&x)[kChunk / 2]) {
  float f[kChunk];
#pragma unroll
  for (int i = 0; i < kChunk / 2; ++i) {
    const float2 p = split(x[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
  Chunk<DT> c;
  c.pack(f);
  return c;
}
__device__ __forceinline__ float sumOf(F2 a) {
  const float2 p = split(a);
  return p.x + p.y;
}
template <int DT>
__device__ __forceinline__ void addTo(Chunk<DT>& x, const Chunk<DT>& r) {  // rounded to the type
#pragma unroll
  for (int i = 0; i < Chunk<DT>::NW; ++i) x.w[i] = combineWord<DT, vrcclSum>(x.w[i], r.w[i]);
}
// The largest |a| of a chunk's pairs, NaN if one is.
__device__ __forceinline__ float largest(const F2 (&x)[kChunk / 2]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kChunk / 2; ++i) {
    const float2 p = split(x[i]);
    m = maxOrNan(m, maxOrNan(fabsf(p.x), fabsf(p.y)));
  }
  return m;
}
template <int G>
__device__ __forceinline__ float largestOfLanes(float x) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) x = maxOrNan(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
template <int G>
__device__ __forceinline__ float sumOfLanes(float x) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// VEC: every operand's rows are whole chunks and start on 16-byte boundaries.
// Chunk j of a team's thread t (of `warps`); what the last lane of a warp holds beyond `step` is another warp's.
template <bool VEC>
__device__ __forceinline__ int chunkOf(const RmsArgs& a, int j, int warps, int t) {
  return VEC ? (j * warps * 32 + t) : (j * warps + (t >> 5)) * a.step + (t & 31);
}
template <bool VEC>
__device__ __forceinline__ bool ownChunk(const RmsArgs& a, int t) {
  return VEC || (t & 31) < a.step;
}
template <int DT, bool VEC>
__device__ __forceinline__ void putChunk(const RmsArgs& a, char* rows, size_t ld, size_t row, const Chunk<DT>& c, int ci) {
  char* p = rows + row * ld * Chunk<DT>::E + (size_t)ci * (kChunk * Chunk<DT>::E);
  if constexpr (VEC) {
    if (ci < a.chunks)
#pragma unroll
      for (int b = 0; b < Chunk<DT>::NB; ++b) __stcs(reinterpret_cast<uint4*>(p) + b, c.block(b));
  } else {
    const Place at = {(int)(threadIdx.x & 31), 32, ci, a.step};
    storeChunk<DT>(p, c, a.cols - ci * kChunk, at, innerChunks(row, a.rows, ci - at.lane, a.cols));
  }
}

// ------------------------------------------------------------ 8 bits
// The scale of a group whose largest |y| is given: no smaller than the least normal number, so that its reciprocal is
// finite (a group of zeros has that one); not finite where a y is not, so that it shows in whatever the codes stand for.
__device__ __forceinline__ float scaleOf(float most, int quant) {
  return maxOrNan(most * (quant == vrcclQuantInt8 ? 1.f / 127.f : 1.f / 448.f), FLT_MIN);
}
// Eight codes at p, `left` of them to the row's end.
__device__ __forceinline__ void storeCodes(unsigned char* p, const F2 (&y)[kChunk / 2], float scale, int quant, int left) {
  float inv;  // (a unit or two off, which moves a code where y lies that near the middle of two; normal, as the scale is below 2^122)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 a = split(y[2 * h]), b = split(y[2 * h + 1]);
    const float f[4] = {a.x * inv, a.y * inv, b.x * inv, b.y * inv};
    if (quant == vrcclQuantInt8) {
      w[h] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int q;
        asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(q) : "f"(f[e]));
        w[h] |= (uint32_t)(q & 0xff) << (8 * e);
      }
    } else {
      unsigned short lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[1]), "f"(f[0]));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[3]), "f"(f[2]));
      w[h] = lo | (uint32_t)hi << 16;
    }
  }
  if (left >= kChunk && (uintptr_t)p % 8 == 0) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
  } else {
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
      if (e < left) p[e] = (unsigned char)(w[e / 4] >> (8 * (e % 4)));
  }
}
// The codes of chunk ci and, by its first lane, the group's scale; `rowMost`: the row's largest |y|. Groups lie within a
// warp, one chunk a lane. All lanes call it.
__device__ __forceinline__ void storeGroup(const RmsArgs& a, size_t row, int ci, const F2 (&y)[kChunk / 2], float rowMost, bool own) {
  const int left = a.cols - ci * kChunk;
  float most = rowMost;
  if (a.group) {
    most = largest(y);
    most = maxOrNan(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = maxOrNan(most, __shfl_xor_sync(0xffffffffu, most, 2));
    if (a.group > 32) most = maxOrNan(most, __shfl_xor_sync(0xffffffffu, most, 4));
    if (a.group > 64) most = maxOrNan(most, __shfl_xor_sync(0xffffffffu, most, 8));
  }
  if (left <= 0 || !own) return;
  const float scale = scaleOf(most, a.quant);
  const int lanes = a.group / kChunk;
  if (a.group ? ci % lanes == 0 : ci == 0) a.scales[row * a.ldsc + (a.group ? ci / lanes : 0)] = scale;
  storeCodes(a.codes + row * a.ldc + (size_t)ci * kChunk, y, scale, a.quant, left);
}

// ------------------------------------------------------------ the ring of rows

// Thread 0 of a team: row `row` of N sources into a stage.
template <int E, int N>
__device__ __forceinline__ void fillStage(const RmsArgs& a, unsigned char* stage, size_t row, unsigned long long* bar,
                                          unsigned long long policy) {
  if (row >= a.rows) return;
  if (a.aligned) {
    const unsigned bytes = a.cols * E;
    expectBytes(bar, N * bytes);
#pragma unroll
    for (int n = 0; n < N; ++n) bulkLoadOnce(stage + n * a.slot, a.src[n].p + row * a.src[n].ld * E, bytes, bar, policy);
    return;
  }
  Window w[N];
  unsigned bytes = 0;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const Source& s = a.src[n];
    w[n] = rowWindow((uintptr_t)s.p, s.ld, row, a.rows, a.cols, E, s.cut);
    bytes += w[n].hi - w[n].lo;
    if (!maybeCut(row, a.rows, s.cut)) continue;
    // what a bulk copy may not take; this thread's arrival at the barrier makes it visible with the rest
    using S = std::conditional_t<E == 4, uint32_t, unsigned short>;
    S* v = reinterpret_cast<S*>(stage + n * a.slot + (w[n].row & 15));
    for (uintptr_t at = w[n].row; at < w[n].headEnd(); at += E) v[(at - w[n].row) / E] = *(const S*)at;
    for (uintptr_t at = w[n].tailBegin(); at < w[n].end; at += E) v[(at - w[n].row) / E] = *(const S*)at;
    fenceProxyAsync();  // a later row's copy into this slot comes after these writes
  }
  expectBytes(bar, bytes);
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (w[n].hi > w[n].lo)
      bulkLoadOnce(stage + n * a.slot + (w[n].lo - (w[n].row & ~(uintptr_t)15)), (const void*)w[n].lo, w[n].hi - w[n].lo, bar, policy);
}
// Chunk ci of source n's row in a stage; elements past the row's end zero.
template <int DT, bool VEC>
__device__ __forceinline__ Chunk<DT> taken(const RmsArgs& a, const unsigned char* stage, int n, size_t row, int ci) {
  using C = Chunk<DT>;
  constexpr int NB = C::NB;
  C c;
  const int left = a.cols - ci * kChunk;
  if (left <= 0) {
    c.clear();
    return c;
  }
  const uint4* b = reinterpret_cast<const uint4*>(stage + n * a.slot) + ci * NB;
  const unsigned skew = VEC ? 0 : ((unsigned)(uintptr_t)a.src[n].p + (unsigned)row * (unsigned)a.src[n].ld * C::E) & 15;
  if (skew == 0) {
#pragma unroll
    for (int i = 0; i < NB; ++i) c.set(i, b[i]);
  } else {
    uint32_t v[4 * NB + 4];
#pragma unroll
    for (int i = 0; i <= NB; ++i) {
      const uint4 q = b[i];
      v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
    }
    shiftedWords(v, skew, c.w);
  }
  if (!VEC) c.cut(left);
  return c;
}
__device__ __forceinline__ void teamSync(int team, int threads) {
  if (threads == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

// What forward and backward share: a team's place, its stages and their barriers. LATE: a row stays in its stage until the
// next one's barrier, which every thread reaches with the row's work done, and is then replaced.
template <int E, int N, bool LATE>
struct Ring {
  const RmsArgs& a;
  unsigned char* mine;
  unsigned long long* bar;
  int* dead;
  unsigned long long policy;
  int team, t, stage, round, turn;
  size_t stride, first;

  __device__ __forceinline__ Ring(const RmsArgs& a, unsigned char* smem, unsigned long long* full, int* deadWord)
      : a(a), policy(0), stage(0), round(0), turn(0) {
    team = threadIdx.x / a.threads;
    t = threadIdx.x - team * a.threads;
    mine = smem + (size_t)team * a.stages * N * a.slot;
    bar = full + team * kMaxStages;
    dead = deadWord + team;
    stride = (size_t)gridDim.x * a.teams;
    first = (size_t)blockIdx.x * a.teams + team;
    if (t == 0) {
      for (int s = 0; s < a.stages; ++s) mbarInit(&bar[s], 1);
      *dead = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      policy = evictFirstPolicy();
      for (int s = 0; s < a.stages; ++s) fill(s, first + s * stride);
    }
  }
  __device__ __forceinline__ void fill(int s, size_t row) {
    fillStage<E, N>(a, mine + (size_t)s * N * a.slot, row, &bar[s], policy);
  }
  __device__ __forceinline__ const unsigned char* wait() {
    waitRow(&bar[stage], round & 1, dead, turn);
    return mine + (size_t)stage * N * a.slot;
  }
  // The team's barrier of a turn, after which the stage takes a later row. true: a wait was given up, and the team leaves.
  __device__ __forceinline__ bool sync(size_t row) {
    teamSync(team, a.threads);
    // (before giving up is asked for, so that then every stage has been filled again)
    if (LATE && t == 0 && row >= first + stride) fill(stage ? stage - 1 : a.stages - 1, row - stride + a.stages * stride);
    if (givenUp(*reinterpret_cast<volatile int*>(dead), turn)) {
      abandon(bar, a.stages, stage, round, t == 0, dead, turn);
      return true;
    }
    if (!LATE && t == 0) fill(stage, row + a.stages * stride);
    return false;
  }
  __device__ __forceinline__ void next() {
    turn ^= 1;
    if (++stage == a.stages) {
      stage = 0;
      ++round;
    }
  }
};

template <int DT, bool RES, bool Q, bool VEC, bool WIDE>
__global__ void __launch_bounds__(32 * forwardWarps(VEC, Q, WIDE)) rmsForward(const __grid_constant__ RmsArgs a) {
  using C = Chunk<DT>;
  constexpr int E = C::E, NP = kChunk / 2;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ unsigned long long full[kMaxTeams * kMaxStages];
  __shared__ float2 red[2][32];  // turn, warp: (sum of squares, largest)
  __shared__ int deadWord[kMaxTeams];
  Ring<E, RES ? 2 : 1, false> ring(a, smem, full, deadWord);
  const int t = ring.t, T = a.threads, lane = t & 31, warps = T / 32;
  F2 g[kHeld][NP];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) gammaOf<DT>(a, chunkOf<VEC>(a, j, warps, t), g[j]);
  const float inv = 1.f / (float)a.cols;
  teamSync(ring.team, T);
  for (size_t row = ring.first; row < a.rows; row += ring.stride, ring.next()) {
    const unsigned char* stage = ring.wait();
    C s[kHeld];
    F2 squares = 0;
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int ci = chunkOf<VEC>(a, j, warps, t);
      s[j] = taken<DT, VEC>(a, stage, 0, row, ci);
      if constexpr (RES) addTo(s[j], taken<DT, VEC>(a, stage, 1, row, ci));
      F2 x[NP];
      pairsOf(s[j], x);
      if (ownChunk<VEC>(a, t))
#pragma unroll
        for (int i = 0; i < NP; ++i) squares = fma2(x[i], x[i], squares);
      if constexpr (Q) {
#pragma unroll
        for (int i = 0; i < NP; ++i) x[i] = mul2(x[i], g[j][i]);
        if (a.group == 0) most = maxOrNan(most, largest(x));
      }
      // (in place: the row is in shared memory)
      if (RES && a.sum) putChunk<DT, VEC>(a, a.sum, a.lds, row, s[j], ci);
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
      const int ci = chunkOf<VEC>(a, j, warps, t);
      F2 x[NP];
      pairsOf(s[j], x);
#pragma unroll
      for (int i = 0; i < NP; ++i) x[i] = mul2(mul2(x[i], scale), g[j][i]);
      if (!RES && a.sum) putChunk<DT, VEC>(a, a.sum, a.lds, row, s[j], ci);
      if (!Q || a.y) putChunk<DT, VEC>(a, a.y, a.ldy, row, packed<DT>(x), ci);
      if constexpr (Q) storeGroup(a, row, ci, x, w.y * rstd, ownChunk<VEC>(a, t));
    }
  }
}

// A thread's sums of its columns, laid out by column.
__device__ __forceinline__ void layOut(float* p, const F2 (&dg)[kChunk / 2], int ci, int cols) {
#pragma unroll
  for (int i = 0; i < kChunk / 2; ++i) {
    const float2 v = split(dg[i]);
    const int c = ci * kChunk + 2 * i;
    if (c < cols) p[c] = v.x;
    if (c + 1 < cols) p[c + 1] = v.y;
  }
}

template <int DT, bool DSUM, bool VEC, bool HOLD>
__global__ void __launch_bounds__(32 * backwardWarps(VEC, HOLD)) rmsBackward(const __grid_constant__ RmsArgs a) {
  using C = Chunk<DT>;
  constexpr int E = C::E, NP = kChunk / 2;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ unsigned long long full[kMaxTeams * kMaxStages];
  __shared__ float red[2][32];
  __shared__ int deadWord[kMaxTeams];
  Ring<E, DSUM ? 3 : 2, !HOLD> ring(a, smem, full, deadWord);
  const int t = ring.t, T = a.threads, lane = t & 31, warps = T / 32;
  F2 g[kHeld][NP], dg[kHeld][NP];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    gammaOf<DT>(a, chunkOf<VEC>(a, j, warps, t), g[j]);
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
      const int ci = chunkOf<VEC>(a, j, warps, t);
      C sj = taken<DT, VEC>(a, stage, 0, row, ci), dj = taken<DT, VEC>(a, stage, 1, row, ci);
      if constexpr (HOLD) {
        s[j] = sj, d[j] = dj;
        if constexpr (DSUM) r[j] = taken<DT, VEC>(a, stage, 2, row, ci);
      }
      if (!ownChunk<VEC>(a, t)) continue;
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
      const int ci = chunkOf<VEC>(a, j, warps, t);
      F2 xh[NP], dy[NP], add[NP];
      pairsOf(HOLD ? s[j] : taken<DT, VEC>(a, stage, 0, row, ci), xh);
      pairsOf(HOLD ? d[j] : taken<DT, VEC>(a, stage, 1, row, ci), dy);
      if constexpr (DSUM) pairsOf(HOLD ? r[j] : taken<DT, VEC>(a, stage, 2, row, ci), add);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const F2 v = fma2(mul2(xh[i], scale), minus, mul2(dy[i], g[j][i]));
        dy[i] = DSUM ? fma2(v, scale, add[i]) : mul2(v, scale);
      }
      putChunk<DT, VEC>(a, a.y, a.ldy, row, packed<DT>(dy), ci);
    }
  }
  if (!a.partial) return;
  // the teams own the same columns: every team lays its sums out, and the block adds them in the teams' order
  float* sum = reinterpret_cast<float*>(smem);
  __syncthreads();  // no team reads its ring any more
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    if (ownChunk<VEC>(a, t)) layOut(sum + (size_t)ring.team * a.cols, dg[j], chunkOf<VEC>(a, j, warps, t), a.cols);
  __syncthreads();
  float* p = a.partial + (size_t)blockIdx.x * a.cols;
  for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
    float x = sum[c];
    for (int w = 1; w < a.teams; ++w) x += sum[(size_t)w * a.cols + c];
    p[c] = x;
  }
}

// ------------------------------------------------------------ narrow rows
// Rows of at most 16 whole chunks on 16-byte boundaries (heads, and their
// like): G lanes a row, 32 / G rows a warp at a time and kNarrowTurn such steps
// in flight. Such rows reduce within a warp; there is nothing to wait for.
constexpr int kNarrowTurn = 4, kNarrowThreads = 256, kNarrowCols = 16 * kChunk;

template <int DT>
__device__ __forceinline__ Chunk<DT> narrowChunk(const Source& s, size_t row, int own, bool there) {
  Chunk<DT> c;
  c.clear();
  if (there) {
    const uint4* p = reinterpret_cast<const uint4*>(s.p + row * s.ld * Chunk<DT>::E) + own * Chunk<DT>::NB;
#pragma unroll
    for (int b = 0; b < Chunk<DT>::NB; ++b) c.set(b, __ldcs(p + b));
  }
  return c;
}
template <int DT>
__device__ __forceinline__ void storeNarrow(char* rows, size_t row, size_t ld, int own, const Chunk<DT>& c) {
  uint4* p = reinterpret_cast<uint4*>(rows + row * ld * Chunk<DT>::E) + own * Chunk<DT>::NB;
#pragma unroll
  for (int b = 0; b < Chunk<DT>::NB; ++b) __stcs(p + b, c.block(b));
}

template <int DT, int G, bool RES, bool Q>
__global__ void __launch_bounds__(kNarrowThreads) rmsForwardNarrow(const __grid_constant__ RmsArgs a) {
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
          storeCodes(a.codes + row * a.ldc + own * kChunk, x, q, a.quant, kChunk);
        }
      }
    }
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

// ------------------------------------------------------------ long rows
// A block a row, chunks of the row in turn, twice: once for the sums, once more
// (from L2) for what is written.
constexpr int kLongThreads = 1024;
constexpr int kLongHeld = kLongThreads * kHeld * kChunk;  // columns whose sums a block's threads hold

template <int DT>
__device__ __forceinline__ Chunk<DT> longChunk(const RmsArgs& a, int n, size_t row, int ci) {
  constexpr int E = Chunk<DT>::E;
  const Source& s = a.src[n];
  return loadChunk<DT>(s.p + (row * s.ld + (size_t)ci * kChunk) * E, a.cols - ci * kChunk, (uintptr_t)s.p,
                       (uintptr_t)s.p + ((a.rows - 1) * s.ld + a.cols) * E, threadIdx.x & 31, 32, innerChunks(row, a.rows, ci - (threadIdx.x & 31), a.cols));
}

template <int DT, bool RES, bool Q>
__global__ void __launch_bounds__(kLongThreads) rmsForwardLong(const __grid_constant__ RmsArgs a) {
  using C = Chunk<DT>;
  constexpr int E = C::E, NP = kChunk / 2;
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
      if (a.sum) putChunk<DT, false>(a, a.sum, a.lds, row, s, ci);
      if (!Q || a.y) putChunk<DT, false>(a, a.y, a.ldy, row, packed<DT>(x), ci);
      if constexpr (Q) storeGroup(a, row, ci, x, w.y * rstd, true);
    }
  }
}

// HOLD: the columns' sums in registers, for rows of up to kLongHeld; else rmsColumns makes them first.
template <int DT, bool DSUM, bool HOLD>
__global__ void __launch_bounds__(kLongThreads) rmsBackwardLong(const __grid_constant__ RmsArgs a) {
  using C = Chunk<DT>;
  constexpr int E = C::E, NP = kChunk / 2;
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
      putChunk<DT, false>(a, a.y, a.ldy, row, packed<DT>(dy), ci);
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

// ------------------------------------------------------------ host

enum Walk { kNarrow, kRing, kLong };
struct Shape {
  Walk walk;
  bool vec;
  int lanes;    // narrow: of a row
  int threads;  // of a team (narrow, long: of a block)
  int teams;    // of a block; narrow: the rows it takes at a time
  int step;     // chunks of its own that a warp takes
  bool wide, hold;  // ring: variants
  int stages, smem, resident;
};
// `sources`: matrices a row is read from; `aligned`: all rows of all operands start on 16-byte boundaries; `grouped`: scales
// of groups of columns, which lie in a warp as they do in the row.
Shape rmsShape(size_t rows, int cols, int elem, int sources, bool aligned, bool forward, bool quantized, bool grouped) {
  Shape s = {};
  const int chunks = (cols + kChunk - 1) / kChunk;
  s.vec = aligned && cols % kChunk == 0;
  s.step = s.vec || grouped ? 32 : 31;
  const int warps = (chunks + kHeld * s.step - 1) / (kHeld * s.step);
  s.wide = forward && !quantized && warps > forwardWarps(s.vec, false, false);
  s.hold = s.vec && warps <= backwardWarps(true, true);
  const int most = forward ? forwardWarps(s.vec, quantized, s.wide) : backwardWarps(s.vec, s.hold);
  const int row = (chunks * (kChunk * elem / 16) + 1) * 16 * sources;
  const int least = forward || s.hold ? 1 : 2;  // stages
  if (s.vec && cols <= kNarrowCols) {
    s.walk = kNarrow;
    s.lanes = chunks <= 4 ? 4 : chunks <= 8 ? 8 : 16;
    s.threads = kNarrowThreads;
    s.teams = kNarrowThreads / s.lanes * kNarrowTurn;
    s.resident = 4;
  } else if (warps <= most && row * least <= kRingSmem) {
    s.walk = kRing;
    s.threads = warps * 32;
    // a block an SM: as many teams as its warps make and as have a row, with no more stages than a team has rows
    s.resident = 1;
    s.teams = std::min(std::min(kMaxTeams, most / warps), kRingSmem / (row * least));
    s.teams = (int)std::min<size_t>(s.teams, (rows + smCount() - 1) / smCount());
    const size_t all = (size_t)smCount() * s.teams, turns = (rows + all - 1) / all;
    s.stages = (int)std::min<size_t>(std::min(kMaxStages, kRingSmem / (s.teams * row)), std::max<size_t>(turns, least));
    s.smem = std::max(s.teams * s.stages * row, forward ? 0 : s.teams * cols * 4);
  } else {
    s.walk = kLong;
    s.step = 32;
    s.threads = kLongThreads;
    s.teams = 1;
    s.resident = 2;
  }
  return s;
}
int rmsBlocks(size_t rows, const Shape& s) {
  return (int)std::min<size_t>((rows + s.teams - 1) / s.teams, (size_t)smCount() * s.resident);
}
// Row blocks of the partial sums, whatever the strides and the type of a call.
int mostBlocks(size_t rows, int cols) {
  int most = 0;
  for (int elem : {2, 4})
    for (int sources : {2, 3})
      for (bool aligned : {false, true}) most = std::max(most, rmsBlocks(rows, rmsShape(rows, cols, elem, sources, aligned, false, false, false)));
  return most;
}

using RmsFn = void (*)(RmsArgs);
template <int DT, bool RES, bool Q>
RmsFn pickForward(const Shape& s) {
  if (s.walk == kRing) {
    if constexpr (!Q)
      if (s.wide) return s.vec ? rmsForward<DT, RES, Q, true, true> : rmsForward<DT, RES, Q, false, true>;
    return s.vec ? rmsForward<DT, RES, Q, true, false> : rmsForward<DT, RES, Q, false, false>;
  }
  if (s.walk == kLong) return rmsForwardLong<DT, RES, Q>;
  return s.lanes == 4 ? rmsForwardNarrow<DT, 4, RES, Q> : s.lanes == 8 ? rmsForwardNarrow<DT, 8, RES, Q> : rmsForwardNarrow<DT, 16, RES, Q>;
}
template <int DT, bool DSUM>
RmsFn pickBackward(const Shape& s, int cols) {
  if (s.walk == kRing)
    return s.hold ? rmsBackward<DT, DSUM, true, true> : s.vec ? rmsBackward<DT, DSUM, true, false> : rmsBackward<DT, DSUM, false, false>;
  if (s.walk == kLong) return cols <= kLongHeld ? rmsBackwardLong<DT, DSUM, true> : rmsBackwardLong<DT, DSUM, false>;
  return s.lanes == 4 ? rmsBackwardNarrow<DT, 4, DSUM> : s.lanes == 8 ? rmsBackwardNarrow<DT, 8, DSUM> : rmsBackwardNarrow<DT, 16, DSUM>;
}
template <typename Fn>
auto forType(int dtype, Fn fn) {
  return dtype == vrcclFloat32    ? fn(std::integral_constant<int, vrcclFloat32>{})
         : dtype == vrcclBfloat16 ? fn(std::integral_constant<int, vrcclBfloat16>{})
                                  : fn(std::integral_constant<int, vrcclFloat16>{});
}
vrcclResult_t launchRms(RmsFn fn, const Shape& s, unsigned blocks, RmsArgs& a, int elem, cudaStream_t st) {
  if (s.smem > 32 * 1024) {  // (beside static shared memory, 48 KB come without asking)
    const vrcclResult_t r = allowSharedMemory((const void*)fn);
    if (r != vrcclSuccess) return r;
  }
  a.stages = s.stages;
  a.teams = s.teams;
  a.threads = s.threads;
  a.step = s.step;
  a.slot = (a.chunks * (kChunk * elem / 16) + 1) * 16;
  const int threads = s.walk == kRing ? s.threads * s.teams : s.threads;
  return launchShaped(fn, {dim3(blocks), threads, s.smem, 0, false}, st, a);
}

bool goodSizes(size_t rows, size_t cols, int dtype, int ptype) {
  return rows < kMaxExtent && cols < (size_t(1) << 31) - 65536 && isOperatorType(dtype) && isOperatorType(ptype);
}
Source sourceOf(const void* p, size_t ld, int elem) {
  return {static_cast<const char*>(p), ld, p ? cutRows(ld, elem) : 0};
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
  const bool aligned = rowsAligned(x, ldx, E) && (!residual || rowsAligned(residual, ldr, E)) && (!sum || rowsAligned(sum, lds, E)) &&
                       (!y || rowsAligned(y, ldy, E));
  const Shape s = rmsShape(rows, (int)cols, E, residual ? 2 : 1, aligned, true, codes, codes && group);
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

extern "C" vrcclResult_t vrcclRmsNormWorkspace(size_t rows, size_t cols, size_t* bytes) {
  if (!bytes || !goodSizes(rows, cols, vrcclFloat32, vrcclFloat32)) return vrcclInvalidArgument;
  *bytes = size_t(mostBlocks(rows, (int)cols)) * cols * sizeof(float);
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
  const Shape shape = rmsShape(rows, (int)cols, E, dsum ? 3 : 2, sources && rowsAligned(dx, lddx, E), false, false, false);
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

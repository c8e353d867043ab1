// RMS norm: what its two directions share. (ops_rmsnorm.cu says how rows are walked.)
#pragma once

#include <algorithm>
#include <cfloat>
#include <initializer_list>

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
// How the rows of a call's matrices lie: whole chunks on 16-byte boundaries; each number of row on the same skew in all of
// them; anyhow.
enum Lie { kWhole, kSame, kAny };
// Warps of a block (one an SM), and so the registers of a thread: what is left of 65536, in steps of four warps. Forward:
// 32768 x 4096 bf16 with residual 16 warps 175 us, 20: 179, 24: 170, 28: 175, 32: 182; 16384 x 4097 20: 88, 24: 93, 28: 97, 32:
// 104, and 65536 x 1025 83, 74, 92, 94; anyhow (three teams of nine from 27 on) 20: 136, 24: 142, 28: 118, 32: 132; 16384 x 5120
// to e4m3 20: 100, 24: 100, 28: 135, 32: 110, and x 4096 91, 76, 94, 86. Rows that need more warps have 32 (wide).
constexpr int forwardWarps(Lie lie, bool wide) { return wide ? 32 : lie == kAny ? 28 : 24; }
// Backward keeps a row's chunks in registers (hold) where 16 warps do and teams of them leave few idle: 16384 x 8192 bf16
// 159 us (20 warps: 205), 20000 x 2500 fp32 141 (not held 169). Else it reads them from the stage once more: 16384 x 5120 20
// warps 104 us (held 118), 16384 x 4097 20: 133, 24: 147, 28: 132, held 192; 8192 x 9001 20: 135, 24: 147, 28: 170. Rows that need
// more warps have 32 (wide): 4096 x 16384 110 us, read twice 200.
constexpr int backwardWarps(bool hold, bool wide) { return hold ? 16 : wide ? 32 : 20; }
constexpr int kMaxTeams = 15;  // (as many named barriers, and the block's)
constexpr int kRingSmem = 208 * 1024;  // of the 227 KB a block may have
// Bytes of a row of `chunks` in a stage: one block more where it starts within one, a chunk more where chunks start on blocks.
constexpr int slotOf(Lie lie, int chunks, int elem) { return ((chunks + (lie == kSame)) * (kChunk * elem / 16) + (lie != kSame)) * 16; }

// Gamma of chunk ci of rows that begin `shift` columns into their first chunk; 0 beside the row.
template <int DT>
__device__ __forceinline__ void gammaOf(const RmsArgs& a, int ci, F2 (&g)[kChunk / 2], int shift = 0) {
  float f[kChunk];
  const int first = ci * kChunk - shift;
  if (shift == 0 && first + kChunk <= a.cols) {
    loadParams<kChunk>(a.gamma, a.ptype, a.wideParams, first, 1.f, f);
  } else {
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
      f[e] = (unsigned)(first + e) >= (unsigned)a.cols ? 0.f : a.gamma ? loadParam(a.gamma, a.ptype, first + e) : 1.f;
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

// Chunk j of a team's thread t (of `warps`). kAny: what the last lane of a warp holds beyond `step` is another warp's.
template <Lie LIE>
__device__ __forceinline__ int chunkOf(const RmsArgs& a, int j, int warps, int t) {
  return LIE != kAny ? (j * warps * 32 + t) : (j * warps + (t >> 5)) * a.step + (t & 31);
}
template <Lie LIE>
__device__ __forceinline__ bool ownChunk(const RmsArgs& a, int t) {
  return LIE != kAny || (t & 31) < a.step;
}
// kSame: a row begins `shift` columns into its first chunk, which starts on a 16-byte boundary in every matrix.
template <int DT, Lie LIE>
__device__ __forceinline__ void putChunk(const RmsArgs& a, char* rows, size_t ld, size_t row, const Chunk<DT>& c, int ci, int shift) {
  constexpr int E = Chunk<DT>::E, NB = Chunk<DT>::NB;
  char* p = rows + row * ld * E + ((ptrdiff_t)ci * kChunk - shift) * E;
  if constexpr (LIE == kAny) {
    const Place at = {(int)(threadIdx.x & 31), 32, ci, a.step};
    storeChunk<DT>(p, c, a.cols - ci * kChunk, at, innerChunks(row, a.rows, ci - at.lane, a.cols));
  } else if (LIE == kWhole) {
    if (ci < a.chunks)
#pragma unroll
      for (int b = 0; b < NB; ++b) __stcs(reinterpret_cast<uint4*>(p) + b, c.block(b));
  } else {
    storeElements<DT>(p, c, shift - ci * kChunk, a.cols + shift - ci * kChunk);
  }
}

// ------------------------------------------------------------ 8 bits
// The scale of a group whose largest |y| is given: no smaller than the least normal number, so that its reciprocal is
// finite (a group of zeros has that one); not finite where a y is not, so that it shows in whatever the codes stand for.
__device__ __forceinline__ float scaleOf(float most, int quant) {
  return maxOrNan(most * (quant == vrcclQuantInt8 ? 1.f / 127.f : 1.f / 448.f), FLT_MIN);
}
// a / b rounded once, from 1 / b rounded once: the product's remainder is exact, and what it adds decides the last bit (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990). Where the remainder falls below binary32's
// range (b near its least normal number) the last bit may be another. NaN for b infinite or a NaN.
__device__ __forceinline__ F2 quotient2(F2 a, F2 minusB, F2 inv) {
  const F2 q = mul2(a, inv);
  return fma2(fma2(minusB, q, a), inv, q);
}
// Those of eight codes at p from number `from` on and before number `to`: y / scale rounded to binary32, then to a code. (By the
// product with an approximate reciprocal nearly twice as many int8 codes of 16384 x 5120 bf16 lay on the other side of a middle
// between two as by the division, 105 in a million for 61, in 96 us for 102; e4m3 96 for 100.)
__device__ __forceinline__ void storeCodes(unsigned char* p, const F2 (&y)[kChunk / 2], float scale, int quant, int from, int to) {
  float inv;  // within a unit, and rounded once after a step of Newton's (the scale is below 2^122: all of it is normal)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
  inv = fmaf(fmaf(-scale, inv, 1.f), inv, inv);
  const F2 inv2 = pair(inv, inv), minus = pair(-scale, -scale);
  uint32_t w[2];
  if (quant == vrcclQuantInt8) {
    // 1.5 2^23 + q has q, rounded to the nearest (even), in its lowest bits; codes of a scale that is not finite are 0
    const F2 round = pair(12582912.f, 12582912.f);
    const bool finite = scale < INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 a = split(add2(quotient2(y[2 * h], minus, inv2), round)), b = split(add2(quotient2(y[2 * h + 1], minus, inv2), round));
      const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040), hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
      w[h] = finite ? __byte_perm(lo, hi, 0x5410) : 0;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 a = split(quotient2(y[2 * h], minus, inv2)), b = split(quotient2(y[2 * h + 1], minus, inv2));
      unsigned short lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
      w[h] = lo | (uint32_t)hi << 16;
    }
  }
  if (from <= 0 && to >= kChunk && (uintptr_t)p % 8 == 0) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
  } else {
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
      if (e >= from && e < to) p[e] = (unsigned char)(w[e / 4] >> (8 * (e % 4)));
  }
}
// The codes of chunk ci and, by its first lane, the group's scale; `rowMost`: the row's largest |y|. Groups lie within a
// warp, one chunk a lane. All lanes call it.
__device__ __forceinline__ void storeGroup(const RmsArgs& a, size_t row, int ci, const F2 (&y)[kChunk / 2], float rowMost, bool own, int shift = 0) {
  const int left = a.cols + shift - ci * kChunk;
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
  const int shares = a.group == 32 ? 2 : a.group == 64 ? 3 : a.group == 128 ? 4 : 31;  // 2^that lanes have one scale
  if ((ci & ((1u << shares) - 1)) == 0) a.scales[row * a.ldsc + (ci >> shares)] = scale;
  storeCodes(a.codes + row * a.ldc + (ptrdiff_t)ci * kChunk - shift, y, scale, a.quant, shift - ci * kChunk, left);
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
// Chunk ci of source n's row in a stage; elements beside the row zero.
template <int DT, Lie LIE>
__device__ __forceinline__ Chunk<DT> taken(const RmsArgs& a, const unsigned char* stage, int n, size_t row, int ci, int shift) {
  using C = Chunk<DT>;
  constexpr int NB = C::NB;
  C c;
  const int left = a.cols + shift - ci * kChunk;
  if (left <= 0) {
    c.clear();
    return c;
  }
  const uint4* b = reinterpret_cast<const uint4*>(stage + n * a.slot) + ci * NB;
  const unsigned skew = LIE != kAny ? 0 : ((unsigned)(uintptr_t)a.src[n].p + (unsigned)row * (unsigned)a.src[n].ld * C::E) & 15;
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
  if (LIE != kWhole) c.cut(left);
  if (LIE == kSame && ci * kChunk < shift) c.cutHead(shift);
  return c;
}
__device__ __forceinline__ void teamSync(int team, int threads) {
  if (threads == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

// kSame: how many columns into its first chunk each of a team's rows begins.
template <int DT, Lie LIE>
__device__ __forceinline__ int shiftOf(const RmsArgs& a, size_t first) {
  constexpr int E = Chunk<DT>::E;
  return LIE == kSame ? (int)(((unsigned)(uintptr_t)a.src[0].p + (unsigned)first * (unsigned)a.src[0].ld * E) & 15) / E : 0;
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

// A thread's sums of its columns, laid out by column.
__device__ __forceinline__ void layOut(float* p, const F2 (&dg)[kChunk / 2], int ci, int cols, int shift = 0) {
#pragma unroll
  for (int i = 0; i < kChunk / 2; ++i) {
    const float2 v = split(dg[i]);
    const int c = ci * kChunk + 2 * i - shift;
    if ((unsigned)c < (unsigned)cols) p[c] = v.x;
    if ((unsigned)(c + 1) < (unsigned)cols) p[c + 1] = v.y;
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

// ------------------------------------------------------------ host

enum Walk { kNarrow, kRing, kLong };
struct Shape {
  Walk walk;
  Lie lie;
  int lanes;    // narrow: of a row
  int threads;  // of a team (narrow, long: of a block)
  int teams;    // of a block; narrow: the rows it takes at a time
  int step;     // chunks of its own that a warp takes
  bool wide, hold;  // ring: variants
  int stages, smem, resident;
};
// `sources`: matrices a row is read from; `grouped`: scales of groups of columns, which lie in a warp as they do in the row.
inline Shape rmsShape(size_t rows, int cols, int elem, int sources, Lie lie, bool forward, bool grouped) {
  Shape s = {};
  const int E16 = 16 / elem;
  // a row's skew comes again E16 rows on, if not before: a team's step is a multiple of that, or it takes one row
  if (lie == kSame && (grouped || smCount() % E16)) lie = kAny;
  s.lie = lie;
  s.step = lie != kAny || grouped ? 32 : 31;
  const int chunks = (cols + kChunk - 1) / kChunk, most = (cols + (lie == kSame ? E16 - 1 : 0) + kChunk - 1) / kChunk;
  const int warps = (most + kHeld * s.step - 1) / (kHeld * s.step);
  s.hold = !forward && lie != kAny && warps <= 16 && 16 / warps * warps >= 12;
  s.wide = forward ? warps > forwardWarps(lie, false) : !s.hold && lie != kAny && warps > backwardWarps(false, false);
  const int room = forward ? forwardWarps(lie, s.wide) : backwardWarps(s.hold, s.wide);
  const int row = slotOf(lie, chunks, elem) * sources;
  const int least = forward || s.hold ? 1 : 2;  // stages
  if (lie == kWhole && cols <= kNarrowCols) {
    s.walk = kNarrow;
    s.lanes = chunks <= 4 ? 4 : chunks <= 8 ? 8 : 16;
    s.threads = kNarrowThreads;
    s.teams = kNarrowThreads / s.lanes * kNarrowTurn;
    s.resident = 4;
  } else if (warps <= room && row * least <= kRingSmem) {
    s.walk = kRing;
    s.threads = warps * 32;
    // a block an SM: as many teams as its warps make and as have a row, with no more stages than a team has rows
    s.resident = 1;
    s.teams = std::min(std::min(kMaxTeams, room / warps), kRingSmem / (row * least));
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
inline int rmsBlocks(size_t rows, const Shape& s) {
  return (int)std::min<size_t>((rows + s.teams - 1) / s.teams, (size_t)smCount() * s.resident);
}
// Row blocks of the partial sums, whatever the strides and the type of a call.
inline int mostBlocks(size_t rows, int cols) {
  int most = 0;
  for (int elem : {2, 4})
    for (int sources : {2, 3})
      for (Lie lie : {kWhole, kSame, kAny}) most = std::max(most, rmsBlocks(rows, rmsShape(rows, cols, elem, sources, lie, false, false)));
  return most;
}

using RmsFn = void (*)(RmsArgs);
template <typename Fn>
auto forType(int dtype, Fn fn) {
  return dtype == vrcclFloat32    ? fn(std::integral_constant<int, vrcclFloat32>{})
         : dtype == vrcclBfloat16 ? fn(std::integral_constant<int, vrcclBfloat16>{})
                                  : fn(std::integral_constant<int, vrcclFloat16>{});
}
inline vrcclResult_t launchRms(RmsFn fn, const Shape& s, unsigned blocks, RmsArgs& a, int elem, cudaStream_t st) {
  if (s.smem > 32 * 1024) {  // (beside static shared memory, 48 KB come without asking)
    const vrcclResult_t r = allowSharedMemory((const void*)fn);
    if (r != vrcclSuccess) return r;
  }
  a.stages = s.stages;
  a.teams = s.teams;
  a.threads = s.threads;
  a.step = s.step;
  a.slot = slotOf(s.lie, a.chunks, elem);
  const int threads = s.walk == kRing ? s.threads * s.teams : s.threads;
  return launchShaped(fn, {dim3(blocks), threads, s.smem, 0, false}, st, a);
}

inline bool goodSizes(size_t rows, size_t cols, int dtype, int ptype) {
  return rows < kMaxExtent && cols < (size_t(1) << 31) - 65536 && isOperatorType(dtype) && isOperatorType(ptype);
}
inline Source sourceOf(const void* p, size_t ld, int elem) {
  return {static_cast<const char*>(p), ld, p ? cutRows(ld, elem) : 0};
}

// How a call's matrices lie together.
struct Matrix {
  const void* p;  // NULL: none
  size_t ld;
};
inline Lie lieOf(std::initializer_list<Matrix> all, size_t cols, int elem) {
  bool whole = cols % kChunk == 0, same = true;
  const Matrix& first = *all.begin();
  for (const Matrix& m : all) {
    if (!m.p) continue;
    whole &= rowsAligned(m.p, m.ld, elem);
    same &= sameSkew(m.p, m.ld, first.p, first.ld, elem);
  }
  return whole ? kWhole : same ? kSame : kAny;
}

}  // namespace
}  // namespace vrccl

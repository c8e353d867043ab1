// Linear layer: a matrix product with bias, activation and residual in its
// epilogue, and its gradients.
//
//   z = x W^T + b,  y = act(z) + r                   x [rows, ins], W [outs, ins]
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum over rows of dz
//
// All three products are D[M, N] = A B^T with a contraction of length K, run by
// one persistent tcgen05 kernel. An operand is "K-major" where the contraction
// runs along its rows in memory (x and W forward, dz in dx) and "MN-major"
// where it runs down its columns (W in dx, both operands of dW); the tensor
// cores read either from the same 128-byte-swizzled tiles, so no operand is
// ever transposed in memory.
//
// Warp roles of a block: one warp issues the TMA copies of slices of A and B
// into a ring of shared-memory stages, one issues the MMAs, eight read finished
// accumulators out of TMEM, apply the epilogue and store by TMA. TMEM holds two
// accumulators, so a tile's epilogue runs under the next one's products.
//
// Large products are bound by the tensor cores, and, a second into a run, by
// the 1400 W limit. Beside a library's plain product in the same state, normal
// inputs: 8192 cubed 583 us after a pause (1.89 PFLOP/s; the library 565), 662
// over seconds (636); 8192 x 8192 x 2048 with the bias 163 us after a pause
// (167), 167 over seconds (158), 175 with gelu-tanh, 181 where z is stored too
// (268 MB written in all); both gradients of 8192 x 4096 x 4096 337 us over seconds
// (335).
//
// A call with few rows (one token and its like) is bound by reading W once:
// linearFew streams W with wide loads, productSplit (below) feeds it to the
// tensor cores from all multiprocessors: 1, 2, 16 and 64 rows of 4096 x 4096
// in 7.2, 8.2, 9.6 and 10.6 us (33.5 MB, 5.0 us from memory; eight weights in
// turn, which L2 does not hold).
#include <cuda.h>

#include <atomic>
#include <cstring>
#include <utility>

#include "ops_common.cuh"

namespace vrccl {
namespace {

// ------------------------------------------------------------ activations

// Two values at a time (F2). What an epilogue or the pass over dy and z has to
// compute for an element shares its multiprocessor with loads, stores and
// MMAs; in pairs it takes half the instructions.
__device__ __forceinline__ F2 both(float x) { return pair(x, x); }
// 2^x on the special function unit, relative error about 2^-22; 2^inf = inf
__device__ __forceinline__ F2 exp2Pair(F2 x) {
  const float2 v = split(x);
  float a, b;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(v.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(v.y));
  return pair(a, b);
}
// 1 / x, relative error about 2^-23; 1 / inf = 0
__device__ __forceinline__ F2 reciprocal(F2 x) {
  const float2 v = split(x);
  float a, b;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(v.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(v.y));
  return pair(a, b);
}
constexpr float kLog2e = 1.4426950408889634f;

// Phi(z), the normal distribution, and exp(-z^2/2), which its slope needs too:
//   Phi(-x) = exp(-x^2/2) t P(t), t = 1 / (1 + 0.304 x), x = |z| >= 0,
// with P a polynomial through the scaled complementary error function
// exp(x^2/2) Phi(-x) / t on 0 <= x <= 13.3 (beyond, the density is below the
// normal numbers), fitted by least squares reweighted to an even relative
// error, 8.3e-8. The relative error stays small in the tail, where
// 1 + erf(z / sqrt(2)) cancels: with the arithmetic's own 6e-7 at z = -2 and
// 2e-6 at -6 (the density's argument is rounded), so that one rounding to 16
// bits is all that shows. It costs two special-function instructions and
// fifteen others where erff costs some forty, which made the gradient's pass
// over dy and z compute bound.
__device__ __forceinline__ F2 normalPhi(F2 z, F2& density) {
  const float2 v = split(z);
  const F2 x = pair(fabsf(v.x), fabsf(v.y));
  const F2 t = reciprocal(fma2(x, both(0.304f), both(1.f)));
  density = exp2Pair(mul2(mul2(z, z), both(-0.5f * kLog2e)));
  F2 p = fma2(t, both(0.0368631847f), both(-0.155317998f));
  p = fma2(t, p, both(0.192221078f));
  p = fma2(t, p, both(-0.0431591134f));
  p = fma2(t, p, both(0.123568846f));
  p = fma2(t, p, both(0.102417924f));
  p = fma2(t, p, both(0.122171489f));
  p = fma2(t, p, both(0.121234632f));
  const float2 tail = split(mul2(mul2(p, t), density));  // Phi(-|z|)
  return pair(v.x > 0.f ? 1.f - tail.x : tail.x, v.y > 0.f ? 1.f - tail.y : tail.y);
}
// 1 / (1 + exp(-w)) with w = 2 sqrt(2/pi) (z + 0.044715 z^3): (1 + tanh(w / 2)) / 2, which loses nothing where the tanh
// nears -1; w itself, and for silu w = z.
constexpr float kTanhScale = 1.5957691216057308f;
template <int ACT>
__device__ __forceinline__ F2 logisticOf(F2 z) {
  F2 w = mul2(z, both(-kLog2e));
  if constexpr (ACT == vrcclActGeluTanh)
    w = mul2(z, fma2(mul2(z, z), both(-kTanhScale * kLog2e * 0.044715f), both(-kTanhScale * kLog2e)));
  return reciprocal(add2(exp2Pair(w), both(1.f)));
}

template <int ACT>
__device__ __forceinline__ F2 activate(F2 z) {
  if constexpr (ACT == vrcclActRelu) {
    const float2 v = split(z);
    return pair(v.x > 0.f ? v.x : (v.x != v.x ? v.x : 0.f), v.y > 0.f ? v.y : (v.y != v.y ? v.y : 0.f));
  }
  if constexpr (ACT == vrcclActGelu) {
    F2 density;
    return mul2(z, normalPhi(z, density));
  }
  if constexpr (ACT == vrcclActGeluTanh || ACT == vrcclActSilu) return mul2(z, logisticOf<ACT>(z));
  return z;
}
template <int ACT>
__device__ __forceinline__ F2 slope(F2 z) {
  if constexpr (ACT == vrcclActRelu) {
    const float2 v = split(z);
    return pair(v.x > 0.f ? 1.f : 0.f, v.y > 0.f ? 1.f : 0.f);
  }
  if constexpr (ACT == vrcclActGelu) {
    F2 density;
    const F2 phi = normalPhi(z, density);
    return fma2(mul2(z, density), both(0.39894228040143268f), phi);
  }
  // y = z s(w): y' = s + z s (1 - s) w'
  if constexpr (ACT == vrcclActGeluTanh || ACT == vrcclActSilu) {
    const F2 s = logisticOf<ACT>(z);
    const F2 bell = mul2(mul2(s, fma2(s, both(-1.f), both(1.f))), z);  // exactly 0 long before z^2 is large
    if constexpr (ACT == vrcclActGeluTanh) {
      const float2 q = split(mul2(z, z));  // held below infinity, which bell's 0 would make NaN of
      const F2 zz = pair(fminf(q.x, 1e30f), fminf(q.y, 1e30f));
      return fma2(bell, fma2(zz, both(kTanhScale * 3.f * 0.044715f), both(kTanhScale)), s);
    }
    return add2(bell, s);
  }
  return both(1.f);
}
template <int ACT>
__device__ __forceinline__ float activate(float z) {
  return split(activate<ACT>(both(z))).x;
}

__device__ __forceinline__ float activateBy(int act, float z) {
  switch (act) {
    case vrcclActRelu: return activate<vrcclActRelu>(z);
    case vrcclActGelu: return activate<vrcclActGelu>(z);
    case vrcclActGeluTanh: return activate<vrcclActGeluTanh>(z);
    case vrcclActSilu: return activate<vrcclActSilu>(z);
  }
  return z;
}

// ------------------------------------------------------------ tcgen05, TMA

// A wait that has not come true after so many cycles (a second and more) never
// will: the kernel then records a timeout, drains what it has in flight and
// ends. (The cycle counter: reading the global timer costs as much as a copy.)
constexpr long long kWaitCycles = 3000000000ll, kDrainCycles = 200000000ll;

__device__ int gLinearStatus;  // vrcclResult_t of the first device-side failure

// false = gave up (this wait, or another one of the block)
__device__ __forceinline__ bool waitBar(unsigned long long* bar, unsigned parity, volatile int* dead,
                                        long long limit = kWaitCycles) {
  if (mbarTryWait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbarTryWait(bar, parity)) {
    if (*dead) return false;
    if (clock64() - t0 > limit) {
      *dead = 1;
      atomicCAS(&gLinearStatus, 0, (int)vrcclTimeout);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void mbarArriveExpect(unsigned long long* bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smemAddr(bar)), "r"(bytes) : "memory");
}
// One lane of a converged warp. The TMA and MMA warps run their loops whole, so
// that addresses and descriptors stay in uniform registers, and only the
// copies and MMAs themselves are one lane's: with the loop in a single lane's
// branch every MMA waited for its operands to be moved there, and a 64-deep
// step took 650 cycles whatever the tile.
__device__ __forceinline__ bool electOne() {
  uint32_t p;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t clusterRank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void clusterSync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this shared variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t inBlock(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smemAddr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbarArriveAt(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// `bar`: a shared::cluster address; in a pair of blocks it may be the other block's.
template <int CG>
__device__ __forceinline__ void tmaLoad2d(const CUtensorMap* map, void* dst, uint32_t bar, int x, int y) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4}], [%2];" ::"r"(smemAddr(dst)),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            smemAddr(dst)),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void tmaStore2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(smemAddr(src)), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void tcFenceBefore() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcFenceAfter() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Arrives on `bar` (in a pair: on both blocks') once the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void tcCommit(unsigned long long* bar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smemAddr(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smemAddr(bar))
                 : "memory");
}
template <int CG>
__device__ __forceinline__ void tcMma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void tmemAlloc(uint32_t* slot, int cols) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smemAddr(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smemAddr(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmemFree(uint32_t addr, int cols) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tcLoad32(uint32_t addr, float (&f)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]);
}

// Shared-memory operand descriptor of a tile with 128-byte swizzle. K-major:
// rows of 64 contraction elements (128 bytes), eight rows to a swizzle block,
// blocks 1024 bytes apart. MN-major: rows of 64 M (or N) elements, one row a
// contraction index; eight of them make a swizzle block (1024 bytes apart),
// and the next 64 M elements start a box of 64 x depth elements on.
__device__ __forceinline__ uint64_t operandDesc(uint32_t addr, bool mn, int depth) {
  uint64_t d = (addr >> 4) & 0x3fff;
  d |= (uint64_t)(mn ? depth * 128 >> 4 : 1) << 16;  // leading dimension
  d |= (uint64_t)(1024 >> 4) << 32;           // stride dimension
  d |= (uint64_t)1 << 46;                     // descriptor version
  d |= (uint64_t)2 << 61;                     // 128-byte swizzle
  return d;
}

// ------------------------------------------------------------ the product

constexpr int kBM = 128;  // rows of A a block
constexpr int kEpilogueWarps = 8;
constexpr int kProductThreads = 32 * (2 + kEpilogueWarps);  // TMA warp, MMA warp, epilogue warps
constexpr int kStoreBytes = 32 * 32 * 2;                    // one warp's 32 rows x 32 columns on the way out

struct Problem {
  CUtensorMap a, b, dMap, zMap;
  void* d;               // [M, N]
  void* z;               // the sums before activation, or NULL
  const void* bias;      // [N] or NULL
  const void* residual;  // [M, N] or NULL
  size_t ldd, ldz, ldr;
  int M, N, K;
  bool aMN, bMN;         // operand majors
  bool wideD, wideZ;     // d / z may be stored by TMA
  bool wideR;            // the residual's rows start on 16-byte boundaries
  int act;
  int tilesM, tilesN, tiles, steps;
};

// A launch computes one product or two (a linear layer's two gradients, which
// would each leave part of the GPU idle in its last round of tiles). The first
// one's tiles are dealt out in turn; unit u (a block, or a pair) then takes
// tiles from[u] to from[u + 1] of the second, so that all end together.
constexpr int kMaxUnits = 256;
struct ProductArgs {
  Problem p[2];
  unsigned short from[kMaxUnits + 1];
};

// A unit's tiles in order.
struct Walk {
  int which, tile, stride, end;
  __device__ __forceinline__ Walk(const ProductArgs& a, int unit, int units)
      : which(0), tile(unit), stride(units), end(a.p[0].tiles) {
    settle(a, unit);
  }
  __device__ __forceinline__ void settle(const ProductArgs& a, int unit) {
    if (which == 0 && tile >= end) {
      which = 1;
      tile = a.from[unit];
      end = a.from[unit + 1];
      stride = 1;
    }
  }
  __device__ __forceinline__ bool more() const { return tile < end; }
  // The tile's place: columns of GROUP tiles down, so that the tiles at work at a time make up a block of the result and
  // read few different rows of either operand.
  template <int GROUP>
  __device__ __forceinline__ void place(const Problem& a, int& m, int& n) const {
    const int column = GROUP * a.tilesN, group = tile / column, r = tile - group * column;
    const int down = min(GROUP, a.tilesM - group * GROUP);
    n = r / down;
    m = group * GROUP + r - n * down;
  }
  __device__ __forceinline__ void next(const ProductArgs& a, int unit) {
    tile += stride;
    settle(a, unit);
  }
};

// A tile is CG x 128 rows of A by BN rows of B. In a pair of blocks (CG = 2)
// each holds its 128 rows of A and half of B's, and one thread issues MMAs
// that run on both multiprocessors: B crosses into shared memory once for the
// two of them, which a single block's 128 x 256 tile cannot afford (its stages
// would take 1.5 times the L2 bandwidth for the same arithmetic).
template <int CG, int BN>
struct ProductShape {
  static constexpr int kBRows = BN / CG;
  // Contraction elements a stage. Waiting for a stage and signalling it free costs its MMA warp some 150 cycles: nothing
  // under the MMAs of the wider tiles (which gain more from many shallow stages than from two deep ones: 4096 cubed on
  // 128 x 128 tiles 107 us against 147), but as much again under a narrow one's.
  static constexpr int kBK = BN <= 64 ? 128 : 64;
  static constexpr int kStageBytes = (kBM + kBRows) * kBK * 2;
  static constexpr int kStages = BN == 64 ? 3 : 6;
  static constexpr int kSmem = kStages * kStageBytes + kEpilogueWarps * 2 * kStoreBytes + 1024;
  static constexpr int kTmemCols = BN == 192 ? 512 : 2 * BN;  // a power of two
  // Tiles of a column (Walk::place). Pairs, over seconds, 8 against 16: 8192 x 8192 x 2048 with gelu-tanh and z 187.3 and
  // 183.6 us, 4096 cubed 89.3 and 87.5, both gradients of 8192 x 4096 x 4096 with gelu 356.4 and 358.4.
  static constexpr int kGroup = CG == 2 ? 16 : 12;
};

// A warp's staging buffer: 32 rows of 64 bytes, their 16-byte pieces swizzled
// as a TMA map of 64-byte swizzle has them, so that lanes that each write or
// read a piece of their own row meet different banks.
__device__ __forceinline__ int pieceAt(int row, int piece) { return row * 64 + ((piece ^ (row >> 1 & 3)) << 4); }

// Writes one warp's finished 32 x 32 elements from its staging buffer to memory.
__device__ __forceinline__ void storeBox(const Problem& a, const CUtensorMap* map, void* out, size_t ld, bool wide,
                                         const unsigned char* buf, int m, int n, int lane) {
  if (wide) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      tmaStore2d(map, buf, n, m);  // what lies outside the matrix is not written
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  } else {
    __syncwarp();
    unsigned short* o = static_cast<unsigned short*>(out) + (size_t)m * ld + n + lane;
    const int rows = n + lane < a.N ? min(32, a.M - m) : 0;
#pragma unroll 8
    for (int r = 0; r < rows; ++r)
      o[(size_t)r * ld] = *reinterpret_cast<const unsigned short*>(buf + pieceAt(r, lane >> 3) + ((lane & 7) << 1));
    __syncwarp();
  }
}
template <int DT>
__device__ __forceinline__ void stage32(unsigned char* buf, int lane, const float (&f)[32]) {
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    float g[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = f[v * 8 + e];
    *reinterpret_cast<uint4*>(buf + pieceAt(lane, v)) = Vec16<DT>::pack(g);
  }
}

template <int ACT>
__device__ __forceinline__ void activate32(float (&f)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 y = split(activate<ACT>(pair(f[i], f[i + 1])));
    f[i] = y.x;
    f[i + 1] = y.y;
  }
}
// One warp's 32 x 32 elements of the residual, rows m.. and columns n..: read
// along the rows, asked for before the tile's products are waited for, and
// handed to the lanes that own the rows through the staging buffer.
template <int DT>
struct Residual {
  uint32_t w[16];
  static __device__ __forceinline__ bool pieces(const Problem& a, int n) { return a.wideR && a.N - n >= 32; }
  __device__ __forceinline__ void load(const Problem& a, int m, int n, int lane) {
    const unsigned short* r = static_cast<const unsigned short*>(a.residual) + (size_t)m * a.ldr + n;
    const int rows = min(32, a.M - m);
    if (pieces(a, n)) {  // a piece of 16 bytes a lane, eight rows at a time
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = i * 8 + (lane >> 2);
        const uint4 v = row < rows ? __ldg(reinterpret_cast<const uint4*>(r + (size_t)row * a.ldr) + (lane & 3)) : make_uint4(0, 0, 0, 0);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    } else {  // a column a lane, two rows at a time
      const bool exists = n + lane < a.N;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const unsigned short* p = r + (size_t)(2 * i) * a.ldr + lane;
        const uint32_t lo = exists && 2 * i < rows ? p[0] : 0u, hi = exists && 2 * i + 1 < rows ? p[a.ldr] : 0u;
        w[i] = lo | hi << 16;
      }
    }
  }
  __device__ __forceinline__ void put(const Problem& a, int n, unsigned char* buf, int lane) const {
    if (pieces(a, n)) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(buf + pieceAt(i * 8 + (lane >> 2), lane & 3)) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        *reinterpret_cast<unsigned short*>(buf + pieceAt(2 * i, lane >> 3) + ((lane & 7) << 1)) = (unsigned short)(w[i] & 0xffffu);
        *reinterpret_cast<unsigned short*>(buf + pieceAt(2 * i + 1, lane >> 3) + ((lane & 7) << 1)) = (unsigned short)(w[i] >> 16);
      }
    }
  }
  static __device__ __forceinline__ void add(const unsigned char* buf, int lane, float (&f)[32]) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float g[8];
      Vec16<DT>::expand(*reinterpret_cast<const uint4*>(buf + pieceAt(lane, v)), g);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[v * 8 + e] += g[e];
    }
  }
};
// The bias of 64 columns from n on, a pair a lane, asked for before a tile's products are waited for; a column's value
// then comes from its lane. (Loaded where it is used, each 32 columns waited 1200 cycles for it.)
template <int DT>
__device__ __forceinline__ uint32_t biasPair(const Problem& a, int n, int lane) {
  const unsigned short* p = static_cast<const unsigned short*>(a.bias) + n + 2 * lane;
  const uint32_t lo = n + 2 * lane < a.N ? p[0] : 0u, hi = n + 2 * lane + 1 < a.N ? p[1] : 0u;
  return lo | hi << 16;
}
template <int DT>
__device__ __forceinline__ void addBias(float (&f)[32], uint32_t pair, int half) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float2 v = unpack2<DT>(__shfl_sync(0xffffffffu, pair, half * 16 + j));
    f[2 * j] += v.x;
    f[2 * j + 1] += v.y;
  }
}

// One stage of a block's operands: rows m.. of A and n.. of B, contraction elements k..k + BK. A K-major operand comes as
// boxes of 64 contraction elements (one swizzled row each), an MN-major one as boxes of 64 rows.
template <int CG, int BN>
__device__ __forceinline__ void loadStage(const Problem& a, unsigned char* sa, uint32_t bar, int m, int n, int k) {
  using Sh = ProductShape<CG, BN>;
  constexpr int BK = Sh::kBK;
  unsigned char* sb = sa + kBM * BK * 2;
  if (!a.aMN) {
#pragma unroll
    for (int i = 0; i < BK / 64; ++i) tmaLoad2d<CG>(&a.a, sa + i * kBM * 128, bar, k + i * 64, m);
  } else {
#pragma unroll
    for (int i = 0; i < kBM / 64; ++i) tmaLoad2d<CG>(&a.a, sa + i * BK * 128, bar, m + i * 64, k);
  }
  if (!a.bMN) {
#pragma unroll
    for (int i = 0; i < BK / 64; ++i) tmaLoad2d<CG>(&a.b, sb + i * Sh::kBRows * 128, bar, k + i * 64, n);
  } else {
#pragma unroll
    for (int i = 0; i < Sh::kBRows / 64; ++i) tmaLoad2d<CG>(&a.b, sb + i * BK * 128, bar, n + i * 64, k);
  }
}
// How the MMAs of a problem address a stage: 16 contraction elements on are 32 bytes along a K-major row (and the next box
// after four of them), 16 rows of an MN-major tile.
struct Issue {
  uint64_t descA, descB;
  uint32_t idesc;
  uint32_t aStep, bStep, aBox, bBox;
};
template <int DT, int CG, int BN>
__device__ __forceinline__ Issue makeIssue(const Problem& a, uint32_t smem) {
  using Sh = ProductShape<CG, BN>;
  constexpr uint32_t kType = DT == vrcclBfloat16 ? 1u : 0u;
  Issue q;
  // f32 accumulators; A and B of the element type; majors; N / 8, M / 16
  q.idesc = 1u << 4 | kType << 7 | kType << 10 | (a.aMN ? 1u : 0u) << 15 | (a.bMN ? 1u : 0u) << 16 |
            (uint32_t)(BN / 8) << 17 | (uint32_t)(CG * kBM / 16) << 24;
  q.descA = operandDesc(smem, a.aMN, Sh::kBK);
  q.descB = operandDesc(smem + kBM * Sh::kBK * 2, a.bMN, Sh::kBK);
  q.aStep = a.aMN ? 2048 >> 4 : 32 >> 4;
  q.bStep = a.bMN ? 2048 >> 4 : 32 >> 4;
  q.aBox = a.aMN ? 4 * 2048 >> 4 : kBM * 128 >> 4;
  q.bBox = a.bMN ? 4 * 2048 >> 4 : Sh::kBRows * 128 >> 4;
  return q;
}
template <int CG, int BN>
__device__ __forceinline__ void issueStage(const Issue& q, uint32_t d, int stage, bool fresh) {
  using Sh = ProductShape<CG, BN>;
  const uint64_t da = q.descA + stage * (Sh::kStageBytes >> 4), db = q.descB + stage * (Sh::kStageBytes >> 4);
#pragma unroll
  for (int i = 0; i < Sh::kBK / 16; ++i)
    tcMma<CG>(d, da + (i >> 2) * q.aBox + (i & 3) * q.aStep, db + (i >> 2) * q.bBox + (i & 3) * q.bStep, q.idesc,
              !fresh || i > 0);
}

template <int DT, int CG, int BN>
__global__ void __launch_bounds__(kProductThreads, 1) productKernel(const __grid_constant__ ProductArgs args) {
  using Sh = ProductShape<CG, BN>;
  constexpr int kStages = Sh::kStages;
  extern __shared__ unsigned char dyn[];
  __shared__ unsigned long long full[kStages], empty[kStages], accFull[2], accEmpty[2], drained;
  __shared__ uint32_t tmemSlot;
  __shared__ int deadWord;
  volatile int* dead = &deadWord;
  unsigned char* smem = dyn + ((1024 - (smemAddr(dyn) & 1023)) & 1023);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? clusterRank() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbarInit(&full[s], 1);
      mbarInit(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbarInit(&accFull[s], 1);
      mbarInit(&accEmpty[s], kEpilogueWarps * CG);
    }
    mbarInit(&drained, 1);
    deadWord = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmemAlloc<CG>(&tmemSlot, Sh::kTmemCols);
  tcFenceBefore();
  __syncwarp();
  if constexpr (CG == 2) clusterSync();
  __syncthreads();
  tcFenceAfter();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmemSlot, 0);
  letNextIn();
  waitForPrevious();

  const int unit = blockIdx.x / CG;

  if (warp == 0) {
    const bool one = electOne();
    const uint32_t firstBar = CG == 2 ? inBlock(&full[0], 0) : smemAddr(&full[0]);
    int stage = 0, round = 0;
    bool ok = true;
    for (Walk w(args, unit, gridDim.x / CG); w.more() && ok; w.next(args, unit)) {
      const Problem& a = args.p[w.which];
      int m, n;
      w.place<Sh::kGroup>(a, m, n);
      m = m * (CG * kBM) + (int)rank * kBM;
      n = n * BN + (int)rank * Sh::kBRows;
      for (int k = 0; k < a.steps; ++k) {
        if (round > 0 && !(ok = __all_sync(0xffffffffu, waitBar(&empty[stage], (round - 1) & 1, dead)))) break;
        if (one) {
          // both blocks' copies count on the first block's barrier, which its MMA warp waits on
          if (rank == 0) mbarArriveExpect(&full[stage], Sh::kStageBytes * CG);
          loadStage<CG, BN>(a, smem + stage * Sh::kStageBytes, firstBar + stage * 8, m, n, k * Sh::kBK);
        }
        if (++stage == kStages) {
          stage = 0;
          ++round;
        }
      }
    }
    // given up: no copy may land after the block has gone
    if (!ok && rank == 0 && lane == 0) {
      int quiet = 0;
      for (int s = 0; s < kStages; ++s) {
        const int issued = round + (s < stage ? 1 : 0);
        if (issued > 0) waitBar(&full[s], (issued - 1) & 1, &quiet, kDrainCycles);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      const bool one = electOne();
      int stage = 0, round = 0, turn = 0;
      bool ok = true;
      for (Walk w(args, unit, gridDim.x / CG); w.more() && ok; w.next(args, unit), ++turn) {
        const Problem& a = args.p[w.which];
        const Issue q = makeIssue<DT, CG, BN>(a, smemAddr(smem));
        const int acc = turn & 1, use = turn >> 1;
        if (use > 0 && !(ok = __all_sync(0xffffffffu, waitBar(&accEmpty[acc], (use - 1) & 1, dead)))) break;
        tcFenceAfter();
        const uint32_t d = tmem + acc * BN;
        for (int k = 0; k < a.steps; ++k) {
          if (!(ok = __all_sync(0xffffffffu, waitBar(&full[stage], round & 1, dead)))) break;
          tcFenceAfter();
          if (one) {
            issueStage<CG, BN>(q, d, stage, k == 0);
            tcCommit<CG>(&empty[stage]);
          }
          if (++stage == kStages) {
            stage = 0;
            ++round;
          }
        }
        if (ok && one) tcCommit<CG>(&accFull[acc]);
      }
      if (!ok && one) {  // given up: the products in flight end before TMEM is freed
        int quiet = 0;
        tcCommit<CG>(&drained);
        waitBar(&drained, 0, &quiet, kDrainCycles);
      }
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    const int part = (warp - 2) >> 2;
    constexpr int kCols = BN / (kEpilogueWarps / 4);  // columns a warp finishes, 32 at a time
    unsigned char* buf = smem + kStages * Sh::kStageBytes + (warp - 2) * 2 * kStoreBytes;
    int turn = 0, which = 0;
    for (Walk w(args, unit, gridDim.x / CG); w.more(); w.next(args, unit), ++turn) {
      const Problem& a = args.p[w.which];
      int m0, n0;
      w.place<Sh::kGroup>(a, m0, n0);
      m0 = m0 * (CG * kBM) + (int)rank * kBM + quarter * 32;
      n0 = n0 * BN + part * kCols;
      const int acc = turn & 1, use = turn >> 1;
      uint32_t bias[(kCols + 63) / 64];
      if (a.bias)
#pragma unroll
        for (int i = 0; i < (kCols + 63) / 64; ++i) bias[i] = biasPair<DT>(a, n0 + i * 64, lane);
      Residual<DT> residual;
      if (a.residual && m0 < a.M && n0 < a.N) residual.load(a, m0, n0, lane);
      // (every lane waits: the barrier orders the products before the loads of the thread that has seen it)
      if (!__all_sync(0xffffffffu, waitBar(&accFull[acc], use & 1, dead))) break;
      tcFenceAfter();
      const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + acc * BN + part * kCols;
      if (m0 < a.M) {
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          const int n = n0 + c;
          if (n >= a.N) break;
          // the buffers take turns; the store that last read one has to be done with it
          unsigned char* zb = buf + which * kStoreBytes;
          if (a.z) which ^= 1;
          unsigned char* yb = buf + which * kStoreBytes;
          which ^= 1;
          if (lane == 0) {
            if (a.z)
              asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            else
              asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          }
          __syncwarp();
          if (a.residual) {
            residual.put(a, n, yb, lane);
            __syncwarp();
            if (c + 32 < kCols && n + 32 < a.N) residual.load(a, m0, n + 32, lane);
          }
          float f[32];
          tcLoad32(from + c, f);
          if (a.bias) addBias<DT>(f, bias[c / 64], c / 32 & 1);
          if (a.z) {
            stage32<DT>(zb, lane, f);
            storeBox(a, &a.zMap, a.z, a.ldz, a.wideZ, zb, m0, n, lane);
          }
          switch (a.act) {
            case vrcclActRelu: activate32<vrcclActRelu>(f); break;
            case vrcclActGelu: activate32<vrcclActGelu>(f); break;
            case vrcclActGeluTanh: activate32<vrcclActGeluTanh>(f); break;
            case vrcclActSilu: activate32<vrcclActSilu>(f); break;
            default: break;
          }
          if (a.residual) Residual<DT>::add(yb, lane, f);
          stage32<DT>(yb, lane, f);
          storeBox(a, &a.dMap, a.d, a.ldd, a.wideD, yb, m0, n, lane);
        }
      }
      tcFenceBefore();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2)
          mbarArriveAt(inBlock(&accEmpty[acc], 0));
        else
          mbarArrive(&accEmpty[acc]);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  tcFenceBefore();
  __syncthreads();
  if constexpr (CG == 2) clusterSync();  // no block leaves while the other may still signal it or use its operands
  tcFenceAfter();
  if (warp == 1) tmemFree<CG>(tmem, Sh::kTmemCols);
}

// ------------------------------------------------------------ split contraction

// Few tiles and a long contraction: the blocks of a cluster take a part of it
// each for one tile of 128 x BN, lay their sums out in shared memory, and each
// finishes its share of the tile from everyone's, added in the blocks' order,
// through distributed shared memory. One launch, no workspace, the same bits
// every time.
//
// With few rows of x a tile of 128 of them would be mostly padding, and the
// stages that hold it are missing for W, which is all such a call has to read.
// Then the operands change places (SWAP): W gives the tile's 128 rows, x its
// columns, and the result is turned back on the way out.
constexpr int kMaxSplit = 8;
template <int BN, bool SWAP>
struct SplitShape {
  static constexpr int kStages = BN == 32 ? 5 : 4;
  static constexpr int kSmem = kStages * ProductShape<1, BN>::kStageBytes + 1024;
  // floats from one row of the sums to the next (SWAP: from one column): 16-byte accesses fall on different banks
  static constexpr int kRow = SWAP ? kBM + 4 : BN + 4;
};

template <int DT>
__device__ __forceinline__ void finish4(const Problem& a, float (&f)[4], size_t m, int n, int cols) {
  using S = typename Ty<DT>::S;
  const int left = min(4, cols - n);
  auto put = [&](void* out, size_t ld) {
    S* o = static_cast<S*>(out) + m * ld + n;
    if (left == 4 && ((uintptr_t)o & 7) == 0) {
      *reinterpret_cast<uint2*>(o) = make_uint2(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) o[i] = Ty<DT>::fromF(f[i]);
    }
  };
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) f[i] += loadOne<DT>(a.bias, n + i);
  }
  if (a.z) put(a.z, a.ldz);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = activateBy(a.act, f[i]);
  if (a.residual) {
    const S* r = static_cast<const S*>(a.residual) + m * a.ldr + n;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) f[i] += Ty<DT>::toF(r[i]);
  }
  put(a.d, a.ldd);
}

template <int DT, int BN, bool SWAP>
__global__ void __launch_bounds__(kProductThreads, 1) productSplit(const __grid_constant__ Problem a, int parts) {
  using Sh = ProductShape<1, BN>;
  using Sp = SplitShape<BN, SWAP>;
  constexpr int kStages = Sp::kStages;
  extern __shared__ unsigned char dyn[];
  __shared__ unsigned long long full[kStages], empty[kStages], accFull, drained;
  __shared__ uint32_t tmemSlot;
  __shared__ int deadWord;
  volatile int* dead = &deadWord;
  unsigned char* smem = dyn + ((1024 - (smemAddr(dyn) & 1023)) & 1023);
  float* part = reinterpret_cast<float*>(smem);  // over the stages, once they have all been used
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = clusterRank(), tile = blockIdx.x / parts;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbarInit(&full[s], 1);
      mbarInit(&empty[s], 1);
    }
    mbarInit(&accFull, 1);
    mbarInit(&drained, 1);
    deadWord = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmemAlloc<1>(&tmemSlot, BN);
  tcFenceBefore();
  __syncthreads();
  tcFenceAfter();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmemSlot, 0);
  letNextIn();
  waitForPrevious();
  const int m0 = tile % a.tilesM * kBM, n0 = tile / a.tilesM * BN;
  const int rows = SWAP ? a.N : a.M, cols = SWAP ? a.M : a.N;  // of the result
  const int per = (a.steps + parts - 1) / parts, lo = min(a.steps, rank * per), hi = min(a.steps, lo + per);
  if (warp == 0) {
    const bool one = electOne();
    int stage = 0, round = 0;
    bool ok = true;
    for (int k = lo; k < hi; ++k) {
      if (round > 0 && !(ok = __all_sync(0xffffffffu, waitBar(&empty[stage], (round - 1) & 1, dead)))) break;
      if (one) {
        mbarArriveExpect(&full[stage], Sh::kStageBytes);
        loadStage<1, BN>(a, smem + stage * Sh::kStageBytes, smemAddr(&full[stage]), m0, n0, k * Sh::kBK);
      }
      if (++stage == kStages) {
        stage = 0;
        ++round;
      }
    }
    if (!ok && lane == 0) {  // given up: no copy may land after the block has gone
      int quiet = 0;
      for (int s = 0; s < kStages; ++s) {
        const int issued = round + (s < stage ? 1 : 0);
        if (issued > 0) waitBar(&full[s], (issued - 1) & 1, &quiet, kDrainCycles);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    const bool one = electOne();
    const Issue q = makeIssue<DT, 1, BN>(a, smemAddr(smem));
    int stage = 0, round = 0;
    bool ok = true;
    for (int k = lo; k < hi; ++k) {
      if (!(ok = __all_sync(0xffffffffu, waitBar(&full[stage], round & 1, dead)))) break;
      tcFenceAfter();
      if (one) {
        issueStage<1, BN>(q, tmem, stage, k == lo);
        tcCommit<1>(&empty[stage]);
      }
      if (++stage == kStages) {
        stage = 0;
        ++round;
      }
    }
    if (one) {
      if (ok) {
        tcCommit<1>(&accFull);
      } else {  // given up: the products in flight end before TMEM is freed
        int quiet = 0;
        tcCommit<1>(&drained);
        waitBar(&drained, 0, &quiet, kDrainCycles);
      }
    }
    __syncwarp();
  } else if (warp < 6) {
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    const bool ok = __all_sync(0xffffffffu, waitBar(&accFull, 0, dead));
    tcFenceAfter();
    const int r = quarter * 32 + lane;
#pragma unroll
    for (int h = 0; h < BN / 32 && ok; ++h) {
      float f[32];
      if (lo < hi) {
        tcLoad32(tmem + ((uint32_t)(quarter * 32) << 16) + h * 32, f);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = 0.f;
      }
      if constexpr (SWAP) {
#pragma unroll
        for (int i = 0; i < 32; ++i) part[(h * 32 + i) * Sp::kRow + r] = f[i];
      } else {
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<float4*>(part + r * Sp::kRow + h * 32 + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
      }
    }
    tcFenceBefore();
  }
  __syncthreads();
  clusterSync();
  if (warp >= 2) {
    // groups of four outputs along a row of the result, dealt to the blocks in runs
    constexpr int kAcross = SWAP ? kBM / 4 : BN / 4, kDown = SWAP ? BN : kBM;
    const int share = kAcross * kDown / parts;
    for (int g = rank * share + threadIdx.x - 64; g < (rank + 1) * share; g += kProductThreads - 64) {
      const int r = g / kAcross, c = g % kAcross * 4;
      const int m = (SWAP ? n0 : m0) + r, n = (SWAP ? m0 : n0) + c;
      if (m >= rows || n >= cols) continue;
      float f[4] = {0.f, 0.f, 0.f, 0.f};
      for (int s = 0; s < parts; ++s) {
        float4 v;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(inBlock(part + r * Sp::kRow + c, s))
                     : "memory");
        f[0] += v.x;
        f[1] += v.y;
        f[2] += v.z;
        f[3] += v.w;
      }
      finish4<DT>(a, f, m, n, cols);
    }
  }
  __syncwarp();
  clusterSync();  // no block leaves while another reads its sums
  tcFenceAfter();
  if (warp == 1) tmemFree<1>(tmem, BN);
}

// ------------------------------------------------------------ few rows

// One or two rows: 4096 x 4096 in 7.2 and 8.2 us where the split product takes 9.2 and 9.6. Up to eight where W would first
// have to be copied for TMA, which alone reads and writes it once more.
constexpr int kFewRows = 2, kFewRowsUnaligned = 8;
// Outputs a block, as many rows of W a thread has in flight: eight for one row of x (4096 x 4096 in 7.2 us against 8.8 with
// four), four for more (two rows 8.2 us against 12.6 with eight, whose sums crowd the registers).
constexpr int fewOuts(int rows) { return rows == 1 ? 8 : 4; }
constexpr int kFewThreads = 256;

struct FewArgs {
  const void* x;
  const void* w;
  const void* bias;
  const void* residual;
  void* y;
  void* z;
  size_t ldx, ldw, ldr, ldy, ldz;
  int rows, outs, ins, act;
};

// The warp's sums of N values a lane, value i in the lanes i (32 / N) and on: at every step a lane gives half of its values
// to its partner and keeps the other half, N - 1 shuffles and a few where N separate sums would take 5 N.
template <int N>
__device__ __forceinline__ float laneSums(float (&v)[N], int lane) {
  int o = 16;
#pragma unroll
  for (int half = N / 2; half > 0; half /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float give = upper ? v[i] : v[i + half], keep = upper ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  for (; o > 0; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// MR rows of x against a few rows of W a block, the contraction dealt to the
// threads in 16-byte vectors (WIDE) or single elements, joined at the end.
template <int DT, int MR, bool WIDE>
__global__ void __launch_bounds__(kFewThreads) linearFew(const __grid_constant__ FewArgs a) {
  using S = typename Ty<DT>::S;
  constexpr int V = WIDE ? 8 : 1, kOuts = fewOuts(MR);
  __shared__ float part[kFewThreads / 32][kOuts * MR];
  const S* x = static_cast<const S*>(a.x);
  const S* w = static_cast<const S*>(a.w);
  const int n0 = blockIdx.x * kOuts;
  float acc[kOuts][MR] = {};
  const int nvec = a.ins / V;
  for (int i = threadIdx.x; i < nvec; i += kFewThreads) {
    float wf[kOuts][V];
#pragma unroll
    for (int o = 0; o < kOuts; ++o) {
      const S* row = w + (size_t)min(n0 + o, a.outs - 1) * a.ldw + (size_t)i * V;
      if constexpr (WIDE)
        Vec16<DT>::expand(__ldg(reinterpret_cast<const uint4*>(row)), wf[o]);
      else
        wf[o][0] = Ty<DT>::toF(*row);
    }
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      float xf[V];
      const S* row = x + (size_t)min(m, a.rows - 1) * a.ldx + (size_t)i * V;
      if constexpr (WIDE)
        Vec16<DT>::expand(__ldg(reinterpret_cast<const uint4*>(row)), xf);
      else
        xf[0] = Ty<DT>::toF(*row);
#pragma unroll
      for (int o = 0; o < kOuts; ++o)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[o][m] += wf[o][e] * xf[e];
    }
  }
  const float s = laneSums(reinterpret_cast<float(&)[kOuts * MR]>(acc), threadIdx.x & 31);
  constexpr int kLanes = 32 / (kOuts * MR);  // lanes that hold the same sum
  if (threadIdx.x % kLanes == 0) part[threadIdx.x >> 5][(threadIdx.x & 31) / kLanes] = s;
  __syncthreads();
  if (threadIdx.x < kOuts * MR) {
    const int n = n0 + threadIdx.x / MR, m = threadIdx.x % MR;
    if (n >= a.outs || m >= a.rows) return;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kFewThreads / 32; ++i) s += part[i][threadIdx.x];
    if (a.bias) s += loadOne<DT>(a.bias, n);
    if (a.z) static_cast<S*>(a.z)[(size_t)m * a.ldz + n] = Ty<DT>::fromF(s);
    s = activateBy(a.act, s);
    if (a.residual) s += loadOne<DT>(a.residual, (size_t)m * a.ldr + n);
    static_cast<S*>(a.y)[(size_t)m * a.ldy + n] = Ty<DT>::fromF(s);
  }
}

// ------------------------------------------------------------ operands and the bias gradient

// Eight consecutive elements from a row that starts on any element, those past `left` as zeros.
__device__ __forceinline__ uint4 gather8(const unsigned short* p, int left) {
  unsigned short e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = i < left ? p[i] : (unsigned short)0;
  return make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16,
                    e[6] | (uint32_t)e[7] << 16);
}

// Copies whose rows start on 16-byte boundaries, which TMA needs; one launch
// for all operands of a call. A thread gathers eight elements (its warp's
// loads lie next to one another, in L1 after the first) and writes them as one
// piece.
struct PackJob {
  const unsigned short* src;
  unsigned short* dst;
  size_t lds, groups;      // groups: pieces of the copy
  unsigned cols, perRow;   // perRow: pieces a row
};
constexpr int kPackTurn = 2;  // pieces a thread has in flight
struct PackArgs {
  PackJob job[3];
};
__global__ void __launch_bounds__(256) packRows(const __grid_constant__ PackArgs a) {
  const PackJob& j = a.job[blockIdx.y];
  letNextIn();
  waitForPrevious();
  const size_t step = (size_t)gridDim.x * 256;
  for (size_t g0 = (size_t)blockIdx.x * 256 + threadIdx.x; g0 < j.groups; g0 += kPackTurn * step) {
    uint4 v[kPackTurn];
#pragma unroll
    for (int u = 0; u < kPackTurn; ++u) {
      const size_t g = g0 + u * step;
      if (g >= j.groups) continue;
      const size_t r = j.groups >> 32 ? g / j.perRow : (unsigned)g / j.perRow;
      const unsigned c = (unsigned)(g - r * j.perRow) * 8;
      v[u] = gather8(j.src + r * j.lds + c, (int)min(8u, j.cols - c));
    }
#pragma unroll
    for (int u = 0; u < kPackTurn; ++u)
      if (g0 + u * step < j.groups) reinterpret_cast<uint4*>(j.dst)[g0 + u * step] = v[u];
  }
}

struct SlopeArgs {
  const void* dy;
  const void* z;
  void* dz;        // NULL: only the sums
  float* partial;  // [blocks][cols] or NULL
  size_t lddy, ldz, lddz, rows;
  int cols;
};
constexpr int kSlopeRows = 8;  // row groups of a block; 32 lanes of 8 columns across
constexpr int kSlopeTurn = 4;  // rows a thread has in flight

// dz = dy act'(z), rounded to the element type: the tensor cores take their
// operands in it. The bias gradient sums the unrounded values. A thread has
// eight columns; WIDE: rows of dy and z start on 16-byte boundaries (and end
// on them), else their elements are gathered. dz always does. Bound by memory:
// for 8192 x 4096 bf16 with gelu (201 MB) it takes 36 us with cold caches and adds 21 to the products.
template <int DT, int ACT, bool WIDE>
__global__ void __launch_bounds__(256, 4) linearSlope(const __grid_constant__ SlopeArgs a) {
  using S = typename Ty<DT>::S;
  __shared__ float part[kSlopeRows][256];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * 8;
  F2 sum[4] = {};
  letNextIn();
  if (c < a.cols) {
    const int left = min(8, a.cols - c);
    const size_t step = (size_t)gridDim.y * kSlopeRows;
    for (size_t r0 = (size_t)blockIdx.y * kSlopeRows + g; r0 < a.rows; r0 += kSlopeTurn * step) {
      uint4 d[kSlopeTurn], z[kSlopeTurn];  // the rows of a turn are all asked for before the first is used
#pragma unroll
      for (int u = 0; u < kSlopeTurn; ++u) {
        const size_t r = r0 + u * step;
        if (r < a.rows) {
          const unsigned short* dy = static_cast<const unsigned short*>(a.dy) + r * a.lddy + c;
          d[u] = WIDE ? __ldg(reinterpret_cast<const uint4*>(dy)) : gather8(dy, left);
          if constexpr (ACT != vrcclActNone) {
            const unsigned short* zp = static_cast<const unsigned short*>(a.z) + r * a.ldz + c;
            z[u] = WIDE ? __ldcs(reinterpret_cast<const uint4*>(zp)) : gather8(zp, left);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kSlopeTurn; ++u) {
        const size_t r = r0 + u * step;
        if (r >= a.rows) break;
        float f[8], h[8];
        Vec16<DT>::expand(d[u], f);
        if constexpr (ACT != vrcclActNone) Vec16<DT>::expand(z[u], h);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          F2 x = pair(f[2 * e], f[2 * e + 1]);
          if constexpr (ACT != vrcclActNone) x = mul2(x, slope<ACT>(pair(h[2 * e], h[2 * e + 1])));
          sum[e] = add2(sum[e], x);
          const float2 y = split(x);
          f[2 * e] = y.x;
          f[2 * e + 1] = y.y;
        }
        if (a.dz) *reinterpret_cast<uint4*>(static_cast<S*>(a.dz) + r * a.lddz + c) = Vec16<DT>::pack(f);
      }
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) *reinterpret_cast<float2*>(&part[g][lane * 8 + 2 * e]) = split(sum[e]);
  __syncthreads();
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col >= a.cols) return;
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < kSlopeRows; ++k) s += part[k][threadIdx.x];
  a.partial[(size_t)blockIdx.y * a.cols + col] = s;
}

template <int DT>
__global__ void __launch_bounds__(1024) linearBiasJoin(const float* partial, int blocks, int cols, void* db) {
  const int c = blockIdx.x * 32 + (threadIdx.x & 31);
  waitForPrevious();
  const float s = columnSum(partial + c, blocks, cols, c < cols);
  if (threadIdx.x < 32 && c < cols) static_cast<typename Ty<DT>::S*>(db)[c] = Ty<DT>::fromF(s);
}

// ------------------------------------------------------------ host

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// (Asked for again after a failure: the driver may not have been there yet.)
EncodeFn encodeFn() {
  static std::atomic<EncodeFn> known{nullptr};
  EncodeFn fn = known.load(std::memory_order_relaxed);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    known.store(fn = (EncodeFn)p, std::memory_order_relaxed);
  }
  return fn;
}

// Tiles of boxCols (64: operands, 32: results) x boxRows out of a [rows, cols]
// matrix of 2-byte elements whose rows start on 16-byte boundaries, swizzled
// over their rows' bytes; what lies outside reads as zero.
bool makeMap(CUtensorMap* map, int dtype, const void* p, size_t ld, size_t rows, size_t cols, int boxRows,
             int boxCols = 64) {
  const EncodeFn fn = encodeFn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * 2};
  const cuuint32_t box[2] = {(cuuint32_t)boxCols, (cuuint32_t)boxRows}, step[2] = {1, 1};
  return fn(map, dtype == vrcclBfloat16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
            const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            boxCols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operand {
  const void* p;
  size_t ld, rows, cols;  // as it lies in memory
  bool mn;                // the contraction runs over its rows
};

size_t packedLd(size_t cols) { return (cols + 7) / 8 * 8; }
size_t packedBytes(size_t rows, size_t cols) { return (rows * packedLd(cols) * 2 + 255) / 256 * 256; }

// Hands out the workspace in order.
struct Scratch {
  unsigned char* p;
  size_t left;
  void* take(size_t bytes) {
    if (!p || bytes > left) return nullptr;
    void* r = p;
    p += bytes;
    left -= bytes;
    return r;
  }
};

// Workspace that a copy of an operand takes.
size_t packNeed(const void* p, size_t ld, size_t rows, size_t cols) {
  return rowsAligned(p, ld, 2) ? 0 : packedBytes(rows, cols);
}
// Operands to be copied before a call's products.
struct Packing {
  PackArgs args = {};
  int jobs = 0;
  // The operand as the products will find it; false: the workspace is too small.
  bool add(Operand& o, Scratch& ws) {
    if (rowsAligned(o.p, o.ld, 2)) return true;
    unsigned short* q = static_cast<unsigned short*>(ws.take(packedBytes(o.rows, o.cols)));
    if (!q) return false;
    const size_t perRow = packedLd(o.cols) / 8;
    args.job[jobs++] = {static_cast<const unsigned short*>(o.p), q, o.ld, o.rows * perRow, (unsigned)o.cols, (unsigned)perRow};
    o.p = q;
    o.ld = packedLd(o.cols);
    return true;
  }
  vrcclResult_t launch(bool after, cudaStream_t st) const {
    if (!jobs) return vrcclSuccess;
    size_t most = 0;
    for (int i = 0; i < jobs; ++i) most = std::max(most, args.job[i].groups);
    const size_t blocks = std::min((most + 256 * kPackTurn - 1) / (256 * kPackTurn), (size_t)smCount() * 8);
    const dim3 grid((unsigned)std::max<size_t>(1, blocks), (unsigned)jobs);
    return launchShaped(packRows, {grid, 256, 0, 0, after}, st, args);
  }
};

// A product and where its operands lie.
struct Product {
  Problem p;
  Operand A, B;
};
Product makeProduct(const Operand& A, const Operand& B, void* d, size_t ldd, size_t M, size_t N, size_t K) {
  Product q = {};
  q.A = A;
  q.B = B;
  q.p.d = d;
  q.p.ldd = ldd;
  q.p.M = (int)M;
  q.p.N = (int)N;
  q.p.K = (int)K;
  q.p.aMN = A.mn;
  q.p.bMN = B.mn;
  return q;
}

long long tileCount(const Problem& p, int bm, int bn) {
  return (long long)((p.M + bm - 1) / bm) * ((p.N + bn - 1) / bn);
}

template <int DT, int CG, int BN>
vrcclResult_t launchProducts(const Product* q, int n, bool after, cudaStream_t st) {
  using Sh = ProductShape<CG, BN>;
  const vrcclResult_t allowed = allowSharedMemory((const void*)productKernel<DT, CG, BN>);
  if (allowed != vrcclSuccess) return allowed;
  ProductArgs args;
  memset(&args, 0, sizeof(args));
  long long total = 0;
  for (int i = 0; i < n; ++i) {
    Problem& p = args.p[i];
    const Operand &A = q[i].A, &B = q[i].B;
    p = q[i].p;
    p.wideR = p.residual && rowsAligned(p.residual, p.ldr, 2);
    // a TMA store writes whole 16-byte pieces: rows that end inside one are stored by the warps
    p.wideD = p.N % 8 == 0 && rowsAligned(p.d, p.ldd, 2);
    p.wideZ = p.z && p.N % 8 == 0 && rowsAligned(p.z, p.ldz, 2);
    p.tilesM = (p.M + CG * kBM - 1) / (CG * kBM);
    p.tilesN = (p.N + BN - 1) / BN;
    p.tiles = (int)tileCount(p, CG * kBM, BN);
    p.steps = (p.K + Sh::kBK - 1) / Sh::kBK;
    total += p.tiles;
    if (!makeMap(&p.a, DT, A.p, A.ld, A.rows, A.cols, A.mn ? Sh::kBK : kBM) ||
        !makeMap(&p.b, DT, B.p, B.ld, B.rows, B.cols, B.mn ? Sh::kBK : Sh::kBRows) ||
        (p.wideD && !makeMap(&p.dMap, DT, p.d, p.ldd, p.M, p.N, 32, 32)) ||
        (p.wideZ && !makeMap(&p.zMap, DT, p.z, p.ldz, p.M, p.N, 32, 32)))
      return vrcclInternalError;
  }
  const int units = (int)std::min<long long>(total, std::min(smCount() / CG, kMaxUnits));
  if (n == 2) {
    // every unit's share of the second product tops up what it has of the first, to the smallest common level
    const long long steps0 = args.p[0].steps, steps1 = args.p[1].steps;
    auto has = [&](int u) { return (args.p[0].tiles - u + units - 1) / units * steps0; };
    auto holds = [&](long long level) {
      long long t = 0;
      for (int u = 0; u < units; ++u) t += std::max(0ll, level - has(u)) / steps1;
      return t;
    };
    long long lo = 0, hi = has(0) + (long long)args.p[1].tiles * steps1;
    while (lo < hi) {
      const long long mid = (lo + hi) / 2;
      if (holds(mid) >= args.p[1].tiles)
        hi = mid;
      else
        lo = mid + 1;
    }
    long long given = 0;
    for (int u = 0; u < units; ++u) {
      args.from[u] = (unsigned short)given;
      given = std::min<long long>(args.p[1].tiles, given + std::max(0ll, lo - has(u)) / steps1);
    }
    args.from[units] = (unsigned short)given;
  }
  return launchShaped(productKernel<DT, CG, BN>, {dim3((unsigned)(units * CG)), kProductThreads, Sh::kSmem, CG, after}, st,
                      args);
}

template <int DT, int BN, bool SWAP>
vrcclResult_t launchSplit(const Product& q, int parts, bool after, cudaStream_t st) {
  using Sh = ProductShape<1, BN>;
  using Sp = SplitShape<BN, SWAP>;
  const vrcclResult_t allowed = allowSharedMemory((const void*)productSplit<DT, BN, SWAP>);
  if (allowed != vrcclSuccess) return allowed;
  Problem p = q.p;
  const Operand &A = SWAP ? q.B : q.A, &B = SWAP ? q.A : q.B;
  if (SWAP) {
    std::swap(p.M, p.N);
    std::swap(p.aMN, p.bMN);
  }
  p.tilesM = (p.M + kBM - 1) / kBM;
  p.tiles = (int)tileCount(p, kBM, BN);
  p.steps = (p.K + Sh::kBK - 1) / Sh::kBK;
  if (!makeMap(&p.a, DT, A.p, A.ld, A.rows, A.cols, A.mn ? Sh::kBK : kBM) ||
      !makeMap(&p.b, DT, B.p, B.ld, B.rows, B.cols, B.mn ? Sh::kBK : Sh::kBRows))
    return vrcclInternalError;
  return launchShaped(productSplit<DT, BN, SWAP>,
                      {dim3((unsigned)(p.tiles * parts)), kProductThreads, Sp::kSmem, parts, after}, st, p, parts);
}

// Blocks to a cluster for `tiles` tiles of `steps` stages: as many as find a multiprocessor each and two stages of work.
// (Eight blocks that fill a multiprocessor each are hard to place: 16 clusters of them took 15 us where 16 of four took 11,
// so they are left to calls with few tiles.)
int splitParts(long long tiles, long long steps) {
  int parts = 1;
  while (parts < kMaxSplit && tiles * parts * 2 <= smCount() && parts * 4 <= steps && (parts < 4 || tiles <= 8)) parts *= 2;
  return parts;
}

// Which tile: the one whose last unit ends first, by measured cycles: a step
// of 64 contraction elements and a tile's epilogue (which runs under the next
// tile's steps where they take longer). At 4096 cubed: pairs 81 us, 128 x 128
// tiles 102, 128 x 64 tiles 166; at 1024 cubed 12.4, 10.3 and 8.3. A pair's tile
// of 192 columns is for counts that leave most of a round of 256-wide ones
// empty: 1921 x 2544 x 2808, 80 of those on 76 pairs, 41 us, 37 with 112.
enum Tile { kPair256, kPair192, kBlock128, kBlock64, kSplit64, kSwap32, kSwap64 };
struct Choice {
  Tile tile;
  int parts;
  double cycles;
};
Choice chooseTile(const Product* q, int n) {
  struct Kind {
    Tile tile;
    int bm, bn, blocks, step, end;
  };
  static const Kind kinds[4] = {{kPair256, 256, 256, 2, 520, 6000}, {kPair192, 256, 192, 2, 420, 5000}, {kBlock128, 128, 128, 1, 420, 3000}, {kBlock64, 128, 64, 1, 341, 2200}};
  constexpr double kJoin = 3000;  // the sums' way through distributed shared memory
  if (n == 1 && q->p.M <= 64 && !q->p.aMN) {
    const int parts = splitParts((q->p.N + kBM - 1) / kBM, (q->p.K + 127) / 128);
    const long long rounds = ((q->p.N + kBM - 1) / kBM * (long long)parts + smCount() - 1) / smCount();
    return {q->p.M <= 32 ? kSwap32 : kSwap64, parts, (double)rounds * ((q->p.K + 63) / 64 / parts * 300 + 2200) + kJoin};
  }
  Choice best = {kPair256, 1, 1e300};
  for (const Kind& k : kinds) {
    // (half of its 192 rows of B is no whole number of the 64-wide boxes an MN-major operand comes in)
    if (k.tile == kPair192 && (q[0].p.bMN || q[n - 1].p.bMN)) continue;
    const int units = smCount() / k.blocks;
    double cycles = 0, longest = 0;
    long long tiles = 0;
    for (int i = 0; i < n; ++i) {
      const double tile = std::max<double>((q[i].p.K + 63) / 64 * k.step, k.end);
      const long long t = tileCount(q[i].p, k.bm, k.bn);
      // one product: whole rounds of tiles; two: the second evens out the end
      cycles += tile * (n == 1 ? (double)((t + units - 1) / units) : (double)t / units);
      longest = std::max(longest, tile);
      tiles += t;
    }
    cycles = std::max(n == 1 ? cycles : cycles + longest / 4, longest) + k.end;
    if (cycles < best.cycles) best = {k.tile, 1, cycles};
    if (k.tile == kBlock64 && n == 1) {
      const int parts = splitParts(tiles, (q->p.K + 127) / 128);
      const double split = longest / parts + k.end + kJoin;
      if (parts > 1 && split < best.cycles) best = {kSplit64, parts, split};
    }
  }
  return best;
}

// `after`: the stream's last kernel is this call's own and lets the next one in.
template <int DT>
vrcclResult_t products(const Product* q, int n, bool after, cudaStream_t st) {
  const Choice c = chooseTile(q, n);
  if (n == 2) {
    // One by one where that is shorter (a few rows' dx is one long contraction that wants splitting, their dW is none at
    // all: 16 rows of 4096 x 4096) or where there are more tiles than a launch counts. A launch costs some 3000 cycles.
    const bool many = tileCount(q[0].p, 128, 64) + tileCount(q[1].p, 128, 64) > 60000;
    if (many || chooseTile(q, 1).cycles + chooseTile(q + 1, 1).cycles + 3000 < c.cycles) {
      const vrcclResult_t r = products<DT>(q, 1, after, st);
      return r == vrcclSuccess ? products<DT>(q + 1, 1, true, st) : r;
    }
  }
  switch (c.tile) {
    case kPair256: return launchProducts<DT, 2, 256>(q, n, after, st);
    case kPair192: return launchProducts<DT, 2, 192>(q, n, after, st);
    case kBlock128: return launchProducts<DT, 1, 128>(q, n, after, st);
    case kBlock64: return launchProducts<DT, 1, 64>(q, n, after, st);
    case kSplit64: return launchSplit<DT, 64, false>(q[0], c.parts, after, st);
    case kSwap32: return launchSplit<DT, 32, true>(q[0], c.parts, after, st);
    case kSwap64: return launchSplit<DT, 64, true>(q[0], c.parts, after, st);
  }
  return vrcclInternalError;
}

template <int DT, int MR, bool WIDE>
vrcclResult_t launchFew(const FewArgs& a, cudaStream_t st) {
  return launchShaped(linearFew<DT, MR, WIDE>, {dim3((unsigned)((a.outs + fewOuts(MR) - 1) / fewOuts(MR))), kFewThreads, 0, 0, false}, st, a);
}
template <int DT>
vrcclResult_t few(const FewArgs& a, bool wide, cudaStream_t st) {
  if (wide && a.rows <= 2) return a.rows == 1 ? launchFew<DT, 1, true>(a, st) : launchFew<DT, 2, true>(a, st);
  if (a.rows <= 2) return a.rows == 1 ? launchFew<DT, 1, false>(a, st) : launchFew<DT, 2, false>(a, st);
  return a.rows <= 4 ? launchFew<DT, 4, false>(a, st) : launchFew<DT, 8, false>(a, st);
}

// Row blocks of linearSlope: enough for two waves of blocks.
int slopeBlocks(size_t rows, size_t cols) {
  const size_t across = (cols + 255) / 256;
  const size_t want = std::max<size_t>(1, (size_t)smCount() * 8 / across);
  return (int)std::min<size_t>(want, (rows + kSlopeRows - 1) / kSlopeRows);
}

// Workspace of the bias gradient's partial sums.
size_t biasBytes(size_t rows, size_t outs) { return (size_t(slopeBlocks(rows, outs)) * outs * 4 + 255) / 256 * 256; }

template <int DT, bool WIDE>
vrcclResult_t launchSlope(int act, dim3 grid, const SlopeArgs& a, cudaStream_t st) {
  void (*fn)(SlopeArgs) = act == vrcclActRelu       ? linearSlope<DT, vrcclActRelu, WIDE>
                          : act == vrcclActGelu     ? linearSlope<DT, vrcclActGelu, WIDE>
                          : act == vrcclActGeluTanh ? linearSlope<DT, vrcclActGeluTanh, WIDE>
                          : act == vrcclActSilu     ? linearSlope<DT, vrcclActSilu, WIDE>
                                                    : linearSlope<DT, vrcclActNone, WIDE>;
  return launchShaped(fn, {grid, 256, 0, 0, false}, st, a);
}

bool goodLinear(size_t rows, size_t outs, size_t ins, int dtype, int act) {
  const size_t most = (size_t(1) << 31) - 65536;
  return rows < most && outs < most && ins < most && isOperatorType(dtype) && (unsigned)act < (unsigned)vrcclNumActs;
}

template <int DT>
vrcclResult_t backward(const void* dy, size_t lddy, const void* z, size_t ldz, const void* x, size_t ldx, const void* w,
                       size_t ldw, void* dx, size_t lddx, void* dw, size_t lddw, void* dbias, size_t rows, size_t outs,
                       size_t ins, int act, Scratch ws, cudaStream_t st) {
  Operand g = {dy, lddy, rows, outs, false};
  const float* partial = nullptr;
  int blocks = 0;
  bool after = false;
  const bool rewrite = act != vrcclActNone && (dx || dw);
  if (rewrite || dbias) {
    SlopeArgs s = {};
    s.dy = dy;
    s.z = z;
    s.lddy = lddy;
    s.ldz = ldz;
    s.rows = rows;
    s.cols = (int)outs;
    if (rewrite) {
      s.lddz = packedLd(outs);
      if (!(s.dz = ws.take(packedBytes(rows, outs)))) return vrcclInvalidArgument;
      g.p = s.dz;
      g.ld = s.lddz;
    }
    if (dbias && !(s.partial = static_cast<float*>(ws.take(biasBytes(rows, outs)))))
      return vrcclInvalidArgument;
    const bool wide = outs % 8 == 0 && rowsAligned(dy, lddy, 2) && (act == vrcclActNone || rowsAligned(z, ldz, 2));
    const dim3 grid((unsigned)((outs + 255) / 256), (unsigned)slopeBlocks(rows, outs));
    const vrcclResult_t r = wide ? launchSlope<DT, true>(act, grid, s, st) : launchSlope<DT, false>(act, grid, s, st);
    if (r != vrcclSuccess) return r;
    partial = s.partial;
    blocks = (int)grid.y;
    after = true;
  }
  Packing pack;
  Operand wt = {w, ldw, outs, ins, true}, xt = {x, ldx, rows, ins, true};
  if (((dx || dw) && !pack.add(g, ws)) || (dx && !pack.add(wt, ws)) || (dw && !pack.add(xt, ws))) return vrcclInvalidArgument;
  if (pack.launch(after, st) != vrcclSuccess) return vrcclCudaError;
  after |= pack.jobs > 0;
  Product q[2];
  int n = 0;
  if (dx) q[n++] = makeProduct(g, wt, dx, lddx, rows, ins, outs);
  if (dw) {
    g.mn = true;
    q[n++] = makeProduct(g, xt, dw, lddw, outs, ins, rows);
  }
  if (n == 2 && q[0].p.K < q[1].p.K) std::swap(q[0], q[1]);  // the longer tiles first: the shorter ones even out the end
  if (n) {
    const vrcclResult_t r = products<DT>(q, n, after, st);
    if (r != vrcclSuccess) return r;
  }
  // last: nothing waits for it, and its launch runs under the products
  if (dbias)
    return launchShaped(linearBiasJoin<DT>, {dim3((unsigned)((outs + 31) / 32)), 1024, 0, 0, true}, st, partial, blocks,
                        (int)outs, dbias);
  return vrcclSuccess;
}

vrcclResult_t zeroRows(void* p, size_t ld, size_t rows, size_t cols, cudaStream_t st) {
  if (cudaMemset2DAsync(p, ld * 2, 0, cols * 2, rows, st) != cudaSuccess) {
    cudaGetLastError();
    return vrcclCudaError;
  }
  return vrcclSuccess;
}

}  // namespace
}  // namespace vrccl

using namespace vrccl;

extern "C" vrcclResult_t vrcclLinearWorkspace(int backward, size_t rows, size_t outs, size_t ins, vrcclDataType_t dtype,
                                              vrcclActivation_t act, size_t* bytes) {
  if (!bytes || !goodLinear(rows, outs, ins, dtype, act)) return vrcclInvalidArgument;
  if (dtype == vrcclFloat32) return vrcclInvalidUsage;
  *bytes = packedBytes(rows, ins) + packedBytes(outs, ins);
  if (backward) *bytes += packedBytes(rows, outs) + biasBytes(rows, outs);
  return vrcclSuccess;
}

extern "C" vrcclResult_t vrcclLinearForward(const void* x, size_t ldx, const void* w, size_t ldw, const void* bias,
                                            const void* residual, size_t ldr, void* y, size_t ldy, void* z, size_t ldz,
                                            size_t rows, size_t outs, size_t ins, vrcclDataType_t dtype,
                                            vrcclActivation_t act, void* workspace, size_t workspaceBytes,
                                            vrcclStream_t stream) {
  if (!goodLinear(rows, outs, ins, dtype, act)) return vrcclInvalidArgument;
  if (dtype == vrcclFloat32) return vrcclInvalidUsage;
  if (rows == 0 || outs == 0) return vrcclSuccess;
  if ((ins && (!goodMatrix(x, ldx, rows, ins, 2) || !goodMatrix(w, ldw, outs, ins, 2))) || !goodMatrix(y, ldy, rows, outs, 2) ||
      (bias && !goodVector(bias, 2)) || (residual && !goodMatrix(residual, ldr, rows, outs, 2)) ||
      (z && !goodMatrix(z, ldz, rows, outs, 2)) || (workspace && !goodVector(workspace, 256)))
    return vrcclInvalidArgument;
  const Span spanR = matrixSpan(residual, ldr, rows, outs, 2), spanZ = matrixSpan(z, ldz, rows, outs, 2);
  const Span out[] = {matrixSpan(y, ldy, rows, outs, 2), spanZ, vectorSpan(workspace, workspaceBytes)};
  const Span in[] = {matrixSpan(x, ldx, rows, ins, 2), matrixSpan(w, ldw, outs, ins, 2), vectorSpan(bias, outs * 2),
                     unlessInPlace(spanR, ldr, y, ldy)};
  if (!apart(out, in) || overlap(spanZ, spanR) || overlap(out[2], spanR)) return vrcclInvalidArgument;
  cudaStream_t st = (cudaStream_t)stream;
  const bool apart = rowsAligned(x, ldx, 2) && rowsAligned(w, ldw, 2);
  if (rows <= (size_t)(apart ? kFewRows : kFewRowsUnaligned) || ins == 0) {
    // ins == 0 is a sum over nothing: the epilogue of zeros, a few rows a launch
    const bool wide = ins % 8 == 0 && apart && rows <= (size_t)kFewRows;
    for (size_t r = 0; r < rows; r += kFewRowsUnaligned) {
      FewArgs a = {};
      a.x = static_cast<const char*>(x) + r * ldx * 2 * (ins != 0);
      a.w = w;
      a.bias = bias;
      a.residual = residual ? static_cast<const char*>(residual) + r * ldr * 2 : nullptr;
      a.y = static_cast<char*>(y) + r * ldy * 2;
      a.z = z ? static_cast<char*>(z) + r * ldz * 2 : nullptr;
      a.ldx = ldx;
      a.ldw = ldw;
      a.ldr = ldr;
      a.ldy = ldy;
      a.ldz = ldz;
      a.rows = (int)std::min<size_t>(kFewRowsUnaligned, rows - r);
      a.outs = (int)outs;
      a.ins = (int)ins;
      a.act = act;
      const vrcclResult_t res =
          dtype == vrcclBfloat16 ? few<vrcclBfloat16>(a, wide, st) : few<vrcclFloat16>(a, wide, st);
      if (res != vrcclSuccess) return res;
    }
    return vrcclSuccess;
  }
  const size_t need = packNeed(x, ldx, rows, ins) + packNeed(w, ldw, outs, ins);
  if (need && (!workspace || workspaceBytes < need)) return vrcclInvalidArgument;
  Scratch ws = {static_cast<unsigned char*>(workspace), workspaceBytes};
  Operand A = {x, ldx, rows, ins, false}, B = {w, ldw, outs, ins, false};
  Packing pack;
  if (!pack.add(A, ws) || !pack.add(B, ws)) return vrcclInvalidArgument;
  if (pack.launch(false, st) != vrcclSuccess) return vrcclCudaError;
  Product q = makeProduct(A, B, y, ldy, rows, outs, ins);
  q.p.z = z;
  q.p.bias = bias;
  q.p.residual = residual;
  q.p.ldz = ldz;
  q.p.ldr = ldr;
  q.p.act = act;
  return dtype == vrcclBfloat16 ? products<vrcclBfloat16>(&q, 1, pack.jobs > 0, st)
                                : products<vrcclFloat16>(&q, 1, pack.jobs > 0, st);
}

extern "C" vrcclResult_t vrcclLinearBackward(const void* dy, size_t lddy, const void* z, size_t ldz, const void* x,
                                             size_t ldx, const void* w, size_t ldw, void* dx, size_t lddx, void* dw,
                                             size_t lddw, void* dbias, size_t rows, size_t outs, size_t ins,
                                             vrcclDataType_t dtype, vrcclActivation_t act, void* workspace,
                                             size_t workspaceBytes, vrcclStream_t stream) {
  if (!goodLinear(rows, outs, ins, dtype, act)) return vrcclInvalidArgument;
  if (dtype == vrcclFloat32) return vrcclInvalidUsage;
  const bool acts = act != vrcclActNone;
  if ((dx && !goodMatrix(dx, lddx, rows, ins, 2)) || (dw && !goodMatrix(dw, lddw, outs, ins, 2)) || (dbias && !goodVector(dbias, 2)) ||
      (workspace && !goodVector(workspace, 256)))
    return vrcclInvalidArgument;
  cudaStream_t st = (cudaStream_t)stream;
  // a sum over no rows, or over no outputs, is zero
  if (rows == 0 || outs == 0 || ins == 0) {
    vrcclResult_t r = vrcclSuccess;
    if (dx && rows && ins) r = zeroRows(dx, lddx, rows, ins, st);
    if (r == vrcclSuccess && dw && outs && ins) r = zeroRows(dw, lddw, outs, ins, st);
    if (r != vrcclSuccess || !dbias || !outs) return r;
    if (rows == 0) return zeroRows(dbias, outs, 1, outs, st);
    dx = dw = nullptr;  // ins == 0: the bias gradient is all there is
  }
  if (!goodMatrix(dy, lddy, rows, outs, 2) || (acts && !goodMatrix(z, ldz, rows, outs, 2)) || (dw && !goodMatrix(x, ldx, rows, ins, 2)) ||
      (dx && !goodMatrix(w, ldw, outs, ins, 2)))
    return vrcclInvalidArgument;
  const Span out[] = {matrixSpan(dx, lddx, rows, ins, 2), matrixSpan(dw, lddw, outs, ins, 2), vectorSpan(dbias, outs * 2),
                      vectorSpan(workspace, workspaceBytes)};
  const Span in[] = {matrixSpan(dy, lddy, rows, outs, 2), matrixSpan(acts ? z : nullptr, ldz, rows, outs, 2),
                     matrixSpan(dw ? x : nullptr, ldx, rows, ins, 2), matrixSpan(dx ? w : nullptr, ldw, outs, ins, 2)};
  if (!apart(out, in)) return vrcclInvalidArgument;
  size_t need = dbias ? biasBytes(rows, outs) : 0;
  if (dx || dw) need += acts ? packedBytes(rows, outs) : packNeed(dy, lddy, rows, outs);
  if (dx) need += packNeed(w, ldw, outs, ins);
  if (dw) need += packNeed(x, ldx, rows, ins);
  if (need && (!workspace || workspaceBytes < need)) return vrcclInvalidArgument;
  Scratch ws = {static_cast<unsigned char*>(workspace), workspaceBytes};
  return dtype == vrcclBfloat16 ? backward<vrcclBfloat16>(dy, lddy, z, ldz, x, ldx, w, ldw, dx, lddx, dw, lddw, dbias,
                                                          rows, outs, ins, act, ws, st)
                                : backward<vrcclFloat16>(dy, lddy, z, ldz, x, ldx, w, ldw, dx, lddx, dw, lddw, dbias,
                                                         rows, outs, ins, act, ws, st);
}

extern "C" vrcclResult_t vrcclReplicaGetAsyncError(vrcclResult_t* asyncErr) {
  if (!asyncErr) return vrcclInvalidArgument;
  int code = 0, norm = 0, rms = 0, rmsBackward = 0;
  // (the copies alone run on the legacy default stream, which does not wait for non-blocking ones)
  if (cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpyFromSymbol(&code, gLinearStatus, sizeof(code)) != cudaSuccess || normStatus(&norm) != cudaSuccess ||
      rmsStatus(&rms) != cudaSuccess || rmsBackwardStatus(&rmsBackward) != cudaSuccess) {
    cudaGetLastError();
    return vrcclCudaError;
  }
  *asyncErr = (vrcclResult_t)(code ? code : norm ? norm : rms ? rms : rmsBackward);
  return vrcclSuccess;
}

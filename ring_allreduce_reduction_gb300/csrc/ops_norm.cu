// Layer norm over the columns of a [rows, cols] matrix, forward and backward.
//
//   xh = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   y  = xh gamma + beta
//   g  = dy gamma
//   dx = rstd (g - mean(g) - xh mean(g xh))
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Both directions are bound by memory: forward reads x and writes y, backward
// reads dy and x and writes dx. A row is loaded once and held in registers
// (packed, as it came) while its sums are formed, so that the mean is known
// before the squares are taken: sum((x - mean)^2) loses nothing to
// cancellation where sum(x^2) - mean^2 would. All sums are binary32.
//
// The weight's gradient is a sum down the columns. Every block owns a fixed
// set of columns a thread, walks rows with the grid's stride and keeps the two
// sums in registers; it writes them once, as one row of a [blocks, 2, cols]
// workspace, and a second kernel adds those rows in order. No atomics: the
// same call gives the same bits.
#include "ops_common.cuh"

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

template <int V>
__device__ __forceinline__ void loadParams(const void* p, int ptype, int c, float dflt, float (&f)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = p ? loadParam(p, ptype, c + e) : dflt;
}

// One row a block, or one row a warp (WARP) where 32 lanes hold it.
template <int DT, bool VEC, int EPT, bool WARP>
__global__ void __launch_bounds__(1024) normForward(const __grid_constant__ NormArgs a) {
  using H = Held<DT, VEC, EPT>;
  constexpr int V = H::V, NV = H::NV, E = floatTypeSize(DT);
  __shared__ float red[2][32];
  const int T = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const size_t per = WARP ? blockDim.x >> 5 : 1;
  const float inv = 1.f / (float)a.cols;
  for (size_t row = blockIdx.x * per + (WARP ? threadIdx.x >> 5 : 0); row < a.rows; row += gridDim.x * per) {
    H h;
    h.load(static_cast<const char*>(a.x) + row * a.ldx * E, t, T, a.cols);
    float f[V], s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      h.get(j, f);
#pragma unroll
      for (int e = 0; e < V; ++e) s += f[e];
    }
    s = WARP ? warpSum(s) : blockSum(s, red[0]);
    const float mean = s * inv;
    s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if ((j * T + t) * V < a.cols) {
        h.get(j, f);
#pragma unroll
        for (int e = 0; e < V; ++e) s += (f[e] - mean) * (f[e] - mean);
      }
    }
    s = WARP ? warpSum(s) : blockSum(s, red[1]);
    const float rstd = 1.f / sqrtf(s * inv + a.eps);
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
        loadParams<V>(a.gamma, a.ptype, i * V, 1.f, g);
        loadParams<V>(a.beta, a.ptype, i * V, 0.f, b);
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

template <int DT, bool VEC, int EPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 1024) normBackward(const __grid_constant__ NormArgs a) {
  using H = Held<DT, VEC, EPT>;
  constexpr int V = H::V, NV = H::NV, E = floatTypeSize(DT);
  __shared__ float2 red[2][32];
  const int T = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const size_t per = WARP ? blockDim.x >> 5 : 1;
  const float inv = 1.f / (float)a.cols;
  float dg[EPT], db[EPT];
#pragma unroll
  for (int i = 0; i < EPT; ++i) dg[i] = db[i] = 0.f;
  int turn = 0;
  for (size_t row = blockIdx.x * per + (WARP ? threadIdx.x >> 5 : 0); row < a.rows; row += gridDim.x * per) {
    H hx, hd;
    hx.load(static_cast<const char*>(a.x) + row * a.ldx * E, t, T, a.cols);
    hd.load(static_cast<const char*>(a.dy) + row * a.lddy * E, t, T, a.cols);
    const float mean = a.mean[row], rstd = a.rstd[row];
    float fx[V], fd[V], g[V];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * T + t) * V;
      if (c < a.cols) {
        loadParams<V>(a.gamma, a.ptype, c, 1.f, g);
        hx.get(j, fx);
        hd.get(j, fd);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xh = (fx[e] - mean) * rstd, gd = fd[e] * g[e];
          s.x += gd;
          s.y += gd * xh;
          dg[j * V + e] += fd[e] * xh;
          db[j * V + e] += fd[e];
        }
      }
    }
    s = WARP ? warpSum2(s) : blockSum2(s, red[turn ^= 1]);
    const float m1 = s.x * inv, m2 = s.y * inv;
    void* out = static_cast<char*>(a.y) + row * a.ldy * E;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = j * T + t;
      if (i * V < a.cols) {
        loadParams<V>(a.gamma, a.ptype, i * V, 1.f, g);
        hx.get(j, fx);
        hd.get(j, fd);
#pragma unroll
        for (int e = 0; e < V; ++e) fx[e] = rstd * (fd[e] * g[e] - m1 - (fx[e] - mean) * rstd * m2);
        H::put(out, i, fx);
      }
    }
  }
  if (!a.partial) return;
  float* p = a.partial + (size_t)blockIdx.x * 2 * a.cols;
  if constexpr (WARP) {
    // the block's warps own the same columns: add them up in warp order
    __shared__ float sum[2 * 32 * EPT];
    for (int w = 0; w < (int)per; ++w) {
      if ((int)(threadIdx.x >> 5) == w) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          float* q = sum + i * 32 + t;
          q[0] = w ? q[0] + dg[i] : dg[i];
          q[32 * EPT] = w ? q[32 * EPT] + db[i] : db[i];
        }
      }
      __syncthreads();
    }
    if (threadIdx.x < 32) {
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const int c = ((i / V) * T + t) * V + i % V;
        if (c < a.cols) {
          p[c] = sum[i * 32 + t];
          p[a.cols + c] = sum[32 * EPT + i * 32 + t];
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int c = ((i / V) * T + t) * V + i % V;
      if (c < a.cols) {
        p[c] = dg[i];
        p[a.cols + c] = db[i];
      }
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
// partial rows split over its 8 warps and joined in warp order.
__global__ void __launch_bounds__(256) normJoin(const float* partial, int blocks, int cols, void* dgamma, void* dbeta,
                                                int ptype) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int which = blockIdx.y;
  float s = 0.f;
  if (c < cols)
    for (int b = w; b < blocks; b += 8) s += partial[(size_t)b * 2 * cols + (size_t)which * cols + c];
  part[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += part[i][lane];
    void* out = which ? dbeta : dgamma;
    if (out) storeParam(out, ptype, c, s);
  }
}

// ------------------------------------------------------------ host

constexpr int kWarpRowCols = 1024;  // a warp holds 32 lanes x 32 elements

struct Shape {
  bool vec, warp, held;
  int ept, threads, perBlock;
};
Shape normShape(int cols, int elem, bool aligned) {
  Shape s;
  const int v = 16 / elem;
  s.vec = aligned && cols % v == 0;
  s.held = cols <= kMaxHeldCols;
  s.warp = cols <= kWarpRowCols;
  if (s.warp) {
    s.ept = cols <= 256 ? 8 : cols <= 512 ? 16 : 32;
    s.threads = 128;
    s.perBlock = 4;
  } else {
    s.ept = cols <= 8192 ? 8 : cols <= 16384 ? 16 : 32;
    s.threads = std::max(64, ((cols + s.ept - 1) / s.ept + 31) / 32 * 32);
    s.perBlock = 1;
  }
  return s;
}
// Blocks that walk the rows of a backward pass, each with one row of partial sums.
int normBlocks(size_t rows, int cols) {
  const size_t groups = cols <= kWarpRowCols ? (rows + 3) / 4 : rows;
  return (int)std::min<size_t>(groups, (size_t)smCount() * 2);
}

using NormFn = void (*)(NormArgs);
template <int DT, bool VEC, bool WARP, bool FWD>
NormFn pickEpt(int ept) {
  if constexpr (FWD)
    return ept == 8 ? normForward<DT, VEC, 8, WARP> : ept == 16 ? normForward<DT, VEC, 16, WARP> : normForward<DT, VEC, 32, WARP>;
  else
    return ept == 8 ? normBackward<DT, VEC, 8, WARP> : ept == 16 ? normBackward<DT, VEC, 16, WARP> : normBackward<DT, VEC, 32, WARP>;
}
template <int DT, bool FWD>
NormFn pickShape(const Shape& s) {
  if (s.vec) return s.warp ? pickEpt<DT, true, true, FWD>(s.ept) : pickEpt<DT, true, false, FWD>(s.ept);
  return s.warp ? pickEpt<DT, false, true, FWD>(s.ept) : pickEpt<DT, false, false, FWD>(s.ept);
}
template <bool FWD>
NormFn pickKernel(int dt, const Shape& s) {
  if (!s.held) {
    if constexpr (FWD)
      return dt == vrcclFloat32 ? normForwardLong<vrcclFloat32>
             : dt == vrcclBfloat16 ? normForwardLong<vrcclBfloat16> : normForwardLong<vrcclFloat16>;
    else
      return dt == vrcclFloat32 ? normBackwardLong<vrcclFloat32>
             : dt == vrcclBfloat16 ? normBackwardLong<vrcclBfloat16> : normBackwardLong<vrcclFloat16>;
  }
  return dt == vrcclFloat32 ? pickShape<vrcclFloat32, FWD>(s)
         : dt == vrcclBfloat16 ? pickShape<vrcclBfloat16, FWD>(s) : pickShape<vrcclFloat16, FWD>(s);
}

bool goodSizes(size_t rows, size_t cols, int dtype, int ptype) {
  return rows < kMaxExtent && cols < (size_t(1) << 31) - 65536 && isOperatorType(dtype) && isOperatorType(ptype);
}

}  // namespace

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
  if (!goodMatrix(x, ldx, cols, E) || !goodMatrix(y, ldy, cols, E)) return vrcclInvalidArgument;
  if ((gamma && !goodVector(gamma, PE)) || (beta && !goodVector(beta, PE)) || (mean && !goodVector(mean, 4)) ||
      (rstd && !goodVector(rstd, 4)))
    return vrcclInvalidArgument;
  if (!(x == y && ldx == ldy) && overlap(x, spanBytes(ldx, rows, cols, E), y, spanBytes(ldy, rows, cols, E)))
    return vrcclInvalidArgument;
  const Shape s = normShape((int)cols, E, rowsAligned(x, ldx, E) && rowsAligned(y, ldy, E));
  NormArgs a = {};
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.ldx = ldx;
  a.ldy = ldy;
  a.rows = rows;
  a.cols = (int)cols;
  a.ptype = paramType;
  a.eps = eps;
  const size_t blocks = std::min<size_t>((rows + s.perBlock - 1) / s.perBlock, size_t(1) << 30);
  const int threads = s.held ? s.threads : 1024;
  pickKernel<true>(dtype, s)<<<(unsigned)blocks, threads, 0, (cudaStream_t)stream>>>(a);
  return launchResult();
}

extern "C" vrcclResult_t vrcclLayerNormWorkspace(size_t rows, size_t cols, size_t* bytes) {
  if (!bytes || !goodSizes(rows, cols, vrcclFloat32, vrcclFloat32)) return vrcclInvalidArgument;
  *bytes = size_t(normBlocks(rows, (int)cols)) * 2 * cols * sizeof(float);
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
  if (!goodMatrix(dy, lddy, cols, E) || !goodMatrix(x, ldx, cols, E) || !goodMatrix(dx, lddx, cols, E) ||
      !goodVector(mean, 4) || !goodVector(rstd, 4))
    return vrcclInvalidArgument;
  const size_t outSpan = spanBytes(lddx, rows, cols, E);
  if ((!(dx == dy && lddx == lddy) && overlap(dx, outSpan, dy, spanBytes(lddy, rows, cols, E))) ||
      (!(dx == x && lddx == ldx) && overlap(dx, outSpan, x, spanBytes(ldx, rows, cols, E))))
    return vrcclInvalidArgument;
  const int blocks = normBlocks(rows, (int)cols);
  if (weights && (!goodVector(workspace, 16) || workspaceBytes < size_t(blocks) * 2 * cols * sizeof(float)))
    return vrcclInvalidArgument;
  const Shape s = normShape((int)cols, E, rowsAligned(dy, lddy, E) && rowsAligned(x, ldx, E) && rowsAligned(dx, lddx, E));
  NormArgs a = {};
  a.x = x;
  a.dy = dy;
  a.gamma = gamma;
  a.y = dx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.partial = weights ? static_cast<float*>(workspace) : nullptr;
  a.ldx = ldx;
  a.lddy = lddy;
  a.ldy = lddx;
  a.rows = rows;
  a.cols = (int)cols;
  a.ptype = paramType;
  if (!s.held && weights) {
    const dim3 grid((unsigned)((cols + 255) / 256), (unsigned)blocks);
    if (dtype == vrcclFloat32)
      normColumns<vrcclFloat32><<<grid, 256, 0, st>>>(a);
    else if (dtype == vrcclBfloat16)
      normColumns<vrcclBfloat16><<<grid, 256, 0, st>>>(a);
    else
      normColumns<vrcclFloat16><<<grid, 256, 0, st>>>(a);
  }
  pickKernel<false>(dtype, s)<<<(unsigned)blocks, s.held ? s.threads : 1024, 0, st>>>(a);
  if (weights)
    normJoin<<<dim3((unsigned)((cols + 31) / 32), 2), 256, 0, st>>>(static_cast<const float*>(workspace), blocks,
                                                                    (int)cols, dgamma, dbeta, paramType);
  return launchResult();
}

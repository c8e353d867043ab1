// Building blocks of the operators a replica runs between two AllReduces
// (layer norm, linear layer, distillation loss): element access, reductions
// over a warp or a block, and the host checks they share.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "device_common.cuh"
#include "ops_rows.h"

namespace vrccl {

// Largest row count, row length and row stride an operator takes: products
// of two of them and an element size stay far inside 64 bits.
constexpr size_t kMaxExtent = size_t(1) << 40;

__host__ __device__ constexpr int floatTypeSize(int dt) { return dt == vrcclFloat32 ? 4 : 2; }
inline bool isOperatorType(int dt) { return dt == vrcclFloat32 || dt == vrcclBfloat16 || dt == vrcclFloat16; }

// A [rows, cols] operand: present, its address a multiple of its elements'
// size, its row stride no shorter than a row, and all of it within 2^46
// elements (so that no offset, in bytes, comes near 64 bits).
inline bool goodMatrix(const void* p, size_t ld, size_t rows, size_t cols, int elemSize) {
  return p && (uintptr_t)p % elemSize == 0 && ld >= cols && ld < kMaxExtent &&
         (rows == 0 || ld <= (size_t(1) << 46) / rows);
}
inline bool goodVector(const void* p, int elemSize) { return p && (uintptr_t)p % elemSize == 0; }
// Every row of a matrix starts on a 16-byte boundary.
inline bool rowsAligned(const void* p, size_t ld, int elemSize) {
  return ((uintptr_t)p | (uintptr_t)(ld * elemSize)) % 16 == 0;
}
// No output touches an input or another output. (An input that an output may
// take the place of is left out by its caller where it does.)
template <int O, int I>
inline bool apart(const Span (&out)[O], const Span (&in)[I]) {
  for (int i = 0; i < O; ++i) {
    for (int j = 0; j < I; ++j)
      if (overlap(out[i], in[j])) return false;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return false;
  }
  return true;
}
// `in`, unless `out` lies in its place.
inline Span unlessInPlace(const Span& in, size_t ldin, const void* out, size_t ldout) {
  return in.p == out && ldin == ldout ? vectorSpan(nullptr, 0) : in;
}

// A failed wait of the layer norm's kernels (each translation unit holds its own device-side word).
int normStatus(int* code);
// Multiprocessors of the current device (asked for once a device).
int smCount();
// Lets a kernel's blocks ask for all the dynamic shared memory there is on the current device; once a kernel and device.
vrcclResult_t allowSharedMemory(const void* fn);

// A kernel that may be launched while the one before it on its stream still
// runs (LaunchShape::after): waits for that one's results. And in the one before: the
// rest of this block's work needs no multiprocessor's worth of room, so the
// next kernel's blocks may come in and wait.
__device__ __forceinline__ void waitForPrevious() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void letNextIn() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Launch with a block's dynamic shared memory and cluster; `after`: without waiting for the stream's previous kernel to end
// (`fn` calls waitForPrevious() before it touches memory), so that the launch runs under that kernel.
struct LaunchShape {
  dim3 grid;
  int threads, smem, cluster;  // cluster: blocks, or 0
  bool after;
};
template <typename... Params, typename... Args>
vrcclResult_t launchShaped(void (*fn)(Params...), const LaunchShape& s, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = s.grid;
  cfg.blockDim = dim3((unsigned)s.threads);
  cfg.dynamicSmemBytes = (size_t)s.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (s.after) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (s.cluster) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = (unsigned)s.cluster;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (cudaLaunchKernelEx(&cfg, fn, Params(args)...) != cudaSuccess) {
    cudaGetLastError();
    return vrcclCudaError;
  }
  return vrcclSuccess;
}

// ------------------------------------------------------------ element access
// N consecutive elements of type DT as binary32. With N elements in 16 (or
// 8, 4) bytes one wide load; the caller guarantees the alignment.

template <int DT>
__device__ __forceinline__ float loadOne(const void* p, size_t i) {
  using S = typename Ty<DT>::S;
  return Ty<DT>::toF(reinterpret_cast<const S*>(p)[i]);
}
__device__ __forceinline__ float loadParam(const void* p, int dt, size_t i) {
  return dt == vrcclFloat32    ? reinterpret_cast<const float*>(p)[i]
         : dt == vrcclBfloat16 ? loadOne<vrcclBfloat16>(p, i)
                               : loadOne<vrcclFloat16>(p, i);
}
__device__ __forceinline__ void storeParam(void* p, int dt, size_t i, float x) {
  if (dt == vrcclFloat32)
    reinterpret_cast<float*>(p)[i] = x;
  else
    reinterpret_cast<unsigned short*>(p)[i] =
        dt == vrcclBfloat16 ? Ty<vrcclBfloat16>::fromF(x) : Ty<vrcclFloat16>::fromF(x);
}

// The two elements of a packed word (2-byte types).
template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (DT == vrcclBfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    return make_float2(Ty<DT>::toF((unsigned short)(w & 0xffffu)), Ty<DT>::toF((unsigned short)(w >> 16)));
  }
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  if constexpr (DT == vrcclBfloat16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// A 16-byte vector of elements <-> binary32.
template <int DT>
struct Vec16 {
  static constexpr int N = 16 / floatTypeSize(DT);
  static __device__ __forceinline__ void expand(const uint4& v, float (&f)[N]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (N == 4) {
        f[i] = __uint_as_float(w[i]);
      } else {
        const float2 p = unpack2<DT>(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
      }
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[N]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (N == 4)
        w[i] = __float_as_uint(f[i]);
      else
        w[i] = pack2<DT>(f[2 * i], f[2 * i + 1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Two binary32 values in one register pair: Blackwell adds and multiplies both
// in one instruction. The passes that read 2-byte elements are bound by issue
// slots nearly as much as by memory, and this halves their arithmetic.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// ------------------------------------------------------------ reductions

__device__ __forceinline__ float warpSum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float2 warpSum2(float2 x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
    x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
  }
  return x;
}
// Sums over a block of up to 32 warps, the result in every thread. `s` holds
// 32 entries; calls that follow one another take turns between two arrays, so
// that one barrier a call is enough.
__device__ __forceinline__ float2 blockSum2(float2 x, float2* s) {
  x = warpSum2(x);
  const int lane = threadIdx.x & 31, warps = (blockDim.x + 31) >> 5;
  if (lane == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  return warpSum2(lane < warps ? s[lane] : make_float2(0.f, 0.f));
}
__device__ __forceinline__ float blockSum(float x, float* s) {
  x = warpSum(x);
  const int lane = threadIdx.x & 31, warps = (blockDim.x + 31) >> 5;
  if (lane == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  return warpSum(lane < warps ? s[lane] : 0.f);
}

// The sum of `rows` values `stride` apart, one column a lane, the rows dealt to
// a block's 32 warps and joined in warp order; the result in warp 0.
__device__ __forceinline__ float columnSum(const float* p, int rows, size_t stride, bool exists) {
  __shared__ float part[32][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float s = 0.f;
  if (exists)
#pragma unroll 8
    for (int r = w; r < rows; r += 32) s += p[r * stride];
  part[w][lane] = s;
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += part[i][lane];
  }
  return s;
}

}  // namespace vrccl

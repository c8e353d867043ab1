// Rows that arrive in shared memory by bulk copies, several ahead, for the
// teams of threads that walk them (layer norm, RMS norm): the waits for them
// and how a team gives up.
#pragma once

#include "ops_common.cuh"

namespace vrccl {
namespace {

constexpr int kMaxStages = 8;
constexpr long long kRowWaitCycles = 3000000000ll, kDrainCycles = 200000000ll;  // a second and more

__device__ int gRingStatus;  // vrcclResult_t of the first device-side failure of this translation unit's kernels

// Sets *dead (givenUpWord) when the copy has not come after a time in which it must have.
__device__ __forceinline__ void waitRow(unsigned long long* bar, unsigned parity, int* dead, int turn,
                                        long long limit = kRowWaitCycles) {
  if (mbarTryWait(bar, parity)) return;
  const long long t0 = clock64();
  while (!mbarTryWait(bar, parity))
    if (clock64() - t0 > limit) {
      *reinterpret_cast<volatile int*>(dead) = givenUpWord(turn);
      return;
    }
}
// Given up with the ring at (stage, round): records it, and lets no copy that
// is in flight land after the block has gone.
__device__ __noinline__ void abandon(unsigned long long* full, int stages, int stage, int round, bool first, int* dead,
                                     int turn) {
  if (!first) return;
  atomicCAS(&gRingStatus, 0, (int)vrcclTimeout);
  for (int s = 0; s < stages; ++s) waitRow(&full[s], (round + (s < stage ? 1 : 0)) & 1, dead, turn, kDrainCycles);
}
__device__ __forceinline__ void expectBytes(unsigned long long* bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smemAddr(bar)), "r"(bytes) : "memory");
}

}  // namespace
}  // namespace vrccl

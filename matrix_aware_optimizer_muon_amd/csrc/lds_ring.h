// A ring of K stages in LDS, filled by direct-to-LDS loads: the loads, their
// waits and the barrier between stages, shared by the kernels that stage tiles
// so.
#pragma once

#include "device_common.h"

namespace muon {

// Wait until at most N vector-memory operations of this wave are pending
// (asm, so the compiler, which does not see the asm loads, keeps it).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Workgroup barrier for the stage ring.  A __syncthreads fence would also
// wait for every direct-to-LDS load in flight (they count as LDS writes)
// and drain the ring; here each wave only completes its own LDS reads
// (lgkmcnt(0): the buffer refilled after the barrier was read before it),
// and callers wait for the loads they need with wait_vmcnt.  The asm
// memory clobbers keep the compiler from moving memory accesses across.
__device__ __forceinline__ void ring_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Direct-to-LDS load: lane l's 16 bytes at base + voff go to lds + 16 l.
// The instruction is written as inline asm (it has no register result): the
// compiler treats the builtin form as an LDS store and puts a wait for every
// outstanding vector-memory operation in front of the next LDS read, which
// would drain the ring.  The stage waits are therefore explicit
// (wait_vmcnt), and the asm's memory clobber keeps LDS accesses in order
// around it.  The load needs one wait state behind the write of M0, which the
// compiler puts between its own instructions but not into an asm block.
__device__ __forceinline__ void dma16(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(lds)
               : "memory", "m0");
}

// LDS byte address of a shared-memory pointer.
template <typename E>
__device__ __forceinline__ uint32_t lds_addr(const E* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const E*)(p)));
}

}  // namespace muon

// ptx_stream.cuh -- what kernels that pass over memory use: launches that overlap, asynchronous copies, products of packed
// fp32 pairs.  Apart from ptx.cuh, which the attention's forward and backward are made of.
#pragma once

#include <cstdint>

namespace attn {
namespace ptx {

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// 16 bytes from global to shared memory without registers; `there` false writes zeros and reads nothing (a predicate: a
// size in a register took 13 instructions a row more).  A thread's copies since its last commit are a group, and it sees
// them once at most kLeft later groups are under way.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool there) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %2, 0;\n\tcp.async.cg.shared.global [%0], [%1], 16, p;\n\t}" ::"r"(dst), "l"(src),
                 "r"((uint32_t)there)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Launched with the attribute that lets its blocks start while the kernel before still runs: `launch_next` lets the kernel after
// do so too, `wait_previous` ends when everything before has ended and is visible.  Nothing global is read or written
// before that, and nothing that a kernel before may have written is read through the non-coherent path (__ldg), which
// asks for data that stays the same from the launch on.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace ptx
}  // namespace attn

// ptx_cache.cuh -- the inline-PTX wrappers that only the cache kernels need,
// beside ptx.cuh: 8- and 16-column TMEM loads and stores, E4M3 products with
// both operands in shared memory for either operand order, and block-level
// votes.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace attn {
namespace ptx {

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// N consecutive columns (8, 16 or 32) of the warp's 32 lanes, and the wait
// for them: no use of the registers is scheduled before it.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t* r) {
    if constexpr (N == 8) tmem_ld8(taddr, r);
    if constexpr (N == 16) tmem_ld16(taddr, r);
    if constexpr (N == 32) tmem_ld32(taddr, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t* r) {
    if constexpr (N == 8) tmem_st8(taddr, r);
    if constexpr (N == 16) tmem_st16(taddr, r);
    if constexpr (N == 32) tmem_st32(taddr, r);
    tmem_st_wait();
}

// One E4M3 product step (K = 32), A and B in shared memory.
__device__ __forceinline__ void mma_ss_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Four steps over 128 keys, the operands' descriptors advancing by kA and kB
// (in 16-byte units) each.
template <int kA, int kB>
__device__ __forceinline__ void mma_ss_f8_x4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "add.s64 a, %1, %5; add.s64 b, %2, %6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t"
        "add.s64 a, a, %5; add.s64 b, b, %6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t"
        "add.s64 a, a, %5; add.s64 b, b, %6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(kA), "n"(kB)
        : "memory");
}
// Instruction descriptor for kind::f8f6f4, E4M3 A and B, fp32 D; bit 15: A is
// MN-major, bit 16: B is.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn) {
    return idesc_e4m3_f32(M, N, b_mn) | (a_mn ? 1u << 15 : 0u);
}
// Instruction descriptor for kind::f16, f16 A (K-major) and B, fp32 D; bit 16: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Two floats -> packed f16x2 (round to nearest even); `lo` in bits 0-15.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Shared-memory descriptor of an operand with rows of 128, 64 or 32 bytes in the
// swizzle of that width (16-byte piece i of row k sits at i ^ (k mod 8), i ^
// (k / 2 mod 4) or i ^ (k / 4 mod 2)), groups of eight rows next to each other;
// fields as in sdesc_sw128, layout 2, 4 or 6.
template <int kRowBytes>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t saddr) {
    static_assert(kRowBytes == 128 || kRowBytes == 64 || kRowBytes == 32, "swizzled rows");
    constexpr uint64_t layout = kRowBytes == 128 ? 2 : kRowBytes == 64 ? 4 : 6;
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(8 * kRowBytes >> 4) << 32) | (1ull << 46) |
           (layout << 61);
}

// mbar_wait (ptx.cuh) as a first probe in place and a call for the rest: the
// cache kernels wait in many places, and their roles share an instruction cache.
// The clock is read only after many probes: a read of the global timer takes
// longer than most waits.
__device__ __noinline__ bool mbar_wait_rest(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                            unsigned int* status, uint64_t limit_ns) {
    uint64_t t0 = 0;
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        const uint64_t t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > limit_ns) {
            *abort_flag = 1;
            atomicOr(status, kStatusTimeout);
            return false;
        }
    }
}
__device__ __forceinline__ bool mbar_wait_call(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                               unsigned int* status, uint64_t limit_ns) {
    return mbar_test_wait(bar, parity) || mbar_wait_rest(bar, parity, abort_flag, status, limit_ns);
}

// Launched with the attribute that lets its blocks start while the kernel before still runs: `launch_next` lets the kernel after
// do so too, `wait_previous` ends when everything before has ended and is visible.  Nothing global is read or written
// before that, and nothing that a kernel before may have written is read through the non-coherent path (__ldg), which
// asks for data that stays the same from the launch on.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void bar_sync(int id, int threads) {
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Barrier over `threads` threads that tells each whether any of them passed true.
__device__ __forceinline__ bool bar_any(int id, int threads, bool x) {
    uint32_t any;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)x), "r"(id), "r"(threads)
        : "memory");
    return any != 0;
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(x));
    return x != 0;
}
__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t x) {
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace ptx
}  // namespace attn

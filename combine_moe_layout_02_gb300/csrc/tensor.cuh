// tensor.cuh -- what the tcgen05 products share (product.cu, product_int8.cu): bounded
// waits of whole warps on barriers of a CTA pair, descriptors, tensor memory to
// bf16 rows, and the encoder of tensor maps.
//
// A kernel's barriers B hold a word `abort`, its arguments A the error word `err`
// and the bound `wait_cycles` of a wait.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "experts.cuh"

namespace moe {

constexpr long long kWaitCycles = 1ll << 32;  // bound of a wait, about two seconds

// Arrival on a barrier of the leading CTA, released at the CTA's scope (at the cluster's it
// waits for all that the thread has stored: about a microsecond per tile where a thread stores
// results, 128 tokens, 1024 -> 14336: 456 us against 299). It hands over
// - tensor memory that has been read: ordered by the tcgen05 fences, no data;
// - in product_int8.cu also operands of the arriving CTA, f16 rows in its shared memory and weights in its
//   tensor memory, for an instruction that the leading CTA issues. The scope alone does not promise those to
//   another CTA. No thread of the other CTA reads them, though: each SM's tensor core reads its own SM's
//   memories, of which there is no second copy, and before the arrival every writer has completed the proxy fence (rows) and
//   tcgen05.wait::st (weights), so nothing is on its way when the arrival leaves.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// A wait has run out: the CTA's other roles are told, and the caller.
template <typename B, typename A>
__device__ __forceinline__ void give_up(B* b, const A& a) {
    *reinterpret_cast<volatile uint32_t*>(&b->abort) = 1u;
    raise_error(a.err, MOE_ERR_DEVICE_TIMEOUT);
}

// Bounded wait of a whole warp, by polls and by time (about two seconds: a poll
// may itself sleep); false if it ran out or another role of the CTA gave up.
template <bool CLUSTER, typename B, typename A>
__device__ __forceinline__ bool wait_in(B* b, uint64_t* bar, uint32_t parity, const A& a) {
    auto done = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    if (__all_sync(0xffffffffu, done())) return true;
    const long long began = clock64();
    for (uint32_t i = 0; i < kSpinLimit; ++i) {
        if (__all_sync(0xffffffffu, done())) return true;
        if (__any_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(&b->abort) != 0u)) return false;
        if (__any_sync(0xffffffffu, clock64() - began > a.wait_cycles)) break;
    }
    give_up(b, a);
    return false;
}
template <typename B, typename A>
__device__ __forceinline__ bool wait_for(B* b, uint64_t* bar, uint32_t parity, const A& a) {
    return wait_in<true>(b, bar, parity, a);
}
// The same, acquiring at the CTA's scope: for what this CTA's own threads, loads and
// products hand over, and for tensor memory.
template <typename B, typename A>
__device__ __forceinline__ bool wait_here(B* b, uint64_t* bar, uint32_t parity, const A& a) {
    return wait_in<false>(b, bar, parity, a);
}

// Arrival on a barrier of this CTA.
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Whether all 128 threads that meet at barrier `id` say so.
__device__ __forceinline__ bool all_agree(int id, bool yes) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "bar.red.and.pred q, %1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(id), "r"(static_cast<uint32_t>(yes))
        : "memory");
    return all != 0;
}

// After a failed wait: what is in flight ends within microseconds, or (a peer
// gave up first) never.
__device__ __forceinline__ void drained(uint64_t* bar, uint32_t parity) {
    const long long began = clock64();
    while (!__any_sync(0xffffffffu, mbar_try_wait_cluster(bar, parity)) &&
           !__any_sync(0xffffffffu, clock64() - began > kWaitCycles / 64)) {
    }
}

// One lane of a converged warp. The loading and the issuing warp run their
// loops as whole warps on warp-uniform values and only the instructions
// themselves are one lane's: in a branch of one lane the compiler cannot keep
// descriptors in uniform registers, and each product then took about 100
// cycles to issue and each scale copy 80 (of 128 cycles of work; measured).
__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

__device__ __forceinline__ int32_t uniform(int32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Shared-memory matrix descriptor: rows of 128 bytes, swizzled, 8 rows to 1024 bytes.
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// Arrives on `bar` of both CTAs once every product and copy issued so far is done.
__device__ __forceinline__ void commit_to(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 lanes x 16 columns of tensor memory: v[4 i + j], column 8 i + 2 (lane % 4) + j % 2,
// lane row lane / 4 + 8 (j / 2).
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(addr)
                 : "memory");
}

// Four 8 x 8 blocks of 16-bit values, transposed: lane 8 q + j gives the address
// of the 16 bytes that column j of block q goes to.
__device__ __forceinline__ void store_turned(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// silu(g) * u. e^-|g| <= 1, so nothing overflows and the denominator is in [1, 2].
// The hardware's exponential and quotient are off by 2 + 1.173 |g| and 2 units, far below the result's rounding to bf16; expf and a
// rounded division change no digit of the int8 chain's error (500 rows 7168 -> 2048 -> 7168: 0.0018 against 64 bits, as binary32 torch) and cost
// 262144 rows 7168 -> 4096 9.2 ms against 8.2.
__device__ __forceinline__ float gate_times_up(float g, float u) {
    const float e = __expf(-fabsf(g));
    return __fdividef(g < 0.f ? g * e : g, 1.f + e) * u;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The CUDA driver's encoder, looked up once per process.
inline EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

}  // namespace moe

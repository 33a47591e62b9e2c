// kda_mla_sm100.cuh -- what the latent-attention kernels add to kda_sm100.cuh: tensor-core products of bf16 and
// e4m3 operands (kind::f16, kind::f8f6f4), untiled bulk copies, and bounded waits that end together.
#pragma once

#include "kda.h"
#include "kda_common.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace sm100 {

// Instruction descriptors with fp32 accumulation for bf16 and e4m3 operands.  a_mn / b_mn: the operand is stored
// MN-major (M or N contiguous) instead of K-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn) {
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// K = 16 bf16 values, both operands in shared memory
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// A in tensor memory: lane = row, each 32-bit column two consecutive values along K
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// K = 32 e4m3 values
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Shared-memory matrix descriptor for 64-byte rows with the 64-byte swizzle (offsets as in sw128_desc).
__device__ __forceinline__ uint64_t sw64_desc(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((lbo_bytes >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>((sbo_bytes >> 4) & 0x3FFFu) << 32;
    d |= static_cast<uint64_t>(1) << 46;  // version
    d |= static_cast<uint64_t>(4) << 61;  // swizzle 64B
    return d;
}
// Byte offset of byte `col` of row `row` in a tile of 64-byte rows whose 16-byte chunks are permuted by XOR with
// (row / 2 % 4) (tile base 512-byte aligned).
__device__ __forceinline__ uint32_t sw64_byte(int row, int col) {
    return static_cast<uint32_t>(row * 64 + ((((col >> 4) ^ (row >> 1)) & 3) << 4) + (col & 15));
}

// Registers -> tensor memory: 32 lanes x 16 consecutive 32-bit columns per warp.
__device__ __forceinline__ void tmem_st16_nw(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

__device__ __forceinline__ void tmem_st32_nw(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
                 "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
                 "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
                 : "memory");
}

// 16 lanes read twice, as tmem_ld16_x2, without waiting.
template <int SPLIT>
__device__ __forceinline__ void tmem_ld16_x2_nw(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], %17;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr), "n"(SPLIT));
}

template <int SPLIT>
__device__ __forceinline__ void tmem_ld8_x2_nw(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], %9;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr), "n"(SPLIT));
}

// One lane of a converged warp.  Products issued under this predicate keep their descriptors in uniform registers:
// 64 x 32 x 16 products measured 31 cycles apart, against 56 under a lane == 0 test.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(p));
    return p != 0u;
}

// Untiled copy into shared memory (16-byte aligned addresses and size), counted in bytes on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// The waits of a block whose warps have different roles.  A wait that gives up (after `polls` polls or 2 s) raises
// KDA_DEVFLAG_TIMEOUT and the block's abort word, at which every other wait of the block gives up too, so that
// all roles leave their loops, drain what they have in flight (drain(), default bound) and meet at the end.  Only the
// first look is inlined: with some thirty waits in a kernel, the loops would be most of its code, and warps would stand
// without instructions.
struct RoleWait {
    uint32_t polls;
    volatile uint32_t* abort_word;  // shared memory
    unsigned int* flags;

    __device__ __noinline__ static bool keep_looking(uint64_t* bar, uint32_t parity, uint32_t polls,
                                                     volatile uint32_t* abort_word, unsigned int* flags) {
        WaitBudget budget;
        bool done = false;
        for (uint32_t i = 1; i < polls; ++i) {
            done = mbar_poll(bar, parity);
            if (done || ((i & 7u) == 7u && *abort_word != 0u) || budget.expired()) break;
        }
        done = __all_sync(0xffffffffu, done);
        if (!done) {
            *abort_word = 1u;
            raise_flag(flags, KDA_DEVFLAG_TIMEOUT);
        }
        return done;
    }
    // For a converged warp, whose lanes all look and get the same answer.  (One lane that looks for all, the others waiting
    // for it, took 35% longer in kda_mla_prefill.cu: the hardware suspends a whole warp at a barrier, not one lane.)
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        if (polls > 0 && __all_sync(0xffffffffu, mbar_poll(bar, parity))) return true;
        return keep_looking(bar, parity, polls, abort_word, flags);
    }
    // Two barriers, looked at together: a look takes some 250 cycles beside busy warps.
    __device__ __forceinline__ bool both(uint64_t* one, uint32_t one_parity, uint64_t* two, uint32_t two_parity) const {
        if (polls > 0) {
            const bool first = mbar_poll(one, one_parity), second = mbar_poll(two, two_parity);
            if (__all_sync(0xffffffffu, first && second)) return true;
        }
        return keep_looking(one, one_parity, polls, abort_word, flags) &&
               keep_looking(two, two_parity, polls, abort_word, flags);
    }
};
static __device__ __noinline__ void drain(uint64_t* bar, uint32_t parity) { mbar_wait(bar, parity, 1u << 26); }

// Byte offset of byte `col` of row `row` in a tile of 128-byte rows whose 16-byte chunks are permuted by XOR with
// (row % 8): the 128-byte swizzle of TMA and of the matrix descriptors (tile base 1024-byte aligned).
__device__ __forceinline__ uint32_t sw128_byte(int row, int col) {
    return static_cast<uint32_t>(row * 128 + ((((col >> 4) ^ row) & 7) << 4) + (col & 15));
}

}  // namespace sm100
}  // namespace kda

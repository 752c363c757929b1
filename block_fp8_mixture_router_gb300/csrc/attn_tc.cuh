// Tensor-core and TMA helpers of the attention kernels, beside tc_ptx.cuh.
#pragma once

#include "attn_device.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace tc {

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// This thread's shared-memory writes before an async-proxy read of them (an MMA's
// operands) that a later barrier arrival releases.
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

__device__ __forceinline__ void wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

#define MOE_TC_O8(v, o)                                                                 \
  "=r"(v[o + 0]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]),       \
      "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define MOE_TC_I8(v, o)                                                                 \
  "r"(v[o + 0]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]),            \
      "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])

// 8, 16 or 32 consecutive columns of this warp's TMEM lanes, not waited for.
__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
      : MOE_TC_O8(v, 0)
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];\n"
      : MOE_TC_O8(v, 0), MOE_TC_O8(v, 8)
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : MOE_TC_O8(v, 0), MOE_TC_O8(v, 8), MOE_TC_O8(v, 16), MOE_TC_O8(v, 24)
      : "r"(taddr)
      : "memory");
}

// 8, 16 or 32 consecutive columns of this warp's TMEM lanes; wait_st() completes it.
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr),
      MOE_TC_I8(v, 0)
      : "memory");
}

__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};\n" ::"r"(taddr),
      MOE_TC_I8(v, 0), MOE_TC_I8(v, 8)
      : "memory");
}

__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(
          taddr),
      MOE_TC_I8(v, 0), MOE_TC_I8(v, 8), MOE_TC_I8(v, 16), MOE_TC_I8(v, 24)
      : "memory");
}

#undef MOE_TC_O8
#undef MOE_TC_I8

// Shared-memory matrix descriptor under the 128- or the 64-byte swizzle.  K-major
// (rows of 128 or 64 bytes along K): the 8-row atoms lie 1024 or 512 bytes apart.
// M-major (rows of 128 or 64 bytes along M, one for each k): the groups of 8 k lie
// as far apart; `next_m` is the offset to the M values behind the row.
__device__ __forceinline__ uint64_t swz_desc(uint32_t saddr, bool wide, uint32_t next_m = 16) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(next_m >> 4) << 16) |
         ((uint64_t)((wide ? 1024 : 512) >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)(wide ? 2 : 4) << 61);
}

// MMAs and commits issued by the lane whose `leader` is set, of a warp that runs them in
// uniform control flow.  Descriptors are taken apart into the changing low word (start
// address and the offset to the next M or N) and the constant high one, and the leader is
// found once: an MMA that looks up its lane and builds its descriptors in 64 bits takes
// the issuing warp about 75 cycles, more than the product takes the tensor cores.
struct Desc {
  uint32_t lo, hi;
};

__device__ __forceinline__ Desc desc_of(uint32_t saddr, bool wide, uint32_t next_m = 16) {
  const uint64_t d = swz_desc(saddr, wide, next_m);
  return Desc{(uint32_t)d, (uint32_t)(d >> 32)};
}

// The same operand `bytes` further on.
__device__ __forceinline__ Desc operator+(Desc d, uint32_t bytes) {
  return Desc{d.lo + (bytes >> 4), d.hi};
}

template <bool kF8>
__device__ __forceinline__ void mma_ss(uint32_t d, Desc a, Desc b, uint32_t idesc,
                                       uint32_t accumulate, uint32_t leader) {
  if constexpr (kF8)
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 x, y;\n setp.ne.b32 p, %6, 0;\n setp.ne.b32 e, %7, 0;\n"
        " mov.b64 x, {%1, %2};\n mov.b64 y, {%3, %4};\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %5, p;\n}\n" ::"r"(d),
        "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 x, y;\n setp.ne.b32 p, %6, 0;\n setp.ne.b32 e, %7, 0;\n"
        " mov.b64 x, {%1, %2};\n mov.b64 y, {%3, %4};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n}\n" ::"r"(d),
        "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}

// A in tensor memory, fp16.
__device__ __forceinline__ void mma_ts_f16(uint32_t d, uint32_t a, Desc b, uint32_t idesc,
                                           uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 e, %6, 0;\n"
      " mov.b64 y, {%2, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}

__device__ __forceinline__ void commit_by(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_u32(bar)),
      "r"(leader)
      : "memory");
}

// Instruction descriptor bits beside idesc_f8: A stored M-major, B of type e5m2.
constexpr uint32_t kIdescAMajorM = 1u << 15;
constexpr uint32_t kIdescBE5m2 = 1u << 10;

}  // namespace tc
}  // namespace moe

// Packed codes as fp16 levels, and the operands made of them: helpers of the
// tensor-core kernels that dequantise to fp16 (shared-prefix attention,
// attention weights).
#pragma once
#include <type_traits>

#include "common.cuh"
#include "tc_decode.cuh"
#include "tc_ptx.cuh"

namespace fsq {
namespace tc {

using namespace ptx;

// A ring position: slot and the parity of its current round.
struct Ring {
  int slot = 0;
  uint32_t par = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      par ^= 1u;
    }
  }
};

// Bounded waits of a whole warp, with one answer: its lanes leave a loop
// together, also when some of them saw the phase complete and others the abort.
__device__ __forceinline__ bool warp_wait(uint64_t *b, uint32_t par, volatile uint32_t *abort, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, wait_bar(b, par, abort, limit_ns));
}
__device__ __forceinline__ bool warp_wait(uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1,
                                          volatile uint32_t *abort, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, wait_bars(b0, p0, b1, p1, abort, limit_ns));
}

// Waits for this thread's tcgen05.ld's; the registers they fill may not be used
// before, also where other work stands between a load and its wait.
#define FSQ_RW8(a, o) "+r"(a[o + 0]), "+r"(a[o + 1]), "+r"(a[o + 2]), "+r"(a[o + 3]), "+r"(a[o + 4]), "+r"(a[o + 5]), "+r"(a[o + 6]), "+r"(a[o + 7])
__device__ __forceinline__ void tmem_ld_wait16(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : FSQ_RW8(r, 0), FSQ_RW8(r, 8)::"memory");
}
// More registers of loads that such a wait covers.
__device__ __forceinline__ void tmem_held16(uint32_t *r) { asm volatile("" : FSQ_RW8(r, 0), FSQ_RW8(r, 8)); }

// f(std::integral_constant<int, n>) for n in [LO, HI]: a loop whose step count the
// compiler knows, for a count known at launch.
template <int LO, int HI, class F>
__device__ __forceinline__ void with_count(int n, F f) {
  if constexpr (LO == HI) {
    f(std::integral_constant<int, LO>());
  } else {
    constexpr int MID = (LO + HI) / 2;
    if (n <= MID) with_count<LO, MID>(n, f);
    else with_count<MID + 1, HI>(n, f);
  }
}

// 128-byte-swizzled operand B of an MMA, as the two words of its descriptor.
// K-major: atoms of 8 rows are 1024 bytes apart (lbo unused).  MN-major: atoms
// of 64 MN-coordinates are `lbo` bytes apart, groups of 8 along K 1024 bytes.
// Moving along the operand adds (bytes / 16) to the low word.
constexpr uint32_t kSwzHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t swz_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }

// D[tmem] (+)= A[tmem] B[smem], run by a whole converged warp and issued by its
// elected lane (el != 0).  An MMA takes its operands from uniform registers: with
// the warp converged, constant steps and a base column that is known to be 0, a
// step costs a few uniform additions and the tensor core runs at its rate (32
// cycles for N = 64, K = 16; from one diverged lane, with descriptors in ordinary
// registers, the same loop issued one every 85-180 cycles).
__device__ __forceinline__ void mma_ts_warp(uint32_t el, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kSwzHi), "r"(el)
      : "memory");
}
// D[tmem] (+)= A[smem] B[smem], both operands K-major atoms; issued alike.
__device__ __forceinline__ void mma_ss_warp(uint32_t el, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kSwzHi), "r"(el)
      : "memory");
}

__device__ __forceinline__ uint32_t hfma2(uint32_t x, uint32_t m, uint32_t a) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&m),
                            *reinterpret_cast<const __half2 *>(&a));
  return *reinterpret_cast<const uint32_t *>(&r);
}
// fp16 pairs as constants
constexpr uint32_t kOne = 0x3C003C00u;
template <int BITS>
__host__ __device__ constexpr int order_of(int c) {  // physical place of coordinate c in its group of 8
  return BITS == 8 ? c : (c & 3) * 2 + (c >> 2);
}

// Eight codes -> four words of fp16 levels in physical order.  BITS = 8: w and
// w2 hold codes 0-3 and 4-7; 4: w holds all; 2: the low 16 bits of w.
template <int BITS>
__device__ __forceinline__ uint4 levels8(uint32_t w, uint32_t w2) {
  constexpr uint32_t M = 0x64006400u;  // 1024.0, whose last mantissa bits take the code
  if constexpr (BITS == 8) {
    constexpr uint32_t kOff = 0xE480E480u;  // -1152 = -(1024 + 128)
    return make_uint4(hfma2(__byte_perm(w, M, 0x7150), kOne, kOff), hfma2(__byte_perm(w, M, 0x7352), kOne, kOff),
                      hfma2(__byte_perm(w2, M, 0x7150), kOne, kOff), hfma2(__byte_perm(w2, M, 0x7352), kOne, kOff));
  } else if constexpr (BITS == 4) {
    const uint32_t v = w >> 8;
    // codes at bit 0: 1024 + n - 1032; at bit 4: (1024 + 16 n) / 16 - 72
    return make_uint4(hfma2((w & 0x000F000Fu) | M, kOne, 0xE408E408u), hfma2((w & 0x00F000F0u) | M, 0x2C002C00u, 0xD480D480u),
                      hfma2((v & 0x000F000Fu) | M, kOne, 0xE408E408u), hfma2((v & 0x00F000F0u) | M, 0x2C002C00u, 0xD480D480u));
  } else {
    const uint32_t v = (w & 0xFFFFu) | (w << 8);  // codes 4-7 beside codes 0-3, 16 bits up
    // code k at bit 2k: (1024 + 4^k n) / 4^k - (1024 / 4^k + 2)
    return make_uint4(hfma2((v & 0x00030003u) | M, kOne, 0xE402E402u), hfma2((v & 0x000C000Cu) | M, 0x34003400u, 0xDC08DC08u),
                      hfma2((v & 0x00300030u) | M, 0x2C002C00u, 0xD420D420u), hfma2((v & 0x00C000C0u) | M, 0x24002400u, 0xCC80CC80u));
  }
}

// The BITS bytes of group u (8 codes) of the token at `row`, whose address and
// whose neighbours' are multiples of `align`
template <int BITS>
__device__ __forceinline__ void group_words(const uint8_t *row, int u, int align, uint32_t (&w)[2]) {
  const uint8_t *p = row + u * BITS;
  w[0] = w[1] = 0u;
  if (align >= 4 && BITS >= 4) {
#pragma unroll
    for (int i = 0; i < BITS / 4; ++i) w[i] = *reinterpret_cast<const uint32_t *>(p + 4 * i);
  } else if (align >= 2) {
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i) w[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(p + 2 * i) << (16 * (i & 1));
  } else {
#pragma unroll
    for (int i = 0; i < BITS; ++i) w[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
  }
}

}  // namespace tc
}  // namespace fsq

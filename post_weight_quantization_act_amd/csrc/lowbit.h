// What the kernels of the low-bit layers share: codes to 16-bit integers c - z, matrix
// instructions on 16-byte fragments, transfers from memory into LDS.
#pragma once

#include <type_traits>

#include "common.h"

namespace awq {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf162v __attribute__((ext_vector_type(2)));

// The AND-OR of the unpacking as one v_and_or_b32, mask in an SGPR and
// exponent in a VGPR.  Written out because the compiler splits (w & mask) |
// expo into a v_and_b32 and a v_or_b32 with literal operands, which measured
// slower (the 70B decode call took 36.5 us that way, 30.3 us with the single
// instruction).
// The constants come from magic_ops(), built once per kernel.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t smask, uint32_t vexpo) {
  uint32_t r;
  asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(w), "s"(smask), "v"(vexpo));
  return r;
}

// Masks (SGPRs) and exponents (VGPRs) of the window offsets sh = BITS t.
template <int BITS, int N>
struct MagicOps {
  uint32_t mask[N];
  uint32_t expo[N];
};
template <int BITS, int N>
__device__ __forceinline__ MagicOps<BITS, N> magic_ops() {
  MagicOps<BITS, N> o;
#pragma unroll
  for (int t = 0; t < N; ++t) {
    asm("s_mov_b32 %0, %1" : "=s"(o.mask[t]) : "i"(((1u << BITS) - 1u) << (BITS * t)));
    asm("v_mov_b32 %0, %1" : "=v"(o.expo[t]) : "i"((uint32_t)(150 - BITS * t) << 23));
  }
  return o;
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Buffer resource of a raw byte range: loads at offsets >= num_bytes return 0.
__device__ __forceinline__ i32x4 byte_range(const void* base, uint32_t num_bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  return i32x4{(int)(uint32_t)b, (int)(uint32_t)(b >> 32), (int)num_bytes, 0x00020000};
}

// 16 bytes per lane from rsrc + voff into LDS at lds_addr + 16 * lane.  Inline
// asm, so that the compiler does not wait for every transfer before each LDS
// read; the kernel waits with explicit counts.  m0 is declared clobbered (the
// compiler keeps nothing of its own in it across the transfer and pads its own
// next use), and the SALU write of m0 gets the one wait state an LDS-DMA load
// needs before it reads m0.  clang warns about any reserved register in a
// clobber list; the clobber is honoured all the same.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void to_lds16(i32x4 rsrc, uint32_t lds_addr, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds_addr), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Wait until at most n transfers of this lane are outstanding.
template <int n>
__device__ __forceinline__ void vm_wait() {
  static_assert(n >= 0 && n < 64, "vmcnt is 6 bits");
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}

template <typename S>
__device__ __forceinline__ f32x16 mfma32(i32x4 a, i32x4 b, f32x16 c);
template <>
__device__ __forceinline__ f32x16 mfma32<_Float16>(i32x4 a, i32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a),
                                                __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16 mfma32<__bf16>(i32x4 a, i32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <typename S>
__device__ __forceinline__ f32x4 mfma16x32(i32x4 a, i32x4 b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mfma16x32<_Float16>(i32x4 a, i32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mfma16x32<__bf16>(i32x4 a, i32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <int BITS>
struct QuarterWindows {
  static constexpr int kPer = (23 - BITS) / BITS + 1;   // codes per window
};
template <int BITS>
using QuarterOps = MagicOps<BITS, QuarterWindows<BITS>::kPer>;

// Code T of 16 consecutive ones held in bits [T BITS, T BITS + BITS) of sw.
template <int BITS, int NW, int T>
__device__ __forceinline__ uint32_t code_in(const uint32_t (&sw)[NW]) {
  constexpr int b = T * BITS, w = b >> 5, o = b & 31;
  constexpr uint32_t mask = (1u << BITS) - 1u;
  if constexpr (o + BITS <= 32) return (sw[w] >> o) & mask;
  else return __builtin_amdgcn_alignbit(sw[w + 1], sw[w], o) & mask;
}

// Code T of the run as fp32 (c - z) in the magic-exponent form of the
// quarter unpacking: windows of QuarterWindows<BITS>::kPer codes start at code
// boundaries, sub[sh / BITS] = 2^(23 - sh) + z.
template <int BITS, int NW, int T>
__device__ __forceinline__ float small_cz(const uint32_t (&sw)[NW], const float* sub,
                                          const QuarterOps<BITS>& ops) {
  constexpr int kPer = QuarterWindows<BITS>::kPer;
  constexpr int w0 = (T / kPer) * kPer * BITS, wi = w0 >> 5, o = w0 & 31;
  constexpr int sh = T * BITS - w0;
  uint32_t win;
  if constexpr (o == 0) win = sw[wi];
  else if constexpr (wi + 1 >= NW || o + sh + BITS <= 32) win = sw[wi] >> o;
  else win = __builtin_amdgcn_alignbit(sw[wi + 1], sw[wi], o);
  return __uint_as_float(and_or(win, ops.mask[sh / BITS], ops.expo[sh / BITS])) - sub[sh / BITS];
}

// Codes 2P and 2P + 1 of the run as two S values (c - z), exact.
template <typename S, int BITS, int NW, int P>
__device__ __forceinline__ int small_pair(const uint32_t (&sw)[NW], half2v negz, const float* sub,
                                          const QuarterOps<BITS>& ops) {
  if constexpr (std::is_same<S, _Float16>::value) {
    const uint32_t c0 = code_in<BITS, NW, 2 * P>(sw), c1 = code_in<BITS, NW, 2 * P + 1>(sw);
    const uint32_t v = c0 | (c1 << 16) | 0x64006400u;
    return (int)__builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, v) + negz);
  } else {
    // small integers are exact in fp32 and their upper halves are exact bf16
    const float f0 = small_cz<BITS, NW, 2 * P>(sw, sub, ops);
    const float f1 = small_cz<BITS, NW, 2 * P + 1>(sw, sub, ops);
    return (int)__builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u);
  }
}

}  // namespace awq

// What the wide GEMMs and the tiled projection share: int4 codes -> bf16
// weights w = q s + b with one rounding, and buffer loads.
#pragma once

#include "device.h"

namespace moe {

struct WideExpand {
  uint32_t mask_lo, magic;  // 0x000F000F, fp16 1024 | 1024
};

// Hidden from the optimiser so that (w & mask) | magic is selected as one
// bitwise three-input op with register operands.
__device__ inline WideExpand wide_expand_consts() {
  WideExpand k;
  asm volatile("v_mov_b32 %0, 0x000F000F" : "=v"(k.mask_lo));
  asm volatile("v_mov_b32 %0, 0x64006400" : "=v"(k.magic));
  return k;
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Per column and group: the scale s and the offset b - 1024 s (exact in fp32
// for the bf16 inputs' exponent spans).
struct ColAffine {
  float s, c;
};

__device__ inline ColAffine col_affine(float s, float b) {
  return ColAffine{s, __builtin_fmaf(-1024.0f, s, b)};
}

// One packed word (eight codes of one column, k = 8 consecutive inputs, code
// o at nibble (o & 1) * 4 + (o >> 1)) -> the eight bf16 weights in k order:
// ((w >> 4d) & 0x000F000F) | 0x64006400 is the fp16 pair (1024 + q_2d,
// 1024 + q_2d+1), and (1024 + q) s + (b - 1024 s) = q s + b with one rounding;
// expand_bf16x2 forms the d-th pair.
__device__ inline uint32_t expand_bf16x2(uint32_t w, int d, const ColAffine& c, const WideExpand& k) {
  const f16x2 h = __builtin_bit_cast(f16x2, ((w >> (4 * d)) & k.mask_lo) | k.magic);
  return pack_bf16x2(__builtin_fmaf((float)h.x, c.s, c.c), __builtin_fmaf((float)h.y, c.s, c.c));
}

__device__ inline u32x4 expand_bf16(uint32_t w, const ColAffine& c, const WideExpand& k) {
  u32x4 r;
#pragma unroll
  for (int d = 0; d < 4; ++d) r[d] = expand_bf16x2(w, d, c, k);
  return r;
}

// Buffer resources: 32-bit offsets from a uniform base, and reads past
// `bytes` return zero instead of touching memory.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ inline rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ inline u32x4 bload(rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, (int)soff, 0));
}
__device__ inline u32x2 bload2(rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)voff, (int)soff, 0));
}
__device__ inline uint32_t bload1(rsrc_t r, uint32_t voff, uint32_t soff) {
  return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, (int)voff, (int)soff, 0);
}

// 64 x 16 bytes straight to LDS: lane l's 16 bytes at `voff` go to dst + 16 l
// (dst the same in every lane). Counted by vmcnt; the compiler does not wait
// for it.
__device__ inline void bload_lds(rsrc_t r, void* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, (int)voff, (int)soff, 0, 0);
}

}  // namespace moe

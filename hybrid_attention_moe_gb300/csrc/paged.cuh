// The paged key-value cache: geometry, argument checks and the formats' small conversions,
// shared by the write and read kernels (paged.cu) and the decode attention (paged_attn.cu).
#pragma once

#include "common.cuh"

namespace beam {

// out[T][H] = og[T][HD] W_o^T in bf16: the output projection of both attention calls (attn.cu).
cudaError_t o_proj(const uint16_t* og, int T, int HD, const uint16_t* w_o, int H, uint16_t* out,
                   cudaStream_t st);

namespace paged {

constexpr int kFmtBF16 = BEAM_PAGED_BF16, kFmtFP8 = BEAM_PAGED_FP8, kFmtNVFP4 = BEAM_PAGED_NVFP4;

// Bytes of one row's codes.
__host__ __device__ constexpr int row_bytes(int fmt, int D) {
  return fmt == kFmtBF16 ? 2 * D : (fmt == kFmtFP8 ? D : D / 2);
}

inline int log2i(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

inline beam_status check(const beam_paged_kv* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr || c->page_table == nullptr ||
      c->num_pages <= 0 || c->page_size <= 0 || c->n_kv <= 0 || c->head_dim <= 0 ||
      c->num_seqs <= 0 || c->table_stride <= 0 || c->window < 0)
    return BEAM_ERR_INVALID_ARG;
  if (c->dtype != kFmtBF16 && c->dtype != kFmtFP8 && c->dtype != kFmtNVFP4) return BEAM_ERR_INVALID_ARG;
  if ((c->dtype != kFmtBF16) != (c->row_scale != nullptr) ||
      (c->dtype == kFmtNVFP4) != (c->block_scale != nullptr))
    return BEAM_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16_or_null(c->row_scale) ||
      !aligned16_or_null(c->block_scale) || (reinterpret_cast<uintptr_t>(c->page_table) & 3u))
    return BEAM_ERR_INVALID_ARG;
  if (!head_dim_ok(c->head_dim)) return BEAM_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) ||
      c->page_size * row_bytes(c->dtype, c->head_dim) < 1024)
    return BEAM_ERR_UNSUPPORTED;
  // positions are 32-bit: page_size * table_stride must not pass them
  if (int64_t(c->table_stride) * c->page_size > INT32_MAX - 256) return BEAM_ERR_UNSUPPORTED;
  // (page, head) indexes are 32-bit
  if (int64_t(c->num_pages) * c->n_kv > INT32_MAX) return BEAM_ERR_UNSUPPORTED;
  return BEAM_OK;
}

// 2^(b - 127) of a row's scale byte; NaN for 255.
__device__ __forceinline__ float pow2_of(unsigned b) {
  const unsigned n = b == 0 ? 0x00400000u : b << 23;
  return __uint_as_float(b == 255 ? 0x7FFFFFFFu : n);
}

// Two e4m3 codes (low byte first) -> f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{.reg .b16 c; cvt.u16.u32 c, %1; cvt.rn.f16x2.e4m3x2 %0, c;}" : "=r"(r) : "r"(codes));
  return r;
}
// Four e4m3 codes -> two f16x2 words, exactly.
__device__ __forceinline__ void e4m3x4_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
// Eight e2m1 codes (four bytes, even element in the low nibble) -> four f16x2 words, exactly.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t* r) {
  asm("{.reg .b8 b0, b1, b2, b3; mov.b32 {b0, b1, b2, b3}, %4; cvt.rn.f16x2.e2m1x2 %0, b0;"
      " cvt.rn.f16x2.e2m1x2 %1, b1; cvt.rn.f16x2.e2m1x2 %2, b2; cvt.rn.f16x2.e2m1x2 %3, b3;}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
__device__ __forceinline__ void unpack_f16(uint32_t w, float& lo, float& hi) {
  asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}"
      : "=f"(lo), "=f"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace paged
}  // namespace beam

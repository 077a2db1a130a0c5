// The paged key-value cache: geometry, argument checks, a slot's page, and the formats' small conversions both ways,
// shared by the write and read kernels (paged.cu), the append (paged_append.cu), the attentions (paged_attn.cu,
// paged_tree.cu) and the trees' bookkeeping (tree.cu).
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

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Where a token's rows go: the page of its 1-based slot p, or -1 (padding, or out of range: the bit to
// set in bad).
__device__ __forceinline__ int page_of(const beam_paged_kv& c, int s, int p, int shift,
                                       unsigned& bad) {
  bad = 0;
  if (p == 0) return -1;
  if (p < 0 || ((p - 1) >> shift) >= c.table_stride) {
    bad = BEAM_DEV_BAD_POSITION;
    return -1;
  }
  if (s < 0 || s >= c.num_seqs) {
    bad = BEAM_DEV_BAD_SEQ;
    return -1;
  }
  const int pg = c.page_table[size_t(s) * c.table_stride + ((p - 1) >> shift)];
  if (pg < 0 || pg >= c.num_pages) {
    bad = BEAM_DEV_BAD_PAGE;
    return -1;
  }
  return pg;
}

// ---- rows to codes. Magnitudes are compared as bf16 patterns without their signs (they order like
// the values, and infinities and NaNs come out on top); a row's power of two follows from the largest
// pattern's exponent and fraction alone, so nothing is rounded before the codes are.

// The larger patterns of even and odd elements of two registers of four words.
__device__ __forceinline__ unsigned abs_max(const uint4& x) {
  constexpr unsigned kAbs = 0x7FFF7FFFu;
  return __vmaxu2(__vmaxu2(x.x & kAbs, x.y & kAbs), __vmaxu2(x.z & kAbs, x.w & kAbs));
}
// The byte of a row with the largest pattern rm: most = 448 = 1.75 * 2^8 (fraction 96 / 128), or
// 2688 = 1.3125 * 2^11 (fraction 40 / 128).
template <int FMT>
__device__ __forceinline__ int row_byte(unsigned rm) {
  constexpr int kExp = FMT == kFmtFP8 ? 8 : 11, kFrac = FMT == kFmtFP8 ? 96 : 40;
  return max(0, int(rm >> 7) - kExp + (int(rm & 127u) > kFrac ? 1 : 0));
}
// Four e4m3 codes of y * inv.
__device__ __forceinline__ uint32_t fp8x4(const float* y, float inv) {
  return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(y[0] * inv, y[1] * inv), __NV_SATFINITE, __NV_E4M3)) |
         uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(y[2] * inv, y[3] * inv), __NV_SATFINITE, __NV_E4M3)) << 16;
}
// x to 14 significant bits (to nearest, ties away from zero).
__device__ __forceinline__ float round14(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x200u) & 0xFFFFFC00u);
}
// The e4m3 scale s of a block of 16 with the largest pattern bm (inv = 2^(127 - b)), and rs = 1 / s. The
// sixth of the block's largest value is rounded to 14 bits on its way: a midpoint of e4m3 has 5 bits, and
// any other sixth is 2^-8 of it away (the dividend has 8 bits, 6 midpoints 7).
__device__ __forceinline__ unsigned block_scale_of(unsigned bm, float inv, bool finite, float& rs) {
  const float q6 = round14(__uint_as_float(bm << 16) * inv * (1.f / 6.f));
  const unsigned s = finite ? __nv_cvt_float_to_fp8(q6, __NV_SATFINITE, __NV_E4M3) : 0u;
  float sf, unused;
  unpack_f16(e4m3x2_f16x2(s), sf, unused);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(sf));
  return s;
}
// Eight e2m1 codes of y * rs, rs the reciprocal of the block's scale times the row's power of two.
// Quotients are rounded to f16 on their way. One that is a midpoint of two codes (3 bits) comes back exactly; any
// other one is 2^-8 of the midpoint or more away from it (the dividend has 8 bits, s 4), which the
// reciprocal's error (2^-21) and half a step of f16 (2^-11) do not reach, so the code is that of the
// exact quotient.
__device__ __forceinline__ uint32_t fp4x8(const float* y, float rs) {
  uint32_t q[4], w;
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = pack_f16x2(y[2 * e] * rs, y[2 * e + 1] * rs);
  asm("{.reg .b8 a, b, c, d;"
      " cvt.rn.satfinite.e2m1x2.f16x2 a, %1; cvt.rn.satfinite.e2m1x2.f16x2 b, %2;"
      " cvt.rn.satfinite.e2m1x2.f16x2 c, %3; cvt.rn.satfinite.e2m1x2.f16x2 d, %4;"
      " mov.b32 %0, {a, b, c, d};}"
      : "=r"(w)
      : "r"(q[0]), "r"(q[1]), "r"(q[2]), "r"(q[3]));
  return w;
}

}  // namespace paged
}  // namespace beam

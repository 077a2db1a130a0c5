// Paged key-value cache: rows quantised as they are written, and read back into a contiguous
// BF16 cache. The formats are those of include/beam.h (beam_paged_kv).
//
// Both kernels move bytes once: bounded by HBM for long calls and by the launch for short ones.
#include "paged.cuh"

namespace beam {
namespace paged {
namespace {

struct WriteParams {
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* seq_id;
  const int32_t* pos;
  beam_paged_kv c;
  int64_t token_stride;
  int rows;   // T * n_kv * 2
  int shift;  // log2(page_size)
};

// Where a token's rows go: the page, or -1 (padding, or out of range: the bit to set in bad).
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

// D / 8 lanes hold one row, eight elements each, so a warp takes 2 (D 128) or 4 (D 64) rows, in
// the order (token, head, K | V). The row's largest magnitude is an integer maximum of the
// bf16 patterns without their signs (they order like the values, and infinities and NaNs come
// out on top); the row's power of two follows from that pattern's exponent and fraction alone,
// so nothing is rounded before the codes are.
template <int FMT, int D>
__global__ void __launch_bounds__(256) paged_write_kernel(const WriteParams P) {
  pdl_trigger();
  pdl_wait();
  constexpr int LPR = D / 8;
  const int lane = threadIdx.x & 31, sub = lane % LPR;
  const int warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int row = warp * (32 / LPR) + lane / LPR;
  const bool live = row < P.rows;
  const int r = live ? row : P.rows - 1;   // idle lanes repeat the last row and store nothing
  const int kv = r & 1, th = r >> 1;
  const int t = th / P.c.n_kv, hk = th - t * P.c.n_kv;
  const uint4 x = *reinterpret_cast<const uint4*>((kv ? P.v : P.k) + t * P.token_stride +
                                                  hk * D + sub * 8);
  const int p = P.pos[t];
  unsigned bad;
  const int pg = page_of(P.c, P.seq_id[t], p, P.shift, bad);
  if (bad && live && hk == 0 && kv == 0 && sub == 0) flag(bad);
  const bool store = live && pg >= 0;
  const int off = (p - 1) & (P.c.page_size - 1);
  const size_t head = size_t(store ? pg : 0) * P.c.n_kv + hk;
  const size_t at = head * P.c.page_size + (store ? off : 0);          // row of k or v
  const size_t sat = (head * 2 + kv) * P.c.page_size + (store ? off : 0);   // row of the scales
  uint8_t* dst = static_cast<uint8_t*>(kv ? P.c.v : P.c.k) + at * row_bytes(FMT, D);
  if constexpr (FMT == kFmtBF16) {
    if (store) *reinterpret_cast<uint4*>(dst + sub * 16) = x;
  } else {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    unsigned mx = 0;   // the lane's largest magnitude, as a bf16 pattern
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mx = max(mx, w[i] & 0x7FFFu);
      mx = max(mx, (w[i] >> 16) & 0x7FFFu);
    }
    unsigned rm = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));   // of the block of 16
    const unsigned bm = rm;
#pragma unroll
    for (int o = 2; o < LPR; o <<= 1) rm = max(rm, __shfl_xor_sync(0xffffffffu, rm, o));
    const bool finite = rm < 0x7F80u;
    // most = 448 = 1.75 * 2^8 (fraction 96 / 128), or 2688 = 1.3125 * 2^11 (fraction 40 / 128)
    constexpr int kExp = FMT == kFmtFP8 ? 8 : 11, kFrac = FMT == kFmtFP8 ? 96 : 40;
    const int b = max(0, int(rm >> 7) - kExp + (int(rm & 127u) > kFrac ? 1 : 0));
    const float inv = __uint_as_float(unsigned(254 - b) << 23);   // 2^(127 - b)
    float y[8];
    unpack8(x, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = finite ? y[i] * inv : 0.f;
    if constexpr (FMT == kFmtFP8) {
      uint32_t c2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c2[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i], y[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      if (store)
        *reinterpret_cast<uint2*>(dst + sub * 8) = make_uint2(c2[0] | (c2[1] << 16), c2[2] | (c2[3] << 16));
    } else {
      const float bmax = finite ? __uint_as_float(bm << 16) * inv : 0.f;
      const unsigned s = __nv_cvt_float_to_fp8(__fdiv_rn(bmax, 6.f), __NV_SATFINITE, __NV_E4M3);
      float sf, unused;
      unpack_f16(e4m3x2_f16x2(s), sf, unused);
      const float rs = s ? __fdiv_rn(1.f, sf) : 0.f;
      uint32_t codes = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // y / s from the reciprocal, then to 14 significant bits. A quotient that is a midpoint
        // of two codes has 3 bits and comes back exactly; any other one is further from every
        // midpoint (2^-8 of it: y has 8 bits, s 4, the midpoint 3) than the two errors
        // (2^-22 and 2^-14) reach, so the code is that of the exact quotient.
        float q[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          q[e] = __uint_as_float((__float_as_uint(y[2 * i + e] * rs) + 0x200u) & 0xFFFFFC00u);
        uint32_t c;
        asm("{.reg .b8 z; cvt.rn.satfinite.e2m1x2.f32 z, %2, %1; cvt.u32.u8 %0, z;}"
            : "=r"(c)
            : "f"(q[0]), "f"(q[1]));
        codes |= (c & 0xFFu) << (8 * i);
      }
      if (store) {
        *reinterpret_cast<uint32_t*>(dst + sub * 4) = s ? codes : 0u;
        if ((sub & 1) == 0) P.c.block_scale[sat * (D / 16) + (sub >> 1)] = uint8_t(s);
      }
    }
    if (store && sub == 0) P.c.row_scale[sat] = finite ? uint8_t(b) : uint8_t(255);
  }
}

struct ReadParams {
  beam_paged_kv c;
  const int32_t* seq_id;
  const int32_t* first;
  const int32_t* last;
  uint16_t* k;
  uint16_t* v;
  int cap, max_len, shift;
};

// A CTA takes kReadKeys consecutive positions of one (row, KV head), K and V. A thread holds
// eight elements of a key: 16, 8 or 4 bytes of codes in, 16 bytes out.
constexpr int kReadKeys = 64;

template <int FMT, int D>
__global__ void __launch_bounds__(256) paged_read_kernel(const ReadParams P) {
  pdl_trigger();
  pdl_wait();
  constexpr int TPR = D / 8, KPP = 256 / TPR, NP = kReadKeys / KPP;   // keys per pass, passes
  const int i = blockIdx.z, hk = blockIdx.y;
  const int first = P.first[i], last = P.last[i], s = P.seq_id[i];
  if (last < first) return;
  unsigned bad = 0;
  if (first < 1 || ((last - 1) >> P.shift) >= P.c.table_stride || last - first >= P.cap ||
      last - first >= P.max_len)
    bad = BEAM_DEV_BAD_POSITION;
  else if (s < 0 || s >= P.c.num_seqs)
    bad = BEAM_DEV_BAD_SEQ;
  if (bad) {
    if (blockIdx.x == 0 && hk == 0 && threadIdx.x == 0) flag(bad);
    return;
  }
  if (int(blockIdx.x) * kReadKeys > last - first) return;
  const int p0 = first + int(blockIdx.x) * kReadKeys;
  const int sub = threadIdx.x % TPR, key = threadIdx.x / TPR;
  const int32_t* table = P.c.page_table + size_t(s) * P.c.table_stride;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int p = p0 + j * KPP + key;
    if (p > last) break;
    const int pg = table[(p - 1) >> P.shift];
    if (pg < 0 || pg >= P.c.num_pages) {
      if (hk == 0 && sub == 0) flag(BEAM_DEV_BAD_PAGE);
      continue;
    }
    const size_t head = size_t(pg) * P.c.n_kv + hk;
    const int off = (p - 1) & (P.c.page_size - 1);
    const size_t to = ((size_t(i) * P.c.n_kv + hk) * P.cap + (p - 1) % P.cap) * D + sub * 8;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint8_t* src = static_cast<const uint8_t*>(kv ? P.c.v : P.c.k) +
                           (head * P.c.page_size + off) * row_bytes(FMT, D);
      uint4 o;
      if constexpr (FMT == kFmtBF16) {
        o = *reinterpret_cast<const uint4*>(src + sub * 16);
      } else {
        const size_t sat = (head * 2 + kv) * P.c.page_size + off;
        float f = pow2_of(P.c.row_scale[sat]);
        uint32_t h[4];
        if constexpr (FMT == kFmtFP8) {
          const uint2 c = *reinterpret_cast<const uint2*>(src + sub * 8);
          e4m3x4_f16(c.x, h[0], h[1]);
          e4m3x4_f16(c.y, h[2], h[3]);
        } else {
          e2m1x8_f16(*reinterpret_cast<const uint32_t*>(src + sub * 4), h);
        }
        float bs = 1.f, unused;
        if constexpr (FMT == kFmtNVFP4)
          unpack_f16(e4m3x2_f16x2(P.c.block_scale[sat * (D / 16) + (sub >> 1)]), bs, unused);
        uint32_t r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float a, b;
          unpack_f16(h[e], a, b);
          // code * s is exact, so the only rounding is that to bf16
          r[e] = pack_bf2(a * bs * f, b * bs * f);
        }
        o = make_uint4(r[0], r[1], r[2], r[3]);
      }
      *reinterpret_cast<uint4*>((kv ? P.v : P.k) + to) = o;
    }
  }
}

template <int FMT, int D>
cudaError_t launch_write(const WriteParams& p, cudaStream_t st) {
  const int per = 8 * (32 / (D / 8));
  return launch_pdl(paged_write_kernel<FMT, D>, dim3((p.rows + per - 1) / per), dim3(256), 0, st, p);
}
template <int FMT, int D>
cudaError_t launch_read(const ReadParams& p, int N, cudaStream_t st) {
  return launch_pdl(paged_read_kernel<FMT, D>,
                    dim3((p.max_len + kReadKeys - 1) / kReadKeys, p.c.n_kv, N), dim3(256), 0, st, p);
}

}  // namespace
}  // namespace paged
}  // namespace beam

extern "C" size_t beam_paged_kv_bytes(int num_pages, int n_kv, int page_size, int head_dim,
                                      int dtype) {
  using namespace beam::paged;
  if (num_pages <= 0 || n_kv <= 0 || page_size <= 0 || head_dim <= 0) return 0;
  if (dtype != kFmtBF16 && dtype != kFmtFP8 && dtype != kFmtNVFP4) return 0;
  const size_t row = size_t(row_bytes(dtype, head_dim)) + (dtype != kFmtBF16 ? 1 : 0) +
                     (dtype == kFmtNVFP4 ? head_dim / 16 : 0);
  return 2 * size_t(num_pages) * n_kv * page_size * row;
}

extern "C" beam_status beam_paged_kv_write(const beam_bf16* k, const beam_bf16* v,
                                           int token_stride, const int32_t* seq_id,
                                           const int32_t* pos, int T, const beam_paged_kv* cache,
                                           beam_stream_t stream) {
  using namespace beam;
  using namespace beam::paged;
  const beam_status st = check(cache);
  if (st != BEAM_OK) return st;
  if (T == 0) return BEAM_OK;
  if (T < 0 || !k || !v || !seq_id || !pos || !aligned16(k) || !aligned16(v) ||
      (token_stride & 7) || token_stride < cache->n_kv * cache->head_dim)
    return BEAM_ERR_INVALID_ARG;
  if (int64_t(T) * cache->n_kv * 2 > INT32_MAX - 64) return BEAM_ERR_UNSUPPORTED;
  const WriteParams p{k, v, seq_id, pos, *cache, token_stride, T * cache->n_kv * 2,
                      log2i(cache->page_size)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = cache->head_dim == 128;
  cudaError_t e;
  if (cache->dtype == kFmtBF16) e = wide ? launch_write<kFmtBF16, 128>(p, s) : launch_write<kFmtBF16, 64>(p, s);
  else if (cache->dtype == kFmtFP8) e = wide ? launch_write<kFmtFP8, 128>(p, s) : launch_write<kFmtFP8, 64>(p, s);
  else e = wide ? launch_write<kFmtNVFP4, 128>(p, s) : launch_write<kFmtNVFP4, 64>(p, s);
  return cuda_status(e);
}

extern "C" beam_status beam_paged_kv_read(const beam_paged_kv* cache, const int32_t* seq_id,
                                          const int32_t* first, const int32_t* last, int N,
                                          int max_len, const beam_kv_cache* dst,
                                          beam_stream_t stream) {
  using namespace beam;
  using namespace beam::paged;
  const beam_status st = check(cache);
  if (st != BEAM_OK) return st;
  if (N == 0) return BEAM_OK;
  if (N < 0 || max_len < 0 || !seq_id || !first || !last || !dst || !dst->k || !dst->v ||
      !aligned16(dst->k) || !aligned16(dst->v) || dst->num_seqs < N || dst->capacity <= 0)
    return BEAM_ERR_INVALID_ARG;
  if (dst->dtype != BEAM_KV_BF16) return BEAM_ERR_UNSUPPORTED;
  if (N > 65535 || cache->n_kv > 65535) return BEAM_ERR_UNSUPPORTED;   // grid limits
  if (max_len == 0) return BEAM_OK;
  // no range is longer than the page table or the destination: the rest of the grid is not needed
  const int64_t table = int64_t(cache->table_stride) * cache->page_size;
  if (max_len > table) max_len = int(table);
  if (max_len > dst->capacity) max_len = dst->capacity;
  const ReadParams p{*cache, seq_id, first, last, static_cast<uint16_t*>(dst->k),
                     static_cast<uint16_t*>(dst->v), dst->capacity, max_len,
                     log2i(cache->page_size)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = cache->head_dim == 128;
  cudaError_t e;
  if (cache->dtype == kFmtBF16) e = wide ? launch_read<kFmtBF16, 128>(p, N, s) : launch_read<kFmtBF16, 64>(p, N, s);
  else if (cache->dtype == kFmtFP8) e = wide ? launch_read<kFmtFP8, 128>(p, N, s) : launch_read<kFmtFP8, 64>(p, N, s);
  else e = wide ? launch_read<kFmtNVFP4, 128>(p, N, s) : launch_read<kFmtNVFP4, 64>(p, N, s);
  return cuda_status(e);
}

// Paged key-value cache: rows quantised as they are written, and read back into a contiguous
// BF16 cache. The formats are those of include/beam.h (beam_paged_kv).
//
// Both kernels move bytes once and do little with them. Reading back is bounded by HBM (192,000
// tokens of 8 heads from FP8: 176.6 us, 99% of the copy rate; 16,384 from BF16 20.0, 99%). Writing
// 16,384 tokens of 8 heads: BF16 20.4 us, FP8 16.5, NVFP4 15.5 with the input in L2 and 21.5 from HBM
// (59% of the copy rate), where the quantisation's ~180 warp instructions for 512 elements keep the
// issue slots 54% busy.
// A decode step's rows (32 tokens) take 2.3 us, most of it the launch and three dependent loads.
#include "mma.cuh"
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
  int T, parts;   // parts: warps of one token
  int shift;      // log2(page_size)
};

// A warp takes up to kHeads KV heads of one token, K and V, and issues all its loads before the
// page is looked up. A lane holds 16 elements of a row (an NVFP4 block; a BF16 row, which is only
// moved, is taken 8 a lane).
constexpr int kHeads = 8;
template <int FMT, int D>
__global__ void __launch_bounds__(128, 8) paged_write_kernel(const WriteParams P) {
  pdl_trigger();
  pdl_wait();
  constexpr int EPL = FMT == kFmtBF16 ? 8 : 16, NV = EPL / 8;
  constexpr int LPR = D / EPL, HPI = 16 / LPR;          // lanes of a row, heads of a step
  constexpr int U = kHeads > HPI ? kHeads / HPI : 1;
  const int lane = threadIdx.x & 31, sub = lane % LPR, kv = (lane / LPR) & 1;
  const int warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int t = warp / P.parts, h0 = (warp - t * P.parts) * kHeads + lane / (2 * LPR);
  if (t >= P.T) return;
  const int n_kv = P.c.n_kv;
  const uint16_t* src = (kv ? P.v : P.k) + t * P.token_stride + sub * EPL;
  uint4 x[U][NV];
#pragma unroll
  for (int u = 0; u < U; ++u)   // heads past the last repeat it and store nothing
#pragma unroll
    for (int a = 0; a < NV; ++a)
      x[u][a] = reinterpret_cast<const uint4*>(src + min(h0 + u * HPI, n_kv - 1) * D)[a];
  const int p = P.pos[t];
  unsigned bad;
  const int pg = page_of(P.c, P.seq_id[t], p, P.shift, bad);
  if (bad && h0 == 0 && lane == 0) flag(bad);
  if (pg < 0) return;   // the whole warp: one token
  const int off = (p - 1) & (P.c.page_size - 1);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int hk = h0 + u * HPI;
    const bool store = hk < n_kv;
    const size_t head = size_t(pg) * n_kv + (store ? hk : 0);
    const size_t sat = (head * 2 + kv) * P.c.page_size + off;   // row of the scales
    uint8_t* dst = static_cast<uint8_t*>(kv ? P.c.v : P.c.k) + (head * P.c.page_size + off) * row_bytes(FMT, D);
    if constexpr (FMT == kFmtBF16) {
      if (store) *reinterpret_cast<uint4*>(dst + sub * 16) = x[u][0];
    } else {
      unsigned mx = 0;   // largest patterns of even and odd elements
#pragma unroll
      for (int a = 0; a < NV; ++a) mx = __vmaxu2(mx, abs_max(x[u][a]));
      const unsigned bm = max(mx & 0xFFFFu, mx >> 16);   // of the block of 16
      unsigned rm = bm;
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) rm = max(rm, __shfl_xor_sync(0xffffffffu, rm, o));
      const bool finite = rm < 0x7F80u;
      const int b = row_byte<FMT>(rm);
      float inv = __uint_as_float(unsigned(254 - b) << 23);   // 2^(127 - b)
      float y[EPL];
#pragma unroll
      for (int a = 0; a < NV; ++a) unpack8(x[u][a], y + 8 * a);
      if constexpr (FMT == kFmtFP8) {
        uint32_t w[EPL / 4];
#pragma unroll
        for (int i = 0; i < EPL / 4; ++i) {
          w[i] = fp8x4(y + 4 * i, inv);
          if (!finite) w[i] = 0u;
        }
        if (store) *reinterpret_cast<uint4*>(dst + sub * EPL) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        float rs;
        const unsigned s = block_scale_of(bm, inv, finite, rs);
        if (b < 16) {   // 2^(127 - b) / s may pass FP32's range: part of it goes to the elements
          inv *= 0x1p-32f;
#pragma unroll
          for (int i = 0; i < EPL; ++i) y[i] *= 0x1p32f;
        }
        rs *= inv;
        uint32_t w[EPL / 8];
#pragma unroll
        for (int i = 0; i < EPL / 8; ++i) {
          w[i] = fp4x8(y + 8 * i, rs);
          if (s == 0) w[i] = 0u;   // the block is zeros, or the row holds no numbers
        }
        if (store) {
          *reinterpret_cast<uint2*>(dst + sub * (EPL / 2)) = make_uint2(w[0], w[1]);
          P.c.block_scale[sat * (D / 16) + sub] = uint8_t(s);
        }
      }
      if (store && sub == 0) P.c.row_scale[sat] = finite ? uint8_t(b) : uint8_t(255);
    }
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

// A CTA takes read_keys consecutive positions of one (row, KV head), K and V, in passes. A thread
// holds two chunks of eight elements of a key, half a row apart (so that a warp's stores are
// whole sectors): 2 x 16, 8 or 4 bytes of codes in, 2 x 16 bytes out.
constexpr int read_passes(int fmt) { return fmt == kFmtNVFP4 ? 4 : 2; }
constexpr int read_keys(int fmt, int D) { return read_passes(fmt) * (256 / (D / 16)); }

template <int FMT, int D>
__global__ void __launch_bounds__(256) paged_read_kernel(const ReadParams P) {
  pdl_trigger();
  pdl_wait();
  constexpr int TPR = D / 16, KPP = 256 / TPR, NP = read_passes(FMT), KEYS = read_keys(FMT, D);
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
  if (int(blockIdx.x) * KEYS > last - first) return;
  const int p0 = first + int(blockIdx.x) * KEYS;
  const int sub = threadIdx.x % TPR, key = threadIdx.x / TPR;
  const int32_t* table = P.c.page_table + size_t(s) * P.c.table_stride;
  // all pages, then all codes and scales, then the stores: each step's loads are in flight at once
  size_t at[NP];   // the key's row of codes; scale rows follow from it
  bool ok[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int p = p0 + j * KPP + key;
    ok[j] = p <= last;
    const int pg = ok[j] ? table[(p - 1) >> P.shift] : 0;
    if (pg < 0 || pg >= P.c.num_pages) {
      if (hk == 0 && sub == 0) flag(BEAM_DEV_BAD_PAGE);
      ok[j] = false;
    }
    at[j] = (size_t(ok[j] ? pg : 0) * P.c.n_kv + hk) * P.c.page_size + ((p - 1) & (P.c.page_size - 1));
  }
  constexpr int CW = FMT == kFmtBF16 ? 4 : (FMT == kFmtFP8 ? 2 : 1);   // words of eight codes
  constexpr int ROWB = row_bytes(FMT, D);
  uint32_t w[NP][2][2][CW], rs[NP][2], bs[NP][2][2];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    if (!ok[j]) continue;
    // [page][head][key] -> [page][head][K | V][key]
    const size_t sat = 2 * at[j] - (at[j] & size_t(P.c.page_size - 1));
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint8_t* src = static_cast<const uint8_t*>(kv ? P.c.v : P.c.k) + at[j] * ROWB + sub * CW * 4;
#pragma unroll
      for (int h = 0; h < 2; ++h, src += ROWB / 2) {
        if constexpr (CW == 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(src);
          w[j][kv][h][0] = x.x; w[j][kv][h][1] = x.y; w[j][kv][h][2] = x.z; w[j][kv][h][3] = x.w;
        } else if constexpr (CW == 2) {
          const uint2 x = *reinterpret_cast<const uint2*>(src);
          w[j][kv][h][0] = x.x; w[j][kv][h][1] = x.y;
        } else {
          w[j][kv][h][0] = *reinterpret_cast<const uint32_t*>(src);
        }
      }
      if constexpr (FMT != kFmtBF16) {
        const size_t r = sat + (kv ? P.c.page_size : 0);
        rs[j][kv] = P.c.row_scale[r];
        if constexpr (FMT == kFmtNVFP4) {
          const uint8_t* b = P.c.block_scale + r * (D / 16) + (sub >> 1);
          bs[j][kv][0] = b[0];
          bs[j][kv][1] = b[D / 32];
        }
      }
    }
  }
  const int slot0 = (p0 - 1) % P.cap;
  const size_t row = (size_t(i) * P.c.n_kv + hk) * P.cap;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    if (!ok[j]) continue;
    int slot = slot0 + j * KPP + key;   // the range is no longer than the ring: one lap at most
    if (slot >= P.cap) slot -= P.cap;
    const size_t to = (row + slot) * D + sub * 8;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint16_t* dst = (kv ? P.v : P.k) + to;
      const float f = FMT == kFmtBF16 ? 1.f : pow2_of(rs[j][kv]);
#pragma unroll
      for (int h = 0; h < 2; ++h, dst += D / 2) {
        uint32_t r[4];
        if constexpr (FMT == kFmtBF16) {
#pragma unroll
          for (int e = 0; e < 4; ++e) r[e] = w[j][kv][h][e];
        } else {
          uint32_t c[4];
          float unit = f;
          if constexpr (FMT == kFmtFP8) {
            e4m3x4_f16(w[j][kv][h][0], c[0], c[1]);
            e4m3x4_f16(w[j][kv][h][CW - 1], c[2], c[3]);
          } else {
            float sf, unused;
            unpack_f16(e4m3x2_f16x2(bs[j][kv][h]), sf, unused);
            e2m1x8_f16(w[j][kv][h][0], c);
            unit = sf * f;
          }
          // code * unit has 6 bits: exact down to FP32's smallest 2^-149, which no stored value
          // passes (2^-10 * 2^-127), so the only rounding is that to bf16
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float a, b;
            unpack_f16(c[e], a, b);
            r[e] = pack_bf16x2(a * unit, b * unit);
          }
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(r[0], r[1], r[2], r[3]);
      }
    }
  }
}

template <int FMT, int D>
cudaError_t launch_write(const WriteParams& p, cudaStream_t st) {
  const int warps = p.T * p.parts;
  return launch_pdl(paged_write_kernel<FMT, D>, dim3((warps + 3) / 4), dim3(128), 0, st, p);
}
template <int FMT, int D>
cudaError_t launch_read(const ReadParams& p, int N, cudaStream_t st) {
  return launch_pdl(paged_read_kernel<FMT, D>,
                    dim3((p.max_len + read_keys(FMT, D) - 1) / read_keys(FMT, D), p.c.n_kv, N), dim3(256), 0, st, p);
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
  const WriteParams p{k, v, seq_id, pos, *cache, token_stride, T,
                      (cache->n_kv + kHeads - 1) / kHeads, log2i(cache->page_size)};
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

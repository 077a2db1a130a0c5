// New tokens of a paged layer: per-head Q/K RMSNorm, RoPE or the SSMax query scale, and K and V into the
// pages, quantised on the way, in one pass over the packed projection rows.
//
//   x <- x (mean(x^2) + eps)^-1/2 w;  RoPE: (a, b) <- (a cos - b sin, b cos + a sin), pairs (i, i + D/2), angle
//   (p - 1) theta^(-2i/D);  SSMax: q <- q (1 + p / base)^e
//
// A CTA takes one token. A lane holds eight elements of a row's lower half and the eight that they pair
// with, so the rotation stays in the lane. Rows are loaded before the angles are worked out. All is FP32 (the angle is reduced in
// FP64), off by 2^-19 (|a| + |b|) at most before the one rounding to bf16. Of 2,097,152 keys without rotation 15 land a bf16 step from
// the exact value's (11 with a correctly rounded root, which costs a prefill chunk 2 %; elementary FP32 operations 9), with it 98:
// the angle's rounding to FP32. What bounds it is
// memory: two batches of rows are in flight in each warp, and registers decide how many warps there are (64 each: 1024
// threads an SM; at 120, with the lane's sines and cosines kept over the rows, half as many took 203 us for 149).
#include <math.h>

#include "gemm_tc.cuh"
#include "gemv.cuh"
#include "mma.cuh"
#include "paged.cuh"

namespace beam {
namespace paged {
namespace {

constexpr int kMaxHalf = 64;
struct RopeTab {
  double inv[kMaxHalf];   // theta^(-2i/D), from the host in double
};

struct AppendParams {
  const uint16_t* z;
  const uint16_t* qnw;
  const uint16_t* knw;
  const int32_t* seq_id;
  const int32_t* pos;
  const int32_t* slot;
  uint16_t* q_out;
  uint16_t* g_out;
  beam_paged_kv c;
  int64_t stride;
  int T, n_q, rows, shift, nope;   // rows: of z that are read, Q | K | V (| gate)
  float eps, ss_base, ss_exp;
  RopeTab rope;
};

template <int FMT, int D>
__global__ void __launch_bounds__(512, 2) paged_append_kernel(const __grid_constant__ AppendParams P) {
  pdl_trigger();
  pdl_wait();
  constexpr int LPR = D / 16, RPW = 32 / LPR, HALF = D / 2;   // lanes of a row, rows of a warp
  constexpr int U = 2;                                        // row groups in flight of a warp
  __shared__ __align__(16) float2 turn[HALF];   // read where they are used: registers are what limits the loads in flight
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, sub = lane % LPR;
  const int n_q = P.n_q, n_kv = P.c.n_kv;
  const uint16_t* z = P.z + t * P.stride + sub * 8;
  const int groups = (P.rows + RPW - 1) / RPW;
  uint4 lo[U], hi[U];
  auto load = [&](int g0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {   // rows past the last repeat it and store nothing
      const uint16_t* src = z + min((g0 + warps * u) * RPW + lane / LPR, P.rows - 1) * D;
      lo[u] = ld_stream(src);
      hi[u] = ld_stream(src + HALF);
    }
  };
  load(warp);
  const int p = P.pos[t], s = P.seq_id[t], sl = P.slot ? P.slot[t] : p;
  float ss = 1.f;
  if (P.nope) ss = ssmax_scale(max(p, 0), P.ss_base, P.ss_exp);
  else if (threadIdx.x < HALF) {
    float sv, cv;
    sincosf(rope_angle(p, P.rope.inv[threadIdx.x]), &sv, &cv);
    turn[threadIdx.x] = make_float2(cv, sv);
  }
  unsigned bad;
  const int pg = page_of(P.c, s, sl, P.shift, bad);
  if (bad == 0 && p < 0) bad = BEAM_DEV_BAD_POSITION;
  if (bad && threadIdx.x == 0) flag(bad);
  const bool keep = pg >= 0 && bad == 0;
  const int off = (sl - 1) & (P.c.page_size - 1);
  __syncthreads();
  for (int g0 = warp; g0 < groups; g0 += warps * U) {
    if (g0 != warp) load(g0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r0 = (g0 + warps * u) * RPW, row = r0 + lane / LPR;
      if (r0 >= P.rows) break;
      uint4 a = lo[u], b = hi[u];
      if (r0 < n_q + n_kv) {   // a group with Q or K rows
        const bool turned = row < n_q + n_kv;
        float x[8], y[8];
        unpack8(a, x);
        unpack8(b, y);
        if (P.qnw != nullptr) {
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], fmaf(y[e], y[e], sum));
#pragma unroll
          for (int o = 1; o < LPR; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          const float f = rsqrtf(sum * (1.f / D) + P.eps);
          const uint16_t* gw = (row < n_q ? P.qnw : P.knw) + sub * 8;
          float wx[8], wy[8];
          unpack8(*reinterpret_cast<const uint4*>(gw), wx);
          unpack8(*reinterpret_cast<const uint4*>(gw + HALF), wy);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] *= f * wx[e];
            y[e] *= f * wy[e];
          }
        }
        if (!P.nope) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float4 w = *reinterpret_cast<const float4*>(turn + sub * 8 + e);   // cosine, sine of two
            const float c0 = x[e], d0 = y[e], c1 = x[e + 1], d1 = y[e + 1];
            x[e] = c0 * w.x - d0 * w.y;
            y[e] = d0 * w.x + c0 * w.y;
            x[e + 1] = c1 * w.z - d1 * w.w;
            y[e + 1] = d1 * w.z + c1 * w.w;
          }
        } else if (row < n_q) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] *= ss;
            y[e] *= ss;
          }
        }
        if (turned) {
          a = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
          b = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        }
      }
      const bool kv_row = row >= n_q && row < n_q + 2 * n_kv;
      if (row < P.rows && !kv_row) {
        uint16_t* dst = row < n_q ? P.q_out + (size_t(t) * n_q + row) * D
                                  : P.g_out + (size_t(t) * n_q + row - n_q - 2 * n_kv) * D;
        *reinterpret_cast<uint4*>(dst + sub * 8) = a;
        *reinterpret_cast<uint4*>(dst + HALF + sub * 8) = b;
      }
      if (!keep || r0 + RPW <= n_q || r0 >= n_q + 2 * n_kv) continue;   // the whole warp: no row for the pages
      const int kv = row >= n_q + n_kv, hk = kv_row ? row - n_q - kv * n_kv : 0;
      const size_t head = size_t(pg) * n_kv + hk, sat = (head * 2 + kv) * P.c.page_size + off;
      uint8_t* dst = static_cast<uint8_t*>(kv ? P.c.v : P.c.k) + (head * P.c.page_size + off) * row_bytes(FMT, D);
      if constexpr (FMT == kFmtBF16) {
        if (kv_row) {
          *reinterpret_cast<uint4*>(dst + sub * 16) = a;
          *reinterpret_cast<uint4*>(dst + D + sub * 16) = b;
        }
      } else {
        unsigned ma = abs_max(a), mb = abs_max(b);
        ma = max(ma & 0xFFFFu, ma >> 16);
        mb = max(mb & 0xFFFFu, mb >> 16);
        // blocks of 16: the lane's and its neighbour's eight
        ma = max(ma, __shfl_xor_sync(0xffffffffu, ma, 1));
        mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
        unsigned rm = max(ma, mb);
#pragma unroll
        for (int o = 2; o < LPR; o <<= 1) rm = max(rm, __shfl_xor_sync(0xffffffffu, rm, o));
        const bool finite = rm < 0x7F80u;
        const int rb = row_byte<FMT>(rm);
        float inv = __uint_as_float(unsigned(254 - rb) << 23);   // 2^(127 - rb)
        float x[8], y[8];
        unpack8(a, x);
        unpack8(b, y);
        if constexpr (FMT == kFmtFP8) {
          const uint2 wa = finite ? make_uint2(fp8x4(x, inv), fp8x4(x + 4, inv)) : make_uint2(0, 0);
          const uint2 wb = finite ? make_uint2(fp8x4(y, inv), fp8x4(y + 4, inv)) : make_uint2(0, 0);
          if (kv_row) {
            *reinterpret_cast<uint2*>(dst + sub * 8) = wa;
            *reinterpret_cast<uint2*>(dst + HALF + sub * 8) = wb;
          }
        } else {
          float ra, rbk;
          const unsigned sa = block_scale_of(ma, inv, finite, ra), sb = block_scale_of(mb, inv, finite, rbk);
          if (rb < 16) {   // 2^(127 - rb) / s may pass FP32's range: part of it goes to the elements
            inv *= 0x1p-32f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              x[e] *= 0x1p32f;
              y[e] *= 0x1p32f;
            }
          }
          const uint32_t wa = sa == 0 ? 0u : fp4x8(x, ra * inv), wb = sb == 0 ? 0u : fp4x8(y, rbk * inv);
          if (kv_row) {
            *reinterpret_cast<uint32_t*>(dst + sub * 4) = wa;
            *reinterpret_cast<uint32_t*>(dst + D / 4 + sub * 4) = wb;
            if ((sub & 1) == 0) {
              P.c.block_scale[sat * (D / 16) + sub / 2] = uint8_t(sa);
              P.c.block_scale[sat * (D / 16) + D / 32 + sub / 2] = uint8_t(sb);
            }
          }
        }
        if (kv_row && sub == 0) P.c.row_scale[sat] = finite ? uint8_t(rb) : uint8_t(255);
      }
    }
  }
}

beam_status append(const beam_layer_cfg* cfg, const uint16_t* z, int64_t stride, const uint16_t* qnw,
                   const uint16_t* knw, const int32_t* seq_id, const int32_t* pos, const int32_t* slot,
                   int T, uint16_t* q_out, uint16_t* g_out, const beam_paged_kv* cache, cudaStream_t st) {
  const int D = cfg->head_dim;
  AppendParams p{z, qnw, knw, seq_id, pos, slot, q_out, g_out, *cache, stride, T, cfg->n_q,
                 cfg->n_q * (g_out ? 2 : 1) + 2 * cfg->n_kv, log2i(cache->page_size),
                 cfg->kind == BEAM_ATTN_NOPE_SSMAX, cfg->eps, cfg->ssmax_base, cfg->ssmax_exp, {}};
  for (int i = 0; i < D / 2; ++i) p.rope.inv[i] = pow(double(cfg->rope_theta), -2.0 * double(i) / double(D));
  const bool wide = D == 128;
  // The widest block of which all tokens are in flight at once (1024 threads of an SM): a token alone is latency, its rows
  // in one batch of loads; past that the narrowest, whose barrier holds up the fewest loads. us of BF16 rows, 48 + 8 + 8 + 48 heads of
  // 128, by threads of a block:
  //   tokens    64     128     256     512
  //        1   8.7     6.1     4.7     4.1
  //      304  11.3     7.8     5.9     5.2
  //      512  11.9     9.3     7.3     8.3
  //     1024  14.7    11.7    12.4    13.9
  //     2048  20.3    21.0    22.4    25.2
  //    16384   149     156     165     195   (943 MB: 6.3 TB/s)
  const int sms = num_sms_cached(), threads = T <= 2 * sms ? 512 : T <= 4 * sms ? 256 : T <= 8 * sms ? 128 : 64;
  auto go = [&](auto kern) { return launch_pdl(kern, dim3(T), dim3(threads), 0, st, p); };
  cudaError_t e;
  if (cache->dtype == kFmtBF16) e = wide ? go(paged_append_kernel<kFmtBF16, 128>) : go(paged_append_kernel<kFmtBF16, 64>);
  else if (cache->dtype == kFmtFP8) e = wide ? go(paged_append_kernel<kFmtFP8, 128>) : go(paged_append_kernel<kFmtFP8, 64>);
  else e = wide ? go(paged_append_kernel<kFmtNVFP4, 128>) : go(paged_append_kernel<kFmtNVFP4, 64>);
  return cuda_status(e);
}

}  // namespace
}  // namespace paged
}  // namespace beam

extern "C" beam_status beam_paged_append(const beam_layer_cfg* cfg, const beam_bf16* qkv, int token_stride,
                                         const beam_bf16* q_norm_w, const beam_bf16* k_norm_w,
                                         const int32_t* seq_id, const int32_t* pos, const int32_t* slot,
                                         int T, beam_bf16* q_out, beam_bf16* g_out,
                                         const beam_paged_kv* cache, beam_stream_t stream) {
  using namespace beam;
  using namespace beam::paged;
  beam_status st = check_cfg_attn(cfg);
  if (st != BEAM_OK) return st;
  if ((st = check(cache)) != BEAM_OK) return st;
  if (cache->n_kv != cfg->n_kv || cache->head_dim != cfg->head_dim || T < 0) return BEAM_ERR_INVALID_ARG;
  if (T == 0) return BEAM_OK;
  const int64_t row = int64_t(cfg->n_q * (g_out ? 2 : 1) + 2 * cfg->n_kv) * cfg->head_dim;
  if (!qkv || !seq_id || !pos || !q_out || (q_norm_w == nullptr) != (k_norm_w == nullptr) || !aligned16(qkv) ||
      !aligned16_or_null(q_norm_w) || !aligned16_or_null(k_norm_w) || !aligned16(q_out) ||
      !aligned16_or_null(g_out) || (token_stride & 7) || token_stride < row)
    return BEAM_ERR_INVALID_ARG;
  return append(cfg, qkv, token_stride, q_norm_w, k_norm_w, seq_id, pos, slot, T, q_out, g_out, cache,
                reinterpret_cast<cudaStream_t>(stream));
}

extern "C" beam_status beam_paged_qkv_gate(const beam_layer_cfg* cfg, const beam_bf16* u,
                                           const beam_bf16* w_qkvg, const beam_bf16* q_norm_w,
                                           const beam_bf16* k_norm_w, const int32_t* seq_id,
                                           const int32_t* pos, const int32_t* slot, int T, beam_bf16* q_out,
                                           beam_bf16* g_out, const beam_paged_kv* cache, void* ws,
                                           size_t ws_bytes, beam_stream_t stream) {
  using namespace beam;
  using namespace beam::paged;
  beam_status st = check_cfg_attn(cfg);
  if (st != BEAM_OK) return st;
  if ((st = check(cache)) != BEAM_OK) return st;
  if (cache->n_kv != cfg->n_kv || cache->head_dim != cfg->head_dim || T < 0) return BEAM_ERR_INVALID_ARG;
  if (T == 0) return BEAM_OK;
  if (!u || !w_qkvg || !q_norm_w || !k_norm_w || !seq_id || !pos || !q_out || !g_out || !ws || !aligned16(u) ||
      !aligned16(w_qkvg) || !aligned16(q_norm_w) || !aligned16(k_norm_w) || !aligned16(q_out) ||
      !aligned16(g_out) || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return BEAM_ERR_INVALID_ARG;
  const int H = cfg->hidden, rows = (2 * cfg->n_q + 2 * cfg->n_kv) * cfg->head_dim;
  Carver cv{static_cast<char*>(ws), ws_bytes};
  uint16_t* z = cv.take<uint16_t>(size_t(T) * rows);
  if (!cv.ok) return BEAM_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = T >= kGemmMinT && tc::gemm_supported(u, H, w_qkvg, H, H)
                            ? tc::gemm_bf16(u, T, H, H, w_qkvg, rows, H, z, rows, true, s)
                            : launch_gemv<kOutBF16>(w_qkvg, rows, H, u, T, nullptr, z, rows, s);
  if (e != cudaSuccess) return cuda_status(e);
  return append(cfg, z, rows, q_norm_w, k_norm_w, seq_id, pos, slot, T, q_out, g_out, cache, s);
}

// Attention of a drafted tree over the paged cache: what its kernel (paged_tree.cu) and the join of its partials
// (paged_tree_join.cu) share. The kernel is compiled as a unit of its own, without relocatable device code, since the
// split of its registers between warps (setmaxnreg) needs that; so it does not reach the device status word, and hands the
// bits to the join.
#pragma once

#include <math.h>

#include "mma.cuh"
#include "paged.cuh"

namespace beam {
namespace paged {
namespace tree {

constexpr int BK = 64;            // keys of a block
constexpr int ROWS = 128;         // rows of a tile
constexpr int kNodes = 64;        // tree rows of a sequence at most
constexpr int kMaxSeqs = 256;     // sequences of one launch
// What an item costs beside its blocks (filling and draining the streams, queries, references, output), in blocks of one
// tile; a range costs four blocks more at least. In us, 32 sequences of 1 to 16 nodes over up to 16K keys / 8 over up to 2K:
//   cost             8         12         14         16         20         24         36
//   D 128  BF16   295/30    251/30     234/29     234/30     219/33     215/33     202/39
//          FP8    326/34    271/35     259/36     259/39     266/45     269/46     278/54
//          NVFP4  335/34    280/35     272/36     270/39     270/45     272/46     280/54
//   D 64   BF16   174/21    147/22     146/22     146/24     147/26     149/27     154/31
//          FP8    240/26    241/29     244/31     247/34     245/37     250/39     253/45
// A full batch gains from a high cost up to the item's own, above all at D 128 (below it the last ranges, of short sequences,
// take twice as long as the others); a small one loses by it, as it then has fewer ranges than there are SMs.
constexpr int kItemBF16 = 20, kItemQuant = 14;
constexpr int kGrid = 152;        // CTAs at most (the workspace is sized for this many)
constexpr int kFlush = 128;       // blocks of a stream between flushes of O: 1024 MMAs
constexpr float kNegInf = -INFINITY;
constexpr int kRescale = 8;       // log2 of what a block's weights may come to before the running max is taken anew
// Over quantised pages: log2 of the largest P when the references are taken (it may be just below twice that when they are
// taken anew). f16 rounds a P below its normal range by up to 2^-25, and once more where a block's first half is brought
// to new references: 1.5 x 2^-25 in all, less than 2^-32 of the largest.
constexpr int kBias = 8;
constexpr unsigned kMostP = 0x7BFFu;   // f16's largest number: past it (an infinity) the references are taken anew
constexpr int kRise = 15 - kBias;      // where another row has them looked at, P may rise by this power: to 2^15, a number of f16

struct Params {
  const uint16_t* q;
  const uint16_t* g;
  const uint16_t* gate_bias;
  const int32_t* seq_id;
  const int32_t* row_start;
  const int32_t* base;
  const uint64_t* mask;
  uint16_t* og;
  float* part_acc;   // [kGrid][2][2][ROWS][D]: partials of a range's first and last item, by tile
  float2* part_ml;   // [kGrid][2][2][ROWS]
  float* flush;      // [kGrid][2][ROWS][D]
  int4* join;        // [kGrid][2]: item that begins in the range and runs on: (head, item, parts, tiles), (row0, n, status bits of the CTA, -)
  beam_paged_kv c;
  int N, T, n_q, n_kv, G, max_pos, shift;
  int least, item;   // least cost of a range; cost of an item beside its blocks, in blocks of one tile
  int head_rows, tail_rows;   // whether rows before the first and behind the last sequence are this launch's
  float sl2;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Four neighbouring outputs, gated, rounded once.
__device__ __forceinline__ uint2 finish4(bool gated, float4 o, uint2 g, float bias) {
  if (gated) {
    o.x *= rcp(1.f + __expf(-(bf_lo(g.x) + bias)));
    o.y *= rcp(1.f + __expf(-(bf_hi(g.x) + bias)));
    o.z *= rcp(1.f + __expf(-(bf_lo(g.y) + bias)));
    o.w *= rcp(1.f + __expf(-(bf_hi(g.y) + bias)));
  }
  return make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}
// Joins the partials of a launch of the kernel with `grid` CTAs.
cudaError_t join(const Params& p, int grid, cudaStream_t st);

}  // namespace tree
}  // namespace paged
}  // namespace beam

// Attention over key ranges: what its kernels and their host side share.
#pragma once
#include <cuda.h>

#include "ops.h"

namespace httm {

constexpr int kAttnTile = 128;          // keys, or query rows, of one tensor-core tile
constexpr int kAttnD = 64;              // channels of a tile; narrower heads are padded with zeros
constexpr int kAttnMaxQ = 1 << 21;      // queries of one sequence
constexpr int kAttnMaxParts = 64;       // key splits of one forward work item

// One call, passed to the kernels by value.
struct AttnArgs {
  int B, H, K, G, L, N, d;              // G = H / K query heads share a key head
  float scale, scale_log2;              // softmax scale; times log2(e)
  const int32_t *kb, *ke;               // [B, L], or null
  View q, k, v, out, dout, dq, dk, dv;
  const float* lse_in;
  float* lse;
  DevState* st;
};

// The 4-D tensor map (channels, tokens, heads, batch) of a bf16 view, boxes
// of `box` tokens x 64 channels with 128-byte swizzle; what lies behind the
// last token or channel reads as zero.  A broadcast dimension (stride 0) has
// extent 1 in the map: its coordinate is multiplied by 0.  `spare`: the base
// address where the view has none (no tokens: nothing is loaded through it).
struct AttnMap {
  CUtensorMap map;
  int hmul, bmul;
};
bool attn_map(AttnMap* m, const View& v, const void* spare, int d, int tokens, int heads, int batch, int box);

// Forward: work items of up to tile_rows query rows, each in `parts` key ranges.
// With at most kAttnFewRows rows a key head the kernel for few rows runs.
constexpr int kAttnFewRows = 32;
constexpr int kAttnCluster = 8;         // parts of few rows that are added up inside one launch
constexpr int kAttnRangePart = 68;     // floats of a partial row: O (64), sum, maximum (log2), 2 unused
struct AttnFwdPlan {
  bool few, pair;                       // the kernel: for few rows, two blocks an SM, else one
  int rows, tile_rows, row_tiles, parts;   // rows = L * G of one key head
  long long items;                      // B * K * row_tiles
  size_t part_bytes;
};
// `ranges`: are there key ranges (few rows are split otherwise then)?
AttnFwdPlan attn_fwd_plan(const httm_attention& a, bool ranges);
int attn_rows_parts(const httm_attention& a, bool ranges);
cudaError_t launch_attn_rows(const AttnArgs& a, const AttnFwdPlan& p, float* part_out, cudaStream_t s);
cudaError_t launch_attn_fwd(const AttnArgs& a, const AttnFwdPlan& p, void* ws, cudaStream_t s);

// Backward workspace: per query row -lse * log2(e) and -D (D = dout . out),
// padded to whole steps, both again as tensor-core operands, the key range of
// every query row and of every step, then the partial sums of split key
// tiles.
struct AttnTileRange {
  int lo, hi;      // union of the live rows' ranges (lo >= hi: none)
  int flo, fhi;    // intersection: keys [flo, fhi) are seen by every live row
  int dead;        // rows of the sequence with an empty range
  int pad[3];
};
struct AttnBwdPlan {
  int kv_groups, q_groups;              // groups a block of the two kernels (1 or 2)
  int step, q_tiles, k_tiles, Lp;       // tiles of `step` queries, of 128 keys; Lp: rows kept per head
  int kv_parts;                         // splits of the queries of one key tile
  size_t stat, extra, range, tiles, part, total;
};
AttnBwdPlan attn_bwd_plan(const httm_attention& a);
cudaError_t launch_attn_bwd(const AttnArgs& a, const AttnBwdPlan& p, void* ws, cudaStream_t s);

}  // namespace httm

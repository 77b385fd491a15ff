// How moe_shared_gemm_lora_bf16 computes a shape: the kernels and splits that lora.hip launches and
// the workspace that they fill, from one function, so that no launch writes more than the size that was
// asked of the caller.  Host code without HIP.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/moeq_lora.h"

namespace moeq {

struct LoraShape {
  int M, N, K, L, slices, r;
  int64_t ld_a;
  int epilogue;
};

constexpr int kSlotK = 64;                               // K of a slot of the LDS rings
constexpr int kMaxSplits = 4;                            // of K, of more than kFewRows rows

// One launch for K up to 256, if a workgroup has at most 8 pieces of 16 ranks to form (two a wave; an
// adapter per row at most) and the workgroups, which all read x and W, fit the card in one go.  us in one
// launch against two: 3 rows x 192 x 256 5.7 and 7.2 (with the host's time 8.6 and 11.8), 64 x 4096 x 256
// 7.6 and 12.6, 512 x 1024 x 256 8.3 and 12.5, 1024 x 512 x 64 8.1 and 11.9; 16 rows x 1024 x 256 with 4 / 8 /
// 16 pieces 7.1 / 8.3 / 10.7 against 9.1 / 9.2 / 9.3, 16 x 1024 x 64 with 32 15.0 and 11.6; 768 workgroups
// (192 x 4096 x 256) 11.3 and 15.0, 1024 (256 x 4096 x 128) 15.4 and 9.7.  K = 512 with operands of all of K
// in flight (16 x 1024): 10.4 and 9.2.
constexpr int kShortK = 256, kShortItems = 8, kShortGrid = 768;
inline bool is_short(const LoraShape& s) {
  const int64_t cols = s.epilogue == MOEQ_EPI_SILU_MUL ? s.N / 2 : s.N;
  return s.K <= kShortK && std::min(s.L, std::min(s.M, 16)) * ((s.slices * s.r + 15) / 16) <= kShortItems &&
         int64_t((s.M + 15) / 16) * ((cols + 63) / 64) <= kShortGrid;
}

// Up to 64 rows are multiplied by lora_few_kernel.  Against the tiles, us: 33 rows x 8192 x 4096 22.9 and
// 26.9, 48 rows 24.6 and 28.0, 64 rows 27.6 and 29.9, 64 rows of rank 64 x 4096 x 4096 23.4 and 32.5.
constexpr int kFewRows = 64, kFewCols = 64;

// The few rows' u: a wave takes 16 rows of one adapter x 16 columns x a piece of 512 K (several, if there
// are more than 16)
constexpr int kUPiece = 512, kUSplits = 16;

// Splits of K of the few-row product: 16 slots (1024 K) each, as that is long enough for a ring's start
// to weigh little and short enough for the parts (8 bytes of traffic an element and split), but at least
// 128 workgroups and at most 8 splits, which the join loads at once.  us by splits 2 / 3 / 4 / 8:
// 16 rows x 8192 x 4096 22.9 / 20.7 / 20.0 / 22.5, 64 x 4096 x 4096 23.5 / 20.6 / 18.4 / 20.0, 16 x 2048 x
// 2048 10.8 / 10.4 / 10.1 / 11.7, 16 x 1024 x 4096 13.8 / 12.4 / 10.9 / 10.2, 16 x 2048 x 8192 21.8 / 18.0 /
// 16.8 / 15.7, 1 x 16384 x 4096 37.5 / 30.7 / 29.9 / 33.5.
// Splits of u: one piece each.  16 splits against 4: 18.8 against 20.8 us for 1 row, 20.0 against 21.6
// for 16 (x 8192 x 4096).
struct FewSplit {
  int splits, slots;                                     // slots of 64 K per split
  int u_splits, u_pieces;                                // pieces of 512 K per split of u
};
inline FewSplit few_split(const LoraShape& s) {
  const int ntiles = (s.N + kFewCols - 1) / kFewCols;
  const int slots = s.K / kSlotK > 0 ? s.K / kSlotK : 1;
  const int want = std::min(slots, std::min(8, std::max(slots / 16, (128 + ntiles - 1) / ntiles)));
  const int per = (slots + want - 1) / want;
  const int pieces = (s.K + kUPiece - 1) / kUPiece;
  const int u_per = (pieces + kUSplits - 1) / kUSplits;
  return {(slots + per - 1) / per, per, (pieces + u_per - 1) / u_per, u_per};
}

// Splits of K of the shrink, at most 4 (the tiles add them): for up to 4096 rows, whose blocks of 32 alone
// would leave CUs idle.  Call, us, by splits 1 / 2 / 4: 777 rows x 1504 x 1448 23.2 / 22.0 / 20.9, 1024 x
// 8192 x 4096 93.6 / 87.3 / 84.7, 2048 x 8192 x 4096 135.8 / 129.0 / 130.1, 8192 x 4096 x 4096 274.0 / 275.5 /
// 279.1.
constexpr int kShrinkPiece = 128;
inline int shrink_splits(const LoraShape& s) {
  const int pieces = (s.K + 4 * kShrinkPiece - 1) / (4 * kShrinkPiece);
  return s.M > 4096 ? 1 : std::min(pieces, kMaxSplits);
}

inline int64_t tiles_of(const LoraShape& s, int bm, int bn) {
  return int64_t((s.M + bm - 1) / bm) * ((s.N + bn - 1) / bn);
}

// How more than 64 rows are multiplied: tiles of bm x bn by `groups` groups of waves, K split over
// `splits` workgroups (1: whole tiles, the shrink ahead of them).  The larger the tile the fewer bytes
// reach LDS per product, and a CU takes in some 45 KB of them a microsecond whatever it has in flight
// (rows that L2 has wait behind the w rows that it has not); but there are 256 CUs to fill.  So the
// largest tile that is met often enough, and below that K is divided: between two groups of waves of a
// workgroup while one tile a CU fills the card in one go, else between workgroups.  us, K = 4096, one
// slice, 16 adapters mixed, rows x columns:
//                 256   256x128   128   128, 2 groups   128 / 2   128 / 4   64    64 / 2   64 / 4
//    2048 x 8192  128     141     160        182           240      310     330
//    1280 x 8192  108     132     125        130           148      187     201
//    1024 x 8192  105      75      83         95           116      150     154     202     231
//     768 x 8192  106      70      79         93            94      112     120     142     172
//     640 x 8192           65      76                       86               99
//     512 x 8192  107      68      62         53            67       78      84      99     127
//     512 x 4096  105              58         51            39       44      47      53      66
//     256 x 8192  111              60         55            42       48      51      57      65
//     128 x 8192  113              62         57            39       36      37      41      44
//     128 x 4096  112              60         55            32       27      34      26      28
//     128 x 2048  101              51         40            24       17      26      17      15
//    1024 x 9216  104             114
//     600 x 12800 104     114      80
//     300 x 19456 109     119      85
//     256 x 18432 116      75      88        100            92             101
//     512 x 7168           56      47         41            46              60      67
//     512 x 6144           56      47         39            43              49      60
//     512 x 4224           56      46         39            41              50      50
//     100 x 65536 170     154     141
//      72 x 40960 124     133     104        119           121             101     121
//      72 x 20480 110      72      68         64            69              64      67
//      72 x 16384 110      68      65         59            50              55      56
// and at K = 1024:
//    1024 x 9216   46              43
//     600 x 12800  47      45      30
//     256 x 18432  60*     37*     39*        47*           50*             44*           (* K = 1536)
//     512 x 8192                              22                            29
//     512 x 7168           28      24         22            28              28      35
//     512 x 4224           27      23         21            25              25      27
//     512 x 4096           27      23         21            19              19      23
//      72 x 20480  48      31      29         25            30              28      33
// Tiles of 128 rows and columns take half of a CU: up to 512 of them are one go, and quicker than larger
// tiles that one go of 256 does not fill; a tile of 256 rows for up to 128 is half empty.  From 129 to 199
// of them at long K groups and splits are within a tenth, either way by the adapters' ranks (512 x 6144
// 39.3 and 43.4 with rank 16, 512 x 4224 with two slices of rank 64 91 and 84).  Tiles that the last rows
// leave mostly empty weigh less: hence the bound on tiles of 64 (300 x 6400, 150 tiles of 128 and 500 of 64,
// K = 2048: 26.2 in groups, 24.1 in tiles of 64).  64 for short K while it fills the card: 512 x 4096 x
// 2048 24.2 against 26.5 (128, 2 groups) and 23.5 (128 / 2); x 1024 18.7, 21.0, 18.9.
struct TilePlan {
  int bm, bn, groups, splits;
};
inline TilePlan tile_plan(const LoraShape& s) {
  const int64_t t256 = tiles_of(s, 256, 256), t256x128 = tiles_of(s, 256, 128), t128 = tiles_of(s, 128, 128),
                t64 = tiles_of(s, 64, 64);
  if (t128 > 512 && s.M > 128 && (t256 >= 150 || s.K > 2048)) return {256, 256, 1, 1};
  if (t128 > 256) return t256x128 <= 256 ? TilePlan{256, 128, 1, 1} : TilePlan{128, 128, 1, 1};
  if (t64 > 512 && (t128 >= 200 || s.M <= 128 || s.K <= 2048)) return {128, 128, 2, 1};
  if (t64 >= 200 && s.K <= 2048) return {64, 64, 1, 1};
  if (t128 >= 64) return {128, 128, 1, t128 >= 128 ? 2 : 4};
  return {64, 64, 1, t64 >= 100 ? 2 : 4};
}

// Parts are joined by lora_join_kernel up to this many of its workgroups, by 64 x 64 tiles from there
// on: its workgroups end sooner, but one per 16 rows and columns each read u and the plan (128 rows x
// 2048, 1024 workgroups: 15.7 us for the call against 20.9; x 4096, 2048: 26.7 against 29.4; 192 rows of
// gate/up 8192: 45.9 against 43.0; 256 rows, 4096: 51.7 against 44.9).
constexpr int kJoinBlocks = 2400;

struct LoraPath {
  bool one_launch;                                       // lora_short_kernel, which takes no workspace
  bool few;                                              // lora_few_kernel and lora_join_kernel
  int bm, bn, groups;                                    // else tiles
  int splits, slots;                                     // of the product; slots per split (few)
  int u_splits, u_pieces;                                // of u; pieces per split (few)
  bool join_rows;                                        // parts of tiles: joined by lora_join_kernel
  size_t u_bytes, part_bytes;                            // the workspace: u's parts, the product's
  size_t ws_bytes() const { return u_bytes + part_bytes + (few ? 256 : 0); }   // (not 0 for M = 0)
};
// (The workspace is that of the shape without its epilogue: the epilogue decides on one_launch and
// join_rows only.)
inline LoraPath lora_path(const LoraShape& s) {
  LoraPath p = {};
  p.one_launch = is_short(s);
  p.few = s.M <= kFewRows;
  if (p.few) {
    const FewSplit fs = few_split(s);
    p.splits = fs.splits;
    p.slots = fs.slots;
    p.u_splits = fs.u_splits;
    p.u_pieces = fs.u_pieces;
  } else {
    const TilePlan tp = tile_plan(s);
    p.bm = tp.bm;
    p.bn = tp.bn;
    p.groups = tp.groups;
    p.splits = tp.splits;
    p.u_splits = shrink_splits(s);
    const int64_t cols = s.epilogue == MOEQ_EPI_SILU_MUL ? s.N / 2 : s.N;
    p.join_rows = int64_t((s.M + 15) / 16) * (cols / 16) <= kJoinBlocks;
  }
  const auto align256 = [](size_t n) { return (n + 255) & ~size_t(255); };
  p.u_bytes = align256(size_t(p.u_splits) * s.M * s.slices * s.r * sizeof(float));
  if (p.few || p.splits > 1)
    p.part_bytes = align256(size_t(p.splits) * ((s.M + 15) / 16 * 16) * s.N * sizeof(float));
  return p;
}

}  // namespace moeq

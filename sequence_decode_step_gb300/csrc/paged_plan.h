// Which kernel a launch of qw_paged_attention takes (host code, without CUDA headers).
#pragma once
#include <algorithm>
#include <cmath>

namespace qw {

constexpr int kPagedMaxSms = 192;  // that a launch uses at most

constexpr int paged_tc_keys(bool kv_bf16) { return kv_bf16 ? 128 : 64; }  // per tensor-core tile
constexpr int paged_tc_rows(bool act_bf16, bool kv_bf16) {               // query rows per item of them
  return act_bf16 && kv_bf16 ? 256 : 128;
}

// Keys per tile, query rows per item, CTAs and an item's own cost of a launch.
struct PagedPlan {
  bool tc;  // paged_attention_tc.cu, else paged_attention.cu
  int kt, rows, grid, item_units, least_units;
};

// Tiles of 32 KB that an item's q, join and output cost a CTA: 6 us against 1.3 us a tile (3 to 5 give
// the same within 2 % on the ragged cases).
constexpr int kDecodeItemUnits = 5;

// The plan of a launch over `n_seqs` sequences with `n_tokens` new tokens, at most `max_new` of one sequence,
// that meet up to `keys` keys each (the most that the table can hold, as the lengths are on the device; so
// the width of a table has a say). A shared prefix is one sequence with all the tokens.
//
// bf16 pages: up to 16 rows (tokens x heads of a KV head) of a sequence run the mma.sync kernel, in items of 8
// rows that each read its keys; more than 16 the tensor-core tiles, unless there is so little of it that their
// start (5 to 8.5 us more, with q, first product and output) is most of the time.
// Measured per tile and CTA: 1.3 us for 64 keys here, and for 128 keys there 1.5 us (bf16) or 2.9 us (f32 in
// three terms). Calls with 4K prefix keys: 32 rows 20.6 us against 22.5 there, 64 rows 27.4 against 22.9 (f32
// 30.8 and 27.6), 128 rows 44 against 28.7; one chunk of 64 tokens behind 2K keys 26.7 against 21, 512 keys 16.8
// against 20.5. An item of tensor-core tiles costs about 7 us beside them; a share of 2 instead of 4 tiles at
// least lets a 4K prefix of 128 rows use all SMs (36.8 us instead of 40.8 with f32 q).
// f32 pages: the least tile that holds the rows: 2 or 4 with FMAs, 8 or 32 with mma.sync. More than 16
// rows by the same estimate: 3.3 us for 32 rows x 32 keys on mma.sync, 2.5 us for 128 rows x 64 keys on the
// tensor-core tiles, whose start takes 2 us more. Measured, with a key of each sequence's own: a prefix of
// 1K keys and 32 rows 20 us against 27, 256 rows 49 against 37; of 16K keys 66 against 56 and 381 against 103.
//
// The items are those of the whole batch: the rows of all tokens, and at least those of as many sequences as
// have max_new tokens if the tokens are spread evenly. Measured, 16 tokens x 8 heads per KV head behind 4K
// keys: one sequence 19.6 us here and 20.5 there, 32 sequences 204 and 49, 160 sequences 1 421 and 158 (bf16).
// Over 84 batches of 1 to 160 sequences with 3 to 32 tokens and 256 to 4K keys for each pair of types the choice is
// 0.1 % (bf16), 1.2 % (f32 q, bf16 pages) and 4 % (f32) slower than the better kernel in the mean.
inline PagedPlan plan_paged_pass(bool kv_bf16, bool act_bf16, int nkv, int gq, int n_tokens, int n_seqs, int max_new,
                                 long long keys, int sms) {
  sms = std::min(sms, kPagedMaxSms);
  const bool f32 = !kv_bf16;
  const int new_tokens = std::min(max_new, n_tokens);
  const long long rows = (long long)new_tokens * gq, all_rows = (long long)n_tokens * gq;
  const long long seqs = std::min(n_seqs, (n_tokens - 1) / new_tokens + 1);
  PagedPlan p{false, f32 ? 32 : 64, 8, 3 * sms, kDecodeItemUnits, 4};
  if (f32) {
    p.rows = rows <= 2 ? 2 : rows <= 4 ? 4 : rows <= 8 ? 8 : 32;
    if (p.rows > 4) p.grid = 2 * sms;
    if (p.rows > 8) p.least_units = 2;  // (a tile takes 3.3 us: 32 rows x 1K keys 22.5 -> 19.7 us)
  }
  if (rows > 16) {
    auto us = [&](double start, double tile, int kt, int item_rows, int units, int grid) {
      auto tiles_of = [&](long long r) { return (r + item_rows - 1) / item_rows; };
      const double items = (double)nkv * std::max(tiles_of(all_rows), seqs * tiles_of(rows));
      return start + tile * std::ceil(items * (keys / kt + 1 + units) / grid);
    };
    const PagedPlan t{true, paged_tc_keys(!f32), paged_tc_rows(act_bf16, !f32), sms,
                      f32 ? 4 : act_bf16 ? 5 : 3, 2};
    if (us(f32 ? 6 : act_bf16 ? 12.5 : 9, f32 ? 2.5 : act_bf16 ? 1.5 : 2.9, t.kt, t.rows, t.item_units, t.grid) <
        us(4, f32 ? 3.3 : 1.3, p.kt, p.rows, p.item_units, p.grid))
      p = t;
  }
  return p;
}

}  // namespace qw

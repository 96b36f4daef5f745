// How dkv_block_append's launch is divided: host code, apart from the kernels so that it runs without a GPU.
#pragma once

namespace dkv {

constexpr int kAppendWarps = 8;  // of a CTA
constexpr int kAppendIterQ = 8;  // query rows of a lane group for one token
constexpr int kUnit = 16;        // tokens that append_blocks' warps look at together for blocks that begin there
constexpr int kLook = kAppendWarps * 16;  // and a CTA of append_tokens in long calls
// Calls of kLong rows and more look for short blocks with a warp for 16 tokens, not one for each: 4096 rows of one sequence
// 26.8 us, 35.8 with a warp each; 2048 18.1 and 21.4; 1024 10.3 and 11.4; 512 8.4 and 7.5.  About kLookCtas CTAs share
// what there is: 4096 single rows 42 us, 41 with a warp each, by block 179; 1024 16.1 and 15.5; 512 11.1 and 9.1.  (256 CTAs:
// 4096 rows of one sequence 28.6, single ones 40.7.)
constexpr int kLong = 1024, kLookCtas = 128;

// Warps that share a run: with heads of 128 four of four rows each, so that a lane holds 16 fp32 values (4096 rows of 32/8 heads
// 26.8 us; with two warps 27 to 28, with one and two CTAs an SM instead of three 38.7).  Of 64 one (16384 rows of 32 heads
// 88 us, 103 with two: what a warp does once for a run counts more).
constexpr int append_share(int head_dim) { return head_dim == 128 ? 4 : 1; }

struct AppendGeometry {
  int q_items;      // groups of query heads
  int heads;        // of a unit of append_blocks
  int span;         // groups of heads of a unit of append_tokens, 0: short calls, whose units are a token and a group
  int parts;        // CTAs that share what a look of append_tokens finds, in long calls
  int block_ctas, token_ctas, q_ctas;  // CTAs of keys, and of values: by block, by token; of queries
  int grid;
};

// q_heads 0: no queries.
inline AppendGeometry append_geometry(int rows, int q_heads, int kv_heads, int head_dim) {
  constexpr long long kMost = 16 * 3 * 152;  // CTAs of a kind
  const int group_q = kAppendIterQ * 32 / (head_dim / 8), share = append_share(head_dim);
  auto ctas = [&](long long units, int each) {
    const long long c = (units + each - 1) / each;
    return (int)(c < kMost ? c : kMost);
  };
  AppendGeometry a;
  a.q_items = (q_heads + group_q - 1) / group_q;
  const bool all = rows >= kLong;
  const long long chunks = (rows + kUnit - 1) / kUnit;
  a.heads = 1;
  // What a warp finds out about its tokens serves up to four heads, while 2048 warps are left to do so.  In us with one, two and
  // four: 4096 rows of 8 heads of 128 33.8, 29.4, 26.5 (the rule takes four), 2048 rows 19.7, 18.0, 21.2 (two), 1024
  // rows 10.1, 9.3, 12.9 (one), 4096 rows of 2 heads 11.1, 11.6, 11.5 (one); 16384 rows of 32 heads of 64 115, 98, 87
  // (four), 8192 rows of 8 33, 29, 40 (two).
  while (a.heads < 4 && chunks * kv_heads / (2 * a.heads) * share >= 2048) a.heads *= 2;
  a.block_ctas = ctas(chunks * ((kv_heads + a.heads - 1) / a.heads), kAppendWarps / share);
  const long long groups = (kv_heads + 256 / head_dim - 1) / (256 / head_dim), looks = (rows + kLook - 1) / kLook;
  a.span = 0;
  a.parts = 1;
  if (all) {
    // groups of heads that share a look, while kLookCtas are left (16384 rows of 32 heads of 64: 88 us; with a look for
    // each 100)
    for (a.span = 1; a.span < groups && looks * groups / (2 * a.span) >= kLookCtas;) a.span *= 2;
    while (a.parts < 16 && looks * groups / a.span * a.parts < kLookCtas) a.parts *= 2;
    a.token_ctas = ctas(looks * ((groups + a.span - 1) / a.span) * a.parts, 1);
  } else {
    a.token_ctas = ctas(rows * groups, kAppendWarps);
  }
  const long long tokens = (rows + kAppendWarps - 1) / kAppendWarps;
  const long long per = a.q_items ? (kMost + a.q_items - 1) / a.q_items : 0;
  a.q_ctas = (int)(tokens < per ? tokens : per) * a.q_items;
  a.grid = 2 * (a.block_ctas + a.token_ctas) + a.q_ctas;
  return a;
}

}  // namespace dkv

// shared.h -- attention over a shared prefix: the tensor-core pass's plan and launch.
#pragma once

#include "visible.cuh"

namespace attn {
namespace shr {

constexpr int kRows = 128;    // query rows of a tile
constexpr int kKeys = 128;    // keys of a tile
constexpr int kSms = 152;

// How a problem is divided into items, by value to the kernel.  A row is a
// (entry, query, head of the kv head's group) triple, in this order.  Prefix
// items pack the rows of all entries into blocks of two row tiles and walk a part
// of the prefix's key tiles; entry items take the rows of one entry and walk
// its own key tiles, behind the prefix's with `joined`.  A block of one row
// tile (alt) deals its key tiles to both row tiles of the kernel in turn, which
// then hold the same rows and give a partial result each.
struct Work {
  int blocks_a, parts_a, alt_a;   // prefix items: row blocks of a kv head, parts of the prefix
  int blocks_b, parts_b, alt_b;   // entry items: row blocks of an entry and kv head, parts of its list
  int joined;
  int n_a, n_items;               // prefix items (in front), all items
  int piece;                      // rows of a copy: the largest power of two up to 128 that divides a page
  int splits;                     // partial results of a row (1: the items write O)
};

}  // namespace shr

// The pass's plan, from the shape alone.  False: another pass takes the problem.
bool shared_tc_plan(const Problem& p, int page_size, shr::Work& w);
// As prefill_tc_try.  s: room for the plan's partial results.
int shared_tc_try(const Problem& p, const Ext& x, const shr::Work& w, const Split& s, cudaStream_t st, int* used);

}  // namespace attn

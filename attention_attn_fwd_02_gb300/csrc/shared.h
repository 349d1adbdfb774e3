// shared.h -- attention over a shared prefix: the tensor-core pass's plan and launch.
#pragma once

#include "paged.cuh"
#include "visible.cuh"

namespace attn {
namespace shr {

constexpr int kRows = 128;    // query rows of a tile
constexpr int kKeys = 128;    // keys of a tile
constexpr int kSms = 152;

// How the CTAs share the prefix.  A row is a (entry, query, head of the kv
// head's group) triple, in this order; the rows of all entries are packed into
// blocks of two row tiles, and a unit -- a block of a kv head -- walks all of the
// prefix's key tiles.  The tiles of all units, laid end to end, are cut into shares of
// equal cost, one a CTA; a unit's result is the merge of its fragments, one of
// each CTA that has tiles of it.
struct Shares {
  // Costs, about 0.2 us each: a key tile of both row tiles, of the one row tile that a kv head's last block may have,
  // and what an item costs besides.
  static constexpr int kTile = 7, kTileAlt = 3, kEnd = 10;
  int ctas, tiles;        // shares; key tiles of the prefix
  int blocks, alt;        // row blocks of a kv head; 1: the last has one row tile
  // Share c begins at tile `tile[c]` of unit `unit[c]`; the first fragment's number in its unit.  (Worked out on the
  // host: the kernels' registers have no room for 64-bit divisions.)
  int unit[kSms + 1];
  int16_t frag[kSms];
  int tile[kSms + 1];

  __host__ __device__ bool is_alt(int u) const { return alt && u % blocks == blocks - 1; }
  // Cuts the tiles of `heads` kv heads; ctas has to leave every share a tile's cost at least.  Returns the most
  // fragments of a unit.
  int cut(int heads);
};

// How a problem is divided into items, by value to the kernels.  Prefix items are
// fragments of units (above).  Entry items take the rows of one entry and walk a
// part of its own key tiles, behind the prefix's with `joined`.  An item of one
// row tile (alt) deals its key tiles to both row tiles of the kernel in turn,
// which then hold the same rows and give a partial result each.  A row's
// partial results are its unit's fragments, then its entry items'.
struct Work {
  Shares pre;                     // pre.ctas = 0: no prefix items
  int blocks_b, parts_b, alt_b;   // entry items: row blocks of an entry and kv head, parts of its list
  int joined;
  int n_b;                        // entry items
  int piece;                      // rows of a copy: the largest power of two up to 128 that divides a page
  int own_slot;                   // first partial result of the entry items (or of the decode pass over own keys)
  int splits;                     // partial results of a row (1: the items write O)
  int one_tile;                   // every item has one row tile
  int own_sms;                    // SMs that the decode pass over own keys is planned for
};

}  // namespace shr

// The pass's plan, from the shape alone.  False: another pass takes the problem.
bool shared_tc_plan(const Problem& p, int page_size, shr::Work& w);
// Enqueues a plan's passes; s: room for its partial results.  own, x_own, ws_own: for one query an entry, the problem of
// the entries' own keys and the decode pass's workspace.  As prefill_tc_try.
int shared_tc_try(const Problem& p, const Ext& x, const shr::Work& w, const Split& s, const Problem& own, const Ext& x_own,
                  void* ws_own, cudaStream_t st, int* used);
// Merges a plan's partial results, as the programmatic dependent of the pass in front.  own: the decode pass over own
// keys, whose cut units it joins too (null: there was none).
cudaError_t launch_shared_merge(const Problem& p, const shr::Work& w, const Split& s, const paged::Work* own,
                                cudaStream_t st);

}  // namespace attn

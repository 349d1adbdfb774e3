// shared.h -- attention over a shared prefix: the tensor-core pass's plan and launch.
#pragma once

#include "paged.cuh"
#include "visible.cuh"

namespace attn {
namespace shr {

constexpr int kRows = 128;    // query rows of a tile
constexpr int kKeys = 128;    // keys of a tile
constexpr int kSms = paged::kSms;

// A list of units cut into shares of equal cost, one a CTA: a unit is a block of
// rows, of one or two row tiles, with its key tiles.  Units lie end to end;
// share c begins at tile `tile[c]` of unit `unit[c]`, and what it has of a unit
// is a fragment, the first of them number frag[c] of its unit.  (Worked out on
// the host: the kernel's registers have no room for 64-bit divisions.)
struct Shares {
  // Costs, about 0.2 us each: a key tile of both row tiles, of one, and what a fragment costs besides.
  static constexpr int kTile = 7, kTileAlt = 4, kEnd = 20;
  int ctas;               // 0: there is no list
  int unit[kSms + 1];
  int tile[kSms + 1];
  int16_t frag[kSms];
  int n_cut;              // joined: the shares that end a unit which an earlier one began
  int16_t cut[kSms];
};

// How a problem is divided, by value to the kernels.  A row is a (entry, query,
// head of the kv head's group) triple, in this order.
//   packed   The rows of all entries are packed into blocks of 256, and a unit
//            (kv head by kv head, its blocks in turn) walks the prefix's key tiles.
//            The entries' own keys are walked by entry items, rows of one entry
//            (in turn over the CTAs), or by the decode pass for one query an
//            entry.  A row's partial results, its unit's fragments and then its
//            own keys', are merged.
//   joined   A unit is a block of 256 rows of one entry (the last blocks, which
//            see the most keys, in front, then entry by entry, kv head by kv
//            head) and walks the prefix's tiles and behind them its own.  As many
//            units as every CTA can have the same number of are dealt whole
//            (entry items) and write O.  The list has those left over, as if every
//            entry had the k_len own keys it may have; the tiles of one that has fewer are
//            cut in the same proportions.  A share keeps its first fragment,
//            where it began in the middle of a unit, and its last, where it
//            ends in one, for the merge.
// A block whose rows fit one row tile (`alt`: the last one) deals its key tiles
// to both row tiles of the kernel, which then hold the same rows, in turn.
struct Work {
  Shares list;
  int joined;
  int blocks, alt;                // row blocks of a kv head (packed) or of an entry and kv head (joined)
  int blocks_b, alt_b, parts_b;   // entry items: row blocks of an entry and kv head, parts of their lists
  int n_b, first_b;               // entry items, and the first one's number
  int piece;                      // rows of a copy: the largest power of two up to 128 that divides a page
  int own_slot;                   // packed: first partial result of own keys
  int splits;                     // packed: partial results of a row.  joined: 1 if a share keeps any
  int one_tile;                   // every item has one row tile
  int own_sms;                    // SMs that the decode pass over own keys is planned for
  // Partial results: numerators over their sums, natural maxima (-inf: no visible key), sums.  packed: [B H q_len][splits]
  // in (entry, head, query) order; joined: [ctas][2][256].  note: packed, the number of each unit's fragments.
  // (float32 has no list: every row has own_slot results of the prefix, and note is null)
  float *part_o, *part_m, *part_l;
  int* note;

  __host__ __device__ int block_of(int u, int B, int G) const { return joined ? blocks - 1 - u / (B * G) : u % blocks; }
  __host__ __device__ bool is_alt(int block) const { return alt && block == blocks - 1; }
};

// joined: the tiles of a unit of block `block`, at most, behind `pre` tiles of the prefix (rows without keys have one too).
__host__ __device__ inline int most_tiles(const Problem& p, int block, int pre) {
  const int64_t rows = (int64_t)p.Sq * p.qpg, end = (int64_t)(block + 1) * 2 * kRows;
  const int64_t q = ((end < rows ? end : rows) - 1) / p.qpg;   // the block's last query
  int64_t own = p.Sk - p.prefix;
  if (p.causal) own = clamp64(q + 1 + (p.align_klens ? own - p.Sq : p.coff - p.prefix), 0, own);
  const int tiles = pre + (int)((own + kKeys - 1) / kKeys);
  return tiles > 0 ? tiles : 1;
}

// Time of the decode pass over pages where it takes the prefix's keys too, once an entry and `per` heads of a kv head, in
// us: out of L2 (l2: bytes a us), and at least once out of HBM.  Long lists (over `uncut` keys, more than a cluster takes) of
// few units are cut into many fragments, which one CTA a unit joins.  (One entry of 8/2 heads, head_dim 64, bf16, behind 42382
// keys: 34.8 us, of them some 24 the join; 4 of 8/1 heads, head_dim 128, behind 49285: 49.2, some 30.)
inline double decode_us(const Problem& p, int per, int es, double l2, int uncut) {
  const double units = (double)p.B * p.G * ((p.qpg + per - 1) / per), keys = (double)p.prefix * p.D * 2 * es;
  const double far = p.G * keys / 6.5e6, near = units * keys / l2;
  double join = 0.0;
  if (units * 8 <= 3 * kSms && p.Sk > uncut) {
    const double width = (double)(p.qpg < per ? p.qpg : per) * p.D / 4 / 256;   // of the joining CTA's threads
    join = 4.0 + 0.2 * 3 * kSms / units * (width < 0.25 ? 0.25 : width > 1 ? 1 : width);
  }
  return (near > far ? near : far) + join;
}

}  // namespace shr

// The pass's plan, from the shape alone.  False: another pass takes the problem.
bool shared_tc_plan(const Problem& p, int page_size, shr::Work& w);
// Bytes of a plan's partial results and notes.
size_t shared_tc_bytes(const Problem& p, const shr::Work& w);
// Enqueues a plan's passes.  own, x_own: for one query an entry, the problem of the entries' own keys, whose decode pass
// has its workspace behind the plan's.  As prefill_tc_try.
int shared_tc_try(const Problem& p, const Ext& x, shr::Work& w, const Problem& own, const Ext& x_own, void* workspace,
                  cudaStream_t st, int* used);
// float32: the pass over each entry by itself and its merge (s: parts of the entries' tile lists), and the packed plan
// with its bytes and passes, as for the tensor cores.
int shared_f32_try(const Problem& p, const Ext& x, const Split& s, cudaStream_t st, int* used);
int shared_f32_parts(const Problem& p);
bool shared_f32_plan(const Problem& p, shr::Work& w);
size_t shared_f32_bytes(const Problem& p, const shr::Work& w);
int shared_f32_packed(const Problem& p, const Ext& x, shr::Work& w, const Problem& own, const Ext& x_own, void* workspace,
                      cudaStream_t st, int* used);
// Merges a plan's partial results, as the programmatic dependent of the pass in front.  own: the decode pass over own
// keys, whose cut units it joins too (null: there was none).
cudaError_t launch_shared_merge(const Problem& p, const shr::Work& w, const paged::Work* own, cudaStream_t st);

}  // namespace attn

// pct_cache.h -- kernel arguments and launchers of the paged key-value
// cache: page plan, row writes, tree attention, commit of accepted paths.
#pragma once

#include "pct_internal.h"

namespace pct {

// profiler kinds after those of ProfKind
constexpr int PROF_PLAN = 12, PROF_CACHE_WRITE = 13, PROF_ATTEND = 14,
              PROF_JOIN = 15, PROF_COMMIT = 16, PROF_ROTARY = 17, PROF_RELEASE = 18,
              PROF_FORK = 19, PROF_COMPACT = 20, PROF_SHARE = 21;

constexpr int kMaxTokens = 1 << 30;  // positions of a request at most

// Paged cache geometry shared by the kernels.
struct PageGeom {
  int batch, N, n_pages, max_pages;
  int shift;  // log2 of the page size
  int Hkv, D;
  const int32_t* table;    // [batch][max_pages]
  const int32_t* ctx_len;  // [batch]
  const int32_t* n_nodes;  // [batch] or null (N in every request)
};

struct PlanArgs {
  PageGeom g;  // table unused
  const int32_t* depth;
  int32_t *table, *held, *ring, *ring_state;
  int64_t* slot;
  int32_t *pos, *missing;
  int32_t* served;  // [batch] or null
  int4* req;   // [batch] {first taken, first given back, held before, after}
  int2* ring0; // ring head and count before the call
};
hipError_t launch_cache_plan(const PlanArgs& a, hipStream_t s);

struct WriteArgs {
  int64_t rows;
  int64_t n_slots;
  int shift, Hkv, D;
  const uint4 *k, *v;      // 8 elements each
  int64_t ks, vs;          // row strides in 8-element chunks
  const int64_t* slot;
  uint4 *kc, *vc;
};
hipError_t launch_cache_write(const WriteArgs& a, hipStream_t s);

// Rotation of rows on their way into the cache.
struct RotaryArgs {
  int64_t rows, n_slots;
  int shift, Hq, Hkv, D, bf16;
  int rot;            // rotated elements of a head
  int pairs;          // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
  const uint64_t* freq;  // [rot / 2] turns per position in units of 2^-64
  float amp, eps;
  const float *qw, *kw;  // [D] norm weights or null
  const void *q, *k, *v;
  int64_t qs, ks, vs, os;  // row strides in elements
  const int32_t* pos;
  const int64_t* slot;
  void *out, *kc, *vc;
};
hipError_t launch_cache_rotary(const RotaryArgs& a, hipStream_t s);

struct CommitArgs {
  PageGeom g;
  int layers, B;
  int64_t layer_stride;  // in 8-element chunks
  const int32_t *tau, *accept;
  uint4 *kc, *vc;
  int32_t* ctx_out;
};
hipError_t launch_cache_commit(const CommitArgs& a, hipStream_t s);

// Pages that several requests hold.
struct PagesArgs {
  PageGeom g;  // n_nodes: of a trim; table and ctx_len unused
  int32_t *ctx, *table, *held, *ring, *ring_state, *extra;
  int m;                  // places of a free or pairs of a fork, else batch
  const int32_t* places;  // [m] of a free, null: a trim
  int layers;
  int64_t layer_stride;   // in 8-element chunks
  uint4 *kc, *vc;
  int32_t* count;         // scratch of the scans, per segment of pages
};
hipError_t launch_release(const PagesArgs& a, hipStream_t s);
size_t release_workspace(const pct_cache_shape& sh);

struct ForkArgs {
  PagesArgs a;
  const int32_t *src, *dst, *length;  // [m]; length or null
  int32_t* done;
  int4* req;       // [m] {source or -1, place, positions, page of the rest}
  int32_t* claim;  // [batch] first pair that names the place
};
hipError_t launch_fork(const ForkArgs& f, hipStream_t s);

struct CompactArgs {
  PagesArgs a;
  int32_t* table_out;
  int32_t *hole, *high, *rank;  // [n_pages] moves: high[k] to hole[k]
  int32_t* info;                // pages in use, moves
};
hipError_t launch_compact(const CompactArgs& c, hipStream_t s);
size_t compact_workspace(const pct_cache_shape& sh);

// What a share plan leaves for the round's attention.
constexpr int kMaxShareBatch = 1024;
struct ShareView {
  int4* req;          // [batch] {context, nodes, shared pages, packed rows of
                      // its group before its own, or -1: no group}
  int4* groups;       // [batch] {leader, shared positions, rows (0: no such
                      // group), first packed row}
  int2* group_of;     // [batch] {group or -1, its first packed row}
  float* totals;      // positions of the own keys of all requests, requests
                      // with rows, rows times shared positions, unused
  int32_t* rows;      // [batch * (N + 1)] row of each packed row
};
struct ShareArgs {
  PageGeom g;
  int least;                 // positions that a pick must promise
  uint64_t* best;            // [blocks][batch] picks of groups of places
  int blocks;
  int32_t *place, *joined;   // [batch]
  int32_t *leader, *shared;       // [batch]
  ShareView view;
};
constexpr int kShareBlocks = 512;
int share_blocks(const pct_cache_shape& sh);
hipError_t launch_share(const ShareArgs& a, hipStream_t s);

struct AttendArgs {
  PageGeom g;
  int Hq, G;        // query heads, query heads per key-value head
  int bf16;         // element type: 1 bf16, 0 fp16
  float c;          // |scale| * log2(e); 1 for a scale of zero
  uint32_t qand, qxor;  // bits that carry the scale's sign into two elements
  const void* q;
  int64_t qs;       // row stride in elements
  const void *kc, *vc;
  const uint64_t* mask;
  int words;        // 64-bit words of a mask row
  void* out;
  float* lse;
  ShareView share;  // of attention in two parts
};
// Which positions a launch goes through: all of a request's, or, where
// requests share a prefix, the shared ones of a group (whose rows are packed
// as if they were one request's) or a request's own ones behind them.
constexpr int kAllKeys = 0, kSharedKeys = 1, kOwnKeys = 2;
// Tile of a call: heads padded to dp elements, mt rows per workgroup (16: all
// waves hold these rows and have keys of their own; 64, 128: they hold
// different ones and share the keys), steps of ks keys, n_wg runs at most (a multiple of 8); the join
// goes through the `tiles` row tiles (row_tiles of a request at most), or
// through the runs where these are fewer (row_tiles 0), and adds so many
// groups of runs side by side.
struct AttendPlan {
  int dp, mt, ks, n_wg, row_tiles, tiles, groups;
};
// Keys of a tile: of a wave's own one, of one that the waves share.
constexpr int kRowsKb = 32, kTilesKb = 64;
// Steps of a run at least while runs are few, and beyond (runs_for).  Tiles of
// 64 rows, 16 rows of 4 heads over 1 k positions, from 6 or from 2 steps on:
// 20 or 14 us; from 5, 6 and 8 on with many runs: 65 rows over 4 k 29.6,
// 28.9, 27.0, 4 requests of 65 rows over up to 2 k 31.7, 31.4, 32.2 us.  Of
// 128 rows, 65 rows over 4 k, from 3, 4, 6 on: 35, 29, 34 us.  Runs of the
// rows kernel leave a few rows only.
constexpr int kRowsFew = 1, kRowsLeast = 1, kTilesFew = 2;
// Up to so many tiles of 128 rows by 64 keys, if requests are as long as the
// block table allows, rows are cut into tiles of 64: more runs with a shorter
// chain of steps each, for twice the reads of keys (from the L2) and of
// operands.  4 requests of 256 rows over 656 positions (2816 tiles) 54 us
// with 128, 37 with 64; 65 rows over 2 k (792) 29, 23; 256 rows over 9 k
// (9280) 79, 82, over 32 k (32 k tiles) 168, 214.  Not for heads past 128,
// whose 64 rows leave one wave per SIMD (256 rows over 2 k, D = 256: 53, 67).
constexpr int kHalfUnits = 6144;
constexpr int kWhole = 6;  // a row tile of so few steps stays in one run
constexpr int tiles_least(int mt) { return mt == 64 ? 8 : 4; }
constexpr int kCus = 256;  // compute units of an MI355X
// In two parts (below) a row tile counts as so many steps more than it has, for
// its beginning and its end, or runs of many short row tiles would end last.
// (In two launches: 123 requests of one token over 64 .. 4096 own keys each and
// two shared prefixes 255 us without, 16 requests of 65 rows 218; with 1 / 1
// step of few rows / of shared tiles 216 and 210, with 1 / 3 209 and 202, with
// 2 / 2 213 and 204, with 1 / 6 210 and 208.)
constexpr int kRowsExtra = 1, kTilesExtra = 3;
// fp16 holds probabilities times 2^kLift (k_attend_impl.h has the reason).
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;
// Per run two row tiles of sums (times 2^kLift) that other runs continue: slot 0 of a tile
// that an earlier run began, slot 1 of one that this run began and did not
// end.  meta {request, head << 20 | row tile, first run, last run} of a row
// tile that is cut, w < 0: it is not; its index is the row tile's if
// row_tiles > 0, else the first run's.
//
// In two parts every row tile leaves sums, those that are not cut in a slot
// of their own behind the runs' (2 n_wg + index).  meta {first run, last run
// or -1: not cut}.  A group's row tiles begin at index first packed row * G /
// mt + group within those of a head: no fewer than it has lie before the next
// group's.
struct AttendWs {
  float* o;    // [2 n_wg (+ tiles)][mt][dp]
  float2* ml;  // [2 n_wg (+ tiles)][mt] {m, sum}
  int4* meta;  // [n_wg] or [tiles]
  int row_tiles;  // of a request at most (shared keys: of all groups)
  int n_wg;
};
hipError_t launch_attend_d64(const AttendArgs&, const AttendPlan&,
                             const AttendWs&, hipStream_t);
hipError_t launch_attend_d96(const AttendArgs&, const AttendPlan&,
                             const AttendWs&, hipStream_t);
hipError_t launch_attend_d128(const AttendArgs&, const AttendPlan&,
                              const AttendWs&, hipStream_t);
hipError_t launch_attend_d192(const AttendArgs&, const AttendPlan&,
                              const AttendWs&, hipStream_t);
hipError_t launch_attend_d256(const AttendArgs&, const AttendPlan&,
                              const AttendWs&, hipStream_t);
// The two parts of a call: arguments, tiles and workspaces of the shared keys
// (no workgroups: no part) and of the own ones.
struct AttendParts {
  AttendArgs a[2];
  AttendPlan p[2];
  AttendWs ws[2];
};
hipError_t launch_parts_d64(const AttendParts&, hipStream_t);
hipError_t launch_parts_d96(const AttendParts&, hipStream_t);
hipError_t launch_parts_d128(const AttendParts&, hipStream_t);
hipError_t launch_parts_d192(const AttendParts&, hipStream_t);
hipError_t launch_parts_d256(const AttendParts&, hipStream_t);
hipError_t launch_tree_attention(const AttendArgs& a, void* ws,
                                 hipStream_t s);
size_t tree_attention_workspace(const pct_cache_shape& sh);
AttendPlan plan_attend(int requests, int64_t rows, int64_t cap, int Hkv,
                       int D);
hipError_t launch_shared_attention(const AttendArgs& a, void* ws,
                                   hipStream_t s);
size_t shared_attention_workspace(const pct_cache_shape& sh);

// A request's lengths, clamped to what the calls accept.
__host__ __device__ inline int clamp_ctx(int c) {
  return c < 0 ? 0 : (c > kMaxTokens ? kMaxTokens : c);
}
__host__ __device__ inline int clamp_nodes(int n, int N) {
  return n < -1 ? -1 : (n > N ? N : n);
}

}  // namespace pct

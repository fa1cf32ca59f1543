// tree_shares.cuh -- how the tree attention's work is shared out.
//
// A unit is one (batch element, layer, KV head); its query rows are the
// element's nodes of the unit's g query heads.  An item is a part of a unit's
// rows that one CTA takes at a time, with all of the unit's key tiles (first
// the cached rows, then the nodes).  The items of all units, in the order
// (batch element, layer, KV head, rows, key tile), form one line of jobs, and
// CTA c takes the jobs [c * share, (c + 1) * share): ragged lengths balance,
// and a few long sequences still fill the GPU.  The line follows from seq_lens
// on the device.
//   narrow kernel (PAIRS false): an item is one row tile, a job one key tile
//   wide kernel (PAIRS true):    row tiles of 128, two to an item while there
//     are two left (a job is then one (row tile, key tile); a border between
//     shares falls on the key tile that holds it)
#pragma once

#include "common.cuh"
#include "paged.cuh"

namespace spk {

// Jobs that a share may have more where that makes it whole units (of like
// lengths), so that nothing is cut and joined.  With 0, 3, 6 and 12 jobs: 16 nodes
// over 320 rows, 512 units, 45.9, 39.1, 39.0, 39.1 us; 8 nodes over 1000 rows, 160
// units, 37.0, 37.1, 37.0, 41.2; 24 nodes over 3000 rows, 256 units, 89.0, 90.1,
// 89.9, 79.4; one node over 320 rows, 512 units, 24.3, 22.6, 22.6, 22.6.
constexpr int kJoinJobs = 6;

struct TreeElement {       // a batch element
  int seq, len, live, tiles;
};

// Length and live nodes of batch element b; an element whose sequence, length
// or node count is out of range has no rows (its outputs stay unwritten).
// The nodes lie in the last cached tile, at the next multiple of 8 rows, where
// all T of them fit behind its rows; otherwise in tiles of their own.
template <int KEYS>
__device__ __forceinline__ bool tree_fused(const TreeParams& p, int len) {
  const int rest = len % KEYS;
  return p.has_tree && rest > 0 && ((rest + 7) & ~7) + p.node_rows <= KEYS && p.T <= KEYS;
}

template <int KEYS>
__device__ __forceinline__ TreeElement tree_element(const TreeParams& p, int b, bool record) {
  TreeElement e;
  e.seq = p.seqs != nullptr ? __ldg(p.seqs + b) : b;
  e.live = p.n_live != nullptr ? __ldg(p.n_live + b) : p.T;
  bool ok = e.seq >= 0 && e.seq < p.n_seqs;
  e.len = ok ? __ldg(p.lens + e.seq) : 0;
  ok = ok && e.live >= 0 && e.live <= p.T && e.len >= 0 && e.len <= static_cast<long long>(p.max_pages) * p.page_rows;
  if (!ok) {
    if (record) record_error(SPK_DEVERR_INDEX, b);
    e.seq = 0;
    e.len = 0;
    e.live = 0;
  }
  const int nodes = p.has_tree && !tree_fused<KEYS>(p, e.len) ? (e.live + KEYS - 1) / KEYS : 0;
  const int t = (e.len + KEYS - 1) / KEYS + nodes;
  e.tiles = e.live == 0 ? 0 : (t > 0 ? t : 1);   // rows without any key still get their zeros
  return e;
}

// Key tile t of an element, by columns: [0, rows) the cached rows first ..,
// [off, off + nodes) the nodes node0 .., nothing behind n.
struct TreeTile {
  int first, rows;
  int node0, nodes, off;
  int n;
};
template <int KEYS>
__device__ __forceinline__ TreeTile tree_tile(const TreeParams& p, const TreeElement& e, int t) {
  TreeTile k;
  const int cached = (e.len + KEYS - 1) / KEYS;
  k.first = t * KEYS;
  k.rows = t < cached ? min(KEYS, e.len - k.first) : 0;
  k.node0 = k.nodes = k.off = 0;
  if (t >= cached) {
    k.node0 = (t - cached) * KEYS;
    k.nodes = p.has_tree ? min(KEYS, e.live - k.node0) : 0;
  } else if (k.rows < KEYS && tree_fused<KEYS>(p, e.len)) {
    k.off = (k.rows + 7) & ~7;
    k.nodes = e.live;
  }
  k.n = k.nodes > 0 ? k.off + k.nodes : k.rows;
  return k;
}

// Which of the columns c0 .. c0 + 31 of a tile the row of node i sees (`there`:
// the row exists): the cached rows, and the nodes by its visibility words.
__device__ __forceinline__ uint32_t tree_word(const TreeParams& p, int b, const TreeTile& t, int c0, int i, bool there) {
  const int rows = t.rows - c0, left = t.n - c0;
  uint32_t w = rows >= 32 ? 0xffffffffu : rows > 0 ? (1u << rows) - 1u : 0u;
  if (t.nodes == 0 || left <= 0 || !there) return w;
  const int s = t.node0 + c0 - t.off;            // node of column c0 (below 0: the gap and the rows before it)
  if (s <= -32) return w;
  uint32_t v;
  if (p.mask != nullptr) {
    const uint32_t* row = p.mask + (static_cast<size_t>(b) * p.T + i) * p.words;
    const int k = s >> 5;
    const uint32_t lo = k >= 0 ? __ldg(row + k) : 0u, hi = k + 1 < p.words ? __ldg(row + k + 1) : 0u;
    v = __funnelshift_r(lo, hi, s & 31);
  } else {                                       // a chain: nodes 0 .. i
    v = i < s ? 0u : i - s >= 31 ? 0xffffffffu : (2u << (i - s)) - 1u;
    if (s < 0) v &= 0xffffffffu << -s;
  }
  if (left < 32) v &= (1u << left) - 1u;
  return w | v;
}

// Jobs of one unit of an element, and of all its units.
__device__ __forceinline__ int tree_unit_jobs(const TreeParams& p, int tiles, int extra) {
  return tiles == 0 ? 0 : tiles * p.row_tiles + extra * p.items;
}
__device__ __forceinline__ int tree_jobs(const TreeParams& p, const TreeElement& e, int extra) {
  return tree_unit_jobs(p, e.tiles, extra) * p.layers * p.hkv;
}

struct TreeStart {
  int total, share;
  int extra;               // jobs in front of an item's tiles
  int begin, end;          // the CTA's jobs
  int b, base;             // the batch element that holds `begin`, and the jobs before it
  TreeElement e;           // that element
};

// The share of CTA `cta`, by the calling warp (every lane gets it).
template <int KEYS>
__device__ __forceinline__ TreeStart tree_start(const TreeParams& p, int cta, bool record) {
  const int lane = threadIdx.x & 31;
  TreeStart s;
  TreeElement first = {0, 0, 0, 0};
  if (lane < p.batch) first = tree_element<KEYS>(p, lane, record);
  int jobs = tree_jobs(p, first, 0), full = first.tiles > 0;     // tiles; elements with any
  for (int b = lane + 32; b < p.batch; b += 32) {
    const TreeElement e = tree_element<KEYS>(p, b, record);
    jobs += tree_jobs(p, e, 0);
    full += e.tiles > 0;
  }
  jobs = __reduce_add_sync(0xffffffffu, jobs);
  // What starting an item costs (Q, the first loads, the outputs: 4 to 5 us) goes
  // into the line as jobs in front of its tiles, where shares are long enough:
  // otherwise the CTAs whose share falls on many short sequences end last.  With
  // 0, 2, 4 and 6 jobs: 16 ragged sequences of up to 8192 rows, 24 nodes, 73.5,
  // 63.6, 60.2, 60.7 us; narrow kernel, 64 sequences of up to 2048 rows, 8 nodes,
  // 109.8, 82.9, 76.2, 78.3; 24 sequences of up to 1000 rows, 24 nodes, 51.1, 36.5,
  // 35.9, 51.3; two of 6000 rows, 24 nodes, 26.6, 27.6, 27.7, 26.8.  (Below as many
  // jobs a share as an item starts with, the start could fill a share.)
  s.extra = jobs / p.ctas >= kTreeItemJobs ? kTreeItemJobs : 0;
  s.total = jobs;
  if (s.extra > 0) s.total += __reduce_add_sync(0xffffffffu, full) * s.extra * p.items * p.layers * p.hkv;
  // (two jobs at least where items are pairs: no share inside an item is then without a tile)
  s.share = max(p.row_tiles > 1 ? 2 : 1, (s.total + p.ctas - 1) / p.ctas);
  // whole units where that costs few jobs more: no unit is then cut and joined
  const int tiles = __shfl_sync(0xffffffffu, first.tiles, 0), unit = tree_unit_jobs(p, tiles, s.extra);
  bool same = unit > 0;
  for (int b = lane; b < p.batch; b += 32) same = same && (b < 32 ? first : tree_element<KEYS>(p, b, false)).tiles == tiles;
  if (__all_sync(0xffffffffu, same)) {
    const int whole = (s.share + unit - 1) / unit * unit;
    if (whole - s.share <= kJoinJobs) s.share = whole;
  }
  const long long begin = static_cast<long long>(s.share) * cta;
  s.begin = begin < s.total ? static_cast<int>(begin) : s.total;
  s.end = s.begin + min(s.total - s.begin, s.share);
  s.b = 0;
  s.base = 0;
  s.e = {0, 0, 0, 0};
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const int b = b0 + lane;
    TreeElement e = {0, 0, 0, 0};
    if (b0 == 0) e = first; else if (b < p.batch) e = tree_element<KEYS>(p, b, false);
    const int x = tree_jobs(p, e, s.extra);
    int sum = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const int base = s.base + sum - x;                         // jobs before element b
    const uint32_t in = __ballot_sync(0xffffffffu, s.begin >= base && s.begin < base + x);
    if (in != 0) {
      const int at = __ffs(in) - 1;
      s.b = b0 + at;
      s.base = __shfl_sync(0xffffffffu, base, at);
      s.e.seq = __shfl_sync(0xffffffffu, e.seq, at);
      s.e.len = __shfl_sync(0xffffffffu, e.len, at);
      s.e.live = __shfl_sync(0xffffffffu, e.live, at);
      s.e.tiles = __shfl_sync(0xffffffffu, e.tiles, at);
      return s;
    }
    s.base += __shfl_sync(0xffffffffu, sum, 31);
  }
  return s;                                                    // no jobs: begin == end == total
}

// An item as the line holds it: jobs [first, first + jobs), `extra` of them
// before its tiles.
struct TreeItem {
  int unit, row0;          // unit = (b * layers + l) * hkv + h
  bool pair;
  int first, jobs, extra;
};

// The item that holds job x of batch element b, whose jobs begin at base.
template <bool PAIRS>
__device__ __forceinline__ TreeItem tree_item(const TreeParams& p, const TreeElement& e, int b, int base, int x, int extra) {
  TreeItem i;
  const int per = tree_unit_jobs(p, e.tiles, extra);           // jobs of a unit
  const int y = x - base;
  const int lh = y / per;
  const int z = y - lh * per;
  i.unit = b * p.layers * p.hkv + lh;
  i.extra = extra;
  const int jobs = (PAIRS ? 2 : 1) * e.tiles + extra, k = z / jobs;
  i.first = base + lh * per + k * jobs;
  i.pair = PAIRS && 2 * k + 1 < p.row_tiles;
  i.row0 = k * (PAIRS ? 256 : p.tile_rows);
  i.jobs = PAIRS && !i.pair ? e.tiles + extra : jobs;
  return i;
}

// Key tiles [t0, t1) of an item that lie in the jobs [begin, end), and whether
// they are its slot 1 (the item starts behind the share's first job) or 0 of
// the share's two places for partial results.
__device__ __forceinline__ void tree_part(const TreeItem& i, int tiles, int begin, int end, int& t0, int& t1, int& slot) {
  const int last = i.jobs - i.extra;
  const int lo = max(0, max(begin, i.first) - i.first - i.extra), hi = max(0, min(end, i.first + i.jobs) - i.first - i.extra);
  t0 = i.pair ? lo >> 1 : lo;
  t1 = hi == last ? tiles : (i.pair ? hi >> 1 : hi);
  slot = i.first > begin ? 1 : 0;
}

// The shares [from, to] that hold tiles of an item (a border before or, of a
// pair, inside its first tile leaves the share before it without one, and so
// for the last; a share is longer than that part).
__device__ __forceinline__ void tree_spread(const TreeItem& i, int tiles, int share, int& from, int& to) {
  int t0, t1, slot;
  from = i.first / share;
  to = (i.first + i.jobs - 1) / share;
  tree_part(i, tiles, from * share, (from + 1) * share, t0, t1, slot);
  if (t0 == t1) ++from;
  tree_part(i, tiles, to * share, (to + 1) * share, t0, t1, slot);
  if (t0 == t1) --to;
}

struct TreeRun {           // a part of an item that a CTA works on
  int b, unit, row0, t0, t1, slot;
  int pool;                // (layer * n_pages) * hkv + KV head: the unit of page 0 in the pages' maps
  int c0, slot0;           // the share in which the item begins, and its slot there
  int from, to;            // the shares that hold some of its tiles (equal: the run is the whole item)
  bool pair;
  TreeElement e;
  __device__ __forceinline__ int jobs() const { return (t1 - t0) * (pair ? 2 : 1); }
};

template <int KEYS, bool PAIRS>
struct TreeWalker {
  int begin, end, x, b, base, share, extra;
  TreeElement e;
  __device__ __forceinline__ explicit TreeWalker(const TreeStart& s)
      : begin(s.begin), end(s.end), x(s.begin), b(s.b), base(s.base), share(s.share), extra(s.extra), e(s.e) {}
  __device__ __forceinline__ bool next(const TreeParams& p, TreeRun& r) {
    while (x < end) {
      int jobs = tree_jobs(p, e, extra);
      while (x >= base + jobs) {
        base += jobs;
        e = tree_element<KEYS>(p, ++b, false);
        jobs = tree_jobs(p, e, extra);
      }
      const TreeItem i = tree_item<PAIRS>(p, e, b, base, x, extra);
      tree_part(i, e.tiles, begin, end, r.t0, r.t1, r.slot);
      r.b = b;
      r.unit = i.unit;
      r.row0 = i.row0;
      r.pair = i.pair;
      const int lh = i.unit - b * p.layers * p.hkv, layer = lh / p.hkv;
      r.pool = layer * p.n_pages * p.hkv + lh - layer * p.hkv;
      r.e = e;
      x = min(end, i.first + i.jobs);
      if (r.t0 >= r.t1) continue;
      if (r.t0 == 0 && r.t1 == e.tiles) {
        r.c0 = r.slot0 = r.from = r.to = 0;
      } else {
        r.c0 = i.first / share;
        r.slot0 = i.first > r.c0 * share ? 1 : 0;
        tree_spread(i, e.tiles, share, r.from, r.to);
      }
      return true;
    }
    return false;
  }
};

// Whether node i sees node j.
__device__ __forceinline__ bool tree_sees(const TreeParams& p, int b, int i, int j) {
  if (p.mask == nullptr) return j <= i;
  return (__ldg(p.mask + (static_cast<size_t>(b) * p.T + i) * p.words + (j >> 5)) >> (j & 31)) & 1u;
}

// Clears what is not finite among eight 16-bit values; true if there was any.
// (expo: the type's exponent bits.)  A row of V that some query rows see and
// others do not must not reach the others as 0 * NaN, so such values leave the
// product, and the rows that see them get their sum (tree_patch).
__device__ __forceinline__ bool tree_clear_wild(uint4& w, uint32_t expo) {
  uint32_t* const x = reinterpret_cast<uint32_t*>(&w);
  bool any = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if ((x[k] & expo) == expo) {
      x[k] &= 0xffff0000u;
      any = true;
    }
    if ((x[k] >> 16 & expo) == expo) {
      x[k] &= 0xffffu;
      any = true;
    }
  }
  return any;
}

// Whether the V rows of nodes [lo, hi) of a unit hold something that is not
// finite, by a warp.
template <int D>
__device__ __forceinline__ bool tree_wild(const TreeParams& p, int unit, int lo, int hi, uint32_t expo) {
  const uint4* const v = reinterpret_cast<const uint4*>(p.v_tree) + (static_cast<size_t>(unit) * p.T + lo) * (D / 8);
  bool any = false;
#pragma unroll 4
  for (int k = threadIdx.x & 31; k < (hi - lo) * (D / 8); k += 32) {
    uint4 w = __ldg(v + k);
    any |= tree_clear_wild(w, expo);
  }
  return __any_sync(0xffffffffu, any);
}

// The nodes [lo, hi) that lie in key tiles [t0, t1) of an element.
template <int KEYS>
__device__ __forceinline__ void tree_nodes(const TreeParams& p, const TreeElement& e, int t0, int t1, int& lo, int& hi) {
  lo = hi = 0;
  if (!p.has_tree || t1 * KEYS <= e.len) return;
  const int cached = (e.len + KEYS - 1) / KEYS;
  const bool fused = tree_fused<KEYS>(p, e.len);               // all of them lie with the last rows
  lo = fused ? 0 : max(0, t0 - cached) * KEYS;
  hi = fused ? e.live : min(e.live, (t1 - cached) * KEYS);
}

// What is not finite among the V values of nodes [lo, hi) that node i sees, added
// to the row's output (or partial result) of the others: an infinity stays one, a
// NaN of the logits or of another row stays NaN.
// Columns d0, d0 + step, .. below d1; column d lies at
// out[(d / run) * stride + d % run].
template <typename V, typename O>
__device__ __noinline__ void tree_patch(const TreeParams& p, int b, int unit, int i, int lo, int hi, int d0, int d1, int step,
                                        int D, O* out, int run, size_t stride) {
#pragma unroll 1
  for (int d = d0; d < d1; d += step) {
    float sum = 0.f;
#pragma unroll 1
    for (int j = lo; j < hi; ++j) {
      if (!tree_sees(p, b, i, j)) continue;
      const float v = static_cast<float>(static_cast<const V*>(p.v_tree)[(static_cast<size_t>(unit) * p.T + j) * D + d]);
      if (!isfinite(v)) sum += v;
    }
    if (sum != 0.f) {                                          // (true for NaN too)
      O& at = out[(d / run) * stride + d % run];
      at = static_cast<O>(static_cast<float>(at) + sum);
    }
  }
}

// Where the partial results of share c of an item lie.
__device__ __forceinline__ size_t tree_place(const TreeRun& r, int c) {
  return static_cast<size_t>(c) * 2 + (c == r.c0 ? r.slot0 : 0);
}

// Four columns of a row of a cut item, `sum`, from its shares [from, to] again
// where adding them gave NaN: where a share's weight underflows to 0, what is
// finite counts for nothing and what is not stays as it is (0 * inf made NaN of
// it; in an item that one share holds whole it is inf). c0, slot0: see TreeRun.
static __device__ __noinline__ float4 tree_join_again(const TreeParams& p, int from, int to, int c0, int slot0, int row,
                                                      int col4, int cols4, float4 sum) {
  TreeRun r;
  r.c0 = c0;
  r.slot0 = slot0;
  float m = -INFINITY;
#pragma unroll 1
  for (int c = from; c <= to; ++c) m = fmaxf(m, __ldcg(p.part_ml + (tree_place(r, c) * p.item_rows + row) * 2));
  const float ref = m == -INFINITY ? 0.f : m;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int c = from; c <= to; ++c) {
    const size_t at = tree_place(r, c);
    const float f = ex2_approx(__ldcg(p.part_ml + (at * p.item_rows + row) * 2) - ref);
    const float4 o = __ldcg(reinterpret_cast<const float4*>(p.part_o) + (at * cols4 + col4) * p.item_rows + row);
    acc.x += f != 0.f ? o.x * f : isfinite(o.x) ? 0.f : o.x;
    acc.y += f != 0.f ? o.y * f : isfinite(o.y) ? 0.f : o.y;
    acc.z += f != 0.f ? o.z * f : isfinite(o.z) ? 0.f : o.z;
    acc.w += f != 0.f ? o.w * f : isfinite(o.w) ? 0.f : o.w;
  }
  return make_float4(isnan(sum.x) ? acc.x : sum.x, isnan(sum.y) ? acc.y : sum.y, isnan(sum.z) ? acc.z : sum.z,
                     isnan(sum.w) ? acc.w : sum.w);
}

// One more share of a cut item has left its results; true for the last one,
// which joins them.  A word holds the call's number and a count; a word with
// another number counts as 0, so the workspace needs no clearing, and the last
// arrival leaves 0, so that a captured call can be replayed.  Which share is
// the last does not change a result: the shares are added in their order.
__device__ __forceinline__ bool tree_arrive(const TreeParams& p, const TreeRun& r) {
  unsigned long long* const word = p.arrived + r.c0;
  const unsigned long long call = p.call << 16;
  const int parts = r.to - r.from + 1;
  __threadfence();
  unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(word);
  while (true) {
    const unsigned long long count = (old & ~0xffffull) == call ? old & 0xffffull : 0;
    const bool last = static_cast<int>(count) + 1 == parts;
    const unsigned long long seen = atomicCAS(word, old, call | (last ? 0ull : count + 1));
    if (seen == old) {
      __threadfence();
      return last;
    }
    old = seen;
  }
}

}  // namespace spk

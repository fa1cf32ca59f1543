// tree_umma.cu -- tree attention for units of many query rows, on tcgen05.
//
// The same attention, work split and partial results as tree.cu (see there);
// this kernel takes over where a unit has more query rows than a narrow
// mma.sync tile holds.  Tiles are 128 query rows by 128 keys:
//   S = Q K^T   A = Q, B = K from shared memory, S in TMEM (fp32)
//   O += P V    A = P from TMEM (in the element type's 16 bits, as tree_kernel's
//               is, and over the second half of S), B = V from
//               shared memory as it lies ([key][d], MN-major), O in TMEM
// with two softmax groups of four warps (thread = query row), so that one
// group's exponentials run under the other's products.  Rows of a unit are
// taken 256 at a time while there are more than 128 of them (a PAIR: group x
// has query tile x, both use every K/V tile), the rest 128 at a time (ALONE:
// both groups have the query tile, group x the key tiles x, x + 2, ...; their
// states are joined at the end).  A job is one (query tile, key tile) product
// pair; the products go out in the order S0(0), S1(0), PV0(0), S0(1), PV1(0),
// S1(1), ...: when a group's S(i + 1) has landed, its O is quiescent and may be
// rescaled.
//   warps 0-3, 4-7  softmax groups 0, 1
//   warps 8, 9      TMA producers: Q and the K tiles, the V tiles, page by page
//                   through one ring
//   warp 10         TMEM allocation, UMMA issue
//   warp 11         the runs (tree_shares.cuh), ahead of the others, which read
//                   them from shared memory
// TMEM (512 columns): group x's S at 256 x, its O at 256 x + 128.
// The one atomic counts a cut item's shares (tree_arrive); which of them is the
// last does not change a result.
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "exp2_poly.cuh"   // f2, exp2_mufu_pair
#include "mma.cuh"
#include "paged.cuh"
#include "tree_shares.cuh"

namespace spk {

SPK_ERROR_READER(device_errors_tree_umma)

namespace {

constexpr int kKeys = 128;               // keys of a tile
constexpr int kGroupWarps = 4;
constexpr int kProducerWarp = 8;         // K; 9: V
constexpr int kMmaWarp = 10;
constexpr int kRunWarp = 11;
constexpr int kUmmaThreads = 12 * 32;
constexpr int kRunSlots = 4;
constexpr int kRunReaders = 2 * kGroupWarps + 3;
constexpr float kRescaleLog2 = 8.f;      // O and the sum are rescaled when the maximum grew by more (P <= 2^8)

__device__ __forceinline__ int umma_site(int role, int which) { return 620 + role * 10 + which; }

// Bounded wait with little code: the hardware suspends the thread for a while at
// each try; from the 4097th on each is followed by a millisecond by the timer, up
// to the library's limit.  (Items are short, so this kernel's speed hangs on how
// much of its code stays in the instruction cache; mbar_wait, inlined at every
// wait, is several times as long.  16 nodes over 320 rows, 512 KV heads; 24 nodes,
// 16 ragged sequences; 64 nodes over 64K rows: 39.3, 59.4 and 216 us; with the
// timer read in the loop 39.4, 59.7 and 216; with a function that takes the wait
// over 39.4, 60.2 and 222; without a limit in time 38.8, 59.1 and 219.)
constexpr int kShortTries = 4096;
constexpr uint32_t kPauseNs = 1000000;
__device__ __noinline__ void pause() {
  const uint64_t t0 = global_timer_ns();
  while (global_timer_ns() - t0 < kPauseNs) __nanosleep(1000);
}
__device__ __noinline__ bool give_up(volatile int* abort_flag, int site) {
  if (*abort_flag == 0) {
    record_error(SPK_DEVERR_TIMEOUT, site);
    *abort_flag = 1;
  }
  return false;
}
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int site) {
#pragma unroll 1
  for (int tries = 0; tries < kShortTries + static_cast<int>(SPK_WAIT_LIMIT_NS / kPauseNs); ++tries) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (tries >= kShortTries) pause();
  }
  return give_up(abort_flag, site);
}

// Shared memory behind the tiles.  (All of it is dynamic, so that the tiles
// begin at its start, which is 1024-byte aligned.)
template <int SLOTS>
struct UmmaShared {
  uint64_t q_full, q_empty, full[SLOTS], empty[SLOTS], s_full[2], p_half[2], p_full[2], run_done, o_empty, ml_ready,
      parts_in, joined, run_full[kRunSlots], run_empty[kRunSlots], wild_full[kRunSlots];
  TreeRun run[kRunSlots];
  float2 ml[2][128];          // both groups' row states, for the other
  uint32_t tmem_holder;
  int abort_flag, last;
  int arrived;                // cut items of which this CTA's share has been counted (tree_arrive)
  int wild[kRunSlots];        // of each run: whether V of its nodes holds something that is not finite
};

// QT query tiles of a unit share the K/V tiles (1: no unit has more than 128
// rows; its place goes to the ring, whose depth hides the memory's latency).
template <int D, int QT>
struct UmmaCfg {
  static constexpr int kTileBytes = 128 * D * 2;          // 128 rows of Q, K or V
  static constexpr int kAtoms = D / 64;
  static constexpr int kSlots = (QT == 1 ? 6 : 5) * (128 / D);
  static constexpr int kSmemBytes = (QT + kSlots) * kTileBytes + sizeof(UmmaShared<kSlots>);
  static_assert(kSmemBytes <= 227 * 1024, "fits one CTA");
  static_assert(kSlots >= 5, "K(t), V(t), K(t + 1), V(t + 1), K(t + 2) are in use together");
};

// Matrix descriptors (shared memory, 128-byte swizzle): the low word has the
// address and the leading offset, the high word is the same for all of them:
// 8-row atoms 1024 bytes apart, version 1, swizzle 2.
//   K-major (Q, K): leading offset unused (1)
//   MN-major (V as it lies, [key][d]): 64-column blocks 16384 bytes apart
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kKMajorLo = 1u << 16, kMnMajorLo = (16384u >> 4) << 16;

// D[tmem] (+)= A[smem] B[smem]^T; a, b: low descriptor words.
// The whole warp executes these, `leader` alone issues: without a branch, what
// is the same in every lane can stay in uniform registers.
__device__ __forceinline__ void umma_ss(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(kDescHi), "r"(leader)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]^T
__device__ __forceinline__ void umma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(kDescHi), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tma_load_if(uint32_t leader, uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0,
                                            int c1, int c2) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(leader)
      : "memory");
}
// Arrive on `bar` when the products issued so far are done.
__device__ __forceinline__ void commit_if(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(one));
  return one;
}
// A value that is the same in every lane, as one the compiler knows to be.
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

template <typename T>
constexpr uint32_t kFormats = 0;                          // operand formats: f16
template <>
constexpr uint32_t kFormats<__nv_bfloat16> = (1u << 7) | (1u << 10);

template <typename T>
__host__ __device__ constexpr uint32_t idesc_of(int M, int N) {
  return (1u << 4) | kFormats<T> | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 4 x 4 transpose of 16-byte vectors among each group of four lanes.
__device__ __forceinline__ uint4 shfl_xor4(const uint4& v, int o) {
  return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o),
                    __shfl_xor_sync(0xffffffffu, v.z, o), __shfl_xor_sync(0xffffffffu, v.w, o));
}
__device__ __forceinline__ uint4 pick4(bool a, const uint4& x, const uint4& y) {
  return make_uint4(a ? x.x : y.x, a ? x.y : y.y, a ? x.z : y.z, a ? x.w : y.w);
}
__device__ __forceinline__ void transpose4(uint4 (&v)[4], int lane) {
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & o) continue;
      // this lane keeps one of v[i], v[i + o] and swaps the other with lane ^ o
      const uint4 got = shfl_xor4(pick4(up, v[i], v[i + o]), o);
      if (up) v[i] = got; else v[i + o] = got;
    }
  }
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A CTA that gave up counts its shares of the cut items that it did not come to,
// so that the counts end at 0: a replay of the call has its number, and would
// take what is left in the workspace for shares of its own.  (By a warp.)
__device__ __noinline__ void count_the_rest(const TreeParams& p, int arrived) {
  const TreeStart start = tree_start<kKeys>(p, blockIdx.x, false);
  if ((threadIdx.x & 31) != 0) return;
  TreeWalker<kKeys, true> walk(start);
  TreeRun r;
  while (walk.next(p, r))
    if (r.from != r.to && --arrived < 0) tree_arrive(p, r);
}

// --------------------------------------------------------------------------
// LOSES: a self-test of the waits. CTA c (0 or 1) publishes only its first c runs;
// what the others wait for never comes.
template <typename T, int D, int QT, bool LOSES>
__global__ void __launch_bounds__(kUmmaThreads, 1)
    tree_umma_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap ktmap,
                     const __grid_constant__ CUtensorMap vtmap, const __grid_constant__ CUtensorMap k8map,
                     const __grid_constant__ CUtensorMap v8map, const __grid_constant__ TreeParams p) {
  using C = UmmaCfg<D, QT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const Q_s = smem;                                  // [QT tiles]
  uint8_t* const ring = smem + QT * C::kTileBytes;            // K(0), V(0), K(1), V(1), ...
  UmmaShared<C::kSlots>& sh = *reinterpret_cast<UmmaShared<C::kSlots>*>(ring + C::kSlots * C::kTileBytes);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh.s_full[x], 1);
      mbar_init(&sh.p_half[x], kGroupWarps);
      mbar_init(&sh.p_full[x], kGroupWarps);
    }
    mbar_init(&sh.run_done, 1);
    mbar_init(&sh.o_empty, 2 * kGroupWarps);
    mbar_init(&sh.ml_ready, 2 * kGroupWarps);
    mbar_init(&sh.parts_in, 2 * kGroupWarps);
    mbar_init(&sh.joined, 1);
    for (int s = 0; s < kRunSlots; ++s) {
      mbar_init(&sh.run_full[s], 1);
      mbar_init(&sh.run_empty[s], kRunReaders);
      mbar_init(&sh.wild_full[s], 1);
    }
    sh.abort_flag = 0;
    sh.arrived = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem_holder, 512);
    tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_map(&qmap);
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
  }
  TreeStart start{};
  if (warp == kRunWarp) start = tree_start<kKeys>(p, blockIdx.x, blockIdx.x == 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!p.join_inside) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // (all 512 columns: the allocation begins at column 0)
  const uint32_t tmem = 0;
  volatile int* const abort_v = &sh.abort_flag;
  TreeRun run;
  uint32_t taken = 0;
  // the next run; false behind the last one, or when the CTA gives up (ok)
  auto next_run = [&](bool& ok) -> bool {
    const uint32_t s = taken % kRunSlots;
    ok = __all_sync(0xffffffffu, bar_wait(&sh.run_full[s], (taken / kRunSlots) & 1, abort_v, umma_site(5, 0)));
    if (!ok) return false;
    run = sh.run[s];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.run_empty[s]);
    ++taken;
    return run.t0 >= 0;
  };

  if (warp == kRunWarp) {
    // -------------------------------------------------------------------- runs
    // lane 0 finds them; the warp looks whether V of a run's nodes holds something
    // that is not finite, when the next run is out
    TreeWalker<kKeys, true> walk(start);
    int lo = 0, hi = 0, unit = 0;
    bool go = true;
    for (uint32_t k = 0; go; ++k) {
      if (LOSES && blockIdx.x < 2 && k == blockIdx.x) break;
      const uint32_t s = k % kRunSlots;
      const int old_lo = lo, old_hi = hi, old_unit = unit;
      lo = hi = unit = 0;
      if (lane == 0) {
        TreeRun r;
        go = walk.next(p, r);
        if (!go) r.t0 = -1;
        go = bar_wait(&sh.run_empty[s], ((k / kRunSlots) & 1) ^ 1, abort_v, umma_site(5, 1)) && go;
        if (go) {
          tree_nodes<kKeys>(p, r.e, r.t0, r.t1, lo, hi);
          unit = r.unit;
        }
        sh.run[s] = r;
        mbar_arrive(&sh.run_full[s]);
      }
      go = __shfl_sync(0xffffffffu, go, 0);
      lo = __shfl_sync(0xffffffffu, lo, 0);
      hi = __shfl_sync(0xffffffffu, hi, 0);
      unit = __shfl_sync(0xffffffffu, unit, 0);
      if (k == 0) continue;
      const bool wild = old_lo < old_hi && tree_wild<D>(p, old_unit, old_lo, old_hi, Half16<T>::kExponent);
      if (lane == 0) {
        sh.wild[(k - 1) % kRunSlots] = wild;
        mbar_arrive(&sh.wild_full[(k - 1) % kRunSlots]);
      }
    }
  } else if (warp == kProducerWarp || warp == kProducerWarp + 1) {
    // --------------------------------------------------------------- producers
    const uint32_t leader = elect_one();
    const int v = uniform(warp - kProducerWarp);               // 0: K (and Q), 1: V
    const CUtensorMap* const pages = v ? &vmap : &kmap;
    const CUtensorMap* const pages8 = v ? &v8map : &k8map;     // in parts of 8 rows, for a tile that ends early
    const CUtensorMap* const nodes = v ? &vtmap : &ktmap;
    uint32_t seq = v;              // K and V tiles in their order: slot seq % kSlots
    int runs = 0, q_last = -1;
    bool ok = true;
    const int per_tile = kKeys / p.box_rows;                   // parts of a full tile
    while (ok && next_run(ok)) {
      if (v == 0) {
        ok = __all_sync(0xffffffffu, bar_wait(&sh.q_empty, (runs & 1) ^ 1, abort_v, umma_site(0, 0)));
        if (!ok) break;
        if (lane == 0) {
          const int tiles = run.pair ? 2 : 1;
          mbar_arrive_expect_tx(&sh.q_full, tiles * C::kTileBytes);
#pragma unroll 1
          for (int x = 0; x < tiles; ++x)
#pragma unroll
            for (int a = 0; a < C::kAtoms; ++a)
              tma_load_3d(Q_s + x * C::kTileBytes + a * 16384, &qmap, &sh.q_full, a * 64, run.row0 + x * 128, run.unit);
        }
        q_last = runs & 1;
      }
      const int full = run.e.len / kKeys;
      // lane i has the place of part `at` + i of the sequence's full tiles (its page's
      // unit in the pages' map, the row in the page): the page table is read for 32
      // parts at a time
      int at = -64, unit = 0, row = 0;
#pragma unroll 1
      for (int t = run.t0; t < run.t1; ++t) {
        int parts = per_tile, more = 0, from = t * per_tile;
        TreeTile tile;
        tile.nodes = 0;
        const bool last = t >= full;                           // the last rows, or nodes: see tree_tile
        if (last) {
          tile = tree_tile<kKeys>(p, run.e, t);
          parts = tile.rows / p.box_rows;                      // then the rest in parts of 8 rows
          more = (tile.rows - parts * p.box_rows + 7) / 8;
        }
        if (last || from + per_tile > at + 32) {
          at = last ? 0 : from;
          const int t_row = !last ? (from + lane) * p.box_rows
                            : lane < parts ? tile.first + lane * p.box_rows
                            : lane < parts + more ? tile.first + parts * p.box_rows + (lane - parts) * 8 : 0x7fffffff;
          unit = row = 0;
          if (t_row < run.e.len) {
            const int pg = t_row / p.page_rows;
            row = t_row - pg * p.page_rows;
            const int page = __ldg(p.table + static_cast<size_t>(run.e.seq) * p.max_pages + pg);
            if (page < 0 || page >= p.n_pages) {
              if (v == 0) record_error(SPK_DEVERR_INDEX, run.b);
              unit = p.layers * p.n_pages * p.hkv;             // outside the map: the part reads as zeros
            } else {
              unit = run.pool + page * p.hkv;
            }
          }
        }
        from = last ? 0 : from - at;
        const int slot = seq % C::kSlots;
        ok = __all_sync(0xffffffffu, bar_wait(&sh.empty[slot], ((seq / C::kSlots) & 1) ^ 1, abort_v, umma_site(0, 1 + v)));
        if (!ok) break;
        uint64_t* const bar = &sh.full[slot];
        uint8_t* const dst = ring + slot * C::kTileBytes;
        const int bytes = (parts * p.box_rows + more * 8 + (tile.nodes > 0 ? p.node_rows : 0)) * 128 * C::kAtoms;
        if (leader) {
          if (bytes == 0)
            mbar_arrive(bar);
          else
            mbar_arrive_expect_tx(bar, bytes);
        }
        // whole parts, then parts of 8 rows (places from lane 0: of the last rows)
        const uint32_t d0 = smem_u32(dst), b0 = smem_u32(bar);
#pragma unroll 1
        for (int k = 0; k < parts; ++k) {
          const int u = uniform(lane == from + k ? unit : -1), f = uniform(lane == from + k ? row : -1);
#pragma unroll
          for (int a = 0; a < C::kAtoms; ++a)
            tma_load_if(leader, d0 + a * 16384 + k * p.box_rows * 128, pages, b0, a * 64, f, u);
        }
        if (last) {
#pragma unroll 1
          for (int k = parts; k < parts + more; ++k) {
            const int u = uniform(lane == k ? unit : -1), f = uniform(lane == k ? row : -1);
#pragma unroll
            for (int a = 0; a < C::kAtoms; ++a)
              tma_load_if(leader, d0 + a * 16384 + (parts * p.box_rows + (k - parts) * 8) * 128, pages8, b0, a * 64, f, u);
          }
          if (tile.nodes > 0) {
#pragma unroll
            for (int a = 0; a < C::kAtoms; ++a)
              tma_load_if(leader, d0 + a * 16384 + tile.off * 128, nodes, b0, a * 64, tile.node0, run.unit);
          }
          at = -64;
        }
        __syncwarp();
        seq += 2;
      }
      ++runs;
    }
    if (!ok && lane == 0) {        // let the copies in flight land before the block ends
      volatile int never = 0;
      if (q_last >= 0) mbar_wait(&sh.q_full, q_last, &never, umma_site(0, 7), 100000000ull);
      for (uint32_t s = seq > 2 * C::kSlots ? seq - 2 * C::kSlots : v; s < seq; s += 2)
        if (s + C::kSlots >= seq) mbar_wait(&sh.full[s % C::kSlots], (s / C::kSlots) & 1, &never, umma_site(0, 8), 100000000ull);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------- UMMA issuer
    // The whole warp goes through the jobs, so that what an instruction needs is
    // the same in every lane and stays in uniform registers; one lane issues.
    // (With one lane in the branch each product took 85 clocks to issue, more
    // than its 64 to run.)
    const uint32_t leader = elect_one();
    bool ok = true;
    int runs = 0;
    constexpr uint32_t idesc_s = idesc_of<T>(128, 128);
    constexpr uint32_t idesc_pv = idesc_of<T>(128, D) | (1u << 16);       // B (V) MN-major
    const uint32_t q_lo = smem_u32(Q_s) >> 4, ring_lo = smem_u32(ring) >> 4;
    // the slots of the next K and V tile, with the parity of their barriers
    int ks = 0, vs = 1;
    uint32_t kph = 0, vph = 0, pph = 0;                        // pph: bit x = parity of group x's P
    auto advance = [](int& slot, uint32_t& ph) {
      slot += 2;
      if (slot >= C::kSlots) {
        slot -= C::kSlots;
        ph ^= 1u;
      }
    };
    auto wait = [&](uint64_t* bar, uint32_t parity, int which) -> bool {
      return __all_sync(0xffffffffu, bar_wait(bar, parity, abort_v, umma_site(1, which)));
    };
    // S of group x = its Q tile times the next K tile
    auto issue_s = [&](auto X, bool pair) -> bool {
      constexpr int x = decltype(X)::value;
      if (!(pair && x == 1) && !wait(&sh.full[ks], kph, 1)) return false;
      tc_fence_after();
      const uint32_t qa = QT == 2 && x == 1 && pair ? q_lo + (C::kTileBytes >> 4) : q_lo;
      const uint32_t ka = ring_lo + ks * (C::kTileBytes >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
        umma_ss(leader, x * 256, (qa + off) | kKMajorLo, (ka + off) | kKMajorLo, idesc_s, kk > 0);
      }
      commit_if(leader, &sh.s_full[x]);
      if (!pair || x == 1) {                                   // the K tile's last use
        commit_if(leader, &sh.empty[ks]);
        advance(ks, kph);
      }
      return true;
    };
    // O of group x += P V(next tile, of n keys), in two halves: keys 64 .. 127 as
    // soon as the softmax has stored their P, then keys 0 .. 63; only the k-steps
    // that hold a key
    auto issue_pv = [&](auto X, bool pair, int n, bool fresh) -> bool {
      constexpr int x = decltype(X)::value;
      const uint32_t ph = (pph >> x) & 1u;
      pph ^= 1u << x;
      const uint32_t va = ring_lo + vs * (C::kTileBytes >> 4);
      if (!(pair && x == 1) && !wait(&sh.full[vs], vph, 6)) return false;
      // the previous run's O has been read before O is restarted
      if (fresh && x == 0 && runs > 0 && !wait(&sh.o_empty, (runs - 1) & 1, 7)) return false;
      if (n > 64) {
        if (!wait(&sh.p_half[x], ph, 2 + x)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 4; kk < 8; ++kk)
          umma_ts(kk * 16 < n ? leader : 0u, x * 256 + 128, x * 256 + 64 + kk * 8, (va + kk * (2048 >> 4)) | kMnMajorLo,
                  idesc_pv, kk > 4 || !fresh);
      }
      if (!wait(&sh.p_full[x], ph, 4 + x)) return false;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        umma_ts(kk * 16 < n ? leader : 0u, x * 256 + 128, x * 256 + 64 + kk * 8, (va + kk * (2048 >> 4)) | kMnMajorLo,
                idesc_pv, kk > 0 || n > 64 || !fresh);
      if (!pair || x == 1) {
        commit_if(leader, &sh.empty[vs]);
        advance(vs, vph);
      }
      return true;
    };
    constexpr std::integral_constant<int, 0> G0{};
    constexpr std::integral_constant<int, 1> G1{};
    while (ok && next_run(ok)) {
      const bool pair = QT == 2 && __any_sync(0xffffffffu, run.pair);
      const int tiles = uniform(run.t1 - run.t0), full = uniform(run.e.len / kKeys - run.t0);   // tiles before it have kKeys keys
      const int j0 = pair ? tiles : (tiles + 1) / 2, j1 = pair ? tiles : tiles / 2;
      auto keys_of = [&](int t) { return t < full ? kKeys : uniform(tree_tile<kKeys>(p, run.e, run.t0 + t).n); };
      if (!(ok = wait(&sh.q_full, runs & 1, 0))) break;
      // S(i + 1) goes out behind PV(i)
#pragma unroll 1
      for (int i = -1; ok && i < j0; ++i) {
        if (i >= 0) ok = issue_pv(G0, pair, keys_of(pair ? i : 2 * i), i == 0);
        if (ok && i + 1 < j0) ok = issue_s(G0, pair);
        if (ok && i >= 0 && i < j1) ok = issue_pv(G1, pair, keys_of(pair ? i : 2 * i + 1), i == 0);
        if (ok && i + 1 < j1) ok = issue_s(G1, pair);
        if (i + 2 == j0) commit_if(leader, &sh.q_empty);                       // the last S is out
      }
      if (!ok) break;
      commit_if(leader, &sh.run_done);
      ++runs;
    }
    if (!ok && leader) {             // the products in flight end before the block does
      umma_commit(&sh.run_done);
      volatile int never = 0;
      mbar_wait(&sh.run_done, runs & 1, &never, umma_site(1, 9), 100000000ull);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- softmax groups
    const int x = warp >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;                              // TMEM lane = row of the query tile
    const uint32_t lanes = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t mine = lanes + x * 256;                     // S; O at + 128
    bool ok = true;
    uint32_t job = 0, base = 0;                                // jobs of this group, K/V tiles, before the run
    int runs = 0, alone_runs = 0, cut_runs = 0;
    auto wait_all = [&](uint64_t* bar, uint32_t parity, int which) -> bool {
      return __all_sync(0xffffffffu, bar_wait(bar, parity, abort_v, umma_site(2 + x, which)));
    };
    // (the run stays in shared memory until its end: its fields would cost 16 registers)
    for (;; ++taken) {
      const TreeRun& run = sh.run[taken % kRunSlots];
      if (!(ok = wait_all(&sh.run_full[taken % kRunSlots], (taken / kRunSlots) & 1, 7))) break;
      if (run.t0 < 0) break;
      const bool pair = QT == 2 && run.pair, alone = !pair;
      const int tiles = run.t1 - run.t0, jobs = pair ? tiles : (tiles + 1 - x) / 2;
      const int row = run.row0 + (pair ? x * 128 : 0) + r;      // row of the unit
      const bool there = row < p.rows;
      const bool idle = row - lane >= p.rows;                  // no row of this warp's exists
      const int node = there ? row % p.T : 0;
      float m = -INFINITY, l = 0.f;                            // running maximum of c2 s, sum
      const uint32_t wild_slot = taken % kRunSlots, wild_parity = (taken / kRunSlots) & 1;
      bool wild = false;                                       // V of the run's nodes holds something that is not finite
      for (int i = 0; i < jobs; ++i, ++job) {
        const TreeTile tile = tree_tile<kKeys>(p, run.e, run.t0 + (pair ? i : 2 * i + x));
        const bool full_tile = tile.rows == kKeys;
        // before S is there: which keys this row sees, as words of 32 columns
        uint32_t w0 = 0, w1 = 0, w2 = 0, w3 = 0;
        if (!full_tile) {
          w0 = tree_word(p, run.b, tile, 0, node, there);
          w1 = tree_word(p, run.b, tile, 32, node, there);
          w2 = tree_word(p, run.b, tile, 64, node, there);
          w3 = tree_word(p, run.b, tile, 96, node, there);
        }
        if (!(ok = wait_all(&sh.s_full[x], job & 1, 0))) break;
        tc_fence_after();
        if (!full_tile) {
          // Zeros in V's rows without a key, up to the end of the last k-step: whatever
          // the slot holds there (it may be NaN) must not meet the zeros of P. Not before
          // S of this tile: only then have the products of the slot's last V retired, and
          // only then does the barrier's parity tell this V from that one.
          const int end = (tile.n + 15) & ~15, gap = tile.nodes > 0 ? tile.off - tile.rows : 0, bad = gap + end - tile.n;
          bool clear = false;
          if (tile.nodes > 0) {
            if (!(ok = wait_all(&sh.wild_full[wild_slot], wild_parity, 6))) break;
            clear = sh.wild[wild_slot] != 0;
            wild = wild || clear;
          }
          if ((bad > 0 || clear) && !(pair && x == 1)) {       // (a pair's group 1 comes behind group 0's products)
            const uint32_t seq = 2 * (base + (pair ? i : 2 * i + x)) + 1;
            const int slot = seq % C::kSlots;
            if (!(ok = wait_all(&sh.full[slot], (seq / C::kSlots) & 1, 1))) break;
            for (int k = r; k < bad * (D / 8); k += 128) {
              const int b = k / (D / 8), ch = k % (D / 8);
              const int vr = b < gap ? tile.rows + b : tile.n + b - gap;
              *reinterpret_cast<uint4*>(ring + slot * C::kTileBytes + (ch >> 3) * 16384 + vr * 128 +
                                        (((ch & 7) ^ (vr & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
            // and in the nodes' rows what is not finite, if there is any: not every row sees them
            for (int k = r; k < (clear ? tile.nodes * (D / 8) : 0); k += 128) {
              const int vr = tile.off + k / (D / 8), ch = k % (D / 8);
              uint4* const at = reinterpret_cast<uint4*>(ring + slot * C::kTileBytes + (ch >> 3) * 16384 + vr * 128 +
                                                         (((ch & 7) ^ (vr & 7)) << 4));
              uint4 w = *at;
              if (tree_clear_wild(w, Half16<T>::kExponent)) *at = w;
            }
            fence_proxy_async_smem();
          }
        }
        auto rescale = [&](float mt) {
          const bool need = mt > m + kRescaleLog2;             // the first key of a row: m = -inf
          if (__any_sync(0xffffffffu, need)) {
            const float alpha = need ? ex2_approx(m - mt) : 1.f;
            if (i > 0) {                                       // O holds this run's products
#pragma unroll 1
              for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t o[32];
                tmem_ld32(mine + 128 + ch * 32, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                tmem_st32(mine + 128 + ch * 32, o);
              }
              tmem_st_wait();
            }
            if (need) {
              l *= alpha;
              m = mt;
            }
          }
        };
        auto max32 = [&](const uint32_t (&a)[32], float mx) {
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            mx = fmaxf(mx, max3f(__uint_as_float(a[k]), __uint_as_float(a[k + 1]),
                                 fmaxf(__uint_as_float(a[k + 2]), __uint_as_float(a[k + 3]))));
          return mx;
        };
        // The row's maximum, then P = 2^(c2 s - m) in 16 bits over the second half of S.
        float2 acc = f2(0.f, 0.f);
        auto exp32 = [&](const uint32_t (&a)[32], float2 nm, int c) {
          const float2 c2v = f2(p.c2, p.c2);
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 e = exp2_mufu_pair(__ffma2_rn(f2(__uint_as_float(a[2 * k]), __uint_as_float(a[2 * k + 1])), c2v, nm));
            acc = __fadd2_rn(acc, e);
            pk[k] = Half16<T>::pack(e.x, e.y);
          }
          tmem_st16(mine + 64 + c * 16, pk);
        };
        auto half_done = [&]() {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_half[x]);
        };
        if (idle) {
          // (rows of a product depend on their own row of P only: nothing to store)
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_half[x]);
        } else if (full_tile) {
          // columns 64 .. 127 stay in registers, 0 .. 63 are read twice, the second
          // time under the exponentials of the others
          uint32_t a[32], b[32], c[32], d[32];
          tmem_ld32(mine, a);
          tmem_ld32(mine + 32, b);
          tmem_ld_wait2(a, b);
          tmem_ld32(mine + 64, c);
          tmem_ld32(mine + 96, d);
          const float mx = max32(b, max32(a, -INFINITY));
          tmem_ld_wait2(c, d);
          rescale(max32(d, max32(c, mx)) * p.c2);
          const float ref = m == -INFINITY ? 0.f : m;          // (every logit so far -inf: the weights are 2^-inf = 0)
          const float2 nm = f2(-ref, -ref);
          tmem_ld32(mine + 32, b);
          exp32(d, nm, 3);
          exp32(c, nm, 2);
          tmem_ld_wait(b);                                     // (read before P of columns 64 .. 127 is used)
          half_done();
          tmem_ld32(mine, a);
          exp32(b, nm, 1);
          tmem_ld_wait(a);
          exp32(a, nm, 0);
        } else {
          // what a row does not see becomes -inf
          const int chunks = (tile.n + 31) / 32;               // of 32 columns that hold a key
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            const uint32_t w = c == 0 ? w0 : c == 1 ? w1 : c == 2 ? w2 : w3;
            uint32_t a[32];
            tmem_ld32(mine + c * 32, a);
            tmem_ld_wait(a);
#pragma unroll
            for (int k = 0; k < 32; ++k) a[k] = (w >> k) & 1u ? a[k] : __float_as_uint(-INFINITY);
            tmem_st32(mine + c * 32, a);
            mx = max32(a, mx);
          }
          tmem_st_wait();
          rescale(mx * p.c2);
          const float ref = m == -INFINITY ? 0.f : m;          // no key yet: every weight is 2^-inf = 0
          // from the last chunk down: P of chunk c lies over S of chunk c / 2 + 2
#pragma unroll 1
          for (int c = chunks - 1; c >= 0; --c) {
            uint32_t a[32];
            tmem_ld32(mine + c * 32, a);
            tmem_ld_wait(a);
            exp32(a, f2(-ref, -ref), c);
            if (c == 2) half_done();                           // keys 64 .. 127 are in
          }
          if (chunks < 3) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_half[x]);
          }
        }
        l += acc.x + acc.y;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[x]);
      }
      if (!ok) break;
      // ---- the run's outputs; ALONE: of both groups' states together, half the columns each
      if (!(ok = wait_all(&sh.run_done, runs & 1, 2))) break;
      tc_fence_after();
      float f0 = 1.f, f1 = 0.f;                                // weights of O_0 and O_1 (ALONE)
      if (alone) {
        // (the other group read the previous run's states before run_done of this one)
        sh.ml[x][r] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.ml_ready);
        if (!(ok = wait_all(&sh.ml_ready, alone_runs & 1, 3))) break;
        ++alone_runs;
        const float2 s0 = sh.ml[0][r], s1 = sh.ml[1][r];
        const float M = fmaxf(s0.x, s1.x), ref = M == -INFINITY ? 0.f : M;
        f0 = ex2_approx(s0.x - ref);
        f1 = ex2_approx(s1.x - ref);
        l = s0.y * f0 + s1.y * f1;
        m = M;
      }
      const bool whole = run.from == run.to;
      const bool live = there && node < run.e.live;
      const float scale = whole ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;
      f0 *= scale;
      f1 *= scale;
      const bool any = l != 0.f;                               // a row without keys: zeros, whatever O holds
      const bool both = alone && tiles > 1;                 // group 1 had a job
      const uint32_t o_at = (alone ? lanes : mine) + 128;
      const size_t place = static_cast<size_t>(blockIdx.x) * 2 + run.slot;
      const int part_row = (pair ? x * 128 : 0) + r;
      const int c_end = alone ? (x + 1) * (D / 2) : D;
      const uint32_t lives = __ballot_sync(0xffffffffu, live);
      if (alone && p.has_tree && run.t1 * kKeys > run.e.len) { // (the nodes may have been the other group's)
        if (!(ok = wait_all(&sh.wild_full[wild_slot], wild_parity, 6))) break;
        wild = sh.wild[wild_slot] != 0;
      }
      // 32 columns of the rows, 8 (16 bytes) to a vector: four lanes exchange vectors
      // so that each store covers 64 bytes of eight rows
      auto store32 = [&](const uint32_t (&o)[32], int c) {
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k].x = Half16<T>::pack(__uint_as_float(o[8 * k + 0]), __uint_as_float(o[8 * k + 1]));
          v[k].y = Half16<T>::pack(__uint_as_float(o[8 * k + 2]), __uint_as_float(o[8 * k + 3]));
          v[k].z = Half16<T>::pack(__uint_as_float(o[8 * k + 4]), __uint_as_float(o[8 * k + 5]));
          v[k].w = Half16<T>::pack(__uint_as_float(o[8 * k + 6]), __uint_as_float(o[8 * k + 7]));
        }
        transpose4(v, lane);
        T* const dst = static_cast<T*>(p.out) + (static_cast<size_t>(run.unit) * p.rows + row - (lane & 3)) * D + c + (lane & 3) * 8;
#pragma unroll
        for (int k = 0; k < 4; ++k)                            // of row (lane & ~3) + k
          if ((lives >> ((lane & ~3) + k)) & 1u) *reinterpret_cast<uint4*>(dst + k * D) = v[k];
      };
      if (lives != 0) {
#pragma unroll 1
        for (int c = alone ? x * (D / 2) : 0; c < c_end; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_at + c, o);
          if (both) {
            uint32_t o1[32];
            tmem_ld32(lanes + 256 + 128 + c, o1);
            tmem_ld_wait2(o, o1);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(fmaf(__uint_as_float(o1[k]), f1, __uint_as_float(o[k]) * f0));
          } else {
            tmem_ld_wait(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f0);
          }
          if (!any) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          if (whole) {
            store32(o, c);
          } else if (live) {
            // partial results lie [4 columns][row]: a store covers 32 rows together
            float4* const dst = reinterpret_cast<float4*>(p.part_o) + (place * (D / 4) + c / 4) * p.item_rows + part_row;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k * p.item_rows] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                                 __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
          }
        }
      }
      if (wild) {
        __syncwarp();                                          // (the row's outputs are other lanes' stores)
        const int d0 = alone ? x * (D / 2) : 0;
        int lo, hi;
        tree_nodes<kKeys>(p, run.e, run.t0, run.t1, lo, hi);
        if (live && whole)
          tree_patch<T>(p, run.b, run.unit, node, lo, hi, d0, c_end, 1, D,
                        static_cast<T*>(p.out) + (static_cast<size_t>(run.unit) * p.rows + row) * D, D, size_t(0));
        else if (live)
          tree_patch<T>(p, run.b, run.unit, node, lo, hi, d0, c_end, 1, D,
                        p.part_o + (place * (D / 4) * p.item_rows + part_row) * 4, 4, static_cast<size_t>(p.item_rows) * 4);
      }
      if (live && (!alone || x == 0)) {
        if (!whole)
          reinterpret_cast<float2*>(p.part_ml)[place * p.item_rows + part_row] = make_float2(m, l);
        else if (p.lse2 != nullptr)
          p.lse2[static_cast<size_t>(run.unit) * p.rows + row] = l == 0.f ? -INFINITY : m + lg2_approx(l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_empty);
      if (!whole && p.join_inside) {
        // The last of the item's shares joins them (the products of the next run go
        // on meanwhile): M = max m_c, out = sum 2^(m_c - M) o_c / sum 2^(m_c - M) l_c
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.parts_in);
        if (threadIdx.x == 0) {
          ok = bar_wait(&sh.parts_in, cut_runs & 1, abort_v, umma_site(2, 4));
          sh.last = ok && tree_arrive(p, run);
          sh.arrived += ok;
          mbar_arrive(&sh.joined);
        }
        __syncwarp();
        if (!(ok = wait_all(&sh.joined, cut_runs & 1, 5))) break;
        ++cut_runs;
        if (sh.last && lives != 0) {
          const float2* const ml = reinterpret_cast<const float2*>(p.part_ml) + part_row;
          float M = -INFINITY, L = 0.f;
          for (int k = run.from; k <= run.to; ++k) M = fmaxf(M, live ? __ldcg(ml + tree_place(run, k) * p.item_rows).x : 0.f);
          const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 1
          for (int c = alone ? x * (D / 2) : 0; c < c_end; c += 32) {
            float a[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) a[k] = 0.f;
            L = 0.f;
#pragma unroll 2
            for (int q = run.from; q <= run.to; ++q) {
              const size_t at = tree_place(run, q);
              float2 s = make_float2(-INFINITY, 0.f);
              float4 o[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (live) {
                s = __ldcg(ml + at * p.item_rows);
                const float4* const src = reinterpret_cast<const float4*>(p.part_o) + (at * (D / 4) + c / 4) * p.item_rows + part_row;
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = __ldcg(src + k * p.item_rows);
              }
              const float f = ex2_approx(s.x - ref);
              L = fmaf(s.y, f, L);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                a[4 * k] = fmaf(o[k].x, f, a[4 * k]);
                a[4 * k + 1] = fmaf(o[k].y, f, a[4 * k + 1]);
                a[4 * k + 2] = fmaf(o[k].z, f, a[4 * k + 2]);
                a[4 * k + 3] = fmaf(o[k].w, f, a[4 * k + 3]);
              }
            }
            const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
            bool again = false;
#pragma unroll
            for (int k = 0; k < 32; ++k) again |= isnan(a[k]);
            if (again && live) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 o = tree_join_again(p, run.from, run.to, run.c0, run.slot0, part_row, c / 4 + k, D / 4,
                                                 make_float4(a[4 * k], a[4 * k + 1], a[4 * k + 2], a[4 * k + 3]));
                a[4 * k] = o.x;
                a[4 * k + 1] = o.y;
                a[4 * k + 2] = o.z;
                a[4 * k + 3] = o.w;
              }
            }
            uint32_t o[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(a[k] * inv);
            store32(o, c);
          }
          if (live && (!alone || x == 0) && p.lse2 != nullptr)
            p.lse2[static_cast<size_t>(run.unit) * p.rows + row] = L == 0.f ? -INFINITY : M + lg2_approx(L);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.run_empty[taken % kRunSlots]);
      base += tiles;
      ++runs;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(sh.tmem_holder, 512);
  }
  if (warp == kRunWarp && p.join_inside && sh.abort_flag != 0) count_the_rest(p, sh.arrived);
}

template <typename T, int D, int QT, bool LOSES>
cudaError_t launch_qt(const CUtensorMap (&maps)[7], const TreeParams& p, cudaStream_t stream) {
  using C = UmmaCfg<D, QT>;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(tree_umma_kernel<T, D, QT, LOSES>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  tree_umma_kernel<T, D, QT, LOSES><<<p.ctas, kUmmaThreads, C::kSmemBytes, stream>>>(maps[4], maps[0], maps[1], maps[2],
                                                                                    maps[3], maps[5], maps[6], p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_d(const CUtensorMap (&maps)[7], const TreeParams& p, cudaStream_t stream) {
  return p.rows > 128 ? launch_qt<T, D, 2, false>(maps, p, stream) : launch_qt<T, D, 1, false>(maps, p, stream);
}

}  // namespace

cudaError_t launch_tree_umma(bool fp16, int head_dim, const CUtensorMap (&maps)[7], const TreeParams& p,
                             cudaStream_t stream) {
  if (head_dim == 128) return fp16 ? launch_d<__half, 128>(maps, p, stream) : launch_d<__nv_bfloat16, 128>(maps, p, stream);
  if (head_dim == 64) return fp16 ? launch_d<__half, 64>(maps, p, stream) : launch_d<__nv_bfloat16, 64>(maps, p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_tree_umma_loses(const CUtensorMap (&maps)[7], const TreeParams& p, cudaStream_t stream) {
  return launch_qt<__nv_bfloat16, 64, 1, true>(maps, p, stream);
}

}  // namespace spk

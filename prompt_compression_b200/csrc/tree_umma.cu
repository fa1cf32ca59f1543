// tree_umma.cu -- tree attention for units of many query rows, on tcgen05.
//
// The same attention, work split and partial results as tree.cu (see there);
// this kernel takes over where a unit has more query rows than a narrow
// mma.sync tile holds.  Tiles are 128 query rows by 128 keys:
//   S = Q K^T   A = Q, B = K from shared memory, S in TMEM (fp32)
//   O += P V    A = P from TMEM (16-bit, over the second half of S), B = V from
//               shared memory as it lies ([key][d], MN-major), O in TMEM
// with two softmax groups of four warps (thread = query row), so that one
// group's exponentials run under the other's products.  Rows of a unit are
// taken 256 at a time while there are more than 128 of them (a PAIR: group x
// has the query tile x, both use every K/V tile), the rest 128 at a time
// (ALONE: both groups have the same query tile, group x the key tiles t = x
// mod 2, and their states are joined at the end).  A job is one (query tile,
// key tile) product pair; job j belongs to group j mod 2, and the products are
// issued in the order S(0), S(1), PV(0), S(2), PV(1), S(3), ...: when S(j + 2)
// has landed, O of its group is quiescent and may be rescaled.
//   warps 0-3, 4-7  softmax groups 0, 1
//   warps 8, 9      TMA producers: Q and the K tiles, the V tiles, page by page
//                   through one ring
//   warp 10         TMEM allocation, UMMA issue
//   warp 11         the runs (tree_shares.cuh), ahead of the others, which read
//                   them from shared memory
// TMEM (512 columns): group x's S at 256 x, its O at 256 x + 128.
// No atomics: the result is deterministic.
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

// Bounded wait with little code: the hardware suspends the thread for up to a
// microsecond a try.  (Items are short, so this kernel's speed hangs on how
// much of its code stays in the instruction cache; mbar_wait, inlined at every
// wait, is several times as long.)
__device__ __noinline__ bool give_up(volatile int* abort_flag, int site) {
  if (*abort_flag == 0) {
    record_error(SPK_DEVERR_TIMEOUT, site);
    *abort_flag = 1;
  }
  return false;
}
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int site) {
  uint32_t ok = 0;
#pragma unroll 1
  for (int tries = 0; tries < 2000000; ++tries) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
  }
  return give_up(abort_flag, site);
}

// Shared memory behind the tiles.  (All of it is dynamic, so that the tiles
// begin at its start, which is 1024-byte aligned.)
template <int SLOTS>
struct UmmaShared {
  uint64_t q_full, q_empty, full[SLOTS], empty[SLOTS], s_full[2], p_half[2], p_full[2], run_done, o_empty, ml_ready,
      run_full[kRunSlots], run_empty[kRunSlots];
  TreeRun run[kRunSlots];
  float2 ml[2][128];          // both groups' row states, for the other
  uint32_t tmem_holder;
  int abort_flag;
};

// QT query tiles of a unit share the K/V tiles (1: no unit has more than 128 rows).
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
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(kDescHi)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]^T
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(one));
  return one != 0;
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

// --------------------------------------------------------------------------
template <typename T, int D, int QT>
__global__ void __launch_bounds__(kUmmaThreads, 1)
    tree_umma_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap ktmap,
                     const __grid_constant__ CUtensorMap vtmap, const __grid_constant__ TreeParams p) {
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
    for (int s = 0; s < kRunSlots; ++s) {
      mbar_init(&sh.run_full[s], 1);
      mbar_init(&sh.run_empty[s], kRunReaders);
    }
    sh.abort_flag = 0;
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // (all 512 columns: the allocation begins at column 0)
  const uint32_t tmem = 0;
  volatile int* const abort_v = &sh.abort_flag;
  TreeRun run;
  uint32_t taken = 0;
  // the next run; false behind the last one (or when the CTA gives up: ok)
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
    if (lane == 0) {
      TreeWalker<kKeys, true> walk(start);
      for (uint32_t k = 0;; ++k) {
        const uint32_t s = k % kRunSlots;
        TreeRun r;
        const bool more = walk.next(p, r);
        if (!more) r.t0 = -1;
        if (!bar_wait(&sh.run_empty[s], ((k / kRunSlots) & 1) ^ 1, abort_v, umma_site(5, 1))) break;
        sh.run[s] = r;
        mbar_arrive(&sh.run_full[s]);
        if (!more) break;
      }
    }
  } else if (warp == kProducerWarp || warp == kProducerWarp + 1) {
    // --------------------------------------------------------------- producers
    const int v = warp - kProducerWarp;                        // 0: K (and Q), 1: V
    const CUtensorMap* const pages = v ? &vmap : &kmap;
    const CUtensorMap* const nodes = v ? &vtmap : &ktmap;
    uint32_t seq = v;              // K and V tiles in their order: slot seq % kSlots
    int runs = 0, q_last = -1;
    bool ok = true;
    while (ok && next_run(ok)) {
      const int* const table = p.table + static_cast<size_t>(run.e.seq) * p.max_pages;
      const int lh = run.unit - run.b * p.layers * p.hkv;
      const int layer = lh / p.hkv, head = lh - layer * p.hkv;
      if (v == 0) {
        ok = __all_sync(0xffffffffu, bar_wait(&sh.q_empty, (runs & 1) ^ 1, abort_v, umma_site(0, 0)));
        if (!ok) break;
        if (lane == 0) {
          const int tiles = run.pair ? 2 : 1;
          mbar_arrive_expect_tx(&sh.q_full, tiles * C::kTileBytes);
          for (int x = 0; x < tiles; ++x)
            for (int a = 0; a < C::kAtoms; ++a)
              tma_load_3d(Q_s + x * C::kTileBytes + a * 16384, &qmap, &sh.q_full, a * 64, run.row0 + x * 128, run.unit);
        }
        q_last = runs & 1;
      }
      for (int t = run.t0; t < run.t1; ++t) {
        const TreeTile tile = tree_tile<kKeys>(p, run.e, t);
        // lane i: where part i of the tile is
        const int boxes = tile.cached ? (tile.n + p.box_rows - 1) / p.box_rows : tile.n > 0 ? 1 : 0;
        int unit = run.unit, first = tile.first;
        if (tile.cached && lane < boxes) {
          const int t_row = tile.first + lane * p.box_rows;
          const int at = t_row / p.page_rows;
          first = t_row - at * p.page_rows;
          const int page = __ldg(table + at);
          if (page < 0 || page >= p.n_pages) {
            if (v == 0) record_error(SPK_DEVERR_INDEX, run.b);
            unit = p.layers * p.n_pages * p.hkv;             // outside the map: the box reads as zeros
          } else {
            unit = (layer * p.n_pages + page) * p.hkv + head;
          }
        }
        const int slot = seq % C::kSlots;
        ok = __all_sync(0xffffffffu, bar_wait(&sh.empty[slot], ((seq / C::kSlots) & 1) ^ 1, abort_v, umma_site(0, 1 + v)));
        if (!ok) break;
        if (lane == 0) {
          if (boxes == 0)
            mbar_arrive(&sh.full[slot]);
          else
            mbar_arrive_expect_tx(&sh.full[slot], tile.cached ? boxes * p.box_rows * 128 * C::kAtoms : C::kTileBytes);
        }
        const CUtensorMap* const map = tile.cached ? pages : nodes;
        uint8_t* const dst = ring + slot * C::kTileBytes;
        for (int i = 0; i < boxes; ++i) {                      // lane 0 copies part after part
          const int u = __shfl_sync(0xffffffffu, unit, i), f = __shfl_sync(0xffffffffu, first, i);
          if (lane == 0) {
#pragma unroll
            for (int a = 0; a < C::kAtoms; ++a)
              tma_load_3d(dst + a * 16384 + i * p.box_rows * 128, map, &sh.full[slot], a * 64, f, u);
          }
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
    const bool leader = elect_one();
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
      const bool last = !pair || x == 1;                       // of this K tile
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          umma_ss(x * 256, (qa + off) | kKMajorLo, (ka + off) | kKMajorLo, idesc_s, kk > 0);
        }
        umma_commit(&sh.s_full[x]);
        if (last) umma_commit(&sh.empty[ks]);
      }
      __syncwarp();
      if (last) advance(ks, kph);
      return true;
    };
    // O of group x += P V(next tile, of n keys), in two halves: keys 64 .. 127 as
    // soon as the softmax has stored their P, then keys 0 .. 63; only the k-steps
    // that hold a key
    auto issue_pv = [&](auto X, bool pair, int n, bool first, bool fresh) -> bool {
      constexpr int x = decltype(X)::value;
      const uint32_t ph = (pph >> x) & 1u;
      pph ^= 1u << x;
      const uint32_t va = ring_lo + vs * (C::kTileBytes >> 4);
      const bool last = !pair || x == 1;
      if (!(pair && x == 1) && !wait(&sh.full[vs], vph, 6)) return false;
      // the previous run's O has been read before O is restarted
      if (first && runs > 0 && !wait(&sh.o_empty, (runs - 1) & 1, 7)) return false;
      if (!wait(&sh.p_half[x], ph, 2 + x)) return false;
      tc_fence_after();
      if (leader && n > 64) {
#pragma unroll
        for (int kk = 4; kk < 8; ++kk)
          if (kk * 16 < n) umma_ts(x * 256 + 128, x * 256 + 64 + kk * 8, (va + kk * (2048 >> 4)) | kMnMajorLo, idesc_pv, kk > 4 || !fresh);
      }
      __syncwarp();
      if (!wait(&sh.p_full[x], ph, 4 + x)) return false;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (kk * 16 < n) umma_ts(x * 256 + 128, x * 256 + 64 + kk * 8, (va + kk * (2048 >> 4)) | kMnMajorLo, idesc_pv, kk > 0 || n > 64 || !fresh);
        if (last) umma_commit(&sh.empty[vs]);
      }
      __syncwarp();
      if (last) advance(vs, vph);
      return true;
    };
    constexpr std::integral_constant<int, 0> G0{};
    constexpr std::integral_constant<int, 1> G1{};
    while (ok && next_run(ok)) {
      const bool pair = __any_sync(0xffffffffu, run.pair);
      const int jobs = uniform(run.jobs());
      const int full_end = uniform(run.e.len / kKeys) - uniform(run.t0);   // tiles before it hold kKeys keys
      auto keys_of = [&](int t) { return t < full_end ? kKeys : uniform(tree_tile<kKeys>(p, run.e, run.t0 + t).n); };
      if (!(ok = wait(&sh.q_full, runs & 1, 0))) break;
      // S(j + 2) goes out behind PV(j)
      for (int j = -2; ok && j < jobs; j += 2) {
        const int t = pair ? j >> 1 : j;
        if (j >= 0) ok = issue_pv(G0, pair, keys_of(t), j == 0, j == 0);
        if (ok && j + 2 < jobs) ok = issue_s(G0, pair);
        if (ok && j >= 0 && j + 1 < jobs) ok = issue_pv(G1, pair, keys_of(pair ? t : t + 1), false, j == 0);
        if (ok && j + 3 < jobs) ok = issue_s(G1, pair);
        if (leader && j + 2 < jobs && j + 4 >= jobs) umma_commit(&sh.q_empty);    // the last S is out
        __syncwarp();
      }
      if (!ok) break;
      if (leader) umma_commit(&sh.run_done);
      __syncwarp();
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
    int runs = 0, alone_runs = 0;
    auto wait_all = [&](uint64_t* bar, uint32_t parity, int which) -> bool {
      return __all_sync(0xffffffffu, bar_wait(bar, parity, abort_v, umma_site(2 + x, which)));
    };
    while (ok && next_run(ok)) {
      const int row = run.row0 + (run.pair ? x * 128 : 0) + r;  // row of the unit
      const bool there = row < p.rows;
      const int node = there ? row % p.T : 0;
      const int n_jobs = run.jobs();
      float m = -INFINITY, l = 0.f;                            // running maximum of c2 s, sum
      bool fresh = true;                                       // O holds nothing yet
      for (int j = x; ok && j < n_jobs; j += 2, ++job) {
        const int t = run.pair ? j >> 1 : j;
        const TreeTile tile = tree_tile<kKeys>(p, run.e, run.t0 + t);
        const bool full_tile = tile.cached && tile.n == kKeys;
        // before S is there: which keys this row sees, as words of 32 columns ...
        uint32_t w0 = 0, w1 = 0, w2 = 0, w3 = 0;
        if (!full_tile) {
          auto word = [&](int c) -> uint32_t {
            const int left = tile.n - c * 32;
            if (left <= 0) return 0u;
            const uint32_t here = left >= 32 ? 0xffffffffu : (1u << left) - 1u;
            if (tile.cached) return here;
            if (!there) return 0u;
            const int n0 = tile.first + c * 32;
            if (p.mask != nullptr)
              return here & __ldg(p.mask + (static_cast<size_t>(run.b) * p.T + node) * p.words + (n0 >> 5));
            return node < n0 ? 0u : here & (node - n0 >= 31 ? 0xffffffffu : (2u << (node - n0)) - 1u);
          };
          w0 = word(0);
          w1 = word(1);
          w2 = word(2);
          w3 = word(3);
          // ... and zeros in V's rows behind the last key, up to the end of its k-step:
          // whatever the slot holds there (it may be NaN) must not meet the zeros of P
          const int bad = (16 - (tile.n & 15)) & 15;
          if (bad > 0 && !(run.pair && x == 1)) {              // (a pair's group 1 comes behind group 0's products)
            const uint32_t seq = 2 * (base + t) + 1;
            const int slot = seq % C::kSlots;
            if (!(ok = wait_all(&sh.full[slot], (seq / C::kSlots) & 1, 1))) break;
            for (int i = r; i < bad * (D / 8); i += 128) {
              const int vr = tile.n + i / (D / 8), ch = i % (D / 8);
              *reinterpret_cast<uint4*>(ring + slot * C::kTileBytes + (ch >> 3) * 16384 + vr * 128 +
                                        (((ch & 7) ^ (vr & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
        }
        if (!(ok = wait_all(&sh.s_full[x], job & 1, 0))) break;
        tc_fence_after();
        auto rescale = [&](float mt) {
          const bool need = mt > m + kRescaleLog2;             // the first key of a row: m = -inf
          if (__any_sync(0xffffffffu, need)) {
            const float alpha = need ? ex2_approx(m - mt) : 1.f;
            if (!fresh) {
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
        // 32 columns at a time, those that hold a key (loops, not straight code: see
        // bar_wait).  First the row's maximum; what a row does not see becomes -inf
        const int chunks = (tile.n + 31) / 32;
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          uint32_t a[32];
          tmem_ld32(mine + c * 32, a);
          tmem_ld_wait(a);
          if (!full_tile) {
            const uint32_t w = c == 0 ? w0 : c == 1 ? w1 : c == 2 ? w2 : w3;
#pragma unroll
            for (int i = 0; i < 32; ++i) a[i] = (w >> i) & 1u ? a[i] : __float_as_uint(-INFINITY);
            tmem_st32(mine + c * 32, a);
          }
          mx = max32(a, mx);
        }
        if (!full_tile) tmem_st_wait();
        rescale(mx * p.c2);
        // then P = 2^(c2 s - m), from the last chunk down: P of chunk c lies over S of
        // chunk c / 2 + 2
        const float ref = m == -INFINITY ? 0.f : m;            // no key yet: every weight is 2^-inf = 0
        const float2 c2v = f2(p.c2, p.c2), nm = f2(-ref, -ref);
        float2 acc = f2(0.f, 0.f);
#pragma unroll 1
        for (int c = chunks - 1; c >= 0; --c) {
          uint32_t a[32], pk[16];
          tmem_ld32(mine + c * 32, a);
          tmem_ld_wait(a);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e = exp2_mufu_pair(__ffma2_rn(f2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1])), c2v, nm));
            acc = __fadd2_rn(acc, e);
            pk[i] = Half16<T>::pack(e.x, e.y);
          }
          tmem_st16(mine + 64 + c * 16, pk);
          if (c == 2) {                                        // keys 64 .. 127 are in
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_half[x]);
          }
        }
        l += acc.x + acc.y;
        if (chunks < 3) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_half[x]);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[x]);
        fresh = false;
      }
      if (!ok) break;
      // ---- the run's outputs: a pair's groups have a query tile each; ALONE, both
      // groups' states together, half the columns each
      if (!(ok = wait_all(&sh.run_done, runs & 1, 2))) break;
      tc_fence_after();
      float f0 = 1.f, f1 = 0.f;                                // weights of O_0 and O_1 (ALONE)
      if (!run.pair) {
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
      const bool whole = run.t0 == 0 && run.t1 == run.e.tiles;
      const bool live = there && node < run.e.live;
      const float scale = whole ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;
      f0 *= scale;
      f1 *= scale;
      const bool any = l != 0.f;                               // a row without keys: zeros, whatever O holds
      const bool both = !run.pair && n_jobs > 1;               // group 1 had a job
      const uint32_t o_at = (run.pair ? mine : lanes) + 128;
      const size_t part = static_cast<size_t>(blockIdx.x) * 2 + run.slot;
      const int part_row = (run.pair ? x * 128 : 0) + r;
      const int c_end = run.pair ? D : (x + 1) * (D / 2);
      const uint32_t lives = __ballot_sync(0xffffffffu, live);
#pragma unroll 1
      for (int c = run.pair ? 0 : x * (D / 2); c < c_end; c += 32) {
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
          // 32 columns a row, 8 (16 bytes) to a vector: four lanes exchange vectors so
          // that each store covers 64 bytes of eight rows
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i].x = Half16<T>::pack(__uint_as_float(o[8 * i + 0]), __uint_as_float(o[8 * i + 1]));
            v[i].y = Half16<T>::pack(__uint_as_float(o[8 * i + 2]), __uint_as_float(o[8 * i + 3]));
            v[i].z = Half16<T>::pack(__uint_as_float(o[8 * i + 4]), __uint_as_float(o[8 * i + 5]));
            v[i].w = Half16<T>::pack(__uint_as_float(o[8 * i + 6]), __uint_as_float(o[8 * i + 7]));
          }
          transpose4(v, lane);
          T* const dst = static_cast<T*>(p.out) + (static_cast<size_t>(run.unit) * p.rows + row - (lane & 3)) * D + c + (lane & 3) * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i)                          // of row (lane & ~3) + i
            if ((lives >> ((lane & ~3) + i)) & 1u) *reinterpret_cast<uint4*>(dst + i * D) = v[i];
        } else if (live) {
          // partial results lie [4 columns][row]: a store covers 32 rows together
          float4* const dst = reinterpret_cast<float4*>(p.part_o) + (part * (D / 4) + c / 4) * (QT * 128) + part_row;
#pragma unroll
          for (int v = 0; v < 8; ++v)
            dst[v * (QT * 128)] = make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                              __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
        }
      }
      if (live && (run.pair || x == 0)) {
        if (!whole)
          reinterpret_cast<float2*>(p.part_ml)[part * (QT * 128) + part_row] = make_float2(m, l);
        else if (p.lse2 != nullptr)
          p.lse2[static_cast<size_t>(run.unit) * p.rows + row] = l == 0.f ? -INFINITY : m + lg2_approx(l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_empty);
      base += run.t1 - run.t0;
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
}

template <typename T, int D, int QT>
cudaError_t launch_qt(const CUtensorMap (&maps)[5], const TreeParams& p, cudaStream_t stream) {
  using C = UmmaCfg<D, QT>;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(tree_umma_kernel<T, D, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  tree_umma_kernel<T, D, QT><<<p.ctas, kUmmaThreads, C::kSmemBytes, stream>>>(maps[4], maps[0], maps[1], maps[2],
                                                                             maps[3], p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_umma(bool fp16, int head_dim, const CUtensorMap (&maps)[5], const TreeParams& p,
                             cudaStream_t stream) {
  const bool pairs = p.rows > 128;
  if (head_dim == 128) {
    if (fp16) return pairs ? launch_qt<__half, 128, 2>(maps, p, stream) : launch_qt<__half, 128, 1>(maps, p, stream);
    return pairs ? launch_qt<__nv_bfloat16, 128, 2>(maps, p, stream) : launch_qt<__nv_bfloat16, 128, 1>(maps, p, stream);
  }
  if (head_dim == 64) {
    if (fp16) return pairs ? launch_qt<__half, 64, 2>(maps, p, stream) : launch_qt<__half, 64, 1>(maps, p, stream);
    return pairs ? launch_qt<__nv_bfloat16, 64, 2>(maps, p, stream) : launch_qt<__nv_bfloat16, 64, 1>(maps, p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace spk

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
//   warp 8          TMA producer: Q, and K and V tiles through one ring, page
//                   by page (lane i copies the boxes of page part i)
//   warp 9          TMEM allocation, UMMA issue (one thread)
// TMEM (512 columns): group x's S at 256 x, its O at 256 x + 128.
// No atomics: the result is deterministic.
#include <cuda_bf16.h>

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
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kUmmaThreads = 10 * 32;
constexpr float kRescaleLog2 = 8.f;      // O and the sum are rescaled when the maximum grew by more (P <= 2^8)

__device__ __forceinline__ int umma_site(int role, int which) { return 620 + role * 10 + which; }

// QT query tiles of a unit share the K/V tiles (1: no unit has more than 128 rows).
template <int D, int QT>
struct UmmaCfg {
  static constexpr int kTileBytes = 128 * D * 2;          // 128 rows of Q, K or V
  static constexpr int kAtoms = D / 64;
  static constexpr int kSlots = (QT == 1 ? 6 : 5) * (128 / D);
  static constexpr int kSmemBytes = 1024 + (QT + kSlots) * kTileBytes;
  static_assert(kSmemBytes <= 227 * 1024 - 1400, "fits one CTA beside the static shared memory");
  static_assert(kSlots >= 5, "K(t), V(t), K(t + 1), V(t + 1), K(t + 2) are in use together");
};

// MN-major operand in the 128-byte-swizzled layout TMA writes: 128-byte rows
// along K (keys), 8-row atoms stacked along K, 64-column blocks lbo apart.
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t smem_addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

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
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// --------------------------------------------------------------------------
template <typename T, int D, int QT>
__global__ void __launch_bounds__(kUmmaThreads, 1)
    tree_umma_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap ktmap,
                     const __grid_constant__ CUtensorMap vtmap, const __grid_constant__ TreeParams p) {
  using C = UmmaCfg<D, QT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const Q_s = smem;                                  // [QT tiles]
  uint8_t* const ring = smem + QT * C::kTileBytes;            // K(0), V(0), K(1), V(1), ...

  __shared__ __align__(8) uint64_t q_full, q_empty, full[C::kSlots], empty[C::kSlots], s_full[2], p_half[2], p_full[2],
      run_done, o_empty, ml_ready;
  __shared__ TreeStart start_s;
  __shared__ float2 ml_s[128];               // group 1's row states, for group 0
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_half[x], kGroupWarps);
      mbar_init(&p_full[x], kGroupWarps);
    }
    mbar_init(&run_done, 1);
    mbar_init(&o_empty, 2 * kGroupWarps);
    mbar_init(&ml_ready, kGroupWarps);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    const TreeStart s = tree_start<kKeys>(p, blockIdx.x, blockIdx.x == 0);
    if (lane == 0) start_s = s;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_holder, 512);
    tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_map(&qmap);
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = tmem_holder;
  volatile int* const abort_v = &abort_flag;
  TreeWalker<kKeys, true> walk(start_s);
  TreeRun run;

  if (warp == kProducerWarp) {
    // ---------------------------------------------------------------- producer
    uint32_t seq = 0;              // K and V tiles loaded: slot seq % kSlots
    int runs = 0, q_last = -1;
    uint32_t issued = 0;           // slots that a copy was started into
    bool ok = true;
    // K or V tile: waits for its slot, then every lane copies its part
    auto load = [&](const CUtensorMap* pages, const CUtensorMap* nodes, const TreeTile& tile, int boxes, int in_page,
                    int unit) -> bool {
      const int slot = seq % C::kSlots;
      bool w = mbar_wait(&empty[slot], ((seq / C::kSlots) & 1) ^ 1, abort_v, umma_site(0, 1));
      if (!__all_sync(0xffffffffu, w)) return false;
      if (lane == 0) {
        if (tile.n == 0)
          mbar_arrive(&full[slot]);
        else
          mbar_arrive_expect_tx(&full[slot], tile.cached ? boxes * p.box_rows * 128 * C::kAtoms : C::kTileBytes);
      }
      __syncwarp();
      uint8_t* const dst = ring + slot * C::kTileBytes;
      if (lane < boxes) {
#pragma unroll
        for (int a = 0; a < C::kAtoms; ++a)
          tma_load_3d(dst + a * 16384 + lane * p.box_rows * 128, pages, &full[slot], a * 64, in_page, unit);
      } else if (!tile.cached && tile.n > 0 && lane == 0) {
#pragma unroll
        for (int a = 0; a < C::kAtoms; ++a)
          tma_load_3d(dst + a * 16384, nodes, &full[slot], a * 64, tile.first, run.unit);
      }
      ++seq;
      issued = seq;
      return true;
    };
    while (ok && walk.next(p, run)) {
      const int* table = p.table + static_cast<size_t>(run.e.seq) * p.max_pages;
      const int lh = run.unit - run.b * p.layers * p.hkv;
      const int layer = lh / p.hkv, head = lh - layer * p.hkv;
      ok = __all_sync(0xffffffffu, mbar_wait(&q_empty, (runs & 1) ^ 1, abort_v, umma_site(0, 0)));
      if (!ok) break;
      if (lane == 0) {
        const int tiles = run.pair ? 2 : 1;
        mbar_arrive_expect_tx(&q_full, tiles * C::kTileBytes);
        for (int x = 0; x < tiles; ++x)
          for (int a = 0; a < C::kAtoms; ++a)
            tma_load_3d(Q_s + x * C::kTileBytes + a * 16384, &qmap, &q_full, a * 64, run.row0 + x * 128, run.unit);
      }
      q_last = runs & 1;
      for (int t = run.t0; ok && t < run.t1; ++t) {
        const TreeTile tile = tree_tile<kKeys>(p, run.e, t);
        const int boxes = tile.cached ? (tile.n + p.box_rows - 1) / p.box_rows : 0;
        int unit = 0, in_page = 0;
        if (lane < boxes) {
          const int t_row = tile.first + lane * p.box_rows;
          const int at = t_row / p.page_rows;
          in_page = t_row - at * p.page_rows;
          const int page = __ldg(table + at);
          if (page < 0 || page >= p.n_pages) {
            record_error(SPK_DEVERR_INDEX, run.b);
            unit = p.layers * p.n_pages * p.hkv;             // outside the map: the box reads as zeros
          } else {
            unit = (layer * p.n_pages + page) * p.hkv + head;
          }
        }
        ok = load(&kmap, &ktmap, tile, boxes, in_page, unit);
        if (ok) ok = load(&vmap, &vtmap, tile, boxes, in_page, unit);
      }
      ++runs;
    }
    if (!ok && lane == 0) {        // let the copies in flight land before the block ends
      volatile int never = 0;
      if (q_last >= 0) mbar_wait(&q_full, q_last, &never, umma_site(0, 7), 100000000ull);
      for (uint32_t s = issued > C::kSlots ? issued - C::kSlots : 0; s < issued; ++s)
        mbar_wait(&full[s % C::kSlots], (s / C::kSlots) & 1, &never, umma_site(0, 8), 100000000ull);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------- UMMA issuer
    if (lane == 0) {
      bool ok = true;
      uint32_t base = 0;           // K/V tiles of this CTA before the run
      uint32_t jobs_of[2] = {0, 0};
      int runs = 0;
      constexpr uint32_t idesc_s = idesc_of<T>(128, 128);
      constexpr uint32_t idesc_pv = idesc_of<T>(128, D) | (1u << 16);     // B (V) MN-major
      auto issue_s = [&](int j) -> bool {
        const int x = j & 1, t = run.pair ? j >> 1 : j;
        const uint32_t seq = 2 * (base + t);
        const int slot = seq % C::kSlots;
        if (!(run.pair && x == 1) && !mbar_wait(&full[slot], (seq / C::kSlots) & 1, abort_v, umma_site(1, 1)))
          return false;
        tc_fence_after();
        const uint64_t q_desc = sw128_kmajor_desc(smem_u32(Q_s + (QT == 2 && run.pair ? x : 0) * C::kTileBytes));
        const uint64_t k_desc = sw128_kmajor_desc(smem_u32(ring + slot * C::kTileBytes));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          umma_bf16_ss(tmem + x * 256, q_desc + off, k_desc + off, idesc_s, kk > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[x]);
        if (!run.pair || x == 1) umma_commit(&empty[slot]);
        return true;
      };
      // A full tile in two halves: keys 64 .. 127 as soon as the softmax has
      // stored their P, then keys 0 .. 63.  A tile that ends earlier: the
      // k-steps that hold a key.
      auto issue_pv = [&](int j) -> bool {
        const int x = j & 1, t = run.pair ? j >> 1 : j;
        const uint32_t seq = 2 * (base + t) + 1;
        const int slot = seq % C::kSlots;
        const uint32_t ph = jobs_of[x] & 1;
        ++jobs_of[x];
        const TreeTile tile = tree_tile<kKeys>(p, run.e, run.t0 + t);
        const uint32_t v_base = smem_u32(ring + slot * C::kTileBytes);
        bool fresh = j < 2;        // O of this group starts with this job
        auto steps = [&](int k0, int k1) {
#pragma unroll 4
          for (int kk = k0; kk < k1; ++kk) {
            umma_bf16_ts(tmem + x * 256 + 128, tmem + x * 256 + 64 + kk * 8, mnmajor_desc(v_base + kk * 2048, 16384),
                         idesc_pv, fresh ? 0u : 1u);
            fresh = false;
          }
        };
        const bool whole = tile.n == kKeys;
        if (whole && !mbar_wait(&p_half[x], ph, abort_v, umma_site(1, 2 + x))) return false;
        if (!whole && !mbar_wait(&p_full[x], ph, abort_v, umma_site(1, 4 + x))) return false;
        if (!(run.pair && x == 1) && !mbar_wait(&full[slot], (seq / C::kSlots) & 1, abort_v, umma_site(1, 6)))
          return false;
        // both groups have read the previous run's O before it is restarted
        if (j == 0 && runs > 0 && !mbar_wait(&o_empty, (runs - 1) & 1, abort_v, umma_site(1, 7))) return false;
        tc_fence_after();
        if (whole) {
          steps(4, 8);
          if (!mbar_wait(&p_full[x], ph, abort_v, umma_site(1, 4 + x))) return false;
          tc_fence_after();
          steps(0, 4);
        } else {
          steps(0, (tile.n + 15) / 16);
        }
        if (!run.pair || x == 1) umma_commit(&empty[slot]);
        return true;
      };
      while (ok && walk.next(p, run)) {
        if (!(ok = mbar_wait(&q_full, runs & 1, abort_v, umma_site(1, 0)))) break;
        const int n = run.jobs();
        for (int j = 0; ok && j < 2 && j < n; ++j) ok = issue_s(j);
        if (ok && n <= 2) umma_commit(&q_empty);
        for (int j = 0; ok && j < n; ++j) {
          ok = issue_pv(j);
          if (ok && j + 2 < n) {
            ok = issue_s(j + 2);
            if (ok && j + 3 == n) umma_commit(&q_empty);
          }
        }
        if (!ok) break;
        umma_commit(&run_done);
        base += run.t1 - run.t0;
        ++runs;
      }
      if (!ok) {                   // the products in flight end before the block does
        umma_commit(&run_done);
        volatile int never = 0;
        mbar_wait(&run_done, runs & 1, &never, umma_site(1, 9), 100000000ull);
      }
    }
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
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_v, umma_site(2 + x, which)));
    };
    while (ok && walk.next(p, run)) {
      const int row = run.row0 + (run.pair ? x * 128 : 0) + r;  // row of the unit
      const bool there = row < p.rows;
      const int node = there ? row % p.T : 0;
      const int n_jobs = run.jobs();
      float m = -INFINITY, l = 0.f;                            // running maximum of c2 s, sum
      bool fresh = true;                                       // O holds nothing yet
      for (int j = x; ok && j < n_jobs; j += 2, ++job) {
        const int t = run.pair ? j >> 1 : j;
        const TreeTile tile = tree_tile<kKeys>(p, run.e, run.t0 + t);
        if (!(ok = wait_all(&s_full[x], job & 1, 0))) break;
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
        if (tile.cached && tile.n == kKeys) {
          // every row sees every key: no masks.  Columns [64, 128) stay in
          // registers, [0, 64) are read twice
          float mx;
          uint32_t b0[32], b1[32];
          {
            uint32_t a0[32], a1[32];
            tmem_ld32(mine, a0);
            tmem_ld32(mine + 32, a1);
            tmem_ld_wait2(a0, a1);
            mx = max32(a1, max32(a0, -INFINITY));
          }
          tmem_ld32(mine + 64, b0);
          tmem_ld32(mine + 96, b1);
          tmem_ld_wait2(b0, b1);
          mx = max32(b1, max32(b0, mx));
          rescale(mx * p.c2);
          const float2 c2v = f2(p.c2, p.c2), nm = f2(-m, -m);
          float2 acc = f2(0.f, 0.f);
          auto exp32 = [&](const uint32_t (&a)[32], uint32_t (&pk)[32], int at) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 tt = __ffma2_rn(f2(__uint_as_float(a[2 * k]), __uint_as_float(a[2 * k + 1])), c2v, nm);
              const float2 e = exp2_mufu_pair(tt);
              acc = __fadd2_rn(acc, e);
              pk[at + k] = Half16<T>::pack(e.x, e.y);
            }
          };
          {
            uint32_t pk[32];
            exp32(b0, pk, 0);
            exp32(b1, pk, 16);
            tmem_st32(mine + 96, pk);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_half[x]);
          {
            uint32_t a0[32], a1[32], pk[32];
            tmem_ld32(mine, a0);
            tmem_ld32(mine + 32, a1);
            tmem_ld_wait2(a0, a1);
            exp32(a0, pk, 0);
            exp32(a1, pk, 16);
            tmem_st32(mine + 64, pk);
          }
          l += acc.x + acc.y;
        } else {
          // a tile that ends early, or the nodes: 32 columns at a time, those
          // that hold a key; which of them this row sees, as a word
          const int chunks = (tile.n + 31) / 32;
          auto word = [&](int c) -> uint32_t {
            const int left = tile.n - c * 32;
            const uint32_t here = left >= 32 ? 0xffffffffu : (1u << left) - 1u;     // left >= 1
            if (tile.cached) return here;
            if (!there) return 0u;
            const int n0 = tile.first + c * 32;
            if (p.mask != nullptr)
              return here & __ldg(p.mask + (static_cast<size_t>(run.b) * p.T + node) * p.words + (n0 >> 5));
            return node < n0 ? 0u : here & (node - n0 >= 31 ? 0xffffffffu : (2u << (node - n0)) - 1u);
          };
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            const uint32_t w = word(c);
            uint32_t a[32];
            tmem_ld32(mine + c * 32, a);
            tmem_ld_wait(a);
#pragma unroll
            for (int k = 0; k < 32; ++k) mx = (w >> k) & 1u ? fmaxf(mx, __uint_as_float(a[k])) : mx;
          }
          rescale(mx * p.c2);
          const float ref = m == -INFINITY ? 0.f : m;          // no key yet: every weight is 0
          // from the last chunk down: P of chunk c lies over S of chunk c / 2 + 2
#pragma unroll 1
          for (int c = chunks - 1; c >= 0; --c) {
            const uint32_t w = word(c);
            uint32_t a[32], pk[16];
            tmem_ld32(mine + c * 32, a);
            tmem_ld_wait(a);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float e0 = (w >> (2 * k)) & 1u ? ex2_approx(fmaf(__uint_as_float(a[2 * k]), p.c2, -ref)) : 0.f;
              const float e1 = (w >> (2 * k + 1)) & 1u ? ex2_approx(fmaf(__uint_as_float(a[2 * k + 1]), p.c2, -ref)) : 0.f;
              l += e0 + e1;
              pk[k] = Half16<T>::pack(e0, e1);
            }
            tmem_st16(mine + 64 + c * 16, pk);
          }
          // V rows behind the last key, up to the end of its k-step: whatever the
          // slot holds (it may be NaN) must not meet the zeros of P
          const int bad = (16 - (tile.n & 15)) & 15;
          if (bad > 0 && !(run.pair && x == 1)) {              // (a pair's group 1 comes behind group 0's products)
            const uint32_t seq = 2 * (base + t) + 1;
            const int slot = seq % C::kSlots;
            if (!(ok = wait_all(&full[slot], (seq / C::kSlots) & 1, 1))) break;
            for (int i = r; i < bad * (D / 8); i += 128) {
              const int vr = tile.n + i / (D / 8), ch = i % (D / 8);
              *reinterpret_cast<uint4*>(ring + slot * C::kTileBytes + (ch >> 3) * 16384 + vr * 128 +
                                        (((ch & 7) ^ (vr & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_half[x]);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
        fresh = false;
      }
      if (!ok) break;
      // ---- the run's outputs: a pair's groups have a query tile each; ALONE,
      // group 0 joins both groups' states (group 1 may go on)
      if (!(ok = wait_all(&run_done, runs & 1, 2))) break;
      tc_fence_after();
      float f0 = 1.f, f1 = 0.f;                                // weights of O_0 and O_1 (ALONE)
      if (!run.pair) {
        if (x == 1) {
          // (group 0 read the previous run's states before run_done of this one)
          ml_s[r] = make_float2(m, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(&ml_ready);
        } else {
          if (!(ok = wait_all(&ml_ready, alone_runs & 1, 3))) break;
          ++alone_runs;
          const float2 other = ml_s[r];
          const float M = fmaxf(m, other.x), ref = M == -INFINITY ? 0.f : M;
          f0 = ex2_approx(m - ref);
          f1 = ex2_approx(other.x - ref);
          l = l * f0 + other.y * f1;
          m = M;
        }
      }
      if (run.pair || x == 0) {
        const bool whole = run.t0 == 0 && run.t1 == run.e.tiles;
        const bool live = there && node < run.e.live;
        const float scale = whole ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;
        f0 *= scale;
        f1 *= scale;
        const bool any = l != 0.f;                             // a row without keys: zeros, whatever O holds
        const bool both = !run.pair && n_jobs > 1;             // group 1 had a job
        const size_t slot_row = (static_cast<size_t>(blockIdx.x) * 2 + run.slot) * (QT * 128) + (run.pair ? x * 128 : 0) + r;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(mine + 128 + c, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = any ? __float_as_uint(__uint_as_float(o[k]) * f0) : 0u;
          if (both) {
            uint32_t o1[32];
            tmem_ld32(lanes + 256 + 128 + c, o1);
            tmem_ld_wait(o1);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (any) o[k] = __float_as_uint(fmaf(__uint_as_float(o1[k]), f1, __uint_as_float(o[k])));
          }
          if (live) {
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (static_cast<size_t>(run.unit) * p.rows + row) * D + c);
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                uint4 w;
                w.x = Half16<T>::pack(__uint_as_float(o[8 * v + 0]), __uint_as_float(o[8 * v + 1]));
                w.y = Half16<T>::pack(__uint_as_float(o[8 * v + 2]), __uint_as_float(o[8 * v + 3]));
                w.z = Half16<T>::pack(__uint_as_float(o[8 * v + 4]), __uint_as_float(o[8 * v + 5]));
                w.w = Half16<T>::pack(__uint_as_float(o[8 * v + 6]), __uint_as_float(o[8 * v + 7]));
                dst[v] = w;
              }
            } else {
              uint4* dst = reinterpret_cast<uint4*>(p.part_o + slot_row * D + c);
#pragma unroll
              for (int v = 0; v < 8; ++v) dst[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
            }
          }
        }
        if (live) {
          if (!whole)
            *reinterpret_cast<float2*>(p.part_ml + slot_row * 2) = make_float2(m, l);
          else if (p.lse2 != nullptr)
            p.lse2[static_cast<size_t>(run.unit) * p.rows + row] = l == 0.f ? -INFINITY : m + lg2_approx(l);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty);
      base += run.t1 - run.t0;
      ++runs;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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

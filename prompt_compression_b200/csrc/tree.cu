// tree.cu -- attention for a tree of drafted tokens over a paged KV cache.
//
// Row r = (query head, node i) of a unit (batch element, layer, KV head):
//   z_j  = scale * q_r . k_j   over the n cached rows and the tree's nodes j
//                              with bit j of the visibility words of node i
//   out  = sum_j 2^(c2 s_j - m) v_j / sum_j 2^(c2 s_j - m),  lse2 = m + log2 sum,
// in one pass with the running maximum m and sum (log2 domain, fp32).
//
// This kernel has the units of few query rows (row tiles of 8, 16 or 32, on
// mma.sync); tree_umma.cu has the others.  How the work is shared out:
// tree_shares.cuh.  An item inside one share is finished there; the others
// leave (m, sum, unnormalised output) of each share in the workspace, to be
// added in the order of the shares, so that the results do not depend on
// timing.  Where there are at least twice as many items as CTAs the share that
// arrives last does it, one share after the other: with items of like lengths
// an item is then in two shares at most; one long sequence among short ones is
// in many, which costs time but is right.  Otherwise tree_join_kernel does it,
// which spreads the many shares of an item over the GPU.
// (The one way and the other, us: 16 nodes over 320 rows, 512 KV heads, 39.5 and
// 45.2; one node over 16K rows, 8 KV heads in 37 shares each, 41.2 and 20.2; over
// 80 sequences of 1500 rows 86.3 and 84.8; over 79 sequences of 300 rows and one of
// 65,536, whose items lie in 22 shares, 75.5 and 68.6.  One of 16K rows beside 73
// elements without a live node, about 32 shares: 37 joined inside, 20 by itself.)
#include <type_traits>

#include "common.cuh"
#include "mma.cuh"
#include "paged.cuh"
#include "tree_shares.cuh"

namespace spk {

SPK_ERROR_READER(device_errors_tree)

namespace {

constexpr int kTreeKeys = 64;                   // keys of a tile
constexpr int kWarps = 4;                       // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;     // and the producer warp
constexpr int kSmemPerCta = 113 * 1024;         // two CTAs share an SM

__device__ __forceinline__ int site(int which) { return 600 + which; }

// --------------------------------------------------------------------------
// main kernel
// --------------------------------------------------------------------------
template <int D, int NT>
struct TreeCfg {
  static constexpr int kRows = 8 * NT;                  // query rows of a tile
  static constexpr int kHalf = kTreeKeys * 128;         // 64 keys x 64 columns
  static constexpr int kAtoms = D / 64;
  static constexpr int kStageBytes = 2 * kAtoms * kHalf;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kPBytes = kRows * kTreeKeys * 2;
  static constexpr int kStages = (kSmemPerCta - 2048 - 1024 - 4 * kRows * 4 - kQBytes - kPBytes) /
                                 kStageBytes;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kQBytes + kPBytes;
  static_assert(kStages >= 2, "a tile is loaded while another is used");
};

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Four consumer warps.  Per tile, warp w takes 16 of its keys for the logits
//   S^T[key][row] = K Q^T               (A = K by ldmatrix, B = Q)
// the four warps exchange their column maxima, leave P = 2^(c2 s - m) in shared
// memory as 16-bit values, and then each takes a quarter of head_dim for
//   O^T[d][row] = alpha O^T + V^T P^T   (A = V^T by ldmatrix.trans, B = P^T),
// so no state is merged at the end of a unit.  P is rounded to the element
// type for the product (the largest weight is 1 exactly, the others are off by
// half a step at most, and the errors average over the keys: outputs in bf16 are
// 2.2e-3 off, relative, of which their own rounding makes 1.7e-3); the sum is
// formed from the fp32 values, so lse2 keeps 32 bits.
// LOSES: a self-test of the waits. The second tile of CTA 0 never comes.
template <typename T, int D, int NT, bool LOSES>
__global__ void __launch_bounds__(kThreads, 2)
    tree_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                const __grid_constant__ CUtensorMap ktmap, const __grid_constant__ CUtensorMap vtmap,
                const __grid_constant__ CUtensorMap k8map, const __grid_constant__ CUtensorMap v8map,
                const __grid_constant__ TreeParams p) {
  using C = TreeCfg<D, NT>;
  constexpr int KS = D / 16;              // k-steps of the logits
  constexpr int DW = D / kWarps;          // head_dim columns of a warp
  constexpr int MT = DW / 16;             // their m-tiles
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t stage_s = smem_u32(smem);
  uint8_t* const q_p = smem + C::kStages * C::kStageBytes;
  const uint32_t q_s = smem_u32(q_p), p_s = q_s + C::kQBytes;

  __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages];
  __shared__ TreeStart start_s;
  __shared__ __align__(16) float wmax[kWarps][C::kRows];   // read and written in pairs
  __shared__ int abort_flag, last_s;
  __shared__ int wild_s[2];      // nodes [x, y) whose V holds something that is not finite (y 0: none)

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    abort_flag = 0;
    wild_s[0] = kTreeMaxNodes;
    wild_s[1] = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    const TreeStart s = tree_start<kTreeKeys>(p, blockIdx.x, blockIdx.x == 0);
    if (lane == 0) start_s = s;
  }
  if (warp == kWarps && lane == 0) {
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
  }
  __syncthreads();
  volatile int* const abort_v = &abort_flag;
  if (!p.join_inside) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  TreeWalker<kTreeKeys, false> walk(start_s);
  TreeRun run;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    uint32_t count = 0;
    bool ok = true;
    int last[C::kStages];
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) last[s] = -1;
    while (ok && walk.next(p, run)) {
      const int* row = p.table + static_cast<size_t>(run.e.seq) * p.max_pages;
      for (int t = run.t0; t < run.t1; ++t, ++count) {
        const TreeTile tile = tree_tile<kTreeKeys>(p, run.e, t);
        const int st = count % C::kStages;
        const uint32_t ph = (count / C::kStages) & 1;
        // lane i: the page of box i of the tile's cached rows
        // (a tile that ends early in parts of 8 rows: the nodes may lie right behind)
        const int part_rows = tile.rows == kTreeKeys ? p.box_rows : 8, boxes = (tile.rows + part_rows - 1) / part_rows;
        const CUtensorMap* const km = tile.rows == kTreeKeys ? &kmap : &k8map;
        const CUtensorMap* const vm = tile.rows == kTreeKeys ? &vmap : &v8map;
        int unit = 0, in_page = 0;
        if (lane < boxes) {
          const int t_row = tile.first + lane * part_rows;
          const int slot = t_row / p.page_rows;
          in_page = t_row - slot * p.page_rows;
          const int page = __ldg(row + slot);
          if (page < 0 || page >= p.n_pages) {
            record_error(SPK_DEVERR_INDEX, run.b);
            unit = p.layers * p.n_pages * p.hkv;     // outside the map: the box reads as zeros
          } else {
            unit = run.pool + page * p.hkv;
          }
        }
        ok = !(LOSES && blockIdx.x == 0 && count == 1) && mbar_wait(&empty[st], ph ^ 1, abort_v, site(0));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int bytes = (boxes * part_rows + (tile.nodes > 0 ? p.node_rows : 0)) * 128 * 2 * C::kAtoms;
        if (lane == 0) {
          if (bytes > 0)
            mbar_arrive_expect_tx(&full[st], bytes);
          else
            mbar_arrive(&full[st]);
        }
        __syncwarp();
        uint8_t* const kp = smem + st * C::kStageBytes;
        if (lane < boxes) {
          uint8_t* const dst = kp + lane * part_rows * 128;
#pragma unroll
          for (int a = 0; a < C::kAtoms; ++a) {
            tma_load_3d(dst + a * C::kHalf, km, &full[st], a * 64, in_page, unit);
            tma_load_3d(dst + (C::kAtoms + a) * C::kHalf, vm, &full[st], a * 64, in_page, unit);
          }
        }
        if (tile.nodes > 0 && lane == 0) {
#pragma unroll
          for (int a = 0; a < C::kAtoms; ++a) {
            tma_load_3d(kp + a * C::kHalf + tile.off * 128, &ktmap, &full[st], a * 64, tile.node0, run.unit);
            tma_load_3d(kp + (C::kAtoms + a) * C::kHalf + tile.off * 128, &vtmap, &full[st], a * 64, tile.node0, run.unit);
          }
        }
#pragma unroll
        for (int s = 0; s < C::kStages; ++s)
          if (s == st) last[s] = static_cast<int>(ph);
      }
    }
    if (!ok && lane == 0) {   // let the copies in flight land before the block ends
      volatile int never = 0;
#pragma unroll
      for (int s = 0; s < C::kStages; ++s)
        if (last[s] >= 0) mbar_wait(&full[s], last[s], &never, site(1), 100000000ull);
    }
  } else {
    // --------------------------------------------------------------- consumers
    // A wait that runs out raises the abort flag; the warps go on through their
    // barriers (every later wait returns at once) and the error word says so.
    const int gr = lane >> 2, gc = lane & 3;
    uint32_t count = 0;
    while (walk.next(p, run)) {
      const int rows = min(C::kRows, p.rows - run.row0);     // rows of this tile that exist
      // Q rows of the tile (they lie together: a unit's heads and nodes), zeros behind them
      {
        const uint4* src = reinterpret_cast<const uint4*>(p.q) +
                           (static_cast<size_t>(run.unit) * p.rows + run.row0) * (D / 8);
        for (int x = threadIdx.x; x < C::kRows * (D / 8); x += kWarps * 32) {
          const int row = x / (D / 8), ch = x % (D / 8);
          const uint4 w = row < rows ? __ldg(src + x) : make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(q_p + row * (D * 2) + ((ch ^ (row & 7)) << 4)) = w;
        }
      }
      consumers_sync();
      float o[MT][NT][4];
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int j = 0; j < MT; ++j) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.f;
      }
      for (int t = run.t0; t < run.t1; ++t, ++count) {
        const TreeTile tile = tree_tile<kTreeKeys>(p, run.e, t);
        const int st = count % C::kStages;
        const uint32_t ks = stage_s + st * C::kStageBytes, vs = ks + C::kAtoms * C::kHalf;
        const int key0 = warp * 16;
        // which of keys gr, gr + 8 each row sees
        uint32_t sees[NT][2];
        if (tile.rows == kTreeKeys) {
#pragma unroll
          for (int n = 0; n < NT; ++n) sees[n][0] = sees[n][1] = 3u;
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int r = run.row0 + 8 * n + 2 * gc + c;
              const uint32_t w = tree_word(p, run.b, tile, key0, r % p.T, r < p.rows);
              sees[n][c] = ((w >> gr) & 1u) | (((w >> (gr + 8)) & 1u) << 1);
            }
          }
        }
        mbar_wait(&full[st], (count / C::kStages) & 1, abort_v, site(2));

        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        if (key0 < tile.n) {
          const int arow = key0 + (lane & 15);
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint32_t a[4], b[4];
            const int ch = 2 * k + (lane >> 4);
            ldsm_x4(ks + (ch >> 3) * C::kHalf + arow * 128 + (((ch & 7) ^ (arow & 7)) << 4), a);
            const int ch2 = ch + 2;
            ldsm_x4(ks + (ch2 >> 3) * C::kHalf + arow * 128 + (((ch2 & 7) ^ (arow & 7)) << 4), b);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint32_t q[4];
              const int row = 8 * n + (lane & 7);
              ldsm_x4(q_s + row * (D * 2) + (((2 * k + (lane >> 3)) ^ (row & 7)) << 4), q);
              Half16<T>::mma(s[n], a, q[0], q[1]);
              Half16<T>::mma(s[n], b, q[2], q[3]);
            }
          }
        }
        // this warp's maximum of each row, then all four warps'
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float mx[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            s[n][c] = (sees[n][c] & 1u) ? s[n][c] * p.c2 : -INFINITY;
            s[n][2 + c] = (sees[n][c] & 2u) ? s[n][2 + c] * p.c2 : -INFINITY;
            mx[c] = fmaxf(s[n][c], s[n][2 + c]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], x));
          }
          if (gr == 0) *reinterpret_cast<float2*>(&wmax[warp][8 * n + 2 * gc]) = make_float2(mx[0], mx[1]);
        }
        consumers_sync();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float mx[2] = {m[n][0], m[n][1]};
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 y = *reinterpret_cast<const float2*>(&wmax[w][8 * n + 2 * gc]);
            mx[0] = fmaxf(mx[0], y.x);
            mx[1] = fmaxf(mx[1], y.y);
          }
          float ref[2], alpha[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            ref[c] = mx[c] == -INFINITY ? 0.f : mx[c];     // no key yet: every weight is 2^-inf = 0
            alpha[c] = ex2_approx(m[n][c] - ref[c]);
            m[n][c] = mx[c];
          }
          float e[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) e[x] = ex2_approx(s[n][x] - ref[x & 1]);
          const uint32_t lo = Half16<T>::pack(e[0], e[1]), hi = Half16<T>::pack(e[2], e[3]);
          l[n][0] = fmaf(l[n][0], alpha[0], e[0] + e[2]);
          l[n][1] = fmaf(l[n][1], alpha[1], e[1] + e[3]);
          const int row = 8 * n + (lane & 7);
          stsm_x2_t(p_s + row * 128 + (((2 * warp + ((lane >> 3) & 1)) ^ (row & 7)) << 4), lo, hi);
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            o[j][n][0] *= alpha[0];
            o[j][n][1] *= alpha[1];
            o[j][n][2] *= alpha[0];
            o[j][n][3] *= alpha[1];
          }
        }
        // V rows without a key: whatever the slot holds (it may be NaN) must not meet
        // the zeros of P, so they are cleared, up to the end of the last k-step
        const int steps = (tile.n + 15) / 16;
        const int gap = tile.nodes > 0 ? tile.off - tile.rows : 0, bad = gap + steps * 16 - tile.n;
        if (bad > 0) {
          constexpr int kCh = DW / 8;            // this warp's 16-byte columns
          for (int x = lane; x < bad * kCh; x += 32) {
            const int b = x / kCh, ch = warp * kCh + x % kCh;
            const int row = b < gap ? tile.rows + b : tile.n + b - gap;
            uint8_t* at = smem + st * C::kStageBytes + C::kAtoms * C::kHalf + (ch >> 3) * C::kHalf + row * 128 +
                          (((ch & 7) ^ (row & 7)) << 4);
            *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();              // before the slot's next copy
        }
        if (tile.nodes > 0) {                    // and in the nodes' rows what is not finite: not every row sees them
          constexpr int kCh = DW / 8;
          bool found = false;
          for (int x = lane; x < tile.nodes * kCh; x += 32) {
            const int row = tile.off + x / kCh, ch = warp * kCh + x % kCh;
            uint4* const at = reinterpret_cast<uint4*>(smem + st * C::kStageBytes + C::kAtoms * C::kHalf + (ch >> 3) * C::kHalf +
                                                       row * 128 + (((ch & 7) ^ (row & 7)) << 4));
            uint4 w = *at;
            if (tree_clear_wild(w, Half16<T>::kExponent)) {
              *at = w;
              found = true;
            }
          }
          if (found) {
            atomicMin(&wild_s[0], tile.node0);
            atomicMax(&wild_s[1], tile.node0 + tile.nodes);
            fence_proxy_async_smem();
          }
        }
        consumers_sync();
#pragma unroll
        for (int k = 0; k < kTreeKeys / 16; k += 2) {
          if (k >= steps) break;
          uint32_t b[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int row = 8 * n + (lane & 7);
            ldsm_x4(p_s + row * 128 + (((2 * k + (lane >> 3)) ^ (row & 7)) << 4), b[n]);
          }
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            if (k + kk >= steps) break;
            const int vrow = (k + kk) * 16 + (lane & 7) + (lane >> 4) * 8;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              uint32_t a[4];
              const int ch = warp * (DW / 8) + 2 * j + ((lane >> 3) & 1);
              ldsm_x4_t(vs + (ch >> 3) * C::kHalf + vrow * 128 + (((ch & 7) ^ (vrow & 7)) << 4), a);
#pragma unroll
              for (int n = 0; n < NT; ++n) Half16<T>::mma(o[j][n], a, b[n][2 * kk], b[n][2 * kk + 1]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }

      // row sums over the keys of all warps (wmax is free: every warp is past the last tile's maxima)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], x);
        if (gr == 0) *reinterpret_cast<float2*>(&wmax[warp][8 * n + 2 * gc]) = make_float2(l[n][0], l[n][1]);
      }
      consumers_sync();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 y = *reinterpret_cast<const float2*>(&wmax[w][8 * n + 2 * gc]);
          l[n][0] += y.x;
          l[n][1] += y.y;
        }
      }
      // rows that see a node whose V is not finite (thread = row, every fourth column)
      auto patch = [&]() {
        const int lo = wild_s[0], hi = wild_s[1];
        if (hi == 0) return;
        consumers_sync();                        // the outputs are there
#pragma unroll 1
        for (int y = threadIdx.x; y < rows * 4; y += kWarps * 32) {
          const int row = y >> 2, r = run.row0 + row, i = r % p.T;
          if (i >= run.e.live) continue;
          if (run.from == run.to)
            tree_patch<T>(p, run.b, run.unit, i, lo, hi, y & 3, D, 4, D,
                          static_cast<T*>(p.out) + (static_cast<size_t>(run.unit) * p.rows + r) * D, D, size_t(0));
          else
            tree_patch<T>(p, run.b, run.unit, i, lo, hi, y & 3, D, 4, D,
                          p.part_o + ((static_cast<size_t>(blockIdx.x) * 2 + run.slot) * (D / 4) * C::kRows + row) * 4, 4,
                          static_cast<size_t>(C::kRows) * 4);
        }
        consumers_sync();
        if (threadIdx.x == 0) {
          wild_s[0] = kTreeMaxNodes;
          wild_s[1] = 0;
        }
      };
      if (run.from == run.to) {
        // the whole unit: outputs through shared memory (over Q), 16 bytes a store
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float i0 = l[n][0] > 0.f ? 1.f / l[n][0] : (l[n][0] == 0.f ? 0.f : l[n][0]);
          const float i1 = l[n][1] > 0.f ? 1.f / l[n][1] : (l[n][1] == 0.f ? 0.f : l[n][1]);
          const int row = 8 * n + (lane & 7);
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            const int ch = warp * (DW / 8) + 2 * j + ((lane >> 3) & 1);
            stsm_x2_t(q_s + row * (D * 2) + ((ch ^ (row & 7)) << 4), Half16<T>::pack(o[j][n][0] * i0, o[j][n][1] * i1),
                      Half16<T>::pack(o[j][n][2] * i0, o[j][n][3] * i1));
          }
          if (warp == 0 && gr == 0 && p.lse2 != nullptr) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int r = run.row0 + 8 * n + 2 * gc + c;
              if (r < p.rows && r % p.T < run.e.live)
                p.lse2[static_cast<size_t>(run.unit) * p.rows + r] =
                    l[n][c] == 0.f ? -INFINITY : m[n][c] + lg2_approx(l[n][c]);
            }
          }
        }
        consumers_sync();
        uint4* dst = reinterpret_cast<uint4*>(p.out) + (static_cast<size_t>(run.unit) * p.rows + run.row0) * (D / 8);
        for (int x = threadIdx.x; x < rows * (D / 8); x += kWarps * 32) {
          const int row = x / (D / 8), ch = x % (D / 8);
          if ((run.row0 + row) % p.T < run.e.live)
            dst[x] = *reinterpret_cast<const uint4*>(q_p + row * (D * 2) + ((ch ^ (row & 7)) << 4));
        }
        patch();
      } else {
        const size_t part = static_cast<size_t>(blockIdx.x) * 2 + run.slot;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int row = 8 * n + 2 * gc + c;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              const int d = warp * DW + 16 * j + gr;           // [4 columns][row], as the join reads it
              p.part_o[((part * (D / 4) + d / 4) * C::kRows + row) * 4 + d % 4] = o[j][n][c];
              p.part_o[((part * (D / 4) + d / 4 + 2) * C::kRows + row) * 4 + d % 4] = o[j][n][2 + c];
            }
            if (warp == 0 && gr == 0)
              *reinterpret_cast<float2*>(p.part_ml + (part * C::kRows + row) * 2) = make_float2(m[n][c], l[n][c]);
          }
        }
        patch();
        // the last of the item's shares joins them:
        //   M = max m_c,  out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c
        bool join = false;
        if (p.join_inside) {
          __threadfence();
          consumers_sync();
          if (threadIdx.x == 0) last_s = tree_arrive(p, run);
          consumers_sync();
          join = last_s;
        }
        if (join) {
#pragma unroll 1
          for (int y = threadIdx.x; y < C::kRows * (D / 4); y += kWarps * 32) {
            const int row = y % C::kRows, col4 = y / C::kRows, r = run.row0 + row;
            if (r >= p.rows || r % p.T >= run.e.live) continue;
            const float2* const ml = reinterpret_cast<const float2*>(p.part_ml) + row;
            const float4* const po = reinterpret_cast<const float4*>(p.part_o) + static_cast<size_t>(col4) * C::kRows + row;
            float M = -INFINITY, L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = run.from; c <= run.to; ++c) {
              const size_t at = tree_place(run, c);
              const float2 s = __ldcg(ml + at * C::kRows);
              const float4 o = __ldcg(po + at * (D / 4) * C::kRows);
              const float mx = fmaxf(M, s.x), ref = mx == -INFINITY ? 0.f : mx;
              const float f0 = ex2_approx(M - ref), f = ex2_approx(s.x - ref);
              M = mx;
              L = fmaf(s.y, f, L * f0);
              acc = make_float4(fmaf(o.x, f, acc.x * f0), fmaf(o.y, f, acc.y * f0), fmaf(o.z, f, acc.z * f0),
                                fmaf(o.w, f, acc.w * f0));
            }
            if (isnan(acc.x + acc.y + acc.z + acc.w))
              acc = tree_join_again(p, run.from, run.to, run.c0, run.slot0, row, col4, D / 4, acc);
            const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
            const size_t at = static_cast<size_t>(run.unit) * p.rows + r;
            reinterpret_cast<uint2*>(p.out)[at * (D / 4) + col4] =
                make_uint2(Half16<T>::pack(acc.x * inv, acc.y * inv), Half16<T>::pack(acc.z * inv, acc.w * inv));
            if (col4 == 0 && p.lse2 != nullptr) p.lse2[at] = L == 0.f ? -INFINITY : M + lg2_approx(L);
          }
        }
      }
      consumers_sync();                          // Q, the staged outputs and the sums are free
    }
  }
}

// --------------------------------------------------------------------------
// the items that several shares hold
// --------------------------------------------------------------------------
// A row's shares are added in their order:
//   M = max m_c,  out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c.
// A block has eight rows of one item at a time; a thread has four columns of a
// row, and adds them over the shares, four shares' loads in flight together.
// MANY (an item has many shares): a block has 16 columns, and eight groups of
// such threads, each with every eighth share and eight loads in flight, joined
// through shared memory in the groups' order; blocks of 256 threads, so that
// they are resident beside the main kernel's.  (One node over 16K rows, 8 KV
// heads in 37 shares each: 19.7 us; blocks of 1024 threads with all columns
// and four groups, which start only when the main kernel's end: 22.0 us.)
// by_border: the item that the border between shares c and c + 1 cuts, if this
// is the first border inside it; otherwise item c of the call.  The blocks
// start while the main kernel still runs and find their item (the line does
// not depend on it), and wait before they read; every block waits, so the
// join ends after the main kernel.
constexpr int kJoinRows = 8;
constexpr int kJoinGroups = 8;                  // MANY
constexpr int kJoinCols = 4;                    // MANY: columns of a block, in fours (part blockIdx.z of them)

template <typename T, int D, int KEYS, bool PAIRS, bool MANY>
__global__ void __launch_bounds__(kJoinRows *(MANY ? kJoinCols * kJoinGroups : D / 4))
    tree_join_kernel(const __grid_constant__ TreeParams p, int item_rows, bool by_border) {
  constexpr int kGroup = kJoinRows * (MANY ? kJoinCols : D / 4);   // threads that hold eight rows
  constexpr int G = MANY ? kJoinGroups : 1;
  __shared__ float4 acc_s[MANY ? kGroup * (G - 1) : 1];
  __shared__ float2 ml_s[MANY ? kGroup * (G - 1) : 1];
  const int lane = threadIdx.x & 31;
  const int group = threadIdx.x / kGroup, me = threadIdx.x % kGroup;
  const int col4 = (MANY ? blockIdx.z * kJoinCols : 0) + me / kJoinRows;
  TreeStart s = tree_start<KEYS>(p, by_border ? blockIdx.x + 1 : 0, false);
  int x = s.begin;
  if (!by_border) {                             // every unit has the same number of items
    const int per = p.items;
    const int unit = blockIdx.x / per, k = blockIdx.x - unit * per, of_b = p.layers * p.hkv;
    s.b = unit / of_b;
    int before = 0;
    for (int b = lane; b < s.b; b += 32) before += tree_jobs(p, tree_element<KEYS>(p, b, false), s.extra);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    s.base = before;
    s.e = tree_element<KEYS>(p, s.b, false);
    x = s.e.tiles == 0 ? s.total
                       : before + (unit - s.b * of_b) * tree_unit_jobs(p, s.e.tiles, s.extra) +
                             k * (s.e.tiles * (PAIRS ? 2 : 1) + s.extra);
  }
  TreeItem item{};
  int c0 = 0, c1 = 0;
  if (x < s.total) {
    item = tree_item<PAIRS>(p, s.e, s.b, s.base, x, s.extra);
    const bool mine = !by_border || (item.first != x && item.first / s.share == static_cast<int>(blockIdx.x));
    if (mine) tree_spread(item, s.e.tiles, s.share, c0, c1);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c0 == c1) return;                         // no item, or one share has it
  const int rows_here = min(PAIRS ? (item.pair ? 256 : 128) : item_rows, p.rows - item.row0);
  for (int row0 = blockIdx.y * kJoinRows; row0 < rows_here; row0 += gridDim.y * kJoinRows) {
    const int row = row0 + me % kJoinRows;                   // in the item
    const int r = item.row0 + row;                           // in the unit
    const bool on = row < rows_here && r % p.T < s.e.live;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float2 ml, float4 o) {
      const float M = fmaxf(m, ml.x), ref = M == -INFINITY ? 0.f : M;
      const float a = ex2_approx(m - ref), f = ex2_approx(ml.x - ref);
      l = fmaf(l, a, ml.y * f);
      acc.x = fmaf(acc.x, a, o.x * f);
      acc.y = fmaf(acc.y, a, o.y * f);
      acc.z = fmaf(acc.z, a, o.z * f);
      acc.w = fmaf(acc.w, a, o.w * f);
      m = M;
    };
    if (on) {
      constexpr int U = MANY ? 8 : 4;
      for (int i0 = c0 + group; i0 <= c1; i0 += U * G) {
        float2 ml[U];
        float4 o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * G;
          int t0 = 0, t1 = 0, slot = 0;
          if (i <= c1) tree_part(item, s.e.tiles, i * s.share, (i + 1) * s.share, t0, t1, slot);
          ml[u] = make_float2(-INFINITY, 0.f);
          o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (t0 < t1) {
            const size_t part = static_cast<size_t>(i) * 2 + slot;
            ml[u] = __ldcs(reinterpret_cast<const float2*>(p.part_ml) + part * item_rows + row);
            o[u] = __ldcs(reinterpret_cast<const float4*>(p.part_o) + (part * (D / 4) + col4) * item_rows + row);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) add(ml[u], o[u]);
      }
    }
    if (MANY) {
      if (group > 0) {
        acc_s[MANY ? (group - 1) * kGroup + me : 0] = acc;
        ml_s[MANY ? (group - 1) * kGroup + me : 0] = make_float2(m, l);
      }
      __syncthreads();
      if (group == 0)
        for (int g = 0; g < G - 1; ++g) add(ml_s[MANY ? g * kGroup + me : 0], acc_s[MANY ? g * kGroup + me : 0]);
      __syncthreads();
    }
    if (!on || group > 0) continue;
    if (isnan(acc.x + acc.y + acc.z + acc.w)) {
      const int first = item.first / s.share;
      acc = tree_join_again(p, c0, c1, first, item.first > first * s.share ? 1 : 0, row, col4, D / 4, acc);
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const size_t at = static_cast<size_t>(item.unit) * p.rows + r;
    reinterpret_cast<uint2*>(p.out)[at * (D / 4) + col4] =
        make_uint2(Half16<T>::pack(acc.x * inv, acc.y * inv), Half16<T>::pack(acc.z * inv, acc.w * inv));
    if (col4 == 0 && p.lse2 != nullptr) p.lse2[at] = l == 0.f ? -INFINITY : m + lg2_approx(l);
  }
}

template <typename T, int D, int KEYS, bool PAIRS>
cudaError_t launch_join(const TreeParams& p, const TreePlan& plan, cudaStream_t stream) {
  if (plan.ctas == 1) return cudaSuccess;
  const long long items = static_cast<long long>(p.batch) * p.layers * p.hkv * plan.items;
  const bool by_border = items > plan.ctas - 1;
  const int rows = p.rows < plan.item_rows ? p.rows : plan.item_rows;
  // Many shares an item.  The join for few shares and the one for many, us: one node
  // over 16K rows, 2 items 32.5 and 11.1; 8 items 25.8 and 19.5; 16 items 32.1 and
  // 29.2; over 8K rows, 32 items 32.6 and 30.1, 64 items 51.0 and 53.8; 16 nodes
  // (148 CTAs), 8 items 30.4 and 29.7, 16 items 29.0 and 33.2, 32 items 38.8 and 49.1.
  const bool many = items * 16 <= plan.ctas;
  cudaLaunchConfig_t cfg = {};
  // blocks that are resident together, beside the main kernel's: six an SM
  const unsigned x = by_border ? plan.ctas - 1 : static_cast<unsigned>(items);
  const unsigned z = many ? D / 4 / kJoinCols : 1;
  const unsigned most = (6u * p.sms + x * z - 1) / (x * z), want = (rows + kJoinRows - 1) / kJoinRows;
  cfg.gridDim = dim3(x, want < most ? want : most, z);
  cfg.blockDim = dim3(kJoinRows * (many ? kJoinCols * kJoinGroups : D / 4));
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, tree_join_kernel<T, D, KEYS, PAIRS, true>, p, plan.item_rows, by_border)
              : cudaLaunchKernelEx(&cfg, tree_join_kernel<T, D, KEYS, PAIRS, false>, p, plan.item_rows, by_border);
}

template <typename T, int D, int NT, bool LOSES = false>
cudaError_t launch_nt(const CUtensorMap (&maps)[7], const TreeParams& p, const TreePlan& plan, cudaStream_t stream) {
  using C = TreeCfg<D, NT>;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(tree_kernel<T, D, NT, LOSES>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  tree_kernel<T, D, NT, LOSES><<<plan.ctas, kThreads, C::kSmemBytes, stream>>>(maps[0], maps[1], maps[2], maps[3], maps[5],
                                                                              maps[6], p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_d(const CUtensorMap (&maps)[7], const TreeParams& p, const TreePlan& plan, cudaStream_t stream) {
  cudaError_t e;
  if (plan.wide) {
    e = launch_tree_umma(std::is_same<T, __half>::value, D, maps, p, stream);
  } else {
    switch (plan.tile_rows) {
      case 8: e = launch_nt<T, D, 1>(maps, p, plan, stream); break;
      case 16: e = launch_nt<T, D, 2>(maps, p, plan, stream); break;
      default: e = launch_nt<T, D, 4>(maps, p, plan, stream); break;
    }
  }
  if (e != cudaSuccess || p.join_inside) return e;
  return plan.wide ? launch_join<T, D, 128, true>(p, plan, stream) : launch_join<T, D, kTreeKeys, false>(p, plan, stream);
}

// --------------------------------------------------------------------------
// visibility words
// --------------------------------------------------------------------------
// Thread = node: walk the parents up to the root, one bit a step.  A parent
// stands before its child, so the words are met from the last to the first
// and each is written once.  Latency bound: one shared-memory load a step.
__global__ void __launch_bounds__(128) tree_mask_kernel(const int* __restrict__ parents, const int* __restrict__ n_live,
                                                        int T, int words, uint32_t* __restrict__ mask,
                                                        int* __restrict__ depth) {
  __shared__ int parent_s[kTreeMaxNodes];
  const int b = blockIdx.x;
  int live = n_live != nullptr ? __ldg(n_live + b) : T;
  if (live < 0 || live > T) {
    if (threadIdx.x == 0 && blockIdx.y == 0) record_error(SPK_DEVERR_INDEX, b);
    live = live < 0 ? 0 : T;
  }
  const int i = blockIdx.y * blockDim.x + threadIdx.x;
  const int upto = min(live, static_cast<int>((blockIdx.y + 1) * blockDim.x));
  for (int x = threadIdx.x; x < upto; x += blockDim.x) {
    int q = __ldg(parents + static_cast<size_t>(b) * T + x);
    if (q < -1 || q >= x) {
      record_error(SPK_DEVERR_INDEX, b);
      q = -1;
    }
    parent_s[x] = q;
  }
  __syncthreads();
  if (i >= T) return;
  uint32_t* row = mask + (static_cast<size_t>(b) * T + i) * words;
  int steps = 0, at = words - 1;
  if (i < live) {
    uint32_t w = 0;
    int q = i;
    while (q >= 0) {
      while ((q >> 5) < at) {
        row[at--] = w;
        w = 0;
      }
      w |= 1u << (q & 31);
      q = parent_s[q];
      ++steps;
    }
    row[at--] = w;
    --steps;
  }
  while (at >= 0) row[at--] = 0;
  if (depth != nullptr) depth[static_cast<size_t>(b) * T + i] = steps;
}

}  // namespace

// Up to 32 rows a unit fit one narrow tile, which wastes less than a tile of
// 128 rows; above that the tcgen05 kernel.  Narrow and wide, us, of 8 KV heads:
//   rows a unit                        10         16         24         32         33         64
//   16 sequences of 4096 rows       52,  53    51,  53    66,  54    68,  55   124,  57   126,  58
//   one of 16,384 rows              21,  26    21,  26    26,  26    27,  26    43,  27    44,  30
//   64 layers over 320 rows         27,  41    28,  40    39,  40    41,  40    65,  41    69,  39
// (between 17 and 32 rows the wide kernel gains on long sequences in batches only)
TreePlan tree_plan(int rows, int head_dim, int sms) {
  TreePlan plan;
  plan.wide = rows > 32;
  plan.keys = plan.wide ? 128 : kTreeKeys;
  plan.tile_rows = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 128;
  plan.row_tiles = (rows + plan.tile_rows - 1) / plan.tile_rows;
  plan.item_rows = plan.wide && rows > 128 ? 256 : plan.tile_rows;
  plan.items = (rows + plan.item_rows - 1) / plan.item_rows;
  plan.ctas = plan.wide ? sms : 2 * sms;
  return plan;
}

size_t tree_ws_bytes(const TreePlan& plan, int head_dim) {
  return static_cast<size_t>(plan.ctas) * (2 * plan.item_rows * (head_dim + 2) * sizeof(float) + sizeof(long long));
}

cudaError_t launch_tree_attention(bool fp16, int head_dim, const CUtensorMap (&maps)[7], const TreeParams& p,
                                  const TreePlan& plan, cudaStream_t stream) {
  if (head_dim == 128)
    return fp16 ? launch_d<__half, 128>(maps, p, plan, stream) : launch_d<__nv_bfloat16, 128>(maps, p, plan, stream);
  if (head_dim == 64)
    return fp16 ? launch_d<__half, 64>(maps, p, plan, stream) : launch_d<__nv_bfloat16, 64>(maps, p, plan, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_tree_loses(const CUtensorMap (&maps)[7], const TreeParams& p, const TreePlan& plan, cudaStream_t stream) {
  return plan.wide ? launch_tree_umma_loses(maps, p, stream) : launch_nt<__nv_bfloat16, 64, 1, true>(maps, p, plan, stream);
}

cudaError_t launch_tree_mask(const int* parents, const int* n_live, int batch, int T, uint32_t* mask, int* depth,
                             cudaStream_t stream) {
  tree_mask_kernel<<<dim3(batch, (T + 127) / 128), 128, 0, stream>>>(parents, n_live, T, (T + 31) / 32, mask, depth);
  return cudaGetLastError();
}

}  // namespace spk

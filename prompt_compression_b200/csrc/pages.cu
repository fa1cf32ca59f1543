// pages.cu -- the pages of a KV cache: reserving, forking and freeing them,
// writing rows into them, and compacting a sequence to the rows that the
// selection kept.
//
// Bookkeeping (page table, lengths, reference counts) lives on the device and
// every change is made there, so a decoding loop never waits for the host and
// can be captured.  One CTA makes a change, or a cluster of eight where the
// tables are large (a cluster's barriers cost more than the loads of a small
// table); pages are taken lowest number first, and counts change by integer
// additions, so the result does not depend on timing.  A call that cannot be
// carried out (too few free pages, a bad argument) leaves everything as it was
// and says so in *result.  Latency bound: a chain of dependent loads.
// Rows are copied as bytes, 16 at a time per thread: bound by HBM bandwidth.
#include "common.cuh"
#include "paged.cuh"

namespace spk {

SPK_ERROR_READER(device_errors_pages)

namespace {

constexpr int kBookThreads = 512;
constexpr int kBadCall = -1;

// CTAS: 1, or the CTAs of the cluster.
template <int CTAS>
__device__ __forceinline__ int book_rank() {
  return CTAS == 1 ? 0 : static_cast<int>(cluster_ctarank());
}
template <int CTAS>
__device__ __forceinline__ void book_sync() {
  if (CTAS == 1)
    __syncthreads();
  else
    cluster_sync();
}

// Workspace of a call over n sequences: [n][max_pages] page numbers, then
// [n][4] words a sequence.
__host__ __device__ __forceinline__ int* ws_words(void* ws, int n, int max_pages) {
  return static_cast<int*>(ws) + ((static_cast<size_t>(n) * max_pages + 3) & ~size_t(3));
}

// The rows' kernel starts while the bookkeeping's runs, and waits for its end.
// What the bookkeeping leaves for it (words, old) comes by plain pointers:
// `const __restrict__` says that nobody writes the data while the kernel runs,
// and lets the compiler load it from the non-coherent cache or above the wait.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// The sum of one value a thread over the CTA, for every thread.
__device__ __forceinline__ int block_sum(int v, int* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kBookThreads / 32; ++w) s += scratch[w];
  return s;
}

// Exclusive prefix sums of x[0..n) in shared memory, by one warp; x[n] = total.
__device__ __forceinline__ void warp_exclusive(int* x, int n) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int v = i < n ? x[i] : 0;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    if (i < n) x[i] = base + s - v;
    base += __shfl_sync(0xffffffffu, s, 31);
  }
  if (lane == 0) x[n] = base;
}

// The free pages (reference count 0) of the whole pool, and before this CTA's
// part of it; every CTA of the cluster calls it.
struct FreePages {
  int all, before;
};
template <int CTAS>
__device__ __forceinline__ FreePages count_free(const int* refs, int n_pages, int* scratch, int* mine_s) {
  const int rank = book_rank<CTAS>();
  const int part = ceil_div(n_pages, CTAS);
  const int lo = min(n_pages, rank * part), hi = min(n_pages, lo + part);
  int c = 0;
  for (int i = lo + threadIdx.x; i < hi; i += kBookThreads) c += refs[i] == 0;
  c = block_sum(c, scratch);
  if (CTAS == 1) return {c, 0};
  if (threadIdx.x == 0) *mine_s = c;
  cluster_sync();
  FreePages f{0, 0};
  for (int r = 0; r < CTAS; ++r) {
    const int v = static_cast<int>(dsmem_ld(dsmem_addr(smem_u32(mine_s), r)));
    f.all += v;
    if (r < rank) f.before += v;
  }
  cluster_sync();            // nobody leaves (or reuses mine_s) while it is read
  return f;
}

// take(rank, page) for the first `want` free pages, in ascending order: each
// gets the count 1 and is handed out by the thread that found it.
template <int CTAS, typename F>
__device__ __forceinline__ void take_free(int* refs, int n_pages, int before, int want, int* scratch, F take) {
  const int part = ceil_div(n_pages, CTAS);
  const int lo = min(n_pages, book_rank<CTAS>() * part), hi = min(n_pages, lo + part);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int rank0 = before;
  for (int i0 = lo; i0 < hi && rank0 < want; i0 += kBookThreads) {
    const int i = i0 + threadIdx.x;
    const bool is_free = i < hi && refs[i] == 0;
    const uint32_t votes = __ballot_sync(0xffffffffu, is_free);
    __syncthreads();
    if (lane == 0) scratch[warp] = __popc(votes);
    __syncthreads();
    int rank = rank0 + __popc(votes & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kBookThreads / 32; ++w) {
      if (w < warp) rank += scratch[w];
      rank0 += scratch[w];
    }
    if (is_free && rank < want) {
      refs[i] = 1;
      take(rank, i);
    }
  }
}

// Whether an entry of list[0..n) is outside [0, n_seqs) or stands twice.
__device__ __forceinline__ bool bad_list(const int* list_s, int n, int n_seqs, bool unique) {
  bool bad = false;
  for (int i = threadIdx.x; i < n; i += kBookThreads) {
    const int s = list_s[i];
    bad |= s < 0 || s >= n_seqs;
    if (unique)
      for (int j = 0; j < i; ++j) bad |= list_s[j] == s;
  }
  return bad;
}

template <int CTAS>
__device__ __forceinline__ void refuse(int* result) {
  if (book_rank<CTAS>() == 0 && threadIdx.x == 0) {
    record_error(SPK_DEVERR_INDEX, 700);
    *result = kBadCall;
  }
}

// --------------------------------------------------------------------------
// reserve
// --------------------------------------------------------------------------
// Sequence i grows by n_new[i] rows: pages for the rows that have none, and a
// page of its own for a partially filled last page that other sequences hold
// too (its rows are copied by copy_tail_kernel, from the words left here:
// {from, to or -1, rows}).  The sequences leave a shared page in the list's
// order; the last holder keeps it.
template <int CTAS>
__global__ void __launch_bounds__(kBookThreads)
    reserve_kernel(PagesShape s, PagesBook b, const int* __restrict__ seqs, const int* __restrict__ n_new, int n,
                   int* __restrict__ result, int* __restrict__ words) {
  launch_next();
  __shared__ int seq_s[kPagesMaxCall], first_s[kPagesMaxCall + 1], tail_s[kPagesMaxCall];
  __shared__ int scratch[kBookThreads / 32], mine_s;
  for (int i = threadIdx.x; i < n; i += kBookThreads) seq_s[i] = seqs[i];
  __syncthreads();
  bool bad = bad_list(seq_s, n, s.n_seqs, true);
  const long long most = static_cast<long long>(s.max_pages) * s.page_rows;
  for (int i = threadIdx.x; i < n; i += kBookThreads) {
    int tail = -1;
    if (seq_s[i] >= 0 && seq_s[i] < s.n_seqs) {
      const int len = b.lens[seq_s[i]], more = n_new[i];
      if (len < 0 || more < 0 || static_cast<long long>(len) + more > most) {
        bad = true;
      } else if (more > 0 && len % s.page_rows != 0) {
        tail = b.table[static_cast<size_t>(seq_s[i]) * s.max_pages + len / s.page_rows];
        bad |= tail < 0 || tail >= s.n_pages;
      }
    }
    tail_s[i] = tail;
  }
  if (__syncthreads_or(bad)) {      // every CTA finds the same
    refuse<CTAS>(result);
    for (int i = threadIdx.x; i < n; i += kBookThreads)
      if (book_rank<CTAS>() == 0) words[4 * i + 1] = -1;
    return;
  }
  for (int i = threadIdx.x; i < n; i += kBookThreads) {
    const int len = b.lens[seq_s[i]];
    int want = ceil_div(len + n_new[i], s.page_rows) - ceil_div(len, s.page_rows);
    if (tail_s[i] >= 0) {
      int holders = b.refs[tail_s[i]];
      for (int j = 0; j < i; ++j) holders -= tail_s[j] == tail_s[i];
      if (holders > 1) want |= 1 << 30;
    }
    first_s[i] = want;
  }
  __syncthreads();
  // tail_s: from now on only where the page is copied
  for (int i = threadIdx.x; i < n; i += kBookThreads) {
    const bool copy = (first_s[i] >> 30) & 1;
    if (!copy) tail_s[i] = -1;
    first_s[i] = (first_s[i] & ~(1 << 30)) + (copy ? 1 : 0);
  }
  __syncthreads();
  if (threadIdx.x < 32) warp_exclusive(first_s, n);
  __syncthreads();
  const int want = first_s[n];
  const FreePages f = count_free<CTAS>(b.refs, s.n_pages, scratch, &mine_s);   // orders the reads above before the changes
  const bool first_cta = book_rank<CTAS>() == 0;
  if (f.all < want) {
    if (first_cta) {
      if (threadIdx.x == 0) *result = want - f.all;
      for (int i = threadIdx.x; i < n; i += kBookThreads) words[4 * i + 1] = -1;
    }
    return;
  }
  take_free<CTAS>(b.refs, s.n_pages, f.before, want, scratch, [&](int rank, int page) {
    int lo = 0, hi = n;                       // the sequence whose pages hold this rank
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first_s[mid] <= rank) lo = mid; else hi = mid;
    }
    const int len = b.lens[seq_s[lo]];
    int at = rank - first_s[lo];
    int* row = b.table + static_cast<size_t>(seq_s[lo]) * s.max_pages;
    if (tail_s[lo] >= 0) {
      if (at == 0) {
        row[len / s.page_rows] = page;
        words[4 * lo] = tail_s[lo];
        words[4 * lo + 1] = page;
        words[4 * lo + 2] = len % s.page_rows;
        return;
      }
      --at;
    }
    row[ceil_div(len, s.page_rows) + at] = page;
  });
  book_sync<CTAS>();                             // lens and the tails' counts have been read
  if (!first_cta) return;
  for (int i = threadIdx.x; i < n; i += kBookThreads) {
    b.lens[seq_s[i]] += n_new[i];
    if (tail_s[i] >= 0)
      atomicSub(b.refs + tail_s[i], 1);
    else
      words[4 * i + 1] = -1;
  }
  if (threadIdx.x == 0) *result = 0;
}

// Block (i, y): rows 0 .. rows-1 of the copied page of sequence i, for the
// (layer, KV head) blocks y, y + gridDim.y, ... of K and V.
__global__ void __launch_bounds__(256)
    copy_tail_kernel(PagesShape s, const int* words, uint4* __restrict__ k, uint4* __restrict__ v) {
  wait_for_previous();
  const int from = words[4 * blockIdx.x], to = words[4 * blockIdx.x + 1];
  if (to < 0) return;
  const int vecs = words[4 * blockIdx.x + 2] * s.row_vecs;
  const size_t block = static_cast<size_t>(s.page_rows) * s.row_vecs;
  for (int lh = blockIdx.y; lh < s.layers * s.hkv; lh += gridDim.y) {
    const int l = lh / s.hkv, h = lh - l * s.hkv;
    const size_t src = ((static_cast<size_t>(l) * s.n_pages + from) * s.hkv + h) * block;
    const size_t dst = ((static_cast<size_t>(l) * s.n_pages + to) * s.hkv + h) * block;
    for (int x = threadIdx.x; x < vecs; x += blockDim.x) {
      k[dst + x] = k[src + x];
      v[dst + x] = v[src + x];
    }
  }
}

// --------------------------------------------------------------------------
// fork
// --------------------------------------------------------------------------
// Sequence dst[i] becomes the first n_rows[i] rows (all of them where n_rows
// is null) that src[i] had before the call, by holding their pages; what
// dst[i] held is released.  The sources' rows of the table are copied first,
// so a sequence may be a source and a destination.
template <int CTAS>
__global__ void __launch_bounds__(kBookThreads)
    fork_kernel(PagesShape s, PagesBook b, const int* __restrict__ src, const int* __restrict__ dst,
                const int* __restrict__ n_rows, int n, int* __restrict__ result, int* __restrict__ old) {
  __shared__ int src_s[kPagesMaxCall], dst_s[kPagesMaxCall], len_s[kPagesMaxCall];
  for (int i = threadIdx.x; i < n; i += kBookThreads) {
    src_s[i] = src[i];
    dst_s[i] = dst[i];
  }
  __syncthreads();
  bool bad = bad_list(src_s, n, s.n_seqs, false) | bad_list(dst_s, n, s.n_seqs, true);
  for (int i = threadIdx.x; i < n; i += kBookThreads) {
    int len = 0;
    if (src_s[i] >= 0 && src_s[i] < s.n_seqs) {
      len = b.lens[src_s[i]];
      bad |= len < 0 || len > static_cast<long long>(s.max_pages) * s.page_rows;
      if (n_rows != nullptr) {
        bad |= n_rows[i] < 0;
        len = min(len, n_rows[i]);
      }
    }
    len_s[i] = len;
  }
  if (__syncthreads_or(bad)) {
    refuse<CTAS>(result);
    return;
  }
  const size_t cells = static_cast<size_t>(n) * s.max_pages;
  const size_t me = static_cast<size_t>(book_rank<CTAS>()) * kBookThreads + threadIdx.x;
  for (size_t x = me; x < cells; x += CTAS * kBookThreads) {
    const int i = static_cast<int>(x / s.max_pages), at = static_cast<int>(x % s.max_pages);
    int page = at < ceil_div(len_s[i], s.page_rows) ? b.table[static_cast<size_t>(src_s[i]) * s.max_pages + at] : -1;
    if (page < 0 || page >= s.n_pages) page = -1;
    old[x] = page;
    if (page >= 0) atomicAdd(b.refs + page, 1);
  }
  book_sync<CTAS>();
  for (size_t x = me; x < cells; x += CTAS * kBookThreads) {
    const int i = static_cast<int>(x / s.max_pages), at = static_cast<int>(x % s.max_pages);
    int* cell = b.table + static_cast<size_t>(dst_s[i]) * s.max_pages + at;
    const int gone = *cell;
    if (gone >= 0 && gone < s.n_pages) atomicSub(b.refs + gone, 1);
    *cell = old[x];
  }
  if (book_rank<CTAS>() == 0) {
    for (int i = threadIdx.x; i < n; i += kBookThreads) b.lens[dst_s[i]] = len_s[i];
    if (threadIdx.x == 0) *result = 0;
  }
}

// --------------------------------------------------------------------------
// free
// --------------------------------------------------------------------------
// A page is released by the thread that took its cell out of the table, so a
// sequence may stand in the list twice.
__global__ void __launch_bounds__(256)
    free_kernel(PagesShape s, PagesBook b, const int* __restrict__ seqs, const int* __restrict__ keep_rows) {
  const int i = blockIdx.x;
  const int seq = seqs[i], keep = keep_rows != nullptr ? keep_rows[i] : 0;
  if (seq < 0 || seq >= s.n_seqs || keep < 0) {
    if (blockIdx.y == 0 && threadIdx.x == 0) record_error(SPK_DEVERR_INDEX, 701);
    return;
  }
  for (int at = ceil_div(keep, s.page_rows) + blockIdx.y * blockDim.x + threadIdx.x; at < s.max_pages;
       at += gridDim.y * blockDim.x) {
    const int page = atomicExch(b.table + static_cast<size_t>(seq) * s.max_pages + at, -1);
    if (page >= 0 && page < s.n_pages) atomicSub(b.refs + page, 1);
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) atomicMin(b.lens + seq, keep);
}

// --------------------------------------------------------------------------
// compact
// --------------------------------------------------------------------------
// The table's side of compacting src[i] to dst[i] (n_idx rows each): the
// sources' pages are held while what the destinations held is released and
// new pages are taken, so a destination's old pages can be used again unless
// a source of this call needs them (dst[i] == src[i]: compacting in place).
// Leaves the sources' rows of the table in `old` and their lengths (or -1:
// nothing to copy) in words[4 i].
template <int CTAS>
__global__ void __launch_bounds__(kBookThreads)
    compact_book_kernel(PagesShape s, PagesBook b, const int* __restrict__ src, const int* __restrict__ dst, int n,
                        int n_idx, int* __restrict__ result, int* __restrict__ old, int* __restrict__ words) {
  launch_next();
  __shared__ int src_s[kPagesMaxCall], dst_s[kPagesMaxCall];
  __shared__ int scratch[kBookThreads / 32], mine_s;
  for (int i = threadIdx.x; i < n; i += kBookThreads) {
    src_s[i] = src[i];
    dst_s[i] = dst[i];
  }
  __syncthreads();
  bool bad = bad_list(src_s, n, s.n_seqs, false) | bad_list(dst_s, n, s.n_seqs, true);
  for (int i = threadIdx.x; i < n; i += kBookThreads) {
    if (src_s[i] < 0 || src_s[i] >= s.n_seqs) continue;
    const int len = b.lens[src_s[i]];           // the rows' kernel finds pages by it
    bad |= len < 0 || len > static_cast<long long>(s.max_pages) * s.page_rows;
  }
  const bool first_cta = book_rank<CTAS>() == 0;
  if (__syncthreads_or(bad)) {
    refuse<CTAS>(result);
    if (first_cta)
      for (int i = threadIdx.x; i < n; i += kBookThreads) words[4 * i] = -1;
    return;
  }
  const int per = ceil_div(n_idx, s.page_rows);
  const size_t cells = static_cast<size_t>(n) * s.max_pages;
  const size_t me = static_cast<size_t>(book_rank<CTAS>()) * kBookThreads + threadIdx.x;
  for (size_t x = me; x < cells; x += CTAS * kBookThreads) {      // hold the sources
    const int i = static_cast<int>(x / s.max_pages), at = static_cast<int>(x % s.max_pages);
    int page = b.table[static_cast<size_t>(src_s[i]) * s.max_pages + at];
    if (page < 0 || page >= s.n_pages) page = -1;
    old[x] = page;
    if (page >= 0) atomicAdd(b.refs + page, 1);
  }
  for (size_t x = me; x < cells; x += CTAS * kBookThreads) {      // release the destinations
    const int i = static_cast<int>(x / s.max_pages), at = static_cast<int>(x % s.max_pages);
    const int page = b.table[static_cast<size_t>(dst_s[i]) * s.max_pages + at];
    if (page >= 0 && page < s.n_pages) atomicSub(b.refs + page, 1);
  }
  book_sync<CTAS>();
  const int want = n * per;
  const FreePages f = count_free<CTAS>(b.refs, s.n_pages, scratch, &mine_s);
  const bool done = f.all >= want;
  if (done)
    take_free<CTAS>(b.refs, s.n_pages, f.before, want, scratch, [&](int rank, int page) {
      b.table[static_cast<size_t>(dst_s[rank / per]) * s.max_pages + rank % per] = page;
    });
  book_sync<CTAS>();
  for (size_t x = me; x < cells; x += CTAS * kBookThreads) {
    const int i = static_cast<int>(x / s.max_pages), at = static_cast<int>(x % s.max_pages);
    if (old[x] >= 0) atomicSub(b.refs + old[x], 1);
    int* cell = b.table + static_cast<size_t>(dst_s[i]) * s.max_pages + at;
    if (done) {
      if (at >= per) *cell = -1;
    } else {                                           // as it was
      const int page = *cell;
      if (page >= 0 && page < s.n_pages) atomicAdd(b.refs + page, 1);
    }
  }
  if (first_cta) {
    for (int i = threadIdx.x; i < n; i += kBookThreads) words[4 * i] = done ? b.lens[src_s[i]] : -1;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kBookThreads)
      if (done) b.lens[dst_s[i]] = n_idx;
    if (threadIdx.x == 0) *result = done ? 0 : want - f.all;
  }
}

// Rows of one unit in blocks of kCopyRows: the block finds where each row comes
// from and goes to once (vectors, in shared memory; -1: not copied), then its
// threads move 16 bytes of K and of V each, four of either in flight.
// (2048 rows a unit, 128 units, 269 MB read and written: 45 us, 6.0 TB/s; with
// the three dependent loads in front of every vector it was 60 us.)
constexpr int kCopyRows = 64;

__device__ __forceinline__ void copy_rows(const long long* from_s, const long long* to_s, int rows, int row_vecs,
                                          const uint4* __restrict__ k, const uint4* __restrict__ v,
                                          uint4* __restrict__ kd, uint4* __restrict__ vd) {
  const int total = rows * row_vecs;
  for (int e0 = threadIdx.x; e0 < total; e0 += 4 * blockDim.x) {
    uint4 a[4], b[4];
    long long to[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = e0 + u * blockDim.x;
      to[u] = -1;
      if (e < total) {
        const int row = e / row_vecs, vec = e - row * row_vecs;
        const long long from = from_s[row];
        if (from >= 0) {
          to[u] = to_s[row] + vec;
          a[u] = __ldcs(k + from + vec);
          b[u] = __ldcs(v + from + vec);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (to[u] >= 0) {
        kd[to[u]] = a[u];
        vd[to[u]] = b[u];
      }
    }
  }
}

// Vector of the pools at which row `row` of page `page` lies, for unit lh = (layer, KV head).
__device__ __forceinline__ long long pool_row(const PagesShape& s, int lh, int page, int row) {
  const int l = lh / s.hkv, h = lh - l * s.hkv;
  return (((static_cast<long long>(l) * s.n_pages + page) * s.hkv + h) * s.page_rows + row) * s.row_vecs;
}

// Block: rows c * kCopyRows .. of one (layer, KV head) of dst[i], from the pages
// that src[i] had (`old`).
__global__ void __launch_bounds__(256)
    compact_rows_kernel(PagesShape s, PagesBook b, const int* __restrict__ dst, int n_idx, const int* __restrict__ idx,
                        int units_per_idx, const int* old, const int* words, uint4* k, uint4* v) {
  __shared__ long long from_s[kCopyRows], to_s[kCopyRows];
  const int chunks = (n_idx + kCopyRows - 1) / kCopyRows;
  const int lh_all = s.layers * s.hkv;
  const size_t u = blockIdx.x / chunks;
  const int t0 = static_cast<int>(blockIdx.x - u * chunks) * kCopyRows, rows = min(kCopyRows, n_idx - t0);
  const int i = static_cast<int>(u / lh_all), lh = static_cast<int>(u - static_cast<size_t>(i) * lh_all);
  int from = -1;
  if (threadIdx.x < rows) from = __ldg(idx + (u / units_per_idx) * n_idx + t0 + threadIdx.x);
  wait_for_previous();
  const int len = words[4 * i];
  if (len < 0) return;                          // refused
  if (threadIdx.x < rows) {
    const int t = t0 + threadIdx.x;
    const int page = from >= 0 && from < len ? old[static_cast<size_t>(i) * s.max_pages + from / s.page_rows] : -1;
    if (page < 0) record_error(SPK_DEVERR_INDEX, static_cast<int>(u));
    const int to = b.table[static_cast<size_t>(dst[i]) * s.max_pages + t / s.page_rows];
    from_s[threadIdx.x] = page < 0 ? -1 : pool_row(s, lh, page, from % s.page_rows);
    to_s[threadIdx.x] = pool_row(s, lh, to, t % s.page_rows);
  }
  __syncthreads();
  copy_rows(from_s, to_s, rows, s.row_vecs, k, v, k, v);
}

// --------------------------------------------------------------------------
// write
// --------------------------------------------------------------------------
// Block: kCopyRows of the rows (i, layer, KV head, t), in that order.  Row
// t < counts[i] goes to row lens[seq] - counts[i] + t of sequence seqs[i].  A
// page that other sequences hold too is not written, nor a sequence that an
// earlier entry names, nor anything where room was missing (*reserved).  (A 16K prompt, 32 layers x 8 KV heads, 4.3 GB read and
// written: 631 us, 6.8 TB/s.)
__global__ void __launch_bounds__(256)
    write_kernel(PagesShape s, PagesBook b, const uint4* __restrict__ k, const uint4* __restrict__ v, int n_src,
                 const int* __restrict__ idx, int n_idx, int units_per_idx, const int* __restrict__ counts,
                 const int* __restrict__ seqs, int n, uint4* __restrict__ kp, uint4* __restrict__ vp, const int* __restrict__ reserved) {
  __shared__ long long from_s[kCopyRows], to_s[kCopyRows];
  const int lh_all = s.layers * s.hkv;
  const long long all = static_cast<long long>(n) * lh_all * n_idx;
  const long long f0 = static_cast<long long>(blockIdx.x) * kCopyRows;
  const int rows = static_cast<int>(min(static_cast<long long>(kCopyRows), all - f0));
  const long long per = static_cast<long long>(lh_all) * n_idx;      // rows of an entry
  const bool room = reserved == nullptr || *reserved == 0;
  long long from = -1, to = -1;
  int mine = -1;
  if (threadIdx.x < rows) {
    const long long f = f0 + threadIdx.x, u = f / n_idx;
    const int t = static_cast<int>(f - u * n_idx), i = static_cast<int>(u / lh_all);
    mine = i;
    const int count = counts != nullptr ? __ldg(counts + i) : n_idx, seq = __ldg(seqs + i);
    bool ok = seq >= 0 && seq < s.n_seqs && count >= 0 && count <= n_idx;
    if (!ok || t < count) {
      const int src = idx != nullptr ? __ldg(idx + (u / units_per_idx) * n_idx + t) : t;
      const int pos = ok ? b.lens[seq] - count + t : -1;
      ok = pos >= 0 && pos < static_cast<long long>(s.max_pages) * s.page_rows && src >= 0 && src < n_src;
      const int page = ok ? b.table[static_cast<size_t>(seq) * s.max_pages + pos / s.page_rows] : -1;
      ok = ok && page >= 0 && page < s.n_pages && b.refs[page] == 1;
      if (ok) {
        from = (u * n_src + src) * s.row_vecs;
        to = pool_row(s, static_cast<int>(u - static_cast<long long>(i) * lh_all), page, pos % s.page_rows);
      } else if (room) {
        record_error(SPK_DEVERR_INDEX, static_cast<int>(u));
      }
    }
  }
  if (!room) return;
  for (int i = static_cast<int>(f0 / per); i <= static_cast<int>((f0 + rows - 1) / per); ++i) {
    bool twice = false;
    for (int j = threadIdx.x; j < i; j += blockDim.x) twice |= __ldg(seqs + j) == __ldg(seqs + i);
    if (__syncthreads_or(twice)) {
      if (mine == i) from = -1;
      if (threadIdx.x == 0) record_error(SPK_DEVERR_INDEX, i);
    }
  }
  if (threadIdx.x < rows) {
    from_s[threadIdx.x] = from;
    to_s[threadIdx.x] = to;
  }
  __syncthreads();
  copy_rows(from_s, to_s, rows, s.row_vecs, k, v, kp, vp);
}

// One CTA, or a cluster of eight for large tables.  One and eight, us: reserve and
// free of 32 sequences, 2048 pages 7.8 and 8.9, 8192 pages 9.8 and 8.9, 16,384
// pages 13.4 and 9.6; fork and compact of 1024 cells 4.6 and 4.3, 9.3 and 10.1, of
// 2048 cells 6.1 and 4.3, 11.7 and 10.6, of 4096 cells 9.5 and 4.4, 17.6 and 11.0.
template <typename K, typename... A>
cudaError_t launch_book(K one, K eight, const PagesShape& s, int n, bool tables, cudaStream_t stream, A... args) {
  const long long cells = static_cast<long long>(n) * s.max_pages;
  const bool big = s.n_pages > 8192 || (tables && cells > 2048);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(big ? 8 : 1);
  cfg.blockDim = dim3(kBookThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 8;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = big ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, big ? eight : one, args...);
}

// A kernel that starts under the one before it (wait_for_previous).
template <typename... P, typename... A>
cudaError_t launch_under(void (*kernel)(P...), dim3 grid, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace

size_t pages_ws_bytes(int n, int max_pages) {
  return (((static_cast<size_t>(n) * max_pages + 3) & ~size_t(3)) + static_cast<size_t>(n) * 4) * sizeof(int);
}

cudaError_t launch_pages_reserve(const PagesShape& s, const PagesBook& b, void* k_pages, void* v_pages,
                                 const int* seqs, const int* n_new, int n, int* result, void* ws,
                                 cudaStream_t stream) {
  int* words = ws_words(ws, n, s.max_pages);
  cudaError_t e = launch_book(reserve_kernel<1>, reserve_kernel<8>, s, n, false, stream, s, b, seqs, n_new, n, result, words);
  if (e != cudaSuccess || n == 0) return e;
  const int lh = s.layers * s.hkv;
  return launch_under(copy_tail_kernel, dim3(n, lh < 1024 ? lh : 1024), stream, s, words, k_pages, v_pages);
}

cudaError_t launch_pages_fork(const PagesShape& s, const PagesBook& b, const int* src, const int* dst,
                              const int* n_rows, int n, int* result, void* ws, cudaStream_t stream) {
  return launch_book(fork_kernel<1>, fork_kernel<8>, s, n, true, stream, s, b, src, dst, n_rows, n, result,
                     static_cast<int*>(ws));
}

cudaError_t launch_pages_free(const PagesShape& s, const PagesBook& b, const int* seqs, const int* keep_rows, int n,
                              cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  const int y = (s.max_pages + 255) / 256;
  free_kernel<<<dim3(n, y < 16 ? y : 16), 256, 0, stream>>>(s, b, seqs, keep_rows);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PagesShape& s, const PagesBook& b, void* k_pages, void* v_pages,
                                 const int* src, const int* dst, int n, const int* idx, int n_idx,
                                 int units_per_idx, int* result, void* ws, cudaStream_t stream) {
  int* old = static_cast<int*>(ws);
  int* words = ws_words(ws, n, s.max_pages);
  cudaError_t e = launch_book(compact_book_kernel<1>, compact_book_kernel<8>, s, n, true, stream, s, b, src, dst, n, n_idx,
                              result, old, words);
  const long long blocks = static_cast<long long>(n) * s.layers * s.hkv * ((n_idx + kCopyRows - 1) / kCopyRows);
  if (e != cudaSuccess || blocks == 0) return e;
  return launch_under(compact_rows_kernel, dim3(static_cast<unsigned>(blocks)), stream, s, b, dst, n_idx, idx, units_per_idx,
                      old, words, k_pages, v_pages);
}

cudaError_t launch_pages_write(const PagesShape& s, const PagesBook& b, const void* k, const void* v, int n_src,
                               const int* idx, int n_idx, int units_per_idx, const int* counts, const int* seqs,
                               int n, void* k_pages, void* v_pages, const int* reserved, cudaStream_t stream) {
  const long long rows = static_cast<long long>(n) * s.layers * s.hkv * n_idx;
  if (rows == 0) return cudaSuccess;
  write_kernel<<<static_cast<unsigned>((rows + kCopyRows - 1) / kCopyRows), 256, 0, stream>>>(
      s, b, static_cast<const uint4*>(k), static_cast<const uint4*>(v), n_src, idx, n_idx, units_per_idx, counts, seqs, n,
      static_cast<uint4*>(k_pages), static_cast<uint4*>(v_pages), reserved);
  return cudaGetLastError();
}

}  // namespace spk

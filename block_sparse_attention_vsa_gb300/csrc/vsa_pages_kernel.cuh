// vsa_pages_kernel.cuh -- the pages of the 8-bit cache: mapping them ahead of a write, letting
// them go, forking sequences that share them, and closing up a pool.
//
// A pool's state is refs[p], the table entries that name page p, and a bitmap of the pages that
// none names.  Taking always the lowest free page makes every outcome unique: counts change by
// integer atomics, whose order does not matter, and the r-th page asked for is the r-th set bit
// of the bitmap, found by counting.  A whole pool's bitmap is small (a pool of 100,000 pages:
// 12.5 KB), so every CTA counts all of it for itself, and only the rows of the tables (or the
// pages) are divided among them.  Where the bitmap is changed as well the CTAs are one cluster,
// whose barrier tells that all have read it.
//
// Launched with programmatic serialization, like the other serving kernels: everything is read
// by ordinary loads behind the wait for the predecessor.
#pragma once

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "vsa_warp_ptx.cuh"

namespace vsa {

constexpr int kPagesThreads = 1024;  // of a CTA that counts
constexpr int kPagesCluster = 8;
constexpr int kEntries = 8;  // table entries a lane has under way at a time
constexpr int kFew = 4;      // blocks of a row that one lane looks after

struct Pool {
  int32_t* refs;
  uint32_t* free;
  int pages;
};

__device__ __forceinline__ bool is_page(int p, int pages) { return p >= 0 && p < pages; }

// Blocks that `tokens` tokens fill or begin, max_blocks at most.
__device__ __forceinline__ int blocks_of(long long tokens, int block, int max_blocks) {
  const long long n = tokens <= 0 ? 0 : (tokens + block - 1) / block;
  return n < max_blocks ? (int)n : max_blocks;
}

// The word w of the bitmap; bits past the pool count as not free.
__device__ __forceinline__ uint32_t free_word(const Pool& p, long long w) {
  const uint32_t x = read_global(p.free + w);
  const long long left = p.pages - w * 32;
  return left >= 32 ? x : x & ((1u << left) - 1u);
}

// The position of the n-th (from 0) set bit; there is one.
__device__ __forceinline__ int nth_bit(uint32_t x, int n) {
  int at = 0;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const int c = __popc(x & ((1u << s) - 1u));
    if (n >= c) {
      n -= c;
      x >>= s;
      at += s;
    }
  }
  return at;
}

// Sum over the CTA's threads before this one; *total of all.  s_warp [33] is scratch.
__device__ __forceinline__ int block_before(int x, int* s_warp, int* total) {
  const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
  int sum = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) s_warp[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    const int n = (int)blockDim.x >> 5;
    const int t = lane < n ? s_warp[lane] : 0;
    int run = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    s_warp[lane] = run - t;
    if (lane == 31) s_warp[32] = run;
  }
  __syncthreads();
  const int before = s_warp[warp] + sum - x;
  *total = s_warp[32];
  __syncthreads();
  return before;
}

// Free pages counted: thread t of the CTA has the words [t * per, (t + 1) * per), and
// before[t] free pages come before them (before[kPagesThreads]: all).
struct FreeCount {
  int* before;
  long long words;
  int per, total;
};
__device__ __forceinline__ FreeCount count_free(const Pool& p, int* s_before, int* s_warp) {
  FreeCount f;
  f.before = s_before;
  f.words = ((long long)p.pages + 31) / 32;
  f.per = (int)((f.words + kPagesThreads - 1) / kPagesThreads);
  const long long w0 = (long long)threadIdx.x * f.per;
  int n = 0;
#pragma unroll 4
  for (int i = 0; i < f.per; ++i)
    if (w0 + i < f.words) n += __popc(free_word(p, w0 + i));
  s_before[threadIdx.x] = block_before(n, s_warp, &f.total);
  if (threadIdx.x == 0) s_before[kPagesThreads] = f.total;
  __syncthreads();
  return f;
}
// The r-th free page; -1 where there are not as many.
__device__ __forceinline__ int nth_free(const Pool& p, const FreeCount& f, int r) {
  int lo = 0;
#pragma unroll
  for (int s = kPagesThreads / 2; s > 0; s >>= 1)
    if (f.before[lo + s] <= r) lo += s;
  int left = r - f.before[lo];
  for (long long w = (long long)lo * f.per; w < f.words; ++w) {
    const uint32_t x = free_word(p, w);
    const int n = __popc(x);
    if (left < n) return (int)(w * 32) + nth_bit(x, left);
    left -= n;
  }
  return -1;
}
// Consecutive free pages for a warp: those of 16 words of the bitmap, half a word a lane, written
// out in their order, so that looking one up is a load.  (Searching the words' counts and then the
// bits of one: 16 prompts of 50,000 tokens in 18.7 us, written out 14.7.)
constexpr int kWindowWords = 16;
struct FreeWindow {
  const Pool& p;
  const FreeCount& f;
  uint16_t* list;        // [32 * kWindowWords] of the warp: pages behind the window's first
  long long w0 = 0;      // first word
  int base = 0, end = 0; // free pages before the window; before it and in it

  // (places that lanes write, or read, together lie in different banks)
  static __device__ __forceinline__ int place(int i) { return i ^ ((i >> 6 & 7) << 1); }
  __device__ __forceinline__ void load() {
    const int lane = (int)threadIdx.x & 31;
    const long long w = w0 + (lane >> 1);
    uint32_t x = w < f.words ? free_word(p, w) : 0u;
    x = lane & 1 ? x >> 16 : x & 0xffffu;
    int at = __popc(x);
    const int mine = at;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    end = base + __shfl_sync(0xffffffffu, at, 31);
    __syncwarp();  // (the list has been read)
    for (at -= mine; x != 0; x &= x - 1)
      list[place(at++)] = (uint16_t)(16 * lane + __ffs((int)x) - 1);
    __syncwarp();
  }
  // places the window on the r-th free page's thread
  __device__ __forceinline__ void seek(int r) {
    int lo = 0;
#pragma unroll
    for (int s = kPagesThreads / 2; s > 0; s >>= 1)
      if (f.before[lo + s] <= r) lo += s;
    w0 = (long long)lo * f.per;
    base = f.before[lo];
    load();
  }
  // The r-th free page for the lanes that want one (ranks ascend with the lane and from call
  // to call; all are below `upto`); -1 where there are not as many.
  __device__ __forceinline__ int get(bool want, int r, int upto) {
    int page = -1;
    if (upto <= end) return want ? (int)(w0 * 32) + list[place(r - base)] : page;
    bool open = want && r < f.total;
    while (true) {
      if (open && r < end) {
        page = (int)(w0 * 32) + list[place(r - base)];
        open = false;
      }
      if (!__any_sync(0xffffffffu, open) || w0 + kWindowWords >= f.words) return page;
      w0 += kWindowWords;
      base = end;
      load();
    }
  }
};

// The first n free pages are free no more (by all CTAs of the cluster, a share each, once
// every one has read the bitmap for the last time).
__device__ __forceinline__ void clear_first(const Pool& p, const FreeCount& f, int n, int rank,
                                            int ctas) {
  if ((int)threadIdx.x % ctas != rank) return;
  int left = n - f.before[threadIdx.x];
  const long long w0 = (long long)threadIdx.x * f.per;
  for (int i = 0; i < f.per && left > 0; ++i) {
    if (w0 + i >= f.words) return;
    uint32_t x = free_word(p, w0 + i);
    const int c = __popc(x);
    if (c == 0) continue;
    if (left >= c) {
      x = 0;
    } else {
      for (int k = 0; k < left; ++k) x &= x - 1;
    }
    left -= c;
    p.free[w0 + i] = x;
  }
}

// ------------------------------------------------------------------------------- free
struct FreeArgs {
  Pool pool;
  int32_t* table;
  const int32_t* lens;  // or null: every entry goes
  unsigned entries;
  int Hkv, max_blocks, block;
};
// One reference less for every entry behind its sequence's last block, which becomes -1.  A
// page given up more often than it was taken stays at 0.
__global__ void __launch_bounds__(256) pages_free_kernel(const FreeArgs a) {
  after_predecessor();
  for (unsigned e = blockIdx.x * 256 + threadIdx.x; e < a.entries; e += gridDim.x * 256) {
    if (a.lens != nullptr) {
      const unsigned row = e / (unsigned)a.max_blocks;
      const int j = (int)(e - row * (unsigned)a.max_blocks);
      if (j < blocks_of(read_global(a.lens + row / (unsigned)a.Hkv), a.block, a.max_blocks))
        continue;
    }
    const int p = read_global(a.table + e);
    if (p == -1) continue;
    a.table[e] = -1;
    if (!is_page(p, a.pool.pages)) continue;
    const int had = atomicSub(a.pool.refs + p, 1);
    if (had == 1)
      atomicOr(a.pool.free + (p >> 5), 1u << (p & 31));
    else if (had <= 0)
      atomicAdd(a.pool.refs + p, 1);
  }
}

// ---------------------------------------------------------------------------- reserve
struct ReserveArgs {
  Pool pool;
  int32_t* table;
  const int32_t *lens, *n_new;  // n_new or null: one token each
  int32_t* lacking;
  int B, Hkv, max_blocks, block;
};
// What the cluster shares: the pages that each CTA asks for.
struct PagesShared {
  int before[kPagesThreads + 1];
  int warp[33];
  int asked;
};
// Pages asked for by the CTAs before this one; *all of them.  (A barrier of a cluster of several.)
__device__ __forceinline__ int cluster_before(PagesShared& s, int asked, int* all) {
  auto cluster = cooperative_groups::this_cluster();
  *all = asked;
  if (cluster.num_blocks() == 1) return 0;
  if (threadIdx.x == 0) s.asked = asked;
  cluster.sync();
  const int rank = (int)cluster.block_rank();
  int before = 0, sum = 0;
  for (int c = 0; c < (int)cluster.num_blocks(); ++c) {
    const int n = *cluster.map_shared_rank(&s.asked, c);
    if (c < rank) before += n;
    sum += n;
  }
  *all = sum;
  return before;
}

// The rows are divided among the cluster's warps in order.  A warp looks up 32 rows' ranges at a
// time, a lane each; short ranges (a token each) stay with the lane, of long ones (a prompt) the
// warp takes one after another, several entries a lane under way.
// The block that the next token falls in may be there already, and shared, where a sequence's length
// has been set back: it is not to be written, and counts as lacking.  (It is looked up beside what
// is needed anyway, and nothing waits for it before the end.)
__global__ void __launch_bounds__(kPagesThreads) pages_reserve_kernel(const ReserveArgs a) {
  __shared__ PagesShared s;
  __shared__ uint16_t s_list[kPagesThreads / 32][32 * kWindowWords];
  auto cluster = cooperative_groups::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int lane = (int)threadIdx.x & 31;
  const unsigned warps = ctas * (kPagesThreads / 32),
                 warp = rank * (kPagesThreads / 32) + (threadIdx.x >> 5);
  // few rows are cut into parts, so that all warps have some
  const unsigned heads = a.Hkv, whole = a.B * heads;
  const unsigned parts = whole > 0 && 2 * warps > whole && a.max_blocks > 32 ? 2 * warps / whole : 1;
  const unsigned rows = whole * parts;
  const unsigned r0 = (unsigned)((unsigned long long)rows * warp / warps),
                 r1 = (unsigned)((unsigned long long)rows * (warp + 1) / warps);
  after_predecessor();
  for (int b = rank * kPagesThreads + (int)threadIdx.x; b < a.B; b += ctas * kPagesThreads)
    a.lacking[b] = 0;
  struct Range {
    int first, last, b;  // blocks [first, last) of the part hold tokens to come
    int32_t* row;
    bool next;           // the first of them is the next token's
  };
  auto range = [&](unsigned part) {
    Range x{0, 0, 0, a.table, false};
    if (part >= r1) return x;
    const unsigned row = part / parts;
    x.b = (int)(row / heads);
    x.row = a.table + (size_t)row * a.max_blocks;
    const int held = read_global(a.lens + x.b);
    const int more = a.n_new != nullptr ? read_global(a.n_new + x.b) : 1;
    const long long len = held > 0 ? held : 0;
    // (blocks are of 64 or 128 tokens)
    const int shift = a.block == 64 ? 6 : 7;
    x.first = (int)(len >> shift) < a.max_blocks ? (int)(len >> shift) : a.max_blocks;
    const long long end = (len + (more > 0 ? more : 0) + a.block - 1) >> shift;
    x.last = end < a.max_blocks ? (int)end : a.max_blocks;
    const int next = x.first;
    if (parts > 1) {
      const unsigned n = x.last - x.first, q = part - row * parts;
      x.last = x.first + (int)((unsigned long long)n * (q + 1) / parts);
      x.first += (int)((unsigned long long)n * q / parts);
    }
    x.next = x.first == next && x.first < x.last;
    return x;
  };
  auto of_lane = [&](const Range& x, int k) {
    Range y;
    y.first = __shfl_sync(0xffffffffu, x.first, k);
    y.last = __shfl_sync(0xffffffffu, x.last, k);
    y.b = __shfl_sync(0xffffffffu, x.b, k);
    y.next = false;
    y.row = reinterpret_cast<int32_t*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(x.row), k));
    return y;
  };
  // the lane's entries j, j + 32, .. that want a page (of a range that is not empty)
  auto batch = [&](const Range& x, int j, bool (&want)[kEntries]) {
    int v[kEntries];
#pragma unroll
    for (int i = 0; i < kEntries; ++i)
      v[i] = read_global(x.row + (j + 32 * i < x.last ? j + 32 * i : x.first));
#pragma unroll
    for (int i = 0; i < kEntries; ++i)
      want[i] = j + 32 * i < x.last && !is_page(v[i], a.pool.pages);
  };
  // a short range, as a mask
  auto few = [&](const Range& x) {
    uint32_t mask = 0;
    if (x.first < x.last) {
      int v[kFew];
#pragma unroll
      for (int i = 0; i < kFew; ++i)
        v[i] = read_global(x.row + (x.first + i < x.last ? x.first + i : x.first));
#pragma unroll
      for (int i = 0; i < kFew; ++i)
        mask |= x.first + i < x.last && !is_page(v[i], a.pool.pages) ? 1u << i : 0u;
    }
    return mask;
  };
  int asked = 0;
  int next = -1, named = 0;  // the page of the lane's next token, and the entries that name it
  Range x{0, 0, 0, a.table, false};
  uint32_t mask = 0;
  for (unsigned rb = r0; rb < r1; rb += 32) {
    x = range(rb + lane);
    if (x.next) next = read_global(x.row + x.first);
    if (__all_sync(0xffffffffu, x.last - x.first <= kFew)) {
      mask = few(x);
      asked += (int)__reduce_add_sync(0xffffffffu, (unsigned)__popc(mask));
      continue;
    }
    for (unsigned k = 0; k < 32 && rb + k < r1; ++k) {
      const Range y = of_lane(x, (int)k);
      for (int j = y.first + lane; j - lane < y.last; j += 32 * kEntries) {
        bool want[kEntries];
        batch(y, j, want);
#pragma unroll
        for (int i = 0; i < kEntries; ++i) asked += __popc(__ballot_sync(0xffffffffu, want[i]));
      }
    }
  }
  const FreeCount f = count_free(a.pool, s.before, s.warp);
  if (is_page(next, a.pool.pages)) named = read_global(a.pool.refs + next);
  int in_cta, all;
  int at = block_before(lane == 0 ? asked : 0, s.warp, &in_cta);
  at = __shfl_sync(0xffffffffu, at, 0);
  at += cluster_before(s, in_cta, &all);
  if (asked > 0) {
    FreeWindow window{a.pool, f, s_list[threadIdx.x >> 5]};
    for (unsigned rb = r0; rb < r1; rb += 32) {
      if (r1 - r0 > 32) x = range(rb + lane);
      if (__all_sync(0xffffffffu, x.last - x.first <= kFew)) {
        if (r1 - r0 > 32) mask = few(x);
        int r = __popc(mask), none = 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, r, o);
          if (lane >= o) r += y;
        }
        const int sum = __shfl_sync(0xffffffffu, r, 31);
        r += at - __popc(mask);
        at += sum;
        for (; mask; mask &= mask - 1) {
          const int p = r < f.total ? nth_free(a.pool, f, r) : -1;
          ++r;
          if (p >= 0)
            a.pool.refs[p] = 1;
          else
            ++none;
          x.row[x.first + __ffs((int)mask) - 1] = p;
        }
        if (none) atomicAdd(a.lacking + x.b, none);
        continue;
      }
      window.seek(at);
      for (unsigned k = 0; k < 32 && rb + k < r1; ++k) {
        const Range y = of_lane(x, (int)k);
        for (int j = y.first + lane; j - lane < y.last; j += 32 * kEntries) {
          bool want[kEntries];
          batch(y, j, want);
#pragma unroll
          for (int i = 0; i < kEntries; ++i) {
            const uint32_t votes = __ballot_sync(0xffffffffu, want[i]);
            if (votes == 0) continue;
            const int r = at + __popc(votes & ((1u << lane) - 1u));
            at += __popc(votes);
            const int p = window.get(want[i], r, at);
            if (want[i]) {
              if (p >= 0) a.pool.refs[p] = 1;
              y.row[j + 32 * i] = p;
            }
            if (at <= f.total) continue;
            const uint32_t none = __ballot_sync(0xffffffffu, want[i] && p < 0);
            if (none && lane == 0) atomicAdd(a.lacking + y.b, __popc(none));
          }
        }
      }
    }
  }
  const bool again = r1 - r0 > 32;  // more rows than lanes: looked up now
  for (unsigned rb = r0; rb < r1; rb += 32) {
    if (again) {
      x = range(rb + lane);
      next = x.next ? read_global(x.row + x.first) : -1;
      named = is_page(next, a.pool.pages) ? read_global(a.pool.refs + next) : 0;
    }
    if (named > 1) atomicAdd(a.lacking + x.b, 1);
  }
  if (ctas > 1)
    cluster.sync();
  else
    __syncthreads();
  clear_first(a.pool, f, all, rank, ctas);
}

// ------------------------------------------------------------------------------- fork
struct CachePtrs {
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  uint16_t* k_mean;  // or null
};
struct ForkArgs {
  Pool pool;
  CachePtrs cache;
  const int32_t *table, *lens, *parent;
  int32_t *table_out, *lens_out, *lacking;
  int B, N, Hkv, max_blocks, block;
};
// A child's parent and tokens (none for a parent that is not there).
__device__ __forceinline__ int fork_parent(const ForkArgs& a, int i, int* tokens) {
  const int p = read_global(a.parent + i);
  if (p < 0 || p >= a.B) {
    *tokens = 0;
    return -1;
  }
  const long long most = (long long)a.max_blocks * a.block, n = read_global(a.lens + p);
  *tokens = n < 0 ? 0 : (int)(n < most ? n : most);
  return p;
}
// Pages for the part-full blocks of the children: entry `tokens / block` of their rows.
__global__ void __launch_bounds__(kPagesThreads) pages_fork_kernel(const ForkArgs a) {
  __shared__ PagesShared s;
  auto cluster = cooperative_groups::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int lane = (int)threadIdx.x & 31;
  const unsigned warps = ctas * (kPagesThreads / 32),
                 warp = rank * (kPagesThreads / 32) + (threadIdx.x >> 5);
  const unsigned heads = a.Hkv, rows = a.N * heads;
  const unsigned r0 = (unsigned)((unsigned long long)rows * warp / warps),
                 r1 = (unsigned)((unsigned long long)rows * (warp + 1) / warps);
  after_predecessor();
  for (int i = rank * kPagesThreads + (int)threadIdx.x; i < a.N; i += ctas * kPagesThreads) {
    int n;
    fork_parent(a, i, &n);
    a.lens_out[i] = n;
    a.lacking[i] = 0;
  }
  auto wanted = [&](unsigned row, int* full) {
    if (row >= r1) return false;
    const int i = (int)(row / heads), h = (int)(row - i * heads);
    int n;
    const int p = fork_parent(a, i, &n);
    *full = n / a.block;
    return n % a.block != 0 &&
           is_page(read_global(a.table + ((long long)p * a.Hkv + h) * a.max_blocks + *full),
                   a.pool.pages);
  };
  int asked = 0, full = 0;
  bool want = false;
  for (unsigned row = r0; row < r1; row += 32) {
    want = wanted(row + lane, &full);
    asked += __popc(__ballot_sync(0xffffffffu, want));
  }
  const FreeCount f = count_free(a.pool, s.before, s.warp);
  int in_cta, all;
  int at = block_before(lane == 0 ? asked : 0, s.warp, &in_cta);
  at = __shfl_sync(0xffffffffu, at, 0);
  at += cluster_before(s, in_cta, &all);
  for (unsigned row = r0; row < r1; row += 32) {
    if (r1 - r0 > 32) want = wanted(row + lane, &full);
    const uint32_t votes = __ballot_sync(0xffffffffu, want);
    const int r = at + __popc(votes & ((1u << lane) - 1u));
    at += __popc(votes);
    if (want) {
      const int p = r < f.total ? nth_free(a.pool, f, r) : -1;
      if (p >= 0)
        a.pool.refs[p] = 1;
      else
        atomicAdd(a.lacking + (row + lane) / heads, 1);
      a.table_out[(size_t)(row + lane) * a.max_blocks + full] = p;
    }
  }
  if (ctas > 1)
    cluster.sync();
  else
    __syncthreads();
  clear_first(a.pool, f, all, rank, ctas);
}

// `tokens` tokens of page src to page dst, with the page's scales and mean, by a CTA.
__device__ __forceinline__ void copy_page(const CachePtrs& c, int block, int src, int dst,
                                          int tokens) {
  const int n = tokens * 8;  // pieces of 16 bytes in the keys, and as many in the values
  const long long s = (long long)src * block * 8, d = (long long)dst * block * 8;
  const uint4* k = reinterpret_cast<const uint4*>(c.k) + s;
  const uint4* v = reinterpret_cast<const uint4*>(c.v) + s;
  uint4* ko = reinterpret_cast<uint4*>(c.k) + d;
  uint4* vo = reinterpret_cast<uint4*>(c.v) + d;
  for (int i = (int)threadIdx.x; i < n; i += 2 * (int)blockDim.x) {
    const int i2 = i + (int)blockDim.x;
    const bool two = i2 < n;
    const uint4 k1 = k[i], v1 = v[i];
    uint4 k2, v2;
    if (two) {
      k2 = k[i2];
      v2 = v[i2];
    }
    ko[i] = k1;
    vo[i] = v1;
    if (two) {
      ko[i2] = k2;
      vo[i2] = v2;
    }
  }
  if (threadIdx.x < 16 && c.k_mean != nullptr)
    reinterpret_cast<uint4*>(c.k_mean)[(long long)dst * 16 + threadIdx.x] =
        reinterpret_cast<const uint4*>(c.k_mean)[(long long)src * 16 + threadIdx.x];
  if (threadIdx.x == 32) c.k_scale[dst] = c.k_scale[src];
  if (threadIdx.x == 33) c.v_scale[dst] = c.v_scale[src];
}

// A CTA a row: the entries of full blocks, each with a reference more, -1 behind, and what the
// part-full block holds.
__global__ void __launch_bounds__(256) cache_fork_kernel(const ForkArgs a) {
  const long long row = blockIdx.x;
  const int i = (int)(row / a.Hkv), h = (int)(row - (long long)i * a.Hkv);
  after_predecessor();
  int n;
  const int p = fork_parent(a, i, &n);
  const int full = n / a.block;
  const bool part = n % a.block != 0;
  const int32_t* from = a.table + ((long long)(p < 0 ? 0 : p) * a.Hkv + h) * a.max_blocks;
  int32_t* to = a.table_out + row * a.max_blocks;
  int src = -1, dst = -1;
  if (part) {
    src = read_global(from + full);
    if (is_page(src, a.pool.pages)) dst = read_global(to + full);
  }
  for (int j = (int)threadIdx.x; j < a.max_blocks; j += 256) {
    if (j == full && dst >= 0) continue;
    int page = -1;
    if (j < full) {
      page = read_global(from + j);
      if (is_page(page, a.pool.pages))
        atomicAdd(a.pool.refs + page, 1);
      else
        page = -1;
    }
    to[j] = page;
  }
  if (dst >= 0) copy_page(a.cache, a.block, src, dst, n % a.block);
}

// ---------------------------------------------------------------------------- compact
struct CompactArgs {
  Pool pool;
  CachePtrs cache;
  int32_t *table, *to, *n_used;
  long long entries;
  int block;
};
// With U pages in use: where each goes.  Those below U stay, the r-th in use from U on goes to
// the r-th free one (there are as many below U).
__global__ void __launch_bounds__(kPagesThreads) pages_compact_kernel(const CompactArgs a) {
  __shared__ PagesShared s;
  after_predecessor();
  const FreeCount f = count_free(a.pool, s.before, s.warp);
  const int used = a.pool.pages - f.total;
  // free pages before page p
  auto free_before = [&](int p) {
    const long long w = p >> 5, t = w / f.per;
    int n = f.before[t];
    for (long long i = t * f.per; i < w; ++i) n += __popc(free_word(a.pool, i));
    return n + __popc(free_word(a.pool, w) & ((1u << (p & 31)) - 1u));
  };
  // pages in use below U (U itself may be the pool's end)
  const int below = used < a.pool.pages ? used - free_before(used) : used;
  for (long long q = (long long)blockIdx.x * kPagesThreads + threadIdx.x; q < a.pool.pages;
       q += (long long)gridDim.x * kPagesThreads) {
    const int p = (int)q;
    int to = -1;
    if (!((free_word(a.pool, p >> 5) >> (p & 31)) & 1u))
      to = p < used ? p : nth_free(a.pool, f, p - free_before(p) - below);
    a.to[p] = to;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_used = used;
}
// The moves, the counts, the bitmap and the table.
__global__ void __launch_bounds__(256) cache_compact_kernel(const CompactArgs a) {
  after_predecessor();
  const int used = read_global(a.n_used);
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x, all = (long long)gridDim.x * 256;
  for (long long e = id; e < a.entries; e += all) {
    const int p = read_global(a.table + e);
    if (is_page(p, a.pool.pages)) {
      const int to = read_global(a.to + p);
      if (to != p) a.table[e] = to;
    }
  }
  for (long long w = id; w < ((long long)a.pool.pages + 31) / 32; w += all) {
    const long long first = w * 32;
    uint32_t x = 0xffffffffu;
    if (first + 32 <= used)
      x = 0;
    else if (first < used)
      x <<= used - first;
    if (first + 32 > a.pool.pages) x &= (1u << (a.pool.pages - first)) - 1u;
    a.pool.free[w] = x;
  }
  for (long long p = used + (long long)blockIdx.x; p < a.pool.pages; p += gridDim.x) {
    const int to = read_global(a.to + p);
    if (to < 0) continue;
    copy_page(a.cache, a.block, (int)p, to, a.block);
    if (threadIdx.x == 64) {
      a.pool.refs[to] = a.pool.refs[p];
      a.pool.refs[p] = 0;
    }
  }
}

}  // namespace vsa

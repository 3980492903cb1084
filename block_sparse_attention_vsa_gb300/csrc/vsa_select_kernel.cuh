// vsa_select_kernel.cuh -- block means and the choice of key blocks by a cheap score.
//
//   block_mean_kernel    m_j = (1/n_j) sum of the block's first n_j tokens (bf16 in and out,
//                        fp32 sums)
//   select_kernel        LUT rows: the topk key blocks j of highest q_mean_i . k_mean_j
//   cache_select_kernel  the same for one token per sequence over the pages of a cache
//
// The choice is that of fp64 sums, ties to the lowest index: scores are first computed on the
// tensor cores with fp32 sums, and only where the error bound of that arithmetic leaves the
// border open are the blocks near it scored again (fp32 with a tighter bound, then fp64, in
// which the products of bf16 values are exact, and their sum while they differ by less than
// 2^30 in size: 16 bits of a product and 7 of 128 terms fit 53).  The fp64 sum has one order
// everywhere, that of 8 lanes with 16 products each.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "vsa_warp_ptx.cuh"

namespace vsa {

// ------------------------------------------------------------------ block means
// One CTA per block, 8 rows a thread: a thread holds 8 of the 128 columns (16 bytes) of
// rows t/16, t/16 + threads/16, ...  The 8 loads of a thread are independent, and that many
// small CTAs keep enough of them in flight: bound by DRAM, 86 us and 7.1 TB/s for 24 heads
// of 98,304 tokens, 9.3 us (5.5 TB/s) for 12 of 16,384.
template <int BLOCK>
__global__ void __launch_bounds__(BLOCK * 2)
    block_mean_kernel(const uint16_t* x, const int32_t* sizes, int S, int nb, uint16_t* mean) {
  after_predecessor();
  constexpr int kThreads = BLOCK * 2, kRowsPerPass = kThreads / 16, kWarps = kThreads / 32;
  __shared__ float part[kWarps][128];
  const long long blk = blockIdx.x;
  const long long bh = blk / nb;
  const int j = (int)(blk - bh * nb);
  int n = S - j * BLOCK;
  n = n < BLOCK ? n : BLOCK;
  if (sizes != nullptr) {
    const int s = sizes[j];
    n = s < n ? (s < 0 ? 0 : s) : n;
  }
  const int c = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const uint4* src = reinterpret_cast<const uint4*>(x + (bh * S + (long long)j * BLOCK) * 128) + c;
  uint4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + i * kRowsPerPass;
    w[i] = r < n ? read_global(src + r * 16) : make_uint4(0, 0, 0, 0);
  }
  float a[8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[2 * e] += bf16_lo(u[e]);
      a[2 * e + 1] += bf16_hi(u[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) a[e] += __shfl_xor_sync(0xffffffffu, a[e], 16);
  if ((threadIdx.x & 31) < 16) {
    float4* p = reinterpret_cast<float4*>(&part[threadIdx.x >> 5][c * 8]);
    p[0] = make_float4(a[0], a[1], a[2], a[3]);
    p[1] = make_float4(a[4], a[5], a[6], a[7]);
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int p = 0; p < kWarps; ++p) {
      lo += part[p][2 * threadIdx.x];
      hi += part[p][2 * threadIdx.x + 1];
    }
    const float d = (float)(n > 0 ? n : 1);
    const __nv_bfloat162 m = __floats2bfloat162_rn(lo / d, hi / d);
    reinterpret_cast<__nv_bfloat162*>(mean + blk * 128)[threadIdx.x] = m;
  }
}

// ------------------------------------------------------------------ order and selection
// Order-preserving whole numbers of finite fp32 / fp64 values (-0 counts as +0); 0 is kept
// for "not eligible" and the largest for "chosen whatever its score".
constexpr int kMaxBlocks = 2048;
constexpr uint32_t kForced32 = 0xffffffffu;
constexpr uint64_t kForced64 = ~0ull;
__device__ __forceinline__ uint32_t order32(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unorder32(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t order64(double f) {
  if (f != f) return 0;  // a NaN score leaves the block out
  const uint64_t b = (uint64_t)__double_as_longlong(f + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}

constexpr int kSelThreads = 256;  // of the kernels that choose within one row

// The helpers below are called by every thread of a CTA of 256 or more.
struct KthScratch {
  unsigned int hist[256];
  unsigned int warp_sum[32];
  int digit, rest, count;
};

// Which of 256 counted digits, from the largest down, holds the rest-th key, and which of
// its keys that is, of how many: s.digit, s.rest and s.count.  One warp.
__device__ __forceinline__ void digit_of(KthScratch& s, int rest, int lane) {
  // lane l holds digits 255-8l down to 248-8l
  unsigned int h[8], sum = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    h[e] = s.hist[255 - 8 * lane - e];
    sum += h[e];
  }
  unsigned int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  unsigned int before = upto - sum;
  if (before < (unsigned)rest && upto >= (unsigned)rest) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (before < (unsigned)rest && before + h[e] >= (unsigned)rest) {
        s.digit = 255 - 8 * lane - e;
        s.rest = rest - (int)before;
        s.count = (int)h[e];
      }
      before += h[e];
    }
  }
}

// The k-th largest of keys[0..n) (1 <= k <= n) and how many keys are larger: a radix
// descent, 8 bits a pass.  Every thread of the CTA calls it and gets the same answer.
template <typename K>
__device__ void kth_largest(const K* keys, int n, int k, KthScratch& s, K* thr, int* larger) {
  K prefix = 0, mask = 0;
  int rest = k;
  for (int shift = 8 * (int)sizeof(K) - 8; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) s.hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const K key = keys[i];
      if ((key & mask) == prefix) atomicAdd(&s.hist[(unsigned)(key >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (threadIdx.x < 32) digit_of(s, rest, threadIdx.x);
    __syncthreads();
    prefix |= (K)s.digit << shift;
    mask |= (K)255 << shift;
    rest = s.rest;
  }
  *thr = prefix;
  *larger = k - rest;
}

// The value of rank `within` (1 = largest) among members[0..count), count <= kRanked and
// none of them 0: to *thr, and which of those equal to it that is to s.rest.  `members` is
// 16-byte aligned with room for kRanked.
constexpr int kRanked = 128;
__device__ __forceinline__ void rank_members(uint32_t* members, int count, int within,
                                             KthScratch& s, uint32_t* thr) {
  if (threadIdx.x < 4 && count + (int)threadIdx.x < kRanked) members[count + threadIdx.x] = 0;
  __syncthreads();
  if ((int)threadIdx.x < count) {
    const uint32_t mine = members[threadIdx.x];
    int gt = 0, ge = 0;
#pragma unroll 4
    for (int o = 0; o < count; o += 4) {
      const uint4 y = *reinterpret_cast<const uint4*>(members + o);
      gt += (y.x > mine) + (y.y > mine) + (y.z > mine) + (y.w > mine);
      ge += (y.x >= mine) + (y.y >= mine) + (y.z >= mine) + (y.w >= mine);
    }
    if (gt < within && within <= ge) {  // the same from every thread that gets here
      *thr = mine;
      s.rest = within - gt;
    }
  }
  __syncthreads();
}

// kth_largest of the keys in [base, top], whose least and largest these are: 256 even steps
// between those, then between the ends of the step that the k-th falls into, until that
// holds few enough to rank.  *n_members is 0 before.
__device__ __forceinline__ void kth_between(const uint32_t* keys, int n, int k, uint32_t base,
                                            uint32_t top, KthScratch& s, uint32_t* members,
                                            int* n_members, uint32_t* s_thr, uint32_t* thr,
                                            int* larger) {
  int bits = 32 - __clz(top - base), rest = k, count;
  do {
    const int shift = max(0, bits - 8);
    if (threadIdx.x < 256) s.hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const uint32_t key = keys[i], off = key - base;
      if (key >= base && key <= top && (bits >= 32 || off >> bits == 0))
        atomicAdd(&s.hist[off >> shift], 1u);
    }
    __syncthreads();
    if (threadIdx.x < 32) digit_of(s, rest, threadIdx.x);
    __syncthreads();
    base += (uint32_t)s.digit << shift;
    bits = shift;
    rest = s.rest;
    count = s.count;
  } while (bits > 0 && count > kRanked);
  if (bits > 0) {
    for (int i = threadIdx.x; i < n; i += blockDim.x)
      if (keys[i] >= base && keys[i] <= top && (keys[i] - base) >> bits == 0)
        members[atomicAdd(n_members, 1)] = keys[i];
    rank_members(members, count, rest, s, s_thr);
    base = *s_thr;
    rest = s.rest;
  }
  *thr = base;
  *larger = k - rest;
}

// Exclusive sum over the CTA's threads.
__device__ __forceinline__ unsigned int cta_exclusive(unsigned int v, KthScratch& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s.warp_sum[warp] = x;
  __syncthreads();
  unsigned int before = 0;
  for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
  return before + x - v;
}

// Ascending walk over keys[0..n): those above `thr` and the first `n_eq` equal to it go to
// chosen(position, i), the others to rest(position, i).
template <typename K, typename F, typename R>
__device__ void partition_ascending(const K* keys, int n, K thr, int n_eq, KthScratch& s,
                                    F chosen, R rest) {
  const int per = (n + (int)blockDim.x - 1) / (int)blockDim.x;
  const int a = min(n, (int)threadIdx.x * per), e = min(n, a + per);
  unsigned int mine = 0;  // larger in the low half, equal in the high half
  for (int i = a; i < e; ++i) mine += keys[i] > thr ? 1u : (keys[i] == thr ? 0x10000u : 0u);
  const unsigned int before = cta_exclusive(mine, s);
  int gt = (int)(before & 0xffffu), eq = (int)(before >> 16);
  for (int i = a; i < e; ++i) {
    const bool g = keys[i] > thr, q = keys[i] == thr;
    const int at = gt + min(eq, n_eq);
    if (g || (q && eq < n_eq))
      chosen(at, i);
    else
      rest(i - at, i);
    gt += g;
    eq += q;
  }
}

// The bound of |fp32 tensor-core dot - exact| for 128 products, relative to sum |q||k| <=
// (sum |q|) max|k|: 8 steps of 16 products, each step's terms aligned to the largest and
// cut at 24 bits or more -- at most 17 * 8 * 2^-23 < 2^-15.
constexpr float kDotBound = 3.0517578125e-5f;  // 2^-15
constexpr float kFinite = 1e38f;  // scores and bounds beyond it are computed in fp64
// What products and sums that fall below the normal fp32 range may lose in all.
constexpr float kTiny = 1e-35f;

// ------------------------------------------------------------------ LUT rows
struct SelectArgs {
  const uint16_t* q;      // [B, Hq, nq, 128]
  const uint16_t* k;      // [B, Hkv, nk, 128]
  const int32_t* sizes;   // [nk] or null
  int32_t* idx;           // [B, Hq, nq, topk]
  int32_t* num;           // [B, Hq, nq]
  int Hq, Hkv, group, nq, nk, topk, causal, n_first, n_near, tiles;
};

constexpr int kSelRowThreads = 512;

__host__ __device__ constexpr int select_stride(int nreg) { return nreg * 64 + 8; }
__host__ __device__ constexpr size_t select_smem(int nreg, int rows) {
  return (size_t)rows * select_stride(nreg) * 2;
}

// Whether block e may be chosen by a row whose diagonal is d, and whether it must be.
__device__ __forceinline__ bool select_allowed(const SelectArgs& a, int e, int d) {
  return e >= 0 && e < a.nk && (a.sizes == nullptr || a.sizes[e] > 0) && (!a.causal || e <= d);
}
__device__ __forceinline__ bool select_forced(const SelectArgs& a, int e, int d) {
  return e < a.n_first || (e > d - a.n_near && e < d + a.n_near);
}

// fp16 values in the order of 16-bit whole numbers.
__device__ __forceinline__ uint16_t f16_unorder(uint32_t o) {
  return (uint16_t)((o & 0x8000u) ? o & 0x7fffu : ~o & 0xffffu);
}
__device__ __forceinline__ float f16_value(uint16_t b) {
  return __half2float(__ushort_as_half(b));
}
__device__ __forceinline__ __half2 f16_pair(uint16_t b) {
  return __half2half2(__ushort_as_half(b));
}
__device__ __forceinline__ __half2 as_half2(uint32_t w) {
  return *reinterpret_cast<const __half2*>(&w);
}
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) {
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}

// How many of the warp's 64*NREG keys are >= the threshold (NaN keys never count).
template <int NREG>
__device__ __forceinline__ int count_ge(const uint32_t (&key)[NREG], uint16_t thr) {
  const __half2 t = f16_pair(thr);
  __half2 c = as_half2(0), d = as_half2(0);
#pragma unroll
  for (int j = 0; j < NREG; j += 2) {
    c = __hadd2(c, __hge2(as_half2(key[j]), t));
    d = __hadd2(d, __hge2(as_half2(key[j + 1]), t));
  }
  c = __hadd2(c, d);
  return __reduce_add_sync(0xffffffffu, (int)(__low2float(c) + __high2float(c)));
}

// Bit i of x to bit 2 i.
__device__ __forceinline__ uint32_t spread16(uint32_t x) {
  x = (x | x << 8) & 0x00ff00ffu;
  x = (x | x << 4) & 0x0f0f0f0fu;
  x = (x | x << 2) & 0x33333333u;
  return (x | x << 1) & 0x55555555u;
}

// A lane's 2*NREG flags, ascending.
template <int NREG>
struct LaneSet {
  static constexpr int kWords = (NREG + 15) / 16;
  uint32_t w[kWords];
  // from masks of pairs: bit j of the low half the even element of pair j, of the high
  // half the odd one (16 pairs a word)
  __device__ __forceinline__ void from_pairs(const uint32_t (&m)[kWords]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = spread16(m[i] & 0xffffu) | spread16(m[i] >> 16) << 1;
  }
  __device__ __forceinline__ int count() const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) n += __popc(w[i]);
    return n;
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      for (uint32_t r = w[i]; r != 0; r &= r - 1) f(32 * i + __ffs(r) - 1, i, r & (0u - r));
  }
};

__device__ __forceinline__ int warp_exclusive(int v, int lane) {
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x - v;
}

// One CTA: ROWS (32, or 16 where that leaves SMs idle) query-block rows of one head against
// all nk <= 64*NREG key blocks.
//   1. scores on the tensor cores: a warp walks key tiles of 16 against the rows, whose
//      operands lie in shared memory; operands are read 16 bytes a thread with the
//      contraction index permuted the same way on both sides, so no shuffle or
//      transposition is needed.  Scores go to shared memory as fp16, times a power of two
//      per row that brings them into its range (32 x nk x 2 bytes fit twice on an SM, fp32
//      would not; the rounding only widens the band that is scored again).
//   2. a warp per row, a lane with 2*NREG consecutive keys in NREG registers of pairs.
//      The border is bracketed in the 16-bit order of the keys by counting, two keys an
//      instruction: outwards from where a normal distribution of the row's mean and mean
//      deviation (of a third of its keys) has it, then by interpolation, aimed at either
//      side of the border in turn, until at most 2 keys lie between the bracket's ends.
//      Blocks surely above the bracket are in; those that the error bound leaves open are
//      scored again.
// Both parts wait for latencies more than for any unit: 16 warps of 64 registers a CTA,
// two CTAs on an SM.  24 heads of 1,536 x 1,536 blocks: 149 us, of which the scores are
// about 64 (the L1 and shared memory's data path: 6 KB read for 16 keys x 32 rows), the
// border 33, the blocks scored again 18, masks and output 17.  With the scores in bf16, 8
// warps and 128 registers, and a bisection of all 16 bits it was 267 us.
template <int NREG, int ROWS>
__global__ void __launch_bounds__(kSelRowThreads, NREG <= 24 ? 2 : 1)
    select_kernel(const SelectArgs a) {
  after_predecessor();
  extern __shared__ __align__(16) uint16_t s_key[];  // [ROWS][stride]
  constexpr int kStride = select_stride(NREG), kWarps = kSelRowThreads / 32;
  constexpr int kQStride = 160;  // 320 bytes: rows g and g + 1 in different halves of the banks
  __shared__ __align__(16) uint16_t s_q[ROWS][kQStride];
  __shared__ uint32_t s_fair[kMaxBlocks / 32];
  __shared__ float s_q1[ROWS];
  __shared__ uint32_t s_kmax[kWarps];
  __shared__ unsigned int s_slow, s_sample;
  __shared__ uint16_t s_cand[kWarps][32];
  __shared__ KthScratch s_kth;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, i4 = lane & 3;
  const long long bh = blockIdx.x / a.tiles;  // b * Hq + hq
  const int row0 = (int)(blockIdx.x - bh * a.tiles) * ROWS;
  const long long b = bh / a.Hq;
  const int hkv = (int)(bh - b * a.Hq) / a.group;
  const uint16_t* qh = a.q + (bh * a.nq) * 128;
  const uint16_t* kh = a.k + ((b * a.Hkv + hkv) * (long long)a.nk) * 128;
  if (tid == 0) s_slow = s_sample = 0;
  __syncthreads();

  auto abs_max = [](__nv_bfloat162 m, const uint4& v) {
    m = __hmax2(m, __habs2(as_bf162(v.x)));
    m = __hmax2(m, __habs2(as_bf162(v.y)));
    m = __hmax2(m, __habs2(as_bf162(v.z)));
    return __hmax2(m, __habs2(as_bf162(v.w)));
  };
  {  // the rows and their sums of |q|; the largest |k| of 32 blocks from all over
    const int r = tid >> 4, c = tid & 15;
    const uint4 v =
        r < ROWS && row0 + r < a.nq
            ? read_global(reinterpret_cast<const uint4*>(qh + (long long)(row0 + r) * 128) + c)
            : make_uint4(0, 0, 0, 0);
    const uint4 w =
        a.nk > 0 ? read_global(reinterpret_cast<const uint4*>(
                                   kh + (long long)(r * a.nk / 32) * 128) + c)
                 : make_uint4(0, 0, 0, 0);
    if (r < ROWS) reinterpret_cast<uint4*>(s_q[r])[c] = v;
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) s += fabsf(bf16_lo(u[e])) + fabsf(bf16_hi(u[e]));
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    if (c == 0 && r < ROWS) s_q1[r] = s;
    const __nv_bfloat162 m = abs_max(as_bf162(0), w);
    const uint32_t mm = __reduce_max_sync(
        0xffffffffu, __float_as_uint(fmaxf(__low2float(m), __high2float(m))));
    if (lane == 0) atomicMax(&s_sample, mm);
  }
  // what may be chosen at all
  int n_fair = 0;
#pragma unroll
  for (int e0 = 0; e0 < NREG * 64; e0 += kSelRowThreads) {
    const int e = e0 + tid;
    const bool fair = e < a.nk && (a.sizes == nullptr || a.sizes[e] > 0);
    const unsigned int m = __ballot_sync(0xffffffffu, fair);
    if (lane == 0 && e < NREG * 64) s_fair[e >> 5] = m;
    n_fair += __syncthreads_count(fair);
  }
  // the power of two that brings a row's largest possible score, were the sampled |k| the
  // largest, to 2^13
  auto factor_of = [&](int r) {
    const uint32_t e = __float_as_uint(s_q1[r] * __uint_as_float(s_sample)) >> 23 & 0xffu;
    return __uint_as_float((uint32_t)(127 + min(100, max(-100, 127 + 13 - (int)e))) << 23);
  };

  // scores
  {
    constexpr int kM = ROWS / 16;
    float f[2 * kM];
#pragma unroll
    for (int r = 0; r < 2 * kM; ++r) f[r] = factor_of(g + 8 * r);
    __nv_bfloat162 kmax = as_bf162(0);
    unsigned int bad = 0;
    for (int t = warp; t * 16 < a.nk; t += kWarps) {
      uint4 kb[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int key = t * 16 + 8 * x + g;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          kb[x][j] = key < a.nk
                         ? read_global(reinterpret_cast<const uint4*>(kh + (long long)key * 128) +
                                       i4 + 4 * j)
                         : make_uint4(0, 0, 0, 0);
      }
      float d[kM][2][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          const uint4 qa = reinterpret_cast<const uint4*>(s_q[16 * m + g])[i4 + 4 * j];
          const uint4 qb = reinterpret_cast<const uint4*>(s_q[16 * m + 8 + g])[i4 + 4 * j];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            mma_bf16(d[m][x], qa.x, qb.x, qa.y, qb.y, kb[x][j].x, kb[x][j].y);
            mma_bf16(d[m][x], qa.z, qb.z, qa.w, qb.w, kb[x][j].z, kb[x][j].w);
          }
        }
        kmax = abs_max(kmax, kb[0][j]);
        kmax = abs_max(kmax, kb[1][j]);
      }
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * m + 8 * h + g;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float u = d[m][x][2 * h], v = d[m][x][2 * h + 1];
            const float fu = u * f[2 * m + h], fv = v * f[2 * m + h];
            if (!(fabsf(u) < kFinite && fabsf(v) < kFinite && fabsf(fu) < 65000.0f &&
                  fabsf(fv) < 65000.0f))
              bad |= 1u << (2 * m + h);
            *reinterpret_cast<uint32_t*>(s_key + r * kStride + t * 16 + 8 * x + 2 * i4) =
                pack_f16x2(fu, fv);
          }
        }
    }
#pragma unroll
    for (int r = 0; r < 2 * kM; ++r)
      if (bad >> r & 1u) atomicOr(&s_slow, 1u << (g + 8 * r));
    const uint32_t mm = __reduce_max_sync(
        0xffffffffu, __float_as_uint(fmaxf(__low2float(kmax), __high2float(kmax))));
    if (lane == 0) s_kmax[warp] = mm;
  }
  __syncthreads();
  for (int e = tid; e < NREG * 64; e += kSelRowThreads)
    if (!(s_fair[e >> 5] >> (e & 31) & 1u))
      for (int r = 0; r < ROWS; ++r) s_key[r * kStride + e] = 0x7fff;
  __syncthreads();

  uint32_t kmax_bits = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) kmax_bits = max(kmax_bits, s_kmax[w]);
  const float kmax = __uint_as_float(kmax_bits);
  constexpr uint32_t kLowest = 0x03ffu, kHighest = 0xfc00u;  // order of -inf and +inf

  for (int r = warp; r < ROWS; r += kWarps) {
    const int row = row0 + r;
    if (row >= a.nq) break;
    if ((s_slow >> r) & 1u) continue;
    const float q1 = s_q1[r], bound = q1 * kmax;
    if (!(bound < kFinite)) {
      if (lane == 0) atomicOr(&s_slow, 1u << r);
      continue;
    }
    const float f = factor_of(r);
    const int d = row + a.nk - a.nq;
    uint16_t* krow = s_key + r * kStride;
    auto force = [&](int e) {
      if ((s_fair[e >> 5] >> (e & 31) & 1u) && (!a.causal || e <= d)) krow[e] = 0x7c00;
    };
    for (int e = lane; e < a.n_first; e += 32) force(e);
    for (int e = max(0, d - a.n_near + 1) + lane; e < min(a.nk, d + a.n_near); e += 32) force(e);
    __syncwarp();
    const int base = lane * 2 * NREG;
    uint32_t key[NREG];
#pragma unroll
    for (int j = 0; j < NREG; j += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(krow + base + 2 * j);
      key[j] = v.x;
      key[j + 1] = v.y;
      key[j + 2] = v.z;
      key[j + 3] = v.w;
    }
    int n_ok = n_fair;
    if (a.causal) {
#pragma unroll
      for (int j = 0; j < NREG; ++j) {
        if (base + 2 * j > d) key[j] |= 0x00007fffu;
        if (base + 2 * j + 1 > d) key[j] |= 0x7fff0000u;
      }
      n_ok = count_ge<NREG>(key, f16_unorder(kLowest));
    }
    const int k = min(a.topk, n_ok);
    uint16_t in_thr, cand_thr;  // in: key > in_thr, candidate: the others >= cand_thr
    bool ties = false;          // candidates are equal: the lowest indices
    if (n_ok <= a.topk) {
      in_thr = cand_thr = f16_unorder(kLowest);  // all are in
    } else {
      uint32_t lo = kLowest, hi = kHighest;  // count(>= lo) >= k > count(>= hi)
      int c_lo = n_ok, c_hi = 0;
      if (a.n_first + 2 * a.n_near >= k) c_hi = count_ge<NREG>(key, f16_unorder(kHighest));
      if (c_hi >= k) {  // more forced blocks than places
        in_thr = cand_thr = 0x7c00u;
        ties = true;
      } else {
        // of a third of the keys, the finite ones: mean and mean deviation from 0
        __half2 sum2 = as_half2(0), dev2 = as_half2(0), num2 = as_half2(0);
#pragma unroll
        for (int j = 0; j < NREG; j += 3) {
          const __half2 one = __float2half2_rn(1.0f), most = __float2half2_rn(65504.0f);
          const uint32_t on = __hle2_mask(__habs2(as_half2(key[j])), most);
          const __half2 x = as_half2(key[j] & on);
          sum2 = __hadd2(sum2, x);
          dev2 = __hadd2(dev2, __habs2(x));
          num2 = __hadd2(num2, as_half2(*reinterpret_cast<const uint32_t*>(&one) & on));
        }
        float sum = __low2float(sum2) + __high2float(sum2);
        float dev = __low2float(dev2) + __high2float(dev2);
        float num = __low2float(num2) + __high2float(num2);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, x);
          dev += __shfl_xor_sync(0xffffffffu, dev, x);
          num += __shfl_xor_sync(0xffffffffu, num, x);
        }
        num = fmaxf(num, 1.0f);
        const float mean = sum / num, sigma = fmaxf(1.2533f * dev / num, fabsf(mean) * 0.01f);
        const float z = normcdfinvf(1.0f - (float)k / (float)n_ok);
        // keys lie this far apart around there
        const float gap = sigma * 2.5066f * __expf(0.5f * z * z) / (float)n_ok;
        float at_value = mean + z * sigma;
        float reach = 2.0f;  // keys to go beyond the border by
        if (!(fabsf(at_value) < 60000.0f && gap < 60000.0f)) at_value = 0.0f;
        auto order_of = [&](float x) {
          const uint32_t h = __half_as_ushort(__float2half_rn(x));
          return (h & 0x8000u) ? ~h & 0xffffu : h | 0x8000u;
        };
        uint32_t at = min(max(order_of(at_value), kLowest + 1), kHighest - 1);
        int tries = 0;
        while (hi - lo > 1 && c_lo - c_hi > 2) {
          const int c = count_ge<NREG>(key, f16_unorder(at));
          const bool above = c >= k;
          if (above) {
            lo = at;
            c_lo = c;
          } else {
            hi = at;
            c_hi = c;
          }
          const uint32_t half = (lo + hi) >> 1;
          if (lo == kLowest || hi == kHighest) {  // out to the border and `reach` keys beyond
            at_value += above ? ((float)(c - k) + reach) * gap : -((float)(k - c) + reach) * gap;
            reach *= 4.0f;
            at = ++tries < 6 && fabsf(at_value) < 65000.0f ? order_of(at_value) : half;
          } else if (++tries > 8) {
            at = half;
          } else {  // half a key past the border, on the side that moved less
            const float aim = (float)(c_lo - k) + (above ? 1.0f : 0.0f);
            at = lo + (uint32_t)((float)(hi - lo) * aim / (float)(c_lo - c_hi));
          }
          at = min(max(at, lo + 1), hi - 1);
        }
        if (q1 == 0.0f || kmax == 0.0f) {  // every score is 0
          in_thr = 0x0000u;
          cand_thr = 0x8000u;
          ties = true;
        } else {
          // a key is off by half an fp16 step, 2^-11 of it or 2^-25, and what the fp32 sum
          // was; s - bound(s) and s + bound(s) grow with s, so the true k-th score lies
          // between those of the bracket's ends
          const float c = 0.00049f;
          const float eps = (kDotBound * bound + kTiny) * f + 3.1e-8f;
          const float t = f16_value(f16_unorder(lo)), u = f16_value(f16_unorder(hi - 1));
          const float up = u + c * fabsf(u) + 2.0f * eps, dn = t - c * fabsf(t) - 2.0f * eps;
          in_thr = __half_as_ushort(__float2half_ru(up / (up > 0.0f ? 1.0f - c : 1.0f + c)));
          cand_thr = __half_as_ushort(__float2half_rd(dn / (dn > 0.0f ? 1.0f + c : 1.0f - c)));
          if (hi == kHighest || in_thr == 0x7c00u) in_thr = 0x7bffu;  // the forced ones
        }
      }
    }
    LaneSet<NREG> in, cand;
    {
      const __half2 ti = f16_pair(in_thr), tc = f16_pair(cand_thr);
      uint32_t mi[LaneSet<NREG>::kWords] = {}, mc[LaneSet<NREG>::kWords] = {};
#pragma unroll
      for (int j = 0; j < NREG; ++j) {
        mi[j / 16] |= __hgt2_mask(as_half2(key[j]), ti) & (0x00010001u << (j & 15));
        mc[j / 16] |= __hge2_mask(as_half2(key[j]), tc) & (0x00010001u << (j & 15));
      }
#pragma unroll
      for (int i = 0; i < LaneSet<NREG>::kWords; ++i) mc[i] &= ~mi[i];
      in.from_pairs(mi);
      cand.from_pairs(mc);
    }
    const int my_cand = cand.count();
    const int n_in = __reduce_add_sync(0xffffffffu, in.count());
    const int n_cand = __reduce_add_sync(0xffffffffu, my_cand);
    const int need = k - n_in;
    if (n_cand == need) {
#pragma unroll
      for (int i = 0; i < LaneSet<NREG>::kWords; ++i) in.w[i] |= cand.w[i];
    } else {
      int at = warp_exclusive(my_cand, lane);
      if (ties) {
        cand.each([&](int, int i, uint32_t bit) {
          if (at < need) in.w[i] |= bit;
          ++at;
        });
      } else if (n_cand > 32) {
        if (lane == 0) atomicOr(&s_slow, 1u << r);
        continue;
      } else {
        // candidate c in lane c, ascending; scored 4 at a time, 8 lanes and 16 products each
        const int at0 = at;
        cand.each([&](int e, int, uint32_t) { s_cand[warp][at++] = (uint16_t)(base + e); });
        __syncwarp();
        const uint4* qp = reinterpret_cast<const uint4*>(s_q[r]) + (lane & 7);
        auto score = [&](int c, auto zero) {
          using T = decltype(zero);
          const uint4* kp = reinterpret_cast<const uint4*>(kh + (long long)s_cand[warp][c] * 128) +
                            (lane & 7);
          T s = zero;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint4 kw = read_global(kp + 8 * x), qw = qp[8 * x];
            const uint32_t ku[4] = {kw.x, kw.y, kw.z, kw.w}, qu[4] = {qw.x, qw.y, qw.z, qw.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              s = fma((T)bf16_lo(qu[y]), (T)bf16_lo(ku[y]), s);
              s = fma((T)bf16_hi(qu[y]), (T)bf16_hi(ku[y]), s);
            }
          }
#pragma unroll
          for (int x = 4; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
          return s;
        };
        auto rank_of = [&](auto zero) {
          using T = decltype(zero);
          T mine = zero;
          for (int c0 = 0; c0 < n_cand; c0 += 4) {
            const T s = score(min(c0 + (lane >> 3), n_cand - 1), zero);
            const T t = __shfl_sync(0xffffffffu, s, (lane & 3) * 8);
            if (lane >> 2 == c0 >> 2) mine = t;
          }
          // (need lies in [1, n_cand): the border has a block on either side)
          int rank = 0;
          for (int c = 0; c < n_cand; ++c) {
            const T o = __shfl_sync(0xffffffffu, mine, c);
            rank += o > mine || (o == mine && c < lane);
          }
          const bool take = lane < n_cand && rank < need;
          // the gap at the border: 19 roundings of partial sums of at most sum |q||k|
          const T worst = __shfl_sync(
              0xffffffffu, mine, __ffs(__ballot_sync(0xffffffffu, take && rank == need - 1)) - 1);
          const T best = __shfl_sync(
              0xffffffffu, mine,
              __ffs(__ballot_sync(0xffffffffu, lane < n_cand && rank == need)) - 1);
          const bool sure =
              sizeof(T) == 8 || worst - best > (T)(2.0f * 19.5f * 5.9604645e-8f * bound + kTiny);
          return (sure ? 0x100 : 0) | (take ? 1 : 0);
        };
        int got = rank_of(0.0f);
        if (!(got & 0x100)) got = rank_of(0.0);
        const unsigned int taken = __ballot_sync(0xffffffffu, got & 1);
        at = at0;
        cand.each([&](int, int i, uint32_t bit) {
          if (taken >> at & 1u) in.w[i] |= bit;
          ++at;
        });
        __syncwarp();
      }
    }
    // ascending indices, -1 behind (by way of the row's keys, which are in registers)
    int32_t* out = a.idx + (bh * a.nq + row) * (long long)a.topk;
    int at = warp_exclusive(in.count(), lane);
    in.each([&](int e, int, uint32_t) { krow[at++] = (uint16_t)(base + e); });
    __syncwarp();
    for (int s = lane; s < a.topk; s += 32) out[s] = s < k ? krow[s] : -1;
    if (lane == 0) a.num[bh * a.nq + row] = k;
  }
  __syncthreads();

  // Rows whose scores overflow fp32 or fp16, or with more than 32 blocks inside the error
  // band (equal blocks, or means with a large common part): every score in fp64, one row at a
  // time by the whole CTA.  With every row here 43 ms for 24 heads of 1,536 x 1,536 blocks
  // (14.5 GFLOP, 0.34 TFLOP/s), 0.94 ms for 12 heads of 256 x 256.
  unsigned int slow = s_slow;
  uint64_t* key64 = reinterpret_cast<uint64_t*>(s_key);  // nk * 8 <= 32 * stride * 2 bytes
  while (slow != 0) {
    const int r = __ffs(slow) - 1;
    slow &= slow - 1;
    const int row = row0 + r;
    if (row >= a.nq) break;
    const int d = row + a.nk - a.nq;
    __syncthreads();
    int n_ok = 0;
    for (int e0 = 0; e0 < a.nk; e0 += kSelRowThreads) {
      const int e = e0 + tid;
      uint64_t key = 0;
      if (e < a.nk && select_allowed(a, e, d)) {
        if (select_forced(a, e, d)) {
          key = kForced64;
        } else {
          const uint4* qp = reinterpret_cast<const uint4*>(qh + (long long)row * 128);
          const uint4* kp = reinterpret_cast<const uint4*>(kh + (long long)e * 128);
          // summed in the order of the 8 lanes that score a candidate above, so that equal rows
          // have equal scores on either path where the sum is not exact
          double s = 0.0, one = 0.0, two = 0.0, four = 0.0;
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const int l = (i & 1) << 2 | (i & 2) | i >> 2;
            s = 0.0;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint4 qw = read_global(qp + l + 8 * x), kw = read_global(kp + l + 8 * x);
              const uint32_t qu[4] = {qw.x, qw.y, qw.z, qw.w}, ku[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                s = fma((double)bf16_lo(qu[y]), (double)bf16_lo(ku[y]), s);
                s = fma((double)bf16_hi(qu[y]), (double)bf16_hi(ku[y]), s);
              }
            }
            // lanes 0 and 4 and so on in pairs, pairs in fours, fours
            if (i & 1) s += one; else one = s;
            if ((i & 3) == 3) s += two; else if (i & 1) two = s;
            if (i == 7) s += four; else if (i == 3) four = s;
          }
          key = order64(s);
        }
      }
      if (e < a.nk) key64[e] = key;
      n_ok += __syncthreads_count(key != 0);
    }
    const int k = min(a.topk, n_ok);
    uint64_t thr = 0;
    int larger = 0;
    if (n_ok > a.topk) kth_largest<uint64_t>(key64, a.nk, k, s_kth, &thr, &larger);
    int32_t* out = a.idx + (bh * a.nq + row) * (long long)a.topk;
    partition_ascending<uint64_t>(
        key64, a.nk, thr, n_ok > a.topk ? k - larger : 0, s_kth,
        [&](int at, int e) { out[at] = e; },
        [](int, int) {});
    for (int s = k + tid; s < a.topk; s += kSelRowThreads) out[s] = -1;
    if (tid == 0) a.num[bh * a.nq + row] = k;
  }
}

// ------------------------------------------------------------------ single tokens
struct CacheSelectArgs {
  const uint16_t* q;       // [B, Hq, 1, 128]
  const uint16_t* k_mean;  // [pages, 128]
  const int32_t* table;    // [B, Hkv, max_blocks]
  const int32_t* lens;     // [B]
  int32_t* idx;            // [B, Hkv, topk]
  int32_t* num;            // [B, Hkv]
  int Hkv, group, pages, max_blocks, block, topk, n_first, n_near;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// A block's score in T: the largest over the group's heads, NaN if any is.  One warp, four
// heads at a time on 8 lanes each; every lane gets it.
template <typename T>
__device__ __forceinline__ T cache_score(const uint16_t* q, int group, const uint16_t* mean,
                                         int lane) {
  const uint4* kp = reinterpret_cast<const uint4*>(mean) + (lane & 7);
  const uint4 kw[2] = {read_global(kp), read_global(kp + 8)};
  T best = (T)-INFINITY;
  bool nan = false;
  for (int h0 = 0; h0 < group; h0 += 4) {
    const int h = min(h0 + (lane >> 3), group - 1);
    const uint4* qp = reinterpret_cast<const uint4*>(q + (long long)h * 128) + (lane & 7);
    const uint4 qw[2] = {read_global(qp), read_global(qp + 8)};
    T s = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t ku[4] = {kw[x].x, kw[x].y, kw[x].z, kw[x].w};
      const uint32_t qu[4] = {qw[x].x, qw[x].y, qw[x].z, qw[x].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        s = fma((T)bf16_lo(qu[y]), (T)bf16_lo(ku[y]), s);
        s = fma((T)bf16_hi(qu[y]), (T)bf16_hi(ku[y]), s);
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    nan |= s != s;
    best = s > best ? s : best;
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    const T y = __shfl_xor_sync(0xffffffffu, best, o);
    best = y > best ? y : best;
  }
  return __any_sync(0xffffffffu, nan) ? (T)NAN : best;
}

// A cluster of CTAs per (sequence, key/value head), up to 2048 blocks: the CTAs score the
// blocks between them on the tensor cores (16 blocks x 8 query heads a tile, the pages'
// means gathered through the table) into the first CTA's shared memory, as ordered 32-bit
// keys of the largest over the heads; the first CTA chooses.  The k-th key is found from
// one histogram of 256 even steps of value and a ranking of the step it falls into (where
// that holds too many, by radix descent); blocks inside the error band of it are scored
// again, in fp32 and where that leaves the order open in fp64.  Bound by latencies one
// after another (table, means, two cluster barriers, the histogram's barriers): 15.8 us for
// 128 rows of up to 1,536 blocks (ragged, 26 MB), where one CTA a row and a radix descent
// took 32.6 us.
__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(const CacheSelectArgs a) {
  after_predecessor();
  __shared__ uint32_t s_key[kMaxBlocks];
  __shared__ uint64_t s_key64[kMaxBlocks];
  __shared__ uint16_t s_cand[kMaxBlocks];
  __shared__ KthScratch s_kth;
  constexpr int kWarps = kSelThreads / 32, kMostCtas = 8;
  __shared__ uint32_t s_kmax[kMostCtas * kWarps], s_q1[kWarps], s_lo[kWarps], s_hi[kWarps];
  __shared__ uint32_t s_bad;
  __shared__ int s_n_cand, s_ok, s_forced;
  __shared__ uint32_t s_thr;
  __shared__ __align__(16) uint32_t s_members[kRanked];
  auto cluster = cooperative_groups::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, i4 = lane & 3;
  const long long bh = blockIdx.x / ctas;
  const int b = (int)(bh / a.Hkv);
  const long long len = max(0, a.lens[b]);
  const int n = (int)min((len + a.block - 1) / a.block, (long long)a.max_blocks);
  const uint16_t* q = a.q + bh * a.group * 128;
  const int32_t* table = a.table + bh * a.max_blocks;
  int32_t* out = a.idx + bh * a.topk;
  uint32_t* const first_key = cluster.map_shared_rank(s_key, 0);
  uint32_t* const first_kmax = cluster.map_shared_rank(s_kmax, 0);
  uint32_t* const first_bad = cluster.map_shared_rank(&s_bad, 0);

  if (tid == 0) s_n_cand = s_ok = s_forced = s_bad = 0;
  cluster.barrier_arrive();

  auto emit = [&](auto* keys, auto thr, int n_eq, int k) {
    partition_ascending(
        keys, n, thr, n_eq, s_kth, [&](int at, int e) { out[at] = e; }, [](int, int) {});
    for (int s = k + tid; s < a.topk; s += kSelThreads) out[s] = -1;
    if (tid == 0) a.num[bh] = k;
  };
  auto forced = [&](int e) { return e < a.n_first || e > n - 1 - a.n_near; };

  bool bad = false;
  __nv_bfloat162 kmax2 = as_bf162(0);
  float q1max = 0.0f;
  const int step = ctas * kWarps;
  uint4 qb[4];
  auto heads_from = [&](int h0) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      qb[j] = h0 + g < a.group
                  ? read_global(reinterpret_cast<const uint4*>(q + (long long)(h0 + g) * 128) +
                                i4 + 4 * j)
                  : make_uint4(0, 0, 0, 0);
  };
  auto page_of = [&](int t, int r) {
    const int e = t * 16 + g + 8 * r;
    return e < n ? read_global(table + e) : -1;
  };
  int page[2];
  uint4 ka[2][4];
  bool ok[2];
  auto means_at = [&]() {  // of page[]
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      ok[r] = page[r] >= 0 && page[r] < a.pages;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        ka[r][j] = ok[r] ? read_global(reinterpret_cast<const uint4*>(
                                           a.k_mean + (long long)page[r] * 128) +
                                       i4 + 4 * j)
                         : make_uint4(0, 0, 0, 0);
    }
  };
  // the first tile is fetched while the cluster's CTAs start: only the first CTA's shared
  // memory has to wait for that (15.8 us; 17.1 with the means behind the barrier, 18.6 with
  // all three there)
#pragma unroll
  for (int r = 0; r < 2; ++r) page[r] = page_of(rank * kWarps + warp, r);
  heads_from(0);
  means_at();
  bool fetched = true;
  cluster.barrier_wait();  // the first CTA runs and has cleared s_bad
  for (int h0 = 0; h0 < a.group; h0 += 8) {
    if (h0 > 0) {
      heads_from(h0);
#pragma unroll
      for (int r = 0; r < 2; ++r) page[r] = page_of(rank * kWarps + warp, r);
    }
    float q1 = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u[4] = {qb[j].x, qb[j].y, qb[j].z, qb[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) q1 += fabsf(bf16_lo(u[e])) + fabsf(bf16_hi(u[e]));
    }
    q1 += __shfl_xor_sync(0xffffffffu, q1, 1);
    q1 += __shfl_xor_sync(0xffffffffu, q1, 2);
    q1max = fmaxf(q1max, q1);
    bad |= !(q1 < kFinite);
    const bool c0 = h0 + 2 * i4 < a.group, c1 = h0 + 2 * i4 + 1 < a.group;
    for (int t = rank * kWarps + warp; t * 16 < n; t += step) {
      float d[4] = {};
      if (!fetched) means_at();
      fetched = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) page[r] = page_of(t + step, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mma_bf16(d, ka[0][j].x, ka[1][j].x, ka[0][j].y, ka[1][j].y, qb[j].x, qb[j].y);
        mma_bf16(d, ka[0][j].z, ka[1][j].z, ka[0][j].w, ka[1][j].w, qb[j].z, qb[j].w);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          kmax2 = __hmax2(kmax2, __habs2(as_bf162(ka[r][j].x)));
          kmax2 = __hmax2(kmax2, __habs2(as_bf162(ka[r][j].y)));
          kmax2 = __hmax2(kmax2, __habs2(as_bf162(ka[r][j].z)));
          kmax2 = __hmax2(kmax2, __habs2(as_bf162(ka[r][j].w)));
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x = max_nan(c0 ? d[2 * r] : -INFINITY, c1 ? d[2 * r + 1] : -INFINITY);
        x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, 2));
        const int e = t * 16 + g + 8 * r;
        if (i4 == 0 && e < n) {
          bad |= ok[r] && !(fabsf(x) < kFinite);
          uint32_t key = ok[r] ? order32(x) : 0u;
          if (h0 > 0) key = max(key, first_key[e]);  // this thread's own, of the heads before
          first_key[e] = key;
        }
      }
    }
  }
  {
    const float m = fmaxf(__low2float(kmax2), __high2float(kmax2));
    const uint32_t mm = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
    const uint32_t qq = __reduce_max_sync(0xffffffffu, __float_as_uint(q1max));
    if (lane == 0) {
      first_kmax[rank * kWarps + warp] = mm;
      s_q1[warp] = qq;
    }
    if (bad) atomicOr(first_bad, 1u);
  }
  cluster.sync();
  if (rank != 0) return;

  uint32_t km = 0, qm = 0;
  for (int w = 0; w < ctas * kWarps; ++w) km = max(km, s_kmax[w]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) qm = max(qm, s_q1[w]);
  const float sum_bound = __uint_as_float(qm) * __uint_as_float(km);
  const float eps = kDotBound * sum_bound + kTiny;

  if (s_bad != 0 || !(sum_bound < kFinite)) {  // scores that overflow fp32, or are not numbers
    int n_ok = 0;
    for (int e = warp; e < n; e += kWarps) {
      uint64_t key = 0;
      const int page = read_global(table + e);
      if (page >= 0 && page < a.pages)
        key = forced(e) ? kForced64
                        : order64(cache_score<double>(
                              q, a.group, a.k_mean + (long long)page * 128, lane));
      if (lane == 0) s_key64[e] = key;
    }
    __syncthreads();
    for (int e0 = 0; e0 < n; e0 += kSelThreads)
      n_ok += __syncthreads_count(e0 + tid < n && s_key64[e0 + tid] != 0);
    const int k = min(a.topk, n_ok);
    uint64_t thr = 0;
    int larger = 0;
    if (n_ok > a.topk) kth_largest<uint64_t>(s_key64, n, k, s_kth, &thr, &larger);
    emit(s_key64, thr, n_ok > a.topk ? k - larger : 0, k);
    return;
  }
  // mark the forced ones; count, and the least and largest of the others
  {
    int ok = 0, sure = 0;
    uint32_t lo = kForced32, hi = 0;
    for (int e = tid; e < n; e += kSelThreads) {
      const uint32_t key = s_key[e];
      if (key == 0) continue;
      ++ok;
      if (forced(e)) {
        s_key[e] = kForced32;
        ++sure;
      } else {
        lo = min(lo, key);
        hi = max(hi, key);
      }
    }
    ok = __reduce_add_sync(0xffffffffu, ok);
    sure = __reduce_add_sync(0xffffffffu, sure);
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      atomicAdd(&s_ok, ok);
      atomicAdd(&s_forced, sure);
      s_lo[warp] = lo;
      s_hi[warp] = hi;
    }
  }
  s_kth.hist[tid] = 0;
  __syncthreads();
  const int n_ok = s_ok, k = min(a.topk, n_ok);
  if (n_ok <= a.topk) {
    emit(s_key, 0u, 0, k);
    return;
  }
  if (s_forced >= k) {  // more forced blocks than places
    emit(s_key, kForced32, k, k);
    return;
  }
  uint32_t lo_key = kForced32, hi_key = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    lo_key = min(lo_key, s_lo[w]);
    hi_key = max(hi_key, s_hi[w]);
  }
  // 256 even steps of value: the step of a key never falls as the key grows
  const float low = unorder32(lo_key), span = unorder32(hi_key) - low;
  const float per = span > 0.0f && span < kFinite ? 255.0f / span : 0.0f;
  auto step_of = [&](uint32_t key) {
    return min(255, (int)((unorder32(key) - low) * per));
  };
  for (int e = tid; e < n; e += kSelThreads) {
    const uint32_t key = s_key[e];
    if (key != 0 && key != kForced32) atomicAdd(&s_kth.hist[step_of(key)], 1u);
  }
  __syncthreads();
  const int rest = k - s_forced;
  if (warp == 0) digit_of(s_kth, rest, lane);
  __syncthreads();
  const int digit = s_kth.digit, within = s_kth.rest, members = s_kth.count;
  uint32_t thr;
  int larger;
  if (members <= kRanked && per < INFINITY) {
    for (int e = tid; e < n; e += kSelThreads) {
      const uint32_t key = s_key[e];
      if (key != 0 && key != kForced32 && step_of(key) == digit)
        s_members[atomicAdd(&s_n_cand, 1)] = key;
    }
    rank_members(s_members, members, within, s_kth, &s_thr);
    thr = s_thr;
    larger = k - s_kth.rest;
    if (tid == 0) s_n_cand = 0;
  } else {
    kth_largest<uint32_t>(s_key, n, k, s_kth, &thr, &larger);
  }
  if (qm == 0 || km == 0) {  // every score is 0
    emit(s_key, thr, k - larger, k);
    return;
  }
  const float t = unorder32(thr);
  const uint32_t hi = order32(__fadd_ru(t, 2.0f * eps)), lo = order32(__fadd_rd(t, -2.0f * eps));
  // above the band in the low half, inside it in the high half
  unsigned int mine = 0;
  for (int e = tid; e < n; e += kSelThreads) {
    const uint32_t key = s_key[e];
    mine += key > hi ? 1u : (key >= lo ? 0x10000u : 0u);
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  __syncthreads();
  if (lane == 0) s_kth.warp_sum[warp] = mine;
  __syncthreads();
  unsigned int both = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) both += s_kth.warp_sum[w];
  const int n_cand = (int)(both >> 16), need = k - (int)(both & 0xffffu);
  if (n_cand == need) {
    emit(s_key, lo - 1, 0, k);
    return;
  }
  for (int e = tid; e < n; e += kSelThreads)
    if (s_key[e] >= lo && s_key[e] <= hi) s_cand[atomicAdd(&s_n_cand, 1)] = (uint16_t)e;
  __syncthreads();
  for (int e = tid; e < n; e += kSelThreads) s_key[e] = s_key[e] > hi ? 2u : 0u;
  // the candidates' scores from fp32 sums of 19 roundings at most, and from fp64 where the
  // border's gap is not beyond those
  auto mean_of = [&](int c) { return a.k_mean + (long long)read_global(table + s_cand[c]) * 128; };
  const float tight = 2.0f * 19.5f * 5.9604645e-8f * sum_bound + kTiny;
  for (int pass = 0; pass < 2; ++pass) {
    for (int c = warp; c < n_cand; c += kWarps) {
      const uint64_t key = pass == 0 ? order32(cache_score<float>(q, a.group, mean_of(c), lane))
                                     : order64(cache_score<double>(q, a.group, mean_of(c), lane));
      if (lane == 0) s_key64[c] = key;
    }
    __syncthreads();
    for (int c = tid; c < n_cand; c += kSelThreads) {
      const uint64_t own = s_key64[c];
      const int e = s_cand[c];
      int place = 0;
      for (int o = 0; o < n_cand; ++o)
        place += s_key64[o] > own || (s_key64[o] == own && s_cand[o] < e);
      s_key[e] = place < need ? 2u : 0u;
      if (place == need - 1) s_lo[0] = (uint32_t)own;
      if (place == need) s_hi[0] = (uint32_t)own;
    }
    __syncthreads();
    if (pass == 0 && unorder32(s_lo[0]) - unorder32(s_hi[0]) > tight) break;
    __syncthreads();  // both ends are read before they are written again
  }
  emit(s_key, 1u, 0, k);
}

}  // namespace vsa

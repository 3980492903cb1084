// vsa_select_kernel.cuh -- block means and the choice of key blocks by a cheap score.
//
//   block_mean_kernel    m_j = (1/n_j) sum of the block's first n_j tokens (bf16 in and out,
//                        fp32 sums)
//   select_kernel        LUT rows: the topk key blocks j of highest q_mean_i . k_mean_j
//   cache_select_kernel  the same for one token per sequence over the pages of a cache
//
// The choice is that of the real numbers, ties to the lowest index: scores are first
// computed on the tensor cores with fp32 sums, and only where the error bound of that
// arithmetic leaves the border open are the blocks near it scored again (fp32 with a
// tighter bound, then fp64, in which the products of bf16 values are exact).
#pragma once

#include <cuda_bf16.h>

#include "vsa_warp_ptx.cuh"

namespace vsa {

// ------------------------------------------------------------------ block means
// One CTA per block, 8 rows a thread: a thread holds 8 of the 128 columns (16 bytes) of
// rows t/16, t/16 + threads/16, ...  The 8 loads of a thread are independent.
template <int BLOCK>
__global__ void __launch_bounds__(BLOCK * 2)
    block_mean_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ sizes, int S,
                      int nb, uint16_t* __restrict__ mean) {
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
    w[i] = r < n ? __ldg(src + r * 16) : make_uint4(0, 0, 0, 0);
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

constexpr int kSelThreads = 256;

struct KthScratch {
  unsigned int hist[256];
  unsigned int warp_sum[kSelThreads / 32];
  int digit, rest;
};

// The k-th largest of keys[0..n) (1 <= k <= n) and how many keys are larger: a radix
// descent, 8 bits a pass.  Every thread of the CTA calls it and gets the same answer.
template <typename K>
__device__ void kth_largest(const K* keys, int n, int k, KthScratch& s, K* thr, int* larger) {
  K prefix = 0, mask = 0;
  int rest = k;
  for (int shift = 8 * (int)sizeof(K) - 8; shift >= 0; shift -= 8) {
    s.hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kSelThreads) {
      const K key = keys[i];
      if ((key & mask) == prefix) atomicAdd(&s.hist[(unsigned)(key >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      // lane l holds digits 255-8l down to 248-8l
      unsigned int h[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[e] = s.hist[255 - 8 * (int)threadIdx.x - e];
        sum += h[e];
      }
      unsigned int upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned int y = __shfl_up_sync(0xffffffffu, upto, o);
        if ((int)threadIdx.x >= o) upto += y;
      }
      unsigned int before = upto - sum;
      if (before < (unsigned)rest && upto >= (unsigned)rest) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (before < (unsigned)rest && before + h[e] >= (unsigned)rest) {
            s.digit = 255 - 8 * (int)threadIdx.x - e;
            s.rest = rest - (int)before;
          }
          before += h[e];
        }
      }
    }
    __syncthreads();
    prefix |= (K)s.digit << shift;
    mask |= (K)255 << shift;
    rest = s.rest;
  }
  *thr = prefix;
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
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w)
    if (w < warp) before += s.warp_sum[w];
  return before + x - v;
}

// Ascending walk over keys[0..n): those above `thr` and the first `n_eq` equal to it go to
// chosen(position, i), the others to rest(position, i).
template <typename K, typename F, typename R>
__device__ void partition_ascending(const K* keys, int n, K thr, int n_eq, KthScratch& s,
                                    F chosen, R rest) {
  const int per = (n + kSelThreads - 1) / kSelThreads;
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

constexpr int kSelRows = 32;

__host__ __device__ constexpr int select_stride(int nreg) { return nreg * 64 + 8; }
__host__ __device__ constexpr size_t select_smem(int nreg) {
  return (size_t)kSelRows * select_stride(nreg) * 2;
}

// Whether block e may be chosen by a row whose diagonal is d, and whether it must be.
__device__ __forceinline__ bool select_allowed(const SelectArgs& a, int e, int d) {
  return e >= 0 && e < a.nk && (a.sizes == nullptr || a.sizes[e] > 0) && (!a.causal || e <= d);
}
__device__ __forceinline__ bool select_forced(const SelectArgs& a, int e, int d) {
  return e < a.n_first || (e > d - a.n_near && e < d + a.n_near);
}

__device__ __forceinline__ uint16_t bf16_unorder(uint32_t o) {
  return (uint16_t)((o & 0x8000u) ? o & 0x7fffu : ~o & 0xffffu);
}
__device__ __forceinline__ uint32_t bf16_pair(uint16_t b) { return (uint32_t)b << 16 | b; }
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) {
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) {
  return *reinterpret_cast<const uint32_t*>(&v);
}

// How many of the warp's 64*NREG keys are >= the threshold (NaN keys never count).
template <int NREG>
__device__ __forceinline__ int count_ge(const uint32_t (&key)[NREG], uint16_t thr) {
  const __nv_bfloat162 t = as_bf162(bf16_pair(thr));
  __nv_bfloat162 c = as_bf162(0);  // at most NREG <= 32 per half: exact
#pragma unroll
  for (int j = 0; j < NREG; ++j) c = __hadd2(c, __hge2(as_bf162(key[j]), t));
  return __reduce_add_sync(0xffffffffu, (int)(__low2float(c) + __high2float(c)));
}

// One CTA: 32 query-block rows of one head against all nk <= 64*NREG key blocks.
//   1. scores on the tensor cores: a warp holds the 32 rows' operands in registers and
//      walks key tiles of 8; scores go to shared memory rounded to bf16 (32 x nk x 2 bytes
//      fit where fp32 would not; the rounding only widens the band that is scored again).
//      Operands are read 16 bytes a thread with the contraction index permuted the same
//      way on both sides, so no shuffle or transposition is needed.
//   2. a warp per row: 64*NREG keys in NREG registers of pairs; the k-th largest key by
//      bisection over the 16-bit order; blocks surely above it are in, the others within
//      the error bound are scored again.
template <int NREG>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) uint16_t s_key[];  // [32][stride]
  constexpr int kStride = select_stride(NREG);
  __shared__ float s_q1[kSelRows];
  __shared__ uint32_t s_kmax[kSelThreads / 32];
  __shared__ unsigned int s_slow;
  __shared__ uint16_t s_cand[kSelThreads / 32][32];
  __shared__ KthScratch s_kth;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, i4 = lane & 3;
  const long long bh = blockIdx.x / a.tiles;  // b * Hq + hq
  const int row0 = (int)(blockIdx.x - bh * a.tiles) * kSelRows;
  const long long b = bh / a.Hq;
  const int hkv = (int)(bh - b * a.Hq) / a.group;
  const uint16_t* qh = a.q + (bh * a.nq) * 128;
  const uint16_t* kh = a.k + ((b * a.Hkv + hkv) * (long long)a.nk) * 128;
  if (tid == 0) s_slow = 0;

  // rows g, g+8, g+16, g+24; 16-byte chunks i4, i4+4, i4+8, i4+12
  uint4 qa[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = row0 + g + 8 * r;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      qa[r][j] = row < a.nq
                     ? __ldg(reinterpret_cast<const uint4*>(qh + (long long)row * 128) + i4 + 4 * j)
                     : make_uint4(0, 0, 0, 0);
  }
  if (warp == 0) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u[4] = {qa[r][j].x, qa[r][j].y, qa[r][j].z, qa[r][j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) s += fabsf(bf16_lo(u[e])) + fabsf(bf16_hi(u[e]));
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (i4 == 0) s_q1[g + 8 * r] = s;
    }
  }
  __syncthreads();

  // scores
  {
    const int nt = (a.nk + 7) / 8;
    __nv_bfloat162 kmax = as_bf162(0);
    bool bad[4] = {false, false, false, false};
    uint4 kb[4];
    auto load = [&](int t) {
      const int key = t * 8 + g;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        kb[j] = key < a.nk
                    ? __ldg(reinterpret_cast<const uint4*>(kh + (long long)key * 128) + i4 + 4 * j)
                    : make_uint4(0, 0, 0, 0);
    };
    if (warp < nt) load(warp);
    for (int t = warp; t < nt; t += kSelThreads / 32) {
      uint4 cur[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) cur[j] = kb[j];
      if (t + kSelThreads / 32 < nt) load(t + kSelThreads / 32);
      float d0[4] = {}, d1[4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mma_bf16(d0, qa[0][j].x, qa[1][j].x, qa[0][j].y, qa[1][j].y, cur[j].x, cur[j].y);
        mma_bf16(d1, qa[2][j].x, qa[3][j].x, qa[2][j].y, qa[3][j].y, cur[j].x, cur[j].y);
        mma_bf16(d0, qa[0][j].z, qa[1][j].z, qa[0][j].w, qa[1][j].w, cur[j].z, cur[j].w);
        mma_bf16(d1, qa[2][j].z, qa[3][j].z, qa[2][j].w, qa[3][j].w, cur[j].z, cur[j].w);
        kmax = __hmax2(kmax, __habs2(as_bf162(cur[j].x)));
        kmax = __hmax2(kmax, __habs2(as_bf162(cur[j].y)));
        kmax = __hmax2(kmax, __habs2(as_bf162(cur[j].z)));
        kmax = __hmax2(kmax, __habs2(as_bf162(cur[j].w)));
      }
      uint16_t* out = s_key + t * 8 + 2 * i4;
      auto put = [&](int r, float x, float y) {
        bad[r] |= !(fabsf(x) < kFinite) | !(fabsf(y) < kFinite);
        *reinterpret_cast<uint32_t*>(out + (g + 8 * r) * kStride) =
            as_u32(__floats2bfloat162_rn(x, y));
      };
      put(0, d0[0], d0[1]);
      put(1, d0[2], d0[3]);
      put(2, d1[0], d1[1]);
      put(3, d1[2], d1[3]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (bad[r]) atomicOr(&s_slow, 1u << (g + 8 * r));
    const float m = fmaxf(__low2float(kmax), __high2float(kmax));
    const uint32_t mm = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
    if (lane == 0) s_kmax[warp] = mm;
  }
  __syncthreads();
  // what may not be chosen by any row
  for (int e = tid; e < NREG * 64; e += kSelThreads)
    if (e >= a.nk || (a.sizes != nullptr && a.sizes[e] <= 0))
      for (int r = 0; r < kSelRows; ++r) s_key[r * kStride + e] = 0x7fff;
  __syncthreads();

  uint32_t kmax_bits = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) kmax_bits = max(kmax_bits, s_kmax[w]);
  const float kmax = __uint_as_float(kmax_bits);
  const unsigned int lt = (1u << lane) - 1u;

  for (int r = warp; r < kSelRows; r += kSelThreads / 32) {
    const int row = row0 + r;
    if (row >= a.nq) break;
    if ((s_slow >> r) & 1u) continue;
    const float q1 = s_q1[r], eps = kDotBound * q1 * kmax + kTiny;
    if (!(q1 * kmax < kFinite)) {
      if (lane == 0) atomicOr(&s_slow, 1u << r);
      continue;
    }
    const int d = row + a.nk - a.nq;
    uint16_t* krow = s_key + r * kStride;
    for (int e = lane; e < min(a.n_first, a.nk); e += 32)
      if (select_allowed(a, e, d)) krow[e] = 0x7f80;
    for (int e = max(0, d - a.n_near + 1) + lane; e < min(a.nk, d + a.n_near); e += 32)
      if (select_allowed(a, e, d)) krow[e] = 0x7f80;
    __syncwarp();
    uint32_t key[NREG];
#pragma unroll
    for (int j = 0; j < NREG; ++j) {
      key[j] = reinterpret_cast<const uint32_t*>(krow)[j * 32 + lane];
      if (a.causal) {
        const int e = 2 * (j * 32 + lane);
        if (e > d) key[j] |= 0x00007fffu;
        if (e + 1 > d) key[j] |= 0x7fff0000u;
      }
    }
    const int n_ok = count_ge<NREG>(key, 0xff80);  // all but the NaN keys
    const int k = min(a.topk, n_ok);
    uint32_t in_lo = 0, in_hi = 0, cand_lo = 0, cand_hi = 0;
    int by_index = 0;  // candidates to take from the lowest index on
    bool slow = false;
    if (n_ok <= a.topk) {
#pragma unroll
      for (int j = 0; j < NREG; ++j) {
        in_lo |= (uint32_t)((key[j] & 0x7fffu) <= 0x7f80u) << j;
        in_hi |= (uint32_t)((key[j] >> 16 & 0x7fffu) <= 0x7f80u) << j;
      }
    } else {
      // largest t with count(>= t) >= k, over the order of bf16 values
      uint32_t lo = 0x007fu, hi = 0xff81u;
      while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (count_ge<NREG>(key, bf16_unorder(mid)) >= k) lo = mid; else hi = mid;
      }
      const float t = __uint_as_float((uint32_t)bf16_unorder(lo) << 16);
      uint32_t in_thr, cand_thr;  // in: key > in_thr, candidate: the others >= cand_thr
      bool ties = true;
      if (isinf(t)) {
        in_thr = cand_thr = 0x7f80u;  // more forced blocks than places
      } else if (q1 == 0.0f || kmax == 0.0f) {
        in_thr = cand_thr = (uint32_t)bf16_unorder(lo);  // every score is 0
      } else {
        // bf16 rounding is off by at most 2^-9 of the value; s - bound(s) and s + bound(s)
        // grow with s, so the true k-th score lies between those of t
        ties = false;
        const float c = 0.00196f;
        const float up = t + c * fabsf(t) + 2.0f * eps, dn = t - c * fabsf(t) - 2.0f * eps;
        in_thr = __bfloat16_as_ushort(__float2bfloat16_ru(up / (up > 0.0f ? 1.0f - c : 1.0f + c)));
        cand_thr = __bfloat16_as_ushort(__float2bfloat16_rd(dn / (dn > 0.0f ? 1.0f + c : 1.0f - c)));
      }
      const __nv_bfloat162 ti = as_bf162(bf16_pair((uint16_t)in_thr));
      const __nv_bfloat162 tc = as_bf162(bf16_pair((uint16_t)cand_thr));
#pragma unroll
      for (int j = 0; j < NREG; ++j) {
        const uint32_t gi = __hgt2_mask(as_bf162(key[j]), ti);
        const uint32_t gc = __hge2_mask(as_bf162(key[j]), tc) & ~gi;
        in_lo |= (gi & 1u) << j;
        in_hi |= (gi >> 31) << j;
        cand_lo |= (gc & 1u) << j;
        cand_hi |= (gc >> 31) << j;
      }
      const int n_in = __reduce_add_sync(0xffffffffu, __popc(in_lo) + __popc(in_hi));
      const int n_cand = __reduce_add_sync(0xffffffffu, __popc(cand_lo) + __popc(cand_hi));
      const int need = k - n_in;
      if (n_cand == need) {
        in_lo |= cand_lo;
        in_hi |= cand_hi;
        cand_lo = cand_hi = 0;
      } else if (ties) {
        by_index = need;
      } else if (n_cand > 32) {
        slow = true;
      } else {
        // gather the candidates' indices, one per lane
        int at = 0;
#pragma unroll
        for (int j = 0; j < NREG; ++j) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const bool c = ((p ? cand_hi : cand_lo) >> j) & 1u;
            const unsigned int m = __ballot_sync(0xffffffffu, c);
            if (c) s_cand[warp][at + __popc(m & lt)] = (uint16_t)(2 * (j * 32 + lane) + p);
            at += __popc(m);
          }
        }
        __syncwarp();
        const int mine = lane < n_cand ? s_cand[warp][lane] : 0x7fffffff;
        const uint2 qw = __ldg(reinterpret_cast<const uint2*>(qh + (long long)row * 128) + lane);
        const float qf[4] = {bf16_lo(qw.x), bf16_hi(qw.x), bf16_lo(qw.y), bf16_hi(qw.y)};
        // fp32 sums of 128 exact products: 4 in a lane, 5 levels across lanes
        float sc = 0.0f;
        for (int c = 0; c < n_cand; ++c) {
          const uint2 kw = __ldg(
              reinterpret_cast<const uint2*>(kh + (long long)s_cand[warp][c] * 128) + lane);
          float s = qf[0] * bf16_lo(kw.x);
          s = fmaf(qf[1], bf16_hi(kw.x), s);
          s = fmaf(qf[2], bf16_lo(kw.y), s);
          s = fmaf(qf[3], bf16_hi(kw.y), s);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (lane == c) sc = s;
        }
        int rank = 0;
        for (int c = 0; c < n_cand; ++c) {
          const float o = __shfl_sync(0xffffffffu, sc, c);
          const int oi = __shfl_sync(0xffffffffu, mine, c);
          rank += o > sc || (o == sc && oi < mine);
        }
        bool take = lane < n_cand && rank < need;
        // 9 roundings of partial sums of at most sum |q||k|
        const float tight = 2.0f * 9.5f * 5.9604645e-8f * q1 * kmax + kTiny;
        float worst_in = take ? sc : INFINITY, best_out = lane < n_cand && !take ? sc : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          worst_in = fminf(worst_in, __shfl_xor_sync(0xffffffffu, worst_in, o));
          best_out = fmaxf(best_out, __shfl_xor_sync(0xffffffffu, best_out, o));
        }
        if (worst_in - best_out <= tight) {
          double sd = 0.0;
          for (int c = 0; c < n_cand; ++c) {
            const uint2 kw = __ldg(
                reinterpret_cast<const uint2*>(kh + (long long)s_cand[warp][c] * 128) + lane);
            double s = (double)qf[0] * (double)bf16_lo(kw.x);
            s = fma((double)qf[1], (double)bf16_hi(kw.x), s);
            s = fma((double)qf[2], (double)bf16_lo(kw.y), s);
            s = fma((double)qf[3], (double)bf16_hi(kw.y), s);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == c) sd = s;
          }
          rank = 0;
          for (int c = 0; c < n_cand; ++c) {
            const double o = __shfl_sync(0xffffffffu, sd, c);
            const int oi = __shfl_sync(0xffffffffu, mine, c);
            rank += o > sd || (o == sd && oi < mine);
          }
          take = lane < n_cand && rank < need;
        }
        cand_lo = cand_hi = 0;
        unsigned int taken = __ballot_sync(0xffffffffu, take);
        while (taken != 0) {
          const int e = s_cand[warp][__ffs(taken) - 1];
          taken &= taken - 1;
          if (((e >> 1) & 31) == lane) {
            if (e & 1) in_hi |= 1u << (e >> 6); else in_lo |= 1u << (e >> 6);
          }
        }
        __syncwarp();
      }
    }
    if (slow) {
      if (lane == 0) atomicOr(&s_slow, 1u << r);
      continue;
    }
    // ascending indices, -1 behind
    int32_t* out = a.idx + (bh * a.nq + row) * (long long)a.topk;
    int at = 0, seen = 0;
#pragma unroll
    for (int j = 0; j < NREG; ++j) {
      bool lo = (in_lo >> j) & 1u, hi = (in_hi >> j) & 1u;
      if (by_index > 0) {
        const bool cl = (cand_lo >> j) & 1u, ch = (cand_hi >> j) & 1u;
        const unsigned int ml = __ballot_sync(0xffffffffu, cl), mh = __ballot_sync(0xffffffffu, ch);
        const int before = seen + __popc(ml & lt) + __popc(mh & lt);
        lo |= cl && before < by_index;
        hi |= ch && before + cl < by_index;
        seen += __popc(ml) + __popc(mh);
      }
      const unsigned int ml = __ballot_sync(0xffffffffu, lo), mh = __ballot_sync(0xffffffffu, hi);
      const int pos = at + __popc(ml & lt) + __popc(mh & lt), e = 2 * (j * 32 + lane);
      if (lo) out[pos] = e;
      if (hi) out[pos + lo] = e + 1;
      at += __popc(ml) + __popc(mh);
    }
    for (int s = k + lane; s < a.topk; s += 32) out[s] = -1;
    if (lane == 0) a.num[bh * a.nq + row] = k;
  }
  __syncthreads();

  // Rows whose fp32 scores overflow, or with more than 32 blocks inside the error band
  // (equal blocks, say): every score in fp64, one row at a time by the whole CTA.
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
    for (int e0 = 0; e0 < a.nk; e0 += kSelThreads) {
      const int e = e0 + tid;
      uint64_t key = 0;
      if (e < a.nk && select_allowed(a, e, d)) {
        if (select_forced(a, e, d)) {
          key = kForced64;
        } else {
          const uint32_t* qp = reinterpret_cast<const uint32_t*>(qh + (long long)row * 128);
          const uint32_t* kp = reinterpret_cast<const uint32_t*>(kh + (long long)e * 128);
          double s = 0.0;
#pragma unroll 8
          for (int c = 0; c < 64; ++c) {
            const uint32_t qw = __ldg(qp + c), kw = __ldg(kp + c);
            s = fma((double)bf16_lo(qw), (double)bf16_lo(kw), s);
            s = fma((double)bf16_hi(qw), (double)bf16_hi(kw), s);
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
        key64, a.nk, thr, n_ok > a.topk ? k - larger : 0, s_kth, [&](int at, int e) { out[at] = e; },
        [](int, int) {});
    for (int s = k + tid; s < a.topk; s += kSelThreads) out[s] = -1;
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

constexpr int kMaxBlocks = 2048;

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The exact score of a block: the largest over the group's heads (NaN if any is), as an
// ordered whole number.  One warp.
__device__ __forceinline__ uint64_t cache_score64(const uint16_t* q, int group,
                                                  const uint16_t* mean, int lane) {
  const uint2 kw = __ldg(reinterpret_cast<const uint2*>(mean) + lane);
  const double k0 = bf16_lo(kw.x), k1 = bf16_hi(kw.x), k2 = bf16_lo(kw.y), k3 = bf16_hi(kw.y);
  double best = -INFINITY;
  bool nan = false;
  for (int h = 0; h < group; ++h) {
    const uint2 qw = __ldg(reinterpret_cast<const uint2*>(q + (long long)h * 128) + lane);
    double s = (double)bf16_lo(qw.x) * k0;
    s = fma((double)bf16_hi(qw.x), k1, s);
    s = fma((double)bf16_lo(qw.y), k2, s);
    s = fma((double)bf16_hi(qw.y), k3, s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    nan |= s != s;
    best = fmax(best, s);
  }
  return nan ? 0 : order64(best);
}

// One CTA per (sequence, key/value head): scores of its n <= 2048 blocks on the tensor
// cores (16 blocks x 8 query heads a tile, the pages' means gathered through the table),
// the largest over the heads as an ordered 32-bit key in shared memory, then a radix
// descent to the k-th; blocks inside the error band of it are scored again in fp64.
__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(const CacheSelectArgs a) {
  __shared__ uint32_t s_key[kMaxBlocks];
  __shared__ uint64_t s_key64[kMaxBlocks];
  __shared__ uint16_t s_cand[kMaxBlocks];
  __shared__ KthScratch s_kth;
  __shared__ uint32_t s_kmax[kSelThreads / 32], s_q1[kSelThreads / 32];
  __shared__ int s_n_cand;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, i4 = lane & 3;
  const long long bh = blockIdx.x;
  const int b = (int)(bh / a.Hkv);
  int len = a.lens[b];
  len = len < 0 ? 0 : len;
  const int n = (int)min(((long long)len + a.block - 1) / a.block, (long long)a.max_blocks);
  const uint16_t* q = a.q + bh * a.group * 128;
  const int32_t* table = a.table + bh * a.max_blocks;
  int32_t* out = a.idx + bh * a.topk;

  auto emit = [&](auto* keys, auto thr, int n_eq, int k) {
    partition_ascending(
        keys, n, thr, n_eq, s_kth, [&](int at, int e) { out[at] = e; }, [](int, int) {});
    for (int s = k + tid; s < a.topk; s += kSelThreads) out[s] = -1;
    if (tid == 0) a.num[bh] = k;
  };
  if (tid == 0) s_n_cand = 0;

  bool bad = false;
  __nv_bfloat162 kmax2 = as_bf162(0);
  float q1max = 0.0f;
  for (int h0 = 0; h0 < a.group; h0 += 8) {
    uint4 qb[4];
    float q1 = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      qb[j] = h0 + g < a.group
                  ? __ldg(reinterpret_cast<const uint4*>(q + (long long)(h0 + g) * 128) + i4 + 4 * j)
                  : make_uint4(0, 0, 0, 0);
      const uint32_t u[4] = {qb[j].x, qb[j].y, qb[j].z, qb[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) q1 += fabsf(bf16_lo(u[e])) + fabsf(bf16_hi(u[e]));
    }
    q1 += __shfl_xor_sync(0xffffffffu, q1, 1);
    q1 += __shfl_xor_sync(0xffffffffu, q1, 2);
    q1max = fmaxf(q1max, q1);
    bad |= !(q1 < kFinite);
    for (int t = warp; t * 16 < n; t += kSelThreads / 32) {
      float d[4] = {};
      uint4 ka[2][4];
      bool ok[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int e = t * 16 + g + 8 * r;
        const int page = e < n ? __ldg(table + e) : -1;
        ok[r] = page >= 0 && page < a.pages;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ka[r][j] = ok[r] ? __ldg(reinterpret_cast<const uint4*>(a.k_mean + (long long)page * 128) +
                                   i4 + 4 * j)
                           : make_uint4(0, 0, 0, 0);
      }
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
      const bool c0 = h0 + 2 * i4 < a.group, c1 = h0 + 2 * i4 + 1 < a.group;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x = max_nan(c0 ? d[2 * r] : -INFINITY, c1 ? d[2 * r + 1] : -INFINITY);
        x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, 2));
        const int e = t * 16 + g + 8 * r;
        if (i4 == 0 && e < n) {
          bad |= ok[r] && !(fabsf(x) < kFinite);
          const uint32_t key = ok[r] ? order32(x) : 0u;
          s_key[e] = h0 == 0 ? key : max(s_key[e], key);
        }
      }
    }
  }
  {
    const float m = fmaxf(__low2float(kmax2), __high2float(kmax2));
    const uint32_t mm = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
    const uint32_t qq = __reduce_max_sync(0xffffffffu, __float_as_uint(q1max));
    if (lane == 0) {
      s_kmax[warp] = mm;
      s_q1[warp] = qq;
    }
  }
  const bool any_bad = __syncthreads_or(bad);
  uint32_t km = 0, qm = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    km = max(km, s_kmax[w]);
    qm = max(qm, s_q1[w]);
  }
  const float sum_bound = __uint_as_float(qm) * __uint_as_float(km);
  const float eps = kDotBound * sum_bound + kTiny;
  auto forced = [&](int e) { return e < a.n_first || e > n - 1 - a.n_near; };
  int n_ok = 0;
  for (int e0 = 0; e0 < n; e0 += kSelThreads) {
    const int e = e0 + tid;
    bool ok = false;
    if (e < n) {
      ok = s_key[e] != 0;
      if (ok && forced(e)) s_key[e] = kForced32;
    }
    n_ok += __syncthreads_count(ok);
  }

  if (any_bad || !(sum_bound < kFinite)) {  // scores that overflow fp32, or are not numbers
    n_ok = 0;
    for (int e = warp; e < n; e += kSelThreads / 32) {
      uint64_t key = 0;
      const int page = __ldg(table + e);
      if (page >= 0 && page < a.pages)
        key = forced(e) ? kForced64
                        : cache_score64(q, a.group, a.k_mean + (long long)page * 128, lane);
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
  const int k = min(a.topk, n_ok);
  if (n_ok <= a.topk) {
    emit(s_key, 0u, 0, k);
    return;
  }
  uint32_t thr;
  int larger;
  kth_largest<uint32_t>(s_key, n, k, s_kth, &thr, &larger);
  if (thr == kForced32 || qm == 0 || km == 0) {
    emit(s_key, thr, k - larger, k);
    return;
  }
  const float t = unorder32(thr);
  const uint32_t hi = order32(__fadd_ru(t, 2.0f * eps)), lo = order32(__fadd_rd(t, -2.0f * eps));
  int n_in = 0, n_cand = 0;
  for (int e0 = 0; e0 < n; e0 += kSelThreads) {
    const uint32_t key = e0 + tid < n ? s_key[e0 + tid] : 0u;
    n_in += __syncthreads_count(key > hi);
    n_cand += __syncthreads_count(key >= lo && key <= hi);
  }
  const int need = k - n_in;
  if (n_cand == need) {
    emit(s_key, lo - 1, 0, k);
    return;
  }
  for (int e = tid; e < n; e += kSelThreads)
    if (s_key[e] >= lo && s_key[e] <= hi) s_cand[atomicAdd(&s_n_cand, 1)] = (uint16_t)e;
  __syncthreads();
  for (int c = warp; c < n_cand; c += kSelThreads / 32) {
    const uint64_t key = cache_score64(
        q, a.group, a.k_mean + (long long)__ldg(table + s_cand[c]) * 128, lane);
    if (lane == 0) s_key64[c] = key;
  }
  __syncthreads();
  for (int e = tid; e < n; e += kSelThreads) s_key[e] = s_key[e] > hi ? 2u : 0u;
  __syncthreads();
  for (int c = tid; c < n_cand; c += kSelThreads) {
    const uint64_t mine = s_key64[c];
    const int e = s_cand[c];
    int rank = 0;
    for (int o = 0; o < n_cand; ++o)
      rank += s_key64[o] > mine || (s_key64[o] == mine && s_cand[o] < e);
    if (rank < need) s_key[e] = 2u;
  }
  __syncthreads();
  emit(s_key, 1u, 0, k);
}

}  // namespace vsa

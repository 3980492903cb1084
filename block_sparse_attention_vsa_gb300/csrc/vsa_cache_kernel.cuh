// vsa_cache_kernel.cuh -- the 8-bit key/value cache: writing tokens into it, attention of
// single tokens over it, and eviction of blocks from it.
//
// A page holds `block` tokens of one sequence and key/value head: e4m3 codes [block][128]
// for keys and for values, one fp32 scale each (value = code * scale), and the bf16 mean
// of its keys.  table[b, h, j] is the page of block j of sequence b.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/vsa.h"
#include "sm103_ptx.cuh"
#include "vsa_select_kernel.cuh"
#include "vsa_warp_ptx.cuh"

namespace vsa {

// ------------------------------------------------------------------ writing
struct CacheWriteArgs {
  const uint16_t* k;     // [B, Hkv, T, 128]
  const uint16_t* v;
  const int32_t* table;  // [B, Hkv, max_blocks]
  const int32_t* lens;   // [B] tokens held before the call
  const int32_t* n_new;  // [B] or null (T each)
  uint8_t* k_cache;      // [pages, block, 128]
  uint8_t* v_cache;
  float* k_scale;        // [pages]
  float* v_scale;
  uint16_t* k_mean;      // [pages, 128] or null
  int Hkv, T, slots, pages, max_blocks;
};

// The least exponent e >= -100 with amax <= 448 * 2^e, for the largest finite |x| given as
// bf16 bits: 448 = 1.75 * 2^8, so e is amax's own exponent less 8, one more where its
// significand exceeds 1.75.
__device__ __forceinline__ int cache_exponent(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7fu) > 0x60u ? 1 : 0);
  return e < -100 ? -100 : e;
}

// One CTA per touched page and tensor (blockIdx.y: 0 keys, 1 values); a thread holds 8
// columns of 8 rows.  The scale is a power of two, so dividing by it and moving held codes
// to a larger one are exact but for codes that fall below the smallest subnormal, and a
// page written token by token ends as one written at once.  Bound by the bytes: bf16 in,
// codes out.
template <int BLOCK>
__global__ void __launch_bounds__(BLOCK * 2) cache_write_kernel(const CacheWriteArgs a) {
  constexpr int kThreads = BLOCK * 2, kRowsPerPass = kThreads / 16, kWarps = kThreads / 32;
  __shared__ uint32_t s_amax[kWarps];
  __shared__ float s_sum[kWarps][128];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long bh = blockIdx.x / a.slots;
  const int b = (int)(bh / a.Hkv);
  const int len = max(0, a.lens[b]);
  int n = a.T;
  if (a.n_new != nullptr) n = min(n, max(0, a.n_new[b]));
  const long long j = len / BLOCK + (blockIdx.x - bh * a.slots);  // the block written
  if (j >= a.max_blocks) return;
  const long long start = j * BLOCK;
  const int n_old = (int)max(0ll, min((long long)BLOCK, len - start));
  const int n_all = (int)min((long long)BLOCK, (long long)len + n - start);
  if (n_all <= n_old) return;
  const int page = a.table[bh * a.max_blocks + j];
  if (page < 0 || page >= a.pages) return;
  const bool values = blockIdx.y != 0;
  const int c = tid & 15, r0 = tid >> 4;
  const uint16_t* x = (values ? a.v : a.k) + bh * a.T * 128;  // row r of the page: start-len+r
  uint8_t* codes = (values ? a.v_cache : a.k_cache) + (long long)page * BLOCK * 128;
  float* scale = (values ? a.v_scale : a.k_scale) + page;

  uint4 w[8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + i * kRowsPerPass;
    w[i] = r >= n_old && r < n_all
               ? __ldg(reinterpret_cast<const uint4*>(x + (start - len + r) * 128) + c)
               : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = u[e] & 0x7fffu, hi = u[e] >> 16 & 0x7fffu;
      if (lo < 0x7f80u) amax = max(amax, lo);  // infinities saturate, NaN stays NaN
      if (hi < 0x7f80u) amax = max(amax, hi);
    }
  }
  const float s_old = n_old > 0 ? *scale : 0.0f;
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (lane == 0) s_amax[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) amax = max(amax, s_amax[i]);
  const int e2 = cache_exponent(amax);
  float s = __uint_as_float((uint32_t)(e2 + 127) << 23);
  if (n_old > 0) s = fmaxf(s, s_old);
  const float inv = 1.0f / s, move = n_old > 0 ? s_old / s : 1.0f;
  const bool moved = n_old > 0 && s != s_old;
  const bool mean = !values && a.k_mean != nullptr;
  float sum[8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + i * kRowsPerPass;
    if (r >= n_all) continue;
    uint2* at = reinterpret_cast<uint2*>(codes + r * 128) + c;
    uint2 o;
    if (r >= n_old) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = f32x2_to_e4m3x2(bf16_lo(u[e]) * inv, bf16_hi(u[e]) * inv);
      o = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
      *at = o;
    } else {
      if (!moved && !mean) continue;
      o = *at;
      if (moved) {
        uint32_t h[4];
        const uint32_t u[2] = {o.x, o.y};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t p, q;
          e4m3x4_to_f16x2(u[e], p, q);
          const float2 fp = __half22float2(*reinterpret_cast<const __half2*>(&p));
          const float2 fq = __half22float2(*reinterpret_cast<const __half2*>(&q));
          h[2 * e] = f32x2_to_e4m3x2(fp.x * move, fp.y * move);
          h[2 * e + 1] = f32x2_to_e4m3x2(fq.x * move, fq.y * move);
        }
        o = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
        *at = o;
      }
    }
    if (mean) {
      const uint32_t u[2] = {o.x, o.y};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t p, q;
        e4m3x4_to_f16x2(u[e], p, q);
        const float2 fp = __half22float2(*reinterpret_cast<const __half2*>(&p));
        const float2 fq = __half22float2(*reinterpret_cast<const __half2*>(&q));
        sum[4 * e] += fp.x;
        sum[4 * e + 1] += fp.y;
        sum[4 * e + 2] += fq.x;
        sum[4 * e + 3] += fq.y;
      }
    }
  }
  if (tid == 0) *scale = s;
  if (!mean) return;
  // codes are whole multiples of 2^-9: their sums are exact, whatever the order (for 128
  // tokens, up to a sum of 2^15)
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 16);
  if (lane < 16) {
    float4* p = reinterpret_cast<float4*>(&s_sum[warp][c * 8]);
    p[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
    p[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
  }
  __syncthreads();
  if (tid < 64) {
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int p = 0; p < kWarps; ++p) {
      lo += s_sum[p][2 * tid];
      hi += s_sum[p][2 * tid + 1];
    }
    const float d = (float)n_all;
    reinterpret_cast<__nv_bfloat162*>(a.k_mean + (long long)page * 128)[tid] =
        __floats2bfloat162_rn(lo / d * s, hi / d * s);
  }
}

// ------------------------------------------------------------------ attention
struct CacheFwdArgs {
  const uint16_t* q;       // [B, Hq, 1, 128]
  const uint8_t* k_cache;  // [pages, block, 128]
  const uint8_t* v_cache;
  const float* k_scale;    // [pages]
  const float* v_scale;
  const int32_t* table;    // [B, Hkv, max_blocks]
  const int32_t* lens;     // [B]
  const int32_t* idx;      // [B, Hkv, max_sel] or null (all blocks)
  const int32_t* num;      // [B, Hkv]
  uint16_t* out;           // [B, Hq, 1, 128]
  float* lse;              // [B, Hq, 1] or null
  float* weight;           // [B, Hkv, max_blocks] or null
  unsigned int* counters;  // [B, Hkv, chunks + 1], zero before and after
  float* part;             // [B, Hkv, chunks, splits][8 * 128 + 16]
  float* lse_ws;           // [B, Hkv, group] (with weight)
  float2* mass;            // [B, Hkv, max_blocks, 8 * chunks] (with weight)
  int Hkv, group, chunks, splits, pages, max_blocks, max_sel;
  float scale_log2, keep;
};

constexpr int kCacheWarps = 4;
constexpr int kCacheStages = 3;
constexpr int kCacheTile = 32;                           // tokens a stage
constexpr int kCacheStageBytes = 2 * kCacheTile * 128;   // keys, then values
constexpr int kCacheList = 512;                          // blocks a CTA walks at most
constexpr int kCachePartFloats = 8 * 128 + 16;           // O [8][128], m [8], l [8]
constexpr int kCacheMinBlocks = 4;                       // blocks a split has at least
constexpr size_t kCacheSmem = (size_t)kCacheWarps * kCacheStages * kCacheStageBytes;

// One CTA: one 8-head chunk of a (sequence, key/value head) and one contiguous range of
// its listed blocks; a warp takes every fourth block of the range, alone: its own ring of
// asynchronous copies (32 tokens a stage: 4 KB of keys, 4 KB of values, two stages in
// flight while one is used), its own running maximum and sums, no barrier until the end.
//
// Codes become fp16 in registers (exact) and both products run on m16n8k16 tensor
// products with the heads as the 8 columns:
//   S^T [tokens x heads] = K [tokens x 128] (A operand) * Q^T
//   O^T [128 x heads]   += V^T [128 x tokens] (A operand) * P^T
// The contraction index of the first and the rows of the second are permuted so that a
// thread reads 16 bytes of a token at a time.  q is scaled by a power of two per head into
// fp16's range (8 significant bits fit 11).  P is fp16 with the running maximum set
// 4 below the largest score and moved only when a score exceeds it by 10, so that
// 2^-28 of the largest weight is still held and the rescaling of O is rare; the rounding
// of P (2^-12 of a weight) is below that of the bf16 output.  Sums are fp32.
//
// The 8-bit values are the only large traffic; everything else is arranged so that they
// arrive without a pause.
template <int BLOCK, bool WEIGHT>
__global__ void __launch_bounds__(kCacheWarps * 32, 2) cache_fwd_kernel(const CacheFwdArgs a) {
  constexpr int kThreads = kCacheWarps * 32;
  constexpr int kHalves = BLOCK / kCacheTile;
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ uint32_t s_bits[kMaxBlocks / 32];
  __shared__ int s_page[kCacheList];
  __shared__ float s_ks[kCacheList], s_vs[kCacheList];
  __shared__ uint16_t s_blk[kCacheList];
  __shared__ float s_qf[8];
  __shared__ float s_m[kCacheWarps][8], s_l[kCacheWarps][8];
  __shared__ int s_last;
  __shared__ int s_n;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, i4 = lane & 3;
  int u = blockIdx.x;
  const int split = u % a.splits;
  u /= a.splits;
  const int chunk = u % a.chunks;
  const long long bh = u / a.chunks;
  const int b = (int)(bh / a.Hkv);
  const int len = max(0, a.lens[b]);
  const int held = (int)min(((long long)len + BLOCK - 1) / BLOCK, (long long)a.max_blocks);
  const int32_t* table = a.table + bh * a.max_blocks;

  // the row's blocks: all it holds, or the listed ones as a set, ascending
  int n = held;
  if (a.idx != nullptr) {
    for (int i = tid; i < kMaxBlocks / 32; i += kThreads) s_bits[i] = 0;
    __syncthreads();
    const int cnt = min(max(0, a.num[bh]), a.max_sel);
    const int32_t* idx = a.idx + bh * a.max_sel;
    for (int i = tid; i < cnt; i += kThreads) {
      const int e = idx[i];
      if (e >= 0 && e < held) atomicOr(&s_bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (warp == 0) {
      const int c = __reduce_add_sync(0xffffffffu, __popc(s_bits[lane]) + __popc(s_bits[lane + 32]));
      if (lane == 0) s_n = c;
    }
    __syncthreads();
    n = s_n;
  }
  const int splits = max(1, min(a.splits, (n + kCacheMinBlocks - 1) / kCacheMinBlocks));
  if (split >= splits) return;
  const int lo = (int)((long long)n * split / splits);
  const int cnt = (int)((long long)n * (split + 1) / splits) - lo;
  // the range's list
  if (a.idx == nullptr) {
    for (int i = tid; i < cnt; i += kThreads) s_blk[i] = (uint16_t)(lo + i);
  } else if (warp < 2) {
    const uint32_t w = s_bits[lane + 32 * warp];
    int at = __popc(w);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    at -= __popc(w);
    if (warp == 1) at += __reduce_add_sync(0xffffffffu, __popc(s_bits[lane]));
    for (uint32_t r = w; r != 0; r &= r - 1, ++at)
      if (at >= lo && at < lo + cnt)
        s_blk[at - lo] = (uint16_t)((lane + 32 * warp) * 32 + __ffs(r) - 1);
  }
  __syncthreads();
  for (int i = tid; i < cnt; i += kThreads) {
    int page = table[s_blk[i]];
    if (page < 0 || page >= a.pages) page = -1;
    s_page[i] = page;
    s_ks[i] = page >= 0 ? a.k_scale[page] : 0.0f;
    s_vs[i] = page >= 0 ? a.v_scale[page] : 0.0f;
  }

  // q of this thread's head column g: columns 16 * (i4 + 4 j) + 0..15
  const int heads = min(8, a.group - chunk * 8);
  const long long head0 = bh * a.group + chunk * 8;
  uint32_t qb[2][4][2];
  {
    uint4 w[2][2];
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        w[j][p] = g < heads ? __ldg(reinterpret_cast<const uint4*>(a.q + (head0 + g) * 128) +
                                    2 * (i4 + 4 * j) + p)
                            : make_uint4(0, 0, 0, 0);
        const uint32_t e[4] = {w[j][p].x, w[j][p].y, w[j][p].z, w[j][p].w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t p0 = e[x] & 0x7fffu, p1 = e[x] >> 16 & 0x7fffu;
          if (p0 < 0x7f80u) amax = max(amax, p0);
          if (p1 < 0x7f80u) amax = max(amax, p1);
        }
      }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // the largest |q| lands in [2^7, 2^8)
    const int e2 = max(-100, min(119, (int)(amax >> 7) - 127 - 7));
    const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
    if (warp == 0 && i4 == 0) s_qf[g] = __uint_as_float((uint32_t)(e2 + 127) << 23) * a.scale_log2;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint4 ww = w[j][x >> 1];
        const uint32_t e0 = (x & 1) ? ww.z : ww.x, e1 = (x & 1) ? ww.w : ww.y;
        qb[j][x][0] = pack_f16x2(bf16_lo(e0) * down, bf16_hi(e0) * down);
        qb[j][x][1] = pack_f16x2(bf16_lo(e1) * down, bf16_hi(e1) * down);
      }
  }
  __syncthreads();
  const float qf0 = s_qf[2 * i4], qf1 = s_qf[2 * i4 + 1];

  float o[8][4] = {};
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;

  // this warp's stages: block entries warp, warp + 4, ...; kHalves stages each
  const int mine = cnt > warp ? (cnt - warp + kCacheWarps - 1) / kCacheWarps : 0;
  const int n_stage = mine * kHalves;
  uint8_t* ring = s_ring + warp * (kCacheStages * kCacheStageBytes);
  auto valid_of = [&](int entry, int half) {  // tokens of the stage that exist
    const long long left = (long long)len - (long long)s_blk[entry] * BLOCK - half * kCacheTile;
    return s_page[entry] < 0 ? 0 : (int)max(0ll, min((long long)kCacheTile, left));
  };
  // Keys: token r, chunk c at chunk c ^ 4 (r & 1); values: c ^ 2 ((r >> 1) & 3) -- each
  // makes its own reads (below) touch all banks.
  auto issue = [&](int st) {
    if (st < n_stage) {
      const int entry = warp + (st / kHalves) * kCacheWarps, half = st % kHalves;
      const int ok = valid_of(entry, half);
      if (ok > 0) {
        const uint32_t dst = smem_addr(ring + (st % kCacheStages) * kCacheStageBytes);
        const long long off = ((long long)s_page[entry] * BLOCK + half * kCacheTile) * 128;
        const int c = lane & 7;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + (lane >> 3);
          const uint32_t nb = r < ok ? 16u : 0u;
          cp_async16(dst + r * 128 + ((c ^ ((r & 1) << 2)) << 4),
                     a.k_cache + off + (nb ? r * 128 + c * 16 : 0), nb);
          cp_async16(dst + kCacheTile * 128 + r * 128 + ((c ^ (((r >> 1) & 3) << 1)) << 4),
                     a.v_cache + off + (nb ? r * 128 + c * 16 : 0), nb);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int st = 0; st < kCacheStages - 1; ++st) issue(st);
  float mass0 = 0.0f, mass1 = 0.0f;
  for (int st = 0; st < n_stage; ++st) {
    cp_async_wait<kCacheStages - 2>();
    __syncwarp();
    issue(st + kCacheStages - 1);
    const int entry = warp + (st / kHalves) * kCacheWarps, half = st % kHalves;
    const int ok = valid_of(entry, half);
    if (ok > 0) {
      const uint8_t* kt = ring + (st % kCacheStages) * kCacheStageBytes;
      const uint8_t* vt = kt + kCacheTile * 128;
      const float f0 = qf0 * s_ks[entry], f1 = qf1 * s_ks[entry];
      float s[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
        const int ra = t * 16 + g, rb = ra + 8;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = (i4 + 4 * j) ^ ((g & 1) << 2);
          const uint4 xa = *reinterpret_cast<const uint4*>(kt + ra * 128 + c * 16);
          const uint4 xb = *reinterpret_cast<const uint4*>(kt + rb * 128 + c * 16);
          const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x2(wa[x], a0, a2);
            e4m3x4_to_f16x2(wb[x], a1, a3);
            mma_f16(s[t], a0, a1, a2, a3, qb[j][x][0], qb[j][x][1]);
          }
        }
      }
      // scores in log2 units; tokens past the sequence's end are left out
      float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const bool in = t * 16 + r * 8 + g < ok;
          s[t][2 * r] = in ? s[t][2 * r] * f0 : -INFINITY;
          s[t][2 * r + 1] = in ? s[t][2 * r + 1] * f1 : -INFINITY;
          top0 = fmaxf(top0, s[t][2 * r]);
          top1 = fmaxf(top1, s[t][2 * r + 1]);
        }
      if (__any_sync(0xffffffffu, top0 > m0 + 10.0f || top1 > m1 + 10.0f)) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, x));
          top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, x));
        }
        const float n0 = top0 > m0 + 10.0f ? top0 - 4.0f : m0;
        const float n1 = top1 > m1 + 10.0f ? top1 - 4.0f : m1;
        const float c0 = n0 > m0 ? fast_exp2(m0 - n0) : 1.0f;
        const float c1 = n1 > m1 ? fast_exp2(m1 - n1) : 1.0f;
        m0 = n0;
        m1 = n1;
        l0 *= c0;
        l1 *= c1;
        if (WEIGHT) {
          mass0 *= c0;
          mass1 *= c1;
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          o[t][0] *= c0;
          o[t][1] *= c1;
          o[t][2] *= c0;
          o[t][3] *= c1;
        }
      }
      const float z0 = m0 == -INFINITY ? 0.0f : m0, z1 = m1 == -INFINITY ? 0.0f : m1;
      float acc[8][4] = {};
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float p0 = fast_exp2(s[t][0] - z0), p1 = fast_exp2(s[t][1] - z1);
        const float p2 = fast_exp2(s[t][2] - z0), p3 = fast_exp2(s[t][3] - z1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        if (WEIGHT) {
          mass0 += p0 + p2;
          mass1 += p1 + p3;
        }
        const uint32_t b0 = transpose_8x8(pack_f16x2(p0, p1));
        const uint32_t b1 = transpose_8x8(pack_f16x2(p2, p3));
        // tokens 2 i4, 2 i4 + 1, and 8 further; columns 16 g .. 16 g + 15
        uint32_t w[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = t * 16 + 2 * i4 + (x & 1) + 8 * (x >> 1);
          const uint4 y = *reinterpret_cast<const uint4*>(vt + r * 128 + ((g ^ (i4 << 1)) << 4));
          w[x][0] = y.x;
          w[x][1] = y.y;
          w[x][2] = y.z;
          w[x][3] = y.w;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x2(__byte_perm(w[0][x], w[1][x], 0x5140), a0, a1);
          e4m3x4_to_f16x2(__byte_perm(w[2][x], w[3][x], 0x5140), a2, a3);
          mma_f16(acc[2 * x], a0, a1, a2, a3, b0, b1);
          e4m3x4_to_f16x2(__byte_perm(w[0][x], w[1][x], 0x7362), a0, a1);
          e4m3x4_to_f16x2(__byte_perm(w[2][x], w[3][x], 0x7362), a2, a3);
          mma_f16(acc[2 * x + 1], a0, a1, a2, a3, b0, b1);
        }
      }
      const float vs = s_vs[entry];
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[t][x] = fmaf(acc[t][x], vs, o[t][x]);
    }
    if (WEIGHT && half == kHalves - 1) {
      // the block's weight under the running maximum, per head
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        mass0 += __shfl_xor_sync(0xffffffffu, mass0, x);
        mass1 += __shfl_xor_sync(0xffffffffu, mass1, x);
      }
      if (g == 0) {
        float4* to = reinterpret_cast<float4*>(
            a.mass + ((bh * a.max_blocks + s_blk[entry]) * a.chunks + chunk) * 8 + 2 * i4);
        *to = make_float4(mass0, m0, mass1, m1);
      }
      mass0 = mass1 = 0.0f;
    }
    __syncwarp();
  }

  // join the warps
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, x);
    l1 += __shfl_xor_sync(0xffffffffu, l1, x);
  }
  if (g == 0) {
    s_m[warp][2 * i4] = m0;
    s_m[warp][2 * i4 + 1] = m1;
    s_l[warp][2 * i4] = l0;
    s_l[warp][2 * i4 + 1] = l1;
  }
  cp_async_wait<0>();
  __syncthreads();
  float* s_o = reinterpret_cast<float*>(s_ring);  // [warp][8][128]
  auto joint_m = [&](int h) {
    float m = s_m[0][h];
#pragma unroll
    for (int w = 1; w < kCacheWarps; ++w) m = fmaxf(m, s_m[w][h]);
    return m;
  };
  {
    const float t0 = joint_m(2 * i4), t1 = joint_m(2 * i4 + 1);
    const float c0 = m0 == -INFINITY ? 0.0f : fast_exp2(m0 - t0);
    const float c1 = m1 == -INFINITY ? 0.0f : fast_exp2(m1 - t1);
    float* to = s_o + warp * 1024;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      *reinterpret_cast<float2*>(to + (2 * i4) * 128 + 16 * g + 2 * t) =
          make_float2(o[t][0] * c0, o[t][2] * c0);
      *reinterpret_cast<float2*>(to + (2 * i4 + 1) * 128 + 16 * g + 2 * t) =
          make_float2(o[t][1] * c1, o[t][3] * c1);
    }
  }
  __syncthreads();
  const long long bc = bh * a.chunks + chunk;
  // thread: head h, columns c4 .. c4+3
  auto finish = [&](int h, int c4, float4 v, float m, float l) {
    if (h >= heads) return;
    const float r = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    uint2 w;
    w.x = pack_bf16x2(v.x * r, v.y * r);
    w.y = pack_bf16x2(v.z * r, v.w * r);
    reinterpret_cast<uint2*>(a.out + (head0 + h) * 128)[c4 >> 2] = w;
    if (c4 == 0) {
      const float lse = l == 0.0f ? VSA_LSE_EMPTY : m + log2f(l);
      if (a.lse != nullptr) a.lse[head0 + h] = lse;
      if (WEIGHT) a.lse_ws[head0 + h] = lse;
    }
  };
  for (int e = tid; e < 256; e += kThreads) {
    const int h = e >> 5, c4 = (e & 31) * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
    const float m = joint_m(h);
#pragma unroll
    for (int w = 0; w < kCacheWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(s_o + w * 1024 + h * 128 + c4);
      v.x += y.x;
      v.y += y.y;
      v.z += y.z;
      v.w += y.w;
      if (s_m[w][h] != -INFINITY) l += s_l[w][h] * fast_exp2(s_m[w][h] - m);
    }
    if (splits == 1) {
      finish(h, c4, v, m, l);
    } else {
      float* p = a.part + (bc * a.splits + split) * kCachePartFloats;
      *reinterpret_cast<float4*>(p + h * 128 + c4) = v;
      if (c4 == 0) {
        p[1024 + h] = m;
        p[1032 + h] = l;
      }
    }
  }
  if (splits > 1) {
    // the last of the row's splits to arrive joins them, in their order
    __threadfence();
    __syncthreads();
    unsigned int* counter = a.counters + bh * (a.chunks + 1) + chunk;
    if (tid == 0) {
      const bool last = atomicAdd(counter, 1u) == (unsigned)splits - 1u;
      if (last) *counter = 0;
      s_last = last;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    for (int e = tid; e < 256; e += kThreads) {
      const int h = e >> 5, c4 = (e & 31) * 4;
      const float* p = a.part + bc * a.splits * kCachePartFloats;
      float m = -INFINITY;
      for (int s = 0; s < splits; ++s) m = fmaxf(m, __ldcg(p + s * kCachePartFloats + 1024 + h));
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float l = 0.0f;
      for (int s = 0; s < splits; ++s) {
        const float* ps = p + s * kCachePartFloats;
        const float ms = __ldcg(ps + 1024 + h);
        if (ms == -INFINITY) continue;
        const float c = fast_exp2(ms - m);
        const float4 y = __ldcg(reinterpret_cast<const float4*>(ps + h * 128 + c4));
        v.x = fmaf(y.x, c, v.x);
        v.y = fmaf(y.y, c, v.y);
        v.z = fmaf(y.z, c, v.z);
        v.w = fmaf(y.w, c, v.w);
        l = fmaf(__ldcg(ps + 1032 + h), c, l);
      }
      finish(h, c4, v, m, l);
    }
  }
  if (WEIGHT) {
    // the last chunk of the group adds each block's share of the weights
    __threadfence();
    __syncthreads();
    if (a.chunks > 1) {
      unsigned int* counter = a.counters + bh * (a.chunks + 1) + a.chunks;
      if (tid == 0) {
        const bool last = atomicAdd(counter, 1u) == (unsigned)a.chunks - 1u;
        if (last) *counter = 0;
        s_last = last;
      }
      __syncthreads();
      if (!s_last) return;
      __threadfence();
    }
    float* weight = a.weight + bh * a.max_blocks;
    for (int j = tid; j < a.max_blocks; j += kThreads) {
      float w = a.keep == 0.0f ? 0.0f : a.keep * weight[j];
      bool on = j < held && (a.idx == nullptr || (s_bits[j >> 5] >> (j & 31) & 1u));
      if (on) {
        const int page = table[j];
        on = page >= 0 && page < a.pages;
      }
      if (on) {
        float share = 0.0f;
        const float2* ms = a.mass + (bh * a.max_blocks + j) * a.chunks * 8;
        for (int h = 0; h < a.group; ++h) {
          const float2 y = __ldcg(ms + h);
          const float z = __ldcg(a.lse_ws + bh * a.group + h);
          if (y.x != 0.0f) share = fmaf(y.x, exp2f(y.y - z), share);
        }
        w += share;
      }
      weight[j] = w;
    }
  }
}

// ------------------------------------------------------------------ eviction
struct CacheEvictArgs {
  const float* weight;   // [B, Hkv, max_blocks]
  const int32_t* table;  // [B, Hkv, max_blocks]
  const int32_t* lens;   // [B]
  int32_t* table_out;
  float* weight_out;
  int32_t* lens_out;     // [B]
  int32_t* freed;        // [B, Hkv, max_blocks]
  int32_t* n_freed;      // [B]
  int Hkv, max_blocks, block, budget, n_first, n_last;
};

// One CTA per (sequence, key/value head): weights as ordered whole numbers in shared
// memory (sure ones above all, NaN below all), the budget-th largest by radix descent,
// then one ascending walk that writes what stays and what goes.
__global__ void __launch_bounds__(kSelThreads) cache_evict_kernel(const CacheEvictArgs a) {
  __shared__ uint32_t s_key[kMaxBlocks];
  __shared__ KthScratch s_kth;
  const int tid = threadIdx.x;
  const long long bh = blockIdx.x, row = bh * a.max_blocks;
  const int b = (int)(bh / a.Hkv);
  const int len = max(0, a.lens[b]);
  const int n = (int)min(((long long)len + a.block - 1) / a.block, (long long)a.max_blocks);
  const int gone = max(0, n - a.budget), stay = n - gone;
  for (int e = tid; e < n; e += kSelThreads) {
    const float w = a.weight[row + e];
    const bool sure = e < a.n_first || e >= n - a.n_last;
    s_key[e] = sure ? kForced32 : (w != w ? 1u : order32(w));
  }
  __syncthreads();
  uint32_t thr = 0;
  int larger = n;
  if (gone > 0) kth_largest<uint32_t>(s_key, n, stay, s_kth, &thr, &larger);
  partition_ascending<uint32_t>(
      s_key, n, thr, stay - larger, s_kth,
      [&](int at, int e) {
        a.table_out[row + at] = a.table[row + e];
        a.weight_out[row + at] = a.weight[row + e];
      },
      [&](int at, int e) { a.freed[row + at] = a.table[row + e]; });
  for (int e = stay + tid; e < a.max_blocks; e += kSelThreads) {
    a.table_out[row + e] = -1;
    a.weight_out[row + e] = 0.0f;
  }
  for (int e = gone + tid; e < a.max_blocks; e += kSelThreads) a.freed[row + e] = -1;
  if (tid == 0 && bh % a.Hkv == 0) {
    a.lens_out[b] = len - gone * a.block;
    a.n_freed[b] = gone;
  }
}

}  // namespace vsa

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
// columns of 8 rows.  The scale is a power of two, so dividing by it is exact, and so is
// moving held codes to a larger one while they stay normal (2^-6 or more); those that become
// subnormal are rounded to a multiple of 2^-9 at each move, each move halving the errors of
// those before: one step in all.  Up to that a page written token by token ends as one
// written at once.  Bound by the bytes, bf16 in and
// codes out, once the arithmetic is packed: 31 us and 6.4 TB/s for two prompts of about
// 12,700 tokens and 8 heads (36 us with 16-bit values taken apart one by one), 3.7 us for one
// token of 32 sequences.
template <int BLOCK>
__global__ void __launch_bounds__(BLOCK * 2) cache_write_kernel(const CacheWriteArgs a) {
  after_predecessor();
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
  const bool values = blockIdx.y != 0;
  const int c = tid & 15, r0 = tid >> 4;
  const uint16_t* x = (values ? a.v : a.k) + bh * a.T * 128;  // row r of the page: start-len+r
  uint4 w[8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + i * kRowsPerPass;
    w[i] = r >= n_old && r < n_all
               ? read_global(reinterpret_cast<const uint4*>(x + (start - len + r) * 128) + c)
               : make_uint4(0, 0, 0, 0);
  }
  const int page = a.table[bh * a.max_blocks + j];
  if (page < 0 || page >= a.pages) return;
  uint8_t* codes = (values ? a.v_cache : a.k_cache) + (long long)page * BLOCK * 128;
  float* scale = (values ? a.v_scale : a.k_scale) + page;
  {  // the largest |x|: NaN does not count; where an infinity does, once more without those
    __nv_bfloat162 m = as_bf162(0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m = __hmax2(m, __habs2(as_bf162(w[i].x)));
      m = __hmax2(m, __habs2(as_bf162(w[i].y)));
      m = __hmax2(m, __habs2(as_bf162(w[i].z)));
      m = __hmax2(m, __habs2(as_bf162(w[i].w)));
    }
    amax = __float_as_uint(fmaxf(__low2float(m), __high2float(m))) >> 16;
    if (amax >= 0x7f80u) {
      amax = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = u[e] & 0x7fffu, hi = u[e] >> 16 & 0x7fffu;
          if (lo < 0x7f80u) amax = max(amax, lo);
          if (hi < 0x7f80u) amax = max(amax, hi);
        }
      }
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
  const uint64_t inv2 = f32x2(inv, inv);
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
      for (int e = 0; e < 4; ++e) {
        float lo, hi;
        split_f32x2(mul_f32x2(bf16x2_to_f32x2(u[e]), inv2), lo, hi);
        h[e] = f32x2_to_e4m3x2(lo, hi);
      }
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
        add_f16x2_to_f32(p, sum[4 * e], sum[4 * e + 1]);
        add_f16x2_to_f32(q, sum[4 * e + 2], sum[4 * e + 3]);
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
  unsigned int* counters;  // zero before and after
  float* part;             // [2 pieces][8 * 128 + 16], then [pieces / 8 + 2] more
  float* lse_ws;           // [B, Hkv, group] (with weight)
  float2* mass;            // [B, Hkv, max_blocks, 8 * chunks] (with weight)
  int rows;                // B * Hkv * chunks
  int Hkv, group, chunks, pages, max_blocks, max_sel;
  int pieces;              // the most there can be
  float scale_log2, keep;
};

constexpr int kCacheWarps = 4;
constexpr int kCacheStages = 3;
constexpr int kCacheTile = 32;                           // tokens a stage
constexpr int kCacheStageBytes = 2 * kCacheTile * 128;   // keys, then values
constexpr int kCacheList = 256;                          // blocks listed at a time
constexpr int kCachePartFloats = 8 * 128 + 16;           // O [8][128], m [8], l [8]
constexpr int kCacheResident = 2;                        // CTAs an SM holds
constexpr int kCacheGrid = 152 * kCacheResident;
constexpr int kCacheRowCost = 12;                        // blocks' time that a row costs, at most
constexpr int kCacheFan = 16;                            // partial results joined at a time
constexpr int kCacheRingBytes = kCacheWarps * kCacheStages * kCacheStageBytes;
constexpr float kNoWeight = -3.4028234663852886e38f;     // the maximum of scores of -infinity
constexpr int kCacheJoinHeads = 4;                       // heads joined at a time
constexpr size_t kCacheSmem =
    (size_t)kCacheRingBytes + kCacheWarps * kCacheJoinHeads * 128 * sizeof(float);
// counters: groups of a row's pieces, rows, chunks of a head group
constexpr int kCacheRowCounters = 1024, kCacheChunkCounters = 2048;

// A stretch of listed blocks of one row, up to kCacheList of them.
struct CacheSeg {
  int row, blocks;            // the row's blocks, as stated
  long long row_at;           // the row's first unit
  int first, from, past, to;  // blocks of the row: the piece's part [first, to), this stretch
  int len, held, cnt;         // tokens and blocks of the sequence, blocks in the list
};

// A row is an 8-head chunk of a (sequence, key/value head).  All rows form one sequence of
// units, a row's being a few for what it costs whatever its length and one for each of its
// blocks, and the sequence is cut into equal pieces, one for each CTA (two per SM, one
// wave): whatever the lengths, every CTA does the same amount.  A piece may hold several
// rows and begin and end inside one; a row spread over several pieces leaves a partial
// result in each, and the last one to arrive joins them in order (beyond 32 in groups of
// 16, then the groups).  Rows whose listing holds duplicates or bad entries count by their
// stated number; the places that are not there do nothing.
// (Pieces of a last part handed out at run time, to even out SMs that differ by a tenth,
// made no call faster: 193 us with and without for 1.24 GB.)
//
// Within a stretch of a row each warp works alone on every fourth block: its own ring of
// asynchronous copies (32 tokens a stage: 4 KB of keys and of values), its own running
// maximum and sums, no barrier until the row's end.  The next stretch's list is made
// before this one's blocks are worked on, and the ring runs on into it, so that copies
// are in flight while a row is joined and the next one set up.
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
// arrive without a pause.  Measured: 1.24 GB (8 sequences of up to 98,304 tokens, 64 heads
// on 8) in 193 us, 6.4 TB/s, which is what DRAM gives to pages in random order; 0.6 GB of 32
// ragged sequences with weights in 107 us; 50 MB of one sequence's chosen blocks in 19.5
// us, of which about 5 lie before the first stage and 5 behind the last, mostly a chain of
// dependent loads and the join (107.5 and 19.9 us without the tables fetched early).
// (Three CTAs an SM of shorter ranges: 207 us and more; one range a row on the hardware's
// scheduler: 210 us; a fifth warp for the lists: 205 us, it costs the others registers.)
template <int BLOCK, bool WEIGHT>
__global__ void __launch_bounds__(kCacheWarps * 32, kCacheResident)
    cache_fwd_kernel(const CacheFwdArgs a) {
  {  // the row that this piece begins in, were the rows equal
    const long long bh = (long long)blockIdx.x * a.rows / gridDim.x / a.chunks;
    prefetch_l2(a.table + bh * a.max_blocks, (size_t)a.max_blocks * 4, threadIdx.x, blockDim.x);
    if (a.idx != nullptr)
      prefetch_l2(a.idx + bh * a.max_sel, (size_t)min(a.max_sel, a.max_blocks) * 4, threadIdx.x,
                  blockDim.x);
    prefetch_l2(a.q + bh * a.group * 128, (size_t)a.group * 256, threadIdx.x, blockDim.x);
  }
  after_predecessor();
  constexpr int kThreads = kCacheWarps * 32;
  constexpr int kHalves = BLOCK / kCacheTile;
  constexpr int N = kCacheStages;
  extern __shared__ __align__(128) uint8_t s_ring[];
  float* const s_o = reinterpret_cast<float*>(s_ring + kCacheRingBytes);
  __shared__ uint32_t s_bits[2][kMaxBlocks / 32];
  __shared__ int s_page[2][kCacheList];
  __shared__ uint16_t s_blk[2][kCacheList];
  __shared__ float s_scale[kCacheWarps][N][2];
  // per list buffer: a warp may be through with its part of the next row before another has
  // read those of this one
  __shared__ float s_m[2][kCacheWarps][8], s_l[2][kCacheWarps][8];
  __shared__ long long s_scan[kCacheWarps];
  __shared__ long long s_at;
  __shared__ int s_row, s_last;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, i4 = lane & 3;

  auto held_of = [&](int b) {
    const long long len = max(0, a.lens[b]);
    return (int)min((len + BLOCK - 1) / BLOCK, (long long)a.max_blocks);
  };
  // a row's blocks as stated, 1 at least
  auto blocks_of = [&](int row) {
    const int bh = row / a.chunks;
    int n = held_of(bh / a.Hkv);
    if (a.idx != nullptr) n = min(n, min(a.num[bh], a.max_sel));
    return max(1, n);
  };

  // ---- the pieces
  const int per = (a.rows + kThreads - 1) / kThreads;
  const int my0 = min(a.rows, tid * per), my1 = min(a.rows, my0 + per);
  long long mine_before, mine_sum = 0, total = 0;
  int pieces, cost;
  {
    for (int r = my0; r < my1; ++r) mine_sum += blocks_of(r);
    long long x = mine_sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    mine_before = x - mine_sum;
#pragma unroll
    for (int w = 0; w < kCacheWarps; ++w) {
      if (w < warp) mine_before += s_scan[w];
      total += s_scan[w];
    }
    pieces = (int)max(1ll, min((long long)gridDim.x, total / 2));
    // no more than an eighth of a piece
    cost = total >= 8ll * kCacheRowCost * pieces ? kCacheRowCost : (int)((int)total / (8 * pieces));
    total += (long long)a.rows * cost;
    mine_before += (long long)my0 * cost;
    mine_sum += (long long)(my1 - my0) * cost;
  }
  // (a 64-bit division takes a few hundred cycles, one of 32 bits some tens)
  auto quotient = [](long long x, long long y) {
    return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
  };
  auto begin_of = [&](int p) { return quotient(total * p, pieces); };
  auto piece_of = [&](long long u) { return (int)quotient((u + 1) * pieces - 1, total); };
  const int piece = blockIdx.x;
  if (piece >= pieces) return;
  const long long piece_from = begin_of(piece), piece_to = begin_of(piece + 1);

  // ---- from one stretch to the next; false when there is none.  Uniform over the CTA.
  // The row's part that lies in the piece, from unit `unit` on (none where the piece ends
  // among the units before the row's first block).
  auto enter_row = [&](CacheSeg& s, long long unit) {
    s.blocks = blocks_of(s.row);
    const long long at = s.row_at + cost;
    s.first = s.from = (int)max(0ll, unit - at);
    s.to = (int)max(0ll, min((long long)s.blocks, piece_to - at));
    s.past = min(s.to, s.from + kCacheList);
    return s.from < s.to;
  };
  auto advance = [&](CacheSeg& s) {
    if (s.past < s.to) {  // more of the same row
      s.from = s.past;
      s.past = min(s.to, s.from + kCacheList);
      return true;
    }
    s.row_at += cost + s.blocks;
    if (s.row_at >= piece_to) return false;
    ++s.row;
    return enter_row(s, s.row_at);
  };
  // ---- a stretch's list of pages, in buffer `buf`
  auto list = [&](CacheSeg& s, int buf) {
    const long long bh = s.row / a.chunks;
    s.len = max(0, a.lens[bh / a.Hkv]);
    s.held = held_of((int)(bh / a.Hkv));
    const int32_t* table = a.table + bh * a.max_blocks;
    uint32_t* bits = s_bits[buf];
    __syncthreads();  // the buffer's last user is through
    if (a.idx == nullptr) {
      s.cnt = min(s.past, s.held) - s.from;  // held may be 0, with one unit all the same
      for (int i = tid; i < s.cnt; i += kThreads) {
        const int page = table[s.from + i];
        s_blk[buf][i] = (uint16_t)(s.from + i);
        s_page[buf][i] = page >= 0 && page < a.pages ? page : -1;
      }
    } else {
      const int listed = min(max(0, a.num[bh]), a.max_sel);
      const int32_t* idx = a.idx + bh * a.max_sel;
      const int idx0 = tid < a.max_sel ? idx[tid] : -1;
      for (int i = tid; i < kMaxBlocks / 32; i += kThreads) bits[i] = 0;
      __syncthreads();
      if (tid < listed && idx0 >= 0 && idx0 < s.held)
        atomicOr(&bits[idx0 >> 5], 1u << (idx0 & 31));
      for (int i = tid + kThreads; i < listed; i += kThreads) {
        const int e = idx[i];
        if (e >= 0 && e < s.held) atomicOr(&bits[e >> 5], 1u << (e & 31));
      }
      __syncthreads();
      int n = 0;
#pragma unroll
      for (int i = 0; i < kMaxBlocks / 1024; ++i)
        n += __reduce_add_sync(0xffffffffu, __popc(bits[lane + 32 * i]));
      s.cnt = max(0, min(s.past, n) - s.from);
      if (warp < kMaxBlocks / 1024) {
        const uint32_t w = bits[lane + 32 * warp];
        int at = __popc(w);
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, at, x);
          if (lane >= x) at += y;
        }
        at -= __popc(w);
        for (int i = 0; i < warp; ++i)
          at += __reduce_add_sync(0xffffffffu, __popc(bits[lane + 32 * i]));
        for (uint32_t r = w; r != 0; r &= r - 1, ++at)
          if (at >= s.from && at < s.from + s.cnt) {
            const int e = (lane + 32 * warp) * 32 + __ffs(r) - 1, page = table[e];
            s_blk[buf][at - s.from] = (uint16_t)e;
            s_page[buf][at - s.from] = page >= 0 && page < a.pages ? page : -1;
          }
      }
    }
    __syncthreads();
  };
  // a stretch's stages for this warp: every fourth block, kHalves stages each
  auto stages_of = [&](const CacheSeg& s) {
    return s.cnt > warp ? (s.cnt - warp + kCacheWarps - 1) / kCacheWarps * kHalves : 0;
  };
  auto valid_of = [&](const CacheSeg& s, int buf, int entry, int half) {  // tokens that exist
    const int left = s.len - (int)s_blk[buf][entry] * BLOCK - half * kCacheTile;
    return s_page[buf][entry] < 0 ? 0 : max(0, min(kCacheTile, left));
  };
  // Copy stage st into a slot.  Keys: token r, chunk c at chunk c ^ 4 (r & 1); values:
  // c ^ 2 ((r >> 1) & 3) -- each makes its own reads (below) touch all banks.
  uint8_t* const ring = s_ring + warp * (N * kCacheStageBytes);
  auto copy = [&](const CacheSeg& s, int buf, int st, int slot) {
    const int entry = warp + (st / kHalves) * kCacheWarps, half = st % kHalves;
    const int ok = valid_of(s, buf, entry, half);
    if (ok > 0) {
      const int page = s_page[buf][entry];
      const uint32_t dst = smem_addr(ring + slot * kCacheStageBytes);
      const long long off = ((long long)page * BLOCK + half * kCacheTile) * 128;
      if (lane < 2)
        cp_async4(smem_addr(&s_scale[warp][slot][lane]),
                  (lane == 0 ? a.k_scale : a.v_scale) + page);
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
  };

  // q of this thread's head column g: columns 16 * (i4 + 4 j) + 0..15
  auto fetch_q = [&](const CacheSeg& s, uint4 (&qw)[2][2]) {
    const int chunk = s.row % a.chunks;
    const long long head = (long long)(s.row / a.chunks) * a.group + chunk * 8 + g;
    const bool on = g < a.group - chunk * 8;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        qw[j][p] = on ? read_global(reinterpret_cast<const uint4*>(a.q + head * 128) +
                                    2 * (i4 + 4 * j) + p)
                      : make_uint4(0, 0, 0, 0);
  };

  CacheSeg cur, nxt;
  uint4 qw[2][2];
  int buf = 0, slot = 0;  // the list in use; the slot of the next stage to be used
  if (mine_before <= piece_from && piece_from < mine_before + mine_sum) {
    long long at = mine_before;
    int r = my0;
    for (;; ++r) {
      const int n = cost + blocks_of(r);
      if (piece_from < at + n) break;
      at += n;
    }
    s_row = r;
    s_at = at;
  }
  __syncthreads();
  cur.row = s_row;
  cur.row_at = s_at;
  bool more = enter_row(cur, piece_from);
  if (more) {
    fetch_q(cur, qw);
    list(cur, 0);
  }
  int n_cur = more ? stages_of(cur) : 0;
  // N groups of copies are always outstanding, some of them empty
#pragma unroll
  for (int st = 0; st < N; ++st) {
    if (st < n_cur) copy(cur, 0, st, st);
    cp_async_commit();
  }
  float o[8][4];
  float m0, m1, l0, l1, mass0 = 0.0f, mass1 = 0.0f;
  bool any = false;  // whether this warp has attended a token of the row

  while (more) {
    nxt = cur;
    const bool follows = advance(nxt);
    if (follows) list(nxt, buf ^ 1);
    const int n_nxt = follows ? stages_of(nxt) : 0;
    auto wrap = [&](int x) { return x >= N ? x - N : x; };
    // the slots that this stretch is too short to fill
    for (int st = n_cur; st < N; ++st) {
      if (st - n_cur < n_nxt) copy(nxt, buf ^ 1, st - n_cur, wrap(slot + st));
      cp_async_commit();
    }

    const int chunk = cur.row % a.chunks;
    const long long bh = cur.row / a.chunks;
    const int heads = min(8, a.group - chunk * 8);
    const long long head0 = bh * a.group + chunk * 8;
    const int32_t* table = a.table + bh * a.max_blocks;
    uint32_t qb[2][4][2];
    float qf0, qf1;  // what turns the products of heads 2 i4, 2 i4 + 1 into log2 units
    {
      uint32_t amax = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t e[4] = {qw[j][p].x, qw[j][p].y, qw[j][p].z, qw[j][p].w};
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
      const float f = __uint_as_float((uint32_t)(e2 + 127) << 23) * a.scale_log2;
      qf0 = __shfl_sync(0xffffffffu, f, 8 * i4);
      qf1 = __shfl_sync(0xffffffffu, f, 8 * i4 + 4);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint4 ww = qw[j][x >> 1];
          const uint32_t e0 = (x & 1) ? ww.z : ww.x, e1 = (x & 1) ? ww.w : ww.y;
          qb[j][x][0] = pack_f16x2(bf16_lo(e0) * down, bf16_hi(e0) * down);
          qb[j][x][1] = pack_f16x2(bf16_lo(e1) * down, bf16_hi(e1) * down);
        }
    }
    if (cur.from == cur.first) {
#pragma unroll
      for (int t = 0; t < 8; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.0f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.0f;
      any = false;
    }

    for (int st = 0; st < n_cur; ++st) {
      cp_async_wait<N - 1>();
      __syncwarp();
      const int entry = warp + (st / kHalves) * kCacheWarps, half = st % kHalves;
      const int ok = valid_of(cur, buf, entry, half);
      if (ok > 0) {
        any = true;
        const uint8_t* kt = ring + slot * kCacheStageBytes;
        const uint8_t* vt = kt + kCacheTile * 128;
        const float f0 = qf0 * s_scale[warp][slot][0], f1 = qf1 * s_scale[warp][slot][0];
        const float vs = s_scale[warp][slot][1];
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
          const float c0_ = n0 > m0 ? fast_exp2(m0 - n0) : 1.0f;
          const float c1_ = n1 > m1 ? fast_exp2(m1 - n1) : 1.0f;
          m0 = n0;
          m1 = n1;
          l0 *= c0_;
          l1 *= c1_;
          if (WEIGHT) {
            mass0 *= c0_;
            mass1 *= c1_;
          }
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            o[t][0] *= c0_;
            o[t][1] *= c1_;
            o[t][2] *= c0_;
            o[t][3] *= c1_;
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
              a.mass + ((bh * a.max_blocks + s_blk[buf][entry]) * a.chunks + chunk) * 8 + 2 * i4);
          *to = make_float4(mass0, m0, mass1, m1);
        }
        mass0 = mass1 = 0.0f;
      }
      __syncwarp();
      const int ahead = st + N;  // the stage that takes the slot's place
      if (ahead < n_cur)
        copy(cur, buf, ahead, slot);
      else if (ahead - n_cur < n_nxt)
        copy(nxt, buf ^ 1, ahead - n_cur, slot);
      cp_async_commit();
      slot = wrap(slot + 1);
    }

    if (cur.past == cur.to) {  // the piece's part of the row ends here
      // ---- join the warps, four heads at a time: thread e has head e / 32, columns
      // 4 (e % 32)..; x counts the two rounds
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, x);
        l1 += __shfl_xor_sync(0xffffffffu, l1, x);
      }
      // weights that are not numbers, and scores that are all -infinity, leave the maximum where
      // it was: never as if there were none
      if (any && m0 == -INFINITY) m0 = l0 != l0 ? 0.0f : kNoWeight;
      if (any && m1 == -INFINITY) m1 = l1 != l1 ? 0.0f : kNoWeight;
      if (g == 0) {
        s_m[buf][warp][2 * i4] = m0;
        s_m[buf][warp][2 * i4 + 1] = m1;
        s_l[buf][warp][2 * i4] = l0;
        s_l[buf][warp][2 * i4 + 1] = l1;
      }
      __syncthreads();
      auto joint_m = [&](int h) {
        float m = s_m[buf][0][h];
#pragma unroll
        for (int w = 1; w < kCacheWarps; ++w) m = fmaxf(m, s_m[buf][w][h]);
        return m;
      };
      const float t0 = joint_m(2 * i4), t1 = joint_m(2 * i4 + 1);
      const float d0 = m0 == -INFINITY ? 0.0f : fast_exp2(m0 - t0);
      const float d1 = m1 == -INFINITY ? 0.0f : fast_exp2(m1 - t1);
      const int c4 = lane * 4;
      float4 v[2];
      float vm[2], vl[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (i4 >> 1 == x) {
          float* to = s_o + (warp * kCacheJoinHeads + 2 * (i4 & 1)) * 128 + 16 * g;
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            *reinterpret_cast<float2*>(to + 2 * t) = make_float2(o[t][0] * d0, o[t][2] * d0);
            *reinterpret_cast<float2*>(to + 128 + 2 * t) = make_float2(o[t][1] * d1, o[t][3] * d1);
          }
        }
        __syncthreads();
        const int h = 4 * x + warp;
        v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        vl[x] = 0.0f;
        vm[x] = joint_m(h);
#pragma unroll
        for (int w = 0; w < kCacheWarps; ++w) {
          const float4 y =
              *reinterpret_cast<const float4*>(s_o + (w * kCacheJoinHeads + warp) * 128 + c4);
          v[x].x += y.x;
          v[x].y += y.y;
          v[x].z += y.z;
          v[x].w += y.w;
          const float wm = s_m[buf][w][h];
          if (wm != -INFINITY) vl[x] += s_l[buf][w][h] * fast_exp2(wm - vm[x]);
        }
        if (x == 0) __syncthreads();
      }

      // ---- join the row's pieces
      const int piece0 = piece_of(cur.row_at + cost);
      const int piece1 = piece_of(cur.row_at + cost + cur.blocks - 1);
      auto leave = [&](float* p) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int h = 4 * x + warp;
          *reinterpret_cast<float4*>(p + h * 128 + c4) = v[x];
          if (lane == 0) {
            p[1024 + h] = vm[x];
            p[1032 + h] = vl[x];
          }
        }
      };
      // whether this CTA is the last of `of` to arrive at a counter, which it then clears;
      // what the others wrote before they arrived is visible then
      auto last_at = [&](unsigned int* counter, int of) {
        __syncthreads();
        if (tid == 0) {
          __threadfence();
          const bool last = atomicAdd(counter, 1u) == (unsigned)of - 1u;
          if (last) *counter = 0;
          __threadfence();
          s_last = last;
        }
        __syncthreads();
        return s_last != 0;
      };
      // A part's place: twice its piece, one more for a row's first part that does not open
      // its piece (another row's last part does).
      const int odd = begin_of(piece0) != cur.row_at + cost ? 1 : 0;
      auto place_of = [&](int p) { return 2 * p + (p == piece0 ? odd : 0); };
      // `count` <= 32 partial results in order: the s-th at place(s)
      auto join = [&](const float* base, auto place, int count) {
        constexpr int kBatch = 8;
        float4 y[kBatch][2];
        auto fetch = [&](int s0) {
#pragma unroll
          for (int s = 0; s < kBatch; ++s)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              y[s][x] = s0 + s < count
                            ? __ldcg(reinterpret_cast<const float4*>(
                                  base + (long long)place(s0 + s) * kCachePartFloats +
                                  (4 * x + warp) * 128 + c4))
                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        };
        float pm[2], pl[2], w[2];  // a lane per source: its maximum, sum and weight
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          pm[x] = -INFINITY;
          pl[x] = 0.0f;
          if (lane < count) {
            const float* p = base + (long long)place(lane) * kCachePartFloats + 4 * x + warp;
            pm[x] = __ldcg(p + 1024);
            pl[x] = __ldcg(p + 1032);
          }
        }
        fetch(0);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float m = pm[x];
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
          w[x] = pm[x] == -INFINITY ? 0.0f : fast_exp2(pm[x] - m);
          float l = pl[x] * w[x];
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
          vm[x] = m;
          vl[x] = l;
          v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        for (int s0 = 0; s0 < count; s0 += kBatch) {
          if (s0 > 0) fetch(s0);
#pragma unroll
          for (int s = 0; s < kBatch; ++s)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float c = __shfl_sync(0xffffffffu, w[x], (s0 + s) & 31);
              v[x].x = fmaf(y[s][x].x, c, v[x].x);
              v[x].y = fmaf(y[s][x].y, c, v[x].y);
              v[x].z = fmaf(y[s][x].z, c, v[x].z);
              v[x].w = fmaf(y[s][x].w, c, v[x].w);
            }
        }
      };
      const int sharers = piece1 - piece0 + 1;
      bool finish = true;
      if (sharers > 1) {
        leave(a.part + (long long)place_of(piece) * kCachePartFloats);
        unsigned int* counter = a.counters + kCacheRowCounters + place_of(piece0);
        if (sharers <= 2 * kCacheFan) {
          finish = last_at(counter, sharers);
          if (finish) join(a.part, [&](int s) { return place_of(piece0 + s); }, sharers);
        } else {
          const int group = (piece - piece0) / kCacheFan, lead = piece0 + group * kCacheFan;
          const int groups = (sharers + kCacheFan - 1) / kCacheFan;
          const int count = min(kCacheFan, piece1 + 1 - lead);
          float* wide = a.part + (long long)2 * a.pieces * kCachePartFloats;
          // 16 pieces hold the leads of two rows at most: one's last group, another's first
          auto group_place = [&](int s) {
            return 2 * ((piece0 + s * kCacheFan) / kCacheFan) + (s == 0 ? 1 : 0);
          };
          finish = last_at(a.counters + place_of(lead), count);
          if (finish) {
            join(a.part, [&](int s) { return place_of(lead + s); }, count);
            leave(wide + (long long)group_place(group) * kCachePartFloats);
            finish = last_at(counter, groups);
            if (finish) join(wide, group_place, groups);
          }
        }
      }
      if (finish) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int h = 4 * x + warp;
          if (h >= heads) continue;
          // (tokens, but no weight among them: 0 / 0)
          const float l = vl[x] == 0.0f && vm[x] != -INFINITY ? NAN : vl[x];
          const float r = l > 0.0f || l != l ? 1.0f / l : 0.0f;
          uint2 w;
          w.x = pack_bf16x2(v[x].x * r, v[x].y * r);
          w.y = pack_bf16x2(v[x].z * r, v[x].w * r);
          reinterpret_cast<uint2*>(a.out + (head0 + h) * 128)[lane] = w;
          if (lane == 0) {
            const float lse = l == 0.0f ? VSA_LSE_EMPTY : vm[x] + log2f(l);
            if (a.lse != nullptr) a.lse[head0 + h] = lse;
            if (WEIGHT) a.lse_ws[head0 + h] = lse;
          }
        }
      }
      // the last chunk of the group adds each block's share of the weights
      if (WEIGHT && finish && last_at(a.counters + kCacheChunkCounters + bh, a.chunks)) {
        float* weight = a.weight + bh * a.max_blocks;
        const uint32_t* bits = s_bits[buf];
        for (int j = tid; j < a.max_blocks; j += kThreads) {
          float w = a.keep == 0.0f ? 0.0f : a.keep * weight[j];
          bool on = j < cur.held && (a.idx == nullptr || (bits[j >> 5] >> (j & 31) & 1u));
          if (on) {
            const int page = table[j];
            on = page >= 0 && page < a.pages;
          }
          if (on) {
            // eight heads of a chunk at a time, in pairs of (sum, maximum)
            float share = 0.0f;
            const float4* ms = reinterpret_cast<const float4*>(
                a.mass + (bh * a.max_blocks + j) * a.chunks * 8);
            for (int h = 0; h < a.group; h += 8) {
              float4 y[4];
              float z[8];
#pragma unroll
              for (int x = 0; x < 4; ++x) y[x] = __ldcg(ms + h / 2 + x);
#pragma unroll
              for (int x = 0; x < 8; ++x)
                z[x] = h + x < a.group ? __ldcg(a.lse_ws + bh * a.group + h + x) : 0.0f;
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                // (a head whose weights are not numbers makes the share none, be its sum 0)
                if ((y[x].x != 0.0f || z[2 * x] != z[2 * x]) && h + 2 * x < a.group)
                  share = fmaf(y[x].x, exp2f(y[x].y - z[2 * x]), share);
                if ((y[x].z != 0.0f || z[2 * x + 1] != z[2 * x + 1]) && h + 2 * x + 1 < a.group)
                  share = fmaf(y[x].z, exp2f(y[x].w - z[2 * x + 1]), share);
              }
            }
            w += share;
          }
          weight[j] = w;
        }
      }
    }
    cur = nxt;
    buf ^= 1;
    n_cur = n_nxt;
    more = follows;
    if (more) fetch_q(cur, qw);
  }
  cp_async_wait<0>();
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
// memory (sure ones above all, NaN below all) beside the table's row; the last of those
// that stay is found between the least and the largest weight; then one ascending walk
// orders what stays and what goes.  Bound by its barriers more than by its bytes: 3.2 us for
// one sequence of 255 blocks and 8 heads, 8.5 us for 64 of up to 1,536 (12 MB).
constexpr int kEvictThreads = 256;
__global__ void __launch_bounds__(kEvictThreads) cache_evict_kernel(const CacheEvictArgs a) {
  prefetch_l2(a.weight + (long long)blockIdx.x * a.max_blocks, (size_t)a.max_blocks * 4,
              threadIdx.x, kEvictThreads);
  prefetch_l2(a.table + (long long)blockIdx.x * a.max_blocks, (size_t)a.max_blocks * 4,
              threadIdx.x, kEvictThreads);
  after_predecessor();
  constexpr int kWarps = kEvictThreads / 32, kEach = kMaxBlocks / kEvictThreads;
  __shared__ uint32_t s_key[kMaxBlocks];
  __shared__ float s_weight[kMaxBlocks];
  __shared__ int32_t s_table[kMaxBlocks];
  __shared__ uint16_t s_order[kMaxBlocks];
  __shared__ __align__(16) uint32_t s_list[kRanked];
  __shared__ KthScratch s_kth;
  __shared__ uint32_t s_lo[kWarps], s_hi[kWarps], s_thr;
  __shared__ int s_sure[kWarps], s_members;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long bh = blockIdx.x, row = bh * a.max_blocks;
  const int b = (int)(bh / a.Hkv);
  // the whole row, before its length is known
  float weight[kEach];
  int32_t page[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = tid + i * kEvictThreads;
    weight[i] = e < a.max_blocks ? read_global(a.weight + row + e) : 0.0f;
    page[i] = e < a.max_blocks ? read_global(a.table + row + e) : -1;
  }
  const int len = max(0, a.lens[b]);
  const int n = (int)min(((long long)len + a.block - 1) / a.block, (long long)a.max_blocks);
  const int gone = max(0, n - a.budget), stay = n - gone;
  uint32_t lo = kForced32, hi = 0;
  int sure = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = tid + i * kEvictThreads;
    if (e >= n) continue;
    const float w = weight[i];
    s_weight[e] = w;
    s_table[e] = page[i];
    uint32_t key = w != w ? 1u : order32(w);
    if (e < a.n_first || e >= n - a.n_last) {
      key = kForced32;
      ++sure;
    } else {
      lo = min(lo, key);
      hi = max(hi, key);
    }
    s_key[e] = key;
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  sure = __reduce_add_sync(0xffffffffu, sure);
  if (lane == 0) {
    s_lo[warp] = lo;
    s_hi[warp] = hi;
    s_sure[warp] = sure;
  }
  if (tid == 0) s_members = 0;
  __syncthreads();
  uint32_t thr = 0;
  int larger = n;
  if (gone > 0) {
    sure = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      lo = min(lo, s_lo[w]);
      hi = max(hi, s_hi[w]);
      sure += s_sure[w];
    }
    if (stay > sure) {
      kth_between(s_key, n, stay - sure, lo, hi, s_kth, s_list, &s_members, &s_thr, &thr, &larger);
      larger += sure;
    } else {  // only the sure ones stay (they are fewer than the budget or as many)
      thr = kForced32 - 1;
      larger = stay;
    }
  }
  // the order of those that stay, then of those that go, so that the writes run through
  partition_ascending<uint32_t>(
      s_key, n, thr, stay - larger, s_kth, [&](int at, int e) { s_order[at] = (uint16_t)e; },
      [&](int at, int e) { s_order[stay + at] = (uint16_t)e; });
  __syncthreads();
  for (int at = tid; at < a.max_blocks; at += kEvictThreads) {
    const int e = at < stay ? s_order[at] : -1, f = at < gone ? s_order[stay + at] : -1;
    a.table_out[row + at] = e >= 0 ? s_table[e] : -1;
    a.weight_out[row + at] = e >= 0 ? s_weight[e] : 0.0f;
    a.freed[row + at] = f >= 0 ? s_table[f] : -1;
  }
  if (tid == 0 && bh % a.Hkv == 0) {
    a.lens_out[b] = len - gone * a.block;
    a.n_freed[b] = gone;
  }
}

}  // namespace vsa

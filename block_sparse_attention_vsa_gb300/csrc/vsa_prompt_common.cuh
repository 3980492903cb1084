// vsa_prompt_common.cuh -- what the forward and the backward of the attention over whole
// prompts share: where the sequences lie, how query tiles are numbered, bounded waits.
//
// Sequences are packed one behind the other along the token axis (their starts in a device
// array) or lie in a padded batch (their lengths in one); neither is known to the host.
// A query tile is 128 rows, the M of one tcgen05 MMA: `heads` = 2^pack query heads that share
// a key/value head, times 128 / heads consecutive tokens, row = head * tokens + token.  A
// short sequence, or one token of it, then still fills a tile with the heads of its group.
//
// Tile slots.  With T tokens a tile (or item), sequence b owns the slots from
// A_b = floor(start_b / T) + b on (packed), or b * ceil(S / T) (padded).  For packed sequences
// ceil(len_b / T) <= A_{b+1} - A_b, as len_b = start_{b+1} - start_b, so slots never meet,
// there are floor(S / T) + B of them, and a slot's sequence is found from the starts alone by
// a search; slots that hold no token are passed over.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "sm103_ptx.cuh"
#include "vsa_warp_ptx.cuh"

namespace vsa {
namespace prompt {

constexpr uint64_t kWaitLimitNs = 1000000000ull;  // one second per wait (for up to 2^25 keys)
constexpr unsigned kErrTimeout = 0x100u;          // | code of the wait that gave up
constexpr uint32_t kSleepNs = 20000;              // a waiting thread looks up this often
constexpr uint32_t kTile = 128 * 128 * 2;         // 128 rows of Q, K, V or dO
constexpr float kLseEmpty = -3.402823466e+38f;

struct SeqArgs {
  const int32_t *q_seq, *k_seq;  // packed: starts [B + 1]; padded: lengths [B] or null
  int packed, B, Sq, Sk;         // rows of the token axis
  int causal;
  int sort;                      // bring the longest sequences first (32 or fewer)
};

struct Seq {
  int z, q0, nq, k0, nk;  // batch coordinate, first row and number of queries / keys
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) {
  return x < lo ? lo : (x > hi ? hi : x);
}

// Whatever the arrays hold, the rows lie inside the tensors.
__device__ __forceinline__ Seq load_seq(const SeqArgs& a, int b) {
  Seq s;
  if (a.packed) {
    const int q0 = read_global(a.q_seq + b), q1 = read_global(a.q_seq + b + 1),
              k0 = read_global(a.k_seq + b), k1 = read_global(a.k_seq + b + 1);
    s.z = 0;
    s.q0 = clampi(q0, 0, a.Sq);
    s.nq = clampi(q1, s.q0, a.Sq) - s.q0;
    s.k0 = clampi(k0, 0, a.Sk);
    s.nk = clampi(k1, s.k0, a.Sk) - s.k0;
  } else {
    s.z = b;
    s.q0 = s.k0 = 0;
    s.nq = a.q_seq ? clampi(read_global(a.q_seq + b), 0, a.Sq) : a.Sq;
    s.nk = a.k_seq ? clampi(read_global(a.k_seq + b), 0, a.Sk) : a.Sk;
  }
  return s;
}

__host__ __device__ inline long long tile_slots(int packed, long long B, long long S, int T) {
  return packed ? S / T + B : B * ((S + T - 1) / T);
}

// The packed sequence that owns a slot, by a whole warp: 32 candidates a step.
// `seq` holds starts, S bounds them; *tile is the slot's place in the sequence (it can lie
// outside of it).
__device__ __forceinline__ int find_slot(const int32_t* seq, int B, int S, int T, int slot,
                                         int* tile) {
  const int lane = (int)lane_id();
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    bool below = false;
    if (i < n) below = clampi(read_global(seq + lo + i), 0, S) / T + lo + i <= slot;
    const uint32_t votes = __ballot_sync(0xffffffffu, below);
    const int at = votes ? 31 - __clz((int)votes) : 0;
    lo += at * step;
    n = n - at * step < step ? n - at * step : step;
  }
  *tile = slot - (clampi(read_global(seq + lo), 0, S) / T + lo);
  return lo;
}

// Which tile a CTA (or an item) works on, by a whole warp.  Tiles of 1 << lt tokens, of queries or
// of keys; the n-th in an order that brings the long work first, as what is started last ends last:
// sequences by what their tiles walk over (queries' tiles over keys, keys' over queries), longest
// first, and inside one the last query tiles, which causal masks leave the most keys, or the first
// key tiles, which they leave the most queries.  With more than 32 sequences, or CTAs for all tiles
// at once, sequences come as they are: in a tight loop the order takes 4 prompts of up to 2,000
// tokens behind 4,001 to 16,411 held from 1,845 us to 1,652 and a training step on 3 clips from
// 1,035 to 990 (1,780 and 1,041 as a program calls them, a pass among others), but 88 short items,
// which start together, from 10.1 to 11.2.
struct Place {
  Seq s;
  int b, tile;
  bool there;  // (a packed batch has fewer tiles than slots)
};
__device__ __forceinline__ Place find_tile(const SeqArgs& a, int n, int lt, bool keys) {
  const int lane = (int)lane_id();
  const int S = keys ? a.Sk : a.Sq;
  const int up = (1 << lt) - 1;  // (rows stay that far below 2^31)
  const int per = (S + up) >> lt;  // tiles of a padded sequence
  Place p;
  if (a.sort) {
    const Seq s = load_seq(a, lane < a.B ? lane : a.B - 1);
    const int mine = keys ? s.nk : s.nq, walked = keys ? s.nq : s.nk;
    const int tiles = lane >= a.B ? 0 : a.packed ? (mine + up) >> lt : per;
    int before = 0;
#pragma unroll 1
    for (int j = 0; j < a.B; ++j) {
      const int w = __shfl_sync(0xffffffffu, walked, j), t = __shfl_sync(0xffffffffu, tiles, j);
      if (w > walked || (w == walked && j < lane)) before += t;
    }
    const uint32_t owner = __ballot_sync(0xffffffffu, n >= before && n - before < tiles);
    const int at = owner ? __ffs((int)owner) - 1 : 0;
    const int place = n - __shfl_sync(0xffffffffu, before, at);
    const int all = __shfl_sync(0xffffffffu, tiles, at);
    p.s.z = a.packed ? 0 : at;
    p.s.q0 = __shfl_sync(0xffffffffu, s.q0, at);
    p.s.nq = __shfl_sync(0xffffffffu, s.nq, at);
    p.s.k0 = __shfl_sync(0xffffffffu, s.k0, at);
    p.s.nk = __shfl_sync(0xffffffffu, s.nk, at);
    p.b = at;
    p.tile = keys ? place : all - 1 - place;
    p.there = owner != 0;
    return p;
  }
  if (a.packed) {
    const int slots = (S >> lt) + a.B;
    p.b = find_slot(keys ? a.k_seq : a.q_seq, a.B, S, 1 << lt, keys ? n : slots - 1 - n, &p.tile);
  } else {
    p.tile = n / a.B;
    p.b = n - p.tile * a.B;
    if (!keys) p.tile = per - 1 - p.tile;
  }
  p.s = load_seq(a, p.b);
  p.there = p.tile >= 0 && p.tile < per &&
            (!a.packed || ((long long)p.tile << lt) < (keys ? p.s.nk : p.s.nq));
  return p;
}

// Bounded wait on an mbarrier phase: gives up after `limit_ns`, recording `code` in the status
// word and raising the abort flag, or as soon as another role has raised the flag -- unless
// `drain`, for copies and MMAs in flight, which always runs to the full limit.
struct WaitCtx {
  int* abort_flag;
  unsigned int* status;
  unsigned long long limit_ns;
};
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const WaitCtx& w,
                                     unsigned code, bool drain = false) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t limit = drain ? kWaitLimitNs : w.limit_ns;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (mbar_sleep_wait(bar, parity, kSleepNs)) return true;
    if (!drain && *reinterpret_cast<volatile int*>(w.abort_flag)) return false;
    if (global_timer_ns() - t0 > limit) {
      *reinterpret_cast<volatile int*>(w.abort_flag) = 1;
      atomicCAS(w.status, 0u, kErrTimeout | code);
      return false;
    }
  }
}
// The same by every lane of a warp that goes on to warp-collective instructions: it goes on
// only if every lane saw the phase complete, so an abort cannot split it.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const WaitCtx& w,
                                          unsigned code) {
  const bool ok = wait(bar, parity, w, code);
  return __all_sync(0xffffffffu, ok);
}

// Box of a 4-D view (d, token, head, batch) -> shared; what lies outside the tensor reads 0.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// A 128-row tile as two halves of 64 columns (128-byte rows, 128-byte swizzle).
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar,
                                          int token, int head, int z) {
  tma_load_4d(dst, map, bar, 0, token, head, z);
  tma_load_4d(dst + kTile / 2, map, bar, 64, token, head, z);
}

// Rows [n, 128) of a tile to zero, by one warp (the rows' bytes are the same under the
// swizzle, which moves 16-byte pieces inside a row only), ordered before later MMAs.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int n) {
  const int lane = (int)lane_id();
  for (int i = n * 8 + lane; i < 128 * 8; i += 32) {
    reinterpret_cast<uint4*>(tile)[i] = make_uint4(0, 0, 0, 0);
    reinterpret_cast<uint4*>(tile + kTile / 2)[i] = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// The rows of a query tile (row = head * T + token) whose token is not in [from, to).
__device__ __forceinline__ void zero_tokens(uint8_t* tile, int from, int to, int T) {
  const int lane = (int)lane_id();
  for (int i = lane; i < 128 * 8; i += 32) {
    const int t = (i >> 3) & (T - 1);
    if (t < from || t >= to) {
      reinterpret_cast<uint4*>(tile)[i] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(tile + kTile / 2)[i] = make_uint4(0, 0, 0, 0);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// 32 columns of a warp's 32 rows, fp32 in registers (a row a lane), times f to bf16 in global
// memory, through 2 KB of shared memory, so that a store is 8 rows of 64 bytes and not 32 of 16
// (the forward's results took 6,000 cycles an item that way).  `to` gives where a row's columns
// go, or null.  (Pieces of 16 bytes are turned by the row so that eight rows' meet all banks.)
template <class To>
__device__ __forceinline__ void store_columns(uint8_t* stage, const uint32_t (&x)[32], float f,
                                              bool some, To to) {
  const uint32_t lane = lane_id();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = some ? pack_bf16x2(__uint_as_float(x[8 * c + 2 * i]) * f,
                                __uint_as_float(x[8 * c + 2 * i + 1]) * f)
                  : 0u;
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) * 16)) =
        make_uint4(y[0], y[1], y[2], y[3]);
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = 8 * i + (lane >> 2), c = lane & 3;
    const uint4 y = *reinterpret_cast<const uint4*>(stage + r * 64 + ((c ^ ((r >> 1) & 3)) * 16));
    uint16_t* dst = to((int)r);
    if (dst != nullptr) *reinterpret_cast<uint4*>(dst + 8 * c) = y;
  }
  __syncwarp();
}

}  // namespace prompt
}  // namespace vsa

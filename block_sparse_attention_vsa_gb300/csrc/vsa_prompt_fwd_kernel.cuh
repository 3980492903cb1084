// vsa_prompt_fwd_kernel.cuh -- attention over whole prompts: every query of a sequence against
// the sequence's keys, causal or not, grouped heads, ragged lengths.
//
//   out_i = sum_j p_ij v_j,  p_ij = 2^(c q_i.k_j - lse_i),  c = scale log2 e,
//   lse_i = log2 sum_j 2^(c q_i.k_j)  over j < nk, with causal j <= i + nk - nq
//
// computed in one pass over the keys: with a reference m that follows the running maximum (it
// may lag by up to 2^32, in log2 units 32, so that the accumulator is rarely rescaled),
// P = 2^(S - m) is rounded to bf16 for the product with V, out = O / l and lse = m + log2 l
// with l the sum of the fp32 weights.  (A sum of the rounded ones as well, for out, takes a
// quarter of the loop's instructions -- 1492 TFLOP/s instead of 1647 -- and gains nothing
// where many keys count: out is off by 0.0023 of its norm either way, 0.0017 of it from its own
// rounding.)  S, O, m and l are fp32.
//
// An item is two query tiles of 128 rows (neighbours in the sequence) that share every K and V
// tile: an SS product of 128 x 128 x 128 takes the tensor core 512 cycles and reads 64 KB of
// shared memory, as much as that gives in 512 cycles, so what the two tiles share is what
// keeps the copies' writes affordable.  A warpgroup per query tile works on its scores while
// the tensor core works for the other one.
//
// A CTA per item is launched, and one that has done its own takes over those not launched yet
// (cluster launch control), so a CTA per SM stays and work is handed out as it is done.  12 warps:
//   warps 0-3, 4-7  softmax warpgroups of query tile 0 and 1 (thread = query row)
//   warp 8          decodes items and copies: Q tiles, and K, V alternating through a ring
//   warps 9, 10     MMA issuers of query tile 0 and 1: S_t(0), then per key tile j a unit of
//                   O_t += P_t(j) V_j and S_t(j + 1).  MMAs of one warp run in order, so
//                   S_t(j + 1) may overwrite P_t(j), and S_t(j + 1) complete says that O_t
//                   holds tile j.  The warps take turns, a unit each, which keeps the two softmax
//                   warpgroups half a period apart: without turns they fall into step, and the
//                   tensor core idles meanwhile; one issuer for both spends longer between its
//                   waits than the products take (1325 and 1356 TFLOP/s, 1475 in turns).  The
//                   warps run converged and elect.sync picks the lane that issues.
//   warp 11         hands landed tiles on to the MMA warps, and zeroes the rows of a V tile
//                   behind the sequence's last key: their weight is 0, but 0 times what lies
//                   there (another sequence, padding) may be NaN
// With 19 heads of 8,192 tokens (all pairs) this runs at 1,650 TFLOP/s: the tensor pipe is busy
// 68 % of the time at 1.9 GHz, 3,000 cycles a key tile of both query tiles against 2,048 of
// products; bound by the chain of a tile -- S read, maximum, exponentials, P written, O += P V, S
// again -- of which the other tile's covers most.
// TMEM (512 columns): S_0, S_1 (P over the first 64 columns of S), O_0, O_1.
#pragma once

#include "vsa_prompt_common.cuh"

namespace vsa {
namespace prompt {

struct FwdArgs {
  SeqArgs seq;
  uint16_t* out;
  float* lse;  // [Hq, Sq] or [B, Hq, Sq], or null
  long long out_b, out_h, out_t;  // strides in elements
  unsigned int* status;
  int Hq, group, pack;  // query heads a key/value head; log2 of the heads in a tile
  int n_packs;           // head packs
  int n_items;
  int splits;       // ranges of an item's key tiles, a unit of work each
  float* part;      // [n_items * splits] partial results, if there are several
  float scale_log2;
  unsigned long long wait_ns;
  int stall;
};

namespace fwd {

constexpr unsigned kSms = 152;
constexpr int kThreads = 384;
constexpr int kStages = 4;
constexpr uint32_t kOffQ = 0;  // [2]
constexpr uint32_t kOffKV = 2 * kTile;
constexpr uint32_t kOffOut = kOffKV + kStages * kTile;  // 32 rows of 32 columns a softmax warp
constexpr uint32_t kOffCtl = kOffOut + 8 * 2048;
constexpr uint32_t kSmemBytes = kOffCtl + 1024 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
constexpr uint32_t kSoftmaxRegs = 216, kOtherRegs = 56;
constexpr uint32_t kRegPoolNeeded = 256 * kSoftmaxRegs + 128 * kOtherRegs;
constexpr float kRescale = 32.0f;
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;

struct Item {
  int head0, kv_head, z;  // first query head of the pack, key/value head, batch coordinate
  int tok, q0, nq;        // first token, first row and number of queries of the sequence
  int k0, nk;
  int n0, n1;             // key tiles of the two query tiles
  int unit;
  int go;
};
// A unit's partial result: O [256][128] relative to the row's m, then m [256] and l [256].
constexpr int kPartFloats = 256 * 128 + 512;

struct Ctl {
  uint64_t item_full[2], item_empty[2];
  uint64_t q_full[2], q_empty[2];  // per query tile
  uint64_t kv_full[kStages], ready[kStages], kv_empty[kStages];
  uint64_t s_full[2];      // S_t is in TMEM (and O_t holds the tile before)
  uint64_t p_full[4];      // [2 t + h]: half h of P_t is in TMEM
  uint64_t o_full[2], o_empty[2];
  uint64_t turn[2];        // of the MMA warps
  uint64_t drain[2], never;
  alignas(16) uint8_t next[16];  // the answer to a request for work
  uint64_t next_full;
  Item own, item[2];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Ctl) <= 1024, "control block");

__device__ __forceinline__ bool decode_item(const FwdArgs& a, int id, Item& it) {
  const int half = 128 >> a.pack;
  const int slot = id / a.n_packs;
  const int hp = id - slot * a.n_packs;
  const Place p = find_tile(a.seq, slot, 8 - a.pack, false);
  const Seq& s = p.s;
  it.z = s.z;
  it.q0 = s.q0;
  it.nq = s.nq;
  it.k0 = s.k0;
  it.nk = s.nk;
  it.tok = p.tile << (8 - a.pack);
  it.head0 = hp << a.pack;
  it.kv_head = it.head0 / a.group;
  it.go = 1;
  auto key_tiles = [&](int t0) {
    const int last = (t0 + half < s.nq ? t0 + half : s.nq) - 1;  // its last query
    int keys = s.nk;
    if (a.seq.causal) keys = clampi(last + 1 + s.nk - s.nq, 0, s.nk);
    return t0 < s.nq ? (keys + 127) / 128 : 0;
  };
  it.n0 = key_tiles(it.tok);
  it.n1 = key_tiles(it.tok + half);
  return p.there;
}
// A unit: an item, or a range of its key tiles -- the item of a sequence whose keys begin with
// the range's first (a query attends keys up to its distance from the end, so nothing else
// changes).
__device__ __forceinline__ bool decode(const FwdArgs& a, int id, Item& it) {
  it.unit = id;
  if (a.splits == 1) return decode_item(a, id, it);
  const int item = id / a.splits, s = id - item * a.splits;
  if (!decode_item(a, item, it)) return false;
  const int n = it.n0 > it.n1 ? it.n0 : it.n1;
  const int lo = (int)((long long)n * s / a.splits), hi = (int)((long long)n * (s + 1) / a.splits);
  it.k0 += 128 * lo;
  it.nk = it.nk > 128 * lo ? it.nk - 128 * lo : 0;
  it.n0 = clampi(it.n0 - lo, 0, hi - lo);
  it.n1 = clampi(it.n1 - lo, 0, hi - lo);
  return true;
}

// The items of a CTA (by a whole warp): its own, and then those of CTAs not yet launched, in
// the order of their indices, each asked for while the one before is worked on.
struct Items {
  const FwdArgs& a;
  Ctl* ctl;
  const WaitCtx& w;
  uint32_t asked = 0;
  bool pending = false;

  __device__ __forceinline__ void ask() {
    if (lane_id() == 0) {
      fence_proxy_async_smem();  // the last answer has been read
      mbar_arrive_expect_tx(&ctl->next_full, 16);
      try_cancel(ctl->next, &ctl->next_full);
    }
    __syncwarp();
    pending = true;
  }
  // false: a wait has run out
  __device__ __forceinline__ bool next(Item& it) {
    while (pending) {
      if (!wait_warp(&ctl->next_full, asked & 1, w, 0x15)) return false;
      ++asked;
      pending = false;
      const int id = canceled_cta(ctl->next);
      __syncwarp();
      if (id < 0) break;
      ask();
      if (decode(a, id, it)) return true;
    }
    it.go = 0;
    return true;
  }
  __device__ __forceinline__ void drain() {
    if (pending) wait(&ctl->next_full, asked & 1, w, 0x16, true);
  }
};

__device__ __forceinline__ void load_role(const FwdArgs& a, uint8_t* smem, Ctl* ctl,
                                          const WaitCtx& w, const CUtensorMap* tq,
                                          const CUtensorMap* tk, const CUtensorMap* tv) {
  const bool leader = lane_id() == 0;
  uint32_t st = 0, ph = 0, fills = 0, nq0 = 0, nq1 = 0;  // ring position; loads of Q tiles
  const int half = 128 >> a.pack;
  Items items{a, ctl, w};
  // With an SM for each CTA there is nothing to take over: a CTA not launched yet waits only for the
  // kernel before to leave its SM.
  if (gridDim.x > kSms) items.ask();
  Item it = ctl->own;
  bool ok = it.go || items.next(it);
  for (uint32_t i = 0; ok; ++i) {
    const uint32_t buf = i & 1;
    if (i >= 2 && !wait_warp(&ctl->item_empty[buf], ((i >> 1) + 1) & 1, w, 0x01)) break;
    if (leader) {
      ctl->item[buf] = it;
      mbar_arrive(&ctl->item_full[buf]);
    }
    if (!it.go) break;
    const Item cur = it;
    const int n = cur.n0 > cur.n1 ? cur.n0 : cur.n1;
    auto put = [&](const CUtensorMap* map, int j) {
      if (fills >= (uint32_t)kStages && !wait_warp(&ctl->kv_empty[st], ph ^ 1, w, 0x03)) return false;
      if (leader) {
        mbar_arrive_expect_tx(&ctl->kv_full[st], kTile);
        load_tile(smem + kOffKV + st * kTile, map, &ctl->kv_full[st], cur.k0 + 128 * j,
                  cur.kv_head, cur.z);
      }
      ++fills;
      if (++st == kStages) st = 0, ph ^= 1;
      return true;
    };
    auto put_q = [&](int t, uint32_t& count) {
      if (count > 0 && !wait_warp(&ctl->q_empty[t], (count - 1) & 1, w, 0x04)) return false;
      if (leader) {
        mbar_arrive_expect_tx(&ctl->q_full[t], kTile);
        load_tile(smem + kOffQ + t * kTile, tq, &ctl->q_full[t], cur.q0 + cur.tok + t * half,
                  cur.head0, cur.z);
      }
      ++count;
      return true;
    };
    // K of the first tile ahead of Q: its stage is free long before the Q buffers are
    if (n > 0) {
      ok = put(tk, 0);
      if (ok && cur.n0 > 0) ok = put_q(0, nq0);
      if (ok && cur.n1 > 0) ok = put_q(1, nq1);
      if (ok) ok = put(tv, 0);
    }
    ok = ok && items.next(it);
    for (int j = 1; j < n && ok; ++j) ok = put(tk, j) && put(tv, j);
  }
  items.drain();
  // every copy issued has landed before the CTA exits
  for (uint32_t s = 0; s < (uint32_t)kStages; ++s) {
    const uint32_t f = fills > s ? (fills - s + kStages - 1) / kStages : 0;
    if (f) wait(&ctl->kv_full[s], (f - 1) & 1, w, 0x05, true);
  }
  if (nq0) wait(&ctl->q_full[0], (nq0 - 1) & 1, w, 0x06, true);
  if (nq1) wait(&ctl->q_full[1], (nq1 - 1) & 1, w, 0x06, true);
}

// Query tile t's products.  A unit is O += P(j) V_j and S(j + 1); units of the two tiles
// alternate, a warp passing the turn on when it has issued one.
__device__ __forceinline__ void mma_role(const FwdArgs& a, uint8_t* smem, Ctl* ctl,
                                         const WaitCtx& w, uint32_t tmem, int t) {
  constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128, false, true);
  const uint32_t qd = desc_low(smem_addr(smem + kOffQ + t * kTile), 16);
  const uint32_t kd = desc_low(smem_addr(smem + kOffKV), 16);
  const uint32_t vd = desc_low(smem_addr(smem + kOffKV), kTile / 2);
  const uint32_t tS = tmem + kColS + 128 * t, tO = tmem + kColO + 128 * t;
  const bool leader = lane_id() == 0;
  uint32_t st = 0, ph = 0;        // ring position
  uint32_t items = 0, tiles = 0;  // with keys for this query tile; its key tiles so far
  uint32_t turns = 0;
  auto take = [&] {
    // tile 0 has the first turn
    const bool mine = (t == 0 && turns == 0) ||
                      wait_warp(&ctl->turn[t], (t == 0 ? turns - 1 : turns) & 1, w, 0x0c);
    ++turns;
    return mine;
  };
  auto pass = [&] {
    if (leader) mbar_arrive(&ctl->turn[t ^ 1]);
  };
  auto qk = [&] {
    warp_mma8_ss(tS, qd, kd + st * (kTile >> 4), kIdescS, kTile / 2);
    warp_mma_commit(&ctl->s_full[t]);
  };
  if (a.stall) {  // test hook: a barrier that nothing completes
    wait_warp(&ctl->never, 0, w, 0x1f);
  } else {
    for (uint32_t i = 0;; ++i) {
      const uint32_t buf = i & 1;
      if (!wait_warp(&ctl->item_full[buf], (i >> 1) & 1, w, 0x07)) break;
      const int n0 = ctl->item[buf].n0, n1 = ctl->item[buf].n1, go = ctl->item[buf].go;
      __syncwarp();
      if (leader) mbar_arrive(&ctl->item_empty[buf]);
      if (!go) break;
      const int n = n0 > n1 ? n0 : n1, nt = t ? n1 : n0;
      if (n == 0) continue;
      bool ok = wait_warp(&ctl->ready[st], ph, w, 0x08) &&
                (nt == 0 || wait_warp(&ctl->q_full[t], items & 1, w, 0x09)) && take();
      if (!ok) break;
      if (nt > 0) {
        tc_fence_after();
        qk();
      }
      pass();
      if (nt > 0) {
        warp_mma_commit(&ctl->kv_empty[st]);
        if (nt == 1) warp_mma_commit(&ctl->q_empty[t]);
      } else if (leader) {
        mbar_arrive(&ctl->kv_empty[st]);
      }
      if (++st == kStages) st = 0, ph ^= 1;
      for (int j = 0; j < n; ++j) {
        // V_j has landed, the first half of P(j) is there, and (an item's first product
        // overwrites O) what O held has been read
        ok = wait_warp(&ctl->ready[st], ph, w, 0x0e) &&
             (j >= nt || wait_warp(&ctl->p_full[2 * t], tiles & 1, w, 0x0b)) &&
             (j > 0 || nt == 0 || items == 0 ||
              wait_warp(&ctl->o_empty[t], (items - 1) & 1, w, 0x0a)) &&
             take();
        if (!ok) break;
        const uint32_t vst = st;
        if (j < nt) {
          tc_fence_after();
          warp_mma4_ts(tO, tS, vd + st * (kTile >> 4), kIdescPV, j > 0 ? 1u : 0u);
          ok = wait_warp(&ctl->p_full[2 * t + 1], tiles & 1, w, 0x0b);
          if (!ok) break;
          tc_fence_after();
          warp_mma4_ts(tO, tS + 32, vd + st * (kTile >> 4) + 512, kIdescPV, 1u);
          ++tiles;
        }
        if (++st == kStages) st = 0, ph ^= 1;
        if (j + 1 < n) {
          ok = wait_warp(&ctl->ready[st], ph, w, 0x08);
          if (!ok) break;
          if (j + 1 < nt) {
            tc_fence_after();
            qk();
          }
        }
        pass();
        // (the commits also cover the other product of the unit, issued since)
        if (j < nt) {
          warp_mma_commit(&ctl->kv_empty[vst]);
          if (j + 1 == nt) warp_mma_commit(&ctl->o_full[t]);
        } else if (leader) {
          mbar_arrive(&ctl->kv_empty[vst]);
        }
        if (j + 1 < n) {
          if (j + 1 < nt) {
            warp_mma_commit(&ctl->kv_empty[st]);
            if (j + 2 == nt) warp_mma_commit(&ctl->q_empty[t]);
          } else if (leader) {
            mbar_arrive(&ctl->kv_empty[st]);
          }
          if (++st == kStages) st = 0, ph ^= 1;
        }
      }
      if (!ok) break;
      if (nt > 0) ++items;
    }
  }
  // every MMA issued has completed before TMEM can be released
  warp_mma_commit(&ctl->drain[t]);
  wait(&ctl->drain[t], 0, w, 0x0d, true);
  __syncwarp();
}

// Hands landed tiles on to the MMA warps.
__device__ __forceinline__ void clean_role(uint8_t* smem, Ctl* ctl, const WaitCtx& w) {
  uint32_t st = 0, ph = 0;
  for (uint32_t i = 0;; ++i) {
    const uint32_t buf = i & 1;
    if (!wait_warp(&ctl->item_full[buf], (i >> 1) & 1, w, 0x13)) return;
    const int n0 = ctl->item[buf].n0, n1 = ctl->item[buf].n1;
    const int nk = ctl->item[buf].nk, go = ctl->item[buf].go;
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(&ctl->item_empty[buf]);
    if (!go) return;
    const int n = n0 > n1 ? n0 : n1;
    for (int x = 0; x < 2 * n; ++x) {
      if (!wait_warp(&ctl->kv_full[st], ph, w, 0x14)) return;
      const int rows = nk - 128 * (x >> 1);
      if ((x & 1) && rows < 128) zero_rows(smem + kOffKV + st * kTile, rows);
      if (lane_id() == 0) mbar_arrive(&ctl->ready[st]);
      if (++st == kStages) st = 0, ph ^= 1;
    }
  }
}

__device__ __forceinline__ void softmax_role(const FwdArgs& a, uint8_t* smem, Ctl* ctl,
                                             const WaitCtx& w, uint32_t tmem, int t) {
  const int row = (int)(threadIdx.x & 127);
  const uint32_t lanes = (uint32_t)(((threadIdx.x >> 5) & 3) * 32) << 16;
  const uint32_t tS = tmem + lanes + kColS + 128 * t, tO = tmem + lanes + kColO + 128 * t;
  const float sl2 = a.scale_log2;
  uint32_t done = 0, tiles = 0;  // items with keys, key tiles so far
  const int half = 128 >> a.pack;
  for (uint32_t i = 0;; ++i) {
    const uint32_t buf = i & 1;
    if (!wait_warp(&ctl->item_full[buf], (i >> 1) & 1, w, 0x10)) break;
    // (what only the end needs is read again there: registers are short in the loop)
    if (!ctl->item[buf].go) break;
    const int n = t ? ctl->item[buf].n1 : ctl->item[buf].n0;
    int lim;  // keys this row attends
    {
      const int nq = ctl->item[buf].nq, nk = ctl->item[buf].nk;
      const int tok = ctl->item[buf].tok + t * half + (row & (half - 1));
      lim = a.seq.causal ? clampi(tok + 1 + nk - nq, 0, nk) : nk;
      if (tok >= nq) lim = 0;
    }
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < n; ++j, ++tiles) {
      if (!wait_warp(&ctl->s_full[t], tiles & 1, w, 0x11)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t r[128];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tmem_ld_32x32b_x32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&r[32 * c]));
      tmem_wait_ld();
      float s[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) s[c] = __uint_as_float(r[c]);
      const int left = lim - 128 * j;
      if (__any_sync(0xffffffffu, left < 128)) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= left) s[c] = -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c + 1 < 128; c += 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + 2 * e + 1 < 128) mx[e] = fmax3(mx[e], s[c + 2 * e], s[c + 2 * e + 1]);
      }
      const float top = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * sl2;
      float alpha = 1.0f;
      if (top > m + kRescale) {
        if (m != -INFINITY) alpha = fast_exp2(m - top);
        m = top;
      }
      if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
        // S_t(j) complete: so is the product that O_t held last
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tO + 32 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st_32x32b_x32(tO + 32 * c, o);
        }
      }
      const float neg = m == -INFINITY ? 0.0f : -m;
      const uint64_t c2 = f32x2(sl2, sl2), neg2 = f32x2(neg, neg);
      uint64_t acc_e[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int c = 64 * h + 2 * e;
          float y0, y1;
          split_f32x2(fma_f32x2(f32x2(s[c], s[c + 1]), c2, neg2), y0, y1);
          const float e0 = fast_exp2(y0), e1 = fast_exp2(y1);
          acc_e[e & 1] = add_f32x2(acc_e[e & 1], f32x2(e0, e1));
          pk[e] = pack_bf16x2(e0, e1);
        }
        tmem_st_32x32b_x32(tS + 32 * h, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane_id() == 0) mbar_arrive(&ctl->p_full[2 * t + h]);
      }
      float e0, e1, e2, e3;
      split_f32x2(acc_e[0], e0, e1);
      split_f32x2(acc_e[1], e2, e3);
      l = l * alpha + ((e0 + e1) + (e2 + e3));
    }
    if (!ok) break;
    // a row that attends nothing gets +0 and the sentinel; scores that are no numbers, or all
    // -infinity, give NaN
    const bool some = lim > 0;
    const float inv = some ? 1.0f / l : 0.0f;
    if (n > 0) {
      if (!wait_warp(&ctl->o_full[t], done & 1, w, 0x12)) break;
      ++done;
      tc_fence_after();
    }
    const Item it = ctl->item[buf];
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(&ctl->item_empty[buf]);
    if (a.splits > 1) {
      float* part = a.part + (long long)it.unit * kPartFloats;
      const int at = 128 * t + row;
      part[256 * 128 + at] = m;
      part[256 * 128 + 256 + at] = l;
#pragma unroll 1
      for (int c = 0; c < 4 && n > 0; ++c) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(tO + 32 * c, o);
        tmem_wait_ld();
        if (c == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane_id() == 0) mbar_arrive(&ctl->o_empty[t]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          reinterpret_cast<uint4*>(part + at * 128 + 32 * c)[e] =
              make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
      continue;
    }
    const int n_rows = a.seq.packed ? it.nq : a.seq.Sq;  // tokens that are written
    const int tok = it.tok + t * half + (row & (half - 1));
    const int head = it.head0 + (row >> (7 - a.pack));
    if (tok < n_rows && a.lse != nullptr)
      a.lse[((long long)it.z * a.Hq + head) * a.seq.Sq + it.q0 + tok] =
          some ? (l > 0.0f ? m + log2f(l) : __int_as_float(0x7fffffff)) : kLseEmpty;
    // 32 columns at a time through shared memory, so that a warp's store is 8 rows of 64 bytes,
    // not 32 of 16 (which took 6,000 cycles an item).  (What store_columns does, written out: with
    // that in its place 4 prompts of up to 157 tokens take 10.4 us for 10.0, 19 heads of 8,192 390.5
    // for 389.2.)
    uint8_t* stage = smem + kOffOut + (threadIdx.x >> 5) * 2048;
    const uint32_t lane = lane_id();
    const int r0 = (int)(threadIdx.x & 96);  // the warp's first row of the tile
    uint16_t* base = a.out + it.z * a.out_b + (long long)(it.q0 + it.tok + t * half) * a.out_t;
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {
      uint32_t o[32];
      if (n > 0) {
        tmem_ld_32x32b_x32(tO + 32 * h, o);
        tmem_wait_ld();
        if (h == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->o_empty[t]);
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t x[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          x[y] = some && n > 0 ? pack_bf16x2(__uint_as_float(o[8 * c + 2 * y]) * inv,
                                             __uint_as_float(o[8 * c + 2 * y + 1]) * inv)
                               : 0u;
        // (pieces of 16 bytes, turned by the row so that eight rows' meet all banks)
        *reinterpret_cast<uint4*>(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) * 16)) =
            make_uint4(x[0], x[1], x[2], x[3]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t rr = 8 * i + (lane >> 2), c = lane & 3;
        const uint4 x =
            *reinterpret_cast<const uint4*>(stage + rr * 64 + ((c ^ ((rr >> 1) & 3)) * 16));
        const int row = r0 + (int)rr, off = row & (half - 1);
        if (it.tok + t * half + off < n_rows)
          *reinterpret_cast<uint4*>(base + (it.head0 + (row >> (7 - a.pack))) * a.out_h +
                                    (long long)off * a.out_t + 32 * h + 8 * c) = x;
      }
      __syncwarp();
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    prompt_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const FwdArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + kOffCtl);
  const uint32_t warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->item_full[i], 1);
      mbar_init(&ctl->item_empty[i], 11);  // 2 MMA and 8 softmax warps, warp 11
      mbar_init(&ctl->turn[i], 1);
      mbar_init(&ctl->drain[i], 1);
      mbar_init(&ctl->q_full[i], 1);
      mbar_init(&ctl->q_empty[i], 1);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[2 * i], 4);
      mbar_init(&ctl->p_full[2 * i + 1], 4);
      mbar_init(&ctl->o_full[i], 1);
      mbar_init(&ctl->o_empty[i], 4);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&ctl->kv_full[i], 1);
      mbar_init(&ctl->ready[i], 1);
      mbar_init(&ctl->kv_empty[i], 2);  // both MMA warps
    }
    mbar_init(&ctl->never, 1);
    mbar_init(&ctl->next_full, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane_id() == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 9) {
    tmem_alloc(&ctl->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  // What comes before runs while the predecessor in the stream ends.  (A successor may not start
  // up likewise: CTAs of this grid that are taken over are never launched.)
  wait_predecessor();
  if (warp == 8) {  // the CTA's own item is looked up while the others get ready
    Item it;
    const bool holds = decode(a, (int)blockIdx.x, it);
    it.go = holds ? 1 : 0;
    if (lane_id() == 0) ctl->own = it;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const WaitCtx w{&ctl->abort_flag, a.status, a.wait_ns};

  if (warp < 8) {
    regs_increase<kSoftmaxRegs>();
    softmax_role(a, smem, ctl, w, tmem, (int)(warp >> 2));
  } else {
    regs_decrease<kOtherRegs>();
    if (warp == 8)
      load_role(a, smem, ctl, w, &tq, &tk, &tv);
    else if (warp < 11)
      mma_role(a, smem, ctl, w, tmem, (int)warp - 9);
    else
      clean_role(smem, ctl, w);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, kTmemCols);
}

// Joins the ranges of split items, a warp a row: with M = max m_s and c_s = 2^(m_s - M), out =
// sum c_s O_s / sum c_s l_s and lse = M + log2 sum c_s l_s, in the order of the ranges.
__global__ void __launch_bounds__(256) prompt_join_kernel(const FwdArgs a) {
  after_predecessor();
  const int item = (int)(blockIdx.x >> 5);
  const int at = (int)((blockIdx.x & 31) * 8 + (threadIdx.x >> 5)), t = at >> 7, row = at & 127;
  const int lane = (int)lane_id();
  Item it;
  if (!decode_item(a, item, it)) return;
  const int half = 128 >> a.pack;
  const int tok = it.tok + t * half + (row & (half - 1));
  const int head = it.head0 + (row >> (7 - a.pack));
  if (tok >= (a.seq.packed ? it.nq : a.seq.Sq)) return;
  int lim = a.seq.causal ? clampi(tok + 1 + it.nk - it.nq, 0, it.nk) : it.nk;
  if (tok >= it.nq) lim = 0;
  const float* part = a.part + (long long)item * a.splits * kPartFloats;
  float m = -INFINITY, l = 0.0f;
  if (lane < a.splits) {
    m = part[(long long)lane * kPartFloats + 256 * 128 + at];
    l = part[(long long)lane * kPartFloats + 256 * 128 + 256 + at];
  }
  float top = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  // (a range that the row attends nothing of has l = 0, and its O may not have been written; a
  // sum that is no number stays one)
  const float c = l != l ? 1.0f : (l == 0.0f ? 0.0f : fast_exp2(m - top));
  float sum = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < a.splits; ++s) {
    const float cs = __shfl_sync(0xffffffffu, c, s), ls = __shfl_sync(0xffffffffu, l, s);
    if (cs == 0.0f) continue;
    const float4 o = reinterpret_cast<const float4*>(part + (long long)s * kPartFloats +
                                                     at * 128)[lane];
    sum = fmaf(cs, ls, sum);
    acc.x = fmaf(cs, o.x, acc.x);
    acc.y = fmaf(cs, o.y, acc.y);
    acc.z = fmaf(cs, o.z, acc.z);
    acc.w = fmaf(cs, o.w, acc.w);
  }
  const bool some = lim > 0;
  const float inv = 1.0f / sum;
  uint2 x = make_uint2(0u, 0u);
  if (some) x = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  reinterpret_cast<uint2*>(a.out + it.z * a.out_b + head * a.out_h +
                           (long long)(it.q0 + tok) * a.out_t)[lane] = x;
  if (lane == 0 && a.lse != nullptr)
    a.lse[((long long)it.z * a.Hq + head) * a.seq.Sq + it.q0 + tok] =
        some ? (sum > 0.0f ? top + log2f(sum) : __int_as_float(0x7fffffff)) : kLseEmpty;
}

}  // namespace fwd
}  // namespace prompt
}  // namespace vsa

// vsa_prompt_bwd_kernel.cuh -- gradient of the attention over whole prompts.
//
// With p_ij = 2^(c q_i.k_j - lse_i) over the attended pairs (c = scale log2 e), D_i = dout_i .
// out_i and ds_ij = p_ij (dout_i . v_j - D_i):
//   dv_j = sum_i p_ij dout_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j,
// dk and dv summed over the query heads of a key/value head.
//
// Two kernels, without atomics, so results do not depend on timing:
//   prompt_dq_kernel    a CTA per query tile: Q and dO stay, dQ adds up in TMEM while it
//                       walks the key tiles: S = Q K^T, dP = dO V^T, dS, dQ += dS K.  It sets
//                       out with the rows' D and leaves -lse and -D for the other kernel, in
//                       the order of the query tiles.
//                       out is rounded to bf16, and D with it; but where a row's p add up to 1
//                       its dS add up to 0, so what they come to is that error: it is taken off
//                       D for the next kernel, and here off the dS of rows of one key tile.
//                       (Relative errors in norm, with and without: 12 heads of up to 411 tokens
//                       dk and dq 0.0024 and 0.0026, sequences of 2 to 16 tokens 0.0024 and
//                       0.0030; inputs three times as large, 400 tokens, dk 0.0023 and 0.0055.)
//                       Where they add up to something else, lse being over more keys than this
//                       call's, D stays as it is.  kWhole tells the two apart: a row whose other
//                       keys weigh that little or less has D off by kWhole dout . (what out is
//                       over these keys, less what over those), about half of the rounding's.
//   prompt_dkv_kernel   a CTA per key tile of 128 keys and key/value head: K and V stay in
//                       shared memory, dK and dV add up in TMEM while it walks the query
//                       tiles that see the keys.  Per step, transposed (lanes = keys):
//                         S^T = K Q^T, dP^T = V dO^T           (SS, both K-major)
//                         P^T = 2^(c S^T - lse), dS^T = P^T (dP^T - D)  -> bf16 over S^T, dP^T
//                         dV += P^T dO, dK += dS^T Q           (TS, A from TMEM)
// That is seven products where one kernel with atomic sums of dQ takes five, but those sums
// are 64 KB of L2 reductions a step, and their order would be anyone's.  P and dS are rounded
// to bf16 for the products, everything else is fp32.
//
// A step's products take 512 tensor cycles each (128 x 128 x 128), issued by two warps that run
// converged (elect.sync picks the lane: one lane issuing for itself took 60 cycles and more a
// product's sixteenth, and the kernels ran at 0.78 of what they do):
//   dkv  warp 9 dV_g, S_{g+1}; warp 10 dK_g, dP_{g+1}; a unit each in turn.  P_{g+1} may take as
//        long as warp 10's unit, dS_{g+1} as long as warp 9's.  S_{g+1} overwrites P_g, dP_{g+1}
//        overwrites dS_g: MMAs of one warp run in order.
//   dq   warp 9 S_{g+1}, dP_{g+1} (two buffers of dP / dS; the one that dQ_{g-1} read), warp 10
//        dQ_g.
// With 19 heads of 8,192 tokens the tensor pipe is busy 73 % (dkv) and 70 % (dq) of the time at
// 1.9 GHz, 1,720 and 1,625 TFLOP/s of their own products; what is left are the round trips through
// barriers and TMEM of a step's chain, and 4 us a CTA of start and end.
//
// Where there are fewer tiles than SMs the steps of each are cut into ranges, a CTA each, and a
// kernel more adds up what they leave, in order.
//
// 12 warps: 0-7 gradient warps (thread = lane of the tile, warpgroup w = columns 64 w ..),
// 8 TMA, 9 and 10 MMA issuers, 11 hands landed tiles on to them and zeroes rows that are not the
// sequence's, and queries that attend nothing, first: they get weight 0, but 0 times what lies
// there (another sequence, padding, a dout of anything) may be NaN.
#pragma once

#include "vsa_prompt_common.cuh"

namespace vsa {
namespace prompt {
namespace bwd {

constexpr int kThreads = 384;
constexpr uint32_t kGradRegs = 216, kOtherRegs = 56;
constexpr uint32_t kRegPoolNeeded = 256 * kGradRegs + 128 * kOtherRegs;
constexpr uint32_t kTmemCols = 512;

struct Args {
  SeqArgs seq;
  float* stats;  // [n_packs][n_tslots][-lse | -D][128]
  int splits;    // ranges of a tile's steps, a CTA each
  float* part;   // their partial results, if there are several
  uint16_t *d0, *d1;   // dkv: dk, dv; dq: dq, null
  long long d0_b, d0_h, d0_t, d1_b, d1_h, d1_t;  // strides in elements
  const uint16_t *out, *dout;  // read row by row by dq
  const float* lse;
  long long o_b, o_h, o_t, g_b, g_h, g_t;
  unsigned int* status;
  int Hq, Hkv, group, pack, n_packs, n_tslots;  // query tiles of 128 >> pack tokens
  float scale, scale_log2;
  unsigned long long wait_ns;
  int stall;
};

// the slot of a sequence's query tile (as tile_slots numbers them)
__device__ __forceinline__ long long query_slot(const Args& a, int b, int q0, int tile) {
  const int T = 128 >> a.pack;
  return a.seq.packed ? (long long)(q0 / T) + b + tile
                      : (long long)b * ((a.seq.Sq + T - 1) / T) + tile;
}

// --------------------------------------------------------------------------- dK and dV
namespace dkv {

constexpr int kQStages = 3, kGStages = 2;
constexpr uint32_t kOffK = 0, kOffV = kTile, kOffQ = 2 * kTile;
constexpr uint32_t kOffG = kOffQ + kQStages * kTile;
constexpr uint32_t kOffStats = kOffG + kGStages * kTile;  // [kGStages] -lse[128], -D[128]
constexpr uint32_t kOffCtl = kOffStats + kGStages * 1024;
constexpr uint32_t kSmemBytes = kOffCtl + 1024;  // (no room for slack: the base is aligned)
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 384;

struct Ctl {
  uint64_t kv_full;
  uint64_t q_full[kQStages], q_ready[kQStages], q_empty[kQStages];
  uint64_t g_full[kGStages], g_ready[kGStages], g_empty[kGStages];
  uint64_t s_full, dp_full, p_full, ds_full, acc_full, turn[2], drain[2], never;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Ctl) <= 1024, "control block");

// A CTA's work: key tile `tile` of sequence b, and the query tiles that see it.
struct Work {
  Seq s;
  int b, tile, hk;
  int first, n_tok;   // first query tile and their number, for each head pack
  int hp0;            // first head pack
  int step0, steps;   // first step of the CTA's range, and their number
  int nk;             // keys of the tile
  bool there;
};

__global__ void __launch_bounds__(kThreads, 1)
    prompt_dkv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tg,
                      const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                      const Args a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_addr(smem) & 1023u) {  // the swizzle goes by address bits
    atomicCAS(a.status, 0u, kErrTimeout | 0xffu);
    return;
  }
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + kOffCtl);
  const int warp = (int)(threadIdx.x >> 5);
  const uint32_t lane = lane_id();
  const int T = 128 >> a.pack;

  if (threadIdx.x == 0) {
    mbar_init(&ctl->kv_full, 1);
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(&ctl->q_full[i], 1);
      mbar_init(&ctl->q_ready[i], 1);
      mbar_init(&ctl->q_empty[i], 1);
    }
    for (int i = 0; i < kGStages; ++i) {
      mbar_init(&ctl->g_full[i], 1);
      mbar_init(&ctl->g_ready[i], 1);
      mbar_init(&ctl->g_empty[i], 9);  // dV done; the gradient warps have read -D
    }
    mbar_init(&ctl->s_full, 1);
    mbar_init(&ctl->dp_full, 1);
    mbar_init(&ctl->p_full, 8);
    mbar_init(&ctl->ds_full, 8);
    mbar_init(&ctl->acc_full, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->turn[i], 1);
      mbar_init(&ctl->drain[i], 1);
    }
    mbar_init(&ctl->never, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tg);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 9) {
    tmem_alloc(&ctl->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const WaitCtx w{&ctl->abort_flag, a.status, a.wait_ns};
  // (what comes before may run while the predecessor ends)
  after_predecessor();
  Work k;
  const unsigned item = blockIdx.x / (unsigned)a.splits, split = blockIdx.x - item * a.splits;
  {
    const int slot = (int)(item / (unsigned)a.Hkv);
    k.hk = (int)(item - (unsigned)slot * (unsigned)a.Hkv);
    const Place p = find_tile(a.seq, slot, 7, true);
    k.s = p.s;
    k.b = p.b;
    k.tile = p.tile;
    k.there = p.there;
    k.nk = clampi(k.s.nk - 128 * k.tile, 0, 128);
    int first = 0;
    if (a.seq.causal) first = clampi(128 * k.tile - (k.s.nk - k.s.nq), 0, k.s.nq);
    k.first = first / T;
    k.n_tok = k.nk > 0 && first < k.s.nq ? (k.s.nq + T - 1) / T - k.first : 0;
    if (!k.there) k.n_tok = 0;
    k.hp0 = (k.hk * a.group) >> a.pack;
    const long long all = (long long)k.n_tok * (a.group >> a.pack);
    k.step0 = (int)(all * split / a.splits);
    k.steps = (int)(all * (split + 1) / a.splits) - k.step0;
  }
  const int off = k.s.nk - k.s.nq;

  if (warp < 8) {
    regs_increase<kGradRegs>();
    const int wg = warp >> 2;
    const int r = (warp & 3) * 32 + (int)lane;  // key of the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + kColS + 64 * wg, tDP = tmem + lanes + kColDP + 64 * wg;
    const uint64_t c2 = f32x2(a.scale_log2, a.scale_log2);
    bool ok = true;
    int ti = k.n_tok ? k.first + k.step0 % k.n_tok : 0;
    for (int g = 0; g < k.steps; ++g) {
      const int st = g & 1;
      const float* nlse = reinterpret_cast<const float*>(smem + kOffStats + st * 1024) + 64 * wg;
      const float* nD = nlse + 128;
      if (!wait_warp(&ctl->g_full[st], (g >> 1) & 1, w, 0x20) ||
          !wait_warp(&ctl->s_full, g & 1, w, 0x21)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t x[64];
      tmem_ld_32x32b_x32(tS, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
      tmem_ld_32x32b_x32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
      tmem_wait_ld();
      float p[64];
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        const float4 l = *reinterpret_cast<const float4*>(nlse + c);
        float y0, y1, y2, y3;
        split_f32x2(fma_f32x2(f32x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), c2,
                              f32x2(l.x, l.y)), y0, y1);
        split_f32x2(fma_f32x2(f32x2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), c2,
                              f32x2(l.z, l.w)), y2, y3);
        p[c] = fast_exp2(y0);
        p[c + 1] = fast_exp2(y1);
        p[c + 2] = fast_exp2(y2);
        p[c + 3] = fast_exp2(y3);
      }
      // causal: query token t sees this key from t = 128 tile + r - off on
      if (a.seq.causal && 128 * k.tile + 127 > ti * T + off) {
        const int from = 128 * k.tile + r - off - ti * T;
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (((64 * wg + c) & (T - 1)) < from) p[c] = 0.0f;
      }
      uint32_t pk[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) pk[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
      tmem_st_32x32b_x32(tS, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->p_full);
      if (!wait_warp(&ctl->dp_full, g & 1, w, 0x22)) {
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_ld_32x32b_x32(tDP, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
      tmem_ld_32x32b_x32(tDP + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        const float4 d = *reinterpret_cast<const float4*>(nD + c);
        float y0, y1, y2, y3;
        split_f32x2(mul_f32x2(f32x2(p[c], p[c + 1]),
                              add_f32x2(f32x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])),
                                        f32x2(d.x, d.y))), y0, y1);
        split_f32x2(mul_f32x2(f32x2(p[c + 2], p[c + 3]),
                              add_f32x2(f32x2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])),
                                        f32x2(d.z, d.w))), y2, y3);
        pk[c / 2] = pack_bf16x2(y0, y1);
        pk[c / 2 + 1] = pack_bf16x2(y2, y3);
      }
      tmem_st_32x32b_x32(tDP, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl->ds_full);
        mbar_arrive(&ctl->g_empty[st]);
      }
      if (++ti == k.first + k.n_tok) ti = k.first;
    }
    // dV (warpgroup 0) and dK (warpgroup 1)
    if (k.steps > 0 && ok) ok = wait_warp(&ctl->acc_full, 0, w, 0x23);
    if (ok && k.there) {
      tc_fence_after();
      const int rows = a.seq.packed ? k.nk : a.seq.Sk - 128 * k.tile;  // that are written
      uint16_t* base = (wg ? a.d0 + k.s.z * a.d0_b + k.hk * a.d0_h
                           : a.d1 + k.s.z * a.d1_b + k.hk * a.d1_h) +
                       (k.s.k0 + 128ll * k.tile) * (wg ? a.d0_t : a.d1_t);
      const long long stride = wg ? a.d0_t : a.d1_t;
      const float f = wg ? a.scale : 1.0f;
      float* part = a.part + ((long long)blockIdx.x * 2 + (wg ? 0 : 1)) * (128 * 128) + r * 128;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32];
        if (k.steps > 0) {
          tmem_ld_32x32b_x32(tmem + lanes + (wg ? kColDK : kColDV) + 32 * c, x);
          tmem_wait_ld();
        }
        if (a.splits == 1) {
          // (the Q stages are free by now)
          store_columns(smem + kOffQ + warp * 2048, x, f, k.steps > 0 && r < k.nk, [&](int i) {
            const int rr = (warp & 3) * 32 + i;
            return rr < rows ? base + rr * stride + 32 * c : nullptr;
          });
        } else if (k.steps > 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            reinterpret_cast<uint4*>(part + 32 * c)[e] =
                make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        }
      }
    }
  } else {
    regs_decrease<kOtherRegs>();
    if (warp == 8) {
      if (lane == 0 && k.steps > 0) {
        mbar_arrive_expect_tx(&ctl->kv_full, 2 * kTile);
        load_tile(smem + kOffK, &tk, &ctl->kv_full, k.s.k0 + 128 * k.tile, k.hk, k.s.z);
        load_tile(smem + kOffV, &tv, &ctl->kv_full, k.s.k0 + 128 * k.tile, k.hk, k.s.z);
        int ti = k.first + k.step0 % k.n_tok, hp = k.hp0 + k.step0 / k.n_tok, g = 0;
        const long long slot0 = query_slot(a, k.b, k.s.q0, 0);
        for (; g < k.steps; ++g) {
          const int qs = g % kQStages, gs = g % kGStages;
          if (g >= kQStages && !wait(&ctl->q_empty[qs], (g / kQStages + 1) & 1, w, 0x24)) break;
          mbar_arrive_expect_tx(&ctl->q_full[qs], kTile);
          load_tile(smem + kOffQ + qs * kTile, &tq, &ctl->q_full[qs], k.s.q0 + ti * T,
                    hp << a.pack, k.s.z);
          if (g >= kGStages && !wait(&ctl->g_empty[gs], (g / kGStages + 1) & 1, w, 0x25)) {
            wait(&ctl->q_full[qs], (g / kQStages) & 1, w, 0x26, true);  // this one has no pair
            break;
          }
          mbar_arrive_expect_tx(&ctl->g_full[gs], kTile + 1024);
          load_tile(smem + kOffG + gs * kTile, &tg, &ctl->g_full[gs], k.s.q0 + ti * T,
                    hp << a.pack, k.s.z);
          bulk_load(smem + kOffStats + gs * 1024,
                    a.stats + ((long long)hp * a.n_tslots + slot0 + ti) * 256, 1024,
                    &ctl->g_full[gs]);
          if (++ti == k.first + k.n_tok) {
            ti = k.first;
            ++hp;
          }
        }
        // every copy issued has landed before the CTA exits
        wait(&ctl->kv_full, 0, w, 0x27, true);
        for (int i = 0; i < kQStages; ++i) {
          const int fills = g > i ? (g - i + kQStages - 1) / kQStages : 0;
          if (fills) wait(&ctl->q_full[i], (fills - 1) & 1, w, 0x28, true);
        }
        for (int i = 0; i < kGStages; ++i) {
          const int fills = g > i ? (g - i + kGStages - 1) / kGStages : 0;
          if (fills) wait(&ctl->g_full[i], (fills - 1) & 1, w, 0x29, true);
        }
      }
      __syncwarp();
    } else if (warp == 9 || warp == 10) {
      // warp 9: dV_g, S_{g+1}; warp 10: dK_g, dP_{g+1}; a unit each in turn
      if (k.steps > 0) {
        constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t kIdescG = idesc_bf16_f32(128, 128, false, true);
        const int x = warp - 9;
        const uint32_t sa = smem_addr(smem);
        // A of the scores (K or V), the ring that both of the warp's products read
        const uint32_t ad = desc_low(sa + (x ? kOffV : kOffK), 16);
        const uint32_t b_k = desc_low(sa + (x ? kOffG : kOffQ), 16);          // K-major
        const uint32_t b_mn = desc_low(sa + (x ? kOffQ : kOffG), kTile / 2);  // MN-major
        const uint32_t col = x ? kColDP : kColS, acc = x ? kColDK : kColDV;
        uint64_t* const full = x ? &ctl->dp_full : &ctl->s_full;
        uint64_t* const ready = x ? &ctl->ds_full : &ctl->p_full;
        auto q_in = [&](int g) {
          return wait_warp(&ctl->q_ready[g % kQStages], (g / kQStages) & 1, w, 0x2a);
        };
        auto g_in = [&](int g) {
          return wait_warp(&ctl->g_ready[g % kGStages], (g / kGStages) & 1, w, 0x2b);
        };
        // S^T or dP^T of step g
        auto scores = [&](int g) {
          const uint32_t st = x ? (uint32_t)(g % kGStages) : (uint32_t)(g % kQStages);
          tc_fence_after();
          warp_mma8_ss(tmem + col, ad, b_k + st * (kTile >> 4), kIdescS, kTile / 2);
          warp_mma_commit(full);
        };
        bool ok = a.stall ? wait_warp(&ctl->never, 0, w, 0x3f)
                          : wait_warp(&ctl->kv_full, 0, w, 0x2c) && (x ? g_in(0) : q_in(0));
        if (ok) scores(0);
        for (int g = 0; g < k.steps && ok; ++g) {
          const bool more = g + 1 < k.steps;
          // the next scores' operands; P or dS; the gradient product's own tile, which for dK is
          // there already (g_in(g) was waited for, and warp 11 hands Q on before dO)
          ok = (!more || (x ? g_in(g + 1) : q_in(g + 1))) && (x || g_in(g)) &&
               wait_warp(ready, g & 1, w, 0x2d) &&
               ((x == 0 && g == 0) || wait_warp(&ctl->turn[x], (x ? g : g - 1) & 1, w, 0x32));
          if (!ok) break;
          const uint32_t st = x ? (uint32_t)(g % kQStages) : (uint32_t)(g % kGStages);
          tc_fence_after();
          warp_mma4_ts(tmem + acc, tmem + col, b_mn + st * (kTile >> 4), kIdescG, g > 0 ? 1u : 0u);
          warp_mma4_ts(tmem + acc, tmem + col + 64, b_mn + st * (kTile >> 4) + 512, kIdescG, 1u);
          if (more) scores(g + 1);
          if (lane == 0) mbar_arrive(&ctl->turn[x ^ 1]);
          // (the commit also covers the next scores, issued since)
          warp_mma_commit(x ? &ctl->q_empty[st] : &ctl->g_empty[st]);
          if (!more) warp_mma_commit(&ctl->acc_full);
        }
        warp_mma_commit(&ctl->drain[x]);
        wait(&ctl->drain[x], 0, w, 0x2f, true);
      }
      __syncwarp();
    } else if (warp == 11) {
      int ti = k.n_tok ? k.first + k.step0 % k.n_tok : 0;
      const int none = a.seq.causal ? k.s.nq - k.s.nk : 0;  // first queries, that attend nothing
      for (int g = 0; g < k.steps; ++g) {
        const int qs = g % kQStages, gs = g % kGStages;
        const int from = none - ti * T, to = k.s.nq - ti * T;  // tokens of the tile that count
        const bool clean = from > 0 || to < T;
        if (!wait_warp(&ctl->q_full[qs], (g / kQStages) & 1, w, 0x30)) break;
        if (clean) zero_tokens(smem + kOffQ + qs * kTile, from, to, T);
        if (lane == 0) mbar_arrive(&ctl->q_ready[qs]);
        if (!wait_warp(&ctl->g_full[gs], (g / kGStages) & 1, w, 0x31)) break;
        if (clean) zero_tokens(smem + kOffG + gs * kTile, from, to, T);
        if (lane == 0) mbar_arrive(&ctl->g_ready[gs]);
        if (++ti == k.first + k.n_tok) ti = k.first;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, kTmemCols);
}

// Adds up the ranges of a tile's steps, in their order: a warp a row, dk and dv.
__global__ void __launch_bounds__(256) prompt_dkv_join_kernel(const Args a) {
  after_predecessor();
  const unsigned item = blockIdx.x >> 5;
  const int at = (int)((blockIdx.x & 31) * 8 + (threadIdx.x >> 5)), r = at & 127;
  const int lane = (int)lane_id();
  const int slot = (int)(item / (unsigned)a.Hkv), hk = (int)(item - (unsigned)slot * a.Hkv);
  const Place p = find_tile(a.seq, slot, 7, true);
  const Seq& s = p.s;
  const int tile = p.tile;
  if (!p.there || 128ll * tile + r >= (a.seq.packed ? s.nk : a.seq.Sk)) return;
  const int T = 128 >> a.pack;
  int first = 0;
  if (a.seq.causal) first = clampi(128 * tile - (s.nk - s.nq), 0, s.nq);
  const int n_tok = first < s.nq && 128 * tile + r < s.nk ? (s.nq + T - 1) / T - first / T : 0;
  const long long all = (long long)n_tok * (a.group >> a.pack);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < a.splits; ++i) {
    if (all * (i + 1) / a.splits == all * i / a.splits) continue;  // a range of nothing
    const float4 x = reinterpret_cast<const float4*>(
        a.part + (((long long)item * a.splits + i) * 2 + (at >> 7)) * (128 * 128) + r * 128)[lane];
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
  }
  const float f = at < 128 ? a.scale : 1.0f;
  const long long row = s.k0 + 128ll * tile + r;
  uint16_t* dst = at < 128 ? a.d0 + s.z * a.d0_b + hk * a.d0_h + row * a.d0_t
                           : a.d1 + s.z * a.d1_b + hk * a.d1_h + row * a.d1_t;
  reinterpret_cast<uint2*>(dst)[lane] =
      make_uint2(pack_bf16x2(acc.x * f, acc.y * f), pack_bf16x2(acc.z * f, acc.w * f));
}

}  // namespace dkv

// ---------------------------------------------------------------------------------- dQ
namespace dq {

constexpr int kKStages = 3, kVStages = 2;
constexpr uint32_t kOffQ = 0, kOffG = kTile, kOffK = 2 * kTile;
constexpr uint32_t kOffV = kOffK + kKStages * kTile;
constexpr uint32_t kOffXch = kOffV + kVStages * kTile;  // a row's sums, of a warpgroup each
constexpr uint32_t kOffCtl = kOffXch + 2048;
constexpr uint32_t kSmemBytes = kOffCtl + 1024;  // (the base is aligned)
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
constexpr uint32_t kColS = 0, kColDP = 128, kColDQ = 384;  // dP twice
constexpr int kPartFloats = 128 * 128 + 128;  // of a range: dQ (and 128 that stay unused)
constexpr float kWhole = 1.0f / 2048.0f;

struct Ctl {
  uint64_t q_full;
  uint64_t k_full[kKStages], k_ready[kKStages], k_empty[kKStages];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t s_full, s_empty, dp_full[2], ds_full[2], ds_empty[2], x_full[4], acc_full, drain[2];
  uint64_t never;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Ctl) <= 1024, "control block");

__global__ void __launch_bounds__(kThreads, 1)
    prompt_dq_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tg,
                     const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                     const Args a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_addr(smem) & 1023u) {  // the swizzle goes by address bits
    atomicCAS(a.status, 0u, kErrTimeout | 0xffu);
    return;
  }
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + kOffCtl);
  const int warp = (int)(threadIdx.x >> 5);
  const uint32_t lane = lane_id();
  const int T = 128 >> a.pack;

  if (threadIdx.x == 0) {
    mbar_init(&ctl->q_full, 1);
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&ctl->k_full[i], 1);
      mbar_init(&ctl->k_ready[i], 1);
      mbar_init(&ctl->k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&ctl->v_full[i], 1);
      mbar_init(&ctl->v_empty[i], 1);
      mbar_init(&ctl->dp_full[i], 1);
      mbar_init(&ctl->ds_full[i], 8);
      mbar_init(&ctl->ds_empty[i], 1);
      mbar_init(&ctl->drain[i], 1);
    }
    mbar_init(&ctl->s_full, 1);
    mbar_init(&ctl->s_empty, 8);
    for (int i = 0; i < 4; ++i) mbar_init(&ctl->x_full[i], 2);
    mbar_init(&ctl->acc_full, 1);
    mbar_init(&ctl->never, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tg);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 9) {
    tmem_alloc(&ctl->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const WaitCtx w{&ctl->abort_flag, a.status, a.wait_ns};
  // (what comes before may run while the predecessor ends)
  after_predecessor();
  const unsigned item = blockIdx.x / (unsigned)a.splits, split = blockIdx.x - item * a.splits;
  const int rank = (int)(item / (unsigned)a.n_packs);
  const int hp = (int)(item - (unsigned)rank * (unsigned)a.n_packs);
  const Place place = find_tile(a.seq, rank, 7 - a.pack, false);
  const Seq s = place.s;
  const int b = place.b, tile = place.tile;
  const bool there = place.there;
  const int off = s.nk - s.nq;
  const int tok0 = tile * T, head0 = hp << a.pack, hk = head0 / a.group;
  int keys = there && tok0 < s.nq ? s.nk : 0;
  if (a.seq.causal) keys = clampi((tok0 + T < s.nq ? tok0 + T : s.nq) + off, 0, keys);
  const int all_steps = (keys + 127) / 128;
  const int step0 = (int)((long long)all_steps * split / a.splits);
  const int steps = (int)((long long)all_steps * (split + 1) / a.splits) - step0;
  const int k_first = s.k0 + 128 * step0, nk = s.nk - 128 * step0;  // of the CTA's range


  if (warp < 8) {
    regs_increase<kGradRegs>();
    const int wg = warp >> 2;
    const int r = (warp & 3) * 32 + (int)lane;  // row of the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + kColS + 64 * wg, tDP = tmem + lanes + kColDP + 64 * wg;
    const int tok = tok0 + (r & (T - 1));
    float* st = a.stats + ((long long)hp * a.n_tslots + query_slot(a, b, s.q0, tile)) * 256;
    float* xch = reinterpret_cast<float*>(smem + kOffXch);  // [2][2][128]
    uint64_t sum2 = f32x2(0.0f, 0.0f), sump = sum2;         // of the row's dS, of its p
    // with the warp that has the rows' other columns
    auto meet = [&](uint32_t parity) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->x_full[warp & 3]);
      return wait_warp(&ctl->x_full[warp & 3], parity, w, 0x50);
    };
    // what the row's dS come to, if that is the rounding of out in D, else 0
    float rest = 0.0f;
    auto find_rest = [&] {
      float s0, s1, p0, p1;
      split_f32x2(sum2, s0, s1);
      split_f32x2(sump, p0, p1);
      // (where D was, once the other warp has read it)
      if (!wait_warp(&ctl->x_full[warp & 3], 1, w, 0x50)) return false;
      xch[128 * wg + r] = s0 + s1;
      xch[256 + 128 * wg + r] = p0 + p1;
      if (!meet(0)) return false;
      const float all = xch[256 + r] + xch[384 + r];
      if (fabsf(all - 1.0f) <= kWhole) rest = xch[r] + xch[128 + r];
      return true;
    };
    int lim = s.nk;  // keys this row attends
    if (a.seq.causal) lim = clampi(tok + 1 + off, 0, s.nk);
    // the row's -lse (-infinity where it attends nothing, or is none of the sequence's, so that
    // every p of it is 0) and -D = -sum_d dout out (0 there, whatever dout holds), this
    // warpgroup's half of the columns
    const bool in = there && tok < s.nq && lim > 0;
    float nlse = -INFINITY, part_d = 0.0f;
    if (in) {
      const int head = head0 + (r >> (7 - a.pack));
      const long long row = s.q0 + tok;
      const uint4* o = reinterpret_cast<const uint4*>(a.out + s.z * a.o_b + head * a.o_h +
                                                      row * a.o_t + 64 * wg);
      const uint4* g = reinterpret_cast<const uint4*>(a.dout + s.z * a.g_b + head * a.g_h +
                                                      row * a.g_t + 64 * wg);
      const float l = read_global(a.lse + ((long long)s.z * a.Hq + head) * a.seq.Sq + row);
      if (!(l <= -3.0e38f)) nlse = -l;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = read_global(o + 4 * h + i);
          y[i] = read_global(g + 4 * h + i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t ow[4] = {x[i].x, x[i].y, x[i].z, x[i].w},
                         gw[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            part_d = fmaf(bf16_lo(ow[e]), bf16_lo(gw[e]), part_d);
            part_d = fmaf(bf16_hi(ow[e]), bf16_hi(gw[e]), part_d);
          }
        }
      }
    }
    xch[128 * wg + r] = part_d;
    bool ok = meet(0);
    const float nD = -(part_d + xch[128 * (wg ^ 1) + r]);
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->x_full[warp & 3]);
    if (wg == 0 && split + 1 == (unsigned)a.splits && there) {  // (the last range has a row's last key)
      st[r] = nlse;
      st[128 + r] = in ? nD : 0.0f;
    }
    lim -= 128 * step0;  // counted from the range's first key
    const uint64_t c2 = f32x2(a.scale_log2, a.scale_log2), l2 = f32x2(nlse, nlse),
                   d2 = f32x2(nD, nD);
    for (int g = 0; g < steps && ok; ++g) {
      if (!wait_warp(&ctl->s_full, g & 1, w, 0x40)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t x[64];
      tmem_ld_32x32b_x32(tS, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
      tmem_ld_32x32b_x32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->s_empty);
      float p[64];
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        float y0, y1;
        split_f32x2(fma_f32x2(f32x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), c2, l2),
                    y0, y1);
        p[c] = fast_exp2(y0);
        p[c + 1] = fast_exp2(y1);
      }
      if (!wait_warp(&ctl->dp_full[g & 1], (g >> 1) & 1, w, 0x41)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t t = tDP + 128 * (g & 1);
      tmem_ld_32x32b_x32(t, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
      tmem_ld_32x32b_x32(t + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
      tmem_wait_ld();
      const int left = lim - 128 * g - 64 * wg;
      if (__any_sync(0xffffffffu, left < 64)) {
        // a masked pair: p = 0, and dP, where v may be no number, likewise
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c >= left) {
            p[c] = 0.0f;
            x[c] = 0u;
          }
      }
      uint32_t pk[32];
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        const uint64_t ds = mul_f32x2(
            f32x2(p[c], p[c + 1]),
            add_f32x2(f32x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), d2));
        sum2 = add_f32x2(sum2, ds);
        sump = add_f32x2(sump, f32x2(p[c], p[c + 1]));
        float y0, y1;
        split_f32x2(ds, y0, y1);
        pk[c / 2] = pack_bf16x2(y0, y1);
        x[c] = __float_as_uint(y0);
        x[c + 1] = __float_as_uint(y1);
      }
      if (all_steps == 1) {
        // the row is here as a whole
        if (!find_rest()) {
          ok = false;
          break;
        }
#pragma unroll
        for (int c = 0; c < 64; c += 2)
          pk[c / 2] = pack_bf16x2(fmaf(-p[c], rest, __uint_as_float(x[c])),
                                  fmaf(-p[c + 1], rest, __uint_as_float(x[c + 1])));
      }
      tmem_st_32x32b_x32(t, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->ds_full[g & 1]);
    }
    // D for the dkv kernel.  (Rows whose keys are cut into ranges keep the D that they have.)
    const bool whole = steps > 0 && steps == all_steps;
    if (whole && all_steps > 1 && ok) ok = find_rest();
    if (whole && ok && wg == 0 && in) st[128 + r] = nD - rest;
    float* part = a.part + (long long)blockIdx.x * kPartFloats;
    if (steps > 0 && ok) ok = wait_warp(&ctl->acc_full, 0, w, 0x42);
    if (ok && there) {
      tc_fence_after();
      const int rows = a.seq.packed ? s.nq : a.seq.Sq;  // tokens that are written
      uint16_t* base =
          a.d0 + s.z * a.d0_b + (long long)(s.q0 + tok0) * a.d0_t + head0 * a.d0_h + 64 * wg;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t x[32];
        if (steps > 0) {
          tmem_ld_32x32b_x32(tmem + lanes + kColDQ + 64 * wg + 32 * c, x);
          tmem_wait_ld();
        }
        if (a.splits == 1) {
          // (the K stages are free by now)
          store_columns(smem + kOffK + warp * 2048, x, a.scale, steps > 0 && tok < s.nq,
                        [&](int i) {
                          const int rr = (warp & 3) * 32 + i, t = rr & (T - 1);
                          return tok0 + t < rows ? base + (rr >> (7 - a.pack)) * a.d0_h +
                                                       t * a.d0_t + 32 * c
                                                 : nullptr;
                        });
        } else if (steps > 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            reinterpret_cast<uint4*>(part + r * 128 + 64 * wg + 32 * c)[e] =
                make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        }
      }
    }
  } else {
    regs_decrease<kOtherRegs>();
    if (warp == 8) {
      if (lane == 0 && steps > 0) {
        mbar_arrive_expect_tx(&ctl->q_full, 2 * kTile);
        load_tile(smem + kOffQ, &tq, &ctl->q_full, s.q0 + tok0, head0, s.z);
        load_tile(smem + kOffG, &tg, &ctl->q_full, s.q0 + tok0, head0, s.z);
        int g = 0;
        for (; g < steps; ++g) {
          const int ks = g % kKStages, vs = g % kVStages;
          if (g >= kKStages && !wait(&ctl->k_empty[ks], (g / kKStages + 1) & 1, w, 0x43)) break;
          mbar_arrive_expect_tx(&ctl->k_full[ks], kTile);
          load_tile(smem + kOffK + ks * kTile, &tk, &ctl->k_full[ks], k_first + 128 * g, hk, s.z);
          if (g >= kVStages && !wait(&ctl->v_empty[vs], (g / kVStages + 1) & 1, w, 0x44)) {
            wait(&ctl->k_full[ks], (g / kKStages) & 1, w, 0x45, true);  // this one has no pair
            break;
          }
          mbar_arrive_expect_tx(&ctl->v_full[vs], kTile);
          load_tile(smem + kOffV + vs * kTile, &tv, &ctl->v_full[vs], k_first + 128 * g, hk, s.z);
        }
        wait(&ctl->q_full, 0, w, 0x46, true);
        for (int i = 0; i < kKStages; ++i) {
          const int fills = g > i ? (g - i + kKStages - 1) / kKStages : 0;
          if (fills) wait(&ctl->k_full[i], (fills - 1) & 1, w, 0x47, true);
        }
        for (int i = 0; i < kVStages; ++i) {
          const int fills = g > i ? (g - i + kVStages - 1) / kVStages : 0;
          if (fills) wait(&ctl->v_full[i], (fills - 1) & 1, w, 0x48, true);
        }
      }
      __syncwarp();
    } else if (warp == 9) {
      // S_g, dP_g
      if (steps > 0) {
        constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
        const uint32_t sa = smem_addr(smem);
        const uint32_t qd = desc_low(sa + kOffQ, 16), gd = desc_low(sa + kOffG, 16),
                       kd = desc_low(sa + kOffK, 16), vd = desc_low(sa + kOffV, 16);
        bool ok = a.stall ? wait_warp(&ctl->never, 0, w, 0x5f)
                          : wait_warp(&ctl->q_full, 0, w, 0x4c);
        for (int g = 0; g < steps && ok; ++g) {
          const uint32_t ks = (uint32_t)(g % kKStages), vs = (uint32_t)(g % kVStages);
          ok = wait_warp(&ctl->k_ready[ks], (g / kKStages) & 1, w, 0x49) &&
               (g == 0 || wait_warp(&ctl->s_empty, (g - 1) & 1, w, 0x4a));
          if (!ok) break;
          tc_fence_after();
          warp_mma8_ss(tmem + kColS, qd, kd + ks * (kTile >> 4), kIdescS, kTile / 2);
          warp_mma_commit(&ctl->s_full);
          // the buffer's dS (of step g - 2) has been read
          ok = wait_warp(&ctl->v_full[vs], (g / kVStages) & 1, w, 0x4b) &&
               (g < 2 || wait_warp(&ctl->ds_empty[g & 1], ((g - 2) >> 1) & 1, w, 0x51));
          if (!ok) break;
          tc_fence_after();
          warp_mma8_ss(tmem + kColDP + 128 * (g & 1), gd, vd + vs * (kTile >> 4), kIdescS, kTile / 2);
          warp_mma_commit(&ctl->dp_full[g & 1]);
          warp_mma_commit(&ctl->v_empty[vs]);
        }
        warp_mma_commit(&ctl->drain[0]);
        wait(&ctl->drain[0], 0, w, 0x4e, true);
      }
      __syncwarp();
    } else if (warp == 10) {
      // dQ += dS_g K
      if (steps > 0) {
        constexpr uint32_t kIdescG = idesc_bf16_f32(128, 128, false, true);
        const uint32_t kd = desc_low(smem_addr(smem) + kOffK, kTile / 2);
        for (int g = 0; g < steps; ++g) {
          const uint32_t ks = (uint32_t)(g % kKStages);
          if (!wait_warp(&ctl->ds_full[g & 1], (g >> 1) & 1, w, 0x4d)) break;
          tc_fence_after();
          const uint32_t t = tmem + kColDP + 128 * (g & 1);
          warp_mma4_ts(tmem + kColDQ, t, kd + ks * (kTile >> 4), kIdescG, g > 0 ? 1u : 0u);
          warp_mma4_ts(tmem + kColDQ, t + 64, kd + ks * (kTile >> 4) + 512, kIdescG, 1u);
          warp_mma_commit(&ctl->ds_empty[g & 1]);
          warp_mma_commit(&ctl->k_empty[ks]);
          if (g + 1 == steps) warp_mma_commit(&ctl->acc_full);
        }
        warp_mma_commit(&ctl->drain[1]);
        wait(&ctl->drain[1], 0, w, 0x4e, true);
      }
      __syncwarp();
    } else if (warp == 11) {
      for (int g = 0; g < steps; ++g) {
        const int ks = g % kKStages;
        if (!wait_warp(&ctl->k_full[ks], (g / kKStages) & 1, w, 0x4f)) break;
        if (nk - 128 * g < 128) zero_rows(smem + kOffK + ks * kTile, nk - 128 * g);
        if (lane == 0) mbar_arrive(&ctl->k_ready[ks]);
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, kTmemCols);
}

// Adds up the ranges of a tile's key tiles, in their order: a warp a row.
__global__ void __launch_bounds__(256) prompt_dq_join_kernel(const Args a) {
  after_predecessor();
  const unsigned item = blockIdx.x >> 4;
  const int r = (int)((blockIdx.x & 15) * 8 + (threadIdx.x >> 5)), lane = (int)lane_id();
  const int T = 128 >> a.pack;
  const int rank = (int)(item / (unsigned)a.n_packs),
            hp = (int)(item - (unsigned)rank * (unsigned)a.n_packs);
  const Place place = find_tile(a.seq, rank, 7 - a.pack, false);
  const Seq& s = place.s;
  const int tok0 = place.tile * T, tok = tok0 + (r & (T - 1)), head = (hp << a.pack) + (r >> (7 - a.pack));
  if (!place.there || tok >= (a.seq.packed ? s.nq : a.seq.Sq)) return;
  int keys = tok0 < s.nq ? s.nk : 0;
  if (a.seq.causal) keys = clampi((tok0 + T < s.nq ? tok0 + T : s.nq) + s.nk - s.nq, 0, keys);
  const int steps = (keys + 127) / 128;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < a.splits && tok < s.nq; ++i) {
    if ((long long)steps * (i + 1) / a.splits == (long long)steps * i / a.splits) continue;
    const float* part = a.part + ((long long)item * a.splits + i) * kPartFloats;
    const float4 x = reinterpret_cast<const float4*>(part + r * 128)[lane];
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
  }
  reinterpret_cast<uint2*>(a.d0 + s.z * a.d0_b + head * a.d0_h +
                           (long long)(s.q0 + tok) * a.d0_t)[lane] =
      make_uint2(pack_bf16x2(acc.x * a.scale, acc.y * a.scale),
                 pack_bf16x2(acc.z * a.scale, acc.w * a.scale));
}

}  // namespace dq
}  // namespace bwd
}  // namespace prompt
}  // namespace vsa

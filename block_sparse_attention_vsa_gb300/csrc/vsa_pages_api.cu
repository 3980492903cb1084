// vsa_pages_api.cu -- the C ABI of the 8-bit cache's pages (declared in include/vsa.h):
// host-side argument checks and launches.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/vsa.h"
#include "vsa_host.h"
#include "vsa_launch.h"
#include "vsa_pages_kernel.cuh"

using namespace vsa;

namespace {

constexpr int kSms = 152;  // of a GB300, which host_device() asks for

bool block_ok(int block) { return block == 64 || block == 128; }

// CTAs that divide the rows of a table among them, one cluster: one CTA where its barriers would
// take longer than the rows (us of one CTA and of eight: room for a token in 512 rows 6.2 and 7.6,
// 2,048 rows 11.5 and 7.8; forks of 512 rows 8.0 and 9.8, 2,048 rows 15.8 and 14.6) or, of long
// prompts, their entries.  How many of those are asked for only the device knows: a token in each of
// 512 rows of 129 blocks takes 5.9 and 7.6, 8,000 tokens 49 and 13; the former come far more often.
int pages_ctas(long long rows, long long entries) {
  return rows <= 1024 && entries <= (1 << 17) ? 1 : kPagesCluster;
}

size_t words(int pages) { return ((size_t)pages + 31) / 32; }

// The cache's buffers as ranges.
struct CacheRanges {
  Range r[5];
  CacheRanges(const uint8_t* k, const uint8_t* v, const float* ks, const float* vs,
              const vsa_bf16* km, int pages, int block)
      : r{{k, (size_t)pages * block * VSA_HEAD_DIM},
          {v, (size_t)pages * block * VSA_HEAD_DIM},
          {ks, (size_t)pages * 4},
          {vs, (size_t)pages * 4},
          {km, (size_t)pages * VSA_HEAD_DIM * 2}} {}
};
vsa_status cache_ok(const void* k, const void* v, const void* ks, const void* vs, const void* km) {
  if (!k || !v || !ks || !vs) return VSA_ERR_INVALID_ARG;
  if (!host_aligned16(k) || !host_aligned16(v) || !host_aligned4(ks) || !host_aligned4(vs) ||
      !host_aligned16(km))
    return VSA_ERR_INVALID_ARG;
  return VSA_OK;
}

}  // namespace

extern "C" {

vsa_status vsa_pages_free(int32_t* table, const int32_t* lens, int B, int Hkv, int max_blocks,
                          int block, int pages, int32_t* refs, uint32_t* free_bits,
                          vsa_stream_t stream) {
  host_set_launches(0);
  if (B < 0 || Hkv < 0 || max_blocks < 0 || pages < 0) return VSA_ERR_INVALID_ARG;
  if (!block_ok(block)) return VSA_ERR_UNSUPPORTED;
  if ((long long)B * Hkv > INT_MAX) return VSA_ERR_UNSUPPORTED;
  const long long entries = (long long)B * Hkv * max_blocks;
  if (entries > INT_MAX) return VSA_ERR_UNSUPPORTED;
  if (entries == 0) return VSA_OK;
  if (!table || !host_aligned4(table) || !host_aligned4(lens)) return VSA_ERR_INVALID_ARG;
  if (pages > 0 && (!refs || !free_bits || !host_aligned4(refs) || !host_aligned4(free_bits)))
    return VSA_ERR_INVALID_ARG;
  const Range out[] = {{table, (size_t)entries * 4}, {refs, (size_t)pages * 4},
                       {free_bits, words(pages) * 4}};
  const Range in[] = {{lens, lens ? (size_t)B * 4 : 0}};
  if (!outputs_clear(out, in)) return VSA_ERR_INVALID_ARG;
  int dev = 0;
  const vsa_status st = host_device(&dev);
  if (st != VSA_OK) return st;
  const FreeArgs a{{refs, free_bits, pages}, table, lens, (unsigned)entries, Hkv, max_blocks,
                   block};
  const long long ctas = (entries + 255) / 256;
  return launch(pages_free_kernel, dim3((unsigned)(ctas < 8 * kSms ? ctas : 8 * kSms)), 256, 0,
                reinterpret_cast<cudaStream_t>(stream), 0, a);
}

vsa_status vsa_pages_reserve(int32_t* table, const int32_t* lens, const int32_t* n_new, int B,
                             int Hkv, int max_blocks, int block, int pages, int32_t* refs,
                             uint32_t* free_bits, int32_t* lacking, vsa_stream_t stream) {
  host_set_launches(0);
  if (B < 0 || Hkv < 0 || max_blocks < 0 || pages < 0) return VSA_ERR_INVALID_ARG;
  if (!block_ok(block)) return VSA_ERR_UNSUPPORTED;
  if ((long long)B * Hkv > INT_MAX) return VSA_ERR_UNSUPPORTED;
  const long long entries = (long long)B * Hkv * max_blocks;
  if (entries > INT_MAX) return VSA_ERR_UNSUPPORTED;
  if (B == 0) return VSA_OK;
  if (!lens || !lacking || !host_aligned4(lens) || !host_aligned4(n_new) ||
      !host_aligned4(lacking))
    return VSA_ERR_INVALID_ARG;
  if (entries > 0 && (!table || !host_aligned4(table))) return VSA_ERR_INVALID_ARG;
  if (pages > 0 && (!refs || !free_bits || !host_aligned4(refs) || !host_aligned4(free_bits)))
    return VSA_ERR_INVALID_ARG;
  const Range out[] = {{table, (size_t)entries * 4}, {refs, (size_t)pages * 4},
                       {free_bits, words(pages) * 4}, {lacking, (size_t)B * 4}};
  const Range in[] = {{lens, (size_t)B * 4}, {n_new, n_new ? (size_t)B * 4 : 0}};
  if (!outputs_clear(out, in)) return VSA_ERR_INVALID_ARG;
  int dev = 0;
  const vsa_status st = host_device(&dev);
  if (st != VSA_OK) return st;
  const ReserveArgs a{{refs, free_bits, pages}, table, lens, n_new, lacking, B, Hkv, max_blocks,
                      block};
  const int ctas = pages_ctas((long long)B * Hkv, entries);
  return launch(pages_reserve_kernel, dim3(ctas), kPagesThreads, 0,
                reinterpret_cast<cudaStream_t>(stream), ctas, a);
}

vsa_status vsa_cache_fork(const int32_t* table, const int32_t* lens, const int32_t* parent, int B,
                          int N, int Hkv, int D, int max_blocks, int block, int pages,
                          uint8_t* k_cache, uint8_t* v_cache, float* k_scale, float* v_scale,
                          vsa_bf16* k_mean, int32_t* refs, uint32_t* free_bits,
                          int32_t* table_out, int32_t* lens_out, int32_t* lacking,
                          vsa_stream_t stream) {
  host_set_launches(0);
  if (B < 0 || N < 0 || Hkv < 0 || max_blocks < 0 || pages < 0) return VSA_ERR_INVALID_ARG;
  if (D != VSA_HEAD_DIM || !block_ok(block)) return VSA_ERR_UNSUPPORTED;
  const long long rows = (long long)N * Hkv;
  if (rows > INT_MAX || (long long)B * Hkv > INT_MAX) return VSA_ERR_UNSUPPORTED;
  const long long entries = rows * max_blocks, held = (long long)B * Hkv * max_blocks;
  if (entries > INT_MAX || held > INT_MAX || (long long)max_blocks * block > INT_MAX)
    return VSA_ERR_UNSUPPORTED;
  if (N == 0) return VSA_OK;
  if (!parent || !lens_out || !lacking || !host_aligned4(parent) || !host_aligned4(lens_out) ||
      !host_aligned4(lacking) || !host_aligned4(lens))
    return VSA_ERR_INVALID_ARG;
  if (B > 0 && !lens) return VSA_ERR_INVALID_ARG;
  if (entries > 0 && (!table_out || !host_aligned4(table_out) || (held > 0 && !table) ||
                      !host_aligned4(table)))
    return VSA_ERR_INVALID_ARG;
  if (pages > 0) {
    if (!refs || !free_bits || !host_aligned4(refs) || !host_aligned4(free_bits))
      return VSA_ERR_INVALID_ARG;
    const vsa_status st = cache_ok(k_cache, v_cache, k_scale, v_scale, k_mean);
    if (st != VSA_OK) return st;
  }
  const CacheRanges c(k_cache, v_cache, k_scale, v_scale, k_mean, pages, block);
  const Range out[] = {{table_out, (size_t)entries * 4}, {lens_out, (size_t)N * 4},
                       {lacking, (size_t)N * 4}, {refs, (size_t)pages * 4},
                       {free_bits, words(pages) * 4}, c.r[0], c.r[1], c.r[2], c.r[3], c.r[4]};
  const Range in[] = {{table, (size_t)held * 4}, {lens, (size_t)B * 4}, {parent, (size_t)N * 4}};
  if (!outputs_clear(out, in)) return VSA_ERR_INVALID_ARG;
  int dev = 0;
  vsa_status st = host_device(&dev);
  if (st != VSA_OK) return st;
  const ForkArgs a{{refs, free_bits, pages}, {k_cache, v_cache, k_scale, v_scale, k_mean},
                   table, lens, parent, table_out, lens_out, lacking, B, N, Hkv,
                   max_blocks, block};
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int ctas = pages_ctas(rows, 0);
  st = launch(pages_fork_kernel, dim3(ctas), kPagesThreads, 0, s, ctas, a);
  if (st != VSA_OK || entries == 0) return st;
  st = launch(cache_fork_kernel, dim3((unsigned)rows), 256, 0, s, 0, a);
  if (st == VSA_OK) host_set_launches(2);
  return st;
}

vsa_status vsa_cache_compact(int32_t* table, int B, int Hkv, int D, int max_blocks, int block,
                             int pages, uint8_t* k_cache, uint8_t* v_cache, float* k_scale,
                             float* v_scale, vsa_bf16* k_mean, int32_t* refs,
                             uint32_t* free_bits, int32_t* to, int32_t* n_used,
                             vsa_stream_t stream) {
  host_set_launches(0);
  if (B < 0 || Hkv < 0 || max_blocks < 0 || pages < 0) return VSA_ERR_INVALID_ARG;
  if (D != VSA_HEAD_DIM || !block_ok(block)) return VSA_ERR_UNSUPPORTED;
  if ((long long)B * Hkv > INT_MAX) return VSA_ERR_UNSUPPORTED;
  const long long entries = (long long)B * Hkv * max_blocks;
  if (entries > INT_MAX) return VSA_ERR_UNSUPPORTED;
  if (!n_used || !host_aligned4(n_used)) return VSA_ERR_INVALID_ARG;
  if (entries > 0 && (!table || !host_aligned4(table))) return VSA_ERR_INVALID_ARG;
  if (pages > 0) {
    if (!refs || !free_bits || !to || !host_aligned4(refs) || !host_aligned4(free_bits) ||
        !host_aligned4(to))
      return VSA_ERR_INVALID_ARG;
    const vsa_status st = cache_ok(k_cache, v_cache, k_scale, v_scale, k_mean);
    if (st != VSA_OK) return st;
  }
  const CacheRanges c(k_cache, v_cache, k_scale, v_scale, k_mean, pages, block);
  const Range out[] = {{table, (size_t)entries * 4}, {to, (size_t)pages * 4}, {n_used, 4},
                       {refs, (size_t)pages * 4}, {free_bits, words(pages) * 4},
                       c.r[0], c.r[1], c.r[2], c.r[3], c.r[4]};
  const Range in[] = {{nullptr, 0}};
  if (!outputs_clear(out, in)) return VSA_ERR_INVALID_ARG;
  int dev = 0;
  vsa_status st = host_device(&dev);
  if (st != VSA_OK) return st;
  const CompactArgs a{{refs, free_bits, pages}, {k_cache, v_cache, k_scale, v_scale, k_mean},
                      table, to, n_used, entries, block};
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // a CTA a thousand pages, one wave at most
  const int ctas = pages < kSms * kPagesThreads ? (pages + kPagesThreads - 1) / kPagesThreads : kSms;
  st = launch(pages_compact_kernel, dim3(ctas < 1 ? 1 : ctas), kPagesThreads, 0, s, 0, a);
  if (st != VSA_OK || (pages == 0 && entries == 0)) return st;
  long long most = (entries + 255) / 256;
  if (pages > most) most = pages;
  st = launch(cache_compact_kernel, dim3((unsigned)(most < 8 * kSms ? most : 8 * kSms)), 256, 0, s,
              0, a);
  if (st == VSA_OK) host_set_launches(2);
  return st;
}

}  // extern "C"

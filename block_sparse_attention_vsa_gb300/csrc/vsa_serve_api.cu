// vsa_serve_api.cu -- the C ABI of the operators around the attention (declared in
// include/vsa.h): block means, the choice of key blocks, the 8-bit key/value cache and
// eviction from it.  Host-side argument checks and launches.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/vsa.h"
#include "vsa_cache_kernel.cuh"
#include "vsa_host.h"
#include "vsa_select_kernel.cuh"

using namespace vsa;

namespace {

// Byte ranges of a call's buffers: an output may overlap nothing else.
struct Range {
  const void* p;
  size_t n;
};
bool meets(const Range& x, const Range& y) {
  if (!x.p || !y.p || !x.n || !y.n) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return a < b + y.n && b < a + x.n;
}
template <int NO, int NI>
bool outputs_clear(const Range (&out)[NO], const Range (&in)[NI]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (meets(out[o], in[i])) return false;
    for (int p = o + 1; p < NO; ++p)
      if (meets(out[o], out[p])) return false;
  }
  return true;
}

constexpr int kSms = 152;  // of a GB300, which host_device() asks for

std::mutex g_attr_mu;
enum AttrSlot { kAttrSelect, kAttrFwd = kAttrSelect + 8, kAttrSlots = kAttrFwd + 4 };
bool g_attr[64][kAttrSlots];

// The dynamic shared-memory limit of a kernel, raised once per device.
template <typename Kern>
vsa_status smem_limit(Kern kern, size_t bytes, int dev, int slot) {
  std::lock_guard<std::mutex> lk(g_attr_mu);
  if (!g_attr[dev][slot]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) !=
        cudaSuccess)
      return VSA_ERR_CUDA;
    g_attr[dev][slot] = true;
  }
  return VSA_OK;
}

// One launch; the kernel may start up while its predecessor in the stream ends (each begins
// with after_predecessor()).  `cluster` CTAs form a cluster.
template <typename... P, typename... A>
vsa_status launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                  int cluster, A... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, P(args)...) != cudaSuccess) {
    cudaGetLastError();
    return VSA_ERR_CUDA;
  }
  host_set_launches(1);
  return VSA_OK;
}

bool heads_ok(int Hq, int Hkv) { return Hkv >= 1 && Hq % Hkv == 0; }

template <int NREG, int ROWS>
vsa_status launch_select_rows(SelectArgs& a, long long heads, int dev, int slot, cudaStream_t s) {
  a.tiles = (a.nq + ROWS - 1) / ROWS;
  const vsa_status st =
      smem_limit(select_kernel<NREG, ROWS>, select_smem(NREG, ROWS), dev, slot);
  if (st != VSA_OK) return st;
  return launch(select_kernel<NREG, ROWS>, dim3((unsigned)(heads * a.tiles)), kSelRowThreads,
                select_smem(NREG, ROWS), s, 0, a);
}
// 32 rows a CTA, or 16 where the CTAs of 32 would hardly fill the SMs once: 256 x 256 blocks
// of 12 / 20 / 32 heads took 14.6 / 19.8 / 20.7 us with 32 rows, 13.1 / 17.8 / 23.4 with 16.
template <int NREG>
vsa_status launch_select(SelectArgs& a, long long heads, int dev, int slot, cudaStream_t s) {
  if (heads * ((a.nq + 31) / 32) > kSms + kSms / 8)
    return launch_select_rows<NREG, 32>(a, heads, dev, slot, s);
  return launch_select_rows<NREG, 16>(a, heads, dev, slot + 1, s);
}

template <int BLOCK, bool WEIGHT>
vsa_status launch_cache_fwd(const CacheFwdArgs& a, int dev, cudaStream_t s) {
  auto kern = cache_fwd_kernel<BLOCK, WEIGHT>;
  const vsa_status st =
      smem_limit(kern, kCacheSmem, dev, kAttrFwd + (BLOCK == 128 ? 1 : 0) + (WEIGHT ? 2 : 0));
  if (st != VSA_OK) return st;
  // one wave, two units a CTA at least; a multiple of the rows where there are fewer of
  // them, so that rows of one length end where pieces do: 24 / 12 rows of 128 blocks take
  // 18.4 / 14.5 us, 24.1 / 20.3 on all CTAs; 24 of 256 25.0 and 27.4; long rows are even
  // (12 of 1,536 56.4 and 56.9, 24 of them 100.5 and 99.0)
  const int n_max = a.idx != nullptr && a.max_sel < a.max_blocks ? a.max_sel : a.max_blocks;
  const long long most = (long long)a.rows * n_max / 2;
  int grid = most < 1 ? 1 : (most < kCacheGrid ? (int)most : kCacheGrid);
  if (a.rows <= grid / 8) grid -= grid % a.rows;
  return launch(kern, dim3(grid), kCacheWarps * 32, kCacheSmem, s, 0, a);
}

// Workspace: counters (at one place whatever the shape, so that a workspace may serve calls
// of several shapes in turn), partial results, log-sum-exps and block weights.
constexpr long long kCacheCounters = 65536;
struct CacheLayout {
  size_t part, lse, mass, total;
  int chunks, pieces;
};
CacheLayout cache_layout(long long B, long long Hq, long long Hkv, long long max_blocks,
                         bool weight) {
  auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  CacheLayout l;
  l.chunks = (int)((Hq / Hkv + 7) / 8);
  l.part = (size_t)kCacheCounters * sizeof(unsigned int);
  // pieces of the unit sequence: one a CTA, two blocks or more each
  const long long most = B * Hkv * l.chunks * (max_blocks > 0 ? max_blocks : 1);
  l.pieces = (int)(most < kCacheGrid ? most : kCacheGrid);
  l.lse = l.part + up((size_t)(2 * l.pieces + l.pieces / 8 + 2) * kCachePartFloats * sizeof(float));
  l.mass = l.lse + (weight ? up((size_t)(B * Hq) * sizeof(float)) : 0);
  l.total = l.mass +
            (weight ? (size_t)(B * Hkv * max_blocks * l.chunks) * 8 * sizeof(float2) : 0);
  return l;
}

// Shape checks shared by the cache entry points.
vsa_status check_cache(int B, int Hkv, int D, int pages, int max_blocks, int block) {
  if (B < 0 || Hkv < 0 || pages < 0 || max_blocks < 0) return VSA_ERR_INVALID_ARG;
  if (D != VSA_HEAD_DIM || (block != 64 && block != 128)) return VSA_ERR_UNSUPPORTED;
  if (max_blocks > VSA_MAX_BLOCKS || (long long)B * Hkv > INT_MAX / 8) return VSA_ERR_UNSUPPORTED;
  return VSA_OK;
}

}  // namespace

extern "C" {

vsa_status vsa_block_mean(const vsa_bf16* x, const int32_t* sizes, int B, int H, int S, int D,
                          int block, vsa_bf16* mean, vsa_stream_t stream) {
  host_set_launches(0);
  if (B < 0 || H < 0 || S < 0) return VSA_ERR_INVALID_ARG;
  if (D != VSA_HEAD_DIM || (block != 64 && block != 128)) return VSA_ERR_UNSUPPORTED;
  if ((long long)B * H > INT_MAX) return VSA_ERR_UNSUPPORTED;
  const long long nb = ((long long)S + block - 1) / block, ctas = (long long)B * H * nb;
  if (ctas > INT_MAX) return VSA_ERR_UNSUPPORTED;
  if (ctas == 0) return VSA_OK;
  if (!x || !mean || !host_aligned16(x) || !host_aligned4(mean) || !host_aligned4(sizes))
    return VSA_ERR_INVALID_ARG;
  const Range out[1] = {{mean, (size_t)ctas * 256}};
  const Range in[2] = {{x, (size_t)B * H * S * 256}, {sizes, (size_t)nb * 4}};
  if (!outputs_clear(out, in)) return VSA_ERR_INVALID_ARG;
  int dev;
  const vsa_status st = host_device(&dev);
  if (st != VSA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launch(block == 64 ? block_mean_kernel<64> : block_mean_kernel<128>,
                dim3((unsigned)ctas), block * 2, 0, s, 0, x, sizes, S, (int)nb, mean);
}

vsa_status vsa_select_blocks(const vsa_bf16* q_mean, const vsa_bf16* k_mean, const int32_t* sizes,
                             int B, int Hq, int Hkv, int nq, int nk, int D, int topk, int causal,
                             int n_first, int n_near, int32_t* q2k_idx, int32_t* q2k_num,
                             vsa_stream_t stream) {
  host_set_launches(0);
  if (B < 0 || Hq < 0 || Hkv < 0 || nq < 0 || nk < 0 || topk < 1 || n_first < 0 || n_near < 0)
    return VSA_ERR_INVALID_ARG;
  if (D != VSA_HEAD_DIM || nk > VSA_MAX_BLOCKS) return VSA_ERR_UNSUPPORTED;
  if (nq > (1 << 24) || topk > (1 << 24) || (long long)B * Hq > INT_MAX)
    return VSA_ERR_UNSUPPORTED;
  const long long heads = (long long)B * Hq, rows = heads * nq;
  if (heads * (((long long)nq + 15) / 16) > INT_MAX) return VSA_ERR_UNSUPPORTED;
  if (rows == 0) return VSA_OK;
  if (!heads_ok(Hq, Hkv)) return VSA_ERR_INVALID_ARG;
  if (!q_mean || (nk > 0 && !k_mean) || !q2k_idx || !q2k_num || !host_aligned16(q_mean) ||
      !host_aligned16(k_mean) || !host_aligned4(sizes) || !host_aligned4(q2k_idx) ||
      !host_aligned4(q2k_num))
    return VSA_ERR_INVALID_ARG;
  const Range out[2] = {{q2k_idx, (size_t)rows * topk * 4}, {q2k_num, (size_t)rows * 4}};
  const Range in[3] = {{q_mean, (size_t)rows * 256},
                       {k_mean, (size_t)B * Hkv * nk * 256},
                       {sizes, (size_t)nk * 4}};
  if (!outputs_clear(out, in)) return VSA_ERR_INVALID_ARG;
  int dev;
  const vsa_status st = host_device(&dev);
  if (st != VSA_OK) return st;
  SelectArgs a{};
  a.q = q_mean;
  a.k = k_mean;
  a.sizes = sizes;
  a.idx = q2k_idx;
  a.num = q2k_num;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.nq = nq;
  a.nk = nk;
  a.topk = topk;
  a.causal = causal != 0;
  // no more than there are blocks on either side: e - n_near and the like stay in range
  a.n_first = n_first < nk ? n_first : nk;
  a.n_near = n_near < nk + nq ? n_near : nk + nq;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (nk <= 512) return launch_select<8>(a, heads, dev, kAttrSelect, s);
  if (nk <= 1024) return launch_select<16>(a, heads, dev, kAttrSelect + 2, s);
  if (nk <= 1536) return launch_select<24>(a, heads, dev, kAttrSelect + 4, s);
  return launch_select<32>(a, heads, dev, kAttrSelect + 6, s);
}

vsa_status vsa_cache_select(const vsa_bf16* q, const vsa_bf16* k_mean, const int32_t* table,
                            const int32_t* lens, int B, int Hq, int Hkv, int D, int pages,
                            int max_blocks, int block, int topk, int n_first, int n_near,
                            int32_t* idx, int32_t* num, vsa_stream_t stream) {
  host_set_launches(0);
  if (Hq < 0 || topk < 1 || n_first < 0 || n_near < 0) return VSA_ERR_INVALID_ARG;
  vsa_status st = check_cache(B, Hkv, D, pages, max_blocks, block);
  if (st != VSA_OK) return st;
  if (topk > (1 << 24)) return VSA_ERR_UNSUPPORTED;
  const long long rows = (long long)B * Hkv;
  if (rows == 0) return VSA_OK;
  if (Hq < 1 || !heads_ok(Hq, Hkv)) return VSA_ERR_INVALID_ARG;
  if (!q || (pages > 0 && !k_mean) || (max_blocks > 0 && !table) || !lens || !idx || !num ||
      !host_aligned16(q) || !host_aligned16(k_mean) || !host_aligned4(table) ||
      !host_aligned4(lens) || !host_aligned4(idx) || !host_aligned4(num))
    return VSA_ERR_INVALID_ARG;
  const Range out[2] = {{idx, (size_t)rows * topk * 4}, {num, (size_t)rows * 4}};
  const Range in[4] = {{q, (size_t)B * Hq * 256},
                       {k_mean, (size_t)pages * 256},
                       {table, (size_t)rows * max_blocks * 4},
                       {lens, (size_t)B * 4}};
  if (!outputs_clear(out, in)) return VSA_ERR_INVALID_ARG;
  int dev;
  st = host_device(&dev);
  if (st != VSA_OK) return st;
  CacheSelectArgs a{};
  a.q = q;
  a.k_mean = k_mean;
  a.table = table;
  a.lens = lens;
  a.idx = idx;
  a.num = num;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.pages = pages;
  a.max_blocks = max_blocks;
  a.block = block;
  a.topk = topk;
  a.n_first = n_first < max_blocks ? n_first : max_blocks;
  a.n_near = n_near < max_blocks ? n_near : max_blocks;
  // CTAs that share a row's blocks: 1 up to 256 blocks (128 rows of 128 blocks: 9.0 us with
  // one, 11.1 with four), else 4 (32 rows of 1,536: 17.2 with one, 11.4 with four, 12.1 with
  // eight), or 8 for few rows (8 rows of 1,536: 10.4 with four, 9.9 with eight)
  const int ctas = max_blocks <= 256 ? 1 : (rows * 8 <= kSms ? 8 : 4);
  if (rows * ctas > INT_MAX) return VSA_ERR_UNSUPPORTED;
  return launch(cache_select_kernel, dim3((unsigned)(rows * ctas)), kSelThreads, 0,
                reinterpret_cast<cudaStream_t>(stream), ctas, a);
}

vsa_status vsa_cache_write(const vsa_bf16* k, const vsa_bf16* v, const int32_t* table,
                           const int32_t* lens, const int32_t* n_new, int B, int Hkv, int T, int D,
                           int pages, int max_blocks, int block, uint8_t* k_cache,
                           uint8_t* v_cache, float* k_scale, float* v_scale, vsa_bf16* k_mean,
                           vsa_stream_t stream) {
  host_set_launches(0);
  if (T < 0) return VSA_ERR_INVALID_ARG;
  vsa_status st = check_cache(B, Hkv, D, pages, max_blocks, block);
  if (st != VSA_OK) return st;
  // blocks that T tokens can touch, wherever the first one falls
  const long long slots = ((long long)T + 2 * block - 2) / block;
  const long long ctas = (long long)B * Hkv * slots;
  if (ctas > INT_MAX) return VSA_ERR_UNSUPPORTED;
  if (ctas == 0 || T == 0 || pages == 0 || max_blocks == 0) return VSA_OK;
  if (!k || !v || !table || !lens || !k_cache || !v_cache || !k_scale || !v_scale)
    return VSA_ERR_INVALID_ARG;
  if (!host_aligned16(k) || !host_aligned16(v) || !host_aligned16(k_cache) ||
      !host_aligned16(v_cache) || !host_aligned4(k_scale) || !host_aligned4(v_scale) ||
      !host_aligned4(k_mean) || !host_aligned4(table) || !host_aligned4(lens) ||
      !host_aligned4(n_new))
    return VSA_ERR_INVALID_ARG;
  const size_t codes = (size_t)pages * block * 128, rows = (size_t)B * Hkv;
  const Range out[5] = {{k_cache, codes},
                        {v_cache, codes},
                        {k_scale, (size_t)pages * 4},
                        {v_scale, (size_t)pages * 4},
                        {k_mean, (size_t)pages * 256}};
  const Range in[5] = {{k, rows * T * 256},
                       {v, rows * T * 256},
                       {table, rows * max_blocks * 4},
                       {lens, (size_t)B * 4},
                       {n_new, (size_t)B * 4}};
  if (!outputs_clear(out, in)) return VSA_ERR_INVALID_ARG;
  int dev;
  st = host_device(&dev);
  if (st != VSA_OK) return st;
  const CacheWriteArgs a{k,       v,       table,   lens,   n_new,      k_cache, v_cache,
                         k_scale, v_scale, k_mean,  Hkv,    T,          (int)slots, pages,
                         max_blocks};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)ctas, 2);
  return launch(block == 64 ? cache_write_kernel<64> : cache_write_kernel<128>, grid, block * 2, 0,
                s, 0, a);
}

size_t vsa_cache_workspace_bytes(int B, int Hq, int Hkv, int max_blocks, int weight) {
  if (check_cache(B, Hkv, VSA_HEAD_DIM, 0, max_blocks, 64) != VSA_OK || Hq < 1 ||
      !heads_ok(Hq, Hkv))
    return 0;
  return cache_layout(B, Hq, Hkv, max_blocks, weight != 0).total;
}

vsa_status vsa_fwd_cache(const vsa_bf16* q, const uint8_t* k_cache, const uint8_t* v_cache,
                         const float* k_scale, const float* v_scale, const int32_t* table,
                         const int32_t* lens, const int32_t* idx, const int32_t* num, int max_sel,
                         int B, int Hq, int Hkv, int D, int pages, int max_blocks, int block,
                         float scale, float keep, vsa_bf16* out, float* lse, float* weight,
                         void* workspace, size_t workspace_bytes, vsa_stream_t stream) {
  host_set_launches(0);
  if (Hq < 0) return VSA_ERR_INVALID_ARG;
  vsa_status st = check_cache(B, Hkv, D, pages, max_blocks, block);
  if (st != VSA_OK) return st;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return VSA_ERR_INVALID_ARG;
  if (weight && !std::isfinite(keep)) return VSA_ERR_INVALID_ARG;
  if (B == 0 || Hq == 0) return VSA_OK;
  if (!heads_ok(Hq, Hkv)) return VSA_ERR_INVALID_ARG;
  if (idx && (!num || max_sel < 1)) return VSA_ERR_INVALID_ARG;
  const bool some = pages > 0 && max_blocks > 0;
  if (!q || !lens || !out || (some && (!k_cache || !v_cache || !k_scale || !v_scale)) ||
      (max_blocks > 0 && !table))
    return VSA_ERR_INVALID_ARG;
  if (!host_aligned16(q) || !host_aligned16(k_cache) || !host_aligned16(v_cache) ||
      !host_aligned16(out) || !host_aligned4(k_scale) || !host_aligned4(v_scale) ||
      !host_aligned4(table) || !host_aligned4(lens) || !host_aligned4(idx) ||
      !host_aligned4(num) || !host_aligned4(lse) || !host_aligned4(weight))
    return VSA_ERR_INVALID_ARG;
  if ((long long)B * Hq > INT_MAX / 128) return VSA_ERR_UNSUPPORTED;
  const CacheLayout l = cache_layout(B, Hq, Hkv, max_blocks, weight != nullptr);
  if ((long long)B * Hkv * (l.chunks + 1) > kCacheCounters) return VSA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < l.total || !host_aligned16(workspace))
    return VSA_ERR_INVALID_ARG;
  const size_t codes = (size_t)pages * block * 128, rows = (size_t)B * Hkv;
  const Range outs[4] = {{out, (size_t)B * Hq * 256},
                         {lse, (size_t)B * Hq * 4},
                         {weight, rows * max_blocks * 4},
                         {workspace, l.total}};
  const Range ins[9] = {{q, (size_t)B * Hq * 256},
                        {k_cache, codes},
                        {v_cache, codes},
                        {k_scale, (size_t)pages * 4},
                        {v_scale, (size_t)pages * 4},
                        {table, rows * max_blocks * 4},
                        {lens, (size_t)B * 4},
                        {idx, idx ? rows * max_sel * 4 : 0},
                        {num, idx ? rows * 4 : 0}};
  if (!outputs_clear(outs, ins)) return VSA_ERR_INVALID_ARG;
  int dev;
  st = host_device(&dev);
  if (st != VSA_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  CacheFwdArgs a{};
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.table = table;
  a.lens = lens;
  a.idx = idx;
  a.num = num;
  a.out = out;
  a.lse = lse;
  a.weight = weight;
  a.counters = reinterpret_cast<unsigned int*>(ws);
  a.part = reinterpret_cast<float*>(ws + l.part);
  a.lse_ws = reinterpret_cast<float*>(ws + l.lse);
  a.mass = reinterpret_cast<float2*>(ws + l.mass);
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.chunks = l.chunks;
  a.rows = (int)((long long)B * Hkv * l.chunks);
  a.pieces = l.pieces;
  a.pages = pages;
  a.max_blocks = max_blocks;
  a.max_sel = max_sel;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.keep = keep;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (weight)
    return block == 64 ? launch_cache_fwd<64, true>(a, dev, s)
                       : launch_cache_fwd<128, true>(a, dev, s);
  return block == 64 ? launch_cache_fwd<64, false>(a, dev, s)
                     : launch_cache_fwd<128, false>(a, dev, s);
}

vsa_status vsa_cache_evict(const float* weight, const int32_t* table, const int32_t* lens, int B,
                           int Hkv, int max_blocks, int block, int budget, int n_first, int n_last,
                           int32_t* table_out, float* weight_out, int32_t* lens_out,
                           int32_t* freed, int32_t* n_freed, vsa_stream_t stream) {
  host_set_launches(0);
  vsa_status st = check_cache(B, Hkv, VSA_HEAD_DIM, 0, max_blocks, block);
  if (st != VSA_OK) return st;
  // the last block may be part full: only whole blocks may go
  if (n_first < 0 || n_last < 1 || budget < 1 || (long long)n_first + n_last > budget)
    return VSA_ERR_INVALID_ARG;
  const size_t rows = (size_t)B * Hkv, cells = rows * max_blocks;
  if (rows == 0) return VSA_OK;
  if (!lens || !lens_out || !n_freed ||
      (cells > 0 && (!weight || !table || !table_out || !weight_out || !freed)))
    return VSA_ERR_INVALID_ARG;
  const void* all[8] = {weight, table, lens, table_out, weight_out, lens_out, freed, n_freed};
  for (const void* p : all)
    if (!host_aligned4(p)) return VSA_ERR_INVALID_ARG;
  const Range out[5] = {{table_out, cells * 4},
                        {weight_out, cells * 4},
                        {lens_out, (size_t)B * 4},
                        {freed, cells * 4},
                        {n_freed, (size_t)B * 4}};
  const Range in[3] = {{weight, cells * 4}, {table, cells * 4}, {lens, (size_t)B * 4}};
  if (!outputs_clear(out, in)) return VSA_ERR_INVALID_ARG;
  int dev;
  st = host_device(&dev);
  if (st != VSA_OK) return st;
  const CacheEvictArgs a{weight,     table,    lens,  table_out, weight_out, lens_out, freed,
                         n_freed,    Hkv,      max_blocks, block, budget,    n_first,  n_last};
  return launch(cache_evict_kernel, dim3((unsigned)rows), kEvictThreads, 0,
                reinterpret_cast<cudaStream_t>(stream), 0, a);
}

}  // extern "C"

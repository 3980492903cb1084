// vsa_prompt_api.cu -- the C ABI of the attention over whole prompts and its gradient
// (declared in include/vsa.h): host-side argument checks, TMA tensor maps and launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <utility>

#include "../../include/vsa.h"
#include "vsa_host.h"
#include "vsa_launch.h"
#include "vsa_prompt_bwd_kernel.cuh"
#include "vsa_prompt_fwd_kernel.cuh"

using namespace vsa;

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// A bf16 tensor [batch, heads, tokens, 128] with strides in elements.
struct View {
  const void* p;
  long long nb, nh, nt;
  long long sb, sh, st;
  bool empty() const { return nb == 0 || nh == 0 || nt == 0; }
  long long last() const {  // elements from the first to behind the last one
    return (nb - 1) * sb + (nh - 1) * sh + (nt - 1) * st + VSA_HEAD_DIM;
  }
};

View view(const void* p, const int64_t* s, long long nb, long long nh, long long nt) {
  View v{p, nb, nh, nt, s[0], s[1], s[2]};
  // the stride of an axis of one is free: any valid one serves
  if (nb == 1) v.sb = VSA_HEAD_DIM;
  if (nh == 1) v.sh = VSA_HEAD_DIM;
  if (nt == 1) v.st = VSA_HEAD_DIM;
  return v;
}

// Address and strides: 16-byte steps, rows that do not overlap, what a tensor map can hold.
bool view_ok(const View& v) {
  if (v.empty()) return true;
  if (!v.p || !host_aligned16(v.p)) return false;
  for (long long s : {v.sb, v.sh, v.st})
    if (s < VSA_HEAD_DIM || s % 8 != 0 || s >= (1ll << 38)) return false;
  // (beyond any address; what is left adds up in 64 bits)
  constexpr double kMost = 1ll << 56;
  return (double)v.nb * v.sb < kMost && (double)v.nh * v.sh < kMost && (double)v.nt * v.st < kMost;
}

// Whether the rows of a result lie apart: every stride spans what the smaller ones reach.
bool rows_apart(const View& v) {
  if (v.empty()) return true;
  std::pair<long long, long long> d[3] = {{v.sb, v.nb}, {v.sh, v.nh}, {v.st, v.nt}};
  std::sort(d, d + 3);
  long long reach = VSA_HEAD_DIM;
  for (const auto& e : d) {
    if (e.second <= 1) continue;
    if (e.first < reach) return false;
    reach += (e.second - 1) * e.first;
  }
  return true;
}

// Whether two tensors share memory.  Ranges that meet may still be parts of one larger tensor:
// slices of the heads of one token (or of one batch's heads) repeat with the same stride and
// lie apart inside it.
bool views_meet(const View& x, const View& y) {
  if (x.empty() || y.empty()) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  if (a >= b + 2 * (uintptr_t)y.last() || b >= a + 2 * (uintptr_t)x.last()) return false;
  // modulo a period, an axis whose stride is a multiple of it adds nothing, and the others span
  // an interval: two intervals that lie apart inside one period never share an element
  auto span = [](const View& v, long long period) {
    long long n = VSA_HEAD_DIM;
    for (const auto& e : {std::pair<long long, long long>(v.nb, v.sb), {v.nh, v.sh}, {v.nt, v.st}})
      if (e.first > 1 && e.second % period != 0) n += (e.first - 1) * e.second;
    return n;
  };
  for (long long period : {x.sb, x.sh, x.st}) {
    const long long nx = span(x, period), ny = span(y, period);
    const long long apart = ((long long)(b - a) / 2 % period + period) % period;  // y behind x
    if (apart >= nx && apart + ny <= period) return false;
  }
  return true;
}

// Tiles of `heads` heads times `tokens` tokens, 64 of the 128 columns at a time.
bool make_map(CUtensorMap* m, const View& v, int tokens, int heads) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[4] = {VSA_HEAD_DIM, (cuuint64_t)v.nt, (cuuint64_t)v.nh, (cuuint64_t)v.nb};
  cuuint64_t strides[3] = {(cuuint64_t)v.st * 2, (cuuint64_t)v.sh * 2, (cuuint64_t)v.sb * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)tokens, (cuuint32_t)heads, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(v.p), dims, strides, box,
            es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::mutex g_attr_mu;
constexpr int kKernels = 3;
struct KernelInfo {
  bool ready;
  int regs;
} g_kernel[64][kKernels];

// Dynamic shared memory and the register pool that the kernel's re-balancing draws on.
template <typename Kern>
vsa_status prepare(Kern kern, int dev, int slot, uint32_t smem, int threads, uint32_t pool) {
  std::lock_guard<std::mutex> lk(g_attr_mu);
  KernelInfo& k = g_kernel[dev][slot];
  if (!k.ready) {
    cudaFuncAttributes fa;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess ||
        cudaFuncGetAttributes(&fa, kern) != cudaSuccess) {
      cudaGetLastError();
      return VSA_ERR_CUDA;
    }
    k.regs = fa.numRegs;
    k.ready = true;
  }
  return (long long)k.regs * threads < (long long)pool ? VSA_ERR_UNSUPPORTED : VSA_OK;
}

// (More rows than any memory holds are refused, so that counts of them fit 64 bits.)
bool too_many(int packed, int B, int Hq, int Hkv, int Sq, int Sk) {
  constexpr double kMost = 1ll << 40;
  const double n = packed ? 1 : B;
  return n * Hq * Sq > kMost || n * Hkv * Sk > kMost || (double)B * Hq > kMost;
}
// What both directions check: sizes, heads, types of sequence arrays.
struct Shape {
  const int32_t *q_seq, *k_seq;
  int packed, B, Hq, Hkv, Sq, Sk, D, causal;
  float scale;
};
vsa_status check_shape(const Shape& p) {
  if (p.B < 0 || p.Hq < 0 || p.Hkv < 0 || p.Sq < 0 || p.Sk < 0) return VSA_ERR_INVALID_ARG;
  if (p.D != VSA_HEAD_DIM) return VSA_ERR_UNSUPPORTED;
  if (!(p.scale > 0.0f) || !std::isfinite(p.scale)) return VSA_ERR_INVALID_ARG;
  if (p.Hq > 0 && (p.Hkv < 1 || p.Hq % p.Hkv != 0)) return VSA_ERR_INVALID_ARG;
  if (!host_aligned4(p.q_seq) || !host_aligned4(p.k_seq)) return VSA_ERR_INVALID_ARG;
  if (p.packed && p.B > 0 && (!p.q_seq || !p.k_seq)) return VSA_ERR_INVALID_ARG;
  // row coordinates, and with 128 rows behind them, stay below 2^31
  const long long most = INT_MAX - 1024;
  if (p.Sq > most || p.Sk > most || too_many(p.packed, p.B, p.Hq, p.Hkv, p.Sq, p.Sk))
    return VSA_ERR_UNSUPPORTED;
  return VSA_OK;
}
prompt::SeqArgs seq_args(const Shape& p) {
  return prompt::SeqArgs{p.q_seq, p.k_seq, p.packed ? 1 : 0, p.B, p.Sq, p.Sk, p.causal ? 1 : 0, 0};
}

// Heads that share a tile: the largest power of two, 16 at most, that divides a group.  A
// packed tile costs no more than one of a single head, and fills up where tokens are few.
int pack_log(int group) {
  int l = 0;
  while (l < 4 && (group >> l) % 2 == 0) ++l;
  return l;
}

constexpr int kSms = 152;     // of a GB300, which host_device() asks for
constexpr int kMaxSplits = 32;  // a lane each where they are joined

// Into how many ranges of `least` tiles or more the tiles of so many items are cut: as many as
// give each SM `each` of them.
int splits(long long items, long long tiles, int each, int least) {
  const long long fill = items > 0 ? (long long)kSms * each / items : 1, most = tiles / least;
  const long long n = fill < most ? fill : most;
  return n < 2 ? 1 : (n < kMaxSplits ? (int)n : kMaxSplits);
}
// Keys of the forward and of dq: ranges of eight tiles, one an SM.  One token of 12 heads against
// 16,384 keys takes 36 us cut and 228 whole; with two an SM 46, 2,048 tokens of 12 heads 44
// where one an SM (whole) takes 33; in ranges of four tiles 300 tokens of 8 heads against 1,000
// keys take 23, whole 21.
int key_splits(long long items, long long Sk) { return splits(items, (Sk + 127) / 128, 1, 8); }
// Steps of (dk, dv): likewise, and two an SM where ranges keep 32 steps, which evens out what
// causal tiles differ by (8,192 tokens, 12 heads on 2: 501 us of the whole gradient, 751 with
// one an SM).
int step_splits(long long items, long long steps) {
  const int a = splits(items, steps, 1, 8), b = splits(items, steps, 2, 32);
  return a > b ? a : b;
}
// Whether CTAs look up the order of the sequences by length (see find_tile).
int sorted(int B, long long ctas) { return B > 1 && B <= 32 && ctas > kSms; }
long long fwd_items(int packed, long long B, int Hq, int Hkv, long long Sq) {
  const int pack = pack_log(Hq / Hkv);
  return prompt::tile_slots(packed, B, Sq, 256 >> pack) * (Hq >> pack);
}

// Backward: the tiles of both kernels, into how many ranges their steps are cut, and the
// workspace: the rows' statistics, and behind them the ranges' results (of one kernel at a time).
// dq's ranges are chosen as the forward's, dkv's likewise among its steps, one a query tile and
// head pack of its group.
struct BwdLayout {
  long long q_tiles, k_tiles;
  int q_splits, k_splits;
  size_t part, total;
};
BwdLayout bwd_layout(int packed, long long B, int Hq, int Hkv, long long Sq, long long Sk) {
  const int pack = pack_log(Hq / Hkv);
  BwdLayout l;
  l.q_tiles = prompt::tile_slots(packed, B, Sq, 128 >> pack) * (Hq >> pack);
  l.k_tiles = prompt::tile_slots(packed, B, Sk, 128) * Hkv;
  l.q_splits = key_splits(l.q_tiles, Sk);
  l.k_splits = step_splits(l.k_tiles, (Sq * (Hq / Hkv) + 127) / 128);
  l.part = (size_t)l.q_tiles * 1024;
  const size_t dq = l.q_splits > 1 ? (size_t)(l.q_tiles * l.q_splits) *
                                         prompt::bwd::dq::kPartFloats * sizeof(float)
                                   : 0;
  const size_t dkv = l.k_splits > 1 ? (size_t)(l.k_tiles * l.k_splits) * 2 * 128 * 128 * sizeof(float)
                                    : 0;
  l.total = l.part + (dq > dkv ? dq : dkv);
  return l;
}

bool meets(const View& x, const void* p, long long bytes) {
  if (x.empty() || !p || bytes <= 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(p);
  return a < b + (uintptr_t)bytes && b < a + 2 * (uintptr_t)x.last();
}

long long seq_bytes(const Shape& p, const int32_t* s) {
  return s ? ((long long)p.B + (p.packed ? 1 : 0)) * 4 : 0;
}
// Whether a contiguous output shares memory with the sequences' starts or lengths.
bool meets_seq(const Shape& p, const void* x, long long bytes) {
  auto apart = [&](const void* y, long long n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    return !x || !y || a + (uintptr_t)bytes <= b || b + (uintptr_t)n <= a;
  };
  return !apart(p.q_seq, seq_bytes(p, p.q_seq)) || !apart(p.k_seq, seq_bytes(p, p.k_seq));
}

}  // namespace

extern "C" {

size_t vsa_fwd_prompt_workspace_bytes(int packed, int B, int Hq, int Hkv, int Sq, int Sk) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Sq < 1 || Sk < 0 ||
      too_many(packed, B, Hq, Hkv, Sq, Sk))
    return 0;
  const long long items = fwd_items(packed, B, Hq, Hkv, Sq);
  const int n = key_splits(items, Sk);
  return n > 1 ? (size_t)(items * n) * prompt::fwd::kPartFloats * sizeof(float) : 0;
}

vsa_status vsa_fwd_prompt(const vsa_bf16* q, const vsa_bf16* k, const vsa_bf16* v,
                          const int64_t* strides, const int32_t* q_seq, const int32_t* k_seq,
                          int packed, int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal,
                          float scale, vsa_bf16* out, float* lse, void* workspace,
                          size_t workspace_bytes, vsa_stream_t stream) {
  host_set_launches(0);
  const Shape p{q_seq, k_seq, packed, B, Hq, Hkv, Sq, Sk, D, causal, scale};
  vsa_status st = check_shape(p);
  if (st != VSA_OK) return st;
  if (B == 0 || Hq == 0 || Sq == 0) return VSA_OK;
  if (!strides) return VSA_ERR_INVALID_ARG;
  const long long nb = packed ? 1 : B;
  const View vq = view(q, strides, nb, Hq, Sq), vk = view(k, strides + 3, nb, Hkv, Sk),
             vv = view(v, strides + 6, nb, Hkv, Sk), vo = view(out, strides + 9, nb, Hq, Sq);
  for (const View* x : {&vq, &vk, &vv, &vo})
    if (!view_ok(*x)) return VSA_ERR_INVALID_ARG;
  if (!rows_apart(vo) || !host_aligned4(lse)) return VSA_ERR_INVALID_ARG;
  const long long lse_bytes = lse ? nb * Hq * Sq * 4 : 0;
  for (const View* x : {&vq, &vk, &vv})
    if (views_meet(vo, *x) || meets(*x, lse, lse_bytes)) return VSA_ERR_INVALID_ARG;
  if (meets(vo, lse, lse_bytes) || meets(vo, q_seq, seq_bytes(p, q_seq)) ||
      meets(vo, k_seq, seq_bytes(p, k_seq)) || meets_seq(p, lse, lse_bytes))
    return VSA_ERR_INVALID_ARG;

  prompt::FwdArgs a{};
  a.seq = seq_args(p);
  a.out = out;
  a.lse = lse;
  a.out_b = vo.sb;
  a.out_h = vo.sh;
  a.out_t = vo.st;
  a.Hq = Hq;
  a.group = Hq / Hkv;
  a.pack = pack_log(a.group);
  a.n_packs = Hq >> a.pack;
  const long long slots = prompt::tile_slots(packed, B, Sq, 256 >> a.pack);
  if (slots * a.n_packs > INT_MAX) return VSA_ERR_UNSUPPORTED;
  a.n_items = (int)(slots * a.n_packs);
  a.splits = 1;
  if (workspace != nullptr) {
    const size_t need = vsa_fwd_prompt_workspace_bytes(packed, B, Hq, Hkv, Sq, Sk);
    if (!host_aligned16(workspace) || workspace_bytes < need) return VSA_ERR_INVALID_ARG;
    const long long n = (long long)need;
    for (const View* x : {&vq, &vk, &vv, &vo})
      if (meets(*x, workspace, n)) return VSA_ERR_INVALID_ARG;
    const uintptr_t w0 = reinterpret_cast<uintptr_t>(workspace), l0 = reinterpret_cast<uintptr_t>(lse);
    if (meets_seq(p, workspace, n) ||
        (lse && w0 < l0 + (uintptr_t)lse_bytes && l0 < w0 + (uintptr_t)n))
      return VSA_ERR_INVALID_ARG;
    a.splits = key_splits(a.n_items, Sk);
    a.part = static_cast<float*>(workspace);
  }
  a.scale_log2 = scale * 1.4426950408889634f;
  // The softmax warps of a query tile without queries wait while its item's other tile walks over
  // the keys, 1.7 us per 128: a second more for every 2^25 of them (0.45 s).
  a.wait_ns = host_wait_ns(prompt::kWaitLimitNs * (1 + (Sk >> 25)));
  a.stall = host_stall();

  a.seq.sort = sorted(B, (long long)a.n_items * a.splits);

  int dev = 0;
  st = host_device(&dev);
  if (st != VSA_OK) return st;
  a.status = host_status_word();
  if (a.status == nullptr) return VSA_ERR_CUDA;
  st = prepare(prompt::fwd::prompt_fwd_kernel, dev, 0, prompt::fwd::kSmemBytes,
               prompt::fwd::kThreads, prompt::fwd::kRegPoolNeeded);
  if (st != VSA_OK) return st;
  CUtensorMap tq, tk, tv;
  // without keys nothing is fetched through their maps, which only have to encode
  if (!make_map(&tq, vq, 128 >> a.pack, 1 << a.pack) || !make_map(&tk, vk.empty() ? vq : vk, 128, 1) ||
      !make_map(&tv, vv.empty() ? vq : vv, 128, 1))
    return VSA_ERR_CUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = launch(prompt::fwd::prompt_fwd_kernel, dim3((unsigned)(a.n_items * a.splits)),
              prompt::fwd::kThreads, prompt::fwd::kSmemBytes, s, 0, tq, tk, tv, a);
  if (st == VSA_OK && a.splits > 1)
    st = launch(prompt::fwd::prompt_join_kernel, dim3((unsigned)(a.n_items * 32)), 256, 0, s, 0, a);
  if (st != VSA_OK) return st;
  host_set_launches(a.splits > 1 ? 2 : 1);
  return VSA_OK;
}

size_t vsa_bwd_prompt_workspace_bytes(int packed, int B, int Hq, int Hkv, int Sq, int Sk) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Sq < 0 || Sk < 0 ||
      too_many(packed, B, Hq, Hkv, Sq, Sk))
    return 0;
  return bwd_layout(packed, B, Hq, Hkv, Sq, Sk).total;
}

vsa_status vsa_bwd_prompt(const vsa_bf16* q, const vsa_bf16* k, const vsa_bf16* v,
                          const vsa_bf16* out, const vsa_bf16* dout, const float* lse,
                          const int64_t* strides, const int32_t* q_seq, const int32_t* k_seq,
                          int packed, int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal,
                          float scale, vsa_bf16* dq, vsa_bf16* dk, vsa_bf16* dv, void* workspace,
                          size_t workspace_bytes, vsa_stream_t stream) {
  host_set_launches(0);
  const Shape p{q_seq, k_seq, packed, B, Hq, Hkv, Sq, Sk, D, causal, scale};
  vsa_status st = check_shape(p);
  if (st != VSA_OK) return st;
  if (B == 0 || Hq == 0 || (Sq == 0 && Sk == 0)) return VSA_OK;
  if (!strides) return VSA_ERR_INVALID_ARG;
  const long long nb = packed ? 1 : B;
  const View vq = view(q, strides, nb, Hq, Sq), vk = view(k, strides + 3, nb, Hkv, Sk),
             vv = view(v, strides + 6, nb, Hkv, Sk), vo = view(out, strides + 9, nb, Hq, Sq),
             vg = view(dout, strides + 12, nb, Hq, Sq), wq = view(dq, strides + 15, nb, Hq, Sq),
             wk = view(dk, strides + 18, nb, Hkv, Sk), wv = view(dv, strides + 21, nb, Hkv, Sk);
  const View* in[5] = {&vq, &vk, &vv, &vo, &vg};
  const View* res[3] = {&wq, &wk, &wv};
  for (const View* x : in)
    if (!view_ok(*x)) return VSA_ERR_INVALID_ARG;
  for (const View* x : res)
    if (!view_ok(*x) || !rows_apart(*x)) return VSA_ERR_INVALID_ARG;
  const BwdLayout l = bwd_layout(packed, B, Hq, Hkv, Sq, Sk);
  const size_t need = l.total;
  const long long lse_bytes = nb * Hq * Sq * 4;
  if (Sq > 0 && (!lse || !host_aligned4(lse) || !workspace || workspace_bytes < need ||
                 !host_aligned16(workspace)))
    return VSA_ERR_INVALID_ARG;
  for (const View* y : res) {
    for (const View* x : in)
      if (views_meet(*y, *x)) return VSA_ERR_INVALID_ARG;
    for (const View* x : res)
      if (x != y && views_meet(*y, *x)) return VSA_ERR_INVALID_ARG;
    if (meets(*y, lse, lse_bytes) || meets(*y, workspace, (long long)need) ||
        meets(*y, q_seq, seq_bytes(p, q_seq)) || meets(*y, k_seq, seq_bytes(p, k_seq)))
      return VSA_ERR_INVALID_ARG;
  }
  for (const View* x : in)
    if (meets(*x, workspace, (long long)need)) return VSA_ERR_INVALID_ARG;
  const uintptr_t w0 = reinterpret_cast<uintptr_t>(workspace), l0 = reinterpret_cast<uintptr_t>(lse);
  if (Sq > 0 && ((w0 < l0 + (uintptr_t)lse_bytes && l0 < w0 + need) ||
                 meets_seq(p, workspace, (long long)need)))
    return VSA_ERR_INVALID_ARG;

  prompt::bwd::Args a{};
  a.seq = seq_args(p);
  a.stats = static_cast<float*>(workspace);
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.pack = pack_log(a.group);
  a.n_packs = Hq >> a.pack;
  if (l.q_tiles > INT_MAX || l.k_tiles > INT_MAX) return VSA_ERR_UNSUPPORTED;
  a.n_tslots = (int)(l.q_tiles / a.n_packs);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + l.part);
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.wait_ns = host_wait_ns(prompt::kWaitLimitNs);
  a.stall = host_stall();

  int dev = 0;
  st = host_device(&dev);
  if (st != VSA_OK) return st;
  a.status = host_status_word();
  if (a.status == nullptr) return VSA_ERR_CUDA;
  namespace pb = prompt::bwd;
  st = prepare(pb::dkv::prompt_dkv_kernel, dev, 1, pb::dkv::kSmemBytes, pb::kThreads,
               pb::kRegPoolNeeded);
  if (st != VSA_OK) return st;
  st = prepare(pb::dq::prompt_dq_kernel, dev, 2, pb::dq::kSmemBytes, pb::kThreads,
               pb::kRegPoolNeeded);
  if (st != VSA_OK) return st;
  CUtensorMap tq, tg, tk, tv;
  // what is empty is not fetched: its map only has to encode
  const View &mq = vq.empty() ? vk : vq, &mg = vg.empty() ? vk : vg, &mk = vk.empty() ? vq : vk,
             &mv = vv.empty() ? vq : vv;
  if (!make_map(&tq, mq, 128 >> a.pack, 1 << a.pack) ||
      !make_map(&tg, mg, 128 >> a.pack, 1 << a.pack) || !make_map(&tk, mk, 128, 1) ||
      !make_map(&tv, mv, 128, 1))
    return VSA_ERR_CUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int launches = 0;
  // each starts up while the one before ends; dkv takes the D that dq leaves
  if (Sq > 0) {
    a.out = out;
    a.dout = dout;
    a.lse = lse;
    a.o_b = vo.sb;
    a.o_h = vo.sh;
    a.o_t = vo.st;
    a.g_b = vg.sb;
    a.g_h = vg.sh;
    a.g_t = vg.st;
    a.d0 = dq;
    a.d0_b = wq.sb;
    a.d0_h = wq.sh;
    a.d0_t = wq.st;
    a.splits = l.q_splits;
    a.seq.sort = sorted(B, l.q_tiles * a.splits);
    st = launch(pb::dq::prompt_dq_kernel, dim3((unsigned)(l.q_tiles * a.splits)), pb::kThreads,
                pb::dq::kSmemBytes, s, 0, tq, tg, tk, tv, a);
    if (st != VSA_OK) return st;
    ++launches;
    if (a.splits > 1) {
      st = launch(pb::dq::prompt_dq_join_kernel, dim3((unsigned)(l.q_tiles * 16)), 256, 0, s, 0, a);
      if (st != VSA_OK) return st;
      ++launches;
    }
  }
  if (Sk > 0) {
    a.d0 = dk;
    a.d0_b = wk.sb;
    a.d0_h = wk.sh;
    a.d0_t = wk.st;
    a.d1 = dv;
    a.d1_b = wv.sb;
    a.d1_h = wv.sh;
    a.d1_t = wv.st;
    a.splits = Sq > 0 ? l.k_splits : 1;
    a.seq.sort = sorted(B, l.k_tiles * a.splits);
    st = launch(pb::dkv::prompt_dkv_kernel, dim3((unsigned)(l.k_tiles * a.splits)), pb::kThreads,
                pb::dkv::kSmemBytes, s, 0, tq, tg, tk, tv, a);
    if (st != VSA_OK) return st;
    ++launches;
    if (a.splits > 1) {
      st = launch(pb::dkv::prompt_dkv_join_kernel, dim3((unsigned)(l.k_tiles * 32)), 256, 0, s, 0, a);
      if (st != VSA_OK) return st;
      ++launches;
    }
  }
  host_set_launches(launches);
  return VSA_OK;
}

}  // extern "C"

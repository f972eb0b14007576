// Host side of the serving entries of the C ABI (rotation and append, decode, prompts): argument
// validation and kernel launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <exception>
#include <mutex>
#include <utility>
#include <vector>

// s2_device.cuh defines this one function out of line; the library's other translation unit has
// it under its own name.
#define wait_slow wait_slow_serve

#include "../../include/s2attn.h"
#include "s2_append.cuh"
#include "s2_decode.cuh"
#include "s2_host.h"
#include "s2_prompt.cuh"

namespace {

using s2host::aligned16;
using s2host::cuda_fail;
using s2host::device_state;
using s2host::kMaxDevices;

struct ServeDevice {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
ServeDevice g_serve_dev[kMaxDevices];

template <int D>
cudaError_t serve_smem_attrs() {
  cudaError_t e = cudaFuncSetAttribute(
      s2::s2_decode_kernel<D, 8>, cudaFuncAttributeMaxDynamicSharedMemorySize, s2::DecodeLayout<D, 8>::kBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(s2::s2_decode_kernel<D, 16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           s2::DecodeLayout<D, 16>::kBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(s2::s2_prompt_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           s2::PromptLayout<D>::kLaunchBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(s2::s2_prompt_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              s2::PromptLayout<D>::kLaunchBytes);
}

// The error word and SM count of the current device, with the serving kernels set up on it.
s2attn_status serve_device(unsigned int** err, int* num_sms) {
  int dev = 0;
  const s2attn_status s = device_state(err, num_sms, &dev);
  if (s != S2ATTN_OK) return s;
  ServeDevice& d = g_serve_dev[dev];
  std::call_once(d.once, [&] {
    d.err = serve_smem_attrs<64>();
    if (d.err == cudaSuccess) d.err = serve_smem_attrs<128>();
  });
  return d.err == cudaSuccess ? S2ATTN_OK : cuda_fail(d.err, "device set-up");
}

// A launch that may start before the kernel in front of it has ended (the kernel waits: pdl_wait).
template <class... Params, class... Args>
s2attn_status launch_early(const char* what, void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                           cudaStream_t stream, Args&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  return e == cudaSuccess ? S2ATTN_OK : cuda_fail(e, what);
}

s2attn_status check_heads(int Hq, int Hkv, int d) {
  if (Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv != 0) return S2ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return S2ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(Hq) * d >= (1ll << 31)) return S2ATTN_ERR_UNSUPPORTED;
  return S2ATTN_OK;
}

bool too_many_rows(int B, int Hq) { return static_cast<long long>(B) * Hq >= (1ll << 31); }

// A token (or batch row) stride: whole 16-byte chunks, rows that do not overlap.
bool bad_row_stride(long long st, int heads, int d) {
  return st % 8 != 0 || st < static_cast<long long>(heads) * d;
}

// The paged cache's shape and {page, token} strides of K and V (null: contiguous).
s2attn_status check_cache(int Hkv, int d, int pages, int page_size, int max_pages,
                          const long long* strides, s2::PagedRef& kc, s2::PagedRef& vc) {
  if (pages <= 0 || page_size <= 0 || max_pages <= 0) return S2ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * page_size > INT_MAX - 128) return S2ATTN_ERR_UNSUPPORTED;
  const long long st = static_cast<long long>(Hkv) * d;
  kc.st = vc.st = st;
  kc.sp = vc.sp = st * page_size;
  if (strides) {
    for (int i = 0; i < 4; i += 2) {
      const long long sp = strides[i], tt = strides[i + 1];
      // tokens of a page may interleave with other tensors, pages may not overlap
      if (bad_row_stride(tt, Hkv, d) || sp % 8 != 0 || sp <= 0) return S2ATTN_ERR_INVALID_ARG;
      if (pages > 1 && sp < (page_size - 1) * tt + st) return S2ATTN_ERR_INVALID_ARG;
    }
    kc.sp = strides[0]; kc.st = strides[1];
    vc.sp = strides[2]; vc.st = strides[3];
  }
  return S2ATTN_OK;
}

s2::FastDiv fast_div_by(int d) {
  int l = 0;
  while ((1ll << l) < d) ++l;
  s2::FastDiv f;
  f.shift = 31 + l;
  f.mul = static_cast<unsigned int>(((1ull << f.shift) + d - 1) / d);
  return f;
}

// F_i of s2_append.cuh for one (base, pi_scale, d); the last one is kept by each host thread.
const unsigned long long* turns(double base, double pi_scale, int d) {
  static thread_local struct { double base, pi; int d; unsigned long long f[64]; } last = {0.0, 0.0, 0, {}};
  if (last.base != base || last.pi != pi_scale || last.d != d) {
    const long double two_pi = 6.283185307179586476925286766559L;
    for (int i = 0; i < d / 2; ++i) {
      long double x = static_cast<long double>(pi_scale) *
                      powl(static_cast<long double>(base), -2.0L * i / d) / two_pi;
      x = (x - floorl(x)) * 18446744073709551616.0L;
      last.f[i] = x >= 18446744073709551615.0L ? 0ull : static_cast<unsigned long long>(x + 0.5L);
    }
    last.base = base;
    last.pi = pi_scale;
    last.d = d;
  }
  return last.f;
}

// Where one token's heads leave more than half of a block idle, a block takes as many groups of tokens as give
// each thread one unit, but no more than leave two blocks per SM; the heads split over the second axis until
// two blocks per SM exist.
template <int D>
s2attn_status launch_append(s2::AppendParams& p, int num_sms, cudaStream_t stream) {
  const int items = (p.Hq + 2 * p.Hkv) * (D / 16);
  p.subs = std::max(1, std::min({s2::kAppendThreads / items, s2::kAppendMaxTokens / s2::kAppendUnit,
                                 p.T / (2 * num_sms * s2::kAppendUnit)}));
  const int groups = (p.T - 1) / (p.subs * s2::kAppendUnit) + 1;
  const int most = (items * p.subs + s2::kAppendThreads - 1) / s2::kAppendThreads;
  const dim3 grid(groups, std::max(1, std::min(most, 2 * num_sms / groups)));
  return launch_early("s2_append_kernel launch",
                      p.subs > 1 ? s2::s2_append_kernel<D, true> : s2::s2_append_kernel<D, false>, grid,
                      s2::kAppendThreads, 0, stream, p);
}

constexpr size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
// Workspace of the decode: first pieces | partial outputs | partial {max, sum} | tails.
struct DecodeSpace {
  size_t first, part, ml, tail;
};
DecodeSpace decode_space(int group, int d) {
  const size_t ctas = s2::kDecodeMaxCtas, rows = std::min(group, s2::kDecodeRows);
  return {round256(ctas * s2::kDecodeWarps * rows * d * sizeof(float)),
          round256(ctas * 2 * rows * d * sizeof(float)), round256(ctas * 2 * rows * sizeof(float2)),
          round256(ctas * sizeof(s2::DecodeTail))};
}

template <int D>
s2attn_status launch_decode(const s2::DecodeParams& p, int grid, cudaStream_t stream) {
  const s2attn_status s = launch_early(
      "s2_decode_kernel launch", p.rows <= 8 ? s2::s2_decode_kernel<D, 8> : s2::s2_decode_kernel<D, 16>, dim3(grid),
      s2::kDecodeThreads, p.rows <= 8 ? s2::DecodeLayout<D, 8>::kBytes : s2::DecodeLayout<D, 16>::kBytes, stream, p);
  if (s != S2ATTN_OK || grid == 1 || p.whole) return s;   // one CTA, or whole segments: nothing crosses CTAs
  return launch_early("s2_decode_join_kernel launch", s2::s2_decode_join_kernel<D>, dim3(grid - 1, p.rows),
                      s2::kDecodeJoinThreads, 0, stream, p);
}

// Tensor map over the rows of a packed bf16 [T, H, d] tensor: dims (d, H, T, 1), box (64, 1, rows, 1),
// 128-byte swizzle, zeros out of bounds.
s2attn_status encode_rows(CUtensorMap* m, const void* base, int T, int H, int d, int box_rows, long long st) {
  const auto encode = s2host::encoder();
  if (!encode) return S2ATTN_ERR_CUDA;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T, 1};
  cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)st * 2, (cuuint64_t)st * 2 * T};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
                            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? S2ATTN_OK : s2host::fail(S2ATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed");
}

// K and V of the kv heads that are taken together stay below this: half of L2.
constexpr long long kPromptL2Bytes = 64ll << 20;

// One launch per kPromptMaxSeqs sequences and kPromptMaxTiles query tiles.
template <int D>
s2attn_status launch_prompt(s2::PromptParams& p, const CUtensorMap (&maps)[4], const int* cu, int n_seqs,
                            cudaStream_t stream) {
  static thread_local s2::PromptWork work;
  static thread_local std::vector<int> order;
  const bool heads = p.group % 2 == 0;
  const int rows = heads ? s2::kTileRows : 2 * s2::kTileRows, per_kv = heads ? p.group / 2 : p.group;
  order.clear();
  for (int i = 0; i < n_seqs; ++i)
    if (cu[i + 1] > cu[i]) order.push_back(i);
  std::stable_sort(order.begin(), order.end(),
                   [&](int a, int b) { return cu[a + 1] - cu[a] > cu[b + 1] - cu[b]; });
  auto launch = [&]() -> s2attn_status {
    const unsigned grid = static_cast<unsigned>(p.Hkv) * per_kv * p.n_tiles;
    const s2attn_status s = launch_early(
        "s2_prompt_kernel launch", heads ? s2::s2_prompt_kernel<D, true> : s2::s2_prompt_kernel<D, false>, dim3(grid),
        s2::PromptLayout<D>::kThreads, s2::PromptLayout<D>::kLaunchBytes, stream, maps[0], maps[1], maps[2], maps[3], p,
        work);
    p.n_tiles = 0;
    return s;
  };
  for (size_t at = 0; at < order.size(); at += s2::kPromptMaxSeqs) {
    const int count = static_cast<int>(std::min<size_t>(s2::kPromptMaxSeqs, order.size() - at));
    long long tokens = 0;
    for (int i = 0; i < count; ++i) {
      const int s = order[at + i];
      work.start[i] = cu[s];
      work.len[i] = cu[s + 1] - cu[s];
      tokens += work.len[i];
    }
    p.kv_chunk = static_cast<int>(std::max(1ll, std::min<long long>(p.Hkv, kPromptL2Bytes / (tokens * 4 * D))));
    p.n_tiles = 0;
    int live = 0;   // the sequences (longest first) that have a tile t
    for (int t = (work.len[0] - 1) / rows; t >= 0; --t) {
      while (live < count && (work.len[live] - 1) / rows >= t) ++live;
      for (int i = 0; i < live; ++i) {
        work.tile[p.n_tiles++] = static_cast<unsigned>(i) << 16 | static_cast<unsigned>(t);
        if (p.n_tiles == s2::kPromptMaxTiles) {
          const s2attn_status s = launch();
          if (s != S2ATTN_OK) return s;
        }
      }
    }
    if (p.n_tiles > 0) {
      const s2attn_status s = launch();
      if (s != S2ATTN_OK) return s;
    }
  }
  return S2ATTN_OK;
}

s2attn_status rope_append(const void* q, void* q_rot, const void* k, void* k_rot, const void* v, void* k_cache,
                          void* v_cache, const int* block_table, const int* cu_seqlens, const int* cache_lens, int T,
                          int B, int Hq, int Hkv, int d, int pages, int page_size, int max_pages, double base,
                          double pi_scale, const long long* strides, void* stream) {
  if (!k || !v || !k_cache || !v_cache || !block_table || !cache_lens) return S2ATTN_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_rot == nullptr)) return S2ATTN_ERR_INVALID_ARG;
  const void* ptrs[7] = {q, q_rot, k, k_rot, v, k_cache, v_cache};
  for (const void* x : ptrs)
    if (!aligned16(x)) return S2ATTN_ERR_INVALID_ARG;
  if (T <= 0 || B <= 0 || (!cu_seqlens && T != B)) return S2ATTN_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base) || !(pi_scale > 0.0) || !std::isfinite(pi_scale))
    return S2ATTN_ERR_INVALID_ARG;
  s2attn_status s = check_heads(Hq, Hkv, d);
  if (s != S2ATTN_OK) return s;
  s2::AppendParams p{};
  if ((s = check_cache(Hkv, d, pages, page_size, max_pages, strides ? strides + 5 : nullptr, p.kc,
                       p.vc)) != S2ATTN_OK)
    return s;
  const long long q_st = static_cast<long long>(Hq) * d, k_st = static_cast<long long>(Hkv) * d;
  long long st[5] = {q_st, q_st, k_st, k_st, k_st};   // q, q_rot, k, k_rot, v
  if (strides)
    for (int i = 0; i < 5; ++i) {
      st[i] = strides[i];
      if (bad_row_stride(st[i], i < 2 ? Hq : Hkv, d)) return S2ATTN_ERR_INVALID_ARG;
    }
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_rot = static_cast<__nv_bfloat16*>(q_rot);
  p.k_rot = static_cast<__nv_bfloat16*>(k_rot);
  p.q_st = st[0]; p.qr_st = st[1]; p.k_st = st[2]; p.kr_st = st[3]; p.v_st = st[4];
  p.kc.p = static_cast<__nv_bfloat16*>(k_cache);
  p.vc.p = static_cast<__nv_bfloat16*>(v_cache);
  p.table = block_table; p.cu = cu_seqlens; p.lens = cache_lens;
  p.T = T; p.B = B; p.Hq = q ? Hq : 0; p.Hkv = Hkv;
  p.pages = pages; p.page_size = page_size; p.max_pages = max_pages;
  const unsigned long long* f = turns(base, pi_scale, d);
  std::copy(f, f + d / 2, p.turn);
  int num_sms = 0;
  if ((s = serve_device(&p.err, &num_sms)) != S2ATTN_OK) return s;
  cudaStream_t sm = static_cast<cudaStream_t>(stream);
  return d == 64 ? launch_append<64>(p, num_sms, sm) : launch_append<128>(p, num_sms, sm);
}

}  // namespace

extern "C" {

s2attn_status s2attn_rope_append(const void* q, void* q_rot, const void* k, void* k_rot,
                                 const void* v, void* k_cache, void* v_cache,
                                 const int* block_table, const int* cu_seqlens,
                                 const int* cache_lens, int T, int B, int Hq, int Hkv, int d,
                                 int pages, int page_size, int max_pages, float base,
                                 float pi_scale, const long long* strides, void* stream) {
  return rope_append(q, q_rot, k, k_rot, v, k_cache, v_cache, block_table, cu_seqlens, cache_lens, T, B, Hq, Hkv, d,
                     pages, page_size, max_pages, base, pi_scale, strides, stream);
}

s2attn_status s2attn_rope_append_f64(const void* q, void* q_rot, const void* k, void* k_rot,
                                     const void* v, void* k_cache, void* v_cache,
                                     const int* block_table, const int* cu_seqlens,
                                     const int* cache_lens, int T, int B, int Hq, int Hkv, int d,
                                     int pages, int page_size, int max_pages, double base,
                                     double pi_scale, const long long* strides, void* stream) {
  return rope_append(q, q_rot, k, k_rot, v, k_cache, v_cache, block_table, cu_seqlens, cache_lens, T, B, Hq, Hkv, d,
                     pages, page_size, max_pages, base, pi_scale, strides, stream);
}

size_t s2attn_decode_workspace_size(int B, int Hq, int Hkv, int d) {
  if (B <= 0 || check_heads(Hq, Hkv, d) != S2ATTN_OK || too_many_rows(B, Hq)) return 0;
  const DecodeSpace w = decode_space(Hq / Hkv, d);
  return w.first + w.part + w.ml + w.tail;
}

s2attn_status s2attn_decode(const void* q, const void* k_cache, const void* v_cache,
                            const int* block_table, const int* cache_lens, void* o, float* lse,
                            int B, int Hq, int Hkv, int d, int pages, int page_size, int max_pages,
                            float scale, const long long* strides, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !block_table || !cache_lens || !o || !workspace)
    return S2ATTN_ERR_INVALID_ARG;
  const void* ptrs[4] = {q, k_cache, v_cache, o};
  for (const void* x : ptrs)
    if (!aligned16(x)) return S2ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return S2ATTN_ERR_INVALID_ARG;
  if (B <= 0 || !(scale > 0.f) || !std::isfinite(scale)) return S2ATTN_ERR_INVALID_ARG;
  s2attn_status s = check_heads(Hq, Hkv, d);
  if (s != S2ATTN_OK) return s;
  if (too_many_rows(B, Hq)) return S2ATTN_ERR_UNSUPPORTED;
  s2::DecodeParams p{};
  if ((s = check_cache(Hkv, d, pages, page_size, max_pages, strides ? strides + 2 : nullptr, p.kc,
                       p.vc)) != S2ATTN_OK)
    return s;
  p.q_sb = p.o_sb = static_cast<long long>(Hq) * d;
  if (strides) {
    p.q_sb = strides[0];
    p.o_sb = strides[1];
    if (bad_row_stride(p.q_sb, Hq, d) || bad_row_stride(p.o_sb, Hq, d)) return S2ATTN_ERR_INVALID_ARG;
  }
  if (workspace_bytes < s2attn_decode_workspace_size(B, Hq, Hkv, d)) return S2ATTN_ERR_INVALID_ARG;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.kc.p = static_cast<__nv_bfloat16*>(const_cast<void*>(k_cache));
  p.vc.p = static_cast<__nv_bfloat16*>(const_cast<void*>(v_cache));
  p.table = block_table; p.lens = cache_lens;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv;
  p.pages = pages; p.page_size = page_size; p.max_pages = max_pages;
  p.group = Hq / Hkv;
  p.chunks = (p.group + s2::kDecodeRows - 1) / s2::kDecodeRows;
  p.rows = std::min(p.group, s2::kDecodeRows);
  p.by_page = fast_div_by(page_size);
  p.scale_log2 = scale * 1.4426950408889634f;
  const DecodeSpace w = decode_space(p.group, d);
  char* ws = static_cast<char*>(workspace);
  p.first_o = reinterpret_cast<float*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + w.first);
  p.part_ml = reinterpret_cast<float2*>(ws + w.first + w.part);
  p.tail = reinterpret_cast<s2::DecodeTail*>(ws + w.first + w.part + w.ml);
  int num_sms = 0;
  if ((s = serve_device(&p.err, &num_sms)) != S2ATTN_OK) return s;
  // No more CTAs than the longest batch the block table can describe has work for.
  const long long tiles = static_cast<long long>(B) * Hkv * p.chunks *
                          ((static_cast<long long>(max_pages) * page_size - 1) / s2::kDecodeTile + 1 +
                           s2::kDecodeGap);
  const long long segments = static_cast<long long>(B) * Hkv * p.chunks;
  const int most = std::min(num_sms, s2::kDecodeMaxCtas);
  p.whole = segments <= most && max_pages * page_size <= s2::kDecodeWholeTokens;
  const int grid = static_cast<int>(p.whole ? segments : std::min<long long>(most, tiles));
  cudaStream_t sm = static_cast<cudaStream_t>(stream);
  return d == 64 ? launch_decode<64>(p, grid, sm) : launch_decode<128>(p, grid, sm);
}

s2attn_status s2attn_prompt_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                                const int* cu_seqlens, int n_seqs, int T, int Hq, int Hkv, int d,
                                float scale, const long long* strides, void* stream) {
  if (!q || !k || !v || !o || !lse || !cu_seqlens) return S2ATTN_ERR_INVALID_ARG;
  const void* ptrs[4] = {q, k, v, o};
  for (const void* x : ptrs)
    if (!aligned16(x)) return S2ATTN_ERR_INVALID_ARG;
  if (n_seqs <= 0 || T <= 0 || !(scale > 0.f) || !std::isfinite(scale)) return S2ATTN_ERR_INVALID_ARG;
  s2attn_status s = check_heads(Hq, Hkv, d);
  if (s != S2ATTN_OK) return s;
  // units of one launch are counted, and query tiles of a sequence numbered, in 31 and 16 bits
  if (Hq >= (1 << 20) || T > (1 << 23)) return S2ATTN_ERR_UNSUPPORTED;
  if (cu_seqlens[0] < 0 || cu_seqlens[n_seqs] > T) return S2ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < n_seqs; ++i)
    if (cu_seqlens[i + 1] < cu_seqlens[i]) return S2ATTN_ERR_INVALID_ARG;
  const int head_count[4] = {Hq, Hkv, Hkv, Hq};
  long long st[4];   // q, k, v, o
  for (int i = 0; i < 4; ++i) {
    st[i] = strides ? strides[i] : static_cast<long long>(head_count[i]) * d;
    if (bad_row_stride(st[i], head_count[i], d)) return S2ATTN_ERR_INVALID_ARG;
  }
  CUtensorMap maps[4];
  if ((s = encode_rows(&maps[0], q, T, Hq, d, s2::kTileRows, st[0])) != S2ATTN_OK) return s;
  if ((s = encode_rows(&maps[1], k, T, Hkv, d, s2::kPromptKeys, st[1])) != S2ATTN_OK) return s;
  if ((s = encode_rows(&maps[2], v, T, Hkv, d, s2::kPromptKeys, st[2])) != S2ATTN_OK) return s;
  if ((s = encode_rows(&maps[3], o, T, Hq, d, 8, st[3])) != S2ATTN_OK) return s;
  s2::PromptParams p{};
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.v_st = st[2];
  p.o = static_cast<__nv_bfloat16*>(o);
  p.o_st = st[3];
  p.lse = lse;
  p.T = T; p.Hq = Hq; p.Hkv = Hkv; p.group = Hq / Hkv;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.timeout_ns = s2host::wait_timeout_ns();
  int num_sms = 0;
  if ((s = serve_device(&p.err, &num_sms)) != S2ATTN_OK) return s;
  cudaStream_t sm = static_cast<cudaStream_t>(stream);
  try {
    return d == 64 ? launch_prompt<64>(p, maps, cu_seqlens, n_seqs, sm)
                   : launch_prompt<128>(p, maps, cu_seqlens, n_seqs, sm);
  } catch (const std::exception&) {   // the sequences' order is host memory
    return s2host::fail(S2ATTN_ERR_CUDA, "s2attn_prompt_fwd: out of host memory");
  }
}

}  // extern "C"

// Rotation and append: the step between the projections and the attention when a model answers.
// Each new token's query and key heads turn by the rotary angle of its position (Position
// Interpolation, LongLoRA summary page, §4 "Model setup"), and the turned key and the value go to
// the token's slot of a paged cache.
//
// For position t and i < D/2 the pair (x[i], x[i + D/2]) turns by t * pi_scale * base^(-2i/D).
// Positions reach 10^5 and more, where an fp32 product is off by 1e-2 rad; the angle is instead
// formed in turns, as 64-bit fixed point: F_i = frac(pi_scale * base^(-2i/D) / 2 pi) * 2^64 (on the
// host, from base and pi_scale in 64 bits, rounded once), and t * F_i modulo 2^64 is the exact
// fraction of a turn (error t * 2^-64). Its upper 32 bits, as a signed number, are sincospif's argument.
//
// Memory bound: every element is read once and written once or twice. A block takes a few tokens;
// one lane per token finds its sequence (binary search of cu_seqlens) and slot, and all threads the
// tokens' angles, shared by all heads through shared memory. The work then is units of one 16-byte
// chunk of a head's first half and its partner D/2 columns on, for 4 tokens: 8 loads of 16 bytes in
// flight a thread, 128 KB an SM, the first ones issued before the slots and angles are known. 4 tokens a
// block where the heads give a block's threads work, up to 32 where they do not, as many as give every
// thread one unit. A grid of few blocks splits the heads over its second axis.
// 64 registers a thread keep four blocks on an SM; 4 to 20 bytes of them spill.
// Measured (device time): 32768 tokens of 64 + 2 x 8 heads, d = 128: 217 us, 6.5 TB/s (8-token units and
// blocks: 218 us, and 4.8 against 3.6 us for a batch of 64 tokens); 9830 tokens of 4 + 2 x 4 heads, d = 64:
// 10.0 us, bound by the chain of lookups of a single wave of blocks.
#pragma once

#include "s2_serve_common.cuh"

namespace s2 {

constexpr int kAppendUnit = 4;            // tokens of a work unit
constexpr int kAppendThreads = 256;
constexpr int kAppendMaxTokens = 32;      // of a block

struct AppendParams {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_rot, *k_rot;          // k_rot null: the turned keys go to the cache only
  long long q_st, k_st, v_st, qr_st, kr_st;
  PagedRef kc, vc;
  const int *table, *cu, *lens;          // cu null: one token per sequence
  int T, B, Hq, Hkv, pages, page_size, max_pages;
  int subs;                              // units of 4 tokens a block takes (of each head's chunk)
  unsigned int* err;
  unsigned long long turn[64];           // F_i
};

// The number of i in [1, B] with cu[i] <= t: the sequence that holds token t, B behind the last.
__device__ __forceinline__ int find_sequence(const int* cu, int B, int t) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (cu[mid + 1] <= t) lo = mid + 1; else hi = mid;
  }
  return lo;
}

// kWide: p.subs units of 4 tokens a block, else one.
template <int D, bool kWide>
__global__ void __launch_bounds__(kAppendThreads, 4) s2_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kHalf = D / 2;
  constexpr int kChunks = D / 16;        // work items of a head: a 16-byte chunk and its partner
  constexpr int kTok = kWide ? kAppendMaxTokens : kAppendUnit;   // room in shared memory
  const int subs = kWide ? p.subs : 1, tok = subs * kAppendUnit;
  __shared__ float s_cos[kTok][kHalf], s_sin[kTok][kHalf];
  __shared__ long long s_slot_k[kTok], s_slot_v[kTok];   // -1: not to be cached
  __shared__ int s_pos[kTok];                            // -1: to be skipped
  pdl_wait();
  const int t_block = blockIdx.x * tok;
  const int items = (p.Hq + 2 * p.Hkv) * kChunks, units = items * subs;
  const int step = gridDim.y * kAppendThreads;
  int w = blockIdx.y * kAppendThreads + threadIdx.x;

  uint4 lo[kAppendUnit], hi[kAppendUnit];
  auto load = [&](int unit) {
    const int sub = kWide ? unit / items : 0, item = unit - sub * items;
    const int t0 = t_block + sub * kAppendUnit;
    const int h = item / kChunks, c = item % kChunks;
    const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
    const __nv_bfloat16* src = is_q ? p.q : is_k ? p.k : p.v;
    const long long st = is_q ? p.q_st : is_k ? p.k_st : p.v_st;
    const int hh = is_q ? h : is_k ? h - p.Hq : h - p.Hq - p.Hkv;
    src += t0 * st + static_cast<long long>(hh) * D + 8 * c;
#pragma unroll
    for (int tt = 0; tt < kAppendUnit; ++tt)
      if (t0 + tt < p.T) {
        lo[tt] = *reinterpret_cast<const uint4*>(src + tt * st);
        hi[tt] = *reinterpret_cast<const uint4*>(src + tt * st + kHalf);
      }
  };
  if (w < units) load(w);

  // ---- the tokens' positions and slots, one lane each ----
  if (threadIdx.x < tok) {
    const int t = t_block + threadIdx.x;
    long long pos = -1;
    int seq = t, len = 0;
    if (t < p.T) {
      if (p.cu) {
        seq = find_sequence(p.cu, p.B, t);
        if (seq < p.B && t >= p.cu[seq]) {
          len = p.lens[seq];
          pos = static_cast<long long>(len) - p.cu[seq + 1] + t;
        }
      } else {
        len = p.lens[seq];
        pos = static_cast<long long>(len) - 1;
      }
      // a row without a position: of an idle sequence if the length is 0, else of a length that cannot be
      if (pos < 0 && len != 0) report_bad_index(p.err, KID_APPEND, kSiteBadLength);
    }
    long long sk = -1, sv = -1;
    if (pos >= static_cast<long long>(p.max_pages) * p.page_size) {
      report_bad_index(p.err, KID_APPEND, kSiteBadLength);
    } else if (pos >= 0) {
      const int i = static_cast<int>(pos) / p.page_size, at = static_cast<int>(pos) % p.page_size;
      const int page = p.table[static_cast<long long>(seq) * p.max_pages + i];
      if (page < 0 || page >= p.pages) {
        report_bad_index(p.err, KID_APPEND, kSiteBadPage);
      } else {
        sk = page * p.kc.sp + at * p.kc.st;
        sv = page * p.vc.sp + at * p.vc.st;
      }
    }
    s_slot_k[threadIdx.x] = sk;
    s_slot_v[threadIdx.x] = sv;
    // (a position past 2^31 is reported above; it turns by the angle of the largest one)
    s_pos[threadIdx.x] = pos < 0 ? -1 : pos > 0x7fffffff ? 0x7fffffff : static_cast<int>(pos);
  }
  __syncthreads();
  for (int k = threadIdx.x; k < tok * kHalf; k += kAppendThreads) {
    const int tt = k / kHalf, i = k % kHalf, pos = s_pos[tt];
    if (pos < 0) continue;
    const unsigned long long turns = static_cast<unsigned long long>(pos) * p.turn[i];
    float sv, cv;
    sincospif(static_cast<float>(static_cast<int>(turns >> 32)) * 0x1p-31f, &sv, &cv);
    s_cos[tt][i] = cv;
    s_sin[tt][i] = sv;
  }
  __syncthreads();

  for (; w < units; w += step) {
    if (w >= step) load(w);
    const int part = kWide ? w / items : 0, item = w - part * items, sub = part * kAppendUnit;
    const int h = item / kChunks, c = item % kChunks;
    const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
    const int hh = is_q ? h : is_k ? h - p.Hq : h - p.Hq - p.Hkv;
    const long long col = static_cast<long long>(hh) * D + 8 * c;
#pragma unroll
    for (int i = 0; i < kAppendUnit; ++i) {
      const int tt = sub + i;
      if (s_pos[tt] < 0) continue;
      uint4 olo = lo[i], ohi = hi[i];
      if (is_q || is_k) {
        const __nv_bfloat162* l2 = reinterpret_cast<const __nv_bfloat162*>(&lo[i]);
        const __nv_bfloat162* h2 = reinterpret_cast<const __nv_bfloat162*>(&hi[i]);
        __nv_bfloat162* ol = reinterpret_cast<__nv_bfloat162*>(&olo);
        __nv_bfloat162* oh = reinterpret_cast<__nv_bfloat162*>(&ohi);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // fp32 rotation, one rounding to bf16
          const float2 a = __bfloat1622float2(l2[j]), b = __bfloat1622float2(h2[j]);
          const float2 cs = *reinterpret_cast<const float2*>(&s_cos[tt][8 * c + 2 * j]);
          const float2 sn = *reinterpret_cast<const float2*>(&s_sin[tt][8 * c + 2 * j]);
          ol[j] = __floats2bfloat162_rn(a.x * cs.x - b.x * sn.x, a.y * cs.y - b.y * sn.y);
          oh[j] = __floats2bfloat162_rn(b.x * cs.x + a.x * sn.x, b.y * cs.y + a.y * sn.y);
        }
      }
      auto store = [&](__nv_bfloat16* dst) {
        *reinterpret_cast<uint4*>(dst) = olo;
        *reinterpret_cast<uint4*>(dst + kHalf) = ohi;
      };
      if (is_q) {
        store(p.q_rot + (t_block + tt) * p.qr_st + col);
      } else if (is_k) {
        if (p.k_rot) store(p.k_rot + (t_block + tt) * p.kr_st + col);
        if (s_slot_k[tt] >= 0) store(p.kc.p + s_slot_k[tt] + col);
      } else if (s_slot_v[tt] >= 0) {
        store(p.vc.p + s_slot_v[tt] + col);
      }
    }
  }
  // (only now: blocks of the next kernel that are resident early crowd the SMs that are free first, 14.6
  // against 12.6 us for two batches of small heads in a row)
  pdl_launch_dependents();
}

}  // namespace s2

// Causal attention over packed prompts of different lengths (O and row log-sum-exp), sm_100a
// tensor cores.
//
// The sequences' rows follow one another in q, k, v [T, heads, D]; row i of a sequence sees its
// rows 0..i: o_i = sum_j p_ij v_j / l_i, p_ij = exp(scale q_i . k_j), l_i = sum_j p_ij, lse_i = log l_i.
// 4 D flops per visible (query head, row, key): bound by the tensor cores, and next to them by
// the exponentials (2 x 128 x 128 on 16 lanes a cycle are 2048 cycles per step of 256 rows x 128 keys,
// whose 32 MMAs take 2048 to 2750).
//
// A work unit is two 128-row query tiles that share their key/value tiles: the same rows of two
// query heads of one kv head where the group is even (both tiles then see the same keys), or 256
// consecutive rows of one head. Each CTA (one per SM) goes on to the next unit by cancelling the launch of
// a block that has not started yet (cluster launch control): units are balanced at run time, in
// the order of the grid, with no counter in memory. The order is by chunks of kv heads whose K and V
// fit L2 together, the heaviest query tiles of all sequences first in each chunk.
//
// Warp roles (384 threads):
//   warps 0-3, 4-7  softmax of query tile 0 / 1: thread i owns row i (TMEM lane i), fp32 online
//                   softmax, P written to TMEM as bf16 over S, epilogue.
//   warp 8          producer: next unit, TMA loads (Q tiles, K ring, V ring).
//   warps 9, 10     MMA issuer of query tile 0 / 1 (one lane): S_t(0), then PV_t(j), S_t(j + 1), ...
//   warp 11         looks through the value tiles that a query tile sees in part.
// TMEM columns: S0/P0 [0,128), S1/P1 [128,256), O0 [256,256+D), O1 [256+D, 256+2D).
//
// One tile's MMAs run beside the other tile's softmax. Each tile has an issuer of its own, so that neither
// waits for the other tile's P, and one's waits and descriptor arithmetic pass while the other's MMAs
// run (one issuer for both: 109 cycles per 128 x 128 x 16 MMA even with no softmax at all, against 64).
//
// Softmax pass: the exponentials are taken against a reference that need not be the maximum: the maximum
// of the row's first 16 scores. It only has to keep the sums inside fp32, where products and sums have the
// same relative precision at any scale, so no maximum is searched for as long as a tile's row sum stays
// below 2^30; else the pass is repeated from S, which is still in TMEM, against the maximum so far, and
// O and l are rescaled. The price is range: O's sums of weights up to 2^30 a tile times values stay finite for
// |v| < 2^98 / tiles (against the running maximum: 2^128 / keys).
//
// Measured, in a loop over three inputs: one prompt of 8192 tokens, 32 heads, d = 128: 0.556 ms, 0.99 PFLOP/s of visible
// work; 39k tokens in two prompts, 64 / 8 heads: 11.3 to 11.7 ms, 1.07 to 1.11; 12 prompts of 1 to 4999 tokens, 32 heads:
// 0.267 ms, 0.84; 64 prompts of 128 tokens, 32 heads: 49 us, 5.5 TB/s (there the loads' latency and the memory bound it,
// and what a short unit costs in sequence: 200 prompts of 40, 109 us).
// What bounds it: tensor pipe and exponential unit are each 55 % busy, counted in their own cycles. One tile's step is a
// chain, S product, pass, all of P stored, PV product, next S into the same columns, of some 3500 cycles, where the two
// tiles' products take 2048 to 2750 and their exponentials 2048. In a loop the GPU sits at its power cap besides (990 W,
// 1.7 GHz, 0.54 J a pass over the 8192 tokens; the MMAs alone, the same launch with the softmax left out, 0.36 J); a call
// on its own, which the cap does not reach, takes 0.50 ms. Scores are loaded 16
// columns at a time so that nothing spills (164 registers; 32 at a time: 4 % slower). Tried without gain: key
// tiles of 64 with two score buffers per query tile (N = 64 MMAs: 0.79 ms), a warpgroup of its own for the
// epilogue (128 registers a thread at launch spill the softmax: 0.79 ms), turns taken by the MMA issuers
// instead of the softmax (0.59 ms).
//
// Masked places hold anything. Keys are masked by selection. Values would reach a product as 0 * NaN: warp 11
// looks through the diagonal V tiles, which hold rows that some query rows do not see, and, where a sequence
// ends inside the tile (its last tile is always a diagonal one), rows behind it that none sees: infinities and
// NaN are replaced by zeros there, and in a unit whose own rows held some, a rare one, the warp adds them to the
// stored rows that do see them. (8192 tokens: no time; it has a step's time to look at 32 KB. Rows behind the
// end kept out by loads in boxes of 8 rows instead: a prompt of 40 tokens spent 4100 of its unit's 6100 cycles
// on their issue.)
#pragma once

#include "s2_common.cuh"
#include "s2_serve_common.cuh"
#include "s2_tmem_wide.cuh"

namespace s2 {

constexpr int kPromptMaxSeqs = 512;       // sequences and query tiles of one launch
constexpr int kPromptMaxTiles = 2048;
constexpr int kPromptKeys = 128;          // keys of a K/V tile

struct PromptParams {
  const __nv_bfloat16* v;
  long long v_st;
  __nv_bfloat16* o;
  long long o_st;
  float* lse;                             // [Hq, T]
  int T, Hq, Hkv, group;
  int n_tiles, kv_chunk;                  // entries of `tile`; kv heads taken together
  float scale_log2;
  unsigned int* err;
  unsigned long long timeout_ns;
};
// What the host lays out for one launch: the sequences, and their query tiles (128 or 256 rows), the
// heaviest first: sequence << 16 | tile.
struct PromptWork {
  int start[kPromptMaxSeqs], len[kPromptMaxSeqs];
  unsigned int tile[kPromptMaxTiles];
};

// A tile's row sum above which its pass is repeated against the tile's own maximum. (2^12 in its place would leave
// values 2^18 more room: 8192 tokens, 32 heads, scores of 1, 2, 4, 8 times unit variance: 472, 480 to 544, 1004 to
// 1067, 998 us against 472, 503 to 522, 540 to 550, 832 to 846.)
constexpr float kPromptMaxSum = 1073741824.f;   // 2^30

// One unit as the roles read it from the ring.
struct PromptUnit {
  int live;                               // 0: no unit is left
  int kvh, h[2];
  int start, len;                         // the sequence's rows
  int qt[2], n[2];                        // query tile of 128 rows, and its key tiles (0: no such tile)
};

template <int D>
struct PromptLayout {
  static constexpr uint32_t kTile = Tile<D>::kBytes;
  static constexpr int kStages = 2;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + 2 * kTile;
  static constexpr uint32_t kV = kK + kStages * kTile;
  static constexpr uint32_t kStageWarp = 32 * 128;          // O staging: 32 rows x 64 columns
  static constexpr uint32_t kStage = kV + kStages * kTile;
  static constexpr uint32_t kClc = kStage + 8 * kStageWarp; // response of the launch control, 16 bytes
  static constexpr uint32_t kRing = kClc + 16;
  static constexpr uint32_t kBad = kRing + kUnitRing * sizeof(PromptUnit);   // units' diagonal tiles
  enum { B_Q = 0, B_QE = 2, B_K = 4, B_KE = B_K + kStages, B_V = B_KE + kStages, B_VE = B_V + kStages,
         B_S = B_VE + kStages, B_P = B_S + 2, B_ODONE = B_P + 2, B_UF = B_ODONE + 2,
         B_UE = B_UF + kUnitRing, B_CLC = B_UE + kUnitRing, B_DRAIN, B_TURN = B_DRAIN + 2,
         B_VC = B_TURN + 2, B_BAD = B_VC + kStages,
         B_FIX = B_BAD + kUnitRing, B_COUNT = B_FIX + 2 };
  static constexpr uint32_t kBar = (kBad + kUnitRing * 4 + 7) / 8 * 8;
  static constexpr uint32_t kTmemSlot = kBar + B_COUNT * 8;
  static constexpr uint32_t kAbort = kTmemSlot + 4;
  static constexpr uint32_t kBytes = kAbort + 4;
  // (at least 116 KB, so that one CTA is resident per SM: each takes all of TMEM)
  static constexpr uint32_t kLaunchBytes = kBytes + 1024 > 116 * 1024 ? kBytes + 1024 : 116 * 1024;
  static constexpr int kThreads = 384;
  static_assert(kLaunchBytes <= 227 * 1024, "shared memory of one CTA");
};

// Cluster launch control: ask for a block that has not started; 16 bytes arrive at `dst`, counted on
// `bar`. After an answer without a block no further request may follow.
__device__ __forceinline__ void clc_request(uint32_t dst, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
      "r"(bar)
      : "memory");
}
// The block's x index, or -1.
__device__ __forceinline__ int clc_answer(uint32_t src) {
  int x, got;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 a, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.s32 %1, 1, 0, p;\n\t"
      "mov.s32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, a;\n\t}"
      : "=r"(x), "=r"(got)
      : "r"(src)
      : "memory");
  return got ? x : -1;
}

// kHeads: the unit's two tiles are two heads' same rows (else 256 rows of one head).
template <bool kHeads>
__device__ __forceinline__ PromptUnit prompt_unit(const PromptParams& p, const PromptWork& w, int u) {
  const int per_kv = kHeads ? p.group / 2 : p.group;
  const int full = p.kv_chunk * per_kv * p.n_tiles;
  const int kv0 = u / full * p.kv_chunk;
  const int in = u % full, here = min(p.kv_chunk, p.Hkv - kv0) * per_kv;
  const int head = in % here;
  const unsigned int e = w.tile[in / here];
  PromptUnit r;
  r.live = 1;
  r.kvh = kv0 + head / per_kv;
  const int h0 = r.kvh * p.group + (head % per_kv) * (kHeads ? 2 : 1);
  r.h[0] = h0;
  r.h[1] = kHeads ? h0 + 1 : h0;
  r.start = w.start[e >> 16];
  r.len = w.len[e >> 16];
  const int t = static_cast<int>(e & 0xFFFFu);
  r.qt[0] = kHeads ? t : 2 * t;
  r.qt[1] = kHeads ? t : 2 * t + 1;
  r.n[0] = r.qt[0] + 1;
  r.n[1] = r.qt[1] * kTileRows < r.len ? r.qt[1] + 1 : 0;
  return r;
}

// The not finite halves of a bf16 pair: bits 15 and 31; and the pair with zeros in their place.
__device__ __forceinline__ uint32_t bf16x2_not_finite(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t bf16x2_finite_part(uint32_t w) {
  const uint32_t x = bf16x2_not_finite(w);
  return w & ~((x & 0x80000000u ? 0xffff0000u : 0u) | (x & 0x8000u ? 0xffffu : 0u));
}

// Adds to the stored rows of O of query tile t the infinities and NaN of the value rows they see in the unit's
// diagonal tiles that were found to hold some (weights are positive: inf stays inf). One warp: a lane has D / 32
// columns (pairs 64 apart), whose sum over the value rows runs along with the query rows, eight rows' loads in
// flight. Two full tiles take some 40 us more, however many values are not finite (8192 tokens, 32 heads, nothing
// but NaN: 0.84 ms, 0.50 with finite values).
template <int D>
__device__ __noinline__ void prompt_add_not_finite(const PromptParams& p, const PromptUnit& u, int bad, int t, int lane) {
  constexpr int kPer = D / 32, kWords = kPer / 2, kAhead = 8;
  float sum[kPer] = {};
  auto add = [&](uint32_t w, int i) {                // the pair i of a value row
    const uint32_t x = bf16x2_not_finite(w);
    if (x & 0x8000u) sum[2 * i] += __uint_as_float(w << 16);
    if (x & 0x80000000u) sum[2 * i + 1] += __uint_as_float(w & 0xffff0000u);
  };
  const uint32_t* v = reinterpret_cast<const uint32_t*>(p.v + u.start * p.v_st + static_cast<long long>(u.kvh) * D) +
                      lane;
  uint32_t* o = reinterpret_cast<uint32_t*>(p.o + u.start * p.o_st + static_cast<long long>(u.h[t]) * D) + lane;
  const long long v_st = p.v_st / 2, o_st = p.o_st / 2;
  // an earlier tile than its own is seen by all of its rows
  const int x = t ^ 1;
  if (((bad >> x) & 1) && u.n[x] < u.n[t]) {
    const int first = (u.n[x] - 1) * kTileRows;
    for (int r = 0; r < kTileRows; r += kAhead) {
      uint32_t w[kAhead][kWords];
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[a][i] = v[(first + r + a) * v_st + 32 * i];
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
#pragma unroll
        for (int i = 0; i < kWords; ++i) add(w[a][i], i);
    }
  }
  const bool own = (bad >> t) & 1;
  const int first = u.qt[t] * kTileRows, left = min(kTileRows, u.len - first);
  for (int r = 0; r < left; r += kAhead) {
    uint32_t w[kAhead][kWords], y[kAhead][kWords];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const bool in = r + a < left;
        w[a][i] = in && own ? v[(first + r + a) * v_st + 32 * i] : 0u;
        y[a][i] = in ? __ldcg(o + (first + r + a) * o_st + 32 * i) : 0u;
      }
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        add(w[a][i], i);
        const float s0 = sum[2 * i], s1 = sum[2 * i + 1];
        if (r + a >= left || (s0 == 0.f && s1 == 0.f)) continue;
        const uint32_t z = pack_bf16(__uint_as_float(y[a][i] << 16) + s0, __uint_as_float(y[a][i] & 0xffff0000u) + s1);
        o[(first + r + a) * o_st + 32 * i] =
            (s0 == 0.f ? y[a][i] & 0xffffu : z & 0xffffu) | (s1 == 0.f ? y[a][i] & 0xffff0000u : z & 0xffff0000u);
      }
  }
}

// Tensor memory loads whose results may be used after tmem_ld_done.
#define S2_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), \
                 "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
__device__ __forceinline__ void tmem_ld16_begin(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : S2_R8(0), S2_R8(8)
      : "r"(taddr)
      : "memory");
}
#undef S2_R8
#define S2_U8(i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), \
                 "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void tmem_ld_done(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : S2_U8(0), S2_U8(8)::"memory");
}
#undef S2_U8

// 16 scores of a row: P = exp2(c s - m) as bf16 pairs into pk, the sums into acc. Scores behind column
// `lim` are masked. P is rounded to the tensor cores' 8 bits, as in the training forward (the sums are of the fp32
// values): output error against 64 bits 0.0020, with fp32 weights it would be that of its own rounding, 0.0016.
template <bool kMask>
__device__ __forceinline__ void softmax16(const uint32_t (&r)[16], int lim, uint64_t c2, uint64_t nm2,
                                          uint32_t* pk, uint64_t (&acc)[2]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float s0 = __uint_as_float(r[2 * i]), s1 = __uint_as_float(r[2 * i + 1]);
    if (kMask) {
      s0 = 2 * i > lim ? -INFINITY : s0;
      s1 = 2 * i + 1 > lim ? -INFINITY : s1;
    }
    const uint64_t a = f2_fma(f2_pack(s0, s1), c2, nm2);
    const float e0 = fast_exp2(f2_lo(a)), e1 = fast_exp2(f2_hi(a));
    acc[i & 1] = f2_add(acc[i & 1], f2_pack(e0, e1));
    pk[i] = pack_bf16(e0, e1);
  }
}
// The pass over a row's 128 scores, 16 at a time, the next 16 on their way; the first ones are in `a`.
template <bool kMask>
__device__ __forceinline__ void softmax_row(uint32_t s_col, uint32_t (&a)[16], uint32_t (&b)[16], int lim, uint64_t c2,
                                            uint64_t nm2, uint32_t (&pk)[64], uint64_t (&acc)[2]) {
#pragma unroll
  for (int q = 0; q < 8; q += 2) {
    tmem_ld16_begin(s_col + 16 * q + 16, b);
    softmax16<kMask>(a, lim - 16 * q, c2, nm2, pk + 8 * q, acc);
    tmem_ld_done(b);
    if (q < 6) tmem_ld16_begin(s_col + 16 * q + 32, a);
    softmax16<kMask>(b, lim - 16 * q - 16, c2, nm2, pk + 8 * q + 8, acc);
    if (q < 6) tmem_ld_done(a);
  }
}

template <int D, bool kHeads>
__global__ void __launch_bounds__(384, 1)
    s2_prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO8,
                     const __grid_constant__ PromptParams p, const __grid_constant__ PromptWork work) {
  using L = PromptLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = aligned_smem(smem_raw);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto bar = [&](int i) { return sbase + L::kBar + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);
  PromptUnit* ring = reinterpret_cast<PromptUnit*>(smem + L::kRing);
  volatile int* bad_tiles = reinterpret_cast<volatile int*>(smem + L::kBad);
  const WaitCtx ctx{abort_flag, p.err, p.timeout_ns, KID_PROMPT};

  if (warp == 8 && lane == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(L::B_Q + s), 1);
      mbar_init(bar(L::B_QE + s), 1);
      mbar_init(bar(L::B_S + s), 1);
      mbar_init(bar(L::B_P + s), 4);
      mbar_init(bar(L::B_ODONE + s), 1);
    }
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(L::B_K + s), 1);
      mbar_init(bar(L::B_KE + s), 2);     // both issuers
      mbar_init(bar(L::B_V + s), 1);
      mbar_init(bar(L::B_VE + s), 3);     // ... and warp 11
      mbar_init(bar(L::B_VC + s), 1);
    }
    for (int s = 0; s < kUnitRing; ++s) {
      mbar_init(bar(L::B_UF + s), 1);
      mbar_init(bar(L::B_UE + s), 11);    // the eight softmax warps, the two issuers and warp 11
      mbar_init(bar(L::B_BAD + s), 1);
    }
    mbar_init(bar(L::B_CLC), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(L::B_TURN + s), 4);
      mbar_init(bar(L::B_FIX + s), 4);
      mbar_init(bar(L::B_DRAIN + s), 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
    tma_prefetch_map(&tmO8);
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();                             // (after the set-up, which touches no memory of the caller's)
  const uint32_t tmem = *tmem_slot;

  // The k-th unit of this CTA, for a whole warp or one thread.
  auto read_rec = [&](int k, PromptUnit& u, bool whole_warp, uint32_t site) -> bool {
    const int slot = k % kUnitRing;
    bool ok = wait_bar(bar(L::B_UF + slot), (k / kUnitRing) & 1, ctx, site);
    if (whole_warp) ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    u = ring[slot];
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(bar(L::B_UE + slot));
    return u.live != 0;
  };

  if (warp == 8) {
    // ---------------- producer (the whole warp; lane 0 issues) ----------------
    int k_issued = 0, v_issued = 0, q_loads[2] = {0, 0};
    int clc_asked = -1;                   // the last request's number
    bool ok = true, clc_open = false;
    PromptUnit u = prompt_unit<kHeads>(p, work, blockIdx.x);
    // A unit of one tile only (a prompt's odd last rows; each unit of prompts of up to 128 tokens) goes to the
    // tile that the unit before left free, so that two such units are on their way at a time: 200 prompts of
    // 40 tokens, 32 heads, 109 against 162 us.
    int last = -1;                        // the tile that the last unit had to itself
    auto place = [&]() {
      if (kHeads || u.n[1] != 0) {
        last = -1;
        return;
      }
      last = last == 0 ? 1 : 0;
      if (last == 1) {
        u.n[1] = u.n[0];
        u.qt[1] = u.qt[0];
        u.n[0] = 0;
      }
    };
    place();
    auto load_box = [&](uint32_t dst, const CUtensorMap* m, int b, int h, int row) {
      if (lane == 0) {
        mbar_expect_tx(bar(b), Tile<D>::kBytes);
#pragma unroll
        for (int half = 0; half < Tile<D>::kHalves; ++half)
          tma_load_4d(dst + half * Tile<D>::kHalfBytes, m, bar(b), half * 64, h, row, 0);
      }
      __syncwarp();
    };
    auto issue_k = [&](int j) -> bool {
      const int i = k_issued, st = i % L::kStages;
      if (i >= L::kStages && !warp_wait(bar(L::B_KE + st), ((i / L::kStages) - 1) & 1, ctx, 1)) return false;
      load_box(sbase + L::kK + st * L::kTile, &tmK, L::B_K + st, u.kvh, u.start + j * kTileRows);
      ++k_issued;
      return true;
    };
    auto issue_v = [&](int j) -> bool {
      const int i = v_issued, st = i % L::kStages;
      if (i >= L::kStages && !warp_wait(bar(L::B_VE + st), ((i / L::kStages) - 1) & 1, ctx, 2)) return false;
      const uint32_t dst = sbase + L::kV + st * L::kTile;
      load_box(dst, &tmV, L::B_V + st, u.kvh, u.start + j * kTileRows);
      ++v_issued;
      return true;
    };
    auto publish = [&](int k) -> bool {
      const int slot = k % kUnitRing;
      if (k >= kUnitRing && !warp_wait(bar(L::B_UE + slot), ((k / kUnitRing) - 1) & 1, ctx, 3)) return false;
      if (lane == 0) {
        ring[slot] = u;
        mbar_arrive(bar(L::B_UF + slot));
      }
      __syncwarp();
      return true;
    };
    ok = publish(0);
    for (int k = 0; ok && u.live; ++k) {
      const int n = max(u.n[0], u.n[1]);
      ok = issue_k(0);
      for (int t = 0; ok && t < 2; ++t) {
        if (u.n[t] == 0) continue;
        if (q_loads[t] > 0 && !warp_wait(bar(L::B_QE + t), (q_loads[t] - 1) & 1, ctx, 4)) {
          ok = false;
          break;
        }
        load_box(sbase + L::kQ + t * L::kTile, &tmQ, L::B_Q + t, u.h[t], u.start + u.qt[t] * kTileRows);
        ++q_loads[t];
      }
      for (int j = 0; ok && j < n; ++j) {
        if (j + 2 >= n && clc_asked < k) {
          // Ask for the next unit while the last two tiles are still to come: late, so that the units
          // left go to the CTAs that are done first.
          if (lane == 0) {
            mbar_expect_tx(bar(L::B_CLC), 16);
            clc_request(sbase + L::kClc, bar(L::B_CLC));
          }
          clc_asked = k;
          clc_open = true;
          __syncwarp();
        }
        if (j + 1 < n) ok = issue_k(j + 1);
        if (ok) ok = issue_v(j);
      }
      if (!ok || !warp_wait(bar(L::B_CLC), k & 1, ctx, 5)) {
        ok = false;
        break;
      }
      clc_open = false;
      const int next = clc_answer(sbase + L::kClc);
      __syncwarp();
      fence_async_smem();                 // read before the next request may write
      if (next >= 0) {
        u = prompt_unit<kHeads>(p, work, next);
        place();
      } else {
        u.live = 0;
      }
      ok = publish(k + 1);
    }
    // Every issued copy lands before the CTA can exit.
    for (int t = 0; t < 2; ++t)
      if (q_loads[t] > 0) drain_wait(bar(L::B_Q + t), (q_loads[t] - 1) & 1, p.timeout_ns);
    for (int i = k_issued - L::kStages; i < k_issued; ++i)
      if (i >= 0) drain_wait(bar(L::B_K + i % L::kStages), (i / L::kStages) & 1, p.timeout_ns);
    for (int i = v_issued - L::kStages; i < v_issued; ++i)
      if (i >= 0) drain_wait(bar(L::B_V + i % L::kStages), (i / L::kStages) & 1, p.timeout_ns);
    if (clc_open) drain_wait(bar(L::B_CLC), clc_asked & 1, p.timeout_ns);
  } else if (warp == 11) {
    // ---------------- the diagonal value tiles ----------------
    int v_seen = 0, fixed[2] = {0, 0};    // V tiles, and units mended, so far
    bool ok = true;
    for (int ku = 0; ok; ++ku) {
      PromptUnit u;
      if (!read_rec(ku, u, true, 16)) break;
      int bad = 0;                        // bit t: query tile t's diagonal tile holds infinities or NaN
      const int n = max(u.n[0], u.n[1]);
      for (int j = 0; j < n; ++j, ++v_seen) {
        // (it waits for every tile and releases it too, so that it never falls a phase behind)
        const int st = v_seen % L::kStages;
        if (!warp_wait(bar(L::B_V + st), (v_seen / L::kStages) & 1, ctx, 17)) { ok = false; break; }
        const int diag = (j + 1 == u.n[0] ? 1 : 0) | (j + 1 == u.n[1] ? 2 : 0);
        if (diag) {
          uint4* tile = reinterpret_cast<uint4*>(smem + L::kV + st * L::kTile);
          // 0 * x summed over the tile: NaN if some x is infinite or NaN. Only then a closer look.
          const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
          __nv_bfloat162 sum[4] = {zero, zero, zero, zero};
#pragma unroll 8
          for (int x = lane; x < static_cast<int>(L::kTile / 16); x += 32) {
            uint4 w = tile[x];
            sum[0] = __hfma2(reinterpret_cast<__nv_bfloat162&>(w.x), zero, sum[0]);
            sum[1] = __hfma2(reinterpret_cast<__nv_bfloat162&>(w.y), zero, sum[1]);
            sum[2] = __hfma2(reinterpret_cast<__nv_bfloat162&>(w.z), zero, sum[2]);
            sum[3] = __hfma2(reinterpret_cast<__nv_bfloat162&>(w.w), zero, sum[3]);
          }
          const float2 found = __bfloat1622float2(__hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3])));
          if (__any_sync(0xffffffffu, !(found.x + found.y == 0.f))) {
            const int valid = u.len - j * kTileRows;   // rows of the sequence in the tile
            uint32_t seen = 0;
            for (int x = lane; x < static_cast<int>(L::kTile / 16); x += 32) {
              const uint4 w = tile[x];
              if (x / 8 % kTileRows < valid)
                seen |= bf16x2_not_finite(w.x) | bf16x2_not_finite(w.y) | bf16x2_not_finite(w.z) | bf16x2_not_finite(w.w);
              tile[x] = make_uint4(bf16x2_finite_part(w.x), bf16x2_finite_part(w.y), bf16x2_finite_part(w.z),
                                   bf16x2_finite_part(w.w));
            }
            if (__any_sync(0xffffffffu, seen != 0)) bad |= diag;
            fence_async_smem();           // the MMAs read the tile through the async proxy
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::B_VC + st));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::B_VE + st));
      }
      if (!ok) break;
      if (lane == 0) {
        bad_tiles[ku % kUnitRing] = bad;
        mbar_arrive(bar(L::B_BAD + ku % kUnitRing));
      }
      __syncwarp();
      for (int t = 0; bad && t < 2; ++t) {           // the rare unit: once its rows are stored
        if (u.n[t] == 0) continue;
        if (!warp_wait(bar(L::B_FIX + t), fixed[t]++ & 1, ctx, 20)) { ok = false; break; }
        prompt_add_not_finite<D>(p, u, bad, t, lane);
      }
    }
  } else if (warp == 9 || warp == 10) {
    // ---------------- MMA issuers ----------------
    const int t = warp - 9;
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16(128, D, false, true);
      const uint32_t s_tmem = tmem + t * 128, o_tmem = tmem + 256 + t * D, q_smem = sbase + L::kQ + t * L::kTile;
      int k0 = 0, q_used = 0, p_used = 0;  // K/V tiles before this unit; query and P tiles used
      int checked[L::kStages] = {};        // tiles of each V slot that warp 11 has looked through
      bool ok = true;
      auto wait_tile = [&](int full0, int i, uint32_t site) {
        return wait_bar(bar(full0 + i % L::kStages), (i / L::kStages) & 1, ctx, site);
      };
      for (int ku = 0; ok; ++ku) {
        PromptUnit u;
        if (!read_rec(ku, u, false, 6)) break;
        const int n = max(u.n[0], u.n[1]), mine = u.n[t];
        // S = Q K(j)^T into this tile's columns
        auto issue_s = [&](int j) -> bool {
          if (!wait_tile(L::B_K, k0 + j, 7)) return false;
          tc_fence_after();
          gemm_ss_k<D>(s_tmem, q_smem, sbase + L::kK + ((k0 + j) % L::kStages) * L::kTile, idesc_qk);
          mma_commit(bar(L::B_S + t));
          mma_commit(bar(L::B_KE + (k0 + j) % L::kStages));
          if (j + 1 == mine) mma_commit(bar(L::B_QE + t));   // last S on this query tile
          return true;
        };
        // V(j) is there, and, if it is a query tile's diagonal one, has been looked through.
        auto wait_v = [&](int j) -> bool {
          const int st = (k0 + j) % L::kStages;
          if (!wait_tile(L::B_V, k0 + j, 10)) return false;
          if (j + 1 != u.n[0] && j + 1 != u.n[1]) return true;
          int k = 0;
#pragma unroll
          for (int x = 0; x < L::kStages; ++x)
            if (x == st) k = checked[x]++;
          return wait_bar(bar(L::B_VC + st), k & 1, ctx, 18);
        };
        if (mine > 0) ok = wait_bar(bar(L::B_Q + t), q_used++ & 1, ctx, 8) && issue_s(0);
        for (int j = 0; ok && j < n; ++j) {
          const int vi = k0 + j, vst = vi % L::kStages;
          if (j >= mine) {
            // The tile does not see these keys: they are released once they are there (a release ahead
            // of the load would count for the slot's last tile).
            if (!wait_tile(L::B_K, vi, 7) || !wait_v(j)) { ok = false; break; }
            mbar_arrive(bar(L::B_KE + vst));
            mbar_arrive(bar(L::B_VE + vst));
            continue;
          }
          if (!wait_v(j)) { ok = false; break; }
          if (!wait_bar(bar(L::B_P + t), p_used++ & 1, ctx, 9)) { ok = false; break; }
          tc_fence_after();
          gemm_ts_mn<D>(o_tmem, s_tmem, sbase + L::kV + vst * L::kTile, idesc_pv, j > 0);
          if (j + 1 == mine) mma_commit(bar(L::B_ODONE + t));
          mma_commit(bar(L::B_VE + vst));                    // V(j) has been read by this tile
          if (j + 1 < mine && !issue_s(j + 1)) { ok = false; break; }
        }
        k0 += n;
      }
    }
  } else {
    // ---------------- softmax warps ----------------
    const int wg = warp / 4;
    const int row = threadIdx.x % 128;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
    const uint32_t s_col = t_lane + wg * 128;
    const uint32_t o_col = t_lane + 256 + wg * D;
    const float c = p.scale_log2;
    const uint64_t c2 = f2_pack(c, c);
    int s_cnt = 0, o_cnt = 0, turn = 0;
    bool ok = true;
    for (int ku = 0; ok; ++ku) {
      // Of the unit only its tile counts are held through the passes (registers); the rest is read in the
      // epilogue, and the ring's slot released after it.
      const int slot = ku % kUnitRing;
      if (!warp_wait(bar(L::B_UF + slot), (ku / kUnitRing) & 1, ctx, 11) || !ring[slot].live) break;
      const int n = ring[slot].n[wg], n_other = ring[slot].n[wg ^ 1];
      const bool turns = kHeads || (n != 0 && n_other != 0);     // a unit of one tile only takes none
      const int n_all = turns ? max(n, n_other) : n;
      float m_run = -INFINITY, l_run = 0.f;
      // The two tiles' passes take turns (tile 0's pass k, tile 1's pass k, tile 0's k + 1, ...): each then
      // has the exponential units to itself while the other tile's MMAs run. Left alone, both warpgroups
      // fall into step, and their MMAs too: 666 against 549 us on one 8192-token prompt of 32 heads.
      auto my_turn = [&]() -> bool {
        if (!turns) return true;
        const int k = wg == 0 ? turn - 1 : turn;     // the other tile's pass that has to be over
        ++turn;
        return k < 0 || warp_wait(bar(L::B_TURN + (wg ^ 1)), k & 1, ctx, 15);
      };
      auto pass_turn = [&]() {
        __syncwarp();
        if (turns && lane == 0) mbar_arrive(bar(L::B_TURN + wg));
      };
      for (int j = 0; j < n_all; ++j) {
        if (j >= n) {                                // no pass of this tile here
          if (!my_turn()) { ok = false; break; }
          pass_turn();
          continue;
        }
        if (!warp_wait(bar(L::B_S + wg), s_cnt & 1, ctx, 12)) { ok = false; break; }
        ++s_cnt;
        if (!my_turn()) { ok = false; break; }
        tc_fence_after();
        uint32_t pk[64];
        uint64_t acc[2] = {0, 0};
        bool need;
        {
          uint32_t a[16], b[16];
          const bool diag = j + 1 == n;              // the last tile is the diagonal one
          tmem_ld16_begin(s_col, a);
          tmem_ld_done(a);
          if (j == 0) {                              // a first reference, the maximum of 16 scores
            float m0 = -INFINITY, m1 = -INFINITY;
            const int lim = diag ? row : kTileRows;
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              m0 = max3f(m0, i > lim ? -INFINITY : __uint_as_float(a[i]), i + 1 > lim ? -INFINITY : __uint_as_float(a[i + 1]));
              m1 = max3f(m1, i + 2 > lim ? -INFINITY : __uint_as_float(a[i + 2]), i + 3 > lim ? -INFINITY : __uint_as_float(a[i + 3]));
            }
            m_run = fmaxf(m0, m1) * c;
          }
          const uint64_t nm2 = f2_pack(-m_run, -m_run);
          if (diag) softmax_row<true>(s_col, a, b, row, c2, nm2, pk, acc);
          else softmax_row<false>(s_col, a, b, 0, c2, nm2, pk, acc);
          // (also where it is infinite or NaN)
          const uint64_t both = f2_add(acc[0], acc[1]);
          need = !(f2_lo(both) + f2_hi(both) <= kPromptMaxSum);
        }
        if (__any_sync(0xffffffffu, need)) {
          const int lim = j + 1 == n ? row : kTileRows;
          float mx = -INFINITY;
          uint32_t a[16], b[16];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            tmem_ld16_begin(s_col + 16 * q, a);
            tmem_ld_done(a);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float s0 = 16 * q + i > lim ? -INFINITY : __uint_as_float(a[i]);
              const float s1 = 16 * q + i + 1 > lim ? -INFINITY : __uint_as_float(a[i + 1]);
              mx = max3f(mx, s0, s1);
            }
          }
          // (the warp's other rows keep their reference, and so their bits)
          const float m_cand = need ? fmaxf(m_run, mx * c) : m_run;
          if (__any_sync(0xffffffffu, m_cand != m_run)) {
            // 0 when m_run = -inf; 1 for a row whose scores are all -inf so far
            const float alpha = m_cand == -INFINITY ? 1.f : fast_exp2(m_run - m_cand);
            if (j > 0) {
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                uint32_t ov[32];
                tmem_ld32(o_col + 32 * q, ov);
#pragma unroll
                for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                tmem_st32(o_col + 32 * q, ov);
              }
            }
            l_run *= alpha;
            m_run = m_cand;
          }
          const float m_use = m_run == -INFINITY ? 0.f : m_run;
          const uint64_t nm2 = f2_pack(-m_use, -m_use);
          acc[0] = acc[1] = 0;
          tmem_ld16_begin(s_col, a);
          tmem_ld_done(a);
          softmax_row<true>(s_col, a, b, lim, c2, nm2, pk, acc);
        }
        pass_turn();
        tmem_st32(s_col, *reinterpret_cast<uint32_t(*)[32]>(pk));
        tmem_st32(s_col + 32, *reinterpret_cast<uint32_t(*)[32]>(pk + 32));
        acc[0] = f2_add(acc[0], acc[1]);
        l_run += f2_lo(acc[0]) + f2_hi(acc[0]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::B_P + wg));
      }
      if (n == 0) {
        if (lane == 0) mbar_arrive(bar(L::B_UE + slot));
        continue;
      }
      if (!ok || !warp_wait(bar(L::B_ODONE + wg), o_cnt & 1, ctx, 13)) { ok = false; break; }
      ++o_cnt;
      tc_fence_after();
      // Epilogue: O / l in bf16 through this warp's staging area (128-byte-swizzled rows of 64
      // columns): atoms of 8 rows inside the sequence go out as TMA boxes, the rows of the atom that
      // the sequence's end cuts as row stores, and rows behind the end not at all.
      const PromptUnit u = ring[slot];
      const float inv_l = 1.f / l_run;
      uint8_t* stage = smem + L::kStage + warp * L::kStageWarp;
      const uint32_t stage_s = sbase + L::kStage + warp * L::kStageWarp;
      const int r_warp = u.qt[wg] * kTileRows + (warp % 4) * 32;
      const int left = u.len - r_warp;               // rows of this warp inside the sequence
      const int tok = u.start + r_warp;
#pragma unroll 1
      for (int half = 0; half < D / 64; ++half) {
        uint32_t w[32];
#pragma unroll
        for (int q2 = 0; q2 < 2; ++q2) {
          uint32_t ov[32];
          tmem_ld32(o_col + 64 * half + 32 * q2, ov);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[16 * q2 + i] = pack_bf16(__uint_as_float(ov[2 * i]) * inv_l, __uint_as_float(ov[2 * i + 1]) * inv_l);
        }
        if (lane == 0) bulk_wait_read_all();         // the boxes sent before have been read out
        __syncwarp();
#pragma unroll
        for (int chunk = 0; chunk < 8; ++chunk)
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((chunk ^ (lane & 7)) * 16)) =
              make_uint4(w[4 * chunk], w[4 * chunk + 1], w[4 * chunk + 2], w[4 * chunk + 3]);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int a = 0; a < 4; ++a)
            if (8 * a + 8 <= left) tma_store_4d(&tmO8, stage_s + a * 1024, 64 * half, u.h[wg], tok + 8 * a, 0);
          bulk_commit();
        }
        if (left > 0 && left < 32 && (left & 7) != 0) {
          const int rr0 = left & ~7;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int rr = rr0 + 4 * i + (lane >> 3), chunk = lane & 7;
            if (rr < left)
              *reinterpret_cast<uint4*>(p.o + (tok + rr) * p.o_st + static_cast<long long>(u.h[wg]) * D + 64 * half +
                                        8 * chunk) =
                  *reinterpret_cast<const uint4*>(stage + rr * 128 + ((chunk ^ (rr & 7)) * 16));
          }
        }
        __syncwarp();
      }
      if (lane < left)
        p.lse[static_cast<long long>(u.h[wg]) * p.T + tok + lane] = (m_run + log2f(l_run)) * 0.6931471805599453f;
      if (!warp_wait(bar(L::B_BAD + slot), (ku / kUnitRing) & 1, ctx, 19)) { ok = false; break; }
      if (bad_tiles[slot] != 0) {                    // warp 11 has to see the warp's stored rows
        if (lane == 0) {
          bulk_wait_all();
          asm volatile("fence.proxy.async;" ::: "memory");
        }
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::B_FIX + wg));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::B_UE + slot));
      tc_fence_before();                  // O is read: the next PV on it waits for this warp's P
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  // ---------------- teardown ----------------
  if (warp == 9 || warp == 10) {          // each issuer's MMAs are done (a commit covers its own thread's)
    if (lane == 0) {
      mma_commit(bar(L::B_DRAIN + warp - 9));
      drain_wait(bar(L::B_DRAIN + warp - 9), 0, p.timeout_ns);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace s2

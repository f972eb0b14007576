// Attention of one new token per sequence over a paged key/value cache.
//
// For sequence b with n = lens[b] cached tokens, query head h and its key/value head g = h / (Hq /
// Hkv): s_j = scale * q_h . k_{j,g}, o_h = sum_j exp(s_j) v_{j,g} / sum_j exp(s_j), lse_h = log
// sum_j exp(s_j), j < n. Every cache row is read once for all heads of its group, so the bytes of
// K and V bound the kernel: two multiply-adds per element and query head.
//
// Split over the length: the batch is one list of 16-token tiles, sequence by sequence and inside
// it head by head (a segment is one (sequence, head) pair's tiles, with kDecodeGap empty places
// before them for what a segment's start and end cost). The list is cut into equal contiguous
// ranges, one per CTA and in it one per warp, whatever the lengths are, so a ragged batch and a
// single long sequence load every SM alike. The lengths are read on the device: one launch, and a
// captured graph, serves every length. A segment inside one warp's range is finished by that warp.
// The pieces (running maximum, sum and unnormalised output in fp32) of the others are joined first
// inside the CTA, through shared memory; of the segments that cross CTAs, at most two a CTA, the
// partial results go to the workspace, and a second small kernel, one block per CTA boundary and
// query row, joins them. Pieces are always added in the list's order, with no atomics: the same
// bits every time.
// Where the block table holds few tokens a sequence and there are no more segments than SMs, each CTA
// takes a whole segment instead and the second kernel falls away.
//
// A warp is on its own: it copies its tiles' rows to its part of shared memory with 16-byte
// asynchronous copies (the row's page looked up one tile ahead), three tiles deep at D = 128 and six
// at 64, across segment boundaries, and there is no barrier between warps. Copies of single rows take
// any page size and any stride. The products run on mma.sync (16 query rows x 8 keys x 16): at 6.5
// TB/s the products of 16 padded rows need about 100 TFLOP/s, far below what it reaches, and the
// fragment of the scores is the fragment of P in the second product, in registers. Scores, maxima,
// sums and outputs are fp32; P is rounded to bf16 for the tensor cores, to twice bf16 where the MMA's
// rows have room (8 query rows and less: output error against 64 bits 0.0017, that of its own rounding; with
// 16 rows 0.0023).
//
// Measured: 16 sequences of about 8k tokens, 32 kv heads, 2.0 GB: 312 to 318 us, 6.4 to 6.5 TB/s (of measured
// copy bandwidth: 0.97 to 0.99). One sequence of 102400 tokens, 8 kv heads, 419 MB: 73 us; the stream itself
// runs at 7.3 TB/s, 2 us pass before the first copy is on its way, 3 before it is there, 4 at the ranges'
// uneven ends and joins and 5 in the second kernel. 64 sequences of 1 to 32768 tokens, 662 MB: 110 to 114 us.
// Tried: 12 warps two tiles deep and K and V copied in groups of their own (not faster), wider L2 fetches
// (no change), a dry round at the start to warm the instruction caches (3 us slower).
#pragma once

#include "s2_device.cuh"
#include "s2_serve_common.cuh"

namespace s2 {

constexpr int kDecodeWarps = 8;
constexpr int kDecodeThreads = 32 * kDecodeWarps;
constexpr int kDecodeTile = 16;           // tokens
constexpr int kDecodeRows = 16;           // query heads a warp takes at a time (one MMA's rows)
// (1 to 3 places: 114 to 117 us on the ragged batch, 73 to 79 us on the long sequence, 1 best over both)
constexpr int kDecodeGap = 1;
// At most this many tokens a sequence, and no more segments than SMs: a CTA takes a whole segment. Device time
// of the two ways, 8 kv heads, d = 128 (whole / split, us): 256 tokens 6.7 / 7.6 (one sequence), 6.9 / 7.8 (4),
// 7.3 / 10.3 (16); 512 tokens 8.7 / 7.7, 9.0 / 9.1, 9.3 / 12.6; 1024 tokens 13.4 / 8.2, 13.6 / 9.8, 14.0 / 17.3.
// A whole segment saves the second launch's 3 us of host time too; a longer limit would leave a batch of one
// long and many short sequences to one CTA. The host sees the table's width only, not the lengths: a table of more
// than 512 tokens a sequence is split however short they are, and the rule loses where the figures above cross it
// (one sequence of 512 tokens, 16 of 1024).
constexpr int kDecodeWholeTokens = 512;
constexpr int kDecodeMaxCtas = 148;       // the workspace has room for this many CTAs' partials
constexpr int kDecodeJoinThreads = 256;

// n / d for 0 <= n < 2^31 as a multiplication: mul = ceil(2^(31 + l) / d), 2^l >= d.
struct FastDiv {
  unsigned int mul;
  int shift;
};
__device__ __forceinline__ int fast_div(int n, const FastDiv& f) {
  return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned int>(n)) * f.mul) >> f.shift);
}

// The segment that begins in a CTA's range and goes on behind it.
struct DecodeTail {
  long long begin;                        // list place of its first tile
  long long cta_range;                    // places of a CTA's range
  int b, hv, tiles, valid;
};

struct DecodeParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;                             // may be null
  long long q_sb, o_sb;
  PagedRef kc, vc;
  const int *table, *lens;
  int B, Hq, Hkv, pages, page_size, max_pages;
  int group, chunks;                      // query heads per kv head, and their chunks of 16
  int whole;                              // a CTA takes a whole segment
  FastDiv by_page;
  float scale_log2;
  float* first_o;                         // [warps][rows][D]: pieces of a warp's first segment (16 rows, D = 128)
  float* part_o;                          // [CTAs][2][rows][D]: partials of segments across CTAs
  float2* part_ml;                        // [CTAs][2][rows]: running maximum (log2 units), sum
  struct DecodeTail* tail;                // [CTAs]
  int rows;                               // query rows of a partial: min(group, 16)
  unsigned int* err;
};

template <int D, int ROWS>
struct DecodeLayout {
  static constexpr int kStages = 24 * 128 / (8 * D);      // 24 KB a warp
  static constexpr uint32_t kHalf = kDecodeTile * D * 2;  // the K or V rows of a tile
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr uint32_t kRing = kDecodeWarps * kStages * kStage;
  // The pieces of the warps' first segments stay in shared memory where it has room (a load from global memory
  // takes 3 us while the other SMs stream), else they go to the workspace.
  static constexpr uint32_t kFirst = ROWS * D * 4;        // of a warp
  static constexpr bool kFirstShared = kRing + kDecodeWarps * kFirst <= 225 * 1024;
  // (the list's prefix sums lie there before: 257 of 8 bytes)
  static constexpr uint32_t kBytes = kRing + (kFirstShared ? kDecodeWarps * kFirst : 2304);
  static_assert(kBytes + 3072 <= 227 * 1024 && kBytes - kRing >= 8 * (kDecodeThreads + 1), "shared memory of one CTA");
};

__device__ __forceinline__ void decode_copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A sequence's length as the kernels use it: never outside [0, the block table's row].
__device__ __forceinline__ int decode_len(const DecodeParams& p, int b) {
  const int n = p.lens[b];
  const long long most = static_cast<long long>(p.max_pages) * p.page_size;
  return n < 0 ? 0 : n > most ? static_cast<int>(most) : n;
}
__device__ __forceinline__ int decode_tiles(int len) { return len / kDecodeTile + (len % kDecodeTile != 0); }

// n / d, by a 32-bit division where n fits (a 64-bit one takes hundreds of cycles at the kernel's start).
__device__ __forceinline__ unsigned long long div_near(unsigned long long n, unsigned int d) {
  return n >> 32 ? n / d : static_cast<unsigned int>(n) / d;
}

// A tile: its sequence, head, number in the segment, and its place in the list.
struct DecodeAt {
  int b, hv, tile, tiles, len;            // hv = kv head * chunks + chunk of its query heads
  long long place;
};

// The query heads of a segment: the first one, and how many.
__device__ __forceinline__ int decode_heads(const DecodeParams& p, int hv, int& h0) {
  const int kvh = p.chunks == 1 ? hv : hv / p.chunks;
  h0 = kvh * p.group + (hv - kvh * p.chunks) * kDecodeRows;
  return min(kDecodeRows, (kvh + 1) * p.group - h0);
}

// ROWS: 8 or 16 query rows a warp computes (the MMA has 16).
template <int D, int ROWS>
__global__ void __launch_bounds__(kDecodeThreads, 1) s2_decode_kernel(const __grid_constant__ DecodeParams p) {
  using L = DecodeLayout<D, ROWS>;
  constexpr int kSteps = D / 16, kHalves = ROWS / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_warp[kDecodeWarps];
  long long* const s_pre = reinterpret_cast<long long*>(smem + L::kRing);
  // The pieces of segments that did not end where they began: of each warp's first segment and of
  // its last. kind 0: none, 1: the first one's output, 2: the last one's, in the warp's ring.
  __shared__ struct { long long begin; int b, hv, tiles, kind; } s_piece[2 * kDecodeWarps];
  __shared__ float2 s_ml[2 * kDecodeWarps][ROWS];
  __shared__ unsigned int s_segment[2 * kDecodeWarps];   // the pieces of each segment
  __shared__ int s_segments;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x < 2 * kDecodeWarps) s_piece[threadIdx.x].kind = 0;
  if (threadIdx.x == 0) p.tail[blockIdx.x].valid = 0;

  const int hv_count = p.Hkv * p.chunks;
  // ---- the list: places before every run of `per` sequences ----
  const int per = (p.B + kDecodeThreads - 1) / kDecodeThreads;
  auto places = [](int tiles) { return tiles == 0 ? 0 : tiles + kDecodeGap; };   // of one segment
  if (!p.whole) {
    long long sum = 0;
    for (int i = 0; i < per; ++i) {
      const int b = threadIdx.x * per + i;
      if (b >= p.B) break;
      const int n = p.lens[b], len = decode_len(p, b);
      if (blockIdx.x == 0 && n != len) report_bad_index(p.err, KID_DECODE, kSiteBadLength);
      sum += places(decode_tiles(len));
    }
    long long inc = sum;                  // inclusive scan: in the warp, then over the warps
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    for (int i = 0; i < warp; ++i) inc += s_warp[i];
    s_pre[threadIdx.x + 1] = inc;
    if (threadIdx.x == 0) s_pre[0] = 0;
    __syncthreads();
  }
  long long cta_first = 0, cta_last = 0, cta_range;
  int own_b = 0, own_len = 0;             // of a CTA that takes a whole segment: its places begin at 0
  if (p.whole) {
    own_b = blockIdx.x / hv_count;
    own_len = decode_len(p, own_b);
    if (threadIdx.x == 0 && own_len != p.lens[own_b]) report_bad_index(p.err, KID_DECODE, kSiteBadLength);
    cta_range = cta_last = decode_tiles(own_len);
    __syncthreads();
  } else {
    const long long total = s_pre[kDecodeThreads] * hv_count;
    cta_range = static_cast<long long>(div_near(total + gridDim.x - 1, gridDim.x));
    cta_first = blockIdx.x * cta_range;
    cta_last = cta_first + cta_range < total ? cta_first + cta_range : total;
  }
  const long long warp_range = (cta_range + kDecodeWarps - 1) / kDecodeWarps;
  const long long first = cta_first + warp * warp_range;
  const long long last = first + warp_range < cta_last ? first + warp_range : cta_last;

  // ---- where the range begins ----
  DecodeAt at{};
  at.place = last;                        // nothing to do
  if (first < last && p.whole) {
    at = DecodeAt{own_b, static_cast<int>(blockIdx.x) % hv_count, static_cast<int>(first),
                  static_cast<int>(cta_last), own_len, first};
  } else if (first < last) {
    // the last run that begins at or before the range: eight runs a lane
    int below = 0;
#pragma unroll
    for (int i = 0; i < kDecodeThreads / 32; ++i) below += s_pre[32 * i + lane] * hv_count <= first;
    const int lo = __reduce_add_sync(0xffffffffu, below) - 1;
    long long begin = s_pre[lo];
    at.b = lo * per;
    for (;;) {
      at.len = decode_len(p, at.b);
      at.tiles = decode_tiles(at.len);
      if (first < (begin + places(at.tiles)) * hv_count) break;
      begin += places(at.tiles);
      ++at.b;
    }
    const unsigned long long in = first - begin * hv_count;
    const unsigned int each = places(at.tiles);
    at.hv = static_cast<int>(div_near(in, each));
    at.tile = static_cast<int>(in - static_cast<unsigned long long>(at.hv) * each) - kDecodeGap;
    at.place = first;
    if (at.tile < 0) {                    // in the gap before a segment
      at.place -= at.tile;
      at.tile = 0;
    }
  }
  auto advance = [&](DecodeAt& a) {       // the next tile, if its place is still in the range
    ++a.place;
    if (++a.tile < a.tiles) return;
    a.place += kDecodeGap;
    if (a.place >= last) return;
    a.tile = 0;
    if (++a.hv < hv_count) return;
    a.hv = 0;
    do {
      ++a.b;
      a.len = decode_len(p, a.b);
      a.tiles = decode_tiles(a.len);
    } while (a.tiles == 0);
  };

  __syncthreads();                        // the prefix sums' place is free

  // ---- copies ----
  constexpr int kChunks = D / 8;                     // 16-byte chunks of a row
  constexpr int kRowsPer = 32 / kChunks;             // rows a warp copies with one instruction
  uint8_t* const ring_p = smem + warp * (L::kStages * L::kStage);
  const uint32_t ring = smem_u32(ring_p);
  int page, slot;                                    // of row lane % 16 of the load cursor's tile
  auto look_up = [&](const DecodeAt& a) {
    const int t = a.tile * kDecodeTile + (lane & 15);
    page = -1;
    slot = 0;
    if (t < a.len) {
      const int i = fast_div(t, p.by_page);
      slot = t - i * p.page_size;
      page = p.table[static_cast<long long>(a.b) * p.max_pages + i];
      if (page < 0 || page >= p.pages) {
        report_bad_index(p.err, KID_DECODE, kSiteBadPage);
        page = -1;
      }
    }
  };
  DecodeAt ld = at;
  int load_stage = 0;
  if (ld.place < last) look_up(ld);
  auto issue = [&]() {                               // the next tile's rows into its stage
    if (ld.place < last) {
      const uint32_t dst = ring + load_stage * L::kStage;
      load_stage = load_stage + 1 == L::kStages ? 0 : load_stage + 1;
      const int kvh = p.chunks == 1 ? ld.hv : ld.hv / p.chunks;
      const int c = lane % kChunks;
      const long long col = static_cast<long long>(kvh) * D + 8 * c;
#pragma unroll
      for (int i = 0; i < kDecodeTile / kRowsPer; ++i) {
        const int row = i * kRowsPer + lane / kChunks;
        const int pg = __shfl_sync(0xffffffffu, page, row), sl = __shfl_sync(0xffffffffu, slot, row);
        const bool on = pg >= 0;                     // rows past the length become zeros
        const int pz = on ? pg : 0;
        const uint32_t off = row * (D * 2) + ((c ^ (row & 7)) * 16);
        decode_copy16(dst + off, p.kc.p + pz * p.kc.sp + sl * p.kc.st + col, on);
        decode_copy16(dst + L::kHalf + off, p.vc.p + pz * p.vc.sp + sl * p.vc.st + col, on);
      }
      advance(ld);
      if (ld.place < last) look_up(ld);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < L::kStages - 1; ++s) issue();

  // Rows of empty sequences, while the first copies are on their way.
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (decode_len(p, b) != 0) continue;
    for (int i = threadIdx.x; i < p.Hq * D; i += kDecodeThreads) p.o[b * p.o_sb + i] = __float2bfloat16(0.f);
    if (p.lse)
      for (int i = threadIdx.x; i < p.Hq; i += kDecodeThreads) p.lse[static_cast<long long>(b) * p.Hq + i] = -INFINITY;
  }

  // Where a warp leaves the piece of its first segment.
  auto first_piece = [&](int w) -> float* {
    if (L::kFirstShared) return reinterpret_cast<float*>(smem + L::kRing + w * L::kFirst);
    return p.first_o + (static_cast<long long>(blockIdx.x) * kDecodeWarps + w) * p.rows * D;
  };

  // ---- the range, tile by tile ----
  const int r0 = lane / 4, c0 = 2 * (lane % 4);
  uint32_t qf[kSteps][4];
  float acc[D / 8][4];
  float m[kHalves], l[kHalves];
  int stage = 0;
  bool fresh = true;                                 // a segment begins here, for this warp
  int seg_tile = 0;                                  // ... at this tile of it
  while (at.place < last) {
    int h0;
    const int rows = decode_heads(p, at.hv, h0);
    if (fresh) {                                     // its queries, empty state
      const __nv_bfloat16* qb = p.q + at.b * p.q_sb + static_cast<long long>(h0) * D + c0;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = r0 + 8 * (e & 1);
          qf[k][e] = row < ROWS && row < rows
                         ? *reinterpret_cast<const uint32_t*>(qb + row * D + 16 * k + 8 * (e >> 1)) : 0u;
        }
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
#pragma unroll
      for (int i = 0; i < kHalves; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
      }
      seg_tile = at.tile;
      fresh = false;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(L::kStages - 2) : "memory");
    __syncwarp();                                    // every lane's copies, and the stage freed below
    issue();
    const uint32_t ks = ring + stage * L::kStage, vs = ks + L::kHalf;
    stage = stage + 1 == L::kStages ? 0 : stage + 1;

    float s[2][4] = {};
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      uint32_t kb[4];
      const int row = (lane >> 4) * 8 + (lane & 7), ch = 2 * k + ((lane >> 3) & 1);
      ldsm4(kb, ks + row * (D * 2) + ((ch ^ (row & 7)) * 16));
      mma_bf16(s[0], qf[k], kb[0], kb[1]);
      mma_bf16(s[1], qf[k], kb[2], kb[3]);
    }
    const int left = at.len - at.tile * kDecodeTile;
    if (left < kDecodeTile) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * t + c0 + (e & 1) >= left) s[t][e] = -INFINITY;
    }
    uint32_t pf[4] = {0, 0, 0, 0};
#pragma unroll
    for (int half = 0; half < kHalves; ++half) {     // rows r0 and r0 + 8
      float mx = fmaxf(fmaxf(s[0][2 * half], s[0][2 * half + 1]), fmaxf(s[1][2 * half], s[1][2 * half + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float cand = fmaxf(m[half], mx * p.scale_log2);
      // the sums keep an old maximum until it has grown by 2^8: exp2 stays far inside fp32
      if (__any_sync(0xffffffffu, cand > m[half] + 8.f)) {
        const float alpha = cand == -INFINITY ? 1.f : fast_exp2(m[half] - cand);
        l[half] *= alpha;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          acc[j][2 * half] *= alpha;
          acc[j][2 * half + 1] *= alpha;
          if (ROWS == 8) {
            acc[j][2] *= alpha;
            acc[j][3] *= alpha;
          }
        }
        m[half] = cand;
      }
      const float mu = m[half] == -INFINITY ? 0.f : m[half];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float e0 = fast_exp2(fmaf(s[t][2 * half], p.scale_log2, -mu));
        const float e1 = fast_exp2(fmaf(s[t][2 * half + 1], p.scale_log2, -mu));
        l[half] += e0 + e1;
        const uint32_t hi = pack_bf16(e0, e1);
        pf[2 * t + half] = hi;
        // With 8 rows the MMA's other 8 carry what the rounding of P to bf16 leaves, so that the product
        // has P to 16 bits at no cost (output error 0.0023 -> 0.0017, that of its own rounding).
        if (ROWS == 8) pf[2 * t + 1] = pack_bf16(e0 - __uint_as_float(hi << 16), e1 - __uint_as_float(hi & 0xffff0000u));
      }
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      uint32_t vb[4];
      const int row = ((lane >> 3) & 1) * 8 + (lane & 7), ch = 2 * j + (lane >> 4);
      ldsm4_t(vb, vs + row * (D * 2) + ((ch ^ (row & 7)) * 16));
      mma_bf16(acc[2 * j], pf, vb[0], vb[1]);
      mma_bf16(acc[2 * j + 1], pf, vb[2], vb[3]);
    }

    const DecodeAt now = at;
    advance(at);
    const bool seg_end = now.tile + 1 == now.tiles, end = at.place >= last;
    if (!seg_end && !end) continue;
    fresh = true;
    if (ROWS == 8) {
      // (where a value was infinite the product with the rounded P is the result: the rest of P may be 0 or
      // negative, and its product NaN or of the other sign)
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        if (isfinite(acc[j][0])) acc[j][0] += acc[j][2];
        if (isfinite(acc[j][1])) acc[j][1] += acc[j][3];
      }
    }
    const bool whole = seg_end && seg_tile == 0;
    const int piece = 2 * warp + (end ? 1 : 0);
    float* out = first_piece(warp);
    if (!whole) {
      if (end) {                                     // the ring is free: every tile has been used
        __syncwarp();
        out = reinterpret_cast<float*>(ring_p);
      }
      if (lane == 0) {
        s_piece[piece].begin = now.place - now.tile;
        s_piece[piece].b = now.b;
        s_piece[piece].hv = now.hv;
        s_piece[piece].tiles = now.tiles;
        s_piece[piece].kind = end ? 2 : 1;
      }
    }
#pragma unroll
    for (int half = 0; half < kHalves; ++half) {
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
      const int row = r0 + 8 * half;
      if (row >= rows) continue;
      if (whole) {
        const float inv = 1.f / l[half];
        __nv_bfloat16* ob = p.o + now.b * p.o_sb + static_cast<long long>(h0 + row) * D + c0;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
          *reinterpret_cast<uint32_t*>(ob + 8 * j) = pack_bf16(acc[j][2 * half] * inv, acc[j][2 * half + 1] * inv);
        if (p.lse && lane % 4 == 0)
          p.lse[static_cast<long long>(now.b) * p.Hq + h0 + row] = (m[half] + log2f(l[half])) * 0.6931471805599453f;
      } else {
        float* ob = out + row * D + c0;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
          *reinterpret_cast<float2*>(ob + 8 * j) = make_float2(acc[j][2 * half], acc[j][2 * half + 1]);
        if (lane % 4 == 0) s_ml[piece][row] = make_float2(m[half], l[half]);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  // ---- join the CTA's pieces ----
  // Lane x of the first warp looks at piece x: `live` are the pieces there are, `heads` the first ones of
  // their segments; each head notes its segment's pieces.
  if (warp == 0) {
    const int x = lane & (2 * kDecodeWarps - 1);
    const bool is_piece = lane < 2 * kDecodeWarps && s_piece[x].kind != 0;
    const long long begin = s_piece[x].begin;
    const unsigned int live = __ballot_sync(0xffffffffu, is_piece);
    const unsigned int before = live & ((1u << lane) - 1u);
    const long long last_begin = __shfl_sync(0xffffffffu, begin, before ? 31 - __clz(before) : 0);
    const bool head = is_piece && (before == 0 || last_begin != begin);
    const unsigned int heads = __ballot_sync(0xffffffffu, head);
    const unsigned int behind = heads & ~((2u << lane) - 1u);
    if (head)
      s_segment[__popc(heads & ((1u << lane) - 1u))] =
          live & ~((1u << lane) - 1u) & (behind ? (1u << (__ffs(behind) - 1)) - 1u : 0xffffffffu);
    if (lane == 0) s_segments = __popc(heads);
  }
  __syncthreads();
  // Four columns of a row of a segment each time, all segments side by side.
  const int places_each = p.rows * (D / 4);
#pragma unroll 1
  for (int u = threadIdx.x; u < s_segments * places_each; u += kDecodeThreads) {
    const int g = u / places_each, in = u - g * places_each;
    const int row = in / (D / 4), col = 4 * (in % (D / 4));
    const unsigned int mine = s_segment[g];
    const int i = __ffs(mine) - 1;
    const long long begin = s_piece[i].begin;
    const int b = s_piece[i].b, hv = s_piece[i].hv, tiles = s_piece[i].tiles;
    int h0;
    if (row >= decode_heads(p, hv, h0)) continue;
    float mt = -INFINITY, lt = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (unsigned int m = mine; m; m &= m - 1) {
      const int k = __ffs(m) - 1;
      const float* src = s_piece[k].kind == 1
          ? first_piece(k / 2)
          : reinterpret_cast<const float*>(smem + (k / 2) * (L::kStages * L::kStage));
      const float4 v = *reinterpret_cast<const float4*>(src + row * D + col);
      const float2 ml = s_ml[k][row];
      const float mn = fmaxf(mt, ml.x), mu = mn == -INFINITY ? 0.f : mn;
      const float alpha = fast_exp2(mt - mu), w = fast_exp2(ml.x - mu);
      mt = mn;
      lt = lt * alpha + ml.y * w;
      sum.x = sum.x * alpha + v.x * w;
      sum.y = sum.y * alpha + v.y * w;
      sum.z = sum.z * alpha + v.z * w;
      sum.w = sum.w * alpha + v.w * w;
    }
    const bool starts = begin >= cta_first, ends = begin + tiles <= cta_last;
    if (starts && ends) {
      const float inv = 1.f / lt;
      uint2 w2;
      w2.x = pack_bf16(sum.x * inv, sum.y * inv);
      w2.y = pack_bf16(sum.z * inv, sum.w * inv);
      *reinterpret_cast<uint2*>(p.o + b * p.o_sb + static_cast<long long>(h0 + row) * D + col) = w2;
      if (p.lse && col == 0)
        p.lse[static_cast<long long>(b) * p.Hq + h0 + row] = (mt + log2f(lt)) * 0.6931471805599453f;
    } else {
      const long long part = (blockIdx.x * 2ll + (starts ? 1 : 0)) * p.rows + row;
      *reinterpret_cast<float4*>(p.part_o + part * D + col) = sum;
      if (col == 0) p.part_ml[part] = make_float2(mt, lt);
      if (starts && in == 0) p.tail[blockIdx.x] = DecodeTail{begin, cta_range, b, hv, tiles, 1};
    }
  }
}

// Joins the partials of the segments that cross CTAs: block (c, row) that query row of the segment
// that begins in CTA c's range and goes on behind it, if there is one. Each warp takes every eighth
// partial's row (a float4 or float2 a lane), then the warps' sums are added in order.
template <int D>
__global__ void __launch_bounds__(kDecodeJoinThreads) s2_decode_join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kWarps = kDecodeJoinThreads / 32;
  constexpr int kPer = D / 32;
  __shared__ float s_o[kWarps][D];
  __shared__ float2 s_ml[kWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x, row = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  const DecodeTail t = p.tail[cta];
  if (!t.valid) return;
  int h0;
  if (row >= decode_heads(p, t.hv, h0)) return;
  // partial 0: CTA `cta`, where the segment begins (its second slot); i: CTA `cta` + i's first slot
  const int n = static_cast<int>((t.begin + t.tiles - 1) / t.cta_range) - cta + 1;
  auto part = [&](int i) { return ((cta + i) * 2ll + (i == 0 ? 1 : 0)) * p.rows + row; };
  float m = -INFINITY, l = 0.f, acc[kPer] = {};
#pragma unroll 4
  for (int i = warp; i < n; i += kWarps) {
    const float2 ml = p.part_ml[part(i)];
    const float* src = p.part_o + part(i) * D + lane * kPer;
    float v[kPer];
    if constexpr (kPer == 4) {
      const float4 x = *reinterpret_cast<const float4*>(src);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(src);
      v[0] = x.x; v[1] = x.y;
    }
    const float mn = fmaxf(m, ml.x), mu = mn == -INFINITY ? 0.f : mn;
    const float alpha = fast_exp2(m - mu), w = fast_exp2(ml.x - mu);
    l = l * alpha + ml.y * w;
    m = mn;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = acc[e] * alpha + v[e] * w;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) s_o[warp][lane * kPer + e] = acc[e];
  if (lane == 0) s_ml[warp] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x < D) {
    float mt = -INFINITY;
    for (int i = 0; i < kWarps; ++i) mt = fmaxf(mt, s_ml[i].x);
    const float mu = mt == -INFINITY ? 0.f : mt;
    float lt = 0.f, ot = 0.f;
    for (int i = 0; i < kWarps; ++i) {
      const float w = fast_exp2(s_ml[i].x - mu);
      lt = fmaf(s_ml[i].y, w, lt);
      ot = fmaf(s_o[i][threadIdx.x], w, ot);
    }
    p.o[t.b * p.o_sb + static_cast<long long>(h0 + row) * D + threadIdx.x] = __float2bfloat16(ot / lt);
    if (p.lse && threadIdx.x == 0)
      p.lse[static_cast<long long>(t.b) * p.Hq + h0 + row] = (mt + log2f(lt)) * 0.6931471805599453f;
  }
}

}  // namespace s2

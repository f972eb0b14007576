// Attention of one new token per sequence over a paged key/value cache.
//
// For sequence b with n = lens[b] cached tokens, query head h and its key/value head g = h / (Hq /
// Hkv): s_j = scale * q_h . k_{j,g}, o_h = sum_j exp(s_j) v_{j,g} / sum_j exp(s_j), lse_h = log
// sum_j exp(s_j), j < n. Every cache row is read once for all heads of its group, so the bytes of
// K and V bound the kernel: two multiply-adds per element and query head.
//
// Split over the length: the batch is one list of 16-token tiles, sequence by sequence and inside
// it head by head (a segment is one (sequence, head) pair's tiles). The list is cut into equal
// contiguous ranges, one per warp of the grid, whatever the lengths are, so a ragged batch and a
// single long sequence load every SM alike. The lengths are read on the device: one launch, and a
// captured graph, serves every length. A segment inside one range is finished by its warp; of the
// others each warp leaves at most two partial results (running maximum, sum and unnormalised
// output in fp32) in the workspace, which a second small kernel joins in the order of the ranges
// (no atomics: the same bits every time). It is launched programmatically early and waits there.
//
// A warp is on its own: it copies its tiles' rows to its part of shared memory with 16-byte
// asynchronous copies (the row's page looked up one tile ahead), kDecodeStages tiles deep, so
// copies run ahead across segment boundaries, and there is no barrier between warps. Copies of single rows take any page size and any
// stride. The products run on mma.sync (16 query rows x 8 keys x 16): at 6.5 TB/s the products of
// 16 padded rows need about 100 TFLOP/s, far below what it reaches, and the fragment of the scores
// is the fragment of P in the second product, in registers. Scores, maxima, sums and outputs are
// fp32; P is rounded to bf16 for the tensor cores as in the other attention kernels.
#pragma once

#include "s2_device.cuh"
#include "s2_serve_common.cuh"

namespace s2 {

constexpr int kDecodeWarps = 8;
constexpr int kDecodeThreads = 32 * kDecodeWarps;
constexpr int kDecodeTile = 16;           // tokens
constexpr int kDecodeRows = 16;           // query heads a warp takes at a time (one MMA's rows)
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

struct DecodeParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;                             // may be null
  long long q_sb, o_sb;
  PagedRef kc, vc;
  const int *table, *lens;
  int B, Hq, Hkv, pages, page_size, max_pages;
  int group, chunks;                      // query heads per kv head, and their chunks of 16
  FastDiv by_page;
  float scale_log2;
  float* part_o;                          // [warps][2][rows][D]
  float2* part_ml;                        // [warps][2][rows]: running maximum (log2 units), sum
  long long* plan;                        // [0]: tiles per warp; [1 + b]: first tile of sequence b / (Hkv chunks)
  int rows;                               // query rows of a partial: min(group, 16)
  unsigned int* err;
};

template <int D>
struct DecodeLayout {
  static constexpr int kStages = 24 * 128 / (8 * D);      // 24 KB a warp
  static constexpr uint32_t kHalf = kDecodeTile * D * 2;  // the K or V rows of a tile
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr uint32_t kBytes = kDecodeWarps * kStages * kStage;
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

// A place in the list of tiles.
struct DecodeAt {
  int b, hv, tile, tiles, len;            // hv = kv head * chunks + chunk of its query heads
};

template <int D>
__global__ void __launch_bounds__(kDecodeThreads, 1) s2_decode_kernel(const __grid_constant__ DecodeParams p) {
  using L = DecodeLayout<D>;
  constexpr int kSteps = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_pre[kDecodeThreads + 1];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  pdl_launch_dependents();

  // ---- the plan: tiles before every run of `per` sequences ----
  const int hv_count = p.Hkv * p.chunks;
  const int per = (p.B + kDecodeThreads - 1) / kDecodeThreads;
  {
    long long sum = 0;
    for (int i = 0; i < per; ++i) {
      const int b = threadIdx.x * per + i;
      if (b >= p.B) break;
      const int n = p.lens[b], len = decode_len(p, b);
      if (blockIdx.x == 0 && n != len) report_bad_index(p.err, KID_DECODE, kSiteBadLength);
      sum += decode_tiles(len);
    }
    long long inc = sum;                  // inclusive scan: in the warp, then over the warps
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    __shared__ long long s_warp[kDecodeWarps];
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    for (int i = 0; i < warp; ++i) inc += s_warp[i];
    s_pre[threadIdx.x + 1] = inc;
    if (threadIdx.x == 0) s_pre[0] = 0;
    __syncthreads();
    if (blockIdx.x == 0) {                // for the joining kernel
      long long at = inc - sum;
      for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b >= p.B) break;
        p.plan[1 + b] = at;
        at += decode_tiles(decode_len(p, b));
      }
    }
  }
  const long long total = s_pre[kDecodeThreads] * hv_count;
  const long long n_warps = static_cast<long long>(gridDim.x) * kDecodeWarps;
  const long long range = (total + n_warps - 1) / n_warps;
  if (blockIdx.x == 0 && threadIdx.x == 0) p.plan[0] = range;
  // neighbouring ranges on different SMs: a short list spreads over all of them
  const long long gw = static_cast<long long>(warp) * gridDim.x + blockIdx.x;
  const long long first = gw * range, last = first + range < total ? first + range : total;
  if (first >= last) return;

  // ---- where the range begins ----
  DecodeAt at;
  long long seg_begin;                    // the list index of the current segment's first tile
  {
    const long long x = first;
    int lo = 0, hi = kDecodeThreads;      // the last run that begins at or before x
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s_pre[mid] * hv_count <= x) lo = mid; else hi = mid;
    }
    long long begin = s_pre[lo];
    at.b = lo * per;
    for (;;) {
      at.len = decode_len(p, at.b);
      at.tiles = decode_tiles(at.len);
      if (x < (begin + at.tiles) * hv_count) break;
      begin += at.tiles;
      ++at.b;
    }
    const long long in = x - begin * hv_count;
    at.hv = static_cast<int>(in / at.tiles);
    at.tile = static_cast<int>(in % at.tiles);
    seg_begin = x - at.tile;
  }
  auto advance = [&](DecodeAt& a) {       // the next tile (only while one is left in the range)
    if (++a.tile < a.tiles) return;
    a.tile = 0;
    if (++a.hv < hv_count) return;
    a.hv = 0;
    do {
      ++a.b;
      a.len = decode_len(p, a.b);
      a.tiles = decode_tiles(a.len);
    } while (a.tiles == 0);
  };

  // ---- copies ----
  constexpr int kChunks = D / 8;                     // 16-byte chunks of a row
  constexpr int kRowsPer = 32 / kChunks;             // rows a warp copies with one instruction
  const uint32_t ring = smem_u32(smem) + warp * (L::kStages * L::kStage);
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
  const int n_tiles = static_cast<int>(last - first);
  int loaded = 0;
  look_up(ld);
  auto issue = [&]() {                               // the next tile's rows into its stage
    if (loaded < n_tiles) {
      const uint32_t dst = ring + (loaded % L::kStages) * L::kStage;
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
      if (++loaded < n_tiles) {
        advance(ld);
        look_up(ld);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < L::kStages - 1; ++s) issue();

  // ---- the range, tile by tile ----
  const int r0 = lane / 4, c0 = 2 * (lane % 4);
  uint32_t qf[kSteps][4];
  float acc[D / 8][4];
  float m[2], l[2];
  for (int n = 0; n < n_tiles; ++n) {
    const int kvh = p.chunks == 1 ? at.hv : at.hv / p.chunks;
    const int h0 = kvh * p.group + (at.hv - kvh * p.chunks) * kDecodeRows;
    const int rows = min(kDecodeRows, (kvh + 1) * p.group - h0);
    if (n == 0 || at.tile == 0) {                    // a segment begins: its queries, empty state
      const __nv_bfloat16* qb = p.q + at.b * p.q_sb + static_cast<long long>(h0) * D + c0;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = r0 + 8 * (e & 1);
          qf[k][e] = row < rows ? *reinterpret_cast<const uint32_t*>(qb + row * D + 16 * k + 8 * (e >> 1)) : 0u;
        }
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(L::kStages - 2) : "memory");
    __syncwarp();                                    // every lane's copies, and the stage freed below
    issue();
    const uint32_t ks = ring + (n % L::kStages) * L::kStage, vs = ks + L::kHalf;

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
    uint32_t pf[4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {           // rows r0 and r0 + 8
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
        }
        m[half] = cand;
      }
      const float mu = m[half] == -INFINITY ? 0.f : m[half];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float e0 = fast_exp2(fmaf(s[t][2 * half], p.scale_log2, -mu));
        const float e1 = fast_exp2(fmaf(s[t][2 * half + 1], p.scale_log2, -mu));
        l[half] += e0 + e1;
        pf[2 * t + half] = pack_bf16(e0, e1);
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

    const bool seg_end = at.tile + 1 == at.tiles;
    if (seg_end || n + 1 == n_tiles) {
      const bool whole = seg_end && seg_begin >= first;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
        l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
        const int row = r0 + 8 * half;
        if (row >= rows) continue;
        if (whole) {
          const float inv = 1.f / l[half];
          __nv_bfloat16* ob = p.o + at.b * p.o_sb + static_cast<long long>(h0 + row) * D + c0;
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<uint32_t*>(ob + 8 * j) = pack_bf16(acc[j][2 * half] * inv, acc[j][2 * half + 1] * inv);
          if (p.lse && lane % 4 == 0)
            p.lse[static_cast<long long>(at.b) * p.Hq + h0 + row] =
                (m[half] + log2f(l[half])) * 0.6931471805599453f;
        } else {
          // partial 0: the segment holds the range's first tile; 1: it begins inside the range
          const long long part = (gw * 2 + (seg_begin > first ? 1 : 0)) * p.rows + row;
          float* ob = p.part_o + part * D + c0;
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<float2*>(ob + 8 * j) = make_float2(acc[j][2 * half], acc[j][2 * half + 1]);
          if (lane % 4 == 0) p.part_ml[part] = make_float2(m[half], l[half]);
        }
      }
    }
    if (n + 1 < n_tiles) {
      if (seg_end) seg_begin = first + n + 1;
      advance(at);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Joins the partials of the segments that more than one warp worked on, and writes the rows of
// empty sequences (o = 0, lse = -inf). One block per (sequence, query head): each warp takes every
// eighth partial's row (a float4 or float2 a lane), then the warps' sums are added in order.
template <int D>
__global__ void __launch_bounds__(kDecodeJoinThreads) s2_decode_join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kWarps = kDecodeJoinThreads / 32;
  constexpr int kPer = D / 32;
  __shared__ float s_o[kWarps][D];
  __shared__ float2 s_ml[kWarps];
  const int b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int kvh = h / p.group, in_group = h - kvh * p.group;
  const int hv = kvh * p.chunks + in_group / kDecodeRows, row = in_group % kDecodeRows;
  const int tiles = decode_tiles(decode_len(p, b));
  pdl_wait();
  if (tiles == 0) {
    for (int c = threadIdx.x; c < D; c += kDecodeJoinThreads)
      p.o[b * p.o_sb + static_cast<long long>(h) * D + c] = __float2bfloat16(0.f);
    if (p.lse && threadIdx.x == 0) p.lse[static_cast<long long>(b) * p.Hq + h] = -INFINITY;
    return;
  }
  const long long range = p.plan[0];
  const long long t0 = p.plan[1 + b] * (p.Hkv * p.chunks) + static_cast<long long>(hv) * tiles;
  const long long w0 = t0 / range, w1 = (t0 + tiles - 1) / range;
  if (w0 == w1) return;                   // one warp had it all and wrote the result
  const int n = static_cast<int>(w1 - w0) + 1;
  auto part = [&](int i) {
    return ((w0 + i) * 2 + (i == 0 && t0 > w0 * range ? 1 : 0)) * p.rows + row;
  };
  float m = -INFINITY, l = 0.f, acc[kPer] = {};
  for (int base = warp; base < n; base += 32 * kWarps) {
    const int i = base + kWarps * lane, cnt = min(32, (n - base + kWarps - 1) / kWarps);
    const float2 ml = i < n ? p.part_ml[part(i)] : make_float2(-INFINITY, 0.f);
    float mx = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
    const float alpha = fast_exp2(m - mu), w = fast_exp2(ml.x - mu);
    l = l * alpha + ml.y * w;             // this lane's partials
    m = mn;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= alpha;
#pragma unroll 8
    for (int k = 0; k < cnt; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const float* src = p.part_o + part(base + kWarps * k) * D + lane * kPer;
      float v[kPer];
      if constexpr (kPer == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        v[0] = x.x; v[1] = x.y;
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = fmaf(v[e], wk, acc[e]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
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
    p.o[b * p.o_sb + static_cast<long long>(h) * D + threadIdx.x] = __float2bfloat16(ot / lt);
    if (p.lse && threadIdx.x == 0)
      p.lse[static_cast<long long>(b) * p.Hq + h] = (mt + log2f(lt)) * 0.6931471805599453f;
  }
}

}  // namespace s2

// kv4_attn.cu -- attention of the newest tokens over the 4-bit KV cache.
//
// For token i of the T newest of a sequence of n keys, and query head h of KV
// head g = h / G:
//   S[j] = scale q . k_j  (j < n - T + i + 1),  p = softmax(S),  out = sum p_j v_j,
// and, if asked, score[g][j] += the sum of p_j over the T * G rows of g.
//
// What bounds it: the cache is read once, 2 (d/2 + d/16) bytes a key and KV
// head.  An SM's share of the copy rate is ~23 bytes a clock, a key of 144
// bytes (d = 128) each 6.2 clocks, in which 256 values must be widened and
// used by G query rows.  FMAs alone would take 8 clocks at G = 4, so the
// products run on the tensor cores with mma.sync m16n8k16 (fp16, fp32 sums):
// keys (or dims) are the 16 rows and the query rows the 8 columns, 1 mma a key
// for up to 8 rows, ~2 clocks.  tcgen05 would want the widened values in shared memory
// (a write and a read of four times the cache's bytes) and 128 columns for
// these 8; here they go from registers into the mma as they are widened.
//
//  - S^T (16 keys x 8 rows) = K (16 x 16 dims) Q^T.  Which dims a step
//    contracts is free as long as K and Q agree: thread (r, t) = (lane / 4,
//    lane % 4) takes 32 consecutive dims of its key, one 16-byte load.
//  - P^T comes out with keys down the lanes and is needed with keys across
//    them: movmatrix transposes each 8 x 8.
//  - O^T (16 dims x 8 rows) += V^T (16 x 16 keys) P^T.  Which key is which k
//    is free too: thread t takes keys t, t+4, t+8, t+12 of its 16, and lane r
//    the 16 dims that share a scale; the nibbles of two keys are woven into
//    bytes, so that one cvt gives the mma's pair.
//
// Precision: code * scale is exact in fp16.  A query row is scaled by a power
// of two to the top of fp16's range; bf16 and fp16 queries are then exact,
// fp32 ones are the sum of two fp16 parts (22 bits).  Probabilities, as
// 2^(S - max + 15) so that small ones stay normal, are one fp16 part for bf16
// results (an error of 2^-12 beside the result's 2^-9) and two for fp16 and
// fp32.  Scores, maxima, sums and outputs are fp32.
//
// Work: a unit is a block of 32 keys of one (sequence, row tile, KV head).
// All units of the call stand in one line, cut into equal contiguous ranges
// for every warp of one wave of CTAs -- the ranges come from the lengths on
// the device, so ragged batches are balanced and a graph may be replayed with
// other lengths.  A warp keeps its own ring of blocks (cp.async, no barrier
// between warps).  A range that ends inside a row of units leaves a partial
// (unnormalised output, maximum, sum); the warps of a CTA merge theirs in
// shared memory, and a second kernel merges what CTAs share and adds the
// weights to the scores.  No atomics: results do not depend on timing.
#include <math.h>

#include <type_traits>

#include "kv4.cuh"
#include "pdl.cuh"

namespace mk {
namespace {

constexpr int kWarps = 8;
constexpr int kThreadsA = kWarps * 32;
constexpr int kStages = 3;        // blocks of a warp's ring
constexpr int kMaxCtas = 320;     // partials are laid out for this many CTAs
constexpr int kMaxRows = 1024;    // query rows of a KV head: q_len * group
constexpr float kBias = 15.f;     // probabilities are 2^(S - max + kBias)

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_half2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

struct AttnArgs {
  Kv4 c;
  const uint8_t* q;
  uint8_t* out;
  size_t q_stride;       // bytes between tokens
  int32_t q_len, group, rows, tiles;   // rows = q_len * group, in `tiles` row tiles
  float s_mul;           // scale * log2(e) * 2^k_log2
  float o_mul;           // 2^v_log2
  int32_t max_ctas;
  int32_t accumulate;
  // workspace
  float* warp_part;      // [max_ctas * kWarps][R][d + 2]: a warp's first, unfinished piece
  float* cta_part;       // [max_ctas][2][R][d + 2]: a CTA's first and last, unfinished
  float* stats;          // [n_seq * tiles * heads][R][2]: max and sum of rows that one CTA finished
  float* s_all;          // [units][32][stored rows]: scores in log2 units
  int32_t s_rows;
};

// The line of units: sequence by sequence, in it row tile by row tile, KV head
// by KV head, block by block.
struct Line {
  long long total;   // units
  int ctas;          // CTAs that have any: at least kWarps units each, one a warp
};

__device__ __forceinline__ int blocks_of(int n) { return (n + kKv4Block - 1) / kKv4Block; }
__device__ __forceinline__ long long cut(const Line& l, int i, int parts) { return l.total * i / parts; }

// Sums the sequences' units over the CTA: every thread holds a run of
// consecutive sequences, `base` the units before them.
template <int THREADS>
__device__ __forceinline__ void line_scan(const AttnArgs& a, Line& l, long long& base, long long& mine, int& s0,
                                          int& s1) {
  __shared__ long long warp_sum[THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int run = (a.c.n_seq + THREADS - 1) / THREADS;
  s0 = min(a.c.n_seq, (int)threadIdx.x * run);
  s1 = min(a.c.n_seq, s0 + run);
  mine = 0;
  for (int s = s0; s < s1; ++s) mine += blocks_of(a.c.len(s));
  mine *= (long long)a.tiles * a.c.heads;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  base = inc - mine;
  l.total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) base += warp_sum[w];
    l.total += warp_sum[w];
  }
  const long long want = (l.total + kWarps - 1) / kWarps;
  l.ctas = (int)(want < a.max_ctas ? want : a.max_ctas);
}

// If unit u lies in this thread's run of sequences: its sequence and the units before that sequence.
__device__ __forceinline__ bool line_find(const AttnArgs& a, long long u, long long base, long long mine, int s0,
                                          int s1, int& seq, long long& start) {
  if (u < base || u >= base + mine) return false;
  for (int s = s0; s < s1; ++s) {
    const long long n = (long long)blocks_of(a.c.len(s)) * a.tiles * a.c.heads;
    if (u < base + n) { seq = s; start = base; return true; }
    base += n;
  }
  return false;
}

template <int R>
__device__ __forceinline__ bool row_of(const AttnArgs& a, int tile, int n, int& token, int& head) {
  const int row = tile * R + n;
  token = row / a.group;
  head = row - token * a.group;
  return row < a.rows;
}

__device__ __forceinline__ void store_out(const AttnArgs& a, size_t at, int dtype, float x) {
  if (dtype == MK_DTYPE_F32) reinterpret_cast<float*>(a.out)[at] = x;
  else if (dtype == MK_DTYPE_BF16) {
    unsigned short h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
    reinterpret_cast<unsigned short*>(a.out)[at] = h;
  } else reinterpret_cast<__half*>(a.out)[at] = __float2half_rn(x);
}

// out and, for the scores, (max, sum) of one finished row element.
template <int D, int DT, int R>
__device__ __forceinline__ void finish(const AttnArgs& a, int seq, int tile, int kvh, int n, int dim, float o,
                                       float sum) {
  int token, head;
  if (!row_of<R>(a, tile, n, token, head)) return;
  const size_t at = (((size_t)seq * a.q_len + token) * a.c.heads * a.group + (size_t)kvh * a.group + head) * D + dim;
  // a row that sees nothing has sum 0; NaN goes through
  store_out(a, at, DT, sum == 0.f ? 0.f : o / sum * a.o_mul);
}

template <int D, int R>
__device__ __forceinline__ float* part_at(float* base, size_t i) { return base + i * ((size_t)R * (D + 2)); }

// D: head dim.  DT: MK_DTYPE_* of queries and outputs.  NT: 8-row tiles of query rows.
template <int D, int DT, int NT>
__global__ void __launch_bounds__(kThreadsA, NT == 1 ? 2 : 1) kv4_attn_kernel(const AttnArgs a) {
  using S = Kv4Shape<D>;
  constexpr int R = 8 * NT;
  constexpr int QP = DT == MK_DTYPE_F32 ? 2 : 1;   // fp16 parts of a query
  constexpr int PP = DT == MK_DTYPE_BF16 ? 1 : 2;  // and of a probability
  constexpr int KS = D / 16;                       // contraction steps, and 16-dim tiles of O
  constexpr int kPart = R * (D + 2);
  static_assert(kPart * 4 <= kStages * S::kBytes, "a warp's last piece takes the place of its ring");
  extern __shared__ __align__(16) uint8_t ring_all[];
  __shared__ int found_seq[kWarps];
  __shared__ long long found_start[kWarps];
  // pieces that a warp leaves: [0] its first, in global memory, [1] its last, in its ring's place
  __shared__ int piece_item[2][kWarps];    // block index in the line's items, -1: none
  __shared__ int piece_seq[2][kWarps], piece_tile[2][kWarps], piece_head[2][kWarps];
  __shared__ int piece_begins[2][kWarps];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, t = lane & 3;
  Line line;
  long long base, mine;
  int s0, s1;
  line_scan<kThreadsA>(a, line, base, mine, s0, s1);

  // sequences without a key: their outputs are zero and no unit covers them
  for (int s = blockIdx.x; s < a.c.n_seq; s += gridDim.x) {
    if (a.c.len(s) > 0) continue;
    const size_t n = (size_t)a.rows * a.c.heads * D;
    for (size_t i = threadIdx.x; i < n; i += kThreadsA) store_out(a, s * n + i, DT, 0.f);
  }
  if ((int)blockIdx.x >= line.ctas) return;

  // this warp's range
  const int parts = line.ctas * kWarps;
  for (int w = 0; w < kWarps; ++w) {
    const long long u = cut(line, blockIdx.x * kWarps + w, parts);
    int seq;
    long long start;
    if (line_find(a, u, base, mine, s0, s1, seq, start)) { found_seq[w] = seq; found_start[w] = start; }
  }
  if (threadIdx.x < 2 * kWarps) piece_item[threadIdx.x / kWarps][threadIdx.x % kWarps] = -1;
  __syncthreads();
  long long u = cut(line, blockIdx.x * kWarps + warp, parts);
  const long long u_end = cut(line, blockIdx.x * kWarps + warp + 1, parts);

  uint8_t* ring = ring_all + (size_t)warp * kStages * S::kBytes;
  const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));

  int seq = u < u_end ? found_seq[warp] : 0;
  long long start = u < u_end ? found_start[warp] : 0;
  while (u < u_end) {
    // ---- the piece of one (sequence, row tile, KV head) that this range covers
    int n = a.c.len(seq);
    while (n == 0) n = a.c.len(++seq);   // u < total: a sequence with keys follows
    const int nb = blocks_of(n);
    const long long in_seq = u - start;
    const int item = (int)(in_seq / nb), b0 = (int)(in_seq - (long long)item * nb);
    const int tile = item / a.c.heads, kvh = item - tile * a.c.heads;
    const int b1 = (int)(u_end - u < nb - b0 ? b0 + (u_end - u) : nb);
    const int nblk = b1 - b0;
    const int per = a.c.page_tokens / kKv4Block;

    // physical blocks, 32 at a time: lane i holds the page of block b0 + 32 k + i
    int pages = -1, pages_from = 0;
    auto fetch_pages = [&](int from) {
      pages_from = from;
      pages = from + lane < b1 ? a.c.page(seq, (from + lane) / per) : -1;
    };
    fetch_pages(b0);
    auto issue = [&](int b) {   // block b into its ring slot; its page, -1 where there is none
      if (b - pages_from >= 32) fetch_pages(b);
      const int page = __shfl_sync(0xFFFFFFFFu, pages, b - pages_from);
      if (page >= 0) {
        const uint8_t* src = kv4_block<D>(a.c, page, kvh, b % per);
        const uint32_t dst = ring_s + (b - b0) % kStages * S::kBytes;
#pragma unroll
        for (int i = 0; i < (S::kBytes / 16 + 31) / 32; ++i) {
          const int at = i * 32 + lane;
          if (S::kBytes / 16 % 32 == 0 || at < S::kBytes / 16) cp16(dst + at * 16, src + at * 16);
        }
      }
      return page >= 0;
    };
    uint32_t have = 0;   // bit: the ring slot holds a block
    __syncwarp();        // the slots' last readers are done
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (i < nblk && issue(b0 + i)) have |= 1u << i;
      cp_commit();
    }

    // ---- query rows: column n = r of each 8-row tile, 2 * KS dims from t * 2 * KS
    uint32_t qf[QP][NT][2 * KS];
    float mul[NT][2];                // S -> log2 units, for this thread's columns 2t, 2t + 1
    int limit[NT][2];                // keys those columns see
    int see_all = n;                 // keys that every row sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      int token, head;
      const bool ok = row_of<R>(a, tile, nt * 8 + r, token, head);
      float x[4 * KS];
      const uint8_t* row = a.q + ((size_t)seq * a.q_len + token) * a.q_stride;
      const int dim0 = (kvh * a.group + head) * D + t * 4 * KS;
      if (DT == MK_DTYPE_F32) {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const float4 v = ok ? __ldcg(reinterpret_cast<const float4*>(row + (size_t)dim0 * 4) + i)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
          x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) {
          const uint4 v = ok ? __ldcg(reinterpret_cast<const uint4*>(row + (size_t)dim0 * 2) + i)
                             : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (DT == MK_DTYPE_BF16) {
              x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
              x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            } else {
              const float2 f = unpack_half2(w[j]);
              x[8 * i + 2 * j] = f.x; x[8 * i + 2 * j + 1] = f.y;
            }
          }
        }
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * KS; ++i) top = fmaxf(top, fabsf(x[i]));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      // 2^e with max |q| * 2^e in [2^13, 2^14); the exponent kept inside fp32's own
      int e = 13 - ((__float_as_int(top) >> 23) - 127);
      e = min(max(e, -120), 120);
      const float up = __int_as_float((127 + e) << 23);
      const float down = __int_as_float((127 - e) << 23) * a.s_mul;
#pragma unroll
      for (int i = 0; i < 2 * KS; ++i) {
        const float f0 = x[2 * i] * up, f1 = x[2 * i + 1] * up;
        const uint32_t h = pack_half2(f0, f1);
        qf[0][nt][i] = h;
        if (QP == 2) {
          const float2 b = unpack_half2(h);
          qf[QP - 1][nt][i] = pack_half2(f0 - b.x, f1 - b.y);
        }
      }
      const int lim = ok ? max(0, min(n, n - a.q_len + token + 1)) : n;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mul[nt][c] = __shfl_sync(0xFFFFFFFFu, down, (2 * t + c) * 4);
        limit[nt][c] = __shfl_sync(0xFFFFFFFFu, lim, (2 * t + c) * 4);
      }
      see_all = min(see_all, lim);
    }
    see_all = __reduce_min_sync(0xFFFFFFFFu, see_all);

    float o[NT][KS][4];
    float mx[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][j][i] = 0.f;
      mx[nt][0] = mx[nt][1] = -INFINITY;
      sum[nt][0] = sum[nt][1] = 0.f;
    }

    for (int b = b0; b < b1; ++b) {
      const int slot = (b - b0) % kStages;
      cp_wait<kStages - 2>();
      __syncwarp();
      {
        const int next = b + kStages - 1, ns = (next - b0) % kStages;
        if (next < b1) {
          if (issue(next)) have |= 1u << ns; else have &= ~(1u << ns);
        }
        cp_commit();
      }
      const bool there = have >> slot & 1u;
      const uint8_t* blk = ring + slot * S::kBytes;
      const bool masked = !there || (b + 1) * kKv4Block > see_all;   // some row does not see some key

      // S^T, 16 keys at a time
      float sc[2][NT][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int ka = half * 16 + (r >> 1) + (r & 1) * 4, kb = ka + 8;   // mma rows r and r + 8
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[half][nt][i] = 0.f;
        uint32_t wa[KS / 2], wb[KS / 2], sa[2], sb[2];
        if (D == 128) {
          const uint4 va = *reinterpret_cast<const uint4*>(blk + ka * S::kCodes + t * 16);
          const uint4 vb = *reinterpret_cast<const uint4*>(blk + kb * S::kCodes + t * 16);
          wa[0] = va.x; wa[1] = va.y; wa[KS / 2 - 2] = va.z; wa[KS / 2 - 1] = va.w;
          wb[0] = vb.x; wb[1] = vb.y; wb[KS / 2 - 2] = vb.z; wb[KS / 2 - 1] = vb.w;
          const uint32_t ha = e4m3x2(*reinterpret_cast<const uint16_t*>(blk + S::kKs + ka * S::kScales + 2 * t));
          const uint32_t hb = e4m3x2(*reinterpret_cast<const uint16_t*>(blk + S::kKs + kb * S::kScales + 2 * t));
          sa[0] = __byte_perm(ha, 0, 0x1010); sa[1] = __byte_perm(ha, 0, 0x3232);
          sb[0] = __byte_perm(hb, 0, 0x1010); sb[1] = __byte_perm(hb, 0, 0x3232);
        } else {
          const uint2 va = *reinterpret_cast<const uint2*>(blk + ka * S::kCodes + t * 8);
          const uint2 vb = *reinterpret_cast<const uint2*>(blk + kb * S::kCodes + t * 8);
          wa[0] = va.x; wa[1] = va.y; wb[0] = vb.x; wb[1] = vb.y;
          const uint32_t ha = e4m3x2(blk[S::kKs + ka * S::kScales + t]);
          const uint32_t hb = e4m3x2(blk[S::kKs + kb * S::kScales + t]);
          sa[0] = sa[1] = __byte_perm(ha, 0, 0x1010);
          sb[0] = sb[1] = __byte_perm(hb, 0, 0x1010);
        }
#pragma unroll
        for (int w = 0; w < KS / 2; ++w) {
          uint32_t ha[4], hb[4];
          e2m1x8(wa[w], ha);
          e2m1x8(wb[w], hb);
          const int g = w >> 1;   // 16 dims: two words
#pragma unroll
          for (int i = 0; i < 4; ++i) { ha[i] = hmul2(ha[i], sa[g]); hb[i] = hmul2(hb[i], sb[g]); }
#pragma unroll
          for (int p = 0; p < QP; ++p)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816(sc[half][nt], ha[0], hb[0], ha[1], hb[1], qf[p][nt][4 * w], qf[p][nt][4 * w + 1]);
              mma16816(sc[half][nt], ha[2], hb[2], ha[3], hb[3], qf[p][nt][4 * w + 2], qf[p][nt][4 * w + 3]);
            }
        }
      }

      // log2 units, masks, running maximum
      float up[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float m = -INFINITY;
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float& x = sc[half][nt][2 * i + c];
              x *= mul[nt][c];
              if (masked) {
                const int key = b * kKv4Block + half * 16 + (r >> 1) + (r & 1) * 4 + 8 * i;
                if (!there || key >= limit[nt][c]) x = -INFINITY;
              }
              m = fmaxf(m, x);
            }
          up[nt][c] = m;
        }
      if (a.accumulate) {
        float* to = a.s_all + ((size_t)(u + (b - b0)) * kKv4Block) * a.s_rows;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = half * 16 + (r >> 1) + (r & 1) * 4 + 8 * i;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (nt * 8 + 2 * t < a.s_rows)
                *reinterpret_cast<float2*>(to + (size_t)key * a.s_rows + nt * 8 + 2 * t) =
                    make_float2(sc[half][nt][2 * i], sc[half][nt][2 * i + 1]);
          }
      }
      bool moved = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float m = up[nt][c];
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
          moved |= m > mx[nt][c];
          up[nt][c] = fmaxf(m, mx[nt][c]);
        }
      if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            // nothing seen so far: nothing to rescale
            const float f = mx[nt][c] == -INFINITY ? 1.f : ex2(mx[nt][c] - up[nt][c]);
            mx[nt][c] = up[nt][c];
            sum[nt][c] *= f;
#pragma unroll
            for (int j = 0; j < KS; ++j) { o[nt][j][c] *= f; o[nt][j][2 + c] *= f; }
          }
      }

      // P^T as the mma's columns
      uint32_t pf[PP][2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float m0 = mx[nt][0] == -INFINITY ? 0.f : mx[nt][0] - kBias;
        const float m1 = mx[nt][1] == -INFINITY ? 0.f : mx[nt][1] - kBias;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p0 = ex2(sc[half][nt][2 * i] - m0), p1 = ex2(sc[half][nt][2 * i + 1] - m1);
            sum[nt][0] += p0;
            sum[nt][1] += p1;
            const uint32_t h = pack_half2(p0, p1);
            pf[0][half][nt][i] = transpose8(h);
            if (PP == 2) {
              const float2 f = unpack_half2(h);
              pf[PP - 1][half][nt][i] = transpose8(pack_half2(p0 - f.x, p1 - f.y));
            }
          }
      }

      // O^T, 16 keys at a time
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        constexpr int W = D / 64;   // words of a key's dims that lane r holds: 16 dims or 8
        uint32_t w[4][W], s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = half * 16 + t + 4 * i;
          const uint8_t* row = blk + S::kVc + key * S::kCodes;
          if (D == 128) {
            const uint2 v = *reinterpret_cast<const uint2*>(row + r * 8);
            w[i][0] = v.x; w[i][W - 1] = v.y;
            s[i] = blk[S::kVs + key * S::kScales + r];
          } else {
            w[i][0] = *reinterpret_cast<const uint32_t*>(row + r * 4);
            s[i] = blk[S::kVs + key * S::kScales + (r >> 1)];
          }
          if (masked) {
            // A value that no row sees must not count, whatever it is (a page's
            // leftovers may be NaN, and 0 * NaN is).  One that only some rows
            // see is NaN for those alone: it leaves the product and is set below.
            const int at = b * kKv4Block + key;
            const bool seen = there && at < n;
            if (!seen || (at >= see_all && (s[i] & 0x7Fu) == 0x7Fu)) s[i] = 0u;
          }
        }
        const uint32_t s01 = e4m3x2(s[0] | s[1] << 8), s23 = e4m3x2(s[2] | s[3] << 8);
#pragma unroll
        for (int x = 0; x < W; ++x) {
          // bytes j: (key 0, key 1) of an even dim, of an odd one, and the same of keys 2, 3
          const uint32_t e01 = (w[0][x] & 0x0F0F0F0Fu) | ((w[1][x] << 4) & 0xF0F0F0F0u);
          const uint32_t d01 = ((w[0][x] >> 4) & 0x0F0F0F0Fu) | (w[1][x] & 0xF0F0F0F0u);
          const uint32_t e23 = (w[2][x] & 0x0F0F0F0Fu) | ((w[3][x] << 4) & 0xF0F0F0F0u);
          const uint32_t d23 = ((w[2][x] >> 4) & 0x0F0F0F0Fu) | (w[3][x] & 0xF0F0F0F0u);
          uint32_t a0[4], a1[4], a2[4], a3[4];
          e2m1x8(e01, a0); e2m1x8(d01, a1); e2m1x8(e23, a2); e2m1x8(d23, a3);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a0[j] = hmul2(a0[j], s01); a1[j] = hmul2(a1[j], s01);
            a2[j] = hmul2(a2[j], s23); a3[j] = hmul2(a3[j], s23);
#pragma unroll
            for (int p = 0; p < PP; ++p)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(o[nt][4 * x + j], a0[j], a1[j], a2[j], a3[j], pf[p][half][nt][0], pf[p][half][nt][1]);
          }
        }
      }
      if (masked && there && see_all < n) {
        // NaN values among keys that only some rows see
        for (int key = 0; key < kKv4Block; ++key) {
          const int at = b * kKv4Block + key;
          if (at < see_all || at >= n) continue;
          if ((blk[S::kVs + key * S::kScales + (D == 128 ? r : r >> 1)] & 0x7Fu) != 0x7Fu) continue;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (at < limit[nt][c]) {
#pragma unroll
                for (int j = 0; j < KS; ++j) o[nt][j][c] = o[nt][j][2 + c] = __int_as_float(0x7FC00000);
              }
        }
      }
    }
    cp_wait<0>();
    __syncwarp();

    // ---- the piece is done: sums over the lanes that share a column
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = sum[nt][c];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
        sum[nt][c] = x;
      }
    const bool begins = b0 == 0, ends = b1 == nb;
    const size_t stat = ((size_t)seq * a.tiles * a.c.heads + item) * R;
    // dims of o[.][j]: lane r holds D / 8 consecutive ones, two a tile j
    auto dim_of = [&](int j, int i) { return r * (D / 8) + 2 * j + (i >> 1); };
    if (begins && ends) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            finish<D, DT, R>(a, seq, tile, kvh, nt * 8 + 2 * t + (i & 1), dim_of(j, i), o[nt][j][i], sum[nt][i & 1]);
      if (a.accumulate && r == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            a.stats[(stat + nt * 8 + 2 * t + c) * 2] = mx[nt][c];
            a.stats[(stat + nt * 8 + 2 * t + c) * 2 + 1] = sum[nt][c];
          }
      }
    } else {
      const int last = !ends;
      float* to = last ? reinterpret_cast<float*>(ring)
                       : part_at<D, R>(a.warp_part, (size_t)blockIdx.x * kWarps + warp);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) to[(nt * 8 + 2 * t + (i & 1)) * D + dim_of(j, i)] = o[nt][j][i];
        if (r == 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            to[R * D + nt * 8 + 2 * t + c] = mx[nt][c];
            to[R * D + R + nt * 8 + 2 * t + c] = sum[nt][c];
          }
        }
      }
      if (lane == 0) {
        piece_item[last][warp] = (int)((size_t)seq * a.tiles * a.c.heads + item);
        piece_seq[last][warp] = seq;
        piece_tile[last][warp] = tile;
        piece_head[last][warp] = kvh;
        piece_begins[last][warp] = begins;
      }
    }
    u += nblk;
    if (ends && item + 1 == a.tiles * a.c.heads) {
      start += (long long)nb * a.tiles * a.c.heads;
      ++seq;
    }
  }
  __syncthreads();

  // ---- pieces of the CTA's warps that belong together, in order: the last
  // of a warp, those of warps that lie whole in the item, the first of the one
  // where it ends
  int from[kWarps + 1], count = 0, item = -1, begins = 0, who = 0;
  auto piece = [&](int code) -> const float* {
    const int w = code >> 1;
    return code & 1 ? reinterpret_cast<const float*>(ring_all + (size_t)w * kStages * S::kBytes)
                    : part_at<D, R>(a.warp_part, (size_t)blockIdx.x * kWarps + w);
  };
  auto merge = [&](bool ends) {
    const int seq = piece_seq[who & 1][who >> 1], tile = piece_tile[who & 1][who >> 1],
              kvh = piece_head[who & 1][who >> 1];
    float* slot = part_at<D, R>(a.cta_part, (size_t)blockIdx.x * 2 + (ends ? 0 : 1));
    for (int e = threadIdx.x; e < R * D; e += kThreadsA) {
      const int row = e / D;
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i <= kWarps; ++i)
        if (i < count) m = fmaxf(m, piece(from[i])[R * D + row]);
      float x = 0.f, l = 0.f;
#pragma unroll
      for (int i = 0; i <= kWarps; ++i)
        if (i < count) {
          const float* p = piece(from[i]);
          const float mi = p[R * D + row], f = mi == -INFINITY ? (m == -INFINITY ? 1.f : 0.f) : ex2(mi - m);
          x = fmaf(f, p[e], x);
          l = fmaf(f, p[R * D + R + row], l);
        }
      const bool one = e - row * D == 0;
      if (begins && ends) {
        finish<D, DT, R>(a, seq, tile, kvh, row, e - row * D, x, l);
        if (one && a.accumulate) {
          a.stats[((size_t)item * R + row) * 2] = m;
          a.stats[((size_t)item * R + row) * 2 + 1] = l;
        }
      } else {
        slot[e] = x;
        if (one) { slot[R * D + row] = m; slot[R * D + R + row] = l; }
      }
    }
  };
#pragma unroll 1
  for (int w = 0; w < kWarps; ++w) {
#pragma unroll
    for (int last = 0; last < 2; ++last) {
      const int it = piece_item[last][w];
      if (it < 0) continue;
      if (count == 0) { item = it; begins = piece_begins[last][w]; who = 2 * w + last; }
      from[count++] = 2 * w + last;
      if (!last) { merge(true); count = 0; }
    }
  }
  if (count) merge(false);
}

// ---- what CTAs share: the first CTA boundary inside an item merges its
// pieces; then, if asked, every key's weights go to its score.
constexpr int kThreadsM = 512;

template <int D, int DT, int R>
__global__ void __launch_bounds__(kThreadsM, 1) kv4_attn_merge_kernel(const AttnArgs a) {
  __shared__ int f_seq[3];
  __shared__ long long f_start[3];
  __shared__ float stat_m[kMaxRows], stat_l[kMaxRows];
  pdl_trigger();
  pdl_wait();
  Line line;
  long long base, mine;
  int s0, s1;
  line_scan<kThreadsM>(a, line, base, mine, s0, s1);
  if (line.total == 0) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_item = a.tiles * a.c.heads;
  // units of all row tiles share their keys: scores go by (sequence, KV head, block)
  const long long keys_total = line.total / a.tiles;
  const long long v0 = keys_total * blockIdx.x / gridDim.x, v1 = keys_total * (blockIdx.x + 1) / gridDim.x;
  const int c = blockIdx.x + 1;   // the boundary between CTAs c - 1 and c
  const int parts = line.ctas * kWarps;
  const long long edge = c < line.ctas ? cut(line, c * kWarps, parts) : -1;
  {
    const long long u[2] = {edge, v0 < v1 && a.accumulate ? v0 * a.tiles : -1};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int seq;
      long long start;
      if (u[i] >= 0 && line_find(a, u[i], base, mine, s0, s1, seq, start)) { f_seq[i] = seq; f_start[i] = start; }
    }
  }
  __syncthreads();

  // CTA whose range holds unit u
  auto cta_of = [&](long long u) {
    int i = (int)(((double)u + 0.5) * line.ctas / line.total);
    i = min(max(i, 0), line.ctas - 1);
    while (i > 0 && u < cut(line, i * kWarps, parts)) --i;
    while (i + 1 < line.ctas && u >= cut(line, (i + 1) * kWarps, parts)) ++i;
    return i;
  };
  // a CTA's piece of an item that goes on behind it is its last, else its first
  auto slot_of = [&](int cta, int c1) { return part_at<D, R>(a.cta_part, (size_t)cta * 2 + (cta < c1 ? 1 : 0)); };

  if (edge >= 0) {
    const int seq = f_seq[0], nb = blocks_of(a.c.len(seq));
    const long long in_seq = edge - f_start[0];
    const int item = (int)(in_seq / nb);
    const long long i0 = f_start[0] + (long long)item * nb, i1 = i0 + nb;
    // strictly inside, and the first such boundary of the item
    if (edge > i0 && cut(line, (c - 1) * kWarps, parts) <= i0) {
      const int c0 = c - 1, c1 = cta_of(i1 - 1);
      const int tile = item / a.c.heads, kvh = item - tile * a.c.heads;
      for (int e = tid; e < R * D; e += kThreadsM) {
        const int row = e / D;
        float m = -INFINITY, x = 0.f, l = 0.f;
        for (int i = c0; i <= c1; ++i) m = fmaxf(m, __ldcg(slot_of(i, c1) + R * D + row));
#pragma unroll 4
        for (int i = c0; i <= c1; ++i) {
          const float* p = slot_of(i, c1);
          const float mi = __ldcg(p + R * D + row), f = mi == -INFINITY ? (m == -INFINITY ? 1.f : 0.f) : ex2(mi - m);
          x = fmaf(f, __ldcg(p + e), x);
          l = fmaf(f, __ldcg(p + R * D + R + row), l);
        }
        finish<D, DT, R>(a, seq, tile, kvh, row, e - row * D, x, l);
      }
    }
  }
  if (!a.accumulate) return;

  long long v = v0;
  int seq = v < v1 ? f_seq[1] : 0;
  long long start = v < v1 ? f_start[1] : 0;   // in units of all row tiles
  while (v < v1) {
    int n = a.c.len(seq);
    while (n == 0) n = a.c.len(++seq);
    const int nb = blocks_of(n);
    const long long in_seq = v - start / a.tiles;
    const int kvh = (int)(in_seq / nb), b0 = (int)(in_seq - (long long)kvh * nb);
    const int b1 = (int)(v1 - v < nb - b0 ? b0 + (v1 - v) : nb);
    // each row's maximum and the reciprocal of its sum, one warp a row
    __syncthreads();
    for (int row = warp; row < a.tiles * R; row += kThreadsM / 32) {
      const int tile = row / R, rr = row - tile * R;
      const int item = tile * a.c.heads + kvh;
      const long long i0 = start + (long long)item * nb;
      const int c0 = cta_of(i0), c1 = cta_of(i0 + nb - 1);
      float m = -INFINITY, l = 0.f;
      if (c0 == c1) {
        const float* p = a.stats + (((size_t)seq * per_item + item) * R + rr) * 2;
        m = __ldcg(p); l = __ldcg(p + 1);
      } else {
        for (int i = c0 + lane; i <= c1; i += 32) m = fmaxf(m, __ldcg(slot_of(i, c1) + R * D + rr));
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        for (int i = c0 + lane; i <= c1; i += 32) {
          const float* p = slot_of(i, c1);
          const float mi = __ldcg(p + R * D + rr);
          l += (mi == -INFINITY ? (m == -INFINITY ? 1.f : 0.f) : ex2(mi - m)) * __ldcg(p + R * D + R + rr);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
      }
      // sums carry the bias of the probabilities; rows behind the last add nothing
      if (lane == 0 && row < kMaxRows) {
        stat_m[row] = m == -INFINITY ? 0.f : m - kBias;
        stat_l[row] = row < a.rows && l != 0.f ? 1.f / l : 0.f;
      }
    }
    __syncthreads();
    float* score = a.c.scores + ((size_t)seq * a.c.heads + kvh) * a.c.capacity();
    for (int key = b0 * kKv4Block + tid; key < min(n, b1 * kKv4Block); key += kThreadsM) {
      float w = 0.f;
      for (int tile = 0; tile < a.tiles; ++tile) {
        const long long unit = start + (long long)(tile * a.c.heads + kvh) * nb + key / kKv4Block;
        const float* s = a.s_all + ((size_t)unit * kKv4Block + key % kKv4Block) * a.s_rows;
        for (int i = 0; i < a.s_rows; i += 2) {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(s + i));
          const int row = tile * R + i;
          if (row < a.rows) w += ex2(x.x - stat_m[row]) * stat_l[row];
          if (row + 1 < a.rows) w += ex2(x.y - stat_m[row + 1]) * stat_l[row + 1];
        }
      }
      score[key] = __ldcg(score + key) + w;
    }
    v += b1 - b0;
    if (b1 == nb && kvh + 1 == a.c.heads) {
      start += (long long)nb * per_item;
      ++seq;
    }
  }
}

struct Layout {
  int R, tiles, s_rows;
  size_t warp_part, cta_part, stats, s_all, bytes;   // byte offsets
};

// Query rows of a KV head: one tile of 8 columns up to 8, else tiles of 16
// (rows beyond share the widened cache of their tile; a tile of 32 would hold
// 128 sums a thread and halve the warps).
Layout layout_of(const mk_kv4_cache* c, int q_len, int group, bool accumulate) {
  Layout l;
  const int rows = q_len * group, d = c->head_dim;
  l.R = rows <= 8 ? 8 : 16;
  l.tiles = (rows + l.R - 1) / l.R;
  l.s_rows = l.tiles > 1 ? l.R : (rows + 1) & ~1;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t part = (size_t)l.R * (d + 2) * sizeof(float);
  size_t at = 0;
  l.warp_part = at; at = up(at + (size_t)kMaxCtas * kWarps * part);
  l.cta_part = at; at = up(at + (size_t)kMaxCtas * 2 * part);
  l.stats = l.s_all = at;
  if (accumulate) {
    const size_t items = (size_t)c->n_seq * l.tiles * c->n_kv_heads;
    at = up(at + items * l.R * 2 * sizeof(float));
    l.s_all = at;
    const size_t blocks = ((size_t)c->pages_per_seq * c->page_tokens + kKv4Block - 1) / kKv4Block;
    at = up(at + items * blocks * kKv4Block * l.s_rows * sizeof(float));
  }
  l.bytes = at;
  return l;
}

int check_shape(const mk_kv4_cache* c, int q_len, int n_q_heads, const char* who) {
  if (int rc = kv4_check(c, who)) return rc;
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "n_q_heads is a multiple of n_kv_heads");
  if (q_len < 1 || (long long)q_len * (n_q_heads / c->n_kv_heads) > kMaxRows)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "q_len times the query heads of a KV head is 1 to 1024");
  return MK_OK;
}

template <int D, int DT, int NT>
cudaError_t launch(const AttnArgs& a, int sms, cudaStream_t st) {
  constexpr int smem = kWarps * kStages * Kv4Shape<D>::kBytes;
  AttnArgs args = a;
  const int ctas = sms * (NT == 1 ? 2 : 1);
  args.max_ctas = ctas < kMaxCtas ? ctas : kMaxCtas;
  cudaError_t e = cudaFuncSetAttribute(kv4_attn_kernel<D, DT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = pdl_launch(kv4_attn_kernel<D, DT, NT>, dim3(args.max_ctas), dim3(kThreadsA), smem, st, args);
  if (e != cudaSuccess) return e;
  return pdl_launch(kv4_attn_merge_kernel<D, DT, 8 * NT>, dim3(args.max_ctas), dim3(kThreadsM), 0, st, args);
}

template <int D, int DT>
cudaError_t launch_rows(const AttnArgs& a, int R, int sms, cudaStream_t st) {
  return R == 8 ? launch<D, DT, 1>(a, sms, st) : launch<D, DT, 2>(a, sms, st);
}

template <int D>
cudaError_t launch_type(const AttnArgs& a, int dtype, int R, int sms, cudaStream_t st) {
  if (dtype == MK_DTYPE_F32) return launch_rows<D, MK_DTYPE_F32>(a, R, sms, st);
  if (dtype == MK_DTYPE_BF16) return launch_rows<D, MK_DTYPE_BF16>(a, R, sms, st);
  return launch_rows<D, MK_DTYPE_F16>(a, R, sms, st);
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" size_t mk_attention_kv4_workspace_bytes(const mk_kv4_cache* cache, int q_len, int n_q_heads,
                                                   int accumulate) {
  if (check_shape(cache, q_len, n_q_heads, "mk_attention_kv4_workspace_bytes")) return 0;
  return layout_of(cache, q_len, n_q_heads / cache->n_kv_heads, accumulate != 0).bytes;
}

extern "C" int mk_attention_kv4(const mk_kv4_cache* cache, const void* q_dev, int dtype, int q_len,
                                int n_q_heads, long long q_stride, float scale, int accumulate,
                                void* workspace_dev, size_t workspace_bytes, void* out_dev, void* stream) {
  const char* who = "mk_attention_kv4";
  if (int rc = check_shape(cache, q_len, n_q_heads, who)) return rc;
  if (dtype != MK_DTYPE_F32 && dtype != MK_DTYPE_BF16 && dtype != MK_DTYPE_F16)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "dtype is one of MK_DTYPE_*");
  if (!q_dev || !out_dev) return kv4_fail(MK_ERR_INVALID_ARG, who, "no queries or output");
  const int esz = dtype == MK_DTYPE_F32 ? 4 : 2;
  if (q_stride < (long long)n_q_heads * cache->head_dim || q_stride > (1ll << 40))
    return kv4_fail(MK_ERR_INVALID_ARG, who, "a token's stride is at least n_q_heads * head_dim");
  if ((reinterpret_cast<uintptr_t>(q_dev) & 15u) || (q_stride * esz) % 16 ||
      (reinterpret_cast<uintptr_t>(out_dev) & (esz - 1)))
    return kv4_fail(MK_ERR_INVALID_ARG, who, "queries of a token are 16-byte aligned, outputs to their type");
  if (!(scale > 0.f) || !(scale <= 3.0e38f)) return kv4_fail(MK_ERR_INVALID_ARG, who, "scale is positive and finite");
  if (accumulate && !cache->scores_dev)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "weights are added to a cache's scores, and this one has none");
  const int group = n_q_heads / cache->n_kv_heads;
  const Layout l = layout_of(cache, q_len, group, accumulate != 0);
  if (!workspace_dev || (reinterpret_cast<uintptr_t>(workspace_dev) & 15u) || workspace_bytes < l.bytes)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "the workspace is 16-byte aligned and of the bytes asked for");
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return kv4_fail(MK_ERR_CUDA, who, "no device");
  uint8_t* ws = static_cast<uint8_t*>(workspace_dev);
  AttnArgs a;
  a.c = kv4_of(cache);
  a.q = static_cast<const uint8_t*>(q_dev);
  a.out = static_cast<uint8_t*>(out_dev);
  a.q_stride = (size_t)q_stride * esz;
  a.q_len = q_len; a.group = group; a.rows = q_len * group; a.tiles = l.tiles;
  a.s_mul = (float)((double)scale * 1.4426950408889634074 * exp2((double)cache->k_log2));
  a.o_mul = (float)exp2((double)cache->v_log2);
  a.max_ctas = 0;
  a.accumulate = accumulate != 0;
  a.warp_part = reinterpret_cast<float*>(ws + l.warp_part);
  a.cta_part = reinterpret_cast<float*>(ws + l.cta_part);
  a.stats = reinterpret_cast<float*>(ws + l.stats);
  a.s_all = reinterpret_cast<float*>(ws + l.s_all);
  a.s_rows = l.s_rows;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->head_dim == 128 ? launch_type<128>(a, dtype, l.R, sms, st)
                                               : launch_type<64>(a, dtype, l.R, sms, st);
  return e == cudaSuccess ? MK_OK : kv4_fail(MK_ERR_CUDA, who, cudaGetErrorString(e));
}

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
// of two that puts its largest element between 2^13 and 2^14.  bf16 elements are then
// exact down to 2^-30 of the largest and fp16 ones to 2^-27; fp32 ones are the sum of two fp16
// parts, 22 bits down to 2^-15 of the largest; anything smaller is off by at most 2^-38 of it
// (half of fp16's last step).  Probabilities, 2^11 to 2^15 at the row's highest score, are
// one fp16 part for bf16 results (an error of 2^-12 beside the result's 2^-9) and two for fp16
// and fp32 (2^-22 down to 2^-13 of the highest); smaller ones are off by at most 2^-36 of it, and
// vanish below that, while the sum still counts them.  Scores, maxima, sums and outputs are fp32.
//
// Work: the blocks of 32 keys of all (sequence, row tile, KV head) items stand
// in one line, each item preceded by a few units for what starting it costs,
// and the line is cut into equal ranges, one for every warp of one wave of
// CTAs -- from the lengths on the device, so ragged batches are balanced and a
// graph may be replayed with other lengths.  A warp keeps its own ring of
// blocks (cp.async, no barrier between warps).  A range that begins or ends
// inside an item leaves a partial (unnormalised output, maximum, sum); the
// warps of a CTA merge theirs in shared memory, and a second kernel merges
// what CTAs share and adds the weights to the scores.  No atomics: results do
// not depend on timing.
#include <math.h>

#include <type_traits>

#include "kv4.cuh"
#include "pdl.cuh"

namespace mk {
namespace {

constexpr int kWarps = 8;
constexpr int kThreadsA = kWarps * 32;
constexpr int kStages = 2;        // blocks of a warp's ring: one loads while the other is used (the code below counts on two)
constexpr int kMaxCtas = 320;     // partials are laid out for this many CTAs
constexpr int kMaxRows = 1024;    // query rows of a KV head: q_len * group
// Probabilities are 2^(S - ref + kBias), S at most kSlack above the reference:
// fp16 holds up to 2^15, with all its bits down to 2^-25 of the reference.
constexpr float kBias = 11.f;
constexpr float kSlack = 4.f;

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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
  float* cta_part;       // [max_ctas][2][R][d + 2]: a CTA's first and last, unfinished
  float2* stats;         // [n_seq * tiles * heads][R]: max and sum of rows that one CTA finished
  float* s_all;          // [units][32][stored rows]: scores in log2 units
  int32_t s_rows;
  // what the first kernel found out, for the second
  int4* line;            // total, each, rest, ctas (Line)
  int4* edges;           // [max_ctas]: the item that a CTA leaves unfinished: sequence, item, first block's
                         // unit, blocks; item -1: none
  int4* begins;          // [max_ctas]: where a CTA's share of the scores begins: sequence, its first unit, keys
};

// Starting an item (its pages, its queries, its result) takes about as long as
// this many blocks; with items of one block and no such units, a warp that got 14
// of them ran 10 times as long as one with 14 blocks of a long item.
constexpr int kStart = 3;

// The line of units: sequence by sequence, in it row tile by row tile, KV head
// by KV head: kStart units, then the item's blocks.
struct Line {
  int32_t total, each, rest;   // units; per range, and ranges that get one more
  int32_t ctas;                // CTAs that have any: kWarps units each, or all
  __device__ __forceinline__ int cut(int i) const { return each * i + min(i, rest); }
  // range that holds unit u
  __device__ __forceinline__ int range_of(int u) const {
    const int big = (each + 1) * rest;
    return u < big ? u / (each + 1) : rest + (u - big) / each;
  }
  __device__ __forceinline__ int cta_of(int u) const { return range_of(u) / kWarps; }
};

// First unit of a CTA's share of the scores.
__device__ __forceinline__ int scores_cut(int total, int i, int ctas) { return (int)((long long)total * i / ctas); }

__device__ __forceinline__ int blocks_of(int n) { return (n + kKv4Block - 1) / kKv4Block; }
__device__ __forceinline__ int units_of(int n) { return n ? blocks_of(n) + kStart : 0; }

// One warp's view of the line: lane i holds a run of consecutive sequences, `base`
// the units before them, n the keys of the first.
struct Scan {
  int32_t s0, s1, base, mine, n;
};

__device__ __forceinline__ Scan line_scan(const AttnArgs& a, Line& l) {
  const int lane = threadIdx.x & 31;
  const int run = (a.c.n_seq + 31) >> 5, items = a.tiles * a.c.heads;
  Scan z;
  z.s0 = min(a.c.n_seq, lane * run);
  z.s1 = min(a.c.n_seq, z.s0 + run);
  z.n = z.s0 < z.s1 ? a.c.len(z.s0) : 0;
  z.mine = units_of(z.n);
#pragma unroll 4
  for (int s = z.s0 + 1; s < z.s1; ++s) z.mine += units_of(a.c.len(s));
  z.mine *= items;
  int inc = z.mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += up;
  }
  z.base = inc - z.mine;
  l.total = __shfl_sync(0xFFFFFFFFu, inc, 31);
  const int want = (l.total + kWarps - 1) / kWarps;
  l.ctas = min(want, a.max_ctas);
  const int parts = max(l.ctas * kWarps, 1);
  l.each = l.total / parts;
  l.rest = l.total - l.each * parts;
  return z;
}

// The sequence that unit u lies in, the units before it and its keys.
__device__ __forceinline__ void line_find(const AttnArgs& a, const Scan& z, int u, int& seq, int& start, int& n) {
  const bool here = u >= z.base && u < z.base + z.mine;
  int s = z.s0, b = z.base, m = z.n;
  if (here && z.s0 + 1 < z.s1) {
    const int items = a.tiles * a.c.heads;
    for (;;) {
      const int len = units_of(m) * items;
      if (u < b + len) break;
      b += len;
      m = a.c.len(++s);
    }
  }
  const int who = max(__ffs(__ballot_sync(0xFFFFFFFFu, here)) - 1, 0);
  seq = __shfl_sync(0xFFFFFFFFu, s, who);
  start = __shfl_sync(0xFFFFFFFFu, b, who);
  n = __shfl_sync(0xFFFFFFFFu, m, who);
}

// Four (or N) consecutive output elements, rounded once.
template <int DT, int N>
__device__ __forceinline__ void store_out(uint8_t* out, size_t at, const float (&x)[N]) {
  if (DT == MK_DTYPE_F32) {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
    uint2* p = reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(out) + at);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      uint32_t w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (DT == MK_DTYPE_BF16)
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(x[4 * i + 2 * j + 1]), "f"(x[4 * i + 2 * j]));
        else
          w[j] = pack_half2(x[4 * i + 2 * j], x[4 * i + 2 * j + 1]);
      }
      p[i] = make_uint2(w[0], w[1]);
    }
  }
}

// Element offset of an output row, false behind the last.
template <int D, int R>
__device__ __forceinline__ bool out_row(const AttnArgs& a, int seq, int tile, int kvh, int n, size_t& at) {
  const int row = tile * R + n, token = row / a.group, head = row - token * a.group;
  at = (((size_t)seq * a.q_len + token) * a.c.heads * a.group + (size_t)kvh * a.group + head) * D;
  return row < a.rows;
}

// What a sum of weighted values is multiplied with; a row that sees nothing
// has sum 0, NaN goes through.
__device__ __forceinline__ float inverse(const AttnArgs& a, float sum) { return sum == 0.f ? 0.f : a.o_mul / sum; }

// What is added to a score to get its probability's exponent.  Rounded down: with a reference
// past 2^24 the bias goes (the nearest step of fp32 could be 16 above it), and a
// probability stays below 2^16.  No reference yet: nothing is added.
__device__ __forceinline__ float exponent_of(float ref) { return ref == -INFINITY ? 0.f : __fadd_rd(kBias, -ref); }

// Weight of a partial with maximum mi under the common maximum m.
__device__ __forceinline__ float rescale(float mi, float m) {
  return mi == -INFINITY ? (m == -INFINITY ? 1.f : 0.f) : ex2(mi - m);
}

template <int D, int R>
__device__ __forceinline__ float* part_at(float* base, int i) { return base + (size_t)i * (R * (D + 2)); }

__device__ __forceinline__ uint32_t scaled(uint32_t codes, __half2 s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&codes), s);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ __half2 scales2(uint32_t two) {
  const uint32_t h = e4m3x2(two);
  return *reinterpret_cast<const __half2*>(&h);
}

// Shared memory of a warp: the ring and behind it the query fragments (more than
// one 8-row tile), which a last piece may overwrite; a first piece.
template <int D, int DT, int NT>
struct AttnSmem {
  static constexpr int kRing = kStages * Kv4Shape<D>::kBytes;
  static constexpr int kQ = NT > 1 ? (DT == MK_DTYPE_F32 ? 2 : 1) * NT * (D / 32) * 512 : 0;
  static constexpr int kPiece = 8 * NT * D * 4;
  static constexpr int kFirst = kRing + kQ > kPiece ? kRing + kQ : kPiece;
  static constexpr int kWarp = kFirst + kPiece;
  static constexpr int kBytes = kWarps * kWarp;
};

// D: head dim.  DT: MK_DTYPE_* of queries and outputs.  NT: 8-row tiles of query rows.
template <int D, int DT, int NT>
__global__ void __launch_bounds__(kThreadsA, NT == 1 ? 2 : 1) kv4_attn_kernel(const AttnArgs a) {
  using S = Kv4Shape<D>;
  constexpr int R = 8 * NT;
  constexpr int QP = DT == MK_DTYPE_F32 ? 2 : 1;   // fp16 parts of a query
  constexpr int PP = DT == MK_DTYPE_BF16 ? 1 : 2;  // and of a probability
  constexpr int KS = D / 16;                       // contraction steps, and 16-dim tiles of O
  using M = AttnSmem<D, DT, NT>;
  // Query fragments: registers for one row tile; for more, shared memory, which both
  // halves of a block read them from once
  constexpr bool kQShared = NT > 1;
  extern __shared__ __align__(16) uint8_t ring_all[];
  // pieces that a warp leaves: even its first, in a place of its own, odd its last, in its ring's
  __shared__ int4 piece_of[2 * kWarps];    // sequence, item (-1: none), first block's unit, blocks
  __shared__ float piece_max[2 * kWarps][R], piece_sum[2 * kWarps][R];
  __shared__ float total[R];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, t = lane & 3;
  Line line;
  const Scan scan = line_scan(a, line);
  const int items = a.tiles * a.c.heads;

  if (blockIdx.x == 0 && threadIdx.x == 0) *a.line = make_int4(line.total, line.each, line.rest, line.ctas);
  if (a.accumulate && warp == kWarps - 1) {
    // units of all row tiles share their keys: the line without row tiles
    const int v = scores_cut(line.total / a.tiles, blockIdx.x, gridDim.x);
    int4 z;
    line_find(a, scan, v * a.tiles, z.x, z.y, z.z);
    if (lane == 0) a.begins[blockIdx.x] = z;
  }
  if ((int)blockIdx.x >= line.ctas) {
    if (threadIdx.x == 0) a.edges[blockIdx.x] = make_int4(0, -1, 0, 0);
    return;
  }

  // this warp's range
  int u = line.cut(blockIdx.x * kWarps + warp);
  const int u_end = line.cut(blockIdx.x * kWarps + warp + 1);
  int seq = 0, start = 0, n = 0;
  if (u < u_end) line_find(a, scan, u, seq, start, n);
  if (lane < 2) piece_of[2 * warp + lane] = make_int4(0, -1, 0, 0);

  uint8_t* ring = ring_all + warp * M::kWarp;
  uint4* q_shared = reinterpret_cast<uint4*>(ring + M::kRing) + lane;
  const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const int per = a.c.page_tokens / kKv4Block;

  while (u < u_end) {
    // ---- the piece of one item that this range covers
    while (n == 0) n = a.c.len(++seq);   // u < total: a sequence with keys follows
    const int nb = blocks_of(n);
    const int item = (u - start) / (nb + kStart), item_at = start + item * (nb + kStart);
    const int tile = item / a.c.heads, kvh = item - tile * a.c.heads;
    const int stop = min(u_end, item_at + nb + kStart);
    const int b0 = max(u - item_at - kStart, 0), b1 = stop - item_at - kStart;
    const bool last_item = item + 1 == items;
    u = stop;
    const bool ends = b1 == nb;
    const int this_seq = seq, this_n = n;
    if (ends && last_item) {
      start += (nb + kStart) * items;
      ++seq;
      n = u < u_end ? a.c.len(seq) : 0;
    }
    if (b1 <= b0) continue;   // units of the start alone

    // ---- query rows: column r of each 8-row tile, 4 * KS dims from t * 4 * KS; in flight
    // while the pages are looked up
    constexpr int kRaw = KS * (DT == MK_DTYPE_F32 ? 1 : 2) / (DT == MK_DTYPE_F32 ? 1 : 4);
    uint4 raw[NT][kRaw];
    int lim[NT];
    bool row_ok[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = tile * R + nt * 8 + r, token = row / a.group, head = row - token * a.group;
      row_ok[nt] = row < a.rows;
      lim[nt] = row_ok[nt] ? max(0, min(this_n, this_n - a.q_len + token + 1)) : this_n;
      const uint8_t* p = a.q + ((size_t)this_seq * a.q_len + token) * a.q_stride +
                         (size_t)((kvh * a.group + head) * D + t * 4 * KS) * (DT == MK_DTYPE_F32 ? 4 : 2);
#pragma unroll
      for (int i = 0; i < kRaw; ++i)
        raw[nt][i] = row_ok[nt] ? __ldcg(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0u, 0u, 0u, 0u);
    }

    // ---- the ring: block b of the item is in_page blocks into logical page lp;
    // lane i holds the physical page of lp0 + i
    int lp0 = b0 / per, rel = 0, in_page = b0 - lp0 * per;
    const int lp_last = (b1 - 1) / per;
    int pages = lp0 + lane <= lp_last ? a.c.page(this_seq, lp0 + lane) : -1;
    int page = __shfl_sync(0xFFFFFFFFu, pages, 0);
    uint32_t fill = ring_s;
    auto issue = [&]() {   // the next block into the ring slot at `fill`; false where it has no page
      if (page >= 0) {
        const uint8_t* src = kv4_block<D>(a.c, page, kvh, in_page) + lane * 16;
        const uint32_t dst = fill + lane * 16;
#pragma unroll
        for (int i = 0; i < (S::kBytes / 16 + 31) / 32; ++i)
          if (S::kBytes / 16 % 32 == 0 || i * 32 + lane < S::kBytes / 16) cp16(dst + i * 512, src + i * 512);
      }
      const bool there = page >= 0;
      fill = fill == ring_s + (kStages - 1) * S::kBytes ? ring_s : fill + S::kBytes;
      if (++in_page == per) {
        in_page = 0;
        if (++rel == 32) {
          rel = 0;
          lp0 += 32;
          pages = lp0 + lane <= lp_last ? a.c.page(this_seq, lp0 + lane) : -1;
        }
        page = __shfl_sync(0xFFFFFFFFu, pages, rel);
      }
      return there;
    };
    uint32_t have = 0;   // bit i: the block i ahead of the current one has a page
    __syncwarp();        // the slots' last readers are done
    // One block now, the next when this one is in: copies are served in order, so a warp's
    // second block would hold up the first one of the warps behind it.
    if (issue()) have |= 1u;
    cp_commit();

    uint32_t qf[QP][kQShared ? 1 : NT][2 * KS];
    float mul[NT][2];                // S -> log2 units, for this thread's columns 2t, 2t + 1
    int limit[NT][2];                // keys those columns see
    int see_all = this_n;            // keys that every row sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[4 * KS];
#pragma unroll
      for (int i = 0; i < kRaw; ++i) {
        const uint32_t w[4] = {raw[nt][i].x, raw[nt][i].y, raw[nt][i].z, raw[nt][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (DT == MK_DTYPE_F32) x[4 * i + j] = __uint_as_float(w[j]);
          else if (DT == MK_DTYPE_BF16) {
            x[(8 * i + 2 * j) % (4 * KS)] = __uint_as_float(w[j] << 16);
            x[(8 * i + 2 * j + 1) % (4 * KS)] = __uint_as_float(w[j] & 0xFFFF0000u);
          } else {
            const float2 f = unpack_half2(w[j]);
            x[(8 * i + 2 * j) % (4 * KS)] = f.x;
            x[(8 * i + 2 * j + 1) % (4 * KS)] = f.y;
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
      // A row with an infinity becomes NaN, as one with a NaN is: scores that were all
      // -inf would pass for those of a row that sees nothing.
      const float up = top <= 3.402823466e38f ? __int_as_float((127 + e) << 23) : __int_as_float(0x7FC00000);
      // not 0: masked scores are -inf and their product has to stay it; at most 2^94:
      // a product q k is below 2^33 (14 + 11.4 + 7 bits), so no score passes fp32's range.
      // What is cut still tells scores apart: they are multiples of 2^-34, and 2^60 log2 units
      // are as good as any number of them.
      const float down = fminf(fmaxf(__int_as_float((127 - e) << 23) * a.s_mul, 1.17549435e-38f), 1.9807040628566084e28f);
#pragma unroll
      for (int i = 0; i < 2 * KS; ++i) {
        const float f0 = x[2 * i] * up, f1 = x[2 * i + 1] * up;
        const uint32_t h = pack_half2(f0, f1);
        qf[0][kQShared ? 0 : nt][i] = h;
        if (QP == 2) {
          const float2 b = unpack_half2(h);
          qf[QP - 1][kQShared ? 0 : nt][i] = pack_half2(f0 - b.x, f1 - b.y);
        }
      }
      if (kQShared) {
#pragma unroll
        for (int p = 0; p < QP; ++p)
#pragma unroll
          for (int w = 0; w < KS / 2; ++w)
            q_shared[((p * NT + nt) * (KS / 2) + w) * 32] =
                make_uint4(qf[p][0][4 * w], qf[p][0][4 * w + 1], qf[p][0][4 * w + 2], qf[p][0][4 * w + 3]);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mul[nt][c] = __shfl_sync(0xFFFFFFFFu, down, (2 * t + c) * 4);
        limit[nt][c] = __shfl_sync(0xFFFFFFFFu, lim[nt], (2 * t + c) * 4);
      }
      see_all = min(see_all, lim[nt]);
    }
    see_all = __reduce_min_sync(0xFFFFFFFFu, see_all);

    float o[NT][KS][4];
    float ref[NT][2], sum[NT][2];    // reference of the probabilities (log2 units), their sum
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][j][i] = 0.f;
      ref[nt][0] = ref[nt][1] = -INFINITY;
      sum[nt][0] = sum[nt][1] = 0.f;
    }
    // this thread's keys of a half block: mma rows r and r + 8
    const int key_r = (r >> 1) + (r & 1) * 4;
    float* s_to = a.accumulate
                      ? a.s_all + ((size_t)(item_at + kStart + b0) * kKv4Block + key_r) * a.s_rows + 2 * t : nullptr;
    const uint8_t* blk = ring;

    for (int b = b0; b < b1; ++b) {
      cp_wait<kStages - 2>();
      __syncwarp();
      if (b + kStages - 1 < b1 && issue()) have |= 1u << (kStages - 1);
      cp_commit();
      const bool there = have & 1u;
      have >>= 1;
      const bool masked = !there || (b + 1) * kKv4Block > see_all;   // some row does not see some key

      // S^T: 16 keys (a half) are an mma's rows; a word holds 8 of a key's dims
      float sc[2][NT][4];
      {
        uint32_t wa[2][KS / 2], wb[2][KS / 2];   // keys of mma rows r and r + 8
        __half2 sa[2], sb[2];   // scales of this thread's two groups (d = 64: one)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int ka = half * 16 + key_r, kb = ka + 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[half][nt][i] = 0.f;
          if (D == 128) {
            const uint4 va = *reinterpret_cast<const uint4*>(blk + ka * S::kCodes + t * 16);
            const uint4 vb = *reinterpret_cast<const uint4*>(blk + kb * S::kCodes + t * 16);
            wa[half][0] = va.x; wa[half][1] = va.y; wa[half][KS / 2 - 2] = va.z; wa[half][KS / 2 - 1] = va.w;
            wb[half][0] = vb.x; wb[half][1] = vb.y; wb[half][KS / 2 - 2] = vb.z; wb[half][KS / 2 - 1] = vb.w;
            sa[half] = scales2(*reinterpret_cast<const uint16_t*>(blk + S::kKs + ka * S::kScales + 2 * t));
            sb[half] = scales2(*reinterpret_cast<const uint16_t*>(blk + S::kKs + kb * S::kScales + 2 * t));
          } else {
            const uint2 va = *reinterpret_cast<const uint2*>(blk + ka * S::kCodes + t * 8);
            const uint2 vb = *reinterpret_cast<const uint2*>(blk + kb * S::kCodes + t * 8);
            wa[half][0] = va.x; wa[half][1] = va.y; wb[half][0] = vb.x; wb[half][1] = vb.y;
            sa[half] = scales2(blk[S::kKs + ka * S::kScales + t]);
            sb[half] = scales2(blk[S::kKs + kb * S::kScales + t]);
          }
        }
#pragma unroll
        for (int w = 0; w < KS / 2; ++w) {
          uint4 qw[QP][NT];
#pragma unroll
          for (int p = 0; p < QP; ++p)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t* f = qf[p][kQShared ? 0 : nt];
              qw[p][nt] = kQShared ? q_shared[((p * NT + nt) * (KS / 2) + w) * 32]
                                   : make_uint4(f[4 * w], f[4 * w + 1], f[4 * w + 2], f[4 * w + 3]);
            }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t ha[4], hb[4];
            e2m1x8(wa[half][w], ha);
            e2m1x8(wb[half][w], hb);
            // 16 dims, two words, share a scale
            const __half2 pa = w < 2 ? __low2half2(sa[half]) : __high2half2(sa[half]);
            const __half2 pb = w < 2 ? __low2half2(sb[half]) : __high2half2(sb[half]);
#pragma unroll
            for (int i = 0; i < 4; ++i) { ha[i] = scaled(ha[i], pa); hb[i] = scaled(hb[i], pb); }
#pragma unroll
            for (int p = 0; p < QP; ++p)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816(sc[half][nt], ha[0], hb[0], ha[1], hb[1], qw[p][nt].x, qw[p][nt].y);
                mma16816(sc[half][nt], ha[2], hb[2], ha[3], hb[3], qw[p][nt].z, qw[p][nt].w);
              }
          }
        }
      }

      if (masked) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = b * kKv4Block + half * 16 + key_r + 8 * i;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (!there || key >= limit[nt][c]) sc[half][nt][2 * i + c] = -INFINITY;
          }
      }
      if (a.accumulate) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (nt * 8 + 2 * t < a.s_rows)
                *reinterpret_cast<float2*>(s_to + (half * 16 + 8 * i) * a.s_rows + nt * 8) =
                    make_float2(sc[half][nt][2 * i] * mul[nt][0], sc[half][nt][2 * i + 1] * mul[nt][1]);
        s_to += kKv4Block * a.s_rows;
      }

      // The reference of a column moves only when a score passes it by kSlack:
      // then, and in the first block, the lanes' maxima meet.
      float top[NT][2];
      bool moves = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          top[nt][c] = __fmul_rn(mul[nt][c], fmaxf(fmaxf(sc[0][nt][c], sc[0][nt][2 + c]), fmaxf(sc[1][nt][c], sc[1][nt][2 + c])));
          moves |= top[nt][c] - ref[nt][c] > kSlack;
        }
      if (__any_sync(0xFFFFFFFFu, moves)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float m = top[nt][c];
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
            m = fmaxf(m, ref[nt][c]);
            const float f = ref[nt][c] == -INFINITY ? 1.f : ex2(ref[nt][c] - m);   // nothing to rescale before the first
            ref[nt][c] = m;
            sum[nt][c] *= f;
#pragma unroll
            for (int j = 0; j < KS; ++j) { o[nt][j][c] *= f; o[nt][j][2 + c] *= f; }
          }
      }

      // P^T as the mma's columns
      uint32_t pf[PP][2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // Scores are rounded before the reference is taken off, as the reference was: one
        // fma would keep bits that the reference has lost, many log2 units of a large score.
        const float m0 = exponent_of(ref[nt][0]), m1 = exponent_of(ref[nt][1]);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p0 = ex2(__fadd_rn(__fmul_rn(sc[half][nt][2 * i], mul[nt][0]), m0));
            const float p1 = ex2(__fadd_rn(__fmul_rn(sc[half][nt][2 * i + 1], mul[nt][1]), m1));
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
      bool some_nan = false;   // among the values that only some rows see
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
        }
        if (masked) {
          // A value that no row sees must not count, whatever it is (a page's
          // leftovers may be NaN, and 0 * NaN is).  One that only some rows
          // see is NaN for those alone: it leaves the product and is set below.
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = b * kKv4Block + half * 16 + t + 4 * i;
            const bool apart = there && at >= see_all && at < this_n && (s[i] & 0x7Fu) == 0x7Fu;
            if (!there || at >= this_n || apart) s[i] = 0u;
            some_nan |= apart;
          }
        }
        const __half2 s01 = scales2(s[0] | s[1] << 8), s23 = scales2(s[2] | s[3] << 8);
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
            a0[j] = scaled(a0[j], s01); a1[j] = scaled(a1[j], s01);
            a2[j] = scaled(a2[j], s23); a3[j] = scaled(a3[j], s23);
#pragma unroll
            for (int p = 0; p < PP; ++p)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(o[nt][4 * x + j], a0[j], a1[j], a2[j], a3[j], pf[p][half][nt][0], pf[p][half][nt][1]);
          }
        }
      }
      if (masked && __any_sync(0xFFFFFFFFu, some_nan)) {
        for (int at = max(see_all, b * kKv4Block); at < min(this_n, (b + 1) * kKv4Block); ++at) {
          const int key = at - b * kKv4Block;
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
      blk = blk == ring + (kStages - 1) * S::kBytes ? ring : blk + S::kBytes;
    }
    cp_wait<0>();
    __syncwarp();

    // ---- the piece is done: sums over the lanes that share a column
    const bool begins = b0 == 0;
    float* to = reinterpret_cast<float*>(ring + (ends ? M::kFirst : 0));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = sum[nt][c];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
        const int col = nt * 8 + 2 * t + c;
        // lane r holds D / 8 consecutive dims of it, two of each 16-dim tile
        float y[D / 8];
#pragma unroll
        for (int j = 0; j < KS; ++j) { y[2 * j] = o[nt][j][c]; y[2 * j + 1] = o[nt][j][2 + c]; }
        if (begins && ends) {
          size_t at;
          if (out_row<D, R>(a, this_seq, tile, kvh, col, at)) {
            const float f = inverse(a, x);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) y[i] *= f;
            store_out<DT, D / 8>(a.out, at + r * (D / 8), y);
          }
          if (a.accumulate && r == 0) {
            a.stats[((size_t)this_seq * items + item) * R + col] = make_float2(ref[nt][c], x);
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            *reinterpret_cast<float4*>(to + col * D + r * (D / 8) + 4 * i) =
                make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          if (r == 0) {
            piece_max[2 * warp + !ends][col] = ref[nt][c];
            piece_sum[2 * warp + !ends][col] = x;
          }
        }
      }
    if (lane == 0 && !(begins && ends))
      piece_of[2 * warp + !ends] = make_int4(this_seq, item, item_at + kStart, begins ? -nb : nb);   // < 0: begins here
  }
  __syncthreads();

  // ---- pieces of the CTA's warps that belong together, in order: the last of
  // a warp, those of warps that lie whole in the item, the first of the one
  // where it ends
  // pieces in `mask`, in order: `count` of warps that follow one another; the final
  // one ends the item, or not
  auto merge = [&](uint32_t mask, bool ends) {
    const int c0 = __ffs(mask) - 1, count = __popc(mask);
    const int4 who = piece_of[c0];
    const bool done = who.w < 0 && ends;   // begins and ends in this CTA
    const int tile = who.y / a.c.heads, kvh = who.y - tile * a.c.heads;
    const int rows = min(R, a.rows - tile * R);
    float* slot = part_at<D, R>(a.cta_part, blockIdx.x * 2 + (ends ? 0 : 1));
    // weights: 16 lanes to a row, a possible piece each
    for (int row = threadIdx.x >> 4; row < (R + 15) / 16 * 16; row += kThreadsA / 16) {
      const int code = threadIdx.x & 15;
      const bool in = row < R && (mask >> code & 1u);
      const float mi = in ? piece_max[code][row] : -INFINITY;
      float m = mi;
#pragma unroll
      for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const float f = in ? rescale(mi, m) : 0.f;
      float l = in ? f * piece_sum[code][row] : 0.f;
#pragma unroll
      for (int o = 8; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
      if (in) piece_max[code][row] = f;   // from here on its weight
      if (code == 0 && row < R) {
        total[row] = l;
        if (!done) {
          slot[R * D + row] = m;
          slot[R * D + R + row] = l;
        } else if (a.accumulate) {
          a.stats[((size_t)who.x * items + who.y) * R + row] = make_float2(m, l);
        }
      }
    }
    if (!ends && threadIdx.x == 0) a.edges[blockIdx.x] = make_int4(who.x, who.y, who.z, abs(who.w));
    __syncthreads();
    for (int e = threadIdx.x * 4; e < rows * D; e += kThreadsA * 4) {
      const int row = e / D;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int i = 0; i < count; ++i) {
        const int code = i == 0 ? c0 : (c0 & ~1) + 2 * i + (ends && i == count - 1 ? 0 : 1);
        const float4 v = *reinterpret_cast<const float4*>(ring_all + (code >> 1) * M::kWarp + (code & 1 ? 0 : M::kFirst) + e * 4);
        const float f = piece_max[code][row];
        x[0] = fmaf(f, v.x, x[0]); x[1] = fmaf(f, v.y, x[1]);
        x[2] = fmaf(f, v.z, x[2]); x[3] = fmaf(f, v.w, x[3]);
      }
      if (done) {
        size_t at;
        out_row<D, R>(a, who.x, tile, kvh, row, at);
        const float f = inverse(a, total[row]);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] *= f;
        store_out<DT, 4>(a.out, at + e - row * D, x);
      } else {
        *reinterpret_cast<float4*>(slot + e) = make_float4(x[0], x[1], x[2], x[3]);
      }
    }
    __syncthreads();   // the sums are free
  };
  uint32_t pieces = __ballot_sync(0xFFFFFFFFu, lane < 2 * kWarps && piece_of[lane & (2 * kWarps - 1)].y >= 0);
  bool open = false;
#pragma unroll 1
  while (pieces) {   // up to the next first piece (an even one), which ends its item
    const uint32_t even = pieces & 0x55555555u;
    const uint32_t now = even ? pieces & (even ^ (even - 1u)) : pieces;
    merge(now, even != 0u);
    pieces &= ~now;
    open = even == 0u;
  }
  if (!open && threadIdx.x == 0) a.edges[blockIdx.x] = make_int4(0, -1, 0, 0);
}

// ---- what CTAs share.  Blocks [0, max_ctas): the CTAs that leave an item
// unfinished split its merge among them (and zero what no unit covers).
// Blocks behind them, if asked: every key's weights go to its score.  All they
// read of the first kernel's is found by one load, so that the rest is in
// flight at once.
constexpr int kThreadsM = 256;
constexpr int kWarpsM = kThreadsM / 32;

// Running (maximum, sum) pairs of two partials.
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2);
  l = l * rescale(m, top) + l2 * rescale(m2, top);
  m = top;
}

template <int D, int DT, int R>
__global__ void __launch_bounds__(kThreadsM, 4) kv4_attn_merge_kernel(const AttnArgs a) {
  __shared__ float2 stat[kMaxRows + 24];
  pdl_trigger();
  pdl_wait();
  const bool merges = (int)blockIdx.x < a.max_ctas;
  const int me = merges ? blockIdx.x : blockIdx.x - a.max_ctas;
  const int4 head = __ldcg(a.line), rec = __ldcg((merges ? a.edges : a.begins) + me);
  const Line line = {head.x, head.y, head.z, head.w};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = a.tiles * a.c.heads;
  // a CTA's piece of an item that goes on behind it is its last, else its first
  auto slot_of = [&](int cta, int c1) { return part_at<D, R>(a.cta_part, cta * 2 + (cta < c1 ? 1 : 0)); };

  if (merges) {
    // sequences without a key: their outputs are zero and no unit covers them
    for (int s = blockIdx.x; s < a.c.n_seq; s += a.max_ctas) {
      if (a.c.len(s) > 0) continue;
      const size_t n = (size_t)a.rows * a.c.heads * D;
      const float zero[4] = {0.f, 0.f, 0.f, 0.f};
      for (size_t i = tid * 4; i < n; i += kThreadsM * 4) store_out<DT, 4>(a.out, s * n + i, zero);
    }
    if (rec.y < 0) return;
    const int seq = rec.x, item = rec.y, i0 = rec.z, nb = rec.w;
    const int c0 = line.cta_of(i0), c1 = line.cta_of(i0 + nb - 1);   // c0 <= me < c1
    const int tile = item / a.c.heads, kvh = item - tile * a.c.heads;
    const int fours = min(R, a.rows - tile * R) * D / 4, share = c1 - c0;
    const int e0 = fours * (me - c0) / share, e1 = fours * (me - c0 + 1) / share;
    // `wide` lanes to four elements, up to 4 partials each (their loads in flight together)
    int wide = 1;
    while (wide < 32 && wide * 4 < c1 - c0 + 1) wide <<= 1;
    const int sub = lane & (wide - 1), at_once = kWarpsM * (32 / wide);
    for (int base = e0; base < e1; base += at_once) {   // the same number of rounds for every lane
      const int e = base + warp * (32 / wide) + lane / wide;
      const bool ok = e < e1;
      const int row = ok ? e * 4 / D : 0;
      float m = -INFINITY, l = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
      if (ok) {
#pragma unroll 4
        for (int i = c0 + sub; i <= c1; i += wide) {
          const float* p = slot_of(i, c1);
          const float4 v = __ldcg(reinterpret_cast<const float4*>(p) + e);
          const float m2 = __ldcg(p + R * D + row), l2 = __ldcg(p + R * D + R + row);
          const float top = fmaxf(m, m2), f = rescale(m, top), g = rescale(m2, top);
          m = top;
          l = fmaf(g, l2, l * f);
          x[0] = fmaf(g, v.x, x[0] * f); x[1] = fmaf(g, v.y, x[1] * f);
          x[2] = fmaf(g, v.z, x[2] * f); x[3] = fmaf(g, v.w, x[3] * f);
        }
      }
      for (int s = wide >> 1; s; s >>= 1) {
        const float m2 = __shfl_xor_sync(0xFFFFFFFFu, m, s), l2 = __shfl_xor_sync(0xFFFFFFFFu, l, s);
        const float top = fmaxf(m, m2), f = rescale(m, top), g = rescale(m2, top);
        m = top;
        l = f * l + g * l2;
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = f * x[k] + g * __shfl_xor_sync(0xFFFFFFFFu, x[k], s);
      }
      if (ok && sub == 0) {
        size_t at;
        out_row<D, R>(a, seq, tile, kvh, row, at);
        const float f = inverse(a, l);
        const float y[4] = {x[0] * f, x[1] * f, x[2] * f, x[3] * f};
        store_out<DT, 4>(a.out, at + e * 4 - row * D, y);
      }
    }
    return;
  }

  const int keys_total = line.total / a.tiles;
  int v = scores_cut(keys_total, me, a.max_ctas);
  const int v_end = scores_cut(keys_total, me + 1, a.max_ctas);
  if (v >= v_end) return;
  int seq = rec.x, start = rec.y, n = rec.z;   // start: in units of all row tiles
  while (v < v_end) {
    while (n == 0) n = a.c.len(++seq);
    const int nb = blocks_of(n), in_seq = v - start / a.tiles;
    const int kvh = in_seq / (nb + kStart), head_at = start / a.tiles + kvh * (nb + kStart);
    const int stop = min(v_end, head_at + nb + kStart);
    const int b0 = max(v - head_at - kStart, 0), b1 = stop - head_at - kStart;
    if (b1 > b0) {
      const int k0 = b0 * kKv4Block + tid, k_end = min(n, b1 * kKv4Block);
      float* score = a.c.scores + ((size_t)seq * a.c.heads + kvh) * a.c.capacity();
      // up to 8 rows: the scores of this thread's first keys load beside the statistics
      constexpr int kAhead = R == 8 ? 4 : 0;
      float2 s[kAhead + 1][4];
      float old[kAhead + 1];
      const float* s_at = a.s_all + (size_t)(start + kvh * (nb + kStart) + kStart) * kKv4Block * a.s_rows;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int key = k0 + i * kThreadsM;
        if (key < k_end) {
          old[i] = __ldcg(score + key);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (2 * j < a.s_rows) s[i][j] = __ldcg(reinterpret_cast<const float2*>(s_at + (size_t)key * a.s_rows) + j);
        }
      }
      // each row's maximum and the reciprocal of its sum, one warp a row
      __syncthreads();
      for (int row = warp; row < a.rows; row += kWarpsM) {
        const int tile = row / R, rr = row - tile * R, item = tile * a.c.heads + kvh;
        const int i0 = start + item * (nb + kStart) + kStart;
        const int c0 = line.cta_of(i0), c1 = line.cta_of(i0 + nb - 1);
        float m = -INFINITY, l = 0.f;
        if (c0 == c1) {
          const float2 st = __ldcg(a.stats + ((size_t)seq * items + item) * R + rr);
          m = st.x; l = st.y;
        } else {
#pragma unroll 2
          for (int i = c0 + lane; i <= c1; i += 32) {
            const float* p = slot_of(i, c1) + R * D + rr;
            join(m, l, __ldcg(p), __ldcg(p + R));
          }
#pragma unroll
          for (int o = 16; o; o >>= 1)
            join(m, l, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, l, o));
        }
        // Sums carry the bias of the probabilities.  No maximum: every score that the row sees is
        // NaN (a bad query), or it sees none.  A factor of 1 then, as a NaN sum would spread to the
        // keys that it does not see (score -inf, whose weight is 0).
        if (lane == 0) stat[row] = make_float2(exponent_of(m), m == -INFINITY ? 1.f : 1.f / l);
      }
      __syncthreads();
      auto weigh = [&](float w, float2 x, int row) {
        if (row < a.rows) w = fmaf(ex2(x.x + stat[row].x), stat[row].y, w);
        if (row + 1 < a.rows) w = fmaf(ex2(x.y + stat[row + 1].x), stat[row + 1].y, w);
        return w;
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int key = k0 + i * kThreadsM;
        if (key < k_end) {
          float w = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (2 * j < a.s_rows) w = weigh(w, s[i][j], 2 * j);
          score[key] = old[i] + w;
        }
      }
      for (int key = k0 + kAhead * kThreadsM; key < k_end; key += kThreadsM) {
        const float was = __ldcg(score + key);
        float w = 0.f;
        for (int tile = 0; tile < a.tiles; ++tile) {
          const float* p = s_at + ((size_t)tile * a.c.heads * (nb + kStart) * kKv4Block + key) * a.s_rows;
#pragma unroll 4
          for (int i = 0; i < a.s_rows; i += 2)
            w = weigh(w, __ldcg(reinterpret_cast<const float2*>(p + i)), tile * R + i);
        }
        score[key] = was + w;
      }
    }
    v = stop;
    if (b1 == nb && kvh + 1 == a.c.heads) {
      start += (nb + kStart) * items;
      ++seq;
      n = v < v_end ? a.c.len(seq) : 0;
    }
  }
}

struct Layout {
  int R, tiles, s_rows;
  size_t line, cta_part, stats, s_all, bytes;   // byte offsets
};

// Query rows of a KV head: tiles of 8, 16 or 24, as many as share one widened
// cache (32 would hold 128 sums a thread beside 64 scores and probabilities);
// the shared memory of 24 fp32 rows of 128 dims is too much.
int rows_of_tile(long long rows, int dtype, int d) {
  return rows <= 8 ? 8 : rows <= 16 || (dtype == MK_DTYPE_F32 && d == 128) ? 16 : 24;
}

Layout layout_of(const mk_kv4_cache* c, int dtype, int q_len, int group, bool accumulate) {
  Layout l;
  const int rows = q_len * group, d = c->head_dim;
  l.R = rows_of_tile(rows, dtype, d);
  l.tiles = (rows + l.R - 1) / l.R;
  l.s_rows = l.tiles > 1 ? l.R : (rows + 1) & ~1;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t part = (size_t)l.R * (d + 2) * sizeof(float);
  size_t at = 0;
  l.line = at; at = up(at + (1 + 2 * kMaxCtas) * sizeof(int4));
  l.cta_part = at; at = up(at + (size_t)kMaxCtas * 2 * part);
  l.stats = l.s_all = at;
  if (accumulate) {
    const size_t items = (size_t)c->n_seq * l.tiles * c->n_kv_heads;
    at = up(at + items * l.R * 2 * sizeof(float));
    l.s_all = at;
    const size_t units = (size_t)c->pages_per_seq * c->page_tokens / kKv4Block + kStart;
    at = up(at + items * units * kKv4Block * l.s_rows * sizeof(float));
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
  const long long rows = (long long)q_len * (n_q_heads / c->n_kv_heads);
  const double units = ((double)c->pages_per_seq * c->page_tokens / kKv4Block + kStart) * c->n_seq * c->n_kv_heads *
                       (double)(rows <= 8 ? 1 : (rows + 15) / 16);
  if (units > 2147483000.0) return kv4_fail(MK_ERR_UNSUPPORTED, who, "more than 2^31 blocks of keys and rows in one call");
  return MK_OK;
}

template <int D, int DT, int NT>
cudaError_t launch(const AttnArgs& a, int sms, cudaStream_t st) {
  constexpr int smem = AttnSmem<D, DT, NT>::kBytes;
  static_assert(smem <= (NT == 1 ? 112 : 224) * 1024, "two CTAs an SM, or one");
  AttnArgs args = a;
  const int ctas = sms * (NT == 1 ? 2 : 1);
  args.max_ctas = ctas < kMaxCtas ? ctas : kMaxCtas;
  cudaError_t e = cudaFuncSetAttribute(kv4_attn_kernel<D, DT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = pdl_launch(kv4_attn_kernel<D, DT, NT>, dim3(args.max_ctas), dim3(kThreadsA), smem, st, args);
  if (e != cudaSuccess) return e;
  return pdl_launch(kv4_attn_merge_kernel<D, DT, 8 * NT>, dim3(args.max_ctas * (args.accumulate ? 2 : 1)),
                    dim3(kThreadsM), 0, st, args);
}

template <int D, int DT>
cudaError_t launch_rows(const AttnArgs& a, int R, int sms, cudaStream_t st) {
  if (R == 8) return launch<D, DT, 1>(a, sms, st);
  if constexpr (D == 64 || DT != MK_DTYPE_F32)
    if (R == 24) return launch<D, DT, 3>(a, sms, st);
  return launch<D, DT, 2>(a, sms, st);
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
  // enough for every type
  const int group = n_q_heads / cache->n_kv_heads;
  const size_t a = layout_of(cache, MK_DTYPE_F32, q_len, group, accumulate != 0).bytes;
  const size_t b = layout_of(cache, MK_DTYPE_BF16, q_len, group, accumulate != 0).bytes;
  return a > b ? a : b;
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
      (reinterpret_cast<uintptr_t>(out_dev) & 15u))
    return kv4_fail(MK_ERR_INVALID_ARG, who, "queries of a token and the outputs are 16-byte aligned");
  if (!(scale >= 1e-18f) || !(scale <= 1e18f)) return kv4_fail(MK_ERR_INVALID_ARG, who, "scale is 1e-18 to 1e18");
  if (accumulate && !cache->scores_dev)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "weights are added to a cache's scores, and this one has none");
  const int group = n_q_heads / cache->n_kv_heads;
  const Layout l = layout_of(cache, dtype, q_len, group, accumulate != 0);
  if (!workspace_dev || (reinterpret_cast<uintptr_t>(workspace_dev) & 15u) || workspace_bytes < l.bytes)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "the workspace is 16-byte aligned and of the bytes asked for");
  const int sms = device_sms();
  if (!sms) return kv4_fail(MK_ERR_CUDA, who, "no device");
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
  a.cta_part = reinterpret_cast<float*>(ws + l.cta_part);
  a.line = reinterpret_cast<int4*>(ws + l.line);
  a.edges = a.line + 1;
  a.begins = a.edges + kMaxCtas;
  a.stats = reinterpret_cast<float2*>(ws + l.stats);
  a.s_all = reinterpret_cast<float*>(ws + l.s_all);
  a.s_rows = l.s_rows;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->head_dim == 128 ? launch_type<128>(a, dtype, l.R, sms, st)
                                               : launch_type<64>(a, dtype, l.R, sms, st);
  return e == cudaSuccess ? MK_OK : kv4_fail(MK_ERR_CUDA, who, cudaGetErrorString(e));
}

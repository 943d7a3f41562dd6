// beam.cu -- beam search: the selection over beams and vocabulary, and the
// reordering of the beams' states.
#include <math.h>
#include <stdio.h>

#include "kv4.cuh"
#include "pdl.cuh"
#include "beam.h"

namespace mk {
namespace {

// ------------------------------------------------------------------ select
//
// Candidate (b, v) of a search has the score cum[b] + logit[b][v] - lse(logit[b]);
// the W highest are wanted.  Inside a beam the order is that of the logits, so
// no score is needed to find a beam's own W best: the vocabulary is read once,
// in chunks of 16 KB that stay in registers, and each chunk gives its W
// highest logits, its maximum and its sum of exponentials.  The W-th highest
// maximum of the chunk's 32 groups of 8 threads bounds the W-th highest logit
// from below, so only logits from that bound on are looked at again, a few
// more than W (taking W rounds of maxima over all logits of a warp instead
// took twice the time: 16 x 4 rows of 151,936 in bf16 27 us).  Where
// ties make them too many, rounds over all logits find the lowest places.  A
// second kernel, one CTA a search and one warp a beam, joins the chunks: the
// log-sum-exp, the beam's W best (they lie in the W chunks with the highest
// heads), then the best of W * W scores.  The chunks' sums are fp32 sums; where
// their error could decide between candidates of two beams the join takes those
// beams' sums again, in 64 bits and in no order: never does that error order them.
//
// Bound: the logits' bytes once (4.1 MB for 8 beams of 128,256 in fp32: under
// 1 us) beside two launches and W rounds of warp maxima in each.

constexpr int kThreadsS = 256;
constexpr int kWarpsS = kThreadsS / 32;
// A chunk is 16 KB of logits: 64 bytes a thread.
__host__ __device__ constexpr int per_thread(int dtype) { return dtype == MK_DTYPE_F32 ? 16 : 32; }
__host__ __device__ constexpr int chunk_of(int dtype) { return kThreadsS * per_thread(dtype); }
constexpr int kMaxBeams = 16;
constexpr int kFound = 128;                     // logits from the bound on that a chunk keeps
static_assert(kWarpsS * 4 == 32, "a group's maximum for every lane");
constexpr int kMaxChunks = 256;
constexpr int kMaxVocab = 1 << 20;
static_assert(kMaxVocab <= chunk_of(MK_DTYPE_F32) * kMaxChunks, "chunk heads that a join holds");

// fp32 to an integer of the same order; 0 for what is no candidate (-inf, NaN).
__device__ __forceinline__ uint32_t logit_key(float f) {
  if (!(f > -INFINITY)) return 0u;
  if (f == 0.f) return 0x80000000u;
  const uint32_t b = __float_as_uint(f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// The lane whose (key, index) is first: highest key, then lowest index.
__device__ __forceinline__ void warp_first(uint32_t key, uint32_t idx, uint32_t& k, uint32_t& i) {
  k = __reduce_max_sync(0xFFFFFFFFu, key);
  i = __reduce_min_sync(0xFFFFFFFFu, key == k ? idx : 0xFFFFFFFFu);
}

struct SelectArgs {
  const void* logits;
  size_t stride;              // bytes between rows
  const float* cum;
  const uint8_t* finished;    // null: none
  int32_t* tokens;
  int32_t* parents;
  float* scores;
  uint8_t* done;              // null: not wanted
  int32_t beams, vocab, chunks, eos, dtype;
  // workspace
  float2* sums;               // [rows][chunks]: maximum, sum of exp(x - maximum)
  uint2* lists;               // [rows][chunks][beams]: key, token, highest first
};

// T: MK_DTYPE_* of the logits.  WIDE: rows allow 16-byte loads.
template <int T, bool WIDE>
__global__ void __launch_bounds__(kThreadsS) beam_chunk_kernel(const SelectArgs a) {
  constexpr int kPer = per_thread(T), kChunk = chunk_of(T);
  __shared__ uint2 best[kWarpsS][kMaxBeams], list[kFound];
  __shared__ float tops[32], parts[kWarpsS];
  __shared__ uint2 borders;   // keys of the highest logit and of the bound
  __shared__ int found;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = a.beams;
  const size_t row = blockIdx.y;
  if (a.finished && __ldcg(a.finished + row)) return;   // has its one candidate
  const int c0 = blockIdx.x * kChunk;
  const uint8_t* base = static_cast<const uint8_t*>(a.logits) + row * a.stride;
  float x[kPer];
  // element e of load j is c0 + (j * threads + tid) * kLoad + e
  constexpr int kSize = T == MK_DTYPE_F32 ? 4 : 2, kLoad = WIDE ? 16 / kSize : 1;
  auto at = [&](int i) { return c0 + ((i / kLoad) * kThreadsS + (int)threadIdx.x) * kLoad + i % kLoad; };
  auto widen = [&](uint32_t h) {
    return T == MK_DTYPE_F32 ? __uint_as_float(h)
           : T == MK_DTYPE_BF16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((unsigned short)h));
  };
  auto one = [&](int i) {
    if (i >= a.vocab) return -INFINITY;
    return widen(kSize == 4 ? __ldcg(reinterpret_cast<const uint32_t*>(base) + i)
                            : (uint32_t)__ldcg(reinterpret_cast<const uint16_t*>(base) + i));
  };
  if (WIDE && c0 + kChunk <= a.vocab) {
    uint4 v[kPer / kLoad];
#pragma unroll
    for (int j = 0; j < kPer / kLoad; ++j)
      v[j] = __ldcg(reinterpret_cast<const uint4*>(base + (size_t)c0 * kSize) + j * kThreadsS + threadIdx.x);
#pragma unroll
    for (int j = 0; j < kPer / kLoad; ++j) {
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (kSize == 4) {
          x[kLoad * j + e] = __uint_as_float(w[e]);
        } else {
          x[(kLoad * j + 2 * e) % kPer] = T == MK_DTYPE_BF16 ? __uint_as_float(w[e] << 16) : widen(w[e] & 0xFFFFu);
          x[(kLoad * j + 2 * e + 1) % kPer] = T == MK_DTYPE_BF16 ? __uint_as_float(w[e] & 0xFFFF0000u) : widen(w[e] >> 16);
        }
      }
    }
  } else {   // a row's last chunk, or rows at odd places
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = one(at(i));
  }

  // maxima of the threads (fmaxf passes NaN by), the groups, the chunk
  float top = x[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i) top = fmaxf(top, x[i]);
  float group = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  group = fmaxf(group, __shfl_xor_sync(0xFFFFFFFFu, group, 2));
  group = fmaxf(group, __shfl_xor_sync(0xFFFFFFFFu, group, 4));
  if ((lane & 7) == 0) tops[warp * 4 + (lane >> 3)] = group;
  if (threadIdx.x == 0) found = 0;
  __syncthreads();
  if (warp == 0) {
    uint32_t left = logit_key(tops[lane]);   // a group a lane
    const uint32_t first = __reduce_max_sync(0xFFFFFFFFu, left);
    uint32_t last = first;
    for (int j = 0; j < W; ++j) {
      last = __reduce_max_sync(0xFFFFFFFFu, left);
      if (last == 0u) break;   // fewer groups with a candidate: look at every one
      if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, left == last)) - 1) left = 0u;
    }
    if (lane == 0) borders = make_uint2(first, last);
  }
  __syncthreads();
  const uint32_t highest = borders.x, bound = borders.y;
  const float mx = highest ? key_logit(highest) : 0.f;
  // the W-th highest maximum, or everything
  const float least = bound ? key_logit(bound) : -INFINITY;
  if (__any_sync(0xFFFFFFFFu, top >= least && top > -INFINITY)) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool hit = x[i] >= least && x[i] > -INFINITY;
      if (__any_sync(0xFFFFFFFFu, hit)) {   // few of a warp's elements: the rest costs a vote
        if (hit) {
          const int to = atomicAdd(&found, 1);   // any order: places decide below
          if (to < kFound) list[to] = make_uint2(logit_key(x[i]), at(i));
        }
      }
    }
  }
  float part[4] = {0.f, 0.f, 0.f, 0.f};   // -inf adds 0, NaN goes through
#pragma unroll
  for (int i = 0; i < kPer; ++i) part[i & 3] += ex2((x[i] - mx) * 1.44269504f);
  float sum = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) parts[warp] = sum;
  __syncthreads();
  const size_t chunk = row * a.chunks + blockIdx.x;
  uint2* out = a.lists + chunk * W;
  if (threadIdx.x == 0) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarpsS; ++w) s += parts[w];
    a.sums[chunk] = make_float2(highest ? mx : -INFINITY, s);
  }
  if (found <= kFound) {
    // each one's rank by counting those before it
    if ((int)threadIdx.x < found) {
      const uint2 mine = list[threadIdx.x];
      int rank = 0;
      for (int j = 0; j < found; ++j) {
        const uint2 o = list[j];
        rank += o.x > mine.x || (o.x == mine.x && o.y < mine.y);
      }
      if (rank < W) out[rank] = mine;
    } else if ((int)threadIdx.x < W) {
      out[threadIdx.x] = make_uint2(0u, 0u);
    }
    return;
  }

  // more logits on the bound than the list holds: rounds of maxima, a warp's W
  // highest first, then those of the warps
  uint32_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = logit_key(x[i]);
  uint32_t mine = 0, which = 0;   // this lane's first: the lowest index of its highest key
  auto rescan = [&]() {
    mine = 0; which = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (key[i] > mine) { mine = key[i]; which = i; }   // at() grows with i
  };
  rescan();
  for (int j = 0; j < W; ++j) {
    uint32_t k, i;
    warp_first(mine, at(which), k, i);
    if (lane == 0) best[warp][j] = make_uint2(k, i);
    if (k == 0u) {   // no more candidates
      for (int z = j + 1 + lane; z < W; z += 32) best[warp][z] = make_uint2(0u, 0u);
      break;
    }
    if (mine == k && (uint32_t)at(which) == i) {
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (e == (int)which) key[e] = 0u;
      rescan();
    }
  }
  __syncthreads();
  if (warp) return;
  // lane l (of kWarpsS) walks list l
  int head = 0;
  uint2 h = lane < kWarpsS ? best[lane][0] : make_uint2(0u, 0u);
  for (int j = 0; j < W; ++j) {
    uint32_t k, i;
    warp_first(h.x, h.y, k, i);
    if (lane == 0) out[j] = make_uint2(k, k ? i : 0u);
    if (k && h.x == k && h.y == i) {
      ++head;
      h = head < W ? best[lane][head] : make_uint2(0u, 0u);
    }
  }
}

// 64-bit scores to integers of the same order; 0 for what is no candidate.
__device__ __forceinline__ unsigned long long score_key64(double s) {
  if (!(s > -INFINITY)) return 0ull;
  if (s == 0.0) return 0x8000000000000000ull;
  const unsigned long long b = __double_as_longlong(s);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

__device__ __forceinline__ double key_score64(unsigned long long k) {
  return __longlong_as_double((long long)(k >> 63 ? k & 0x7FFFFFFFFFFFFFFFull : ~k));
}

// Largest error of a beam's log-sum-exp as the chunks give it.  Exponents carry
// 2.3 x 2^-24 of their size (difference, product, the rounded log2(e)), and
// their mean size under a chunk's softmax is at most the logarithm of its 8,192
// logits, 9.1 nats (the entropy is that mean plus the sum's logarithm): 21 x
// 2^-24 of the sum.  ex2.approx adds 4 x 2^-24 and 23 additions in a row 23 x
// 2^-24; the chunks are added in 64 bits.
constexpr double kSumError = 1.0 / (1 << 18);

// This thread's part of the sum of exp(logit - mx) over a row, in units of 2^-43
// (x) and of 2^-86 (y, what those leave, of either sign): whole numbers, so that
// the sum does not depend on the order and rows of the same logits have the
// same one.  At most 2^20 terms of at most 2^43: modulo 2^64 they fit.  A term is
// rounded to either unit by an addition that leaves it in the last bits of the
// sum (with conversions to integers and loads of single logits, 8 rows of 128,256
// in fp32 took 1,250 us instead of 706).
__device__ __noinline__ ulonglong2 exact_sum(const uint8_t* base, int dtype, int vocab, float mx) {
  constexpr double kOne = 0x1p9, kTwo = 1.5 * 0x1p-34;   // last bits 2^-43 and 2^-86
  ulonglong2 sum = {0ull, 0ull};
  auto add = [&](float x) {
    const double t = exp((double)x - (double)mx);
    const double a = __dadd_rn(t, kOne), b = __dadd_rn(__dsub_rn(t, __dsub_rn(a, kOne)), kTwo);
    sum.x += __double_as_longlong(a) - __double_as_longlong(kOne);
    sum.y += __double_as_longlong(b) - __double_as_longlong(kTwo);
  };
  auto widen = [&](uint32_t h) {
    return dtype == MK_DTYPE_BF16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((unsigned short)h));
  };
  const int size = dtype == MK_DTYPE_F32 ? 4 : 2, of16 = 16 / size;
  const int whole = (reinterpret_cast<uintptr_t>(base) & 15u) ? 0 : vocab / of16;
#pragma unroll 2
  for (int i = threadIdx.x; i < whole; i += blockDim.x) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(base) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (size == 4) {
        add(__uint_as_float(w[e]));
      } else {
        add(widen(w[e] & 0xFFFFu));
        add(widen(w[e] >> 16));
      }
    }
  }
  for (int i = whole * of16 + threadIdx.x; i < vocab; i += blockDim.x)
    add(size == 4 ? __ldcg(reinterpret_cast<const float*>(base) + i)
                  : widen(__ldcg(reinterpret_cast<const uint16_t*>(base) + i)));
  return sum;
}

__device__ __forceinline__ bool finished_of(const SelectArgs& a, size_t row) {
  return a.finished && __ldcg(a.finished + row);
}

// Warps of a join beside those of its beams help with sums that are taken again.
__host__ __device__ constexpr int join_threads(int beams) { return beams == 1 ? 32 : beams > 4 ? beams * 32 : 128; }

// One CTA a search, one warp a beam.  HEADS: chunk heads of a lane.  WT: most beams.
// Where candidates of two beams are closer than the error of their sums
// (neighbours 0.1 apart on average are that close once in 13,000 times), those
// beams' sums are taken again in 64 bits and the choice is made again.  It costs 0.2 to
// 0.8 us where nothing is close (8 beams of 128,256 fp32 10.1 -> 10.5 us) and
// 90 to 130 us for each such beam of that size (8 that hold the same logits 706 us).
template <int HEADS, int WT>
__global__ void __launch_bounds__(join_threads(WT)) beam_join_kernel(const SelectArgs a) {
  constexpr int kOwn = WT * WT < 32 ? 1 : WT * WT / 32;   // candidates of a lane
  __shared__ __align__(16) uint2 few[WT][HEADS * 32 > WT * WT ? HEADS * 32 : WT * WT];   // heads, then candidates
  __shared__ int chosen[WT][WT];
  __shared__ uint32_t bound[WT];
  __shared__ double cand_score[WT][WT];
  __shared__ float cand_logit[WT][WT];
  __shared__ int32_t cand_token[WT][WT];
  __shared__ float highest[WT];
  __shared__ unsigned long long total[2];
  __shared__ uint32_t unsure;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, beam = threadIdx.x >> 5, W = a.beams;
  const size_t row = (size_t)blockIdx.x * W + beam;
  // all in flight at once (a finished beam's sums and lists are not written: not used)
  const double cum = beam < W ? __ldcg(a.cum + row) : 0.0;
  const bool ended = beam == 0 && lane < W && finished_of(a, (size_t)blockIdx.x * W + lane);
  if (beam < W) {
    const float2* sums = a.sums + row * a.chunks;
    const uint2* lists = a.lists + row * a.chunks * W;
    const bool finished = finished_of(a, row);
    float2 sum_of[HEADS];
    uint2 head[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      const int c = i * 32 + lane;
      sum_of[i] = c < a.chunks ? __ldcg(sums + c) : make_float2(-INFINITY, 0.f);
      head[i] = c < a.chunks ? __ldcg(lists + (size_t)c * W) : make_uint2(0u, 0u);
    }
    for (int j = lane; j < W; j += 32) {   // no candidates so far
      cand_score[beam][j] = -INFINITY;
      chosen[beam][j] = -1;
    }
    if (lane == 0) bound[beam] = 0u;
    if (finished) {
      __syncwarp();
      if (lane == 0) {
        cand_score[beam][0] = cum;
        cand_token[beam][0] = a.eos;
      }
    } else {
#pragma unroll
      for (int i = 0; i < HEADS; ++i) few[beam][i * 32 + lane] = head[i];
      __syncwarp();
      // the W chunks with the highest heads, by counting the heads before each (a
      // head's token tells ties apart); the last of them bounds the beam's W best
      const uint4* two = reinterpret_cast<const uint4*>(few[beam]);
      int rank[HEADS];
#pragma unroll
      for (int i = 0; i < HEADS; ++i) rank[i] = 0;
      const int pairs = (min(a.chunks, HEADS * 32) + 1) / 2;
#pragma unroll 4
      for (int j = 0; j < pairs; ++j) {
        const uint4 o = two[j];
#pragma unroll
        for (int i = 0; i < HEADS; ++i) {
          rank[i] += o.x > head[i].x || (o.x == head[i].x && o.y < head[i].y);
          rank[i] += o.z > head[i].x || (o.z == head[i].x && o.w < head[i].y);
        }
      }
#pragma unroll
      for (int i = 0; i < HEADS; ++i)
        if (head[i].x && rank[i] < W) {
          chosen[beam][rank[i]] = i * 32 + lane;
          if (rank[i] == W - 1) bound[beam] = head[i].x;
        }
      __syncwarp();
      // their lists, in flight during the log-sum-exp over all chunks
      uint2 c[kOwn];
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int e = i * 32 + lane, from = e / W;
        const int chunk = e < W * W ? chosen[beam][from] : -1;
        c[i] = chunk >= 0 ? __ldcg(lists + (size_t)chunk * W + (e - from * W)) : make_uint2(0u, 0u);
      }
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < HEADS; ++i) mx = fmaxf(mx, sum_of[i].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < HEADS; ++i)
        // a chunk without a candidate has maximum -inf and adds its sum: 0, or a NaN
        sum += sum_of[i].x > -INFINITY ? (double)sum_of[i].y * exp((double)sum_of[i].x - (double)mx) : (double)sum_of[i].y;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      // log-probability: (logit - mx) - log(sum), the first difference exact, so that a constant
      // on all logits of a row changes nothing
      const double log_sum = log(sum);
      if (lane == 0) highest[beam] = mx;
      // the beam's W best: of the few from the bound on, again by counting
      const uint32_t least = max(bound[beam], 1u);
      int n = 0;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const uint32_t in = __ballot_sync(0xFFFFFFFFu, c[i].x >= least);
        if (c[i].x >= least) few[beam][n + __popc(in & ((1u << lane) - 1u))] = c[i];
        n += __popc(in);
      }
      __syncwarp();
      for (int e = lane; e < n; e += 32) {
        const uint2 me = few[beam][e];
        int before = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
          const uint2 o = few[beam][j];
          before += o.x > me.x || (o.x == me.x && o.y < me.y);
        }
        if (before < W) {
          cand_score[beam][before] = cum + (((double)key_logit(me.x) - (double)mx) - log_sum);
          cand_logit[beam][before] = key_logit(me.x);
          cand_token[beam][before] = (int32_t)me.y;
        }
      }
    }
  }
  // beams whose scores carry no error of a sum (the first warp's)
  uint32_t exact = __ballot_sync(0xFFFFFFFFu, ended);
#pragma unroll 1
  for (;;) {
    __syncthreads();
    if (beam == 0) {
      // W rounds over the beams' lists, a lane each: highest score, then lowest beam
      int at = 0;
      double mine = lane < W ? cand_score[lane][0] : -INFINITY;
      unsigned long long chosen_key = 0ull;   // lane j: the j-th choice, 0 a dead one
      int chosen_beam = 0;
      for (int j = 0; j < W; ++j) {
        const unsigned long long key = score_key64(mine);
        const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(key >> 32));
        const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(key >> 32) == hi ? (uint32_t)key : 0u);
        const unsigned long long best = (unsigned long long)hi << 32 | lo;
        const bool real = best != 0ull;
        const int who = __ffs(__ballot_sync(0xFFFFFFFFu, key == best)) - 1;
        if (lane == j) {
          chosen_key = best;
          chosen_beam = who;
        }
        // fewer candidates than beams: a dead one, which keeps its own state
        if (real ? lane == who : lane == j) {
          const size_t to = (size_t)blockIdx.x * W + j;
          const int token = real ? cand_token[lane][at] : max(a.eos, 0);
          a.tokens[to] = token;
          a.parents[to] = lane;
          a.scores[to] = real ? (float)mine : -INFINITY;
          if (a.done) a.done[to] = ended || (a.eos >= 0 && token == a.eos);
          if (real) {
            ++at;
            mine = at < W ? cand_score[lane][at] : -INFINITY;
          }
        }
      }
      // Beams that a choice could have gone the other way for: of neighbours in the
      // order, and of the last choice and each beam's next candidate.  (What is close
      // to a choice further off is close to all in between.)
      uint32_t close = 0u;
      if (W > 1) {
        auto close_to = [&](unsigned long long key, int b, double below, int b2) -> uint32_t {
          const bool e = exact >> b & 1u, e2 = exact >> b2 & 1u;
          const double from = key_score64(key) - (e || e2 ? kSumError : 2 * kSumError);
          return key && b != b2 && !(e && e2) && below >= from ? 1u << b | 1u << b2 : 0u;
        };
        const unsigned long long next_key = __shfl_down_sync(0xFFFFFFFFu, chosen_key, 1),
                                 last_key = __shfl_sync(0xFFFFFFFFu, chosen_key, W - 1);
        const int next_beam = __shfl_down_sync(0xFFFFFFFFu, chosen_beam, 1),
                  last_beam = __shfl_sync(0xFFFFFFFFu, chosen_beam, W - 1);
        if (lane < W) close = close_to(last_key, last_beam, mine, lane);
        if (lane + 1 < W && next_key) close |= close_to(chosen_key, chosen_beam, key_score64(next_key), next_beam);
        close = __reduce_or_sync(0xFFFFFFFFu, close) & ~exact;
      }
      exact |= close;
      if (lane == 0) unsure = close;
    }
    __syncthreads();
    uint32_t left = unsure;   // the same for all, and new beams each time round
    if (left == 0u) return;
    for (; left; left &= left - 1u) {
      const int b = __ffs(left) - 1;
      if (threadIdx.x < 2) total[threadIdx.x] = 0ull;
      __syncthreads();
      ulonglong2 sum = exact_sum(static_cast<const uint8_t*>(a.logits) + ((size_t)blockIdx.x * W + b) * a.stride,
                                a.dtype, a.vocab, highest[b]);
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        sum.x += __shfl_xor_sync(0xFFFFFFFFu, sum.x, o);
        sum.y += __shfl_xor_sync(0xFFFFFFFFu, sum.y, o);
      }
      if (lane == 0) {
        atomicAdd(&total[0], sum.x);
        atomicAdd(&total[1], sum.y);
      }
      __syncthreads();
      if (beam == b && lane < W && cand_score[b][lane] > -INFINITY) {
        const double all = ((double)total[0] + (double)(long long)total[1] * 0x1p-43) * 0x1p-43;
        cand_score[b][lane] = cum + (((double)cand_logit[b][lane] - (double)highest[b]) - log(all));
      }
      __syncthreads();
    }
  }
}

// ----------------------------------------------------------------- reorder
//
// Beam b gets the state of beam parents[b], in place.  A thread owns one
// 16-byte column of the states: it reads that column of every parent that some
// other beam wants, and only then writes, so no beam's state is overwritten
// before it is read and no copy of the states is kept.  Beams that stay are neither
// read nor written.  Bound: the moved bytes, read (once from HBM per parent) and written.

constexpr int kThreadsR = 256;

// Physical byte address of logical offset `o` (in the beam's segment `seg`).
__device__ __forceinline__ uint8_t* state_at(const ReorderState& s, int beam, int seg, uint32_t o16) {
  int slot = s.slots ? s.slot[beam] : beam;
  uint32_t page = (uint32_t)slot;
  if (s.page16) {   // pages of a segment: page16 16-byte columns each
    const uint32_t lp = o16 / s.page16;
    o16 -= lp * s.page16;
    if (s.table) {
      const int p = __ldcg(s.table + (size_t)slot * s.pps + lp);
      if (p < 0 || p >= s.pages) return nullptr;
      page = (uint32_t)p;
    } else {
      page = (uint32_t)slot * s.pps + lp;
    }
  }
  return s.base + page * s.stride + seg * s.seg_stride + (size_t)o16 * 16;
}

template <int W>
__global__ void __launch_bounds__(kThreadsR) beam_reorder_kernel(const ReorderArgs a) {
  __shared__ int par[W];
  pdl_trigger();
  pdl_wait();
  const ReorderState& s = a.state[blockIdx.z % a.n_states];
  const int batch = blockIdx.z / a.n_states;
  if (threadIdx.y == 0 && threadIdx.x < W) {
    const int b = threadIdx.x;
    int p = b < a.beams ? __ldcg(a.parents + (size_t)batch * a.beams + b) : b;
    par[b] = p < 0 || p >= a.beams ? b : p;   // no such beam: it stays
  }
  __syncthreads();
  const int seg = blockIdx.y * blockDim.y + threadIdx.y;
  const uint32_t col = blockIdx.x * blockDim.x + threadIdx.x;
  if (seg >= s.segments || col >= s.count16) return;
  const uint32_t o = s.first16 + col;
  uint4 v[W];
  uint32_t moves = 0;
#pragma unroll
  for (int b = 0; b < W; ++b) {
    const int p = par[b];
    if (b < a.beams && p != b) {
      const uint8_t* from = state_at(s, batch * a.beams + p, seg, o);
      if (from) { v[b] = __ldcg(reinterpret_cast<const uint4*>(from)); moves |= 1u << b; }
    }
  }
#pragma unroll
  for (int b = 0; b < W; ++b)
    if (moves >> b & 1u) {
      uint8_t* to = state_at(s, batch * a.beams + b, seg, o);
      if (to) *reinterpret_cast<uint4*>(to) = v[b];
    }
}

int fail(int code, const char* who, const char* why) { return kv4_fail(code, who, why); }

}  // namespace

cudaError_t launch_reorder(const ReorderArgs& a, int n_batch, cudaStream_t st) {
  uint32_t cols = 0;
  int segs = 0;
  for (int i = 0; i < a.n_states; ++i) {
    if (a.state[i].count16 > cols) cols = a.state[i].count16;
    if (a.state[i].segments > segs) segs = a.state[i].segments;
  }
  if (cols == 0 || segs == 0 || a.beams < 2) return cudaSuccess;
  int x = 32;   // short segments share a block
  while (x < kThreadsR && (uint32_t)x < cols) x <<= 1;
  const int y = kThreadsR / x;
  const dim3 grid((cols + x - 1) / x, (segs + y - 1) / y, n_batch * a.n_states), block(x, y);
  if (grid.y > 65535u || grid.z > 65535u) return cudaErrorInvalidValue;
  auto kernel = a.beams <= 2 ? beam_reorder_kernel<2> : a.beams <= 4 ? beam_reorder_kernel<4>
                : a.beams <= 8 ? beam_reorder_kernel<8> : beam_reorder_kernel<16>;
  return pdl_launch(kernel, grid, block, 0, st, a);
}

}  // namespace mk

using namespace mk;

extern "C" size_t mk_beam_select_workspace_bytes(int n_batch, int beams, int vocab) {
  if (n_batch < 1 || beams < 1 || beams > kMaxBeams || vocab < 1 || vocab > kMaxVocab ||
      (long long)n_batch * beams > 65535)
    return 0;
  const int per = chunk_of(MK_DTYPE_F32);   // enough for every type
  const size_t chunks = (vocab + per - 1) / per, rows = (size_t)n_batch * beams;
  return rows * chunks * (sizeof(float2) + beams * sizeof(uint2));
}

extern "C" int mk_beam_select(const void* logits_dev, int dtype, long long row_stride, const float* cum_dev,
                              const uint8_t* finished_dev, int n_batch, int beams, int vocab, int eos,
                              int32_t* tokens_dev, int32_t* parents_dev, float* scores_dev,
                              uint8_t* finished_out_dev, void* workspace_dev, size_t workspace_bytes,
                              void* stream) {
  const char* who = "mk_beam_select";
  if (n_batch < 1 || beams < 1 || beams > kMaxBeams || (long long)n_batch * beams > 65535)
    return fail(MK_ERR_INVALID_ARG, who, "1 to 16 beams, and at most 65535 rows");
  if (vocab < 1 || vocab > kMaxVocab) return fail(MK_ERR_INVALID_ARG, who, "vocab is 1 to 1048576");
  const int esz = dtype == MK_DTYPE_F32 ? 4 : (dtype == MK_DTYPE_BF16 || dtype == MK_DTYPE_F16) ? 2 : 0;
  if (!esz) return fail(MK_ERR_INVALID_ARG, who, "dtype is one of MK_DTYPE_*");
  if (!logits_dev || !cum_dev || !tokens_dev || !parents_dev || !scores_dev)
    return fail(MK_ERR_INVALID_ARG, who, "logits, sums, tokens, parents and scores are wanted");
  if (row_stride < vocab || row_stride > (1ll << 40)) return fail(MK_ERR_INVALID_ARG, who, "rows are at least vocab apart");
  if (eos < -1 || eos >= vocab) return fail(MK_ERR_INVALID_ARG, who, "eos is -1 or a token");
  if (finished_dev && eos < 0) return fail(MK_ERR_INVALID_ARG, who, "finished beams need an eos");
  if (finished_dev && (const uint8_t*)finished_out_dev == finished_dev)
    return fail(MK_ERR_INVALID_ARG, who, "finished flags are read while the new ones are written: two arrays");
  if (static_cast<const float*>(scores_dev) == cum_dev)
    return fail(MK_ERR_INVALID_ARG, who, "sums are read while the new ones are written: two arrays");
  if ((reinterpret_cast<uintptr_t>(logits_dev) & (esz - 1)) ||
      ((reinterpret_cast<uintptr_t>(cum_dev) | reinterpret_cast<uintptr_t>(tokens_dev) |
        reinterpret_cast<uintptr_t>(parents_dev) | reinterpret_cast<uintptr_t>(scores_dev)) & 3u))
    return fail(MK_ERR_INVALID_ARG, who, "arrays are aligned to their type");
  const size_t need = mk_beam_select_workspace_bytes(n_batch, beams, vocab);
  if (!workspace_dev || (reinterpret_cast<uintptr_t>(workspace_dev) & 15u) || workspace_bytes < need)
    return fail(MK_ERR_INVALID_ARG, who, "the workspace is 16-byte aligned and of the bytes asked for");
  SelectArgs a;
  a.logits = logits_dev; a.stride = (size_t)row_stride * esz;
  a.cum = cum_dev; a.finished = finished_dev;
  a.tokens = tokens_dev; a.parents = parents_dev; a.scores = scores_dev; a.done = finished_out_dev;
  a.beams = beams; a.vocab = vocab; a.eos = eos; a.dtype = dtype;
  a.chunks = (vocab + chunk_of(dtype) - 1) / chunk_of(dtype);
  const bool wide = ((reinterpret_cast<uintptr_t>(logits_dev) | a.stride) & 15u) == 0;
  const size_t rows = (size_t)n_batch * beams;
  a.sums = static_cast<float2*>(workspace_dev);
  a.lists = reinterpret_cast<uint2*>(a.sums + rows * a.chunks);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto chunk = dtype == MK_DTYPE_F32 ? (wide ? beam_chunk_kernel<MK_DTYPE_F32, true> : beam_chunk_kernel<MK_DTYPE_F32, false>)
               : dtype == MK_DTYPE_BF16 ? (wide ? beam_chunk_kernel<MK_DTYPE_BF16, true> : beam_chunk_kernel<MK_DTYPE_BF16, false>)
                                        : (wide ? beam_chunk_kernel<MK_DTYPE_F16, true> : beam_chunk_kernel<MK_DTYPE_F16, false>);
  cudaError_t e = pdl_launch(chunk, dim3(a.chunks, (unsigned)rows), dim3(kThreadsS), 0, st, a);
  auto join = beams <= 4 ? (a.chunks <= 64 ? beam_join_kernel<2, 4> : beam_join_kernel<8, 4>)
              : beams <= 8 ? (a.chunks <= 64 ? beam_join_kernel<2, 8> : beam_join_kernel<8, 8>)
                           : (a.chunks <= 64 ? beam_join_kernel<2, 16> : beam_join_kernel<8, 16>);
  if (e == cudaSuccess) e = pdl_launch(join, dim3(n_batch), dim3(join_threads(beams)), 0, st, a);
  return e == cudaSuccess ? MK_OK : fail(MK_ERR_CUDA, who, cudaGetErrorString(e));
}

extern "C" int mk_beam_reorder(void* state_dev, const int32_t* parents_dev, int n_batch, int beams,
                               size_t beam_stride, int n_segments, size_t segment_stride,
                               size_t segment_bytes, void* stream) {
  const char* who = "mk_beam_reorder";
  if (n_batch < 1 || n_batch > 32767 || beams < 1 || beams > kMaxBeams)
    return fail(MK_ERR_INVALID_ARG, who, "1 to 16 beams and 1 to 32767 searches");
  if (n_segments < 0 || n_segments > 65535) return fail(MK_ERR_INVALID_ARG, who, "0 to 65535 segments");
  if (!state_dev || !parents_dev) return fail(MK_ERR_INVALID_ARG, who, "no state or parents");
  if ((reinterpret_cast<uintptr_t>(state_dev) | beam_stride | segment_stride | segment_bytes) & 15u)
    return fail(MK_ERR_INVALID_ARG, who, "the state, its strides and a segment's bytes are multiples of 16");
  if (reinterpret_cast<uintptr_t>(parents_dev) & 3u) return fail(MK_ERR_INVALID_ARG, who, "parents are 4-byte aligned");
  if (segment_bytes > (size_t)1 << 34) return fail(MK_ERR_INVALID_ARG, who, "a segment has at most 2^34 bytes");
  if (n_segments > 1 && segment_stride < segment_bytes)
    return fail(MK_ERR_INVALID_ARG, who, "segments of a beam do not overlap");
  if (n_segments && n_batch * beams > 1 && beam_stride < (n_segments - 1) * segment_stride + segment_bytes &&
      !(n_segments > 1 && segment_stride >= (size_t)(n_batch * beams - 1) * beam_stride + segment_bytes &&
        beam_stride >= segment_bytes))
    return fail(MK_ERR_INVALID_ARG, who, "beams do not overlap");
  ReorderArgs a = {};
  a.parents = parents_dev; a.beams = beams; a.n_states = 1;
  ReorderState& s = a.state[0];
  s.base = static_cast<uint8_t*>(state_dev);
  s.stride = beam_stride; s.seg_stride = segment_stride;
  s.segments = n_segments; s.count16 = (uint32_t)(segment_bytes / 16);
  const cudaError_t e = launch_reorder(a, n_batch, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MK_OK : fail(MK_ERR_CUDA, who, cudaGetErrorString(e));
}

extern "C" int mk_kv4_reorder(const mk_kv4_cache* cache, const int32_t* parents_dev, int beams, int first,
                              int n_keys, void* stream) {
  const char* who = "mk_kv4_reorder";
  if (int rc = kv4_check(cache, who)) return rc;
  if (beams < 1 || beams > kMaxBeams || cache->n_seq % beams)
    return fail(MK_ERR_INVALID_ARG, who, "1 to 16 beams, and whole searches of them in the cache");
  const long long capacity = (long long)cache->pages_per_seq * cache->page_tokens;
  if (first < 0 || n_keys < first || n_keys > capacity)
    return fail(MK_ERR_INVALID_ARG, who, "keys [first, n_keys) of the cache");
  if (!parents_dev || (reinterpret_cast<uintptr_t>(parents_dev) & 3u))
    return fail(MK_ERR_INVALID_ARG, who, "parents are a 4-byte aligned array");
  if (n_keys == first) return MK_OK;
  const int b0 = first / kKv4Block, b1 = (n_keys + kKv4Block - 1) / kKv4Block;
  const uint32_t block16 = kKv4Block * (cache->head_dim + cache->head_dim / 8) / 16;
  if ((long long)b1 * block16 > 0x7FFFFFFFll) return fail(MK_ERR_INVALID_ARG, who, "too many keys in one call");
  ReorderArgs a = {};
  a.parents = parents_dev; a.beams = beams; a.n_states = 1;
  ReorderState& s = a.state[0];
  s.base = static_cast<uint8_t*>(cache->pool_dev);
  s.table = cache->table_dev; s.pps = cache->pages_per_seq; s.pages = cache->n_pages;
  s.page16 = cache->page_tokens / kKv4Block * block16;
  s.seg_stride = (size_t)s.page16 * 16;
  s.stride = s.seg_stride * cache->n_kv_heads;
  s.segments = cache->n_kv_heads;
  s.first16 = b0 * block16; s.count16 = (b1 - b0) * block16;
  if (cache->scores_dev) {   // a page is a multiple of 32 keys: rows of scores are whole 16-byte columns
    if (reinterpret_cast<uintptr_t>(cache->scores_dev) & 15u)
      return fail(MK_ERR_INVALID_ARG, who, "scores are 16-byte aligned");
    ReorderState& w = a.state[a.n_states++];
    w.base = reinterpret_cast<uint8_t*>(cache->scores_dev);
    w.seg_stride = (size_t)capacity * 4;
    w.stride = w.seg_stride * cache->n_kv_heads;
    w.segments = cache->n_kv_heads;
    w.first16 = b0 * (kKv4Block / 4); w.count16 = (b1 - b0) * (kKv4Block / 4);
  }
  const cudaError_t e = launch_reorder(a, cache->n_seq / beams, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MK_OK : fail(MK_ERR_CUDA, who, cudaGetErrorString(e));
}

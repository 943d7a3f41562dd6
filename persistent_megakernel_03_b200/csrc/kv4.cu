// kv4.cu -- the 4-bit KV cache's writers and readers: append, read, eviction.
#include <math.h>
#include <stdio.h>

#include <atomic>
#include <type_traits>

#include "kv4.cuh"
#include "pdl.cuh"

namespace mk {

int kv4_fail(int code, const char* who, const char* why) {
  char msg[256];
  snprintf(msg, sizeof msg, "%s: %s", who, why);
  set_last_error(msg);
  return code;
}

int device_sms() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];   // 0: not asked yet
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < kDevices && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < kDevices) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

int kv4_check(const mk_kv4_cache* c, const char* who) {
  if (!c) return kv4_fail(MK_ERR_INVALID_ARG, who, "no cache");
  if (!c->pool_dev || !c->lens_dev) return kv4_fail(MK_ERR_INVALID_ARG, who, "a cache has a pool and lengths");
  if (c->head_dim != 64 && c->head_dim != 128)
    return kv4_fail(MK_ERR_UNSUPPORTED, who, "head_dim is 64 or 128");
  if (c->n_kv_heads < 1 || c->n_kv_heads > 1024)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "n_kv_heads is 1 to 1024");
  if (c->page_tokens < kKv4Block || c->page_tokens % kKv4Block)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "page_tokens is a positive multiple of 32");
  if (c->n_seq < 1 || c->n_seq > kKv4MaxSeq) return kv4_fail(MK_ERR_INVALID_ARG, who, "n_seq is 1 to 4096");
  if (c->n_pages < 1 || c->pages_per_seq < 1)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "n_pages and pages_per_seq are positive");
  if ((long long)c->pages_per_seq * c->page_tokens > (1ll << 30))
    return kv4_fail(MK_ERR_INVALID_ARG, who, "a sequence holds at most 2^30 keys");
  if (!c->table_dev && (long long)c->n_seq * c->pages_per_seq > c->n_pages)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "without a table the pool has n_seq * pages_per_seq pages");
  if (c->k_log2 < -32 || c->k_log2 > 32 || c->v_log2 < -32 || c->v_log2 > 32)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "k_log2 and v_log2 are -32 to 32");
  if (reinterpret_cast<uintptr_t>(c->pool_dev) & 15u)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "the pool is 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(c->table_dev) | reinterpret_cast<uintptr_t>(c->lens_dev) |
       reinterpret_cast<uintptr_t>(c->scores_dev)) & 3u)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "table, lengths and scores are 4-byte aligned");
  return MK_OK;
}

Kv4 kv4_of(const mk_kv4_cache* c) {
  Kv4 k;
  k.pool = static_cast<uint8_t*>(c->pool_dev);
  k.table = c->table_dev; k.lens = c->lens_dev; k.scores = c->scores_dev;
  k.heads = c->n_kv_heads; k.page_tokens = c->page_tokens; k.pages = c->n_pages;
  k.n_seq = c->n_seq; k.pps = c->pages_per_seq;
  return k;
}

// ------------------------------------------------------------------ append

// 32 bytes.  A thread's 16 elements are one or two such pieces: as one access
// each they are whole sectors, while 16-byte accesses 32 bytes apart move every sector
// twice.  Addresses that are only 16-byte aligned take those.
__device__ __forceinline__ void load32(const uint8_t* p, bool whole, uint4& a, uint4& b) {
  if (whole) {
    asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
  } else {
    a = __ldcg(reinterpret_cast<const uint4*>(p));
    b = __ldcg(reinterpret_cast<const uint4*>(p) + 1);
  }
}
__device__ __forceinline__ void store32(uint8_t* p, bool whole, uint4 a, uint4 b) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w), "l"(p)
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = a;
    reinterpret_cast<uint4*>(p)[1] = b;
  }
}

// 16 input elements, raw, as fp32.
template <int DT, int N>
__device__ __forceinline__ void widen_input(const uint4 (&raw)[N], float (&x)[16]) {
  constexpr int kPer = 16 / N;   // elements of 16 bytes
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == MK_DTYPE_F32) {
        x[kPer * i + j] = __uint_as_float(w[j]);
      } else if constexpr (DT == MK_DTYPE_BF16) {
        x[kPer * i + 2 * j] = __uint_as_float(w[j] << 16);
        x[kPer * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        x[kPer * i + 2 * j] = f.x; x[kPer * i + 2 * j + 1] = f.y;
      }
    }
  }
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// One group: the scale is e4m3(max |x| / 6), rounded to nearest even and at
// most 448; a code is the e2m1 value nearest x / scale, halves to the even
// code.  Both come out exactly.  A quotient a / b of fp32 numbers is on a
// midpoint m of either grid (at most 5 significant bits) or at least 0.53 of
// fp32's steps away from it, as a and m * b are fp32 numbers too; so it is
// enough to round the quotient correctly, and then to the grid.  For the
// codes the reciprocal's product is corrected once by its exact remainder,
// which leaves an error of 2^-47 before the rounding.  Comparing x with the
// seven products midpoint * scale instead (exact as well) took 31 us where
// this takes 14 (8 prompts, 7,292 tokens of 8 heads, d = 128): 21 integer
// instructions an element at half rate.  A NaN or infinity makes the scale NaN:
// the whole group then reads back as NaN.
__device__ __forceinline__ void quantize16(float (&x)[16], int neg_log2, uint2& codes, uint32_t& scale) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(x[i])));
  if (!(top <= 3.402823466e38f)) {
    scale = 0x7Fu;
    codes = make_uint2(0u, 0u);
    return;
  }
  if (neg_log2) {
    const float f = __int_as_float((127 + neg_log2) << 23);
    // far past saturation and far from overflow
    const float most = 1.2e28f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fminf(fmaxf(x[i], -most), most) * f;
    top = fminf(top, most) * f;
  }
  unsigned short two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(__fdiv_rn(top, 6.f)));
  scale = two & 0x7Fu;
  const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2(scale) & 0xFFFFu)));
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;   // a scale of 0 makes every code 0
  const uint64_t inv2 = pack2(inv, inv), minus_s2 = pack2(-s, -s);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {   // two at a time (FFMA2)
      const uint64_t u = pack2(x[8 * i + j], x[8 * i + j + 1]), q = mul2(u, inv2);
      unpack2(fma2(fma2(q, minus_s2, u), inv2, q), y[j], y[j + 1]);
    }
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w[i])
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  }
  codes = make_uint2(w[0], w[1]);
}

constexpr int kAppendThreads = 256;
constexpr int kAppendSmemSeq = 512;   // offsets kept in shared memory up to this many sequences

// One thread per 16 dims of one token's key and value (one KV head).  The
// input is read once and 9 bytes written for its 32 or 64; threads of a warp
// hold consecutive groups of the token, so reads are contiguous and a row's
// codes are written as whole 32-byte sectors.  One wave of CTAs goes over the
// tokens: where a token goes takes three dependent loads (offsets, length,
// page), of which a CTA makes the first two once, and each thread's next
// input is in flight while it rounds the current one.
template <int D, int DT>
__global__ void __launch_bounds__(kAppendThreads, DT == MK_DTYPE_F32 ? 3 : 4)
    kv4_append_kernel(Kv4 c, const uint8_t* k, const uint8_t* v, size_t k_stride, size_t v_stride,
                      bool whole, const int32_t* offsets, int n_tokens, int k_neg, int v_neg) {
  using S = Kv4Shape<D>;
  __shared__ int32_t offs[kAppendSmemSeq + 1], lens[kAppendSmemSeq];
  pdl_trigger();
  pdl_wait();
  constexpr int G = D / kKv4Group, esz = DT == MK_DTYPE_F32 ? 4 : 2;
  // a thread keeps its part of a token (a head's group) and goes from token to
  // token; a token of more parts than threads takes several CTAs
  const int per = c.heads * G, at_once = max(kAppendThreads / per, 1), cuts = (per + kAppendThreads - 1) / kAppendThreads;
  const int part = per <= kAppendThreads ? (int)threadIdx.x % per : (int)(blockIdx.x % cuts) * kAppendThreads + threadIdx.x;
  int tok = per <= kAppendThreads ? (int)blockIdx.x * at_once + (int)threadIdx.x / per : (int)(blockIdx.x / cuts);
  const int step = gridDim.x / cuts * at_once;
  const bool mine = per <= kAppendThreads ? (int)threadIdx.x < at_once * per
                                          : part < per && (int)blockIdx.x < (int)gridDim.x / cuts * cuts;
  const int head = part / G, g = part % G;
  k += (size_t)part * kKv4Group * esz;
  v += (size_t)part * kKv4Group * esz;
  uint4 raw[2][esz];
  auto fetch = [&](int i) {
    if (!mine || i >= n_tokens) return;
#pragma unroll
    for (int j = 0; j < esz; j += 2) {
      load32(k + (size_t)i * k_stride + 16 * j, whole, raw[0][j], raw[0][j + 1]);
      load32(v + (size_t)i * v_stride + 16 * j, whole, raw[1][j], raw[1][j + 1]);
    }
  };
  fetch(tok);
  const bool near = c.n_seq <= kAppendSmemSeq;
  if (near) {
    for (int i = threadIdx.x; i <= c.n_seq; i += kAppendThreads) {
      offs[i] = __ldcg(offsets + i);
      if (i < c.n_seq) lens[i] = __ldcg(c.lens + i);
    }
    __syncthreads();
  }
  if (!mine) return;
  auto at = [&](int i) { return near ? offs[i] : __ldcg(offsets + i); };
  for (; tok < n_tokens; tok += step) {
    int lo = 0, hi = c.n_seq - 1;   // the last sequence whose offset is <= tok
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (at(mid) <= tok) lo = mid; else hi = mid - 1;
    }
    const int first = at(lo), end = at(lo + 1);
    const long long slot = (long long)(near ? lens[lo] : __ldcg(c.lens + lo)) - end + tok;
    // tokens before the first sequence or behind the last, slots out of range: nothing
    const bool ok = tok >= first && tok < end && slot >= 0 && slot < c.capacity();
    const int lp = ok ? (int)((uint32_t)slot / (uint32_t)c.page_tokens) : 0, in = (int)slot - lp * c.page_tokens;
    const int page = ok ? c.page(lo, lp) : -1;
    uint2 codes[2];
    uint32_t scale[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x[16];
      widen_input<DT>(raw[i], x);
      quantize16(x, i ? v_neg : k_neg, codes[i], scale[i]);
    }
    fetch(tok + step);
    if (page < 0) continue;
    uint8_t* b = kv4_block<D>(c, page, head, in / kKv4Block);
    const int row = in % kKv4Block;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<uint2*>(b + (i ? S::kVc : 0) + row * S::kCodes + g * 8) = codes[i];
      b[(i ? S::kVs : S::kKs) + row * S::kScales + g] = (uint8_t)scale[i];
    }
    if (c.scores && g == 0) c.scores[((size_t)lo * c.heads + head) * c.capacity() + slot] = 0.f;
  }
}

// -------------------------------------------------------------------- read

__device__ __forceinline__ void store16(uint8_t* p, int dtype, bool whole, const float (&x)[16]) {
  uint32_t w[16];
  if (dtype == MK_DTYPE_F32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(x[i]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (dtype == MK_DTYPE_BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(x[2 * j + 1]), "f"(x[2 * j]));
      else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(x[2 * j + 1]), "f"(x[2 * j]));
    }
  }
  store32(p, whole, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
  if (dtype == MK_DTYPE_F32)
    store32(p + 32, whole, make_uint4(w[8], w[9], w[10], w[11]), make_uint4(w[12], w[13], w[14], w[15]));
}

__device__ __forceinline__ void widen16(uint2 codes, uint32_t scale, float mul, float (&x)[16]) {
  const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2(scale) & 0xFFFFu))) * mul;
  const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[4];
    e2m1x8(w[i], h);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      x[8 * i + 2 * j] = f.x * s; x[8 * i + 2 * j + 1] = f.y * s;
    }
  }
}

constexpr int kReadThreads = 256;

// One thread per 16 dims of one slot's key and value.  Groups of a row, then
// rows of a block, run along the threads: a warp reads 256 contiguous bytes
// of codes and writes whole rows.  A slot's bytes are found by two dependent
// loads (length and page, then the row), so many warps an SM matter more than
// work per thread: four slots a thread took the same time for a ragged batch of
// 7,292 slots and 5 to 10 us more for one of 4,096.
template <int D>
__global__ void __launch_bounds__(kReadThreads)
    kv4_read_kernel(Kv4 c, int dtype, int n, uint8_t* k_out, uint8_t* v_out, bool whole, float k_mul, float v_mul) {
  using S = Kv4Shape<D>;
  constexpr int G = D / kKv4Group, kRows = kReadThreads / G;
  pdl_trigger();
  pdl_wait();
  const int g = threadIdx.x % G;
  const int slot = blockIdx.x * kRows + threadIdx.x / G;
  const int head = blockIdx.y, s = blockIdx.z;
  const int lp = min(slot, c.capacity() - 1) / c.page_tokens, in = slot - lp * c.page_tokens;
  const int len = c.len(s), page = c.page(s, lp);   // both in flight
  if (slot >= n || slot >= len || page < 0) return;
  const uint8_t* b = kv4_block<D>(c, page, head, in / kKv4Block);
  const int row = in % kKv4Block;
  const uint2 kc = __ldcg(reinterpret_cast<const uint2*>(b + row * S::kCodes + g * 8));
  const uint2 vc = __ldcg(reinterpret_cast<const uint2*>(b + S::kVc + row * S::kCodes + g * 8));
  const uint32_t ks = __ldcg(b + S::kKs + row * S::kScales + g), vs = __ldcg(b + S::kVs + row * S::kScales + g);
  const size_t at = ((((size_t)s * n + slot) * c.heads + head) * D + g * kKv4Group) *
                    (dtype == MK_DTYPE_F32 ? 4 : 2);
  float x[16];
  widen16(kc, ks, k_mul, x);
  store16(k_out + at, dtype, whole, x);
  widen16(vc, vs, v_mul, x);
  store16(v_out + at, dtype, whole, x);
}

// ---------------------------------------------------------------- eviction

// fp32 to an integer of the same order; NaN lowest, both zeros equal.
__device__ __forceinline__ uint32_t score_key(float f) {
  if (f != f) return 0u;
  if (f == 0.f) return 0x80000000u;
  const uint32_t b = __float_as_uint(f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelCtas = 8;   // most CTAs of a head: a portable cluster

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void store_peer(void* mine, int rank, unsigned long long v) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(mine)), b;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(b), "l"(v) : "memory");
}

__device__ __forceinline__ uint32_t load_peer(const void* mine, int rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(mine)), b, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(b) : "memory");
  return v;
}

// Which slots a head keeps: the `take` highest scores between the protected
// ends.  A head's keys are cut into contiguous parts, one for each CTA of a
// cluster, and stay in registers (KPT a thread; longer parts are read from L2
// again for each digit).  The threshold -- the `take`-th highest key -- is found
// a digit of 8 bits at a time from the top: a histogram of the keys that
// share the digits so far in each CTA's shared memory, summed over the
// cluster's.  Accumulated weights share their exponents, so the first digit's
// adds meet on few bins (~10 of a warp's 32 lanes on one); that still costs
// less than counting keys above candidate thresholds bit by bit, which the
// integer pipe bounds: 8 heads of 32,768 keys, one bit a step on one SM each 47
// us, two bits a step over 8 SMs 21 us, digits 13 us (each with cold caches).  A warp whose keys all
// have one digit (scores that are all equal) adds them once.  Slots above the threshold,
// and the lowest of those on it, are then written in slot order by prefix
// sums: position = (# above before) + min(# equal before, equals wanted).
template <int KPT>
__global__ void __launch_bounds__(kSelThreads, 1)
    kv4_select_kernel(Kv4 c, int budget, int first, int last, int ctas, int32_t* kept) {
  __shared__ uint32_t hist[4][256];    // a digit each: no CTA clears one that another still reads
  __shared__ uint32_t cnt[KPT][kSelWarps], sums[kSelWarps], above_warp[8];
  __shared__ uint32_t digit_found, above_found, here_found;
  __shared__ unsigned long long by_cta[kSelCtas];
  pdl_trigger();
  for (int i = threadIdx.x; i < 4 * 256; i += kSelThreads) (&hist[0][0])[i] = 0u;
  pdl_wait();
  const int rank = ctas > 1 ? blockIdx.x % ctas : 0, head = blockIdx.x / ctas, s = blockIdx.y, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int n = c.len(s);
  int32_t* out = kept + ((size_t)s * c.heads + head) * budget;
  const int step = ctas * kSelThreads, from = rank * kSelThreads + tid;
  if (n <= budget) {
    for (int i = from; i < budget; i += step) out[i] = i < n ? i : -1;
    return;
  }
  const int m_all = n - first - last, take = budget - first - last;   // take < m_all
  for (int i = from; i < first; i += step) out[i] = i;
  for (int i = from; i < last; i += step) out[budget - last + i] = n - last + i;
  if (take == 0) return;
  // this CTA's part
  const int part = (m_all + ctas - 1) / ctas, p0 = min(m_all, rank * part), m = min(m_all, p0 + part) - p0;
  const float* sc = c.scores + ((size_t)s * c.heads + head) * c.capacity() + first + p0;
  const bool whole = part <= KPT * kSelThreads;
  uint32_t key[KPT];
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    const int i = j * kSelThreads + tid;
    key[j] = whole && i < m ? score_key(__ldcg(sc + i)) : 0u;
  }
  __syncthreads();   // the histograms are clear

  uint32_t T = 0, want = (uint32_t)take;   // digits so far; the threshold's rank among the keys that have them
  bool exact = false;                      // all keys with these digits are kept: none is on a border
  int shift = 32;
#pragma unroll 1
  for (int d = 0; d < 4 && !exact; ++d) {
    shift -= 8;
    auto add = [&](uint32_t k, bool in) {
      in = in && (d == 0 || k >> (shift + 8) == T >> (shift + 8));
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, in);
      if (mask == 0u) return;
      const uint32_t b = k >> shift & 255u, b0 = __shfl_sync(0xFFFFFFFFu, b, __ffs(mask) - 1);
      if (__all_sync(0xFFFFFFFFu, !in || b == b0)) {
        if (lane == 0) atomicAdd(&hist[d][b0], (uint32_t)__popc(mask));
      } else if (in) {
        atomicAdd(&hist[d][b], 1u);
      }
    };
    if (whole) {
#pragma unroll
      for (int j = 0; j < KPT; ++j) add(key[j], j * kSelThreads + tid < m);
    } else {
      for (int i = tid; i < ((m + 31) & ~31); i += kSelThreads) add(i < m ? score_key(__ldcg(sc + i)) : 0u, i < m);
    }
    if (ctas > 1) { cluster_arrive(); cluster_wait(); }
    else __syncthreads();
    uint32_t mine = 0, inc = 0;
    if (tid < 256) {   // a thread a bin, the highest first
      const int bin = 255 - tid;
      if (ctas > 1) {
        for (int i = 0; i < ctas; ++i) mine += load_peer(&hist[d][bin], i);
      } else {
        mine = hist[d][bin];
      }
      inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += up;
      }
      if (lane == 31) above_warp[warp] = inc;
    }
    __syncthreads();
    if (tid < 256) {
      for (int w = 0; w < warp; ++w) inc += above_warp[w];
      if (inc >= want && inc - mine < want) {
        digit_found = 255 - tid;
        above_found = inc - mine;
        here_found = mine;
      }
    }
    __syncthreads();
    T |= digit_found << shift;
    want -= above_found;
    exact = here_found == want;
  }
  // `want` of the keys with T's digits are kept besides all above them
  auto is_gt = [&](uint32_t k) { return exact ? k >= T : k > T; };
  auto is_eq = [&](uint32_t k) { return !exact && k == T; };
  uint32_t base_gt = 0, base_eq = 0;   // in the CTAs before
  const uint32_t equals = exact ? 0u : want;
  if (ctas > 1) {
    uint32_t gt = 0, eq = 0;
    if (whole) {
#pragma unroll
      for (int j = 0; j < KPT; ++j) {
        const bool in = j * kSelThreads + tid < m;
        gt += in && is_gt(key[j]);
        eq += in && is_eq(key[j]);
      }
    } else {
      for (int i = tid; i < m; i += kSelThreads) {
        const uint32_t k = score_key(__ldcg(sc + i));
        gt += is_gt(k);
        eq += is_eq(k);
      }
    }
    gt = __reduce_add_sync(0xFFFFFFFFu, gt);
    eq = __reduce_add_sync(0xFFFFFFFFu, eq);
    if (lane == 0) { cnt[0][warp] = gt; sums[warp] = eq; }
    __syncthreads();
    if (warp == 0) {
      const unsigned long long t = (unsigned long long)__reduce_add_sync(0xFFFFFFFFu, cnt[0][lane]) |
                                   (unsigned long long)__reduce_add_sync(0xFFFFFFFFu, sums[lane]) << 32;
      if (lane < ctas) store_peer(&by_cta[rank], lane, t);
    }
    cluster_arrive();   // also: no CTA leaves while another reads its histograms
    cluster_wait();
    for (int i = 0; i < rank; ++i) {
      base_gt += (uint32_t)by_cta[i];
      base_eq += (uint32_t)(by_cta[i] >> 32);
    }
  }
  for (int base = 0; base < m; base += KPT * kSelThreads) {
    if (!whole) {
#pragma unroll
      for (int j = 0; j < KPT; ++j) {
        const int i = base + j * kSelThreads + tid;
        key[j] = i < m ? score_key(__ldcg(sc + i)) : 0u;
      }
    }
    uint32_t g_bits = 0, e_bits = 0;   // a bit per j
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const bool in = base + j * kSelThreads + tid < m;
      const bool g = in && is_gt(key[j]), e = in && is_eq(key[j]);
      g_bits |= (uint32_t)g << j;
      e_bits |= (uint32_t)e << j;
      const uint32_t bg = __ballot_sync(0xFFFFFFFFu, g), be = __ballot_sync(0xFFFFFFFFu, e);
      if (lane == 0) cnt[j][warp] = (uint32_t)__popc(bg) << 16 | (uint32_t)__popc(be);
    }
    __syncthreads();
    // exclusive prefix over (j, warp), counts above in the high half (at most 16,384 of each)
    const bool mine = tid < KPT * kSelWarps;
    const uint32_t own = mine ? cnt[tid >> 5][lane] : 0u;
    uint32_t inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    const uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sums[lane] : 0u);
    if (mine) cnt[tid >> 5][lane] = before + inc - own;
    const uint32_t all = __reduce_add_sync(0xFFFFFFFFu, sums[lane]);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const uint32_t bg = __ballot_sync(0xFFFFFFFFu, g_bits >> j & 1u),
                     be = __ballot_sync(0xFFFFFFFFu, e_bits >> j & 1u);
      const uint32_t lt = (1u << lane) - 1u, p = cnt[j][warp];
      const uint32_t ng = base_gt + (p >> 16) + __popc(bg & lt), ne = base_eq + (p & 0xFFFFu) + __popc(be & lt);
      if ((g_bits >> j & 1u) || ((e_bits >> j & 1u) && ne < equals))
        out[first + ng + min(ne, equals)] = first + p0 + base + j * kSelThreads + tid;
    }
    base_gt += all >> 16;
    base_eq += all & 0xFFFFu;
    __syncthreads();
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveLanes = 8;    // threads of a row
constexpr int kMoveRows = 4;     // rows of a thread, their loads in flight together

// Copies the kept rows to their place in the other cache: 8 threads a row, 16
// (d = 128) or 8 bytes of codes each, the scales beside the first of K and V.
// A row that has no page, here or there, is skipped: callers give every slot that lens counts one.
template <int D>
__global__ void __launch_bounds__(kMoveThreads)
    kv4_move_kernel(Kv4 src, Kv4 dst, int budget, const int32_t* kept) {
  using S = Kv4Shape<D>;
  using Code = typename std::conditional<D == 128, uint4, uint2>::type;
  using Scale = typename std::conditional<D == 128, uint2, uint32_t>::type;
  constexpr int kPer = kMoveThreads / kMoveLanes;
  pdl_trigger();
  pdl_wait();
  const int head = blockIdx.y, s = blockIdx.z;
  const int t = threadIdx.x % kMoveLanes, which = t / 4, piece = t % 4;
  const int32_t* list = kept + ((size_t)s * src.heads + head) * budget;
  const size_t row_of_scores = (size_t)s * src.heads + head;
  int from[kMoveRows], to[kMoveRows];
  Code code[kMoveRows];
  Scale scale[kMoveRows];
  float score[kMoveRows];
#pragma unroll
  for (int i = 0; i < kMoveRows; ++i) {
    to[i] = (blockIdx.x * kMoveRows + i) * kPer + threadIdx.x / kMoveLanes;
    from[i] = to[i] < budget ? __ldcg(list + to[i]) : -1;
  }
#pragma unroll
  for (int i = 0; i < kMoveRows; ++i) {
    if (from[i] < 0 || from[i] >= src.capacity()) { from[i] = -1; continue; }
    const int lp = from[i] / src.page_tokens, in = from[i] - lp * src.page_tokens;
    const int page = src.page(s, lp);
    if (piece == 1 && which == 0 && src.scores) score[i] = __ldcg(src.scores + row_of_scores * src.capacity() + from[i]);
    if (page < 0) { from[i] = -2; continue; }
    const uint8_t* b = kv4_block<D>(src, page, head, in / kKv4Block);
    const int row = in % kKv4Block;
    code[i] = __ldcg(reinterpret_cast<const Code*>(b + (which ? S::kVc : 0) + row * S::kCodes) + piece);
    if (piece == 0) scale[i] = __ldcg(reinterpret_cast<const Scale*>(b + (which ? S::kVs : S::kKs) + row * S::kScales));
  }
#pragma unroll
  for (int i = 0; i < kMoveRows; ++i) {
    if (from[i] == -1 || to[i] >= dst.capacity()) continue;
    if (piece == 1 && which == 0 && dst.scores) dst.scores[row_of_scores * dst.capacity() + to[i]] = src.scores ? score[i] : 0.f;
    const int lp = to[i] / dst.page_tokens, in = to[i] - lp * dst.page_tokens;
    const int page = dst.page(s, lp);
    if (page < 0 || from[i] == -2) continue;
    uint8_t* b = kv4_block<D>(dst, page, head, in / kKv4Block);
    const int row = in % kKv4Block;
    *(reinterpret_cast<Code*>(b + (which ? S::kVc : 0) + row * S::kCodes) + piece) = code[i];
    if (piece == 0) *reinterpret_cast<Scale*>(b + (which ? S::kVs : S::kKs) + row * S::kScales) = scale[i];
  }
}

static int dtype_bytes(int dtype) {
  return dtype == MK_DTYPE_F32 ? 4 : (dtype == MK_DTYPE_BF16 || dtype == MK_DTYPE_F16) ? 2 : 0;
}

}  // namespace mk

using namespace mk;

extern "C" size_t mk_kv4_page_bytes(int n_kv_heads, int head_dim, int page_tokens) {
  if (n_kv_heads < 1 || n_kv_heads > 1024 || (head_dim != 64 && head_dim != 128) ||
      page_tokens < kKv4Block || page_tokens % kKv4Block)
    return 0;
  return (size_t)n_kv_heads * page_tokens * (head_dim + head_dim / 8);
}

extern "C" int mk_kv4_append(const mk_kv4_cache* cache, const void* k_dev, const void* v_dev, int dtype,
                             long long k_stride, long long v_stride, const int32_t* offsets_dev,
                             int n_tokens, void* stream) {
  const char* who = "mk_kv4_append";
  if (int rc = kv4_check(cache, who)) return rc;
  const int esz = dtype_bytes(dtype);
  if (!esz) return kv4_fail(MK_ERR_INVALID_ARG, who, "dtype is one of MK_DTYPE_*");
  if (n_tokens < 0 || n_tokens > 1 << 30) return kv4_fail(MK_ERR_INVALID_ARG, who, "n_tokens is 0 to 2^30");
  if (!offsets_dev || (reinterpret_cast<uintptr_t>(offsets_dev) & 3u))
    return kv4_fail(MK_ERR_INVALID_ARG, who, "offsets are a 4-byte aligned array");
  if (n_tokens == 0) return MK_OK;
  if (!k_dev || !v_dev) return kv4_fail(MK_ERR_INVALID_ARG, who, "no keys or values");
  const long long row = (long long)cache->n_kv_heads * cache->head_dim;
  if (k_stride < row || v_stride < row || k_stride > (1ll << 40) || v_stride > (1ll << 40))
    return kv4_fail(MK_ERR_INVALID_ARG, who, "a token's stride is at least n_kv_heads * head_dim");
  if (((reinterpret_cast<uintptr_t>(k_dev) | reinterpret_cast<uintptr_t>(v_dev)) & 15u) ||
      (k_stride * esz) % 16 || (v_stride * esz) % 16)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "keys and values of a token are 16-byte aligned");
  const Kv4 c = kv4_of(cache);
  const int per = c.heads * (cache->head_dim / kKv4Group);   // threads of a token
  const int at_once = per < kAppendThreads ? kAppendThreads / per : 1, cuts = (per + kAppendThreads - 1) / kAppendThreads;
  const int sms = device_sms();
  if (!sms) return kv4_fail(MK_ERR_CUDA, who, "no device");
  const int wave = (dtype == MK_DTYPE_F32 ? 3 : 4) * sms;
  long long blocks = ((long long)n_tokens + at_once - 1) / at_once * cuts;
  if (blocks > wave) blocks = wave > cuts ? wave / cuts * cuts : cuts;
  const uint8_t* k = static_cast<const uint8_t*>(k_dev);
  const uint8_t* v = static_cast<const uint8_t*>(v_dev);
  const size_t ks = (size_t)k_stride * esz, vs = (size_t)v_stride * esz;
  const bool whole = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | ks | vs) & 31u) == 0;
  const bool wide = cache->head_dim == 128;
  auto kernel = dtype == MK_DTYPE_F32 ? (wide ? kv4_append_kernel<128, MK_DTYPE_F32> : kv4_append_kernel<64, MK_DTYPE_F32>)
                : dtype == MK_DTYPE_BF16 ? (wide ? kv4_append_kernel<128, MK_DTYPE_BF16> : kv4_append_kernel<64, MK_DTYPE_BF16>)
                                         : (wide ? kv4_append_kernel<128, MK_DTYPE_F16> : kv4_append_kernel<64, MK_DTYPE_F16>);
  const cudaError_t e = pdl_launch(kernel, dim3((unsigned)blocks), dim3(kAppendThreads), 0,
                                   static_cast<cudaStream_t>(stream), c, k, v, ks, vs, whole, offsets_dev,
                                   n_tokens, -cache->k_log2, -cache->v_log2);
  return e == cudaSuccess ? MK_OK : kv4_fail(MK_ERR_CUDA, who, cudaGetErrorString(e));
}

extern "C" int mk_kv4_read(const mk_kv4_cache* cache, int dtype, int n, void* k_out_dev, void* v_out_dev,
                           void* stream) {
  const char* who = "mk_kv4_read";
  if (int rc = kv4_check(cache, who)) return rc;
  if (!dtype_bytes(dtype)) return kv4_fail(MK_ERR_INVALID_ARG, who, "dtype is one of MK_DTYPE_*");
  if (n < 0) return kv4_fail(MK_ERR_INVALID_ARG, who, "n is not negative");
  if (n == 0) return MK_OK;
  if (!k_out_dev || !v_out_dev) return kv4_fail(MK_ERR_INVALID_ARG, who, "no outputs");
  if ((reinterpret_cast<uintptr_t>(k_out_dev) | reinterpret_cast<uintptr_t>(v_out_dev)) & 15u)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "outputs are 16-byte aligned");
  const Kv4 c = kv4_of(cache);
  const int rows = kReadThreads / (cache->head_dim / kKv4Group);
  const int most = n < c.capacity() ? n : c.capacity();
  const bool whole = ((reinterpret_cast<uintptr_t>(k_out_dev) | reinterpret_cast<uintptr_t>(v_out_dev)) & 31u) == 0;
  auto kernel = cache->head_dim == 128 ? kv4_read_kernel<128> : kv4_read_kernel<64>;
  const cudaError_t e = pdl_launch(kernel, dim3((unsigned)((most + rows - 1) / rows), c.heads, c.n_seq),
                                   dim3(kReadThreads), 0, static_cast<cudaStream_t>(stream), c, dtype, n,
                                   static_cast<uint8_t*>(k_out_dev), static_cast<uint8_t*>(v_out_dev), whole,
                                   ldexpf(1.f, cache->k_log2), ldexpf(1.f, cache->v_log2));
  return e == cudaSuccess ? MK_OK : kv4_fail(MK_ERR_CUDA, who, cudaGetErrorString(e));
}

extern "C" int mk_kv4_evict(const mk_kv4_cache* src, const mk_kv4_cache* dst, int budget, int keep_first,
                            int keep_last, int32_t* kept_dev, void* stream) {
  const char* who = "mk_kv4_evict";
  if (int rc = kv4_check(src, who)) return rc;
  if (int rc = kv4_check(dst, who)) return rc;
  if (src->n_kv_heads != dst->n_kv_heads || src->head_dim != dst->head_dim || src->n_seq != dst->n_seq ||
      src->k_log2 != dst->k_log2 || src->v_log2 != dst->v_log2)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "both caches have the same heads, head_dim, sequences and log2");
  if (!src->scores_dev) return kv4_fail(MK_ERR_INVALID_ARG, who, "the source has scores");
  if (budget < 1 || budget > (long long)dst->pages_per_seq * dst->page_tokens)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "budget is 1 to the destination's capacity");
  if (keep_first < 0 || keep_last < 0 || (long long)keep_first + keep_last > budget)
    return kv4_fail(MK_ERR_INVALID_ARG, who, "keep_first + keep_last is 0 to budget");
  if (!kept_dev || (reinterpret_cast<uintptr_t>(kept_dev) & 3u))
    return kv4_fail(MK_ERR_INVALID_ARG, who, "kept is a 4-byte aligned array");
  if (dst->scores_dev == src->scores_dev ||
      (src->pool_dev == dst->pool_dev && src->table_dev == dst->table_dev))
    return kv4_fail(MK_ERR_INVALID_ARG, who, "the destination has pages and scores of its own");
  const Kv4 a = kv4_of(src), b = kv4_of(dst);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // 2 or 4 keys a thread in as many CTAs as the longest head can need (the fewer keys
  // an SM counts, the faster); past 8 CTAs of them 16 keys a thread
  const int per_cta = 4 * kSelThreads;
  int ctas = 1;
  while (ctas < kSelCtas && (long long)ctas * per_cta < a.capacity()) ctas <<= 1;
  auto select = a.capacity() <= 2 * kSelThreads ? kv4_select_kernel<2>
                : (long long)ctas * per_cta < a.capacity() ? kv4_select_kernel<16> : kv4_select_kernel<4>;
  cudaError_t e = pdl_launch_cluster(select, dim3(a.heads * ctas, a.n_seq), dim3(kSelThreads), ctas, st, a, budget,
                                     keep_first, keep_last, ctas, kept_dev);
  if (e != cudaSuccess) return kv4_fail(MK_ERR_CUDA, who, cudaGetErrorString(e));
  const int rows = kMoveThreads / kMoveLanes * kMoveRows;
  auto move = src->head_dim == 128 ? kv4_move_kernel<128> : kv4_move_kernel<64>;
  e = pdl_launch(move, dim3((budget + rows - 1) / rows, a.heads, a.n_seq), dim3(kMoveThreads), 0, st, a, b,
                 budget, kept_dev);
  return e == cudaSuccess ? MK_OK : kv4_fail(MK_ERR_CUDA, who, cudaGetErrorString(e));
}

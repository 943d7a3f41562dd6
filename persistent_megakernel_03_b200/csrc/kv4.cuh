// kv4.cuh -- the 4-bit KV cache: its layout and the code that every kernel on
// it shares.
//
// 16 consecutive dims of a key (or value) row share one e4m3 scale; each dim
// is an e2m1 code (0 .5 1 1.5 2 3 4 6 and a sign), so a value is
//   code * scale * 2^log2,
// 4.5 bits.  A code has 2 significant bits and a scale 4: the product has at
// most 6 and a unit of at least 2^-10, which fp16 and bf16 both hold exactly.
// Kernels therefore widen to 16 bits without a rounding.
//
// A block is kKv4Block keys of one KV head, contiguous:
//   K codes [32][d/2], K scales [32][d/16], V codes [32][d/2], V scales [32][d/16]
// (byte i of a row of codes: dim 2i in the low nibble).  A page is
// [n_kv_heads][page_tokens / 32] blocks, so the 64 to 128 bytes that a step
// appends per head are whole sectors, and a warp of the attention streams
// 4,608 contiguous bytes (d = 128) for 32 keys and their values.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mk.h"

namespace mk {

void set_last_error(const char* msg);  // api.cu: the message mk_last_error(NULL) returns

constexpr int kKv4Block = 32;   // keys of a block
constexpr int kKv4Group = 16;   // dims that share a scale
constexpr int kKv4MaxSeq = 4096;

// What the kernels need of an mk_kv4_cache.
struct Kv4 {
  uint8_t* pool;
  const int32_t* table;   // null: sequence s owns pages s * pps ...
  const int32_t* lens;
  float* scores;
  int32_t heads, page_tokens, pages, n_seq, pps;

  __host__ __device__ int capacity() const { return pps * page_tokens; }
  // Physical page of a sequence's logical page, -1 where it has none.
  __device__ __forceinline__ int page(int s, int lp) const {
    const int p = table ? __ldcg(table + (size_t)s * pps + lp) : s * pps + lp;
    return p >= 0 && p < pages ? p : -1;
  }
  // Keys of a sequence; a length out of range is cut to it.
  __device__ __forceinline__ int len(int s) const {
    const int n = __ldcg(lens + s);
    return n < 0 ? 0 : (n > capacity() ? capacity() : n);
  }
};

template <int D>
struct Kv4Shape {
  static constexpr int kCodes = D / 2;                    // bytes of a row's codes
  static constexpr int kScales = D / kKv4Group;           // and of its scales
  static constexpr int kKs = kKv4Block * kCodes;          // offsets inside a block
  static constexpr int kVc = kKs + kKv4Block * kScales;
  static constexpr int kVs = kVc + kKv4Block * kCodes;
  static constexpr int kBytes = kVs + kKv4Block * kScales;
};

template <int D>
__device__ __forceinline__ uint8_t* kv4_block(const Kv4& c, int page, int head, int in_page) {
  const int per = c.page_tokens / kKv4Block;
  return c.pool + (((size_t)page * c.heads + head) * per + in_page) * Kv4Shape<D>::kBytes;
}

// Two e2m1 codes of a byte as fp16 values (low nibble in the low half), for
// each byte of a word: cvt converts 42 pairs a clock and SM, shifts and masks of the
// nibbles 25 (the probe's own three instructions counted in both).
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two e4m3 scales (low byte in the low half) as fp16.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
  return h;
}

// 2^x: 2^-22 of the value, 0 for -inf.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Checks an mk_kv4_cache; 0 or an MK_ERR_* code, with the reason in
// mk_last_error(NULL).  `who` names the entry point.
int kv4_check(const mk_kv4_cache* c, const char* who);
// SMs of the current device (asked for once a device), 0 without one.
int device_sms();
int kv4_fail(int code, const char* who, const char* why);
Kv4 kv4_of(const mk_kv4_cache* c);

}  // namespace mk

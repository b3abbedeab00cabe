// Shared by the kernels of the 8-bit key/value cache (cosmot_kv8_*).
//
// A cached element is an e4m3 byte times the float32 scale of its (sequence,
// head, block of rows), keys and values apart.  e4m3 -> f16 is exact, so the
// tensor cores see f16 operands (or the bytes themselves) and the scales act
// on the float32 side: a key block's scale multiplies its scores, and a value
// block's scale is added to the exponent of its softmax weights,
//     p vs = 2^(x - m + log2 vs),   sum p = sum (p vs) / vs,
// so that no element needs a multiplication of its own.  P is f16 or bf16 for the
// tensor cores: each kernel says how it keeps the spread of the scales out of
// their range.  The store writes powers of two in [2^-40, 2^40]; with those every
// sum stays inside float32.
#pragma once

#include <cuda_fp16.h>

#include "cosmot_internal.h"
#include "ptx.cuh"

namespace cosmot {
namespace kv8 {

constexpr int kScaleExpLo = -40, kScaleExpHi = 40;
constexpr float kE4m3Max = 448.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Cache {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;  // [batch][n_kv_heads][n_blocks]
  float* v_scale;
  const int32_t* lens;
  int64_t ld, bstride;  // elements between rows, rows between sequences
  int32_t batch, capacity, n_kv, hd, block, n_blocks;
};

// Query-side parameters of attention and weighing.  Rows are packed per key
// head: row r of (sequence, key head g) is query r / group of head g * group +
// r % group, so that the heads that share a key head share its tiles.
struct Query {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;  // [batch][n_heads][n_q], NULL: not written
  int64_t ld_q, ld_o, q_bstride, o_bstride;
  int64_t n_q, n_rows;  // n_rows = n_q * group
  int32_t n_heads, group, n_new;
  int32_t causal;
  float scale_log2;  // softmax scale * log2(e)
  // split of the keys (workspace): O'' [split][batch][n_kv][n_rows][hd] and (m, l)
  int32_t splits, chunk;  // chunk: keys of a split (register-tile kernels)
  float* part_o;
  float2* part_ml;
  int64_t part_rows;  // rows that the workspace has room for (debug store checks)
  int* status;
};

// Rows that sequence b shows: lens[b] + n_new, held inside the cache whatever
// the device array says (a value outside reports COSMOT_ERR_BOUNDS).
__device__ __forceinline__ int32_t shown_rows(const Cache& c, int32_t b, int32_t n_new, int* status, bool report) {
  const int32_t held = c.lens[b];
  if (held >= 0 && held <= c.capacity - n_new) return held + n_new;
  if (report) report_status(status, COSMOT_ERR_BOUNDS, kWhereKv8Lens);
  return held < 0 ? 0 : c.capacity;
}

// Query and head (within its key head's group) of packed row r.  n_rows < 2^30:
// 32-bit division, which a warp's short prologue notices.
__device__ __forceinline__ int32_t row_query(const Query& p, int64_t r) { return (int32_t)((uint32_t)r / (uint32_t)p.group); }
__device__ __forceinline__ int32_t row_head(const Query& p, int64_t r) { return (int32_t)((uint32_t)r % (uint32_t)p.group); }

// First hidden key of packed row r (n_rows and beyond: padding, sees nothing).
__device__ __forceinline__ int32_t row_limit(const Query& p, int64_t r, int32_t len) {
  if (r >= p.n_rows) return 0;
  if (!p.causal) return len;
  const int32_t lim = len - (int32_t)p.n_q + row_query(p, r) + 1;
  return lim < 0 ? 0 : (lim < len ? lim : len);
}

// (e4m3, e4m3) -> (f16, f16), exact; byte 0 goes to the low half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(b));
  return r;
}
__device__ __forceinline__ uint32_t cvt_lo(uint32_t w) { return e4m3x2_to_f16x2((uint16_t)(w & 0xffffu)); }
__device__ __forceinline__ uint32_t cvt_hi(uint32_t w) { return e4m3x2_to_f16x2((uint16_t)(w >> 16)); }

// (lo, hi) floats -> two e4m3 bytes, to nearest even, saturating.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// 2^x of a whole x in [-126, 127] held as a float.
__device__ __forceinline__ float exp2_whole(float x) {
  return __int_as_float(__float_as_int(x + (12582912.f + 127.f)) << 23);  // 1.5 * 2^23: the sum's low bits are x + 127
}

// log2 of a positive scale and the factor 2^-log2, both exact for a power of two.
__device__ __forceinline__ void scale_log2_parts(float s, float& log2s, float& inv) {
  const uint32_t u = __float_as_uint(s);
  int e = (int)((u >> 23) & 255u) - 127;
  e = e < -126 ? -126 : (e > 126 ? 126 : e);
  const float frac = __log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u));  // 0 for a power of two
  log2s = (float)e + frac;
  inv = exp2_int(-e) * ex2_approx(-frac);
}

// Smallest e in [kScaleExpLo, kScaleExpHi] with amax <= 448 * 2^e (448 = 0.875 * 2^9).
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int x = (int)(u >> 23) - 126;  // amax = m * 2^x, m in [0.5, 1)
  int e = (u & 0x7fffffu) <= 0x600000u ? x - 9 : x - 8;  // m <= 0.875
  if (amax == 0.f) e = kScaleExpLo;
  return e < kScaleExpLo ? kScaleExpLo : (e > kScaleExpHi ? kScaleExpHi : e);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Natural logarithm of l 2^ref, where l is near 2^bias and ref near -bias: the
// whole bias (exact in both) goes before the logarithm, so that a sum near one
// keeps its last digits.
__device__ __forceinline__ float log_sum(float ref, float l, float bias) {
  return ((ref + bias) + log2f(l * exp2_whole(-bias))) * kLn2;
}

// Key splits of a row: split s gives o_s = sum 2^(x - ref_s) v8 and (ref_s,
// l_s) with l_s = sum 2^(x - ref_s) / vs; where a split shows the row nothing,
// l_s = 0 and o_s is zero or was not written (each kernel says which).
constexpr int kMaxSplits = 256;

// Checked host-side views of the public structs.
cosmot_status make_cache(const cosmot_kv8_cache* c, Cache& out);
cosmot_status make_query(const cosmot_kv8_cache* c, const cosmot_kv8_query* d, Query& out);
// Register-tile kernels (kv8_rows.cu): few packed rows.
cosmot_status rows_attention(const Cache& c, const Query& p, cudaStream_t s);
cosmot_status rows_weigh(const Cache& c, const Query& p, float decay, float* weight, int32_t max_len, cudaStream_t s);
// Sets the key split of a register-tile attention call.
void rows_plan(const Cache& c, Query& p, int32_t max_len);
// tcgen05 kernels (kv8_tile.cu): many packed rows.  max_len: what the host
// takes the longest sequence to show; it sizes the split of the work only.
bool tile_fits(const Cache& c, const Query& p);  // else UNSUPPORTED: more work items than a grid counts
size_t tile_workspace(const Cache& c, const Query& p, int32_t max_len);
cosmot_status tile_attention(const Cache& c, const Query& p, int32_t max_len, void* workspace, cudaStream_t s);
cosmot_status tile_weigh(const Cache& c, const Query& p, float decay, float* weight, int32_t max_len, cudaStream_t s);

}  // namespace kv8
}  // namespace cosmot

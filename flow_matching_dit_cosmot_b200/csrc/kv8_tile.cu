// Attention and weighing over the 8-bit cache for many query rows, on the
// tcgen05 tensor cores (TMEM accumulators).
//
// Attention.  One CTA per (sequence, key head, 256 packed query rows) and, for
// the items of the last wave, per key split.  512 threads in four warpgroups:
//   warp 0       owns TMEM and issues the MMAs:
//                  S_t = Q_t K_j^T   (M 128, N 128, K head_dim; both in smem)
//                  O_t += P_t V_j    (A = P in TMEM over S)
//                in the order S0 S1 | PV0 S0' PV1 S1' | ..., so that one tile's
//                products run beside the other tile's softmax.
//   warps 1-7    read the cache's bytes (16 a load), widen them to f16 (exact)
//                and write the 128-byte-swizzled tiles that the MMAs read, a K
//                and a V tile ahead in registers and four slots ahead in smem.
//   warps 8-11   softmax of rows 0-127, warps 12-15 of rows 128-255, a row per
//                thread; first they bring their rows of Q into smem as f16, by a
//                power of two per row (its largest magnitude in [2^13, 2^14):
//                exact down to 2^-31 of it).
// The scales of a 128-key tile come with its keys, one for each 128 / NG keys:
//     x = s (q factor)(ks) + y,   p 2^y = 2^(x - m + 10)  (f16 in TMEM),
// m the running maximum of x; it is followed only when it grows by more than
// 2^5, so p 2^y stays below 2^15.  l = sum (p 2^y) / 2^y stays in float32.
// Where the value scales of a CTA's keys lie within 2^2 of one another (warp 0
// looks at them all while the queries come in), vs = 2^(y + unit), unit the
// largest's log2 and O in units of 2^unit: f16 keeps full precision down to 2^-22
// of the largest weight, a step of 2^-32 of it below.  Otherwise vs = 2^(y + shift
// + unit) with -1 < y <= 0: V's tile is widened times 2^shift, exact from 2^-15 to
// 2^7, and the unit moves from tile to tile so that the tile's scales fit (O
// changes by a power of two then, like for a maximum that moved).  Only blocks of
// one tile further apart than 2^22 leave a rest in y, and the smaller ones'
// weights lose digits by it.
// 1,560 queries x 14,106 rows x 32 heads: 365 us with near scales, 380 with random
// ones in 2^4, 427 in 2^40; 363 where any spread went into y, which is wrong for
// far ones.  P as two bf16 where scales are far took 10 % more with near ones too
// (the softmax's registers), the same shifts for every CTA 6 to 10 %.
// bound: the chain S -> softmax -> PV of a query tile, two tiles half a period
// apart: 3,340 cycles a key tile (2,800 without the exponentials; the products
// alone 2,048).  The same sizes: 409 us = 880 TFLOP/s in long runs under the power
// cap, 365 us (986) on a cool card; tensor pipe and SFU at 50 %.
// Registers a thread: 176 for the softmax and 80 for the other warps measured
// best (184 / 72 +2 %, 192 / 64 +6 %, 168 / 88 +5 %).
//
// Weighing.  One CTA per (sequence, key head, 256 keys): the keys are widened
// to bf16 once and stay in smem, the queries' tiles come by TMA as they are
// (bf16), and every thread of four warpgroups owns one query row of a tile:
// per group of 16 keys it adds 2^(s f - lse).  Nothing but the sums leaves the
// CTA; a cluster may share the queries of one key range, and the sums are
// joined in a fixed order.  A quarter of the exponentials runs on the FMA pipe.
// bound: the SFU (62 % busy) and the issue slots (64 %).  The same sizes: 230 us
// in long runs, 213 on a cool card (an SFU floor of 156; the products alone 131);
// with every exponential on the SFU 257 where a quarter off it took 233, three
// eighths 244.
#include "kv8.cuh"

#include <climits>
#include <mutex>

namespace cosmot {
namespace kv8 {
namespace {

constexpr int kTile = 128;                    // rows of a query tile, keys of a key tile
constexpr int kSlots = 4;
constexpr int kBoxBytes = 128 * 64 * 2;       // 128 rows x 64 columns of 16 bits, 128-byte swizzle
constexpr float kTileBias = 10.f;
constexpr float kFollow = 5.f;                // log2 units
constexpr float kFold = 2.f;                  // spread of the value scales' log2 that the weights' exponents take
constexpr int kShiftLo = -15, kShiftHi = 7;   // powers of two by which e4m3 stays exact in f16

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Byte offset of 16-byte piece `piece` (of 8 columns) of `row` in a tile of boxes of 64 columns.
template <int BOX = kBoxBytes>
__device__ __forceinline__ uint32_t sw_offset(int row, int piece) {
  return (uint32_t)((piece >> 3) * BOX + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// 32 bytes to a 32-byte-aligned address.
__device__ __forceinline__ void st_global32(void* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int* status, int where) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, where));
}

// ------------------------------------------------------------------ attention
// Registers: 256 threads x (kRegsIo + kRegsSoftmax) must not exceed the launch's pool (the launch checks it).
constexpr int kAttnThreads = 512;
constexpr int kRegsIo = 80, kRegsSoftmax = 176;
constexpr int kConvWarps = 7;

struct TilePlan {
  int32_t pairs;    // pairs of query tiles of a (sequence, key head)
  int32_t n_full;   // leading items that one CTA takes whole
  int32_t n_lo;     // the next ones, `splits` CTAs each
  int32_t n_hi;     // the last ones, splits + 1 CTAs each
  int32_t splits;
  // CTAs behind the whole items; each writes 2 * kTile rows of partial results
  __host__ __device__ int32_t n_parts() const { return n_lo * splits + n_hi * (splits + 1); }
};

template <int HD>
struct AttnCfg {
  static constexpr int kTileBytes = kTile * HD * 2;
  static constexpr int kScaleBytes = 4 * 8 * 16;  // four key tiles in flight, eight groups each
  static constexpr int kSmem = (2 + kSlots) * kTileBytes + 256 + kScaleBytes + 1024;
  static constexpr uint32_t kIdescS = idesc_f16_f32(kTile, kTile, false);
  static constexpr uint32_t kIdescO = idesc_f16_f32(kTile, HD, true);
  __device__ static constexpr uint32_t s_col(int t) { return (uint32_t)t * 128u; }
  __device__ static constexpr uint32_t o_col(int t) { return 256u + (uint32_t)t * HD; }
};

// NG: groups of keys with their own scale in a key tile, 128 / block.
template <int HD, int NG>
__global__ void __launch_bounds__(kAttnThreads, 1)
    tile_attention_kernel(const __grid_constant__ Cache c, const __grid_constant__ Query p,
                          const __grid_constant__ TilePlan plan) {
  using C = AttnCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = smem_u32(smem);
  const uint32_t sKV = sQ + 2 * C::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (2 + kSlots) * C::kTileBytes);
  const uint32_t bar_q = smem_u32(bars);
  const uint32_t bar_kv_full = bar_q + 8;                 // [kSlots]
  const uint32_t bar_kv_empty = bar_kv_full + 8 * kSlots; // [kSlots]
  const uint32_t bar_s_full = bar_kv_empty + 8 * kSlots;  // [2]
  const uint32_t bar_p_half = bar_s_full + 16;            // [2] P of keys 0-63 written
  const uint32_t bar_p_full = bar_p_half + 16;            // [2] P of keys 64-127 written
  const uint32_t bar_o_done = bar_p_full + 16;            // [1]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 1 + 2 * kSlots + 7);
  const uint32_t bar_span = smem_u32(bars + 24);            // [1] vs_top is written
  volatile int32_t* vs_top = reinterpret_cast<int32_t*>(bars + 25);  // log2 of the largest value scale; whether all are near
  // [4][NG] (ks, y, 2^-y, unit)
  float4* scales = reinterpret_cast<float4*>(smem + (2 + kSlots) * C::kTileBytes + 256);
  constexpr int kGroupKeys = kTile / NG;

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
  // work item: the pairs of all heads in turn (causal: the longest first)
  int32_t item = (int32_t)blockIdx.x, split = 0, splits = 1;
  const int32_t slot_of_part = item - plan.n_full;
  if (slot_of_part >= 0) {
    const int32_t lo = plan.n_lo * plan.splits;
    splits = slot_of_part < lo ? plan.splits : plan.splits + 1;
    const int32_t t = slot_of_part < lo ? slot_of_part : slot_of_part - lo;
    split = t % splits;
    item = plan.n_full + (slot_of_part < lo ? 0 : plan.n_lo) + t / splits;
  }
  const int32_t heads = c.batch * c.n_kv;
  const int32_t bg = item % heads, b = bg / c.n_kv, kvh = bg % c.n_kv;
  const int32_t pair = p.causal ? plan.pairs - 1 - item / heads : item / heads;
  const int64_t r0 = (int64_t)pair * 2 * kTile;
  const bool two = r0 + kTile < p.n_rows;

  if (threadIdx.x == 0) {
    mbar_init(bar_q, 8);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar_kv_full + 8 * s, kConvWarps);
      mbar_init(bar_kv_empty + 8 * s, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_s_full + 8 * t, 1);
      mbar_init(bar_p_half + 8 * t, 4);
      mbar_init(bar_p_full + 8 * t, 4);
    }
    mbar_init(bar_o_done, 1);
    mbar_init(bar_span, 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // up to here only the CTA's own shared and tensor memory and the parameters were touched
  pdl_trigger();
  pdl_wait();
  const int32_t len = shown_rows(c, b, p.n_new, p.status, threadIdx.x == 0);
  const int64_t r_end = r0 + 2 * kTile < p.n_rows ? r0 + 2 * kTile : p.n_rows;
  const int32_t kend = row_limit(p, r_end - 1, len);
  const int32_t n_kt = (kend + kTile - 1) / kTile;
  const int32_t kt0 = (int32_t)((int64_t)split * n_kt / splits), kt1 = (int32_t)((int64_t)(split + 1) * n_kt / splits);
  const int32_t n_vis = __shfl_sync(0xffffffffu, kt1 - kt0, 0);  // key tiles of this CTA
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(tmem_slot), 0);

  if (warp < 8) {
    setmaxnreg_dec<kRegsIo>();
    if (warp == 0) {
    // The whole warp walks the loop and one lane issues: with uniform control flow
    // the operands stay in uniform registers.
    if (n_vis > 0) {
      const uint32_t leader = elect_one();
      auto issue_s = [&](int t, int slot) {
        const uint32_t qa = sw128_desc_lo(sQ + t * C::kTileBytes, 16), ka = sw128_desc_lo(sKV + slot * C::kTileBytes, 16);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t off = ((k >> 2) * kBoxBytes + (k & 3) * 32) >> 4;
          umma_ss_lo(leader, tmem_base + C::s_col(t), qa + off, ka + off, C::kIdescS, k > 0 ? 1u : 0u);
        }
      };
      auto issue_pv = [&](int t, int slot, bool acc, int half) {  // keys 64 half .. 64 half + 63
        const uint32_t va = sw128_desc_lo(sKV + slot * C::kTileBytes, kBoxBytes);
#pragma unroll
        for (int k = 4 * half; k < 4 * half + 4; ++k)  // 16 keys: two 8-row swizzle atoms = 2048 bytes
          umma_ts_lo(leader, tmem_base + C::o_col(t), tmem_base + C::s_col(t) + 8 * k, va + (2048 >> 4) * k, C::kIdescO,
                     (acc || k > 0) ? 1u : 0u);
      };
      auto wait = [&](uint32_t bar, uint32_t par) { return warp_wait(bar, par, p.status, kWhereKv8Mma); };
      auto kv_wait = [&](int L) { return wait(bar_kv_full + 8 * (L % kSlots), (L / kSlots) & 1); };
      {  // the value scales of this CTA's keys, mostly near one another
        const float* vsp = c.v_scale + (int64_t)bg * c.n_blocks;
        const int32_t end = min(kt1 * NG, (kend + kGroupKeys - 1) / kGroupKeys);
        int hi = INT_MIN, lo = INT_MAX;  // positive floats order like their bits
#pragma unroll 8
        for (int32_t i = kt0 * NG + lane; i < end; i += 32) {
          const int v = __float_as_int(load_global(vsp + i));
          hi = max(hi, v);
          lo = min(lo, v);
        }
        hi = __reduce_max_sync(0xffffffffu, hi);
        lo = __reduce_min_sync(0xffffffffu, lo);
        float top, low, inv;
        scale_log2_parts(__int_as_float(hi), top, inv);
        scale_log2_parts(__int_as_float(lo), low, inv);
        if (lane == 0) {
          vs_top[0] = (int)ceilf(top);
          vs_top[1] = top - low <= kFold;
          mbar_arrive(bar_span);
        }
        __syncwarp();
      }
      bool ok = wait(bar_q, 0) && kv_wait(0);
      if (ok) {
        tc_fence_after();
        issue_s(0, 0);
        umma_commit_if(leader, bar_s_full);
        if (two) {
          issue_s(1, 0);
          umma_commit_if(leader, bar_s_full + 8);
        }
        umma_commit_if(leader, bar_kv_empty);
      }
      for (int j = 0; j < n_vis && ok; ++j) {
        const int LV = 2 * j + 1, LK = 2 * j + 2;
        const bool has_next = j + 1 < n_vis;
        const uint32_t par = j & 1;
        if (!kv_wait(LV) || !wait(bar_p_half, par)) break;
        tc_fence_after();
        issue_pv(0, LV % kSlots, j > 0, 0);
        if (!wait(bar_p_full, par)) break;
        tc_fence_after();
        issue_pv(0, LV % kSlots, true, 1);
        if (has_next) {
          if (!kv_wait(LK)) break;
          tc_fence_after();
          issue_s(0, LK % kSlots);
          umma_commit_if(leader, bar_s_full);
        }
        if (two) {
          if (!wait(bar_p_half + 8, par)) break;
          tc_fence_after();
          issue_pv(1, LV % kSlots, j > 0, 0);
          if (!wait(bar_p_full + 8, par)) break;
          tc_fence_after();
          issue_pv(1, LV % kSlots, true, 1);
        }
        umma_commit_if(leader, bar_kv_empty + 8 * (LV % kSlots));
        if (has_next) {
          if (two) {
            issue_s(1, LK % kSlots);
            umma_commit_if(leader, bar_s_full + 8);
          }
          umma_commit_if(leader, bar_kv_empty + 8 * (LK % kSlots));
        }
      }
      umma_commit_if(leader, bar_o_done);
      mbar_drain(bar_o_done, 0, p.status, kWhereKv8Drain);
    }
    __syncwarp();
    } else {
    // ---------------------------------------------------------- widening
    // The widening warps live on 80 registers: addresses that step along keep them
    // from spilling in this loop, which costs up to 10 % where it paces the tile.
    // A warp takes 32 pieces of 16 bytes at a time, kRows whole rows; the tile's
    // row groups go round the seven warps.  Eight neighbouring lanes write two
    // rows' pieces of one box: their chunks of 16 bytes fall on all banks (four
    // pieces give every other chunk of a row).
    constexpr int kRows = HD == 128 ? 4 : 8, kRowGroups = kTile / kRows;
    constexpr int kLoads = (kRowGroups + kConvWarps - 1) / kConvWarps, kStep = kConvWarps * kRows;
    const int cw = warp - 1;
    const int u = HD == 128 ? (lane & 3) | ((lane >> 1) & 4) : lane & 3;
    const int row = cw * kRows + (HD == 128 ? ((lane >> 2) & 1) | ((lane >> 4) << 1) : lane >> 2);
    const int64_t start = ((int64_t)b * c.bstride + (int64_t)kt0 * kTile + row) * c.ld + (int64_t)kvh * HD + u * 16;
    const uint8_t* kp = c.k + start;  // this lane's first row of the next tile to load
    const uint8_t* vp = c.v + start;
    int32_t left_k = kend - kt0 * kTile - row, left_v = left_k;  // rows from there to the end
    uint4 wk[kLoads], wv[kLoads];
    auto load = [&](uint4 (&w)[kLoads], const uint8_t*& from, int32_t& left) {
      const uint8_t* at = from;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        w[i] = make_uint4(0, 0, 0, 0);
        if (row + i * kStep < kTile && i * kStep < left) w[i] = load_global(reinterpret_cast<const uint4*>(at));
        at += (int64_t)kStep * c.ld;
      }
      from += (int64_t)kTile * c.ld;
      left -= kTile;
    };
    // A row's place in a tile: kStep rows on, the swizzle's row bits change by kStep & 7, which is 0 or 4.
    static_assert(kStep % 4 == 0, "the swizzle of a lane's next row");
    const uint32_t place = sKV + sw_offset(row, 2 * u);
    auto widen = [&](const uint4 (&w)[kLoads], int slot) {
      const uint32_t dst = place + slot * C::kTileBytes;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (row + i * kStep >= kTile) break;
        const uint32_t to = (dst ^ ((i * kStep & 4) << 4)) + i * kStep * 128;
        st_shared16(to, cvt_lo(w[i].x), cvt_hi(w[i].x), cvt_lo(w[i].y), cvt_hi(w[i].y));
        st_shared16(to ^ 16, cvt_lo(w[i].z), cvt_hi(w[i].z), cvt_lo(w[i].w), cvt_hi(w[i].w));
      }
    };
    // the same times 2^shift, the lane's shift that of its group of keys
    auto widen_shifted = [&](const uint4 (&w)[kLoads], int slot, int shift) {
      const uint32_t dst = place + slot * C::kTileBytes;
      const uint32_t by = pack_f16x2(exp2_int(shift), exp2_int(shift));
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = row + i * kStep;
        const uint32_t f = __shfl_sync(0xffffffffu, by, NG == 1 ? 0 : min(r / kGroupKeys, NG - 1));
        if (r >= kTile) break;
        const uint32_t to = (dst ^ ((i * kStep & 4) << 4)) + i * kStep * 128;
        st_shared16(to, mul_f16x2(cvt_lo(w[i].x), f), mul_f16x2(cvt_hi(w[i].x), f), mul_f16x2(cvt_lo(w[i].y), f),
                    mul_f16x2(cvt_hi(w[i].y), f));
        st_shared16(to ^ 16, mul_f16x2(cvt_lo(w[i].z), f), mul_f16x2(cvt_hi(w[i].z), f), mul_f16x2(cvt_lo(w[i].w), f),
                    mul_f16x2(cvt_hi(w[i].w), f));
      }
    };
    auto empty = [&](int L) {
      return warp_wait(bar_kv_empty + 8 * (L % kSlots), ((L / kSlots) & 1) ^ 1, p.status, kWhereKv8Widen);
    };
    auto full = [&](int L) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_kv_full + 8 * (L % kSlots));
    };
    if (n_vis > 0) {
      load(wk, kp, left_k);
      load(wv, vp, left_v);
    }
    if (n_vis > 0 && warp_wait(bar_span, 0, p.status, kWhereKv8Widen) && !vs_top[1]) {
      int unit = vs_top[0];  // (every warp finds the same units and shifts: nothing is exchanged for them)
#pragma unroll 1
      for (int j = 0; j < n_vis; ++j) {
        float4 sc = make_float4(1.f, 0.f, 0.f, 0.f);  // a group behind the end: finite, and every key masked
        int shift = 0;
        const int32_t g = (kt0 + j) * NG + lane;
        const bool live = lane < NG && g * kGroupKeys < kend;
        if (live) {
          sc.x = load_global(c.k_scale + (int64_t)bg * c.n_blocks + g);
          scale_log2_parts(load_global(c.v_scale + (int64_t)bg * c.n_blocks + g), sc.y, sc.z);
        }
        const int e = live ? (int)ceilf(sc.y) : INT_MIN;
        const int hi = __reduce_max_sync(0xffffffffu, e), lo = __reduce_min_sync(0xffffffffu, live ? e : INT_MAX);
        unit = max(hi - kShiftHi, min(unit, lo - kShiftLo));
        sc.w = (float)unit;
        if (live) {
          const int by = max(e, unit + kShiftLo);
          shift = by - unit;
          sc.y -= (float)by;
          sc.z *= exp2_int(min(max(by, -126), 127));
        }
        if (!empty(2 * j)) break;
        widen(wk, (2 * j) % kSlots);
        if (cw == 0 && lane < NG) scales[(j & 3) * NG + lane] = sc;
        full(2 * j);
        if (j + 1 < n_vis) load(wk, kp, left_k);
        if (!empty(2 * j + 1)) break;
        widen_shifted(wv, (2 * j + 1) % kSlots, shift);
        full(2 * j + 1);
        if (j + 1 < n_vis) load(wv, vp, left_v);
      }
    } else {
      for (int j = 0; j < n_vis; ++j) {
        const int32_t kt = kt0 + j;
        float4 sc = make_float4(1.f, 0.f, 0.f, (float)vs_top[0]);  // a group behind the end: finite, and every key masked
        if (cw == 0 && lane < NG && kt * kTile + lane * kGroupKeys < kend) {
          const int64_t at = (int64_t)bg * c.n_blocks + kt * NG + lane;
          sc.x = load_global(c.k_scale + at);
          scale_log2_parts(load_global(c.v_scale + at), sc.y, sc.z);
          sc.y -= sc.w;
          sc.z *= exp2_whole(sc.w);
        }
        if (!empty(2 * j)) break;
        widen(wk, (2 * j) % kSlots);
        if (cw == 0 && lane < NG) scales[(j & 3) * NG + lane] = sc;
        full(2 * j);
        if (j + 1 < n_vis) load(wk, kp, left_k);
        if (!empty(2 * j + 1)) break;
        widen(wv, (2 * j + 1) % kSlots);
        full(2 * j + 1);
        if (j + 1 < n_vis) load(wv, vp, left_v);
      }
    }
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ---------------------------------------------------------- softmax
    const int t = (warp - 8) >> 2;           // query tile
    const int lane_base = (warp & 3) * 32;   // TMEM lanes this warp may access
    const int64_t r = r0 + t * kTile + lane_base + lane;
    const bool valid = r < p.n_rows;
    const int32_t qi = valid ? row_query(p, r) : 0;
    const int32_t h = kvh * p.group + (valid ? (int32_t)r - qi * p.group : 0);
    // Q: a warp's 32 rows come into their places as bf16, whole rows at a time;
    // then every lane turns its own row into f16 where it lies.  Short loops: a
    // CTA runs this once, and code that was never run comes in slowly.
    float fac = p.scale_log2;
    if (n_vis > 0 && (t == 0 || two)) {
      constexpr int kLanes = HD / 8, kRows = 32 / kLanes;  // lanes of a row, rows of one copy
      const int64_t at = (int64_t)(b * p.q_bstride + qi) * p.ld_q + (int64_t)h * HD;  // this lane's own row
      const uint32_t tile = sQ + t * C::kTileBytes;
      const int piece = lane % kLanes;
#pragma unroll 2
      for (int i = 0; i < 32 / kRows; ++i) {
        const int row = i * kRows + lane / kLanes;
        const int64_t from = __shfl_sync(0xffffffffu, at, row);
        const int live = __shfl_sync(0xffffffffu, (int)valid, row) ? 16 : 0;  // 0: zeros
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tile + sw_offset(lane_base + row, piece)),
                     "l"(p.q + from + piece * 8), "r"(live)
                     : "memory");
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      uint32_t mag = 0;  // magnitudes of bf16 order like their bits
#pragma unroll 4
      for (int i = 0; i < kLanes; ++i) {
        const uint4 x = ld_shared16(tile + sw_offset(lane_base + lane, i));
        mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
      }
      mag = max(mag & 0xffffu, mag >> 16);
      // below 2^-47 a row loses bits of less than 2^-85: nothing that a key could raise to a visible score
      int e2 = (int)(mag >> 7) - 127 - 13;
      e2 = e2 < -60 ? -60 : (e2 > 114 ? 114 : e2);
      const float down = exp2_int(-e2);
      fac = mag < 0x7f80u ? fmaxf(p.scale_log2 * exp2_int(e2), 1e-25f) : __int_as_float(0x7fc00000);
#pragma unroll 2
      for (int i = 0; i < kLanes; ++i) {
        const uint32_t where = tile + sw_offset(lane_base + lane, i);
        const uint4 x = ld_shared16(where);
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = unpack_bf16x2(w[e]);
          y[e] = pack_f16x2(v.x * down, v.y * down);
        }
        st_shared16(where, y[0], y[1], y[2], y[3]);
      }
      fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_q);

    const uint32_t s_addr = tmem_base + ((uint32_t)lane_base << 16) + C::s_col(t);
    const uint32_t o_addr = tmem_base + ((uint32_t)lane_base << 16) + C::o_col(t);
    const int32_t lim = valid ? row_limit(p, r, len) : kend;  // padding rows see all: they never force the masks
    const bool live = __any_sync(0xffffffffu, valid);  // the warp has a row to answer for
    float m = -INFINITY, l = 0.f, unit = 0.f;  // O is in units of 2^unit
    bool ok = true;
    if (t == 0 || two) {
#pragma unroll 1
      for (int j = 0; j < n_vis; ++j) {
        const int32_t kbase = (kt0 + j) * kTile;
        // warp-uniform decisions only: every tcgen05.ld/st below is .sync.aligned
        if (!warp_wait(bar_s_full + 8 * t, j & 1, p.status, kWhereKv8Softmax)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (!live) {  // what P and O hold in these lanes reaches no other row
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar_p_half + 8 * t);
            mbar_arrive(bar_p_full + 8 * t);
          }
          continue;
        }
        uint32_t s[128];
        tmem_ld32(s_addr + 0, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
        tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
        tmem_ld32(s_addr + 64, *reinterpret_cast<uint32_t(*)[32]>(&s[64]));
        tmem_ld32(s_addr + 96, *reinterpret_cast<uint32_t(*)[32]>(&s[96]));
        const float4* sc = scales + (j & 3) * NG;
        tmem_ld_wait();
        if (kbase + kTile > lim) {
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (kbase + e >= lim) s[e] = 0xff800000u;
        }
        float4 kept[NG];  // the tile's scales, for the exponentials (16-key groups read them again)
        float m_new = m;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          constexpr int kChains = NG == 1 ? 4 : 2;  // independent three-input chains
          float mx[kChains];
#pragma unroll
          for (int q = 0; q < kChains; ++q) mx[q] = -INFINITY;
#pragma unroll
          for (int e = 0; e < kGroupKeys; e += 2 * kChains)
#pragma unroll
            for (int q = 0; q < kChains; ++q)
              mx[q] = fmax3(mx[q], __uint_as_float(s[kGroupKeys * g + e + 2 * q]), __uint_as_float(s[kGroupKeys * g + e + 2 * q + 1]));
          float x = fmaxf(mx[0], mx[1]);
          if constexpr (kChains == 4) x = fmaxf(x, fmaxf(mx[2], mx[3]));
          const float4 k = sc[g];
          if constexpr (NG <= 4) kept[g] = k;
          m_new = fmaxf(m_new, fmaf(x, fac * k.x, k.y));
        }
        const float unit_now = sc[0].w;
        const bool moved = unit_now != unit && j > 0;
        const bool first = m == -INFINITY;
        const bool need = !first && m_new > m + kFollow;
        float factor = 1.f;
        if (first) {
          m = m_new;
        } else if (need) {
          factor = ex2_approx(m - m_new);
          m = m_new;
          l *= factor;
        }
        if (__any_sync(0xffffffffu, need || moved)) {
          if (moved) factor *= exp2_whole(fminf(fmaxf(unit - unit_now, -126.f), 126.f));
#pragma unroll 1
          for (int i = 0; i < HD / 32; ++i) {
            uint32_t ov[32];
            tmem_ld32(o_addr + 32 * i, ov);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * factor);
            tmem_st32(o_addr + 32 * i, ov);
          }
          tmem_st_wait();
        }
        unit = unit_now;
        const float mu = m == -INFINITY ? 0.f : m - kTileBias;
#pragma unroll
        for (int g2 = 0; g2 < 4; ++g2) {  // 32 keys
          uint32_t pk[16];
          constexpr int kRun = kGroupKeys < 32 ? kGroupKeys : 32;  // keys of one scale
#pragma unroll
          for (int g = 0; g < 32 / kRun; ++g) {
            float4 k;
            if constexpr (NG <= 4)
              k = kept[(32 * g2 + kRun * g) / kGroupKeys];
            else
              k = sc[(32 * g2 + kRun * g) / kGroupKeys];
            const float f = fac * k.x, off = k.y - mu;
            const uint64_t f2 = pack_f32x2(f, f), off2 = pack_f32x2(off, off);
            float rs0 = 0.f, rs1 = 0.f;  // (packed sums measured slower)
#pragma unroll
            for (int e = 0; e < kRun / 2; ++e) {
              const int at = 32 * g2 + kRun * g + 2 * e;
              float p0, p1;
              unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), f2, off2), p0, p1);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              rs0 += p0;
              rs1 += p1;
              pk[kRun / 2 * g + e] = pack_f16x2(p0, p1);
            }
            l = fmaf(rs0 + rs1, k.z, l);
          }
          tmem_st16(s_addr + 16 * g2, pk);
          if (g2 == 1) {  // P of keys 0-63 is in TMEM: PV over them may start
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_p_half + 8 * t);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p_full + 8 * t);
      }
    }
    const float ref = m - kTileBias;  // o = sum 2^(x - ref) v8, l = sum 2^(x - ref) / vs
    if (t == 0 || two) {
      if (n_vis > 0) {
        ok = ok && warp_wait(bar_o_done, 0, p.status, kWhereKv8Softmax);
        tc_fence_after();
      }
      const bool none = l == 0.f;  // the row saw nothing here
      const int64_t pr = (int64_t)slot_of_part * 2 * kTile + t * kTile + lane_base + lane;
      const bool store = valid && dcheck(qi < p.n_q && h < p.n_heads && (splits == 1 || (pr >= 0 && pr < p.part_rows)),
                                         p.status, kWhereKv8Store);
      const float inv = (splits > 1 ? 1.f : 1.f / l) * exp2_whole(unit);
      if (store && ok) {
        if (splits > 1)
          p.part_ml[pr] = make_float2(none ? -INFINITY : ref, l);
        else if (p.lse)
          p.lse[((int64_t)b * p.n_heads + h) * p.n_q + qi] = none ? -INFINITY : log_sum(ref, l, kTileBias);
      }
      __nv_bfloat16* dst = p.o + (b * p.o_bstride + qi) * p.ld_o + (int64_t)h * HD;
      float* pdst = p.part_o + pr * HD;
      const bool wide = (((uintptr_t)p.o | (uintptr_t)(p.ld_o * 2)) & 31) == 0;  // whole sectors: 32 bytes a store
      if (ok) {
#pragma unroll 1
        for (int i = 0; i < HD / 32; ++i) {
          uint32_t ov[32];
          if (n_vis > 0) {
            tmem_ld32(o_addr + 32 * i, ov);
            tmem_ld_wait();
          }
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = none ? 0.f : __uint_as_float(ov[e]) * inv;
          if (store && splits > 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) st_global32(pdst + 32 * i + 8 * e, reinterpret_cast<const uint32_t*>(v) + 8 * e);
          } else if (store) {
            uint32_t y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
            if (wide) {
              st_global32(dst + 32 * i, y);
              st_global32(dst + 32 * i + 16, y + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint4*>(dst + 32 * i + 8 * e) = make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem_base, 512);
}

// Joins the key splits, in their order: hd / 4 lanes a row of a split item, 4
// columns each.  (The few-row join's CTA a row took 23 us where this takes 11,
// for 76 items of three or four splits.)
constexpr int kTileJoinThreads = 256;

template <int HD>
__global__ void __launch_bounds__(kTileJoinThreads) tile_join_kernel(const __grid_constant__ Cache c,
                                                                     const __grid_constant__ Query p,
                                                                     const __grid_constant__ TilePlan plan) {
  pdl_trigger();
  pdl_wait();
  constexpr int kLanes = HD / 4, kRowsOfCta = kTileJoinThreads / kLanes;
  constexpr int kCtas = 2 * kTile / kRowsOfCta;  // of an item
  const int32_t i = (int32_t)(blockIdx.x / kCtas);
  const int32_t row = (int32_t)(blockIdx.x % kCtas) * kRowsOfCta + (int32_t)threadIdx.x / kLanes;
  const bool lo = i < plan.n_lo;
  const int splits = lo ? plan.splits : plan.splits + 1;
  const int64_t part = lo ? (int64_t)i * plan.splits
                          : (int64_t)plan.n_lo * plan.splits + (int64_t)(i - plan.n_lo) * (plan.splits + 1);
  const int32_t heads = c.batch * c.n_kv, item = plan.n_full + i, bg = item % heads, b = bg / c.n_kv, kvh = bg % c.n_kv;
  const int32_t pair = p.causal ? plan.pairs - 1 - item / heads : item / heads;
  const int64_t r = (int64_t)pair * 2 * kTile + row;
  if (r >= p.n_rows) return;
  const int64_t pr = part * 2 * kTile + row;
  const int col = ((int)threadIdx.x % kLanes) * 4;
  const float2* ml = p.part_ml + pr;
  float ref = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float2 x = ml[(int64_t)s * 2 * kTile];
    if (x.y != 0.f) ref = fmaxf(ref, x.x);
  }
  float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  const float* src = p.part_o + pr * HD + col;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float2 m = ml[(int64_t)s * 2 * kTile];
    // (a range that shows the row nothing wrote zeros)
    const float4 x = *reinterpret_cast<const float4*>(src + (int64_t)s * 2 * kTile * HD);
    const float f = m.y == 0.f ? 0.f : ex2_approx(m.x - ref);
    l = fmaf(f, m.y, l);
    acc[0] = fmaf(f, x.x, acc[0]);
    acc[1] = fmaf(f, x.y, acc[1]);
    acc[2] = fmaf(f, x.z, acc[2]);
    acc[3] = fmaf(f, x.w, acc[3]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int32_t qi = row_query(p, r), h = kvh * p.group + (int32_t)r - qi * p.group;
  if (!dcheck(qi < p.n_q && h < p.n_heads, p.status, kWhereKv8Store)) return;
  *reinterpret_cast<uint2*>(p.o + (b * p.o_bstride + qi) * p.ld_o + (int64_t)h * HD + col) =
      make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  if (col == 0 && p.lse)
    p.lse[((int64_t)b * p.n_heads + h) * p.n_q + qi] = l == 0.f ? -INFINITY : log_sum(ref, l, kTileBias);
}

// ------------------------------------------------------------------ weighing
// Warp 0 loads the queries' tiles (TMA), warp 1 issues the products, warps 2-7
// widen the next item's keys, four warpgroups (warps 8-23) own the rows of two
// query tiles x two key tiles; warp 3 adds their sums up, two items behind.
// Items (256 keys of a sequence and key head) go round the CTAs; nothing drains
// between two.
// Registers: 256 x kWeighRegsIo + 512 x kWeighRegsRows out of the launch's pool.
constexpr int kWeighThreads = 768, kWeighConvWarps = 6;
constexpr int kWeighRegsIo = 64, kWeighRegsRows = 88;
constexpr int kWeighMaxCluster = 4;
constexpr int kQSlots = 3;
constexpr int kWeighLens = 64;
constexpr int kPolyPairs = 2;  // of 8 pairs of exponentials, those on the FMA pipe

template <int HD>
struct WeighCfg {
  static constexpr int kTileBytes = kTile * HD * 2;
  static constexpr int kBars = (4 + kQSlots) * kTileBytes;  // two buffers of two key tiles, the queries' ring
  static constexpr int kSums = kBars + 192;                 // [2][4 warpgroups][4 warps][8 groups]
  static constexpr int kParts = kSums + 2 * 4 * 4 * 8 * 4;  // [2][cluster][16 groups]
  static constexpr int kLens = kParts + 2 * kWeighMaxCluster * 16 * 4;  // the first sequences' lengths
  static constexpr int kSmem = kLens + kWeighLens * 4 + 1024;
  static constexpr int kBoxK = 2 * kBoxBytes;  // 256 keys x 64 columns
  static constexpr uint32_t kIdesc2 = idesc_bf16_f32(kTile, 2 * kTile, false, false);  // both key tiles at once
  static constexpr uint32_t kIdesc1 = idesc_bf16_f32(kTile, kTile, false, false);
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

constexpr float kExp2C1 = 6.931470037e-01f, kExp2C2 = 2.402224243e-01f, kExp2C3 = 5.550733581e-02f, kExp2C4 = 9.671512991e-03f, kExp2C5 = 1.326472731e-03f;

// Into [-127, 128], NaN kept.
__device__ __forceinline__ float clamp_exp2(float x) {
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;\n\tmin.NaN.f32 %0, %0, 0f43000000;" : "+f"(x));
  return x;
}

// 2^x of a pair on the FMA pipe: n = round(x), 2^n by its exponent bits (zero
// at -127, infinity at 128), 2^(x - n) by a polynomial of degree 5
// with constant 1, fitted here for the least relative error on [-1/2, 1/2]
// (1.9e-7 of the value, float32 arithmetic included).
__device__ __forceinline__ void exp2_fma(uint64_t x, float& y0, float& y1) {
  float a, b;
  unpack_f32x2(x, a, b);
  x = pack_f32x2(clamp_exp2(a), clamp_exp2(b));
  const uint64_t magic = pack_f32x2(12582912.f, 12582912.f);  // 1.5 * 2^23: the sum's low bits are round(x)
  const uint64_t t = add_f32x2(x, magic);
  const uint64_t f = fma_f32x2(add_f32x2(t, pack_f32x2(-12582912.f, -12582912.f)), pack_f32x2(-1.f, -1.f), x);
  uint64_t r = pack_f32x2(kExp2C5, kExp2C5);
  r = fma_f32x2(r, f, pack_f32x2(kExp2C4, kExp2C4));
  r = fma_f32x2(r, f, pack_f32x2(kExp2C3, kExp2C3));
  r = fma_f32x2(r, f, pack_f32x2(kExp2C2, kExp2C2));
  r = fma_f32x2(r, f, pack_f32x2(kExp2C1, kExp2C1));
  r = fma_f32x2(r, f, pack_f32x2(1.f, 1.f));
  float t0, t1, r0, r1;
  unpack_f32x2(t, t0, t1);
  unpack_f32x2(r, r0, r1);
  y0 = r0 * __int_as_float((__float_as_int(t0) << 23) + 0x3f800000);
  y1 = r1 * __int_as_float((__float_as_int(t1) << 23) + 0x3f800000);
}

struct WeighItem {
  int32_t bg, b, k0, k_end, len, i0, n_i;  // keys [k0, k_end), query tiles [i0, i0 + n_i) of this CTA; k_end = k0: none
  bool two;
};

// (32-bit arithmetic: every warp does this for every item)
__device__ __forceinline__ WeighItem weigh_item(const Cache& c, const Query& p, uint32_t item, int32_t q_tile, int32_t n_all,
                                                int32_t rank, int32_t ranks, const int32_t* lens) {
  WeighItem w;
  const uint32_t heads = (uint32_t)c.batch * (uint32_t)c.n_kv;  // one key range of every head, then the next
  w.bg = (int32_t)(item % heads);
  w.b = c.batch == 1 ? 0 : (int32_t)((uint32_t)w.bg / (uint32_t)c.n_kv);
  w.k0 = (int32_t)(item / heads) * 2 * kTile;
  w.len = w.b < kWeighLens ? lens[w.b] : shown_rows(c, w.b, p.n_new, p.status, threadIdx.x == 0 && rank == 0);
  w.len = __shfl_sync(0xffffffffu, w.len, 0);
  w.k_end = min(w.len, w.k0 + 2 * kTile);
  if (w.k0 >= w.len) w.k_end = w.k0;
  w.two = w.k0 + kTile < w.k_end;
  // query tiles that see a key of the range (causal: the last ones), shared by the cluster
  int32_t first = w.k_end > w.k0 ? 0 : n_all;
  if (p.causal && w.k_end > w.k0) {  // query i sees keys <= len - n_q + i
    const int32_t q_first = w.k0 - (w.len - (int32_t)p.n_q);
    if (q_first > 0) first = (int32_t)((uint32_t)q_first / (uint32_t)q_tile);  // < n_all as k0 < len
  }
  w.i0 = first;
  w.n_i = n_all - first;
  if (ranks > 1) {
    const int32_t n = n_all - first;
    w.i0 = first + (int32_t)((int64_t)n * rank / ranks);
    w.n_i = first + (int32_t)((int64_t)n * (rank + 1) / ranks) - w.i0;
  }
  return w;
}

// q_tile: queries of a tile (kTile / group), its rows q_tile * group <= 128;
// n_all: the query tiles; ranges: key ranges of 256 in the capacity.
template <int HD>
__global__ void __launch_bounds__(kWeighThreads, 1)
    tile_weigh_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ Cache c,
                      const __grid_constant__ Query p, float decay, float* weight, int32_t q_tile,
                      int32_t n_all, int32_t ranges) {
  using C = WeighCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sK = smem_u32(smem);
  const uint32_t sQ = sK + 4 * C::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars);
  const uint32_t bar_q_full = smem_u32(bars);              // [kQSlots]
  const uint32_t bar_q_empty = bar_q_full + 8 * kQSlots;   // [kQSlots]
  const uint32_t bar_s_full = bar_q_empty + 8 * kQSlots;   // [2]
  const uint32_t bar_s_empty = bar_s_full + 16;            // [2]
  const uint32_t bar_k_full = bar_s_empty + 16;            // [2]
  const uint32_t bar_k_empty = bar_k_full + 16;            // [2]
  const uint32_t bar_sum_full = bar_k_empty + 16;          // [2]
  const uint32_t bar_sum_empty = bar_sum_full + 16;        // [2]
  const uint32_t bar_done = bar_sum_empty + 16;            // [1]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kQSlots + 13);
  float* sums = reinterpret_cast<float*>(smem + C::kSums);
  float* parts = reinterpret_cast<float*>(smem + C::kParts);
  int32_t* lens = reinterpret_cast<int32_t*>(smem + C::kLens);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int32_t ranks = gridDim.y, rank = blockIdx.y;  // the cluster runs along y
  const uint32_t items = (uint32_t)c.batch * (uint32_t)c.n_kv * (uint32_t)ranges;  // < 2^31
  const int32_t tile_rows = q_tile * p.group;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kQSlots; ++s) {
      mbar_init(bar_q_full + 8 * s, 1);
      mbar_init(bar_q_empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_s_full + 8 * s, 1);
      mbar_init(bar_s_empty + 8 * s, 8);
      mbar_init(bar_k_full + 8 * s, kWeighConvWarps);
      mbar_init(bar_k_empty + 8 * s, 1);
      mbar_init(bar_sum_full + 8 * s, 16);
      mbar_init(bar_sum_empty + 8 * s, 1);
    }
    mbar_init(bar_done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp >= 8 && tile_rows < kTile) {  // the rows of a query tile that TMA never writes
    const int pieces = (kTile - tile_rows) * (HD / 8);
    for (int i = (int)threadIdx.x - 256; i < kQSlots * pieces; i += 512) {
      const int q = i % pieces;
      st_shared16(sQ + (i / pieces) * C::kTileBytes + sw_offset(tile_rows + q / (HD / 8), q % (HD / 8)), 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  pdl_trigger();
  pdl_wait();
  for (int i = (int)threadIdx.x; i < kWeighLens && i < c.batch; i += kWeighThreads)
    lens[i] = shown_rows(c, i, p.n_new, p.status, blockIdx.x == 0 && rank == 0);
  tc_fence_before();
  if (ranks > 1)
    cluster_sync();  // every CTA of the cluster has started before anything is written to it
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(tmem_slot), 0);

  if (warp < 8) {
  setmaxnreg_dec<kWeighRegsIo>();
  if (warp == 0) {
    tma_prefetch_desc(&tmap_q);
    int n = 0;  // tiles so far
    bool ok = true;
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
      const WeighItem w = weigh_item(c, p, item, q_tile, n_all, rank, ranks, lens);
      for (int i = 0; i < w.n_i && ok; ++i, ++n) {
        const int slot = n % kQSlots;
        ok = warp_wait(bar_q_empty + 8 * slot, ((n / kQSlots) & 1) ^ 1, p.status, kWhereKv8Widen);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar_q_full + 8 * slot, (uint32_t)tile_rows * HD * 2);
          for (int bx = 0; bx < HD / 64; ++bx)
            tma_load_4d(sQ + slot * C::kTileBytes + bx * kBoxBytes, &tmap_q, bar_q_full + 8 * slot, bx * 64,
                        (w.bg % c.n_kv) * p.group, (w.i0 + i) * q_tile, w.b);
        }
        __syncwarp();
      }
      if (ranks > 1) cluster_sync();
    }
    // every copy lands before the CTA may exit
    for (int i = n > kQSlots ? n - kQSlots : 0; i < n; ++i)
      mbar_drain(bar_q_full + 8 * (i % kQSlots), (i / kQSlots) & 1, p.status, kWhereKv8Drain);
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t leader = elect_one();
    int n = 0, done = 0;  // query tiles, items
    bool ok = true;
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
      const WeighItem w = weigh_item(c, p, item, q_tile, n_all, rank, ranks, lens);
      if (w.n_i > 0 && ok) {
        const int kbuf = done & 1;
        const uint32_t idesc = w.two ? C::kIdesc2 : C::kIdesc1;
        const uint32_t ka = sw128_desc_lo(sK + 2 * kbuf * C::kTileBytes, 16);
        ok = warp_wait(bar_k_full + 8 * kbuf, (done >> 1) & 1, p.status, kWhereKv8Mma);
        for (int i = 0; i < w.n_i && ok; ++i, ++n) {
          const int slot = n % kQSlots, phase = n & 1;
          ok = warp_wait(bar_q_full + 8 * slot, (n / kQSlots) & 1, p.status, kWhereKv8Mma) &&
               warp_wait(bar_s_empty + 8 * phase, ((n >> 1) & 1) ^ 1, p.status, kWhereKv8Mma);
          if (!ok) break;
          tc_fence_after();
          const uint32_t qa = sw128_desc_lo(sQ + slot * C::kTileBytes, 16);
#pragma unroll
          for (int k = 0; k < HD / 16; ++k)
            umma_ss_lo(leader, tmem_base + 256u * phase, qa + (((k >> 2) * kBoxBytes + (k & 3) * 32) >> 4),
                       ka + (((k >> 2) * C::kBoxK + (k & 3) * 32) >> 4), idesc, k > 0 ? 1u : 0u);
          umma_commit_if(leader, bar_s_full + 8 * phase);
          umma_commit_if(leader, bar_q_empty + 8 * slot);
        }
        if (ok) umma_commit_if(leader, bar_k_empty + 8 * kbuf);
        ++done;
      }
      if (ranks > 1) cluster_sync();
    }
    umma_commit_if(leader, bar_done);
    mbar_drain(bar_done, 0, p.status, kWhereKv8Drain);
    __syncwarp();
  } else {
    // keys to bf16 (exact), rows behind the end zero; the warps take four (hd 64: eight) rows in turn
    constexpr int kRows = HD == 128 ? 4 : 8, kStep = kWeighConvWarps * kRows, kAhead = 6;
    const int u = HD == 128 ? (lane & 3) | ((lane >> 1) & 4) : lane & 3;
    const int row0 = (warp - 2) * kRows + (HD == 128 ? ((lane >> 2) & 1) | ((lane >> 4) << 1) : lane >> 2);
    int done = 0, live = 0, added = 0;  // items converted, items with keys, items whose sums were added up
    bool ok = true;
    WeighItem last[2];
    // 16 group sums of this CTA, then of the cluster, each added in a fixed order
    auto add_up = [&](const WeighItem& w, int at) {
      if (warp == 3) ok = ok && warp_wait(bar_sum_full + 8 * (at & 1), (at >> 1) & 1, p.status, kWhereKv8Softmax);
      float* my_parts = parts + (at & 1) * kWeighMaxCluster * 16;
      if (warp == 3) {
        const float* my_sums = sums + (at & 1) * 128;
        const int kt = (lane >> 3) & 1, g = lane & 7;
        float x = 0.f;
#pragma unroll
        for (int ph = 0; ph < 2; ++ph)
#pragma unroll
          for (int q = 0; q < 4; ++q) x += my_sums[((2 * ph + kt) * 4 + q) * 8 + g];
        if (lane < 16) {
          if (ranks > 1)
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(my_parts + rank * 16 + lane), 0)),
                         "f"(x)
                         : "memory");
          else
            my_parts[lane] = x;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_sum_empty + 8 * (at & 1));
      }
      if (ranks > 1) cluster_sync();
      if (warp == 3 && rank == 0 && ok) {
        const int n_groups = c.block / 16;  // groups of a block
        const int32_t key = w.k0 + lane * c.block;
        if (lane < 16 / n_groups && key < w.k_end) {
          float y = 0.f;
          for (int r = 0; r < ranks; ++r)
            for (int e = 0; e < n_groups; ++e) y += my_parts[r * 16 + lane * n_groups + e];
          const int32_t blk = key / c.block;
          if (dcheck(blk < c.n_blocks, p.status, kWhereKv8Store)) {
            float* out = weight + (int64_t)w.bg * c.n_blocks + blk;
            *out = fmaf(decay, *out, y);
          }
        }
      }
      __syncwarp();
    };
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
      const WeighItem w = weigh_item(c, p, item, q_tile, n_all, rank, ranks, lens);
      const uint8_t* src = c.k + (int64_t)w.b * c.bstride * c.ld + (int64_t)(w.bg % c.n_kv) * HD + u * 16;
      const int rows = w.two ? 2 * kTile : kTile;
      uint4 x[kAhead];
      auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int row = r0 + kStep * i;
          x[i] = make_uint4(0, 0, 0, 0);
          if (w.k0 + row < w.k_end) x[i] = load_global(reinterpret_cast<const uint4*>(src + (int64_t)(w.k0 + row) * c.ld));
        }
      };
      if (w.n_i > 0) load(row0);  // on their way while the buffer empties
      if (ranks == 1 && live - added == 2) {  // its keys' buffer is free about when its sums are there
        add_up(last[0], added++);
        last[0] = last[1];
      }
      if (w.n_i > 0 && ok) {
        const uint32_t dst = sK + (done & 1) * 2 * C::kTileBytes;
        ok = warp_wait(bar_k_empty + 8 * (done & 1), ((done >> 1) & 1) ^ 1, p.status, kWhereKv8Widen);
        for (int r0 = row0; r0 < rows && ok; r0 += kStep * kAhead) {
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const int row = r0 + kStep * i;
            if (row >= rows) break;
            const uint32_t* z = reinterpret_cast<const uint32_t*>(&x[i]);
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t lo = cvt_lo(z[e]), hi = cvt_hi(z[e]);
              const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&lo));
              const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              y[2 * e] = pack_bf16x2(f0.x, f0.y);
              y[2 * e + 1] = pack_bf16x2(f1.x, f1.y);
            }
            st_shared16(dst + sw_offset<C::kBoxK>(row, 2 * u), y[0], y[1], y[2], y[3]);
            st_shared16(dst + sw_offset<C::kBoxK>(row, 2 * u + 1), y[4], y[5], y[6], y[7]);
          }
          if (r0 + kStep * kAhead < rows) load(r0 + kStep * kAhead);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar_k_full + 8 * (done & 1));
        ++done;
      }
      if (w.k_end == w.k0) {
        if (ranks > 1) cluster_sync();
      } else if (ranks > 1) {
        add_up(w, live++);
      } else {
        last[live - added] = w;
        ++live;
      }
    }
    if (ranks == 1)
      for (int i = 0; added < live; ++i) add_up(last[i], added++);
  }
  } else {
    setmaxnreg_inc<kWeighRegsRows>();
    const int wg = (warp - 8) >> 2, t = wg & 1, phase = wg >> 1;
    const int lane_base = (warp & 3) * 32, row = lane_base + lane;
    const int block_shift = 31 - __clz(c.block);
    const int32_t qr = row / p.group, hr = row % p.group;  // query and head of this row in a tile
    const uint32_t addr = tmem_base + ((uint32_t)lane_base << 16) + 128u * wg;
    int n = 0, done = 0;  // query tiles, items
    bool ok = true;
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
      const WeighItem w = weigh_item(c, p, item, q_tile, n_all, rank, ranks, lens);
      if (w.k_end == w.k0) {
        if (ranks > 1) cluster_sync();
        continue;
      }
      const int32_t kbase = w.k0 + t * kTile;
      float acc[8], f[8];
      const float* ks = c.k_scale + (int64_t)w.bg * c.n_blocks;
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        acc[g] = 0.f;
        const int32_t key = kbase + 16 * g;
        f[g] = key < w.k_end ? p.scale_log2 * load_global(ks + (key >> block_shift)) : 0.f;
      }
      const float* lse_row = p.lse + ((int64_t)w.b * p.n_heads + (w.bg % c.n_kv) * p.group + hr) * p.n_q;
      {
        // rows that are not there weigh 2^-inf; a tile's lse is loaded one tile ahead
        auto load_lse = [&](int i) {
          const int64_t qi = (int64_t)(w.i0 + i) * q_tile + qr;
          return row < tile_rows && qi < p.n_q ? load_global(lse_row + qi) : INFINITY;
        };
        const int first = (phase ^ n) & 1;
        float ls_next = first < w.n_i ? load_lse(first) : 0.f;
#pragma unroll 1
        for (int i = first; i < w.n_i && ok; i += 2) {
          const float ls = ls_next * kLog2e;
          if (i + 2 < w.n_i) ls_next = load_lse(i + 2);
          int32_t lim = w.k_end;
          if (p.causal) {
            const int64_t x = (int64_t)w.len - p.n_q + (int64_t)(w.i0 + i) * q_tile + qr + 1;
            lim = x < 0 ? 0 : (x < w.k_end ? (int32_t)x : w.k_end);
          }
          if (ls == -INFINITY) lim = 0;  // a row that saw nothing is hidden from every key
          const bool masked = kbase + kTile > lim;
          // (not so for a tile of keys behind the end, nor for a warp whose rows are not there)
          const bool any = __any_sync(0xffffffffu, lim > kbase && row < tile_rows && (int64_t)(w.i0 + i) * q_tile + qr < p.n_q);
          ok = warp_wait(bar_s_full + 8 * phase, ((n + i) >> 1) & 1, p.status, kWhereKv8Softmax);
          if (!ok) break;
          tc_fence_after();
          if (!any) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_s_empty + 8 * phase);
            continue;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            // (four warps a sub-partition cover the loads; a second buffer of 32 measured no faster)
            uint32_t x[32];
            tmem_ld32(addr + 32 * q, x);
            tmem_ld_wait();
            if (q == 3) {  // S is in registers: the next product may overwrite it
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar_s_empty + 8 * phase);
            }
            if (masked) {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float pe = ex2_approx(fmaf(__uint_as_float(x[e]), f[2 * q + (e >> 4)], -ls));
                acc[2 * q + (e >> 4)] += kbase + 32 * q + e < lim ? pe : 0.f;
              }
            } else {
              const uint64_t ls2 = pack_f32x2(-ls, -ls);
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const uint64_t f2 = pack_f32x2(f[2 * q + g], f[2 * q + g]);
                float a0 = 0.f, a1 = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const uint64_t v = fma_f32x2(
                      pack_f32x2(__uint_as_float(x[16 * g + 2 * e]), __uint_as_float(x[16 * g + 2 * e + 1])), f2, ls2);
                  float p0, p1;
                  if (e % 4 == 1 && e / 4 < kPolyPairs) {
                    exp2_fma(v, p0, p1);
                  } else {
                    unpack_f32x2(v, p0, p1);
                    p0 = ex2_approx(p0);
                    p1 = ex2_approx(p1);
                  }
                  a0 += p0;
                  a1 += p1;
                }
                acc[2 * q + g] += a0 + a1;
              }
            }
          }
        }
      }
      n += w.n_i;
      ok = ok && warp_wait(bar_sum_empty + 8 * (done & 1), ((done >> 1) & 1) ^ 1, p.status, kWhereKv8Softmax);
#pragma unroll
      for (int g = 0; g < 8; ++g) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) acc[g] += __shfl_xor_sync(0xffffffffu, acc[g], off);
        if (lane == g) sums[(done & 1) * 128 + (wg * 4 + (warp & 3)) * 8 + g] = acc[g];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_sum_full + 8 * (done & 1));
      ++done;
      if (ranks > 1) cluster_sync();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, 512);
  if (ranks > 1) cluster_sync();  // nothing is written to a CTA that has left
}

// ------------------------------------------------------------------ host

TilePlan make_plan(const Cache& c, const Query& p, int32_t max_len) {
  TilePlan t{};
  t.pairs = (int32_t)((p.n_rows + 2 * kTile - 1) / (2 * kTile));
  const int64_t heads = (int64_t)c.batch * c.n_kv, items = heads * t.pairs, sms = num_sms();
  const int64_t n_kt = ((int64_t)max_len + kTile - 1) / kTile;
  t.splits = 1;
  t.n_full = (int32_t)items;
  // Items of a last wave that does not fill the SMs are split over the keys into
  // m full waves of CTAs, so that m (the longest range + a start and an end, about
  // four key tiles) and the join, about one for every 48 CTAs, take the least.
  const int64_t tail = items % sms;
  double best = (double)(n_kt + 4);
  for (int64_t m = 1; tail > 0 && m <= 6; ++m) {
    int64_t k = m * sms / tail, hi = m * sms - k * tail;  // hi items take one range more
    if (k > kMaxSplits - 1) k = kMaxSplits - 1;
    if (2 * k > n_kt) k = n_kt / 2;  // two key tiles a range at least
    if (k != m * sms / tail || 2 * (k + 1) > n_kt) hi = 0;
    if (k < 1 || (k == 1 && hi < tail)) continue;
    const double first = (double)((n_kt + k - 1) / k), rest = (double)((n_kt + (hi > 0 ? k : k - 1)) / (hi > 0 ? k + 1 : k));
    const double cost = first + (double)(m - 1) * rest + 4.0 * (double)m + (double)(tail * k + hi) / 48 + 2;
    if (cost < best) {
      best = cost;
      t.splits = (int32_t)k;
      t.n_lo = (int32_t)(tail - hi);
      t.n_hi = (int32_t)hi;
      t.n_full = (int32_t)(items - tail);
    }
  }
  return t;
}

size_t plan_o_bytes(const TilePlan& t, int hd) {
  return ((size_t)t.n_parts() * 2 * kTile * hd * 4 + 255) & ~size_t(255);
}

// Sets a kernel's shared-memory limit once per device; `regs` is the sum that
// its register hand-over needs of the launch.
template <typename K>
cosmot_status prepare(K kern, int smem, int64_t regs, int threads, uint64_t& done) {
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return COSMOT_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  if (dev < 64 && (done & (1ull << dev))) return COSMOT_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return COSMOT_ERR_CUDA;
  // a build whose register count cannot fund the hand-over is not launched
  cudaFuncAttributes fa{};
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess || regs > (int64_t)threads * fa.numRegs) return COSMOT_ERR_CUDA;
  if (dev < 64) done |= 1ull << dev;
  return COSMOT_OK;
}

template <int HD, int NG>
cosmot_status launch_tiles(const Cache& c, const Query& p, const TilePlan& t, cudaStream_t s) {
  static uint64_t done = 0;
  const cosmot_status st = prepare(tile_attention_kernel<HD, NG>, AttnCfg<HD>::kSmem, 256 * (kRegsIo + kRegsSoftmax),
                                   kAttnThreads, done);
  if (st != COSMOT_OK) return st;
  const int64_t grid = (int64_t)t.n_full + t.n_parts();
  return launch_status(launch_pdl(tile_attention_kernel<HD, NG>, dim3((unsigned)grid), dim3(kAttnThreads),
                                  AttnCfg<HD>::kSmem, s, nullptr, c, p, t));
}

template <int HD>
cosmot_status launch_attention(const Cache& c, const Query& p, const TilePlan& t, cudaStream_t s) {
  const cosmot_status st = c.block == 128  ? launch_tiles<HD, 1>(c, p, t, s)
                           : c.block == 64 ? launch_tiles<HD, 2>(c, p, t, s)
                           : c.block == 32 ? launch_tiles<HD, 4>(c, p, t, s)
                                           : launch_tiles<HD, 8>(c, p, t, s);
  if (st != COSMOT_OK || t.n_parts() == 0) return st;
  return launch_status(launch_pdl(tile_join_kernel<HD>, dim3((unsigned)(t.n_lo + t.n_hi) * (unsigned)(2 * kTile * (HD / 4) / kTileJoinThreads)),
                                  dim3(kTileJoinThreads), 0, s, nullptr, c,
                                  p, t));
}

template <int HD>
cosmot_status launch_weigh(const Cache& c, const Query& p, float decay, float* weight, int32_t max_len, cudaStream_t s) {
  static uint64_t done = 0;
  cosmot_status st = prepare(tile_weigh_kernel<HD>, WeighCfg<HD>::kSmem, 256 * kWeighRegsIo + 512 * kWeighRegsRows,
                             kWeighThreads, done);
  if (st != COSMOT_OK) return st;
  const int32_t q_tile = kTile / p.group;
  CUtensorMap map;
  st = make_tmap_bf16_4d(&map, p.q, (uint64_t)HD, (uint64_t)p.n_heads, (uint64_t)p.n_q, (uint64_t)c.batch, (uint64_t)p.ld_q,
                         (uint64_t)(c.batch > 1 ? p.q_bstride : p.n_q), 64, (uint32_t)p.group, (uint32_t)q_tile);
  if (st != COSMOT_OK) return st;
  const int64_t heads = (int64_t)c.batch * c.n_kv, n_all = (p.n_q + q_tile - 1) / q_tile;
  const int32_t ranges = (c.capacity + 2 * kTile - 1) / (2 * kTile);
  const int64_t live = heads * (((int64_t)max_len + 2 * kTile - 1) / (2 * kTile)), items = heads * ranges, sms = num_sms();
  if (items > INT32_MAX / 2) return COSMOT_ERR_UNSUPPORTED;
  // a key range's queries are shared by a cluster where there are fewer key ranges than SMs
  int ranks = 1;
  while (ranks < kWeighMaxCluster && live * ranks * 2 <= sms && n_all >= 4 * ranks) ranks *= 2;
  cudaLaunchAttribute cl{};
  cl.id = cudaLaunchAttributeClusterDimension;
  cl.val.clusterDim.x = 1;
  cl.val.clusterDim.y = (unsigned)ranks;
  cl.val.clusterDim.z = 1;
  const dim3 grid((unsigned)(items < sms / ranks ? items : sms / ranks), (unsigned)ranks);
  return launch_status(launch_pdl(tile_weigh_kernel<HD>, grid, dim3(kWeighThreads), WeighCfg<HD>::kSmem, s, &cl, map, c, p,
                                  decay, weight, q_tile, (int32_t)n_all, ranges));
}

}  // namespace

bool tile_fits(const Cache& c, const Query& p) {
  return (int64_t)c.batch * c.n_kv * ((p.n_rows + 2 * kTile - 1) / (2 * kTile)) <= INT32_MAX / 64;
}

size_t tile_workspace(const Cache& c, const Query& p, int32_t max_len) {
  const TilePlan t = make_plan(c, p, max_len);
  return t.n_parts() == 0 ? 0 : plan_o_bytes(t, c.hd) + (size_t)t.n_parts() * 2 * kTile * sizeof(float2);
}

cosmot_status tile_attention(const Cache& c, const Query& p0, int32_t max_len, void* workspace, cudaStream_t s) {
  Query p = p0;
  const TilePlan t = make_plan(c, p, max_len);
  if (t.n_parts()) {
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + plan_o_bytes(t, c.hd));
    p.part_rows = (int64_t)t.n_parts() * 2 * kTile;
  }
  return c.hd == 128 ? launch_attention<128>(c, p, t, s) : launch_attention<64>(c, p, t, s);
}

cosmot_status tile_weigh(const Cache& c, const Query& p, float decay, float* weight, int32_t max_len, cudaStream_t s) {
  return c.hd == 128 ? launch_weigh<128>(c, p, decay, weight, max_len, s)
                     : launch_weigh<64>(c, p, decay, weight, max_len, s);
}

}  // namespace kv8
}  // namespace cosmot

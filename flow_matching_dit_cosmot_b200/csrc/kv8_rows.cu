// Attention and weighing over the 8-bit cache for few query rows (single
// tokens), bound by the cache's bytes.
//
// A warp takes 16 keys at a time.  Keys are the M dimension of mma.m16n8k16 and
// eight packed query rows its N dimension, so that a row tile costs no more
// products than it has to:
//   S^T = K Q^T    lane (g, j) (g = lane / 4, j = lane % 4) holds bytes 16j ..
//                  16j+15 of each 64-dim half of keys g and g + 8; chunk c of 4
//                  bytes is k-step c, slots (2j, 2j+1, 2j+8, 2j+9) = dims
//                  16j + 4c + (0, 1, 2, 3); Q is laid out the same way once.
//   O^T += V^T P^T P^T (f16) is S^T's accumulator, transposed in registers
//                  (movmatrix); lane (g, j) holds piece g (hd/8 bytes) of the
//                  rows of its four keys 2j, 2j+1, 8 + 2j, 8 + 2j + 1; row tile
//                  i is bytes 2i and 2i + 1 of every piece.
// The contracted dimension's order and the output rows' order are free, so
// every lane needs just the bytes that it loads itself: they go through a ring
// of cp.async stages in shared memory that no other lane reads, with no
// barrier, and leave the registers to the products.
// Q (bf16) becomes f16 by a power of two per row that puts its largest
// magnitude in [2^13, 2^14): exact down to 2^-31 of it.
// P (f16) is 2^11 times the weight relative to the running maximum of the
// scores, which follows only when it grows by more than 2^4, times the block's
// value scale in units of 2^v_exp, at most 1 and more than 2^-3: below 2^15, full
// precision for weights down to 2^-22 of the largest, and a step of 2^-32 of it
// below.  O^T is in those units too.  A block whose scale lies outside the window
// moves it: the accumulators change by a power of two, which float32 holds
// exactly, so that scales far apart cost the weights no digits.  (It costs 0.5 %
// for one token and 4 % at 32 rows x 32 heads; with every scale in the exponent,
// whatever their spread, small ones lose their digits.  A unit that follows every
// block's scale took 10 % more where neighbours differ by one; to bring every 16
// keys' share in by its own scale 2 % and 12 %; to follow the maximum at 2^7 saves
// 1.5 % and costs three digits.)
#include "kv8.cuh"

#include <mutex>

namespace cosmot {
namespace kv8 {
namespace {

constexpr int kWarps = 4;
constexpr int kRing = 3;  // stages of 16 keys
constexpr int ctas_per_sm(int nt) { return nt == 1 ? 4 : 3; }  // shared memory and registers allow
constexpr float kPBias = 11.f, kFollow = 4.f, kVWindow = 2.f;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8x8 matrix of 16-bit elements held two a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool live) {
  const int n = live ? BYTES : 0;  // nothing is read for n = 0: the destination becomes zeros
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_shared8(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// One row's 16-dim pieces for this lane (its j), scaled into f16; returns the
// factor that takes the scaled scores back (NaN for a row that is not finite).
template <int HD>
__device__ __forceinline__ float load_q_row(const __nv_bfloat16* row, bool valid, int j, uint32_t (&f)[HD / 16][2]) {
  uint32_t w[HD / 64][8];
  float amax = 0.f;
  bool finite = true;
#pragma unroll
  for (int h = 0; h < HD / 64; ++h) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[h][i] = 0;
    if (valid) {
      const uint4* p = reinterpret_cast<const uint4*>(row + 64 * h + 16 * j);
      *reinterpret_cast<uint4*>(&w[h][0]) = load_global(p);
      *reinterpret_cast<uint4*>(&w[h][4]) = load_global(p + 1);
    }
  }
#pragma unroll
  for (int h = 0; h < HD / 64; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = unpack_bf16x2(w[h][i]);
      amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
      finite = finite && fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY;
    }
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    finite = __shfl_xor_sync(0xffffffffu, (int)finite, off) && finite;
  }
  int e = (int)((__float_as_uint(amax) >> 23) & 255u) - 127 - 13;
  e = e < -100 ? -100 : (e > 114 ? 114 : e);
  if (amax == 0.f) e = 0;
  const float down = exp2_int(-e);
#pragma unroll
  for (int h = 0; h < HD / 64; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = unpack_bf16x2(w[h][i]);
      f[4 * h + (i >> 1)][i & 1] = pack_f16x2(v.x * down, v.y * down);
    }
  return finite ? exp2_int(e) : __int_as_float(0x7fc00000);
}

// NT tiles of eight packed rows from r0: B fragments (this lane's row g), and
// the score factors of the rows of its accumulator columns 2j and 2j + 1.
template <int HD, int NT>
__device__ __forceinline__ void load_q_tile(const Cache& c, const Query& p, int32_t b, int32_t kvh, int64_t r0, int g,
                                            int j, uint32_t (&q)[NT][HD / 16][2], float (&fac)[NT][2]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int64_t r = r0 + 8 * n + g;
    const bool valid = r < p.n_rows;
    const int64_t qi = valid ? row_query(p, r) : 0;
    const int32_t h = kvh * p.group + (valid ? row_head(p, r) : 0);
    const float f = p.scale_log2 * load_q_row<HD>(p.q + (b * p.q_bstride + qi) * p.ld_q + (int64_t)h * HD, valid, j, q[n]);
    fac[n][0] = __shfl_sync(0xffffffffu, f, 8 * j);
    fac[n][1] = __shfl_sync(0xffffffffu, f, 8 * j + 4);
  }
}

// S^T of 16 keys: ka, kb the 16-byte pieces of keys g and g + 8.
template <int HD, int NT>
__device__ __forceinline__ void scores(float (&s)[NT][4], const uint4 (&ka)[HD / 64], const uint4 (&kb)[HD / 64],
                                       const uint32_t (&q)[NT][HD / 16][2]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
  for (int h = 0; h < HD / 64; ++h) {
    const uint32_t* a = reinterpret_cast<const uint32_t*>(&ka[h]);
    const uint32_t* d = reinterpret_cast<const uint32_t*>(&kb[h]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a0 = cvt_lo(a[k]), a1 = cvt_lo(d[k]), a2 = cvt_hi(a[k]), a3 = cvt_hi(d[k]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(s[n], a0, a1, a2, a3, q[n][4 * h + k][0], q[n][4 * h + k][1]);
    }
  }
}

// ------------------------------------------------------------------ attention
template <int HD>
struct Ring {
  static constexpr int kPieceK = 512;               // 16 bytes a lane
  static constexpr int kPieceV = HD == 128 ? 512 : 256;
  static constexpr int kOffV = 2 * (HD / 64) * kPieceK;
  static constexpr int kStage = kOffV + 4 * kPieceV;
  static constexpr int kScales = 256;               // blocks whose scales are kept in shared memory
  static constexpr int kRowPitch = HD + 4;           // floats between rows of the warps' parts
  static constexpr int smem(int nt) {
    const int ring = kWarps * kRing * kStage, parts = kWarps * 8 * nt * (kRowPitch * 4 + 8);
    return kScales * 16 + (ring > parts ? ring : parts);
  }
};

// One CTA per (key range, 8 NT packed rows, sequence and key head); its warps
// take 16 keys in turn.
// bound: HBM.  One token behind 130,999 rows (8 key heads of 128): 57.5 us with
// the join, the ranges alone 51 us = 5.2 TB/s; without the arithmetic the same
// loads take 46.  Three stages at four CTAs an SM, four at three and six at two
// are within 2 % of one another.
template <int HD, int NT>
__global__ void __launch_bounds__(32 * kWarps, ctas_per_sm(NT)) rows_attention_kernel(const __grid_constant__ Cache c,
                                                                                 const __grid_constant__ Query p) {
  pdl_trigger();
  pdl_wait();
  using R = Ring<HD>;
  extern __shared__ __align__(16) uint8_t sm_raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, j = lane & 3;
  const int32_t split = blockIdx.x;
  const int32_t b = blockIdx.z / c.n_kv, kvh = blockIdx.z % c.n_kv;
  const int64_t r0 = (int64_t)blockIdx.y * 8 * NT;
  const int32_t len = shown_rows(c, b, p.n_new, p.status, threadIdx.x == 0);
  const int64_t r_end = r0 + 8 * NT < p.n_rows ? r0 + 8 * NT : p.n_rows;
  const int32_t shown = row_limit(p, r_end - 1, len);  // the tile's last row sees the most
  // this CTA's keys; the last range takes what is left of a sequence longer than the host said
  const int32_t k0 = (int32_t)min((int64_t)shown, (int64_t)split * p.chunk);
  const int32_t kend = split == p.splits - 1 ? shown : (int32_t)min((int64_t)shown, (int64_t)(split + 1) * p.chunk);
  if (p.splits > 1 && k0 >= kend) {  // nothing here: the join leaves this range out
    const int64_t pr = ((int64_t)split * c.batch * c.n_kv + blockIdx.z) * p.n_rows + r0 + threadIdx.x;
    if (r0 + threadIdx.x < r_end && threadIdx.x < 8 * NT && dcheck(pr < p.part_rows, p.status, kWhereKv8Store))
      p.part_ml[pr] = make_float2(-INFINITY, 0.f);
    return;
  }

  const uint8_t* kb = c.k + (int64_t)b * c.bstride * c.ld + (int64_t)kvh * HD;
  const uint8_t* vb = c.v + (int64_t)b * c.bstride * c.ld + (int64_t)kvh * HD;
  const float* ksp = c.k_scale + (int64_t)blockIdx.z * c.n_blocks;
  const float* vsp = c.v_scale + (int64_t)blockIdx.z * c.n_blocks;
  const int block_shift = 31 - __clz(c.block);
  float4* scales = reinterpret_cast<float4*>(sm_raw);  // (ks, log2 vs, 1/vs, log2 vs rounded up)
  const uint32_t ring = smem_u32(sm_raw) + R::kScales * 16 + warp * kRing * R::kStage;
  // V pieces: a row's eight pieces side by side, turned by the row so that the
  // lanes' reads fall on all banks too
  const uint32_t v_at = R::kOffV + (uint32_t)(j * 8 + (g ^ (2 * j))) * (HD / 8);

  auto fetch = [&](int32_t key0, int slot) {
    if (key0 < kend) {
      const uint32_t st = ring + slot * R::kStage + lane * 16;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int32_t key = key0 + 8 * t + g;
        const bool live = key < kend;
        const uint8_t* src = kb + (int64_t)(live ? key : key0) * c.ld + 16 * j;
#pragma unroll
        for (int h = 0; h < HD / 64; ++h) cp_async<16>(st + (t * (HD / 64) + h) * R::kPieceK, src + 64 * h, live);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int32_t key = key0 + 8 * (s >> 1) + 2 * j + (s & 1);
        const bool live = key < kend;
        cp_async<HD / 8>(ring + slot * R::kStage + v_at + s * R::kPieceV, vb + (int64_t)(live ? key : key0) * c.ld + g * (HD / 8),
                         live);
      }
    }
    cp_async_commit();  // a group per stage, whether it holds anything or not
  };
  constexpr int kStep = 16 * kWarps;
  const int32_t first = k0 + 16 * warp;
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch(first + i * kStep, i);
  auto scale_of = [&](int32_t blk) {
    float4 s;
    s.x = load_global(ksp + blk);
    scale_log2_parts(load_global(vsp + blk), s.y, s.z);
    s.w = ceilf(s.y);
    return s;
  };
  const int32_t blk0 = k0 >> block_shift, blk1 = ((kend - 1) >> block_shift) + 1;
  for (int32_t i = blk0 + (int32_t)threadIdx.x; i < min(blk1, blk0 + R::kScales); i += 32 * kWarps) scales[i - blk0] = scale_of(i);

  uint32_t q[NT][HD / 16][2];
  float fac[NT][2];
  load_q_tile<HD, NT>(c, p, b, kvh, r0, g, j, q, fac);
  // columns 2j, 2j + 1 of each row tile; rows that are not there see every key (they force no mask)
  int32_t lim[NT][2], lim_min = kend;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t r = r0 + 8 * n + 2 * j + i;
      lim[n][i] = r < p.n_rows ? row_limit(p, r, len) : kend;
      lim_min = min(lim_min, lim[n][i]);
    }
  lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 1));
  lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 2));

  constexpr int kTiles = HD / 16;  // row tiles of O^T
  constexpr int VW = HD / 32;      // 32-bit words of a V piece
  float o[NT][kTiles][4];
  float m[NT][2], l[NT][2], v_exp = 0.f;  // o is in units of 2^v_exp
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
  }

  __syncthreads();  // the scales
  int slot = 0;
#pragma unroll 1
  for (int32_t key0 = first; key0 < kend; key0 += kStep) {
    fetch(key0 + (kRing - 1) * kStep, slot == 0 ? kRing - 1 : slot - 1);
    cp_async_wait<kRing - 1>();  // this stage's group has landed; a lane reads its own bytes alone
    const uint32_t st = ring + slot * R::kStage;
    slot = slot == kRing - 1 ? 0 : slot + 1;
    uint4 ka[HD / 64], kc[HD / 64];
#pragma unroll
    for (int h = 0; h < HD / 64; ++h) {
      ka[h] = ld_shared16(st + h * R::kPieceK + lane * 16);
      kc[h] = ld_shared16(st + (HD / 64 + h) * R::kPieceK + lane * 16);
    }
    const int32_t blk = key0 >> block_shift;
    const float4 sc = blk - blk0 < R::kScales ? scales[blk - blk0] : scale_of(blk);
    const float ks = sc.x;
    // (the warp's 16 keys have one value scale)
    const bool moved = sc.w > v_exp || sc.w < v_exp - kVWindow;
    const float v_by = moved ? v_exp - sc.w : 0.f;
    v_exp = moved ? sc.w : v_exp;
    // the scale's log2 in units of 2^v_exp, in (-kVWindow - 1, 0], and 2^-it
    const float p_bias = kPBias + (sc.y - v_exp), v_inv = sc.z * exp2_whole(v_exp);

    float s[NT][4];
    scores<HD, NT>(s, ka, kc, q);
    uint32_t pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // s[n][0], [1]: key g, columns 2j, 2j + 1; [2], [3]: key g + 8
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f = fac[n][i] * ks;
        s[n][i] *= f;
        s[n][2 + i] *= f;
      }
      if (key0 + 16 > lim_min) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (key0 + g >= lim[n][i]) s[n][i] = -INFINITY;
          if (key0 + 8 + g >= lim[n][i]) s[n][2 + i] = -INFINITY;
        }
      }
      const float t0 = fmaxf(s[n][0], s[n][2]), t1 = fmaxf(s[n][1], s[n][3]);
      // (-inf > -inf + 4 is false: a row that has seen nothing stays where it is)
      if (__any_sync(0xffffffffu, moved || t0 > m[n][0] + kFollow || t1 > m[n][1] + kFollow)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float t = i ? t1 : t0;
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
          const float to = t > m[n][i] + kFollow ? t : m[n][i];  // a row of its own: whatever the others do
          const float corr = to == m[n][i] ? 1.f : ex2_approx(m[n][i] - to);  // 0 from -inf
          m[n][i] = to;
          l[n][i] *= corr;
          const float o_by = corr * exp2_whole(fminf(fmaxf(v_by, -126.f), 126.f));
#pragma unroll
          for (int d = 0; d < kTiles; ++d) {
            o[n][d][i] *= o_by;
            o[n][d][2 + i] *= o_by;
          }
        }
      }
      float pr[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mu = m[n][i] == -INFINITY ? 0.f : m[n][i] - p_bias;
        pr[i] = ex2_approx(s[n][i] - mu);
        pr[2 + i] = ex2_approx(s[n][2 + i] - mu);
        l[n][i] = fmaf(pr[i] + pr[2 + i], v_inv, l[n][i]);
      }
      pb[n][0] = transpose8x8(pack_f16x2(pr[0], pr[1]));
      pb[n][1] = transpose8x8(pack_f16x2(pr[2], pr[3]));
    }
    uint32_t vw[4][VW];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t at = st + v_at + k * R::kPieceV;
      if constexpr (HD == 128) {
        *reinterpret_cast<uint4*>(vw[k]) = ld_shared16(at);
      } else {
        *reinterpret_cast<uint2*>(vw[k]) = ld_shared8(at);
      }
    }
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      // bytes 4w .. 4w+3 of the pieces of keys (2j, 2j+1) and (8 + 2j, 8 + 2j + 1)
      const uint32_t lo0 = __byte_perm(vw[0][w], vw[1][w], 0x5140), hi0 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
      const uint32_t lo1 = __byte_perm(vw[2][w], vw[3][w], 0x5140), hi1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
      const uint32_t a0 = cvt_lo(lo0), a1 = cvt_hi(lo0), a2 = cvt_lo(lo1), a3 = cvt_hi(lo1);
      const uint32_t b0 = cvt_lo(hi0), b1 = cvt_hi(hi0), b2 = cvt_lo(hi1), b3 = cvt_hi(hi1);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_f16(o[n][2 * w], a0, a1, a2, a3, pb[n][0], pb[n][1]);
        mma_f16(o[n][2 * w + 1], b0, b1, b2, b3, pb[n][0], pb[n][1]);
      }
    }
  }
  const float v_unit = exp2_whole(v_exp);
  cp_async_wait<0>();
  __syncthreads();  // the ring's memory takes the warps' parts now

  // lane (g, j): rows 2j, 2j + 1 of each tile, dims hd/8 g + (2i, 2i + 1)
  float* sm_o = reinterpret_cast<float*>(sm_raw + R::kScales * 16);
  float2* sm_ml = reinterpret_cast<float2*>(sm_o + kWarps * 8 * NT * R::kRowPitch);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float lr = l[n][i];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) lr += __shfl_xor_sync(0xffffffffu, lr, off);
      const int row = warp * 8 * NT + 8 * n + 2 * j + i;
      if (g == 0) sm_ml[row] = make_float2(m[n][i], lr);
#pragma unroll
      for (int d = 0; d < kTiles; ++d)
        *reinterpret_cast<float2*>(sm_o + row * R::kRowPitch + g * (HD / 8) + 2 * d) = make_float2(o[n][d][i] * v_unit, o[n][d][2 + i] * v_unit);
    }
  __syncthreads();
  // a thread joins the warps' parts of 4 columns of a row, in warp order
  for (int u = threadIdx.x; u < 8 * NT * (HD / 4); u += 32 * kWarps) {
    const int row = u / (HD / 4), col = (u % (HD / 4)) * 4;
    const int64_t r = r0 + row;
    if (r >= p.n_rows) break;
    float ref = -INFINITY, lsum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sm_ml[w * 8 * NT + row];
      if (ml.y != 0.f) ref = fmaxf(ref, ml.x);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sm_ml[w * 8 * NT + row];
      const float f = ml.y == 0.f ? 0.f : ex2_approx(ml.x - ref);
      lsum = fmaf(f, ml.y, lsum);
      const float4 x = *reinterpret_cast<const float4*>(sm_o + (w * 8 * NT + row) * R::kRowPitch + col);
      acc[0] = fmaf(f, x.x, acc[0]);
      acc[1] = fmaf(f, x.y, acc[1]);
      acc[2] = fmaf(f, x.z, acc[2]);
      acc[3] = fmaf(f, x.w, acc[3]);
    }
    ref -= kPBias;
    if (p.splits > 1) {
      const int64_t pr = ((int64_t)split * c.batch * c.n_kv + blockIdx.z) * p.n_rows + r;
      if (!dcheck(pr < p.part_rows, p.status, kWhereKv8Store)) continue;
      *reinterpret_cast<float4*>(p.part_o + pr * HD + col) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (col == 0) p.part_ml[pr] = make_float2(lsum == 0.f ? -INFINITY : ref, lsum);
    } else {
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
      const int64_t qi = row_query(p, r);
      const int32_t h = kvh * p.group + row_head(p, r);
      if (!dcheck(qi < p.n_q && h < p.n_heads, p.status, kWhereKv8Store)) continue;
      *reinterpret_cast<uint2*>(p.o + (b * p.o_bstride + qi) * p.ld_o + (int64_t)h * HD + col) =
          make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
      if (col == 0 && p.lse)
        p.lse[((int64_t)b * p.n_heads + h) * p.n_q + qi] = lsum == 0.f ? -INFINITY : log_sum(ref, lsum, kPBias);
    }
  }
}

constexpr int kJoinThreads = 128;

// One row a CTA: its threads are hd / 4 columns of 4 by groups that take the
// splits in turn; the groups' sums are added in order.  (A split without a key
// for the row may have written nothing: it is not read.)
template <int HD>
__global__ void __launch_bounds__(kJoinThreads) rows_join_kernel(const __grid_constant__ Cache c,
                                                                 const __grid_constant__ Query p) {
  pdl_trigger();
  pdl_wait();
  const int64_t stride = (int64_t)c.batch * c.n_kv * p.n_rows, pr = blockIdx.x, r = pr % p.n_rows, bg = pr / p.n_rows;
  const int32_t b = (int32_t)(bg / c.n_kv), kvh = (int32_t)(bg % c.n_kv);
  const int splits = p.splits;
  constexpr int kCols = HD / 4, kGroups = kJoinThreads / kCols;
  __shared__ float wgt[kMaxSplits];
  __shared__ float red[2][4];
  __shared__ float4 part[kGroups][kCols];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float2 ml[kMaxSplits / kJoinThreads];
  float ref = -INFINITY;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kJoinThreads; ++i) {
    const int s = tid + kJoinThreads * i;
    ml[i] = s < splits ? p.part_ml[s * stride + pr] : make_float2(-INFINITY, 0.f);
    if (ml[i].y != 0.f) ref = fmaxf(ref, ml[i].x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, off));
  if (lane == 0) red[0][warp] = ref;
  __syncthreads();
  ref = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  float lsum = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kJoinThreads; ++i) {
    const float f = ml[i].y == 0.f ? 0.f : ex2_approx(ml[i].x - ref);
    wgt[tid + kJoinThreads * i] = f;
    lsum = fmaf(f, ml[i].y, lsum);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, off);
  if (lane == 0) red[1][warp] = lsum;
  __syncthreads();
  lsum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  const int grp = tid / kCols, col = tid % kCols;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* src = p.part_o + pr * HD + col * 4;
#pragma unroll 8
  for (int s = grp; s < splits; s += kGroups) {
    const float f = wgt[s];
    if (f != 0.f) {
      const float4 x = *reinterpret_cast<const float4*>(src + (int64_t)s * stride * HD);
      acc.x = fmaf(f, x.x, acc.x);
      acc.y = fmaf(f, x.y, acc.y);
      acc.z = fmaf(f, x.z, acc.z);
      acc.w = fmaf(f, x.w, acc.w);
    }
  }
  part[grp][col] = acc;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int i = 1; i < kGroups; ++i) {
    const float4 x = part[i][col];
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
  }
  const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
  const int64_t qi = row_query(p, r);
  const int32_t h = kvh * p.group + row_head(p, r);
  if (!dcheck(qi < p.n_q && h < p.n_heads, p.status, kWhereKv8Store)) return;
  *reinterpret_cast<uint2*>(p.o + (b * p.o_bstride + qi) * p.ld_o + (int64_t)h * HD + col * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (col == 0 && p.lse)
    p.lse[((int64_t)b * p.n_heads + h) * p.n_q + qi] = lsum == 0.f ? -INFINITY : log_sum(ref, lsum, kPBias);
}

// ------------------------------------------------------------------ weighing
// A warp owns whole blocks of rows and sums 2^(s - lse) over their keys and
// eight NT query rows, so that nothing is added by two threads.  The keys come
// through a ring of 16-key stages, as above.  More query rows take more passes
// over the keys (from L2).
// bound: HBM.  One token of 16 sequences (132 MB of keys): 24-28 us.
constexpr int kWeighRing = 5;

template <int HD>
struct WeighRing {
  static constexpr int kStage = 2 * (HD / 64) * 512;
  static constexpr int kSmem = kWarps * kWeighRing * kStage;
};

template <int HD, int NT>
__global__ void __launch_bounds__(32 * kWarps) rows_weigh_kernel(const __grid_constant__ Cache c,
                                                                const __grid_constant__ Query p, float decay,
                                                                float* weight) {
  pdl_trigger();
  pdl_wait();
  using R = WeighRing<HD>;
  extern __shared__ __align__(16) uint8_t sm_raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, j = lane & 3;
  const int32_t b = blockIdx.y / c.n_kv, kvh = blockIdx.y % c.n_kv;
  const int32_t len = shown_rows(c, b, p.n_new, p.status, threadIdx.x == 0);
  // blocks blk0 + warp, + kWarps, ... of this CTA's p.chunk keys (a whole number of blocks)
  const int32_t per = p.chunk / c.block, blk0 = (int32_t)blockIdx.x * per + warp;
  const int32_t blk1 = min((len + c.block - 1) / c.block, ((int32_t)blockIdx.x + 1) * per);
  if (blk0 >= blk1) return;
  const int stages = c.block >> 4, n = ((blk1 - blk0 + kWarps - 1) / kWarps) * stages;  // stages of 16 keys
  const int shift = 31 - __clz(stages);
  const uint8_t* kb = c.k + (int64_t)b * c.bstride * c.ld + (int64_t)kvh * HD + 16 * j;
  const float* ksp = c.k_scale + (int64_t)blockIdx.y * c.n_blocks;
  float* wp = weight + (int64_t)blockIdx.y * c.n_blocks;
  const uint32_t ring = smem_u32(sm_raw) + warp * kWeighRing * R::kStage;

  auto fetch = [&](int t, int slot) {
    if (t < n) {
      const int32_t blk = blk0 + (t >> shift) * kWarps, key0 = blk * c.block + (t & (stages - 1)) * 16;
      const uint32_t st = ring + slot * R::kStage + lane * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t key = key0 + 8 * i + g;
        const bool live = key < len;
        const uint8_t* src = kb + (int64_t)(live ? key : blk * c.block) * c.ld;
#pragma unroll
        for (int h = 0; h < HD / 64; ++h) cp_async<16>(st + (i * (HD / 64) + h) * 512, src + 64 * h, live);
      }
    }
    cp_async_commit();
  };

  for (int64_t r0 = 0; r0 == 0 || r0 < p.n_rows; r0 += 8 * NT) {
#pragma unroll
    for (int i = 0; i < kWeighRing - 1; ++i) fetch(i, i);
    uint32_t q[NT][HD / 16][2];
    float fac[NT][2], lse[NT][2];
    int32_t lim[NT][2], lim_min = len;
    load_q_tile<HD, NT>(c, p, b, kvh, r0, g, j, q, fac);
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t r = r0 + 8 * m + 2 * j + i;
        lim[m][i] = len;
        lse[m][i] = INFINITY;  // rows that are not there: 2^-inf
        if (r < p.n_rows) {
          const int64_t qi = row_query(p, r);
          const int32_t h = kvh * p.group + row_head(p, r);
          lse[m][i] = p.lse[((int64_t)b * p.n_heads + h) * p.n_q + qi] * kLog2e;
          lim[m][i] = lse[m][i] == -INFINITY ? 0 : row_limit(p, r, len);  // a row that saw nothing weighs nothing
        }
        lim_min = min(lim_min, lim[m][i]);
      }
    lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 1));
    lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 2));
    float sum = 0.f, ks = 0.f, before = 0.f;
    // a block's scale and old weight are loaded one block ahead
    float ks_next = load_global(ksp + blk0), before_next = wp[blk0];
    int slot = 0;
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
      if ((t & (stages - 1)) == 0) {
        ks = ks_next;
        before = before_next;
        const int32_t ahead = blk0 + ((t >> shift) + 1) * kWarps;
        if (ahead < blk1) {
          ks_next = load_global(ksp + ahead);
          before_next = wp[ahead];
        }
      }
      fetch(t + kWeighRing - 1, slot == 0 ? kWeighRing - 1 : slot - 1);
      cp_async_wait<kWeighRing - 1>();
      const uint32_t st = ring + slot * R::kStage;
      slot = slot == kWeighRing - 1 ? 0 : slot + 1;
      uint4 ka[HD / 64], kc[HD / 64];
#pragma unroll
      for (int h = 0; h < HD / 64; ++h) {
        ka[h] = ld_shared16(st + h * 512 + lane * 16);
        kc[h] = ld_shared16(st + (HD / 64 + h) * 512 + lane * 16);
      }
      const int32_t blk = blk0 + (t >> shift) * kWarps, key0 = blk * c.block + (t & (stages - 1)) * 16;
      float s[NT][4];
      scores<HD, NT>(s, ka, kc, q);
      const bool masked = key0 + 16 > lim_min;
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // key g + 8 (e / 2), column 2j + e % 2
          const float x = ex2_approx(fmaf(s[m][e], fac[m][e & 1] * ks, -lse[m][e & 1]));
          sum += masked && key0 + 8 * (e >> 1) + g >= lim[m][e & 1] ? 0.f : x;
        }
      if ((t & (stages - 1)) == stages - 1) {  // the block's last keys
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        // (in a later pass lane 0 reads back what it wrote in the one before)
        if (lane == 0 && dcheck(blk < c.n_blocks, p.status, kWhereKv8Store))
          wp[blk] = fmaf(r0 == 0 ? decay : 1.f, before, sum);
        sum = 0.f;
      }
    }
  }
  cp_async_wait<0>();
}

int rows_tiles(const Query& p) { return p.n_rows <= 8 ? 1 : 2; }  // row tiles of a CTA

template <int HD, int NT>
cosmot_status launch_attention(const Cache& c, const Query& p, cudaStream_t s) {
  constexpr int smem = Ring<HD>::smem(NT);
  static std::mutex mu;
  static uint64_t done = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return COSMOT_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (dev >= 64 || !(done & (1ull << dev))) {
      if (cudaFuncSetAttribute(rows_attention_kernel<HD, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return COSMOT_ERR_CUDA;
      if (dev < 64) done |= 1ull << dev;
    }
  }
  const dim3 grid((unsigned)p.splits, (unsigned)((p.n_rows + 8 * NT - 1) / (8 * NT)), (unsigned)(c.batch * c.n_kv));
  return launch_status(launch_pdl(rows_attention_kernel<HD, NT>, grid, dim3(32 * kWarps), smem, s, nullptr, c, p));
}

}  // namespace

void rows_plan(const Cache& c, Query& p, int32_t max_len) {
  const int64_t per = 8 * rows_tiles(p), tiles = (p.n_rows + per - 1) / per * c.batch * c.n_kv;
  p.splits = 1;
  p.chunk = max_len;
  if (tiles <= 0) return;
  // As many key ranges as fill the SMs once (a batch of unequal lengths: four
  // times, so that the long ones are not left alone).  A range has 256 keys at
  // least: 768 keys x 8 key heads take 6.8 us so, 7.7 as one range, but 512 take
  // 6.2 as one and 6.6 as two; and 1,024 where the rows alone fill half the SMs:
  // 768 keys x 512 heads take 17 us as one range, 23 in ranges of 256.
  const int64_t slots = (int64_t)num_sms() * ctas_per_sm(rows_tiles(p)), want = slots * (c.batch > 1 ? 4 : 1) / tiles;
  const int64_t n = want < 1 ? 1 : (want > kMaxSplits ? kMaxSplits : want);
  const int64_t least = 2 * tiles >= slots ? 1024 : (max_len <= 512 ? 512 : 256);
  int64_t chunk = ((max_len + n - 1) / n + 63) & ~int64_t(63);
  if (chunk < least) chunk = least;
  p.chunk = (int32_t)(chunk < INT32_MAX ? chunk : INT32_MAX);
  p.splits = (int32_t)((max_len + chunk - 1) / chunk);
  if (p.splits < 1) p.splits = 1;
}

cosmot_status rows_attention(const Cache& c, const Query& p, cudaStream_t s) {
  const bool one = rows_tiles(p) == 1;
  cosmot_status st;
  if (c.hd == 128)
    st = one ? launch_attention<128, 1>(c, p, s) : launch_attention<128, 2>(c, p, s);
  else
    st = one ? launch_attention<64, 1>(c, p, s) : launch_attention<64, 2>(c, p, s);
  if (st != COSMOT_OK || p.splits == 1) return st;
  const dim3 jgrid((unsigned)((int64_t)c.batch * c.n_kv * p.n_rows));
  return launch_status(c.hd == 128 ? launch_pdl(rows_join_kernel<128>, jgrid, dim3(kJoinThreads), 0, s, nullptr, c, p)
                                   : launch_pdl(rows_join_kernel<64>, jgrid, dim3(kJoinThreads), 0, s, nullptr, c, p));
}

cosmot_status rows_weigh(const Cache& c, const Query& p0, float decay, float* weight, int32_t max_len, cudaStream_t s) {
  Query p = p0;
  // CTAs for eight warps' worth of work an SM and sub-partition, of one block a warp at least
  const int64_t heads = (int64_t)c.batch * c.n_kv, want = (int64_t)num_sms() * 16 / heads;
  const int64_t span = (int64_t)kWarps * c.block;
  int64_t chunk = max_len / (want < 1 ? 1 : want) / span * span;
  if (chunk < span) chunk = span;
  p.chunk = (int32_t)chunk;
  const dim3 grid((unsigned)((c.capacity + chunk - 1) / chunk), (unsigned)heads);
  const bool one = rows_tiles(p) == 1;
  if (c.hd == 128)
    return launch_status(one ? launch_pdl(rows_weigh_kernel<128, 1>, grid, dim3(32 * kWarps), WeighRing<128>::kSmem, s,
                                          nullptr, c, p, decay, weight)
                             : launch_pdl(rows_weigh_kernel<128, 2>, grid, dim3(32 * kWarps), WeighRing<128>::kSmem, s,
                                          nullptr, c, p, decay, weight));
  return launch_status(one ? launch_pdl(rows_weigh_kernel<64, 1>, grid, dim3(32 * kWarps), WeighRing<64>::kSmem, s, nullptr,
                                        c, p, decay, weight)
                           : launch_pdl(rows_weigh_kernel<64, 2>, grid, dim3(32 * kWarps), WeighRing<64>::kSmem, s, nullptr,
                                        c, p, decay, weight));
}

}  // namespace kv8
}  // namespace cosmot

// Attention and weighing over the 8-bit cache for few query rows (single
// tokens), bound by the cache's bytes.
//
// A warp takes 16 keys at a time, straight from global memory into registers:
// the fragment layouts of mma.m16n8k16 leave the order of the contracted
// dimension and of the output columns free, so each lane loads 16 contiguous
// bytes of a row and those bytes are its operands.
//   S = Q K^T    lane (g, j) (g = lane / 4, j = lane % 4) loads dims 16j..16j+15
//                of each 64-dim half of key g of an 8-key tile; chunk c of 4
//                bytes is k-step c, slots (2j, 2j+1, 2j+8, 2j+9) = dims
//                16j + 4c + (0, 1, 2, 3); Q is laid out the same way once.
//   O += P V     the accumulator of S is the A operand of PV; lane (g, j) loads
//                piece g (hd/8 bytes) of the rows of its four keys 2j, 2j+1,
//                8 + 2j, 8 + 2j + 1; column tile i is byte i of every piece.
// Q (bf16) becomes f16 by a power of two per row that puts its largest
// magnitude in [2^13, 2^14): exact down to 2^-31 of it.  P (f16) is kept times
// 2^15: full precision for weights down to 2^-29 of the largest.
#include "kv8.cuh"

namespace cosmot {
namespace kv8 {
namespace {

constexpr int kWarps = 4;
constexpr float kPBias = 15.f;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
      *reinterpret_cast<uint4*>(&w[h][0]) = __ldg(p);
      *reinterpret_cast<uint4*>(&w[h][4]) = __ldg(p + 1);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = unpack_bf16x2(w[h][i]);
      amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
      finite = finite && fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY;
    }
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

template <int HD>
struct KFrag {
  uint4 w[2][HD / 64];  // [8-key tile][64-dim half]
};

template <int HD>
__device__ __forceinline__ void load_k(KFrag<HD>& f, const uint8_t* base, int64_t ld, int32_t key0, int32_t kend, int g,
                                       int j) {
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int h = 0; h < HD / 64; ++h) {
      f.w[t][h] = make_uint4(0, 0, 0, 0);
      if (key0 + 8 * t + g < kend)
        f.w[t][h] = __ldg(reinterpret_cast<const uint4*>(base + (int64_t)(key0 + 8 * t + g) * ld + 64 * h + 16 * j));
    }
}

// S of one 8-key tile for MT tiles of 16 rows.
template <int HD, int MT>
__device__ __forceinline__ void scores(float (&s)[MT][4], const KFrag<HD>& f, int t, const uint32_t (&q)[MT][HD / 16][4]) {
#pragma unroll
  for (int m = 0; m < MT; ++m) s[m][0] = s[m][1] = s[m][2] = s[m][3] = 0.f;
#pragma unroll
  for (int h = 0; h < HD / 64; ++h) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&f.w[t][h]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t b0 = cvt_lo(w[c]), b1 = cvt_hi(w[c]);
#pragma unroll
      for (int m = 0; m < MT; ++m) mma_f16(s[m], q[m][4 * h + c], b0, b1);
    }
  }
}

template <int HD, int MT>
__device__ __forceinline__ void load_q_tile(const Cache& c, const Query& p, int32_t b, int32_t kvh, int64_t r0, int g,
                                            int j, uint32_t (&q)[MT][HD / 16][4], float (&fac)[MT][2]) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t r = r0 + 16 * m + 8 * i + g;
      const bool valid = r < p.n_rows;
      const int64_t qi = valid ? r / p.group : 0;
      const int32_t h = kvh * p.group + (int32_t)(valid ? r % p.group : 0);
      uint32_t f[HD / 16][2];
      fac[m][i] = p.scale_log2 * load_q_row<HD>(p.q + (b * p.q_bstride + qi) * p.ld_q + (int64_t)h * HD, valid, j, f);
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) {
        q[m][k][i] = f[k][0];
        q[m][k][2 + i] = f[k][1];
      }
    }
}

// ------------------------------------------------------------------ attention
template <int HD, int MT>
__global__ void __launch_bounds__(32 * kWarps) rows_attention_kernel(const Cache c, const Query p) {
  pdl_trigger();
  pdl_wait();
  constexpr int NT = HD / 8;  // column tiles of O = bytes of a V piece
  extern __shared__ float sm[];
  float* sm_o = sm;                                  // [kWarps][16 MT][HD]
  float2* sm_ml = reinterpret_cast<float2*>(sm + kWarps * 16 * MT * HD);  // [kWarps][16 MT]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, j = lane & 3;
  const int32_t split = blockIdx.x;
  const int32_t b = blockIdx.z / c.n_kv, kvh = blockIdx.z % c.n_kv;
  const int64_t r0 = (int64_t)blockIdx.y * 16 * MT;
  const int32_t len = shown_rows(c, b, p.n_new, p.status, threadIdx.x == 0);
  const int64_t r_last = (r0 + 16 * MT < p.n_rows ? r0 + 16 * MT : p.n_rows) - 1;
  const int32_t kend = row_limit(p, r_last, len);
  const int32_t n_grp = (kend + 15) >> 4;
  const int32_t g0 = (int32_t)((int64_t)split * n_grp / p.splits);
  const int32_t g1 = (int32_t)((int64_t)(split + 1) * n_grp / p.splits);

  uint32_t q[MT][HD / 16][4];
  float fac[MT][2];
  load_q_tile<HD, MT>(c, p, b, kvh, r0, g, j, q, fac);
  int32_t lim[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) lim[m][i] = row_limit(p, r0 + 16 * m + 8 * i + g, len);

  const uint8_t* kb = c.k + (int64_t)b * c.bstride * c.ld + (int64_t)kvh * HD;
  const uint8_t* vb = c.v + (int64_t)b * c.bstride * c.ld + (int64_t)kvh * HD;
  const float* ksp = c.k_scale + (int64_t)blockIdx.z * c.n_blocks;
  const float* vsp = c.v_scale + (int64_t)blockIdx.z * c.n_blocks;

  float o[MT][NT][4];
  float mx[MT][2], l[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int i = 0; i < NT; ++i) o[m][i][0] = o[m][i][1] = o[m][i][2] = o[m][i][3] = 0.f;
    mx[m][0] = mx[m][1] = -INFINITY;
    l[m][0] = l[m][1] = 0.f;
  }

  constexpr int VW = HD / 32;  // 32-bit words of a V piece
  for (int32_t grp = g0 + warp; grp < g1; grp += kWarps) {
    const int32_t key0 = grp * 16;
    KFrag<HD> kf;
    load_k<HD>(kf, kb, c.ld, key0, kend, g, j);
    uint32_t vw[4][VW];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int32_t key = key0 + 8 * (s >> 1) + 2 * j + (s & 1);
#pragma unroll
      for (int i = 0; i < VW; ++i) vw[s][i] = 0;
      if (key < kend) {
        const uint8_t* src = vb + (int64_t)key * c.ld + g * (HD / 8);
        if constexpr (HD == 128) {
          *reinterpret_cast<uint4*>(vw[s]) = __ldg(reinterpret_cast<const uint4*>(src));
        } else {
          *reinterpret_cast<uint2*>(vw[s]) = __ldg(reinterpret_cast<const uint2*>(src));
        }
      }
    }
    const float ks = __ldg(ksp + key0 / c.block);
    float vlog, vinv;
    scale_log2_parts(__ldg(vsp + key0 / c.block), vlog, vinv);

    float s[2][MT][4];
    scores<HD, MT>(s[0], kf, 0, q);
    scores<HD, MT>(s[1], kf, 1, q);
    uint32_t a[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // row g + 8 i
        const float f = fac[m][i] * ks;
        float x[4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int32_t key = key0 + 8 * t + 2 * j + e;
            x[2 * t + e] = key < lim[m][i] ? fmaf(s[t][m][2 * i + e], f, vlog) : -INFINITY;
          }
        float mt = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
        const float m_new = fmaxf(mx[m][i], mt);
        if (__any_sync(0xffffffffu, m_new > mx[m][i])) {
          const float corr = mx[m][i] == m_new ? 1.f : ex2_approx(mx[m][i] - m_new);  // 0 from -inf
          l[m][i] *= corr;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[m][n][2 * i] *= corr;
            o[m][n][2 * i + 1] *= corr;
          }
          mx[m][i] = m_new;
        }
        const float mu = m_new == -INFINITY ? 0.f : m_new - kPBias;
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[e] = ex2_approx(x[e] - mu);
        l[m][i] = fmaf((pr[0] + pr[1]) + (pr[2] + pr[3]), vinv, l[m][i]);
        a[m][i] = pack_f16x2(pr[0], pr[1]);
        a[m][2 + i] = pack_f16x2(pr[2], pr[3]);
      }
    }
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      // bytes 4w .. 4w+3 of the pieces of keys (0, 1) and (2, 3)
      const uint32_t lo0 = __byte_perm(vw[0][w], vw[1][w], 0x5140), hi0 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
      const uint32_t lo1 = __byte_perm(vw[2][w], vw[3][w], 0x5140), hi1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mma_f16(o[m][4 * w + 0], a[m], cvt_lo(lo0), cvt_lo(lo1));
        mma_f16(o[m][4 * w + 1], a[m], cvt_hi(lo0), cvt_hi(lo1));
        mma_f16(o[m][4 * w + 2], a[m], cvt_lo(hi0), cvt_lo(hi1));
        mma_f16(o[m][4 * w + 3], a[m], cvt_hi(hi0), cvt_hi(hi1));
      }
    }
  }

  // each warp's part to shared memory; accumulator column (tile i, 2j + e) is dim (2j + e) * (HD / 8) + i
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float lr = l[m][i];
      lr += __shfl_xor_sync(0xffffffffu, lr, 1);
      lr += __shfl_xor_sync(0xffffffffu, lr, 2);
      const int row = 16 * m + 8 * i + g;
      if (j == 0) sm_ml[warp * 16 * MT + row] = make_float2(mx[m][i], lr);
      float* dst = sm_o + (warp * 16 * MT + row) * HD;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) dst[(2 * j + e) * (HD / 8) + n] = o[m][n][2 * i + e];
    }
  __syncthreads();
  // a thread joins the warps' parts of 8 columns of a row, in warp order
  for (int u = threadIdx.x; u < 16 * MT * (HD / 8); u += 32 * kWarps) {
    const int row = u / (HD / 8), col = (u % (HD / 8)) * 8;
    const int64_t r = r0 + row;
    if (r >= p.n_rows) continue;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm_ml[w * 16 * MT + row].x);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sm_ml[w * 16 * MT + row];
      const float f = ml.x == -INFINITY && ml.y == 0.f ? 0.f : ex2_approx(ml.x - m);
      lsum = fmaf(f, ml.y, lsum);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(f, sm_o[(w * 16 * MT + row) * HD + col + e], acc[e]);
    }
    if (p.splits > 1) {
      const int64_t pr = ((int64_t)split * c.batch * c.n_kv + blockIdx.z) * p.n_rows + r;
      float4* dst = reinterpret_cast<float4*>(p.part_o + pr * HD + col);
      dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (col == 0) p.part_ml[pr] = make_float2(lsum == 0.f ? -INFINITY : m - kPBias, lsum);
    } else {
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] *= inv;
      const int64_t qi = r / p.group;
      const int32_t h = kvh * p.group + (int32_t)(r % p.group);
      if (!dcheck(qi < p.n_q && h < p.n_heads, p.status, kWhereKv8Store)) continue;
      store_o8(p.o + (b * p.o_bstride + qi) * p.ld_o + (int64_t)h * HD + col, acc);
      if (col == 0 && p.lse)
        p.lse[((int64_t)b * p.n_heads + h) * p.n_q + qi] =
            lsum == 0.f ? -INFINITY : (m - kPBias + log2f(lsum)) * kLn2;
    }
  }
}

// Joins the key splits of every row, in split order; a thread has 8 columns.
template <int HD>
__global__ void __launch_bounds__(256) rows_join_kernel(const Cache c, const Query p) {
  pdl_trigger();
  pdl_wait();
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t rows = (int64_t)c.batch * c.n_kv * p.n_rows;
  if (u >= rows * (HD / 8)) return;
  const int64_t pr = u / (HD / 8);
  const int col = (int)(u % (HD / 8)) * 8;
  float acc[8], lse;
  join_row<HD>(p.part_o, p.part_ml, p.splits, rows, pr, col, acc, lse);
  const int64_t bg = pr / p.n_rows, r = pr % p.n_rows;
  const int32_t b = (int32_t)(bg / c.n_kv), kvh = (int32_t)(bg % c.n_kv);
  const int64_t qi = r / p.group;
  const int32_t h = kvh * p.group + (int32_t)(r % p.group);
  if (!dcheck(qi < p.n_q && h < p.n_heads, p.status, kWhereKv8Store)) return;
  store_o8(p.o + (b * p.o_bstride + qi) * p.ld_o + (int64_t)h * HD + col, acc);
  if (col == 0 && p.lse) p.lse[((int64_t)b * p.n_heads + h) * p.n_q + qi] = lse;
}

// ------------------------------------------------------------------ weighing
// A warp owns a block of rows: it walks the query rows 16 MT at a time and sums
// 2^(s - lse) over them and its keys, so that nothing is added by two threads.
template <int HD, int MT>
__global__ void __launch_bounds__(32 * kWarps) rows_weigh_kernel(const Cache c, const Query p, float decay,
                                                                float* __restrict__ weight) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, j = lane & 3;
  const int32_t b = blockIdx.y / c.n_kv, kvh = blockIdx.y % c.n_kv;
  const int32_t len = shown_rows(c, b, p.n_new, p.status, threadIdx.x == 0);
  const int32_t blk = (int32_t)blockIdx.x * kWarps + warp;
  const int32_t k0 = blk * c.block, k1 = min(len, k0 + c.block);
  if (k0 >= len) return;
  const uint8_t* kb = c.k + (int64_t)b * c.bstride * c.ld + (int64_t)kvh * HD;
  const float ks = __ldg(c.k_scale + (int64_t)blockIdx.y * c.n_blocks + blk);
  float sum = 0.f;
  for (int64_t r0 = 0; r0 < p.n_rows; r0 += 16 * MT) {
    const int64_t r_last = (r0 + 16 * MT < p.n_rows ? r0 + 16 * MT : p.n_rows) - 1;
    if (row_limit(p, r_last, len) <= k0) continue;  // the tile's last row sees the most
    uint32_t q[MT][HD / 16][4];
    float fac[MT][2], lse[MT][2];
    int32_t lim[MT][2];
    load_q_tile<HD, MT>(c, p, b, kvh, r0, g, j, q, fac);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t r = r0 + 16 * m + 8 * i + g;
        lim[m][i] = row_limit(p, r, len);
        lse[m][i] = 0.f;
        if (r < p.n_rows) {
          const int64_t qi = r / p.group;
          const int32_t h = kvh * p.group + (int32_t)(r % p.group);
          lse[m][i] = p.lse[((int64_t)b * p.n_heads + h) * p.n_q + qi];
        }
        if (lse[m][i] == -INFINITY) lim[m][i] = 0;  // a row that saw nothing weighs nothing
        lse[m][i] *= kLog2e;
        fac[m][i] *= ks;
      }
    float part = 0.f;
    for (int32_t key0 = k0; key0 < k1; key0 += 16) {
      KFrag<HD> kf;
      load_k<HD>(kf, kb, c.ld, key0, k1, g, j);
      float s[2][MT][4];
      scores<HD, MT>(s[0], kf, 0, q);
      scores<HD, MT>(s[1], kf, 1, q);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int32_t key = key0 + 8 * t + 2 * j + e;
              if (key < lim[m][i]) part += ex2_approx(fmaf(s[t][m][2 * i + e], fac[m][i], -lse[m][i]));
            }
    }
    sum += part;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0 && dcheck(blk < c.n_blocks, p.status, kWhereKv8Store)) {
    float* w = weight + (int64_t)blockIdx.y * c.n_blocks + blk;
    *w = fmaf(decay, *w, sum);
  }
}

}  // namespace

int32_t rows_splits(const Cache& c, const Query& p, int32_t max_len) {
  const int64_t tiles = (p.n_rows + 15) / 16 * c.batch * c.n_kv;
  if (tiles <= 0) return 1;
  const int64_t want = (2 * (int64_t)num_sms() + tiles - 1) / tiles;
  const int64_t most = ((int64_t)max_len + 255) / 256;
  const int64_t s = want < most ? want : most;
  return (int32_t)(s < 1 ? 1 : (s > 512 ? 512 : s));
}

cosmot_status rows_attention(const Cache& c, const Query& p, cudaStream_t s) {
  constexpr int MT = 1;
  const int64_t tiles = (p.n_rows + 16 * MT - 1) / (16 * MT);
  if (tiles > 65535) return COSMOT_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)p.splits, (unsigned)tiles, (unsigned)(c.batch * c.n_kv));
  const size_t smem = (size_t)kWarps * 16 * MT * (c.hd * 4 + 8);
  cosmot_status st = launch_status(
      c.hd == 128 ? launch_pdl(rows_attention_kernel<128, MT>, grid, dim3(32 * kWarps), smem, s, nullptr, c, p)
                  : launch_pdl(rows_attention_kernel<64, MT>, grid, dim3(32 * kWarps), smem, s, nullptr, c, p));
  if (st != COSMOT_OK || p.splits == 1) return st;
  const int64_t units = (int64_t)c.batch * c.n_kv * p.n_rows * (c.hd / 8);
  const dim3 jgrid((unsigned)((units + 255) / 256));
  return launch_status(c.hd == 128 ? launch_pdl(rows_join_kernel<128>, jgrid, dim3(256), 0, s, nullptr, c, p)
                                   : launch_pdl(rows_join_kernel<64>, jgrid, dim3(256), 0, s, nullptr, c, p));
}

cosmot_status rows_weigh(const Cache& c, const Query& p, float decay, float* weight, cudaStream_t s) {
  const dim3 grid((unsigned)((c.n_blocks + kWarps - 1) / kWarps), (unsigned)(c.batch * c.n_kv));
  return launch_status(
      c.hd == 128 ? launch_pdl(rows_weigh_kernel<128, 1>, grid, dim3(32 * kWarps), 0, s, nullptr, c, p, decay, weight)
                  : launch_pdl(rows_weigh_kernel<64, 1>, grid, dim3(32 * kWarps), 0, s, nullptr, c, p, decay, weight));
}

}  // namespace kv8
}  // namespace cosmot

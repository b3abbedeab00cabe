// The 8-bit key/value cache: storing rows, evicting blocks, and the argument
// checks and dispatch of its attention and weighing.
#include "kv8.cuh"

namespace cosmot {
namespace kv8 {

// ------------------------------------------------------------------ store
// One CTA per (block of rows, sequence x head, K or V), the heads of a block one
// after another, so that CTAs that run together read whole rows.  Each thread
// owns kUnits pieces of 8 elements: 16 bytes read, 8 written, neighbours side by
// side.  The block's largest magnitude is reduced over the CTA, then the
// elements, still in registers, are rounded against the scale, so every input
// byte is read once.  Rows of the block that were there before are read only if
// the scale grows.
// bound: HBM (4 bytes read and 2 written for each K and V element), the issue
// slots next (78 % busy).  18,978 rows x 32 heads of 128: 82 to 89 us = 5.7 to
// 5.3 TB/s.  256 threads at four CTAs an SM; 512 took 99 us where they took 82,
// 128 the same; magnitudes on packed bits saved 12 us.  1,560 rows: 9.8 to 10.8
// us at six CTAs an SM, 11.9 at four.
constexpr int kStoreThreads = 256;

// Largest of the CTA's values: magnitudes of bf16 order like their bits.
__device__ __forceinline__ uint32_t cta_max_bf16(uint32_t mag, uint32_t* part) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mag = __vmaxu2(mag, __shfl_xor_sync(0xffffffffu, mag, off));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = mag;
  __syncthreads();
  for (int i = 0; i < (int)blockDim.x >> 5; ++i) mag = __vmaxu2(mag, part[i]);
  return max(mag & 0xffffu, mag >> 16);
}

template <int kUnits>
__global__ void __launch_bounds__(kStoreThreads, kUnits <= 4 ? 6 : 4)
    store_kernel(const __grid_constant__ Cache c, const __nv_bfloat16* ksrc,
                 const __nv_bfloat16* vsrc, int64_t ld_src, int64_t src_bstride, int32_t n, int* status) {
  pdl_trigger();
  pdl_wait();
  __shared__ uint32_t part[2][kStoreThreads / 32];
  const uint32_t sides = 2u * c.batch * c.n_kv;  // K and V of every head
  const uint32_t side = blockIdx.x % sides;
  const bool is_v = side & 1;
  const int32_t bg = side >> 1, b = bg / c.n_kv, g = bg % c.n_kv;
  const int32_t held = c.lens[b];
  if (held < 0 || held > c.capacity - n) {
    if (threadIdx.x == 0) report_status(status, COSMOT_ERR_BOUNDS, kWhereKv8Lens);
    return;
  }
  const int32_t blk = held / c.block + (int32_t)(blockIdx.x / sides);
  const int32_t row0 = blk * c.block, end = held + n;
  if (row0 >= end) return;
  const int per_row = c.hd >> 3;  // pieces a row
  const int step = (int)blockDim.x / per_row;
  const int32_t first = row0 + (int32_t)threadIdx.x / per_row;
  const int col = ((int)threadIdx.x % per_row) * 8;
  const __nv_bfloat16* src =
      (is_v ? vsrc : ksrc) + ((int64_t)b * src_bstride + (first - held)) * ld_src + (int64_t)g * c.hd + col;
  uint8_t* dst = (is_v ? c.v : c.k) + ((int64_t)b * c.bstride + first) * c.ld + (int64_t)g * c.hd + col;
  float* scale = (is_v ? c.v_scale : c.k_scale) + (int64_t)bg * c.n_blocks + blk;

  uint4 x[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int32_t row = first + u * step;
    x[u] = make_uint4(0, 0, 0, 0);
    if (row >= held && row < end) x[u] = load_global(reinterpret_cast<const uint4*>(src + (int64_t)(u * step) * ld_src));
  }
  const float old = row0 < held ? *scale : 0.f;  // read by every thread before thread 0 writes it
  uint32_t mag = 0;
#pragma unroll
  for (int u = 0; u < kUnits; ++u)
    mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(x[u].x & 0x7fff7fffu, x[u].y & 0x7fff7fffu),
                                 __vmaxu2(x[u].z & 0x7fff7fffu, x[u].w & 0x7fff7fffu)));
  mag = cta_max_bf16(mag, part[0]);
  if (mag >= 0x7f80u) {  // infinities saturate like any other large value and NaN stays NaN: neither sets the scale
    mag = 0;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = w[i] & 0x7fff7fffu;
        mag = __vmaxu2(mag, a & ~__vcmpgeu2(a, 0x7f807f80u));
      }
    }
    mag = cta_max_bf16(mag, part[1]);
  }
  const float amax = __uint_as_float(mag << 16);
  const float fresh = exp2_int(scale_exponent(amax));
  const bool have_old = old > 0.f && old < INFINITY;
  const float now = have_old && old > fresh ? old : fresh;
  const bool again = have_old && now > old;  // the rows that were there are rounded again
  const float inv = 1.f / now;
  if (threadIdx.x == 0 && dcheck(blk < c.n_blocks, status, kWhereKv8Store)) *scale = now;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int32_t row = first + u * step;
    if (row >= end || (row < held && !again)) continue;
    uint2* out = reinterpret_cast<uint2*>(dst + (int64_t)(u * step) * c.ld);
    uint32_t y[2];
    if (row >= held) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[u]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 f0 = unpack_bf16x2(w[2 * i]), f1 = unpack_bf16x2(w[2 * i + 1]);
        y[i] = (uint32_t)f32x2_to_e4m3x2(f0.x * inv, f0.y * inv) |
               ((uint32_t)f32x2_to_e4m3x2(f1.x * inv, f1.y * inv) << 16);
      }
    } else {
      const uint2 o2 = *out;
      const uint32_t w[2] = {o2.x, o2.y};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t a = cvt_lo(w[i]), d = cvt_hi(w[i]);
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&a));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&d));
        y[i] = (uint32_t)f32x2_to_e4m3x2(f0.x * old * inv, f0.y * old * inv) |
               ((uint32_t)f32x2_to_e4m3x2(f1.x * old * inv, f1.y * old * inv) << 16);
      }
    }
    if (dcheck(row < c.capacity, status, kWhereKv8Store)) *out = make_uint2(y[0], y[1]);
  }
}

// ------------------------------------------------------------------ evict
// Two kernels.  The first, one CTA per (sequence, head), finds which blocks
// stay.  Up to kSelectThreads free blocks every thread counts the blocks that
// come before its own (one pass over shared memory); above, a radix select over
// the ordered bits of the weights (four passes of 8 bits) gives the threshold.
// Then one pass in index order lists the blocks that stay and moves their scales
// and weights.  The second kernel moves the rows.
// 1,560 of 14,106 rows x 32 heads go: 47 to 49 us, the moves 41 of them (198 MB,
// read and write in turn) against 30 at the copy's rate.
constexpr int kSelectThreads = 512;

struct EvictPlan {  // per sequence and head, in the workspace
  int32_t len, nb, count;
  int32_t first;  // the first kept block that moves
};

// Orders like torch's descending sort: NaN above infinity, both zeros equal.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelectThreads)
    evict_select_kernel(const __grid_constant__ Cache c, const float* weight, int32_t keep, int32_t first_rows,
                        int32_t last_rows, float* weight_out, EvictPlan* plan, int32_t* list, int* status) {
  pdl_trigger();
  pdl_wait();
  __shared__ uint32_t hist[256];
  __shared__ __align__(16) uint32_t keys[kSelectThreads];
  __shared__ uint32_t sh_prefix, sh_need;
  __shared__ int32_t sh_first;
  __shared__ uint32_t warp_cnt[2][kSelectThreads / 32];
  const int32_t b = blockIdx.x / c.n_kv;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int64_t base = (int64_t)blockIdx.x * c.n_blocks;
  const float* w = weight + base;
  // the first kSelectThreads blocks' values, on their way with the length
  float w0 = 0.f, ks0 = 0.f, vs0 = 0.f;
  if (tid < c.n_blocks) {
    w0 = w[tid];
    ks0 = c.k_scale[base + tid];
    vs0 = c.v_scale[base + tid];
  }
  const int32_t len = shown_rows(c, b, 0, status, tid == 0);
  const int32_t nb = (len + c.block - 1) / c.block;
  // fixed blocks: [0, head) and [tail, nb)
  const int32_t head = min(nb, (int32_t)(((int64_t)first_rows + c.block - 1) / c.block));
  const int32_t tail = max(head, min(nb, (len - min(len, last_rows)) / c.block));
  const int32_t n_fixed = nb - (tail - head);
  const int32_t count = min(nb, max(keep, n_fixed));
  int32_t* out = list + base;
  if (tid == 0) sh_first = count;

  // threshold: the (count - n_fixed)-th largest key of [head, tail)
  uint32_t prefix = 0, need = (uint32_t)(count - n_fixed);
  const bool all = (int32_t)need >= tail - head;
  const bool count_ranks = !all && need > 0 && tail - head <= kSelectThreads;
  if (count_ranks) {
    const bool mine = tid < tail - head;
    const uint32_t k = mine ? weight_key(head == 0 ? w0 : w[head + tid]) : 0u;
    keys[tid] = k;
    __syncthreads();
    uint32_t before = 0;
    // keys behind the last free block are 0: below every weight's
    for (int i = 0; i < tail - head; i += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(keys + i);
      before += (x.x > k || (x.x == k && i < tid) ? 1u : 0u) + (x.y > k || (x.y == k && i + 1 < tid) ? 1u : 0u) +
                (x.z > k || (x.z == k && i + 2 < tid) ? 1u : 0u) + (x.w > k || (x.w == k && i + 3 < tid) ? 1u : 0u);
    }
    __syncthreads();
    keys[tid] = mine && before < need ? 1u : 0u;  // block head + tid is among the first `need`
    __syncthreads();
  } else if (!all && need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
      for (int32_t j = head + tid; j < tail; j += kSelectThreads) {
        const uint32_t k = weight_key(w[j]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (wid == 0) {  // lane l holds digits 255 - 8l .. 248 - 8l, the largest first
        uint32_t d[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += d[i] = hist[255 - 8 * lane - i];
        uint32_t before = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint32_t t = __shfl_up_sync(0xffffffffu, before, off);
          if (lane >= off) before += t;
        }
        before -= sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < need && need <= before + d[i]) {
            sh_prefix = prefix | ((uint32_t)(255 - 8 * lane - i) << shift);
            sh_need = need - before;
          }
          before += d[i];
        }
      }
      __syncthreads();
      prefix = sh_prefix;
      need = sh_need;
      __syncthreads();
    }
  }
  // kept blocks in index order
  uint32_t kept = 0, ties = 0;
  for (int32_t j0 = 0; j0 < nb; j0 += kSelectThreads) {
    const int32_t j = j0 + tid;
    // read before anything of this chunk is written (destinations lie at or before their sources)
    if (j0 > 0 && j < nb) {
      w0 = w[j];
      ks0 = c.k_scale[base + j];
      vs0 = c.v_scale[base + j];
    }
    bool sure = j < nb && (j < head || j >= tail || all), tie = false;
    if (count_ranks) {
      sure = sure || (j >= head && j < tail && keys[j - head] != 0);
    } else if (j < nb && !sure && count > n_fixed) {
      const uint32_t k = weight_key(j0 == 0 ? w0 : w[j]);
      sure = k > prefix;
      tie = k == prefix;
    }
    const uint32_t tie_votes = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) warp_cnt[0][wid] = __popc(tie_votes);
    __syncthreads();
    uint32_t rank = ties, total = ties;
    for (int i = 0; i < kSelectThreads / 32; ++i) {
      if (i < wid) rank += warp_cnt[0][i];
      total += warp_cnt[0][i];
    }
    ties = total;
    rank += __popc(tie_votes & ((1u << lane) - 1u));
    const bool stay = sure || (tie && rank < need);
    const uint32_t votes = __ballot_sync(0xffffffffu, stay);
    if (lane == 0) warp_cnt[1][wid] = __popc(votes);
    __syncthreads();
    uint32_t at = kept;
    total = kept;
    for (int i = 0; i < kSelectThreads / 32; ++i) {
      if (i < wid) at += warp_cnt[1][i];
      total += warp_cnt[1][i];
    }
    kept = total;
    at += __popc(votes & ((1u << lane) - 1u));
    if (stay && dcheck((int32_t)at < count, status, kWhereKv8Store)) {
      out[at] = j;
      if ((int32_t)at < j) {
        c.k_scale[base + at] = ks0;
        c.v_scale[base + at] = vs0;
        atomicMin(&sh_first, (int32_t)at);
      }
      weight_out[base + at] = w0;
    }
  }
  __syncthreads();
  for (int32_t j = count + tid; j < c.n_blocks; j += kSelectThreads) {
    if (!dcheck(j >= 0 && count <= nb && nb <= c.n_blocks, status, kWhereKv8Store)) break;
    if (j < nb)
      weight_out[base + j] = 0.f;  // blocks that a later store begins anew
    else if (weight_out != weight)
      weight_out[base + j] = w[j];
  }
  if (tid == 0) plan[blockIdx.x] = EvictPlan{len, nb, count, sh_first};
}

// Blocks move towards the front: the source of the j-th kept block is list[j]
// >= j, ascending.  A thread owns one 16-byte piece of one row of every block
// and walks j upwards, kMoveTurn blocks a turn; it has begun to read the sources
// of a turn and of the ones after it before it writes the turn's blocks, and no
// later source is a block that it has written, so the move is in place without any thread waiting
// for another.  The pieces wait in the thread's own slots of shared memory.
// 24 pieces on their way take 49 us where 16 take 59 and 8 take 62.  Eight blocks
// a turn count where few threads walk far: 20,000 rows in blocks of 16, 2 heads
// of 64, 600 kept: 70 us, with two a turn 89-94, with twelve 79.
constexpr int kMoveThreads = 128, kMoveTurn = 8, kMoveRing = 24;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ Cache c,
                                                                  const EvictPlan* plan,
                                                                  const int32_t* list, int32_t* lens_out,
                                                                  int* status) {
  pdl_trigger();
  pdl_wait();
  const int32_t b = blockIdx.y / c.n_kv, g = blockIdx.y % c.n_kv;
  const EvictPlan pl = plan[blockIdx.y];
  const int32_t* src = list + (int64_t)blockIdx.y * c.n_blocks;
  const int32_t part = pl.len - (pl.nb - 1) * c.block;  // rows of the last block, which stays if it is not full
  if (blockIdx.x == 0 && blockIdx.z == 0 && g == 0 && threadIdx.x == 0)
    lens_out[b] = pl.nb == 0 ? 0 : (pl.count - 1) * c.block + part;
  const int per_row = c.hd >> 4;
  const int unit = (int)blockIdx.x * (int)blockDim.x + (int)threadIdx.x;
  const int32_t r = unit / per_row;
  if (r >= c.block) return;
  uint8_t* base = (blockIdx.z ? c.v : c.k) + ((int64_t)b * c.bstride + r) * c.ld + (int64_t)g * c.hd +
                  (unit % per_row) * 16;
  const int64_t step = (int64_t)c.block * c.ld;
  const int32_t lo = pl.first, end = pl.count - (r >= part ? 1 : 0);
  __shared__ __align__(16) uint4 ring[kMoveRing][kMoveThreads];
  const uint32_t at = smem_u32(&ring[0][threadIdx.x]);
  // the list is read one turn ahead: its latency would pace the thread
  int32_t next[kMoveTurn];
  auto look = [&](int32_t j) {
#pragma unroll
    for (int i = 0; i < kMoveTurn; ++i) {
      next[i] = j + i < end ? src[j + i] : 0;
      // a source behind its destination, both inside the cache; else (debug build) the block stays as it is
      if (j + i < end && !dcheck(next[i] >= j + i && (int64_t)next[i] * c.block + r < c.capacity, status, kWhereKv8Store))
        next[i] = j + i;
    }
  };
  auto read = [&](int32_t j, int slot) {  // kMoveTurn blocks from j on, whose sources `next` holds
#pragma unroll
    for (int i = 0; i < kMoveTurn; ++i)
      if (j + i < end)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + (slot * kMoveTurn + i) * (kMoveThreads * 16)),
                     "l"(base + next[i] * step)
                     : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  constexpr int kTurns = kMoveRing / kMoveTurn;  // on their way at any time
  look(lo);
#pragma unroll
  for (int i = 0; i < kTurns - 1; ++i) {
    read(lo + i * kMoveTurn, i);
    look(lo + (i + 1) * kMoveTurn);
  }
  int slot = 0;
#pragma unroll 2
  for (int32_t j = lo; j < end; j += kMoveTurn) {
    read(j + (kTurns - 1) * kMoveTurn, slot == 0 ? kTurns - 1 : slot - 1);
    look(j + kTurns * kMoveTurn);
    asm volatile("cp.async.wait_group %0;" ::"n"(kTurns - 1) : "memory");
#pragma unroll
    for (int i = 0; i < kMoveTurn; ++i) {
      uint4 x;
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                   : "r"(at + (slot * kMoveTurn + i) * (kMoveThreads * 16))
                   : "memory");
      if (j + i < end && dcheck((int64_t)(j + i) * c.block + r < c.capacity, status, kWhereKv8Store))
        *reinterpret_cast<uint4*>(base + (j + i) * step) = x;
    }
    slot = slot == kTurns - 1 ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------------ host
cosmot_status make_cache(const cosmot_kv8_cache* c, Cache& o) {
  if (!c) return COSMOT_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return COSMOT_ERR_UNSUPPORTED;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return COSMOT_ERR_UNSUPPORTED;
  if (c->batch < 1 || c->capacity < 1 || c->n_kv_heads < 1) return COSMOT_ERR_INVALID_ARG;
  if (c->ld < (int64_t)c->n_kv_heads * c->head_dim || c->ld % 16) return COSMOT_ERR_INVALID_ARG;
  if (c->batch > 1 && c->batch_stride < c->capacity) return COSMOT_ERR_INVALID_ARG;
  if ((int64_t)c->batch * c->n_kv_heads > 65535) return COSMOT_ERR_UNSUPPORTED;
  // row indices of the key tiles are 32 bits wide
  if (c->capacity > INT32_MAX - 256 ||
      (c->batch > 1 && c->batch_stride > (INT32_MAX - 256 - (int64_t)c->capacity) / (c->batch - 1)))
    return COSMOT_ERR_UNSUPPORTED;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->lens) return COSMOT_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return COSMOT_ERR_INVALID_ARG;
  o = Cache{};
  o.k = static_cast<uint8_t*>(c->k);
  o.v = static_cast<uint8_t*>(c->v);
  o.k_scale = c->k_scale;
  o.v_scale = c->v_scale;
  o.lens = c->lens;
  o.ld = c->ld;
  o.bstride = c->batch > 1 ? c->batch_stride : 0;
  o.batch = c->batch;
  o.capacity = c->capacity;
  o.n_kv = c->n_kv_heads;
  o.hd = c->head_dim;
  o.block = c->block;
  o.n_blocks = (c->capacity + c->block - 1) / c->block;
  return COSMOT_OK;
}

cosmot_status make_query(const cosmot_kv8_cache* c, const cosmot_kv8_query* d, Query& o) {
  if (!c || !d) return COSMOT_ERR_INVALID_ARG;
  if (d->n_heads < 1 || c->n_kv_heads < 1 || d->n_heads % c->n_kv_heads) return COSMOT_ERR_INVALID_ARG;
  if (d->n_q < 0 || d->n_new < 0 || d->n_new > c->capacity || d->max_len < 0) return COSMOT_ERR_INVALID_ARG;
  if (d->mask_mode != COSMOT_KV8_FULL && d->mask_mode != COSMOT_KV8_CAUSAL) return COSMOT_ERR_INVALID_ARG;
  if (c->batch > 1 && (d->q_batch_stride < d->n_q || d->o_batch_stride < d->n_q)) return COSMOT_ERR_INVALID_ARG;
  if (!(d->softmax_scale >= 0.f) || d->softmax_scale > 1e30f) return COSMOT_ERR_INVALID_ARG;
  o = Query{};
  o.n_q = d->n_q;
  o.group = d->n_heads / c->n_kv_heads;
  if (d->n_q > INT32_MAX / 2 / o.group) return COSMOT_ERR_UNSUPPORTED;
  o.n_rows = d->n_q * o.group;
  o.n_heads = d->n_heads;
  o.n_new = d->n_new;
  o.causal = d->mask_mode == COSMOT_KV8_CAUSAL;
  o.q_bstride = c->batch > 1 ? d->q_batch_stride : 0;
  o.o_bstride = c->batch > 1 ? d->o_batch_stride : 0;
  o.scale_log2 = (d->softmax_scale > 0.f ? d->softmax_scale : 1.0f / sqrtf((float)c->head_dim)) * kLog2e;
  o.splits = 1;
  return COSMOT_OK;
}

namespace {

// Rows that the host may take any sequence to show (it sizes splits only).
int32_t bound_len(const cosmot_kv8_cache* c, const cosmot_kv8_query* d) {
  return d->max_len > 0 && d->max_len < c->capacity ? d->max_len : c->capacity;
}

cosmot_status check_q(const cosmot_kv8_cache* c, const cosmot_kv8_query* d, const void* q, int64_t ld_q) {
  if (!q || !aligned16(q) || ld_q % 8 || ld_q < (int64_t)d->n_heads * c->head_dim) return COSMOT_ERR_INVALID_ARG;
  return COSMOT_OK;
}

size_t o_part_bytes(const Cache& c, const Query& p) {
  return ((size_t)p.splits * c.batch * c.n_kv * p.n_rows * c.hd * 4 + 255) & ~size_t(255);
}
size_t part_bytes(const Cache& c, const Query& p) {
  return p.splits == 1 ? 0 : o_part_bytes(c, p) + (size_t)p.splits * c.batch * c.n_kv * p.n_rows * 8;
}

// Up to kRowsMax packed rows the register-tile kernels run, above it the tcgen05
// ones.  Attention, 14,106 rows x 32 heads: 53 against 61 us at 32 rows, 71
// against 63 at 48.  Weighing, 32 heads: 44 against 57 at 32, 63 against 57 at 48.
// The rule looks at the rows alone: x 8 heads the register tiles take 23 us where
// the others take 30 at 32 rows and still 31 against 32 at 64, so that 33 to 63
// rows on few heads would go a little faster there.
constexpr int64_t kRowsMax = 32;
bool use_tiles(const Query& p) { return p.n_rows > kRowsMax; }

// A range of 256 keys is weighed by all the rows in one go, 1.5 us for 128 of
// them, and the warps that wait for its end do so for a second at most: 2^25 rows
// take 0.4 s.
constexpr int64_t kWeighRowsMax = int64_t(1) << 25;

size_t evict_list_offset(const Cache& c) { return ((size_t)c.batch * c.n_kv * sizeof(EvictPlan) + 255) & ~size_t(255); }

}  // namespace
}  // namespace kv8
}  // namespace cosmot

using namespace cosmot;

extern "C" cosmot_status cosmot_kv8_store(const cosmot_kv8_cache* cache, const void* k, const void* v, int64_t ld_src,
                                          int64_t src_batch_stride, int32_t n_rows, cosmot_stream_t stream) {
  kv8::Cache c;
  cosmot_status st = kv8::make_cache(cache, c);
  if (st != COSMOT_OK) return st;
  if (!k || !v || !aligned16(k) || !aligned16(v) || ld_src % 8 || ld_src < (int64_t)c.n_kv * c.hd)
    return COSMOT_ERR_INVALID_ARG;
  if (n_rows < 0 || n_rows > c.capacity || (c.batch > 1 && src_batch_stride < n_rows)) return COSMOT_ERR_INVALID_ARG;
  if (n_rows == 0) return COSMOT_OK;
  int* status = device_status_ptr();
  if (!status) return COSMOT_ERR_CUDA;
  const int pieces = c.block * c.hd / 8;  // 128 .. 2048
  const int64_t ctas = 2 * (int64_t)c.batch * c.n_kv * (((int64_t)n_rows + 2 * c.block - 2) / c.block);
  if (ctas > INT32_MAX) return COSMOT_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)ctas);
  const dim3 block((unsigned)(pieces < kv8::kStoreThreads ? pieces : kv8::kStoreThreads));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t bs = c.batch > 1 ? src_batch_stride : 0;
  const auto* ks = static_cast<const __nv_bfloat16*>(k);
  const auto* vs = static_cast<const __nv_bfloat16*>(v);
  auto* kern = pieces <= 256    ? kv8::store_kernel<1>
               : pieces == 512  ? kv8::store_kernel<2>
               : pieces == 1024 ? kv8::store_kernel<4>
                                : kv8::store_kernel<8>;
  const cudaError_t e = launch_pdl(kern, grid, block, 0, s, nullptr, c, ks, vs, ld_src, bs, n_rows, status);
  return launch_status(e);
}

extern "C" cosmot_status cosmot_kv8_attention_workspace(const cosmot_kv8_cache* cache, const cosmot_kv8_query* query,
                                                        size_t* bytes) {
  kv8::Cache c;
  kv8::Query p;
  if (!bytes) return COSMOT_ERR_INVALID_ARG;
  cosmot_status st = kv8::make_cache(cache, c);
  if (st == COSMOT_OK) st = kv8::make_query(cache, query, p);
  if (st != COSMOT_OK) return st;
  if (kv8::use_tiles(p)) {
    if (!kv8::tile_fits(c, p)) return COSMOT_ERR_UNSUPPORTED;
    *bytes = kv8::tile_workspace(c, p, kv8::bound_len(cache, query));
    return COSMOT_OK;
  }
  kv8::rows_plan(c, p, kv8::bound_len(cache, query));
  *bytes = kv8::part_bytes(c, p);
  return COSMOT_OK;
}

extern "C" cosmot_status cosmot_kv8_attention(const cosmot_kv8_cache* cache, const cosmot_kv8_query* query,
                                              const void* q, int64_t ld_q, void* o, int64_t ld_o, float* lse,
                                              void* workspace, size_t workspace_bytes, cosmot_stream_t stream) {
  kv8::Cache c;
  kv8::Query p;
  cosmot_status st = kv8::make_cache(cache, c);
  if (st == COSMOT_OK) st = kv8::make_query(cache, query, p);
  if (st == COSMOT_OK) st = kv8::check_q(cache, query, q, ld_q);
  if (st != COSMOT_OK) return st;
  if (!o || !aligned16(o) || ld_o % 8 || ld_o < (int64_t)p.n_heads * c.hd) return COSMOT_ERR_INVALID_ARG;
  const int32_t max_len = kv8::bound_len(cache, query);
  const bool tiles = kv8::use_tiles(p);
  if (tiles && !kv8::tile_fits(c, p)) return COSMOT_ERR_UNSUPPORTED;
  if (!tiles) kv8::rows_plan(c, p, max_len);
  const size_t need = tiles ? kv8::tile_workspace(c, p, max_len) : kv8::part_bytes(c, p);
  if (need > 0) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return COSMOT_ERR_INVALID_ARG;
    if (workspace_bytes < need) return COSMOT_ERR_WORKSPACE;
  }
  if (!tiles && need > 0) {
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + kv8::o_part_bytes(c, p));
    p.part_rows = (int64_t)p.splits * c.batch * c.n_kv * p.n_rows;
  }
  if (p.n_q == 0) return COSMOT_OK;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.ld_q = ld_q;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.ld_o = ld_o;
  p.lse = lse;
  p.status = device_status_ptr();
  if (!p.status) return COSMOT_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return tiles ? kv8::tile_attention(c, p, max_len, workspace, s) : kv8::rows_attention(c, p, s);
}

extern "C" cosmot_status cosmot_kv8_weigh(const cosmot_kv8_cache* cache, const cosmot_kv8_query* query, const void* q,
                                          int64_t ld_q, const float* lse, float decay, float* weight,
                                          cosmot_stream_t stream) {
  kv8::Cache c;
  kv8::Query p;
  cosmot_status st = kv8::make_cache(cache, c);
  if (st == COSMOT_OK) st = kv8::make_query(cache, query, p);
  if (st == COSMOT_OK) st = kv8::check_q(cache, query, q, ld_q);
  if (st != COSMOT_OK) return st;
  if (!lse || !weight || !(decay >= 0.f) || decay > 1e30f) return COSMOT_ERR_INVALID_ARG;
  if (p.n_rows > kv8::kWeighRowsMax) return COSMOT_ERR_UNSUPPORTED;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.ld_q = ld_q;
  p.lse = const_cast<float*>(lse);
  p.status = device_status_ptr();
  if (!p.status) return COSMOT_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return kv8::use_tiles(p) && p.group <= 128
             ? kv8::tile_weigh(c, p, decay, weight, kv8::bound_len(cache, query), s)
             : kv8::rows_weigh(c, p, decay, weight, kv8::bound_len(cache, query), s);
}

extern "C" cosmot_status cosmot_kv8_evict_workspace(const cosmot_kv8_cache* cache, size_t* bytes) {
  kv8::Cache c;
  if (!bytes) return COSMOT_ERR_INVALID_ARG;
  const cosmot_status st = kv8::make_cache(cache, c);
  if (st != COSMOT_OK) return st;
  *bytes = kv8::evict_list_offset(c) + (size_t)c.batch * c.n_kv * c.n_blocks * sizeof(int32_t);
  return COSMOT_OK;
}

extern "C" cosmot_status cosmot_kv8_evict(const cosmot_kv8_cache* cache, const float* weight, int32_t keep_blocks,
                                          int32_t first_rows, int32_t last_rows, float* weight_out, int32_t* lens_out,
                                          void* workspace, size_t workspace_bytes, cosmot_stream_t stream) {
  kv8::Cache c;
  cosmot_status st = kv8::make_cache(cache, c);
  if (st != COSMOT_OK) return st;
  if (!weight || !weight_out || !lens_out || keep_blocks < 1 || first_rows < 0 || last_rows < 0)
    return COSMOT_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return COSMOT_ERR_INVALID_ARG;
  size_t need = 0;
  if (cosmot_kv8_evict_workspace(cache, &need) != COSMOT_OK || workspace_bytes < need) return COSMOT_ERR_WORKSPACE;
  int* status = device_status_ptr();
  if (!status) return COSMOT_ERR_CUDA;
  auto* plan = static_cast<kv8::EvictPlan*>(workspace);
  auto* list = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + kv8::evict_list_offset(c));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = launch_status(launch_pdl(kv8::evict_select_kernel, dim3((unsigned)(c.batch * c.n_kv)),
                                dim3(kv8::kSelectThreads), 0, s, nullptr, c, weight, keep_blocks, first_rows, last_rows,
                                weight_out, plan, list, status));
  if (st != COSMOT_OK) return st;
  const unsigned slices = (unsigned)((c.block * c.hd / 16 + kv8::kMoveThreads - 1) / kv8::kMoveThreads);  // 64 .. 1024 pieces
  return launch_status(launch_pdl(kv8::evict_move_kernel, dim3(slices, (unsigned)(c.batch * c.n_kv), 2),
                                  dim3(kv8::kMoveThreads), 0, s, nullptr, c, (const kv8::EvictPlan*)plan,
                                  (const int32_t*)list, lens_out, status));
}

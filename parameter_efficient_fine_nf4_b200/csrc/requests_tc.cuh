// The many-adapter products on tensor cores (tcgen05), for batches of more
// than a few tokens: tiles of up to 128 tokens of one adapter.
//
//   shrink:  V = s X A_a^T        (128 tokens x rank, K columns split over a cluster)
//   expand:  Y = base + V Bt_a    (128 tokens x a range of columns)
//   grads:   dA_a = V^T X         (256 columns x rank, the tokens of all units cut into equal parts, one per CTA;
//                                  a second kernel adds up the units that were cut)
// The backward is the same three kernels with A and Bt, X and dY exchanged.
//
// V is a 32-bit value kept as three bf16 terms, v = hi + mid + lo (8 bits of
// significand each), so that products with bf16 factors are exact in fp32:
// expand multiplies hi and mid (2^-16 of the term, far below the one rounding
// of its bf16 output), grads all three (its outputs are fp32).  A row of V
// holds, for each 64 of the adapter's rank (rounded to 16), 64 columns for hi,
// then mid | lo side by side.  Rows are tile by tile, 128 each, and zero behind a tile's
// tokens.  So V is an ordinary TMA operand for expand (K-major) and for grads
// (MN-major), with no gather, and only X, dY, base and the outputs are
// addressed by token.
//
// Token rows come in by TMA, 32 at a time where they are consecutive and whole
// (a request's tokens are) and four at a time (gather4) elsewhere; a gathered
// row behind the tile's tokens repeats the last one, so nothing that the tile
// does not own is ever multiplied.
//
// The tensor core adds into its 32-bit accumulator by cutting, not rounding:
// measured, a sum over 5,500 tokens in one accumulator is 7e-5 off, always
// towards zero.  So an accumulator whose result is kept in 32 bits takes a
// short piece of the long sum only (shrink: 64 columns; grads: 128 tokens); two
// alternate, and the epilogue warps add each to registers, rounding to nearest,
// while the other one fills.
#pragma once
#include "ptx.cuh"
#include "requests_kernels.cuh"

namespace qlora {

constexpr int kReqTile = 128;
// warp 0: TMA, warp 1: MMA, the others: epilogue
constexpr int kExpandThreads = 320;          // warps 2-9: epilogue, 32 rows x 32 columns of a stage each
constexpr int kShrinkThreads = 320;          // warps 2-9: epilogue, two per quarter of the rows
constexpr int kReqRows = 128 * 128;          // bytes of 128 rows x 64 bf16 columns

// Columns of a V row, from the widest adapter of the pool.
__host__ __device__ __forceinline__ int terms_ld(int width) {
  return width <= 64 ? 64 + (2 * width + 63) / 64 * 64 : (width + 63) / 64 * 192;
}
// Column of term `part` of rank index j for an adapter of r16 (rank rounded to 16).
__device__ __forceinline__ int term_col(int j, int part, int r16) {
  const int c = j >> 6;
  const int rc = min(64, r16 - 64 * c);
  return 192 * c + (part == 0 ? 0 : 64 + (part - 1) * rc) + (j & 63);
}

__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, const int (&y)[4]) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
      : "memory");
}

// Four consecutive rows of a group of tokens for this lane: rows 4 i .. 4 i + 3
// of `count`, token numbers from order[first ...]; `whole`: the 32 rows of
// this lane's group of 8 lanes are all there and consecutive.
struct RowLane {
  int tok[4];
  bool whole;
};
__device__ __forceinline__ void row_tokens(RowLane& r, const int32_t* order, int first, int count, int i) {
#pragma unroll
  for (int j = 0; j < 4; ++j) r.tok[j] = __ldcg(order + first + max(0, min(4 * i + j, count - 1)));
}
__device__ __forceinline__ void row_whole(RowLane& r, int count, int i) {
  const int lane = threadIdx.x & 31;
  const int a = __shfl_sync(0xFFFFFFFFu, r.tok[0], lane & ~7);
  const int b = __shfl_sync(0xFFFFFFFFu, r.tok[3], lane | 7);
  r.whole = (i / 8 + 1) * 32 <= count && b - a == 31;
}
__device__ __forceinline__ RowLane row_lane(const int32_t* order, int first, int count, int i) {
  RowLane r;
  row_tokens(r, order, first, count, i);
  row_whole(r, count, i);
  return r;
}
// This lane's part of one 64-column block of token rows (rounded up to 16).
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* box, const CUtensorMap* row, uint32_t bar, int x,
                                          const RowLane& r, int i, int count) {
  if (r.whole) {
    if (i % 8 == 0) tma_load_2d(dst + (uint32_t)i * 512u, box, bar, x, r.tok[0]);
  } else if (4 * i < (count + 15) / 16 * 16) {
    tma_gather4(dst + (uint32_t)i * 512u, row, bar, x, r.tok);
  }
}
__device__ __forceinline__ uint32_t row_bytes(int count) { return (uint32_t)((count + 15) / 16 * 16 * 128); }

__device__ __forceinline__ float bf16_round(float v, uint16_t& bits) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  bits = *reinterpret_cast<const uint16_t*>(&h);
  return __bfloat162float(h);
}

// Writes four consecutive rank values (j % 4 == 0) of one V row as three terms.
__device__ __forceinline__ void store_terms(uint16_t* row, int j, int r16, const float (&v)[4]) {
  uint16_t t[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float h = bf16_round(v[i], t[0][i]);
    const float rest = __fsub_rn(v[i], h);
    const float m = bf16_round(rest, t[1][i]);
    bf16_round(__fsub_rn(rest, m), t[2][i]);
  }
#pragma unroll
  for (int part = 0; part < 3; ++part)
    *reinterpret_cast<uint2*>(row + term_col(j, part, r16)) =
        make_uint2((uint32_t)t[part][0] | ((uint32_t)t[part][1] << 16), (uint32_t)t[part][2] | ((uint32_t)t[part][3] << 16));
}

// A shared-memory ring of stages with full and empty barriers.
struct Ring {
  uint32_t full, empty;          // first barrier of each, 8 bytes apart
  int stages;
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ uint32_t full_bar() const { return full + 8u * at; }
  __device__ __forceinline__ uint32_t empty_bar() const { return empty + 8u * at; }
  __device__ __forceinline__ void next() {
    if (++at == stages) {
      at = 0;
      phase ^= 1u;
    }
  }
};

// Four values of every CTA of the cluster, added in rank order, the loads together.
template <int CS>
__device__ __forceinline__ float4 cluster_sum(uint32_t at) {
  float4 f[CS];
#pragma unroll
  for (int c = 0; c < CS; ++c) f[c] = ld_shared_cluster_f4(mapa_shared(at, (uint32_t)c));
  float4 v = f[0];
#pragma unroll
  for (int c = 1; c < CS; ++c) {
    v.x += f[c].x; v.y += f[c].y; v.z += f[c].z; v.w += f[c].w;
  }
  return v;
}

// ---------------------------------------------------------------------- shrink
struct ShrinkArgs {
  const int32_t* order;
  const int4* tiles;
  PoolArgs pool;
  int K, width, csize, stages, tmem_cols, stage_bytes, ld;
  float* U;                     // T x width, or null: the unscaled product
  uint16_t* V;                  // terms of scale * product
  const float* U_in;            // T x width, or null: a saved U ...
  uint16_t* V_in;               // ... whose terms (times the scale) are laid out as well
};

// X is streamed once; the factor's rows come from L2; the split over the cluster
// only makes enough CTAs.  Reading X is what has to be done, but no unit is near
// its peak (46 % of DRAM at 8192 tokens of 11008 columns): set-up, the first loads
// and the cluster's exchange are some 10 us of a launch, and above that a little over
// one wave of CTAs leaves SMs idle at the end.  NI: 32 columns of
// the rank per step of the epilogue's registers (width <= 32 NI).  Measured
// (alone, between two events, L2 flushed): 4096 tokens of 4096 columns, ranks 8
// to 64, 21 us; 16384 tokens of rank 64, 8192 columns 74 us (3.6 TB/s of X) and
// 22016 columns 171 us (4.2 TB/s).
template <int NI>
__global__ void __launch_bounds__(kShrinkThreads) requests_shrink_kernel(const __grid_constant__ CUtensorMap box,
                                                                      const __grid_constant__ CUtensorMap row,
                                                                      const __grid_constant__ CUtensorMap weight,
                                                                      const __grid_constant__ ShrinkArgs p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[2 * 8 + 4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - smem_u32(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = (int)(blockIdx.x % p.csize), u = (int)(blockIdx.x / p.csize);
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&box);
    tma_prefetch_desc(&row);
    tma_prefetch_desc(&weight);
  }
  volatile int* abort_flag = &s_abort;

  Ring ring;
  ring.full = smem_u32(&s_bar[0]);
  ring.empty = smem_u32(&s_bar[8]);
  ring.stages = p.stages;
  const uint32_t acc_full = smem_u32(&s_bar[16]), acc_empty = smem_u32(&s_bar[18]);   // two each
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(ring.full + 8u * i, 1);
      mbar_init(ring.empty + 8u * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8u * i, 1);
      mbar_init(acc_empty + 8u * i, 8);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), (uint32_t)p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  griddep_wait();
  // (behind the allocation: a dependent that allocates early must not take Tensor Memory this CTA still needs)
  griddep_launch_dependents();
  const int4 tile = p.tiles[u];
  if (tile.z <= 0) {                             // the whole cluster
    if (warp == 1) tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
    return;
  }
  const int count = min(tile.z, kReqTile);
  const AdapterRows ad = adapter_rows(p.pool, tile.x, p.width);
  if (ad.rank == 0) {
    if (p.U && q == 0)
      for (int e = threadIdx.x; e < count * p.width; e += kShrinkThreads)
        p.U[(int64_t)p.order[tile.y + e / p.width] * p.width + e % p.width] = 0.f;
    if (warp == 1) tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
    return;
  }
  const int r16 = (ad.rank + 15) & ~15;
  const int kper = ((p.K + p.csize - 1) / p.csize + 63) / 64 * 64;
  const int k0 = min(p.K, q * kper), k1 = min(p.K, k0 + kper);
  const int steps = (k1 - k0 + 63) / 64;

  if (warp == 0) {
    const RowLane r = row_lane(p.order, tile.y, count, lane);
    const uint32_t bytes = row_bytes(count) + (uint32_t)r16 * 128u;
    int issued = 0;
    for (int s = 0; s < steps; ++s) {
      int ok = 1;
      if (lane == 0) {
        ok = mbar_wait_bounded(ring.empty_bar(), ring.phase ^ 1u, abort_flag);
        if (ok) mbar_arrive_expect_tx(ring.full_bar(), bytes);
      }
      if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
      const uint32_t st = sbase + (uint32_t)(ring.at * p.stage_bytes);
      const int x = k0 + s * 64;
      load_rows(st, &box, &row, ring.full_bar(), x, r, lane, count);
      if (lane < r16 / 16)
        tma_load_2d(st + kReqRows + (uint32_t)lane * 2048u, &weight, ring.full_bar(), x, ad.first + 16 * lane);
      ring.next();
      ++issued;
    }
    if (*abort_flag && lane == 0) {              // let copies in flight land
      for (int i = 0; i < min(issued, p.stages); ++i) {
        const int last = (issued - 1 - i) / p.stages;      // last use of stage i counts from 0
        mbar_wait_bounded(ring.full + 8u * i, (uint32_t)(last & 1), nullptr);
      }
    }
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_bf16_f32(128, r16, 0, 0);
    const uint64_t a0 = smem_desc_sw128(sbase, 16, 1024), b0 = smem_desc_sw128(sbase + kReqRows, 16, 1024);
    bool ok = true;
    int last = -1;
    for (int s = 0; s < steps && ok; ++s) {
      const int buf = s & 1;
      ok = mbar_wait_bounded(acc_empty + 8u * buf, (uint32_t)(((s >> 1) & 1) ^ 1), abort_flag) &&
           mbar_wait_bounded(ring.full_bar(), ring.phase, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const uint32_t off = (uint32_t)(ring.at * p.stage_bytes) >> 4;
      const uint64_t a = a0 + off, b = b0 + off;
#pragma unroll
      for (int j = 0; j < 4; ++j) umma_bf16(tmem + (uint32_t)(buf * r16), a + 2u * j, b + 2u * j, idesc, j ? 1u : 0u);
      last = s;
      umma_commit(ring.empty_bar());
      umma_commit(acc_full + 8u * buf);
      ring.next();
    }
    if (!ok && last >= 0) mbar_wait_bounded(acc_full + 8u * (last & 1), (uint32_t)((last >> 1) & 1), nullptr);
  }
  __syncwarp();

  // the stages' products added up in registers, then to shared memory (all
  // stages are free once the last MMA is done)
  const int pitch = r16 + 4;
  float* s_part = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    const int quarter = warp & 3, half = (warp - 2) >> 2, rowi = quarter * 32 + lane;
    float acc[NI][16];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[i][j] = 0.f;
    for (int s = 0; s < steps; ++s) {
      const int buf = s & 1;
      if (!mbar_wait_bounded(acc_full + 8u * buf, (uint32_t)((s >> 1) & 1), abort_flag)) break;
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int c = 32 * i + 16 * half;
        if (c < r16) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * r16 + c), v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[i][j] += __uint_as_float(v[j]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + 8u * buf);
    }
    // the partial sums lie over the stages: every epilogue warp has seen the last product
    named_bar_sync(1, 256);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = 32 * i + 16 * half;
      if (c < r16)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(s_part + rowi * pitch + c + 4 * j) =
              make_float4(acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]);
    }
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
  if (p.csize > 1) cluster_sync();

  // this CTA's share of the rows: partials added in rank order
  const int rows = kReqTile / p.csize, w4 = p.width / 4;
  const uint32_t part = smem_u32(s_part);
  for (int e = threadIdx.x; e < rows * w4; e += kShrinkThreads) {
    const int i = q * rows + e / w4, j = (e % w4) * 4;
    const bool valid = i < count;
    const int64_t tok = valid ? p.order[tile.y + i] : 0;
    float4 saved = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.V_in && valid && j < r16) saved = *reinterpret_cast<const float4*>(p.U_in + tok * p.width + j);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (valid && j < r16) {
      const uint32_t at = part + (uint32_t)(i * pitch + j) * 4u;
      const float4 f = p.csize == 8 ? cluster_sum<8>(at) : p.csize == 4 ? cluster_sum<4>(at) : p.csize == 2 ? cluster_sum<2>(at)
                       : *reinterpret_cast<const float4*>(s_part + i * pitch + j);
      v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
#pragma unroll
      for (int n = 0; n < 4; ++n)
        if (j + n >= ad.rank) v[n] = 0.f;
    }
    if (p.U && valid) *reinterpret_cast<float4*>(p.U + tok * p.width + j) = make_float4(v[0], v[1], v[2], v[3]);
    if (j < r16) {
      const int64_t vrow = ((int64_t)u * kReqTile + i) * p.ld;
#pragma unroll
      for (int n = 0; n < 4; ++n) v[n] = __fmul_rn(ad.scale, v[n]);
      store_terms(p.V + vrow, j, r16, v);
      if (p.V_in) {
        float w[4] = {saved.x, saved.y, saved.z, saved.w};
#pragma unroll
        for (int n = 0; n < 4; ++n) w[n] = j + n < ad.rank ? __fmul_rn(ad.scale, w[n]) : 0.f;
        store_terms(p.V_in + vrow, j, r16, w);
      }
    }
  }
  if (p.csize > 1) cluster_sync();               // partials stay until every CTA has read them
}

// ---------------------------------------------------------------------- expand
struct ExpandArgs {
  const int32_t* order;
  const int4* tiles;
  const int32_t* n_tiles;
  PoolArgs pool;
  int N, width, stages, stage_bytes, v_bytes;
  const uint16_t* base;
  uint16_t* out;
};

// A CTA's share: pieces of consecutive 64-column blocks of one tile each.  The
// blocks of all tiles, tile by tile, are cut into equal parts, one per CTA, so
// no CTA starts late or ends early and set-up and first loads are paid once.
struct ExpandPiece {
  long long at, end;            // blocks left to this CTA
  int chunks;                   // blocks of a tile
  int u, c, count_c;            // the piece: tile, first block, blocks
  int4 tile;
  AdapterRows ad;
};
__device__ __forceinline__ bool expand_piece(const ExpandArgs& p, ExpandPiece& s) {
  if (s.at >= s.end) return false;
  s.u = (int)(s.at / s.chunks);
  s.c = (int)(s.at % s.chunks);
  s.count_c = (int)min((long long)(s.chunks - s.c), s.end - s.at);
  s.at += s.count_c;
  // (maps and tables past L1: they are read ahead of the dependency wait)
  s.tile = __ldcg(p.tiles + s.u);
  s.tile.z = min(s.tile.z, kReqTile);
  s.ad = adapter_rows(p.pool, s.tile.x, p.width);
  return true;
}
__device__ __forceinline__ ExpandPiece expand_share(const ExpandArgs& p) {
  ExpandPiece s;
  s.chunks = (p.N + 63) / 64;
  const long long all = (long long)__ldcg(p.n_tiles) * s.chunks;
  s.at = all * blockIdx.x / gridDim.x;
  s.end = all * (blockIdx.x + 1) / gridDim.x;
  return s;
}

// Streams base in and Y out, 64 columns of the tile's rows a stage, with a few
// small MMAs (two per 16 of the rank) in between.  Bound by DRAM on large batches, in
// 128-byte pieces of rows (4.8 to 5.2 of the 6.5 TB/s of a copy); at 8192 tokens of
// 4096 columns (35 us, 33 % of DRAM) by the first loads and the last stores.  Measured
// (alone, between two events, L2 flushed): 75 us for 8192 tokens x 11008 columns of rank
// 16 (4.8 TB/s in and out), 279 us for 16384 x 22016 of rank 64 (5.2 TB/s).  Two
// CTAs an SM, so that one's loads run beside the other's epilogue.
__global__ void __launch_bounds__(kExpandThreads, 2) requests_expand_kernel(const __grid_constant__ CUtensorMap box,
                                                                            const __grid_constant__ CUtensorMap row,
                                                                            const __grid_constant__ CUtensorMap weight,
                                                                            const __grid_constant__ CUtensorMap terms,
                                                                            const __grid_constant__ ExpandArgs p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[2 * 8 + 6];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - smem_u32(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &s_abort;

  Ring ring;
  ring.full = smem_u32(&s_bar[0]);
  ring.empty = smem_u32(&s_bar[8]);
  ring.stages = p.stages;
  const uint32_t v_full = smem_u32(&s_bar[16]), v_empty = smem_u32(&s_bar[17]);
  const uint32_t acc_full = smem_u32(&s_bar[18]), acc_empty = smem_u32(&s_bar[20]);   // two each
  const uint32_t stage0 = sbase + (uint32_t)p.v_bytes;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(ring.full + 8u * i, 1);
      mbar_init(ring.empty + 8u * i, 8);
    }
    mbar_init(v_full, 1);
    mbar_init(v_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8u * i, 1);
      mbar_init(acc_empty + 8u * i, 8);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&box);
    tma_prefetch_desc(&row);
    tma_prefetch_desc(&weight);
    tma_prefetch_desc(&terms);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();                   // (behind the allocation, as above)
  const uint32_t tmem = s_tmem;
  // Everything but V was there before the kernel in front started, which waited
  // for it: only V's loads wait for that kernel.
  ExpandPiece s = expand_share(p);

  if (warp == 0) {
    int issued = 0, pieces = 0, ok = 1;
    bool waited = false;
    while (ok && expand_piece(p, s)) {
      if (s.ad.rank == 0) continue;
      const int count = s.tile.z, r16 = (s.ad.rank + 15) & ~15;
      const RowLane r = row_lane(p.order, s.tile.y, count, lane);
      const uint32_t bytes = (p.base ? row_bytes(count) : 0u) + (uint32_t)r16 * 128u;
      // V: hi and mid of every 64 of the rank; for the first piece behind the first stages' loads
      auto load_v = [&] {
        if (!waited) griddep_wait();
        waited = true;
        if (lane == 0) {
          ok = mbar_wait_bounded(v_empty, (uint32_t)((pieces & 1) ^ 1), abort_flag);
          if (ok) {
            const int boxes = 2 * ((r16 + 63) / 64);
            mbar_arrive_expect_tx(v_full, (uint32_t)(boxes * kReqRows));
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(sbase + (uint32_t)(i * kReqRows), &terms, v_full, (i >> 1) * 192 + (i & 1) * 64, s.u * kReqTile);
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      };
      const int v_at = min(waited ? 1 : p.stages, s.count_c - 1);
      for (int c = 0; c < s.count_c; ++c) {
        if (c == v_at) load_v();
        if (!ok) break;
        if (lane == 0) {
          ok = mbar_wait_bounded(ring.empty_bar(), ring.phase ^ 1u, abort_flag);
          if (ok) mbar_arrive_expect_tx(ring.full_bar(), bytes);
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!ok) break;
        const uint32_t st = stage0 + (uint32_t)(ring.at * p.stage_bytes);
        const int x = (s.c + c) * 64;
        if (p.base) load_rows(st, &box, &row, ring.full_bar(), x, r, lane, count);
        if (lane < r16 / 16)
          tma_load_2d(st + kReqRows + (uint32_t)lane * 2048u, &weight, ring.full_bar(), x, s.ad.first + 16 * lane);
        ring.next();
        ++issued;
      }
      ++pieces;
    }
    if (!waited) griddep_wait();
    if (*abort_flag && lane == 0) {
      // copies in flight: the last piece's V may or may not have been asked for
      for (int i = 0; i < min(issued, p.stages); ++i) {
        const int last = (issued - 1 - i) / p.stages;
        mbar_wait_bounded(ring.full + 8u * i, (uint32_t)(last & 1), nullptr);
      }
      if (pieces > 0) mbar_wait_bounded(v_full, (uint32_t)((pieces - 1) & 1), nullptr);
    }
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_bf16_f32(128, 64, 0, 1);
    const uint64_t v0 = smem_desc_sw128(sbase, 16, 1024), w0 = smem_desc_sw128(stage0 + kReqRows, 8192, 1024);
    bool ok = true;
    int n = 0, pieces = 0;
    while (ok && expand_piece(p, s)) {
      if (s.ad.rank == 0) continue;
      const int r16 = (s.ad.rank + 15) & ~15;
      ok = mbar_wait_bounded(v_full, (uint32_t)(pieces & 1), abort_flag);
      ++pieces;
      for (int c = 0; c < s.count_c && ok; ++c, ++n) {
        const int buf = n & 1;
        ok = mbar_wait_bounded(acc_empty + 8u * buf, (uint32_t)(((n >> 1) & 1) ^ 1), abort_flag) &&
             mbar_wait_bounded(ring.full_bar(), ring.phase, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * 64);
        const uint64_t w = w0 + ((uint32_t)(ring.at * p.stage_bytes) >> 4);
        uint32_t acc = 0;
        for (int j = 0; j < r16; j += 64) {
          const int ks = min(64, r16 - j) / 16;
          // hi, then mid (a box further); 16 of the rank are 32 bytes of V's rows and 16 rows of the factor
          const uint64_t v = v0 + (uint64_t)(j / 64 * (2 * kReqRows / 16)), wj = w + (uint64_t)(j * 8);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < ks) {
              umma_bf16(d, v + (uint64_t)(2 * k), wj + (uint64_t)(128 * k), idesc, acc);
              acc = 1;
              umma_bf16(d, v + (uint64_t)(kReqRows / 16 + 2 * k), wj + (uint64_t)(128 * k), idesc, 1u);
            }
        }
        if (c == s.count_c - 1) umma_commit(v_empty);
        umma_commit(acc_full + 8u * buf);
        ring.next();
      }
    }
    if (!ok && n > 0) mbar_wait_bounded(acc_full + 8u * ((n - 1) & 1), (uint32_t)(((n - 1) >> 1) & 1), nullptr);
  } else if (warp >= 2) {
    const int quarter = warp & 3, half = (warp - 2) >> 2, rowi = quarter * 32 + lane;
    bool ok = true;
    int n = 0;
    while (ok && expand_piece(p, s)) {
      const int count = s.tile.z, x0 = s.c * 64, x1 = min(p.N, x0 + s.count_c * 64);
      if (s.ad.rank == 0) {
        // no adapter: the base's rows as they are, eight 16-byte words of a lane in flight
        if (p.out == p.base) continue;
        // (the warp's rows are warp - 2 + 8 j, row j's token in lane j)
        const int rows = (count - (warp - 2) + 7) / 8, words = (x1 - x0) / 8, total = max(0, rows) * words;
        const int tok = lane < rows ? __ldcg(p.order + s.tile.y + warp - 2 + 8 * lane) : 0;
        for (int e0 = 0; e0 < total; e0 += 8 * 32) {
          uint4 v[8];
          int64_t at[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = min(e0 + 32 * i + lane, total - 1);
            at[i] = (int64_t)__shfl_sync(0xFFFFFFFFu, tok, e / words) * p.N + x0 + (e % words) * 8;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = p.base ? __ldcs(reinterpret_cast<const uint4*>(p.base + at[i])) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (e0 + 32 * i + lane < total) __stcs(reinterpret_cast<uint4*>(p.out + at[i]), v[i]);
        }
        continue;
      }
      const int tok = __ldcg(p.order + s.tile.y + min(rowi, count - 1));
      for (int c = 0; c < s.count_c; ++c, ++n) {
        const int buf = n & 1;
        ok = mbar_wait_bounded(acc_full + 8u * buf, (uint32_t)((n >> 1) & 1), abort_flag) &&
             mbar_wait_bounded(ring.full_bar(), ring.phase, abort_flag);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * 64 + half * 32), v);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + 8u * buf);
        // base + term, in place in the stage (128B-swizzled rows: conflict-free)
        uint8_t* st = smem + p.v_bytes + ring.at * p.stage_bytes;
        uint8_t* mine = st + rowi * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4* at = reinterpret_cast<uint4*>(mine + (((4 * half + i) ^ (rowi & 7)) << 4));
          uint4 b = p.base ? *at : make_uint4(0, 0, 0, 0);
          uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 o = __floats2bfloat162_rn(bf_lo(w[j]) + __uint_as_float(v[8 * i + 2 * j]),
                                                           bf_hi(w[j]) + __uint_as_float(v[8 * i + 2 * j + 1]));
            w[j] = *reinterpret_cast<const uint32_t*>(&o);
          }
          *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        // this warp's 32 rows x 64 bytes, eight rows at a time
        const int piece = 4 * half + (lane & 3), x = x0 + c * 64 + piece * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = quarter * 32 + i * 8 + lane / 4;
          const int64_t t = __shfl_sync(0xFFFFFFFFu, tok, i * 8 + lane / 4);
          if (r < count && x < x1)
            __stcs(reinterpret_cast<uint4*>(p.out + t * p.N + x),
                   *reinterpret_cast<const uint4*>(st + r * 128 + ((piece ^ (r & 7)) << 4)));
        }
        fence_proxy_async_smem();                // the next copy into this stage comes by TMA
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.empty_bar());
        ring.next();
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 128);
}

// ----------------------------------------------------------------------- grads
struct GradArgs {
  const int32_t* order;
  const int32_t* seg;
  const int32_t* tile_first;
  PoolArgs pool;
  int cols[2], blocks[2];       // columns of the two factors, and their blocks of 256
  float* dW[2];
  float* part;                  // [CTA][2][64 or width][256]: sums of units that CTAs share
  int4* cut;                    // [CTA]: {factor, row, column, rank | CTAs that go on << 16} of its last unit, if that is cut
  int width, stages, stage_bytes, tmem_cols;
};
constexpr int kGradCols = 256;
constexpr int kReqGradThreads = 320;            // warps 2-9: epilogue, one per 128 columns and quarter of their rows

// A unit is one adapter, 64 of its rank and 256 columns of one factor; its work
// is one step per 64 tokens (an adapter without tokens: one step that only
// writes zeros).  The steps of all units, unit by unit, are cut into equal
// parts, one per CTA, whatever the adapters' lengths are.  A CTA that has all
// steps of a unit writes its gradient; the sums of a unit that is cut go to
// the workspace (slot 0: the unit began in an earlier CTA, slot 1: it goes on in
// a later one), and requests_grads_join_kernel adds them in order.
struct GradUnit {
  int a, unit, units;           // adapter; block + per * (64 of the rank); how many it has
  int steps, lo, cnt;           // steps of a unit; the adapter's tokens in `order`
  AdapterRows ad;
};
__device__ __forceinline__ int grad_per(const GradArgs& p) { return p.blocks[0] + p.blocks[1]; }
__device__ __forceinline__ void grad_adapter(const GradArgs& p, GradUnit& g, int a) {
  g.a = a;
  g.ad = adapter_rows(p.pool, a, p.width);
  g.lo = p.seg[a];
  g.cnt = p.seg[a + 1] - g.lo;
  g.units = (g.ad.rank + 63) / 64 * grad_per(p);
  g.steps = max(1, (g.cnt + 63) / 64);
}
__device__ __forceinline__ void grad_next_unit(const GradArgs& p, GradUnit& g) {
  if (++g.unit < g.units) return;
  g.unit = 0;
  int a = g.a;
  do grad_adapter(p, g, ++a);
  while (g.units == 0);         // never past the last: the caller knows that steps are left
}
// Where part `part` of the steps begins: step `at` of all `total`, in adapter a,
// whose first step is `base`.  As many parts as there are CTAs, or steps if
// these are fewer.  The whole block calls it.
struct GradScan {
  long long warp[32];
  long long at, base, total;
  int a, parts;
};
__device__ __forceinline__ void grad_locate(const GradArgs& p, GradScan& s, int part, int parts) {
  const int per = (p.pool.n + blockDim.x - 1) / blockDim.x;
  const int a0 = min(p.pool.n, (int)threadIdx.x * per), a1 = min(p.pool.n, a0 + per);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long sum = 0;
  for (int a = a0; a < a1; ++a) {
    GradUnit g;
    grad_adapter(p, g, a);
    sum += (long long)g.units * g.steps;
  }
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) s.warp[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) {
    if (w < warp) before += s.warp[w];
    total += s.warp[w];
  }
  long long base = before + inc - sum;
  parts = (int)min((long long)parts, max(1ll, total));
  const long long at = part < parts ? total * part / parts : total;
  if (at >= base && at < base + sum) {
    for (int a = a0; a < a1; ++a) {
      GradUnit g;
      grad_adapter(p, g, a);
      const long long w = (long long)g.units * g.steps;
      if (at < base + w) {
        s.a = a;
        s.base = base;
        break;
      }
      base += w;
    }
  }
  if (threadIdx.x == 0) {
    s.at = at;
    s.total = total;
    s.parts = parts;
  }
  __syncthreads();
}
struct GradPlace {
  int z, c0, cols, rc0, rc;
};
__device__ __forceinline__ GradPlace grad_place(const GradArgs& p, const GradUnit& g) {
  GradPlace w;
  const int per = grad_per(p), block = g.unit % per;
  w.rc0 = g.unit / per * 64;
  w.z = block >= p.blocks[0] ? 1 : 0;
  w.cols = w.z ? p.cols[1] : p.cols[0];
  w.c0 = (w.z ? block - p.blocks[0] : block) * kGradCols;
  w.rc = min(64, ((g.ad.rank + 15) & ~15) - w.rc0);
  return w;
}

// D[column][hi .. 64 | mid | lo] (A operand: token rows, MN-major; B operand: V,
// MN-major): one MMA takes the three parts of V, so the token rows are read
// from shared memory once.  The 256 columns are two accumulators; two steps
// (128 tokens) go into the first, then into the second, and while one fills the
// epilogue warps move the other to registers.  (With the parts in MMAs of their
// own and the accumulators changing by step, operand reads beside the arriving
// loads made a step 2,180 cycles.)  Measured (alone, between
// two events, L2 flushed): both factors' gradients 257 us at 16384 tokens of rank 64, 8192
// and 22016 columns (3.9 TB/s of token rows, and V's rows, as many bytes again, from L2:
// what bounds it), 32 us at 4096 tokens, 4096 columns.
template <int NI>                                // 16 of the rank each: 1 or 4
__global__ void __launch_bounds__(kReqGradThreads, NI == 1 ? 2 : 1) requests_grads_kernel(
    const __grid_constant__ CUtensorMap box0, const __grid_constant__ CUtensorMap row0, const __grid_constant__ CUtensorMap terms0,
    const __grid_constant__ CUtensorMap box1, const __grid_constant__ CUtensorMap row1, const __grid_constant__ CUtensorMap terms1,
    const __grid_constant__ GradArgs p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[2 * 8 + 4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ GradScan s_scan;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &s_abort;

  Ring ring;
  ring.full = smem_u32(&s_bar[0]);
  ring.empty = smem_u32(&s_bar[8]);
  ring.stages = p.stages;
  // by half of the columns; Tensor Memory likewise
  const uint32_t acc_full = smem_u32(&s_bar[16]), acc_empty = smem_u32(&s_bar[18]);
  const uint32_t half_cols = 64u + 2u * (uint32_t)min(64, p.width);
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(ring.full + 8u * i, 1);
      mbar_init(ring.empty + 8u * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8u * i, 1);
      mbar_init(acc_empty + 8u * i, 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), (uint32_t)p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();
  const uint32_t tmem = s_tmem;
  griddep_wait();
  grad_locate(p, s_scan, (int)blockIdx.x, (int)gridDim.x);
  const long long at = s_scan.at, total = s_scan.total;
  const int parts = s_scan.parts;
  const long long left0 = (int)blockIdx.x < parts ? total * (blockIdx.x + 1) / parts - at : 0;
  if (threadIdx.x == 0) p.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (left0 <= 0) {
    if (warp == 1) tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
    return;
  }
  GradUnit g;
  grad_adapter(p, g, s_scan.a);
  g.unit = (int)((at - s_scan.base) / g.steps);
  int step0 = (int)((at - s_scan.base) % g.steps);
  long long left = left0;

  if (warp == 0) {
    const int i = lane & 15;                     // four token rows of 64
    int issued = 0, ok = 1;
    while (left > 0 && ok) {
      const GradPlace w = grad_place(p, g);
      const int step1 = (int)min((long long)g.steps, step0 + left);
      const CUtensorMap* box = w.z ? &box1 : &box0;
      const CUtensorMap* rowm = w.z ? &row1 : &row0;
      const CUtensorMap* terms = w.z ? &terms1 : &terms0;
      const int blocks64 = min(4, (w.cols - w.c0 + 63) / 64);       // (an unloaded last block is never stored)
      const int vboxes = 1 + (2 * w.rc + 63) / 64;
      const int vrow0 = p.tile_first[g.a] * kReqTile;
      RowLane ahead;                             // the next step's tokens, on their way while this one waits
      if (g.cnt > 0) row_tokens(ahead, p.order, g.lo + step0 * 64, min(64, g.cnt - step0 * 64), i);
      for (int s = step0; s < step1 && g.cnt > 0; ++s) {
        const int first = s * 64;
        const int m = min(64, g.cnt - first);
        RowLane r = ahead;
        if (s + 1 < step1) row_tokens(ahead, p.order, g.lo + first + 64, min(64, g.cnt - first - 64), i);
        row_whole(r, m, i);
        if (lane == 0) {
          ok = mbar_wait_bounded(ring.empty_bar(), ring.phase ^ 1u, abort_flag);
          if (ok) mbar_arrive_expect_tx(ring.full_bar(), row_bytes(m) * blocks64 + (uint32_t)vboxes * 8192u);
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!ok) break;
        const uint32_t st = sbase + (uint32_t)(ring.at * p.stage_bytes);
        for (int c = lane >> 4; c < blocks64; c += 2)
          load_rows(st + (uint32_t)c * 8192u, box, rowm, ring.full_bar(), w.c0 + c * 64, r, i, m);
        if (lane < vboxes)
          tma_load_2d(st + 4u * 8192u + (uint32_t)lane * 8192u, terms, ring.full_bar(), w.rc0 * 3 + 64 * lane, vrow0 + first);
        ring.next();
        ++issued;
      }
      left -= step1 - step0;
      step0 = 0;
      if (left > 0) grad_next_unit(p, g);
    }
    if (*abort_flag && lane == 0) {
      for (int k = 0; k < min(issued, p.stages); ++k) {
        const int last = (issued - 1 - k) / p.stages;
        mbar_wait_bounded(ring.full + 8u * k, (uint32_t)(last & 1), nullptr);
      }
    }
  } else if (warp == 1 && lane == 0) {
    // descriptors of stage 0: one thread issues, so an address costs it an addition
    const uint64_t xd0 = smem_desc_sw128(sbase, 8192, 1024), vd0 = smem_desc_sw128(sbase + 4u * 8192u, 8192, 1024);
    bool ok = true;
    int n[2] = {0, 0};                           // times that an accumulator was filled
    while (left > 0 && ok) {
      const GradPlace w = grad_place(p, g);
      const int step1 = (int)min((long long)g.steps, step0 + left);
      const int halves = w.cols - w.c0 > 128 ? 2 : 1;               // 128-column MMAs in use
      const uint32_t idesc = idesc_bf16_f32(128, 64 + 2 * w.rc, 1, 1);
      for (int s = step0; s < step1 && g.cnt > 0 && ok; s += 2) {
        const int two = min(2, step1 - s);
        const int stage[2] = {ring.at, ring.at + 1 == p.stages ? 0 : ring.at + 1};
        const uint32_t phase[2] = {ring.phase, ring.at + 1 == p.stages ? ring.phase ^ 1u : ring.phase};
        for (int h = 0; h < halves && ok; ++h) {
          ok = mbar_wait_bounded(acc_empty + 8u * h, (uint32_t)((n[h] & 1) ^ 1), abort_flag);
          for (int i = 0; i < two && ok; ++i) {
            if (h == 0) ok = mbar_wait_bounded(ring.full + 8u * stage[i], phase[i], abort_flag);
            if (!ok) break;
            tc_fence_after();
            const int ks = (min(64, g.cnt - (s + i) * 64) + 15) / 16;
            const uint32_t off = (uint32_t)(stage[i] * p.stage_bytes) >> 4;
            const uint64_t xd = xd0 + off + (uint64_t)(h * 1024), vd = vd0 + off;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < ks) umma_bf16(tmem + (uint32_t)h * half_cols, xd + (uint64_t)(k * 128), vd + (uint64_t)(k * 128), idesc, (i | k) ? 1u : 0u);
            if (h == halves - 1) umma_commit(ring.empty + 8u * stage[i]);
          }
          if (ok) {
            umma_commit(acc_full + 8u * h);
            ++n[h];
          }
        }
        ring.next();
        if (two == 2) ring.next();
      }
      left -= step1 - step0;
      step0 = 0;
      if (left > 0 && ok) grad_next_unit(p, g);
    }
    if (!ok) {
      // MMAs already issued, before Tensor Memory is released
      umma_commit(acc_full);
      mbar_wait_bounded(acc_full, (uint32_t)(n[0] & 1), nullptr);
    }
  } else if (warp >= 2) {
    const int quarter = warp & 3, h = (warp - 2) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    bool ok = true;
    int n = 0;
    while (left > 0 && ok) {
      const GradPlace w = grad_place(p, g);
      const int step1 = (int)min((long long)g.steps, step0 + left);
      const bool mine = h * 128 < w.cols - w.c0;
      float acc[NI][16];
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] = 0.f;
      for (int s = step0; s < step1 && g.cnt > 0 && mine; s += 2, ++n) {
        ok = mbar_wait_bounded(acc_full + 8u * h, (uint32_t)(n & 1), abort_flag);
        __syncwarp();
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (16 * i >= w.rc) break;
          uint32_t v[3][16];
          const uint32_t t = lanes + (uint32_t)h * half_cols + 16u * i;
          tmem_ld_32x32b_x16(t, v[0]);
          tmem_ld_32x32b_x16(t + 64u, v[1]);
          tmem_ld_32x32b_x16(t + 64u + (uint32_t)w.rc, v[2]);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            acc[i][j] += __uint_as_float(v[0][j]) + (__uint_as_float(v[1][j]) + __uint_as_float(v[2][j]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + 8u * h);
      }
      if (ok) {
        const bool whole = step0 == 0 && step1 == g.steps;
        float* out;
        int64_t ld;
        if (whole) {
          ld = w.cols;
          out = (w.z ? p.dW[1] : p.dW[0]) + (int64_t)(g.ad.first + w.rc0) * ld + w.c0;
        } else {
          ld = kGradCols;
          out = p.part + ((int64_t)blockIdx.x * 2 + (step0 > 0 ? 0 : 1)) * (int64_t)min(64, p.width) * kGradCols;
          if (step0 == 0 && warp == 2 && lane == 0) {
            // the CTAs behind this one that have a part of the unit
            const long long end = total * (blockIdx.x + 1) / parts + g.steps - step1;
            int more = 0;
            for (int k = blockIdx.x + 1; k < parts && total * k / parts < end; ++k) ++more;
            p.cut[blockIdx.x] = make_int4(w.z, g.ad.first + w.rc0, w.c0, w.rc | more << 16);
          }
        }
        // rows behind the rank are zero, also where a token holds an infinity
        const int c = h * 128 + quarter * 32 + lane, live = g.ad.rank - w.rc0;
        if (w.c0 + c < w.cols)
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if (16 * i < w.rc)
#pragma unroll
              for (int j = 0; j < 16; ++j) out[(int64_t)(16 * i + j) * ld + c] = 16 * i + j < live ? acc[i][j] : 0.f;
      }
      left -= step1 - step0;
      step0 = 0;
      if (left > 0 && ok) grad_next_unit(p, g);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
}

// Adds the parts of the unit that CTA blockIdx.x began and others went on with;
// blockIdx.y takes a quarter of the rows.  Latency: 9.6 us alone
// between two events, L2 flushed, some 4 us in the chain.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) requests_grads_join_kernel(const GradArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  const int4 cut = p.cut[blockIdx.x];
  const int rc = cut.w & 0xFFFF, more = cut.w >> 16;
  if (rc == 0) return;
  const int cols = cut.x ? p.cols[1] : p.cols[0];
  const int64_t slot = (int64_t)min(64, p.width) * kGradCols;
  float* out = (cut.x ? p.dW[1] : p.dW[0]) + (int64_t)cut.y * cols + cut.z;
  const int rows = rc / 4;
  for (int e = threadIdx.x; e < rows * (kGradCols / 4); e += kJoinThreads) {
    const int j = blockIdx.y * rows + e / (kGradCols / 4), c = (e % (kGradCols / 4)) * 4;
    if (cut.z + c >= cols) continue;
    const float* in = p.part + (int64_t)blockIdx.x * 2 * slot + (int64_t)j * kGradCols + c;
    float4 v = *reinterpret_cast<const float4*>(in + slot);
    for (int k = 1; k <= more; ++k) {
      const float4 f = *reinterpret_cast<const float4*>(in + (int64_t)k * 2 * slot);
      v.x += f.x; v.y += f.y; v.z += f.z; v.w += f.w;
    }
    *reinterpret_cast<float4*>(out + (int64_t)j * cols + c) = v;
  }
}

}  // namespace qlora

// Many adapters at once beside a shared projection: the maps of a batch, and
// the kernels for few tokens.
//
// [P2] "The LoRA hypothesis": serving many tasks keeps the adapters unmerged,
// one base in memory and a small adapter chosen per request.  A batch is a
// row of requests; request i owns lens[i] consecutive tokens and one adapter
// (or none).  The adapters of one linear live in a pool of rows: adapter a
// owns rows first[a] .. first[a] + rank[a] of A (rows x k) and of B
// transposed (rows x d).  With B transposed the forward and the backward are
// the same two products with A and Bt exchanged:
//   U = X A_a^T,   Y  = base + s_a U Bt_a
//   G = dY Bt_a^T, dX = base + s_a G A_a,   dA_a = s_a G^T X, dBt_a = s_a U^T dY.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace qlora {

// ------------------------------------------------------------------- the maps
// starts, idx, order, seg as documented in qlora.h, and the work list of the
// kernels below: groups 0 .. n-1 are the adapters, group n the tokens without
// one; tile_first[g] (n + 2 entries) is the first tile of group g, and tile u
// is {group, first position in order, tokens, 0}; unused tiles hold 0 tokens.
constexpr int kReqMax = 4096;        // requests, and adapters, of one batch
constexpr int kPlanThreads = 256;

struct PlanArgs {
  const int32_t* lens;
  const int32_t* ids;
  int n_req, n, T;
  int tile, max_tiles, slice;
  int32_t* starts;
  int32_t* idx;
  int32_t* order;
  int32_t* seg;
  int32_t* tile_first;
  int4* tiles;
};

__host__ __device__ __forceinline__ size_t plan_smem_bytes(int n_req, int n) {
  return (size_t)4 * (3 * (n_req + 1) + 2 * (n + 2));
}

// Exclusive sum of one value per thread over the block, and the block's total.
template <typename V>
__device__ __forceinline__ V block_exclusive(V v, V* s_warp, V& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();                       // s_warp may still be read from the last call
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  V before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  return before + inc - v;
}

// Largest i in [0, count) with v[i] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int last_not_above(const int* v, int count, int x) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Every block scans the requests for itself (a few thousand at most, read
// from L2) and then writes its own slice of the tokens and of the tiles, so
// nothing is exchanged between blocks and one launch does it all.  Where a
// request's tokens land in `order` needs the tokens of earlier requests with
// the same adapter: a warp sums them straight from shared memory, only for
// the requests of its slice.  Bound by latency, two dependent scans: in a chain
// of launches 4.4 us for 64 requests of one token, 5.1 us for 300 requests of
// 16384 tokens (8.4 and 9.2 us alone between two events, L2 flushed).
__global__ void __launch_bounds__(kPlanThreads) requests_plan_kernel(const PlanArgs p) {
  extern __shared__ int32_t s_mem[];
  __shared__ long long s_warp64[kPlanThreads / 32];
  __shared__ int s_warp[kPlanThreads / 32];
  int* s_start = s_mem;                          // n_req + 1
  int* s_id = s_start + p.n_req + 1;             // n_req + 1
  int* s_pos = s_id + p.n_req + 1;               // n_req + 1
  int* s_seg = s_pos + p.n_req + 1;              // n + 2
  int* s_tile = s_seg + p.n + 2;                 // n + 2
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  for (int i = tid; i < p.n_req; i += kPlanThreads) {
    s_start[i] = max(0, p.lens[i]);
    const int a = p.ids[i];
    s_id[i] = (a >= 0 && a < p.n) ? a : p.n;
  }
  for (int g = tid; g < p.n + 2; g += kPlanThreads) s_seg[g] = 0;
  __syncthreads();

  // first rows: a 64-bit sum, cut at T, so that no lengths can overflow it
  {
    const int per = (p.n_req + kPlanThreads - 1) / kPlanThreads;
    const int i0 = min(p.n_req, tid * per), i1 = min(p.n_req, i0 + per);
    long long sum = 0;
    for (int i = i0; i < i1; ++i) sum += s_start[i];
    long long total;
    long long run = block_exclusive<long long>(sum, s_warp64, total);
    for (int i = i0; i < i1; ++i) {
      const int len = s_start[i];
      s_start[i] = (int)min(run, (long long)p.T);
      run += len;
    }
    if (tid == 0) s_start[p.n_req] = (int)min(total, (long long)p.T);
  }
  __syncthreads();
  // tokens of each group (integer sums: their order does not matter)
  for (int i = tid; i < p.n_req; i += kPlanThreads) {
    const int len = s_start[i + 1] - s_start[i];
    if (len > 0) atomicAdd(&s_seg[s_id[i]], len);
  }
  __syncthreads();
  {
    const int per = (p.n + 2 + kPlanThreads - 1) / kPlanThreads;
    const int g0 = min(p.n + 2, tid * per), g1 = min(p.n + 2, g0 + per);
    int sum = 0, tiles = 0;
    for (int g = g0; g < g1; ++g) {
      sum += s_seg[g];
      tiles += (s_seg[g] + p.tile - 1) / p.tile;
    }
    int total;
    int run = block_exclusive<int>(sum, s_warp, total);
    int trun = block_exclusive<int>(tiles, s_warp, total);
    for (int g = g0; g < g1; ++g) {
      const int c = s_seg[g];
      s_seg[g] = run;
      s_tile[g] = trun;
      run += c;
      trun += (c + p.tile - 1) / p.tile;
    }
  }
  __syncthreads();
  const int total = s_start[p.n_req];

  if (blockIdx.x == 0) {
    for (int i = tid; i <= p.n_req; i += kPlanThreads) p.starts[i] = s_start[i];
    for (int g = tid; g < p.n + 2; g += kPlanThreads) {
      p.seg[g] = s_seg[g];                       // entry n + 1 is the group behind the last: the total
      p.tile_first[g] = s_tile[g];
    }
  }
  for (int u = blockIdx.x * kPlanThreads + tid; u < p.max_tiles; u += gridDim.x * kPlanThreads) {
    int4 t = make_int4(-1, 0, 0, 0);
    if (u < s_tile[p.n + 1]) {
      const int g = last_not_above(s_tile, p.n + 1, u);
      const int at = s_seg[g] + (u - s_tile[g]) * p.tile;
      t = make_int4(g < p.n ? g : -1, at, min(p.tile, s_seg[g + 1] - at), 0);
    }
    p.tiles[u] = t;
  }

  const int t0 = blockIdx.x * p.slice, t1 = min(p.T, t0 + p.slice);
  if (t0 >= t1) return;
  if (t0 < total) {
    const int lo = last_not_above(s_start, p.n_req, t0);
    const int hi = last_not_above(s_start, p.n_req, min(t1, total) - 1);
    for (int i = lo + (tid >> 5); i <= hi; i += kPlanThreads / 32) {
      if (s_start[i + 1] == s_start[i]) continue;
      const int id = s_id[i];
      int before = 0;
      for (int j = tid & 31; j < i; j += 32)
        if (s_id[j] == id) before += s_start[j + 1] - s_start[j];
      before = __reduce_add_sync(0xFFFFFFFFu, before);
      if ((tid & 31) == 0) s_pos[i] = s_seg[id] + before;
    }
  }
  __syncthreads();
  for (int t = t0 + tid; t < t1; t += kPlanThreads) {
    int a = -1;
    if (t < total) {
      const int i = last_not_above(s_start, p.n_req, t);
      if (s_id[i] < p.n) a = s_id[i];
      p.order[s_pos[i] + (t - s_start[i])] = t;
    } else {
      p.order[t] = -1;
    }
    p.idx[t] = a;
  }
}

// ----------------------------------------------------------------- the adapters
struct PoolArgs {
  const int32_t* first;
  const int32_t* rank;
  const float* scale;
  int n, rows;
};

struct AdapterRows {
  int first, rank;
  float scale;
};
// Adapter a's rows; an entry that does not lie within the pool counts as rank
// 0 (no term), so no table can make a kernel read outside the pool.
__device__ __forceinline__ AdapterRows adapter_rows(const PoolArgs& p, int a, int width) {
  AdapterRows r{0, 0, 0.f};
  if (a < 0 || a >= p.n) return r;
  const int f = __ldcg(p.first + a), k = __ldcg(p.rank + a);
  const float scale = __ldcg(p.scale + a);       // (with the others, not behind them)
  if (f < 0 || k < 1 || k > width || f > p.rows - ((k + 15) & ~15)) return r;
  r.first = f;
  r.rank = k;
  r.scale = scale;
  return r;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// ------------------------------------------------------------------ few tokens
// Tiles of up to 8 tokens of one adapter.  A cluster of CTAs takes one tile:
// each CTA sums U over its share of the K columns and sends the sums to every
// CTA of the cluster, which adds them in rank order and writes its share of the
// N output columns.  (The sums travel as asynchronous stores that count down
// the receiver's barrier: no cluster-wide fence, 0.9 us less than a cluster
// barrier and remote loads.)  One launch, the factors read once.
//
// The factors are what has to be read (a few tokens' X is nothing), so a
// producer thread streams this CTA's part of both through a ring of TMA boxes,
// 16 rows x 256 columns a stage: 40 KB are in flight per CTA from the first
// moment, and the second factor arrives while the cluster still adds up U.
// What is left is the time a stage takes the warps, so the products go through
// m16n8k16 tensor instructions with the factor's rows (U) or columns (output)
// as M and the tokens as N = 8: a tenth of the instructions of multiply-adds,
// too small a product for tcgen05's 128 rows.  Measured: 12.2 us in
// a chain, 20.5 us alone with L2 flushed, for 64 tokens of 48 adapters, 4096 x 4096; 3.3
// us in a chain for 16 tokens, 256 x 256.  Of 9.5 us for 16 adapters of rank 64, 4.9
// are the launch, the exchange and the output rows, 2.5 the ring's barriers, 1.8 the
// products and 0.3 the loads.  The tensor core cuts what it adds up, so U leaves
// the accumulator every 32 columns and is summed in registers, rounded to nearest:
// in one accumulator, sums of one sign over 65536 columns were 2.5e-5 off, all
// towards zero; now 1.4e-7 at worst and 2e-9 in the mean, at the same speed.  For the
// output, U enters as two bf16 terms (2^-16, far below the one rounding of the bf16 output).
constexpr int kFewTile = 8;
constexpr int kFewWarps = 8;                   // consumers; one more warp produces
constexpr int kFewThreads = 32 * (kFewWarps + 1);
constexpr int kFewRows = 16;                   // rows of a stage
constexpr int kFewCols = 256;                  // columns of a stage, 32 per warp
constexpr int kFewStages = 5;
constexpr int kFewStageBytes = kFewRows * kFewCols * 2;
constexpr int kFewGroup = 32;                  // rows of U whose sums are exchanged at once

struct FewArgs {
  const uint16_t* X;       // T x K
  const uint16_t* base;    // T x N, or null (zero)
  uint16_t* out;           // T x N
  float* U;                // T x width: U of each token (zeros beyond its rank), or null
  float* sU;               // the same times the adapter's scale, or null
  int K, N, width, csize;
  const int32_t* order;
  const int4* tiles;
  PoolArgs pool;
};

struct alignas(128) FewShared {
  // [4 blocks of 64 columns][2 x 8 rows][128 bytes], 128B-swizzled
  uint8_t ring[kFewStages * kFewStageBytes];
  float red[kFewWarps * kFewGroup * kFewTile];   // [warp][row][token]; later [warp][token][32 columns]
  uint64_t full[kFewStages], empty[kFewStages], ready;
  int abort_flag, unused[3];
  // behind it, by the pool's width: what the cluster's CTAs sent, float
  // part[CTA][row][token], then scaled U as bf16 [hi, mid][token][width + 8]
  __device__ __forceinline__ float* part() { return reinterpret_cast<float*>(this + 1); }
  __device__ __forceinline__ uint16_t* u(int width, int csize) {
    return reinterpret_cast<uint16_t*>(part() + csize * width * kFewTile);
  }
};
__host__ __device__ __forceinline__ size_t few_smem_bytes(int width, int csize) {
  return 1024 + sizeof(FewShared) + (size_t)csize * kFewTile * width * 4 + (size_t)2 * kFewTile * (width + 8) * 2;
}

// Four floats to shared memory of another CTA of the cluster, counted on its barrier.
__device__ __forceinline__ void store_async4(uint32_t cluster_addr, float4 v, uint32_t cluster_bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                   cluster_addr),
               "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)), "r"(__float_as_uint(v.w)),
               "r"(cluster_bar)
               : "memory");
}
// d += A (16 x 16) B (16 x 8), bf16 in, fp32 out.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}

static_assert(sizeof(FewShared) % 128 == 0, "what lies behind it is read in 16-byte words");

struct FewRing {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == kFewStages) {
      at = 0;
      phase ^= 1u;
    }
  }
};

// Stages of one factor for this CTA (one warp): for the first factor all
// columns of 16 rows, then the next rows; for the second all rows of 256
// columns.  Boxes of 64 columns x 16 rows, or 8 where the rank ends in a
// stage's first 8; columns only up to the share's end.  A lane issues one box:
// with one lane for all four, and its position by division, issuing took longer
// than the warps' products.
__device__ __forceinline__ bool few_produce(FewShared& s, FewRing& ring, int& issued, const CUtensorMap* w8,
                                            const CUtensorMap* w16, int first, int rank, int c0, int c1, bool rows_first) {
  const int lane = threadIdx.x & 31;
  int r = 0, c = c0;
  while (r < rank && c < c1) {
    const bool two = rank - r > 8;
    const int blocks = min(4, (c1 - c + 63) / 64);
    const uint32_t full = smem_u32(&s.full[ring.at]);
    const bool ok = mbar_wait_bounded(smem_u32(&s.empty[ring.at]), ring.phase ^ 1u, &s.abort_flag);
    if (!__all_sync(0xFFFFFFFFu, ok)) return false;
    if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(blocks * (two ? 2048 : 1024)));
    if (lane < blocks)
      tma_load_2d(smem_u32(s.ring) + (uint32_t)(ring.at * kFewStageBytes + lane * 2048), two ? w16 : w8, full, c + 64 * lane,
                  first + r);
    __syncwarp();
    ring.next();
    ++issued;
    if (rows_first) {
      r += kFewRows;
      if (r >= rank) r = 0, c += kFewCols;
    } else {
      c += kFewCols;
      if (c >= c1) c = c0, r += kFewRows;
    }
  }
  return true;
}

// The consumers' side of a tile (warps 0 .. 7).  X's values stay in L1.
__device__ __forceinline__ void few_consume(const FewArgs& p, FewShared& s, const AdapterRows& ad, const int4& tile, int count,
                                            int q, int k0, int k1, int n0, int n1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hi = lane >> 2, lo = lane & 3;
  float* s_part = s.part();
  uint16_t* s_u = s.u(p.width, p.csize);
  const int upitch = p.width + 8;                // bf16 values; rows of U in distinct banks
  const int quads = count <= 4 ? 1 : 2;          // fours of tokens in use
  if (p.csize > 1 && threadIdx.x == 0)
    mbar_arrive_expect_tx(smem_u32(&s.ready), (uint32_t)((p.csize - 1) * ad.rank * quads * 16));
  const int tokn = p.order[tile.y + min(hi, count - 1)];      // the token of this lane's column
  const uint16_t* xrow = p.X + (int64_t)tokn * p.K;
  FewRing ring;
  bool ok = true;
  // U: a warp takes 32 columns of a stage; a lane's 8 consecutive columns are
  // the 4 values of two k-steps (any order of the columns gives the same sum)
  const uint32_t a_off = (uint32_t)((warp >> 1) * 2048 + hi * 128 + ((((warp & 1) * 4 + lo) ^ hi) << 4));
  for (int g = 0; g < ad.rank; g += kFewGroup) {
    for (int r = g; r < min(ad.rank, g + kFewGroup) && ok; r += kFewRows) {
      const bool two = ad.rank - r > 8;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int c = k0; c < k1; c += kFewCols) {
        const int x0 = c + warp * 32 + lo * 8;
        const uint4 x = x0 < k1 ? __ldg(reinterpret_cast<const uint4*>(xrow + x0)) : make_uint4(0, 0, 0, 0);
        ok = mbar_wait_bounded(smem_u32(&s.full[ring.at]), ring.phase, &s.abort_flag);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        if (c + (warp >> 1) * 64 < k1) {         // (a block behind the share's end is not loaded)
          const uint8_t* st = s.ring + ring.at * kFewStageBytes + a_off;
          const uint4 w0 = *reinterpret_cast<const uint4*>(st);
          const uint4 w1 = two ? *reinterpret_cast<const uint4*>(st + 1024) : make_uint4(0, 0, 0, 0);
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          mma16816(acc, w0.x, w1.x, w0.y, w1.y, x.x, x.y);
          mma16816(acc, w0.z, w1.z, w0.w, w1.w, x.z, x.w);
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[j] += acc[j];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.empty[ring.at]));
        ring.next();
      }
      float* red = s.red + (warp * kFewGroup + (r - g) + hi) * kFewTile + 2 * lo;
      *reinterpret_cast<float2*>(red) = make_float2(sum[0], sum[1]);
      *reinterpret_cast<float2*>(red + 8 * kFewTile) = make_float2(sum[2], sum[3]);
    }
    named_bar_sync(1, 32 * kFewWarps);
    // the warps' sums of four tokens of a row, added in order, to every CTA
    const int rows = min(kFewGroup, ad.rank - g);
    if ((int)threadIdx.x < rows * quads) {
      const int i = threadIdx.x / quads, t = threadIdx.x % quads * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const float4 f = *reinterpret_cast<const float4*>(s.red + (w * kFewGroup + i) * kFewTile + t);
        v.x += f.x; v.y += f.y; v.z += f.z; v.w += f.w;
      }
      float* at = s_part + (q * p.width + g + i) * kFewTile + t;
      *reinterpret_cast<float4*>(at) = v;
      const uint32_t a = smem_u32(at), bar = smem_u32(&s.ready);
      for (int c = 1; c < p.csize; ++c) {
        const uint32_t to = (uint32_t)((q + c) & (p.csize - 1));
        store_async4(mapa_shared(a, to), v, mapa_shared(bar, to));
      }
    }
    named_bar_sync(1, 32 * kFewWarps);
  }
  // base comes in while the cluster's sums do: lane: token pair half, 2 columns
  const int th = lane >> 4, x2 = warp * 32 + (lane & 15) * 2;
  int tokb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) tokb[i] = __shfl_sync(0xFFFFFFFFu, tokn, (2 * i + th) * 4);
  uint32_t ahead[4];                             // base's values of the next 256 columns
  auto load_base = [&](int c) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ahead[i] = p.base && 2 * i + th < count && c + x2 < n1
                     ? *reinterpret_cast<const uint32_t*>(p.base + (int64_t)tokb[i] * p.N + c + x2) : 0u;
  };
  load_base(n0);
  // (acquire at cluster scope: the sums read below were written by the other CTAs)
  if (p.csize > 1) ok = mbar_wait_bounded<true>(smem_u32(&s.ready), 0, &s.abort_flag) && ok;
  __syncwarp();
  ok = __all_sync(0xFFFFFFFFu, ok);
  const int r16 = (ad.rank + 15) & ~15;
  for (int e = threadIdx.x; e < r16 * kFewTile; e += 32 * kFewWarps) {
    const int r = e / kFewTile, t = e % kFewTile;
    float v = 0.f;                               // rows behind the rank and tokens behind the tile's count for nothing
    if (r < ad.rank && t < count) {
#pragma unroll 8
      for (int c = 0; c < p.csize; ++c) v += s_part[(c * p.width + r) * kFewTile + t];
      if (q == 0) {
        const int64_t at = (int64_t)p.order[tile.y + t] * p.width + r;
        if (p.U) p.U[at] = v;
        if (p.sU) p.sU[at] = ad.scale * v;
      }
      v *= ad.scale;
    }
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    const __nv_bfloat16 m = __float2bfloat16_rn(v - __bfloat162float(h));
    s_u[t * upitch + r] = *reinterpret_cast<const uint16_t*>(&h);
    s_u[(kFewTile + t) * upitch + r] = *reinterpret_cast<const uint16_t*>(&m);
  }
  named_bar_sync(1, 32 * kFewWarps);
  // output: a warp's 32 columns are two M of 16 (transposed fragments), the rows K
  const int lr = (lane & 7) + ((lane >> 4) << 3), lj = ((lane >> 3) & 1) * 8;   // this lane's row and column of a 16 x 16 block
  for (int c = n0; c < n1; c += kFewCols) {
    uint32_t base[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) base[i] = ahead[i];
    load_base(c + kFewCols);
    float acc[2][4] = {};
    for (int r = 0; r < ad.rank && ok; r += kFewRows) {
      ok = mbar_wait_bounded(smem_u32(&s.full[ring.at]), ring.phase, &s.abort_flag);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      if (c + (warp >> 1) * 64 < n1) {
        const bool two = ad.rank - r > 8;
        const uint16_t* u = s_u + hi * upitch + r + 2 * lo;
        const uint32_t h0 = *reinterpret_cast<const uint32_t*>(u), h1 = *reinterpret_cast<const uint32_t*>(u + 8);
        const uint32_t m0 = *reinterpret_cast<const uint32_t*>(u + kFewTile * upitch);
        const uint32_t m1 = *reinterpret_cast<const uint32_t*>(u + kFewTile * upitch + 8);
        const uint32_t st = smem_u32(s.ring) + (uint32_t)(ring.at * kFewStageBytes + (warp >> 1) * 2048 + (lr >> 3) * 1024 + (lr & 7) * 128);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t a[4];
          ldmatrix4_trans(a, st + (uint32_t)((((warp & 1) * 4 + 2 * j + (lj >> 3)) ^ (lr & 7)) << 4));
          if (!two) a[2] = a[3] = 0u;            // (rows that were not loaded)
          mma16816(acc[j], a[0], a[1], a[2], a[3], h0, h1);
          mma16816(acc[j], a[0], a[1], a[2], a[3], m0, m1);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.empty[ring.at]));
      ring.next();
    }
    // [token][column] of this warp, then rows of 64 bytes
    float* tr = s.red + warp * (kFewTile * 32);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      tr[(2 * lo) * 32 + 16 * j + hi] = acc[j][0];
      tr[(2 * lo + 1) * 32 + 16 * j + hi] = acc[j][1];
      tr[(2 * lo) * 32 + 16 * j + hi + 8] = acc[j][2];
      tr[(2 * lo + 1) * 32 + 16 * j + hi + 8] = acc[j][3];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = *reinterpret_cast<const float2*>(tr + (2 * i + th) * 32 + (lane & 15) * 2);
      if (2 * i + th < count && c + x2 < n1) {
        const __nv_bfloat162 o = __floats2bfloat162_rn(bf_lo(base[i]) + v.x, bf_hi(base[i]) + v.y);
        *reinterpret_cast<uint32_t*>(p.out + (int64_t)tokb[i] * p.N + c + x2) = *reinterpret_cast<const uint32_t*>(&o);
      }
    }
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kFewThreads, 3) requests_few_kernel(const __grid_constant__ CUtensorMap w1a,
                                                                      const __grid_constant__ CUtensorMap w1b,
                                                                      const __grid_constant__ CUtensorMap w2a,
                                                                      const __grid_constant__ CUtensorMap w2b,
                                                                      const __grid_constant__ FewArgs p) {
  extern __shared__ uint8_t smem_raw[];
  FewShared& s = *reinterpret_cast<FewShared*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int csize = p.csize;                   // CTAs of a cluster
  const int q = (int)(blockIdx.x % csize);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kFewStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), kFewWarps);
    }
    mbar_init(smem_u32(&s.ready), 1);
    s.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&w1b);
    tma_prefetch_desc(&w2b);
  }
  __syncwarp();
  cluster_sync();                              // every CTA's barriers are set up
  griddep_wait();
  griddep_launch_dependents();
  const int4 tile = p.tiles[blockIdx.x / csize];
  if (tile.z <= 0) return;                     // the whole cluster leaves
  const int count = min(tile.z, kFewTile);
  const AdapterRows ad = adapter_rows(p.pool, tile.x, p.width);
  // columns of U beyond the rank are zero
  if (q == 0 && (p.U || p.sU)) {
    const int rest = p.width - ad.rank;
    for (int e = threadIdx.x; e < count * rest; e += kFewThreads) {
      const int64_t row = p.order[tile.y + e / rest];
      const int r = ad.rank + e % rest;
      if (p.U) p.U[row * p.width + r] = 0.f;
      if (p.sU) p.sU[row * p.width + r] = 0.f;
    }
  }
  if (ad.rank == 0) {
    // no adapter: the base's rows as they are
    if (p.out != p.base) {
      const int n8 = p.N / 8, stride = csize * kFewThreads;
      for (int t = 0; t < count; ++t) {
        const int64_t row = (int64_t)p.order[tile.y + t] * p.N;
        for (int c = q * kFewThreads + threadIdx.x; c < n8; c += stride)
          reinterpret_cast<uint4*>(p.out + row)[c] =
              p.base ? reinterpret_cast<const uint4*>(p.base + row)[c] : make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  // shares of the columns: whole 16-byte words
  const int kc = ((p.K / 8 + csize - 1) / csize) * 8, nc = ((p.N / 8 + csize - 1) / csize) * 8;
  const int k0 = min(p.K, q * kc), k1 = min(p.K, k0 + kc);
  const int n0 = min(p.N, q * nc), n1 = min(p.N, n0 + nc);
  if (threadIdx.x >= 32 * kFewWarps) {
    FewRing ring;
    int issued = 0;
    if (!few_produce(s, ring, issued, &w1a, &w1b, ad.first, ad.rank, k0, k1, false) ||
        !few_produce(s, ring, issued, &w2a, &w2b, ad.first, ad.rank, n0, n1, true))
      for (int i = 0; i < min(issued, kFewStages); ++i)        // let copies in flight land
        mbar_wait_bounded(smem_u32(&s.full[i]), (uint32_t)((issued - 1 - i) / kFewStages & 1), nullptr);
  } else {
    few_consume(p, s, ad, tile, count, q, k0, k1, n0, n1);
  }
  __syncwarp();
  cluster_sync();                              // no CTA leaves while another may still send to it
}

// Gradients of few tokens: dW[first + r][c] = sum over the adapter's tokens of
// V[t][r] X[t][c], fp32 on CUDA cores, tokens in order.  A block takes 16 rows
// of one adapter (blockIdx.x: 4096 adapters of rank 256 are more than y may
// count) and 512 columns (y) of one of the two factors (z); rows between the
// rank and its multiple of 16 get zeros, and so do all rows of an adapter
// without tokens.  Tensor cores would need V in three terms for a handful of
// tokens; this is bound by latency: 13.5 us alone between two events, L2 flushed,
// for 48 tokens of 6 adapters, 4096 x 4096 (some 4 us of them the events').
struct FewGradArgs {
  const uint16_t* X[2];
  const float* V[2];        // T x width, scaled by v_scale ? the adapter's scale : 1
  float* dW[2];
  int cols[2];
  int scale_v[2];
  int width, row_blocks;
  const int32_t* order;
  const int32_t* seg;
  PoolArgs pool;
};
constexpr int kFewGradThreads = 128;
constexpr int kFewGradTokens = 32;

__global__ void __launch_bounds__(kFewGradThreads, 2) requests_few_grads_kernel(const FewGradArgs p) {
  __shared__ __align__(16) float s_v[kFewGradTokens][16];
  __shared__ int s_tok[kFewGradTokens];
  griddep_wait();
  griddep_launch_dependents();
  const int z = blockIdx.z;
  const int a = blockIdx.x / p.row_blocks, rb = blockIdx.x % p.row_blocks;
  const AdapterRows ad = adapter_rows(p.pool, a, p.width);
  if (rb * 16 >= ad.rank) return;
  const int cols = z ? p.cols[1] : p.cols[0];
  const uint16_t* X = z ? p.X[1] : p.X[0];
  const float* V = z ? p.V[1] : p.V[0];
  float* dW = z ? p.dW[1] : p.dW[0];
  const float vs = (z ? p.scale_v[1] : p.scale_v[0]) ? ad.scale : 1.f;
  const int c = (blockIdx.y * kFewGradThreads + threadIdx.x) * 4;
  if ((int)(blockIdx.y * kFewGradThreads * 4) >= cols) return;
  const int lo = p.seg[a], hi = p.seg[a + 1];
  float acc[16][4];
#pragma unroll
  for (int r = 0; r < 16; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[r][j] = 0.f;
  for (int t0 = lo; t0 < hi; t0 += kFewGradTokens) {
    const int m = min(kFewGradTokens, hi - t0);
    __syncthreads();
    for (int e = threadIdx.x; e < m * 16; e += kFewGradThreads) {
      const int t = e / 16, r = e % 16;
      const int row = p.order[t0 + t];
      if (r == 0) s_tok[t] = row;
      s_v[t][r] = rb * 16 + r < ad.rank ? vs * V[(int64_t)row * p.width + rb * 16 + r] : 0.f;
    }
    __syncthreads();
    if (c < cols) {
#pragma unroll 4
      for (int t = 0; t < m; ++t) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(X + (int64_t)s_tok[t] * cols + c));
        const float f[4] = {bf_lo(x.x), bf_hi(x.x), bf_lo(x.y), bf_hi(x.y)};
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float v = s_v[t][r];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[r][j] = __fmaf_rn(v, f[j], acc[r][j]);
        }
      }
    }
  }
  if (c < cols) {
#pragma unroll
    for (int r = 0; r < 16; ++r)
      *reinterpret_cast<float4*>(dW + (int64_t)(ad.first + rb * 16 + r) * cols + c) =
          rb * 16 + r < ad.rank ? make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3])
                                : make_float4(0.f, 0.f, 0.f, 0.f);        // (also where a token holds an infinity)
  }
}

}  // namespace qlora

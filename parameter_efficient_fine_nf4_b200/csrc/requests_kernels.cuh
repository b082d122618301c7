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
// the requests of its slice.  Bound by latency: two dependent scans.
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
// barrier and remote loads.)  One launch, the factors read once, all
// arithmetic in fp32 on CUDA cores.
//
// The factors are what has to be read (a few tokens' X is nothing), so a
// producer thread streams this CTA's part of both through a ring of TMA boxes,
// 16 rows x 256 columns a stage: 48 KB are in flight per CTA from the first
// moment, and the second factor arrives while the cluster still adds up U.
constexpr int kFewTile = 8;
constexpr int kFewWarps = 8;                   // consumers; one more warp produces
constexpr int kFewThreads = 32 * (kFewWarps + 1);
constexpr int kFewRows = 16;                   // rows of a stage
constexpr int kFewCols = 256;                  // columns of a stage
constexpr int kFewStages = 6;
constexpr int kFewStageBytes = kFewRows * kFewCols * 2;

struct FewArgs {
  const uint16_t* X;       // T x K
  const uint16_t* base;    // T x N, or null (zero)
  uint16_t* out;           // T x N
  float* U;                // T x width: U of each token (zeros beyond its rank), or null
  float* sU;               // the same times the adapter's scale, or null
  int K, N, T, width, csize;
  const int32_t* order;
  const int4* tiles;
  PoolArgs pool;
};

struct FewShared {
  uint64_t full[kFewStages], empty[kFewStages], ready;
  int abort_flag;
  alignas(16) float red[kFewTile * kFewCols];    // the second half of the rows' sums
  alignas(128) uint8_t ring[kFewStages * kFewStageBytes];
  // behind it, by the pool's width: float u[8][width] (scaled U), then what the
  // cluster's CTAs sent, part[CTA][row][tokens of the tile, a power of two]
  __device__ __forceinline__ float* u() { return reinterpret_cast<float*>(ring + kFewStages * kFewStageBytes); }
  __device__ __forceinline__ float* part(int width) { return u() + kFewTile * width; }
};
__host__ __device__ __forceinline__ size_t few_smem_bytes(int width, int csize) {
  return sizeof(FewShared) + (size_t)(1 + csize) * kFewTile * width * 4;
}

// N floats to shared memory of a CTA of the cluster, counted on its barrier.
template <int N>
__device__ __forceinline__ void store_async(uint32_t cluster_addr, const float* v, uint32_t cluster_bar) {
  if (N == 1)
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(cluster_addr),
                 "r"(__float_as_uint(v[0])), "r"(cluster_bar)
                 : "memory");
  else if (N == 2)
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(cluster_addr),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(cluster_bar)
                 : "memory");
  else
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                       cluster_addr + 4u * i),
                   "r"(__float_as_uint(v[i])), "r"(__float_as_uint(v[i + 1])), "r"(__float_as_uint(v[i + 2])),
                   "r"(__float_as_uint(v[i + 3])), "r"(cluster_bar)
                   : "memory");
}

// Two products and sums at once: d.{lo,hi} += a.{lo,hi} * b.{lo,hi}.
__device__ __forceinline__ void fma2(float2& d, float2 a, float2 b) {
  uint64_t x = *reinterpret_cast<uint64_t*>(&d);
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(x) : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  d = *reinterpret_cast<float2*>(&x);
}

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

// Stages of one factor for this CTA (one thread): for the first factor all
// columns of 16 rows, then the next rows; for the second all rows of 256
// columns.  Boxes of 8 rows: a stage's second one only where the rank has it.
__device__ __forceinline__ bool few_produce(FewShared& s, FewRing& ring, int& issued, const CUtensorMap* w, int first, int rank,
                                            int c0, int c1, bool rows_first) {
  const int rb = (rank + kFewRows - 1) / kFewRows, cb = (c1 - c0 + kFewCols - 1) / kFewCols;
  for (int i = 0; i < rb * cb; ++i) {
    const int r = (rows_first ? i % rb : i / cb) * kFewRows, c = c0 + (rows_first ? i / rb : i % cb) * kFewCols;
    const bool two = rank - r > 8;
    const uint32_t full = smem_u32(&s.full[ring.at]);
    if (!mbar_wait_bounded(smem_u32(&s.empty[ring.at]), ring.phase ^ 1u, &s.abort_flag)) return false;
    mbar_arrive_expect_tx(full, two ? kFewStageBytes : kFewStageBytes / 2);
    const uint32_t dst = smem_u32(s.ring) + (uint32_t)(ring.at * kFewStageBytes);
    tma_load_2d(dst, w, full, c, first + r);
    if (two) tma_load_2d(dst + kFewStageBytes / 2, w, full, c, first + r + 8);
    ring.next();
    ++issued;
  }
  return true;
}

// The consumers' side of a tile (warps 0 .. 7).  X's values stay in L1.
template <int NT>
__device__ __forceinline__ void few_consume(const FewArgs& p, FewShared& s, const AdapterRows& ad, const int (&tok)[kFewTile],
                                            int count, int q, int k0, int k1, int n0, int n1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rb = (ad.rank + kFewRows - 1) / kFewRows;
  float* s_u = s.u();
  float* s_part = s.part(p.width);
  if (p.csize > 1 && threadIdx.x == 0)
    mbar_arrive_expect_tx(smem_u32(&s.ready), (uint32_t)((p.csize - 1) * ad.rank * NT * 4));
  FewRing ring;
  bool ok = true;
  // U: a warp takes rows w and w + 8 of a stage, a lane 8 columns
  for (int r = 0; r < ad.rank && ok; r += kFewRows) {
    float2 acc[2][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[0][t] = acc[1][t] = make_float2(0.f, 0.f);
    for (int c = k0; c < k1; c += kFewCols) {
      const int x0 = c + lane * 8;
      const bool in = x0 < k1;
      uint4 xv[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
        xv[t] = in ? __ldg(reinterpret_cast<const uint4*>(p.X + (int64_t)tok[t] * p.K + x0)) : make_uint4(0, 0, 0, 0);
      ok = mbar_wait_bounded(smem_u32(&s.full[ring.at]), ring.phase, &s.abort_flag);
      if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
      const uint8_t* st = s.ring + ring.at * kFewStageBytes + warp * (kFewCols * 2) + lane * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (in && r + warp + 8 * i < ad.rank) {
          const uint4 w = *reinterpret_cast<const uint4*>(st + i * 8 * kFewCols * 2);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 wf = make_float2(bf_lo(ws[j]), bf_hi(ws[j]));
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint32_t xs[4] = {xv[t].x, xv[t].y, xv[t].z, xv[t].w};
              fma2(acc[i][t], wf, make_float2(bf_lo(xs[j]), bf_hi(xs[j])));
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.empty[ring.at]));
      ring.next();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = r + warp + 8 * i;
      if (row >= ad.rank) break;
      float v[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        v[t] = acc[i][t].x + acc[i][t].y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[t] += __shfl_xor_sync(0xFFFFFFFFu, v[t], o);
      }
      // lane c sends the row's sums to CTA c, this CTA's own are plain stores
      if (lane == q) {
#pragma unroll
        for (int t = 0; t < NT; ++t) s_part[(q * p.width + row) * NT + t] = v[t];
      } else if (lane < p.csize)
        store_async<NT>(mapa_shared(smem_u32(s_part + (q * p.width + row) * NT), (uint32_t)lane), v,
                        mapa_shared(smem_u32(&s.ready), (uint32_t)lane));
      __syncwarp();
    }
  }
  // base comes in while the cluster meets
  const int g = threadIdx.x >> 7, x2 = (threadIdx.x & 127) * 2;     // half of a stage's rows, 2 columns
  uint32_t base[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
    base[t] = g == 0 && p.base && t < count && n0 + x2 < n1
                  ? *reinterpret_cast<const uint32_t*>(p.base + (int64_t)tok[t] * p.N + n0 + x2) : 0u;
  named_bar_sync(1, 32 * kFewWarps);
  if (p.csize > 1) ok = mbar_wait_bounded(smem_u32(&s.ready), 0, &s.abort_flag) && ok;
  __syncwarp();
  for (int e = threadIdx.x; e < ad.rank * NT; e += 32 * kFewWarps) {
    const int r = e / NT, t = e % NT;
    float v = 0.f;
#pragma unroll 8
    for (int c = 0; c < p.csize; ++c) v += s_part[(c * p.width + r) * NT + t];
    s_u[t * p.width + r] = ad.scale * v;
    if (q == 0 && t < count) {
      if (p.U) p.U[(int64_t)tok[t] * p.width + r] = v;
      if (p.sU) p.sU[(int64_t)tok[t] * p.width + r] = ad.scale * v;
    }
  }
  // rows up to the stage's 16 multiply whatever the stage holds: make that nothing
  for (int e = threadIdx.x; e < (rb * kFewRows - ad.rank) * NT; e += 32 * kFewWarps)
    s_u[(e % NT) * p.width + ad.rank + e / NT] = 0.f;
  named_bar_sync(1, 32 * kFewWarps);
  for (int c = n0; c < n1; c += kFewCols) {
    const int x = c + x2;
    const bool in = x < n1;
    if (c > n0) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        base[t] = g == 0 && p.base && t < count && in ? *reinterpret_cast<const uint32_t*>(p.base + (int64_t)tok[t] * p.N + x) : 0u;
    }
    float acc[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = 0.f;
    for (int r = 0; r < ad.rank && ok; r += kFewRows) {
      ok = mbar_wait_bounded(smem_u32(&s.full[ring.at]), ring.phase, &s.abort_flag);
      if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
      if (in && r + 8 * g < ad.rank) {
        const uint8_t* st = s.ring + ring.at * kFewStageBytes + 8 * g * (kFewCols * 2) + x2 * 2;
        const int m = min(8, ad.rank - r - 8 * g);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = i < m ? *reinterpret_cast<const uint32_t*>(st + i * kFewCols * 2) : 0u;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float4 a = *reinterpret_cast<const float4*>(s_u + t * p.width + r + 8 * g);
          const float4 b = *reinterpret_cast<const float4*>(s_u + t * p.width + r + 8 * g + 4);
          const float u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[t][0] = __fmaf_rn(u[i], bf_lo(w[i]), acc[t][0]);
            acc[t][1] = __fmaf_rn(u[i], bf_hi(w[i]), acc[t][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.empty[ring.at]));
      ring.next();
    }
    if (rb * kFewRows > 8 && ad.rank > 8) {      // the second half's sums
      named_bar_sync(1, 32 * kFewWarps);
      if (g == 1) {
#pragma unroll
        for (int t = 0; t < NT; ++t) *reinterpret_cast<float2*>(s.red + t * kFewCols + x2) = make_float2(acc[t][0], acc[t][1]);
      }
      named_bar_sync(1, 32 * kFewWarps);
      if (g == 0) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float2 v = *reinterpret_cast<const float2*>(s.red + t * kFewCols + x2);
          acc[t][0] += v.x;
          acc[t][1] += v.y;
        }
      }
    }
    if (g == 0 && in) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t >= count) break;
        const __nv_bfloat162 o = __floats2bfloat162_rn(bf_lo(base[t]) + acc[t][0], bf_hi(base[t]) + acc[t][1]);
        *reinterpret_cast<uint32_t*>(p.out + (int64_t)tok[t] * p.N + x) = *reinterpret_cast<const uint32_t*>(&o);
      }
    }
  }
}

__global__ void __launch_bounds__(kFewThreads, 3) requests_few_kernel(const __grid_constant__ CUtensorMap w1,
                                                                      const __grid_constant__ CUtensorMap w2,
                                                                      const __grid_constant__ FewArgs p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  FewShared& s = *reinterpret_cast<FewShared*>(smem_raw);
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
  }
  cluster_sync();                              // every CTA's barriers are set up
  griddep_wait();
  griddep_launch_dependents();
  const int4 tile = p.tiles[blockIdx.x / csize];
  if (tile.z <= 0) return;                     // the whole cluster leaves
  const int count = min(tile.z, kFewTile);
  int tok[kFewTile];
#pragma unroll
  for (int t = 0; t < kFewTile; ++t) tok[t] = p.order[tile.y + min(t, count - 1)];
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
    if ((threadIdx.x & 31) == 0) {
      FewRing ring;
      int issued = 0;
      if (!few_produce(s, ring, issued, &w1, ad.first, ad.rank, k0, k1, false) ||
          !few_produce(s, ring, issued, &w2, ad.first, ad.rank, n0, n1, true))
        for (int i = 0; i < min(issued, kFewStages); ++i)        // let copies in flight land
          mbar_wait_bounded(smem_u32(&s.full[i]), (uint32_t)((issued - 1 - i) / kFewStages & 1), nullptr);
    }
    __syncwarp();
  } else {
    if (count == 1) few_consume<1>(p, s, ad, tok, count, q, k0, k1, n0, n1);
    else if (count == 2) few_consume<2>(p, s, ad, tok, count, q, k0, k1, n0, n1);
    else if (count <= 4) few_consume<4>(p, s, ad, tok, count, q, k0, k1, n0, n1);
    else few_consume<8>(p, s, ad, tok, count, q, k0, k1, n0, n1);
  }
  __syncwarp();
  cluster_sync();                              // no CTA leaves while another may still send to it
}

// Gradients of few tokens: dW[first + r][c] = sum over the adapter's tokens of
// V[t][r] X[t][c], fp32 on CUDA cores, tokens in order.  A block takes 16 rows
// of one adapter and 512 columns of one of the two factors (blockIdx.z); rows
// between the rank and its multiple of 16 get zeros (V is zero there), and so
// do all rows of an adapter without tokens.
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

__global__ void __launch_bounds__(kFewGradThreads) requests_few_grads_kernel(const FewGradArgs p) {
  __shared__ __align__(16) float s_v[kFewGradTokens][16];
  __shared__ int s_tok[kFewGradTokens];
  griddep_wait();
  griddep_launch_dependents();
  const int z = blockIdx.z;
  const int a = blockIdx.y / p.row_blocks, rb = blockIdx.y % p.row_blocks;
  const AdapterRows ad = adapter_rows(p.pool, a, p.width);
  if (rb * 16 >= ad.rank) return;
  const int cols = z ? p.cols[1] : p.cols[0];
  const uint16_t* X = z ? p.X[1] : p.X[0];
  const float* V = z ? p.V[1] : p.V[0];
  float* dW = z ? p.dW[1] : p.dW[0];
  const float vs = (z ? p.scale_v[1] : p.scale_v[0]) ? ad.scale : 1.f;
  const int c = (blockIdx.x * kFewGradThreads + threadIdx.x) * 4;
  if ((int)(blockIdx.x * kFewGradThreads * 4) >= cols) return;
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
          make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
  }
}

}  // namespace qlora

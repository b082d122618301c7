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

  // first rows: a 64-bit sum, cut at T, so that no lengths can overflow it
  {
    const int per = (p.n_req + kPlanThreads - 1) / kPlanThreads;
    const int i0 = min(p.n_req, tid * per), i1 = min(p.n_req, i0 + per);
    long long sum = 0;
    for (int i = i0; i < i1; ++i) sum += max(0, p.lens[i]);
    long long total;
    long long run = block_exclusive<long long>(sum, s_warp64, total);
    for (int i = i0; i < i1; ++i) {
      s_start[i] = (int)min(run, (long long)p.T);
      run += max(0, p.lens[i]);
      const int a = p.ids[i];
      s_id[i] = (a >= 0 && a < p.n) ? a : p.n;
    }
    if (tid == 0) s_start[p.n_req] = (int)min(total, (long long)p.T);
  }
  for (int g = tid; g < p.n + 2; g += kPlanThreads) s_seg[g] = 0;
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
  const int f = p.first[a], k = p.rank[a];
  if (f < 0 || k < 1 || k > width || f > p.rows - ((k + 15) & ~15)) return r;
  r.first = f;
  r.rank = k;
  r.scale = p.scale[a];
  return r;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// ------------------------------------------------------------------ few tokens
// Tiles of up to 8 tokens of one adapter.  A cluster of CTAs takes one tile:
// each CTA sums U over its share of the K columns, the shares are added in
// rank order over the cluster's shared memory, and each CTA then writes its
// share of the N output columns.  One launch, X and the factors read once,
// everything in fp32 on CUDA cores.
constexpr int kFewTile = 8;
constexpr int kFewThreads = 256;

struct FewArgs {
  const uint16_t* W1;      // rows x K
  const uint16_t* W2;      // rows x N
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

// Rows of 8 consecutive bf16 values times NT tokens: acc[row][token] += w . x
template <int NT>
__device__ __forceinline__ void few_shrink(const FewArgs& p, const AdapterRows& ad, const int (&tok)[kFewTile], int k0,
                                           int k1, float* s_part) {
  constexpr int RB = NT >= 4 ? 2 : 4;          // rows per pass share the loaded x
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r0 = warp * RB; r0 < ad.rank; r0 += (kFewThreads / 32) * RB) {
    float acc[RB][NT];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[i][t] = 0.f;
    const uint16_t* w0 = p.W1 + (int64_t)(ad.first + r0) * p.K;
#pragma unroll 2
    for (int c = k0 + lane * 8; c < k1; c += 256) {
      uint4 w[RB];
#pragma unroll
      for (int i = 0; i < RB; ++i)
        w[i] = r0 + i < ad.rank ? __ldg(reinterpret_cast<const uint4*>(w0 + (int64_t)i * p.K + c)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p.X + (int64_t)tok[t] * p.K + c));
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[i][t] = __fmaf_rn(bf_lo(ws[j]), bf_lo(xs[j]), acc[i][t]);
            acc[i][t] = __fmaf_rn(bf_hi(ws[j]), bf_hi(xs[j]), acc[i][t]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float v = acc[i][t];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if (lane == 0 && r0 + i < ad.rank) s_part[(r0 + i) * kFewTile + t] = v;
      }
  }
}

// out[tok][c..c+3] for this CTA's columns; RG groups of threads share the
// adapter's rows and are summed in group order.
template <int NT>
__device__ __forceinline__ void few_expand(const FewArgs& p, const AdapterRows& ad, const int (&tok)[kFewTile], int count,
                                           int n0, int n1, const float* s_u, float* s_red) {
  const int cols4 = (n1 - n0) / 4;
  int groups = 1;
  while (groups < 8 && cols4 * groups * 2 <= kFewThreads) groups *= 2;
  const int per = kFewThreads / groups;        // threads of a group
  const int g = threadIdx.x / per, x = threadIdx.x % per;
  for (int cb = 0; cb < cols4; cb += per) {
    const int c4 = cb + x;
    const bool ok = c4 < cols4;
    const int c = n0 + c4 * 4;
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t][j] = 0.f;
    if (ok) {
      const uint16_t* w = p.W2 + (int64_t)ad.first * p.N + c;
#pragma unroll 4
      for (int r = g; r < ad.rank; r += groups) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(w + (int64_t)r * p.N));
        const float f[4] = {bf_lo(v.x), bf_hi(v.x), bf_lo(v.y), bf_hi(v.y)};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float u = s_u[r * kFewTile + t];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[t][j] = __fmaf_rn(u, f[j], acc[t][j]);
        }
      }
    }
    if (groups > 1) {
      __syncthreads();
      if (ok && g > 0) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          *reinterpret_cast<float4*>(s_red + (((g - 1) * NT + t) * per + x) * 4) =
              make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
      }
      __syncthreads();
      if (ok && g == 0) {
        for (int q = 1; q < groups; ++q)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float4 v = *reinterpret_cast<const float4*>(s_red + (((q - 1) * NT + t) * per + x) * 4);
            acc[t][0] += v.x; acc[t][1] += v.y; acc[t][2] += v.z; acc[t][3] += v.w;
          }
      }
    }
    if (ok && g == 0) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t >= count) break;
        const int64_t at = (int64_t)tok[t] * p.N + c;
        uint2 b = make_uint2(0, 0);
        if (p.base) b = *reinterpret_cast<const uint2*>(p.base + at);
        uint2 o;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(bf_lo(b.x) + acc[t][0], bf_hi(b.x) + acc[t][1]);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(bf_lo(b.y) + acc[t][2], bf_hi(b.y) + acc[t][3]);
        o.x = *reinterpret_cast<const uint32_t*>(&lo);
        o.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(p.out + at) = o;
      }
    }
  }
}

template <int NT>
__device__ __forceinline__ void few_tile(const FewArgs& p, const AdapterRows& ad, const int (&tok)[kFewTile], int count,
                                         int q, int csize, float* s_part, float* s_u, float* s_red) {
  // shares of the columns: whole 16-byte words
  const int kc = ((p.K / 8 + csize - 1) / csize) * 8, nc = ((p.N / 8 + csize - 1) / csize) * 8;
  const int k0 = min(p.K, q * kc), k1 = min(p.K, k0 + kc);
  const int n0 = min(p.N, q * nc), n1 = min(p.N, n0 + nc);
  few_shrink<NT>(p, ad, tok, k0, k1, s_part);
  cluster_sync();
  const uint32_t part = smem_u32(s_part);
  for (int e = threadIdx.x; e < ad.rank * NT; e += kFewThreads) {
    const int r = e / NT, t = e % NT;
    float v = 0.f;
    for (int c = 0; c < csize; ++c)
      v += ld_shared_cluster_f32(mapa_shared(part + (uint32_t)(r * kFewTile + t) * 4u, (uint32_t)c));
    s_u[r * kFewTile + t] = ad.scale * v;
    if (q == 0 && t < count) {
      if (p.U) p.U[(int64_t)tok[t] * p.width + r] = v;
      if (p.sU) p.sU[(int64_t)tok[t] * p.width + r] = ad.scale * v;
    }
  }
  __syncthreads();
  few_expand<NT>(p, ad, tok, count, n0, n1, s_u, s_red);
}

__global__ void __launch_bounds__(kFewThreads) requests_few_kernel(const FewArgs p) {
  __shared__ __align__(16) float s_part[256 * kFewTile];
  __shared__ __align__(16) float s_u[256 * kFewTile];
  __shared__ __align__(16) float s_red[kFewTile * kFewThreads * 4];
  const int csize = p.csize;                   // CTAs of a cluster
  const int q = (int)(blockIdx.x % csize);
  griddep_wait();
  const int4 tile = p.tiles[blockIdx.x / csize];
  if (tile.z <= 0) return;                     // the whole cluster leaves
  const int count = min(tile.z, kFewTile);
  int tok[kFewTile];
#pragma unroll
  for (int t = 0; t < kFewTile; ++t) tok[t] = p.order[tile.y + min(t, count - 1)];
  const AdapterRows ad = adapter_rows(p.pool, tile.x, p.width);
  // columns of U beyond the rank are zero
  if (q == 0) {
    for (int e = threadIdx.x; e < count * (p.width - ad.rank); e += kFewThreads) {
      const int t = e / (p.width - ad.rank), r = ad.rank + e % (p.width - ad.rank);
      int row = 0;
#pragma unroll
      for (int j = 0; j < kFewTile; ++j)
        if (j == t) row = tok[j];
      if (p.U) p.U[(int64_t)row * p.width + r] = 0.f;
      if (p.sU) p.sU[(int64_t)row * p.width + r] = 0.f;
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
  if (count == 1) few_tile<1>(p, ad, tok, count, q, csize, s_part, s_u, s_red);
  else if (count == 2) few_tile<2>(p, ad, tok, count, q, csize, s_part, s_u, s_red);
  else if (count <= 4) few_tile<4>(p, ad, tok, count, q, csize, s_part, s_u, s_red);
  else few_tile<8>(p, ad, tok, count, q, csize, s_part, s_u, s_red);
  cluster_sync();                              // no CTA leaves while its sums may still be read
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

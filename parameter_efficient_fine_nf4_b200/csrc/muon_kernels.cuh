// The optimiser step that orthogonalises a factor's momentum (the Muon rule),
// for a stack of n equal matrices: the update of an adapter factor is
// replaced by the nearest matrix with equal singular values, found by
// Newton-Schulz iterations of an odd quintic.
//
//   m = mu m + g,  u = g + mu m (Nesterov) or m,  x0 = u / (|u|_F + eps)
//   x <- a x + b (x x^T) x + c (x x^T)^2 x          (steps times)
//   master = (1 - lr wd) master - lr scale x,  w16 = bf16(master)
//
// A factor is long and thin (one side is the rank), so the iterations never
// touch the long side here.  With R = x x^T (r x r) every iterate is x = P x0
// with P a polynomial in R0, and
//   Q = a I + b R + c R^2,   P <- Q P,   R <- Q R Q,
// all symmetric and commuting.  The long side is read once for R0 and once
// for P x0.  Small singular values grow some fivehundredfold, and P depends on
// them through their squares, so R0 and the r x r products are held in 64
// bits: rounding R0 to 32 bits alone would leave errors of 1e-3 in directions
// a thousand times smaller than the largest.
//
// "Wide" matrices (rows <= cols) use x x^T; tall ones the same formulas on
// their transpose.  Element (i, c): i on the short side, c on the long one.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace qlora {

struct MuonArgs {
  float* master;
  uint16_t* w16;
  float* m;
  const float* g;
  int r, rp;               // short side, and its multiple of 16
  int64_t len;             // long side
  int tall, nesterov, chunks;
  int64_t chunk;           // long-side elements per block of the Gram kernel
  float mu, keep, step;    // keep = 1 - lr wd, step = lr scale
  double eps, a, b, c;
  double* part;            // [n][chunks][rp][rp] partial Gram matrices
  double* R;               // [n][rp][rp]
  double* P;
  double* Q;
  double* H;
};

__device__ __forceinline__ int64_t muon_at(const MuonArgs& p, int64_t mat, int i, int64_t c) {
  const int64_t base = mat * (int64_t)p.r * p.len;
  return base + (p.tall ? c * p.r + i : (int64_t)i * p.len + c);
}
__device__ __forceinline__ float muon_u(const MuonArgs& p, float g, float m_new) {
  return p.nesterov ? __fmaf_rn(p.mu, m_new, g) : m_new;
}

// m = mu m + g over all elements.
__global__ void __launch_bounds__(256) muon_momentum_kernel(float* __restrict__ m, const float* __restrict__ g, float mu,
                                                            int64_t count) {
  griddep_wait();
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < count; i += stride)
    m[i] = __fmaf_rn(mu, m[i], g[i]);
}

// One 64 x 64 block (i0, j0) of the partial Gram matrix of one chunk of the
// long side: products and sums in 64 bits (the products of two 32-bit values
// are exact).  A thread holds 4 x 4 sums; 32 long-side elements are staged at
// a time.
constexpr int kGramThreads = 256;
constexpr int kGramStep = 32;
constexpr int kGramPitch = 66;             // doubles per staged long-side element
__global__ void __launch_bounds__(kGramThreads) muon_gram_kernel(const MuonArgs p) {
  __shared__ __align__(16) double s_i[kGramStep][kGramPitch];
  __shared__ __align__(16) double s_j[kGramStep][kGramPitch];
  griddep_wait();
  const int blocks = (p.rp + 63) / 64;
  int bi = 0, bj = blockIdx.y;             // upper triangle, row by row
  while (bj >= blocks - bi) { bj -= blocks - bi; ++bi; }
  bj += bi;
  const int64_t mat = blockIdx.z;
  const int64_t c0 = (int64_t)blockIdx.x * p.chunk, c1 = min(p.len, c0 + p.chunk);
  const int ti = (threadIdx.x / 16) * 4, tj = (threadIdx.x % 16) * 4;
  double acc[4][4] = {};
  for (int64_t cb = c0; cb < c1; cb += kGramStep) {
    __syncthreads();
    for (int side = 0; side < (bi == bj ? 1 : 2); ++side) {
      double(*s)[kGramPitch] = side ? s_j : s_i;
      const int base = (side ? bj : bi) * 64;
      for (int e = threadIdx.x; e < 64 * kGramStep; e += kGramThreads) {
        const int i = p.tall ? e % 64 : e / kGramStep, c = p.tall ? e / 64 : e % kGramStep;
        double v = 0.0;
        if (base + i < p.r && cb + c < c1) {
          const int64_t at = muon_at(p, mat, base + i, cb + c);
          v = (double)muon_u(p, p.g[at], p.m[at]);
        }
        s[c][i] = v;
      }
    }
    __syncthreads();
    const double(*sj)[kGramPitch] = bi == bj ? s_i : s_j;
#pragma unroll 4
    for (int c = 0; c < kGramStep; ++c) {
      double x[4], y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[q] = s_i[c][ti + q];
        y[q] = sj[c][tj + q];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int w = 0; w < 4; ++w) acc[q][w] = fma(x[q], y[w], acc[q][w]);
    }
  }
  double* out = p.part + ((mat * p.chunks + blockIdx.x) * p.rp) * (int64_t)p.rp;
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int i = bi * 64 + ti + q, j = bj * 64 + tj + w;
      if (i < p.rp && j < p.rp) {
        out[(int64_t)i * p.rp + j] = acc[q][w];
        if (bi != bj) out[(int64_t)j * p.rp + i] = acc[q][w];
      }
    }
}

// R0 = (sum of the partials in chunk order) / (|u|_F + eps)^2; P starts as I.
__global__ void __launch_bounds__(256) muon_norm_kernel(const MuonArgs p) {
  __shared__ double s_sum[256];
  griddep_wait();
  const int64_t mat = blockIdx.y, sq = (int64_t)p.rp * p.rp;
  const double* part = p.part + mat * p.chunks * sq;
  double t = 0.0;
  for (int i = threadIdx.x; i < p.r; i += 256)
    for (int c = 0; c < p.chunks; ++c) t += part[c * sq + (int64_t)i * p.rp + i];
  s_sum[threadIdx.x] = t;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) s_sum[threadIdx.x] += s_sum[threadIdx.x + o];
    __syncthreads();
  }
  const double f = sqrt(s_sum[0]) + p.eps, inv = 1.0 / f;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < sq; e += (int64_t)gridDim.x * 256) {
    double v = 0.0;
    for (int c = 0; c < p.chunks; ++c) v += part[c * sq + e];
    p.R[mat * sq + e] = v * inv * inv;
    p.P[mat * sq + e] = (e / p.rp == e % p.rp) ? inv : 0.0;   // P carries the norm of x0 = u inv
  }
}

// One 32 x 32 block of an r x r product; what: 0: Q = a I + b R + c R R,
// 1: H = Q R (z < n) and the next P = Q P (z >= n, into `out2`), 2: R = Q H.
__global__ void __launch_bounds__(256) muon_square_kernel(const MuonArgs p, int what, const double* pin, double* pout, int n) {
  __shared__ double s_a[32][33];
  __shared__ double s_b[32][33];
  griddep_wait();
  const int64_t sq = (int64_t)p.rp * p.rp;
  const bool second = (int)blockIdx.z >= n;
  const int64_t mat = second ? blockIdx.z - n : blockIdx.z;
  const double* A = (what == 0 ? p.R : p.Q) + mat * sq;
  const double* B = (what == 0 ? p.R : what == 2 ? p.H : second ? pin : p.R) + mat * sq;
  double* O = (what == 0 ? p.Q : what == 2 ? p.R : second ? pout : p.H) + mat * sq;
  const int i0 = blockIdx.y * 32, j0 = blockIdx.x * 32;
  const int ti = threadIdx.x / 16 * 2, tj = threadIdx.x % 16 * 2;
  double acc[2][2] = {};
  for (int kb = 0; kb < p.rp; kb += 32) {
    __syncthreads();
    for (int e = threadIdx.x; e < 1024; e += 256) {
      const int x = e / 32, y = e % 32;
      s_a[x][y] = (i0 + x < p.rp && kb + y < p.rp) ? A[(int64_t)(i0 + x) * p.rp + kb + y] : 0.0;
      s_b[x][y] = (kb + x < p.rp && j0 + y < p.rp) ? B[(int64_t)(kb + x) * p.rp + j0 + y] : 0.0;
    }
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < 32; ++k)
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int w = 0; w < 2; ++w) acc[q][w] = fma(s_a[ti + q][k], s_b[k][tj + w], acc[q][w]);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int i = i0 + ti + q, j = j0 + tj + w;
      if (i >= p.rp || j >= p.rp) continue;
      double v = acc[q][w];
      if (what == 0) v = p.c * v + p.b * A[(int64_t)i * p.rp + j] + (i == j ? p.a : 0.0);
      O[(int64_t)i * p.rp + j] = v;
    }
}

// x = P u for 64 short-side rows and 32 long-side elements, and the update of
// the master and of its 16-bit copy.
__global__ void __launch_bounds__(256) muon_apply_kernel(const MuonArgs p, const double* P) {
  __shared__ double s_p[64][33];           // P[i0 + i][kb + k]
  __shared__ double s_u[32][33];           // u[kb + k][c0 + c]
  griddep_wait();
  const int64_t mat = blockIdx.z, sq = (int64_t)p.rp * p.rp;
  const int i0 = blockIdx.y * 64;
  const int64_t c0 = (int64_t)blockIdx.x * 32;
  const int ti = threadIdx.x / 16 * 4, tc = threadIdx.x % 16 * 2;
  double acc[4][2] = {};
  for (int kb = 0; kb < p.r; kb += 32) {
    __syncthreads();
    for (int e = threadIdx.x; e < 64 * 32; e += 256) {
      const int i = e / 32, k = e % 32;
      s_p[i][k] = (i0 + i < p.rp && kb + k < p.rp) ? P[mat * sq + (int64_t)(i0 + i) * p.rp + kb + k] : 0.0;
    }
    for (int e = threadIdx.x; e < 32 * 32; e += 256) {
      const int k = p.tall ? e % 32 : e / 32, c = p.tall ? e / 32 : e % 32;
      double v = 0.0;
      if (kb + k < p.r && c0 + c < p.len) {
        const int64_t at = muon_at(p, mat, kb + k, c0 + c);
        v = (double)muon_u(p, p.g[at], p.m[at]);
      }
      s_u[k][c] = v;
    }
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < 32; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int w = 0; w < 2; ++w) acc[q][w] = fma(s_p[ti + q][k], s_u[k][tc + w], acc[q][w]);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int i = i0 + ti + q;
      const int64_t c = c0 + tc + w;
      if (i >= p.r || c >= p.len) continue;
      const int64_t at = muon_at(p, mat, i, c);
      const float v = __fmaf_rn(p.keep, p.master[at], -__fmul_rn(p.step, (float)acc[q][w]));
      p.master[at] = v;
      const __nv_bfloat16 h = __float2bfloat16_rn(v);
      p.w16[at] = *reinterpret_cast<const uint16_t*>(&h);
    }
}

}  // namespace qlora

// CUDA-core kernels of the product Y = act(X W^T + bias) + residual in fp32 (the
// tensor cores' TF32 does not keep fp32's precision).
//
//   linear_gemv_kernel  up to 8 rows of X: a CTA's four warps share four rows of W
//       and split K; W streams from HBM once, 16 bytes a lane.  Bound by W's bytes up to
//       four rows (9728 -> 2560 with bias and residual 21 us, 15.2 at HBM's copy rate);
//       eight rows take 57 us.
//   linear_f32_kernel   BM x BN tiles, TM x TN outputs a thread, the next 16
//       columns of K in registers while the present ones are multiplied.  The
//       CTAs of a cluster split K where there are few tiles and join their sums
//       through distributed shared memory, in rank order.  Bound by the CUDA cores and
//       the shared-memory reads that feed them, a word a product: 333 x 1000 x 1001 with
//       bias and gelu 25.9 us (9.0 us at 128 products a clock and SM), 1154 x 2168 x
//       2547 309 us (171).  Two products an instruction leave issue slots to the loads
//       (28.3 and 373 us with one); 8 x 16 outputs a thread, which read less but leave
//       half the warps, were slower (480 us and more for the second).
#pragma once

#include "common.cuh"
#include "mixer.cuh"

namespace ittt {

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t cluster_address) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_address));
  return v;
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

template <int ACT>
__device__ __forceinline__ void linear_finish(const LinearArgs<float>& a, int m, int n, float v) {
  if (a.bias) v += a.bias[n];
  v = activate<ACT>(v);
  if (a.residual) v += a.residual[m * a.ldr + n];
  a.Y[m * a.ldy + n] = v;
}

// VEC: 16-byte pieces of the rows of X and W.
template <int ACT, int MB, bool VEC>
__global__ void __launch_bounds__(128) linear_gemv_kernel(const LinearArgs<float> a) {
  constexpr int NB = 4;
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * NB;
  float acc[MB][NB] = {};
  // rows past the end repeat the last one; their sums are not stored
  const float *w[NB], *x[MB];
#pragma unroll
  for (int j = 0; j < NB; ++j) w[j] = a.W + (long long)min(n0 + j, a.N - 1) * a.K;
#pragma unroll
  for (int i = 0; i < MB; ++i) x[i] = a.X + min(i, a.M - 1) * a.ldx;
  if (VEC) {
#pragma unroll 2
    for (int k = (warp * 32 + lane) * 4; k < a.K; k += 512) {
      float4 wv[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) wv[j] = __ldg(reinterpret_cast<const float4*>(w[j] + k));
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const float4 xv = *reinterpret_cast<const float4*>(x[i] + k);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          acc[i][j] = fmaf(xv.x, wv[j].x, acc[i][j]);
          acc[i][j] = fmaf(xv.y, wv[j].y, acc[i][j]);
          acc[i][j] = fmaf(xv.z, wv[j].z, acc[i][j]);
          acc[i][j] = fmaf(xv.w, wv[j].w, acc[i][j]);
        }
      }
    }
  } else {
#pragma unroll 4
    for (int k = warp * 32 + lane; k < a.K; k += 128) {
      float wv[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) wv[j] = __ldg(w[j] + k);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const float xv = x[i][k];
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = fmaf(xv, wv[j], acc[i][j]);
      }
    }
  }
  __shared__ float part[4][MB * NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      float v = acc[i][j];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) part[warp][i * NB + j] = v;
    }
  __syncthreads();
  if (threadIdx.x < MB * NB) {
    const int i = threadIdx.x / NB, n = n0 + threadIdx.x % NB;
    if (i < a.M && n < a.N)
      linear_finish<ACT>(a, i, n, (part[0][threadIdx.x] + part[1][threadIdx.x]) +
                                 (part[2][threadIdx.x] + part[3][threadIdx.x]));
  }
}

template <int BM, int BN, int TM, int TN>
struct F32Tile {
  static constexpr int THREADS = (BM / TM) * (BN / TN);
  static constexpr int KT = 16;
  static constexpr int LDM = BM + 4, LDN = BN + 4;  // 4 floats more a row: other banks
  static constexpr int SMEM = 2 * KT * (LDM + LDN) * 4;
  static_assert(BM * KT % (4 * THREADS) == 0 && BN * KT % (4 * THREADS) == 0, "whole passes");
  static_assert(TM % 4 == 0 && TN % 4 == 0, "16-byte fragments");
};

// Four floats of row r from column k (zeros past the end).
template <bool VEC>
__device__ __forceinline__ float4 f32_quad(const float* p, long long ld, int r, int rows, int k, int K) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r >= rows) return v;
  p += r * ld + k;
  if (VEC) {
    if (k < K) v = *reinterpret_cast<const float4*>(p);
  } else {
    if (k < K) v.x = p[0];
    if (k + 1 < K) v.y = p[1];
    if (k + 2 < K) v.z = p[2];
    if (k + 3 < K) v.w = p[3];
  }
  return v;
}

// The rows rank, rank + S, ... of a tile: the S sums of each value in rank order, 32
// remote loads in flight.
template <int ACT, int BM, int BN, int TH, int S>
__device__ __forceinline__ void f32_join(const LinearArgs<float>& a, uint32_t sums, int rank, int m0,
                                         int n0) {
  constexpr int MINE = BM * BN / S / TH, BATCH = MINE < 32 / S ? MINE : 32 / S;
  static_assert(BM % S == 0 && BM * BN % (S * TH) == 0 && MINE % BATCH == 0, "whole passes");
#pragma unroll 1
  for (int i0 = 0; i0 < MINE; i0 += BATCH) {
    float part[BATCH][S];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int e = (i0 + i) * TH + static_cast<int>(threadIdx.x);
      const uint32_t at = sums + static_cast<uint32_t>((e / BN * S + rank) * BN + e % BN) * 4u;
#pragma unroll
      for (int s = 0; s < S; ++s) part[i][s] = ld_shared_cluster_f32(cluster_addr(at, s));
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int e = (i0 + i) * TH + static_cast<int>(threadIdx.x);
      const int m = m0 + e / BN * S + rank, n = n0 + e % BN;
      float v = part[i][0];
#pragma unroll
      for (int s = 1; s < S; ++s) v += part[i][s];
      if (m < a.M && n < a.N) linear_finish<ACT>(a, m, n, v);
    }
  }
}

template <int ACT, int BM, int BN, int TM, int TN, bool VEC>
__global__ void __launch_bounds__(F32Tile<BM, BN, TM, TN>::THREADS)
    linear_f32_kernel(const LinearArgs<float> a, int m_tiles) {
  using S = F32Tile<BM, BN, TM, TN>;
  constexpr int KT = S::KT, TH = S::THREADS;
  constexpr int QA = BM * KT / (4 * TH), QB = BN * KT / (4 * TH);
  __shared__ __align__(16) float smem[S::SMEM / 4];
  float* As = smem;                        // [2][KT][LDM]
  float* Bs = smem + 2 * KT * S::LDM;      // [2][KT][LDN]
  const int splits = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_cta_rank());
  const int tile = blockIdx.x / splits;
  const int m0 = (tile % m_tiles) * BM, n0 = (tile / m_tiles) * BN;
  const int steps = (a.K + KT - 1) / KT;
  const int s0 = static_cast<int>((long long)steps * rank / splits);
  const int s1 = static_cast<int>((long long)steps * (rank + 1) / splits);
  const int tid = threadIdx.x;
  // a thread's outputs: fragments of 4, spread over the tile so that a quarter
  // warp's 16-byte reads fall on different banks
  constexpr int NX = BN / TN, NY = BM / TM;
  const int tx = tid % NX, ty = tid / NX;
  float4 ra[QA], rb[QB];
  auto load = [&](int step) {
    const int k = step * KT;
#pragma unroll
    for (int i = 0; i < QA; ++i) {
      const int e = i * TH + tid;
      ra[i] = f32_quad<VEC>(a.X, a.ldx, m0 + e / (KT / 4), a.M, k + (e % (KT / 4)) * 4, a.K);
    }
#pragma unroll
    for (int i = 0; i < QB; ++i) {
      const int e = i * TH + tid;
      rb[i] = f32_quad<VEC>(a.W, a.K, n0 + e / (KT / 4), a.N, k + (e % (KT / 4)) * 4, a.K);
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < QA; ++i) {
      const int e = i * TH + tid;
      float* d = As + (buf * KT + (e % (KT / 4)) * 4) * S::LDM + e / (KT / 4);
      d[0] = ra[i].x, d[S::LDM] = ra[i].y, d[2 * S::LDM] = ra[i].z, d[3 * S::LDM] = ra[i].w;
    }
#pragma unroll
    for (int i = 0; i < QB; ++i) {
      const int e = i * TH + tid;
      float* d = Bs + (buf * KT + (e % (KT / 4)) * 4) * S::LDN + e / (KT / 4);
      d[0] = rb[i].x, d[S::LDN] = rb[i].y, d[2 * S::LDN] = rb[i].z, d[3 * S::LDN] = rb[i].w;
    }
  };
  f32x2 acc2[TM][TN / 2] = {};  // two neighbouring columns
  grid_dependency_wait();
  if (s0 < s1) {
    load(s0);
    put(0);
  }
  __syncthreads();
  for (int s = s0; s < s1; ++s) {
    const int buf = (s - s0) & 1;
    if (s + 1 < s1) load(s + 1);
    const float* Ab = As + buf * KT * S::LDM + ty * 4;
    const float* Bb = Bs + buf * KT * S::LDN + tx * 4;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      float x[TM];
      f32x2 w[TN / 2];
#pragma unroll
      for (int i = 0; i < TM; i += 4)
        *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(Ab + k * S::LDM + i * NY);
#pragma unroll
      for (int j = 0; j < TN; j += 4)
        *reinterpret_cast<ulonglong2*>(w + j / 2) =
            *reinterpret_cast<const ulonglong2*>(Bb + k * S::LDN + j * NX);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const f32x2 xx = pack2(x[i], x[i]);
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) acc2[i][j] = fma2(xx, w[j], acc2[i][j]);
      }
    }
    if (s + 1 < s1) put(buf ^ 1);
    __syncthreads();
  }
  float acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN / 2; ++j) unpack2(acc2[i][j], acc[i][2 * j], acc[i][2 * j + 1]);
  auto row_of = [&](int i) { return (i / 4) * 4 * NY + ty * 4 + i % 4; };
  auto col_of = [&](int j) { return (j / 4) * 4 * NX + tx * 4 + j % 4; };
  if (splits == 1) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int m = m0 + row_of(i);
      if (m >= a.M) continue;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int n = n0 + col_of(j);
        if (n < a.N) linear_finish<ACT>(a, m, n, acc[i][j]);
      }
    }
    return;
  }
  // join the cluster's sums (only tiles whose sums fit the operands' place are split)
  if constexpr (BM * BN * 4 <= S::SMEM) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) smem[row_of(i) * BN + col_of(j)] = acc[i][j];
    cluster_sync_all();
    switch (splits) {
      case 2: f32_join<ACT, BM, BN, TH, 2>(a, smem_u32(smem), rank, m0, n0); break;
      case 4: f32_join<ACT, BM, BN, TH, 4>(a, smem_u32(smem), rank, m0, n0); break;
      default: f32_join<ACT, BM, BN, TH, 8>(a, smem_u32(smem), rank, m0, n0); break;
    }
    cluster_sync_all();  // no CTA leaves while a peer may still read its sums
  }
}

}  // namespace ittt

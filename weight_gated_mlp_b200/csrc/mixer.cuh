// Kernels of the operators around the layer: the product with bias, activation
// and residual, the short causal convolution and the selective state space
// scan.
#pragma once

#include "common.cuh"

namespace ittt {

template <typename T_>
__device__ __forceinline__ float to_f32(T_ v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T_>
__device__ __forceinline__ T_ from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// act(x) in fp32.  SiLU at -inf: e^inf = inf, x / inf would be NaN in a quotient
// of infinities; the limit, 0, is taken there.
__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case ITTT_ACT_RELU: return x < 0.f ? 0.f : x;  // NaN stays NaN
    case ITTT_ACT_SILU: return x == -INFINITY ? 0.f : x / (1.f + expf(-x));
    case ITTT_ACT_GELU: return x == -INFINITY ? 0.f : 0.5f * x * (1.f + erff(x * 0.70710678118654752f));
    case ITTT_ACT_GELU_TANH: {
      if (x == -INFINITY) return 0.f;
      const float a = 0.79788456080286536f * (x + 0.044715f * x * x * x);
      return 0.5f * x * (1.f + tanhf(a));
    }
    default: return x;
  }
}

// ------------------------------------------------------------------ linear

template <typename T_>
struct LinearArgs {
  const T_ *X, *W, *bias, *residual;
  T_* Y;
  long long ldx, ldr, ldy;
  int M, N, K, act;
};

// One 64 x 64 tile of Y per CTA on the CUDA cores, 4 x 4 outputs a thread.
template <typename T_>
__global__ void __launch_bounds__(256) linear_simt_kernel(const LinearArgs<T_> a) {
  __shared__ float xs[16][64 + 4], ws[16][64 + 4];
  grid_dependency_wait();
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += 16) {
    for (int e = threadIdx.x; e < 16 * 64; e += 256) {
      const int kk = e % 16, r = e / 16;
      const int m = m0 + r, n = n0 + r, k = k0 + kk;
      xs[kk][r] = (m < a.M && k < a.K) ? to_f32(a.X[m * a.ldx + k]) : 0.f;
      ws[kk][r] = (n < a.N && k < a.K) ? to_f32(a.W[(long long)n * a.K + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk) {
      float x[4], w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = xs[kk][ty * 4 + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = ws[kk][tx * 4 + j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], w[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= a.M || n >= a.N) continue;
      float v = acc[i][j];
      if (a.bias) v += to_f32(a.bias[n]);
      v = activate(v, a.act);
      if (a.residual) v += to_f32(a.residual[m * a.ldr + n]);
      a.Y[m * a.ldy + n] = from_f32<T_>(v);
    }
}

// ------------------------------------------------------------- causal conv

template <typename T_>
struct CausalConvArgs {
  const T_ *X, *w, *bias, *state_in;
  const int32_t* lengths;
  T_ *Y, *state_out;
  long long ldx, ldy;
  int B, T, d, k, act;
};

__device__ __forceinline__ int sequence_length(const int32_t* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

// One output per thread.  The threads of token 0 also move the state: each reads
// its channel's state_in before it writes the same channel's state_out, so the
// two may be one buffer (the outputs of the first k - 1 tokens need state_in
// too and are computed by the same thread).
template <typename T_>
__global__ void __launch_bounds__(256) causal_conv_kernel(const CausalConvArgs<T_> a) {
  grid_dependency_wait();
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  const int b = blockIdx.z;
  if (c >= a.d) return;
  const int len = sequence_length(a.lengths, b, a.T);
  const T_* X = a.X + (long long)b * a.T * a.ldx + c;
  T_* Y = a.Y + (long long)b * a.T * a.ldy + c;
  const T_* w = a.w + (long long)c * a.k;
  const T_* s_in = a.state_in ? a.state_in + (long long)b * (a.k - 1) * a.d + c : nullptr;
  const int back = a.k - 1;
  // CTA row 0: tokens 0..k-2 and the state; row r > 0: token k - 2 + r on
  const int t_first = blockIdx.y == 0 ? 0 : back + (blockIdx.y - 1) * 16;
  const int t_last = min(len, blockIdx.y == 0 ? back : t_first + 16);
  for (int t = t_first; t < t_last; ++t) {
    float acc = a.bias ? to_f32(a.bias[c]) : 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int s = t - back + j;
      float x = 0.f;
      if (s >= 0) x = to_f32(X[s * a.ldx]);
      else if (s_in) x = to_f32(s_in[(long long)(s + back) * a.d]);
      acc = fmaf(to_f32(w[j]), x, acc);
    }
    Y[t * a.ldy] = from_f32<T_>(activate(acc, a.act));
  }
  if (blockIdx.y == 0 && a.state_out) {
    T_* s_out = a.state_out + (long long)b * back * a.d + c;
    for (int j = 0; j < back; ++j) {  // slot j is read (as slot j' >= j) before it is written
      const int s = len - back + j;
      T_ x = from_f32<T_>(0.f);
      if (s >= 0) x = X[s * a.ldx];
      else if (s_in) x = s_in[(long long)(s + back) * a.d];
      s_out[(long long)j * a.d] = x;
    }
  }
}

}  // namespace ittt

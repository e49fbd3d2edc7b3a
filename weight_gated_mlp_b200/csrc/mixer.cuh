// What the kernels of the operators around the layer share (conversions, activations,
// paired arithmetic), and the short causal convolution.
#pragma once

#include <type_traits>

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

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x / (1 + e^-x) by the hardware's reciprocal (2 ulp).  The reciprocal of a denominator
// above 2^126 is 0 (the value is under 2^-119).  Below -126 the value is under
// 2^-174, and the quotient by an infinite denominator gives the 0 it rounds to; the
// argument is held there so that -inf gives 0 too (NaN stays NaN).
__device__ __forceinline__ float silu_fast(float x) {
  asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(x));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp2_approx(-kLog2e * x)));
  return x * r;
}

// act(x) in fp32; at -inf the limit (0 for all but the identity).  A template
// argument, so that a kernel holds the instructions of its own activation only: with
// all of them behind a switch in an unrolled epilogue, a short launch spent more
// time fetching instructions than computing.
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if (ACT == ITTT_ACT_RELU) return x < 0.f ? 0.f : x;  // NaN stays NaN
  if (ACT == ITTT_ACT_SILU) return silu_fast(x);
  if (ACT == ITTT_ACT_GELU)
    return x == -INFINITY ? 0.f : 0.5f * x * (1.f + erff(x * 0.70710678118654752f));
  if (ACT == ITTT_ACT_GELU_TANH) {
    const float t = 0.79788456080286536f * (x + 0.044715f * x * x * x);
    return x == -INFINITY ? 0.f : 0.5f * x * (1.f + tanhf(t));
  }
  return x;
}

// The same by a run-time act, out of line.
__device__ __noinline__ float activate_any(float x, int act) {
  switch (act) {
    case ITTT_ACT_RELU: return activate<ITTT_ACT_RELU>(x);
    case ITTT_ACT_SILU: return activate<ITTT_ACT_SILU>(x);
    case ITTT_ACT_GELU: return activate<ITTT_ACT_GELU>(x);
    case ITTT_ACT_GELU_TANH: return activate<ITTT_ACT_GELU_TANH>(x);
    default: return x;
  }
}

// Two fp32 values in one 64-bit register and the paired instructions on them
// (one issue slot for two products).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float x, float y) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Two neighbouring channels of a row.
__device__ __forceinline__ float2 load_two(const __nv_bfloat16* p) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 load_two(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ void store_two(__nv_bfloat16* p, float x, float y) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(x, y);
}
__device__ __forceinline__ void store_two(float* p, float x, float y) {
  *reinterpret_cast<float2*>(p) = make_float2(x, y);
}

// ------------------------------------------------------------------ linear

template <typename T_>
struct LinearArgs {
  const T_ *X, *W, *bias, *residual;
  T_* Y;
  long long ldx, ldr, ldy;
  int M, N, K, act;
};

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

// Bound by reading X and writing Y once, with the activation's two special-function
// results a value close behind: 8192 x 5120 in bf16 with four taps and silu 35.3 us, 4.75
// TB/s (torch's copy of the same bytes 27.2 us; 37.3 us with one channel an instruction
// and eight steps a thread).  A thread owns V neighbouring channels (16 bytes; 1
// where widths or alignment do not allow that) over `steps` times four tokens.  It
// holds the KT - 1 rows before and four more, and asks for the next four before it
// computes, so that loads and arithmetic overlap; a thread's first KT - 1 rows are
// the only ones read twice.
// The threads of token 0 also move the state: each reads its channels' state_in
// (nobody else does: the others start at token 8 or later) before it writes the same
// channels' state_out, so the two may be one buffer.
template <typename T_, int V, int KT, int ACT>
__global__ void __launch_bounds__(128, V > 1 && KT <= 4 ? 4 : 1)
    causal_conv_vec_kernel(const CausalConvArgs<T_> a, unsigned total, unsigned groups, unsigned runs,
                           int steps) {
  using Row = std::conditional_t<V == 1, T_, uint4>;
  constexpr int R = 4;  // tokens a step
  grid_dependency_wait();
  const unsigned e = blockIdx.x * 128u + threadIdx.x;
  if (e >= total) return;
  const unsigned rest = e / groups;
  const int c = static_cast<int>(e - rest * groups) * V;
  const int b = static_cast<int>(rest / runs);
  const int t0 = static_cast<int>(rest - unsigned(b) * runs) * steps * R;
  const int len = sequence_length(a.lengths, b, a.T);
  const T_* X = a.X + (long long)b * a.T * a.ldx + c;
  const T_* s_in = a.state_in ? a.state_in + (long long)b * (KT - 1) * a.d + c : nullptr;
  auto before = [&](int t) -> Row {  // the inputs of a token -(KT - 1) <= t < len
    if (t >= 0) return *reinterpret_cast<const Row*>(X + t * a.ldx);
    if (s_in) return *reinterpret_cast<const Row*>(s_in + (long long)(t + KT - 1) * a.d);
    return Row{};
  };
  if (t0 < len) {
    const int t_end = min(len, t0 + steps * R);
    Row rows[R + KT - 1], next[R];
    const T_* xp = X + t0 * a.ldx;
#pragma unroll
    for (int i = 0; i < R; ++i)
      next[i] = t0 + i < t_end ? *reinterpret_cast<const Row*>(xp + i * a.ldx) : Row{};
#pragma unroll
    for (int i = 0; i < KT - 1; ++i) rows[R + i] = before(t0 + i - (KT - 1));
    float bias[V];
    float w1[KT];                 // V == 1
    f32x2 w2[KT][(V + 1) / 2];    // V > 1
    {
      // the taps of V channels are V * KT contiguous elements
      const Row* wp = reinterpret_cast<const Row*>(a.w + (long long)c * KT);
      alignas(16) T_ taps[V * KT];
#pragma unroll
      for (int i = 0; i < KT; ++i) *reinterpret_cast<Row*>(taps + i * V) = __ldg(wp + i);
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        w1[j] = to_f32(taps[j]);
#pragma unroll
        for (int i = 0; i + 1 < V; i += 2)
          w2[j][i / 2] = pack2(to_f32(taps[i * KT + j]), to_f32(taps[(i + 1) * KT + j]));
      }
#pragma unroll
      for (int i = 0; i < V; ++i) bias[i] = a.bias ? to_f32(a.bias[c + i]) : 0.f;
    }
    T_* Y = a.Y + ((long long)b * a.T + t0) * a.ldy + c;
#pragma unroll 1
    for (int t = t0; t < t_end; t += R) {
#pragma unroll
      for (int i = 0; i < KT - 1; ++i) rows[i] = rows[R + i];
#pragma unroll
      for (int i = 0; i < R; ++i) rows[KT - 1 + i] = next[i];
      xp += R * a.ldx;
#pragma unroll
      for (int i = 0; i < R; ++i)
        next[i] = t + R + i < t_end ? *reinterpret_cast<const Row*>(xp + i * a.ldx) : Row{};
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (t + r < t_end) {
          float y[V];
          if (V == 1) {
            y[0] = bias[0];
#pragma unroll
            for (int j = 0; j < KT; ++j)
              y[0] = fmaf(w1[j], to_f32(*reinterpret_cast<const T_*>(&rows[r + j])), y[0]);
          } else {
            // two channels an instruction
#pragma unroll
            for (int i = 0; i + 1 < V; i += 2) {
              f32x2 acc = pack2(bias[i], bias[i + 1]);
#pragma unroll
              for (int j = 0; j < KT; ++j) {
                const float2 x = load_two(reinterpret_cast<const T_*>(&rows[r + j]) + i);
                acc = fma2(w2[j][i / 2], pack2(x.x, x.y), acc);
              }
              unpack2(acc, y[i], y[i + 1]);
            }
          }
          Row out;
          T_* o = reinterpret_cast<T_*>(&out);
          if (ACT == ITTT_ACT_SILU) {
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = silu_fast(y[i]);
          } else if (ACT != ITTT_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = activate_any(y[i], a.act);
          }
          if (V == 1) o[0] = from_f32<T_>(y[0]);
#pragma unroll
          for (int i = 0; i + 1 < V; i += 2) store_two(o + i, y[i], y[i + 1]);
          *reinterpret_cast<Row*>(Y + r * a.ldy) = out;
        }
      }
      Y += R * a.ldy;
    }
  }
  if (KT > 1 && t0 == 0 && a.state_out) {
    Row keep[KT > 1 ? KT - 1 : 1];
#pragma unroll
    for (int j = 0; j < KT - 1; ++j) keep[j] = before(len - (KT - 1) + j);
    T_* s_out = a.state_out + (long long)b * (KT - 1) * a.d + c;
#pragma unroll
    for (int j = 0; j < KT - 1; ++j) *reinterpret_cast<Row*>(s_out + (long long)j * a.d) = keep[j];
  }
}

// More than eight taps: one channel a thread, 16 tokens (or, in
// CTA row 0, the first k - 1 tokens and the state, with the same order of reads
// and writes).
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
    Y[t * a.ldy] = from_f32<T_>(activate_any(acc, a.act));
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

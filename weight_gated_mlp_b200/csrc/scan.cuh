// Kernels of the selective state space scan
//   h_t[c, n] = exp(s_t[c] A[c, n]) h_(t-1)[c, n] + s_t[c] u_t[c] B_t[n],
//   y_t[c]    = sum_n h_t[c, n] C_t[n] + D[c] u_t[c],  Y = y silu(z).
//
// One exponential per state element and token is the largest cost (the unit that
// computes it takes 16 a clock and SM), so no kernel computes one twice.
//
//   scan_serial_kernel  short calls and single tokens: lanes over the state, four
//       or eight elements a lane, token after token.  Bound by the state's bytes.
//   scan_chunk_kernel   prompts: 16 channels a CTA, 128 tokens at a time.  A
//       thread owns one channel and 8 consecutive tokens; for four state elements
//       at once it runs the recurrence from zero over its tokens, keeping the
//       exponentials, the CTA joins the 16 spans (a span's decay is
//       exp(A sum s), one exponential and one rounding for 8 tokens), and the
//       thread runs its tokens again from the true state, with the kept
//       exponentials, into y.  The lanes of a half warp are neighbouring channels,
//       so a row of U, delta, Z and Y is read in whole 32-byte sectors, and B and C
//       come from shared memory as broadcasts of four state elements.
#pragma once

#include "common.cuh"
#include "mixer.cuh"

namespace ittt {

constexpr float kLog2e = 1.4426950408889634f;

template <typename T_>
struct ScanArgs {
  const T_ *U, *delta, *Bm, *Cm, *Z;
  const float *A, *D, *dt_bias, *state_in;
  const int32_t* lengths;
  T_* Y;
  float* state_out;
  long long ldu, ldt, ldb, ldc, ldz, ldy;
  int B, T, d, N, G, softplus;
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// softplus(x) = max(x, 0) + log(1 + e^-|x|).  log(1 + e) = e q(e) on [0, 1], q of
// degree 9 fitted to least relative error (2^-23 in fp32 Horner steps): small
// steps keep their relative precision, which a logarithm of 1 + e would lose.
__device__ __forceinline__ float softplus_f32(float x) {
  const float e = exp2_approx(-kLog2e * fabsf(x));
  float q = -0.0032440319f;
  q = fmaf(q, e, 0.0198514927f);
  q = fmaf(q, e, -0.0569595918f);
  q = fmaf(q, e, 0.1060366035f);
  q = fmaf(q, e, -0.1530559659f);
  q = fmaf(q, e, 0.1967594028f);
  q = fmaf(q, e, -0.2495413423f);
  q = fmaf(q, e, 0.3332996368f);
  q = fmaf(q, e, -0.4999990165f);
  q = fmaf(q, e, 1.0f);
  // NaN stays NaN (fmaxf alone would drop it)
  return fmaf(q, e, x != x ? x : fmaxf(x, 0.f));
}

// z / (1 + e^-z) by the hardware's quotient (2 ulp; a denominator past 2^126 gives 0).
__device__ __forceinline__ float silu_gate(float z) {
  return __fdividef(z, 1.f + exp2_approx(-kLog2e * z));
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

// ------------------------------------------------------------ short calls

// NPL state elements a lane, `lanes` (a power of two) lanes a channel.
template <typename T_, int NPL>
__global__ void __launch_bounds__(128) scan_serial_kernel(const ScanArgs<T_> a, int lanes,
                                                          int aligned) {
  grid_dependency_wait();
  const long long gid = (blockIdx.x * 128ll + threadIdx.x) / lanes;
  const int sub = threadIdx.x & (lanes - 1);
  // every thread of a warp stays for the shuffles; those past the end repeat the last channel
  const bool real = gid < (long long)a.B * a.d;
  const long long w = real ? gid : (long long)a.B * a.d - 1;
  const int b = static_cast<int>(w / a.d), c = static_cast<int>(w % a.d);
  const int g = c / (a.d / a.G);
  const int n0 = sub * NPL;
  const int live = min(NPL, a.N - n0);  // elements of this lane (may be <= 0)
  const int len = sequence_length(a.lengths, b, a.T);
  const bool vec = aligned && live == NPL && (a.N & 3) == 0;
  float h[NPL], A2[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) h[i] = A2[i] = 0.f;
  if (vec) {
    const float4* Ap = reinterpret_cast<const float4*>(a.A + (long long)c * a.N + n0);
    const float4* hp =
        a.state_in ? reinterpret_cast<const float4*>(a.state_in + w * a.N + n0) : nullptr;
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
      const float4 v = __ldg(Ap + i / 4);
      A2[i] = v.x, A2[i + 1] = v.y, A2[i + 2] = v.z, A2[i + 3] = v.w;
      if (hp) {
        const float4 s = hp[i / 4];
        h[i] = s.x, h[i + 1] = s.y, h[i + 2] = s.z, h[i + 3] = s.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (i < live) {
        A2[i] = a.A[(long long)c * a.N + n0 + i];
        if (a.state_in) h[i] = a.state_in[w * a.N + n0 + i];
      }
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) A2[i] *= kLog2e;
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
  const float skip = a.D ? a.D[c] : 0.f;
  const long long row0 = (long long)b * a.T;
  // the lanes of a warp may belong to sequences of different lengths
  const int warp_len = __reduce_max_sync(0xffffffffu, len);
  for (int t = 0; t < warp_len; ++t) {
    float y = 0.f, u = 0.f;
    if (t < len) {
      const long long row = row0 + t;
      u = to_f32(a.U[row * a.ldu + c]);
      float s = to_f32(a.delta[row * a.ldt + c]) + bias;
      if (a.softplus) s = softplus_f32(s);
      const float su = s * u;
      const T_* Bp = a.Bm + row * a.ldb + (long long)g * a.N + n0;
      const T_* Cp = a.Cm + row * a.ldc + (long long)g * a.N + n0;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (i < live) {
          h[i] = fmaf(exp2_approx(s * A2[i]), h[i], su * to_f32(Bp[i]));
          y = fmaf(h[i], to_f32(Cp[i]), y);
        }
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (t < len && sub == 0 && real) {
      const long long row = row0 + t;
      if (a.D) y = fmaf(skip, u, y);
      if (a.Z) y *= silu_gate(to_f32(a.Z[row * a.ldz + c]));
      a.Y[row * a.ldy + c] = from_f32<T_>(y);
    }
  }
  if (a.state_out && real) {
    if (vec) {
      float4* hp = reinterpret_cast<float4*>(a.state_out + w * a.N + n0);
#pragma unroll
      for (int i = 0; i < NPL; i += 4) hp[i / 4] = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (i < live) a.state_out[w * a.N + n0 + i] = h[i];
    }
  }
}

// ---------------------------------------------------------------- prompts

constexpr int kScanCh = 16;                       // channels a CTA
constexpr int kScanSegs = 16;                     // spans of a chunk
constexpr int kScanK = 8;                         // tokens a span
constexpr int kScanChunk = kScanSegs * kScanK;    // tokens a chunk
constexpr int kScanThreads = kScanCh * kScanSegs;
constexpr int kScanSlab = 16;                     // state elements of B and C staged at once

// How the work of a call is cut.  A task is one channel block of one sequence
// over one run of tokens; tasks are handed out run by run.
struct ScanPlan {
  int blocks;      // channel blocks of one sequence (none crosses a group)
  int per_group;   // channel blocks of one group
  int runs;        // runs of run_tokens tokens (the last may be short)
  int run_tokens;  // a multiple of kScanChunk
  int chained;     // 1: a run starts from the state that the run before leaves in
                   // `carry`; 0: run r from carry[r - 1] (filled by scan_join_kernel)
  float* carry;    // chained: [B blocks][16][NP]; else [runs - 1][B, d, N]
  float* step_sum; // state pass: [runs - 1][B, d], the runs' sums of s
  unsigned* flags; // chained: [0] the next task, [1 + B blocks] runs finished
};

// Rows of the staged tiles: a span's 8 tokens side by side, the spans 16 (raw
// rows) or 4 (B and C in fp32) elements further apart than that, so that the two
// spans of a warp read different banks.
constexpr int kRawSpan = kScanK * kScanCh + 16;
constexpr int kRawTile = kScanSegs * kRawSpan;        // elements of one of U, delta, Z
constexpr int kSlabSpan = kScanK * kScanSlab + 4;
constexpr int kSlabTile = kScanSegs * kSlabSpan;      // fp32 elements of one of B, C
constexpr int kSlabRaw = kScanChunk * kScanSlab;      // bf16 elements of one of B, C

// Shared memory.  Two buffers of what arrives while the step before is computed
// (U, delta, Z of a chunk; 16 state elements of B and C: fp32 lands in its final
// place, bf16 is widened into one more tile), two buffers of the spans' end states
// and decays, the state and A log2(e) of the CTA's channels.
template <typename T_>
struct ScanShape {
  static constexpr bool WIDEN = sizeof(T_) == 2;
  static constexpr int RAW = 2 * 3 * kRawTile * int(sizeof(T_));
  static constexpr int BC = 2 * 2 * (WIDEN ? kSlabRaw * 2 : kSlabTile * 4);
  static constexpr int TILES = WIDEN ? 2 * kSlabTile * 4 : 0;
  static constexpr int ENDS = 2 * 2 * kScanThreads * 16;
};
__host__ __device__ constexpr int scan_np(int N) { return (N + 3) & ~3; }
template <typename T_>
__host__ __device__ constexpr int scan_smem_bytes(int N) {
  using S = ScanShape<T_>;
  return S::RAW + S::BC + S::TILES + S::ENDS + 2 * kScanCh * (scan_np(N) + 4) * 4;
}

// 16 bytes global -> shared, not waited for; zeros where valid is false.
__device__ __forceinline__ void copy16_async(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// What the copies of one operand may assume: 16-byte pieces of its rows.
template <typename T_>
__device__ __forceinline__ bool pieces_ok(const T_* p, long long ld, int unit) {
  constexpr int V = 16 / int(sizeof(T_));
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % V == 0 && unit % V == 0;
}

// [tokens][nch] of one of U, delta, Z into a raw tile (zeros elsewhere).
template <typename T_>
__device__ __forceinline__ void fetch_rows(T_* tile, const T_* src, long long ld, int tokens, int nch,
                                           bool pieces) {
  constexpr int V = 16 / int(sizeof(T_));
  if (pieces) {
    constexpr int P = kScanCh / V;
    static_assert(kScanChunk * P % kScanThreads == 0, "whole passes");
#pragma unroll
    for (int i = 0; i < kScanChunk * P / kScanThreads; ++i) {
      const int e = i * kScanThreads + static_cast<int>(threadIdx.x);
      const int t = e / P, c = (e % P) * V;
      const bool in = t < tokens && c < nch;
      copy16_async(tile + (t / kScanK) * kRawSpan + (t % kScanK) * kScanCh + c,
                   src + (in ? t * ld + c : 0), in);
    }
  } else {
    for (int e = threadIdx.x; e < kScanChunk * kScanCh; e += kScanThreads) {
      const int t = e / kScanCh, c = e % kScanCh;
      tile[(t / kScanK) * kRawSpan + (t % kScanK) * kScanCh + c] =
          (t < tokens && c < nch) ? src[t * ld + c] : from_f32<T_>(0.f);
    }
  }
}

// State elements [n0, n0 + 16) of B or C of a chunk's tokens (zeros behind the
// end and past N): fp32 into its final tile, bf16 as it is.
template <typename T_>
__device__ __forceinline__ void fetch_slab(T_* dst, const T_* src, long long ld, int tokens, int N,
                                           int n0, bool pieces) {
  constexpr int V = 16 / int(sizeof(T_)), P = kScanSlab / V;
  constexpr bool WIDEN = ScanShape<T_>::WIDEN;
  auto place = [](int t, int n) {
    return WIDEN ? t * kScanSlab + n : (t / kScanK) * kSlabSpan + (t % kScanK) * kScanSlab + n;
  };
  if (pieces) {
#pragma unroll
    for (int i = 0; i < kScanChunk * P / kScanThreads; ++i) {
      const int e = i * kScanThreads + static_cast<int>(threadIdx.x);
      const int t = e / P, n = (e % P) * V;
      const bool in = t < tokens && n0 + n < N;
      copy16_async(dst + place(t, n), src + (in ? t * ld + n0 + n : 0), in);
    }
  } else {
    for (int e = threadIdx.x; e < kSlabRaw; e += kScanThreads) {
      const int t = e / kScanSlab, n = e % kScanSlab;
      dst[place(t, n)] = (t < tokens && n0 + n < N) ? src[t * ld + n0 + n] : from_f32<T_>(0.f);
    }
  }
}

// bf16 B or C into its fp32 tile: eight elements a thread.
__device__ __forceinline__ void widen_slab(float* tile, const __nv_bfloat16* raw) {
  static_assert(kSlabRaw == 8 * kScanThreads, "eight elements a thread");
  const int e = threadIdx.x * 8, t = e / kScanSlab, n = e % kScanSlab;
  const uint4 v = *reinterpret_cast<const uint4*>(raw + e);
  float4* dst = reinterpret_cast<float4*>(tile + (t / kScanK) * kSlabSpan + (t % kScanK) * kScanSlab + n);
  dst[0] = make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  dst[1] = make_float4(__uint_as_float(v.z << 16), __uint_as_float(v.z & 0xffff0000u),
                       __uint_as_float(v.w << 16), __uint_as_float(v.w & 0xffff0000u));
}
__device__ __forceinline__ void widen_slab(float*, const float*) {}

// STATE_ONLY: the first of the two passes of a call that is split over time: every
// run from a zero state, its end state and sum of steps written, no outputs.
template <typename T_, bool STATE_ONLY>
__global__ void __launch_bounds__(kScanThreads, 2)
    scan_chunk_kernel(const ScanArgs<T_> a, const ScanPlan pl, unsigned long long wait_ns) {
  using S = ScanShape<T_>;
  extern __shared__ __align__(16) uint8_t scan_smem[];
  const int NP = scan_np(a.N);
  T_* raw = reinterpret_cast<T_*>(scan_smem);                       // [2][3][kRawTile]
  T_* bc = reinterpret_cast<T_*>(scan_smem + S::RAW);               // [2][2][one slab]
  constexpr int kBc = S::WIDEN ? kSlabRaw : kSlabTile;
  float* tiles = reinterpret_cast<float*>(scan_smem + S::RAW + S::BC);
  float4* ends = reinterpret_cast<float4*>(scan_smem + S::RAW + S::BC + S::TILES);
  float4* decays = ends + 2 * kScanThreads;                         // both [2][segs][ch]
  float* state = reinterpret_cast<float*>(decays + 2 * kScanThreads);  // [ch][NP + 4]
  float* A2s = state + kScanCh * (NP + 4);
  __shared__ int next_task, aborted;

  const int tid = threadIdx.x;
  const int ch = tid & 15, seg = tid >> 4;
  const int groups = a.B * pl.blocks;
  const int tasks = groups * (STATE_ONLY ? pl.runs - 1 : pl.runs);
  const int dg = a.d / a.G;
  const bool pieces_u = pieces_ok(a.U, a.ldu, dg);
  const bool pieces_t = pieces_ok(a.delta, a.ldt, dg);
  const bool pieces_z = pieces_ok(a.Z, a.ldz, dg);
  const bool pieces_b = pieces_ok(a.Bm, a.ldb, a.N), pieces_c = pieces_ok(a.Cm, a.ldc, a.N);
  if (tid == 0) aborted = 0;
  grid_dependency_wait();

  for (int turn = 0;; ++turn) {
    // handed out by a counter, in order: what a task waits for has been taken by
    // a CTA that runs already, so the waits end whatever else is on the GPU
    int task;
    __syncthreads();  // the task before is done with the shared memory
    if (!STATE_ONLY && pl.chained && pl.runs > 1) {
      if (tid == 0) next_task = static_cast<int>(atomicAdd(pl.flags, 1u));
      __syncthreads();
      task = next_task;
    } else {
      task = static_cast<int>(blockIdx.x) + turn * static_cast<int>(gridDim.x);
    }
    if (task >= tasks) return;
    const int run = task / groups, gb = task - run * groups;
    const int b = gb / pl.blocks, blk = gb - b * pl.blocks;
    const int g = blk / pl.per_group;
    const int in_group = (blk - g * pl.per_group) * kScanCh;
    const int c0 = g * dg + in_group;
    const int nch = min(kScanCh, dg - in_group);
    const bool mine = ch < nch;
    const int c = c0 + (mine ? ch : 0);
    const int len = sequence_length(a.lengths, b, a.T);
    const int t_begin = run * pl.run_tokens;
    const int t_end = min(len, t_begin + pl.run_tokens);
    const bool first = run == 0;
    const bool last = len <= t_begin + pl.run_tokens;  // the run that holds the sequence's end
    if (!first && t_begin >= len) {
      if (!STATE_ONLY) continue;
      // a run behind the end joins as nothing
      for (int e = tid; e < nch * a.N; e += kScanThreads)
        pl.carry[((long long)run * a.B + b) * a.d * a.N + (long long)c0 * a.N + e] = 0.f;
      if (tid < nch) pl.step_sum[((long long)run * a.B + b) * a.d + c0 + tid] = 0.f;
      continue;
    }

    const long long row0 = (long long)b * a.T;
    // the copies of one step: a chunk's rows with its first slab, or a further slab
    auto fetch = [&](int t0, int n0, int rows_buf, int bc_buf) {
      const int tokens = min(kScanChunk, t_end - t0);
      const long long row = row0 + t0;
      if (n0 == 0) {
        T_* r = raw + rows_buf * 3 * kRawTile;
        fetch_rows(r, a.U + row * a.ldu + c0, a.ldu, tokens, nch, pieces_u);
        fetch_rows(r + kRawTile, a.delta + row * a.ldt + c0, a.ldt, tokens, nch, pieces_t);
        if (!STATE_ONLY && a.Z)
          fetch_rows(r + 2 * kRawTile, a.Z + row * a.ldz + c0, a.ldz, tokens, nch, pieces_z);
      }
      T_* dst = bc + bc_buf * 2 * kBc;
      const long long gn = (long long)g * a.N;
      fetch_slab(dst, a.Bm + row * a.ldb + gn, a.ldb, tokens, a.N, n0, pieces_b);
      if (!STATE_ONLY)
        fetch_slab(dst + kBc, a.Cm + row * a.ldc + gn, a.ldc, tokens, a.N, n0, pieces_c);
      copy_commit();
    };
    if (t_begin < t_end) fetch(t_begin, 0, 0, 0);

    if (!STATE_ONLY && pl.chained && !first) {
      if (tid == 0) {
        const WaitCtl wc{&aborted, wait_ns};
        flag_wait_geq(pl.flags + 1 + gb, static_cast<uint32_t>(run), wc);
      }
      __syncthreads();
      if (*const_cast<volatile int*>(&aborted)) {
        copy_wait_all();
        return;
      }
    }
    for (int e = tid; e < kScanCh * NP; e += kScanThreads) {
      const int i = e / NP, n = e - i * NP;
      float h = 0.f, A2 = 0.f;
      if (i < nch && n < a.N) {
        A2 = a.A[(long long)(c0 + i) * a.N + n] * kLog2e;
        const long long at = ((long long)b * a.d + c0 + i) * a.N + n;
        if (!STATE_ONLY) {
          if (first) h = a.state_in ? a.state_in[at] : 0.f;
          else if (pl.chained) h = __ldcg(pl.carry + ((long long)gb * kScanCh + i) * NP + n);
          else h = pl.carry[(long long)(run - 1) * a.B * a.d * a.N + at];
        }
      }
      state[i * (NP + 4) + n] = h;
      A2s[i * (NP + 4) + n] = A2;
    }

    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
    const float skip = a.D ? a.D[c] : 0.f;
    float steps_total = 0.f;  // STATE_ONLY: this thread's share of the run's sum of s
    int rows_buf = 0, bc_buf = 0;

    for (int t0 = t_begin; t0 < t_end; t0 += kScanChunk, rows_buf ^= 1) {
      const int tokens = min(kScanChunk, t_end - t0);
      const int mine0 = seg * kScanK;  // this thread's first token of the chunk
      f32x2 s2[kScanK], su2[kScanK], y2[kScanK];
      float sum = 0.f;
      const T_* rows = raw + rows_buf * 3 * kRawTile + seg * kRawSpan + ch;

      for (int n0 = 0; n0 < NP; n0 += kScanSlab, bc_buf ^= 1) {
        copy_wait_all();
        __syncthreads();  // this step's copies are in; the readers of the step before are done
        if (n0 + kScanSlab < NP) fetch(t0, n0 + kScanSlab, rows_buf, bc_buf ^ 1);
        else if (t0 + kScanChunk < t_end) fetch(t0 + kScanChunk, 0, rows_buf ^ 1, bc_buf ^ 1);
        const float *Bs, *Cs;
        if (S::WIDEN) {
          widen_slab(tiles, bc + bc_buf * 2 * kBc);
          if (!STATE_ONLY) widen_slab(tiles + kSlabTile, bc + (bc_buf * 2 + 1) * kBc);
          Bs = tiles;
        } else {
          Bs = reinterpret_cast<const float*>(bc + bc_buf * 2 * kBc);
        }
        Cs = Bs + kSlabTile;
        if (n0 == 0) {
#pragma unroll
          for (int k = 0; k < kScanK; ++k) {
            const float u = to_f32(rows[k * kScanCh]);
            float s = to_f32(rows[kRawTile + k * kScanCh]) + bias;
            if (a.softplus) s = softplus_f32(s);
            if (mine0 + k >= tokens) s = 0.f;  // behind the end: the state passes unchanged
            sum += s;
            s2[k] = pack2(s, s);
            const float su = s * u;
            su2[k] = pack2(su, su);
            y2[k] = pack2(a.D ? skip * u : 0.f, 0.f);  // no 0 * inf where there is no skip
          }
          if (STATE_ONLY) steps_total += sum;
        }
        if (S::WIDEN) __syncthreads();
        const int blocks = min(kScanSlab, NP - n0) >> 2;
#pragma unroll 1
        for (int nb = 0; nb < blocks; ++nb) {
          const int buf = (nb & 1) * kScanThreads;
          const float4 A4 = *reinterpret_cast<const float4*>(A2s + ch * (NP + 4) + n0 + nb * 4);
          const f32x2 A01 = pack2(A4.x, A4.y), A23 = pack2(A4.z, A4.w);
          const float* bp = Bs + seg * kSlabSpan + nb * 4;
          f32x2 a01[kScanK], a23[kScanK];
          f32x2 h01 = 0ull, h23 = 0ull;
#pragma unroll
          for (int k = 0; k < kScanK; ++k) {
            const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(bp + k * kScanSlab);
            float x0, x1, x2, x3;
            unpack2(mul2(s2[k], A01), x0, x1);
            unpack2(mul2(s2[k], A23), x2, x3);
            a01[k] = pack2(exp2_approx(x0), exp2_approx(x1));
            a23[k] = pack2(exp2_approx(x2), exp2_approx(x3));
            h01 = fma2(a01[k], h01, mul2(su2[k], b4.x));
            h23 = fma2(a23[k], h23, mul2(su2[k], b4.y));
          }
          float4 e4;
          unpack2(h01, e4.x, e4.y);
          unpack2(h23, e4.z, e4.w);
          ends[buf + tid] = e4;
          decays[buf + tid] = make_float4(exp2_approx(sum * A4.x), exp2_approx(sum * A4.y),
                                          exp2_approx(sum * A4.z), exp2_approx(sum * A4.w));
          __syncthreads();
          if (tid < kScanCh * 4) {
            // one state element of one channel: the spans in order
            float* e = reinterpret_cast<float*>(ends + buf) + tid;
            const float* p = reinterpret_cast<const float*>(decays + buf) + tid;
            float* st = state + (tid >> 2) * (NP + 4) + n0 + nb * 4 + (tid & 3);
            float h = *st;
#pragma unroll
            for (int i = 0; i < kScanSegs; ++i) {
              const float end = e[i * kScanCh * 4];
              if (!STATE_ONLY) e[i * kScanCh * 4] = h;
              h = fmaf(p[i * kScanCh * 4], h, end);
            }
            *st = h;
          }
          if (STATE_ONLY) continue;  // two buffers: the next block writes the other one
          __syncthreads();
          const ulonglong2 start = *reinterpret_cast<const ulonglong2*>(ends + buf + tid);
          h01 = start.x;
          h23 = start.y;
          const float* cp = Cs + seg * kSlabSpan + nb * 4;
#pragma unroll
          for (int k = 0; k < kScanK; ++k) {
            const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(bp + k * kScanSlab);
            const ulonglong2 c4 = *reinterpret_cast<const ulonglong2*>(cp + k * kScanSlab);
            h01 = fma2(a01[k], h01, mul2(su2[k], b4.x));
            h23 = fma2(a23[k], h23, mul2(su2[k], b4.y));
            y2[k] = fma2(h01, c4.x, y2[k]);
            y2[k] = fma2(h23, c4.y, y2[k]);
          }
        }
      }

      if (!STATE_ONLY && mine) {
        T_* yp = a.Y + (row0 + t0 + mine0) * a.ldy + c;
#pragma unroll
        for (int k = 0; k < kScanK; ++k, yp += a.ldy) {
          if (mine0 + k < tokens) {
            float lo, hi;
            unpack2(y2[k], lo, hi);
            float y = lo + hi;
            if (a.Z) y *= silu_gate(to_f32(rows[2 * kRawTile + k * kScanCh]));
            *yp = from_f32<T_>(y);
          }
        }
      }
    }

    __syncthreads();  // the state of the run's last token is complete
    if (STATE_ONLY) {
      float* sums = reinterpret_cast<float*>(ends);
      sums[tid] = steps_total;
      __syncthreads();
      const long long at = ((long long)run * a.B + b) * a.d + c0;
      if (tid < nch) {
        float s = 0.f;
        for (int i = 0; i < kScanSegs; ++i) s += sums[i * kScanCh + tid];
        pl.step_sum[at + tid] = s;
      }
      for (int e = tid; e < nch * a.N; e += kScanThreads)
        pl.carry[at * a.N + e] = state[(e / a.N) * (NP + 4) + e % a.N];
      continue;
    }
    if (last) {
      if (a.state_out)
        for (int e = tid; e < nch * a.N; e += kScanThreads)
          a.state_out[((long long)b * a.d + c0) * a.N + e] = state[(e / a.N) * (NP + 4) + e % a.N];
    } else if (pl.chained) {
      for (int e = tid; e < kScanCh * NP; e += kScanThreads)
        pl.carry[(long long)gb * kScanCh * NP + e] = state[(e / NP) * (NP + 4) + e % NP];
      __threadfence();
      __syncthreads();
      if (tid == 0) red_release_gpu_add(pl.flags + 1 + gb, 1u);
    }
  }
}

// Between the two passes: carry[run] becomes the state before run, from the runs'
// own end states and sums of steps.
template <typename T_>
__global__ void __launch_bounds__(256) scan_join_kernel(const ScanArgs<T_> a, const ScanPlan pl) {
  grid_dependency_wait();
  const long long e = blockIdx.x * 256ll + threadIdx.x, total = (long long)a.B * a.d * a.N;
  if (e >= total) return;
  const long long bd = e / a.N;
  const float A2 = a.A[(bd % a.d) * a.N + e % a.N] * kLog2e;
  float h = a.state_in ? a.state_in[e] : 0.f;
  for (int r = 0; r < pl.runs - 1; ++r) {
    const float end = pl.carry[r * total + e];
    h = fmaf(exp2_approx(pl.step_sum[(long long)r * a.B * a.d + bd] * A2), h, end);
    pl.carry[r * total + e] = h;  // the state before run r + 1
  }
}

}  // namespace ittt

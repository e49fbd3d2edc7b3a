// Kernels of the selective state space scan
//   h_t[c, n] = exp(s_t[c] A[c, n]) h_(t-1)[c, n] + s_t[c] u_t[c] B_t[n],
//   y_t[c]    = sum_n h_t[c, n] C_t[n] + D[c] u_t[c],  Y = y silu(z).
//
// One exponential per state element and token is the largest cost (the unit that
// computes it takes 16 a clock and SM), so no pass over the tokens computes one twice.  A
// call that is cut into independent runs makes two passes over all runs but the last,
// and a join costs one exponential more for 8 tokens.
//
//   scan_token_kernel   single tokens: lanes over the state, sequence after sequence.
//       Bound by the state's bytes (64 sequences of 5120 x 16: 13.7 us, 6.9 us at HBM's
//       copy rate).
//   scan_serial_kernel  short calls: lanes over the state, four or eight elements a
//       lane, four tokens at a time.  Bound by the latency of one token after the other
//       (0.24 us each), or by the exponentials where there are many sequences.
//   scan_chunk_kernel   prompts: 256 tokens at a time.  A thread owns two neighbouring
//       channels and 8 consecutive tokens, a warp two channels and the whole chunk, a
//       CTA one or two such pairs of channels a warp.  For four state elements at once a
//       thread runs the recurrence of its tokens from zero into y, and keeps for each
//       token g = C times the decay since the span's start; the warp joins its 32 spans
//       (a span's decay is exp(A sum s): one exponential and one rounding for 8
//       tokens); then y += g h with the span's true start h.  Two channels a thread halve
//       what a state element costs in shared-memory reads of B and C (32 words a
//       clock and SM, however many lanes read the same word), and the joins stay
//       inside a warp, so the CTA meets four times a chunk only.
//       8192 x 5120 x 16 in bf16: 480 us, where the exponentials alone need 150 us and
//       the bytes 51 us.  About 15 instructions an element go out in 56% of the issue
//       slots; the exponentials' unit is 40% busy.  What remains is latency: a warp's
//       join is a chain of shuffles, and three CTAs an SM (the registers' limit) do
//       not cover it.
#pragma once

#include "common.cuh"
#include "mixer.cuh"

namespace ittt {

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

// ------------------------------------------------------------ short calls

// Four neighbouring values as they are in memory.  The short kernels issue every
// load before the first use of one, without branches between them: a conversion or a
// condition after each load would wait for it.
template <typename T_>
struct alignas(4 * sizeof(T_)) Quad {
  T_ v[4];
  // VEC: one load of four values; else the first `live` >= 1 of them, the last repeated.
  template <bool VEC>
  __device__ __forceinline__ void load(const T_* p, int live) {
    if (VEC) {
      *this = *reinterpret_cast<const Quad*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = p[min(i, live - 1)];
    }
  }
};

// NPL state elements a lane, `lanes` (a power of two) lanes a channel, four tokens at
// a time: the loads of the next four are under way while four are computed.
template <typename T_, int NPL, bool VEC>
__global__ void __launch_bounds__(128) scan_serial_kernel(const ScanArgs<T_> a, int lanes) {
  constexpr int Q = NPL / 4, TOK = 4;
  grid_dependency_wait();
  const long long gid = (blockIdx.x * 128ll + threadIdx.x) / lanes;
  const int sub = threadIdx.x & (lanes - 1);
  // every thread of a warp stays for the shuffles; those past the end repeat the last channel
  const bool real = gid < (long long)a.B * a.d;
  const long long w = real ? gid : (long long)a.B * a.d - 1;
  const int b = static_cast<int>(w / a.d), c = static_cast<int>(w % a.d);
  const int g = c / (a.d / a.G);
  const int len = sequence_length(a.lengths, b, a.T);
  int n0[Q], live[Q];  // first element and number of elements (may be <= 0) of each quad
  float h[Q][4] = {}, A2[Q][4];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    live[q] = a.N - (sub * NPL + 4 * q);
    n0[q] = live[q] > 0 ? sub * NPL + 4 * q : 0;  // a quad past the end reads the first and drops it
    Quad<float> v;
    v.load<VEC>(a.A + (long long)c * a.N + n0[q], live[q] > 0 ? live[q] : a.N);
#pragma unroll
    for (int j = 0; j < 4; ++j) A2[q][j] = v.v[j] * kLog2e;
    if (a.state_in) {
      v.load<VEC>(a.state_in + w * a.N + n0[q], live[q] > 0 ? live[q] : a.N);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[q][j] = v.v[j];
    }
  }
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
  const float skip = a.D ? a.D[c] : 0.f;
  const long long row0 = (long long)b * a.T;
  // the lanes of a warp may belong to sequences of different lengths
  const int warp_len = __reduce_max_sync(0xffffffffu, len);
  if (warp_len > 0) {
    T_ u[TOK], s[TOK], z[TOK];
    Quad<T_> Bq[TOK][Q], Cq[TOK][Q];
    const T_* zp = a.Z ? a.Z : a.U;  // a row of something where there is no gate
    const long long ldz = a.Z ? a.ldz : a.ldu;
    // tokens behind the end repeat the last one (an empty sequence its first row) and are dropped
    auto load = [&](int t0) {
#pragma unroll
      for (int i = 0; i < TOK; ++i) {
        const long long row = row0 + max(min(t0 + i, len - 1), 0);
        u[i] = a.U[row * a.ldu + c];
        s[i] = a.delta[row * a.ldt + c];
        z[i] = zp[row * ldz + c];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const long long at = (long long)g * a.N + n0[q];
          Bq[i][q].template load<VEC>(a.Bm + row * a.ldb + at, live[q] > 0 ? live[q] : a.N);
          Cq[i][q].template load<VEC>(a.Cm + row * a.ldc + at, live[q] > 0 ? live[q] : a.N);
        }
      }
    };
    load(0);
    for (int t0 = 0; t0 < warp_len; t0 += TOK) {
      float uf[TOK], sf[TOK], zf[TOK], Bf[TOK][Q][4], Cf[TOK][Q][4], y[TOK];
#pragma unroll
      for (int i = 0; i < TOK; ++i) {
        uf[i] = to_f32(u[i]);
        sf[i] = to_f32(s[i]) + bias;
        zf[i] = to_f32(z[i]);
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            Bf[i][q][j] = to_f32(Bq[i][q].v[j]);
            Cf[i][q][j] = to_f32(Cq[i][q].v[j]);
          }
      }
      load(t0 + TOK);
#pragma unroll
      for (int i = 0; i < TOK; ++i) {
        const float st = a.softplus ? softplus_f32(sf[i]) : sf[i];
        const float su = st * uf[i];
        const bool in = t0 + i < len;
        y[i] = 0.f;
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float hn = fmaf(exp2_approx(st * A2[q][j]), h[q][j], su * Bf[i][q][j]);
            if (in && j < live[q]) {
              h[q][j] = hn;
              y[i] = fmaf(hn, Cf[i][q][j], y[i]);
            }
          }
      }
      for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < TOK; ++i) y[i] += __shfl_xor_sync(0xffffffffu, y[i], o);
#pragma unroll
      for (int i = 0; i < TOK; ++i)
        if (real && t0 + i < len && (i & (lanes - 1)) == sub) {
          float v = y[i];
          if (a.D) v = fmaf(skip, uf[i], v);
          if (a.Z) v *= silu_fast(zf[i]);
          a.Y[(row0 + t0 + i) * a.ldy + c] = from_f32<T_>(v);
        }
    }
  }
  if (a.state_out && real) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float* p = a.state_out + w * a.N + n0[q];
      if (VEC && live[q] > 0) {
        *reinterpret_cast<float4*>(p) = make_float4(h[q][0], h[q][1], h[q][2], h[q][3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < live[q]) p[j] = h[q][j];
      }
    }
  }
}

// Single tokens (N <= 128): four state elements a lane of one channel.  A thread keeps
// its channel (A, D and the bias are read once) and walks over the sequences
// blockIdx.y, blockIdx.y + gridDim.y, ..., the next one's loads under way while one is
// computed.  Bound by reading and writing the state.
template <typename T_, bool VEC>
__global__ void __launch_bounds__(128) scan_token_kernel(const ScanArgs<T_> a, int lanes) {
  grid_dependency_wait();
  const int gid = static_cast<int>((blockIdx.x * 128ll + threadIdx.x) / lanes);
  const int sub = threadIdx.x & (lanes - 1);
  // every thread of a warp stays for the shuffles; those past the end repeat the last channel
  const bool real = gid < a.d;
  const int c = real ? gid : a.d - 1;
  const int g = c / (a.d / a.G);
  const int live = a.N - 4 * sub;                 // elements of this lane's quad (may be <= 0)
  const int n0 = live > 0 ? 4 * sub : 0, some = live > 0 ? live : a.N;
  const long long cn = (long long)c * a.N + n0, gn = (long long)g * a.N + n0;
  const T_* zp = a.Z ? a.Z : a.U;  // a row of something where there is no gate
  const long long ldz = a.Z ? a.ldz : a.ldu;
  const float* sp = a.state_in ? a.state_in : a.A;
  const long long sequence = a.state_in ? (long long)a.d * a.N : 0;
  struct Item {
    Quad<float> h;
    Quad<T_> B, C;
    T_ u, s, z;
    int len;
  } next;
  auto load = [&](int b) {
    const long long row = min(b, a.B - 1);  // past the batch: the last sequence again
    next.h.template load<VEC>(sp + row * sequence + cn, some);
    next.B.template load<VEC>(a.Bm + row * a.ldb + gn, some);
    next.C.template load<VEC>(a.Cm + row * a.ldc + gn, some);
    next.u = a.U[row * a.ldu + c];
    next.s = a.delta[row * a.ldt + c];
    next.z = zp[row * ldz + c];
    next.len = a.lengths ? a.lengths[row] : 1;
  };
  load(blockIdx.y);
  Quad<float> A;
  A.load<VEC>(a.A + cn, some);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
  const float skip = a.D ? a.D[c] : 0.f;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    Item now = next;
    load(b + gridDim.y);
    const bool on = real && now.len > 0;
    const float uf = to_f32(now.u);
    float st = to_f32(now.s) + bias;
    if (a.softplus) st = softplus_f32(st);
    const float su = st * uf;
    float y = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float before = a.state_in ? now.h.v[j] : 0.f;
      const float after = fmaf(exp2_approx(st * (A.v[j] * kLog2e)), before, su * to_f32(now.B.v[j]));
      if (j < live) y = fmaf(after, to_f32(now.C.v[j]), y);
      now.h.v[j] = on ? after : before;  // an empty sequence passes its state through
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (on && sub == 0) {
      if (a.D) y = fmaf(skip, uf, y);
      if (a.Z) y *= silu_fast(to_f32(now.z));
      a.Y[b * a.ldy + c] = from_f32<T_>(y);
    }
    if (a.state_out && real) {
      float* p = a.state_out + (long long)b * a.d * a.N + cn;
      if (VEC && live > 0) {
        *reinterpret_cast<Quad<float>*>(p) = now.h;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < live) p[j] = now.h.v[j];
      }
    }
  }
}

// ---------------------------------------------------------------- prompts

// Four warps, two pairs of state elements at once, and in bf16 168 registers a thread
// and three CTAs an SM.  8192 x 5120 x 16, one pass, each against 470 us in the build it
// was tried in: one pair at once 491 us, with 128 registers and four CTAs 534 us (584 us
// with two pairs, which then spill), eight warps and 128 registers 514 us, 255 registers
// and two CTAs 532 us, spans of four tokens 517 us.  fp32 holds twice the values of B and
// C and wants the registers: 81 us with two CTAs for 1667 tokens x 1000 x 32, 105 us with
// three.
constexpr int kScanWarps = 4;
constexpr int kScanThreads = 32 * kScanWarps;
// Channels a CTA: a warp takes P pairs of channels one after the other.  Two halve
// what staging B and C costs a channel (8 x 1024 x 5120 x 16: 436 us, 474 with one);
// one makes twice as many tasks (1 x 8192 x 5120: 480 us, 543 with two, whose 320
// channel blocks leave CTAs without work).  Two are for a state of one slab of B and C,
// which the second finds laid out.
__host__ __device__ constexpr int scan_ch(int P) { return 2 * kScanWarps * P; }
constexpr int kScanK = 8;                // tokens a span, one span a lane
constexpr int kScanChunk = 32 * kScanK;  // tokens a chunk
constexpr int kScanJ = 2;                // pairs of state elements at once

// How the work of a call is cut.  A task is one channel block of one sequence
// over one run of tokens; tasks are handed out run by run.
struct ScanPlan {
  int blocks;      // channel blocks of one sequence (none crosses a group)
  int per_group;   // channel blocks of one group
  int runs;        // runs of run_tokens tokens (the last may be short)
  int run_tokens;  // a multiple of kScanChunk
  int chained;     // 1: a run starts from the state that the run before leaves in
                   // `carry`; 0: run r from carry[r] (filled by scan_join_kernel), run 0
                   // too, since state_in may be the state_out that the last run's CTA,
                   // which nothing orders behind run 0's, writes
  float* carry;    // chained: [B blocks][channels a block, NP]; else [runs][B, d, N]
  float* step_sum; // state pass: [runs - 1][B, d], the runs' sums of s
  unsigned* flags; // chained: [0] the next task, [1 + B blocks] runs finished
};

// A slab: the 32 bytes of state elements of B and C that are staged at once (16
// bf16, 8 fp32).  Staged rows arrive as they are; B and C are then laid out as
// [pair of state elements][span][token], so that a lane reads the pair of 4 (or 2)
// tokens with one 16-byte load; the spans stand 12 (20) words apart, which puts the
// eight lanes of a quarter warp on different banks.
template <typename T_, int P>
struct ScanShape {
  static constexpr int CH = scan_ch(P);                      // channels
  static constexpr int ES = int(sizeof(T_));
  static constexpr int SLAB = 32 / ES;                       // state elements
  static constexpr int CTAS = ES == 2 ? 3 : 2;               // CTAs an SM
  static constexpr int PAIRS = SLAB / 2;
  static constexpr int ROW_SPAN = kScanK * CH + 16 / ES;  // elements between spans of raw rows
  static constexpr int ROW_TILE = 32 * ROW_SPAN;
  static constexpr int PAIR_SPAN = kScanK * 2 * ES / 4 + 4;  // words between spans of laid out pairs
  static constexpr int PAIR_TILE = 32 * PAIR_SPAN;           // words of one pair
  static constexpr int ROWS = 3 * ROW_TILE * ES;             // bytes: U, delta, Z (and Y)
  static constexpr int RAW = 2 * kScanChunk * 32;            // bytes: B and C as they come
  static constexpr int TILES = 2 * PAIRS * PAIR_TILE * 4;    // bytes: B and C laid out
};
// A join: a lane takes one of the 4 J state elements (of two channels) that are
// computed at once, over kJoinSpans neighbouring spans; 32 / (4 J) lanes share one.
constexpr int kJoinSpans = 4 * kScanJ;
constexpr int kEndsSpan = 4 * kScanJ;                       // floats of a span's end states
constexpr int kEndsGroup = kJoinSpans * kEndsSpan + kEndsSpan;  // the groups on different banks
constexpr int kEndsWarp = 32 / kJoinSpans * kEndsGroup;
__host__ __device__ constexpr int scan_np(int N) { return (N + 2 * kScanJ - 1) / (2 * kScanJ) * (2 * kScanJ); }
template <typename T_, int P>
__host__ __device__ constexpr int scan_smem_bytes(int N) {
  using S = ScanShape<T_, P>;
  return S::ROWS + S::RAW + S::TILES + kScanWarps * kEndsWarp * 4 + 2 * S::CH * scan_np(N) * 4 +
         3 * S::CH * 4;
}

// 16 bytes global -> shared, not waited for; zeros where valid is false.
__device__ __forceinline__ void copy16_async(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most N of this thread's committed groups are still on their way.
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What the copies of one operand may assume: 16-byte pieces of its rows.
template <typename T_>
__device__ __forceinline__ bool pieces_ok(const T_* p, long long ld, int unit) {
  constexpr int V = 16 / int(sizeof(T_));
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % V == 0 && unit % V == 0;
}

// [tokens][nch] of one of U, delta, Z into a tile of rows (zeros elsewhere).
template <typename T_, int PASSES>
__device__ __forceinline__ void fetch_rows(T_* tile, const T_* src, long long ld, int tokens, int nch,
                                           bool pieces) {
  using S = ScanShape<T_, PASSES>;
  constexpr int V = 16 / S::ES, P = S::CH / V;
  if (pieces) {
#pragma unroll
    for (int i = 0; i < kScanChunk * P / kScanThreads; ++i) {
      const int e = i * kScanThreads + static_cast<int>(threadIdx.x);
      const int t = e / P, c = (e % P) * V;
      const bool in = t < tokens && c < nch;
      copy16_async(tile + (t / kScanK) * S::ROW_SPAN + (t % kScanK) * S::CH + c,
                   src + (in ? t * ld + c : 0), in);
    }
  } else {
    for (int e = threadIdx.x; e < kScanChunk * S::CH; e += kScanThreads) {
      const int t = e / S::CH, c = e % S::CH;
      tile[(t / kScanK) * S::ROW_SPAN + (t % kScanK) * S::CH + c] =
          (t < tokens && c < nch) ? src[t * ld + c] : from_f32<T_>(0.f);
    }
  }
}

// A tile of rows to Y: the counterpart of fetch_rows.
template <typename T_, int PASSES>
__device__ __forceinline__ void store_rows(T_* dst, const T_* tile, long long ld, int tokens, int nch,
                                           bool pieces) {
  using S = ScanShape<T_, PASSES>;
  constexpr int V = 16 / S::ES, P = S::CH / V;
  if (pieces) {
#pragma unroll
    for (int i = 0; i < kScanChunk * P / kScanThreads; ++i) {
      const int e = i * kScanThreads + static_cast<int>(threadIdx.x);
      const int t = e / P, c = (e % P) * V;
      if (t < tokens && c < nch)
        *reinterpret_cast<uint4*>(dst + t * ld + c) = *reinterpret_cast<const uint4*>(
            tile + (t / kScanK) * S::ROW_SPAN + (t % kScanK) * S::CH + c);
    }
  } else {
    for (int e = threadIdx.x; e < kScanChunk * S::CH; e += kScanThreads) {
      const int t = e / S::CH, c = e % S::CH;
      if (t < tokens && c < nch)
        dst[t * ld + c] = tile[(t / kScanK) * S::ROW_SPAN + (t % kScanK) * S::CH + c];
    }
  }
}

// The slab [n0, n0 + SLAB) of B or C of a chunk's tokens, as it comes: [token][SLAB]
// (zeros behind the end and past N).
template <typename T_, int PASSES>
__device__ __forceinline__ void fetch_slab(T_* dst, const T_* src, long long ld, int tokens, int N,
                                           int n0, bool pieces) {
  using S = ScanShape<T_, PASSES>;
  constexpr int V = 16 / S::ES;
  if (pieces) {
#pragma unroll
    for (int i = 0; i < 2 * kScanChunk / kScanThreads; ++i) {
      const int e = i * kScanThreads + static_cast<int>(threadIdx.x);
      const int t = e >> 1, n = (e & 1) * V;
      const bool in = t < tokens && n0 + n < N;
      copy16_async(dst + t * S::SLAB + n, src + (in ? t * ld + n0 + n : 0), in);
    }
  } else {
    for (int e = threadIdx.x; e < kScanChunk * S::SLAB; e += kScanThreads) {
      const int t = e / S::SLAB, n = e % S::SLAB;
      dst[e] = (t < tokens && n0 + n < N) ? src[t * ld + n0 + n] : from_f32<T_>(0.f);
    }
  }
}

// [token][SLAB] -> [pair][span][token].
template <typename T_, int PASSES>
__device__ __forceinline__ void lay_out(uint32_t* tile, const T_* raw) {
  using S = ScanShape<T_, PASSES>;
#pragma unroll
  for (int t = threadIdx.x; t < kScanChunk; t += kScanThreads) {
    const uint4* src = reinterpret_cast<const uint4*>(raw + t * S::SLAB);
    const uint4 lo = src[0], hi = src[1];
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t* dst = tile + (t / kScanK) * S::PAIR_SPAN + (t % kScanK) * (S::ES / 2);
    if (S::ES == 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[i * S::PAIR_TILE] = w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint2*>(dst + i * S::PAIR_TILE) = make_uint2(w[2 * i], w[2 * i + 1]);
    }
  }
}

// One pair's values of a span's eight tokens.
template <typename T_>
struct PairSpan;
template <>
struct PairSpan<__nv_bfloat16> {
  uint32_t w[8];
  __device__ __forceinline__ explicit PairSpan(const uint32_t* p) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
  __device__ __forceinline__ float lo(int k) const { return __uint_as_float(w[k] << 16); }
  __device__ __forceinline__ float hi(int k) const { return __uint_as_float(w[k] & 0xffff0000u); }
};
template <>
struct PairSpan<float> {
  float w[16];
  __device__ __forceinline__ explicit PairSpan(const uint32_t* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = reinterpret_cast<const float4*>(p)[i];
      w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
    }
  }
  __device__ __forceinline__ float lo(int k) const { return w[2 * k]; }
  __device__ __forceinline__ float hi(int k) const { return w[2 * k + 1]; }
};

// STATE_ONLY: the first of the two passes of a call that is split over time: every
// run from a zero state, its end state and sum of steps written, no outputs.
template <typename T_, int P, bool STATE_ONLY>
__global__ void __launch_bounds__(kScanThreads, ScanShape<T_, P>::CTAS)
    scan_chunk_kernel(const ScanArgs<T_> a, const ScanPlan pl, unsigned long long wait_ns) {
  using S = ScanShape<T_, P>;
  extern __shared__ __align__(16) uint8_t scan_smem[];
  const int NP = scan_np(a.N);
  T_* rows = reinterpret_cast<T_*>(scan_smem);                        // U, delta, Z (then Y)
  T_* raw = reinterpret_cast<T_*>(scan_smem + S::ROWS);               // B, C as they come
  uint32_t* tiles = reinterpret_cast<uint32_t*>(scan_smem + S::ROWS + S::RAW);
  float* ends_all = reinterpret_cast<float*>(scan_smem + S::ROWS + S::RAW + S::TILES);
  float* state = ends_all + kScanWarps * kEndsWarp;                            // [ch][NP]
  float* A2s = state + S::CH * NP;                                  // [ch][NP], A log2(e)
  float* biases = A2s + S::CH * NP;                                 // [ch]
  float* skips = biases + S::CH;                                    // [ch]
  float* totals = skips + S::CH;                                    // [ch], STATE_ONLY: sums of s
  __shared__ int next_task, aborted;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = a.B * pl.blocks;
  const int tasks = groups * (STATE_ONLY ? pl.runs - 1 : pl.runs);
  const int dg = a.d / a.G;
  const bool pieces_u = pieces_ok(a.U, a.ldu, dg), pieces_t = pieces_ok(a.delta, a.ldt, dg);
  const bool pieces_z = pieces_ok(a.Z, a.ldz, dg), pieces_y = pieces_ok(a.Y, a.ldy, dg);
  const bool pieces_b = pieces_ok(a.Bm, a.ldb, a.N), pieces_c = pieces_ok(a.Cm, a.ldc, a.N);
  // joins: lane -> one state element of one channel (q = 2 element + channel)
  float* ends = ends_all + warp * kEndsWarp;
  float* my_end = ends + (lane / kJoinSpans) * kEndsGroup + (lane % kJoinSpans) * kEndsSpan;
  const int q = lane % kEndsSpan, first_span = lane / kEndsSpan * kJoinSpans;
  float* join_ends = ends + (lane / kEndsSpan) * kEndsGroup + q;
  const int join_at = (q & 1) * NP + (q >> 1);
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
    const int in_group = (blk - g * pl.per_group) * S::CH;
    const int c0 = g * dg + in_group;
    const int nch = min(S::CH, dg - in_group);
    const int len = sequence_length(a.lengths, b, a.T);
    const int t_begin = run * pl.run_tokens;
    const int t_end = min(len, t_begin + pl.run_tokens);
    const bool first = run == 0;
    const bool last = len <= t_begin + pl.run_tokens;  // the run that holds the sequence's end
    if (!first && t_begin >= len) {
      if constexpr (STATE_ONLY) {  // a run behind the end joins as nothing
        const long long at = ((long long)run * a.B + b) * a.d + c0;
        float* end = pl.carry + (at + (long long)a.B * a.d) * a.N;
        for (int e = tid; e < nch * a.N; e += kScanThreads) end[e] = 0.f;
        if (tid < nch) pl.step_sum[at + tid] = 0.f;
      }
      continue;
    }

    const long long row0 = (long long)b * a.T;
    auto fetch_inputs = [&](int t0) {
      const int tokens = min(kScanChunk, t_end - t0);
      const long long row = row0 + t0;
      fetch_rows<T_, P>(rows, a.U + row * a.ldu + c0, a.ldu, tokens, nch, pieces_u);
      fetch_rows<T_, P>(rows + S::ROW_TILE, a.delta + row * a.ldt + c0, a.ldt, tokens, nch, pieces_t);
    };
    auto fetch_bc = [&](int t0, int n0) {
      const int tokens = min(kScanChunk, t_end - t0);
      const long long row = row0 + t0, gn = (long long)g * a.N;
      fetch_slab<T_, P>(raw, a.Bm + row * a.ldb + gn, a.ldb, tokens, a.N, n0, pieces_b);
      if (!STATE_ONLY)
        fetch_slab<T_, P>(raw + kScanChunk * S::SLAB, a.Cm + row * a.ldc + gn, a.ldc, tokens, a.N, n0,
                          pieces_c);
    };
    if (t_begin < t_end) {
      fetch_inputs(t_begin);
      fetch_bc(t_begin, 0);
      copy_commit();
    }

    if (!STATE_ONLY && pl.chained && !first) {
      if (tid == 0) {
        const WaitCtl wc{&aborted, wait_ns};
        flag_wait_geq(pl.flags + 1 + gb, static_cast<uint32_t>(run), wc);
      }
      __syncthreads();
      if (*const_cast<volatile int*>(&aborted)) {
        copy_wait<0>();
        return;
      }
    }
    for (int e = tid; e < S::CH * NP; e += kScanThreads) {
      const int i = e / NP, n = e - i * NP;
      float h = 0.f, A2 = 0.f;
      if (i < nch && n < a.N) {
        A2 = a.A[(long long)(c0 + i) * a.N + n] * kLog2e;
        const long long at = ((long long)b * a.d + c0 + i) * a.N + n;
        if (!STATE_ONLY) {
          if (pl.runs > 1 && !pl.chained) h = pl.carry[(long long)run * a.B * a.d * a.N + at];
          else if (first) h = a.state_in ? a.state_in[at] : 0.f;
          else h = __ldcg(pl.carry + ((long long)gb * S::CH + i) * NP + n);
        }
      }
      state[e] = h;
      A2s[e] = A2;
    }

    if (tid < S::CH) {
      biases[tid] = (a.dt_bias && tid < nch) ? a.dt_bias[c0 + tid] : 0.f;
      skips[tid] = (a.D && tid < nch) ? a.D[c0 + tid] : 0.f;
      totals[tid] = 0.f;
    }

    for (int t0 = t_begin; t0 < t_end; t0 += kScanChunk) {
      const int tokens = min(kScanChunk, t_end - t0);
      const int mine0 = lane * kScanK;  // this thread's first token of the chunk
      f32x2 s2[kScanK];                 // (channel, next channel)
      f32x2 y2[kScanK];
      float2 su[kScanK];
      float join_sum[kJoinSpans];       // sums of s of the spans that this lane joins

#pragma unroll 1
      for (int pass = 0; pass < P; ++pass) {
        // this thread's two channels (past nch: zeros in, nothing out)
        const int ch = 2 * (warp + kScanWarps * pass);
        const T_* my_rows = rows + lane * S::ROW_SPAN + ch;
        float* join_state = state + ch * NP + join_at;
        const float* join_A2 = A2s + ch * NP + join_at;
        const bool last_pass = pass == P - 1;
#pragma unroll 1
        for (int n0 = 0; n0 < NP; n0 += S::SLAB) {
          const bool fresh = pass == 0;  // else B and C, one slab, are laid out already
          if (fresh) {
            copy_wait<0>();
            __syncthreads();  // the copies are in; the tiles' readers of the step before are done
          }
          if (n0 == 0) {
            if (!STATE_ONLY && a.Z && pass == 0) {
              fetch_rows<T_, P>(rows + 2 * S::ROW_TILE, a.Z + (row0 + t0) * a.ldz + c0, a.ldz, tokens, nch,
                                pieces_z);
              copy_commit();
            }
            const float2 bias = *reinterpret_cast<const float2*>(biases + ch);
            const float2 skip = *reinterpret_cast<const float2*>(skips + ch);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kScanK; ++k) {
              const float2 u = load_two(my_rows + k * S::CH);
              float2 s = load_two(my_rows + S::ROW_TILE + k * S::CH);
              s.x += bias.x;
              s.y += bias.y;
              if (a.softplus) {
                s.x = softplus_f32(s.x);
                s.y = softplus_f32(s.y);
              }
              if (mine0 + k >= tokens) s = make_float2(0.f, 0.f);  // behind the end: the state passes
              sum.x += s.x;
              sum.y += s.y;
              s2[k] = pack2(s.x, s.y);
              su[k] = make_float2(s.x * u.x, s.y * u.y);
              // no 0 * inf where there is no skip
              y2[k] = a.D ? pack2(skip.x * u.x, skip.y * u.y) : pack2(0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < kJoinSpans; ++i) {
              const float x = __shfl_sync(0xffffffffu, sum.x, first_span + i);
              const float z = __shfl_sync(0xffffffffu, sum.y, first_span + i);
              join_sum[i] = (q & 1) ? z : x;
            }
            if constexpr (STATE_ONLY) {
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) {
                sum.x += __shfl_xor_sync(0xffffffffu, sum.x, o);
                sum.y += __shfl_xor_sync(0xffffffffu, sum.y, o);
              }
              if (lane == 0) {
                totals[ch] += sum.x;
                totals[ch + 1] += sum.y;
              }
            }
          }
          if (fresh) {
            lay_out<T_, P>(tiles, raw);
            if (!STATE_ONLY) lay_out<T_, P>(tiles + S::PAIRS * S::PAIR_TILE, raw + kScanChunk * S::SLAB);
          }
          // before the tiles are read, and before the rows, read above by all, are replaced
          if (fresh || last_pass) __syncthreads();
          // what comes next arrives during the recurrences
          if (n0 + S::SLAB < NP) {
            fetch_bc(t0, n0 + S::SLAB);
          } else if (last_pass && t0 + kScanChunk < t_end) {
            fetch_inputs(t0 + kScanChunk);
            fetch_bc(t0 + kScanChunk, 0);
          }
          copy_commit();

          const int pairs = min(S::PAIRS, (NP - n0) >> 1);
#pragma unroll 1
          for (int p = 0; p < pairs; p += kScanJ) {
            const int n = n0 + 2 * p;
            // the recurrence from zero, its outputs, and g = C times the decay since the
            // span's start, which the start state is multiplied with once it is known
            f32x2 g[kScanJ][2][kScanK], h[kScanJ][2];
#pragma unroll
            for (int j = 0; j < kScanJ; ++j) {
              const uint32_t* bp = tiles + (p + j) * S::PAIR_TILE + lane * S::PAIR_SPAN;
              const float2 Ax = *reinterpret_cast<const float2*>(A2s + ch * NP + n + 2 * j);
              const float2 Ay = *reinterpret_cast<const float2*>(A2s + (ch + 1) * NP + n + 2 * j);
              const f32x2 A0 = pack2(Ax.x, Ay.x), A1 = pack2(Ax.y, Ay.y);
              const PairSpan<T_> B(bp), C(bp + S::PAIRS * S::PAIR_TILE);
              f32x2 h0 = 0ull, h1 = 0ull, p0 = 0ull, p1 = 0ull;
#pragma unroll
              for (int k = 0; k < kScanK; ++k) {
                float x, z;
                unpack2(mul2(s2[k], A0), x, z);
                const f32x2 a0 = pack2(exp2_approx(x), exp2_approx(z));
                unpack2(mul2(s2[k], A1), x, z);
                const f32x2 a1 = pack2(exp2_approx(x), exp2_approx(z));
                h0 = fma2(a0, h0, pack2(su[k].x * B.lo(k), su[k].y * B.lo(k)));
                h1 = fma2(a1, h1, pack2(su[k].x * B.hi(k), su[k].y * B.hi(k)));
                if (!STATE_ONLY) {
                  p0 = k ? mul2(p0, a0) : a0;
                  p1 = k ? mul2(p1, a1) : a1;
                  float y0, y1;
                  unpack2(y2[k], y0, y1);
                  unpack2(h0, x, z);
                  y0 = fmaf(x, C.lo(k), y0);
                  y1 = fmaf(z, C.lo(k), y1);
                  unpack2(h1, x, z);
                  y2[k] = pack2(fmaf(x, C.hi(k), y0), fmaf(z, C.hi(k), y1));
                  unpack2(p0, x, z);
                  g[j][0][k] = pack2(x * C.lo(k), z * C.lo(k));
                  unpack2(p1, x, z);
                  g[j][1][k] = pack2(x * C.hi(k), z * C.hi(k));
                }
              }
              h[j][0] = h0;
              h[j][1] = h1;
            }
            // join the warp's spans
            __syncwarp();  // the starts of the pairs before have been read
#pragma unroll
            for (int j = 0; j < kScanJ; ++j)
              *reinterpret_cast<ulonglong2*>(my_end + 4 * j) = make_ulonglong2(h[j][0], h[j][1]);
            __syncwarp();
            {
              const float A2 = join_A2[n], h_in = join_state[n];
              float e[kJoinSpans], d[kJoinSpans];
#pragma unroll
              for (int i = 0; i < kJoinSpans; ++i) {
                e[i] = join_ends[i * kEndsSpan];
                d[i] = exp2_approx(join_sum[i] * A2);
              }
              // this lane's spans as one: E + D h
              float E = e[0], D = d[0];
#pragma unroll
              for (int i = 1; i < kJoinSpans; ++i) {
                E = fmaf(d[i], E, e[i]);
                D *= d[i];
              }
              // and the lanes before it
#pragma unroll
              for (int o = kEndsSpan; o < 32; o <<= 1) {
                const float Eo = __shfl_up_sync(0xffffffffu, E, o), Do = __shfl_up_sync(0xffffffffu, D, o);
                if (lane >= o) {
                  E = fmaf(D, Eo, E);
                  D *= Do;
                }
              }
              if (lane >= 32 - kEndsSpan) join_state[n] = fmaf(D, h_in, E);
              if (!STATE_ONLY) {
                const float Eo = __shfl_up_sync(0xffffffffu, E, kEndsSpan);
                const float Do = __shfl_up_sync(0xffffffffu, D, kEndsSpan);
                float start = lane >= kEndsSpan ? fmaf(Do, h_in, Eo) : h_in;
#pragma unroll
                for (int i = 0; i < kJoinSpans; ++i) {
                  join_ends[i * kEndsSpan] = start;
                  start = fmaf(d[i], start, e[i]);
                }
              }
            }
            if (STATE_ONLY) continue;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kScanJ; ++j) {
              const ulonglong2 start = *reinterpret_cast<const ulonglong2*>(my_end + 4 * j);
#pragma unroll
              for (int k = 0; k < kScanK; ++k)
                y2[k] = fma2(g[j][1][k], start.y, fma2(g[j][0][k], start.x, y2[k]));
            }
          }
        }

        if (!STATE_ONLY) {
          if (pass == 0) {
            copy_wait<1>();   // Z is in (the next step's copies may still run)
            __syncthreads();
          }
          T_* zy = const_cast<T_*>(my_rows) + 2 * S::ROW_TILE;  // Z's place becomes Y's
#pragma unroll
          for (int k = 0; k < kScanK; ++k) {
            float y0, y1;
            unpack2(y2[k], y0, y1);
            if (a.Z) {
              const float2 z = load_two(zy + k * S::CH);
              y0 *= silu_fast(z.x);
              y1 *= silu_fast(z.y);
            }
            store_two(zy + k * S::CH, y0, y1);
          }
        }
      }
      if (!STATE_ONLY) {
        __syncthreads();
        store_rows<T_, P>(a.Y + (row0 + t0) * a.ldy + c0, rows + 2 * S::ROW_TILE, a.ldy, tokens, nch, pieces_y);
      }
    }

    __syncthreads();  // the state of the run's last token is complete
    if (STATE_ONLY) {
      const long long at = ((long long)run * a.B + b) * a.d + c0;
      if (tid < nch) pl.step_sum[at + tid] = totals[tid];
      float* end = pl.carry + (at + (long long)a.B * a.d) * a.N;  // carry[run + 1]
      for (int e = tid; e < nch * a.N; e += kScanThreads) end[e] = state[(e / a.N) * NP + e % a.N];
      continue;
    }
    if (last) {
      if (a.state_out)
        for (int e = tid; e < nch * a.N; e += kScanThreads)
          a.state_out[((long long)b * a.d + c0) * a.N + e] = state[(e / a.N) * NP + e % a.N];
    } else if (pl.chained) {
      for (int e = tid; e < S::CH * NP; e += kScanThreads)
        pl.carry[(long long)gb * S::CH * NP + e] = state[e];
      __threadfence();
      __syncthreads();
      if (tid == 0) red_release_gpu_add(pl.flags + 1 + gb, 1u);
    }
  }
}

// Between the two passes: carry[run + 1], which holds run's own end state, becomes the
// state before run + 1, by the runs' sums of steps, and carry[0] the state before the
// call.
template <typename T_>
__global__ void __launch_bounds__(256) scan_join_kernel(const ScanArgs<T_> a, const ScanPlan pl) {
  grid_dependency_wait();
  const long long e = blockIdx.x * 256ll + threadIdx.x, total = (long long)a.B * a.d * a.N;
  if (e >= total) return;
  const long long bd = e / a.N;
  const float A2 = a.A[(bd % a.d) * a.N + e % a.N] * kLog2e;
  float h = a.state_in ? a.state_in[e] : 0.f;
  pl.carry[e] = h;
  for (int r = 0; r < pl.runs - 1; ++r) {
    const float end = pl.carry[(r + 1) * total + e];
    const float x = pl.step_sum[(long long)r * a.B * a.d + bd] * A2;
    if (x > 126.f) {
      // a run may grow by more than fp32 holds while what it multiplies is zero or small:
      // three factors, none infinite (past 378 every h but 0 goes to infinity)
      const float third = exp2_approx(fminf(x, 378.f) * (1.f / 3.f));
      h = fmaf(third, third * (third * h), end);
    } else {
      h = fmaf(exp2_approx(x), h, end);
    }
    pl.carry[(r + 1) * total + e] = h;
  }
}

}  // namespace ittt

// Tensor-core kernels of the product Y = act(X W^T + bias) + residual (bf16).
//
// Both compute the transposed tile D = W X^T: the 128 TMEM lanes are output
// columns n, the TMEM columns are rows m of X.  The epilogue's warp then holds
// 32 neighbouring outputs of one row of Y: its loads of the residual and its
// stores are whole 64-byte segments for any row stride, alignment and width of
// Y (no store map, no staging), a lane keeps its one bias value, and few tokens
// make a narrow tile (16 columns) instead of a 128-row one that is mostly
// padding, so one kernel serves one token and many.
//
//   linear_split_kernel  one 128 x MT tile per CTA; the CTAs of a cluster share a
//       tile and split K, their sums joined through distributed shared memory in
//       rank order (the same bits every time, no workspace, one launch).  For few
//       rows it is bound by reading W once from HBM, and by what a launch costs before
//       its first bytes arrive and after its last: 1 x 9728 x 2560 with bias and residual
//       12.3 us (4.0 TB/s; 7.6 us at HBM's copy rate), 64 x 2560 x 10240 15.5 us (8.3).
//   linear_pair_kernel   persistent CTA pairs (two SMs, one 256-lane tile, 256
//       columns, two TMEM slots so that a tile's epilogue overlaps the next tile's main
//       loop).  For many rows: bound by the tensor cores.  8192 x 9728 x 2560 with
//       residual: 349 us in a loop of calls, 1.17 PFLOP/s (cuBLAS's bare product 267 us);
//       under the power cap, where the measured peak is 1.40 PFLOP/s, that is 0.83 of it.
//       Its last wave is part full (320 tiles on 74 pairs).
#pragma once

#include "common.cuh"
#include "linear_f32.cuh"
#include "mixer.cuh"

namespace ittt {

// Outputs (m, n) for m in [m0, m0 + count) of one lane's column n: acc holds the
// sums of 32 rows of X.
template <int ACT>
__device__ __forceinline__ void linear_store32(const LinearArgs<__nv_bfloat16>& a,
                                               const uint32_t (&acc)[32], int n, int m0, int count,
                                               float bias) {
  if (n >= a.N || count <= 0) return;
  __nv_bfloat16* y = a.Y + (long long)m0 * a.ldy + n;
  const __nv_bfloat16* r = a.residual ? a.residual + (long long)m0 * a.ldr + n : nullptr;
  if (count >= 32) {
    float res[32];
    if (r) {
#pragma unroll
      for (int j = 0; j < 32; ++j) res[j] = __bfloat162float(r[j * a.ldr]);
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      float v = activate<ACT>(__uint_as_float(acc[j]) + bias);
      if (r) v += res[j];
      y[j * a.ldy] = __float2bfloat16_rn(v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j < count) {
        float v = activate<ACT>(__uint_as_float(acc[j]) + bias);
        if (r) v += __bfloat162float(r[j * a.ldr]);
        y[j * a.ldy] = __float2bfloat16_rn(v);
      }
    }
  }
}

// Shared-memory pipeline depth: up to 74 KB, so that three CTAs share an SM (two at
// 128 rows) and enough bytes are in flight to cover HBM latency.  A pipeline as deep as
// the shared memory that the launch leaves free measured the same (12.0, 14.3 us).
template <int MT>
struct SplitShape {
  static constexpr int STAGE_BYTES = 128 * 128 + MT * 128;  // 64 bf16 of 128 rows of W, MT of X
  static constexpr int STAGES = MT <= 16 ? 4 : 3;
  static constexpr int CTAS = MT <= 64 ? 3 : 2;  // an SM
  static constexpr int SMEM = STAGES * STAGE_BYTES + 1024 + 256;
  static constexpr int TMEM_COLS = MT < 32 ? 32 : MT;
  static_assert(STAGES * STAGE_BYTES >= MT * 512, "the joined sums fit the pipeline's memory");
};

// One lane's column n of the rows rank, rank + S, ... of a tile: the S sums of each
// row in rank order.  16 remote loads are in flight at once (one at a time, the
// join of 64 rows took longer than the product's own pipeline).
template <int MT, int S, int ACT>
__device__ __forceinline__ void linear_join(const LinearArgs<__nv_bfloat16>& a, uint32_t mine, int rank,
                                            int n, int m0, float bias) {
  constexpr int ROWS = MT / S, BATCH = ROWS < 16 / S ? ROWS : 16 / S;
#pragma unroll 1
  for (int i0 = 0; i0 < ROWS; i0 += BATCH) {
    const int c0 = rank + i0 * S;
    if (m0 + c0 >= a.M) return;
    float part[BATCH][S];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
#pragma unroll
      for (int s = 0; s < S; ++s)
        part[i][s] = ld_shared_cluster_f32(cluster_addr(mine + (c0 + i * S) * 512u, s));
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const long long m = m0 + c0 + i * S;
      if (m >= a.M) break;
      float v = part[i][0];
#pragma unroll
      for (int s = 1; s < S; ++s) v += part[i][s];
      v = activate<ACT>(v + bias);
      if (a.residual) v += __bfloat162float(a.residual[m * a.ldr + n]);
      a.Y[m * a.ldy + n] = __float2bfloat16_rn(v);
    }
  }
}

template <int MT, int ACT>
__global__ void __launch_bounds__(192, SplitShape<MT>::CTAS)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmW,
                        const __grid_constant__ CUtensorMap tmX,
                        const LinearArgs<__nv_bfloat16> a, int m_tiles, int num_kb,
                        unsigned long long wait_ns) {
  using S = SplitShape<MT>;
  constexpr uint32_t IDESC = make_idesc_bf16(128, MT, false, false);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + S::STAGES * S::STAGE_BYTES);
  uint64_t* empty_bar = full_bar + S::STAGES;
  uint64_t* tfull = empty_bar + S::STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int splits = static_cast<int>(cluster_size());
  const int rank = static_cast<int>(cluster_cta_rank());
  const int tile = blockIdx.x / splits;
  const int m0 = (tile % m_tiles) * MT;
  const int n0 = (tile / m_tiles) * 128;
  // this CTA's share of the k-blocks
  const int kb0 = static_cast<int>((long long)num_kb * rank / splits);
  const int kb1 = static_cast<int>((long long)num_kb * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(tfull, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, S::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  grid_dependency_wait();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl wc{abort_flag, wait_ns};

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int last_parity[S::STAGES];
      for (int s = 0; s < S::STAGES; ++s) last_parity[s] = -1;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty_bar[stage], phase ^ 1, wc)) break;
        mbar_arrive_expect_tx(&full_bar[stage], S::STAGE_BYTES);
        last_parity[stage] = static_cast<int>(phase);
        uint8_t* sa = smem + stage * S::STAGE_BYTES;
        tma_load_2d(sa, &tmW, &full_bar[stage], kb * 64, n0);
        tma_load_2d(sa + 128 * 128, &tmX, &full_bar[stage], kb * 64, m0);
        if (++stage == S::STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (*abort_flag) {
        for (int s = 0; s < S::STAGES; ++s)
          if (last_parity[s] >= 0) mbar_wait_teardown(&full_bar[s], last_parity[s], wait_ns);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = mbar_wait(&full_bar[stage], phase, wc))) break;
        tc_fence_after_sync();
        const uint32_t wa = smem_u32(smem + stage * S::STAGE_BYTES);
        const uint32_t xa = wa + 128 * 128;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16(tmem_base, make_sdesc_sw128(wa + kk * 32, 16, 1024),
                    make_sdesc_sw128(xa + kk * 32, 16, 1024), IDESC, (kb > kb0 || kk > 0) ? 1u : 0u);
        umma_commit(&empty_bar[stage]);
        if (++stage == S::STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      umma_commit(tfull);
      if (!ok) mbar_wait_teardown(tfull, 0, wait_ns);
    }
    __syncwarp();
  }
  // The next kernel's CTAs may take free slots and set up (every CTA of this one holds
  // its TMEM): 11.9 us a call instead of 13.7 for one row of 9728 -> 2560 in a chain of
  // calls.  Before the wait above it is 12.4, and in the other kernels of these
  // operators, which leave no slot unused, it costs time.
  grid_launch_dependents();

  // every MMA has completed, and with them every read of the pipeline's memory
  bool ok = false;
  if (warp >= 2) {
    ok = mbar_wait(tfull, 0, wc);
    __syncwarp();
    tc_fence_after_sync();
  }
  const int q = warp & 3;
  const int r = q * 32 + lane;  // this thread's column of Y within the tile (warps 2..5)
  const int n = n0 + r;
  const float bias = (warp >= 2 && a.bias && n < a.N) ? __bfloat162float(a.bias[n]) : 0.f;
  const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
  if (splits == 1) {
    if (ok) {
#pragma unroll 1
      for (int c0 = 0; c0 < MT; c0 += 32) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(tbase + c0, v);
        tmem_ld_wait();
        linear_store32<ACT>(a, v, n, m0 + c0, min(MT - c0, a.M - (m0 + c0)), bias);
      }
    }
  } else {
    float* red = reinterpret_cast<float*>(smem);  // [MT][128], this CTA's sums
    if (ok) {
#pragma unroll 1
      for (int c0 = 0; c0 < MT; c0 += 32) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(tbase + c0, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c0 + j < MT) red[(c0 + j) * 128 + r] = __uint_as_float(v[j]);
      }
    }
    __syncwarp();
    cluster_sync_all();
    // rank i finishes the rows i, i + splits, ... of X
    if (ok && n < a.N) {
      const uint32_t mine = smem_u32(red) + static_cast<uint32_t>(r) * 4u;
      switch (splits) {
        case 2: linear_join<MT, 2, ACT>(a, mine, rank, n, m0, bias); break;
        case 4: linear_join<MT, 4, ACT>(a, mine, rank, n, m0, bias); break;
        default: linear_join<MT, 8, ACT>(a, mine, rank, n, m0, bias); break;
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while a peer may still read its sums
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem_base, S::TMEM_COLS);
  }
}

// ------------------------------------------------------------------ pairs

struct PairTile {
  int m_tiles, n_tiles;       // tiles of 256 rows of X and of 256 outputs
  int group_n;                // n-tiles per rasterisation group (0 = all): their rows of W
                              // stay in L2 while the rows of X pass
  int num_kb;
};

constexpr int kPairRows = 256;  // rows of X a tile: 128 and 224 take as long per step of K (0.4 us)
constexpr int kPairStages = 6;
constexpr int kPairStageBytes = 2 * 128 * 128;
constexpr int kPairSmem = kPairStages * kPairStageBytes + 1024 + 256;

__device__ __forceinline__ void pair_decode(const PairTile& t, int u, int& mt, int& nt) {
  const int gn = (t.group_n > 0 && t.group_n < t.n_tiles) ? t.group_n : t.n_tiles;
  const int per_group = gn * t.m_tiles;
  const int g = u / per_group, r = u - g * per_group;
  const int cols = min(gn, t.n_tiles - g * gn);
  nt = g * gn + r % cols;
  mt = r / cols;
}

template <int ACT>
__global__ void __launch_bounds__(192, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmX,
                       const LinearArgs<__nv_bfloat16> a, const PairTile t,
                       unsigned long long wait_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + kPairStages * kPairStageBytes);
  uint64_t* empty_bar = full_bar + kPairStages;
  uint64_t* tfull = empty_bar + kPairStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done_bar = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_cta_rank();
  const bool leader = rank == 0;
  constexpr int half = kPairRows / 2;  // rows of X each CTA of the pair loads

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], 8);  // four epilogue warps of each CTA
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc<true>(tmem_slot, 512);
    tmem_relinquish<true>();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // the peer's barriers exist before anyone signals them
  tc_fence_after_sync();
  grid_dependency_wait();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl wc{abort_flag, wait_ns};
  auto leader_bar = [&](uint64_t* bar) { return cluster_addr(smem_u32(bar), 0u); };
  const int units = t.m_tiles * t.n_tiles;
  const int worker = blockIdx.x >> 1, workers = gridDim.x >> 1;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int last_parity[kPairStages];
      for (int s = 0; s < kPairStages; ++s) last_parity[s] = -1;
      bool ok = true;
      for (int u = worker; u < units && ok; u += workers) {
        int mt, nt;
        pair_decode(t, u, mt, nt);
        const int n0 = nt * 256 + static_cast<int>(rank) * 128;
        const int m0 = mt * kPairRows + static_cast<int>(rank) * half;
        for (int kb = 0; kb < t.num_kb; ++kb) {
          if (!(ok = mbar_wait(&empty_bar[stage], phase ^ 1, wc))) break;
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2u * kPairStageBytes);
          last_parity[stage] = static_cast<int>(phase);
          uint8_t* sa = smem + stage * kPairStageBytes;
          const uint32_t fb = leader_bar(&full_bar[stage]);
          tma_load_2d_pair(sa, &tmW, fb, kb * 64, n0);
          tma_load_2d_pair(sa + 128 * 128, &tmX, fb, kb * 64, m0);
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (*abort_flag && leader) {
        for (int s = 0; s < kPairStages; ++s)
          if (last_parity[s] >= 0) mbar_wait_teardown(&full_bar[s], last_parity[s], wait_ns);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // 256 lanes x 256 columns over the two SMs
      constexpr uint32_t idesc = make_idesc_bf16(256, kPairRows, false, false);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t count[2] = {0, 0};
      int slot = 0;
      bool ok = true;
      for (int u = worker; u < units && ok; u += workers) {
        if (!(ok = mbar_wait(&tempty[slot], count[slot] & 1, wc))) break;
        count[slot]++;
        tc_fence_after_sync();
        const uint32_t dtm = tmem_base + static_cast<uint32_t>(slot) * 256u;
        for (int kb = 0; kb < t.num_kb; ++kb) {
          if (!(ok = mbar_wait(&full_bar[stage], phase, wc))) break;
          tc_fence_after_sync();
          const uint32_t wa = smem_u32(smem + stage * kPairStageBytes);
          const uint32_t xa = wa + 128 * 128;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_pair(dtm, make_sdesc_sw128(wa + kk * 32, 16, 1024),
                           make_sdesc_sw128(xa + kk * 32, 16, 1024), idesc,
                           (kb > 0 || kk > 0) ? 1u : 0u);
          umma_commit_pair_both(smem_u32(&empty_bar[stage]));
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        umma_commit_pair_both(smem_u32(&tfull[slot]));
        slot ^= 1;
      }
      // every MMA issued above has completed once done_bar flips
      umma_commit_pair_both(smem_u32(done_bar));
      mbar_wait_teardown(done_bar, 0, wait_ns);
    }
  } else {
    const int q = warp & 3;
    const int r = q * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    auto release = [&](int slot) {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_bar(&tempty[slot]));
    };
    release(0);
    release(1);
    uint32_t count[2] = {0, 0};
    int slot = 0;
    for (int u = worker; u < units; u += workers) {
      int mt, nt;
      pair_decode(t, u, mt, nt);
      const int n = nt * 256 + static_cast<int>(rank) * 128 + r;
      const int m0 = mt * kPairRows;
      const float bias = (a.bias && n < a.N) ? __bfloat162float(a.bias[n]) : 0.f;
      // this warp's 64 bytes of the tile's residual rows come into L2 during the main loop
      if (a.residual && n - lane < a.N)
        for (int i = lane; i < kPairRows && m0 + i < a.M; i += 32)
          prefetch_l2(a.residual + (long long)(m0 + i) * a.ldr + n - lane);
      const bool ok = mbar_wait(&tfull[slot], count[slot] & 1, wc);
      __syncwarp();
      if (!ok) break;
      count[slot]++;
      tc_fence_after_sync();
      const uint32_t tbase = tmem_base + lane_addr + static_cast<uint32_t>(slot) * 256u;
#pragma unroll 1
      for (int c0 = 0; c0 < kPairRows; c0 += 32) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(tbase + c0, v);
        tmem_ld_wait();
        if (c0 + 32 == kPairRows) release(slot);
        linear_store32<ACT>(a, v, n, m0 + c0, min(kPairRows - c0, a.M - (m0 + c0)), bias);
      }
      slot ^= 1;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its peer may still signal it
  tc_fence_after_sync();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc<true>(tmem_base, 512);
  }
}

}  // namespace ittt

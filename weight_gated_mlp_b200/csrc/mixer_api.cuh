// C ABI of the operators around the layer: validation, and dispatch of the kernels of
// tc_linear.cuh, linear_f32.cuh, mixer.cuh and scan.cuh.  Included at the end of api.cu,
// whose helpers it uses.
#pragma once

namespace {

bool valid_dtype_act(int32_t dtype, int32_t act) {
  return (dtype == ITTT_F32 || dtype == ITTT_BF16) && act >= ITTT_ACT_NONE &&
         act <= ITTT_ACT_GELU_TANH;
}

// The row stride that 0 stands for.
long long stride_or(int64_t ld, int64_t dense) { return ld == 0 ? dense : ld; }

// Bytes from the first to the last element of `rows` rows of `width` elements,
// `ld` apart.
size_t span_bytes(long long rows, long long ld, long long width, size_t es) {
  return (size_t(rows - 1) * size_t(ld) + size_t(width)) * es;
}

// Row and column numbers, rounded up to a tile, fit 32 bits; offsets are 64-bit.
bool fits(int64_t rows, int64_t width, int64_t ld) {
  constexpr int64_t most = (1ll << 31) - 1024;
  return rows > 0 && width > 0 && rows < most && width < most && (ld == 0 || (ld >= width && ld < most));
}

// ------------------------------------------------------------------ linear

ittt_status validate_linear(const ittt_linear_problem* p) {
  if (!p || p->M <= 0 || p->N <= 0 || p->K <= 0 || p->ldx < 0 || p->ldr < 0 || p->ldy < 0 ||
      !valid_dtype_act(p->dtype, p->act))
    return ITTT_ERR_INVALID_ARG;
  if ((p->ldx && p->ldx < p->K) || (p->ldr && p->ldr < p->N) || (p->ldy && p->ldy < p->N))
    return ITTT_ERR_INVALID_ARG;
  if (!fits(p->M, p->K, p->ldx) || !fits(p->M, p->N, p->ldr) || !fits(p->M, p->N, p->ldy) ||
      !fits(p->N, p->K, 0))
    return ITTT_ERR_UNSUPPORTED;
  if (p->dtype == ITTT_BF16 && (p->K % 8 || p->ldx % 8)) return ITTT_ERR_UNSUPPORTED;
  return ITTT_OK;
}

template <typename T_>
LinearArgs<T_> linear_args(const ittt_linear_problem* p, const void* X, const void* W,
                           const void* bias, const void* residual, void* Y) {
  LinearArgs<T_> a{};
  a.X = static_cast<const T_*>(X);
  a.W = static_cast<const T_*>(W);
  a.bias = static_cast<const T_*>(bias);
  a.residual = static_cast<const T_*>(residual);
  a.Y = static_cast<T_*>(Y);
  a.ldx = stride_or(p->ldx, p->K);
  a.ldr = stride_or(p->ldr, p->N);
  a.ldy = stride_or(p->ldy, p->N);
  a.M = int(p->M);
  a.N = int(p->N);
  a.K = int(p->K);
  a.act = p->act;
  return a;
}

// A launch in clusters of `cluster` CTAs, its prologue overlapping the kernel before.
template <typename... KArgs, typename... Args>
ittt_status launch_clusters(void (*kern)(KArgs...), unsigned grid, unsigned cluster, unsigned threads,
                            int smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = ITTT_PDL;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...) != cudaSuccess)
    return ITTT_ERR_CUDA;
  return launch_status();
}

constexpr int kSmemMost = 232448;  // the most dynamic shared memory of a CTA

// Dynamic shared memory above the default, granted once per kernel and device.
template <typename Kern>
bool grant_smem(Kern kern, int smem, std::atomic<bool>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  if (done[dev].load(std::memory_order_relaxed)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return false;
  done[dev].store(true, std::memory_order_relaxed);
  return true;
}

template <int ACT, int MB, bool VEC>
ittt_status linear_gemv(const LinearArgs<float>& a, cudaStream_t st) {
  return launch_pdl(linear_gemv_kernel<ACT, MB, VEC>, dim3(unsigned(cdiv(a.N, 4))), dim3(128), st, a);
}

template <int ACT, int BM, int BN, int TM, int TN, bool VEC>
ittt_status linear_tiles_f32(const LinearArgs<float>& a, int splits, cudaStream_t st) {
  const long long m_tiles = cdiv(a.M, BM), grid = m_tiles * cdiv(a.N, BN) * splits;
  if (grid >= (1ll << 31)) return ITTT_ERR_UNSUPPORTED;
  return launch_clusters(linear_f32_kernel<ACT, BM, BN, TM, TN, VEC>, unsigned(grid), unsigned(splits),
                         F32Tile<BM, BN, TM, TN>::THREADS, 0, st, a, int(m_tiles));
}

// Up to 8 rows: the kernel that streams W.  Else 64 x 64 tiles, K split over clusters
// while the CTAs stay within six an SM and every CTA keeps at least 64 columns of K, or,
// so that the last wave is a small part of the whole, within 21 an SM at 128 columns
// (us, unsplit and split: 333 x 1000 x 1001 63 and 25 in 8; 1154 x 2168 x 2547 338 and 309
// in 4; 2048 x 2048 x 2048 430 and 372 in 2, 395 in 4; 4096 x 1024 x 2368, 16 tiles an SM,
// 419 and 425 in 2).  128 x 128 tiles were slower (422, 386 and 465 us for the
// last three).
template <int ACT, bool VEC>
ittt_status linear_f32_sized(const LinearArgs<float>& a, int sms, cudaStream_t st) {
  if (a.M == 1) return linear_gemv<ACT, 1, VEC>(a, st);
  if (a.M == 2) return linear_gemv<ACT, 2, VEC>(a, st);
  if (a.M <= 4) return linear_gemv<ACT, 4, VEC>(a, st);
  if (a.M <= 8) return linear_gemv<ACT, 8, VEC>(a, st);
  const long long tiles = cdiv(a.M, 64) * cdiv(a.N, 64);
  int splits = 1;
  auto twice = [&](int ctas, int columns) {
    return tiles * splits * 2 <= (long long)ctas * sms && a.K / columns >= splits * 2;
  };
  while (splits < 8 && (twice(6, 64) || twice(21, 128))) splits *= 2;
  return linear_tiles_f32<ACT, 64, 64, 8, 8, VEC>(a, splits, st);
}

template <int ACT>
ittt_status linear_f32(const LinearArgs<float>& a, cudaStream_t st) {
  const int sms = num_sms();
  if (sms <= 0) return ITTT_ERR_CUDA;
  if (aligned16(a.X) && aligned16(a.W) && a.K % 4 == 0 && a.ldx % 4 == 0)
    return linear_f32_sized<ACT, true>(a, sms, st);
  return linear_f32_sized<ACT, false>(a, sms, st);
}

// Never launched: place_kernel stands in for linear_split_kernel in questions about how
// many clusters fit, which for a kernel with tensor memory are answered as if an SM
// held one CTA of it.
__global__ void __launch_bounds__(192) place_kernel() {}

// Dynamic shared memory at which an SM holds `per_sm` CTAs and no more (1 KB of an SM's 228
// is reserved for each).
int smem_for(int per_sm) { return std::min(kSmemMost, (233472 / per_sm - 1024) / 1024 * 1024); }

// Clusters of `cluster` CTAs that the current device holds at once with per_sm CTAs an SM
// (-1: it does not say).  Fewer than the SMs divided, since no cluster leaves its part of the
// GPU: of 8, 15 at one CTA an SM, 33 at two and 48 at three, where 148 SMs would give 18,
// 37 and 55.
int cluster_places(int per_sm, int cluster) {
  static std::atomic<bool> granted[kMaxDevices] = {};
  static std::atomic<int> known[kMaxDevices][4][9] = {};
  if (!grant_smem(place_kernel, kSmemMost, granted)) return -1;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  std::atomic<int>& places = known[dev][per_sm][cluster];
  if ((n = places.load(std::memory_order_relaxed)) > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(cluster) * 1024, 1, 1);
  cfg.blockDim = dim3(192, 1, 1);
  cfg.dynamicSmemBytes = smem_for(per_sm);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, place_kernel, &cfg) != cudaSuccess) return -1;
  places.store(n, std::memory_order_relaxed);
  return n;
}

// One 128 x MT tile per CTA, K split over clusters.  The split is the widest of
// 1, 2, 4, 8 CTAs whose clusters the GPU holds all at once and that leaves at least four
// k-blocks to each CTA.  A call asks for the shared memory that lets no SM hold more CTAs
// than that takes: clusters are otherwise packed onto fewer SMs (777 x 5120 x 192, 208
// CTAs: 12.8 us, 13.7 without).  Two CTAs always find room, so that the next launch's, or
// another stream's, can start beside a CTA that has its SM to itself (128 x 4096 x 1024, 64
// CTAs: 10.2 us in a chain of calls, 10.5 where the memory let an SM hold one).  Counted by
// SMs alone, clusters that found no place ran behind the others (1 x 9728 x 2304, 18
// clusters of 8: 20.3 us, 12.2 in two CTAs an SM; 1 x 4096 x 6400, 50 of 8: 15.7 us, 12.3 in
// clusters of 4).
template <int MT, int ACT>
ittt_status linear_split(const LinearArgs<__nv_bfloat16>& a, int sms, cudaStream_t st) {
  using S = SplitShape<MT>;
  static std::atomic<bool> granted[kMaxDevices] = {};
  auto kern = linear_split_kernel<MT, ACT>;
  if (!grant_smem(kern, kSmemMost, granted)) return ITTT_ERR_CUDA;
  const int num_kb = int(cdiv(a.K, 64));
  const long long m_tiles = cdiv(a.M, MT), tiles = m_tiles * cdiv(a.N, 128);
  int splits = 1, per_sm = 2;
  while (splits < 8 && num_kb >= 4 * splits * 2) {
    const int places = cluster_places(S::CTAS, splits * 2);
    if (places < 0) return ITTT_ERR_CUDA;
    if (tiles > places) break;
    splits *= 2;
  }
  while (per_sm < S::CTAS) {
    const int places = splits == 1 ? per_sm * sms : cluster_places(per_sm, splits);
    if (places < 0) return ITTT_ERR_CUDA;
    if (tiles <= places) break;
    ++per_sm;
  }
  if (tiles * splits >= (1ll << 31)) return ITTT_ERR_UNSUPPORTED;
  CUtensorMap w, x;
  if (!make_map(&w, a.W, a.K, a.N, a.K, 64, 128) || !make_map(&x, a.X, a.K, a.M, a.ldx, 64, MT))
    return ITTT_ERR_CUDA;
  return launch_clusters(kern, unsigned(tiles * splits), unsigned(splits), 192,
                         std::max(S::SMEM, smem_for(per_sm)), st, w, x, a,
                         int(m_tiles), num_kb, g_wait_ns.load());
}

// CTA pairs of linear_pair_kernel that the current device holds at once (0: none).
template <int ACT>
int resident_pairs(int sms) {
  static std::atomic<bool> granted[kMaxDevices] = {};
  static std::atomic<int> pairs[kMaxDevices] = {};
  if (!grant_smem(linear_pair_kernel<ACT>, kPairSmem, granted)) return 0;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if ((n = pairs[dev].load(std::memory_order_relaxed)) > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(2 * (sms / 2)), 1, 1);
  cfg.blockDim = dim3(192, 1, 1);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, linear_pair_kernel<ACT>, &cfg) != cudaSuccess || n <= 0) return 0;
  pairs[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Persistent CTA pairs.
template <int ACT>
ittt_status linear_pairs(const LinearArgs<__nv_bfloat16>& a, int pairs, cudaStream_t st) {
  PairTile t{};
  t.m_tiles = int(cdiv(a.M, kPairRows));
  t.n_tiles = int(cdiv(a.N, 256));
  t.num_kb = int(cdiv(a.K, 64));
  // a group's rows of W (about 32 MiB) stay in L2 while the rows of X pass once
  const long long tile_bytes = 256ll * a.K * 2;
  if (tile_bytes * t.n_tiles > (48ll << 20)) t.group_n = int(std::max(1ll, (32ll << 20) / tile_bytes));
  if ((long long)t.m_tiles * t.n_tiles >= (1ll << 31)) return ITTT_ERR_UNSUPPORTED;
  CUtensorMap w, x;
  if (!make_map(&w, a.W, a.K, a.N, a.K, 64, 128) || !make_map(&x, a.X, a.K, a.M, a.ldx, 64, kPairRows / 2))
    return ITTT_ERR_CUDA;
  const long long units = (long long)t.m_tiles * t.n_tiles;
  return launch_clusters(linear_pair_kernel<ACT>, unsigned(2 * std::min<long long>(units, pairs)), 2, 192,
                         kPairSmem, st, w, x, a, t, g_wait_ns.load());
}

// Up to 128 rows: one narrow tile of all rows per 128 outputs, so that W is read
// once.  More: split tiles of 128 x 128 while K can still be split over two CTAs (the
// pairs' 256 x 256 tiles leave most SMs empty there: 512 x 9728 x 2560 takes 40 us
// split and 50 in pairs, but 69 and 56 with a residual, which the split's join loads a
// row at a time), of 128 x 64 where even eight-fold splits of those leave SMs empty;
// from there on pairs (1024 x 9728 x 2560: 52 us, 80 us in unsplit tiles).
template <int ACT>
ittt_status linear_bf16(const LinearArgs<__nv_bfloat16>& a, cudaStream_t st) {
  const int sms = num_sms();
  if (sms <= 0) return ITTT_ERR_CUDA;
  if (a.M <= 16) return linear_split<16, ACT>(a, sms, st);
  if (a.M <= 32) return linear_split<32, ACT>(a, sms, st);
  if (a.M <= 64) return linear_split<64, ACT>(a, sms, st);
  if (a.M <= 128) return linear_split<128, ACT>(a, sms, st);
  const int pairs = resident_pairs<ACT>(sms);
  if (pairs <= 0) return ITTT_ERR_CUDA;
  if (cdiv(a.N, 128) * cdiv(a.M, 128) > sms) return linear_pairs<ACT>(a, pairs, st);
  if (cdiv(a.N, 128) * cdiv(a.M, 128) * 8 < sms) return linear_split<64, ACT>(a, sms, st);
  return linear_split<128, ACT>(a, sms, st);
}

template <int ACT>
ittt_status linear_typed(const LinearArgs<__nv_bfloat16>& a, cudaStream_t st) {
  return linear_bf16<ACT>(a, st);
}
template <int ACT>
ittt_status linear_typed(const LinearArgs<float>& a, cudaStream_t st) {
  return linear_f32<ACT>(a, st);
}

template <typename T_>
ittt_status linear_by_act(const LinearArgs<T_>& a, cudaStream_t st) {
  switch (a.act) {
    case ITTT_ACT_RELU: return linear_typed<ITTT_ACT_RELU>(a, st);
    case ITTT_ACT_SILU: return linear_typed<ITTT_ACT_SILU>(a, st);
    case ITTT_ACT_GELU: return linear_typed<ITTT_ACT_GELU>(a, st);
    case ITTT_ACT_GELU_TANH: return linear_typed<ITTT_ACT_GELU_TANH>(a, st);
    default: return linear_typed<ITTT_ACT_NONE>(a, st);
  }
}

// ------------------------------------------------------------- causal conv

ittt_status validate_conv(const ittt_conv_problem* p) {
  if (!p || p->B <= 0 || p->T <= 0 || p->d <= 0 || p->k <= 0 || p->ldx < 0 || p->ldy < 0 ||
      p->reserved != 0 || !valid_dtype_act(p->dtype, p->act))
    return ITTT_ERR_INVALID_ARG;
  if ((p->ldx && p->ldx < p->d) || (p->ldy && p->ldy < p->d)) return ITTT_ERR_INVALID_ARG;
  if (p->k > 16 || p->B > 65535 || p->T > (1ll << 30) ||
      !fits(p->B * p->T, p->d, p->ldx) || !fits(p->B * p->T, p->d, p->ldy))
    return ITTT_ERR_UNSUPPORTED;
  return ITTT_OK;
}

// CTAs of a kernel without dynamic shared memory that an SM of the current device holds
// (0: the device does not say).
template <typename Kern>
int resident_ctas(Kern kern, int threads, std::atomic<int>* known) {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, 0) != cudaSuccess) return 0;
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Steps of four tokens a thread: 8 while that leaves every SM 16 warps, down to 2.  More
// CTAs than the GPU holds at once: the number from 6 to 18 that wastes least of the last
// wave (a thread's start counts as one step): 8192 x 5120 takes 35.2 us in one wave of 18
// steps and 35.1 us in two of 9, but 36.4 us in 8 steps, whose third wave is a sixth
// full, and 40.4 us in 16.
template <typename T_, int V, int KT, int ACT>
ittt_status causal_conv_vec(const CausalConvArgs<T_>& a, cudaStream_t st) {
  const int sms = num_sms();
  if (sms <= 0) return ITTT_ERR_CUDA;
  const long long groups = a.d / V;
  int steps = 8;
  while (steps > 2 && a.B * cdiv(a.T, 4 * steps) * groups < 512ll * sms) steps /= 2;
  auto kern = causal_conv_vec_kernel<T_, V, KT, ACT>;
  static std::atomic<int> known[kMaxDevices] = {};
  const long long slots = (long long)resident_ctas(kern, 128, known) * sms;
  if (slots <= 0) return ITTT_ERR_CUDA;
  auto ctas = [&](int n) { return cdiv(a.B * cdiv(a.T, 4 * n) * groups, 128); };
  if (ctas(steps) > slots) {
    long long best = 0;
    for (int n = 6; n <= 18; ++n) {
      const long long cost = cdiv(ctas(n), slots) * (n + 1);
      if (n == 6 || cost < best) best = cost, steps = n;
    }
  }
  const long long runs = cdiv(a.T, 4 * steps), total = a.B * runs * groups;
  if (total >= (1ll << 32) - 128) return ITTT_ERR_UNSUPPORTED;
  return launch_pdl(kern, dim3(unsigned(cdiv(total, 128))), dim3(128), st, a, unsigned(total),
                    unsigned(groups), unsigned(runs), steps);
}

template <typename T_, int V, int KT>
ittt_status causal_conv_act(const CausalConvArgs<T_>& a, cudaStream_t st) {
  if (a.act == ITTT_ACT_SILU) return causal_conv_vec<T_, V, KT, ITTT_ACT_SILU>(a, st);
  if (a.act == ITTT_ACT_NONE) return causal_conv_vec<T_, V, KT, ITTT_ACT_NONE>(a, st);
  return causal_conv_vec<T_, V, KT, -1>(a, st);  // by a.act
}

template <typename T_, int V>
ittt_status causal_conv_taps(const CausalConvArgs<T_>& a, cudaStream_t st) {
  switch (a.k) {
    case 1: return causal_conv_act<T_, V, 1>(a, st);
    case 2: return causal_conv_act<T_, V, 2>(a, st);
    case 3: return causal_conv_act<T_, V, 3>(a, st);
    case 4: return causal_conv_act<T_, V, 4>(a, st);
    case 5: return causal_conv_act<T_, V, 5>(a, st);
    case 6: return causal_conv_act<T_, V, 6>(a, st);
    case 7: return causal_conv_act<T_, V, 7>(a, st);
    default: return causal_conv_act<T_, V, 8>(a, st);
  }
}

template <typename T_>
ittt_status causal_conv_launch(const ittt_conv_problem* p, const void* X, const void* w,
                               const void* bias, const void* state_in, const int32_t* lengths,
                               void* Y, void* state_out, cudaStream_t st) {
  CausalConvArgs<T_> a{};
  a.X = static_cast<const T_*>(X);
  a.w = static_cast<const T_*>(w);
  a.bias = static_cast<const T_*>(bias);
  a.state_in = p->k > 1 ? static_cast<const T_*>(state_in) : nullptr;
  a.lengths = lengths;
  a.Y = static_cast<T_*>(Y);
  a.state_out = p->k > 1 ? static_cast<T_*>(state_out) : nullptr;
  a.ldx = stride_or(p->ldx, p->d);
  a.ldy = stride_or(p->ldy, p->d);
  a.B = int(p->B);
  a.T = int(p->T);
  a.d = int(p->d);
  a.k = p->k;
  a.act = p->act;
  constexpr int V = 16 / int(sizeof(T_));
  const bool vec = p->d % V == 0 && a.ldx % V == 0 && a.ldy % V == 0 && aligned16(X) &&
                   aligned16(w) && aligned16(Y) && aligned16(a.state_in) && aligned16(a.state_out);
  if (p->k <= 8) return vec ? causal_conv_taps<T_, V>(a, st) : causal_conv_taps<T_, 1>(a, st);
  const long long rest = p->T - (p->k - 1);
  const long long gy = 1 + (rest > 0 ? cdiv(rest, 16) : 0);
  if (gy > 65535) return ITTT_ERR_UNSUPPORTED;
  return launch_pdl(causal_conv_kernel<T_>,
                    dim3(unsigned(cdiv(p->d, 256)), unsigned(gy), unsigned(p->B)), dim3(256), st, a);
}

// ---------------------------------------------------------- selective scan

ittt_status validate_scan(const ittt_scan_problem* p) {
  if (!p || p->B <= 0 || p->T <= 0 || p->d <= 0 || p->N <= 0 || p->G <= 0 ||
      (p->dtype != ITTT_F32 && p->dtype != ITTT_BF16) || (p->flags & ~ITTT_SCAN_SOFTPLUS) != 0)
    return ITTT_ERR_INVALID_ARG;
  const int64_t gn = int64_t(p->G) * p->N;
  const int64_t ld[] = {p->ldu, p->ldt, p->ldz, p->ldy, p->ldb, p->ldc};
  for (int i = 0; i < 6; ++i)
    if (ld[i] < 0 || (ld[i] && ld[i] < (i < 4 ? p->d : gn))) return ITTT_ERR_INVALID_ARG;
  if (p->d % p->G != 0) return ITTT_ERR_INVALID_ARG;
  // the walk over sequences (and the one over tokens) may step past its end in 32 bits
  if (p->N > 256 || p->B > (1ll << 30) || p->T > (1ll << 30)) return ITTT_ERR_UNSUPPORTED;
  for (int i = 0; i < 6; ++i)
    if (!fits(p->B * p->T, i < 4 ? p->d : gn, ld[i])) return ITTT_ERR_UNSUPPORTED;
  if (p->B * p->d >= (1ll << 31)) return ITTT_ERR_UNSUPPORTED;
  return ITTT_OK;
}

template <typename T_>
ScanArgs<T_> scan_args(const ittt_scan_problem* p, const void* U, const void* delta, const float* A,
                       const void* Bm, const void* Cm, const float* D, const float* dt_bias,
                       const void* Z, const float* state_in, const int32_t* lengths, void* Y,
                       float* state_out) {
  ScanArgs<T_> a{};
  a.U = static_cast<const T_*>(U);
  a.delta = static_cast<const T_*>(delta);
  a.Bm = static_cast<const T_*>(Bm);
  a.Cm = static_cast<const T_*>(Cm);
  a.Z = static_cast<const T_*>(Z);
  a.A = A;
  a.D = D;
  a.dt_bias = dt_bias;
  a.state_in = state_in;
  a.lengths = lengths;
  a.Y = static_cast<T_*>(Y);
  a.state_out = state_out;
  const long long gn = (long long)p->G * p->N;
  a.ldu = stride_or(p->ldu, p->d);
  a.ldt = stride_or(p->ldt, p->d);
  a.ldb = stride_or(p->ldb, gn);
  a.ldc = stride_or(p->ldc, gn);
  a.ldz = stride_or(p->ldz, p->d);
  a.ldy = stride_or(p->ldy, p->d);
  a.B = int(p->B);
  a.T = int(p->T);
  a.d = int(p->d);
  a.N = p->N;
  a.G = p->G;
  a.softplus = p->flags & ITTT_SCAN_SOFTPLUS;
  return a;
}

// How a call is cut (see ScanPlan).  short_call: the serial kernel.
struct ScanCut {
  bool short_call, chained;
  int passes;                            // the chunk kernel's P
  int runs, run_tokens, blocks, per_group;
  size_t flags, carry, step_sum, total;  // workspace offsets and size
};

ScanCut scan_cut(const ittt_scan_problem* p, int sms) {
  ScanCut c{};
  const int ctas = p->dtype == ITTT_BF16 ? ScanShape<__nv_bfloat16, 1>::CTAS : ScanShape<float, 1>::CTAS;
  const long long workers = (long long)ctas * sms;
  // the wider channel blocks where they still fill the GPU (few, long sequences: as
  // independent runs), the narrow ones else; a state of more than one slab of B and C
  // would be staged once a pass and gain nothing, and the kernel has no code for it
  const long long wide = p->B * p->G * cdiv(p->d / p->G, scan_ch(2));
  const bool few = wide * 4 < workers && cdiv(p->T, kScanChunk) * wide >= 4 * workers;
  c.passes = p->dtype == ITTT_BF16 && p->N <= ScanShape<__nv_bfloat16, 2>::SLAB && (wide >= workers || few) ? 2 : 1;
  c.per_group = int(cdiv(p->d / p->G, scan_ch(c.passes)));
  c.blocks = c.per_group * p->G;
  const long long groups = p->B * c.blocks;
  // Token after token, or chunks.  Measured at N = 4, 16, 64, B = 1, 8, 32 and d = 512
  // to 5120 (us): the serial kernel takes 0.24 a token, or 1.4e-6 a state element and
  // token where that is more; a wave of chunks 4 + 0.42 N, at least 7.5 in all.
  // (B 8, d 5120, N 16: 60 and 116 at T = 64, 117 and 120 at 128, 229 and 138 at 256;
  // B 1, d 512: 7.8 and 7.6 at T = 33.  B 32, d 1024, N 4: 57 and 97 at T = 256.)
  const double elements = double(p->B) * p->d * p->T * double((p->N + 3) / 4 * 4);
  const double serial_us = std::max(2.0 + 0.24 * p->T, 1.4e-6 * elements);
  // Rows of channels that do not split into 16-byte pieces are staged element by element:
  // 7 more a pass (B 9, T 3432, d 3033, N 4: 1526 in chunks, 28 a wave instead of 13.5;
  // 739 token after token).
  const int64_t V = p->dtype == ITTT_BF16 ? 8 : 4;
  const bool pieces = (p->d / p->G) % V == 0 && stride_or(p->ldu, p->d) % V == 0 &&
                      stride_or(p->ldt, p->d) % V == 0 && stride_or(p->ldz, p->d) % V == 0 &&
                      stride_or(p->ldy, p->d) % V == 0;
  const double wave = (c.passes == 2 ? 11.7 + 0.45 * p->N : 4.0 + 0.42 * p->N) + (pieces ? 0.0 : 7.0 * c.passes);
  const double chunk_us = std::max(c.passes == 2 ? 13.0 : 7.5,
                                   double(groups) * cdiv(p->T, kScanChunk) / workers * wave);
  c.short_call = p->T == 1 || serial_us < chunk_us;
  if (c.short_call) return c;
  const long long chunks = cdiv(p->T, kScanChunk);
  long long run_chunks = chunks;
  // One pass over whole sequences, or independent runs whose two passes and join cost
  // less.  A chunk takes a CTA 0.6 of a wave's time when it has the SM to itself, all of
  // it when the SM is full; the state pass does 0.6 of the other's work, and a task
  // costs half a chunk more than its chunks.
  auto chunk_time = [&](double tasks) { return wave * (0.6 + 0.4 * std::min(1.0, tasks / workers)); };
  double best = double(chunks) * chunk_time(double(groups)) * std::max(1.0, double(groups) / workers);
  bool split = false;
  for (long long rc = 1; rc < chunks; rc += std::max(1ll, rc / 8)) {
    const long long tasks = groups * cdiv(chunks, rc);
    const double cost =
        1.6 * (double(rc) + 0.5) * double(cdiv(tasks, workers)) * chunk_time(double(tasks)) + 4.0;
    if (cost < best) {
      best = cost;
      run_chunks = rc;
      split = true;
    }
  }
  if (!split && groups >= sms && groups < 6 * workers) {
    // runs of four chunks, chained, so that the work is dealt out evenly however many
    // channel blocks there are
    c.chained = true;
    run_chunks = std::min(chunks, 4ll);
  }
  c.run_tokens = int(run_chunks * kScanChunk);
  c.runs = int(cdiv(chunks, run_chunks));
  if (c.runs == 1) return c;
  const long long np = scan_np(p->N);
  size_t off = 0;
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  if (c.chained) {
    c.flags = take(size_t(1 + groups) * 4);
    c.carry = take(size_t(groups) * scan_ch(c.passes) * np * 4);
  } else {
    c.carry = take(size_t(c.runs) * p->B * p->d * p->N * 4);
    c.step_sum = take(size_t(c.runs - 1) * p->B * p->d * 4);
  }
  c.total = off;
  return c;
}

template <typename T_, bool VEC>
ittt_status scan_short_sized(const ScanArgs<T_>& a, int sms, cudaStream_t st) {
  const int npl = a.N <= 128 ? 4 : 8;
  int lanes = 1;
  while (lanes * npl < a.N) lanes *= 2;
  const long long threads = (long long)a.d * lanes;
  auto launch = [&](auto kern, long long batches) {
    return launch_pdl(kern, dim3(unsigned(cdiv(batches * threads, 128))), dim3(128), st, a, lanes);
  };
  if (a.T == 1 && npl == 4) {
    // ten CTAs of 128 threads an SM, all resident, share the sequences (64 sequences of
    // 5120 x 16: 12.9 us, 13.2 with eight, 14.0 with six or with all sequences at once)
    const long long x = cdiv(threads, 128);
    const long long y = std::max(1ll, std::min<long long>(a.B, 10ll * sms / x));
    return launch_pdl(scan_token_kernel<T_, VEC>, dim3(unsigned(x), unsigned(std::min(y, 65535ll))),
                      dim3(128), st, a, lanes);
  }
  if (npl == 4) return launch(scan_serial_kernel<T_, 4, VEC>, a.B);
  return launch(scan_serial_kernel<T_, 8, VEC>, a.B);
}

template <typename T_>
ittt_status scan_short(const ScanArgs<T_>& a, int sms, cudaStream_t st) {
  constexpr uintptr_t quad = 4 * sizeof(T_) - 1;
  const bool vec = a.N % 4 == 0 && a.ldb % 4 == 0 && a.ldc % 4 == 0 && aligned16(a.A) &&
                   aligned16(a.state_in) && aligned16(a.state_out) &&
                   ((reinterpret_cast<uintptr_t>(a.Bm) | reinterpret_cast<uintptr_t>(a.Cm)) & quad) == 0;
  return vec ? scan_short_sized<T_, true>(a, sms, st) : scan_short_sized<T_, false>(a, sms, st);
}

template <typename T_, int P, bool STATE_ONLY>
ittt_status scan_chunks_wide(const ScanArgs<T_>& a, const ScanPlan& pl, long long tasks, int sms,
                             cudaStream_t st) {
  static std::atomic<bool> granted[kMaxDevices] = {};
  auto kern = scan_chunk_kernel<T_, P, STATE_ONLY>;
  if (!grant_smem(kern, scan_smem_bytes<T_, P>(256), granted)) return ITTT_ERR_CUDA;
  const long long grid = std::min<long long>(tasks, (long long)ScanShape<T_, P>::CTAS * sms);
  return launch_clusters(kern, unsigned(grid), 1, kScanThreads, scan_smem_bytes<T_, P>(a.N), st, a, pl,
                         g_wait_ns.load());
}

template <typename T_, bool STATE_ONLY>
ittt_status scan_chunks(const ScanArgs<T_>& a, const ScanPlan& pl, int passes, long long tasks, int sms,
                        cudaStream_t st) {
  if constexpr (sizeof(T_) == 2) {
    if (passes == 2) return scan_chunks_wide<T_, 2, STATE_ONLY>(a, pl, tasks, sms, st);
  }
  return scan_chunks_wide<T_, 1, STATE_ONLY>(a, pl, tasks, sms, st);
}

template <typename T_>
ittt_status scan_launch(const ittt_scan_problem* p, const ScanArgs<T_>& a, void* workspace,
                        size_t workspace_bytes, cudaStream_t st) {
  const int sms = num_sms();
  if (sms <= 0) return ITTT_ERR_CUDA;
  const ScanCut c = scan_cut(p, sms);
  if (c.total && (!workspace || workspace_bytes < c.total)) return ITTT_ERR_WORKSPACE;
  if (c.total && !aligned16(workspace)) return ITTT_ERR_UNSUPPORTED;
  if (c.short_call) return scan_short(a, sms, st);
  char* ws = static_cast<char*>(workspace);
  ScanPlan pl{};
  pl.blocks = c.blocks;
  pl.per_group = c.per_group;
  pl.runs = c.runs;
  pl.run_tokens = c.run_tokens;
  pl.chained = c.chained;
  const long long groups = p->B * c.blocks;
  if (groups * c.runs >= (1ll << 31)) return ITTT_ERR_UNSUPPORTED;
  if (c.runs > 1) {
    pl.carry = reinterpret_cast<float*>(ws + c.carry);
    if (c.chained) {
      pl.flags = reinterpret_cast<unsigned*>(ws + c.flags);
      if (cudaMemsetAsync(pl.flags, 0, size_t(1 + groups) * 4, st) != cudaSuccess) return ITTT_ERR_CUDA;
    } else {
      pl.step_sum = reinterpret_cast<float*>(ws + c.step_sum);
      ittt_status s = scan_chunks<T_, true>(a, pl, c.passes, groups * (c.runs - 1), sms, st);
      if (s != ITTT_OK) return s;
      s = launch_pdl(scan_join_kernel<T_>, dim3(unsigned(cdiv((long long)a.B * a.d * a.N, 256))),
                     dim3(256), st, a, pl);
      if (s != ITTT_OK) return s;
    }
  }
  return scan_chunks<T_, false>(a, pl, c.passes, groups * c.runs, sms, st);
}

}  // namespace

extern "C" {

ittt_status ittt_linear(const ittt_linear_problem* p, const void* X, const void* W,
                        const void* bias, const void* residual, void* Y, void* stream) {
  const NvtxRange nvtx_range("ittt_linear");
  ittt_status s = validate_linear(p);
  if (s != ITTT_OK) return s;
  if (!X || !W || !Y || Y == X || Y == W || Y == bias) return ITTT_ERR_INVALID_ARG;
  if (residual == Y && stride_or(p->ldr, p->N) != stride_or(p->ldy, p->N)) return ITTT_ERR_INVALID_ARG;
  const size_t es = p->dtype == ITTT_BF16 ? 2 : 4;
  if ((s = check_buffers({{X, span_bytes(p->M, stride_or(p->ldx, p->K), p->K, es)},
                          {W, size_t(p->N) * p->K * es},
                          {bias, size_t(p->N) * es},
                          {residual, span_bytes(p->M, stride_or(p->ldr, p->N), p->N, es)},
                          {Y, span_bytes(p->M, stride_or(p->ldy, p->N), p->N, es)}})) != ITTT_OK)
    return s;
  if (p->dtype == ITTT_BF16) {
    if (!aligned16(X) || !aligned16(W)) return ITTT_ERR_UNSUPPORTED;
    return linear_by_act(linear_args<__nv_bfloat16>(p, X, W, bias, residual, Y), as_stream(stream));
  }
  return linear_by_act(linear_args<float>(p, X, W, bias, residual, Y), as_stream(stream));
}

ittt_status ittt_causal_conv(const ittt_conv_problem* p, const void* X, const void* conv_kernel,
                             const void* bias, const void* state_in, const int32_t* lengths,
                             void* Y, void* state_out, void* stream) {
  const NvtxRange nvtx_range("ittt_causal_conv");
  ittt_status s = validate_conv(p);
  if (s != ITTT_OK) return s;
  if (!X || !conv_kernel || !Y || X == Y || Y == state_in || Y == state_out || Y == conv_kernel || Y == bias)
    return ITTT_ERR_INVALID_ARG;
  if (state_out && p->k > 1 && (state_out == X || state_out == conv_kernel || state_out == bias))
    return ITTT_ERR_INVALID_ARG;
  const size_t es = p->dtype == ITTT_BF16 ? 2 : 4;
  const long long rows = p->B * p->T;
  const size_t state = size_t(p->B) * size_t(p->k - 1) * p->d * es;
  if ((s = check_buffers({{X, span_bytes(rows, stride_or(p->ldx, p->d), p->d, es)},
                          {conv_kernel, size_t(p->d) * p->k * es},
                          {bias, size_t(p->d) * es},
                          {state_in, state},
                          {lengths, size_t(p->B) * 4},
                          {Y, span_bytes(rows, stride_or(p->ldy, p->d), p->d, es)},
                          {state_out, state}})) != ITTT_OK)
    return s;
  if (p->dtype == ITTT_BF16)
    return causal_conv_launch<__nv_bfloat16>(p, X, conv_kernel, bias, state_in, lengths, Y,
                                             state_out, as_stream(stream));
  return causal_conv_launch<float>(p, X, conv_kernel, bias, state_in, lengths, Y, state_out,
                                   as_stream(stream));
}

ittt_status ittt_selective_scan_workspace_size(const ittt_scan_problem* p, size_t* bytes) {
  if (!bytes) return ITTT_ERR_INVALID_ARG;
  const ittt_status s = validate_scan(p);
  if (s != ITTT_OK) return s;
  const int sms = num_sms();
  if (sms <= 0) return ITTT_ERR_CUDA;
  *bytes = scan_cut(p, sms).total;
  return ITTT_OK;
}

ittt_status ittt_selective_scan(const ittt_scan_problem* p, const void* U, const void* delta,
                                const float* A, const void* Bm, const void* Cm, const float* D,
                                const float* dt_bias, const void* Z, const float* state_in,
                                const int32_t* lengths, void* Y, float* state_out, void* workspace,
                                size_t workspace_bytes, void* stream) {
  const NvtxRange nvtx_range("ittt_selective_scan");
  ittt_status s = validate_scan(p);
  if (s != ITTT_OK) return s;
  if (!U || !delta || !A || !Bm || !Cm || !Y) return ITTT_ERR_INVALID_ARG;
  if (Y == state_in || Y == state_out) return ITTT_ERR_INVALID_ARG;
  for (const void* in : {U, delta, Z, Bm, Cm, static_cast<const void*>(A), static_cast<const void*>(D),
                         static_cast<const void*>(dt_bias)})
    if (in && (Y == in || state_out == in)) return ITTT_ERR_INVALID_ARG;
  const size_t es = p->dtype == ITTT_BF16 ? 2 : 4;
  const long long rows = p->B * p->T, gn = (long long)p->G * p->N;
  const size_t state = size_t(p->B) * p->d * p->N * 4;
  if ((s = check_buffers({{U, span_bytes(rows, stride_or(p->ldu, p->d), p->d, es)},
                          {delta, span_bytes(rows, stride_or(p->ldt, p->d), p->d, es)},
                          {A, size_t(p->d) * p->N * 4},
                          {Bm, span_bytes(rows, stride_or(p->ldb, gn), gn, es)},
                          {Cm, span_bytes(rows, stride_or(p->ldc, gn), gn, es)},
                          {D, size_t(p->d) * 4},
                          {dt_bias, size_t(p->d) * 4},
                          {Z, span_bytes(rows, stride_or(p->ldz, p->d), p->d, es)},
                          {state_in, state},
                          {lengths, size_t(p->B) * 4},
                          {Y, span_bytes(rows, stride_or(p->ldy, p->d), p->d, es)},
                          {state_out, state},
                          {workspace, workspace_bytes}})) != ITTT_OK)
    return s;
  if (p->dtype == ITTT_BF16)
    return scan_launch(p, scan_args<__nv_bfloat16>(p, U, delta, A, Bm, Cm, D, dt_bias, Z, state_in,
                                                   lengths, Y, state_out),
                       workspace, workspace_bytes, as_stream(stream));
  return scan_launch(p, scan_args<float>(p, U, delta, A, Bm, Cm, D, dt_bias, Z, state_in, lengths, Y,
                                         state_out),
                     workspace, workspace_bytes, as_stream(stream));
}

}  // extern "C"

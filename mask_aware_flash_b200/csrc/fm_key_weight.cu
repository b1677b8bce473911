// Attention weight that each key of a prompt receives (fm_attn_key_weight), for sm_100a (tcgen05 + TMEM + TMA).
//
//   weight_j = sum over heads h of the group, rows i of  exp(scale q_i.k_j - LSE_i)   [unmasked pairs]
//
// One key tile of 128 keys and K/V head per CTA (or per cluster of CTAs that share its work): the tile's K stays
// in shared memory, the query tiles of its column lists (skip tiles never loaded) stream past it, head by head:
//   S^T = K Q^T  (tcgen05, M = 128 keys, N = 128 queries) -> one of four TMEM buffers
// so a thread holds one key: its sum stays in registers, its mask bounds too, and the interval test is a word of
// bits per 32 queries.  Per score there is one exponential against 2 D flops of the tensor core: for D = 128 the
// exponentials bound the kernel (16384 per tile at 16 per clock on the MUFU unit = 1024 clocks, against 512 of
// the product).
// Warps 0-3 / 4-7 take the even / odd query tiles, warp 8 issues the TMA loads, warp 9 the MMAs.
#include "fm_common.cuh"

namespace fm {
fm_status check_attn_args(const fm_attn_args* a, const fm_mask_meta* meta, const int32_t* const vec[4]);

namespace {

constexpr int kTile = 128;
constexpr int kThreads = 320;
constexpr int kBufs = 4;  // TMEM score buffers of 128 columns
constexpr float kNegInf = -__builtin_huge_valf();

struct KeyWeightParams {
  const int32_t* col_count;    // [B, Hm, T_k]
  const int32_t* col_entries;  // [B, Hm, T_k, T_q]
  const int32_t* order;        // [B, Hm, T_k] key tiles, longest first
  const int32_t* vec[4];       // [B, Hm, n_k] or null
  const float* lse;            // [B, H, n_q]
  float* weight;
  int64_t weight_stride;
  int* status;
  int H, Hm, H_kv, q_per_kv, n_q, n_k, T_q, T_k, accumulate;
  float scale_log2;
};

template <int D>
struct KeyWeightSmem {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 256 ? 2 : D == 128 ? 5 : 8;  // query tiles in flight
  static constexpr int kK = 0;
  static constexpr int kQ = kK + kTileBytes;
  static constexpr int kLse = kQ + kStages * kTileBytes;  // [2 warpgroups][2][128] -log2 LSE
  static constexpr int kSum = kLse + 2 * 2 * kTile * 4;   // [128] sums of the second warpgroup / of the CTA
  static constexpr int kBar = kSum + kTile * 4;
  enum { K_FULL, Q_FULL, Q_EMPTY = Q_FULL + kStages, S_FULL = Q_EMPTY + kStages, S_EMPTY = S_FULL + kBufs,
         DRAIN = S_EMPTY + kBufs, kNumBars };
  static constexpr int kMisc = kBar + kNumBars * 8;  // [0] TMEM base, [1] abort flag, [2] zero
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {  // another CTA's shared memory
  float v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [a];\n\t}"
      : "=f"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// The items (query head of the group, query tile) of one key tile in their fixed order; CTA `rank` of a cluster
// of `step` takes items rank, rank + step, ...
struct ItemWalk {
  const int32_t* count;    // column count of the first head's list
  const int32_t* entries;
  int64_t head_count, head_entries;  // distance to the next head's (0 when all heads share one mask)
  int heads;
  int head, n, at;
  __device__ __forceinline__ void start(int rank) {
    head = -1;
    n = 0;
    at = rank;
  }
  // moves to the item `at`; false behind the last one
  __device__ __forceinline__ bool get(int& hg, int& entry) {
    while (at >= n) {
      if (head + 1 >= heads) return false;
      at -= n;
      ++head;
      n = __ldg(count + head * head_count);
    }
    hg = head;
    entry = __ldg(entries + head * head_entries + at);
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    key_weight_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const KeyWeightParams p) {
  using S = KeyWeightSmem<D>;
  constexpr int kAtoms = D / 64;  // 128-byte swizzle-atom columns of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_base_1024(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), step = (int)cluster_size();
  const int hk = blockIdx.y, b = blockIdx.z;
  const int64_t bhm0 = (int64_t)b * p.Hm + (p.Hm == 1 ? 0 : hk * p.q_per_kv);
  const int kt = __ldg(p.order + bhm0 * p.T_k + blockIdx.x / step);

  ItemWalk walk;
  walk.count = p.col_count + bhm0 * p.T_k + kt;
  walk.entries = p.col_entries + (bhm0 * p.T_k + kt) * p.T_q;
  walk.head_count = p.Hm == 1 ? 0 : p.T_k;
  walk.head_entries = p.Hm == 1 ? 0 : (int64_t)p.T_k * p.T_q;
  walk.heads = p.q_per_kv;

  const uint32_t bar0 = smem_u32(smem + S::kBar);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  const volatile int* never = reinterpret_cast<const volatile int*>(misc + 2);
  const uint32_t k_s = smem_u32(smem + S::kK), q_s = smem_u32(smem + S::kQ);
  float* lse_s = reinterpret_cast<float*>(smem + S::kLse);
  float* sum_s = reinterpret_cast<float*>(smem + S::kSum);

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kNumBars; ++i) mbar_init(bar(i), 1);
    for (int i = 0; i < kBufs; ++i) mbar_init(bar(S::S_EMPTY + i), kTile);
    *abort_flag = 0;
    misc[2] = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  float sum = 0.f;

  if (warp == 8) {
    // ------------------------------------------------------------ load role
    if (lane == 0) {
      int hg, entry;
      walk.start(rank);
      bool ok = true;
      int i = 0;
      for (; walk.get(hg, entry); ++i, walk.at += step) {
        if (i == 0) {
          mbar_arrive_expect_tx(bar(S::K_FULL), S::kTileBytes);
          for (int c = 0; c < kAtoms; ++c) tma_load_4d(k_s + c * 16384, &tm_k, bar(S::K_FULL), c * 64, hk, kt * kTile, b);
        }
        const int st = i % S::kStages;
        if (i >= S::kStages && !mbar_wait(bar(S::Q_EMPTY + st), (i / S::kStages - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(bar(S::Q_FULL + st), S::kTileBytes);
        for (int c = 0; c < kAtoms; ++c)
          tma_load_4d(q_s + st * S::kTileBytes + c * 16384, &tm_q, bar(S::Q_FULL + st), c * 64, hk * p.q_per_kv + hg,
                      (entry >> 1) * kTile, b);
      }
      if (!ok) record_failure(p.status, abort_flag, 61);
      // the copies in flight land before this role ends (a consumer that gave up may leave some unread)
      if (i > 0) mbar_wait(bar(S::K_FULL), 0, never);
      for (int x = max(i - S::kStages, 0); x < i; ++x) mbar_wait(bar(S::Q_FULL + x % S::kStages), (x / S::kStages) & 1, never);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------- MMA role
    if (lane == 0) {
      constexpr uint32_t kIdesc = idesc_bf16(128, 128, false, false);
      constexpr uint32_t kHi = desc_hi(1024);
      const uint32_t lo_k = desc_lo(k_s, 16), lo_q = desc_lo(q_s, 16);
      int hg, entry;
      walk.start(rank);
      bool ok = true;
      int i = 0;
      for (; walk.get(hg, entry); ++i, walk.at += step) {
        const int st = i % S::kStages, buf = i % kBufs;
        if ((i == 0 && !mbar_wait(bar(S::K_FULL), 0, abort_flag)) ||
            !mbar_wait(bar(S::Q_FULL + st), (i / S::kStages) & 1, abort_flag) ||
            (i >= kBufs && !mbar_wait(bar(S::S_EMPTY + buf), (i / kBufs - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t qa = lo_q + st * (S::kTileBytes >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
          umma_ss_w(tmem + buf * 128, lo_k + off, kHi, qa + off, kHi, kIdesc, k > 0 ? 1u : 0u);
        }
        umma_commit(bar(S::Q_EMPTY + st));
        umma_commit(bar(S::S_FULL + buf));
      }
      if (!ok) record_failure(p.status, abort_flag, 62);
      umma_commit(bar(S::DRAIN));  // every MMA has finished before TMEM is released
      mbar_wait(bar(S::DRAIN), 0, never);
    }
  } else {
    // ------------------------------------------------------- exponentials and sums: one key per thread
    const int wg = warp >> 2, r = threadIdx.x & 127;
    const int key = kt * kTile + r;
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    float* my_lse = lse_s + wg * 2 * kTile;
    const uint64_t sc2 = f2pack(p.scale_log2, p.scale_log2);
    uint64_t acc[4] = {0, 0, 0, 0};
    int at_head = -1;
    int32_t lts = 0, lte = 0, uts = 0, ute = 0;
    walk.start(rank);
    int hg, entry;
    bool ok = true;
    for (int i = 0; walk.get(hg, entry); ++i, walk.at += step) {
      if ((i & 1) != wg) continue;
      const int qt = entry >> 1, q0 = qt * kTile, buf = i % kBufs, lb = (i >> 1) & 1;
      const bool ragged = q0 + kTile > p.n_q, partial = (entry & 1) || ragged;
      // -LSE in log2 units, -inf for rows that see no key and rows past n_q (their p is 0)
      {
        const int row = q0 + r;
        const float x = row < p.n_q ? __ldg(p.lse + ((int64_t)b * p.H + hk * p.q_per_kv + hg) * p.n_q + row) : kNegInf;
        my_lse[lb * kTile + r] = x == kNegInf ? kNegInf : -x * 1.4426950408889634f;
      }
      if (partial && hg != at_head) {  // this key's bounds
        const int64_t at = (bhm0 + (p.Hm == 1 ? 0 : hg)) * p.n_k + key;
        const bool in = key < p.n_k;
        lts = in && p.vec[0] ? __ldg(p.vec[0] + at) : p.n_q;
        lte = in && p.vec[1] ? __ldg(p.vec[1] + at) : p.n_q;
        uts = in && p.vec[2] ? __ldg(p.vec[2] + at) : 0;
        ute = in && p.vec[3] ? __ldg(p.vec[3] + at) : 0;
        at_head = hg;
      }
      named_bar_sync(1 + wg, 128);  // the values are there; the pair before last has been read
      ok = __all_sync(0xffffffffu, mbar_wait(bar(S::S_FULL + buf), (i / kBufs) & 1, abort_flag)) && ok;
      tc_fence_after();
      uint32_t s[128];
      tmem_ld128(tmem + buf * 128 + lane_addr, s);
      tc_fence_before();
      mbar_arrive(bar(S::S_EMPTY + buf));
      const float4* nl = reinterpret_cast<const float4*>(my_lse + lb * kTile);
#pragma unroll
      for (int c = 0; c < kTile; c += 4) {
        const float4 v = nl[c / 4];
        const uint64_t x0 = fma2(f2pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, f2pack(v.x, v.y));
        const uint64_t x1 = fma2(f2pack(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), sc2, f2pack(v.z, v.w));
        s[c] = __float_as_uint(ex2(f2lo(x0)));
        s[c + 1] = __float_as_uint(ex2(f2hi(x0)));
        s[c + 2] = __float_as_uint(ex2(f2lo(x1)));
        s[c + 3] = __float_as_uint(ex2(f2hi(x1)));
      }
      if (partial) {
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
          const int base = q0 + jb * 32;
          uint32_t mw = interval_bits32(lts, lte, base) | interval_bits32(uts, ute, base);
          if (ragged) mw |= base + 32 <= p.n_q ? 0u : base >= p.n_q ? 0xFFFFFFFFu : 0xFFFFFFFFu << (p.n_q - base);
          if (__any_sync(0xffffffffu, mw != 0u)) {
#pragma unroll
            for (int c = 0; c < 32; ++c) s[jb * 32 + c] = ((mw >> c) & 1u) ? 0u : s[jb * 32 + c];
          }
        }
      }
#pragma unroll
      for (int c = 0; c < kTile; c += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          acc[u] = add2(acc[u], f2pack(__uint_as_float(s[c + 2 * u]), __uint_as_float(s[c + 2 * u + 1])));
    }
    if (!ok && lane == 0) record_failure(p.status, abort_flag, 63);
    const uint64_t a = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
    sum = f2lo(a) + f2hi(a);
    if (wg == 1) sum_s[r] = sum;
  }

  __syncthreads();  // (also: the MMA warp has drained)
  if (warp < 4) {
    sum += sum_s[threadIdx.x];
    if (step > 1) sum_s[threadIdx.x] = sum;
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (step > 1) cluster_sync_all();
  const int key = kt * kTile + (int)threadIdx.x;
  if (rank == 0 && warp < 4 && key < p.n_k) {
    for (int c = 1; c < step; ++c) sum += ld_cluster_f32(smem_u32(sum_s + threadIdx.x), c);
    float* w = p.weight + ((int64_t)b * p.H_kv + hk) * p.weight_stride + key;
    *w = p.accumulate ? *w + sum : sum;
  }
  if (step > 1) cluster_sync_all();  // no CTA leaves while its sums are read
}

template <int D>
fm_status launch_key_weight(const fm_attn_args* a, const KeyWeightParams& p, int H_kv, cudaStream_t stream) {
  using S = KeyWeightSmem<D>;
  static_assert(S::kAlloc <= 227 * 1024, "shared memory exceeds the per-CTA limit");
  CUtensorMap tq, tk;
  if (!encode_tmap_bf16_4d(&tq, a->q, D, a->H, a->n_q, a->B, kTile) ||
      !encode_tmap_bf16_4d(&tk, a->k, D, H_kv, a->n_k, a->B, kTile))
    return FM_ERR_CUDA;
  if (!smem_opt_in<key_weight_kernel<D>>(S::kAlloc)) return FM_ERR_CUDA;
  // A key tile's query tiles are shared by a cluster of CTAs where there are too few key tiles for the SMs.
  const int64_t tiles = (int64_t)p.T_k * H_kv * a->B;
  int cluster = 1;
  while (cluster < 8 && tiles * cluster * 2 <= 148) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.T_k * cluster), H_kv, a->B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, key_weight_kernel<D>, tq, tk, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

}  // namespace
}  // namespace fm

extern "C" fm_status fm_attn_key_weight(const fm_attn_args* a, const fm_mask_meta* meta, const int32_t* const vec[4],
                                        const float* lse, float* weight, int64_t weight_stride, int32_t accumulate,
                                        fm_stream_t stream) {
  if (!a) return FM_ERR_INVALID_ARG;
  fm_attn_args args = *a;
  if (!args.v) args.v = args.k;  // not read
  const fm_status st = fm::check_attn_args(&args, meta, vec);
  if (st != FM_OK) return st;
  if (args.dtype != 0) return FM_ERR_UNSUPPORTED;
  if (!lse || !weight || ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(weight)) & 3))
    return FM_ERR_INVALID_ARG;
  if (weight_stride < args.n_k || (accumulate != 0 && accumulate != 1)) return FM_ERR_INVALID_ARG;
  const int H_kv = args.H_kv ? args.H_kv : args.H;
  fm::KeyWeightParams p;
  p.col_count = meta->col_count;
  p.col_entries = meta->col_entries;
  p.order = meta->bwd_order;
  for (int c = 0; c < 4; ++c) p.vec[c] = vec ? vec[c] : nullptr;
  p.lse = lse;
  p.weight = weight;
  p.weight_stride = weight_stride;
  p.status = fm::device_status_ptr();
  p.H = args.H;
  p.Hm = meta->d.Hm;
  p.H_kv = H_kv;
  p.q_per_kv = args.H / H_kv;
  p.n_q = args.n_q;
  p.n_k = args.n_k;
  p.T_q = (args.n_q + fm::kTile - 1) / fm::kTile;
  p.T_k = (args.n_k + fm::kTile - 1) / fm::kTile;
  p.accumulate = accumulate;
  p.scale_log2 = args.scale * 1.4426950408889634f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (args.D == 64) return fm::launch_key_weight<64>(&args, p, H_kv, s);
  if (args.D == 128) return fm::launch_key_weight<128>(&args, p, H_kv, s);
  return fm::launch_key_weight<256>(&args, p, H_kv, s);
}

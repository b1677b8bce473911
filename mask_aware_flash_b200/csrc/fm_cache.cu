// The paged 8-bit K/V cache: writing new tokens (fm_cache_append) and evicting the keys that
// received the least attention (fm_cache_evict).
#include "fm_cache.cuh"

namespace fm {

fm_status check_cache(const fm_kv_cache* c) {
  if (!c) return FM_ERR_INVALID_ARG;
  if (c->B < 1 || c->H_kv < 1 || c->n_pages < 1 || c->max_pages < 1) return FM_ERR_INVALID_ARG;
  if (c->code_type != 0 && c->code_type != 1) return FM_ERR_UNSUPPORTED;
  if (c->D != 64 && c->D != 128 && c->D != 256) return FM_ERR_UNSUPPORTED;
  if (c->B > kMaxCacheB || c->H_kv > 65535) return FM_ERR_UNSUPPORTED;
  // rows of the pools, and slots of the tables, in 32 bits; the slots with room for the strides that loops add to them
  if ((int64_t)c->n_pages * c->H_kv >= ((int64_t)1 << 31) / kPage) return FM_ERR_UNSUPPORTED;
  constexpr int64_t kSlotPages = ((int64_t)1 << 30) / kPage;
  if ((int64_t)c->B * c->H_kv >= kSlotPages || (int64_t)c->B * c->H_kv * c->max_pages >= kSlotPages)
    return FM_ERR_UNSUPPORTED;
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !c->page_table) return FM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(c->k_codes) | reinterpret_cast<uintptr_t>(c->v_codes)) & 15) return FM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale) |
       reinterpret_cast<uintptr_t>(c->page_table) | reinterpret_cast<uintptr_t>(c->weight) |
       reinterpret_cast<uintptr_t>(c->pos)) & 3)
    return FM_ERR_INVALID_ARG;
  return FM_OK;
}

namespace {

// a[which] without a dynamic index into the kernel's parameters (which would copy them to local memory)
template <typename T>
__device__ __forceinline__ T pick(T const (&a)[2], int which) {
  return which ? a[1] : a[0];
}

// Block-wide maximum of the bit patterns of non-negative floats (their order, with infinity and then NaN on top);
// every thread gets it.  `red`: one word per warp; it may be used again after the next __syncthreads.
template <int kThreads>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v = max(v, red[w]);
  return v;
}
constexpr uint32_t kInfBits = 0x7F800000u;

// ------------------------------------------------------------------------------------------ append
struct AppendParams {
  const void* src[2];  // k, v [B, n_new, H_kv, D]
  uint8_t* codes[2];
  float* scale[2];
  const int32_t* page_table;
  const int32_t* start;
  const int32_t* count;
  const int32_t* row;
  float* weight;
  int32_t* pos;
  int n_new, H_kv, n_pages, max_pages;
};

// 16 consecutive elements as they lie in memory, and as fp32
template <typename T>
struct Raw16;
template <>
struct Raw16<__nv_bfloat16> {
  uint4 v[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v[0] = *(reinterpret_cast<const uint4*>(p));
    v[1] = *(reinterpret_cast<const uint4*>(p) + 1);
  }
  // bit pattern (as fp32) of the largest |x|: both halves of a word at once
  __device__ __forceinline__ uint32_t max_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m = __vmaxu2(m, v[i].x & 0x7FFF7FFFu);
      m = __vmaxu2(m, v[i].y & 0x7FFF7FFFu);
      m = __vmaxu2(m, v[i].z & 0x7FFF7FFFu);
      m = __vmaxu2(m, v[i].w & 0x7FFF7FFFu);
    }
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * i + 2 * j] = bf16_lo(w[j]);
        x[8 * i + 2 * j + 1] = bf16_hi(w[j]);
      }
    }
  }
};
template <>
struct Raw16<float> {
  float4 v[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *(reinterpret_cast<const float4*>(p) + i);
  }
  __device__ __forceinline__ uint32_t max_bits() const {
    float x[16];
    get(x);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = v[i].x;
      x[4 * i + 1] = v[i].y;
      x[4 * i + 2] = v[i].z;
      x[4 * i + 3] = v[i].w;
    }
  }
};

template <bool E4M3, bool kSafe>
__device__ __forceinline__ uint4 encode16(const float (&x)[16], float f) {
  uint4 r;
  r.x = encode4<E4M3, kSafe>(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
  r.y = encode4<E4M3, kSafe>(x[4] * f, x[5] * f, x[6] * f, x[7] * f);
  r.z = encode4<E4M3, kSafe>(x[8] * f, x[9] * f, x[10] * f, x[11] * f);
  r.w = encode4<E4M3, kSafe>(x[12] * f, x[13] * f, x[14] * f, x[15] * f);
  return r;
}
template <bool E4M3>
__device__ __forceinline__ void decode16(const uint4& v, float (&x)[16]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y[4];
    decode4f<E4M3>(w[i], y);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[4 * i + j] = y[j];
  }
}

// code = round(x / s), s = 2^e the scale of the (block, head): a maximum over 64 x D values, then one multiplication and one
// rounding each.  One CTA per (cache block that gets tokens, K or V, head, sequence): a thread holds two 16-element
// pieces of the block's values in registers from the one load to the one store, so each new token is read once and its code
// written once, and the maximum costs one barrier.  Bound by memory: 3 bytes a bf16 value.  32768 tokens x 16 heads, D = 128: 64 us
// for 407 MB, 6.4 TB/s (0.97 of the measured copy rate); 8 prompts of up to 4096 x 8 heads: 24 us for 131 MB; one token for
// each of 64 sequences: 4.1 us, a launch and two dependent loads.
template <int D, typename T, bool E4M3>
__global__ void __launch_bounds__(2 * D) append_kernel(const AppendParams p) {
  constexpr int kThreads = 2 * D, kPieces = D / 16;
  __shared__ uint32_t red[2][kThreads / 32];
  grid_wait();
  grid_launch_next();
  const int which = blockIdx.x & 1, hk = blockIdx.y, b = blockIdx.z;
  const int start = *(p.start + b);
  const int count = p.count ? min(max(*(p.count + b), 0), p.n_new) : p.n_new;
  const int block = (start >> 6) + (int)(blockIdx.x >> 1);
  if (block < 0 || block >= p.max_pages) return;
  const int64_t t0 = (int64_t)block * kPage - start;  // token of the block's first slot (negative: older slots)
  if (t0 >= count || t0 + kPage <= 0) return;
  const int page = *(p.page_table + (int64_t)b * p.max_pages + block);
  Raw16<T> x[2];
  bool fresh[2];
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int piece = threadIdx.x + i * kThreads;
    const int64_t t = t0 + piece / kPieces;
    fresh[i] = t >= 0 && t < count;
    if (fresh[i])
      x[i].load(static_cast<const T*>(pick(p.src, which)) + (((int64_t)b * p.n_new + t) * p.H_kv + hk) * D +
                piece % kPieces * 16);
  }
  if (page < 0 || page >= p.n_pages) return;
  const int64_t at = (int64_t)page * p.H_kv + hk;
  const float s_old = t0 < 0 ? pick(p.scale, which)[at] : 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (fresh[i]) bits = max(bits, x[i].max_bits());
  bits = block_max<kThreads>(bits, red[0]);
  const bool safe = bits >= kInfBits;  // an infinity or a NaN is among the values: they do not count
  if (safe) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (fresh[i]) {
        float y[16];
        x[i].get(y);
#pragma unroll
        for (int j = 0; j < 16; ++j) amax = fmaxf(amax, finite_abs(y[j]));
      }
    bits = block_max<kThreads>(__float_as_uint(amax), red[1]);
  }
  const float s = fmaxf(s_old, scale_rule<E4M3>(__uint_as_float(bits)));
  const float inv = s > 0.f ? 1.f / s : 0.f;
  const bool grow = t0 < 0 && s != s_old;  // older codes move to the larger scale
  uint4* codes = reinterpret_cast<uint4*>(pick(p.codes, which) + at * (kPage * D));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int piece = threadIdx.x + i * kThreads;
    float y[16];
    if (fresh[i]) {
      x[i].get(y);
      codes[piece] = safe ? encode16<E4M3, true>(y, inv) : encode16<E4M3, false>(y, inv);
    } else if (grow && t0 + piece / kPieces < 0) {
      decode16<E4M3>(codes[piece], y);
      codes[piece] = encode16<E4M3, true>(y, s_old * inv);
    }
  }
  if (threadIdx.x == 0) pick(p.scale, which)[at] = s;
  if (which == 0 && threadIdx.x < kPage) {
    const int64_t t = t0 + threadIdx.x;
    if (t >= 0 && t < count) {
      const int64_t slot = ((int64_t)b * p.H_kv + hk) * p.max_pages * kPage + (int64_t)block * kPage + threadIdx.x;
      if (p.weight) p.weight[slot] = 0.f;
      if (p.pos) p.pos[slot] = (p.row ? *(p.row + b) : start) + (int)t;
    }
  }
}

template <int D>
cudaError_t launch_append(const AppendParams& p, int B, int dtype, int code_type, cudaStream_t s) {
  EarlyLaunch launch(s);
  // a run of n tokens touches at most ceil((63 + n) / 64) blocks
  launch.cfg.gridDim = dim3(2 * (unsigned)(((int64_t)p.n_new + kPage - 1 + kPage - 1) / kPage), p.H_kv, B);
  launch.cfg.blockDim = dim3(2 * D);
  if (dtype == 0)
    return code_type ? cudaLaunchKernelEx(&launch.cfg, append_kernel<D, __nv_bfloat16, true>, p)
                     : cudaLaunchKernelEx(&launch.cfg, append_kernel<D, __nv_bfloat16, false>, p);
  return code_type ? cudaLaunchKernelEx(&launch.cfg, append_kernel<D, float, true>, p)
                   : cudaLaunchKernelEx(&launch.cfg, append_kernel<D, float, false>, p);
}

// ------------------------------------------------------------------------------------------- evict
struct EvictParams {
  const int32_t* src_table;
  const int32_t* dst_table;
  const uint8_t* src_codes[2];
  const float* src_scale[2];
  uint8_t* dst_codes[2];
  float* dst_scale[2];
  const float* src_weight;
  const int32_t* src_pos;
  float* dst_weight;
  int32_t* dst_pos;
  const int32_t* len;
  int32_t* new_len;
  int32_t* kept;    // ws: [B, H_kv, budget] the kept slots' rows (page * 64 + slot % 64; -1: no page), ascending slots
  int32_t* n_kept;  // ws: [B, H_kv]
  int H_kv, src_pages, dst_pages, src_max, dst_max, budget, recent;
  int chunk;  // slots of a CTA of the selection (a multiple of 32)
};

// Unsigned key that orders weights as the selection does: larger weight, larger key; -0 equals +0;
// NaN above everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

constexpr int kDigitBits = 11;      // a pass
constexpr int kBins = 1 << kDigitBits;
constexpr int kSelMaxKeys = 49152;  // keys a CTA can hold in shared memory
constexpr int kMaxCluster = 8;      // CTAs of a cluster (a power of two of them)

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
__device__ __forceinline__ uint32_t ld_cluster(const uint32_t* p, uint32_t rank) {  // another CTA's shared memory
  uint32_t v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.u32 %0, [a];\n\t}"
      : "=r"(v)
      : "r"(smem_u32(p)), "r"(rank)
      : "memory");
  return v;
}

__device__ __forceinline__ uint4 ld_cluster4(const uint32_t* p, uint32_t rank) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "r"(smem_u32(p)), "r"(rank)
      : "memory");
  return v;
}

struct SelSmem {
  uint32_t hist[2][kBins];  // of this CTA's slots: passes alternate, so that the others may still read the last one's
  uint32_t digit, left;     // the pass's result: its digit, how many of the keys with it are taken,
  uint32_t all;             // whether those are all
  uint32_t lowest, highest;
  uint32_t above, equal;    // of this CTA's slots
  uint32_t first, last;     // its part of the kept list
  uint32_t warp_a[32], warp_b[32];
};
// Sum of v[0 .. n) for n <= 32, by every lane of a warp.
__device__ __forceinline__ uint32_t sum_before(const uint32_t* v, int n, int lane) {
  return __reduce_add_sync(0xffffffffu, lane < n ? v[lane] : 0u);
}

// The budget - recent largest weights of the older slots of one (head, sequence) by a radix selection, up to 11 bits
// of the keys a pass, then one ordered pass that writes the kept slots ascending.  A cluster of CTAs shares the slots
// (contiguous runs); histograms and counts are exchanged through distributed shared memory.  kHeld: the keys stay in
// shared memory after the one read of the weights (else every pass reads them again; 49152 keys are what a CTA can hold).
// Bound by latency: 4 bytes a slot are read once, but each pass is a histogram (shared-memory atomics), a cluster barrier, the
// other CTAs' counts and a scan, one after the other.  Digits relative to the lowest key with an early end make that two
// passes for 131072 random weights and one for 4200 (fixed digits: three), 11 bits a pass where 8 would take a pass more.
// 8 heads of 131072 slots: some 19 us of the call's 31; 256 lists of 4200: some 14 of 63.
template <bool kHeld, int kSelThreads>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictParams p) {
  constexpr int kSelWarps = kSelThreads / 32;
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) SelSmem sm;
  grid_wait();
  grid_launch_next();
  const int rank = (int)cluster_rank(), size = (int)cluster_size();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int64_t bh = (int64_t)b * p.H_kv + hk;
  const int n = min(max(*(p.len + b), 0), p.src_max * kPage);
  if (threadIdx.x == 0 && rank == 0) p.n_kept[bh] = min(n, p.budget);
  int32_t* kept = p.kept + bh * p.budget;
  const float* w = p.src_weight + bh * p.src_max * kPage;
  const int32_t* pos = p.src_pos ? p.src_pos + bh * p.src_max * kPage : nullptr;
  float* to_w = p.dst_weight ? p.dst_weight + bh * p.dst_max * kPage : nullptr;
  int32_t* to_pos = p.dst_pos ? p.dst_pos + bh * p.dst_max * kPage : nullptr;
  const int32_t* table = p.src_table + (int64_t)b * p.src_max;
  // What the new cache takes of the slots from(first), from(first + step), ... for its slots first, first + step, ... < end:
  // four at a time, so that their loads overlap.
  auto keep = [&](int first, int end, int step, auto from) {
    for (int to = first; to < end; to += 4 * step) {
      int f[4], page[4], q[4];
      float x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) f[u] = to + u * step < end ? from(to + u * step) : -1;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        page[u] = f[u] >= 0 ? *(table + f[u] / kPage) : -1;
        x[u] = to_w && f[u] >= 0 ? *(w + f[u]) : 0.f;
        q[u] = to_pos && pos && f[u] >= 0 ? *(pos + f[u]) : f[u];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (f[u] >= 0) {
          kept[to + u * step] = page[u] >= 0 && page[u] < p.src_pages ? page[u] * kPage + f[u] % kPage : -1;
          if (to_w) to_w[to + u * step] = x[u];
          if (to_pos) to_pos[to + u * step] = q[u];
        }
    }
  };
  if (n <= p.budget) {  // (the same for every CTA of the cluster)
    keep(rank * kSelThreads + threadIdx.x, n, size * kSelThreads, [](int i) { return i; });
    return;
  }
  const int older = n - p.recent, want = p.budget - p.recent;  // older > want >= 0
  keep(want + rank * kSelThreads + threadIdx.x, p.budget, size * kSelThreads, [&](int i) { return older + i - want; });
  if (want == 0) return;
  // this CTA's run of slots; a length below the table's leaves CTAs fewer slots, not other ones without any
  const int run = min(p.chunk, (((older + size - 1) / size) + 31) / 32 * 32);
  const int i0 = min(rank * run, older), mine = min(i0 + run, older) - i0;
  auto key = [&](int i) { return kHeld ? keys[i] : weight_key(*(w + i0 + i)); };
  // The range of the keys: digits are taken of key - lowest, from the highest bit that occurs, so that a pass tells as many
  // keys apart as its bins can (of weights within a few octaves, the top bits of the key itself would fill a few bins).
  uint32_t lowest = 0xFFFFFFFFu, highest = 0;
  for (int i = threadIdx.x; i < mine; i += 8 * kSelThreads) {
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = i + u * kSelThreads < mine ? *(w + i0 + i + u * kSelThreads) : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i + u * kSelThreads < mine) {
        const uint32_t k = weight_key(x[u]);
        if (kHeld) keys[i + u * kSelThreads] = k;
        lowest = min(lowest, k);
        highest = max(highest, k);
      }
  }
  lowest = __reduce_min_sync(0xffffffffu, lowest);
  highest = __reduce_max_sync(0xffffffffu, highest);
  if (lane == 0) {
    sm.warp_a[warp] = lowest;
    sm.warp_b[warp] = highest;
  }
  __syncthreads();
  lowest = __reduce_min_sync(0xffffffffu, sm.warp_a[lane % kSelWarps]);
  highest = __reduce_max_sync(0xffffffffu, sm.warp_b[lane % kSelWarps]);
  if (size > 1) {
    if (threadIdx.x == 0) {
      sm.lowest = lowest;
      sm.highest = highest;
    }
    cluster_sync_all();
    lowest = __reduce_min_sync(0xffffffffu, ld_cluster(&sm.lowest, lane % size));
    highest = __reduce_max_sync(0xffffffffu, ld_cluster(&sm.highest, lane % size));
  } else {
    __syncthreads();
  }
  // prefix: the digits found so far of the last key that is taken; `need`: how many are taken of the keys that share them
  uint32_t prefix = 0, need = want;
  int shift = 32 - __clz((int)(highest - lowest)), above_shift = 32;
  uint32_t* hist = sm.hist[0];
  for (bool more = shift > 0; more; hist = hist == sm.hist[0] ? sm.hist[1] : sm.hist[0]) {
    above_shift = shift;
    shift = max(shift - kDigitBits, 0);
    for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i - lane < mine; i += 4 * kSelThreads) {
      uint32_t k[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) k[u] = i + u * kSelThreads < mine ? key(i + u * kSelThreads) - lowest : 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool in = i + u * kSelThreads < mine &&
                        (above_shift == 32 ? 0u : k[u] >> above_shift) == (above_shift == 32 ? 0u : prefix >> above_shift);
        const uint32_t d = (k[u] >> shift) & ((1u << (above_shift - shift)) - 1u), who = __ballot_sync(0xffffffffu, in);
        if (who == 0) continue;
        const int leader = __ffs(who) - 1;
        const uint32_t d_leader = __shfl_sync(0xffffffffu, d, leader);  // (by every lane: not behind the && below)
        const uint32_t same = __ballot_sync(0xffffffffu, in && d == d_leader);
        if (same == who) {  // all the same (zeros, say): one addition for the warp
          if (lane == leader) atomicAdd(&hist[d], (uint32_t)__popc(who));
        } else if (in) {
          atomicAdd(&hist[d], 1u);
        }
      }
    }
    if (size > 1) cluster_sync_all();
    else __syncthreads();
    // The digit at which the count from the top reaches `need`: every CTA adds up the whole histogram, thread i the i-th
    // four bins from the top.
    {
      constexpr int kQuads = kBins / 4;
      const int quad = kQuads - 1 - (int)threadIdx.x;
      uint32_t t[4] = {0, 0, 0, 0};
      if (quad >= 0) {
        // the CTAs' counts all in flight at once, each CTA beginning at another one
        uint4 v[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
          v[c] = c < size ? ld_cluster4(hist + 4 * quad, (rank + c) & (size - 1)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          t[0] += v[c].w;
          t[1] += v[c].z;
          t[2] += v[c].y;
          t[3] += v[c].x;
        }
      }
      const uint32_t own = t[0] + t[1] + t[2] + t[3];
      uint32_t x = own;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, s);
        if (lane >= s) x += y;
      }
      if (lane == 31) sm.warp_a[warp] = x;
      __syncthreads();
      uint32_t before = x - own + sum_before(sm.warp_a, warp, lane);
      if (before < need && before + own >= need) {  // one thread
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (before < need && before + t[j] >= need) {
            sm.digit = (uint32_t)(4 * quad + 3 - j);
            sm.left = need - before;
            sm.all = t[j] == need - before;
          }
          before += t[j];
        }
      }
      __syncthreads();
    }
    prefix |= sm.digit << shift;
    need = sm.left;
    more = shift > 0 && !sm.all;  // all the keys with these digits are taken: the rest does not matter
  }
  auto rank_of = [&](int i) { return (key(i) - lowest) >> shift; };
  prefix >>= shift;
  // Keys above the prefix are taken, and `need` of those that share it, lowest slots first.
  // Counts of each warp's run of slots, of the CTA, and of the CTAs before it
  const int per_warp = ((run + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int a0 = min(warp * per_warp, mine), a1 = min(a0 + per_warp, mine);
  uint32_t above = 0, equal = 0;
#pragma unroll 4
  for (int i = a0 + lane; i < a1; i += 32) {
    const uint32_t k = rank_of(i);
    above += k > prefix;
    equal += k == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    sm.warp_a[warp] = above;
    sm.warp_b[warp] = equal;
  }
  __syncthreads();
  if (size > 1 && warp == kSelWarps - 1) {
    const uint32_t a = sum_before(sm.warp_a, kSelWarps, lane), e = sum_before(sm.warp_b, kSelWarps, lane);
    if (lane == 0) {
      sm.above = a;
      sm.equal = e;
    }
  }
  above = sum_before(sm.warp_a, warp, lane);
  equal = sum_before(sm.warp_b, warp, lane);
  if (size > 1) {
    cluster_sync_all();
    above += __reduce_add_sync(0xffffffffu, lane < rank ? ld_cluster(&sm.above, lane) : 0u);
    equal += __reduce_add_sync(0xffffffffu, lane < rank ? ld_cluster(&sm.equal, lane) : 0u);
  }
  // the kept slots in order, then (in parallel again) what the new cache takes of each
  if (threadIdx.x == 0) sm.first = above + min(equal, need);
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
  for (int i = a0; i < a1; i += 32) {
    const uint32_t k = i + lane < a1 ? rank_of(i + lane) : 0;
    const bool in = i + lane < a1;
    const uint32_t ba = __ballot_sync(0xffffffffu, in && k > prefix), be = __ballot_sync(0xffffffffu, in && k == prefix);
    const uint32_t before_a = above + __popc(ba & below), before_e = equal + __popc(be & below);
    if (in && (k > prefix || (k == prefix && before_e < need))) kept[before_a + min(before_e, need)] = i0 + i + lane;
    above += __popc(ba);
    equal += __popc(be);
  }
  if (threadIdx.x == kSelThreads - 1) sm.last = above + min(equal, need);
  __syncthreads();
  keep((int)sm.first + threadIdx.x, (int)sm.last, kSelThreads, [&](int i) { return kept[i]; });
  if (size > 1) cluster_sync_all();  // no CTA leaves while its counts are read
}

// Byte permutation whose selectors with the top bit set give the sign of a byte, eight times.
template <uint32_t kSel>
__device__ __forceinline__ uint32_t bytes_signed(uint32_t w) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "n"(kSel));
  return r;
}

// The largest magnitude of four times four codes, as a number in code units.  int8: the bytes go to 16-bit pairs with their
// signs, a running maximum and minimum of each; e4m3: magnitudes are ordered as their 7-bit patterns.
template <bool E4M3>
__device__ __forceinline__ float max_code(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (E4M3) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, __vmaxu2(w[i] & 0x007F007Fu, (w[i] >> 8) & 0x007F007Fu));
    float y[4];
    decode4f<E4M3>(max(m & 0xFFu, m >> 16), y);
    return y[0];
  } else {
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = bytes_signed<0x9180>(w[i]), b = bytes_signed<0xB3A2>(w[i]);
      hi = __vmaxs2(hi, __vmaxs2(a, b));
      lo = __vmins2(lo, __vmins2(a, b));
    }
    const int top = max((int)(int16_t)(hi & 0xFFFFu), (int)(int16_t)(hi >> 16));
    const int low = min((int)(int16_t)(lo & 0xFFFFu), (int)(int16_t)(lo >> 16));
    return (float)max(top, -low);
  }
}

// The kept slots' values code * s_old, re-quantised by the scale rule over the 64 that now share a block: since scales are powers
// of two, value / s_new = code * (s_old / s_new) exactly, and a code is rounded once.  One CTA per (dst block, head, sequence)
// gathers the K and V codes together (they share the list and its latency: 20 -> 10 us against a CTA each for 8 heads x 8192
// slots), keeps them in registers and writes the block once.  Bound by memory: the kept rows are D bytes each, two dependent
// loads away (list, then scale and codes); 32 x 8 heads x 2048 slots, D = 128: 268 MB read and written in some 46 us, 5.8 TB/s.
template <int D, bool E4M3>
__global__ void __launch_bounds__(2 * D, 1024 / (2 * D)) compact_kernel(const EvictParams p) {
  constexpr int kThreads = 2 * D, kPieces = D / 16;
  __shared__ uint32_t red[2][kThreads / 32];
  grid_wait();
  grid_launch_next();
  const int block = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
  const int64_t bh = (int64_t)b * p.H_kv + hk;
  const int n = __ldcg(p.n_kept + bh);
  const int page = *(p.dst_table + (int64_t)b * p.dst_max + block);
  int row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // (entries behind the n-th are there, without a meaning)
    const int to = block * kPage + (threadIdx.x + i * kThreads) / kPieces;
    row[i] = to < p.budget ? __ldcg(p.kept + bh * p.budget + to) : -1;
  }
  if (block == 0 && hk == 0 && threadIdx.x == 0) p.new_len[b] = n;
  if (block * kPage >= n || page < 0 || page >= p.dst_pages) return;
  uint4 raw[2][2];
  float scale[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int piece = threadIdx.x + i * kThreads;
    if (block * kPage + piece / kPieces >= n) row[i] = -1;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      raw[x][i] = make_uint4(0, 0, 0, 0);  // (code 0 of both formats)
      scale[x][i] = 0.f;
      if (row[i] >= 0) {
        const int64_t at = (int64_t)(row[i] / kPage) * p.H_kv + hk;
        scale[x][i] = *(p.src_scale[x] + at);
        raw[x][i] = *(reinterpret_cast<const uint4*>(p.src_codes[x] + (at * kPage + row[i] % kPage) * D) + piece % kPieces);
      }
    }
  }
  uint32_t bits[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    bits[x] = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      bits[x] = max(bits[x], __float_as_uint(fabsf(max_code<E4M3>(raw[x][i]) * scale[x][i])));
    bits[x] = __reduce_max_sync(0xffffffffu, bits[x]);
    if ((threadIdx.x & 31) == 0) red[x][threadIdx.x >> 5] = bits[x];
  }
  __syncthreads();
  const int64_t at = (int64_t)page * p.H_kv + hk;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) bits[x] = max(bits[x], red[x][w]);
    // (a product that overflows, from scales no append writes: the largest finite scale, its codes saturate)
    const bool safe = bits[x] >= kInfBits;
    const float s = scale_rule<E4M3>(__uint_as_float(min(bits[x], kInfBits - 1)));
    const float inv = s > 0.f ? 1.f / s : 0.f;
    uint4* codes = reinterpret_cast<uint4*>(p.dst_codes[x] + at * (kPage * D));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float y[16];
      decode16<E4M3>(raw[x][i], y);
      const float f = scale[x][i] * inv;
      codes[threadIdx.x + i * kThreads] = safe ? encode16<E4M3, true>(y, f) : encode16<E4M3, false>(y, f);
    }
    if (threadIdx.x == 0) p.dst_scale[x][at] = s;
  }
}

template <bool kHeld, int kThreads>
cudaError_t launch_select(const EvictParams& p, int B, int cluster, cudaStream_t s) {
  EarlyLaunch launch(s, cluster);
  cudaLaunchConfig_t& cfg = launch.cfg;
  cfg.gridDim = dim3(cluster, p.H_kv, B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kHeld ? p.chunk * 4 : 0;
  if (kHeld && !smem_opt_in<select_kernel<kHeld, kThreads>>(kSelMaxKeys * 4)) return cudaErrorInvalidValue;
  return cudaLaunchKernelEx(&cfg, select_kernel<kHeld, kThreads>, p);
}

// Do two caches' tables of a word per slot (weight, pos) share any word?
bool slot_words_overlap(const fm_kv_cache* a, const void* x, const fm_kv_cache* b, const void* y) {
  if (!x || !y) return false;
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), y0 = reinterpret_cast<uintptr_t>(y);
  auto bytes = [](const fm_kv_cache* c) { return (uintptr_t)c->B * c->H_kv * c->max_pages * kPage * 4; };
  return x0 < y0 + bytes(b) && y0 < x0 + bytes(a);
}

size_t evict_n_kept_offset(const fm_kv_cache* src, int32_t budget) {
  return ((size_t)src->B * src->H_kv * budget * 4 + 255) / 256 * 256;
}

}  // namespace
}  // namespace fm

extern "C" {

fm_status fm_cache_append(const fm_kv_cache* c, const void* k, const void* v, int32_t dtype, int32_t n_new,
                          const int32_t* start, const int32_t* count, const int32_t* row, fm_stream_t stream) {
  fm_status st = fm::check_cache(c);
  if (st != FM_OK) return st;
  if (dtype != 0 && dtype != 1) return FM_ERR_UNSUPPORTED;
  if (n_new < 1 || !k || !v || !start) return FM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) return FM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(start) | reinterpret_cast<uintptr_t>(count) | reinterpret_cast<uintptr_t>(row)) & 3)
    return FM_ERR_INVALID_ARG;
  fm::AppendParams p;
  p.src[0] = k;
  p.src[1] = v;
  p.codes[0] = static_cast<uint8_t*>(c->k_codes);
  p.codes[1] = static_cast<uint8_t*>(c->v_codes);
  p.scale[0] = c->k_scale;
  p.scale[1] = c->v_scale;
  p.page_table = c->page_table;
  p.start = start;
  p.count = count;
  p.row = row;
  p.weight = c->weight;
  p.pos = c->pos;
  p.n_new = n_new;
  p.H_kv = c->H_kv;
  p.n_pages = c->n_pages;
  p.max_pages = c->max_pages;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c->D == 64    ? fm::launch_append<64>(p, c->B, dtype, c->code_type, s)
                        : c->D == 128 ? fm::launch_append<128>(p, c->B, dtype, c->code_type, s)
                                      : fm::launch_append<256>(p, c->B, dtype, c->code_type, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

size_t fm_cache_evict_workspace_bytes(const fm_kv_cache* src, int32_t budget) {
  if (fm::check_cache(src) != FM_OK || budget < 1) return 0;
  return fm::evict_n_kept_offset(src, budget) + ((size_t)src->B * src->H_kv * 4 + 255) / 256 * 256;
}

fm_status fm_cache_evict(const fm_kv_cache* src, const fm_kv_cache* dst, const int32_t* len, int32_t budget,
                         int32_t recent, int32_t* new_len, void* ws, size_t ws_bytes, fm_stream_t stream) {
  fm_status st = fm::check_cache(src);
  if (st == FM_OK) st = fm::check_cache(dst);
  if (st != FM_OK) return st;
  if (src->B != dst->B || src->H_kv != dst->H_kv || src->D != dst->D || src->code_type != dst->code_type)
    return FM_ERR_INVALID_ARG;
  if (src->page_table == dst->page_table && src->k_codes == dst->k_codes) return FM_ERR_INVALID_ARG;
  if (!src->weight || !len || !new_len) return FM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(len) | reinterpret_cast<uintptr_t>(new_len)) & 3) return FM_ERR_INVALID_ARG;
  if (fm::slot_words_overlap(src, src->weight, dst, dst->weight) || fm::slot_words_overlap(src, src->weight, dst, dst->pos) ||
      fm::slot_words_overlap(src, src->pos, dst, dst->weight) || fm::slot_words_overlap(src, src->pos, dst, dst->pos))
    return FM_ERR_INVALID_ARG;
  if (budget < 1 || budget > (int64_t)dst->max_pages * fm::kPage || recent < 0 || recent > budget)
    return FM_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || ws_bytes < fm_cache_evict_workspace_bytes(src, budget))
    return FM_ERR_WORKSPACE;
  fm::EvictParams p;
  p.src_table = src->page_table;
  p.dst_table = dst->page_table;
  p.src_codes[0] = static_cast<const uint8_t*>(src->k_codes);
  p.src_codes[1] = static_cast<const uint8_t*>(src->v_codes);
  p.src_scale[0] = src->k_scale;
  p.src_scale[1] = src->v_scale;
  p.dst_codes[0] = static_cast<uint8_t*>(dst->k_codes);
  p.dst_codes[1] = static_cast<uint8_t*>(dst->v_codes);
  p.dst_scale[0] = dst->k_scale;
  p.dst_scale[1] = dst->v_scale;
  p.src_weight = src->weight;
  p.src_pos = src->pos;
  p.dst_weight = dst->weight;
  p.dst_pos = dst->pos;
  p.len = len;
  p.new_len = new_len;
  p.kept = static_cast<int32_t*>(ws);
  p.n_kept = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + fm::evict_n_kept_offset(src, budget));
  p.H_kv = src->H_kv;
  p.src_pages = src->n_pages;
  p.dst_pages = dst->n_pages;
  p.src_max = src->max_pages;
  p.dst_max = dst->max_pages;
  p.budget = budget;
  p.recent = recent;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // The CTAs of a selection: one per 2048 to 4096 slots of the table, as far as a cluster goes and all clusters run at once.  (8
  // heads: 131072 slots 31 us with clusters of 8, 184 with a CTA each; 2 x 8 heads of 40000: 24 us with clusters of 4, of
  // which 16 run at once, 39 with 8, of which they do not; 2 heads of 4000: 10.8 us with a CTA each, 12.2 with clusters of 2.)
  const int64_t slots = (int64_t)src->max_pages * fm::kPage, lists = (int64_t)src->B * src->H_kv;
  constexpr int kHeldBytes = fm::kSelMaxKeys * 4;
  if (!fm::smem_opt_in<fm::select_kernel<true, 1024>>(kHeldBytes)) return FM_ERR_CUDA;
  int cluster = fm::kMaxCluster;
  while (cluster > 1 && (slots <= 2048 * (int64_t)cluster ||
                         lists > fm::clusters_at_once<fm::select_kernel<true, 1024>>(cluster, 1024, kHeldBytes)))
    cluster /= 2;
  p.chunk = (int)(((slots + cluster - 1) / cluster + 31) / 32 * 32);
  const bool held = p.chunk <= fm::kSelMaxKeys;
  // 1024 threads a CTA where there is one CTA per SM at most (2 x 8 heads of 40000 slots: 24 us, with 512 threads 28), 512
  // where two share one (32 x 8 heads of 4200: 62.0 us, with 1024 threads 63.2)
  const bool wide = lists * cluster <= 148;
  cudaError_t e = held ? (wide ? fm::launch_select<true, 1024>(p, src->B, cluster, s) : fm::launch_select<true, 512>(p, src->B, cluster, s))
                       : fm::launch_select<false, 1024>(p, src->B, cluster, s);
  if (e != cudaSuccess) return FM_ERR_CUDA;
  fm::EarlyLaunch launch(s);
  cudaLaunchConfig_t& cfg = launch.cfg;
  cfg.gridDim = dim3((unsigned)((budget + fm::kPage - 1) / fm::kPage), src->H_kv, src->B);
  cfg.blockDim = dim3(2 * src->D);
  if (src->D == 64)
    e = src->code_type ? cudaLaunchKernelEx(&cfg, fm::compact_kernel<64, true>, p) : cudaLaunchKernelEx(&cfg, fm::compact_kernel<64, false>, p);
  else if (src->D == 128)
    e = src->code_type ? cudaLaunchKernelEx(&cfg, fm::compact_kernel<128, true>, p) : cudaLaunchKernelEx(&cfg, fm::compact_kernel<128, false>, p);
  else
    e = src->code_type ? cudaLaunchKernelEx(&cfg, fm::compact_kernel<256, true>, p) : cudaLaunchKernelEx(&cfg, fm::compact_kernel<256, false>, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

}  // extern "C"

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
  constexpr int64_t kLimit = (int64_t)1 << 31;
  if ((int64_t)c->n_pages * c->H_kv >= kLimit / kPage) return FM_ERR_UNSUPPORTED;
  if ((int64_t)c->B * c->H_kv >= kLimit / kPage || (int64_t)c->B * c->H_kv * c->max_pages >= kLimit / kPage)
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

// Block-wide maximum of non-negative values; every thread gets it.  `red`: one float per warp.
template <int kThreads>
__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v = fmaxf(v, red[w]);
  return v;
}

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

// 16 consecutive elements as fp32
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * i + 2 * j] = bf16_lo(w[j]);
      x[8 * i + 2 * j + 1] = bf16_hi(w[j]);
    }
  }
}
__device__ __forceinline__ void load16(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
    x[4 * i] = v.x;
    x[4 * i + 1] = v.y;
    x[4 * i + 2] = v.z;
    x[4 * i + 3] = v.w;
  }
}

template <bool E4M3>
__device__ __forceinline__ uint4 encode16(const float (&x)[16], float inv) {
  uint4 r;
  r.x = encode4<E4M3>(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
  r.y = encode4<E4M3>(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
  r.z = encode4<E4M3>(x[8] * inv, x[9] * inv, x[10] * inv, x[11] * inv);
  r.w = encode4<E4M3>(x[12] * inv, x[13] * inv, x[14] * inv, x[15] * inv);
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

// One CTA per (cache block that gets tokens, K or V, head, sequence): a thread holds two 16-element
// pieces of the block's 64 x D values in registers from the one load to the one store, so each new
// token is read once and its code written once.
template <int D, typename T, bool E4M3>
__global__ void __launch_bounds__(2 * D) append_kernel(const AppendParams p) {
  constexpr int kThreads = 2 * D, kPieces = D / 16;
  __shared__ float red[kThreads / 32];
  const int which = blockIdx.x & 1, hk = blockIdx.y, b = blockIdx.z;
  const int start = __ldg(p.start + b);
  const int count = p.count ? min(max(__ldg(p.count + b), 0), p.n_new) : p.n_new;
  const int block = (start >> 6) + (int)(blockIdx.x >> 1);
  if (block < 0 || block >= p.max_pages) return;
  const int64_t t0 = (int64_t)block * kPage - start;  // token of the block's first slot (negative: older slots)
  if (t0 >= count || t0 + kPage <= 0) return;
  const int page = __ldg(p.page_table + (int64_t)b * p.max_pages + block);
  if (page < 0 || page >= p.n_pages) return;
  const int64_t at = (int64_t)page * p.H_kv + hk;
  const float s_old = t0 < 0 ? pick(p.scale, which)[at] : 0.f;
  float x[2][16];
  bool fresh[2];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int piece = threadIdx.x + i * kThreads;
    const int64_t t = t0 + piece / kPieces;
    fresh[i] = t >= 0 && t < count;
    if (!fresh[i]) continue;
    load16(static_cast<const T*>(pick(p.src, which)) + (((int64_t)b * p.n_new + t) * p.H_kv + hk) * D + piece % kPieces * 16, x[i]);
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = fmaxf(amax, finite_abs(x[i][j]));
  }
  amax = block_max<kThreads>(amax, red);
  const float s = fmaxf(s_old, scale_rule<E4M3>(amax));
  const float inv = s > 0.f ? 1.f / s : 0.f;
  const bool grow = t0 < 0 && s != s_old;  // older codes move to the larger scale
  uint4* codes = reinterpret_cast<uint4*>(pick(p.codes, which) + at * (kPage * D));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int piece = threadIdx.x + i * kThreads;
    if (fresh[i]) {
      codes[piece] = encode16<E4M3>(x[i], inv);
    } else if (grow && t0 + piece / kPieces < 0) {
      decode16<E4M3>(codes[piece], x[i]);
      codes[piece] = encode16<E4M3>(x[i], s_old * inv);
    }
  }
  if (threadIdx.x == 0) pick(p.scale, which)[at] = s;
  if (which == 0 && threadIdx.x < kPage) {
    const int64_t t = t0 + threadIdx.x;
    if (t >= 0 && t < count) {
      const int64_t slot = ((int64_t)b * p.H_kv + hk) * p.max_pages * kPage + (int64_t)block * kPage + threadIdx.x;
      if (p.weight) p.weight[slot] = 0.f;
      if (p.pos) p.pos[slot] = (p.row ? __ldg(p.row + b) : start) + (int)t;
    }
  }
}

template <int D>
void launch_append(const AppendParams& p, int B, int dtype, int code_type, cudaStream_t s) {
  // a run of n tokens touches at most ceil((63 + n) / 64) blocks
  const dim3 grid(2 * (unsigned)(((int64_t)p.n_new + kPage - 1 + kPage - 1) / kPage), p.H_kv, B);
  if (dtype == 0)
    code_type ? append_kernel<D, __nv_bfloat16, true><<<grid, 2 * D, 0, s>>>(p)
              : append_kernel<D, __nv_bfloat16, false><<<grid, 2 * D, 0, s>>>(p);
  else
    code_type ? append_kernel<D, float, true><<<grid, 2 * D, 0, s>>>(p)
              : append_kernel<D, float, false><<<grid, 2 * D, 0, s>>>(p);
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
  int32_t* kept;    // ws: [B, H_kv, budget] source slots, ascending
  int32_t* n_kept;  // ws: [B, H_kv]
  int H_kv, src_pages, dst_pages, src_max, dst_max, budget, recent;
};

// Unsigned key that orders weights as the selection does: larger weight, larger key; -0 equals +0;
// NaN above everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024;

// Exclusive prefix sum over the block of a pair packed into 64 bits; `total` gets the block's sum.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* red, uint64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += y;
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint64_t w = red[lane];
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, w, s);
      if (lane >= s) w += y;
    }
    red[lane] = w;
  }
  __syncthreads();
  total = red[31];
  return x - v + (warp ? red[warp - 1] : 0);
}

// One CTA per (head, sequence): the budget - recent largest weights of the older slots by a radix
// selection (four passes of 8 bits over the keys, a 256-bin histogram in shared memory), then one
// ordered pass that writes the kept slots ascending.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_prefix, s_need;
  __shared__ uint64_t red[32];
  const int hk = blockIdx.x, b = blockIdx.y;
  const int64_t bh = (int64_t)b * p.H_kv + hk;
  const int n = min(max(__ldg(p.len + b), 0), p.src_max * kPage);
  int32_t* kept = p.kept + bh * p.budget;
  if (threadIdx.x == 0) p.n_kept[bh] = min(n, p.budget);
  if (n <= p.budget) {
    for (int i = threadIdx.x; i < n; i += kSelThreads) kept[i] = i;
    return;
  }
  const int older = n - p.recent, want = p.budget - p.recent;  // older > want >= 0
  const float* w = p.src_weight + bh * p.src_max * kPage;
  uint32_t prefix = 0, need = want;
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < older; i += kSelThreads) {
        const uint32_t k = weight_key(__ldg(w + i));
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        uint32_t left = need;
        int d = 255;
        while (hist[d] < left) left -= hist[d--];
        s_prefix = prefix | ((uint32_t)d << shift);
        s_need = left;
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
  }
  // prefix: the key of the last one taken; `need` of the keys equal to it are taken, lowest slots first
  const int per = (older + kSelThreads - 1) / kSelThreads;
  const int i0 = min((int)threadIdx.x * per, older), i1 = min(i0 + per, older);
  uint64_t mine = 0;  // above | equal << 32
  if (want > 0)
    for (int i = i0; i < i1; ++i) {
      const uint32_t k = weight_key(__ldg(w + i));
      mine += k > prefix ? 1ull : (k == prefix ? (1ull << 32) : 0ull);
    }
  uint64_t total;
  uint64_t before = block_scan(mine, red, total);
  if (want > 0)
    for (int i = i0; i < i1; ++i) {
      const uint32_t k = weight_key(__ldg(w + i));
      const uint32_t above = (uint32_t)before, equal = (uint32_t)(before >> 32);
      if (k > prefix || (k == prefix && equal < need)) kept[above + min(equal, need)] = i;
      before += k > prefix ? 1ull : (k == prefix ? (1ull << 32) : 0ull);
    }
  for (int i = threadIdx.x; i < p.recent; i += kSelThreads) kept[want + i] = older + i;
}

// One CTA per (dst block, K or V, head, sequence): gathers the kept slots' codes, re-quantises them
// together (values stay in registers) and writes the block once.
template <int D, bool E4M3>
__global__ void __launch_bounds__(2 * D) compact_kernel(const EvictParams p) {
  constexpr int kThreads = 2 * D, kPieces = D / 16;
  __shared__ float red[kThreads / 32];
  const int which = blockIdx.x & 1, block = blockIdx.x >> 1, hk = blockIdx.y, b = blockIdx.z;
  const int64_t bh = (int64_t)b * p.H_kv + hk;
  const int n = __ldg(p.n_kept + bh);
  if (block == 0 && which == 0 && hk == 0 && threadIdx.x == 0) p.new_len[b] = n;
  if (block * kPage >= n) return;
  const int32_t* kept = p.kept + bh * p.budget;
  if (which == 0 && threadIdx.x < kPage && block * kPage + (int)threadIdx.x < n) {
    const int to = block * kPage + threadIdx.x, from = __ldg(kept + to);
    const int64_t src = bh * p.src_max * kPage + from, dst = bh * p.dst_max * kPage + to;
    if (p.dst_weight) p.dst_weight[dst] = __ldg(p.src_weight + src);
    if (p.dst_pos) p.dst_pos[dst] = p.src_pos ? __ldg(p.src_pos + src) : from;
  }
  const int page = __ldg(p.dst_table + (int64_t)b * p.dst_max + block);
  if (page < 0 || page >= p.dst_pages) return;
  float x[2][16];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int piece = threadIdx.x + i * kThreads, to = block * kPage + piece / kPieces;
#pragma unroll
    for (int j = 0; j < 16; ++j) x[i][j] = 0.f;
    if (to >= n) continue;
    const int from = __ldg(kept + to);
    const int sp = __ldg(p.src_table + (int64_t)b * p.src_max + from / kPage);
    if (sp < 0 || sp >= p.src_pages) continue;
    const int64_t at = (int64_t)sp * p.H_kv + hk;
    const float s = __ldg(pick(p.src_scale, which) + at);
    decode16<E4M3>(__ldg(reinterpret_cast<const uint4*>(pick(p.src_codes, which) + (at * kPage + from % kPage) * D) + piece % kPieces),
                   x[i]);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      x[i][j] *= s;
      amax = fmaxf(amax, finite_abs(x[i][j]));
    }
  }
  amax = block_max<kThreads>(amax, red);
  const float s = scale_rule<E4M3>(amax);
  const float inv = s > 0.f ? 1.f / s : 0.f;
  const int64_t at = (int64_t)page * p.H_kv + hk;
  uint4* codes = reinterpret_cast<uint4*>(pick(p.dst_codes, which) + at * (kPage * D));
#pragma unroll
  for (int i = 0; i < 2; ++i) codes[threadIdx.x + i * kThreads] = encode16<E4M3>(x[i], inv);
  if (threadIdx.x == 0) pick(p.dst_scale, which)[at] = s;
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
  if (c->D == 64) fm::launch_append<64>(p, c->B, dtype, c->code_type, s);
  else if (c->D == 128) fm::launch_append<128>(p, c->B, dtype, c->code_type, s);
  else fm::launch_append<256>(p, c->B, dtype, c->code_type, s);
  return cudaGetLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
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
  if (dst->weight == src->weight || (dst->pos && dst->pos == src->pos)) return FM_ERR_INVALID_ARG;
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
  fm::select_kernel<<<dim3(src->H_kv, src->B), fm::kSelThreads, 0, s>>>(p);
  const dim3 grid(2 * (unsigned)((budget + fm::kPage - 1) / fm::kPage), src->H_kv, src->B);
  if (src->D == 64)
    src->code_type ? fm::compact_kernel<64, true><<<grid, 128, 0, s>>>(p) : fm::compact_kernel<64, false><<<grid, 128, 0, s>>>(p);
  else if (src->D == 128)
    src->code_type ? fm::compact_kernel<128, true><<<grid, 256, 0, s>>>(p) : fm::compact_kernel<128, false><<<grid, 256, 0, s>>>(p);
  else
    src->code_type ? fm::compact_kernel<256, true><<<grid, 512, 0, s>>>(p) : fm::compact_kernel<256, false><<<grid, 512, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

}  // extern "C"

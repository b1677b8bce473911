// Attention of a few query rows per sequence over the paged 8-bit K/V cache (fm_cache_attn).
//
//   O = sum_j p_j v_j / sum_j p_j,   p_j = 2^(s_j - m),   s_j = scale log2(e) (q . code_j) kscale_j,   m >= max_j s_j - 14
// in one pass over the keys: a running maximum m, the sum of p in fp32, O rescaled whenever m or its unit moves.
// Bound by the bytes of the cache: every live key's K and V codes are read once, 2 D bytes per key and K/V head, and each is used
// for the n_q * H / H_kv rows that share the head.  So the design starts from the copies:
//   * blocks that no row sees are found from the mask vectors by a kernel of its own (only where there is a
//     mask) before anything of them is loaded; it leaves the list of the others.
//   * the listed (sequence, K/V head, 64-token block) units of the whole batch form one flat order that is
//     cut into equal runs, one per CTA (one CTA per SM): ragged lengths, sparse masks and long single
//     sequences load every SM alike.  A (sequence, head) cut by a run's border is joined by the last kernel.
//   * each warp owns a ring of K and V pieces in shared memory, filled by TMA (a piece's keys by up to 128 bytes a box, 64- or
//     128-byte swizzle) through mbarriers, and works through its share of the run's blocks alone: no CTA
//     barrier until a (sequence, head) ends.
// The products run on mma.sync m16n8k16 with fp16 operands and fp32 accumulation, as
//   S^T [keys x rows] = K Q^T   and   O^T [d x rows] += V^T P^T,
// so that the 8 columns of the instruction are the few query rows and no row of it is padding for up to
// 8 rows.  (tcgen05 wants its operands as 16-bit tiles in shared memory or TMEM: converting the codes
// there and back would move three times the bytes per block that this form does, for a path whose tensor pipe is busy 17% of the
// time as it is.)  Both 8-bit formats are exact in fp16, so a score is the exact
// product of q and the cached key, summed in fp32.  The contraction orders are permuted so that a thread's
// operands are 16 consecutive bytes of a row: over d for K; for V by pairing the bytes of two tokens.
//
// Device time (graph of back-to-back calls; D = 128, 8 K/V heads of 4 query heads): one sequence of 131072 tokens 52 us, 5.2 TB/s
// of codes, of which some 8 us are the start (launch, dependent loads, first copies) and the join; 64 ragged ones of up to 8192
// (e4m3) with weights 146 us, without 122.  One of 517 tokens (D = 64): 9.5 us, all of it latency.
#include "fm_cache.cuh"

namespace fm {
namespace {

constexpr int kSMs = 148;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// P is held as 2^14 p in fp16: p down to 2^-28 keeps all 11 bits (a rounding is at most 2^-11 of p), and 2^14 is
// exact, so a row that sees one key returns its value unrounded.
constexpr float kPBias = 14.f;
// That is with O in units of the block's V scale.  In general a row's O is held in units of 2^u, u a whole number of the row's own, and
// its P is 2^14 p vscale / 2^u.  u stays while the largest P of the row's live keys in a block lies in [1, 2^15.5] (fp16 ends at 65504:
// p down to 2^-14 of the block's largest keeps all its bits), and otherwise moves so that the largest comes to 2^14: no key's share is
// lost where V's scales or the softmax weights of two blocks are far apart, in either order, and a block that a row does not see does
// not matter to it.  O moves with u, in fp32, as far as 2^kORoom; so what a block adds loses bits only where it is under 2^-118 of the
// largest element of the row's O.  (One unit for all rows, the block's scale, loses rows whose scales are 2^80 under another row's; a
// unit per row costs up to 1% at 8 rows, 3% at 32 rows of D = 64: 32 sequences of 8192 tokens 74.2 -> 76.4 us.)
constexpr float kPMid = 7.75f;  // half of 15.5
constexpr int kORoom = 118, kUnitMax = 126;

struct CacheAttnParams {
  const __nv_bfloat16* q;
  const int32_t* len;
  const int32_t* row;
  const int32_t* vec[4];
  const int32_t* page_table;
  const float* k_scale;
  const float* v_scale;
  const int32_t* pos;
  float* weight;
  __nv_bfloat16* o;
  float* lse;
  // workspace
  int32_t* units;    // [B * H_kv + 1] units before each (sequence, head)
  int32_t* chunk_n;  // [B * H_kv][n_chunk] listed blocks of each chunk of blocks (mask)
  int32_t* listed;   // [B * H_kv][n_chunk][chunk] those blocks, ascending: block << 1 | some row does not see some key (mask)
  float* part_o;     // [n_work][2][n_rows_pad][D] O over the keys of runs that end inside a (sequence, head)
  float2* part_ml;   // [n_work][2][n_rows_pad] their running maximum (log2) and sum of p
  float2* whole_ml;  // [B * H_kv][n_rows_pad] the same for (sequence, head)s inside one run (accumulate)
  float* score;      // [B * H_kv][max_pages * 64][rows4] scores in log2 units (accumulate)
  uint8_t* live;     // [B * H_kv][max_pages] block was read (accumulate)
  int* status;
  int B, H, H_kv, n_q, group, n_rows, n_rows_pad, rows4, Hm, n_k, n_pages, max_pages, n_work, n_row_chunks;
  int run_min;         // units of a run at least
  int n_chunk, chunk;  // chunks of blocks per (sequence, head), blocks of a chunk (n_chunk = 1 without a mask)
  int masked, causal, accumulate;
  float scale_log2;
};

template <int D, int NT>
struct CacheAttnCfg {
  // a warp's piece of work: a block, or at D = 256 half a one, since a ring of whole ones would leave shared memory for half the
  // warps (16 sequences of 16384 tokens under a window of 4096, 4 rows: 38 us against 42)
  static constexpr int kKeys = D == 256 ? kPage / 2 : kPage;
  static constexpr int kParts = kPage / kKeys;
  static constexpr int kWarps = 8;
  static constexpr int kThreads = kWarps * 32;
  // ring slots of a warp (each one K or one V block): what shared memory holds
  static constexpr int kSlots = D == 64 ? 4 : 2;
  static constexpr int kBox = D < 128 ? D : 128;     // bytes of a TMA box row (= swizzle span)
  static constexpr int kBoxes = D / kBox;
  static constexpr int kSlotBytes = kKeys * D;
  static constexpr int kRows = 8 * NT;               // query rows a CTA holds
  static constexpr int kKSteps = D / 16;
  static constexpr int kCap = (256 + kThreads - 1) / kThreads * kThreads - 2;  // units listed at a time
  static constexpr int kRing = 0;
  static constexpr int kQ = kRing + kWarps * kSlots * kSlotBytes;       // fragments [NT][D / 16][32] x 8 bytes
  static constexpr int kJoin = kQ + NT * kKSteps * 32 * 8;              // [warps][regs][32] fp32
  static constexpr int kRegs = D / 16 * NT * 4;
  static constexpr int kList = kJoin + kWarps * kRegs * 32 * 4;         // int4 entries
  static constexpr int kSegStart = kList + kCap * 16;                   // int [kCap + 1] (padded)
  static constexpr int kSegBh = kSegStart + (kCap + 4) * 4;             // int [kCap]
  static constexpr int kSegFlag = kSegBh + kCap * 4;                    // int [kCap]
  static constexpr int kUnitBh = kSegFlag + kCap * 4;                   // int [kCap + 2]: of the units, one before and one behind
  static constexpr int kMl = kUnitBh + (kCap + 4) * 4;                  // float4 [warps][rows]: maximum, sum, unit of O
  static constexpr int kQs = kMl + kWarps * kRows * 16;                 // float [rows]
  static constexpr int kBits = kQs + kRows * 4;                         // uint2 [warps][rows] mask bits
  static constexpr int kBar = kBits + kWarps * kRows * 8;               // mbarriers [warps][slots]
  static constexpr int kMisc = kBar + kWarps * kSlots * 8;              // abort, zero
  static constexpr int kRed = kMisc + 16;                               // int [32]
  static constexpr int kBefore = kRed + 128;                            // int [threads]: units before each thread's lists
  static constexpr int kBytes = kBefore + kThreads * 4;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kList % 16 == 0 && kMl % 16 == 0 && kBits % 8 == 0 && kBar % 8 == 0, "shared memory alignment");
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::
          "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
// D (fp32, 16 x 8) += A (fp16, 16 x 16) B (fp16, 16 x 8)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// transpose of the 8 x 8 matrix of 16-bit elements that the warp holds one pair per lane
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127
__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23 & 255u) - 127; }

// Bounds of one cached key: its row index and its two masked stretches.
struct KeyBounds {
  int j, lts, lte, uts, ute;
  bool in;  // slot in use
};
__device__ __forceinline__ void load_pos(const CacheAttnParams& p, KeyBounds& k, int64_t bh, int slot, int len) {
  k.in = slot < len;
  k.j = slot;
  if (k.in && p.pos) k.j = *(p.pos + bh * p.max_pages * kPage + slot);
}
__device__ __forceinline__ void load_vectors(const CacheAttnParams& p, KeyBounds& k, int64_t bhm) {
  k.lts = k.lte = 0x7FFFFFFF;  // canonical empty stretches; also those of keys outside the vectors
  k.uts = k.ute = 0;
  if (k.in && k.j >= 0 && k.j < p.n_k) {
    const int64_t at = bhm * p.n_k + k.j;
    if (p.vec[0]) k.lts = *(p.vec[0] + at);
    if (p.vec[1]) k.lte = *(p.vec[1] + at);
    if (p.vec[2]) k.uts = *(p.vec[2] + at);
    if (p.vec[3]) k.ute = *(p.vec[3] + at);
  }
}
__device__ __forceinline__ bool key_seen(const CacheAttnParams& p, const KeyBounds& k, int i) {
  return k.in && !(p.causal && k.j > i) && !(k.lts <= i && i < k.lte) && !(k.uts <= i && i < k.ute);
}

// Units of a run: an equal share of all, but no fewer than an equal cut of the average (sequence, head) into pieces of a turn of
// the CTA's warps (a run of less than a turn takes as long as one unit and leaves more partial sums to join, and a CTA takes
// the (sequence, head)s it holds one after the other); beyond a turn in whole ones (a part of one takes as long, and borders fall on
// sequences' ends more often: one sequence of 16384 tokens, 8 K/V heads: 14.7 us, with the bare share 17.3; 8 of 4000: 23.6
// and 22.3); or the average itself where that is at most one turn more (16 sequences of 1000 tokens, 8 K/V heads: 14 us, with
// equal shares 18).
__device__ __forceinline__ int units_per_run(const CacheAttnParams& p, int total) {
  const int average = total / (p.B * p.H_kv), pieces = max((average + p.run_min - 1) / p.run_min, 1);
  int share = max(max((total + p.n_work - 1) / p.n_work, (average + pieces - 1) / pieces), 1);
  if (share > p.run_min) share = (share + p.run_min - 1) / p.run_min * p.run_min;
  return share < average && average <= share + p.run_min && p.B * p.H_kv * 2 > p.n_work ? average : share;
}

// How many of the rows [i0, i1) see the key: those not before its pos (causal), less the union of its two stretches.
__device__ __forceinline__ int rows_seen(const CacheAttnParams& p, const KeyBounds& k, int i0, int i1) {
  if (p.causal) i0 = max(i0, k.j);
  if (!k.in || i0 >= i1) return 0;
  const int a0 = min(max(k.lts, i0), i1), a1 = max(min(k.lte, i1), a0);
  const int b0 = min(max(k.uts, i0), i1), b1 = max(min(k.ute, i1), b0);
  const int both = max(min(a1, b1) - max(a0, b0), 0);
  return (i1 - i0) - (a1 - a0) - (b1 - b0) + both;
}

// The lists of units: list e is chunk e % n_chunk of (sequence, head) e / n_chunk.
__device__ __forceinline__ int list_len(const CacheAttnParams& p, int e) {
  if (p.masked) return __ldcg(p.chunk_n + e);
  return (min(max(*(p.len + e / p.H_kv), 0), p.max_pages * kPage) + kPage - 1) / kPage;
}
// List and place in it of unit u.  before[t]: units before list t * per.
__device__ __forceinline__ int2 find_unit(const CacheAttnParams& p, const int* before, int threads, int per, int u) {
  int lo = 0, hi = threads - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (before[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  int e = lo * per, at = u - before[lo];
  for (int n = list_len(p, e); at >= n; n = list_len(p, ++e)) at -= n;
  return make_int2(e, at);
}

// First kernel of a call with a mask: a CTA classifies one chunk of a (sequence, head)'s blocks and lists those that some row
// sees.  Per key, a row i0 + t sees it unless t lies in one of two intervals, so the number of rows that see it is interval
// arithmetic whatever n_q; a block is listed where some key's is above 0, and its mask is left out later where all are n_q.  A
// warp takes kGang blocks at a time (their loads in flight together), two keys per lane: 20 bytes a key (pos, four bounds),
// against 2 D of codes, but three dependent loads: latency is what it costs, some 9 us of the call for 16 x 16384 slots x 4 heads.
constexpr int kPlanThreads = 256;
constexpr int kMaxChunk = 1024;
__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const CacheAttnParams p) {
  constexpr int kGang = 4;
  __shared__ uint8_t cls[kMaxChunk];
  grid_wait();
  grid_launch_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int64_t bh = (int64_t)b * p.H_kv + hk;
  const int len = min(max(*(p.len + b), 0), p.max_pages * kPage), nb = (len + kPage - 1) / kPage;
  const int first = blockIdx.x * p.chunk, n = min(nb - first, p.chunk);
  const int64_t list = bh * p.n_chunk + blockIdx.x;
  if (n <= 0) {
    if (threadIdx.x == 0) p.chunk_n[list] = 0;
    return;
  }
  const int row0 = *(p.row + b), head = b * p.Hm + (p.Hm > 1 ? hk * p.group : 0);
  for (int x0 = warp * kGang; x0 < n; x0 += kPlanThreads / 32 * kGang) {
    KeyBounds k[kGang][2];
    bool any[kGang], all[kGang];
    int page[kGang];
#pragma unroll
    for (int x = 0; x < kGang; ++x) {
      const int blk = first + min(x0 + x, n - 1);
      page[x] = *(p.page_table + (int64_t)b * p.max_pages + blk);
#pragma unroll
      for (int i = 0; i < 2; ++i) load_pos(p, k[x][i], bh, blk * kPage + lane + 32 * i, len);
      any[x] = false;
      all[x] = true;
    }
#pragma unroll 1
    for (int hg = 0; hg < (p.Hm > 1 ? p.group : 1); ++hg) {
#pragma unroll
      for (int x = 0; x < kGang; ++x)
#pragma unroll
        for (int i = 0; i < 2; ++i) load_vectors(p, k[x][i], head + hg);
#pragma unroll
      for (int x = 0; x < kGang; ++x)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int seen = rows_seen(p, k[x][i], row0, row0 + p.n_q);
          any[x] |= seen > 0;
          all[x] &= seen == p.n_q;
        }
    }
#pragma unroll
    for (int x = 0; x < kGang; ++x) {
      const bool some = __any_sync(0xffffffffu, any[x]), every = __all_sync(0xffffffffu, all[x]);
      if (lane == 0 && x0 + x < n) cls[x0 + x] = some && page[x] >= 0 && page[x] < p.n_pages ? (every ? 2 : 1) : 0;
    }
  }
  __syncthreads();
  if (p.accumulate)
    for (int x = threadIdx.x; x < n; x += kPlanThreads) p.live[bh * p.max_pages + first + x] = cls[x] != 0;
  if (warp == 0) {
    int32_t* out = p.listed + list * p.chunk;
    int count = 0;
    for (int x = lane; x - lane < n; x += 32) {
      const int c = x < n ? cls[x] : 0;
      const uint32_t there = __ballot_sync(0xffffffffu, c != 0);
      if (c) out[count + __popc(there & ((1u << lane) - 1u))] = (first + x) << 1 | (c == 1 ? 1 : 0);
      count += __popc(there);
    }
    if (lane == 0) p.chunk_n[list] = count;
  }
}

// What a segment (the units of one (sequence, head) in one list of a CTA) is to its CTA and to its (sequence, head).
constexpr int kReset = 1;   // the CTA's first units of it
constexpr int kDone = 2;    // the CTA's last ones: its sums are written
constexpr int kBegin = 4;   // its first units at all
constexpr int kEndAll = 8;  // its last ones
constexpr int kInside = 16; // kBegin, and not at the run's first unit

// Moves the units of rows whose largest P of this block would be out of range (see kPMid), with their O, and with alpha, which is 1
// afterwards.  The eight lanes of a row hold other elements of its O and decide alike: all else is the same to them.
template <int NT, int kTiles>
__device__ __forceinline__ void move_units(float (&o)[kTiles][NT][4], float (&alpha)[NT][2], const float (&above)[NT][2],
                                           float (&per_unit)[NT][2], float vs) {
  const int v_exp = exponent_of(vs);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) big = fmaxf(big, fmaxf(fabsf(o[i][nt][x]), fabsf(o[i][nt][2 + x])));
#pragma unroll
      for (int y = 4; y < 32; y <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, y));
      big *= alpha[nt][x];
      const int u = -exponent_of(per_unit[nt][x]);
      const float top = above[nt][x] + lg2(fabsf(vs * pow2i(-v_exp))) + (float)(v_exp - u);  // of P
      int to = u;
      if (above[nt][x] != kNegInf && fabsf(top - kPMid) > kPMid) {
        to = u + (int)rintf(top - kPBias);
        if (big > 0.f) to = max(to, u + exponent_of(big) - kORoom);
        to = min(max(max(to, v_exp - kUnitMax), -kUnitMax), kUnitMax);  // (vs / 2^u and 2^-u stay finite)
        per_unit[nt][x] = pow2i(-to);
      }
      // in two steps that neither overflow nor lose what the end keeps
      const int d = u - to, d1 = d / 2;
      const float f0 = alpha[nt][x] * pow2i(d1), f1 = pow2i(d - d1);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        o[i][nt][x] = o[i][nt][x] * f0 * f1;
        o[i][nt][2 + x] = o[i][nt][2 + x] * f0 * f1;
      }
      alpha[nt][x] = 1.f;
    }
}

template <int D, int NT, bool E4M3>
__global__ void __launch_bounds__(CacheAttnCfg<D, NT>::kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const CacheAttnParams p) {
  using C = CacheAttnCfg<D, NT>;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads, kSlots = C::kSlots;
  constexpr int kTiles = D / 16;  // 16-row tiles of O^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_base_1024(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int work = blockIdx.x / p.n_row_chunks, chunk = blockIdx.x % p.n_row_chunks;
  const int row_base = chunk * C::kRows;  // first query row of this CTA

  uint2* q_s = reinterpret_cast<uint2*>(smem + C::kQ);
  float* join = reinterpret_cast<float*>(smem + C::kJoin);
  int4* list = reinterpret_cast<int4*>(smem + C::kList);
  int* seg_start = reinterpret_cast<int*>(smem + C::kSegStart);
  int* seg_bh = reinterpret_cast<int*>(smem + C::kSegBh);
  int* seg_flag = reinterpret_cast<int*>(smem + C::kSegFlag);
  int* unit_bh = reinterpret_cast<int*>(smem + C::kUnitBh) + 1;  // [-1 .. kCap]
  float4* ml_s = reinterpret_cast<float4*>(smem + C::kMl);
  float* qs_s = reinterpret_cast<float*>(smem + C::kQs);
  uint2* bits_s = reinterpret_cast<uint2*>(smem + C::kBits) + warp * C::kRows;
  int* misc = reinterpret_cast<int*>(smem + C::kMisc);
  volatile int* abort_flag = misc;
  const volatile int* never = misc + 1;
  int* red = reinterpret_cast<int*>(smem + C::kRed);
  int* before = reinterpret_cast<int*>(smem + C::kBefore);
  const uint32_t ring = smem_u32(smem + C::kRing) + warp * kSlots * C::kSlotBytes;
  uint8_t* ring_p = smem + C::kRing + warp * kSlots * C::kSlotBytes;
  const uint32_t bar0 = smem_u32(smem + C::kBar) + warp * kSlots * 8;

  if (threadIdx.x == 0) {
    misc[0] = misc[1] = 0;
    for (int i = 0; i < kWarps * kSlots; ++i) mbar_init(smem_u32(smem + C::kBar) + 8 * i, 1);
    fence_barrier_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  const int cap = p.max_pages * kPage;
  grid_wait();
  grid_launch_next();
  // units before each thread's share of the lists, and in all
  const int n_lists = p.B * p.H_kv * p.n_chunk, lists_per = (n_lists + kThreads - 1) / kThreads;
  int total;
  {
    const int e0 = min((int)threadIdx.x * lists_per, n_lists), e1 = min(e0 + lists_per, n_lists);
    int mine = 0;
    for (int e = e0; e < e1; ++e) mine += list_len(p, e);
    int x = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, s);
      if (lane >= s) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int pre = x - mine;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) pre += red[w];
      total += red[w];
    }
    before[threadIdx.x] = pre;
    __syncthreads();
  }
  const int per = units_per_run(p, total);
  const int c0 = min((int64_t)work * per, (int64_t)total), c1 = min(c0 + per, total);
  if (total == 0 && blockIdx.x == 0)
    for (int e = threadIdx.x; e <= p.B * p.H_kv; e += kThreads) p.units[e] = 0;
  float o[kTiles][NT][4];
  float m[NT][2], l[NT][2];
  float per_unit[NT][2];            // 2^-u of the row's unit of O
  int item = 0;                     // ring items consumed by this warp so far
  int begun = 0;                    // flags of the current segment's first units
  bool ok = true;

  for (int w0 = c0; w0 < c1; w0 += C::kCap) {
    const int nu = min(C::kCap, c1 - w0);
    // ------------------------------------------------------------------------ list the run's next units
    if (w0 != c0) __syncthreads();  // the last list has been read
    constexpr int kPer = (C::kCap + 2) / kThreads;
    float scale_k[kPer], scale_v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int u = i * kThreads + (int)threadIdx.x - 1;  // -1 and nu: the unit before and the one behind
      if (u <= nu && (w0 + u < 0 || w0 + u >= total)) unit_bh[u] = -1;
      else if (u <= nu) {
        const int2 at = find_unit(p, before, kThreads, lists_per, w0 + u);
        const int bh = at.x / p.n_chunk;
        unit_bh[u] = bh;
        if (u < 0 || u == nu) continue;
        const int b = bh / p.H_kv, hk = bh - b * p.H_kv;
        const int len = min(max(*(p.len + b), 0), cap);
        int blk = at.y, partial = 0;
        if (p.masked) {
          const int w = __ldcg(p.listed + (int64_t)at.x * p.chunk + at.y);
          blk = w >> 1;
          partial = w & 1;
        } else {
          partial = (blk + 1) * kPage > len;
        }
        int page = *(p.page_table + (int64_t)b * p.max_pages + blk);
        const bool there = page >= 0 && page < p.n_pages;
        if (!there) page = 0;  // read, but no key of it is seen
        const int row = page * p.H_kv + hk;
        *reinterpret_cast<int2*>(&list[u]) = make_int2(row * kPage, blk * kPage + (there ? partial : 3));
        scale_k[i] = there ? *(p.k_scale + row) : 0.f;  // (stored once the ring has started)
        scale_v[i] = there ? *(p.v_scale + row) : 0.f;
        if (p.accumulate && !p.masked && chunk == 0) p.live[(int64_t)bh * p.max_pages + blk] = there;
      }
    }
    __syncthreads();
    // ---------------------------------------------------------------- the ring of this warp
    const int n_pieces = nu * C::kParts, n_items = 2 * (n_pieces > warp ? (n_pieces - warp + kWarps - 1) / kWarps : 0);
    int issued = 0, done = 0;
    auto issue = [&]() {  // the next item: K of a piece, then its V
      if (issued < n_items && ok) {
        if (lane == 0) {
          const int piece = warp + kWarps * (issued >> 1), row = list[piece / C::kParts].x + piece % C::kParts * C::kKeys;
          const int slot = (item + issued) % kSlots;
          const uint32_t bar = bar0 + 8 * slot;
          mbar_arrive_expect_tx(bar, C::kSlotBytes);
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x)
            tma_load_2d(ring + slot * C::kSlotBytes + x * C::kKeys * C::kBox, (issued & 1) ? &tm_v : &tm_k, bar, x * C::kBox,
                        row);
        }
        ++issued;
      }
    };
    auto wait = [&]() {  // the item to be consumed next has arrived
      const int it = item + done;
      if (ok && !__all_sync(0xffffffffu, mbar_wait(bar0 + 8 * (it % kSlots), (it / kSlots) & 1, abort_flag))) {
        // gave up: the warp goes on to take part in the CTA's barriers, but issues nothing more; its copies in
        // flight must land before the ring can be left
        ok = false;
        if (lane == 0) {
          record_failure(p.status, abort_flag, 51);
          for (int i = done; i < issued; ++i) mbar_wait(bar0 + 8 * ((item + i) % kSlots), ((item + i) / kSlots) & 1, never);
        }
      }
    };
    for (int i = 0; i < kSlots; ++i) issue();

    // query rows of a segment into shared memory as fragments: row n of tile n / 8, scaled by a power of
    // two that puts its largest element into [2^14, 2^15) (exact; bf16's range is wider than fp16's, and
    // elements under 2^-28 of the largest lose low bits, at most 2^-39 of the row's largest)
    constexpr int kQRows = (C::kRows + kWarps - 1) / kWarps;
    constexpr int kQElems = D / 32;  // consecutive elements per lane
    uint32_t qreg[kQRows][kQElems / 2];
    auto load_q = [&](int bh) {
#pragma unroll
      for (int i = 0; i < kQRows; ++i) {
        const int n = warp + kWarps * i, r = row_base + n;
#pragma unroll
        for (int x = 0; x < kQElems / 2; ++x) qreg[i][x] = 0;
        if (n < C::kRows && r < p.n_rows) {
          const int b = bh / p.H_kv, hk = bh % p.H_kv;
          const int h = hk * p.group + r / p.n_q, tq = r % p.n_q;
          const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + (((int64_t)b * p.n_q + tq) * p.H + h) * D) +
                                lane * (kQElems / 2);
#pragma unroll
          for (int x = 0; x < kQElems / 2; ++x) qreg[i][x] = *(src + x);
        }
      }
    };
    auto store_q = [&]() {
#pragma unroll
      for (int i = 0; i < kQRows; ++i) {
        const int n = warp + kWarps * i;
        if (n >= C::kRows) continue;
        float amax = 0.f;
#pragma unroll
        for (int x = 0; x < kQElems / 2; ++x) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(qreg[i][x])), fabsf(bf16_hi(qreg[i][x]))));
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
        int e = 14 - ((int)(__float_as_uint(amax) >> 23) - 127);
        e = amax > 0.f && amax <= 3.402823466e38f ? min(max(e, -126), 126) : 0;
        const float f = __uint_as_float((uint32_t)(e + 127) << 23), back = __uint_as_float((uint32_t)(127 - e) << 23);
        if (lane == 0) qs_s[n] = p.scale_log2 * back;
        uint32_t h[kQElems / 2];
#pragma unroll
        for (int x = 0; x < kQElems / 2; ++x) h[x] = pack_f16(bf16_lo(qreg[i][x]) * f, bf16_hi(qreg[i][x]) * f);
        // element d: 16-byte piece c = d / 16 of its box row; word s of the piece is k-step (.., s)
#pragma unroll
        for (int x = 0; x < kQElems / 2; ++x) {
          const int d = lane * kQElems + 2 * x, in_box = d % C::kBox, c = in_box >> 4, s = (d & 15) >> 2;
          const int tt = C::kBox == 128 ? c >> 1 : c, hh = C::kBox == 128 ? c & 1 : 0;
          const int ks = d / C::kBox * (C::kBox / 16) + hh * 4 + s;
          uint32_t* dst = reinterpret_cast<uint32_t*>(q_s + ((n >> 3) * C::kKSteps + ks) * 32 + (n & 7) * 4 + tt);
          dst[(d >> 1) & 1] = h[x];
        }
      }
    };
    int n_seg = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {  // segments: runs of units of one (sequence, head)
      const int u = i * kThreads + (int)threadIdx.x - 1;
      const bool starts = u >= 0 && u < nu && (u == 0 || unit_bh[u] != unit_bh[u - 1]);
      const uint32_t who = __ballot_sync(0xffffffffu, starts);
      if (i > 0) __syncthreads();  // (the counts of the units before have been read)
      if (lane == 0) red[warp] = __popc(who);
      __syncthreads();
      int k = n_seg + __popc(who & ((1u << lane) - 1u));
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) k += red[w];
        n_seg += red[w];
      }
      if (starts) {
        const bool begin = unit_bh[u] != unit_bh[u - 1];
        seg_start[k] = u;
        seg_bh[k] = unit_bh[u];
        seg_flag[k] = (begin || w0 + u == c0 ? kReset : 0) | (begin ? kBegin : 0) | (begin && w0 + u > c0 ? kInside : 0);
      }
    }
    if (threadIdx.x == 0) seg_start[n_seg] = nu;
    __syncthreads();
    for (int k = threadIdx.x; k < n_seg; k += kThreads) {
      const int u = seg_start[k + 1] - 1;  // the segment's last unit
      const bool end = unit_bh[u] != unit_bh[u + 1];
      seg_flag[k] |= (end || w0 + u == c1 - 1 ? kDone : 0) | (end ? kEndAll : 0);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int u = i * kThreads + (int)threadIdx.x - 1;
      if (u >= 0 && u < nu) *(reinterpret_cast<float2*>(&list[u]) + 1) = make_float2(scale_k[i], scale_v[i]);
    }
    if (blockIdx.x == 0 && w0 == 0) {  // units before each (sequence, head), for the last kernel
      const int e0 = min((int)threadIdx.x * lists_per, n_lists), e1 = min(e0 + lists_per, n_lists);
      int pre = before[threadIdx.x];
      for (int e = e0; e < e1; ++e) {
        if (e % p.n_chunk == 0) p.units[e / p.n_chunk] = pre;
        pre += list_len(p, e);
      }
      if (threadIdx.x == 0) p.units[p.B * p.H_kv] = total;
    }
    __syncthreads();

#pragma unroll 1
    for (int sg = -1; sg < n_seg; ++sg) {
      // the rows of the next segment: loaded here, in flight during this one, stored at the end of the loop's body
      if (sg + 1 < n_seg) load_q(seg_bh[sg + 1]);
      if (sg >= 0) {
      const int bh = seg_bh[sg], flag = seg_flag[sg], e1 = seg_start[sg + 1] * C::kParts;
      const int b = bh / p.H_kv, hk = bh % p.H_kv;
      const int len = min(max(*(p.len + b), 0), cap);
      if (flag & kReset) {
        begun = flag;
        const int e = warp + kWarps * (done >> 1);  // the warp's first piece: its scale is the unit to begin with
        const float start = e < e1 ? pow2i(-min(max(exponent_of(__int_as_float(list[e / C::kParts].w)), -kUnitMax), kUnitMax)) : 1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          m[nt][0] = m[nt][1] = kNegInf;
          l[nt][0] = l[nt][1] = 0.f;
          per_unit[nt][0] = per_unit[nt][1] = start;
#pragma unroll
          for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[i][nt][c] = 0.f;
        }
      }
      for (int e = warp + kWarps * (done >> 1); e < e1; e += kWarps) {
        const int4 ent = list[e / C::kParts];
        const int slot0 = (ent.y & ~3) + e % C::kParts * C::kKeys;
        const bool partial = ent.y & 1, missing = ent.y & 2;
        const float ks = __int_as_float(ent.z), vs = __int_as_float(ent.w);
        if (partial) {
          // bit k of row n's word pair: the row sees key k of the block
          KeyBounds k[2];
          if (p.masked) {
#pragma unroll
            for (int i = 0; i < C::kKeys / 32; ++i) load_pos(p, k[i], bh, slot0 + lane + 32 * i, len);
            const int row0 = *(p.row + b);
            // row row_base + n is query tq of head hg of the group (rows behind the last one take its bits)
            int hg = row_base / p.n_q, tq = row_base - hg * p.n_q;
            bool new_head = true;
            uint32_t lo = 0, hi = 0;
#pragma unroll 1
            for (int n = 0; n < C::kRows; ++n) {
              if (row_base + n < p.n_rows) {
                if (new_head) {
                  const int64_t bhm = p.Hm > 1 ? (int64_t)b * p.Hm + hk * p.group + hg : b;
#pragma unroll
                  for (int i = 0; i < C::kKeys / 32; ++i) load_vectors(p, k[i], bhm);
                }
                lo = __ballot_sync(0xffffffffu, key_seen(p, k[0], row0 + tq));
                hi = C::kKeys == 64 ? __ballot_sync(0xffffffffu, key_seen(p, k[1], row0 + tq)) : 0u;
                new_head = false;
                if (++tq == p.n_q) {
                  tq = 0;
                  ++hg;
                  new_head = p.Hm > 1;
                }
              }
              if (lane == (n & 31)) bits_s[n] = make_uint2(lo, hi);
            }
          } else {
            const uint32_t lo = __ballot_sync(0xffffffffu, !missing && slot0 + lane < len);
            const uint32_t hi = __ballot_sync(0xffffffffu, !missing && slot0 + lane + 32 < len);
            if (lane < C::kRows) bits_s[lane] = make_uint2(lo, hi);
          }
          __syncwarp();
        }
        // ------------------------------------------------------------ S^T = K Q^T (the piece's keys x rows)
        wait();
        constexpr int kJ = C::kKeys / 16;  // 16-key tiles of the piece
        float s[kJ][NT][4];
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[j][nt][c] = 0.f;
        {
          const uint8_t* kb = ring_p + (item + done) % kSlots * C::kSlotBytes;
          // (not unrolled: the kernel's code is read once by most calls, and its misses cost more than the loop)
#pragma unroll 1
          for (int x = 0; x < C::kBoxes; ++x)
#pragma unroll 1
            for (int h = 0; h < (C::kBox == 128 ? 2 : 1); ++h) {
              // key 16 j + 8 r + g, 16-byte piece 2 t + h (t for D = 64): no two lanes of a quarter warp
              // share a bank under the swizzle
              uint4 raw[kJ][2];
#pragma unroll
              for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const int key = 16 * j + 8 * r + g;
                  const int c = C::kBox == 128 ? ((2 * t + h) ^ (key & 7)) : (t ^ ((key >> 1) & 3));
                  raw[j][r] = *reinterpret_cast<const uint4*>(kb + x * C::kKeys * C::kBox + key * C::kBox + c * 16);
                }
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const int step = x * (C::kBox / 16) + h * 4 + w;
                uint2 bq[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) bq[nt] = q_s[(nt * C::kKSteps + step) * 32 + lane];
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                  const uint32_t wa = w == 0 ? raw[j][0].x : w == 1 ? raw[j][0].y : w == 2 ? raw[j][0].z : raw[j][0].w;
                  const uint32_t wb = w == 0 ? raw[j][1].x : w == 1 ? raw[j][1].y : w == 2 ? raw[j][1].z : raw[j][1].w;
                  uint32_t a0, a1, a2, a3;
                  decode4<E4M3>(wa, a0, a2);
                  decode4<E4M3>(wb, a1, a3);
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) mma_f16(s[j][nt], a0, a1, a2, a3, bq[nt].x, bq[nt].y);
                }
              }
            }
        }
        __syncwarp();
        issue();  // K's slot is free
        ++done;
        // ------------------------------------------------------------ softmax: this thread's rows 2t, 2t+1
        uint32_t pb[kJ][NT][2];  // P^T fragments
        bool moved = false, far = false;
        float alpha[NT][2], above[NT][2];  // above: the block's largest score over m (-inf: the row sees no key)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float cf = qs_s[nt * 8 + 2 * t + x] * ks;
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
              s[j][nt][x] *= cf;
              s[j][nt][2 + x] *= cf;
            }
            if (partial) {
              const uint2 bits = bits_s[nt * 8 + 2 * t + x];
#pragma unroll
              for (int j = 0; j < kJ; ++j) {
                const uint32_t w = j < 2 ? bits.x : bits.y;
                if (!((w >> (16 * (j & 1) + g)) & 1u)) s[j][nt][x] = kNegInf;
                if (!((w >> (16 * (j & 1) + 8 + g)) & 1u)) s[j][nt][2 + x] = kNegInf;
              }
            }
          }
          if (p.accumulate && row_base + nt * 8 + 2 * t < p.rows4) {
            float* dst = p.score + ((int64_t)bh * cap + slot0 + g) * p.rows4 + row_base + nt * 8 + 2 * t;
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
              *reinterpret_cast<float2*>(dst + (int64_t)(16 * j) * p.rows4) = make_float2(s[j][nt][0], s[j][nt][1]);
              *reinterpret_cast<float2*>(dst + (int64_t)(16 * j + 8) * p.rows4) = make_float2(s[j][nt][2], s[j][nt][3]);
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float mx = fmaxf(s[0][nt][x], s[0][nt][2 + x]);
#pragma unroll
            for (int j = 1; j < kJ; ++j) mx = fmaxf(mx, fmaxf(s[j][nt][x], s[j][nt][2 + x]));
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
            const float m_new = fmaxf(m[nt][x], mx - kPBias);
            const float m_use = m_new == kNegInf ? 0.f : m_new;
            alpha[nt][x] = ex2(m[nt][x] - m_use);
            moved |= m_new != m[nt][x];
            m[nt][x] = m_new;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
              s[j][nt][x] = ex2(s[j][nt][x] - m_use);
              s[j][nt][2 + x] = ex2(s[j][nt][2 + x] - m_use);
              sum += s[j][nt][x] + s[j][nt][2 + x];
            }
            l[nt][x] = fmaf(l[nt][x], alpha[nt][x], sum);
            above[nt][x] = mx - m_use;
            // log2 of the block's largest P, outside [0, 2 kPMid]?
            far |= mx != kNegInf && fabsf(above[nt][x] + (lg2(fabsf(vs * per_unit[nt][x])) - kPMid)) > kPMid;
          }
        }
        if (__any_sync(0xffffffffu, far) && vs != 0.f) move_units<NT, kTiles>(o, alpha, above, per_unit, vs);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float pf0 = above[nt][0] != kNegInf ? vs * per_unit[nt][0] : 0.f;  // P / p
          const float pf1 = above[nt][1] != kNegInf ? vs * per_unit[nt][1] : 0.f;
#pragma unroll
          for (int j = 0; j < kJ; ++j) {  // keys 16 j + 2t, +1 and + 8, + 9 of row g, as the product reads them
            pb[j][nt][0] = transpose8x8(pack_f16(s[j][nt][0] * pf0, s[j][nt][1] * pf1));
            pb[j][nt][1] = transpose8x8(pack_f16(s[j][nt][2] * pf0, s[j][nt][3] * pf1));
          }
        }
        // O moves to the new maximum
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float f0 = alpha[nt][0], f1 = alpha[nt][1];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
              o[i][nt][0] *= f0;
              o[i][nt][1] *= f1;
              o[i][nt][2] *= f0;
              o[i][nt][3] *= f1;
            }
          }
        }
        // ------------------------------------------------------------ O^T += V^T P^T
        wait();
        {
          uint8_t* vb = ring_p + (item + done) % kSlots * C::kSlotBytes;
          const int valid = missing ? 0 : len - slot0;
          if (partial && valid < C::kKeys) {  // slots never written may hold any bytes, a NaN's among them
            for (int x = lane; x < (C::kKeys - max(valid, 0)) * (D / 16); x += 32) {
              const int row = max(valid, 0) + x / (D / 16), piece = x % (D / 16);
              *reinterpret_cast<uint4*>(vb + piece / (C::kBox / 16) * C::kKeys * C::kBox + row * C::kBox + piece % (C::kBox / 16) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();  // (the slot's next copy comes after these)
            __syncwarp();
          }
          constexpr int kWords = C::kBox / 32;  // 32-bit words of a row's piece that belongs to lane group g
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x)
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
              uint32_t raw[4][kWords];  // keys 16 j + 2t, + 1, + 8, + 9
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int key = 16 * j + 2 * t + (r & 1) + 8 * (r >> 1);
                if constexpr (C::kBox == 128) {
                  const uint4 v = *reinterpret_cast<const uint4*>(vb + x * C::kKeys * 128 + key * 128 + ((g ^ (key & 7)) << 4));
                  raw[r][0] = v.x;
                  raw[r][1] = v.y;
                  raw[r][2] = v.z;
                  raw[r][3] = v.w;
                } else {
                  const uint2 v = *reinterpret_cast<const uint2*>(vb + key * 64 + (((g >> 1) ^ ((key >> 1) & 3)) << 4) + (g & 1) * 8);
                  raw[r][0] = v.x;
                  raw[r][1] = v.y;
                }
              }
#pragma unroll
              for (int w = 0; w < kWords; ++w) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {  // bytes 2u, 2u + 1: d rows of tile 2 w + u
                  const uint32_t sel = u ? 0x7362u : 0x5140u;
                  uint32_t a0, a1, a2, a3;
                  decode4<E4M3>(__byte_perm(raw[0][w], raw[1][w], sel), a0, a1);
                  decode4<E4M3>(__byte_perm(raw[2][w], raw[3][w], sel), a2, a3);
                  const int tile = x * (C::kBox / 16) + 2 * w + u;
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) mma_f16(o[tile][nt], a0, a1, a2, a3, pb[j][nt][0], pb[j][nt][1]);
                }
              }
            }
        }
        __syncwarp();
        issue();
        ++done;
      }
      if (!(flag & kDone)) break;  // the list's last one: goes on in the next list

      // -------------------------------------------------- the segment's end: join the warps
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int y = 4; y < 32; y <<= 1) l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], y);
          if (g == 0)
            ml_s[warp * C::kRows + nt * 8 + 2 * t + x] =
                make_float4(m[nt][x], l[nt][x], pow2i(-exponent_of(per_unit[nt][x])), 0.f);
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) join[(warp * C::kRegs + (i * NT + nt) * 4 + c) * 32 + lane] = o[i][nt][c];
      }
      __syncthreads();
      // each warp adds up a share of the accumulators' places (pairs: the same row, d and d + 1) over the warps, in order
      const bool whole = (begun & kBegin) && (flag & kEndAll);
      const int64_t part = ((int64_t)work * 2 + (begun & kInside ? 1 : 0)) * p.n_rows_pad;
#pragma unroll 1
      for (int pair = warp; pair < C::kRegs / 2; pair += kWarps) {
        const int x = pair & 1, nt = pair / 2 % NT, i = pair / (2 * NT);
        const int n = nt * 8 + 2 * t + x, r = row_base + n;
        float mm = kNegInf;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml_s[w * C::kRows + n].x);
        const float use = mm == kNegInf ? 0.f : mm;
        float f[kWarps], unit[kWarps], ll = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 v = ml_s[w * C::kRows + n];
          f[w] = ex2(v.x - use);
          unit[w] = v.z;
          ll += v.y * f[w];
        }
        // The division by the sum comes before the unit: the quotient is an average of codes, and its product with the unit no
        // larger than the largest value, where 2^14 n times that may be past fp32's range.
        const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);  // (a NaN stays one)
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* src = join + (w * C::kRegs + (i * NT + nt) * 4 + x) * 32 + lane;
          const float fo = f[w] * inv;
          y0 = fmaf(src[0] * fo, unit[w], y0);
          y1 = fmaf(src[64] * fo, unit[w], y1);
        }
        const int d = i / (C::kBox / 16) * C::kBox + g * (C::kBox / 8) + 2 * (i % (C::kBox / 16));
        if (whole) {
          if (r >= p.n_rows) continue;
          const int h = hk * p.group + r / p.n_q, tq = r % p.n_q;
          *reinterpret_cast<uint32_t*>(p.o + (((int64_t)b * p.n_q + tq) * p.H + h) * D + d) = pack_bf16(y0, y1);
          if (i == 0 && g == 0) {
            p.lse[((int64_t)b * p.H + h) * p.n_q + tq] = (mm + log2f(ll)) * kLn2;
            if (p.accumulate) p.whole_ml[(int64_t)bh * p.n_rows_pad + r] = make_float2(mm, ll);
          }
        } else {
          *reinterpret_cast<float2*>(p.part_o + (part + r) * D + d) = make_float2(y0, y1);
          if (i == 0 && g == 0) p.part_ml[part + r] = make_float2(mm, ll);
        }
      }
      }
      if (sg + 1 < n_seg) store_q();  // (every warp is done with the old rows)
      __syncthreads();
    }
    item += done;
  }
}

// Last kernel (it may be resident before the one before ends, so what that wrote is read through L2).  The first CTAs join
// the rows of the (sequence, head)s that several runs share, a CTA per row: with M the largest of the runs' maxima,
// l = sum_c l_c 2^(m_c - M), O = sum_c O_c (l_c 2^(m_c - M) / l), O_c the run's own quotient (of a value's size, so no sum
// overflows).  The others add the softmax weights 2^(s - M) / l of kWeightSlots keys each to the cache's, from the stored scores:
// 4 bytes per key and row written and read (for 4 rows 32 bytes beside a key's 256 of codes), against reading K again and forming
// its products twice.  1024 slots a CTA, 8 a thread, for up to 8 rows: 64 ragged sequences of up to 8192 tokens, 8 K/V heads, 4
// rows: 145 us for the call (five CTAs an SM instead of six: 148); 512 slots: 150; 2048: 4 sequences of 2048 take 15.0 us instead
// of 13.7.  512 slots and more CTAs on an SM beyond, where a CTA's time is its rows': 21 sequences of
// up to 19055 tokens, 80 rows: 305 us; with 1024 slots 347.
constexpr int kJoinThreads = 128;
constexpr int weight_slots(int n_rows) { return n_rows <= 8 ? 1024 : 512; }
constexpr int kMaxRows = 1024;

struct Span {  // the runs that hold a (sequence, head), and where their partial sums are
  int first, last;     // last < first: no units
  int64_t part0;    // first row of run `first`'s partial sums; run c > first has them in its first place
};
__device__ __forceinline__ Span span_of(const CacheAttnParams& p, int bh) {
  const int u0 = __ldcg(p.units + bh), u1 = __ldcg(p.units + bh + 1);
  const int per = units_per_run(p, __ldcg(p.units + p.B * p.H_kv));
  Span s;
  s.first = u0 / per;
  s.last = u1 > u0 ? (u1 - 1) / per : s.first - 1;
  s.part0 = ((int64_t)s.first * 2 + (u0 > s.first * per ? 1 : 0)) * p.n_rows_pad;
  return s;
}
__device__ __forceinline__ int64_t part_of(const CacheAttnParams& p, const Span& s, int c) {
  return c == s.first ? s.part0 : (int64_t)c * 2 * p.n_rows_pad;
}
// Maximum and sum of row r over its runs, by a warp (the same order for every caller).
__device__ __forceinline__ float2 join_ml(const CacheAttnParams& p, const Span& s, int r, int lane) {
  float2 v = make_float2(kNegInf, 0.f);  // of run first + lane
  if (s.first + lane <= s.last) v = __ldcg(&p.part_ml[part_of(p, s, s.first + lane) + r]);
  float m = v.x;
  for (int c = s.first + lane + 32; c <= s.last; c += 32) m = fmaxf(m, __ldcg(&p.part_ml[part_of(p, s, c) + r].x));
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float use = m == kNegInf ? 0.f : m;
  float l = v.y * ex2(v.x - use);
  for (int c = s.first + lane + 32; c <= s.last; c += 32) {
    const float2 w = __ldcg(&p.part_ml[part_of(p, s, c) + r]);
    l += w.y * ex2(w.x - use);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  return make_float2(m, l);
}

// The same by a thread, over at most 8 runs.
__device__ __forceinline__ float2 join_ml_few(const CacheAttnParams& p, const Span& s, int r) {
  float2 v[8];
  float m = kNegInf;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = s.first + i <= s.last ? __ldcg(&p.part_ml[part_of(p, s, s.first + i) + r]) : make_float2(kNegInf, 0.f);
    m = fmaxf(m, v[i].x);
  }
  const float use = m == kNegInf ? 0.f : m;
  float l = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) l += v[i].y * ex2(v[i].x - use);
  return make_float2(m, l);
}

template <int D, int kWeightSlots>
__global__ void __launch_bounds__(kJoinThreads, kWeightSlots == 512 ? 8 : 6) cache_join_kernel(const CacheAttnParams p) {
  __shared__ float2 ml[kMaxRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_wait();
  grid_launch_next();
  const int n_join = p.B * p.H_kv * p.n_rows;
  if ((int)blockIdx.x < n_join) {
    // every warp finds the row's maximum and sum, then adds up every fourth run's part
    constexpr int kPer = D / 32;  // consecutive d of a lane
    __shared__ float part[kJoinThreads / 32][D];
    const int bh = blockIdx.x / p.n_rows, r = blockIdx.x % p.n_rows, b = bh / p.H_kv, hk = bh % p.H_kv;
    const Span s = span_of(p, bh);
    if (s.first == s.last) return;  // written by its one run
    const float2 t = join_ml(p, s, r, lane);
    const float use = t.x == kNegInf ? 0.f : t.x, inv = t.y > 0.f ? 1.f / t.y : (t.y == 0.f ? 0.f : t.y);
    float x[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = 0.f;
#pragma unroll 4
    for (int c = s.first + warp; c <= s.last; c += kJoinThreads / 32) {
      const int64_t at = part_of(p, s, c) + r;
      const float2 ml_c = __ldcg(&p.part_ml[at]);
      const float f = ml_c.y * ex2(ml_c.x - use) * inv;
      const float2* src = reinterpret_cast<const float2*>(p.part_o + at * D + lane * kPer);
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        const float2 v = __ldcg(src + i / 2);
        x[i] = fmaf(v.x, f, x[i]);
        x[i + 1] = fmaf(v.y, f, x[i + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) part[warp][lane * kPer + i] = x[i];
    __syncthreads();
    const int h = hk * p.group + r / p.n_q, tq = r % p.n_q;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (((int64_t)b * p.n_q + tq) * p.H + h) * D);
    for (int d = threadIdx.x; d < D / 2; d += kJoinThreads) {
      float y0 = 0.f, y1 = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinThreads / 32; ++w) {
        y0 += part[w][2 * d];
        y1 += part[w][2 * d + 1];
      }
      dst[d] = pack_bf16(y0, y1);
    }
    if (threadIdx.x == 0) p.lse[((int64_t)b * p.H + h) * p.n_q + tq] = t.y == 0.f ? kNegInf : (t.x + log2f(t.y)) * kLn2;
    return;
  }
  // Weights.  kWeightSlots / kJoinThreads keys a thread; what does not depend on anything is loaded first, so that there are two memory latencies
  // on the way, not one for each of length, runs, sums, liveness, scores.
  constexpr int kKeys = kWeightSlots / kJoinThreads;
  const int cap = p.max_pages * kPage, per_bh = (cap + kWeightSlots - 1) / kWeightSlots;
  const int w = blockIdx.x - n_join, bh = w / per_bh, s0 = w % per_bh * kWeightSlots, b = bh / p.H_kv;
  const int len = min(max(*(p.len + b), 0), cap);
  const Span s = span_of(p, bh);
  float* weight = p.weight + (int64_t)bh * cap;
  float x[kKeys];
  uint8_t live[kKeys];
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const int slot = s0 + i * kJoinThreads + threadIdx.x;
    live[i] = slot < cap ? __ldcg(p.live + (int64_t)bh * p.max_pages + slot / kPage) : 0;
    x[i] = slot < cap ? weight[slot] : 0.f;
  }
  if (s0 >= len) return;
  const float4* sc = reinterpret_cast<const float4*>(p.score + ((int64_t)bh * cap + s0 + threadIdx.x) * p.rows4);
  float4 v[kKeys];
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    live[i] = live[i] && s0 + i * kJoinThreads + (int)threadIdx.x < len;
    v[i] = live[i] ? __ldcg(sc + i * kJoinThreads * p.rows4 / 4) : make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
  }
  // a warp per row, or where there are more rows than warps and few runs a thread per row, their loads in flight together (80 rows
  // over 21 sequences of up to 19055 tokens, 2 K/V heads: 346 us for the call, 369 with a warp per row, both with 1024 slots a CTA)
  const bool few = p.rows4 > kJoinThreads / 32 && s.last - s.first < 8;
  const int r_step = few ? kJoinThreads : kJoinThreads / 32;
  for (int r = few ? threadIdx.x : warp; r < p.rows4; r += r_step) {
    float2 t = make_float2(kNegInf, 0.f);
    if (r < p.n_rows)
      t = s.first == s.last ? __ldcg(&p.whole_ml[(int64_t)bh * p.n_rows_pad + r])
          : few             ? join_ml_few(p, s, r)
                            : join_ml(p, s, r, lane);
    if (few || lane == 0) ml[r] = make_float2(t.x == kNegInf ? 0.f : t.x, t.y > 0.f ? 1.f / t.y : (t.y == 0.f ? 0.f : t.y));
  }
  __syncthreads();
#pragma unroll 1
  for (int r = 0; r < p.rows4; r += 4) {
    const float2 m0 = ml[r], m1 = ml[r + 1], m2 = ml[r + 2], m3 = ml[r + 3];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      float y = ex2(v[i].x - m0.x) * m0.y;
      // rows behind the last one hold no score
      if (r + 1 < p.n_rows) y += ex2(v[i].y - m1.x) * m1.y;
      if (r + 2 < p.n_rows) y += ex2(v[i].z - m2.x) * m2.y;
      if (r + 3 < p.n_rows) y += ex2(v[i].w - m3.x) * m3.y;
      x[i] += y;
      if (r + 4 < p.rows4 && live[i]) v[i] = __ldcg(sc + (i * kJoinThreads * p.rows4 + r + 4) / 4);
    }
  }
#pragma unroll
  for (int i = 0; i < kKeys; ++i)
    if (live[i]) weight[s0 + i * kJoinThreads + threadIdx.x] = x[i];
}

// ------------------------------------------------------------------------------------------- host
// Tiles of 8 query rows that a CTA holds.  More than one spares reading (through L2) and decoding the cache again for the next
// rows, as far as the accumulators fit the registers: 32 sequences of 8192 tokens, 4 K/V heads, D = 128, 16 rows: 66 us with two
// tiles, 89 with one; D = 64, 32 rows: 76 us with four, 88 with two, 125 with one.  At D = 256 two tiles leave room for half the
// warps, which costs what they spare (16 rows: 92 us either way).  Where the table is so small that the rows' CTAs all
// end after one turn of their warps, a tile each: 500 tokens, 8 K/V heads, D = 128, 16 rows: 10.8 us against 12.3; D = 64, 32
// rows: 9.8 against 13.4.
int row_tiles(const fm_kv_cache* c, int n_rows) {
  const int need = (n_rows + 7) / 8;
  if (c->D == 256 || (int64_t)c->B * c->H_kv * c->max_pages * need <= kSMs * 8) return 1;
  const int most = c->D == 64 ? 4 : 2;
  return need >= most ? most : need == 3 ? 4 : need;
}

struct Layout {
  int nt, n_row_chunks, n_work, n_rows, n_rows_pad, rows4;
  int n_chunk, chunk;
  size_t units, chunk_n, listed, part_o, part_ml, whole_ml, score, live, total;
};

Layout layout_of(const fm_kv_cache* c, const fm_cache_attn_args* a) {
  Layout L;
  const size_t bh = (size_t)c->B * c->H_kv;
  L.n_rows = a->n_q * (a->H / c->H_kv);
  L.nt = row_tiles(c, L.n_rows);
  L.n_row_chunks = (L.n_rows + 8 * L.nt - 1) / (8 * L.nt);
  L.n_rows_pad = L.n_row_chunks * 8 * L.nt;
  L.rows4 = (L.n_rows + 3) / 4 * 4;
  const int64_t most = (int64_t)bh * c->max_pages;
  L.n_work = L.n_row_chunks >= kSMs ? 1 : kSMs / L.n_row_chunks;
  if (L.n_work > most) L.n_work = (int)most;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += (bytes + 255) / 256 * 256;
    return r;
  };
  L.units = take((bh + 1) * 4);
  // chunks of 32 blocks, which a CTA of the plan lists in one go (2 sequences of 34954 tokens under a window per head, 8 heads: 34.5 us
  // for the call, 45.8 with chunks of 64); larger ones where that would make more than 1024 lists, and of 64 than 8192: every CTA of
  // the main kernel adds up all their lengths; none longer than the table
  L.chunk = 32;
  while (L.chunk < kMaxChunk && L.chunk < c->max_pages &&
         bh * ((c->max_pages + L.chunk - 1) / L.chunk) > (L.chunk < 64 ? 1024 : 8192))
    L.chunk *= 2;
  if (L.chunk > c->max_pages) L.chunk = c->max_pages;
  L.n_chunk = (c->max_pages + L.chunk - 1) / L.chunk;
  L.chunk_n = take(bh * L.n_chunk * 4);
  L.listed = take(bh * L.n_chunk * L.chunk * 4);
  L.part_o = take((size_t)L.n_work * 2 * L.n_rows_pad * c->D * 4);
  L.part_ml = take((size_t)L.n_work * 2 * L.n_rows_pad * 8);
  const bool acc = a->accumulate != 0;
  L.whole_ml = take(acc ? bh * L.n_rows_pad * 8 : 0);
  L.live = take(acc ? bh * c->max_pages : 0);
  L.score = take(acc ? bh * c->max_pages * kPage * L.rows4 * 4 : 0);
  L.total = at;
  return L;
}

fm_status check_cache_attn(const fm_kv_cache* c, const fm_cache_attn_args* a) {
  const fm_status st = check_cache(c);
  if (st != FM_OK) return st;
  if (!a || a->n_q < 1 || a->H < 1 || a->H > 65535 || a->H % c->H_kv) return FM_ERR_INVALID_ARG;
  if (a->dtype != 0) return FM_ERR_UNSUPPORTED;
  if (a->H / c->H_kv > 64 || a->n_q > kMaxRows || a->n_q * (a->H / c->H_kv) > kMaxRows) return FM_ERR_UNSUPPORTED;
  if ((int64_t)c->B * a->H * a->n_q >= ((int64_t)1 << 30)) return FM_ERR_UNSUPPORTED;
  if (!(a->scale > 0.f) || a->scale > 3.0e38f) return FM_ERR_INVALID_ARG;
  if ((a->causal != 0 && a->causal != 1) || (a->accumulate != 0 && a->accumulate != 1)) return FM_ERR_INVALID_ARG;
  if (a->accumulate && !c->weight) return FM_ERR_INVALID_ARG;
  if (a->Hm == 0 ? a->n_k != 0 : ((a->Hm != 1 && a->Hm != a->H) || a->n_k < 1)) return FM_ERR_INVALID_ARG;
  return FM_OK;
}

// Tensor map over a code pool: rows of D bytes (page, head, slot), boxes of a piece's keys, 64- or 128-byte swizzle.
bool encode_pool(CUtensorMap* map, const fm_kv_cache* c, const void* base, int keys) {
  return encode_tmap_u8_rows(map, base, c->D, (uint64_t)c->n_pages * c->H_kv * kPage, keys);
}

template <int D, int NT, bool E4M3>
fm_status launch(const fm_kv_cache* c, CacheAttnParams p, cudaStream_t s) {
  using C = CacheAttnCfg<D, NT>;
  p.run_min = C::kWarps / C::kParts;
  static_assert(C::kAlloc <= 227 * 1024, "shared memory exceeds the per-CTA limit");
  CUtensorMap tk, tv;
  if (!encode_pool(&tk, c, c->k_codes, C::kKeys) || !encode_pool(&tv, c, c->v_codes, C::kKeys)) return FM_ERR_CUDA;
  if (!smem_opt_in<cache_attn_kernel<D, NT, E4M3>>(C::kAlloc)) return FM_ERR_CUDA;
  EarlyLaunch launch(s);
  cudaLaunchConfig_t& cfg = launch.cfg;
  cudaError_t e;
  if (p.masked) {
    cfg.gridDim = dim3(p.n_chunk, p.H_kv, p.B);
    cfg.blockDim = dim3(kPlanThreads);
    e = cudaLaunchKernelEx(&cfg, cache_plan_kernel, p);
    if (e != cudaSuccess) return FM_ERR_CUDA;
  }
  cfg.gridDim = dim3(p.n_work * p.n_row_chunks);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kAlloc;
  e = cudaLaunchKernelEx(&cfg, cache_attn_kernel<D, NT, E4M3>, tk, tv, p);
  if (e != cudaSuccess) return FM_ERR_CUDA;
  const int64_t bh = (int64_t)p.B * p.H_kv;
  int64_t grid = bh * p.n_rows;
  if (p.accumulate) grid += bh * ((p.max_pages * kPage + weight_slots(p.n_rows) - 1) / weight_slots(p.n_rows));
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  e = weight_slots(p.n_rows) == 512 ? cudaLaunchKernelEx(&cfg, cache_join_kernel<D, 512>, p)
                                    : cudaLaunchKernelEx(&cfg, cache_join_kernel<D, 1024>, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

template <int D, bool E4M3>
fm_status launch_nt(int nt, const fm_kv_cache* c, const CacheAttnParams& p, cudaStream_t s) {
  if constexpr (D == 64) {
    if (nt == 4) return launch<D, 4, E4M3>(c, p, s);
  }
  if constexpr (D < 256) {
    if (nt == 2) return launch<D, 2, E4M3>(c, p, s);
  }
  return launch<D, 1, E4M3>(c, p, s);
}

}  // namespace
}  // namespace fm

extern "C" {

size_t fm_cache_attn_workspace_bytes(const fm_kv_cache* cache, const fm_cache_attn_args* a) {
  return fm::check_cache_attn(cache, a) == FM_OK ? fm::layout_of(cache, a).total : 0;
}

fm_status fm_cache_attn(const fm_kv_cache* c, const fm_cache_attn_args* a, void* o, float* lse, void* ws,
                        size_t ws_bytes, fm_stream_t stream) {
  const fm_status st = fm::check_cache_attn(c, a);
  if (st != FM_OK) return st;
  bool vecs = false;
  uintptr_t low = reinterpret_cast<uintptr_t>(a->len) | reinterpret_cast<uintptr_t>(a->row) | reinterpret_cast<uintptr_t>(lse);
  for (int i = 0; i < 4; ++i) {
    vecs = vecs || a->vec[i];
    low |= reinterpret_cast<uintptr_t>(a->vec[i]);
  }
  if (!a->q || !a->len || !o || !lse || (low & 3)) return FM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(o)) & 15) return FM_ERR_INVALID_ARG;
  if (vecs && a->Hm == 0) return FM_ERR_INVALID_ARG;
  if ((a->Hm != 0 || a->causal) && !a->row) return FM_ERR_INVALID_ARG;
  const fm::Layout L = fm::layout_of(c, a);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || ws_bytes < L.total) return FM_ERR_WORKSPACE;
  uint8_t* base = static_cast<uint8_t*>(ws);
  fm::CacheAttnParams p;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.len = a->len;
  p.row = a->row;
  for (int i = 0; i < 4; ++i) p.vec[i] = a->vec[i];
  p.page_table = c->page_table;
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.pos = c->pos;
  p.weight = c->weight;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.units = reinterpret_cast<int32_t*>(base + L.units);
  p.part_o = reinterpret_cast<float*>(base + L.part_o);
  p.part_ml = reinterpret_cast<float2*>(base + L.part_ml);
  p.whole_ml = reinterpret_cast<float2*>(base + L.whole_ml);
  p.score = reinterpret_cast<float*>(base + L.score);
  p.live = base + L.live;
  p.status = fm::device_status_ptr();
  p.masked = a->Hm != 0 || a->causal;
  p.B = c->B;
  p.H = a->H;
  p.H_kv = c->H_kv;
  p.n_q = a->n_q;
  p.group = a->H / c->H_kv;
  p.n_rows = L.n_rows;
  p.n_rows_pad = L.n_rows_pad;
  p.rows4 = L.rows4;
  p.Hm = a->Hm;
  p.n_k = a->n_k;
  p.n_pages = c->n_pages;
  p.max_pages = c->max_pages;
  p.n_work = L.n_work;
  p.n_chunk = p.masked ? L.n_chunk : 1;
  p.chunk = L.chunk;
  p.chunk_n = reinterpret_cast<int32_t*>(base + L.chunk_n);
  p.listed = reinterpret_cast<int32_t*>(base + L.listed);
  p.n_row_chunks = L.n_row_chunks;
  p.causal = a->causal;
  p.accumulate = a->accumulate;
  p.scale_log2 = a->scale * fm::kLog2e;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (c->D * 2 + c->code_type) {
    case 128: return fm::launch_nt<64, false>(L.nt, c, p, s);
    case 129: return fm::launch_nt<64, true>(L.nt, c, p, s);
    case 256: return fm::launch_nt<128, false>(L.nt, c, p, s);
    case 257: return fm::launch_nt<128, true>(L.nt, c, p, s);
    case 512: return fm::launch_nt<256, false>(L.nt, c, p, s);
    default: return fm::launch_nt<256, true>(L.nt, c, p, s);
  }
}

}  // extern "C"

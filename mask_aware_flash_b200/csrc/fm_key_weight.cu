// Attention weight that each key of a prompt receives (fm_attn_key_weight), for sm_100a (tcgen05 + TMEM + TMA).
//
//   weight_j = sum over heads h of the group, rows i of  exp(scale q_i.k_j - LSE_i)   [unmasked pairs]
//
// The work is cut into (key tile of 128 keys, K/V head): its K stays in shared memory, the query tiles of its column
// lists (skip tiles never loaded) stream past it, head by head:
//   S^T = K Q^T  (tcgen05, M = 128 keys, N = 128 queries) -> one of four TMEM buffers
// so a thread holds one key: its sum stays in registers, its mask bounds too, and the interval test is a word of
// bits per 32 queries.  One CTA per SM works through a fixed share of the key tiles, longest lists first, and the
// copies and products of the next key tile start while the last one is still being summed.  Where there are too few
// key tiles for the SMs a cluster of CTAs shares each one's query tiles and adds up through distributed shared memory.
// Bound by the exponentials: per score there is one against 2 D flops of the tensor core, and for D = 128 the MUFU unit takes 1024
// clocks for a tile's 16384 (16 a clock) against 512 of the product.  8192 tokens in documents, 16 heads, D = 128: 50 us, 7888
// tiles, 0.56 of that rate at 1965 MHz; the rest are a tile's other instructions (TMEM loads, multiply-adds and additions share the issue
// slots with them: without the exponentials it takes 37 us, without the products too 25) and the ends of 1024 uneven lists.
// 2 x 3996 tokens, 16 heads, D = 64: 53 us, the same unit.  1024 tokens, 8 heads: 13 us, latency (launch, lists, one or two tiles
// a warpgroup, the cluster's sum).
// Four warpgroups take the query tiles in turn (so that one's waits hide behind the others' exponentials; three: slower); one
// warp lists the items for everybody, some key tiles ahead, one issues the TMA loads, one the MMAs.
#include "fm_common.cuh"

namespace fm {
fm_status check_attn_args(const fm_attn_args* a, const fm_mask_meta* meta, const int32_t* const vec[4]);

namespace {

constexpr int kTile = 128;
constexpr int kGroups = 4;    // warpgroups of sums
constexpr int kThreads = kGroups * 128 + 96;
constexpr int kListWarp = kGroups * 4, kLoadWarp = kListWarp + 1, kMmaWarp = kListWarp + 2;
constexpr int kSMs = 148;
constexpr int kBufs = kGroups;  // TMEM score buffers of 128 columns, one per warpgroup
constexpr int kRing = 8;      // listed items of a reader
constexpr int kReaders = kGroups + 1;  // the warpgroups of sums, the load role
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
  int n_work, n_bh, group;  // key tiles of all heads; B * H_kv; how many of those are dispatched together
  float scale_log2;
};

template <int D>
struct KeyWeightSmem {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kKBufs = D == 256 ? 1 : 2;                  // key tiles held
  static constexpr int kStages = D == 256 ? 2 : D == 128 ? 4 : 8;  // query tiles in flight
  static constexpr int kK = 0;
  static constexpr int kQ = kK + kKBufs * kTileBytes;
  static constexpr int kLse = kQ + kStages * kTileBytes;     // [warps of sums][128] -log2 LSE
  static constexpr int kSum = kLse + kGroups * 4 * kTile * 4;  // [2][warpgroups - 1][128] sums; [0][0]: of the CTA
  static constexpr int kItems = kSum + 2 * (kGroups - 1) * kTile * 4;  // int4 [readers][kRing]: listed items
  static constexpr int kBar = kItems + kReaders * kRing * 16;
  enum { K_FULL, K_EMPTY = K_FULL + kKBufs, Q_FULL = K_EMPTY + kKBufs, Q_EMPTY = Q_FULL + kStages,
         S_FULL = Q_EMPTY + kStages, S_EMPTY = S_FULL + kBufs, ITEM = S_EMPTY + kBufs, ITEM_FREE = ITEM + kReaders * kRing,
         SUM_FULL = ITEM_FREE + kReaders * kRing, SUM_EMPTY = SUM_FULL + 2, DRAIN = SUM_EMPTY + 2, kNumBars };
  static constexpr int kMisc = kBar + kNumBars * 8;  // [0] TMEM base, [1] abort flag, [2] zero
  static constexpr int kFlags = kMisc + 16;          // int [kStages]: flags of the query tiles in flight
  static constexpr int kBytes = kFlags + kStages * 4;
  static constexpr int kAlloc = kBytes + 1024;
};
// An item: .x query-tile entry (qt << 1 | partial), .y query head of the group and flags, .z key tile, .w b << 16 | hk.
// Each reader has a ring of its own: the load role gets every query tile, with kFirst and kLast of its key tile (and passes
// those on to the MMA role with the tile); a
// warpgroup of sums gets its query tiles, with kLast at its last one of the key tile, or a kLast | kEmpty item if it has none.
constexpr int kFirst = 1 << 8, kLast = 2 << 8, kEmpty = 4 << 8, kEnd = 8 << 8;

// One lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xFFFFFFFF;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}
// Has the phase of the given parity completed?  (Never waits, as try_wait may.)
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait for the two roles of one thread, which are usually ahead: their polling takes no issue slots from the sums.
__device__ __forceinline__ bool mbar_wait_idle(uint32_t bar, uint32_t parity, const volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    __nanosleep(32);
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      if (globaltimer() - t0 > kTimeoutNs) return false;
    }
  }
}

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

// Adds the weights of 32 scores to the four running sums; bit i of `masked` (only of a partial tile): query i does not see
// the key.  nl: -LSE of the queries in log2 units.  (One score an instruction: packed pairs would halve the multiply-adds and
// additions, but cost more register moves than that.)  Scale and LSE come in log2 units, rounded to fp32 first: a weight is off by a
// few 2^-24 of |s| + |LSE| and by the exponential's 2^-22 (the weights by 1.3e-7 to 1.9e-7 of their norm, an fp32 form with an exact
// exponential by 0.6e-7).
__device__ __forceinline__ void add_block(const uint32_t (&s)[32], const float* nl, float scale, bool partial, uint32_t masked,
                                          float (&acc)[4]) {
  float w[32];
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    const float4 v = *reinterpret_cast<const float4*>(nl + c);
    w[c] = ex2(fmaf(__uint_as_float(s[c]), scale, v.x));
    w[c + 1] = ex2(fmaf(__uint_as_float(s[c + 1]), scale, v.y));
    w[c + 2] = ex2(fmaf(__uint_as_float(s[c + 2]), scale, v.z));
    w[c + 3] = ex2(fmaf(__uint_as_float(s[c + 3]), scale, v.w));
  }
  if (partial) {
#pragma unroll
    for (int c = 0; c < 32; ++c) w[c] = ((masked >> c) & 1u) ? 0.f : w[c];
  }
#pragma unroll
  for (int c = 0; c < 32; ++c) acc[c & 3] += w[c];
}

// The key tile and head of piece of work `w`: groups of heads, in each the key tiles by rank (longest lists first).
__device__ __forceinline__ void work_of(const KeyWeightParams& p, int w, int& bh, int& kt) {
  const int per_group = p.group * p.T_k, grp = w / per_group, first = grp * p.group;
  const int heads = min(p.group, p.n_bh - first), in = w - grp * per_group;
  bh = first + in % heads;
  const int b = bh / p.H_kv, hk = bh % p.H_kv;
  const int64_t bhm = (int64_t)b * p.Hm + (p.Hm == 1 ? 0 : hk * p.q_per_kv);
  kt = *(p.order + bhm * p.T_k + in / heads);
}

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
  const int work0 = blockIdx.x / step, work_step = gridDim.x / step;

  const uint32_t bar0 = smem_u32(smem + S::kBar);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  const volatile int* never = reinterpret_cast<const volatile int*>(misc + 2);
  const uint32_t k_s = smem_u32(smem + S::kK), q_s = smem_u32(smem + S::kQ);
  float* lse_s = reinterpret_cast<float*>(smem + S::kLse);
  float* sum_s = reinterpret_cast<float*>(smem + S::kSum);
  int4* items = reinterpret_cast<int4*>(smem + S::kItems);
  volatile int* stage_flags = reinterpret_cast<volatile int*>(smem + S::kFlags);

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kNumBars; ++i) mbar_init(bar(i), 1);
    for (int i = 0; i < kBufs; ++i) mbar_init(bar(S::S_EMPTY + i), kTile);
    for (int i = 0; i < kGroups * kRing; ++i) mbar_init(bar(S::ITEM_FREE + i), 4);  // a warpgroup's warps
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(S::SUM_FULL + i), 4 * (kGroups - 1));
      mbar_init(bar(S::SUM_EMPTY + i), 4);
    }
    *abort_flag = 0;
    misc[2] = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  grid_wait();
  grid_launch_next();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  float sum = 0.f;    // of this thread's key (the last key tile's stays for the cluster's exchange)
  int64_t key_at = -1;  // where it goes

  if (warp == kListWarp) {
    // ------------------------------------------------------------ list role
    // The whole warp reads the lists (32 entries at a time) and hands out eight items at a time, a lane each: this warp shares
    // its scheduler with four busy ones, and one thread's instructions per item would pace the kernel.
    int qi = 0;  // query tiles so far
    int pushed[kGroups];  // items of each warpgroup's ring so far (the other two rings: qi)
#pragma unroll
    for (int i = 0; i < kGroups; ++i) pushed[i] = 0;
    bool ok = true;
    // puts `e` into place n of a reader's ring, by the calling lane
    auto put = [&](int reader, int n, const int4& e) {
      const int at = reader * kRing + n % kRing;
      ok = ok && (n < kRing || mbar_wait_idle(bar(S::ITEM_FREE + at), (n / kRing - 1) & 1, abort_flag));
      if (ok) {
        items[at] = e;
        mbar_arrive(bar(S::ITEM + at));
      }
    };
    int bh = 0, kt = 0;
    if (work0 < p.n_work) work_of(p, work0, bh, kt);
    // rounds of one key tile per CTA, every other one in reverse: the first of a round has its longest list
    for (int round = 0, w = work0; ok && w < p.n_work; ++round) {
      int bh_next = 0, kt_next = 0;
      const int w_next = (round + 1) * work_step + ((round & 1) ? work0 : work_step - 1 - work0);
      if (w_next < p.n_work) work_of(p, w_next, bh_next, kt_next);  // (in flight until it is used)
      const int b = bh / p.H_kv, hk = bh % p.H_kv;
      const int b_hk = (int)((uint32_t)b << 16 | (uint32_t)hk);
      const int64_t bhm0 = (int64_t)b * p.Hm + (p.Hm == 1 ? 0 : hk * p.q_per_kv);
      const int32_t* counts = p.col_count + bhm0 * p.T_k + kt;
      const int32_t* entries = p.col_entries + (bhm0 * p.T_k + kt) * p.T_q;
      // list lengths of the group's heads (at most 64) in two registers of the lanes, and their sum
      int n0 = 0, n1 = 0;
      if (lane < p.q_per_kv) n0 = *(counts + (p.Hm == 1 ? 0 : (int64_t)lane * p.T_k));
      if (lane + 32 < p.q_per_kv) n1 = *(counts + (p.Hm == 1 ? 0 : (int64_t)(lane + 32) * p.T_k));
      const int total = __reduce_add_sync(0xffffffffu, n0 + n1);
      const int n_items = total > rank ? (total - rank + step - 1) / step : 0;  // of this CTA
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
        if ((g - qi % kGroups + kGroups) % kGroups >= n_items) {
          if (lane == 0) put(g, pushed[g], make_int4(0, kLast | kEmpty, kt, b_hk));
          ++pushed[g];
        }
      int item = 0, skip = rank;  // items handed out; entries to pass over before the next one
      for (int hg = 0; hg < p.q_per_kv; ++hg) {
        const int n = __shfl_sync(0xffffffffu, hg < 32 ? n0 : n1, hg & 31);
        const int32_t* list = entries + (p.Hm == 1 ? 0 : (int64_t)hg * p.T_k * p.T_q);
        int at = skip;
        for (; at < n; at += 32 * step) {
          const int mine = at + lane * step < n ? *(list + at + lane * step) : 0;
          const int here = min(32, (n - at + step - 1) / step);
          for (int j0 = 0; j0 < here; j0 += 8) {
            const int n_now = min(8, here - j0), entry = __shfl_sync(0xffffffffu, mine, j0 + (lane & 7));
            if (lane < n_now) {
              const int q = qi + lane, reader = q % kGroups, i = item + lane;
              const int4 e = make_int4(entry, hg | (i == 0 ? kFirst : 0) | (i + 1 == n_items ? kLast : 0), kt, b_hk);
              put(kGroups, q, e);
              int n_before = pushed[0];
#pragma unroll
              for (int g = 1; g < kGroups; ++g) n_before = reader == g ? pushed[g] : n_before;
              put(reader, n_before + lane / kGroups, make_int4(entry, hg | (i + kGroups >= n_items ? kLast : 0), kt, b_hk));
            }
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
              const int first = (g - qi % kGroups + kGroups) % kGroups;  // this warpgroup's first item of the eight
              pushed[g] += first < n_now ? (n_now - 1 - first) / kGroups + 1 : 0;
            }
            item += n_now;
            qi += n_now;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          if (!ok) break;
        }
        // the first entry of the next head's list that is this CTA's
        skip = skip >= n ? skip - n : (step - (n - skip) % step) % step;
        if (!ok) break;
      }
      bh = bh_next;
      kt = kt_next;
      w = w_next;
      ok = __all_sync(0xffffffffu, ok);  // (the lanes leave the loop together)
    }
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < kGroups; ++i) put(i, pushed[i], make_int4(0, kEnd, 0, 0));
      put(kGroups, qi, make_int4(0, kEnd, 0, 0));
    }
    if (!ok && lane == 0) record_failure(p.status, abort_flag, 61);
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------ load role
    if (lane == 0) {
      bool ok = true;
      int qi = 0, wk = 0;
      for (int it = 0;; ++it) {
        const int slot = kGroups * kRing + it % kRing;
        if (!mbar_wait_idle(bar(S::ITEM + slot), (it / kRing) & 1, abort_flag)) {
          ok = false;
          break;
        }
        const int4 e = items[slot];
        mbar_arrive(bar(S::ITEM_FREE + slot));
        const int b = (int)((uint32_t)e.w >> 16), hk = e.w & 0xFFFF;
        const int kb = wk % S::kKBufs, st = qi % S::kStages;
        if ((e.y & kFirst) && wk >= S::kKBufs && !mbar_wait_idle(bar(S::K_EMPTY + kb), (wk / S::kKBufs - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        if (e.y & kFirst) {
          mbar_arrive_expect_tx(bar(S::K_FULL + kb), S::kTileBytes);
          for (int c = 0; c < kAtoms; ++c)
            tma_load_4d(k_s + kb * S::kTileBytes + c * 16384, &tm_k, bar(S::K_FULL + kb), c * 64, hk, e.z * kTile, b);
          ++wk;
        }
        if (qi >= S::kStages && !mbar_wait_idle(bar(S::Q_EMPTY + st), (qi / S::kStages - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        stage_flags[st] = e.y;
        if (e.y & kEnd) {  // (the MMA role's end: a stage without a tile)
          mbar_arrive(bar(S::Q_FULL + st));
          break;
        }
        mbar_arrive_expect_tx(bar(S::Q_FULL + st), S::kTileBytes);
        for (int c = 0; c < kAtoms; ++c)
          tma_load_4d(q_s + st * S::kTileBytes + c * 16384, &tm_q, bar(S::Q_FULL + st), c * 64,
                      hk * p.q_per_kv + (e.y & 255), (e.x >> 1) * kTile, b);
        ++qi;
      }
      if (!ok) record_failure(p.status, abort_flag, 64);
      // the copies in flight land before this role ends (a consumer that gave up may leave some unread)
      for (int x = max(wk - S::kKBufs, 0); x < wk; ++x) mbar_wait(bar(S::K_FULL + x % S::kKBufs), (x / S::kKBufs) & 1, never);
      // (the end's stage held the tile kStages before, which the wait for the stage has seen through)
      for (int x = max(qi - S::kStages + (ok ? 1 : 0), 0); x < qi; ++x)
        mbar_wait(bar(S::Q_FULL + x % S::kStages), (x / S::kStages) & 1, never);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------- MMA role
    // The whole warp runs it, so that descriptors and addresses stay in uniform registers; one elected lane issues.
    constexpr uint32_t kIdesc = idesc_bf16(128, 128, false, false);
    constexpr uint32_t kHi = desc_hi(1024);
    const uint32_t lo_k = desc_lo(k_s, 16), lo_q = desc_lo(q_s, 16);
    bool ok = true;
    int wk = 0;
    for (int qi = 0;; ++qi) {
      const int st = qi % S::kStages, buf = qi % kBufs, kb = wk % S::kKBufs;
      ok = __all_sync(0xffffffffu, mbar_wait(bar(S::Q_FULL + st), (qi / S::kStages) & 1, abort_flag));
      if (!ok) break;
      const int flags = __shfl_sync(0xffffffffu, stage_flags[st], 0);
      if (flags & kEnd) break;
      ok = (!(flags & kFirst) || mbar_wait(bar(S::K_FULL + kb), (wk / S::kKBufs) & 1, abort_flag)) &&
           (qi < kBufs || mbar_wait(bar(S::S_EMPTY + buf), (qi / kBufs - 1) & 1, abort_flag));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t qa = lo_q + st * (S::kTileBytes >> 4), ka = lo_k + kb * (S::kTileBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
          umma_ss_w(tmem + buf * 128, ka + off, kHi, qa + off, kHi, kIdesc, k > 0 ? 1u : 0u);
        }
        umma_commit(bar(S::S_FULL + buf));
        umma_commit(bar(S::Q_EMPTY + st));
        if (flags & kLast) umma_commit(bar(S::K_EMPTY + kb));
      }
      __syncwarp();
      if (flags & kLast) ++wk;
    }
    if (!ok && lane == 0) record_failure(p.status, abort_flag, 62);
    if (elect_one()) {
      umma_commit(bar(S::DRAIN));  // every MMA has finished before TMEM is released
      mbar_wait(bar(S::DRAIN), 0, never);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------- exponentials and sums: one key per thread
    const int wg = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    float* nl = lse_s + warp * kTile;  // (each warp has its own: no barrier between the warps for it)
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    int ends = 0;
    bool ok = true;
    // The first warpgroup adds the others' sums of a key tile when the next one ends: they have long arrived then.
    auto finish = [&](int end) {
      const int sb = end & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(bar(S::SUM_FULL + sb), (end >> 1) & 1, abort_flag)) && ok;
      const float* others = sum_s + sb * (kGroups - 1) * kTile;
#pragma unroll
      for (int g = 0; g < kGroups - 1; ++g) sum += others[g * kTile + r];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(S::SUM_EMPTY + sb));
      if (step == 1 && key_at >= 0) p.weight[key_at] = p.accumulate ? p.weight[key_at] + sum : sum;
    };
    int mine = 0;  // query tiles so far
    // LSE of four rows of an item's query tile (lane, lane + 32, ..); -inf past n_q (and for rows that see no key): their p is 0
    auto load_lse = [&](const int4& e) {
      const int row = (e.x >> 1) * kTile + lane, h = (e.w & 0xFFFF) * p.q_per_kv + (e.y & 255);
      const float* src = p.lse + ((int64_t)((uint32_t)e.w >> 16) * p.H + h) * p.n_q + row;
      const int n = e.y & (kEmpty | kEnd) ? 0 : p.n_q - row;
      return make_float4(n > 0 ? *src : kNegInf, n > 32 ? *(src + 32) : kNegInf, n > 64 ? *(src + 64) : kNegInf,
                         n > 96 ? *(src + 96) : kNegInf);
    };
    // bounds of this thread's key for an item: lts, lte, uts, ute
    auto load_bounds = [&](const int4& e) {
      const int b = (int)((uint32_t)e.w >> 16), key = e.z * kTile + r;
      const int hm = p.Hm == 1 ? 0 : (e.w & 0xFFFF) * p.q_per_kv + (e.y & 255);
      const int64_t at = ((int64_t)b * p.Hm + hm) * p.n_k + key;
      const bool in = key < p.n_k && !(e.y & (kEmpty | kEnd));
      int4 v;
      v.x = in && p.vec[0] ? *(p.vec[0] + at) : p.n_q;
      v.y = in && p.vec[1] ? *(p.vec[1] + at) : p.n_q;
      v.z = in && p.vec[2] ? *(p.vec[2] + at) : 0;
      v.w = in && p.vec[3] ? *(p.vec[3] + at) : 0;
      return v;
    };
    int4 e_next, bounds_next;
    float4 x_next;
    bool have_next = false;
    for (int it = 0; ok; ++it) {
      auto take = [&](int i) {  // reads a listed item and gives its place back
        const int slot = wg * kRing + i % kRing;
        const int4 v = items[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::ITEM_FREE + slot));
        return v;
      };
      int4 e, bounds;
      float4 x;
      if (have_next) {
        e = e_next;
        x = x_next;
        bounds = bounds_next;
      } else {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(S::ITEM + wg * kRing + it % kRing), (it / kRing) & 1, abort_flag));
        if (!ok) break;
        e = take(it);
        x = load_lse(e);
        bounds = load_bounds(e);
      }
      if (e.y & kEnd) break;
      const int b = (int)((uint32_t)e.w >> 16), hk = e.w & 0xFFFF, key = e.z * kTile + r;
      auto log2_neg = [](float v) { return v == kNegInf ? kNegInf : -v * 1.4426950408889634f; };
      __syncwarp();  // (the last item's have been read)
      nl[lane] = log2_neg(x.x);
      nl[lane + 32] = log2_neg(x.y);
      nl[lane + 64] = log2_neg(x.z);
      nl[lane + 96] = log2_neg(x.w);
      __syncwarp();
      // the next item, if it is listed already: its LSE and bounds are in flight during this one's exponentials
      have_next = __all_sync(0xffffffffu, mbar_test(bar(S::ITEM + wg * kRing + (it + 1) % kRing), ((it + 1) / kRing) & 1));
      if (have_next) {
        e_next = take(it + 1);
        x_next = load_lse(e_next);
        // (the bounds stay while the key tile and the mask do)
        const bool same = e_next.z == e.z && e_next.w == e.w && !(e.y & kEmpty) && (p.Hm == 1 || ((e_next.y ^ e.y) & 255) == 0);
        bounds_next = bounds;
        if (!same) bounds_next = load_bounds(e_next);
      }
      if (!(e.y & kEmpty)) {
        const int q0 = (e.x >> 1) * kTile;
        const bool ragged = q0 + kTile > p.n_q, partial = (e.x & 1) || ragged;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(S::S_FULL + wg), mine & 1, abort_flag));
        if (!ok) break;
        auto mask_word = [&](int jb) {  // bit i: query q0 + 32 jb + i does not see this key
          const int base = q0 + jb * 32;
          const uint32_t mw = interval_bits32(bounds.x, bounds.y, base) | interval_bits32(bounds.z, bounds.w, base);
          return !ragged || base + 32 <= p.n_q ? mw : mw | (base >= p.n_q ? 0xFFFFFFFFu : 0xFFFFFFFFu << (p.n_q - base));
        };
        tc_fence_after();
        // (not unrolled: the code of one block stays in the instruction cache)
        const uint32_t t0 = tmem + wg * 128 + lane_addr;
#pragma unroll 1
        for (int jb = 0; jb < 4; ++jb) {
          uint32_t s[32];
          tmem_ld32(t0 + jb * 32, s);
          if (jb == 3) {
            tc_fence_before();
            mbar_arrive(bar(S::S_EMPTY + wg));
          }
          add_block(s, nl + jb * 32, p.scale_log2, partial, partial ? mask_word(jb) : 0u, acc);
        }
        ++mine;
      }
      if (e.y & kLast) {  // the key tile is done: the other warpgroups' sums go to the first
        const float mine_sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        if (wg > 0) {
          const int sb = ends & 1, turn = ends >> 1;
          if (turn > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(S::SUM_EMPTY + sb), (turn - 1) & 1, abort_flag));
          sum_s[(sb * (kGroups - 1) + wg - 1) * kTile + r] = mine_sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(S::SUM_FULL + sb));
        } else {
          if (ends > 0) finish(ends - 1);
          sum = mine_sum;
          key_at = key < p.n_k ? ((int64_t)b * p.H_kv + hk) * p.weight_stride + key : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[u] = 0.f;
        ++ends;
      }
    }
    if (wg == 0 && ends > 0 && ok) finish(ends - 1);
    if (!ok && lane == 0) record_failure(p.status, abort_flag, 63);
  }

  __syncthreads();  // (also: the MMA warp has drained)
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (step > 1) {  // one key tile per cluster
    if (warp < 4) sum_s[threadIdx.x] = sum;
    cluster_sync_all();
    if (rank == 0 && warp < 4 && key_at >= 0) {
      for (int c = 1; c < step; ++c) sum += ld_cluster_f32(smem_u32(sum_s + threadIdx.x), c);
      p.weight[key_at] = p.accumulate ? p.weight[key_at] + sum : sum;
    }
    cluster_sync_all();  // no CTA leaves while its sums are read
  }
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
  // A key tile's query tiles are shared by a cluster of CTAs where there are too few key tiles for the SMs: the largest of
  // which all run at once.  (1024 tokens, 2 K/V heads: 16 clusters of 4 CTAs 12.9 us, of 8, of which 15 run at once, 16.9, a CTA
  // each 29.3; 512 tokens: 9.1 with 8, 10.4 with 4, 17.1 with one.)
  int cluster = 8;
  while (cluster > 1 && p.n_work > clusters_at_once<key_weight_kernel<D>>(cluster, kThreads, S::kAlloc)) cluster /= 2;
  EarlyLaunch launch(stream, cluster);
  cudaLaunchConfig_t& cfg = launch.cfg;
  cfg.gridDim = dim3((unsigned)(cluster > 1 ? p.n_work * cluster : p.n_work < kSMs ? p.n_work : kSMs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kAlloc;
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
  if ((int64_t)args.B * args.H * ((args.n_k + 127) / 128) >= ((int64_t)1 << 31)) return FM_ERR_UNSUPPORTED;
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
  p.n_bh = args.B * H_kv;
  p.n_work = p.T_k * p.n_bh;
  p.group = fm::dispatch_group(p.n_bh, 2.0 * args.n_q * args.D * p.q_per_kv);
  p.scale_log2 = args.scale * 1.4426950408889634f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (args.D == 64) return fm::launch_key_weight<64>(&args, p, H_kv, s);
  if (args.D == 128) return fm::launch_key_weight<128>(&args, p, H_kv, s);
  return fm::launch_key_weight<256>(&args, p, H_kv, s);
}

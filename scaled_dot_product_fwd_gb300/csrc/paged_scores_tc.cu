// paged_scores_tc.cu — accumulated attention weights over the paged KV cache
// on the 5th-generation tensor cores (fp16/bf16, head_dim 64/128):
//     scores[key] += sum over rows of 2^(S^T[key, row] * scale*log2e - lse2[row])
// with S^T = K Q^T, 128 keys on the lanes of TMEM and a chunk of query rows
// (tokens x heads of the kv head) on its columns.  A thread owns a key (two
// threads do, one for the even steps and one for the odd: their waits and
// their arithmetic then alternate on an SM sub-partition): it
// reads its row of S^T, subtracts the rows' log-sum-exp (shared memory, the
// same address for a whole warp), and adds the exponentials up in registers
// over all chunks, so no value crosses lanes and nothing is added atomically.
//
// A unit is 256 keys (two TMEM tiles, one a warpgroup): each query chunk that
// is brought in meets both, which halves the query traffic out of L2.  Its
// steps are the chunks of w tokens x gu heads that see a key of it, and the
// work is divided among the CTAs as paged.cuh describes.  The K tiles of one
// unit and four query chunks are in shared memory (head_dim 128); S^T is
// double-buffered, so the products of a step run while the exponentials of
// the one before do.  Chunks (8192 tokens over themselves, 32 heads over 8,
// head_dim 128: 213 us, 1290 TFLOP/s): bound by the issue and latency of the
// exponentials' loop; its floors are 1024 clk of products a step and about
// 1100 of exponentials, and it takes about 1800.  Few rows a sequence (single
// tokens): the chunk has R = 16, 32 or 64 columns and K streams once, bound by
// HBM (8 x 32768 keys: 102 us, 5.4 TB/s).
//
// Rows that do not exist (past the sequence's tokens, another head's) take no
// part: their limit is 0, and a chunk that holds one, or a key that some row
// does not see, takes the path with a comparison for every column.  Keys past
// the length produce sums that are never written.
#include "paged.cuh"
#include "prefill_tc.cuh"

namespace gb300 {
namespace paged {
namespace {

constexpr int kUnitKeys = 256;
constexpr int kLgUnit = 8;
constexpr int kNL = 4;  // slots of the rows' log-sum-exp

template <int D, int R>
struct ScCfg {
  static constexpr int CB = D / 64;
  static constexpr int TILE = 128 * D * 2;  // a key tile
  static constexpr int QTILE = R * D * 2;   // a query chunk
  // units whose keys are in flight, and query chunks
  static constexpr int NK = (R <= 32 ? 3 : R == 64 ? 2 : 1) * (D == 64 ? 2 : 1);
  static constexpr int NQS = R == 128 && D == 64 ? 6 : R == 32 ? 2 : 4;
  static constexpr int Q_OFF = NK * 2 * TILE;
  static constexpr int BAR_OFF = Q_OFF + NQS * QTILE;
  // k_full[NK], k_empty[NK], q_full[NQS], q_empty[NQS], s_full[2 tiles][2],
  // l_full[kNL], l_empty[kNL], drain
  static constexpr int NBARS = 2 * NK + 2 * NQS + 4 + 2 * kNL + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  // warps of the exponentials: four for each key tile, or four for each tile
  // and parity of the step
  static constexpr int GROUPS = R >= 64 ? 2 : 1;
  static constexpr int EW = 8 * GROUPS;
  static constexpr int WARPS = EW + 4;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int SHARE_OFF = (MISC_OFF + 16 + 15) / 16 * 16;
  static constexpr int SCRATCH_OFF = SHARE_OFF + static_cast<int>(sizeof(Share));
  static constexpr int MIN_OFF = SCRATCH_OFF + (WARPS + 1) * 8;  // int[kNL]
  static constexpr int WALK_OFF = (MIN_OFF + kNL * 4 + 15) / 16 * 16;
  static constexpr int UNIT_OFF = WALK_OFF + WARPS * static_cast<int>(sizeof(Walk<ScoreUnits>));
  // per slot: -lse2[R], then the rows' limits [R]
  static constexpr int LSE_OFF =
      (UNIT_OFF + WARPS * static_cast<int>(sizeof(Unit)) + 15) / 16 * 16;
  static constexpr int SUM_OFF = LSE_OFF + kNL * R * 8;  // float[2][128]
  static constexpr int SMEM = SUM_OFF + 2 * 128 * 4 + 1024;
  static_assert(SMEM <= 232448, "shared memory budget");
};

// N columns (16 or 32) of this thread's row of S^T.
template <int N>
__device__ __forceinline__ void load_cols(uint32_t t0, uint32_t (&s)[N]) {
  if constexpr (N == 32) {
    tmem_ld32_sync(t0, s);
  } else {
    static_assert(N == 16, "columns of a chunk");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3]), "=r"(s[4]), "=r"(s[5]), "=r"(s[6]),
          "=r"(s[7]), "=r"(s[8]), "=r"(s[9]), "=r"(s[10]), "=r"(s[11]), "=r"(s[12]),
          "=r"(s[13]), "=r"(s[14]), "=r"(s[15])
        : "r"(t0)
        : "memory");
  }
}

// Sum over N columns of 2^(s * sl2 + nl), with kMasked of those whose limit
// is above `key`.
template <int N, bool kMasked>
__device__ __forceinline__ float weights(const uint32_t (&s)[N], float sl2, const float* nl,
                                         const int* lim, int key) {
  const uint64_t SL = f2_pack(sl2, sl2);
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 l4 = *reinterpret_cast<const float4*>(nl + i);
    const uint64_t x0 = f2_fma(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), SL,
                               f2_pack(l4.x, l4.y));
    const uint64_t x1 = f2_fma(f2_pack(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), SL,
                               f2_pack(l4.z, l4.w));
    float e0, e1, e2, e3;
    f2_unpack(x0, e0, e1);
    f2_unpack(x1, e2, e3);
    e0 = ex2(e0);
    e1 = ex2(e1);
    e2 = ex2(e2);
    e3 = ex2(e3);
    if constexpr (kMasked) {
      const int4 m4 = *reinterpret_cast<const int4*>(lim + i);
      e0 = key < m4.x ? e0 : 0.f;
      e1 = key < m4.y ? e1 : 0.f;
      e2 = key < m4.z ? e2 : 0.f;
      e3 = key < m4.w ? e3 : 0.f;
    }
    acc[(i >> 1) & 3] = f2_add(acc[(i >> 1) & 3], f2_pack(e0, e1));
    acc[((i >> 1) + 1) & 3] = f2_add(acc[((i >> 1) + 1) & 3], f2_pack(e2, e3));
  }
  const uint64_t x = f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3]));
  float x0, x1;
  f2_unpack(x, x0, x1);
  return x0 + x1;
}

__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t nthreads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}
// named barriers: kBarS + 2 t + buffer: the warps of key tile t have read
// that buffer of S^T; kBarQ: stage helper with the MMA warp
constexpr uint32_t kBarS = 1;
constexpr uint32_t kBarQ = 5;
constexpr uint32_t kBarC = 6;  // + t: the two groups of key tile t

template <int D, bool BF16, int R>
__global__ void __launch_bounds__(ScCfg<D, R>::THREADS, 1)
    paged_scores_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                           const __grid_constant__ CUtensorMap tmK, const Args a,
                           const int lg_box, const CacheBlocks kb) {
  using C = ScCfg<D, R>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* sK = smem;
  uint8_t* sQ = smem + C::Q_OFF;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* k_empty = k_full + C::NK;
  uint64_t* q_full = k_empty + C::NK;
  uint64_t* q_empty = q_full + C::NQS;
  uint64_t* s_full = q_empty + C::NQS;  // [tile][buffer]
  uint64_t* l_full = s_full + 4;
  uint64_t* l_empty = l_full + kNL;
  uint64_t* drain = l_empty + kNL;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  Share* sh = reinterpret_cast<Share*>(smem + C::SHARE_OFF);
  int* sMin = reinterpret_cast<int*>(smem + C::MIN_OFF);
  float* sLse = reinterpret_cast<float*>(smem + C::LSE_OFF);
  constexpr int kLoad = C::EW, kMma = kLoad + 1, kHelp = kLoad + 2, kLse = kLoad + 3;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::NQS; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&s_full[i], 1);
    for (int i = 0; i < kNL; ++i) {
      mbar_init(&l_full[i], 32);
      mbar_init(&l_empty[i], 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == kLoad && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
  }
  // rows of a chunk that no box writes stay zero (finite scores)
  if (a.gu * a.w < R) {
    for (int i = threadIdx.x; i < C::NQS * C::QTILE / 16; i += C::THREADS)
      reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_shared();
  }
  tc_fence_before();
  griddep_launch_dependents();
  griddep_wait();
  const ScoreUnits units{a.by_w, kLgUnit, a.causal, a.nsub, 4};
  plan_share<C::THREADS>(a, units, a.Hkv, 2,
                         reinterpret_cast<long long*>(smem + C::SCRATCH_OFF), sh);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{a.wait_ns, abort_flag, a.status};
  using W = Walk<ScoreUnits>;
  W* walk = reinterpret_cast<W*>(smem + C::WALK_OFF) + warp;
  Unit* unit = reinterpret_cast<Unit*>(smem + C::UNIT_OFF) + warp;
  if (lane == 0) *walk = W(*sh);
  auto next = [&]() {
    __syncwarp();
    bool more = false;
    if (lane == 0) more = walk->next(a, units, *sh, a.Hkv, unit);
    return __shfl_sync(0xffffffffu, more ? 1 : 0, 0) != 0;
  };
  // the two key tiles of unit j, or one where the length ends in the first
  auto tiles_of = [&](const Unit& u) { return u.s.nk - u.j * kUnitKeys > 128 ? 2 : 1; };
  int k_fills = 0, q_fills = 0;  // producer: fills of the two rings so far

  if (warp == kLoad) {
    // ------------------------------------------------------------ producer
    const int nbox = 128 >> lg_box;
    const uint32_t box_bytes = (C::CB * 128u) << lg_box;
    bool ok = true;
    int ku = 0, g = 0;  // units, steps
    while (ok && next()) {
      const Unit u = *unit;
      const int first = units.first(u.s, u.j);
      // this lane's box: of tile lane / nbox
      const int key = u.j * kUnitKeys + (lane << lg_box);
      int page = -1, row = 0;
      if (lane < 2 * nbox && key < u.s.nk) {
        page = page_of(a, u.b, key);
        row = key - a.by_page.div(key) * a.page_size;
        if (page < 0) page = -2;  // the table names none: reads as zero
      }
      const int boxes = min(2 * nbox, (u.s.nk - u.j * kUnitKeys + (1 << lg_box) - 1) >> lg_box);
      const int ks = ku % C::NK;
      if (lane == 0) {
        if (ku >= C::NK) ok = mbar_wait(&k_empty[ks], ((ku / C::NK) - 1) & 1, wc);
        if (ok) mbar_arrive_expect_tx(&k_full[ks], box_bytes * boxes);
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      if (page != -1)
        load_box(sK + ks * 2 * C::TILE + lane * box_bytes, &tmK, &k_full[ks], row,
                 page < 0 ? kb.blocks : page * kb.page_mul + u.h * kb.head_mul);
      ++ku;
      k_fills = ku;
      if (lane == 0) {
        for (int t = u.s0; t < u.s1 && ok; ++t, ++g) {
          const int qs = g % C::NQS;
          if (g >= C::NQS) ok = mbar_wait(&q_empty[qs], ((g / C::NQS) - 1) & 1, wc);
          if (!ok) break;
          mbar_arrive_expect_tx(&q_full[qs], static_cast<uint32_t>(C::CB * a.gu * a.w * 128));
          const int tok = u.s.q0 + (first + a.by_nsub.div(t)) * a.w;
          const int head = u.h * a.G + (a.by_nsub.mod(t)) * a.gu;
          for (int cb = 0; cb < C::CB; ++cb)
            tma_load_4d(sQ + qs * C::QTILE + cb * R * 128, &tmQ, &q_full[qs], cb * 64, head,
                        tok, 0);
          q_fills = g + 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    }
  } else if (warp == kMma) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t idS = idesc_f16(BF16, 128, R, false, false);
    // K tiles: 8-key groups CB * 1024 bytes apart, 64-column blocks 1024
    const uint64_t k_desc = sdesc(smem_addr(sK), 16, C::CB * 1024, kSwizzle128B);
    const uint64_t q_desc = sdesc(smem_addr(sQ), 16, 1024, kSwizzle128B);
    const uint32_t k_hi = static_cast<uint32_t>(k_desc >> 32);
    const uint32_t q_hi = static_cast<uint32_t>(q_desc >> 32);
    const uint32_t k_lo = static_cast<uint32_t>(k_desc);
    const uint32_t q_lo = static_cast<uint32_t>(q_desc);
    auto desc = [](uint32_t hi, uint32_t lo) { return (static_cast<uint64_t>(hi) << 32) | lo; };
    int ku = 0, g = 0;
    int uses[4] = {0, 0, 0, 0};  // of each (tile, buffer)
    while (next()) {
      const int nt = tiles_of(*unit), n = unit->s1 - unit->s0;
      for (int t = 0; t < n; ++t, ++g) {
        named_bar_sync(kBarQ, 64);  // the chunk, its constants and the unit's keys have landed
        tc_fence_after();
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          if (kt >= nt) continue;
          const int buf = 2 * kt + (g & 1);
          // the buffer's previous scores have been read
          if ((g & 1) ? uses[2 * kt + 1]++ : uses[2 * kt]++) {
            named_bar_sync(kBarS + buf, 160);
            tc_fence_after();
          }
          const uint32_t kd = k_lo + static_cast<uint32_t>((((ku % C::NK) * 2 + kt) * C::TILE) >> 4);
          const uint32_t qd = q_lo + static_cast<uint32_t>(((g % C::NQS) * C::QTILE) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ko = ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4;
            const uint32_t qo = ((kk >> 2) * (R * 128) + (kk & 3) * 32) >> 4;
            mma_f16_ss_elect(tmem + buf * 128, desc(k_hi, kd + ko), desc(q_hi, qd + qo), idS,
                             kk > 0 ? 1u : 0u, 1u);
          }
          mma_commit_elect(&s_full[buf], 1u);
        }
        mma_commit_elect(&q_empty[g % C::NQS], 1u);
      }
      mma_commit_elect(&k_empty[ku % C::NK], 1u);
      ++ku;
    }
    // meet the last readers of each buffer
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (uses[i] > 0) named_bar_sync(kBarS + i, 160);
    mma_commit_elect(drain, 1u);
    if (lane == 0) drain_wait(drain, 0, kDrainNs);
    __syncwarp();
  } else if (warp == kHelp) {
    // -------------------------------------------------------- stage helper
    bool ok = true;
    int ku = 0, g = 0;
    while (next()) {
      ok = ok && mbar_wait(&k_full[ku % C::NK], static_cast<uint32_t>((ku / C::NK) & 1), wc);
      const int n = unit->s1 - unit->s0;
      for (int t = 0; t < n; ++t, ++g) {
        ok = ok && mbar_wait(&q_full[g % C::NQS], static_cast<uint32_t>((g / C::NQS) & 1), wc);
        ok = ok && mbar_wait(&l_full[g % kNL], static_cast<uint32_t>((g / kNL) & 1), wc);
        __syncwarp();
        named_bar_sync(kBarQ, 64);
      }
      ++ku;
    }
  } else if (warp == kLse) {
    // ------------------------------------- the rows' log-sum-exp and limits
    // this lane's rows of a chunk: token and head (token past every
    // sequence's for rows that no chunk has)
    constexpr int N = (R + 31) / 32;
    int row_t[N], row_e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = i * 32 + lane;
      row_t[i] = a.by_gu.div(r);
      row_e[i] = a.by_gu.mod(r);
    }
    bool ok = true;
    int g = 0;
    while (ok && next()) {
      const Unit u = *unit;
      const int first = units.first(u.s, u.j);
      // the next step's values are on their way while this one's are stored
      float nxt[N];
      auto fetch = [&](int t) {
        const int tok0 = (first + a.by_nsub.div(t)) * a.w, e0 = a.by_nsub.mod(t) * a.gu;
        const float* p =
            a.lse + static_cast<size_t>(u.s.q0 + tok0) * a.Hq + u.h * a.G + e0;
        const int nt = t < u.s1 ? min(a.w, u.s.nq - tok0) : 0, ne = a.G - e0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          nxt[i] = 0.f;
          if (row_t[i] < nt && row_e[i] < ne) nxt[i] = p[row_t[i] * a.Hq + row_e[i]];
        }
      };
      fetch(u.s0);
      for (int t = u.s0; t < u.s1 && ok; ++t, ++g) {
        const int slot = g % kNL;
        float* dst = sLse + slot * 2 * R;
        const int tok0 = (first + a.by_nsub.div(t)) * a.w;
        const int nt = min(a.w, u.s.nq - tok0), ne = a.G - a.by_nsub.mod(t) * a.gu;
        const int lim0 = u.s.off + tok0 + 1;
        float v[N];
        int lim[N];
        int mn = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const bool there = row_t[i] < nt && row_e[i] < ne;
          const float x = nxt[i] * kLog2e;
          // (a row that saw nothing adds nothing)
          v[i] = there && x != -INFINITY ? -x : -INFINITY;
          lim[i] = !there ? 0 : a.causal ? min(u.s.nk, lim0 + row_t[i]) : u.s.nk;
          if (row_t[i] < a.w) mn = min(mn, lim[i]);
        }
        fetch(t + 1);
        mn = __reduce_min_sync(0xffffffffu, mn);
        if (g >= kNL) ok = __all_sync(0xffffffffu, mbar_wait(&l_empty[slot], ((g / kNL) - 1) & 1, wc));
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int r = i * 32 + lane;
          if (r < R) {
            dst[r] = v[i];
            reinterpret_cast<int*>(dst)[R + r] = lim[i];
          }
        }
        if (lane == 0) sMin[slot] = mn;
        mbar_arrive(&l_full[slot]);
      }
    }
  } else {
    // -------------------------------------------------------- exponentials
    const int kt = warp / (C::EW / 2);
    const int grp = (warp >> 2) % C::GROUPS;  // takes the steps of its parity
    const int r = (warp & 3) * 32 + lane;
    float* sSum = reinterpret_cast<float*>(smem + C::SUM_OFF) + kt * 128;
    const uint32_t t0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    bool ok = true;
    int g = 0;
    int ph[2] = {0, 0};  // phases of s_full consumed, per buffer
    bool began = false;
    while (next()) {
      const int key = unit->j * kUnitKeys + kt * 128 + r;
      const int n = unit->s1 - unit->s0;
      const bool mine = kt < tiles_of(*unit);
      const bool whole = unit->whole();
      float* dst = a.scores + unit->b * a.ss[0] + unit->h * a.ss[1] + key;
      const bool live = mine && key < unit->s.nk && key < a.score_len;
      float old = 0.f;
      if (live && whole && grp == 0) old = *dst;  // on its way while the scores are computed
      float sum = 0.f;
      for (int t = 0; t < n; ++t, ++g) {
        if (C::GROUPS == 2 && (g & 1) != grp) continue;
        const int slot = g % kNL;
        // (a warp without a tile waits for the constants all the same: its
        // arrival below counts for this use of the slot)
        if (!mine)
          ok = ok && mbar_wait(&l_full[slot], static_cast<uint32_t>((g / kNL) & 1), wc);
        if (mine) {
          const int buf = 2 * kt + (g & 1);
          const int p = (g & 1) ? ph[1]++ : ph[0]++;
          ok = __all_sync(0xffffffffu, ok && mbar_wait(&s_full[buf], static_cast<uint32_t>(p & 1), wc));
          // 32 columns at a time, so that registers are left to have the
          // rows' constants (which landed before s_full) on their way
          constexpr int kPart = R < 32 ? R : 32;
          const float* nl = sLse + slot * 2 * R;
          const int* lim = reinterpret_cast<const int*>(nl) + R;
          const bool inside = __all_sync(0xffffffffu, key < sMin[slot]);
#pragma unroll
          for (int c = 0; c < R; c += kPart) {
            uint32_t s[kPart];
            if (ok) {
              tc_fence_after();
              __syncwarp();
              load_cols<kPart>(t0 + buf * 128 + c, s);
              tc_fence_before();
            }
            if (c + kPart == R) named_bar_arrive(kBarS + buf, 160);
            if (ok) sum += inside ? weights<kPart, false>(s, a.sl2, nl + c, lim + c, key)
                                  : weights<kPart, true>(s, a.sl2, nl + c, lim + c, key);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_empty[slot]);
      }
      if (!whole && unit->s0 == 0 && threadIdx.x == 0) {
        int* d = a.desc + blockIdx.x * kDesc;
        d[0] = pieces_of(*unit, *sh);
        d[1] = unit->b;
        d[2] = unit->h;
        d[3] = unit->j;
        d[6] = unit->s.nk;
        began = true;
      }
      if constexpr (C::GROUPS == 2) {
        // the groups' sums meet (a unit's end; `mine` is the same for both)
        if (mine) {
          if (grp == 1) sSum[r] = sum;
          named_bar_sync(kBarC + kt, 256);
          if (grp == 0) sum += sSum[r];
          named_bar_sync(kBarC + kt, 256);
        }
      }
      if (ok && live && grp == 0) {
        if (whole)
          *dst = old + sum;
        else
          a.ws[static_cast<size_t>(blockIdx.x * 2 + unit->slot()) * kUnitKeys + kt * 128 + r] =
              sum;
      }
    }
    if (threadIdx.x == 0 && !began) a.desc[blockIdx.x * kDesc] = 0;
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (warp == kLoad && lane == 0 && *abort_flag) {
    // a role gave up: every copy the producer issued lands before the CTA exits
    for (int i = max(0, k_fills - C::NK); i < k_fills; ++i)
      drain_wait(&k_full[i % C::NK], static_cast<uint32_t>((i / C::NK) & 1), kDrainNs);
    for (int i = max(0, q_fills - C::NQS); i < q_fills; ++i)
      drain_wait(&q_full[i % C::NQS], static_cast<uint32_t>((i / C::NQS) & 1), kDrainNs);
  }
}

template <int D, bool BF16, int R>
sdpa_status_t launch_sc(const Args& a, const CUtensorMap& tq, const CUtensorMap& tk,
                        int lg_box, const CacheBlocks& kb, const LaunchEnv& env) {
  using C = ScCfg<D, R>;
  auto kern = paged_scores_tc_kernel<D, BF16, R>;
  if (!allow_smem<paged_scores_tc_kernel<D, BF16, R>>(C::SMEM)) return SDPA_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.nctas));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = env.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, tq, tk, a, lg_box, kb) != cudaSuccess) return SDPA_ERR_CUDA;
  return launch_paged_scores_merge(a, kUnitKeys, env.stream);
}

template <int D>
sdpa_status_t launch_scores(Args& a, int dtype, const LaunchEnv& env) {
  // Columns of a chunk: the fewest that hold a sequence's rows (a
  // column costs an exponential whether its row exists or not: 10 x 34 tokens
  // over up to 24727 keys, one head a kv head, took 106 us with 128 columns
  // and 67 with 64).
  int cols = 16;
  while (cols < 128 && (a.G > cols || call_rows(a) > cols)) cols *= 2;
  fit_rows(a, cols);
  const bool bf16 = dtype == SDPA_BF16;
  const CUtensorMapDataType dt =
      bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int lg_box = box_log2(a.page_size);
  CacheBlocks kb;
  long long ku;
  if (!cache_blocks(a.ks, a.num_pages, a.Hkv, &kb, &ku))
    return SDPA_ERR_UNSUPPORTED;  // (the caller has checked)
  CUtensorMap tq, tk;
  // a stride of a dimension of one element is never followed: any valid one
  auto st = [](long long s, long long n) { return static_cast<uint64_t>(n > 1 ? s : D); };
  if (!encode_tiled_4d_box(&tq, dt, a.q, D, a.Hq, a.T, 1, 2, 64, static_cast<uint32_t>(a.gu),
                           static_cast<uint32_t>(a.w), st(a.qs[1], a.Hq), st(a.qs[0], a.T), D) ||
      !encode_row_blocks(&tk, dt, a.k, D / 64, a.page_size, kb.blocks, 1 << lg_box,
                         st(a.ks[2], a.page_size), ku))
    return SDPA_ERR_CUDA;
#define GB300_SCORES(R)                                                 \
  (bf16 ? launch_sc<D, true, R>(a, tq, tk, lg_box, kb, env)             \
        : launch_sc<D, false, R>(a, tq, tk, lg_box, kb, env))
  switch (cols) {
    case 16: return GB300_SCORES(16);
    case 32: return GB300_SCORES(32);
    case 64: return GB300_SCORES(64);
    default: return GB300_SCORES(128);
  }
#undef GB300_SCORES
}

}  // namespace
}  // namespace paged

sdpa_status_t launch_paged_scores_tc(paged::Args a, int head_dim, int dtype,
                                     const LaunchEnv& env) {
  return head_dim == 64 ? paged::launch_scores<64>(a, dtype, env)
                        : paged::launch_scores<128>(a, dtype, env);
}

}  // namespace gb300

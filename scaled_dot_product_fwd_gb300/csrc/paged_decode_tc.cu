// paged_decode_tc.cu — attention over the paged KV cache where a sequence has
// few query rows (single tokens: the G heads of a kv head): fp16/bf16,
// head_dim 64/128, up to NR = 8 or 16 rows of (token, head) a tile, on the
// 5th-generation tensor cores.
//
// The rows are the narrow side of both products, as in the contiguous decode
// (decode_tc128.cu):
//     S^T  = K Q^T     M = 128 keys,       N = 16 rows, K = D
//     O^T += V^T P^T   M = 128 head dims,  N = 16 rows, K = 128 keys
// so each of 128 threads has one key of a tile and NR exponentials, instead
// of one warp having 128 for each of a few rows (64 x 4096 keys, 16 heads over
// 2, head_dim 64: 32.8 us; with rows on the lanes 36.8).
//
// A CTA walks its share of the line of key tiles (paged.cuh), so the running
// form of the softmax is needed: every thread holds the rows' reference
// maxima, and a tile only asks, by one barrier with a vote, whether any score
// passes its row's reference by more than 8 (log2 units; P stays <= 2^8).
// If so the tile's maxima are taken across the CTA and O^T (16 columns of
// TMEM) is rescaled; after a row's first tile that is rare.  The sums stay
// per thread until the unit ends.
//
// P enters the value product rounded to the cache's type, for the reason and
// at the cost that paged_tc.cuh gives; the sums take it unrounded.
//
// Bound by HBM (8 x 32768 keys, head_dim 128, bf16: 164-170 us, 6.3-6.5
// TB/s): six 32 KB K/V slots in flight (twelve of 16 KB at head_dim 64), S
// three tiles ahead of P V; TMEM holds eight S^T tiles and O^T.
#include "paged.cuh"
#include "prefill_tc.cuh"

namespace gb300 {
namespace paged {
namespace {

template <int D>
struct DecCfg {
  static constexpr int CB = D / 64;
  static constexpr int TILE = 128 * D * 2;
  static constexpr int NS = D == 64 ? 12 : 6;  // ring slots (K or V tile)
  static constexpr int LA = 3;                 // key tiles that S runs ahead
  static constexpr int NSB = 8;                // S^T tiles in TMEM
  static constexpr int NP = 4;                 // P^T tiles
  static constexpr int QT = 16 * D * 2;        // query tile (two: this unit's, the next one's)
  static constexpr int PT = 16 * 256;          // P^T tile: 2 chunks of 16 rows x 64 keys
  static constexpr int Q_OFF = NS * TILE;
  static constexpr int P_OFF = Q_OFF + 2 * QT;
  static constexpr int BAR_OFF = P_OFF + NP * PT;
  // q_full[2], q_empty[2], full[NS], empty[NS], s_full[NSB], p_ready[NP],
  // p_free[NP], o_done, drain
  static constexpr int NBARS = 4 + 2 * NS + NSB + 2 * NP + 2;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int WARPS = 6;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int SHARE_OFF = (MISC_OFF + 16 + 15) / 16 * 16;
  static constexpr int SCRATCH_OFF = SHARE_OFF + static_cast<int>(sizeof(Share));
  static constexpr int RED_OFF = (SCRATCH_OFF + WARPS * 8 + 15) / 16 * 16;  // float[2][4][16]
  static constexpr int SMEM = RED_OFF + 2 * 4 * 16 * 4 + 16 * 4 + 1024;  // + float[16]
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(Q_OFF % 1024 == 0 && P_OFF % 1024 == 0, "swizzle atoms 1024-aligned");
};
constexpr uint32_t kDecCols = 256;             // TMEM: S^T tiles, then O^T
constexpr float kAlarm = 8.f;                  // log2 units

template <int NR>
__device__ __forceinline__ void ld_rows(uint32_t t0, uint32_t (&r)[NR]) {
  if constexpr (NR == 8) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(t0)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t0)
        : "memory");
  }
}
template <int NR>
__device__ __forceinline__ void st_rows(uint32_t t0, const uint32_t (&r)[NR]) {
  if constexpr (NR == 8) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t0),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(t0),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
  }
}

// Whether `v` holds in any of the 128 threads that meet at barrier `id`.
__device__ __forceinline__ bool bar_any(uint32_t id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(v ? 1u : 0u), "r"(id)
      : "memory");
  return r != 0;
}

// Butterfly reduce-scatter of NR values over a warp (max or sum): lane l
// holds the reduction of value l / (32 / NR).
template <int NR, bool kMax>
__device__ __forceinline__ float reduce_rows(float (&v)[NR], int lane) {
#pragma unroll
  for (int n = NR, msk = 16; n > 1; n >>= 1, msk >>= 1) {
    const bool upper = (lane & msk) != 0;
#pragma unroll
    for (int k = 0; k < n / 2; ++k) {
      const float send = upper ? v[k] : v[k + n / 2];
      const float keep = upper ? v[k + n / 2] : v[k];
      const float got = __shfl_xor_sync(0xffffffffu, send, msk);
      v[k] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
#pragma unroll
  for (int msk = 16 / NR; msk >= 1; msk >>= 1) {
    const float got = __shfl_xor_sync(0xffffffffu, v[0], msk);
    v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
  }
  return v[0];
}

// Ring positions of the unit's tiles: K_0 .. K_LA-1, then V_j, K_j+LA for
// every j.
struct RingPos {
  int n, ahead;
  __device__ __forceinline__ int v(int j) const { return ahead + j + min(j, n - ahead); }
  __device__ __forceinline__ int k(int j) const { return j < ahead ? j : v(j - ahead) + 1; }
};

template <int D, bool BF16, int NR>
__global__ void __launch_bounds__(DecCfg<D>::THREADS, 1)
    paged_decode_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                           const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const Args a,
                           const int lg_box, const CacheBlocks kb, const CacheBlocks vb) {
  using C = DecCfg<D>;
  using T = typename Elem<BF16>::T;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* sRing = smem;
  uint8_t* sQ = smem + C::Q_OFF;
  uint8_t* sP = smem + C::P_OFF;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* q_empty = q_full + 2;
  uint64_t* full = q_empty + 2;
  uint64_t* empty = full + C::NS;
  uint64_t* s_full = empty + C::NS;
  uint64_t* p_ready = s_full + C::NSB;
  uint64_t* p_free = p_ready + C::NP;
  uint64_t* o_done = p_free + C::NP;
  uint64_t* drain = o_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  Share* sh = reinterpret_cast<Share*>(smem + C::SHARE_OFF);
  float* red = reinterpret_cast<float*>(smem + C::RED_OFF);
  constexpr int kLoad = 4, kMma = 5;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::NSB; ++i) mbar_init(&s_full[i], 1);
    for (int i = 0; i < C::NP; ++i) {
      mbar_init(&p_ready[i], 128);
      mbar_init(&p_free[i], 1);
    }
    mbar_init(o_done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(tmem_slot, kDecCols);
    tmem_relinquish();
  }
  if (warp == kLoad && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // query rows that no box writes stay zero: finite scores that nobody reads
  for (int i = threadIdx.x; i < 2 * C::QT / 16; i += C::THREADS)
    reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_shared();
  tc_fence_before();
  griddep_launch_dependents();
  griddep_wait();
  const AttendUnits units{a.by_w, 7, a.causal, 2};
  const int heads = a.Hkv * a.nsub;
  plan_share<C::THREADS>(a, units, heads, 2,
                         reinterpret_cast<long long*>(smem + C::SCRATCH_OFF), sh);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{a.wait_ns, abort_flag, a.status};
  // every warp walks the share on its own
  Walk<AttendUnits> walk(*sh);
  Unit u;
  auto next = [&]() { return walk.next(a, units, *sh, heads, &u); };
  auto ring_of = [&](int n) { return RingPos{n, min(C::LA, n)}; };
  int fills = 0, qfills = 0;  // producer: ring slots and query tiles filled

  if (warp == kLoad) {
    // ------------------------------------------------------------ producer
    const int nbox = 128 >> lg_box;
    const uint32_t box_bytes = (C::CB * 128u) << lg_box;
    int g = 0;
    bool ok = true;
    for (int it = 0; ok && next(); ++it) {
      const int kvh = a.by_nsub.div(u.h), sub = a.by_nsub.mod(u.h);
      const int n = u.s1 - u.s0;
      struct Box {
        int page, row;  // page -2: the table names none; -1: past the length
      };
      Boxes boxes_of(a, u.b, u.s0 * 128, u.s.nk, lg_box, lane);
      auto lookup = [&](int j) {
        Box x{-1, 0};
        if (j < n && boxes_of.tile(j, &x.page, &x.row)) {
          if (x.page < 0) x.page = -2;
        } else {
          x.page = -1;
        }
        return x;
      };
      auto load = [&](const CUtensorMap* map, const CacheBlocks& c, int j, const Box& x) {
        const int s = g % C::NS, use = g / C::NS;
        const int boxes = min(nbox, (u.s.nk - (u.s0 + j) * 128 + (1 << lg_box) - 1) >> lg_box);
        ok = __all_sync(0xffffffffu, ok && (use == 0 || mbar_wait(&empty[s], (use - 1) & 1, wc)));
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], box_bytes * boxes);
        __syncwarp();
        if (x.page != -1)
          load_box(sRing + s * C::TILE + lane * box_bytes, map, &full[s], x.row,
                   x.page < 0 ? c.blocks : x.page * c.page_mul + kvh * c.head_mul);
        fills = ++g;
      };
      Box bx[C::LA + 1];  // boxes of tiles j .. j + LA
#pragma unroll
      for (int i = 0; i <= C::LA; ++i) bx[i] = lookup(i);
      if (lane == 0) {
        const int qb = it & 1;
        if (it >= 2) ok = mbar_wait(&q_empty[qb], ((it >> 1) - 1) & 1, wc);
        if (ok) {
          qfills = it + 1;
          mbar_arrive_expect_tx(&q_full[qb], static_cast<uint32_t>(C::CB * a.gu * a.w * 128));
          for (int cb = 0; cb < C::CB; ++cb)
            tma_load_4d(sQ + qb * C::QT + cb * 16 * 128, &tmQ, &q_full[qb], cb * 64,
                        kvh * a.G + sub * a.gu, u.s.q0 + u.j * a.w, 0);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
#pragma unroll
      for (int i = 0; i < C::LA; ++i)
        if (ok && i < n) load(&tmK, kb, i, bx[i]);
      for (int j = 0; ok && j < n; ++j) {
        const Box nx = lookup(j + C::LA + 1);
        load(&tmV, vb, j, bx[0]);
        if (ok && j + C::LA < n) load(&tmK, kb, j + C::LA, bx[C::LA]);
#pragma unroll
        for (int i = 0; i < C::LA; ++i) bx[i] = bx[i + 1];
        bx[C::LA] = nx;
      }
    }
  } else if (warp == kMma) {
    // ---------------------------------------------------------- MMA issuer
    // (the whole warp in step; one lane, elected inside each instruction,
    // issues)
    constexpr uint32_t idS = idesc_f16(BF16, 128, 16, false, false);
    constexpr uint32_t idO = idesc_f16(BF16, 128, 16, true, false);
    const uint64_t k_desc = sdesc(smem_addr(sRing), 16, C::CB * 1024, kSwizzle128B);
    const uint64_t q_desc = sdesc(smem_addr(sQ), 16, 1024, kSwizzle128B);
    // V^T: 64-column blocks 1024 bytes apart, 8-key groups CB * 1024 (at
    // head_dim 64 the second block is the next group: rows of O^T that are
    // never read)
    const uint64_t v_desc = sdesc(smem_addr(sRing), 1024, C::CB * 1024, kSwizzle128B);
    const uint64_t p_desc = sdesc(smem_addr(sP), 16, 1024, kSwizzle128B);
    bool ok = true;
    int p0 = 0, g0 = 0;
    auto landed = [&](int p) {
      const int s = p % C::NS;
      ok = ok && mbar_wait(&full[s], static_cast<uint32_t>((p / C::NS) & 1), wc);
      return s;
    };
    for (int it = 0; next(); ++it) {
      const int n = u.s1 - u.s0, s0 = u.s0, nk = u.s.nk;
      const RingPos rp = ring_of(n);
      const int qb = it & 1;
      ok = ok && mbar_wait(&q_full[qb], static_cast<uint32_t>((it >> 1) & 1), wc);
      auto scores = [&](int j) {
        const int s = landed(p0 + rp.k(j));
        __syncwarp();
        tc_fence_after();
        const int buf = (g0 + j) % C::NSB;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ko = s * C::TILE + (kk >> 2) * 1024 + (kk & 3) * 32;
          const uint32_t qo = qb * C::QT + (kk >> 2) * 2048 + (kk & 3) * 32;
          mma_f16_ss_elect(tmem + buf * 16, k_desc + (ko >> 4), q_desc + (qo >> 4), idS,
                           kk > 0 ? 1u : 0u, ok ? 1u : 0u);
        }
        mma_commit_elect(&s_full[buf], 1u);
        mma_commit_elect(&empty[s], 1u);
        if (j == n - 1) mma_commit_elect(&q_empty[qb], 1u);
      };
      if (n == 0) mma_commit_elect(&q_empty[qb], 1u);
      for (int j = 0; j < rp.ahead; ++j) scores(j);
      for (int j = 0; j < n; ++j) {
        const int pb = (g0 + j) % C::NP;
        const int s = landed(p0 + rp.v(j));
        const int keys = nk - (s0 + j) * 128;
        if (keys < 128 && (keys & 15)) {
          // value rows between the length and the end of its group of 16
          uint8_t* v = sRing + s * C::TILE;
          const int rows = 16 - (keys & 15);
          for (int i = lane; i < rows * C::CB * 8; i += 32) {
            const int key = keys + i / (C::CB * 8), cb = (i >> 3) % C::CB;
            *reinterpret_cast<uint4*>(v + ((key >> 3) * C::CB + cb) * 1024 + (key & 7) * 128 +
                                      (i & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_shared();
        }
        ok = ok && mbar_wait(&p_ready[pb], static_cast<uint32_t>(((g0 + j) / C::NP) & 1), wc);
        __syncwarp();
        tc_fence_after();
        const int groups = min(8, (keys + 15) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t vo = s * C::TILE + kk * 2 * C::CB * 1024;
          const uint32_t po = pb * C::PT + (kk >> 2) * 2048 + (kk & 3) * 32;
          mma_f16_ss_elect(tmem + C::NSB * 16, v_desc + (vo >> 4), p_desc + (po >> 4), idO,
                           (j > 0 || kk > 0) ? 1u : 0u, ok && kk < groups ? 1u : 0u);
        }
        mma_commit_elect(&p_free[pb], 1u);
        mma_commit_elect(&empty[s], 1u);
        if (j + rp.ahead < n) scores(j + rp.ahead);
      }
      // (a unit without keys hands over nothing: the softmax warps, who did not
      // hold this warp up there, could miss a phase)
      if (n > 0) mma_commit_elect(o_done, 1u);
      p0 += 2 * n;
      g0 += n;
    }
    // every product completes before TMEM is freed
    mma_commit_elect(drain, 1u);
    if (lane == 0) drain_wait(drain, 0, kDrainNs);
    __syncwarp();
  } else {
    // ------------------------------------------------ softmax and epilogue
    const int i = threadIdx.x;  // key of a tile; head dimension of O^T
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tO = tmem + lane_off + C::NSB * 16;
    bool ok = true, began = false;
    int g = 0, units_done = 0;
    while (next()) {
      const Seq s = u.s;
      const int n = u.s1 - u.s0;
      const int tok0 = u.j * a.w;
      // visible keys of each row, counted from the piece's first key; rows
      // that do not exist are given every key (never read)
      int lim[NR];
#pragma unroll
      for (int c = 0; c < NR; ++c) {
        const int tok = tok0 + a.by_gu.div(c);
        const int l = a.causal ? min(s.nk, s.off + tok + 1) : s.nk;
        lim[c] = l - u.s0 * 128;
      }
      float m[NR], l[NR];
#pragma unroll
      for (int c = 0; c < NR; ++c) {
        m[c] = -INFINITY;
        l[c] = 0.f;
      }
      for (int j = 0; j < n; ++j, ++g) {
        const int buf = g % C::NSB, pb = g % C::NP;
        ok = __all_sync(0xffffffffu,
                        ok && mbar_wait(&s_full[buf], static_cast<uint32_t>((g / C::NSB) & 1), wc));
        tc_fence_after();
        __syncwarp();
        uint32_t sv[NR];
        ld_rows<NR>(tmem + lane_off + buf * 16, sv);
        float x[NR];
        bool over = false;
        if ((j + 1) * 128 <= lim[0]) {  // (the first row sees the fewest keys)
#pragma unroll
          for (int c = 0; c < NR; ++c) {
            x[c] = __uint_as_float(sv[c]) * a.sl2;
            over |= x[c] > m[c] + kAlarm;
          }
        } else {
          const int key = j * 128 + i;
#pragma unroll
          for (int c = 0; c < NR; ++c) {
            x[c] = key < lim[c] ? __uint_as_float(sv[c]) * a.sl2 : -INFINITY;
            over |= x[c] > m[c] + kAlarm;
          }
        }
        if (bar_any(1, over)) {
          float t[NR];
#pragma unroll
          for (int c = 0; c < NR; ++c) t[c] = x[c];
          const float mx = reduce_rows<NR, true>(t, lane);
          if ((lane & (32 / NR - 1)) == 0) red[warp * 16 + lane / (32 / NR)] = mx;
          named_bar_sync(2, 128);
          float alpha[NR];
#pragma unroll
          for (int c = 0; c < NR; ++c) {
            const float mn = fmaxf(fmaxf(fmaxf(red[c], red[16 + c]), fmaxf(red[32 + c], red[48 + c])),
                                   m[c]);
            alpha[c] = mn == m[c] ? 1.f : ex2(m[c] - mn);
            m[c] = mn;
            l[c] *= alpha[c];
          }
          if (j > 0) {
            // O^T through the previous tile, rescaled
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&p_free[(g - 1) % C::NP],
                                                         static_cast<uint32_t>(((g - 1) / C::NP) & 1),
                                                         wc));
            tc_fence_after();
            __syncwarp();
            uint32_t o[NR];
            ld_rows<NR>(tO, o);
#pragma unroll
            for (int c = 0; c < NR; ++c)
              o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha[c]);
            st_rows<NR>(tO, o);
            tmem_wait_st();
          }
          named_bar_sync(2, 128);  // `red` is read
        }
        // the P buffer's previous tile has been read by its products
        if (g >= C::NP)
          ok = __all_sync(0xffffffffu,
                          ok && mbar_wait(&p_free[pb], static_cast<uint32_t>((g / C::NP - 1) & 1), wc));
        // P^T: row c, key i at chunk i / 64, 16-byte unit ((i % 64) / 8) ^ (c % 8)
        uint8_t* pcol = sP + pb * C::PT + (i >> 6) * 2048 + (i & 7) * 2;
        const int un = (i & 63) >> 3;
#pragma unroll
        for (int c = 0; c < NR; ++c) {
          const float p = ex2(x[c] - (m[c] == -INFINITY ? 0.f : m[c]));
          l[c] += p;
          *reinterpret_cast<uint16_t*>(pcol + c * 128 + ((un ^ (c & 7)) << 4)) =
              static_cast<uint16_t>(Elem<BF16>::pack(p, 0.f));
        }
        fence_proxy_async_shared();
        tc_fence_before();
        // every thread arrives every tile, also after a failed wait
        mbar_arrive(&p_ready[pb]);
      }
      // sums over the tiles' keys
      {
        const float v = reduce_rows<NR, false>(l, lane);
        if ((lane & (32 / NR - 1)) == 0) red[64 + warp * 16 + lane / (32 / NR)] = v;
      }
      const bool whole = u.whole();
      const int kvh = a.by_nsub.div(u.h), e0 = a.by_nsub.mod(u.h) * a.gu;
      float* slot = a.ws + static_cast<size_t>(blockIdx.x * 2 + u.slot()) * (NR * (D + 2));
      if (!whole && u.s0 == 0 && i == 0) {
        int* d = a.desc + blockIdx.x * kDesc;
        d[0] = pieces_of(u, *sh);
        d[1] = u.b;
        d[2] = u.h;
        d[3] = u.j;
        d[4] = s.q0;
        d[5] = s.nq;
        began = true;
      }
      named_bar_sync(2, 128);
      // Thread c finishes row c: its sum, the factor of its output (0 where
      // it saw no key: O^T may never have been written), its LSE.
      if (i < NR) {
        float M = 0.f;  // (m is indexed by constants only)
#pragma unroll
        for (int c = 0; c < NR; ++c)
          if (i == c) M = m[c];
        float L = (red[64 + i] + red[80 + i]) + (red[96 + i] + red[112 + i]);
        const int t = a.by_gu.div(i), e = e0 + a.by_gu.mod(i);
        const bool row_ok = i < a.gu * a.w && tok0 + t < s.nq && e < a.G;
        float f = L != 0.f ? 1.f : 0.f;
        if (!whole) {
          if (row_ok) {
            slot[NR * D + i] = M;
            slot[NR * (D + 1) + i] = L;
          }
        } else if (row_ok) {
          const int hq = kvh * a.G + e;
          if (a.sinks) f *= add_sink(a.sinks[hq], M, L);
          f = L != 0.f ? f / L : 0.f;
          if (a.lse)
            a.lse[static_cast<long long>(s.q0 + tok0 + t) * a.Hq + hq] =
                L != 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
        }
        red[128 + i] = f;
      }
      if (n > 0) {
        ok = __all_sync(0xffffffffu,
                        ok && mbar_wait(o_done, static_cast<uint32_t>(units_done & 1), wc));
        ++units_done;
      }
      tc_fence_after();
      __syncwarp();
      uint32_t ov[NR];
      ld_rows<NR>(tO, ov);
      tc_fence_before();
      named_bar_sync(2, 128);
      if (ok && i < D) {
        // rows in order: token t, head e of the group
        T* orow = static_cast<T*>(a.o) + (s.q0 + tok0) * a.os[0] + (kvh * a.G + e0) * a.os[1] + i;
        int t = 0, e = 0;
#pragma unroll
        for (int c = 0; c < NR; ++c) {
          const float f = red[128 + c];
          const float v = f != 0.f ? __uint_as_float(ov[c]) * f : 0.f;
          if (t < a.w && tok0 + t < s.nq && e0 + e < a.G) {
            if (!whole)
              slot[c * D + i] = v;
            else
              *reinterpret_cast<uint16_t*>(orow + t * a.os[0] + e * a.os[1]) =
                  static_cast<uint16_t>(Elem<BF16>::pack(v, 0.f));
          }
          if (++e == a.gu) {
            e = 0;
            ++t;
          }
        }
      }
      named_bar_sync(2, 128);  // `red` is read
    }
    if (i == 0 && !began) a.desc[blockIdx.x * kDesc] = 0;
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kDecCols);
  }
  if (warp == kLoad && lane == 0 && *abort_flag) {
    // a role gave up: every copy the producer issued lands before the CTA exits
    for (int i = max(0, qfills - 2); i < qfills; ++i)
      drain_wait(&q_full[i & 1], static_cast<uint32_t>((i >> 1) & 1), kDrainNs);
    for (int i = max(0, fills - C::NS); i < fills; ++i)
      drain_wait(&full[i % C::NS], static_cast<uint32_t>((i / C::NS) & 1), kDrainNs);
  }
}

template <int D, bool BF16, int NR>
sdpa_status_t launch_dec(const Args& a, const CUtensorMap& tq, const CUtensorMap& tk,
                         const CUtensorMap& tv, int lg_box, const CacheBlocks& kb,
                         const CacheBlocks& vb, const LaunchEnv& env) {
  using C = DecCfg<D>;
  auto kern = paged_decode_tc_kernel<D, BF16, NR>;
  if (!allow_smem<paged_decode_tc_kernel<D, BF16, NR>>(C::SMEM)) return SDPA_ERR_CUDA;
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
  if (cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, a, lg_box, kb, vb) != cudaSuccess)
    return SDPA_ERR_CUDA;
  return launch_paged_merge(a, D, BF16 ? SDPA_BF16 : SDPA_F16, NR, 1, env.stream);
}

template <int D>
sdpa_status_t launch_decode_of(Args a, int dtype, int rows, const LaunchEnv& env) {
  fit_rows(a, rows);
  const bool bf16 = dtype == SDPA_BF16;
  const CUtensorMapDataType dt =
      bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int lg_box = box_log2(a.page_size);
  CacheBlocks kb, vb;
  long long ku, vu;
  if (!cache_blocks(a.ks, a.num_pages, a.Hkv, &kb, &ku) ||
      !cache_blocks(a.vs, a.num_pages, a.Hkv, &vb, &vu))
    return SDPA_ERR_UNSUPPORTED;  // (the caller has checked)
  CUtensorMap tq, tk, tv;
  // a stride of a dimension of one element is never followed: any valid one
  auto st = [](long long s, long long n) { return static_cast<uint64_t>(n > 1 ? s : D); };
  if (!encode_tiled_4d_box(&tq, dt, a.q, D, a.Hq, a.T, 1, 2, 64, static_cast<uint32_t>(a.gu),
                           static_cast<uint32_t>(a.w), st(a.qs[1], a.Hq), st(a.qs[0], a.T), D) ||
      !encode_row_blocks(&tk, dt, a.k, D / 64, a.page_size, kb.blocks, 1 << lg_box,
                         st(a.ks[2], a.page_size), ku) ||
      !encode_row_blocks(&tv, dt, a.v, D / 64, a.page_size, vb.blocks, 1 << lg_box,
                         st(a.vs[2], a.page_size), vu))
    return SDPA_ERR_CUDA;
  if (rows == 8)
    return bf16 ? launch_dec<D, true, 8>(a, tq, tk, tv, lg_box, kb, vb, env)
                : launch_dec<D, false, 8>(a, tq, tk, tv, lg_box, kb, vb, env);
  return bf16 ? launch_dec<D, true, 16>(a, tq, tk, tv, lg_box, kb, vb, env)
              : launch_dec<D, false, 16>(a, tq, tk, tv, lg_box, kb, vb, env);
}

}  // namespace
}  // namespace paged

int paged_decode_rows(const paged::Args& a) {
  // Against the 128-row form of paged_tc.cuh (us): 4 sequences of up to 1000 keys, 4 rows,
  // 10.9 and 13.7; 16 x 4096 keys, 16 rows, 52.5 and 56.6.  Eight rows a tile
  // against sixteen: 10.9 and 12.1, and 32.8 and 35.1 at 64 x 4096 keys, 8
  // rows, head_dim 64.
  const long long rows = paged::call_rows(a);
  return a.G > 16 ? 0 : a.G <= 8 && rows <= 8 ? 8 : rows <= 16 ? 16 : 0;
}

sdpa_status_t launch_paged_decode_tc(const paged::Args& a, int head_dim, int dtype, int rows,
                                     const LaunchEnv& env) {
  return head_dim == 64 ? paged::launch_decode_of<64>(a, dtype, rows, env)
                        : paged::launch_decode_of<128>(a, dtype, rows, env);
}

}  // namespace gb300

// paged_tc.cuh — attention of packed new tokens over the paged KV cache for
// fp16/bf16, head_dim 64/128, on the 5th-generation tensor cores: the kernel
// and its launch, instantiated per head size in paged_tc_d64.cu and
// paged_tc_d128.cu.
//
// The rows of a 128-row query tile are (token, query head) pairs of one kv
// head: w = 128 / gu tokens times gu heads, row = token * gu + head, which a
// TMA box of w tokens x gu heads lays down in that order.  So the tokens and
// heads that read the same keys share every K and V tile.  The work is divided
// as paged.cuh describes (equal shares of all key tiles of all units, cut
// units merged after); calls of up to 16 rows a sequence and kv head take
// paged_decode_tc.cu.
//
// Two forms:
//  NT = 2  (sequences of more than 128 rows): a unit is two query
//          tiles that share each K/V tile; S_0 | S_1 | O_0 | O_1 in TMEM, and
//          the softmax of one tile overlaps the products of the other.  Bound
//          by the tensor pipe, 71 % active, the softmax warps and the clock
//          under that load (4096 tokens over 32768 keys, 32 heads over 8,
//          head_dim 128, bf16: 1190 to 1374 us from one GPU to the next, 1730
//          to 1500 TFLOP/s).
//  NT = 1  (short chunks, 17 to 128 rows): one query tile; S is
//          double-buffered over the key tiles (S_j+1 is computed while the
//          softmax works on S_j), six 32 KB K/V slots in flight at head_dim
//          128.  Bound by the softmax chain of a key tile where HBM is not
//          (8 x 16 tokens over 4096 keys: 37 us, 3.6 TB/s); warps without a
//          row do no arithmetic.
// K and V have ring slots of their own, each released when its products are
// done: loads then run a step further ahead than with a slot for both (the
// 4096-token chunk above 1715 -> 1210 us).
//
// Key tiles are 128 keys in boxes of R = gcd(page_size, 128) rows, each
// inside a page; one lane of the producer warp looks up and loads each box, in
// one copy for both 64-column halves of its rows (a tile lies as [16 groups
// of 8 keys][D / 64][8][64], which both operand descriptors take).  With a
// copy per half, 16-row pages cost 30 % more: a copy has a price of its own.
// Boxes past the sequence's length are not loaded.  What the last tile holds
// behind it (a page's rows of no sequence yet: anything, NaN included) is kept
// out of the results: such scores are replaced by -inf, the value product
// stops at the last group of 16 keys in use, and the rows of that group past
// the length are zeroed in shared memory before it.
//
// Warp roles and the issue loop (a whole warp in step, no shared-memory access
// between MMAs, named barriers) are those of the prefill kernel
// (prefill_tc.cuh), whose softmax arithmetic this one uses: p = 2^(s * scale *
// log2e - m) against a reference max m that moves only when a row sum passes
// 2^15, so P stays in the exact range of fp16 and bf16.
//
// Rounding: P goes into the value product in the cache's type, since the
// product takes one type for both operands (half a step of it, 2^-8 relative
// in bf16 and 2^-11 in fp16, on each weight; a second product for the rest of P
// would add half of the tensor pipe's work).  The sums take P before that
// rounding.  Relative error of O against 64 bits: 2.3e-3 in bf16 and 2.9e-4 in
// fp16, where rounding the exact O once gives 1.7e-3 and 2.1e-4.
#pragma once

#include <atomic>

#include "paged.cuh"
#include "prefill_tc.cuh"

namespace gb300 {
namespace paged {
namespace {

template <int D, int NT>
struct TcCfg {
  static constexpr int CB = D / 64;        // 128-byte column blocks of a row
  static constexpr int TILE = 128 * D * 2;
  // Ring of K and V tiles (a slot each), in the order of their use: K_0 ..
  // K_LA-1, then V_j, K_j+LA for every j: S runs LA key tiles ahead of P V.
  static constexpr int NS = NT == 2 ? (D == 64 ? 8 : 4) : (D == 64 ? 12 : 6);
  static constexpr int LA = NT == 2 ? 1 : 2;
  static constexpr int RING_OFF = NT * TILE;
  static constexpr int BAR_OFF = RING_OFF + NS * TILE;
  // q_full, q_empty, full[NS], empty[NS], s_full[2], o_done[2], pv_done, drain
  static constexpr int NBARS = 2 + 2 * NS + 2 + 2 + 1 + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int SOFT_WARPS = 4 * NT;
  static constexpr int WARPS = SOFT_WARPS + 4;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int SHARE_OFF = (MISC_OFF + 16 + 15) / 16 * 16;
  static constexpr int SCRATCH_OFF = SHARE_OFF + static_cast<int>(sizeof(Share));
  static constexpr int WALK_OFF = (SCRATCH_OFF + (WARPS + 1) * 8 + 15) / 16 * 16;
  static constexpr int UNIT_OFF =
      WALK_OFF + WARPS * static_cast<int>(sizeof(Walk<AttendUnits>));
  static constexpr int SMEM = UNIT_OFF + WARPS * static_cast<int>(sizeof(Unit)) + 1024;
  static_assert(SMEM <= 232448, "shared memory budget");
  static constexpr uint32_t s_col(int i) { return static_cast<uint32_t>(i * 128); }
  static constexpr uint32_t o_col(int t) { return static_cast<uint32_t>(256 + t * D); }
  static constexpr int SLOT = 128 * NT * (D + 2);  // floats of a partial result
};

// Fixed cost of a unit (query tiles, the first scores, the output) in key
// tiles: 8 chunks of 64 tokens over 4096 keys took 60 us with 6, 69 with 2.
constexpr int kUnitSteps = 6;
constexpr uint32_t kPBar = 1;  // + t: softmax warps of tile t with the MMA warp
constexpr uint32_t kKBar = 3;  // stage helper with the MMA warp

// What a role needs of a unit.
struct TileGeo {
  int nt;       // active query tiles
  int s0;       // first key tile
  int n[2];     // key tiles of each query tile, from s0
  int nmax;     // key tiles loaded
  int nk;
  // ring positions of V_j and K_j, counted from the unit's first slot
  template <int LA>
  __device__ __forceinline__ int v_pos(int j) const {
    const int ahead = min(LA, nmax);
    return ahead + j + min(j, nmax - ahead);
  }
  template <int LA>
  __device__ __forceinline__ int k_pos(int j) const {
    return j < LA ? j : v_pos<LA>(j - LA) + 1;
  }
};
template <int NT>
__device__ __forceinline__ TileGeo tile_geo(const Args& a, const Unit& u) {
  TileGeo g;
  g.s0 = u.s0;
  g.nk = u.s.nk;
  g.nmax = u.s1 - u.s0;
  const int tok0 = u.j * a.w * NT;
  g.nt = NT == 2 && tok0 + a.w < u.s.nq ? 2 : 1;
  g.n[0] = g.n[1] = g.nmax;
  if (NT == 2 && a.causal && g.nt == 2) {  // the first tile may see fewer keys
    const int lim = min(u.s.nk, max(0, u.s.off + tok0 + a.w));
    g.n[0] = max(0, min(u.s1, (lim + 127) >> 7) - u.s0);
  }
  return g;
}

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(TcCfg<D, NT>::THREADS, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const Args a, const int lg_box,
                    const CacheBlocks kb, const CacheBlocks vb) {
  using C = TcCfg<D, NT>;
  using E = Elem<BF16>;
  using T = typename E::T;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + C::RING_OFF;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* q_empty = q_full + 1;
  uint64_t* full = q_empty + 1;
  uint64_t* empty = full + C::NS;
  uint64_t* s_full = empty + C::NS;
  uint64_t* o_done = s_full + 2;
  uint64_t* pv_done = o_done + 2;
  uint64_t* drain = pv_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  Share* sh = reinterpret_cast<Share*>(smem + C::SHARE_OFF);
  constexpr int kLoad = C::SOFT_WARPS, kMma = kLoad + 1, kHelp = kLoad + 2;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(pv_done, 1);
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
    tma_prefetch_desc(&tmV);
  }
  // query rows that no box writes stay zero: finite scores that nobody reads
  if (a.gu * a.w < 128) {
    for (int i = threadIdx.x; i < NT * C::TILE / 16; i += C::THREADS)
      reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_shared();
  }
  tc_fence_before();
  griddep_launch_dependents();
  griddep_wait();
  const AttendUnits units{a.by_w, 7, a.causal, kUnitSteps};
  const int heads = a.Hkv * a.nsub;
  plan_share<C::THREADS>(a, units, heads, 2,
                         reinterpret_cast<long long*>(smem + C::SCRATCH_OFF), sh);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{a.wait_ns, abort_flag, a.status};
  // Each warp walks the share on its own; the walk's state lives in shared
  // memory, so that it holds no registers between units.
  using W = Walk<AttendUnits>;
  W* walk = reinterpret_cast<W*>(smem + C::WALK_OFF) + warp;
  Unit* unit = reinterpret_cast<Unit*>(smem + C::UNIT_OFF) + warp;
  if (lane == 0) *walk = W(*sh);
  auto next = [&]() {
    __syncwarp();
    bool more = false;
    if (lane == 0) more = walk->next(a, units, *sh, heads, unit);
    return __shfl_sync(0xffffffffu, more ? 1 : 0, 0) != 0;
  };
  int fills = 0;    // producer: ring slots filled
  int last_q = -1;  // and last unit whose Q it loaded

  if (warp >= C::SOFT_WARPS) {
    if constexpr (NT == 2) setmaxnreg_dec<kControlRegs>();
    if (warp == kLoad) {
      // ---------------------------------------------------------- producer
      const int nbox = 128 >> lg_box;
      const uint32_t box_bytes = (C::CB * 128u) << lg_box;
      int g = 0;  // ring slots filled
      bool ok = true;
      for (int it = 0; ok && next(); ++it) {
        const Unit u = *unit;
        const TileGeo tg = tile_geo<NT>(a, u);
        const int kvh = a.by_nsub.div(u.h), sub = a.by_nsub.mod(u.h);
        // Page and row of this lane's box of key tile t (page -2: the table
        // names none; -1: past the length).
        struct Box {
          int page, row;
        };
        Boxes boxes_of(a, u.b, tg.s0 * 128, u.s.nk, lg_box, lane);
        auto lookup = [&](int j) {
          Box x{-1, 0};
          if (j < tg.nmax && boxes_of.tile(j, &x.page, &x.row)) {
            if (x.page < 0) x.page = -2;
          } else {
            x.page = -1;
          }
          return x;
        };
        auto load = [&](const CUtensorMap* map, const CacheBlocks& c, int j, const Box& x) {
          const int s = g % C::NS, use = g / C::NS;
          const int boxes = min(nbox, (u.s.nk - (tg.s0 + j) * 128 + (1 << lg_box) - 1) >> lg_box);
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
        for (int i = 0; i < C::LA; ++i) bx[i] = lookup(i);
        if (lane == 0) {
          if (it > 0) ok = mbar_wait(q_empty, (it - 1) & 1, wc);
          if (ok) {
            last_q = it;
            mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(tg.nt * C::CB * a.gu * a.w * 128));
            for (int t = 0; t < tg.nt; ++t)
              for (int cb = 0; cb < C::CB; ++cb)
                tma_load_4d(sQ + t * C::TILE + cb * 128 * 128, &tmQ, q_full, cb * 64,
                            kvh * a.G + sub * a.gu, u.s.q0 + (u.j * NT + t) * a.w, 0);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
#pragma unroll
        for (int i = 0; i < C::LA; ++i)
          if (ok && i < tg.nmax) load(&tmK, kb, i, bx[i]);
        bx[C::LA] = lookup(C::LA);
        for (int j = 0; ok && j < tg.nmax; ++j) {
          const Box nx = lookup(j + C::LA + 1);
          load(&tmV, vb, j, bx[0]);
          if (ok && j + C::LA < tg.nmax) load(&tmK, kb, j + C::LA, bx[C::LA]);
#pragma unroll
          for (int i = 0; i < C::LA; ++i) bx[i] = bx[i + 1];
          bx[C::LA] = nx;
        }
      }
    } else if (warp == kMma) {
      // -------------------------------------------------------- MMA issuer
      constexpr uint32_t idS = idesc_f16(BF16, 128, 128, false, false);
      constexpr uint32_t idO = idesc_f16(BF16, 128, D, false, true);
      const uint64_t q_desc = sdesc(smem_addr(sQ), 16, 1024, kSwizzle128B);
      // K and V tiles: 8-key groups CB * 1024 bytes apart, 64-column blocks
      // 1024
      const uint64_t k_desc = sdesc(smem_addr(sRing), 16, C::CB * 1024, kSwizzle128B);
      const uint64_t v_desc = sdesc(smem_addr(sRing), 1024, C::CB * 1024, kSwizzle128B);
      const uint32_t q_hi = static_cast<uint32_t>(q_desc >> 32);
      const uint32_t k_hi = static_cast<uint32_t>(k_desc >> 32);
      const uint32_t v_hi = static_cast<uint32_t>(v_desc >> 32);
      const uint32_t q_lo = static_cast<uint32_t>(q_desc);
      const uint32_t k_lo = static_cast<uint32_t>(k_desc);
      const uint32_t v_lo = static_cast<uint32_t>(v_desc);
      auto desc = [](uint32_t hi, uint32_t lo) { return (static_cast<uint64_t>(hi) << 32) | lo; };
      // S (columns of slot i) = Q_t K^T, K in ring slot s
      auto issue_s = [&](int t, int i, int s) {
        const uint32_t qd = q_lo + static_cast<uint32_t>((t * C::TILE) >> 4);
        const uint32_t kd = k_lo + static_cast<uint32_t>((s * C::TILE) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t qo = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
          const uint32_t ko = ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4;
          mma_f16_ss_elect(tmem + C::s_col(i), desc(q_hi, qd + qo), desc(k_hi, kd + ko), idS,
                           kk > 0 ? 1u : 0u, 1u);
        }
      };
      // O_t += P V, P in slot i, V in ring slot s, keys in groups of 16
      auto issue_pv = [&](int t, int i, int s, bool first, int groups) {
        const uint32_t vd = v_lo + static_cast<uint32_t>((s * C::TILE) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_f16_ts_elect(tmem + C::o_col(t), tmem + C::s_col(i) + kk * 8,
                           desc(v_hi, vd + ((kk * 2 * C::CB * 1024) >> 4)), idO,
                           (!first || kk > 0) ? 1u : 0u, kk < groups ? 1u : 0u);
      };
      int p0 = 0;  // ring slots of earlier units
      int g0 = 0;  // key tiles of earlier units
      while (next()) {
        const TileGeo tg = tile_geo<NT>(a, *unit);
        auto groups = [&](int j) { return min(8, (tg.nk - (tg.s0 + j) * 128 + 15) >> 4); };
        auto kslot = [&](int j) { return (p0 + tg.k_pos<C::LA>(j)) % C::NS; };
        auto vslot = [&](int j) { return (p0 + tg.v_pos<C::LA>(j)) % C::NS; };
        named_bar_sync(kKBar, 64);  // Q and K_0 have landed
        tc_fence_after();
        if constexpr (NT == 2) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t >= tg.nt) continue;
            // (a tile without keys hands over nothing: its softmax warps, who
            // would not hold this warp up, could miss a phase of o_done)
            if (tg.n[t] > 0) {
              issue_s(t, t, kslot(0));
              mma_commit_elect(&s_full[t], 1u);
            }
          }
          if (tg.nmax > 0) mma_commit_elect(&empty[kslot(0)], 1u);
          if (tg.nmax <= 1) mma_commit_elect(q_empty, 1u);
          for (int j = 0; j < tg.nmax; ++j) {
            bool waited = false;
            const int ks = kslot(j + 1), vs = vslot(j);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (t >= tg.nt || j >= tg.n[t]) continue;
              named_bar_sync(kPBar + t, 32 * 5);
              if (!waited) {  // V_j and K_j+1 have landed
                named_bar_sync(kKBar, 64);
                waited = true;
              }
              tc_fence_after();
              issue_pv(t, t, vs, j == 0, groups(j));
              if (j + 1 < tg.n[t]) {
                issue_s(t, t, ks);
                mma_commit_elect(&s_full[t], 1u);
              } else {
                mma_commit_elect(&o_done[t], 1u);
              }
            }
            // K_j+1 and V_j are free once these land (S_1,j+1 is the last
            // of them, or the P V products where the unit ends)
            if (j + 1 < tg.nmax) mma_commit_elect(&empty[ks], 1u);
            if (j == tg.nmax - 2) mma_commit_elect(q_empty, 1u);
            mma_commit_elect(&empty[vs], 1u);
          }
        } else {
          if (tg.nmax == 0) {
            mma_commit_elect(q_empty, 1u);
          } else {
            issue_s(0, g0 & 1, kslot(0));
            mma_commit_elect(&s_full[g0 & 1], 1u);
            mma_commit_elect(&empty[kslot(0)], 1u);
            if (tg.nmax > 1) {
              named_bar_sync(kKBar, 64);
              tc_fence_after();
              issue_s(0, (g0 + 1) & 1, kslot(1));
              mma_commit_elect(&s_full[(g0 + 1) & 1], 1u);
              mma_commit_elect(&empty[kslot(1)], 1u);
            }
            if (tg.nmax <= 2) mma_commit_elect(q_empty, 1u);
            for (int j = 0; j < tg.nmax; ++j) {
              const int i = (g0 + j) & 1;
              named_bar_sync(kPBar, 32 * 5);
              named_bar_sync(kKBar, 64);  // V_j and K_j+2 have landed
              tc_fence_after();
              issue_pv(0, i, vslot(j), j == 0, groups(j));
              mma_commit_elect(pv_done, 1u);
              mma_commit_elect(&empty[vslot(j)], 1u);
              if (j + 2 < tg.nmax) {
                issue_s(0, i, kslot(j + 2));
                mma_commit_elect(&s_full[i], 1u);
                mma_commit_elect(&empty[kslot(j + 2)], 1u);
                if (j + 3 == tg.nmax) mma_commit_elect(q_empty, 1u);
              }
            }
            mma_commit_elect(&o_done[0], 1u);
          }
        }
        p0 += 2 * tg.nmax;
        g0 += tg.nmax;
      }
      // every MMA issued by this warp completes before TMEM is freed
      mma_commit_elect(drain, 1u);
      if (lane == 0) drain_wait(drain, 0, kDrainNs);
      __syncwarp();
    } else if (warp == kHelp) {
      // ------------------------------------------------------ stage helper
      // Waits for the tiles that the MMA warp's next products read, zeroes
      // the last tile's value rows between the length and the end of its
      // group of 16 keys, and meets the MMA warp (the same number of times,
      // also after a failed wait).
      bool ok = true;
      int p0 = 0;
      auto landed = [&](int p) {
        const int s = p % C::NS;
        ok = ok && mbar_wait(&full[s], static_cast<uint32_t>((p / C::NS) & 1), wc);
        return s;
      };
      for (int it = 0; next(); ++it) {
        const TileGeo tg = tile_geo<NT>(a, *unit);
        ok = ok && mbar_wait(q_full, static_cast<uint32_t>(it & 1), wc);
        if (tg.nmax > 0) landed(p0);
        __syncwarp();
        named_bar_sync(kKBar, 64);
        if (NT == 1 && tg.nmax > 1) {
          landed(p0 + 1);
          __syncwarp();
          named_bar_sync(kKBar, 64);
        }
        for (int j = 0; j < tg.nmax; ++j) {
          const int s = landed(p0 + tg.v_pos<C::LA>(j));
          const int keys = tg.nk - (tg.s0 + j) * 128;
          if (keys < 128 && (keys & 15)) {
            uint8_t* v = sRing + s * C::TILE;
            const int rows = 16 - (keys & 15);
            for (int i = lane; i < rows * C::CB * 8; i += 32) {
              const int key = keys + i / (C::CB * 8), cb = (i >> 3) % C::CB;
              *reinterpret_cast<uint4*>(v + ((key >> 3) * C::CB + cb) * 1024 + (key & 7) * 128 +
                                        (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_shared();
          }
          if (j + C::LA < tg.nmax) landed(p0 + tg.k_pos<C::LA>(j + C::LA));
          __syncwarp();
          named_bar_sync(kKBar, 64);
        }
        p0 += 2 * tg.nmax;
      }
    }
  } else {
    if constexpr (NT == 2) setmaxnreg_inc<kSoftmaxRegs>();
    // --------------------------------------------------------------- softmax
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lane_off + C::o_col(t);
    bool ok = true;
    int g0 = 0;   // steps of earlier units (NT = 2: of this tile)
    int oph = 0;  // phases of o_done[t] consumed
    bool began = false;  // this CTA wrote its descriptor
    while (next()) {
      const TileGeo tg = tile_geo<NT>(a, *unit);
      if (t >= tg.nt) continue;
      const int tok0 = (unit->j * NT + t) * a.w;  // first token of the tile
      const int nq = unit->s.nq;
      const int tok = tok0 + a.by_gu.div(r);
      // rows of this warp that exist
      const bool live = (warp & 3) * 32 < min(a.w, nq - tok0) * a.gu;
      // visible keys of the row, counted from the piece's first key
      const int limit =
          (a.causal ? min(tg.nk, unit->s.off + tok + 1) : tg.nk) - tg.s0 * 128;
      float m = -INFINITY, l = 0.f;
      const int n = tg.n[t];
      for (int j = 0; j < n; ++j) {
        const int g = g0 + j;
        const int slot = NT == 2 ? t : g & 1;
        const uint32_t tS = tmem + lane_off + C::s_col(slot);
        if (live) {
          ok = __all_sync(0xffffffffu,
                          ok && mbar_wait(&s_full[slot], (NT == 2 ? g : g >> 1) & 1, wc));
          if (ok) {
            tc_fence_after();
            uint32_t s[128];
            __syncwarp();
            tmem_ld4x32_sync(tS, tS + 32, tS + 64, tS + 96,
                             *reinterpret_cast<uint32_t(*)[32]>(&s[0]),
                             *reinterpret_cast<uint32_t(*)[32]>(&s[32]),
                             *reinterpret_cast<uint32_t(*)[32]>(&s[64]),
                             *reinterpret_cast<uint32_t(*)[32]>(&s[96]));
            const int vis = limit - j * 128;  // visible keys of the row in this tile
            if (__any_sync(0xffffffffu, vis < 128)) {
#pragma unroll
              for (int i = 0; i < 128; ++i)
                if (i >= vis) s[i] = 0xff800000u;  // -inf
            }
            float alpha = 1.f, rs;
            uint32_t pk[64];
            bool resc = !(m > -INFINITY);
            if (!resc) {
              softmax_pairs<BF16, 128>(s, a.sl2, m, pk, rs);
              resc = !(rs <= kFusedSumLimit);
            }
            if (resc) {
              const float mx = row_max_raw(s) * a.sl2;  // -inf: no visible key
              if (mx > -INFINITY) {
                alpha = ex2(m - mx);  // 0 when m = -inf
                m = mx;
              }
              softmax_pairs<BF16, 128>(s, a.sl2, m == -INFINITY ? 0.f : m, pk, rs);
            }
            __syncwarp();
            l = l * alpha + rs;
            // O_t through step j - 1 (NT = 2: complete, the commit behind
            // s_full tracks it); rescaled where a row's max moved
            if (j > 0 && __any_sync(0xffffffffu, resc)) {
              if constexpr (NT == 1) {
                ok = __all_sync(0xffffffffu, ok && mbar_wait(pv_done, (g - 1) & 1, wc));
                tc_fence_after();
              }
              __syncwarp();
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t ob[32];
                tmem_ld32_sync(tO + c * 32, ob);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  ob[i] = __float_as_uint(__uint_as_float(ob[i]) * alpha);
                tmem_st32(tO + c * 32, ob);
              }
            }
            tmem_st32(tS, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
            tmem_st32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
            tmem_wait_st();
            tc_fence_before();
          }
        }
        // hand P_j to the MMA warp; met every step, also after a failed wait
        named_bar_sync(kPBar + (NT == 2 ? t : 0), 32 * 5);
      }
      if (n > 0) {
        ok = ok && mbar_wait(&o_done[t], static_cast<uint32_t>(oph & 1), wc);
        ok = __all_sync(0xffffffffu, ok);
        ++oph;
      }
      g0 += n;
      // ------------------------------------------------------------ epilogue
      const bool whole = unit->whole();
      if (!whole && unit->s0 == 0 && threadIdx.x == 0) {
        int* d = a.desc + blockIdx.x * kDesc;
        d[0] = pieces_of(*unit, *sh);
        d[1] = unit->b;
        d[2] = unit->h;
        d[3] = unit->j;
        d[4] = unit->s.q0;
        d[5] = nq;
        began = true;
      }
      if (!ok || !live) continue;
      const int sub = a.by_nsub.mod(unit->h);
      const int e = sub * a.gu + a.by_gu.mod(r);
      const bool row_ok = r < a.w * a.gu && tok < nq && e < a.G;
      tc_fence_after();
      __syncwarp();
      if (!whole) {
        // unnormalised O (relative to 2^m), m and l
        float* slot = a.ws + static_cast<size_t>(blockIdx.x * 2 + unit->slot()) * C::SLOT;
        float* orow = slot + (t * 128 + r) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ob[32];
          tmem_ld32_sync(tO + c * 32, ob);
          if (row_ok) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<uint4*>(orow + c * 32)[i] =
                  make_uint4(ob[4 * i], ob[4 * i + 1], ob[4 * i + 2], ob[4 * i + 3]);
          }
        }
        if (row_ok) {
          slot[NT * 128 * D + t * 128 + r] = m;
          slot[NT * 128 * (D + 1) + t * 128 + r] = l;
        }
      } else {
        const int hq = (a.by_nsub.div(unit->h)) * a.G + e;
        float f = 1.f;
        const float own = l;
        if (a.sinks && row_ok) f = add_sink(a.sinks[hq], m, l);
        const float inv = own != 0.f ? f / l : 0.f;
        const long long q = unit->s.q0 + tok;
        T* orow = static_cast<T*>(a.o) + q * a.os[0] + hq * a.os[1];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ob[32];
          tmem_ld32_sync(tO + c * 32, ob);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            // (a row that saw no key: O may never have been written)
            const float x0 = own != 0.f ? __uint_as_float(ob[2 * i]) * inv : 0.f;
            const float x1 = own != 0.f ? __uint_as_float(ob[2 * i + 1]) * inv : 0.f;
            w[i] = E::pack(x0, x1);
          }
          if (row_ok) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              reinterpret_cast<uint4*>(orow + c * 32)[i] =
                  make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        }
        if (row_ok && a.lse) a.lse[q * a.Hq + hq] = l != 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
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
    if (last_q >= 0) drain_wait(q_full, static_cast<uint32_t>(last_q & 1), kDrainNs);
    for (int i = max(0, fills - C::NS); i < fills; ++i)
      drain_wait(&full[i % C::NS], static_cast<uint32_t>((i / C::NS) & 1), kDrainNs);
  }
}

template <int D, bool BF16, int NT>
sdpa_status_t launch_tc_impl(Args& a, const CUtensorMap& tq, const CUtensorMap& tk,
                             const CUtensorMap& tv, int lg_box, const CacheBlocks& kb,
                             const CacheBlocks& vb, const LaunchEnv& env) {
  using C = TcCfg<D, NT>;
  auto kern = paged_tc_kernel<D, BF16, NT>;
  // The setmaxnreg split must fit the registers the kernel is launched with
  // (an increase beyond them would wait forever).
  static std::atomic<uint64_t> ready{0};  // devices on which this holds and is set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SDPA_ERR_CUDA;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(ready.load() & bit)) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return SDPA_ERR_CUDA;
    const long have = static_cast<long>((fa.numRegs + 7) & ~7) * C::THREADS;
    const long need = 32L * (C::SOFT_WARPS * static_cast<long>(kSoftmaxRegs) + 4L * kControlRegs);
    if (NT == 2 && have < need) return SDPA_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
        cudaSuccess)
      return SDPA_ERR_CUDA;
    ready.fetch_or(bit);
  }
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
  return launch_paged_merge(a, D, BF16 ? SDPA_BF16 : SDPA_F16, 128, NT, env.stream);
}

template <int D>
sdpa_status_t launch_tc(Args a, int dtype, const LaunchEnv& env) {
  fit_rows(a, 128);
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
  // A stride of a dimension of one element is never followed: any valid one.
  auto st = [](long long s, long long n) { return static_cast<uint64_t>(n > 1 ? s : D); };
  if (!encode_tiled_4d_box(&tq, dt, a.q, D, a.Hq, a.T, 1, 2, 64, static_cast<uint32_t>(a.gu),
                           static_cast<uint32_t>(a.w), st(a.qs[1], a.Hq), st(a.qs[0], a.T), D) ||
      !encode_row_blocks(&tk, dt, a.k, D / 64, a.page_size, kb.blocks, 1 << lg_box,
                         st(a.ks[2], a.page_size), ku) ||
      !encode_row_blocks(&tv, dt, a.v, D / 64, a.page_size, vb.blocks, 1 << lg_box,
                         st(a.vs[2], a.page_size), vu))
    return SDPA_ERR_CUDA;
  // More than 128 rows a sequence and head unit on average: two tiles a unit.
  // 16 sequences over 4096 keys, two tiles against one (us): 96 rows 69 and 61,
  // 192 rows 78 and 104.
  const bool two = static_cast<long long>(a.T) * a.gu > 128LL * a.B;
  if (two) fit_rows(a, 128, 2);
  if (bf16)
    return two ? launch_tc_impl<D, true, 2>(a, tq, tk, tv, lg_box, kb, vb, env)
               : launch_tc_impl<D, true, 1>(a, tq, tk, tv, lg_box, kb, vb, env);
  return two ? launch_tc_impl<D, false, 2>(a, tq, tk, tv, lg_box, kb, vb, env)
             : launch_tc_impl<D, false, 1>(a, tq, tk, tv, lg_box, kb, vb, env);
}

}  // namespace
}  // namespace paged

}  // namespace gb300

// paged_fp4_tc.cuh — attention of packed new tokens over the 4-bit paged cache
// on the 5th-generation tensor cores, for more rows a sequence than
// paged_fp4_decode.cu takes: the kernel and its launch, instantiated per head
// size in paged_fp4_tc_d64.cu and paged_fp4_tc_d128.cu.
//
// The rows, the division of the work, the issue loop and the softmax are those
// of paged_tc.cuh.  What differs:
//  - A loader warp brings the codes of the 128-key tiles to a staging ring
//    (tensor copies), and four warps widen them: a lane has a row of a tile,
//    reads its scales a tile ahead and writes it as fp16 where tcgen05.mma
//    reads it (128-byte swizzle).  Code times scale is exact in fp16 (fp4.cuh).
//    Rows past the length, or of a page that the table does not name, become
//    zeros there.
//  - Both products are in fp16 whatever the type of q.  The softmax warps lay
//    down the query tiles while the products of the unit before end (whole rows
//    by asynchronous copies, then each lane its own row in place): fp16 rows as
//    they are, bf16 ones times a power of two a row that brings the row's
//    largest to [2^14, 2^15) (what fp16 then drops is below 2^-39 of it); fp32
//    ones likewise as a sum of two fp16 parts (2^-22 of an element, or 2^-39 of
//    the row's largest), each multiplied with K, and so do their weights with V
//    (NT = 1).
//    A row's score factor is scale * gain / that power; its sign goes into the
//    row, so that the largest raw score is the largest score.
//  - Weights are 2^kHead at the reference maximum, so that fp16 holds them to
//    2^-11 relative down to 2^-18 of the largest, and to 2^-29 of it below that;
//    the two parts of fp32 calls (kRestScale) to 2^-22, and to 2^-41.
// Two query tiles a unit (NT = 2) share each widened tile.
//
// What bounds it: no unit is full (2048 tokens over 16384 keys, head_dim 128 /
// 64: tensor pipe 58 / 33 % active, issue 50 / 49 %, XU 29 / 33 %, ALU 34 / 31 %,
// shared-memory wavefronts 27 / 17 %).  In a build with clock stamps, which takes
// 1.5 and 1.1 times as long, the issuing warp waits for widened tiles (700 of 5000
// clocks a key tile, 910 of 2900) and never for weights (14, 16), and the widening
// warps are busy all the time, with their rows' pages and scales for a third of
// it: the chain of a widened tile sets the pace.
//
// 4096 tokens over 32768 keys, 32 heads over 8, head_dim 128, bf16: 1450 us, 1420
// TFLOP/s (the 16-bit cache's kernel 1190 to 1374 us).  Four ragged chunks of up to
// 700 tokens over 5000 keys: 150 us, 737 TFLOP/s.  Head_dim 64, 2048 tokens over
// 16384 keys: bf16 344 us (750 TFLOP/s), fp16 307 (840).  fp32, 4 x 300 tokens over
// 3000 keys: 180 us, and 54 for 8 heads of head_dim 64.  The steps (us, the first case): copies and widening
// by the same four warps 1975; a loader warp, scales read by the widening lanes,
// all scores in one load, and the registers split anew 1505; queries by the
// softmax warps, a row a lane in 16-byte loads, 1465; queries by asynchronous
// copies of whole rows 1530, but the chunks 156 -> 151, 300 tokens over themselves
// 28 -> 24, 8 x 16 tokens over 4096 keys 45 -> 37 and head_dim 64 (4 x 700 over
// 5000) 222 -> 200; these in a function of their own 1450.  The split of the
// registers counts (spills of the softmax or of the issuing warps; a thread of the
// softmax, control and widening warps): 184 / 80 / 64 (kept) 1452, 176 / 80 / 80 1449,
// 184 / 72 / 72 1473, 176 / 88 / 72 1519 to 1529; the four chunks 149, 148, 148, 152.
#pragma once

#include <atomic>
#include <type_traits>

#include "fp4.cuh"
#include "paged.cuh"
#include "paged_fp4.cuh"
#include "prefill_tc.cuh"

namespace gb300 {
namespace paged {
namespace {

template <int D, int NT, bool X2>
struct F4Cfg {
  static constexpr int CB = D / 64;        // 128-byte column blocks of a row
  static constexpr int TILE = 128 * D * 2;
  static constexpr int QN = X2 ? 2 : 1;    // fp16 parts of a query
  // Ring of widened K and V tiles in the order of their use: K_0 .. K_LA-1, then
  // V_j, K_j+LA for every j: S runs LA key tiles ahead of P V.
  static constexpr int NS = D == 64 ? 8 : NT == 2 || X2 ? 4 : 5;
  static constexpr int LA = NT == 2 ? 1 : 2;
  static constexpr int RING_OFF = NT * QN * TILE;
  // staging: a tile's codes, ST stages
  static constexpr int ROW = D / 2;
  static constexpr int SC = D / 16;  // bytes of a row's scales
  static constexpr int ST = 3;
  static constexpr int STAGE = 128 * ROW;
  static constexpr int STAGE_OFF = RING_OFF + NS * TILE;
  static constexpr int BAR_OFF = STAGE_OFF + ST * STAGE;
  // q_full, q_empty, full[NS], empty[NS], s_full[2], o_done[2], pv_done, drain,
  // st_full[ST], st_empty[ST]
  static constexpr int NBARS = 2 + 2 * NS + 2 + 2 + 1 + 1 + 2 * ST;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int SOFT_WARPS = 4 * NT;
  static constexpr int WARPS = SOFT_WARPS + 8;
  static constexpr int THREADS = 32 * WARPS;
  // registers of a thread by warpgroup (their sum is the launch's)
  static constexpr uint32_t SOFT_REGS = NT == 2 ? 184 : 232;
  static constexpr uint32_t CONTROL_REGS = NT == 2 ? 80 : 136;
  static constexpr uint32_t WIDEN_REGS = NT == 2 ? 64 : 136;
  static constexpr int SHARE_OFF = (MISC_OFF + 16 + 15) / 16 * 16;
  static constexpr int SCRATCH_OFF = SHARE_OFF + static_cast<int>(sizeof(Share));
  static constexpr int WALK_OFF = (SCRATCH_OFF + (WARPS + 1) * 8 + 15) / 16 * 16;
  static constexpr int UNIT_OFF =
      WALK_OFF + WARPS * static_cast<int>(sizeof(Walk<AttendUnits>));
  // (a softmax warp has its unit and the next one)
  static constexpr int SMEM =
      UNIT_OFF + (WARPS + SOFT_WARPS) * static_cast<int>(sizeof(Unit)) + 1024;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(STAGE % 512 == 0 && STAGE_OFF % 512 == 0, "swizzle atoms aligned");
  static constexpr uint32_t s_col(int i) { return static_cast<uint32_t>(i * 128); }
  static constexpr uint32_t o_col(int t) { return static_cast<uint32_t>(256 + t * D); }
  static constexpr int SLOT = 128 * NT * (D + 2);  // floats of a partial result
};

constexpr int kUnitSteps = 6;    // fixed cost of a unit in key tiles
constexpr uint32_t kPBar = 1;    // + t: softmax warps of tile t with the MMA warp
constexpr uint32_t kKBar = 3;    // stage helper with the MMA warp
// A row's weights are 2^kHead at its reference maximum, and their sum over a key
// tile at most kFusedSumLimit, past which the reference moves.  With 2^7 small
// weights were held to 2^-32 of the largest, but scores that grow along the keys
// would move it more often: 2 x 1024 tokens over 8192 such keys, 16 heads over 4,
// head_dim 128, 178 us and 203; where they do not grow, or grow at once, both take
// the same.
constexpr float kHead = 4.f;

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

// Tiles in ring order: the next one is K_k or V_v.
template <int LA>
struct Order {
  int n, k = 0, v = 0;
  __device__ __forceinline__ explicit Order(int tiles) : n(tiles) {}
  __device__ __forceinline__ bool more() const { return v < n; }
  __device__ __forceinline__ bool is_k() const { return k < n && k < v + LA; }
  __device__ __forceinline__ int tile() const { return is_k() ? k : v; }
  __device__ __forceinline__ void next() {
    if (is_k()) ++k; else ++v;
  }
};

// p = 2^(s f - m) of N raw scores as fp16 pairs, added to rs.  X2: and what fp16
// leaves of them, times kRestScale.  (4 x 300 fp32 tokens over 3000 keys, 8 heads of
// 64 / 32 over 8 of 128: 54 and 180 us; with the first part widened to fp32 and
// subtracted before the scaling 60 and 192; with p times kRestScale from the
// exponential on 57 and 181, and exponents near 16, whose rounding raised O's error
// from 5.5e-7 to 6.2e-7.)
template <bool X2, int N>
__device__ __forceinline__ void weights(const uint32_t (&s)[N], float f, float m, uint32_t* pk,
                                        uint32_t* lo, float& rs) {
  const uint64_t F = f2_pack(f, f), NM = f2_pack(-m, -m);
  uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const uint64_t X =
        f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), F, NM);
    float x0, x1;
    f2_unpack(X, x0, x1);
    const float p0 = ex2(x0), p1 = ex2(x1);
    acc[i & 1] = f2_add(acc[i & 1], f2_pack(p0, p1));
    const __half2 h = __floats2half2_rn(p0, p1);
    pk[i] = fp4::as_u32(h);
    if constexpr (X2)
      lo[i] = fp4::as_u32(__floats2half2_rn(rest_of(p0 * kRestScale, __low2half(h)),
                                            rest_of(p1 * kRestScale, __high2half(h))));
  }
  float t0, t1;
  f2_unpack(f2_add(acc[0], acc[1]), t0, t1);
  rs += t0 + t1;
}

// 32 bytes, a whole sector (p 32-byte aligned).
__device__ __forceinline__ void store32(float* p, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// A warp's 32 query rows (q: this lane's, or null; any: an address to name where
// there is none) times mul, -1, 0 or 1, as fp16 rows of the query tile `tile`.
// Returns two factors that a row's scores take for it (as one, 2^-127 would be
// subnormal).
template <typename T, int D, int NT>
__device__ __forceinline__ float2 lay_down(uint8_t* tile, int quarter, const T* q, const void* any,
                                        float mul) {
  constexpr bool X2 = sizeof(T) == 4;
  using C = F4Cfg<D, NT, X2>;
  const int lane = threadIdx.x & 31, r = quarter * 32 + lane;
  float f = 1.f, f2 = 1.f;
  // the power of two that brings `top` to [2^14, 2^15) (at most 2^126), into mul
  // and, inverted, f f2
  auto scale_by = [&](float top) {
    const int ex = static_cast<int>(__float_as_uint(top) >> 23);
    const int up = ex == 0 ? 126 : ex == 255 ? 0 : min(127 + 14 - ex, 126);
    mul *= __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
    f = __uint_as_float(static_cast<uint32_t>(127 - up / 2) << 23);
    f2 = __uint_as_float(static_cast<uint32_t>(127 - (up - up / 2)) << 23);
  };
  // 16-byte piece c of the fp16 row rr
  auto at = [&](int rr, int c) {
    return tile + (c >> 3) * (128 * 128) + (rr >> 3) * 1024 + (rr & 7) * 128 +
           (((c & 7) ^ (rr & 7)) * 16);
  };
  // The warp's rows as they are, whole rows at a time (zeros where there is
  // none), then each lane's own in place.  Pieces 2 c and 2 c + 1 of an fp32
  // row come where its fp16 parts' pieces c will be.
  constexpr int LR = D * sizeof(T) / 16;  // pieces of a row
  const unsigned long long src = reinterpret_cast<unsigned long long>(q);
#pragma unroll 2
  for (int i = 0; i < LR; ++i) {
    const int from = i * (32 / LR) + lane / LR, p = lane % LR;
    const unsigned long long s = __shfl_sync(0xffffffffu, src, from);
    const uint8_t* dst = X2 ? at(quarter * 32 + from, p >> 1) + (p & 1) * NT * C::TILE
                            : at(quarter * 32 + from, p);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)),
                 "l"(s ? s + p * 16 : reinterpret_cast<unsigned long long>(any)),
                 "r"(s ? 16 : 0)
                 : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  // the 8 elements of piece c
  auto load = [&](int c, float (&x)[8]) {
    if constexpr (X2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 v = *reinterpret_cast<const float4*>(at(r, c) + h * NT * C::TILE);
        x[4 * h] = v.x, x[4 * h + 1] = v.y, x[4 * h + 2] = v.z, x[4 * h + 3] = v.w;
      }
    } else {
      const uint4 raw = *reinterpret_cast<const uint4*>(at(r, c));
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = to_float(reinterpret_cast<const T*>(&raw)[k]);
    }
  };
  constexpr bool kHalf = std::is_same<T, __half>::value;
  if constexpr (!kHalf) {
    float top = 0.f;
#pragma unroll 2
    for (int c = 0; c < D / 8; ++c) {
      float x[8];
      load(c, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[k]));
    }
    scale_by(top);
  }
  if (!kHalf || mul != 1.f) {
#pragma unroll 2
    for (int c = 0; c < D / 8; ++c) {
      float x[8];
      load(c, x);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x0 = x[2 * k] * mul, x1 = x[2 * k + 1] * mul;
        const __half2 h = __floats2half2_rn(x0, x1);
        hi[k] = fp4::as_u32(h);
        if constexpr (X2)
          lo[k] = fp4::as_u32(__floats2half2_rn(x0 - __low2float(h), x1 - __high2float(h)));
      }
      uint8_t* dst = at(r, c);
      *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if constexpr (X2)
        *reinterpret_cast<uint4*>(dst + NT * C::TILE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  return make_float2(f, f2);
}
// Two tiles of head_dim 128 have it in a function of its own: the compiler's
// schedule of the softmax turns on what else that role's loop holds.  Apart and
// inside: 4096 tokens over 32768 keys 1450 and 1530 us; head_dim 64, 2048 tokens
// over 16384 keys, bf16 395 and 344, fp16 404 and 307; one tile, 8 x 16 tokens over
// 4096 keys 41 and 38.
template <typename T, int D, int NT>
__device__ __noinline__ float2 lay_down_apart(uint8_t* tile, int quarter, const T* q,
                                              const void* any, float mul) {
  return lay_down<T, D, NT>(tile, quarter, q, any, mul);
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(F4Cfg<D, NT, sizeof(T) == 4>::THREADS, 1)
    paged_fp4_tc_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const Args a,
                        const CodeMaps cm) {
  constexpr bool X2 = sizeof(T) == 4;
  using C = F4Cfg<D, NT, X2>;
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
  uint64_t* st_full = drain + 1;
  uint64_t* st_empty = st_full + C::ST;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  Share* sh = reinterpret_cast<Share*>(smem + C::SHARE_OFF);
  constexpr int kMma = C::SOFT_WARPS, kHelp = kMma + 1, kLoad = kMma + 2, kWiden = kMma + 4;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, C::SOFT_WARPS);
    mbar_init(q_empty, 1);
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&full[s], 4);
      mbar_init(&empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(pv_done, 1);
    mbar_init(drain, 1);
    for (int i = 0; i < C::ST; ++i) {
      mbar_init(&st_full[i], cm.lg >= 0 ? 1 : 33);  // (or 32 lanes' copies as well)
      mbar_init(&st_empty[i], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
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
  // Each warp walks the share on its own (state in shared memory).
  using W = Walk<AttendUnits>;
  W* walk = reinterpret_cast<W*>(smem + C::WALK_OFF) + warp;
  Unit* unit = reinterpret_cast<Unit*>(smem + C::UNIT_OFF) + warp;
  if (lane == 0) *walk = W(*sh);
  auto next_to = [&](Unit* u) {
    __syncwarp();
    bool more = false;
    if (lane == 0) more = walk->next(a, units, *sh, heads, u);
    return __shfl_sync(0xffffffffu, more ? 1 : 0, 0) != 0;
  };
  auto next = [&]() { return next_to(unit); };

  int fills = 0;  // loader: stages filled

  if (warp >= kWiden) {
    setmaxnreg_dec<C::WIDEN_REGS>();
    // -------------------------------------------------------------- widening
    const int w = warp - kWiden;
    const uint8_t* stages = smem + C::STAGE_OFF;
    constexpr int P = C::ROW / 16;  // 16-byte pieces of a row
    int g = 0;                      // ring slots filled
    bool ok = true;
    for (int it = 0; next(); ++it) {
      const Unit u = *unit;
      const TileGeo tg = tile_geo<NT>(a, u);
      const int kvh = a.by_nsub.div(u.h);
      // The scales of this lane's row, read a tile before they are needed, and
      // its page, looked up two before.
      Order<C::LA> order(tg.nmax), of_scales(tg.nmax), of_pages(tg.nmax);
      uint32_t sb_next[D / 64];
      int page = -1, row = 0;
      auto lookup = [&]() {
        const int key = (tg.s0 + of_pages.tile()) * 128 + w * 32 + lane;
        page = -1;
        if (of_pages.more()) {
          if (key < tg.nk) {
            const int i = a.by_page.div(key);
            row = key - i * a.page_size;
            page = a.table[u.b * a.table_stride + i];
          }
          of_pages.next();
        }
      };
      auto fetch_scales = [&]() {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) sb_next[i] = 0;
        if (page >= 0 && page < a.num_pages) {
          const bool is_k = of_scales.is_k();
          const char* src = (is_k ? a.k_scales : a.v_scales) + page * (is_k ? a.kss[0] : a.vss[0]) +
                            kvh * (is_k ? a.kss[1] : a.vss[1]) + row * (is_k ? a.kss[2] : a.vss[2]);
          if constexpr (D == 128) {
            const uint2 y = *reinterpret_cast<const uint2*>(src);
            sb_next[0] = y.x;
            sb_next[1] = y.y;
          } else {
            sb_next[0] = *reinterpret_cast<const uint32_t*>(src);
          }
        }
        of_scales.next();
        lookup();
      };
      lookup();
      fetch_scales();
      // ------------------------------------------------------- key tiles
      for (; order.more(); order.next()) {
        uint32_t sb[D / 64];  // the row's scales, four a word
#pragma unroll
        for (int i = 0; i < D / 64; ++i) sb[i] = sb_next[i];
        fetch_scales();
        const int x = g % C::ST;
        const int s = g % C::NS, use = g / C::NS;
        ok = __all_sync(0xffffffffu,
                        ok && mbar_wait(&st_full[x], (g / C::ST) & 1, wc) &&
                            (use == 0 || mbar_wait(&empty[s], (use - 1) & 1, wc)));
        const int r = w * 32 + lane;
        const uint8_t* src = stages + x * C::STAGE + r * C::ROW;
        uint8_t* dst = sRing + s * C::TILE + (r >> 3) * (C::CB * 1024) + (r & 7) * 128;
        uint4 codes[P];
#pragma unroll
        for (int c = 0; c < P; ++c) {  // (pieces swapped by row: see the maps' swizzle)
          const int pc = P == 4 ? c ^ ((lane >> 1) & 3) : c ^ ((lane >> 2) & 1);
          codes[c] = *reinterpret_cast<const uint4*>(src + pc * 16);
        }
        if (ok) {
#pragma unroll
          for (int c = 0; c < P; ++c) {  // 32 codes, two scales
            const uint4 x = codes[c];
            const __half2 sc = fp4::as_half2(fp4::scales_f16(sb[c >> 1] >> (16 * (c & 1))));
            const __half2 s0 = __low2half2(sc), s1 = __high2half2(sc);
            const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // 8 elements: a 16-byte piece
              uint32_t o[4];
              fp4::codes_f16(wd[k], o);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                o[i] = fp4::as_u32(__hmul2(fp4::as_half2(o[i]), k < 2 ? s0 : s1));
              const int piece = (c & 1) * 4 + k;
              *reinterpret_cast<uint4*>(dst + (c >> 1) * 1024 + ((piece ^ (r & 7)) * 16)) =
                  make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[s]);
          mbar_arrive(&st_empty[x]);
        }
        ++g;
      }
    }
  } else if (warp >= C::SOFT_WARPS) {
    setmaxnreg_dec<C::CONTROL_REGS>();
    if (warp == kMma) {
      // -------------------------------------------------------- MMA issuer
      constexpr uint32_t idS = idesc_f16(false, 128, 128, false, false);
      constexpr uint32_t idO = idesc_f16(false, 128, D, false, true);
      const uint64_t q_desc = sdesc(smem_addr(sQ), 16, 1024, kSwizzle128B);
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
        const uint32_t kd = k_lo + static_cast<uint32_t>((s * C::TILE) >> 4);
#pragma unroll
        for (int p = C::QN - 1; p >= 0; --p) {  // (the small part first)
          const uint32_t qd = q_lo + static_cast<uint32_t>(((p * NT + t) * C::TILE) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t qo = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
            const uint32_t ko = ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4;
            mma_f16_ss_elect(tmem + C::s_col(i), desc(q_hi, qd + qo), desc(k_hi, kd + ko), idS,
                             kk > 0 || p < C::QN - 1 ? 1u : 0u, 1u);
          }
        }
      };
      // O_t += P V, P in slot i, V in ring slot s, keys in groups of 16.  X2: the
      // weights' second part lies 64 columns on and has an O of its own (in the
      // place of tile 1's): it is kRestScale times larger, and half as many sums are
      // rounded at O's size.
      auto issue_pv = [&](int t, int i, int s, bool first, int groups) {
        const uint32_t vd = v_lo + static_cast<uint32_t>((s * C::TILE) >> 4);
#pragma unroll
        for (int p = 0; p < C::QN; ++p)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_ts_elect(tmem + C::o_col(X2 ? p : t), tmem + C::s_col(i) + p * 64 + kk * 8,
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
        named_bar_sync(kKBar, 64);  // Q and K_0 are there
        tc_fence_after();
        if constexpr (NT == 2) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t >= tg.nt) continue;
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
              if (!waited) {  // V_j and K_j+1 are there
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
              named_bar_sync(kKBar, 64);  // V_j and K_j+2 are there
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
    } else if (warp == kLoad) {
      // ---------------------------------------------------------- loader
      // Codes of the tiles in ring order to the staging ring.  Boxes past the
      // length are not loaded: scales are zero there, so whatever codes a stage
      // holds widen to zero.
      bool ok = true;
      int g = 0;
      while (next()) {
        const Unit u = *unit;
        const TileGeo tg = tile_geo<NT>(a, u);
        const int kvh = a.by_nsub.div(u.h);
        const int* table = a.table + u.b * a.table_stride;
        struct Box {
          int page, row;  // as looked up (row -1: past the length); checked():
        };                // page -1 past the length, -2 not the cache's
        const int lg = max(cm.lg, 0);
        const int nbox = cm.lg < 0 ? 0 : 128 >> lg;
        auto lookup = [&](int j) {  // box `lane` of key tile j
          Box x{0, -1};
          const int key = (tg.s0 + j) * 128 + (lane << lg);
          if (j < tg.nmax && lane < nbox && key < tg.nk) {
            const int i = a.by_page.div(key);
            x.row = key - i * a.page_size;
            x.page = table[i];
          }
          return x;
        };
        auto checked = [&](Box x) {
          if (x.row < 0) {
            x.page = -1;
          } else if (x.page < 0 || x.page >= a.num_pages) {
            atomicExch(a.status, kStatusPageTable);
            x.page = -2;
          }
          return x;
        };
        auto load = [&](bool is_k, int j, const Box& x) {
          const int s = g % C::ST, use = g / C::ST;
          ok = __all_sync(0xffffffffu,
                          ok && (use == 0 || mbar_wait(&st_empty[s], (use - 1) & 1, wc)));
          if (!ok) return;
          uint8_t* dst = smem + C::STAGE_OFF + s * C::STAGE;
          const int key0 = (tg.s0 + j) * 128;
          if (cm.lg >= 0) {
            const int boxes = min(nbox, (tg.nk - key0 + (1 << lg) - 1) >> lg);
            if (lane == 0)
              mbar_arrive_expect_tx(&st_full[s], static_cast<uint32_t>(boxes * C::ROW) << lg);
            __syncwarp();
            if (x.page != -1)
              tma_load_4d(dst + (lane * C::ROW << lg), is_k ? &tmK : &tmV, &st_full[s], 0, x.row,
                          kvh * (is_k ? cm.k_head_mul : cm.v_head_mul),
                          x.page < 0 ? (is_k ? cm.k_no_page : cm.v_no_page)
                                     : x.page * (is_k ? cm.k_page_mul : cm.v_page_mul));
          } else {
            const char* codes = static_cast<const char*>(is_k ? a.k : a.v);
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const int r = i * 32 + lane, key = key0 + r;
              Box y{0, -1};
              if (key < tg.nk) {
                const int n = a.by_page.div(key);
                y.row = key - n * a.page_size;
                y.page = table[n];
              }
              y = checked(y);
              const char* src = y.page < 0 ? codes
                                           : codes + y.page * (is_k ? a.ks[0] : a.vs[0]) +
                                                 kvh * (is_k ? a.ks[1] : a.vs[1]) +
                                                 y.row * (is_k ? a.ks[2] : a.vs[2]);
#pragma unroll 1
              for (int c = 0; c < C::ROW / 16; ++c) {
                const int pc = C::ROW == 64 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 smem_addr(dst + r * C::ROW + pc * 16)),
                             "l"(src + (y.page < 0 ? 0 : c * 16)), "r"(y.page < 0 ? 0 : 16)
                             : "memory");
              }
            }
            if (lane == 0) mbar_arrive(&st_full[s]);
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                             smem_addr(&st_full[s]))
                         : "memory");
          }
          fills = ++g;
        };
        Box bx[C::LA + 1];  // boxes of tiles j .. j + LA
#pragma unroll
        for (int i = 0; i <= C::LA; ++i) bx[i] = lookup(i);
#pragma unroll
        for (int i = 0; i < C::LA; ++i)
          if (ok && i < tg.nmax) load(true, i, checked(bx[i]));
        for (int j = 0; ok && j < tg.nmax; ++j) {
          const Box nx = lookup(j + C::LA + 1);
          load(false, j, checked(bx[0]));
          if (ok && j + C::LA < tg.nmax) load(true, j + C::LA, checked(bx[C::LA]));
#pragma unroll
          for (int i = 0; i < C::LA; ++i) bx[i] = bx[i + 1];
          bx[C::LA] = nx;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kHelp) {
      // ------------------------------------------------------ stage helper
      // Waits for the tiles that the MMA warp's next products read and meets
      // the MMA warp (the same number of times, also after a failed wait).
      bool ok = true;
      int p0 = 0;
      auto landed = [&](int p) {
        ok = ok && mbar_wait(&full[p % C::NS], static_cast<uint32_t>((p / C::NS) & 1), wc);
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
          landed(p0 + tg.v_pos<C::LA>(j));
          if (j + C::LA < tg.nmax) landed(p0 + tg.k_pos<C::LA>(j + C::LA));
          __syncwarp();
          named_bar_sync(kKBar, 64);
        }
        p0 += 2 * tg.nmax;
      }
    }
  } else {
    setmaxnreg_inc<C::SOFT_REGS>();
    // --------------------------------------------------------------- softmax
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lane_off + C::o_col(t);
    bool ok = true;
    int g0 = 0;   // steps of earlier units (NT = 2: of this tile)
    int oph = 0;  // phases of o_done[t] consumed
    bool began = false;  // this CTA wrote its descriptor
    // Row r of the unit's query tile t as fp16 (see the top), while the products
    // of the unit before end; returns the row's score factor.
    auto load_q = [&](const Unit& u, int it) {
      const TileGeo tg = tile_geo<NT>(a, u);
      const int kvh = a.by_nsub.div(u.h), e = a.by_nsub.mod(u.h) * a.gu + a.by_gu.mod(r);
      const int tok = (u.j * NT + t) * a.w + a.by_gu.div(r);
      const T* q = r < a.w * a.gu && tok < u.s.nq && e < a.G
                       ? static_cast<const T*>(a.q) + (u.s.q0 + tok) * a.qs[0] +
                             static_cast<long long>(kvh * a.G + e) * a.qs[1]
                       : nullptr;
      const float sc = a.sl2 * (a.k_gain ? a.k_gain[kvh] : 1.f);
      const float mul = sc < 0.f ? -1.f : sc == 0.f ? 0.f : 1.f;
      float f = sc == 0.f ? 1.f : fabsf(sc);
      if (it > 0) ok = ok && mbar_wait(q_empty, (it - 1) & 1, wc);
      ok = __all_sync(0xffffffffu, ok);
      if (t < tg.nt) {
        constexpr auto lay = D == 128 && NT == 2 ? lay_down_apart<T, D, NT> : lay_down<T, D, NT>;
        const float2 x = lay(sQ + t * C::TILE, warp & 3, q, a.q, mul);
        f = f * x.x * x.y;
        fence_proxy_async_shared();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      return fmaxf(f, 0x1p-149f);  // (never 0, which would make a hidden score, -inf, NaN)
    };
    Unit* const units2 = reinterpret_cast<Unit*>(smem + C::UNIT_OFF) + C::WARPS;
    bool more = next_to(unit);
    float f_next = 1.f;
    if (more) f_next = load_q(*unit, 0);
    for (int it = 0; more; ++it) {
      Unit* const unit = (it & 1) ? units2 + warp
                                  : reinterpret_cast<Unit*>(smem + C::UNIT_OFF) + warp;
      Unit* const after = (it & 1) ? reinterpret_cast<Unit*>(smem + C::UNIT_OFF) + warp
                                   : units2 + warp;
      const TileGeo tg = tile_geo<NT>(a, *unit);
      const float f = f_next;
      if (t >= tg.nt) {
        more = next_to(after);
        if (more) f_next = load_q(*after, it + 1);
        continue;
      }
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
            const int vis = limit - j * 128;  // visible keys of the row in this tile
            const bool edge = __any_sync(0xffffffffu, vis < 128);
            // (the weights take the scores' registers; X2 has none left for
            // all of them at once, and a moved reference reads them again)
            constexpr int N = X2 ? 64 : 128;
            uint32_t s[N];
            auto scores = [&](int c) {  // scores c * N .. + N - 1
              __syncwarp();
              if constexpr (X2)
                tmem_ld2x32_sync(tS + c * 64, tS + c * 64 + 32,
                                 *reinterpret_cast<uint32_t(*)[32]>(&s[0]),
                                 *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
              else
                tmem_ld4x32_sync(tS, tS + 32, tS + 64, tS + 96,
                                 *reinterpret_cast<uint32_t(*)[32]>(&s[0]),
                                 *reinterpret_cast<uint32_t(*)[32]>(&s[32]),
                                 *reinterpret_cast<uint32_t(*)[32]>(&s[N - 64]),
                                 *reinterpret_cast<uint32_t(*)[32]>(&s[N - 32]));
              if (edge) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                  if (c * N + i >= vis) s[i] = 0xff800000u;  // -inf
              }
            };
            float alpha = 1.f, rs = 0.f;
            uint32_t pk[64], lo[X2 ? 64 : 1];
            bool resc = !(m > -INFINITY);
            if (!__all_sync(0xffffffffu, resc)) {
#pragma unroll
              for (int c = 0; c < 128 / N; ++c) {
                scores(c);
                weights<X2>(s, f, m == -INFINITY ? 0.f : m, pk + c * 32, lo + (X2 ? c * 32 : 0),
                            rs);
              }
              resc = resc || !(rs <= kFusedSumLimit);
            }
            if (__any_sync(0xffffffffu, resc)) {
              float mx = -INFINITY;
#pragma unroll 1
              for (int c = 0; c < 128 / N; ++c) {
                scores(c);
                mx = fmaxf(mx, row_max_raw(s));
              }
              mx = mx * f - kHead;  // -inf: no visible key
              if (resc && mx > -INFINITY) {
                alpha = ex2(m - mx);  // 0 when m = -inf
                m = mx;
              }
              rs = 0.f;
#pragma unroll
              for (int c = 0; c < 128 / N; ++c) {
                scores(c);
                weights<X2>(s, f, m == -INFINITY ? 0.f : m, pk + c * 32, lo + (X2 ? c * 32 : 0),
                            rs);
              }
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
#pragma unroll 1
              for (int c = 0; c < C::QN * D / 32; ++c) {
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
            if constexpr (X2) {
              tmem_st32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&lo[0]));
              tmem_st32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&lo[32]));
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        // hand P_j to the MMA warp; met every step, also after a failed wait
        named_bar_sync(kPBar + (NT == 2 ? t : 0), 32 * 5);
      }
      more = next_to(after);
      if (more) f_next = load_q(*after, it + 1);
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
      const int kvh = a.by_nsub.div(unit->h), sub = a.by_nsub.mod(unit->h);
      const int e = sub * a.gu + a.by_gu.mod(r);
      const bool row_ok = r < a.w * a.gu && tok < nq && e < a.G;
      auto load_o = [&](int c, uint32_t (&x)[32]) {  // columns c * 32 .. + 31
        tmem_ld32_sync(tO + c * 32, x);
        if constexpr (X2) {
          uint32_t y[32];
          tmem_ld32_sync(tO + D + c * 32, y);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            x[i] = __float_as_uint(
                fmaf(__uint_as_float(y[i]), 1.f / kRestScale, __uint_as_float(x[i])));
        }
      };
      tc_fence_after();
      __syncwarp();
      if (!whole) {
        // unnormalised O (relative to 2^m, without the gain), m and l
        float* slot = a.ws + static_cast<size_t>(blockIdx.x * 2 + unit->slot()) * C::SLOT;
        float* orow = slot + (t * 128 + r) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ob[32];
          load_o(c, ob);
          if (row_ok) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) store32(orow + c * 32 + i, ob + i);
          }
        }
        if (row_ok) {
          slot[NT * 128 * D + t * 128 + r] = m;
          slot[NT * 128 * (D + 1) + t * 128 + r] = l;
        }
      } else {
        const int hq = kvh * a.G + e;
        float z = 1.f;
        const float own = l;
        if (a.sinks && row_ok) z = add_sink(a.sinks[hq], m, l);
        // (apart from the gain: a sum of weights times its inverse, or over it,
        // would be past fp32's range where O is not)
        const float inv = own != 0.f ? z / l : 0.f;
        const float gain = a.v_gain ? a.v_gain[kvh] : 1.f;
        const long long q = unit->s.q0 + tok;
        T* orow = static_cast<T*>(a.o) + q * a.os[0] + hq * a.os[1];
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ob[32];
          load_o(c, ob);
          // (a row that saw no key: O may never have been written)
          float x[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            x[i] = own != 0.f ? __uint_as_float(ob[i]) * inv * gain : 0.f;
          if (row_ok) {
            if constexpr (X2) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                reinterpret_cast<float4*>(orow + c * 32)[i] =
                    make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            } else {
              using E = Elem<std::is_same<T, __nv_bfloat16>::value>;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                reinterpret_cast<uint4*>(orow + c * 32)[i] =
                    make_uint4(E::pack(x[8 * i], x[8 * i + 1]), E::pack(x[8 * i + 2], x[8 * i + 3]),
                               E::pack(x[8 * i + 4], x[8 * i + 5]),
                               E::pack(x[8 * i + 6], x[8 * i + 7]));
            }
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
    // a role gave up: every copy that was asked for lands before the CTA exits
    for (int i = max(0, fills - C::ST); i < fills; ++i)
      drain_wait(&st_full[i % C::ST], static_cast<uint32_t>((i / C::ST) & 1), kDrainNs);
  }
}

template <typename T, int D, int NT>
sdpa_status_t launch_f4(Args& a, const LaunchEnv& env) {
  using C = F4Cfg<D, NT, sizeof(T) == 4>;
  auto kern = paged_fp4_tc_kernel<T, D, NT>;
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
    const long need = 32L * (C::SOFT_WARPS * static_cast<long>(C::SOFT_REGS) +
                             4L * C::CONTROL_REGS + 4L * C::WIDEN_REGS);
    if (have < need) return SDPA_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
        cudaSuccess)
      return SDPA_ERR_CUDA;
    ready.fetch_or(bit);
  }
  a.nctas = a.max_ctas < env.num_sms ? a.max_ctas : env.num_sms;
  CUtensorMap tk = {}, tv = {};
  const CodeMaps cm = encode_code_maps(
      a, D / 2, 7, D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B, &tk, &tv);
  const sdpa_status_t st = launch_overlapped(kern, dim3(static_cast<unsigned>(a.nctas)), C::THREADS,
                                             C::SMEM, env.stream, tk, tv, a, cm);
  if (st != SDPA_OK) return st;
  const int dtype = sizeof(T) == 4                      ? SDPA_F32
                    : std::is_same<T, __half>::value ? SDPA_F16
                                                     : SDPA_BF16;
  return launch_paged_merge(a, D, dtype, 128, NT, env.stream);
}

template <int D>
sdpa_status_t launch_fp4_tc(Args a, int dtype, const LaunchEnv& env) {
  fit_rows(a, 128);
  if (dtype == SDPA_F32) return launch_f4<float, D, 1>(a, env);
  // More than 128 rows a sequence and head unit on average: two tiles a unit.
  // 16 sequences over 4096 keys, one tile against two (us): 96 rows 62 and 74, 128
  // rows 64 and 76, 144 rows 102 and 89, 256 rows 105 and 97.
  const bool two = static_cast<long long>(a.T) * a.gu > 128LL * a.B;
  if (two) fit_rows(a, 128, 2);
  if (dtype == SDPA_F16)
    return two ? launch_f4<__half, D, 2>(a, env) : launch_f4<__half, D, 1>(a, env);
  return two ? launch_f4<__nv_bfloat16, D, 2>(a, env) : launch_f4<__nv_bfloat16, D, 1>(a, env);
}

}  // namespace
}  // namespace paged

}  // namespace gb300

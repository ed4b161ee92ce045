// paged_fp4_decode.cu — attention over the 4-bit paged cache where a sequence
// has few query rows (single tokens: the heads of a kv head), 8 or 16 rows of
// (token, head) a unit; every element type, head_dim 64/128.
//
// A key and kv head is 2 (D / 2 + D / 16) bytes, 3.6 times fewer than in 16
// bits, so the widening of its 2 D codes is what a kernel has to keep beside
// HBM: 41 elements a clock and SM at 6.7 TB/s.  Widened tiles in shared memory
// for tcgen05.mma would be written and read again at 2 bytes an element, more
// than its bandwidth.  So the codes become operand fragments in registers, one
// conversion and one multiplication by the scale for two elements, and go
// straight into mma.sync (a quarter of its rate is enough):
//     S^T  = K Q^T     M = 16 keys, N = 8 rows, K = 16 dims a step
//     O^T += V^T P^T   M = 16 dims, N = 8 rows, K = 16 keys a step
//  - K: a lane reads a quarter row, 16 bytes; which elements form a step is
//    free as long as Q's fragments, laid out once a unit, agree.
//  - V: a lane reads the same D / 8 elements of four keys; two shifts and two
//    three-input logic operations a word pair up the codes of two keys before
//    they are widened, so no transpose is needed.
//  - P: from S^T's layout to its operand's by movmatrix.
// Products of codes and scales are exact in fp16 (fp4.cuh).  fp16 queries enter
// as they are; bf16 ones times a power of two a row that brings the row's
// largest to 2^14 (what fp16 then drops is below 2^-39 of it); fp32 ones as a
// sum of two fp16 parts, likewise scaled (2^-22 of an element, or 2^-39 of the
// row's largest), and so do their weights.
// Weights are 2^(x - m + 7) against a reference maximum m that moves only when a
// score passes it by 8.  fp16 then holds them to 2^-11 relative down to 2^-21 of
// the largest, and to 2^-32 of it below; two parts (kRestScale) to 2^-22 relative,
// or 2^-44.  (A second part for 16-bit calls too would be half as many
// mma.sync again, for an O that is then rounded to 16 bits.)
// The gains enter with the score factor and, last, with the output.
//
// A CTA of 8 warps walks its share of the line of 256-key tiles (paged.cuh); a
// warp has 32 keys of a tile and a ring of its own in shared memory, filled by
// asynchronous copies one step ahead (head_dim 128; 64: three, in as many
// bytes), so nothing but the end of a unit meets a CTA barrier.
//
// 8 sequences of 32768 keys, 32 heads over 8, head_dim 128, bf16: 75.5 us a call,
// 4.0 TB/s, of which this kernel 71.5.  No unit is full: issue 62 % of the slots
// (380 instructions a warp for 16 keys: 110 scores, 124 values, 29 softmax, the
// rest copies and lookups), the ALU pipe, which converts the codes, 56 %, DRAM
// 62 % of the copy rate; of 14.7 resident warps an SM most wait for their turn
// (1.2 for each instruction issued), fixed latencies (1.1) or the conversions'
// pipe (0.9), memory least (0.3).  What brought it there (us): cp.async by each
// lane 115, by rows of neighbouring heads 102, tensor copies 90, copies issued
// without a loop over lanes and a merge over the whole grid 81, overlapped launches
// 77.  A ring of three stages instead of two, three CTAs an SM (80 registers, spills) and
// the next unit's copies beside the last one's end gave nothing or cost time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "fp4.cuh"
#include "paged.cuh"
#include "paged_fp4.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace paged {
namespace {

constexpr int kT = 256;
constexpr int kWarps = kT / 32;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kHead = 7.f;    // weights are 2^kHead at the reference maximum
constexpr float kLimit = 15.f;  // and at most 2^kLimit

template <int D>
struct Cfg {
  static constexpr int ROW = D / 2;   // bytes of a row's codes
  static constexpr int SC = D / 16;   // of its scales
  static constexpr int V_OFF = 32 * ROW;  // a warp's 32 keys: K, V, scales of K and V
  static constexpr int KS_OFF = 2 * V_OFF;
  static constexpr int VS_OFF = KS_OFF + 32 * SC;
  static constexpr int CELL = VS_OFF + 32 * SC;
  static constexpr int NS = D == 128 ? 2 : 4;
  static constexpr int RING = kWarps * NS * CELL;
  static constexpr int SMEM = RING + 512;
  static_assert(CELL % 128 == 0 && (D == 64 || CELL % 512 == 0), "swizzle atoms aligned");
};

// Row of a 16-key group in which slot s (row of an operand fragment) keeps its
// key.  A lane of the value product reads slots 2 t, 2 t + 1, 2 t + 8, 2 t + 9, of
// the score product slots g and g + 8, and neither may meet a bank twice:
// D = 128: 64-byte rows under the 64-byte swizzle (16-byte piece c of row r at
// c ^ (r / 2 % 4)); D = 64: 32-byte rows as they are.
template <int D>
__device__ __forceinline__ int even_row(int t) {  // slot 2 t
  return D == 128 ? (t & 1) + 2 * (t & 2) : t;    // 0 1 4 5; 0 1 2 3
}
template <int D>
__device__ __forceinline__ int odd_row(int t) {  // slot 2 t + 1
  return even_row<D>(t) ^ (D == 128 ? 3 : 6);    // 3 2 7 6; 6 7 4 5
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > limit_ns) break;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The same with nothing to add to.
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Issued by one lane of a warp in step: a tensor copy, and the bytes that a
// barrier's phase waits for (operands the same in every lane; a branch on the
// lane would have the copy issued in a loop over lanes).
__device__ __forceinline__ void tma_load_4d_elect(void* dst, const CUtensorMap* map, uint64_t* bar,
                                                  int c1, int c2, int c3) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];\n\t}\n" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void mbar_expect_elect(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;\n\t}\n" ::"r"(
          smem_addr(bar)),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ uint32_t mul2(uint32_t x, __half2 s) {
  return fp4::as_u32(__hmul2(fp4::as_half2(x), s));
}
// Four bytes of code pairs as fp16 pairs times s.
__device__ __forceinline__ void widen4(uint32_t w, __half2 s, uint32_t (&o)[4]) {
  fp4::codes_f16(w, o);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = mul2(o[i], s);
}
__device__ __forceinline__ float wide(float x) { return x; }
__device__ __forceinline__ float wide(__half x) { return __half2float(x); }
__device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put4(float* p, const float4& v) {
  *reinterpret_cast<float4*>(p) = v;
}
__device__ __forceinline__ void put2(float* p, const float2& v) {
  *reinterpret_cast<float2*>(p) = v;
}
__device__ __forceinline__ void put2(__half* p, const float2& v) {
  *reinterpret_cast<__half2*>(p) = __floats2half2_rn(v.x, v.y);
}
__device__ __forceinline__ void put2(__nv_bfloat16* p, const float2& v) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}
__device__ __forceinline__ void put4(__half* p, const float4& v) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2(fp4::as_u32(__floats2half2_rn(v.x, v.y)), fp4::as_u32(__floats2half2_rn(v.z, v.w)));
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, const float4& v) {
  __nv_bfloat162 x[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(x);
}

// NT: row tiles of 8.  hw: 2^lg_hw kv heads are a unit, a warp's keys and head
// are number warp >> lg_hw and warp & (hw - 1).
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kT, NT == 1 && sizeof(T) == 2 ? 2 : 1)
    paged_fp4_decode_kernel(const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const Args a,
                            const CodeMaps cm, const int lg_hw) {
  using C = Cfg<D>;
  constexpr int NR = 8 * NT;
  constexpr bool kSplit = sizeof(T) == 4;
  constexpr int QN = kSplit ? 2 : 1;  // fp16 parts of a query
  constexpr int KW = D / 32;          // words of a lane's part of a K row
  constexpr int VW = D / 64;          // and of its part of a V row
  constexpr int MT = D / 16;          // 16-row tiles of O^T
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long scratch[kWarps];
  __shared__ Share sh;
  __shared__ float s_m[kWarps][NR], s_l[kWarps][NR];
  __shared__ uint64_t s_full[kWarps][C::NS];
  __shared__ int s_abort;
  uint8_t* smem = smem_raw + ((512u - (smem_addr(smem_raw) & 511u)) & 511u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int hw = 1 << lg_hw, lg_tile = 8 - lg_hw;
  uint8_t* ring = smem + warp * (C::NS * C::CELL);
  uint64_t* full = s_full[warp];
  if (lane == 0) {
    for (int i = 0; i < C::NS; ++i) mbar_init(&full[i], 1);
    if (warp == 0) s_abort = 0;
    fence_mbar_init();
  }
  const WaitCtl wc{a.wait_ns, &s_abort, a.status};
  griddep_launch_dependents();
  griddep_wait();
  const AttendUnits units{a.by_w, lg_tile, a.causal, 1};
  const int heads = ((a.Hkv + hw - 1) >> lg_hw) * a.nsub;
  plan_share<kT>(a, units, heads, 1, scratch, &sh);  // (ends with a CTA barrier)
  if (tid == 0) a.desc[blockIdx.x * kDesc] = 0;
  Walk<AttendUnits> walk(sh);
  Unit u;
  // ring slots filled and read (their stage and the parity of its barrier)
  int fill = 0, read = 0;
  uint32_t read_par = 0;
  bool ok_wait = true;
  while (walk.next(a, units, sh, heads, &u)) {
    const int h0 = a.by_nsub.div(u.h) << lg_hw, e0 = a.by_nsub.mod(u.h) * a.gu;
    const int kvh = h0 + (warp & (hw - 1));  // this warp's head (it may be past the last)
    const bool head_ok = kvh < a.Hkv;
    const int tok0 = u.j * a.w;
    auto row_ok = [&](int h, int c) {
      const int tk = a.by_gu.div(c);
      return h < a.Hkv && c < a.gu * a.w && tok0 + tk < u.s.nq && e0 + a.by_gu.mod(c) < a.G;
    };
    // ------------------------------------------------------------- copies
    // Lane i looks up key i of its warp's 32 a step before their copies, copies
    // its scales, and brings the box of codes that begins there.
    const int sub = warp >> lg_hw;
    int nx_page = -1, nx_row = 0;
    auto lookup = [&](int step) {
      const int key = (step << lg_tile) + sub * 32 + lane;
      nx_page = -1;
      if (head_ok && step < u.s1 && key < u.s.nk) {
        const int i = a.by_page.div(key);
        nx_row = key - i * a.page_size;
        nx_page = a.table[u.b * a.table_stride + i];
        if (nx_page < 0 || nx_page >= a.num_pages) nx_page = -2;
      }
    };
    const char* ksc = a.k_scales + kvh * a.kss[1];
    const char* vsc = a.v_scales + kvh * a.vss[1];
    auto copy_scales = [&](uint8_t* dst, const char* src, bool ok) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_addr(dst)), "l"(src),
                   "n"(C::SC), "r"(ok ? C::SC : 0)
                   : "memory");
    };
    auto copy = [&](int step) {  // (every call commits one group of copies)
      if (step < u.s1) {
        if (nx_page == -2) atomicExch(a.status, kStatusPageTable);
        const bool own = nx_page >= 0;
        uint8_t* cell = ring + fill * C::CELL;
        copy_scales(cell + C::KS_OFF + lane * C::SC,
                    own ? ksc + nx_page * a.kss[0] + nx_row * a.kss[2] : a.k_scales, own);
        copy_scales(cell + C::VS_OFF + lane * C::SC,
                    own ? vsc + nx_page * a.vss[0] + nx_row * a.vss[2] : a.v_scales, own);
        if (cm.lg >= 0) {
          const int keys = head_ok ? u.s.nk - ((step << lg_tile) + sub * 32) : 0;
          const int boxes = keys <= 0 ? 0 : min(32 >> cm.lg, (keys + (1 << cm.lg) - 1) >> cm.lg);
          mbar_expect_elect(&full[fill], static_cast<uint32_t>(boxes * 2 * C::ROW) << cm.lg);
#pragma unroll 1
          for (int i = 0; i < boxes; ++i) {
            const int page = __shfl_sync(0xffffffffu, nx_page, i << cm.lg);
            const int row = __shfl_sync(0xffffffffu, nx_row, i << cm.lg);
            uint8_t* dst = cell + (i << cm.lg) * C::ROW;
            tma_load_4d_elect(dst, &tmK, &full[fill], row, kvh * cm.k_head_mul,
                              page >= 0 ? page * cm.k_page_mul : cm.k_no_page);
            tma_load_4d_elect(dst + C::V_OFF, &tmV, &full[fill], row, kvh * cm.v_head_mul,
                              page >= 0 ? page * cm.v_page_mul : cm.v_no_page);
          }
        } else {
          constexpr int P = C::ROW / 16;  // 16-byte pieces of a row
          const long long ko = own ? nx_page * a.ks[0] + kvh * a.ks[1] + nx_row * a.ks[2] : -1;
          const long long vo = nx_page * a.vs[0] + kvh * a.vs[1] + nx_row * a.vs[2];
#pragma unroll 1
          for (int i = 0; i < P; ++i) {
            const int x = i * 32 + lane, r = x / P, c = x % P, pc = P == 4 ? c ^ ((r >> 1) & 3) : c;
            const long long k = __shfl_sync(0xffffffffu, ko, r);
            const long long v = __shfl_sync(0xffffffffu, vo, r);
            const char* src = static_cast<const char*>(a.k);
            uint8_t* dst = cell + r * C::ROW + pc * 16;
#pragma unroll 1
            for (int y = 0; y < 2; ++y) {
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)),
                           "l"(k >= 0 ? src + (y ? v : k) + c * 16 : src), "r"(k >= 0 ? 16 : 0)
                           : "memory");
              src = static_cast<const char*>(a.v);
              dst += C::V_OFF;
            }
          }
          if (lane == 0) mbar_arrive(&full[fill]);
        }
        fill = fill + 1 == C::NS ? 0 : fill + 1;
        lookup(step + 1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    lookup(u.s0);
#pragma unroll 1
    for (int i = 0; i < C::NS - 1; ++i) copy(u.s0 + i);
    // ------------------------------------------------------------ queries
    // Lane (g, t) has quarter t of row g (of each tile): steps of 4 elements.
    uint32_t q[QN][NT][D / 16][2];
    float f[NT][2];  // score factors of this lane's columns 2 t, 2 t + 1 of S
    int lim[NT][2];  // and their visible keys
    int lim_min = u.s.nk;
    const float gain = a.k_gain && head_ok ? a.k_gain[kvh] : 1.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int c = n * 8 + g;
      const bool ok = row_ok(kvh, c);
      const int tok = tok0 + a.by_gu.div(c);
      float x[D / 4];
#pragma unroll
      for (int i = 0; i < D / 4; ++i) x[i] = 0.f;
      if (ok) {
        const T* src = static_cast<const T*>(a.q) + (u.s.q0 + tok) * a.qs[0] +
                       (kvh * a.G + e0 + a.by_gu.mod(c)) * a.qs[1] + t * (D / 4);
        constexpr int N = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < D / 4; i += N) {
          const uint4 raw = *reinterpret_cast<const uint4*>(src + i);
          const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
          for (int k = 0; k < N; ++k) x[i + k] = wide(e[k]);
        }
      }
      float factor = ok ? a.sl2 * gain : 0.f;
      if constexpr (!std::is_same<T, __half>::value) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the power of two that brings `top` to [2^14, 2^15) (at most 2^126)
        const int ex = static_cast<int>(__float_as_uint(top) >> 23);
        int up = ex == 0 ? 126 : ex == 255 ? 0 : min(127 + 14 - ex, 126);
        const float mul = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[i] *= mul;
        // 2^-up (subnormal at 127): two factors
        factor *= __uint_as_float(static_cast<uint32_t>(127 - up / 2) << 23);
        factor *= __uint_as_float(static_cast<uint32_t>(127 - (up - up / 2)) << 23);
      }
#pragma unroll
      for (int i = 0; i < D / 4; i += 2) {
        const __half2 hi = __floats2half2_rn(x[i], x[i + 1]);
        q[0][n][i / 4][(i >> 1) & 1] = fp4::as_u32(hi);
        if constexpr (kSplit)
          q[1][n][i / 4][(i >> 1) & 1] = fp4::as_u32(
              __floats2half2_rn(x[i] - __low2float(hi), x[i + 1] - __high2float(hi)));
      }
      const int own = ok && a.causal ? min(u.s.nk, u.s.off + tok + 1) : u.s.nk;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        f[n][k] = __shfl_sync(0xffffffffu, factor, (2 * t + k) * 4);
        lim[n][k] = __shfl_sync(0xffffffffu, own, (2 * t + k) * 4);
        lim_min = min(lim_min, lim[n][k]);
      }
    }
    lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 1));
    lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 2));
    // per column: reference (x - mb are the weights' exponents), its alarm, sum
    float mb[NT][2], alarm[NT][2], l[NT][2];
    float o[NT][MT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        mb[n][k] = 0.f;
        alarm[n][k] = -INFINITY;  // no reference yet
        l[n][k] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[n][i][k] = 0.f;
    }
    // addresses in a cell: this lane's piece of K slots g (and g + 8, 8 rows on),
    // of V slots 2 t and 2 t + 1, and of their scales
    const int k_row = (g & 1) ? odd_row<D>(g >> 1) : even_row<D>(g >> 1);
    const int v_even = even_row<D>(t), v_odd = odd_row<D>(t);
    auto v_at = [&](int row) {
      return C::V_OFF + row * C::ROW +
             (D == 128 ? (((g >> 1) ^ ((row >> 1) & 3)) * 16 + (g & 1) * 8) : g * 4);
    };
    const int k_off = k_row * C::ROW + (D == 128 ? (t ^ ((k_row >> 1) & 3)) * 16 : t * 8);
    const int v_off[2] = {v_at(v_even), v_at(v_odd)};
    const int ks_off = C::KS_OFF + k_row * C::SC + (D == 128 ? 2 * t : t);
    const int vs_off[2] = {C::VS_OFF + v_even * C::SC + (D == 128 ? g : g >> 1),
                           C::VS_OFF + v_odd * C::SC + (D == 128 ? g : g >> 1)};
    // ------------------------------------------------------------- steps
#pragma unroll 1
    for (int step = u.s0; step < u.s1; ++step) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::NS - 2) : "memory");
      ok_wait = ok_wait && mbar_wait(&full[read], read_par, wc);
      __syncwarp();  // every lane's copies of this step have landed, and the last step is read
      copy(step + C::NS - 1);
      const int key0 = (step << lg_tile) + sub * 32;
      const uint8_t* st = ring + read * C::CELL;
      if (++read == C::NS) {
        read = 0;
        read_par ^= 1;
      }
      if (key0 >= u.s.nk || !head_ok) continue;
      float s[2][NT][4];
      {
        uint32_t w[2][2][KW];
        __half2 sc[2][2][2];
#pragma unroll
        for (int kg = 0; kg < 2; ++kg)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = kg * 16 + r * 8;
            const uint8_t* p = st + k_off + row * C::ROW;
            if constexpr (D == 128) {
              const uint4 x = *reinterpret_cast<const uint4*>(p);
              w[kg][r][0] = x.x;
              w[kg][r][1] = x.y;
              w[kg][r][2] = x.z;
              w[kg][r][3] = x.w;
              const __half2 h = fp4::as_half2(fp4::scales_f16(
                  *reinterpret_cast<const uint16_t*>(st + ks_off + row * C::SC)));
              sc[kg][r][0] = __low2half2(h);
              sc[kg][r][1] = __high2half2(h);
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(p);
              w[kg][r][0] = x.x;
              w[kg][r][1] = x.y;
              sc[kg][r][0] = sc[kg][r][1] =
                  __low2half2(fp4::as_half2(fp4::scales_f16(st[ks_off + row * C::SC])));
            }
          }
#pragma unroll
        for (int i = 0; i < KW; ++i)
#pragma unroll
          for (int kg = 0; kg < 2; ++kg) {
            uint32_t x[4], y[4];
            widen4(w[kg][0][i], sc[kg][0][i >> 1], x);
            widen4(w[kg][1][i], sc[kg][1][i >> 1], y);
#pragma unroll
            for (int p = QN - 1; p >= 0; --p)  // (the small part first)
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                if (i == 0 && p == QN - 1)
                  mma16816_first(s[kg][n], x[0], y[0], x[1], y[1], q[p][n][0][0], q[p][n][0][1]);
                else
                  mma16816(s[kg][n], x[0], y[0], x[1], y[1], q[p][n][2 * i][0],
                           q[p][n][2 * i][1]);
                mma16816(s[kg][n], x[2], y[2], x[3], y[3], q[p][n][2 * i + 1][0],
                         q[p][n][2 * i + 1][1]);
              }
          }
      }
      // exponents of the weights, x - mb; element k of a fragment: slot g + 8 (k / 2), column k & 1
      bool over = false;
#pragma unroll
      for (int kg = 0; kg < 2; ++kg)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[kg][n][k] = fmaf(s[kg][n][k], f[n][k & 1], -mb[n][k & 1]);
          }
      if (key0 + 32 > lim_min) {
#pragma unroll
        for (int kg = 0; kg < 2; ++kg)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (key0 + kg * 16 + (k >> 1) * 8 + k_row >= lim[n][k & 1]) s[kg][n][k] = -INFINITY;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float mx = fmaxf(fmaxf(s[0][n][k], s[0][n][k + 2]), fmaxf(s[1][n][k], s[1][n][k + 2]));
          over |= mx > alarm[n][k];
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float mx =
                fmaxf(fmaxf(s[0][n][k], s[0][n][k + 2]), fmaxf(s[1][n][k], s[1][n][k + 2]));
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            // (a column whose keys are all hidden keeps what it has)
            if (mx > alarm[n][k]) {
              const float by = mx - kHead;  // the exponents fall by it
              const float fall = alarm[n][k] == -INFINITY ? 0.f : ex2(-by);
              mb[n][k] += by;
              alarm[n][k] = kLimit;
              l[n][k] *= fall;
#pragma unroll
              for (int kg = 0; kg < 2; ++kg) {
                s[kg][n][k] -= by;
                s[kg][n][k + 2] -= by;
              }
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[n][i][k] *= fall;
                o[n][i][k + 2] *= fall;
              }
            }
          }
      }
      uint32_t p[QN][2][NT][2];
#pragma unroll
      for (int kg = 0; kg < 2; ++kg)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = ex2(s[kg][n][2 * h]), p1 = ex2(s[kg][n][2 * h + 1]);
            l[n][0] += p0;
            l[n][1] += p1;
            const __half2 hi = __floats2half2_rn(p0, p1);
            p[0][kg][n][h] = transpose8(fp4::as_u32(hi));
            if constexpr (kSplit)
              p[1][kg][n][h] = transpose8(
                  fp4::as_u32(__floats2half2_rn(rest_of(p0 * kRestScale, __low2half(hi)),
                                                rest_of(p1 * kRestScale, __high2half(hi)))));
          }
#pragma unroll
      for (int kg = 0; kg < 2; ++kg) {
        uint32_t w[4][VW];
        uint32_t sb[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // slots 2 t, 2 t + 1, 2 t + 8, 2 t + 9
          const int row = kg * 16 + (k >> 1) * 8;
          const uint8_t* x = st + v_off[k & 1] + row * C::ROW;
          if constexpr (D == 128) {
            const uint2 y = *reinterpret_cast<const uint2*>(x);
            w[k][0] = y.x;
            w[k][1] = y.y;
          } else {
            w[k][0] = *reinterpret_cast<const uint32_t*>(x);
          }
          sb[k] = st[vs_off[k & 1] + row * C::SC];
        }
        const __half2 s0 = fp4::as_half2(fp4::scales_f16(__byte_perm(sb[0], sb[1], 0x0040)));
        const __half2 s1 = fp4::as_half2(fp4::scales_f16(__byte_perm(sb[2], sb[3], 0x0040)));
#pragma unroll
        for (int i = 0; i < VW; ++i) {
          // the codes of two keys side by side: even elements, odd elements
          uint32_t e0_[4], o0_[4], e1_[4], o1_[4];
          constexpr uint32_t L = 0x0f0f0f0fu, H = 0xf0f0f0f0u;
          widen4((w[0][i] & L) | ((w[1][i] << 4) & H), s0, e0_);
          widen4(((w[0][i] >> 4) & L) | (w[1][i] & H), s0, o0_);
          widen4((w[2][i] & L) | ((w[3][i] << 4) & H), s1, e1_);
          widen4(((w[2][i] >> 4) & L) | (w[3][i] & H), s1, o1_);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(o[n][4 * i + b], e0_[b], o0_[b], e1_[b], o1_[b], p[0][kg][n][0],
                       p[0][kg][n][1]);
            if constexpr (kSplit) {
              // the weights' second part, times values scaled back (multiples of
              // 2^-10 below 2^12: exact in fp16 at 2^-12 of them too)
              const __half2 z = __float2half2_rn(1.f / kRestScale);
              const uint32_t e0 = mul2(e0_[b], z), o0 = mul2(o0_[b], z), e1 = mul2(e1_[b], z),
                             o1 = mul2(o1_[b], z);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816(o[n][4 * i + b], e0, o0, e1, o1, p[1][kg][n][0], p[1][kg][n][1]);
            }
          }
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // ------------------------------------------- the warps' results meet
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], d);
        if (g == 0) {
          s_m[warp][n * 8 + 2 * t + k] = mb[n][k];
          s_l[warp][n * 8 + 2 * t + k] = l[n][k];
        }
      }
    __syncthreads();  // every warp has left its loop: the rings are free
    float* red = reinterpret_cast<float*>(smem);
    // lane (g, t): elements D / 8 * g .. of columns 2 t and 2 t + 1
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float* dst = red + (warp * NR + n * 8 + 2 * t + k) * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < MT; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) =
              make_float4(o[n][i][k], o[n][i][k + 2], o[n][i + 1][k], o[n][i + 1][k + 2]);
      }
    __syncthreads();
    const bool whole = u.whole();
    const int rows = NR << lg_hw;
    float* slot = a.ws + static_cast<size_t>(blockIdx.x * 2 + u.slot()) * (rows * (D + 2));
    for (int x = tid; x < rows * (D / 4); x += kT) {
      const int row = x / (D / 4), col = (x % (D / 4)) * 4;
      const int hi = row / NR, c = row % NR, head = h0 + hi;
      if (!row_ok(head, c)) continue;
      float M = -INFINITY, L = 0.f;
      for (int w = hi; w < kWarps; w += hw)
        if (s_l[w][c] != 0.f) M = fmaxf(M, s_m[w][c]);
      float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = hi; w < kWarps; w += hw) {
        if (s_l[w][c] == 0.f) continue;  // this warp's keys are not seen
        const float z = ex2(s_m[w][c] - (M == -INFINITY ? 0.f : M));
        const float4 v = *reinterpret_cast<const float4*>(red + (w * NR + c) * D + col);
        L = fmaf(s_l[w][c], z, L);
        r.x = fmaf(v.x, z, r.x);
        r.y = fmaf(v.y, z, r.y);
        r.z = fmaf(v.z, z, r.z);
        r.w = fmaf(v.w, z, r.w);
      }
      if (!whole) {  // (without the gain, which may be large)
        put4(slot + row * D + col, r);
        if (col == 0) {
          slot[rows * D + row] = M;
          slot[rows * (D + 1) + row] = L;
        }
        continue;
      }
      const long long tok = u.s.q0 + tok0 + a.by_gu.div(c);
      const int hq = head * a.G + e0 + a.by_gu.mod(c);
      float z = L != 0.f ? 1.f : 0.f;
      if (a.sinks) z *= add_sink(a.sinks[hq], M, L);
      z = L != 0.f ? z / L : 0.f;
      const float gain = a.v_gain ? a.v_gain[head] : 1.f;
      put4(static_cast<T*>(a.o) + tok * a.os[0] + hq * a.os[1] + col,
           make_float4(r.x * z * gain, r.y * z * gain, r.z * z * gain, r.w * z * gain));
      if (a.lse && col == 0)
        a.lse[tok * a.Hq + hq] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
    }
    if (!whole && u.s0 == 0 && tid == 0) {
      int* d = a.desc + blockIdx.x * kDesc;
      d[0] = pieces_of(u, sh);
      d[1] = u.b;
      d[2] = u.h;
      d[3] = u.j;
      d[4] = u.s.q0;
      d[5] = u.s.nq;
    }
    fence_proxy_async_shared();
    __syncthreads();  // the rings are free for the next unit
  }
  // a wait that gave up: what was asked for lands before the CTA leaves
  if (s_abort && lane == 0)
    for (int i = 0; i < C::NS; ++i) {
      drain_wait(&full[i], 0, kDrainNs / 8);
      drain_wait(&full[i], 1, kDrainNs / 8);
    }
}

constexpr int kMaxUnits = 1024;  // CTAs of a call, at most

// Joins the partial results of the units that CTAs began and did not finish
// (their descriptors are compacted first): M = max of the m's, weights 2^(m -
// M), in the order of the pieces.  Bound by the latency of its three dependent
// loads, so a row is spread over as many warps of a block as leave all warps of
// the grid with at most one row (8 units of 32 rows in 38 pieces, cold: 13 us
// against 19 with 16 blocks a unit; 16 units of 16 rows in 19 pieces: 10 against
// 13).
template <typename T, int D>
__global__ void __launch_bounds__(kT) paged_fp4_merge_kernel(const Args a, const int nr,
                                                             const int lg_hw) {
  constexpr int E = D / 32;  // columns of a lane
  __shared__ short s_unit[kMaxUnits];
  __shared__ bool s_cut[kMaxUnits];
  __shared__ int s_count;
  __shared__ float s_ml[kWarps][2], s_o[kWarps][D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  for (int c = tid; c < a.nctas; c += kT) s_cut[c] = a.desc[c * kDesc] != 0;
  __syncthreads();
  if (warp == 0) {  // (the same order in every block)
    int count = 0;
    for (int c0 = 0; c0 < a.nctas; c0 += 32) {
      const int c = c0 + lane;
      const bool cut = c < a.nctas && s_cut[c];
      const uint32_t all = __ballot_sync(0xffffffffu, cut);
      if (cut) s_unit[count + __popc(all & ((1u << lane) - 1))] = static_cast<short>(c);
      count += __popc(all);
    }
    if (lane == 0) s_count = count;
  }
  __syncthreads();
  const int live = a.gu * a.w;  // rows of a head's tile
  const int per = live << lg_hw;
  const int tasks = s_count * per, warps = gridDim.x * kWarps;
  int lg = 3;  // log2 of the warps of a row
  while (lg > 0 && (tasks << lg) > warps) --lg;
  const int part = warp & ((1 << lg) - 1), step = 1 << lg;
  const int rows = nr << lg_hw;
  const size_t slot_floats = static_cast<size_t>(rows) * (D + 2);
  for (int base = blockIdx.x * (kWarps >> lg); base < tasks; base += warps >> lg) {
    const int task = base + (warp >> lg);
    bool ok = task < tasks;
    int c = 0, row = 0, tok = 0, hq = 0, head = 0, n = 0;
    const int* d = a.desc;
    if (ok) {
      const int unit = task / per, x = task - unit * per;
      c = s_unit[unit];
      d = a.desc + c * kDesc;
      n = d[0];
      const int hi = x / live, r = x - hi * live;
      row = hi * nr + r;
      const int g = a.by_gu.div(r), e = a.by_nsub.mod(d[2]) * a.gu + r - g * a.gu;
      head = (a.by_nsub.div(d[2]) << lg_hw) + hi;
      tok = d[3] * a.w + g;
      hq = head * a.G + e;
      ok = tok < d[5] && e < a.G && head < a.Hkv;
    }
    float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.f;
    if (ok) {
      auto piece = [&](int p) {
        return a.ws +
               (p == 0 ? static_cast<size_t>(c * 2 + 1) : static_cast<size_t>((c + p) * 2)) *
                   slot_floats;
      };
      for (int p0 = part; p0 < n; p0 += 32 * step) {  // 32 pieces of this warp's
        const int mine = p0 + lane * step;
        float m = -INFINITY, l = 0.f;
        if (mine < n) {
          const float* s = piece(mine);
          m = s[static_cast<size_t>(rows) * D + row];
          l = s[static_cast<size_t>(rows) * (D + 1) + row];
        }
        if (l == 0.f) m = -INFINITY;  // (a piece whose keys the row does not see)
        float mn = m;
#pragma unroll
        for (int i = 16; i >= 1; i >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, i));
        mn = fmaxf(mn, M);
        const float fall = M == -INFINITY ? 0.f : ex2(M - mn);
        M = mn;
        const float wgt = l != 0.f ? ex2(m - (mn == -INFINITY ? 0.f : mn)) : 0.f;
        L *= fall;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] *= fall;
        const int count = min(32, (n - p0 + step - 1) >> lg);
#pragma unroll 5
        for (int k = 0; k < count; ++k) {
          const float w = __shfl_sync(0xffffffffu, wgt, k), lk = __shfl_sync(0xffffffffu, l, k);
          if (lk != 0.f) {
            const float* s = piece(p0 + k * step) + static_cast<size_t>(row) * D + lane * E;
            L = fmaf(lk, w, L);
#pragma unroll
            for (int i = 0; i < E; i += 2) {
              const float2 v = *reinterpret_cast<const float2*>(s + i);
              acc[i] = fmaf(v.x, w, acc[i]);
              acc[i + 1] = fmaf(v.y, w, acc[i + 1]);
            }
          }
        }
      }
    }
    if (lg > 0) {  // the parts of a row meet
      if (lane == 0) {
        s_ml[warp][0] = M;
        s_ml[warp][1] = L;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) s_o[warp][lane * E + i] = acc[i];
      __syncthreads();
      if (part == 0) {
        for (int w = 1; w < step; ++w) {
          const float m = s_ml[warp + w][0], l = s_ml[warp + w][1];
          if (l == 0.f) continue;
          const float mn = fmaxf(M, m);
          const float f = M == -INFINITY ? 0.f : ex2(M - mn), z = ex2(m - (mn == -INFINITY ? 0.f : mn));
          L = L * f + l * z;
#pragma unroll
          for (int i = 0; i < E; ++i) acc[i] = acc[i] * f + s_o[warp + w][lane * E + i] * z;
          M = mn;
        }
      }
    }
    if (ok && part == 0) {
      const bool any = L != 0.f;
      float f = 1.f;
      if (a.sinks) f = add_sink(a.sinks[hq], M, L);
      const float inv = any ? f / L : 0.f;
      const float gain = a.v_gain ? a.v_gain[head] : 1.f;
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] *= inv;
      const long long q = d[4] + tok;
      T* o = static_cast<T*>(a.o) + q * a.os[0] + hq * a.os[1] + lane * E;
      if constexpr (E == 4) {
        put4(o, make_float4(acc[0] * gain, acc[1] * gain, acc[2] * gain, acc[3] * gain));
      } else {
        put2(o, make_float2(acc[0] * gain, acc[1] * gain));
      }
      if (a.lse && lane == 0) a.lse[q * a.Hq + hq] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
    }
    if (lg > 0) __syncthreads();  // (the meeting place is read)
  }
}

// Kv heads of a unit (log2).  Where a token's heads lie next to one another,
// a run of up to 4 heads' rows is read as one piece of memory (8 x 32768 keys of
// 8 kv heads, 1, 2, 4 and 8 heads a unit: 128, 88, 81 and 87 us); where a head's
// tokens do, one.
int unit_heads(const Args& a) {
  int lg = 2;
  if (a.ks[1] >= a.ks[2] && a.page_size > 1) return 0;
  // (the last unit's missing heads leave warps idle)
  while (lg > 0 && (a.Hkv >> lg == 0 || (a.Hkv % (1 << lg) != 0 && a.Hkv < (4 << lg)))) --lg;
  return lg;
}

template <typename T, int D, int NT>
sdpa_status_t launch(Args& a, const LaunchEnv& env) {
  auto kern = paged_fp4_decode_kernel<T, D, NT>;
  constexpr int smem = std::max(Cfg<D>::SMEM, kWarps * 8 * NT * D * 4 + 512);
  fit_rows(a, 8 * NT);
  a.nctas = std::min(a.max_ctas, (NT == 1 && sizeof(T) == 2 ? 2 : 1) * env.num_sms);
  if (a.nctas > kMaxUnits) a.nctas = kMaxUnits;
  const int lg_hw = unit_heads(a);
  if (!allow_smem<paged_fp4_decode_kernel<T, D, NT>>(smem)) return SDPA_ERR_CUDA;
  CUtensorMap tk = {}, tv = {};
  const CodeMaps cm = encode_code_maps(
      a, D / 2, 5, D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE, &tk, &tv);
  const sdpa_status_t st =
      launch_overlapped(kern, dim3(a.nctas), kT, smem, env.stream, tk, tv, a, cm, lg_hw);
  if (st != SDPA_OK) return st;
  return launch_overlapped(paged_fp4_merge_kernel<T, D>, dim3(2 * env.num_sms), kT, 0, env.stream,
                           a, 8 * NT, lg_hw);
}

template <typename T>
sdpa_status_t by_size(Args& a, int head_dim, int rows, const LaunchEnv& env) {
  if (head_dim == 64) return rows == 8 ? launch<T, 64, 1>(a, env) : launch<T, 64, 2>(a, env);
  return rows == 8 ? launch<T, 128, 1>(a, env) : launch<T, 128, 2>(a, env);
}

}  // namespace
}  // namespace paged

int paged_fp4_decode_rows(const paged::Args& a, int dtype) {
  // 16 sequences of 4096 keys (us): 8 rows a tile, 16 rows, the kernel of many
  // rows.  32 heads over 8, head_dim 128, bf16: 8 rows a sequence and kv head 35,
  // 42, 56; 16 rows 52, 46, 56; 24 rows 71, 71, 56.  16 heads over 4, head_dim 64,
  // fp32, whose many-row kernel does twice the work: 8 rows 21, 27, 46; 16 rows
  // 29, 28, 46; 32 rows 45, 38, 47 (before fp32 weights kept their small parts;
  // since then, on other inputs, 4, 16 and 32 rows 21, 29 and 42, 36 rows, by the
  // other kernel, 47).  A step of single tokens and a long chunk goes by the average
  // and loses by it: 128 tokens over 512 keys and a chunk of 384 over 32768, 32 heads
  // over 8, bf16, 1434, in two calls 40 and 172.
  const long long rows = paged::call_rows(a);
  const int most = dtype == SDPA_F32 ? 32 : 16;
  return a.G > 16 ? 0 : a.G <= 8 && rows <= 8 ? 8 : rows <= most ? 16 : 0;
}

sdpa_status_t launch_paged_fp4_decode(paged::Args a, int head_dim, int dtype, int rows,
                                      const LaunchEnv& env) {
  using namespace paged;
  if (dtype == SDPA_F32) return by_size<float>(a, head_dim, rows, env);
  return dtype == SDPA_F16 ? by_size<__half>(a, head_dim, rows, env)
                           : by_size<__nv_bfloat16>(a, head_dim, rows, env);
}

}  // namespace gb300

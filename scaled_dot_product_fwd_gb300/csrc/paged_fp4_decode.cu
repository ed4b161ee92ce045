// paged_fp4_decode.cu — attention over the 4-bit paged cache where a sequence
// has few query rows (single tokens: the heads of a kv head), up to 8 or 16
// rows of (token, head) a unit; every element type, head_dim 64/128.
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
// sum of two fp16 parts, likewise scaled (22 bits), and so do their weights.
// Weights are 2^(x - m + 7) against a reference maximum m that moves only when a
// score passes it by 8 (fp16 then holds them to 2^-11 relative down to 2^-21 of
// the largest).  The gains enter with the score factor and the output.
//
// A CTA of 8 warps walks its share of the line of 256-key tiles (paged.cuh); a
// warp has 32 keys of a tile and a ring of its own in shared memory, filled by
// asynchronous copies two steps ahead, so nothing but the end of a unit meets
// a CTA barrier.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "fp4.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace paged {
namespace {

constexpr int kT = 256;
constexpr int kWarps = kT / 32;
constexpr int kLgTile = 8;  // keys of a CTA's step (32 a warp)
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kHead = 7.f;    // weights are 2^kHead at the reference maximum
constexpr float kLimit = 15.f;  // and at most 2^kLimit

template <int D>
struct Cfg {
  static constexpr int ROW = D / 2;                 // bytes of a row's codes
  static constexpr int SC = D / 16;                 // of its scales
  static constexpr int STAGE = 32 * 2 * (ROW + SC);  // a warp's 32 keys: K, V, scales
  static constexpr int NS = D == 128 ? 3 : 5;
  static constexpr int V_OFF = 32 * ROW;
  static constexpr int KS_OFF = 2 * V_OFF;
  static constexpr int VS_OFF = KS_OFF + 32 * SC;
  static constexpr int SMEM = kWarps * NS * STAGE;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
__device__ __forceinline__ void put4(__half* p, const float4& v) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2(fp4::as_u32(__floats2half2_rn(v.x, v.y)), fp4::as_u32(__floats2half2_rn(v.z, v.w)));
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, const float4& v) {
  __nv_bfloat162 x[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(x);
}

// NT: row tiles of 8.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kT, NT == 1 && sizeof(T) == 2 ? 2 : 1)
    paged_fp4_decode_kernel(const Args a) {
  using C = Cfg<D>;
  constexpr int NR = 8 * NT;
  constexpr bool kSplit = sizeof(T) == 4;
  constexpr int QN = kSplit ? 2 : 1;  // fp16 parts of a query
  constexpr int KW = D / 32;          // words of a lane's part of a K row
  constexpr int VW = D / 64;          // and of its part of a V row
  constexpr int MT = D / 16;          // 16-row tiles of O^T
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ long long scratch[kWarps];
  __shared__ Share sh;
  __shared__ float s_m[kWarps][NR], s_l[kWarps][NR];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem_raw + warp * C::NS * C::STAGE;
  griddep_launch_dependents();
  const AttendUnits units{a.by_w, kLgTile, a.causal, 1};
  const int heads = a.Hkv * a.nsub;
  plan_share<kT>(a, units, heads, 1, scratch, &sh);
  if (tid == 0) a.desc[blockIdx.x * kDesc] = 0;
  Walk<AttendUnits> walk(sh);
  Unit u;
  while (walk.next(a, units, sh, heads, &u)) {
    const int kvh = a.by_nsub.div(u.h), e0 = a.by_nsub.mod(u.h) * a.gu;
    const int tok0 = u.j * a.w;
    auto row_ok = [&](int c) {
      const int tk = a.by_gu.div(c);
      return c < a.gu * a.w && tok0 + tk < u.s.nq && e0 + a.by_gu.mod(c) < a.G;
    };
    // ------------------------------------------------------------- copies
    // A lane looks up one key of its warp's 32, a step before its copies.
    const char* kc = static_cast<const char*>(a.k) + kvh * a.ks[1];
    const char* vc = static_cast<const char*>(a.v) + kvh * a.vs[1];
    const char* ksc = a.k_scales + kvh * a.kss[1];
    const char* vsc = a.v_scales + kvh * a.vss[1];
    int nx_page = -1, nx_row = 0;
    auto lookup = [&](int step) {
      const int key = (step << kLgTile) + warp * 32 + lane;
      nx_page = -1;
      if (step < u.s1 && key < u.s.nk) {
        const int i = a.by_page.div(key);
        nx_row = key - i * a.page_size;
        nx_page = a.table[u.b * a.table_stride + i];
        if (nx_page < 0 || nx_page >= a.num_pages) nx_page = -2;
      }
    };
    auto copy16 = [&](uint8_t* dst, const char* src, bool ok) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
                   "r"(ok ? 16 : 0)
                   : "memory");
    };
    auto copy_scales = [&](uint8_t* dst, const char* src, bool ok) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_addr(dst)), "l"(src),
                   "n"(C::SC), "r"(ok ? C::SC : 0)
                   : "memory");
    };
    auto copy = [&](int step) {  // (every call commits one group of copies)
      if (step < u.s1) {
        if (nx_page == -2) atomicExch(a.status, kStatusPageTable);
        const bool own = nx_page >= 0;
        const long long ko = own ? nx_page * a.ks[0] + nx_row * a.ks[2] : -1;
        const long long vo = own ? nx_page * a.vs[0] + nx_row * a.vs[2] : 0;
        uint8_t* st = ring + ((step - u.s0) % C::NS) * C::STAGE;
        constexpr int P = C::ROW / 16;  // 16-byte pieces of a row
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int x = i * 32 + lane, r = x / P, c = x % P;
          const long long k = __shfl_sync(0xffffffffu, ko, r), v = __shfl_sync(0xffffffffu, vo, r);
          copy16(st + r * C::ROW + c * 16, kc + (k >= 0 ? k + c * 16 : 0), k >= 0);
          // V rows: keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of 16 lie in rows t, t + 4,
          // t + 8, t + 12, and the halves of 64-byte rows 2 and 3 of four are
          // swapped, so that a warp's reads of four keys meet no bank twice
          const int pr = (r & 16) | ((r & 1) << 2) | (r & 8) | ((r >> 1) & 3);
          const int pc = P == 4 ? c ^ (pr & 2) : c;
          copy16(st + C::V_OFF + pr * C::ROW + pc * 16, vc + (k >= 0 ? v + c * 16 : 0), k >= 0);
        }
        const int pr = (lane & 16) | ((lane & 1) << 2) | (lane & 8) | ((lane >> 1) & 3);
        copy_scales(st + C::KS_OFF + lane * C::SC,
                    ksc + (own ? nx_page * a.kss[0] + nx_row * a.kss[2] : 0), own);
        copy_scales(st + C::VS_OFF + pr * C::SC,
                    vsc + (own ? nx_page * a.vss[0] + nx_row * a.vss[2] : 0), own);
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
    const float gain = a.k_gain ? a.k_gain[kvh] : 1.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int c = n * 8 + g;
      const bool ok = row_ok(c);
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
    const int v_off = C::V_OFF + t * C::ROW +
                      (D == 128 ? (((g >> 1) ^ (t & 2)) * 16 + (g & 1) * 8) : g * 4);
    const int vs_off = C::VS_OFF + t * C::SC + (D == 128 ? g : g >> 1);
    // ------------------------------------------------------------- steps
#pragma unroll 1
    for (int step = u.s0; step < u.s1; ++step) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::NS - 2) : "memory");
      __syncwarp();  // every lane's copies of this step have landed, and the last step is read
      copy(step + C::NS - 1);
      const int key0 = (step << kLgTile) + warp * 32;
      if (key0 >= u.s.nk) continue;
      const uint8_t* st = ring + ((step - u.s0) % C::NS) * C::STAGE;
      float s[2][NT][4];
#pragma unroll
      for (int kg = 0; kg < 2; ++kg) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[kg][n][k] = 0.f;
        uint32_t w[2][KW];
        __half2 sc[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = kg * 16 + r * 8 + g;
          const uint8_t* p = st + row * C::ROW + t * (C::ROW / 4);
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            w[r][0] = x.x;
            w[r][1] = x.y;
            w[r][2] = x.z;
            w[r][3] = x.w;
            const __half2 h = fp4::as_half2(
                fp4::scales_f16(*reinterpret_cast<const uint16_t*>(st + C::KS_OFF + row * 8 + 2 * t)));
            sc[r][0] = __low2half2(h);
            sc[r][1] = __high2half2(h);
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[r][0] = x.x;
            w[r][1] = x.y;
            sc[r][0] = sc[r][1] =
                __low2half2(fp4::as_half2(fp4::scales_f16(st[C::KS_OFF + row * 4 + t])));
          }
        }
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          uint32_t x[4], y[4];
          widen4(w[0][i], sc[0][i >> 1], x);
          widen4(w[1][i], sc[1][i >> 1], y);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < QN; ++p) {
              mma16816(s[kg][n], x[0], y[0], x[1], y[1], q[p][n][2 * i][0], q[p][n][2 * i][1]);
              mma16816(s[kg][n], x[2], y[2], x[3], y[3], q[p][n][2 * i + 1][0],
                       q[p][n][2 * i + 1][1]);
            }
        }
      }
      // exponents of the weights, x - mb; element k of a fragment: key g + 8 (k / 2), column k & 1
      bool over = false;
#pragma unroll
      for (int kg = 0; kg < 2; ++kg)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float x = fmaf(s[kg][n][k], f[n][k & 1], -mb[n][k & 1]);
            s[kg][n][k] = x;
          }
      if (key0 + 32 > lim_min) {
#pragma unroll
        for (int kg = 0; kg < 2; ++kg)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (key0 + kg * 16 + (k >> 1) * 8 + g >= lim[n][k & 1]) s[kg][n][k] = -INFINITY;
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
                  fp4::as_u32(__floats2half2_rn(p0 - __low2float(hi), p1 - __high2float(hi))));
          }
#pragma unroll
      for (int kg = 0; kg < 2; ++kg) {
        uint32_t w[4][VW];
        uint32_t sb[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // rows t + 4 k: keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
          const uint8_t* x = st + v_off + (kg * 16 + 4 * k) * C::ROW;
          if constexpr (D == 128) {
            const uint2 y = *reinterpret_cast<const uint2*>(x);
            w[k][0] = y.x;
            w[k][1] = y.y;
          } else {
            w[k][0] = *reinterpret_cast<const uint32_t*>(x);
          }
          sb[k] = st[vs_off + (kg * 16 + 4 * k) * C::SC];
        }
        const __half2 s0 = fp4::as_half2(fp4::scales_f16(sb[0] | (sb[1] << 8)));
        const __half2 s1 = fp4::as_half2(fp4::scales_f16(sb[2] | (sb[3] << 8)));
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
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int y = 0; y < QN; ++y)
                mma16816(o[n][4 * i + b], e0_[b], o0_[b], e1_[b], o1_[b], p[y][kg][n][0],
                         p[y][kg][n][1]);
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
    float* red = reinterpret_cast<float*>(smem_raw);
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
    const float v_gain = a.v_gain ? a.v_gain[kvh] : 1.f;
    float* slot = a.ws + static_cast<size_t>(blockIdx.x * 2 + u.slot()) * (NR * (D + 2));
    for (int x = tid; x < NR * (D / 4); x += kT) {
      const int c = x / (D / 4), col = (x % (D / 4)) * 4;
      if (!row_ok(c)) continue;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (s_l[w][c] != 0.f) M = fmaxf(M, s_m[w][c]);
      float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (s_l[w][c] == 0.f) continue;  // this warp's keys are not seen
        const float z = ex2(s_m[w][c] - (M == -INFINITY ? 0.f : M));
        const float4 v = *reinterpret_cast<const float4*>(red + (w * NR + c) * D + col);
        L = fmaf(s_l[w][c], z, L);
        r.x = fmaf(v.x, z, r.x);
        r.y = fmaf(v.y, z, r.y);
        r.z = fmaf(v.z, z, r.z);
        r.w = fmaf(v.w, z, r.w);
      }
      if (!whole) {
        put4(slot + c * D + col,
             make_float4(r.x * v_gain, r.y * v_gain, r.z * v_gain, r.w * v_gain));
        if (col == 0) {
          slot[NR * D + c] = M;
          slot[NR * (D + 1) + c] = L;
        }
        continue;
      }
      const long long tok = u.s.q0 + tok0 + a.by_gu.div(c);
      const int hq = kvh * a.G + e0 + a.by_gu.mod(c);
      float z = L != 0.f ? 1.f : 0.f;
      if (a.sinks) z *= add_sink(a.sinks[hq], M, L);
      z = L != 0.f ? z / L * v_gain : 0.f;
      put4(static_cast<T*>(a.o) + tok * a.os[0] + hq * a.os[1] + col,
           make_float4(r.x * z, r.y * z, r.z * z, r.w * z));
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
    __syncthreads();  // the rings are free for the next unit
  }
}

template <typename T, int D, int NT>
sdpa_status_t launch(Args& a, const LaunchEnv& env) {
  auto kern = paged_fp4_decode_kernel<T, D, NT>;
  constexpr int smem = std::max(Cfg<D>::SMEM, kWarps * 8 * NT * D * 4);
  fit_rows(a, 8 * NT);
  a.nctas = std::min(a.max_ctas, (NT == 1 && sizeof(T) == 2 ? 2 : 1) * env.num_sms);
  if (!allow_smem<paged_fp4_decode_kernel<T, D, NT>>(smem)) return SDPA_ERR_CUDA;
  kern<<<a.nctas, kT, smem, env.stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return SDPA_ERR_CUDA;
  const int dtype = sizeof(T) == 4                      ? SDPA_F32
                    : std::is_same<T, __half>::value ? SDPA_F16
                                                     : SDPA_BF16;
  return launch_paged_merge(a, D, dtype, 8 * NT, 1, env.stream);
}

template <typename T>
sdpa_status_t by_size(Args& a, int head_dim, int rows, const LaunchEnv& env) {
  if (head_dim == 64) return rows == 8 ? launch<T, 64, 1>(a, env) : launch<T, 64, 2>(a, env);
  return rows == 8 ? launch<T, 128, 1>(a, env) : launch<T, 128, 2>(a, env);
}

}  // namespace
}  // namespace paged

int paged_fp4_decode_rows(const paged::Args& a) {
  const long long rows = paged::call_rows(a);
  return a.G > 16 ? 0 : a.G <= 8 && rows <= 8 ? 8 : rows <= 16 ? 16 : 0;
}

sdpa_status_t launch_paged_fp4_decode(paged::Args a, int head_dim, int dtype, int rows,
                                      const LaunchEnv& env) {
  using namespace paged;
  if (dtype == SDPA_F32) return by_size<float>(a, head_dim, rows, env);
  return dtype == SDPA_F16 ? by_size<__half>(a, head_dim, rows, env)
                           : by_size<__nv_bfloat16>(a, head_dim, rows, env);
}

}  // namespace gb300

// paged_append.cu — a step's new tokens on their way to the paged cache: q
// rotated, k rotated and written to its page row, v written; and the same into
// the 4-bit cache, where the rows of k and v become codes and scales.
//
// Bound by HBM where there are many tokens (each row in and out once), by the
// chain of dependent loads (sequence, length, page; position, table) where
// there are few.  A warp takes rows of one token, D / 16 lanes a row
// (rotate.cuh), so the lookups are made once a warp, beside the rows' loads.
//
// Four chunks of up to 2048 tokens, 32 heads over 8, head_dim 128, fp16: 26 us
// (131 MB, 5.0 TB/s; the kernel alone 24), into the 4-bit cache 36 us (139 MB with
// the values read back, 3.9 TB/s), where the exact rotation of k and the quotients
// count too: true divisions 62, corrected products 47, three CTAs an SM 40, queries
// without the exact sums 38, overlapped launches 35 (35.8 with sums that are not
// finite kept apart).  There the issue slots are 70 % busy and no pipe above 51 %;
// the 20 resident warps an SM wait for their turn (1.9 for each instruction issued),
// the sums' and quotients' fixed latencies (1.4) and memory (0.9).  64 single tokens:
// 10 and 14 us a call, the host's.
#include <cuda_runtime.h>

#include <algorithm>

#include "fp4.cuh"
#include "paged.cuh"
#include "paged_append.cuh"
#include "ptx.cuh"
#include "rotate.cuh"

namespace gb300 {
namespace paged {
namespace {

using namespace rotary;

constexpr int kWarps = 8;

struct AppendArgs {
  Args a;
  Rotation rot;
  int times;   // groups of 32 * 16 / D rows that a warp takes
  int rows;    // rows of a token: q heads, k heads, v heads
  const char* k;
  const char* v;
  char* q_out;
  // byte strides: q, q_out, new k and v (token, head); pages (page, head, row)
  long long qi[2], qo[2], kn[2], vn[2], kb[3], vb[3];
  char* pages[2];
  // 4-bit cache
  char* scales[2];
  long long sb[2][3];
  const float* gain[2];
  char* value[2];  // k_out and v_out, or null
  long long vo[2];
};

__device__ __forceinline__ void put8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void get8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x;
  x[1] = a.y;
  x[2] = a.z;
  x[3] = a.w;
  x[4] = b.x;
  x[5] = b.y;
  x[6] = b.z;
  x[7] = b.w;
}

// x / d for r the reciprocal of d rounded once: the quotient x r, corrected by
// its exact remainder (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990).  One correction is within a unit of
// a product of two rounded numbers and, where d has 4 significant bits, meets
// every number of few bits that the quotient equals and passes none; the
// second leaves the quotient rounded to nearest.
template <int kSteps>
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float q0 = __fmul_rn(x, r);
  float q = q0;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) q = __fmaf_rn(__fmaf_rn(-q, d, x), r, q);
  if (kSteps > 1) return fabsf(q0) < INFINITY ? q : q0;  // (an infinity has no remainder)
  return q;
}

template <typename T, int D, bool kFp4>
__global__ void __launch_bounds__(kWarps * 32, kFp4 ? 3 : 4) paged_append_kernel(const AppendArgs w) {
  constexpr int U = D / 16;    // pieces of a row
  constexpr int RW = 32 / U;   // rows of a warp at a time
  const Args& a = w.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = lane % U;
  // a warp's rows in fp32 where 16 consecutive elements of a rotated row come
  // from two lanes
  __shared__ __align__(16) float s_rows[kFp4 ? kWarps * 512 : 4];
  griddep_launch_dependents();
  griddep_wait();
  const long long tt = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (tt >= a.T) return;
  const int t = static_cast<int>(tt);
  const int row0 = blockIdx.y * w.times * RW + lane / U;
  // (a group of the 4-bit cache is 16 consecutive elements)
  const Piece pc = piece_of<kFp4>(w.rot, D, u);
  const Piece plain = kFp4 ? Piece{16 * u, 16 * u + 8, false} : Piece{8 * u, D / 2 + 8 * u, false};
  // what row r is: 0 a query, 1 a key, 2 a value
  auto kind = [&](int r) { return r < a.Hq ? 0 : r < a.Hq + a.Hkv ? 1 : 2; };
  Raw<T> lo, hi, nlo, nhi;
  auto load = [&](int r, Raw<T>& x0, Raw<T>& x1) {
    if (r >= w.rows) return;
    const int kd = kind(r);
    const char* x = kd == 0   ? static_cast<const char*>(a.q) + t * w.qi[0] + r * w.qi[1]
                    : kd == 1 ? w.k + t * w.kn[0] + (r - a.Hq) * w.kn[1]
                              : w.v + t * w.vn[0] + (r - a.Hq - a.Hkv) * w.vn[1];
    const Piece p = kd == 2 ? plain : pc;
    x0 = load8(reinterpret_cast<const T*>(x) + p.lo);
    x1 = load8(reinterpret_cast<const T*>(x) + p.hi);
  };
  load(row0, lo, hi);
  const int b = find_seq(a, t, lane);
  if (b < 0) return;
  const Seq s = seq_of(a, b);
  // the token's position (seq_of ends the keys at the table's end, not this)
  const long long own = static_cast<long long>(max(a.lens[b], 0)) - s.nq + (t - s.q0);
  const long long pos = w.rot.positions ? w.rot.positions[t] : own;
  Angles ang = {};
  bool turned = pc.turned && pos >= 0 && pos < w.rot.len;
  if (turned) ang = load_angles(w.rot, pos, pc);
  if (pc.turned && !turned && u == 0 && (w.rot.positions || pos >= 0))
    atomicExch(a.status, kStatusPosition);
  int page = -1, prow = 0;
  if (own >= 0 && own < a.cap) {
    page = page_of(a, b, static_cast<int>(own));
    prow = a.by_page.mod(static_cast<int>(own));
  }
  for (int i = 0; i < w.times; ++i) {
    const int r = row0 + i * RW;
    if (i + 1 < w.times) load(r + RW, nlo, nhi);  // (on their way meanwhile)
    const bool live = r < w.rows;
    if (!kFp4 && !live) break;  // (so are the lane's later rows)
    const int kd = kind(r);
    const int h = r - (kd == 0 ? 0 : kd == 1 ? a.Hq : a.Hq + a.Hkv);
    const Piece p = kd == 2 ? plain : pc;
    Values x;
    const bool tn = turned && kd != 2;
    if (live && (tn || (kFp4 && kd != 0))) {
      widen8(lo, x.lo);
      widen8(hi, x.hi);
      if (tn) {
        if (kFp4 && kd == 1)
          turn_piece<kFp4>(x, ang, w.rot.interleaved, 1.f);
        else
          turn_piece<false>(x, ang, w.rot.interleaved, 1.f);
        lo = narrow8<T>(x.lo);
        hi = narrow8<T>(x.hi);
      }
    }
    if (live && (kd == 0 || !kFp4)) {
      char* dst = nullptr;
      if (kd == 0)
        dst = w.q_out + t * w.qo[0] + h * w.qo[1];
      else if (page >= 0)
        dst = w.pages[kd - 1] + page * (kd == 1 ? w.kb : w.vb)[0] +
              h * (kd == 1 ? w.kb : w.vb)[1] + prow * (kd == 1 ? w.kb : w.vb)[2];
      if (dst) {
        store8(reinterpret_cast<T*>(dst) + p.lo, lo);
        store8(reinterpret_cast<T*>(dst) + p.hi, hi);
      }
    }
    if constexpr (kFp4) {
      const bool mine = live && kd != 0;
      if (mine && tn) {  // the row as its type holds it
        widen8(lo, x.lo);
        widen8(hi, x.hi);
      }
      if (__any_sync(0xffffffffu, mine && p.hi != 16 * u + 8)) {
        float* row = s_rows + warp * 512 + (lane / U) * D;
        __syncwarp();
        if (mine) {
          put8(row + p.lo, x.lo);
          put8(row + p.hi, x.hi);
        }
        __syncwarp();
        if (mine) {
          get8(row + 16 * u, x.lo);
          get8(row + 16 * u + 8, x.hi);
        }
      }
      if (mine) {
        const int c = kd - 1;
        const float g = w.gain[c] ? w.gain[c][h] : 1.f;
        float top = 0.f;
        if (w.gain[c]) {
          const float rg = __frcp_rn(g);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x.lo[k] = quotient<2>(x.lo[k], g, rg);
            x.hi[k] = quotient<2>(x.hi[k], g, rg);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, fmaxf(fabsf(x.lo[k]), fabsf(x.hi[k])));
        float sc;
        const uint32_t sbyte = fp4::scale_of(top, &sc);
        const float rs = __frcp_rn(sc);
#pragma unroll
        for (int k = 0; k < 8; ++k) {  // (what is past the largest value ends there)
          x.lo[k] = quotient<1>(fminf(fmaxf(x.lo[k], -4096.f), 4096.f), sc, rs);
          x.hi[k] = quotient<1>(fminf(fmaxf(x.hi[k], -4096.f), 4096.f), sc, rs);
        }
        const uint32_t c0 = fp4::codes_of(x.lo), c1 = fp4::codes_of(x.hi);
        if (page >= 0) {
          const long long* st = c == 0 ? w.kb : w.vb;
          char* dst = w.pages[c] + page * st[0] + h * st[1] + prow * st[2] + 8 * u;
          *reinterpret_cast<uint2*>(dst) = make_uint2(c0, c1);
          w.scales[c][page * w.sb[c][0] + h * w.sb[c][1] + prow * w.sb[c][2] + u] =
              static_cast<char>(sbyte);
        }
        if (w.value[c]) {
          uint32_t f[8];
          fp4::codes_f16(c0, reinterpret_cast<uint32_t(&)[4]>(f[0]));
          fp4::codes_f16(c1, reinterpret_cast<uint32_t(&)[4]>(f[4]));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 y0 = __half22float2(fp4::as_half2(f[k]));
            const float2 y1 = __half22float2(fp4::as_half2(f[4 + k]));
            x.lo[2 * k] = y0.x * sc * g;
            x.lo[2 * k + 1] = y0.y * sc * g;
            x.hi[2 * k] = y1.x * sc * g;
            x.hi[2 * k + 1] = y1.y * sc * g;
          }
          T* dst = reinterpret_cast<T*>(w.value[c] + t * w.vo[0] + h * w.vo[1]) + 16 * u;
          store8(dst, narrow8<T>(x.lo));
          store8(dst + 8, narrow8<T>(x.hi));
        }
      }
    }
    lo = nlo;
    hi = nhi;
  }
}

template <typename T, int D, bool kFp4>
sdpa_status_t launch(AppendArgs& w, const LaunchEnv& env) {
  constexpr int RW = 512 / D;
  const long long blocks = (static_cast<long long>(w.a.T) + kWarps - 1) / kWarps;
  const int groups = (w.rows + RW - 1) / RW;
  // Groups of rows of a warp: one where the call is small (the shortest
  // chain), more where that still fills the GPU.  Four chunks of up to 2048
  // tokens, 32 heads over 8, head_dim 128: 2, 4, 6 and 12 groups 27.6, 27.4, 28.2
  // and 28.5 us, into the 4-bit cache, whose rows cost more, 44, 42, 40 and 40.
  int times = kFp4 ? 8 : 4;
  while (times > 1 && blocks * ((groups + times - 1) / times) < 8LL * env.num_sms) times >>= 1;
  times = std::max(times, (groups + 65534) / 65535);
  const int parts = (groups + times - 1) / times;
  times = (groups + parts - 1) / parts;  // (even shares)
  w.times = times;
  const dim3 grid(static_cast<unsigned>(blocks),
                  static_cast<unsigned>((groups + times - 1) / times));
  return launch_overlapped(paged_append_kernel<T, D, kFp4>, grid, kWarps * 32, 0, env.stream, w);
}

template <typename T>
sdpa_status_t by_dim(AppendArgs& w, int head_dim, bool fp4, const LaunchEnv& env) {
  if (head_dim == 64) return fp4 ? launch<T, 64, true>(w, env) : launch<T, 64, false>(w, env);
  return fp4 ? launch<T, 128, true>(w, env) : launch<T, 128, false>(w, env);
}

}  // namespace
}  // namespace paged

sdpa_status_t launch_paged_append(const paged::Args& a, int head_dim, int dtype,
                                  const paged::AppendIo& io, const LaunchEnv& env) {
  using namespace paged;
  const int es = dtype == SDPA_F32 ? 4 : 2;
  const int cs = io.fp4 ? 1 : es;  // bytes of the pages' stride unit
  AppendArgs w = {};
  w.a = a;
  w.rot = make_rotation(io.rotation);
  w.rows = a.Hq + 2 * a.Hkv;
  w.k = static_cast<const char*>(io.k);
  w.v = static_cast<const char*>(io.v);
  w.q_out = static_cast<char*>(io.q_out);
  for (int i = 0; i < 2; ++i) {
    w.qi[i] = a.qs[i] * es;
    w.qo[i] = a.os[i] * es;
    w.kn[i] = io.k_new_stride[i] * es;
    w.vn[i] = io.v_new_stride[i] * es;
  }
  for (int i = 0; i < 3; ++i) {
    w.kb[i] = a.ks[i] * cs;
    w.vb[i] = a.vs[i] * cs;
  }
  w.pages[0] = static_cast<char*>(io.fp4 ? io.fp4->k_codes : io.k_pages);
  w.pages[1] = static_cast<char*>(io.fp4 ? io.fp4->v_codes : io.v_pages);
  if (io.fp4) {
    w.scales[0] = static_cast<char*>(io.fp4->k_scales);
    w.scales[1] = static_cast<char*>(io.fp4->v_scales);
    for (int i = 0; i < 3; ++i) {
      w.sb[0][i] = io.fp4->k_scale_stride[i];
      w.sb[1][i] = io.fp4->v_scale_stride[i];
    }
    w.gain[0] = io.fp4->k_gain;
    w.gain[1] = io.fp4->v_gain;
    w.value[0] = static_cast<char*>(io.k_out);
    w.value[1] = static_cast<char*>(io.v_out);
    for (int i = 0; i < 2; ++i) w.vo[i] = io.out_stride ? io.out_stride[i] * es : 0;
  }
  if (dtype == SDPA_F32) return by_dim<float>(w, head_dim, io.fp4 != nullptr, env);
  return dtype == SDPA_F16 ? by_dim<__half>(w, head_dim, io.fp4 != nullptr, env)
                           : by_dim<__nv_bfloat16>(w, head_dim, io.fp4 != nullptr, env);
}

}  // namespace gb300

// paged_simt.cu — attention and score sums over the paged KV cache on the
// CUDA cores, in fp32 arithmetic: every element type, head dimension 64 and
// 128, any page size.  fp32 caches always run here; fp16/bf16 ones where a
// page's rows do not fall into whole groups of 8 (the tensor-core kernels'
// layout).  And the kernels that join the partial results of cut units.
//
// Attention: a CTA of 256 threads holds a tile of RM query rows (RM / gu
// tokens times gu heads of one kv head) and walks the unit's key tiles of
// 64 keys with a running maximum m and sum l per row; K and V tiles are
// widened to fp32 in shared memory.  A thread owns RM / 16 rows x 4 keys of
// the scores, and the same rows x D / 16 columns of the output.  RM = 64
// reuses each K and V value for 64 rows (bound by the FMA pipes: 2048 tokens
// over 4096 keys, 16 heads over 4, head_dim 128, fp32: 1294 us, 40 TFLOP/s);
// RM = 16, for calls of few rows a sequence, does a quarter of that arithmetic
// on the same bytes (bound by the shared-memory reads of K and V).  fp32 calls
// of up to 8 rows take paged_vector_f32.cu.  Score sums of the same 2048 tokens
// in fp32: 705 us, 37 TFLOP/s.
//
// 16-bit caches in pages of other than whole groups of 8 rows pay for the fp32
// arithmetic and the widening of each row: 2048 tokens over 4096 keys, 32 heads
// over 8, head_dim 128, bf16, pages of 20: 2926 us (35 TFLOP/s), score sums
// 1339 (38); single tokens over 8 x 32768 keys: 1273 us and 700, 0.8 TB/s (168
// and 103 on the tensor cores with pages of 16).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace paged {
namespace {

constexpr int kT = 256;   // threads of a CTA
constexpr int kKT = 64;   // keys of a tile
constexpr int kLgKT = 6;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half narrow<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// 16 bytes of T widened to fp32 at dst (zeros where src is null).
template <typename T>
__device__ __forceinline__ void widen16(float* dst, const T* src) {
  constexpr int N = 16 / sizeof(T);
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (src) raw = *reinterpret_cast<const uint4*>(src);
  const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<float4*>(dst + i) =
        make_float4(widen(e[i]), widen(e[i + 1]), widen(e[i + 2]), widen(e[i + 3]));
}

// Element offsets of a key tile's rows in k_pages and v_pages (-1: at or past
// nk, or in a bad page), by the first kKT threads: the page lookups of the
// next tile run beside this tile's arithmetic.
__device__ __forceinline__ void row_offsets(const Args& a, int b, int kvh, int key0, int nk,
                                            long long* off_k, long long* off_v) {
  const int r = threadIdx.x;
  if (r >= kKT) return;
  const int key = key0 + r;
  const int page = key < nk ? page_of(a, b, key) : -1;
  const int row = key - a.by_page.div(key) * a.page_size;
  off_k[r] = page < 0 ? -1 : page * a.ks[0] + kvh * a.ks[1] + row * a.ks[2];
  off_v[r] = page < 0 ? -1 : page * a.vs[0] + kvh * a.vs[1] + row * a.vs[2];
}

// The rows at `off` as fp32 rows of `pitch` floats; zeros where there is none.
template <typename T, int D>
__device__ void load_rows(const void* base, const long long* off, float* dst, int pitch) {
  constexpr int N = 16 / sizeof(T);
  constexpr int C = D / N;  // 16-byte pieces of a row
#pragma unroll 4
  for (int i = threadIdx.x; i < kKT * C; i += kT) {
    const int r = i / C, c = (i % C) * N;
    const long long o = off[r];
    widen16<T>(dst + r * pitch + c, o >= 0 ? static_cast<const T*>(base) + o + c : nullptr);
  }
}

// The same for fp32 caches as asynchronous copies straight into shared memory
// (nothing to widen), zeros where there is no row.
template <int D>
__device__ void copy_rows(const void* base, const long long* off, float* dst, int pitch) {
  constexpr int C = D / 4;  // 16-byte pieces of a row
#pragma unroll 4
  for (int i = threadIdx.x; i < kKT * C; i += kT) {
    const int r = i / C, c = (i % C) * 4;
    const long long o = off[r];
    const float* src = static_cast<const float*>(base) + (o >= 0 ? o + c : 0);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     smem_addr(dst + r * pitch + c)),
                 "l"(src), "r"(o >= 0 ? 16 : 0)
                 : "memory");
  }
}

// Query rows of tile (first token tok0) of head unit (kvh, sub) as fp32 rows
// of D floats; rows that do not exist are zero.
template <typename T, int D, int RM>
__device__ void load_queries(const Args& a, const Seq& s, int tok0, int kvh, int sub,
                             float* dst) {
  constexpr int N = 16 / sizeof(T);
  constexpr int C = D / N;
  for (int i = threadIdx.x; i < RM * C; i += kT) {
    const int r = i / C, c = (i % C) * N;
    const int tok = tok0 + a.by_gu.div(r), e = sub * a.gu + a.by_gu.mod(r);
    const T* src = nullptr;
    if (r < a.w * a.gu && tok < s.nq && e < a.G)
      src = static_cast<const T*>(a.q) + (s.q0 + tok) * a.qs[0] +
            static_cast<long long>(kvh * a.G + e) * a.qs[1] + c;
    widen16<T>(dst + r * D + c, src);
  }
}

// s[i][jj] = q_row(ty * RPT + i) . k_key(tx + 16 jj)
template <int D, int RPT>
__device__ __forceinline__ void scores_tile(const float* sQ, const float* sK, int ty, int tx,
                                            float (&s)[RPT][4]) {
#pragma unroll
  for (int i = 0; i < RPT; ++i)
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) s[i][jj] = 0.f;
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    float4 q[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
      q[i] = *reinterpret_cast<const float4*>(sQ + (ty * RPT + i) * D + d);
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const float4 k = *reinterpret_cast<const float4*>(sK + (tx + 16 * jj) * (D + 4) + d);
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        s[i][jj] = fmaf(q[i].x, k.x, s[i][jj]);
        s[i][jj] = fmaf(q[i].y, k.y, s[i][jj]);
        s[i][jj] = fmaf(q[i].z, k.z, s[i][jj]);
        s[i][jj] = fmaf(q[i].w, k.w, s[i][jj]);
      }
    }
  }
}

// fp32 tiles are double-buffered (copies of the next beside the arithmetic on
// this one)
template <typename T, int D, int RM>
constexpr int attend_smem() {
  return (RM * D + (sizeof(T) == 4 ? 2 : 1) * kKT * (2 * D + 4) + RM * (kKT + 4)) * 4;
}

// CTAs an SM: what the shared memory and the registers of a tile allow (one of
// 8 warps alone leaves the FMA pipes waiting for shared memory).
template <typename T, int D, int RM>
constexpr int attend_ctas() {
  if (sizeof(T) == 4) return D == 64 ? 2 : 1;
  return RM == 16 ? (D == 64 ? 4 : 2) : (D == 64 ? 2 : 1);
}
template <int D, int RM>
constexpr int scores_ctas() {
  return RM == 16 ? 4 : D == 64 ? 3 : 2;
}

template <typename T, int D, int RM>
__global__ void __launch_bounds__(kT, attend_ctas<T, D, RM>()) paged_simt_kernel(const Args a) {
  constexpr int RPT = RM / 16;
  constexpr int CG = D / 64;  // float4 column groups of a thread
  constexpr int kSlot = RM * (D + 2);
  extern __shared__ float smem[];
  float* sQ = smem;
  float* sK = sQ + RM * D;
  constexpr bool kAsync = sizeof(T) == 4;
  constexpr int kTile = kKT * (2 * D + 4);  // a K and a V tile
  float* sP = sK + (kAsync ? 2 : 1) * kTile;
  __shared__ long long off_k[2][kKT], off_v[2][kKT];
  __shared__ long long scratch[kT / 32 + 1];
  __shared__ Share sh;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  griddep_launch_dependents();
  const AttendUnits units{a.by_w, kLgKT, a.causal, 1};
  const int heads = a.Hkv * a.nsub;
  plan_share<kT>(a, units, heads, 1, scratch, &sh);
  if (tid == 0) a.desc[blockIdx.x * kDesc] = 0;
  Walk<AttendUnits> walk(sh);
  Unit u;
  while (walk.next(a, units, sh, heads, &u)) {
    const int kvh = a.by_nsub.div(u.h), sub = a.by_nsub.mod(u.h);
    const int tok0 = u.j * a.w;
    __syncthreads();  // the previous unit's tiles are read
    load_queries<T, D, RM>(a, u.s, tok0, kvh, sub, sQ);
    row_offsets(a, u.b, kvh, u.s0 * kKT, u.s.nk, off_k[0], off_v[0]);
    __syncthreads();
    int limit[RPT];  // keys below it are visible to the row
    float m[RPT], l[RPT], o[RPT][CG][4];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = ty * RPT + i, tok = tok0 + a.by_gu.div(r);
      limit[i] = a.causal ? min(u.s.nk, u.s.off + tok + 1) : u.s.nk;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < CG; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][c][e] = 0.f;
    }
    auto copy_tile = [&](int par) {
      float* k = sK + par * kTile;
      copy_rows<D>(a.k, off_k[par], k, D + 4);
      copy_rows<D>(a.v, off_v[par], k + kKT * (D + 4), D);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (kAsync && u.s0 < u.s1) {
      copy_tile(0);
      if (u.s0 + 1 < u.s1)
        row_offsets(a, u.b, kvh, (u.s0 + 1) * kKT, u.s.nk, off_k[1], off_v[1]);
    }
    for (int t = u.s0; t < u.s1; ++t) {
      const int key0 = t * kKT;
      const int par = (t - u.s0) & 1;
      float* sKt = sK;
      if constexpr (kAsync) {
        // this tile's copies have landed, and the last tile's buffers are read
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        sKt = sK + par * kTile;
        if (t + 1 < u.s1) copy_tile(par ^ 1);
        if (t + 2 < u.s1)
          row_offsets(a, u.b, kvh, key0 + 2 * kKT, u.s.nk, off_k[par], off_v[par]);
      } else {
        if (t > u.s0) __syncthreads();
        load_rows<T, D>(a.k, off_k[par], sK, D + 4);
        load_rows<T, D>(a.v, off_v[par], sK + kKT * (D + 4), D);
        __syncthreads();
        if (t + 1 < u.s1)
          row_offsets(a, u.b, kvh, key0 + kKT, u.s.nk, off_k[par ^ 1], off_v[par ^ 1]);
      }
      const float* sV = sKt + kKT * (D + 4);
      float s[RPT][4];
      scores_tile<D, RPT>(sQ, sKt, ty, tx, s);
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          s[i][jj] = key0 + tx + 16 * jj < limit[i] ? s[i][jj] * a.sl2 : -INFINITY;
          mx = fmaxf(mx, s[i][jj]);
        }
#pragma unroll
        for (int d = 8; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m[i], mx);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float alpha = ex2(m[i] - base);  // 0 when m = -inf
        float rs = 0.f;
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const float p = ex2(s[i][jj] - base);
          rs += p;
          sP[(ty * RPT + i) * (kKT + 4) + tx + 16 * jj] = p;
        }
#pragma unroll
        for (int d = 8; d >= 1; d >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, d);
        l[i] = l[i] * alpha + rs;
        m[i] = mn;
#pragma unroll
        for (int c = 0; c < CG; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][c][e] *= alpha;
      }
      __syncwarp();  // a row's probabilities come from 16 lanes of one warp
#pragma unroll 2
      for (int k4 = 0; k4 < kKT; k4 += 4) {
        float4 p[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i)
          p[i] = *reinterpret_cast<const float4*>(sP + (ty * RPT + i) * (kKT + 4) + k4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int c = 0; c < CG; ++c) {
            const float4 v =
                *reinterpret_cast<const float4*>(sV + (k4 + kk) * D + c * 64 + tx * 4);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
              const float pv = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
              o[i][c][0] = fmaf(pv, v.x, o[i][c][0]);
              o[i][c][1] = fmaf(pv, v.y, o[i][c][1]);
              o[i][c][2] = fmaf(pv, v.z, o[i][c][2]);
              o[i][c][3] = fmaf(pv, v.w, o[i][c][3]);
            }
          }
      }
    }
    const bool whole = u.whole();
    float* slot = a.ws + static_cast<size_t>(blockIdx.x * 2 + u.slot()) * kSlot;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = ty * RPT + i, tok = tok0 + a.by_gu.div(r), e = sub * a.gu + a.by_gu.mod(r);
      if (r >= a.w * a.gu || tok >= u.s.nq || e >= a.G) continue;
      if (!whole) {
#pragma unroll
        for (int c = 0; c < CG; ++c)
          *reinterpret_cast<float4*>(slot + r * D + c * 64 + tx * 4) =
              make_float4(o[i][c][0], o[i][c][1], o[i][c][2], o[i][c][3]);
        if (tx == 0) {
          slot[RM * D + r] = m[i];
          slot[RM * D + RM + r] = l[i];
        }
        continue;
      }
      const int hq = kvh * a.G + e;
      float mm = m[i], ll = l[i], f = 1.f;
      if (a.sinks) f = add_sink(a.sinks[hq], mm, ll);
      const float inv = l[i] != 0.f ? f / ll : 0.f;  // (a NaN sum stays one)
      T* orow = static_cast<T*>(a.o) + (u.s.q0 + tok) * a.os[0] + hq * a.os[1];
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        T x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = narrow<T>(o[i][c][k] * inv);
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<uint4*>(orow + c * 64 + tx * 4) = *reinterpret_cast<uint4*>(x);
        else
          *reinterpret_cast<uint2*>(orow + c * 64 + tx * 4) = *reinterpret_cast<uint2*>(x);
      }
      if (a.lse && tx == 0)
        a.lse[static_cast<size_t>(u.s.q0 + tok) * a.Hq + hq] =
            ll != 0.f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
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
  }
}

// Joins the partial results of the units that CTAs of the attention kernels
// began and did not finish: M = max of the m's, weights 2^(m - M), in the
// order of the pieces.  Block (c, y) takes a part of the rows of the unit that
// CTA c began.  Bound by the latency of its few loads, so a warp takes two rows
// and has their (m, l), a piece a lane, and up to kAhead pieces of their
// outputs on their way at once.  A unit of more than kWide pieces (a few rows
// of a long sequence spread over the whole GPU): a row at a time, its pieces
// spread over the block's warps.
constexpr int kWide = 12;
constexpr int kAhead = 3;
constexpr int kMergeRows = 2;

template <int D>
struct MergeVec;
template <>
struct MergeVec<128> {
  using V = float4;
};
template <>
struct MergeVec<64> {
  using V = float2;
};

template <typename T, int D>
__global__ void __launch_bounds__(256, 4)
    paged_merge_kernel(const Args a, int tile_rows, int tiles) {
  using V = typename MergeVec<D>::V;
  constexpr int E = D / 32;  // columns of a lane
  griddep_wait();
  const int c = blockIdx.x;
  const int* d = a.desc + c * kDesc;
  const int n = d[0];
  if (n == 0) return;
  const int b_h = d[2], j = d[3], q0 = d[4], nq = d[5];
  const int kvh = a.by_nsub.div(b_h), sub = a.by_nsub.mod(b_h);
  const int rows = tile_rows * tiles;
  const size_t slot_floats = static_cast<size_t>(rows) * (D + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto piece = [&](int p) {
    return a.ws + (p == 0 ? static_cast<size_t>(c * 2 + 1) : static_cast<size_t>((c + p) * 2)) *
                      slot_floats;
  };
  // token and head of row rr (false: no such row)
  auto locate = [&](int rr, int* tok, int* head) {
    const int t = rr >= tile_rows ? rr / tile_rows : 0, r = rr - t * tile_rows;
    const int g = a.by_gu.div(r), e = sub * a.gu + r - g * a.gu;
    *tok = (j * tiles + t) * a.w + g;
    *head = kvh * a.G + e;
    return rr < rows && g < a.w && *tok < nq && e < a.G;
  };
  // O, LSE of a row from its joined accumulator
  auto finish = [&](int tok, int hq, float M, float L, const float (&acc)[E]) {
    const bool any = L != 0.f;
    float f = 1.f;
    if (a.sinks) f = add_sink(a.sinks[hq], M, L);
    const float inv = any ? f / L : 0.f;
    const float gain = a.v_gain ? a.v_gain[kvh] : 1.f;  // (of a 4-bit cache)
    T* orow = static_cast<T*>(a.o) + static_cast<long long>(q0 + tok) * a.os[0] + hq * a.os[1];
    T x[E];
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = narrow<T>(acc[i] * inv * gain);
    if constexpr (E * sizeof(T) == 16)
      *reinterpret_cast<uint4*>(orow + lane * E) = *reinterpret_cast<uint4*>(x);
    else if constexpr (E * sizeof(T) == 8)
      *reinterpret_cast<uint2*>(orow + lane * E) = *reinterpret_cast<uint2*>(x);
    else
      *reinterpret_cast<uint32_t*>(orow + lane * E) = *reinterpret_cast<uint32_t*>(x);
    if (a.lse && lane == 0)
      a.lse[static_cast<size_t>(q0 + tok) * a.Hq + hq] =
          L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
  };
  if (n <= kWide) {
    for (int r0 = (blockIdx.y * 8 + warp) * kMergeRows; r0 < rows;
         r0 += gridDim.y * 8 * kMergeRows) {
      int tok[kMergeRows], head[kMergeRows];
      bool live[kMergeRows];
      float m[kMergeRows], l[kMergeRows], acc[kMergeRows][E];
      V v[kAhead][kMergeRows];
      auto fetch = [&](int p, V (&x)[kMergeRows]) {
        const float* s = piece(p) + static_cast<size_t>(r0) * D + lane * E;
#pragma unroll
        for (int k = 0; k < kMergeRows; ++k)
          if (p < n && live[k]) x[k] = *reinterpret_cast<const V*>(s + k * D);
      };
#pragma unroll
      for (int k = 0; k < kMergeRows; ++k) {
        live[k] = locate(r0 + k, &tok[k], &head[k]);
        m[k] = -INFINITY;
        l[k] = 0.f;
        if (live[k] && lane < n) {
          const float* s = piece(lane);
          m[k] = s[static_cast<size_t>(rows) * D + r0 + k];
          l[k] = s[static_cast<size_t>(rows) * (D + 1) + r0 + k];
        }
#pragma unroll
        for (int i = 0; i < E; ++i) acc[k][i] = 0.f;
      }
#pragma unroll
      for (int p = 0; p < kAhead; ++p) fetch(p, v[p]);
      float wgt[kMergeRows], L[kMergeRows], M[kMergeRows];
#pragma unroll
      for (int k = 0; k < kMergeRows; ++k) {
        // (a piece whose keys the row does not see holds nothing)
        M[k] = l[k] != 0.f ? m[k] : -INFINITY;
#pragma unroll
        for (int i = 16; i >= 1; i >>= 1)
          M[k] = fmaxf(M[k], __shfl_xor_sync(0xffffffffu, M[k], i));
        wgt[k] = l[k] != 0.f ? ex2(m[k] - M[k]) : 0.f;
        L[k] = 0.f;
      }
      for (int p0 = 0; p0 < n; p0 += kAhead) {
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
          const int p = p0 + x;
          if (p < n) {
#pragma unroll
            for (int k = 0; k < kMergeRows; ++k) {
              const float w = __shfl_sync(0xffffffffu, wgt[k], p);
              const float lp = __shfl_sync(0xffffffffu, l[k], p);
              if (live[k] && lp != 0.f) {
                L[k] += lp * w;
                const float* e = reinterpret_cast<const float*>(&v[x][k]);
#pragma unroll
                for (int i = 0; i < E; ++i) acc[k][i] = fmaf(e[i], w, acc[k][i]);
              }
            }
            fetch(p + kAhead, v[x]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kMergeRows; ++k)
        if (live[k]) finish(tok[k], head[k], M[k], L[k], acc[k]);
    }
    return;
  }
  __shared__ float sM[8], sL[8], sO[8][D];
  for (int rr = blockIdx.y; rr < rows; rr += gridDim.y) {
    int tok, head;
    if (!locate(rr, &tok, &head)) continue;  // the same for every warp
    float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.f;
    auto join = [&](float m, float l, const float* v) {
      if (l != 0.f) {
        const float mn = fmaxf(M, m);
        const float f = ex2(M - mn), g = ex2(m - mn);
        L = L * f + l * g;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = acc[i] * f + v[i] * g;
        M = mn;
      }
    };
#pragma unroll 4
    for (int p = warp; p < n; p += 8) {
      const float* s = piece(p);
      const V v = *reinterpret_cast<const V*>(s + static_cast<size_t>(rr) * D + lane * E);
      join(s[static_cast<size_t>(rows) * D + rr], s[static_cast<size_t>(rows) * (D + 1) + rr],
           reinterpret_cast<const float*>(&v));
    }
    __syncthreads();
    if (lane == 0) {
      sM[warp] = M;
      sL[warp] = L;
    }
    *reinterpret_cast<V*>(&sO[warp][lane * E]) = *reinterpret_cast<V*>(acc);
    __syncthreads();
    if (warp != 0) continue;
    for (int w = 1; w < 8; ++w) join(sM[w], sL[w], &sO[w][lane * E]);
    finish(tok, head, M, L, acc);
  }
}

// Score sums: a unit is 64 keys, its steps the chunks of RM query rows that
// see them; a thread's 4 keys x RM / 16 rows of each score tile become
// probabilities against the rows' log-sum-exp and are added up in registers,
// and the 16 row groups meet in shared memory at the end of the unit.
template <int D, int RM>
constexpr int scores_smem() {
  return (RM * D + kKT * (D + 4) + 16 * kKT) * 4;
}

template <typename T, int D, int RM>
__global__ void __launch_bounds__(kT, scores_ctas<D, RM>())
    paged_scores_simt_kernel(const Args a) {
  constexpr int RPT = RM / 16;
  extern __shared__ float smem[];
  float* sQ = smem;
  float* sK = sQ + RM * D;
  float* sR = sK + kKT * (D + 4);
  __shared__ float sLse[RM];
  __shared__ int sLim[RM];
  __shared__ long long off_k[kKT], off_v[kKT];
  __shared__ long long scratch[kT / 32 + 1];
  __shared__ Share sh;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  griddep_launch_dependents();
  const ScoreUnits units{a.by_w, kLgKT, a.causal, a.nsub, 1};
  plan_share<kT>(a, units, a.Hkv, 1, scratch, &sh);
  if (tid == 0) a.desc[blockIdx.x * kDesc] = 0;
  Walk<ScoreUnits> walk(sh);
  Unit u;
  while (walk.next(a, units, sh, a.Hkv, &u)) {
    const int key0 = u.j * kKT;
    const int first = units.first(u.s, u.j);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    __syncthreads();
    row_offsets(a, u.b, u.h, key0, u.s.nk, off_k, off_v);
    __syncthreads();
    load_rows<T, D>(a.k, off_k, sK, D + 4);
    for (int t = u.s0; t < u.s1; ++t) {
      const int tok0 = (first + a.by_nsub.div(t)) * a.w, sub = a.by_nsub.mod(t);
      if (t > u.s0) __syncthreads();
      load_queries<T, D, RM>(a, u.s, tok0, u.h, sub, sQ);
      if (tid < RM) {
        const int tok = tok0 + a.by_gu.div(tid), e = sub * a.gu + a.by_gu.mod(tid);
        float ls = INFINITY;  // rows that do not exist add nothing
        int lim = 0;
        if (tid < a.w * a.gu && tok < u.s.nq && e < a.G) {
          ls = a.lse[static_cast<size_t>(u.s.q0 + tok) * a.Hq + u.h * a.G + e] * kLog2e;
          if (ls == -INFINITY) ls = INFINITY;
          lim = a.causal ? min(u.s.nk, u.s.off + tok + 1) : u.s.nk;
        }
        sLse[tid] = ls;
        sLim[tid] = lim;
      }
      __syncthreads();
      float s[RPT][4];
      scores_tile<D, RPT>(sQ, sK, ty, tx, s);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        float add = 0.f;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const int r = ty * RPT + i;
          const bool vis = key0 + tx + 16 * jj < sLim[r];
          add += vis ? ex2(fmaf(s[i][jj], a.sl2, -sLse[r])) : 0.f;
        }
        sum[jj] += add;
      }
    }
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) sR[ty * kKT + tx + 16 * jj] = sum[jj];
    __syncthreads();
    if (tid < kKT) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) x += sR[i * kKT + tid];
      const int key = key0 + tid;
      if (!u.whole())
        a.ws[static_cast<size_t>(blockIdx.x * 2 + u.slot()) * kKT + tid] = x;
      else if (key < u.s.nk && key < a.score_len)
        a.scores[u.b * a.ss[0] + u.h * a.ss[1] + key] += x;
    }
    if (!u.whole() && u.s0 == 0 && tid == 0) {
      int* d = a.desc + blockIdx.x * kDesc;
      d[0] = pieces_of(u, sh);
      d[1] = u.b;
      d[2] = u.h;
      d[3] = u.j;
      d[6] = u.s.nk;
    }
  }
}

// Adds the partial sums of a cut unit, in the order of its pieces.
__global__ void __launch_bounds__(256)
    paged_scores_merge_kernel(const Args a, int tile_keys) {
  griddep_wait();
  const int c = blockIdx.x;
  const int* d = a.desc + c * kDesc;
  const int n = d[0];
  if (n == 0) return;
  for (int i = threadIdx.x; i < tile_keys; i += blockDim.x) {
    const int key = d[3] * tile_keys + i;
    if (key >= d[6] || key >= a.score_len) continue;
    float x = a.ws[static_cast<size_t>(c * 2 + 1) * tile_keys + i];
#pragma unroll 4
    for (int p = 1; p < n; ++p) x += a.ws[static_cast<size_t>(c + p) * 2 * tile_keys + i];
    a.scores[d[1] * a.ss[0] + d[2] * a.ss[1] + key] += x;
  }
}

// Launch with programmatic stream serialization (the kernel waits for the
// previous grid itself, before it touches global memory).
template <typename... P, typename... V>
sdpa_status_t launch_after(void (*kern)(P...), dim3 grid, int threads, cudaStream_t stream,
                           V... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

template <auto kKernel>
sdpa_status_t start(Args& a, int smem, int ctas, cudaStream_t stream) {
  a.nctas = std::min(a.max_ctas, ctas);
  if (!allow_smem<kKernel>(smem)) return SDPA_ERR_CUDA;
  kKernel<<<a.nctas, kT, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

template <typename T, int D>
sdpa_status_t attend(Args& a, const LaunchEnv& env) {
  // few rows a sequence (decode): the 16-row tile, see the top of the file
  const int rows = a.G <= 16 && call_rows(a) <= 16 ? 16 : 64;
  fit_rows(a, rows);
  const sdpa_status_t st =
      rows == 16 ? start<paged_simt_kernel<T, D, 16>>(
                       a, attend_smem<T, D, 16>(), attend_ctas<T, D, 16>() * env.num_sms, env.stream)
                 : start<paged_simt_kernel<T, D, 64>>(
                       a, attend_smem<T, D, 64>(), attend_ctas<T, D, 64>() * env.num_sms, env.stream);
  if (st != SDPA_OK) return st;
  const int dtype = sizeof(T) == 4 ? SDPA_F32 : std::is_same<T, __half>::value ? SDPA_F16 : SDPA_BF16;
  return launch_paged_merge(a, D, dtype, rows, 1, env.stream);
}

template <typename T, int D>
sdpa_status_t score(Args& a, const LaunchEnv& env) {
  const bool few = a.G <= 16 && call_rows(a) <= 16;
  fit_rows(a, few ? 16 : 64);
  const sdpa_status_t st =
      few ? start<paged_scores_simt_kernel<T, D, 16>>(
                a, scores_smem<D, 16>(), scores_ctas<D, 16>() * env.num_sms, env.stream)
          : start<paged_scores_simt_kernel<T, D, 64>>(
                a, scores_smem<D, 64>(), scores_ctas<D, 64>() * env.num_sms, env.stream);
  return st != SDPA_OK ? st : launch_paged_scores_merge(a, kKT, env.stream);
}

}  // namespace
}  // namespace paged

sdpa_status_t launch_paged_merge(const paged::Args& a, int head_dim, int dtype, int tile_rows,
                                 int tiles, cudaStream_t stream) {
  using namespace paged;
  const dim3 grid(a.nctas, tile_rows * tiles > 16 ? 16 : 8);
  auto go = [&](auto kern) { return launch_after(kern, grid, 256, stream, a, tile_rows, tiles); };
  if (head_dim == 64) {
    if (dtype == SDPA_F32) return go(paged_merge_kernel<float, 64>);
    return dtype == SDPA_F16 ? go(paged_merge_kernel<__half, 64>)
                             : go(paged_merge_kernel<__nv_bfloat16, 64>);
  }
  if (dtype == SDPA_F32) return go(paged_merge_kernel<float, 128>);
  return dtype == SDPA_F16 ? go(paged_merge_kernel<__half, 128>)
                           : go(paged_merge_kernel<__nv_bfloat16, 128>);
}

sdpa_status_t launch_paged_scores_merge(const paged::Args& a, int tile_keys,
                                        cudaStream_t stream) {
  return paged::launch_after(paged::paged_scores_merge_kernel, dim3(a.nctas), 256, stream, a,
                             tile_keys);
}

sdpa_status_t launch_paged_simt(paged::Args a, int head_dim, int dtype, const LaunchEnv& env) {
  using namespace paged;
  if (head_dim == 64) {
    if (dtype == SDPA_F32) return attend<float, 64>(a, env);
    return dtype == SDPA_F16 ? attend<__half, 64>(a, env) : attend<__nv_bfloat16, 64>(a, env);
  }
  if (dtype == SDPA_F32) return attend<float, 128>(a, env);
  return dtype == SDPA_F16 ? attend<__half, 128>(a, env) : attend<__nv_bfloat16, 128>(a, env);
}

sdpa_status_t launch_paged_scores_simt(paged::Args a, int head_dim, int dtype,
                                       const LaunchEnv& env) {
  using namespace paged;
  if (head_dim == 64) {
    if (dtype == SDPA_F32) return score<float, 64>(a, env);
    return dtype == SDPA_F16 ? score<__half, 64>(a, env) : score<__nv_bfloat16, 64>(a, env);
  }
  if (dtype == SDPA_F32) return score<float, 128>(a, env);
  return dtype == SDPA_F16 ? score<__half, 128>(a, env) : score<__nv_bfloat16, 128>(a, env);
}

}  // namespace gb300

// paged_vector_f32.cu — attention (and accumulated weights, further down) over
// a paged fp32 KV cache where a sequence has few query rows (single tokens, up
// to NR = 4 or 8 rows of (token, head) of a kv head), on the CUDA cores.
//
// Every warp is a reader of its own: of each tile of 64 keys it takes 8, whose
// K and V rows it brings into its part of shared memory with asynchronous
// copies some tiles ahead, and it keeps a running softmax of its own for the
// NR rows, so that no barrier stands in the loop; the eight warps' results
// meet at the end of a unit.  A lane owns D / 32 columns: it holds that slice
// of the NR queries and of the NR outputs in registers, and reads that slice
// of every K and V row once for all NR rows.  The 8 x NR dot products are
// summed over the lanes by one reduce-scatter (62 shuffles for 64 sums), which
// leaves key l / 4 with lane l.
//
// Bound by HBM and by the copies' latency; the tile kernel of paged_simt.cu,
// made for 16 and 64 rows, reads K and V out of shared memory once for every
// two rows and was bound by that (8 x 16384 keys, 16 heads over 4, head_dim
// 128: 308 us, here 93).
#include <cuda_runtime.h>

#include "paged.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace paged {
namespace {

constexpr int kVT = 256;  // threads of a CTA
constexpr int kVWarps = kVT / 32;
constexpr int kVKeys = 8;  // keys of a warp in a tile
constexpr int kVLg = 6;    // tiles of 64 keys
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
constexpr int vector_stages() {
  return D == 128 ? 3 : 6;
}
// floats of a warp's stage: K rows, then V rows
template <int D>
constexpr int vector_stage() {
  return 2 * kVKeys * D;
}
template <int D>
constexpr int vector_smem() {
  return (vector_stages<D>() * kVWarps * vector_stage<D>() + kVWarps * 64) * 4;
}

template <int E>
__device__ __forceinline__ void ld_cols(const float* p, float (&x)[E]) {
  if constexpr (E == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x;
    x[1] = v.y;
  }
}

template <int D, int NR>
__global__ void __launch_bounds__(kVT, 1) paged_vector_f32_kernel(const Args a) {
  constexpr int E = D / 32;  // columns of a lane
  constexpr int NS = vector_stages<D>();
  constexpr int PL = NR / 4;  // scores of a lane: rows PL * (lane % 4) ..
  extern __shared__ float smem[];
  __shared__ long long scratch[kVWarps];
  __shared__ Share sh;
  __shared__ float s_m[kVWarps][NR], s_l[kVWarps][NR];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* ring = smem + warp * vector_stage<D>();  // stage s at + s * kVWarps * vector_stage
  constexpr int kNext = kVWarps * vector_stage<D>();
  float* s_p = smem + NS * kNext + warp * 64;
  griddep_launch_dependents();
  const AttendUnits units{a.by_w, kVLg, a.causal, 2};
  const int heads = a.Hkv * a.nsub;
  plan_share<kVT>(a, units, heads, 2, scratch, &sh);
  if (tid == 0) a.desc[blockIdx.x * kDesc] = 0;
  Walk<AttendUnits> walk(sh);
  Unit u;
  while (walk.next(a, units, sh, heads, &u)) {
    const int kvh = a.by_nsub.div(u.h), e0 = a.by_nsub.mod(u.h) * a.gu;
    const int tok0 = u.j * a.w;
    auto row_ok = [&](int c) {
      const int t = a.by_gu.div(c);
      return c < a.gu * a.w && tok0 + t < u.s.nq && e0 + a.by_gu.mod(c) < a.G;
    };
    // this lane's slice of the queries, in log2 units
    float q[NR][E], acc[NR][E];
#pragma unroll
    for (int c = 0; c < NR; ++c) {
#pragma unroll
      for (int e = 0; e < E; ++e) q[c][e] = acc[c][e] = 0.f;
      if (row_ok(c)) {
        const float* src = static_cast<const float*>(a.q) +
                           (u.s.q0 + tok0 + a.by_gu.div(c)) * a.qs[0] +
                           (kvh * a.G + e0 + a.by_gu.mod(c)) * a.qs[1] + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) q[c][e] = src[e] * a.sl2;
      }
    }
    // rows of this lane's scores: keys below their limits are visible
    int lim[PL];
    float m[PL], l[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int tok = tok0 + a.by_gu.div(PL * (lane & 3) + i);
      lim[i] = a.causal ? min(u.s.nk, u.s.off + tok + 1) : u.s.nk;
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    // Rows of the next group (lanes 0 .. 7: one each), looked up one group
    // before its copies.
    int nx_page = -1, nx_row = 0;
    auto lookup = [&](int t) {
      const int key = (t << kVLg) + warp * kVKeys + lane;
      nx_page = -1;
      if (lane < kVKeys && t < u.s1 && key < u.s.nk) {
        const int i = a.by_page.div(key);
        nx_row = key - i * a.page_size;
        nx_page = a.table[u.b * a.table_stride + i];
        if (nx_page < 0 || nx_page >= a.num_pages) nx_page = -2;
      }
    };
    auto copy = [&](int t) {  // (every call commits one group of copies)
      if (t < u.s1) {
        if (nx_page == -2) atomicExch(a.status, kStatusPageTable);
        const long long ko = nx_page < 0 ? -1 : nx_page * a.ks[0] + kvh * a.ks[1] + nx_row * a.ks[2];
        const long long vo = nx_page * a.vs[0] + kvh * a.vs[1] + nx_row * a.vs[2];
        float* dst = ring + ((t - u.s0) % NS) * kNext;
        constexpr int P = D / 4;  // 16-byte pieces of a row
#pragma unroll
        for (int i = 0; i < kVKeys * P / 32; ++i) {
          const int x = i * 32 + lane, r = x / P, c = (x % P) * 4;
          const long long k = __shfl_sync(0xffffffffu, ko, r), v = __shfl_sync(0xffffffffu, vo, r);
          const int n = k >= 0 ? 16 : 0;  // zeros where there is no row
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           smem_addr(dst + r * D + c)),
                       "l"(static_cast<const float*>(a.k) + (k >= 0 ? k + c : 0)), "r"(n)
                       : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           smem_addr(dst + (kVKeys + r) * D + c)),
                       "l"(static_cast<const float*>(a.v) + (k >= 0 ? v + c : 0)), "r"(n)
                       : "memory");
        }
        lookup(t + 1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    lookup(u.s0);
#pragma unroll 1
    for (int i = 0; i < NS - 1; ++i) copy(u.s0 + i);
#pragma unroll 1
    for (int t = u.s0; t < u.s1; ++t) {
      asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
      __syncwarp();  // every lane's copies of this group have landed, and the last group is read
      copy(t + NS - 1);
      const float* K = ring + ((t - u.s0) % NS) * kNext;
      const float* V = K + kVKeys * D;
      float s[kVKeys * NR];  // [key][row]
#pragma unroll
      for (int k = 0; k < kVKeys; ++k) {
        float x[E];
        ld_cols<E>(K + k * D + lane * E, x);
#pragma unroll
        for (int c = 0; c < NR; ++c) {
          float d = q[c][0] * x[0];
#pragma unroll
          for (int e = 1; e < E; ++e) d = fmaf(q[c][e], x[e], d);
          s[k * NR + c] = d;
        }
      }
      // reduce-scatter: lane l keeps key l / 4, rows PL (l % 4) ..
#pragma unroll
      for (int n = kVKeys * NR, msk = 16; msk >= 1; n >>= 1, msk >>= 1) {
        const bool upper = (lane & msk) != 0;
#pragma unroll
        for (int k = 0; k < n / 2; ++k) {
          const float send = upper ? s[k] : s[k + n / 2];
          const float keep = upper ? s[k + n / 2] : s[k];
          s[k] = keep + __shfl_xor_sync(0xffffffffu, send, msk);
        }
      }
      const int key = (t << kVLg) + warp * kVKeys + (lane >> 2);
      float alpha[PL];
      bool moved = false;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const float x = key < lim[i] ? s[i] : -INFINITY;
        float mx = x;
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m[i], mx);
        const float base = mn == -INFINITY ? 0.f : mn;
        alpha[i] = mn == m[i] ? 1.f : ex2(m[i] - base);
        moved |= mn != m[i];
        m[i] = mn;
        const float p = ex2(x - base);
        l[i] = l[i] * alpha[i] + p;
        s_p[(lane >> 2) * NR + PL * (lane & 3) + i] = p;
      }
      __syncwarp();
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int c = 0; c < NR; ++c) {
          const float f = __shfl_sync(0xffffffffu, alpha[c % PL], c / PL);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[c][e] *= f;
        }
      }
#pragma unroll
      for (int k = 0; k < kVKeys; ++k) {
        float x[E], p[NR];
        ld_cols<E>(V + k * D + lane * E, x);
#pragma unroll
        for (int c = 0; c < NR; c += 4)
          *reinterpret_cast<float4*>(&p[c]) = *reinterpret_cast<const float4*>(s_p + k * NR + c);
#pragma unroll
        for (int c = 0; c < NR; ++c)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[c][e] = fmaf(p[c], x[e], acc[c][e]);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // the warps' results meet in the ring
#pragma unroll
    for (int i = 0; i < PL; ++i) {
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      if (lane < 4) {
        s_m[warp][PL * lane + i] = m[i];
        s_l[warp][PL * lane + i] = l[i];
      }
    }
    __syncthreads();  // every warp has left its loop
#pragma unroll
    for (int c = 0; c < NR; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) smem[(warp * NR + c) * D + lane * E + e] = acc[c][e];
    __syncthreads();
    const bool whole = u.whole();
    float* slot = a.ws + static_cast<size_t>(blockIdx.x * 2 + u.slot()) * (NR * (D + 2));
    for (int x = tid; x < NR * (D / 4); x += kVT) {
      const int c = x / (D / 4), col = (x % (D / 4)) * 4;
      if (!row_ok(c)) continue;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < kVWarps; ++w)
        if (s_l[w][c] != 0.f) M = fmaxf(M, s_m[w][c]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kVWarps; ++w) {
        if (s_l[w][c] == 0.f) continue;  // this warp's keys are not seen
        const float f = ex2(s_m[w][c] - (M == -INFINITY ? 0.f : M));
        const float4 v = *reinterpret_cast<const float4*>(smem + (w * NR + c) * D + col);
        L = fmaf(s_l[w][c], f, L);
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z);
        o.w = fmaf(v.w, f, o.w);
      }
      if (!whole) {
        *reinterpret_cast<float4*>(slot + c * D + col) = o;
        if (col == 0) {
          slot[NR * D + c] = M;
          slot[NR * (D + 1) + c] = L;
        }
        continue;
      }
      const long long tok = u.s.q0 + tok0 + a.by_gu.div(c);
      const int hq = kvh * a.G + e0 + a.by_gu.mod(c);
      float f = L != 0.f ? 1.f : 0.f;
      if (a.sinks) f *= add_sink(a.sinks[hq], M, L);
      f = L != 0.f ? f / L : 0.f;
      *reinterpret_cast<float4*>(static_cast<float*>(a.o) + tok * a.os[0] + hq * a.os[1] + col) =
          make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
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
    __syncthreads();  // the ring is free for the next unit
  }
}

// Accumulated weights with few rows a sequence: a unit is a (sequence, kv
// head); its steps are, for every tile of 64 keys, the sequence's blocks of
// rows, of which a warp takes 8 keys as above.  A tile is whole in the share
// that its first step lies in: every key has one owner, who adds its sum to the
// scores at once, and nothing is left to merge.
// 8 x 16384 keys, 16 heads over 4, D = 128: 66 us, 4.1 TB/s (195 us with the
// 16-row tiles); 32 heads over 8, D = 64: 108 us (210), where the products and
// their reduction bound it.  A chunk of 9 tokens among 16 single ones, 4096
// keys: 146 us (228); of 257 among 255, 32 heads over 8, D = 128: 4578 us
// (3391), for a block's queries come from L2 every time.
struct KeyTileUnits {
  FastDiv by_w;
  int cost;
  __host__ __device__ int count(const Seq& s) const { return s.nq > 0; }
  __host__ __device__ int steps(const Seq& s, int) const {
    return ((s.nk + (1 << kVLg) - 1) >> kVLg) * by_w.ceil(s.nq);
  }
  __host__ __device__ long long before(const Seq& s, int j) const {
    return j <= 0 ? 0 : steps(s, 0);
  }
};
template <int D>
constexpr int score_stages() {
  return D == 128 ? 6 : 8;
}
template <int D>
constexpr int score_vector_smem() {
  return score_stages<D>() * kVWarps * kVKeys * D * 4;
}

template <int D, int NR>
__global__ void __launch_bounds__(kVT, 1) paged_scores_vector_f32_kernel(const Args a) {
  constexpr int E = D / 32;
  constexpr int NS = score_stages<D>();
  constexpr int PL = NR / 4;
  extern __shared__ float smem[];
  __shared__ long long scratch[kVWarps];
  __shared__ Share sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* ring = smem + warp * kVKeys * D;
  constexpr int kNext = kVWarps * kVKeys * D;
  const KeyTileUnits units{a.by_w, 2};
  plan_share<kVT>(a, units, a.Hkv, 2, scratch, &sh);
  Walk<KeyTileUnits> walk(sh);
  Unit u;
  while (walk.next(a, units, sh, a.Hkv, &u)) {
    float q[NR][E], nl[PL];  // queries in log2 units; -lse in log2 units
    int lim[PL];
    const int blocks = a.by_w.ceil(u.s.nq);
    const int t0 = (u.s0 + blocks - 1) / blocks, t1 = (u.s1 + blocks - 1) / blocks;
    if (t0 == t1) continue;  // a part of a tile that another CTA has
    auto load_block = [&](int blk) {
      const int tok0 = blk * a.w;
      auto row_ok = [&](int c) { return c < a.G * a.w && tok0 + a.by_gu.div(c) < u.s.nq; };
#pragma unroll
      for (int c = 0; c < NR; ++c) {
#pragma unroll
        for (int e = 0; e < E; ++e) q[c][e] = 0.f;
        if (row_ok(c)) {
          const float* src = static_cast<const float*>(a.q) +
                             (u.s.q0 + tok0 + a.by_gu.div(c)) * a.qs[0] +
                             (u.h * a.G + a.by_gu.mod(c)) * a.qs[1] + lane * E;
#pragma unroll
          for (int e = 0; e < E; ++e) q[c][e] = src[e] * a.sl2;
        }
      }
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const int c = PL * (lane & 3) + i, tok = tok0 + a.by_gu.div(c);
        nl[i] = 0.f;
        lim[i] = 0;  // a row that does not exist adds nothing
        if (row_ok(c)) {
          const float x = a.lse[static_cast<size_t>(u.s.q0 + tok) * a.Hq + u.h * a.G +
                                a.by_gu.mod(c)] * 1.4426950408889634f;
          nl[i] = x == -INFINITY ? x : -x;  // nor does one that saw nothing
          lim[i] = a.causal ? min(u.s.nk, u.s.off + tok + 1) : u.s.nk;
        }
      }
    };
    load_block(0);
    int nx_page = -1, nx_row = 0;
    auto lookup = [&](int t) {
      const int key = (t << kVLg) + warp * kVKeys + lane;
      nx_page = -1;
      if (lane < kVKeys && t < t1 && key < u.s.nk) {
        const int i = a.by_page.div(key);
        nx_row = key - i * a.page_size;
        nx_page = a.table[u.b * a.table_stride + i];
        if (nx_page < 0 || nx_page >= a.num_pages) nx_page = -2;
      }
    };
    auto copy = [&](int t) {  // (every call commits one group of copies)
      if (t < t1) {
        if (nx_page == -2) atomicExch(a.status, kStatusPageTable);
        const long long ko =
            nx_page < 0 ? -1 : nx_page * a.ks[0] + u.h * a.ks[1] + nx_row * a.ks[2];
        float* dst = ring + ((t - t0) % NS) * kNext;
        constexpr int P = D / 4;  // 16-byte pieces of a row
#pragma unroll
        for (int i = 0; i < kVKeys * P / 32; ++i) {
          const int x = i * 32 + lane, r = x / P, c = (x % P) * 4;
          const long long k = __shfl_sync(0xffffffffu, ko, r);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           smem_addr(dst + r * D + c)),
                       "l"(static_cast<const float*>(a.k) + (k >= 0 ? k + c : 0)),
                       "r"(k >= 0 ? 16 : 0)
                       : "memory");
        }
        lookup(t + 1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    lookup(t0);
#pragma unroll 1
    for (int i = 0; i < NS - 1; ++i) copy(t0 + i);
    float* out = a.scores + u.b * a.ss[0] + u.h * a.ss[1];
#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
      asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
      __syncwarp();  // every lane's copies of this group have landed, and the last group is read
      copy(t + NS - 1);
      const float* K = ring + ((t - t0) % NS) * kNext;
      const int key = (t << kVLg) + warp * kVKeys + (lane >> 2);
      const bool mine = (lane & 3) == 0 && key < u.s.nk && key < a.score_len;
      const float old = mine ? out[key] : 0.f;
      float sum = 0.f;
      const int behind = (t << kVLg) - u.s.off;  // first token that sees the tile
      const int blk0 = a.causal && behind > 0 ? a.by_w.div(behind) : 0;
#pragma unroll 1
      for (int blk = blk0; blk < blocks; ++blk) {
        if (blocks > 1) load_block(blk);
        float s[kVKeys * NR];
#pragma unroll
        for (int k = 0; k < kVKeys; ++k) {
          float x[E];
          ld_cols<E>(K + k * D + lane * E, x);
#pragma unroll
          for (int c = 0; c < NR; ++c) {
            float d = q[c][0] * x[0];
#pragma unroll
            for (int e = 1; e < E; ++e) d = fmaf(q[c][e], x[e], d);
            s[k * NR + c] = d;
          }
        }
#pragma unroll
        for (int n = kVKeys * NR, msk = 16; msk >= 1; n >>= 1, msk >>= 1) {
          const bool upper = (lane & msk) != 0;
#pragma unroll
          for (int k = 0; k < n / 2; ++k) {
            const float send = upper ? s[k] : s[k + n / 2];
            const float keep = upper ? s[k + n / 2] : s[k];
            s[k] = keep + __shfl_xor_sync(0xffffffffu, send, msk);
          }
        }
        float p = 0.f;
#pragma unroll
        for (int i = 0; i < PL; ++i) p += key < lim[i] ? ex2(s[i] + nl[i]) : 0.f;
        p += __shfl_xor_sync(0xffffffffu, p, 1);
        p += __shfl_xor_sync(0xffffffffu, p, 2);
        sum += p;
      }
      if (mine) out[key] = old + sum;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();  // the ring is free for the next unit
  }
}

template <int D, int NR>
sdpa_status_t launch_vector(Args& a, const LaunchEnv& env) {
  fit_rows(a, NR);
  a.nctas = a.max_ctas < env.num_sms ? a.max_ctas : env.num_sms;
  if (!allow_smem<paged_vector_f32_kernel<D, NR>>(vector_smem<D>())) return SDPA_ERR_CUDA;
  paged_vector_f32_kernel<D, NR><<<a.nctas, kVT, vector_smem<D>(), env.stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return SDPA_ERR_CUDA;
  return launch_paged_merge(a, D, SDPA_F32, NR, 1, env.stream);
}

template <int D, int NR>
sdpa_status_t launch_scores_vector(Args& a, const LaunchEnv& env) {
  fit_rows(a, NR);
  a.nctas = a.max_ctas < env.num_sms ? a.max_ctas : env.num_sms;
  if (!allow_smem<paged_scores_vector_f32_kernel<D, NR>>(score_vector_smem<D>()))
    return SDPA_ERR_CUDA;
  paged_scores_vector_f32_kernel<D, NR>
      <<<a.nctas, kVT, score_vector_smem<D>(), env.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

}  // namespace
}  // namespace paged

// Rows of a tile of these kernels for a call (4 or 8; 0: the tile kernel's).
int paged_vector_rows(const paged::Args& a) {
  if (debug_option(SDPA_DEBUG_PAGED_SIMT) == 1) return 0;  // test hook
  const long long rows = paged::call_rows(a);
  return a.G <= 4 && rows <= 4 ? 4 : a.G <= 8 && rows <= 8 ? 8 : 0;
}

sdpa_status_t launch_paged_vector_f32(paged::Args a, int head_dim, int rows,
                                      const LaunchEnv& env) {
  using namespace paged;
  if (head_dim == 64)
    return rows == 4 ? launch_vector<64, 4>(a, env) : launch_vector<64, 8>(a, env);
  return rows == 4 ? launch_vector<128, 4>(a, env) : launch_vector<128, 8>(a, env);
}

sdpa_status_t launch_paged_scores_vector_f32(paged::Args a, int head_dim, int rows,
                                             const LaunchEnv& env) {
  using namespace paged;
  if (head_dim == 64)
    return rows == 4 ? launch_scores_vector<64, 4>(a, env) : launch_scores_vector<64, 8>(a, env);
  return rows == 4 ? launch_scores_vector<128, 4>(a, env) : launch_scores_vector<128, 8>(a, env);
}

}  // namespace gb300

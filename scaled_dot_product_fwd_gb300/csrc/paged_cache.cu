// paged_cache.cu — the paged KV cache's own operators: writing the new
// tokens' rows into their pages, and eviction by accumulated attention
// weight.  Both only move bytes: bound by HBM.
//
// Write: one warp a token; its lanes bring the token's K and V rows (all kv
// heads) with 16-byte loads, issued before the warp looks its sequence up.
//
// Eviction, three kernels:
//  - select (a CTA per (sequence, kv head)): the threshold weight is the
//    keep'-th largest of the candidates, found digit by digit (11, 11 and 10
//    bits) from histograms of the weights' order-preserving integer form,
//    which up to 48 Ki positions stay in shared memory; then one
//    ordered pass over the positions writes the kept ones (above the
//    threshold, the first of those equal to it, and the newest) in ascending
//    order by a scan, and the weights' new places.
//  - move (a CTA per (sequence, kv head), K or V, slice of the rows): row
//    kept[i] goes to row i, for the kept[i] below `keep`, whose rows other
//    moves overwrite.  kept[i] >= i, and the sources of a chunk lie behind the
//    destinations of every earlier chunk, so a CTA that takes the chunks in
//    order, loads the next one early and writes a chunk only when every thread
//    has its rows in registers, moves in place without losing a row.
//  - far: the rows from positions at or past `keep`, which no move writes, in
//    any order over the whole GPU.
#include <cuda_runtime.h>

#include "paged.cuh"
#include "ptx.cuh"

namespace gb300 {
namespace paged {
namespace {

// ------------------------------------------------------------------- write
constexpr int kWriteWarps = 8;

struct WriteArgs {
  Args a;
  const char* k;
  const char* v;
  char* kp;
  char* vp;
  long long kn[2], vn[2];  // byte strides of the new rows (token, head)
  long long kb[3], vb[3];  // byte strides of the cache (page, head, row)
  int pieces;              // 16-byte pieces of a row (a power of two)
  int lg;                  // its log2
};

__global__ void __launch_bounds__(kWriteWarps * 32) paged_write_kernel(const WriteArgs w) {
  const Args& a = w.a;
  const int lane = threadIdx.x & 31;
  const long long tt = static_cast<long long>(blockIdx.x) * kWriteWarps + (threadIdx.x >> 5);
  if (tt >= a.T) return;
  const int t = static_cast<int>(tt);
  const int total = a.Hkv << w.lg;  // 16-byte pieces of a token
  const char* ksrc = w.k + t * w.kn[0];
  const char* vsrc = w.v + t * w.vn[0];
  constexpr int U = 4;
  uint4 kr[U], vr[U];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int x = base + i * 32 + lane;
      if (x < total) {
        const int h = x >> w.lg, c = x & (w.pieces - 1);
        kr[i] = *reinterpret_cast<const uint4*>(ksrc + h * w.kn[1] + c * 16);
        vr[i] = *reinterpret_cast<const uint4*>(vsrc + h * w.vn[1] + c * 16);
      }
    }
  };
  load(0);
  const int b = find_seq(a, t, lane);
  if (b < 0) return;
  const Seq s = seq_of(a, b);
  const int pos = s.off + (t - s.q0);
  if (pos < 0 || pos >= s.nk) return;  // (at or past the table's end: no place)
  const int page = page_of(a, b, pos);
  if (page < 0) return;
  const int row = pos % a.page_size;
  char* kdst = w.kp + page * w.kb[0] + row * w.kb[2];
  char* vdst = w.vp + page * w.vb[0] + row * w.vb[2];
  for (int base = 0; base < total; base += 32 * U) {
    if (base > 0) load(base);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int x = base + i * 32 + lane;
      if (x < total) {
        const int h = x >> w.lg, c = x & (w.pieces - 1);
        *reinterpret_cast<uint4*>(kdst + h * w.kb[1] + c * 16) = kr[i];
        *reinterpret_cast<uint4*>(vdst + h * w.vb[1] + c * 16) = vr[i];
      }
    }
  }
}

// ---------------------------------------------------------------- eviction
struct EvictArgs {
  Args a;
  int keep, recent;
  int near;  // positions below it are the ordered kernel's
  const float* scores;
  float* scores_out;
  long long ss[2];
  int score_len;
  int* kept;
  int* lens_out;
  char* kp;
  char* vp;
  long long kb[3], vb[3];  // byte strides of the cache (page, head, row)
  int slices;  // parts of a row, a CTA each (ordered kernel)
};

// Integer whose order is the weights' order: sign bit flipped for positive
// numbers, all bits for negative ones; NaN as -inf, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) x = -INFINITY;
  if (x == 0.f) x = 0.f;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelE = 4;  // positions of a thread in the ordered pass
constexpr int kBins = 2048;
// weights that the select kernel keeps in shared memory (more are read from
// global memory again for each digit)
constexpr int kSelCache = 48 * 1024;

template <int kSelT>
__global__ void __launch_bounds__(kSelT)
    paged_evict_select_kernel(const EvictArgs e, const int cache) {
  const Args& a = e.a;
  const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  extern __shared__ float s_weight[];  // [cache]
  __shared__ int hist[kBins];
  __shared__ int warp_sum[32];
  __shared__ uint32_t s_digit;
  __shared__ int s_want;
  griddep_launch_dependents();
  const int nk = min(max(a.lens[b], 0), a.cap);
  int* kept = e.kept + static_cast<size_t>(blockIdx.x) * e.keep;
  const float* sc = e.scores + b * e.ss[0] + h * e.ss[1];
  float* out = e.scores_out ? e.scores_out + b * e.ss[0] + h * e.ss[1] : nullptr;
  if (nk <= e.keep) {  // nothing to evict
    for (int i = tid; i < e.keep; i += kSelT) kept[i] = i < nk ? i : -1;
    if (out) {
      if (out != sc)
        for (int i = tid; i < min(nk, e.score_len); i += kSelT) out[i] = sc[i];
      for (int i = nk + tid; i < e.score_len; i += kSelT) out[i] = 0.f;
    }
    return;
  }
  const int rec = min(e.recent, e.keep);
  const int cand = nk - rec;  // positions below it compete
  int want = e.keep - rec;    // for these places
  const bool cached = nk <= cache;
  if (cached) {
#pragma unroll 8
    for (int i = tid; i < nk; i += kSelT) s_weight[i] = i < e.score_len ? sc[i] : 0.f;
    __syncthreads();
  }
  auto weight = [&](int i) {
    return cached ? s_weight[i] : i < e.score_len ? sc[i] : 0.f;
  };
  auto key_of = [&](int i) { return order_key(weight(i)); };

  // exclusive sum of v over the CTA's threads, and its total
  auto scan = [&](int v, int* total) {
    int incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += t;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    const int w = lane < kSelT / 32 ? warp_sum[lane] : 0;
    int wi = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, wi, d);
      if (lane >= d) wi += t;
    }
    if (total) *total = __shfl_sync(0xffffffffu, wi, 31);
    return incl - v + __shfl_sync(0xffffffffu, wi - w, warp);
  };

  // the want-th largest key, from its top digit down (11, 11 and 10 bits)
  uint32_t prefix = 0, mask = 0;
  if (want > 0) {
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
      const uint32_t dmask = d == 2 ? 1023u : 2047u;
      for (int i = tid; i < kBins; i += kSelT) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int i0 = 0; i0 < cand; i0 += kSelT) {
        const int i = i0 + tid;
        const uint32_t key = i < cand ? key_of(i) : 0u;
        const bool in = i < cand && (key & mask) == prefix;
        const uint32_t digit = (key >> shift) & dmask;
        // one add for a warp of one digit (equal weights)
        int same;
        __match_all_sync(0xffffffffu, in ? digit : 0x80000000u + lane, &same);
        if (same) {
          if (lane == 0) atomicAdd(&hist[digit], 32);
        } else if (in) {
          atomicAdd(&hist[digit], 1);
        }
      }
      __syncthreads();
      // how many keys have a larger digit: thread t holds the kBT digits
      // from 2047 - kBT t down
      constexpr int kBT = kBins / kSelT;
      int c[kBT], sum = 0;
#pragma unroll
      for (int k = 0; k < kBT; ++k) {
        c[k] = hist[kBins - 1 - kBT * tid - k];
        sum += c[k];
      }
      int before = scan(sum, nullptr);
#pragma unroll
      for (int k = 0; k < kBT; ++k) {
        if (before < want && want <= before + c[k]) {
          s_digit = static_cast<uint32_t>(kBins - 1 - kBT * tid - k);
          s_want = want - before;
        }
        before += c[k];
      }
      __syncthreads();
      prefix |= s_digit << shift;
      mask |= dmask << shift;
      want = s_want;
    }
  }
  // `want` keys equal to the threshold are kept, the first ones.  Every
  // position in order: place = kept before it (those above the threshold or
  // recent, and of the equal ones at most `want`).
  const bool none = e.keep == rec;  // only the newest stay
  int run_gt = 0, run_eq = 0;
  for (int i0 = 0; i0 < nk; i0 += kSelT * kSelE) {
    uint32_t gt = 0, eq = 0;  // a bit for each of the thread's positions
    float x[kSelE];
#pragma unroll
    for (int k = 0; k < kSelE; ++k) {
      const int i = i0 + tid * kSelE + k;
      x[k] = 0.f;
      if (i < nk) {
        x[k] = weight(i);
        if (i >= cand) {
          gt |= 1u << k;
        } else if (!none) {
          const uint32_t key = order_key(x[k]);
          if (key > prefix) gt |= 1u << k;
          if (key == prefix) eq |= 1u << k;
        }
      }
    }
    const int mine = __popc(gt) | (__popc(eq) << 16);
    // (its barrier: every weight of this chunk is read; `out` may be `sc`)
    int total;
    const int before = scan(mine, &total);
    int ng = run_gt + (before & 0xffff), ne = run_eq + (before >> 16);
#pragma unroll
    for (int k = 0; k < kSelE; ++k) {
      const bool g = (gt >> k) & 1u, q = (eq >> k) & 1u;
      if (g || (q && ne < want)) {
        const int place = ng + min(ne, want);
        kept[place] = i0 + tid * kSelE + k;
        if (out && place < e.score_len) out[place] = x[k];
      }
      ng += g;
      ne += q;
    }
    run_gt += total & 0xffff;
    run_eq += total >> 16;
    __syncthreads();
  }
  if (out)
    for (int i = e.keep + tid; i < e.score_len; i += kSelT) out[i] = 0.f;
}

// Where row `src` of a sequence comes from and row `dst` goes to, as byte
// offsets into the cache of one head.  A page that the table does not name
// sets the status word: one to be read gives zeros (`from` kZeros), one to be
// written drops the row (`from` kNoMove).
constexpr long long kNoMove = -1, kZeros = -2;
__device__ __forceinline__ void locate_move(const Args& a, const int* table, const long long* st,
                                            int src, int dst, long long* from, long long* to) {
  const int ps = table[a.by_page.div(src)], pd = table[a.by_page.div(dst)];
  const bool ok_s = ps >= 0 && ps < a.num_pages, ok_d = pd >= 0 && pd < a.num_pages;
  if (!ok_s || !ok_d) atomicExch(a.status, kStatusPageTable);
  if (!ok_d) return;
  *from = ok_s ? ps * st[0] + a.by_page.mod(src) * st[2] : kZeros;
  *to = pd * st[0] + a.by_page.mod(dst) * st[2];
}

constexpr int kMoveT = 256;
constexpr int kMoveRows = 8;  // rows of a thread in a chunk
// rows of a chunk where a CTA takes 16 * lanes bytes of a row
constexpr int move_chunk(int lanes) { return kMoveRows * kMoveT / lanes; }

template <int kLanes>
__global__ void __launch_bounds__(kMoveT, 2) paged_evict_move_kernel(const EvictArgs e) {
  constexpr int kSlice = 16 * kLanes;         // bytes of a row that the CTA moves
  constexpr int kMoveStep = kMoveT / kLanes;  // rows at a time
  constexpr int kMoveChunk = move_chunk(kLanes);
  constexpr int kRows = kMoveChunk < kMoveT ? kMoveT : kMoveChunk;
  const Args& a = e.a;
  // Where a chunk's rows come from and go to (locate_move), looked up two
  // chunks ahead by one thread a row; four chunks' worth, so that the writes
  // for chunk n + 2 never meet the last reads for chunk n - 1.
  __shared__ long long s_from[4][kRows], s_to[4][kRows];
  __shared__ int s_more[4];
  griddep_wait();
  griddep_launch_dependents();
  int x = blockIdx.x;
  const int slice = x % e.slices;
  x /= e.slices;
  const bool is_v = x & 1;
  const int bh = x >> 1;
  const int b = bh / a.Hkv, h = bh % a.Hkv;
  const int tid = threadIdx.x;
  const int* kept = e.kept + static_cast<size_t>(bh) * e.keep;
  if (h == 0 && slice == 0 && !is_v && tid == 0 && e.lens_out)
    e.lens_out[b] = min(min(max(a.lens[b], 0), a.cap), e.keep);
  const long long* st = is_v ? e.vb : e.kb;
  char* base = (is_v ? e.vp : e.kp) + h * st[1] + slice * kSlice + (tid % kLanes) * 16;
  const int* table = a.table + b * a.table_stride;
  const int r0 = tid / kLanes;
  auto lookup = [&](int n) {
    constexpr int N = kRows / kMoveT;
    int src[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int r = k * kMoveT + tid;
      const long long i = static_cast<long long>(n) * kMoveChunk + r;
      src[k] = r < kMoveChunk && i < e.keep ? kept[i] : -1;
    }
    // (the positions ascend: the first at or past `keep`, the second kernel's,
    // or the end of a short sequence ends this kernel's part)
    if (tid == 0) s_more[n & 3] = src[0] >= 0 && src[0] < e.near;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int r = k * kMoveT + tid, i = n * kMoveChunk + r;
      long long from = kNoMove, to = 0;
      if (src[k] > i && src[k] < e.near)  // (a row that stays needs no move)
        locate_move(a, table, st, src[k], i, &from, &to);
      s_from[n & 3][r] = from;
      s_to[n & 3][r] = to;
    }
  };
  auto load = [&](int n, uint4 (&data)[kMoveRows]) {
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      const long long from = s_from[n & 3][r0 + k * kMoveStep];
      data[k] = make_uint4(0, 0, 0, 0);
      if (from >= 0) data[k] = *reinterpret_cast<const uint4*>(base + from);
    }
  };
  auto store = [&](int n, uint4 (&data)[kMoveRows]) {
    // every row of the chunk is in registers before any thread writes
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k)
      asm volatile("" : "+r"(data[k].x), "+r"(data[k].y), "+r"(data[k].z), "+r"(data[k].w)
                   : : "memory");
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      const int r = r0 + k * kMoveStep;
      if (s_from[n & 3][r] != kNoMove) *reinterpret_cast<uint4*>(base + s_to[n & 3][r]) = data[k];
    }
  };
  lookup(0);
  lookup(1);
  __syncthreads();
  uint4 d0[kMoveRows], d1[kMoveRows];
  load(0, d0);
  for (int n = 0; s_more[n & 3]; n += 2) {
    load(n + 1, d1);
    lookup(n + 2);
    store(n, d0);
    if (!s_more[(n + 1) & 3]) break;
    load(n + 2, d0);
    lookup(n + 3);
    store(n + 1, d1);
  }
}

// Rows from positions at or past `keep`: no move writes there, so they go in
// any order once the rows above have been read.  A warp takes 32 rows: a lane
// looks one row's pages up, and the warp copies the rows two to eight at a
// time.
constexpr int kFarT = 256;
constexpr int kFarPer = 32 * kFarT / 32;  // rows of a CTA

__global__ void __launch_bounds__(kFarT) paged_evict_far_kernel(const EvictArgs e, int lg_lanes) {
  const Args& a = e.a;
  griddep_wait();
  const int chunks = (e.keep + kFarPer - 1) / kFarPer;
  const int chunk = blockIdx.x % chunks;
  const int x = blockIdx.x / chunks;
  const bool is_v = x & 1;
  const int bh = x >> 1;
  const int b = bh / a.Hkv, h = bh % a.Hkv;
  const int lane = threadIdx.x & 31;
  const long long* st = is_v ? e.vb : e.kb;
  char* base = (is_v ? e.vp : e.kp) + h * st[1] + (lane & ((1 << lg_lanes) - 1)) * 16;
  const int* table = a.table + b * a.table_stride;
  const int i = chunk * kFarPer + (threadIdx.x & ~31) + lane;
  const int src = i < e.keep ? e.kept[static_cast<size_t>(bh) * e.keep + i] : -1;
  long long from = kNoMove, to = 0;
  if (src >= e.keep) locate_move(a, table, st, src, i, &from, &to);
  if (__all_sync(0xffffffffu, from == kNoMove)) return;
  const int rows = 32 >> lg_lanes;  // rows at a time (2 lanes << lg_lanes = 32)
  constexpr int U = 8;
  for (int r0 = 0; r0 < 32; r0 += U * rows) {
    uint4 data[U];
    long long dst[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int r = r0 + k * rows + (lane >> lg_lanes);
      const long long f = __shfl_sync(0xffffffffu, from, r & 31);
      dst[k] = __shfl_sync(0xffffffffu, to, r & 31);
      data[k] = make_uint4(0, 0, 0, 0);
      if (r >= 32 || f == kNoMove)
        dst[k] = -1;
      else if (f >= 0)
        data[k] = *reinterpret_cast<const uint4*>(base + f);
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (dst[k] >= 0) *reinterpret_cast<uint4*>(base + dst[k]) = data[k];
  }
}

}  // namespace
}  // namespace paged

sdpa_status_t launch_paged_write(const paged::Args& a, int row_bytes, const void* k,
                                 const void* v, const int64_t* kn, const int64_t* vn,
                                 void* k_pages, void* v_pages, int elem,
                                 cudaStream_t stream) {
  using namespace paged;
  WriteArgs w;
  w.a = a;
  w.k = static_cast<const char*>(k);
  w.v = static_cast<const char*>(v);
  w.kp = static_cast<char*>(k_pages);
  w.vp = static_cast<char*>(v_pages);
  for (int i = 0; i < 2; ++i) {
    w.kn[i] = kn[i] * elem;
    w.vn[i] = vn[i] * elem;
  }
  for (int i = 0; i < 3; ++i) {
    w.kb[i] = a.ks[i] * elem;
    w.vb[i] = a.vs[i] * elem;
  }
  w.pieces = row_bytes / 16;
  w.lg = 0;
  while ((1 << w.lg) < w.pieces) ++w.lg;
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.T) + kWriteWarps - 1) /
                                              kWriteWarps);
  paged_write_kernel<<<grid, kWriteWarps * 32, 0, stream>>>(w);
  return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

sdpa_status_t launch_paged_evict(const paged::Args& a, int row_bytes, int elem, int keep,
                                 int recent, void* k_pages, void* v_pages, const float* scores,
                                 float* scores_out, const int64_t* ss, int score_len, int* kept,
                                 int* lens_out, cudaStream_t stream, int* launches) {
  using namespace paged;
  EvictArgs e;
  e.a = a;
  e.keep = keep;
  e.recent = recent;
  e.scores = scores;
  e.scores_out = scores_out;
  e.ss[0] = ss[0];
  e.ss[1] = ss[1];
  e.score_len = score_len;
  e.kept = kept;
  e.lens_out = lens_out;
  e.kp = static_cast<char*>(k_pages);
  e.vp = static_cast<char*>(v_pages);
  for (int i = 0; i < 3; ++i) {
    e.kb[i] = a.ks[i] * elem;
    e.vb[i] = a.vs[i] * elem;
  }
  // Lanes of a row in the ordered kernel: a whole row where the budget is one
  // chunk then (fewer CTAs), else 64 bytes (more bytes on their way; 8 x 16384
  // keys in 128-byte slices: 85 us against 89).
  const int row_lanes = row_bytes / 16;
  const int lanes = keep <= move_chunk(row_lanes) ? row_lanes : 4;
  e.slices = row_lanes / lanes;
  // A budget of up to two chunks moves in the ordered kernel alone: a launch
  // less (measured at 2 x 1500 keys, budget 1024: 12.4 us against 16.7), while
  // at 8 x 16384 keys and a budget of 4096 the two take 71 us against 89.
  e.near = keep <= 2 * move_chunk(lanes) ? 0x7fffffff : keep;
  const unsigned bh = static_cast<unsigned>(a.B) * a.Hkv;
  const int cache = a.cap < kSelCache ? a.cap : kSelCache;
  if (!allow_smem<paged_evict_select_kernel<1024>>(kSelCache * 4)) return SDPA_ERR_CUDA;
  // (checked before the first launch, so that a refused call moves nothing)
  if (static_cast<long long>(bh) * 2 * ((keep - 1) / kFarPer + 1) > 0x7fffffffLL)
    return SDPA_ERR_UNSUPPORTED;
  // many short sequences: small CTAs, several an SM (1406 rows of 7 keys 84 ->
  // 32 us; 16 rows of 1500 take 12.0 us with 1024 threads and 13.4 with 256)
  if (a.cap <= 4096 && bh > 256)
    paged_evict_select_kernel<256><<<bh, 256, cache * 4, stream>>>(e, cache);
  else
    paged_evict_select_kernel<1024><<<bh, 1024, cache * 4, stream>>>(e, cache);
  if (cudaGetLastError() != cudaSuccess) return SDPA_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(bh * 2 * e.slices);
  cfg.blockDim = dim3(kMoveT);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto move = lanes == 4    ? paged_evict_move_kernel<4>
              : lanes == 8  ? paged_evict_move_kernel<8>
              : lanes == 16 ? paged_evict_move_kernel<16>
                            : paged_evict_move_kernel<32>;
  if (cudaLaunchKernelEx(&cfg, move, e) != cudaSuccess) return SDPA_ERR_CUDA;
  *launches = 2;
  if (e.near != keep) return SDPA_OK;
  *launches = 3;
  int lg = 0;  // lanes of a row
  while ((16 << lg) < row_bytes) ++lg;
  cfg.gridDim = dim3(bh * 2 * static_cast<unsigned>((keep - 1) / kFarPer + 1));
  cfg.blockDim = dim3(kFarT);
  return cudaLaunchKernelEx(&cfg, paged_evict_far_kernel, e, lg) == cudaSuccess ? SDPA_OK
                                                                                : SDPA_ERR_CUDA;
}

}  // namespace gb300

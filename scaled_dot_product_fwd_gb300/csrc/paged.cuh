// paged.cuh — what the kernels over the paged KV cache share: their
// arguments, the lengths of a sequence, and the division of the work.
//
// Division of the work.  The units of a call are (sequence, kv head, block):
// a block of query rows for attention, a run of keys for the score sums.  A
// unit takes a number of equal steps (key tiles, or query chunks) that
// follows from the lengths and the causal rule, and the lengths are known on
// the device only.  So every CTA computes the whole call's cost (a fixed
// cost and the steps of every unit, summed per sequence in closed form), takes its equal share
// of the line of all units, finds where it begins, and walks on from there.
// A unit that crosses the end of a share is finished by the next CTAs: each
// leaves a partial result in the workspace (slot 1 of the CTA that began the
// unit, slot 0 of those that continue it) and a merge kernel joins them in
// order.  Every CTA is busy equally long whatever the lengths, the workspace
// has a fixed size, and the summation order depends on the lengths alone.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"
#include "sdpa.h"

namespace gb300 {
namespace paged {

constexpr int kStatusPageTable = 7;  // SDPA_ERR_PAGE_TABLE

// Division of n < 2^31 by a number known on the host: a high product, an add
// and a shift (Granlund and Montgomery, "Division by Invariant Integers using
// Multiplication", 1994).  The kernels' single-token paths are chains of
// index arithmetic, in which the divide instruction sequence is several times
// as long.
struct FastDiv {
  uint32_t d, m;
  int l;
  __host__ __device__ __forceinline__ int div(int n) const {
    const uint32_t u = static_cast<uint32_t>(n);
#ifdef __CUDA_ARCH__
    return static_cast<int>((__umulhi(m, u) + u) >> l);
#else
    return static_cast<int>(((static_cast<uint64_t>(m) * u >> 32) + u) >> l);
#endif
  }
  __host__ __device__ __forceinline__ int mod(int n) const {
    return n - div(n) * static_cast<int>(d);
  }
  __host__ __device__ __forceinline__ int ceil(int n) const {
    return div(n + static_cast<int>(d) - 1);
  }
};
inline FastDiv fast_div(int d) {
  FastDiv f;
  f.d = static_cast<uint32_t>(d);
  f.l = 0;
  while ((1u << f.l) < f.d) ++f.l;
  f.m = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << f.l) - f.d)) / f.d + 1);
  return f;
}

struct Args {
  int B, T, Hq, Hkv, G;
  int causal;
  int num_pages, page_size, max_pages;
  int cap;  // max_pages * page_size, at most 2^30
  const int* table;
  long long table_stride;
  const int* cu;    // or nullptr: one token a sequence
  const int* lens;
  const float* sinks;
  long long qs[2], os[2], ks[3], vs[3];
  float sl2;  // scale * log2(e)
  // Query heads of a kv head are taken `gu` at a time (the whole group when
  // it fits a tile's rows), `nsub` times; a tile of `rows` rows holds w =
  // rows / gu tokens, row r = token r / gu, head r % gu.
  int gu, nsub, w;
  FastDiv by_page, by_gu, by_nsub;
  FastDiv by_w;  // tokens of a unit (attention: of all its tiles)
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  float* ws;   // partial results (see the kernels)
  int* desc;   // [CTAs][kDesc]: the unit that a CTA began and did not finish
  int nctas;
  int max_ctas;  // (a test hook may ask for fewer than the plan's)
  // score sums
  float* scores;
  long long ss[2];
  int score_len;
  int* status;
  unsigned long long wait_ns;
};

// Descriptor of a cut unit, written by the CTA that began it: partial
// results it has (0: this CTA cut none), sequence, head unit, block, first
// token row, query tokens, keys.
constexpr int kDesc = 8;

// First packed row, new tokens and keys of a sequence, and the position of its
// first token (negative where the tokens are more than its length).  A length
// past the table's end leaves the tokens their positions: only the keys end
// there (`off` stops at the end too, from where every key is seen).
struct Seq {
  int q0, nq, nk, off;
};
__device__ __forceinline__ Seq seq_of(const Args& a, int b) {
  Seq s;
  if (a.cu) {
    s.q0 = min(max(a.cu[b], 0), a.T);
    s.nq = min(max(a.cu[b + 1], s.q0), a.T) - s.q0;
  } else {
    s.q0 = min(b, a.T);
    s.nq = b < a.T ? 1 : 0;
  }
  const int len = max(a.lens[b], 0);
  s.nk = min(len, a.cap);
  s.off = min(len - s.nq, a.cap);
  return s;
}

// sum over i in [0, n) of floor((a i + b) / m), for n, a, b >= 0 and m >= 1:
// whole parts of a and b are summed directly, and what is left counts the
// lattice points under a line, which swaps the roles of a and m (the steps
// of Euclid's algorithm).
__host__ __device__ inline long long floor_sum(long long n, long long m, long long a,
                                               long long b) {
  long long r = 0;
  while (n > 0) {
    r += (a / m) * (n * (n - 1) / 2) + (b / m) * n;
    a %= m;
    b %= m;
    const long long top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const long long t = m;
    m = a;
    a = t;
  }
  return r;
}

// Steps of the units of one (sequence, kv head).  Attention: block j holds
// `w` tokens and reads the key tiles of `tile` keys up to its last visible
// key.
struct AttendUnits {
  FastDiv by_w;
  int lg, causal;  // tiles of 2^lg keys
  int cost;        // fixed cost of a unit, in steps
  __host__ __device__ int count(const Seq& s) const { return by_w.ceil(s.nq); }
  __host__ __device__ int steps(const Seq& s, int j) const {
    int lim = s.nk;
    if (causal) {
      const long long last = static_cast<long long>(j + 1) * by_w.d;
      lim = last < s.nk - s.off ? s.off + static_cast<int>(last) : s.nk;
    }
    return lim <= 0 ? 0 : (lim + (1 << lg) - 1) >> lg;
  }
  // steps of the blocks before j
  __host__ __device__ long long before(const Seq& s, int j) const {
    if (j <= 0) return 0;
    const long long all = (s.nk + (1 << lg) - 1) >> lg;
    if (!causal) return j * all;
    // blocks whose last token does not see every key: (i + 1) w < nk - off
    const int cut = s.nk > s.off ? by_w.div(s.nk - s.off - 1) : 0;
    const int part = j < cut ? j : cut;
    long long r = (j - part) * all;
    const int off = s.off, w = static_cast<int>(by_w.d);
    const int i0 = off + w > 0 ? 0 : by_w.div(-off);  // first block that sees a key
    if (part > i0)
      r += floor_sum(part - i0, 1LL << lg, w,
                     off + static_cast<long long>(i0 + 1) * w + (1 << lg) - 1);
    return r;
  }
};
// Score sums: unit j holds 2^lg keys and reads the chunks of `w` tokens
// (times nsub head groups) from the first that sees one of its keys.
struct ScoreUnits {
  FastDiv by_w;
  int lg, causal, nsub, cost;
  __host__ __device__ int count(const Seq& s) const {
    return s.nq > 0 ? (s.nk + (1 << lg) - 1) >> lg : 0;
  }
  __host__ __device__ int first(const Seq& s, int j) const {
    const int d = (j << lg) - s.off;
    return causal && d > 0 ? by_w.div(d) : 0;
  }
  __host__ __device__ int steps(const Seq& s, int j) const {
    return (by_w.ceil(s.nq) - first(s, j)) * nsub;
  }
  __host__ __device__ long long before(const Seq& s, int j) const {
    if (j <= 0) return 0;
    long long r = static_cast<long long>(j) * by_w.ceil(s.nq);
    if (causal) {
      const int off = s.off;
      const int i0 = off > 0 ? (off + (1 << lg) - 1) >> lg : 0;  // first j with a cut
      if (j > i0)
        r -= floor_sum(j - i0, by_w.d, 1LL << lg, (static_cast<long long>(i0) << lg) - off);
    }
    return r * nsub;
  }
};

// One unit of a CTA's share, and the steps [s0, s1) of it that are the CTA's.
struct Unit {
  int b, h, j;
  Seq s;
  int steps, s0, s1;
  long long pos;  // position of its step 0 on the line
  __device__ bool whole() const { return s0 == 0 && s1 == steps; }
  __device__ int slot() const { return s0 > 0 ? 0 : 1; }
};

// A CTA's share [begin, end) of the line and where it begins (shared memory;
// made once by plan_share, then every role walks it with Walk).
struct Share {
  long long begin, end, size;
  long long pos;  // start of the first unit
  int b, h, j;    // the first unit (b = B: none)
  int n;          // units of its (sequence, head)
  Seq s;
};

// Units whose cost reaches into the share, in order.
template <typename Units>
struct Walk {
  long long pos;
  int b, h, j, n;
  Seq s;
  __device__ __forceinline__ explicit Walk(const Share& sh)
      : pos(sh.pos), b(sh.b), h(sh.h), j(sh.j), n(sh.n), s(sh.s) {}
  // heads: units of one sequence and block number (kv heads, times nsub)
  __device__ __forceinline__ bool next(const Args& a, const Units& u, const Share& sh, int heads,
                                       Unit* out) {
    while (b < a.B && pos < sh.end) {
      if (j >= n) {
        j = 0;
        if (++h >= heads || n == 0) {
          h = 0;
          if (++b >= a.B) return false;
          s = seq_of(a, b);
          n = u.count(s);
        }
        continue;
      }
      out->b = b;
      out->h = h;
      out->j = j;
      out->s = s;
      const int steps = u.steps(s, j);
      const long long p0 = pos + u.cost;
      const long long lo = sh.begin - p0, hi = sh.end - p0;
      out->steps = steps;
      out->s0 = lo <= 0 ? 0 : lo >= steps ? steps : static_cast<int>(lo);
      out->s1 = hi <= 0 ? 0 : hi >= steps ? steps : static_cast<int>(hi);
      out->pos = p0;
      const bool mine = steps == 0 ? pos >= sh.begin : out->s1 > out->s0;
      pos = p0 + steps;
      ++j;
      if (mine) return true;
    }
    return false;
  }
};

// a / b for a >= 0, b > 0: 32-bit where the numbers allow it (the 64-bit
// sequence is several times as long).
__device__ __forceinline__ long long div_nonneg(long long a, long long b) {
  if (((a | b) >> 31) == 0)
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Divide the line among the grid's CTAs and find this CTA's share.  Every
// thread of the CTA calls it (kThreads of them, whole warps); `scratch`
// holds kThreads / 32 numbers.  Ends with a CTA barrier.
template <int kThreads, typename Units>
__device__ __forceinline__ void plan_share(const Args& a, const Units& u, int heads,
                                           int min_share, long long* scratch, Share* sh) {
  const int tid = threadIdx.x;
  const int per = (a.B + kThreads - 1) / kThreads;  // sequences of a thread
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  auto cost = [&](const Seq& s, int n) {
    return (u.before(s, n) + static_cast<long long>(n) * u.cost) * heads;
  };
  long long mine = 0;
  Seq s{0, 0, 0, 0};
  int n = 0;
  for (int b = b0; b < b1; ++b) {
    s = seq_of(a, b);
    n = u.count(s);
    mine += cost(s, n);
  }
  long long incl = mine;  // inclusive scan over the threads
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, d);
    if ((tid & 31) >= d) incl += t;
  }
  if ((tid & 31) == 31) scratch[tid >> 5] = incl;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i == (tid >> 5)) incl += total;
    total += scratch[i];
  }
  long long size = div_nonneg(total + gridDim.x - 1, gridDim.x);
  if (size < min_share) size = min_share;
  const long long begin = size * blockIdx.x;
  const long long end = begin + size < total ? begin + size : total;
  if (tid == 0) {
    sh->begin = begin;
    sh->end = end;
    sh->size = size;
    if (begin >= total) {
      sh->pos = total;
      sh->b = a.B;
      sh->h = sh->j = sh->n = 0;
      sh->s = Seq{0, 0, 0, 0};
    }
  }
  long long pos = incl - mine;
  if (begin < total && begin >= pos && begin < incl) {
    for (int b = b0; b < b1; ++b) {
      if (b1 - b0 > 1) {
        s = seq_of(a, b);
        n = u.count(s);
      }
      const long long c = b1 - b0 > 1 ? cost(s, n) : mine;
      if (begin < pos + c) {
        const long long per_head = div_nonneg(c, heads);
        const int h = static_cast<int>(div_nonneg(begin - pos, per_head));
        pos += h * per_head;
        // last block that starts at or before `begin`
        int lo = 0, hi = n - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          const long long at = pos + u.before(s, mid) + static_cast<long long>(mid) * u.cost;
          if (at <= begin) lo = mid; else hi = mid - 1;
        }
        sh->b = b;
        sh->h = h;
        sh->j = lo;
        sh->n = n;
        sh->s = s;
        sh->pos = pos + u.before(s, lo) + static_cast<long long>(lo) * u.cost;
        break;
      }
      pos += c;
    }
  }
  __syncthreads();
}

// Partial results that a unit has: the CTAs from the one that holds its
// first step to the one that holds its last.
__device__ __forceinline__ int pieces_of(const Unit& u, const Share& sh) {
  return static_cast<int>(div_nonneg(u.pos + u.steps - 1, sh.size) -
                          div_nonneg(u.pos, sh.size)) + 1;
}

// The sink logit joins a row's denominator (its value row is zero): m, l
// become those of the row with it, and the factor of what was summed before
// is returned.  A sink of -inf adds nothing, also to a row that saw no key.
__device__ __forceinline__ float add_sink(float sink, float& m, float& l) {
  const float sk = sink * 1.4426950408889634f;
  const float mn = fmaxf(m, sk);
  if (mn == -INFINITY) return 1.f;
  const float f = m == -INFINITY ? 0.f : ex2(m - mn);
  l = l * f + ex2(sk - mn);
  m = mn;
  return f;
}

// Page of position p, or -1 (and the status word set) where the table names
// none of the cache's.
__device__ __forceinline__ int page_of(const Args& a, int b, int p) {
  const int page = a.table[b * a.table_stride + a.by_page.div(p)];
  if (page < 0 || page >= a.num_pages) {
    atomicExch(a.status, kStatusPageTable);
    return -1;
  }
  return page;
}

// One copy of box_rows rows of a cache block (encode_row_blocks).
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, uint64_t* bar, int row,
                                         int block) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %3, %3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(row >> 3), "r"(block)
      : "memory");
}

// The page table as a producer warp reads it: the entries of 32 boxes of a
// piece at a time, one a lane, fetched one batch before their use (a lookup a
// tile, its load and its divisions, held a tile's copies back by more than a
// microsecond).
struct Boxes {
  const Args& a;
  const int* table;  // the sequence's row
  int key0, nk;      // first key of the piece, keys of the sequence
  int lg, nbox, lane;  // boxes of 2^lg rows, boxes of a tile
  int cur_page, cur_row, nxt_page, nxt_row;
  __device__ __forceinline__ Boxes(const Args& args, int b, int first_key, int keys, int lg_rows,
                                   int lane_)
      : a(args), table(args.table + b * args.table_stride), key0(first_key), nk(keys),
        lg(lg_rows), nbox(128 >> lg_rows), lane(lane_), cur_page(-1), cur_row(0) {
    fetch(0);
  }
  __device__ __forceinline__ void fetch(int batch) {
    const int key = key0 + ((batch * 32 + lane) << lg);
    nxt_page = -1;
    nxt_row = 0;
    if (key < nk) {
      const int i = a.by_page.div(key);
      nxt_row = key - i * a.page_size;
      nxt_page = table[i];
    }
  }
  // Box `lane` of the piece's key tile j (asked for in order): false where
  // there is none; page -1 where the table names none of the cache's.
  __device__ __forceinline__ bool tile(int j, int* page, int* row) {
    const int q = j * nbox;
    if ((q & 31) == 0) {
      cur_page = nxt_page;
      cur_row = nxt_row;
      fetch((q >> 5) + 1);
    }
    const int src = (q & 31) + (lane & (nbox - 1));
    *page = __shfl_sync(0xffffffffu, cur_page, src);
    *row = __shfl_sync(0xffffffffu, cur_row, src);
    if (lane >= nbox || key0 + ((q + lane) << lg) >= nk) return false;
    if (*page < 0 || *page >= a.num_pages) {
      atomicExch(a.status, kStatusPageTable);
      *page = -1;
    }
    return true;
  }
};

}  // namespace paged

// Launchers (host side).  `a` holds the problem and the workspace; the
// attention and score launchers fill in the tile's rows (gu, nsub, w).
sdpa_status_t launch_paged_simt(paged::Args a, int head_dim, int dtype, const LaunchEnv& env);
int paged_vector_rows(const paged::Args& a);
sdpa_status_t launch_paged_vector_f32(paged::Args a, int head_dim, int rows,
                                      const LaunchEnv& env);
sdpa_status_t launch_paged_scores_vector_f32(paged::Args a, int head_dim, int rows,
                                             const LaunchEnv& env);
sdpa_status_t launch_paged_scores_simt(paged::Args a, int head_dim, int dtype,
                                       const LaunchEnv& env);
sdpa_status_t launch_paged_tc_d64(paged::Args a, int dtype, const LaunchEnv& env);
sdpa_status_t launch_paged_tc_d128(paged::Args a, int dtype, const LaunchEnv& env);
// Rows of a tile of the few-row kernel for this call (8 or 16; 0: the calls
// of more rows take paged_tc.cuh).
int paged_decode_rows(const paged::Args& a);
sdpa_status_t launch_paged_decode_tc(const paged::Args& a, int head_dim, int dtype, int rows,
                                     const LaunchEnv& env);
sdpa_status_t launch_paged_scores_tc(paged::Args a, int head_dim, int dtype,
                                     const LaunchEnv& env);
sdpa_status_t launch_paged_merge(const paged::Args& a, int head_dim, int dtype, int tile_rows,
                                 int tiles, cudaStream_t stream);
sdpa_status_t launch_paged_scores_merge(const paged::Args& a, int tile_keys,
                                        cudaStream_t stream);
sdpa_status_t launch_paged_write(const paged::Args& a, int row_bytes, const void* k,
                                 const void* v, const int64_t* kn, const int64_t* vn,
                                 void* k_pages, void* v_pages, int elem, cudaStream_t stream);
sdpa_status_t launch_paged_evict(const paged::Args& a, int row_bytes, int elem, int keep,
                                 int recent, void* k_pages, void* v_pages, const float* scores,
                                 float* scores_out, const int64_t* ss, int score_len, int* kept,
                                 int* lens_out, cudaStream_t stream, int* launches);

namespace paged {
// The tensor-core kernels see a cache as blocks of page_size rows, block (page,
// head) at unit * (page * page_mul + head * head_mul) elements, the unit
// being the greatest common divisor of the two strides.  `blocks` is one past
// the last; a copy of that block reads zero (a bad page).
struct CacheBlocks {
  int page_mul, head_mul, blocks;
};
inline bool cache_blocks(const long long (&st)[3], int pages, int heads, CacheBlocks* c,
                         long long* unit) {
  long long x = pages > 1 ? st[0] : 0, y = heads > 1 ? st[1] : 0;
  long long u = x, v = y;
  while (v) {
    const long long t = u % v;
    u = v;
    v = t;
  }
  if (u == 0) u = 64;  // one block
  const long long last = (pages - 1) * (x / u) + (heads - 1) * (y / u);
  if (x / u > 0x7fffffffLL || y / u > 0x7fffffffLL || last >= 0x7fffffffLL) return false;
  c->page_mul = static_cast<int>(x / u);
  c->head_mul = static_cast<int>(y / u);
  c->blocks = static_cast<int>(last) + 1;
  *unit = u;
  return true;
}

// Heads per tile and tokens per tile of `rows` query rows.
inline void fit_rows(Args& a, int rows, int tiles = 1) {
  a.nsub = (a.G + rows - 1) / rows;
  a.gu = (a.G + a.nsub - 1) / a.nsub;
  a.w = rows / a.gu;
  a.by_gu = fast_div(a.gu);
  a.by_nsub = fast_div(a.nsub);
  a.by_w = fast_div(a.w * tiles);
}
// Lets a kernel have `bytes` of dynamic shared memory on the current device;
// done once a device.
template <auto kKernel>
bool allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load() & bit) return true;
  if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return false;
  done.fetch_or(bit);
  return true;
}

// Query rows (tokens times heads of a kv head) of a sequence on average, by
// which a kernel is chosen: the offsets are on the device.  A chunk among
// single tokens is read in passes of few rows then.  Where the chunk's keys are
// about as many as theirs, its passes weigh about what the single tokens do;
// where they are many more, the passes are the call's whole time, and the
// kernels of many rows would be several times as fast.  Attention / score sums
// (us) with the kernels chosen here and with those of many rows, 32 heads over
// 8, head_dim 128, bf16, and 16 heads over 4 in fp32:
//   255 single tokens and a chunk of 257, all over 4096 keys:
//       bf16 687 / 521 and 671 / 912; fp32 1066 / 2540 and 3573 / 3176
//   128 single tokens over 512 keys and a chunk of 384 over 32768:
//       bf16 1398 / 337 and 272 / 147; fp32 7083 / 3210 and 2753 / 1604
//   255 single tokens over 64 keys and a chunk of 257 over 32768:
//       bf16 1789 / 245 and 249 / 132; fp32 3340 / 4586 and 1904 / 1042
inline long long call_rows(const Args& a) {
  return a.cu ? (static_cast<long long>(a.T) * a.G + a.B - 1) / a.B : a.G;
}

// Rows of a page box: log2 of gcd(page_size, 128).
inline int box_log2(int page_size) {
  int lg = 7;
  while (page_size & ((1 << lg) - 1)) --lg;
  return lg;
}
// Largest tile whose partial results a CTA may leave, in query rows: two
// 128-row tiles.  (Score sums leave one number a key, at most 256.)
constexpr int kMaxRows = 256;
// CTAs an SM that share a call's work, at most (their slots' rows together
// are at most kMaxRows an SM).
constexpr int kMaxCtas = 4;
}  // namespace paged

}  // namespace gb300

// rope.cu — rotary positions of q and k (and the transposed rotation, for
// their gradients), and the table of cosines and sines that the rotary calls
// read.
//
// Rotation: bound by HBM (q and k in and out).  A thread takes a 16-element
// piece of a row (rotate.cuh), holds its 8 cosines and sines in registers and
// walks over `per` heads with them (RopeArgs, chosen at the launch), so that a
// pair's 8 bytes of the table are read once for `per` heads.  A warp's D / 16 lanes a
// row leave it 32 * 16 / D rows at a time: consecutive tokens where a head's
// tokens lie next to one another, consecutive heads where a token's heads do,
// so that a warp's accesses are runs of 1 KB in either order.
// 2 x 76 heads x 4250 tokens x 64, fp16: 28.0 us a call (166 MB, 5.9 TB/s; the
// kernel alone 25.2, the copy rate); gradients of 8192 tokens, 40 heads, head_dim
// 128, bf16, token after token: 31.0 us (5.5 TB/s; 38.9 before a thread had its
// next heads' pieces on their way and the heads were shared out evenly).  One,
// two and four pieces at a time: 31.7, 30.3 and 31.7 us (the first case, before
// launches overlapped).
#include <cuda_runtime.h>

#include <algorithm>

#include "paged.cuh"
#include "rotate.cuh"

namespace gb300 {
namespace rotary {
namespace {

using paged::FastDiv;
using paged::fast_div;

constexpr int kWarps = 8;

struct RopeArgs {
  Rotation rot;
  long long pos_stride;  // of a batch
  int n;                 // tokens (batch * seq_len)
  int Hq, H;             // query heads, all heads
  int lg_u;              // log2 of the pieces of a row
  int lg_t;              // log2 of a warp's tokens
  int per;               // heads of a thread
  float sign;
  FastDiv by_len;
  const char* in[2];
  char* out[2];
  long long is[2][3], os[2][3];  // byte strides (batch, head, row)
  int* status;
};

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const RopeArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = lane & ((1 << a.lg_u) - 1), r = lane >> a.lg_u;
  const int lg_h = 5 - a.lg_u - a.lg_t;  // log2 of heads at a time
  griddep_launch_dependents();
  griddep_wait();
  const long long t =
      ((static_cast<long long>(blockIdx.x) * kWarps + warp) << a.lg_t) + (r & ((1 << a.lg_t) - 1));
  if (t >= a.n) return;
  const int b = a.by_len.div(static_cast<int>(t));
  const int l = static_cast<int>(t) - b * static_cast<int>(a.by_len.d);
  const Piece pc = piece_of<false>(a.rot, 16 << a.lg_u, u);
  const int h0 = blockIdx.y * a.per * (1 << lg_h) + (r >> a.lg_t);
  constexpr int U = sizeof(T) == 4 ? 1 : 2;  // heads at a time
  Raw<T> lo[U], hi[U];
  auto load = [&](int i, Raw<T>& x0, Raw<T>& x1) {  // head number i of this thread
    const int h = h0 + (i << lg_h);
    if (i < a.per && h < a.H) {
      const int w = h >= a.Hq, g = w ? h - a.Hq : h;
      const T* x = reinterpret_cast<const T*>(a.in[w] + b * a.is[w][0] + g * a.is[w][1] +
                                              l * a.is[w][2]);
      x0 = load8(x + pc.lo);
      x1 = load8(x + pc.hi);
    }
  };
#pragma unroll
  for (int k = 0; k < U; ++k) load(k, lo[k], hi[k]);
  bool turned = pc.turned;
  Angles ang = {};
  {
    const long long pos = a.rot.positions ? a.rot.positions[b * a.pos_stride + l] : l;
    if (pos < 0 || pos >= a.rot.len) {
      if (u == 0 && turned) atomicExch(a.status, kStatusPosition);
      turned = false;
    }
    if (turned) ang = load_angles(a.rot, pos, pc);
  }
  for (int i = 0; i < a.per; i += U) {
    Raw<T> nlo[U], nhi[U];  // the next heads' pieces are on their way meanwhile
#pragma unroll
    for (int k = 0; k < U; ++k) load(i + U + k, nlo[k], nhi[k]);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int h = h0 + ((i + k) << lg_h);
      if (i + k < a.per && h < a.H) {
        const int w = h >= a.Hq, g = w ? h - a.Hq : h;
        T* x = reinterpret_cast<T*>(a.out[w] + b * a.os[w][0] + g * a.os[w][1] + l * a.os[w][2]);
        if (turned) {
          Values v;
          widen8(lo[k], v.lo);
          widen8(hi[k], v.hi);
          turn_piece<false>(v, ang, a.rot.interleaved, a.sign);
          lo[k] = narrow8<T>(v.lo);
          hi[k] = narrow8<T>(v.hi);
        }
        store8(x + pc.lo, lo[k]);
        store8(x + pc.hi, hi[k]);
      }
      lo[k] = nlo[k];
      hi[k] = nhi[k];
    }
  }
}

// The table: a thread an entry, the angle and its functions in fp64 (a
// position of 10^6 leaves an fp32 angle 2 decimal digits).  Made once for a
// model, so its time (131072 x 64 entries) does not count.
constexpr int kMaxPairs = 256;
struct Frequencies {
  double f[kMaxPairs];
};
__global__ void __launch_bounds__(256)
    rope_table_kernel(float2* table, long long length, int half, const Frequencies w,
                      double gain) {
  const long long n = length * half;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const long long p = i / half;
    double s, c;
    sincos(static_cast<double>(p) * w.f[i - p * half], &s, &c);
    table[i] = make_float2(static_cast<float>(gain * c), static_cast<float>(gain * s));
  }
}

}  // namespace
}  // namespace rotary

sdpa_status_t launch_rope_table(float* table, long long length, int rotary_dim,
                                const double* inv_freq, double gain, cudaStream_t stream) {
  using namespace rotary;
  Frequencies w = {};
  for (int i = 0; i < rotary_dim / 2; ++i) w.f[i] = inv_freq[i];
  const long long blocks = (length * (rotary_dim / 2) + 255) / 256;
  rope_table_kernel<<<static_cast<unsigned>(std::min(blocks, 1LL << 16)), 256, 0, stream>>>(
      reinterpret_cast<float2*>(table), length, rotary_dim / 2, w, gain);
  return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

sdpa_status_t launch_rope(const sdpa_rope_params_t& p, const void* q, const void* k, void* q_out,
                          void* k_out, const LaunchEnv& env) {
  using namespace rotary;
  const int es = p.dtype == SDPA_F32 ? 4 : 2;
  RopeArgs a = {};
  a.rot = make_rotation(&p.rotation);
  a.pos_stride = p.position_stride;
  a.n = p.batch * p.seq_len;
  a.Hq = p.num_q_heads;
  a.H = p.num_q_heads + p.num_kv_heads;
  a.lg_u = p.head_dim == 64 ? 2 : p.head_dim == 128 ? 3 : 5;
  a.sign = p.transpose ? -1.f : 1.f;
  a.by_len = paged::fast_div(p.seq_len);
  a.in[0] = static_cast<const char*>(q);
  a.in[1] = static_cast<const char*>(k);
  a.out[0] = static_cast<char*>(q_out);
  a.out[1] = static_cast<char*>(k_out);
  for (int i = 0; i < 3; ++i) {
    a.is[0][i] = p.q_stride[i] * es;
    a.is[1][i] = p.k_stride[i] * es;
    a.os[0][i] = p.q_out_stride[i] * es;
    a.os[1][i] = p.k_out_stride[i] * es;
  }
  a.status = env.status;
  // a warp's rows: tokens where the next token is nearer than the next head
  const bool tokens = p.seq_len > 1 && p.q_stride[2] <= p.q_stride[1];
  const int lg_rows = 5 - a.lg_u;
  a.lg_t = tokens ? lg_rows : 0;
  const int heads = (a.H + (1 << (lg_rows - a.lg_t)) - 1) >> (lg_rows - a.lg_t);  // times
  const long long warps = (static_cast<long long>(a.n) + (1 << a.lg_t) - 1) >> a.lg_t;
  // Heads of a thread: 8 (the table then costs 1 / 8 of the row's bytes again,
  // from L2), fewer where the call would not fill the GPU.  4, 8 and 16 heads: 31.5,
  // 30.3 and 32.3 us on the first case above, 33.4, 33.7 and 32.4 on the second.
  int per = 8;
  while (per > 1 && warps * ((heads + per - 1) / per) < 32LL * env.num_sms) per >>= 1;
  per = std::max(per, (heads + 65534) / 65535);
  per = (heads + (heads + per - 1) / per - 1) / ((heads + per - 1) / per);  // (even shares)
  a.per = per;
  const dim3 grid(static_cast<unsigned>((warps + kWarps - 1) / kWarps),
                  static_cast<unsigned>((heads + per - 1) / per));
  auto go = [&](auto kern) {
    return paged::launch_overlapped(kern, grid, kWarps * 32, 0, env.stream, a);
  };
  if (p.dtype == SDPA_F32) return go(rope_kernel<float>);
  return p.dtype == SDPA_F16 ? go(rope_kernel<__half>) : go(rope_kernel<__nv_bfloat16>);
}

}  // namespace gb300

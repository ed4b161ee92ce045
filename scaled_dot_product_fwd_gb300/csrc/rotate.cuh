// rotate.cuh — the rotation of a head's pairs as the rotary kernels share it.
//
// A row of D elements is D / 16 pieces, one a thread: two runs of 8 elements,
// half of the rotated (or of the other) elements apart, so that neighbouring
// lanes' 16-byte accesses are neighbours in memory.  In the halves form the
// runs are each other's partners, in the interleaved form each holds whole
// pairs; either way a thread needs 64 bytes of the table.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "sdpa.h"

namespace gb300 {
namespace rotary {

constexpr int kStatusPosition = 8;  // SDPA_ERR_POSITION

struct Rotation {
  const float* table;
  long long len;
  int R;            // 0: no rotation
  int interleaved;
  const int* positions;
};
inline Rotation make_rotation(const sdpa_rotation_t* r) {
  Rotation x = {};
  if (r) x = Rotation{r->table, r->table_len, r->rotary_dim, r->interleaved ? 1 : 0, r->positions};
  return x;
}

// Elements of piece u of a row of D: the runs of 8 from lo and from hi.
// kWhole: 16 consecutive elements where the pairs allow it.
struct Piece {
  int lo, hi;
  bool turned;
};
template <bool kWhole>
__device__ __forceinline__ Piece piece_of(const Rotation& r, int D, int u) {
  const bool turned = 16 * u < r.R;
  if (kWhole && !(turned && !r.interleaved)) return Piece{16 * u, 16 * u + 8, turned};
  const int first = turned ? 0 : r.R, count = turned ? r.R : D - r.R;
  const int lo = first + 8 * (u - first / 16);
  return Piece{lo, lo + count / 2, turned};
}

// Eight elements of a row in fp32 (lo, hi: the piece's runs).
struct Values {
  float lo[8], hi[8];
};

template <typename T>
struct Raw {  // eight elements as they lie in memory
  uint4 r[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load8(const T* p) {
  Raw<T> x;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    x.r[i] = reinterpret_cast<const uint4*>(p)[i];
  return x;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Raw<T>& x) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    reinterpret_cast<uint4*>(p)[i] = x.r[i];
}
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float v, float* x) { *x = v; }
__device__ __forceinline__ void from_float(float v, __half* x) { *x = __float2half_rn(v); }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16* x) {
  *x = __float2bfloat16_rn(v);
}
template <typename T>
__device__ __forceinline__ void widen8(const Raw<T>& x, float (&v)[8]) {
  const T* e = reinterpret_cast<const T*>(&x);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_float(e[i]);
}
template <typename T>
__device__ __forceinline__ Raw<T> narrow8(const float (&v)[8]) {
  Raw<T> x;
  T* e = reinterpret_cast<T*>(&x);
#pragma unroll
  for (int i = 0; i < 8; ++i) from_float(v[i], &e[i]);
  return x;
}

// (x, y) turned by (c, s).  kExact: the two sums of products rounded once from
// about 48 bits (the products' and the sum's rounding errors are computed with
// fma and added up: Dekker 1971, Knuth's two-sum), so that a 4-bit code next to
// a border does not turn on the order of operations.  A sum that is not finite
// has no such errors (inf - inf): it is what the plain form makes of it.
template <bool kExact>
__device__ __forceinline__ float dot2(float x, float c, float y, float s) {  // x c + y s
  if constexpr (!kExact) return fmaf(x, c, y * s);
  const float p = __fmul_rn(x, c), pe = __fmaf_rn(x, c, -p);
  const float q = __fmul_rn(y, s), qe = __fmaf_rn(y, s, -q);
  const float t = __fadd_rn(p, q);
  const float b = __fsub_rn(t, p);
  const float e = __fadd_rn(__fsub_rn(p, __fsub_rn(t, b)), __fsub_rn(q, b));
  const float r = __fadd_rn(t, __fadd_rn(e, __fadd_rn(pe, qe)));
  return fabsf(t) < INFINITY ? r : __fmaf_rn(x, c, q);
}
template <bool kExact>
__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float rx = dot2<kExact>(x, c, -y, s), ry = dot2<kExact>(y, c, x, s);
  x = rx;
  y = ry;
}

// Cosines and sines of a piece's 8 pairs.
struct Angles {
  float4 cs[4];
};
__device__ __forceinline__ Angles load_angles(const Rotation& r, long long pos, const Piece& p) {
  Angles a;
  // pair i of the halves form at 2 i, of the interleaved form at its element
  const float* t = r.table + pos * r.R;
  const float4* lo = reinterpret_cast<const float4*>(t + (r.interleaved ? p.lo : 2 * p.lo));
  const float4* hi = r.interleaved ? reinterpret_cast<const float4*>(t + p.hi) : lo + 2;
  a.cs[0] = __ldg(lo);
  a.cs[1] = __ldg(lo + 1);
  a.cs[2] = __ldg(hi);
  a.cs[3] = __ldg(hi + 1);
  return a;
}
template <bool kExact>
__device__ __forceinline__ void turn_piece(Values& v, const Angles& a, bool interleaved,
                                           float sign) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4& f = a.cs[i >> 1];
    const float c = i & 1 ? f.z : f.x, s = (i & 1 ? f.w : f.y) * sign;
    if (interleaved) {
      if (i < 4)
        turn<kExact>(v.lo[2 * i], v.lo[2 * i + 1], c, s);
      else
        turn<kExact>(v.hi[2 * i - 8], v.hi[2 * i - 7], c, s);
    } else {
      turn<kExact>(v.lo[i], v.hi[i], c, s);
    }
  }
}

}  // namespace rotary

// Checks of a rotation's description for rows of head_dim elements (host).
sdpa_status_t check_rotation(const sdpa_rotation_t& r, int head_dim);
// Launchers (host side).
sdpa_status_t launch_rope_table(float* table, long long length, int rotary_dim,
                                const double* inv_freq, double gain, cudaStream_t stream);
sdpa_status_t launch_rope(const sdpa_rope_params_t& p, const void* q, const void* k, void* q_out,
                          void* k_out, const LaunchEnv& env);

}  // namespace gb300

// paged_fp4.cuh — what the attention kernels over the 4-bit paged cache share:
// the second part of fp32 calls' weights, and the codes as tensor copies see them.
#pragma once

#include <algorithm>

#include "paged.cuh"
#include "tensor_map.h"

namespace gb300 {
namespace paged {

// fp32 calls multiply a softmax weight with its value as two fp16 parts.  The
// second, what the first leaves, is this times larger than the first before it
// is rounded: below 2^-14 the first part's steps stay 2^-24, and the second, at
// the same scale, would be 0.  (The first is at most 2^15, so what it leaves at
// most 2^3, and the second at most 2^15.)  The two hold a weight to 2^-22 of
// itself, or to 2^-37 of the first part's unit where it is small.
constexpr float kRestScale = 0x1p12f;

// What h, p rounded, leaves of p, times kRestScale (exact; given p times that).
__device__ __forceinline__ float rest_of(float scaled, __half h) {
  float r;
  asm("fma.rn.f32.f16 %0, %1, %2, %3;"
      : "=f"(r)
      : "h"(__half_as_ushort(h)), "h"(__half_as_ushort(__float2half_rn(-kRestScale))),
        "f"(scaled));
  return r;
}

// How codes reach shared memory: a tensor copy of 2^lg rows of one head at
// coordinates {0, row, head, page}, or, where no 8 rows are sure to share a page
// (lg < 0), 16-byte copies.  A dimension of stride 0 has an extent of 1 and its
// coordinate times 0.
struct CodeMaps {
  int lg;
  int k_page_mul, k_head_mul, k_no_page;  // no_page: a page that reads as zeros
  int v_page_mul, v_head_mul, v_no_page;
};

namespace {
// Maps for boxes of at most 2^max_lg rows (null maps, lg = -1: see above).
inline CodeMaps encode_code_maps(const Args& a, int row_bytes, int max_lg,
                                 CUtensorMapSwizzle swizzle, CUtensorMap* tk, CUtensorMap* tv) {
  CodeMaps m = {};
  m.lg = std::min(box_log2(a.page_size), max_lg);
  auto encode = [&](CUtensorMap* map, const void* base, const long long (&st)[3], int* page_mul,
                    int* head_mul, int* no_page) {
    for (int i = 0; i < 3; ++i)
      if (st[i] >= (1LL << 40)) return false;
    if (a.page_size > 1 && st[2] == 0) return false;
    const bool flat_page = a.num_pages > 1 && st[0] == 0, flat_head = a.Hkv > 1 && st[1] == 0;
    *page_mul = flat_page ? 0 : 1;
    *head_mul = flat_head ? 0 : 1;
    *no_page = flat_page ? 1 : a.num_pages;
    auto s = [&](long long x) { return static_cast<uint64_t>(x > 0 ? x : row_bytes); };
    return encode_tiled_4d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, row_bytes, a.page_size,
                           flat_head ? 1 : a.Hkv, *no_page, 1, row_bytes, 1u << m.lg, s(st[2]),
                           s(st[1]), s(st[0]), swizzle);
  };
  if (a.num_pages < 1 || m.lg < 3 ||
      !encode(tk, a.k, a.ks, &m.k_page_mul, &m.k_head_mul, &m.k_no_page) ||
      !encode(tv, a.v, a.vs, &m.v_page_mul, &m.v_head_mul, &m.v_no_page))
    m.lg = -1;
  return m;
}
}  // namespace

}  // namespace paged
}  // namespace gb300

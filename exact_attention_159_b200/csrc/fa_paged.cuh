// fa_paged.cuh -- what the kernels of the paged key/value cache share: the ragged batch, its checks on
// the device, and the e4m3 conversions.
//
// A cache is K and V pages [num_pages, Hkv, page_size, D] (bf16 or e4m3), for e4m3 with one fp32 scale per
// page and head; sequence b's token p lives in slot p % page_size of page block_table[b][p / page_size].
// Everything a kernel reads from those index arrays is checked before it addresses memory with it; what is
// out of range is left out and recorded in the status word (sites kSitePaged | n), never followed.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "sm100.cuh"

#define FA_HD __host__ __device__ __forceinline__

namespace fa {

enum : int {
  kSitePaged = 0xE00,
  kBadRows = kSitePaged | 1,      // cu_q decreases, leaves [0, T], or a sequence has more than max_q rows
  kBadLength = kSitePaged | 2,    // a length below 0, beyond the block table, or (append) below the new rows
  kBadPage = kSitePaged | 3,      // a page number outside [0, num_pages)
  kBadPosition = kSitePaged | 4,  // a position beyond the rotation's tables
};

// The next kernel of the stream, if it was launched to overlap with this one, may be scheduled from here on.
__device__ __forceinline__ void grid_dependency_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Waits for the kernel before, if this one was launched to overlap with it, to end, its writes visible.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// a / b, of 32 bits where both are (64-bit divisions are a long dependent sequence at every CTA's start).
FA_HD long long divide(long long a, long long b) {
  return ((a | b) >> 31) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

struct PagedBatch {
  const int* table;  // [B, max_pages]
  const int* cu_q;   // [B + 1]
  const int* lens;   // [B]
  int B, T, max_q, max_pages;
  int num_pages, page_shift, Hkv;
  int* status;
};

struct SeqInfo {
  int row0, rows, len;  // first token row, new rows, tokens in all
  bool cut;             // the length is not the one given, which was below 0 or beyond the block table
};

FA_HD void record(int* status, int what) {
#ifdef __CUDA_ARCH__
  atomicCAS(status, 0, what);
#else  // the plans are also run on the host, by their tests
  if (*status == 0) *status = what;
#endif
}

// Sequence b, reduced to what is safe to read: no rows where cu_q cannot be trusted, and no more keys than the
// block table names (a length cut to it moves the new rows' positions, so nothing may be written by it).
FA_HD SeqInfo load_seq(const PagedBatch& p, int b) {
  SeqInfo s;
  const int r0 = p.cu_q[b], r1 = p.cu_q[b + 1];
  s.len = p.lens[b];
  s.row0 = r0;
  s.rows = r1 - r0;
  if (r0 < 0 || r1 < r0 || r1 > p.T || s.rows > p.max_q) {
    s.row0 = s.rows = 0;
    record(p.status, kBadRows);
  }
  const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
  s.cut = s.len < 0 || s.len > cap;
  if (s.cut) {
    s.len = s.len < 0 ? 0 : static_cast<int>(cap);
    record(p.status, kBadLength);
  }
  return s;
}

// The page holding the tokens of block `i` of sequence b, or -1 (recorded) when its number is out of range.
FA_HD int load_page(const PagedBatch& p, int b, int i) {
  const int page = p.table[static_cast<size_t>(b) * p.max_pages + i];
  if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) return page;
  record(p.status, kBadPage);
  return -1;
}

// e4m3 of two floats (round to nearest even, saturating; NaN stays NaN), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// The four e4m3 values of a word as halves (exact: e4m3's values and subnormals are normal halves), the low
// two in `lo`.
__device__ __forceinline__ void halves_of_e4m3(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

// The smallest scale a page gets, and the exponent of the smallest power of two 2^e >= 2^kScaleMinExp with
// amax <= 448 * 2^e: 448 = 1.75 * 2^8, so the exponent of amax minus 8, one more when its mantissa is
// above 1.75.  Powers of two cost e4m3 no precision (its steps are relative, only the bottom of its
// 2^18 range moves by at most one binade) and make growing a page's scale exact for its earlier codes
// except those that fall among e4m3's subnormals.
constexpr int kScaleMinExp = -100;
__device__ __forceinline__ float needed_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < kScaleMinExp ? kScaleMinExp : e;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

}  // namespace fa

// fa_paged_join.cuh -- joins the parts of the items that the paged kernels' cuts divide.
//
// A part holds, for each of its rows, O = sum w v unnormalised, the reference m (log2 units) that w is
// relative to, and l = sum w; the row's result is sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.  Blocks look at
// one cut each and join the item it falls into when no earlier cut does; a thread takes four columns of a
// row.  Bound by the latency of a few dependent loads (few rows), or by reading the parts (many rows).
#pragma once

#include "fa_paged_decode.cuh"
#include "fa_paged_prefill.cuh"

namespace fa {

constexpr int kJoinThreads = 128;
constexpr int kJoinSplit = 8;  // blocks that share the rows of a cut of the kernel of many rows

struct JoinItem {
  const float* part_o;
  const float2* part_ml;
  int first, last;     // shares that hold parts of it
  int slot_rows;       // rows of a slot
  int row0, rows;      // the item's first row among the sequence's rows * G, and its number of rows
  int token0, G, Hq, h;
  __nv_bfloat16* O;
  float* LSE;
};

template <int D>
__device__ __forceinline__ void join_rows(const JoinItem& it, int begin, int end) {
  auto slot = [&](int cta) { return static_cast<size_t>(decode_slot(cta, cta - it.first)) * it.slot_rows; };
  for (int i = begin * (D / 4) + threadIdx.x; i < end * (D / 4); i += kJoinThreads) {
    const int lr = i / (D / 4), col = (i % (D / 4)) * 4;
    float m = -INFINITY;
#pragma unroll 4
    for (int k = it.first; k <= it.last; ++k) m = fmaxf(m, it.part_ml[slot(k) + lr].x);
    float l = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = it.first; k <= it.last; ++k) {
      const float2 ml = it.part_ml[slot(k) + lr];
      if (ml.x == -INFINITY) continue;  // a part in which the row sees no key; its O may not be written
      const float4 v = *reinterpret_cast<const float4*>(it.part_o + (slot(k) + lr) * D + col);
      const float f = exp2f(ml.x - m);
      l = fmaf(f, ml.y, l);
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int row = it.row0 + lr;
    const size_t at = static_cast<size_t>(it.token0 + row / it.G) * it.Hq + it.h * it.G + row % it.G;
    *reinterpret_cast<uint2*>(it.O + at * D + col) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (col == 0) it.LSE[at] = l > 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
}

// Blocks 0 .. n_dec - 2: the cuts of decode_kernel's n_dec shares; after them kJoinSplit blocks for each cut
// of prefill_kernel's.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const DecodeParams dec, const PrefillParams pre, int n_dec) {
  __shared__ long long scratch[kJoinThreads / 32 + 2];
  grid_dependency_wait();  // the parts are written
  JoinItem it;
  if (static_cast<int>(blockIdx.x) < n_dec - 1) {
    const int c = blockIdx.x + 1;
    const DecodeShare s = decode_share<kJoinThreads>(dec, c, n_dec, scratch);
    if (s.b >= dec.b.B) return;
    const DecodeSeq d = decode_seq(dec, s.b);
    const DecodeCut cut = decode_cut(s.per, c, s.off, d.tiles);
    if (cut.last < c || cut.first != c - 1) return;
    const int rb = cut.item / dec.b.Hkv;
    it.part_o = dec.part_o;
    it.part_ml = dec.part_ml;
    it.first = cut.first;
    it.last = cut.last;
    it.slot_rows = dec.rows;
    it.row0 = rb * dec.rows;
    it.rows = min(dec.rows, d.s.rows * dec.G - it.row0);
    it.token0 = d.s.row0;
    it.h = cut.item % dec.b.Hkv;
    it.G = dec.G;
    it.Hq = dec.Hq;
    it.O = dec.O;
    it.LSE = dec.LSE;
    join_rows<D>(it, 0, it.rows);
    return;
  }
  const int i = blockIdx.x - (n_dec - 1), c = i / kJoinSplit + 1, part = i % kJoinSplit;
  const PrefillShare s = prefill_share<kJoinThreads>(pre, c, scratch);
  if (s.b >= pre.b.B) return;
  const PrefillSeq d = prefill_seq(pre, s.b);
  const PrefillAt a = prefill_at(d, s.off);
  const PrefillCut cut = prefill_cut(s.per, c, a, d.count(a.p));
  if (cut.last < c || cut.first != c - 1) return;
  it.part_o = pre.part_o;
  it.part_ml = pre.part_ml;
  it.first = cut.first;
  it.last = cut.last;
  it.slot_rows = kPreRows;
  it.row0 = a.p * kPreRows;
  it.rows = min(kPreRows, d.s.rows * pre.G - it.row0);
  it.token0 = d.s.row0;
  it.h = a.h;
  it.G = pre.G;
  it.Hq = pre.Hq;
  it.O = pre.O;
  it.LSE = pre.LSE;
  constexpr int R = kPreRows / kJoinSplit;
  join_rows<D>(it, min(part * R, it.rows), min((part + 1) * R, it.rows));
}

}  // namespace fa

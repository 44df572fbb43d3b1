// fa_paged_join.cuh -- joins the parts of the items that the paged kernels' cuts divide.
//
// A part holds, for each of its rows, O = sum w v unnormalised, the reference m (log2 units) that w is
// relative to, and l = sum w; the row's result is sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.  Blocks look at
// one cut each and join the item it falls into when no earlier cut does.  Few rows have many parts (a long
// cache over all SMs: 37 of them) and what counts is how many loads are under way: a block of four warps
// takes one row, a quarter of its parts each, lanes holding the parts' weights.  Many rows mostly have two or three
// parts: a warp takes two rows, and adds their parts one after the other (up to 148 where one short chunk lies over
// a long cache: 16 tokens of 8 heads over 131072 keys are 128).  Where a cut falls was left in the workspace by the
// CTA whose share begins there: making the plan again in every block cost more than the join (65 us for a batch of
// prompts).
#pragma once

#include "fa_paged_decode.cuh"
#include "fa_paged_prefill.cuh"

namespace fa {

constexpr int kJoinThreads = 128;
constexpr int kJoinPreRows = 8;                        // rows of a block of the kernel of many rows
constexpr int kJoinPreSplit = kPreRows / kJoinPreRows;  // its blocks for a cut

struct JoinItem {
  const float* part_o;
  const float2* part_ml;
  int first, last;  // shares that hold parts of it
  int slot_rows;    // rows of a slot
  CutPlan plan;
  int G, Hq;
  __nv_bfloat16* O;
  float* LSE;
};

// The item that the cut before share c divides; false when there is none or an earlier cut joins it.
template <typename P>
__device__ __forceinline__ bool join_item(JoinItem& it, const P& prm, int c, int slot_rows) {
  it.plan = prm.plan[c];
  if (it.plan.tile == 0) return false;
  const Cut cut = cut_of(it.plan.per, c, it.plan.tile, it.plan.n);
  it.part_o = prm.part_o;
  it.part_ml = prm.part_ml;
  it.first = cut.first;
  it.last = cut.last;
  it.slot_rows = slot_rows;
  it.G = prm.G;
  it.Hq = prm.Hq;
  it.O = prm.O;
  it.LSE = prm.LSE;
  return cut.first == c - 1;
}

// One warp: the weighted sum of parts `begin`, begin + stride, ... of row lr, D / 32 columns a lane; m and l over
// all parts.
template <int D>
__device__ __forceinline__ void join_row(const JoinItem& it, int lr, int begin, int stride, float (&o)[D / 32], float& m,
                                         float& l) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31, n = it.last - it.first + 1;
  auto at = [&](int k) { return static_cast<size_t>(decode_slot(it.first + k, k)) * it.slot_rows + lr; };
  m = -INFINITY;
  for (int k = lane; k < n; k += 32) m = fmaxf(m, it.part_ml[at(k)].x);
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  l = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.0f;
  for (int k0 = 0; k0 < n; k0 += 32) {
    const float2 ml = k0 + lane < n ? it.part_ml[at(k0 + lane)] : make_float2(-INFINITY, 0.0f);
    // l = 0: the row sees no key of the part, whose O may not be written
    const Exp2Pair by(ml.x - (m == -INFINITY ? 0.0f : m));
    const float w = ml.y == 0.0f ? 0.0f : by.times(1.0f);
    l += by.times(ml.y);
    const int here = min(32, n - k0);
#pragma unroll 8
    for (int k = begin; k < here; k += stride) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      float v[C];
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = 0.0f;
      if (wk > 0.0f) {
        const float* p = it.part_o + at(k0 + k) * D + lane * C;
        if constexpr (C == 4) {
          const float4 x = *reinterpret_cast<const float4*>(p);
          v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(p);
          v[0] = x.x, v[1] = x.y;
        }
      }
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = fmaf(wk, v[c], o[c]);
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
}

template <int D>
__device__ __forceinline__ void join_store(const JoinItem& it, int lr, const float (&o)[D / 32], float m, float l) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31, row = it.plan.row0 + lr;
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  const size_t at = static_cast<size_t>(it.plan.token0 + row / it.G) * it.Hq + it.plan.h * it.G + row % it.G;
  uint32_t* to = reinterpret_cast<uint32_t*>(it.O + at * D + lane * C);
  if constexpr (C == 4) {
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  } else {
    *to = pack_bf16x2(o[0] * inv, o[1] * inv);
  }
  if (lane == 0) it.LSE[at] = l != 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// Blocks 0 .. (n_dec - 1) * dec.rows - 1: the cuts of decode_kernel's n_dec shares, a block a row; after them
// kJoinPreSplit blocks for each cut of prefill_kernel's.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const DecodeParams dec, const PrefillParams pre, int n_dec) {
  constexpr int C = D / 32;
  __shared__ float sums[3][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int dec_blocks = (n_dec - 1) * dec.rows;
  JoinItem it;
  float o[C], m, l;
  grid_dependency_wait();  // the parts and where they lie are written
  if (static_cast<int>(blockIdx.x) < dec_blocks) {
    const int lr = blockIdx.x % dec.rows;
    if (!join_item(it, dec, blockIdx.x / dec.rows + 1, dec.rows) || lr >= it.plan.rows) return;
    join_row<D>(it, lr, warp, 4, o, m, l);
    if (warp > 0)
#pragma unroll
      for (int i = 0; i < C; ++i) sums[warp - 1][lane * C + i] = o[i];
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] += sums[0][lane * C + i] + sums[1][lane * C + i] + sums[2][lane * C + i];
    join_store<D>(it, lr, o, m, l);
    return;
  }
  const int i = blockIdx.x - dec_blocks, part = i % kJoinPreSplit;
  if (!join_item(it, pre, i / kJoinPreSplit + 1, kPreRows)) return;
#pragma unroll
  for (int k = 0; k < kJoinPreRows / 4; ++k) {
    const int lr = part * kJoinPreRows + k * 4 + warp;
    if (lr >= it.plan.rows) return;
    join_row<D>(it, lr, 0, 1, o, m, l);
    join_store<D>(it, lr, o, m, l);
  }
}

}  // namespace fa

// fa_append.cuh -- new keys and values into the paged cache, keys and queries rotated on the way.
//
//   rot(x, p): for each pair (i, j) of the first rot columns, x_i' = x_i cos - x_j sin, x_j' = x_j cos +
//   x_i sin with the position's table entries; (i, j) = (i, i + rot/2), or (2i, 2i+1) when interleaved.
//   bf16 cache: one rounding of the rotated value.  e4m3 cache: one scale for each page and head,
//   scale' = max(scale of the page's earlier tokens, what the new values need), new codes e4m3(x / scale'),
//   and, when the scale grew, the earlier codes brought to it: e4m3(code * scale / scale').
//
// A block owns one page of one sequence and one key/value head, since a page's scale is a maximum over all its
// new tokens and growing it touches all its earlier ones; the G query heads of that head ride along and
// reuse the angles.  A thread holds 8 columns (16 bytes) of ITEMS tokens; a pair's other half is in
// another lane of the same warp (a row is D / 8 consecutive lanes) and comes by shuffle, so every input is
// read once and Q may be rotated in place.  What a block waits for is two dependent loads, the batch's
// indices and then everything else at once (keys, values, angles, four query heads and the page number);
// the rotated keys are not kept but rotated again after the maximum, which keeps four blocks on an SM.
// One or two new tokens a sequence (a decode batch) take blocks of one warp.  Bound by HBM for prompts
// (each row is read once and written once), by the two loads' latency for single tokens.
#pragma once

#include "fa_paged.cuh"

namespace fa {

struct AppendParams {
  PagedBatch b;
  const __nv_bfloat16 *K, *V, *Q;  // token-major rows [T, heads, D], `ld*` elements apart
  __nv_bfloat16* Qo;
  long long ldk, ldv, ldq, ldqo;
  const float *cosp, *sinp;  // [n_pos, rot / 2]
  int rot, interleaved, n_pos;
  void *Kc, *Vc;
  float *Ks, *Vs;
  int G;          // query heads per key/value head (0: no queries)
  int max_touched;  // pages a sequence's new rows can touch
};

// Rotated fp32 values of this lane's 8 columns.  All 32 lanes call it together (shuffles).
template <int D>
__device__ __forceinline__ void rotate8(const uint4& raw, float (&x)[8], const float (&c)[8], const float (&s)[8],
                                        int vec, int rot, int interleaved) {
  constexpr int VPR = D / 8;
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  if (rot == 0) return;
  if (interleaved) {
    if (vec * 8 < rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * c[i] - b * s[i];
        x[2 * i + 1] = b * c[i] + a * s[i];
      }
    }
    return;
  }
  const int half = rot / 16;  // lanes of half the rotated columns
  const int other = vec < half ? vec + half : vec < 2 * half ? vec - half : vec;
  const float sign = vec < half ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t o = __shfl_sync(0xffffffffu, w[i], other, VPR);
    if (vec < 2 * half) {
      x[2 * i] = x[2 * i] * c[2 * i] + sign * __uint_as_float(o << 16) * s[2 * i];
      x[2 * i + 1] = x[2 * i + 1] * c[2 * i + 1] + sign * __uint_as_float(o & 0xFFFF0000u) * s[2 * i + 1];
    }
  }
}

// This lane's table entries of position p (8 angles, 4 when interleaved).
__device__ __forceinline__ void load_angles(const AppendParams& prm, int p, int vec, float (&c)[8], float (&s)[8]) {
  const int half = prm.rot / 2;
  const int first = prm.interleaved ? vec * 4 : (vec * 8 < half ? vec * 8 : vec * 8 - half);
  const float4* cp = reinterpret_cast<const float4*>(prm.cosp + static_cast<size_t>(p) * half + first);
  const float4* sp = reinterpret_cast<const float4*>(prm.sinp + static_cast<size_t>(p) * half + first);
  const float4 c0 = __ldg(cp), s0 = __ldg(sp);
  c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w;
  s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w;
  if (!prm.interleaved) {
    const float4 c1 = __ldg(cp + 1), s1 = __ldg(sp + 1);
    c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
  }
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float inv) {
  return make_uint2(e4m3x2(x[0] * inv, x[1] * inv) | (e4m3x2(x[2] * inv, x[3] * inv) << 16),
                    e4m3x2(x[4] * inv, x[5] * inv) | (e4m3x2(x[6] * inv, x[7] * inv) << 16));
}
// The largest finite magnitude: an infinity saturates its own code and leaves the page's scale to the others.
__device__ __forceinline__ float amax8(const float (&x)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    m = fmaxf(m, a < INFINITY ? a : 0.0f);
  }
  return m;
}

// Earlier codes of a page and head, `n` bytes (a multiple of 16), times ratio (below 1).
__device__ __forceinline__ void rescale_codes(uint8_t* codes, int n, float ratio, int t, int threads) {
#pragma unroll 4
  for (int i = t * 16; i < n; i += threads * 16) {
    uint4 v = *reinterpret_cast<uint4*>(codes + i);
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t lo, hi;
      halves_of_e4m3(w[j], lo, hi);
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      w[j] = e4m3x2(a.x * ratio, a.y * ratio) | (e4m3x2(b.x * ratio, b.y * ratio) << 16);
    }
    *reinterpret_cast<uint4*>(codes + i) = v;
  }
}

constexpr int kAppendThreads = 256;
constexpr int kAppendQ = 4;  // query heads whose rows are loaded together

template <int D, bool FP8, int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS, THREADS == kAppendThreads && ITEMS == 1 ? 4 : 1)
    append_kernel(const AppendParams prm) {
  constexpr int VPR = D / 8;
  constexpr int ROWS = THREADS / VPR;  // tokens of a page the block takes at a time
  const PagedBatch& pb = prm.b;
  const int h = blockIdx.x % pb.Hkv;
  const int unit = blockIdx.x / pb.Hkv;
  const int b = unit / prm.max_touched, ordinal = unit % prm.max_touched;
  const SeqInfo s = load_seq(pb, b);
  const int start = s.len - s.rows;  // position of the first new row
  if (s.rows == 0) return;
  if (start < 0) {
    record(pb.status, kBadLength);
    return;
  }
  const int block = (start >> pb.page_shift) + ordinal;
  const int base = block << pb.page_shift;  // position of the page's first slot
  if (base >= s.len) return;
  const int page = pb.table[static_cast<size_t>(b) * pb.max_pages + block];  // checked below, with the loads under way
  const int first = max(start, base) - base, last = min(s.len, base + (1 << pb.page_shift)) - base;  // slots [first, last)
  const int vec = threadIdx.x % VPR, slot0 = first + threadIdx.x / VPR;
  const size_t row0 = static_cast<size_t>(s.row0 + base + slot0 - start);  // this thread's first token row

  uint4 kraw[ITEMS], vraw[ITEMS], qraw[kAppendQ];
  auto live = [&](int i) { return slot0 + i * ROWS < last && (prm.rot == 0 || base + slot0 + i * ROWS < prm.n_pos); };
  auto load_q = [&](int i, int g0) {
#pragma unroll
    for (int g = 0; g < kAppendQ; ++g)
      qraw[g] = live(i) && g0 + g < prm.G
                    ? *reinterpret_cast<const uint4*>(prm.Q + (row0 + i * ROWS) * prm.ldq + (h * prm.G + g0 + g) * D + vec * 8)
                    : make_uint4(0u, 0u, 0u, 0u);
  };
  auto angles = [&](int i, float (&c)[8], float (&sn)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = sn[j] = 0.0f;
    if (live(i) && vec * 8 < prm.rot) load_angles(prm, base + slot0 + i * ROWS, vec, c, sn);
  };
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    kraw[i] = vraw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (live(i)) {
      kraw[i] = *reinterpret_cast<const uint4*>(prm.K + (row0 + i * ROWS) * prm.ldk + h * D + vec * 8);
      vraw[i] = *reinterpret_cast<const uint4*>(prm.V + (row0 + i * ROWS) * prm.ldv + h * D + vec * 8);
    }
    if (prm.rot > 0 && slot0 + i * ROWS < last && base + slot0 + i * ROWS >= prm.n_pos) record(pb.status, kBadPosition);
  }
  float c[8], sn[8];
  angles(0, c, sn);
  load_q(0, 0);
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(pb.num_pages)) {
    record(pb.status, kBadPage);
    return;
  }
  const size_t head_at = (static_cast<size_t>(page) * pb.Hkv + h) << pb.page_shift;  // row of slot 0 in the cache
  float ak = 0.0f, av = 0.0f;
  float ks_old = 0.0f, vs_old = 0.0f;
  if (FP8 && first > 0) {
    ks_old = prm.Ks[static_cast<size_t>(page) * pb.Hkv + h];
    vs_old = prm.Vs[static_cast<size_t>(page) * pb.Hkv + h];
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if (i > 0) {
      angles(i, c, sn);
      load_q(i, 0);
    }
    float x[8];
    rotate8<D>(kraw[i], x, c, sn, vec, prm.rot, prm.interleaved);
    if constexpr (FP8) {
      ak = amax8(x, ak);
      float vx[8];
      rotate8<D>(vraw[i], vx, c, sn, vec, 0, 0);
      av = amax8(vx, av);
    } else if (live(i)) {
      const size_t at = (head_at + slot0 + i * ROWS) * D + vec * 8;
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(prm.Kc) + at) = pack8_bf16(x);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(prm.Vc) + at) = vraw[i];
    }
    for (int g0 = 0; g0 < prm.G; g0 += kAppendQ) {
      if (g0 > 0) load_q(i, g0);
#pragma unroll
      for (int g = 0; g < kAppendQ; ++g) {
        rotate8<D>(qraw[g], x, c, sn, vec, prm.rot, prm.interleaved);
        if (live(i) && g0 + g < prm.G)
          *reinterpret_cast<uint4*>(prm.Qo + (row0 + i * ROWS) * prm.ldqo + (h * prm.G + g0 + g) * D + vec * 8) =
              pack8_bf16(x);
      }
    }
  }
  if constexpr (FP8) {
    __shared__ float red[2][THREADS / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ak = fmaxf(ak, __shfl_xor_sync(0xffffffffu, ak, o));
      av = fmaxf(av, __shfl_xor_sync(0xffffffffu, av, o));
    }
    if (THREADS > 32) {
      if ((threadIdx.x & 31) == 0) {
        red[0][threadIdx.x >> 5] = ak;
        red[1][threadIdx.x >> 5] = av;
      }
      __syncthreads();  // also: every thread has read the old scales
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) {
        ak = fmaxf(ak, red[0][w]);
        av = fmaxf(av, red[1][w]);
      }
    } else {
      __syncwarp();
    }
    const float ks = fmaxf(ks_old, needed_scale(ak)), vs = fmaxf(vs_old, needed_scale(av));
    uint8_t* kc = static_cast<uint8_t*>(prm.Kc) + head_at * D;
    uint8_t* vc = static_cast<uint8_t*>(prm.Vc) + head_at * D;
    if (threadIdx.x == 0) {
      prm.Ks[static_cast<size_t>(page) * pb.Hkv + h] = ks;
      prm.Vs[static_cast<size_t>(page) * pb.Hkv + h] = vs;
    }
    if (first > 0 && ks > ks_old) rescale_codes(kc, first * D, ks_old / ks, threadIdx.x, THREADS);
    if (first > 0 && vs > vs_old) rescale_codes(vc, first * D, vs_old / vs, threadIdx.x, THREADS);
    const float ki = 1.0f / ks, vi = 1.0f / vs;  // exact for the powers of two written here
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (ITEMS > 1) angles(i, c, sn);
      float x[8], vx[8];
      rotate8<D>(kraw[i], x, c, sn, vec, prm.rot, prm.interleaved);
      rotate8<D>(vraw[i], vx, c, sn, vec, 0, 0);
      if (!live(i)) continue;
      const size_t at = static_cast<size_t>(slot0 + i * ROWS) * D + vec * 8;
      *reinterpret_cast<uint2*>(kc + at) = pack8_e4m3(x, ki);
      *reinterpret_cast<uint2*>(vc + at) = pack8_e4m3(vx, vi);
    }
  }
}

}  // namespace fa

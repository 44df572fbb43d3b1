// fa_append.cuh -- new keys and values into the paged cache, keys and queries rotated on the way.
//
//   rot(x, p): for each pair (i, j) of the first rot columns, x_i' = x_i cos - x_j sin, x_j' = x_j cos +
//   x_i sin with the position's table entries; (i, j) = (i, i + rot/2), or (2i, 2i+1) when interleaved.
//   bf16 cache: one rounding of the rotated value.  e4m3 cache: one scale for each page and head,
//   scale' = max(scale of the page's earlier tokens, what the new values need), new codes e4m3(x / scale'),
//   and, when the scale grew, the earlier codes brought to it: e4m3(code * scale / scale').
//
// A page's scale is a maximum over all its new tokens, and growing it touches all its earlier ones, so the unit
// is one page of one sequence and one key/value head; the G query heads of that head ride along and reuse
// the angles.  A block takes 16 tokens (D = 128; 32 at D = 64), a thread 8 columns (16 bytes) of one; the blocks
// of a longer page are a cluster and exchange their maxima through shared memory (one block holding a whole
// page had 148 to 245 registers a thread and reached 2.5 TB/s).  A pair's other half is in another lane of the
// same warp (a row is D / 8 consecutive lanes) and comes by shuffle, so every input is read once and Q may be
// rotated in place.  What a block waits for is two dependent loads, the batch's indices and then everything
// else at once (keys, values, angles, four query heads and the page number); 64 registers keep four blocks on an
// SM, for 16 (bf16) or 36 to 44 bytes (e4m3) of spills a thread.  Batches of no more than two new tokens a sequence
// (four at D = 64) take blocks of one warp.  Bound by HBM for prompts (each row is read once and written once), in
// an e4m3 cache by the loads' latency before it (28.7 warps an SM wait for them most of the time; 2.5 of 4
// instructions a cycle are issued), and by that latency for single tokens.  22 K tokens of 32 + 2 x 8 heads into
// pages of 16: bf16 95 us (5.9 of 6.56 TB/s measured copy), e4m3 110 to 115 us (4.5 to 4.7 TB/s); one token 3.2 us.
// The grid has max_q tokens' pages for every sequence: a long prompt among many single tokens launches as many empty
// blocks.
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
  int subs;         // blocks of a page
};

// Sequence b's new rows: none where their positions cannot be trusted (a length below 0, beyond the block table or
// below the rows), since live tokens of this sequence, or of one that shares its full pages, lie at any others.
FA_HD SeqInfo append_seq(const PagedBatch& p, int b) {
  SeqInfo s = load_seq(p, b);
  if (s.rows > 0 && (s.cut || s.len < s.rows)) {
    s.rows = 0;
    record(p.status, kBadLength);
  }
  return s;
}

// This lane's 8 columns as fp32 pairs.
struct Eight {
  float2 v[4];
};
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ Eight unpack8(const uint4& raw) {
  return Eight{{unpack2(raw.x), unpack2(raw.y), unpack2(raw.z), unpack2(raw.w)}};
}

// This lane's angles of one position: cosines and sines of its 8 columns (of its 4 pairs when interleaved),
// the sines with the sign of the pair's first or second half.
struct Angles {
  float2 c[4], s[4];
};
__device__ __forceinline__ Angles load_angles(const AppendParams& prm, int p, int vec) {
  const int half = prm.rot / 2;
  const bool first = vec * 8 < half;
  const size_t at = static_cast<size_t>(p) * half + (prm.interleaved ? vec * 4 : first ? vec * 8 : vec * 8 - half);
  const float4* cp = reinterpret_cast<const float4*>(prm.cosp + at);
  const float4* sp = reinterpret_cast<const float4*>(prm.sinp + at);
  const float4 c0 = __ldg(cp), s0 = __ldg(sp);
  Angles a;
  if (prm.interleaved) {
    a.c[0] = make_float2(c0.x, c0.x), a.c[1] = make_float2(c0.y, c0.y);
    a.c[2] = make_float2(c0.z, c0.z), a.c[3] = make_float2(c0.w, c0.w);
    a.s[0] = make_float2(-s0.x, s0.x), a.s[1] = make_float2(-s0.y, s0.y);
    a.s[2] = make_float2(-s0.z, s0.z), a.s[3] = make_float2(-s0.w, s0.w);
    return a;
  }
  const float4 c1 = __ldg(cp + 1), s1 = __ldg(sp + 1);
  const float g = first ? -1.0f : 1.0f;
  a.c[0] = make_float2(c0.x, c0.y), a.c[1] = make_float2(c0.z, c0.w);
  a.c[2] = make_float2(c1.x, c1.y), a.c[3] = make_float2(c1.z, c1.w);
  a.s[0] = make_float2(g * s0.x, g * s0.y), a.s[1] = make_float2(g * s0.z, g * s0.w);
  a.s[2] = make_float2(g * s1.x, g * s1.y), a.s[3] = make_float2(g * s1.z, g * s1.w);
  return a;
}

// Rotated values of this lane's 8 columns: x cos + (its pair's other half) sin.  All 32 lanes call it together;
// `other` is the lane (of the row's VPR) with the other halves, `turns` whether this lane's columns are rotated.
template <int VPR>
__device__ __forceinline__ Eight rotate8(const uint4& raw, const Angles& a, int other, bool turns, bool interleaved) {
  Eight x = unpack8(raw);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 o;
    if (interleaved) {
      o = make_float2(x.v[i].y, x.v[i].x);
    } else {
      o = unpack2(__shfl_sync(0xffffffffu, w[i], other, VPR));
    }
    if (turns) x.v[i] = __ffma2_rn(o, a.s[i], __fmul2_rn(x.v[i], a.c[i]));
  }
  return x;
}

__device__ __forceinline__ uint4 pack8_bf16(const Eight& x) {
  return make_uint4(pack_bf16x2(x.v[0].x, x.v[0].y), pack_bf16x2(x.v[1].x, x.v[1].y),
                    pack_bf16x2(x.v[2].x, x.v[2].y), pack_bf16x2(x.v[3].x, x.v[3].y));
}
// x times the scale's reciprocal: the quotient itself for a power of two, which every scale is that this kernel wrote;
// by another (a caller's, kept while it is large enough) a value next to a tie may go to the other neighbour.
__device__ __forceinline__ uint2 pack8_e4m3(const Eight& x, float inv) {
  const float2 f = make_float2(inv, inv);
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = __fmul2_rn(x.v[i], f);
    h[i] = e4m3x2(y.x, y.y);
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}
// The largest finite magnitude: an infinity saturates its own code and leaves the page's scale to the others.
// (NaN never wins a maximum; an infinity shows in the result, and only then is each value looked at.)
__device__ __forceinline__ float amax8(const Eight& x, float m) {
  float a = fmaxf(fabsf(x.v[0].x), fabsf(x.v[0].y));
#pragma unroll
  for (int i = 1; i < 4; ++i) a = fmax3(a, fabsf(x.v[i].x), fabsf(x.v[i].y));
  if (!(a < INFINITY)) {
    a = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (fabsf(x.v[i].x) < INFINITY) a = fmaxf(a, fabsf(x.v[i].x));
      if (fabsf(x.v[i].y) < INFINITY) a = fmaxf(a, fabsf(x.v[i].y));
    }
  }
  return fmaxf(m, a);
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

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

constexpr int kAppendThreads = 256;
constexpr int kAppendQ = 4;  // query heads whose rows are loaded together

// CL: blocks of a cluster, which are a page's (e4m3; a bf16 page's blocks need not know of each other).
template <int D, bool FP8, int THREADS, int CL>
__global__ void __launch_bounds__(THREADS, THREADS == kAppendThreads ? 4 : 1) append_kernel(const AppendParams prm) {
  constexpr int VPR = D / 8;
  constexpr int ROWS = THREADS / VPR;  // tokens of the block
  const PagedBatch& pb = prm.b;
  if (CL > 1) cluster_arrive();  // this block runs: the others may write to its shared memory
  // a cluster's blocks are neighbours; otherwise the heads are, whose rows of a token lie side by side
  unsigned rest = blockIdx.x;
  const int fast = FP8 ? prm.subs : pb.Hkv, slow = FP8 ? pb.Hkv : prm.subs;
  unsigned q = rest / fast;
  const int i0 = rest - q * fast;
  rest = q;
  q = rest / slow;
  const int i1 = rest - q * slow;
  rest = q;
  const int h = FP8 ? i1 : i0, blk = FP8 ? i0 : i1;
  const int b = rest / static_cast<unsigned>(prm.max_touched), ordinal = rest - b * prm.max_touched;
  const SeqInfo s = append_seq(pb, b);
  const int start = s.len - s.rows;  // position of the first new row
  if (s.rows == 0) return;
  const int block = (start >> pb.page_shift) + ordinal;
  const int base = block << pb.page_shift;  // position of the page's first slot
  if (base >= s.len) return;
  const int page = pb.table[static_cast<size_t>(b) * pb.max_pages + block];  // checked below, with the loads under way
  const int first = max(start, base) - base, last = min(s.len, base + (1 << pb.page_shift)) - base;  // slots [first, last)
  const int vec = threadIdx.x % VPR, slot = first + blk * ROWS + threadIdx.x / VPR;
  const size_t row0 = static_cast<size_t>(s.row0 + base + slot - start);  // this thread's token row
  // the lane with the other halves of this lane's pairs, and whether its columns turn at all
  const int half = prm.rot / 16;
  const bool turns = vec * 8 < prm.rot, inter = prm.interleaved;
  const int other = vec < half ? vec + half : vec < 2 * half ? vec - half : vec;
  const __nv_bfloat16* kp = prm.K + row0 * prm.ldk + h * D + vec * 8;
  const __nv_bfloat16* vp = prm.V + row0 * prm.ldv + h * D + vec * 8;
  const __nv_bfloat16* qp = prm.Q + row0 * prm.ldq + h * prm.G * D + vec * 8;
  __nv_bfloat16* qop = prm.Qo + row0 * prm.ldqo + h * prm.G * D + vec * 8;
  const int limit = prm.rot > 0 ? min(last, prm.n_pos - base) : last;  // slots behind it are not written
  const bool live = slot < limit;

  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4 kraw = live ? *reinterpret_cast<const uint4*>(kp) : zero;
  const uint4 vraw = live ? *reinterpret_cast<const uint4*>(vp) : zero;
  uint4 qraw[kAppendQ];
  auto load_q = [&](int g0) {
#pragma unroll
    for (int g = 0; g < kAppendQ; ++g)
      qraw[g] = live && g0 + g < prm.G ? *reinterpret_cast<const uint4*>(qp + (g0 + g) * D) : zero;
  };
  Angles ang;
#pragma unroll
  for (int j = 0; j < 4; ++j) ang.c[j] = ang.s[j] = make_float2(0.0f, 0.0f);
  if (live && turns) ang = load_angles(prm, base + slot, vec);
  load_q(0);
  if (limit < last && threadIdx.x == 0) record(pb.status, kBadPosition);
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(pb.num_pages)) {
    record(pb.status, kBadPage);
    return;
  }
  const size_t head_at = (static_cast<size_t>(page) * pb.Hkv + h) << pb.page_shift;  // row of slot 0 in the cache
  float ks_old = 0.0f, vs_old = 0.0f;
  if (FP8 && first > 0) {
    ks_old = prm.Ks[static_cast<size_t>(page) * pb.Hkv + h];
    vs_old = prm.Vs[static_cast<size_t>(page) * pb.Hkv + h];
  }
  const Eight kx = rotate8<VPR>(kraw, ang, other, turns, inter);
  if (!FP8 && live) {
    const size_t at = (head_at + slot) * D + vec * 8;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(prm.Kc) + at) = pack8_bf16(kx);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(prm.Vc) + at) = vraw;
  }
  auto queries = [&] {
    for (int g0 = 0; g0 < prm.G; g0 += kAppendQ) {
      if (g0 > 0) load_q(g0);
#pragma unroll
      for (int g = 0; g < kAppendQ; ++g) {
        const uint4 y = pack8_bf16(rotate8<VPR>(qraw[g], ang, other, turns, inter));
        if (live && g0 + g < prm.G) *reinterpret_cast<uint4*>(qop + (g0 + g) * D) = y;
      }
    }
  };
  if (!FP8) queries();
  if constexpr (FP8) {
    float ak = amax8(kx, 0.0f), av = amax8(unpack8(vraw), 0.0f);
    __shared__ float2 red[THREADS / 32], all[CL];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ak = fmaxf(ak, __shfl_xor_sync(0xffffffffu, ak, o));
      av = fmaxf(av, __shfl_xor_sync(0xffffffffu, av, o));
    }
    if (THREADS > 32) {
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(ak, av);
      __syncthreads();  // also: every thread has read the old scales
      if (CL == 1 || threadIdx.x < CL) {
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
          ak = fmaxf(ak, red[w].x);
          av = fmaxf(av, red[w].y);
        }
      }
      if constexpr (CL > 1) {
        // thread r leaves this block's maxima in block r's shared memory (once all blocks run); after the barrier
        // all are local.  The queries are turned while it completes.
        cluster_wait();
        if (threadIdx.x < CL)
          asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(peer_smem(smem_u32(&all[blk]), threadIdx.x)),
                       "f"(ak), "f"(av)
                       : "memory");
        cluster_arrive();
        queries();
        cluster_wait();
        ak = av = 0.0f;
#pragma unroll
        for (int w = 0; w < CL; ++w) {
          ak = fmaxf(ak, all[w].x);
          av = fmaxf(av, all[w].y);
        }
      }
    } else {
      __syncwarp();
    }
    if (CL == 1) queries();
    const float ks = fmaxf(ks_old, needed_scale(ak)), vs = fmaxf(vs_old, needed_scale(av));
    uint8_t* kc = static_cast<uint8_t*>(prm.Kc) + head_at * D;
    uint8_t* vc = static_cast<uint8_t*>(prm.Vc) + head_at * D;
    const int t = blk * THREADS + threadIdx.x;
    if (t == 0) {
      prm.Ks[static_cast<size_t>(page) * pb.Hkv + h] = ks;
      prm.Vs[static_cast<size_t>(page) * pb.Hkv + h] = vs;
    }
    if (first > 0 && ks > ks_old) rescale_codes(kc, first * D, ks_old / ks, t, THREADS * CL);
    if (first > 0 && vs > vs_old) rescale_codes(vc, first * D, vs_old / vs, t, THREADS * CL);
    if (live) {
      const size_t at = static_cast<size_t>(slot) * D + vec * 8;
      *reinterpret_cast<uint2*>(kc + at) = pack8_e4m3(kx, 1.0f / ks);
      *reinterpret_cast<uint2*>(vc + at) = pack8_e4m3(unpack8(vraw), 1.0f / vs);
    }
  }
}

}  // namespace fa

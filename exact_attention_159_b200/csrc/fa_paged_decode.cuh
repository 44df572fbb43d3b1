// fa_paged_decode.cuh -- attention of few query rows (single tokens, a few drafted tokens) over the paged
// cache: one pass over the keys and values with a running maximum and sum, the long axis split evenly
// over the GPU and joined by a second small kernel.
//
// With few rows the work is reading the cache once, so everything here serves that: TMA brings 64-key
// tiles of a page list into a ring of shared-memory stages (96 KB of loads in flight per CTA, two CTAs an
// SM), and the arithmetic runs on mma.sync m16n8k16, whose 16 rows fit the query heads that share a
// key/value head, where a tcgen05 tile would be 128 rows of padding.
//
// Rows: the R = rows * G (token, query head) pairs that read one key/value head, in blocks of 16.  One
// (sequence, row block, key/value head) is an item of ceil(len / 64) tiles; the items' tiles laid end to
// end are cut into equal runs, one per CTA, so a batch of ragged lengths loads every SM alike.  An item
// that a cut divides leaves its unnormalised sums in the workspace, at most two a CTA, for the join.
//
// Each of the four consumer warps takes 16 keys of every tile and keeps its own maximum, sum and output
// accumulators; they meet once, at the item's end.
//   S = Q K^T:  A = Q (16 rows, registers for the whole item), B = 16 keys
//   O += P V:   A = P straight from S's accumulators, B = V
// e4m3 pages: codes become halves exactly (one conversion for two codes) and the scales stay outside the
// products: K's multiplies the scores, V's joins the exponent, w = 2^(s + log2 vs - m), so w <= 1 whatever
// the scales, O = sum w * code, and the softmax's sum is sum w / vs.  Q is brought to [-1, 1] by a power of
// two per row before it becomes halves.  P is rounded to half (11 bits; bf16 for a bf16 cache, as the
// other forwards round it); m, the sums and O are fp32.
// To feed B from bytes without a transposing load, columns are permuted: a lane's 16-byte chunk of a key
// row holds its k indices of four MMAs, and a lane's 16-byte chunk of a value row holds its column n of
// 16 output tiles.  Keys 0..7 of a tile's octet go to n = 0,2,4,6,1,3,5,7, which with TMA's 128-byte
// swizzle puts the eight lanes of a load phase on eight different chunks.
#pragma once

#include "exp2_poly.cuh"
#include "fa_paged.cuh"

namespace fa {

constexpr int kSiteDecode = 0xD00;
constexpr int kDecTile = 64;       // keys of a tile
constexpr int kDecRows = 16;       // query rows of an item
constexpr int kDecCtas = 2 * 148;  // two on each SM
constexpr int kDecThreads = 160;   // four consumer warps, one producer warp
constexpr int kDecStageBytes = 98304;
constexpr int kDecMinTiles = 2;    // a CTA's share is at least this many tiles
constexpr float kScaleFloor = 7.8886090522101181e-31f;  // 2^-100: smaller value scales count as this

struct DecodeParams {
  PagedBatch b;
  const __nv_bfloat16* Q;  // [T, Hq, D], ldq elements between tokens
  long long ldq;
  __nv_bfloat16* O;   // [T, Hq, D]
  float* LSE;         // [T, Hq]
  const float *Ks, *Vs;
  float* part_o;      // [2 * n_cta][16][D] unnormalised sums
  float2* part_ml;    // [2 * n_cta][16] (m in log2 units, l)
  int G, Hq;
  int max_rows;       // sequences of more rows * G are another kernel's
  int causal, whole;  // whole: shares are whole items (short caches), nothing is joined
  float scale_log2;
};

template <int D, bool FP8>
struct DecodeLayout {
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  static constexpr int kHalf = kDecTile * 128;  // bytes of a 128-byte-wide column block of a tile
  static constexpr int kTileBytes = kDecTile * kRowBytes;
  static constexpr int kStages = kDecStageBytes / (2 * kTileBytes) < 6 ? kDecStageBytes / (2 * kTileBytes) : 6;
  static constexpr int kV = kStages * kTileBytes;
  static constexpr int kMerge = 2 * kV;                      // two warps' accumulators
  static constexpr int kMergeWarp = 16 * D * 4 + 512;        // float4 per lane and column tile, then (m, l) x 2
  static constexpr int kMeta = kMerge + 2 * kMergeWarp;      // [stage][4 boxes] (K scale, V scale)
  static constexpr int kBar = kMeta + kStages * 4 * 8;
  static constexpr int kMisc = kBar + 2 * kStages * 8;
  static constexpr int kBytes = kMisc + 96;
};

// ------------------------------------------------------------------------------------- the plan
struct DecodeSeq {
  SeqInfo s;
  int tiles, items;  // items 0: no rows, or too many for this kernel
};
FA_HD DecodeSeq decode_seq(const DecodeParams& p, int b) {
  DecodeSeq d;
  d.s = load_seq(p.b, b);
  const long long rows = static_cast<long long>(d.s.rows) * p.G;
  const bool mine = rows > 0 && rows <= p.max_rows;
  d.tiles = max(1, (d.s.len + kDecTile - 1) / kDecTile);  // a sequence of no keys still gets its rows written
  d.items = mine ? static_cast<int>((rows + kDecRows - 1) / kDecRows) * p.b.Hkv : 0;
  return d;
}
FA_HD long long decode_units(const DecodeParams& p, const DecodeSeq& d) {
  return static_cast<long long>(d.items) * (p.whole ? 1 : d.tiles);
}
FA_HD long long decode_per(const DecodeParams& p, long long total, int n_cta) {
  const long long per = (total + n_cta - 1) / n_cta;
  return !p.whole && per < kDecMinTiles ? kDecMinTiles : per;
}

struct DecodeShare {
  long long total, per;
  int b;          // sequence holding the wanted unit (B when there is none)
  long long off;  // the unit within that sequence
};
// The total of all units, a CTA's share of them, and where unit index * share lies.  Each thread sums a run
// of sequences; the one whose run holds the unit walks it.  All threads of the block call it.
template <int THREADS>
__device__ __forceinline__ DecodeShare decode_share(const DecodeParams& p, int index, int n_cta, long long* scratch) {
  constexpr int W = THREADS / 32;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int run = (p.b.B + THREADS - 1) / THREADS;
  const int b0 = min(t * run, p.b.B), b1 = min(b0 + run, p.b.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += decode_units(p, decode_seq(p, b));
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) scratch[warp] = inc;
  if (t == 0) scratch[W] = p.b.B, scratch[W + 1] = 0;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  DecodeShare r;
  r.total = total;
  r.per = decode_per(p, total, n_cta);
  const long long want = r.per * index;
  const long long lo = before + inc - mine;
  if (want >= lo && want < lo + mine) {
    long long at = lo;
    for (int b = b0; b < b1; ++b) {
      const long long u = decode_units(p, decode_seq(p, b));
      if (want < at + u) {
        scratch[W] = b;
        scratch[W + 1] = want - at;
        break;
      }
      at += u;
    }
  }
  __syncthreads();
  r.b = static_cast<int>(scratch[W]);
  r.off = scratch[W + 1];
  return r;
}

// Where CTA `cta` leaves the part of an item that starts at tile t0 of it: its share has at most one part
// whose item began in an earlier share and one whose item goes on in the next.
FA_HD int decode_slot(int cta, int t0) { return 2 * cta + (t0 == 0 ? 1 : 0); }

// The item that the cut before share c divides: `first`..`last` are the shares it lies in.  first < c - 1
// when an earlier cut divides it too, last < c when the cut falls between two items.
struct DecodeCut {
  int item, first, last;
};
FA_HD DecodeCut decode_cut(long long per, int c, long long off, int tiles) {
  DecodeCut r;
  r.item = static_cast<int>(off / tiles);
  const long long tile = off % tiles, begin = per * c - tile;
  r.first = static_cast<int>(begin / per);
  r.last = tile == 0 ? c - 1 : static_cast<int>((begin + tiles - 1) / per);
  return r;
}

// Walks a CTA's share: one segment (an item's tiles [t0, t1)) after another.
struct DecodeWalk {
  long long left;
  int b, item, t0, t1;
  DecodeSeq d;
  bool whole;
  FA_HD void start(const DecodeParams& p, const DecodeShare& s, int index) {
    left = min(s.per, s.total - s.per * index);
    b = s.b;
    d = decode_seq(p, b);
    if (p.whole) {
      item = static_cast<int>(s.off);
      t0 = 0;
    } else {
      item = static_cast<int>(s.off / d.tiles);
      t0 = static_cast<int>(s.off % d.tiles);
    }
    cut(p);
  }
  FA_HD void cut(const DecodeParams& p) {
    t1 = p.whole ? d.tiles : static_cast<int>(min(static_cast<long long>(d.tiles), t0 + left));
    whole = t0 == 0 && t1 == d.tiles;
  }
  // False when the share is done.
  FA_HD bool next(const DecodeParams& p) {
    left -= p.whole ? 1 : t1 - t0;
    if (left <= 0) return false;
    t0 = 0;
    if (++item == d.items) {
      item = 0;
      do {
        if (++b >= p.b.B) return false;
        d = decode_seq(p, b);
      } while (d.items == 0);
    }
    cut(p);
    return true;
  }
};

// ------------------------------------------------------------------------------ fragments and MMA
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
template <bool FP8>  // halves for an e4m3 cache, bf16 for a bf16 cache
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (FP8)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Octet position of key (or chunk) n: 0,4,1,5,2,6,3,7.
__device__ __forceinline__ int spread8(int n) { return ((n & 1) << 2) | (n >> 1); }

// One item's running state in one warp.  o[j]: accumulator of output column tile j; rows g and g + 8.
template <int D>
struct DecodeAcc {
  float o[D / 8][4];
  float m[2], l[2];
};

// Output column of element e (0, 1) of column tile j in lane quarter t.
template <int D, bool FP8>
__device__ __forceinline__ int out_col(int j, int t, int e) {
  if constexpr (!FP8) return 8 * j + 2 * t + e;
  constexpr int RUN = D / 8;  // columns that one lane's chunk of a value row holds
  return RUN * (t + 4 * e) + j;
}

// The other's state into this one's (both hold the same rows and columns).
template <int D>
__device__ __forceinline__ void absorb(DecodeAcc<D>& a, const uint8_t* from, int lane) {
  const float4* f = reinterpret_cast<const float4*>(from);
  const float4 ml = f[(D / 8) * 32 + lane];
  float ca[2], cb[2];
  const float mb[2] = {ml.x, ml.z}, lb[2] = {ml.y, ml.w};
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float mx = fmaxf(a.m[r], mb[r]);
    const float ms = mx == -INFINITY ? 0.0f : mx;
    ca[r] = exp2f(a.m[r] - ms);
    cb[r] = exp2f(mb[r] - ms);
    a.l[r] = a.l[r] * ca[r] + lb[r] * cb[r];
    a.m[r] = mx;
  }
#pragma unroll
  for (int j = 0; j < D / 8; ++j) {
    const float4 v = f[j * 32 + lane];
    a.o[j][0] = a.o[j][0] * ca[0] + v.x * cb[0];
    a.o[j][1] = a.o[j][1] * ca[0] + v.y * cb[0];
    a.o[j][2] = a.o[j][2] * ca[1] + v.z * cb[1];
    a.o[j][3] = a.o[j][3] * ca[1] + v.w * cb[1];
  }
}
template <int D>
__device__ __forceinline__ void leave(const DecodeAcc<D>& a, uint8_t* to, int lane) {
  float4* f = reinterpret_cast<float4*>(to);
#pragma unroll
  for (int j = 0; j < D / 8; ++j) f[j * 32 + lane] = make_float4(a.o[j][0], a.o[j][1], a.o[j][2], a.o[j][3]);
  f[(D / 8) * 32 + lane] = make_float4(a.m[0], a.l[0], a.m[1], a.l[1]);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kDecThreads, 2)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const DecodeParams prm) {
  using L = DecodeLayout<D, FP8>;
  constexpr int S = L::kStages, KS = D / 16, NJ = D / 8;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + S;
  float2* meta = reinterpret_cast<float2*>(smem + L::kMeta);
  int* abort_flag = reinterpret_cast<int*>(smem + L::kMisc);
  long long* scratch = reinterpret_cast<long long*>(smem + L::kMisc + 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if ((smem_u32(smem) & 1023u) != 0) {  // swizzled tiles need a 1024-byte aligned base
    if (threadIdx.x == 0) atomicCAS(prm.b.status, 0, kSiteDecode | 0x7F);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  const DecodeShare share = decode_share<kDecThreads>(prm, blockIdx.x, gridDim.x, scratch);  // has the barriers
  if (share.b >= prm.b.B) return;
  const Guard g{abort_flag, prm.b.status};
  DecodeWalk w;
  w.start(prm, share, blockIdx.x);
  const int box_rows = min(1 << prm.b.page_shift, kDecTile);
  const int box_shift = min(prm.b.page_shift, 6);
  int it = 0;  // tiles since the start: stage it % S

  if (warp == 4) {
    // ------------------------------------------------------------------------------- producer
    bool ok = true;
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    do {
      const int h = w.item % prm.b.Hkv;
      const int n_pages = (w.d.s.len + (1 << prm.b.page_shift) - 1) >> prm.b.page_shift;
      int held = -1;  // the 32 pages whose numbers and scales the lanes hold
      int page = -1;
      float2 sc = make_float2(1.0f, 1.0f);
      for (int tile = w.t0; tile < w.t1; ++tile, ++it) {
        const int keys = min(kDecTile, w.d.s.len - tile * kDecTile);  // <= 0: a sequence of no keys
        if (keys <= 0) {
          --it;
          continue;
        }
        const int boxes = (keys + box_rows - 1) >> box_shift;
        const int first_page = (tile * kDecTile) >> prm.b.page_shift;
        if ((first_page >> 5) != held) {  // a tile's pages lie in one aligned run of 32
          held = first_page >> 5;
          const int i = held * 32 + lane;
          page = i < n_pages ? load_page(prm.b, w.b, i) : -1;
          if (FP8 && page >= 0) {
            const size_t at = static_cast<size_t>(page) * prm.b.Hkv + h;
            sc = make_float2(prm.Ks[at], fmaxf(prm.Vs[at], kScaleFloor));
          }
        }
        const int my_page = __shfl_sync(0xffffffffu, page, (first_page + lane) & 31);
        const float2 my_sc = make_float2(__shfl_sync(0xffffffffu, sc.x, (first_page + lane) & 31),
                                         __shfl_sync(0xffffffffu, sc.y, (first_page + lane) & 31));
        const int st = it % S;
        if (!(ok = wait_warp(&empty[st], ((it / S) & 1) ^ 1, g, kSiteDecode | 1))) break;
        if (FP8 && lane < boxes) meta[st * 4 + lane] = my_sc;
        __syncwarp();
        if (lane == 0) mbar_expect_tx(&full[st], 2 * boxes * box_rows * L::kRowBytes);
        __syncwarp();
        if (lane < boxes) {
          // a page out of range reads as zeros beyond the map's last head
          const int z = my_page >= 0 ? my_page * prm.b.Hkv + h : prm.b.num_pages * prm.b.Hkv;
          const int y = (tile * kDecTile) & ((1 << prm.b.page_shift) - 1);
          constexpr int kCols = FP8 ? D : 64;
#pragma unroll
          for (int c = 0; c < D / kCols; ++c) {
            const int at = st * L::kTileBytes + c * L::kHalf + lane * box_rows * (kCols * (FP8 ? 1 : 2));
            tma_load_3d(smem + at, &tmK, c * kCols, y, z, &full[st]);
            tma_load_3d(smem + L::kV + at, &tmV, c * kCols, y, z, &full[st]);
          }
        }
      }
    } while (ok && w.next(prm));
    if (!ok) {  // let copies already in flight land before the CTA exits
      const uint64_t t0 = globaltimer();
      for (int i = max(it - S, 0); i < it; ++i)
        while (!mbar_try_wait(&full[i % S], (i / S) & 1) && globaltimer() - t0 < 200000000ull) {
        }
    }
    return;
  }

  // ---------------------------------------------------------------------------------- consumers
  const int gid = lane >> 2, t = lane & 3;
  bool ok = true;
  do {
    const int h = w.item % prm.b.Hkv, rb = w.item / prm.b.Hkv;
    const int rows = w.d.s.rows * prm.G - rb * kDecRows;  // real rows of the block
    const int len = w.d.s.len;
    // this lane's rows: query pointers, last visible key, score factor
    uint32_t qf[KS][4];
    float rowfac[2];
    int lim[2];
    float amax[2] = {0.0f, 0.0f};
    const __nv_bfloat16* qrow[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = rb * kDecRows + gid + 8 * r;
      const bool real = gid + 8 * r < rows;
      const int token = real ? row / prm.G : 0, head = h * prm.G + (real ? row % prm.G : 0);
      qrow[r] = real ? prm.Q + static_cast<size_t>(w.d.s.row0 + token) * prm.ldq + head * D : nullptr;
      lim[r] = prm.causal && real ? len - w.d.s.rows + token : len - 1;
      rowfac[r] = prm.scale_log2;
    }
    if constexpr (FP8) {
      uint2 qw[2][KS];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int col = 16 * (t + 4 * (s >> 2)) + (s & 3) * 4;
          qw[r][s] = qrow[r] ? *reinterpret_cast<const uint2*>(qrow[r] + col) : make_uint2(0u, 0u);
          const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qw[r][s].x));
          const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qw[r][s].y));
          amax[r] = fmaxf(fmaxf(amax[r], fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
        }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        amax[r] = fmaxf(amax[r], __shfl_xor_sync(0xffffffffu, amax[r], 1));
        amax[r] = fmaxf(amax[r], __shfl_xor_sync(0xffffffffu, amax[r], 2));
        // a power of two above the row's largest magnitude (kept where its inverse is normal)
        const int e = min(max(static_cast<int>(__float_as_uint(amax[r]) >> 23) + 1, 2), 252);
        const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        rowfac[r] = prm.scale_log2 * up;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qw[r][s].x));
          const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qw[r][s].y));
          qf[s][r] = pack_half2(a.x * down, a.y * down);
          qf[s][2 + r] = pack_half2(b.x * down, b.y * down);
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const __nv_bfloat16* q = qrow[r] ? qrow[r] + 16 * s + 2 * t : nullptr;
          qf[s][r] = q ? *reinterpret_cast<const uint32_t*>(q) : 0u;
          qf[s][2 + r] = q ? *reinterpret_cast<const uint32_t*>(q + 8) : 0u;
        }
    }
    const int lim_min = prm.causal ? len - w.d.s.rows + rb * kDecRows / prm.G : len - 1;
    DecodeAcc<D> acc;
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc.o[j][0] = acc.o[j][1] = acc.o[j][2] = acc.o[j][3] = 0.0f;
    acc.m[0] = acc.m[1] = -INFINITY;
    acc.l[0] = acc.l[1] = 0.0f;

    for (int tile = w.t0; tile < w.t1; ++tile, ++it) {
      const int key0 = tile * kDecTile + warp * 16;
      if (tile * kDecTile >= len) {
        --it;
        continue;
      }
      const int st = it % S;
      if (!(ok = wait_warp(&full[st], (it / S) & 1, g, kSiteDecode | 2))) break;
      if (key0 < len) {
        const uint32_t sK = smem_u32(smem + st * L::kTileBytes), sV = smem_u32(smem + L::kV + st * L::kTileBytes);
        if (key0 + 16 > len) {
          // slots behind the sequence's end hold whatever the page holds: their values become zeros, since
          // a weight of zero times an infinity or NaN is not zero
          constexpr int kCols = FP8 ? D : 128;  // bytes of a row in a column block
          for (int i = lane; i < 16 * L::kRowBytes / 16; i += 32) {
            const int row = warp * 16 + (i / (kCols / 16)) % 16, blk = i / (kCols / 16) / 16;
            if (tile * kDecTile + row >= len)
              *reinterpret_cast<uint4*>(smem + L::kV + st * L::kTileBytes + blk * L::kHalf + row * kCols +
                                        (i % (kCols / 16)) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
        }
        // ---- S = Q K^T: two octets of keys
        float c[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
        if constexpr (FP8) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int row = warp * 16 + n * 8 + spread8(gid);
#pragma unroll
            for (int cc = 0; cc < KS / 4; ++cc) {
              const int chunk = t + 4 * cc;
              const uint32_t a = D == 128 ? sK + row * 128 + ((chunk ^ (row & 7)) << 4)
                                          : sK + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
              const uint4 v = lds128(a);
              const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma16816<FP8>(c[n], qf[cc * 4 + i], half2_of_e4m3(x[i]), half2_of_e4m3(x[i] >> 16));
            }
          }
        } else {
          const int row = warp * 16 + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            uint32_t kf[4];
            const int chunk = (s & 3) * 2 + ((lane >> 3) & 1);
            ldsm4(sK + (s >> 2) * L::kHalf + row * 128 + ((chunk ^ (row & 7)) << 4), kf);
            mma16816<FP8>(c[0], qf[s], kf[0], kf[1]);
            mma16816<FP8>(c[1], qf[s], kf[2], kf[3]);
          }
        }
        // ---- softmax: scores in log2 units (plus log2 of the value scale)
        float ks = 1.0f, lv = 0.0f, inv_vs = 1.0f;
        if constexpr (FP8) {
          const float2 sc = meta[st * 4 + ((warp * 16) >> box_shift)];
          ks = sc.x;
          lv = log2f(sc.y);
          inv_vs = 1.0f / sc.y;
        }
        const float f0 = rowfac[0] * ks, f1 = rowfac[1] * ks;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          c[n][0] = fmaf(c[n][0], f0, lv);
          c[n][1] = fmaf(c[n][1], f0, lv);
          c[n][2] = fmaf(c[n][2], f1, lv);
          c[n][3] = fmaf(c[n][3], f1, lv);
        }
        if (key0 + 15 > lim_min) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = key0 + n * 8 + (FP8 ? t + 4 * (i & 1) : 2 * t + (i & 1));
              if (key > lim[i >> 1]) c[n][i] = -INFINITY;
            }
        }
        float mx[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] = fmaxf(fmaxf(c[0][2 * r], c[0][2 * r + 1]), fmaxf(c[1][2 * r], c[1][2 * r + 1]));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > acc.m[0] || mx[1] > acc.m[1])) {
          float al[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float m = fmaxf(acc.m[r], mx[r]);
            al[r] = m == -INFINITY ? 1.0f : exp2_sfu(acc.m[r] - m);
            acc.m[r] = m;
            acc.l[r] *= al[r];
          }
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            acc.o[j][0] *= al[0];
            acc.o[j][1] *= al[0];
            acc.o[j][2] *= al[1];
            acc.o[j][3] *= al[1];
          }
        }
        const float m0 = acc.m[0] == -INFINITY ? 0.0f : acc.m[0], m1 = acc.m[1] == -INFINITY ? 0.0f : acc.m[1];
        float p[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          p[n][0] = exp2_sfu(c[n][0] - m0);
          p[n][1] = exp2_sfu(c[n][1] - m0);
          p[n][2] = exp2_sfu(c[n][2] - m1);
          p[n][3] = exp2_sfu(c[n][3] - m1);
        }
        acc.l[0] = fmaf(p[0][0] + p[0][1] + (p[1][0] + p[1][1]), inv_vs, acc.l[0]);
        acc.l[1] = fmaf(p[0][2] + p[0][3] + (p[1][2] + p[1][3]), inv_vs, acc.l[1]);
        uint32_t pf[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          pf[2 * n] = FP8 ? pack_half2(p[n][0], p[n][1]) : pack_bf16x2(p[n][0], p[n][1]);
          pf[2 * n + 1] = FP8 ? pack_half2(p[n][2], p[n][3]) : pack_bf16x2(p[n][2], p[n][3]);
        }
        // ---- O += P V
        if constexpr (FP8) {
          constexpr int WORDS = D / 32;  // 4-byte words of a lane's chunk of a value row
          uint32_t v[4][WORDS];
          const int chunk = spread8(gid);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = warp * 16 + t + 4 * i;
            if constexpr (D == 128) {
              const uint4 x = lds128(sV + row * 128 + ((chunk ^ (row & 7)) << 4));
              v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
            } else {
              const uint2 x = lds64(sV + row * 64 + (((chunk >> 1) ^ ((row >> 1) & 3)) << 4) + (chunk & 1) * 8);
              v[i][0] = x.x, v[i][1] = x.y;
            }
          }
#pragma unroll
          for (int i = 0; i < WORDS; ++i) {
            // bytes of two keys interleaved: column 4i in the low half, 4i + 1 in the high one; then 4i + 2, 4i + 3
            const uint32_t a0 = __byte_perm(v[0][i], v[1][i], 0x5140), a1 = __byte_perm(v[0][i], v[1][i], 0x7362);
            const uint32_t b0 = __byte_perm(v[2][i], v[3][i], 0x5140), b1 = __byte_perm(v[2][i], v[3][i], 0x7362);
            mma16816<FP8>(acc.o[4 * i], pf, half2_of_e4m3(a0), half2_of_e4m3(b0));
            mma16816<FP8>(acc.o[4 * i + 1], pf, half2_of_e4m3(a0 >> 16), half2_of_e4m3(b0 >> 16));
            mma16816<FP8>(acc.o[4 * i + 2], pf, half2_of_e4m3(a1), half2_of_e4m3(b1));
            mma16816<FP8>(acc.o[4 * i + 3], pf, half2_of_e4m3(a1 >> 16), half2_of_e4m3(b1 >> 16));
          }
        } else {
          const int row = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
          for (int j = 0; j < NJ; j += 2) {
            uint32_t vf[4];
            const int chunk = (j & 7) + (lane >> 4);
            ldsm4_t(sV + (j >> 3) * L::kHalf + row * 128 + ((chunk ^ (row & 7)) << 4), vf);
            mma16816<FP8>(acc.o[j], pf, vf[0], vf[1]);
            mma16816<FP8>(acc.o[j + 1], pf, vf[2], vf[3]);
          }
        }
        // zeros written above must be done before TMA writes the stage again
        if (key0 + 16 > len) fence_proxy_async();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---- the four warps meet: 2 and 3 into 0 and 1, then 1 into 0
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      acc.l[r] += __shfl_xor_sync(0xffffffffu, acc.l[r], 1);
      acc.l[r] += __shfl_xor_sync(0xffffffffu, acc.l[r], 2);
    }
    uint8_t* box = smem + L::kMerge + (warp & 1) * L::kMergeWarp;
    if (warp >= 2) leave<D>(acc, box, lane);
    if (!(ok = group_and(1, 128, ok))) break;
    if (warp < 2) absorb<D>(acc, box, lane);
    named_barrier(1, 128);
    if (warp == 1) leave<D>(acc, box, lane);
    named_barrier(1, 128);
    if (warp == 0) {
      absorb<D>(acc, smem + L::kMerge + L::kMergeWarp, lane);
      const int slot = decode_slot(blockIdx.x, w.t0);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int lr = gid + 8 * r;
        if (lr >= rows) continue;
        const float scale = !w.whole ? 1.0f : acc.l[r] > 0.0f ? 1.0f / acc.l[r] : 0.0f;
        float x[NJ][2];
#pragma unroll
        for (int j = 0; j < NJ; ++j) x[j][0] = acc.o[j][2 * r] * scale, x[j][1] = acc.o[j][2 * r + 1] * scale;
        if (w.whole) {
          const int row = rb * kDecRows + lr;
          const size_t at = static_cast<size_t>(w.d.s.row0 + row / prm.G) * prm.Hq + h * prm.G + row % prm.G;
          __nv_bfloat16* o = prm.O + at * D;
          if constexpr (FP8) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < NJ; j += 8)
                *reinterpret_cast<uint4*>(o + out_col<D, FP8>(j, t, e)) =
                    make_uint4(pack_bf16x2(x[j][e], x[j + 1][e]), pack_bf16x2(x[j + 2][e], x[j + 3][e]),
                               pack_bf16x2(x[j + 4][e], x[j + 5][e]), pack_bf16x2(x[j + 6][e], x[j + 7][e]));
          } else {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
              *reinterpret_cast<uint32_t*>(o + out_col<D, FP8>(j, t, 0)) = pack_bf16x2(x[j][0], x[j][1]);
          }
          if (t == 0)
            prm.LSE[at] = acc.l[r] > 0.0f ? (acc.m[r] + log2f(acc.l[r])) * 0.69314718055994531f : -INFINITY;
        } else {
          float* o = prm.part_o + (static_cast<size_t>(slot) * kDecRows + lr) * D;
          if constexpr (FP8) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < NJ; j += 4)
                *reinterpret_cast<float4*>(o + out_col<D, FP8>(j, t, e)) =
                    make_float4(x[j][e], x[j + 1][e], x[j + 2][e], x[j + 3][e]);
          } else {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
              *reinterpret_cast<float2*>(o + out_col<D, FP8>(j, t, 0)) = make_float2(x[j][0], x[j][1]);
          }
          if (t == 0) prm.part_ml[static_cast<size_t>(slot) * kDecRows + lr] = make_float2(acc.m[r], acc.l[r]);
        }
      }
    }
    named_barrier(1, 128);  // the merge area is free again
  } while (w.next(prm));
}

// Joins the items that cuts divide: block c looks at the cut before CTA c's share, and joins the item it
// falls into when no earlier cut does.  One thread per four columns of a row.
constexpr int kJoinThreads = 128;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const DecodeParams prm, int n_cta) {
  __shared__ long long scratch[kJoinThreads / 32 + 2];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the shares' sums are written
  const int c = blockIdx.x + 1;
  const DecodeShare s = decode_share<kJoinThreads>(prm, c, n_cta, scratch);
  if (s.b >= prm.b.B) return;
  const DecodeSeq d = decode_seq(prm, s.b);
  const DecodeCut cut = decode_cut(s.per, c, s.off, d.tiles);
  if (cut.last < c || cut.first != c - 1) return;
  const int item = cut.item, last = cut.last;
  const int h = item % prm.b.Hkv, rb = item / prm.b.Hkv;
  const int rows = min(kDecRows, d.s.rows * prm.G - rb * kDecRows);
  auto slot = [&](int cta) { return static_cast<size_t>(decode_slot(cta, cta - (c - 1))) * kDecRows; };
  for (int i = threadIdx.x; i < rows * (D / 4); i += kJoinThreads) {
    const int lr = i / (D / 4), col = (i % (D / 4)) * 4;
    float m = -INFINITY;
    for (int k = c - 1; k <= last; ++k) m = fmaxf(m, prm.part_ml[slot(k) + lr].x);
    const float ms = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = c - 1; k <= last; ++k) {
      const float2 ml = prm.part_ml[slot(k) + lr];
      const float4 v = *reinterpret_cast<const float4*>(prm.part_o + (slot(k) + lr) * D + col);
      const float f = exp2f(ml.x - ms);
      l = fmaf(f, ml.y, l);
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int row = rb * kDecRows + lr;
    const size_t at = static_cast<size_t>(d.s.row0 + row / prm.G) * prm.Hq + h * prm.G + row % prm.G;
    *reinterpret_cast<uint2*>(prm.O + at * D + col) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (col == 0) prm.LSE[at] = l > 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace fa

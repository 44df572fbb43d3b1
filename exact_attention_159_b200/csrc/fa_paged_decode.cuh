// fa_paged_decode.cuh -- attention of few query rows (single tokens, a few drafted tokens) over the paged
// cache: one pass over the keys and values with a running maximum and sum, the long axis split evenly
// over the GPU and joined by a second small kernel.
//
// With few rows the work is reading the cache once, so everything here serves that: TMA brings tiles of
// 64 keys (bf16) or 128 keys (e4m3) of a page list into a ring of shared-memory stages (96 KB of loads in
// flight per CTA, two CTAs an SM), and the arithmetic runs on mma.sync m16n8k16 with keys (then value
// columns) as its 16 rows and the query rows as its 8 columns: the query heads that share a key/value head
// fit one or two such column tiles, where a tcgen05 tile would be 128 rows of padding.
//
// Rows: the R = rows * G (token, query head) pairs that read one key/value head, in blocks of 8 * NT.  One
// (sequence, row block, key/value head) is an item of ceil(len / tile) tiles; the items' tiles laid end to
// end, each with a unit more for its start and end, are cut into equal runs, one per CTA, so a batch of ragged
// lengths loads every SM alike.  An item
// that a cut divides leaves its unnormalised sums in the workspace, at most two a CTA, for the join.
//
// Each of the four consumer warps takes a quarter of every tile's keys and keeps its own maximum, sum and
// output accumulators; they meet once, at the item's end.
//   S^T = K Q^T:   A = 16 keys, B = Q (registers for the whole item)
//   O^T += V^T P^T: A = 16 columns of 16 values, B = P^T, S^T's accumulators transposed 8 x 8 at a time
// The maximum is a reference that moves only when a score passes it by 2^8 (as in the other forwards): the
// lanes of a row then agree on the new one; otherwise no lane has to ask another.
// e4m3 pages: codes become halves exactly (one conversion for two codes) and the scales stay outside the
// products: K's multiplies the scores, V's joins the exponent, w = 2^(s + log2 vs - m), so w <= 2^8 whatever
// the scales, O = sum w * code, and the softmax's sum is sum w / vs.  Q is brought to [-1, 1] by a power of
// two per row before it becomes halves.  P is rounded to half (11 bits; bf16 for a bf16 cache, as the
// other forwards round it); m, the sums and O are fp32.
// To feed A from bytes without a transposing load, columns are permuted: a lane's 16-byte chunk of a key
// row holds its k indices of four MMAs, and a lane's 16-byte chunk of a value row holds its rows of eight
// output tiles.  Keys 0..7 of an octet go to rows 0,2,4,6,1,3,5,7, which with TMA's 128-byte swizzle puts
// the eight lanes of a load phase on eight different chunks.
// Measured: 64 sequences of 200 to 8192 e4m3 tokens, 32 over 8 heads (555 MB), 90 to 97 us (5.8 to 6.1 of 6.56
// TB/s measured copy).  The whole call took 263 us with query rows on the MMA's rows and one CTA an SM, 124 us
// with two CTAs and cheaper conversions, 102 us with keys on the rows.  (Two column tiles of e4m3 at D = 128 take all
// 168 registers of two CTAs an SM and spill 22 bytes a thread.)
#pragma once

#include "exp2_poly.cuh"
#include "fa_paged.cuh"

namespace fa {

constexpr int kSiteDecode = 0xD00;
constexpr int kDecRows = 16;       // most query rows of an item
constexpr int kDecCtas = 2 * 148;  // two on each SM
constexpr int kDecThreads = 192;   // four consumer warps, a producer warp for K and one for V
constexpr int kDecStageBytes = 98304;
constexpr int kDecMinUnits = 2;    // a CTA's share is at least this many
constexpr int kDecItemCost = 1;    // tiles' worth of time that starting and ending an item takes
constexpr float kDecTau = 8.0f;    // log2 units
constexpr float kScaleFloor = 7.8886090522101181e-31f;  // 2^-100: smaller value scales count as this
constexpr float kBoost = 100.0f, kUnboost = kScaleFloor;

// What the softmax needs of a page's scales: K's, log2 of V's, and, since w = 2^(s + log2 vs - m) of a page
// of tiny values (a page of zeros has the smallest scale) would vanish beside others' while its keys still
// count in the sum, a boost: w' = 2^(s + log2 vs + boost - m), w = w' 2^-boost, sum += w' (2^-boost / vs).
// x: K scale, y: log2 of V's, z: 2^-boost / V scale, w: boost (0, or 100 for scales below 2^-40).
__device__ __forceinline__ float4 page_scales(float ks, float vs) {
  vs = fmaxf(vs, kScaleFloor);
  const float lv = log2f(vs);
  const bool tiny = lv < -40.0f;
  return make_float4(ks, lv, (tiny ? kUnboost : 1.0f) / vs, tiny ? kBoost : 0.0f);
}

// 2^d for d <= 0 as two factors, the second 1 down to the smallest normal.  A softmax's sum counts a key by 1 / (its
// value scale), up to 2^100, in units of a reference that holds the scale's logarithm: when the reference moves from
// a page of zeros to one of scale 2^60, by 2^-160, what that leaves of the sum still counts, and the one factor would
// flush to zero.  (O's terms hold no 1 / scale: what flushes there is nothing beside the largest weight's rounding.)
struct Exp2Pair {
  float a, b;
  __device__ __forceinline__ explicit Exp2Pair(float d) : a(exp2_sfu(fmaxf(d, -126.0f))), b(exp2_sfu(fminf(d + 126.0f, 0.0f))) {}
  __device__ __forceinline__ float times(float x) const { return x * a * b; }
};

// What the join needs of the cut before share c, left in the workspace by CTA c, whose share begins with tile
// `tile` of an item of n.
struct alignas(16) CutPlan {
  long long per;
  int tile, n;     // tile 0 (or no tile in the share at all): nothing is divided here
  int h;           // key/value head
  int row0, rows;  // the item's first row among the sequence's rows * G, and its number of rows
  int token0;      // the sequence's first token row
};
// The shares `first`..`last` that an item lies in; first < c - 1: an earlier cut divides it too.
struct Cut {
  int first, last;
};
FA_HD Cut cut_of(long long per, int c, int tile, int n) {
  const long long begin = per * c - tile;
  return Cut{static_cast<int>(divide(begin, per)), static_cast<int>(divide(begin + n - 1, per))};
}

struct DecodeParams {
  PagedBatch b;
  const __nv_bfloat16* Q;  // [T, Hq, D], ldq elements between tokens
  long long ldq;
  __nv_bfloat16* O;   // [T, Hq, D]
  float* LSE;         // [T, Hq]
  const float *Ks, *Vs;
  float* part_o;      // [2 * n_cta][rows][D] unnormalised sums
  float2* part_ml;    // [2 * n_cta][rows] (m in log2 units, l)
  CutPlan* plan;      // [n_cta]
  int G, Hq;
  int tile, rows;     // keys of a tile (DecodeLayout::kTile), query rows of an item (8 * NT)
  int max_rows;       // sequences of more rows * G are another kernel's
  int causal, whole;  // whole: shares are whole items (short caches), nothing is joined
  float scale_log2;
};

template <int D, bool FP8>
struct DecodeLayout {
  static constexpr int kTile = FP8 ? 128 : 64;       // keys: a quarter is one warp's, 32 or 16
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  static constexpr int kHalf = kTile * 128;          // bytes of a 128-byte-wide column block of a tile
  static constexpr int kTileBytes = kTile * kRowBytes;
  static constexpr int kStages = kDecStageBytes / (2 * kTileBytes);
  static constexpr int kBoxes = kTile / 16;          // pages of a tile, at most
  static constexpr int kV = kStages * kTileBytes;
  static constexpr int kMerge = 2 * kV;              // two warps' accumulators, eight query rows at a time
  static constexpr int kMergeWarp = (D / 16) * 512 + 512;  // a float4 per lane and column tile, then (m, l) x 2
  static constexpr int kMeta = kMerge + 2 * kMergeWarp;    // [stage][box] page_scales
  static constexpr int kBar = kMeta + kStages * kBoxes * 16;
  static constexpr int kMisc = kBar + 2 * kStages * 8;
  static constexpr int kBytes = kMisc + 96;
  static_assert(kBytes <= (233472 - 2 * 1024) / 2, "two CTAs must fit an SM");
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
  d.tiles = max(1, (d.s.len + p.tile - 1) / p.tile);  // a sequence of no keys still gets its rows written
  d.items = mine ? static_cast<int>((rows + p.rows - 1) / p.rows) * p.b.Hkv : 0;
  return d;
}
FA_HD long long decode_units(const DecodeParams& p, const DecodeSeq& d) {
  return static_cast<long long>(d.items) * (p.whole ? 1 : d.tiles + kDecItemCost);
}
FA_HD long long decode_per(const DecodeParams& p, long long total, int n_cta) {
  const long long per = divide(total + n_cta - 1, n_cta);
  return !p.whole && per < kDecMinUnits ? kDecMinUnits : per;
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

// Walks a CTA's share: one segment (an item's tiles [t0, t1)) after another.
struct DecodeWalk {
  long long left;  // units
  int b, item, u0, t0, t1;
  DecodeSeq d;
  bool whole;
  // False when the share holds no tile.
  FA_HD bool start(const DecodeParams& p, const DecodeShare& s, int index) {
    left = min(s.per, s.total - s.per * index);
    b = s.b;
    d = decode_seq(p, b);
    const int units = d.tiles + kDecItemCost;
    item = static_cast<int>(p.whole ? s.off : divide(s.off, units));
    u0 = p.whole ? 0 : static_cast<int>(s.off - static_cast<long long>(item) * units);
    cut(p);
    return t1 > 0 || next(p);
  }
  FA_HD void cut(const DecodeParams& p) {
    t0 = max(0, u0 - kDecItemCost);
    t1 = p.whole ? d.tiles : max(0, static_cast<int>(min(static_cast<long long>(d.tiles + kDecItemCost), u0 + left)) - kDecItemCost);
    whole = t0 == 0 && t1 == d.tiles;
  }
  // False when the share is done.
  FA_HD bool next(const DecodeParams& p) {
    do {
      left -= p.whole ? 1 : d.tiles + kDecItemCost - u0;
      if (left <= 0) return false;
      u0 = 0;
      if (++item == d.items) {
        item = 0;
        do {
          if (++b >= p.b.B) return false;
          d = decode_seq(p, b);
        } while (d.items == 0);
      }
      cut(p);
    } while (t1 == 0);
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

// 8 x 8 halves (or bf16) transposed across the warp: lane 4i + j gives row i, columns 2j and 2j + 1.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// One item's running state in one warp, query rows 8 n + 2t and 8 n + 2t + 1 of lane quarter t.
template <int D, int NT>
struct DecodeAcc {
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];
};

// Warp `gives`'s state into warp `takes`'s (both hold the same rows and columns), eight query rows at a
// time through `box`; every consumer warp calls it.
template <int D, int NT>
__device__ __forceinline__ void meet(DecodeAcc<D, NT>& a, uint8_t* box, int lane, bool gives, bool takes) {
  constexpr int N = D / 16;
  float4* f = reinterpret_cast<float4*>(box);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (gives) {
#pragma unroll
      for (int j = 0; j < N; ++j) f[j * 32 + lane] = make_float4(a.o[n][j][0], a.o[n][j][1], a.o[n][j][2], a.o[n][j][3]);
      f[N * 32 + lane] = make_float4(a.m[n][0], a.l[n][0], a.m[n][1], a.l[n][1]);
    }
    named_barrier(1, 128);
    if (takes) {
      const float4 ml = f[N * 32 + lane];
      const float mb[2] = {ml.x, ml.z}, lb[2] = {ml.y, ml.w};
      float ca[2], cb[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mx = fmaxf(a.m[n][e], mb[e]);
        const float ms = mx == -INFINITY ? 0.0f : mx;
        const Exp2Pair pa(a.m[n][e] - ms), pb(mb[e] - ms);
        ca[e] = pa.times(1.0f);
        cb[e] = pb.times(1.0f);
        a.l[n][e] = pa.times(a.l[n][e]) + pb.times(lb[e]);
        a.m[n][e] = mx;
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float4 v = f[j * 32 + lane];
        float* o = a.o[n][j];
        o[0] = o[0] * ca[0] + v.x * cb[0];
        o[1] = o[1] * ca[1] + v.y * cb[1];
        o[2] = o[2] * ca[0] + v.z * cb[0];
        o[3] = o[3] * ca[1] + v.w * cb[1];
      }
    }
    named_barrier(1, 128);
  }
}

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(kDecThreads, 2)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const DecodeParams prm) {
  using L = DecodeLayout<D, FP8>;
  constexpr int S = L::kStages, KS = D / 16, NJ = D / 16, TILE = L::kTile, NS = TILE / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + S;
  float4* meta = reinterpret_cast<float4*>(smem + L::kMeta);
  int* abort_flag = reinterpret_cast<int*>(smem + L::kMisc);
  long long* scratch = reinterpret_cast<long long*>(smem + L::kMisc + 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_launch();
  if ((smem_u32(smem) & 1023u) != 0) {  // swizzled tiles need a 1024-byte aligned base
    if (threadIdx.x == 0) {
      atomicCAS(prm.b.status, 0, kSiteDecode | 0x7F);
      prm.plan[blockIdx.x] = CutPlan{};
    }
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 2);   // both producers
      mbar_init(&empty[i], 4);  // the consumer warps
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  const DecodeShare share = decode_share<kDecThreads>(prm, blockIdx.x, gridDim.x, scratch);  // has the barriers
  DecodeWalk w;
  if (share.b >= prm.b.B || !w.start(prm, share, blockIdx.x)) {
    if (threadIdx.x == 0) prm.plan[blockIdx.x] = CutPlan{};
    grid_dependency_wait();
    return;
  }
  const Guard g{abort_flag, prm.b.status};
  if (threadIdx.x == 0) {
    const int row0 = w.item / prm.b.Hkv * prm.rows;
    prm.plan[blockIdx.x] = CutPlan{share.per, w.t0, w.d.tiles, w.item % prm.b.Hkv, row0,
                                   min(prm.rows, w.d.s.rows * prm.G - row0), w.d.s.row0};
  }
  const int box_shift = min(prm.b.page_shift, FP8 ? 7 : 6), box_rows = 1 << box_shift;
  int it = 0;  // tiles since the start: stage it % S

  if (warp >= 4) {
    // ------------------------------------------------------------------ producers: K (with the scales), V
    // A lane issues the boxes of one page; an issue takes about 95 clocks, which for pages of 16 bf16 slots is
    // 0.8 us a tile from one warp (half from two).
    const bool is_v = warp == 5;
    const CUtensorMap* map = is_v ? &tmV : &tmK;
    bool ok = true;
    prefetch_tmap(map);
    do {
      const int h = w.item % prm.b.Hkv;
      const int n_pages = (w.d.s.len + (1 << prm.b.page_shift) - 1) >> prm.b.page_shift;
      int held = -1;  // the 32 pages whose numbers and scales the lanes hold
      int page = -1;
      float4 sc = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
      for (int tile = w.t0; tile < w.t1; ++tile, ++it) {
        const int keys = min(TILE, w.d.s.len - tile * TILE);  // <= 0: a sequence of no keys
        if (keys <= 0) {
          --it;
          continue;
        }
        const int boxes = (keys + box_rows - 1) >> box_shift;
        const int first_page = (tile * TILE) >> prm.b.page_shift;
        if ((first_page >> 5) != held) {  // a tile's pages lie in one aligned run of 32
          held = first_page >> 5;
          const int i = held * 32 + lane;
          page = i < n_pages ? load_page(prm.b, w.b, i) : -1;
          if (FP8 && !is_v && page >= 0) {
            const size_t at = static_cast<size_t>(page) * prm.b.Hkv + h;
            sc = page_scales(prm.Ks[at], prm.Vs[at]);
          }
        }
        const int my_page = __shfl_sync(0xffffffffu, page, (first_page + lane) & 31);
        float4 my_sc = sc;
        if (FP8 && !is_v) {
          my_sc.x = __shfl_sync(0xffffffffu, sc.x, (first_page + lane) & 31);
          my_sc.y = __shfl_sync(0xffffffffu, sc.y, (first_page + lane) & 31);
          my_sc.z = __shfl_sync(0xffffffffu, sc.z, (first_page + lane) & 31);
          my_sc.w = __shfl_sync(0xffffffffu, sc.w, (first_page + lane) & 31);
        }
        const int st = it % S;
        if (!(ok = wait_warp(&empty[st], ((it / S) & 1) ^ 1, g, kSiteDecode | 1))) break;
        if (FP8 && !is_v && lane < boxes) meta[st * L::kBoxes + lane] = my_sc;
        __syncwarp();
        if (lane == 0) mbar_expect_tx(&full[st], boxes * box_rows * L::kRowBytes);
        __syncwarp();
        if (lane < boxes) {
          // a page out of range reads as zeros beyond the map's last head
          const int z = my_page >= 0 ? my_page * prm.b.Hkv + h : prm.b.num_pages * prm.b.Hkv;
          const int y = (tile * TILE) & ((1 << prm.b.page_shift) - 1);
          constexpr int kCols = FP8 ? D : 64;
          uint8_t* to = smem + (is_v ? L::kV : 0) + st * L::kTileBytes + lane * box_rows * (kCols * (FP8 ? 1 : 2));
#pragma unroll
          for (int c = 0; c < D / kCols; ++c) tma_load_3d(to + c * L::kHalf, map, c * kCols, y, z, &full[st]);
        }
      }
    } while (ok && w.next(prm));
    if (!ok) {  // let copies already in flight land before the CTA exits
      const uint64_t t0 = globaltimer();
      for (int i = max(it - S, 0); i < it; ++i)
        while (!mbar_try_wait(&full[i % S], (i / S) & 1) && globaltimer() - t0 < 200000000ull) {
        }
    }
    // when another kernel of the call runs alongside, this one ends after it: what follows may rely on both
    grid_dependency_wait();
    return;
  }

  // ---------------------------------------------------------------------------------- consumers
  const int gid = lane >> 2, t = lane & 3;
  bool ok = true;
  do {
    const int h = w.item % prm.b.Hkv, rb = w.item / prm.b.Hkv;
    const int rows = w.d.s.rows * prm.G - rb * (8 * NT);  // real rows of the block
    const int len = w.d.s.len;
    // Q: row 8 n + gid; what the scores need of rows 8 n + 2t + e: last visible key, factor
    uint32_t qf[NT][KS][2];
    float rowfac[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = rb * (8 * NT) + 8 * n + gid;
      const __nv_bfloat16* q = nullptr;
      if (8 * n + gid < rows)
        q = prm.Q + static_cast<size_t>(w.d.s.row0 + row / prm.G) * prm.ldq + (h * prm.G + row % prm.G) * D;
      if constexpr (FP8) {
        uint2 qw[KS];
        float amax = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int col = 16 * (t + 4 * (s >> 2)) + (s & 3) * 4;
          qw[s] = q ? *reinterpret_cast<const uint2*>(q + col) : make_uint2(0u, 0u);
          const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qw[s].x));
          const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qw[s].y));
          amax = fmaxf(fmaxf(amax, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // a power of two above the row's largest magnitude (kept where its inverse is normal)
        const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) + 1, 2), 252);
        const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qw[s].x));
          const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qw[s].y));
          qf[n][s][0] = pack_half2(a.x * down, a.y * down);
          qf[n][s][1] = pack_half2(b.x * down, b.y * down);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          rowfac[n][i] = prm.scale_log2 * __shfl_sync(0xffffffffu, up, (2 * t + i) * 4);
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          qf[n][s][0] = q ? *reinterpret_cast<const uint32_t*>(q + 16 * s + 2 * t) : 0u;
          qf[n][s][1] = q ? *reinterpret_cast<const uint32_t*>(q + 16 * s + 2 * t + 8) : 0u;
        }
        rowfac[n][0] = rowfac[n][1] = prm.scale_log2;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int lr = 8 * n + 2 * t + e;
        lim[n][e] = prm.causal && lr < rows ? len - w.d.s.rows + (rb * (8 * NT) + lr) / prm.G : len - 1;
      }
    }
    const int lim_min = prm.causal ? len - w.d.s.rows + rb * (8 * NT) / prm.G : len - 1;
    DecodeAcc<D, NT> acc;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc.o[n][j][0] = acc.o[n][j][1] = acc.o[n][j][2] = acc.o[n][j][3] = 0.0f;
      acc.m[n][0] = acc.m[n][1] = -INFINITY;
      acc.l[n][0] = acc.l[n][1] = 0.0f;
    }

    for (int tile = w.t0; tile < w.t1; ++tile, ++it) {
      const int row0 = warp * (16 * NS), key0 = tile * TILE + row0;  // this warp's first row of the tile
      if (tile * TILE >= len) {
        --it;
        continue;
      }
      const int st = it % S;
      if (!(ok = wait_warp(&full[st], (it / S) & 1, g, kSiteDecode | 2))) break;
      if (key0 < len) {
        const uint32_t sK = smem_u32(smem + st * L::kTileBytes), sV = smem_u32(smem + L::kV + st * L::kTileBytes);
        if (key0 + 16 * NS > len) {
          // slots behind the sequence's end hold whatever the page holds: their values become zeros, since
          // a weight of zero times an infinity or NaN is not zero
          constexpr int kCols = FP8 ? D : 128;  // bytes of a row in a column block
          for (int i = lane; i < NS * L::kRowBytes; i += 32) {
            const int row = row0 + (i / (kCols / 16)) % (16 * NS), blk = i / (kCols / 16) / (16 * NS);
            if (tile * TILE + row >= len)
              *reinterpret_cast<uint4*>(smem + L::kV + st * L::kTileBytes + blk * L::kHalf + row * kCols +
                                        (i % (kCols / 16)) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
        }
        // ---- S^T = K Q^T: 16 keys at a time; c[.][.][2r + e] is key (row of lane) + 8r, query row 2t + e
        float c[NS][NT][4];
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int n = 0; n < NT; ++n) c[s][n][0] = c[s][n][1] = c[s][n][2] = c[s][n][3] = 0.0f;
        if constexpr (FP8) {
#pragma unroll
          for (int cc = 0; cc < KS / 4; ++cc) {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
              uint32_t x[2][4];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const int row = row0 + 16 * s + 8 * r + spread8(gid), chunk = t + 4 * cc;
                const uint4 v = lds128(D == 128 ? sK + row * 128 + ((chunk ^ (row & 7)) << 4)
                                                : sK + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
                x[r][0] = v.x, x[r][1] = v.y, x[r][2] = v.z, x[r][3] = v.w;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t a[4];
                halves_of_e4m3(x[0][i], a[0], a[2]);
                halves_of_e4m3(x[1][i], a[1], a[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816<FP8>(c[s][n], a, qf[n][cc * 4 + i][0], qf[n][cc * 4 + i][1]);
              }
            }
          }
        } else {
          const int row = row0 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t a[4];
            const int chunk = (k & 3) * 2 + (lane >> 4);
            ldsm4(sK + (k >> 2) * L::kHalf + row * 128 + ((chunk ^ (row & 7)) << 4), a);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<FP8>(c[0][n], a, qf[n][k][0], qf[n][k][1]);
          }
        }
        // ---- softmax: scores in log2 units (plus log2 of the value scale)
        float inv_vs[NS], boost[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          float ks = 1.0f, lv = 0.0f;
          inv_vs[s] = 1.0f;
          boost[s] = 0.0f;
          if constexpr (FP8) {
            if (s == 0 || key0 + 16 * s < len) {  // a page behind the end brought no scales
              const float4 sc = meta[st * L::kBoxes + ((row0 + 16 * s) >> box_shift)];
              ks = sc.x;
              lv = sc.y;
              inv_vs[s] = sc.z;
              boost[s] = sc.w;
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float f0 = rowfac[n][0] * ks, f1 = rowfac[n][1] * ks;
            c[s][n][0] = fmaf(c[s][n][0], f0, lv);
            c[s][n][1] = fmaf(c[s][n][1], f1, lv);
            c[s][n][2] = fmaf(c[s][n][2], f0, lv);
            c[s][n][3] = fmaf(c[s][n][3], f1, lv);
          }
        }
        if (key0 + 16 * NS - 1 > lim_min) {
#pragma unroll
          for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = key0 + 16 * s + 8 * (i >> 1) + (FP8 ? spread8(gid) : gid);
                if (key > lim[n][i & 1]) c[s][n][i] = -INFINITY;
              }
        }
        float mx[NT][2];
        bool passed = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[n][e] = fmaxf(c[0][n][e], c[0][n][2 + e]);
#pragma unroll
            for (int s = 1; s < NS; ++s) mx[n][e] = fmax3(mx[n][e], c[s][n][e], c[s][n][2 + e]);
            passed |= mx[n][e] > acc.m[n][e] + kDecTau;
          }
        if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float al[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float m = mx[n][e];
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
              m = fmaxf(m, acc.m[n][e]);
              const Exp2Pair by(m == -INFINITY ? 0.0f : acc.m[n][e] - m);
              al[e] = by.times(1.0f);
              acc.m[n][e] = m;
              acc.l[n][e] = by.times(acc.l[n][e]);
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              acc.o[n][j][0] *= al[0];
              acc.o[n][j][1] *= al[1];
              acc.o[n][j][2] *= al[0];
              acc.o[n][j][3] *= al[1];
            }
          }
        }
        uint32_t pf[NS][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float m0 = acc.m[n][0] == -INFINITY ? 0.0f : acc.m[n][0];
          const float m1 = acc.m[n][1] == -INFINITY ? 0.0f : acc.m[n][1];
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const float d0 = FP8 ? boost[s] - m0 : -m0, d1 = FP8 ? boost[s] - m1 : -m1;
            float p0 = exp2_sfu(c[s][n][0] + d0), p1 = exp2_sfu(c[s][n][1] + d1);
            float p2 = exp2_sfu(c[s][n][2] + d0), p3 = exp2_sfu(c[s][n][3] + d1);
            acc.l[n][0] = FP8 ? fmaf(p0 + p2, inv_vs[s], acc.l[n][0]) : acc.l[n][0] + (p0 + p2);
            acc.l[n][1] = FP8 ? fmaf(p1 + p3, inv_vs[s], acc.l[n][1]) : acc.l[n][1] + (p1 + p3);
            if (FP8 && boost[s] > 0.0f) p0 *= kUnboost, p1 *= kUnboost, p2 *= kUnboost, p3 *= kUnboost;
            pf[s][n][0] = transpose8x8(FP8 ? pack_half2(p0, p1) : pack_bf16x2(p0, p1));
            pf[s][n][1] = transpose8x8(FP8 ? pack_half2(p2, p3) : pack_bf16x2(p2, p3));
          }
        }
        // ---- O^T += V^T P^T
        if constexpr (FP8) {
          constexpr int WORDS = D / 32;  // 4-byte words of a lane's chunk of a value row
          const int chunk = spread8(gid);
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            uint32_t v[4][WORDS];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = row0 + 16 * s + t + 4 * i;
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
              // bytes of two keys interleaved: columns 4i (row gid of the tile) and 4i + 1 (row gid + 8), then two more
              uint32_t a[2][4];
              halves_of_e4m3(__byte_perm(v[0][i], v[1][i], 0x5140), a[0][0], a[0][1]);
              halves_of_e4m3(__byte_perm(v[2][i], v[3][i], 0x5140), a[0][2], a[0][3]);
              halves_of_e4m3(__byte_perm(v[0][i], v[1][i], 0x7362), a[1][0], a[1][1]);
              halves_of_e4m3(__byte_perm(v[2][i], v[3][i], 0x7362), a[1][2], a[1][3]);
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816<FP8>(acc.o[n][2 * i + e], a[e], pf[s][n][0], pf[s][n][1]);
            }
          }
        } else {
          const int row = row0 + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            uint32_t a[4];
            const int chunk = (2 * j & 7) + ((lane >> 3) & 1);
            ldsm4_t(sV + (j >> 2) * L::kHalf + row * 128 + ((chunk ^ (row & 7)) << 4), a);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<FP8>(acc.o[n][j], a, pf[0][n][0], pf[0][n][1]);
          }
        }
        // zeros written above must be done before TMA writes the stage again
        if (key0 + 16 * NS > len) fence_proxy_async();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ---- the lanes of a row add up, then the four warps meet: 2 and 3 into 0 and 1, then 1 into 0
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) acc.l[n][e] += __shfl_xor_sync(0xffffffffu, acc.l[n][e], o);
    if (!(ok = group_and(1, 128, ok))) break;
    meet<D, NT>(acc, smem + L::kMerge + (warp & 1) * L::kMergeWarp, lane, warp >= 2, warp < 2);
    meet<D, NT>(acc, smem + L::kMerge, lane, warp == 1, warp == 0);
    if (warp == 0) {
      const size_t slot = static_cast<size_t>(decode_slot(blockIdx.x, w.t0)) * prm.rows;
      constexpr int RUN = D / 8;  // e4m3: consecutive columns of a lane, from RUN * spread8(gid)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (FP8) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int lr = 8 * n + 2 * t + e, row = rb * (8 * NT) + lr;
            if (lr >= rows) continue;
            float x[RUN];
            const float scale = !w.whole ? 1.0f : acc.l[n][e] != 0.0f ? 1.0f / acc.l[n][e] : 0.0f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) x[2 * j] = acc.o[n][j][e] * scale, x[2 * j + 1] = acc.o[n][j][2 + e] * scale;
            if (w.whole) {
              const size_t at = static_cast<size_t>(w.d.s.row0 + row / prm.G) * prm.Hq + h * prm.G + row % prm.G;
#pragma unroll
              for (int j = 0; j < RUN; j += 8)
                *reinterpret_cast<uint4*>(prm.O + at * D + RUN * spread8(gid) + j) =
                    make_uint4(pack_bf16x2(x[j], x[j + 1]), pack_bf16x2(x[j + 2], x[j + 3]),
                               pack_bf16x2(x[j + 4], x[j + 5]), pack_bf16x2(x[j + 6], x[j + 7]));
            } else {
#pragma unroll
              for (int j = 0; j < RUN; j += 4)
                *reinterpret_cast<float4*>(prm.part_o + (slot + lr) * D + RUN * spread8(gid) + j) =
                    make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
            }
          }
        } else if (w.whole) {
          // two rows' values of one column become two columns of one row, so that a lane stores pairs
          const float i0 = acc.l[n][0] != 0.0f ? 1.0f / acc.l[n][0] : 0.0f;
          const float i1 = acc.l[n][1] != 0.0f ? 1.0f / acc.l[n][1] : 0.0f;
          const int row = rb * (8 * NT) + 8 * n + gid;
          const size_t at = static_cast<size_t>(w.d.s.row0 + row / prm.G) * prm.Hq + h * prm.G + row % prm.G;
#pragma unroll
          for (int j = 0; j < 2 * NJ; ++j) {
            const float* o = acc.o[n][j >> 1] + 2 * (j & 1);
            const uint32_t y = transpose8x8(pack_bf16x2(o[0] * i0, o[1] * i1));
            if (8 * n + gid < rows) *reinterpret_cast<uint32_t*>(prm.O + at * D + 8 * j + 2 * t) = y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int lr = 8 * n + 2 * t + e;
            if (lr >= rows) continue;
#pragma unroll
            for (int j = 0; j < 2 * NJ; ++j)
              prm.part_o[(slot + lr) * D + 8 * j + gid] = acc.o[n][j >> 1][2 * (j & 1) + e];
          }
        }
        if (gid == 0)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int lr = 8 * n + 2 * t + e, row = rb * (8 * NT) + lr;
            if (lr >= rows) continue;
            if (w.whole)
              prm.LSE[static_cast<size_t>(w.d.s.row0 + row / prm.G) * prm.Hq + h * prm.G + row % prm.G] =
                  acc.l[n][e] != 0.0f ? (acc.m[n][e] + log2f(acc.l[n][e])) * 0.69314718055994531f : -INFINITY;
            else
              prm.part_ml[slot + lr] = make_float2(acc.m[n][e], acc.l[n][e]);
          }
      }
    }
  } while (w.next(prm));
}

}  // namespace fa

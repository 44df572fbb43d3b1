// fa_paged_prefill.cuh -- attention of many query rows (prompt chunks, verified drafts of wide groups) over
// the paged cache on the 5th-generation tensor cores.
//
// The pipeline is that of the contiguous forward (fa_fwd.cuh): two 128-row query tiles in flight per CTA,
// S = Q K^T into TMEM, one thread per score row for the online softmax with conditional rescaling, P back
// over S in TMEM, O += P V.  What the cache changes:
//   Rows.  The R = rows * G (token, query head) pairs that read one key/value head are the rows, so a key
//     tile is read once for all G heads; 256 of them are a pair of tiles.
//   Work.  A CTA per SM walks an equal share of all (sequence, key/value head, pair) items' key tiles laid
//     end to end, each item with kPreItemCost units more for its start (Q) and end (O), so neither a batch of ragged prompts nor a single chunk of few pairs leaves SMs idle; an
//     item that a cut divides leaves unnormalised fp32 sums for the join.  The number of tiles that a pair
//     sees under the causal mask is a floor of a linear function, whose sums have a closed form, so every
//     CTA finds its share by itself.
//   Pages.  A 128-key tile is one TMA box for each of its pages.  Slots behind the sequence's end may hold
//     anything: their scores are masked, and their values are zeroed in shared memory before the MMA (a
//     weight of zero times a NaN is not zero).
//   e4m3.  S comes from the codes themselves: a row of Q, brought to 256 by a power of two, is the sum of two
//     e4m3 rows (its 8-bit significands in two parts; what is below 2^-18 of the row's largest is rounded off),
//     so S = Q1 K^T + Q2 K^T on the 8-bit tensor pipe, as fast as one 16-bit product and with no conversion of
//     K.  V's codes land in a staging ring and two warps turn them into halves (exact).  The scales stay outside
//     the products: K's multiplies the scores of its 16 columns or more, V's joins the exponent (w = 2^(s +
//     log2 vs - m), O = sum w * code, the softmax's sum is sum w / vs).  P is rounded to half.
// Measured: 2048 tokens over 16384 keys, 32 over 8 heads (515 GFLOP): bf16 473 us at 1.955 GHz in
// short runs, 528 us at the 1.75 GHz that the power cap leaves a loop of seconds (925 K cycles either way, 4420
// per pair of tiles and key tile; the contiguous forward takes 928 K; tensor pipe 54 % active), e4m3 514 to 536
// us.  An earlier form of the e4m3 kernel, which converted K to halves as it does V, took 757 us.
#pragma once

#include "exp2_poly.cuh"
#include "fa_fwd.cuh"
#include "fa_paged.cuh"
#include "fa_paged_decode.cuh"

namespace fa {

constexpr int kSitePrefill = 0xC00;
constexpr int kPreCtas = 148;
constexpr int kPreRows = 256;     // query rows of an item: two tiles
constexpr int kPreItemCost = 4;   // key tiles' worth of time that starting and ending an item takes

// Register split (setmaxnreg), the launch's total.  The issuing thread keeps its loop state and the
// descriptors that the compiler holds: at the contiguous forward's 56 it spilled 28 words and reloaded them
// between UMMAs (a 2048-token chunk over 16384 bf16 keys: 554 us against 493 us); the softmax fits 208.
constexpr int kPreRegsCtl = 88, kPreRegsSoftmax = 208;
static_assert(128 * kPreRegsCtl + 256 * kPreRegsSoftmax <= 384 * ((65536 / 384) / 8 * 8),
              "prefill register split exceeds the launch's");

struct PrefillParams {
  PagedBatch b;
  const __nv_bfloat16* Q;  // [T, Hq, D], ldq elements between tokens
  long long ldq;
  __nv_bfloat16* O;   // [T, Hq, D]
  float* LSE;         // [T, Hq]
  const float *Ks, *Vs;
  float* part_o;      // [2 * kPreCtas][kPreRows][D] unnormalised sums
  float2* part_ml;    // [2 * kPreCtas][kPreRows] (m in log2 units, l)
  CutPlan* plan;      // [kPreCtas]
  int G, Hq;
  int min_rows;       // sequences of no more rows * G are the other kernel's
  int causal;
  float scale_log2;
};

template <int D, bool FP8>
struct PrefillLayout {
  static constexpr int kQBytes = kTile * D * 2;             // a tile of Q: bf16, or two parts of e4m3
  static constexpr int kKBytes = kTile * D * (FP8 ? 1 : 2);
  static constexpr int kVBytes = kTile * D * 2;             // bf16 or halves
  static constexpr int kRawBytes = FP8 ? kTile * D : 0;     // e4m3 staging of a tile of V
  static constexpr int kStagesK = (D == 128 ? 2 : 3) + (FP8 ? 1 : 0);
  static constexpr int kStagesV = D == 128 ? 2 : 3;
  static constexpr int kRaws = 2;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kQBytes;
  static constexpr int kV = kK + kStagesK * kKBytes;
  static constexpr int kRaw = kV + kStagesV * kVBytes;
  static constexpr int kMeta = kRaw + kRaws * kRawBytes;  // [8 tiles][8 groups of 16 keys] page_scales
  static constexpr int kBar = kMeta + (FP8 ? 8 * 8 * 16 : 0);
  // q_full[2], k_full[], v_full[], k_empty[], v_empty[], v_land[], s_full[2], p_full[2], o_full[2], drain, raw_empty[],
  // seg_full[kSegs], seg_empty[kSegs]
  static constexpr int kSegs = 4;
  static constexpr int kNumBars = 2 + 2 * kStagesK + 3 * kStagesV + 6 + 1 + kRaws + 2 * kSegs;
  static constexpr int kSeg = kBar + kNumBars * 8 + (kNumBars & 1) * 8;
  static constexpr int kMl = kSeg + kSegs * 48;  // (m, l) of a split item's second half
  static constexpr int kMisc = kMl + kTile * 8;
  static constexpr int kBytes = kMisc + 16 + 16 * 8;
  static constexpr int kThreads = 384;
  static constexpr int kLaunchRegs = (65536 / kThreads) / 8 * 8;
  static_assert(kBytes <= 232448, "more shared memory than a CTA may have");
};

// Halves: the instruction descriptor of bf16 without its two type bits.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn_major, bool b_mn_major) {
  return idesc_bf16_f32(M, N, a_mn_major, b_mn_major) & ~((1u << 7) | (1u << 10));
}

// e4m3 operands (kind::f8f6f4, both of type 0), fp32 accumulate; 32 of K an instruction.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void mma_ss_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, "
      "p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// K-major rows of 64 bytes under the 64-byte swizzle (8-row groups of 512 bytes).
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(512 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(4) << 61);
}

// ------------------------------------------------------------------------------------- the plan
// Sum of floor((a i + b) / m) over i = 0 .. n - 1 (all non-negative, m > 0), by the well-known recursion that counts
// the lattice points under the line with the steps of Euclid's algorithm.  Here n < 2^24, b < 2^31 and a, m are small, so the divisions are of 32 bits.
FA_HD long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  long long sum = 0;
  while (n > 0) {
    sum += static_cast<long long>(n) * (n - 1) / 2 * (a / m) + static_cast<long long>(n) * (b / m);
    a %= m;
    b %= m;
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const uint32_t x = m;
    m = a;
    a = x;
  }
  return sum;
}

struct PrefillSeq {
  SeqInfo s;
  int pairs;       // 0: no rows, or too few for this kernel
  int tiles;       // key tiles of the whole sequence (1 when it has no key: its rows are written)
  int half;        // the last pair has one tile of rows: its steps are two key tiles each
  int linear;      // pair p counts (x + 2 p) / G + 1 tiles, the last one all; otherwise every pair counts all
  int x;
  int G;
  // Units counted before pair p (p < pairs), and pair p's steps (key tiles, or two of them); a pair's rows see no
  // key beyond its own steps.
  FA_HD long long before(int p) const {
    return static_cast<long long>(p) * kPreItemCost +
           (linear ? p + floor_sum(p, G, 2, x) : static_cast<long long>(p) * tiles);
  }
  FA_HD int count(int p) const {
    if (p == pairs - 1) return half ? (tiles + 1) / 2 : tiles;
    return linear ? static_cast<int>((x + 2 * p) / G) + 1 : tiles;
  }
  FA_HD long long head_units() const { return pairs == 0 ? 0 : before(pairs - 1) + count(pairs - 1) + kPreItemCost; }
};
FA_HD PrefillSeq prefill_seq(const PrefillParams& p, int b) {
  PrefillSeq d;
  d.s = load_seq(p.b, b);
  d.G = p.G;
  const long long rows = static_cast<long long>(d.s.rows) * p.G;
  d.pairs = rows > p.min_rows ? static_cast<int>((rows + kPreRows - 1) / kPreRows) : 0;
  d.tiles = max(1, (d.s.len + 127) / 128);
  d.half = d.pairs > 0 && rows - static_cast<long long>(d.pairs - 1) * kPreRows <= kTile;
  // pair p's last row (when the pair is full) is token (256 (p + 1) - 1) / G, which sees keys up to len - rows +
  // that; a tile has 128 keys, and 256 p is a multiple of 128, which leaves (x + 2 p) / G
  // (groups so wide and sequences so long that x would not fit count every tile for every pair)
  const long long x = (static_cast<long long>(d.s.len - d.s.rows) * p.G + 255) / 128;
  d.linear = p.causal && d.s.len >= d.s.rows && x < (1 << 30);
  d.x = d.linear ? static_cast<int>(x) : 0;
  return d;
}
FA_HD long long prefill_per(long long total) {
  return divide(total + kPreCtas - 1, kPreCtas);  // down to one step: 32 tokens over 2048 keys 26 us, at least two 28 us
}
// Unit `off` of a sequence: head, pair and unit of the item.
struct PrefillAt {
  int h, p, unit;
};
template <typename F>
FA_HD PrefillAt prefill_at(const PrefillSeq& d, long long off, const F& find) {
  PrefillAt a;
  const long long head = d.head_units();
  a.h = static_cast<int>(divide(off, head));
  const long long r = off - a.h * head;
  a.p = find(d, r);
  a.unit = static_cast<int>(r - d.before(a.p));
  return a;
}
// The last pair that begins at unit r of a head or before: by halving, and by a warp's lanes together.
struct FindPairAlone {
  FA_HD int operator()(const PrefillSeq& d, long long r) const {
    int lo = 0, hi = d.pairs - 1;
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (d.before(mid) <= r) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};
struct FindPairWarp {
  __device__ __forceinline__ int operator()(const PrefillSeq& d, long long r) const {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = d.pairs;  // in [lo, lo + n)
    while (n > 1) {
      const int step = (n + 31) / 32, p = lo + lane * step;
      const uint32_t yes = __ballot_sync(0xffffffffu, lane * step < n && d.before(p) <= r);  // lane 0's always
      const int last = 31 - __clz(yes);
      n = min(step, n - last * step);
      lo += last * step;
    }
    return lo;
  }
};

struct PrefillShare {
  long long total, per, off;
  int b;
};
// As decode_share, over the units of this kernel.
template <int THREADS>
__device__ __forceinline__ PrefillShare prefill_share(const PrefillParams& p, int index, long long* scratch) {
  constexpr int W = THREADS / 32;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int run = (p.b.B + THREADS - 1) / THREADS;
  const int b0 = min(t * run, p.b.B), b1 = min(b0 + run, p.b.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += prefill_seq(p, b).head_units() * p.b.Hkv;
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
  PrefillShare r;
  r.total = total;
  r.per = prefill_per(total);
  const long long want = r.per * index;
  const long long lo = before + inc - mine;
  if (want >= lo && want < lo + mine) {
    long long at = lo;
    for (int b = b0; b < b1; ++b) {
      const long long u = prefill_seq(p, b).head_units() * p.b.Hkv;
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

// Walks a CTA's share: one segment (steps [t0, t1) of an item) after another.
struct PrefillWalk {
  long long left;  // units
  int b, h, p, u0, t0, t1, n;  // t0, t1: steps; n: the item's steps
  bool whole;
  PrefillSeq d;
  // False when the share holds no tile.
  template <typename F>
  FA_HD bool start(const PrefillParams& prm, const PrefillShare& s, int index, const F& find) {
    left = min(s.per, s.total - s.per * index);
    b = s.b;
    d = prefill_seq(prm, b);
    const PrefillAt a = prefill_at(d, s.off, find);
    h = a.h;
    p = a.p;
    u0 = a.unit;
    cut();
    return t1 > 0 || next(prm);
  }
  FA_HD void cut() {
    n = d.count(p);
    t0 = max(0, u0 - kPreItemCost);
    t1 = max(0, static_cast<int>(min(static_cast<long long>(n + kPreItemCost), u0 + left)) - kPreItemCost);
    whole = t0 == 0 && t1 == n;
  }
  FA_HD bool next(const PrefillParams& prm) {
    do {
      left -= n + kPreItemCost - u0;
      if (left <= 0) return false;
      u0 = 0;
      if (++p == d.pairs) {
        p = 0;
        if (++h == prm.b.Hkv) {
          h = 0;
          do {
            if (++b >= prm.b.B) return false;
            d = prefill_seq(prm, b);
          } while (d.pairs == 0);
        }
      }
      cut();
    } while (t1 == 0);
    return true;
  }
  FA_HD bool split() const { return d.half && p == d.pairs - 1; }
  FA_HD int first() const { return split() ? 2 * t0 : t0; }  // first key tile
  // The first key tile that query tile t does not see within this segment (first(): it sees none of it).
  FA_HD int end(const PrefillParams& prm, int t) const {
    const int rows = d.s.rows * prm.G, row0 = p * kPreRows + (split() ? 0 : t * kTile);
    if (row0 >= rows) return first();
    const int last_row = min(row0 + kTile, rows) - 1;
    const int last = prm.causal ? d.s.len - d.s.rows + last_row / prm.G : d.s.len - 1;
    const int seen = last < 0 ? 0 : min(last / kTile + 1, (d.s.len + kTile - 1) / kTile);
    return max(first(), min(split() ? 2 * t1 : t1, seen));
  }
};

// A segment as the producer publishes it to the other warps.
struct alignas(16) PrefillSegment {
  int row0, rows, len;  // the sequence
  int h, p;             // key/value head, pair of query tiles
  int t0;               // first key tile; below 0: the share is done
  int end[2];           // the first one that each query tile does not see
  int whole;            // the item is whole: results, not parts
  int split;            // one tile of rows: query tile t takes every second key tile from t0 + t
  int step0;            // first step of the item
  int pad;
};
static_assert(sizeof(PrefillSegment) == 48, "segment slots are 48 bytes");

// --------------------------------------------------------------------------------------- kernel
template <int D, bool FP8>
__global__ void __launch_bounds__(384, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const PrefillParams prm) {
  using L = PrefillLayout<D, FP8>;
  constexpr int SK = L::kStagesK, SV = L::kStagesV, TK = L::kKBytes, TV = L::kVBytes;
  extern __shared__ __align__(1024) uint8_t smem[];
  grid_dependency_launch();
  if ((smem_u32(smem) & 1023u) != 0) {  // swizzled tiles need a 1024-byte aligned base
    if (threadIdx.x == 0) {
      atomicCAS(prm.b.status, 0, kSitePrefill | 0x7F);
      prm.plan[blockIdx.x] = CutPlan{};
    }
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 2;
  uint64_t* k_empty = k_full + SK;
  uint64_t* v_full = k_empty + SK;  // V's tile is ready: halves of e4m3 codes, or zeros behind the end
  uint64_t* v_empty = v_full + SV;
  uint64_t* v_land = v_empty + SV;  // V's copies have landed (e4m3: in the staging ring, kRaws of them)
  uint64_t* s_full = v_land + SV;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* drain = o_full + 2;
  uint64_t* raw_empty = drain + 1;
  uint64_t* seg_full = raw_empty + L::kRaws;
  uint64_t* seg_empty = seg_full + L::kSegs;
  PrefillSegment* segs = reinterpret_cast<PrefillSegment*>(smem + L::kSeg);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  int* abort_flag = reinterpret_cast<int*>(smem + L::kMisc + 4);
  long long* scratch = reinterpret_cast<long long*>(smem + L::kMisc + 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const PrefillShare share = prefill_share<384>(prm, blockIdx.x, scratch);
  if (share.b >= prm.b.B) {
    if (threadIdx.x == 0) prm.plan[blockIdx.x] = CutPlan{};
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < SK; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < SV; ++s) {
      mbar_init(&v_full[s], FP8 ? 2 : 1);  // both converting warps, or the one that zeroes
      mbar_init(&v_empty[s], 1);
      mbar_init(&v_land[s], 1);
    }
    for (int i = 0; i < L::kRaws; ++i) mbar_init(&raw_empty[i], 2);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 128);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 128);
      mbar_init(&o_full[t], 1);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < L::kSegs; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 11);  // the MMA thread, warps 2 and 3, eight softmax warps
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Guard g{abort_flag, prm.b.status};
  // The producer walks the share and publishes its segments; the others read them, each in turn.
  int seg_n = 0;
  auto segment = [&](bool& ok, auto whole_warp) -> const PrefillSegment* {  // null: the share is done, or a wait failed
    const int i = seg_n % L::kSegs;
    const uint32_t ph = (seg_n / L::kSegs) & 1;
    ok = decltype(whole_warp)::value ? wait_warp(&seg_full[i], ph, g, kSitePrefill | 15)
                                     : wait(&seg_full[i], ph, g, kSitePrefill | 15);
    return !ok || segs[i].t0 < 0 ? nullptr : &segs[i];
  };
  constexpr std::true_type kWarp{};
  constexpr std::false_type kThread{};
  auto segment_done = [&](bool arrives) {  // this thread (or warp) has read all it needs of the segment
    if (arrives) mbar_arrive(&seg_empty[seg_n % L::kSegs]);
    ++seg_n;
  };

  if (warp < 4) {
    regs_to<kPreRegsCtl, L::kLaunchRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------------------------- producer
      // Lane i issues the boxes of a tile's i-th page.
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      PrefillWalk w;
      bool ok = true, more = w.start(prm, share, blockIdx.x, FindPairWarp{});
      if (lane == 0)
        prm.plan[blockIdx.x] = more ? CutPlan{share.per, w.t0, w.n, w.h, w.p * kPreRows,
                                              min(kPreRows, w.d.s.rows * prm.G - w.p * kPreRows), w.d.s.row0}
                                    : CutPlan{};
      const int shift = min(prm.b.page_shift, 7), box_rows = 1 << shift;
      constexpr int kCols = FP8 ? D : 64;
      int kt = 0, kn = 0, vn = 0;  // key tiles since the start, loads issued
      while (ok) {
        const int si = seg_n % L::kSegs;
        if (!(ok = wait_warp(&seg_empty[si], ((seg_n / L::kSegs) & 1) ^ 1, g, kSitePrefill | 16))) break;
        ++seg_n;
        const int end = more ? max(w.end(prm, 0), w.end(prm, 1)) : 0;
        if (lane == 0) {
          PrefillSegment& x = segs[si];
          x.row0 = w.d.s.row0;
          x.rows = w.d.s.rows;
          x.len = w.d.s.len;
          x.h = w.h;
          x.p = w.p;
          x.t0 = more ? w.first() : -1;
          x.split = w.split();
          x.step0 = w.t0;
          x.end[0] = w.end(prm, 0);
          x.end[1] = w.end(prm, 1);
          x.whole = w.whole;
          mbar_arrive(&seg_full[si]);
        }
        if (!more) break;
        // the segment's rows of Q on their way to L2: they are read when the segment before has ended
        for (int r = lane; r < kPreRows; r += 32) {
          const int row = w.p * kPreRows + r, token = row / prm.G;
          if (token >= w.d.s.rows) break;
          const __nv_bfloat16* q =
              prm.Q + static_cast<size_t>(w.d.s.row0 + token) * prm.ldq + (w.h * prm.G + row % prm.G) * D;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
          if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
        }
        __syncwarp();
        for (int j = w.first(); j < end && ok; ++j, ++kt) {
          const int keys = min(kTile, w.d.s.len - j * kTile);
          const int boxes = (keys + box_rows - 1) >> shift;
          int z = 0, y = 0;
          float4 sc = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
          if (lane < boxes) {
            const int key = j * kTile + (lane << shift);
            const int page = load_page(prm.b, w.b, key >> prm.b.page_shift);
            // a page out of range reads as zeros beyond the map's last head
            z = page >= 0 ? page * prm.b.Hkv + w.h : prm.b.num_pages * prm.b.Hkv;
            y = key & ((1 << prm.b.page_shift) - 1);
            if (FP8 && page >= 0) sc = page_scales(prm.Ks[z], prm.Vs[z]);
          }
          constexpr int kSize = FP8 ? 1 : 2, VR = FP8 ? L::kRaws : SV;
          const int sk = kt % SK, sv = kt % VR, bytes = boxes * box_rows * D * kSize;
          if (!(ok = wait_warp(&k_empty[sk], ((kt / SK) & 1) ^ 1, g, kSitePrefill | 1))) break;
          if (FP8 && lane < (kTile >> shift)) {
            // the scales of the page's groups of 16 keys (neutral ones behind the last page); of the eight slots
            // the one written here was last read for tile kt - 8, and the S of tile kt - SK that freed the stage
            // came after that
            float4* m = reinterpret_cast<float4*>(smem + L::kMeta) + (kt & 7) * 8 + (lane << (shift - 4));
            for (int i = 0; i < 1 << (shift - 4); ++i) m[i] = sc;
          }
          __syncwarp();
          if (lane == 0) mbar_expect_tx(&k_full[sk], bytes);
          __syncwarp();
          const int at = lane * box_rows * kCols * kSize;
          if (lane < boxes)
            for (int c = 0; c < D / kCols; ++c)
              tma_load_3d(smem + L::kK + sk * TK + c * 16384 + at, &tmK, c * kCols, y, z, &k_full[sk]);
          ++kn;
          if (!(ok = wait_warp(FP8 ? &raw_empty[sv] : &v_empty[sv], ((kt / VR) & 1) ^ 1, g, kSitePrefill | 2))) break;
          if (lane == 0) mbar_expect_tx(&v_land[sv], bytes);
          __syncwarp();
          if (lane < boxes)
            for (int c = 0; c < D / kCols; ++c)
              tma_load_3d(smem + (FP8 ? L::kRaw + sv * L::kRawBytes : L::kV + sv * TV) + c * 16384 + at, &tmV, c * kCols,
                          y, z, &v_land[sv]);
          ++vn;
        }
        if (ok) more = w.next(prm);
      }
      if (!ok) {  // let copies already in flight land before the CTA exits
        constexpr int VR = FP8 ? L::kRaws : SV;
        for (int i = max(kn - SK, 0); i < kn; ++i) drain_wait(&k_full[i % SK], (i / SK) & 1);
        for (int i = max(vn - VR, 0); i < vn; ++i) drain_wait(&v_land[i % VR], (i / VR) & 1);
      }
    } else if (warp == 1) {
      // --------------------------------------------------------------------------------- MMA
      // One thread issues every UMMA, in the order of the contiguous forward.
      if (lane == 0) {
        constexpr uint32_t idS = FP8 ? idesc_e4m3_f32(128, 128) : idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t idO = FP8 ? idesc_f16_f32(128, D, false, true) : idesc_bf16_f32(128, D, false, true);
        const uint32_t sQ = smem_u32(smem + L::kQ), sK = smem_u32(smem + L::kK), sV = smem_u32(smem + L::kV);
        auto issue_s = [&](int t, int s) {
          if constexpr (FP8) {
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk) {
                const uint32_t a = sQ + t * L::kQBytes + part * (kTile * D) + kk * 32, b = sK + s * TK + kk * 32;
                mma_ss_e4m3(tmem + 128 * t, D == 128 ? sdesc_sw128(a, 16, 1024) : sdesc_sw64(a),
                            D == 128 ? sdesc_sw128(b, 16, 1024) : sdesc_sw64(b), idS, part + kk > 0);
              }
          } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
              mma_ss(tmem + 128 * t, sdesc_sw128(sQ + t * L::kQBytes + off, 16, 1024),
                     sdesc_sw128(sK + s * TK + off, 16, 1024), idS, kk > 0);
            }
          }
        };
        auto issue_pv = [&](int t, int s, bool acc) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ts(tmem + 256 + D * t, tmem + 128 * t + 8 * kk, sdesc_sw128(sV + s * TV + kk * 2048, 16384, 1024), idO,
                   (acc || kk > 0) ? 1u : 0u);
        };
        // Per-tile state is kept in bits and selected, not indexed: an indexed array would live in local memory,
        // and every load of it would delay the thread that feeds the tensor core.
        bool ok = true;
        int kt = 0;
        uint32_t q_ph = 0, p_ph = 0;  // bit t: parity of the tile's next q_full, p_full
        while (const PrefillSegment* w = segment(ok, kThread)) {
          const int t0 = w->t0, end0 = w->end[0], end1 = w->end[1];
          const int last = max(end0, end1);
          const bool split = w->split;
          segment_done(true);
          if (last == t0) continue;
          if (split) {
            // key tile i of the segment is query tile (i & 1)'s alone: S two tiles ahead of P V
            const int n = last - t0;
            auto score = [&](int i) {
              const int t = i & 1, s = (kt + i) % SK;
              if (i < 2) {
                if (!(ok = wait(&q_full[t], (q_ph >> t) & 1, g, kSitePrefill | 4))) return;
                q_ph ^= 1u << t;
              }
              if (!(ok = wait(&k_full[s], ((kt + i) / SK) & 1, g, kSitePrefill | 3))) return;
              tc_fence_after();
              issue_s(t, s);
              tc_commit(&s_full[t]);
              tc_commit(&k_empty[s]);
            };
            // a segment of one key tile leaves the second half's Q unused: its barrier still has to turn
            if (n == 1) {
              if (!(ok = wait(&q_full[1], (q_ph >> 1) & 1, g, kSitePrefill | 4))) break;
              q_ph ^= 2u;
            }
            score(0);
            if (ok && n > 1) score(1);
#pragma unroll 1
            for (int i = 0; ok && i < n; ++i) {
              const int t = i & 1, s = (kt + i) % SV;
              if (!(ok = wait(&v_full[s], ((kt + i) / SV) & 1, g, kSitePrefill | 5))) break;
              if (!(ok = wait(&p_full[t], (p_ph >> t) & 1, g, kSitePrefill | 7))) break;
              p_ph ^= 1u << t;
              tc_fence_after();
              issue_pv(t, s, i > 1);
              tc_commit(&o_full[t]);
              tc_commit(&v_empty[s]);
              if (i + 2 < n) score(i + 2);
            }
            if (!ok) break;
            kt += n;
            continue;
          }
          if (!(ok = wait(&k_full[kt % SK], (kt / SK) & 1, g, kSitePrefill | 3))) break;
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (ok && (t ? end1 : end0) > t0) {
              if (!(ok = wait(&q_full[t], (q_ph >> t) & 1, g, kSitePrefill | 4))) break;
              q_ph ^= 1u << t;
              tc_fence_after();
              issue_s(t, kt % SK);
              tc_commit(&s_full[t]);
            }
          if (!ok) break;
          tc_commit(&k_empty[kt % SK]);
          for (int j = t0; j < last; ++j, ++kt) {
            const int s = kt % SV, s1 = (kt + 1) % SK;
            if (!(ok = wait(&v_full[s], (kt / SV) & 1, g, kSitePrefill | 5))) break;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int end = t ? end1 : end0;
              if (!ok || j >= end) continue;
              if (!(ok = wait(&p_full[t], (p_ph >> t) & 1, g, kSitePrefill | 7))) continue;
              p_ph ^= 1u << t;
              tc_fence_after();
              issue_pv(t, s, j > t0);
              tc_commit(&o_full[t]);
              if (j + 1 < end) {
                if (!(ok = wait(&k_full[s1], ((kt + 1) / SK) & 1, g, kSitePrefill | 8))) continue;
                tc_fence_after();
                issue_s(t, s1);
                tc_commit(&s_full[t]);
              }
            }
            if (!ok) break;
            tc_commit(&v_empty[s]);
            if (j + 1 < last) tc_commit(&k_empty[s1]);
          }
          if (!ok) break;
        }
        tc_commit(drain);
        drain_wait(drain, 0);
      }
    } else if constexpr (FP8) {
      // -------------------- V's codes to halves: warp 2 the first 64 keys of a tile, warp 3 the others
      const int first = (warp - 2) * 64;
      bool ok = true;
      int kt = 0;
      while (const PrefillSegment* w = segment(ok, kWarp)) {
        const int t0 = w->t0, end = max(w->end[0], w->end[1]), len = w->len;
        __syncwarp();
        segment_done(lane == 0);
        for (int j = t0; j < end && ok; ++j, ++kt) {
          const int s = kt % SV, rs = kt % L::kRaws;
          if (!(ok = wait_warp(&v_land[rs], (kt / L::kRaws) & 1, g, kSitePrefill | 9))) break;
          if (!(ok = wait_warp(&v_empty[s], ((kt / SV) & 1) ^ 1, g, kSitePrefill | 10))) break;
          const int live = len - j * kTile;  // rows behind it become zeros
          const uint32_t raw = smem_u32(smem + L::kRaw + rs * L::kRawBytes), to = smem_u32(smem + L::kV + s * TV);
          constexpr int CH = D / 16;  // 16-byte chunks of a row of codes
          // eight lanes store rows r and r + 1 (of 4 chunks each): no two to the same bank
#pragma unroll 4
          for (int i = 0; i < 64 * CH / 32; ++i) {
            int r, c;
            if constexpr (D == 128) {
              r = first + (i >> 1) * 8 + (lane >> 2), c = (lane & 3) + 4 * (i & 1);
            } else {
              r = first + i * 8 + (lane >> 2), c = lane & 3;
            }
            uint4 x = lds128(D == 128 ? raw + r * 128 + ((c ^ (r & 7)) << 4) : raw + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
            if (r >= live) x = make_uint4(0u, 0u, 0u, 0u);
            uint32_t h[8];
            halves_of_e4m3(x.x, h[0], h[1]);
            halves_of_e4m3(x.y, h[2], h[3]);
            halves_of_e4m3(x.z, h[4], h[5]);
            halves_of_e4m3(x.w, h[6], h[7]);
            const uint32_t at = to + (c >> 2) * 16384 + r * 128, c2 = 2 * (c & 3);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + (((c2) ^ (r & 7)) << 4)), "r"(h[0]),
                         "r"(h[1]), "r"(h[2]), "r"(h[3])
                         : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + (((c2 + 1) ^ (r & 7)) << 4)), "r"(h[4]),
                         "r"(h[5]), "r"(h[6]), "r"(h[7])
                         : "memory");
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&v_full[s]);
            mbar_arrive(&raw_empty[rs]);
          }
        }
        if (!ok) break;
      }
    } else if (warp == 3) {
      // ------------------------------------------- values behind a sequence's end become zeros
      bool ok = true;
      int kt = 0;
      while (const PrefillSegment* w = segment(ok, kWarp)) {
        const int t0 = w->t0, end = max(w->end[0], w->end[1]), len = w->len;
        __syncwarp();
        segment_done(lane == 0);
        for (int j = t0; j < end && ok; ++j, ++kt) {
          const int live = len - j * kTile, s = kt % SV;
          if (!(ok = wait_warp(&v_land[s], (kt / SV) & 1, g, kSitePrefill | 11))) break;
          if (live < kTile) {
            for (int i = lane; i < (kTile - live) * 8; i += 32)
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                *reinterpret_cast<uint4*>(smem + L::kV + s * TV + c * 16384 + live * 128 + i * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&v_full[s]);
        }
        if (!ok) break;
      }
    }
    if (!FP8 && warp == 2 && lane == 0) {  // takes part in the segments' hand-over only
      bool ok = true;
      while (segment(ok, kThread)) segment_done(true);
    }
  } else {
    regs_to<kPreRegsSoftmax, L::kLaunchRegs>();
    // ------------------------------------------- Q, softmax / correction / epilogue: a thread a row
    const int t = (warp - 4) >> 2;   // query tile
    const int quarter = warp & 3;    // TMEM lanes this warp may touch
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + 128 * t + lane_off;
    const uint32_t tO = tmem + 256 + D * t + lane_off;
    const float4* meta = reinterpret_cast<const float4*>(smem + L::kMeta);
    bool ok = true;
    bool met = false;       // left by the softmax warps' common decision
    int step = 0, kt0 = 0;  // this tile's steps, key tiles of the CTA before the segment
    while (const PrefillSegment* w = segment(ok, kWarp)) {
      const int t0 = w->t0, end = w->end[t], len = w->len;
      const bool split = w->split;
      const int j0 = split ? t0 + t : t0, dj = split ? 2 : 1;  // this tile's key tiles: j0, j0 + dj, ... < end
      // this thread's row of the sequence's rows * G: its token and query head
      const int row0 = w->p * kPreRows + (split ? 0 : t * kTile);
      const int token = (row0 + r) / prm.G, head = (row0 + r) % prm.G + w->h * prm.G;
      const bool real = token < w->rows;
      const int lim = prm.causal && real ? len - w->rows + token : len - 1;  // last visible key
      const int lim_min = prm.causal ? len - w->rows + row0 / prm.G : len - 1;
      float sl2 = prm.scale_log2;
      // Rows go between global and shared memory by the warp, LPR lanes a row, so that a load or store covers
      // whole lines (a thread a row took 32 lines an instruction: 4 us a segment for Q, as much for O).
      constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes of a row, rows of an instruction
      const int chunk = lane % LPR, sub = lane / LPR;
      const uint32_t reals = __ballot_sync(0xffffffffu, real);
      if (end > t0) {
        // the tile's last S is done, since these threads have seen its scores
        const __nv_bfloat16* mine = prm.Q + (real ? static_cast<size_t>(w->row0 + token) * prm.ldq + head * D : 0);
        // four rows at a time, the next four on their way: unrolled over all rows the code, run once a segment,
        // took longer to fetch than to run
        uint4 x[4], ahead[4];
        auto load = [&](uint4(&y)[4], int i0) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int from = (i0 + k) * RPI + sub;
            const auto* q = reinterpret_cast<const __nv_bfloat16*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), from));
            y[k] = (reals >> from) & 1 ? __ldg(reinterpret_cast<const uint4*>(q) + chunk) : make_uint4(0u, 0u, 0u, 0u);
          }
        };
        load(ahead, 0);
#pragma unroll 1
        for (int i0 = 0; i0 < LPR; i0 += 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = ahead[k];
          if (i0 + 4 < LPR) load(ahead, i0 + 4);
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const int i = i0 + k4;
            const int row = quarter * 32 + i * RPI + sub;  // of the tile
            uint8_t* to = smem + L::kQ + t * L::kQBytes;
            if constexpr (FP8) {
              const uint32_t v[4] = {x[k4].x, x[k4].y, x[k4].z, x[k4].w};
              float f[8], amax = 0.0f;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                f[2 * k] = __uint_as_float(v[k] << 16);
                f[2 * k + 1] = __uint_as_float(v[k] & 0xFFFF0000u);
                amax = fmaxf(amax, fmaxf(fabsf(f[2 * k]), fabsf(f[2 * k + 1])));
              }
#pragma unroll
              for (int o = 1; o < LPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
              // q * 256 / (a power of two above the row's largest magnitude) = first part + second part, both e4m3
              const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) + 1, 8), 255);
              const float down = __uint_as_float(static_cast<uint32_t>(262 - e) << 23);
              const int e_row = __shfl_sync(0xffffffffu, e, (lane % RPI) * LPR);  // for the row's own thread
              if (i == lane / RPI) sl2 = prm.scale_log2 * __uint_as_float(static_cast<uint32_t>(e_row - 8) << 23);
              uint32_t part[2][2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int n = 0; n < 4; ++n) f[4 * k + n] *= down;
                part[0][k] = e4m3x2(f[4 * k], f[4 * k + 1]) | (e4m3x2(f[4 * k + 2], f[4 * k + 3]) << 16);
                uint32_t h0, h1;
                halves_of_e4m3(part[0][k], h0, h1);
                const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
                const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
                part[1][k] = e4m3x2(f[4 * k] - a.x, f[4 * k + 1] - a.y) |
                             (e4m3x2(f[4 * k + 2] - b.x, f[4 * k + 3] - b.y) << 16);
              }
              const int c = chunk >> 1;  // 16 bytes are two lanes' eight codes
              to += (D == 128 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ ((row >> 1) & 3)) << 4)) + (chunk & 1) * 8;
              *reinterpret_cast<uint2*>(to) = make_uint2(part[0][0], part[0][1]);
              *reinterpret_cast<uint2*>(to + kTile * D) = make_uint2(part[1][0], part[1][1]);
            } else {
              *reinterpret_cast<uint4*>(to + (chunk >> 3) * 16384 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)) = x[k4];
            }
          }
        }
        fence_proxy_async();
        mbar_arrive(&q_full[t]);
      }
      float m_ref = -INFINITY, l = 0.0f;
      for (int j = j0; j < end; j += dj, ++step) {
        if (!(ok = wait_warp(&s_full[t], step & 1, g, kSitePrefill | 12))) break;
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, sr[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_fence(sr[c]);
#define S(c) __uint_as_float(sr[(c) >> 5][(c) & 31])
        if (j * kTile + kTile - 1 > lim_min) {
#pragma unroll
          for (int c = 0; c < kTile; ++c)
            if (j * kTile + c > lim) sr[c >> 5][c & 31] = __float_as_uint(-INFINITY);
        }
        const float4* mt = meta + ((kt0 + j - t0) & 7) * 8;
        // row maximum (e4m3: of each group of 16 keys, then with the group's scales)
        float top;
        float fg[FP8 ? 8 : 1];  // e4m3: each group's score factor
        bool tiny = false;      // e4m3: a group's value scale needs the boost (page_scales)
        if constexpr (FP8) {
          float mg[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float m0 = fmax3(S(16 * q), S(16 * q + 1), S(16 * q + 2)), m1 = fmax3(S(16 * q + 3), S(16 * q + 4), S(16 * q + 5));
            m0 = fmax3(m0, S(16 * q + 6), S(16 * q + 7));
            m1 = fmax3(m1, S(16 * q + 8), S(16 * q + 9));
            m0 = fmax3(m0, S(16 * q + 10), S(16 * q + 11));
            m1 = fmax3(m1, S(16 * q + 12), S(16 * q + 13));
            m0 = fmax3(m0, S(16 * q + 14), S(16 * q + 15));
            const float4 sc = mt[q];
            fg[q] = fmaxf(sl2 * sc.x, 1e-37f);  // not zero, which a masked score would turn into NaN
            mg[q] = fmaf(fmaxf(m0, m1), fg[q], sc.y);
            tiny |= sc.w > 0.0f;
          }
          top = fmaxf(fmax3(mg[0], mg[1], mg[2]), fmax3(mg[3], mg[4], fmax3(mg[5], mg[6], mg[7])));
        } else {
          float mx[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            mx[q] = S(32 * q);
#pragma unroll
            for (int c = 32 * q + 1; c < 32 * q + 31; c += 2) mx[q] = fmax3(mx[q], S(c), S(c + 1));
            mx[q] = fmaxf(mx[q], S(32 * q + 31));
          }
          top = fmax3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * sl2;
        }
        const float m_new = fmaxf(m_ref, top);
        const bool need = m_new > m_ref + kRescaleTau;
        const float alpha = need ? exp2_sfu(m_ref - m_new) : 1.0f;
        if (need) {
          l = FP8 ? Exp2Pair(m_ref - m_new).times(l) : l * alpha;
          m_ref = m_new;
        }
        const float m_sub = m_ref == -INFINITY ? 0.0f : m_ref;
        float2 ls0 = make_float2(0.f, 0.f), ls1 = make_float2(0.f, 0.f);
        // P, 32 keys -> 16 columns at a time, over S
        auto exp_store = [&](auto tiny_tag) {
          [[maybe_unused]] constexpr bool kTiny = decltype(tiny_tag)::value;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t pk[16];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              float2 c2 = make_float2(sl2, sl2), nm2 = make_float2(-m_sub, -m_sub), gs = make_float2(0.f, 0.f);
              float4 sc = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
              if constexpr (FP8) {
                sc = mt[2 * cc + hh];
                const float n = (kTiny ? sc.y + sc.w : sc.y) - m_sub;
                c2 = make_float2(fg[2 * cc + hh], fg[2 * cc + hh]);
                nm2 = make_float2(n, n);
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int c = 32 * cc + 16 * hh + 2 * e;
                const float2 x = __ffma2_rn(make_float2(S(c), S(c + 1)), c2, nm2);
                float2 p;
                p.x = exp2_sfu(x.x);
                p.y = exp2_sfu(x.y);
                if constexpr (FP8) {
                  gs = __fadd2_rn(gs, p);
                  if (kTiny && sc.w > 0.0f) p.x *= kUnboost, p.y *= kUnboost;
                  pk[8 * hh + e] = pack_half2(p.x, p.y);
                } else {
                  if (e & 1) ls1 = __fadd2_rn(ls1, p);
                  else ls0 = __fadd2_rn(ls0, p);
                  pk[8 * hh + e] = pack_bf16x2(p.x, p.y);
                }
              }
              if constexpr (FP8) ls0 = __ffma2_rn(gs, make_float2(sc.z, sc.z), ls0);
            }
            tmem_st16(tS + 16 * cc, pk);
          }
        };
        if (FP8 && tiny) exp_store(std::true_type{});
        else exp_store(std::false_type{});
#undef S
        const float2 ls = __fadd2_rn(ls0, ls1);
        l += ls.x + ls.y;
        if (j > j0 && __any_sync(0xffffffffu, need)) {
          // O_t *= alpha once the previous P.V has landed (before p_full lets the next one add to it)
          ok = wait_warp(&o_full[t], (step - 1) & 1, g, kSitePrefill | 13);
          tc_fence_after();
          if (ok) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + 32 * c, o);
              tmem_wait_ld();
              reg_fence(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + 32 * c, o);
            }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        if (!ok) break;
        mbar_arrive(&p_full[t]);
      }
      if (ok && j0 < end) ok = wait_warp(&o_full[t], (step - 1) & 1, g, kSitePrefill | 14);
      if (split && end > t0) {
        // the second half's O, m and l through shared memory (the tiles of Q, which no MMA reads any more) into
        // the first half's
        tc_fence_after();
        float4* ring = reinterpret_cast<float4*>(smem + L::kQ + r * (4 * D));
        float2* ml = reinterpret_cast<float2*>(smem + L::kMl);
        if (ok && t == 1 && j0 < end) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
            reg_fence(o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              ring[(8 * c + i) ^ (r & 7)] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                        __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
          }
        }
        if (t == 1) ml[r] = make_float2(m_ref, l);
        if (!(ok = group_and(2, 256, ok))) {
          met = true;
          break;
        }
        if (t == 0 && t0 + 1 < end) {
          const float2 other = ml[r];
          const float m = fmaxf(m_ref, other.x), ms = m == -INFINITY ? 0.0f : m;
          const Exp2Pair pa(m_ref - ms), pb(other.x - ms);
          const float ca = pa.times(1.0f), cb = pb.times(1.0f);
          l = pa.times(l) + pb.times(other.y);
          m_ref = m;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
            reg_fence(o);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 v = ring[(8 * c + i) ^ (r & 7)];
              o[4 * i] = __float_as_uint(__uint_as_float(o[4 * i]) * ca + v.x * cb);
              o[4 * i + 1] = __float_as_uint(__uint_as_float(o[4 * i + 1]) * ca + v.y * cb);
              o[4 * i + 2] = __float_as_uint(__uint_as_float(o[4 * i + 2]) * ca + v.z * cb);
              o[4 * i + 3] = __float_as_uint(__uint_as_float(o[4 * i + 3]) * ca + v.w * cb);
            }
            tmem_st32(tO + 32 * c, o);
          }
          tmem_wait_st();
        }
        named_barrier(2, 256);
      }
      if (!ok) break;
      const bool stores = !(split && t == 1);  // a split item's second half is in the first's
      const size_t at = static_cast<size_t>(w->row0 + token) * prm.Hq + head;
      const bool whole = w->whole;
      const size_t slot = static_cast<size_t>(decode_slot(blockIdx.x, w->step0)) * kPreRows + (split ? 0 : t * kTile) + r;
      if (end > t0 && stores) {
        tc_fence_after();
        const float scale = !whole ? 1.0f : l != 0.0f ? 1.0f / l : 0.0f;
        // rows of W bytes (results in one go, parts, fp32 and twice as wide, in two) through the shared memory that
        // held these same rows of Q: no MMA reads them any more, and no other warp writes there when it goes on
        // to the next segment's
        constexpr int W = 2 * D, RB = FP8 ? D : 128;  // a row of Q: RB bytes in each of W / RB parts
        auto stage = [&](int lr, int k) {
          const int part = k / (RB / 16), kk = k % (RB / 16), x = RB == 128 ? lr & 7 : (lr >> 1) & 3;
          return reinterpret_cast<uint4*>(smem + L::kQ + t * L::kQBytes + part * (kTile * RB) + (quarter * 32 + lr) * RB +
                                          ((kk ^ x) << 4));
        };
        const auto mine = reinterpret_cast<unsigned long long>(whole ? static_cast<void*>(prm.O + at * D)
                                                                     : static_cast<void*>(prm.part_o + slot * D));
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + (D / 2) * half + 32 * c, o);
            tmem_wait_ld();
            reg_fence(o);
            if (whole) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  v[k] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * scale, __uint_as_float(o[8 * i + 2 * k + 1]) * scale);
                const int k = (D / 16) * half + 4 * c + i;
                *stage(lane, k) = make_uint4(v[0], v[1], v[2], v[3]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *stage(lane, 8 * c + i) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          }
          if (whole && half == 0) continue;
          __syncwarp();
#pragma unroll 4
          for (int i = 0; i < LPR; ++i) {
            const int from = i * RPI + sub;
            auto* to = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, mine, from));
            const uint4 v = *stage(from, chunk);
            if ((reals >> from) & 1) *reinterpret_cast<uint4*>(to + (whole ? 0 : half * W) + chunk * 16) = v;
          }
          __syncwarp();
        }
        tc_fence_before();
      } else if (real && whole && stores) {  // no key is visible to any row of the tile
#pragma unroll
        for (int i = 0; i < D / 8; ++i) reinterpret_cast<uint4*>(prm.O + at * D)[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (real && stores) {
        if (whole) prm.LSE[at] = l != 0.0f ? (m_ref + log2f(l)) * 0.69314718055994531f : -INFINITY;
        else prm.part_ml[slot] = make_float2(m_ref, l);  // l = 0: the join takes nothing from this part
      }
      kt0 += max(w->end[0], w->end[1]) - t0;
      __syncwarp();
      segment_done(lane == 0);
    }
    // a warp that leaves on a failed wait of its own still meets those that wait for it in a split segment
    if (!met) group_and(2, 256, ok);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa

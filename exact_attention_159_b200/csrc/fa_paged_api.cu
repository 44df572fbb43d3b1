// fa_paged_api.cu -- host side of the paged key/value cache: argument checks, plans, launches.
// See include/fa.h for the contract of every entry point.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/fa.h"
#include "fa_append.cuh"
#include "fa_host.h"
#include "fa_paged.cuh"
#include "fa_paged_decode.cuh"
#include "fa_paged_join.cuh"
#include "fa_paged_prefill.cuh"

using namespace fa_host;

namespace {

// Short caches (by the block table's width) are not cut along the keys: each CTA takes whole items and
// nothing is joined.  A step of 1, 32 and 128 sequences over 512 bf16 keys (8 x 4 heads), whole against cut:
// 9.1 / 9.4, 10.7 / 15.7 and 50 / 53 us; over 1024 keys: 12.7 / 11.1, 26.9 / 31.8 and 93 / 91 us, so twice the
// width where there are many items (from 64 on: between the 8 and the 256 that were measured).
constexpr int kWholeKeys = 512, kWholeItems = 64;

// Sequences of at most this many rows (new tokens x query heads of a key/value head) go to the kernel of few
// rows, longer ones to the tensor-core tiles, whose time hardly depends on the rows up to 128.  24 sequences
// of 4096 keys, 8 x 4 heads, and one of 65536, few rows against tiles: e4m3 at 32 rows 92 / 98 us and 67 / 74
// us, at 48 rows 119 / 98 us and 86 / 74 us; bf16 at 16 rows 83 / 99 us and 59 / 79 us, at 24 rows 94 / 101 us
// and 99 / 80 us.
constexpr int kDecodeMaxRowsBf16 = 16, kDecodeMaxRowsE4m3 = 32;
int decode_max_rows(const fa_paged_cache* c) {
  return c->type == FA_CACHE_E4M3 ? kDecodeMaxRowsE4m3 : kDecodeMaxRowsBf16;
}

struct Sizes {
  size_t cache, scales, table;
};

// Checks shared by both operators; *empty set when there is nothing to do.
int check_paged(const fa_paged_cache* c, const fa_paged_batch* b, int T, int Hq, bool queries, bool* empty, Sizes* z) {
  *empty = false;
  if (!c || !b) return FA_ERR_INVALID_ARG;
  if (c->type != FA_CACHE_BF16 && c->type != FA_CACHE_E4M3) return FA_ERR_INVALID_ARG;
  if (c->num_pages < 0 || c->heads < 0 || b->B < 0 || b->max_pages < 0 || b->max_q < 0 || T < 0 || Hq < 0)
    return FA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return FA_ERR_UNSUPPORTED;
  if (queries && (c->heads == 0 ? Hq != 0 : Hq % c->heads != 0)) return FA_ERR_INVALID_ARG;
  if (T == 0 || b->B == 0 || c->heads == 0 || b->max_q == 0 || (queries && Hq == 0)) {
    *empty = true;
    return FA_OK;
  }
  if (!c->K || !c->V || !b->block_table || !b->cu_q || !b->seq_lens) return FA_ERR_INVALID_ARG;
  if (c->type == FA_CACHE_E4M3 && (!c->K_scale || !c->V_scale)) return FA_ERR_INVALID_ARG;
  if (c->num_pages == 0 || b->max_pages == 0) return FA_ERR_INVALID_ARG;
  if (!aligned16(c->K) || !aligned16(c->V)) return FA_ERR_ALIGNMENT;
  // int lengths, offsets within a row and tensor-map extents stay in range
  if (static_cast<long long>(queries && Hq > c->heads ? Hq : c->heads) * c->d > INT_MAX) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->num_pages) * c->heads > INT_MAX / 2) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(b->max_pages) * c->page_size > INT_MAX / 2) return FA_ERR_UNSUPPORTED;
  z->cache = static_cast<size_t>(c->num_pages) * c->heads * c->page_size * c->d * (c->type == FA_CACHE_BF16 ? 2 : 1);
  z->scales = static_cast<size_t>(c->num_pages) * c->heads * 4;
  z->table = static_cast<size_t>(b->B) * b->max_pages * 4;
  if (overlaps(c->K, z->cache, c->V, z->cache)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

bool meets_batch(const void* p, size_t n, const fa_paged_batch* b, const Sizes& z) {
  return overlaps(p, n, b->block_table, z.table) || overlaps(p, n, b->cu_q, (static_cast<size_t>(b->B) + 1) * 4) ||
         overlaps(p, n, b->seq_lens, static_cast<size_t>(b->B) * 4);
}

// A written range against everything of the cache and the batch.
bool meets(const void* p, size_t n, const fa_paged_cache* c, const fa_paged_batch* b, const Sizes& z) {
  if (overlaps(p, n, c->K, z.cache) || overlaps(p, n, c->V, z.cache)) return true;
  if (c->type == FA_CACHE_E4M3 && (overlaps(p, n, c->K_scale, z.scales) || overlaps(p, n, c->V_scale, z.scales)))
    return true;
  return meets_batch(p, n, b, z);
}

// The ranges that an append writes against one another and the batch's arrays (check_paged has K against V).
bool written_meet(const fa_paged_cache* c, const fa_paged_batch* b, const Sizes& z) {
  if (meets_batch(c->K, z.cache, b, z) || meets_batch(c->V, z.cache, b, z)) return true;
  if (c->type != FA_CACHE_E4M3) return false;
  for (const float* p : {c->K_scale, c->V_scale})
    if (overlaps(p, z.scales, c->K, z.cache) || overlaps(p, z.scales, c->V, z.cache) || meets_batch(p, z.scales, b, z))
      return true;
  return overlaps(c->K_scale, z.scales, c->V_scale, z.scales);
}

size_t rows_bytes(int T, int64_t ld, int heads, int d) {
  return (static_cast<size_t>(T - 1) * ld + static_cast<size_t>(heads) * d) * 2;
}

// Whether T rows of `na` elements, lda apart, may share an element with T rows of `nb`, ldb apart: of equal
// strides (a fused projection's slices) those that lie side by side within a row do not.
bool rows_meet(const void* a, int64_t lda, int64_t na, const void* b, int64_t ldb, int64_t nb, int T) {
  const size_t sa = (static_cast<size_t>(T - 1) * lda + na) * 2, sb = (static_cast<size_t>(T - 1) * ldb + nb) * 2;
  if (!overlaps(a, sa, b, sb)) return false;
  if (lda != ldb) return true;
  const int64_t apart = (static_cast<int64_t>(reinterpret_cast<uintptr_t>(b)) -
                         static_cast<int64_t>(reinterpret_cast<uintptr_t>(a))) / 2 % lda;  // both 16-byte aligned
  const int64_t off = apart < 0 ? apart + lda : apart;
  return off < na || off + nb > lda;
}

int shift_of(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }

fa::PagedBatch device_batch(const fa_paged_cache* c, const fa_paged_batch* b, int T, int* status) {
  fa::PagedBatch p;
  p.table = b->block_table;
  p.cu_q = b->cu_q;
  p.lens = b->seq_lens;
  p.B = b->B;
  p.T = T;
  p.max_q = b->max_q;
  p.max_pages = b->max_pages;
  p.num_pages = c->num_pages;
  p.page_shift = shift_of(c->page_size);
  p.Hkv = c->heads;
  p.status = status;
  return p;
}

// 3-D map over the pages [num_pages * heads, page_size, d]: box of a row's 128 bytes (64 when a whole row
// is 64 bytes) x `rows` slots, swizzled by the box's width.
bool make_page_map(CUtensorMap* map, const void* base, const fa_paged_cache* c, int rows) {
  const bool fp8 = c->type == FA_CACHE_E4M3;
  const MapKey key{base, c->num_pages * c->heads, c->page_size, c->d, rows, kMapPages + (fp8 ? 1 : 0)};
  if (map_lookup(key, map)) return true;
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t size = fp8 ? 1 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(c->page_size),
                              static_cast<cuuint64_t>(c->num_pages) * c->heads};
  const cuuint64_t strides[2] = {c->d * size, static_cast<cuuint64_t>(c->page_size) * c->d * size};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(fp8 ? c->d : 64), static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  if (fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
         fp8 && c->d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  map_store(key, *map);
  return true;
}

template <int D, bool FP8, int THREADS, int CL>
int launch_append_blocks(fa::AppendParams prm, long long units, int subs, cudaStream_t st) {
  prm.subs = subs;
  if (units * subs > INT_MAX) return FA_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * subs));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = CL;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = CL > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fa::append_kernel<D, FP8, THREADS, CL>, prm) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
// units: pages x key/value heads; most: new tokens of a sequence, at most.
template <int D, bool FP8>
int launch_append(const fa::AppendParams& prm, long long units, int most, cudaStream_t st) {
  constexpr int N = fa::kAppendThreads, VPR = D / 8;
  const int rows = most < (1 << prm.b.page_shift) ? most : 1 << prm.b.page_shift;  // new tokens that a page can get
  if (rows <= 32 / VPR) return launch_append_blocks<D, FP8, 32, 1>(prm, units, 1, st);
  const int subs = (rows + N / VPR - 1) / (N / VPR);
  if constexpr (!FP8) {
    return launch_append_blocks<D, FP8, N, 1>(prm, units, subs, st);
  } else {
    constexpr int kMost = 128 / (N / VPR);  // blocks of the longest page: 8, or 4 at D = 64
    if (subs == 1) return launch_append_blocks<D, FP8, N, 1>(prm, units, 1, st);
    if (subs == 2) return launch_append_blocks<D, FP8, N, 2>(prm, units, 2, st);
    if (subs <= 4) return launch_append_blocks<D, FP8, N, 4>(prm, units, 4, st);
    return launch_append_blocks<D, FP8, N, kMost>(prm, units, kMost, st);
  }
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
struct PagedWs {
  size_t dec_plan, dec_o, dec_ml, pre_plan, pre_o, pre_ml, total;
};
// The kernel of many rows has its parts only where a sequence may have as many.
PagedWs paged_ws(int d, bool many) {
  PagedWs w;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  };
  const size_t dec = static_cast<size_t>(2) * fa::kDecCtas * fa::kDecRows;
  const size_t pre = many ? static_cast<size_t>(2) * fa::kPreCtas * fa::kPreRows : 0;
  w.dec_plan = take(fa::kDecCtas * sizeof(fa::CutPlan));
  w.dec_o = take(dec * d * 4);
  w.dec_ml = take(dec * 8);
  w.pre_plan = take(fa::kPreCtas * sizeof(fa::CutPlan));
  w.pre_o = take(pre * d * 4);
  w.pre_ml = take(pre * 8);
  w.total = at;
  return w;
}
bool many_rows(const fa_paged_cache* c, const fa_paged_batch* b, int T, int G) {
  return static_cast<long long>(b->max_q < T ? b->max_q : T) * G > decode_max_rows(c);
}
bool whole_items(const fa_paged_cache* c, const fa_paged_batch* b) {
  const long long keys = static_cast<long long>(b->max_pages) * c->page_size;
  return keys <= (static_cast<long long>(b->B) * c->heads >= kWholeItems ? 2 * kWholeKeys : kWholeKeys);
}

struct FwdMaps {
  CUtensorMap dec_k, dec_v, pre_k, pre_v;
};

// A launch that may be scheduled while the stream's kernel before it still runs.
template <typename... P>
bool launch_overlapped(void (*kern)(P...), int grid, int threads, int smem, cudaStream_t st, const P&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

template <int D, bool FP8, int NT>
int launch_fwd_paged(const FwdMaps& m, const fa::DecodeParams& dec, const fa::PrefillParams& pre, bool many,
                     cudaStream_t st) {
  using LD = fa::DecodeLayout<D, FP8>;
  using LP = fa::PrefillLayout<D, FP8>;
  auto dkern = fa::decode_kernel<D, FP8, NT>;
  auto pkern = fa::prefill_kernel<D, FP8>;
  if (set_smem(dkern, LD::kBytes) != cudaSuccess) return FA_ERR_CUDA;
  if (many) {
    if (set_smem(pkern, LP::kBytes) != cudaSuccess) return FA_ERR_CUDA;
    pkern<<<fa::kPreCtas, LP::kThreads, LP::kBytes, st>>>(m.pre_k, m.pre_v, pre);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    // the two share no data: the few rows' blocks fill SMs as the many rows' ones leave them
    if (!launch_overlapped(dkern, fa::kDecCtas, fa::kDecThreads, LD::kBytes, st, m.dec_k, m.dec_v, dec)) return FA_ERR_CUDA;
  } else {
    dkern<<<fa::kDecCtas, fa::kDecThreads, LD::kBytes, st>>>(m.dec_k, m.dec_v, dec);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  }
  const int dec_cuts = dec.whole ? 0 : fa::kDecCtas - 1, pre_cuts = many ? fa::kPreCtas - 1 : 0;
  if (dec_cuts + pre_cuts == 0) return FA_OK;
  return launch_overlapped(fa::join_kernel<D>, dec_cuts * dec.rows + pre_cuts * fa::kJoinPreSplit, fa::kJoinThreads, 0,
                           st, dec, pre, dec_cuts + 1)
             ? FA_OK
             : FA_ERR_CUDA;
}
template <int NT>
int launch_fwd_paged_type(int d, bool fp8, const FwdMaps& m, const fa::DecodeParams& dec, const fa::PrefillParams& pre,
                          bool many, cudaStream_t st) {
  if (d == 128)
    return fp8 ? launch_fwd_paged<128, true, NT>(m, dec, pre, many, st)
               : launch_fwd_paged<128, false, NT>(m, dec, pre, many, st);
  return fp8 ? launch_fwd_paged<64, true, NT>(m, dec, pre, many, st)
             : launch_fwd_paged<64, false, NT>(m, dec, pre, many, st);
}

}  // namespace

extern "C" {

int fa_cache_append(const fa_paged_cache* cache, const fa_paged_batch* batch, int T, const void* K, int64_t ldk,
                    const void* V, int64_t ldv, const void* Q, int64_t ldq, void* Q_out, int64_t ldqo, int Hq,
                    const float* cosine, const float* sine, int rot_dim, int interleaved, int n_pos, void* stream) {
  bool empty = false;
  Sizes z;
  int rc = check_paged(cache, batch, T, Hq, Q != nullptr && Hq > 0, &empty, &z);
  if (rc != FA_OK) return rc;
  if (rot_dim < 0 || n_pos < 0 || (interleaved != 0 && interleaved != 1)) return FA_ERR_INVALID_ARG;
  if (rot_dim > cache->d || rot_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
  if ((Q == nullptr) != (Q_out == nullptr) || (Q ? rot_dim == 0 : Hq != 0)) return FA_ERR_INVALID_ARG;
  if (empty) return FA_OK;
  if (Hq == 0) Q = Q_out = nullptr;  // no head to turn, but keys and values to append
  if (!K || !V || (rot_dim > 0 && (!cosine || !sine))) return FA_ERR_INVALID_ARG;
  const int Hkv = cache->heads, d = cache->d;
  const int64_t kv_row = static_cast<int64_t>(Hkv) * d, q_row = static_cast<int64_t>(Hq) * d;
  if (ldk < kv_row || ldv < kv_row || (Q && (ldq < q_row || ldqo < q_row))) return FA_ERR_INVALID_ARG;
  if (ldk % 8 || ldv % 8 || (Q && (ldq % 8 || ldqo % 8))) return FA_ERR_ALIGNMENT;
  for (const void* p : {K, V, Q, static_cast<const void*>(Q_out), static_cast<const void*>(rot_dim ? cosine : nullptr),
                        static_cast<const void*>(rot_dim ? sine : nullptr)})
    if (!aligned16(p)) return FA_ERR_ALIGNMENT;
  for (const int64_t ld : {ldk, ldv, Q ? ldq : 0, Q ? ldqo : 0})
    if (ld > (1LL << 40) / T) return FA_ERR_UNSUPPORTED;
  const size_t kb = rows_bytes(T, ldk, Hkv, d), vb = rows_bytes(T, ldv, Hkv, d);
  const size_t tb = static_cast<size_t>(n_pos) * (rot_dim / 2) * 4;
  if (written_meet(cache, batch, z) || meets(K, kb, cache, batch, z) || meets(V, vb, cache, batch, z))
    return FA_ERR_INVALID_ARG;
  if (Q) {
    const size_t qb = rows_bytes(T, ldq, Hq, d), ob = rows_bytes(T, ldqo, Hq, d);
    if (meets(Q, qb, cache, batch, z) || meets(Q_out, ob, cache, batch, z)) return FA_ERR_INVALID_ARG;
    // in place the rows of a fused projection lie between K's and V's, and only Q's own elements are written
    if (Q_out == Q && ldqo == ldq &&
        (rows_meet(Q, ldq, q_row, K, ldk, kv_row, T) || rows_meet(Q, ldq, q_row, V, ldv, kv_row, T)))
      return FA_ERR_INVALID_ARG;
    if (!(Q_out == Q && ldqo == ldq) &&
        (overlaps(Q_out, ob, Q, qb) || overlaps(Q_out, ob, K, kb) || overlaps(Q_out, ob, V, vb)))
      return FA_ERR_INVALID_ARG;
    if (overlaps(Q_out, ob, cosine, tb) || overlaps(Q_out, ob, sine, tb)) return FA_ERR_INVALID_ARG;
  }
  if (rot_dim && (meets(cosine, tb, cache, batch, z) || meets(sine, tb, cache, batch, z))) return FA_ERR_INVALID_ARG;
  int* status = device_status(&rc);
  if (!status) return rc;
  fa::AppendParams prm;
  prm.b = device_batch(cache, batch, T, status);
  prm.K = static_cast<const __nv_bfloat16*>(K);
  prm.V = static_cast<const __nv_bfloat16*>(V);
  prm.Q = static_cast<const __nv_bfloat16*>(Q);
  prm.Qo = static_cast<__nv_bfloat16*>(Q_out);
  prm.ldk = ldk;
  prm.ldv = ldv;
  prm.ldq = ldq;
  prm.ldqo = ldqo;
  prm.cosp = cosine;
  prm.sinp = sine;
  prm.rot = rot_dim;
  prm.interleaved = interleaved;
  prm.n_pos = n_pos;
  prm.Kc = cache->K;
  prm.Vc = cache->V;
  prm.Ks = cache->K_scale;
  prm.Vs = cache->V_scale;
  prm.G = Q ? Hq / Hkv : 0;
  // max_q consecutive slots starting anywhere in a page, no more than the table is wide
  const int most = batch->max_q < T ? batch->max_q : T;
  prm.max_touched = (most + cache->page_size - 2) / cache->page_size + 1;
  if (prm.max_touched > batch->max_pages) prm.max_touched = batch->max_pages;
  const long long units = static_cast<long long>(batch->B) * prm.max_touched * Hkv;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool fp8 = cache->type == FA_CACHE_E4M3;
  if (d == 128) return fp8 ? launch_append<128, true>(prm, units, most, st) : launch_append<128, false>(prm, units, most, st);
  return fp8 ? launch_append<64, true>(prm, units, most, st) : launch_append<64, false>(prm, units, most, st);
}

size_t fa_fwd_paged_workspace_size(const fa_paged_cache* cache, const fa_paged_batch* batch, int T, int Hq) {
  bool empty = false;
  Sizes z;
  if (check_paged(cache, batch, T, Hq, true, &empty, &z) != FA_OK || empty) return 0;
  return paged_ws(cache->d, many_rows(cache, batch, T, Hq / cache->heads)).total;
}

int fa_fwd_paged(const void* Q, int64_t ldq, const fa_paged_cache* cache, const fa_paged_batch* batch, int T, void* O,
                 float* LSE, void* workspace, size_t workspace_bytes, int Hq, float scale, int causal, void* stream) {
  bool empty = false;
  Sizes z;
  int rc = check_paged(cache, batch, T, Hq, true, &empty, &z);
  if (rc != FA_OK) return rc;
  if ((causal != 0 && causal != 1) || !(scale > 0.0f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (empty) return FA_OK;
  if (!Q || !O || !LSE || !workspace) return FA_ERR_INVALID_ARG;
  if (ldq < static_cast<int64_t>(Hq) * cache->d) return FA_ERR_INVALID_ARG;
  if (ldq % 8 || !aligned16(Q) || !aligned16(O) || !aligned16(LSE) || !aligned16(workspace)) return FA_ERR_ALIGNMENT;
  if (ldq > (1LL << 40) / T || static_cast<long long>(T) * Hq > INT_MAX) return FA_ERR_UNSUPPORTED;
  const int G = Hq / cache->heads;
  const bool many = many_rows(cache, batch, T, G);
  const PagedWs ws = paged_ws(cache->d, many);
  if (workspace_bytes < ws.total) return FA_ERR_INVALID_ARG;
  const size_t qb = rows_bytes(T, ldq, Hq, cache->d), ob = static_cast<size_t>(T) * Hq * cache->d * 2;
  const size_t lb = static_cast<size_t>(T) * Hq * 4;
  const void* outs[3] = {O, LSE, workspace};
  const size_t osz[3] = {ob, lb, ws.total};
  for (int i = 0; i < 3; ++i) {
    if (meets(outs[i], osz[i], cache, batch, z) || overlaps(outs[i], osz[i], Q, qb)) return FA_ERR_INVALID_ARG;
    for (int j = i + 1; j < 3; ++j)
      if (overlaps(outs[i], osz[i], outs[j], osz[j])) return FA_ERR_INVALID_ARG;
  }
  int* status = device_status(&rc);
  if (!status) return rc;
  const bool fp8 = cache->type == FA_CACHE_E4M3;
  const int tile = fp8 ? fa::DecodeLayout<128, true>::kTile : fa::DecodeLayout<128, false>::kTile;
  FwdMaps m;
  const int box = cache->page_size < tile ? cache->page_size : tile;
  if (!make_page_map(&m.dec_k, cache->K, cache, box) || !make_page_map(&m.dec_v, cache->V, cache, box) ||
      (many && (!make_page_map(&m.pre_k, cache->K, cache, cache->page_size) || !make_page_map(&m.pre_v, cache->V, cache, cache->page_size))))
    return FA_ERR_CUDA;
  uint8_t* wsb = static_cast<uint8_t*>(workspace);
  fa::DecodeParams dec;
  dec.b = device_batch(cache, batch, T, status);
  dec.Q = static_cast<const __nv_bfloat16*>(Q);
  dec.ldq = ldq;
  dec.O = static_cast<__nv_bfloat16*>(O);
  dec.LSE = LSE;
  dec.Ks = cache->K_scale;
  dec.Vs = cache->V_scale;
  dec.plan = reinterpret_cast<fa::CutPlan*>(wsb + ws.dec_plan);
  dec.part_o = reinterpret_cast<float*>(wsb + ws.dec_o);
  dec.part_ml = reinterpret_cast<float2*>(wsb + ws.dec_ml);
  dec.G = G;
  dec.Hq = Hq;
  dec.tile = tile;
  // eight rows an item where single tokens fit them and are most of what comes; sixteen for a few tokens
  dec.rows = G <= 8 && (many || static_cast<long long>(batch->max_q) * G <= 8) ? 8 : 16;
  dec.max_rows = decode_max_rows(cache);
  dec.causal = causal;
  dec.whole = whole_items(cache, batch) ? 1 : 0;
  dec.scale_log2 = scale * 1.4426950408889634f;
  fa::PrefillParams pre;
  pre.b = dec.b;
  pre.Q = dec.Q;
  pre.ldq = ldq;
  pre.O = dec.O;
  pre.LSE = LSE;
  pre.Ks = dec.Ks;
  pre.Vs = dec.Vs;
  pre.plan = reinterpret_cast<fa::CutPlan*>(wsb + ws.pre_plan);
  pre.part_o = reinterpret_cast<float*>(wsb + ws.pre_o);
  pre.part_ml = reinterpret_cast<float2*>(wsb + ws.pre_ml);
  pre.G = G;
  pre.Hq = Hq;
  pre.min_rows = decode_max_rows(cache);
  pre.causal = causal;
  pre.scale_log2 = dec.scale_log2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dec.rows == 8 ? launch_fwd_paged_type<1>(cache->d, fp8, m, dec, pre, many, st)
                       : launch_fwd_paged_type<2>(cache->d, fp8, m, dec, pre, many, st);
}

}  // extern "C"

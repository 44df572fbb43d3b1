// fa_host.h -- host-side pieces that the library's translation units share (defined in fa_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <cstdint>

namespace fa_host {

constexpr int kMaxDevices = 64;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Status word of the current device (set up once per device); null with *err_out set on failure.
int* device_status(int* err_out);

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// Encoded tensor maps of recent calls, keyed by (address, extents, box, element kind): callers that
// reuse their buffers (training loops, graph replays, the ring steps, a cache) skip cuTensorMapEncodeTiled.
// A map holds only the address and geometry it was encoded from, so a hit is exactly the map a
// fresh encode would produce.  Small, round-robin replacement, one lock for the operands' maps and one for the pages'.
constexpr int kMapPages = 2;  // kinds from here on are cache pages
struct MapKey {
  const void* base;
  // kind 0: bf16 operand, 1: fp32 dQ accumulator, 2 / 3: bf16 / e4m3 cache pages (BH pages * heads, N = page size)
  int BH, N, d, rows, kind;
  bool operator==(const MapKey& o) const {
    return base == o.base && BH == o.BH && N == o.N && d == o.d && rows == o.rows && kind == o.kind;
  }
};
bool map_lookup(const MapKey& k, CUtensorMap* out);
void map_store(const MapKey& k, const CUtensorMap& m);

// Sets a kernel's dynamic shared memory limit, once per (kernel, device).
cudaError_t set_smem_limit(const void* kernel, int bytes);
template <typename K>
cudaError_t set_smem(K kernel, int bytes) {
  return set_smem_limit(reinterpret_cast<const void*>(kernel), bytes);
}

}  // namespace fa_host

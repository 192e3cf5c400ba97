// What the paged-cache kernels share: the cache as a kernel sees it, the
// checks a kernel makes because lengths and page tables live on the device,
// and the host checks of an rkv_paged_cache.
#pragma once

#include <atomic>
#include <initializer_list>

#include "common.cuh"

namespace rkv {
namespace paged {

constexpr int kHD = 128;                  // head dim
constexpr uint32_t kRowBytes = kHD * 2;   // one token of one key head: the unit rows are counted in
constexpr int64_t kMaxSpan = int64_t(1) << 58;   // elements from a tensor's first row to its last: bytes stay within 64 bits

struct CacheDev {
  uint8_t* k;
  uint8_t* v;
  const int32_t* table;
  int64_t table_stride;
  int32_t* status;
  uint32_t page_units;   // head rows (of kRowBytes) between pages
  uint32_t n_pages;
  uint32_t P;            // tokens per page
  FastDiv div_P;
  int32_t H, n_seqs, capacity;
};

// Where a device-side finding was made (status word: RKV_ERR_DEVICE_CHECK in
// the low byte, this above it).
enum : int { kBadLength = 1, kBadPage = 2 };

__device__ __forceinline__ void record(const CacheDev& c, int what) {
  if (c.status) atomicCAS(c.status, 0, int(RKV_ERR_DEVICE_CHECK) | (what << 8));
}

// Length of sequence s, brought into [0, capacity].
__device__ __forceinline__ int seq_len(const CacheDev& c, const int32_t* seq_lens, int s) {
  const int L = seq_lens[s];
  if (L < 0 || L > c.capacity) {
    record(c, kBadLength);
    return L < 0 ? 0 : c.capacity;
  }
  return L;
}

// Page of token j of sequence s (j < capacity), and the head row of (page,
// token, head h) counted from the start of the pool (below 2^32, checked on
// the host).
__device__ __forceinline__ uint32_t page_of(const CacheDev& c, int s, uint32_t j) {
  return uint32_t(c.table[int64_t(s) * c.table_stride + fdiv(j, c.div_P)]);
}
__device__ __forceinline__ uint32_t row_unit(const CacheDev& c, uint32_t page, uint32_t j, int h) {
  const uint32_t tok = j - fdiv(j, c.div_P) * c.P;
  return page * c.page_units + tok * uint32_t(c.H) + uint32_t(h);
}

// ---- host -------------------------------------------------------------------------
rkv_status check_cache(const rkv_paged_cache* c);
CacheDev cache_dev(const rkv_paged_cache* c);   // of a checked cache
// Bytes that a call reads or writes: `rows` runs of `width` bytes, `stride`
// bytes apart; p = null: none.
struct Bytes {
  const char* name;
  const void* p;
  int64_t rows, stride, width;
};
inline Bytes run_of(const char* name, const void* p, uint64_t bytes) { return {name, p, 1, int64_t(bytes), int64_t(bytes)}; }
Bytes pool_k(const rkv_paged_cache* c);
Bytes pool_v(const rkv_paged_cache* c);
Bytes table_of(const rkv_paged_cache* c);
Bytes status_of(const rkv_paged_cache* c);
// What a call writes shares no byte with anything else it writes or reads.
rkv_status check_apart(std::initializer_list<Bytes> writes, std::initializer_list<Bytes> reads);
int sm_count();

// Allow kernel kKern `bytes` of dynamic shared memory on the current device:
// once per device, since the call takes as long as a small launch.
template <auto kKern>
inline cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};   // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kKern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launch that may overlap the end of the stream's previous launch (the kernel
// waits for it before it reads anything), as clusters of `cluster` blocks.
template <class Args>
inline cudaError_t launch_overlapped(void (*kern)(Args), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                     const Args& args, int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = uint32_t(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(uint32_t(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline int64_t capacity(const rkv_paged_cache* c) { return int64_t(c->max_pages) * c->page_tokens; }

}  // namespace paged
}  // namespace rkv

// Launch parameters of the 8-bit cache's kernels (host and device side).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "kv8.cuh"

namespace tq {

// Allows kernel k `smem` bytes of dynamic shared memory, once a device (seen: bit of each device).
template <typename K>
cudaError_t allow_smem(K* k, int smem, std::atomic<uint64_t>& seen) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (seen.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) seen.fetch_or(bit, std::memory_order_release);
  return e;
}

struct Kv8AppendParams {
  const void* x[2];                                   // new keys, new values
  int64_t stride_b[2], stride_h[2], stride_t[2];      // elements
  int dtype, B, T, blocks;                            // blocks: that T new tokens can touch
  const int32_t* kv_lens;
  const int32_t* new_lens;                            // or nullptr: T
  bool empty_ok;                                      // a sequence of no tokens brings none (decode steps)
  uint8_t* codes[2];
  float* scales[2];
  Kv8Map map;
  int* status;
};
cudaError_t launch_kv8_append(const Kv8AppendParams& p, int d, cudaStream_t s);

// Attention of B sequences whose query heads share Hkv key heads; rows of a key head are its
// T * G queries (r = i * G + g), G = Hq / Hkv.
struct Kv8AttnParams {
  const void* q;
  int64_t q_stride_b, q_stride_h, q_stride_t;         // elements
  int dtype, Hq, G, T;
  // the launch works on virtual sequences v0 .. v0 + VB - 1; sequence v / RG, row group v % RG
  int v0, VB, RG;
  const float* kscales;
  const float* vscales;
  Kv8Scoring sc;
  Kv8Map map;
  void* out;                                          // [B][Hq][T][d], dtype
  float* lse;                                         // [B][Hq][T] or nullptr
  float* part_o;                                      // partial results of split rows
  float* part_lse;
  int* plan;                                          // where the launch's work is split
  int* status;
  long long wait_limit;
  int run_cost;                                       // decode: see plan_attn
  bool appended;                                      // behind an append of the same call
};
// Groups of 16 rows a key head (decode; fp32 queries).  kmap / vmap: the codes as [records][d]
// bytes in boxes of 16 rows.
constexpr int kKv8DecodeRows = 16;
__host__ __device__ constexpr int kv8_decode_tile(int d) { return d == 64 ? 64 : 32; }       // tokens
constexpr int kKv8DecodeMaxVB = 1024;                 // virtual sequences a launch
// Warps of a CTA.  Their instructions' latency bounds a tile, so as many as the registers allow.
__host__ __device__ constexpr int kv8_decode_warps(int64_t rows, bool f32) { return rows <= 8 && !f32 ? 12 : 8; }
// team: the warps of a CTA share each run, else each has its own.
cudaError_t launch_kv8_decode(const CUtensorMap& kmap, const CUtensorMap& vmap, const Kv8AttnParams& p, int d, bool team,
                              int grid, cudaStream_t s);


// Groups of 256 rows a key head, 16-bit queries (prefill).
constexpr int kKv8PrefillRows = 256;
constexpr int kKv8PrefillMaxVB = 512;
cudaError_t launch_kv8_prefill(const uint8_t* kcodes, const uint8_t* vcodes, const Kv8AttnParams& p, int d, int grid,
                               cudaStream_t s);

}  // namespace tq

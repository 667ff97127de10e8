// Append to the 8-bit block-scaled cache.
//
//   s(x) = min{2^e >= 2^-126 : max|x| <= 448 * 2^e},   code = rn_e4m3(x / s)
//
// over a block of 16 tokens of a head.  Tokens arrive behind those that the cache holds; a
// block that already holds some keeps s' = max(s_old, s(new)) and, where that is larger, its
// old codes are rounded again to it: rn_e4m3(code * s_old / s').  Scales are powers of two so
// that this second rounding is exact except for values that fall below e4m3's normal range; a
// free scale would round every held code anew each time a block grows.
//
// One warp owns one block of one side: it reads the block's new rows once into registers (16
// bytes a lane and load), takes the maximum, converts and stores 8 bytes a lane.  No two warps
// share a block, so nothing is synchronised.  Bytes bound it: 2 to 4 in and 1 out an element.
#include <cuda_runtime.h>

#include "kv8.cuh"
#include "kv8_launch.h"
#include "launchers.h"

namespace tq {
namespace {

constexpr int kWarps = 8;

// Biased exponent of the smallest power of two s >= 2^-126 with amax <= 448 s
// (448 = 1.75 * 2^8; amax >= 0).
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, 1);
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Four codes times r, rounded again.
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float r) {
  const uint32_t h0 = e4m3x2_to_h2(w), h1 = e4m3x2_to_h2(w >> 16);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
  return to_e4m3x4(a.x * r, a.y * r, b.x * r, b.y * r);
}

template <int D, int DT>
__global__ void __launch_bounds__(kWarps * 32) kv8_append_kernel(const Kv8AppendParams p) {
  constexpr int LPR = D / 8;          // lanes a row
  constexpr int RPP = 32 / LPR;       // rows a pass
  constexpr int NP = kKv8Block / RPP;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t per_side = static_cast<int64_t>(p.B) * p.map.Hkv * p.blocks;
  const int side = w >= per_side ? 1 : 0;
  w -= side * per_side;
  if (w >= per_side) return;
  const int j = static_cast<int>(w % p.blocks);
  const int bh = static_cast<int>(w / p.blocks);
  const int b = bh / p.map.Hkv, h = bh - b * p.map.Hkv;

  const int len = __ldg(p.kv_lens + b);
  const int fresh = p.new_lens ? __ldg(p.new_lens + b) : p.T;
  if (fresh < 0 || fresh > p.T || len < fresh || len > p.map.cap) {
    report_status(p.status, TQ_ERR_INVALID_ARG);
    return;
  }
  const int p0 = len - fresh;                            // first new token
  const int t0 = (p0 / kKv8Block + j) * kKv8Block;       // first token of the block
  if (fresh == 0 || t0 >= len) return;
  const int held = max(0, p0 - t0), end = min(kKv8Block, len - t0);

  const int64_t rec = kv8_record(p.map, b, h, t0, p.status);
  uint8_t* codes = p.codes[side] + rec * D;
  float* scale = p.scales[side] + rec / kKv8Block;

  const int row0 = lane / LPR, col = (lane % LPR) * 8;
  const int64_t base = b * p.stride_b[side] + h * p.stride_h[side] + col;
  float v[NP][8];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int r = k * RPP + row0;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = 0.f;
    if (r >= held && r < end) {
      const int64_t at = base + static_cast<int64_t>(t0 + r - p0) * p.stride_t[side];
      if constexpr (DT == TQ_F32) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p.x[side]) + at);
        const float4 a = __ldg(s), c = __ldg(s + 1);
        v[k][0] = a.x; v[k][1] = a.y; v[k][2] = a.z; v[k][3] = a.w;
        v[k][4] = c.x; v[k][5] = c.y; v[k][6] = c.z; v[k][7] = c.w;
      } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x[side]) + at));
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (DT == TQ_BF16) {
            v[k][2 * i] = __uint_as_float(u[i] << 16);
            v[k][2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
          } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            v[k][2 * i] = f.x;
            v[k][2 * i + 1] = f.y;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[k][i]));
    }
  }
  const int need = scale_exponent(warp_max(amax));
  int e = need;
  if (held) {
    const int old = static_cast<int>((__float_as_uint(*scale) >> 23) & 0xffu);
    e = max(need, old);
    if (need > old) {
      // 2^(old - need); below 2^-126 every held code rounds to 0 either way
      const float r = __uint_as_float(static_cast<uint32_t>(max(127 + old - need, 0)) << 23);
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int row = k * RPP + row0;
        if (row < held) {
          uint2* c = reinterpret_cast<uint2*>(codes + row * D + col);
          const uint2 w2 = *c;
          *c = make_uint2(rescale_e4m3x4(w2.x, r), rescale_e4m3x4(w2.y, r));
        }
      }
    }
  }
  __syncwarp();
  // e is 1..248, so 2^(127 - e) is a normal number and v * inv is exact where it matters
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int r = k * RPP + row0;
    if (r >= held && r < end)
      *reinterpret_cast<uint2*>(codes + r * D + col) =
          make_uint2(to_e4m3x4(v[k][0] * inv, v[k][1] * inv, v[k][2] * inv, v[k][3] * inv),
                     to_e4m3x4(v[k][4] * inv, v[k][5] * inv, v[k][6] * inv, v[k][7] * inv));
  }
  if (lane == 0) *scale = __uint_as_float(static_cast<uint32_t>(e) << 23);
}

template <int D>
cudaError_t go(const Kv8AppendParams& p, unsigned grid, cudaStream_t s) {
  const dim3 g(grid), t(kWarps * 32);
  if (p.dtype == TQ_F32) return launch_pdl(kv8_append_kernel<D, TQ_F32>, g, t, 0, s, p);
  if (p.dtype == TQ_BF16) return launch_pdl(kv8_append_kernel<D, TQ_BF16>, g, t, 0, s, p);
  return launch_pdl(kv8_append_kernel<D, TQ_F16>, g, t, 0, s, p);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendParams& p, int d, cudaStream_t s) {
  const int64_t warps = 2ll * p.B * p.map.Hkv * p.blocks;
  const unsigned grid = static_cast<unsigned>((warps + kWarps - 1) / kWarps);
  return d == 128 ? go<128>(p, grid, s) : go<64>(p, grid, s);
}

}  // namespace tq

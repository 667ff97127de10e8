// Shared pieces of the 8-bit block-scaled cache (append, decode and prefill attention).
//
// A side of the cache (keys or values) is e4m3 codes [records][d] with one fp32 scale, a power
// of two, for each block of 16 records of a head: x^ = code * scale.  Record of token t of
// sequence b and head h: (page * Hkv + h) * page_size + t % page_size, page = block_table[b *
// max_pages + t / page_size]; without a block table page = b and page_size = Nmax, which is the
// contiguous layout [B][Hkv][Nmax].
#pragma once

#include <cuda_fp8.h>

#include "device_common.cuh"

namespace tq {

constexpr int kKv8Block = TQ_KV8_BLOCK;
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Kv8Map {
  const int32_t* table;   // [B][max_pages], or nullptr (contiguous)
  int64_t page;           // page_size, or Nmax
  int max_pages;
  int64_t num_pages;      // pages of the pool, or B
  int Hkv;
  int64_t cap;            // tokens a sequence can hold
};

// Which tokens a query at `pos` sees, and how its scores are formed.
struct Kv8Scoring {
  const int32_t* kv_lens;   // [B]
  const int32_t* q_pos;     // [B][T], or nullptr: the sequence's last token
  const int32_t* first;     // [B][T] or nullptr
  const int32_t* prefix;    // [B] or nullptr
  const float* slopes;      // [Hq] or nullptr
  int window;
  float scale_log2;         // scale * log2(e): scores in powers of two
  float cap;                // 0: none.  scores are cap * tanh(score / cap)
};

// Visible tokens [lo, hi) of query (b, i); hi <= lo: none.  len is already within capacity.
__device__ __forceinline__ void kv8_range(const Kv8Scoring& s, int b, int i, int T, int len, int& lo, int& hi, int& pos) {
  pos = s.q_pos ? __ldg(s.q_pos + static_cast<int64_t>(b) * T + i) : len - 1;
  lo = 0;
  hi = 0;
  if (pos < 0) return;                       // padding
  int64_t end = static_cast<int64_t>(pos) + 1;
  if (s.prefix) end = max(end, static_cast<int64_t>(__ldg(s.prefix + b)));
  hi = static_cast<int>(min(end, static_cast<int64_t>(len)));
  if (s.window > 0) lo = max(lo, pos - s.window + 1);
  if (s.first) lo = max(lo, __ldg(s.first + static_cast<int64_t>(b) * T + i));
}

// Length of sequence b; one outside 0..capacity is reported and read as the nearest bound.
__device__ __forceinline__ int kv8_len(const int32_t* lens, int b, int64_t cap, int* status) {
  const int n = __ldg(lens + b);
  if (n < 0 || n > cap) {
    report_status(status, TQ_ERR_INVALID_ARG);
    return n < 0 ? 0 : static_cast<int>(cap);
  }
  return n;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two floats an instruction.
__device__ __forceinline__ float2 pair(float x, float y) { return make_float2(x, y); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ uint64_t bits2(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 floats2(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return floats2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return floats2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return floats2(r);
}

// tanh from 1 - 2 / (1 + e^2x): absolute error near 2^-22.  A NaN stays one.
__device__ __forceinline__ float kv8_tanh(float x) {
  float e;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(e) : "f"(x * (2.f * kLog2E)), "f"(80.f));
  return 1.f - __fdividef(2.f, 1.f + ex2(e));
}

// Capped scores, out * tanh(z).  A cap may be far above the scores, so the error is kept relative: for
// |z| <= 1/2 the series to z^11, whose next term is below 2^-20 of the result, else kv8_tanh of |z|.
__device__ __forceinline__ float2 kv8_cap_series(float2 z, float out) {
  const float2 u = mul2(z, z), y = mul2(z, both(out));
  float2 q = fma2(u, both(-1382.f / 155925.f), both(62.f / 2835.f));
  q = fma2(u, q, both(-17.f / 315.f));
  q = fma2(u, q, both(2.f / 15.f));
  q = fma2(u, q, both(-1.f / 3.f));
  return fma2(mul2(y, u), q, y);
}
__device__ __forceinline__ float2 kv8_cap(float2 z, float out) {
  const float2 near = kv8_cap_series(z, out);
  return make_float2(fabsf(z.x) <= 0.5f ? near.x : copysignf(out * kv8_tanh(fabsf(z.x)), z.x),
                     fabsf(z.y) <= 0.5f ? near.y : copysignf(out * kv8_tanh(fabsf(z.y)), z.y));
}

// Two e4m3 codes (low 16 bits) as two halves; every e4m3 value is exact in half precision.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

// The line of tiles that a launch cuts into equal runs: virtual sequences v in order, for each its
// key heads, for each the tiles of its visible tokens.
struct Kv8Place {
  int v, h, tile, n;      // virtual sequence, key head, tile and tiles of the sequence
};

// pref[v]: tiles of one key head before virtual sequence v (pref[VB]: all).
__device__ __forceinline__ Kv8Place kv8_place_of(int64_t u, const int* pref, int VB, int Hkv) {
  int lo = 0, hi = VB - 1;
  while (lo < hi) {                       // last v with Hkv * pref[v] <= u
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(pref[mid]) * Hkv <= u) lo = mid; else hi = mid - 1;
  }
  Kv8Place p;
  p.v = lo;
  p.n = pref[lo + 1] - pref[lo];
  const int rem = static_cast<int>(u - static_cast<int64_t>(pref[lo]) * Hkv);
  p.h = p.n ? rem / p.n : 0;
  p.tile = p.n ? rem - p.h * p.n : 0;
  return p;
}

// Counts pref[1 .. VB] to sums (one warp).
__device__ __forceinline__ void kv8_prefix(int* pref, int VB) {
  const int lane = threadIdx.x & 31;
  int run = 0;
  for (int v = 0; v < VB; v += 32) {
    int x = v + lane < VB ? pref[v + lane + 1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (v + lane < VB) pref[v + lane + 1] = run + x;
    run += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) pref[0] = 0;
}

// A part (a CTA's or a warp's) that starts inside a key head's units says so for the kernel that joins:
// plan[c] = {v, h, c0, c1}, the parts that the key head is cut into, if c is the second of them, else
// v = -1.  A key head has `cost` units before its tiles.
__device__ __forceinline__ void kv8_plan_split(int* plan, int c, int64_t u0, int64_t u1, int64_t per, const int* pref, int VB, int Hkv,
                                               int cost) {
  int4 s = make_int4(-1, 0, 0, 0);
  if (u0 < u1 && u0 > 0) {
    const Kv8Place p = kv8_place_of(u0, pref, VB, Hkv);
    const int64_t start = u0 - p.tile;
    s.z = static_cast<int>((start + cost) / per);
    s.w = static_cast<int>((start + p.n - 1) / per);
    if (p.tile > 0 && s.z + 1 == c) {
      s.x = p.v;
      s.y = p.h;
    }
  }
  reinterpret_cast<int4*>(plan)[c] = s;
}

// Tiles [tile, tile + tiles) of the n of key head h of virtual sequence v: what a part does from unit u
// of the line to u1 or to the end of the key head, which has `cost` units before those of its tiles.
struct Kv8Run {
  int v, h, tile, tiles, n, units;
};

__device__ __forceinline__ Kv8Run kv8_run_at(int64_t u, int64_t u1, const int* pref, int VB, int Hkv, int cost) {
  const Kv8Place p = kv8_place_of(u, pref, VB, Hkv);
  Kv8Run r;
  r.v = p.v;
  r.h = p.h;
  r.n = p.n - cost;
  r.units = static_cast<int>(min(u1 - u, static_cast<int64_t>(p.n - p.tile)));
  r.tile = max(0, p.tile - cost);
  r.tiles = max(0, p.tile + r.units - cost) - r.tile;
  return r;
}

// The NaN codes (0x7f, 0xff) of four bytes as 0.
__device__ __forceinline__ uint32_t e4m3_nan_to_zero(uint32_t w) {
  const uint32_t nan = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
  return w & ~(nan * 0xffu);
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {   // a in the low half
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace tq

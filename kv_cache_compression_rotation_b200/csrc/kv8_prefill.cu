// Attention of many query rows a key head over the 8-bit block-scaled cache, on the tensor cores
// with accumulators in tensor memory (16-bit queries).
//
//   S = Q K^T,  l_t = scale s_k(t) S_t (capped, biased),  O = sum_t e^{l_t} v^_t,  out = O / sum
//
// 4 d operations a (row, token) and one exponential bound it: a tile pair of 2 x 128 rows and 128
// tokens at d = 128 takes the tensor core 2048 cycles and the exponentials, 16 a cycle, as many.
//
// A CTA an SM (persistent) takes runs of the line of (256-row group, key head, 128-token tile) as
// the decode kernel does.  Its roles:
//   warps 0-3, 4-7   softmax of row tile 0 and 1, a row a thread: scores from tensor memory,
//                    running maximum and sum, probabilities back into tensor memory as halves
//   warps 8-11       codes to halves: 16 bytes of codes become 32 of a 128-byte-swizzled operand
//                    tile in shared memory; the next tile's codes are already in registers
//   warp 12          the tensor core's issuing thread
// The two row tiles alternate: while one tile's scores are in the softmax, the tensor core works
// for the other.  Tensor memory (512 columns): S 0, S 1 (128 each; the tile's probabilities
// overwrite its scores, two a column), O 0, O 1.  K is a row-major operand, V the same bytes read
// transposed.
//
// A row's reference stays while no score exceeds it by 2^8, so the outputs are seldom rescaled.
// The value scales 2^e of 16-token blocks join the exponent: P = 2^(l - m + 7 + e - E), E the
// largest e of the run, at most 2^15 in halves of 11 bits; row sums are fp32.  q is divided by a
// power of two a row, as in the decode kernel.
#include <cuda_runtime.h>

#include "kv8_launch.h"
#include "launchers.h"
#include "quantize_umma.cuh"

namespace tq {
namespace {

constexpr int kThreads = 13 * 32;
constexpr int kTile = 128;                   // tokens, and rows of a row tile
constexpr int kBlocks = kTile / kKv8Block;
constexpr float kLazy = 8.f;                 // a reference may lag by this many powers of two
constexpr int kHead = 7;                     // P <= 2^(kLazy + kHead)
constexpr int kScaleSlots = 4;               // tiles whose scales are kept: a slot is filled again when the
                                             // first product of the tile two before is done, so none in use
constexpr int kSlot = 2 * kBlocks + 4;       // key scales, exponents of the probabilities, E

struct PrefillSmem {
  uint32_t q, k, v, scales, bars, lo, hi, in_lo, in_hi, pref, misc, total;
};
__host__ __device__ constexpr PrefillSmem prefill_smem(int D) {
  PrefillSmem L{};
  const uint32_t tile = kTile * D * 2;
  uint32_t at = 0;
  L.q = at; at += 2 * tile;
  L.k = at; at += 2 * tile;
  L.v = at; at += 2 * tile;
  L.scales = at; at += kScaleSlots * kSlot * 4;
  L.bars = at; at += 16 * 8;
  L.lo = at; at += kKv8PrefillMaxVB * 4;
  L.hi = at; at += kKv8PrefillMaxVB * 4;
  L.in_lo = at; at += kKv8PrefillMaxVB * 4;
  L.in_hi = at; at += kKv8PrefillMaxVB * 4;
  L.pref = at; at += (kKv8PrefillMaxVB + 4) * 4;
  L.misc = at; at += 64;
  L.total = at + 1024;
  return L;
}
static_assert(prefill_smem(128).total <= 232448, "shared memory");

enum : int { KFULL = 0, KEMPTY = 2, VFULL = 4, VEMPTY = 6, SFULL = 8, PFULL = 10, OFULL = 12, QFULL = 14 };

// Operand tile of 128 rows of D halves: D / 64 parts of [128][64], 16-byte chunks XORed with the
// row within 8.  Byte offset of chunk c (8 halves) of row r.
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  return (c >> 3) * 16384u + r * 128u + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Shared-memory descriptor of an operand whose rows are the contraction (V: tokens): atoms of 64
// columns x 8 rows, the next 64 columns 16 KB on, the next 8 rows 1 KB on, 128-byte swizzle.
__device__ __forceinline__ uint64_t sw128_desc_t(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(16384u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// D f32, A and B f16, M = 128, N = n; tb: B's rows are the contraction.
__device__ __forceinline__ uint32_t idesc_f16(uint32_t n, uint32_t tb) {
  return (1u << 4) | (tb << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void tmem_st32(uint32_t a, const float (&v)[32]) {
  uint32_t r[16];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[16 * h + i]);
    tmem_st16(a + 16 * h, r);
  }
}

// GEN: scores are capped or biased.
template <int D, bool GEN>
__global__ void __launch_bounds__(kThreads, 1)
kv8_prefill_kernel(const uint8_t* __restrict__ kcodes, const uint8_t* __restrict__ vcodes, const Kv8AttnParams p) {
  constexpr PrefillSmem L = prefill_smem(D);
  constexpr uint32_t TB = kTile * D * 2;     // bytes of an operand tile
  extern __shared__ unsigned char psm_raw[];
  const uint32_t raw = smem_u32(psm_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* sm = psm_raw + (base - raw);
  float* s_scale = reinterpret_cast<float*>(sm + L.scales);
  int* s_lo = reinterpret_cast<int*>(sm + L.lo);                // tokens that some row of the group sees
  int* s_hi = reinterpret_cast<int*>(sm + L.hi);
  int* s_in_lo = reinterpret_cast<int*>(sm + L.in_lo);          // tokens that all rows see
  int* s_in_hi = reinterpret_cast<int*>(sm + L.in_hi);
  int* s_pref = reinterpret_cast<int*>(sm + L.pref);
  int* s_e = reinterpret_cast<int*>(sm + L.misc);               // [4] largest value scale that each converting warp saw
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L.misc + 32);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L.misc + 36);
  const uint32_t bar0 = base + L.bars;
  auto bar = [&](int id) { return bar0 + 8u * id; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(KFULL + i), 128);
      mbar_init(bar(KEMPTY + i), 1);
      mbar_init(bar(VFULL + i), 128);
      mbar_init(bar(VEMPTY + i), 1);
      mbar_init(bar(SFULL + i), 1);
      mbar_init(bar(PFULL + i), 128);
      mbar_init(bar(OFULL + i), 1);
      mbar_init(bar(QFULL + i), 128);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  if (warp == 12) {                          // behind the kernel before, which may want tensor memory
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // ---- how the work is cut
  const int VB = p.VB, Hkv = p.map.Hkv, R = p.T * p.G;
  for (int v = warp; v < VB; v += kThreads / 32) {
    const int gv = p.v0 + v, b = gv / p.RG, r0 = (gv - b * p.RG) * kKv8PrefillRows;
    const int len = kv8_len(p.sc.kv_lens, b, p.map.cap, p.status);
    int lo = INT32_MAX, hi = 0, in_lo = 0, in_hi = INT32_MAX;
    const int i1 = min(R - 1, r0 + kKv8PrefillRows - 1) / p.G;
    for (int i = r0 / p.G + lane; i <= i1; i += 32) {
      int a, z, pos;
      kv8_range(p.sc, b, i, p.T, len, a, z, pos);
      if (z > a) { lo = min(lo, a); hi = max(hi, z); }
      in_lo = max(in_lo, a);
      in_hi = min(in_hi, z);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    in_lo = __reduce_max_sync(0xffffffffu, in_lo);
    in_hi = __reduce_min_sync(0xffffffffu, in_hi);
    if (lane == 0) {
      s_lo[v] = hi > 0 ? lo : 0;
      s_hi[v] = hi;
      s_in_lo[v] = in_lo;
      s_in_hi[v] = in_hi;
      s_pref[v + 1] = hi > 0 ? (hi + kTile - 1) / kTile - lo / kTile : 0;
    }
  }
  __syncthreads();
  if (warp == 0) kv8_prefix(s_pref, VB);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int64_t total = static_cast<int64_t>(s_pref[VB]) * Hkv;
  const int64_t per = max((total + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(1));
  if (blockIdx.x == 0) {
    for (int v = tid; v <= VB; v += kThreads) p.plan[kKv8PlanHead + v] = s_pref[v];
    if (tid == 0) *reinterpret_cast<int64_t*>(p.plan) = per;
  }
  pdl_trigger();
  const int64_t u0 = min(total, per * blockIdx.x), u1 = min(total, u0 + per);
  const long long lim = p.wait_limit;

  if (warp < 8) {
    // ================================================================ softmax
    const int rt = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + rt * 128, to = tmem + lanes + 256 + rt * D;
    const uint32_t qa = base + L.q + rt * TB;
    int64_t kt = 0;                          // tiles of the CTA so far
    int own = 0, seg = 0;                    // tiles and runs of this row tile
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok;) {
      const Kv8Place sp = kv8_place_of(u, s_pref, VB, Hkv);
      const int64_t seg_end = min(u1, u + sp.n - sp.tile);
      const int tiles = static_cast<int>(seg_end - u);
      const int gv = p.v0 + sp.v, b = gv / p.RG, r0 = (gv - b * p.RG) * kKv8PrefillRows;
      if (r0 + rt * kTile >= R) {            // this row tile is empty
        kt += tiles;
        u = seg_end;
        continue;
      }
      const int r = r0 + rt * kTile + row;
      const bool on = r < R;
      const int i = on ? r / p.G : 0, hq = sp.h * p.G + (on ? r - i * p.G : 0);
      const int len = kv8_len(p.sc.kv_lens, b, p.map.cap, nullptr);
      int lo = 0, hi = 0, pos = 0;
      float slope = 0.f;
      if (on) {
        kv8_range(p.sc, b, i, p.T, len, lo, hi, pos);
        if (GEN && p.sc.slopes) slope = __ldg(p.sc.slopes + hq) * kLog2E;
      }
      // ---- the row of q, divided by a power of two
      float rowc;
      {
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(p.q) + b * p.q_stride_b + hq * p.q_stride_h + i * p.q_stride_t);
        const bool bf = p.dtype == TQ_BF16;
        auto unpack = [&](uint32_t w) {
          return bf ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u))
                    : __half22float2(*reinterpret_cast<const __half2*>(&w));
        };
        uint4 x[D / 8];
        float mx = 0.f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          x[c] = on ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack(w[k]);
            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23), 1), 253);
        float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        rowc = __uint_as_float(static_cast<uint32_t>(e) << 23) * fabsf(p.sc.scale_log2);
        if (p.sc.scale_log2 < 0.f) down = -down;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack(w[k]);
            y[k] = pack_h2(f.x * down, f.y * down);
          }
          sts128(qa + tile_off(row, c), y[0], y[1], y[2], y[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(bar(QFULL + rt));
      }
      // tokens that all rows of this warp see
      const int w_lo = __reduce_max_sync(0xffffffffu, on ? lo : 0);
      const int w_hi = __reduce_min_sync(0xffffffffu, on ? hi : INT32_MAX);
      const int tile0 = s_lo[sp.v] / kTile + sp.tile;

      float m = -INFINITY, l = 0.f, E = 1.f;
      for (int j = 0; j < tiles; ++j, ++kt, ++own) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(SFULL + rt), own & 1, lim, p.status, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const float* sc = s_scale + (kt % kScaleSlots) * kSlot;
        E = sc[2 * kBlocks];
        const int t0 = (tile0 + j) * kTile;
        const bool masked = t0 < w_lo || t0 + kTile > w_hi;
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < kTile / 32; ++c) {
          float s[32];
          tmem_ld32(ts + 32 * c, s);
          tmem_wait_ld();
          const float c0 = sc[2 * c] * rowc, c1 = sc[2 * c + 1] * rowc;
          if (GEN || masked) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const int t = t0 + 32 * c + k;
              float x = s[k] * (k < 16 ? c0 : c1);
              if (GEN) {
                if (p.sc.cap > 0.f) x = p.sc.cap * kLog2E * kv8_tanh(x * (kLn2 / p.sc.cap));
                if (p.sc.slopes) x -= slope * static_cast<float>(abs(pos - t));
              }
              if (masked && (t < lo || t >= hi)) x = -INFINITY;
              s[k] = x;
              mx = fmaxf(mx, x);
            }
            tmem_st32(ts + 32 * c, s);
          } else {
            float a = s[0], d = s[16];
#pragma unroll
            for (int k = 1; k < 16; ++k) { a = fmaxf(a, s[k]); d = fmaxf(d, s[16 + k]); }
            mx = fmaxf(mx, fmaxf(a * c0, d * c1));
          }
        }
        if (GEN || masked) tmem_wait_st();
        // ---- the reference, and what was summed against the old one
        const bool grow = mx > m + kLazy || m == -INFINITY;
        const float m1 = grow ? fmaxf(m, mx) : m;
        const float ref = m1 == -INFINITY ? 0.f : m1;
        if (j > 0 && __any_sync(0xffffffffu, grow && mx > m)) {
          const float a = ex2(m - ref);      // 1 where the reference stays, 0 where there was none
          l *= a;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tmem_ld32(to + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= a;
            tmem_st32(to + 32 * c, o);
          }
        }
        m = m1;
        // ---- probabilities
#pragma unroll 1
        for (int c = 0; c < kTile / 32; ++c) {
          float s[32];
          tmem_ld32(ts + 32 * c, s);
          tmem_wait_ld();
          uint32_t out[16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float f = sc[kBlocks + 2 * c + h];
            const float cc = (GEN || masked) ? 1.f : sc[2 * c + h] * rowc;
            const float off = f - ref;
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float x = ex2(fmaf(s[16 * h + k], cc, off)), y = ex2(fmaf(s[16 * h + k + 1], cc, off));
              sum += x + y;
              out[8 * h + k / 2] = pack_h2(x, y);
            }
            l = fmaf(sum, ex2(-f), l);
          }
          tmem_st16(ts + 16 * c, out);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(PFULL + rt));
      }
      if (!ok) break;
      // ---- the run's result
      ok = __all_sync(0xffffffffu, mbar_wait(bar(OFULL + rt), seg & 1, lim, p.status, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const bool whole = sp.tile == 0 && tiles == sp.n;
      // O is in units of 2^(E - 127 - kHead); two factors, so that neither leaves the normal range
      const float unit = __uint_as_float(static_cast<uint32_t>(E) << 23);
      const float inv = l == 0.f ? 0.f : 1.f / (l * (1 << kHead));
      const float ls2 = l == 0.f ? -INFINITY : m + __log2f(l);
      const int64_t at = (static_cast<int64_t>(b) * p.Hq + hq) * p.T + i;
      const int slot = blockIdx.x * 2 + (sp.tile == 0 ? 1 : 0);
      const int64_t prow = static_cast<int64_t>(slot) * kKv8PrefillRows + rt * kTile + row;
      if (on) {
        if (whole) { if (p.lse) p.lse[at] = ls2 * kLn2; }
        else p.part_lse[prow] = ls2;
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        tmem_ld32(to + 32 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = o[k] * inv * unit;
        if (on && whole) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            if (p.dtype == TQ_BF16) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]);
              w[k] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
              w[k] = pack_h2(o[2 * k], o[2 * k + 1]);
            }
          }
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * D + 32 * c);
#pragma unroll
          for (int k = 0; k < 4; ++k) dst[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        } else if (on) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D + 32 * c);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
        __syncwarp();
      }
      tc_fence_before();                     // before the next run's products overwrite O
      ++seg;
      u = seg_end;
    }
  } else if (warp < 12) {
    // ================================================================ codes to halves
    const int w = warp - 8;
    int64_t kt = 0;
    bool ok = true;                          // a thread that gave up still takes part in the barriers
    constexpr int NL = D / 16;               // 16-byte loads a thread and tile: rows 8 (w + 4 k) + lane % 8
    constexpr int NH = D / 64;
    for (int64_t u = u0; u < u1;) {
      const Kv8Place sp = kv8_place_of(u, s_pref, VB, Hkv);
      const int64_t seg_end = min(u1, u + sp.n - sp.tile);
      const int tiles = static_cast<int>(seg_end - u);
      const int b = (p.v0 + sp.v) / p.RG;
      const int b_lo = s_lo[sp.v] / kKv8Block, b_hi = (s_hi[sp.v] - 1) / kKv8Block;
      const int tile0 = s_lo[sp.v] / kTile + sp.tile;
      // record of a block; one outside the visible tokens may have no page: the nearest visible
      auto block_rec = [&](int blk) {
        return kv8_record(p.map, b, sp.h, static_cast<int64_t>(min(max(blk, b_lo), b_hi)) * kKv8Block, p.status);
      };
      // largest value scale of the run
      int E = 1;
      for (int blk = max(tile0 * kBlocks, b_lo) + w * 32 + lane; blk <= min((tile0 + tiles) * kBlocks - 1, b_hi); blk += 128)
        E = max(E, static_cast<int>((__float_as_uint(__ldg(p.vscales + block_rec(blk) / kKv8Block)) >> 23) & 0xffu));
      E = __reduce_max_sync(0xffffffffu, E);
      if (lane == 0) s_e[w] = E;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      E = max(max(s_e[0], s_e[1]), max(s_e[2], s_e[3]));
      asm volatile("bar.sync 1, 128;" ::: "memory");

      // row 8 (w + 4 k) + lane % 8 of a tile lies in block (w + 4 k) / 2
      uint4 raw_k[NL], raw_v[NL];
      float next_scale = 0.f;
      auto load = [&](const uint8_t* codes, int tile, uint4 (&x)[NL]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = 8 * (w + 4 * k) + (lane & 7);
          const int64_t rec = block_rec(tile * kBlocks + rr / kKv8Block) + rr % kKv8Block;
#pragma unroll
          for (int h = 0; h < NH; ++h)
            x[k * NH + h] = __ldg(reinterpret_cast<const uint4*>(codes + rec * D + h * 64 + (lane >> 3) * 16));
        }
      };
      auto load_scales = [&](int tile) {     // threads 0..7 key scales, 8..15 value scales
        if (w == 0 && lane < 2 * kBlocks)
          next_scale = __ldg((lane < kBlocks ? p.kscales : p.vscales) + block_rec(tile * kBlocks + lane % kBlocks) / kKv8Block);
      };
      auto convert = [&](uint4 (&x)[NL], uint32_t dst, bool clean) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = 8 * (w + 4 * k) + (lane & 7);
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            uint4 y = x[k * NH + h];
            if (clean) {
              y.x = e4m3_nan_to_zero(y.x);
              y.y = e4m3_nan_to_zero(y.y);
              y.z = e4m3_nan_to_zero(y.z);
              y.w = e4m3_nan_to_zero(y.w);
            }
            const int c = h * 8 + (lane >> 3) * 2;
            sts128(dst + tile_off(rr, c), e4m3x2_to_h2(y.x), e4m3x2_to_h2(y.x >> 16), e4m3x2_to_h2(y.y),
                   e4m3x2_to_h2(y.y >> 16));
            sts128(dst + tile_off(rr, c + 1), e4m3x2_to_h2(y.z), e4m3x2_to_h2(y.z >> 16), e4m3x2_to_h2(y.w),
                   e4m3x2_to_h2(y.w >> 16));
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      };
      if (ok) {
        load_scales(tile0);
        load(kcodes, tile0, raw_k);
      }
      for (int j = 0; j < tiles && ok; ++j, ++kt) {
        const int st = static_cast<int>(kt & 1);
        const uint32_t ph = static_cast<uint32_t>((kt >> 1) - 1) & 1u;
        const int t0 = (tile0 + j) * kTile;
        load(vcodes, tile0 + j, raw_v);
        if (kt >= 2 && !mbar_wait(bar(KEMPTY + st), ph, lim, p.status, abort_flag)) { ok = false; break; }
        if (w == 0 && lane <= 2 * kBlocks) {
          float x = next_scale;
          if (lane == 2 * kBlocks) x = static_cast<float>(E);
          else if (lane >= kBlocks)          // exponent of the block's probabilities
            x = static_cast<float>(kHead + max(static_cast<int>((__float_as_uint(x) >> 23) & 0xffu) - E, -100));
          s_scale[(kt % kScaleSlots) * kSlot + lane] = x;
        }
        convert(raw_k, base + L.k + st * TB, false);
        mbar_arrive(bar(KFULL + st));
        if (j + 1 < tiles) {
          load_scales(tile0 + j + 1);
          load(kcodes, tile0 + j + 1, raw_k);
        }
        if (kt >= 2 && !mbar_wait(bar(VEMPTY + st), ph, lim, p.status, abort_flag)) { ok = false; break; }
        // a masked token's NaN stays out of the rows that do not see it
        convert(raw_v, base + L.v + st * TB, t0 < s_in_lo[sp.v] || t0 + kTile > s_in_hi[sp.v]);
        mbar_arrive(bar(VFULL + st));
      }
      u = seg_end;
    }
  } else if (lane == 0) {
    // ================================================================ tensor core
    const uint32_t id_qk = idesc_f16(kTile, 0), id_pv = idesc_f16(D, 1);
    int64_t kt = 0;
    int own[2] = {0, 0}, seg[2] = {0, 0};
    bool ok = true;
    auto qk = [&](int rt, int st) {
      const uint32_t a = base + L.q + rt * TB, bq = base + L.k + st * TB;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (k >> 2) * 16384u + (k & 3) * 32u;
        umma_f16(tmem + rt * 128, sw128_desc(a + off), sw128_desc(bq + off), id_qk, k > 0);
      }
    };
    for (int64_t u = u0; u < u1 && ok;) {
      const Kv8Place sp = kv8_place_of(u, s_pref, VB, Hkv);
      const int64_t seg_end = min(u1, u + sp.n - sp.tile);
      const int tiles = static_cast<int>(seg_end - u);
      const int gv = p.v0 + sp.v, r0 = (gv % p.RG) * kKv8PrefillRows;
      const int nrt = r0 + kTile < R ? 2 : 1;
      for (int j = -1; j < tiles && ok; ++j) {
        // tile j's second product, then tile j + 1's first
        const int64_t kn = kt + j + 1;
        const int st = static_cast<int>((kt + j) & 1), stn = static_cast<int>(kn & 1);
        for (int rt = 0; rt < nrt && ok; ++rt) {
          if (j >= 0) {
            if (rt == 0) ok = mbar_wait(bar(VFULL + st), ((kt + j) >> 1) & 1, lim, p.status, abort_flag);
            if (ok) ok = mbar_wait(bar(PFULL + rt), own[rt] & 1, lim, p.status, abort_flag);
            if (!ok) break;
            ++own[rt];
            tc_fence_after();
            const uint32_t bv = base + L.v + st * TB;
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              umma_f16_ts(tmem + 256 + rt * D, tmem + rt * 128 + k * 8, sw128_desc_t(bv + k * 2048u), id_pv, j > 0 || k > 0);
            if (rt == nrt - 1) umma_commit(bar(VEMPTY + st));
            if (j + 1 == tiles) umma_commit(bar(OFULL + rt));
          } else {
            ok = mbar_wait(bar(QFULL + rt), seg[rt] & 1, lim, p.status, abort_flag);
            if (!ok) break;
            ++seg[rt];
            tc_fence_after();
          }
          if (j + 1 < tiles) {
            if (rt == 0) ok = mbar_wait(bar(KFULL + stn), (kn >> 1) & 1, lim, p.status, abort_flag);
            if (!ok) break;
            tc_fence_after();
            qk(rt, stn);
            umma_commit(bar(SFULL + rt));
            if (rt == nrt - 1) umma_commit(bar(KEMPTY + stn));
          }
        }
      }
      kt += tiles;
      u = seg_end;
    }
    // all products end before tensor memory is given back
    const uint32_t end_bar = base + L.misc + 48;
    mbar_init(end_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    umma_commit(end_bar);
    for (long long i = 0; !mbar_try(end_bar, 0) && i < kDrainLimit; ++i) {}
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the partial results of a (256-row group, key head) that several CTAs worked on; one warp
// a row.  Groups with no visible token get zeros.
template <int D>
__global__ void __launch_bounds__(256) kv8_prefill_join_kernel(const Kv8AttnParams p) {
  pdl_wait();
  pdl_trigger();
  const int Hkv = p.map.Hkv, v = blockIdx.x / Hkv, h = blockIdx.x - v * Hkv;
  const int64_t per = __ldg(reinterpret_cast<const int64_t*>(p.plan));
  const int t0 = __ldg(p.plan + kKv8PlanHead + v), n = __ldg(p.plan + kKv8PlanHead + v + 1) - t0;
  const int64_t u = static_cast<int64_t>(t0) * Hkv + static_cast<int64_t>(h) * n;
  const int c0 = static_cast<int>(u / per), c1 = n ? static_cast<int>((u + n - 1) / per) : c0;
  if (n && c0 == c1) return;
  const int gv = p.v0 + v, b = gv / p.RG, r0 = (gv - b * p.RG) * kKv8PrefillRows, R = p.T * p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int PL = D / 32;
  const int rl = blockIdx.y * 8 + warp;
  if (r0 + rl >= R) return;
  const int r = r0 + rl, i = r / p.G;
  const int64_t row = (static_cast<int64_t>(b) * p.Hq + h * p.G + (r - i * p.G)) * p.T + i;
  float mx = -INFINITY, sum = 0.f, o[PL];
#pragma unroll
  for (int k = 0; k < PL; ++k) o[k] = 0.f;
  auto prow = [&](int c) { return static_cast<int64_t>(c * 2 + (c == c0 ? 1 : 0)) * kKv8PrefillRows + rl; };
  if (n) {
    for (int c = c0 + lane; c <= c1; c += 32) mx = fmaxf(mx, __ldg(p.part_lse + prow(c)));
    mx = warp_max(mx);
    if (mx > -INFINITY)
      for (int c = c0; c <= c1; ++c) {
        const float w = ex2(__ldg(p.part_lse + prow(c)) - mx);
        sum += w;
        const float* src = p.part_o + prow(c) * D + lane * PL;
#pragma unroll
        for (int k = 0; k < PL; ++k) o[k] += w * __ldg(src + k);
      }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  if (p.lse && lane == 0) p.lse[row] = sum > 0.f ? (mx + __log2f(sum)) * kLn2 : -INFINITY;
#pragma unroll
  for (int k = 0; k < PL; ++k) {
    const float x = o[k] * inv;
    if (p.dtype == TQ_BF16) static_cast<__nv_bfloat16*>(p.out)[row * D + lane * PL + k] = __float2bfloat16_rn(x);
    else static_cast<__half*>(p.out)[row * D + lane * PL + k] = __float2half_rn(x);
  }
}

template <int D, bool GEN>
cudaError_t go(const uint8_t* kc, const uint8_t* vc, const Kv8AttnParams& p, int grid, cudaStream_t s) {
  auto k = kv8_prefill_kernel<D, GEN>;
  constexpr uint32_t smem = prefill_smem(D).total;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3(grid), dim3(kThreads), smem, s, kc, vc, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv8_prefill_join_kernel<D>, dim3(static_cast<unsigned>(p.VB) * p.map.Hkv, kKv8PrefillRows / 8), dim3(256), 0,
                    s, p);
}

}  // namespace

cudaError_t launch_kv8_prefill(const uint8_t* kcodes, const uint8_t* vcodes, const Kv8AttnParams& p, int d, int grid,
                               cudaStream_t s) {
  const bool gen = p.sc.cap > 0.f || p.sc.slopes;
  if (d == 128) return gen ? go<128, true>(kcodes, vcodes, p, grid, s) : go<128, false>(kcodes, vcodes, p, grid, s);
  return gen ? go<64, true>(kcodes, vcodes, p, grid, s) : go<64, false>(kcodes, vcodes, p, grid, s);
}

}  // namespace tq

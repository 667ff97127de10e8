// Attention of many query rows a key head over the 8-bit block-scaled cache, on the tensor cores
// with accumulators in tensor memory (16-bit queries).
//
//   S = Q K^T,  l_t = scale s_k(t) S_t (capped, biased),  O = sum_t e^{l_t} v^_t,  out = O / sum
//
// 4 d operations a (row, token) and one exponential bound it: 2 x 128 rows and 128 tokens at d = 128
// take the tensor core 2048 cycles and the exponentials, 16 a cycle, as many.  Measured: 4000 to 4300
// cycles, of which a row tile's softmax is 2400 and its two products, which share the memory they
// read with the conversion of the codes, 1500 (causal 8192 tokens, 32 heads: 537 us, 1.02 PFLOP/s;
// two times 512 queries over 32768 tokens: 505 us, 1.08).
//
// A CTA an SM (persistent) takes runs of the line of (256-row group, key head, 128-token tile) as
// the decode kernel does.  Its roles, with register shares of their own (setmaxnreg):
//   warps 0-3, 4-7   softmax of row tile 0 and 1, a row a thread: the scores of a tile are read from
//                    tensor memory at once and stay in registers; running maximum and sum; the
//                    probabilities go back into tensor memory as halves.  Between runs: q and results
//   warps 8-11       codes to halves, in place: a tile's codes arrive in one half of its operand
//                    tile and are expanded to all of it (128-byte swizzle)
//   warp 12          issues the products
//   warp 13          prepares runs: what their rows see
//   warps 14, 15     ask for keys and scales, and for values (bulk copies of blocks, or of as many as
//                    follow one another in the cache)
// The two row tiles alternate: while one tile's scores are in the softmax, the tensor core works
// for the other.  (A warp issuing for each row tile lets both fall into step: 606 us in place of 524.)
// The second product begins with the first half of the probabilities (521 without, 512 with).  Tensor
// memory (512 columns): S 0, S 1 (128 each; the tile's probabilities overwrite its scores, two a
// column), O 0, O 1.  K is a row-major operand, V the same bytes read transposed.
//
// A row's reference stays while no score exceeds it by 2^8, so the outputs are seldom rescaled.
// The value scales 2^e of 16-token blocks join the exponent: P = 2^(l - m + 7 + e - E), E the
// largest e so far, at most 2^15 in halves of 11 bits (a probability below 2^-21 of the row's largest
// loses bits to the halves' subnormal step, 2^-32 of it); row sums are fp32.  q is divided by a power
// of two a row, as in the decode kernel.  A capped score is a series where it is at most cap / 2, else
// exponential and division (kv8_cap); where 1024 of them are small at once, the series alone.  So a row's
// bits do not depend on its neighbours' scores, or on those that a mask hides.
#include <cuda_runtime.h>

#include "kv8_launch.h"
#include "launchers.h"
#include "quantize_umma.cuh"

namespace tq {
namespace {

constexpr int kThreads = 16 * 32;
constexpr int kTile = 128;                   // tokens, and rows of a row tile
constexpr int kBlocks = kTile / kKv8Block;
constexpr float kLazy = 8.f;                 // a reference may lag by this many powers of two
constexpr int kHead = 7;                     // P <= 2^(kLazy + kHead)
constexpr int kScaleSlots = 4;               // tiles whose scales are kept: a slot is filled again when the
                                             // first product of the tile two before is done, so none in use
constexpr int kSlot = 3 * kBlocks + 4;       // key scales, exponents f of the probabilities, 2^-f, E
// What a run costs beside its tiles, in tiles: q, the first copies, the result.  (8k tokens, causal, d = 128:
// 775 us with 2, 589 with 4, 605 with 7; where the tiles cost more, capped d = 64: 114 with 2, 125 with 4.)
__host__ __device__ constexpr int run_cost(bool gen) { return gen ? 2 : 4; }
// Registers a thread of the roles' warpgroups; the launch has 128 for each of 512 threads.
constexpr int kRegsSoftmax = 192, kRegsConvert = 72, kRegsRest = 56, kRegsLaunch = 128;
static_assert(2 * kRegsSoftmax + kRegsConvert + kRegsRest <= 4 * kRegsLaunch, "registers");
constexpr int kScouts = 32;                  // the warp that prepares runs

// A run, on rows r0 .. of sequence b; its first tile starts at token t0.  tiles = 0: no more.
struct Run : Kv8Run {
  int b, r0, t0;
  int lo, hi;                                // tokens that some row sees
  int in_lo, in_hi;                          // tokens that all rows see
};

struct RowMeta {                             // of 256 rows
  Run run;
  int lo[kKv8PrefillRows], hi[kKv8PrefillRows], pos[kKv8PrefillRows];
  float slope[kKv8PrefillRows];
  int i[kKv8PrefillRows], hq[kKv8PrefillRows];       // query and head; i = -1: no row
};

struct PrefillSmem {
  uint32_t q, k, v, stage, meta, scales, bars, pref, misc, total;
};
__host__ __device__ constexpr PrefillSmem prefill_smem(int D) {
  PrefillSmem L{};
  const uint32_t tile = kTile * D * 2;
  uint32_t at = 0;
  L.q = at; at += 2 * tile;
  L.k = at; at += 2 * tile;
  L.v = at; at += 2 * tile;
  L.stage = at; at += 8 * 2048;              // results on their way out, 64 bytes of 32 rows a warp
  L.meta = at; at += 2 * sizeof(RowMeta);
  L.scales = at; at += kScaleSlots * kSlot * 4;
  L.bars = at; at += 26 * 8;
  L.pref = at; at += (kKv8PrefillMaxVB + 4) * 4;
  L.misc = at; at += 64;
  L.total = at + 1024;
  return L;
}
static_assert(prefill_smem(128).total <= 232448, "shared memory");

enum : int { KFULL = 0, KEMPTY = 2, VFULL = 4, VEMPTY = 6, SFULL = 8, PFULL = 10, OFULL = 12, QFULL = 14, MEMPTY = 16, DFULL = 18, PHALF = 20, KRAW = 22, VRAW = 24 };

// Operand tile of 128 rows of D halves: D / 64 parts of [128][64], 16-byte chunks XORed with the
// row within 8.  Byte offset of chunk c (8 halves) of row r.
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  return (c >> 3) * 16384u + r * 128u + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
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

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// 16 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t a, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
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

// No use of v before this point (the wait for its load from tensor memory).
__device__ __forceinline__ void pin(float (&v)[32]) {
#pragma unroll
  for (int k = 0; k < 32; ++k) asm volatile("" : "+f"(v[k]));
}

// Bounded wait of a warp; one that gives up raises the flag, which ends the others' (the status is
// reported at the end).  Kept short: its copies and the unrolled softmax share the instruction cache.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, int limit, volatile int* abort_flag) {
  bool done = false;
#pragma unroll 1
  for (int i = 0; i < limit; ++i) {
    done = mbar_try(bar, parity);
    if (done || *abort_flag) break;
  }
  if (__all_sync(0xffffffffu, done)) return true;
  *abort_flag = 1;
  return false;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(on));
  return on != 0;
}

// out * tanh(in * x) of 16 values, |in * x| <= 1/2: the series to z^11, whose next term is below 2^-21.
// Step by step for all, so that no step waits for the one before.
__device__ __forceinline__ void tanh_small(float (&s)[32], int at, float in, float out) {
  float2 z[8], u[8], q[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) z[k] = mul2(pair(s[at + 2 * k], s[at + 2 * k + 1]), both(in));
#pragma unroll
  for (int k = 0; k < 8; ++k) u[k] = mul2(z[k], z[k]);
#pragma unroll
  for (int k = 0; k < 8; ++k) q[k] = fma2(u[k], both(-1382.f / 155925.f), both(62.f / 2835.f));
#pragma unroll
  for (int k = 0; k < 8; ++k) q[k] = fma2(u[k], q[k], both(-17.f / 315.f));
#pragma unroll
  for (int k = 0; k < 8; ++k) q[k] = fma2(u[k], q[k], both(2.f / 15.f));
#pragma unroll
  for (int k = 0; k < 8; ++k) q[k] = fma2(u[k], q[k], both(-1.f / 3.f));
#pragma unroll
  for (int k = 0; k < 8; ++k) z[k] = mul2(z[k], both(out));
#pragma unroll
  for (int k = 0; k < 8; ++k) u[k] = mul2(z[k], u[k]);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 y = fma2(u[k], q[k], z[k]);
    s[at + 2 * k] = y.x;
    s[at + 2 * k + 1] = y.y;
  }
}

// GEN: scores are capped or biased.
template <int D, bool GEN>
__global__ void __launch_bounds__(kThreads, 1)
kv8_prefill_kernel(const uint8_t* __restrict__ kcodes, const uint8_t* __restrict__ vcodes, const Kv8AttnParams p) {
  constexpr PrefillSmem L = prefill_smem(D);
  constexpr uint32_t TB = kTile * D * 2;     // bytes of an operand tile
  constexpr uint32_t BB = kKv8Block * D;     // bytes of a block's codes, which arrive
  constexpr uint32_t kRaw = D == 128 ? 16384u : 0u;    // there in the tile, and 2048 further for each block
  extern __shared__ unsigned char psm_raw[];
  const uint32_t raw = smem_u32(psm_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* sm = psm_raw + (base - raw);
  RowMeta* s_meta = reinterpret_cast<RowMeta*>(sm + L.meta);
  float* s_scale = reinterpret_cast<float*>(sm + L.scales);
  int* s_pref = reinterpret_cast<int*>(sm + L.pref);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L.misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L.misc + 4);
  const uint32_t bar0 = base + L.bars;
  auto bar = [&](int id) { return bar0 + 8u * id; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(KFULL + i), 128);
      mbar_init(bar(KEMPTY + i), 4);
      mbar_init(bar(VFULL + i), 128);
      mbar_init(bar(VEMPTY + i), 4);
      mbar_init(bar(SFULL + i), 1);
      mbar_init(bar(PFULL + i), 128);
      mbar_init(bar(OFULL + i), 1);
      mbar_init(bar(QFULL + i), 128);
      mbar_init(bar(MEMPTY + i), 256 + 4 + 1 + 2);     // softmax threads; converting, issuing and fetching warps
      mbar_init(bar(PHALF + i), 128);
      mbar_init(bar(DFULL + i), kScouts);
      mbar_init(bar(KRAW + i), 1);
      mbar_init(bar(VRAW + i), 1);
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
  // Tokens that some row, and that all rows, of a group see (one warp).
  auto group_range = [&](int b, int r0, int len, int& lo, int& hi, int& in_lo, int& in_hi) {
    lo = INT32_MAX, hi = 0, in_lo = 0, in_hi = INT32_MAX;
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
  };
  for (int v = warp; v < VB; v += kThreads / 32) {
    const int gv = p.v0 + v, b = gv / p.RG, r0 = (gv - b * p.RG) * kKv8PrefillRows;
    const int len = kv8_len(p.sc.kv_lens, b, p.map.cap, p.status);
    int lo, hi, in_lo, in_hi;
    group_range(b, r0, len, lo, hi, in_lo, in_hi);
    if (lane == 0) s_pref[v + 1] = hi > 0 ? (hi + kTile - 1) / kTile - lo / kTile + run_cost(GEN) : 0;
  }
  __syncthreads();
  if (warp == 0) kv8_prefix(s_pref, VB);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int64_t total = static_cast<int64_t>(s_pref[VB]) * Hkv;
  const int64_t per = max((total + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(1));
  const int64_t u0 = min(total, per * blockIdx.x), u1 = min(total, u0 + per);
  pdl_trigger();
  const int lim = static_cast<int>(min(p.wait_limit, static_cast<long long>(INT32_MAX)));
  auto wait_for = [&](int id, uint32_t parity) { return wait_bar(bar(id), parity & 1u, lim, abort_flag); };

  if (warp < 8) {
    // ================================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int rt = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + rt * 128, to = tmem + lanes + 256 + rt * D;
    int kt = 0, own = 0, oseg = 0;           // tiles of the CTA, tiles and runs of this row tile
    const bool bf = p.dtype == TQ_BF16;
    const int rr = rt * kTile + row;
    const uint32_t qa = base + L.q + rt * TB;
    float rowc = 0.f;
    bool asked = false;                      // the run was waited for, its q asked for
    // The warp's 32 rows of q, each by D / 8 neighbouring lanes, to where they will stand as an operand.
    auto ask_q = [&](const RowMeta& meta) {
      constexpr int LPR = D / 8;
      const int64_t at_b = meta.run.b * p.q_stride_b;
#pragma unroll 4
      for (int k = 0; k < LPR; ++k) {
        const int r = (warp & 3) * 32 + k * (32 / LPR) + lane / LPR, c = lane % LPR;
        const int i = max(meta.i[rt * kTile + r], 0);        // (a row that is none: another one's q, not used)
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + at_b + meta.hq[rt * kTile + r] * p.q_stride_h + i * p.q_stride_t;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(qa + tile_off(r, c)), "l"(src + c * 8) : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // This thread's row divided by a power of two, its largest entry in [1, 2).
    auto scale_q = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      auto unpack = [&](uint32_t w) {
        return bf ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u))
                  : __half22float2(*reinterpret_cast<const __half2*>(&w));
      };
      float mx = 0.f;
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = lds128(qa + tile_off(row, c));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
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
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = lds128(qa + tile_off(row, c));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
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
    };
    bool ok = true;
    for (int seg = 0;; ++seg) {
      const RowMeta& meta = s_meta[seg & 1];
      const Run& run = meta.run;
      if (!asked) ok = wait_for(DFULL + (seg & 1), (seg >> 1) & 1);
      const int tiles = run.tiles;
      if (!ok || tiles == 0) break;
      if (run.r0 + rt * kTile >= R) {        // this row tile is empty
        kt += tiles;
        asked = false;
        mbar_arrive(bar(MEMPTY + (seg & 1)));
        continue;
      }
      if (!asked) ask_q(meta);
      scale_q();
      asked = false;
      int t0 = run.t0;
      const int lo = meta.lo[rr], hi = meta.hi[rr], pos = GEN ? meta.pos[rr] : 0;
      const float slope = GEN ? meta.slope[rr] : 0.f;
      const bool last = rt == 1 || run.r0 + kTile >= R;
      float m = -INFINITY, l = 0.f, E = 1.f;
      for (int j = 0; j < tiles; ++j, ++kt, ++own, t0 += kTile) {
        ok = wait_for(SFULL + rt, own & 1);
        if (!ok) break;
        tc_fence_after();
        // The last row tile's first product is done: so are all that read the keys, and the values of
        // the tile before.
        if (last && lane == 0) {
          mbar_arrive(bar(KEMPTY + (kt & 1)));
          if (j > 0) mbar_arrive(bar(VEMPTY + ((kt - 1) & 1)));
        }
        const float* sc = s_scale + (kt % kScaleSlots) * kSlot;
        const float E1 = sc[3 * kBlocks];
        const bool masked = __any_sync(0xffffffffu, t0 < lo || t0 + kTile > hi);
        const bool formed = GEN || masked;   // scores are formed here, else their scale joins the exponent
        // Rolled, by way of tensor memory: copies of this for each 32 tokens cost the plain path its
        // registers and its place in the instruction cache (561 us became 661).
        if (formed) {
#pragma unroll 1
          for (int c = 0; c < kTile / 32; ++c) {
            const int from = lo - t0 - 32 * c, to = hi - t0 - 32 * c;          // visible ones of the 32
            const bool cut = masked && __any_sync(0xffffffffu, from > 0 || to < 32);
            float s[32];
            if (cut && __all_sync(0xffffffffu, from >= 32 || to <= 0)) {
#pragma unroll
              for (int k = 0; k < 32; ++k) s[k] = -INFINITY;
            } else {
              tmem_ld32(ts + 32 * c, s);
              tmem_wait_ld();
              pin(s);
              if (GEN && p.sc.cap > 0.f) {
                const float by_cap = kLn2 / p.sc.cap * rowc, cap2 = p.sc.cap * kLog2E;
                const float z0 = sc[2 * c] * by_cap, z1 = sc[2 * c + 1] * by_cap;
                float far = 0.f, far1 = 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  far = fmaxf(far, fabsf(s[k]));
                  far1 = fmaxf(far1, fabsf(s[16 + k]));
                }
                if (__all_sync(0xffffffffu, fmaxf(far * z0, far1 * z1) <= 0.5f)) {
                  tanh_small(s, 0, z0, cap2);
                  tanh_small(s, 16, z1, cap2);
                } else {
#pragma unroll
                  for (int k = 0; k < 32; k += 2) {      // (the series' bits where a score is small)
                    const float2 y = kv8_cap(mul2(pair(s[k], s[k + 1]), both(k < 16 ? z0 : z1)), cap2);
                    s[k] = y.x;
                    s[k + 1] = y.y;
                  }
                }
              } else {
                const float z0 = sc[2 * c] * rowc, z1 = sc[2 * c + 1] * rowc;
#pragma unroll
                for (int k = 0; k < 32; ++k) s[k] *= k < 16 ? z0 : z1;
              }
              if (GEN && p.sc.slopes) {
                const float far0 = static_cast<float>(pos - t0 - 32 * c);
#pragma unroll
                for (int k = 0; k < 32; ++k) s[k] = fmaf(-slope, fabsf(far0 - k), s[k]);
              }
              if (cut) {
                const uint32_t seen = (to >= 32 ? ~0u : to <= 0 ? 0u : (1u << to) - 1u) &
                                      (from <= 0 ? ~0u : from >= 32 ? 0u : ~0u << from);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (!(seen & (1u << k))) s[k] = -INFINITY;
              }
            }
            tmem_st32(ts + 32 * c, s);
          }
          tmem_wait_st();
        }
        // the row's scores stay in registers (the probabilities overwrite them in tensor memory)
        float s0[32], s1[32], s2[32], s3[32];
        tmem_ld32(ts, s0);
        tmem_ld32(ts + 32, s1);
        tmem_ld32(ts + 64, s2);
        tmem_ld32(ts + 96, s3);
        tmem_wait_ld();
        pin(s0);
        pin(s1);
        pin(s2);
        pin(s3);
        auto top = [&](const float (&s)[32], int c) {
          float a = s[0], b = s[16];
#pragma unroll
          for (int k = 1; k < 16; ++k) {
            a = fmaxf(a, s[k]);
            b = fmaxf(b, s[16 + k]);
          }
          return formed ? fmaxf(a, b) : fmaxf(a * (sc[2 * c] * rowc), b * (sc[2 * c + 1] * rowc));
        };
        const float mx = fmaxf(fmaxf(top(s0, 0), top(s1, 1)), fmaxf(top(s2, 2), top(s3, 3)));
        // ---- the reference, and what was summed against the old one and the old E
        const bool grow = mx > m + kLazy || m == -INFINITY;
        const float m1 = grow ? fmaxf(m, mx) : m;
        const float ref = m1 == -INFINITY ? 0.f : m1;
        if (j > 0 && __any_sync(0xffffffffu, (grow && mx > m) || E1 != E)) {
          const float a = ex2(m - ref);      // 1 where the reference stays, 0 where there was none
          l *= a;
          const float ae = a * ex2(E - E1);
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            float o[16];
            tmem_ld16(to + 16 * c, o);
            tmem_wait_ld();
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k] * ae);
            tmem_st16(to + 16 * c, w);
          }
        }
        m = m1;
        E = E1;
        // ---- probabilities
        // The exponentials of 32 tokens stand between the sums and the rounding of the 32 before, so
        // that their unit, which bounds this part, is not left waiting.
        auto arg = [&](float (&s)[32], int c) {
          const float2 off0 = both(sc[kBlocks + 2 * c] - ref), off1 = both(sc[kBlocks + 2 * c + 1] - ref);
          const float2 cb0 = both(formed ? 1.f : sc[2 * c] * rowc), cb1 = both(formed ? 1.f : sc[2 * c + 1] * rowc);
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float2 x = fma2(pair(s[k], s[k + 1]), k < 16 ? cb0 : cb1, k < 16 ? off0 : off1);
            s[k] = x.x;
            s[k + 1] = x.y;
          }
        };
        auto ex2_at = [](float& x) { asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(x)); };
        uint32_t out[16];
        float2 sum;
        auto finish_at = [&](const float (&s)[32], int c, int k) {         // the pair k of 16
          const float2 x = pair(s[2 * k], s[2 * k + 1]);
          asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(out[k]) : "f"(x.y), "f"(x.x));
          sum = (k & 7) ? add2(sum, x) : x;
          if ((k & 7) == 7) l = fmaf(sum.x + sum.y, sc[2 * kBlocks + 2 * c + (k >> 3)], l);
        };
        arg(s0, 0);
#pragma unroll
        for (int k = 0; k < 32; ++k) ex2_at(s0[k]);
        arg(s1, 1);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          ex2_at(s1[k]);
          if (k & 1) finish_at(s0, 0, k >> 1);
        }
        tmem_st16(ts, out);
        arg(s2, 2);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          ex2_at(s2[k]);
          if (k & 1) finish_at(s1, 1, k >> 1);
        }
        tmem_st16(ts + 16, out);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(PHALF + rt));        // the second product may begin
        arg(s3, 3);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          ex2_at(s3[k]);
          if (k & 1) finish_at(s2, 2, k >> 1);
        }
        tmem_st16(ts + 32, out);
#pragma unroll
        for (int k = 0; k < 16; ++k) finish_at(s3, 3, k);
        tmem_st16(ts + 48, out);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(PFULL + rt));
      }
      if (!ok) break;
      // ---- the next run's row of q is asked for before this run's result is waited for
      const RowMeta& after = s_meta[(seg & 1) ^ 1];
      ok = wait_for(DFULL + ((seg + 1) & 1), ((seg + 1) >> 1) & 1);
      if (!ok) break;
      asked = true;
      if (after.run.tiles > 0 && after.run.r0 + rt * kTile < R) ask_q(after);
      // ---- the run's result
      ok = wait_for(OFULL + rt, oseg & 1);
      if (!ok) break;
      ++oseg;
      if (last && lane == 0) mbar_arrive(bar(VEMPTY + ((kt - 1) & 1)));
      tc_fence_after();
      const bool whole = tiles == run.n;
      // O is in units of 2^(E - 127 - kHead); two factors, so that neither leaves the normal range
      const float unit = __uint_as_float(static_cast<uint32_t>(E) << 23);
      const float inv = l == 0.f ? 0.f : 1.f / (l * (1 << kHead));
      const float ls2 = l == 0.f ? -INFINITY : m + __log2f(l);
      const bool on = meta.i[rr] >= 0;
      const int slot = blockIdx.x * 2 + (run.tile == 0 ? 1 : 0);
      const int64_t prow = static_cast<int64_t>(slot) * kKv8PrefillRows + rr;
      auto out_row = [&](int rr) { return (static_cast<int64_t>(run.b) * p.Hq + meta.hq[rr]) * p.T + meta.i[rr]; };
      if (on) {
        if (whole) { if (p.lse) p.lse[out_row(rr)] = ls2 * kLn2; }
        else p.part_lse[prow] = ls2;
      }
      // 64 bytes a row at a time, by way of shared memory, so that four lanes write them together
      const uint32_t stage = base + L.stage + warp * 2048;
      const int per = whole ? 32 : 16;       // dims
#pragma unroll 1
      for (int c = 0; c < D; c += per) {
        uint32_t w[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !whole) break;
          float o[16];
          tmem_ld16(to + c + 16 * h, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = o[k] * inv * unit;
          if (whole) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const __nv_bfloat162 y = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]);
              w[8 * h + k] = bf ? *reinterpret_cast<const uint32_t*>(&y) : pack_h2(o[2 * k], o[2 * k + 1]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          sts128(stage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4), w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = 8 * k + (lane >> 2), x = lane & 3, ra = rt * kTile + (warp & 3) * 32 + r;
          const uint4 v = lds128(stage + r * 64 + ((x ^ ((r >> 1) & 3)) << 4));
          if (meta.i[ra] < 0) continue;
          if (whole) reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out_row(ra) * D + c)[x] = v;
          else reinterpret_cast<uint4*>(p.part_o + (prow - lane + r) * D + c)[x] = v;
        }
        __syncwarp();
      }
      mbar_arrive(bar(MEMPTY + (seg & 1)));  // (behind the last use of run and meta)
      tc_fence_before();                     // before the next run's products overwrite O
    }
    // ---- groups that see nothing
    for (int v = blockIdx.x; v < VB; v += gridDim.x) {
      if (s_pref[v + 1] != s_pref[v]) continue;
      const int gv = p.v0 + v, b = gv / p.RG, r = (gv - b * p.RG) * kKv8PrefillRows + tid;
      if (r >= R) continue;
      const int i = r / p.G, g = r - i * p.G;
      for (int h = 0; h < Hkv; ++h) {
        const int64_t at = (static_cast<int64_t>(b) * p.Hq + h * p.G + g) * p.T + i;
        if (p.lse) p.lse[at] = -INFINITY;
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * D);
        for (int k = 0; k < D / 8; ++k) dst[k] = make_uint4(0, 0, 0, 0);
      }
    }
  } else if (warp < 12) {
    // ================================================================ codes to halves
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
    // Warp w takes blocks w and w + 4 of each tile.  A block's codes stand where its halves will
    // (in the operand's last 64 dims).
    const int w = warp - 8;
    constexpr int LPR = D / 16, RPL = 32 / LPR, NL = BB / 512;       // lanes a row, rows a step, steps a block
    int kt = 0;
    bool ok = true;
    auto wait = [&](int id, uint32_t parity) {
      ok = wait_for(id, parity);
      return ok;
    };
    auto convert = [&](int side, bool clean) {
      const int st = kt & 1;
      if (!wait((side ? VRAW : KRAW) + st, kt >> 1)) return;
      const uint32_t dst = base + (side ? L.v : L.k) + st * TB;
      uint4 x[2][NL];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int k = 0; k < NL; ++k)
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(x[b][k].x), "=r"(x[b][k].y), "=r"(x[b][k].z), "=r"(x[b][k].w)
                       : "r"(dst + kRaw + (w + 4 * b) * 2048 + k * 512 + lane * 16));
      __syncwarp();                          // (each lane's codes are read before any is overwritten)
      if (clean) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int k = 0; k < NL; ++k) {
            x[b][k].x = e4m3_nan_to_zero(x[b][k].x);
            x[b][k].y = e4m3_nan_to_zero(x[b][k].y);
            x[b][k].z = e4m3_nan_to_zero(x[b][k].z);
            x[b][k].w = e4m3_nan_to_zero(x[b][k].w);
          }
      }
      // Lanes of a row's second 64 dims store their odd chunk first: the two parts of the operand
      // tile lie in the same banks.
      const int c = (lane % LPR) * 2;
      const bool odd = D == 128 && (lane & 4);
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int k = 0; k < NL; ++k) {
          const int rr = (w + 4 * b) * kKv8Block + k * RPL + lane / LPR;
          const uint4 a = x[b][k], y = odd ? make_uint4(a.z, a.w, a.x, a.y) : a;
          sts128(dst + tile_off(rr, c + odd), e4m3x2_to_h2(y.x), e4m3x2_to_h2(y.x >> 16), e4m3x2_to_h2(y.y),
                 e4m3x2_to_h2(y.y >> 16));
          sts128(dst + tile_off(rr, c + !odd), e4m3x2_to_h2(y.z), e4m3x2_to_h2(y.z >> 16), e4m3x2_to_h2(y.w),
                 e4m3x2_to_h2(y.w >> 16));
        }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(bar((side ? VFULL : KFULL) + st));
    };
    for (int seg = 0; ok; ++seg) {
      if (!wait(DFULL + (seg & 1), seg >> 1)) break;
      const Run& run = s_meta[seg & 1].run;
      const int tiles = run.tiles, in_lo = run.in_lo, in_hi = run.in_hi;
      int t0 = run.t0;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(MEMPTY + (seg & 1)));
      if (tiles == 0) break;
      for (int j = 0; j < tiles && ok; ++j, ++kt, t0 += kTile) {
        // a masked token's NaN stays out of the rows that do not see it (scores are replaced)
#pragma unroll 1
        for (int side = 0; side < 2 && ok; ++side) convert(side, side && (t0 < in_lo || t0 + kTile > in_hi));
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == 12) {
      // ============================================================== tensor core
      // The whole warp waits; one lane issues.  The row tiles' products alternate, which also keeps
      // their softmax half a period apart.
      const uint32_t id_qk = idesc_f16(kTile, 0), id_pv = idesc_f16(D, 1);
      const bool leader = elect_one();
      int kt = 0;
      uint32_t own = 0, seg = 0;             // bit rt: parity of the row tile's tiles and runs
      bool ok = true;
      auto wait = [&](int id, uint32_t parity) {
        if (ok) ok = wait_for(id, parity);
        return ok;
      };
      for (int sg = 0; ok; ++sg) {
        if (!wait(DFULL + (sg & 1), sg >> 1)) break;
        const int tiles = s_meta[sg & 1].run.tiles, nrt = s_meta[sg & 1].run.r0 + kTile < R ? 2 : 1;
        __syncwarp();
        if (leader) mbar_arrive(bar(MEMPTY + (sg & 1)));
        if (tiles == 0) break;
        for (int j = -1; j < tiles && ok; ++j) {
          // tile j's second product, then tile j + 1's first
          const int kn = kt + j + 1;
          const int st = (kt + j) & 1, stn = kn & 1;
          // (the converting warps are done with a tile's values before the next tile's keys)
          if (j + 1 < tiles) wait(KFULL + stn, kn >> 1);
          else wait(VFULL + st, (kt + j) >> 1);
          const uint64_t dv = sw128_desc_t(base + L.v + st * TB), dk = sw128_desc(base + L.k + stn * TB);
#pragma unroll 1
          for (int rt = 0; rt < nrt && ok; ++rt) {
            const uint32_t ts = tmem + rt * 128, to = tmem + 256 + rt * D;
            if (j >= 0) {
              if (!wait(PHALF + rt, own >> rt)) break;
              tc_fence_after();
              if (leader) {
#pragma unroll
                for (int k = 0; k < 4; ++k) umma_f16_ts(to, ts + k * 8, dv + k * (2048u >> 4), id_pv, j > 0 || k > 0);
              }
              __syncwarp();
              if (!wait(PFULL + rt, own >> rt)) break;
              own ^= 1u << rt;
            } else {
              if (!wait(QFULL + rt, seg >> rt)) break;
              seg ^= 1u << rt;
            }
            tc_fence_after();
            if (leader) {
              if (j >= 0) {
#pragma unroll
                for (int k = 4; k < 8; ++k) umma_f16_ts(to, ts + k * 8, dv + k * (2048u >> 4), id_pv, 1);
              }
              if (j + 1 < tiles) {
                const uint64_t dq = sw128_desc(base + L.q + rt * TB);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                  const uint32_t off = ((k >> 2) * 16384u + (k & 3) * 32u) >> 4;
                  umma_f16(ts, dq + off, dk + off, id_qk, k > 0);
                }
                umma_commit(bar(SFULL + rt));
              } else {
                umma_commit(bar(OFULL + rt));
              }
            }
            __syncwarp();
          }
        }
        kt += tiles;
      }
      // all products end before tensor memory is given back
      if (leader) {
        const uint32_t end_bar = base + L.misc + 32;
        mbar_init(end_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        umma_commit(end_bar);
        for (long long i = 0; !mbar_try(end_bar, 0) && i < kDrainLimit; ++i) {}
      }
      __syncwarp();
    } else if (warp >= 14) {
      // ============================================================== codes and scales from the cache
      // Warp 14 asks for keys, and all scales, warp 15 for values: a tile's codes as soon as the
      // products of two tiles before are done.
      const int side = warp - 14;
      const uint8_t* codes = side ? vcodes : kcodes;
      const int page = static_cast<int>(p.map.page), ppb = page / kKv8Block, num_pages = static_cast<int>(p.map.num_pages);
      int kt = 0;
      bool ok = true;
      for (int seg = 0;; ++seg) {
        ok = wait_for(DFULL + (seg & 1), seg >> 1);
        if (!ok) break;
        const Run& run = s_meta[seg & 1].run;
        const int tiles = run.tiles, b = run.b, head = run.h;
        const int b_lo = run.lo / kKv8Block, b_hi = (run.hi - 1) / kKv8Block;
        int blk = run.t0 / kKv8Block + lane % kBlocks;       // lane k (of 8): block k of the tile
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(MEMPTY + (seg & 1)));
        if (tiles == 0) break;
        const int32_t* row = p.map.table ? p.map.table + static_cast<int64_t>(b) * p.map.max_pages : nullptr;
        int in;
        auto ask = [&]() {                     // the block's page and its place there
          // a block outside the visible tokens may have no page: the nearest visible one is taken
          const int c = min(max(blk, b_lo), b_hi), col = c / ppb;
          in = c - col * ppb;
          blk += kBlocks;
          return row ? __ldg(row + col) : b;
        };
        auto record = [&](int id) {
          if (id < 0 || id >= num_pages) {
            report_status(p.status, TQ_ERR_INVALID_ARG);
            id = 0;
          }
          return (id * Hkv + head) * page + in * kKv8Block;          // (a side has fewer than 2^31 records)
        };
        auto load_scale = [&](int rec) {       // lanes 0..7: key scales, 8..15: value scales
          return side == 0 && lane < 2 * kBlocks ? __ldg((lane < kBlocks ? p.kscales : p.vscales) + rec / kKv8Block) : 0.f;
        };
        int rec = record(ask());
        float scale = load_scale(rec);
        int id = ask();
        int E = 1;                             // largest value scale so far
        for (int j = 0; j < tiles; ++j, ++kt) {
          const int st = kt & 1;
          if (kt >= 2 && !(ok = wait_for((side ? VEMPTY : KEMPTY) + st, (kt >> 1) - 1))) break;
          if (side == 0) {
            // The scales' slot is free: its last readers, the softmax of four tiles before, are done,
            // because the first product of two tiles before is.
            const int e = static_cast<int>((__float_as_uint(scale) >> 23) & 0xffu);
            E = max(E, __reduce_max_sync(0xffffffffu, lane >= kBlocks && lane < 2 * kBlocks ? e : 0));
            float* slot = s_scale + (kt % kScaleSlots) * kSlot;
            if (lane < kBlocks) slot[lane] = scale;
            else if (lane < 2 * kBlocks) {     // f: exponent of the block's probabilities
              const int f = kHead + max(e - E, -100);
              slot[lane] = static_cast<float>(f);
              slot[lane + kBlocks] = __uint_as_float(static_cast<uint32_t>(127 - f) << 23);
            } else if (lane == 2 * kBlocks) {
              slot[3 * kBlocks] = static_cast<float>(E);
            }
            __syncwarp();
          }
          // blocks that follow one another in the cache come in one copy (where they do in the tile: d = 128)
          const uint32_t full = bar((side ? VRAW : KRAW) + st);
          const int before = __shfl_up_sync(0xffffffffu, rec, 1);
          const bool head_of = lane < kBlocks && (D == 64 || lane == 0 || rec != before + kKv8Block);
          const uint32_t heads = __ballot_sync(0xffffffffu, head_of) | (1u << kBlocks);
          const int len = __ffs(heads >> (lane + 1) % 32);
          if (lane == 0) mbar_expect_tx(full, kBlocks * BB);
          __syncwarp();
          if (head_of)
            bulk_load(base + (side ? L.v : L.k) + st * TB + kRaw + lane * 2048, codes + static_cast<int64_t>(rec) * D, len * BB, full);
          rec = record(id);
          scale = load_scale(rec);
          id = ask();
        }
        if (!ok) break;
      }
      // copies still in flight land before the CTA ends (none, unless a wait gave up)
      for (int k = max(0, kt - 2); k < kt; ++k)
        for (long long i = 0; !mbar_try(bar((side ? VRAW : KRAW) + (k & 1)), (k >> 1) & 1) && i < kDrainLimit; ++i) {}
    } else {
      // ============================================================== runs, and what their rows see
      const int lt = lane;
      int seg = 0;
      for (int64_t u = u0;;) {
        Run run{};
        int len = 0;
        if (u < u1) {
          static_cast<Kv8Run&>(run) = kv8_run_at(u, u1, s_pref, VB, Hkv, run_cost(GEN));
          u += run.units;
          if (run.tiles == 0) continue;
          const int gv = p.v0 + run.v;
          run.b = gv / p.RG;
          run.r0 = (gv - run.b * p.RG) * kKv8PrefillRows;
          len = kv8_len(p.sc.kv_lens, run.b, p.map.cap, nullptr);
          group_range(run.b, run.r0, len, run.lo, run.hi, run.in_lo, run.in_hi);
          run.t0 = (run.lo / kTile + run.tile) * kTile;
        }
        const int mb = seg & 1;
        RowMeta& meta = s_meta[mb];
        if (seg >= 2 && !wait_for(MEMPTY + mb, (seg >> 1) - 1)) break;
        ++seg;
        if (lt == 0) meta.run = run;
        if (run.tiles > 0) {
          const int b = run.b;
#pragma unroll 2
          for (int rr = lt; rr < kKv8PrefillRows; rr += kScouts) {
            const int r = run.r0 + rr;
            int lo = 0, hi = INT32_MAX, pos = 0;
            float slope = 0.f;
            int i = -1, hq = 0;
            if (r < R) {
              i = r / p.G;
              hq = run.h * p.G + r - i * p.G;
              kv8_range(p.sc, b, i, p.T, len, lo, hi, pos);
              if (GEN && p.sc.slopes) slope = __ldg(p.sc.slopes + hq) * kLog2E;
            }
            meta.lo[rr] = lo;
            meta.hi[rr] = hi;
            meta.pos[rr] = pos;
            meta.slope[rr] = slope;
            meta.i[rr] = i;
            meta.hq[rr] = hq;
          }
        }
        mbar_arrive(bar(DFULL + mb));
        if (run.tiles == 0) break;
      }
      if (lane == 0) kv8_plan_split(p.plan, blockIdx.x, u0, u1, per, s_pref, VB, Hkv, run_cost(GEN));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) report_status(p.status, kDevTimeout);
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the partial results of a (256-row group, key head) that several CTAs worked on, one warp a
// row: out = sum_c w_c out_c / sum_c w_c, w_c = 2^(lse_c - max).  Blocks x: the CTAs' boundaries.
template <int D>
__global__ void __launch_bounds__(256) kv8_prefill_join_kernel(const Kv8AttnParams p) {
  pdl_wait();
  pdl_trigger();
  const int4 split = __ldcg(reinterpret_cast<const int4*>(p.plan) + blockIdx.x + 1);
  if (split.x < 0) return;
  const int h = split.y, c0 = split.z, c1 = split.w;
  const int gv = p.v0 + split.x, b = gv / p.RG, r0 = (gv - b * p.RG) * kKv8PrefillRows, R = p.T * p.G;
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
  bool bad = false;                          // a NaN among the scores stays one
  for (int c = c0 + lane; c <= c1; c += 32) {
    const float x = __ldcg(p.part_lse + prow(c));
    bad |= x != x;
    mx = fmaxf(mx, x);
  }
  mx = warp_max(mx);
  bad = __any_sync(0xffffffffu, bad);
  if (mx > -INFINITY)
    for (int c = c0; c <= c1; ++c) {
      const float w = ex2(__ldcg(p.part_lse + prow(c)) - mx);
      sum += w;
      const float* src = p.part_o + prow(c) * D + lane * PL;
#pragma unroll
      for (int k = 0; k < PL; ++k) o[k] += w * __ldcg(src + k);
    }
  const float inv = bad ? NAN : sum > 0.f ? 1.f / sum : 0.f;
  if (p.lse && lane == 0) p.lse[row] = bad ? NAN : sum > 0.f ? (mx + __log2f(sum)) * kLn2 : -INFINITY;
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
  // the roles' register shares must fit what the launch has, or their exchange would not end
  static std::atomic<uint64_t> seen{0};
  static std::atomic<int> regs{0};
  cudaError_t e = cudaSuccess;
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, k)) != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) < kRegsLaunch) return cudaErrorLaunchOutOfResources;
  e = allow_smem(k, smem, seen);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3(grid), dim3(kThreads), smem, s, kc, vc, p);
  if (e != cudaSuccess || grid == 1) return e;
  return launch_pdl(kv8_prefill_join_kernel<D>, dim3(grid - 1, kKv8PrefillRows / 8), dim3(256), 0, s, p);
}

}  // namespace

cudaError_t launch_kv8_prefill(const uint8_t* kcodes, const uint8_t* vcodes, const Kv8AttnParams& p, int d, int grid,
                               cudaStream_t s) {
  const bool gen = p.sc.cap > 0.f || p.sc.slopes;
  if (d == 128) return gen ? go<128, true>(kcodes, vcodes, p, grid, s) : go<128, false>(kcodes, vcodes, p, grid, s);
  return gen ? go<64, true>(kcodes, vcodes, p, grid, s) : go<64, false>(kcodes, vcodes, p, grid, s);
}

}  // namespace tq

// Attention of up to 16 query rows a key head over the 8-bit block-scaled cache: decode steps,
// short query blocks, and fp32 queries of any length in groups of 16 rows.
//
//   l_t = scale q.k^_t (capped, biased),  out = sum_t softmax(l)_t v^_t,  lse = ln sum_t e^{l_t}
//
// Bytes bound it: each token of a key head is 2 d codes and 2 / 16 scales, read once for all its
// query rows (d = 128, eight sequences of 131072 tokens: 322 us, 6.7 TB/s).  Tiles of 8 KB of codes
// (32 tokens at d = 128, 64 at d = 64) of all (sequence, key head) pairs form one line that is cut
// into equal parts, so ragged lengths and few long sequences load every SM alike: a part for each
// CTA, whose warps take its tiles in turn, or one for each warp (the rule stands in plan_attn).  A
// pair that one part covers is finished there; the others leave at most two partial results a part,
// joined by a second, small kernel.  In the line a pair has a few tiles' length more than its own,
// for what a run costs beside them.
//
// The warps work without meeting: each keeps its own ring of tiles, copied by the tensor-map engine
// into swizzled rows (the swizzle frees the reads of the value operand from bank conflicts).  What
// bounds a warp is the latency of its instructions, hence twelve where registers allow (eight: 400
// us in place of 345 at 131072 tokens).  A tile's scores are S^T = K Q^T with 16 tokens as the rows
// of an m16n8k16 product and eight query rows as its columns, so small groups of query heads waste
// little of it (the tensor-memory instructions' 128 rows would be nine tenths empty); then
// O^T += V^T P^T with the dims as rows.  Codes become halves (exact) on the way into the registers.
// The order of the 16 dims of a step is free, as long as q has it too: a lane reads 16 consecutive
// bytes of a row.
//
// Number ranges.  q is divided by a power of two a row so that its largest entry is in [1, 2) as
// a half (entries below 2^-14 of it round to 2^-25 of it).  A value block's scale 2^e joins its
// probabilities: P = p 2^(15 + e - E) with E the largest e so far, in halves of 11 bits down to
// p 2^(e - E) = 2^-29.  fp32 queries take q and P as two halves each (22 bits).  Scores, maxima,
// sums and outputs are fp32.
#include <cuda_runtime.h>

#include "kv8_launch.h"
#include "launchers.h"
#include "quantize_umma.cuh"

namespace tq {
namespace {

// Tokens of a tile: what it costs a warp beside its tokens is shared by 8 KB of codes.
__host__ __device__ constexpr int tile_of(int D) { return kv8_decode_tile(D); }
__host__ __device__ constexpr int warps_of(int NT, int W) { return kv8_decode_warps(8 * NT, W == 2); }
constexpr int kMinTiles = 8;               // a CTA's tiles, where there is little work
// Outputs of 8 * NT rows on their way to the sum over the warps: a lane of the product holds two
// neighbouring dims of row 2 (lane % 4) + c and eighth lane / 4 of the dims; the padding keeps the
// lanes' banks apart.
__host__ __device__ constexpr int eighth(int D) { return D / 8 + 2; }
__host__ __device__ constexpr int out_stride(int D) { return 8 * eighth(D) + 4; }

__host__ __device__ constexpr int ring_stages(int NT, int W) { return warps_of(NT, W) == 8 ? 3 : 2; }
__host__ __device__ constexpr uint32_t stage_bytes(int D) { return 2u * tile_of(D) * D; }

struct DecodeSmem {
  uint32_t scales, bars, lo, hi, pref, ml, fin, o, total;
};
__host__ __device__ constexpr DecodeSmem decode_smem(int D, int NT, int W) {
  const int ns = NT == 2 ? 2 : ring_stages(NT, W), kWarps = warps_of(NT, W);
  DecodeSmem L{};
  uint32_t at = kWarps * ns * stage_bytes(D);
  L.o = at; at += 4u * 8 * NT * out_stride(D) * 4;             // four warps' outputs
  L.scales = at; at += kWarps * ns * (tile_of(D) / kKv8Block) * 8;
  L.bars = at; at += kWarps * ns * 8;
  L.ml = at; at += kWarps * (16 * 2 + 1) * 4;                  // m, l of 16 rows and E
  L.fin = at; at += 16 * 2 * 4;                                // 1 / sum and lse of 16 rows
  L.lo = at; at += kKv8DecodeMaxVB * 4;
  L.hi = at; at += kKv8DecodeMaxVB * 4;
  L.pref = at; at += (kKv8DecodeMaxVB + 1) * 4;
  L.total = at + 16 + 1024;                                    // abort flag, alignment
  return L;
}
static_assert(decode_smem(128, 1, 1).total <= 232448 && decode_smem(128, 1, 2).total <= 232448 &&
              decode_smem(128, 2, 1).total <= 232448 && decode_smem(64, 1, 1).total <= 232448, "shared memory");

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ float h_lo(float x) { return x - __half2float(__float2half_rn(x)); }

// Address of byte `off` (16-byte chunk aligned) of row r in a tile of rows of D bytes, as the
// tensor-map engine swizzles them: 16-byte chunks XORed with the row within 8 rows of 128 bytes
// (D = 128) or with the pair of rows within 8 of 64 bytes (D = 64).
template <int D>
__device__ __forceinline__ uint32_t swz(int r, uint32_t off) {
  return D == 128 ? r * 128u + (off ^ ((r & 7u) << 4)) : r * 64u + (off ^ (((r >> 1) & 3u) << 4));
}

// Four outputs at element `at`; W == 2: fp32.
template <int W>
__device__ __forceinline__ void store4(void* out, int dtype, int64_t at, float2 x, float2 y) {
  if (W == 2) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(x.x, x.y, y.x, y.y);
  } else if (dtype == TQ_BF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(y.x, y.y);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack_h2(x.x, x.y), pack_h2(y.x, y.y));
  }
}

// TEAM: a CTA's warps share each run, else each warp has runs of its own.
template <int D, int NT, int W, bool TEAM>
__global__ void __launch_bounds__(warps_of(NT, W) * 32, 1)
kv8_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const Kv8AttnParams p) {
  constexpr int NS = NT == 2 ? 2 : ring_stages(NT, W), kWarps = warps_of(NT, W);
  constexpr int STEP = TEAM ? kWarps : 1;  // a warp takes every STEP-th tile of its runs
  constexpr uint32_t SB = stage_bytes(D);
  constexpr int kTile = tile_of(D), NB = kTile / kKv8Block;            // tokens and blocks of a tile
  constexpr DecodeSmem L = decode_smem(D, NT, W);
  constexpr int KJ = D / 64;               // 64-dim halves of a row
  constexpr int MT = D / 16;               // 16-dim rows of the output product
  extern __shared__ unsigned char dsm_raw[];
  const uint32_t raw = smem_u32(dsm_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* sm = dsm_raw + (base - raw);
  int* s_lo = reinterpret_cast<int*>(sm + L.lo);         // visible tokens [lo, hi) of a virtual sequence
  int* s_hi = reinterpret_cast<int*>(sm + L.hi);
  int* s_pref = reinterpret_cast<int*>(sm + L.pref);
  float* s_ml = reinterpret_cast<float*>(sm + L.ml);
  float* s_o = reinterpret_cast<float*>(sm + L.o);
  float* s_fin = reinterpret_cast<float*>(sm + L.fin);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L.total - 1024 - 16);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, qd = lane & 3;
  const uint32_t ring = base + warp * NS * SB;
  const uint32_t bar0 = base + L.bars + warp * NS * 8;
  const uint32_t sc0 = base + L.scales + warp * NS * NB * 8;
  const int ppb = static_cast<int>(p.map.page / kKv8Block);
  if (lane == 0) {                           // (each warp's own barriers; the fence is for the thread's own)
    for (int s = 0; s < NS; ++s) mbar_init(bar0 + 8 * s, 1 + 2 * NB);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 0) *abort_flag = 0;
  if (!p.appended) pdl_wait();               // (behind an append nothing that it writes is read before the second wait)

  // ---- how the work is cut
  const int VB = p.VB, Hkv = p.map.Hkv, R = p.T * p.G;
  for (int v = tid; v < VB; v += kWarps * 32) {
    const int gv = p.v0 + v, b = gv / p.RG, r0 = (gv - b * p.RG) * kKv8DecodeRows;
    const int len = kv8_len(p.sc.kv_lens, b, p.map.cap, p.status);
    int lo = INT32_MAX, hi = 0;
    const int i1 = min(R - 1, r0 + kKv8DecodeRows - 1) / p.G;
    for (int i = r0 / p.G; i <= i1; ++i) {
      int a, z, pos;
      kv8_range(p.sc, b, i, p.T, len, a, z, pos);
      if (z > a) { lo = min(lo, a); hi = max(hi, z); }
    }
    s_lo[v] = hi > 0 ? lo : 0;
    s_hi[v] = hi;
    s_pref[v + 1] = hi > 0 ? (hi + kTile - 1) / kTile - lo / kTile + p.run_cost : 0;
  }
  __syncthreads();
  if (warp == 0) kv8_prefix(s_pref, VB);
  __syncthreads();
  const int64_t total = static_cast<int64_t>(s_pref[VB]) * Hkv;
  // Neighbouring parts of the line go to different SMs, so that a short one is spread over all.
  const int parts = TEAM ? gridDim.x : gridDim.x * kWarps, part = TEAM ? blockIdx.x : warp * gridDim.x + blockIdx.x;
  const int64_t per = max((total + parts - 1) / parts, static_cast<int64_t>(TEAM ? kMinTiles : 1));
  const int64_t u0 = min(total, per * part), u1 = min(total, u0 + per);
  if (p.appended) pdl_wait();
  pdl_trigger();

  // ---- issue side: the warp's share of the tiles of the CTA's runs
  int64_t iu = u0;
  Kv8Run ir{};
  int ij = TEAM ? warp : 0, issued = 0, used = 0;
  // Lane k (of NB) follows block k of the warp's tiles: its page's column and its place in the page.
  int blk = 0, col = 0, in = 0, b_lo = 0, b_hi = 0, seq = 0;
  const int32_t* row = nullptr;
  const int step_col = STEP * NB / ppb, step_in = STEP * NB - step_col * ppb;
  struct Next {                              // the warp's next tile: page and place of the lane's block, key head
    int id, place, h;                        // h < 0: no more
  };
  auto ask = [&]() {
    Next n{0, 0, -1};
    if (iu >= u1) return n;                  // (asked again behind the last tile)
    bool moved = false;
    while (ij >= ir.tiles) {
      ij -= ir.tiles;
      iu += ir.units;
      if (iu >= u1) return n;
      ir = kv8_run_at(iu, u1, s_pref, VB, Hkv, p.run_cost);
      moved = true;
    }
    if (moved) {
      const int lo = s_lo[ir.v];
      seq = (p.v0 + ir.v) / p.RG;
      b_lo = lo / kKv8Block;
      b_hi = (s_hi[ir.v] - 1) / kKv8Block;
      row = p.map.table ? p.map.table + static_cast<int64_t>(seq) * p.map.max_pages : nullptr;
      blk = (lo / kTile + ir.tile + ij) * NB + lane % NB;
      col = blk / ppb;
      in = blk - col * ppb;
    } else {
      blk += STEP * NB;
      col += step_col;
      in += step_in;
      if (in >= ppb) {
        in -= ppb;
        ++col;
      }
    }
    int c = col;
    n.place = in;
    if (blk < b_lo || blk > b_hi) {          // it may have no page: the nearest visible block instead
      const int x = blk < b_lo ? b_lo : b_hi;
      c = x / ppb;
      n.place = x - c * ppb;
    }
    n.id = row ? __ldg(row + c) : seq;
    n.h = ir.h;
    ij += STEP;
    return n;
  };
  auto issue = [&](Next n) {
    if (n.h < 0) return;
    const int st = issued % NS;
    const uint32_t bar = bar0 + 8 * st, dst = ring + st * SB;
    if (n.id < 0 || n.id >= p.map.num_pages) {
      report_status(p.status, TQ_ERR_INVALID_ARG);
      n.id = 0;
    }
    // (a side has fewer than 2^31 records)
    const int rec = (n.id * Hkv + n.h) * static_cast<int>(p.map.page) + n.place * kKv8Block;
    if (lane == 0) mbar_expect_tx(bar, SB);
    __syncwarp();
    if (lane < 2 * NB) {
      if (lane < NB) {
        tma_load_2d(dst + lane * kKv8Block * D, &kmap, 0, rec, bar);
        tma_load_2d(dst + (kTile + lane * kKv8Block) * D, &vmap, 0, rec, bar);
      }
      const float* src = (lane < NB ? p.kscales : p.vscales) + rec / kKv8Block;
      const uint32_t to = sc0 + (st * 2 * NB + lane) * 4;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(src) : "memory");
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
    }
    __syncwarp();
    ++issued;
  };
  Next next;
  {
    Next n[NS];                              // (all asked for before the first is needed)
#pragma unroll
    for (int s = 0; s < NS; ++s) n[s] = ask();
    next = ask();
#pragma unroll
    for (int s = 0; s < NS; ++s) issue(n[s]);
  }

  // ---- consume side, one (sequence, key head) at a time
  int cj = TEAM ? warp : 0;
  bool dead = false;
  for (int64_t u = u0; u < u1;) {
    const Kv8Run sp = kv8_run_at(u, u1, s_pref, VB, Hkv, p.run_cost);
    u += sp.units;
    if (sp.tiles == 0) continue;
    const int gv = p.v0 + sp.v, b = gv / p.RG, r0 = (gv - b * p.RG) * kKv8DecodeRows;
    const int len = kv8_len(p.sc.kv_lens, b, p.map.cap, nullptr);

    // the query rows as the columns of the score product: row nt * 8 + g
    uint32_t qf[W][NT][KJ * 8];
    float qs[NT];                              // of row nt * 8 + g, then of this lane's score columns
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + nt * 8 + g;
      float x[KJ][16];
      float mx = 0.f;
      const bool on = r < R;
      const int i = on ? r / p.G : 0, hq = sp.h * p.G + (on ? r - i * p.G : 0);
      const int64_t at = b * p.q_stride_b + hq * p.q_stride_h + i * p.q_stride_t;
#pragma unroll
      for (int j = 0; j < KJ; ++j)
#pragma unroll
        for (int k = 0; k < 16; k += 8) {
          const int64_t e = at + 64 * j + 16 * qd + k;
          if (!on) {
#pragma unroll
            for (int z = 0; z < 8; ++z) x[j][k + z] = 0.f;
          } else if (W == 2) {
            const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + e);
            const float4 a = __ldg(s), c = __ldg(s + 1);
            x[j][k] = a.x; x[j][k + 1] = a.y; x[j][k + 2] = a.z; x[j][k + 3] = a.w;
            x[j][k + 4] = c.x; x[j][k + 5] = c.y; x[j][k + 6] = c.z; x[j][k + 7] = c.w;
          } else {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + e));
            const uint32_t w4[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              float2 f;
              if (p.dtype == TQ_BF16) f = make_float2(__uint_as_float(w4[z] << 16), __uint_as_float(w4[z] & 0xffff0000u));
              else f = __half22float2(*reinterpret_cast<const __half2*>(&w4[z]));
              x[j][k + 2 * z] = f.x;
              x[j][k + 2 * z + 1] = f.y;
            }
          }
        }
#pragma unroll
      for (int j = 0; j < KJ; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) mx = fmaxf(mx, fabsf(x[j][k]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23), 1), 253);
      const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
      qs[nt] = __uint_as_float(static_cast<uint32_t>(e) << 23) * p.sc.scale_log2;
#pragma unroll
      for (int j = 0; j < KJ; ++j)
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const float a = x[j][k] * down, c = x[j][k + 1] * down;
          qf[0][nt][j * 8 + k / 2] = pack_h2(a, c);
          if constexpr (W == 2) qf[1][nt][j * 8 + k / 2] = pack_h2(h_lo(a), h_lo(c));
        }
    }
    // this lane's score columns: rows nt * 8 + 2 qd + c
    float cs[NT][2], slope[NT][2], m[NT][2], l[NT][2];
    int lo[NT][2], hi[NT][2], pos[NT][2];
    int in_lo = 0, in_hi = INT32_MAX;            // tokens that every row sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        cs[nt][c] = __shfl_sync(0xffffffffu, qs[nt], (2 * qd + c) * 4);
        const int r = r0 + nt * 8 + 2 * qd + c;
        lo[nt][c] = hi[nt][c] = pos[nt][c] = 0;
        slope[nt][c] = 0.f;
        if (r < R) {
          const int i = r / p.G;
          kv8_range(p.sc, b, i, p.T, len, lo[nt][c], hi[nt][c], pos[nt][c]);
          if (p.sc.slopes) slope[nt][c] = __ldg(p.sc.slopes + sp.h * p.G + r - i * p.G) * kLog2E;
          in_lo = max(in_lo, lo[nt][c]);
          in_hi = min(in_hi, hi[nt][c]);
        }
        m[nt][c] = -INFINITY;
        l[nt][c] = 0.f;
      }
    in_lo = __reduce_max_sync(0xffffffffu, in_lo);
    in_hi = __reduce_min_sync(0xffffffffu, in_hi);
    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][nt][k] = 0.f;
    int E = 1;                                   // largest value-scale exponent so far (biased)

    for (; cj < sp.tiles; cj += STEP) {
      const int st = used % NS;
      const uint32_t bar = bar0 + 8 * st, ks_a = ring + st * SB, vs_a = ks_a + kTile * D;
      if (!dead && !mbar_wait(bar, (used / NS) & 1, p.wait_limit, p.status, abort_flag)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      if (dead) continue;
      ++used;
      const int t0 = (s_lo[sp.v] / kTile + sp.tile + cj) * kTile;
      const bool masked = t0 < in_lo || t0 + kTile > in_hi;
      float ksc[NB], vsc[NB];                    // scales of the blocks
#pragma unroll
      for (int i = 0; i < NB; i += 2) {
        asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(ksc[i]), "=f"(ksc[i + 1]) : "r"(sc0 + (st * 2 * NB + i) * 4));
        asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(vsc[i]), "=f"(vsc[i + 1]) : "r"(sc0 + (st * 2 * NB + NB + i) * 4));
      }

      // scores
      float s[NB][NT][4];
#pragma unroll
      for (int bl = 0; bl < NB; ++bl) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[bl][nt][k] = 0.f;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          const int row = bl * 16 + g;
          const uint4 ka = lds128(ks_a + swz<D>(row, 64 * j + 16 * qd));
          const uint4 kb = lds128(ks_a + swz<D>(row + 8, 64 * j + 16 * qd));
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a0 = e4m3x2_to_h2(wa[k]), a1 = e4m3x2_to_h2(wb[k]);
            const uint32_t a2 = e4m3x2_to_h2(wa[k] >> 16), a3 = e4m3x2_to_h2(wb[k] >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(s[bl][nt], a0, a1, a2, a3, qf[0][nt][j * 8 + 2 * k], qf[0][nt][j * 8 + 2 * k + 1]);
              if constexpr (W == 2)
                mma_f16(s[bl][nt], a0, a1, a2, a3, qf[1][nt][j * 8 + 2 * k], qf[1][nt][j * 8 + 2 * k + 1]);
            }
          }
        }
      }
      // Capped ones: most are below half the cap, and where all are the series alone does (the same bits either way).
      if (p.sc.cap > 0.f) {
        const float in = kLn2 / p.sc.cap, out = p.sc.cap * kLog2E;
        float far = 0.f;
#pragma unroll
        for (int bl = 0; bl < NB; ++bl)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const float2 z = mul2(mul2(pair(s[bl][nt][k], s[bl][nt][k + 1]), pair(ksc[bl] * cs[nt][0], ksc[bl] * cs[nt][1])), both(in));
              s[bl][nt][k] = z.x;
              s[bl][nt][k + 1] = z.y;
              far = fmaxf(far, fmaxf(fabsf(z.x), fabsf(z.y)));
            }
        const bool near = __all_sync(0xffffffffu, far <= 0.5f);
#pragma unroll
        for (int bl = 0; bl < NB; ++bl)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const float2 z = pair(s[bl][nt][k], s[bl][nt][k + 1]);
              const float2 y = near ? kv8_cap_series(z, out) : kv8_cap(z, out);
              s[bl][nt][k] = y.x;
              s[bl][nt][k + 1] = y.y;
            }
      }
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
      for (int bl = 0; bl < NB; ++bl) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int c = k & 1, t = t0 + bl * 16 + g + (k >> 1) * 8;
            float x = s[bl][nt][k] * (p.sc.cap > 0.f ? 1.f : ksc[bl] * cs[nt][c]);
            if (p.sc.slopes) x -= slope[nt][c] * static_cast<float>(abs(pos[nt][c] - t));
            if (masked && (t < lo[nt][c] || t >= hi[nt][c])) x = -INFINITY;
            s[bl][nt][k] = x;
            mx[nt][c] = fmaxf(mx[nt][c], x);
          }
      }
      // the running maxima, and the largest value scale
      int E1 = E;
#pragma unroll
      for (int i = 0; i < NB; ++i) E1 = max(E1, static_cast<int>((__float_as_uint(vsc[i]) >> 23) & 0xffu));
      bool grown = E1 > E;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx[nt][c] = fmaxf(mx[nt][c], __shfl_xor_sync(0xffffffffu, mx[nt][c], o));
          grown |= mx[nt][c] > m[nt][c];
        }
      if (__any_sync(0xffffffffu, grown)) {
        const float de = ex2(static_cast<float>(E - E1));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float nm = fmaxf(m[nt][c], mx[nt][c]);
            const float a = nm == -INFINITY ? 1.f : ex2(m[nt][c] - nm);
            m[nt][c] = nm;
            l[nt][c] *= a;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              acc[i][nt][c] *= a * de;
              acc[i][nt][2 + c] *= a * de;
            }
          }
        E = E1;
      }
      // probabilities, times their block's value scale, as the second product's columns
      uint32_t pf[W][NB][NT][2];
#pragma unroll
      for (int bl = 0; bl < NB; ++bl) {
        const int ev = static_cast<int>((__float_as_uint(vsc[bl]) >> 23) & 0xffu) - E;
        const float f = ev < -120 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + 15 + ev) << 23);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w4[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float nm = m[nt][k & 1];
            const float x = ex2(s[bl][nt][k] - (nm == -INFINITY ? 0.f : nm));
            l[nt][k & 1] += x;
            w4[k] = x * f;
          }
          pf[0][bl][nt][0] = transpose8(pack_h2(w4[0], w4[1]));
          pf[0][bl][nt][1] = transpose8(pack_h2(w4[2], w4[3]));
          if constexpr (W == 2) {
            pf[1][bl][nt][0] = transpose8(pack_h2(h_lo(w4[0]), h_lo(w4[1])));
            pf[1][bl][nt][1] = transpose8(pack_h2(h_lo(w4[2]), h_lo(w4[3])));
          }
        }
      }
      // O^T += V^T P^T: lane g holds dims (D / 8) g .. of the four tokens 2 qd, + 1, + 8, + 9
#pragma unroll
      for (int bl = 0; bl < NB; ++bl) {
        constexpr int VW = D / 32;             // words a lane and token
        uint32_t v4[4][VW];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = bl * 16 + 2 * qd + (k & 1) + (k >> 1) * 8;
          if constexpr (D == 128) {
            const uint4 x = lds128(vs_a + swz<D>(row, 16 * g));
            v4[k][0] = x.x; v4[k][1] = x.y; v4[k][2] = x.z; v4[k][3] = x.w;
          } else {
            const uint2 x = lds64(vs_a + swz<D>(row, (8 * g) & ~15) + ((8 * g) & 15));
            v4[k][0] = x.x; v4[k][1] = x.y;
          }
          if (masked)                          // a masked token's NaN stays out of the other rows
#pragma unroll
            for (int z = 0; z < VW; ++z) v4[k][z] = e4m3_nan_to_zero(v4[k][z]);
        }
#pragma unroll
        for (int z = 0; z < VW; ++z) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7362u : 0x5140u;
            const uint32_t x = __byte_perm(v4[0][z], v4[1][z], sel), y = __byte_perm(v4[2][z], v4[3][z], sel);
            const uint32_t a0 = e4m3x2_to_h2(x), a1 = e4m3x2_to_h2(x >> 16);
            const uint32_t a2 = e4m3x2_to_h2(y), a3 = e4m3x2_to_h2(y >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(acc[2 * z + half][nt], a0, a1, a2, a3, pf[0][bl][nt][0], pf[0][bl][nt][1]);
              if constexpr (W == 2)
                mma_f16(acc[2 * z + half][nt], a0, a1, a2, a3, pf[1][bl][nt][0], pf[1][bl][nt][1]);
            }
          }
        }
      }
      __syncwarp();
      issue(next);                              // into the stage just read
      next = ask();
    }

    cj -= sp.tiles;
    const bool whole = sp.tiles == sp.n;
    const int slot = part * 2 + (sp.tile == 0 ? 1 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], o);
    if constexpr (!TEAM) {
      // ---- the warp's result: a lane has D / 8 neighbouring dims of each of its rows
      const float unit = __uint_as_float(static_cast<uint32_t>(E) << 23);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int rl = nt * 8 + 2 * qd + c, r = r0 + rl, col = (D / 8) * g;
          if (r >= R) continue;
          const float inv = l[nt][c] == 0.f ? 0.f : 1.f / (l[nt][c] * 32768.f);
          const float ls2 = l[nt][c] == 0.f ? -INFINITY : m[nt][c] + __log2f(l[nt][c]);
          const int i = r / p.G;
          const int64_t row = (static_cast<int64_t>(b) * p.Hq + sp.h * p.G + (r - i * p.G)) * p.T + i;
          if (g == 0) {
            if (!whole) p.part_lse[slot * kKv8DecodeRows + rl] = ls2;
            else if (p.lse) p.lse[row] = ls2 * kLn2;
          }
          // (in units of 2^(E - 127 - 15); two factors, so that neither leaves the normal range)
#pragma unroll
          for (int k = 0; k < MT; k += 2) {
            const float2 x = make_float2(acc[k][nt][c] * inv * unit, acc[k][nt][2 + c] * inv * unit);
            const float2 y = make_float2(acc[k + 1][nt][c] * inv * unit, acc[k + 1][nt][2 + c] * inv * unit);
            if (whole) store4<W>(p.out, p.dtype, row * D + col + 2 * k, x, y);
            else
              *reinterpret_cast<float4*>(p.part_o + (static_cast<int64_t>(slot) * kKv8DecodeRows + rl) * D + col + 2 * k) =
                  make_float4(x.x, x.y, y.x, y.y);
          }
        }
    } else {
      // ---- join the warps: common maximum and value scale, then sums in a fixed order
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (g == 0) {
            s_ml[warp * 33 + nt * 8 + 2 * qd + c] = m[nt][c];
            s_ml[warp * 33 + 16 + nt * 8 + 2 * qd + c] = l[nt][c];
          }
        }
      if (lane == 0) s_ml[warp * 33 + 32] = static_cast<float>(E);
      __syncthreads();
      float Em = 1.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) Em = fmaxf(Em, s_ml[w * 33 + 32]);
      const float unit = __uint_as_float(static_cast<uint32_t>(Em) << 23);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = nt * 8 + 2 * qd + c;
          float mm = -INFINITY, ll = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_ml[w * 33 + r]);
          const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) ll += s_ml[w * 33 + 16 + r] * ex2(s_ml[w * 33 + r] - ref);
          if (warp == 0 && g == 0) {
            s_fin[2 * r] = ll == 0.f ? 0.f : 1.f / (ll * 32768.f);
            s_fin[2 * r + 1] = ll == 0.f ? -INFINITY : mm + __log2f(ll);
          }
          const float a = ex2(m[nt][c] - ref + (static_cast<float>(E) - Em));
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            acc[i][nt][c] *= a;
            acc[i][nt][2 + c] *= a;
          }
        }
      // The last four warps leave their outputs, four by four the others add theirs to them; then every
      // thread sums four.
      constexpr int RS = out_stride(D);
#pragma unroll
      for (int four = kWarps / 4 - 1; four >= 0; --four) {
        if (warp / 4 == four) {
          float* o = s_o + (warp & 3) * 8 * NT * RS + eighth(D) * g;
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float2* at = reinterpret_cast<float2*>(o + (nt * 8 + 2 * qd + c) * RS + 2 * i);
                float2 x = make_float2(acc[i][nt][c], acc[i][nt][2 + c]);
                if (four < kWarps / 4 - 1) {
                  x.x += at->x;
                  x.y += at->y;
                }
                *at = x;
              }
        }
        __syncthreads();
      }
      for (int e = tid; e < 8 * NT * (D / 4); e += kWarps * 32) {
        const int rl = e / (D / 4), col = (e - rl * (D / 4)) * 4, r = r0 + rl;
        if (r >= R) break;
        const float* o = s_o + rl * RS + eighth(D) * (col / (D / 8)) + col % (D / 8);
        float2 x = make_float2(0.f, 0.f), y = x;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 a = *reinterpret_cast<const float2*>(o + w * 8 * NT * RS);
          const float2 c = *reinterpret_cast<const float2*>(o + w * 8 * NT * RS + 2);
          x.x += a.x; x.y += a.y; y.x += c.x; y.y += c.y;
        }
        // the sums are in units of 2^(Em - 127 - 15); two factors, so that neither leaves the normal range
        const float inv = s_fin[2 * rl], ls2 = s_fin[2 * rl + 1];
        x.x = x.x * inv * unit; x.y = x.y * inv * unit; y.x = y.x * inv * unit; y.y = y.y * inv * unit;
        if (whole) {
          const int i = r / p.G;
          const int64_t row = (static_cast<int64_t>(b) * p.Hq + sp.h * p.G + (r - i * p.G)) * p.T + i;
          if (p.lse && col == 0) p.lse[row] = ls2 * kLn2;
          store4<W>(p.out, p.dtype, row * D + col, x, y);
        } else {
          if (col == 0) p.part_lse[slot * kKv8DecodeRows + rl] = ls2;
          *reinterpret_cast<float4*>(p.part_o + (static_cast<int64_t>(slot) * kKv8DecodeRows + rl) * D + col) =
              make_float4(x.x, x.y, y.x, y.y);
        }
      }
    }
  }
  if (part > 0 && (TEAM ? tid : lane) == 0) kv8_plan_split(p.plan, part, u0, u1, per, s_pref, VB, Hkv, p.run_cost);
  // ---- groups that see nothing
  for (int v = blockIdx.x; v < VB; v += gridDim.x) {
    if (s_pref[v + 1] != s_pref[v]) continue;
    const int gv = p.v0 + v, b = gv / p.RG, r0 = (gv - b * p.RG) * kKv8DecodeRows, n = min(R - r0, kKv8DecodeRows);
    for (int e = tid; e < Hkv * n * (D / 4); e += kWarps * 32) {
      const int hr = e / (D / 4), h = hr / n, r = r0 + hr - h * n, i = r / p.G, col = (e - hr * (D / 4)) * 4;
      const int64_t row = (static_cast<int64_t>(b) * p.Hq + h * p.G + (r - i * p.G)) * p.T + i;
      if (p.lse && col == 0) p.lse[row] = -INFINITY;
      store4<W>(p.out, p.dtype, row * D + col, make_float2(0.f, 0.f), make_float2(0.f, 0.f));
    }
  }
  // copies still in flight land before the CTA ends (none, unless a wait gave up)
  for (; used < issued; ++used)
    for (long long i = 0; !mbar_try(bar0 + 8 * (used % NS), (used / NS) & 1) && i < kDrainLimit; ++i) {}
}

// Joins the partial results of a (virtual sequence, key head) that several CTAs worked on:
// out = sum_c w_c out_c / sum_c w_c, w_c = 2^(lse_c - max).  Blocks: the CTAs' boundaries.
template <int D>
__global__ void __launch_bounds__(256) kv8_decode_join_kernel(const Kv8AttnParams p) {
  pdl_wait();
  pdl_trigger();
  const int4 split = __ldcg(reinterpret_cast<const int4*>(p.plan) + blockIdx.x + 1);
  if (split.x < 0) return;
  const int h = split.y, c0 = split.z, c1 = split.w;
  const int gv = p.v0 + split.x, b = gv / p.RG, r0 = (gv - b * p.RG) * kKv8DecodeRows;
  const int R = p.T * p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int PL = D / 32;                   // dims a lane
  for (int rl = warp; rl < kKv8DecodeRows && r0 + rl < R; rl += 8) {
    const int r = r0 + rl, i = r / p.G;
    const int64_t row = (static_cast<int64_t>(b) * p.Hq + h * p.G + (r - i * p.G)) * p.T + i;
    float mx = -INFINITY, sum = 0.f, o[PL];
#pragma unroll
    for (int k = 0; k < PL; ++k) o[k] = 0.f;
    auto slot_of = [&](int c) { return c * 2 + (c == c0 ? 1 : 0); };
    bool bad = false;                          // a NaN among the scores stays one
    for (int c = c0 + lane; c <= c1; c += 32) {
      const float x = __ldcg(p.part_lse + slot_of(c) * kKv8DecodeRows + rl);
      bad |= x != x;
      mx = fmaxf(mx, x);
    }
    mx = warp_max(mx);
    bad = __any_sync(0xffffffffu, bad);
    if (mx > -INFINITY) {
#pragma unroll 4
      for (int c = c0; c <= c1; ++c) {
        const int slot = slot_of(c);
        const float w = ex2(__ldcg(p.part_lse + slot * kKv8DecodeRows + rl) - mx);
        sum += w;
        const float* src = p.part_o + (static_cast<int64_t>(slot) * kKv8DecodeRows + rl) * D + lane * PL;
#pragma unroll
        for (int k = 0; k < PL; ++k) o[k] += w * __ldcg(src + k);
      }
    }
    const float inv = bad ? NAN : sum > 0.f ? 1.f / sum : 0.f;
    if (p.lse && lane == 0) p.lse[row] = bad ? NAN : sum > 0.f ? (mx + __log2f(sum)) * kLn2 : -INFINITY;
    const int64_t at = row * D + lane * PL;
#pragma unroll
    for (int k = 0; k < PL; ++k) {
      const float x = o[k] * inv;
      if (p.dtype == TQ_F32) static_cast<float*>(p.out)[at + k] = x;
      else if (p.dtype == TQ_BF16) static_cast<__nv_bfloat16*>(p.out)[at + k] = __float2bfloat16_rn(x);
      else static_cast<__half*>(p.out)[at + k] = __float2half_rn(x);
    }
  }
}

template <int D, int NT, int W, bool TEAM>
cudaError_t go(const CUtensorMap& km, const CUtensorMap& vm, const Kv8AttnParams& p, int grid, cudaStream_t s) {
  auto k = kv8_decode_kernel<D, NT, W, TEAM>;
  constexpr uint32_t smem = decode_smem(D, NT, W).total;
  static std::atomic<uint64_t> seen{0};
  cudaError_t e = allow_smem(k, smem, seen);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3(grid), dim3(warps_of(NT, W) * 32), smem, s, km, vm, p);
  const int parts = TEAM ? grid : grid * warps_of(NT, W);
  if (e != cudaSuccess || parts == 1) return e;
  return launch_pdl(kv8_decode_join_kernel<D>, dim3(parts - 1), dim3(256), 0, s, p);
}

template <int D, int NT, int W>
cudaError_t go_w(const CUtensorMap& km, const CUtensorMap& vm, const Kv8AttnParams& p, bool team, int grid, cudaStream_t s) {
  return team ? go<D, NT, W, true>(km, vm, p, grid, s) : go<D, NT, W, false>(km, vm, p, grid, s);
}

template <int D>
cudaError_t go_d(const CUtensorMap& km, const CUtensorMap& vm, const Kv8AttnParams& p, bool team, int grid, cudaStream_t s) {
  const bool two = p.T * p.G > 8;            // more than one product column block of 8 rows
  if (p.dtype == TQ_F32) return two ? go_w<D, 2, 2>(km, vm, p, team, grid, s) : go_w<D, 1, 2>(km, vm, p, team, grid, s);
  return two ? go_w<D, 2, 1>(km, vm, p, team, grid, s) : go_w<D, 1, 1>(km, vm, p, team, grid, s);
}

}  // namespace

cudaError_t launch_kv8_decode(const CUtensorMap& kmap, const CUtensorMap& vmap, const Kv8AttnParams& p, int d, bool team,
                              int grid, cudaStream_t s) {
  return d == 128 ? go_d<128>(kmap, vmap, p, team, grid, s) : go_d<64>(kmap, vmap, p, team, grid, s);
}

}  // namespace tq

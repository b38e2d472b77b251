// Decode attention over the 4-bit KV cache: one query per sequence,
//   o[b, h, :] = softmax_s(q[b, h] . k^[b, j, s] / sqrt(128)) v^[b, j, s],  j = h / (H / Hkv),
// with k^, v^ = offset + scale * code, a scale and an offset per 32 channels (kv4.cu).
//
// The codes never become scaled values: with the group's scale s_g and offset z_g of a key,
//   q . k^  = sum_g s_g (sum_{c in g} q_c code_c) + sum_g z_g qsum_g,   qsum_g = sum_{c in g} q_c
//   out_c   = sum_s (p_s s_g) (code_c - 8) + sum_s p_s z_g + 8 sum_s p_s s_g   (8: smaller numbers)
// so the tensor core multiplies codes, which 16-bit floats hold exactly, and scales touch one
// score per key and group (or one probability) instead of 32 values. A code becomes a number
// by placing its nibble under an exponent (an and-or for two codes) and taking the exponent's
// value off again (one packed add, on the otherwise idle fp32 pipe; the integer pipe has the most
// to do in the unpacking): the known way from an integer to a float without a conversion, published
// for 4-bit weights by Kim et al. 2022 ("Who Says Elephants Can't Run"). K in fp16, whose mantissa also takes a nibble 4 bits up without a
// shift (1024 + 16 code); q is scaled by a power of two per head to use fp16's whole range.
// V in bf16 (128 + code): p s_g keeps its exponent range whatever the values' size. p is rounded
// to bf16 once, for all terms of a value alike; the 16-bit product p s_g goes in as two bf16
// numbers, its rounding and the rest (8 products and 8 packed operations more for 16 keys; with
// p s_g rounded, and codes counted from the end of their range, the mean error of an output was
// 0.0050 of it, so 0.0022, of which storing it in bf16 takes 0.0016).
//
// Keys sit on the rows of the products and the group's query heads on their columns
// (m16n8k16: S^T = K q^T, out^T = V^T P^T), so that 8 heads cost what one does. The score
// tile turns into the second product's operand with two 8x8 transposes.
//
// Work: the 128-key tiles of all (sequence, KV head) pairs form one line, cut into equal
// stretches, one per CTA, whatever the lengths; a pair that lies within one stretch is
// finished there, one that is cut leaves partial results (at most two per CTA) that a small
// second kernel joins. No counter, no atomics: the same to the bit on every run.
// A CTA is four warps, each of which owns 32 keys of every tile: it copies their codes and
// scales (5 KB) into its own two-stage ring with 16-byte asynchronous copies, a tile ahead,
// and meets the other warps only when a pair's stretch ends, to merge their softmax states.
// Rows behind the last key are filled with zeros, so nothing they hold is ever read.
// Small batches take clusters instead (see CL below). 160 bytes a key and KV head. No unit is at its
// limit: DRAM 64% of the copy rate, issue slots 62%, the integer pipe 54%, the matrix pipe about
// 31%; what is left are the four warps of a scheduler, each a chain of dependent steps (scores,
// softmax, transposes, products). 64 ragged sequences of up to 8192 keys, 32 heads over 8: 98.2 us,
// 4.3 TB/s; one of 4000 keys in a cache of that capacity: 7.0 us (the kernel is chosen by the
// capacity, which the host knows: 1000 keys take 7.8 us in a cache of 32768). Measured and
// not kept: a producer warp with a ring for all warps (93 us against 90.5); before that, against
// 96 us, three stages (97), two CTAs of 200 registers (100), one of eight warps (103); and e4m3
// operands, one product of which takes as long as the two fp16 ones that it would stand for.
#include <cuda_fp16.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace blk {

namespace {

constexpr int kD = 128;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSub = 2;                             // runs of 16 keys a warp owns of every tile
constexpr int kKeys = 16 * kSub;                    // ... and their number
constexpr int kTile = kWarps * kKeys;               // keys per tile
constexpr int kCodeBytes = kKeys * kKv4Codes;       // of a warp's stage: K codes, V codes,
constexpr int kScaleBytes = kKeys * kKv4Scales;     // K scales, V scales
constexpr int kStageBytes = 2 * (kCodeBytes + kScaleBytes);
constexpr int kStages = 2;                          // per warp
constexpr int kMergeHeads = 4;                      // heads merged at a time
constexpr int kMergeFloats = kWarps * kMergeHeads * (kD + 2);
constexpr int kMinTiles = 2;                        // tiles a CTA takes at least, while there are enough
constexpr float kRescaleLog2 = 8.0f;
constexpr float kLog2e = 1.4426950408889634f;

// NT: tiles of 8 query heads (one for groups of up to 8 heads, two for up to 16)
template <int NT>
struct Cfg {
  static constexpr int kCtas = NT == 1 ? 4 : 2;  // per SM (128 or 255 registers)
  static constexpr int kSmem = kWarps * kStages * kStageBytes + kMergeFloats * 4 + kWarps * kStages * 16;
};

// What a warp's stage holds: how many of its keys are real, whose they are, and whether the
// tile is the CTA's first or last one of its pair, or the pair lies within the CTA.
struct __align__(16) TileInfo {
  int valid, b, kvh, flags;
};
constexpr int kFirst = 1, kLast = 2, kWhole = 4;

struct Kv4Params {
  HeadRows q, o;
  Kv4Cache c;
  int B, H, Hkv, window;
  int* prefix;    // [B + 1] tiles of one KV head before each sequence; then the stretches' count
  float* part_ml; // [2 * grid][G][2]
  float* part_o;  // [2 * grid][G][128]
  float sl2;
};

// The keys of sequence b: the last `window` of its lens[b] slots.
__device__ __forceinline__ void keys_of(const Kv4Params& p, int b, int& first, int& n) {
  const int len = max(0, min(p.c.lens[b], p.c.capacity));
  first = p.window > 0 ? max(0, len - p.window) : 0;
  n = len - first;
}
__device__ __forceinline__ int tiles(int keys) { return (keys + kTile - 1) / kTile; }

// How many stretches `total` tiles are cut into, where stretch c begins, whose tile x is in.
__device__ __forceinline__ int stretches(long long total, int grid) {
  return (int)max(1ll, min((long long)grid, total / kMinTiles));
}
__device__ __forceinline__ long long stretch_begin(long long total, int n, int c) { return total * c / n; }
__device__ __forceinline__ int stretch_of(long long total, int n, long long x) {
  return (int)(((x + 1) * n + total - 1) / total) - 1;
}

// One (sequence, KV head) after the other along the line of tiles.
struct Walk {
  int b, kvh, t, n_tiles, first, keys;
  __device__ __forceinline__ void enter(const Kv4Params& p) {  // from b on, the first sequence with keys
    for (;; ++b) {
      keys_of(p, b, first, keys);
      n_tiles = tiles(keys);
      if (n_tiles > 0) return;
    }
  }
  __device__ __forceinline__ void next(const Kv4Params& p) {
    t = 0;
    if (++kvh == p.Hkv) {
      kvh = 0;
      ++b;
      enter(p);
    }
  }
};

// 16 bytes global -> shared, of which the first n (16 or 0) are read and the rest are zeros. The
// cache is read once per step: evict it first.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
               "r"(n), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D = A B + C on fp16 operands
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                        const float (&c)[4]) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// The same on bf16 operands
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                         const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// The 8x8 transpose of a 16-bit fragment (lane 4 r + c holds row r, columns 2c, 2c + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// a b - c exactly, for c = the rounded product a b
__device__ __forceinline__ uint32_t rest_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b),
                                   __hneg2(*reinterpret_cast<const __nv_bfloat162*>(&c)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The codes in the nibbles at bits 0-3 and 16-19, less 8, as a pair of bf16, from 128 + code.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w, uint32_t mask) {
  const uint32_t v = and_or<0x43004300u>(w, mask), c = 0xC308C308u;
  const __nv_bfloat162 r = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The same as fp16, from 1024 + code, and for the nibbles at bits 4-7 and 20-23 (mask << 4),
// from (1024 + 16 code) / 16 - 64 (exact).
__device__ __forceinline__ uint32_t codes_f16_lo(uint32_t w, uint32_t mask) {
  const uint32_t v = and_or<0x64006400u>(w, mask), c = 0xE400E400u;
  const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t codes_f16_hi(uint32_t w, uint32_t mask_hi) {
  const uint32_t v = and_or<0x64006400u>(w, mask_hi), a = 0x2C002C00u, c = 0xD400D400u;
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&a),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <typename T>
__device__ __forceinline__ T ld(const uint8_t* p) {
  return *reinterpret_cast<const T*>(p);
}

// The key (of a warp's 16) on row r of the products: chosen so that the rows that one
// phase of a 16-byte shared load touches (two neighbouring rows for K, four even or four
// odd ones for V) are as even and odd keys, whose 64-byte rows sit on different banks.
__device__ __forceinline__ int key_of_row(int r) { return r ^ ((r >> 1) & 1); }

// CL: the CTAs of a cluster that share one (sequence, KV head), for small batches: equal shares of
// its tiles, joined through their shared memory, so that no second kernel and no workspace
// is needed. CL == 1: a stretch of the line of all tiles per CTA.
template <int NT, int CL>
__global__ void __launch_bounds__(kThreads, Cfg<NT>::kCtas) attn_kv4_kernel(const __grid_constant__ Kv4Params p) {
  pdl_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem + kWarps * kStages * kStageBytes);
  __shared__ int warp_sums[kWarps];
  __shared__ int start[3];  // b, kvh, t of the CTA's first tile
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* ring = smem + warp * kStages * kStageBytes;
  TileInfo* info = reinterpret_cast<TileInfo*>(merge + kMergeFloats) + warp * kStages;
  pdl_wait();
  const int cta = blockIdx.x, rank = CL > 1 ? (int)cluster_ctarank() : 0;
  int n_mine;
  Walk w;
  if constexpr (CL > 1) {
    w.b = cta / CL / p.Hkv;
    w.kvh = cta / CL % p.Hkv;
    keys_of(p, w.b, w.first, w.keys);
    w.n_tiles = tiles(w.keys);
    w.t = w.n_tiles * rank / CL;
    n_mine = w.n_tiles * (rank + 1) / CL - w.t;
  } else {
    // the tiles before each thread's run of sequences
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b_lo = min(p.B, tid * per), b_hi = min(p.B, b_lo + per);
    int mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
      int first, n;
      keys_of(p, b, first, n);
      mine += tiles(n);
    }
    int run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += u;
    }
    if (lane == 31) warp_sums[warp] = run;
    __syncthreads();
    int before = run - mine, all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += warp_sums[i];
      all += warp_sums[i];
    }
    const long long total = (long long)all * p.Hkv;
    const int n_str = total > 0 ? stretches(total, gridDim.x) : 0;
    const long long t_lo = cta < n_str ? stretch_begin(total, n_str, cta) : 0;
    n_mine = cta < n_str ? (int)(stretch_begin(total, n_str, cta + 1) - t_lo) : 0;
    {
      int acc = before;
      for (int b = b_lo; b < b_hi; ++b) {
        int first, n;
        keys_of(p, b, first, n);
        const int nt = tiles(n);
        if (cta == 0) p.prefix[b] = acc;
        const long long lo = (long long)acc * p.Hkv;
        if (nt > 0 && t_lo >= lo && t_lo < lo + (long long)nt * p.Hkv) {
          const int off = (int)(t_lo - lo);
          start[0] = b;
          start[1] = off / nt;
          start[2] = off % nt;
        }
        acc += nt;
      }
      if (cta == 0 && tid == kThreads - 1) {
        p.prefix[p.B] = all;
        p.prefix[p.B + 1] = n_str;
      }
    }
    __syncthreads();
    if (n_mine == 0) return;
    w.b = start[0];
    w.enter(p);
    w.kvh = start[1];
    w.t = start[2];
  }
  const int pair_b = w.b, pair_kvh = w.kvh;  // CL > 1: the cluster's pair
  float* const shared_out = reinterpret_cast<float*>(smem);  // ... and this CTA's share of it, [head][128 + 4]

  // ---- this warp's copies, a tile ahead of its products
  const uint64_t once = l2_policy_evict_first();
  // byte offset of this lane's first copy of codes: a row of codes is four lanes' copies, and a
  // row of scales, a quarter as long, one lane's
  auto row_of = [&] {
    const size_t at = ((size_t)w.b * p.Hkv + w.kvh) * p.c.capacity + w.first + w.t * kTile + warp * kKeys;
    return at * kKv4Codes + 16 * lane;
  };
  size_t row = row_of();
  int loaded = 0;
  bool first = true;
  auto load = [&](int stage) {
    if (loaded < n_mine) {
      const int valid = w.keys - w.t * kTile - warp * kKeys;
      const uint32_t dst = smem_u32(ring + stage * kStageBytes) + 16 * lane;
      const uint8_t *k = p.c.k + row, *v = p.c.v + row, *ks = p.c.k_scale + (row >> 2) + 12 * lane,
                    *vs = p.c.v_scale + (row >> 2) + 12 * lane;
      if (valid >= kKeys) {
#pragma unroll
        for (int i = 0; i < kCodeBytes / 512; ++i) {
          copy16(dst + 512 * i, k + 512 * i, 16, once);
          copy16(dst + kCodeBytes + 512 * i, v + 512 * i, 16, once);
        }
        copy16(dst + 2 * kCodeBytes, ks, 16, once);  // kKeys == 32: a row's scales per lane
        copy16(dst + 2 * kCodeBytes + kScaleBytes, vs, 16, once);
      } else {  // rows that do not exist are not read
#pragma unroll
        for (int i = 0; i < kCodeBytes / 512; ++i) {
          const bool on = (lane >> 2) + 8 * i < valid;
          copy16(dst + 512 * i, on ? k + 512 * i : p.c.k, on ? 16 : 0, once);
          copy16(dst + kCodeBytes + 512 * i, on ? v + 512 * i : p.c.v, on ? 16 : 0, once);
        }
        const bool on = lane < valid;
        copy16(dst + 2 * kCodeBytes, on ? ks : p.c.k_scale, on ? 16 : 0, once);
        copy16(dst + 2 * kCodeBytes + kScaleBytes, on ? vs : p.c.v_scale, on ? 16 : 0, once);
      }
      ++loaded;
      const bool pair_ends = w.t + 1 == w.n_tiles, last = pair_ends || loaded == n_mine;
      if (w.t == 0 || loaded == 1) first = w.t == 0;  // whether the CTA has the pair from its first tile on
      if (lane == 0)
        info[stage] = {valid, w.b, w.kvh,
                       (w.t == 0 || loaded == 1 ? kFirst : 0) | (last ? kLast : 0) | (pair_ends && first ? kWhole : 0)};
      ++w.t;
      row += (size_t)kTile * kKv4Codes;
      if (pair_ends && loaded < n_mine) {
        w.next(p);
        row = row_of();
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(i);

  const int G = p.H / p.Hkv;
  const int g = lane >> 2, tq = lane & 3;
  // this lane's rows of 16 keys: of product rows g, g + 8 (K) and of the operand pairs 2 tq,
  // 2 tq + 1, 2 tq + 8, 2 tq + 9 (V), and their places in a stage
  const int k_lo = key_of_row(g), k_hi = k_lo + 8;
  const int v_key[2] = {key_of_row(2 * tq), key_of_row(2 * tq + 1)};  // and 8 further
  const uint32_t at_k = k_lo * kKv4Codes + 16 * tq, at_ks = 2 * kCodeBytes + k_lo * kKv4Scales,
                 at_kz = at_ks + 8 + 4 * (tq & 1);
  uint32_t at_v[2], at_vs[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    at_v[i] = kCodeBytes + v_key[i] * kKv4Codes + 16 * (g >> 1);
    at_vs[i] = 2 * kCodeBytes + kScaleBytes + v_key[i] * kKv4Scales;
  }
  const uint32_t z_off = g < 4 ? 8 + 2 * g : 2 * (g - 4);  // the offset of group g, the scale of group g - 4
  const uint32_t mask = kept_constant(0x000F000Fu), mask_hi = kept_constant(0x00F000F0u);
  const uint32_t half = (g & 1) ? 0x7632u : 0x5410u;  // which bytes of a word are this row's

  uint32_t qf[NT][8][2], qz[NT][2];
  float sl2[NT][2];  // log2(e) / sqrt(128) over q's power of two, for the heads on this lane's columns
  float acc[NT][8][4], zacc[NT][4], m[NT][2], l[NT][2];
  int stage = 0, parts = 0;  // parts: stretches of pairs finished so far
  for (int it = 0; it < n_mine; ++it) {
    load(stage == 0 ? kStages - 1 : stage - 1);  // the stage that the last tile was in
    copies_wait<kStages - 1>();
    __syncwarp();
    const TileInfo ti = info[stage];
    if (ti.flags & kFirst) {
      // Q as the column operand: head g (+ 8), channels 16 i + 2 tq, + 1 and the two 8 further
      // fp16, times a power of two per head that puts the head's largest channel at 2^14
      {
        const __nv_bfloat16* qg = static_cast<const __nv_bfloat16*>(p.q.ptr) + ti.b * p.q.row;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int h = 8 * n + g;
          const __nv_bfloat16* qh = qg + (long long)(ti.kvh * G + h) * p.q.head + 2 * tq;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            qf[n][i][0] = h < G ? *reinterpret_cast<const uint32_t*>(qh + 16 * i) : 0u;
            qf[n][i][1] = h < G ? *reinterpret_cast<const uint32_t*>(qh + 16 * i + 8) : 0u;
          }
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) top = fmaxf(top, fmaxf(fabsf(bf16_lo(qf[n][i][e])), fabsf(bf16_hi(qf[n][i][e]))));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // 2^(14 - exponent of top), both powers kept normal numbers; an infinity stays one
          const int ex = min(max((int)(__float_as_uint(top) >> 23), 15), 254);  // biased
          const float up = __uint_as_float((uint32_t)(min(127 + 14 + 127 - ex, 254)) << 23);
          const float down = __uint_as_float((uint32_t)(254 - min(127 + 14 + 127 - ex, 253)) << 23);
          sl2[n][0] = p.sl2 * __shfl_sync(0xffffffffu, down, 8 * tq);
          sl2[n][1] = p.sl2 * __shfl_sync(0xffffffffu, down, 8 * tq + 4);
          float sum[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sum[j] = 0.f;
#pragma unroll
            for (int i = 2 * j; i < 2 * j + 2; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float a = bf16_lo(qf[n][i][e]) * up, b = bf16_hi(qf[n][i][e]) * up;
                const __half2 hh = __floats2half2_rn(a, b);
                qf[n][i][e] = *reinterpret_cast<const uint32_t*>(&hh);
                sum[j] += a + b;
              }
            sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
            sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
          }
          // qsum in three bf16 parts (24 bits): product columns 2 tq, 2 tq + 1 carry groups
          // 2 (tq & 1), + 1, the high part for tq < 2, the middle one above; + 8: the low part
          const float x0 = (tq & 1) ? sum[2] : sum[0], x1 = (tq & 1) ? sum[3] : sum[1];
          const float h0 = round_to<__nv_bfloat16>(x0), h1 = round_to<__nv_bfloat16>(x1);
          const float m0 = round_to<__nv_bfloat16>(x0 - h0), m1 = round_to<__nv_bfloat16>(x1 - h1);
          qz[n][0] = tq < 2 ? pack_bf16x2(h0, h1) : pack_bf16x2(m0, m1);
          qz[n][1] = tq < 2 ? pack_bf16x2(x0 - h0 - m0, x1 - h1 - m1) : 0u;
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[n][i][0] = acc[n][i][1] = acc[n][i][2] = acc[n][i][3] = 0.f;
        zacc[n][0] = zacc[n][1] = zacc[n][2] = zacc[n][3] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
      }
    }
    const uint8_t* st = ring + stage * kStageBytes;
    {
        // ---- scores S^T: rows keys, columns heads
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        float sc[kSub][NT][4];
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          const uint8_t *sk = st + at_k + u * 16 * kKv4Codes, *ss = st + at_ks + u * 16 * kKv4Scales,
                        *sz = st + at_kz + u * 16 * kKv4Scales;
          const uint32_t z_lo = ld<uint32_t>(sz), z_hi = ld<uint32_t>(sz + 8 * kKv4Scales);
          const uint2 s_lo = ld<uint2>(ss), s_hi = ld<uint2>(ss + 8 * kKv4Scales);
          const uint4 c_lo = ld<uint4>(sk), c_hi = ld<uint4>(sk + 8 * kKv4Codes);
          const uint32_t za[4] = {z_lo, z_hi, z_lo, z_hi};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_bf16(sc[u][n], za, qz[n][0], qz[n][1], zero);
          const uint32_t wl[4] = {c_lo.x, c_lo.y, c_lo.z, c_lo.w}, wh[4] = {c_hi.x, c_hi.y, c_hi.z, c_hi.w};
          const float fl[4] = {bf16_lo(s_lo.x), bf16_hi(s_lo.x), bf16_lo(s_lo.y), bf16_hi(s_lo.y)};
          const float fh[4] = {bf16_lo(s_hi.x), bf16_hi(s_hi.x), bf16_lo(s_hi.y), bf16_hi(s_hi.y)};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t xl = wl[j] >> 8, xh = wh[j] >> 8;
            const uint32_t a0[4] = {codes_f16_lo(wl[j], mask), codes_f16_lo(wh[j], mask), codes_f16_hi(wl[j], mask_hi),
                                    codes_f16_hi(wh[j], mask_hi)};
            const uint32_t a1[4] = {codes_f16_lo(xl, mask), codes_f16_lo(xh, mask), codes_f16_hi(xl, mask_hi),
                                    codes_f16_hi(xh, mask_hi)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float d[4];
              mma_f16(d, a0, qf[n][2 * j][0], qf[n][2 * j][1], zero);
              mma_f16(d, a1, qf[n][2 * j + 1][0], qf[n][2 * j + 1][1], d);
              sc[u][n][0] += fl[j] * d[0];
              sc[u][n][1] += fl[j] * d[1];
              sc[u][n][2] += fh[j] * d[2];
              sc[u][n][3] += fh[j] * d[3];
            }
          }
        }
        // ---- probabilities against a running reference, moved only when a score passes it
        // by 2^8 (exact: the softmax does not depend on the reference)
        float e[kSub][NT][4];
        auto hide = [&](float (&x)[NT][4], int u) {  // rows behind the last key
          if (ti.valid < kKeys) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (k_lo + 16 * u >= ti.valid) x[n][0] = x[n][1] = -INFINITY;
              if (k_hi + 16 * u >= ti.valid) x[n][2] = x[n][3] = -INFINITY;
            }
          }
        };
        float most = -INFINITY;
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) e[u][n][i] = fmaf(sc[u][n][i], sl2[n][i & 1], -m[n][i & 1]);
          hide(e[u], u);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            most = fmaxf(most, fmaxf(fmaxf(e[u][n][0], e[u][n][1]), fmaxf(e[u][n][2], e[u][n][3])));
        }
        if (__any_sync(0xffffffffu, most > kRescaleLog2)) {
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) e[u][n][i] = sc[u][n][i] * sl2[n][i & 1];
            hide(e[u], u);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float al[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float mx = m[n][r];
#pragma unroll
              for (int u = 0; u < kSub; ++u) mx = fmaxf(mx, fmaxf(e[u][n][r], e[u][n][r + 2]));
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              al[r] = m[n][r] == -INFINITY ? 0.f : ex2(m[n][r] - mx);
              m[n][r] = mx;
              l[n][r] *= al[r];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              zacc[n][i] *= al[i & 1];
#pragma unroll
              for (int j = 0; j < 8; ++j) acc[n][j][i] *= al[i & 1];
            }
          }
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) e[u][n][i] = fmaf(sc[u][n][i], sl2[n][i & 1], -m[n][i & 1]);
            hide(e[u], u);
          }
        }
        uint32_t pb[kSub][NT][2];  // P^T as the column operand: keys 2 tq, 2 tq + 1 (+ 8) of head g
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) e[u][n][i] = ex2(e[u][n][i]);
            l[n][0] += e[u][n][0] + e[u][n][2];
            l[n][1] += e[u][n][1] + e[u][n][3];
            pb[u][n][0] = transpose8(pack_bf16x2(e[u][n][0], e[u][n][1]));
            pb[u][n][1] = transpose8(pack_bf16x2(e[u][n][2], e[u][n][3]));
          }
        // ---- out^T += V^T P^T: rows channels, columns heads
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          uint2 vs[4];
          uint32_t vz[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint8_t* a = st + at_vs[i & 1] + (16 * u + (i >> 1) * 8) * kKv4Scales;
            vs[i] = ld<uint2>(a);
            vz[i] = ld<uint16_t>(a + z_off);
          }
          {
            const uint32_t za[4] = {__byte_perm(vz[0], vz[1], 0x5410), 0u, __byte_perm(vz[2], vz[3], 0x5410), 0u};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_bf16(zacc[n], za, pb[u][n][0], pb[u][n][1], zacc[n]);
          }
          uint4 cv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) cv[i] = ld<uint4>(st + at_v[i & 1] + (16 * u + (i >> 1) * 8) * kKv4Codes);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t word[4] = {j == 0 ? cv[0].x : j == 1 ? cv[0].y : j == 2 ? cv[0].z : cv[0].w,
                                      j == 0 ? cv[1].x : j == 1 ? cv[1].y : j == 2 ? cv[1].z : cv[1].w,
                                      j == 0 ? cv[2].x : j == 1 ? cv[2].y : j == 2 ? cv[2].z : cv[2].w,
                                      j == 0 ? cv[3].x : j == 1 ? cv[3].y : j == 2 ? cv[3].z : cv[3].w};
            const uint32_t x = __byte_perm(word[0], word[1], half), y = __byte_perm(word[2], word[3], half);
            const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
            const uint32_t s0 = __byte_perm(j < 2 ? vs[0].x : vs[0].y, j < 2 ? vs[1].x : vs[1].y, sel);
            const uint32_t s1 = __byte_perm(j < 2 ? vs[2].x : vs[2].y, j < 2 ? vs[3].x : vs[3].y, sel);
            const uint32_t a0[4] = {codes_bf16(x, mask), codes_bf16(x >> 4, mask), codes_bf16(y, mask),
                                    codes_bf16(y >> 4, mask)};
            const uint32_t a1[4] = {codes_bf16(x >> 8, mask), codes_bf16(x >> 12, mask), codes_bf16(y >> 8, mask),
                                    codes_bf16(y >> 12, mask)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t p0 = mul_bf16x2(pb[u][n][0], s0), p1 = mul_bf16x2(pb[u][n][1], s1);
              mma_bf16(acc[n][2 * j], a0, p0, p1, acc[n][2 * j]);
              mma_bf16(acc[n][2 * j + 1], a1, p0, p1, acc[n][2 * j + 1]);
              const uint32_t r0 = rest_bf16x2(pb[u][n][0], s0, p0), r1 = rest_bf16x2(pb[u][n][1], s1, p1);
              mma_bf16(acc[n][2 * j], a0, r0, r1, acc[n][2 * j]);
              mma_bf16(acc[n][2 * j + 1], a1, r0, r1, acc[n][2 * j + 1]);
            }
          }
        }
    }
    if (ti.flags & kLast) {
      // ---- the pair's stretch ends: merge the warps' states, a few heads at a time
      float* sm_ml = merge;                                // [warp][head][2]
      float* sm_o = merge + 2 * kWarps * kMergeHeads;      // [warp][head][128]
      const int slot = 2 * cta + (parts == 0 ? 0 : 1);
      ++parts;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], o);
#pragma unroll
      for (int c = 0; c < 2 * NT; ++c) {
        if (c * kMergeHeads >= G) break;
        const int n = c >> 1;
        float zj[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            zj[j][r] = fmaf(8.f, __shfl_sync(0xffffffffu, zacc[n][r], 4 * (j + 4) + tq),
                            __shfl_sync(0xffffffffu, zacc[n][r], 4 * j + tq));
        if ((tq >> 1) == (c & 1)) {  // the lanes whose columns are these heads
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int hh = warp * kMergeHeads + 2 * (tq & 1) + r;
            if (g == 0) {
              sm_ml[2 * hh] = m[n][r];
              sm_ml[2 * hh + 1] = l[n][r];
            }
            float* so = sm_o + hh * kD + g;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              so[16 * i] = acc[n][i][r] + zj[i >> 1][r];
              so[16 * i + 8] = acc[n][i][r + 2] + zj[i >> 1][r];
            }
          }
        }
        __syncthreads();
        const int h = c * kMergeHeads + warp;  // a warp per head, four channels a lane
        if (h < G) {
          float mm = -INFINITY;
#pragma unroll
          for (int v = 0; v < kWarps; ++v) mm = fmaxf(mm, sm_ml[2 * (v * kMergeHeads + warp)]);
          const float mu = mm == -INFINITY ? 0.f : mm;
          float ll = 0.f;
          float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int v = 0; v < kWarps; ++v) {
            const int hh = v * kMergeHeads + warp;
            const float f = ex2(sm_ml[2 * hh] - mu);
            const float4 x = *reinterpret_cast<const float4*>(sm_o + hh * kD + 4 * lane);
            ll += sm_ml[2 * hh + 1] * f;
            oo = make_float4(oo.x + x.x * f, oo.y + x.y * f, oo.z + x.z * f, oo.w + x.w * f);
          }
          if constexpr (CL > 1) {  // over the stages, which are done with
            float* to = shared_out + h * (kD + 4);
            *reinterpret_cast<float4*>(to + 4 * lane) = oo;
            if (lane == 0) *reinterpret_cast<float2*>(to + kD) = make_float2(mm, ll);
          } else if (ti.flags & kWhole) {
            const float inv = 1.f / ll;
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o.ptr) + ti.b * p.o.row +
                               (long long)(ti.kvh * G + h) * p.o.head + 4 * lane;
            *reinterpret_cast<uint2*>(o) =
                make_uint2(pack_bf16x2(oo.x * inv, oo.y * inv), pack_bf16x2(oo.z * inv, oo.w * inv));
          } else {
            const size_t at = (size_t)slot * G + h;
            *reinterpret_cast<float4*>(p.part_o + at * kD + 4 * lane) = oo;
            if (lane == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(mm, ll);
          }
        }
        __syncthreads();  // the buffer is reused
      }
    }
    __syncwarp();  // every lane is done with the stage: the next copies may overwrite it
    if (++stage == kStages) stage = 0;
  }
  if constexpr (CL > 1) {
    if (n_mine == 0)  // nothing, as a share
      for (int i = tid; i < G * (kD + 4); i += kThreads) shared_out[i] = i % (kD + 4) == kD ? -INFINITY : 0.f;
    __syncwarp();  // the loop's last turn may be half a warp's, and the barrier wants it whole
    cluster_sync_all();
    for (int h = rank + CL * warp; h < G; h += CL * kWarps) {  // a warp per head, four channels a lane
      const uint32_t mine = smem_u32(shared_out + h * (kD + 4));
      float m_of[CL], l_of[CL];
#pragma unroll
      for (int v = 0; v < CL; ++v) {
        const float4 x = ld_dsmem_f4(map_shared_rank(mine, v) + 4 * kD);
        m_of[v] = x.x;
        l_of[v] = x.y;
      }
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int v = 0; v < CL; ++v) mm = fmaxf(mm, m_of[v]);
      const float mu = mm == -INFINITY ? 0.f : mm;
      float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v0 = 0; v0 < CL; v0 += 8) {
        float4 ov[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) ov[v] = ld_dsmem_f4(map_shared_rank(mine, v0 + v) + 16 * lane);
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const float f = ex2(m_of[v0 + v] - mu);
          ll += l_of[v0 + v] * f;
          oo = make_float4(oo.x + ov[v].x * f, oo.y + ov[v].y * f, oo.z + ov[v].z * f, oo.w + ov[v].w * f);
        }
      }
      const float inv = w.n_tiles > 0 ? 1.f / ll : 0.f;  // no keys: a zero row
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o.ptr) + pair_b * p.o.row +
                         (long long)(pair_kvh * G + h) * p.o.head + 4 * lane;
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(oo.x * inv, oo.y * inv), pack_bf16x2(oo.z * inv, oo.w * inv));
    }
    __syncwarp();
    cluster_sync_all();  // nobody leaves while its share may be read
  }
}

// Joins the partial results of the pairs that were cut, W warps per query head (8: a block, for
// long sequences, which many stretches share); a sequence without keys gets its zeros here.
constexpr int kJoinThreads = 256;
constexpr int kJoinBatch = 8;  // partials whose loads are issued together

template <int W>
__global__ void __launch_bounds__(kJoinThreads) attn_kv4_join_kernel(const __grid_constant__ Kv4Params p) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.H / p.Hkv;
  const long long total = (long long)p.prefix[p.B] * p.Hkv;
  const int n_str = p.prefix[p.B + 1];
  static_assert(W == 1 || W == kJoinThreads / 32, "a block's warps share one head, or none");
  const long long pair = W == 1 ? (long long)blockIdx.x * (kJoinThreads / 32) + warp : blockIdx.x;
  const int part = W == 1 ? 0 : warp;
  if (pair >= (long long)p.B * p.H) return;
  const int b = (int)(pair / p.H), h = (int)(pair % p.H), kvh = h / G, hg = h % G;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o.ptr) + b * p.o.row + h * p.o.head + 4 * lane;
  const int nt = p.prefix[b + 1] - p.prefix[b];
  if (nt == 0) {
    *reinterpret_cast<uint2*>(o) = make_uint2(0, 0);
    return;
  }
  const long long s0 = (long long)p.prefix[b] * p.Hkv + (long long)kvh * nt;
  const int c0 = stretch_of(total, n_str, s0), c1 = stretch_of(total, n_str, s0 + nt - 1);
  if (c0 == c1) return;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0 + part * kJoinBatch; c <= c1; c += W * kJoinBatch) {
    float2 ml[kJoinBatch];
    float4 ov[kJoinBatch];
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      ov[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c + i <= c1) {
        // the pair is the stretch's first one unless it begins inside of it
        const int slot = 2 * (c + i) + (s0 > stretch_begin(total, n_str, c + i) ? 1 : 0);
        const size_t at = (size_t)slot * G + hg;
        ml[i] = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
        ov[i] = *reinterpret_cast<const float4*>(p.part_o + at * kD + 4 * lane);
      }
    }
    float gm = m;
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) gm = fmaxf(gm, ml[i].x);
    const float mu = gm == -INFINITY ? 0.f : gm;
    const float sc = ex2(m - mu);  // 0 for the first group
    l *= sc;
    acc = make_float4(acc.x * sc, acc.y * sc, acc.z * sc, acc.w * sc);
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) {
      const float f = ex2(ml[i].x - mu);
      l += ml[i].y * f;
      acc = make_float4(acc.x + ov[i].x * f, acc.y + ov[i].y * f, acc.z + ov[i].z * f, acc.w + ov[i].w * f);
    }
    m = gm;
  }
  if constexpr (W > 1) {
    __shared__ float2 part_ml[W];
    __shared__ float4 part_o[W][32];
    if (lane == 0) part_ml[part] = make_float2(m, l);
    part_o[part][lane] = acc;
    __syncthreads();
    if (part != 0) return;
    float gm = -INFINITY;
#pragma unroll
    for (int i = 0; i < W; ++i) gm = fmaxf(gm, part_ml[i].x);
    const float mu = gm == -INFINITY ? 0.f : gm;
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float f = ex2(part_ml[i].x - mu);
      const float4 x = part_o[i][lane];
      l += part_ml[i].y * f;
      acc = make_float4(acc.x + x.x * f, acc.y + x.y * f, acc.z + x.z * f, acc.w + x.w * f);
    }
  }
  const float inv = 1.f / l;
  *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

int kv4_grid(int H, int Hkv, int num_sms) { return num_sms * (H / Hkv <= 8 ? Cfg<1>::kCtas : Cfg<2>::kCtas); }

struct Kv4Ws {
  size_t prefix, ml, o, bytes;
};
Kv4Ws kv4_ws(int B, int H, int Hkv, int num_sms) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t slots = (size_t)2 * kv4_grid(H, Hkv, num_sms) * (H / Hkv);
  Kv4Ws w;
  w.prefix = 0;
  w.ml = up(((size_t)B + 2) * sizeof(int));
  w.o = w.ml + up(slots * 2 * sizeof(float));
  w.bytes = w.o + slots * kD * sizeof(float);
  return w;
}

// Clusters for small batches: how many CTAs share a pair, 1 for none. 16 for longer caches, while
// the clusters are all resident at once with room to spare in each GPC; 8 for shorter ones; none
// where the tiles of a CTA would be many. us with 32 heads, for 16 | 8 | 1 CTAs a pair: one
// sequence over 8 KV heads of 512 keys 5.3 | 4.6, 4000 keys 7.1 | 7.8, 12000 12.4 | | 13.1, 16384
// 15.2 | | 13.4; four of 8192 17.1 | 23.0 | 21.6. Groups of 16 heads (2 KV heads), whose CTAs take
// half an SM: one sequence of 8192 10.7 | | 11.9, 8 of them 23.8 | 20.4 | 17.4, 16 of 1024 25.0 |
// 8.6.
int kv4_cluster(int B, int H, int Hkv, int capacity, int window, int num_sms) {
  const int span = window > 0 && window < capacity ? window : capacity;
  const int n = (span + kTile - 1) / kTile;
  const long long pairs = (long long)B * Hkv;
  const bool fits16 = H / Hkv <= 8 ? 2 * 16 * pairs <= 7ll * num_sms : 16 * pairs <= num_sms;
  if (fits16 && n >= 16 && n <= 96) return 16;
  return 8 * pairs <= 2ll * num_sms && n <= 32 ? 8 : 1;
}

// Clusters of more than 8 CTAs, allowed once per device (a bit each).
cudaError_t allow_large_clusters_once(const void* kernel, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

template <int NT, int CL>
cudaError_t launch_nt(const Kv4Params& p, int grid, cudaStream_t s) {
  static std::atomic<unsigned long long> configured{0};  // one bit per device
  const auto kernel = attn_kv4_kernel<NT, CL>;
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(kernel), Cfg<NT>::kSmem, configured);
  if (e != cudaSuccess) return e;
  if constexpr (CL == 1) {
    return launch_pdl(kernel, grid, kThreads, Cfg<NT>::kSmem, s, p);
  } else {
    if (CL > 8) {
      static std::atomic<unsigned long long> large{0};
      e = allow_large_clusters_once(reinterpret_cast<const void*>(kernel), large);
      if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<NT>::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
  }
}

}  // namespace

size_t attn_kv4_ws_bytes(int B, int H, int Hkv, int capacity, int window, int num_sms) {
  if (B <= 0 || kv4_cluster(B, H, Hkv, capacity, window, num_sms) > 1) return 0;
  return kv4_ws(B, H, Hkv, num_sms).bytes;
}

cudaError_t launch_attn_decode_kv4(const HeadRows& q, const Kv4Cache& c, const HeadRows& o, int B, int H, int Hkv,
                                   int window, void* ws, int num_sms, cudaStream_t s, const char** why) {
  if (H / Hkv > 16) {
    *why = "4-bit decode attention: at most 16 query heads per KV head";
    return cudaErrorInvalidValue;
  }
  if (B <= 0) return cudaSuccess;
  Kv4Params p{q, o, c, B, H, Hkv, window > 0 ? window : 0, nullptr, nullptr, nullptr, kLog2e / sqrtf((float)kD)};
  const bool wide = H / Hkv > 8;
  const int cluster = kv4_cluster(B, H, Hkv, c.capacity, window, num_sms);
  if (cluster == 16) return wide ? launch_nt<2, 16>(p, B * Hkv * 16, s) : launch_nt<1, 16>(p, B * Hkv * 16, s);
  if (cluster == 8) return wide ? launch_nt<2, 8>(p, B * Hkv * 8, s) : launch_nt<1, 8>(p, B * Hkv * 8, s);
  const Kv4Ws w = kv4_ws(B, H, Hkv, num_sms);
  uint8_t* base = static_cast<uint8_t*>(ws);
  p.prefix = reinterpret_cast<int*>(base + w.prefix);
  p.part_ml = reinterpret_cast<float*>(base + w.ml);
  p.part_o = reinterpret_cast<float*>(base + w.o);
  // a CTA per kMinTiles tiles of the largest cache this could be
  const long long most = (long long)B * Hkv * ((c.capacity + kTile - 1) / kTile);
  const int grid = (int)std::max(1ll, std::min<long long>(kv4_grid(H, Hkv, num_sms), most / kMinTiles));
  cudaError_t e = wide ? launch_nt<2, 1>(p, grid, s) : launch_nt<1, 1>(p, grid, s);
  if (e != cudaSuccess) return e;
  // a block per head where a pair may be cut into more stretches than a warp loads at once (one
  // sequence of 65536 keys 41.2 -> 29.7 us)
  const long long heads = (long long)B * H;
  if (grid >= (long long)kJoinBatch * B * Hkv)
    return launch_pdl(attn_kv4_join_kernel<kJoinThreads / 32>, dim3((unsigned)heads), kJoinThreads, 0, s, p);
  return launch_pdl(attn_kv4_join_kernel<1>, dim3((unsigned)((heads + kJoinThreads / 32 - 1) / (kJoinThreads / 32))),
                    kJoinThreads, 0, s, p);
}

}  // namespace blk

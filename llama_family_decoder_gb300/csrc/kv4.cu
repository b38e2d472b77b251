// The 4-bit KV cache: store (quantise and append) and load (the values the codes
// stand for). A row is one key or value of one KV head, 128 channels in four groups
// of 32. A group keeps scale = bf16((hi - lo) / 15) and offset = bf16(lo) and the
// codes clamp(rint((x - offset) / scale), 0, 15); a code stands for
// offset + scale * code. bf16 scales share the inputs' exponent range, so no scale
// overflows; a group with a NaN or an infinity in it, or whose span hi - lo passes fp32's
// range (from -3.3e38 to 3.3e38), keeps the offset NaN, and one whose scale underflows keeps
// codes 0.
//
// The order of a row's 64 code bytes is the one the decode attention's tensor-core
// fragments want (see kv4_byte_channel): a lane of an 8-row fragment finds all its
// codes of a key in one 16-byte chunk, word j of it holding group j alone.
//
// One pass over the rows: 16 lanes hold a row, 8 neighbouring channels each; a group is 4
// lanes (two shuffles for its extremes), and four more shuffles in the same 4 lanes
// turn their codes into the row's words. A block takes a few token rows, all heads: it looks
// up their slots once (a binary search of cu_seqlens in shared memory) while its first rows
// are already on the way, and loads a row ahead of the one it converts. What bounds it is the
// issue of instructions (70% of the slots, DRAM half busy), about 150 for two rows of a warp:
// hence the packed arithmetic, the extremes on bf16 pairs and the running offsets. 9155 rows of
// 8 KV heads, stored and then loaded: 27.4 us, 3.6 TB/s.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace blk {

namespace {

constexpr int kThreads = 128;
constexpr int kStatusInvalidArg = 1;  // == BLK_ERR_INVALID_ARG
constexpr int kStatusCacheFull = 4;   // == BLK_ERR_CACHE_FULL

constexpr int kMaxBlockRows = 64;     // token rows of a block, at most
constexpr int kSharedSeqs = 1024;     // sequences whose cu_seqlens a block copies to shared memory

// Rows of packed tokens and their slots.
struct RowParams {
  HeadRows k, v;
  const int* cu;      // [B + 1], or null: row b is sequence b
  const int* starts;  // [B] first slots, or null: 0
  Kv4Cache c;
  int rows, B, Hkv, block_rows;
  DevStatus* status;
};

// What a half warp works on in turn: K and V of one row (of the block) and head, and where they
// are. Both halves of a warp take the same number of turns; row >= the block's rows: nothing
// left.
struct Unit {
  int row, head, turns, rows_on, heads_on;
  long long k, v, plane;          // element offsets into k, v; slots before the head's plane
  long long k_on, v_on, plane_on;  // ... from one turn to the next, and on when the head wraps
  long long k_wrap, v_wrap, plane_wrap;
  __device__ __forceinline__ Unit(const RowParams& p, int r0, int n) {
    const int halves = blockDim.x / 16, u = threadIdx.x / 16;
    row = u / p.Hkv;
    head = u - row * p.Hkv;
    rows_on = halves / p.Hkv;
    heads_on = halves - rows_on * p.Hkv;
    turns = (n * p.Hkv - (u & ~1) + halves - 1) / halves;
    k = (r0 + row) * p.k.row + head * p.k.head + 8 * (threadIdx.x & 15);
    v = (r0 + row) * p.v.row + head * p.v.head + 8 * (threadIdx.x & 15);
    plane = (long long)head * p.c.capacity;
    k_on = rows_on * p.k.row + heads_on * p.k.head;
    v_on = rows_on * p.v.row + heads_on * p.v.head;
    plane_on = (long long)heads_on * p.c.capacity;
    k_wrap = p.k.row - p.Hkv * p.k.head;
    v_wrap = p.v.row - p.Hkv * p.v.head;
    plane_wrap = -(long long)p.Hkv * p.c.capacity;
  }
  __device__ __forceinline__ void next(const RowParams& p) {
    row += rows_on;
    k += k_on;
    v += v_on;
    if (heads_on != 0) {  // the same for all
      head += heads_on;
      plane += plane_on;
      if (head >= p.Hkv) {
        head -= p.Hkv;
        ++row;
        k += k_wrap;
        v += v_wrap;
        plane += plane_wrap;
      }
    }
  }
};

// A number of cu_seqlens as it is read.
__device__ __forceinline__ int clamped(int x, int rows) { return min(max(x, 0), rows); }

// Whether cu_seqlens falls somewhere; one that does, or leaves [0, rows], sets the status word, also
// where rows that it misplaced found no slot (CACHE_FULL) first. All threads of the block.
__device__ __forceinline__ bool list_falls(const int* cu, int B, int rows, DevStatus* st) {
  bool bad = false, falls = false;
  for (int i = threadIdx.x; i < B; i += blockDim.x) {
    const int a = cu[i], e = cu[i + 1];
    falls |= e < a;
    bad |= e < a || a < 0 || e > rows;
  }
  if (bad && st && atomicCAS(&st->code, 0, kStatusInvalidArg) == kStatusCacheFull)
    atomicCAS(&st->code, kStatusCacheFull, kStatusInvalidArg);
  return __syncthreads_or(falls);
}

// at[i] := the slot of the block's row i, counted over the whole cache for KV head 0 (-1: a row
// of no sequence, -2: a slot outside the cache).
__device__ __forceinline__ void find_slots(const RowParams& p, int r0, int n, long long* at, int* s_cu) {
  const int tid = threadIdx.x;
  const int* cu = p.cu;
  if (cu && p.B <= kSharedSeqs) {
    for (int i = tid; i <= p.B; i += blockDim.x) s_cu[i] = cu[i];
    __syncthreads();
    cu = s_cu;
  }
  if (tid < n) {
    const int r = r0 + tid;
    int b = r, i = 0;
    bool in = true;
    if (cu) {
      in = r >= cu[0] && r < cu[p.B];
      int lo = 0, hi = p.B;  // the last sequence that begins at or before r
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cu[mid] <= r)
          lo = mid;
        else
          hi = mid;
      }
      b = lo;
      i = r - max(cu[lo], 0);
    }
    long long a = -1;
    if (in) {
      const long long slot = (long long)(p.starts ? p.starts[b] : 0) + i;
      a = slot >= 0 && slot < p.c.capacity ? (long long)b * p.Hkv * p.c.capacity + slot : -2;
    }
    at[tid] = a;
  }
  __syncthreads();
}

__device__ __forceinline__ uint32_t bf16_bits(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

// The correctly rounded quotient d / s from inv = (1 / s)(1 + e), |e| <= 2^-23, s of at most 8
// significant bits, all of them normal numbers: q = RN(d inv) is within a relative 2^-22 of it,
// the remainder d - q s is exact in one fused multiply-add, and q + rem inv misses d / s by a
// relative 2^-45 at most before its rounding (the correction step of Markstein 1990). A
// quotient of a 24-bit by an 8-bit number keeps a relative 2^-34 away from the middle between
// two fp32 numbers, so the rounding is that of d / s. quotient2: two of them, given -s.
__device__ __forceinline__ float quotient(float d, float s, float inv) {
  const float q = d * inv;
  return fmaf(fmaf(-q, s, d), inv, q);
}
__device__ __forceinline__ f32x2 quotient2(f32x2 d, f32x2 minus_s, f32x2 inv) {
  const f32x2 q = f2_mul(d, inv);
  return f2_fma(f2_fma(q, minus_s, d), inv, q);
}
__device__ __forceinline__ float reciprocal(float s) {  // documented to be within 2^-23
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// Packed bf16 least and greatest; a NaN in either operand wins.
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// One row by 16 lanes (m = lane & 15: channels 8 m .. 8 m + 7, in u), all 32 lanes converged.
__device__ __forceinline__ void store_row(const uint4& u, uint8_t* codes, uint8_t* scales, bool on, int lane) {
  const int m = lane & 15, q = lane & 3, j = m >> 2;
  uint32_t lo2 = min2(min2(u.x, u.y), min2(u.z, u.w)), hi2 = max2(max2(u.x, u.y), max2(u.z, u.w));
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo2 = min2(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
    hi2 = max2(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
  }
  const uint32_t zb = min2(lo2, lo2 >> 16) & 0xffffu, tb = max2(hi2, hi2 >> 16);
  const float z = __uint_as_float(zb << 16), span = __uint_as_float(tb << 16) - z;
  f32x2 x[4];  // less the offset
  {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = f2_add(f2_make(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), f2_make(-z, -z));
  }
  uint32_t w = 0, sz;
  if (span >= 1e-28f && span <= 3.402823466e38f) {
    const uint32_t sb = bf16_bits(quotient(span, 15.f, 1.f / 15.f));
    const float s = __uint_as_float(sb << 16), inv = reciprocal(s);
    const f32x2 minus_s2 = f2_make(-s, -s), inv2 = f2_make(inv, inv), magic2 = f2_make(12582912.f, 12582912.f);
    // adding 1.5 * 2^23 rounds a quotient (at most 15.1) to its code, in the sum's low bits; the
    // bits are added up as integers, each 4 bits further, and 0x4B400000 (8 times, likewise
    // shifted: 0x4B400000 * 0x11111111) is taken off
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      float a, b;
      f2_split(f2_add(quotient2(x[i], minus_s2, inv2), magic2), a, b);
      w = (w * 16u + __float_as_uint(b)) * 16u + __float_as_uint(a);
    }
    w -= 0x4B400000u * 0x11111111u;
    sz = sb | zb << 16;
  } else if (span < 1e-28f) {  // quotients and reciprocals may leave the normal numbers
    const uint32_t sb = bf16_bits(span / 15.f);
    const float s = __uint_as_float(sb << 16);
    if (s > 0.f)
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        float a, b;
        f2_split(x[0], a, b);
        w |= (uint32_t)fminf(rintf(a / s), 15.f) << (8 * i) | (uint32_t)fminf(rintf(b / s), 15.f) << (8 * i + 4);
#pragma unroll
        for (int k = 0; k < 3; ++k) x[k] = x[k + 1];
      }
    sz = sb | zb << 16;
  } else {  // a NaN or an infinity, or a span past fp32
    sz = 0x7fc00000u;
  }
  // lanes q = 0, 1 of the group hold the low and high nibbles of its bytes e = 0, lanes
  // 2, 3 those of e = 1 (nibble g = 2 t + u); lane q writes word t = q: byte q of the four
  // lanes' words, their low nibbles (u = 0) side by side, then their high ones
  const uint32_t w0 = __shfl_sync(0xffffffffu, w, lane & ~3), w1 = __shfl_sync(0xffffffffu, w, (lane & ~3) + 1),
                 w2 = __shfl_sync(0xffffffffu, w, (lane & ~3) + 2), w3 = __shfl_sync(0xffffffffu, w, lane | 3);
  const uint32_t pick = q | (4 + q) << 4;
  const uint32_t y = __byte_perm(__byte_perm(w0, w1, pick), __byte_perm(w2, w3, pick), 0x5410);
  const uint32_t n0 = y & 0x0F0F0F0Fu, n1 = y >> 4 & 0x0F0F0F0Fu;
  const uint32_t word = __byte_perm(n0 | n0 >> 4, n1 | n1 >> 4, 0x6420);
  const int pair = (lane & 16) + 8 * (q & 1);  // the groups 2 (q & 1) and 2 (q & 1) + 1
  const uint32_t g0 = __shfl_sync(0xffffffffu, sz, pair), g1 = __shfl_sync(0xffffffffu, sz, pair + 4);
  if (on) {
    *reinterpret_cast<uint32_t*>(codes + 16 * q + 4 * j) = word;
    if (m < 4)  // scales of groups 0, 1 | 2, 3, then offsets likewise
      *reinterpret_cast<uint32_t*>(scales + 4 * m) = m < 2 ? __byte_perm(g0, g1, 0x5410) : __byte_perm(g0, g1, 0x7632);
  }
}

// append: starts is lens itself. Without cu its blocks hold a row each and move lens on; with cu
// a second kernel does. Otherwise a last block without rows looks the list over and writes the new
// lengths, which nobody reads here (a block with rows would be the last one done: 0.2 us more for
// the decode batch).
__global__ void __launch_bounds__(kThreads) kv4_store_kernel(const __grid_constant__ RowParams p, int append) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ long long at[kMaxBlockRows];
  __shared__ int s_cu[kSharedSeqs + 1];
  const int tid = threadIdx.x, lane = tid & 31;
  const int r0 = blockIdx.x * p.block_rows, n = max(0, min(p.block_rows, p.rows - r0));
  Unit un(p, r0, n);
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  auto fetch = [&] {
    if (un.row < n) {
      k = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k.ptr) + un.k);
      v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v.ptr) + un.v);
    }
  };
  fetch();
  find_slots(p, r0, n, at, s_cu);
  if (tid < n && at[tid] == -2 && p.status) atomicCAS(&p.status->code, 0, kStatusCacheFull);
  for (int turn = 0; turn < un.turns; ++turn) {
    const uint4 ku = k, vu = v;
    const long long a = un.row < n ? at[un.row] : -1;
    const size_t to = a >= 0 ? (size_t)(a + un.plane) : 0;
    un.next(p);
    fetch();
    store_row(ku, p.c.k + to * kKv4Codes, p.c.k_scale + to * kKv4Scales, a >= 0, lane);
    store_row(vu, p.c.v + to * kKv4Codes, p.c.v_scale + to * kKv4Scales, a >= 0, lane);
  }
  if (!append) {
    if (blockIdx.x == gridDim.x - 1 && !(p.cu && list_falls(p.cu, p.B, p.rows, p.status)))
      for (int i = tid; i < p.B; i += blockDim.x) {
        const long long e = (long long)p.starts[i] + (p.cu ? clamped(p.cu[i + 1], p.rows) - clamped(p.cu[i], p.rows) : 1);
        p.c.lens[i] = (int)(e < 0 ? 0 : e < p.c.capacity ? e : p.c.capacity);
      }
  } else if (!p.cu && tid == 0 && n > 0 && at[0] >= 0) {  // the block has read its slot (find_slots)
    p.c.lens[r0] += 1;
  }
}

// lens[b] += the rows of sequence b, after a store that read them as first slots. Every block
// looks the whole list over, so there is one per SM at most.
__global__ void kv4_lens_kernel(const int* cu, int* lens, int B, int rows, int capacity, DevStatus* st) {
  pdl_launch_dependents();
  pdl_wait();
  if (list_falls(cu, B, rows, st)) return;
  for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < B; b += gridDim.x * blockDim.x) {
    const long long n = (long long)lens[b] + clamped(cu[b + 1], rows) - clamped(cu[b], rows);
    lens[b] = (int)(n < 0 ? 0 : n < capacity ? n : capacity);
  }
}

// One row by 16 lanes: the code word and the scale and offset bits that a lane holds -> its 8
// channels. All 32 lanes converged.
__device__ __forceinline__ void load_row(__nv_bfloat16* dst, uint32_t word, uint32_t sb, uint32_t zb, bool on, int lane,
                                         uint32_t mask) {
  const int q = lane & 3;
  const float s = __uint_as_float(sb << 16), z = __uint_as_float(zb << 16);
  // lane q wants nibble q (of each 16-bit half: channels g = 2 t, 2 t + 1) of the 4 words t
  uint32_t x[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint32_t w = __shfl_sync(0xffffffffu, word, (lane & ~3) + t) >> (4 * q);
    // a code under the exponent of 2^23, taken off again
    const f32x2 code = f2_add(f2_make(__uint_as_float(and_or<0x4B000000u>(w, mask)),
                                      __uint_as_float(and_or<0x4B000000u>(w >> 16, mask))),
                              f2_make(-8388608.f, -8388608.f));
    float a, b;
    f2_split(f2_fma(f2_make(s, s), code, f2_make(z, z)), a, b);
    x[t] = pack_bf16x2(a, b);
  }
  if (on) *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
}

__global__ void __launch_bounds__(kThreads) kv4_load_kernel(const __grid_constant__ RowParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ long long at[kMaxBlockRows];
  __shared__ int s_cu[kSharedSeqs + 1];
  const int tid = threadIdx.x, lane = tid & 31, q = lane & 3, j = (lane & 15) >> 2;
  const int r0 = blockIdx.x * p.block_rows, n = max(0, min(p.block_rows, p.rows - r0));
  Unit un(p, r0, n);
  find_slots(p, r0, n, at, s_cu);
  if (tid < n && at[tid] == -2 && p.status) atomicCAS(&p.status->code, 0, kStatusInvalidArg);
  if (p.cu && blockIdx.x == gridDim.x - 1) list_falls(p.cu, p.B, p.rows, p.status);  // a block without rows
  const uint32_t mask = kept_constant(15u);
  uint32_t kw = 0, ks = 0, kz = 0, vw = 0, vs = 0, vz = 0;
  auto fetch = [&] {
    kw = ks = kz = vw = vs = vz = 0;
    const long long a = un.row < n ? at[un.row] : -1;
    if (a >= 0) {
      const size_t from = (size_t)(a + un.plane);
      kw = *reinterpret_cast<const uint32_t*>(p.c.k + from * kKv4Codes + 16 * q + 4 * j);
      vw = *reinterpret_cast<const uint32_t*>(p.c.v + from * kKv4Codes + 16 * q + 4 * j);
      const uint16_t* sk = reinterpret_cast<const uint16_t*>(p.c.k_scale + from * kKv4Scales) + j;
      const uint16_t* sv = reinterpret_cast<const uint16_t*>(p.c.v_scale + from * kKv4Scales) + j;
      ks = sk[0], kz = sk[4], vs = sv[0], vz = sv[4];
    }
  };
  fetch();
  for (int turn = 0; turn < un.turns; ++turn) {
    const uint32_t kw0 = kw, ks0 = ks, kz0 = kz, vw0 = vw, vs0 = vs, vz0 = vz;
    const bool on = un.row < n && at[un.row] != -1;  // a row of no sequence is left as it was
    const long long k_to = un.k, v_to = un.v;
    un.next(p);
    fetch();
    load_row(static_cast<__nv_bfloat16*>(p.k.ptr) + k_to, kw0, ks0, kz0, on, lane, mask);
    load_row(static_cast<__nv_bfloat16*>(p.v.ptr) + v_to, vw0, vs0, vz0, on, lane, mask);
  }
}

// Token rows per block: a few, so that a block's look-up serves many rows, but at least about
// twelve blocks per SM while there are enough.
int block_rows(int rows, int Hkv, int num_sms) {
  const int most = Hkv >= 32 ? 1 : 32 / Hkv;  // 32 units, four turns of a block's 8 half warps
  const int fill = rows / (12 * num_sms);
  return fill < 1 ? 1 : fill < most ? fill : most;
}

}  // namespace

cudaError_t launch_kv4_store(const HeadRows& k, const HeadRows& v, int rows, const int* cu, const int* starts, int B,
                             int Hkv, const Kv4Cache& c, int num_sms, DevStatus* st, cudaStream_t s) {
  const bool append = starts == nullptr || starts == c.lens;
  RowParams p{k, v, cu, append ? c.lens : starts, c, rows, B, Hkv, block_rows(rows, Hkv, num_sms), st};
  if (append && !cu) p.block_rows = 1;
  const int grid = rows > 0 ? (rows + p.block_rows - 1) / p.block_rows + (append ? 0 : 1) : 1;
  cudaError_t e = launch_pdl(kv4_store_kernel, grid, kThreads, 0, s, p, append ? 1 : 0);
  if (e != cudaSuccess || !append || !cu) return e;
  return launch_pdl(kv4_lens_kernel, std::min((B - 1) / 256 + 1, num_sms), 256, 0, s, cu, c.lens, B, rows, c.capacity, st);
}

cudaError_t launch_kv4_load(const HeadRows& k, const HeadRows& v, int rows, const int* cu, const int* starts, int B,
                            int Hkv, const Kv4Cache& c, int num_sms, DevStatus* st, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  const RowParams p{k, v, cu, starts, c, rows, B, Hkv, block_rows(rows, Hkv, num_sms), st};
  return launch_pdl(kv4_load_kernel, (rows + p.block_rows - 1) / p.block_rows + (cu ? 1 : 0), kThreads, 0, s, p);
}

}  // namespace blk

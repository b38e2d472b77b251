// The 4-bit KV cache: store (quantise and append) and load (the values the codes
// stand for). A row is one key or value of one KV head, 128 channels in four groups
// of 32. A group keeps scale = bf16((hi - lo) / 15) and offset = bf16(lo) and the
// codes clamp(rint((x - offset) / scale), 0, 15); a code stands for
// offset + scale * code. bf16 scales share the inputs' exponent range, so no finite
// group can overflow them; a group whose span hi - lo is not finite (a NaN or an
// infinity in it) keeps the offset NaN, and one whose scale underflows keeps codes 0.
//
// The order of a row's 64 code bytes is the one the decode attention's tensor-core
// fragments want (see kv4_byte_channel): a lane of an 8-row fragment finds all its
// codes of a key in one 16-byte chunk, word j of it holding group j alone.
//
// HBM-bound, one pass: 16 lanes hold a row, 8 neighbouring channels each; a group is 4
// lanes (two shuffles for its extremes), and four more shuffles in the same 4 lanes
// turn their codes into the row's words.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace blk {

namespace {

constexpr int kThreads = 256;
constexpr int kStatusInvalidArg = 1;  // == BLK_ERR_INVALID_ARG
constexpr int kStatusCacheFull = 4;   // == BLK_ERR_CACHE_FULL

struct StoreParams {
  HeadRows k, v;
  const int* cu;      // [B + 1], or null: row b is sequence b
  const int* starts;  // [B] first slots, or null
  Kv4Cache c;
  int rows, B, Hkv, warps_per_row;
  int first_slot_lens;  // starts is c.lens itself (an append)
  DevStatus* status;
};

// The sequence of packed row r: the number of entries of cu[1 .. B] that are <= r,
// found by a warp 32 at a time. Returns -1 for rows before cu[0] or behind cu[B].
__device__ __forceinline__ int sequence_of_row(const int* cu, int B, int r, int lane) {
  if (r < cu[0] || r >= cu[B]) return -1;
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    // cu[lo + step * (lane + 1)] <= r: the answer is at or past that entry
    const int at = lo + step * (lane + 1);
    const bool past = at < lo + n && cu[at] <= r;
    const int k = __popc(__ballot_sync(0xffffffffu, past));
    const int base = lo + step * k;
    n = min(step, lo + n - base);
    lo = base;
  }
  return lo;
}

__device__ __forceinline__ uint32_t bf16_bits(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

// One row by 16 lanes (m = lane & 15: channels 8 m .. 8 m + 7), all 32 lanes converged.
__device__ __forceinline__ void store_row(const __nv_bfloat16* src, uint8_t* codes, uint8_t* scales, bool on, int lane) {
  const int m = lane & 15, q = lane & 3, j = m >> 2;
  float x[8];
  {
    const uint4 u = on ? *reinterpret_cast<const uint4*>(src + 8 * m) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = unpack_bf16x2(w[i]);
      x[2 * i] = t.x;
      x[2 * i + 1] = t.y;
    }
  }
  float lo = x[0], hi = x[0];
  bool nan = x[0] != x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    nan |= x[i] != x[i];
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const uint32_t nans = __ballot_sync(0xffffffffu, nan);
  const float span = hi - lo;
  const bool finite = ((nans >> (lane & ~3)) & 15u) == 0 && span <= 3.402823466e38f;
  const uint32_t sb = finite ? bf16_bits(span / 15.f) : 0u;
  const uint32_t zb = finite ? bf16_bits(lo) : 0x7fc0u;
  const float s = __uint_as_float(sb << 16), z = __uint_as_float(zb << 16);
  uint32_t w = 0;
  if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = fminf(fmaxf(rintf((x[i] - z) / s), 0.f), 15.f);
      w |= (uint32_t)c << (4 * i);
    }
  }
  // lanes q = 0, 1 of the group hold the low and high nibbles of its bytes e = 0, lanes
  // 2, 3 those of e = 1 (nibble g = 2 t + u); lane q writes word t = q
  uint32_t a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = __shfl_sync(0xffffffffu, w, (lane & ~3) + i) >> (8 * q);
  const uint32_t word = (a[0] & 15u) | (a[1] & 15u) << 4 | (a[2] & 15u) << 8 | (a[3] & 15u) << 12 |
                        (a[0] >> 4 & 15u) << 16 | (a[1] >> 4 & 15u) << 20 | (a[2] >> 4 & 15u) << 24 |
                        (a[3] >> 4 & 15u) << 28;
  const uint32_t sz = sb | zb << 16;
  const int pair = (lane & 16) + 8 * (q & 1);  // the groups 2 (q & 1) and 2 (q & 1) + 1
  const uint32_t g0 = __shfl_sync(0xffffffffu, sz, pair), g1 = __shfl_sync(0xffffffffu, sz, pair + 4);
  if (on) {
    *reinterpret_cast<uint32_t*>(codes + 16 * q + 4 * j) = word;
    if (m < 4)  // scales of groups 0, 1 | 2, 3, then offsets likewise
      *reinterpret_cast<uint32_t*>(scales + 4 * m) = m < 2 ? __byte_perm(g0, g1, 0x5410) : __byte_perm(g0, g1, 0x7632);
  }
}

// A warp takes two KV heads of one row, K and V of both.
__global__ void __launch_bounds__(kThreads) kv4_store_kernel(const __grid_constant__ StoreParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long gw = (long long)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int row = (int)(gw / p.warps_per_row), part = (int)(gw % p.warps_per_row);
  int b = -1, slot = 0;
  if (row < p.rows) {
    b = p.cu ? sequence_of_row(p.cu, p.B, row, lane) : row;
    if (b >= 0) slot = p.starts[b] + (p.cu ? row - p.cu[b] : 0);
  }
  const bool fits = b >= 0 && slot >= 0 && slot < p.c.capacity;
  if (b >= 0 && !fits && lane == 0 && p.status) atomicCAS(&p.status->code, 0, kStatusCacheFull);
  if (fits) {
    for (int h0 = 2 * part; h0 < p.Hkv; h0 += 2 * p.warps_per_row) {
      const int h = h0 + (lane >> 4);
      const bool on = h < p.Hkv;
      const size_t at = ((size_t)b * p.Hkv + (on ? h : 0)) * p.c.capacity + slot;
      const long long off = on ? h : 0;
      store_row(static_cast<const __nv_bfloat16*>(p.k.ptr) + row * p.k.row + off * p.k.head, p.c.k + at * kKv4Codes,
                p.c.k_scale + at * kKv4Scales, on, lane);
      store_row(static_cast<const __nv_bfloat16*>(p.v.ptr) + row * p.v.row + off * p.v.head, p.c.v + at * kKv4Codes,
                p.c.v_scale + at * kKv4Scales, on, lane);
    }
  }
  if (!p.first_slot_lens) {  // the new lengths: nobody reads lens here
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < p.B; i += blockDim.x) {
        const long long n = (long long)p.starts[i] + (p.cu ? p.cu[i + 1] - p.cu[i] : 1);
        p.c.lens[i] = (int)(n < 0 ? 0 : n < p.c.capacity ? n : p.c.capacity);
      }
  } else if (!p.cu) {  // one row per sequence, one block per row: every warp has read its slot
    __syncthreads();
    if (threadIdx.x == 0 && fits) p.c.lens[b] = slot + 1;
  }
}

// lens[b] += the rows of sequence b, after a store that read them as first slots
__global__ void kv4_lens_kernel(const int* cu, int* lens, int B, int capacity) {
  pdl_launch_dependents();
  pdl_wait();
  for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < B; b += gridDim.x * blockDim.x) {
    const long long n = (long long)lens[b] + cu[b + 1] - cu[b];
    lens[b] = (int)(n < 0 ? 0 : n < capacity ? n : capacity);
  }
}

struct LoadParams {
  HeadRows k, v;
  const int* cu;
  const int* starts;  // [B], or null: slot 0
  Kv4Cache c;
  int rows, B, Hkv, warps_per_row;
  DevStatus* status;
};

__device__ __forceinline__ void load_row(__nv_bfloat16* dst, const uint8_t* codes, const uint8_t* scales, bool on,
                                         bool valid, int lane) {
  const int m = lane & 15, q = lane & 3, j = m >> 2;
  uint32_t word = 0;
  float s = 0.f, z = 0.f;
  if (on && valid) {
    word = *reinterpret_cast<const uint32_t*>(codes + 16 * q + 4 * j);
    s = __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t*>(scales + 2 * j) << 16);
    z = __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t*>(scales + 8 + 2 * j) << 16);
  }
  // lane q wants nibble q (of each 16-bit half: channels g = 2 t, 2 t + 1) of the 4 words t
  float x[8];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint32_t w = __shfl_sync(0xffffffffu, word, (lane & ~3) + t) >> (4 * q);
    x[2 * t] = z + s * (float)(w & 15u);
    x[2 * t + 1] = z + s * (float)(w >> 16 & 15u);
  }
  if (on)
    *reinterpret_cast<uint4*>(dst + 8 * m) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                        pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

__global__ void __launch_bounds__(kThreads) kv4_load_kernel(const __grid_constant__ LoadParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long gw = (long long)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int row = (int)(gw / p.warps_per_row), part = (int)(gw % p.warps_per_row);
  if (row >= p.rows) return;
  const int b = p.cu ? sequence_of_row(p.cu, p.B, row, lane) : row;
  if (b < 0) return;  // a row of no sequence is left as it was
  const int slot = (p.starts ? p.starts[b] : 0) + (p.cu ? row - p.cu[b] : 0);
  const bool valid = slot >= 0 && slot < p.c.capacity;
  if (!valid && lane == 0 && p.status) atomicCAS(&p.status->code, 0, kStatusInvalidArg);
  for (int h0 = 2 * part; h0 < p.Hkv; h0 += 2 * p.warps_per_row) {
    const int h = h0 + (lane >> 4);
    const bool on = h < p.Hkv;
    const long long off = on ? h : 0;
    const size_t at = ((size_t)b * p.Hkv + off) * p.c.capacity + (valid ? slot : 0);
    load_row(static_cast<__nv_bfloat16*>(p.k.ptr) + row * p.k.row + off * p.k.head, p.c.k + at * kKv4Codes,
             p.c.k_scale + at * kKv4Scales, on, valid, lane);
    load_row(static_cast<__nv_bfloat16*>(p.v.ptr) + row * p.v.row + off * p.v.head, p.c.v + at * kKv4Codes,
             p.c.v_scale + at * kKv4Scales, on, valid, lane);
  }
}

}  // namespace

cudaError_t launch_kv4_store(const HeadRows& k, const HeadRows& v, int rows, const int* cu, const int* starts, int B,
                             int Hkv, const Kv4Cache& c, DevStatus* st, cudaStream_t s) {
  const bool append = starts == nullptr || starts == c.lens;
  StoreParams p{k, v, cu, append ? c.lens : starts, c, rows, B, Hkv, (Hkv + 1) / 2, append ? 1 : 0, st};
  if (append && !cu) {  // a block per row
    p.warps_per_row = p.warps_per_row < kThreads / 32 ? p.warps_per_row : kThreads / 32;
    return rows > 0 ? launch_pdl(kv4_store_kernel, rows, p.warps_per_row * 32, 0, s, p) : cudaSuccess;
  }
  const long long warps = (long long)rows * p.warps_per_row;
  const long long grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
  cudaError_t e = launch_pdl(kv4_store_kernel, dim3((unsigned)(grid > 0 ? grid : 1)), kThreads, 0, s, p);
  if (e != cudaSuccess || !append) return e;
  return launch_pdl(kv4_lens_kernel, (B + 255) / 256, 256, 0, s, cu, c.lens, B, c.capacity);
}

cudaError_t launch_kv4_load(const HeadRows& k, const HeadRows& v, int rows, const int* cu, const int* starts, int B,
                            int Hkv, const Kv4Cache& c, DevStatus* st, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  LoadParams p{k, v, cu, starts, c, rows, B, Hkv, (Hkv + 1) / 2, st};
  const long long warps = (long long)rows * p.warps_per_row;
  return launch_pdl(kv4_load_kernel, dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32))), kThreads, 0, s, p);
}

}  // namespace blk

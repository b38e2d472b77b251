// Per-head RMSNorm of queries and keys and the rotary in one pass over packed
// token rows ("apertus", "Queries and keys are normed per head, before the
// rotary"; the rotary turns element i together with i + d/2):
//   y = x / sqrt(mean(x^2) + eps) * gain
//   out_i       = y_i cos(a_i) - y_{i+d/2} sin(a_i)
//   out_{i+d/2} = y_{i+d/2} cos(a_i) + y_i sin(a_i),  a_i = pos[axis(i)] * inv_freq_i
// with up to four position axes (image and video models: time, height, width),
// each turning its own pairs. Angles come from the handle's table, computed in
// double (fp32 angles of far positions would lose their turns).
//
// HBM-bound: each value is read and written once. A head's row is held by L lanes,
// each with one 16-byte chunk of the lower half and the matching one of the upper
// half, so that a pair never leaves its thread; the norm's sum takes log2(L)
// shuffles. A lane keeps its pairs' cos and sin in registers over the heads of its
// row, so the table is read once per row and warp, not once per head; a head's values are
// loaded a turn ahead, the first ones before the position and its angles are looked up.
// 8191 rows of 40 heads, norms and three axes: 31.0 us, 5.4 TB/s (35.4 with the loads in turn);
// 16384 rows of 64 heads, no norms: 88.4 us, 6.1 TB/s (95.0).
#include "common.cuh"
#include "kernels.h"

namespace blk {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 4;  // per SM: 64 registers. 5 spill; a turn more in flight takes too many for 4
constexpr int kStatusInvalidArg = 1;  // == BLK_ERR_INVALID_ARG

struct RopeParams {
  HeadRows q, k, qo, ko;
  const void *q_gain, *k_gain;  // null: no norm
  const float2* table;          // [max_pos][half] (cos, sin), or null: no rotary
  const int* pos;               // [n_axes][rows]
  PairAxes axes;
  int rows, H, Hkv, half, max_pos, n_axes;
  int warps_per_row;
  float eps, inv_d;
  DevStatus* status;
};

template <typename T>
struct Chunk;  // 16 bytes of T as floats
template <>
struct Chunk<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = unpack_bf16x2(w[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};

// L: lanes per head row (a power of two); lanes past half / N hold nothing.
template <typename T, int L, bool NORM>
__global__ void __launch_bounds__(kThreads, kBlocks) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  typedef Chunk<T> C;
  constexpr int N = C::N;
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kHeadsPerWarp = 32 / L;
  const int lane = threadIdx.x & 31, sub = lane % L, hw = lane / L;
  const long long gw = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int row = (int)(gw / p.warps_per_row), part = (int)(gw % p.warps_per_row);
  if (row >= p.rows) return;
  const bool mine = sub * N < p.half;
  const int c = mine ? sub * N : 0;
  const int heads = p.H + p.Hkv, h_on = p.warps_per_row * kHeadsPerWarp;
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  auto fetch = [&](int h) {
    if (h < heads && mine) {
      const bool is_q = h < p.H;
      const T* x = static_cast<const T*>(is_q ? p.q.ptr : p.k.ptr) + row * (is_q ? p.q.row : p.k.row) +
                   (long long)(is_q ? h : h - p.H) * (is_q ? p.q.head : p.k.head) + c;
      lo = *reinterpret_cast<const uint4*>(x);
      hi = *reinterpret_cast<const uint4*>(x + p.half);
    }
  };
  int h = part * kHeadsPerWarp + hw;
  fetch(h);  // on the way while the position and then its angles are looked up
  float cs[N], sn[N];
#pragma unroll
  for (int i = 0; i < N; ++i) cs[i] = 1.f, sn[i] = 0.f;
  if (p.table) {
    bool bad = false;
    auto position = [&](int axis) {
      const int x = p.pos[(size_t)axis * p.rows + row];
      bad |= x < 0 || x >= p.max_pos;
      return min(max(x, 0), p.max_pos - 1);  // never read past the table
    };
    if (p.n_axes == 1) {
      const float4* t = reinterpret_cast<const float4*>(p.table + (size_t)position(0) * p.half + c);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float4 v = t[i / 2];
        cs[i] = v.x, sn[i] = v.y, cs[i + 1] = v.z, sn[i + 1] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int pair = c + i;
        const int axis = (p.axes.w[pair >> 4] >> (2 * (pair & 15))) & 3;
        const float2 v = p.table[(size_t)position(axis) * p.half + pair];
        cs[i] = v.x, sn[i] = v.y;
      }
    }
    if (bad && p.status) atomicCAS(&p.status->code, 0, kStatusInvalidArg);
  }
  for (; h - hw < heads; h += h_on) {
    const bool is_q = h < p.H;
    float a[N], b[N];
    C::unpack(lo, a);
    C::unpack(hi, b);
    fetch(h + h_on);
    if constexpr (NORM) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) ss += a[i] * a[i] + b[i] * b[i];
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(ss * p.inv_d + p.eps);
      const T* gain = static_cast<const T*>(is_q ? p.q_gain : p.k_gain) + c;
      float g[N];
      C::unpack(*reinterpret_cast<const uint4*>(gain), g);
#pragma unroll
      for (int i = 0; i < N; ++i) a[i] *= r * g[i];
      C::unpack(*reinterpret_cast<const uint4*>(gain + p.half), g);
#pragma unroll
      for (int i = 0; i < N; ++i) b[i] *= r * g[i];
    }
    if (h < heads && mine) {
      T* y = static_cast<T*>(is_q ? p.qo.ptr : p.ko.ptr) + row * (is_q ? p.qo.row : p.ko.row) +
             (long long)(is_q ? h : h - p.H) * (is_q ? p.qo.head : p.ko.head) + c;
      float u[N];
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] = a[i] * cs[i] - b[i] * sn[i];
      *reinterpret_cast<uint4*>(y) = C::pack(u);
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] = b[i] * cs[i] + a[i] * sn[i];
      *reinterpret_cast<uint4*>(y + p.half) = C::pack(u);
    }
  }
}

template <typename T, int L>
cudaError_t launch_l(RopeParams p, int num_sms, cudaStream_t s) {
  const int groups = (p.H + p.Hkv + 32 / L - 1) / (32 / L);  // warp loads of a row
  // one warp per row when the rows alone bring 24 warps to each SM, more when they do not.
  // 1200 bf16 rows of 40 heads 6.6 us, 2000 in fp32 9.3; with 32 warps an SM 7.9 and 10.1, with 12
  // 7.4 and 11.9.
  int w = 1;
  while (w < groups && (long long)p.rows * w < 24ll * num_sms) w *= 2;
  p.warps_per_row = w < groups ? w : groups;
  const long long warps = (long long)p.rows * p.warps_per_row;
  const long long grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
  return launch_pdl(p.q_gain ? qk_norm_rope_kernel<T, L, true> : qk_norm_rope_kernel<T, L, false>,
                    dim3((unsigned)grid), kThreads, 0, s, p);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const HeadRows& q, const HeadRows& k, const HeadRows& qo, const HeadRows& ko, int rows,
                                int H, int Hkv, int d, const int* pos, int n_axes, const PairAxes& axes,
                                const void* q_gain, const void* k_gain, float eps, const float2* table, int max_pos,
                                bool bf16, int num_sms, DevStatus* st, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  RopeParams p{q, k, qo, ko, q_gain, k_gain, table, pos, axes, rows, H, Hkv, d / 2, max_pos, n_axes, 1, eps,
               1.f / (float)d, st};
  if (bf16) return launch_l<__nv_bfloat16, 8>(p, num_sms, s);  // head_dim 128
  const int lanes = d / 8;  // 4 pairs a lane
  if (lanes <= 2) return launch_l<float, 2>(p, num_sms, s);
  if (lanes <= 4) return launch_l<float, 4>(p, num_sms, s);
  if (lanes <= 8) return launch_l<float, 8>(p, num_sms, s);
  if (lanes <= 16) return launch_l<float, 16>(p, num_sms, s);
  return launch_l<float, 32>(p, num_sms, s);
}

}  // namespace blk

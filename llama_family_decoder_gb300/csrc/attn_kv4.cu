// Decode attention over the 4-bit KV cache: one query per sequence,
//   o[b, h, :] = softmax_s(q[b, h] . k^[b, j, s] / sqrt(128)) v^[b, j, s],  j = h / (H / Hkv),
// with k^, v^ = offset + scale * code (see kv4.cu for the rows).
//
// A warp per (sequence, head) walks the keys; a lane holds two code bytes of each row
// (four channels).
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace blk {

namespace {

constexpr int kD = 128;

struct Kv4Params {
  HeadRows q, o;
  Kv4Cache c;
  int B, H, Hkv, window;
  float sl;
};

__global__ void __launch_bounds__(128) attn_kv4_kernel(const __grid_constant__ Kv4Params p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long u = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (u >= (long long)p.B * p.H) return;
  const int b = (int)(u / p.H), h = (int)(u % p.H), j = h / (p.H / p.Hkv);
  const int len = max(0, min(p.c.lens[b], p.c.capacity));
  const int first = p.window > 0 ? max(0, len - p.window) : 0;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q.ptr) + b * p.q.row + h * p.q.head;
  int ch[4];
  float qv[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    ch[i] = kv4_byte_channel(2 * lane + (i >> 1)) + 8 * (i & 1);
    qv[i] = __bfloat162float(q[ch[i]]);
  }
  const size_t row0 = ((size_t)b * p.Hkv + j) * p.c.capacity;
  auto values = [&](const uint8_t* codes, const uint8_t* scales, size_t row, float (&x)[4]) {
    const uint32_t w = *reinterpret_cast<const uint16_t*>(codes + row * kKv4Codes + 2 * lane);
    const __nv_bfloat16* sc = reinterpret_cast<const __nv_bfloat16*>(scales + row * kKv4Scales);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int g = ch[i] >> 5;
      x[i] = __bfloat162float(sc[4 + g]) + __bfloat162float(sc[g]) * (float)(w >> (4 * i) & 15u);
    }
  };
  for (int s = first; s < len; ++s) {
    float x[4], dot = 0.f;
    values(p.c.k, p.c.k_scale, row0 + s, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) dot += qv[i] * x[i];
    dot = warp_sum(dot) * p.sl;
    const float mn = fmaxf(m, dot), a = __expf(m - mn), e = __expf(dot - mn);
    m = mn;
    values(p.c.v, p.c.v_scale, row0 + s, x);
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = acc[i] * a + e * x[i];
  }
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o.ptr) + b * p.o.row + h * p.o.head;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[ch[i]] = __float2bfloat16_rn(len > first ? acc[i] / l : 0.f);
}

}  // namespace

size_t attn_kv4_ws_bytes(int B, int H, int Hkv, int num_sms) { return 0; }

cudaError_t launch_attn_decode_kv4(const HeadRows& q, const Kv4Cache& c, const HeadRows& o, int B, int H, int Hkv,
                                   int window, void* ws, int num_sms, DevStatus* st, unsigned long long wait_ns,
                                   cudaStream_t s, const char** why) {
  Kv4Params p{q, o, c, B, H, Hkv, window, 1.f / sqrtf((float)kD)};
  return launch_pdl(attn_kv4_kernel, dim3((unsigned)(((long long)B * H + 3) / 4)), 128, 0, s, p);
}

}  // namespace blk

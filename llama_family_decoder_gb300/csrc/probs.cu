// Probabilities of the rows of a model's logits: softmax(x / temperature) in fp32, or for temperature 0 all of it
// on the largest logit (the first one of several). One CTA a row, HBM-bound: the logits are read twice (the second
// time from L2), a running maximum and sum in the log2 domain, then the probabilities.
#include "common.cuh"
#include "kernels.h"

namespace blk {

namespace {

constexpr int kThreads = 512;

struct Peak {  // a maximum, where it is first, and the sum of 2^(x - maximum)
  float m, l;
  int at;
};
__device__ __forceinline__ Peak join(const Peak& a, const Peak& b) {
  const bool first = a.m > b.m || (a.m == b.m && a.at <= b.at);
  const float m = fmaxf(a.m, b.m), mu = m == -INFINITY ? 0.f : m;
  return {m, a.l * exp2f(a.m - mu) + b.l * exp2f(b.m - mu), first ? a.at : b.at};
}

__global__ void __launch_bounds__(kThreads) probs_kernel(const uint4* __restrict__ x, int vocab, float scale,
                                                         int greedy, float4* __restrict__ out) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ Peak sh[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, chunks = vocab / 8;
  const uint4* const row = x + (size_t)blockIdx.x * chunks;
  auto values = [&](int i, float (&f)[8]) {
    const uint4 u = row[i];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 t = unpack_bf16x2(w[k]);
      f[2 * k] = t.x * scale;
      f[2 * k + 1] = t.y * scale;
    }
  };
  Peak p{-INFINITY, 0.f, 0x7fffffff};
  for (int i = threadIdx.x; i < chunks; i += kThreads) {
    float f[8];
    values(i, f);
    float m = p.m;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (f[k] > m) m = f[k], p.at = 8 * i + k;
    const float mu = m == -INFINITY ? 0.f : m;
    p.l *= exp2f(p.m - mu);
#pragma unroll
    for (int k = 0; k < 8; ++k) p.l += exp2f(f[k] - mu);
    p.m = m;
  }
  auto reduce = [&](Peak q, int from) {
    for (int o = from; o > 0; o >>= 1) {
      const Peak r{__shfl_xor_sync(0xffffffffu, q.m, o), __shfl_xor_sync(0xffffffffu, q.l, o),
                   __shfl_xor_sync(0xffffffffu, q.at, o)};
      // the lower lane's first: both lanes of a pair get the same sum
      q = lane & o ? join(r, q) : join(q, r);
    }
    return q;
  };
  p = reduce(p, 16);
  if (lane == 0) sh[warp] = p;
  __syncthreads();
  p = reduce(sh[lane % (kThreads / 32)], kThreads / 64);
  const float mu = p.m == -INFINITY ? 0.f : p.m, inv = 1.f / p.l;
  float4* const to = out + (size_t)blockIdx.x * (vocab / 4);
  for (int i = threadIdx.x; i < chunks; i += kThreads) {
    float f[8];
    if (!greedy) {
      values(i, f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = exp2f(f[k] - mu) * inv;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = 8 * i + k == p.at ? 1.f : 0.f;
    }
    to[2 * i] = make_float4(f[0], f[1], f[2], f[3]);
    to[2 * i + 1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

}  // namespace

cudaError_t launch_probs(const void* logits, int rows, int vocab, float temperature, float* out, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  if (vocab % 8) return cudaErrorInvalidValue;
  const bool greedy = temperature == 0.f;
  return launch_pdl(probs_kernel, rows, kThreads, 0, s, static_cast<const uint4*>(logits), vocab,
                    greedy ? 1.f : 1.4426950408889634f / temperature, greedy ? 1 : 0, reinterpret_cast<float4*>(out));
}

}  // namespace blk

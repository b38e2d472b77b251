// Probabilities of the rows of a model's logits: softmax(x / temperature) in fp32, or for temperature 0 all of it
// on the largest logit (the first one of several; a NaN is not one, and a row with a NaN and nothing above -inf gives NaN).
// A cluster of CTAs takes a row, a stretch each: a running maximum and
// sum in the log2 domain, joined over the CTA and in distributed shared memory, then the probabilities from the logits
// read again (from L1 or L2). Few rows: a launch and two dependent rounds of loads. Many: two waves of CTAs above 304 rows, and each
// value read and its exponential taken twice. What it adds to the model's call: 64 rows of 32000 11.7 us (one CTA a row:
// 14.6; their bytes at HBM's rate 1.8), of 128000 19.8 (36.3; 7.2), 400 rows of 32000 23.5 (11.3).
#include <algorithm>
#include <cfloat>

#include "paged.cuh"

namespace blk {

namespace {

constexpr int kThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kAtOnce = 4;  // chunks of eight values of a thread under way

constexpr int kNowhere = 0x7fffffff;
struct Peak {  // a maximum, where it is first (kNowhere: nothing is above -inf), and the sum of 2^((x - maximum) scale)
  float m, l;
  int at;
};
__device__ __forceinline__ Peak join(const Peak& a, const Peak& b, float scale) {
  const bool first = a.m > b.m || (a.m == b.m && a.at <= b.at);
  const float m = fmaxf(a.m, b.m), mu = m == -INFINITY ? 0.f : m;
  return {m, a.l * exp2f((a.m - mu) * scale) + b.l * exp2f((b.m - mu) * scale), first ? a.at : b.at};
}

__device__ __forceinline__ Peak ld_dsmem_peak(uint32_t addr) {
  Peak p;
  asm volatile("ld.shared::cluster.f32 %0, [%3];\n\tld.shared::cluster.f32 %1, [%3 + 4];\n\tld.shared::cluster.u32 %2, [%3 + 8];"
               : "=f"(p.m), "=f"(p.l), "=r"(p.at)
               : "r"(addr)
               : "memory");
  return p;
}

__global__ void __launch_bounds__(kThreads, 2) probs_kernel(const uint4* __restrict__ x, int vocab, const int* __restrict__ cu,
                                                            int B, float scale, int greedy, float4* __restrict__ out, int size) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ Peak sh[kThreads / 32], own;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, chunks = vocab / 8;
  const int row_at = blockIdx.x / size, rank = blockIdx.x % size, per = (chunks + size - 1) / size;
  if (cu && (row_at < cu[0] || row_at >= cu[B])) return;  // a row of no sequence, the whole cluster alike
  const int first = min(chunks, rank * per) + threadIdx.x, end = min(chunks, (rank + 1) * per);
  const uint4* const row = x + (size_t)row_at * chunks;
  auto values = [&](const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 t = unpack_bf16x2(w[k]);
      f[2 * k] = t.x;
      f[2 * k + 1] = t.y;
    }
  };
  auto each = [&](auto&& use) {  // use(chunk, its values), in order
    for (int i0 = first; i0 < end; i0 += kAtOnce * kThreads) {
      uint4 u[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) u[k] = row[min(i0 + k * kThreads, chunks - 1)];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (i0 + k * kThreads < end) {
          float f[8];
          values(u[k], f);
          use(i0 + k * kThreads, f);
        }
    }
  };
  Peak p{-INFINITY, 0.f, kNowhere};
  each([&](int i, const float (&f)[8]) {
    float m = p.m;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (f[k] > m) m = f[k], p.at = 8 * i + k;
    const float mu = m == -INFINITY ? 0.f : m;
    p.l *= exp2f((p.m - mu) * scale);
#pragma unroll
    for (int k = 0; k < 8; ++k) p.l += exp2f((f[k] - mu) * scale);
    p.m = m;
  });
  auto reduce = [&](Peak q, int from) {
    for (int o = from; o > 0; o >>= 1) {
      const Peak r{__shfl_xor_sync(0xffffffffu, q.m, o), __shfl_xor_sync(0xffffffffu, q.l, o),
                   __shfl_xor_sync(0xffffffffu, q.at, o)};
      // the lower lane's first: both lanes of a pair get the same sum
      q = lane & o ? join(r, q, scale) : join(q, r, scale);
    }
    return q;
  };
  p = reduce(p, 16);
  if (lane == 0) sh[warp] = p;
  __syncthreads();
  p = reduce(sh[lane % (kThreads / 32)], kThreads / 64);
  if (size > 1) {
    if (threadIdx.x == 0) own = p;
    __syncwarp();
    cluster_sync_all();
    Peak q = ld_dsmem_peak(map_shared_rank(smem_u32(&own), 0));
    for (int r = 1; r < size; ++r) q = join(q, ld_dsmem_peak(map_shared_rank(smem_u32(&own), r)), scale);
    p = q;
    __syncwarp();
    cluster_arrive();  // (waited for below: nobody leaves while its peak may be read)
  }
  const float mu = p.m == -INFINITY ? 0.f : p.m, inv = 1.f / p.l;
  // nothing above -inf: the first -inf is the largest, unless the sum (of zeros) tells of a NaN
  const int top = p.at == kNowhere ? 0 : p.at;
  const float none = p.at == kNowhere && p.l != p.l ? p.l : 0.f;
  float4* const to = out + (size_t)row_at * (vocab / 4);
  each([&](int i, float (&f)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = greedy ? (8 * i + k == top ? 1.f + none : none) : exp2f((f[k] - mu) * scale) * inv;
    to[2 * i] = make_float4(f[0], f[1], f[2], f[3]);
    to[2 * i + 1] = make_float4(f[4], f[5], f[6], f[7]);
  });
  if (size > 1) {
    __syncwarp();
    cluster_wait();
  }
}

}  // namespace

cudaError_t launch_probs(const void* logits, int rows, int vocab, const int* cu, int B, float temperature, float* out,
                         int num_sms, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  if (vocab % 8) return cudaErrorInvalidValue;
  const bool greedy = temperature == 0.f;
  if ((long long)rows * kMaxCluster > 0x7fffffff) return cudaErrorInvalidValue;
  // clusters as long as they are all resident (two CTAs an SM) and a thread has a chunk
  int size = 1;
  while (size < kMaxCluster && 2ll * size * rows <= 2ll * num_sms && size * kThreads < vocab / 8) size *= 2;
  // finite and not 0: the largest logit's exponent is 0, an infinite one's stays infinite
  const float scale = greedy ? 1.f : std::min(std::max(1.4426950408889634f / temperature, FLT_MIN), FLT_MAX);
  return launch_clusters(probs_kernel, rows * size, kThreads, 0, size, s, static_cast<const uint4*>(logits), vocab, cu, B, scale,
                         greedy ? 1 : 0, reinterpret_cast<float4*>(out), size);
}

}  // namespace blk

// Attention of a sequence's new rows (one token, a chain or a tree of drafted ones) over the paged
// cache, grouped-query, head_dim 128:
//   o = softmax(q k^T / sqrt(128)) v over the sequence's slots and the row's ancestors and itself.
// A warp takes a row and head, four channels a lane, and goes over the keys one at a time with the
// running maximum and sum of the softmax.
#include "paged.cuh"

namespace blk {

namespace {

constexpr int kThreads = 256;
constexpr float kScaleLog2 = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)

struct PagedAttnParams {
  HeadRows q, o;
  PagedCache c;
  const int *cu, *parents;
  int rows, B, H, Hkv, window;
  DevStatus* status;
};

__global__ void __launch_bounds__(kThreads) attn_paged_kernel(const __grid_constant__ PagedAttnParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  const SeqRows sr = seq_rows(p.cu, b, p.rows);
  const int len = p.c.lens[b];
  const bool tree = p.parents != nullptr;
  const bool fits = len >= 0 && (long long)len + sr.n <= page_slots(p.c);
  const int n = fits ? (tree ? min(sr.n, kMaxNodes) : sr.n) : 0;
  if (blockIdx.x == 0 && threadIdx.x == 0 && (!fits || seq_bad(p.cu, b, p.rows) || n < sr.n))
    record(p.status, fits || len < 0 ? kStatusInvalidArg : kStatusCacheFull);
  for (long long w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < (long long)n * p.H;
       w += gridDim.x * (kThreads / 32)) {
    const int i = (int)(w / p.H), h = (int)(w % p.H), kvh = h / (p.H / p.Hkv);
    unsigned long long kin = 0;
    int depth = i;
    if (tree) {
      depth = 0;
      for (int j = i; j >= 0;) {
        if (p.window == 0 || depth < p.window) kin |= 1ull << j;
        const int up = p.parents[sr.lo + j];
        if (up >= j) record(p.status, kStatusInvalidArg);
        if (up < 0 || up >= j) break;
        j = up;
        ++depth;
      }
    }
    const int first = p.window > 0 ? max(0, len + depth - p.window + 1) : 0;
    const int end = len + (tree ? n : i + 1);
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    auto load4 = [](const __nv_bfloat16* x, float (&f)[4]) {
      const uint2 u = *reinterpret_cast<const uint2*>(x);
      const float2 a = unpack_bf16x2(u.x), c = unpack_bf16x2(u.y);
      f[0] = a.x, f[1] = a.y, f[2] = c.x, f[3] = c.y;
    };
    load4(static_cast<const __nv_bfloat16*>(p.q.ptr) + (sr.lo + i) * p.q.row + h * p.q.head + 4 * lane, q);
    for (int s = first; s < end; ++s) {
      if (tree && s >= len && !(kin >> (s - len) & 1)) continue;
      const PagePlace at = page_place(p.c, b, s);
      if (at.page < 0) {
        record(p.status, kStatusInvalidArg);
        continue;
      }
      const long long row = place_row(p.c, at, p.Hkv, kvh) * 128 + 4 * lane;
      float k[4], v[4];
      load4(static_cast<const __nv_bfloat16*>(p.c.k) + row, k);
      load4(static_cast<const __nv_bfloat16*>(p.c.v) + row, v);
      const float x = warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]) * kScaleLog2;
      const float top = fmaxf(m, x), mu = top == -INFINITY ? 0.f : top;
      const float keep = exp2f(m - mu), e = exp2f(x - mu);
      m = top;
      l = l * keep + e;
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = o[c] * keep + e * v[c];
    }
    uint2 u;
    u.x = pack_bf16x2(o[0] / l, o[1] / l);
    u.y = pack_bf16x2(o[2] / l, o[3] / l);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o.ptr) + (sr.lo + i) * p.o.row + h * p.o.head + 4 * lane) = u;
  }
}

}  // namespace

size_t attn_paged_ws_bytes(int, int, int, int, int) { return 0; }

cudaError_t launch_attn_paged(const HeadRows& q, const PagedCache& c, const HeadRows& o, int rows, const int* cu,
                              const int* parents, int B, int H, int Hkv, int window, void*, int num_sms,
                              DevStatus* st, unsigned long long, cudaStream_t s, const char** why) {
  if (rows <= 0 || B <= 0) return cudaSuccess;
  if (B > 65535) {
    *why = "paged attention: at most 65535 sequences";
    return cudaErrorInvalidValue;
  }
  PagedAttnParams p{q, o, c, cu, parents, rows, B, H, Hkv, window, st};
  return launch_pdl(attn_paged_kernel, dim3(32, (unsigned)B), kThreads, 0, s, p);
}

}  // namespace blk

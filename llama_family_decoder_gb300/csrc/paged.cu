// The paged KV cache: appending rows with their norm and rotary, and keeping an accepted path.
//
// Append: per-head RMSNorm of queries and keys ("apertus", "Queries and keys are normed per head,
// before the rotary") and the rotary over the first `dims` channels of a head in one pass, as in
// qk_rope.cu, here with the positions taken from the cache's lengths, keys and values written to
// their pages instead of dense rows, and two layouts of a pair:
//   y = x / sqrt(mean(x^2) + eps) * gain
//   out_a = y_a cos(t_j) - y_b sin(t_j), out_b = y_b cos(t_j) + y_a sin(t_j),  t_j = pos * inv_freq_j
//   (a, b) = (j, j + dims / 2), or interleaved (2j, 2j + 1); channels from dims on stay as they are.
// HBM-bound: each value is read and written once. L lanes hold a head's row, 2 N channels each in two
// 16-byte chunks that hold both channels of N pairs in either layout, and the same N pairs j =
// N sub .. : the layouts differ in where a lane's chunks are and in which channels of them meet. The
// cos and sin of a lane's pairs stay in registers over the heads of its row; a head's values are
// loaded a turn ahead, the first ones while the row's sequence, length and angles are looked up (a
// search of cu_seqlens 32 numbers at a time, then three dependent loads). Measured (a graph of calls): a token of each of 64
// sequences, 32 + 8 heads with norms 3.8 us, a launch and those loads; 8 prompts of up to 2048 tokens 19.9 us,
// 5.7 TB/s; fp32, 3 of up to 333 with heads of 64 channels 3.6 us. A row's heads go to more warps (24 an SM) while rows are few.
#include "paged.cuh"

namespace blk {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 4;  // per SM: 64 registers

struct AppendParams {
  HeadRows q, k, v, qo;
  const void *q_gain, *k_gain;  // null: no norm
  const float2* table;          // [max_pos][dims / 2] (cos, sin), or null: no rotary
  const int *cu, *depths;       // null: a row per sequence; the row's number in its sequence
  PagedCache c;
  int rows, B, H, Hkv, d, dims, max_pos;
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

// The sequence whose rows hold `row`, or -1 (a whole warp; cu non-null).
__device__ __forceinline__ int find_sequence(const int* cu, int B, int row, int lane) {
  if (row < cu[0]) return -1;
  int lo = 0, hi = B;  // cu[lo] <= row, as far as the list rises
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const int n = __popc(__ballot_sync(0xffffffffu, at < hi && cu[at] <= row));
    lo += n * step;
    hi = min(hi, lo + step);
  }
  return cu[lo] <= row && row < cu[lo + 1] ? lo : -1;
}

// L: lanes per head row (a power of two); lanes past d / (2 N) hold nothing.
template <typename T, int L, bool NORM, bool INTER>
__global__ void __launch_bounds__(kThreads, kBlocks) paged_append_kernel(const __grid_constant__ AppendParams p) {
  typedef Chunk<T> C;
  constexpr int N = C::N;
  constexpr int kHeadsPerWarp = 32 / L;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, sub = lane % L, hw = lane / L;
  const long long gw = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const long long row_l = gw / p.warps_per_row;
  const int part = (int)(gw % p.warps_per_row);
  if (p.cu && blockIdx.x == gridDim.x - 1) {  // the last block, one that the rows need not, looks the list over
    bool bad = false;
    for (int b = threadIdx.x; b < p.B; b += kThreads) bad |= seq_bad(p.cu, b, p.rows);
    if (bad) record(p.status, kStatusInvalidArg);
  }
  if (row_l >= p.rows) return;
  const int row = (int)row_l;
  const bool mine = sub * 2 * N < p.d;
  const bool turns = p.table && sub * 2 * N < p.dims;
  // a lane's two chunks: of the lower and upper half of the pairs, or side by side
  const int c_lo = !mine ? 0 : turns && !INTER ? sub * N : sub * 2 * N;
  const int c_hi = !mine ? 0 : turns && !INTER ? p.dims / 2 + sub * N : c_lo + N;
  const int heads = p.H + 2 * p.Hkv, h_on = p.warps_per_row * kHeadsPerWarp;
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  auto fetch = [&](int h) {
    if (h < heads && mine) {
      const HeadRows& x = h < p.H ? p.q : h < p.H + p.Hkv ? p.k : p.v;
      const int j = h < p.H ? h : h < p.H + p.Hkv ? h - p.H : h - p.H - p.Hkv;
      const T* at = static_cast<const T*>(x.ptr) + row * x.row + j * x.head;
      lo = *reinterpret_cast<const uint4*>(at + c_lo);
      hi = *reinterpret_cast<const uint4*>(at + c_hi);
    }
  };
  int h = part * kHeadsPerWarp + hw;
  fetch(h);
  int b = row, i = 0;
  if (p.cu) {
    b = find_sequence(p.cu, p.B, row, lane);
    if (b < 0) return;  // a row of no sequence
    i = row - max(p.cu[b], 0);
  }
  const int len = p.c.lens[b];
  const long long slot = (long long)len + i;
  const bool fits = len >= 0 && slot < page_slots(p.c);
  PagePlace at{-1, 0};
  if (fits) at = page_place(p.c, b, (int)slot);
  if (at.page < 0) record(p.status, fits || len < 0 ? kStatusInvalidArg : kStatusCacheFull);
  float cs[N], sn[N];
#pragma unroll
  for (int n = 0; n < N; ++n) cs[n] = 1.f, sn[n] = 0.f;
  if (turns) {
    const long long want = (long long)len + (p.depths ? p.depths[row] : i);
    const int pos = (int)(want < 0 ? 0 : want < p.max_pos ? want : p.max_pos - 1);  // never read past the table
    if (pos != want) record(p.status, kStatusInvalidArg);
    const float4* t = reinterpret_cast<const float4*>(p.table + (size_t)pos * (p.dims / 2) + sub * N);
#pragma unroll
    for (int n = 0; n < N; n += 2) {
      const float4 v = t[n / 2];
      cs[n] = v.x, sn[n] = v.y, cs[n + 1] = v.z, sn[n + 1] = v.w;
    }
  }
  for (; h - hw < heads; h += h_on) {
    const bool is_q = h < p.H, is_v = h >= p.H + p.Hkv;
    uint4 u_lo = lo, u_hi = hi;
    fetch(h + h_on);
    float a[N], b2[N];
    C::unpack(u_lo, a);
    C::unpack(u_hi, b2);
    if constexpr (NORM) {
      float ss = 0.f;
#pragma unroll
      for (int n = 0; n < N; ++n) ss += a[n] * a[n] + b2[n] * b2[n];
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!is_v) {
        const float r = rsqrtf(ss * p.inv_d + p.eps);
        const T* gain = static_cast<const T*>(is_q ? p.q_gain : p.k_gain);
        float g[N];
        C::unpack(*reinterpret_cast<const uint4*>(gain + c_lo), g);
#pragma unroll
        for (int n = 0; n < N; ++n) a[n] *= r * g[n];
        C::unpack(*reinterpret_cast<const uint4*>(gain + c_hi), g);
#pragma unroll
        for (int n = 0; n < N; ++n) b2[n] *= r * g[n];
      }
    }
    if (h >= heads || !mine) continue;
    if (!is_v) {
      if constexpr (INTER) {  // pairs (2j, 2j + 1) of the lower chunk, then of the upper one
#pragma unroll
        for (int n = 0; n < N / 2; ++n) {
          const float x0 = a[2 * n], x1 = a[2 * n + 1], y0 = b2[2 * n], y1 = b2[2 * n + 1];
          a[2 * n] = x0 * cs[n] - x1 * sn[n];
          a[2 * n + 1] = x1 * cs[n] + x0 * sn[n];
          b2[2 * n] = y0 * cs[N / 2 + n] - y1 * sn[N / 2 + n];
          b2[2 * n + 1] = y1 * cs[N / 2 + n] + y0 * sn[N / 2 + n];
        }
      } else {
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const float x0 = a[n], x1 = b2[n];
          a[n] = x0 * cs[n] - x1 * sn[n];
          b2[n] = x1 * cs[n] + x0 * sn[n];
        }
      }
      u_lo = C::pack(a);
      u_hi = C::pack(b2);
    }
    T* to;
    if (is_q) {
      to = static_cast<T*>(p.qo.ptr) + row * p.qo.row + h * p.qo.head;
    } else {
      if (at.page < 0) continue;
      const int j = is_v ? h - p.H - p.Hkv : h - p.H;
      to = static_cast<T*>(is_v ? p.c.v : p.c.k) + place_row(p.c, at, p.Hkv, j) * p.d;
    }
    *reinterpret_cast<uint4*>(to + c_lo) = u_lo;
    *reinterpret_cast<uint4*>(to + c_hi) = u_hi;
  }
}

template <typename T, int L>
cudaError_t launch_append(AppendParams p, bool inter, int num_sms, cudaStream_t s) {
  const int groups = (p.H + 2 * p.Hkv + 32 / L - 1) / (32 / L);  // warp loads of a row
  int w = 1;
  while (w < groups && (long long)p.rows * w < 24ll * num_sms) w *= 2;
  p.warps_per_row = w < groups ? w : groups;
  const long long warps = (long long)p.rows * p.warps_per_row;
  const long long grid = (warps + kThreads / 32 - 1) / (kThreads / 32) + (p.cu ? 1 : 0);
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  const bool norm = p.q_gain != nullptr;
  auto kernel = inter ? (norm ? paged_append_kernel<T, L, true, true> : paged_append_kernel<T, L, false, true>)
                      : (norm ? paged_append_kernel<T, L, true, false> : paged_append_kernel<T, L, false, false>);
  return launch_pdl(kernel, dim3((unsigned)grid), kThreads, 0, s, p);
}

// Keep: slot start + path[j] -> slot start + j for the kept nodes j of each sequence, in every layer's
// cache, and lens[b] = start + counts[b]. A cluster of CTAs takes a sequence; a warp takes the rows
// of one (layer, K or V, head) at a time, eight of them loaded before any of the eight is stored:
// path rises, so that no later row's source is behind an earlier row's place. The lengths are written
// once every CTA of the cluster has read them. Latency: a launch, the path, its pages, and then a warp's rows one (layer, K or V,
// head) after the other, the next ones' loads behind this one's stores, in at most 8 CTAs a sequence: 24 layers of one
// sequence 6.0 us, three such turns; 8 layers of 64 sequences 6.6.
constexpr int kKeepThreads = 512;
constexpr int kKeepRows = 128;  // path entries looked up at a time
struct KeepParams {
  void* kv[2 * kKeepLayers];  // k, v of each layer
  PagedCache c;               // the page table and lens they share
  const int *counts, *path, *cu, *starts;
  int n_layers, B, rows, Hkv, row_bytes;
  int write_lens;
  DevStatus* status;
};

__global__ void __launch_bounds__(kKeepThreads, 2) paged_keep_kernel(const __grid_constant__ KeepParams p, int size) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ long long from[kKeepRows], to[kKeepRows];  // rows of head 0; from < 0: nothing to move
  const int tid = threadIdx.x, lane = tid & 31;
  const int b = blockIdx.x / size, rank = blockIdx.x % size;
  const SeqRows sr = seq_rows(p.cu, b, p.rows);
  const int count = p.counts[b], start = p.starts ? p.starts[b] : p.c.lens[b];
  bool bad = count < 0 || start < 0 || seq_bad(p.cu, b, p.rows) || (p.path && count > sr.n);
  // with a path, all the sequence's rows are to have slots: attention gave none of them an output otherwise
  const bool full = !bad && (long long)start + (p.path ? sr.n : count) > page_slots(p.c);
  // the places of row j0 + j and of the one that it comes from; false: a page of theirs is none
  auto look_up = [&](int j0, int j, int x) {
    const PagePlace f = page_place(p.c, b, start + x), t = page_place(p.c, b, start + j0 + j);
    from[j] = x != j0 + j ? place_row(p.c, f, p.Hkv, 0) : -1;
    to[j] = place_row(p.c, t, p.Hkv, 0);
    return f.page >= 0 && t.page >= 0;
  };
  if (p.path && !bad && !full)
    for (int j = tid; j < count; j += kKeepThreads) {
      const int x = p.path[sr.lo + j];
      const bool wrong = x < j || x >= sr.n || (j > 0 && p.path[sr.lo + j - 1] >= x);
      bad |= wrong || (j < kKeepRows ? !look_up(0, j, x)
                                     : page_place(p.c, b, start + x).page < 0 || page_place(p.c, b, start + j).page < 0);
    }
  bad = __syncthreads_or(bad);
  cluster_arrive();
  if (tid == 0 && rank == 0 && (bad || full)) record(p.status, bad ? kStatusInvalidArg : kStatusCacheFull);
  const bool on = !bad && !full;
  if (p.path && on) {
    const int units = p.n_layers * 2 * p.Hkv, warps = kKeepThreads / 32;
    const int chunks = p.row_bytes / 16;  // of a row
    const int page_rows = 1 << p.c.page_shift;
    for (int j0 = 0; j0 < count; j0 += kKeepRows) {
      const int n = min(kKeepRows, count - j0);
      if (j0 > 0) {  // the first ones were looked up above
        for (int j = tid; j < n; j += kKeepThreads) look_up(j0, j, p.path[sr.lo + j0 + j]);
        __syncthreads();
      }
      for (int u = rank * warps + (tid >> 5); u < units; u += size * warps) {
        const int head = u % p.Hkv;
        uint8_t* base = static_cast<uint8_t*>(p.kv[u / p.Hkv]) + (size_t)head * page_rows * p.row_bytes;
        const int work = n * chunks;
        for (int w0 = 0; w0 < work; w0 += 4 * 32) {
          uint4 x[4];
          bool has[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int w = w0 + i * 32 + lane, j = w / chunks;
            has[i] = w < work && from[j] >= 0;
            if (has[i]) x[i] = *reinterpret_cast<const uint4*>(base + from[j] * p.row_bytes + (w - j * chunks) * 16);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int w = w0 + i * 32 + lane, j = w / chunks;
            if (has[i]) *reinterpret_cast<uint4*>(base + to[j] * p.row_bytes + (w - j * chunks) * 16) = x[i];
          }
          __syncwarp();
        }
      }
      __syncthreads();
    }
  }
  cluster_wait();
  if (p.write_lens && on && rank == 0 && tid == 0) p.c.lens[b] = start + count;
}

}  // namespace

cudaError_t launch_paged_append(const HeadRows& q, const HeadRows& k, const HeadRows& v, const HeadRows& qo, int rows,
                                const int* cu, const int* depths, int B, int H, int Hkv, int d, const PagedCache& c,
                                const void* q_gain, const void* k_gain, float eps, const float2* table, int dims,
                                int max_pos, bool interleaved, bool bf16, int num_sms, DevStatus* st, cudaStream_t s) {
  if (rows <= 0 || B <= 0) return cudaSuccess;
  AppendParams p{q, k, v, qo, q_gain, k_gain, table, cu, depths, c, rows, B, H, Hkv, d, dims, max_pos, 1, eps,
                 1.f / (float)d, st};
  if (bf16) return launch_append<__nv_bfloat16, 8>(p, interleaved, num_sms, s);  // head_dim 128
  const int lanes = d / 8;
  if (lanes <= 2) return launch_append<float, 2>(p, interleaved, num_sms, s);
  if (lanes <= 4) return launch_append<float, 4>(p, interleaved, num_sms, s);
  if (lanes <= 8) return launch_append<float, 8>(p, interleaved, num_sms, s);
  if (lanes <= 16) return launch_append<float, 16>(p, interleaved, num_sms, s);
  return launch_append<float, 32>(p, interleaved, num_sms, s);
}

cudaError_t launch_paged_keep(void* const* kv, int n_layers, const PagedCache& c, const int* counts, const int* path,
                              const int* cu, const int* starts, int B, int rows, int Hkv, int row_bytes, int num_sms,
                              DevStatus* st, cudaStream_t s) {
  if (B <= 0) return cudaSuccess;
  for (int l0 = 0; l0 < n_layers; l0 += kKeepLayers) {
    KeepParams p{};
    p.n_layers = n_layers - l0 < kKeepLayers ? n_layers - l0 : kKeepLayers;
    for (int i = 0; i < 2 * p.n_layers; ++i) p.kv[i] = kv[2 * l0 + i];
    p.c = c;
    p.counts = counts;
    p.path = path;
    p.cu = cu;
    p.starts = starts;
    p.B = B;
    p.rows = rows;
    p.Hkv = Hkv;
    p.row_bytes = row_bytes;
    p.write_lens = !path || l0 + kKeepLayers >= n_layers;
    p.status = st;
    // enough CTAs for a warp to have a unit or two, while the clusters of all sequences fit the SMs
    int size = 1;
    if (path)
      while (size < 8 && 2ll * size * B <= 2ll * num_sms && size * (kKeepThreads / 32) < p.n_layers * 2 * Hkv) size *= 2;
    const cudaError_t e = launch_clusters(paged_keep_kernel, B * size, kKeepThreads, 0, size, s, p, size);
    if (e != cudaSuccess || !path) return e;
  }
  return cudaSuccess;
}

}  // namespace blk

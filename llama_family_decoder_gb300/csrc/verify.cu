// Verification of drafted tokens against the target's probabilities (speculative sampling: Leviathan et
// al. 2023, Chen et al. 2023; over several candidates of a node as in SpecInfer, Miao et al. 2024). At
// node cur, with p = target[cur] and its children's tokens x in order, P_0 = p and c_0 = 1:
//   x is accepted if u_x c_k q(x) < P_k(x) and P_k(x) > 0, and becomes cur; else
//   with a draft distribution q = draft[cur]: P_{k+1} = max(0, P_k - c_k q), c_{k+1} = sum P_{k+1};
//   without one (the candidate itself, q(x) = 1): P_{k+1} = P_k with P(x) = 0, c_{k+1} = c_k - P_k(x).
// At the end the next token is the first v with sum_{w <= v} P_k(w) > u_next sum P_k.
// By induction P_k = max(0, p - C_k q), C_0 = 0, C_{k+1} = C_k + c_k (where P_k = 0, p <= C_k q, and so
// P_{k+1} = 0), so a rejection needs no array of its own: one pass over p and q gives the next sum.
//
// The answers are whole numbers, so what decides them has to be known far better than fp32: a sum
// over a vocabulary in fp32 would move about one next token in a thousand. p - C q is held as two
// fp32 numbers (its products and sums with their errors: Dekker 1971, Knuth 1969), sums of 16 of them and then
// of a warp's likewise, to about 2^-45; everything from there on, and every test, is fp64.
//
// A cluster of CTAs takes a sequence. All of them walk the tree alike, from the candidates' p and q
// values gathered beforehand in one round of loads; only a pass over the vocabulary is shared: CTA r
// takes the segments of 512 values r, and the cluster's sums meet in distributed shared memory. The
// pass that ends the walk keeps its segments' sums, from which the next token's segment is found, and
// a warp looks through that one. Latency-bound: a launch, three dependent rounds of loads, and
// per pass a row from HBM (or, from the second on, L2) and a cluster barrier.
#include "paged.cuh"

namespace blk {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSeg = 512;        // values of a segment: 16 a lane
constexpr int kCtaSegs = 1024;   // segments whose sums a CTA keeps
constexpr int kMaxCluster = 8;

struct VerifyParams {
  const float *target, *draft;
  long long target_row, draft_row;
  const int *tokens, *parents, *cu;
  const float *u, *u_next;
  int *counts, *path, *next;
  int rows, vocab, B, size;  // size: CTAs of a cluster
  DevStatus* status;
};

// An unevaluated sum of two fp32 numbers.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  Two s = two_sum(a.hi, b.hi);
  s.lo = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo));
  const float hi = __fadd_rn(s.hi, s.lo);  // |hi| >= |lo|: the error is exact
  return {hi, __fsub_rn(s.lo, __fsub_rn(hi, s.hi))};
}

// max(0, p - C q); C in two numbers, C = 0 for the target's own distribution.
__device__ __forceinline__ Two left_of(float p, float q, Two C) {
  const float x = __fmul_rn(C.hi, q), e = __fadd_rn(__fmaf_rn(C.hi, q, -x), __fmul_rn(C.lo, q));
  Two d = two_sum(p, -x);
  d.lo = __fsub_rn(d.lo, e);
  const float hi = __fadd_rn(d.hi, d.lo);
  const float lo = __fsub_rn(d.lo, __fsub_rn(hi, d.hi));
  return hi > 0.f || !(hi == hi) ? Two{hi, lo} : Two{0.f, 0.f};
}

struct Shared {
  double sums[kCtaSegs];            // of this CTA's segments, in the last pass
  double warp_sums[kWarps];
  double total[2];                  // of this CTA, read by its cluster; two passes in turn
  int parent[kMaxNodes], token[kMaxNodes];
  float u[kMaxNodes], p[kMaxNodes], q[kMaxNodes];  // p, q: of the candidate's token at its parent
  int gone[kMaxNodes];              // tokens of rejected candidates (no draft)
  unsigned long long key;           // the warp's find
};

}  // namespace

__device__ __forceinline__ double ld_dsmem_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}

namespace {

// 16 consecutive values of a lane, from element `at` of a row, those past the vocabulary 0.
__device__ __forceinline__ void load16(const float* row, int at, int vocab, bool wide, float (&x)[16]) {
  if (wide && at + 16 <= vocab) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(row + at) + i);
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = at + i < vocab ? __ldg(row + at + i) : 0.f;
  }
}

__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.size, rank = blockIdx.x % p.size;
  const SeqRows sr = seq_rows(p.cu, b, p.rows);
  const bool bad = seq_bad(p.cu, b, p.rows) || sr.n > kMaxNodes;
  if (bad && tid == 0 && rank == 0) record(p.status, kStatusInvalidArg);
  const int n = sr.n > kMaxNodes ? 0 : sr.n;
  if (n == 0) {  // the whole cluster alike
    if (rank == 0) {
      if (tid == 0) p.counts[b] = 0, p.next[b] = -1;
      for (int i = tid; i < sr.n; i += kThreads) p.path[sr.lo + i] = -1;
    }
    return;
  }
  const bool wide_p = (reinterpret_cast<uintptr_t>(p.target) & 15) == 0 && p.target_row % 4 == 0;
  const bool wide_q = p.draft && (reinterpret_cast<uintptr_t>(p.draft) & 15) == 0 && p.draft_row % 4 == 0;
  if (tid < n) {
    const int row = sr.lo + tid;
    int up = p.parents ? p.parents[row] : tid - 1;
    int x = p.tokens[row];
    // a parent behind its child, or a token that is none, takes the node out of the tree
    if (up >= tid || (tid > 0 && up >= 0 && (x < 0 || x >= p.vocab))) {
      record(p.status, kStatusInvalidArg);
      up = -1;
    }
    sh.parent[tid] = up;
    sh.token[tid] = x;
    sh.u[tid] = p.u[row];
    if (tid > 0 && up >= 0) {
      sh.p[tid] = p.target[(sr.lo + up) * p.target_row + x];
      sh.q[tid] = p.draft ? p.draft[(sr.lo + up) * p.draft_row + x] : 1.f;
    }
  }
  __syncthreads();

  int passes = 0;
  const int segs = (p.vocab + kSeg - 1) / kSeg;
  const int per = (segs + p.size - 1) / p.size;  // segments of a CTA, at most kCtaSegs
  const int s0 = min(segs, rank * per), s1 = min(segs, s0 + per);
  // sums over the cluster of max(0, p - C q) at node cur, less the tokens gone; the CTA's segments in sh.sums
  auto value = [&](float x, float y, Two C) { return C.hi > 0.f ? left_of(x, y, C) : Two{x, 0.f}; };
  auto lane_values = [&](int cur, Two C, int n_gone, int seg, float (&x)[16], float (&y)[16]) {
    const int at = seg * kSeg + lane * 16;
    load16(p.target + (sr.lo + cur) * p.target_row, at, p.vocab, wide_p, x);
    if (C.hi > 0.f) load16(p.draft + (sr.lo + cur) * p.draft_row, at, p.vocab, wide_q, y);
    for (int g = 0; g < n_gone; ++g) {
      const int i = sh.gone[g] - at;
      if (sh.gone[g] / kSeg == seg) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (k == i) x[k] = 0.f;
      }
    }
  };
  auto pass = [&](int cur, Two C, int n_gone) {
    __syncthreads();  // sh.gone is written, the last pass's sums are read
    double mine = 0.0;
    for (int seg = s0 + warp; seg < s1; seg += kWarps) {
      float x[16], y[16];
      lane_values(cur, C, n_gone, seg, x, y);
      Two s = value(x[0], y[0], C);
#pragma unroll
      for (int i = 1; i < 16; ++i) s = add(s, value(x[i], y[i], C));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        s = add(s, Two{__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
      const double d = (double)s.hi + (double)s.lo;
      mine += d;
      if (lane == 0) sh.sums[seg - s0] = d;
    }
    if (lane == 0) sh.warp_sums[warp] = mine;
    __syncthreads();
    if (tid == 0) {
      double t = 0.0;
      for (int w = 0; w < kWarps; ++w) t += sh.warp_sums[w];
      sh.total[passes & 1] = t;
    }
    __syncthreads();
    cluster_sync_all();
    double all = 0.0;
    for (int r = 0; r < p.size; ++r) all += ld_dsmem_f64(map_shared_rank(smem_u32(&sh.total[passes & 1]), r));
    ++passes;
    return all;
  };

  // every thread walks alike
  int cur = 0, kept = 1, n_gone = 0;
  double c = 1.0, C = 0.0, sum = 0.0;
  bool summed = false;
  auto two = [](double x) {
    const float hi = (float)x;
    return Two{hi, (float)(x - (double)hi)};
  };
  if (rank == 0 && tid == 0) p.path[sr.lo] = 0;
  for (int i = 1; i < n; ++i) {
    if (sh.parent[i] != cur) continue;
    const float px = sh.p[i], qx = sh.q[i];
    double here;
    if (p.draft) {
      here = fmax(0.0, (double)px - C * (double)qx);
    } else {
      here = px;
      for (int g = 0; g < n_gone; ++g)
        if (sh.gone[g] == sh.token[i]) here = 0.0;
    }
    if ((double)sh.u[i] * c * (double)qx < here && here > 0.0) {
      cur = i;
      if (rank == 0 && tid == 0) p.path[sr.lo + kept] = i;
      ++kept;
      c = 1.0, C = 0.0, n_gone = 0, summed = false;
    } else if (p.draft) {
      C += c;
      c = sum = pass(cur, two(C), 0);
      summed = true;
    } else {
      c -= here;
      __syncthreads();  // the others have read gone
      if (tid == 0) sh.gone[n_gone] = sh.token[i];
      ++n_gone;
      __syncthreads();
    }
  }
  if (!summed) sum = pass(cur, two(C), n_gone);
  if (!(sum > 0.0) && (C > 0.0 || n_gone > 0)) {  // nothing is left: the target's own distribution
    C = 0.0, n_gone = 0;
    sum = pass(cur, two(0.0), 0);
  }
  if (rank == 0) {
    if (tid == 0) p.counts[b] = kept;
    for (int i = kept + tid; i < n; i += kThreads) p.path[sr.lo + i] = -1;
  }
  // The next token: the CTA, then the segment, then the value where the running sum passes u * sum. Where
  // none does (u = 1, or a NaN) it is the last one.
  const double want = (double)p.u_next[b] * sum;
  double before = 0.0;
  int owner = p.size - 1;
  for (int r = 0; r < p.size; ++r) {
    const double t = ld_dsmem_f64(map_shared_rank(smem_u32(&sh.total[(passes - 1) & 1]), r));
    if (before + t > want) {
      owner = r;
      break;
    }
    if (r + 1 < p.size) before += t;
  }
  cluster_sync_all();  // no CTA leaves while its sums are read
  if (rank != owner || warp != 0) return;
  int seg = max(s1 - 1, s0);
  for (int k = s0; k < s1; ++k) {
    const double t = sh.sums[k - s0];
    if (before + t > want) {
      seg = k;
      break;
    }
    if (k + 1 < s1) before += t;
  }
  float x[16], y[16];
  lane_values(cur, two(C), n_gone, seg, x, y);
  double own = 0.0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const Two v = value(x[i], y[i], two(C));
    own += (double)v.hi + (double)v.lo;
  }
  double upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += t;
  }
  const unsigned past = __ballot_sync(0xffffffffu, before + upto > want);
  const int at = past ? __ffs(past) - 1 : 31;
  if (lane == at) {
    double run = before + upto - own;
    int pick = min(p.vocab, seg * kSeg + lane * 16 + 16) - 1;
    bool found = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const Two v = value(x[i], y[i], two(C));
      run += (double)v.hi + (double)v.lo;
      if (!found && run > want) {
        found = true;
        pick = seg * kSeg + lane * 16 + i;
      }
    }
    p.next[b] = min(max(pick, 0), p.vocab - 1);
  }
}

}  // namespace

cudaError_t launch_verify_drafts(const float* target, long long target_row, const float* draft, long long draft_row,
                                 int rows, int vocab, const int* tokens, const int* parents, const int* cu,
                                 const float* u, const float* u_next, int B, int* counts, int* path, int* next,
                                 int num_sms, DevStatus* st, cudaStream_t s) {
  if (B <= 0) return cudaSuccess;
  VerifyParams p{target, draft, target_row, draft_row, tokens, parents, cu, u, u_next, counts, path, next, rows, vocab, B, 1, st};
  const int segs = (vocab + kSeg - 1) / kSeg;
  while (p.size < kMaxCluster && (2ll * p.size * B <= 2ll * num_sms || (segs + p.size - 1) / p.size > kCtaSegs) &&
         p.size * kWarps < segs)
    p.size *= 2;
  return launch_clusters(verify_kernel, B * p.size, kThreads, 0, p.size, s, p);
}

}  // namespace blk

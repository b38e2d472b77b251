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
// fp32 numbers (its products and sums with their errors: Dekker 1971, Knuth 1969), sums of 8 of them and then
// of a warp's likewise, to about 2^-45; everything from there on, and every test, is fp64.
//
// A cluster of CTAs takes a sequence. Warp 0 of each walks the tree, all of them alike, two nodes a lane, from the
// candidates' p and q values gathered beforehand in one round of loads; fp64 is slow here (two lanes
// a cycle and SM), so no other warp does any of it. A pass over the vocabulary is shared: CTA r takes the r-th run
// of segments of 256 values, a warp a segment, and the CTAs' sums meet in distributed shared memory. The pass
// that ends the walk leaves its segments' sums, in which the next token's segment is found; a warp looks
// through that one. Latency-bound: a launch, three dependent rounds of loads, and per pass a row from HBM (from the
// second on, L2) and a cluster barrier. Measured (a graph of calls): one chain of 5 over 32000 tokens with the draft's
// distributions 7.9 us, 64 chains of up to 6 11.2, 16 trees of up to 64 over 131072 tokens without them 12.2. (One CTA an
// SM 9.3, 17.4, 14.9; sums written to all CTAs instead of read 10.0, 12.3, 13.7; segments of 128 values 9.7, 12.0, 11.9.)
#include "paged.cuh"

namespace blk {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 8;          // values of a segment that a lane has
constexpr int kSeg = 32 * kPer;
constexpr int kCtaSegs = 2048;   // segments whose sums a CTA keeps
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

// What warp 0 asks of all: a pass over the row of node cur, with C and without the gone tokens, or nothing more.
struct Order {
  int cur, n_gone, done;
  Two C;
};
struct Shared {
  Two sums[kCtaSegs];     // of this CTA's segments, in the last pass
  double total[2];        // of this CTA, read by its cluster; two passes in turn
  int gone[kMaxNodes];    // tokens of rejected candidates (no draft)
  Order order;
};

__device__ __forceinline__ double ld_dsmem_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ double value_of(Two x) { return (double)x.hi + (double)x.lo; }
__device__ __forceinline__ Two two_of(double x) {
  const float hi = (float)x;
  return {hi, (float)(x - (double)hi)};
}
__device__ __forceinline__ double scan(double x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// kPer consecutive values of a row, from element `at`, those past the vocabulary 0.
__device__ __forceinline__ void load_values(const float* row, int at, int vocab, bool wide, float (&x)[kPer]) {
  if (wide && at + kPer <= vocab) {
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(row + at) + i);
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = at + i < vocab ? __ldg(row + at + i) : 0.f;
  }
}

// A lane's values of a segment: what is left of the target's distribution at node cur.
struct Row {
  const float *p, *q;
  bool wide_p, wide_q;
};
__device__ __forceinline__ void left_values(const Row& row, const Order& o, const int* gone, int vocab, int seg, int lane,
                                            Two (&v)[kPer]) {
  const int at = seg * kSeg + lane * kPer;
  float x[kPer];
  load_values(row.p, at, vocab, row.wide_p, x);
  if (o.C.hi > 0.f) {
    float y[kPer];
    load_values(row.q, at, vocab, row.wide_q, y);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = left_of(x[i], y[i], o.C);
    return;
  }
  if (o.n_gone > 0) {
#pragma unroll 1
    for (int g0 = 0; g0 < o.n_gone; g0 += 32) {
      const int x_at = g0 + lane < o.n_gone ? gone[g0 + lane] - seg * kSeg : -1;
      for (unsigned in = __ballot_sync(0xffffffffu, x_at >= 0 && x_at < kSeg); in; in &= in - 1) {
        const int i = __shfl_sync(0xffffffffu, x_at, __ffs(in) - 1) - lane * kPer;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (k == i) x[k] = 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = Two{x[i], 0.f};
}
__device__ __forceinline__ Two sum_of(const Two (&v)[kPer]) {
  Two s[kPer / 2];
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) s[i] = add(v[2 * i], v[2 * i + 1]);
#pragma unroll
  for (int n = kPer / 4; n > 0; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) s[i] = add(s[i], s[i + n]);
  return s[0];
}

__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const __grid_constant__ VerifyParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.size, rank = blockIdx.x % p.size;
  const float u_next = p.u_next[b];
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
  const int segs = (p.vocab + kSeg - 1) / kSeg;
  const int per = (segs + p.size - 1) / p.size;  // segments of a CTA, at most kCtaSegs
  const int s0 = min(segs, rank * per), s1 = min(segs, s0 + per);
  const bool wide_p = (reinterpret_cast<uintptr_t>(p.target) & 15) == 0 && p.target_row % 4 == 0;
  const bool wide_q = p.draft && (reinterpret_cast<uintptr_t>(p.draft) & 15) == 0 && p.draft_row % 4 == 0;
  auto row_of = [&](int cur) {
    return Row{p.target + (sr.lo + cur) * p.target_row, p.draft ? p.draft + (sr.lo + cur) * p.draft_row : nullptr, wide_p, wide_q};
  };
  // A pass: the segments' sums to sh.sums, all warps.
  auto pass = [&](const Order& o) {
    const Row row = row_of(o.cur);
    for (int seg = s0 + warp; seg < s1; seg += kWarps) {
      Two v[kPer];
      left_values(row, o, sh.gone, p.vocab, seg, lane, v);
      Two s = sum_of(v);
#pragma unroll
      for (int k = 16; k > 0; k >>= 1)
        s = add(s, Two{__shfl_xor_sync(0xffffffffu, s.hi, k), __shfl_xor_sync(0xffffffffu, s.lo, k)});
      if (lane == 0) sh.sums[seg - s0] = s;
    }
  };
  const int each = (s1 - s0 + 31) / 32;  // of the CTA's segments, a lane of warp 0 has `each`
  int passes = 0;
  double upto = 0.0, own = 0.0;          // sums up to and of the lane's segments
  double cta_upto = 0.0, cta_own = 0.0;  // ... of CTA `lane`
  // Their sum over the cluster, in warp 0 (which has the sums above too).
  auto total = [&] {
    __syncthreads();
    if (warp == 0) {
      own = 0.0;
      for (int k = lane * each; k < min((lane + 1) * each, s1 - s0); ++k) own += value_of(sh.sums[k]);
      upto = scan(own, lane);
      if (lane == 31) sh.total[passes & 1] = upto;
    }
    __syncwarp();
    cluster_sync_all();
    double all = 0.0;
    if (warp == 0) {
      cta_own = lane < p.size ? ld_dsmem_f64(map_shared_rank(smem_u32(&sh.total[passes & 1]), lane)) : 0.0;
      cta_upto = scan(cta_own, lane);
      all = __shfl_sync(0xffffffffu, cta_upto, 31);
    }
    ++passes;
    return all;
  };

  if (warp != 0) {
    for (;;) {
      __syncthreads();  // an order
      const Order o = sh.order;
      if (o.done) break;
      pass(o);
      total();
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    return;
  }
  // ---------------- warp 0
  int parent[2], token[2];
  float u[2], px[2], qx[2];  // px, qx: of the candidate's token at its parent
  bool gone[2] = {false, false};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    parent[h] = -1, token[h] = -1, u[h] = px[h] = qx[h] = 0.f;
    if (i < n) {
      parent[h] = p.parents ? p.parents[sr.lo + i] : i - 1;
      token[h] = p.tokens[sr.lo + i];
      u[h] = p.u[sr.lo + i];
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    // a parent behind its child, or a token that is none, takes the node out of the tree
    if (i < n && (parent[h] >= i || (i > 0 && parent[h] >= 0 && (token[h] < 0 || token[h] >= p.vocab)))) {
      record(p.status, kStatusInvalidArg);
      parent[h] = -1;
    }
    if (i > 0 && parent[h] >= 0) {
      px[h] = p.target[(sr.lo + parent[h]) * p.target_row + token[h]];
      qx[h] = p.draft ? p.draft[(sr.lo + parent[h]) * p.draft_row + token[h]] : 1.f;
    }
  }
  __syncwarp();
  auto pick = [&](auto (&x)[2], int i) { return __shfl_sync(0xffffffffu, i < 32 ? x[0] : x[1], i & 31); };
  Order o{0, 0, 0, {0.f, 0.f}};
  double c = 1.0, C = 0.0, sum = 0.0;
  bool summed = false;
  auto passed = [&] {  // an order and its sum
    if (lane == 0) sh.order = o;
    __syncthreads();
    pass(o);
    return total();
  };
  int kept = 1;
  if (rank == 0 && lane == 0) p.path[sr.lo] = 0;
  for (;;) {
    // the current node's children in order
    unsigned long long left = __ballot_sync(0xffffffffu, lane > 0 && parent[0] == o.cur) |
                              (unsigned long long)__ballot_sync(0xffffffffu, parent[1] == o.cur) << 32;
    int taken = -1;
    for (; left && taken < 0; left &= left - 1) {
      const int i = __ffsll((long long)left) - 1;
      const int x = pick(token, i);
      const double xp = pick(px, i), xq = pick(qx, i), xu = pick(u, i);
      double here = xp;
      if (p.draft) {
        here = fmax(0.0, xp - C * xq);
      } else if (__any_sync(0xffffffffu, (gone[0] && token[0] == x) || (gone[1] && token[1] == x))) {
        here = 0.0;
      }
      if (here > 0.0 && xu * c * xq < here) {
        taken = i;
      } else if (p.draft) {
        C += c;
        o.C = two_of(C);
        c = sum = passed();
        summed = true;
      } else {
        c -= here;
        gone[0] |= lane == i;
        gone[1] |= lane + 32 == i;
        if (lane == 0) sh.gone[o.n_gone] = x;
        ++o.n_gone;
      }
    }
    if (taken < 0) break;
    if (rank == 0 && lane == 0) p.path[sr.lo + kept] = taken;
    ++kept;
    o = Order{taken, 0, 0, {0.f, 0.f}};
    gone[0] = gone[1] = false;
    c = 1.0, C = 0.0;
    summed = false;
  }
  if (!summed) sum = passed();
  if (!(sum > 0.0) && (C > 0.0 || o.n_gone > 0)) {  // nothing is left: the target's own distribution
    o.C = {0.f, 0.f};
    o.n_gone = 0;
    sum = passed();
  }
  if (lane == 0) sh.order.done = 1;
  __syncthreads();
  cluster_arrive();  // the other CTAs' sums have been read
  if (rank == 0) {
    if (lane == 0) p.counts[b] = kept;
    for (int i = kept + lane; i < n; i += 32) p.path[sr.lo + i] = -1;
  }
  // The next token: the CTA, then the segment, then the value where the running sum passes u * sum. Where
  // none does (a NaN) it is the last one.
  const double want = (double)u_next * sum;
  const unsigned ctas = __ballot_sync(0xffffffffu, lane < p.size && cta_upto > want);
  const int owner = ctas ? __ffs(ctas) - 1 : p.size - 1;
  if (rank == owner) {
    const double before = __shfl_sync(0xffffffffu, cta_upto - cta_own, owner);
    const unsigned lanes = __ballot_sync(0xffffffffu, before + upto > want);
    int seg = max(s1 - 1, s0);
    double run = before + __shfl_sync(0xffffffffu, upto, 31);
    if (lanes) {
      const int l = __ffs(lanes) - 1;
      run = before + __shfl_sync(0xffffffffu, upto - own, l);
      seg = s0 + l * each;
      for (const int last = min(s0 + (l + 1) * each, s1) - 1; seg < last; ++seg) {
        const double next = run + value_of(sh.sums[seg - s0]);
        if (next > want) break;
        run = next;
      }
    }
    Two v[kPer];
    left_values(row_of(o.cur), o, sh.gone, p.vocab, seg, lane, v);
    const double mine = value_of(sum_of(v)), here = scan(mine, lane);
    const unsigned past = __ballot_sync(0xffffffffu, run + here > want);
    const int at = past ? __ffs(past) - 1 : 31;
    run += __shfl_sync(0xffffffffu, here - mine, at);
    Two one{0.f, 0.f};  // lane i < kPer: value i of that lane
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const Two x{__shfl_sync(0xffffffffu, v[i].hi, at), __shfl_sync(0xffffffffu, v[i].lo, at)};
      if (lane == i) one = x;
    }
    const double here1 = scan(value_of(one), lane);
    const unsigned found = __ballot_sync(0xffffffffu, lane < kPer && run + here1 > want);
    const int first = seg * kSeg + at * kPer;
    if (lane == 0) p.next[b] = min(max(found ? first + __ffs(found) - 1 : min(first + kPer - 1, p.vocab - 1), 0), p.vocab - 1);
  }
  __syncwarp();
  cluster_wait();
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

// Attention of a sequence's new rows (one token, a chain or a tree of drafted ones) over the paged
// cache on the 5th-generation tensor core (tcgen05 + TMEM), grouped-query ("arcee", "Grouped-query
// attention, 128-wide heads"), head_dim 128:
//   o = softmax(q k^T / sqrt(128)) v over the sequence's slots and the row's ancestors and itself.
//
// Bound by reading the cache once. All heads of a KV head and all new rows of a sequence share its
// keys, so they fold into the rows of one matrix tile: row r of a slot is head r % G of row r / G (G = H / Hkv),
// a slot has 128 of them. A CTA has two slots. Where a sequence has more than 96 such rows on average they hold
// the two halves of its rows and share each tile of 64 keys (units of one slot would read the cache once per 128
// rows: trees of 64 nodes 72 us against 56); else they take the units in turn, so that one's outputs and first tiles run
// beside the other's (256 sequences of up to 300 slots, a token each, 62.7 -> 55.7 us; of up to 20 48 -> 37; 64 of up to
// 8192 199 -> 195). The tensor core's M = 128 costs the same for one row as for 128: 620 cycles a tile and slot, a
// tile (32 KB) takes 1390 to arrive at an SM's share of 6.8 TB/s.
//
// Large batches: work is a line of key tiles, units (sequence, KV head, rows of the slots) one after the other, each as
// many tiles as it has keys. The CTAs, one per SM, take equal stretches of it, whatever the sequences'
// lengths; a unit that lies in several stretches leaves partial results (unnormalised outputs, the
// running maximum and sum), which a second kernel joins in the order of the keys, so results do not
// depend on timing. Lengths are on the device: every CTA adds up the line by itself, and the CTA that goes on with
// another's unit writes down what is to be joined there. (Whole units per CTA instead: trees 73 us.)
// Small batches (plan_of): a cluster of CTAs takes a unit, equal shares of its keys each, joined in the
// cluster's shared memory: no second kernel, one token over 4000 slots 12.2 -> 9.0 us, or where tiles are few too
// one CTA (16 sequences of up to 300 12.8 -> 7.9). With few rows a CTA's two
// slots hold the same rows and take its tiles in turn there.
//
// Warps 0 and 3 load K and V: their lanes look up the pages of the next 32 boxes (a box: the rows of a page in a tile)
// and each issues a TMA copy of a box's half, 128-byte swizzled, into a ring of 16 KB stages. (One warp for
// both: pages of 16 19.7 us against 17.2.) Warps 1 and 2, one a slot, issue the products as they
// become possible: S = Q K^T up to two tiles ahead into TMEM buffers, O += P V with P from TMEM, and
// load the next unit's queries. All its lanes go through that loop and an elected one issues, so that the
// descriptors stay in uniform registers: from one lane's own branch each MMA cost some 100 cycles more (64 ragged
// tokens 238 us against 201). Four warps a slot hold a row a thread: scores
// from TMEM, the running softmax in the log2 domain with a reference that moves only when a
// score passes it by 2^8 (exact: softmax does not depend on it), P as bf16 over the scores (the product takes its operands
// so; the output's error is 0.0022 of its size then, 0.0017 by its own rounding to bf16 alone), and the outputs.
// Every wait is bounded; on expiry the CTA records a timeout, drains its own copies and MMAs, frees its
// TMEM and returns.
//
// Measured (8 KV heads of 4 query heads, a graph of calls on cold caches): 64 sequences of up to 8192 slots, a token
// each, 195 us = 6.6 TB/s, the cache's bandwidth; 16 trees of up to 64 nodes over up to 4096 slots 56 us: two full slots
// take 1900 cycles a tile (scores 768, bound by shared memory's 128 bytes a cycle, products 512, and exponentials
// that run while the pipe waits), one 1240; 32 chains of 5 over windows of 2048 in pages of 16 (2 KV
// heads) 17 us and one token over 4000 slots 9 us: a launch, the list, a page, a tile, one after the other.
#include <algorithm>
#include <cstring>

#include "paged.cuh"

namespace blk {

namespace {

constexpr int kD = 128;
constexpr int kBQ = 128;               // rows of a slot (MMA M)
constexpr int kBK = 64;                // keys of a tile
constexpr int kQSub = kBQ * 128;       // one 64-channel half of a slot's queries (bytes)
constexpr int kQBytes = 2 * kQSub;
constexpr int kKVSub = kBK * 128;      // one 64-channel half of a K or V tile
constexpr int kStageBytes = 4 * kKVSub;
constexpr int kMaxCluster = 16;
constexpr int kClusterTiles = 64;      // a CTA's share of tiles up to which clusters of ragged sequences pay (plan_of)
constexpr int kWholeTiles = 28;        // a unit's tiles up to which it is one CTA's (plan_of)
constexpr float kRescaleLog2 = 8.0f;
constexpr float kScaleLog2 = 1.4426950408889634f * 0.08838834764831845f;  // log2(e) / sqrt(128)
constexpr int kNoBox = -2;             // a box that no row needs; entries below -1 are read as -1
constexpr unsigned long long kDrainNs = 2000000000ULL;
constexpr unsigned long long kShortNs = 100000;  // limits below are for tests of what happens then
struct Join;  // see below
struct AttnParams {
  CUtensorMap tk, tv;  // [n_pages * Hkv * page_size, 128] bf16, boxes of 64 channels x `box` rows
  CUtensorMap tq_map;  // the query rows: boxes of 64 channels x G heads x tq rows
  HeadRows o;
  PagedCache c;
  const int *cu, *parents;
  int rows, B, H, Hkv, G, window;
  int q_bytes;    // of a slot's queries
  int q_shift;    // units in turn: where the second slot's begin (lanes)
  int tq;         // rows of a sequence in a slot: 128 / G
  int slots;      // slots of a CTA
  int box_shift;  // log2 of a box's rows: those of a page, at most 64
  int grid;
  int cluster;    // CTAs that share a unit, 0: the line
  int single;     // no sequence has more than one unit of a KV head
  int unit_cost;  // what a unit counts for on the line besides its tiles, before them
  float2* ml;     // partial results [2 grid][slots][128]: (reference, sum)
  float* acc;     // ... [2 grid][slots][32][128][4]: four channels of each row side by side
  Join* joins;    // [grid]
  int o_wide;     // the outputs' rows start on 32-byte boundaries
  DevStatus* status;
  unsigned long long wait_ns;
};

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// A tile into L2 alone.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* m, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}
// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// 32 bytes in one store (a 32-byte boundary)
__device__ __forceinline__ void st_global_32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem desc], bf16
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ------------------------------------------------------------------ the line of tiles

// A sequence that has something to do: rows [row0, row0 + n) over `len` slots.
struct Seq {
  int row0, n, len;
};
__device__ __forceinline__ Seq seq_of(const AttnParams& p, int b) {
  const SeqRows r = seq_rows(p.cu, b, p.rows);
  const int len = p.c.lens[b];
  const bool fits = len >= 0 && (long long)len + r.n <= page_slots(p.c);
  return {r.lo, fits ? (p.parents ? min(r.n, kMaxNodes) : r.n) : 0, len};
}
__device__ __forceinline__ int units_of(const AttnParams& p, const Seq& s) {
  return (s.n + p.tq * p.slots - 1) / (p.tq * p.slots);
}
// Keys [first, end) that some row of unit t sees, or rather that may be.
struct Keys {
  int first, end;
  __device__ __forceinline__ int tile0() const { return first / kBK; }
  __device__ __forceinline__ int tiles() const { return (end + kBK - 1) / kBK - first / kBK; }
};
__device__ __forceinline__ Keys keys_of(const AttnParams& p, const Seq& s, int t) {
  const int i0 = p.parents ? 0 : t * p.tq * p.slots;
  const int i1 = p.parents ? s.n : min(s.n, i0 + p.tq * p.slots);
  return {p.window > 0 ? max(0, s.len + i0 - p.window + 1) : 0, s.len + i1};
}
__device__ __forceinline__ int head_cost(const AttnParams& p, const Seq& s) {  // of all units of a KV head
  if (s.n == 0) return 0;
  int n = keys_of(p, s, 0).tiles() + p.unit_cost;
  for (int t = 1; t * p.tq * p.slots < s.n; ++t) n += keys_of(p, s, t).tiles() + p.unit_cost;
  return n;
}

// A CTA's stretch [lo, hi) of the line, and the sequence it begins in, whose own tiles begin at `base`. per: the
// stretches' length.
struct Stretch {
  int lo, hi, base, b, per;
};
__device__ __forceinline__ int scan(int n, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, n, o);
    if (lane >= o) n += x;
  }
  return n;
}
// Numbers of the sequences, 32 * kHeld of them looked up once, the others again where they are needed; by one warp.
template <class F>
struct PerSeq {
  static constexpr int kHeld = 4;
  F of;
  int B, lane, held[kHeld];
  __device__ __forceinline__ PerSeq(F f, int B_, int lane_) : of(f), B(B_), lane(lane_) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) held[i] = 32 * i < B ? number(32 * i + lane) : 0;
  }
  __device__ __forceinline__ int number(int b) const {
    const int n = of(min(b, B - 1));  // without a branch: the loads of all are under way together
    return b < B ? n : 0;
  }
  template <int = 0>
  __device__ __forceinline__ int total() const {
    unsigned n = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) n += (unsigned)held[i];
    for (int b = lane + 32 * kHeld; b < B; b += 32) n += (unsigned)number(b);
    return (int)__reduce_add_sync(0xffffffffu, n);
  }
  // The sequence in whose share place x of the sum lies, and the sum before it; false: x is not below the sum.
  __device__ __forceinline__ bool find(int x, int& b, int& before) const {
    before = 0;
    bool found = false;
    auto look = [&](int b0, int n) {
      const int upto = scan(n, lane);
      const unsigned past = __ballot_sync(0xffffffffu, before + upto > x);
      const int at = past ? __ffs(past) - 1 : 31;
      b = b0 + at;
      before += __shfl_sync(0xffffffffu, past ? upto - n : upto, at);
      found = past != 0;
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (!found && 32 * i < B) look(32 * i, held[i]);
    for (int b0 = 32 * kHeld; !found && b0 < B; b0 += 32) look(b0, number(b0 + lane));
    return found;
  }
};
// By one warp. Stretch number `c`; an empty one (lo >= hi) if the line ends before. The line is shorter
// than 2^31 (see plan_of); that of a list that falls need not be, and is not walked.
__device__ __forceinline__ Stretch stretch_of(const AttnParams& p, int c, int lane) {
  const PerSeq costs([&](int b) { return p.Hkv * head_cost(p, seq_of(p, b)); }, p.B, lane);
  const int total = costs.total();
  Stretch s{0, 0, 0, 0, max((int)(((unsigned)total + p.grid - 1) / p.grid), 1)};
  s.lo = (int)min((long long)total, (long long)c * s.per);
  s.hi = (int)min((long long)total, (long long)s.lo + s.per);
  if (s.lo < s.hi && !costs.find(s.lo, s.b, s.base)) s.hi = s.lo;  // lengths that change meanwhile
  return s;
}

// Walks the units of a stretch: unit t of KV head kvh of sequence b, its tiles [j0, j1) of `tiles` (none where
// the stretch ends in a unit's own cost).
struct Walk {
  Seq seq;
  Keys keys;
  int b, kvh, t, tiles, j0, j1;
  int at;  // where in the unit, costs counted, the stretch is
  int left;
  Walk() = default;
  __device__ __forceinline__ void unit(const AttnParams& p) {
    keys = keys_of(p, seq, t);
    tiles = keys.tiles();
  }
  __device__ __forceinline__ void part(const AttnParams& p) {
    j0 = max(0, at - p.unit_cost);
    j1 = min(tiles, max(0, at + left - p.unit_cost));
  }
  __device__ __forceinline__ Walk(const AttnParams& p, const Stretch& s) {
    left = s.hi - s.lo;
    j0 = j1 = tiles = kvh = t = at = 0;
    b = s.b;
    if (left <= 0) return;
    seq = seq_of(p, b);
    const int from = s.lo - s.base;
    const int per_head = head_cost(p, seq);
    if (per_head <= 0) {  // lengths that change meanwhile: no walk leaves the lists
      left = 0;
      return;
    }
    kvh = from / per_head;
    if (kvh >= p.Hkv) {
      left = 0;
      return;
    }
    at = from - kvh * per_head;
    unit(p);
    while (at >= tiles + p.unit_cost) {  // at < per_head: it ends within the units
      at -= tiles + p.unit_cost;
      ++t;
      unit(p);
    }
    part(p);
  }
  // The share of CTA `rank` of a cluster of `size` that takes unit number u, or nothing (seq.n = 0). By one warp.
  __device__ __forceinline__ Walk(const AttnParams& p, int u, int rank, int size, int lane) {
    left = j0 = j1 = tiles = at = b = kvh = t = 0;
    seq = Seq{0, 0, 0};
    int before = 0;
    if (p.single) {
      b = u / p.Hkv;
      before = b * p.Hkv;
    } else {
      const PerSeq units([&](int x) { return p.Hkv * units_of(p, seq_of(p, x)); }, p.B, lane);
      if (!units.find(u, b, before)) return;
    }
    seq = seq_of(p, b);
    const int n = units_of(p, seq);
    if (n == 0) return;  // a sequence without rows
    kvh = (u - before) / n;
    t = u - before - kvh * n;
    unit(p);
    at = (int)((long long)tiles * rank / size);
    left = (int)((long long)tiles * (rank + 1) / size) - at;
    part(p);
  }
  __device__ __forceinline__ bool on() const { return left > 0; }
  __device__ __forceinline__ void next(const AttnParams& p) {
    left -= tiles + p.unit_cost - at;
    if (left <= 0) return;
    if (++t >= units_of(p, seq)) {
      t = 0;
      if (++kvh >= p.Hkv) {
        kvh = 0;
        do {
          if (++b >= p.B) {
            left = 0;
            return;
          }
          seq = seq_of(p, b);
        } while (seq.n == 0);
      }
    }
    at = 0;
    unit(p);
    part(p);
  }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == tiles; }
  // whether a slot has rows to work on, and its first one
  __device__ __forceinline__ bool has(const AttnParams& p, int g) const { return j1 > j0 && node0(p, g) < seq.n; }
  __device__ __forceinline__ int node0(const AttnParams& p, int g) const { return (t * p.slots + g) * p.tq; }
};

// What the second kernel joins at stretch c, written by its CTA: the unit that the stretch goes on with, if stretch
// c - 1 has its first tile; its parts are those of stretches c - 1 (number `first`) to `last`. last < 0: nothing.
struct Join {
  Seq seq;
  int kvh, t, first, last;
};
__device__ __forceinline__ Join join_of(const AttnParams& p, const Stretch& s, const Walk& w, int c) {
  Join j{w.seq, w.kvh, w.t, 0, -1};
  const int tile0 = s.lo - w.at + p.unit_cost;  // the unit's first tile on the line
  if (!w.on() || w.j0 == 0 || tile0 / s.per != c - 1) return j;  // no unit goes over, or an earlier stretch has it
  j.last = min((tile0 + w.tiles - 1) / s.per, p.grid - 1);
  j.first = s.lo - w.at <= (c - 1) * s.per ? 2 * (c - 1) : 2 * (c - 1) + 1;  // was it that stretch's first unit?
  return j;
}

__device__ __forceinline__ unsigned long long bits_from(int lo) {  // bits lo ..
  return lo <= 0 ? ~0ull : lo >= 64 ? 0ull : ~0ull << lo;
}
__device__ __forceinline__ unsigned long long bits_below(int hi) { return ~bits_from(hi); }

// Four channels of a row, joined from parts (reference and sum, unnormalised outputs) one group after
// the other.
struct Joined {
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  template <int N>
  __device__ __forceinline__ void take(const float2 (&ml)[N], const float4 (&a)[N]) {
    float top = m;
#pragma unroll
    for (int j = 0; j < N; ++j) top = fmaxf(top, ml[j].x);
    const float old = m == -INFINITY ? 0.f : ex2_approx(m - top);
    m = top;
    l *= old;
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] *= old;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (ml[j].x == -INFINITY && !(ml[j].y != ml[j].y)) continue;  // a part that saw no key, or is none
      const float wt = ex2_approx(ml[j].x - m);
      l = fmaf(wt, ml[j].y, l);
      o[0] = fmaf(wt, a[j].x, o[0]);
      o[1] = fmaf(wt, a[j].y, o[1]);
      o[2] = fmaf(wt, a[j].z, o[2]);
      o[3] = fmaf(wt, a[j].w, o[3]);
    }
  }
  __device__ __forceinline__ void store(const AttnParams& p, int row, int head, int ch) const {
    const float inv = 1.f / l;
    __nv_bfloat16* const to = static_cast<__nv_bfloat16*>(p.o.ptr) + row * p.o.row + head * p.o.head + 4 * ch;
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  }
};

__device__ __forceinline__ float2 ld_dsmem_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// ------------------------------------------------------------------ the kernel

// TURNS: units have the rows of one slot; the CTA's two take the units in turn, or with clusters the tiles of its one unit.
template <bool CL, bool TURNS>
struct Cfg {
  static constexpr int NS = 2;
  static constexpr int kQueries = (CL && TURNS ? 1 : NS) * kQBytes;
  static constexpr int kStages = kQueries == kQBytes ? 6 : 5;
  static constexpr int kThreads = 128 + 128 * NS;  // at most 12 warps: one more would leave 128 registers
  static constexpr int kBufs = 2;                  // a slot's buffers of scores
  static constexpr int kSlotCols = 64 * kBufs + kD;  // of tensor memory: scores (and P over them), outputs
  static constexpr int kTmemCols = 512;
  static_assert(NS * kSlotCols <= kTmemCols, "tensor memory");
  static constexpr int kBars = 4 * kStages + (6 + 3 * kBufs) * NS;
  static constexpr int kSmem = 1024 + kQueries + kStages * kStageBytes + kBars * 8 + 8 + sizeof(Walk);
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(!(CL && TURNS) || kStages % 2 == 0, "tiles in turn: a stage is always the same slot's, whose waits tell its phases apart");
  static_assert(NS * kBQ * kD * 4 <= kStages * kStageBytes, "clusters: the slots' outputs take the ring's place");
};

template <bool CL, bool TURNS>
__global__ void __launch_bounds__(Cfg<CL, TURNS>::kThreads, 1) attn_paged_kernel(const __grid_constant__ AttnParams p) {
  typedef Cfg<CL, TURNS> C;
  constexpr int NS = C::NS;
  constexpr bool SPLIT = CL && TURNS;  // tiles in turn
  constexpr bool ALT = !CL && TURNS;   // units in turn
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const sQ = smem;
  uint8_t* const ring = smem + C::kQueries;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ring + C::kStages * kStageBytes);
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  Walk* const begin = reinterpret_cast<Walk*>(tmem_holder + 2);  // the CTA's first unit
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto full = [&](int kv, int s) { return bar(kv * C::kStages + s); };  // K (0) or V (1) of a stage
  auto empty = [&](int kv, int s) { return bar((2 + kv) * C::kStages + s); };
  auto mine = [&](int g, int i) { return bar(4 * C::kStages + (6 + 3 * C::kBufs) * g + i); };
  auto q_full = [&](int g) { return mine(g, 0); };
  auto q_free = [&](int g) { return mine(g, 1); };
  auto o_done = [&](int g) { return mine(g, 2); };
  auto o_free = [&](int g) { return mine(g, 3); };
  auto drain = [&](int g) { return mine(g, 4); };
  auto turn_over = [&](int g) { return mine(g, 5 + 3 * C::kBufs); };
  // of the slot's tile number A, in buffer A % kBufs
  auto s_full = [&](int g, int A) { return mine(g, 5 + A % C::kBufs); };
  auto p_ready = [&](int g, int A) { return mine(g, 5 + C::kBufs + A % C::kBufs); };
  auto pv_done = [&](int g, int A) { return mine(g, 5 + 2 * C::kBufs + A % C::kBufs); };
  auto phase = [](int A) { return (uint32_t)(A / C::kBufs) & 1; };
  // the warp's number as the compiler can see that it is the same in all lanes: what the roles compute from it
  // then goes through uniform registers, where the MMA and TMA instructions want their operands
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const unsigned long long budget = p.wait_ns;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(0, s), 1);
      mbar_init(full(1, s), 1);
      mbar_init(empty(0, s), TURNS ? 1 : NS);
      mbar_init(empty(1, s), TURNS ? 1 : NS);
    }
    for (int g = 0; g < NS; ++g) {
      mbar_init(q_full(g), 1);
      mbar_init(q_free(g), 1);
      for (int i = 0; i < C::kBufs; ++i) {
        mbar_init(s_full(g, i), 1);
        mbar_init(p_ready(g, i), 128);
        mbar_init(pv_done(g, i), 1);
      }
      mbar_init(o_done(g), 1);
      mbar_init(o_free(g), 128);
      mbar_init(drain(g), 1);
      mbar_init(turn_over(g), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tk);
    tma_prefetch_desc(&p.tv);
    tma_prefetch_desc(&p.tq_map);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), C::kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();  // queries, cache, lengths and lists come from earlier kernels
  pdl_launch_dependents();
  if (warp == 0) {
    if constexpr (CL) {
      const Walk w(p, blockIdx.x / p.cluster, cluster_ctarank(), p.cluster, lane);
      if (lane == 0) *begin = w;
    } else {
      const Stretch s = stretch_of(p, blockIdx.x, lane);
      const Walk w(p, s);
      if (lane == 0) {
        *begin = w;
        p.joins[blockIdx.x] = join_of(p, s, w, blockIdx.x);
      }
    }
  }
  if (warp == 2 && blockIdx.x == 0) {  // what the lists say that they should not
    bool bad = false, over = false;
    for (int b = lane; b < p.B; b += 32) {
      const SeqRows r = seq_rows(p.cu, b, p.rows);
      const int len = p.c.lens[b];
      bad |= seq_bad(p.cu, b, p.rows) || len < 0 || (p.parents && r.n > kMaxNodes);
      over |= len >= 0 && (long long)len + r.n > page_slots(p.c);
    }
    if (bad) record(p.status, kStatusInvalidArg);
    if (over) record(p.status, kStatusCacheFull);
    __syncwarp();
  }
  // Sequences of a list that falls overlap: neither the line nor the units are as long then as the host has them.
  bool falls = false;
  if (warp == 2 && p.cu)
    for (int b = lane; b < p.B; b += 32) falls |= p.cu[b + 1] < p.cu[b];
  __syncwarp();
  tc_fence_before();
  if (__syncthreads_or(falls)) {  // no row gets an output
    if (threadIdx.x == 0) {
      begin->left = begin->seq.n = 0;
      if (!CL) p.joins[blockIdx.x].last = -1;
    }
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  // What is in flight, for the drain after an abort: the stages issued (with the parity of their last
  // phase), the loads of queries so far and whether any MMA was issued.
  uint32_t issued = 0, parity = 0;
  int q_loads = 0;
  bool mma_issued = false;
  // clusters: a row's reference and sum over the CTA's share (of none, at first)
  float2 share = make_float2(-INFINITY, 0.f);
  bool share_live = false;

  if (warp == 0 || warp == 3) {
    // ---------------- the cache's tiles, all lanes: K by warp 0, V by warp 3 (a warp issues about a copy
    // every 60 cycles: with pages of 16, 8 copies a tile and warp, one warp for both took 1450 cycles a tile)
    const int kv = warp == 0 ? 0 : 1;
    const CUtensorMap* const map = kv ? &p.tv : &p.tk;
    const uint32_t to = smem_u32(ring) + 2 * kv * kKVSub;
    const uint64_t once = l2_policy_evict_first();
    const int page_shift = p.c.page_shift, boxes = kBK >> p.box_shift, box = lane >> 1, half = lane & 1;
    int J = 0;
    bool failed = false;
    for (Walk w = *begin; w.on() && !failed; w.next(p)) {
      const int* const pages = p.c.pages + (size_t)w.b * p.c.max_pages;
      const int box0 = (w.keys.tile0() + w.j0) * boxes;  // the first box of the part
      const int n_boxes = (w.j1 - w.j0) * boxes;
      auto look_up = [&](int i) {  // the page of the part's box i + lane
        const int slot = (box0 + i + lane) << p.box_shift;
        const bool in = i + lane < n_boxes && slot < w.keys.end && slot + (1 << p.box_shift) > w.keys.first;
        return in ? max(pages[slot >> page_shift], -1) : kNoBox;
      };
      int page = look_up(0), ahead = look_up(32);
      for (int i = 0; i < n_boxes; i += boxes, ++J) {
        if (i > 0 && (i & 31) == 0) {
          page = ahead;
          ahead = look_up(i + 32);
        }
        const int s = J % C::kStages;
        const uint32_t ph = (J / C::kStages) & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(empty(kv, s), ph ^ 1, budget, abort_flag))) {
          failed = true;
          break;
        }
        int its = __shfl_sync(0xffffffffu, page, (i & 31) + (box < boxes ? box : 0));
        const bool loads = box < boxes && its != kNoBox;
        if (loads && (its < 0 || its >= p.c.n_pages)) {
          record(p.status, kStatusInvalidArg);
          its = 0;
        }
        const int n = __popc(__ballot_sync(0xffffffffu, loads));
        if (lane == 0) mbar_arrive_expect_tx(full(kv, s), (uint32_t)(n * 128) << p.box_shift);
        __syncwarp();
        if (loads) {
          const int slot = (box0 + i + box) << p.box_shift;
          const int row = ((its * p.Hkv + w.kvh) << page_shift) + (slot & ((1 << page_shift) - 1));
          tma_load_2d_hint(to + s * kStageBytes + half * kKVSub + ((box << p.box_shift) << 7), map, 64 * half, row,
                           full(kv, s), once);
        }
        __syncwarp();
        issued |= 1u << s;
        parity = (parity & ~(1u << s)) | (ph << s);
      }
    }
    if (failed && lane == 0) {
      *abort_flag = 1;
      report_timeout(p.status, 0x50 + 3 * kv);
    }
  } else if (warp >= 1 && warp <= NS) {
    // ---------------- the products of a slot: all lanes go through the loop, one issues
    const int g = warp - 1;
    constexpr uint32_t idesc_s = idesc_bf16_f32(kBQ, kBK);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(kBQ, kD) | (1u << 16);  // B (V) is MN-major
    const int rows = TURNS ? 0 : g, qs = SPLIT ? 0 : g;  // the slot's rows of a unit, and its queries' place
    const uint64_t dq = smem_desc_sw128(smem_u32(sQ + qs * kQBytes));
    const uint64_t dk = smem_desc_sw128(smem_u32(ring));
    const uint64_t dv = smem_desc_sw128_mn(smem_u32(ring + 2 * kKVSub), kKVSub, 1024);
    const uint32_t s_tmem = tmem + C::kSlotCols * g, o_tmem = s_tmem + 64 * C::kBufs;
    constexpr int kStep = SPLIT ? 2 : 1;  // from one of the slot's tiles to the next
    // The time is read every 32 looks in a row that find nothing; under a short limit at each, so that one runs out for
    // certain (a tile's exponentials are longer; a try_wait may sleep past any limit, and the global timer may stand).
    const unsigned look = budget < kShortNs ? 32 : 1;
    int J = 0, A = 0, units = 0;  // tiles of the CTA and of this slot, and its units
    bool failed = false;
    auto there = [](uint32_t bar, uint32_t ph) { return __all_sync(0xffffffffu, mbar_test_wait(bar, ph)) != 0; };
    auto wait = [&](uint32_t bar, uint32_t ph) { return __all_sync(0xffffffffu, mbar_wait(bar, ph, budget, abort_flag)) != 0; };
    // The slot's queries: loaded as soon as the last score product of a unit has read its own, and asked into L2 a
    // unit before that (behind the tiles in flight, a load from HBM would take 4 us).
    Walk ahead = *begin;
    int turn = 0;  // ahead's number
    auto find = [&] {
      while (ahead.on() && !(ahead.has(p, rows) && (!ALT || (turn & 1) == g))) ahead.next(p), ++turn;
      return ahead.on();
    };
    auto load_queries = [&] {
      if (!ahead.on() || (SPLIT && g != 0)) return;
      if (elect_one()) {
        // rows past the sequence's are others' or zeros: their scores are nobody's
        mbar_arrive_expect_tx(q_full(qs), (uint32_t)p.q_bytes);
#pragma unroll
        for (int half = 0; half < 2; ++half)
          tma_load_3d(smem_u32(sQ + qs * kQBytes + half * kQSub) + (ALT && g == 1 ? p.q_shift * 128 : 0), &p.tq_map, 64 * half, ahead.kvh * p.G,
                      ahead.seq.row0 + ahead.node0(p, rows), q_full(qs));
      }
      __syncwarp();
      q_loads++;
      ahead.next(p), ++turn;
      if (!SPLIT && find() && elect_one())
#pragma unroll
        for (int half = 0; half < 2; ++half)
          tma_prefetch_3d(&p.tq_map, 64 * half, ahead.kvh * p.G, ahead.seq.row0 + ahead.node0(p, rows));
      __syncwarp();
    };
    find();
    load_queries();
    int number = 0;
    for (Walk w = *begin; w.on() && !failed; w.next(p), ++number) {
      const int all = w.j1 - w.j0, n = SPLIT ? (all + 1 - g) / 2 : all;
      if (SPLIT && n == 0) break;  // (a cluster's CTA has one unit)
      if (ALT && (number & 1) != g) {
        J += n;
        continue;
      }
      // A slot looks at no tile before all tiles of the unit before have been seen there: a barrier's parity tells only
      // neighbouring phases apart, and no stage is more than one behind then.
      if (ALT && number > 0 && !wait(turn_over(1 - g), ((number - 1) >> 1) & 1)) {
        failed = true;
        break;
      }
      if (ALT && n == 0) {
        if (lane == 0) mbar_arrive(turn_over(g));
        continue;
      }
      if (!w.has(p, rows)) {  // nothing for this slot: the stages go back
        for (int j = 0; j < n && !failed; ++j, ++J)
          for (int kv = 0; kv < 2 && !failed; ++kv) {
            if (!wait(full(kv, J % C::kStages), (J / C::kStages) & 1)) failed = true;
            else if (lane == 0) mbar_arrive(empty(kv, J % C::kStages));
          }
        continue;
      }
      if constexpr (SPLIT) J = g;
      // What can be issued is, whatever it is: scores up to kBufs tiles ahead (their buffer's P has been read: its
      // product was issued before), the product of a tile whose P is there, the next unit's queries.
      if (!wait(q_full(qs), units & 1)) {
        failed = true;
        break;
      }
      int s = 0, v = 0;  // tiles whose scores and products have been issued
      bool q_wanted = false, over = !ALT;
      unsigned long long idle_since = 0;
      unsigned idle = 0;  // looks in a row that found nothing
      while (v < n) {
        bool did = false;
        if (s < n && s < v + C::kBufs) {
          const int at = J + s * kStep, st = at % C::kStages;
          if (there(full(0, st), (at / C::kStages) & 1)) {
            tc_fence_after();
            if (elect_one()) {
              const uint64_t b = dk + (uint64_t)(st * (kStageBytes >> 4));
              const uint32_t d = s_tmem + 64 * ((A + s) % C::kBufs);
#pragma unroll
              for (int kk = 0; kk < kD / 16; ++kk)
                tc_mma_bf16(d, dq + (uint64_t)((kk >> 2) * (kQSub >> 4) + (kk & 3) * 2),
                            b + (uint64_t)((kk >> 2) * (kKVSub >> 4) + (kk & 3) * 2), idesc_s, kk > 0 ? 1u : 0u);
              tc_commit(s_full(g, A + s));
              tc_commit(empty(0, st));
              if (s + 1 == n && !SPLIT) tc_commit(q_free(g));  // no further score product of this unit reads the queries
            }
            __syncwarp();
            mma_issued = true;
            if (++s == n && !SPLIT) q_wanted = true;
            did = true;
          }
        }
        if (v < s && there(p_ready(g, A + v), phase(A + v))) {
          const int at = J + v * kStep, st = at % C::kStages;
          if (there(full(1, st), (at / C::kStages) & 1) && (v > 0 || units == 0 || there(o_free(g), (units - 1) & 1))) {
            tc_fence_after();
            if (elect_one()) {
              const uint64_t b = dv + (uint64_t)(st * (kStageBytes >> 4));
              const uint32_t a = s_tmem + 64 * ((A + v) % C::kBufs);
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk)
                tc_mma_ts(o_tmem, a + kk * 8, b + (uint64_t)(kk * (16 * 128 >> 4)), idesc_pv, (v > 0 || kk > 0) ? 1u : 0u);
              tc_commit(empty(1, st));
              tc_commit(pv_done(g, A + v));
              if (v + 1 == n) tc_commit(o_done(g));
            }
            __syncwarp();
            ++v;
            did = true;
          }
        }
        if (!over && s == n) {  // the next tiles are the other slot's, as soon as V of the last ones is there
          over = true;
          for (int x = v; x < n; ++x) over &= there(full(1, (J + x) % C::kStages), ((J + x) / C::kStages) & 1);
          if (over && lane == 0) mbar_arrive(turn_over(g));
          __syncwarp();
        }
        if (q_wanted && there(q_free(g), units & 1)) {
          load_queries();
          q_wanted = false;
          did = true;
        }
        if (did) {
          idle = 0;
        } else if (((idle += look) & 31) == 0) {
          const unsigned long long now = clock64();
          if (idle == 32) idle_since = now;
          if (__any_sync(0xffffffffu, *abort_flag != 0 || now - idle_since > 2 * budget)) {  // 2.07 cycles a ns at most
            failed = true;
            break;
          }
        }
      }
      // A unit that was given up says nothing on turn_over: the other slot would take stages that are still being filled for
      // its own, and give them back. It sees the abort flag.
      __syncwarp();
      if (!failed && q_wanted) {
        if (wait(q_free(g), units & 1))
          load_queries();
        else
          failed = true;
      }
      J += n * kStep;
      A += n;
      ++units;
    }
    if (failed && lane == 0) {
      *abort_flag = 1;
      report_timeout(p.status, 0x51);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------- a slot's rows, one a thread
    const int g = (warp - 4) >> 2, quarter = warp & 3;
    // the row of a lane; of single tokens, the second slot's begin at lane 64, whose warp is on another quarter of the SM
    // than the first slot's
    const int r = (quarter * 32 + lane - (ALT && g == 1 ? p.q_shift : 0)) & (kBQ - 1);
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_taddr = tmem + lane_off + C::kSlotCols * g, o_taddr = s_taddr + 64 * C::kBufs;
    const int node_of_row = r / p.G, head_of_row = r - node_of_row * p.G;
    int J = 0, A = 0, units = 0, number = 0;
    bool failed = false;
    for (Walk w = *begin; w.on() && !failed; w.next(p), ++number) {
      const int rows = TURNS ? 0 : g, all = w.j1 - w.j0;
      const int n = SPLIT ? (all + 1 - g) / 2 : all, node0 = w.node0(p, rows);
      if (SPLIT && n == 0) break;  // (a cluster's CTA has one unit)
      if (!w.has(p, rows) || (ALT && (number & 1) != g)) {
        J += n;
        continue;
      }
      if constexpr (SPLIT) J = g;
      const int node = node0 + node_of_row;
      const bool valid = node_of_row < p.tq && node < w.seq.n;
      const bool live = __any_sync(0xffffffffu, valid);
      const int len = w.seq.len;
      // what the row sees: slots [low, len) and the nodes in kin (a tree), or slots [low, high) (a chain)
      unsigned long long kin = 0;
      int depth = node;
      if (p.parents && valid) {
        depth = 0;
        for (int x = node;;) {
          if (p.window == 0 || depth < p.window) kin |= 1ull << x;
          const int up = p.parents[w.seq.row0 + x];
          if (up >= x) record(p.status, kStatusInvalidArg);
          if (up < 0 || up >= x) break;
          x = up;
          ++depth;
        }
      }
      __syncwarp();
      const int low = p.window > 0 ? len + depth - p.window + 1 : 0;
      const int high = !valid ? 0 : p.parents ? len : len + node + 1;
      // tiles whose scores are all seen by all rows
      const int last = min(w.seq.n, p.parents ? kMaxNodes : node0 + p.tq) - 1;  // the deepest row, or deeper
      const int plain_lo = p.window > 0 ? len + last - p.window + 1 : 0;
      const int plain_hi = (p.parents ? len : len + node0 + 1) - kBK;
      float m_ref = -INFINITY, l = 0.f;
      constexpr int kStep = SPLIT ? 2 : 1;
      for (int j = 0; j < n; ++j, J += kStep, ++A) {
        const int n0 = (w.keys.tile0() + w.j0 + (SPLIT ? J : j)) * kBK;
        if (!__all_sync(0xffffffffu, mbar_wait(s_full(g, A), phase(A), budget, abort_flag))) {
          failed = true;
          break;
        }
        __syncwarp();
        tc_fence_after();
        // Rows of V that were not loaded, or lie outside the keys, may hold anything: zero, so that P = 0
        // meets finite values. Both slots write the same zeros, each before its own product.
        const int v_lo = w.keys.first - n0, v_hi = w.keys.end - n0;
        if (v_lo > 0 || v_hi < kBK) {
          const int st = J % C::kStages;
          if (!__all_sync(0xffffffffu, mbar_wait(full(1, st), (J / C::kStages) & 1, budget, abort_flag))) {
            failed = true;
            break;
          }
          const int row = r & 63;  // two threads a row, a half each
          if (row < v_lo || row >= v_hi) {
            const uint32_t at = smem_u32(ring + st * kStageBytes + (2 + (r >> 6)) * kKVSub) + row * 128;
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) st_shared_u4(at + (((ch + row) & 7) << 4), 0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!live) {  // nobody reads these rows: whatever the score buffer holds may stand for P
          tc_fence_before();
          mbar_arrive(p_ready(g, A));
          continue;
        }
        const uint32_t s_buf = s_taddr + 64 * (A % C::kBufs);
        float x[kBK];
#pragma unroll
        for (int c = 0; c < kBK; c += 16) tmem_ld16(s_buf + c, *reinterpret_cast<float(*)[16]>(&x[c]));
        tc_wait_ld();
        if (n0 < plain_lo || n0 > plain_hi) {
          unsigned long long seen = bits_from(low - n0) & bits_below(high - n0);
          if (p.parents) {
            const int a = len - n0;  // the column of node 0
            seen |= a >= 64 ? 0ull : a >= 0 ? kin << a : a > -64 ? kin >> -a : 0ull;
          }
#pragma unroll
          for (int c = 0; c < kBK; ++c)
            if (!((seen >> c) & 1)) x[c] = -INFINITY;
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < kBK; c += 2) mx[(c >> 1) & 3] = fmax3(mx[(c >> 1) & 3], x[c], x[c + 1]);
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * kScaleLog2;
        const bool need = mt > m_ref + kRescaleLog2;
        if (__any_sync(0xffffffffu, need)) {
          float alpha = 1.f;
          if (need) {
            alpha = ex2_approx(m_ref - mt);
            m_ref = mt;
          }
          l *= alpha;
          if (j > 0) {  // the products so far are to be complete, then O moves to the new reference
            if (!__all_sync(0xffffffffu, mbar_wait(pv_done(g, A - 1), phase(A - 1), budget, abort_flag))) {
              failed = true;
              break;
            }
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kD; c += 16) {
              float ov[16];
              tmem_ld16(o_taddr + c, ov);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) ov[i] *= alpha;
              tmem_st16(o_taddr + c, ov);
            }
          }
          __syncwarp();
        }
        const float neg_mu = m_ref == -INFINITY ? 0.f : -m_ref;
        const f32x2 scale2 = f2_make(kScaleLog2, kScaleLog2), mu2 = f2_make(neg_mu, neg_mu);
        f32x2 sum2[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float pw[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float t0, t1;
            f2_split(f2_fma(f2_make(x[32 * h + 2 * i], x[32 * h + 2 * i + 1]), scale2, mu2), t0, t1);
            const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
            sum2[i & 1] = f2_add(sum2[i & 1], f2_make(p0, p1));
            pw[i] = __uint_as_float(pack_bf16x2(p0, p1));
          }
          tmem_st16(s_buf + 16 * h, pw);
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(p_ready(g, A));
        float a0, a1, b0, b1;
        f2_split(sum2[0], a0, a1);
        f2_split(sum2[1], b0, b1);
        l += (a0 + a1) + (b0 + b1);
      }
      if (failed) break;
      if (!__all_sync(0xffffffffu, mbar_wait(o_done(g), units & 1, budget, abort_flag))) {
        failed = true;
        break;
      }
      __syncwarp();
      tc_fence_after();
      if (!CL && live) {
        const bool whole = w.whole();
        const size_t part = (size_t)(2 * blockIdx.x + min(number, 1)) * p.slots + rows;
        float* const acc = p.acc + part * kBQ * kD + 4 * r;
        // a row sees itself at least: a sum that is NaN, or 0 where all its scores are -inf, gives NaN
        const float inv = whole ? 1.f / l : 1.f;
        __nv_bfloat16* const o = static_cast<__nv_bfloat16*>(p.o.ptr) + (w.seq.row0 + (valid ? node : 0)) * p.o.row +
                                 (long long)(w.kvh * p.G + head_of_row) * p.o.head;
        if (valid && !whole) p.ml[part * kBQ + r] = make_float2(m_ref, l);
#pragma unroll 1
        for (int c = 0; c < kD; c += 32) {
          float ov[32];
          tmem_ld16(o_taddr + c, *reinterpret_cast<float(*)[16]>(&ov[0]));
          tmem_ld16(o_taddr + c + 16, *reinterpret_cast<float(*)[16]>(&ov[16]));
          tc_wait_ld();
          if (valid && whole) {
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
              uint4 a, b;
              uint32_t* const w8[2] = {&a.x, &b.x};
#pragma unroll
              for (int i = 0; i < 8; ++i) w8[i >> 2][i & 3] = pack_bf16x2(ov[h + 2 * i] * inv, ov[h + 2 * i + 1] * inv);
              if (p.o_wide) {
                st_global_32(o + c + h, a, b);
              } else {
                reinterpret_cast<uint4*>(o + c + h)[0] = a;
                reinterpret_cast<uint4*>(o + c + h)[1] = b;
              }
            }
          } else if (valid) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(acc + (c + i) * kBQ) = make_float4(ov[i], ov[i + 1], ov[i + 2], ov[i + 3]);
          }
          __syncwarp();
        }
      }
      if constexpr (CL) {  // its outputs stay in tensor memory for the cluster (below)
        share_live = live;
        share = make_float2(m_ref, l);
      }
      tc_fence_before();
      mbar_arrive(o_free(g));
      ++units;
    }
    if (failed) {
      *abort_flag = 1;
      if (lane == 0) report_timeout(p.status, 0x52);
    }
  }

  tc_fence_before();
  __syncthreads();
  // Every role has stopped issuing. After an abort, copies and MMAs that nobody waited for may still be in
  // flight: they complete before TMEM is freed and the CTA exits. Every thread reads the same flag.
  if (*abort_flag) {
    volatile int never = 0;
    if ((warp == 0 || warp == 3) && lane == 0) {
      for (int s = 0; s < C::kStages; ++s)
        if (issued & (1u << s)) mbar_wait(full(warp == 0 ? 0 : 1, s), (parity >> s) & 1, kDrainNs, &never);
    } else if (warp >= 1 && warp <= NS) {
      if (q_loads > 0) mbar_wait(q_full(warp - 1), (q_loads - 1) & 1, kDrainNs, &never);
      __syncwarp();
      if (mma_issued) {
        if (elect_one()) tc_commit(drain(warp - 1));  // the lane that issued the products
        __syncwarp();
        mbar_wait(drain(warp - 1), 0, kDrainNs, &never);
      }
      __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
  }
  if (CL && warp >= 4) {
    // the products have read the queries and the ring: a share's sums and outputs take their place
    tc_fence_after();
    const int g = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
    reinterpret_cast<float2*>(sQ)[g * kBQ + r] = share;
    if (share_live && !*abort_flag) {
      const uint32_t o_taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::kSlotCols * g + 64 * C::kBufs;
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        float ov[32];
        tmem_ld16(o_taddr + c, *reinterpret_cast<float(*)[16]>(&ov[0]));
        tmem_ld16(o_taddr + c + 16, *reinterpret_cast<float(*)[16]>(&ov[16]));
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          reinterpret_cast<float4*>(ring)[(g * (kD / 4) + (c + i) / 4) * kBQ + r] = make_float4(ov[i], ov[i + 1], ov[i + 2], ov[i + 3]);
      }
    }
    tc_fence_before();
  }
  if constexpr (CL) {
    // The shares of the cluster's CTAs joined in their order, as the second kernel does with parts: a thread
    // has four channels of a row at a time.
    __syncwarp();
    cluster_sync_all();
    const Walk w = *begin;
    if (w.seq.n > 0) {
      constexpr int kRowSlots = SPLIT ? 1 : NS, kParts = SPLIT ? 2 : 1;  // parts of a CTA
      const int parts = p.cluster * kParts, threads = p.cluster * C::kThreads;
#pragma unroll
      for (int g = 0; g < kRowSlots; ++g) {
        const int n = min(p.tq, w.seq.n - w.node0(p, g)) * p.G;  // rows of the slot
        for (int i = cluster_ctarank() * C::kThreads + threadIdx.x; i < n * (kD / 4); i += threads) {
          const int ch = i / n, r = i - ch * n, nd = r / p.G;
          Joined x;
          constexpr int kAtOnce = 12;
          for (int k0 = 0; k0 < parts; k0 += kAtOnce) {
            float2 ml[kAtOnce];
            float4 a[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
              ml[j] = make_float2(-INFINITY, 0.f);
              a[j] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (k0 + j < parts) {
                const int cta = (k0 + j) / kParts, slot = SPLIT ? (k0 + j) % kParts : g;
                ml[j] = ld_dsmem_f2(map_shared_rank(smem_u32(sQ) + 8 * (slot * kBQ + r), cta));
                a[j] = ld_dsmem_f4(map_shared_rank(smem_u32(ring) + (((slot * (kD / 4) + ch) * kBQ + r) << 4), cta));
              }
            }
            x.take(ml, a);
          }
          x.store(p, w.seq.row0 + w.node0(p, g) + nd, w.kvh * p.G + r - nd * p.G, ch);
        }
      }
    }
    __syncwarp();
    cluster_sync_all();  // nobody leaves while its share may be read
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------ joining partial results

// Block (c - 1, y): what stretch c says (Join), in the order of the parts; a thread has four channels of a row, a
// warp 32 rows, PARTS parts are under way at a time.
constexpr int kJoinThreads = 256;
template <int PARTS>
__global__ void __launch_bounds__(kJoinThreads) attn_paged_join_kernel(const __grid_constant__ AttnParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, c = blockIdx.x + 1;
  const Join w = p.joins[c];
  if (w.last < 0) return;
  const int warp = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5), warps = gridDim.y * (kJoinThreads / 32);
  for (int i = warp; i < p.slots * (kBQ / 32) * (kD / 4); i += warps) {
    const int ch = i % (kD / 4), quarter = i / (kD / 4) % (kBQ / 32), g = i / (kD / 4) / (kBQ / 32);
    const int r = quarter * 32 + lane, nd = r / p.G, node = (w.t * p.slots + g) * p.tq + nd;
    if (nd >= p.tq || node >= w.seq.n) continue;
    Joined x;
    for (int k0 = c - 1; k0 <= w.last; k0 += PARTS) {
      float2 ml[PARTS];
      float4 a[PARTS];
#pragma unroll
      for (int j = 0; j < PARTS; ++j) {
        const int k = k0 + j;
        const size_t at = (size_t)(k == c - 1 ? w.first : 2 * k) * p.slots + g;
        ml[j] = make_float2(-INFINITY, 0.f);
        a[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k <= w.last) {
          ml[j] = p.ml[at * kBQ + r];
          a[j] = reinterpret_cast<const float4*>(p.acc + at * kBQ * kD)[ch * kBQ + r];
        }
      }
      x.take(ml, a);
    }
    x.store(p, w.seq.row0 + node, w.kvh * p.G + r - nd * p.G, ch);
  }
}

// How a call is cut, from what the host knows of it: the sequences' lengths are on the device, so that the page list's length
// (capacity) stands for them. The figures below are with lists as long as the longest sequence. With longer ones: 16
// sequences of up to 300 slots 8.2 -> 12.9 us (lists for 8192), of up to 1000 13.0 -> 17.0; 4 of up to 2000 9.2 -> 12.5
// (131072; 9.1 with 8192), of up to 8000 21.1 -> 22.5; 4 trees over up to 500 15.5 -> 22.3 (131072). One sequence, windows and what
// takes the line anyway: no difference.
struct Plan {
  int slots, grid, unit_cost, units, cluster;
  bool fits;  // the line is shorter than 2^31
};

// Clusters of `size` CTAs of the kernel that are resident at once, 0 if it cannot be launched so; asked once per device.
template <bool TURNS>
int resident_clusters(int size) {
  static std::atomic<int> known[64][kMaxCluster + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int was = known[dev][size].load(std::memory_order_relaxed);
  if (was != 0) return was - 1;
  const auto kernel = attn_paged_kernel<true, TURNS>;
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)size);
  cfg.blockDim = dim3(Cfg<true, TURNS>::kThreads);
  cfg.dynamicSmemBytes = Cfg<true, TURNS>::kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Cfg<true, TURNS>::kSmem) != cudaSuccess ||
      cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  known[dev][size].store(n + 1, std::memory_order_relaxed);
  return n;
}

Plan plan_of(int rows, int B, int H, int Hkv, bool cu, bool tree, long long capacity, int window, int num_sms) {
  Plan pl{};
  const int G = H / Hkv, tq = kBQ / G;
  const long long per_seq = (long long)rows * G;  // matrix rows of all sequences of a KV head
  // A unit of both slots costs 1 to 2 us more where one slot would do (16 trees of 32 nodes over 4096 slots 58.3 us against
  // 56.7), units of one slot read the cache twice where they do not (of 40: 92.1 against 66.4, ragged ones up to 40 of 121 rows
  // on average 55.9 against 51.5).
  pl.slots = per_seq > 96ll * B ? 2 : 1;
  pl.grid = num_sms;
  // A unit's queries, first scores and outputs take the time of about four tiles, of two where the slots take units in
  // turn; where every CTA has about a unit of its own, that shares the work out better. 16 trees of up to 64 nodes: 58.7 us
  // with no tiles, 56.5 with 4, 59 to 62 with 7 to 14. 256 sequences of up to 1000 slots, a token each: 111, 114, 117,
  // 121 and 123 us with 1, 2, 4, 6 and 9, of up to 100 43.6, 40.2, 41.9, 40.4, 42.4. With fewer units it would leave CTAs
  // without tiles.
  pl.unit_cost = 2ll * B * Hkv <= num_sms ? 0 : pl.slots == 2 ? 4 : 2;
  const int nodes = tq * pl.slots, most = tree ? std::min(rows, kMaxNodes) : cu ? rows : 1;
  // units of a KV head: what fills a unit whole, and one more for each sequence
  pl.units = (int)std::min<long long>((long long)B * ((most + nodes - 1) / nodes), (long long)B + rows / nodes);
  const long long keys = std::min(capacity, window > 0 ? (long long)window + (tree ? kMaxNodes : nodes) : capacity);
  const long long tiles = keys / kBK + 2;
  pl.fits = ((long long)B + rows / nodes + 1) * Hkv * (tiles + pl.unit_cost) < 0x7fffffffll;
  // Clusters: a unit each, its keys in equal shares, no list to add up and no second kernel. Where lengths differ
  // their CTAs end at different times, up to where the longest sequence alone costs more than the line's second
  // kernel does (8 KV heads, one token each; the line against clusters, us): 4 sequences of 2000 14.6 against 9.2, of
  // 16000 50 against 43, one of 16000 and three of one slot 42 against 32 (63 tiles a CTA), of 32000 53 against 58.
  // Single CTAs likewise, where a unit has few tiles and one slot: 16 sequences of up to 300 12.8 against 8.0, of up to 1000
  // 18.2 against 13.7, of up to 2000 23.8 against 21.0 (but one of 2000 and 15 of one slot 13.1 against 18.6). Not so trees of two
  // slots (10 over 500 slots 20.9 against 30.7) and more units than SMs (64 sequences of up to 100 14.2 against 28.5).
  pl.cluster = 0;
  const long long units = (long long)Hkv * pl.units;
  for (int size = kMaxCluster; size > 0; --size)
    if (units * size <= num_sms && (size > 1 || pl.slots == 1) &&
        ((B == 1 && size > 1) || tiles <= (size > 1 ? kClusterTiles * size : kWholeTiles)) &&
        (pl.slots == 2 ? resident_clusters<false>(size) : resident_clusters<true>(size)) >= units) {
      pl.cluster = size;
      break;
    }
  return pl;
}

}  // namespace

size_t attn_paged_ws_bytes(int rows, int B, int H, int Hkv, bool cu, bool tree, long long capacity, int window, int num_sms) {
  if (rows <= 0 || B <= 0) return 0;
  const Plan pl = plan_of(rows, B, H, Hkv, cu, tree, capacity, window, num_sms);
  if (!pl.fits) return kAttnPagedTooLong;
  if (pl.cluster > 0) return 0;
  return (size_t)2 * pl.grid * pl.slots * kBQ * (sizeof(float2) + kD * sizeof(float)) + pl.grid * sizeof(Join);
}

cudaError_t launch_attn_paged(const HeadRows& q, const PagedCache& c, const HeadRows& o, int rows, const int* cu,
                              const int* parents, int B, int H, int Hkv, int window, void* ws, int num_sms,
                              DevStatus* st, unsigned long long wait_ns, cudaStream_t s, const char** why) {
  if (rows <= 0 || B <= 0) return cudaSuccess;
  const Plan pl = plan_of(rows, B, H, Hkv, cu != nullptr, parents != nullptr, page_slots(c), window, num_sms);
  AttnParams p;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  const int box = std::min(1 << c.page_shift, kBK);
  const int cache_rows = (c.n_pages * Hkv) << c.page_shift;  // checked by the caller
  p.G = H / Hkv;
  p.tq = kBQ / p.G;
  const int box_rows = cu ? p.tq : 1;  // without a list no sequence has more than a row
  p.q_bytes = box_rows * p.G * kD * 2;
  p.q_shift = cu ? 0 : 64;
  if (!make_tma_2d_16b(&p.tk, c.k, cache_rows, kD, box, false) || !make_tma_2d_16b(&p.tv, c.v, cache_rows, kD, box, false) ||
      !make_tma_heads_bf16(&p.tq_map, q, rows, H, kD, p.G, box_rows)) {
    *why = "cuTensorMapEncodeTiled failed for the cache or the queries";
    return cudaErrorInvalidValue;
  }
  p.o = o;
  p.c = c;
  p.cu = cu;
  p.parents = parents;
  p.rows = rows;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.window = window > 0 ? window : 0;
  p.slots = pl.slots;
  const bool two = pl.slots == 2;
  while ((1 << p.box_shift) < box) ++p.box_shift;
  p.grid = pl.grid;
  p.cluster = pl.cluster;
  p.single = pl.units == B;
  p.unit_cost = pl.cluster > 0 ? 0 : pl.unit_cost;
  p.o_wide = reinterpret_cast<uintptr_t>(o.ptr) % 32 == 0 && (rows == 1 || o.row % 16 == 0) && (H == 1 || o.head % 16 == 0);
  p.status = st;
  p.wait_ns = wait_ns;
  if (pl.cluster > 0)  // configured when the resident clusters were asked for
    return launch_clusters(two ? attn_paged_kernel<true, false> : attn_paged_kernel<true, true>, Hkv * pl.units * pl.cluster,
                           Cfg<true, false>::kThreads, two ? Cfg<true, false>::kSmem : Cfg<true, true>::kSmem, pl.cluster, s, p);
  const int smem = Cfg<false, false>::kSmem, threads = Cfg<false, false>::kThreads;
  static_assert(Cfg<false, true>::kSmem == Cfg<false, false>::kSmem, "of both");
  p.acc = static_cast<float*>(ws);
  p.ml = reinterpret_cast<float2*>(p.acc + (size_t)2 * pl.grid * pl.slots * kBQ * kD);
  p.joins = reinterpret_cast<Join*>(p.ml + (size_t)2 * pl.grid * pl.slots * kBQ);
  const auto kernel = two ? attn_paged_kernel<false, false> : attn_paged_kernel<false, true>;
  static std::atomic<unsigned long long> configured[2];
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(kernel), smem, configured[two]);
  if (e == cudaSuccess) e = launch_pdl(kernel, pl.grid, threads, smem, s, p);
  if (e != cudaSuccess || pl.grid == 1) return e;
  // few units: many parts each, and all of them loaded at once; many units: a few parts each, more blocks per SM
  const bool few = 4ll * B * Hkv <= num_sms;
  return launch_pdl(few ? attn_paged_join_kernel<10> : attn_paged_join_kernel<4>, dim3(pl.grid - 1, two ? 16 : 4),
                    kJoinThreads, 0, s, p);
}

}  // namespace blk

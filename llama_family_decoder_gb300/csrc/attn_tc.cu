// Prefill attention on the 5th-generation tensor core (tcgen05 + TMEM), causal,
// grouped-query, head_dim 128 ("LlamaForCausalLM-32L-4096d" sheet: softmax(q @
// k.T / sqrt(128), mask=causal) @ v per head; "arcee", "Grouped-query attention,
// 128-wide heads": query head h reads KV head h / (H / Hkv)).
//
// Work items of two 128-query slots that share every K/V tile: two query heads of
// one KV group at the same query tile (an even group size), or two consecutive
// query tiles of one head (otherwise). Persistent: one CTA per SM walks the items,
// heaviest first, dealt out in a snake order; barrier phases and ring positions run
// on across items, so that the next item's Q, first K/V tiles and first score
// products overlap the current item's last softmax, PV and output store.
// 352 threads:
//   warp 0      TMA producers: lane 0 both slots' Q tiles once, then K tiles of
//               128 keys through a 2-stage ring; lane 1 the V tiles through their
//               own 2-stage ring (128-byte swizzle, 64-column boxes).
//   warps 1, 10 MMA issuers, lane 0 of warp 1 for slot 0 and of warp 10 for slot 1
//               (warp 1 also allocates TMEM): per key tile j, O_g += P_g V_j (A = P
//               from tensor memory, B = V as an MN-major operand) as soon as the
//               slot's P_j is written, then at once S_g = Q_g K_{j+1}^T (M=128,
//               N=128) into the slot's score buffer.
//   warps 2..9  softmax, four warps per slot, one query row per thread: read S_j
//               from TMEM, mask, exponentiate in the log2 domain against a running
//               reference max, and write P_j (fp16 or bf16 pairs) over the first 64
//               columns of the same TMEM buffer; rescale O in TMEM only when the row
//               max grew by more than 2^8 (exact: softmax does not depend on the
//               reference); finally O / l to the head-major output.
// The slots take turns: while one slot's softmax works on its tile, the tensor
// core runs the other slot's PV and next score product. P never touches shared
// memory, so the tensor core's shared-memory reads are Q, K and V alone. The MMAs
// of one thread run in issue order: S_{j+1} of a slot, issued after that slot's
// PV_j, overwrites P_j only once PV_j has read it, and a commit after S_j also
// covers PV_{j-1} (so O is stable whenever S_j is ready).
// Options of the "afmoe" block ("Rotary runs on the sliding-window blocks only";
// "Attention: per-head q/k norms and a sigmoid gate on every head"): a window
// over the last W positions (key tiles before the first query's oldest key are
// skipped, the rest masked), and a per-channel gate on the output; a padded batch
// hides the keys outside each sequence's run of real tokens.
// Packed sequences (PACKED) go through the same loop with 512 threads (see kPackedThreads):
// whole prompts of any lengths, the heads of a KV head folded into a tile's rows. Bound by the
// chain of a tile pair (scores, softmax, PV: 3400 cycles by clock reads in the kernel, of which the
// tensor core works 2048), and by an item's masked tiles and the start of the next one (3900 cycles
// more than plain tiles take): 410 to 420 us, 1.3 PFLOP/s, for one sequence of 8190 (32 heads of
// their own), 112 us, 1.0 PFLOP/s, for 8 ragged ones of up to 2048 (32 heads over 8), 24.5 us for 48
// turns of up to 200. Measured and not kept: sixteen softmax warps, two threads a row, with the
// scores read twice from tensor memory (498 us for the long one; held in registers they spill, and
// shared memory leaves too little L1 for that: 1167); outputs staged in shared memory for whole-row
// stores (48 short turns 39 -> 41 us); a third Q buffer (27 -> 28 us); masked tiles read by 64 keys
// (24.7 -> 26.8 us) or a quarter ahead (27.4, spills); turns for the exponentials alone (the long
// one 448 us).
// Every wait is bounded; on expiry the CTA records a timeout, drains its own
// copies and MMAs, frees its TMEM and returns.
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace blk {

namespace {

constexpr int kD = 128;
constexpr int kBQ = 128;                    // queries per slot (MMA M)
constexpr int kBK = 128;                    // keys per tile
constexpr int kSlots = 2;
constexpr int kThreads = 64 + kSlots * 128 + 32;  // + warp 10: the second slot's MMA issuer
// Packed sequences: four warpgroups, the softmax in the first two (warps 0..7), then the TMA
// producers, the two MMA issuers and an idle warp, then the epilogue, which reads an item's
// outputs out while the softmax is at the next item (with the softmax warps storing, an item
// boundary took 8500 cycles, two and a half tiles' time). Registers move from the last two to
// the first two, whose scores (128 a thread) and addresses do not fit 128.
constexpr int kPackedThreads = 512;
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 176, kControlRegs = 112, kEpilogueRegs = 48;
static_assert(2 * kSoftmaxRegs + kControlRegs + kEpilogueRegs <= 4 * kLaunchRegs, "the registers the block is launched with");
constexpr int kQSub = kBQ * 128;            // one 64-column half of a Q tile (bytes)
constexpr int kQBytes = 2 * kQSub;          // 128 queries x 128 dims
constexpr int kKVSub = kBK * 128;           // one 64-column half of a K or V tile
constexpr int kKVBytes = 2 * kKVSub;        // 128 keys x 128 dims
constexpr int kKStages = 2;                 // K ring
constexpr int kVStages = 2;                 // V ring
constexpr int kSmem = 1024 + kSlots * kQBytes + (kKStages + kVStages) * kKVBytes + 256;
// + more barriers, the slots' softmax states of an item, and the CTA's own work entries
constexpr int kOwnItems = 256;
// The slots take turns (see the softmax) in a CTA with a sequence longer than this. Tiles that are
// mostly masked are bound by latency, which the slots hide for each other: 64 prompts of 150
// 101.7 us in turns, 91.4 at their own pace (32 heads of their own), of 400 245 and 231; in the
// plain tiles of long ones they fall into step (8190 queries 408 and 489, 32 prompts of 800 in 8
// heads over 2 59.4 and 61.4).
constexpr int kTurnKeys = 512;
constexpr int kSmemPacked = kSmem + 32 + kSlots * kBQ * 8 + kOwnItems * 16;
static_assert(kSmemPacked <= 227 * 1024, "shared memory");
constexpr float kRescaleLog2 = 8.0f;
constexpr int kStatusInvalidArg = 1;        // == BLK_ERR_INVALID_ARG
constexpr unsigned long long kDrainNs = 2000000000ULL;
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kSmem <= 227 * 1024, "shared memory");
static_assert(kQSub == kKVSub && kKStages == 2 && kVStages == 2, "the MMA issuers' descriptor steps and stage selects");

// A query tile of a packed sequence (or, not split, two of them): queries from `query` on of the
// sequence whose len rows start at row0.
struct __align__(16) PackedWork {
  int row0, len, query, unused;
};

struct AttnParams {
  CUtensorMap tq, tk, tv;
  void* o;
  int o_f16;
  int B, H, Hkv, T, n_qtiles;
  int head_pairs;  // 1: the two slots are heads 2i, 2i+1 at one query tile; 0: query tiles 2k, 2k+1 of one head
  int n_items;
  // K/V rows per (sequence, KV head): T, or a cache's capacity; q_off: positions already
  // in that cache per sequence (the T queries sit at q_off[b] ..), or null for 0
  int kv_stride;
  const int* q_off;
  // "afmoe": window > 0 keeps the keys at positions > query - window; gate (fp16, the
  // output's layout) multiplies the output, ungated (bf16) receives it before the gate
  int window;
  const __half* gate;
  __nv_bfloat16* ungated;
  const int2* key_range;  // per sequence [lo, hi): the visible (non-padding) keys, or null
  float sl2;
  DevStatus* status;
  unsigned long long wait_ns;
  // packed sequences: the work list (heaviest first) and its length, both on the device, and
  // the output's strides
  const PackedWork* work;  // null: every CTA makes the list itself from cu (see own_work)
  const int* n_work;
  const int* cu;
  int step, cap;  // queries of an entry, entries at most
  long long o_row, o_head;
  // 2^fold query heads of a KV head share a slot's 128 rows: row r is head r % 2^fold of query
  // r / 2^fold
  int fold;
  int o_wide;  // the output's rows start on 32-byte boundaries
};

// 2^x on the MUFU unit (one instruction; -inf gives +0).
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max of three (one instruction; like fmaxf, a NaN operand is ignored)
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, bool f16) {
  if (f16) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  return pack_bf16x2(lo, hi);
}

// D[tmem] (+)= A[tmem] * B[smem desc]: the A operand (M rows on the TMEM lanes, K
// 16-bit elements packed two per 32-bit column) read from tensor memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 bytes in one store (a 32-byte boundary): a warp's stores of 32 separate rows are bound by
// the rows they touch, so half as many instructions take half the time.
__device__ __forceinline__ void st_global_32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

struct Slot {
  int h, qt, m0, valid;
};

// A work item: two slots over one KV head of one sequence, and its key-tile range.
struct Item {
  Slot sl[kSlots];
  int b, kv_row, off, kv_lo, kv_hi, n_keys, t0, n_tiles;
  int kvh, T, tq;  // the KV head, the sequence's queries, a slot's queries
};

// Item id, heaviest first: the far query tiles (more keys) get the small ids. Reads
// the cache positions and key ranges, so it runs after pdl_wait. PACKED: of work entry `w`.
template <bool PACKED, bool SPLIT>
__device__ __forceinline__ Item item_of(const AttnParams& p, int id, const PackedWork& w) {
  Item it;
  it.T = p.T;
  it.tq = kBQ;
  if constexpr (PACKED) {
    const int h = (id % (p.H >> p.fold)) << p.fold;
    it.tq = kBQ >> p.fold;
    it.T = w.len;
    it.b = w.row0;
#pragma unroll
    for (int g = 0; g < kSlots; ++g) {
      const int m0 = SPLIT ? w.query : w.query + g * it.tq;
      const int ok = m0 < w.len;
      it.sl[g] = {h, 0, ok ? m0 : w.query, ok};
    }
  } else if (p.head_pairs) {
    const int hp_n = p.H / 2;
    const int qt = p.n_qtiles - 1 - id / (p.B * hp_n);
    const int r = id % (p.B * hp_n);
    const int hp = r % hp_n;
    it.b = r / hp_n;
#pragma unroll
    for (int g = 0; g < kSlots; ++g) it.sl[g] = {2 * hp + g, qt, qt * kBQ, 1};
  } else {
    const int np = (p.n_qtiles + 1) / 2;
    const int k = np - 1 - id / (p.B * p.H);
    const int r = id % (p.B * p.H);
    const int h = r % p.H;
    it.b = r / p.H;
#pragma unroll
    for (int g = 0; g < kSlots; ++g) {
      const int qt = 2 * k + g;
      const int ok = qt < p.n_qtiles;
      it.sl[g] = {h, ok ? qt : 2 * k, (ok ? qt : 2 * k) * kBQ, ok};
    }
  }
  it.kvh = it.sl[0].h / (p.H / p.Hkv);
  if constexpr (PACKED) {
    it.kv_row = it.b;  // the sequence's first row: keys and queries are the same rows
    it.off = it.kv_lo = 0;
    it.kv_hi = it.T;
  } else {
    it.kv_row = (it.b * p.Hkv + it.kvh) * p.kv_stride;
    it.off = p.q_off ? p.q_off[it.b] : 0;  // keys 0 .. off - 1 are earlier positions in the cache
    // visible keys: [kv_lo, kv_hi) (an attention_mask's run of real tokens, else all)
    const int2 kr = p.key_range ? p.key_range[it.b] : make_int2(0, it.off + p.T);
    it.kv_lo = kr.x;
    it.kv_hi = kr.y;
  }
  // the key tiles the item needs: the union of both slots' ranges
  int n_keys = 0, first_key = 1 << 30;
#pragma unroll
  for (int g = 0; g < kSlots; ++g) {
    const int kv_end = min(it.T, it.sl[g].m0 + it.tq);
    n_keys = max(n_keys, min(it.off + kv_end, it.kv_hi));
    first_key = min(first_key, max(it.kv_lo, p.window > 0 ? it.off + it.sl[g].m0 - p.window + 1 : 0));
  }
  it.n_keys = n_keys;
  it.t0 = max(0, first_key) / kBK;
  it.n_tiles = max(0, (n_keys + kBK - 1) / kBK - it.t0);  // none when every query is padding
  return it;
}

// Round k of CTA c among G: the heaviest-first ids dealt out in a snake (c, then
// 2G - 1 - c, ...), so that every CTA's rounds sum to about the same work.
__device__ __forceinline__ int item_id(int k, int G, int c) { return k * G + ((k & 1) ? G - 1 - c : c); }

// The work list of packed sequences (heaviest first, an entry per `step` queries, ordered by its
// place in its sequence, which its key count grows with, then by sequence), as far as a CTA
// needs it: mine[k] := the entry of the CTA's item k, longest := the longest of their
// sequences. Returns the number of items. The order
// is the same in every CTA. F(t), the entries at places t and farther, falls with t: the place
// of entry e is the last t with F(t) > e, found by halving, and its sequence is the one number
// e - F(t + 1) of those that reach t. A warp finds an item at a time; `scratch` holds the
// sequences. A cu that does not rise from >= 0 to at most the rows records INVALID_ARG and is read
// as the running maximum of its clamped numbers: sequences never overlap, so that there are at most
// p.cap entries, and the sums fit.
constexpr int kOwnSeqs = 2048;
__device__ __forceinline__ int running_max(int x, int lane) {  // over the lanes up to this one
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = max(x, u);
  }
  return x;
}
__device__ __noinline__ int own_work(const AttnParams& p, uint8_t* scratch, int units, PackedWork* mine, int* longest) {
  int* n_of = reinterpret_cast<int*>(scratch);                 // [B] a sequence's entries
  int2* rows = reinterpret_cast<int2*>(n_of + kOwnSeqs);       // its first row and its length
  static_assert(kOwnSeqs * 12 <= (kKStages + kVStages) * kKVBytes, "scratch");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  bool bad = false, falls = false;
  auto put = [&](int b, int lo, int hi) {
    rows[b] = make_int2(lo, hi - lo);
    n_of[b] = (hi - lo + p.step - 1) / p.step;
  };
  for (int b = tid; b < p.B; b += blockDim.x) {
    const int a = p.cu[b], e = p.cu[b + 1];
    const int lo = min(max(a, 0), p.T), hi = min(max(e, lo), p.T);
    bad |= lo != a || hi != e;
    falls |= e < a;
    put(b, lo, hi);
  }
  if (bad && blockIdx.x == 0 && p.status) atomicCAS(&p.status->code, 0, kStatusInvalidArg);
  if (__syncthreads_or(falls)) {
    if (warp == 0) {
      int top = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane, lo = max(top, running_max(b < p.B ? min(max(p.cu[b], 0), p.T) : 0, lane));
        if (b < p.B) put(b, lo, max(lo, min(max(p.cu[b + 1], 0), p.T)));
        top = __shfl_sync(0xffffffffu, lo, 31);
      }
    }
    __syncthreads();
  }
  auto from = [&](int t) {  // F(t)
    int n = 0;
#pragma unroll 4
    for (int b = lane; b < p.B; b += 32) n += max(n_of[b] - t, 0);
    return (int)__reduce_add_sync(0xffffffffu, n);
  };
  int places = 0;
  for (int b = lane; b < p.B; b += 32) places = max(places, n_of[b]);
  places = __reduce_max_sync(0xffffffffu, places);
  const int n_items = min(from(0), p.cap) * units;  // never more than a CTA keeps entries for
  for (int k = warp; k < kOwnItems; k += warps) {
    const int id = item_id(k, gridDim.x, blockIdx.x);
    if (id >= n_items) break;
    const int e = id / units;
    int lo = 0, hi = places, before = 0;  // F(lo) > e >= F(hi) == before
    while (hi - lo > 1) {
      const int t = (lo + hi) / 2, n = from(t);
      if (n > e) {
        lo = t;
      } else {
        hi = t;
        before = n;
      }
    }
    int left = e - before;
    for (int b = lane; left >= 0 && b - lane < p.B; b += 32) {
      const bool in = b < p.B && n_of[b] > lo;
      const uint32_t all = __ballot_sync(0xffffffffu, in);
      if (in && __popc(all & ((1u << lane) - 1u)) == left) {
        mine[k] = {rows[b].x, rows[b].y, lo * p.step, 0};
        atomicMax(longest, rows[b].y);
      }
      left -= __popc(all);
    }
  }
  return n_items;
}

// F16: q, k, v (and so P) are fp16; otherwise bf16. Persistent: CTA c runs items
// item_id(0, G, c), item_id(1, G, c), ... Barrier phases and ring positions run on
// across items, so that the next item's Q, first K/V tiles and first score products
// overlap the current item's last softmax, PV and output store.
// PACKED: sequences of different lengths packed into one run of rows (see AttnParams::work);
// q, k and v are 3-D maps (channel, head, row), and a slot's rows hold the query heads of a KV
// head side by side (AttnParams::fold): a box of the Q map is 2^fold heads of 128 / 2^fold
// queries, so that short sequences fill the tile and all rows of it share the K/V tiles.
// SPLIT: both slots work on the same queries, slot g on the key tiles j % 2 == g through its own
// K and V stage; the epilogue joins the two results from tensor memory. Twice as many items of
// half the length, for batches whose items are too few to fill the SMs evenly.
template <bool F16, bool PACKED, bool SPLIT>
__global__ void __launch_bounds__(PACKED ? kPackedThreads : kThreads, 1) attn_tc_kernel(const __grid_constant__ AttnParams p) {
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                                   // [slot]: two 64-column halves of 16 KB
  uint8_t* sK = sQ + kSlots * kQBytes;                  // [stage]: two halves of 16 KB
  uint8_t* sV = sK + kKStages * kKVBytes;               // [stage]: two halves of 16 KB
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + kVStages * kKVBytes);
  // q_full, q_empty, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_ready[2][4],
  // o_done[2], o_free[2], drain[2]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 26);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* longest = reinterpret_cast<int*>(bars + 27);  // PACKED: the longest sequence of the CTA's items
  // PACKED: each slot's reference and sum of each row, for the epilogue, and the barriers that
  // announce them
  float2* ml = reinterpret_cast<float2*>(bars + 36);
  auto ml_ready = [&](int g) { return smem_u32(&bars[28 + g]); };
  PackedWork* mine = reinterpret_cast<PackedWork*>(ml + kSlots * kBQ);  // PACKED: the CTA's entries, item by item
  static_assert(27 * 8 + 4 <= 28 * 8, "barriers, the TMEM address, the abort flag, the longest sequence");
  const uint32_t q_full = smem_u32(&bars[0]);
  const uint32_t q_empty = smem_u32(&bars[1]);
  auto k_full = [&](int s) { return smem_u32(&bars[2 + s]); };
  auto k_empty = [&](int s) { return smem_u32(&bars[4 + s]); };
  auto v_full = [&](int s) { return smem_u32(&bars[6 + s]); };
  auto v_empty = [&](int s) { return smem_u32(&bars[8 + s]); };
  auto s_full = [&](int g) { return smem_u32(&bars[10 + g]); };
  // P is released in quarters of 32 keys, each on its own barrier (one phase per tile):
  // the PV steps of a quarter run while the softmax computes the next quarter
  auto p_ready = [&](int g, int q) { return smem_u32(&bars[12 + 4 * g + q]); };
  auto o_done = [&](int g) { return smem_u32(&bars[20 + g]); };
  auto o_free = [&](int g) { return smem_u32(&bars[22 + g]); };
  auto drain = [&](int g) { return smem_u32(&bars[24 + g]); };

  // warp: its role, 0 TMA, 1 and 10 MMA, 2..9 softmax, 12..15 the epilogue of PACKED (11 none)
  const int pw = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warp = !PACKED ? pw : pw < 8 ? pw + 2 : pw == 8 ? 0 : pw == 9 ? 1 : pw;
  const unsigned long long budget = p.wait_ns;
  const int G = gridDim.x, cta = blockIdx.x;
  // one 64-channel half of a Q (or K, V) tile: rows from `row` of a head
  auto load_half = [&](uint32_t dst, const CUtensorMap* m, int half, int head, int row, uint32_t bar) {
    if constexpr (PACKED)
      tma_load_3d(dst, m, 64 * half, head, row, bar);
    else
      tma_load_2d(dst, m, 64 * half, row, bar);
  };

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, kSlots);  // one commit from each slot's MMA issuer after its item's last S
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), SPLIT ? 1 : kSlots);  // one commit from each slot's MMA issuer
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), SPLIT ? 1 : kSlots);
    }
    for (int g = 0; g < kSlots; ++g) {
      mbar_init(s_full(g), 1);
      for (int q = 0; q < 4; ++q) mbar_init(p_ready(g, q), 128);
      mbar_init(o_done(g), 1);
      mbar_init(o_free(g), 128);  // the slot's softmax threads, once they have read O out
      mbar_init(drain(g), 1);
    }
    if constexpr (PACKED) {
      mbar_init(ml_ready(0), 128);
      mbar_init(ml_ready(1), 128);
    }
    *abort_flag = 0;
    if constexpr (PACKED) *longest = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tq);
    tma_prefetch_desc(&p.tk);
    tma_prefetch_desc(&p.tv);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();  // q, k, v (and the cache positions, the key ranges) come from earlier kernels
  const int units = PACKED ? p.H >> p.fold : 1;  // items of a work entry
  int n_items = p.n_items;
  if constexpr (PACKED) {
    if (p.work) {
      n_items = *p.n_work * units;
      for (int k = threadIdx.x; k < kOwnItems; k += blockDim.x) {
        const int id = item_id(k, G, cta);
        if (id < n_items) {
          mine[k] = p.work[id / units];
          atomicMax(longest, mine[k].len);
        }
      }
    } else {
      n_items = own_work(p, sK, units, mine, longest);
      fence_proxy_async_smem();  // the K and V stages served as scratch
    }
    __syncthreads();
  }
  auto entry = [&](int k) {  // the work entry of this CTA's item k
    PackedWork w{};
    if constexpr (PACKED) w = mine[k];
    return w;
  };
  // the ring stage of slot g's tile J (counted over all items) and its phase: the slots share two
  // stages, or (SPLIT) each has one
  auto stage_of = [](int J, int g) { return SPLIT ? g : J % kKStages; };
  auto phase_of = [](int J) { return (uint32_t)(SPLIT ? J & 1 : (J / kKStages) & 1); };
  // quarters (32 keys) of the tile at key n0 that some query of the slot at m0 sees, at least one
  auto quarters = [](const Item& it, int m0, int n0) {
    return min(4, max(1, (min(it.T, m0 + it.tq) - n0 + 31) >> 5));
  };
  // this slot's share of an item's key tiles
  auto my_tiles = [&](const Item& it, int g) { return SPLIT ? (it.n_tiles + 1 - g) / 2 : it.n_tiles; };
  const uint32_t tmem = *tmem_holder;  // S[g] (and P[g] over its first 64 columns): cols 128 g; O[g]: 256 + 128 g
  // What the producer lanes and the MMA lanes have in flight, for the drain after an
  // abort: the ring stages issued (with the parity of their last phase), the last Q
  // load's parity, and whether any MMA was issued.
  uint32_t issued = 0, parity = 0, q_parity = 0;
  bool q_issued = false, mma_issued = false;

  if (PACKED && warp >= 12) {
    if constexpr (PACKED) {
      // ---------------- epilogue: an item's outputs from tensor memory to their rows
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
      const int quarter = pw & 3, r = quarter * 32 + lane;
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 256;
      auto ready = [&](int g, int k) {  // O_g is complete and its rows' sums are known
        const bool ok = mbar_wait(ml_ready(g), k & 1, budget, abort_flag) && mbar_wait(o_done(g), k & 1, budget, abort_flag);
        return __all_sync(0xffffffffu, ok);
      };
      bool failed = false;
      for (int k = 0; !failed; ++k) {
        const int id = item_id(k, G, cta);
        if (id >= n_items) break;
        const Item it = item_of<PACKED, SPLIT>(p, id, entry(k));
#pragma unroll
        for (int g = 0; g < (SPLIT ? 1 : kSlots); ++g) {
          if (!ready(g, k) || (SPLIT && !ready(1, k))) {
            failed = true;
            break;
          }
          __syncwarp();
          tc_fence_after();
          const float2 s0 = ml[g * kBQ + r];
          float w0 = 1.f, w1 = 0.f, l = s0.y;  // the weights of the slots' outputs
          if constexpr (SPLIT) {
            const float2 s1 = ml[kBQ + r];
            const float m = fmaxf(s0.x, s1.x), mu = m == -INFINITY ? 0.f : m;
            w0 = ex2_approx(s0.x - mu);
            w1 = ex2_approx(s1.x - mu);
            l = s0.y * w0 + s1.y * w1;
          }
          // a query sees itself at least: a sum that is NaN (a NaN or infinity in its scores), or 0 (all of
          // them -inf), gives NaN, as the formula does
          const float inv = 1.f / l;
          w0 *= inv;
          w1 *= inv;
          const int query = it.sl[g].m0 + (r >> p.fold), h = it.sl[g].h + (r & ((1 << p.fold) - 1));
          const bool store = it.sl[g].valid && query < it.T;
          uint16_t* const o = static_cast<uint16_t*>(p.o) + (size_t)(it.b + query) * p.o_row + (size_t)h * p.o_head;
          if (__any_sync(0xffffffffu, store)) {
#pragma unroll 1
            for (int c = 0; c < kD; c += 16) {
              float ov[16];
              tmem_ld16(taddr + g * kD + c, ov);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) ov[i] *= w0;
              if (SPLIT && it.n_tiles > 1) {  // O_1 holds something
                float o1[16];
                tmem_ld16(taddr + kD + c, o1);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) ov[i] = fmaf(o1[i], w1, ov[i]);
              }
              if (store) {
                const uint4 a = make_uint4(pack_bf16x2(ov[0], ov[1]), pack_bf16x2(ov[2], ov[3]),
                                           pack_bf16x2(ov[4], ov[5]), pack_bf16x2(ov[6], ov[7]));
                const uint4 b = make_uint4(pack_bf16x2(ov[8], ov[9]), pack_bf16x2(ov[10], ov[11]),
                                           pack_bf16x2(ov[12], ov[13]), pack_bf16x2(ov[14], ov[15]));
                if (p.o_wide) {
                  st_global_32(o + c, a, b);
                } else {
                  reinterpret_cast<uint4*>(o + c)[0] = a;
                  reinterpret_cast<uint4*>(o + c)[1] = b;
                }
              }
              __syncwarp();  // whole again for the next tensor-memory load
            }
          }
          tc_fence_before();
          mbar_arrive(o_free(g));  // O is read out: the next item's first PV may overwrite it
          if constexpr (SPLIT) mbar_arrive(o_free(1));
        }
      }
      if (failed) {
        *abort_flag = 1;
        if (lane == 0) report_timeout(p.status, 0x20 + 4);
      }
    }
  } else if (warp < 2 || warp >= 10) {
  if constexpr (PACKED) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer: each item's Q, then its K tiles through the ring
      bool failed = false;
      int J = 0;  // K tiles issued over all items
      uint32_t used = 0;  // SPLIT: the parity of each stage's next phase
      for (int k = 0; !failed; ++k) {
        const int id = item_id(k, G, cta);
        if (id >= n_items) break;
        const Item it = item_of<PACKED, SPLIT>(p, id, entry(k));
        // the Q buffer is free once both slots' score products of the previous item are done
        if (!mbar_wait(q_empty, (k & 1) ^ 1, budget, abort_flag)) {
          failed = true;
          break;
        }
        mbar_arrive_expect_tx(q_full, (SPLIT ? 1 : kSlots) * kQBytes);
#pragma unroll
        for (int g = 0; g < (SPLIT ? 1 : kSlots); ++g) {
          const int q_row = PACKED ? it.b + it.sl[g].m0 : (it.b * p.H + it.sl[g].h) * p.T + it.sl[g].m0;
          load_half(smem_u32(sQ + g * kQBytes), &p.tq, 0, it.sl[g].h, q_row, q_full);
          load_half(smem_u32(sQ + g * kQBytes + kQSub), &p.tq, 1, it.sl[g].h, q_row, q_full);
        }
        q_issued = true;
        q_parity = k & 1;
        for (int j = 0; j < it.n_tiles; ++j, ++J) {
          const int s = SPLIT ? j & 1 : J % kKStages;
          const uint32_t ph = SPLIT ? (used >> s) & 1 : (J / kKStages) & 1;
          if constexpr (SPLIT) used ^= 1u << s;
          if (!mbar_wait(k_empty(s), ph ^ 1, budget, abort_flag)) {
            failed = true;
            break;
          }
          mbar_arrive_expect_tx(k_full(s), kKVBytes);
          const int row = it.kv_row + (it.t0 + j) * kBK;
          load_half(smem_u32(sK + s * kKVBytes), &p.tk, 0, it.kvh, row, k_full(s));
          load_half(smem_u32(sK + s * kKVBytes + kKVSub), &p.tk, 1, it.kvh, row, k_full(s));
          issued |= 1u << s;
          parity = (parity & ~(1u << s)) | (ph << s);
        }
      }
      if (failed) {  // the loads in flight are drained after the CTA's final barrier
        *abort_flag = 1;
        report_timeout(p.status, 0x20 + 0);
      }
    } else if (lane == 1) {
      // ---------------- TMA producer: the V ring (its own thread, so that K never waits behind V)
      bool failed = false;
      int J = 0;
      uint32_t used = 0;
      for (int k = 0; !failed; ++k) {
        const int id = item_id(k, G, cta);
        if (id >= n_items) break;
        const Item it = item_of<PACKED, SPLIT>(p, id, entry(k));
        for (int j = 0; j < it.n_tiles; ++j, ++J) {
          const int s = SPLIT ? j & 1 : J % kVStages;
          const uint32_t ph = SPLIT ? (used >> s) & 1 : (J / kVStages) & 1;
          if constexpr (SPLIT) used ^= 1u << s;
          if (!mbar_wait(v_empty(s), ph ^ 1, budget, abort_flag)) {
            failed = true;
            break;
          }
          mbar_arrive_expect_tx(v_full(s), kKVBytes);
          const int row = it.kv_row + (it.t0 + j) * kBK;
          load_half(smem_u32(sV + s * kKVBytes), &p.tv, 0, it.kvh, row, v_full(s));
          load_half(smem_u32(sV + s * kKVBytes + kKVSub), &p.tv, 1, it.kvh, row, v_full(s));
          issued |= 1u << s;
          parity = (parity & ~(1u << s)) | (ph << s);
        }
      }
      if (failed) {
        *abort_flag = 1;
        report_timeout(p.status, 0x20 + 3);
      }
    }
  } else if (warp == 1 || warp == 10) {
    if (lane == 0) {
      // ---------------- MMA issuer of slot g (warp 1: slot 0, the last warp: slot 1). Each
      // slot has its own issuing thread, so that a slot whose P is ready never waits
      // behind the other slot's waits and commits: its PV queues on the tensor pipe at once.
      const int g = warp == 1 ? 0 : 1;
      // kind::f16 operand formats: bf16 (1) or fp16 (0) for both A and B
      constexpr uint32_t fmt_clear = F16 ? ~((7u << 7) | (7u << 10)) : ~0u;
      constexpr uint32_t idesc_s = idesc_bf16_f32(kBQ, kBK) & fmt_clear;
      constexpr uint32_t idesc_pv = (idesc_bf16_f32(kBQ, kD) & fmt_clear) | (1u << 16);  // B (V) is MN-major
      // Shared-memory descriptors, built once: a descriptor's start-address field counts
      // 16-byte units, so K step kk of a 128-byte-swizzled operand sits (kk / 4) halves of
      // 16 KB and (kk % 4) 32-byte steps further; V's 16-key steps are 2 KB apart.
      const uint64_t dq = smem_desc_sw128(smem_u32(sQ + (SPLIT ? 0 : g) * kQBytes));
      uint64_t dk[kKStages], dv[kVStages];
#pragma unroll
      for (int st = 0; st < kKStages; ++st) dk[st] = smem_desc_sw128(smem_u32(sK + st * kKVBytes));
#pragma unroll
      for (int st = 0; st < kVStages; ++st) dv[st] = smem_desc_sw128_mn(smem_u32(sV + st * kKVBytes), kKVSub, 1024);
      auto kstep = [](int kk) { return (uint64_t)((kk >> 2) * (kQSub >> 4) + (kk & 3) * 2); };
      const uint32_t s_tmem = tmem + g * kBK, o_tmem = tmem + 256 + g * kD;
      auto issue_s = [&](int J) {  // S of global tile J into the slot's score buffer
        const int s = stage_of(J, g);
        const uint64_t dks = s == 0 ? dk[0] : dk[1];
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) tc_mma_bf16(s_tmem, dq + kstep(kk), dks + kstep(kk), idesc_s, kk > 0 ? 1u : 0u);
        tc_commit(s_full(g));
        tc_commit(k_empty(s));  // this slot is done with the K stage once this S is
        mma_issued = true;
      };
      bool failed = false;
      int J = 0;  // tiles over all items
      for (int k = 0; !failed; ++k) {
        const int id = item_id(k, G, cta);
        if (id >= n_items) break;
        const Item it = item_of<PACKED, SPLIT>(p, id, entry(k));
        if (!mbar_wait(q_full, k & 1, budget, abort_flag)) {
          failed = true;
          break;
        }
        const int n_my = my_tiles(it, g);
        const int m0 = g == 0 ? it.sl[0].m0 : it.sl[1].m0;  // a select, not a run-time index into local memory
        if (n_my > 0) {
          if (!mbar_wait(k_full(stage_of(J, g)), phase_of(J), budget, abort_flag)) {
            failed = true;
            break;
          }
          tc_fence_after();
          issue_s(J);
        }
        if (n_my <= 1) tc_commit(q_empty);  // no further score product of this item reads Q
        for (int j = 0; j < n_my; ++j, ++J) {
          const int nq = PACKED ? quarters(it, m0, (it.t0 + (SPLIT ? 2 * j + g : j)) * kBK) : 4;
          // PV_j as soon as V_j has landed, O is free (the previous item's output read out)
          // and each quarter of P_j is in tensor memory ...
          const int vs = stage_of(J, g);
          if (!mbar_wait(v_full(vs), phase_of(J), budget, abort_flag) ||
              (j == 0 && k >= 1 && !mbar_wait(o_free(g), (k - 1) & 1, budget, abort_flag))) {
            failed = true;
            break;
          }
          const uint64_t dvs = vs == 0 ? dv[0] : dv[1];
          auto pv = [&](int q) {  // a quarter's two K = 16 steps once P's quarter is there
            if (!mbar_wait(p_ready(g, q), J & 1, budget, abort_flag)) return false;
            tc_fence_after();
#pragma unroll
            for (int kk = 2 * q; kk < 2 * q + 2; ++kk)
              tc_mma_ts(o_tmem, s_tmem + kk * 8, dvs + (uint64_t)(kk * (16 * 128 >> 4)), idesc_pv,
                        (j > 0 || kk > 0) ? 1u : 0u);
            return true;
          };
          if (!PACKED || nq == 4) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (!failed && !pv(q)) failed = true;
          } else {
            // the softmax still arrives for a quarter left out, before it arrives for the next
            // tile's first one: no barrier falls a phase behind
            for (int q = 0; q < nq; ++q)
              if (!failed && !pv(q)) failed = true;
          }
          if (failed) break;
          tc_commit(v_empty(vs));  // this slot is done with the V stage once PV_j is
          // ... then S_{j+1}, which overwrites P_j after PV_j has read it (issue order)
          if (j + 1 < n_my) {
            if (!mbar_wait(k_full(stage_of(J + 1, g)), phase_of(J + 1), budget, abort_flag)) {
              failed = true;
              break;
            }
            tc_fence_after();
            issue_s(J + 1);
            if (j + 2 == n_my) tc_commit(q_empty);  // that was the item's last score product
          }
        }
        if (failed) break;
        // An item without key tiles has no PV that waited for the previous item's O to be
        // read out: wait here, so that o_done runs at most one phase ahead of its waiter.
        if (n_my == 0 && k >= 1 && !mbar_wait(o_free(g), (k - 1) & 1, budget, abort_flag)) {
          failed = true;
          break;
        }
        tc_commit(o_done(g));  // every PV of the slot's item is complete
      }
      if (failed) {  // the MMAs in flight are drained after the CTA's final barrier
        *abort_flag = 1;
        report_timeout(p.status, 0x20 + 1);
      }
    }
  }
  } else {
    if constexpr (PACKED) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---------------- softmax / correction / epilogue: slot g, one query row per thread
    const int g = (warp - 2) / 4;
    const int quarter = pw & 3;  // the tensor-memory lanes a warp can reach
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_taddr = tmem + lane_off + g * kBK;
    const uint32_t o_taddr = tmem + lane_off + 256 + g * kD;
    bool failed = false;
    int J = 0;  // tiles over all items
    for (int k = 0; !failed; ++k) {
      const int id = item_id(k, G, cta);
      if (id >= n_items) break;
      const Item it = item_of<PACKED, SPLIT>(p, id, entry(k));
      const Slot me = g == 0 ? it.sl[0] : it.sl[1];  // a select, not a run-time index into local memory
      const int m0 = me.m0;
      const int qi = m0 + (PACKED ? r >> p.fold : r);
      const int n_my = my_tiles(it, g);
      const int qc = min(qi, it.T - 1);
      const int off = it.off, kv_lo = it.kv_lo, kv_hi = it.kv_hi, n_keys = it.n_keys;
      float m_ref = -INFINITY, l = 0.f;
      // whether any of this warp's rows is a query (packed sequences)
      const bool live = me.valid && (!PACKED || m0 + ((quarter * 32) >> p.fold) < it.T);
      // tiles that start in [plain_lo, plain_hi] have no masked score
      const int plain_lo = p.window > 0 ? min(m0 + it.tq - 1, it.T - 1) - p.window + 1 : 0;
      const int plain_hi = live ? min(m0 + 1, it.T) - kBK : -1;
      // Moves the row's reference up to mt where a score passes it by 2^8; PV_{J-1} is done (S_J is
      // ready), so this warp's O rows can be rescaled. Returns the factor.
      auto rescale = [&](float mt, int j) {
        const bool need = mt > m_ref + kRescaleLog2;
        const bool any = __any_sync(0xffffffffu, need);
        float alpha = 1.f;
        if (need) {
          alpha = ex2_approx(m_ref - mt);
          m_ref = mt;
        }
        __syncwarp();
        if (j >= 1 && any) {
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
        return alpha;
      };
      // A masked tile of a packed sequence: keys n0 + c are seen for c in [first, lim]. Quarter by
      // quarter of 32 keys, each read twice from tensor memory (cheap) instead of held, only the
      // nq that some row of the slot sees, the mask as bits that select each score. P's quarter
      // goes to the first 64 columns, over scores that have been read.
      auto masked_tile = [&](int j, int nq, int lim, int first) {
        auto scores = [&](int q4, float (&x)[32]) {
          tmem_ld16(s_taddr + 32 * q4, *reinterpret_cast<float(*)[16]>(&x[0]));
          tmem_ld16(s_taddr + 32 * q4 + 16, *reinterpret_cast<float(*)[16]>(&x[16]));
          const int a = lim - 32 * q4, b = first - 32 * q4;
          const uint32_t bits = (a >= 31 ? ~0u : a < 0 ? 0u : (2u << a) - 1u) & (b <= 0 ? ~0u : b > 31 ? 0u : ~0u << b);
          tc_wait_ld();
          if (!__all_sync(0xffffffffu, bits == ~0u)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(bits & (1u << i))) x[i] = -INFINITY;
          }
        };
        float mraw = -INFINITY;
#pragma unroll 1
        for (int q4 = 0; q4 < nq; ++q4) {
          float x[32];
          scores(q4, x);
          float mx[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = x[i];
#pragma unroll
          for (int c = 4; c < 32; c += 2) mx[(c >> 1) & 3] = fmax3(mx[(c >> 1) & 3], x[c], x[c + 1]);
          mraw = fmaxf(mraw, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
        }
        const float alpha = rescale(mraw * p.sl2, j);
        const float neg_mu = m_ref == -INFINITY ? 0.f : -m_ref;
        const f32x2 sl2x2 = f2_make(p.sl2, p.sl2), mu2 = f2_make(neg_mu, neg_mu);
        f32x2 ls2[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
#pragma unroll 1
        for (int q4 = 0; q4 < nq; ++q4) {
          float x[32], w[16];
          scores(q4, x);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float t0, t1;
            f2_split(f2_fma(f2_make(x[2 * i], x[2 * i + 1]), sl2x2, mu2), t0, t1);
            const float p0 = ex2_approx(t0);
            const float p1 = ex2_approx(t1);
            ls2[i & 1] = f2_add(ls2[i & 1], f2_make(p0, p1));
            w[i] = __uint_as_float(pack2(p0, p1, F16));
          }
          tmem_st16(s_taddr + q4 * 16, w);
          tc_wait_st();
          tc_fence_before();
          mbar_arrive(p_ready(g, q4));
        }
        for (int q4 = nq; q4 < 4; ++q4) mbar_arrive(p_ready(g, q4));
        float ls[4];
        f2_split(ls2[0], ls[0], ls[1]);
        f2_split(ls2[1], ls[2], ls[3]);
        l = l * alpha + ((ls[0] + ls[1]) + (ls[2] + ls[3]));
      };
      for (int j = 0; j < n_my; ++j, ++J) {
        // what needs no score is known before the wait for them
        const int n0 = (it.t0 + (SPLIT ? 2 * j + g : j)) * kBK;
        const bool plain = PACKED && n0 >= plain_lo && n0 <= plain_hi;
        // The slots take turns (slot 0 tile J, slot 1 tile J, slot 0 tile J + 1, ...): each
        // softmax runs alone on the SM's exponential units while the tensor core works on
        // the other slot's PV and next scores. Slot 1 starts tile J once slot 0's P_J is
        // written, slot 0 starts tile J + 1 once slot 1's P_J is. (At their own pace: see kTurnKeys.)
        if ((!PACKED || (!SPLIT && *static_cast<volatile int*>(longest) > kTurnKeys)) && (g == 1 || J >= 1)) {
          if (!__all_sync(0xffffffffu, mbar_wait(p_ready(1 - g, 3), (g == 1 ? J : J - 1) & 1, budget, abort_flag))) {
            failed = true;
            break;
          }
        }
        // warp-uniform: every lane waits, the warp gives up together. S_J ready also means
        // that this slot's PV_{J-1} is done: O is stable and the P buffer free
        if (!__all_sync(0xffffffffu, mbar_wait(s_full(g), J & 1, budget, abort_flag))) {
          failed = true;
          break;
        }
        __syncwarp();
        tc_fence_after();
        if (PACKED && !plain) {
          const int nq = quarters(it, m0, n0);
          if (n0 + kBK > n_keys && nq * 32 > n_keys - n0) {
            // V rows behind the sequence belong to another one, or to none: zero those that P = 0
            // will meet (see below). The 8 chunks of a row in an order that starts at the row's
            // number: eight neighbouring rows' stores go to all banks.
            const int vs = stage_of(J, g);
            if (!__all_sync(0xffffffffu, mbar_wait(v_full(vs), phase_of(J), budget, abort_flag))) {
              failed = true;
              break;
            }
            if (r >= n_keys - n0 && r < nq * 32) {
              uint8_t* vrow = sV + vs * kKVBytes + r * 128;
#pragma unroll
              for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int hb = 0; hb < 2; ++hb)
                  *reinterpret_cast<uint4*>(vrow + hb * kKVSub + ((c + r) & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();  // whole again for the tensor-memory loads, which want that
          }
          if (!live) {  // nobody reads these rows: whatever the score buffer holds may stand for P
            tc_fence_before();
#pragma unroll
            for (int q = 0; q < 4; ++q) mbar_arrive(p_ready(g, q));
            continue;
          }
          masked_tile(j, nq, qc - n0, p.window > 0 ? qc - n0 - p.window + 1 : -kBK);
          continue;
        }
        float x[kBK];
#pragma unroll
        for (int c = 0; c < kBK; c += 16) tmem_ld16(s_taddr + c, *reinterpret_cast<float(*)[16]>(&x[c]));
        tc_wait_ld();
        // raw scores: masked entries become -inf (tiles on the diagonal, past the last key,
        // before the first visible key, or before the window)
        if (!PACKED && ((n0 + kBK - 1 > off + m0) || (n0 + kBK > kv_hi) || n0 < kv_lo ||
            (p.window > 0 && n0 < off + min(m0 + it.tq - 1, it.T - 1) - p.window + 1))) {
          const int causal = off + qc - n0;                    // keys n0 + c with c <= causal are not ahead
          const int lim = min(causal, kv_hi - 1 - n0);         // ... nor padding after the run
          const int first = max(p.window > 0 ? causal - p.window + 1 : -kBK, kv_lo - n0);  // c >= first
#pragma unroll
          for (int c = 0; c < kBK; ++c)
            if (c > lim || c < first) x[c] = -INFINITY;
        }
        float mx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = x[i];
#pragma unroll
        for (int c = 8; c < kBK; c += 2) mx[(c >> 1) & 7] = fmax3(mx[(c >> 1) & 7], x[c], x[c + 1]);
        const float mraw = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                 fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
        const float mt = mraw * p.sl2;  // the scale is positive: the max commutes with it
        const bool need = mt > m_ref + kRescaleLog2;
        const bool any = __any_sync(0xffffffffu, need);
        float alpha = 1.f;
        if (need) {
          alpha = ex2_approx(m_ref - mt);
          m_ref = mt;
        }
        const float neg_mu = m_ref == -INFINITY ? 0.f : -m_ref;
        if (j >= 1 && any) {  // PV_{J-1} is done (see above): rescale this warp's O rows
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
        if (!PACKED && n0 + kBK > n_keys) {
          // V rows past the item's last key may hold anything (unused cache slots): zero them,
          // so that P = 0 meets finite values, once the tile has landed. Both slots write the
          // same zeros, each before its own p_ready (the fence below), as either slot's PV
          // may run first
          const int vs = J % kVStages;
          if (!__all_sync(0xffffffffu, mbar_wait(v_full(vs), (J / kVStages) & 1, budget, abort_flag))) {
            failed = true;
            break;
          }
          if (r >= n_keys - n0) {
            uint8_t* vrow = sV + vs * kKVBytes + r * 128;
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
              for (int c16 = 0; c16 < 8; ++c16) *reinterpret_cast<uint4*>(vrow + hb * kKVSub + c16 * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        // P row r into tensor memory over the scores it came from: 64 columns of element
        // pairs (keys 2c, 2c + 1 in column c), a quarter (16 columns) at a time. Keys 2c and
        // 2c + 1 go as one packed pair through the scale and shift and the row sum. A
        // quarter is released to the PV steps once its store has landed, which the warp
        // waits for only after computing the next quarter.
        const f32x2 sl2x2 = f2_make(p.sl2, p.sl2), mu2 = f2_make(neg_mu, neg_mu);
        f32x2 ls2[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
        float w[2][16];
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = q4 * 32 + 2 * i;
            float t0, t1;
            f2_split(f2_fma(f2_make(x[c], x[c + 1]), sl2x2, mu2), t0, t1);
            const float p0 = ex2_approx(t0);
            const float p1 = ex2_approx(t1);
            ls2[i & 1] = f2_add(ls2[i & 1], f2_make(p0, p1));
            w[q4 & 1][i] = __uint_as_float(pack2(p0, p1, F16));
          }
          if (q4 >= 1) {
            tc_wait_st();  // quarter q4 - 1 of P (and a rescaled O) in tensor memory before its PV steps
            tc_fence_before();
            mbar_arrive(p_ready(g, q4 - 1));
          }
          tmem_st16(s_taddr + q4 * 16, w[q4 & 1]);
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(p_ready(g, 3));
        float ls[4];
        f2_split(ls2[0], ls[0], ls[1]);
        f2_split(ls2[1], ls[2], ls[3]);
        l = l * alpha + ((ls[0] + ls[1]) + (ls[2] + ls[3]));
      }
      if (failed) break;
      if constexpr (PACKED) {
        // the epilogue takes over; it has read this slot's last states once it frees its O
        if (k >= 1 && !__all_sync(0xffffffffu, mbar_wait(o_free(g), (k - 1) & 1, budget, abort_flag))) {
          failed = true;
          break;
        }
        ml[g * kBQ + r] = make_float2(m_ref, l);
        mbar_arrive(ml_ready(g));
        continue;
      }
      // the slot's last PV of this item is complete (every item commits, with tiles or not)
      if (!__all_sync(0xffffffffu, mbar_wait(o_done(g), k & 1, budget, abort_flag))) {
        failed = true;
        break;
      }
      __syncwarp();
      tc_fence_after();
      const bool seen = l > 0.f;  // false: a padding query that sees no key (its output is 0)
      const float inv = seen ? 1.f / l : 0.f;
      const size_t orow_i = (((size_t)it.b * p.T + qi) * p.H + me.h) * kD;
      uint16_t* orow = static_cast<uint16_t*>(p.o) + orow_i;
      const bool of16 = p.o_f16 != 0;
      const bool store = me.valid && qi < it.T;
      auto pack16 = [](const float (&v)[16], bool f16, uint4& w0, uint4& w1) {
        w0 = make_uint4(pack2(v[0], v[1], f16), pack2(v[2], v[3], f16), pack2(v[4], v[5], f16),
                        pack2(v[6], v[7], f16));
        w1 = make_uint4(pack2(v[8], v[9], f16), pack2(v[10], v[11], f16), pack2(v[12], v[13], f16),
                        pack2(v[14], v[15], f16));
      };
#pragma unroll 1
      for (int c = 0; c < kD; c += 16) {
        float ov[16];
        tmem_ld16(o_taddr + c, ov);
        tc_wait_ld();
        if (store) {
#pragma unroll
          for (int i = 0; i < 16; ++i) ov[i] = seen ? ov[i] * inv : 0.f;
          uint4 w0, w1;
          if (p.ungated) {  // the head outputs before the gate (bf16)
            pack16(ov, false, w0, w1);
            reinterpret_cast<uint4*>(p.ungated + orow_i + c)[0] = w0;
            reinterpret_cast<uint4*>(p.ungated + orow_i + c)[1] = w1;
          }
          if (p.gate) {
            const uint4* g4 = reinterpret_cast<const uint4*>(p.gate + orow_i + c);
            const uint4 ga = g4[0], gb = g4[1];
            const uint32_t gw[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 gf = __half22float2(*reinterpret_cast<const __half2*>(&gw[i]));
              ov[2 * i] *= gf.x;
              ov[2 * i + 1] *= gf.y;
            }
          }
          pack16(ov, of16, w0, w1);
          reinterpret_cast<uint4*>(orow + c)[0] = w0;
          reinterpret_cast<uint4*>(orow + c)[1] = w1;
        }
      }
      tc_fence_before();
      mbar_arrive(o_free(g));  // O is read out: the next item's first PV may overwrite it
    }
    if (failed) {
      *abort_flag = 1;
      if (lane == 0) report_timeout(p.status, 0x20 + 2);
    }
  }

  tc_fence_before();
  __syncthreads();
  // Every role has stopped issuing. After an abort (a wait that ran out anywhere in
  // the CTA), copies and MMAs that no role waited for may still be in flight: they
  // complete before TMEM is freed and the CTA exits. Every thread reads the same flag.
  if (*abort_flag) {
    volatile int never = 0;
    if (warp == 0 && lane == 0) {
      if (q_issued) mbar_wait(q_full, q_parity, kDrainNs, &never);
      for (int s = 0; s < kKStages; ++s)
        if (issued & (1u << s)) mbar_wait(k_full(s), (parity >> s) & 1, kDrainNs, &never);
    } else if (warp == 0 && lane == 1) {
      for (int s = 0; s < kVStages; ++s)
        if (issued & (1u << s)) mbar_wait(v_full(s), (parity >> s) & 1, kDrainNs, &never);
    } else if ((warp == 1 || warp == 10) && lane == 0 && mma_issued) {
      const int g = warp == 1 ? 0 : 1;
      tc_commit(drain(g));
      mbar_wait(drain(g), 0, kDrainNs, &never);
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_attn_prefill_tc(const void* q, const void* k, const void* v, void* o, int B, int H, int Hkv, int T,
                                   int d, bool f16, bool o_f16, DevStatus* st, unsigned long long wait_ns,
                                   cudaStream_t s, const char** why, const int* q_off, int kv_stride,
                                   const AttnOpts& opt) {
  if (d != kD) {
    *why = "tcgen05 attention: head_dim must be 128";
    return cudaErrorInvalidValue;
  }
  if (B <= 0 || T <= 0) return cudaSuccess;
  if (kv_stride <= 0) kv_stride = T;
  if (!q_off && kv_stride != T) {
    *why = "tcgen05 attention: K/V rows per head differ from T only with cache positions";
    return cudaErrorInvalidValue;
  }
  AttnParams p;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  if (!make_tma_2d_16b(&p.tq, q, B * H * T, kD, kBQ, f16) ||
      !make_tma_2d_16b(&p.tk, k, B * Hkv * kv_stride, kD, kBK, f16) ||
      !make_tma_2d_16b(&p.tv, v, B * Hkv * kv_stride, kD, kBK, f16)) {
    *why = "cuTensorMapEncodeTiled failed for q/k/v";
    return cudaErrorInvalidValue;
  }
  p.o = o;
  p.o_f16 = o_f16 ? 1 : 0;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.T = T;
  p.kv_stride = kv_stride;
  p.q_off = q_off;
  p.window = opt.window > 0 ? opt.window : 0;
  p.key_range = opt.key_range;
  p.gate = static_cast<const __half*>(opt.gate);
  p.ungated = static_cast<__nv_bfloat16*>(opt.ungated);
  p.n_qtiles = (T + kBQ - 1) / kBQ;
  p.head_pairs = (H / Hkv) % 2 == 0 ? 1 : 0;
  p.n_items = p.head_pairs ? B * (H / 2) * p.n_qtiles : B * H * ((p.n_qtiles + 1) / 2);
  p.sl2 = kLog2e / sqrtf((float)kD);
  p.status = st;
  p.wait_ns = wait_ns;
  static std::atomic<unsigned long long> configured[2];  // per instantiation, one bit per device
  cudaError_t ce = f16 ? set_smem_limit_once(reinterpret_cast<const void*>(attn_tc_kernel<true, false, false>), kSmem, configured[1])
                       : set_smem_limit_once(reinterpret_cast<const void*>(attn_tc_kernel<false, false, false>), kSmem, configured[0]);
  if (ce != cudaSuccess) return ce;
  // persistent: one CTA per SM (at most one per item) walks the items
  int dev = 0, sms = 0;
  ce = cudaGetDevice(&dev);
  if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (ce != cudaSuccess) return ce;
  const int grid = std::min(p.n_items, sms);
  if (f16)
    launch_pdl(attn_tc_kernel<true, false, false>, grid, kThreads, kSmem, s, p);
  else
    launch_pdl(attn_tc_kernel<false, false, false>, grid, kThreads, kSmem, s, p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ packed sequences

namespace {

// 3-D TMA map over bf16 head rows: boxes of 64 channels x box_heads x box_rows rows, 128-byte
// swizzle, zero fill out of bounds. Strides in multiples of 8 elements.
bool make_tma_heads_bf16(CUtensorMap* m, const HeadRows& x, int rows, int heads, int d, int box_heads, int box_rows) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr)
                                                                : nullptr;
  }();
  if (!encode) return false;
  // the stride of a dimension of one element is never used, but has to be a valid one
  const long long head = heads > 1 ? x.head : d, row = rows > 1 ? x.row : (long long)d * heads;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)head * 2, (cuuint64_t)row * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, x.ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 4096;
// The work list of packed sequences, heaviest first: an entry per `step` queries, ordered by its
// place in its sequence, which its key count grows with. One CTA counts the entries of each
// place, sums the counts from the far places down, and deals the entries out; the order within
// a place does not matter (items are independent, so no result depends on it). A cu that is not
// valid is read as by own_work, 1024 sequences at a time.
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const int* __restrict__ cu, int B, int rows, int step,
                                                                   int cap, PackedWork* __restrict__ work,
                                                                   int* __restrict__ n_work, DevStatus* st) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int count[kPlanBins];
  __shared__ int warp_sums[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int places = (rows + step - 1) / step;
  const int per_bin = (places + kPlanBins - 1) / kPlanBins;
  for (int i = tid; i < kPlanBins; i += kPlanThreads) count[i] = 0;
  __syncthreads();
  bool bad = false, falls = false;
  for (int b = tid; b < B; b += kPlanThreads) falls |= cu[b + 1] < cu[b];
  falls = __syncthreads_or(falls);
  for (int pass = 0; pass < 2; ++pass) {
    int top = 0;  // of the sequences before (a list that falls)
    for (long long base = 0; base < B; base += kPlanThreads) {  // 32 sequences a warp, one after another
      const long long b0 = base + 32 * warp, b = b0 + lane;
      const int a = b < B ? cu[b] : 0, e = b < B ? cu[b + 1] : 0;
      int lo = min(max(a, 0), rows);
      if (falls) {
        lo = max(top, running_max(lo, lane));
        if (lane == 31) warp_sums[warp] = lo;
        __syncthreads();
        for (int w = 0; w < kPlanThreads / 32; ++w) {
          if (w < warp) lo = max(lo, warp_sums[w]);
          top = max(top, warp_sums[w]);
        }
        __syncthreads();
      }
      const int len = min(max(e, lo), rows) - lo;
      bad |= b < B && (lo != a || lo + len != e);
      const int n = (len + step - 1) / step;
      const int seqs = (int)min(32ll, B - b0);  // none when it is not positive
      for (int i = 0; i < seqs; ++i) {
        const int row0 = __shfl_sync(0xffffffffu, lo, i), its = __shfl_sync(0xffffffffu, len, i);
        const int last = __shfl_sync(0xffffffffu, n, i);
        for (int t = lane; t < last; t += 32) {
          const int at = atomicAdd(&count[t / per_bin], 1);
          if (pass == 1 && (unsigned)at < (unsigned)cap) work[at] = {row0, its, t * step, 0};
        }
      }
    }
    __syncthreads();
    if (pass == 0) {
      // count[i] := the entries of all farther places (an exclusive sum from the far end)
      constexpr int kPer = kPlanBins / kPlanThreads;
      int v[kPer], sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        v[i] = count[kPlanBins - 1 - (tid * kPer + i)];
        sum += v[i];
      }
      int run = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += u;
      }
      if (lane == 31) warp_sums[warp] = run;
      __syncthreads();
      int before = 0;
      for (int w = 0; w < warp; ++w) before += warp_sums[w];
      if (tid == kPlanThreads - 1) *n_work = min(before + run, cap);
      int x = before + run - sum;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        count[kPlanBins - 1 - (tid * kPer + i)] = x;
        x += v[i];
      }
      __syncthreads();
    }
  }
  if (bad && st) atomicCAS(&st->code, 0, kStatusInvalidArg);
}

constexpr size_t kPackedHead = 256;  // bytes before the work list: its length

// How a packed batch is cut into items, from what the host knows of it.
struct PackedPlan {
  int fold, step, units, cap, grid;
  bool split, own;  // own: every CTA makes the work list itself
};
PackedPlan packed_plan(int rows, int B, int H, int Hkv, int num_sms) {
  PackedPlan p{};
  while (p.fold < 4 && (H / Hkv) % (2 << p.fold) == 0) ++p.fold;
  p.units = H >> p.fold;
  const int tq = kBQ >> p.fold;
  // Two query tiles an item; split when that leaves SMs idle, or with one long item each: below
  // 5/4 items per SM (8 heads over 2: 2000 queries 34.7 -> 25.0 us, 4000 61.9 -> 43.4; above it
  // the split's shorter items do not make up for its second read of K and V: 8000 115 -> 132).
  p.split = 4 * (long long)(rows / (2 * tq) + B) * p.units < 5 * num_sms;
  p.step = p.split ? tq : 2 * tq;
  p.cap = rows / p.step + std::min(B, rows);  // a sequence's rows are its own, and an empty one has no entry
  // one CTA per SM, more only where a CTA would have more items than it keeps entries for
  const long long most = (long long)p.cap * p.units;
  p.grid = (int)std::max(std::min<long long>(most, num_sms), (most + kOwnItems - 1) / kOwnItems);
  // The list costs its sums in every CTA, or a launch of its own before the attention: 48 turns of
  // 10 to 200 queries 25.2 us, 27.5 with that launch; 2000 sequences of 10 (8 heads over 2) 81 and
  // 113; 4000 of 60 (32 over 8) 1479 and 1405.
  p.own = B <= kOwnSeqs;
  return p;
}

}  // namespace

size_t attn_packed_ws_bytes(int rows, int B, int H, int Hkv, int num_sms) {
  if (rows <= 0 || B <= 0) return 0;
  const PackedPlan pl = packed_plan(rows, B, H, Hkv, num_sms);
  return pl.own ? 0 : kPackedHead + (size_t)pl.cap * sizeof(PackedWork);
}

cudaError_t launch_attn_packed(const HeadRows& q, const HeadRows& k, const HeadRows& v, const HeadRows& o, int rows,
                               const int* cu, int B, int H, int Hkv, int d, int window, void* ws, int num_sms,
                               DevStatus* st, unsigned long long wait_ns, cudaStream_t s, const char** why) {
  if (d != kD) {
    *why = "tcgen05 attention: head_dim must be 128";
    return cudaErrorInvalidValue;
  }
  if (B <= 0 || rows <= 0) return cudaSuccess;
  AttnParams p;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  const PackedPlan pl = packed_plan(rows, B, H, Hkv, num_sms);
  p.fold = pl.fold;
  const int tq = kBQ >> p.fold;
  if (!make_tma_heads_bf16(&p.tq, q, rows, H, kD, 1 << p.fold, tq) ||
      !make_tma_heads_bf16(&p.tk, k, rows, Hkv, kD, 1, kBK) || !make_tma_heads_bf16(&p.tv, v, rows, Hkv, kD, 1, kBK)) {
    *why = "cuTensorMapEncodeTiled failed for q/k/v";
    return cudaErrorInvalidValue;
  }
  p.o = o.ptr;
  p.o_row = o.row;
  p.o_head = o.head;
  p.o_wide = reinterpret_cast<uintptr_t>(o.ptr) % 32 == 0 && (rows == 1 || o.row % 16 == 0) && (H == 1 || o.head % 16 == 0);
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.T = rows;
  p.window = window > 0 ? window : 0;
  p.sl2 = kLog2e / sqrtf((float)kD);
  p.status = st;
  p.wait_ns = wait_ns;
  p.cu = cu;
  p.step = pl.step;
  p.cap = pl.cap;
  if (!pl.own) {
    p.n_work = static_cast<int*>(ws);
    p.work = reinterpret_cast<PackedWork*>(static_cast<uint8_t*>(ws) + kPackedHead);
  }
  const int split = pl.split ? 1 : 0;
  const auto kernel = split ? attn_tc_kernel<false, true, true> : attn_tc_kernel<false, true, false>;
  static std::atomic<unsigned long long> configured[2];
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(kernel), kSmemPacked, configured[split]);
  if (e != cudaSuccess) return e;
  // the kernel moves registers between its warpgroups: the launch has to bring as many as it
  // gives out, or the wait for them would not end
  static std::atomic<int> regs[2];
  if (regs[split].load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, reinterpret_cast<const void*>(kernel));
    if (e != cudaSuccess) return e;
    regs[split].store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs[split].load(std::memory_order_relaxed) < kLaunchRegs) {
    *why = "packed attention: the kernel was built with fewer registers than it redistributes";
    return cudaErrorLaunchOutOfResources;
  }
  if (!pl.own) {
    e = launch_pdl(packed_plan_kernel, 1, kPlanThreads, 0, s, cu, B, rows, pl.step, pl.cap,
                   const_cast<PackedWork*>(p.work), static_cast<int*>(ws), st);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, pl.grid, kPackedThreads, kSmemPacked, s, p);
}

}  // namespace blk

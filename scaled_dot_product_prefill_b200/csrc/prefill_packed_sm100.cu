// prefill_packed_sm100.cu -- bf16 attention prefill of packed sequences on the fifth-generation tensor cores.
//
// What is computed: for sequences of different lengths that lie one after
// another in [tokens, heads, D] buffers, O = softmax(Q K^T * scale + mask) V per
// sequence and query head, with the masks and the GQA head map of the public
// header; K and V packed likewise, or in the paged cache.  As in the dense
// kernel (prefill_sm100.cu), whose softmax arithmetic this one repeats step by
// step (equal lengths give equal bits, short of RUNS), the scores stay on the SM and an
// online softmax visits the keys a tile at a time.
//
// How.  A work item is 2 query tiles of one head block.  A query tile is
// 128 / 2^s tokens x 2^s query heads of one kv head (2^s: the largest power of
// two that divides the group), one four-dimensional TMA box.  A sequence of n
// tokens then fills n * 2^s rows of its last tile instead of n, and each K/V
// tile serves 2^s heads at once.  The kernel is persistent, one CTA per SM:
//   warps 0-3, 4-7  softmax of query tiles 0 and 1 (thread t owns row t)
//   warp 8          TMA producer: Q of each item, and a ring of stages
//   warp 9          MMA issuer (one thread) and tensor-memory owner
//   warp 10         scheduler: makes the items (the lengths are on the device)
//   warp 11         zeroes the V rows behind a sequence
// Items.  The scheduler walks the query blocks of all sequences from the
// costliest (last visible key farthest) down, deals them out in a snake over
// the CTAs, and hands each to the other roles through a ring in shared memory.
// Nothing is stored in memory and no other launch precedes this one.
// Stages, D = 128.  The key tiles of all of a CTA's items form one stream.
// Stage g holds V of tile g - 1 and K of tile g, because the MMA thread uses
// them together: P V of one tile, then S of the next, for query tile 0 and then
// 1.  One full and one empty barrier serve two loads, and the next item's first
// K comes with the last V of the item before.  Within a long item that thread never
// waits for a P: a key tile of the pair takes it 2980 cycles, 2048 of them the tensor
// pipe's own (32 MMAs of 64) and the rest its waits (about 100 each, also where
// the phase is complete) and commits (40 to 60); with a barrier for each load it took
// 5 % longer.  The softmax chain of a tile is nearly as long, and an item costs 4.1 us
// beside its tiles (first softmax, last P V, output): tensor pipe 53 % active on
// four prompts of 1733 to 4096 tokens, where 2048 of 2980 would be 69 %.
// At D = 64 a stage is a single K or V tile: S_i(j + 1) runs ahead of P_i(j) V_j, and
// would only wait longer for a V that it does not need (6 % on items of 2 key tiles).
// Tail.  The last key tile of a sequence is followed in memory by the next
// sequence's rows (or by whatever the page holds).  Their scores are masked
// like any others; the V rows are zeroed in shared memory (0 * NaN is NaN) by
// warp 11 while the softmax of that tile runs.
// Output.  64 columns at a time through shared memory, so that 8 lanes write a
// row's 128 bytes together: one thread a row would touch 32 lines with every
// store (4 % of the time of a batch of 1 to 1024-token prompts).
//
// Split.  With so few items that each could have several SMs (a few new tokens
// of a few sequences), the key tiles of an item are dealt to 2 to 16 items
// (SPLIT kernels; packed_splits has the rule and what it measured; at D = 64 they spill one
// 8-byte value, read back 80 times in the code).  Each writes its
// normalised fp32 output rows and base-2 log-sum-exps to the caller's workspace,
// and prefill_packed_combine_kernel joins them.
//
// Runs.  The tensor core aligns 16 products with their sum and drops what lies below 2^-25 of it (as
// measured: a product of 1 is lost beside 2^26, not beside 2^25).  Weights of like size and
// values of one sign so lose 2e-4 of the sum over 2^16 keys, 7e-4 over 2^18, 4e-3 over 2^20, 2 % over
// 2^22, 35 % over 2^26.  Where buffers and window allow a row more than kOneRun key tiles, the
// RUNS kernels begin a new sum every kRun tiles, and the softmax threads add the old one, and
// their sum of weights, to fp32 totals in local memory: 2e-4 at any length.  They are kernels of their
// own because the others are slower for it: 4 % on a batch of 1 to 1024-token prompts, 3 % on
// long ones.
//
// Tensor memory (512 columns x 128 lanes, fp32), as in the dense kernel:
//   D = 128: S_i at 128 i, P_i (bf16) over its first half, O_i at 256 + 128 i
//   D = 64:  S_i at 128 i, P_i at 256 + 64 i, O_i at 384 + 64 i; S_i(j + 1)
//            is computed while the softmax of tile j runs
#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <pthread.h>

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int BM = 128;          // query rows per tile
constexpr int BN = 128;          // keys per tile
constexpr int NQ = 2;            // query tiles per work item
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kSchedWarp = 10;
constexpr int kTailWarp = 11;
constexpr float kTau = 8.0f;     // lazy-rescale threshold, log2 units
constexpr int kRun = 512;        // RUNS: key tiles whose P V one accumulation sums (a power of two)
constexpr int kOneRun = 2048;    // key tiles that need no runs
constexpr int kItemRing = 4;           // items handed out ahead
constexpr int kItemConsumers = 11;     // TMA warp, MMA thread, V-zeroing warp, 8 softmax warps

template <int D>
struct Cfg {
  static constexpr int THREADS = 384;
  static constexpr int SOFTMAX_REGS = 208;            // the dense kernel's register split
  static constexpr int PRODUCER_REGS = 88;
  static constexpr int KATOMS = D / 64;               // 64-column (128-byte) swizzle atoms
  static constexpr int TILE_BYTES = BN * D * 2;       // one K or V tile
  static constexpr int Q_BYTES = BM * D * 2;          // one query tile
  static constexpr int QBUF = (D == 128) ? 1 : 2;     // query buffers (items in flight)
  static constexpr int STAGES = (D == 128) ? 2 : 8;
  static constexpr int STAGE_BYTES = (D == 128) ? 2 * TILE_BYTES : TILE_BYTES;   // V, then K; one tile
  static constexpr bool SEP_P = (D == 64);            // P has tensor memory of its own
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t S_COL = 0;                // + BN * i
  static constexpr uint32_t P_COL = SEP_P ? 256 : 0;  // + P_STRIDE * i
  static constexpr uint32_t P_STRIDE = SEP_P ? 64 : BN;
  static constexpr uint32_t O_COL = SEP_P ? 384 : NQ * BN;  // + D * i
  static constexpr int CONTROL = 1024;                // barriers and the item ring
  static constexpr int OUT_BYTES = 8 * 4096;          // a softmax warp's 32 output rows x 64 columns
  static constexpr size_t SMEM = 1024 /*align*/ + QBUF * NQ * Q_BYTES + STAGES * STAGE_BYTES + CONTROL + OUT_BYTES;
};

struct Params {
  int B, Hq, Hkv, Tq, Tk, causal, window;
  int n_items;              // what sequences that do not overlap can make at most
  float scale_log2;
  __nv_bfloat16* out;
  long long out_stride;     // elements from one token of out to the next
  float* lse;               // [Tq, Hq] natural-log log-sum-exp, or null
  unsigned int* err;
  const int32_t* cu_q;      // [B + 1]: sequence b owns rows [cu_q[b], cu_q[b + 1]) of q and out
  const int32_t* cu_k;      // the same for k and v (not PAGED)
  int pack_log2;            // s: 2^s query heads of a kv head share a tile
  int head_blocks;          // Hq >> s
  // PAGED: K and V come from [num_pages, Hkv, page_size, D] pools through page_table [B, max_pages];
  // sequence b has seq_lens[b] keys (at most max_seq_len)
  const int32_t* page_table;
  const int32_t* seq_lens;
  int page_size, box_rows, max_pages, num_pages, max_seq_len;
  // SPLIT: the items an item's key tiles are dealt to, and their results
  int splits;
  float* ws_o;              // [splits, Tq, Hq, D]
  float* ws_lse;            // [splits, Tq, Hq], log2 units
};

struct Item {
  int b;                // sequence (SPLIT: in the low 16 bits, above them the part); -1 ends the list
  int hb, g;            // head block (heads [hb << s, (hb + 1) << s)) and its kv head
  int row0, end;        // tokens [row0, end) of the sequence
  int q_base, k_base;   // the sequence's first rows
  int sq, sk;           // its queries and keys
  int lo[NQ], hi[NQ];   // key-tile range per query tile (empty if hi <= lo)
  int lo_all, hi_all;   // union; empty (hi_all <= lo_all) if no row sees a key
};

// One sequence of a packed batch: first rows and lengths, cut to the buffers.
// A cumulative length that decreases or passes the buffer is reported, and
// never leads outside it.
struct PackedSpan {
  int q0, sq, k0, sk;
};

template <bool PAGED>
__device__ __forceinline__ PackedSpan packed_span(const Params& p, int b) {
  PackedSpan s;
  const int a = p.cu_q[b], e = p.cu_q[b + 1];
  bool bad = a < 0 || e < a || e > p.Tq;
  s.q0 = min(max(a, 0), p.Tq);
  s.sq = min(max(e, s.q0), p.Tq) - s.q0;
  if constexpr (PAGED) {
    const int L = p.seq_lens[b];
    const long long room = static_cast<long long>(p.max_pages) * p.page_size;
    const int cap = room < p.max_seq_len ? static_cast<int>(room) : p.max_seq_len;
    bad |= L > cap;
    s.k0 = 0;
    s.sk = max(0, min(L, cap));
  } else {
    const int ka = p.cu_k[b], ke = p.cu_k[b + 1];
    bad |= ka < 0 || ke < ka || ke > p.Tk;
    s.k0 = min(max(ka, 0), p.Tk);
    s.sk = min(max(ke, s.k0), p.Tk) - s.k0;
  }
  if (bad) record_error(p.err, ATTN_ERRBIT_BADPAGE);
  return s;
}

// How a sequence's query blocks (of 2^tb_log2 tokens) spread over cost steps.
// Causal: block qb ends at step qb + o, o = ceil((sk - sq) / block), whose last
// visible key lies in key block step - 1; blocks that see no key or only
// the first block's share step 0.  Not causal: all blocks cost the same, one
// step by the number of keys.  A level is 2^shift steps.
struct PackedSteps {
  int o, nb;
};

__device__ __forceinline__ PackedSteps packed_steps(const Params& p, const PackedSpan& s, int tb_log2) {
  const int up = (1 << tb_log2) - 1;
  PackedSteps l;
  l.nb = (s.sq >> tb_log2) + ((s.sq & up) ? 1 : 0);
  l.o = p.causal ? ((s.sk - s.sq) >> tb_log2) + (((s.sk - s.sq) & up) ? 1 : 0)
                 : (s.sk >> tb_log2) + ((s.sk & up) ? 1 : 0);
  return l;
}

// The sequence's highest step (-1: no blocks), and its lowest.  o + nb <= 2^30 + 1: no sum here wraps.
__device__ __forceinline__ int top_step(const PackedSteps& l, int causal) {
  return l.nb == 0 ? -1 : causal ? max(l.o + l.nb - 1, 0) : l.o;
}
__device__ __forceinline__ int low_step(const PackedSteps& l) { return max(l.o, 0); }

// Blocks of the sequence at level q >= 0, and its next level below q (-1: none).
__device__ __forceinline__ int blocks_at(const PackedSteps& l, int causal, int q, int shift) {
  if (!causal) return q == l.o >> shift ? l.nb : 0;
  const int from = q << shift, to = from + (1 << shift);   // steps of the level
  if (q == 0) return min(max(to - l.o, 0), l.nb);
  return max(min(to, l.o + l.nb) - max(from, l.o), 0);
}
__device__ __forceinline__ int next_level(const PackedSteps& l, int causal, int q, int shift) {
  if (l.nb == 0) return -1;
  const int n = min(q - 1, top_step(l, causal) >> shift);
  return n >= low_step(l) >> shift ? n : -1;
}
// The j-th block of the sequence at level q, the costliest first.
__device__ __forceinline__ int block_of(const PackedSteps& l, int causal, int q, int shift, int j) {
  if (!causal) return j;
  return min((q + 1) << shift, l.o + l.nb) - 1 - l.o - j;
}

// A wait for another role's part in a tile (the others are renewed by progress).  Microseconds; but the last V of
// an item comes once the scheduler knows the next item, and it may have many without keys to pass over:
// some half a second of 65535 sequences with 1024 kv heads.
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* err) {
  return mbar_wait_for(bar, parity, abort, err, 8 * ATTN_WAIT_NS);
}

// The key-tile ranges of an item's query tiles: those that hold a key some row sees.
__device__ __forceinline__ void packed_ranges(const Params& p, Item& it) {
  const int off = it.sk - it.sq;
  const int tpt = BM >> p.pack_log2;   // tokens per tile
  it.lo_all = 1 << 30;
  it.hi_all = 0;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int r0 = it.row0 + tpt * i;
    const int r1 = min(r0 + tpt, it.end);   // exclusive
    int lo = 0, hi = 0;
    if (r0 < r1) {
      const int last_key = p.causal ? min(r1 - 1 + off, it.sk - 1) : it.sk - 1;
      const int first_key = (p.causal && p.window > 0) ? max(0, r0 + off - p.window + 1) : 0;
      if (last_key >= first_key) {
        lo = first_key / BN;
        hi = last_key / BN + 1;
      }
    }
    it.lo[i] = lo;
    it.hi[i] = hi;
    if (hi > lo) {
      it.lo_all = min(it.lo_all, lo);
      it.hi_all = max(it.hi_all, hi);
    }
  }
  if (it.hi_all <= 0) it.lo_all = it.hi_all = 0;
}

// SPLIT: the item's ranges cut to share `part` of its key tiles.
__device__ __forceinline__ void cut_to_part(const Params& p, Item& it, int part) {
  const int n = it.hi_all - it.lo_all;
  const int from = it.lo_all + n * part / p.splits, to = it.lo_all + n * (part + 1) / p.splits;
  it.lo_all = 1 << 30;
  it.hi_all = 0;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    it.lo[i] = max(it.lo[i], from);
    it.hi[i] = min(it.hi[i], to);
    if (it.hi[i] > it.lo[i]) {
      it.lo_all = min(it.lo_all, it.lo[i]);
      it.hi_all = max(it.hi_all, it.hi[i]);
    } else {
      it.lo[i] = it.hi[i] = 0;
    }
  }
  if (it.hi_all <= 0) it.lo_all = it.hi_all = 0;
}

// Rows [from, to) of the item's last V tile lie behind its sequence and must be
// zeroed before P V reads them (to <= from: none).  Packed rows behind a
// sequence are the next one's; of paged ones only the box that holds the last
// key brings any, since boxes wholly behind it are filled with zeros.
template <bool PAGED>
__device__ __forceinline__ void v_tail(const Params& p, const Item& it, int& from, int& to) {
  from = it.sk - (it.hi_all - 1) * BN;
  to = BN;
  if constexpr (PAGED) to = min(BN, (from + p.box_rows - 1) / p.box_rows * p.box_rows);
}

__device__ __forceinline__ bool active(const Item& it, int i, int j) { return j >= it.lo[i] && j < it.hi[i]; }

// True if every key of tile j is visible to all of the tokens [t0, t1] of the sequence.
__device__ __forceinline__ bool tile_unmasked(const Params& p, const Item& it, int t0, int t1, int j) {
  const int off = it.sk - it.sq;
  const int k0 = j * BN, k1 = j * BN + BN - 1;
  if (k1 >= it.sk) return false;
  if (!p.causal) return true;
  if (k1 > t0 + off) return false;
  if (p.window > 0 && k0 <= t1 + off - p.window) return false;
  return true;
}

template <int D, bool PAGED, bool SPLIT, bool RUNS>
__global__ void __launch_bounds__(Cfg<D>::THREADS, 1)
    prefill_packed_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_v, const Params p) {
  using C = Cfg<D>;
  constexpr int STAGES = C::STAGES, QBUF = C::QBUF;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                                   // [QBUF][NQ][KATOMS][BM rows x 128 B]
  uint8_t* sRing = smem + QBUF * NQ * C::Q_BYTES;       // [STAGES][one tile, or V and K][KATOMS][BN rows x 128 B]
  uint8_t* control = sRing + STAGES * C::STAGE_BYTES;
  uint8_t* sOut = control + C::CONTROL;                 // [8 softmax warps][4 KB]
  uint64_t* q_full = reinterpret_cast<uint64_t*>(control);   // QBUF
  uint64_t* q_empty = q_full + QBUF;                    // QBUF
  uint64_t* full = q_empty + QBUF;                      // STAGES
  uint64_t* empty = full + STAGES;                      // STAGES
  uint64_t* s_ready = empty + STAGES;                   // NQ
  uint64_t* p_ready = s_ready + NQ;                     // NQ
  uint64_t* o_done = p_ready + NQ;                      // NQ: O_i final (SEP_P: each P_i V done)
  uint64_t* s_free = o_done + NQ;                       // NQ: S_i loaded by the softmax (SEP_P)
  uint64_t* drain = s_free + NQ;                        // 1
  uint64_t* item_full = drain + 1;                      // kItemRing
  uint64_t* item_empty = item_full + kItemRing;         // kItemRing
  uint64_t* tail_go = item_empty + kItemRing;           // 1: a V tile with rows to zero has landed
  uint64_t* tail_done = tail_go + 1;                    // 1: they are zero
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail_done + 1);
  // and behind it the counts that renew the waits (wait_is_over): stages filled, items of a pass looked at
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Item* item_ring = reinterpret_cast<Item*>(tmem_slot + 4);   // kItemRing
  static_assert((2 * QBUF + 2 * STAGES + 4 * NQ + 3 + 2 * kItemRing) * 8 + 16 + kItemRing * sizeof(Item) <= C::CONTROL,
                "barriers and item ring");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int q = 0; q < QBUF; ++q) {
      mbar_init(&q_full[q], 1);
      mbar_init(&q_empty[q], 1);
    }
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&s_ready[i], 1);
      mbar_init(&p_ready[i], 4 * 32);
      mbar_init(&o_done[i], 1);
      mbar_init(&s_free[i], 4 * 32);
    }
    mbar_init(drain, 1);
    for (int s = 0; s < kItemRing; ++s) {
      mbar_init(&item_full[s], 1);
      mbar_init(&item_empty[s], kItemConsumers);
    }
    mbar_init(tail_go, 1);
    mbar_init(tail_done, 32);
    abort_flag[0] = abort_flag[1] = abort_flag[2] = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // set-up above overlaps the tail of the kernel before; global memory only from here on
  grid_dependency_wait();

  // The r-th item from the scheduler's ring; false at the end of the list or if a wait
  // gave up.  whole_warp: all 32 lanes call (one lane arrives for them).
  auto next_item = [&](int r, bool whole_warp, Item& it) -> bool {
    const int slot = r % kItemRing;
    bool got = mbar_wait<true>(&item_full[slot], (r / kItemRing) & 1, abort_flag, p.err);
    if (whole_warp) got = __all_sync(0xffffffffu, got);
    it.b = -1;
    if (!got) return false;
    it = item_ring[slot];
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(&item_empty[slot]);
    return it.b >= 0;
  };
  // The roles that move and multiply tiles: the next item with any.  Those without come
  // last; the first of them ends the role's work, and pass_rest takes what is left.
  auto next_work = [&](int& r, bool whole_warp, Item& it) -> bool {
    return next_item(r++, whole_warp, it) && it.hi_all > it.lo_all;
  };
  auto pass_rest = [&](int& r, bool whole_warp, const Item& last) {
    if (last.b < 0) return;
    Item it;
    while (next_item(r++, whole_warp, it)) {}
  };

  if (warp >= 8) {
   // ------------------------------------------------------------ producer warpgroup
   asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::PRODUCER_REGS));
   if (warp == kTmaWarp) {
    // ------------------------------------------------------------ TMA producer
    // One thread; PAGED: the whole warp, so that the page-table entries of a tile are read by one
    // load and its page boxes issued by one instruction (lane 0 still arms the barriers and loads Q).
    if (PAGED || lane == 0) {
      const bool lead = (lane == 0);
      auto uni = [&](bool v) -> bool {   // one outcome for the whole warp
        if constexpr (PAGED) return __all_sync(0xffffffffu, v);
        return v;
      };
      if (lead) {
        prefetch_tmap(&tmap_q);
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
      }
      const int tpt = BM >> p.pack_log2;   // tokens per query tile
      int r = 0, n = 0, qn = 0;
      bool ok = true;
      auto load_q = [&](const Item& it) -> bool {
        const int qb = qn % QBUF;
        if (qn >= QBUF && !uni(mbar_wait<true>(&q_empty[qb], ((qn / QBUF) - 1) & 1, abort_flag, p.err))) return false;
        if (lead) {
          // a tile without tokens is not loaded; nothing multiplies it either
          const int nt = (it.row0 + tpt < it.end) ? NQ : 1;
          mbar_arrive_expect_tx(&q_full[qb], nt * C::Q_BYTES);
          for (int i = 0; i < nt; ++i)
            for (int a = 0; a < C::KATOMS; ++a)
              tma_load_4d(sQ + ((qb * NQ + i) * C::KATOMS + a) * BM * 128, &tmap_q, &q_full[qb], a * 64, 0,
                          it.q_base + it.row0 + tpt * i, it.hb);
        }
        ++qn;
        return true;
      };
      // PAGED: the physical page of this lane's box of key tile j (lane rb + nb * a copies
      // box rb of swizzle atom a), or the pool size for a box past the end of the sequence.
      // K_j and V_j share it, and it is read a tile ahead of the wait for a free stage.
      auto page_of = [&](const Item& it, int j) -> int {
        if constexpr (!PAGED) {
          return 0;
        } else {
          const int nb = BN / p.box_rows;
          int ph = p.num_pages;                 // plane ph * Hkv + g is past the pool's planes
          if (lane < nb * C::KATOMS) {
            const int key0 = j * BN + (lane % nb) * p.box_rows;
            if (key0 < it.sk) {
              ph = p.page_table[static_cast<size_t>(SPLIT ? it.b & 0xFFFF : it.b) * p.max_pages + key0 / p.page_size];
              if (ph < 0 || ph >= p.num_pages) {  // never read outside the pool
                record_error(p.err, ATTN_ERRBIT_BADPAGE);
                ph = 0;
              }
            }
          }
          return ph;
        }
      };
      auto copy_tile = [&](uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, const Item& it, int j, int ph) {
        if constexpr (!PAGED) {
          for (int a = 0; a < C::KATOMS; ++a)
            tma_load_3d(dst + a * BN * 128, tm, bar, a * 64, it.k_base + j * BN, it.g);
        } else {
          // the key tile is assembled from page boxes of box_rows rows each; a box lands at its row
          // offset inside the swizzled tile, so the MMA sees the layout of a whole load
          const int nb = BN / p.box_rows;
          if (lane < nb * C::KATOMS) {
            const int rb = lane % nb, a = lane / nb;
            const int key0 = j * BN + rb * p.box_rows;
            tma_load_3d(dst + a * BN * 128 + rb * p.box_rows * 128, tm, bar, a * 64, key0 % p.page_size,
                        ph * p.Hkv + it.g);
          }
        }
      };
      // next stage <- V of tile vj of v (unless null), then K of tile kj of k (unless null)
      auto load_stage = [&](const Item* v, int vj, int vph, const Item* k, int kj, int kph) -> bool {
        const int st = n % STAGES;
        if (!uni(mbar_wait<true>(&empty[st], ((n / STAGES) & 1) ^ 1, abort_flag, p.err))) return false;
        if (lead) mbar_arrive_expect_tx(&full[st], (v ? C::TILE_BYTES : 0) + (k ? C::TILE_BYTES : 0));
        if constexpr (PAGED) __syncwarp();   // the barrier is armed before any box can land
        uint8_t* dst = sRing + st * C::STAGE_BYTES;
        if (v) copy_tile(dst, &tmap_v, &full[st], *v, vj, vph);
        if (k) copy_tile(dst + (C::SEP_P ? 0 : C::TILE_BYTES), &tmap_k, &full[st], *k, kj, kph);
        ++n;
        if (lead) abort_flag[1] = n;
        return true;
      };
      Item it;
      bool have = next_work(r, PAGED, it);
      // load order = the MMA thread's consumption order
      if constexpr (C::SEP_P) {   // Q, K_lo, then K_{j+1} ahead of V_j
        while (have && ok) {
          int ph = page_of(it, it.lo_all);
          int ph1 = (it.lo_all + 1 < it.hi_all) ? page_of(it, it.lo_all + 1) : 0;
          ok = load_q(it) && load_stage(nullptr, 0, 0, &it, it.lo_all, ph);
          for (int j = it.lo_all; j < it.hi_all && ok; ++j) {
            const int ph2 = (j + 2 < it.hi_all) ? page_of(it, j + 2) : 0;
            if (j + 1 < it.hi_all) ok = load_stage(nullptr, 0, 0, &it, j + 1, ph1);
            if (ok) ok = load_stage(&it, j, ph, nullptr, 0, 0);
            ph = ph1;
            ph1 = ph2;
          }
          if (ok) have = next_work(r, PAGED, it);
        }
      } else {                    // K_lo, Q, then V_j with K_{j+1} or the next item's first K
        Item nx;
        int ph = 0;
        if (have) {
          ph = page_of(it, it.lo_all);
          ok = load_stage(nullptr, 0, 0, &it, it.lo_all, ph);
        }
        while (have && ok) {
          // Q waits for the S of the item before; this item's first K went ahead of it
          if (!(ok = load_q(it))) break;
          bool more = false;
          int ph1 = (it.lo_all + 1 < it.hi_all) ? page_of(it, it.lo_all + 1) : 0;
          for (int j = it.lo_all; j < it.hi_all && ok; ++j) {
            if (j + 1 < it.hi_all) {
              const int ph2 = (j + 2 < it.hi_all) ? page_of(it, j + 2) : 0;
              ok = load_stage(&it, j, ph, &it, j + 1, ph1);
              ph = ph1;
              ph1 = ph2;
            } else {
              more = next_work(r, PAGED, nx);
              const int phn = more ? page_of(nx, nx.lo_all) : 0;
              ok = load_stage(&it, j, ph, more ? &nx : nullptr, more ? nx.lo_all : 0, phn);
              ph = phn;
            }
          }
          it = nx;
          have = more;
        }
      }
      if (ok) pass_rest(r, PAGED, it);
      // the last loads issued must land before the CTA may exit (normally already consumed)
      for (int k = max(0, n - STAGES); k < n; ++k) mbar_wait(&full[k % STAGES], (k / STAGES) & 1, nullptr, p.err);
    }
   } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BN, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(BM, D, 0, 1);
      constexpr uint32_t kHi = sw128_desc_hi(1024);   // 8-row groups 1024 B apart
      // descriptor low words at K step 0: Q tiles and the stages' K (K-major) and V (MN-major, 64-column
      // blocks BN * 128 bytes apart); a K step adds a compile-time offset in 16-byte units
      const uint32_t q_lo0 = sw128_desc_lo(smem_u32(sQ), 16);
      const uint32_t v_lo0 = sw128_desc_lo(smem_u32(sRing), BN * 128);
      const uint32_t k_lo0 = sw128_desc_lo(smem_u32(sRing) + (C::SEP_P ? 0 : C::TILE_BYTES), 16);
      int r = 0, n = 0, qn = 0, tails = 0;
      uint32_t tp = 0;          // bit i: parity of P_i's next phase
      bool ok = true;

      auto issue_s = [&](int i, int qb, int st) {  // S_i = Q_i K^T with the K of stage st
        const uint32_t d_tmem = tmem + C::S_COL + BN * i;
        const uint32_t a_lo = q_lo0 + (((qb * NQ + i) * C::Q_BYTES) >> 4);
        const uint32_t b_lo = k_lo0 + ((st * C::STAGE_BYTES) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t koff = ((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4;
          mma_ss(d_tmem, desc64(a_lo + koff, kHi), desc64(b_lo + koff, kHi), idesc_s, kk > 0 ? 1u : 0u);
        }
        mma_commit(&s_ready[i]);
      };
      auto issue_pv = [&](int i, int st, uint32_t acc0) {  // O_i (+)= P_i V with the V of stage st
        const uint32_t o_tmem = tmem + C::O_COL + D * i;
        const uint32_t p_tmem = tmem + C::P_COL + C::P_STRIDE * i;
        const uint32_t b_lo = v_lo0 + ((st * C::STAGE_BYTES) >> 4);
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          mma_ts(o_tmem, p_tmem + kk * 8, desc64(b_lo + ((kk * 16 * 128) >> 4), kHi), idesc_pv, kk > 0 ? 1u : acc0);
      };
      // P_i(j) V_j begins a sum
      auto starts = [&](const Item& it, int i, int j) -> bool {
        return RUNS ? ((j - it.lo[i]) & (kRun - 1)) == 0 : j == it.lo[i];
      };
      auto wait_p = [&](int i) -> bool {
        const bool got = tile_wait(&p_ready[i], (tp >> i) & 1, abort_flag, p.err);
        tp ^= 1u << i;
        tc_fence_after();
        return got;
      };
      auto wait_stage = [&](int st) -> bool {
        const bool got = tile_wait(&full[st], (n / STAGES) & 1, abort_flag, p.err);
        tc_fence_after();
        return got;
      };
      // the V rows behind the sequence: warp 11 zeroes them while the softmax of the last tile runs
      auto tail_start = [&](const Item& it) -> bool {
        int from, to;
        v_tail<PAGED>(p, it, from, to);
        if (to <= from) return false;
        mbar_arrive(tail_go);
        return true;
      };
      auto tail_wait = [&]() -> bool {
        const bool got = tile_wait(tail_done, tails & 1, abort_flag, p.err);
        ++tails;
        return got;
      };

      Item it;
      bool have = next_work(r, false, it);
      if constexpr (C::SEP_P) {
        // Per key tile j: S_i(j + 1) as soon as softmax group i has loaded S_i(j) (s_free), then
        // P_i(j) V_j as soon as it has written P_i(j).
        uint32_t used = 0, tf = 0;   // bit i: S_i was written before; parity of s_free's next phase
        auto issue_next_s = [&](int i, int qb, int st) -> bool {
          if (used & (1u << i)) {
            if (!tile_wait(&s_free[i], (tf >> i) & 1, abort_flag, p.err)) return false;
            tf ^= 1u << i;
            tc_fence_after();
          }
          used |= 1u << i;
          issue_s(i, qb, st);
          return true;
        };
        while (have && ok) {
          const int qb = qn % QBUF;
          if (!(ok = tile_wait(&q_full[qb], (qn / QBUF) & 1, abort_flag, p.err))) break;
          tc_fence_after();
          ++qn;
          int st = n % STAGES;
          if (!(ok = wait_stage(st))) break;
#pragma unroll
          for (int i = 0; i < NQ; ++i)
            if (ok && active(it, i, it.lo_all)) ok = issue_next_s(i, qb, st);
          if (!ok) break;
          mma_commit(&empty[st]);
          ++n;
          if (it.hi_all - it.lo_all == 1) mma_commit(&q_empty[qb]);
          for (int j = it.lo_all; j < it.hi_all && ok; ++j) {
            if (j + 1 < it.hi_all) {
              st = n % STAGES;
              if (!(ok = wait_stage(st))) break;
#pragma unroll
              for (int i = 0; i < NQ; ++i)
                if (ok && active(it, i, j + 1)) ok = issue_next_s(i, qb, st);
              if (!ok) break;
              mma_commit(&empty[st]);
              ++n;
              if (j + 1 == it.hi_all - 1) mma_commit(&q_empty[qb]);
            }
            st = n % STAGES;
            if (!(ok = wait_stage(st))) break;
            bool tail = j + 1 == it.hi_all && tail_start(it);
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
              if (!ok || !active(it, i, j)) continue;
              ok = wait_p(i);
              if (ok && tail) {
                ok = tail_wait();
                tail = false;
              }
              if (!ok) continue;
              issue_pv(i, st, starts(it, i, j) ? 0u : 1u);
              mma_commit(&o_done[i]);   // P_i free again, O_i current
            }
            if (!ok) break;
            mma_commit(&empty[st]);
            ++n;
          }
          if (ok) have = next_work(r, false, it);
        }
      } else {
        // Per key tile j and query tile i: P_i(j) V_j as soon as softmax group i has written P_i(j) over
        // S_i(j), then S_i(j + 1); one group's softmax overlaps the other group's products.
        if (have) ok = wait_stage(0);
        while (have && ok) {
          const int qb = qn % QBUF;
          if (!(ok = tile_wait(&q_full[qb], (qn / QBUF) & 1, abort_flag, p.err))) break;
          tc_fence_after();
          ++qn;
          int st = n % STAGES;   // holds the V of the tile before (used up) and this item's first K
#pragma unroll
          for (int i = 0; i < NQ; ++i)
            if (active(it, i, it.lo_all)) issue_s(i, qb, st);
          mma_commit(&empty[st]);
          ++n;
          if (it.hi_all - it.lo_all == 1) mma_commit(&q_empty[qb]);
          for (int j = it.lo_all;; ++j) {
            st = n % STAGES;
            if (!(ok = wait_stage(st))) break;
            const bool next = j + 1 < it.hi_all;
            bool tail = !next && tail_start(it);
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
              if (active(it, i, j)) {
                if (!(ok = wait_p(i))) break;
                if (tail) {
                  tail = false;
                  if (!(ok = tail_wait())) break;
                }
                issue_pv(i, st, starts(it, i, j) ? 0u : 1u);
                if (j == it.hi[i] - 1) mma_commit(&o_done[i]);
              }
              if (next && active(it, i, j + 1)) issue_s(i, qb, st);
            }
            if (!ok || !next) break;
            mma_commit(&empty[st]);
            ++n;
            if (j == it.hi_all - 2) mma_commit(&q_empty[qb]);
          }
          if (!ok) break;
          have = next_work(r, false, it);   // its first K is in the stage of the last V
        }
      }
      // everything issued above must be complete before tensor memory is released
      mma_commit(drain);
      mbar_wait(drain, 0, nullptr, p.err);
      if (ok) pass_rest(r, false, it);
    }
   } else if (warp == kSchedWarp) {
    // ------------------------------------------------------------ item scheduler
    // Blocks are ranked level by level from the highest (costliest) down, within
    // a level by sequence; item k is head block k % head_blocks of the block of
    // rank k / head_blocks.  This CTA's k only grow, so one walk down the levels,
    // and within a level over the sequences, serves all its items.  A level costs two
    // passes over the sequences, 32 at a time: levels get wider (2^shift steps) until
    // there are at most 2048 such chunks to visit in all.  (16384 sequences of one token,
    // 32/8 heads: 4.8 ms; with a search from the first sequence for every item 113 ms.)
    const int tpt = BM >> p.pack_log2;
    const int tb_log2 = 8 - p.pack_log2;   // NQ * BM rows of 2^s heads
    const int chunks = (p.B + 31) / 32;
    // sequence 32 c + lane; the first 32 stay in registers
    auto span_of = [&](int c) -> PackedSpan {
      PackedSpan s = {0, 0, 0, 0};
      if (c * 32 + lane < p.B) s = packed_span<PAGED>(p, c * 32 + lane);
      return s;
    };
    const PackedSpan span0 = span_of(0);
    auto steps_of = [&](int c) -> PackedSteps { return packed_steps(p, c == 0 ? span0 : span_of(c), tb_log2); };
    const int blocks_per_kv = p.Hq / p.Hkv >> p.pack_log2;   // head blocks of a kv head
    int top = -1;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) top = max(top, top_step(steps_of(c), p.causal));
    top = __reduce_max_sync(0xffffffffu, top);
    int shift = 0;
    while (shift < 20 && ((top >> shift) + 1LL) * chunks > 2048) ++shift;
    // the level being dealt out: its blocks, the rank of its first, the next level, and how many of
    // its blocks lie in chunks before `chunk`
    int level = -1, count = 0, base = 0, below = -1, chunk = 0, passed = 0;
    auto visit = [&](int q) {
      int m = 0, nx = -1;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        const PackedSteps l = steps_of(c);
        m += blocks_at(l, p.causal, q, shift);
        nx = max(nx, next_level(l, p.causal, q, shift));
      }
      level = q;
      count = __reduce_add_sync(0xffffffffu, m);
      below = __reduce_max_sync(0xffffffffu, nx);
      chunk = passed = 0;
    };
    // Two passes: the items with key tiles, then (if any) those none of whose rows sees a key, whose
    // zeros the softmax warps write.  The producer and the MMA thread look an item ahead, and
    // must not wait for the softmax to pass items that they have no part in.
    bool none = false;
    int put = 0;   // items handed out
    bool go_on = true;
    for (int pass = 0; pass < (none ? 2 : 1) && go_on; ++pass) {
      const bool rows_left = pass == 1;
      base = 0;
      level = -1;
      if (top >= 0) visit(top >> shift);
      for (int r = 0;; ++r) {
        const int P = gridDim.x, c = blockIdx.x;
        const int k = r * P + ((r & 1) ? (P - 1 - c) : c);
        if (lane == 0) abort_flag[2] = r;
        const int unit = SPLIT ? k / p.splits : k;
        const int rank = unit / p.head_blocks;
        while (level >= 0 && rank >= base + count) {
          base += count;
          if (below < 0) level = -1;
          else visit(below);
        }
        Item it;
        it.b = -1;
        // sequences that do not overlap have at most n_items items: more means malformed lengths
        if (level >= 0 && k >= p.n_items) {
          if (lane == 0) record_error(p.err, ATTN_ERRBIT_BADPAGE);
          level = -1;
        }
        if (level >= 0) {
#pragma unroll 1
          for (; chunk < chunks; ++chunk) {
            int j = rank - base - passed;   // the j-th block of this level from this chunk on
            const PackedSpan sp = chunk == 0 ? span0 : span_of(chunk);
            const PackedSteps l = packed_steps(p, sp, tb_log2);
            const int m = blocks_at(l, p.causal, level, shift);
            // inclusive count over the lanes: of ones where a sequence has one block at most
            int incl = __popc(__ballot_sync(0xffffffffu, m > 0) & (0xffffffffu >> (31 - lane)));
            if (__any_sync(0xffffffffu, m > 1)) {
              incl = m;
#pragma unroll
              for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += v;
              }
            }
            const int total = __shfl_sync(0xffffffffu, incl, 31);
            if (j >= total) {
              passed += total;
              continue;
            }
            const int src = __ffs(__ballot_sync(0xffffffffu, incl > j)) - 1;
            j -= __shfl_sync(0xffffffffu, incl - m, src);
            const int qb = __shfl_sync(0xffffffffu, block_of(l, p.causal, level, shift, j), src);
            const int nb = __shfl_sync(0xffffffffu, l.nb, src);
            // (counts of malformed, overlapping lengths may have wrapped: no block then)
            if (src < 0 || chunk * 32 + src >= p.B || qb < 0 || qb >= nb) break;
            it.b = chunk * 32 + src;
            it.hb = unit - rank * p.head_blocks;
            it.g = blocks_per_kv == 1 ? it.hb : it.hb / blocks_per_kv;
            it.row0 = qb << tb_log2;
            it.q_base = __shfl_sync(0xffffffffu, sp.q0, src);
            it.k_base = __shfl_sync(0xffffffffu, sp.k0, src);
            it.sq = __shfl_sync(0xffffffffu, sp.sq, src);
            it.sk = __shfl_sync(0xffffffffu, sp.sk, src);
            it.end = min(it.sq, it.row0 + NQ * tpt);
            packed_ranges(p, it);
            if constexpr (SPLIT) {
              cut_to_part(p, it, k - unit * p.splits);
              it.b |= (k - unit * p.splits) << 16;
            }
            break;
          }
        }
        if (it.b >= 0 && (it.hi_all <= it.lo_all) != rows_left) {   // not of this pass
          none |= !rows_left;
          continue;
        }
        if (it.b < 0 && none && !rows_left) break;   // the second pass ends the list
        const int slot = put % kItemRing;
        if (!__all_sync(0xffffffffu,
                        mbar_wait_idle<true>(&item_empty[slot], ((put / kItemRing) & 1) ^ 1, abort_flag, p.err))) {
          go_on = false;
          break;
        }
        ++put;
        if (lane == 0) {
          item_ring[slot] = it;
          mbar_arrive(&item_full[slot]);
        }
        if (it.b < 0) break;
      }
    }
   } else if (warp == kTailWarp) {
    // ------------------------------------------------------------ V rows behind a sequence
    int tiles = 0, tails = 0;   // key tiles of the items so far, V tiles zeroed
    for (int r = 0;; ++r) {
      Item it;
      if (!__all_sync(0xffffffffu, mbar_wait_idle<true>(&item_full[r % kItemRing], (r / kItemRing) & 1, abort_flag, p.err)))
        break;
      if (!next_item(r, true, it)) break;
      tiles += it.hi_all - it.lo_all;
      const int n = C::SEP_P ? 2 * tiles - 1 : tiles;   // number of the stage of the item's last V
      int from, to;
      v_tail<PAGED>(p, it, from, to);
      if (to <= from) continue;
      const int st = n % STAGES;
      // the MMA thread has seen the stage land, and frees it only after tail_done
      bool got = mbar_wait_idle<true>(tail_go, tails & 1, abort_flag, p.err);
      got = got && mbar_wait<true>(&full[st], (n / STAGES) & 1, abort_flag, p.err);
      if (!__all_sync(0xffffffffu, got)) break;
      ++tails;
      for (int a = 0; a < C::KATOMS; ++a) {
        const uint32_t rows = smem_u32(sRing + st * C::STAGE_BYTES + a * BN * 128);
        for (int e = from * 128 + lane * 16; e < to * 128; e += 512)   // a row holds its key's values under the swizzle
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(rows + e), "r"(0u) : "memory");
      }
      fence_proxy_async_smem();
      mbar_arrive(tail_done);
    }
   }
  } else {
    // ------------------------------------------------------------ softmax groups
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
    const int i = warp >> 2;                 // query tile
    const int wq = warp & 3;                 // lane quarter of tensor memory
    const int rl = wq * 32 + lane;           // row within the tile
    const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t s_tmem = tmem + lane_bits + C::S_COL + BN * i;
    const uint32_t p_tmem = tmem + lane_bits + C::P_COL + C::P_STRIDE * i;
    const uint32_t o_tmem = tmem + lane_bits + C::O_COL + D * i;
    const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
    int t = 0, oc = 0;
    int pv = 0;   // SEP_P: P_i V products of this tile completed and waited for
    // O_i *= alpha (every row of the warp takes part when any row needs it)
    auto rescale_o = [&](bool later_tile, float alpha) {
      if (!__any_sync(0xffffffffu, later_tile && alpha != 1.f)) return;
      const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(o_tmem + 32 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x0, x1;
          f2_unpack(f2_mul(f2_pack(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), a2), x0, x1);
          o[e] = __float_as_uint(x0);
          o[e + 1] = __float_as_uint(x1);
        }
        tmem_st32(o_tmem + 32 * c, o);
      }
    };
    float bank[RUNS ? D + 2 : 1];   // the runs before: O_i, l, and the maximum that they refer to (local memory, used once a run)
    bool ok = true;

    for (int rr = 0; ok; ++rr) {
      Item it;
      if (!next_item(rr, true, it)) break;
      const int my_lo = (i == 0) ? it.lo[0] : it.lo[1];
      const int my_hi = (i == 0) ? it.hi[0] : it.hi[1];
      // this thread's row: a token of the sequence, one of 2^s heads
      const int tpt = BM >> p.pack_log2;
      const int r0 = it.row0 + tpt * i;
      const int r = r0 + (rl >> p.pack_log2);
      const bool store = r < it.end;
      auto head = [&]() -> int { return (it.hb << p.pack_log2) + (rl & ((1 << p.pack_log2) - 1)); };
      auto lse_at = [&]() -> size_t { return (static_cast<size_t>(it.q_base) + r) * p.Hq + head(); };
      auto ws_at = [&]() -> size_t { return static_cast<size_t>(it.b >> 16) * p.Tq * p.Hq + lse_at(); };   // SPLIT
      if (my_hi <= my_lo) {                  // no visible key for any row of this tile
        if (SPLIT && store) {
          p.ws_lse[ws_at()] = -INFINITY;
        } else if (store) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + (static_cast<size_t>(it.q_base) + r) * p.out_stride +
                                                static_cast<size_t>(head()) * D);
          for (int e = 0; e < D / 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse != nullptr) p.lse[lse_at()] = -INFINITY;
        }
        continue;
      }
      // visible keys of this row: [key_lo, key_hi]
      const int off = it.sk - it.sq;
      const int key_hi = p.causal ? min(r + off, it.sk - 1) : it.sk - 1;
      const int key_lo = (p.causal && p.window > 0) ? r + off - p.window + 1 : 0;
      float m_ref = -INFINITY, l = 0.f;
      // O_i and l into the bank at the end of a run, or out of it at the end of the item
      [[maybe_unused]] auto join_runs = [&](bool first, bool last) {
        const float f = (first || bank[D + 1] == -INFINITY) ? 0.f : ex2(bank[D + 1] - m_ref);
        tmem_wait_st();   // a rescaled O_i
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_tmem + 32 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x = __uint_as_float(o[e]);
            if (!first) x = fmaf(bank[32 * c + e], f, x);
            if (!last) bank[32 * c + e] = x;
            o[e] = __float_as_uint(x);
          }
          if (last) tmem_st32(o_tmem + 32 * c, o);
        }
        if (!first) l = fmaf(bank[D], f, l);
        if (last) {
          tmem_wait_st();
        } else {
          bank[D] = l;
          bank[D + 1] = m_ref;
          l = 0.f;
        }
      };

      for (int j = my_lo; j < my_hi; ++j, ++t) {
        ok = tile_wait(&s_ready[i], t & 1, abort_flag, p.err);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool run_ends = RUNS && j > my_lo && ((j - my_lo) & (kRun - 1)) == 0;
        if constexpr (RUNS && !C::SEP_P) {
          if (run_ends) join_runs(j == my_lo + kRun, false);   // S_i(j) covers P_i V(j-1); P_i V(j) starts from nothing
        }
        float s[BN];
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) tmem_ld32f(s_tmem + 32 * c, s + 32 * c);
        tmem_wait_ld();
        if constexpr (C::SEP_P) {   // S_i may be overwritten by S_i(j+1) from here on
          tc_fence_before();
          mbar_arrive(&s_free[i]);
        }
        if (!tile_unmasked(p, it, r0, r0 + tpt - 1, j)) {
          const int c_lo = key_lo - j * BN, c_hi = key_hi - j * BN;
#pragma unroll
          for (int c = 0; c < BN; ++c) s[c] = (c >= c_lo && c <= c_hi) ? s[c] : -INFINITY;
        }
        // row maximum: four independent chains of three-input max
        // (columns 0-7 start the chains, then 8 columns per step: exactly s[0, BN))
        float mc[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) mc[q] = fmaxf(s[2 * q], s[2 * q + 1]);
#pragma unroll
        for (int c = 8; c < BN; c += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q) mc[q] = fmax3(mc[q], s[c + 2 * q], s[c + 2 * q + 1]);
        const float mx = fmaxf(fmax3(mc[0], mc[1], mc[2]), mc[3]);
        const float m_tile = mx * p.scale_log2;
        float alpha = 1.f;
        if (m_tile > m_ref + kTau) {
          alpha = (m_ref == -INFINITY) ? 0.f : ex2(m_ref - m_tile);
          l *= alpha;
          m_ref = m_tile;
        }
        if constexpr (!C::SEP_P) rescale_o(j > my_lo, alpha);   // O_i is current: S_i(j) covers P_i V(j-1)
        const float mb = (m_ref == -INFINITY) ? 0.f : m_ref;
        const uint64_t nm2 = f2_pack(-mb, -mb);
        uint32_t pk[BN / 2];
        uint64_t sum2[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) sum2[q] = f2_pack(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < BN; c += 2) {
          const uint64_t x2 = f2_fma(f2_pack(s[c], s[c + 1]), c2, nm2);
          float x0, x1;
          f2_unpack(x2, x0, x1);
          const float p0 = ex2(x0), p1 = ex2(x1);
          sum2[(c / 2) % 4] = f2_add(sum2[(c / 2) % 4], f2_pack(p0, p1));
          pk[c / 2] = pack_bf16x2(p0, p1);
        }
        float s0, s1, s2, s3;
        f2_unpack(f2_add(sum2[0], sum2[1]), s0, s1);
        f2_unpack(f2_add(sum2[2], sum2[3]), s2, s3);
        l += (s0 + s1) + (s2 + s3);
        // The exponentials above need nothing from tensor memory; only now must
        // P_i(j-1) V be complete: before O_i is rescaled and (separate P) before
        // P_i is rewritten.  Waiting here hides that product behind them.
        if constexpr (C::SEP_P) {
          if (j > my_lo) {
            ok = tile_wait(&o_done[i], pv & 1, abort_flag, p.err);
            ++pv;
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
        }
        if constexpr (C::SEP_P) rescale_o(j > my_lo, alpha);
        if constexpr (RUNS && C::SEP_P) {
          if (run_ends) join_runs(j == my_lo + kRun, false);
        }
#pragma unroll
        for (int c = 0; c < BN / 64; ++c) tmem_st32(p_tmem + 32 * c, pk + 32 * c);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_ready[i]);
      }
      if (!ok) break;
      // ---- epilogue: O / l -> bf16 (tcgen05.ld is warp-collective: every lane loads)
      if constexpr (C::SEP_P) {
        ok = tile_wait(&o_done[i], pv & 1, abort_flag, p.err);
        ++pv;
      } else {
        ok = tile_wait(&o_done[i], oc & 1, abort_flag, p.err);
        ++oc;
      }
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if constexpr (RUNS) {
        if (my_hi - my_lo > kRun) join_runs(false, true);
      }
      // a row with no visible key is 0 (and its lse -inf)
      const bool has_keys = key_hi >= max(key_lo, 0);
      const float inv = (has_keys && l > 0.f) ? 1.f / l : 0.f;
      if constexpr (SPLIT) {
        const size_t at = ws_at();
        if (store) p.ws_lse[at] = l == 0.f ? -INFINITY : m_ref + log2f(l);   // (NaN stays NaN)
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_tmem + 32 * c, o);
          tmem_wait_ld();
          if (store) {
            float4* dst = reinterpret_cast<float4*>(p.ws_o + at * D + 32 * c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                   __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
          }
        }
      } else {
        if (p.lse != nullptr && store)   // log(sum_j exp(s_ij * scale)) = (m + log2 l) * ln 2
          p.lse[lse_at()] = (!has_keys || l == 0.f) ? -INFINITY : (m_ref + log2f(l)) * 0.6931471805599453f;
        // (64 columns of the warp's 32 rows at a time; the 16-byte pieces of a row are permuted by its
        // number, which keeps both sides free of bank conflicts)
        uint8_t* stage = sOut + warp * 4096;
        const int at0 = wq * 32 + (lane >> 3), piece = lane & 7, mask = (1 << p.pack_log2) - 1;
        __nv_bfloat16* base = p.out + (static_cast<size_t>(it.q_base) + r0) * p.out_stride +
                              (static_cast<size_t>(it.hb) << p.pack_log2) * D + piece * 8;
        const int last = it.end - r0;   // tokens of this tile
        const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll 1
        for (int h = 0; h < D / 64; ++h) {
          uint32_t o[64];
          tmem_ld32(o_tmem + 64 * h, o);
          tmem_ld32(o_tmem + 64 * h + 32, o + 32);
          tmem_wait_ld();
          __syncwarp();   // the warp has read the half before
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              float lo, hi;
              const uint64_t pair = f2_pack(__uint_as_float(o[8 * e + 2 * x]), __uint_as_float(o[8 * e + 2 * x + 1]));
              f2_unpack(f2_mul(pair, inv2), lo, hi);
              w[x] = pack_bf16x2(lo, hi);
            }
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) * 16)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
          uint4 u[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int row = 4 * e + (lane >> 3);
            u[e] = *reinterpret_cast<const uint4*>(stage + row * 128 + ((piece ^ (row & 7)) * 16));
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int at = at0 + 4 * e, tok = at >> p.pack_log2;
            if (tok < last)
              *reinterpret_cast<uint4*>(base + tok * p.out_stride + (at & mask) * D + 64 * h) = u[e];
          }
        }
      }
      tc_fence_before();   // this group's O reads precede the next item's first P_i V product
    }
    // if a wait gave up, the remaining rows stay unwritten and the error word records it
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}


typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encoder = nullptr;

void look_up_encoder() {
  void* ptr = nullptr;
  cudaDriverEntryPointQueryResult q{};
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    g_encoder = reinterpret_cast<EncodeTiledFn>(ptr);
}

// bf16 tensor map over `rank` (3 or 4) dimensions, innermost first, with 128-byte swizzle and zeros out of
// bounds; strides: bytes between elements of dimensions 1 .. rank - 1.  False if the driver's encoder is
// unavailable or rejects the map.
bool encode_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                const cuuint32_t* box) {
  static pthread_once_t once = PTHREAD_ONCE_INIT;
  pthread_once(&once, look_up_encoder);
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return g_encoder != nullptr &&
         g_encoder(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Packed q: [tokens][head blocks of 2^s][D] bf16 rows `stride` elements apart, as
// (column, head of the block, token, head block); a box is one query tile.
bool make_map_packed_q(CUtensorMap* m, const void* base, int D, int tokens, int head_blocks, int pack_log2,
                       long long stride) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), 1ull << pack_log2, static_cast<cuuint64_t>(tokens),
                              static_cast<cuuint64_t>(head_blocks)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2,
                                 (static_cast<cuuint64_t>(D) << pack_log2) * 2};
  const cuuint32_t box[4] = {64, 1u << pack_log2, static_cast<cuuint32_t>(BM >> pack_log2), 1};
  return encode_map(m, base, 4, dims, strides, box);
}

// Packed k or v: [tokens][Hkv][D] bf16 rows `stride` elements apart, as (column, token, head).
bool make_map_packed_kv(CUtensorMap* m, const void* base, int D, int tokens, int Hkv, long long stride, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(tokens),
                              static_cast<cuuint64_t>(Hkv)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride) * 2, static_cast<cuuint64_t>(D) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  return encode_map(m, base, 3, dims, strides, box);
}

// One-time set-up of a kernel on the current device: its shared-memory limit, and the check
// that setmaxnreg.inc can be honoured (as the dense kernel's).
template <int D, bool PAGED, bool SPLIT, bool RUNS>
cudaError_t prepare_kernel() {
  using C = Cfg<D>;
  constexpr int kMaxDevices = 64;
  static int ready[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (__atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE) == 1) return cudaSuccess;
  auto kern = prefill_packed_kernel<D, PAGED, SPLIT, RUNS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa{};
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * C::THREADS < 128 * (2 * C::SOFTMAX_REGS + C::PRODUCER_REGS))
    return cudaErrorInvalidConfiguration;
  __atomic_store_n(&ready[dev], 1, __ATOMIC_RELEASE);
  return cudaSuccess;
}

template <int D, bool PAGED, bool SPLIT, bool RUNS>
cudaError_t launch_s(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const Params& p,
                     cudaStream_t stream) {
  using C = Cfg<D>;
  auto kern = prefill_packed_kernel<D, PAGED, SPLIT, RUNS>;
  cudaError_t e = prepare_kernel<D, PAGED, SPLIT, RUNS>();
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const unsigned grid = static_cast<unsigned>(min(p.n_items, sms));
  return launch_dependent(kern, dim3(grid), dim3(C::THREADS), C::SMEM, stream, mq, mk, mv, p);
}

// Joins the parts of each row of a sequence: a warp a row, its lanes over the columns.
template <int D>
__global__ void __launch_bounds__(128) prefill_packed_combine_kernel(const Params p) {
  constexpr int PER = D / 32;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();   // the parts
  const int t = static_cast<int>(row / p.Hq);
  if (t >= p.Tq || t < p.cu_q[0] || t >= p.cu_q[p.B]) return;   // rows of no sequence stay as they are
  const long long rows = static_cast<long long>(p.Tq) * p.Hq;
  const float lse = lane < p.splits ? p.ws_lse[lane * rows + row] : -INFINITY;   // at most 16 parts
  float M = lse;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float w = (lse == -INFINITY) ? 0.f : ex2(lse - M);
  float sum = w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  float acc[PER];
#pragma unroll
  for (int c = 0; c < PER; ++c) acc[c] = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float ws = __shfl_sync(0xffffffffu, w, s);
    if (ws == 0.f) continue;   // (a part without keys wrote no row)
    const float* src = p.ws_o + (s * rows + row) * D + lane * PER;
#pragma unroll
    for (int c = 0; c < PER; ++c) acc[c] = fmaf(ws, src[c], acc[c]);
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int h = static_cast<int>(row - static_cast<long long>(t) * p.Hq);
  __nv_bfloat16* dst = p.out + t * p.out_stride + static_cast<long long>(h) * D + lane * PER;
#pragma unroll
  for (int c = 0; c < PER; c += 2)
    *reinterpret_cast<uint32_t*>(dst + c) = pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
}

template <int D, bool PAGED>
cudaError_t launch_d(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const Params& p, bool runs,
                     cudaStream_t stream) {
  if (p.splits <= 1)
    return runs ? launch_s<D, PAGED, false, true>(mq, mk, mv, p, stream)
                : launch_s<D, PAGED, false, false>(mq, mk, mv, p, stream);
  const cudaError_t e = runs ? launch_s<D, PAGED, true, true>(mq, mk, mv, p, stream)
                             : launch_s<D, PAGED, true, false>(mq, mk, mv, p, stream);
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(p.Tq) * p.Hq;   // few: a split has at most 148 items of 256 rows
  return launch_dependent(prefill_packed_combine_kernel<D>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0,
                          stream, p);
}

// Whether an item may have more key tiles than one accumulation sums well: from the longest sequence that
// the buffers or the caller's bound allow, and the window (an item of n tokens sees window + n - 1 keys).
bool needs_runs(const Params& p, int max_keys) {
  long long tiles = (static_cast<long long>(max_keys) + BN - 1) / BN;
  if (p.causal && p.window > 0) tiles = min(tiles, (static_cast<long long>(p.window) + NQ * BM) / BN + 2);
  return tiles > static_cast<long long>(kOneRun) * p.splits;
}

// 2^s query heads of a kv head share a tile: the largest power of two that divides the group, at most 128.
int pack_log2_of(int Hq, int Hkv) {
  int s = 0;
  while (s < 7 && ((Hq / Hkv) & (1 << s)) == 0) ++s;
  return s;
}

// Sequences of any lengths make at most Tq / block + B query blocks; times the head blocks.
long long item_bound(int B, int Tq, int Hq, int Hkv) {
  const int s = pack_log2_of(Hq, Hkv);
  const int block = (BM >> s) * NQ;
  return (static_cast<long long>(Tq) / block + B) * (Hq >> s);
}

}  // namespace

// The items that the key tiles of an item are dealt to, from the sizes alone (sequences taken as
// equally long).  All parts run at once (148 SMs): 8 sequences x 16 new tokens over 8192 keys, 32/8
// heads, took 153 us whole, 86 in 2 parts (128 items) and 114 in 3; 4 such sequences 151, 86, 64
// and 50 us in 1 to 4 parts; 2 sequences x 9 tokens, 8/2 heads, 145 us whole and 22 in 16.  With
// the tiles mostly empty (few rows) a part may be a single key tile: 600 keys took 15.9 us whole
// and 12.3 in 5.  With full tiles the parts' rows cost as much to write and join as 4 key
// tiles: a 512-token prompt, 12 heads, took 13.5 us whole and 17.2 in 2, 1024 tokens 20.6 and 19.4.
// With a window (causal) an item has no more parts than key tiles that it sees, and is whole if they are 3: 2
// sequences x 9 tokens over 8192 keys, 8/2 heads, took 12.1 us whole and 12.6 in 16 parts with a window
// of 128, 9.4 and 12.1 with one of 32; 15.0 and 12.8 with one of 256, 4 key tiles.
int packed_splits(int B, int Tq, int Hq, int Hkv, int max_seq_len, int window) {
  if (B <= 0 || Tq <= 0 || Hq <= 0 || Hkv <= 0) return 1;
  const int s = pack_log2_of(Hq, Hkv);
  const int block = (BM >> s) * NQ;
  const long long each = (static_cast<long long>(Tq) + B - 1) / B;
  const long long items = (each + block - 1) / block * B * (Hq >> s);
  const int tiles = (max_seq_len + BN - 1) / BN;
  long long seen = tiles;
  if (window > 0) {   // n tokens see window + n - 1 keys in a row: the tiles that those may touch
    const long long keys = window + (each < block ? each : block) - 1;
    if ((keys + BN - 2) / BN + 1 < seen) seen = (keys + BN - 2) / BN + 1;
  }
  if (seen < 4) return 1;
  const bool few_rows = static_cast<long long>(Tq) * Hq <= items * (NQ * BM / 4);
  long long parts = 148 / items;
  const int most = few_rows ? tiles : tiles / 4;
  if (parts > most) parts = most;
  if (parts > seen) parts = seen;
  if (parts > 16) parts = 16;
  return parts < 2 ? 1 : static_cast<int>(parts);
}

size_t packed_workspace_bytes(int B, int Tq, int Hq, int Hkv, int D, int max_seq_len) {
  const int s = packed_splits(B, Tq, Hq, Hkv, max_seq_len, 0);   // (a window never means more parts)
  return s < 2 ? 0 : static_cast<size_t>(s) * Tq * Hq * (D + 1) * sizeof(float);
}

namespace {

// What the packed launches share: the head packing, the item bound that sizes the grid, the
// split, and the fields of Params that do not depend on where K and V lie.
bool packed_params(Params& p, void* out, float* lse, const int32_t* cu_q, int B, int Hq, int Hkv, int D, int Tq,
                   int max_seq_len, long long out_stride, float scale, int causal, int window, void* workspace,
                   unsigned int* err) {
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Tq = Tq;
  p.causal = causal;
  p.window = window;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.err = err;
  p.cu_q = cu_q;
  p.out_stride = out_stride;
  p.pack_log2 = pack_log2_of(Hq, Hkv);
  p.head_blocks = Hq >> p.pack_log2;
  // the caller's workspace decides whether an item is split (none: never)
  p.splits = workspace != nullptr ? packed_splits(B, Tq, Hq, Hkv, max_seq_len, window) : 1;
  p.ws_o = static_cast<float*>(workspace);
  if (p.splits > 1) p.ws_lse = p.ws_o + static_cast<size_t>(p.splits) * Tq * Hq * D;
  // items are counted in int32, with room for one more round of the grid
  const long long items = item_bound(B, Tq, Hq, Hkv) * p.splits;
  if (items > (1LL << 30)) return false;
  p.n_items = static_cast<int>(items);
  return true;
}

}  // namespace

cudaError_t launch_prefill_tc_packed(const void* q, const void* k, const void* v, const int32_t* cu_q,
                                     const int32_t* cu_k, int B, int Tq, int Tk, int Hq, int Hkv, int D,
                                     long long q_stride, long long k_stride, long long v_stride, long long out_stride,
                                     float scale, int causal, int window, void* workspace, void* out, float* lse,
                                     unsigned int* err, cudaStream_t stream) {
  Params p{};
  if (!packed_params(p, out, lse, cu_q, B, Hq, Hkv, D, Tq, keys_each(Tk, B), out_stride, scale, causal, window,
                     workspace, err))
    return cudaErrorNotSupported;
  p.cu_k = cu_k;
  p.Tk = Tk;
  CUtensorMap mq, mk, mv;
  // without keys the k and v maps are never used: any valid address will do
  const void* kb = Tk > 0 ? k : q;
  const void* vb = Tk > 0 ? v : q;
  const int rows = Tk > 0 ? Tk : 1;
  if (!make_map_packed_q(&mq, q, D, Tq, p.head_blocks, p.pack_log2, q_stride) ||
      !make_map_packed_kv(&mk, kb, D, rows, Hkv, k_stride, BN) ||
      !make_map_packed_kv(&mv, vb, D, rows, Hkv, v_stride, BN))
    return cudaErrorInvalidValue;
  const bool runs = needs_runs(p, Tk);
  return D == 64 ? launch_d<64, false>(mq, mk, mv, p, runs, stream) : launch_d<128, false>(mq, mk, mv, p, runs, stream);
}

cudaError_t launch_prefill_tc_packed_paged(const void* q, const void* k_pool, const void* v_pool, const int32_t* cu_q,
                                           const int32_t* page_table, const int32_t* seq_lens, int page_size, int B,
                                           int Tq, int Hq, int Hkv, int D, long long q_stride, long long out_stride,
                                           int num_pages, int max_pages, int max_seq_len, float scale, int causal,
                                           int window, void* workspace, void* out, float* lse, unsigned int* err,
                                           cudaStream_t stream) {
  Params p{};
  if (!packed_params(p, out, lse, cu_q, B, Hq, Hkv, D, Tq, max_seq_len, out_stride, scale, causal, window, workspace,
                     err))
    return cudaErrorNotSupported;
  p.max_seq_len = max_seq_len;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.page_size = page_size;
  p.box_rows = page_size < BN ? page_size : BN;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  CUtensorMap mq, mk, mv;
  // with max_seq_len 0 nothing is cached and the pools' maps are never used
  const bool any = max_seq_len > 0;
  if (!make_map_packed_q(&mq, q, D, Tq, p.head_blocks, p.pack_log2, q_stride) ||
      !make_tensor_map_3d(&mk, any ? k_pool : q, 2, D, page_size, any ? num_pages * Hkv : 1, 64, p.box_rows) ||
      !make_tensor_map_3d(&mv, any ? v_pool : q, 2, D, page_size, any ? num_pages * Hkv : 1, 64, p.box_rows))
    return cudaErrorInvalidValue;
  const long long room = static_cast<long long>(max_pages) * page_size;
  const bool runs = needs_runs(p, room < max_seq_len ? static_cast<int>(room) : max_seq_len);
  return D == 64 ? launch_d<64, true>(mq, mk, mv, p, runs, stream) : launch_d<128, true>(mq, mk, mv, p, runs, stream);
}

}  // namespace attn

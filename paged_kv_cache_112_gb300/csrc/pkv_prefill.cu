// Attention of many tokens of each sequence over its paged history: prompts,
// chunks of prompts behind a cached prefix, a few drafted tokens.
//
// The n new tokens of sequence s (rows query_start[s] .. of q) are the last n
// of its L; the query of token i, head h sits at position p = L - n + i and sees
//     t <= p and (no window, or t > p - window, or t < sinks):
//     out = sum_t softmax_t(scale * q . k_t) v_t.
//
// Bound: the two products, 4 D flops a visible (query, head, token) on the
// tensor cores; and next to them 32 exponentials a SM and cycle.  8192 tokens of
// 32 + 8 heads of 128: 376 us, 1.46 PFLOP/s; a step of 128 history tokens for two
// tiles takes some 2900 cycles, the products alone 2048.
//
// A CTA works on two tiles of 128 query rows of one KV head: the group's G heads
// of 128 / G tokens, rows ordered (token, head), so that K and V are read once
// for the whole group.  It walks the visible 128-token tiles of the history:
//     S = Q K^T        tcgen05.mma, both from shared memory, S in tensor memory;
//     P = 2^(S - m)    one thread a row, the running maximum and sum in
//                      registers; P goes back as 16-bit pairs;
//     O += P V         tcgen05.mma, P from tensor memory.
// Warps 0 to 3 and 4 to 7 are the threads of the two tiles: while one tile's
// are at the exponentials, the tensor cores work on the other's products.
// Warps 8 and 10 load K and V: TMA boxes of a block's rows of a head, scattered
// by the block table, into a ring of tiles; warp 11 passes a tile on, once it
// has zeroed what nobody sees of it; a thread of warp 9 issues the products.
//
// P overwrites the first half of S.  (With S of the next keys issued in halves,
// one of them beside the exponentials, the products take 48 instructions an
// iteration in place of 32, and the issuing thread is what everybody waits for:
// 690 us for 8192 tokens instead of 400.)  (Leaving out halves of a
// tile that no row sees costs more, in branches and registers, than it saves:
// 413 and 232 us for 384 and 218 at 8192 tokens and 16 windowed prompts.)
//
// The grid has a CTA for each pair of tiles; those on the SMs take over the
// others' work one after another (clusterlaunchcontrol), so that the next
// pair's loads and first products run beside the last rows' stores.
//
// m is raised, and O scaled in tensor memory, only when the row's maximum has
// grown by more than 2^8 since: weights up to 2^8 do as well (a weight is
// rounded relative to itself), and O is read and written rarely.
//
// A row's weight for a token that it does not see is 0, and 0 times an infinite or
// NaN value would be NaN.  Where some rows of a pair see a token and others do not,
// warp 11 looks for such values, makes them 0 and keeps a list of their tokens; the
// rows that see one get it added once the products are done.  (Without all that
// 8192 tokens took 351 us for 358, 16 windowed prompts 172 for 175, 200 prompts of
// 20 tokens behind 50, where warp 11 is what the others wait for, 59 for 64.)
//
// With few query rows a cluster of up to eight CTAs shares a pair of tiles:
// each takes every C-th tile of the history, and their rows meet in distributed
// shared memory.
#include <algorithm>
#include <atomic>

#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

using namespace dev;

constexpr int kRows = 128;     // query rows a tile
constexpr int kKeys = 128;     // history tokens a tile
constexpr int kThreads = 384;  // two tiles' threads, and four warps that load, pass on and multiply
// Registers: 168 a thread at launch; the tiles' threads hold a row of scores.  (216
// and 72: 16 windowed prompts 179 us for 175, 8192 tokens 365 for 358.)
constexpr int kRowRegs = 200, kOtherRegs = 104;
static_assert(256 * kRowRegs + 128 * kOtherRegs <= 384 * 168, "shares of the launch's registers");
constexpr int kMaxCluster = 8;
// Tokens of a pair whose values are not all finite: the number of history tiles
// with some, then of each the place where it begins and a bit a token.  Only tiles
// at the edges of the rows' views are listed: at most 255 tokens lie between the
// first row's end and the last one's, as many between the window's two starts.
constexpr int kListTiles = 6, kListWords = 1 + 5 * kListTiles;

template <int D>
struct Smem {
  static constexpr int kLines = D / 64;                 // 128-byte lines of a row
  static constexpr int kLineBytes = kRows * 128;        // one line of a tile's rows
  static constexpr int kTileBytes = kLines * kLineBytes;
  static constexpr int kSlots = D == 128 ? 5 : 8;       // K and V tiles in flight
  static constexpr int kRing = 2 * kTileBytes;          // after the two query tiles
  static constexpr int kRowState = 0;                   // the cluster's meeting, over the tiles: max and sum of 256 rows,
  static constexpr int kRowsAt = 2048;                  // then 256 x [D] floats, 4 KB a warp
  static constexpr int kStolen = kRing + kSlots * kTileBytes;
  static constexpr int kUnits = kStolen + 16;           // two units of work
  static constexpr int kBars = kUnits + 64;
  static constexpr int kBarCount = 3 * kSlots + 18;
  static constexpr int kWords = kBars + 8 * kBarCount;  // bad blocks of each slot, tensor memory, abort
  static constexpr int kLists = kWords + 4 * (kSlots + 2);
  static constexpr int kBytes = kLists + 2 * 4 * kListWords;
  static_assert(kRowsAt + 2 * kRows * D * 4 + 8 * 4096 <= kStolen, "the cluster's rows fit over the tiles");
  static_assert(kBytes <= 232448, "shared memory of a CTA");
};

__device__ __forceinline__ uint4 load16(uint32_t at) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ void store16(uint32_t at, uint4 x) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}

// 0 for two finite 16-bit values, NaN in the half of one that is not; added to `sum`.
template <bool BF16>
__device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t sum) {
  if constexpr (BF16)
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(x), "r"(0));
  else
    asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(x), "r"(0));
  return sum;
}
// Two 16-bit values, those that are no finite numbers 0.
template <bool BF16>
__device__ __forceinline__ uint32_t finite(uint32_t x) {
  constexpr uint32_t kOdd = BF16 ? 0x7f80u : 0x7c00u;  // magnitudes from here on
  return ((x & 0x7fffu) >= kOdd ? 0u : x & 0xffffu) | (((x >> 16) & 0x7fffu) >= kOdd ? 0u : x & 0xffff0000u);
}

// A pair of tiles of one KV head.
struct Unit {
  int s, g;          // sequence (-1: no more units), KV head
  int first, n;      // first new token of the pair, the sequence's new tokens
  int row0, len;     // the sequence's first row, its length
  int pad[2];
};
static_assert(sizeof(Unit) == 32, "two units in shared memory");

// What the rows of a pair of tiles see.  The history's tiles of 128 are cut from
// an axis of the blocks that some row sees: those of the first tokens, then
// those of the window, with no gap between (tokens 0 .. mid - 1, then mid + gap
// and on).
struct View {
  int per_tile, tokens, ntiles;  // tokens a tile holds, of this pair, tiles with any
  int p0, p1;                    // positions of the pair's first and last token
  int window, sinks_all;
  int low, sinks;                // some row sees [0, sinks) and [low, p1]
  int mid, gap;
  int end, cnt;                  // the axis' length, this CTA's number of tiles
  int C, rank;

  __device__ __forceinline__ View(const Unit& u, const PrefillArgs& pa, int tile_tokens, int block_shift, int c, int r)
      : per_tile(tile_tokens), window(pa.window), C(c), rank(r) {
    tokens = min(2 * per_tile, u.n - u.first);
    ntiles = tokens > per_tile ? 2 : 1;
    p0 = u.len - u.n + u.first;
    p1 = p0 + tokens - 1;
    sinks_all = window > 0 ? pa.sinks : 0;
    low = low_of(p0);
    sinks = min(sinks_all, low);
    const int first = (sinks + (1 << block_shift) - 1) >> block_shift, from = low >> block_shift;  // blocks
    mid = from > first ? first << block_shift : 0;
    gap = from > first ? (from - first) << block_shift : 0;
    end = max(0, p1 + 1 - gap);
    const int count = (end + kKeys - 1) / kKeys;
    cnt = count > rank ? (count - rank + C - 1) / C : 0;
  }
  // The first token of the window at position p (which may lie before the history: p - window need not fit).
  __device__ __forceinline__ int low_of(int p) const { return window > 0 && p >= window ? p - window + 1 : 0; }
  // Where tile j begins on the axis; the token at a place of the axis.
  __device__ __forceinline__ int begin(int j) const { return (j * C + rank) * kKeys; }
  __device__ __forceinline__ int token(int x) const { return x < mid ? x : x + gap; }
  // Places from low - gap on, and those before `sinks`, are seen by some row.
  __device__ __forceinline__ bool seen(int x) const { return x < end && (x >= low - gap || x < sinks); }
  // Places in [all_from(), all_to()), and those of them before sinks_all, are seen by every row.  (Where there is a
  // gap, sinks_all ends before it.)
  __device__ __forceinline__ int all_from() const { return low_of(p1) - gap; }
  __device__ __forceinline__ int all_to() const { return p0 + 1 - gap; }
};

// TWO: a softmax weight enters the product in two 16-bit parts, its rounding and
// what that leaves (2^-17 of it in bf16, 2^-22 in f16), for outputs in 32 bits.  A
// 16-bit output takes the first part alone, off by half a step of its own type
// and, over many tokens, by less of the row than the row's rounding (errors
// against 64 bits: 2.1e-3 for 1.6e-3 in bf16, 2.7e-4 for 2.1e-4 in f16): the second
// part is half as much work again for the tensor cores.  Microseconds with one
// and two: 8192 tokens 363 and 529, 16 windowed prompts 196 and 247, 37 behind
// 2000 16.2 and 18.1 (32-bit outputs both).  Either way the sum is that of the weights
// before their rounding: adding up the rounded ones, which would give a row of one
// token that token's values to the bit, took 381 for 347 at 8192 tokens.
template <int D, bool BF16, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const DecodeArgs a, const PrefillArgs pa,
                                                              const __grid_constant__ CUtensorMap tmap_q,
                                                              const __grid_constant__ CUtensorMap tmap_k,
                                                              const __grid_constant__ CUtensorMap tmap_v) {
  using SM = Smem<D>;
  constexpr int NS = SM::kSlots, NL = SM::kLines;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_misaligned(smem, a.dev_status)) return;  // the same for every CTA
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const uint32_t base = smem_u32(smem), stolen = base + SM::kStolen;
  const uint32_t full = base + SM::kBars, ready = full + 8 * NS, empty = ready + 8 * NS, q_bar = empty + 8 * NS,
                 q_free = q_bar + 8, s_bar = q_free + 8, p_bar = s_bar + 16, o_bar = p_bar + 32, o_free = o_bar + 16,
                 u_full = o_free + 16, u_empty = u_full + 16, steal_bar = u_empty + 16, drain_bar = steal_bar + 8;
  volatile Unit* units = reinterpret_cast<volatile Unit*>(smem + SM::kUnits);
  volatile uint32_t* bad_blocks = reinterpret_cast<volatile uint32_t*>(smem + SM::kWords);
  volatile uint32_t* tmem_at = bad_blocks + NS;
  volatile uint32_t* abort_at = tmem_at + 1;
  volatile uint32_t* lists = reinterpret_cast<volatile uint32_t*>(smem + SM::kLists);  // of two units
  const int G = a.group, per_tile = kRows / G;

  if (tid == 0) {
    *abort_at = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(ready + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    mbar_init(q_bar, 1);
    mbar_init(q_free, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_bar + 8 * t, 1);
      mbar_init(p_bar + 16 * t, kRows);
      mbar_init(p_bar + 16 * t + 8, kRows);
      mbar_init(o_bar + 8 * t, 1);
      mbar_init(o_free + 8 * t, kRows);
      mbar_init(u_full + 8 * t, 1);
      mbar_init(u_empty + 8 * t, 11);  // the eight warps of rows, the loading warps, the issuing thread
    }
    mbar_init(steal_bar, 1);
    mbar_init(drain_bar, 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 9) {
    tc::alloc(smem_u32(const_cast<uint32_t*>(tmem_at)), 512);
    tc::fence_before();
  }
  griddep_wait();  // what is above touches nothing that the last kernel writes
  griddep_launch_dependents();
  __syncthreads();
  tc::fence_after();
  constexpr uint32_t tmem = 0;  // all of it, so it begins at 0
  const bool odd_memory = *tmem_at != tmem;
  if (odd_memory && tid == 0) flag(a.dev_status, 32u);  // PKV_DEV_ERR_SMEM: nothing is done

  // Waits for the phase; gives up at the time limit, or when another thread has.
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    for (;;) {
      for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
      if (*abort_at) return false;
      if (static_cast<long long>(global_timer_ns() - t0) > a.timeout_ns) {
        *abort_at = 1;
        flag(a.dev_status, 16u);  // PKV_DEV_ERR_TIMEOUT; the output is undefined
        return false;
      }
    }
  };
  auto signal = [](uint32_t bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory"); };
  // Unit k of this CTA, from warp 11; false: none, or given up.
  auto next_unit = [&](int k, Unit& u) {
    if (odd_memory) return false;
    if (!wait(u_full + 8 * (k & 1), (k >> 1) & 1)) return false;
    const volatile Unit& v = units[k & 1];
    u.s = v.s;
    u.g = v.g;
    u.first = v.first;
    u.n = v.n;
    u.row0 = v.row0;
    u.len = v.len;
    return u.s >= 0;
  };
  bool met = false;  // there was a unit

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8 || warp == 10) {
      // -------------------------------------------------------------- loads
      // K tiles are 0, 2, 4, ... of the ring, V tiles 1, 3, 5, ...
      const bool is_v = warp == 10;
      const CUtensorMap* map = is_v ? &tmap_v : &tmap_k;
      const int B = 1 << a.block_shift, nblk = kKeys >> a.block_shift;  // blocks of a tile: 2 to 16, one a lane
      Unit u;
      int i = is_v, loaded = 0, k = 0;  // this warp's next tile of the ring; pairs of query tiles
      bool ok = true;
      for (; ok && __all_sync(kFull, next_unit(k, u)); ++k) {
        __syncwarp();
        if (lane == 0) signal(u_empty + 8 * (k & 1));
        met = true;
        const View v(u, pa, per_tile, a.block_shift, C, rank);
        const int32_t* tbl = a.block_tables + static_cast<int64_t>(u.s) * a.max_blocks_per_seq;
        auto entry = [&](int j) {  // this lane's block of tile j: physical block, -1 where no row sees it, -2 outside the pool
          if (j >= v.cnt || lane >= nblk) return -1;
          const int x = v.begin(j) + lane * B;
          if (x >= v.end || !(x + B > v.low - v.gap || x < v.sinks)) return -1;
          const int phys = __ldg(tbl + (v.token(x) >> a.block_shift));
          return static_cast<unsigned>(phys) < static_cast<unsigned>(a.num_blocks) ? phys : -2;
        };
        int phys = entry(0);
        if (!is_v && v.cnt > 0) {
          ok = __all_sync(kFull, wait(q_free, (loaded & 1) ^ 1));
          if (!ok) break;
          if (tc::elect_one()) {
            mbar_arrive_expect_tx(q_bar, v.ntiles * NL * per_tile * G * 128);
            for (int t = 0; t < v.ntiles; ++t)
              for (int l = 0; l < NL; ++l)
                tma_load_4d(base + t * SM::kTileBytes + l * SM::kLineBytes, &tmap_q, 0, l, u.g * G,
                            u.row0 + u.first + t * per_tile, q_bar);
          }
          __syncwarp();
          ++loaded;
        }
        for (int j = 0; j < v.cnt; ++j, i += 2) {
          const uint32_t bad = __ballot_sync(kFull, phys == -2), there = __ballot_sync(kFull, phys >= 0);
          if (bad && lane == 0) flag(a.dev_status, 4u);  // PKV_DEV_ERR_BLOCK; the block counts as zeros
          const int slot = i % NS;
          const uint32_t bar = full + 8 * slot, dst = base + SM::kRing + slot * SM::kTileBytes;
          ok = __all_sync(kFull, wait(empty + 8 * slot, ((i / NS) & 1) ^ 1));
          if (!ok) break;
          if (lane == 0) {
            bad_blocks[slot] = bad;
            mbar_arrive_expect_tx(bar, __popc(there) * NL * B * 128);
          }
          __syncwarp();
          for (int b = 0; b < nblk; ++b) {
            if (!((there >> b) & 1u)) continue;
            const int block = __shfl_sync(kFull, phys, b);
            if (tc::elect_one()) {
#pragma unroll
              for (int l = 0; l < NL; ++l)
                tma_load_4d(dst + l * SM::kLineBytes + b * B * 128, map, 0, 0, u.g * NL + l, block, bar);
            }
          }
          phys = entry(j + 1);
        }
      }
      if (*abort_at && lane == 0) {  // copies in flight land before the CTA leaves
        if (!is_v && loaded > 0) mbar_wait_bounded(q_bar, (loaded - 1) & 1, a.timeout_ns);
        for (int b = i - 2; b >= 0 && b > i - 2 - NS; b -= 2)
          mbar_wait_bounded(full + 8 * (b % NS), (b / NS) & 1, a.timeout_ns);
      }
    } else if (warp == 11) {
      // ------------------------------------------------ units, and what is there
      // Unit x in launch order: pairs of tiles from the last sequence's last
      // (whose history is longest) to the first, the KV heads of each together.
      auto find = [&](int x) {
        Unit r{-1, 0, 0, 0, 0, 0, {0, 0}};
        const int S = a.num_seqs, per_pair = 2 * per_tile;
        r.g = x % a.num_kv_heads;
        int before = x / a.num_kv_heads;  // pairs still to pass over
        for (int top = S - 1; top >= 0; top -= 32) {
          const int s = top - lane;
          int lo = 0, n = 0, len = 0;
          if (s >= 0) {
            const int from = pa.query_start[s], to = pa.query_start[s + 1];
            len = a.context_lens[s];
            lo = min(max(from, 0), pa.num_tokens);
            const int hi = min(max(to, lo), pa.num_tokens);
            n = hi - lo;
          }
          const int mine = (n + per_pair - 1) / per_pair;
          int incl = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
          }
          const uint32_t at = __ballot_sync(kFull, incl > before);
          if (at == 0) {
            before -= __shfl_sync(kFull, incl, 31);
            continue;
          }
          const int who = __ffs(at) - 1;
          const int first = (mine - 1 - (before - (incl - mine))) * per_pair;
          if (lane == who) {
            const bool report = first == 0 && r.g == 0 && rank == 0;
            len = clamp_len(a, len, report);
            if (report && len < n) flag(a.dev_status, 8u);  // PKV_DEV_ERR_LENGTH
          }
          r.s = __shfl_sync(kFull, s, who);
          r.first = __shfl_sync(kFull, first, who);
          r.n = __shfl_sync(kFull, n, who);
          r.row0 = __shfl_sync(kFull, lo, who);
          r.len = __shfl_sync(kFull, len, who);
          break;
        }
        return r;
      };
      // Publishes unit k for the other warps; false: given up.
      auto publish = [&](int k, const Unit& u) {
        if (!__all_sync(kFull, wait(u_empty + 8 * (k & 1), ((k >> 1) & 1) ^ 1))) return false;
        if (lane == 0) {
          volatile Unit& v = units[k & 1];
          v.s = u.s;
          v.g = u.g;
          v.first = u.first;
          v.n = u.n;
          v.row0 = u.row0;
          v.len = u.len;
          signal(u_full + 8 * (k & 1));
        }
        __syncwarp();
        return true;
      };
      int steals = 0;
      bool more = C == 1;  // clusters do the unit they were launched for
      auto steal = [&]() {
        if (lane == 0) {
          fence_proxy_async_smem();  // the last answer has been read
          mbar_arrive_expect_tx(steal_bar, 16);
          tc::steal_cta(stolen, steal_bar);
        }
        ++steals;
        __syncwarp();
      };
      // The next unit that exists, from a CTA that has not started.
      auto take = [&]() {
        Unit u{-1, 0, 0, 0, 0, 0, {0, 0}};
        while (more && u.s < 0) {
          more = __all_sync(kFull, wait(steal_bar, (steals - 1) & 1));
          if (!more) break;
          const int x = tc::stolen_cta(stolen);
          __syncwarp();
          more = x >= 0;
          if (more) {
            steal();
            u = find(x);
          }
        }
        return u;
      };
      if (more) steal();
      Unit u = find(blockIdx.x / C);
      if (u.s < 0) u = take();
      int i = 0;
      bool ok = publish(0, u);
      if (blockIdx.x == 0) {  // while the first tiles are on their way; a sequence without rows has no unit to report it
        for (int s = lane; s < a.num_seqs; s += 32) {
          const int from = pa.query_start[s], to = pa.query_start[s + 1];
          if (from < 0 || to < from || to > pa.num_tokens) flag(a.dev_status, 8u);  // PKV_DEV_ERR_LENGTH
        }
        __syncwarp();
      }
      for (int k = 0; ok && u.s >= 0; ++k) {
        met = true;
        const Unit after = take();
        if (!publish(k + 1, after)) break;
        const View v(u, pa, per_tile, a.block_shift, C, rank);
        // Rows that no row of queries sees and blocks outside the pool become
        // zeros: their weights are zero, but what the pool holds there may be
        // anything, and zero times NaN is NaN.  So do infinite and NaN values that
        // some rows see and others do not: the former get them from the list.
        volatile uint32_t* list = lists + (k & 1) * kListWords;
        int listed = 0;
        if (lane == 0) list[0] = 0;  // the unit before last, whose list this was, is done with
        const int all_from = v.all_from(), all_to = v.all_to();
        for (int j = 0; j < 2 * v.cnt && ok; ++j, ++i) {
          const int slot = i % NS;
          const bool is_v = j & 1;
          ok = __all_sync(kFull, wait(full + 8 * slot, (i / NS) & 1));
          if (!ok) break;
          const uint32_t bad = bad_blocks[slot];
          const int x0 = v.begin(j >> 1);
          const uint32_t at = base + SM::kRing + slot * SM::kTileBytes;
          // A row's 16-byte pieces, rotated by the row: other banks for other lanes.
          auto piece = [&](int r, int c) { return at + (c >> 3) * SM::kLineBytes + r * 128 + ((c + r) & 7) * 16; };
          const bool edge = is_v && (x0 + kKeys > v.end || (x0 < v.low - v.gap && x0 + kKeys > v.sinks));
          bool changed = bad || edge;
          if (changed) {
            for (int r = lane; r < kKeys; r += 32) {
              if (!((bad >> (r >> a.block_shift)) & 1u) && (!is_v || v.seen(x0 + r))) continue;
              for (int c = 0; c < NL * 8; ++c) store16(piece(r, c), make_uint4(0, 0, 0, 0));
            }
            __syncwarp();
          }
          if (is_v && (x0 < all_from || x0 + kKeys > all_to)) {
            // All lanes side by side over the rows of one range of places, then the other's.
            uint32_t nan = 0;
            const uint32_t col = at + ((lane >> 3) & (NL - 1)) * SM::kLineBytes + (lane & 7) * 16;
            int r = max(v.low - v.gap - x0, 0) + lane / (NL * 8), last = min(all_from - x0, kKeys);
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
#pragma unroll 4
              for (; r < last; r += 32 / (NL * 8)) {
                const uint4 w = load16(col + r * 128);
                nan = times_zero<BF16>(w.x, times_zero<BF16>(w.y, times_zero<BF16>(w.z, times_zero<BF16>(w.w, nan))));
              }
              r = max(all_to - x0, 0) + lane / (NL * 8);
              last = min(v.end - x0, kKeys);
            }
            if (__any_sync(kFull, nan != 0)) {
              changed = true;
              if (lane == 0 && listed < kListTiles) list[1 + 5 * listed] = x0;
#pragma unroll 1
              for (int r = lane; r < kKeys; r += 32) {
                const int x = x0 + r;
                bool odd = false;
                if (v.seen(x) && (x >= all_to || (x < all_from && x >= v.sinks_all))) {
#pragma unroll 1
                  for (int c = 0; c < NL * 8; ++c) {
                    const uint4 w = load16(piece(r, c));
                    const uint4 z = make_uint4(finite<BF16>(w.x), finite<BF16>(w.y), finite<BF16>(w.z), finite<BF16>(w.w));
                    odd |= w.x != z.x || w.y != z.y || w.z != z.z || w.w != z.w;
                    store16(piece(r, c), z);
                  }
                }
                const uint32_t m = __ballot_sync(kFull, odd);
                if (lane == 0 && listed < kListTiles) list[2 + 5 * listed + (r >> 5)] = m;
              }
              listed = min(listed + 1, kListTiles);
              if (lane == 0) list[0] = listed;
            }
          }
          if (changed) fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) signal(ready + 8 * slot);
        }
        u = after;
      }
      // No answer is on its way into shared memory when the CTA leaves.
      if (steals > 0 && lane == 0) mbar_wait_bounded(steal_bar, (steals - 1) & 1, a.timeout_ns);
    } else if (tc::elect_one()) {
      // ----------------------------------------------------------- products
      const uint32_t pv = tc::instr_desc(BF16, D, true, false);
      const uint32_t qk = tc::instr_desc(BF16, kKeys, false, pa.negate != 0);
      const uint64_t q_desc = tc::smem_desc(base, 16, 1024), k_desc = tc::smem_desc(base + SM::kRing, 16, 1024);
      const uint64_t v_desc = tc::smem_desc(base + SM::kRing, SM::kLineBytes, 1024);
      constexpr uint32_t kSlotStep = SM::kTileBytes >> 4;  // of a descriptor
      auto arrive = [&](int i) { return wait(ready + 8 * (i % NS), (i / NS) & 1); };
      auto scores = [&](int t, int slot) {  // S_t = Q_t K^T
        const uint64_t qd = q_desc + t * kSlotStep, kd = k_desc + slot * kSlotStep;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t off = ((s / 4) * SM::kLineBytes + (s % 4) * 32) >> 4;
          tc::mma_ss(tmem + t * kKeys, qd + off, kd + off, qk, s > 0);
        }
        tc::commit(s_bar + 8 * t);
      };
      int i = 0, pairs = 0, phase[2] = {0, 0}, outs[2] = {0, 0};
      Unit u;
      bool ok = true;
      for (int k = 0; ok && next_unit(k, u); ++k) {
        signal(u_empty + 8 * (k & 1));
        const View v(u, pa, per_tile, a.block_shift, C, rank);
        const int cnt = v.cnt, ntiles = v.ntiles;
        if (cnt == 0) continue;
        ok = wait(q_bar, pairs & 1) && arrive(i);
        if (!ok) break;
        ++pairs;
        tc::fence_after();
        for (int t = 0; t < ntiles; ++t) scores(t, i % NS);
        tc::commit(empty + 8 * (i % NS));
        if (cnt == 1) tc::commit(q_free);
        for (int t = 0; t < ntiles && ok; ++t) ok = wait(o_free + 8 * t, (outs[t]++ & 1) ^ 1);
        for (int j = 0; j < cnt && ok; ++j, i += 2) {
          const bool last = j + 1 == cnt;
          const int v_slot = (i + 1) % NS, k_slot = (i + 2) % NS;
          const uint64_t vd = v_desc + v_slot * kSlotStep;
          ok = arrive(i + 1) && (last || arrive(i + 2));
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t >= ntiles || !ok) break;
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // O_t += P_t V over keys 64 half .. + 63
              if (!wait(p_bar + 16 * t + 8 * half, phase[t] & 1)) {
                ok = false;
                break;
              }
              tc::fence_after();
#pragma unroll
              for (int s = 4 * half; s < 4 * half + 4; ++s) {
                tc::mma_ts(tmem + 256 + t * D, tmem + t * kKeys + 8 * s, vd + ((s * 2048) >> 4), pv,
                           s > 0 || j > 0);
                if (TWO) tc::mma_ts(tmem + 256 + t * D, tmem + t * kKeys + 64 + 8 * s, vd + ((s * 2048) >> 4), pv, true);
              }
            }
            if (!ok) break;
            ++phase[t];
            if (last)
              tc::commit(o_bar + 8 * t);
            else
              scores(t, k_slot);
          }
          if (!ok) break;
          tc::commit(empty + 8 * v_slot);
          if (!last) tc::commit(empty + 8 * k_slot);
          if (j + 2 == cnt) tc::commit(q_free);
        }
      }
      // Every product has completed before tensor memory is freed.
      tc::commit(drain_bar);
      mbar_wait_bounded(drain_bar, 0, a.timeout_ns);
    }
    __syncwarp();
    if (C > 1) {  // the barriers of the cluster's meeting
      __syncthreads();
      cluster_sync();
      cluster_sync();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    // -------------------------------------------------------------- softmax
    const int t = warp >> 2, r = tid & (kRows - 1);  // tile and row
    const int token = r / G;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t s_at = tmem + t * kKeys + lanes, o_at = tmem + 256 + t * D + lanes;
    const uint32_t my_s = s_bar + 8 * t, my_p = p_bar + 16 * t;
    constexpr float kGrow = 8.f;
    // f16 weights: times 2^7, so that small ones keep their bits (f16 ends at 2^-24).
    constexpr float kUp = BF16 ? 0.f : 7.f;
    const float sl2 = a.scale_log2, grow = kGrow / sl2;
    Unit u{-1, 0, 0, 0, 0, 0, {0, 0}};
    float m = kNegInf, l = 0.f;  // the row's reference, in scores; the sum of its weights
    int seen = 0, outs = 0, ntiles = 0;
    auto row_at = [&](int tile, int row) {  // element index of a live row's first channel
      const int tok = row / G;
      return ((static_cast<int64_t>(u.row0) + u.first + tile * per_tile + tok) * a.num_q_heads + u.g * G + (row - tok * G)) *
             D;
    };
    for (int k = 0; __all_sync(kFull, next_unit(k, u)); ++k) {
      __syncwarp();
      if (lane == 0) signal(u_empty + 8 * (k & 1));
      met = true;
      const View v(u, pa, per_tile, a.block_shift, C, rank);
      ntiles = v.ntiles;
      m = kNegInf;
      l = 0.f;
      if (t >= ntiles) {
        if (C > 1) break;  // keeps the unit
        continue;
      }
      const int pos = v.p0 + t * per_tile + token, my_low = v.low_of(pos), my_sinks = v.sinks_all;
      // The tile's rows: positions first .. last, the widest and the narrowest view.
      const int first = v.p0 + t * per_tile, last_low = v.low_of(first + per_tile - 1);
      bool ok = true;
      for (int j = 0; j < v.cnt; ++j, ++seen) {
        const int x0 = v.begin(j), t0 = v.token(x0), t1 = v.token(x0 + kKeys - 1);
        const bool whole = t1 - t0 == kKeys - 1 && t1 <= first && (t0 >= last_low || t1 < my_sinks);  // for every row
        uint32_t x[kKeys];
        float* y = reinterpret_cast<float*>(x);
        float mx = kNegInf;
        ok = __all_sync(kFull, wait(my_s, seen & 1));
        if (!ok) break;
        tc::fence_after();
        if (!whole) {  // 32 columns that some row does not see go back masked (a loop: this code runs rarely)
#pragma unroll 1
          for (int c = 0; c < kKeys; c += 32) {
            auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? kFull : (1u << n) - 1u; };
            auto from = [&](int at) {  // bit i: this row sees token at + i
              return below(pos + 1 - at) & (~below(my_low - at) | below(my_sinks - at));
            };
            const uint32_t before = below(v.mid - (x0 + c));
            const uint32_t see = (from(x0 + c) & before) | (from(x0 + c + v.gap) & ~before);
            if (__all_sync(kFull, see == kFull)) continue;
            uint32_t o[32];
            tc::ld32(o, s_at + c);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = (see >> i) & 1u ? o[i] : __float_as_uint(kNegInf);
            tc::st32(s_at + c, o);
          }
          tc::wait_st();
        }
        tc::ld32(x, s_at);
        tc::ld32(x + 32, s_at + 32);
        tc::wait_ld();
        tc::ld32(x + 64, s_at + 64);  // on their way while the first half's maximum is taken
        tc::ld32(x + 96, s_at + 96);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half == 1) tc::wait_ld();
          const float* z = y + 64 * half;
          float top[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
          for (int i = 4; i < 60; i += 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q) top[q] = fmaxf(fmaxf(top[q], z[i + q]), z[i + 4 + q]);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) top[q] = fmaxf(top[q], z[60 + q]);
          mx = fmaxf(mx, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
        }
        // The reference moves to mx where that lies far above it.
        const bool raise = mx > m + grow;  // a first one counts: m is -infinity
        if (__any_sync(kFull, raise)) {
          const float mn = raise ? mx : m;
          const float f = raise ? ex2_approx((m - mn) * sl2) : 1.f;  // 0 for a first one
          l *= f;
          m = mn;
          if (j > 0) {  // O is at rest: its last product came before these scores
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tc::ld32(o, o_at + c);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tc::st32(o_at + c, o);
            }
          }
        }
        const float shift = m == kNegInf ? 0.f : kUp - m * sl2;
        const F2 scale2 = pair(sl2, sl2), shift2 = pair(shift, shift);
        F2 sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
        [[maybe_unused]] uint32_t rest[16];
        auto weigh = [&](int i) {  // columns i, i + 1; with TWO, what rounding left of them to `rest`
          const float2 e = halves(fma2(pair(y[i], y[i + 1]), scale2, shift2));
          const float w0 = ex2_approx(e.x), w1 = ex2_approx(e.y);
          sum[(i / 2) & 1] = add2(sum[(i / 2) & 1], pair(w0, w1));
          const uint32_t p = BF16 ? pack_bf16(w0, w1) : pack_f16(w0, w1);
          if constexpr (TWO) {
            const float2 r = BF16 ? unpack_bf16(p) : __half22float2(*reinterpret_cast<const __half2*>(&p));
            const float2 z = halves(fma2(pair(r.x, r.y), pair(-1.f, -1.f), pair(w0, w1)));
            rest[(i / 2) & 15] = BF16 ? pack_bf16(z.x, z.y) : pack_f16(z.x, z.y);
          }
          return p;
        };
        auto pass = [&](int half) {  // the weights of this half are in tensor memory
          tc::wait_st();
          tc::fence_before();
          signal(my_p + 8 * half);
        };
        if constexpr (TWO) {
          uint32_t w[16];
#pragma unroll
          for (int part = 0; part < 4; ++part) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = weigh(32 * part + 2 * i);
            if (part == 2) pass(0);
            tc::st16(s_at + 16 * part, w);
            tc::st16(s_at + 64 + 16 * part, rest);
          }
          pass(1);
        } else {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = weigh(2 * i);
          tc::st32(s_at, w);
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = weigh(64 + 2 * i);
          pass(0);  // a while after its stores
#pragma unroll
          for (int i = 16; i < 32; ++i) w[i] = weigh(64 + 2 * i);
          tc::st32(s_at + 32, w);
          pass(1);
        }
        const float2 s0 = halves(sum[0]), s1 = halves(sum[1]);
        l += (s0.x + s0.y) + (s1.x + s1.y);
      }
      if (!ok) break;
      if (v.cnt > 0) {
        if (!__all_sync(kFull, wait(o_bar + 8 * t, outs++ & 1))) break;
        tc::fence_after();
      }
      // Values that the products left out (see warp 11): added for the rows that see their tokens.
      const volatile uint32_t* list = lists + (k & 1) * kListWords;
      if (__builtin_expect(v.cnt > 0 && list[0] != 0, 0)) {
        const int32_t* tbl = a.block_tables + static_cast<int64_t>(u.s) * a.max_blocks_per_seq;
#pragma unroll 1
        for (int e = 0; e < 4 * min(static_cast<int>(list[0]), kListTiles); ++e) {
          const int x = static_cast<int>(list[1 + 5 * (e >> 2)]) + 32 * (e & 3);
#pragma unroll 1
          for (uint32_t left = list[2 + 5 * (e >> 2) + (e & 3)]; left; left &= left - 1) {
            const int tok = v.token(x + __ffs(left) - 1);
            const bool sees = tok <= pos && (tok >= my_low || tok < my_sinks);
            const uint32_t* row = reinterpret_cast<const uint32_t*>(
                pa.v_pool + __ldg(tbl + (tok >> a.block_shift)) * a.block_stride +
                (static_cast<int64_t>(tok & ((1 << a.block_shift) - 1)) * a.num_kv_heads + u.g) * D);
#pragma unroll 1
            for (int c = 0; c < D; c += 8) {
              uint32_t o[8];
              tc::ld8(o, o_at + c);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 8; i += 2) {
                const uint32_t w = __ldg(row + (c + i) / 2);
                const float2 y = BF16 ? unpack_bf16(w) : __half22float2(*reinterpret_cast<const __half2*>(&w));
                if (sees && !(fabsf(y.x) < INFINITY)) o[i] = __float_as_uint(__uint_as_float(o[i]) + y.x);
                if (sees && !(fabsf(y.y) < INFINITY)) o[i + 1] = __float_as_uint(__uint_as_float(o[i + 1]) + y.y);
              }
              tc::st8(o_at + c, o);
              tc::wait_st();
            }
          }
        }
      }
      if (C > 1) break;  // the rows meet below
      const float f = l == 0.f ? 0.f : 1.f / l;  // a sum that is no number makes the row none
      const int eb = a.out_dtype == 0 ? 4 : 2;
      const bool live = token < per_tile && t * per_tile + token < v.tokens;
      uint8_t* mine = static_cast<uint8_t*>(a.out) +
                      (((static_cast<int64_t>(u.row0) + u.first + t * per_tile + token) * a.num_q_heads + u.g * G +
                        (r - token * G)) * D * eb);
      auto store8 = [&](uint8_t* to, const uint32_t (&x)[8]) {
        if (pa.out_sectors) {
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                       "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                       : "memory");
        } else {
          reinterpret_cast<uint4*>(to)[0] = make_uint4(x[0], x[1], x[2], x[3]);
          reinterpret_cast<uint4*>(to)[1] = make_uint4(x[4], x[5], x[6], x[7]);
        }
      };
      auto free_rows = [&]() {  // the next pair's products may begin
        if (v.cnt == 0) return;
        tc::fence_before();
        signal(o_free + 8 * t);
      };
      if (eb == 2) {
        // A quad of lanes has 64 channels of a row, every fourth pair each; two
        // exchanges give each lane 16 in a row, so that a store is eight lines of
        // 128 bytes.  (Each lane storing its own row: 32 lines a store, 5500
        // cycles a pair of tiles.)
        const uint32_t lives = __ballot_sync(kFull, live), empty_rows = __ballot_sync(kFull, l == 0.f);
        const bool up2 = lane & 2, up1 = lane & 1;
#pragma unroll 1
        for (int part = 0; part < D / 32; ++part) {  // 16 rows, 64 channels
          const int c = (part >> 1) * 64, half = part & 1;
          uint32_t o[32];
          tc::ld16x64(o, o_at + (static_cast<uint32_t>(half) << 20) + c);
          tc::wait_ld();
          if (part + 1 == D / 32) free_rows();
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = 16 * half + 8 * e + (lane >> 2);  // of the warp's
            const float fr = __shfl_sync(kFull, f, row);
            uint8_t* to = reinterpret_cast<uint8_t*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(mine), row));
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float x = __uint_as_float(o[4 * k + 2 * e]) * fr, y = __uint_as_float(o[4 * k + 2 * e + 1]) * fr;
              w[k] = a.out_dtype == 1 ? pack_f16(x, y) : pack_bf16(x, y);
              if ((empty_rows >> row) & 1u) w[k] = 0u;  // no visible token: whatever tensor memory holds
            }
            uint32_t h[8], z[8];  // after the exchange with the lane 2 further: [which of the two][k of four]
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t keep = up2 ? w[k + 4] : w[k], got = __shfl_xor_sync(kFull, up2 ? w[k] : w[k + 4], 2);
              h[k] = up2 ? got : keep;
              h[4 + k] = up2 ? keep : got;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int b = 0; b < 2; ++b) {  // lanes (b, own) and (b, the other's) of the quad
                const uint32_t keep = up1 ? h[4 * b + k + 2] : h[4 * b + k];
                const uint32_t got = __shfl_xor_sync(kFull, up1 ? h[4 * b + k] : h[4 * b + k + 2], 1);
                z[4 * k + 2 * b] = up1 ? got : keep;
                z[4 * k + 2 * b + 1] = up1 ? keep : got;
              }
            if ((lives >> row) & 1u) store8(to + 2 * c + 32 * (lane & 3), z);
          }
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tc::ld32(o, o_at + c);
          tc::wait_ld();
          if (c + 32 == D) free_rows();
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[8 * h + i]) * f);
            if (live) store8(mine + 4 * c + 32 * h, x);
          }
        }
      }
    }

    if (C > 1) {
      // The cluster's rows: each CTA scales its part to the rows' common maximum
      // and sends rows 256 / C i .. to CTA i, which adds the parts up.  32
      // channels of a warp's rows at a time are brought into order first, so that
      // a store's lanes lie side by side (16 bytes of 32 rows a store took 6600
      // cycles in place of 1600).
      float2* state = reinterpret_cast<float2*>(smem + SM::kRowState);
      float* inbox = reinterpret_cast<float*>(smem + SM::kRowsAt);  // [from][256 / C rows][D]
      const int tokens = met ? min(2 * per_tile, u.n - u.first) : 0, rows = 2 * kRows / C;
      __syncthreads();  // the tiles are no longer read
      state[tid] = make_float2(m, l);
      cluster_sync();
      if (t < ntiles && token < per_tile && t * per_tile + token < tokens) {
        float2 part[kMaxCluster];
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
          if (k < C)
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                         : "=f"(part[k].x), "=f"(part[k].y)
                         : "r"(cluster_map(smem_u32(state + tid), k))
                         : "memory");
        float top = kNegInf, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
          if (k < C) top = fmaxf(top, part[k].x);
        const float ref = top == kNegInf ? 0.f : top;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
          if (k < C) sum += part[k].y * ex2_approx((part[k].x - ref) * sl2);
        l = l == 0.f ? 0.f : ex2_approx((m - ref) * sl2) / sum;  // the factor of this part
      }
      const uint32_t stage = base + SM::kRowsAt + 2 * kRows * D * 4 + warp * 4096;  // 32 rows of 128 bytes
      const int owner = warp * 32 / rows, first_row = warp * 32 - owner * rows;
      const uint32_t to = cluster_map(smem_u32(inbox + (rank * rows + first_row) * D), owner);
      if (__any_sync(kFull, t < ntiles && token < per_tile && t * per_tile + token < tokens)) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tc::ld32(o, o_at + c);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            auto val = [&](int e) { return l == 0.f ? 0.f : __uint_as_float(o[4 * i + e]) * l; };
            *reinterpret_cast<float4*>(smem + (stage - base) + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                make_float4(val(0), val(1), val(2), val(3));
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = 4 * i + (lane >> 3);
            cluster_store_float4(to + (row * D + c) * 4 + 16 * (lane & 7),
                                 *reinterpret_cast<const float4*>(smem + (stage - base) + row * 128 +
                                                                  (((lane & 7) ^ (row & 7)) << 4)));
          }
          __syncwarp();
        }
      }
      cluster_sync();
      // 4 channels a thread, D / 4 threads a row.
      constexpr int kWidth = D / 4;
      const int ch = 4 * (tid % kWidth);
      for (int i = tid / kWidth; i < rows; i += 2 * kRows / kWidth) {
        const int row = rank * rows + i, tile = row / kRows, in = row & (kRows - 1), tok = in / G;
        if (tile >= ntiles || tok >= per_tile || tile * per_tile + tok >= tokens) continue;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
          if (k < C) {
            const float4 x = *reinterpret_cast<const float4*>(inbox + (k * rows + i) * D + ch);
            sum.x += x.x;
            sum.y += x.y;
            sum.z += x.z;
            sum.w += x.w;
          }
        const int64_t at = row_at(tile, in) + ch;
        if (a.out_dtype == 0)
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = sum;
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
              a.out_dtype == 1 ? make_uint2(pack_f16(sum.x, sum.y), pack_f16(sum.z, sum.w))
                               : make_uint2(pack_bf16(sum.x, sum.y), pack_bf16(sum.z, sum.w));
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

template <int D, bool BF16, bool TWO>
struct Launch {
  static constexpr auto kernel = prefill_kernel<D, BF16, TWO>;

  static int resident(int C) {
    constexpr int kDevices = 64;
    static std::atomic<int> cache[kDevices][4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) {
      cudaGetLastError();
      return 1;
    }
    std::atomic<int>& slot = cache[dev][C == 1 ? 0 : C == 2 ? 1 : C == 4 ? 2 : 3];
    int n = slot.load(std::memory_order_acquire);
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Smem<D>::kBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      return 1;
    }
    slot.store(n, std::memory_order_release);
    return n;
  }

  static cudaError_t launch(const DecodeArgs& a, const PrefillArgs& pa, const CUtensorMap& tq, const CUtensorMap& tk,
                            const CUtensorMap& tv, cudaStream_t stream) {
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), Smem<D>::kBytes);
    if (e != cudaSuccess) return e;
    const int per_pair = 2 * (kRows / a.group);
    // Pairs of tiles, at most: each sequence with one of a single token, all the others whole.
    const int64_t some = std::min<int64_t>(a.num_seqs, pa.num_tokens);
    const int64_t pairs = some + (pa.num_tokens - some) / per_pair;
    const int64_t units = pairs * a.num_kv_heads;
    int64_t longest = a.max_context_len;  // tokens that a pair of tiles sees
    if (pa.window > 0)  // its blocks' other tokens with them, at both ends
      longest = std::min(longest, static_cast<int64_t>(pa.window) + pa.sinks + per_pair + (2 << a.block_shift));
    const int64_t tiles = (longest + kKeys - 1) / kKeys;
    // Few pairs share their histories over clusters, unless the tiles saved take
    // less time than the rows' meeting.  A pair takes start + step * its CTA's
    // tiles (+ the meeting), microseconds, fitted at 1 to 16 sequences of 4 to 1024
    // new tokens behind 0 to 20000 and 1 to 8 KV heads: of 45 shapes, the choice
    // was within 2% of the fastest form in 44 and 9% off in one.  D = 128, 256
    // tokens alone: 10.9 without clusters, 15.3 in twos; 64 behind 2000: 31.3,
    // 26.3, 19.6 in fours, 18.2 in eights (18.7 now).  D = 64, 64 behind 500: 12.2, 12.8, 10.9.
    constexpr float kStartUs = D == 64 ? 6.7f : 8.2f, kStepUs = (D == 64 ? 1.1f : 1.43f) * (TWO ? 1.4f : 1.f);
    constexpr float kMeetUs = D == 64 ? 2.3f : 5.f, kMeetCtaUs = D == 64 ? 0.f : 0.25f;
    // The most pairs there can be come of odd lengths; as many as are likely
    // have to be resident at once (8 sequences of 32 behind 4000: 37.5 in
    // twos, 51.9 without; were there more pairs, some clusters would wait).
    const int64_t likely =
        std::min(pairs, std::max(some, (2 * pa.num_tokens + some * per_pair + 2 * per_pair - 1) / (2 * per_pair))) *
        a.num_kv_heads;
    int C = 1;
    float best = kStartUs + kStepUs * static_cast<float>(tiles);
    for (int c = 2; c <= kMaxCluster && c <= tiles && likely * c <= current_sm_count(152) && likely <= resident(c); c *= 2) {
      const float cost = kStartUs + kStepUs * static_cast<float>((tiles + c - 1) / c) + kMeetUs + kMeetCtaUs * c;
      if (cost >= best) continue;
      best = cost;
      C = c;
    }
    return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(units * C)), dim3(kThreads), Smem<D>::kBytes, C, stream,
                              a, pa, tq, tk, tv);
  }
};

template <bool TWO>
cudaError_t launch_p(const DecodeArgs& a, const PrefillArgs& pa, const CUtensorMap& tq, const CUtensorMap& tk,
                     const CUtensorMap& tv, int head_dim, bool bf16, cudaStream_t stream) {
  if (head_dim == 128)
    return bf16 ? Launch<128, true, TWO>::launch(a, pa, tq, tk, tv, stream)
                : Launch<128, false, TWO>::launch(a, pa, tq, tk, tv, stream);
  if (head_dim == 64)
    return bf16 ? Launch<64, true, TWO>::launch(a, pa, tq, tk, tv, stream)
                : Launch<64, false, TWO>::launch(a, pa, tq, tk, tv, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_prefill(const DecodeArgs& a, const PrefillArgs& pa, const CUtensorMap& tmap_q,
                           const CUtensorMap& tmap_k, const CUtensorMap& tmap_v, int head_dim, bool bf16,
                           cudaStream_t stream) {
  return a.out_dtype == 0 ? launch_p<true>(a, pa, tmap_q, tmap_k, tmap_v, head_dim, bf16, stream)
                          : launch_p<false>(a, pa, tmap_q, tmap_k, tmap_v, head_dim, bf16, stream);
}

}  // namespace pkv

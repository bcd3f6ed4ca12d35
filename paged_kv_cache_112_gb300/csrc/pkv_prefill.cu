// Attention of many tokens of each sequence over its paged history: prompts,
// chunks of prompts behind a cached prefix, a few drafted tokens.
//
// The n new tokens of sequence s (rows query_start[s] .. of q) are the last n
// of its L; the query of token i, head h sits at position p = L - n + i and sees
//     t <= p and (no window, or t > p - window, or t < sinks):
//     out = sum_t softmax_t(scale * q . k_t) v_t.
//
// Bound: the two products, 4 D flops a visible (query, head, token) on the
// tensor cores; and next to them 32 exponentials a SM and cycle.
//
// A CTA owns two tiles of 128 query rows of one KV head: the group's G heads of
// 128 / G tokens, rows ordered (token, head), so that K and V are read once for
// the whole group.  It walks the visible 128-token tiles of the history:
//     S = Q K^T        tcgen05.mma, both from shared memory, S in tensor memory;
//     P = 2^(S - m)    one thread a row, the running maximum and sum in
//                      registers; P goes back over S as 16-bit pairs;
//     O += P V         tcgen05.mma, P from tensor memory.
// Warps 0 to 3 and 4 to 7 are the threads of the two tiles: while one tile's
// are at the exponentials, the tensor cores work on the other's products.
// Warps 8 and 10 load K and V: TMA boxes of a block's rows of a head, scattered
// by the block table, into a ring of tiles; warp 11 passes a tile on, once it
// has zeroed what nobody sees of it; a thread of warp 9 issues the products.
//
// m is raised, and O scaled in tensor memory, only when the row's maximum has
// grown by more than 2^8 since: weights up to 2^8 do as well (a weight is
// rounded relative to itself), and O is read and written rarely.
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
// Registers: 168 a thread at launch; the tiles' threads hold a row of scores.
constexpr int kRowRegs = 208, kOtherRegs = 80;
static_assert(256 * kRowRegs + 128 * kOtherRegs <= 384 * 168, "shares of the launch's registers");
constexpr int kMaxCluster = 8;

template <int D>
struct Smem {
  static constexpr int kLines = D / 64;                 // 128-byte lines of a row
  static constexpr int kLineBytes = kRows * 128;        // one line of a tile's rows
  static constexpr int kTileBytes = kLines * kLineBytes;
  static constexpr int kSlots = D == 128 ? 5 : 8;       // K and V tiles in flight
  static constexpr int kRing = 2 * kTileBytes;          // after the two query tiles
  static constexpr int kRowState = 0;                   // the cluster's meeting, over the tiles: max and sum of 256 rows,
  static constexpr int kRowsAt = 2048;                  // then [256][D] floats
  static constexpr int kBars = kRing + kSlots * kTileBytes;
  // full[kSlots], ready[kSlots], empty[kSlots], q, s[2], p[2][2], o[2], drain; bad blocks of each slot, tensor
  // memory, abort, unit
  static constexpr int kBytes = kBars + 8 * (3 * kSlots + 10) + 4 * kSlots + 64;
  static_assert(kRowsAt + 2 * kRows * D * 4 <= kBars, "the cluster's rows fit over the tiles");
};

struct Unit {
  int s, first, n;  // sequence, first new token of the pair of tiles, the sequence's new tokens; s < 0: none
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const DecodeArgs a, const PrefillArgs pa,
                                                              const __grid_constant__ CUtensorMap tmap_q,
                                                              const __grid_constant__ CUtensorMap tmap_k,
                                                              const __grid_constant__ CUtensorMap tmap_v) {
  using SM = Smem<D>;
  constexpr int NS = SM::kSlots, NL = SM::kLines;
  extern __shared__ __align__(1024) uint8_t smem[];
  griddep_wait();
  griddep_launch_dependents();
  if (smem_misaligned(smem, a.dev_status)) return;  // the same for every CTA
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const uint32_t base = smem_u32(smem);
  const uint32_t full = base + SM::kBars, ready = full + 8 * NS, empty = ready + 8 * NS, q_bar = empty + 8 * NS,
                 s_bar = q_bar + 8, p_bar = s_bar + 16, o_bar = p_bar + 32, drain_bar = o_bar + 16;
  uint32_t* bad_blocks = reinterpret_cast<uint32_t*>(smem + SM::kBars + 8 * (3 * NS + 10));
  volatile uint32_t* tmem_at = bad_blocks + NS;
  volatile uint32_t* abort_at = tmem_at + 1;
  Unit* unit_at = reinterpret_cast<Unit*>(bad_blocks + NS + 2);
  int* warp_sums = reinterpret_cast<int*>(smem);  // over the tiles, before any copy

  // Which pair of tiles: units count ceil(n / pair) a sequence, the last ones
  // (whose history is longest) first.
  const int G = a.group, per_tile = kRows / G, per_pair = 2 * per_tile;
  const int g = static_cast<int>((blockIdx.x / C) % a.num_kv_heads);
  const int u = static_cast<int>((blockIdx.x / C) / a.num_kv_heads);
  const int S = a.num_seqs;
  auto range = [&](int s, int& lo) {  // new tokens of sequence s; its first row
    lo = min(max(pa.query_start[s], 0), pa.num_tokens);
    const int hi = min(max(pa.query_start[s + 1], lo), pa.num_tokens);
    return hi - lo;
  };
  {
    if (tid == 0) *unit_at = Unit{-1, 0, 0};
    const int chunk = (S + kThreads - 1) / kThreads, b = min(S, tid * chunk), e = min(S, b + chunk);
    int mine = 0, lo;
    for (int s = b; s < e; ++s) mine += (range(s, lo) + per_pair - 1) / per_pair;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int before = incl - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += warp_sums[w];
      total += warp_sums[w];
    }
    const int want = total - 1 - u;
    if (want >= before && want < before + mine) {
      for (int s = b; s < e; ++s) {
        const int n = range(s, lo), c = (n + per_pair - 1) / per_pair;
        if (want < before + c) {
          *unit_at = Unit{s, (want - before) * per_pair, n};
          break;
        }
        before += c;
      }
    }
    if (tid == 0) {
      *abort_at = 0;
      for (int i = 0; i < NS; ++i) {
        mbar_init(full + 8 * i, 1);
        mbar_init(ready + 8 * i, 1);
        mbar_init(empty + 8 * i, 1);
      }
      mbar_init(q_bar, 1);
      for (int t = 0; t < 2; ++t) {
        mbar_init(s_bar + 8 * t, 1);
        mbar_init(p_bar + 16 * t, kRows);
        mbar_init(p_bar + 16 * t + 8, kRows);
        mbar_init(o_bar + 8 * t, 1);
      }
      mbar_init(drain_bar, 1);
      fence_barrier_init();
      fence_proxy_async_smem();
    }
    __syncthreads();
  }
  const Unit unit = *unit_at;
  if (unit.s < 0) return;  // the same for the whole cluster
  if (warp == 9) {
    tc::alloc(smem_u32(const_cast<uint32_t*>(tmem_at)), 512);
    tc::fence_before();
  }
  const int s = unit.s;
  const int32_t raw_len = a.context_lens[s];
  const bool reporter = unit.first == 0 && g == 0 && rank == 0 && tid == 0;
  const int L = clamp_len(a, raw_len, reporter);
  int row0;
  range(s, row0);
  if (reporter && (L < unit.n || pa.query_start[s] != row0 || pa.query_start[s + 1] != row0 + unit.n))
    flag(a.dev_status, 8u);  // PKV_DEV_ERR_LENGTH
  const int tokens = min(per_pair, unit.n - unit.first);  // of this pair
  const int ntiles = tokens > per_tile ? 2 : 1;
  const int p0 = L - unit.n + unit.first, p1 = p0 + tokens - 1;  // positions of the pair's first and last token
  // Tokens that some row sees: [0, sinks) and [low, p1].
  const int low = pa.window > 0 ? max(0, p0 - pa.window + 1) : 0;
  const int sinks = pa.window > 0 ? min(pa.sinks, low) : 0;
  // Their tiles: [0, head), [head + skip, ..), `count` in all; this CTA's are rank, rank + C, ...
  const int head = (sinks + kKeys - 1) / kKeys, skip = max(0, low / kKeys - head);
  const int count = p1 >= 0 ? p1 / kKeys + 1 - skip : 0;
  const int cnt = count > rank ? (count - rank + C - 1) / C : 0;
  auto tile_of = [&](int j) {
    const int i = j * C + rank;
    return i < head ? i : i + skip;
  };
  __syncthreads();  // tensor memory's address
  tc::fence_after();
  const uint32_t tmem = *tmem_at;

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

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8 || warp == 10) {
      // -------------------------------------------------------------- loads
      // K tiles are 0, 2, 4, ... of the ring, V tiles 1, 3, 5, ...
      const bool is_v = warp == 10;
      const int B = 1 << a.block_shift, nblk = kKeys >> a.block_shift;  // blocks of a tile: 2 to 16, one a lane
      const int32_t* tbl = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
      auto entry = [&](int j) {  // this lane's block of tile j: physical block, -1 where no row sees it, -2 outside the pool
        if (j >= cnt || lane >= nblk) return -1;
        const int t = tile_of(j) * kKeys + lane * B;
        if (t > p1 || !(t + B > low || t < sinks)) return -1;
        const int phys = __ldg(tbl + (t >> a.block_shift));
        return static_cast<unsigned>(phys) < static_cast<unsigned>(a.num_blocks) ? phys : -2;
      };
      int phys = entry(0), j = 0;
      fence_proxy_async_smem();  // the search's sums lay where the queries go
      if (!is_v && cnt > 0 && tc::elect_one()) {
        mbar_arrive_expect_tx(q_bar, ntiles * NL * per_tile * G * 128);
        for (int t = 0; t < ntiles; ++t)
          for (int l = 0; l < NL; ++l)
            tma_load_4d(base + t * SM::kTileBytes + l * SM::kLineBytes, &tmap_q, 0, l, g * G,
                        row0 + unit.first + t * per_tile, q_bar);
      }
      __syncwarp();
      const CUtensorMap* map = is_v ? &tmap_v : &tmap_k;
      for (; j < cnt; ++j) {
        const uint32_t bad = __ballot_sync(kFull, phys == -2), there = __ballot_sync(kFull, phys >= 0);
        if (bad && lane == 0) flag(a.dev_status, 4u);  // PKV_DEV_ERR_BLOCK; the block counts as zeros
        const int i = 2 * j + is_v, slot = i % NS;
        const uint32_t bar = full + 8 * slot, dst = base + SM::kRing + slot * SM::kTileBytes;
        if (!__all_sync(kFull, wait(empty + 8 * slot, ((i / NS) & 1) ^ 1))) break;
        if (lane == 0) {
          bad_blocks[slot] = bad;
          mbar_arrive_expect_tx(bar, __popc(there) * NL * B * 128);
        }
        __syncwarp();
        for (int k = 0; k < nblk; ++k) {
          if (!((there >> k) & 1u)) continue;
          const int block = __shfl_sync(kFull, phys, k);
          if (tc::elect_one()) {
#pragma unroll
            for (int l = 0; l < NL; ++l)
              tma_load_4d(dst + l * SM::kLineBytes + k * B * 128, map, 0, 0, g * NL + l, block, bar);
          }
        }
        phys = entry(j + 1);
      }
      if (j < cnt && lane == 0) {  // copies in flight land before the CTA leaves
        if (!is_v) mbar_wait_bounded(q_bar, 0, a.timeout_ns);
        for (int k = max(0, j - NS); k < j; ++k) {
          const int i = 2 * k + is_v;
          if (i + NS > 2 * j + is_v) mbar_wait_bounded(full + 8 * (i % NS), (i / NS) & 1, a.timeout_ns);
        }
      }
    } else if (warp == 11) {
      // --------------------------------------------------------- what is there
      // Rows that no row of queries sees and blocks outside the pool become
      // zeros: their weights are zero, but what the pool holds there may be
      // anything, and zero times NaN is NaN.
      for (int i = 0; i < 2 * cnt; ++i) {
        const int slot = i % NS;
        const bool is_v = i & 1;
        if (!__all_sync(kFull, wait(full + 8 * slot, (i / NS) & 1))) break;
        const uint32_t bad = bad_blocks[slot];
        const int t0 = tile_of(i >> 1) * kKeys;
        const bool edge = is_v && (t0 + kKeys - 1 > p1 || (t0 < low && t0 + kKeys > sinks));
        if (bad || edge) {
          const uint32_t at = base + SM::kRing + slot * SM::kTileBytes;
          for (int r = lane; r < kKeys; r += 32) {
            const int t = t0 + r;
            const bool seen = t <= p1 && (t >= low || t < sinks);
            if (!((bad >> (r >> a.block_shift)) & 1u) && (!is_v || seen)) continue;
            for (int c = 0; c < NL * 8; ++c)  // rotated by the row: other banks for other lanes
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                               at + (c >> 3) * SM::kLineBytes + r * 128 + ((c + r) & 7) * 16),
                           "r"(0)
                           : "memory");
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(ready + 8 * slot) : "memory");
      }
    } else if (tc::elect_one()) {
      // ----------------------------------------------------------- products
      const uint32_t qk = tc::instr_desc(BF16, kKeys, false, pa.negate != 0), pv = tc::instr_desc(BF16, D, true, false);
      auto slot_addr = [&](int i) { return base + SM::kRing + (i % NS) * SM::kTileBytes; };
      auto arrive = [&](int i) { return wait(ready + 8 * (i % NS), (i / NS) & 1); };
      auto scores = [&](int t, int i) {  // S_t = Q_t K^T
        const uint64_t qd = tc::smem_desc(base + t * SM::kTileBytes, 16, 1024), kd = tc::smem_desc(slot_addr(i), 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k / 4) * SM::kLineBytes + (k % 4) * 32) >> 4;
          tc::mma_ss(tmem + t * kKeys, qd + off, kd + off, qk, k > 0);
        }
      };
      auto output = [&](int t, int i, int half, bool add) {  // O_t += P_t V, keys 64 half .. + 63
        const uint64_t vd = tc::smem_desc(slot_addr(i), SM::kLineBytes, 1024);
#pragma unroll
        for (int k = 4 * half; k < 4 * half + 4; ++k)
          tc::mma_ts(tmem + 256 + t * D, tmem + t * kKeys + 8 * k, vd + ((k * 2048) >> 4), pv, add || k > 0);
      };
      bool ok = cnt > 0 && wait(q_bar, 0) && arrive(0);
      if (ok) {
        tc::fence_after();
        for (int t = 0; t < ntiles; ++t) {
          scores(t, 0);
          tc::commit(s_bar + 8 * t);
        }
        tc::commit(empty);
      }
      for (int j = 0; j < cnt && ok; ++j) {
        const int vi = 2 * j + 1, ki = 2 * j + 2;
        ok = arrive(vi) && (j + 1 == cnt || arrive(ki));
        for (int t = 0; t < ntiles && ok; ++t) {
          ok = wait(p_bar + 16 * t, j & 1);
          if (!ok) break;
          tc::fence_after();
          output(t, vi, 0, j > 0);
          ok = wait(p_bar + 16 * t + 8, j & 1);
          if (!ok) break;
          tc::fence_after();
          output(t, vi, 1, true);
          if (j + 1 < cnt) scores(t, ki);
          tc::commit(j + 1 < cnt ? s_bar + 8 * t : o_bar + 8 * t);
        }
        if (ok) {
          tc::commit(empty + 8 * (vi % NS));
          if (j + 1 < cnt) tc::commit(empty + 8 * (ki % NS));
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
      cluster_sync();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    // -------------------------------------------------------------- softmax
    const int t = warp >> 2, r = tid & (kRows - 1);  // tile and row
    const int token = r / G, pos = p0 + t * per_tile + token;
    const bool live = token < per_tile && t * per_tile + token < tokens;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t s_at = tmem + t * kKeys + lanes, o_at = tmem + 256 + t * D + lanes;
    constexpr float kGrow = 8.f;
    // f16 weights: times 2^7, so that small ones keep their bits (f16 ends at 2^-24).
    constexpr float kUp = BF16 ? 0.f : 7.f;
    float m = kNegInf, l = 0.f;  // the row's reference, in scores; the sum of its weights
    if (t < ntiles) {
      const float sl2 = a.scale_log2, grow = kGrow / sl2;
      const int my_low = pa.window > 0 ? max(0, pos - pa.window + 1) : 0, my_sinks = pa.window > 0 ? pa.sinks : 0;
      // The tile's rows: positions first .. last, the widest and the narrowest view.
      const int first = p0 + t * per_tile, last = first + per_tile - 1;
      const int last_low = pa.window > 0 ? max(0, last - pa.window + 1) : 0;
      bool ok = true;
      for (int j = 0; j < cnt; ++j) {
        ok = __all_sync(kFull, wait(s_bar + 8 * t, j & 1));
        if (!ok) break;
        tc::fence_after();
        uint32_t x[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tc::ld32(x + c, s_at + c);
        tc::wait_ld();
        float* v = reinterpret_cast<float*>(x);
        const int t0 = tile_of(j) * kKeys;
        if (!(t0 + kKeys - 1 <= first && (t0 >= last_low || t0 + kKeys <= my_sinks))) {
          auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? kFull : (1u << n) - 1u; };
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            const int at = t0 + c;
            const uint32_t see = below(pos + 1 - at) & (~below(my_low - at) | below(my_sinks - at));
#pragma unroll
            for (int i = 0; i < 32; ++i) v[c + i] = (see >> i) & 1u ? v[c + i] : kNegInf;
          }
        }
        float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int i = 4; i < kKeys - 4; i += 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) top[k] = fmaxf(fmaxf(top[k], v[i + k]), v[i + 4 + k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) top[k] = fmaxf(top[k], v[kKeys - 4 + k]);
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
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
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // the product with V begins on the first half
#pragma unroll
          for (int i = 64 * half; i < 64 * half + 64; i += 2) {
            const float2 e = halves(fma2(pair(v[i], v[i + 1]), scale2, shift2));
            const float p0 = ex2_approx(e.x), p1 = ex2_approx(e.y);
            sum[(i / 2) & 1] = add2(sum[(i / 2) & 1], pair(p0, p1));
            x[i / 2] = BF16 ? pack_bf16(p0, p1) : pack_f16(p0, p1);
          }
          tc::st32(s_at + 32 * half, x + 32 * half);
          tc::wait_st();
          tc::fence_before();
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(p_bar + 16 * t + 8 * half) : "memory");
        }
        const float2 s0 = halves(sum[0]), s1 = halves(sum[1]);
        l += (s0.x + s0.y) + (s1.x + s1.y);
      }
      if (cnt > 0 && ok) ok = __all_sync(kFull, wait(o_bar + 8 * t, 0));
      tc::fence_after();
    }

    // ----------------------------------------------------------------- rows
    auto store_row = [&](int64_t at, const float* o, float f) {  // 32 channels
      if (a.out_dtype == 0) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i] * f, o[4 * i + 1] * f, o[4 * i + 2] * f, o[4 * i + 3] * f);
        return;
      }
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at);
      auto two = [&](int i) {
        return a.out_dtype == 1 ? pack_f16(o[i] * f, o[i + 1] * f) : pack_bf16(o[i] * f, o[i + 1] * f);
      };
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i] = make_uint4(two(8 * i), two(8 * i + 2), two(8 * i + 4), two(8 * i + 6));
    };
    auto row_at = [&](int tile, int row) {  // element index of a live row's first channel
      const int tok = row / G;
      return ((static_cast<int64_t>(row0) + unit.first + tile * per_tile + tok) * a.num_q_heads + g * G + (row - tok * G)) * D;
    };
    if (C == 1) {
      if (t < ntiles) {
        const float f = l > 0.f ? 1.f / l : 0.f;
        const int64_t at = row_at(t, r);
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tc::ld32(o, o_at + c);
          tc::wait_ld();
          if (l == 0.f) {  // no visible token: whatever tensor memory holds
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          if (live) store_row(at + c, reinterpret_cast<const float*>(o), f);
        }
      }
    } else {
      // The cluster's rows: each CTA scales its part to the rows' common maximum
      // and leaves it in its shared memory; CTA r adds up rows r, r + C, ...
      float2* state = reinterpret_cast<float2*>(smem + SM::kRowState);
      float* rows = reinterpret_cast<float*>(smem + SM::kRowsAt);
      __syncthreads();  // the tiles are no longer read
      state[tid] = make_float2(m, l);
      cluster_sync();
      auto remote = [&](uint32_t addr, int from) {
        float2 v;
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                     : "=f"(v.x), "=f"(v.y)
                     : "r"(cluster_map(addr, from))
                     : "memory");
        return v;
      };
      if (t < ntiles) {
        float top = kNegInf, sum = 0.f;
        for (int k = 0; k < C; ++k) top = fmaxf(top, remote(smem_u32(state + tid), k).x);
        const float ref = top == kNegInf ? 0.f : top;
        for (int k = 0; k < C; ++k) {
          const float2 v = remote(smem_u32(state + tid), k);
          sum += v.y * ex2_approx((v.x - ref) * a.scale_log2);
        }
        const float f = l > 0.f ? ex2_approx((m - ref) * a.scale_log2) / sum : 0.f;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tc::ld32(o, o_at + c);
          tc::wait_ld();
          // Rotated by the row, so that a warp's stores meet different banks.
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
            if (l > 0.f)
              w = make_float4(__uint_as_float(o[i]) * f, __uint_as_float(o[i + 1]) * f, __uint_as_float(o[i + 2]) * f,
                              __uint_as_float(o[i + 3]) * f);
            *reinterpret_cast<float4*>(rows + tid * D + ((c + i + 4 * r) & (D - 1))) = w;
          }
        }
      }
      cluster_sync();
      // 4 channels a thread, D / 4 threads a row.
      const int rows_in = ntiles * kRows, width = D / 4;
      for (int e = tid; e < rows_in / C * width; e += 2 * kRows) {
        const int row = (e / width) * C + rank, ch = 4 * (e % width);
        const int tile = row / kRows, in = row & (kRows - 1), tok = in / G;
        if (tok >= per_tile || tile * per_tile + tok >= tokens) continue;
        const uint32_t addr = smem_u32(rows + row * D + ((ch + 4 * in) & (D - 1)));
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < C; ++k) {
          float4 v;
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                       : "r"(cluster_map(addr, k))
                       : "memory");
          sum.x += v.x;
          sum.y += v.y;
          sum.z += v.z;
          sum.w += v.w;
        }
        const int64_t at = row_at(tile, in) + ch;
        store_out(a.out, at, sum.x, a.out_dtype);
        store_out(a.out, at + 1, sum.y, a.out_dtype);
        store_out(a.out, at + 2, sum.z, a.out_dtype);
        store_out(a.out, at + 3, sum.w, a.out_dtype);
      }
      cluster_sync();  // no CTA leaves while its rows are read
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

template <int D, bool BF16>
struct Launch {
  static constexpr auto kernel = prefill_kernel<D, BF16>;

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
    // Pairs of tiles: at most one more than whole ones a sequence.
    const int64_t pairs = pa.num_tokens / per_pair + std::min<int64_t>(a.num_seqs, pa.num_tokens);
    const int64_t units = pairs * a.num_kv_heads, tiles = (static_cast<int64_t>(a.max_context_len) + kKeys - 1) / kKeys;
    int C = 1;
    while (C < kMaxCluster && units * C * 2 <= current_sm_count(152) && 2 * C <= tiles && units <= resident(2 * C)) C *= 2;
    return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(units * C)), dim3(kThreads), Smem<D>::kBytes, C, stream,
                              a, pa, tq, tk, tv);
  }
};

}  // namespace

cudaError_t launch_prefill(const DecodeArgs& a, const PrefillArgs& pa, const CUtensorMap& tmap_q,
                           const CUtensorMap& tmap_k, const CUtensorMap& tmap_v, int head_dim, bool bf16,
                           cudaStream_t stream) {
  if (head_dim == 128)
    return bf16 ? Launch<128, true>::launch(a, pa, tmap_q, tmap_k, tmap_v, stream)
                : Launch<128, false>::launch(a, pa, tmap_q, tmap_k, tmap_v, stream);
  if (head_dim == 64)
    return bf16 ? Launch<64, true>::launch(a, pa, tmap_q, tmap_k, tmap_v, stream)
                : Launch<64, false>::launch(a, pa, tmap_q, tmap_k, tmap_v, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkv

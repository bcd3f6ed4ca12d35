// Block summaries and block selection for sparse decode attention.
//
// summarize_blocks: for a block's keys k_t of KV head g and each channel d,
//     lo_d = min_t k_t[d],  hi_d = max_t k_t[d],
// held as int8 steps of a power of two 2^e (the smallest with every |bound| <=
// 127 * 2^e): lo rounded down, hi rounded up, so the bounds stay bounds.
//
// select_blocks: no key of block b can score above
//     score_h(b) = sum_d max(q_d lo_d, q_d hi_d)
// for query head h; q is rounded to int8 steps of a power of two of its own,
// so the sum is an integer, sum_d q_d^- lo_d + q_d^+ hi_d with q^- = min(q, 0)
// and q^+ = max(q, 0): two integer dot products, below 2^22 in magnitude and
// free of any summation order.  A block's score is the largest over the
// group's heads; the best ones are taken, equal scores by the lowest block.
//
// Bound: HBM bytes of the summaries, 2D + 4 a block and KV head (8 sequences of
// 2048 to 8192 blocks: 27.8 us, 20 of them the scores at 5.2 TB/s, 6 the search
// after them; every sequence has as many CTAs, so the longest ones end last); with few blocks the latency of length -> table -> summary ->
// ranks (64 sequences of up to 128 blocks: 6.2 us).
#include "pkv_device.cuh"

namespace pkv {
namespace {

using namespace dev;

// ------------------------------------------------------------------ summary

// The smallest e >= -126 such that p + r <= 127 * 2^e, where p >= 0 is finite
// and r is the part of an exact product that its float32 rounding p left out;
// 0 for p = 0.  p = m 2^x with m in [1/2, 1): x - 7 while m <= 127/128
// (fraction bits 0x7e0000), else x - 6; a subnormal p is below 127 * 2^-126.
__device__ __forceinline__ int bound_exponent(float p, float r) {
  const uint32_t u = __float_as_uint(p), frac = u & 0x7fffffu;
  const int x = static_cast<int>(u >> 23) - 126;
  const int e = x - 7 + (frac > 0x7e0000u || (frac == 0x7e0000u && r > 0.f));
  return u == 0 ? 0 : max(e, -126);
}

// floor (ceil) of x * f as a byte, |x f| <= 127: added to 1.5 * 2^23 with one
// rounding downwards (upwards), the exact product's integer part is the sum's
// low bits, in two's complement.
__device__ __forceinline__ uint32_t floor_bits(float x, float f) {
  return __float_as_uint(__fmaf_rd(x, f, 12582912.f));
}
__device__ __forceinline__ uint32_t ceil_bits(float x, float f) {
  return __float_as_uint(__fmaf_ru(x, f, 12582912.f));
}
// The low bytes of four words.
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Packed minimum and maximum of two values; a NaN loses against a number.
template <bool BF16>
__device__ __forceinline__ void min_max2(uint32_t& lo, uint32_t& hi, uint32_t v) {
  if constexpr (BF16) {
    __nv_bfloat162 l = *reinterpret_cast<__nv_bfloat162*>(&lo), h = *reinterpret_cast<__nv_bfloat162*>(&hi);
    const __nv_bfloat162 x = *reinterpret_cast<__nv_bfloat162*>(&v);
    l = __hmin2(l, x);
    h = __hmax2(h, x);
    lo = *reinterpret_cast<uint32_t*>(&l);
    hi = *reinterpret_cast<uint32_t*>(&h);
  } else {
    __half2 l = *reinterpret_cast<__half2*>(&lo), h = *reinterpret_cast<__half2*>(&hi);
    const __half2 x = *reinterpret_cast<__half2*>(&v);
    l = __hmin2(l, x);
    h = __hmax2(h, x);
    lo = *reinterpret_cast<uint32_t*>(&l);
    hi = *reinterpret_cast<uint32_t*>(&h);
  }
}

template <bool BF16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  if constexpr (BF16) return unpack_bf16(w);
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}

// A finite number: NaN counts as 0, an infinity as the type's largest value.
__device__ __forceinline__ float finite_bound(float x, float most) {
  return x == x ? fminf(fmaxf(x, -most), most) : 0.f;
}

// A warp takes (listed block, HPT adjacent KV heads) tasks in turn: as many
// heads as make 256 bytes of a row.  The rows are read as 16-byte vectors, two
// rows at a time and 16 rows a step, the next step's rows on their way while
// the current ones are compared.  Each lane keeps the packed min and max of
// its channels; the two row groups then exchange halves, so each lane ends up
// with NW channels, rounds their bounds and stores the codes.  KIND: 0 = f16,
// 1 = bf16, 2 = FP8 (codes compared as f16, which holds every e4m3 value).
//
// Bound: 16-bit pools HBM (8192 blocks of 8 heads in 46.0 us, 6.2 TB/s);
// FP8 pools neither memory nor the issue rate alone (4001 blocks of 8 heads in
// 15.6 us, 4.7 TB/s: a code costs as many instructions as a 16-bit key of
// twice its bytes, 41% of the issue slots with two CTAs of 120 registers a SM).
template <int D, int KIND>
__global__ void __launch_bounds__(256) summarize_blocks_kernel(const SummarizeArgs a) {
  constexpr int EB = KIND == 2 ? 1 : 2;
  constexpr bool BF16 = KIND == 1;
  constexpr int HPT = 256 / (D * EB);  // heads per task
  constexpr int LPR = 16;              // lanes per row
  constexpr int LPH = LPR / HPT;       // lanes per head and row
  constexpr int NL = 8;                // loads per step of 16 rows
  constexpr int NW = KIND == 2 ? 8 : 4;  // packed pairs of channels per lane; channels it ends up with
  constexpr uint32_t kNone = BF16 ? 0x7fc07fc0u : 0x7e007e00u;  // NaN: no number yet
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int H = a.num_kv_heads, GH = (H + HPT - 1) / HPT;  // tasks per block
  const uint32_t first = blockIdx.x * 8 + (threadIdx.x >> 5), stride = gridDim.x * 8;
  const int step_i = static_cast<int>(stride / GH), step_g = static_cast<int>(stride % GH);
  const int64_t row_bytes = static_cast<int64_t>(H) * D * EB;
  const int64_t lane_at = (lane / LPR) * row_bytes + (lane % LPR) * 16;
  const int sub = (lane % LPR) / LPH;  // this lane's head within the task

  struct Task {
    int64_t i;  // index into block_ids
    int g;      // group of HPT heads
  };
  auto after = [&](Task p) {
    p.i += step_i;
    p.g += step_g;
    if (p.g >= GH) {
      p.g -= GH;
      ++p.i;
    }
    return p;
  };
  auto id_of = [&](const Task& p) { return p.i < a.num_ids ? __ldg(a.block_ids + p.i) : -1; };
  // A step's rows; none for a block that is not there (-1 or out of range) or a head past the last.
  auto load = [&](uint4 (&u)[NL], const Task& p, int id, int r0) {
    if (id < 0 || id >= a.num_blocks || p.g * HPT + sub >= H) return;
    const uint8_t* src = a.k_pool + id * a.block_bytes + p.g * 256 + r0 * row_bytes + lane_at;
#pragma unroll
    for (int i = 0; i < NL; ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(src + 2 * i * row_bytes));
  };

  Task now{first / GH, static_cast<int>(first % GH)}, next = after(now), later = after(next);
  int id = id_of(now), next_id = id_of(next), r0 = 0;
  uint4 cur[NL] = {}, nxt[NL] = {};
  load(cur, now, id, 0);
  uint32_t lo[NW], hi[NW];
#pragma unroll
  for (int i = 0; i < NW; ++i) lo[i] = hi[i] = kNone;
  while (now.i < a.num_ids) {
    const bool last = r0 + 16 >= a.block_size;
    const int later_id = last ? id_of(later) : 0;
    if (last)
      load(nxt, next, next_id, 0);
    else
      load(nxt, now, id, r0 + 16);
    const bool there = id >= 0 && id < a.num_blocks;
    if (there) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const uint32_t w[4] = {cur[i].x, cur[i].y, cur[i].z, cur[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (KIND == 2) {
            uint32_t p, q;
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
                "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                : "=r"(p), "=r"(q)
                : "r"(w[j]));
            min_max2<false>(lo[2 * j], hi[2 * j], p);
            min_max2<false>(lo[2 * j + 1], hi[2 * j + 1], q);
          } else {
            min_max2<BF16>(lo[j], hi[j], w[j]);
          }
        }
      }
    } else if (id != -1 && r0 == 0 && now.g == 0 && lane == 0) {
      flag(a.dev_status, 4u);  // PKV_DEV_ERR_BLOCK
    }
    if (last && there) {
      // The row groups exchange halves of their pairs: lanes 16 and up keep the upper.
      const bool upper = lane & 16;
#pragma unroll
      for (int i = 0; i < NW / 2; ++i) {
        const uint32_t l = __shfl_xor_sync(kFull, upper ? lo[i] : lo[i + NW / 2], 16);
        const uint32_t h = __shfl_xor_sync(kFull, upper ? hi[i] : hi[i + NW / 2], 16);
        lo[i] = upper ? lo[i + NW / 2] : lo[i];
        hi[i] = upper ? hi[i + NW / 2] : hi[i];
        uint32_t dump = lo[i];
        min_max2<BF16>(lo[i], dump, l);
        dump = hi[i];
        min_max2<BF16>(dump, hi[i], h);
      }
      // The bounds in float32; a channel without a number counts as 0, an
      // infinity as the type's largest value.
      const int head = now.g * HPT + sub;
      const int64_t at = static_cast<int64_t>(id) * H + min(head, H - 1);
      constexpr float kMost = KIND == 0 ? 65504.f : 3.3895313892515355e38f;
      float vl[NW], vh[NW], top = 0.f;
#pragma unroll
      for (int i = 0; i < NW / 2; ++i) {
        const float2 l = widen2<BF16>(lo[i]), h = widen2<BF16>(hi[i]);
        vl[2 * i] = l.x == l.x ? l.x : 0.f;
        vl[2 * i + 1] = l.y == l.y ? l.y : 0.f;
        vh[2 * i] = l.x == l.x ? h.x : 0.f;
        vh[2 * i + 1] = l.y == l.y ? h.y : 0.f;
      }
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        if constexpr (KIND != 2) {
          vl[j] = fminf(fmaxf(vl[j], -kMost), kMost);
          vh[j] = fminf(fmaxf(vh[j], -kMost), kMost);
        }
        top = fmaxf(top, fmaxf(-vl[j], vh[j]));
      }
      if constexpr (HPT == 1) {
        top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));  // top >= 0: its bits order as it does
      } else {
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
      }
      float factor, ptop = top, rtop = 0.f;  // value = factor * v
      if constexpr (KIND == 2) {
        factor = __ldg(a.k_scale + id * a.scale_stride + min(head, H - 1));
        if (!(factor > 0.f) || factor > 3.4028234e38f) factor = 0.f;  // no such scale: the block counts as zeros
        ptop = top * factor;
        rtop = fmaf(top, factor, -ptop);
        if (ptop > 3.4028234e38f) {  // values beyond float32 count as its largest
          ptop = 3.4028234e38f;
          rtop = 0.f;
#pragma unroll
          for (int j = 0; j < NW; ++j) {
            vl[j] = fminf(fmaxf(vl[j] * factor, -3.4028234e38f), 3.4028234e38f);
            vh[j] = fminf(fmaxf(vh[j] * factor, -3.4028234e38f), 3.4028234e38f);
          }
          factor = 1.f;
        }
      } else {
        factor = 1.f;
      }
      const int e = bound_exponent(ptop, rtop);
      factor *= exp2_int(-e);  // exact: a power of two that keeps top * factor within 127
      uint32_t cl[NW], ch[NW];
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        cl[j] = floor_bits(vl[j], factor);
        ch[j] = ceil_bits(vh[j], factor);
      }
      if (head < H) {
        int8_t* dst = a.summary + at * (2 * D) + (lane % LPH) * (2 * NW) + (upper ? NW : 0);
        if constexpr (NW == 4) {
          *reinterpret_cast<uint32_t*>(dst) = pack_bytes(cl[0], cl[1], cl[2], cl[3]);
          *reinterpret_cast<uint32_t*>(dst + D) = pack_bytes(ch[0], ch[1], ch[2], ch[3]);
        } else {
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(pack_bytes(cl[0], cl[1], cl[2], cl[3]), pack_bytes(cl[4], cl[5], cl[6], cl[7]));
          *reinterpret_cast<uint2*>(dst + D) =
              make_uint2(pack_bytes(ch[0], ch[1], ch[2], ch[3]), pack_bytes(ch[4], ch[5], ch[6], ch[7]));
        }
        if (lane % LPH == 0 && !upper) a.summary_scale[at] = exp2_int(e);
      }
    }
    if (last) {
      now = next;
      next = later;
      later = after(later);
      id = next_id;
      next_id = later_id;
      r0 = 0;
#pragma unroll
      for (int i = 0; i < NW; ++i) lo[i] = hi[i] = kNone;
    } else {
      r0 += 16;
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) cur[i] = nxt[i];
  }
}

// ---------------------------------------------------------------- selection

// Floats in the order of unsigned integers (no NaN); -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// 16 x 8 integer products over 32 channels: c += a b.  (The integer tensor
// path of this GPU is slow -- 115 of these a microsecond and SM, measured --
// but eight of them still score 16 blocks for 8 heads in less time than their
// 4 KB take from memory, and leave the issue slots free; with dp4a the same
// loop was issue-bound at 20 instructions a block.)
__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kBins = 2048;
constexpr int kListed = 512;      // candidates that are listed once no more are left
constexpr int kAhead = 8;         // keys a thread reads ahead of using them
constexpr int kWarpBlocks = 1024;  // up to here one warp searches the threshold
constexpr int kRankBlocks = 256;  // up to here every key is ranked directly

// Exclusive prefix sums of a pair of counts over the CTA's threads.
template <int NT>
__device__ __forceinline__ int2 block_scan(int2 v, int2* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, s.x, o), y = __shfl_up_sync(kFull, s.y, o);
    if (lane >= o) {
      s.x += x;
      s.y += y;
    }
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int2 before = make_int2(s.x - v.x, s.y - v.y);
#pragma unroll
  for (int w = 0; w < NT / 32; ++w)
    if (w < warp) {
      before.x += warp_sums[w].x;
      before.y += warp_sums[w].y;
    }
  return before;
}

// One cluster of C CTAs per (sequence, KV head).  Every CTA scores its share
// of the blocks and stores the order keys into the first CTA's shared
// memory; then the first CTA alone finds the keep-th largest key by
// histograms over ever narrower ranges (2048 bins each) and writes the chosen
// block numbers in order.  (Histograms kept by every CTA and added up through
// distributed shared memory took 25 us of the 79 us that 8 sequences of up to
// 8192 blocks needed: 64 KB of remote loads a CTA and round.)
//
// Scoring: a warp takes 16 blocks at a time as the rows of an m16n8k32 product
// whose columns are the group's heads.  Lane (gr = lane / 4, tq = lane % 4)
// needs rows gr and gr + 8; since any order of the channels will do as long as
// q has the same, it reads 16-byte chunks 4x + tq of a bound straight from
// global memory and uses words 2i, 2i + 1 of chunk x in k-step 2x + i.  The
// next 16 blocks' summaries are loaded before the current ones are used.
// With at most 4 heads (FEW) half of the product's columns would be idle and
// the slow integer tensor path bound the kernel (18 us of an SM's 21 at 8
// sequences of up to 8192 blocks): there the lower bounds take dp4a on the
// same registers instead, the query's words from shared memory.
template <int D, bool BF16, int NT, bool FEW>
__global__ void __launch_bounds__(NT) select_blocks_kernel(const SelectArgs a, int a_keys, int words_max) {
  constexpr int X = D / 64;      // 16-byte chunks of one bound per lane and row
  constexpr int NWARP = NT / 32;
  constexpr int BPT = kBins / NT;  // bins per thread
  extern __shared__ __align__(16) uint32_t keys[];  // read as 16-byte vectors too
  __shared__ __align__(16) int hist[kBins];
  __shared__ __align__(16) uint32_t q_codes[2][8][D / 4];  // negative and positive parts; heads past the group are 0
  __shared__ int q_exp[8];
  __shared__ int2 warp_sums[NWARP];
  __shared__ uint32_t warp_range[2][NWARP];
  __shared__ int found[3];  // the bin, how many keys lie above it and in it
  __shared__ uint2 list[kListed];  // candidates left: key and block
  __shared__ int listed;
  cluster_arrive();  // see the wait before the scores
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int64_t unit = blockIdx.x / C;
  const int s = static_cast<int>(unit / a.num_kv_heads), g = static_cast<int>(unit % a.num_kv_heads);
  int L = a.context_lens[s];
  // The cluster's warps take chunks of 32 blocks in turn.  Where the first ones
  // are does not depend on the length: their table entries are read along with it.
  const int32_t* tbl = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  const int stride = C * NT;
  int b0 = rank * NT + warp * 32;
  const int early = b0 + lane < a.max_blocks_per_seq ? __ldg(tbl + b0 + lane) : -1;

  // Query codes, a head per warp: 4 channels a lane (D = 64: the lower half-warp).
  for (int h = warp; h < 8; h += NWARP) {
    const bool live = h < a.group && lane < D / 4;
    const uint2 w = live ? __ldg(reinterpret_cast<const uint2*>(
                               a.q + (static_cast<int64_t>(s) * a.num_q_heads + g * a.group + h) * D) + lane)
                         : make_uint2(0u, 0u);
    const float2 f0 = widen2<BF16>(w.x), f1 = widen2<BF16>(w.y);
    const float most = BF16 ? __uint_as_float(0x7f7f0000u) : 65504.f;
    float x[4] = {finite_bound(f0.x, most), finite_bound(f0.y, most), finite_bound(f1.x, most),
                  finite_bound(f1.y, most)};
    float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    // Positive floats order as their bits.
    top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));
    const int e = top > 0.f ? bound_exponent(top, 0.f) : -126;
    const float inv = exp2_int(-e);
    uint32_t neg = 0, pos = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = __float2int_rn(x[j] * inv);
      neg |= (static_cast<uint32_t>(min(c, 0)) & 0xffu) << (8 * j);
      pos |= static_cast<uint32_t>(max(c, 0)) << (8 * j);
    }
    if (lane < D / 4) {
      q_codes[0][h][lane] = neg;
      q_codes[1][h][lane] = pos;
    }
    if (lane == 0) q_exp[h] = e;
  }

  const int cap = min(a.max_context_len, a.max_blocks_per_seq << a.block_shift);
  if (L < 0 || L > cap) {
    if (g == 0 && rank == 0 && tid == 0) flag(a.dev_status, 8u);  // PKV_DEV_ERR_LENGTH
    L = L < 0 ? 0 : cap;
  }
  const int n = (L >> a.block_shift) + ((L & ((1 << a.block_shift) - 1)) ? 1 : 0);
  const int count = min(n, a.keep);
  int32_t* out = a.selected + unit * a.keep;
  if (rank == 0 && tid == 0) a.counts[unit] = count;
  if (n <= a.keep) {  // the same for every CTA of the cluster
    for (int i = rank * NT + tid; i < a.keep; i += C * NT) out[i] = i < n ? i : -1;
    cluster_wait();
    return;
  }
  const int first = a.first_blocks, last = n - a.last_blocks;  // blocks outside [first, last) are always taken

  // Lane j holds block j's table entry, fetched two chunks ahead, and its scale, one chunk ahead.
  auto entry = [&](int b) {
    if (b + lane >= n) return -1;
    return __ldg(tbl + b + lane);
  };
  auto checked = [&](int p, int b) {  // PKV_DEV_ERR_BLOCK: the block is scored last
    if (p >= 0 && p < a.num_blocks) return p;
    if (b + lane < n) flag(a.dev_status, 4u);
    return -1;
  };
  // -1 for a block that is scored last: no table entry, or a scale that no
  // summary has (0 times an infinite one is NaN, whose key would end the
  // order of the floats that the searches below rely on).
  auto scale_of = [&](int p) {
    const float x = p >= 0 ? __ldg(a.summary_scale + static_cast<int64_t>(p) * a.num_kv_heads + g) : -1.f;
    return x >= 0.f && x <= 3.4028234e38f ? x : -1.f;
  };
  const int gr = lane >> 2, tq = lane & 3;
  struct Group {
    uint4 lo[2][X], hi[2][X];  // [row gr, gr + 8]
  };
  auto load = [&](Group& u, int p, int half) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int block = max(__shfl_sync(kFull, p, 16 * half + gr + 8 * r), 0);
      const uint4* src = reinterpret_cast<const uint4*>(
                             a.summary + (static_cast<int64_t>(block) * a.num_kv_heads + g) * (2 * D)) + tq;
#pragma unroll
      for (int x = 0; x < X; ++x) {
        u.lo[r][x] = __ldg(src + 4 * x);
        u.hi[r][x] = __ldg(src + D / 16 + 4 * x);
      }
    }
  };
  int phys = b0 + lane < n ? early : -1, ahead = entry(b0 + stride);
  phys = checked(phys, b0);
  float sc = scale_of(phys);
  Group even, odd;
  load(even, phys, 0);
  __syncthreads();  // q_codes

  // Query fragments: this lane's words of head gr.  All heads' scales times
  // 2^-(22 + the largest exponent), down to float32's subnormals: integer *
  // scale * summary scale does not overflow and is exact while scale times
  // summary scale is 2^-149 or more, 2^-22 * 2^-126 for the head with that
  // exponent; below, it rounds, which swaps no two scores.
  uint32_t qf[X][4], qn[X][4];  // positive, negative parts
#pragma unroll
  for (int x = 0; x < X; ++x) {
    const uint4 w = *reinterpret_cast<const uint4*>(&q_codes[1][gr][16 * x + 4 * tq]);
    qf[x][0] = w.x, qf[x][1] = w.y, qf[x][2] = w.z, qf[x][3] = w.w;
    if constexpr (!FEW) {
      const uint4 v = *reinterpret_cast<const uint4*>(&q_codes[0][gr][16 * x + 4 * tq]);
      qn[x][0] = v.x, qn[x][1] = v.y, qn[x][2] = v.z, qn[x][3] = v.w;
    }
  }
  int emax = -126;
#pragma unroll
  for (int h = 0; h < 8; ++h) emax = max(emax, q_exp[h]);
  // The scales of the heads whose sums this lane ends up with: 2 tq and
  // 2 tq + 1, the product's columns; FEW: 2 (tq & 1) and the next.
  const int head_a = 2 * (FEW ? tq & 1 : tq);
  const bool live_a = head_a < a.group, live_b = head_a + 1 < a.group;
  const float scale_a = ldexpf(1.f, q_exp[head_a] - emax - 22);
  const float scale_b = ldexpf(1.f, q_exp[head_a + 1] - emax - 22);

  const uint32_t keys_at = cluster_map(smem_u32(keys), 0);
  cluster_wait();  // the first CTA has begun
  auto score = [&](const Group& u, int half, int base, float scales) {
    int c[4] = {0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < X; ++x) {
      const uint4 h0 = u.hi[0][x], h1 = u.hi[1][x];
      mma_s8(c, h0.x, h1.x, h0.y, h1.y, qf[x][0], qf[x][1]);
      mma_s8(c, h0.z, h1.z, h0.w, h1.w, qf[x][2], qf[x][3]);
      if constexpr (!FEW) {
        const uint4 l0 = u.lo[0][x], l1 = u.lo[1][x];
        mma_s8(c, l0.x, l1.x, l0.y, l1.y, qn[x][0], qn[x][1]);
        mma_s8(c, l0.z, l1.z, l0.w, l1.w, qn[x][2], qn[x][3]);
      }
    }
    if constexpr (FEW) {
      int d[2][4];  // [row gr, gr + 8][head]: this lane's channels
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        d[0][h] = d[1][h] = 0;
#pragma unroll
        for (int x = 0; x < X; ++x) {
          const int4 w = *reinterpret_cast<const int4*>(&q_codes[0][h][16 * x + 4 * tq]);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint4 l = u.lo[r][x];
            d[r][h] = __dp4a(static_cast<int>(l.x), w.x, d[r][h]);
            d[r][h] = __dp4a(static_cast<int>(l.y), w.y, d[r][h]);
            d[r][h] = __dp4a(static_cast<int>(l.z), w.z, d[r][h]);
            d[r][h] = __dp4a(static_cast<int>(l.w), w.w, d[r][h]);
          }
        }
      }
      // Sums over the four lanes of a row pair, halved with each exchange:
      // lane tq ends up with row (tq & 2 ? gr + 8 : gr), heads 2 (tq & 1) and + 1.
      const bool low_row = !(tq & 2), low_pair = !(tq & 1);
      int e[4];
#pragma unroll
      for (int h = 0; h < 4; ++h)
        e[h] = (low_row ? d[0][h] : d[1][h]) + __shfl_xor_sync(kFull, low_row ? d[1][h] : d[0][h], 2);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        e[i] = (low_pair ? e[i] : e[2 + i]) + __shfl_xor_sync(kFull, low_pair ? e[2 + i] : e[i], 1);
      // The product's sums of row gr + 8 move to lanes 2 and 3 (its columns 4 to 7 are padding).
      const int p = __shfl_xor_sync(kFull, c[2], 2), q = __shfl_xor_sync(kFull, c[3], 2);
      const int ta = e[0] + (low_row ? c[0] : p), tb = e[1] + (low_row ? c[1] : q);
      float top = fmaxf(live_a ? static_cast<float>(ta) * scale_a : kNegInf,
                        live_b ? static_cast<float>(tb) * scale_b : kNegInf);
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
      const int row = 16 * half + gr + (low_row ? 0 : 8);
      const float psc = __shfl_sync(kFull, scales, row);
      const int b = base + row;
      // The block's scale after the maximum over heads: it is their common factor.
      if (low_pair && b < n) cluster_store_u32(keys_at + 4 * b, psc >= 0.f ? order_key(top * psc) : 0u);
    } else {
      float best[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        best[r] = fmaxf(live_a ? static_cast<float>(c[2 * r]) * scale_a : kNegInf,
                        live_b ? static_cast<float>(c[2 * r + 1]) * scale_b : kNegInf);
        best[r] = fmaxf(best[r], __shfl_xor_sync(kFull, best[r], 1));
        best[r] = fmaxf(best[r], __shfl_xor_sync(kFull, best[r], 2));
      }
      // Lanes tq = 0 and 1 store rows gr and gr + 8 (the block's scale is the heads' common factor).
      const int row = 16 * half + gr + 8 * (tq & 1);
      const float psc = __shfl_sync(kFull, scales, row);
      const int b = base + row;
      if (tq < 2 && b < n)
        cluster_store_u32(keys_at + 4 * b, psc >= 0.f ? order_key((tq ? best[1] : best[0]) * psc) : 0u);
    }
  };
  while (b0 < n) {
    load(odd, phys, 1);
    const int next = checked(ahead, b0 + stride);
    ahead = entry(b0 + 2 * stride);
    const float next_sc = scale_of(next);
    score(even, 0, b0, sc);
    load(even, next, 0);
    score(odd, 1, b0, sc);
    phys = next;
    sc = next_sc;
    b0 += stride;
  }
  cluster_sync();  // every key has arrived
  if (rank != 0) return;

  // What is taken goes into two bitmaps: blocks taken for sure, and blocks
  // whose key equals the threshold, of which the first `ties` are taken.
  const int words = (n + 31) / 32;
  uint32_t* sure_bits = keys + a_keys;
  uint32_t* tie_bits = sure_bits + words_max;
  int need = a.keep - first - a.last_blocks;  // middle blocks to take
  int ties = 0;
  auto forced = [&](int b) { return b < first || b >= last; };
  if (n <= kRankBlocks) {
    // Few blocks: each thread counts the middle keys above its own.  Forced
    // blocks' keys become 0 first, below every score.
    for (int b = tid; b < words * 32; b += NT)
      if (b >= n || forced(b)) keys[b] = 0;
    if (tid == 0) listed = 0;
    __syncthreads();
    const uint4* all = reinterpret_cast<const uint4*>(keys);
    for (int b = tid; b < words * 32; b += NT) {
      const uint32_t k = keys[b];
      int part[4] = {0, 0, 0, 0};  // independent sums: with one warp a scheduler only these overlap
      for (int j = 0; j < words * 8; j += 8) {
        uint4 o[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) o[u] = all[j + u];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          part[0] += o[u].x > k;
          part[1] += o[u].y > k;
          part[2] += o[u].z > k;
          part[3] += o[u].w > k;
        }
      }
      const int above = part[0] + part[1] + part[2] + part[3];
      const bool middle = b < n && !forced(b);
      const uint32_t w = __ballot_sync(kFull, middle && above < need);
      const uint32_t f = __ballot_sync(kFull, b < n && !middle);
      if (lane == 0) {
        sure_bits[b / 32] = w | f;
        atomicAdd(&listed, __popc(w));
      }
    }
    __syncthreads();
    if (listed > need) {  // equal keys at the threshold: the lowest blocks of them
      for (int b = tid; b < words * 32; b += NT) {
        const uint32_t k = keys[b];
        const bool middle = b < n && !forced(b);
        int before = 0;
        for (int j = first; j < last; ++j) before += keys[j] > k || (keys[j] == k && j < b);
        const uint32_t w = __ballot_sync(kFull, middle ? before < need : b < n);
        if (lane == 0) sure_bits[b / 32] = w;
      }
    }
    __syncthreads();
    for (int b = tid; b < words * 32; b += NT) {
      const uint32_t w = sure_bits[b / 32];
      int at = __popc(w & ((1u << lane) - 1));
      for (int i = 0; i < b / 32; ++i) at += __popc(sure_bits[i]);
      if ((w >> lane) & 1) out[at] = b;
    }
    return;
  }
  if (n <= kWarpBlocks) {
    // One warp holds all keys (0, below every score, for those not to be
    // chosen among) and halves the range until a bound has exactly `need`
    // keys at or above it, or a single value is left: no barrier until then.
    // (1 us less than the histograms below at 400 to 700 blocks, 1 more at 1500.)
    constexpr int GROUP = 8, GROUPS = kWarpBlocks / (32 * GROUP);
    if (warp == 0 && need > 0) {
      uint32_t k[GROUPS][GROUP], low = 0xffffffffu, top = 0;
#pragma unroll
      for (int i = 0; i < GROUPS; ++i)
#pragma unroll
        for (int j = 0; j < GROUP; ++j) {
          const int b = (i * GROUP + j) * 32 + lane;
          const bool middle = b < n && !forced(b);
          k[i][j] = i * GROUP * 32 < n && middle ? keys[b] : 0u;
          low = min(low, middle ? k[i][j] : 0xffffffffu);
          top = max(top, k[i][j]);
        }
      // At least `need` keys are >= lo, `above` (fewer than `need`) are >= hi.
      // (hi does not wrap: a finite float's key is below 0xff800000.)
      uint32_t lo = __reduce_min_sync(kFull, low), hi = __reduce_max_sync(kFull, top) + 1;
      int above = 0;
      uint32_t threshold = 0;
      for (;;) {
        if (hi - lo == 1) {
          threshold = hi;
          ties = need - above;
          break;
        }
        const uint32_t mid = lo + (hi - lo) / 2;
        int part[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < GROUPS; ++i)
          if (i * GROUP * 32 < n) {
#pragma unroll
            for (int j = 0; j < GROUP; ++j) part[j % 4] += k[i][j] >= mid;
          }
        const int c = __reduce_add_sync(kFull, (part[0] + part[1]) + (part[2] + part[3]));
        if (c == need) {
          threshold = mid;
          break;
        }
        if (c > need)
          lo = mid;
        else
          hi = mid, above = c;
      }
      if (lane == 0) {
        found[0] = static_cast<int>(threshold);
        found[1] = ties;
      }
    } else if (tid == 0) {
      found[0] = -1;  // need == 0: no key reaches it
      found[1] = 0;
    }
    __syncthreads();
    const uint32_t threshold = static_cast<uint32_t>(found[0]);
    ties = found[1];
    for (int b = tid; b < words * 32; b += NT) {
      const bool middle = b < n && !forced(b);
      const uint32_t k = middle ? keys[b] : 0u;
      const uint32_t w = __ballot_sync(kFull, middle ? k >= threshold : b < n);
      const uint32_t v = __ballot_sync(kFull, middle && k + 1 == threshold && ties > 0);
      if (lane == 0) {
        sure_bits[b / 32] = w;
        tie_bits[b / 32] = v;
      }
    }
    __syncthreads();
    // Counts before each word of 32 blocks (at most 32 words, one a lane).
    int2* before = reinterpret_cast<int2*>(hist);
    if (warp == 0) {
      const int2 x = lane < words ? make_int2(__popc(sure_bits[lane]), __popc(tie_bits[lane])) : make_int2(0, 0);
      int2 sum = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int p = __shfl_up_sync(kFull, sum.x, o), q = __shfl_up_sync(kFull, sum.y, o);
        if (lane >= o) sum.x += p, sum.y += q;
      }
      before[lane] = make_int2(sum.x - x.x, sum.y - x.y);
    }
    __syncthreads();
    const uint32_t below = (1u << lane) - 1;
    for (int b = tid; b < words * 32; b += NT) {
      const uint32_t w = sure_bits[b / 32], v = tie_bits[b / 32];
      const int2 p = before[b / 32];
      const int at = p.x + __popc(w & below), tie = p.y + __popc(v & below);
      if (((w >> lane) & 1) || (((v >> lane) & 1) && tie < ties)) out[at + min(tie, ties)] = b;
    }
    return;
  }
  {
    // The range of the middle keys.
    uint32_t kmin = 0xffffffffu, kmax = 0u;
#pragma unroll 8
    for (int b = first + tid; b < last; b += NT) {
      const uint32_t k = keys[b];
      kmin = min(kmin, k);
      kmax = max(kmax, k);
    }
    kmin = __reduce_min_sync(kFull, kmin);
    kmax = __reduce_max_sync(kFull, kmax);
    if (lane == 0) {
      warp_range[0][warp] = kmin;
      warp_range[1][warp] = kmax;
    }
    for (int i = tid; i < kBins; i += NT) hist[i] = 0;
    if (tid == 0) listed = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NWARP; ++w) {
      kmin = min(kmin, warp_range[0][w]);
      kmax = max(kmax, warp_range[1][w]);
    }
    // Rounds: the candidates, keys in [lo, lo + width], are counted in 2048
    // bins; the bin of the need-th largest is the next round's range.  Once
    // it holds few enough they are listed, and the rest is settled.
    uint32_t lo = kmin, width = kmax - kmin;
    bool in_list = false;
    int shift = max(0, 32 - __clz(width) - 11);
    if (need == 0) lo = 0xffffffffu, shift = -1;  // no middle block: none lies above
    while (shift >= 0) {
      const int items = in_list ? listed : last - first;
      for (int i0 = tid; i0 < items; i0 += kAhead * NT) {
        uint32_t k[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int i = min(i0 + u * NT, items - 1);
          k[u] = in_list ? list[i].x : keys[first + i];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (i0 + u * NT < items && k[u] >= lo && k[u] - lo <= width) atomicAdd(&hist[(k[u] - lo) >> shift], 1);
      }
      __syncthreads();
      // Thread t owns BPT bins, descending with t.
      int own[BPT], sum = 0;
      int* at = hist + BPT * (NT - 1 - tid);
#pragma unroll
      for (int i = 0; i < BPT; i += 4) {
        const int4 x = *reinterpret_cast<const int4*>(at + i);
        own[BPT - 1 - i] = x.x;
        own[BPT - 2 - i] = x.y;
        own[BPT - 3 - i] = x.z;
        own[BPT - 4 - i] = x.w;
        *reinterpret_cast<int4*>(at + i) = make_int4(0, 0, 0, 0);  // for the next round
      }
#pragma unroll
      for (int i = 0; i < BPT; ++i) sum += own[i];
      int above = block_scan<NT>(make_int2(sum, 0), warp_sums).x;
#pragma unroll
      for (int i = 0; i < BPT; ++i) {
        if (above < need && above + own[i] >= need) {
          found[0] = kBins - 1 - (tid * BPT + i);
          found[1] = above;
          found[2] = own[i];
        }
        above += own[i];
      }
      __syncthreads();
      const int in_bin = found[2];
      need -= found[1];
      lo += static_cast<uint32_t>(found[0]) << shift;
      width = (1u << shift) - 1;
      // Settled: every key of the bin is taken, or the bin is a single key.
      ties = in_bin == need ? 0x7fffffff : need;
      if (in_bin == need || shift == 0) break;
      shift = max(0, shift - 11);
      if (!in_list && in_bin <= kListed) {
        for (int i0 = tid; i0 < words * 32; i0 += 2 * kAhead * NT) {
          uint32_t k[2 * kAhead], open = 0;  // keys; which of them are candidates
#pragma unroll
          for (int u = 0; u < 2 * kAhead; ++u) k[u] = keys[min(i0 + u * NT, n - 1)];
#pragma unroll
          for (int u = 0; u < 2 * kAhead; ++u) {
            const int b = i0 + u * NT;
            if (b < words * 32) {  // the same for a whole warp
              const bool mid = b < n && !forced(b), in = mid && k[u] >= lo;
              const bool above = in && k[u] - lo > width;
              const uint32_t w = __ballot_sync(kFull, (b < n && !mid) || above);
              if (lane == 0) {
                sure_bits[b / 32] = w;
                tie_bits[b / 32] = 0;
              }
              if (in && !above) open |= 1u << u;
            }
          }
          if (open) {  // one atomic a thread that has any; their order in the list does not matter
            int at = atomicAdd(&listed, __popc(open));
#pragma unroll
            for (int u = 0; u < 2 * kAhead; ++u)
              if ((open >> u) & 1) list[at++] = make_uint2(k[u], static_cast<uint32_t>(i0 + u * NT));
          }
        }
        __syncthreads();
        in_list = true;
      }
    }
    if (in_list) {
      for (int i = tid; i < listed; i += NT)
        if (list[i].x >= lo)
          atomicOr((list[i].x > lo ? sure_bits : tie_bits) + list[i].y / 32, 1u << (list[i].y % 32));
    } else {
      for (int b = tid; b < words * 32; b += NT) {
        const uint32_t k = b < n ? keys[b] : 0u;
        const bool mid = b < n && !forced(b);
        const uint32_t w = __ballot_sync(kFull, (b < n && !mid) || (mid && k > lo));
        const uint32_t v = __ballot_sync(kFull, mid && k == lo && need > 0);
        if (lane == 0) {
          sure_bits[b / 32] = w;
          tie_bits[b / 32] = v;
        }
      }
    }
  }
  __syncthreads();

  // Ordered output from the bitmaps, a word of 32 blocks a thread.
  int2 done = make_int2(0, 0);
  for (int w0 = 0; w0 < words; w0 += NT) {
    const int w = w0 + tid;
    const uint32_t su = w < words ? sure_bits[w] : 0u, ti = w < words ? tie_bits[w] : 0u;
    const int2 mine = make_int2(__popc(su), __popc(ti));
    int2 before = block_scan<NT>(mine, warp_sums);
    before.x += done.x;
    before.y += done.y;
    if (tid == NT - 1) {
      found[0] = before.x + mine.x;
      found[1] = before.y + mine.y;
    }
    for (uint32_t m = su | ti; m; m &= m - 1) {
      const uint32_t bit = m & (0u - m);
      if ((su & bit) || before.y < ties) out[before.x + min(before.y, ties)] = w * 32 + __ffs(m) - 1;
      before.x += (su & bit) != 0;
      before.y += (ti & bit) != 0;
    }
    __syncthreads();
    done = make_int2(found[0], found[1]);
  }
}

// CTAs per (sequence, KV head): doubled while all clusters stay resident at 16
// warps a SM and one CTA cannot take the blocks in one pass.  A cluster stays
// within one of the GPU's groups of 18 to 20 SMs: where a CTA takes a whole SM,
// 76 clusters of two fit, 36 of four, but 15 of eight (a sixteenth waits for
// another to end).
constexpr int kSelWarps = 16, kSelMaxCluster = 8;

template <int D, bool BF16, int NT>
cudaError_t launch_select_t(const SelectArgs& a, int64_t cap, cudaStream_t stream) {
  auto kern = a.group <= 4 ? select_blocks_kernel<D, BF16, NT, true> : select_blocks_kernel<D, BF16, NT, false>;
  const int64_t units = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  int C = 1;
  const int64_t warps = static_cast<int64_t>(kSelWarps) * current_sm_count(152);
  auto fits = [&](int c) { return units * c * (NT / 32) * 100 <= warps * (c == 8 ? 79 : c == 4 ? 95 : 100); };
  while (C < kSelMaxCluster && fits(2 * C) && cap > C * NT) C *= 2;
  // Keys of the longest sequence, then the two bitmaps.
  const int words = static_cast<int>((cap + 31) / 32);
  const size_t smem = static_cast<size_t>(34) * words * sizeof(uint32_t);
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(units * C)), dim3(NT), smem, C, stream, a,
                            32 * words, words);
}

// More threads where a sequence may have more blocks: each warp still scores
// four chunks or more, and the first CTA's search of the keys is shared among
// more threads (8 sequences of up to 8192 blocks: 57.7 us with 128 threads, 30.5
// with 256, 27.8 with 512).
template <int D, bool BF16>
cudaError_t launch_select_n(const SelectArgs& a, cudaStream_t stream) {
  const int64_t cap = min(static_cast<int64_t>(a.max_blocks_per_seq),
                          (static_cast<int64_t>(a.max_context_len) + (1 << a.block_shift) - 1) >> a.block_shift);
  return cap <= 512    ? launch_select_t<D, BF16, 128>(a, cap, stream)
         : cap <= 2048 ? launch_select_t<D, BF16, 256>(a, cap, stream)
                       : launch_select_t<D, BF16, 512>(a, cap, stream);
}

template <int D, int KIND>
cudaError_t launch_summarize_t(const SummarizeArgs& a, cudaStream_t stream) {
  auto kern = summarize_blocks_kernel<D, KIND>;
  constexpr int HPT = 256 / (D * (KIND == 2 ? 1 : 2));
  const int64_t ctas = (static_cast<int64_t>(a.num_ids) * ((a.num_kv_heads + HPT - 1) / HPT) + 7) / 8;
  const int64_t most = resident_warp_slots(reinterpret_cast<const void*>(kern), 256, 0) / 8;
  return launch_pdl(kern, dim3(static_cast<unsigned>(min(ctas, most))), dim3(256), 0, stream, a);
}

}  // namespace

cudaError_t launch_summarize_blocks(const SummarizeArgs& a, int head_dim, bool bf16, bool fp8, cudaStream_t stream) {
  if (a.num_ids == 0) return cudaSuccess;
  if (head_dim == 128)
    return fp8 ? launch_summarize_t<128, 2>(a, stream)
               : bf16 ? launch_summarize_t<128, 1>(a, stream) : launch_summarize_t<128, 0>(a, stream);
  if (head_dim == 64)
    return fp8 ? launch_summarize_t<64, 2>(a, stream)
               : bf16 ? launch_summarize_t<64, 1>(a, stream) : launch_summarize_t<64, 0>(a, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_select_blocks(const SelectArgs& a, int head_dim, bool bf16, cudaStream_t stream) {
  if (a.num_seqs == 0) return cudaSuccess;
  if (head_dim == 128) return bf16 ? launch_select_n<128, true>(a, stream) : launch_select_n<128, false>(a, stream);
  if (head_dim == 64) return bf16 ? launch_select_n<64, true>(a, stream) : launch_select_n<64, false>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkv

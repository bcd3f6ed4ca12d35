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
// and q^+ = max(q, 0): two dp4a dot products, below 2^22 in magnitude and
// free of any summation order.  A block's score is the largest over the
// group's heads; the best ones are taken, equal scores by the lowest block.
#include "pkv_device.cuh"

namespace pkv {
namespace {

using namespace dev;

// ------------------------------------------------------------------ summary

// The smallest e >= -126 such that p + r <= 127 * 2^e, where p >= 0 and r is
// the part of an exact product that its float32 rounding p left out.
__device__ __forceinline__ int bound_exponent(float p, float r) {
  if (!(p > 0.f)) return 0;
  int x;
  const float m = frexpf(p, &x);  // p = m 2^x, m in [1/2, 1)
  const int e = (m < 0.9921875f || (m == 0.9921875f && r <= 0.f)) ? x - 7 : x - 6;
  return max(e, -126);
}

// floor (ceil) of (p + r) * 2^-e in int8 steps; r as above.  A power of two
// scales p exactly, so p + r crosses an integer only where p sits on it; a
// result that underflowed still has its sign.
__device__ __forceinline__ int step_down(float p, float r, float inv) {
  const float y = p * inv;
  int c = static_cast<int>(floorf(y));
  if (static_cast<float>(c) == y && (r < 0.f || (c == 0 && p < 0.f))) --c;
  return max(c, -127);
}
__device__ __forceinline__ int step_up(float p, float r, float inv) { return -step_down(-p, -r, inv); }

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

// A finite number for a bound: NaN (a channel without a number) counts as 0,
// an infinity as the type's largest value.
__device__ __forceinline__ float finite_bound(float x, float most) {
  return x == x ? fminf(fmaxf(x, -most), most) : 0.f;
}

// One warp per (listed block, KV head).  Rows of D * EB bytes are read as
// 16-byte vectors, 32 / LPR rows at a time; each lane keeps the packed min
// and max of its channels, the row groups are merged by shuffles, and group 0
// writes the lower bounds, group 1 the upper ones.  KIND: 0 = f16, 1 = bf16,
// 2 = FP8 (codes compared as f16, which holds every e4m3 value).
template <int D, int KIND>
__global__ void __launch_bounds__(256) summarize_blocks_kernel(const SummarizeArgs a) {
  constexpr int EB = KIND == 2 ? 1 : 2;
  constexpr bool BF16 = KIND == 1;
  constexpr int LPR = D * EB / 16;  // lanes per row
  constexpr int RPL = 32 / LPR;     // rows per load
  constexpr int NW = KIND == 2 ? 8 : 4;  // packed pairs of channels per lane
  constexpr int CH = 2 * NW;             // channels per lane
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (task >= static_cast<int64_t>(a.num_ids) * a.num_kv_heads) return;
  const int g = static_cast<int>(task % a.num_kv_heads);
  const int id = a.block_ids[task / a.num_kv_heads];
  if (id < 0 || id >= a.num_blocks) {  // -1: no block
    if (id != -1 && g == 0 && lane == 0) flag(a.dev_status, 4u);  // PKV_DEV_ERR_BLOCK
    return;
  }
  const int64_t row_bytes = static_cast<int64_t>(a.num_kv_heads) * D * EB;
  const uint8_t* src = a.k_pool + id * a.block_bytes + (lane / LPR) * row_bytes + g * (D * EB) + (lane % LPR) * 16;
  uint32_t lo[NW], hi[NW];
#pragma unroll
  for (int i = 0; i < NW; ++i) lo[i] = hi[i] = KIND == 1 ? 0x7fc07fc0u : 0x7e007e00u;  // NaN: no number yet
  for (int r0 = 0; r0 < a.block_size; r0 += 16) {
    uint4 u[16 / RPL];
#pragma unroll
    for (int i = 0; i < 16 / RPL; ++i)
      u[i] = *reinterpret_cast<const uint4*>(src + (r0 + i * RPL) * row_bytes);
#pragma unroll
    for (int i = 0; i < 16 / RPL; ++i) {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
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
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      uint32_t dump = lo[i];
      min_max2<BF16>(lo[i], dump, __shfl_xor_sync(kFull, lo[i], o));
      dump = hi[i];
      min_max2<BF16>(dump, hi[i], __shfl_xor_sync(kFull, hi[i], o));
    }

  // Values p + r, exactly: the keys themselves (r = 0), or code * scale as
  // its float32 product and the remainder.
  const float most = KIND == 0 ? 65504.f : KIND == 1 ? __uint_as_float(0x7f7f0000u) : 448.f;
  float sc = 1.f;
  if constexpr (KIND == 2) {
    sc = a.k_scale[id * a.scale_stride + g];
    if (!(sc > 0.f) || sc > 3.4028234e38f) sc = 0.f;  // no such scale: the block counts as zeros
  }
  const bool upper = (lane / LPR) & 1;
  float v[CH], top = 0.f;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const float2 l = widen2<BF16>(lo[i]), h = widen2<BF16>(hi[i]);
    const float lx = finite_bound(l.x, most), ly = finite_bound(l.y, most);
    const float hx = finite_bound(h.x, most), hy = finite_bound(h.y, most);
    top = fmaxf(top, fmaxf(fmaxf(-lx, hx), fmaxf(-ly, hy)));
    v[2 * i] = upper ? hx : lx;
    v[2 * i + 1] = upper ? hy : ly;
  }
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  const float ptop = fminf(top * sc, 3.4028234e38f);
  const int e = bound_exponent(ptop, KIND == 2 ? fmaf(top, sc, -ptop) : 0.f);
  const float inv = exp2_int(-e);
  uint32_t code[CH / 4];
#pragma unroll
  for (int i = 0; i < CH / 4; ++i) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = v[4 * i + j];
      float p = x, r = 0.f;
      if constexpr (KIND == 2) {
        p = fminf(fmaxf(x * sc, -3.4028234e38f), 3.4028234e38f);
        r = fmaf(x, sc, -p);
      }
      const int c = upper ? step_up(p, r, inv) : step_down(p, r, inv);
      w |= (static_cast<uint32_t>(c) & 0xffu) << (8 * j);
    }
    code[i] = w;
  }
  if (lane / LPR < 2) {
    const int64_t head = static_cast<int64_t>(id) * a.num_kv_heads + g;
    int8_t* dst = a.summary + (head * 2 + (upper ? 1 : 0)) * D + (lane % LPR) * CH;
    if constexpr (CH == 16)
      *reinterpret_cast<uint4*>(dst) = make_uint4(code[0], code[1], code[2], code[3]);
    else
      *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[1]);
    if (lane == 0) a.summary_scale[head] = exp2_int(e);
  }
}

// ---------------------------------------------------------------- selection

// Floats in the order of unsigned integers (no NaN); -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The integer dot products of GP heads, acc[h], summed over the LPB lanes of
// a block: halves of the heads are exchanged while more than one is left, so
// GP + log2 shuffles do instead of GP * log2.  Afterwards this lane holds the
// sums of heads first .. first + left - 1.
template <int GP, int LPB>
__device__ __forceinline__ void reduce_heads(int (&acc)[GP], int lane, int& first) {
  first = 0;
  int left = GP;
#pragma unroll
  for (int o = LPB / 2; o >= 1; o >>= 1) {
    if (left > 1) {
      const int half = left / 2;
      const bool high = lane & o;
#pragma unroll
      for (int i = 0; i < GP / 2; ++i)
        if (i < half) {
          const int send = high ? acc[i] : acc[i + half];
          const int keep = high ? acc[i + half] : acc[i];
          acc[i] = keep + __shfl_xor_sync(kFull, send, o);
        }
      first += high ? half : 0;
      left = half;
    } else {
      acc[0] += __shfl_xor_sync(kFull, acc[0], o);
    }
  }
}

constexpr int kSelThreads = 256;
constexpr int kBins = 2048;

// Exclusive prefix sums of a pair of counts over the CTA's threads.
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
  for (int w = 0; w < kSelThreads / 32; ++w)
    if (w < warp) {
      before.x += warp_sums[w].x;
      before.y += warp_sums[w].y;
    }
  return before;
}

// One cluster of C CTAs per (sequence, KV head), each CTA with a contiguous
// share of the blocks: scores into its shared memory (order keys), the
// keep-th largest key by histograms over ever narrower ranges (2048 bins
// each; every CTA adds up all CTAs' counts through distributed shared memory
// and comes to the same bin), then the chosen block numbers in order.
template <int D, bool BF16, int GP>
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const SelectArgs a) {
  constexpr int LPB = D / 16;    // lanes per block: 16 channels each
  constexpr int BPW = 32 / LPB;  // blocks per warp step
  constexpr int LEFT = GP > LPB ? GP / LPB : 1;
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) int hist[2][kBins];  // the histogram of even and odd rounds
  __shared__ int2 warp_sums[kSelThreads / 32];
  __shared__ uint32_t warp_range[2][kSelThreads / 32];
  __shared__ int2 shared_pair[2];  // what the other CTAs read: the range of keys; the counts of chosen ones
  __shared__ int found[3];  // the bin, how many keys lie above it and in it
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int64_t unit = blockIdx.x / C;
  const int s = static_cast<int>(unit / a.num_kv_heads), g = static_cast<int>(unit % a.num_kv_heads);
  const int cap = min(a.max_context_len, static_cast<int>(min(static_cast<int64_t>(a.max_blocks_per_seq) << a.block_shift,
                                                              static_cast<int64_t>(0x7fffffff))));
  int L = a.context_lens[s];
  if (L < 0 || L > cap) {
    if (g == 0 && rank == 0 && tid == 0) flag(a.dev_status, 8u);  // PKV_DEV_ERR_LENGTH
    L = L < 0 ? 0 : cap;
  }
  const int n = (L >> a.block_shift) + ((L & ((1 << a.block_shift) - 1)) ? 1 : 0);
  const int count = min(n, a.keep);
  int32_t* out = a.selected + unit * a.keep;
  if (rank == 0 && tid == 0) a.counts[unit] = count;
  if (n <= a.keep) {  // the same for every CTA of the cluster
    for (int i = rank * kSelThreads + tid; i < a.keep; i += C * kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  // This CTA's blocks are [lo_b, hi_b), whole steps of 32; keys[] holds theirs.
  const int share = ((n + C - 1) / C + 31) & ~31;
  const int lo_b = min(n, rank * share), hi_b = min(n, lo_b + share);

  // Query codes of this lane's 16 channels: negative and positive parts, and the scale per head.
  const int ch = (lane % LPB) * 16;
  int qn[GP][4], qp[GP][4], qe[GP], emax = -126;
#pragma unroll
  for (int h = 0; h < GP; ++h) {
    float x[16], top = 0.f;
    const bool live = h < a.group;
    const uint16_t* row = a.q + (static_cast<int64_t>(s) * a.num_q_heads + g * a.group + (live ? h : 0)) * D + ch;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = widen2<BF16>(live ? __ldg(reinterpret_cast<const uint32_t*>(row) + i) : 0u);
      const float most = BF16 ? __uint_as_float(0x7f7f0000u) : 65504.f;
      x[2 * i] = finite_bound(f.x, most);
      x[2 * i + 1] = finite_bound(f.y, most);
      top = fmaxf(top, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
    }
#pragma unroll
    for (int o = 1; o < LPB; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    qe[h] = top > 0.f ? bound_exponent(top, 0.f) : -126;
    emax = max(emax, qe[h]);
    const float inv = exp2_int(-qe[h]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      qn[h][w] = qp[h][w] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = __float2int_rn(x[4 * w + j] * inv);
        if (c < 0)
          qn[h][w] |= (c & 0xff) << (8 * j);
        else
          qp[h][w] |= c << (8 * j);
      }
    }
  }

  // All heads' scales times 2^-(22 + the largest exponent): the order stays,
  // and integer * scale * summary scale neither overflows nor, for the head
  // with that exponent, loses a bit (2^-22 * 2^-126 is a subnormal float32).
  float qs[GP];
#pragma unroll
  for (int h = 0; h < GP; ++h) qs[h] = exp2_int(max(qe[h] - emax - 22, -126));

  // Scores.  A warp takes 32 consecutive blocks at a time (lane j: block j's table entry and scale).
  const int first = a.first_blocks, last = n - a.last_blocks;  // blocks outside [first, last) are always taken
  const int32_t* tbl = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  uint32_t kmin = 0xffffffffu, kmax = 0u;
  for (int b0 = lo_b + warp * 32; b0 < hi_b; b0 += kSelThreads) {
    int phys = b0 + lane < hi_b ? __ldg(tbl + b0 + lane) : -1;
    if (phys < 0 || phys >= a.num_blocks) {
      if (b0 + lane < hi_b) flag(a.dev_status, 4u);  // PKV_DEV_ERR_BLOCK: the block is scored last
      phys = -1;
    }
    const float sc = phys >= 0 ? __ldg(a.summary_scale + static_cast<int64_t>(phys) * a.num_kv_heads + g) : 0.f;
#pragma unroll 4
    for (int j = 0; j < LPB; ++j) {
      const int mine = j * BPW + lane / LPB;  // which of the 32 blocks
      const int p = __shfl_sync(kFull, phys, mine);
      const float psc = __shfl_sync(kFull, sc, mine);
      const int8_t* sum = a.summary + ((static_cast<int64_t>(max(p, 0)) * a.num_kv_heads + g) * 2) * D + ch;
      const uint4 lo = *reinterpret_cast<const uint4*>(sum), hi = *reinterpret_cast<const uint4*>(sum + D);
      const int lw[4] = {static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z),
                         static_cast<int>(lo.w)};
      const int hw[4] = {static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z),
                         static_cast<int>(hi.w)};
      int acc[GP];
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        acc[h] = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) acc[h] = __dp4a(hw[w], qp[h][w], __dp4a(lw[w], qn[h][w], acc[h]));
      }
      int h0;
      reduce_heads<GP, LPB>(acc, lane, h0);
      float best = kNegInf;
#pragma unroll
      for (int i = 0; i < LEFT; ++i) {
        float f = 0.f;
        bool live = false;
#pragma unroll
        for (int h = 0; h < GP; ++h)
          if (h == h0 + i && h < a.group) {
            f = qs[h];
            live = true;
          }
        if (live) best = fmaxf(best, static_cast<float>(acc[i]) * f * psc);
      }
#pragma unroll
      for (int o = 1; o < LPB; o <<= 1) best = fmaxf(best, __shfl_xor_sync(kFull, best, o));
      const int b = b0 + mine;
      if (lane % LPB == 0 && b < hi_b) {
        const uint32_t key = p >= 0 ? order_key(best) : 0u;
        keys[b - lo_b] = key;
        if (b >= first && b < last) {
          kmin = min(kmin, key);
          kmax = max(kmax, key);
        }
      }
    }
  }
  kmin = __reduce_min_sync(kFull, kmin);
  kmax = __reduce_max_sync(kFull, kmax);
  if (lane == 0) {
    warp_range[0][warp] = kmin;
    warp_range[1][warp] = kmax;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    kmin = min(kmin, warp_range[0][w]);
    kmax = max(kmax, warp_range[1][w]);
  }
  if (tid == 0) shared_pair[0] = make_int2(static_cast<int>(kmin), static_cast<int>(kmax));
  for (int i = tid; i < kBins; i += kSelThreads) hist[0][i] = 0;
  cluster_sync();
  for (int r = 0; r < C; ++r) {
    const int2 p = cluster_load_int2(cluster_map(smem_u32(&shared_pair[0]), r));
    kmin = min(kmin, static_cast<uint32_t>(p.x));
    kmax = max(kmax, static_cast<uint32_t>(p.y));
  }
  // This CTA's middle blocks, as indices of keys[].
  const int mid0 = max(first, lo_b) - lo_b, mid1 = min(last, hi_b) - lo_b;

  // The threshold: `need` of the middle keys are taken.  Keys above `lo` are
  // taken whole, `ties` of those equal to it (lowest block first).
  int need = a.keep - a.first_blocks - a.last_blocks;
  uint32_t lo = kmin;
  int ties = 0;
  if (need > 0) {
    const int bits = 32 - __clz(kmax - kmin);
    int shift = max(0, bits - 11);
    uint32_t width = 0xffffffffu;  // keys in [lo, lo + width] are still candidates
    for (int round = 0;; ++round) {
      int* mine = hist[round & 1];  // zeroed one cluster barrier ago
      for (int b = mid0 + tid; b < mid1; b += kSelThreads) {
        const uint32_t d = keys[b] - lo;
        if (keys[b] >= lo && d <= width) atomicAdd(&mine[d >> shift], 1);
      }
      cluster_sync();
      // The other buffer was last read before this barrier.
      for (int i = tid; i < kBins; i += kSelThreads) hist[(round + 1) & 1][i] = 0;
      // Thread t owns bins 8 (255 - t) .. + 7: descending with t.
      int own[8] = {}, sum = 0;
      const uint32_t at = smem_u32(mine + 8 * (kSelThreads - 1 - tid));
      for (int r = 0; r < C; ++r) {
        const uint32_t p = cluster_map(at, r);
        const int4 x = cluster_load_int4(p), y = cluster_load_int4(p + 16);
        own[0] += y.w;
        own[1] += y.z;
        own[2] += y.y;
        own[3] += y.x;
        own[4] += x.w;
        own[5] += x.z;
        own[6] += x.y;
        own[7] += x.x;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += own[i];
      int above = block_scan(make_int2(sum, 0), warp_sums).x;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (above < need && above + own[i] >= need) {
          found[0] = kBins - 1 - (tid * 8 + i);
          found[1] = above;
          found[2] = own[i];
        }
        above += own[i];
      }
      __syncthreads();
      const int bin = found[0], in_bin = found[2];
      need -= found[1];
      lo += static_cast<uint32_t>(bin) << shift;
      if (in_bin == need || shift == 0) break;
      width = (1u << shift) - 1;
      shift = max(0, shift - 11);
    }
    // Either every key of the last bin is taken, or the bin is a single key and `need` of them are.
    ties = need;
    if (shift > 0) ties = 0x7fffffff;
  } else {
    lo = 0xffffffffu;  // no middle block: no key is above it, none of those equal is taken
  }

  // Ordered output: thread t owns a run of this CTA's consecutive blocks.
  const int run = (hi_b - lo_b + kSelThreads - 1) / kSelThreads;
  const int i1 = min(hi_b - lo_b, (tid + 1) * run);
  int2 mine = make_int2(0, 0);  // (taken for sure, equal to the threshold)
  for (int i = tid * run; i < i1; ++i) {
    if (i < mid0 || i >= mid1 || keys[i] > lo)
      ++mine.x;
    else if (keys[i] == lo)
      ++mine.y;
  }
  __syncthreads();  // warp_sums is reused
  int2 before = block_scan(mine, warp_sums);
  if (tid == kSelThreads - 1) shared_pair[1] = make_int2(before.x + mine.x, before.y + mine.y);
  cluster_sync();
  for (int r = 0; r < rank; ++r) {
    const int2 p = cluster_load_int2(cluster_map(smem_u32(&shared_pair[1]), r));
    before.x += p.x;
    before.y += p.y;
  }
  for (int i = tid * run; i < i1; ++i) {
    const bool sure = i < mid0 || i >= mid1 || keys[i] > lo;
    const bool tie = !sure && keys[i] == lo;
    if (sure || (tie && before.y < ties)) out[before.x + min(before.y, ties)] = lo_b + i;
    before.x += sure;
    before.y += tie;
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
}

// CTAs per (sequence, KV head): doubled while the batch has fewer than
// kSelTarget CTAs a SM and a CTA keeps at least kSelLeast blocks, and until
// its keys fit kSelKeys.
constexpr int kSelTarget = 3, kSelLeast = 128, kSelKeys = 1 << 15, kSelMaxCluster = 8;

template <int D, bool BF16, int GP>
cudaError_t launch_select_t(const SelectArgs& a, cudaStream_t stream) {
  auto kern = select_blocks_kernel<D, BF16, GP>;
  const int64_t cap = min(static_cast<int64_t>(a.max_blocks_per_seq),
                          (static_cast<int64_t>(a.max_context_len) + (1 << a.block_shift) - 1) >> a.block_shift);
  const int64_t units = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  int C = 1;
  while (C < kSelMaxCluster &&
         ((units * C < kSelTarget * current_sm_count(152) && cap >= 2 * C * kSelLeast) || cap > C * static_cast<int64_t>(kSelKeys)))
    C *= 2;
  const size_t smem = (static_cast<size_t>((cap + C - 1) / C) + 32) * sizeof(uint32_t);
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(units * C)), dim3(kSelThreads), smem, C, stream, a);
}

template <int D, bool BF16>
cudaError_t launch_select_g(const SelectArgs& a, cudaStream_t stream) {
  if (a.group == 1) return launch_select_t<D, BF16, 1>(a, stream);
  if (a.group == 2) return launch_select_t<D, BF16, 2>(a, stream);
  if (a.group <= 4) return launch_select_t<D, BF16, 4>(a, stream);
  return launch_select_t<D, BF16, 8>(a, stream);
}

template <int D, int KIND>
cudaError_t launch_summarize_t(const SummarizeArgs& a, cudaStream_t stream) {
  const int64_t tasks = static_cast<int64_t>(a.num_ids) * a.num_kv_heads;
  return launch_pdl(summarize_blocks_kernel<D, KIND>, dim3(static_cast<unsigned>((tasks + 7) / 8)), dim3(256), 0,
                    stream, a);
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
  if (head_dim == 128) return bf16 ? launch_select_g<128, true>(a, stream) : launch_select_g<128, false>(a, stream);
  if (head_dim == 64) return bf16 ? launch_select_g<64, true>(a, stream) : launch_select_g<64, false>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkv

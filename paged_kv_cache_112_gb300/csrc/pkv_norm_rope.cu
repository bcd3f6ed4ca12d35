// Norms of queries and keys per head, position rotation and the write path in
// one pass over a step's new rows.
//
// For every token t and head (x: the head's D values, float32 throughout):
//     q, k:  y = x * rsqrt(mean(x^2) + eps) * w            (with a weight)
//            (a, b) -> (a cos - b sin, b cos + a sin)      (the first rot_dim channels)
//     q -> q_out;  k -> its slot of the K pool (and k_out);  v -> its slot of the V pool.
// One rounding to 16 bits at the end; into FP8 pools the float32 value is
// divided by the block's scale and rounded once to e4m3.
//
// Bound: HBM bytes (each row read and written once, ~3 flops a byte): 16384
// tokens of 32 + 16 heads in 64.7 us, 6.35 TB/s.  Head counts whose groups do
// not divide into equal parts stay further from it, as a streaming warp then
// has parts of unequal size (8192 tokens: 32 + 16 heads 1.13 times the bytes'
// time, 40 + 16 1.24, 16 + 4 1.67, 6 + 12 1.85).  4097 tokens of 32 + 8 heads
// into FP8 pools take 20.0 us, 1.65 times their bytes' time, on the direct
// kernel: 52% of the issue slots, 28% of DRAM, and loads that wait for one
// another (position -> angles, sum -> weights, slot -> scale) as the largest
// stall.  With few tokens that latency alone (1.7 us for one, 3.4 for 256).
//
// Layout: D/16 lanes share a head, each holding two 16-byte chunks chosen so
// that both members of every rotated pair (i, i + rot_dim/2) sit in one lane:
// the rotation needs no exchange and the norm log2(D/16) shuffles.  A warp
// serves groups of 32 / (D/16) adjacent heads of one token and reads the
// token's angle row once for all of them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pkv_device.cuh"
#include "pkv_fp8.cuh"

namespace pkv {
namespace {

using namespace dev;

// Pairs of floats, two operations an instruction (the kernel is as near the
// issue limit as the memory's).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pair(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 halves(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& u, F2 (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[i] = pair(f.x, f.y);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(F2 a) {
  const float2 f = halves(a);
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const F2 (&x)[4]) {
  return make_uint4(narrow2<BF16>(x[0]), narrow2<BF16>(x[1]), narrow2<BF16>(x[2]), narrow2<BF16>(x[3]));
}

// Eight e4m3 codes of x / scale, the division in IEEE float32.  x times the
// reciprocal moved by 2^-21 either way is below and above the quotient (the
// reciprocal, its move and the product round by 2^-24 each, as the division
// does).  Where both have the same code, the quotient has it too; only
// elsewhere (one element in some 10^5, next to a rounding border) is the
// division carried out.  Scales whose reciprocal is not a normal number always
// divide.
__device__ __forceinline__ uint2 codes8(const F2 (&x)[4], float scale) {
  const float inv = __frcp_rn(scale);
  const float below = inv * (1.f - 4.76837158203125e-7f), above = inv * (1.f + 4.76837158203125e-7f);
  const F2 lo = pair(below, below), hi = pair(above, above);
  uint32_t c[4], differ = fabsf(inv) < 1.17549435e-38f || fabsf(inv) > 3.4e38f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = halves(mul2(x[i], lo)), q = halves(mul2(x[i], hi));
    c[i] = fp8::e4m3x2_satfinite(p.x, p.y);
    differ |= c[i] ^ fp8::e4m3x2_satfinite(q.x, q.y);
  }
  if (differ) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = halves(x[i]);
      c[i] = fp8::e4m3x2_satfinite(__fdiv_rn(f.x, scale), __fdiv_rn(f.y, scale));
    }
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// One lane's work on a head: the norm, the rotation and the stores of its two
// chunks of the head's D values, with the token's angles and the norm weights
// kept from head to head.  All lanes of a warp call together.
template <int D, bool BF16, bool FP8>
struct LaneWork {
  static constexpr int LPH = D / 16;    // lanes per head
  static constexpr int HPW = 32 / LPH;  // heads per warp
  const NormRopeArgs& a;
  int l, rc, c0, c1;  // lane of the head; rotated chunks / 2; this lane's chunks
  int first_k, first_v, heads;
  int64_t t, at, block;  // token; its row in the pools and its block
  bool writes;
  F2 cs[4], sn[4], ns[4];
  const uint16_t* w_now = nullptr;  // whose weights w0 and w1 hold
  F2 w0[4], w1[4];

  __device__ __forceinline__ LaneWork(const NormRopeArgs& args, int lane) : a(args) {
    l = lane % LPH;
    // Chunks (l, l + rot/16) while l < rot/16, then the unrotated rest in pairs.
    rc = a.rot_dim / 16;
    c0 = l < rc ? l : 2 * rc + 2 * (l - rc);
    c1 = l < rc ? l + rc : c0 + 1;
    first_k = a.num_q_heads;
    first_v = first_k + a.num_kv_heads;
    heads = first_v + a.num_kv_heads;
  }

  // Whether a token with this position is worked on: -1 marks a padding
  // token, for which nothing is written; any other position outside the
  // table (negative, where nothing is rotated) is treated alike and reported.
  __device__ __forceinline__ bool in_table(int pos) const {
    return pos >= 0 && (a.rot_dim == 0 || pos < a.max_positions);
  }
  __device__ __forceinline__ void report(int pos, int slot) const {
    if (!in_table(pos)) {
      if (pos != -1) flag(a.dev_status, 64u);  // PKV_DEV_ERR_POSITION
    } else if (slot != -1 && (slot < 0 || slot >= a.num_slots)) {
      flag(a.dev_status, 1u);  // PKV_DEV_ERR_SLOT
    }
  }

  // `row`: the position's cosines, then sines.  This lane's are those of
  // channels 8 c0 .. 8 c0 + 7 (paired with c1's), or, interleaved, of pairs
  // 4 c0 .. + 3 and 4 c1 .. + 3.
  __device__ __forceinline__ void begin(int64_t token, int slot, const float* row) {
    t = token;
    writes = slot >= 0 && slot < a.num_slots;  // -1: the token has no slot
    block = writes ? slot >> a.block_shift : 0;
    at = block * a.block_stride +
         static_cast<int64_t>(writes ? slot & ((1 << a.block_shift) - 1) : 0) * a.num_kv_heads * D;
    if (l >= rc) return;
    const int i0 = a.interleaved ? 4 * c0 : 8 * c0, i1 = a.interleaved ? 4 * c1 : 8 * c0 + 4;
    const float4 x = *reinterpret_cast<const float4*>(row + i0), y = *reinterpret_cast<const float4*>(row + i1);
    row += a.rot_dim / 2;
    const float4 z = *reinterpret_cast<const float4*>(row + i0), w = *reinterpret_cast<const float4*>(row + i1);
    cs[0] = pair(x.x, x.y), cs[1] = pair(x.z, x.w), cs[2] = pair(y.x, y.y), cs[3] = pair(y.z, y.w);
    sn[0] = pair(z.x, z.y), sn[1] = pair(z.z, z.w), sn[2] = pair(w.x, w.y), sn[3] = pair(w.z, w.w);
    ns[0] = pair(-z.x, -z.y), ns[1] = pair(-z.z, -z.w), ns[2] = pair(-w.x, -w.y), ns[3] = pair(-w.z, -w.w);
  }

  __device__ __forceinline__ void head(int h, const uint4& u0, const uint4& u1) {
    const bool is_q = h < first_k, is_v = h >= first_v;
    const int g = is_q ? h : is_v ? h - first_v : h - first_k;
    F2 x0[4], x1[4];
    widen8<BF16>(u0, x0);
    widen8<BF16>(u1, x1);
    const uint16_t* w = is_q ? a.q_weight : is_v ? nullptr : a.k_weight;
    if (__any_sync(kFull, w != nullptr)) {
      F2 ss = mul2(x0[0], x0[0]), st = mul2(x1[0], x1[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) {
        ss = fma2(x0[j], x0[j], ss);
        st = fma2(x1[j], x1[j], st);
      }
      const float2 s0 = halves(ss), s1 = halves(st);
      float sum = (s0.x + s0.y) + (s1.x + s1.y);
#pragma unroll
      for (int o = 1; o < LPH; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
      if (w) {
        if (w != w_now) {
          widen8<BF16>(__ldg(reinterpret_cast<const uint4*>(w) + c0), w0);
          widen8<BF16>(__ldg(reinterpret_cast<const uint4*>(w) + c1), w1);
          w_now = w;
        }
        const float r = rsqrtf(sum * (1.f / D) + a.eps);
        const F2 rr = pair(r, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x0[j] = mul2(mul2(x0[j], rr), w0[j]);
          x1[j] = mul2(mul2(x1[j], rr), w1[j]);
        }
      }
    }
    if (l < rc && !is_v) {
      if (a.interleaved) {  // pairs (2i, 2i + 1): chunk c holds pairs 4c .. 4c + 3
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 c = halves(cs[j / 2]), s = halves(sn[j / 2]), d = halves(cs[2 + j / 2]), e = halves(sn[2 + j / 2]);
          const float ca = j & 1 ? c.y : c.x, sa = j & 1 ? s.y : s.x, cb = j & 1 ? d.y : d.x, sb = j & 1 ? e.y : e.x;
          const float2 p = halves(x0[j]), q = halves(x1[j]);
          x0[j] = pair(p.x * ca - p.y * sa, p.y * ca + p.x * sa);
          x1[j] = pair(q.x * cb - q.y * sb, q.y * cb + q.x * sb);
        }
      } else {  // pairs (i, i + rot/2): element j of chunk c0 with element j of c1
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const F2 p = x0[j], q = x1[j];
          x0[j] = fma2(q, ns[j], mul2(p, cs[j]));
          x1[j] = fma2(p, sn[j], mul2(q, cs[j]));
        }
      }
    }
    if (h >= heads) return;
    if (is_q || (a.k_out && !is_v) || (!FP8 && !is_v && writes)) {
      const uint4 y0 = narrow8<BF16>(x0), y1 = narrow8<BF16>(x1);
      if (is_q || a.k_out) {
        uint16_t* dst = is_q ? a.q_out + t * a.q_out_stride + g * D : a.k_out + t * a.k_out_stride + g * D;
        reinterpret_cast<uint4*>(dst)[c0] = y0;
        reinterpret_cast<uint4*>(dst)[c1] = y1;
      }
      if (!FP8 && !is_q && writes) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k_pool) + at + g * D);
        dst[c0] = y0;
        dst[c1] = y1;
      }
    }
    if (is_q || !writes) return;
    if constexpr (FP8) {
      const float sc = __ldg((is_v ? a.v_scale : a.k_scale) + block * a.scale_stride + g);
      uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.v_pool : a.k_pool) + at + g * D);
      dst[c0] = codes8(x0, sc);
      dst[c1] = codes8(x1, sc);
    } else if (is_v) {  // moves bit by bit
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v_pool) + at + g * D);
      dst[c0] = u0;
      dst[c1] = u1;
    }
  }
};

// Few tokens: a warp per (token, HPW heads), everything straight from global memory.
template <int D, bool BF16, bool FP8>
__global__ void __launch_bounds__(128) norm_rope_write_kernel(const NormRopeArgs a, uint32_t parts) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t task = blockIdx.x * 4 + (threadIdx.x >> 5);
  const uint32_t token = task / parts;
  if (token >= static_cast<uint32_t>(a.num_tokens)) return;
  LaneWork<D, BF16, FP8> work(a, lane);
  const int part = static_cast<int>(task - token * parts);
  const int h = part * work.HPW + lane / work.LPH;
  const int64_t t = token;
  const uint16_t* src = h < work.first_k   ? a.q + t * a.q_stride + h * D
                        : h < work.first_v ? a.k + t * a.kv_stride + (h - work.first_k) * D
                                           : a.v + t * a.kv_stride + (h - work.first_v) * D;
  uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
  if (h < work.heads) {
    u0 = *(reinterpret_cast<const uint4*>(src) + work.c0);
    u1 = *(reinterpret_cast<const uint4*>(src) + work.c1);
  }
  const int slot = __ldg(a.slot_mapping + t);
  const int pos = a.positions ? __ldg(a.positions + t) : 0;
  if (part == 0 && lane == 0) work.report(pos, slot);
  if (!work.in_table(pos)) return;
  work.begin(t, slot, a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim);
  work.head(h, u0, u1);
}

// Many tokens: persistent warps, each streaming its share of the (token, part)
// tasks -- a part is up to kGroups * HPW adjacent heads -- through a private ring of
// bulk copies into shared memory, a stage the part's rows and the token's
// angle row.  What is in flight does not depend on registers then, the chain
// position -> angles is off the path, and no warp waits for another.  (Loaded
// by registers the kernel stayed at 5.0 TB/s whatever the heads per warp, 80
// to 90 us for 16384 tokens of 32 + 16 heads; with a CTA per token and a
// barrier a token it took 73 us.)
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

constexpr int kGroups = 4, kStages = 2, kStreamWarps = 4;

// Shared memory of one warp's ring: rows and angles, then position and slot, then the barrier of each stage.
template <int D>
constexpr int kStageBytes = kGroups * (32 / (D / 16)) * D * 2 + D * 4;
template <int D>
constexpr int kRingBytes = (kStages * (kStageBytes<D> + 16) + 127) / 128 * 128;

template <int D, bool BF16, bool FP8>
__global__ void __launch_bounds__(kStreamWarps * 32) norm_rope_stream_kernel(const NormRopeArgs a, uint32_t parts,
                                                                                int part_groups) {
  using Work = LaneWork<D, BF16, FP8>;
  constexpr int kRowBytes = D * 2, kAngles = kGroups * Work::HPW * kRowBytes;
  const int part_heads = part_groups * Work::HPW;
  extern __shared__ __align__(128) uint8_t smem[];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Work work(a, lane);
  uint8_t* ring = smem + warp * kRingBytes<D>;
  int2* info = reinterpret_cast<int2*>(ring + kStages * kStageBytes<D>);  // position and slot of each stage
  const uint32_t bars = smem_u32(info + kStages);
  if (lane == 0) {
    for (int st = 0; st < kStages; ++st) mbar_init(bars + 8 * st, 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncwarp();

  const uint32_t total = static_cast<uint32_t>(a.num_tokens) * parts;
  const uint32_t step = gridDim.x * kStreamWarps, first = blockIdx.x * kStreamWarps + warp;
  const uint32_t count = first < total ? (total - first + step - 1) / step : 0;  // this warp's tasks
  auto token_of = [&](uint32_t j) { return static_cast<int64_t>((first + j * step) / parts); };
  auto first_head = [&](uint32_t j) { return static_cast<int>((first + j * step) % parts) * part_heads; };
  auto fetch = [&](uint32_t j) {  // task j's position and slot
    if (j >= count) return make_int2(-1, -1);
    const int64_t t = token_of(j);
    return make_int2(a.positions ? __ldg(a.positions + t) : 0, __ldg(a.slot_mapping + t));
  };
  auto issue = [&](uint32_t j, int2 at) {  // lane 0
    if (j >= count) return;
    const int st = j % kStages;
    const uint32_t bar = bars + 8 * st, dst = smem_u32(ring) + st * kStageBytes<D>;
    info[st] = at;
    if (!work.in_table(at.x)) {
      mbar_arrive_expect_tx(bar, 0);
      return;
    }
    const int64_t t = token_of(j);
    const int h0 = first_head(j), h1 = min(h0 + part_heads, work.heads);
    mbar_arrive_expect_tx(bar, (h1 - h0) * kRowBytes + a.rot_dim * 4);
    auto copy = [&](const uint16_t* rows, int lo, int hi) {  // heads [lo, hi) of a kind whose first head `rows` is
      const int from = max(h0, lo), to = min(h1, hi);
      if (from < to) bulk_load(dst + (from - h0) * kRowBytes, rows + (from - lo) * D, (to - from) * kRowBytes, bar);
    };
    copy(a.q + t * a.q_stride, 0, work.first_k);
    copy(a.k + t * a.kv_stride, work.first_k, work.first_v);
    copy(a.v + t * a.kv_stride, work.first_v, work.heads);
    if (a.rot_dim) bulk_load(dst + kAngles, a.cos_sin + static_cast<int64_t>(at.x) * a.rot_dim, a.rot_dim * 4, bar);
  };

  int2 ahead = make_int2(0, 0);
  if (lane == 0) {
    int2 at[kStages];
    for (int j = 0; j < kStages; ++j) at[j] = fetch(j);
    ahead = fetch(kStages);
    for (int j = 0; j < kStages; ++j) issue(j, at[j]);
  }
  __syncwarp();
  for (uint32_t i = 0; i < count; ++i) {
    const int st = i % kStages;
    if (!__all_sync(kFull, mbar_wait_bounded(bars + 8 * st, (i / kStages) & 1, a.timeout_ns))) {
      for (uint32_t j = i; j < min(count, i + kStages); ++j)  // copies in flight land before the warp leaves
        mbar_wait_bounded(bars + 8 * (j % kStages), (j / kStages) & 1, a.timeout_ns);
      if (lane == 0) flag(a.dev_status, 16u);  // PKV_DEV_ERR_TIMEOUT; the output is undefined
      return;
    }
    const uint8_t* stage = ring + st * kStageBytes<D>;
    const int2 at = info[st];
    const int h0 = first_head(i);
    if (h0 == 0 && lane == 0) work.report(at.x, at.y);
    if (work.in_table(at.x)) {
      work.begin(token_of(i), at.y, reinterpret_cast<const float*>(stage + kAngles));
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        const int hh = k * Work::HPW + lane / Work::LPH;  // past the last head: the stage's old contents, not stored
        if (k >= part_groups || h0 + k * Work::HPW >= work.heads) break;
        const uint4* row = reinterpret_cast<const uint4*>(stage + hh * kRowBytes);
        work.head(h0 + hh, row[work.c0], row[work.c1]);
      }
    }
    __syncwarp();  // every lane is done with the stage
    if (lane == 0) {
      issue(i + kStages, ahead);
      ahead = fetch(i + kStages + 1);
    }
    __syncwarp();
  }
}

// The streaming kernel from this many head groups a SM on; below, the direct
// kernel's shorter start counts for more.  Microseconds direct / streaming at
// 81, 162, 323 and 647 groups a SM (32 + 16 heads, 16 bits): 5.8 / 7.1,
// 13.0 / 13.1, 24.0 / 20.2, 45.3 / 34.8; FP8 pools (32 + 8 heads) at 135,
// 270 and 539: 11.0 / 13.1, 20.2 / 21.1, 37.2 / 35.5.
template <bool FP8>
constexpr int kManyTasks = FP8 ? 320 : 160;

template <int D, bool BF16, bool FP8>
cudaError_t launch_t(const NormRopeArgs& a, cudaStream_t stream) {
  constexpr int HPW = 32 / (D / 16);
  const int64_t heads = a.num_q_heads + 2LL * a.num_kv_heads, groups = (heads + HPW - 1) / HPW;
  if (a.num_tokens * groups < static_cast<int64_t>(kManyTasks<FP8>) * current_sm_count(152))
    return launch_pdl(norm_rope_write_kernel<D, BF16, FP8>,
                      dim3(static_cast<unsigned>((a.num_tokens * groups + 3) / 4)), dim3(128), 0, stream, a,
                      static_cast<uint32_t>(groups));
  const int64_t parts = (groups + kGroups - 1) / kGroups, part_groups = (groups + parts - 1) / parts;
  auto kern = norm_rope_stream_kernel<D, BF16, FP8>;
  constexpr size_t smem = static_cast<size_t>(kStreamWarps) * kRingBytes<D>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (a.num_tokens * parts + kStreamWarps - 1) / kStreamWarps;
  const int64_t slots = resident_warp_slots(reinterpret_cast<const void*>(kern), kStreamWarps * 32, smem) / kStreamWarps;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas < slots ? ctas : slots)), dim3(kStreamWarps * 32), smem,
                    stream, a, static_cast<uint32_t>(parts), static_cast<int>(part_groups));
}

}  // namespace

cudaError_t launch_norm_rope_write(const NormRopeArgs& a, int head_dim, bool bf16, bool fp8, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  if (head_dim == 128)
    return fp8 ? (bf16 ? launch_t<128, true, true>(a, stream) : launch_t<128, false, true>(a, stream))
               : (bf16 ? launch_t<128, true, false>(a, stream) : launch_t<128, false, false>(a, stream));
  if (head_dim == 64)
    return fp8 ? (bf16 ? launch_t<64, true, true>(a, stream) : launch_t<64, false, true>(a, stream))
               : (bf16 ? launch_t<64, true, false>(a, stream) : launch_t<64, false, false>(a, stream));
  return cudaErrorInvalidValue;
}

}  // namespace pkv

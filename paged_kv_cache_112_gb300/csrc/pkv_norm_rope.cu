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
// Bound: HBM bytes (each row read and written once, ~3 flops a byte); with few
// tokens the latency of position -> angle row -> store.
//
// Layout: D/16 lanes share a head, each holding two 16-byte chunks chosen so
// that both members of every rotated pair (i, i + rot_dim/2) sit in one lane:
// the rotation needs no exchange and the norm log2(D/16) shuffles.  A warp
// serves 32 / (D/16) adjacent heads of one token and reads the token's angle
// row once for all of them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pkv_fp8.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void flag(int32_t* status, unsigned bit) {
  if (status) atomicOr(reinterpret_cast<unsigned*>(status), bit);
}

// Eight 16-bit values of a 16-byte chunk, widened.
template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = fp8::widen16(w[i] & 0xffffu, BF16);
    x[2 * i + 1] = fp8::widen16(w[i] >> 16, BF16);
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
  return make_uint4(narrow2<BF16>(x[0], x[1]), narrow2<BF16>(x[2], x[3]), narrow2<BF16>(x[4], x[5]),
                    narrow2<BF16>(x[6], x[7]));
}

// Eight e4m3 codes of x / scale (IEEE division).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = fp8::e4m3x2_satfinite(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <int D, bool BF16, bool FP8>
__global__ void __launch_bounds__(128) norm_rope_write_kernel(const NormRopeArgs a) {
  constexpr int LPH = D / 16;    // lanes per head
  constexpr int HPW = 32 / LPH;  // heads per warp
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.num_q_heads + 2 * a.num_kv_heads;
  const int groups = (heads + HPW - 1) / HPW;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * 4 + warp;
  if (task >= static_cast<int64_t>(a.num_tokens) * groups) return;
  const int64_t t = task / groups;
  const int h = static_cast<int>(task % groups) * HPW + lane / LPH;
  const int l = lane % LPH;
  const bool live = h < heads;
  const bool is_q = h < a.num_q_heads;
  const bool is_v = h >= a.num_q_heads + a.num_kv_heads;
  const int g = is_q ? 0 : (h - a.num_q_heads) % a.num_kv_heads;

  // Chunks c0 and c1 of the head: (l, l + rot/16) while l < rot/16, then the unrotated rest in pairs.
  const int rc = a.rot_dim / 16;
  const int c0 = l < rc ? l : 2 * rc + 2 * (l - rc);
  const int c1 = l < rc ? l + rc : c0 + 1;

  const uint16_t* src = is_q   ? a.q + t * a.q_stride + h * D
                        : is_v ? a.v + t * a.kv_stride + g * D
                               : a.k + t * a.kv_stride + g * D;
  uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
  if (live) {
    u0 = *(reinterpret_cast<const uint4*>(src) + c0);
    u1 = *(reinterpret_cast<const uint4*>(src) + c1);
  }
  const int slot = a.slot_mapping[t];
  const int pos = a.rot_dim ? a.positions[t] : 0;
  if (a.rot_dim && (pos < 0 || pos >= a.max_positions)) {
    // -1 marks a padding token; any other position outside the table is an error.  Nothing is written.
    if (pos != -1 && task % groups == 0 && lane == 0) flag(a.dev_status, 64u);  // PKV_DEV_ERR_POSITION
    return;
  }
  float x0[8], x1[8];
  widen8<BF16>(u0, x0);
  widen8<BF16>(u1, x1);

  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss += x0[i] * x0[i] + x1[i] * x1[i];
#pragma unroll
  for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
  const uint16_t* w = is_q ? a.q_weight : is_v ? nullptr : a.k_weight;
  if (w) {
    const float r = rsqrtf(ss * (1.f / D) + a.eps);
    float w0[8], w1[8];
    widen8<BF16>(__ldg(reinterpret_cast<const uint4*>(w) + c0), w0);
    widen8<BF16>(__ldg(reinterpret_cast<const uint4*>(w) + c1), w1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x0[i] *= r * w0[i];
      x1[i] *= r * w1[i];
    }
  }
  if (l < rc && !is_v) {
    const float* cs = a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim;
    const int half = a.rot_dim / 2;
    if (a.interleaved) {  // pairs (2i, 2i + 1): chunk c holds pairs 4c .. 4c + 3
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ca = __ldg(cs + 4 * c0 + i), sa = __ldg(cs + half + 4 * c0 + i);
        const float cb = __ldg(cs + 4 * c1 + i), sb = __ldg(cs + half + 4 * c1 + i);
        const float p = x0[2 * i], q = x0[2 * i + 1], y = x1[2 * i], z = x1[2 * i + 1];
        x0[2 * i] = p * ca - q * sa;
        x0[2 * i + 1] = q * ca + p * sa;
        x1[2 * i] = y * cb - z * sb;
        x1[2 * i + 1] = z * cb + y * sb;
      }
    } else {  // pairs (i, i + rot/2): element i of chunk c0 with element i of c1
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = __ldg(cs + 8 * c0 + i), s = __ldg(cs + half + 8 * c0 + i);
        const float p = x0[i], q = x1[i];
        x0[i] = p * c - q * s;
        x1[i] = q * c + p * s;
      }
    }
  }
  if (!live) return;

  if (is_q || (a.k_out && !is_v)) {
    uint16_t* dst = is_q ? a.q_out + t * a.q_out_stride + h * D : a.k_out + t * a.k_out_stride + g * D;
    reinterpret_cast<uint4*>(dst)[c0] = narrow8<BF16>(x0);
    reinterpret_cast<uint4*>(dst)[c1] = narrow8<BF16>(x1);
  }
  if (is_q) return;
  if (slot < 0 || slot >= a.num_slots) {  // -1: the token has no slot
    if (slot != -1 && !is_v && g == 0 && l == 0) flag(a.dev_status, 1u);  // PKV_DEV_ERR_SLOT
    return;
  }
  const int64_t block = slot >> a.block_shift;
  const int64_t at = block * a.block_stride +
                     (static_cast<int64_t>(slot & ((1 << a.block_shift) - 1)) * a.num_kv_heads + g) * D;
  if constexpr (FP8) {
    const float sc = (is_v ? a.v_scale : a.k_scale)[block * a.scale_stride + g];
    uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.v_pool : a.k_pool) + at);
    dst[c0] = codes8(x0, sc);
    dst[c1] = codes8(x1, sc);
  } else {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.v_pool : a.k_pool) + at);
    dst[c0] = is_v ? u0 : narrow8<BF16>(x0);  // V rows move bit by bit
    dst[c1] = is_v ? u1 : narrow8<BF16>(x1);
  }
}

template <int D, bool BF16, bool FP8>
cudaError_t launch_t(const NormRopeArgs& a, cudaStream_t stream) {
  constexpr int HPW = 32 / (D / 16);
  const int64_t groups = (a.num_q_heads + 2 * a.num_kv_heads + HPW - 1) / HPW;
  const int64_t tasks = a.num_tokens * groups;
  return launch_pdl(norm_rope_write_kernel<D, BF16, FP8>, dim3(static_cast<unsigned>((tasks + 3) / 4)), dim3(128), 0,
                    stream, a);
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

// Per-warp attention over FP8 (e4m3) tiles, shared by the partition kernels
// (pkv_decode_fp8.cu, whose head comment has the layouts and permutations)
// and the sparse decode kernel.
#pragma once

#include "pkv_device.cuh"

namespace pkv {
namespace dev {

// Four e4m3 codes (bytes 0..3 of w) -> two f16x2 (codes 0,1 in lo; 2,3 in hi;
// the lower-addressed code in the lower half).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// 16 bytes of shared memory into r[0..3].
__device__ __forceinline__ void lds128(uint32_t* r, uint32_t addr) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Attention state of one warp serving the G <= 8 query heads of one KV head
// over FP8 tiles (layout and permutations: the head of pkv_decode_fp8.cu).
template <int D>
struct WarpAttentionFp8 : SoftmaxState<D / 16> {
  static_assert(D == 128, "FP8 tiles are one 128-byte line per head row");
  static constexpr int KT = D / 16;
  using Base = SoftmaxState<KT>;
  using Base::acc;
  uint32_t qf[KT][2];  // f16x2: q[head gr][32tq + 4kk + {0,1}] and {2,3}

  // Loads the group's query rows (heads >= G read as 0) in the permuted
  // order and returns the power of two by which they were scaled down (1
  // for f16; for bf16, 2^e with the group's max |q| / 2^e below 2^15).
  // OWN: a power of two per head, that of head gr, from the head's largest
  // finite |q|: a head beside one of far larger or infinite queries keeps its
  // bits.
  template <bool QBF16, bool OWN = false>
  __device__ __forceinline__ float load_q(const uint16_t* qhead0, int G, int lane) {
    const int gr = lane >> 2, tq = lane & 3;
    const bool live = gr < G;
    const uint4* src = reinterpret_cast<const uint4*>(qhead0 + (live ? gr : 0) * D + 32 * tq);
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
    float down = 1.f;
    if constexpr (QBF16) {
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 f = unpack_bf16(w[i]);
        const float x = fabsf(f.x), y = fabsf(f.y);
        if constexpr (OWN)
          amax = fmaxf(amax, fmaxf(x < INFINITY ? x : 0.f, y < INFINITY ? y : 0.f));
        else
          amax = fmaxf(amax, fmaxf(x, y));
      }
#pragma unroll
      for (int o = 1; o < (OWN ? 4 : 32); o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
      // 2^e >= amax / 2^14.99: exponent of amax minus 14, at least 0.
      const int ex = static_cast<int>((__float_as_uint(amax) >> 23) & 0xff) - 127;
      const int e = min(max(ex - 14, OWN ? -100 : 0), 120);
      const float mul = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, exact
      down = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 f = unpack_bf16(w[i]);
        w[i] = pack_f16(f.x * mul, f.y * mul);
      }
    }
#pragma unroll
    for (int kk = 0; kk < KT; ++kk) {
      qf[kk][0] = w[2 * kk];
      qf[kk][1] = w[2 * kk + 1];
    }
    return down;
  }

  // NT tiles at once (independent chains interleave; one softmax update for
  // all of them).  Tile t: K at sK[t], V at sK[t] + VOFF, nv[t] valid
  // tokens (rows >= nv are masked, whatever they hold), sl2k[t] = log2(e) *
  // softmax scale * q prescale * K scale, pv[t] = V scale in the
  // accumulator's unit (a power of two chosen per chunk of tiles).  OWN: sl2k
  // times up_a and up_b for this lane's heads 2tq and 2tq + 1 (load_q's
  // powers); pv[t] times kWeightUp, and lift[t] bounds log2 of pv[t] /
  // kWeightUp: a weight times the V scale is at most 1 then, whatever the
  // scales, so that a tile of large scale and little weight costs the others
  // no bits.
  static constexpr int kWeightUpLog2 = 14;
  template <int NT, int VOFF = 2048, bool OWN = false>
  __device__ __forceinline__ void tiles(const uint32_t (&sK)[NT], const int (&nv)[NT], const float (&sl2k)[NT],
                                        const float (&pv)[NT], int lane, float up_a = 1.f, float up_b = 1.f,
                                        const float* lift = nullptr) {
    const int gr = lane >> 2, tq = lane & 3;
    // K: rows gr and gr+8 (same swizzle phase), chunks 2tq and 2tq+1.
    const uint32_t off0 = gr * 128 + (((2 * tq) ^ gr) << 4);
    const uint32_t off1 = gr * 128 + (((2 * tq + 1) ^ gr) << 4);
    uint32_t kw[NT][2][8];  // words i = codes [32tq + 4i, +4) of rows gr, gr+8
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      lds128(kw[t][0], sK[t] + off0);
      lds128(kw[t][0] + 4, sK[t] + off1);
      lds128(kw[t][1], sK[t] + 1024 + off0);
      lds128(kw[t][1] + 4, sK[t] + 1024 + off1);
    }
    // Scores S^T[token][head]; per tile, even and odd k-steps in separate chains.
    float c[NT][2][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[t][0][j] = c[t][1][j] = 0.f;
#pragma unroll
    for (int kk = 0; kk < KT; ++kk)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint32_t a[4];
        e4m3x4_to_f16x4(kw[t][0][kk], a[0], a[2]);
        e4m3x4_to_f16x4(kw[t][1][kk], a[1], a[3]);
        mma_16816<false>(c[t][kk & 1], a, qf[kk][0], qf[kk][1]);
      }
    // V: rows 2tq, 2tq+1, 2tq+8, 2tq+9, chunk gr (codes of dims 16gr .. 16gr+15).
    const int r0 = 2 * tq;
    const uint32_t voff[4] = {static_cast<uint32_t>(r0 * 128 + ((gr ^ r0) << 4)),
                              static_cast<uint32_t>((r0 + 1) * 128 + ((gr ^ (r0 + 1)) << 4)),
                              static_cast<uint32_t>((r0 + 8) * 128 + ((gr ^ r0) << 4)),
                              static_cast<uint32_t>((r0 + 9) * 128 + ((gr ^ (r0 + 1)) << 4))};
    uint32_t vw[NT][4][4];  // [tile][row 2tq, 2tq+1, 2tq+8, 2tq+9][word]
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) lds128(vw[t][r], sK[t] + VOFF + voff[r]);

    float sc[4 * NT], p[4 * NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float fa = OWN ? sl2k[t] * up_a : sl2k[t], fb = OWN ? sl2k[t] * up_b : sl2k[t];
      sc[4 * t] = (c[t][0][0] + c[t][1][0]) * fa;
      sc[4 * t + 1] = (c[t][0][1] + c[t][1][1]) * fb;
      sc[4 * t + 2] = (c[t][0][2] + c[t][1][2]) * fa;
      sc[4 * t + 3] = (c[t][0][3] + c[t][1][3]) * fb;
      if (gr >= nv[t]) sc[4 * t] = sc[4 * t + 1] = kNegInf;
      if (gr + 8 >= nv[t]) sc[4 * t + 2] = sc[4 * t + 3] = kNegInf;
    }
    this->template online_update_lazy<NT, OWN>(sc, p, lift);

    // P^T (times the V scale) as f16 hi + lo parts, two MMAs per tile: off by
    // 2^-22 of itself or, where f16's subnormals end, by 2^-25 in the
    // accumulator's unit (OWN: 2^-39 of a unit at most twice the largest
    // weight times V scale).
    uint32_t pb[NT][4];  // hi (tokens 0-7, 8-15), lo (tokens 0-7, 8-15)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float q0 = p[4 * t] * pv[t], q1 = p[4 * t + 1] * pv[t];
      const float q2 = p[4 * t + 2] * pv[t], q3 = p[4 * t + 3] * pv[t];
      const uint32_t h0 = pack_f16(q0, q1), h1 = pack_f16(q2, q3);
      const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
      const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
      pb[t][0] = movmatrix_trans(h0);
      pb[t][1] = movmatrix_trans(h1);
      pb[t][2] = movmatrix_trans(pack_f16(q0 - f0.x, q1 - f0.y));
      pb[t][3] = movmatrix_trans(pack_f16(q2 - f1.x, q3 - f1.y));
      // V codes of tokens >= nv may be anything (NaN codes included): zero them.
      if (nv[t] < kBlockSize) {
        const int row[4] = {r0, r0 + 1, r0 + 8, r0 + 9};
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (row[r] >= nv[t]) vw[t][r][0] = vw[t][r][1] = vw[t][r][2] = vw[t][r][3] = 0u;
      }
    }
    // V^T A fragment of M-tile mt: rows gr / gr+8 are dims 16gr+2mt / +1,
    // k = tokens.  A byte permute pairs a dim's codes of tokens 2tq and
    // 2tq+1 (and 2tq+8, 2tq+9), which convert to the f16x2 the MMA wants.
#pragma unroll
    for (int mt = 0; mt < KT; ++mt) {
      const int w = mt >> 1;
      const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint32_t va[4];
        e4m3x4_to_f16x4(__byte_perm(vw[t][0][w], vw[t][1][w], sel), va[0], va[1]);
        e4m3x4_to_f16x4(__byte_perm(vw[t][2][w], vw[t][3][w], sel), va[2], va[3]);
        mma_16816<false>(acc[mt], va, pb[t][0], pb[t][1]);
        mma_16816<false>(acc[mt], va, pb[t][2], pb[t][3]);
      }
    }
  }

  // acc[mt][0..1] hold dim 16gr + 2mt of heads a, b; acc[mt][2..3] dim +1:
  // a lane owns dims [16gr, 16gr+16) of its two heads.
  __device__ __forceinline__ void store_final(void* out, int64_t out_head0, int G, int dtype, int lane) const {
    const int gr = lane >> 2, tq = lane & 3;
    const int ha = 2 * tq, hb = ha + 1;
    const float ia = this->l_a > 0.f ? 1.f / this->l_a : 0.f;
    const float ib = this->l_b > 0.f ? 1.f / this->l_b : 0.f;
#pragma unroll
    for (int mt = 0; mt < KT; ++mt) {
      const int d = 16 * gr + 2 * mt;
      if (ha < G) {
        store_out(out, (out_head0 + ha) * D + d, acc[mt][0] * ia, dtype);
        store_out(out, (out_head0 + ha) * D + d + 1, acc[mt][2] * ia, dtype);
      }
      if (hb < G) {
        store_out(out, (out_head0 + hb) * D + d, acc[mt][1] * ib, dtype);
        store_out(out, (out_head0 + hb) * D + d + 1, acc[mt][3] * ib, dtype);
      }
    }
  }

  __device__ __forceinline__ void store_partial(float* ws_acc, float2* ws_ml, int64_t rec0, int64_t rec_stride,
                                                int G, int lane) const {
    const int gr = lane >> 2, tq = lane & 3;
    const int ha = 2 * tq, hb = ha + 1;
    const int64_t ra = rec0 + ha * rec_stride, rb = rec0 + hb * rec_stride;
#pragma unroll
    for (int j = 0; j < KT / 2; ++j) {  // dims 16gr + 4j .. +3: M-tiles 2j, 2j+1
      if (ha < G)
        *reinterpret_cast<float4*>(ws_acc + ra * D + 16 * gr + 4 * j) =
            make_float4(acc[2 * j][0], acc[2 * j][2], acc[2 * j + 1][0], acc[2 * j + 1][2]);
      if (hb < G)
        *reinterpret_cast<float4*>(ws_acc + rb * D + 16 * gr + 4 * j) =
            make_float4(acc[2 * j][1], acc[2 * j][3], acc[2 * j + 1][1], acc[2 * j + 1][3]);
    }
    if (gr == 0) {
      if (ha < G) ws_ml[ra] = make_float2(this->m_a, this->l_a);
      if (hb < G) ws_ml[rb] = make_float2(this->m_b, this->l_b);
    }
  }
};

// 2^e for an integer e in [-126, 127], exactly.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// The factor 2^(from - to) that moves the accumulator from unit 2^from to
// unit 2^to (to > from), exactly, down to the f32 subnormals and 0 (the
// first unit of a pair starts at 2^-126, so the gap can exceed 126).
__device__ __forceinline__ float unit_change(int from, int to) { return ldexpf(1.f, from - to); }

// The accumulator's unit for a chunk of tiles: 2^-e with 2^e <= the
// largest V scale of the chunk (over the warp) < 2^(e+1), so P * scale /
// unit stays below 2 and well inside the f16 range.
__device__ __forceinline__ int chunk_exponent(float vs) {
  float m = vs;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  const int e = static_cast<int>((__float_as_uint(m) >> 23) & 0xff) - 127;
  return min(max(e, -126), 126);
}

}  // namespace dev
}  // namespace pkv

// 4-bit pools: e2m1 codes (sign, two exponent bits, one mantissa bit: 0, 1/2,
// 1, 3/2, 2, 3, 4, 6) with an e4m3 scale for every 16 channels of a token.
//
// Layout.  A block holds, per KV head and per 16 tokens, one record
//     [16 tokens][D / 2] bytes of codes (the even channel in the low half),
//     [16 tokens][D / 16] bytes of scales,
// 9 D bytes.  A tile (16 tokens of a head) is then one contiguous copy of
// 16-byte pieces, codes and scales together; the records of a block's heads
// follow one another, so the CTAs of neighbouring heads read one range.
#pragma once

#include "pkv_device.cuh"

namespace pkv {
namespace fp4 {

template <int D>
struct Record {
  static constexpr int kRowBytes = D / 2;    // codes of a token
  static constexpr int kRowScales = D / 16;  // scales of a token
  static constexpr int kScalesAt = 16 * kRowBytes;
  static constexpr int kBytes = 9 * D;
};

// Eight values to codes, element i in bits 4i ..: nearest, ties to the even
// code, magnitudes beyond 6 saturate.
__device__ __forceinline__ uint32_t e2m1x8(const float2 (&x)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y));
  return r;
}

// Four bytes of codes to four pairs of f16 (the low half's value in the lower half).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The bits of a where m has ones, those of b elsewhere.
__device__ __forceinline__ uint32_t select(uint32_t a, uint32_t b, uint32_t m) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xe4;" : "=r"(r) : "r"(a), "r"(b), "r"(m));
  return r;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }

}  // namespace fp4

namespace dev {

// Attention state of one warp serving the G <= 8 query heads of one KV head
// over 4-bit tiles (see SoftmaxState; mma.sync m16n8k16 as WarpAttention).
//
// A value is code * scale: two significant bits times four, at most 2688 and
// a multiple of 2^-10, so the f16 product that enters the MMA is exact.  A
// softmax weight enters in two f16 parts, its rounding and what that leaves
// (off by 2^-22 of the weight at most; the first part alone is off by 2^-11,
// which put f16 rows up to 27% further from their values than their own rounding).
// With G <= 4 (NARROW) the parts share a product of eight columns: columns 4 to
// 7 are the same heads once more, so their lanes have the same weights and pass
// on the second parts.  With more heads they take a product each.
// Microseconds with one part, with two in a shared product and in one each: 8
// long contexts of 32 + 8 heads 179.7, 181.9, 192.9, 16 sequences of 8000 tokens
// 35.8, 37.6, 39.7; with 64 + 8 heads, 256 sequences, 136.8 and 144.5.
//
// Order of the fragments: within an MMA, channels, tokens and output dims may
// be permuted as long as both operands agree.  Lane (gr, tq) takes channels
// [D/4 tq, + D/4) of K: 16 bytes a token for D = 128, and the two quantisation
// groups they hold.  MMA row r of a half tile is token r/2 + 4 (r & 1), so a
// lane's V tokens are tq, tq + 4 (+ 8): the four lanes of a quad read adjacent
// rows.  Of V it takes dims [D/8 gr, + D/8): one group's scale a token.  A
// dim's codes of two tokens are brought into one byte by a select, which one
// conversion turns into the f16 pair the MMA wants.
template <int D, bool NARROW>
struct WarpAttentionFp4 : SoftmaxState<D / 16> {
  static constexpr int KT = D / 16;
  using Rec = fp4::Record<D>;
  using Base = SoftmaxState<KT>;
  using Base::acc;
  uint32_t qf[KT][2];  // f16x2: q[head gr][D/4 tq + 4kk + {0,1}] and {2,3}
  float fa, fb;          // log2 units a product with heads 2tq and 2tq + 1
  float grow_a, grow_b;  // kGrow in products
  // Weights lie up to 2^kGrow above the reference m and enter the product
  // times 2^kUp: below 2^15, and f16's floor of 2^-25 is 2^-33 of the largest
  // weight at most.
  static constexpr float kGrow = 7.f, kUp = 8.f;

  // The group's query rows (heads >= G read as 0; NARROW: rows 4 to 7 are 0 to 3 again), the sign of sl2 = log2(e) *
  // softmax scale * the head's K scale with them.  bf16 queries become f16 with
  // a power of two per head, from its largest finite |q|.
  template <bool QBF16>
  __device__ __forceinline__ void load_q(const uint16_t* qhead0, int G, int lane, float sl2) {
    const int gr = lane >> 2, tq = lane & 3, head = NARROW ? gr & 3 : gr;
    const bool live = head < G;
    const uint4* src = reinterpret_cast<const uint4*>(qhead0 + (live ? head : 0) * D + D / 4 * tq);
    uint32_t w[2 * KT];
#pragma unroll
    for (int i = 0; i < KT / 2; ++i) {
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
      for (int i = 0; i < 2 * KT; ++i) {
        const float2 f = unpack_bf16(w[i]);
        const float x = fabsf(f.x), y = fabsf(f.y);
        amax = fmaxf(amax, fmaxf(x < INFINITY ? x : 0.f, y < INFINITY ? y : 0.f));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
      const int ex = static_cast<int>((__float_as_uint(amax) >> 23) & 0xff) - 127;
      const int e = min(max(ex - 14, -100), 120);  // |q| 2^-e is below 2^15
      const float mul = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      down = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
      for (int i = 0; i < 2 * KT; ++i) {
        const float2 f = unpack_bf16(w[i]);
        w[i] = pack_f16(f.x * mul, f.y * mul);
      }
    }
#pragma unroll
    for (int kk = 0; kk < KT; ++kk) {
      qf[kk][0] = w[2 * kk];
      qf[kk][1] = w[2 * kk + 1];
    }
    const uint32_t flip = sl2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int kk = 0; kk < KT; ++kk) {
      qf[kk][0] ^= flip;
      qf[kk][1] ^= flip;
    }
    // A factor of 0 would make a masked score 0 times infinity.
    const float mag = fmaxf(fabsf(sl2), 1e-30f);
    fa = fmaxf(mag * __shfl_sync(kFull, down, 8 * tq), 1e-36f);
    fb = fmaxf(mag * __shfl_sync(kFull, down, 8 * tq + 4), 1e-36f);
    grow_a = kGrow / fa;
    grow_b = kGrow / fb;
  }

  __device__ __forceinline__ static uint32_t lds32(uint32_t addr) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr));
    return r;
  }
  __device__ __forceinline__ static uint32_t lds8(uint32_t addr) {
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(addr));
    return r;
  }
  template <int N>
  __device__ __forceinline__ static void lds(uint32_t (&r)[N], uint32_t addr) {
    if constexpr (N == 4)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                   : "r"(addr));
    else if constexpr (N == 2)
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
    else
      r[0] = lds32(addr);
  }

  // NT tiles at once: K records at sK[t], V records Rec::kBytes further.  With
  // MASKED, bit r of mask[t] is set where token r counts (the others are left
  // out whatever they hold); without, every token does.  m_a and m_b are in
  // products, not in log2 units, until finish().
  template <int NT, bool MASKED>
  __device__ __forceinline__ void tiles(const uint32_t (&sK)[NT], const uint32_t (&mask)[NT], int lane) {
    const int gr = lane >> 2, tq = lane & 3;
    const int tok = (gr >> 1) + 4 * (gr & 1);
    constexpr int KW = D / 32, VW = D / 64;  // words of a lane's codes a K row and a V row
    uint32_t kw[NT][2][KW], ks[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        lds<KW>(kw[t][r], sK[t] + (tok + 8 * r) * Rec::kRowBytes + tq * (D / 8));
        const uint32_t at = sK[t] + Rec::kScalesAt + (tok + 8 * r) * Rec::kRowScales;
        if constexpr (D == 128) {
          asm volatile("{\n\t.reg .u16 h;\n\tld.shared.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}"
                       : "=r"(ks[t][r])
                       : "r"(at + 2 * tq));
        } else {
          ks[t][r] = lds8(at + tq);
        }
      }
    float c[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const __half2 s0 = fp4::as_half2(fp4::e4m3x2_to_f16(ks[t][0])), s1 = fp4::as_half2(fp4::e4m3x2_to_f16(ks[t][1]));
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        uint32_t x[4], y[4];
        fp4::e2m1x8_to_f16(kw[t][0][w], x);
        fp4::e2m1x8_to_f16(kw[t][1][w], y);
        const __half2 f0 = w < 2 ? __low2half2(s0) : __high2half2(s0), f1 = w < 2 ? __low2half2(s1) : __high2half2(s1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // k-step 2w + h
          const uint32_t a[4] = {fp4::mul_f16x2(x[2 * h], f0), fp4::mul_f16x2(y[2 * h], f1),
                                 fp4::mul_f16x2(x[2 * h + 1], f0), fp4::mul_f16x2(y[2 * h + 1], f1)};
          if (w + h == 0)
            mma_16816_first(c[t], a, qf[0][0], qf[0][1]);
          else
            mma_16816<false>(c[t], a, qf[2 * w + h][0], qf[2 * w + h][1]);
        }
      }
    }
    // V: tokens tq, tq + 4, tq + 8, tq + 12, dims [D/8 gr, + D/8).
    uint32_t vw[NT][4][VW], vs[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t sV = sK[t] + Rec::kBytes;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        lds<VW>(vw[t][r], sV + (tq + 4 * r) * Rec::kRowBytes + gr * (D / 16));
        vs[t][r] = lds8(sV + Rec::kScalesAt + (tq + 4 * r) * Rec::kRowScales + (D == 128 ? gr : gr >> 1));
        // A token that does not count may hold anything: its scale is 0.
        if (MASKED && !((mask[t] >> (tq + 4 * r)) & 1u)) vs[t][r] = 0u;
      }
    }
    float mx_a = kNegInf, mx_b = kNegInf;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if constexpr (MASKED) {
        if (!((mask[t] >> tok) & 1u)) c[t][0] = c[t][1] = kNegInf;
        if (!((mask[t] >> (tok + 8)) & 1u)) c[t][2] = c[t][3] = kNegInf;
      }
      mx_a = fmaxf(fmaxf(mx_a, c[t][0]), c[t][2]);
      mx_b = fmaxf(fmaxf(mx_b, c[t][1]), c[t][3]);
    }
    // The reference follows the running maximum only where a score lies more
    // than kGrow above it: few steps exchange maxima and scale the sums.
    if (__any_sync(kFull, (mx_a > this->m_a + grow_a) | (mx_b > this->m_b + grow_b))) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx_a = fmaxf(mx_a, __shfl_xor_sync(kFull, mx_a, o));
        mx_b = fmaxf(mx_b, __shfl_xor_sync(kFull, mx_b, o));
      }
      const float mn_a = fmaxf(this->m_a, mx_a), mn_b = fmaxf(this->m_b, mx_b);
      const float al_a = mn_a > this->m_a ? ex2_approx((this->m_a - mn_a) * fa) : 1.f;  // m = -inf: 0
      const float al_b = mn_b > this->m_b ? ex2_approx((this->m_b - mn_b) * fb) : 1.f;
      this->l_a *= al_a;
      this->l_b *= al_b;
#pragma unroll
      for (int mt = 0; mt < KT; ++mt) {
        acc[mt][0] *= al_a;
        acc[mt][1] *= al_b;
        acc[mt][2] *= al_a;
        acc[mt][3] *= al_b;
      }
      this->m_a = mn_a;
      this->m_b = mn_b;
    }
    const float u_a = this->m_a == kNegInf ? 0.f : kUp - this->m_a * fa;
    const float u_b = this->m_b == kNegInf ? 0.f : kUp - this->m_b * fb;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float q0 = ex2_approx(fmaf(c[t][0], fa, u_a)), q1 = ex2_approx(fmaf(c[t][1], fb, u_b));
      const float q2 = ex2_approx(fmaf(c[t][2], fa, u_a)), q3 = ex2_approx(fmaf(c[t][3], fb, u_b));
      this->l_a += q0 + q2;
      this->l_b += q1 + q3;
      const uint32_t h0 = pack_f16(q0, q1), h1 = pack_f16(q2, q3);
      const uint32_t r0 = rest(q0, q1, h0), r1 = rest(q2, q3, h1);
      const uint32_t p0 = movmatrix_trans(NARROW && tq >= 2 ? r0 : h0), p1 = movmatrix_trans(NARROW && tq >= 2 ? r1 : h1);
      [[maybe_unused]] uint32_t o0, o1;
      if constexpr (!NARROW) {
        o0 = movmatrix_trans(r0);
        o1 = movmatrix_trans(r1);
      }
      const __half2 s0 = fp4::as_half2(fp4::e4m3x2_to_f16(__byte_perm(vs[t][0], vs[t][1], 0x0040)));
      const __half2 s1 = fp4::as_half2(fp4::e4m3x2_to_f16(__byte_perm(vs[t][2], vs[t][3], 0x0040)));
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        constexpr uint32_t kLow = 0x0f0f0f0fu;
        uint32_t x[4][4];  // even dims, odd dims of tokens tq and tq + 4; of tq + 8 and tq + 12
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t A = vw[t][2 * h][w], B = vw[t][2 * h + 1][w];
          fp4::e2m1x8_to_f16(fp4::select(A, B << 4, kLow), x[2 * h]);
          fp4::e2m1x8_to_f16(fp4::select(A >> 4, B, kLow), x[2 * h + 1]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // M-tile 4w + j: rows gr, gr + 8 are dims D/8 gr + 2 (4w + j), + 1
          const uint32_t a[4] = {fp4::mul_f16x2(x[0][j], s0), fp4::mul_f16x2(x[1][j], s0),
                                 fp4::mul_f16x2(x[2][j], s1), fp4::mul_f16x2(x[3][j], s1)};
          mma_16816<false>(acc[4 * w + j], a, p0, p1);
          if constexpr (!NARROW) mma_16816<false>(acc[4 * w + j], a, o0, o1);
        }
      }
    }
  }

  // What rounding to f16 left of two weights.
  __device__ __forceinline__ static uint32_t rest(float x, float y, uint32_t rounded) {
    const float2 r = __half22float2(fp4::as_half2(rounded));
    return pack_f16(x - r.x, y - r.y);
  }

  // The sums of all lanes; the maxima in log2 units.
  __device__ __forceinline__ void finish() {
    this->finish_sums();
    if constexpr (NARROW) {
#pragma unroll
      for (int mt = 0; mt < KT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][i] += __shfl_xor_sync(kFull, acc[mt][i], 2);
    }
    this->m_a *= fa;
    this->m_b *= fb;
  }
};

}  // namespace dev
}  // namespace pkv

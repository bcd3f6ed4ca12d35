// Single-token attention over a range of a sequence's tokens: a sliding
// window and the first tokens (16-bit and 4-bit pools), or a partition of the
// whole history (4-bit pools).
//
// For sequence s of L tokens and each query head h of KV head g's group,
//     out[s][h] = sum_t softmax_t(scale * q[s][h] . k_t) v_t,
//     windows:    t < sinks or t >= L - window     (t < L),
//     partitions: t in [part * size, part * size + size).
//
// Bound over 16-bit pools: HBM bytes of the visible K and V, each read once for
// all query heads of the group (256 windows of 70B-class heads, f16: 290 us, the
// rate of a plain copy).  Over 4-bit pools: the latency of a warp's chain of
// steps (copy, conversion, product, maximum, exponential, product) at 16 warps a
// SM; 304 instructions a warp and tile of 2304 bytes (D = 128), some 144 of them
// conversions, scales, products and fragment loads.  57% of the issue slots and
// 52% of DRAM are used at 2 contexts of 65536 tokens, and a warp's largest stall
// is an instruction's fixed latency.  8 of 32 to 128 thousand, 8 KV heads: 182
// us, 75% of a copy's rate.
//
// A cluster of C CTAs of NW warps serves one (s, g, partition).  The visible
// 16-token tiles are dealt to its warps in turn; each streams its tiles
// through a private ring of copies (16 bits: TMA boxes; 4 bits: records, by
// asynchronous copies of 16 bytes a lane) and keeps its own online-softmax state
// on the tensor cores.  The states meet in shared memory, first a CTA's, then through
// distributed shared memory the cluster's.  Windows need no workspace then;
// partitions write the partial records that the reduce kernel merges.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "pkv_fp4.cuh"

namespace pkv {
namespace {

using namespace dev;

constexpr int kMaxCluster = 8;

// The visible part of a sequence: tokens [0, sinks) and [low, L), as a list of
// tiles [0, head) and [head + skip, ...), `count` in all.
struct Visible {
  int sinks, low, head, skip, count;

  __device__ __forceinline__ Visible(int L, int window, int first) {
    low = max(0, L - window);
    sinks = min(first, low);
    head = (sinks + kTile - 1) / kTile;
    skip = max(0, low / kTile - head);
    count = (L + kTile - 1) / kTile - skip;
  }
  __device__ __forceinline__ int tile(int j) const { return j < head ? j : j + skip; }
  // Bit r: token 16 T + r is visible.
  __device__ __forceinline__ uint32_t mask(int T, int L) const {
    auto below = [&](int x) { return (1u << max(0, min(kTile, x - T * kTile))) - 1u; };
    return below(L) & (below(sinks) | ~below(low));
  }
};

// POOL: 16 or 4 bits.  Warps a CTA NW, stages a warp NST; a stage is NT tiles.
template <int D, int POOL, int NW, int NST, int NT>
struct Ring {
  static constexpr int kTileBytes = POOL == 4 ? fp4::Record<D>::kBytes : kTile * D * 2;
  static constexpr int kStageBytes = 2 * NT * kTileBytes;
  static constexpr int kState = 8 * (D + 4) + 16;  // a warp's saved state: 8 rows, running max and sum of each head
  static constexpr int kWarpBytes = NST * kStageBytes > kState * 4 ? NST * kStageBytes : kState * 4;
  static constexpr size_t kInboxAt = static_cast<size_t>(NW) * (kWarpBytes + 8 * NST);
  static constexpr size_t smem(int C) {
    return kInboxAt + (C > 1 ? (8 * D + 16 * kMaxCluster) * sizeof(float) : 0);
  }
  static_assert(POOL == 4 || kWarpBytes % 1024 == 0, "TMA tiles sit on 1024-byte boundaries");
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int POOL>
constexpr int kTilesAStep = POOL == 4 ? 2 : 1;

// Least CTAs a SM, for the compiler: 16 warps' registers (0: as many as it likes).  4-bit pools with 64 channels
// and more than two warps a CTA do better with what it takes by itself (8 of 60000 tokens 73 us for 76).
template <int D, int POOL, int NW>
constexpr int kLeastCtas = POOL == 4 && (D == 128 || NW == 2) ? 16 / NW : 0;

// NARROW: 4-bit pools with at most four heads a group (WarpAttentionFp4).
template <int D, bool BF16, int POOL, bool NARROW, int NW, int NST>
__global__ void __launch_bounds__(NW * 32, kLeastCtas<D, POOL, NW>)
    decode_window_kernel(const DecodeArgs a, const WindowArgs wa, const __grid_constant__ CUtensorMap tmap_k,
                         const __grid_constant__ CUtensorMap tmap_v) {
  constexpr int NT = kTilesAStep<POOL>;
  using R = Ring<D, POOL, NW, NST, NT>;
  using Att = std::conditional_t<POOL == 4, WarpAttentionFp4<D, NARROW>, WarpAttention<D, BF16, true>>;
  constexpr int kRow = D + 4;  // floats between a saved state's head rows
  extern __shared__ __align__(1024) uint8_t smem[];
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  if (C > 1) cluster_arrive();  // see the wait before the merge
  griddep_wait();
  griddep_launch_dependents();
  if (POOL != 4 && smem_misaligned(smem, a.dev_status)) return;  // the same for every CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Units in ascending partition index: those past a sequence's end come last.
  const int64_t unit = blockIdx.x / C;
  const int g = static_cast<int>(unit % a.num_kv_heads);
  const int64_t rest = unit / a.num_kv_heads;
  const int s = static_cast<int>(rest % a.num_seqs), part = static_cast<int>(rest / a.num_seqs);
  const int G = a.group;
  const int32_t* tbl = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  const int tshift = a.block_shift - 4;         // log2 of tiles per block
  const int W = C * NW, w0 = rank * NW + warp;  // this warp's steps of NT tiles of the list: w0, w0 + W, ...

  const int L = clamp_len(a, a.context_lens[s], part == 0 && g == 0 && rank == 0 && threadIdx.x == 0);
  const int nparts = wa.window > 0 ? 1 : max(1, (L + a.partition_size - 1) / a.partition_size);
  if (part >= nparts) return;  // never with windows or clusters: max_parts is 1 there
  const Visible vis(L, wa.window > 0 ? wa.window : L, wa.sinks);
  const int tile0 = wa.window > 0 ? 0 : part * (a.partition_size / kTile);
  const int tiles = wa.window > 0 ? vis.count : min(vis.count - tile0, a.partition_size / kTile);
  const int steps = (tiles + NT - 1) / NT, cnt = steps > w0 ? (steps - w0 + W - 1) / W : 0;
  // The place in the list of tile n of the warp (tile n % NT of its step n / NT).
  auto place = [&](int n) { return (n / NT * W + w0) * NT + n % NT; };
  // Its table entry: the physical block, or -1: none there, or unusable and left out.
  auto fetch = [&](int n) {
    const int j = place(n);
    if (n >= cnt * NT || j >= tiles) return -1;
    const int phys = __ldg(tbl + (vis.tile(tile0 + j) >> tshift));  // inside the table: L is clamped to it
    if (static_cast<unsigned>(phys) < static_cast<unsigned>(a.num_blocks)) return phys;
    flag(a.dev_status, 4u);  // PKV_DEV_ERR_BLOCK
    return -1;
  };
  uint8_t* mine = smem + static_cast<size_t>(warp) * R::kWarpBytes;
  const uint32_t buf = smem_u32(mine);
  const uint16_t* q0 = a.q + (static_cast<int64_t>(s) * a.num_q_heads + g * G) * D;
  float sl2 = a.scale_log2, post = 1.f;
  uint32_t gone = 0;  // bit st * NT + u: tile u of stage st is not there
  Att at;
  at.reset();
  if constexpr (POOL == 4) {
    // Records by 16-byte asynchronous copies of all lanes: a warp's addresses
    // differ by the lane alone, and a step is waited for without a barrier.
    // (Bulk copies take their operands from uniform registers: some 20
    // instructions to issue one, 40 a tile of the 370 there were.)
    const int per_block = static_cast<int>(a.block_stride / R::kTileBytes);
    auto record = [&](int n) {  // the tile's record in the pool, or -1
      const int phys = fetch(n);
      return phys < 0 ? -1 : phys * per_block + (g << tshift) + (vis.tile(tile0 + place(n)) & ((1 << tshift) - 1));
    };
    const uint8_t* k4 = wa.k4 + 16 * lane;
    const uint8_t* v4 = wa.v4 + 16 * lane;
    // Lane j holds the record of the warp's tile j of a chunk of 32.
    int cur = record(lane), ahead = record(32 + lane);
    auto issue = [&](int i) {
      if (((i * NT) & 31) == 0 && i > 0) {
        cur = ahead;
        ahead = record(i * NT + 32 + lane);
      }
      const int st = i % NST;
      gone &= ~(((1u << NT) - 1u) << (st * NT));
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        const int rec = __shfl_sync(kFull, cur, (i * NT + u) & 31);
        if (rec < 0) {
          gone |= 1u << (st * NT + u);
          continue;
        }
        const int64_t off = static_cast<int64_t>(rec) * R::kTileBytes;
        const uint32_t dst = buf + st * R::kStageBytes + 2 * u * R::kTileBytes + 16 * lane;
#pragma unroll
        for (int c = 0; c < R::kTileBytes; c += 512)
          if (c + 512 <= R::kTileBytes || c + 16 * lane < R::kTileBytes) {
            copy16(dst + c, k4 + off + c);
            copy16(dst + R::kTileBytes + c, v4 + off + c);
          }
      }
    };
#pragma unroll
    for (int i = 0; i < NST; ++i) {
      if (i < cnt) issue(i);
      copies_commit();
    }
    if (a.k_scale) sl2 *= __ldg(a.k_scale + g);
    if (a.v_scale) post *= __ldg(a.v_scale + g);
    at.template load_q<BF16>(q0, G, lane, sl2);
    // Places in the list between which every token is visible: [0, plain_first) and [plain_from, plain_to).
    const int plain_first = vis.sinks / kTile, plain_from = vis.head + ((vis.low & (kTile - 1)) ? 1 : 0);
    const int plain_to = L / kTile - vis.skip;
    for (int i = 0; i < cnt; ++i) {
      copies_wait<NST - 1>();
      __syncwarp();
      const int st = i % NST, j = place(i * NT), jj = tile0 + j;
      const uint32_t absent = (gone >> (st * NT)) & ((1u << NT) - 1u);
      uint32_t m[NT], sK[NT];
#pragma unroll
      for (int u = 0; u < NT; ++u) sK[u] = buf + st * R::kStageBytes + 2 * u * R::kTileBytes;
      if (absent == 0 && jj + NT <= plain_to && (jj >= plain_from || jj + NT <= plain_first)) {
        at.template tiles<NT, false>(sK, m, lane);
      } else {
#pragma unroll
        for (int u = 0; u < NT; ++u) m[u] = (absent >> u) & 1u ? 0u : vis.mask(vis.tile(jj + u), L);
        at.template tiles<NT, true>(sK, m, lane);
      }
      __syncwarp();
      if (i + NST < cnt) issue(i + NST);
      copies_commit();
    }
    copies_wait<0>();
    at.finish();
  } else {
    const uint32_t bars = smem_u32(smem + static_cast<size_t>(NW) * R::kWarpBytes) + 8 * NST * warp;
    if (lane == 0) {
      for (int st = 0; st < NST; ++st) mbar_init(bars + 8 * st, 1);
      fence_barrier_init();
      fence_proxy_async_smem();
    }
    __syncwarp();
    // Lane j holds the table entry of the warp's tile j of a chunk of 32.
    int cur = fetch(lane), ahead = fetch(32 + lane);
    auto issue = [&](int i) {
      if ((i & 31) == 0 && i > 0) {
        cur = ahead;
        ahead = fetch(i + 32 + lane);
      }
      const int st = i % NST;
      const int phys = __shfl_sync(kFull, cur, i & 31);
      gone = (gone & ~(1u << st)) | (phys < 0 ? 1u << st : 0u);
      if (lane != 0) return;
      const uint32_t bar = bars + 8 * st, dst = buf + st * R::kStageBytes;
      const int row0 = (vis.tile(tile0 + place(i)) & ((1 << tshift) - 1)) * kTile;
      mbar_arrive_expect_tx(bar, R::kStageBytes);
      tma_tile<D>(dst, &tmap_k, row0, g, max(phys, 0), bar);
      tma_tile<D>(dst + R::kTileBytes, &tmap_v, row0, g, max(phys, 0), bar);
    };
    auto wait = [&](int i) { return mbar_wait_bounded(bars + 8 * (i % NST), (i / NST) & 1, a.timeout_ns); };
    for (int i = 0; i < min(cnt, NST); ++i) issue(i);
    at.load_q(q0, G, lane);
    for (int i = 0; i < cnt; ++i) {
      if (!__all_sync(kFull, wait(i))) {
        for (int j = i; j < min(cnt, i + NST); ++j) wait(j);  // copies in flight land before the warp goes on
        if (lane == 0) flag(a.dev_status, 16u);               // PKV_DEV_ERR_TIMEOUT; the output is undefined
        break;
      }
      const uint32_t stage = buf + (i % NST) * R::kStageBytes;
      const uint32_t m = (gone >> (i % NST)) & 1u ? 0u : vis.mask(vis.tile(tile0 + place(i)), L);
      if (m) at.template tile<true>(stage, stage + R::kTileBytes, static_cast<int>(m), sl2, lane);
      __syncwarp();
      if (i + NST < cnt) issue(i + NST);
    }
    at.finish_sums();
    post = 1.f / Att::kWeightUp;
  }

  // Save this warp's state: rows [8][kRow], running max [8], running sum [8].
  {
    float* st = reinterpret_cast<float*>(mine);
    const int gr = lane >> 2, tq = lane & 3;
    float* ra = st + (2 * tq) * kRow;
    float* rb = ra + kRow;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      const int d0 = POOL == 4 ? D / 8 * gr + 2 * mt : 16 * mt + gr, d1 = POOL == 4 ? d0 + 1 : d0 + 8;
      ra[d0] = at.acc[mt][0];
      rb[d0] = at.acc[mt][1];
      ra[d1] = at.acc[mt][2];
      rb[d1] = at.acc[mt][3];
    }
    if (gr == 0) {
      st[8 * kRow + 2 * tq] = at.m_a;
      st[8 * kRow + 2 * tq + 1] = at.m_b;
      st[8 * kRow + 8 + 2 * tq] = at.l_a;
      st[8 * kRow + 8 + 2 * tq + 1] = at.l_b;
    }
  }
  __syncthreads();
  // Merge over the warps, four channels a thread:
  //     M = max m_w, acc = sum 2^(m_w - M) acc_w, l = sum 2^(m_w - M) l_w.
  auto merged = [&](int h, int d, float& M, float4& o, float& l) {
    const float* st[NW];
    float m[NW];
    M = kNegInf;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      st[w] = reinterpret_cast<const float*>(smem + static_cast<size_t>(w) * R::kWarpBytes);
      m[w] = st[w][8 * kRow + h];
      M = fmaxf(M, m[w]);
    }
    const float mu = M == kNegInf ? 0.f : M;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    l = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float c = exp2f(m[w] - mu);
      const float4 v = *reinterpret_cast<const float4*>(st[w] + h * kRow + d);
      o.x += v.x * c;
      o.y += v.y * c;
      o.z += v.z * c;
      o.w += v.w * c;
      l += st[w][8 * kRow + 8 + h] * c;
    }
  };
  const int64_t head0 = static_cast<int64_t>(s) * a.num_q_heads + g * G;
  auto store4 = [&](int e, float4 o, float l) {
    const float inv = l == 0.f ? 0.f : post / l;  // a sum that is no number makes the row none
    store_out(a.out, head0 * D + e, o.x * inv, a.out_dtype);
    store_out(a.out, head0 * D + e + 1, o.y * inv, a.out_dtype);
    store_out(a.out, head0 * D + e + 2, o.z * inv, a.out_dtype);
    store_out(a.out, head0 * D + e + 3, o.w * inv, a.out_dtype);
  };
  if (C == 1) {
    for (int e = 4 * threadIdx.x; e < G * D; e += 4 * NW * 32) {
      const int h = e / D, d = e % D;
      float M, l;
      float4 o;
      merged(h, d, M, o, l);
      if (nparts == 1) {
        store4(e, o, l);
      } else {
        const int64_t rec = (head0 + h) * a.max_parts + part;
        *reinterpret_cast<float4*>(a.ws_acc + rec * D + d) = make_float4(o.x * post, o.y * post, o.z * post, o.w * post);
        // A sum that is no number: over the other parts, and above the zero that the join asks of a sum.
        if (d == 0) a.ws_ml[rec] = l == l ? make_float2(M, l) : make_float2(3e38f, __int_as_float(0x7f800000));
      }
    }
    return;
  }
  // CTA r merges elements [r * per, r * per + per) of the group's rows over
  // the cluster: every CTA stores its part of them, and its heads' max and
  // sum, into r's shared memory.
  const int per = G * D / C;  // a multiple of 4: D is at least 64, C at most 8
  float* inbox = reinterpret_cast<float*>(smem + R::kInboxAt);  // [C][per], then [C][8] max, [C][8] sum
  float* inbox_m = inbox + 8 * D;
  float* inbox_l = inbox_m + 8 * kMaxCluster;
  cluster_wait();  // every CTA has begun
  for (int e = 4 * threadIdx.x; e < G * D; e += 4 * NW * 32) {
    const int h = e / D, d = e % D, to = e / per;
    float M, l;
    float4 o;
    merged(h, d, M, o, l);
    cluster_store_float4(cluster_map(smem_u32(inbox + rank * per + (e - to * per)), to), o);
    if (d / 4 < C) {  // head h's max and sum, to CTA d / 4
      cluster_store_float(cluster_map(smem_u32(inbox_m + rank * 8 + h), d / 4), M);
      cluster_store_float(cluster_map(smem_u32(inbox_l + rank * 8 + h), d / 4), l);
    }
  }
  cluster_sync();
  for (int k = 4 * threadIdx.x; k < per; k += 4 * NW * 32) {
    const int e = rank * per + k, h = e / D;
    float M = kNegInf, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < C) M = fmaxf(M, inbox_m[r * 8 + h]);
    const float mu = M == kNegInf ? 0.f : M;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < C) {
        const float c = exp2f(inbox_m[r * 8 + h] - mu);
        const float4 v = *reinterpret_cast<const float4*>(inbox + r * per + k);
        o.x += v.x * c;
        o.y += v.y * c;
        o.z += v.z * c;
        o.w += v.w * c;
        l += inbox_l[r * 8 + h] * c;
      }
    store4(e, o, l);
  }
}

// The kernel with NW warps a CTA, and what launching it in clusters of C takes.
template <int D, bool BF16, int POOL, bool NARROW, int NW>
struct Launch {
  static constexpr int NST = POOL == 4 ? 2 : D == 64 ? 3 : 2;
  using R = Ring<D, POOL, NW, NST, kTilesAStep<POOL>>;
  static constexpr auto kernel = decode_window_kernel<D, BF16, POOL, NARROW, NW, NST>;

  // Clusters of C that the current device holds at a time (a cluster stays
  // within one of the GPU's groups of SMs, so fewer than SMs / C).
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
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = R::smem(C);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), R::smem(kMaxCluster)) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      return 1;
    }
    slot.store(n, std::memory_order_release);
    return n;
  }

  static cudaError_t launch(const DecodeArgs& a, const WindowArgs& w, int C, const CUtensorMap& tk,
                            const CUtensorMap& tv, cudaStream_t stream) {
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), R::smem(kMaxCluster));
    if (e != cudaSuccess) return e;
    const int64_t units = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads * a.max_parts;
    return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(units * C)), dim3(NW * 32), R::smem(C), C, stream, a,
                              w, tk, tv);
  }
};

// Microseconds that `units` units of up to `tiles` tiles take with NW warps a CTA
// and C CTAs a unit, `held` clusters at a time: the sparse decode's estimate
// (pkv_sparse_decode.cu has the reasoning), whose 16-bit constants hold here.
// 4-bit pools: fitted to 18 shapes measured with each NW and C (8 to 2048 units
// of 10 to 514 tiles): the form of the lowest cost is 2% slower than the best
// one in the mean, 10% at the most.  A SM takes its tiles at the rate of the
// conversions, 34 GB a second, not of the memory.  Microseconds, 4 bits (with
// weights in one part, 1 to 5% less than now):
//   8 of 514 tiles: 9.1 with 8 warps in clusters of 8, 13.0 of 4, 37.5 alone;
//   72 of 514: 22.0 with 8 warps of 4, 23.7 of 2, 32.6 with 4 of 2, 39.6 with 8 alone;
//   512 of 258: 60.8 with 4 warps of 2, 65.2 with 8 alone, 89.6 with 2;
//   2048 of 18: 28.9 with 2 warps alone, 45.3 with 8.  16 bits:
//   8 of 514: 11.7 with 8 warps of 8, 17.1 of 4; 72 of 514: 47.9 with 8 of 2, 56.0 alone;
//   512 of 66: 46.3 with 2 alone, 53.1 with 8.
template <int D, int POOL>
float form_cost(int64_t units, int64_t tiles, int group, int NW, int C, int held, int64_t sms) {
  constexpr bool kFour = POOL == 4;
  constexpr float kStartUs = kFour ? 2.5f : 3.5f, kTileUs = D == 64 ? 0.6f : 0.9f;
  constexpr float kSmBytes = kFour ? 34e3f : D == 64 ? 60e3f : 75e3f;  // a microsecond
  constexpr float kTileBytes = 2.f * (kFour ? fp4::Record<D>::kBytes : kTile * D * 2);
  const float bytes_us = kFour ? 4.2e6f : 6.4e6f;
  const int64_t full = (static_cast<int64_t>(held) * C + sms - 1) / sms;  // CTAs a SM holds
  const int64_t per_sm = C == 1 ? std::min((units + sms - 1) / sms, full) : units * C <= sms ? 1 : full;
  constexpr int NT = kTilesAStep<POOL>;
  const int64_t n = NT * (((tiles + NT - 1) / NT + NW * C - 1) / (NW * C));  // tiles of a warp
  const float tile = std::max(kTileUs, static_cast<float>(per_sm * NW) * (kTileBytes / kSmBytes));
  const float start = kStartUs + (C > 1 ? 0.4f + 0.1f * static_cast<float>(group) : 0.f);
  const float wave = start + tile * static_cast<float>(n), waves = static_cast<float>(units) / static_cast<float>(held);
  const float exposed = units > held ? wave * (0.5f + 0.15f * (waves - 1.f)) / static_cast<float>(full) : 0.f;
  const float bytes = static_cast<float>(units) * static_cast<float>(tiles) * kTileBytes;
  return std::max(static_cast<float>((units + held - 1) / held) * wave, start + bytes / bytes_us + exposed) +
         0.25f * wave;
}

struct Form {
  int nw = 8, c = 1;
  float cost = 0.f;  // microseconds
};

// The form of the lowest cost; `clusters`: a unit may be shared by CTAs.
template <int D, bool BF16, int POOL, bool NARROW>
Form best_form(int64_t units, int64_t tiles, int group, bool clusters) {
  using Two = Launch<D, BF16, POOL, NARROW, 2>;
  using Four = Launch<D, BF16, POOL, NARROW, 4>;
  using Eight = Launch<D, BF16, POOL, NARROW, 8>;
  const int64_t sms = current_sm_count(152);
  Form best;
  auto consider = [&](int NW, int C, int held) {
    const float cost = form_cost<D, POOL>(units, tiles, group, NW, C, held, sms);
    if (best.cost == 0.f || cost < best.cost) best = Form{NW, C, cost};
  };
  if (!clusters) {
    // Partitions: alike, and none but the last short.  Once there are more than
    // four-warp CTAs at a time, CTAs of two warps leave less of the last wave empty,
    // and pay for it with twice the chain of a warp's steps: worth it for
    // partitions of up to 512 tokens, and for longer ones while they stay within one
    // wave and groups are small.  Microseconds of one sequence with four warps and
    // two, D = 128, in units (KV heads x partitions) of tokens: G = 4, 784 of
    // 1024 32.5, 30.6, 1000 of 1024 36.8, 37.5, 1400 of 1024 49.6, 52.6, 784 of 512
    // 22.3, 19.5, 1400 of 512 32.7, 32.9, 2400 of 512 48.5, 43.5, 784 of 256 17.3, 14.2,
    // 2400 of 256 34.9, 29.7, but 496 of 1024 23.3, 24.5; G = 8, 784 of 1024 34.7,
    // 38.9, 784 of 512 23.9, 24.0, 1800 of 256 29.7, 27.8.  Of 78 shapes with more units
    // than that, of both head sizes, 68 take two warps by this rule: 8% less time in
    // the mean, 18% less at best, 6% more at worst.
    const int resident = Four::resident(1);
    if (units > resident && (tiles <= 32 || (group <= 4 && units <= Two::resident(1))))
      consider(2, 1, Two::resident(1));
    else
      consider(4, 1, resident);
    return best;
  }
  consider(4, 1, Four::resident(1));
  consider(8, 1, Eight::resident(1));
  consider(2, 1, Two::resident(1));
  for (int C = 2; C <= kMaxCluster && units * C <= 8 * sms; C *= 2) {
    consider(8, C, Eight::resident(C));
    consider(4, C, Four::resident(C));
  }
  return best;
}

int64_t longest_of(const DecodeArgs& a) {
  return std::min<int64_t>(a.max_context_len, static_cast<int64_t>(a.max_blocks_per_seq) << a.block_shift);
}
int64_t tiles_of(int64_t tokens) { return std::max<int64_t>(1, (tokens + kTile - 1) / kTile); }

template <int D, bool BF16, int POOL, bool NARROW>
cudaError_t launch_t(const DecodeArgs& a, const WindowArgs& w, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads * a.max_parts;
  const int64_t seen = w.window > 0 ? static_cast<int64_t>(w.window) + w.sinks : a.partition_size;
  const Form f = best_form<D, BF16, POOL, NARROW>(units, tiles_of(std::min(longest_of(a), seen)), a.group, w.window > 0);
  switch (f.nw) {
    case 2: return Launch<D, BF16, POOL, NARROW, 2>::launch(a, w, 1, tk, tv, stream);
    case 4: return Launch<D, BF16, POOL, NARROW, 4>::launch(a, w, f.c, tk, tv, stream);
    default: return Launch<D, BF16, POOL, NARROW, 8>::launch(a, w, f.c, tk, tv, stream);
  }
}

// A history in partitions takes a second kernel, which joins them, and leaves
// SMs without work where there are few; over a cluster it takes one launch, but
// not more than eight SMs.  Microseconds of histories of 8 KV heads, whole and
// in partitions of 1024: 1 of 4000 tokens 6.3 and 11.0, 4 of 10000 16.1 and
// 19.2, 1 of 40000 26.9 and 19.0, 16 of 8000 39.5 and 36.0, 64 of 2000 alike.
// Lengths differ, and only the longest is known here: whole has to be the
// faster one with every history that long and with one of them, by more than
// the estimates' error where there are many (16 of 8000: 5% apart).
template <int D, bool BF16, bool NARROW>
bool whole_t(const DecodeArgs& a) {
  const int64_t longest = longest_of(a), in_part = std::min<int64_t>(longest, a.partition_size);
  constexpr float kJoinUs = 2.f;
  auto wins = [&](int64_t units) {
    return 1.05f * best_form<D, BF16, 4, NARROW>(units, tiles_of(longest), a.group, true).cost <
           best_form<D, BF16, 4, NARROW>(units * a.max_parts, tiles_of(in_part), a.group, false).cost + kJoinUs;
  };
  return wins(a.num_kv_heads) && wins(static_cast<int64_t>(a.num_seqs) * a.num_kv_heads);
}

template <int POOL, bool NARROW>
cudaError_t launch_p(const DecodeArgs& a, const WindowArgs& w, const CUtensorMap& tk, const CUtensorMap& tv,
                     int head_dim, bool bf16, cudaStream_t stream) {
  if (head_dim == 128)
    return bf16 ? launch_t<128, true, POOL, NARROW>(a, w, tk, tv, stream)
                : launch_t<128, false, POOL, NARROW>(a, w, tk, tv, stream);
  if (head_dim == 64)
    return bf16 ? launch_t<64, true, POOL, NARROW>(a, w, tk, tv, stream)
                : launch_t<64, false, POOL, NARROW>(a, w, tk, tv, stream);
  return cudaErrorInvalidValue;
}

template <bool NARROW>
bool whole_p(const DecodeArgs& a, int head_dim, bool bf16) {
  if (head_dim == 64) return bf16 ? whole_t<64, true, NARROW>(a) : whole_t<64, false, NARROW>(a);
  return bf16 ? whole_t<128, true, NARROW>(a) : whole_t<128, false, NARROW>(a);
}

bool narrow(const DecodeArgs& a) { return a.group <= 4; }

}  // namespace

bool decode_whole_fp4(const DecodeArgs& a, int head_dim, bool bf16) {
  if (a.num_seqs == 0 || a.max_parts <= 1) return true;
  return narrow(a) ? whole_p<true>(a, head_dim, bf16) : whole_p<false>(a, head_dim, bf16);
}

cudaError_t launch_decode_window(const DecodeArgs& a, const WindowArgs& w, const CUtensorMap& tmap_k,
                                 const CUtensorMap& tmap_v, int head_dim, bool bf16, bool fp4, cudaStream_t stream) {
  if (a.num_seqs == 0) return cudaSuccess;
  if (!fp4) return launch_p<16, false>(a, w, tmap_k, tmap_v, head_dim, bf16, stream);
  return narrow(a) ? launch_p<4, true>(a, w, tmap_k, tmap_v, head_dim, bf16, stream)
                   : launch_p<4, false>(a, w, tmap_k, tmap_v, head_dim, bf16, stream);
}

}  // namespace pkv

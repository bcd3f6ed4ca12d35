// Single-token attention over selected blocks.
//
// For each sequence s and KV head g a list of logical blocks is given
// (pkv_select_blocks, or the caller's own choice), and every query head h of
// the group attends to those blocks' tokens alone:
//     out[s][h] = sum_t softmax_t(scale * q[s][h] . k_t) v_t,
//                 t in {b * B + o : b selected, o < B, t < L}.
//
// Bound: HBM bytes of the selected K and V rows (each read once; all query
// heads of the group share them); with few units the latency of length ->
// list -> table entry -> tile.  (256 sequences of 64 blocks, 8 KV heads: 155.6
// us, 6.6 TB/s; 8 of 128 over FP8 pools: 12.3 us, 4 of them before the first
// tile and after the last, on 128 of the SMs; one of 128: 5.4 us.)
//
// One cluster of C CTAs of NW warps per (s, g).  The list's 16-token tiles are
// dealt to the cluster's warps in turn; each warp streams its tiles through a
// private ring of TMA copies and keeps its own online-softmax state on the
// tensor cores (WarpAttention, WarpAttentionFp8).  The states meet in shared
// memory, first a CTA's, then through distributed shared memory the
// cluster's, so one launch writes final rows and no workspace is needed.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "pkv_fp8_attention.cuh"

namespace pkv {
namespace {

using namespace dev;

constexpr int kSparseMaxCluster = 8;

// A tile's place: physical block, or -1 for a tile to be skipped, first row
// and valid rows.
struct TilePlace {
  int phys, row0, nv;
};

template <int D, bool BF16, bool FP8, int NW, int NST>
__global__ void __launch_bounds__(NW * 32) decode_sparse_kernel(const DecodeArgs a, const SparseArgs sp,
                                                                const __grid_constant__ CUtensorMap tmap_k,
                                                                const __grid_constant__ CUtensorMap tmap_v) {
  constexpr int EB = FP8 ? 1 : 2;
  using Geom = TileGeom<D, EB>;
  using Att = std::conditional_t<FP8, WarpAttentionFp8<128>, WarpAttention<D, BF16, true>>;
  constexpr int kRow = D + 4;                    // floats between a saved state's head rows
  constexpr int kState = 8 * kRow + 16;          // 8 rows, then running max and sum of each head
  // Shared memory: rings, barriers, then what the cluster's CTAs send: per
  // CTA its share of the rows, and running max and sum of each head.
  constexpr size_t kInboxAt = static_cast<size_t>(NW) * NST * (Geom::kStageBytes + 8);
  static_assert(kState * 4 <= NST * Geom::kStageBytes, "a saved state must fit its warp's ring");
  extern __shared__ __align__(1024) uint8_t smem[];
  cluster_arrive();  // see the wait before the merge
  griddep_wait();
  griddep_launch_dependents();
  if (smem_misaligned(smem, a.dev_status)) return;  // the same for every CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int64_t unit = blockIdx.x / C;
  const int s = static_cast<int>(unit / a.num_kv_heads), g = static_cast<int>(unit % a.num_kv_heads);
  const int G = a.group, B = 1 << a.block_shift;
  const int32_t* list = sp.selected + unit * sp.keep;
  const int32_t* tbl = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  const int tshift = a.block_shift - 4;     // log2 of tiles per block
  const int W = C * NW, w0 = rank * NW + warp;  // this warp's tiles of the list: w0, w0 + W, ...

  // The list entry of the warp's tile i, the one before it, and its table
  // entry: read before the length and the count are known (inside the list
  // and the table whatever they are), so the chain is list -> table -> tile.
  struct Entry {
    int block, prev, phys;
  };
  auto fetch = [&](int i) {
    Entry r{-1, -1, -1};
    const int64_t e = (static_cast<int64_t>(i) * W + w0) >> tshift;
    if (e >= sp.keep) return r;
    r.block = __ldg(list + e);
    r.prev = e > 0 ? __ldg(list + e - 1) : -1;
    if (r.block >= 0 && r.block < a.max_blocks_per_seq) r.phys = __ldg(tbl + r.block);
    return r;
  };
  const int raw_len = a.context_lens[s];
  int count = sp.counts[unit];
  const Entry first = fetch(lane);
  const int L = clamp_len(a, raw_len, g == 0 && rank == 0 && threadIdx.x == 0);
  const int nblk = (L >> a.block_shift) + ((L & (B - 1)) ? 1 : 0);
  if (count < 0 || count > sp.keep) {
    if (rank == 0 && threadIdx.x == 0) flag(a.dev_status, 128u);  // PKV_DEV_ERR_SELECT
    count = count < 0 ? 0 : sp.keep;
  }
  const int tiles = L > 0 ? count << tshift : 0;
  const int cnt = tiles > w0 ? (tiles - w0 + W - 1) / W : 0;

  // Place of this warp's tile i.  A list entry counts when it is larger than
  // its predecessor and inside the sequence: every entry of an ascending list,
  // no token twice.  A list that is not ascending is flagged where it descends
  // or repeats; as nothing is known of the entries further back, a block that
  // comes again behind another one counts again.
  auto place = [&](int i, const Entry& r) {
    TilePlace p{-1, 0, 0};
    if (i >= cnt) return p;
    if (r.block <= r.prev || r.block < 0 || r.block >= nblk) {
      flag(a.dev_status, 128u);  // PKV_DEV_ERR_SELECT
      return p;
    }
    if (r.phys < 0 || r.phys >= a.num_blocks) {
      flag(a.dev_status, 4u);  // PKV_DEV_ERR_BLOCK
      return p;
    }
    p.phys = r.phys;
    p.row0 = ((i * W + w0) & ((1 << tshift) - 1)) * kTile;
    p.nv = max(0, min(kTile, L - r.block * B - p.row0));
    return p;
  };

  WarpRing<D, NST, EB> ring{smem_u32(smem + static_cast<size_t>(warp) * NST * Geom::kStageBytes),
                            smem_u32(smem + static_cast<size_t>(NW) * NST * Geom::kStageBytes) + 8 * NST * warp};
  ring.init(lane);
  // Lane j holds the place (and scales) of the warp's tile j of a chunk of
  // 32; the previous chunk's scales stay until its last tile is done.
  TilePlace cur = place(lane, first);
  Entry ahead = fetch(32 + lane);
  auto scale_of = [&](const float* sc, int phys) {
    return phys >= 0 ? __ldg(sc + static_cast<int64_t>(phys) * a.scale_stride + g) : 0.f;
  };
  // With each V scale goes its exponent: |v scale| < 2^ve.
  auto exponent_of = [](float x) { return static_cast<float>(static_cast<int>((__float_as_uint(x) >> 23) & 0xff) - 126); };
  float ks = 0.f, vs = 0.f, ve = 0.f, ks_prev = 0.f, vs_prev = 0.f, ve_prev = 0.f;
  int chunk = 0;
  if constexpr (FP8) {
    ks = scale_of(a.k_scale, cur.phys);
    vs = scale_of(a.v_scale, cur.phys);
    ve = exponent_of(vs);
  }
  uint32_t stage_nv = 0;  // 8 bits per stage: valid rows of its tile
  static_assert(NST <= 4, "stage_nv");
  auto issue = [&](int j) {
    if ((j & 31) == 0 && j > 0) {
      cur = place(j + lane, ahead);
      ahead = fetch(j + 32 + lane);
      if constexpr (FP8) {
        ks_prev = ks;
        vs_prev = vs;
        ve_prev = ve;
        ks = scale_of(a.k_scale, cur.phys);
        vs = scale_of(a.v_scale, cur.phys);
        ve = exponent_of(vs);
        chunk = j >> 5;
      }
    }
    const int st = j % NST, from = j & 31;
    const int phys = __shfl_sync(kFull, cur.phys, from);
    const int row0 = __shfl_sync(kFull, cur.row0, from);
    const int nv = __shfl_sync(kFull, cur.nv, from);
    stage_nv = (stage_nv & ~(0xffu << (8 * st))) | (static_cast<uint32_t>(nv) << (8 * st));
    ring.issue(j, max(phys, 0), -1, row0, g, &tmap_k, &tmap_v, lane);
  };
  auto nv_of = [&](int j) { return static_cast<int>((stage_nv >> (8 * (j % NST))) & 0xffu); };

  Att at;
  at.reset();
  for (int j = 0; j < min(cnt, NST); ++j) issue(j);
  const uint16_t* q0 = a.q + (static_cast<int64_t>(s) * a.num_q_heads + g * G) * D;
  if constexpr (!FP8) {
    at.load_q(q0, G, lane);
    for (int i = 0; i < cnt; ++i) {
      if (!__all_sync(kFull, ring.wait(i, a.timeout_ns))) {
        ring.drain(i, min(cnt, i + NST), a.timeout_ns);
        if (lane == 0) flag(a.dev_status, 16u);  // PKV_DEV_ERR_TIMEOUT; the output is undefined
        break;
      }
      const uint32_t sK = ring.k_tile(i);
      const int nv = nv_of(i);
      if (nv > 0) at.tile(sK, sK + Geom::kTileBytes, nv, a.scale_log2, lane);
      __syncwarp();
      if (i + NST < cnt) issue(i + NST);
    }
    if constexpr (!BF16) at.scale_acc(1.f / Att::kWeightUp);
  } else {
    // Two tiles a step.  2^top is above every V scale seen so far; weights and
    // scales enter the product in its unit, times 2^14.  The softmax's shift m
    // follows weight times V scale in that unit (`lift`), so the products keep
    // their f16 bits although scales lie far apart.  When the unit grows by
    // 2^d, lowering m by d (times 2^d for the sum) leaves the accumulator's
    // numbers as they are.  Weights without their scales then exceed 1: lift
    // >= -kSpread and at most kSpread of lowering keep their sum below 2^97 a
    // token.  (Up to the first scale of 2^kLeast and more, zeros among the
    // smaller ones, m is lowered to lift = -kSpread at most and none of that
    // counts.)
    constexpr int kSpread = 48, kLeast = -100;
    const float up = at.template load_q<BF16, true>(q0, G, lane);
    const float up_a = __shfl_sync(kFull, up, 8 * (lane & 3)), up_b = __shfl_sync(kFull, up, 8 * (lane & 3) + 4);
    int vexp = kLeast, room = kSpread;
    float top = kLeast, unit = exp2i(Att::kWeightUpLog2 - kLeast);
    for (int i = 0; i < cnt; i += 2) {
      const bool two = i + 1 < cnt;
      const bool ok = ring.wait(i, a.timeout_ns) && (!two || ring.wait(i + 1, a.timeout_ns));
      if (!__all_sync(kFull, ok)) {
        ring.drain(i, min(cnt, i + NST), a.timeout_ns);
        if (lane == 0) flag(a.dev_status, 16u);
        break;
      }
      const bool now = (i >> 5) == chunk;  // both tiles of a pair lie in one chunk
      const float ksel = now ? ks : ks_prev, vsel = now ? vs : vs_prev, vesel = now ? ve : ve_prev;
      uint32_t sK[2];
      int nv[2];
      float sl2k[2], pv[2], lift[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j = two ? i + u : i;  // a missing second tile reuses the first one's stage, no valid token
        sl2k[u] = a.scale_log2 * __shfl_sync(kFull, ksel, j & 31);
        pv[u] = __shfl_sync(kFull, vsel, j & 31);
        lift[u] = __shfl_sync(kFull, vesel, j & 31);
        nv[u] = u == 1 && !two ? 0 : nv_of(j);
        sK[u] = ring.k_tile(j);
      }
      if (fmaxf(lift[0], lift[1]) > top && vexp < 126) {  // the same for the whole warp
        const int e = min(static_cast<int>(fmaxf(lift[0], lift[1])), 126);
        const bool begun = vexp > kLeast;
        const int d = min(e - vexp, begun ? room : kSpread - (126 + kLeast));
        at.m_a -= static_cast<float>(d);
        at.m_b -= static_cast<float>(d);
        at.l_a *= exp2i(d);
        at.l_b *= exp2i(d);
        at.scale_acc(unit_change(vexp + d, e));
        if (begun) room -= d;
        vexp = e;
        top = static_cast<float>(e);
        unit = exp2i(Att::kWeightUpLog2 - e);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        pv[u] = nv[u] > 0 ? pv[u] * unit : 0.f;
        lift[u] = fmaxf(lift[u] - top, -static_cast<float>(kSpread));
      }
      at.template tiles<2, Geom::kTileBytes, true>(sK, nv, sl2k, pv, lane, up_a, up_b, lift);
      __syncwarp();
      if (i + NST < cnt) issue(i + NST);
      if (i + 1 + NST < cnt) issue(i + 1 + NST);
    }
    // Out of the unit.  Of a very large one (2^60 and more) a part stays in m
    // and the sum: the accumulator adds up tokens before it is divided.
    const int stay = max(vexp - Att::kWeightUpLog2 - 60, 0);
    at.m_a += static_cast<float>(stay);
    at.m_b += static_cast<float>(stay);
    at.l_a *= exp2i(-stay);
    at.l_b *= exp2i(-stay);
    at.scale_acc(exp2i(vexp - Att::kWeightUpLog2 - stay));
  }
  at.finish_sums();

  // Save this warp's state: rows [8][kRow], running max [8], running sum [8].
  {
    float* st = reinterpret_cast<float*>(smem + static_cast<size_t>(warp) * NST * Geom::kStageBytes);
    const int gr = lane >> 2, tq = lane & 3;
    float* ra = st + (2 * tq) * kRow;
    float* rb = ra + kRow;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      const int d0 = FP8 ? 16 * gr + 2 * mt : 16 * mt + gr, d1 = FP8 ? d0 + 1 : d0 + 8;
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
      st[w] = reinterpret_cast<const float*>(smem + static_cast<size_t>(w) * NST * Geom::kStageBytes);
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
  const int64_t row0 = (static_cast<int64_t>(s) * a.num_q_heads + g * G) * D;
  auto store4 = [&](int e, float4 o, float l) {
    const float inv = l > 0.f ? 1.f / l : 0.f;
    store_out(a.out, row0 + e, o.x * inv, a.out_dtype);
    store_out(a.out, row0 + e + 1, o.y * inv, a.out_dtype);
    store_out(a.out, row0 + e + 2, o.z * inv, a.out_dtype);
    store_out(a.out, row0 + e + 3, o.w * inv, a.out_dtype);
  };
  if (C == 1) {
    for (int e = 4 * threadIdx.x; e < G * D; e += 4 * NW * 32) {
      float M, l;
      float4 o;
      merged(e / D, e % D, M, o, l);
      store4(e, o, l);
    }
    cluster_wait();
    return;
  }
  // CTA r merges elements [r * per, r * per + per) of the group's rows over
  // the cluster: every CTA stores its part of them, and its heads' max and
  // sum, into r's shared memory.
  const int per = G * D / C;  // a multiple of 4: D is at least 64, C at most 8
  float* inbox = reinterpret_cast<float*>(smem + kInboxAt);  // [C][per], then [C][8] max, [C][8] sum
  float* inbox_m = inbox + 8 * D;
  float* inbox_l = inbox_m + 8 * kSparseMaxCluster;
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
    for (int r = 0; r < kSparseMaxCluster; ++r)
      if (r < C) M = fmaxf(M, inbox_m[r * 8 + h]);
    const float mu = M == kNegInf ? 0.f : M;
#pragma unroll
    for (int r = 0; r < kSparseMaxCluster; ++r)
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
template <int D, bool BF16, bool FP8, int NW>
struct SparseLaunch {
  using Geom = TileGeom<D, FP8 ? 1 : 2>;
  static constexpr int NST = FP8 ? 4 : D == 64 ? 3 : 2;  // 12 to 16 KB of tiles a warp
  static constexpr auto kernel = decode_sparse_kernel<D, BF16, FP8, NW, NST>;

  static size_t smem(int C) {
    return static_cast<size_t>(NW) * NST * (Geom::kStageBytes + 8) +
           (C > 1 ? (8 * D + 16 * kSparseMaxCluster) * sizeof(float) : 0);
  }

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
    cfg.dynamicSmemBytes = smem(C);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem(kSparseMaxCluster)) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      return 1;
    }
    slot.store(n, std::memory_order_release);
    return n;
  }

  static cudaError_t launch(const DecodeArgs& a, const SparseArgs& sp, int C, const CUtensorMap& tk,
                            const CUtensorMap& tv, cudaStream_t stream) {
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem(kSparseMaxCluster));
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(a.num_seqs) * a.num_kv_heads * C), dim3(NW * 32),
                              smem(C), C, stream, a, sp, tk, tv);
  }
};

// Microseconds that `units` lists of up to `tiles` tiles take with NW warps a
// CTA and C CTAs a list, `held` clusters at a time.  A wave of clusters starts
// (length -> list -> table -> tile; the cluster's meeting), then a warp takes
// kTileUs a tile, or longer where its SM's rate is what it waits for.  All
// waves together are no faster than the memory; the last one, and some of each
// one's start, stay exposed, the less the more CTAs a SM holds.  A quarter of
// a wave is added in any case: a longer chain next to a full memory.  SMs fill
// up with clusters one after another, with single CTAs evenly.
// The constants are fitted to 458 measured shapes (2 to 2000 lists of 2 to 512
// tiles, the three kinds of pool, each NW and C): the form with the lowest cost
// is 1% slower than the best one in the mean, 16% at the most.  (Eight warps up
// to the number of SMs and four or two above it: 11% and 130%.)  Microseconds:
//   8 of 128 tiles: 5.4 with 8 warps in clusters of 8, 6.6 of 4, 9.4 of 2;
//   16 of 128: 6.8 with 8 warps of 4 -- clusters of 8 no longer fit at once: 9.9;
//   38 of 128: 10.8 with 4 warps of 8 -- 15.7 with 8 of 4, 11.8 with 8 of 2;
//   64 of 128 (FP8): 11.8 with 8 warps of 2, 12.6 with 4 of 4;
//   100 of 512 (FP8): 37.7 with 4 warps of 4, 51 with 8 alone;
//   160 of 512 (FP8): 64 with 4 warps of 2, 87 with 4 alone, 142 with 2;
//   912 of 5: 10.3 with 2 warps alone, 12.9 with 4; 2000 of 64: 153 with 4, 157
//   with 2, 171 with 8, 180 with 1.
template <int D, bool FP8>
float sparse_cost(int64_t units, int64_t tiles, int group, int NW, int C, int held, int64_t sms) {
  constexpr float kStartUs = 3.5f, kTileUs = FP8 ? 0.8f : D == 64 ? 0.6f : 0.9f;
  constexpr float kSmBytes = FP8 ? 45e3f : D == 64 ? 60e3f : 75e3f, kBytes = 6.4e6f;  // a microsecond
  constexpr float kTileBytes = TileGeom<D, FP8 ? 1 : 2>::kStageBytes;
  const int64_t full = (static_cast<int64_t>(held) * C + sms - 1) / sms;  // CTAs a SM holds
  const int64_t per_sm = C == 1 ? std::min((units + sms - 1) / sms, full) : units * C <= sms ? 1 : full;
  int64_t n = (tiles + NW * C - 1) / (NW * C);  // tiles of a warp
  if (FP8) n += n & 1;                          // taken in pairs
  const float tile = std::max(kTileUs, static_cast<float>(per_sm * NW) * (kTileBytes / kSmBytes));
  const float meet = 0.4f + 0.1f * static_cast<float>(group);  // rows of `group` heads to send
  const float start = kStartUs + (C > 1 ? meet : 0.f), wave = start + tile * static_cast<float>(n);
  const float waves = static_cast<float>(units) / static_cast<float>(held);
  const float exposed = units > held ? wave * (0.5f + 0.15f * (waves - 1.f)) / static_cast<float>(full) : 0.f;
  const float bytes = static_cast<float>(units) * static_cast<float>(tiles) * kTileBytes;
  return std::max(static_cast<float>((units + held - 1) / held) * wave, start + bytes / kBytes + exposed) +
         0.25f * wave;
}

template <int D, bool BF16, bool FP8>
cudaError_t launch_sparse_t(const DecodeArgs& a, const SparseArgs& sp, const CUtensorMap& tk, const CUtensorMap& tv,
                            cudaStream_t stream) {
  using One = SparseLaunch<D, BF16, FP8, 1>;
  using Two = SparseLaunch<D, BF16, FP8, 2>;
  using Four = SparseLaunch<D, BF16, FP8, 4>;
  using Eight = SparseLaunch<D, BF16, FP8, 8>;
  const int64_t units = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads, sms = current_sm_count(152);
  const int64_t tiles = std::max<int64_t>(1, std::min((static_cast<int64_t>(a.max_context_len) + kTile - 1) / kTile,
                                                      static_cast<int64_t>(sp.keep) << (a.block_shift - 4)));
  int best_nw = 8, best_c = 1;
  float best = 0.f;
  auto consider = [&](int NW, int C, int held) {
    const float cost = sparse_cost<D, FP8>(units, tiles, a.group, NW, C, held, sms);
    if (best > 0.f && cost >= best) return;
    best = cost;
    best_nw = NW;
    best_c = C;
  };
  consider(4, 1, Four::resident(1));
  consider(8, 1, Eight::resident(1));
  if (units > sms) {
    consider(2, 1, Two::resident(1));
    consider(1, 1, One::resident(1));
  }
  for (int C = 2; C <= kSparseMaxCluster && units * C <= 4 * sms; C *= 2) {
    consider(8, C, Eight::resident(C));
    consider(4, C, Four::resident(C));
  }
  switch (best_nw) {
    case 1: return One::launch(a, sp, 1, tk, tv, stream);
    case 2: return Two::launch(a, sp, 1, tk, tv, stream);
    case 4: return Four::launch(a, sp, best_c, tk, tv, stream);
    default: return Eight::launch(a, sp, best_c, tk, tv, stream);
  }
}

}  // namespace

cudaError_t launch_decode_sparse(const DecodeArgs& a, const SparseArgs& sp, const CUtensorMap& tmap_k,
                                 const CUtensorMap& tmap_v, int head_dim, bool bf16, bool fp8, cudaStream_t stream) {
  if (a.num_seqs == 0) return cudaSuccess;
  if (fp8) {
    if (head_dim != 128) return cudaErrorInvalidValue;
    return bf16 ? launch_sparse_t<128, true, true>(a, sp, tmap_k, tmap_v, stream)
                : launch_sparse_t<128, false, true>(a, sp, tmap_k, tmap_v, stream);
  }
  if (head_dim == 128)
    return bf16 ? launch_sparse_t<128, true, false>(a, sp, tmap_k, tmap_v, stream)
                : launch_sparse_t<128, false, false>(a, sp, tmap_k, tmap_v, stream);
  if (head_dim == 64)
    return bf16 ? launch_sparse_t<64, true, false>(a, sp, tmap_k, tmap_v, stream)
                : launch_sparse_t<64, false, false>(a, sp, tmap_k, tmap_v, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkv

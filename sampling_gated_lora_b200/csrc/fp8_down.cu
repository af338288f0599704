// What the 8-bit linear needs of its activations, in one pass over them:
//
//   xq, sx  x [M,K] in 1 x 128 blocks, codes row-major, scales K-block major
//           (the quantiser of fp8_quantize.cu, the same arithmetic)
//   t       scale * gate(m) * (x A^T) [M,r] in bf16: the gated adapter's
//           down-projection (hyper.ai, section "方法"), from x itself
//
// x arrives by TMA; a tensor-core pass takes a tile of BT tokens as one operand
// of x A^T (tokens on the 128-row side, adapter rows on the other, fp32 in TMEM)
// while eight warps read the same tile from shared memory, find each row's
// maximum over the block and write its codes. K is split over a thread-block
// cluster; the CTAs' T meet through distributed shared memory in rank order.
// With few tokens A is most of what is read, and chunks of 32 adapter rows go
// to clusters of their own (the first of them quantises).
// HBM bounds it for many rows (3 bytes an element; two separate passes over x
// measured 43 + 25 us at 4352 x 12288), latency for few.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "per_device.h"

#include "fp8.cuh"

namespace uno {

namespace {

constexpr int kThreads = 320;         // producer, MMA issuer, eight quantising warps
constexpr int kLanes = 128;           // MMA M: token rows, whatever part of them a tile has
constexpr int kPartPad = 4;

struct DownMaps {
  CUtensorMap x, a;
};
struct DownParams {
  int M, K, r, nkb, kb_per_split, splits;
  int ld_sx;
  float scale;
  const uint8_t* gate;
  uint8_t* xq;
  float* sx;
  __nv_bfloat16* t;
};

// A CTA's tile: BT tokens, NA boxes of RC adapter rows.
template <int BT, int RC, int NA>
struct Down {
  static constexpr int kCols = NA * RC;                    // adapter rows: TMEM columns
  static constexpr uint32_t kX = BT * 256, kA = RC * 256;  // 128 k of bf16: two 64-wide boxes
  static constexpr uint32_t kStage = kX + NA * kA;
  // an MMA reads 128 token rows from either box of x: past a smaller tile's, and
  // past the ring's end with the last stage's
  static constexpr int kSlack = BT < kLanes ? kLanes * 128 : 0;
  static constexpr int kFit = (192 * 1024 - kSlack) / static_cast<int>(kStage);
  static constexpr int kStages = kFit < 12 ? kFit : 12;
  static_assert(BT * (kCols + kPartPad) * 4 <= kStages * static_cast<int>(kStage), "T must fit the ring");
};

template <int BT, int RC, int NA>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_down_kernel(const __grid_constant__ DownMaps tm, const DownParams p) {
  using C = Down<BT, RC, NA>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~static_cast<uintptr_t>(1023u));
  __shared__ uint64_t full[S], empty[S], accum;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tok0 = blockIdx.x * BT, j0 = blockIdx.y * C::kCols;
  const bool quantises = blockIdx.y == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), quantises ? 9 : 1);   // the MMAs' commit, eight warps
    }
    mbar_init(smem_u32(&accum), 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_slot), C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int kb0 = blockIdx.z * p.kb_per_split, kb1 = min(p.nkb, kb0 + p.kb_per_split);
  auto fail = [&]() {
    abort_flag = 1;
    raise_status(nullptr, kDevTimeout);
  };

  // A may have been written by the launch before (the input gradient's
  // transposes), so nothing is fetched earlier. The product may start its
  // prologue from here on: its constants are complete when this wait returns.
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ TMA producer
    int s = 0;
    uint32_t ph = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1u) || abort_flag) {
        fail();
        break;
      }
      const uint32_t sa = smem_u32(smem + s * C::kStage), fb = smem_u32(&full[s]);
      mbar_arrive_expect_tx(fb, C::kStage);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        tma_load_2d(sa + h * (C::kX / 2), &tm.x, kb * 128 + 64 * h, tok0, fb);
#pragma unroll
        for (int n = 0; n < NA; ++n)
          tma_load_2d(sa + C::kX + n * C::kA + h * (C::kA / 2), &tm.a, kb * 128 + 64 * h, j0 + n * RC, fb);
      }
      if (++s == S) {
        s = 0;
        ph ^= 1u;
      }
    }
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = idesc_f32acc(kLanes, RC, false);
    int s = 0;
    uint32_t ph = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(smem_u32(&full[s]), ph)) {
        fail();
        break;
      }
      tc_fence_after();
      const uint32_t sa = smem_u32(smem + s * C::kStage);
#pragma unroll
      for (int n = 0; n < NA; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t xd = sdesc_k_sw128(sa + h * (C::kX / 2));
          const uint64_t ad = sdesc_k_sw128(sa + C::kX + n * C::kA + h * (C::kA / 2));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss<false>(tmem + static_cast<uint32_t>(n * RC), xd + 2 * kk, ad + 2 * kk, idesc,
                          (kb > kb0 || h > 0 || kk > 0) ? 1u : 0u);
        }
      mma_commit(smem_u32(&empty[s]));
      if (++s == S) {
        s = 0;
        ph ^= 1u;
      }
    }
    mma_commit(smem_u32(&accum));
  } else if (warp >= 2) {
    // ------------------------------------------------------------ quantisation
    // kPer threads share a row of the tile, each with kCh 8-element chunks of
    // the row's 16; the two halves of a row (boxes) are read in opposite chunk
    // order, so a quarter warp of the 128-token tile touches all banks once
    constexpr int kPer = 256 / BT, kCh = 16 / kPer;
    const int tid = threadIdx.x - 64, row = tid / kPer, part = tid % kPer;
    const int m = tok0 + row;
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int kb = kb0; quantises && kb < kb1; ++kb) {
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[s]), ph));
      if (!ok) break;
      const uint8_t* xs = smem + s * C::kStage;
      uint4 w[kCh];
#pragma unroll
      for (int i = 0; i < kCh; ++i) {
        const int c = part * kCh + (kCh == 8 ? i ^ (4 * part) : i);   // of the row's 16 chunks
        w[i] = *reinterpret_cast<const uint4*>(xs + (c >> 3) * (C::kX / 2) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
      }
      uint32_t top[4] = {};   // pairs of magnitudes
#pragma unroll
      for (int i = 0; i < kCh; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e] = max_nan_bf16x2(top[e], abs_bf16x2(u[e]));
      }
      top[0] = max_nan_bf16x2(max_nan_bf16x2(top[0], top[1]), max_nan_bf16x2(top[2], top[3]));
      float a = max_nan(max_nan(kAmaxFloor, bf16_lo(top[0])), bf16_hi(top[0]));
      // the tile has been read
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[s]));
      if (++s == S) {
        s = 0;
        ph ^= 1u;
      }
#pragma unroll
      for (int o = kPer / 2; o; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
      if (part == 0 && m < p.ld_sx) p.sx[static_cast<size_t>(kb) * p.ld_sx + m] = __fdiv_rn(a, kE4m3Max);
      if (m >= p.M) continue;
      const float inv = __fdiv_rn(kE4m3Max, a);
      uint2 q[kCh];
#pragma unroll
      for (int i = 0; i < kCh; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[2 * e] = bf16_lo(u[e]) * inv;
          f[2 * e + 1] = bf16_hi(u[e]) * inv;
        }
        q[i] = e4m3x8(f);
      }
      uint8_t* dst = p.xq + static_cast<size_t>(m) * p.K + kb * 128;
      if (kCh == 1) {
        if (kb * 128 + part * 8 < p.K) *reinterpret_cast<uint2*>(dst + part * 8) = q[0];
      } else {
#pragma unroll
        for (int i = 0; i < kCh; i += 2) {   // chunks i and i + 1 are neighbours in either order
          const int c = part * kCh + (kCh == 8 ? i ^ (4 * part) : i);
          if (kb * 128 + c * 8 < p.K)
            *reinterpret_cast<uint4*>(dst + c * 8) = make_uint4(q[i].x, q[i].y, q[i + 1 < kCh ? i + 1 : i].x, q[i + 1 < kCh ? i + 1 : i].y);
        }
      }
    }
    // T -> shared memory, [token][adapter row]: the ring is free once the MMAs are done
    ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&accum), 0));
    if (!ok && lane == 0) fail();
    tc_fence_after();
    named_sync(1, 256);   // every warp has read its last tile
    const int quarter = warp & 3, half = (warp - 2) >> 2, token = quarter * 32 + lane;
    if (ok && quarter * 32 < BT) {
      float* stage = reinterpret_cast<float*>(smem) + token * (C::kCols + kPartPad);
      for (int c = half * 16; c < C::kCols; c += 32) {
        float v[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(c), v);
        if (token < BT) {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(stage + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
    }
  }

  if (p.splits > 1) cluster_sync_converged();
  else cta_sync_converged();
  if (!abort_flag) {
    constexpr int kQuads = C::kCols / 4, kGroups = BT * kQuads;
    const int Sp = p.splits;
    const int chunk = (kGroups + Sp - 1) / Sp;
    const int e0 = static_cast<int>(cluster_ctarank()) * chunk, e1 = min(kGroups, e0 + chunk);
    const uint32_t part0 = smem_u32(smem);
    uint32_t peer[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) peer[r] = map_shared_rank(part0, r < Sp ? r : 0);
    for (int e = e0 + static_cast<int>(threadIdx.x); e < e1; e += kThreads) {
      const int token = e / kQuads, j4 = e % kQuads * 4;
      const int m = tok0 + token, j = j0 + j4;
      if (m >= p.M || j >= p.r) continue;
      const uint32_t off = static_cast<uint32_t>((token * (C::kCols + kPartPad) + j4) * 4);
      float4 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < Sp) v[r] = ld_cluster_f32x4(peer[r] + off);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < Sp) {
          a.x += v[r].x; a.y += v[r].y; a.z += v[r].z; a.w += v[r].w;
        }
      const float f = p.scale * static_cast<float>(p.gate[m]);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(f * a.x, f * a.y), hi = __floats2bfloat162_rn(f * a.z, f * a.w);
      *reinterpret_cast<uint2*>(p.t + static_cast<size_t>(m) * p.r + j) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
  }
  if (p.splits > 1) cluster_sync_converged();   // the peers have read this CTA's T
  tc_fence_before();
  cta_sync_converged();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// Clusters of `size` CTAs (along z) of a kernel that `device` (the current one) holds at once.
template <int BT, int RC, int NA>
int resident_clusters(int device, int size) {
  static PerDevice<9> kept;
  using C = Down<BT, RC, NA>;
  return kept.get(device, size, [&] {
    return resident_clusters_of(reinterpret_cast<const void*>(&fp8_down_kernel<BT, RC, NA>), kThreads,
                                static_cast<int>(C::kStages * C::kStage + C::kSlack + 1024), size);
  });
}

template <int BT, int RC, int NA>
uno_status down_launch(const Fp8Down& d, DownParams p, cudaStream_t s) {
  using C = Down<BT, RC, NA>;
  DownMaps tm;
  uno_status st;
  if ((st = make_map(&tm.x, UNO_BF16, d.x, d.K, d.M, d.K, BT)) != UNO_OK) return st;
  if ((st = make_map(&tm.a, UNO_BF16, d.A, d.K, d.r, d.K, RC)) != UNO_OK) return st;
  const int tiles = (p.M + BT - 1) / BT, chunks = (p.r + C::kCols - 1) / C::kCols;
  // as many K-splits as one wave of clusters takes (34 token tiles in four
  // splits fit the SMs but not the clusters' places: 64 us where three take 39)
  int splits = std::min(8, p.nkb);
  const int device = current_device();
  while (splits > 1 && static_cast<int64_t>(tiles) * chunks > resident_clusters<BT, RC, NA>(device, splits)) --splits;
  p.kb_per_split = (p.nkb + splits - 1) / splits;
  p.splits = splits = (p.nkb + p.kb_per_split - 1) / p.kb_per_split;
  const int smem = static_cast<int>(C::kStages * C::kStage + C::kSlack + 1024);
  auto fn = &fp8_down_kernel<BT, RC, NA>;
  static SmemGranted granted;
  cudaError_t e = granted.ask(reinterpret_cast<const void*>(fn), smem);
  if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute(8-bit down-projection smem)");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(tiles, chunks, splits);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = launch_attrs(attr, 1, 1, static_cast<unsigned>(splits));
  cfg.attrs = attr;
  e = cudaLaunchKernelEx(&cfg, fn, tm, p);
  return e == cudaSuccess ? UNO_OK : cuda_error(e, "8-bit down-projection launch");
}

}  // namespace

uno_status fp8_down_launch(const Fp8Down& d, cudaStream_t s) {
  DownParams p{};
  p.M = static_cast<int>(d.M);
  p.K = static_cast<int>(d.K);
  p.r = d.r;
  p.nkb = static_cast<int>((d.K + 127) / 128);
  p.ld_sx = static_cast<int>(d.ld_sx);
  p.scale = d.scale;
  p.gate = d.gate;
  p.xq = d.xq;
  p.sx = d.sx;
  p.t = static_cast<__nv_bfloat16*>(d.t);
  if (d.M <= 16) return down_launch<16, 32, 1>(d, p, s);
  if (d.M <= 32) return down_launch<32, 32, 1>(d, p, s);
  if (d.M <= 64) return down_launch<64, 32, 1>(d, p, s);
  // chunks of 32 adapter rows while they and eight K-splits fit the device
  const int64_t tiles = (d.M + 127) / 128;
  if (tiles * ((d.r + 31) / 32) * 8 <= device_sm_count()) return down_launch<128, 32, 1>(d, p, s);
  return d.r <= 128 ? down_launch<128, 128, 1>(d, p, s) : down_launch<128, 128, 2>(d, p, s);
}

}  // namespace uno

// Gated-LoRA linear on e4m3 operands with block scales (sm_100a).
//
//   y[m,n] = sum_b sx[m,b] sw[n/128,b] sum_{k in block b} xq[m,k] wq[n,k]
//          + sum_j t[m,j] Bl[n,j],       blocks b of 128 consecutive k
//
// xq, sx: the activations in 1 x 128 blocks (fp8_quantize_launch); wq, sw: the
// weight in 128 x 128 blocks; t = scale * gate * (x A^T) in bf16 (the gated
// adapter of hyper.ai, section "方法", fed by the unquantised x).
//
// The scales are arbitrary floats and change every 128 k, so the tensor core
// sums one 128-deep block at a time (exact e4m3 products, fp32 sums) and the
// epilogue warps add factor * block sum into fp32 registers while the tensor
// core works on the next block in another TMEM buffer. A 128-byte K-block is
// 128 e4m3 or 64 bf16 values, so the adapter's K-blocks of [t | Bl] pass
// through the same stages with kind::f16 MMAs and factor 1.
#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"

#include "fp8.cuh"

namespace uno {

namespace {

constexpr int kThreads = 192;
constexpr int kRows = 128;                           // features per tile (MMA M)
constexpr uint32_t kWBytes = kRows * 128;            // one 128-row, 128-byte K-block tile
constexpr int kPartPad = 4;

struct Fp8Maps {
  CUtensorMap x, w, t, b;
};

struct Fp8Params {
  int M, N, nkb, nkr;        // K-blocks of xq wq^T and of t Bl^T
  int kb_per_split, splits;
  int stages;
  int ld_sx, ld_sw;          // sx [nkb, ld_sx], sw [ceil(N/128), ld_sw]
  const float* sx;
  const float* sw;
  __nv_bfloat16* y;
};

// ---------------------------------------------------------------- few tokens
// Weights on the 128-row MMA side, BN tokens on the N side: a lane of TMEM is
// a feature and a column a token. K is split over a thread-block cluster so
// that every SM streams a share of W (HBM bandwidth bounds these sizes); the
// CTAs' fp32 sums meet through distributed shared memory, in rank order.
template <int BN>
struct Narrow {
  static constexpr uint32_t kStage = kWBytes + BN * 128;
  static constexpr int kStride = BN < 32 ? 32 : BN;      // TMEM columns of a buffer
  static constexpr int kBufs = BN <= 64 ? 8 : 4;
  static constexpr int kCols = kStride * kBufs;
};

template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_narrow_kernel(const __grid_constant__ Fp8Maps tm, const Fp8Params p) {
  using C = Narrow<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~static_cast<uintptr_t>(1023u));
  __shared__ float fac[4][2][BN];                        // per epilogue warp: factors of one K-block
  __shared__ uint64_t accf[C::kBufs], acce[C::kBufs];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  const int S = p.stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * C::kStage);
  uint64_t* empty = full + S;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tok0 = blockIdx.x * BN, feat0 = blockIdx.y * kRows;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(smem_u32(&accf[b]), 1);
      mbar_init(smem_u32(&acce[b]), 4);
    }
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
  if (threadIdx.x == 0) pdl_trigger();

  const int kb0 = blockIdx.z * p.kb_per_split;
  const int kb1 = min(p.nkb + p.nkr, kb0 + p.kb_per_split);
  auto fail = [&]() {
    abort_flag = 1;
    raise_status(nullptr, kDevTimeout);
  };

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ TMA producer
    auto load_w = [&](int kb, uint32_t st, uint32_t fb) {
      if (kb < p.nkb) tma_load_2d(st, &tm.w, kb * 128, feat0, fb);
      else tma_load_2d(st, &tm.b, (kb - p.nkb) * 64, feat0, fb);
    };
    auto load_x = [&](int kb, uint32_t st, uint32_t fb) {
      if (kb < p.nkb) tma_load_2d(st + kWBytes, &tm.x, kb * 128, tok0, fb);
      else tma_load_2d(st + kWBytes, &tm.t, (kb - p.nkb) * 64, tok0, fb);
    };
    // weights (constant) of the first stages before waiting for the writer of xq and t
    const int pre = min(S, kb1 - kb0);
    for (int q = 0; q < pre; ++q) {
      mbar_arrive_expect_tx(smem_u32(&full[q]), C::kStage);
      load_w(kb0 + q, smem_u32(smem + q * C::kStage), smem_u32(&full[q]));
    }
    pdl_wait();
    for (int q = 0; q < pre; ++q)
      load_x(kb0 + q, smem_u32(smem + q * C::kStage), smem_u32(&full[q]));
    int it = pre;
    for (int kb = kb0 + pre; kb < kb1; ++kb, ++it) {
      const int s = it % S;
      if (!mbar_wait(smem_u32(&empty[s]), ((it / S) & 1u) ^ 1u) || abort_flag) {
        fail();
        break;
      }
      const uint32_t st = smem_u32(smem + s * C::kStage), fb = smem_u32(&full[s]);
      mbar_arrive_expect_tx(fb, C::kStage);
      load_w(kb, st, fb);
      load_x(kb, st, fb);
    }
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t id8 = idesc_e4m3(kRows, BN), id16 = idesc_f32acc(kRows, BN, false);
    int it = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
      const int s = it % S, b = it % C::kBufs;
      if (!mbar_wait(smem_u32(&acce[b]), ((it / C::kBufs) & 1u) ^ 1u) ||
          !mbar_wait(smem_u32(&full[s]), (it / S) & 1u)) {
        fail();
        break;
      }
      tc_fence_after();
      const uint32_t st = smem_u32(smem + s * C::kStage);
      const uint64_t wd = sdesc_k_sw128(st), xd = sdesc_k_sw128(st + kWBytes);
      const uint32_t d = tmem + static_cast<uint32_t>(b * C::kStride);
      if (kb < p.nkb) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_f8(d, wd + 2 * kk, xd + 2 * kk, id8, kk > 0 ? 1u : 0u);
      } else {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss<false>(d, wd + 2 * kk, xd + 2 * kk, id16, kk > 0 ? 1u : 0u);
      }
      mma_commit(smem_u32(&empty[s]));
      mma_commit(smem_u32(&accf[b]));
    }
  } else if (warp >= 2) {
    // ------------------------------------------------------------ block sums -> registers
    const int quarter = warp & 3;
    const uint32_t trow = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float(*fw)[BN] = fac[quarter];
    const float* sw = p.sw + static_cast<size_t>(blockIdx.y) * p.ld_sw;
    constexpr int kPer = (BN + 31) / 32;
    auto factor = [&](int kb, float (&f)[kPer]) {   // this lane's tokens' factors of K-block kb
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int j = lane + 32 * i;
        f[i] = 1.f;
        if (kb < p.nkb && j < BN)
          f[i] = p.sx[static_cast<size_t>(kb) * p.ld_sx + tok0 + j] * sw[kb];
      }
    };
    float acc[BN];
#pragma unroll
    for (int j = 0; j < BN; ++j) acc[j] = 0.f;
    pdl_wait();
    float f[kPer];
    factor(kb0, f);
    int it = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
      const int b = it % C::kBufs;
      float* fs = fw[it & 1];
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (lane + 32 * i < BN) fs[lane + 32 * i] = f[i];
      if (kb + 1 < kb1) factor(kb + 1, f);
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&accf[b]), (it / C::kBufs) & 1u));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < BN; c += 16) {
        float v[16];
        tmem_ld16(trow + static_cast<uint32_t>(b * C::kStride + c), v);
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[c + j] = fmaf(fs[c + j], v[j], acc[c + j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acce[b]));
    }
    if (!ok && lane == 0) fail();
    // every MMA has finished, so the stage ring is free: stage the sums [token][feature]
    float* stage = reinterpret_cast<float*>(smem);
    if (ok) {
#pragma unroll
      for (int j = 0; j < BN; ++j) stage[j * (kRows + kPartPad) + quarter * 32 + lane] = acc[j];
    }
  }

  if (p.splits > 1) cluster_sync_converged();
  else cta_sync_converged();
  if (!abort_flag) {
    // the CTAs of the cluster share the tile's outputs out, 4 features at a time
    constexpr int kGroups = BN * (kRows / 4);
    const int Sp = p.splits;
    const int chunk = (kGroups + Sp - 1) / Sp;
    const int e0 = static_cast<int>(cluster_ctarank()) * chunk, e1 = min(kGroups, e0 + chunk);
    const uint32_t part0 = smem_u32(smem);
    uint32_t peer[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) peer[r] = map_shared_rank(part0, r < Sp ? r : 0);
    for (int e = e0 + static_cast<int>(threadIdx.x); e < e1; e += kThreads) {
      const int j = e / (kRows / 4), i4 = e % (kRows / 4);
      const int m = tok0 + j, n = feat0 + 4 * i4;
      if (m >= p.M || n >= p.N) continue;
      const uint32_t off = static_cast<uint32_t>((j * (kRows + kPartPad) + 4 * i4) * 4);
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
      const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(a.z, a.w);
      *reinterpret_cast<uint2*>(p.y + static_cast<size_t>(m) * p.N + n) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
  }
  if (p.splits > 1) cluster_sync_converged();   // the peers have read this CTA's sums

  tc_fence_before();
  cta_sync_converged();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int BN>
uno_status narrow_launch(const Fp8Maps& tm, Fp8Params p, cudaStream_t s) {
  using C = Narrow<BN>;
  const int tok_tiles = (p.M + BN - 1) / BN, feat_tiles = (p.N + kRows - 1) / kRows;
  if (feat_tiles > 65535) return set_error(UNO_ERR_UNSUPPORTED, "N too large for the tile grid");
  p.stages = std::min(8, static_cast<int>(200u * 1024u / C::kStage));
  const int smem = static_cast<int>(p.stages * (C::kStage + 16) + 1024);
  const int nkb = p.nkb + p.nkr;
  int splits = std::max(1, std::min({8, device_sm_count() / std::max(1, tok_tiles * feat_tiles), nkb}));
  p.kb_per_split = (nkb + splits - 1) / splits;
  p.splits = splits = (nkb + p.kb_per_split - 1) / p.kb_per_split;
  auto fn = &fp8_narrow_kernel<BN>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute(8-bit GEMM smem)");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(tok_tiles, feat_tiles, splits);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = launch_attrs(attr, 1, 1, static_cast<unsigned>(splits));
  cfg.attrs = attr;
  e = cudaLaunchKernelEx(&cfg, fn, tm, p);
  return e == cudaSuccess ? UNO_OK : cuda_error(e, "8-bit GEMM launch");
}

}  // namespace

uno_status fp8_gemm_launch(const Fp8Gemm& g, cudaStream_t s) {
  Fp8Params p{};
  p.M = static_cast<int>(g.M);
  p.N = static_cast<int>(g.N);
  p.nkb = static_cast<int>((g.K + 127) / 128);
  p.nkr = (g.r + 63) / 64;
  p.ld_sx = static_cast<int>(g.ld_sx);
  p.ld_sw = p.nkb;
  p.sx = g.sx;
  p.sw = g.sw;
  p.y = static_cast<__nv_bfloat16*>(g.y);
  const int bn = g.M <= 16 ? 16 : g.M <= 32 ? 32 : g.M <= 64 ? 64 : 128;
  Fp8Maps tm;
  uno_status st;
  if ((st = make_map_u8(&tm.x, g.xq, g.K, g.M, g.K, bn)) != UNO_OK) return st;
  if ((st = make_map_u8(&tm.w, g.wq, g.K, g.N, g.K, kRows)) != UNO_OK) return st;
  tm.t = tm.x;
  tm.b = tm.w;
  if (g.r > 0) {
    if ((st = make_map(&tm.t, UNO_BF16, g.t, g.r, g.M, g.r, bn)) != UNO_OK) return st;
    if ((st = make_map(&tm.b, UNO_BF16, g.Bl, g.r, g.N, g.r, kRows)) != UNO_OK) return st;
  }
  switch (bn) {
    case 16: return narrow_launch<16>(tm, p, s);
    case 32: return narrow_launch<32>(tm, p, s);
    case 64: return narrow_launch<64>(tm, p, s);
    default: return narrow_launch<128>(tm, p, s);
  }
}

}  // namespace uno

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

constexpr int kRows = 128;                           // features per tile (MMA M)
constexpr uint32_t kWBytes = kRows * 128;            // one 128-row, 128-byte K-block tile
constexpr int kPartPad = 4;

struct Fp8Maps {
  CUtensorMap x, w, t, b;
};

struct Fp8Params {
  int M, N, nkb, nkr;        // K-blocks of xq wq^T and of t Bl^T
  int kb_per_split, splits;
  int ld_sx, ld_sw;          // sx [nkb, ld_sx], sw [ceil(N/128), ld_sw]
  const float* sx;
  const float* sw;
  __nv_bfloat16* y;
  int32_t* status;           // library-wide device status word
};

// This file is compiled without relocatable device code (setmaxnreg needs it),
// so the status word comes as a pointer.
__device__ __forceinline__ void raise_timeout(int32_t* status) { atomicOr(status, kDevTimeout); }

// Position in a ring of N slots and the parity of the current pass over it
// (a running counter: one thread issues every copy and every MMA, and a
// division by the ring's size a K-block would be on its critical path).
struct Ring {
  int i = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      ph ^= 1u;
    }
  }
};

// acc[i] += f * v[i] and acc[i+1] += g * v[i+1], one packed instruction (the
// epilogue's adds are on the path that frees a TMEM buffer: 380 -> 355 us at
// 4352 x 12288 -> 4096 against scalar adds).
__device__ __forceinline__ void fma2(float& a0, float& a1, uint32_t v0, uint32_t v1, uint64_t fg) {
  uint64_t a, v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(v0), "r"(v1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(v), "l"(fg));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}

// ---------------------------------------------------------------- few tokens
// Weights on the 128-row MMA side, BN tokens on the N side: a lane of TMEM is
// a feature and a column a token (all of them: M <= BN). HBM bandwidth bounds
// these sizes, so W is read once. With fewer tiles than SMs, K is split over a thread-block cluster
// so that every SM streams a share, and the CTAs' fp32 sums meet through
// distributed shared memory in rank order; otherwise each CTA walks whole
// tiles, and the stores of one overlap the loads and products of the next.
// Up to 64 tokens four epilogue warps hold the sums, from 128 on eight (halves
// of the columns); the factors of a column's token are staged per warp in
// shared memory and read as broadcasts.
template <int BN>
struct Narrow {
  static constexpr uint32_t kStage = kWBytes + BN * 128;
  static constexpr int kStride = BN < 32 ? 32 : BN;      // TMEM columns of a buffer
  static constexpr int kBufs = BN <= 64 ? 8 : 512 / BN;
  static constexpr int kCols = BN <= 32 ? 256 : 512;
  static constexpr int kEpi = BN <= 64 ? 4 : 8;          // epilogue warps
  static constexpr int kFirst = 4;                       // the first of them
  // K-blocks an epilogue warp takes at a time: at few columns the latencies of
  // a block (barrier, factors, TMEM read) outweigh its adds and would exceed
  // the 0.36 us in which HBM brings an SM the next 16 KB of W
  static constexpr int kBatch = BN <= 16 ? 4 : BN <= 64 ? 2 : 1;
  static constexpr int kStages = 194 * 1024 / static_cast<int>(kStage) < 12 ? 194 * 1024 / static_cast<int>(kStage) : 12;
  // Scales of a K-block's tokens: copied along with its operands into a ring of
  // their own. The copies run at most kStages blocks ahead of the MMAs and the
  // epilogue at most kBufs behind them, so a slot is free when it comes up.
  static constexpr int kSlots = kStages + kBufs;
  static_assert(kBufs <= kStages, "the epilogue has to see every phase of a stage's barrier");
  static constexpr int kCW = BN * 4 / kEpi;              // columns of an epilogue warp
  static constexpr int kThreads = 32 * (kFirst + kEpi);
  static constexpr bool kMoveRegs = BN > 160;            // see kPairThreads
};

template <int BN>
__global__ void __launch_bounds__(Narrow<BN>::kThreads, 1)
    fp8_narrow_kernel(const __grid_constant__ Fp8Maps tm, const Fp8Params p) {
  using C = Narrow<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~static_cast<uintptr_t>(1023u));
  __shared__ alignas(16) float fac[C::kEpi][2][C::kBatch][C::kCW];  // per epilogue warp: factors of a batch
  __shared__ alignas(16) float scl[C::kSlots][BN];
  __shared__ uint64_t sfull[C::kSlots];
  __shared__ uint64_t acce[C::kBufs];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  constexpr int S = C::kStages;
  // full: a stage has been filled; done: the MMAs on it have completed (frees the
  // stage to the producer and shows the block's sum to the epilogue, which is
  // never more than kBufs <= S blocks behind, so it sees every phase); acce: a
  // TMEM buffer has been read
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * C::kStage);
  uint64_t* done = full + S;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = (p.N + kRows - 1) / kRows;   // one token tile: M <= BN

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 2);   // W's producer and x's
      mbar_init(smem_u32(&done[s]), 1);
    }
    for (int b = 0; b < C::kBufs; ++b) mbar_init(smem_u32(&acce[b]), C::kEpi);
    for (int b = 0; b < C::kSlots; ++b) mbar_init(smem_u32(&sfull[b]), 1);
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

  const int nkb = p.nkb + p.nkr;
  const int kb0 = blockIdx.z * p.kb_per_split;
  const int kb1 = min(nkb, kb0 + p.kb_per_split);
  const int step = gridDim.x;   // splits > 1: one tile per cluster
  auto fail = [&]() {
    abort_flag = 1;
    raise_timeout(p.status);
  };

  if (warp < C::kFirst) {
    if (C::kMoveRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- TMA producer of W (and Bl)
      // constant, so the first stages do not wait for the writer of xq and t
      Ring st;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += step)
        for (int kb = kb0; kb < kb1; ++kb, st.next(S)) {
          if (!mbar_wait(smem_u32(&done[st.i]), st.ph ^ 1u) || abort_flag) {
            fail();
            ok = false;
            break;
          }
          const uint32_t sa = smem_u32(smem + st.i * C::kStage), fb = smem_u32(&full[st.i]);
          mbar_arrive_expect_tx(fb, kWBytes);
          if (kb < p.nkb) tma_load_2d(sa, &tm.w, kb * 128, tile * kRows, fb);
          else tma_load_2d(sa, &tm.b, (kb - p.nkb) * 64, tile * kRows, fb);
        }
    } else if (warp == 2 && lane == 0) {
      // ---------------------------------------------------------- TMA producer of x (and t) and its scales
      Ring st, sl;
      bool ok = true;
      pdl_wait();
      for (int tile = blockIdx.x; ok && tile < tiles; tile += step)
        for (int kb = kb0; kb < kb1; ++kb, st.next(S)) {
          if (!mbar_wait(smem_u32(&done[st.i]), st.ph ^ 1u) || abort_flag) {
            fail();
            ok = false;
            break;
          }
          const uint32_t sa = smem_u32(smem + st.i * C::kStage) + kWBytes, fb = smem_u32(&full[st.i]);
          mbar_arrive_expect_tx(fb, BN * 128);
          if (kb < p.nkb) {
            const uint32_t sb = smem_u32(&sfull[sl.i]);
            tma_load_2d(sa, &tm.x, kb * 128, 0, fb);
            mbar_arrive_expect_tx(sb, BN * 4);
            bulk_load(smem_u32(&scl[sl.i]), p.sx + static_cast<size_t>(kb) * p.ld_sx, BN * 4, sb);
            sl.next(C::kSlots);
          } else {
            tma_load_2d(sa, &tm.t, (kb - p.nkb) * 64, 0, fb);
          }
        }
    } else if (warp == 1 && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t id8 = idesc_e4m3(kRows, BN), id16 = idesc_f32acc(kRows, BN, false);
      Ring st, buf;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += step)
        for (int kb = kb0; kb < kb1; ++kb, st.next(S), buf.next(C::kBufs)) {
          if (!mbar_wait(smem_u32(&acce[buf.i]), buf.ph ^ 1u) || !mbar_wait(smem_u32(&full[st.i]), st.ph)) {
            fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + static_cast<uint32_t>(buf.i * C::kStride);
          const uint32_t sa = smem_u32(smem + st.i * C::kStage);
          const uint64_t wd = sdesc_k_sw128(sa), xd = sdesc_k_sw128(sa + kWBytes);
          if (kb < p.nkb) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_f8(d, wd + 2 * kk, xd + 2 * kk, id8, kk > 0 ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_ss<false>(d, wd + 2 * kk, xd + 2 * kk, id16, kk > 0 ? 1u : 0u);
          }
          mma_commit(smem_u32(&done[st.i]));
        }
    }
  } else {
    // ------------------------------------------------------------ block sums -> registers
    if (C::kMoveRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    constexpr int kCW = C::kCW, kPer = (kCW + 31) / 32, kChunk = kCW % 32 ? 16 : 32;
    const int quarter = warp & 3, half = (warp - C::kFirst) >> 2;
    const uint32_t tcol = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * kCW);
    constexpr int kB = C::kBatch;
    float(*fw)[kB][kCW] = fac[warp - C::kFirst];
    const int groups = kb1 - kb0;
    pdl_wait();
    // W's scales: a lane holds one of 32 consecutive K-blocks, the next 32 are on their way
    int ahead_tile = blockIdx.x, ahead_kb = kb0;
    auto load_sw = [&]() -> float {
      float v = 1.f;
      if (ahead_tile < tiles) {
        if (ahead_kb + lane < min(kb1, p.nkb))
          v = p.sw[static_cast<size_t>(ahead_tile) * p.ld_sw + ahead_kb + lane];
        if ((ahead_kb += 32) >= kb1) {
          ahead_kb = kb0;
          ahead_tile += step;
        }
      }
      return v;
    };
    float w_now = 1.f, w_next = load_sw();
    int grp = 0;
    Ring st, buf, sl;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < tiles; tile += step) {
      const int tok0 = half * kCW, feat0 = tile * kRows;
      float acc[kCW];
#pragma unroll
      for (int j = 0; j < kCW; ++j) acc[j] = 0.f;
      for (int g = 0; g < groups; g += kB, ++grp) {
        float(*f)[kCW] = fw[grp & 1];
        if ((g & 31) == 0) {
          w_now = w_next;
          w_next = load_sw();
        }
        // factors of the batch (1 for the adapter's blocks)
        const int left = min(kB, groups - g);
#pragma unroll
        for (int u = 0; u < kB; ++u) {
          if (u >= left) break;
          const float ws = __shfl_sync(0xffffffffu, w_now, (g + u) & 31);
          const bool main = kb0 + g + u < p.nkb;
          ok = ok && (!main || __all_sync(0xffffffffu, mbar_wait(smem_u32(&sfull[sl.i]), sl.ph)));
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < kCW)
              f[u][lane + 32 * i] = main ? scl[sl.i][half * kCW + lane + 32 * i] * ws : 1.f;
          if (main) sl.next(C::kSlots);
        }
        __syncwarp();
        for (int u = 1; u < left; ++u) st.next(S);   // MMAs complete in order: wait for the batch's last
        ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&done[st.i]), st.ph));
        if (!ok) break;
        st.next(S);
        tc_fence_after();
        uint32_t v[2][kChunk];
        auto col = [&](int q) {   // chunk q of the batch, kCW / kChunk of them to a buffer
          const int u = q / (kCW / kChunk);
          int b = buf.i + u;
          if (b >= C::kBufs) b -= C::kBufs;
          return tcol + static_cast<uint32_t>(b * C::kStride + q % (kCW / kChunk) * kChunk);
        };
        constexpr int kN = kB * (kCW / kChunk);
        const int nq = left * (kCW / kChunk);
        tmem_ld_async(col(0), v[0]);
#pragma unroll
        for (int q = 0; q < kN; ++q) {
          if (q >= nq) break;
          uint32_t(&w)[kChunk] = v[q & 1];
          tmem_wait_ld(w);
          if (q + 1 < nq) {
            tmem_ld_async(col(q + 1), v[(q + 1) & 1]);
          } else {   // the buffers have been read: hand them back to the MMA issuer
            tc_fence_before();
            __syncwarp();
            if (lane < left) {
              int b = buf.i + lane;
              if (b >= C::kBufs) b -= C::kBufs;
              mbar_arrive(smem_u32(&acce[b]));
            }
          }
          constexpr int kQ = kCW / kChunk;
          const int c = q % kQ * kChunk;
#pragma unroll
          for (int j = 0; j < kChunk; j += 4) {
            const ulonglong2 h = *reinterpret_cast<const ulonglong2*>(&f[q / kQ][c + j]);
            fma2(acc[c + j], acc[c + j + 1], w[j], w[j + 1], h.x);
            fma2(acc[c + j + 2], acc[c + j + 3], w[j + 2], w[j + 3], h.y);
          }
        }
        for (int u = 0; u < left; ++u) buf.next(C::kBufs);
      }
      if (!ok) break;
      if (p.splits > 1) {
        // every MMA has finished, so the stage ring is free: stage the sums [token][feature]
        float* stage = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int j = 0; j < kCW; ++j)
          stage[(half * kCW + j) * (kRows + kPartPad) + quarter * 32 + lane] = acc[j];
      } else {
        // lanes hold features, so pairs of lanes swap halves of two tokens and
        // store two features each
        const int n = feat0 + quarter * 32 + (lane & ~1);
#pragma unroll
        for (int j = 0; j < kCW; j += 2) {
          if (tok0 + j >= p.M) break;
          const bool odd = lane & 1;
          const float other = __shfl_xor_sync(0xffffffffu, odd ? acc[j] : acc[j + 1], 1);
          const int m = tok0 + j + odd;
          const __nv_bfloat162 o = odd ? __floats2bfloat162_rn(other, acc[j + 1]) : __floats2bfloat162_rn(acc[j], other);
          if (m < p.M && n < p.N) *reinterpret_cast<__nv_bfloat162*>(p.y + static_cast<size_t>(m) * p.N + n) = o;
        }
      }
    }
    if (!ok && lane == 0) fail();
  }

  if (p.splits > 1) {
    cluster_sync_converged();
    if (!abort_flag) {
      // the CTAs of the cluster share the tile's outputs out, 4 features at a time
      const int feat0 = static_cast<int>(blockIdx.x) * kRows;
      constexpr int kGroups = BN * (kRows / 4);
      const int Sp = p.splits;
      const int chunk = (kGroups + Sp - 1) / Sp;
      const int e0 = static_cast<int>(cluster_ctarank()) * chunk, e1 = min(kGroups, e0 + chunk);
      const uint32_t part0 = smem_u32(smem);
      uint32_t peer[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) peer[r] = map_shared_rank(part0, r < Sp ? r : 0);
      for (int e = e0 + static_cast<int>(threadIdx.x); e < e1; e += C::kThreads) {
        const int j = e / (kRows / 4), i4 = e % (kRows / 4);
        const int m = j, n = feat0 + 4 * i4;
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
    cluster_sync_converged();   // the peers have read this CTA's sums
  }

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
  const int64_t tiles = (p.N + kRows - 1) / kRows;
  const int smem = static_cast<int>(C::kStages * (C::kStage + 16) + 1024);
  const int nkb = p.nkb + p.nkr, sms = device_sm_count();
  int splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({8, sms / tiles, nkb})));
  p.kb_per_split = (nkb + splits - 1) / splits;
  p.splits = splits = (nkb + p.kb_per_split - 1) / p.kb_per_split;
  auto fn = &fp8_narrow_kernel<BN>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute(8-bit GEMM smem)");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(splits > 1 ? tiles : std::min<int64_t>(tiles, sms)), 1, splits);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = launch_attrs(attr, 1, 1, static_cast<unsigned>(splits));
  cfg.attrs = attr;
  e = cudaLaunchKernelEx(&cfg, fn, tm, p);
  return e == cudaSuccess ? UNO_OK : cuda_error(e, "8-bit GEMM launch");
}

// ---------------------------------------------------------------- many tokens
// A CTA pair (cta_group::2) computes 256 x 256 tiles: CTA r holds tokens
// [128 r, 128 r + 128) of the A side and features [128 r, 128 r + 128) of the B
// side, its TMEM its 128 token rows over all 256 features. The sum of one
// K-block takes a 256-column buffer; two buffers alternate, so while the tensor
// core works on block b (512 cycles at the full e4m3 rate) the eight epilogue
// warps of each CTA add block b - 1 into their registers: a lane has one token
// row and 128 features (one weight scale), i.e. one factor and 128 fused adds a
// block, 256 cycles an SM sub-partition.
// Roles of the 384 threads: warp 0 TMA producer (both CTAs), warp 1 MMA issuer
// (leader), warps 2 and 3 idle, warps 4..11 epilogue (warp % 4: TMEM lanes, (warp - 4)
// / 4: features). The launch gives every thread 168 registers; the first
// warpgroup hands all but 56 of its own to the two epilogue warpgroups, whose
// 128 sums a thread need more (128 (56 + 2 * 224) = 384 * 168).
constexpr int kPairThreads = 384;
constexpr uint32_t kPairStage = 2 * kWBytes;
constexpr int kPairStages = 6;
constexpr int kPairTile = 256;

__global__ void __launch_bounds__(kPairThreads, 1)
    fp8_pair_kernel(const __grid_constant__ Fp8Maps tm, const Fp8Params p) {
  constexpr int S = kPairStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~static_cast<uintptr_t>(1023u));
  __shared__ uint64_t full[S], done[S], acce[2];   // as in the kernel above
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
  const int tiles_m = (p.M + kPairTile - 1) / kPairTile;
  const int num_tiles = tiles_m * ((p.N + kPairTile - 1) / kPairTile);
  const int nkb = p.nkb + p.nkr;   // stages of a tile

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&done[s]), 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(smem_u32(&acce[b]), 16);   // 8 epilogue warps x 2 CTAs
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc_pair(smem_u32(&tmem_slot), 2 * kPairTile);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (threadIdx.x == 0) pdl_trigger();
  auto fail = [&]() {
    abort_flag = 1;
    raise_timeout(p.status);
  };

  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    Ring st;
    bool ok = true, waited = false;
    for (int tile = pair; ok && tile < num_tiles; tile += num_pairs) {
      const int m0 = (tile % tiles_m) * kPairTile + static_cast<int>(rank) * 128;
      const int n0 = (tile / tiles_m) * kPairTile + static_cast<int>(rank) * 128;
      auto load_x = [&](int kb, uint32_t sa, uint32_t fb) {
        if (kb < p.nkb) tma_load_2d_pair(sa, &tm.x, kb * 128, m0, fb);
        else tma_load_2d_pair(sa, &tm.t, (kb - p.nkb) * 64, m0, fb);
      };
      auto load_w = [&](int kb, uint32_t sa, uint32_t fb) {
        if (kb < p.nkb) tma_load_2d_pair(sa + kWBytes, &tm.w, kb * 128, n0, fb);
        else tma_load_2d_pair(sa + kWBytes, &tm.b, (kb - p.nkb) * 64, n0, fb);
      };
      int kb = 0;
      if (!waited) {   // weights (constant) of the first stages before waiting for xq and t
        const int pre = min(S, nkb);
        for (int q = 0; q < pre; ++q) {
          if (leader) mbar_arrive_expect_tx(smem_u32(&full[q]), 2 * kPairStage);
          load_w(q, smem_u32(smem + q * kPairStage), map_shared_rank(smem_u32(&full[q]), 0));
        }
        pdl_wait();
        waited = true;
        for (; kb < pre; ++kb, st.next(S))
          load_x(kb, smem_u32(smem + kb * kPairStage), map_shared_rank(smem_u32(&full[kb]), 0));
      }
      for (; kb < nkb; ++kb, st.next(S)) {
        if (!mbar_wait(smem_u32(&done[st.i]), st.ph ^ 1u) || abort_flag) {
          fail();
          ok = false;
          break;
        }
        const uint32_t fb = map_shared_rank(smem_u32(&full[st.i]), 0);
        const uint32_t sa = smem_u32(smem + st.i * kPairStage);
        if (leader) mbar_arrive_expect_tx(smem_u32(&full[st.i]), 2 * kPairStage);
        load_x(kb, sa, fb);
        load_w(kb, sa, fb);
      }
    }
    if (!waited) pdl_wait();
  } else if (warp == 1 && lane == 0 && leader) {
    // ------------------------------------------------------------ MMA issuer (leader)
    const uint32_t id8 = idesc_e4m3(kPairTile, kPairTile), id16 = idesc_f32acc(kPairTile, kPairTile, false);
    Ring st, buf;
    bool ok = true;
    for (int tile = pair; ok && tile < num_tiles; tile += num_pairs) {
      for (int kb = 0; kb < nkb; ++kb, st.next(S), buf.next(2)) {
        if (!mbar_wait_cluster(smem_u32(&acce[buf.i]), buf.ph ^ 1u) || !mbar_wait(smem_u32(&full[st.i]), st.ph)) {
          fail();
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(buf.i * kPairTile);
        const uint32_t sa = smem_u32(smem + st.i * kPairStage);
        const uint64_t ad = sdesc_k_sw128(sa), bd = sdesc_k_sw128(sa + kWBytes);
        if (kb < p.nkb) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_pair_f8(d, ad + 2 * kk, bd + 2 * kk, id8, kk > 0 ? 1u : 0u);
        } else {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_pair_bf16(d, ad + 2 * kk, bd + 2 * kk, id16, kk > 0 ? 1u : 0u);
        }
        mma_commit_both(smem_u32(&done[st.i]));
      }
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // ------------------------------------------------------------ block sums -> registers (both CTAs)
    const int quarter = warp & 3, h = (warp - 4) >> 2;
    const uint32_t tcol = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(h * 128);
    Ring st, buf;
    bool ok = true;
    pdl_wait();
    for (int tile = pair; ok && tile < num_tiles; tile += num_pairs) {
      const int m = (tile % tiles_m) * kPairTile + static_cast<int>(rank) * 128 + quarter * 32 + lane;
      const int n0 = (tile / tiles_m) * kPairTile + h * 128;
      const bool have_m = m < p.ld_sx, have_n = n0 < p.N;
      const float* sx = p.sx + (have_m ? m : 0);
      const float* sw = p.sw + (have_n ? static_cast<size_t>(n0 >> 7) * p.ld_sw : 0);
      // a block's two scales are loaded two blocks ahead and multiplied when they
      // are used (a product any earlier would stall on the loads)
      auto load_x = [&](int g) { return g < p.nkb ? sx[static_cast<size_t>(g) * p.ld_sx] : 1.f; };
      auto load_w = [&](int g) { return g < p.nkb ? sw[g] : 1.f; };
      float fx[2] = {load_x(0), load_x(1)}, fw[2] = {load_w(0), load_w(1)};
      float acc[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) acc[c] = 0.f;
      for (int g = 0; g < nkb; ++g, st.next(S), buf.next(2)) {
        const float f = fx[0] * fw[0];
        fx[0] = fx[1];
        fw[0] = fw[1];
        fx[1] = load_x(g + 2);
        fw[1] = load_w(g + 2);
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&done[st.i]), st.ph));
        if (!ok) break;
        tc_fence_after();
        const uint32_t t0 = tcol + static_cast<uint32_t>(buf.i * kPairTile);
        uint32_t v[2][32];
        const uint64_t ff = pack2(f, f);
        auto add = [&](int c) {
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            fma2(acc[32 * c + j], acc[32 * c + j + 1], v[c & 1][j], v[c & 1][j + 1], ff);
        };
        // only half of the adds stand before the buffer is handed back
        tmem_ld_async(t0, v[0]);
        tmem_ld_async(t0 + 32, v[1]);
        tmem_wait_ld(v[0]);
        tmem_wait_ld(v[1]);
        add(0);
        tmem_ld_async(t0 + 64, v[0]);
        add(1);
        tmem_ld_async(t0 + 96, v[1]);
        tmem_wait_ld(v[0]);
        tmem_wait_ld(v[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(map_shared_rank(smem_u32(&acce[buf.i]), 0));
        add(2);
        add(3);
      }
      if (!ok) {
        if (lane == 0) fail();
        break;
      }
      if (m < p.M) {
        __nv_bfloat16* y = p.y + static_cast<size_t>(m) * p.N + n0;
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
          if (n0 + c >= p.N) break;
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 q = __floats2bfloat162_rn(acc[c + 2 * e], acc[c + 2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&q);
          }
          *reinterpret_cast<uint4*>(y + c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }

  tc_fence_before();
  cluster_sync_converged();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * kPairTile);
  }
}

uno_status pair_launch(const Fp8Maps& tm, const Fp8Params& p, cudaStream_t s) {
  const int64_t tiles = static_cast<int64_t>((p.M + kPairTile - 1) / kPairTile) *
                        ((p.N + kPairTile - 1) / kPairTile);
  if (tiles > (1ll << 30)) return set_error(UNO_ERR_UNSUPPORTED, "too many tiles");
  const int pairs = static_cast<int>(std::min<int64_t>(std::max(1, device_sm_count() / 2), tiles));
  const int smem = static_cast<int>(kPairStages * kPairStage + 1024);
  cudaError_t e = cudaFuncSetAttribute(&fp8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute(8-bit pair smem)");
  e = launch_kernel(fp8_pair_kernel, dim3(2 * pairs), dim3(kPairThreads), smem, s, 2, tm, p);
  return e == cudaSuccess ? UNO_OK : cuda_error(e, "8-bit pair GEMM launch");
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
  p.status = g.status;
  const bool pair = g.M > 256 || (g.M > 128 && g.N >= 256 * (device_sm_count() / 2));
  const int bn = g.M <= 16 ? 16 : g.M <= 32 ? 32 : g.M <= 64 ? 64 : g.M <= 128 ? 128 : g.M <= 160 ? 160 : g.M <= 192 ? 192 : 256;
  const int xbox = pair ? 128 : bn;
  Fp8Maps tm;
  uno_status st;
  if ((st = make_map_u8(&tm.x, g.xq, g.K, g.M, g.K, xbox)) != UNO_OK) return st;
  if ((st = make_map_u8(&tm.w, g.wq, g.K, g.N, g.K, kRows)) != UNO_OK) return st;
  tm.t = tm.x;
  tm.b = tm.w;
  if (g.r > 0) {
    if ((st = make_map(&tm.t, UNO_BF16, g.t, g.r, g.M, g.r, xbox)) != UNO_OK) return st;
    if ((st = make_map(&tm.b, UNO_BF16, g.Bl, g.r, g.N, g.r, kRows)) != UNO_OK) return st;
  }
  if (pair) return pair_launch(tm, p, s);
  switch (bn) {
    case 16: return narrow_launch<16>(tm, p, s);
    case 32: return narrow_launch<32>(tm, p, s);
    case 64: return narrow_launch<64>(tm, p, s);
    case 128: return narrow_launch<128>(tm, p, s);
    case 160: return narrow_launch<160>(tm, p, s);
    case 192: return narrow_launch<192>(tm, p, s);
    default: return narrow_launch<256>(tm, p, s);
  }
}

}  // namespace uno

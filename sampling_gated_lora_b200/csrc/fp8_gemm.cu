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
//
// Few tokens: HBM bandwidth bounds it (9 x 4096 -> 151936: 622 MB of codes in
// 129 us, 0.74 of the copy rate). Many: an epilogue warp's wait, TMEM loads and
// adds of a K-block, about 860 cycles where the tensor core needs 512
// (2048 x 12288 -> 4096: 111 us, 130 with the down-projection; 4352 rows: 266;
// single calls after a pause, 150 and 311 in a stream of calls at the clock that the
// power cap leaves).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "per_device.h"

#include "fp8.cuh"

namespace uno {

namespace {

constexpr int kThreads = 384;
constexpr int kRows = 128;                           // token rows of a CTA (MMA M, TMEM lanes)
constexpr int kMaxWidth = 256;                       // features of a tile (MMA N, TMEM columns)
constexpr int kPartPad = 4;
constexpr int kPairStages = 6;

struct Fp8Maps {
  CUtensorMap x, w, t, b;
};

struct Fp8Params {
  int M, N, nkb, nkr;        // K-blocks of xq wq^T and of t Bl^T
  int tiles_m, tiles;        // token tiles, all tiles
  int kb_per_split, splits;
  int stages;
  uint32_t x_bytes, stage_bytes;   // of a stage in one CTA: x, x and W
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

// One tile: 128 token rows (kPair: 256, the pair's CTAs hold 128 each) x kWidth
// features. A TMEM lane is a token and a column a feature, so a lane's
// scale of x is one value a K-block and the columns of an epilogue warp share
// one or two scales of W. The sum of a K-block takes one of two 256-column
// buffers: while the tensor core works on one, the eight epilogue warps (lanes
// by warp % 4, halves of the columns) add the other to their registers.
//
// kPair (cta_group::2, many tokens): CTA r holds tokens [128 r, 128 r + 128) of
// the A side and half of the tile's W rows; each CTA loads 32 KB a K-block for
// what a CTA alone would load 48 KB for, and W passes once for 256 tokens.
// Otherwise one CTA computes the tile; x comes in only as many rows as there are, epilogue warps without tokens only
// pass the buffers on, and with fewer tiles than SMs K is split over a
// thread-block cluster whose sums meet through distributed shared memory in
// rank order.
//
// Threads: warp 0 TMA producer, warp 1 MMA issuer (kPair: the leader's), both
// converged (elect_one), warps 2 and 3 idle, warps 4..11 epilogue (sixteen with
// half the columns each: 141 us where these take 131, 2048 x 12288 -> 4096).
// The launch gives every thread 168 registers; the first warpgroup hands all but
// 56 of its own to the two epilogue warpgroups, whose 128 sums a thread need more
// (128 (56 + 2 * 224) = 384 * 168).
template <bool kPair, int kWidth>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ Fp8Maps tm, const Fp8Params p) {
  constexpr int kMaxStages = 12;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023u) & ~static_cast<uintptr_t>(1023u));
  // full: a stage has been filled; done: the MMAs on it have completed (frees the
  // stage to the producer and shows the block's sum to the epilogue, which is
  // never more than two buffers behind, so it sees every phase); acce: a TMEM
  // buffer has been read
  __shared__ uint64_t full[kMaxStages], done[kMaxStages], acce[2];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0;
  const int S = kPair ? kPairStages : p.stages;
  const uint32_t x_bytes = kPair ? kRows * 128 : p.x_bytes, stage_bytes = kPair ? 2 * kRows * 128 : p.stage_bytes;
  const int first = kPair ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
  const int step = kPair ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);
  const int nkb = p.nkb + p.nkr;
  const int kb0 = kPair ? 0 : static_cast<int>(blockIdx.z) * p.kb_per_split;
  const int kb1 = kPair ? nkb : min(nkb, kb0 + p.kb_per_split);
  const uint32_t row0 = rank * kRows;                // of this CTA's tokens in a tile
  constexpr int kTileRows = kPair ? 2 * kRows : kRows;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&done[s]), 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(smem_u32(&acce[b]), kPair ? 16 : 8);   // epilogue warps
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    if (kPair) {
      tmem_alloc_pair(smem_u32(&tmem_slot), 2 * kMaxWidth);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&tmem_slot), 2 * kMaxWidth);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (kPair) cluster_sync();
  else cta_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (threadIdx.x == 0) pdl_trigger();
  auto fail = [&]() {
    abort_flag = 1;
    raise_timeout(p.status);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer
      auto load = [&](uint32_t dst, const CUtensorMap* map, int c, int r, int s) {
        if (kPair) tma_load_2d_pair(dst, map, c, r, map_shared_rank(smem_u32(&full[s]), 0));
        else tma_load_2d(dst, map, c, r, smem_u32(&full[s]));
      };
      auto load_x = [&](int tile, int kb, int s) {
        const uint32_t dst = smem_u32(smem + s * stage_bytes);
        const int m0 = tile % p.tiles_m * kTileRows + static_cast<int>(row0);
        if (kb < p.nkb) load(dst, &tm.x, kb * 128, m0, s);
        else load(dst, &tm.t, (kb - p.nkb) * 64, m0, s);
      };
      auto load_w = [&](int tile, int kb, int s) {
        const uint32_t dst = smem_u32(smem + s * stage_bytes) + x_bytes;
        const int n0 = tile / p.tiles_m * kWidth + static_cast<int>(rank) * (kWidth / 2);
        if (kb < p.nkb) load(dst, &tm.w, kb * 128, n0, s);
        else load(dst, &tm.b, (kb - p.nkb) * 64, n0, s);
      };
      auto expect = [&](int s) {
        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full[s]), (kPair ? 2 : 1) * stage_bytes);
      };
      // weights (constant) of the first stages before waiting for the writer of xq and t
      Ring st;
      int skip = min(S, kb1 - kb0);   // blocks of the first tile that are on their way
      if (elect_one())
        for (int q = 0; q < skip; ++q) {
          expect(q);
          load_w(first, kb0 + q, q);
        }
      __syncwarp();
      pdl_wait();
      for (int q = 0; q < skip; ++q, st.next(S)) {
        if (elect_one()) load_x(first, kb0 + q, q);
        __syncwarp();
      }
      bool ok = true;
      for (int tile = first; ok && tile < p.tiles; tile += step, skip = 0)
        for (int kb = kb0 + skip; kb < kb1; ++kb, st.next(S)) {
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&done[st.i]), st.ph ^ 1u) && !abort_flag);
          if (!ok) break;
          if (elect_one()) {
            expect(st.i);
            load_w(tile, kb, st.i);
            load_x(tile, kb, st.i);
          }
          __syncwarp();
        }
      if (!ok && lane == 0) fail();
    } else if (warp == 1 && rank == 0) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t id8 = idesc_e4m3(kTileRows, kWidth), id16 = idesc_f32acc(kTileRows, kWidth, false);
      Ring st, buf;
      bool ok = true;
      for (int tile = first; ok && tile < p.tiles; tile += step)
        for (int kb = kb0; kb < kb1; ++kb, st.next(S), buf.next(2)) {
          ok = __all_sync(0xffffffffu, (kPair ? mbar_wait_cluster(smem_u32(&acce[buf.i]), buf.ph ^ 1u)
                                              : mbar_wait(smem_u32(&acce[buf.i]), buf.ph ^ 1u)) &&
                                           mbar_wait(smem_u32(&full[st.i]), st.ph));
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + static_cast<uint32_t>(buf.i * kMaxWidth);
          const uint32_t sa = smem_u32(smem + st.i * stage_bytes);
          const uint64_t xd = sdesc_k_sw128(sa), wd = sdesc_k_sw128(sa + x_bytes);
          if (elect_one()) {
            if (kb < p.nkb) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                if (kPair) mma_pair_f8(d, xd + 2 * kk, wd + 2 * kk, id8, kk > 0 ? 1u : 0u);
                else mma_f8(d, xd + 2 * kk, wd + 2 * kk, id8, kk > 0 ? 1u : 0u);
              }
            } else {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                if (kPair) mma_pair_bf16(d, xd + 2 * kk, wd + 2 * kk, id16, kk > 0 ? 1u : 0u);
                else mma_ss<false>(d, xd + 2 * kk, wd + 2 * kk, id16, kk > 0 ? 1u : 0u);
              }
            }
            if (kPair) mma_commit_both(smem_u32(&done[st.i]));
            else mma_commit(smem_u32(&done[st.i]));
          }
          __syncwarp();
        }
      if (!ok && lane == 0) fail();
    }
  } else {
    // ------------------------------------------------------------ block sums -> registers
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // (from threadIdx: with the shuffled index the accumulators spill; this way the
    // pair form still spills five words, the others none)
    const int quarter = (threadIdx.x >> 5) & 3, half = (static_cast<int>(threadIdx.x >> 5) - 4) >> 2;
    constexpr int kCols = kWidth / 2;        // of this warp
    constexpr bool kOneScale = kCols % 128 == 0 || 128 % kCols == 0;   // they share one scale of W
    const uint32_t tcol = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * kCols);
    Ring st, buf;
    bool ok = true;
    pdl_wait();
    for (int tile = first; ok && tile < p.tiles; tile += step) {
      const int m_warp = tile % p.tiles_m * kTileRows + static_cast<int>(row0) + quarter * 32, m = m_warp + lane;
      const int n0 = tile / p.tiles_m * kWidth + half * kCols;
      const bool work = m_warp < p.M && n0 < p.N;
      // columns below `edge` are in W's scale block n0 / 128, the others in the next
      const int nb = min(n0, p.N - 1) >> 7, edge = ((nb + 1) << 7) - n0;
      const float* sx = p.sx + min(m, p.ld_sx - 1);
      const float* sw0 = p.sw + static_cast<size_t>(nb) * p.ld_sw;
      const float* sw1 = edge < kCols && n0 + edge < p.N ? sw0 + p.ld_sw : sw0;
      // a block's scales are loaded two blocks ahead and multiplied when they are
      // used (a product any earlier would stall on the loads)
      float fx[2], f0[2], f1[2];
      auto load_scales = [&](int kb, int i) {
        const bool main = work && kb < min(kb1, p.nkb);   // the adapter's blocks have factor 1
        fx[i] = main ? sx[static_cast<size_t>(kb) * p.ld_sx] : 1.f;
        f0[i] = main ? sw0[kb] : 1.f;
        if (!kOneScale) f1[i] = main ? sw1[kb] : 1.f;
      };
      load_scales(kb0, 0);
      load_scales(kb0 + 1, 1);
      float acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
      for (int kb = kb0; kb < kb1; ++kb, st.next(S), buf.next(2)) {
        const float g0 = fx[0] * f0[0], g1 = kOneScale ? g0 : fx[0] * f1[0];
        const uint64_t gg0 = pack2(g0, g0), gg1 = pack2(g1, g1);
        fx[0] = fx[1];
        f0[0] = f0[1];
        if (!kOneScale) f1[0] = f1[1];
        load_scales(kb + 2, 1);
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&done[st.i]), st.ph));
        if (!ok) break;
        tc_fence_after();
        const uint32_t t0 = tcol + static_cast<uint32_t>(buf.i * kMaxWidth);
        auto hand_back = [&]() {   // the buffer has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (kPair) mbar_arrive_cluster_relaxed(map_shared_rank(smem_u32(&acce[buf.i]), 0));
            else mbar_arrive(smem_u32(&acce[buf.i]));
          }
        };
        if (!work) {
          hand_back();
          continue;
        }
        // units of kUnit columns, two in flight: of 128 columns, half of the adds
        // stand before the buffer is handed back
        constexpr int kUnit = kCols % 32 ? 16 : 32, kUnits = kCols / kUnit;
        uint32_t v[2][kUnit];
        auto add = [&](int u) {
          const uint64_t g = kOneScale || kUnit * u < edge ? gg0 : gg1;
#pragma unroll
          for (int j = 0; j < kUnit; j += 2)
            fma2(acc[kUnit * u + j], acc[kUnit * u + j + 1], v[u & 1][j], v[u & 1][j + 1], g);
        };
        tmem_ld_async(t0, v[0]);
        tmem_ld_async(t0 + kUnit, v[1]);
#pragma unroll
        for (int u = 0; u < kUnits; u += 2) {
          tmem_wait_ld(v[0]);
          tmem_wait_ld(v[1]);
          if (u + 2 >= kUnits) hand_back();
          add(u);
          if (u + 2 < kUnits) tmem_ld_async(t0 + kUnit * (u + 2), v[0]);
          if (u + 1 < kUnits) add(u + 1);
          if (u + 3 < kUnits) tmem_ld_async(t0 + kUnit * (u + 3), v[1]);
        }
      }
      if (!ok) break;
      if (!kPair && p.splits > 1) {
        // one tile; every MMA has finished, so the stage ring is free: stage the
        // sums [token][feature]
        float* stage = reinterpret_cast<float*>(smem) + (quarter * 32 + lane) * (kWidth + kPartPad) + half * kCols;
        if (m < p.M) {
#pragma unroll
          for (int c = 0; c < kCols; c += 4)
            *reinterpret_cast<float4*>(stage + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
        }
      } else if (m < p.M) {
        __nv_bfloat16* y = p.y + static_cast<size_t>(m) * p.N + n0;
#pragma unroll
        for (int c = 0; c < kCols; c += 8) {
          if (n0 + c >= p.N) break;
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 q = __floats2bfloat162_rn(acc[c + 2 * e], acc[c + 2 * e + 1]);
            o[e] = *reinterpret_cast<const uint32_t*>(&q);
          }
          *reinterpret_cast<uint4*>(y + c) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    if (!ok && lane == 0) fail();
  }

  if (!kPair && p.splits > 1) {
    cluster_sync_converged();
    if (!abort_flag) {
      // the CTAs of the cluster share the tile's outputs out, 4 features at a time
      const int m0 = first % p.tiles_m * kTileRows, n0 = first / p.tiles_m * kWidth;
      const int quads = kWidth / 4, groups = min(kRows, p.M - m0) * quads;
      const int Sp = p.splits;
      const int chunk = (groups + Sp - 1) / Sp;
      const int e0 = static_cast<int>(cluster_ctarank()) * chunk, e1 = min(groups, e0 + chunk);
      const uint32_t part0 = smem_u32(smem);
      uint32_t peer[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) peer[r] = map_shared_rank(part0, r < Sp ? r : 0);
      for (int e = e0 + static_cast<int>(threadIdx.x); e < e1; e += kThreads) {
        const int j = e / quads, n = n0 + 4 * (e % quads);
        if (n >= p.N) continue;
        const uint32_t off = static_cast<uint32_t>((j * (kWidth + kPartPad) + 4 * (e % quads)) * 4);
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
        *reinterpret_cast<uint2*>(p.y + static_cast<size_t>(m0 + j) * p.N + n) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
    cluster_sync_converged();   // the peers have read this CTA's sums
  }

  tc_fence_before();
  if (kPair) cluster_sync_converged();
  else cta_sync_converged();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    if (kPair) tmem_dealloc_pair(tmem, 2 * kMaxWidth);
    else tmem_dealloc(tmem, 2 * kMaxWidth);
  }
}

constexpr int kRing = 196 * 1024;   // bytes of the stage ring
static_assert(kRows * (kMaxWidth + kPartPad) * 4 <= kRing, "the sums of a split tile must fit the ring");

// Clusters of `size` CTAs (along z) that `device` (the current one) holds at once.
int resident_clusters(int device, int size) {
  static PerDevice<9> kept;
  return kept.get(device, size, [&] {
    return resident_clusters_of(reinterpret_cast<const void*>(&fp8_gemm_kernel<false, kMaxWidth>), kThreads,
                                kRing + 1024, size);
  });
}

// The launch form with the least estimated time. A K-block of a tile of w
// features takes about 380 + 0.63 w ns (measured between 128 and 256 features at
// 2048 x 12288 -> 4096: an epilogue warp's wait, loads and adds), and not less
// than the 2.8 w ns in which HBM brings its w rows of W to one SM of 148 when W
// passes by once. CTA pairs take 2 % longer for twice the tokens (544 .. 4352
// rows); up to 256 rows they read W once where two token tiles that drift apart
// read it twice (136 x 4096 -> 151936: 197 us against 221; the 0.97 below is from
// that size alone and stands for every N and K). Single CTAs fill the
// device with half the tokens a tile, and can split K.
struct Plan {
  bool pair;
  int width;
};

Plan plan(Fp8Params* p) {
  const int nkb = p->nkb + p->nkr, sms = device_sm_count(), device = current_device();
  Plan best{};
  double least = -1.;
  auto consider = [&](bool pair, int w, int splits) {
    const int rows = pair ? 2 * kRows : kRows, slots = pair ? std::max(1, sms / 2) : sms;
    const int tiles_m = (p->M + rows - 1) / rows;
    const int64_t tiles = static_cast<int64_t>(tiles_m) * ((p->N + w - 1) / w);
    if (splits > 1 && tiles > resident_clusters(device, splits)) return false;   // one wave of clusters only
    const int per = (nkb + splits - 1) / splits;
    double block = 380. + 0.63 * w;
    if (tiles_m == 1) block = std::max(block, pair ? 1.4 * w : 2.8 * w);
    if (pair) block *= p->M <= 2 * kRows ? 0.97 : 1.02;
    const double cost = static_cast<double>((tiles + slots - 1) / slots) * per * block;
    if (least < 0. || cost < least) {
      least = cost;
      best = Plan{pair, w};
      p->tiles_m = tiles_m;
      p->tiles = static_cast<int>(std::min<int64_t>(tiles, 1ll << 30));
      p->kb_per_split = per;
      p->splits = (nkb + per - 1) / per;
    }
    return true;
  };
  for (int w : {256, 224, 192, 128})
    for (int splits = 1; splits <= std::min(8, nkb) && consider(false, w, splits); ++splits) {
    }
  if (p->M > kRows) consider(true, kMaxWidth, 1);
  return best;
}

template <bool kPair, int kWidth>
uno_status gemm_launch(const Fp8Maps& tm, Fp8Params p, cudaStream_t s) {
  // an MMA reads 128 rows of x whatever the stage holds of them: past x it reads W's
  static_assert(kPair || kWidth >= kRows, "128 rows of a stage that holds any of x must lie within it");
  p.stages = std::min(12, static_cast<int>(kRing / p.stage_bytes));
  const int smem = kRing + 1024;
  auto fn = &fp8_gemm_kernel<kPair, kWidth>;
  static SmemGranted granted;
  cudaError_t e = granted.ask(reinterpret_cast<const void*>(fn), smem);
  if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute(8-bit GEMM smem)");
  const int slots = kPair ? std::max(1, device_sm_count() / 2) : device_sm_count();
  const int ctas = p.splits > 1 ? p.tiles : std::min(p.tiles, slots);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kPair ? 2 * ctas : ctas, 1, p.splits);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = launch_attrs(attr, kPair ? 2 : 1, 1, static_cast<unsigned>(p.splits));
  cfg.attrs = attr;
  e = cudaLaunchKernelEx(&cfg, fn, tm, p);
  return e == cudaSuccess ? UNO_OK : cuda_error(e, "8-bit GEMM launch");
}

}  // namespace

int resident_clusters_of(const void* kernel, int threads, int smem, int size) {
  int n = 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1, 1, size);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = size;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = std::max(1, device_sm_count() / size);
  }
  return n;
}

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
  const Plan form = plan(&p);
  if (p.tiles >= (1 << 30)) return set_error(UNO_ERR_UNSUPPORTED, "too many tiles");
  const int xbox = form.pair ? kRows : static_cast<int>(std::min<int64_t>(kRows, (g.M + 7) / 8 * 8));
  const int wbox = form.pair ? form.width / 2 : form.width;
  p.x_bytes = static_cast<uint32_t>(xbox * 128);
  p.stage_bytes = p.x_bytes + static_cast<uint32_t>(wbox * 128);
  Fp8Maps tm;
  uno_status st;
  if ((st = make_map_u8(&tm.x, g.xq, g.K, g.M, g.K, xbox)) != UNO_OK) return st;
  if ((st = make_map_u8(&tm.w, g.wq, g.K, g.N, g.K, wbox)) != UNO_OK) return st;
  tm.t = tm.x;
  tm.b = tm.w;
  if (g.r > 0) {
    if ((st = make_map(&tm.t, UNO_BF16, g.t, g.r, g.M, g.r, xbox)) != UNO_OK) return st;
    if ((st = make_map(&tm.b, UNO_BF16, g.Bl, g.r, g.N, g.r, wbox)) != UNO_OK) return st;
  }
  if (form.pair) return gemm_launch<true, 256>(tm, p, s);
  switch (form.width) {
    case 256: return gemm_launch<false, 256>(tm, p, s);
    case 224: return gemm_launch<false, 224>(tm, p, s);
    case 192: return gemm_launch<false, 192>(tm, p, s);
    default: return gemm_launch<false, 128>(tm, p, s);
  }
}

}  // namespace uno

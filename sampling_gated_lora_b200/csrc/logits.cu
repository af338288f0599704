// Token counts of running sequences, and the rules a user puts on their
// logits before they are sampled or verified.
//
// A sequence's record is one 16-bit word per vocabulary id: bit 15 = the id
// occurs in the prompt, bits 0..14 = how often it was emitted (it stays at
// 32767). token_counts_add raises it for the ids of a prompt or of a verified
// block; logits_process reads it.
//
// For row j of sequence b (tokens the row's path adds to the record: the first
// j drafted ids, or the row's own list), with n the emitted count of id v:
//   z' = z / rho (z > 0) or z * rho (z <= 0)   if n > 0 or v is in the prompt
//   z' -= frequency n + presence [n > 0]
//   z' += sum of the biases listed for v
//   z' = -inf                                   if the row's mask bit is 0
// computed in float and rounded once to the logits' type.
//
// HBM bandwidth bounds both: every logit is read and written once, the record
// and the mask once. Few ids have a record, a bias or a place on the path, so
// the dense pass only branches per 16-byte vector on "any record here", and
// the ids of the path and the bias list (at most a few hundred) are recomputed
// from the original logits by single threads and overwrite the dense result.
// A vector whose mask bits are all 0 needs no logits at all.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace uno {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kMaxSpecial = kMaxPath + kMaxBias;

// ---------------------------------------------------------------- counts

// Adds are saturating compare-and-swap loops, so any number of equal ids in
// one call, in one sequence or in several that share a slot, are all counted
// and the result does not depend on their order.
__global__ void __launch_bounds__(256)
    counts_add_kernel(unsigned short* __restrict__ counts, int S, int V, const int32_t* __restrict__ tokens,
                      int T, long long total, const int32_t* __restrict__ lens,
                      const int32_t* __restrict__ slots, int prompt, int32_t* dev_status) {
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  pdl_wait();
  if (i >= total) return;
  const int b = static_cast<int>(i / T), pos = static_cast<int>(i - static_cast<long long>(b) * T);
  if (lens && pos >= lens[b]) return;
  const int tok = tokens[i];
  if (tok == -1) return;
  const int slot = slots ? slots[b] : b;
  if (tok < 0 || tok >= V || slot < 0 || slot >= S) {
    raise_status(dev_status, kDevBadIndex);
    return;
  }
  unsigned short* w = counts + static_cast<size_t>(slot) * V + tok;
  unsigned short old = *reinterpret_cast<volatile unsigned short*>(w);
  while (true) {
    unsigned short want;
    if (prompt) {
      if (old & 0x8000u) return;
      want = static_cast<unsigned short>(old | 0x8000u);
    } else {
      if ((old & 0x7fffu) == 0x7fffu) return;
      want = static_cast<unsigned short>(old + 1);
    }
    const unsigned short seen = atomicCAS(w, old, want);
    if (seen == old) return;
    old = seen;
  }
}

// ---------------------------------------------------------------- rules

template <typename T>
struct LogitVec;   // 16 bytes of logits
template <>
struct LogitVec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(uint4 w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(u[i]);
      f[2 * i + 1] = bf16_hi(u[i]);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct LogitVec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(uint4 w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

struct Rules {
  float rho, freq, pres;
};

// n: emitted count; held: emitted or in the prompt
__device__ __forceinline__ float apply_rules(const Rules& r, float z, int n, bool held) {
  if (held) z = z > 0.f ? __fdiv_rn(z, r.rho) : z * r.rho;
  if (n > 0) z = z - r.freq * static_cast<float>(n) - r.pres;
  return z;
}

// kAligned: rows start on 16-byte boundaries (of the logits, the record and,
// bitwise, the mask). Otherwise a row's 16-byte vectors start at a = row * V
// mod kN elements before its first id, the first and last are handled id by
// id, and record words and mask bits are gathered one by one.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(kThreads)
    logits_kernel(const LogitsArgs a, int chunks) {
  using Vec = LogitVec<T>;
  constexpr int kN = Vec::kN;
  constexpr int kChunk = kThreads * kUnroll * kN;
  __shared__ int32_t ids[kMaxSpecial];
  __shared__ float vals[kMaxSpecial];
  const long long row = blockIdx.x / chunks;
  const int chunk = static_cast<int>(blockIdx.x - row * chunks);
  const int b = static_cast<int>(row / a.R), j = static_cast<int>(row - static_cast<long long>(b) * a.R);
  const int V = a.V;
  const T* in = static_cast<const T*>(a.logits) + row * V;
  T* out = static_cast<T*>(a.out) + row * V;
  const int lead = kAligned ? 0 : static_cast<int>((row * V) % kN);
  const int v_begin = chunk * kChunk - lead;   // id of the chunk's first vector element
  pdl_wait();

  const int slot = a.slots ? a.slots[b] : b;
  const bool has_rec = a.counts && slot >= 0 && slot < a.S;
  if (a.counts && !has_rec && chunk == 0 && threadIdx.x == 0) raise_status(a.dev_status, kDevBadIndex);
  const unsigned short* rec = has_rec ? a.counts + static_cast<size_t>(slot) * V : nullptr;
  const int mask_words = (V + 31) / 32;
  const uint32_t* mask = a.mask ? a.mask + row * mask_words : nullptr;
  Rules r;
  r.rho = a.repetition ? a.repetition[b] : 1.f;
  r.freq = a.frequency ? a.frequency[b] : 0.f;
  r.pres = a.presence ? a.presence[b] : 0.f;

  // mask bits of the vector's ids (bit e: id v + e); ids outside the row read 0
  auto allowed = [&](int v) -> uint32_t {
    constexpr uint32_t kAll = (1u << kN) - 1u;
    if (kAligned) {
      if (v >= V) return 0u;
      return mask ? (mask[v >> 5] >> (v & 31)) & kAll : kAll;
    }
    uint32_t bits = 0u;
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const int id = v + e;
      if (id >= 0 && id < V && (!mask || ((mask[id >> 5] >> (id & 31)) & 1u))) bits |= 1u << e;
    }
    return bits;
  };
  auto whole = [&](int v) { return kAligned ? v < V : v >= 0 && v + kN <= V; };

  // dense loads first: they fly while the special ids are looked up
  uint32_t bits[kUnroll];
  uint4 z[kUnroll], c[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    bits[u] = allowed(v_begin + (u * kThreads + static_cast<int>(threadIdx.x)) * kN);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int v = v_begin + (u * kThreads + static_cast<int>(threadIdx.x)) * kN;
    z[u] = c[u] = make_uint4(0u, 0u, 0u, 0u);
    if (bits[u] && whole(v)) {
      z[u] = *reinterpret_cast<const uint4*>(in + v);
      if (kAligned && rec) {
        if (kN == 8) {
          c[u] = *reinterpret_cast<const uint4*>(rec + v);
        } else {
          const uint2 h = *reinterpret_cast<const uint2*>(rec + v);
          c[u].x = h.x;
          c[u].y = h.y;
        }
      }
    }
  }

  // ids of the path and of the bias list that fall into this chunk
  const int np = a.path ? (a.path_per_row ? a.P : min(j, a.P)) : 0;
  const int n_special = np + a.nb;
  if (n_special > 0) {
    const int32_t* path = a.path + (a.path_per_row ? row : b) * a.P;
    const int32_t* bid = a.bias_ids + static_cast<size_t>(b) * a.nb;
    for (int i = threadIdx.x; i < n_special; i += kThreads) {
      int id = i < np ? path[i] : bid[i - np];
      if (id < 0 || id >= V) {
        if (id != -1 && chunk == 0) raise_status(a.dev_status, kDevBadIndex);
        id = -1;
      }
      ids[i] = id;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_special; i += kThreads) {
      const int id = ids[i];
      bool mine = id >= 0 && id >= v_begin && id < v_begin + kChunk;
      for (int q = 0; mine && q < i; ++q) mine = ids[q] != id;   // the first of equal ids acts for all
      if (!mine) continue;
      float v = -INFINITY;
      if (!mask || ((mask[id >> 5] >> (id & 31)) & 1u)) {
        int n = 0;
        for (int q = 0; q < np; ++q) n += ids[q] == id;
        const unsigned short w = rec ? rec[id] : 0;
        n += w & 0x7fff;
        v = apply_rules(r, to_f32<T>(in[id]), n, n > 0 || (w & 0x8000u));
        float add = 0.f;
        bool any = false;
        for (int q = np; q < n_special; ++q)
          if (ids[q] == id) {
            add += a.bias[static_cast<size_t>(b) * a.nb + (q - np)];
            any = true;
          }
        if (any) v += add;
      }
      vals[i] = v;
    }
    __syncthreads();
  }

  // dense results
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int v = v_begin + (u * kThreads + static_cast<int>(threadIdx.x)) * kN;
    if (whole(v)) {
      float f[kN];
      Vec::unpack(z[u], f);
      if (kAligned) {
        if (c[u].x | c[u].y | c[u].z | c[u].w) {
          const uint32_t cw[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            const uint32_t w = (cw[e >> 1] >> (16 * (e & 1))) & 0xffffu;
            f[e] = apply_rules(r, f[e], static_cast<int>(w & 0x7fffu), w != 0);
          }
        }
      } else if (rec && bits[u]) {
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const uint32_t w = rec[v + e];
          f[e] = apply_rules(r, f[e], static_cast<int>(w & 0x7fffu), w != 0);
        }
      }
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (!((bits[u] >> e) & 1u)) f[e] = -INFINITY;
      *reinterpret_cast<uint4*>(out + v) = Vec::pack(f);
    } else if (!kAligned) {
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const int id = v + e;
        if (id < 0 || id >= V) continue;
        float f = -INFINITY;
        if ((bits[u] >> e) & 1u) {
          const uint32_t w = rec ? rec[id] : 0u;
          f = apply_rules(r, to_f32<T>(in[id]), static_cast<int>(w & 0x7fffu), w != 0);
        }
        out[id] = from_f32<T>(f);
      }
    }
  }
  if (n_special > 0) {
    __syncthreads();
    for (int i = threadIdx.x; i < n_special; i += kThreads) {
      const int id = ids[i];
      bool mine = id >= 0 && id >= v_begin && id < v_begin + kChunk;
      for (int q = 0; mine && q < i; ++q) mine = ids[q] != id;
      if (mine) out[id] = from_f32<T>(vals[i]);
    }
  }

  // a row whose mask allows nothing is reported (its logits are all -inf)
  if (mask && chunk == 0) {
    int any = 0;
    for (int w0 = 0; w0 < mask_words && !any; w0 += kThreads) {
      const int w = w0 + static_cast<int>(threadIdx.x);
      uint32_t m = w < mask_words ? mask[w] : 0u;
      if (w == mask_words - 1 && (V & 31)) m &= (1u << (V & 31)) - 1u;
      any = __syncthreads_or(m != 0u);
    }
    if (!any && threadIdx.x == 0) raise_status(a.dev_status, kDevNoToken);
  }
}

template <typename T>
uno_status logits_dispatch(const LogitsArgs& a, cudaStream_t s) {
  constexpr int kN = LogitVec<T>::kN;
  constexpr int kChunk = kThreads * kUnroll * kN;
  const bool aligned = a.V % 8 == 0;   // 16-byte rows of logits and record, whole bytes of mask
  const int chunks = aligned ? (a.V + kChunk - 1) / kChunk : (a.V + kN - 1 + kChunk - 1) / kChunk;
  const int64_t grid = static_cast<int64_t>(a.B) * a.R * chunks;
  if (grid > 0x7fffffffll) return set_error(UNO_ERR_UNSUPPORTED, "too many logit rows");
  const dim3 g(static_cast<unsigned>(grid)), t(kThreads);
  const cudaError_t e = aligned ? launch_kernel(logits_kernel<T, true>, g, t, 0, s, 1, a, chunks)
                                : launch_kernel(logits_kernel<T, false>, g, t, 0, s, 1, a, chunks);
  return e == cudaSuccess ? UNO_OK : cuda_error(e, "logits rules launch");
}

}  // namespace

uno_status logits_process_launch(const LogitsArgs& a, cudaStream_t s) {
  return a.dt == UNO_F32 ? logits_dispatch<float>(a, s) : logits_dispatch<__nv_bfloat16>(a, s);
}

uno_status token_counts_launch(uint16_t* counts, int32_t S, int32_t V, const int32_t* tokens, int32_t B,
                               int32_t T, const int32_t* lens, const int32_t* slots, bool prompt,
                               int32_t* dev_status, cudaStream_t s) {
  const long long total = static_cast<long long>(B) * T;
  const long long grid = (total + 255) / 256;
  if (grid > 0x7fffffffll) return set_error(UNO_ERR_UNSUPPORTED, "too many tokens");
  const cudaError_t e =
      launch_kernel(counts_add_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, 1, counts, S, V,
                    tokens, T, total, lens, slots, prompt ? 1 : 0, dev_status);
  return e == cudaSuccess ? UNO_OK : cuda_error(e, "token counts launch");
}

}  // namespace uno

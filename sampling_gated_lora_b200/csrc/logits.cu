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
constexpr int kUnroll = 2;
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

// One CTA per segment of a row.
// kAligned: rows start on 16-byte boundaries (of the logits, the record and,
// bitwise, the mask). Otherwise a row's 16-byte vectors start at row * V mod kN
// elements before its first id, the first and last are handled id by id, and
// record words and mask bits are gathered one by one.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(kThreads, 6)
    logits_kernel(const LogitsArgs a, int segments, int iters) {
  using Vec = LogitVec<T>;
  constexpr int kN = Vec::kN;
  constexpr int kStep = kThreads * kUnroll * kN;   // ids of one iteration
  __shared__ int32_t sp_id[kMaxSpecial];           // special ids in this segment, in any order,
  __shared__ int32_t sp_src[kMaxSpecial];          // their places in path + bias list,
  __shared__ float sp_val[kMaxSpecial];            // their biases, then their results
  __shared__ int sp_n;
  const long long row = blockIdx.x / segments;
  const int seg = static_cast<int>(blockIdx.x - row * segments);
  const int b = static_cast<int>(row / a.R), j = static_cast<int>(row - static_cast<long long>(b) * a.R);
  const int V = a.V;
  const T* in = static_cast<const T*>(a.logits) + row * V;
  T* out = static_cast<T*>(a.out) + row * V;
  const int lead = kAligned ? 0 : static_cast<int>((row * V) % kN);
  const int v_begin = seg * iters * kStep - lead;  // id of the segment's first vector element
  const int v_end = min(V, v_begin + iters * kStep);
  if (threadIdx.x == 0) sp_n = 0;
  pdl_wait();

  const int slot = a.slots ? a.slots[b] : b;
  const bool has_rec = a.counts && slot >= 0 && slot < a.S;
  if (a.counts && !has_rec && seg == 0 && threadIdx.x == 0) raise_status(a.dev_status, kDevBadIndex);
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
  auto vec_id = [&](int it, int u) {
    return v_begin + ((it * kUnroll + u) * kThreads + static_cast<int>(threadIdx.x)) * kN;
  };

  uint32_t bits[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) bits[u] = allowed(vec_id(0, u));

  // ids of the path and of the bias list that fall into this segment; their
  // results come from the original logits, so before anything is stored
  const int np = a.path ? (a.path_per_row ? a.P : min(j, a.P)) : 0;
  const int n_special = np + a.nb;
  int n_here = 0;
  if (n_special > 0) {
    const int32_t* path = a.path + (a.path_per_row ? row : b) * a.P;
    const size_t bias0 = static_cast<size_t>(b) * a.nb;
    __syncthreads();
    for (int i = threadIdx.x; i < n_special; i += kThreads) {
      const int id = i < np ? path[i] : a.bias_ids[bias0 + (i - np)];
      if (id < 0 || id >= V) {
        if (id != -1 && seg == 0) raise_status(a.dev_status, kDevBadIndex);
      } else if (id >= v_begin && id < v_end) {
        const int k = atomicAdd(&sp_n, 1);
        sp_id[k] = id;
        sp_src[k] = i;
        sp_val[k] = i < np ? 0.f : a.bias[bias0 + (i - np)];
      }
    }
    __syncthreads();
    n_here = sp_n;
    if (n_here > 0) {
      // the first of equal ids acts for all; equal biases add up in list order
      constexpr int kPer = (kMaxSpecial + kThreads - 1) / kThreads;
      float res[kPer];
      uint32_t skip = 0u;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int i = threadIdx.x + q * kThreads;
        res[q] = 0.f;
        if (i >= n_here) continue;
        const int id = sp_id[i], src = sp_src[i];
        const unsigned short w = rec ? rec[id] : 0;
        const float z = to_f32<T>(in[id]);
        const bool on = !mask || ((mask[id >> 5] >> (id & 31)) & 1u);
        int n = w & 0x7fff, first = src, biases = 0;
        float add = 0.f;
        for (int k = 0; k < n_here; ++k)
          if (sp_id[k] == id) {
            first = min(first, sp_src[k]);
            if (sp_src[k] < np) {
              ++n;
            } else {
              ++biases;
              add = sp_val[k];
            }
          }
        if (biases > 1) {
          add = 0.f;
          for (int m = 0, last = np - 1; m < biases; ++m) {
            int at = -1;
            for (int k = 0; k < n_here; ++k)
              if (sp_id[k] == id && sp_src[k] > last && (at < 0 || sp_src[k] < sp_src[at])) at = k;
            last = sp_src[at];
            add += sp_val[at];
          }
        }
        float v = apply_rules(r, z, n, n > 0 || (w & 0x8000u));
        if (biases) v += add;
        res[q] = on ? v : -INFINITY;
        if (first != src) skip |= 1u << q;
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int i = threadIdx.x + q * kThreads;
        if (i < n_here) sp_val[i] = res[q];
        if ((skip >> q) & 1u) sp_id[i] = -1;
      }
    }
  }

  for (int it = 0; it < iters; ++it) {
    if (vec_id(it, 0) - static_cast<int>(threadIdx.x) * kN >= V) break;   // uniform: the row has ended
    uint4 z[kUnroll], c[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = vec_id(it, u);
      z[u] = c[u] = make_uint4(0u, 0u, 0u, 0u);
      if (bits[u] && whole(v)) {
        z[u] = __ldcs(reinterpret_cast<const uint4*>(in + v));
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
    uint32_t now[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      now[u] = bits[u];
      if (it + 1 < iters) bits[u] = allowed(vec_id(it + 1, u));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = vec_id(it, u);
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
        } else if (rec && now[u]) {
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            const uint32_t w = rec[v + e];
            f[e] = apply_rules(r, f[e], static_cast<int>(w & 0x7fffu), w != 0);
          }
        }
#pragma unroll
        for (int e = 0; e < kN; ++e)
          if (!((now[u] >> e) & 1u)) f[e] = -INFINITY;
        __stcs(reinterpret_cast<uint4*>(out + v), Vec::pack(f));
      } else if (!kAligned) {
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const int id = v + e;
          if (id < 0 || id >= V) continue;
          float f = -INFINITY;
          if ((now[u] >> e) & 1u) {
            const uint32_t w = rec ? rec[id] : 0u;
            f = apply_rules(r, to_f32<T>(in[id]), static_cast<int>(w & 0x7fffu), w != 0);
          }
          out[id] = from_f32<T>(f);
        }
      }
    }
  }
  if (n_here > 0) {
    __syncthreads();
    for (int i = threadIdx.x; i < n_here; i += kThreads)
      if (sp_id[i] >= 0) out[sp_id[i]] = from_f32<T>(sp_val[i]);
  }

  // a row whose mask allows nothing is reported (its logits are all -inf)
  if (mask && seg == 0) {
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
  constexpr int kStep = kThreads * kUnroll * kN;
  const bool aligned = a.V % 8 == 0;   // 16-byte rows of logits and record, whole bytes of mask
  const int steps = (a.V + (aligned ? 0 : kN - 1) + kStep - 1) / kStep;
  // Long segments spread a CTA's fixed work (parameters, special ids) over more
  // ids; short ones fill the device when there are few rows.
  const int64_t rows = static_cast<int64_t>(a.B) * a.R, fill = 12 * device_sm_count();
  const int iters = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, rows * steps / fill)));
  const int segments = (steps + iters - 1) / iters;
  if (rows * segments > 0x7fffffffll) return set_error(UNO_ERR_UNSUPPORTED, "too many logit rows");
  const dim3 g(static_cast<unsigned>(rows * segments)), t(kThreads);
  const cudaError_t e = aligned ? launch_kernel(logits_kernel<T, true>, g, t, 0, s, 1, a, segments, iters)
                                : launch_kernel(logits_kernel<T, false>, g, t, 0, s, 1, a, segments, iters);
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

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
// Every logit is read and written once, the record and the mask once; a vector
// whose mask bits are all 0 needs no logits at all. At 256 x 9 rows of 151936, half
// of them with 5 % of the ids allowed, that moves 1.29 GB in 275 us, 0.72 of the
// copy rate (0.67 in a profile of 64 x 9 rows): instruction issue is the nearer
// bound (ALU pipe 0.67 busy; a denser mask or none takes the same time), so what
// follows counts instructions. Few ids have a record, a bias or a place on the path, so
// the dense pass only branches per 16-byte vector on "any record here", and
// the ids of the path and the bias list are recomputed from the original logits by
// single threads and overwrite the dense result. That warp is the bound of small
// vocabularies with long lists: an id that occurs twice in a segment's list makes
// each of its entries search the list (9 rows of 4096, bf16: 300 biases 15 us, with
// one repeat 95; 1024 biases 33 and 815).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace uno {

namespace {

constexpr int kThreads = 256;  // streaming threads
constexpr int kUnroll = 2;    // 16-byte vectors a thread has in flight
constexpr int kMaxIters = 8;  // iterations of a segment
constexpr int kCtas = 5;      // per SM
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

// n: emitted count; held: emitted or in the prompt.
// Float logits are divided by rho. bf16 ones are multiplied by its float
// reciprocal: off by 2^-24 relative more than the quotient (2^-22 for factors above
// 2^126), at most 2^-14 of the half step that rounding to bf16 may take, and a
// division a penalised id makes the dense pass half as long again (256 x 9 rows of
// 151936: 400 us against 288).
template <typename T>
struct Rules {
  float rho, inv_rho, freq, pres;
  __device__ __forceinline__ Rules(const LogitsArgs& a, int b) {
    rho = a.repetition ? a.repetition[b] : 1.f;
    inv_rho = 1.f / rho;
    freq = a.frequency ? a.frequency[b] : 0.f;
    pres = a.presence ? a.presence[b] : 0.f;
  }
  __device__ __forceinline__ float apply(float z, int n, bool held) const {
    if (held) {
      if (std::is_same<T, float>::value) z = z > 0.f ? z / rho : z * rho;
      else z *= z > 0.f ? inv_rho : rho;
    }
    if (n > 0) z = z - freq * static_cast<float>(n) - pres;
    return z;
  }
  __device__ __forceinline__ float apply(float z, uint32_t word) const {
    return apply(z, static_cast<int>(word & 0x7fffu), word != 0u);
  }
};

// 16 bytes of logits, kept packed. About one id in a hundred has a record, so
// nearly every warp meets one: only the pairs of ids with a non-zero record
// word are unpacked and computed (with every id computed, arithmetic instead of
// HBM was the bound).
template <typename T>
struct LogitVec;
template <>
struct LogitVec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ uint4 load_record(const unsigned short* p) {
    return *reinterpret_cast<const uint4*>(p);
  }
  static __device__ __forceinline__ uint32_t two(uint32_t z, uint32_t c, const Rules<__nv_bfloat16>& r) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(r.apply(bf16_lo(z), c & 0xffffu),
                                                   r.apply(bf16_hi(z), c >> 16));
    return *reinterpret_cast<const uint32_t*>(&h);   // an id without a record comes back as it was
  }
  // the first pair with a record each round: a warp whose lanes hold one such
  // pair each, wherever in the vector, takes one round instead of up to four
  static __device__ __forceinline__ void rules(uint4& z, uint4 c, const Rules<__nv_bfloat16>& r) {
    while (c.x | c.y | c.z | c.w) {
      const bool p0 = c.x != 0u, p1 = !p0 && c.y != 0u, p2 = !p0 && !p1 && c.z != 0u, p3 = !p0 && !p1 && !p2;
      const uint32_t v = two(p0 ? z.x : p1 ? z.y : p2 ? z.z : z.w, p0 ? c.x : p1 ? c.y : p2 ? c.z : c.w, r);
      if (p0) z.x = v, c.x = 0u;
      if (p1) z.y = v, c.y = 0u;
      if (p2) z.z = v, c.z = 0u;
      if (p3) z.w = v, c.w = 0u;
    }
  }
  // keep two ids by the sign bits of two bytes of w
  template <uint32_t kSelect>
  static __device__ __forceinline__ uint32_t forbid2(uint32_t z, uint32_t w) {
    uint32_t keep;   // prmt with bit 3 of a selector: eight copies of the byte's sign
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(keep) : "r"(w), "n"(kSelect));
    return (z & keep) | (0xff80ff80u & ~keep);
  }
  static __device__ __forceinline__ void forbid(uint4& z, uint32_t bits) {
    // four bits to the signs of four bytes: bit i times 2^(7 (i + 1)) is bit 8 i + 7,
    // and the four products do not meet
    const uint32_t lo = (bits & 15u) * 0x10204080u, hi = (bits >> 4) * 0x10204080u;
    z = make_uint4(forbid2<0x9988>(z.x, lo), forbid2<0xbbaa>(z.y, lo), forbid2<0x9988>(z.z, hi), forbid2<0xbbaa>(z.w, hi));
  }
};
template <>
struct LogitVec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ uint4 load_record(const unsigned short* p) {
    const uint2 h = *reinterpret_cast<const uint2*>(p);
    return make_uint4(h.x, h.y, 0u, 0u);
  }
  static __device__ __forceinline__ uint32_t one(uint32_t z, uint32_t w, const Rules<float>& r) {
    return w ? __float_as_uint(r.apply(__uint_as_float(z), w)) : z;
  }
  static __device__ __forceinline__ void rules(uint4& z, const uint4& c, const Rules<float>& r) {
    if (c.x) {
      z.x = one(z.x, c.x & 0xffffu, r);
      z.y = one(z.y, c.x >> 16, r);
    }
    if (c.y) {
      z.z = one(z.z, c.y & 0xffffu, r);
      z.w = one(z.w, c.y >> 16, r);
    }
  }
  static __device__ __forceinline__ void forbid(uint4& z, uint32_t bits) {
    const uint32_t inf = 0xff800000u;
    z = make_uint4(bits & 1u ? z.x : inf, bits & 2u ? z.y : inf, bits & 4u ? z.z : inf, bits & 8u ? z.w : inf);
  }
};

// One CTA per segment of a row: eight warps stream it, a ninth works out the
// special ids (path and bias list) meanwhile and overwrites their places when
// the stream has passed.
// kAligned: rows start on 16-byte boundaries (of the logits, the record and,
// bitwise, the mask). Otherwise a row's 16-byte vectors start at row * V mod kN
// elements before its first id, the first and last are handled id by id, and
// record words and mask bits are gathered one by one.
constexpr int kBarRead = 1, kBarStored = 2;   // named barriers of the CTA's nine warps

__device__ __forceinline__ void bar_arrive(int id) {
  asm volatile("barrier.arrive %0, %1;" ::"r"(id), "n"(kThreads + 32) : "memory");
}
__device__ __forceinline__ void bar_wait(int id) {
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "n"(kThreads + 32) : "memory");
}

template <typename T, bool kAligned>
__global__ void __launch_bounds__(kThreads + 32, kAligned ? kCtas : kCtas - 1)
    logits_kernel(const LogitsArgs a, int segments, int iters) {
  using Vec = LogitVec<T>;
  constexpr int kN = Vec::kN;
  constexpr int kStep = kThreads * kUnroll * kN;   // ids of one iteration
  __shared__ int32_t sp_id[kMaxSpecial];           // special ids in this segment, in list order
  __shared__ float sp_bias[kMaxSpecial], sp_res[kMaxSpecial];   // their biases and results
  __shared__ uint32_t seen[kMaxIters * kThreads * kUnroll * 8 / 32];   // ids of the segment met so far
  const long long row = blockIdx.x / segments;
  const int seg = static_cast<int>(blockIdx.x - row * segments);
  const int b = static_cast<int>(row / a.R), j = static_cast<int>(row - static_cast<long long>(b) * a.R);
  const int V = a.V;
  const T* in = static_cast<const T*>(a.logits) + row * V;
  T* out = static_cast<T*>(a.out) + row * V;
  const int lead = kAligned ? 0 : static_cast<int>((row * V) % kN);
  const int v_begin = seg * iters * kStep - lead;  // id of the segment's first vector element
  const int v_end = min(V, v_begin + iters * kStep);
  const int np = a.path ? (a.path_per_row ? a.P : min(j, a.P)) : 0;
  const int n_special = np + a.nb;
  pdl_wait();
  if (v_begin >= V) return;   // an unaligned row that ends before its last segment

  const int slot = a.slots ? a.slots[b] : b;
  const bool has_rec = a.counts && slot >= 0 && slot < a.S;
  const unsigned short* rec = has_rec ? a.counts + static_cast<size_t>(slot) * V : nullptr;
  const int mask_words = (V + 31) / 32;
  const uint32_t* mask = a.mask ? a.mask + row * mask_words : nullptr;
  const Rules<T> r(a, b);

  if (threadIdx.x >= kThreads) {
    // ------------------------------------------------------------ the ninth warp
    const int lane = threadIdx.x & 31;
    if (seg == 0) {
      if (a.counts && !has_rec && lane == 0) raise_status(a.dev_status, kDevBadIndex);
      if (mask) {   // a row whose mask allows nothing is reported (its logits are all -inf)
        bool any = false;
        for (int w0 = 0; w0 < mask_words && !any; w0 += 8 * 32) {
          uint32_t m = 0u;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int w = w0 + 32 * q + lane;
            const uint32_t x = w < mask_words ? mask[w] : 0u;
            m |= w == mask_words - 1 && (V & 31) ? x & ((1u << (V & 31)) - 1u) : x;
          }
          any = __any_sync(0xffffffffu, m != 0u);
        }
        if (!any && lane == 0) raise_status(a.dev_status, kDevNoToken);
      }
    }
    if (n_special == 0) return;
    const int words = (v_end - v_begin + 31) / 32;
    for (int i = lane; i < words; i += 32) seen[i] = 0u;
    __syncwarp();
    const int32_t* path = a.path + (a.path_per_row ? row : b) * a.P;
    const size_t bias0 = static_cast<size_t>(b) * a.nb;
    int n = 0, n_path = 0;
    bool twice = false;   // some id occurs more than once in the list
    for (int i0 = 0; i0 < n_special; i0 += 32) {
      const int i = i0 + lane;
      int id = -1;
      float bias = 0.f;
      if (i < np) {
        id = path[i];
      } else if (i < n_special) {
        id = a.bias_ids[bias0 + (i - np)];
        bias = a.bias[bias0 + (i - np)];
      }
      if (id < -1 || id >= V) {
        if (seg == 0) raise_status(a.dev_status, kDevBadIndex);
        id = -1;
      }
      const bool here = id >= 0 && id >= v_begin && id < v_end;
      const uint32_t m = __ballot_sync(0xffffffffu, here);
      if (here) {
        const int k = n + __popc(m & ((1u << lane) - 1u)), o = id - v_begin;
        sp_id[k] = id;
        sp_bias[k] = bias;
        if (atomicOr(&seen[o >> 5], 1u << (o & 31)) >> (o & 31) & 1u) twice = true;
      }
      n_path += __popc(m & __ballot_sync(0xffffffffu, i < np));
      n += __popc(m);
    }
    twice = __any_sync(0xffffffffu, twice);
    __syncwarp();
    // results from the original logits, before the stream may store (out may be
    // logits): the first entry of an id acts for all, biases add up in list order
    static_assert((kMaxSpecial + 31) / 32 <= 64, "one bit of `acts` a round");
    uint64_t acts = 0ull;
    for (int k0 = 0, q = 0; k0 < n; k0 += 32, ++q) {
      const int k = k0 + lane;
      if (k < n) {
        const int id = sp_id[k];
        const uint32_t w = rec ? rec[id] : 0u;
        const float z = to_f32<T>(in[id]);
        const bool on = !mask || ((mask[id >> 5] >> (id & 31)) & 1u);
        int cnt = static_cast<int>(w & 0x7fffu), first = k;
        float add = 0.f;
        if (twice) {
          for (int e = 0; e < n; ++e)
            if (sp_id[e] == id) {
              first = min(first, e);
              if (e < n_path) ++cnt;
              else add += sp_bias[e];
            }
        } else {
          cnt += k < n_path;
          add = sp_bias[k];
        }
        if (first == k) acts |= 1ull << q;
        const float v = r.apply(z, cnt, cnt > 0 || (w & 0x8000u));
        sp_res[k] = on ? v + add : -INFINITY;
      }
    }
    if (a.logits == a.out) bar_arrive(kBarRead);
    bar_wait(kBarStored);
    for (int k = lane, q = 0; k < n; k += 32, ++q)
      if ((acts >> q) & 1ull) out[sp_id[k]] = from_f32<T>(sp_res[k]);
    return;
  }

  // -------------------------------------------------------------- the stream
  // mask bits of the vector's ids (bit e: id v + e); ids outside the row read 0
  auto allowed = [&](int v) -> uint32_t {
    constexpr uint32_t kAll = (1u << kN) - 1u;
    if (kAligned) {
      if (v >= V) return 0u;
      if (!mask) return kAll;
      const uint32_t byte = reinterpret_cast<const uint8_t*>(mask)[static_cast<uint32_t>(v) >> 3];
      return kN == 8 ? byte : (byte >> (v & 7)) & kAll;
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

  for (int it = 0; it < iters; ++it) {
    if (vec_id(it, 0) - static_cast<int>(threadIdx.x) * kN >= V) break;   // uniform: the row has ended
    // logits and record words (vectors that allow nothing are not read), the
    // next iteration's mask bits
    uint4 z[kUnroll], c[kUnroll];
    uint32_t now[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = vec_id(it, u);
      now[u] = bits[u];
      z[u] = c[u] = make_uint4(0u, 0u, 0u, 0u);
      if (now[u] && whole(v)) {
        z[u] = __ldcs(reinterpret_cast<const uint4*>(in + v));
        if (kAligned && rec) c[u] = Vec::load_record(rec + v);
      }
    }
    if (it + 1 < iters) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) bits[u] = allowed(vec_id(it + 1, u));
    }
    if (it == 0 && n_special > 0 && a.logits == a.out) bar_wait(kBarRead);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = vec_id(it, u);
      if (whole(v)) {
        if (kAligned) {
          if (c[u].x | c[u].y | c[u].z | c[u].w) Vec::rules(z[u], c[u], r);
        } else if (rec && now[u]) {
          uint32_t w[4] = {};
#pragma unroll
          for (int e = 0; e < kN; ++e) w[e >> 1] |= static_cast<uint32_t>(rec[v + e]) << (16 * (e & 1));
          Vec::rules(z[u], make_uint4(w[0], w[1], w[2], w[3]), r);
        }
        if (now[u] != (1u << kN) - 1u) Vec::forbid(z[u], now[u]);
        *reinterpret_cast<uint4*>(out + v) = z[u];
      } else if (!kAligned) {
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const int id = v + e;
          if (id < 0 || id >= V) continue;
          float f = -INFINITY;
          if ((now[u] >> e) & 1u) {
            const uint32_t w = rec ? rec[id] : 0u;
            f = r.apply(to_f32<T>(in[id]), w);
          }
          out[id] = from_f32<T>(f);
        }
      }
    }
  }
  if (n_special > 0) bar_arrive(kBarStored);
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
  const int iters = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxIters, rows * steps / fill)));
  const int segments = (steps + iters - 1) / iters;
  if (rows * segments > 0x7fffffffll) return set_error(UNO_ERR_UNSUPPORTED, "too many logit rows");
  const dim3 g(static_cast<unsigned>(rows * segments)), t(kThreads + 32);
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

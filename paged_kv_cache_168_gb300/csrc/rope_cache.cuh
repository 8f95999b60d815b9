// rope_cache.cuh -- rotary positions on q and k, with or without a norm of each of
// their vectors before it, fused with the cache write; instantiated by rope_cache.cu
// and norm_rope_cache.cu.
//
// A pair (x1, x2) at angle position * frequency becomes (x1 c - x2 s, x2 c +
// x1 s); each pair's position comes from its own axis (time, height, width).
// Every product and sum is rounded to fp32 and never contracted, so a result is
// a pure function of the input bits, like the rest of the cache operations.
//
// Bound: HBM.  A token reads q, k and v and writes q, K and V once; its cosines
// and sines (rotary_dim floats) come from L2, once per token, into shared
// memory, where all heads read them.  A unit is two 16-byte pieces of one head
// vector that hold both halves of their pairs -- pieces u and u + rotary_dim / 16
// when halves pair up, 2u and 2u + 1 when neighbours do -- so a vector is D / 16
// units on neighbouring lanes, and a vector's amax (8-bit caches) or its sum of
// squares (norms) is three shuffles.
#pragma once

#include <float.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

// The two pieces (16 bytes = 8 dims each) of unit u of a head vector.
template <bool kPairs>
__device__ __forceinline__ void unit_pieces(int u, int rot, int& a, int& b, bool& turned) {
  const int half = rot / 16;
  turned = u < half;
  if (kPairs || !turned) {
    a = 2 * u;
    b = 2 * u + 1;
  } else {
    a = u;
    b = u + half;
  }
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Elem<T>::to_float2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(Elem<T>::pack2(x[0], x[1]), Elem<T>::pack2(x[2], x[3]), Elem<T>::pack2(x[4], x[5]),
                    Elem<T>::pack2(x[6], x[7]));
}

// In shared memory a unit's values lie four by four, the units' first fours together, then their second ones: what the
// lanes of a vector read at once is contiguous and no bank is asked twice.
__device__ __forceinline__ int shared_place(int i, int units) { return (i / 4 % 2 * units + i / 8) * 4 + i % 4; }

// x holds the unit's 16 values (piece a, then piece b); cs the token's cosines, then sines (shared_place).
template <bool kPairs>
__device__ __forceinline__ void rotate(float (&x)[16], const float* cs, int u, int units) {
  float c[8], s[8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float4 v = reinterpret_cast<const float4*>(cs)[k * units + u];
    const float4 w = reinterpret_cast<const float4*>(cs)[(k + 2) * units + u];
    c[4 * k] = v.x, c[4 * k + 1] = v.y, c[4 * k + 2] = v.z, c[4 * k + 3] = v.w;
    s[4 * k] = w.x, s[4 * k + 1] = w.y, s[4 * k + 2] = w.z, s[4 * k + 3] = w.w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = kPairs ? 2 * i : i, b = kPairs ? 2 * i + 1 : i + 8;
    const float x1 = x[a], x2 = x[b];
    x[a] = __fsub_rn(__fmul_rn(x1, c[i]), __fmul_rn(x2, s[i]));
    x[b] = __fadd_rn(__fmul_rn(x2, c[i]), __fmul_rn(x1, s[i]));
  }
}

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pack2f(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2f(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2f(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2f(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// x becomes x / sqrt(mean of the vector's squares + eps) w; the vector's D / 16 units are neighbouring lanes.
// False where the vector is not finite.
template <int D>
__device__ __forceinline__ bool normalise(float (&x)[16], const float* weight, int u, float eps, float small) {
  constexpr int kUnits = D / 16;
  const unsigned lanes = ((1u << kUnits) - 1u) << (threadIdx.x & 31 & ~(kUnits - 1));
  auto squares = [&]() {
    uint64_t s[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint64_t v = pack2f(x[2 * k], x[2 * k + 1]);
      s[k & 1] = fma2f(v, v, s[k & 1]);
    }
    float a, b, c, d;
    unpack2f(s[0], a, b);
    unpack2f(s[1], c, d);
    float sum = (a + b) + (c + d);
#pragma unroll
    for (int o = kUnits / 2; o; o >>= 1) sum += __shfl_xor_sync(lanes, sum, o);
    return sum;
  };
  float ss = squares();
  // bf16 reaches 3e38, whose squares do not fit: such a vector is made smaller first,
  // and eps with it (one that holds an infinity stays infinite, r = 0).  In the same way
  // one whose squares are too small is made larger, unless they are nothing beside eps.
  // (`small`: below which they are; one comparison with both ends, in the order of the bits, which takes NaN along.)
  if (__builtin_expect(__float_as_uint(ss) - __float_as_uint(small) >= 0x7f800000u - __float_as_uint(small), 0)) {
    const float by = ss == INFINITY ? 0x1p-80f : 0x1p80f;
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] *= by;
    ss = squares();
    eps = eps * by * by;
  }
  const float r = rsqrtf(fmaf(ss, 1.f / D, eps));
  const uint64_t r2 = pack2f(r, r);
  // (the weights of piece a, then of piece b, each as shared_place has them)
  const float4* w4 = reinterpret_cast<const float4*>(weight);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 v = w4[k * kUnits + u];
    unpack2f(mul2f(pack2f(x[4 * k], x[4 * k + 1]), mul2f(r2, pack2f(v.x, v.y))), x[4 * k], x[4 * k + 1]);
    unpack2f(mul2f(pack2f(x[4 * k + 2], x[4 * k + 3]), mul2f(r2, pack2f(v.z, v.w))), x[4 * k + 2], x[4 * k + 3]);
  }
  return r > 0.f;
}

// A round of a CTA is kTokens tokens: their cosines and sines go to shared memory,
// then every thread takes kDeep units at a time, all their loads before any
// arithmetic.  32768 tokens of 32 + 8 heads in bf16, three axes: 138 us, 5.8 TB/s (one
// token a CTA and round, two barriers for 1.5 units a thread: 185 us).  5001 tokens of
// 32 + 32 heads into an 8-bit cache: 50 us, 4.1 TB/s; 132-byte vectors go to random
// places there.
//
// kNorm: q and k vectors become x / sqrt(mean(x^2) + eps) (weight + offset) first, in
// fp32 and not rounded before the rotation; the weights wait in shared memory.  32768
// tokens of 32 + 8 heads: 165 us, 4.9 TB/s.  Nothing is full there (issue slots 58%,
// DRAM 60%): a round's slots, positions and cosines wait for one another before its
// first vector is loaded.  Three CTAs an SM with more registers 205, five or six with
// fewer 174 to 197.  Into an 8-bit cache 192 us.
template <typename T, int D, bool kPairs, bool kI8, bool kNorm, int kTokens>
__global__ void __launch_bounds__(kThreads, 4) rope_cache_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kUnits = D / 16;                     // units per head vector
  constexpr int kDeep = kNorm ? 2 : 3;               // units a thread has in flight
  __shared__ __align__(16) float cs[kTokens][D];
  __shared__ int64_t slots[kTokens];                 // where the token goes; -1: nowhere
  __shared__ int skip[kTokens];                      // its position is out of range
  __shared__ __align__(16) float weight[kNorm ? 2 : 1][kNorm ? D : 4];      // of q, of k
  const int rot = p.rotary_dim, half_dims = rot / 2;
  const int hq = p.num_q_heads, hkv = p.num_kv_heads, heads = hq + 2 * hkv;
  const int64_t nslots = (int64_t)p.num_blocks * p.block_size;
  const int shift = __ffs(p.block_size) - 1;
  const Layout L{p.block_size, D, hkv};
  const I8Layout L8{p.block_size, hkv};
  const int u = threadIdx.x % kUnits;                // kThreads is a multiple of kUnits
  int a, b;
  bool turns;
  unit_pieces<kPairs>(u, rot, a, b, turns);
  if constexpr (kNorm) {                             // (seen after the first round's barriers)
    static_assert(kThreads >= 2 * D, "a weight a thread");
    if (threadIdx.x < 2 * D) {
      const T* w = static_cast<const T*>(threadIdx.x < D ? p.q_weight : p.k_weight);
      // value i of the unit's two pieces
      const int at = threadIdx.x % D, unit = at / 16, i = at % 16;
      int pa, pb;
      bool unused;
      unit_pieces<kPairs>(unit, rot, pa, pb, unused);
      const int d = (i < 8 ? pa : pb) * 8 + i % 8;
      weight[threadIdx.x / D][(i / 8) * (D / 2) + shared_place(unit * 8 + i % 8, kUnits)] =
          w ? (float)w[d] + p.weight_offset : 1.f;
    }
  }
  for (int tok0 = blockIdx.x * kTokens; tok0 < p.num_tokens; tok0 += gridDim.x * kTokens) {
    const int count = min(kTokens, p.num_tokens - tok0);
    __syncthreads();                                 // the round before has been used
    if (threadIdx.x < count) {
      const int64_t slot = p.slot_mapping[tok0 + threadIdx.x];
      const bool bad = slot != -1 && (slot < 0 || slot >= nslots);
      slots[threadIdx.x] = bad ? -1 : slot;
      if (bad) report(p.dev_err, PA_DEVERR_SLOT);
      skip[threadIdx.x] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < count * rot; i += kThreads) {
      const int k = i / rot, d = i - k * rot;
      const int pos = p.positions[p.pair_axis[d < half_dims ? d : d - half_dims] * p.axis_stride + tok0 + k];
      const bool fine = pos >= 0 && pos < p.max_position;
      cs[k][d < half_dims ? shared_place(d, rot / 16) : half_dims + shared_place(d - half_dims, rot / 16)] =
          fine ? p.cos_sin[(int64_t)pos * rot + d] : 0.f;
      if (!fine) skip[k] = 1;
    }
    __syncthreads();
    if (threadIdx.x < count && skip[threadIdx.x]) {
      slots[threadIdx.x] = -1;
      report(p.dev_err, PA_DEVERR_POSITION);
    }
    __syncthreads();
    const int vectors = count * heads;
    for (int v0 = threadIdx.x / kUnits; v0 < vectors; v0 += kDeep * (kThreads / kUnits)) {
      uint4 va[kDeep], vb[kDeep];
      int tok[kDeep], head[kDeep];
#pragma unroll
      for (int e = 0; e < kDeep; ++e) {
        const int v = v0 + e * (kThreads / kUnits);
        tok[e] = 0;                                  // v / heads, without a division (162 us instead of 170)
#pragma unroll
        for (int k = 1; k < kTokens; ++k) tok[e] += v >= k * heads;
        head[e] = v - tok[e] * heads;
        if (v >= vectors) tok[e] = -1;
        else if (head[e] >= hq && slots[tok[e]] == -1) tok[e] = -1;   // K and V that are not stored
        if (tok[e] < 0) continue;
        const int64_t t = tok0 + tok[e];
        const T* src = head[e] < hq ? static_cast<const T*>(p.q) + t * p.q_stride + (int64_t)head[e] * D
                       : head[e] < hq + hkv
                           ? static_cast<const T*>(p.key) + t * p.key_stride + (int64_t)(head[e] - hq) * D
                           : static_cast<const T*>(p.value) + t * p.value_stride + (int64_t)(head[e] - hq - hkv) * D;
        va[e] = *reinterpret_cast<const uint4*>(src + a * 8);
        vb[e] = *reinterpret_cast<const uint4*>(src + b * 8);
      }
#pragma unroll
      for (int e = 0; e < kDeep; ++e) {
        if (tok[e] < 0) continue;                    // the same for all units of a vector
        const int part = head[e] < hq ? 0 : head[e] < hq + hkv ? 1 : 2;      // q, k, v
        const bool turned = turns && part != 2;
        if (turned || (kI8 && part != 0) || (kNorm && part != 2)) {
          float x[16];
          unpack8<T>(va[e], x);
          unpack8<T>(vb[e], x + 8);
          bool finite = true;
          if (kNorm && part != 2) finite = normalise<D>(x, weight[kNorm ? part : 0], u, p.eps, p.small_squares);
          if (turned) rotate<kPairs>(x, cs[tok[e]], u, rot / 16);
          if (kI8 && part != 0) {
            const int h = head[e] - (part == 1 ? hq : hq + hkv);
            const int64_t slot = slots[tok[e]], block = slot >> shift;
            const int t = (int)(slot & (p.block_size - 1));
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(x[k]));
            const unsigned lanes = ((1u << kUnits) - 1u) << (threadIdx.x & 31 & ~(kUnits - 1));
#pragma unroll
            for (int o = kUnits / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, o));
            uint32_t code[4] = {0, 0, 0, 0};
            float scale = 0.f;
            if (amax > 0.f) {
              // x * inv is at most 127 (1 + 2^-22) in size: added to 1.5 * 2^23 it is
              // rounded half to even into the sum's low byte
              const float inv = fminf(__fmul_rn(127.f, __fdiv_rn(1.f, amax)), FLT_MAX);
              uint32_t r[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(__fadd_rn(__fmul_rn(x[k], inv), 12582912.f));
              // A product is NaN where x is, or where x is infinite (inv is 0 then): code 0.  The
              // sums' exponent field is 150, so bit 26 is set in a NaN alone.
              uint32_t any = 0;
#pragma unroll
              for (int k = 0; k < 16; ++k) any |= r[k];
              if (__builtin_expect(any & 0x04000000u, 0)) {
#pragma unroll
                for (int k = 0; k < 16; ++k) r[k] = r[k] & 0x04000000u ? 0u : r[k];
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
                code[k] = __byte_perm(__byte_perm(r[4 * k], r[4 * k + 1], 0x0040), __byte_perm(r[4 * k + 2], r[4 * k + 3], 0x0040), 0x5410);
              scale = __fmul_rn(amax, 1.f / 127.f);
            }
            // (a norm leaves such a vector 0 and NaN, whose codes are all 0: the scale says what it is)
            if (kNorm && !finite) scale = __int_as_float(0x7fffffff);
            uint8_t* at = p.cache + L8.chunk(block, h) + ((part - 1) * p.block_size + t) * 128;
            *reinterpret_cast<uint2*>(at + ((((a >> 1) ^ (t & 7)) << 4) | (a & 1) << 3)) = make_uint2(code[0], code[1]);
            *reinterpret_cast<uint2*>(at + ((((b >> 1) ^ (t & 7)) << 4) | (b & 1) << 3)) = make_uint2(code[2], code[3]);
            if (u == 0) *reinterpret_cast<float*>(p.cache + L8.scale(block, h, part - 1, t)) = scale;
            continue;
          }
          va[e] = pack8<T>(x);
          vb[e] = pack8<T>(x + 8);
        }
        if (part == 0) {
          T* dst = static_cast<T*>(p.q_out) + (tok0 + tok[e]) * p.q_out_stride + (int64_t)head[e] * D;
          if (skip[tok[e]]) va[e] = vb[e] = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(dst + a * 8) = va[e];
          *reinterpret_cast<uint4*>(dst + b * 8) = vb[e];
        } else {
          const int h = head[e] - (part == 1 ? hq : hq + hkv);
          const int64_t slot = slots[tok[e]], block = slot >> shift;
          const int t = (int)(slot & (p.block_size - 1));
          *reinterpret_cast<uint4*>(p.cache + L.offset(block, h, part - 1, t, a * 8) * 2) = va[e];
          *reinterpret_cast<uint4*>(p.cache + L.offset(block, h, part - 1, t, b * 8) * 2) = vb[e];
        }
      }
    }
  }
}

template <typename T, int D, bool kI8, bool kNorm, int kTokens>
void launch_rounds(const RopeParams& p, int sms, cudaStream_t stream) {
  const int rounds = (p.num_tokens + kTokens - 1) / kTokens;
  const unsigned grid = (unsigned)(rounds < sms * 8 ? rounds : sms * 8);
  if (p.interleaved)
    rope_cache_kernel<T, D, true, kI8, kNorm, kTokens><<<grid, kThreads, 0, stream>>>(p);
  else
    rope_cache_kernel<T, D, false, kI8, kNorm, kTokens><<<grid, kThreads, 0, stream>>>(p);
}

template <typename T, int D, bool kI8, bool kNorm>
cudaError_t launch_pairs(const RopeParams& p, int sms, cudaStream_t stream) {
  // One token a CTA as long as all CTAs run at once (four an SM), for latency: 256
  // tokens of 32 + 8 heads 3.8 us back to back in a graph against 5.9 with four a
  // CTA, 608 (on 152 SMs) 4.8 against 6.0; but 2048 12.0 against 10.9, 4096 26.6 against 21.8.
  if (p.num_tokens <= sms * 4)
    launch_rounds<T, D, kI8, kNorm, 1>(p, sms, stream);
  else
    launch_rounds<T, D, kI8, kNorm, 4>(p, sms, stream);
  return cudaGetLastError();
}

template <bool kNorm, typename T>
cudaError_t launch_typed(const RopeParams& p, bool i8, int sms, cudaStream_t stream) {
  if (i8) return launch_pairs<T, 128, true, kNorm>(p, sms, stream);
  return p.head_size == 128 ? launch_pairs<T, 128, false, kNorm>(p, sms, stream)
                            : launch_pairs<T, 64, false, kNorm>(p, sms, stream);
}

template <bool kNorm>
cudaError_t launch(const RopeParams& p, int act_dtype, bool i8, int sms, cudaStream_t stream) {
  return act_dtype == PA_F16 ? launch_typed<kNorm, __half>(p, i8, sms, stream)
                             : launch_typed<kNorm, __nv_bfloat16>(p, i8, sms, stream);
}

}  // namespace
}  // namespace pkv

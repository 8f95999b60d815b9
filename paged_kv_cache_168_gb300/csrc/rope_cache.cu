// rope_cache.cu -- rotary positions on q and k, fused with the cache write.
//
// A pair (x1, x2) at angle position * frequency becomes (x1 c - x2 s, x2 c +
// x1 s); each pair's position comes from its own axis (time, height, width).
// Every product and sum is rounded to fp32 and never contracted, so a result is
// a pure function of the input bits, like the rest of the cache operations.
//
// Bound: HBM.  A token reads q, k and v and writes q, K and V once; its cosines
// and sines (rotary_dim floats) come from L2, once per token, into shared
// memory, where all heads read them.  One CTA per token (grid-stride): a unit
// is two 16-byte pieces of one head vector that hold both halves of their
// pairs -- pieces u and u + rotary_dim / 16 when halves pair up, 2u and 2u + 1
// when neighbours do -- so a vector is D / 16 units on neighbouring lanes and a
// vector's amax (8-bit caches) is three shuffles.
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

// x holds the unit's 16 values (piece a, then piece b); cs the token's cosines and sines.
template <bool kPairs>
__device__ __forceinline__ void rotate(float (&x)[16], const float* cs, int u, int half_dims) {
  const float* c = cs + u * 8;
  const float* s = cs + half_dims + u * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = kPairs ? 2 * i : i, b = kPairs ? 2 * i + 1 : i + 8;
    const float x1 = x[a], x2 = x[b];
    x[a] = __fsub_rn(__fmul_rn(x1, c[i]), __fmul_rn(x2, s[i]));
    x[b] = __fadd_rn(__fmul_rn(x2, c[i]), __fmul_rn(x1, s[i]));
  }
}

template <typename T, int D, bool kPairs, bool kI8>
__global__ void __launch_bounds__(kThreads) rope_cache_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kUnits = D / 16;                     // units per head vector
  __shared__ __align__(16) float cs[2][D];
  __shared__ int bad_pos[2];
  const int rot = p.rotary_dim, half_dims = rot / 2;
  const int hq = p.num_q_heads, hkv = p.num_kv_heads;
  const int units = (hq + 2 * hkv) * kUnits;
  const int64_t nslots = (int64_t)p.num_blocks * p.block_size;
  const Layout L{p.block_size, D, hkv};
  const I8Layout L8{p.block_size, hkv};
  int buf = 0;
  for (int tok = blockIdx.x; tok < p.num_tokens; tok += gridDim.x, buf ^= 1) {
    const int64_t slot = p.slot_mapping[tok];
    if (threadIdx.x == 0) bad_pos[buf] = 0;
    __syncthreads();
    if (threadIdx.x < rot) {
      const int pair = threadIdx.x < half_dims ? threadIdx.x : threadIdx.x - half_dims;
      const int pos = p.positions[p.pair_axis[pair] * p.axis_stride + tok];
      const bool fine = pos >= 0 && pos < p.max_position;
      cs[buf][threadIdx.x] = fine ? p.cos_sin[(int64_t)pos * rot + threadIdx.x] : 0.f;
      if (!fine) bad_pos[buf] = 1;
    }
    __syncthreads();
    const bool skip = bad_pos[buf] != 0;
    bool store = slot != -1 && !skip;
    if (store && (slot < 0 || slot >= nslots)) {
      store = false;
      if (threadIdx.x == 0) report(p.dev_err, PA_DEVERR_SLOT);
    }
    if (skip && threadIdx.x == 0) report(p.dev_err, PA_DEVERR_POSITION);
    const int64_t block = store ? slot / p.block_size : 0;
    const int t = store ? (int)(slot - block * p.block_size) : 0;
    for (int i = threadIdx.x; i < units; i += kThreads) {
      const int head = i / kUnits, u = i % kUnits;
      const int part = head < hq ? 0 : head < hq + hkv ? 1 : 2;   // q, k, v
      const int h = head - (part == 0 ? 0 : part == 1 ? hq : hq + hkv);
      if (part != 0 && !store) continue;             // the same for all units of a vector
      int a, b;
      bool turned;
      unit_pieces<kPairs>(u, rot, a, b, turned);
      const T* src = part == 0   ? static_cast<const T*>(p.q) + tok * p.q_stride
                     : part == 1 ? static_cast<const T*>(p.key) + tok * p.key_stride
                                 : static_cast<const T*>(p.value) + tok * p.value_stride;
      src += (int64_t)h * D;
      uint4 va = *reinterpret_cast<const uint4*>(src + a * 8), vb = *reinterpret_cast<const uint4*>(src + b * 8);
      turned = turned && part != 2;
      if (kI8 && part != 0) {
        float x[16];
        unpack8<T>(va, x);
        unpack8<T>(vb, x + 8);
        if (turned) rotate<kPairs>(x, cs[buf], u, half_dims);
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
        const unsigned lanes = ((1u << kUnits) - 1u) << (threadIdx.x & 31 & ~(kUnits - 1));
#pragma unroll
        for (int o = kUnits / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, o));
        uint32_t code[4] = {0, 0, 0, 0};
        float scale = 0.f;
        if (amax > 0.f) {
          const float inv = __fmul_rn(127.f, __fdiv_rn(1.f, amax));
#pragma unroll
          for (int e = 0; e < 16; ++e)
            code[e >> 2] |= (uint32_t)(min(127, max(-127, __float2int_rn(__fmul_rn(x[e], inv)))) & 0xff) << (8 * (e & 3));
          scale = __fmul_rn(amax, 1.f / 127.f);
        }
        *reinterpret_cast<uint2*>(p.cache + L8.code(block, h, part - 1, t, a * 8)) = make_uint2(code[0], code[1]);
        *reinterpret_cast<uint2*>(p.cache + L8.code(block, h, part - 1, t, b * 8)) = make_uint2(code[2], code[3]);
        if (u == 0) *reinterpret_cast<float*>(p.cache + L8.scale(block, h, part - 1, t)) = scale;
        continue;
      }
      if (turned) {
        float x[16];
        unpack8<T>(va, x);
        unpack8<T>(vb, x + 8);
        rotate<kPairs>(x, cs[buf], u, half_dims);
        va = pack8<T>(x);
        vb = pack8<T>(x + 8);
      }
      if (part == 0) {
        T* dst = static_cast<T*>(p.q_out) + tok * p.q_out_stride + (int64_t)h * D;
        if (skip) va = vb = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(dst + a * 8) = va;
        *reinterpret_cast<uint4*>(dst + b * 8) = vb;
      } else {
        *reinterpret_cast<uint4*>(p.cache + L.offset(block, h, part - 1, t, a * 8) * 2) = va;
        *reinterpret_cast<uint4*>(p.cache + L.offset(block, h, part - 1, t, b * 8) * 2) = vb;
      }
    }
  }
}

template <typename T, int D, bool kI8>
cudaError_t launch_pairs(const RopeParams& p, cudaStream_t stream) {
  const unsigned grid = (unsigned)(p.num_tokens < 152 * 8 ? p.num_tokens : 152 * 8);
  if (p.interleaved)
    rope_cache_kernel<T, D, true, kI8><<<grid, kThreads, 0, stream>>>(p);
  else
    rope_cache_kernel<T, D, false, kI8><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const RopeParams& p, bool i8, cudaStream_t stream) {
  if (i8) return launch_pairs<T, 128, true>(p, stream);
  return p.head_size == 128 ? launch_pairs<T, 128, false>(p, stream) : launch_pairs<T, 64, false>(p, stream);
}

}  // namespace

cudaError_t launch_rope_cache(const RopeParams& p, int act_dtype, bool i8, cudaStream_t stream) {
  return act_dtype == PA_F16 ? launch_typed<__half>(p, i8, stream) : launch_typed<__nv_bfloat16>(p, i8, stream);
}

}  // namespace pkv

// extend.cu -- attention of a chunk of new tokens per sequence over any paged
// cache: one warp per (token, query head), online softmax over the attended
// positions, fp32 throughout.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace pkv {
namespace {

template <typename T, int D, bool kI8>
__global__ void __launch_bounds__(128) extend_kernel(const __grid_constant__ ExtendParams p) {
  constexpr int kDims = D / 32;                      // dims per lane, consecutive
  const int lane = threadIdx.x & 31;
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int tok = (int)(w / p.num_q_heads), h = (int)(w % p.num_q_heads);
  if (tok >= p.num_tokens || tok >= p.query_start_loc[p.num_seqs]) return;
  int lo = 0, hi = p.num_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.query_start_loc[mid] <= tok) lo = mid; else hi = mid;
  }
  const int s = lo, bs = p.block_size, first = p.query_start_loc[s], q_len = p.query_start_loc[s + 1] - first;
  const int ctx = p.context_lens[s], kvh = h / p.group;
  if (first < 0 || q_len <= 0 || (int64_t)first + q_len > p.num_tokens) {
    if (lane == 0) report(p.dev_err, PA_DEVERR_CONTEXT);
    return;
  }
  bool ok = q_len <= p.max_query_len && q_len <= ctx &&
            (p.ring_blocks > 0 || (int64_t)ctx <= (int64_t)p.bt_stride * bs);
  if (!ok && lane == 0) report(p.dev_err, PA_DEVERR_CONTEXT);
  const int pos = ctx - q_len + (tok - first);
  int t0 = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  if (p.ring_blocks > 0) t0 = max(t0, ((ctx - 1) / bs - p.ring_blocks + 1) * bs);
  const T* q = static_cast<const T*>(p.q) + tok * p.q_token_stride + (int64_t)h * D + lane * kDims;
  float x[kDims], o[kDims], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int d = 0; d < kDims; ++d) {
    x[d] = (float)q[d] * p.scale_log2;
    o[d] = 0.f;
  }
  const Layout L{bs, D, p.num_kv_heads};
  const I8Layout L8{bs, p.num_kv_heads};
  for (int t = t0; ok && t <= pos; ++t) {
    const int b = p.block_tables[(int64_t)s * p.bt_stride + table_index(t / bs, p.ring_blocks)];
    if (b < 0 || b >= p.num_blocks) {
      if (lane == 0) report(p.dev_err, PA_DEVERR_BLOCK_ID);
      ok = false;
      break;
    }
    float k[kDims], v[kDims];
#pragma unroll
    for (int d = 0; d < kDims; ++d) {
      if (kI8) {
        k[d] = (float)reinterpret_cast<const int8_t*>(p.cache)[L8.code(b, kvh, 0, t % bs, lane * kDims + d)] *
               *reinterpret_cast<const float*>(p.cache + L8.scale(b, kvh, 0, t % bs));
        v[d] = (float)reinterpret_cast<const int8_t*>(p.cache)[L8.code(b, kvh, 1, t % bs, lane * kDims + d)] *
               *reinterpret_cast<const float*>(p.cache + L8.scale(b, kvh, 1, t % bs));
      } else {
        k[d] = (float)reinterpret_cast<const T*>(p.cache)[L.offset(b, kvh, 0, t % bs, lane * kDims + d)];
        v[d] = (float)reinterpret_cast<const T*>(p.cache)[L.offset(b, kvh, 1, t % bs, lane * kDims + d)];
      }
    }
    float z = 0.f;
#pragma unroll
    for (int d = 0; d < kDims; ++d) z = fmaf(x[d], k[d], z);
#pragma unroll
    for (int i = 16; i; i >>= 1) z += __shfl_xor_sync(0xffffffffu, z, i);
    const float mn = fmaxf(m, z), a = exp2f(m - mn), e = exp2f(z - mn);
    l = l * a + e;
#pragma unroll
    for (int d = 0; d < kDims; ++d) o[d] = o[d] * a + e * v[d];
    m = mn;
  }
  T* out = static_cast<T*>(p.out) + ((int64_t)tok * p.num_q_heads + h) * D + lane * kDims;
#pragma unroll
  for (int d = 0; d < kDims; ++d) out[d] = Elem<T>::from_float(ok && l > 0.f ? o[d] / l : 0.f);
}

template <typename T>
cudaError_t launch_typed(const ExtendParams& p, int head_size, bool i8, cudaStream_t stream) {
  const int64_t warps = (int64_t)p.num_tokens * p.num_q_heads;
  const unsigned grid = (unsigned)((warps + 3) / 4);
  if (i8) extend_kernel<T, 128, true><<<grid, 128, 0, stream>>>(p);
  else if (head_size == 128) extend_kernel<T, 128, false><<<grid, 128, 0, stream>>>(p);
  else extend_kernel<T, 64, false><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_extend(const ExtendParams& p, int act_dtype, int head_size, bool i8, cudaStream_t stream) {
  return act_dtype == PA_F16 ? launch_typed<__half>(p, head_size, i8, stream)
                             : launch_typed<__nv_bfloat16>(p, head_size, i8, stream);
}

}  // namespace pkv

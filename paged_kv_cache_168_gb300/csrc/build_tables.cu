// build_tables.cu -- block tables, slot mapping and positions of a step from the
// requests' lengths (the KV manager's and model runner's bookkeeping of the
// tiemojia.cn vLLM V1 walkthrough, sections 3.3-3.4, on the device).
//
// Everything follows from two prefix sums over the requests: new tokens (the
// query starts) and blocks handed out.  Every CTA works both out for itself --
// two int32 per request, from L2 -- and keeps them in shared memory with the
// contexts; then each thread takes tokens, finds a token's request by binary
// search there, and derives its block from the free list (a block begun in this
// step) or the table (the request's last, partly filled block).  Every block
// begun in a step is begun by one of its tokens, which writes the table entry,
// so entries read and entries written are disjoint and no pass waits for
// another.  One launch: the CTAs are one cluster, whose barrier separates reading
// the inputs from overwriting them (lengths and free count may be updated in
// place).
//
// Bound: launch latency and the chain lengths -> scan -> search -> store; the
// bytes of a step would take 0.1 us.  Back to back in a graph: 256 decoding
// requests 5.0 us, 2048 of them 7.2, 16 prompts of 1024 or 2048 tokens 5.9 (one CTA
// instead of eight: 5.0, 7.0, and 11.9 for the prompts of 1024).
#include "common.cuh"
#include "kernels.h"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;       // the largest portable cluster
constexpr int kRun = 4;           // consecutive tokens of a thread

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int64_t warp_inclusive(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

__global__ void __launch_bounds__(kThreads, 1) build_tables_kernel(const TablesParams p, bool wide) {
  extern __shared__ int32_t dyn[];
  const int S = p.num_seqs, bs = p.block_size, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int shift = __ffs(bs) - 1;                    // block sizes are powers of two
  const int64_t cap = p.ring_blocks > 0 ? p.ring_blocks : INT64_MAX;
  int32_t* starts = dyn;                              // [S + 1] query starts
  int32_t* first = starts + S + 1;                    // [S] number of the request's first new block
  int32_t* ctxs = first + S;                          // [S]
  __shared__ int64_t wsum[2][kWarps];
  __shared__ uint32_t bad;
  if (tid == 0) bad = 0;
  const int num_free = *p.num_free;
  __syncthreads();

  // ---- scan: thread t owns the requests [t * per, (t + 1) * per)
  const int per = (S + kThreads - 1) / kThreads;
  const int s0 = min(S, tid * per), s1 = min(S, s0 + per);
  int64_t tok = 0, blk = 0;
  uint32_t err = 0;
  for (int s = s0; s < s1; ++s) {
    const int64_t c = p.cached_lens[s], n = p.new_lens[s], ctx = c + n;
    if (c < 0 || n < 0 || ctx > INT32_MAX || (p.ring_blocks == 0 && ctx > (int64_t)p.bt_width * bs)) {
      err = PA_DEVERR_CONTEXT;
      continue;
    }
    ctxs[s] = (int32_t)ctx;
    tok += n;
    blk += min((ctx + bs - 1) >> shift, cap) - min((c + bs - 1) >> shift, cap);
  }
  int64_t itok = warp_inclusive(tok, lane), iblk = warp_inclusive(blk, lane);
  if (lane == 31) {
    wsum[0][warp] = itok;
    wsum[1][warp] = iblk;
  }
  if (err) atomicOr(&bad, err);
  __syncthreads();
  int64_t total = 0, taken = 0;
  {
    const int64_t a = warp_inclusive(wsum[0][lane], lane), b = warp_inclusive(wsum[1][lane], lane);
    total = __shfl_sync(0xffffffffu, a, 31);
    taken = __shfl_sync(0xffffffffu, b, 31);
    const int64_t pa = __shfl_sync(0xffffffffu, a, (warp + 31) & 31), pb = __shfl_sync(0xffffffffu, b, (warp + 31) & 31);
    itok += (warp ? pa : 0) - tok;                    // exclusive over the whole CTA
    iblk += (warp ? pb : 0) - blk;
  }
  err = bad;
  if (total > p.max_tokens) err |= PA_DEVERR_CONTEXT;
  if (num_free < 0 || num_free > p.num_blocks || taken > num_free) err |= PA_DEVERR_OUT_OF_BLOCKS;
  const bool ok = err == 0;                           // the same in every thread of every CTA
  if (ok) {
    for (int s = s0; s < s1; ++s) {
      const int64_t n = p.new_lens[s], ctx = ctxs[s], c = ctx - n;
      starts[s] = (int32_t)itok;
      first[s] = (int32_t)iblk;
      itok += n;
      iblk += min((ctx + bs - 1) >> shift, cap) - min((c + bs - 1) >> shift, cap);
    }
    if (tid == 0) starts[S] = (int32_t)total;
  }
  cluster_sync();                                     // every CTA has read the lengths and the free count
  if (blockIdx.x == 0) {
    // lengths updated in place stay as they are when the step cannot be built: it can be tried again
    const bool keep = !ok && p.context_lens == p.cached_lens;
    for (int s = tid; s < S; s += kThreads) {
      p.query_start_loc[s] = ok ? starts[s] : 0;
      if (!keep) p.context_lens[s] = ok ? ctxs[s] : 0;
    }
    if (tid == 0) {
      p.query_start_loc[S] = ok ? (int32_t)total : 0;
      *p.num_free_out = ok ? num_free - (int32_t)taken : num_free;
      if (err) report(p.dev_err, err);
    }
  }

  // ---- tokens, four in a row a thread: one search, four independent lookups
  const int n_tok = ok ? (int)total : 0;
  for (int64_t i0 = ((int64_t)blockIdx.x * kThreads + tid) * kRun; i0 < p.max_tokens;
       i0 += (int64_t)gridDim.x * kThreads * kRun) {
    int64_t slot[kRun];
    int pos[kRun], s = 0;
    if (i0 < n_tok) {
      int hi = S;                                     // the last request with starts <= i0
      while (hi - s > 1) {
        const int mid = (s + hi) >> 1;
        if (starts[mid] <= i0) s = mid; else hi = mid;
      }
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      slot[k] = -1;
      pos[k] = 0;
      if (i0 + k >= n_tok) continue;
      const int i = (int)i0 + k;
      while (starts[s + 1] <= i) ++s;                 // (ends: i < starts[S])
      const int ctx = ctxs[s];
      const int cached = ctx - (starts[s + 1] - starts[s]);
      pos[k] = cached + (i - starts[s]);
      const int b = pos[k] >> shift;
      const int have = (int)min(((int64_t)cached + bs - 1) >> shift, cap);
      const bool kept = p.ring_blocks == 0 || b > ((ctx - 1) >> shift) - p.ring_blocks;
      const int e = p.ring_blocks > 0 ? b % p.ring_blocks : b;
      int32_t* entry = p.block_tables + s * p.bt_stride + e;
      // begun in this step: logical block b itself, or (ring) the one whose entry b takes over
      const bool fresh = e >= have;
      if (kept || fresh) {
        const int id = fresh ? p.free_blocks[num_free - 1 - (first[s] + e - have)] : *entry;
        if (fresh && b == e && (pos[k] & (bs - 1)) == 0) *entry = id;
        if ((unsigned)id < (unsigned)p.num_blocks) {
          if (kept) slot[k] = ((int64_t)id << shift) + (pos[k] & (bs - 1));
        } else {
          report(p.dev_err, PA_DEVERR_BLOCK_ID);
        }
      }
    }
    if (wide && i0 + kRun <= p.max_tokens) {
#pragma unroll
      for (int k = 0; k < kRun; k += 2)
        *reinterpret_cast<longlong2*>(p.slot_mapping + i0 + k) = make_longlong2(slot[k], slot[k + 1]);
      if (p.positions) *reinterpret_cast<int4*>(p.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kRun; ++k)
        if (i0 + k < p.max_tokens) {
          p.slot_mapping[i0 + k] = slot[k];
          if (p.positions) p.positions[i0 + k] = pos[k];
        }
    }
  }
}

}  // namespace

cudaError_t launch_build_tables(const TablesParams& p, cudaStream_t stream) {
  const size_t smem = (3 * (size_t)p.num_seqs + 1) * sizeof(int32_t);
  cudaError_t e = set_smem_attribute_once<build_tables_kernel>((3 * (size_t)PA_BUILD_TABLES_MAX_SEQS + 1) * sizeof(int32_t));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kCluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const bool wide = ((reinterpret_cast<uintptr_t>(p.slot_mapping) | reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
  return cudaLaunchKernelEx(&cfg, build_tables_kernel, p, wide);
}

}  // namespace pkv

// Block tables and slot maps of a batch, built on the GPU from its requests'
// lengths, with the free cache blocks on a stack in device memory: nothing
// goes through the host, so a step can be captured into a CUDA graph.
//
// extend: request r has c_r tokens cached and brings q_r new ones.
//   have_r = min(ceil(c_r / 64), MB), want_r = min(ceil((c_r + q_r) / 64), MB)
//   first_r = sum of (want - have) over the requests before r
//   block_table[r, j], have_r <= j < want_r, = free_blocks[F - 1 - n], the
//     n = first_r + j - have_r th new block (F = free_count; -1 once n >= F)
//   query_start_r = sum of q over the requests before r (at most T)
//   token t of request r: position c_r + t - query_start_r, its slot
//     block_table[r, position / 64] * 64 + position % 64
// release: the blocks of the released requests, in order, back on the stack.
//
// Both are bound by latency: a few KB to 1 MB are moved.  One launch: every CTA
// makes the prefix sums over the requests in its shared memory (redundantly: no
// exchange through global memory), then all threads share the tokens and blocks,
// each finding its request by a binary search in shared memory.  Where an output
// may overwrite an input (release always counts across CTAs, too) the CTAs form
// one thread-block cluster, and inputs are read before a cluster barrier and
// written after it; extend otherwise takes as many CTAs as the tokens fill.
// Measured, replayed from a graph: extend, 500 requests with 90 000 new tokens 8.4
// us (1.5 MB), 8 single tokens 5.5; release, a third of 700 requests 11.5 us (0.5 MB:
// the table rows, then the stack, three dependent passes through memory), 3 of 8 4.1.
#include <cstdint>
#include <algorithm>
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "smla_common.cuh"
#include "smla_kernels.h"

namespace cg = cooperative_groups;

namespace smla {

namespace {

constexpr int kMaxThreads = 1024;

// a + b, at most cap (both at most cap <= 2^31 - 1): associative, so a prefix
// sum can use it in any grouping.
__device__ __forceinline__ uint32_t add_capped(uint32_t a, uint32_t b, uint32_t cap) { return min(a + b, cap); }

// Exclusive prefix sums of v[0 .. n-1] in place (sums capped), the total in
// v[n]; all threads of the CTA.
__device__ void scan_in_place(uint32_t* v, int n, uint32_t cap) {
  __shared__ uint32_t warp_sum[kMaxThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int per = (n + blockDim.x - 1) / blockDim.x;
  const int beg = min(tid * per, n), end = min(beg + per, n);
  uint32_t sum = 0;
  for (int i = beg; i < end; ++i) sum = add_capped(sum, v[i], cap);
  uint32_t inc = sum;
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc = add_capped(inc, u, cap);
  }
  uint32_t before = __shfl_up_sync(0xffffffffu, inc, 1);
  if (lane == 0) before = 0;
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  uint32_t base = 0;
  for (int w = 0; w < warp; ++w) base = add_capped(base, warp_sum[w], cap);
  uint32_t run = add_capped(base, before, cap);
  for (int i = beg; i < end; ++i) {
    const uint32_t x = v[i];
    v[i] = run;
    run = add_capped(run, x, cap);
  }
  if (tid == 0) {
    uint32_t total = 0;
    for (int w = 0; w < nw; ++w) total = add_capped(total, warp_sum[w], cap);
    v[n] = total;
  }
  __syncthreads();
}

// The last i in [0, n) with v[i] <= x (v non-decreasing, v[0] <= x).
__device__ __forceinline__ int last_not_above(const uint32_t* v, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int blocks_of(int64_t tokens, int MB) {
  return (int)min((tokens + kBlock - 1) / kBlock, (int64_t)MB);
}

__global__ void __launch_bounds__(kMaxThreads) blocks_extend_kernel(const __grid_constant__ BlocksExtendArgs a) {
  extern __shared__ uint32_t smem_blocks[];
  const cg::cluster_group cluster = cg::this_cluster();
  uint32_t* start = smem_blocks;           // [R + 1] first token
  uint32_t* first = start + a.R + 1;       // [R + 1] first new block
  uint32_t* ctx = first + a.R + 1;         // [R] cached tokens
  const int tid = threadIdx.x;
  const int64_t gid = (int64_t)blockIdx.x * blockDim.x + tid, step = (int64_t)gridDim.x * blockDim.x;
  const int free_count = max(0, min(__ldg(a.free_count), a.F));
  for (int r = tid; r < a.R; r += blockDim.x) {
    const int c = max(0, a.context_lens[r]), q = max(0, a.query_lens[r]);
    ctx[r] = (uint32_t)c;
    start[r] = (uint32_t)min(q, a.T);
    first[r] = (uint32_t)(blocks_of((int64_t)c + q, a.MB) - blocks_of(c, a.MB));
  }
  __syncthreads();
  // The length of request gid, read here because seq_lens may be one of the inputs: the cluster has a
  // thread for every request (kMaxPagedRequests is 8 CTAs of 1024).
  int64_t len0 = 0;
  if (gid < a.R) len0 = (int64_t)max(0, a.context_lens[gid]) + max(0, a.query_lens[gid]);
  scan_in_place(start, a.R, (uint32_t)a.T);
  scan_in_place(first, a.R, 0x7fffffffu);
  const uint32_t used = start[a.R], grown = first[a.R];
  cluster.sync();

  for (int64_t r = gid; r <= a.R; r += step) {
    a.query_start[r] = (int32_t)start[r];
    if (r < a.R) a.seq_lens[r] = (int32_t)min(len0, (int64_t)0x7fffffff);
  }
  if (gid == 0) {
    *a.free_count_out = max(0, free_count - (int)grown);
    *a.missing = max(0, (int)grown - free_count);
  }
  for (int64_t n = gid; n < (int64_t)grown; n += step) {
    const int r = last_not_above(first, a.R, (uint32_t)n);
    const int j = blocks_of((int64_t)ctx[r], a.MB) + (int)((uint32_t)n - first[r]);
    const int64_t at = (int64_t)free_count - 1 - n;
    a.block_table[(int64_t)r * a.MB + j] = at >= 0 ? __ldg(a.free_blocks + at) : -1;
  }
  // four tokens a thread: mostly of one request and block, so one search and one table read
  const bool whole = ((reinterpret_cast<uintptr_t>(a.req_id_per_token) | reinterpret_cast<uintptr_t>(a.positions) |
                       reinterpret_cast<uintptr_t>(a.slot_mapping)) & 15u) == 0;  // 16-byte stores
  for (int64_t t0 = 4 * gid; t0 < a.T; t0 += 4 * step) {
    int32_t req[4], pos[4];
    int64_t slot[4];
    int r = -1, have = 0;
    int64_t j_at = -1, b = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t t = t0 + k;
      req[k] = -1;
      pos[k] = 0;
      slot[k] = -1;
      if (t < (int64_t)used) {
        if (r < 0 || (uint32_t)t >= start[r + 1]) {
          r = last_not_above(start, a.R, (uint32_t)t);
          have = blocks_of((int64_t)ctx[r], a.MB);
          j_at = -1;
        }
        const int64_t p = (int64_t)ctx[r] + (t - start[r]), j = p / kBlock;
        if (j != j_at) {
          j_at = j;
          b = -1;
          if (j < have) {
            b = a.block_table[(int64_t)r * a.MB + j];  // not written by this call
          } else if (j < a.MB) {
            const int64_t at = (int64_t)free_count - 1 - ((int64_t)first[r] + (j - have));
            if (at >= 0) b = __ldg(a.free_blocks + at);
          }
        }
        req[k] = r;
        pos[k] = (int32_t)min(p, (int64_t)0x7fffffff);
        if (b >= 0 && b < a.NB) slot[k] = b * kBlock + p % kBlock;
      }
    }
    if (whole && t0 + 4 <= a.T) {
      *reinterpret_cast<int4*>(a.req_id_per_token + t0) = make_int4(req[0], req[1], req[2], req[3]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<longlong2*>(a.slot_mapping + t0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2*>(a.slot_mapping + t0 + 2) = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (t0 + k < a.T) {
          a.req_id_per_token[t0 + k] = req[k];
          a.positions[t0 + k] = pos[k];
          a.slot_mapping[t0 + k] = slot[k];
        }
    }
  }
  // The latent cache's store and decode read these results before they wait for this grid: they begin when its CTAs
  // have ended, and by then the results are there for all.
  __threadfence();
}

// A unit is a run of `chunk` table entries of one request; a warp counts the
// blocks of a unit, and pushes them after the prefix sums over the units.
__global__ void __launch_bounds__(kMaxThreads) blocks_release_kernel(const __grid_constant__ BlocksReleaseArgs a) {
  extern __shared__ uint32_t smem_blocks[];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31;
  const int nw = (int)(gridDim.x * blockDim.x) >> 5, w0 = (int)(blockIdx.x * blockDim.x + tid) >> 5;
  const int nch = (a.MB + a.chunk - 1) / a.chunk, units = a.R * nch;
  uint32_t* count = smem_blocks;       // [units + 1]
  uint32_t* held = count + units + 1;  // [R] table entries to look at
  const int free_count = max(0, min(__ldg(a.free_count), a.F));
  for (int r = tid; r < a.R; r += blockDim.x) held[r] = a.release[r] ? blocks_of(max(0, a.seq_lens[r]), a.MB) : 0;
  // this thread's request (the cluster has a thread for each): its length may be overwritten below
  const int mine = (int)(blockIdx.x * blockDim.x) + tid;
  const int left = mine < a.R && !a.release[mine] ? a.seq_lens[mine] : 0;
  for (int u = tid; u < units; u += blockDim.x) count[u] = 0u;
  cluster.sync();  // every CTA's counts are 0 before others' arrive
  // entries of unit u: the first of them, and their number
  auto entries = [&](int u, const int32_t*& row) {
    const int r = u / nch, j0 = (u - r * nch) * a.chunk;
    row = a.block_table + (int64_t)r * a.MB + j0;
    return max(0, min(a.chunk, (int)held[r] - j0));
  };
  constexpr int kAhead = 4;  // reads in flight a lane
  for (int u = w0; u < units; u += nw) {
    const int32_t* row;
    const int n = entries(u, row);
    if (n == 0) continue;
    int got = 0;
    for (int i0 = 0; i0 < n; i0 += 32 * kAhead) {
      int b[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) b[k] = i0 + 32 * k + lane < n ? row[i0 + 32 * k + lane] : -1;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) got += b[k] >= 0 && b[k] < a.NB;
    }
    got = __reduce_add_sync(0xffffffffu, got);
    if (got > 0 && lane < (int)gridDim.x) cluster.map_shared_rank(count, lane)[u] = (uint32_t)got;
  }
  cluster.sync();
  scan_in_place(count, units, 0x7fffffffu);
  for (int u = w0; u < units; u += nw) {
    if (count[u + 1] == count[u]) continue;
    const int32_t* row;
    const int n = entries(u, row);
    int64_t at = (int64_t)free_count + count[u];
    for (int i0 = 0; i0 < n; i0 += 32 * kAhead) {
      int b[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) b[k] = i0 + 32 * k + lane < n ? row[i0 + 32 * k + lane] : -1;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const bool ok = b[k] >= 0 && b[k] < a.NB;
        const uint32_t who = __ballot_sync(0xffffffffu, ok);
        const int64_t to = at + __popc(who & ((1u << lane) - 1u));
        if (ok && to < a.F) a.free_blocks[to] = b[k];
        at += __popc(who);
      }
    }
  }
  cluster.sync();  // all lengths and the count have been read: context_lens and free_count_out may be the inputs
  if (mine < a.R) a.context_lens[mine] = left;
  if (blockIdx.x == 0 && tid == 0) *a.free_count_out = (int)min((int64_t)a.F, (int64_t)free_count + count[units]);
}

template <typename Args>
cudaError_t launch_cluster(void (*kernel)(Args), const Args& a, int ctas, int cluster, int threads, size_t smem,
                           cudaStream_t stream) {
  // set at every launch: it takes well under a microsecond and needs no per-device record
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// CTAs (1, 2, 4 or 8, a portable cluster) and threads for `work` items.
void size_cluster(int64_t work, int* ctas, int* threads) {
  *threads = work <= 256 ? 256 : kMaxThreads;
  *ctas = 1;
  while (*ctas < 8 && (int64_t)*ctas * *threads < work) *ctas *= 2;
}

}  // namespace

static bool overlap(const void* a, const void* b, size_t a_bytes, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

cudaError_t launch_blocks_extend(const BlocksExtendArgs& a, cudaStream_t stream) {
  const int64_t work = std::max<int64_t>((int64_t)a.R + 1, (a.T + 3) / 4);
  const size_t smem = (size_t)(3 * (int64_t)a.R + 2) * 4, lens = (size_t)a.R * 4;
  int ctas, threads;
  size_cluster(work, &ctas, &threads);
  const bool in_place = overlap(a.seq_lens, a.context_lens, lens, lens) || overlap(a.seq_lens, a.query_lens, lens, lens) ||
                        overlap(a.free_count_out, a.free_count, 4, 4);
  if (in_place || ctas == 1) return launch_cluster(blocks_extend_kernel, a, ctas, ctas, threads, smem, stream);
  // Separate outputs: CTAs of 512 threads, one four-token item a thread, at most 64 of them (each makes the
  // prefix sums); 90 K tokens of 500 requests take 16.5 us in one cluster
  constexpr int kThreads = 512;
  ctas = (int)std::min<int64_t>(64, (work + kThreads - 1) / kThreads);
  return launch_cluster(blocks_extend_kernel, a, ctas, 1, kThreads, smem, stream);
}

cudaError_t launch_blocks_release(BlocksReleaseArgs a, cudaStream_t stream) {
  a.chunk = 512;
  while ((int64_t)a.R * ((a.MB + a.chunk - 1) / a.chunk) > kMaxPagedRequests) a.chunk *= 2;
  const int64_t units = (int64_t)a.R * ((a.MB + a.chunk - 1) / a.chunk);
  int ctas, threads;
  size_cluster(std::max<int64_t>(32 * units, a.R), &ctas, &threads);  // a warp a unit
  return launch_cluster(blocks_release_kernel, a, ctas, ctas, threads, (size_t)(units + 1 + a.R) * 4, stream);
}

}  // namespace smla

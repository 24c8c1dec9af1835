// Eviction from a dense cache by accumulated attention weight, per KV head.
//
// Of the len tokens of a unit (row, KV head), the first `sinks` and the last
// `recent` are kept always; the rest of the `keep` places go to the largest
// running sums, equal ones to the lower position.  Kept tokens stay in order.
//
//   select_kernel  a cluster of up to 8 blocks per unit, a stretch of positions each,
//                  the sums in shared memory.  A radix select over the sums' 32-bit
//                  patterns (monotone for sums >= 0; histograms added up through
//                  distributed shared memory) finds the smallest kept sum and how
//                  many tokens equal to it are kept; then each warp counts its
//                  stretch of positions, the counts are scanned, and each warp
//                  writes its kept positions and sums.  Reads the sums once.
//   gather, move   copy the kept rows of K and V: bound by memory, 4 d bytes read and
//                  written per kept token.
#include <math.h>

#include "dense_attn.h"
#include "kvc_device.cuh"

namespace kvc {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;              // 11 bits a pass: 11 + 11 + 10
constexpr int kStageTok = 48 * 1024;     // sums held in a block's shared memory
constexpr int kMaxBlocks = 8;            // blocks of a cluster

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void add_rank(unsigned* p, unsigned x, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("red.shared::cluster.add.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ uint2 ld_rank(const void* p, int rank) {
  uint32_t a;
  uint2 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ unsigned scan_up(unsigned v) {      // inclusive sum over the lanes up to this one
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, v, o);
    if ((int)(threadIdx.x & 31) >= o) v += x;
  }
  return v;
}

__device__ __forceinline__ int evict_len(const EvictCall& p, int u) {
  int n = p.n_tokens;
  if (p.seq_lens) {
    const int s = p.seq_lens[(u / p.Hkv) % p.B];
    n = s < 0 ? 0 : (s < n ? s : n);
  }
  return n;
}

__device__ __forceinline__ uint32_t sum_key(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

template <bool STAGED>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ EvictCall p) {
  extern __shared__ float sums[];        // STAGED: the block's stretch of the row's sums
  __shared__ __align__(16) unsigned hist[kBins], all[2][kBins];      // the block's counts; block 0: the cluster's
  __shared__ unsigned warp_a[kSelWarps], warp_b[kSelWarps];
  __shared__ uint2 sh_digit;             // block 0: the digit found, and need
  static_assert(kBins == 4 * kSelThreads && kSelWarps <= 32, "a thread owns four bins");
  __shared__ uint2 total;                // this block's kept tokens, and those equal to the boundary
  const int C = p.blocks, rank = blockIdx.x % C, u = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = evict_len(p, u);
  const int new_len = min(len, p.keep);
  int* const kept = p.kept + (size_t)u * p.keep;
  const float* const w = p.w + (size_t)u * p.tmax;
  float* const w2 = p.w2 + (size_t)u * p.tmax2;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (u < p.B * p.Hkv && u % p.Hkv == 0 && rank == 0 && tid == 0) p.new_lens[u / p.Hkv] = new_len;
  // this block's positions [q0, q1)
  const int per_block = ((len + C - 1) / C + 31) & ~31;
  const int q0 = min(len, rank * per_block), q1 = min(len, q0 + per_block);
  if (STAGED)
    for (int t = q0 + tid; t < q1; t += kSelThreads) sums[t - q0] = w[t];
  auto sum_at = [&](int t) { return STAGED ? sums[t - q0] : w[t]; };
  for (int i = new_len + rank * kSelThreads + tid; i < p.keep; i += C * kSelThreads) kept[i] = -1;
  if (len <= p.keep) {                   // the row keeps all
    if (STAGED) cluster_sync();          // in place: read before written
    for (int t = q0 + tid; t < q1; t += kSelThreads) {
      kept[t] = t;
      if (STAGED) w2[t] = sums[t - q0];
    }
  } else {
    // candidates: tokens [c0, c1), of which `need` are kept (sinks + recent <= keep < len)
    const int c0 = p.sinks, c1 = len - p.recent;
    const int h0 = max(q0, c0), h1 = min(q1, c1);
    unsigned need = (unsigned)(p.keep - p.sinks - p.recent);
    // the key of the need-th largest candidate, digit by digit from the top;
    // need becomes the number of candidates equal to it that are kept
    uint32_t prefix = 0;
    int shift = 32;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(&hist[4 * tid]) = *reinterpret_cast<uint4*>(&all[0][4 * tid]) = none;
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass == 2 ? 10 : 11;
      const uint32_t hi = pass == 0 ? 0u : ~0u << shift;
      unsigned* const sum = all[pass & 1];
      shift -= bits;
      __syncthreads();
      for (int t = h0 + tid; t < h1; t += kSelThreads) {
        const uint32_t k = sum_key(sum_at(t));
        if ((k & hi) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
      }
      if (pass == 0) cluster_sync();     // the cluster's blocks run, block 0's counts are zero
      else __syncthreads();
      // counts to block 0, few of them: the sums share most of their leading bits.  (Every
      // block reading all of them: 25 us for 8 rows of 32K tokens where this takes 23.)
      const uint4 x = *reinterpret_cast<const uint4*>(&hist[4 * tid]);
      *reinterpret_cast<uint4*>(&hist[4 * tid]) = none;
      if (x.x) add_rank(&sum[4 * tid], x.x, 0);
      if (x.y) add_rank(&sum[4 * tid + 1], x.y, 0);
      if (x.z) add_rank(&sum[4 * tid + 2], x.z, 0);
      if (x.w) add_rank(&sum[4 * tid + 3], x.w, 0);
      cluster_sync();
      if (rank == 0) {
        *reinterpret_cast<uint4*>(&all[(pass + 1) & 1][4 * tid]) = none;
        // suffix sums of the bins: thread t owns bins 4 t .. 4 t + 3
        const uint4 y = *reinterpret_cast<const uint4*>(&sum[4 * tid]);
        const unsigned bin[4] = {y.x, y.y, y.z, y.w};
        const unsigned own = bin[0] + bin[1] + bin[2] + bin[3];
        unsigned v = own;                // sum over this lane and the lanes above it
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned z = __shfl_down_sync(0xffffffffu, v, o);
          if (lane + o < 32) v += z;
        }
        if (lane == 0) warp_a[warp] = v;
        __syncthreads();
        const unsigned above = __reduce_add_sync(0xffffffffu, lane > warp && lane < kSelWarps ? warp_a[lane] : 0u);
        unsigned over = above + v - own; // candidates in the bins above
#pragma unroll
        for (int k = 3; k >= 0; --k) {
          if (need > over && need <= over + bin[k]) sh_digit = make_uint2(4 * tid + k, need - over);
          over += bin[k];
        }
        if (need == 0 && tid == 0) sh_digit = make_uint2(kBins - 1, 0u);
      }
      cluster_sync();
      const uint2 found = ld_rank(&sh_digit, 0);
      prefix |= (found.x & ((1u << bits) - 1u)) << shift;
      need = found.y;
    }
    // need == 0 (nothing but the protected tokens): the key is above every sum
    if (p.keep == p.sinks + p.recent) prefix = 0xffffffffu;
    // each warp takes a stretch of the block's positions
    const int per = (q1 - q0 + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;
    const int s0 = min(q1, q0 + warp * per), s1 = min(q1, s0 + per);
    // 2: kept, 1: equal to the boundary key, 0: not kept
    auto cls = [&](int t) -> int {
      if (t >= s1) return 0;
      if (t < c0 || t >= c1) return 2;
      const uint32_t k = sum_key(sum_at(t));
      return k > prefix ? 2 : k == prefix ? 1 : 0;
    };
    unsigned n_gt = 0, n_eq = 0;
    for (int t = s0 + lane; t - lane < s1; t += 32) {
      const int c = cls(t);
      n_gt += __popc(__ballot_sync(0xffffffffu, c == 2));
      n_eq += __popc(__ballot_sync(0xffffffffu, c == 1));
    }
    __syncthreads();
    if (lane == 0) warp_a[warp] = n_gt, warp_b[warp] = n_eq;
    __syncthreads();
    // kept and equal tokens before this warp's stretch: of the block's warps, of the blocks
    const unsigned wa = scan_up(lane < kSelWarps ? warp_a[lane] : 0u), wb = scan_up(lane < kSelWarps ? warp_b[lane] : 0u);
    if (tid == 31) total = make_uint2(wa, wb);
    cluster_sync();
    uint2 before = make_uint2(0, 0);
    for (int c = 0; c < rank; ++c) {
      const uint2 x = ld_rank(&total, c);
      before.x += x.x;
      before.y += x.y;
    }
    unsigned eq = before.y + __shfl_sync(0xffffffffu, wb, warp) - n_eq;
    unsigned at = before.x + __shfl_sync(0xffffffffu, wa, warp) - n_gt + min(eq, need);
    for (int t = s0 + lane; t - lane < s1; t += 32) {
      const int c = cls(t);
      const unsigned m1 = __ballot_sync(0xffffffffu, c == 1);
      const unsigned ahead = __popc(m1 & ((1u << lane) - 1u));
      const bool k = c == 2 || (c == 1 && eq + ahead < need);
      const unsigned mk = __ballot_sync(0xffffffffu, k);
      if (k) {
        const unsigned i = at + __popc(mk & ((1u << lane) - 1u));
        kept[i] = t;
        if (STAGED) w2[i] = sum_at(t);
      }
      at += __popc(mk);
      eq += __popc(m1);
    }
  }
  // every block of the cluster has read the sums it needs; tokens appended later start at zero
  cluster_sync();
  if (STAGED)
    for (int i = new_len + rank * kSelThreads + tid; i < p.tmax2; i += C * kSelThreads) w2[i] = 0.f;
}

// Kept rows into another cache: 16 bytes per thread, d / 8 threads per row.  (Copying
// the protected rows before the selection ends takes longer in all: 121 us for 8 rows
// of 32K tokens, 112 so.)
constexpr int kGThreads = 256;
constexpr int kGUnroll = 8;

template <int D>
__global__ void __launch_bounds__(kGThreads) gather_kernel(const __grid_constant__ EvictCall p) {
  constexpr int TPR = D / 8, RPB = kGThreads / TPR;
  const int nb = (p.keep + RPB * kGUnroll - 1) / (RPB * kGUnroll);      // blocks per unit and tensor
  const int u = blockIdx.x / (2 * nb), b = blockIdx.x % (2 * nb), col = threadIdx.x % TPR;
  const uint4* src = reinterpret_cast<const uint4*>(b >= nb ? p.v : p.k) + (size_t)u * p.tmax * TPR + col;
  uint4* dst = reinterpret_cast<uint4*>(b >= nb ? p.v2 : p.k2) + (size_t)u * p.tmax2 * TPR + col;
  const int i0 = b % nb * RPB * kGUnroll + threadIdx.x / TPR;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int* kept = p.kept + (size_t)u * p.keep;
  int t[kGUnroll];
  uint4 x[kGUnroll];
#pragma unroll
  for (int k = 0; k < kGUnroll; ++k) t[k] = i0 + k * RPB < p.keep ? kept[i0 + k * RPB] : -1;
#pragma unroll
  for (int k = 0; k < kGUnroll; ++k)
    if (t[k] >= 0) x[k] = src[(size_t)t[k] * TPR];
#pragma unroll
  for (int k = 0; k < kGUnroll; ++k)
    if (t[k] >= 0) dst[(size_t)(i0 + k * RPB) * TPR] = x[k];
}

// Kept rows moved down within one cache.  A block owns a 64-byte column of a
// unit's rows (so that blocks do not meet) and takes the kept tokens in
// order, a chunk at a time: kept[i] >= i, so a chunk's stores reach no row that
// a later chunk still reads, and its own reads end before its stores begin.
constexpr int kMoveTPR = 4, kMoveRows = kGThreads / kMoveTPR;

template <int D>
__global__ void __launch_bounds__(kGThreads) move_kernel(const __grid_constant__ EvictCall p) {
  constexpr int TPR = D / 8, COLS = TPR / kMoveTPR;
  const int u = blockIdx.x / (2 * COLS), part = blockIdx.x % (2 * COLS);
  const int col = (part % COLS) * kMoveTPR + threadIdx.x % kMoveTPR;
  uint4* rows = reinterpret_cast<uint4*>(part >= COLS ? p.v2 : p.k2) + (size_t)u * p.tmax2 * TPR + col;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int* kept = p.kept + (size_t)u * p.keep;
  for (int i0 = threadIdx.x / kMoveTPR; i0 - (int)(threadIdx.x / kMoveTPR) < p.keep; i0 += kMoveRows * kGUnroll) {
    int t[kGUnroll];
    uint4 x[kGUnroll];
#pragma unroll
    for (int k = 0; k < kGUnroll; ++k) t[k] = i0 + k * kMoveRows < p.keep ? kept[i0 + k * kMoveRows] : -1;
#pragma unroll
    for (int k = 0; k < kGUnroll; ++k)
      if (t[k] >= 0) x[k] = rows[(size_t)t[k] * TPR];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kGUnroll; ++k)
      if (t[k] >= 0) rows[(size_t)(i0 + k * kMoveRows) * TPR] = x[k];
  }
}

// The kept sums of rows too long for shared memory, in order and chunk by chunk as
// above (source and destination may be one array); zero from the new length on.
__global__ void __launch_bounds__(kSelThreads) gather_sums_kernel(const __grid_constant__ EvictCall p) {
  const int u = blockIdx.x;
  const float* src = p.w + (size_t)u * p.tmax;
  float* dst = p.w2 + (size_t)u * p.tmax2;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int* kept = p.kept + (size_t)u * p.keep;
  for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < p.tmax2; i0 += kSelThreads * 4) {
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * kSelThreads;
      const int t = i < p.keep ? kept[i] : -1;
      x[k] = t >= 0 ? src[t] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + k * kSelThreads < p.tmax2) dst[i0 + k * kSelThreads] = x[k];
  }
}

template <int D>
cudaError_t launch_rows(const EvictCall& c, cudaLaunchConfig_t& cfg) {
  if (c.in_place) {
    cfg.gridDim = dim3((unsigned)c.units * (2 * (D / 8) / kMoveTPR));
    return cudaLaunchKernelEx(&cfg, move_kernel<D>, c);
  }
  const int per = kGThreads / (D / 8) * kGUnroll;
  cfg.gridDim = dim3((unsigned)c.units * 2 * ((c.keep + per - 1) / per));
  return cudaLaunchKernelEx(&cfg, gather_kernel<D>, c);
}

}  // namespace

cudaError_t launch_evict(const EvictCall& call, cudaStream_t s) {
  EvictCall c = call;
  // blocks per unit: while they fit the SMs twice over and have 2048 tokens each, and
  // as many as the shared memory asks for
  c.blocks = 1;
  while (c.blocks < kMaxBlocks && ((c.units * c.blocks * 2 <= 2 * kNumSMs && c.n_tokens / (2 * c.blocks) >= 2048) ||
                                   c.n_tokens > c.blocks * kStageTok))
    c.blocks *= 2;
  const bool staged = c.n_tokens <= c.blocks * kStageTok;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)c.blocks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)c.units * c.blocks);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (staged) {
    cfg.dynamicSmemBytes = (size_t)(((c.n_tokens + c.blocks - 1) / c.blocks + 31) & ~31) * sizeof(float);
    e = cudaSuccess;
    if (cfg.dynamicSmemBytes > 16 * 1024)                // with the histograms above what every kernel may have
      e = cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageTok * 4);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, select_kernel<true>, c);
  } else {
    e = cudaLaunchKernelEx(&cfg, select_kernel<false>, c);
  }
  if (e != cudaSuccess) return e;
  // the copies start as the selection ends
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kGThreads);
  cfg.dynamicSmemBytes = 0;
  e = c.d == 128 ? launch_rows<128>(c, cfg) : launch_rows<64>(c, cfg);
  if (e != cudaSuccess || staged) return e;
  gather_sums_kernel<<<c.units, kSelThreads, 0, s>>>(c);
  return cudaGetLastError();
}

}  // namespace kvc

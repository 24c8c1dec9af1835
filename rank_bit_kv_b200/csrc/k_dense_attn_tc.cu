// Attention over a dense bf16 cache for many query rows per KV head, on
// tcgen05: prefill with a window and sinks, and the shared part of a
// shared-prefix decode.  Output in bf16.
//
//   S = Q K^T (fp32, TMEM);  P = 2^(scale log2(e) S - m);  O += P V (fp32, TMEM)
//
// What bounds it is the tensor core together with the exponentials: a 128 x 128
// tile of scores takes 4 * 128^2 * d operations on the tensor core (1024 clocks
// at d = 128) and 128^2 exponentials (1024 clocks at 16 a clock).  So two score
// tiles ("streams") are in flight per CTA, and while the softmax of one runs on
// its four warps the tensor core works on the other:
//   warps 0-3, 4-7  softmax of stream 0 / 1, one thread per row: scores from TMEM,
//                   mask, maximum, exponentials, P back into TMEM over the scores
//   warp 8          issues the MMAs: S = Q K^T from shared memory, O += P V with P
//                   from TMEM
//   warp 9          loads 128-token tiles of K and V by TMA into a ring
// PAIR: the streams are two tiles of 128 query rows and share the K/V tiles.
// Otherwise (up to 128 rows, or too few blocks to fill the SMs) they are the
// same 128 rows over the even and the odd tiles, merged through shared memory.
//
// P is rounded to bf16, the output's own precision, as V's type asks (both
// operands of an MMA have one type); sums are taken before the rounding.
#include <cuda.h>
#include <math.h>

#include "dense_rows.cuh"
#include "tc_util.cuh"

namespace kvc {
namespace {

using namespace tc;

constexpr int kTM = 128;                 // query rows per stream
constexpr int kTN = 128;                 // tokens per tile
constexpr int kWarpMma = 8, kWarpTma = 9;
constexpr int kThreads = 320;
constexpr int kSoftThreads = 256;

template <int D>
struct Cfg {
  static constexpr int kHalfB = kTN * 128;               // 64 elements of 128 rows, 128-byte swizzle
  static constexpr int kTileB = kHalfB * (D / 64);       // a K, V or Q tile
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kSmem = (2 + kStages) * kTileB + 1024;
};

// TMEM columns: the scores of both streams (P over them), then their outputs.
constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int s) { return (uint32_t)s * kTN; }
template <int D>
__device__ __forceinline__ uint32_t col_o(int s) { return 2 * kTN + (uint32_t)s * D; }

constexpr uint32_t idesc_bf16(int n, int b_mn_major) {
  return idesc_f16(kTM, n, 0, b_mn_major) | (1u << 7) | (1u << 10);      // A and B are bf16
}

// 128-byte-swizzled operand tile (K-major: lbo unused).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
          "r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf2(float2 x) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D>
struct __align__(8) Bars {
  uint64_t q_full, full[Cfg<D>::kStages], empty[Cfg<D>::kStages];
  uint64_t s_full[2], p_full[2], o_done[2], drain;
  uint32_t tmem;
  int abort;
  float ml[kTM][2];                      // stream 1's maximum and sum
};

// The tiles of a CTA: range [0, a1) then [b0, b1) of the token span.
struct Tiles {
  TokenSpan sp;
  int n_a, first, n;
  __device__ __forceinline__ void at(int t, int& t0, int& nt) const {
    const int j = first + t;
    t0 = j < n_a ? j * kTN : sp.b0 + (j - n_a) * kTN;
    nt = min(kTN, (j < n_a ? sp.a1 : sp.b1) - t0);
  }
};

// Ring position of K tile t and V tile t of n: K runs `lead` tiles ahead of V
// (K0, V0, K1, V1 ... or K0, K1, V0, K2, V1 ...).
template <bool PAIR>
__device__ __forceinline__ int ring_k(int t) { return PAIR ? 2 * t : (t < 2 ? t : 2 * t - 1); }
template <bool PAIR>
__device__ __forceinline__ int ring_v(int t, int n) { return PAIR ? 2 * t + 1 : min(2 * t + 2, 2 * n - 1); }

template <int D, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    dense_attn_tc_kernel(const __grid_constant__ DenseAttn p, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D>;
  constexpr int RB = PAIR ? 2 * kTM : kTM;
  constexpr int NST = C::kStages;
  extern __shared__ uint8_t dsm_raw[];
  __shared__ Bars<D> bars;
  // swizzled tiles start on 1024-byte boundaries
  uint8_t* const dsm = dsm_raw + ((1024u - (smem_u32(dsm_raw) & 1023u)) & 1023u);
  uint8_t* const sm_q = dsm;
  uint8_t* const ring = dsm + 2 * C::kTileB;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % p.own.splits, ub = blockIdx.x / p.own.splits;
  const int u = ub / p.own.blocks, r0 = (ub % p.own.blocks) * RB;
  const int n_rows = min(RB, p.rows - r0);
  const int len = dense_len(p, u);
  // a kernel that merges with this one's partials may start
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int p_lo = dense_row_pos(p, len, r0), p_hi = dense_row_pos(p, len, r0 + n_rows - 1);
  Tiles tl;
  tl.sp = token_span(p_lo, p_hi, p.window, p.sinks);
  tl.n_a = (tl.sp.a1 + kTN - 1) / kTN;
  {
    const int all = tl.n_a + (tl.sp.b1 - tl.sp.b0 + kTN - 1) / kTN;
    const int per = (all + p.own.splits - 1) / p.own.splits;
    tl.first = min(all, split * per);
    tl.n = min(all, tl.first + per) - tl.first;
  }
  const int n = tl.n;
  volatile int* abort = &bars.abort;
  uint32_t* const err = p.err;
  // the error word is cleared by the first block; a wait gives up only much later
  if (p.clear_err && blockIdx.x == 0 && threadIdx.x == 0) *err = 0u;

  if (threadIdx.x == 0) {
    mbar_init(&bars.q_full, kSoftThreads);
    for (int i = 0; i < NST; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.s_full[s], 1);
      mbar_init(&bars.p_full[s], kTM);
      mbar_init(&bars.o_done[s], 1);
    }
    mbar_init(&bars.drain, 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&bars.tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;

  if (warp == kWarpTma) {
    // ---- K / V tiles into the ring
    if (lane == 0 && n > 0) {
      int pos = 0, issued = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* map, int t) {
        const int st = pos % NST;
        if (pos >= NST && !mbar_wait(&bars.empty[st], ((pos / NST) - 1) & 1, abort, err)) {
          ok = false;
          return;
        }
        int t0, nt;
        tl.at(t, t0, nt);
        mbar_arrive_expect_tx(&bars.full[st], C::kTileB);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tma_tile(smem_u32(ring + st * C::kTileB + h * C::kHalfB), map, 64 * h, t0, u, &bars.full[st]);
        ++pos;
        issued = pos;
      };
      constexpr int lead = PAIR ? 1 : 2;
      for (int t = 0; t < lead && t < n && ok; ++t) load(&map_k, t);
      for (int t = 0; t < n && ok; ++t) {
        load(&map_v, t);
        if (ok && t + lead < n) load(&map_k, t + lead);
      }
      if (!ok) {
        // copies in flight land before the block ends
        volatile int no_abort = 0;
        for (int q = issued > NST ? issued - NST : 0; q < issued; ++q)
          mbar_wait(&bars.full[q % NST], (q / NST) & 1, &no_abort, nullptr);
      }
    }
  } else if (warp == kWarpMma) {
    // ---- MMAs
    if (n > 0) {
      bool ok = __all_sync(0xffffffffu, mbar_wait(&bars.q_full, 0, abort, err));
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err));
      };
      auto qk = [&](int s, int t, bool first_use, bool last_use) {
        const int pos = ring_k<PAIR>(t), st = pos % NST;
        if (first_use) wait(&bars.full[st], (pos / NST) & 1);
        if (!ok) return;
        tc_fence_after();
        if (lane == 0) {
          int t0, nt;
          tl.at(t, t0, nt);
          const uint32_t id = idesc_bf16((nt + 15) & ~15, 0);
          const uint32_t qa = smem_u32(sm_q + (PAIR ? s * C::kTileB : 0));
          const uint32_t ka = smem_u32(ring + st * C::kTileB);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk / 4) * C::kHalfB + (kk % 4) * 32;
            mma_ss(tmem + col_s(s), desc_sw128(qa + off, 0, 1024), desc_sw128(ka + off, 0, 1024), id, kk > 0);
          }
          tc_commit(&bars.s_full[s]);
          if (last_use) tc_commit(&bars.empty[st]);
        }
        __syncwarp();
      };
      auto pv = [&](int s, int j, int t, bool first_use, bool last_use) {
        const int pos = ring_v<PAIR>(t, n), st = pos % NST;
        int t0, nt;
        tl.at(t, t0, nt);
        const int steps = (nt + 15) / 16;
        uint8_t* const vt = ring + st * C::kTileB;
        if (first_use) {
          wait(&bars.full[st], (pos / NST) & 1);
          if (!ok) return;
          if (nt & 15) {
            // rows behind the range, in its last 16: zero, whatever the cache holds there
            const int i0 = nt * 8, i1 = steps * 16 * 8;
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              for (int i = i0 + lane; i < i1; i += 32)
                *reinterpret_cast<uint4*>(vt + h * C::kHalfB + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        wait(&bars.p_full[s], j & 1);
        if (!ok) return;
        tc_fence_after();
        if (lane == 0) {
          constexpr uint32_t id = idesc_bf16(D, 1);
          const uint32_t va = smem_u32(vt);
          for (int ks = 0; ks < steps; ++ks)
            mma_ts(tmem + col_o<D>(s), tmem + col_s(s) + 8 * ks, desc_sw128(va + ks * 2048, C::kHalfB, 1024), id,
                   j > 0 || ks > 0);
          tc_commit(&bars.o_done[s]);
          if (last_use) tc_commit(&bars.empty[st]);
        }
        __syncwarp();
      };
      if (PAIR) {
        qk(0, 0, true, false);
        qk(1, 0, false, true);
        for (int t = 0; t < n && ok; ++t) {
          pv(0, t, t, true, false);
          if (t + 1 < n) qk(0, t + 1, true, false);
          pv(1, t, t, false, true);
          if (t + 1 < n) qk(1, t + 1, false, true);
        }
      } else {
        qk(0, 0, true, true);
        if (n > 1) qk(1, 1, true, true);
        for (int t = 0; t < n && ok; ++t) {
          pv(t & 1, t >> 1, t, true, true);
          if (t + 2 < n) qk(t & 1, t + 2, true, true);
        }
      }
      if (!ok && lane == 0) {
        // MMAs in flight end before the block frees its TMEM
        tc_commit(&bars.drain);
        volatile int no_abort = 0;
        mbar_wait(&bars.drain, 0, &no_abort, nullptr);
      }
    }
  } else {
    // ---- softmax warps
    const int s = warp >> 2;
    const int row = (warp & 3) * 32 + lane;              // row of the stream = TMEM lane
    const uint32_t tl_base = tmem + ((uint32_t)(warp & 3) << 21);
    if (n > 0) {
      // queries, 16 bytes a thread and step; zero past the block's rows
      constexpr int CH = D / 8;                          // 16-byte chunks of a row
      for (int i = threadIdx.x; i < RB * CH; i += kSoftThreads) {
        const int r = i / CH, c = i % CH;
        const bool has = r < n_rows;
        const __nv_bfloat16* src = p.q + dense_row_at(p, u, r0 + (has ? r : 0)) + c * 8;
        uint8_t* dst = sm_q + (r / kTM) * C::kTileB + (c / 8) * C::kHalfB + (r % kTM) * 128 + (((c & 7) ^ (r & 7)) << 4);
        cp_async16(dst, src, has ? 16 : 0);
      }
      cp_async_wait_all();
      fence_proxy_async_smem();
      mbar_arrive(&bars.q_full);
    }
    const int r = (PAIR ? s * kTM : 0) + row;            // row of the block
    const int pos = dense_row_pos(p, len, r0 + min(r, n_rows - 1));
    // positions of the stream's rows
    const int s_lo = PAIR ? dense_row_pos(p, len, r0 + min(s * kTM, n_rows - 1)) : p_lo;
    const int s_hi = PAIR ? dense_row_pos(p, len, r0 + min(s * kTM + kTM, n_rows) - 1) : p_hi;
    const int n_s = PAIR ? n : (n + 1 - s) / 2;
    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_s; ++j) {
      int t0, nt;
      tl.at(PAIR ? j : 2 * j + s, t0, nt);
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars.s_full[s], j & 1, abort, err)))) break;
      tc_fence_after();
      uint32_t x[4][32];
      const int chunks = (nt + 31) >> 5;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < chunks) tmem_ld32(tl_base + col_s(s) + 32 * c, x[c]);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 4; ++c) reg_fence(x[c]);
      // a tile that every row sees whole needs no mask
      if (nt < kTN || t0 + kTN - 1 > s_lo || !(t0 + kTN <= p.sinks || t0 > s_hi - p.window)) {
        const int hi = min(pos - t0, nt - 1), lo = pos - p.window + 1 - t0, sk = p.sinks - t0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int t = 32 * c + i;
            if (!(t <= hi && (t >= lo || t < sk))) x[c][i] = 0xff800000u;
          }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < chunks) {
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; ++i) m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(x[c][i]));
          mx = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
        }
      mx *= p.scale_log2;
      // the reference maximum is raised only by a score more than 2^8 above it
      if (__any_sync(0xffffffffu, mx > m_ref + 8.f)) {
        const float nm = fmaxf(m_ref, mx);
        const float a = nm == -INFINITY ? 1.f : ex2_approx(m_ref - nm);
        m_ref = nm;
        l *= a;
        if (j > 0) {
          // the last product is in the accumulators before they are rescaled
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars.o_done[s], (j - 1) & 1, abort, err)))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld16(tl_base + col_o<D>(s) + c, o);
            tmem_wait_ld();
            reg_fence(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
            tmem_st16(tl_base + col_o<D>(s) + c, o);
          }
          tmem_wait_st();
        }
      }
      const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
      const float2 neg2 = make_float2(neg, neg);
      float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < chunks) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 v = fma2(make_float2(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])), scale2, neg2);
            v.x = ex2_approx(v.x);
            v.y = ex2_approx(v.y);
            sum[i & 1] = add2(sum[i & 1], v);
            w[i] = pack_bf2(v);
          }
          tmem_st16(tl_base + col_s(s) + 16 * c, w);
        }
      sum[0] = add2(sum[0], sum[1]);
      l += sum[0].x + sum[0].y;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars.p_full[s]);
    }
    // ---- epilogue
    if (ok && n_s > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars.o_done[s], (n_s - 1) & 1, abort, err));
    tc_fence_after();
    float* const stage = reinterpret_cast<float*>(ring);  // [D][kTM]: the ring's loads are over
    if (!PAIR) {
      if (s == 1) {
        bars.ml[row][0] = m_ref;
        bars.ml[row][1] = l;
        // stream 0's products may still read the ring: wait for the last of them
        if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars.o_done[0], ((n + 1) / 2 - 1) & 1, abort, err));
        if (ok && n_s > 0) {
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld16(tl_base + col_o<D>(s) + c, o);
            tmem_wait_ld();
            reg_fence(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) stage[(c + i) * kTM + row] = __uint_as_float(o[i]);
          }
        }
      }
      named_bar(1, kSoftThreads);
    }
    if (ok && (PAIR || s == 0) && r - (r & 31) < n_rows) {
      float a0 = 1.f, a1 = 0.f;
      // a stream that saw nothing adds nothing
      const bool mine = !(m_ref == -INFINITY && l == 0.f);
      bool other = false;
      if (!PAIR) {
        const float m1 = bars.ml[row][0], l1 = bars.ml[row][1];
        other = n > 1 && !(m1 == -INFINITY && l1 == 0.f);
        if (other) {
          const float mx = fmaxf(m_ref, m1);
          if (m_ref != -INFINITY) a0 = exp2f(m_ref - mx);
          a1 = m1 == -INFINITY ? 1.f : exp2f(m1 - mx);
          m_ref = mx;
          l = (mine ? a0 * l : 0.f) + a1 * l1;
        }
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const size_t at = (size_t)blockIdx.x * RB + r;
      const long long out_at = dense_row_at(p, u, r0 + min(r, n_rows - 1));
      bool fine = true;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        tmem_ld16(tl_base + col_o<D>(s) + c, o);
        tmem_wait_ld();
        reg_fence(o);
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          f[i] = mine ? __uint_as_float(o[i]) * a0 : 0.f;
          if (other) f[i] = fmaf(a1, stage[(c + i) * kTM + row], f[i]);
          if (l == 0.f) f[i] = 0.f;
        }
        if (p.finish) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 v = make_float2(f[2 * i] * inv, f[2 * i + 1] * inv);
            fine = fine && fabsf(v.x) <= 3.4e38f && fabsf(v.y) <= 3.4e38f;
            w[i] = pack_bf2(v);
          }
          if (r < n_rows) {
            uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + out_at + c);
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        } else if (r < n_rows) {
          float4* dst = reinterpret_cast<float4*>(p.own.part + at * D + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        }
      }
      if (p.finish) {
        // rows that another row's NaN or infinity may have reached: from the definition
        if (p.n_q > 1) {
          unsigned bad = __ballot_sync(0xffffffffu, !fine && r < n_rows);
          __syncwarp();
          while (bad) {
            const int b = __ffs(bad) - 1;
            bad &= bad - 1;
            float o[D / 32];
            const int rr = r0 + r - lane + b;
            dense_row_alone<D>(p, u, rr, o);
            dense_put_row<D>(p, u, rr, o);
          }
        }
      } else if (r < n_rows) {
        *reinterpret_cast<float2*>(p.own.ml + 2 * at) = make_float2(m_ref, l);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// The keys or values of a problem as a 3-D tensor (d, tokens, units); tokens
// past the capacity read as zero.
cudaError_t tensor_map(CUtensorMap* map, const DenseAttn& p, const __nv_bfloat16* base) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
            cudaSuccess || found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (Encode)f;
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)p.d, (cuuint64_t)p.tmax, (cuuint64_t)p.units};
  const cuuint64_t strides[2] = {(cuuint64_t)p.d * 2, (cuuint64_t)p.d * 2 * p.tmax};
  const cuuint32_t box[3] = {64, kTN, 1}, step[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(base), dims, strides,
                            box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, bool PAIR>
cudaError_t launch(const DenseAttn& p, cudaStream_t s) {
  CUtensorMap mk, mv;
  cudaError_t e = tensor_map(&mk, p, p.k);
  if (e == cudaSuccess) e = tensor_map(&mv, p, p.v);
  if (e != cudaSuccess) return e;
  auto* f = dense_attn_tc_kernel<D, PAIR>;
  e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  f<<<(unsigned)((long long)p.units * p.own.blocks * p.own.splits), kThreads, Cfg<D>::kSmem, s>>>(p, mk, mv);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dense_attn_tc(const DenseAttn& p, cudaStream_t s) {
  const bool pair = p.own.row_block == 2 * kTM;
  if (p.d == 128) return pair ? launch<128, true>(p, s) : launch<128, false>(p, s);
  return pair ? launch<64, true>(p, s) : launch<64, false>(p, s);
}

}  // namespace kvc

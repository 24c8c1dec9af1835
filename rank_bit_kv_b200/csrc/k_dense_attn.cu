// Attention over a dense bf16 cache for few query rows per KV head: window
// attention of one or a few tokens, decode with accumulated weights and the
// two parts of a shared-prefix decode.
//
//   o_r = sum_t 2^(s_rt - m_r) v_t / sum_t 2^(s_rt - m_r),
//   s_rt = scale log2(e) q_r . k_t over the tokens t that row r sees
//
// What bounds it is the cache stream: 4 d bytes per token and KV head against
// 4 d operations per row.  So every warp streams 16-token tiles (keys and
// values) through its own cp.async ring, with no block barrier in the loop;
// the rows of a KV head (query heads x query tokens) are the N dimension of the
// MMAs, so a tile is read once for all of them.  A block's warps take the
// tiles of its token range in turn, merge in shared memory, and the block
// writes one partial per row, or the output where nothing is left to merge.
#include <math.h>

#include "dense_rows.cuh"
#include "tc_util.cuh"

namespace kvc {
namespace {

using namespace tc;

constexpr int kTok = 16;                 // tokens per tile
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

enum Mode { kOneToken = 0, kManyTokens = 1, kScores = 2 };

template <int D>
struct Geo {
  static constexpr int kRowB = 2 * D + 16;               // shared bytes per token row (no bank conflicts)
  static constexpr int kTileB = kTok * kRowB;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kWarpB = kStages * 2 * kTileB;
  static constexpr int kSmem = kWarps * kWarpB;
};

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (x, y) rounded to bf16x2; x and y become what the rounding left over.
__device__ __forceinline__ uint32_t split_bf2(float& x, float& y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  x -= __low2float(h);
  y -= __high2float(h);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ bool sees(int t, int pos, int window, int sinks) {
  return t <= pos && (t < sinks || t > pos - window);
}

// NT: 8-row tiles of a row block.  EXACT (fp32 output): the probabilities
// enter the value product in three bf16 parts (24 bits), and each tile's product
// is formed from zero and added in fp32 arithmetic -- the MMA's own accumulation
// truncates, which over a long context adds up to more than fp32's rounding.
// Otherwise two parts (16 bits, well below the output's 8), accumulated by the MMA.
template <int D, int NT, bool EXACT, int MODE>
__global__ void __launch_bounds__(kThreads, 1) dense_attn_kernel(const __grid_constant__ DenseAttn p) {
  using G = Geo<D>;
  constexpr int RB = 8 * NT;
  constexpr int KS = D / 16;             // k-steps of the scores, m-tiles of the values
  constexpr int CPR = D / 8;             // 16-byte chunks per row
  extern __shared__ __align__(128) uint8_t dsm[];
  __shared__ float sm_ml[kWarps][RB][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c4 = lane & 3;
  const int split = blockIdx.x % p.splits, ub = blockIdx.x / p.splits;
  const int u = ub / p.blocks, r0 = (ub % p.blocks) * RB;
  const int n_rows = min(RB, p.rows - r0);
  const int len = dense_len(p, u);

  // positions of this block's rows (ascending)
  int p_lo = len - 1, p_hi = len - 1;
  if (MODE == kManyTokens) p_lo = dense_row_pos(p, len, r0), p_hi = dense_row_pos(p, len, r0 + n_rows - 1);
  const TokenSpan sp = token_span(p_lo, p_hi, p.window, p.sinks);
  const int n_a = (sp.a1 + kTok - 1) / kTok;
  const int n_tiles = n_a + (sp.b1 - sp.b0 + kTok - 1) / kTok;
  const int per = (n_tiles + p.splits - 1) / p.splits;
  const int j_end = min(n_tiles, (split + 1) * per);
  const int j_first = split * per + warp;          // this warp: every kWarps-th tile from here
  const int n_mine = j_first < j_end ? (j_end - j_first + kWarps - 1) / kWarps : 0;

  uint8_t* ring = dsm + warp * G::kWarpB;
  const uint8_t* const kb = reinterpret_cast<const uint8_t*>(p.k + (size_t)u * p.tmax * D);
  const uint8_t* const vb = reinterpret_cast<const uint8_t*>(p.v + (size_t)u * p.tmax * D);
  auto tile_at = [&](int i, int& t0, int& nt) {
    const int j = j_first + i * kWarps;
    t0 = j < n_a ? j * kTok : sp.b0 + (j - n_a) * kTok;
    nt = min(kTok, (j < n_a ? sp.a1 : sp.b1) - t0);
  };
  // copy tile i of this warp into its ring stage (rows past the range are zero)
  auto issue = [&](int i) {
    int t0, nt;
    tile_at(i, t0, nt);
    const uint8_t* ks = kb + (size_t)t0 * (2 * D);
    const uint8_t* vs = vb + (size_t)t0 * (2 * D);
    uint8_t* st = ring + (i % G::kStages) * (2 * G::kTileB);
#pragma unroll
    for (int x = 0; x < kTok * CPR / 32; ++x) {
      const int c = lane + 32 * x, r = c / CPR, col = c % CPR;
      const int nb = r < nt ? 16 : 0;
      const size_t go = (size_t)(r < nt ? r : 0) * (2 * D) + col * 16;
      cp_async16(st + r * G::kRowB + col * 16, ks + go, nb);
      cp_async16(st + G::kTileB + r * G::kRowB + col * 16, vs + go, nb);
    }
  };
#pragma unroll
  for (int i = 0; i < G::kStages - 1; ++i) {
    if (i < n_mine) issue(i);
    cp_commit();
  }

  // queries as B fragments (zero past the block's rows)
  uint32_t qb[KS][NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + g;
    const __nv_bfloat16* qq = p.q + dense_row_at(p, u, r0 + (r < n_rows ? r : 0));
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      qb[kk][nt][0] = r < n_rows ? *reinterpret_cast<const uint32_t*>(qq + 16 * kk + 2 * c4) : 0u;
      qb[kk][nt][1] = r < n_rows ? *reinterpret_cast<const uint32_t*>(qq + 16 * kk + 8 + 2 * c4) : 0u;
    }
  }
  int pos[NT][2];
  if (MODE == kManyTokens) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) pos[nt][e] = dense_row_pos(p, len, min(r0 + 8 * nt + 2 * c4 + e, p.rows - 1));
  }
  float m_ref[NT][2], l_sum[NT][2], acc[KS][NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m_ref[nt][0] = m_ref[nt][1] = -INFINITY;
    l_sum[nt][0] = l_sum[nt][1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.f;
  }

  for (int i = 0; i < n_mine; ++i) {
    if (i + G::kStages - 1 < n_mine) issue(i + G::kStages - 1);
    cp_commit();
    cp_wait<G::kStages - 1>();
    __syncwarp();
    int t0, nt_tok;
    tile_at(i, t0, nt_tok);
    const uint8_t* kt = ring + (i % G::kStages) * (2 * G::kTileB);
    const uint8_t* vt = kt + G::kTileB;
    // ---- scores: rows g, g + 8 = tokens; columns 2 c4, 2 c4 + 1 of n-tile nt = query rows
    float s[NT][4];
    {
      float sb[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = sb[nt][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        uint32_t a[4];
        ldmatrix_x4(a, kt + (lane & 15) * G::kRowB + (2 * kk + (lane >> 4)) * 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (NT < 4 && (kk & 1)) mma_bf16(sb[nt], a, qb[kk][nt][0], qb[kk][nt][1]);
          else mma_bf16(s[nt], a, qb[kk][nt][0], qb[kk][nt][1]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = (NT < 4 ? s[nt][e] + sb[nt][e] : s[nt][e]) * p.scale_log2;
    }
    if (MODE == kManyTokens) {
      // a tile that every row sees whole needs no mask
      const int t1 = t0 + kTok - 1;
      if (nt_tok < kTok || t1 > p_lo || !(t1 < p.sinks || t0 > p_hi - p.window)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tt = g + 8 * (e >> 1);
            if (tt >= nt_tok || !sees(t0 + tt, pos[nt][e & 1], p.window, p.sinks)) s[nt][e] = -INFINITY;
          }
      }
    } else if (nt_tok < kTok) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (g + 8 * (e >> 1) >= nt_tok) s[nt][e] = -INFINITY;
    }
    if (MODE == kScores) {
      float* sc = p.scores + ((size_t)u * p.n_tokens + t0) * p.rows + r0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int tt = g + 8 * h, r = 8 * nt + 2 * c4;
          if (tt < nt_tok) {
            float* dst = sc + (size_t)tt * p.rows + r;
            if (r + 1 < n_rows && (p.rows & 1) == 0) {
              *reinterpret_cast<float2*>(dst) = make_float2(s[nt][2 * h], s[nt][2 * h + 1]);
            } else {
              if (r < n_rows) dst[0] = s[nt][2 * h];
              if (r + 1 < n_rows) dst[1] = s[nt][2 * h + 1];
            }
          }
        }
    }
    // ---- online softmax: the reference maximum is raised only by a score more
    // than 2^8 above it, so that the accumulators are rarely rescaled
    bool need = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) need = need || fmaxf(s[nt][e], s[nt][2 + e]) > m_ref[nt][e] + 8.f;
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(s[nt][e], s[nt][2 + e]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const float nm = fmaxf(m_ref[nt][e], mx);
          const float a = nm == -INFINITY ? 0.f : ex2_approx(m_ref[nt][e] - nm);
          m_ref[nt][e] = nm;
          l_sum[nt][e] *= a;
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            acc[mt][nt][e] *= a;
            acc[mt][nt][2 + e] *= a;
          }
        }
    }
    uint32_t pb[NT][EXACT ? 3 : 2][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = s[nt][e] == -INFINITY ? 0.f : ex2_approx(s[nt][e] - m_ref[nt][e & 1]);
      l_sum[nt][0] += w[0] + w[2];
      l_sum[nt][1] += w[1] + w[3];
#pragma unroll
      for (int part = 0; part < (EXACT ? 3 : 2); ++part) {
        pb[nt][part][0] = movmatrix_trans(split_bf2(w[0], w[1]));
        pb[nt][part][1] = movmatrix_trans(split_bf2(w[2], w[3]));
      }
    }
    // ---- acc^T (dim x row) += V^T (dim x token) P (token x row)
    const int tok = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      uint32_t a[4];
      ldmatrix_x4_trans(a, vt + tok * G::kRowB + (2 * mt + ((lane >> 3) & 1)) * 16);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (EXACT) {
          float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int part = 2; part >= 0; --part) mma_bf16(f, a, pb[nt][part % (EXACT ? 3 : 2)][0], pb[nt][part % (EXACT ? 3 : 2)][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[mt][nt][e] += f[e];
        } else {
          mma_bf16(acc[mt][nt], a, pb[nt][0][0], pb[nt][0][1]);
          mma_bf16(acc[mt][nt], a, pb[nt][1][0], pb[nt][1][1]);
        }
      }
    }
    __syncwarp();                        // this stage is refilled next iteration
  }
  cp_wait<0>();

  // ---- merge the warps: accumulators to shared memory as [warp][row][d]
  constexpr int RS = D + 4;              // floats per staged row
  static_assert(kWarps * RB * RS * 4 <= G::kSmem, "staged accumulators fit the ring");
  float* const stage = reinterpret_cast<float*>(dsm);
  __syncthreads();                       // every warp is done with its ring
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = l_sum[nt][e];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      const int r = 8 * nt + 2 * c4 + e;
      float* dst = stage + (warp * RB + r) * RS;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        dst[16 * mt + g] = acc[mt][nt][e];
        dst[16 * mt + g + 8] = acc[mt][nt][2 + e];
      }
      if (g == 0) {
        sm_ml[warp][r][0] = m_ref[nt][e];
        sm_ml[warp][r][1] = l;
      }
    }
  __syncthreads();
  for (int r = warp; r < n_rows; r += kWarps) {
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm_ml[w][r][0]);
    float l = 0.f, o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = sm_ml[w][r][0];
      // a warp without a visible token holds zeros; NaN scores leave mw at
      // -inf with a NaN sum, which must reach the result
      const float lw = sm_ml[w][r][1];
      if (mw == -INFINITY && lw == 0.f) continue;
      const float a = mw == -INFINITY ? 1.f : exp2f(mw - mx);
      l = fmaf(a, lw, l);
      const float* src = stage + (w * RB + r) * RS + lane;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = fmaf(a, src[32 * i], o[i]);
    }
    if (p.direct) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = l == 0.f ? 0.f : o[i] / l;
      dense_put_row<D>(p, u, r0 + r, o);
    } else {
      const size_t at = (size_t)blockIdx.x * RB + r;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) p.part[at * D + lane + 32 * i] = o[i];
      if (lane == 0) *reinterpret_cast<float2*>(p.ml + 2 * at) = make_float2(mx, l);
    }
  }
}

// ---------------------------------------------------------------- merge

// Row r's split partials in a set: first index, and how many.
struct PartRef {
  const float* part;
  const float* ml;
  size_t first;                          // partial of split 0; split s is s * step further
  int step, n;
};

__device__ __forceinline__ PartRef part_ref(const DenseAttn& p, int u, int r) {
  PartRef f;
  f.part = p.part;
  f.ml = p.ml;
  f.first = ((size_t)u * p.blocks + r / p.row_block) * p.splits * p.row_block + r % p.row_block;
  f.step = p.row_block;
  f.n = p.splits;
  return f;
}

constexpr int kCWarps = 4;

// The largest maximum and the merged sum of a row's partials, by one warp.
__device__ __forceinline__ void merge_ml(const PartRef* set, int n_sets, float& mx, float& l) {
  const int lane = threadIdx.x & 31;
  mx = -INFINITY;
  for (int k = 0; k < n_sets; ++k)
    for (int s = lane; s < set[k].n; s += 32) mx = fmaxf(mx, set[k].ml[2 * (set[k].first + (size_t)s * set[k].step)]);
  mx = warp_max(mx);
  l = 0.f;
  for (int k = 0; k < n_sets; ++k)
    for (int s = lane; s < set[k].n; s += 32) {
      const float2 x = *reinterpret_cast<const float2*>(set[k].ml + 2 * (set[k].first + (size_t)s * set[k].step));
      if (x.x == -INFINITY && x.y == 0.f) continue;
      l = fmaf(x.x == -INFINITY ? 1.f : exp2f(x.x - mx), x.y, l);
    }
  l = warp_sum(l);
}

// One output row by the kCWarps warps of a block: warp w takes every
// kCWarps-th partial, then their sums are added.
template <int D>
__device__ void merge_row(const DenseAttn& p, int u, int r, const PartRef* set, int n_sets,
                          float (*red)[D]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float mx, l, o[D / 32];
  merge_ml(set, n_sets, mx, l);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  for (int k = 0; k < n_sets; ++k)
#pragma unroll 4
    for (int s = warp; s < set[k].n; s += kCWarps) {
      const size_t at = set[k].first + (size_t)s * set[k].step;
      const float2 x = *reinterpret_cast<const float2*>(set[k].ml + 2 * at);
      if (x.x == -INFINITY && x.y == 0.f) continue;
      const float a = x.x == -INFINITY ? 1.f : exp2f(x.x - mx);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = fmaf(a, set[k].part[at * D + lane + 32 * i], o[i]);
    }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) red[warp][lane + 32 * i] = o[i];
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kCWarps; ++w) t += red[w][lane + 32 * i];
      o[i] = l == 0.f ? 0.f : t / l;
    }
    dense_put_row<D>(p, u, r, o);
  }
}

template <int D>
__global__ void __launch_bounds__(32 * kCWarps) dense_combine_kernel(const __grid_constant__ DenseAttn p,
                                                                     const __grid_constant__ DenseAttn pre,
                                                                     int has_prefix) {
  __shared__ float red[kCWarps][D];
  const int u = blockIdx.x / p.rows, r = blockIdx.x % p.rows;
  PartRef set[2];
  set[0] = part_ref(p, u, r);
  if (has_prefix) {
    // the prefix's unit is the KV head, its rows run over the batch's rows too
    const int row = u / p.Hkv, batch = p.units / pre.units, h = u % p.Hkv;
    set[1] = part_ref(pre, (row / batch) * p.Hkv + h, (row % batch) * p.rows + r);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  merge_row<D>(p, u, r, set, has_prefix ? 2 : 1, red);
}

// Blocks of unit u: block c < rows merges output row c (and further rows in
// turn where there are more rows than blocks); every block adds the weights of
// its tokens.
constexpr int kAccTok = 1024;            // tokens per block

template <int D>
__global__ void __launch_bounds__(32 * kCWarps) dense_accum_kernel(const __grid_constant__ DenseAttn p,
                                                                   float* weights, int chunks) {
  extern __shared__ float2 sm_row[];     // per row: maximum, 1 / sum
  __shared__ float red[kCWarps][D];
  const int u = blockIdx.x / chunks, c = blockIdx.x % chunks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int r = c; r < p.rows; r += chunks) {
    const PartRef set = part_ref(p, u, r);
    merge_row<D>(p, u, r, &set, 1, red);
    __syncthreads();
  }
  const int len = dense_len(p, u);
  if (c * kAccTok >= len) return;
  for (int r = warp; r < p.rows; r += kCWarps) {
    const PartRef set = part_ref(p, u, r);
    float mx, l;
    merge_ml(&set, 1, mx, l);
    if (lane == 0) sm_row[r] = make_float2(mx, 1.f / l);
  }
  __syncthreads();
  const int end = min(len, (c + 1) * kAccTok);
  for (int t = c * kAccTok + threadIdx.x; t < end; t += 32 * kCWarps) {
    const float* sc = p.scores + ((size_t)u * p.n_tokens + t) * p.rows;
    float w = 0.f;
    for (int r = 0; r < p.rows; ++r) {
      const float2 x = sm_row[r];
      w = fmaf(exp2f(sc[r] - x.x), x.y, w);
    }
    weights[(size_t)u * p.tmax + t] += w;
  }
}

template <int D, int NT, bool EXACT, int MODE>
cudaError_t launch_one(const DenseAttn& p, cudaLaunchConfig_t& cfg) {
  auto* f = dense_attn_kernel<D, NT, EXACT, MODE>;
  const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kSmem);
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = Geo<D>::kSmem;
  return cudaLaunchKernelEx(&cfg, f, p);
}

template <int D, int NT>
cudaError_t launch_nt(const DenseAttn& p, cudaLaunchConfig_t& cfg) {
  const int mode = p.scores ? kScores : p.n_q > 1 ? kManyTokens : kOneToken;
  if (p.out_bf16) {
    if (mode == kScores) return launch_one<D, NT, false, kScores>(p, cfg);
    if (mode == kManyTokens) return launch_one<D, NT, false, kManyTokens>(p, cfg);
    return launch_one<D, NT, false, kOneToken>(p, cfg);
  }
  if (mode == kScores) return launch_one<D, NT, true, kScores>(p, cfg);
  if (mode == kManyTokens) return launch_one<D, NT, true, kManyTokens>(p, cfg);
  return launch_one<D, NT, true, kOneToken>(p, cfg);
}

template <int D>
cudaError_t launch_d(const DenseAttn& p, cudaLaunchConfig_t& cfg) {
  if (p.row_block == 8) return launch_nt<D, 1>(p, cfg);
  if (p.row_block == 16) return launch_nt<D, 2>(p, cfg);
  return launch_nt<D, 4>(p, cfg);
}

}  // namespace

// The kernel and the split of a problem's tokens.
//
// Warp-level kernel: blocks of up to 32 rows, one block per SM at a time; enough
// splits for every SM, none with fewer tiles than warps; where the blocks alone
// exceed the SMs, as few splits as fill whole waves to nine tenths.
//
// tcgen05 kernel: bf16 output and at least kTensorRows rows per KV head.  256 rows
// per block where rows and tokens give every SM a block, 128 otherwise; splits of
// at least two tiles per score stream up to one block per SM.
DensePlan dense_plan(int units, int rows, long long tokens, int out_bf16) {
  DensePlan f;
  if (out_bf16 && rows >= kTensorRows) {
    const long long tiles = (tokens + 127) / 128, wide = (long long)units * ((rows + 255) / 256);
    f.tensor = 1;
    f.row_block = rows > 128 && wide * (tiles / 2 > 1 ? tiles / 2 : 1) >= kNumSMs ? 256 : 128;
    f.blocks = (rows + f.row_block - 1) / f.row_block;
    const long long ctas = (long long)units * f.blocks, most = tiles / (f.row_block == 256 ? 2 : 4);
    long long s = kNumSMs / ctas;
    s = s < most ? s : most;
    if (s > 1) {
      const long long per = (tiles + s - 1) / s;
      s = (tiles + per - 1) / per;
    }
    f.splits = s > 1 ? (int)s : 1;
    return f;
  }
  f.tensor = 0;
  f.row_block = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
  f.blocks = (rows + f.row_block - 1) / f.row_block;
  const long long blocks = (long long)units * f.blocks;
  const long long most = (tokens + kTok * kWarps - 1) / (kTok * kWarps);
  long long best = 1;
  double best_fill = 0.;
  for (long long s = 1; s <= most && s <= kNumSMs; ++s) {
    const long long waves = (blocks * s + kNumSMs - 1) / kNumSMs;
    const double fill = (double)(blocks * s) / (double)(waves * kNumSMs);
    if (fill > best_fill + 0.02) best = s, best_fill = fill;
    if (fill >= 0.9 || blocks * s > kWaves * kNumSMs) break;
  }
  f.splits = (int)best;
  return f;
}

// Row slots that the partials take in any call of up to `tokens` tokens and, with
// `direct`, of up to `rows` rows (a call of one split then writes its output and
// needs none).
long long dense_part_rows(long long units, long long rows, long long tokens, int out_bf16, bool direct) {
  const long long tiles = tokens > 128 ? (tokens + 127) / 128 : 1;
  if (out_bf16 && rows >= kTensorRows) {
    // splits only while the blocks do not fill the SMs
    const long long wide = units * ((rows + 255) / 256);
    if (wide >= kNumSMs && !direct) return wide * 256;
    return 256 * (wide * tiles < kNumSMs ? wide * tiles : kNumSMs);
  }
  // splits until the blocks pass kWaves waves, and none where they do without
  const int rb = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
  const long long nb = units * ((rows + rb - 1) / rb);
  if (nb > kWaves * kNumSMs && !direct) return nb * rb;
  const long long most = (nb < kWaves * kNumSMs ? nb : kWaves * kNumSMs) + kWaves * kNumSMs;
  return rb * (nb * tiles < most ? nb * tiles : most);
}

cudaError_t launch_dense_attn(const DenseAttn& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p.units * p.blocks * p.splits));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  if (p.tensor) return launch_dense_attn_tc(p, s);
  return p.d == 128 ? launch_d<128>(p, cfg) : launch_d<64>(p, cfg);
}

static void dependent(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr) {
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

cudaError_t launch_dense_combine(const DenseAttn& p, const DenseAttn* prefix, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)((long long)p.units * p.rows));
  cfg.blockDim = dim3(32 * kCWarps);
  cfg.stream = s;
  dependent(cfg, attr);
  const DenseAttn& pre = prefix ? *prefix : p;
  if (p.d == 128) return cudaLaunchKernelEx(&cfg, dense_combine_kernel<128>, p, pre, prefix ? 1 : 0);
  return cudaLaunchKernelEx(&cfg, dense_combine_kernel<64>, p, pre, prefix ? 1 : 0);
}

cudaError_t launch_dense_accum(const DenseAttn& p, float* weights, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  const int chunks = (p.n_tokens + kAccTok - 1) / kAccTok;
  cfg.gridDim = dim3((unsigned)((long long)p.units * (chunks > 0 ? chunks : 1)));
  cfg.blockDim = dim3(32 * kCWarps);
  cfg.dynamicSmemBytes = (size_t)p.rows * sizeof(float2);
  cfg.stream = s;
  dependent(cfg, attr);
  if (p.d == 128) return cudaLaunchKernelEx(&cfg, dense_accum_kernel<128>, p, weights, chunks > 0 ? chunks : 1);
  return cudaLaunchKernelEx(&cfg, dense_accum_kernel<64>, p, weights, chunks > 0 ? chunks : 1);
}

}  // namespace kvc

// Output rows of the dense-cache attention kernels.
#pragma once

#include <math.h>

#include "dense_attn.h"
#include "kvc_device.cuh"

namespace kvc {

// A row of D values over a warp: lane holds E = D / 32 neighbours, dims lane * E + i.
template <int E>
__device__ __forceinline__ void load_row(const float* row, float (&x)[E]) {
  static_assert(E == 2 || E == 4, "");
  const float* at = row + (threadIdx.x & 31) * E;
  if (E == 4) {
    const float4 v = *reinterpret_cast<const float4*>(at);
    x[0] = v.x, x[1] = v.y, x[E - 2] = v.z, x[E - 1] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(at);
    x[0] = v.x, x[1] = v.y;
  }
}
template <int E>
__device__ __forceinline__ void store_row(float* row, const float (&x)[E]) {
  float* at = row + (threadIdx.x & 31) * E;
  if (E == 4) *reinterpret_cast<float4*>(at) = make_float4(x[0], x[1], x[E - 2], x[E - 1]);
  else *reinterpret_cast<float2*>(at) = make_float2(x[0], x[1]);
}
template <int E>
__device__ __forceinline__ void load_row(const __nv_bfloat16* row, float (&x)[E]) {
  const __nv_bfloat162* at = reinterpret_cast<const __nv_bfloat162*>(row + (threadIdx.x & 31) * E);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const __nv_bfloat162 v = at[i];
    x[2 * i] = __low2float(v), x[2 * i + 1] = __high2float(v);
  }
}
template <int E>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, const float (&x)[E]) {
  __nv_bfloat162* at = reinterpret_cast<__nv_bfloat162*>(row + (threadIdx.x & 31) * E);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) at[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
}

// One output row from its definition, by one warp, reading only the tokens the
// row sees.  Taken for a row of a several-token call whose result is not
// finite: a NaN or infinite value of a token that the row does not see, but
// another row of its tile does, enters the tile product as 0 * NaN.
template <int D>
__device__ void dense_row_alone(const DenseAttn& p, int u, int r, float (&o)[D / 32]) {
  constexpr int E = D / 32;
  const int pos = dense_row_pos(p, dense_len(p, u), r);
  float q[E];
  load_row<E>(p.q + dense_row_at(p, u, r), q);
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] *= p.scale_log2;
    o[i] = 0.f;
  }
  const TokenSpan sp = token_span(pos, pos, p.window, p.sinks);
  const size_t row0 = (size_t)u * p.tmax;
  float m = -INFINITY, l = 0.f;
  for (int part = 0; part < 2; ++part) {
    const int end = part ? sp.b1 : sp.a1;
#pragma unroll 4
    for (int t = part ? sp.b0 : 0; t < end; ++t) {
      float k[E], v[E], x = 0.f;
      load_row<E>(p.k + (row0 + t) * D, k);
      load_row<E>(p.v + (row0 + t) * D, v);
#pragma unroll
      for (int i = 0; i < E; ++i) x = fmaf(q[i], k[i], x);
      x = warp_sum(x);
      const float nm = fmaxf(m, x);
      const float a = m == -INFINITY ? 0.f : exp2f(m - nm);
      const float w = x == -INFINITY ? 0.f : exp2f(x - nm);
      l = l * a + w;
#pragma unroll
      for (int i = 0; i < E; ++i) o[i] = o[i] * a + w * v[i];
      m = nm;
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = l == 0.f ? 0.f : o[i] / l;
}

// Write a finished row.
template <int D>
__device__ __forceinline__ void dense_put_row(const DenseAttn& p, int u, int r, float (&o)[D / 32]) {
  if (p.n_q > 1) {
    bool fine = true;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) fine = fine && fabsf(o[i]) <= 3.4e38f;
    if (!__all_sync(0xffffffffu, fine)) dense_row_alone<D>(p, u, r, o);
  }
  const long long at = dense_row_at(p, u, r);
  if (p.out_bf16) store_row(reinterpret_cast<__nv_bfloat16*>(p.out) + at, o);
  else store_row(reinterpret_cast<float*>(p.out) + at, o);
}

}  // namespace kvc

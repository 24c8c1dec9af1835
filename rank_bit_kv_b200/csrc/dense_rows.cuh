// Output rows of the dense-cache attention kernels.
#pragma once

#include <math.h>

#include "dense_attn.h"
#include "kvc_device.cuh"

namespace kvc {

// One output row from its definition, by one warp, reading only the tokens the
// row sees.  Taken for a row of a several-token call whose result is not
// finite: a NaN or infinite value of a token that the row does not see, but
// another row of its tile does, enters the tile product as 0 * NaN.
template <int D>
__device__ void dense_row_alone(const DenseAttn& p, int u, int r, float (&o)[D / 32]) {
  const int lane = threadIdx.x & 31;
  const int pos = dense_row_pos(p, dense_len(p, u), r);
  const __nv_bfloat16* qr = p.q + dense_row_at(p, u, r);
  float qv[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    qv[i] = bf2f(qr[lane + 32 * i]) * p.scale_log2;
    o[i] = 0.f;
  }
  const TokenSpan sp = token_span(pos, pos, p.window, p.sinks);
  float m = -INFINITY, l = 0.f;
  for (int t = sp.a1 ? 0 : sp.b0; t < sp.b1; t = (t + 1 == sp.a1) ? sp.b0 : t + 1) {
    const size_t row = ((size_t)u * p.tmax + t) * D;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) x = fmaf(qv[i], bf2f(p.k[row + lane + 32 * i]), x);
    x = warp_sum(x);
    const float nm = fmaxf(m, x);
    const float a = m == -INFINITY ? 0.f : exp2f(m - nm);
    const float w = x == -INFINITY ? 0.f : exp2f(x - nm);
    l = l * a + w;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = o[i] * a + w * bf2f(p.v[row + lane + 32 * i]);
    m = nm;
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = l == 0.f ? 0.f : o[i] / l;
}

// Write a finished row (value i of lane `lane` is dim lane + 32 i).
template <int D>
__device__ __forceinline__ void dense_put_row(const DenseAttn& p, int u, int r, float (&o)[D / 32]) {
  const int lane = threadIdx.x & 31;
  if (p.n_q > 1) {
    bool fine = true;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) fine = fine && fabsf(o[i]) <= 3.4e38f;
    if (!__all_sync(0xffffffffu, fine)) dense_row_alone<D>(p, u, r, o);
  }
  const long long at = dense_row_at(p, u, r);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    if (p.out_bf16) reinterpret_cast<__nv_bfloat16*>(p.out)[at + lane + 32 * i] = __float2bfloat16_rn(o[i]);
    else reinterpret_cast<float*>(p.out)[at + lane + 32 * i] = o[i];
  }
}

}  // namespace kvc

// The seam between two blocks of linears: the norm after a block, its gate, the scaled residual sum and the norm before
// the next block in one pass over the tokens, and its backward. With G the token's gate row, a = res_scale:
//   r_y = (mean(y^2) + eps)^(-1/2),  h' = a h + G (r_y y w_post),  r_h = (mean(h'^2) + eps)^(-1/2),  x = r_h h' w_pre
// and, with n = r_h h', u = dx w_pre, b = r_y y (gradients of h', x in; of h, y, G, w_post, w_pre out):
//   t = dh' + r_h (u - n mean(u n)),  dh = a t,  dw_pre = sum dx n,
//   v = t G w_post,  dy = r_y (v - b mean(v b)),  dw_post = sum t G b,  dG = sum over the row's tokens of t w_post b.
#include <algorithm>

#include "../../include/poet.h"
#include "internal.h"

namespace poet {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = 0.f;
  for (int i = 0; i < kThreads / 64; ++i) r += red[i];
  __syncthreads();
  return r;
}

template <class TR, class TA>
__global__ __launch_bounds__(kThreads) void k_norm_fwd(const NormArgs a) {
  __shared__ float red[kThreads / 64];
  const int64_t t = blockIdx.x;
  const TR* h = (const TR*)a.h + t * a.ldh;
  TR* ho = a.h_out ? (TR*)a.h_out + t * a.ldh : nullptr;
  const TA* y = a.y ? (const TA*)a.y + t * a.ldy : nullptr;
  const TA* g = a.gate ? (const TA*)a.gate + t / a.gate_tokens * a.ldg : nullptr;
  float ry = 1.f;
  if (a.w_post) {
    float s = 0.f;
    for (int j = threadIdx.x; j < a.d; j += kThreads) { const float v = (float)y[j]; s += v * v; }
    ry = 1.f / sqrtf(block_sum(s, red) / a.d + a.eps);
  }
  float s = 0.f;
  for (int j = threadIdx.x; j < a.d; j += kThreads) {
    float v = (float)h[j];
    if (y) {
      float r = (float)y[j];
      if (a.w_post) r = r * ry * a.w_post[j];
      if (g) r *= (float)g[j];
      const TR o = (TR)(v * a.res_scale + r);
      ho[j] = o;
      v = (float)o;
    }
    s += v * v;
  }
  const float rh = a.x ? 1.f / sqrtf(block_sum(s, red) / a.d + a.eps) : 0.f;
  if (a.x) {
    const TR* src = ho ? ho : h;
    TA* x = (TA*)a.x + t * a.ldx;
    for (int j = threadIdx.x; j < a.d; j += kThreads) x[j] = (TA)((float)src[j] * rh * a.w_pre[j]);
  }
  if (threadIdx.x == 0) { a.rstd[2 * t] = ry; a.rstd[2 * t + 1] = rh; }
}

// the gradient t of h' at column j of token t, from the row's mean c1 = mean(u n)
template <class TR, class TA>
__device__ __forceinline__ float grad_h(const NormArgs& a, int64_t t, int j, float rh, float c1) {
  float g = a.dh_out ? (float)((const TR*)a.dh_out)[t * a.ldh + j] : 0.f;
  if (a.dx) {
    const float n = (float)((const TR*)a.h)[t * a.ldh + j] * rh;
    const float u = (float)((const TA*)a.dx)[t * a.ldx + j] * a.w_pre[j];
    g += rh * (u - n * c1);
  }
  return g;
}

template <class TR, class TA>
__global__ __launch_bounds__(kThreads) void k_norm_bwd(const NormArgs a, float* c1s) {
  __shared__ float red[kThreads / 64];
  const int64_t t = blockIdx.x;
  const float ry = a.rstd[2 * t], rh = a.rstd[2 * t + 1];
  float s = 0.f;
  if (a.dx)
    for (int j = threadIdx.x; j < a.d; j += kThreads)
      s += (float)((const TA*)a.dx)[t * a.ldx + j] * a.w_pre[j] * (float)((const TR*)a.h)[t * a.ldh + j] * rh;
  const float c1 = block_sum(s, red) / a.d;
  const TA* y = a.y ? (const TA*)a.y + t * a.ldy : nullptr;
  const TA* g = a.gate ? (const TA*)a.gate + t / a.gate_tokens * a.ldg : nullptr;
  s = 0.f;
  for (int j = threadIdx.x; j < a.d; j += kThreads)
    if (a.w_post)
      s += grad_h<TR, TA>(a, t, j, rh, c1) * (g ? (float)g[j] : 1.f) * a.w_post[j] * (float)y[j] * ry;
  const float c2 = block_sum(s, red) / a.d;
  for (int j = threadIdx.x; j < a.d; j += kThreads) {
    const float dt = grad_h<TR, TA>(a, t, j, rh, c1);
    if (a.dy) {
      float v = dt * (g ? (float)g[j] : 1.f);
      if (a.w_post) v = ry * (v * a.w_post[j] - (float)y[j] * ry * c2);
      ((TA*)a.dy)[t * a.ldy + j] = (TA)v;
    }
  }
  if (threadIdx.x == 0) c1s[t] = c1;
}

// one thread a column: the sums over the tokens
template <class TR, class TA>
__global__ __launch_bounds__(64) void k_norm_bwd_cols(const NormArgs a, const float* c1s) {
  const int j = blockIdx.x * 64 + threadIdx.x;
  if (j >= a.d) return;
  double pre = 0, post = 0, dg = 0;
  for (int64_t t = 0; t < a.T; ++t) {
    const float ry = a.rstd[2 * t], rh = a.rstd[2 * t + 1];
    if (a.dx) pre += (float)((const TA*)a.dx)[t * a.ldx + j] * (float)((const TR*)a.h)[t * a.ldh + j] * rh;
    if (!a.gate && !a.w_post) continue;
    const float dt = grad_h<TR, TA>(a, t, j, rh, c1s[t]);
    const float b = (float)((const TA*)a.y)[t * a.ldy + j] * (a.w_post ? ry : 1.f);
    const float g = a.gate ? (float)((const TA*)a.gate)[t / a.gate_tokens * a.ldg + j] : 1.f;
    post += dt * g * b;
    if (a.gate) {
      dg += dt * b * (a.w_post ? a.w_post[j] : 1.f);
      if (t + 1 == a.T || (t + 1) % a.gate_tokens == 0) {
        ((TA*)a.dgate)[t / a.gate_tokens * a.ldg + j] = (TA)(float)dg;
        dg = 0;
      }
    }
  }
  if (a.dw_pre) a.dw_pre[j] = (float)pre;
  if (a.dw_post) a.dw_post[j] = (float)post;
}

// last, so that dh may be dh_out
template <class TR, class TA>
__global__ __launch_bounds__(kThreads) void k_norm_bwd_dh(const NormArgs a, const float* c1s) {
  const int64_t t = blockIdx.x;
  for (int j = threadIdx.x; j < a.d; j += kThreads)
    ((TR*)a.dh)[t * a.ldh + j] = (TR)(a.res_scale * grad_h<TR, TA>(a, t, j, a.rstd[2 * t + 1], c1s[t]));
}

template <class F> hipError_t by_types(int rdt, int adt, F f) {
  if (rdt == BF16) {
    if (adt == BF16) f(__bf16(), __bf16()); else f(__bf16(), float());
  } else {
    if (adt == BF16) f(float(), __bf16()); else f(float(), float());
  }
  return hipGetLastError();
}

}  // namespace

size_t block_norm_bytes(int T, int d, int gate_tokens) { (void)d; (void)gate_tokens; return (size_t)T * 4 + 256; }

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
  ProfScope prof(POET_K_NORM, st, 0, 0);
  return by_types(a.res_dt, a.act_dt, [&](auto r, auto v) {
    hipLaunchKernelGGL((k_norm_fwd<decltype(r), decltype(v)>), dim3(a.T), dim3(kThreads), 0, st, a);
  });
}

hipError_t launch_norm_bwd(const NormArgs& a, void* ws, hipStream_t st) {
  float* c1s = reinterpret_cast<float*>(ws);
  ProfScope prof(POET_K_NORM, st, 0, 0);
  return by_types(a.res_dt, a.act_dt, [&](auto r, auto v) {
    using TR = decltype(r);
    using TA = decltype(v);
    hipLaunchKernelGGL((k_norm_bwd<TR, TA>), dim3(a.T), dim3(kThreads), 0, st, a, c1s);
    hipLaunchKernelGGL((k_norm_bwd_cols<TR, TA>), dim3((a.d + 63) / 64), dim3(64), 0, st, a, c1s);
    hipLaunchKernelGGL((k_norm_bwd_dh<TR, TA>), dim3(a.T), dim3(kThreads), 0, st, a, c1s);
  });
}

}  // namespace poet

// What a model's last linear answers with: log-probabilities of given tokens with the entropy and the best
// alternatives of each row of logits, the distillation loss on a teacher's top logits, and the gradients of both.
//
// With z a row of V logits, s = inv_temp, m = max z, d = (z - m) s, Z = sum exp d:
//   log p_j = d_j - log Z,   entropy H = log Z - (1/Z) sum exp(d) d   (both sums have one sign: nothing cancels).
#include <algorithm>
#include <cmath>

#include "../../include/poet.h"
#include "internal.h"

namespace poet {
namespace {

constexpr int kThreads = 256;
constexpr float kLow = -1.0e30f;  // stands in for -inf where it would meet a zero factor, and survives a gradient times it

template <class T> __device__ __forceinline__ float ld(const T* p, int64_t i) { return (float)p[i]; }
template <class T> __device__ __forceinline__ void st(T* p, int64_t i, float v) { p[i] = (T)v; }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
template <class A> __device__ __forceinline__ A wave_sum(A v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor((unsigned long long)v, o);
    v = w > v ? w : v;
  }
  return v;
}

// every thread gets the block's result; red holds one entry per wave, free again after the call
template <class A, class F> __device__ __forceinline__ A block_all(A v, A* red, F f) {
  const int w = threadIdx.x >> 6, n = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) red[w] = v;
  __syncthreads();
  A r = red[0];
  for (int i = 1; i < n; ++i) r = f(r, red[i]);
  __syncthreads();
  return r;
}

// order of the alternatives: larger logit first, then the lower index; NaN after everything else
__device__ __forceinline__ uint64_t rank_key(float z, int j) {
  z += 0.f;  // -0 and +0 are equal
  const uint32_t b = __float_as_uint(z);
  const uint32_t o = z != z ? 0u : (b >> 31 ? ~b : b | 0x80000000u);
  return ((uint64_t)o << 32) | (uint32_t)~j;
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_logprobs(const TokenArgs a) {
  __shared__ double rd[kThreads / 64];
  __shared__ float rf[kThreads / 64];
  __shared__ uint64_t rk[kThreads / 64];
  const int row = blockIdx.x;
  const T* z = (const T*)a.z + row * a.ld;
  float m = -INFINITY;
  for (int j = threadIdx.x; j < a.V; j += kThreads) m = fmaxf(m, ld(z, j));
  m = block_all(wave_max(m), rf, [](float x, float y) { return fmaxf(x, y); });
  const bool empty = m == -INFINITY;
  const float ref = empty ? 0.f : m;
  double Z = 0, S = 0;
  for (int j = threadIdx.x; j < a.V; j += kThreads) {
    const float d = (ld(z, j) - ref) * a.s, e = expf(d);
    Z += e;
    S += e * fmaxf(d, kLow);
  }
  const auto add = [](double x, double y) { return x + y; };
  Z = block_all(wave_sum(Z), rd, add);
  S = block_all(wave_sum(S), rd, add);
  const bool none = empty && Z == 0.0;  // every logit is -inf (a NaN would be in Z)
  const float logZ = (float)log(Z), H = none ? 0.f : (float)(log(Z) - S / Z);
  uint64_t last = ~0ull;
  for (int k = 0; k < a.K; ++k) {
    uint64_t best = 0;
    for (int j = threadIdx.x; j < a.V; j += kThreads) {
      const uint64_t q = rank_key(ld(z, j), j);
      if (q < last && q > best) best = q;
    }
    last = block_all(wave_max64(best), rk, [](uint64_t x, uint64_t y) { return x > y ? x : y; });
    const int j = (int)~(uint32_t)last;
    if (threadIdx.x == 0) {
      a.top_ids[(int64_t)row * a.K + k] = j;
      a.top_logp[(int64_t)row * a.K + k] = none ? -INFINITY : (ld(z, j) - ref) * a.s - logZ;
    }
  }
  if (threadIdx.x) return;
  float* q = a.stats + (int64_t)row * 4;
  q[0] = m; q[1] = logZ; q[2] = H; q[3] = 0.f;
  if (a.entropy) a.entropy[row] = H;
  if (a.logp) {
    const int id = a.ids[row];
    a.logp[row] = id < 0 || id >= a.V ? 0.f : none ? -INFINITY : (ld(z, id) - ref) * a.s - logZ;
  }
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_logprobs_bwd(const TokenArgs a) {
  const int row = blockIdx.x;
  const T* z = (const T*)a.z + row * a.ld;
  T* dz = (T*)a.dz + row * a.ldd;
  const float m = a.stats[(int64_t)row * 4], logZ = a.stats[(int64_t)row * 4 + 1], H = a.stats[(int64_t)row * 4 + 2];
  const int id = a.ids && a.dlogp ? a.ids[row] : -1;
  const float gl = id < 0 || id >= a.V ? 0.f : a.dlogp[row], gh = a.dentropy ? a.dentropy[row] : 0.f;
  const bool none = m == -INFINITY && logZ == -INFINITY, zero = none || (gl == 0.f && gh == 0.f);
  const float ref = m == -INFINITY ? 0.f : m;
  for (int j = threadIdx.x; j < a.V; j += kThreads) {
    float g = 0.f;
    if (!zero) {
      const float lp = (ld(z, j) - ref) * a.s - logZ, p = expf(lp);
      g = -p * (gl + gh * (fmaxf(lp, kLow) + H));
      if (j == id) g += gl;
    }
    st(dz, j, g * a.s);
  }
}

// The teacher's list of one row: q[k] = its probability of entry k (0 for absent ones), log q[k], id[k] (-1 absent).
struct List {
  float q[POET_MAX_TOP], lq[POET_MAX_TOP], z[POET_MAX_TOP];
  int id[POET_MAX_TOP];
  float qt;   // TAIL: what the list leaves
  int some;   // any entry present
};

template <class T>
__device__ void load_list(List& L, const TokenArgs& a, int row, const T* z) {
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    int id = a.t_ids[(int64_t)row * a.K + k];
    if (id < 0 || id >= a.V) id = -1;
    L.id[k] = id;
    L.z[k] = id < 0 ? 0.f : ld(z, id);
    L.lq[k] = id < 0 ? -INFINITY : a.t_z[(int64_t)row * a.K + k];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int some = 0;
    float tm = -INFINITY;
    for (int k = 0; k < a.K; ++k) { some |= L.id[k] >= 0; tm = fmaxf(tm, L.lq[k]); }
    double Q = 0;
    if (a.tail) {
      for (int k = 0; k < a.K; ++k) {
        const double l = (double)L.lq[k] * a.ts - (a.t_lse ? a.t_lse[row] : 0.f);
        L.lq[k] = (float)l; L.q[k] = (float)exp(l);
        Q += exp(l);
      }
      L.qt = some ? fmaxf((float)(1.0 - Q), 0.f) : 0.f;
    } else {
      for (int k = 0; k < a.K; ++k) Q += exp(((double)L.lq[k] - tm) * a.ts);
      for (int k = 0; k < a.K; ++k) {
        const double l = ((double)L.lq[k] - tm) * a.ts - log(Q);
        L.lq[k] = (float)l; L.q[k] = (float)exp(l);
      }
      L.qt = 0.f;
    }
    for (int k = 0; k < a.K; ++k)
      if (L.id[k] < 0) L.q[k] = 0.f;
    L.some = some;
  }
  __syncthreads();
}

__device__ __forceinline__ bool listed(const List& L, int K, int j) {
  for (int k = 0; k < K; ++k)
    if (L.id[k] == j) return true;
  return false;
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_distill(const TokenArgs a) {
  __shared__ double rd[kThreads / 64];
  __shared__ float rf[kThreads / 64];
  __shared__ List L;
  const int row = blockIdx.x;
  const T* z = (const T*)a.z + row * a.ld;
  load_list(L, a, row, z);
  const auto fmx = [](float x, float y) { return fmaxf(x, y); };
  const auto add = [](double x, double y) { return x + y; };
  float m = -INFINITY, mt = -INFINITY;  // of the whole row, of its unlisted part
  for (int j = threadIdx.x; j < a.V; j += kThreads) {
    const float v = ld(z, j);
    m = fmaxf(m, v);
    if (a.tail && !listed(L, a.K, j)) mt = fmaxf(mt, v);
  }
  m = block_all(wave_max(m), rf, fmx);
  mt = block_all(wave_max(mt), rf, fmx);
  const float ref = m == -INFINITY ? 0.f : m, reft = mt == -INFINITY ? 0.f : mt;
  double Z = 0, Zt = 0;
  for (int j = threadIdx.x; j < a.V; j += kThreads) {
    const float v = ld(z, j);
    Z += expf((v - ref) * a.s);
    if (a.tail && !listed(L, a.K, j)) Zt += expf((v - reft) * a.s);
  }
  Z = block_all(wave_sum(Z), rd, add);
  Zt = block_all(wave_sum(Zt), rd, add);
  if (threadIdx.x) return;
  const double logZ = log(Z), logZt = log(Zt);
  const bool none = m == -INFINITY && Z == 0.0;
  double loss = 0;
  for (int k = 0; k < a.K; ++k)
    if (L.q[k] > 0.f) loss += none ? INFINITY : (double)L.q[k] * (L.lq[k] - (((double)L.z[k] - ref) * a.s - logZ));
  if (L.qt > 0.f) loss += none ? INFINITY : L.qt * (log((double)L.qt) - (logZt + ((double)reft - ref) * a.s - logZ));
  a.loss[row] = L.some ? (float)loss : 0.f;
  float* q = a.stats + (int64_t)row * 4;
  q[0] = m; q[1] = (float)logZ; q[2] = a.tail ? mt : 0.f; q[3] = a.tail ? (float)logZt : 0.f;
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_distill_bwd(const TokenArgs a) {
  __shared__ List L;
  const int row = blockIdx.x;
  const T* z = (const T*)a.z + row * a.ld;
  T* dz = (T*)a.dz + row * a.ldd;
  load_list(L, a, row, z);
  const float* q = a.stats + (int64_t)row * 4;
  const float m = q[0], logZ = q[1], mt = q[2], logZt = q[3];
  const float w = L.some ? a.dloss[row] : 0.f;
  const bool zero = w == 0.f || (m == -INFINITY && logZ == -INFINITY);
  const float ref = m == -INFINITY ? 0.f : m, reft = mt == -INFINITY ? 0.f : mt;
  for (int j = threadIdx.x; j < a.V; j += kThreads) {
    float g = 0.f;
    if (!zero) {
      const float v = ld(z, j);
      g = expf((v - ref) * a.s - logZ);
      bool in = false;
      float take = 0.f;
      for (int k = 0; k < a.K; ++k)
        if (L.id[k] == j) { in = true; take += L.q[k]; }
      if (!in && a.tail && L.qt > 0.f && logZt > -INFINITY) take = L.qt * expf((v - reft) * a.s - logZt);
      g = (g - take) * w * a.s;
    }
    st(dz, j, g);
  }
}

template <class F> hipError_t by_type(int dt, F f) {
  if (dt == BF16) f(__bf16()); else f(float());
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs(const TokenArgs& a, hipStream_t st) {
  ProfScope prof(POET_K_HEAD, st, 6.0 * a.T * a.V, (double)a.T * a.V * dtype_size(a.dt));
  return by_type(a.dt, [&](auto t) { hipLaunchKernelGGL(k_logprobs<decltype(t)>, dim3(a.T), dim3(kThreads), 0, st, a); });
}
hipError_t launch_logprobs_bwd(const TokenArgs& a, hipStream_t st) {
  ProfScope prof(POET_K_HEAD, st, 6.0 * a.T * a.V, 2.0 * a.T * a.V * dtype_size(a.dt));
  return by_type(a.dt, [&](auto t) { hipLaunchKernelGGL(k_logprobs_bwd<decltype(t)>, dim3(a.T), dim3(kThreads), 0, st, a); });
}
hipError_t launch_distill(const TokenArgs& a, hipStream_t st) {
  ProfScope prof(POET_K_HEAD, st, 6.0 * a.T * a.V, (double)a.T * a.V * dtype_size(a.dt));
  return by_type(a.dt, [&](auto t) { hipLaunchKernelGGL(k_distill<decltype(t)>, dim3(a.T), dim3(kThreads), 0, st, a); });
}
hipError_t launch_distill_bwd(const TokenArgs& a, hipStream_t st) {
  ProfScope prof(POET_K_HEAD, st, 6.0 * a.T * a.V, 2.0 * a.T * a.V * dtype_size(a.dt));
  return by_type(a.dt, [&](auto t) { hipLaunchKernelGGL(k_distill_bwd<decltype(t)>, dim3(a.T), dim3(kThreads), 0, st, a); });
}

}  // namespace poet

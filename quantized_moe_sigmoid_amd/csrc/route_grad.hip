// route_grad.hip — the gradient of the route from logits (route_logits.hip; colibri-strix README,
// "What's implemented", router item) with respect to the logits.
//
// The taken experts are held fixed, so a weight depends on the taken scores alone (sigmoid, or any
// score over its sum) or on all logits (softmax). With p the scores, S their sum over the taken and
// g the weights' gradient:
//   renorm: scale (g_j - sum_i g_i p_i / S) p_j / S, times 1 - p_j for the sigmoid;
//   else scale g_j p_j (1 - p_j), or p_e scale (g_e - sum_i g_i p_i) for every expert.
// All of it in fp64: what is left of g_j is a difference. A single taken expert has p / S = 1 and so
// exactly 0.
//
// One wavefront a token: its logits in registers, the slots in the first k lanes and handed to all
// by scalar reads, so that an expert in two slots gets their sum in slot order. 8191 tokens over 256
// experts, sigmoid, fp32: 8 to 9 us by the card (17 MB: 2.7; a launch 4): loads of 4 bytes a lane, an id before its
// logit, then fp64. Branches that spare the additions of other lanes' experts and reading the taken logits alone:
// the same.
#include "mxfp4_impl.h"

namespace coli {

constexpr int RG_WAVES = 4;

__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// Sum of the values of the first `many` lanes (a power of two), the others holding 0; in every lane
__device__ __forceinline__ double lanes_total(double v, int many) {
  for (int o = many >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return lane_value(v, 0);
}

// z and dz may be one array: a wavefront has read its row before it writes it
template <int EPL, bool SOFTMAX, typename T>
__global__ __launch_bounds__(64 * RG_WAVES) void route_grad_kernel(RouteGradArgs a, const T *z, T *dz) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * RG_WAVES + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const int E = a.E, k = a.k, many = a.many;
  const T *zt = z + t * E;
  float v[EPL];  // -inf: not there
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; i++) {
    const int e = lane + 64 * i;
    const float x = e < E ? (float)zt[e] : -INFINITY;
    v[i] = x == x ? x : -INFINITY;
    top = fmaxf(top, v[i]);
  }
  int mine = lane < k ? a.idx[t * k + lane] : -1;
  if (mine >= E) mine = -1;
  float zs = mine >= 0 ? (float)zt[mine] : -INFINITY;
  if (!(zs > -INFINITY)) zs = -INFINITY;
  const double g = lane < k && mine >= 0 ? (double)a.dw[t * k + lane] : 0.0;
  double p[SOFTMAX ? EPL : 1], ps, rest = 1.0;  // scores; of this lane's slot; 1 - p of a sigmoid
  if constexpr (SOFTMAX) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    // logits of +inf share everything and move nothing
    const bool some = top > -INFINITY && top < INFINITY;
    ps = some && zs > -INFINITY ? exp((double)zs - (double)top) : 0.0;
    if (!a.renorm) {
      double total = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; i++) {
        p[i] = some && v[i] > -INFINITY ? exp((double)v[i] - (double)top) : 0.0;
        total += p[i];
      }
      total = lanes_total(total, 64);
      const double inv = total > 0.0 ? 1.0 / total : 0.0;
#pragma unroll
      for (int i = 0; i < EPL; i++) p[i] *= inv;
      ps *= inv;
    }
  } else {
    const double x = exp(-fabs((double)zs));
    ps = zs > -INFINITY ? (zs >= 0.0f ? 1.0 : x) / (1.0 + x) : 0.0;
    rest = (zs >= 0.0f ? x : 1.0) / (1.0 + x);
  }
  // what this lane's slot gives its expert
  double mean = 0.0, give;
  if (a.renorm) {
    const double total = lanes_total(ps, many);
    const double share = total > 0.0 ? ps / total : 0.0;
    mean = lanes_total(share > 0.0 ? g * share : 0.0, many);
    give = share > 0.0 ? (double)a.scale * (g - mean) * share * rest : 0.0;
  } else if constexpr (SOFTMAX) {
    mean = lanes_total(ps > 0.0 ? g * ps : 0.0, many) * (double)a.scale;
    give = g * (double)a.scale;
  } else {
    give = ps > 0.0 ? (double)a.scale * g * ps * rest : 0.0;
  }
  double out[EPL] = {};
  for (int j = 0; j < k; j++) {
    const int e = __builtin_amdgcn_readlane(mine, j);
    if (e < 0) continue;
    const double add = lane_value(give, j);
#pragma unroll
    for (int i = 0; i < EPL; i++) out[i] += e == lane + 64 * i ? add : 0.0;
  }
#pragma unroll
  for (int i = 0; i < EPL; i++) {
    const int e = lane + 64 * i;
    if (SOFTMAX && !a.renorm) out[i] = p[i] > 0.0 ? p[i] * (out[i] - mean) : 0.0;
    if (e < E) dz[t * E + e] = (T)out[i];
  }
}

template <typename T>
static hipError_t launch_rg(RouteGradArgs a, const T *z, T *dz, hipStream_t s) {
  for (a.many = 1; a.many < a.k;) a.many *= 2;
  const dim3 grid((unsigned)((a.T + RG_WAVES - 1) / RG_WAVES)), block(64 * RG_WAVES);
  auto go = [&]<int EPL>() {
    if (a.softmax)
      hipLaunchKernelGGL((route_grad_kernel<EPL, true, T>), grid, block, 0, s, a, z, dz);
    else
      hipLaunchKernelGGL((route_grad_kernel<EPL, false, T>), grid, block, 0, s, a, z, dz);
    return hipGetLastError();
  };
  if (a.E <= 64) return go.template operator()<1>();
  if (a.E <= 128) return go.template operator()<2>();
  if (a.E <= 256) return go.template operator()<4>();
  if (a.E <= 512) return go.template operator()<8>();
  return go.template operator()<16>();
}

hipError_t launch_route_grad(const RouteGradArgs &a, const void *z, int dtype, void *dz, hipStream_t s) {
  if (dtype == COLI_F32) return launch_rg(a, (const float *)z, (float *)dz, s);
  if (dtype == COLI_BF16) return launch_rg(a, (const bf16_t *)z, (bf16_t *)dz, s);
  return launch_rg(a, (const f16_t *)z, (f16_t *)dz, s);
}

}  // namespace coli

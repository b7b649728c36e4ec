// route_logits.hip — the route of T tokens from router logits that the caller computed.
//
// The router family of colibri-strix README, "What's implemented", router item, with the
// choices that gates of other models make: sigmoid or softmax scores p in fp64, over the
// experts present (a logit of -inf or NaN takes its expert away); key = the logit, or
// p + bias with a correction bias; groups of E/G contiguous experts scored by the sum of their
// one or two best (the logit or score itself), the Gk best kept; the k best keys inside them
// in descending order, every tie to the lower index; w = p, over the sum of the taken with
// renorm (0 where that sum is 0), times scale. Slots that no expert is left for hold -1 and 0.
//
// One wavefront per token. Lane l holds the EPL contiguous experts l * EPL ..; a slot is one
// maximum over the wavefront, and the lowest lane that holds it wins (its lowest expert).
#include "mxfp4_impl.h"

namespace coli {

constexpr int RL_WAVES = 4;  // tokens per workgroup

__device__ __forceinline__ double dpp_max_step(double v, double w) { return fmax(v, w); }

template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

template <typename Op>
__device__ __forceinline__ double wave_all(double v, Op op) {  // op over the 64 lanes, in every lane
  v = op(v, dpp_d<0xB1>(v));   // l ^ 1
  v = op(v, dpp_d<0x4E>(v));   // l ^ 2
  v = op(v, dpp_d<0x141>(v));  // l ^ 7
  v = op(v, dpp_d<0x140>(v));  // l ^ 15
  v = op(v, __shfl_xor(v, 16));
  return op(v, __shfl_xor(v, 32));
}

__device__ __forceinline__ double wave_max(double v) {
  return wave_all(v, [](double a, double b) { return fmax(a, b); });
}

template <int EPL, typename T>
__global__ __launch_bounds__(64 * RL_WAVES) void route_logits_kernel(RouteLogitsArgs a, const T *__restrict__ z) {
  extern __shared__ double lds[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t0 = blockIdx.x * RL_WAVES + wv, t = min(t0, a.T - 1);  // waves past the end repeat the last token
  const int E = a.E, G = a.G, k = a.k;
  double p[EPL], key[EPL];
  double zmax = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; i++) {
    const int e = lane * EPL + i;
    double v = e < E ? (double)(float)z[(int64_t)t * E + e] : -INFINITY;
    if (!(v > -INFINITY)) v = -INFINITY;  // NaN
    key[i] = v;
    zmax = fmax(zmax, v);
  }
  if (a.softmax) {
    zmax = wave_max(zmax);
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
      // experts with a logit of +inf share everything
      p[i] = key[i] == -INFINITY ? 0.0 : zmax == INFINITY ? (key[i] == INFINITY ? 1.0 : 0.0) : exp(key[i] - zmax);
      s += p[i];
    }
    s = wave_all(s, [](double x, double y) { return x + y; });
#pragma unroll
    for (int i = 0; i < EPL; i++) p[i] = s > 0.0 ? p[i] / s : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; i++) p[i] = 1.0 / (1.0 + exp(-key[i]));
  }
  // what groups and experts are compared by; -inf: not there
  double by[EPL];
#pragma unroll
  for (int i = 0; i < EPL; i++) {
    const int e = lane * EPL + i;
    const bool there = key[i] > -INFINITY;
    double c = p[i];
    if (a.bias && e < E) c += (double)a.bias[e];
    if (a.bias) key[i] = there && c > -INFINITY ? c : -INFINITY;  // a bias of -inf or NaN takes an expert away
    by[i] = a.group_top == 1 || a.E == G ? key[i] : (key[i] > -INFINITY ? c : -INFINITY);
  }
  if (G > 1) {
    const int m = E / G;
    double *by_s = lds + (size_t)wv * E;
    int *keep_s = reinterpret_cast<int *>(lds + (size_t)RL_WAVES * E) + wv * 64;
#pragma unroll
    for (int i = 0; i < EPL; i++)
      if (lane * EPL + i < E) by_s[lane * EPL + i] = by[i];
    __syncthreads();
    double gs = -INFINITY;
    if (lane < G) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int j = 0; j < m; j++) {
        const double v = by_s[lane * m + j];
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
      }
      gs = b1 + (a.group_top == 2 && b2 > -INFINITY ? b2 : 0.0);
    }
    int before = 0;
    for (int j = 0; j < G; j++) {
      const double o = __shfl(gs, j);
      before += (o > gs || (o == gs && j < lane)) ? 1 : 0;
    }
    keep_s[lane] = lane < G && before < a.Gk;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EPL; i++) {
      const int e = lane * EPL + i;
      if (e < E && !keep_s[e / m]) key[i] = -INFINITY;
    }
  }
  int mine = -1;
  double pm = 0.0, total = 0.0;
  for (int j = 0; j < k; j++) {
    double best = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < EPL; i++)
      if (key[i] > best) {
        best = key[i];
        bi = i;
      }
    const double top = wave_max(best);
    if (top == -INFINITY) break;
    const int owner = __builtin_ctzll(__ballot(best == top));
    double pb = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; i++)
      if (i == bi) {
        pb = p[i];
        if (lane == owner) key[i] = -INFINITY;
      }
    pb = __shfl(pb, owner);
    const int e = __shfl(lane * EPL + bi, owner);
    total += pb;
    if (lane == j) {
      mine = e;
      pm = pb;
    }
  }
  if (t0 < a.T && lane < k) {
    double w = a.renorm ? (total > 0.0 ? pm / total : 0.0) : pm;
    a.idx[(int64_t)t * k + lane] = mine;
    a.w[(int64_t)t * k + lane] = (float)(w * (double)a.scale);
  }
}

template <typename T>
static hipError_t launch_rl(const RouteLogitsArgs &a, const T *z, hipStream_t s) {
  const dim3 g((unsigned)((a.T + RL_WAVES - 1) / RL_WAVES)), b(64 * RL_WAVES);
  const size_t lds = a.G > 1 ? (size_t)RL_WAVES * (a.E * sizeof(double) + 64 * sizeof(int)) : 0;
  if (a.E <= 64)
    hipLaunchKernelGGL((route_logits_kernel<1, T>), g, b, lds, s, a, z);
  else if (a.E <= 128)
    hipLaunchKernelGGL((route_logits_kernel<2, T>), g, b, lds, s, a, z);
  else if (a.E <= 256)
    hipLaunchKernelGGL((route_logits_kernel<4, T>), g, b, lds, s, a, z);
  else if (a.E <= 512)
    hipLaunchKernelGGL((route_logits_kernel<8, T>), g, b, lds, s, a, z);
  else
    hipLaunchKernelGGL((route_logits_kernel<16, T>), g, b, lds, s, a, z);
  return hipGetLastError();
}

hipError_t launch_route_logits(const RouteLogitsArgs &a, const void *z, int dtype, hipStream_t s) {
  if (dtype == COLI_F32) return launch_rl(a, (const float *)z, s);
  if (dtype == COLI_BF16) return launch_rl(a, (const bf16_t *)z, s);
  return launch_rl(a, (const f16_t *)z, s);
}

}  // namespace coli

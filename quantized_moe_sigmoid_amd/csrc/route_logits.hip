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
// One wavefront per token, bound by its instructions (a token's logits are 1 KB at most).
// The kernel keeps the whole selection in fp32, a value to a register: one maximum over the
// wavefront (six instructions) per slot. Logits are fp32 numbers, so without a bias it is exact;
// with one (and for sums of two scores) its keys are within a known distance of the fp64 ones,
// and where two keys whose order counts lie closer than that, the token goes through route_exact,
// the same selection in fp64. Only the taken experts' scores are computed in fp64 otherwise.
// 8191 tokens of 256 experts in 8 groups, 8 taken, with a bias: 15 us (20 with the selection in
// fp64); 4093 of 64 experts, and one token, 6 us: the call. The 8.4 MB of logits alone need 1.3.
#include "mxfp4_impl.h"

namespace coli {

constexpr int RL_WAVES = 4;  // tokens per workgroup

template <int CTRL>
__device__ __forceinline__ int dpp_i(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  return __hiloint2double(dpp_i<CTRL>(__double2hiint(v)), dpp_i<CTRL>(__double2loint(v)));
}

// op over the 64 lanes, in every lane: partners l ^ 1, l ^ 2, l ^ 7, l ^ 15 by DPP; the swaps of
// 16- and 32-lane rows of a pair of equal registers leave a value and its partner's
template <typename Op>
__device__ __forceinline__ double wave_all(double v, Op op) {
  v = op(v, dpp_d<0xB1>(v));
  v = op(v, dpp_d<0x4E>(v));
  v = op(v, dpp_d<0x141>(v));
  v = op(v, dpp_d<0x140>(v));
  auto h = __builtin_amdgcn_permlane16_swap(__double2hiint(v), __double2hiint(v), false, false);
  auto l = __builtin_amdgcn_permlane16_swap(__double2loint(v), __double2loint(v), false, false);
  v = op(__hiloint2double(h[0], l[0]), __hiloint2double(h[1], l[1]));
  h = __builtin_amdgcn_permlane32_swap(__double2hiint(v), __double2hiint(v), false, false);
  l = __builtin_amdgcn_permlane32_swap(__double2loint(v), __double2loint(v), false, false);
  return op(__hiloint2double(h[0], l[0]), __hiloint2double(h[1], l[1]));
}
__device__ __forceinline__ double wave_max(double v) {
  return wave_all(v, [](double a, double b) { return fmax(a, b); });
}
__device__ __forceinline__ double wave_sum(double v) {
  return wave_all(v, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ float wave_sum(float v) {
  v += __int_as_float(dpp_i<0xB1>(__float_as_int(v)));
  v += __int_as_float(dpp_i<0x4E>(__float_as_int(v)));
  v += __int_as_float(dpp_i<0x141>(__float_as_int(v)));
  v += __int_as_float(dpp_i<0x140>(__float_as_int(v)));
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_int(v), __float_as_int(v), false, false);
  v = __int_as_float(r[0]) + __int_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_int(v), __float_as_int(v), false, false);
  return __int_as_float(r[0]) + __int_as_float(r[1]);
}
// the largest of the 64 lanes, in a scalar register
__device__ __forceinline__ int wave_max(int v) {
  v = max(v, dpp_i<0xB1>(v));
  v = max(v, dpp_i<0x4E>(v));
  v = max(v, dpp_i<0x141>(v));
  v = max(v, dpp_i<0x140>(v));
  const int a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const int c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  return max(max(a, b), max(c, d));
}

// fp32 values as integers of the same order (-0 as 0), and back
__device__ __forceinline__ int order_of(float f) {
  const int b = __float_as_int(f + 0.0f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float value_of(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7FFFFFFF)); }
constexpr int ABSENT = (int)0x807FFFFF;  // order_of(-inf)

// LDS writes of this wavefront are visible to its own later reads
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The selection in fp64, of the experts lane * EPL + i. Slot j in lane j: expert or -1, and p.
template <int EPL, typename T>
__device__ __forceinline__ void route_exact(const RouteLogitsArgs &a, const T *zt, double *by_s, int &mine,
                                                      double &pm) {
  const int lane = threadIdx.x & 63;
  const int E = a.E, G = a.G, k = a.k;
  double p[EPL], key[EPL];
  double zmax = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; i++) {
    const int e = lane * EPL + i;
    double v = e < E ? (double)(float)zt[e] : -INFINITY;
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
    s = wave_sum(s);
#pragma unroll
    for (int i = 0; i < EPL; i++) p[i] = s > 0.0 ? p[i] / s : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; i++) p[i] = 1.0 / (1.0 + exp(-key[i]));
  }
  if (G > 1) {
    const int m = E / G;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
      const int e = lane * EPL + i;
      const bool there = key[i] > -INFINITY;
      double c = p[i];
      if (a.bias && e < E) c += (double)a.bias[e];
      if (a.bias) key[i] = there && c > -INFINITY ? c : -INFINITY;  // a bias of -inf or NaN takes an expert away
      if (e < E) by_s[e] = a.group_top == 1 || m == 1 ? key[i] : (key[i] > -INFINITY ? c : -INFINITY);
    }
    wave_sync();
    double gs = -INFINITY;
    if (lane < G) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int j = 0; j < m; j++) {
        const double v = by_s[lane * m + j];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
      gs = b1 + (a.group_top == 2 && b2 > -INFINITY ? b2 : 0.0);
    }
    int before = 0;
    for (int j = 0; j < G; j++) {
      const double o = __shfl(gs, j);
      before += (o > gs || (o == gs && j < lane)) ? 1 : 0;
    }
    const uint64_t keep = __ballot(lane < G && before < a.Gk);
#pragma unroll
    for (int i = 0; i < EPL; i++) {
      const int e = min(lane * EPL + i, E - 1);
      if (!((keep >> (e / m)) & 1)) key[i] = -INFINITY;
    }
  } else if (a.bias) {
#pragma unroll
    for (int i = 0; i < EPL; i++) {
      const int e = lane * EPL + i;
      const double c = p[i] + (e < E ? (double)a.bias[e] : 0.0);
      key[i] = key[i] > -INFINITY && c > -INFINITY ? c : -INFINITY;
    }
  }
  mine = -1;
  pm = 0.0;
  for (int j = 0; j < k; j++) {
    double best = key[0], pb = p[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < EPL; i++)
      if (key[i] > best) best = key[i], pb = p[i], bi = i;
    const double top = wave_max(best);
    if (top == -INFINITY) break;
    const int owner = __builtin_ctzll(__ballot(best == top));
#pragma unroll
    for (int i = 0; i < EPL; i++)
      if (i == bi && lane == owner) key[i] = -INFINITY;
    pb = __shfl(pb, owner);
    const int e = __shfl(lane * EPL + bi, owner);
    if (lane == j) {
      mine = e;
      pm = pb;
    }
  }
}

// A lane holds EPL experts of one group: with Gp = the power of two from G up, group g has lanes
// g L .. g L + L - 1 (L = 64 / Gp), lane r of them the experts r EPL .. of the group.
template <int EPL, int EPX, bool SOFTMAX, typename T>
__global__ __launch_bounds__(64 * RL_WAVES) void route_logits_kernel(RouteLogitsArgs a, const T *__restrict__ z) {
  extern __shared__ double lds[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t0 = blockIdx.x * RL_WAVES + wv, t = min(t0, a.T - 1);  // waves past the end repeat the last token
  const int E = a.E, G = a.G, k = a.k, m = a.m;
  const T *zt = z + (int64_t)t * E;
  const int g = lane >> a.lshift, r0 = (lane & ((1 << a.lshift) - 1)) * EPL, e0 = g * m + r0;
  const int mine_n = g < G ? m - r0 : 0;  // experts from e0 on that are in the group
  float key[EPL], sc[EPL];                // what experts, groups are compared by; -inf: not there
  float zmax = -INFINITY;
  float bias[EPL] = {};
  constexpr bool WIDE = EPL > 1 && EPL * sizeof(T) <= 16;
  if (WIDE && a.vec) {  // whole lanes, aligned rows
    typedef T tv __attribute__((ext_vector_type(WIDE ? EPL : 1)));
    typedef float fv __attribute__((ext_vector_type(WIDE && EPL <= 4 ? EPL : 1)));
    const int at = mine_n > 0 ? e0 : 0;
    const tv v = *reinterpret_cast<const tv *>(zt + at);
    if constexpr (EPL <= 4) {
      if (a.bias) {
        const fv b = *reinterpret_cast<const fv *>(a.bias + at);
#pragma unroll
        for (int i = 0; i < EPL; i++) bias[i] = b[i];
      }
    } else if (a.bias) {
#pragma unroll
      for (int i = 0; i < EPL; i++) bias[i] = a.bias[at + i];
    }
#pragma unroll
    for (int i = 0; i < EPL; i++) key[i] = mine_n > 0 ? (float)v[i] : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; i++) {
      key[i] = i < mine_n ? (float)zt[e0 + i] : -INFINITY;
      if (a.bias) bias[i] = i < mine_n ? a.bias[e0 + i] : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; i++) {
    key[i] = key[i] > -INFINITY ? key[i] : -INFINITY;  // NaN
    zmax = fmaxf(zmax, key[i]);
  }
  const bool two = G > 1 && a.group_top == 2 && m > 1;
  const bool scores = a.bias != nullptr || two;  // p is compared, not only z
  double total64 = 1.0;
  if constexpr (SOFTMAX) {
    zmax = value_of(wave_max(order_of(zmax)));
    if (!a.renorm) {  // the weights are p themselves
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; i++)
        s += key[i] == -INFINITY ? 0.0 : zmax == INFINITY ? (key[i] == INFINITY ? 1.0 : 0.0) : exp((double)key[i] - (double)zmax);
      total64 = wave_sum(s);
    }
  }
  // |p in fp32 - p| < delta. Sigmoid: the exponential's argument is off by 2^-23 |z|, which
  // moves p by less than p (1 - p) |z| 2^-23 < 2^-25; exponential, sum and reciprocal by a few
  // 2^-24 of p. Softmax: the sum of E <= 1024 terms in fp32 by less than 2^-18 of it.
  constexpr float delta = SOFTMAX ? 0x1p-17f : 0x1p-20f;
  int ord[EPL], by[EPL];
#pragma unroll
  for (int i = 0; i < EPL; i++) ord[i] = by[i] = order_of(key[i]);
  if (scores) {
    float p[EPL], s = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
      if constexpr (SOFTMAX) {
        p[i] = zmax == INFINITY ? (key[i] == INFINITY ? 1.0f : 0.0f) : __expf(key[i] - zmax);
        s += key[i] > -INFINITY ? p[i] : 0.0f;
      } else {
        p[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-key[i]));
      }
    }
    if constexpr (SOFTMAX) {
      s = 1.0f / wave_sum(s);
#pragma unroll
      for (int i = 0; i < EPL; i++) p[i] *= s;
    }
#pragma unroll
    for (int i = 0; i < EPL; i++) {
      const float c = p[i] + bias[i];
      const bool there = key[i] > -INFINITY && c > -INFINITY;  // a bias of -inf or NaN takes an expert away
      const int o = there ? order_of(c) : ABSENT;
      if (a.bias) ord[i] = o;
      by[i] = a.bias || two ? o : by[i];
    }
  }
  bool close = false;  // an order that counts is within the error
  if (G > 1) {
    int b1 = ABSENT, b2 = ABSENT;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
      b2 = max(b2, min(b1, by[i]));
      b1 = max(b1, by[i]);
    }
    auto join = [&](int p1, int p2, int q1, int q2) {
      b2 = max(max(p2, q2), min(p1, q1));
      b1 = max(p1, q1);
    };
    if (a.lshift > 0) join(b1, b2, dpp_i<0xB1>(b1), dpp_i<0xB1>(b2));
    if (a.lshift > 1) join(b1, b2, dpp_i<0x4E>(b1), dpp_i<0x4E>(b2));
    if (a.lshift > 2) join(b1, b2, dpp_i<0x141>(b1), dpp_i<0x141>(b2));
    if (a.lshift > 3) join(b1, b2, dpp_i<0x140>(b1), dpp_i<0x140>(b2));
    if (a.lshift > 4) {
      const auto x = __builtin_amdgcn_permlane16_swap(b1, b1, false, false);
      const auto y = __builtin_amdgcn_permlane16_swap(b2, b2, false, false);
      join(x[0], y[0], x[1], y[1]);
    }
    int gs = b1;
    if (two && b2 != ABSENT) gs = order_of(value_of(b1) + value_of(b2));
    int before = 0;
    for (int j = 0; j < G; j++) {
      const int o = __builtin_amdgcn_readlane(gs, j << a.lshift);
      before += o >= gs + (j < g ? 0 : 1) ? 1 : 0;  // larger, or equal and lower
    }
    const bool keep = before < a.Gk;
    if (scores) {
      // A group's one or two keys were rounded at their own sizes and may cancel in the sum: its
      // error is below 2 delta + (|b1| + |b2|) 2^-22. Compared are the least that a kept group can
      // be and the most that another can (infinite sizes: close).
      const float f1 = value_of(b1), f2 = two && b2 != ABSENT ? value_of(b2) : 0.0f;
      const float mag = fabsf(f1) + fabsf(f2), err = mag < INFINITY ? mag * 0x1p-21f : INFINITY, sum = value_of(gs);
      const int least = err < INFINITY ? order_of(sum - err) : ABSENT;
      const int most = order_of(err < INFINITY ? sum + err : INFINITY);
      const bool there = g < G && gs != ABSENT;
      const int in = ~wave_max(keep && g < G ? ~(there ? least : ABSENT) : ABSENT);
      const int out = wave_max(!keep && there ? most : ABSENT);
      close = out != ABSENT && !(value_of(in) - value_of(out) > 4 * delta);
    }
#pragma unroll
    for (int i = 0; i < EPL; i++) ord[i] = keep ? ord[i] : ABSENT;
  }
  int mine = -1, tv = ABSENT;  // slot j's expert and its key in lane j
  const int rounds = a.bias && k < 64 ? k + 1 : k;  // with a bias the best that is left out, too
  for (int j = 0; j < rounds; j++) {
    int best = ord[0];
#pragma unroll
    for (int i = 1; i < EPL; i++) best = max(best, ord[i]);
    const int top = wave_max(best);
    if (top == ABSENT) break;
    const uint64_t who = __ballot(best == top);
    const int owner = __builtin_ctzll(who);
    const bool own = lane == owner;
    tv = lane == j ? top : tv;
    int at = EPL - 1;
#pragma unroll
    for (int i = EPL - 2; i >= 0; i--) at = ord[i] == top ? i : at;  // the lane's lowest
    const int e = __builtin_amdgcn_readlane(e0 + at, owner);
    mine = lane == j ? e : mine;
#pragma unroll
    for (int i = 0; i < EPL; i++) ord[i] = own && at == i ? ABSENT : ord[i];
  }
  if (a.bias) {
    const int next = k < 64 ? __shfl_down(tv, 1) : tv;
    const float ft = value_of(tv), fn = value_of(next);
    close = close || (lane < k && next != ABSENT && !(ft - fn > 2 * delta + (fabsf(ft) + fabsf(fn)) * 0x1p-22f));
    if (lane >= k) mine = -1;
  }
  double pm = 0.0;
  if (__ballot(close) != 0) {
    route_exact<EPX>(a, zt, lds + (size_t)wv * E, mine, pm);
  } else if (mine >= 0) {
    const double v = (double)(a.bias ? (float)zt[mine] : value_of(tv));
    if constexpr (!SOFTMAX)
      pm = 1.0 / (1.0 + exp(-v));
    else
      pm = (zmax == INFINITY ? (v == INFINITY ? 1.0 : 0.0) : exp(v - (double)zmax)) / total64;
  }
  const double total = a.renorm ? wave_sum(pm) : 1.0;
  if (t0 < a.T && lane < k) {
    a.idx[(int64_t)t * k + lane] = mine;
    a.w[(int64_t)t * k + lane] = total > 0.0 ? (float)(pm / total * (double)a.scale) : 0.0f;
  }
}

template <int EPL, int EPX, typename T>
static hipError_t launch_rl(const RouteLogitsArgs &a, const T *z, hipStream_t s) {
  const dim3 g((unsigned)((a.T + RL_WAVES - 1) / RL_WAVES)), b(64 * RL_WAVES);
  const size_t lds = a.G > 1 ? (size_t)RL_WAVES * a.E * sizeof(double) : 0;
  const size_t piece = EPL * sizeof(T);
  RouteLogitsArgs r = a;
  r.vec = a.m % EPL == 0 && (uintptr_t)z % piece == 0 && a.E * sizeof(T) % piece == 0 && (uintptr_t)a.bias % 16 == 0;
  if (a.softmax)
    hipLaunchKernelGGL((route_logits_kernel<EPL, EPX, true, T>), g, b, lds, s, r, z);
  else
    hipLaunchKernelGGL((route_logits_kernel<EPL, EPX, false, T>), g, b, lds, s, r, z);
  return hipGetLastError();
}

template <int EPX, typename T>
static hipError_t launch_rl_x(const RouteLogitsArgs &a, int epl, const T *z, hipStream_t s) {
  // a group's lanes are a power of two, so a lane has up to four times an even share
  if (epl <= EPX) return launch_rl<EPX, EPX>(a, z, s);
  if (epl <= 2 * EPX) return launch_rl<2 * EPX, EPX>(a, z, s);
  return launch_rl<4 * EPX, EPX>(a, z, s);
}

template <typename T>
static hipError_t launch_rl_t(RouteLogitsArgs a, const T *z, hipStream_t s) {
  a.m = a.E / a.G;
  int gp = 1;
  while (gp < a.G) gp *= 2;
  a.lshift = __builtin_ctz(64 / gp);
  const int epl = (a.m + (64 / gp) - 1) / (64 / gp);
  if (a.E <= 64) return launch_rl_x<1>(a, epl, z, s);
  if (a.E <= 128) return launch_rl_x<2>(a, epl, z, s);
  if (a.E <= 256) return launch_rl_x<4>(a, epl, z, s);
  if (a.E <= 512) return launch_rl_x<8>(a, epl, z, s);
  return launch_rl_x<16>(a, epl, z, s);
}

hipError_t launch_route_logits(const RouteLogitsArgs &a, const void *z, int dtype, hipStream_t s) {
  if (dtype == COLI_F32) return launch_rl_t(a, (const float *)z, s);
  if (dtype == COLI_BF16) return launch_rl_t(a, (const bf16_t *)z, s);
  return launch_rl_t(a, (const f16_t *)z, s);
}

}  // namespace coli

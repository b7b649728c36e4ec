// pairs.hip — a route's pairs sorted by expert, tokens' rows laid out in that order and summed back,
// and the gradients (batch-union and router items of colibri-strix README, "What's implemented").
//
// All bound by memory: a row is read once for each use and written once. Sums are fp32 in slot order,
// without atomics.
#include "group_impl.h"
#include "mxfp4_impl.h"

namespace coli {

// ------------------------------------------------------------------ sorting
// A stable counting sort in chunks of pairs: counts of every chunk (sort_count_kernel), then each
// chunk's workgroup adds up what lies before its own pairs and places them. One chunk needs no counts
// of others. A wavefront owns consecutive pairs and ranks 64 at a time by ballots (group_impl.h).
constexpr int SORT_WAVES = 4, SORT_NT = 64 * SORT_WAVES;

__global__ __launch_bounds__(SORT_NT) void sort_count_kernel(SortArgs a) {
  extern __shared__ int cnt[];  // [E + 1], the last one: ids out of range
  for (int e = threadIdx.x; e <= a.E; e += SORT_NT) cnt[e] = 0;
  __syncthreads();
  const int first = blockIdx.x * a.chunk, end = min(a.P, first + a.chunk);
  for (int p = first + threadIdx.x; p < end; p += SORT_NT) {
    const int e = a.idx[p];
    if (e >= 0 && e < a.E)
      atomicAdd(&cnt[e], 1);
    else if (e != -1)
      cnt[a.E] = 1;
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= a.E; e += SORT_NT) a.hist[(int64_t)blockIdx.x * (a.E + 1) + e] = cnt[e];
}

// The lanes that hold the same id: ids are below 1 << bits
__device__ __forceinline__ uint64_t same_id(int id, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; b++) {
    const uint64_t bb = __ballot((id >> b) & 1);
    m &= ((id >> b) & 1) ? bb : ~bb;
  }
  return m;
}

__global__ __launch_bounds__(SORT_NT) void sort_place_kernel(SortArgs a) {
  extern __shared__ int at[];  // [SORT_WAVES][E]: counts, then the next place, of each wavefront's pairs
  __shared__ int wsum[SORT_WAVES], wsum2[SORT_WAVES], bad;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, E = a.E;
  const int c = blockIdx.x, chunks = gridDim.x;
  const int seg = a.chunk / SORT_WAVES, first = min(a.P, c * a.chunk + wv * seg), end = min(a.P, first + seg);
  if (tid == 0) bad = 0;
  for (int i = tid; i < SORT_WAVES * E; i += SORT_NT) at[i] = 0;
  __syncthreads();
  for (int p = first + lane; p < end; p += 64) {
    const int e = a.idx[p];
    if (e >= 0 && e < E)
      atomicAdd(&at[wv * E + e], 1);
    else if (e != -1)
      bad = 1;
  }
  __syncthreads();
  // experts e0 .. e1 - 1 of this thread
  const int ept = (E + SORT_NT - 1) / SORT_NT, e0 = min(E, tid * ept), e1 = min(E, e0 + ept);
  int before[4], total[4], sum = 0, hit = 0;  // E <= 1024
#pragma unroll
  for (int i = 0; i < 4; i++) {
    before[i] = total[i] = 0;
    if (e0 + i >= e1) continue;
    if (chunks == 1) {
      for (int w = 0; w < SORT_WAVES; w++) total[i] += at[w * E + e0 + i];
    } else {
      for (int o = 0; o < chunks; o++) {
        const int n = a.hist[(int64_t)o * (E + 1) + e0 + i];
        total[i] += n;
        before[i] += o < c ? n : 0;
      }
    }
    sum += total[i];
    hit += total[i] > 0;
  }
  int incl = sum, hincl = hit;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(incl, o), y = __shfl_up(hincl, o);
    if (lane >= o) incl += x, hincl += y;
  }
  if (lane == 63) wsum[wv] = incl, wsum2[wv] = hincl;
  if (chunks > 1 && c == 0)
    for (int o = tid; o < chunks; o += SORT_NT)
      if (a.hist[(int64_t)o * (E + 1) + E]) bad = 1;
  __syncthreads();
  int run = incl - sum, hrun = hincl - hit;
  for (int i = 0; i < wv; i++) run += wsum[i], hrun += wsum2[i];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if (e0 + i >= e1) continue;
    if (c == 0) {
      a.off[e0 + i] = run;
      if (total[i] > 0) a.active[hrun++] = e0 + i;
    }
    int place = run + before[i];
    for (int w = 0; w < SORT_WAVES; w++) {
      const int n = at[w * E + e0 + i];
      at[w * E + e0 + i] = place;
      place += n;
    }
    run += total[i];
  }
  if (c == 0 && e0 < e1 && e1 == E) {
    a.off[E] = run;
    *a.nact = bad ? -1 : hrun;
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(E);  // ids 0 .. E, E: none
  for (int p0 = first; p0 < end; p0 += 64) {
    const int p = p0 + lane;
    int e = p < end ? a.idx[p] : -1;
    const bool there = e >= 0 && e < E;
    const uint64_t who = same_id(there ? e : E, bits);
    const int rank = __popcll(who & ((1ull << lane) - 1));
    int place = -1;
    if (there) {
      place = at[wv * E + e] + rank;
      a.perm[place] = p;
    }
    if (p < end) a.pos[p] = place;
    __builtin_amdgcn_wave_barrier();
    if (there && rank == 0) at[wv * E + e] = place + __popcll(who);
    __builtin_amdgcn_wave_barrier();
  }
}

// Pairs of a chunk: a multiple of 64 for each wavefront, and so many that no more than SORT_CHUNKS
// rows of counts are read by every workgroup
constexpr int SORT_CHUNKS = 128, SORT_ONE = 1024;
static int sort_chunk(int64_t P) {
  if (P <= SORT_ONE) return SORT_ONE;
  const int64_t c = (P + SORT_CHUNKS - 1) / SORT_CHUNKS;
  return (int)((c + SORT_NT - 1) / SORT_NT * SORT_NT);
}
int sort_chunks(int64_t P) {
  const int c = sort_chunk(P);
  return (int)((P + c - 1) / c);
}
int sort_most_chunks(int64_t P) {
  if (P <= SORT_ONE) return 1;
  return P < (int64_t)SORT_CHUNKS * SORT_NT ? (int)((P + SORT_NT - 1) / SORT_NT) : SORT_CHUNKS;
}

hipError_t launch_sort_pairs(SortArgs a, hipStream_t s) {
  a.chunk = sort_chunk(a.P);
  const int chunks = sort_chunks(a.P);
  if (chunks > 1) {
    hipLaunchKernelGGL(sort_count_kernel, dim3(chunks), dim3(SORT_NT), (a.E + 1) * sizeof(int), s, a);
    if (const hipError_t st = hipGetLastError(); st != hipSuccess) return st;
  }
  hipLaunchKernelGGL(sort_place_kernel, dim3(chunks), dim3(SORT_NT), (size_t)SORT_WAVES * a.E * sizeof(int), s, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------ rows
// A thread takes one piece (16 bytes, or one element where rows are not whole aligned pieces) of a
// token's row for all of its slots.
template <typename U>
__global__ __launch_bounds__(256) void dispatch_kernel(const U *__restrict__ x, uint32_t T_, int k, uint32_t units,
                                                       const int32_t *__restrict__ pos, int64_t rows,
                                                       U *__restrict__ xs) {
  const int64_t n = (int64_t)T_ * units, step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
    const int64_t t = i / units;
    const uint32_t u = (uint32_t)(i - t * units);
    const U v = x[i];
    for (int j = 0; j < k; j++) {
      const int64_t r = pos[t * k + j];
      if (r >= 0 && r < rows) xs[r * units + u] = v;
    }
  }
}

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Piece {
  T v[VEC];
};

template <typename T, int VEC>
__global__ __launch_bounds__(256) void combine_kernel_t(const Piece<T, VEC> *__restrict__ ys, int64_t rows, uint32_t T_,
                                                        int k, uint32_t units, const int32_t *__restrict__ pos,
                                                        const float *__restrict__ w,
                                                        const Piece<T, VEC> *__restrict__ add,
                                                        Piece<T, VEC> *__restrict__ out) {
  const int64_t n = (int64_t)T_ * units, step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
    const int64_t t = i / units;
    const uint32_t u = (uint32_t)(i - t * units);
    float s[VEC] = {};
    for (int j = 0; j < k; j++) {
      const int64_t r = pos[t * k + j];
      if (r < 0 || r >= rows) continue;
      const Piece<T, VEC> y = ys[r * units + u];
      const float wt = w ? w[t * k + j] : 1.0f;
#pragma unroll
      for (int e = 0; e < VEC; e++) s[e] = __builtin_fmaf(wt, (float)y.v[e], s[e]);
    }
    if (add) {
      const Piece<T, VEC> y = add[i];
#pragma unroll
      for (int e = 0; e < VEC; e++) s[e] += (float)y.v[e];
    }
    Piece<T, VEC> o;
#pragma unroll
    for (int e = 0; e < VEC; e++) o.v[e] = (T)s[e];
    out[i] = o;
  }
}

// A wavefront takes a pair: its row of the gradient, and the weight's
template <typename T, int VEC>
__global__ __launch_bounds__(256) void combine_grad_kernel(const Piece<T, VEC> *__restrict__ dout,
                                                           const Piece<T, VEC> *__restrict__ ys, int64_t rows, uint32_t P,
                                                           int k, uint32_t units, const int32_t *__restrict__ pos,
                                                           const float *__restrict__ w, Piece<T, VEC> *__restrict__ dys,
                                                           float *__restrict__ dw) {
  const int lane = threadIdx.x & 63;
  for (uint32_t p = blockIdx.x * 4 + (threadIdx.x >> 6); p < P; p += gridDim.x * 4) {
    const int64_t r = pos[p];
    float sum = 0.0f;
    if (r >= 0 && r < rows) {
      const float wt = w[p];
      const Piece<T, VEC> *d = dout + (int64_t)(p / k) * units;
      for (uint32_t u = lane; u < units; u += 64) {
        const Piece<T, VEC> g = d[u];
        if (dw) {
          const Piece<T, VEC> y = ys[r * units + u];
#pragma unroll
          for (int e = 0; e < VEC; e++) sum = __builtin_fmaf((float)g.v[e], (float)y.v[e], sum);
        }
        if (dys) {
          Piece<T, VEC> o;
#pragma unroll
          for (int e = 0; e < VEC; e++) o.v[e] = (T)(wt * (float)g.v[e]);
          dys[r * units + u] = o;
        }
      }
    }
    if (dw) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
      if (lane == 0) dw[p] = sum;
    }
  }
}

// Workgroups of a launch of 256 threads each, fewer than 2^32 threads; the kernels loop over more
static unsigned groups_of(int64_t n) { return (unsigned)(n < (1 << 23) ? n : (1 << 23)); }

static bool whole(int H, int size, const void *a, const void *b, const void *c = nullptr) {
  return (int64_t)H * size % 16 == 0 && (uintptr_t)a % 16 == 0 && (uintptr_t)b % 16 == 0 && (uintptr_t)c % 16 == 0;
}

hipError_t launch_dispatch(const PairArgs &a, int dtype, const void *x, void *xs, hipStream_t s) {
  const int size = dtype == COLI_F32 ? 4 : 2;
  auto go = [&]<typename U>() {
    const uint32_t units = (uint32_t)((int64_t)a.H * size / (int)sizeof(U));
    const int64_t n = (int64_t)a.T * units;
    hipLaunchKernelGGL(dispatch_kernel<U>, dim3(groups_of((n + 255) / 256)), dim3(256), 0, s, (const U *)x, (uint32_t)a.T,
                       a.k, units, a.pos, a.rows, (U *)xs);
    return hipGetLastError();
  };
  if (whole(a.H, size, x, xs)) return go.template operator()<uint4>();
  return size == 4 ? go.template operator()<uint32_t>() : go.template operator()<uint16_t>();
}

template <typename T>
static hipError_t launch_combine_t(const PairArgs &a, const void *ys, const void *add, void *out, hipStream_t s) {
  auto go = [&]<int VEC>() {
    typedef Piece<T, VEC> piece;
    const uint32_t units = (uint32_t)(a.H / VEC);
    const int64_t n = (int64_t)a.T * units;
    hipLaunchKernelGGL((combine_kernel_t<T, VEC>), dim3(groups_of((n + 255) / 256)), dim3(256), 0, s, (const piece *)ys,
                       a.rows, (uint32_t)a.T, a.k, units, a.pos, a.w, (const piece *)add, (piece *)out);
    return hipGetLastError();
  };
  return whole(a.H, sizeof(T), ys, out, add) ? go.template operator()<16 / sizeof(T)>() : go.template operator()<1>();
}

hipError_t launch_pair_combine(const PairArgs &a, int dtype, const void *ys, const void *add, void *out, hipStream_t s) {
  if (dtype == COLI_F32) return launch_combine_t<float>(a, ys, add, out, s);
  if (dtype == COLI_BF16) return launch_combine_t<bf16_t>(a, ys, add, out, s);
  return launch_combine_t<f16_t>(a, ys, add, out, s);
}

template <typename T>
static hipError_t launch_grad_t(const PairArgs &a, const void *dout, const void *ys, void *dys, float *dw, hipStream_t s) {
  auto go = [&]<int VEC>() {
    typedef Piece<T, VEC> piece;
    const uint32_t units = (uint32_t)(a.H / VEC), P = (uint32_t)a.T * (uint32_t)a.k;
    hipLaunchKernelGGL((combine_grad_kernel<T, VEC>), dim3(groups_of((P + 3) / 4)), dim3(256), 0, s, (const piece *)dout,
                       (const piece *)ys, a.rows, P, a.k, units, a.pos, a.w, (piece *)dys, dw);
    return hipGetLastError();
  };
  return whole(a.H, sizeof(T), dout, ys, dys) ? go.template operator()<16 / sizeof(T)>() : go.template operator()<1>();
}

hipError_t launch_pair_grad(const PairArgs &a, int dtype, const void *dout, const void *ys, void *dys, float *dw,
                            hipStream_t s) {
  if (dtype == COLI_F32) return launch_grad_t<float>(a, dout, ys, dys, dw, s);
  if (dtype == COLI_BF16) return launch_grad_t<bf16_t>(a, dout, ys, dys, dw, s);
  return launch_grad_t<f16_t>(a, dout, ys, dys, dw, s);
}

}  // namespace coli

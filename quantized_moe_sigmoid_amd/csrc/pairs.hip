// pairs.hip — a route's pairs sorted by expert, tokens' rows laid out in that order and summed back,
// and the gradients (batch-union and router items of colibri-strix README, "What's implemented").
//
// All bound by memory: a row is read once for each use and written once. Sums are fp32 in slot order,
// without atomics.
#include <type_traits>

#include "mxfp4_impl.h"

namespace coli {

// ------------------------------------------------------------------ sorting
// A stable counting sort in chunks of pairs, a workgroup each: it counts the pairs before its chunk, in
// it and behind it, which gives every expert's first place, then places its own. A wavefront owns
// consecutive pairs and ranks 64 at a time by ballots. With many pairs the chunks' counts come from a
// kernel of their own (sort_count_kernel), else every workgroup counts all pairs: up to 32768 pairs (32000
// over 256 experts, with a dispatch of short rows: 13.7 us against 17; 65528 over 64 with rows of 2048: 75
// against 59). 65528 pairs: 5 us each kernel; a few hundred pairs in one workgroup 3.6.
constexpr int SORT_WAVES = 16, SORT_NT = 64 * SORT_WAVES;

// One more of expert e of E in cnt; -1 if e is neither an expert nor an empty slot
__device__ __forceinline__ int sort_count(int *cnt, int e, int E) {
  if ((unsigned)e < (unsigned)E) atomicAdd(&cnt[e], 1);
  else if (e != -1) return -1;
  return 0;
}

__global__ __launch_bounds__(SORT_NT) void sort_count_kernel(SortArgs a) {
  extern __shared__ int cnt[];  // [E + 1], the last one: ids out of range
  for (int e = threadIdx.x; e <= a.E; e += SORT_NT) cnt[e] = 0;
  __syncthreads();
  const int first = blockIdx.x * a.chunk, end = min(a.P, first + a.chunk);
  for (int p = first + threadIdx.x; p < end; p += SORT_NT)
    if (sort_count(cnt, a.idx[p], a.E) < 0) cnt[a.E] = 1;
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
  // before [E], total [E]: pairs in earlier chunks, in all; at [SORT_WAVES][E]: counts, then the next
  // place, of each wavefront's pairs
  extern __shared__ int before[];
  __shared__ int wsum[SORT_WAVES], wsum2[SORT_WAVES], bad;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, E = a.E;
  int *total = before + E, *at = total + E, *mine = at + wv * E;
  const int c = blockIdx.x, chunks = gridDim.x;
  const int begin = c * a.chunk, behind = min(a.P, begin + a.chunk);
  const int seg = a.chunk / SORT_WAVES, first = min(a.P, begin + wv * seg), end = min(a.P, first + seg);
  if (tid == 0) bad = 0;
  for (int i = tid; i < (SORT_WAVES + 2) * E; i += SORT_NT) before[i] = 0;
  __syncthreads();
  int wrong = 0;
  for (int p = first + lane; p < end; p += 64) wrong |= sort_count(mine, a.idx[p], E);
  if (a.hist) {
    // rows of counts: a wavefront takes each sixteenth
    for (int e0 = 0; e0 <= E; e0 += 64) {
      const int e = e0 + lane;
      if (e > E) continue;
      int sum = 0, less = 0;
#pragma unroll 4
      for (int o = wv; o < chunks; o += SORT_WAVES) {
        const int n = a.hist[(int64_t)o * (E + 1) + e];
        sum += n;
        less += o < c ? n : 0;
      }
      if (e == E) wrong |= -(sum > 0);
      else if (sum) atomicAdd(&total[e], sum), atomicAdd(&before[e], less);
    }
  } else {
    for (int p = tid; p < begin; p += SORT_NT) wrong |= sort_count(before, a.idx[p], E);
    for (int p = behind + tid; p < a.P; p += SORT_NT) wrong |= sort_count(total, a.idx[p], E);
  }
  if (wrong) bad = 1;
  __syncthreads();
  // thread e: expert e (E <= SORT_NT)
  int n = 0, less = 0;
  if (tid < E) {
    less = before[tid];
    if (a.hist) n = total[tid];
    else {
      n = less + total[tid];
#pragma unroll
      for (int w = 0; w < SORT_WAVES; w++) n += at[w * E + tid];
    }
  }
  const int hit = n > 0;
  int incl = n, hincl = hit;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(incl, o), y = __shfl_up(hincl, o);
    if (lane >= o) incl += x, hincl += y;
  }
  if (lane == 63) wsum[wv] = incl, wsum2[wv] = hincl;
  __syncthreads();
  int run = incl - n, hrun = hincl - hit;
#pragma unroll
  for (int i = 0; i < SORT_WAVES; i++)
    if (i < wv) run += wsum[i], hrun += wsum2[i];
  if (tid < E) {
    if (c == 0) {
      a.off[tid] = run;
      if (hit) a.active[hrun] = tid;
      if (tid == E - 1) {
        a.off[E] = run + n;
        *a.nact = bad ? -1 : hrun + hit;
      }
    }
    int place = run + less;
#pragma unroll
    for (int w = 0; w < SORT_WAVES; w++) {
      const int m = at[w * E + tid];
      at[w * E + tid] = place;
      place += m;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(E);  // ids 0 .. E, E: none
  for (int p0 = first; p0 < end; p0 += 64) {
    const int p = p0 + lane;
    const int e = p < end ? a.idx[p] : -1;
    const bool there = (unsigned)e < (unsigned)E;
    const uint64_t who = same_id(there ? e : E, bits);
    const int rank = __popcll(who & ((1ull << lane) - 1));
    int place = -1;
    if (there) {
      place = mine[e] + rank;
      a.perm[place] = p;
    }
    if (p < end) a.pos[p] = place;
    __builtin_amdgcn_wave_barrier();
    if (there && rank == 0) mine[e] = place + __popcll(who);
    __builtin_amdgcn_wave_barrier();
  }
}

// Pairs of a chunk: 64 for each wavefront, or so many that there are no more than SORT_CHUNKS chunks
constexpr int SORT_SELF = 32768;  // pairs that every workgroup counts itself
static int sort_chunk(int64_t P) {
  const int64_t c = (P + SORT_CHUNKS - 1) / SORT_CHUNKS;
  return (int)((c + SORT_NT - 1) / SORT_NT * SORT_NT);
}
int sort_chunks(int64_t P) {
  const int c = sort_chunk(P);
  return (int)((P + c - 1) / c);
}

hipError_t launch_sort_pairs(SortArgs a, hipStream_t s) {
  a.chunk = sort_chunk(a.P);
  const int chunks = sort_chunks(a.P);
  if (a.P <= SORT_SELF) {
    a.hist = nullptr;
  } else {
    hipLaunchKernelGGL(sort_count_kernel, dim3(chunks), dim3(SORT_NT), (a.E + 1) * sizeof(int), s, a);
    if (const hipError_t st = hipGetLastError(); st != hipSuccess) return st;
  }
  const size_t lds = (size_t)(SORT_WAVES + 2) * a.E * sizeof(int);  // 72 KB for 1024 experts
  static PerDevice allowed;
  if (const hipError_t st = allow_lds(allowed, sort_place_kernel, (SORT_WAVES + 2) * 1024 * sizeof(int)); st != hipSuccess) return st;
  hipLaunchKernelGGL(sort_place_kernel, dim3(chunks), dim3(SORT_NT), lds, s, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------ rows
// A thread takes one piece (16 bytes at any element's address; one element of rows shorter than that) of a
// token's row, for all of its slots. SHIFT: rows are no whole pieces, and the last one is moved back to end
// with its row. Rows of pairs are used once and pass the caches by.
// With rows of no whole pieces taken by element, 4095 tokens, 8 slots, 2047 bf16: combine 152 us, its gradient
// 141, in pieces 36 and 80.
template <typename T, int VEC>
struct VecOf {
  typedef T vec __attribute__((ext_vector_type(VEC)));
  typedef vec type __attribute__((aligned(sizeof(T))));
};
template <typename T>
struct VecOf<T, 1> {
  typedef T type;
};
template <typename T, int VEC>
using piece_of = typename VecOf<T, VEC>::type;

// Piece u of the row at p of H elements
template <typename T, int VEC, bool SHIFT, typename Q>
__device__ __forceinline__ auto piece_at(Q *p, uint32_t u, uint32_t H) {
  const uint32_t at = SHIFT ? min(u * VEC, H - VEC) : u * VEC;
  if constexpr (std::is_const_v<Q>) return reinterpret_cast<const piece_of<T, VEC> *>(p + at);
  else return reinterpret_cast<piece_of<T, VEC> *>(p + at);
}

template <typename T, int VEC>
__device__ __forceinline__ T part(const piece_of<T, VEC> &x, int e) {
  if constexpr (VEC == 1) return x;
  else return x[e];
}
template <typename T, int VEC>
__device__ __forceinline__ void set_part(piece_of<T, VEC> &x, int e, T y) {
  if constexpr (VEC == 1) x = y;
  else x[e] = y;
}

// i = row * units + u; WIDE: i may pass 32 bits
template <bool WIDE>
__device__ __forceinline__ void split(int64_t i, uint32_t units, int64_t &row, uint32_t &u) {
  if constexpr (WIDE) {
    row = i / units;
    u = (uint32_t)(i - row * units);
  } else {
    const uint32_t r = (uint32_t)i / units;
    row = r;
    u = (uint32_t)i - r * units;
  }
}

constexpr int SLOTS = 8;  // rows of a token under way at a time (combine of 2048 x 8 rows of 6144: 4: 42.5 us, 8: 41)

// 8191 tokens, 8 slots, 2048 bf16: 50 to 55 us by the card, 268 MB written and 35 read at 5.5 TB/s. By pair, x
// read eight times through the L2s of other XCDs: 73. Rows of no whole pieces meet in lines, which the L2 puts
// together: 6915 tokens, 8 slots, 406 fp32, with the sort 29 us, past the caches 36, by element 41 (one card).
template <typename T, int VEC, bool SHIFT, bool WIDE>
__global__ __launch_bounds__(256) void dispatch_kernel(const T *__restrict__ x, uint32_t T_, int k, uint32_t H, uint32_t units,
                                                       const int32_t *__restrict__ pos, int64_t rows,
                                                       T *__restrict__ xs) {
  const int64_t n = (int64_t)T_ * units, step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
    int64_t t;
    uint32_t u;
    split<WIDE>(i, units, t, u);
    const piece_of<T, VEC> v = *piece_at<T, VEC, SHIFT>(x + t * H, u, H);
    for (int j0 = 0; j0 < k; j0 += SLOTS) {
      int64_t r[SLOTS];
#pragma unroll
      for (int j = 0; j < SLOTS; j++) r[j] = j0 + j < k ? pos[t * k + j0 + j] : -1;
#pragma unroll
      for (int j = 0; j < SLOTS; j++)
        if (r[j] >= 0 && r[j] < rows) {
          auto *to = piece_at<T, VEC, SHIFT>(xs + r[j] * H, u, H);
          if constexpr (SHIFT) *to = v;
          else __builtin_nontemporal_store(v, to);
        }
    }
  }
}

// 2048 tokens, 8 slots of which a fifth is empty, 6144 fp16, a row added: 40 to 45 us by the card, 211 MB at 4.7
// to 5.3 TB/s; row loads that fill the caches 49, empty slots' loads sent to row 0 instead of left out 41. 4095
// tokens, 8 slots, 2047 bf16: 36 to 40, 140 MB read where 134 are needed: the lines that rows share are not what it
// waits for. add may be out.
template <typename T, int VEC, bool SHIFT, bool WIDE>
__global__ __launch_bounds__(256) void pair_combine_kernel(const T *__restrict__ ys, int64_t rows, uint32_t T_, int k, uint32_t H,
                                                           uint32_t units, const int32_t *__restrict__ pos,
                                                           const float *__restrict__ w, const T *add, T *out) {
  typedef piece_of<T, VEC> piece;
  const int64_t n = (int64_t)T_ * units, step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
    int64_t t;
    uint32_t u;
    split<WIDE>(i, units, t, u);
    float s[VEC] = {};
    for (int j0 = 0; j0 < k; j0 += SLOTS) {
      piece y[SLOTS];
      bool there[SLOTS];
#pragma unroll
      for (int j = 0; j < SLOTS; j++) {
        const int64_t r = j0 + j < k ? pos[t * k + j0 + j] : -1;
        there[j] = r >= 0 && r < rows;
        if (there[j]) y[j] = __builtin_nontemporal_load(piece_at<T, VEC, SHIFT>(ys + r * H, u, H));
      }
#pragma unroll
      for (int j = 0; j < SLOTS; j++) {
        if (!there[j]) continue;
        const float wt = w ? w[t * k + j0 + j] : 1.0f;
#pragma unroll
        for (int e = 0; e < VEC; e++) s[e] = __builtin_fmaf(wt, (float)part<T, VEC>(y[j], e), s[e]);
      }
    }
    if (add) {
      const piece y = *piece_at<T, VEC, SHIFT>(add + t * H, u, H);
#pragma unroll
      for (int e = 0; e < VEC; e++) s[e] += (float)part<T, VEC>(y, e);
    }
    piece o;
#pragma unroll
    for (int e = 0; e < VEC; e++) set_part<T, VEC>(o, e, (T)s[e]);
    T *po = out + t * H;
    if (SHIFT && u == units - 1) {  // the elements before u VEC are another thread's, and add may be out
#pragma unroll
      for (int e = 0; e < VEC; e++)
        if (H - VEC + e >= u * VEC) po[H - VEC + e] = part<T, VEC>(o, e);
    } else {
      __builtin_nontemporal_store(o, piece_at<T, VEC, SHIFT>(po, u, H));
    }
  }
}

// A wavefront takes a pair: its row of the gradient, and the weight's. 4093 tokens, 8 slots, 2048 fp32: 101
// to 110 us by the card, 606 MB moved (570 needed) at 5.6 TB/s. A turn loads 512 pieces and shorter rows repeat their
// last one, so that 16-bit rows of 2048 have half as much under way: 54 us, 285 MB needed; of 2047 80 us.
constexpr int GRAD_AHEAD = 8;  // pieces of a lane under way: 2, 4, 8, 16: 126, 114, 104, 443 us
template <typename T, int VEC, bool SHIFT>
__global__ __launch_bounds__(256) void combine_grad_kernel(const T *__restrict__ dout, const T *__restrict__ ys, int64_t rows,
                                                           uint32_t P, int k, uint32_t H, uint32_t units,
                                                           const int32_t *__restrict__ pos, const float *__restrict__ w,
                                                           T *__restrict__ dys, float *__restrict__ dw) {
  typedef piece_of<T, VEC> piece;
  const int lane = threadIdx.x & 63;
  for (uint32_t p = blockIdx.x * 4 + (threadIdx.x >> 6); p < P; p += gridDim.x * 4) {
    const int64_t r = pos[p];
    float sum = 0.0f;
    if (r >= 0 && r < rows) {
      const float wt = w[p];
      const T *d = dout + (int64_t)(p / k) * H, *yr = ys + r * H;
      for (uint32_t u0 = lane; u0 < units; u0 += 64 * GRAD_AHEAD) {
        piece g[GRAD_AHEAD], y[GRAD_AHEAD];
#pragma unroll
        for (int a = 0; a < GRAD_AHEAD; a++) {
          const uint32_t u = min(u0 + 64 * a, units - 1);
          g[a] = *piece_at<T, VEC, SHIFT>(d, u, H);
          if (dw) y[a] = __builtin_nontemporal_load(piece_at<T, VEC, SHIFT>(yr, u, H));
        }
#pragma unroll
        for (int a = 0; a < GRAD_AHEAD; a++) {
          const uint32_t u = u0 + 64 * a;
          if (u >= units) break;
          if (dw) {
#pragma unroll
            for (int e = 0; e < VEC; e++) {
              const float more = __builtin_fmaf((float)part<T, VEC>(g[a], e), (float)part<T, VEC>(y[a], e), sum);
              sum = !SHIFT || u < units - 1 || H - VEC + e >= u * VEC ? more : sum;  // each element once
            }
          }
          if (dys) {
            piece o;
#pragma unroll
            for (int e = 0; e < VEC; e++) set_part<T, VEC>(o, e, (T)(wt * (float)part<T, VEC>(g[a], e)));
            __builtin_nontemporal_store(o, piece_at<T, VEC, SHIFT>(dys + r * H, u, H));
          }
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

// Rows of H elements of T: go<pieces' elements, whether rows are no whole pieces>()
template <typename T>
static hipError_t by_row(int H, auto go) {
  constexpr int VEC = 16 / sizeof(T);
  if (H < VEC) return go.template operator()<1, false>();
  return H % VEC ? go.template operator()<VEC, true>() : go.template operator()<VEC, false>();
}

template <typename T>
static hipError_t launch_dispatch_t(const PairArgs &a, const T *x, T *xs, hipStream_t s) {
  return by_row<T>(a.H, [&]<int VEC, bool SHIFT>() {
    const uint32_t H = a.H, units = (H + VEC - 1) / VEC;
    const int64_t n = (int64_t)a.T * units;
    auto kernel = n < ((int64_t)1 << 32) ? dispatch_kernel<T, VEC, SHIFT, false> : dispatch_kernel<T, VEC, SHIFT, true>;
    hipLaunchKernelGGL(kernel, dim3(groups_of((n + 255) / 256)), dim3(256), 0, s, x, (uint32_t)a.T, a.k, H, units, a.pos, a.rows, xs);
    return hipGetLastError();
  });
}

hipError_t launch_dispatch(const PairArgs &a, int dtype, const void *x, void *xs, hipStream_t s) {
  if (dtype == COLI_F32) return launch_dispatch_t(a, (const uint32_t *)x, (uint32_t *)xs, s);
  return launch_dispatch_t(a, (const uint16_t *)x, (uint16_t *)xs, s);
}

template <typename T>
static hipError_t launch_combine_t(const PairArgs &a, const void *ys, const void *add, void *out, hipStream_t s) {
  return by_row<T>(a.H, [&]<int VEC, bool SHIFT>() {
    const uint32_t H = a.H, units = (H + VEC - 1) / VEC;
    const int64_t n = (int64_t)a.T * units;
    auto kernel = n < ((int64_t)1 << 32) ? pair_combine_kernel<T, VEC, SHIFT, false> : pair_combine_kernel<T, VEC, SHIFT, true>;
    hipLaunchKernelGGL(kernel, dim3(groups_of((n + 255) / 256)), dim3(256), 0, s, (const T *)ys, a.rows, (uint32_t)a.T, a.k, H,
                       units, a.pos, a.w, (const T *)add, (T *)out);
    return hipGetLastError();
  });
}

hipError_t launch_pair_combine(const PairArgs &a, int dtype, const void *ys, const void *add, void *out, hipStream_t s) {
  if (dtype == COLI_F32) return launch_combine_t<float>(a, ys, add, out, s);
  if (dtype == COLI_BF16) return launch_combine_t<bf16_t>(a, ys, add, out, s);
  return launch_combine_t<f16_t>(a, ys, add, out, s);
}

template <typename T>
static hipError_t launch_grad_t(const PairArgs &a, const void *dout, const void *ys, void *dys, float *dw, hipStream_t s) {
  return by_row<T>(a.H, [&]<int VEC, bool SHIFT>() {
    const uint32_t H = a.H, units = (H + VEC - 1) / VEC, P = (uint32_t)a.T * (uint32_t)a.k;
    hipLaunchKernelGGL((combine_grad_kernel<T, VEC, SHIFT>), dim3(groups_of((P + 3) / 4)), dim3(256), 0, s, (const T *)dout,
                       (const T *)ys, a.rows, P, a.k, H, units, a.pos, a.w, (T *)dys, dw);
    return hipGetLastError();
  });
}

hipError_t launch_pair_grad(const PairArgs &a, int dtype, const void *dout, const void *ys, void *dys, float *dw,
                            hipStream_t s) {
  if (dtype == COLI_F32) return launch_grad_t<float>(a, dout, ys, dys, dw, s);
  if (dtype == COLI_BF16) return launch_grad_t<bf16_t>(a, dout, ys, dys, dw, s);
  return launch_grad_t<f16_t>(a, dout, ys, dys, dw, s);
}

}  // namespace coli

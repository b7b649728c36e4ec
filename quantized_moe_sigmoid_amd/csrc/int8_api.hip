// int8_api.hip — the C entry points of the int8 products with token and channel scales, of the
// pairs' way to their experts and back, and of the route's gradient: host-side validation, workspace
// layout, launches (one stream, no host synchronisation, no device allocation).
#include <algorithm>

#include "coli_internal.h"

namespace coli {

static bool i8_aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
static int i8_dev(hipError_t e) { return e == hipSuccess ? COLI_OK : COLI_E_DEVICE; }
static bool i8_dtype(int d) { return d == COLI_F32 || d == COLI_BF16 || d == COLI_F16; }
static size_t i8_elem(int d) { return d == COLI_F32 ? 4 : 2; }
static size_t i8_al256(size_t v) { return (v + 255) & ~(size_t)255; }

constexpr int32_t I8_MAX_K = 1 << 17;  // 127 * 128 * K < 2^31

// A workspace: quantised activations (codes, scales), the row tiles of a route, then the down product's
// fp32 rows.
struct I8Ws {
  size_t aq, as, tiles, ntiles, y, total;
};

static I8Ws i8_ws(int64_t rows, int K, int64_t tiles, size_t y_bytes) {
  I8Ws L{};
  size_t o = 0;
  L.aq = o;      o = i8_al256(o + (size_t)rows * i8_padded(K));
  L.as = o;      o = i8_al256(o + (size_t)rows * sizeof(float));
  L.tiles = o;   o = i8_al256(o + tiles * sizeof(int4));
  L.ntiles = o;  o = i8_al256(o + (tiles ? sizeof(int32_t) : 0));
  L.y = o;       o = i8_al256(o + y_bytes);
  L.total = o;
  return L;
}

static int64_t i8_rows(const coli_moe_cfg &c, int32_t T) { return (int64_t)T * (c.top_k + c.has_shared); }
static int64_t i8_tiles(const coli_moe_cfg &c, int32_t T) { return i8_tile_cap(T, c.top_k, c.n_experts, c.has_shared); }
static I8Ws i8_ws_gateup(const coli_moe_cfg &c, int32_t T) { return i8_ws(T, c.hidden, i8_tiles(c, T), 0); }
static I8Ws i8_ws_down(const coli_moe_cfg &c, int32_t T) {
  const int64_t R = i8_rows(c, T);
  return i8_ws(R, c.ffn, i8_tiles(c, T), (size_t)R * c.hidden * sizeof(float));
}

static int check_linear(int32_t M, int32_t N, int32_t K) {
  if (M < 0 || N < 0 || K <= 0) return COLI_E_INVALID;
  if (K % 16 || K > I8_MAX_K || M > (1 << 20) || N > (1 << 20)) return COLI_E_UNSUPPORTED;
  if ((int64_t)M * K >= ((int64_t)1 << 37) || (int64_t)N * K >= ((int64_t)1 << 37)) return COLI_E_UNSUPPORTED;
  return COLI_OK;
}

static int check_experts(const coli_moe_cfg *cfg, const coli_moe_weights *w, int dtype, int32_t T) {
  int st;
  if ((st = check_cfg(cfg))) return st;
  if (cfg->wfmt != COLI_W_INT8 || cfg->scale_group != 0 || !i8_dtype(dtype)) return COLI_E_INVALID;
  if ((st = check_T(cfg, T))) return st;
  return T == 0 ? COLI_OK : check_weights(w, true, false);
}

static I8Args expert_args(const coli_moe_cfg &c, const coli_moe_weights &w, int32_t T, const int32_t *off,
                          const int32_t *perm, const int32_t *active, const int32_t *nact) {
  I8Args a{};
  a.wq = static_cast<const int8_t *>(w.experts);
  a.ws = w.scales;
  a.wq_stride = (int64_t)coli_moe_blob_bytes(&c);
  a.ws_stride = (int64_t)coli_moe_scales_per_expert(&c);
  a.M = T;
  a.E = c.n_experts;
  a.k = c.top_k;
  a.has_shared = c.has_shared;
  a.off = off;
  a.perm = perm;
  a.active = active;
  a.nact = nact;
  return a;
}

// A dense product on the tiled kernels? The kernel for few rows goes through the weights once for each 64
// rows. us, few rows and tiled, K = 6144: N = 12288: 2 rows 19 and 21, 4 20 and 21, 16 25 and 22, 64 49 and
// 22; N = 2048: 16 rows 14 and 21, 33 19 and 21, 64 22 and 21; 200 x 512 22 and 21, 1000 x 128 25 and 23.
// K = 2048: 16 x 6144 11 and 12, 16 x 40000 25 and 24, 33 x 512 12 and 12.
static bool i8_linear_tiled(int32_t M, int32_t N) { return M > 48 || (M > 8 && (int64_t)M * N > 150000); }

// The kernel for few rows reads an expert's weights once for each 16 rows, the tiled one fills the card
// with about eight tiles to a CU and reads faster then. us, few rows and tiled, of bf16 (events; down with its
// quantisation and combine):
//   experts, slots to a token                    tokens  gate/up        down
//   256 of 6144 x 2048, 8 and a shared one       17      436 and 406    248 and 243
//                                                24      606 and 566    313 and 302
//                                                64      1013 and 901   494 and 467
//   64 of 2048 x 1024, 8 and a shared one        17      54 and 58      37 and 43
//                                                64      65 and 73      44 and 51
//                                                200     112 and 75     80 and 56
//   32 of 1024 x 512, 1                          300     15 and 20      17 and 20
//   8 of 4096 x 2048, 1                          64      38 and 46      24 and 29
//                                                128     49 and 48      31 and 30
//   8 of 6144 x 2048, 2                          200     138 and 66     93 and 40
// (64 x 64 and 64 x 128 tiles over a route: slower than either but for 600 tokens over 32 of 1024 x 512, 24 and 26.)
static bool i8_experts_tiled(const I8Args &a) {
  const int64_t P = (int64_t)a.M * a.k, hit = std::min<int64_t>(P, a.E);
  return P > 12 * (int64_t)a.E || (P > 128 && hit * a.N >= 2048 * 128);
}

// The tiled kernel's offsets into the activations and the output have 32 bits, which check_cfg's and check_T's
// limits keep: at most 65535 pairs and as many tokens, rows of fewer than 7168 values of 4 bytes.
static_assert(gemv_lds(7168) > GEMV_LDS_LIMIT && 2 * 65535ll * 7168 * 4 < (1ll << 32) - 65536);

static hipError_t launch_experts(I8Mode mode, int dtype, I8Args &a, uint8_t *ws, const I8Ws &L, hipStream_t s) {
  if (!i8_experts_tiled(a)) return launch_i8_gemv(mode, dtype, a, s);
  a.tiles = reinterpret_cast<int4 *>(ws + L.tiles);
  a.ntiles = reinterpret_cast<int32_t *>(ws + L.ntiles);
  return launch_i8_tile(mode, dtype, a, s);
}

static int check_pairs(int dtype, int32_t T, int32_t k, int32_t H, int64_t rows) {
  if (!i8_dtype(dtype) || T < 0 || k <= 0 || H <= 0 || rows < 0) return COLI_E_INVALID;
  if ((int64_t)T * k >= (1 << 30) || (int64_t)T * H >= ((int64_t)1 << 40) || rows >= ((int64_t)1 << 40) / H)
    return COLI_E_UNSUPPORTED;
  return COLI_OK;
}

}  // namespace coli

using namespace coli;

extern "C" {

int coli_moe_int8_quantize(const void *x, int dtype, int64_t rows, int32_t cols, int8_t *codes, float *scales,
                           void *stream) {
  if (rows < 0 || cols <= 0 || !i8_dtype(dtype)) return COLI_E_INVALID;
  if (cols % 16 || cols > I8_MAX_K || rows >= ((int64_t)1 << 31) || rows >= ((int64_t)1 << 40) / cols)
    return COLI_E_UNSUPPORTED;
  if (rows == 0) return COLI_OK;
  if (!x || !codes || !scales) return COLI_E_INVALID;
  if (!i8_aligned(x, 16) || !i8_aligned(codes, 16) || !i8_aligned(scales, 4)) return COLI_E_ALIGN;
  return i8_dev(launch_i8_quantize(x, dtype, rows, cols, cols, codes, scales, static_cast<hipStream_t>(stream)));
}

size_t coli_moe_int8_linear_workspace_bytes(int32_t M_max, int32_t N, int32_t K) {
  if (check_linear(M_max, N, K) != COLI_OK) return 0;
  return i8_ws(M_max > 0 ? M_max : 1, K, 0, 0).total;
}

int coli_moe_int8_linear(const void *x, int dtype, const int8_t *codes, const float *scales, const float *bias, int32_t M,
                         int32_t N, int32_t K, void *y, void *workspace, size_t ws_bytes, void *stream) {
  int st;
  if (!i8_dtype(dtype)) return COLI_E_INVALID;
  if ((st = check_linear(M, N, K))) return st;
  if (M == 0 || N == 0) return COLI_OK;
  if (!x || !codes || !scales || !y) return COLI_E_INVALID;
  if (!i8_aligned(x, 16) || !i8_aligned(codes, 16) || !i8_aligned(y, 16) || !i8_aligned(scales, 4) || !i8_aligned(bias, 4))
    return COLI_E_ALIGN;
  const I8Ws L = i8_ws(M, K, 0, 0);
  if (!workspace || ws_bytes < L.total) return COLI_E_WORKSPACE;
  if (!i8_aligned(workspace, 256)) return COLI_E_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  I8Args a{};
  a.wq = codes;
  a.ws = scales;
  a.bias = bias;
  a.N = N;
  a.K = K;
  a.M = M;
  a.out = y;
  int8_t *aq = reinterpret_cast<int8_t *>(ws + L.aq);
  float *as = reinterpret_cast<float *>(ws + L.as);
  if (i8_gemv_from_x(a))
    a.x = x;
  else if ((st = i8_dev(launch_i8_quantize(x, dtype, M, K, i8_padded(K), aq, as, s))))
    return st;
  a.aq = aq;
  a.as = as;
  return i8_dev(i8_linear_tiled(M, N) ? launch_i8_tile(I8_LINEAR, dtype, a, s) : launch_i8_gemv(I8_LINEAR, dtype, a, s));
}

size_t coli_moe_int8_experts_workspace_bytes(const coli_moe_cfg *cfg, int32_t T_max) {
  if (check_cfg(cfg) != COLI_OK || cfg->wfmt != COLI_W_INT8 || cfg->scale_group != 0 || check_T(cfg, T_max) != COLI_OK)
    return 0;
  const int32_t T = T_max > 0 ? T_max : 1;
  const size_t g = i8_ws_gateup(*cfg, T).total, d = i8_ws_down(*cfg, T).total;
  return g > d ? g : d;
}

int coli_moe_int8_gate_up(const coli_moe_cfg *cfg, const coli_moe_weights *w, const void *x, int dtype, int32_t T,
                          const int32_t *expert_off, const int32_t *pair_perm, const int32_t *active,
                          const int32_t *n_active, void *h, void *workspace, size_t ws_bytes, void *stream) {
  int st;
  if ((st = check_experts(cfg, w, dtype, T))) return st;
  if (T == 0) return COLI_OK;
  if (!x || !expert_off || !pair_perm || !active || !n_active || !h) return COLI_E_INVALID;
  if (!i8_aligned(x, 16) || !i8_aligned(h, 16) || !i8_aligned(expert_off, 4) || !i8_aligned(pair_perm, 4) ||
      !i8_aligned(active, 4) || !i8_aligned(n_active, 4))
    return COLI_E_ALIGN;
  const I8Ws L = i8_ws_gateup(*cfg, T);
  if (!workspace || ws_bytes < L.total) return COLI_E_WORKSPACE;
  if (!i8_aligned(workspace, 256)) return COLI_E_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  I8Args a = expert_args(*cfg, *w, T, expert_off, pair_perm, active, n_active);
  a.N = cfg->ffn;
  a.K = cfg->hidden;
  int8_t *aq = reinterpret_cast<int8_t *>(ws + L.aq);
  float *as = reinterpret_cast<float *>(ws + L.as);
  if (i8_gemv_from_x(a))
    a.x = x;
  else if ((st = i8_dev(launch_i8_quantize(x, dtype, T, cfg->hidden, i8_padded(cfg->hidden), aq, as, s))))
    return st;
  a.aq = aq;
  a.as = as;
  a.out = h;
  return i8_dev(launch_experts(I8_GATEUP, dtype, a, ws, L, s));
}

int coli_moe_int8_down(const coli_moe_cfg *cfg, const coli_moe_weights *w, const void *h, int dtype, int32_t T,
                       const int32_t *topk_idx, const float *topk_w, const int32_t *expert_off,
                       const int32_t *pair_perm, const int32_t *active, const int32_t *n_active, void *out,
                       void *workspace, size_t ws_bytes, void *stream) {
  int st;
  if ((st = check_experts(cfg, w, dtype, T))) return st;
  if (T == 0) return COLI_OK;
  if (!h || !topk_idx || !topk_w || !expert_off || !pair_perm || !active || !n_active || !out) return COLI_E_INVALID;
  if (!i8_aligned(h, 16) || !i8_aligned(out, 16) || !i8_aligned(topk_idx, 4) || !i8_aligned(topk_w, 4) ||
      !i8_aligned(expert_off, 4) || !i8_aligned(pair_perm, 4) || !i8_aligned(active, 4) || !i8_aligned(n_active, 4))
    return COLI_E_ALIGN;
  const I8Ws L = i8_ws_down(*cfg, T);
  if (!workspace || ws_bytes < L.total) return COLI_E_WORKSPACE;
  if (!i8_aligned(workspace, 256)) return COLI_E_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  I8Args a = expert_args(*cfg, *w, T, expert_off, pair_perm, active, n_active);
  a.wq += 2 * (int64_t)cfg->ffn * cfg->hidden;  // gate and up rows
  a.ws += 2 * (int64_t)cfg->ffn;
  a.N = cfg->hidden;
  a.K = cfg->ffn;
  int8_t *aq = reinterpret_cast<int8_t *>(ws + L.aq);
  float *as = reinterpret_cast<float *>(ws + L.as), *y = reinterpret_cast<float *>(ws + L.y);
  const bool fused = i8_down_fused(a);
  if (fused && i8_down_from_x(a))
    a.x = h;
  else if ((st = i8_dev(launch_i8_quantize(h, dtype, i8_rows(*cfg, T), cfg->ffn, i8_padded(cfg->ffn), aq, as, s))))
    return st;
  a.aq = aq;
  a.as = as;
  if (fused) return i8_dev(launch_i8_down(a, topk_idx, topk_w, out, dtype, s));
  a.out = y;
  if ((st = i8_dev(launch_experts(I8_DOWN, dtype, a, ws, L, s)))) return st;
  return i8_dev(launch_mx_combine(y, topk_idx, topk_w, T, cfg->top_k, cfg->n_experts, cfg->hidden, cfg->has_shared, out,
                                  dtype, s));
}

size_t coli_moe_sort_pairs_workspace_bytes(int64_t P, int32_t n_experts) {
  if (P < 0 || P >= (1 << 30) || n_experts <= 0 || n_experts > 1024) return 0;
  // as many chunks as there are at most: enough for fewer pairs too
  return i8_al256((size_t)SORT_CHUNKS * (n_experts + 1) * sizeof(int32_t));
}

int coli_moe_sort_pairs(const int32_t *topk_idx, int32_t T, int32_t k, int32_t n_experts, int32_t *expert_off,
                        int32_t *pair_perm, int32_t *pair_pos, int32_t *active, int32_t *n_active, void *workspace,
                        size_t ws_bytes, void *stream) {
  if (T < 0 || k <= 0 || n_experts <= 0) return COLI_E_INVALID;
  const int64_t P = (int64_t)T * k;
  if (P >= (1 << 30) || n_experts > 1024) return COLI_E_UNSUPPORTED;
  if (T == 0) return COLI_OK;
  if (!topk_idx || !expert_off || !pair_perm || !pair_pos || !active || !n_active) return COLI_E_INVALID;
  if (!i8_aligned(topk_idx, 4) || !i8_aligned(expert_off, 4) || !i8_aligned(pair_perm, 4) || !i8_aligned(pair_pos, 4) ||
      !i8_aligned(active, 4) || !i8_aligned(n_active, 4))
    return COLI_E_ALIGN;
  if (!workspace || ws_bytes < (size_t)sort_chunks(P) * (n_experts + 1) * sizeof(int32_t)) return COLI_E_WORKSPACE;
  if (!i8_aligned(workspace, 256)) return COLI_E_ALIGN;
  SortArgs a{};
  a.idx = topk_idx;
  a.P = (int32_t)P;
  a.E = n_experts;
  a.hist = static_cast<int32_t *>(workspace);
  a.off = expert_off;
  a.perm = pair_perm;
  a.pos = pair_pos;
  a.active = active;
  a.nact = n_active;
  return i8_dev(launch_sort_pairs(a, static_cast<hipStream_t>(stream)));
}

int coli_moe_dispatch(const void *x, int dtype, int32_t T, int32_t k, int32_t H, const int32_t *pair_pos, int64_t rows,
                      void *xs, void *stream) {
  const int st = check_pairs(dtype, T, k, H, rows);
  if (st || T == 0 || rows == 0) return st;
  if (!x || !pair_pos || !xs) return COLI_E_INVALID;
  const size_t e = i8_elem(dtype);
  if (!i8_aligned(x, e) || !i8_aligned(xs, e) || !i8_aligned(pair_pos, 4)) return COLI_E_ALIGN;
  const PairArgs a{T, k, H, pair_pos, nullptr, rows};
  return i8_dev(launch_dispatch(a, dtype, x, xs, static_cast<hipStream_t>(stream)));
}

int coli_moe_combine(const void *ys, int dtype, int64_t rows, int32_t T, int32_t k, int32_t H, const int32_t *pair_pos,
                     const float *topk_w, const void *add, void *out, void *stream) {
  const int st = check_pairs(dtype, T, k, H, rows);
  if (st || T == 0) return st;
  if ((!ys && rows > 0) || !pair_pos || !out) return COLI_E_INVALID;
  const size_t e = i8_elem(dtype);
  if (!i8_aligned(ys, e) || !i8_aligned(add, e) || !i8_aligned(out, e) || !i8_aligned(pair_pos, 4) || !i8_aligned(topk_w, 4))
    return COLI_E_ALIGN;
  const PairArgs a{T, k, H, pair_pos, topk_w, rows};
  return i8_dev(launch_pair_combine(a, dtype, ys, add, out, static_cast<hipStream_t>(stream)));
}

int coli_moe_combine_backward(const void *dout, const void *ys, int dtype, int64_t rows, int32_t T, int32_t k, int32_t H,
                              const int32_t *pair_pos, const float *topk_w, void *dys, float *dtopk_w, void *stream) {
  const int st = check_pairs(dtype, T, k, H, rows);
  if (st || T == 0) return st;
  if (!dout || !pair_pos || !topk_w || (!dys && !dtopk_w) || (dtopk_w && !ys && rows > 0)) return COLI_E_INVALID;
  const size_t e = i8_elem(dtype);
  if (!i8_aligned(dout, e) || !i8_aligned(ys, e) || !i8_aligned(dys, e) || !i8_aligned(pair_pos, 4) ||
      !i8_aligned(topk_w, 4) || !i8_aligned(dtopk_w, 4))
    return COLI_E_ALIGN;
  const PairArgs a{T, k, H, pair_pos, topk_w, rows};
  return i8_dev(launch_pair_grad(a, dtype, dout, ys, dys, dtopk_w, static_cast<hipStream_t>(stream)));
}

int coli_moe_route_logits_backward(const coli_moe_router *r, const void *z, int dtype, int32_t T, const int32_t *topk_idx,
                                   const float *dtopk_w, void *dz, void *stream) {
  int st;
  if (!i8_dtype(dtype) || T < 0) return COLI_E_INVALID;
  if ((st = check_router(r))) return st;
  if (T > (1 << 26) - 4) return COLI_E_UNSUPPORTED;  // 64 threads a token, fewer than 2^32
  if (T == 0) return COLI_OK;
  if (!z || !topk_idx || !dtopk_w || !dz) return COLI_E_INVALID;
  const size_t e = i8_elem(dtype);
  if (!i8_aligned(z, e) || !i8_aligned(dz, e) || !i8_aligned(topk_idx, 4) || !i8_aligned(dtopk_w, 4)) return COLI_E_ALIGN;
  RouteGradArgs a{};
  a.T = T;
  a.E = r->n_experts;
  a.k = r->top_k;
  a.softmax = r->score == COLI_SCORE_SOFTMAX;
  a.renorm = r->renorm;
  a.scale = r->scale;
  a.idx = topk_idx;
  a.dw = dtopk_w;
  return i8_dev(launch_route_grad(a, z, dtype, dz, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

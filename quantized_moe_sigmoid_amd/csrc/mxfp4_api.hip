// mxfp4_api.hip — the C entry points of the route from logits and of the MXFP4 x MXFP4
// operators: host-side validation, workspace layout, launches (one stream, no host
// synchronisation, no device allocation).
#include <algorithm>

#include "coli_internal.h"

namespace coli {

static bool mx_aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
static int mx_dev(hipError_t e) { return e == hipSuccess ? COLI_OK : COLI_E_DEVICE; }
static bool mx_dtype(int d) { return d == COLI_F32 || d == COLI_BF16 || d == COLI_F16; }
static size_t mx_al256(size_t v) { return (v + 255) & ~(size_t)255; }

// A workspace: quantised activations (codes, E8M0 bytes), the row tiles of a route, then the
// down product's fp32 rows or a dense product's padded weight scales.
struct MxWs {
  size_t ac, as, tiles, ntiles, y, total;
};

static MxWs mx_ws(int64_t rows, int K, int64_t tiles, size_t y_bytes) {
  MxWs L{};
  const size_t kp = (size_t)mx_padded(K);
  size_t o = 0;
  L.ac = o;  o = mx_al256(o + rows * (kp / 2));
  L.as = o;  o = mx_al256(o + rows * (kp / 32));
  L.tiles = o;   o = mx_al256(o + tiles * sizeof(int4));
  L.ntiles = o;  o = mx_al256(o + (tiles ? sizeof(int32_t) : 0));
  L.y = o;   o = mx_al256(o + y_bytes);
  L.total = o;
  return L;
}

static int64_t mx_rows(const coli_moe_cfg &c, int32_t T) { return (int64_t)T * (c.top_k + c.has_shared); }
static int64_t mx_tiles(const coli_moe_cfg &c, int32_t T) {
  return mx_tile_cap(T, c.top_k, c.n_experts, c.has_shared);
}
static MxWs mx_ws_gateup(const coli_moe_cfg &c, int32_t T) { return mx_ws(T, c.hidden, mx_tiles(c, T), 0); }
static MxWs mx_ws_down(const coli_moe_cfg &c, int32_t T) {
  const int64_t R = mx_rows(c, T);
  return mx_ws(R, c.ffn, mx_tiles(c, T), (size_t)R * c.hidden * sizeof(float));
}
static MxWs mx_ws_linear(int32_t M, int32_t N, int32_t K) {
  return mx_ws(M, K, 0, mx_linear_tiled(M, N) ? (size_t)N * (mx_padded(K) / 32) : 0);
}

// Blocks of 32 of one launch: two threads each, of fewer than 2^32
constexpr int64_t MX_MAX_BLOCKS = ((int64_t)1 << 31) - 128;

static int check_linear(int32_t M, int32_t N, int32_t K) {
  if (M < 0 || N < 0 || K <= 0) return COLI_E_INVALID;
  if (K % 32 || K > (1 << 20) || M > (1 << 20) || N > (1 << 20)) return COLI_E_UNSUPPORTED;
  const int64_t nbp = mx_padded(K) / 32;
  if (M * nbp > MX_MAX_BLOCKS || N * nbp > 4 * MX_MAX_BLOCKS) return COLI_E_UNSUPPORTED;
  return COLI_OK;
}

static int check_experts(const coli_moe_cfg *cfg, const coli_moe_weights *w, int dtype, int32_t T) {
  int st;
  if ((st = check_cfg(cfg))) return st;
  if (cfg->wfmt != COLI_W_MXFP4 || !mx_dtype(dtype)) return COLI_E_INVALID;
  if ((st = check_T(cfg, T))) return st;
  return T == 0 ? COLI_OK : check_weights(w, true, false);
}

static MxArgs expert_args(const coli_moe_cfg &c, const coli_moe_weights &w, int32_t T, const int32_t *off,
                          const int32_t *perm, const int32_t *active, const int32_t *nact) {
  MxArgs a{};
  a.wc = static_cast<const uint8_t *>(w.experts);
  a.ws = reinterpret_cast<const uint8_t *>(w.scales);
  a.wc_stride = (int64_t)coli_moe_blob_bytes(&c);
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

static hipError_t launch_experts(MxMode mode, int dtype, MxArgs &a, uint8_t *ws, const MxWs &L, hipStream_t s) {
  a.ws_pitch = a.K / 32;
  // The kernel for few rows up to 512 pairs (decode batches), the tiled one past them. What makes
  // the difference is rows to an expert, the shared one's among them: the first kernel reads the
  // weights once for each 16, the second takes at least a whole tile's time. us, few rows and tiled:
  //   experts of 4096 x 2048            gate/up            down (few rows: pairs, combine)
  //   8, 1 to a token: 64 tokens        21 and 30          19 and 22
  //     128 tokens                      33 and 30          23 and 23
  //     500 tokens                      75 and 42          53 and 33
  //     500, with a shared expert       157 and 44         82 and 38
  //   16, 2 to a token: 64 tokens       38 and 40          29 and 23
  //     250 tokens                      82 and 43          56 and 28
  //   64, 8 to a token: 64 tokens       139 and 107        102 and 70
  //   256 of 6144 x 2048, 8: 64 tokens  543 and 533        441 and 292
  // So the bound by pairs is right where an expert has up to about 16 rows, and late for few experts.
  // The tiled kernel's offsets into the activations and the output have 32 bits.
  const int64_t rows = (int64_t)a.M * (a.k + a.has_shared), widest = std::max<int64_t>((int64_t)a.N * 4, mx_padded(a.K) / 2);
  if ((int64_t)a.M * a.k <= LOCAL_GROUP_MAX_P || rows * widest >= ((int64_t)1 << 32) - 65536)
    return launch_mx_gemv(mode, dtype, a, s);
  a.tiles = reinterpret_cast<int4 *>(ws + L.tiles);
  a.ntiles = reinterpret_cast<int32_t *>(ws + L.ntiles);
  return launch_mx_tile(mode, dtype, a, s);
}

}  // namespace coli

using namespace coli;

extern "C" {

int coli_moe_route_logits(const coli_moe_router *r, const void *z, int dtype, int32_t T, const float *bias,
                          int32_t *topk_idx, float *topk_w, void *stream) {
  if (!r || !mx_dtype(dtype) || T < 0) return COLI_E_INVALID;
  if (r->n_experts <= 0 || r->top_k <= 0 || r->n_group <= 0 || r->topk_group <= 0) return COLI_E_INVALID;
  if (r->n_experts % r->n_group || r->topk_group > r->n_group) return COLI_E_INVALID;
  if (r->top_k > r->topk_group * (r->n_experts / r->n_group)) return COLI_E_INVALID;
  if ((r->group_top != 1 && r->group_top != 2) || (r->renorm != 0 && r->renorm != 1)) return COLI_E_INVALID;
  if (r->score != COLI_SCORE_SIGMOID && r->score != COLI_SCORE_SOFTMAX) return COLI_E_INVALID;
  if (!(r->scale == r->scale)) return COLI_E_INVALID;  // NaN
  if (r->n_experts > 1024 || r->n_group > 64 || r->top_k > 64) return COLI_E_UNSUPPORTED;
  if (T > (1 << 26) - 4) return COLI_E_UNSUPPORTED;  // 64 threads a token, fewer than 2^32
  if (T == 0) return COLI_OK;
  if (!z || !topk_idx || !topk_w) return COLI_E_INVALID;
  if (!mx_aligned(z, dtype == COLI_F32 ? 4 : 2) || !mx_aligned(topk_idx, 4) || !mx_aligned(topk_w, 4) ||
      !mx_aligned(bias, 4))
    return COLI_E_ALIGN;
  RouteLogitsArgs a{};
  a.T = T;
  a.E = r->n_experts;
  a.k = r->top_k;
  a.G = r->n_group;
  a.Gk = r->topk_group;
  a.group_top = r->group_top;
  a.softmax = r->score == COLI_SCORE_SOFTMAX;
  a.renorm = r->renorm;
  a.scale = r->scale;
  a.bias = bias;
  a.idx = topk_idx;
  a.w = topk_w;
  return mx_dev(launch_route_logits(a, z, dtype, static_cast<hipStream_t>(stream)));
}

static int check_mx_rows(const void *x, int dtype, int64_t rows, int32_t cols, const void *codes, const void *scales) {
  if (rows < 0 || cols <= 0 || !mx_dtype(dtype)) return COLI_E_INVALID;
  if (cols % 32 || rows > MX_MAX_BLOCKS / (cols / 32)) return COLI_E_UNSUPPORTED;
  if (rows == 0) return COLI_OK;
  if (!x || !codes || !scales) return COLI_E_INVALID;
  if (!mx_aligned(x, 16) || !mx_aligned(codes, 16)) return COLI_E_ALIGN;
  return COLI_OK;
}

int coli_moe_mxfp4_quantize(const void *x, int dtype, int64_t rows, int32_t cols, uint8_t *codes, uint8_t *scales,
                            void *stream) {
  const int st = check_mx_rows(x, dtype, rows, cols, codes, scales);
  if (st || rows == 0) return st;
  return mx_dev(launch_mx_quantize(x, dtype, rows * (cols / 32), codes, scales, static_cast<hipStream_t>(stream)));
}

int coli_moe_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int32_t cols, void *out,
                              int dtype, void *stream) {
  const int st = check_mx_rows(out, dtype, rows, cols, codes, scales);
  if (st || rows == 0) return st;
  return mx_dev(launch_mx_dequantize(codes, scales, rows * (cols / 32), out, dtype, static_cast<hipStream_t>(stream)));
}

size_t coli_moe_mxfp4_linear_workspace_bytes(int32_t M_max, int32_t N, int32_t K) {
  if (check_linear(M_max, N, K) != COLI_OK) return 0;
  return mx_ws_linear(M_max > 0 ? M_max : 1, N, K).total;
}

int coli_moe_mxfp4_linear(const void *x, int dtype, const uint8_t *codes, const uint8_t *scales, int32_t M, int32_t N,
                          int32_t K, void *y, void *workspace, size_t ws_bytes, void *stream) {
  int st;
  if (!mx_dtype(dtype)) return COLI_E_INVALID;
  if ((st = check_linear(M, N, K))) return st;
  if (M == 0 || N == 0) return COLI_OK;
  if (!x || !codes || !scales || !y) return COLI_E_INVALID;
  if (!mx_aligned(x, 16) || !mx_aligned(codes, 16) || !mx_aligned(y, 16)) return COLI_E_ALIGN;
  const MxWs L = mx_ws_linear(M, N, K);
  if (!workspace || ws_bytes < L.total) return COLI_E_WORKSPACE;
  if (!mx_aligned(workspace, 256)) return COLI_E_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  MxArgs a{};
  a.wc = codes;
  a.ws = scales;
  a.N = N;
  a.K = K;
  a.ac = ws + L.ac;
  a.as = ws + L.as;
  a.M = M;
  a.out = y;
  a.ws_pitch = K / 32;
  if (mx_gemv_from_x(a))
    a.x = x;
  else if ((st = mx_dev(launch_mx_quantize_rows(x, dtype, M, K, ws + L.ac, ws + L.as, s))))
    return st;
  if (!mx_linear_tiled(M, N)) return mx_dev(launch_mx_gemv(MX_LINEAR, dtype, a, s));
  if (K % 128 || K < 512 || !mx_aligned(scales, 4)) {  // the tiled kernel loads 16 scales at a dword's address
    if ((st = mx_dev(launch_mx_pad_scales(scales, N, K, ws + L.y, s)))) return st;
    a.ws = ws + L.y;
    a.ws_pitch = mx_padded(K) / 32;
  }
  return mx_dev(launch_mx_tile(MX_LINEAR, dtype, a, s));
}

size_t coli_moe_mxfp4_experts_workspace_bytes(const coli_moe_cfg *cfg, int32_t T_max) {
  if (check_cfg(cfg) != COLI_OK || cfg->wfmt != COLI_W_MXFP4 || check_T(cfg, T_max) != COLI_OK) return 0;
  const int32_t T = T_max > 0 ? T_max : 1;
  const size_t g = mx_ws_gateup(*cfg, T).total, d = mx_ws_down(*cfg, T).total;
  return g > d ? g : d;
}

int coli_moe_mxfp4_gate_up(const coli_moe_cfg *cfg, const coli_moe_weights *w, const void *x, int dtype, int32_t T,
                           const int32_t *expert_off, const int32_t *pair_perm, const int32_t *active,
                           const int32_t *n_active, void *h, void *workspace, size_t ws_bytes, void *stream) {
  int st;
  if ((st = check_experts(cfg, w, dtype, T))) return st;
  if (T == 0) return COLI_OK;
  if (!x || !expert_off || !pair_perm || !active || !n_active || !h) return COLI_E_INVALID;
  if (!mx_aligned(x, 16) || !mx_aligned(h, 16) || !mx_aligned(expert_off, 4) || !mx_aligned(pair_perm, 4) ||
      !mx_aligned(active, 4) || !mx_aligned(n_active, 4))
    return COLI_E_ALIGN;
  const MxWs L = mx_ws_gateup(*cfg, T);
  if (!workspace || ws_bytes < L.total) return COLI_E_WORKSPACE;
  if (!mx_aligned(workspace, 256)) return COLI_E_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  MxArgs a = expert_args(*cfg, *w, T, expert_off, pair_perm, active, n_active);
  a.N = cfg->ffn;
  a.K = cfg->hidden;
  if (mx_gemv_from_x(a))
    a.x = x;
  else if ((st = mx_dev(launch_mx_quantize_rows(x, dtype, T, cfg->hidden, ws + L.ac, ws + L.as, s))))
    return st;
  a.ac = ws + L.ac;
  a.as = ws + L.as;
  a.out = h;
  return mx_dev(launch_experts(MX_GATEUP, dtype, a, ws, L, s));
}

int coli_moe_mxfp4_down(const coli_moe_cfg *cfg, const coli_moe_weights *w, const void *h, int dtype, int32_t T,
                        const int32_t *topk_idx, const float *topk_w, const int32_t *expert_off,
                        const int32_t *pair_perm, const int32_t *active, const int32_t *n_active, void *out,
                        void *workspace, size_t ws_bytes, void *stream) {
  int st;
  if ((st = check_experts(cfg, w, dtype, T))) return st;
  if (T == 0) return COLI_OK;
  if (!h || !topk_idx || !topk_w || !expert_off || !pair_perm || !active || !n_active || !out) return COLI_E_INVALID;
  if (!mx_aligned(h, 16) || !mx_aligned(out, 16) || !mx_aligned(topk_idx, 4) || !mx_aligned(topk_w, 4) ||
      !mx_aligned(expert_off, 4) || !mx_aligned(pair_perm, 4) || !mx_aligned(active, 4) || !mx_aligned(n_active, 4))
    return COLI_E_ALIGN;
  const MxWs L = mx_ws_down(*cfg, T);
  if (!workspace || ws_bytes < L.total) return COLI_E_WORKSPACE;
  if (!mx_aligned(workspace, 256)) return COLI_E_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  MxArgs a = expert_args(*cfg, *w, T, expert_off, pair_perm, active, n_active);
  a.wc += (int64_t)cfg->ffn * cfg->hidden;  // gate and up rows: 2 F H / 2 bytes
  a.ws += (int64_t)cfg->ffn * cfg->hidden / 16;
  a.N = cfg->hidden;
  a.K = cfg->ffn;
  a.ac = ws + L.ac;
  a.as = ws + L.as;
  a.out = ws + L.y;
  const bool fused = mx_down_fused(a);
  if (fused && mx_down_from_x(a))
    a.x = h;
  else if ((st = mx_dev(launch_mx_quantize_rows(h, dtype, mx_rows(*cfg, T), cfg->ffn, ws + L.ac, ws + L.as, s))))
    return st;
  if (fused) return mx_dev(launch_mx_down(a, topk_idx, topk_w, out, dtype, s));
  if ((st = mx_dev(launch_experts(MX_DOWN, dtype, a, ws, L, s)))) return st;
  return mx_dev(launch_mx_combine(reinterpret_cast<float *>(ws + L.y), topk_idx, topk_w, T, cfg->top_k,
                                  cfg->n_experts, cfg->hidden, cfg->has_shared, out, dtype, s));
}

}  // extern "C"

// q8_w4_api.cpp -- host side of the 4-bit weight's calls declared in
// include/q8gemv.h: argument validation before any launch, and which kernel runs.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/q8gemv.h"
#include "q8_checks.h"
#include "q8_w4.h"

namespace {

using namespace q8;

constexpr int64_t kMaxKN = (int64_t)1 << 24;
constexpr int64_t kMax32 = 0xffffffffll;

int check_shape(int64_t K, int64_t N, int group) {
  int st;
  if ((st = check_range(K, 1, kMaxKN, "K"))) return st;
  if (K % Q8_BLOCK)
    return report_error(Q8_ERR_SHAPE, "K = %lld is not whole %d-row blocks: declared %lld, bound %lld",
                        (long long)K, Q8_BLOCK, (long long)K, (long long)round_up(K, Q8_BLOCK));
  if ((st = check_range(N, 1, kMaxKN, "N"))) return st;
  if (K * round_up(N, Q8_TILE_COLS) >= (int64_t)1 << 40)
    return report_error(Q8_ERR_SHAPE, "K*N_pad = %lld exceeds 2^40",
                        (long long)(K * round_up(N, Q8_TILE_COLS)));
  if (group != 32 && group != 64 && group != 128)
    return report_error(Q8_ERR_SHAPE, "group = %d: need 32, 64 or 128 rows", group);
  return Q8_OK;
}

size_t scale_bytes(int64_t K, int64_t N, int group) {
  return (size_t)(round_up(N, Q8_TILE_COLS) / Q8_TILE_COLS) * (size_t)w4_groups(K, group) * 128;
}

// The weight's description; with `out` its pointers too.
int check_weight(const q8_w4_weight *w, const char *name, W4 *out) {
  int st;
  if (!w) return report_error(Q8_ERR_NULL, "%s is NULL", name);
  if ((st = check_shape(w->K, w->N, w->group))) return st;
  if (w->scale_fmt != Q8_W4_SCALE_F16 && w->scale_fmt != Q8_W4_SCALE_BF16)
    return report_error(Q8_ERR_ACT_FMT, "%s scale_fmt = %d: need 0 (fp16) or 1 (bf16)", name,
                        w->scale_fmt);
  if (out) {
    if ((st = check_ptr(w->values, "weight values"))) return st;
    if ((st = check_ptr(w->scales, "weight scales"))) return st;
    out->values = static_cast<const char *>(w->values);
    out->scales = static_cast<const char *>(w->scales);
    out->zeros = w->has_zeros ? out->scales + scale_bytes(w->K, w->N, w->group) : nullptr;
  }
  return Q8_OK;
}

int check_act(int act_fmt) {
  if (act_fmt != Q8_ACT_BF16 && act_fmt != Q8_ACT_Q8_0)
    return report_error(Q8_ERR_ACT_FMT, "act_fmt = %d: a 4-bit weight takes 0 (bf16) or 1 (Q8_0)",
                        act_fmt);
  return Q8_OK;
}

int check_pair(const q8_w4_weight *g, const q8_w4_weight *u) {
  if (g->K != u->K || g->N != u->N || g->group != u->group || g->scale_fmt != u->scale_fmt ||
      !g->has_zeros != !u->has_zeros)
    return report_error(Q8_ERR_SHAPE, "the pair's weights differ in K, N, group, scale_fmt or has_zeros");
  return Q8_OK;
}

// ---- what runs ------------------------------------------------------------------

// The tile kernel's shape changes where the tiles are more than the CUs (us, K = 4096).
//   * Sixteen waves, all of a workgroup's loads in flight sooner, while every tile has a CU
//     of its own; then eight, two workgroups a CU (1 row, 224 tiles 7.0 against 7.7 with
//     eight, 256 6.6 against 8.1, 261 11.1 against 10.5, 383 11.9 against 11.2, 500 13.2
//     against 12.1; 16 rows, 224 tiles 9.2 against 9.6).  With Q8_0 rows above four and
//     groups of 128 they lack registers (11.6 against 9.6).
//   * Above 16 rows one tile a wave, then two that share its activation (32 rows, 256 tiles
//     12.2 against 17.9 with two, 258 21.7 against 18.5, 438 22.3 against 19.2; Q8_0, 258
//     29.2 against 24.7, 501 with K = 5120 35.6 against 29.7).  17 to 24 rows of Q8_0 scale
//     less and keep one tile (24 rows, 258 tiles 19.7 against 21.9, 500 21.8 against 22.7),
//     but for weights with zero points in groups of 64 and 128, whose results take more
//     steps (282 tiles 27.2 against 24.2, 500 28.3 against 25.0).
W4Plan tile_plan(const W4Args &a, bool pair, int act_fmt) {
  const bool q8 = act_fmt == Q8_ACT_Q8_0, more = a.T > 256;
  if (a.m <= 4) return {4, pair || !more ? 16 : 8, pair ? 2 : 1};
  if (a.m <= 8 && q8) return {8, 8, pair ? 2 : 1};
  if (a.m <= 16) return {16, pair || more || (q8 && a.group == 128) ? 8 : 16, pair ? 2 : 1};
  if (a.m <= 24 && q8) return {24, 8, pair || (more && a.w.zeros && a.group > 32) ? 2 : 1};
  if (a.m <= 32 || pair) return {32, 8, pair || more ? 2 : 1};
  return {64, 8, 1};
}

// K splits across workgroups: only where the column tiles leave half of the CUs idle, as in
// the 8-bit tile plans.  The join of more costs more than it spares (us, one split against
// two: 1 row, K = 4096, 172 tiles 6.8 against 9.5, 16 rows 8.5 against 12.1; 1 row, K =
// 14336, 141 tiles 16.0 against 20.1; pairs of 172 tiles, 1 row 11.9 against 16.0, 24 rows of
// Q8_0 25.5 against 36.0).
int tile_splits(int64_t K, int64_t N) {
  const int64_t T = round_up(N, Q8_TILE_COLS) / Q8_TILE_COLS;
  const int64_t quads = (K / Q8_BLOCK + 3) / 4;
  int64_t S = T >= 128 ? 1 : 256 / T;
  S = std::min<int64_t>(S, 8);
  S = std::min<int64_t>(S, std::max<int64_t>(quads / 2, 1));
  return (int)std::max<int64_t>(S, 1);
}

size_t ws_bytes_of(int64_t m, int64_t N, int splits, int nw) {
  if (splits <= 1) return 0;
  return kCounterBytes + (size_t)round_up((int64_t)nw * splits * m * round_up(N, Q8_TILE_COLS) * 4, 256);
}

W4Args args_of(const void *x, const q8_w4_weight *w, float *y, int64_t m, int act_fmt) {
  W4Args a{};
  a.x = x;
  a.y = y;
  a.m = (int)m;
  a.K = (int)w->K;
  a.NB = (int)(w->K / Q8_BLOCK);
  a.Npad = (int)round_up(w->N, Q8_TILE_COLS);
  a.T = a.Npad / Q8_TILE_COLS;
  a.group = w->group;
  a.scale_bf16 = w->scale_fmt == Q8_W4_SCALE_BF16;
  a.split_k = 1;
  if (act_fmt == Q8_ACT_Q8_0) {
    a.act_scale_off = (unsigned)q8_act_scales_offset(m, w->K);
    a.act_view_off = (unsigned)q8_act_view_offset(m, w->K);
  }
  a.ep.N = (int)w->N;
  a.ep.write_y = 1;
  a.ep.nw = 1;
  return a;
}

void output_q8(W4Args &a, void *y_q8) {
  if (!y_q8) return;
  a.ep.yq = static_cast<int8_t *>(y_q8);
  a.ep.yq_scale = reinterpret_cast<float *>(a.ep.yq + q8_act_scales_offset(a.m, a.Npad));
  a.ep.yq_view = a.ep.yq + q8_act_view_offset(a.m, a.Npad);
}

int check_sizes(const q8_w4_weight *w, int64_t m, int64_t most, int act_fmt) {
  int st;
  if ((st = check_range(m, 1, most, "m")) || (st = check_act(act_fmt))) return st;
  if (act_fmt == Q8_ACT_Q8_0 && m * w->K > kMax32 - 512 - m * (w->K / Q8_BLOCK) * 4)
    return report_error(Q8_ERR_SHAPE, "m*K = %lld too large for the quantized layout",
                        (long long)(m * w->K));
  return Q8_OK;
}

int check_out(bool write_y, const float *y, const void *y_q8) {
  int st;
  if (write_y && (st = check_ptr(y, "y"))) return st;
  if (!write_y && !y_q8)
    return report_error(Q8_ERR_NULL, "epilogue writes neither y nor y_q8");
  return check_opt(y_q8, "epilogue y_q8");
}

int run_tile(W4Args &a, int act_fmt, bool pair, int splits, int64_t m, hipStream_t stream,
             void *ws, size_t ws_bytes) {
  const size_t need = ws_bytes_of(m, a.ep.N, splits, pair ? 2 : 1);
  const int st = check_workspace(ws, ws_bytes, need);
  if (st) return st;
  a.split_k = splits;
  if (need) {
    a.counters = static_cast<unsigned *>(ws);
    a.partial = reinterpret_cast<float *>(static_cast<char *>(ws) + kCounterBytes);
  }
  const auto launch = act_fmt == Q8_ACT_BF16 ? launch_w4_tile_bf16 : launch_w4_tile_q8;
  return done(launch(tile_plan(a, pair, act_fmt), pair, a, stream), "4-bit product launch");
}

// Many rows: the GEMM, whose workgroups own 128 rows by 256 columns (the pair 128), or
// the tile kernel in chunks of 64 rows (the pair 32), one workgroup a tile and chunk.  The
// tile kernel takes one step of its time for each 256 workgroups, the GEMM one of its
// (four to five times longer) for each 256.  Measured on MI355X (us, tile kernel against
// GEMM, by workgroups of the former), K = 4096, groups of 128: bf16 224 19 against 65, 448
// 34 against 67, 896 65 against 68, 1024 65 against 69, 1120 81 against 69; the pair 448
// 36 against 73, 896 70 against 76, 1024 66 against 76, 1120 87 against 76.  With Q8_0 or
// groups of 32, whose GEMM scales more: 1120 bf16, groups of 32, 87 against 103; Q8_0 105
// against 109, groups of 32 118 against 127 (the pair 114 against 136); 1344 Q8_0 125
// against 109, the pair 137 against 136.
bool gemm_route(const W4Args &a, int act_fmt, bool pair) {
  const int chunk = pair ? 32 : 64;
  const int64_t workgroups = (int64_t)((a.m + chunk - 1) / chunk) * a.T;
  return a.m > 64 && workgroups > (act_fmt == Q8_ACT_Q8_0 || a.group == 32 ? 1280 : 1024);
}

int run_many(W4Args &a, int act_fmt, bool pair, hipStream_t stream) {
  if (!gemm_route(a, act_fmt, pair)) return run_tile(a, act_fmt, pair, 1, a.m, stream, nullptr, 0);
  return done(launch_w4_gemm(act_fmt, pair, a, stream), "4-bit product launch");
}

int check_pair_args(const void *x, const q8_w4_weight *Wg, const q8_w4_weight *Wu, const float *y,
                    int64_t m, int64_t most, int act_fmt, const q8_glu_epilogue *ep, W4 *g, W4 *u) {
  int st;
  if ((st = check_weight(Wg, "Wg", g)) || (st = check_weight(Wu, "Wu", u)) ||
      (st = check_pair(Wg, Wu)) || (st = check_sizes(Wg, m, most, act_fmt)) ||
      (st = check_ptr(x, "x")))
    return st;
  if ((st = check_out(!ep || ep->write_y, y, ep ? ep->y_q8 : nullptr))) return st;
  if (ep) {
    if ((st = check_opt(ep->bias_g, "epilogue bias_g"))) return st;
    if ((st = check_opt(ep->bias_u, "epilogue bias_u"))) return st;
  }
  return Q8_OK;
}

W4Args pair_args(const void *x, const q8_w4_weight *Wg, const W4 &g, const W4 &u, float *y, int64_t m,
                 int act_fmt, const q8_glu_epilogue *ep) {
  W4Args a = args_of(x, Wg, y, m, act_fmt);
  a.w = g;
  a.w_u = u;
  a.ep.nw = 2;
  if (ep) {
    a.ep.bias = ep->bias_g;
    a.ep.bias_u = ep->bias_u;
    a.ep.write_y = ep->write_y != 0;
    output_q8(a, ep->y_q8);
  }
  return a;
}

}  // namespace

extern "C" {

size_t q8_w4_values_bytes(int64_t K, int64_t N) {
  return check_shape(K, N, 32) ? 0 : (size_t)(K / 2) * (size_t)round_up(N, Q8_TILE_COLS);
}

size_t q8_w4_scales_bytes(int64_t K, int64_t N, int group, int has_zeros) {
  if (check_shape(K, N, group)) return 0;
  const size_t b = scale_bytes(K, N, group);
  return has_zeros ? b + b / 2 : b;
}

int q8_w4_repack(const uint8_t *u_kn, const uint16_t *s_kn, const uint8_t *z_kn,
                 const q8_w4_weight *W, hipStream_t stream) {
  int st;
  W4 w;
  if ((st = check_weight(W, "W", &w)) || (st = check_ptr(u_kn, "u_kn")) ||
      (st = check_ptr(s_kn, "s_kn")) || (W->has_zeros && (st = check_ptr(z_kn, "z_kn"))))
    return st;
  return done(launch_w4_repack(u_kn, s_kn, z_kn, W->K, W->N, W->group, const_cast<char *>(w.values),
                               const_cast<char *>(w.scales), const_cast<char *>(w.zeros), stream),
              "4-bit repack launch");
}

int q8_w4_unpack(const q8_w4_weight *W, uint8_t *u_kn, uint16_t *s_kn, uint8_t *z_kn,
                 hipStream_t stream) {
  int st;
  W4 w;
  if ((st = check_weight(W, "W", &w)) || (st = check_ptr(u_kn, "u_kn")) ||
      (st = check_ptr(s_kn, "s_kn")) || (W->has_zeros && (st = check_ptr(z_kn, "z_kn"))))
    return st;
  return done(launch_w4_unpack(w.values, w.scales, w.zeros, W->K, W->N, W->group, u_kn, s_kn, z_kn,
                               stream),
              "4-bit unpack launch");
}

size_t q8_w4_gemv_workspace_bytes(int64_t m, const q8_w4_weight *W, int act_fmt) {
  if (check_weight(W, "W", nullptr) || check_sizes(W, m, Q8_MAX_ROWS, act_fmt)) return 0;
  return ws_bytes_of(m, W->N, tile_splits(W->K, W->N), 1);
}

size_t q8_w4_glu_workspace_bytes(int64_t m, const q8_w4_weight *W, int act_fmt) {
  if (check_weight(W, "W", nullptr) || check_sizes(W, m, Q8_MAX_ROWS, act_fmt)) return 0;
  return ws_bytes_of(m, W->N, tile_splits(W->K, W->N), 2);
}

int q8_w4_gemv(const void *x, const q8_w4_weight *W, float *y, int64_t m, int act_fmt,
               const q8_epilogue *epilogue, hipStream_t stream, void *workspace, size_t ws_bytes) {
  int st;
  W4 w;
  if ((st = check_weight(W, "W", &w)) || (st = check_sizes(W, m, Q8_MAX_ROWS, act_fmt)) ||
      (st = check_ptr(x, "x")))
    return st;
  const q8_epilogue *ep = epilogue;
  if ((st = check_out(!ep || ep->write_y, y, ep ? ep->y_q8 : nullptr))) return st;
  W4Args a = args_of(x, W, y, m, act_fmt);
  a.w = w;
  if (ep) {
    if ((st = check_opt(ep->bias, "epilogue bias"))) return st;
    if ((st = check_opt(ep->residual, "epilogue residual"))) return st;
    a.ep.bias = ep->bias;
    a.ep.residual = ep->residual;
    a.ep.write_y = ep->write_y != 0;
    output_q8(a, ep->y_q8);
  }
  return run_tile(a, act_fmt, false, tile_splits(W->K, W->N), m, stream, workspace, ws_bytes);
}

int q8_w4_gemv_glu(const void *x, const q8_w4_weight *Wg, const q8_w4_weight *Wu, float *y, int64_t m,
                   int act_fmt, const q8_glu_epilogue *epilogue, hipStream_t stream, void *workspace,
                   size_t ws_bytes) {
  W4 g, u;
  const int st = check_pair_args(x, Wg, Wu, y, m, Q8_MAX_ROWS, act_fmt, epilogue, &g, &u);
  if (st) return st;
  W4Args a = pair_args(x, Wg, g, u, y, m, act_fmt, epilogue);
  return run_tile(a, act_fmt, true, tile_splits(Wg->K, Wg->N), m, stream, workspace, ws_bytes);
}

int q8_w4_gemm(const void *x, const q8_w4_weight *W, float *y, int64_t m, int act_fmt,
               hipStream_t stream) {
  int st;
  W4 w;
  if ((st = check_weight(W, "W", &w)) || (st = check_sizes(W, m, Q8_MAX_GEMM_ROWS, act_fmt)) ||
      (st = check_ptr(x, "x")) || (st = check_ptr(y, "y")))
    return st;
  W4Args a = args_of(x, W, y, m, act_fmt);
  a.w = w;
  return run_many(a, act_fmt, false, stream);
}

int q8_w4_gemm_glu(const void *x, const q8_w4_weight *Wg, const q8_w4_weight *Wu, float *y, int64_t m,
                   int act_fmt, const q8_glu_epilogue *epilogue, hipStream_t stream) {
  W4 g, u;
  const int st = check_pair_args(x, Wg, Wu, y, m, Q8_MAX_GEMM_ROWS, act_fmt, epilogue, &g, &u);
  if (st) return st;
  W4Args a = pair_args(x, Wg, g, u, y, m, act_fmt, epilogue);
  return run_many(a, act_fmt, true, stream);
}

}  // extern "C"

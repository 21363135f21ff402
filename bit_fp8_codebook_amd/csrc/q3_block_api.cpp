// C ABI of q3_block.h: host-side validation, then the launches on the caller's
// stream.  Nothing here allocates device memory or synchronises.
#include <hip/hip_runtime.h>

#include "../../include/q3_block.h"
#include "q3_check.h"
#include "q3_internal.h"

using namespace q3::check;

namespace {

constexpr int64_t kMaxK = int64_t(1) << 21;   // rows and columns: 256 widened rows stay below 2 GiB

// A packed matrix and bf16 token rows of `cols` columns in front of it.  A
// kernel addresses up to 256 rows through one 32-bit buffer resource.
q3_status check_product(const q3_matrix* w, const uint16_t* x, int64_t m, int64_t ldx, int64_t cols) {
  q3_status st = check_matrix(w);
  if (st != Q3_OK) return st;
  if (m < 1 || m >= kMaxM || w->k > kMaxK || w->n > kMaxK) return Q3_ERR_UNSUPPORTED_SHAPE;
  if (!x && cols > 0) return Q3_ERR_INVALID_ARG;
  if (ldx < cols) return Q3_ERR_INVALID_ARG;
  if (ldx % 8 || !aligned(x, 16)) return Q3_ERR_MISALIGNED;
  if (ldx > kMaxPlaneBytes / 512 - cols / 256) return Q3_ERR_UNSUPPORTED_SHAPE;
  return Q3_OK;
}

bool bad_shape(int64_t n, int64_t k, int64_t m) {
  return n < 1 || n > kMaxK || k < 32 || k % 32 || k > kMaxK || m < 1 || m >= kMaxM;
}

bool bad_act(int32_t act) { return act != Q3_ACT_SILU && act != Q3_ACT_GELU_TANH; }

constexpr int64_t kMaxNorm = 16384;

// What both directions of the residual norm share.
q3_status check_norm(const float* y, int64_t ldy, const float* post_weight, const float* gate, int64_t ld_gate,
                     const void* r, int64_t ldr, int32_t r_type, const float* pre_weight, float eps, int64_t m,
                     int64_t n) {
  if (r_type != Q3_F32 && r_type != Q3_BF16) return Q3_ERR_INVALID_ARG;
  if (m < 1 || m >= kMaxM || n < 1 || n > kMaxNorm) return Q3_ERR_UNSUPPORTED_SHAPE;
  if (!r || !(eps >= 0.f)) return Q3_ERR_INVALID_ARG;
  if (!y && (post_weight || gate)) return Q3_ERR_INVALID_ARG;
  if (ldr < n || (y && ldy < n) || (gate && ld_gate != 0 && ld_gate < n)) return Q3_ERR_INVALID_ARG;
  if (!aligned(r, r_type == Q3_BF16 ? 2 : 4) || !aligned(y, 4) || !aligned(post_weight, 4) || !aligned(gate, 4) ||
      !aligned(pre_weight, 4))
    return Q3_ERR_MISALIGNED;
  return Q3_OK;
}

// The forward pass's own outputs.
q3_status check_norm_out(const void* r, int64_t ldr, const void* r_out, int64_t ldr_out, int32_t r_type,
                         const uint16_t* x, int64_t ldx, int64_t n) {
  if ((r_out && ldr_out < n) || (x && ldx < n) || (r_out == r && ldr_out != ldr)) return Q3_ERR_INVALID_ARG;
  if (!aligned(r_out, r_type == Q3_BF16 ? 2 : 4) || !aligned(x, 2)) return Q3_ERR_MISALIGNED;
  return Q3_OK;
}

// Whether rows at p with this pitch all start on four elements of `size` bytes.
bool quads(const void* p, int64_t ld, int size) { return !p || (aligned(p, 4 * size) && ld % 4 == 0); }

q3_status run_norm(const q3::NormArgs& a, int32_t r_type, void* stream) {
  const int e = r_type == Q3_BF16 ? 2 : 4;
  const bool vec = a.n % 4 == 0 && quads(a.y, a.ldy, 4) && quads(a.post_w, 0, 4) && quads(a.gate, a.ld_gate, 4) &&
                   quads(a.r, a.ldr, e) && quads(a.r_out, a.ldr_out, e) && quads(a.pre_w, 0, 4) &&
                   quads(a.x, a.ldx, 2);
  return from_hip(q3::launch_residual_norm(a, r_type, vec, static_cast<hipStream_t>(stream)));
}

// q3_ffn's workspace: x [m][k] and h [m][I] in bf16, y [m][k] in fp32 and what
// the two products need, each from a 256-byte boundary on.
struct FfnSpace {
  int64_t h, y, products, bytes;
};
FfnSpace ffn_space(int64_t n_gu, int64_t k, int64_t m) {
  FfnSpace f;
  f.h = align256(m * k * 2);
  f.y = f.h + align256(m * (n_gu / 2) * 2);
  f.products = f.y + align256(m * k * 4);
  const int64_t up = q3::glu_workspace_bytes(n_gu, k, m), down = q3::gemm_workspace_bytes(k, n_gu / 2, m);
  f.bytes = f.products + (up > down ? up : down);
  return f;
}

}  // namespace

extern "C" {

Q3_API int64_t q3_gemm_workspace_bytes(int64_t n, int64_t k, int64_t m) {
  return bad_shape(n, k, m) ? 0 : q3::gemm_workspace_bytes(n, k, m);
}

Q3_API q3_status q3_gemm(const q3_matrix* w, const uint16_t* x, int64_t m, int64_t ldx, float* y, int64_t ldy,
                         void* workspace, int64_t workspace_bytes, void* stream) {
  q3_status st = check_matrix(w);
  if (st != Q3_OK) return st;
  if ((st = check_product(w, x, m, ldx, w->k)) != Q3_OK) return st;
  if ((!y && w->n > 0) || ldy < w->n) return Q3_ERR_INVALID_ARG;
  if (!aligned(y, 4)) return Q3_ERR_MISALIGNED;
  if ((st = check_workspace(workspace, workspace_bytes, q3_gemm_workspace_bytes(w->n, w->k, m))) != Q3_OK) return st;
  if ((st = check_device()) != Q3_OK) return st;
  return from_hip(q3::launch_gemm(view_of(w), x, m, ldx, y, ldy, workspace, static_cast<hipStream_t>(stream)));
}

Q3_API int64_t q3_gemm_backward_workspace_bytes(int64_t n, int64_t k, int64_t m) {
  return bad_shape(n, k, m) ? 0 : q3::gemm_backward_workspace_bytes(n, k, m);
}

Q3_API q3_status q3_gemm_backward(const q3_matrix* w, const uint16_t* dy, int64_t m, int64_t ld_dy, float* dx,
                                  int64_t ld_dx, void* workspace, int64_t workspace_bytes, void* stream) {
  q3_status st = check_matrix(w);
  if (st != Q3_OK) return st;
  if ((st = check_product(w, dy, m, ld_dy, w->n)) != Q3_OK) return st;
  if (!dx || ld_dx < w->k) return Q3_ERR_INVALID_ARG;
  if (!aligned(dx, 4)) return Q3_ERR_MISALIGNED;
  if ((st = check_workspace(workspace, workspace_bytes, q3_gemm_backward_workspace_bytes(w->n, w->k, m))) != Q3_OK)
    return st;
  if ((st = check_device()) != Q3_OK) return st;
  return from_hip(
      q3::launch_gemm_backward(view_of(w), dy, m, ld_dy, dx, ld_dx, workspace, static_cast<hipStream_t>(stream)));
}

Q3_API int64_t q3_glu_workspace_bytes(int64_t n_gu, int64_t k, int64_t m) {
  return bad_shape(n_gu, k, m) || n_gu % 64 ? 0 : q3::glu_workspace_bytes(n_gu, k, m);
}

Q3_API q3_status q3_glu(const q3_matrix* gate_up, const uint16_t* x, int64_t m, int64_t ldx, int32_t act,
                        uint16_t* h, int64_t ldh, float* pre, int64_t ld_pre, void* workspace,
                        int64_t workspace_bytes, void* stream) {
  q3_status st = check_matrix(gate_up);
  if (st != Q3_OK) return st;
  if ((st = check_product(gate_up, x, m, ldx, gate_up->k)) != Q3_OK) return st;
  if (bad_act(act)) return Q3_ERR_INVALID_ARG;
  if (gate_up->n % 64) return Q3_ERR_UNSUPPORTED_SHAPE;
  if ((!h && gate_up->n > 0) || ldh < gate_up->n / 2 || (pre && ld_pre < gate_up->n)) return Q3_ERR_INVALID_ARG;
  if (ldh % 8 || !aligned(h, 16) || (pre && (ld_pre % 4 || !aligned(pre, 16)))) return Q3_ERR_MISALIGNED;
  if ((st = check_workspace(workspace, workspace_bytes, q3_glu_workspace_bytes(gate_up->n, gate_up->k, m))) != Q3_OK)
    return st;
  if ((st = check_device()) != Q3_OK) return st;
  return from_hip(q3::launch_glu(view_of(gate_up), x, m, ldx, act, h, ldh, pre, ld_pre, workspace,
                                 static_cast<hipStream_t>(stream)));
}

Q3_API q3_status q3_glu_backward(const float* pre, int64_t ld_pre, const float* dh, int64_t ld_dh, int32_t act,
                                 int64_t m, int64_t inter, uint16_t* dpre, int64_t ld_dpre, void* stream) {
  if (bad_act(act)) return Q3_ERR_INVALID_ARG;
  if (m < 1 || m >= kMaxM || inter < 32 || inter % 32 || inter > kMaxK) return Q3_ERR_UNSUPPORTED_SHAPE;
  if (!pre || !dh || !dpre) return Q3_ERR_INVALID_ARG;
  if (ld_pre < 2 * inter || ld_dh < inter || ld_dpre < 2 * inter) return Q3_ERR_INVALID_ARG;
  if (ld_pre % 4 || ld_dh % 4 || ld_dpre % 8 || !aligned(pre, 16) || !aligned(dh, 16) || !aligned(dpre, 16))
    return Q3_ERR_MISALIGNED;
  // One thread per four outputs, and a launch takes less than 2^32 (in blocks of 256).
  if (m * (inter / 4) > int64_t(0xFFFFFF00)) return Q3_ERR_UNSUPPORTED_SHAPE;
  q3_status st = check_device();
  if (st != Q3_OK) return st;
  return from_hip(q3::launch_glu_backward(pre, ld_pre, dh, ld_dh, act, m, inter, dpre, ld_dpre,
                                          static_cast<hipStream_t>(stream)));
}

Q3_API q3_status q3_residual_norm(const float* y, int64_t ldy, const float* post_weight, const float* gate,
                                  int64_t ld_gate, float scale, const void* r, int64_t ldr, void* r_out,
                                  int64_t ldr_out, int32_t r_type, const float* pre_weight, uint16_t* x, int64_t ldx,
                                  float eps, int64_t m, int64_t n, void* stream) {
  q3_status st = check_norm(y, ldy, post_weight, gate, ld_gate, r, ldr, r_type, pre_weight, eps, m, n);
  if (st != Q3_OK) return st;
  if ((y && !r_out) || (pre_weight && !x) || (!r_out && !x)) return Q3_ERR_INVALID_ARG;
  if ((st = check_norm_out(r, ldr, r_out, ldr_out, r_type, x, ldx, n)) != Q3_OK) return st;
  if ((st = check_device()) != Q3_OK) return st;
  q3::NormArgs a{};
  a.y = y;
  a.ldy = ldy;
  a.post_w = post_weight;
  a.gate = gate;
  a.ld_gate = ld_gate;
  a.scale = scale;
  a.eps = eps;
  a.r = r;
  a.ldr = ldr;
  a.r_out = r_out;
  a.ldr_out = ldr_out;
  a.pre_w = pre_weight;
  a.x = x;
  a.ldx = ldx;
  a.m = m;
  a.n = static_cast<int>(n);
  return run_norm(a, r_type, stream);
}

Q3_API int64_t q3_residual_norm_backward_workspace_bytes(int64_t m, int64_t n) {
  if (m < 1 || m >= kMaxM || n < 1 || n > kMaxNorm) return 0;
  return 3 * align256(q3::norm_back_groups(m, static_cast<int>(n)) * n * 4);
}

Q3_API q3_status q3_residual_norm_backward(const float* y, int64_t ldy, const float* post_weight, const float* gate,
                                           int64_t ld_gate, float scale, const void* r_out, int64_t ldr_out,
                                           int32_t r_type, const float* pre_weight, float eps, int64_t m, int64_t n,
                                           const q3_residual_norm_grads* grads, void* workspace,
                                           int64_t workspace_bytes, void* stream) {
  q3_status st = check_norm(y, ldy, post_weight, gate, ld_gate, r_out, ldr_out, r_type, pre_weight, eps, m, n);
  if (st != Q3_OK) return st;
  if (!grads || !grads->dr) return Q3_ERR_INVALID_ARG;
  const q3_residual_norm_grads& g = *grads;
  if ((!y && g.dy) || (!gate && g.dgate) || (!post_weight && g.dpost_weight)) return Q3_ERR_INVALID_ARG;
  if (g.ld_dr < n || (g.dx && g.ld_dx < n) || (g.dr_out && g.ld_dr_out < n) || (g.dy && g.ld_dy < n) ||
      (g.dgate && ld_gate != 0 && g.ld_dgate < n) || (g.dr == g.dr_out && g.ld_dr != g.ld_dr_out))
    return Q3_ERR_INVALID_ARG;
  const int e = r_type == Q3_BF16 ? 2 : 4;
  if (!aligned(g.dr, e) || !aligned(g.dr_out, e) || !aligned(g.dx, 4) || !aligned(g.dy, 2) || !aligned(g.dgate, 4) ||
      !aligned(g.dpost_weight, 4) || !aligned(g.dpre_weight, 4))
    return Q3_ERR_MISALIGNED;
  if ((st = check_workspace(workspace, workspace_bytes, q3_residual_norm_backward_workspace_bytes(m, n))) != Q3_OK)
    return st;
  if ((st = check_device()) != Q3_OK) return st;
  q3::NormBackArgs a{};
  a.y = y;
  a.ldy = ldy;
  a.post_w = post_weight;
  a.gate = gate;
  a.ld_gate = ld_gate;
  a.scale = scale;
  a.eps = eps;
  a.r = r_out;
  a.ldr = ldr_out;
  a.pre_w = pre_weight;
  a.dx = g.dx;
  a.ld_dx = g.ld_dx;
  a.dr_out = g.dr_out;
  a.ld_dr_out = g.ld_dr_out;
  a.dr = g.dr;
  a.ld_dr = g.ld_dr;
  a.dy = g.dy;
  a.ld_dy = g.ld_dy;
  a.dgate = g.dgate;
  a.ld_dgate = g.ld_dgate;
  a.m = m;
  a.n = static_cast<int>(n);
  a.groups = q3::norm_back_groups(m, a.n);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int64_t part = align256(a.groups * n * 4);
  float* gate_row = g.dgate && ld_gate == 0 ? g.dgate : nullptr;
  if (g.dpre_weight) a.part_pre = reinterpret_cast<float*>(ws);
  if (g.dpost_weight) a.part_post = reinterpret_cast<float*>(ws + part);
  if (gate_row) a.part_gate = reinterpret_cast<float*>(ws + 2 * part);
  const bool vec = n % 4 == 0 && quads(y, ldy, 4) && quads(post_weight, 0, 4) && quads(gate, ld_gate, 4) &&
                   quads(r_out, ldr_out, e) && quads(pre_weight, 0, 4) && quads(g.dx, g.ld_dx, 4) &&
                   quads(g.dr_out, g.ld_dr_out, e) && quads(g.dr, g.ld_dr, e) && quads(g.dy, g.ld_dy, 2) &&
                   (!g.dgate || ld_gate == 0 || quads(g.dgate, g.ld_dgate, 4));
  return from_hip(q3::launch_residual_norm_back(a, r_type, vec, g.dpre_weight, g.dpost_weight, gate_row,
                                                static_cast<hipStream_t>(stream)));
}

Q3_API int64_t q3_ffn_workspace_bytes(int64_t n_gu, int64_t k, int64_t m) {
  if (bad_shape(n_gu, k, m) || n_gu % 64 || k > kMaxNorm) return 0;
  return ffn_space(n_gu, k, m).bytes;
}

Q3_API q3_status q3_ffn(const q3_matrix* gate_up, const q3_matrix* down, int32_t act, const q3_ffn_norms* norms,
                        const void* r, int64_t ldr, void* r_out, int64_t ldr_out, int32_t r_type, uint16_t* x_next,
                        int64_t ldx_next, int64_t m, void* workspace, int64_t workspace_bytes, void* stream) {
  q3_status st = check_matrix(gate_up);
  if (st != Q3_OK) return st;
  if ((st = check_matrix(down)) != Q3_OK) return st;
  if (!norms || bad_act(act)) return Q3_ERR_INVALID_ARG;
  const int64_t k = gate_up->k, inter = gate_up->n / 2;
  if (bad_shape(gate_up->n, k, m) || gate_up->n % 64 || k > kMaxNorm || down->n != k || down->k != inter)
    return Q3_ERR_UNSUPPORTED_SHAPE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const FfnSpace at = ffn_space(gate_up->n, k, m);
  if ((st = check_workspace(workspace, workspace_bytes, at.bytes)) != Q3_OK) return st;
  uint16_t* x = reinterpret_cast<uint16_t*>(ws);
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + at.h);
  float* y = reinterpret_cast<float*>(ws + at.y);
  void* rest = ws + at.products;
  if ((st = check_product(gate_up, x, m, k, k)) != Q3_OK) return st;
  if ((st = check_product(down, h, m, inter, inter)) != Q3_OK) return st;
  if ((st = check_norm(y, k, norms->post_weight, norms->gate, norms->ld_gate, r, ldr, r_type, norms->pre_weight,
                       norms->eps, m, k)) != Q3_OK)
    return st;
  if (!r_out || (norms->next_weight && !x_next)) return Q3_ERR_INVALID_ARG;
  if (!aligned(norms->next_weight, 4)) return Q3_ERR_MISALIGNED;
  if ((st = check_norm_out(r, ldr, r_out, ldr_out, r_type, x_next, ldx_next, k)) != Q3_OK) return st;
  if ((st = check_device()) != Q3_OK) return st;

  hipStream_t s = static_cast<hipStream_t>(stream);
  q3::NormArgs a{};
  a.r = r;
  a.ldr = ldr;
  a.pre_w = norms->pre_weight;
  a.eps = norms->eps;
  a.m = m;
  a.n = static_cast<int>(k);
  q3::NormArgs first = a;
  first.x = x;
  first.ldx = k;
  if ((st = run_norm(first, r_type, stream)) != Q3_OK) return st;
  hipError_t e = q3::launch_glu(view_of(gate_up), x, m, k, act, h, inter, nullptr, 0, rest, s);
  if (e == hipSuccess) e = q3::launch_gemm(view_of(down), h, m, inter, y, k, rest, s);
  if (e != hipSuccess) return from_hip(e);
  a.y = y;
  a.ldy = k;
  a.post_w = norms->post_weight;
  a.gate = norms->gate;
  a.ld_gate = norms->ld_gate;
  a.scale = norms->scale;
  a.r_out = r_out;
  a.ldr_out = ldr_out;
  a.pre_w = norms->next_weight;
  a.x = x_next;
  a.ldx = ldx_next;
  return run_norm(a, r_type, stream);
}

Q3_API int64_t q3_sample_workspace_bytes(int64_t m, int64_t n) {
  if (m < 1 || m > 65535 || n < 1 || n > (int64_t(1) << 19)) return 0;
  return q3::sample_workspace_bytes(m, n);
}

Q3_API q3_status q3_sample(const float* logits, int64_t m, int64_t n, int64_t ld, const float* temperature,
                           const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                           void* workspace, int64_t workspace_bytes, int32_t* tokens, float* logprobs, void* stream) {
  if (!logits || !u || !tokens) return Q3_ERR_INVALID_ARG;
  if (m < 1 || m > 65535 || n < 1 || n > (int64_t(1) << 19)) return Q3_ERR_UNSUPPORTED_SHAPE;
  if (ld < n) return Q3_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
      !aligned(min_p, 4) || !aligned(u, 4) || !aligned(tokens, 4) || !aligned(logprobs, 4))
    return Q3_ERR_MISALIGNED;
  q3_status st = check_workspace(workspace, workspace_bytes, q3_sample_workspace_bytes(m, n));
  if (st != Q3_OK) return st;
  if ((st = check_device()) != Q3_OK) return st;
  q3::SampleArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.m = static_cast<int>(m);
  a.n = static_cast<int>(n);
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.u = u;
  a.tokens = tokens;
  a.logprobs = logprobs;
  return from_hip(q3::launch_sample(a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

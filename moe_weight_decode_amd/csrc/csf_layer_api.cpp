// C ABI of the layer operators (norm, router, gated feed-forward half):
// argument checks and launches.  Declarations are in include/csf.h; the
// kernels are in csf_norm.hip, csf_route.hip and csf_gated.hip.
#include "csf.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "csf_layer.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t element_bytes(int32_t dtype) {
    if (dtype == CSF_BF16 || dtype == CSF_F16) return 2;
    return dtype == CSF_F32 ? 4 : 0;
}

// HIP reports the last error of any runtime call on the thread: one left by
// an earlier call must not be taken for a failure of this call's launches.
void clear_stale_error() { (void)hipGetLastError(); }

csf_status launched(hipError_t e) { return e == hipSuccess ? CSF_OK : CSF_E_HIP; }

csf_status norm_shape(int32_t dtype, int32_t tokens, int32_t cols) {
    if (element_bytes(dtype) == 0) return CSF_E_FORMAT;
    if (cols <= 0 || cols > int32_t(csf::kNormMaxCols)) return CSF_E_SHAPE;
    return tokens < 0 ? CSF_E_SIZE : CSF_OK;
}

csf_status norm_impl(int32_t dtype, const void *x, const void *residual, const float *weight, int32_t tokens,
                     int32_t cols, const int32_t *slots, const float *gates, int32_t choices, int64_t x_rows, float eps,
                     void *sum, void *out, uint8_t *scales, float *rstd, void *hip_stream) {
    csf_status st = norm_shape(dtype, tokens, cols);
    if (st != CSF_OK) return st;
    if (slots != nullptr && (choices <= 0 || x_rows < 0)) return CSF_E_SIZE;
    if (weight == nullptr) return CSF_E_NULL;
    if (tokens > 0 && (out == nullptr || (slots != nullptr && gates == nullptr) || (x == nullptr && !(slots && x_rows == 0))))
        return CSF_E_NULL;
    const uintptr_t size = uintptr_t(element_bytes(dtype));
    if (!aligned(x, slots ? 4 : size) || !aligned(residual, size) || !aligned(weight, 4) || !aligned(slots, 4) ||
        !aligned(gates, 4) || !aligned(sum, size) || (scales == nullptr && !aligned(out, size)) || !aligned(rstd, 4))
        return CSF_E_ALIGN;
    if (tokens == 0) return CSF_OK;
    csf::NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.slots = slots;
    a.gates = gates;
    a.sum = sum;
    a.out = out;
    a.scales = scales;
    a.rstd = rstd;
    a.x_rows = x_rows;
    a.eps = eps;
    a.T = uint32_t(tokens);
    a.D = uint32_t(cols);
    a.k = slots ? uint32_t(choices) : 0u;
    clear_stale_error();
    return launched(csf::launch_norm(dtype, a, static_cast<hipStream_t>(hip_stream)));
}

csf_status norm_backward_impl(int32_t dtype, const void *dy, const void *sum, const float *weight, const float *rstd,
                              const void *dsum, int32_t tokens, int32_t cols, void *dx, float *dweight, void *workspace,
                              int64_t workspace_bytes, void *hip_stream) {
    csf_status st = norm_shape(dtype, tokens, cols);
    if (st != CSF_OK) return st;
    if (weight == nullptr || dweight == nullptr || workspace == nullptr) return CSF_E_NULL;
    if (tokens > 0 && (dy == nullptr || sum == nullptr || rstd == nullptr || dx == nullptr)) return CSF_E_NULL;
    if (workspace_bytes < csf_rms_norm_backward_workspace(tokens, cols)) return CSF_E_SIZE;
    const uintptr_t size = uintptr_t(element_bytes(dtype));
    if (!aligned(dy, size) || !aligned(sum, size) || !aligned(weight, 4) || !aligned(rstd, 4) || !aligned(dsum, size) ||
        !aligned(dx, size) || !aligned(dweight, 4) || !aligned(workspace, 4))
        return CSF_E_ALIGN;
    csf::NormBackwardArgs a;
    std::memset(&a, 0, sizeof(a));
    a.dy = dy;
    a.sum = sum;
    a.weight = weight;
    a.rstd = rstd;
    a.dsum = dsum;
    a.dx = dx;
    a.dweight = dweight;
    a.partial = static_cast<float *>(workspace);
    a.T = uint32_t(tokens);
    a.D = uint32_t(cols);
    a.groups = csf::norm_backward_groups(a.T, a.D);
    clear_stale_error();
    return launched(csf::launch_norm_backward(dtype, a, static_cast<hipStream_t>(hip_stream)));
}

uint32_t route_groups(int32_t tokens) { return (uint32_t(tokens) + csf::kRouteTokens - 1u) / csf::kRouteTokens; }

csf_status route_shape(int32_t dtype, int32_t tokens, int32_t num_experts, int32_t topk) {
    if (element_bytes(dtype) == 0) return CSF_E_FORMAT;
    if (num_experts <= 0 || num_experts > CSF_MAX_EXPERTS || topk <= 0 || topk > num_experts ||
        topk > int32_t(csf::kRouteMaxTopk))
        return CSF_E_SHAPE;
    return tokens < 0 || int64_t(tokens) * topk >= (int64_t(1) << 31) ? CSF_E_SIZE : CSF_OK;
}

csf_status route_impl(int32_t dtype, const void *logits, int32_t tokens, int32_t num_experts, int32_t topk,
                      int32_t renorm, int32_t *experts, float *gates, int32_t *expert_start, int32_t *rows,
                      int32_t *slots, void *workspace, int64_t workspace_bytes, void *hip_stream) {
    csf_status st = route_shape(dtype, tokens, num_experts, topk);
    if (st != CSF_OK) return st;
    if (expert_start == nullptr) return CSF_E_NULL;
    if (tokens > 0 && (logits == nullptr || experts == nullptr || gates == nullptr || rows == nullptr || slots == nullptr))
        return CSF_E_NULL;
    const int64_t need = csf_route_workspace(tokens, num_experts);
    if (need > 0 && workspace == nullptr) return CSF_E_NULL;
    if (workspace_bytes < need) return CSF_E_SIZE;
    if (!aligned(logits, uintptr_t(element_bytes(dtype))) || !aligned(experts, 4) || !aligned(gates, 4) ||
        !aligned(expert_start, 4) || !aligned(rows, 4) || !aligned(slots, 4) || !aligned(workspace, 16))
        return CSF_E_ALIGN;
    csf::RouteArgs a;
    std::memset(&a, 0, sizeof(a));
    a.logits = logits;
    a.experts = experts;
    a.gates = gates;
    a.expert_start = expert_start;
    a.rows = rows;
    a.slots = slots;
    a.T = uint32_t(tokens);
    a.E = uint32_t(num_experts);
    a.k = uint32_t(topk);
    a.renorm = renorm != 0;
    a.groups = std::max(1u, route_groups(tokens));  // no tokens: one workgroup writes the offsets
    a.count = static_cast<uint8_t *>(workspace);
    a.base = reinterpret_cast<uint32_t *>(a.count + uint64_t(a.groups) * csf::route_stride(a.E));
    a.total = a.base + uint64_t(a.groups) * a.E;
    clear_stale_error();
    return launched(csf::launch_route(dtype, a, static_cast<hipStream_t>(hip_stream)));
}

csf_status combine_backward_impl(int32_t dtype, const void *dout, const float *y, const int32_t *slots,
                                 const float *gates, int32_t tokens, int32_t choices, int32_t cols, int64_t y_rows,
                                 void *dy, float *dgates, void *hip_stream) {
    if (element_bytes(dtype) == 0) return CSF_E_FORMAT;
    if (cols <= 0) return CSF_E_SHAPE;
    if (tokens < 0 || choices <= 0 || y_rows < 0) return CSF_E_SIZE;
    if (tokens > 0 && (dout == nullptr || slots == nullptr || gates == nullptr || dgates == nullptr)) return CSF_E_NULL;
    if (tokens > 0 && y_rows > 0 && (y == nullptr || dy == nullptr)) return CSF_E_NULL;
    const uintptr_t size = uintptr_t(element_bytes(dtype));
    if (!aligned(dout, size) || !aligned(y, 4) || !aligned(slots, 4) || !aligned(gates, 4) || !aligned(dy, size) ||
        !aligned(dgates, 4))
        return CSF_E_ALIGN;
    if (tokens == 0) return CSF_OK;
    csf::CombineBackwardArgs a;
    std::memset(&a, 0, sizeof(a));
    a.dout = dout;
    a.y = y;
    a.slots = slots;
    a.gates = gates;
    a.dy = dy;
    a.dgates = dgates;
    a.S = y_rows;
    a.T = uint32_t(tokens);
    a.D = uint32_t(cols);
    a.k = uint32_t(choices);
    clear_stale_error();
    return launched(csf::launch_combine_backward(dtype, a, static_cast<hipStream_t>(hip_stream)));
}

csf_status route_backward_impl(int32_t dtype, const float *dgates, const void *logits, const int32_t *experts,
                               const float *gates, int32_t tokens, int32_t num_experts, int32_t topk, int32_t renorm,
                               void *dlogits, void *hip_stream) {
    csf_status st = route_shape(dtype, tokens, num_experts, topk);
    if (st != CSF_OK) return st;
    if (tokens > 0 && (dgates == nullptr || logits == nullptr || experts == nullptr || gates == nullptr || dlogits == nullptr))
        return CSF_E_NULL;
    const uintptr_t size = uintptr_t(element_bytes(dtype));
    if (!aligned(dgates, 4) || !aligned(logits, size) || !aligned(experts, 4) || !aligned(gates, 4) || !aligned(dlogits, size))
        return CSF_E_ALIGN;
    if (tokens == 0) return CSF_OK;
    csf::RouteBackwardArgs a;
    std::memset(&a, 0, sizeof(a));
    a.dgates = dgates;
    a.logits = logits;
    a.experts = experts;
    a.gates = gates;
    a.dlogits = dlogits;
    a.T = uint32_t(tokens);
    a.E = uint32_t(num_experts);
    a.k = uint32_t(topk);
    a.renorm = renorm != 0;
    clear_stale_error();
    return launched(csf::launch_route_backward(dtype, a, static_cast<hipStream_t>(hip_stream)));
}

// The scale stack of a gated projection: 2 F rows of K weights.  need_streams:
// the scales come from the CSF streams (else only the shape is used).
csf_status gated_stack(const csf_stack *s, bool need_streams, int64_t &K) {
    if (s == nullptr) return CSF_E_NULL;
    if (s->format != CSF_NVFP4_E4M3 && s->format != CSF_MXFP4_UE8M0) return CSF_E_FORMAT;
    const bool mx = s->format == CSF_MXFP4_UE8M0;
    if (s->num_experts <= 0 || s->num_experts > CSF_MAX_EXPERTS || s->rows <= 0 || s->rows % 2 != 0 || s->cols <= 0 ||
        int64_t(s->rows) * s->cols >= (int64_t(1) << 24))
        return CSF_E_SHAPE;
    K = (mx ? 32 : 16) * int64_t(s->cols);
    if (K % 32 != 0 || K > int64_t(csf::kGatedMaxK)) return CSF_E_SHAPE;
    if (!need_streams) return CSF_OK;
    if (s->bases == nullptr || s->offsets == nullptr || s->exc_prefix == nullptr || s->tile_index == nullptr)
        return CSF_E_NULL;
    const int64_t G = mx ? 128 : 32;
    const int64_t stride = 16 * ((int64_t(s->rows) * s->cols + G - 1) / G);
    if (s->num_exceptions < 0 || s->num_exceptions >= (int64_t(1) << 31) || s->offsets_stride < stride ||
        s->offsets_stride % 16 != 0 || s->offsets_stride >= (int64_t(1) << 31))
        return CSF_E_SIZE;
    if (s->num_exceptions > 0 && s->exceptions == nullptr) return CSF_E_NULL;
    if (!aligned(s->offsets, 16) || !aligned(s->exceptions, 4) || !aligned(s->exc_prefix, 4) || !aligned(s->tile_index, 4)) return CSF_E_ALIGN;
    return CSF_OK;
}

void fill_stack(csf::StackArgs &a, const csf_stack &s) {
    const uint32_t C = uint32_t(s.cols);
    a.bases = s.bases;
    a.offsets = s.offsets;
    a.exc = s.exceptions;
    a.tile_index = s.tile_index;
    a.stride = s.offsets_stride;
    a.rcp_cols = 1.0 / double(C);
    a.n_exc = uint32_t(s.num_exceptions);
    a.R = uint32_t(s.rows);
    a.C = C;
    a.P = a.R * C;
    a.index_tiles = (a.P + csf::kIndexTile - 1u) / csf::kIndexTile;
    a.wbits = s.format == CSF_NVFP4_E4M3 ? 4u : 1u;
    a.row_mode = C % 16 == 0 ? csf::kRowSplat : (C >= 16 ? csf::kRowTwo : csf::kRowBytes);
}

csf_status gated_impl(const csf_stack *scales, const uint8_t *dense, const uint8_t *weights, const void *x,
                      const uint8_t *x_scales, int32_t num_tokens, const float *alpha, const int32_t *expert_start,
                      const int32_t *rows, int32_t num_slots, uint16_t *h, uint16_t *gate_up, void *workspace,
                      int64_t workspace_bytes, void *hip_stream) {
    int64_t K = 0;
    csf_status st = gated_stack(scales, dense == nullptr, K);
    if (st != CSF_OK) return st;
    const bool mx = scales->format == CSF_MXFP4_UE8M0;
    if (x_scales != nullptr && !mx) return CSF_E_FORMAT;
    if (num_tokens < 0 || num_slots < 0) return CSF_E_SIZE;
    if (weights == nullptr || alpha == nullptr || expert_start == nullptr) return CSF_E_NULL;
    if (num_slots > 0 && num_tokens > 0 && (x == nullptr || rows == nullptr || h == nullptr)) return CSF_E_NULL;
    const int64_t need = dense == nullptr ? csf_moe_gated_workspace(scales, num_slots) : 0;
    if (need > 0 && workspace == nullptr) return CSF_E_NULL;
    if (workspace_bytes < need) return CSF_E_SIZE;
    if (!aligned(weights, 16) || !aligned(x, 16) || !aligned(alpha, 4) || !aligned(expert_start, 4) || !aligned(rows, 4) ||
        !aligned(h, 2) || !aligned(gate_up, 2) || !aligned(workspace, 16))
        return CSF_E_ALIGN;
    if (num_slots == 0 || num_tokens == 0) return CSF_OK;
    csf::GatedArgs a;
    std::memset(&a, 0, sizeof(a));
    fill_stack(a.st, *scales);
    a.dense = dense;
    a.w = weights;
    a.x = x;
    a.x_scales = x_scales;
    a.alpha = alpha;
    a.expert_start = expert_start;
    a.rows = rows;
    a.h = h;
    a.gu = gate_up;
    a.E = uint32_t(scales->num_experts);
    a.F = uint32_t(scales->rows) / 2u;
    a.K = uint32_t(K);
    a.C = uint32_t(scales->cols);
    a.T = uint32_t(num_tokens);
    a.S = uint32_t(num_slots);
    a.mx = mx;
    // the workspace: the tiles' counters, then the scales
    if (workspace != nullptr && workspace_bytes >= int64_t(csf::kGatedQueueBytes)) a.queue = static_cast<uint32_t *>(workspace);
    const bool tiles = csf::gated_by_tiles(a.E, a.S) && csf::tiles_reach(a.T, a.K, x_scales != nullptr);
    if (tiles && dense == nullptr) {
        // the routed experts' scales decoded ahead: one launch, a few per cent of the products' time
        uint8_t *decoded = static_cast<uint8_t *>(workspace) + csf::kGatedQueueBytes;
        st = csf_decode(scales, decoded, expert_start, hip_stream);
        if (st != CSF_OK) return st;
        a.dense = decoded;
    }
    clear_stale_error();
    const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    return launched(tiles ? csf::launch_gated_tiles(a, stream) : csf::launch_gated(a, stream));
}

csf_status gated_backward_impl(const csf_stack *scales, const uint8_t *dense, const uint8_t *weights,
                               const uint16_t *dh, const uint16_t *gate_up, int32_t num_slots, const float *alpha,
                               const int32_t *expert_start, uint16_t *dx, uint16_t *dgate_up, void *hip_stream) {
    int64_t K = 0;
    csf_status st = gated_stack(scales, false, K);
    if (st != CSF_OK) return st;
    if (num_slots < 0) return CSF_E_SIZE;
    if (dense == nullptr || weights == nullptr || alpha == nullptr || expert_start == nullptr) return CSF_E_NULL;
    if (num_slots > 0 && (dh == nullptr || gate_up == nullptr || dx == nullptr || dgate_up == nullptr)) return CSF_E_NULL;
    if (!aligned(weights, 16) || !aligned(dh, 2) || !aligned(gate_up, 2) || !aligned(alpha, 4) || !aligned(expert_start, 4) ||
        !aligned(dx, 16) || !aligned(dgate_up, 4))
        return CSF_E_ALIGN;
    if (num_slots == 0) return CSF_OK;
    csf::GatedBackwardArgs a;
    std::memset(&a, 0, sizeof(a));
    a.dense = dense;
    a.w = weights;
    a.dh = dh;
    a.gu = gate_up;
    a.alpha = alpha;
    a.expert_start = expert_start;
    a.dx = dx;
    a.dgu = dgate_up;
    a.E = uint32_t(scales->num_experts);
    a.F = uint32_t(scales->rows) / 2u;
    a.K = uint32_t(K);
    a.C = uint32_t(scales->cols);
    a.S = uint32_t(num_slots);
    a.mx = scales->format == CSF_MXFP4_UE8M0;
    clear_stale_error();
    return launched(csf::launch_gated_backward(a, static_cast<hipStream_t>(hip_stream)));
}

}  // namespace

extern "C" {

csf_status csf_rms_norm(int32_t dtype, const void *x, const void *residual, const float *weight, int32_t tokens,
                        int32_t cols, const int32_t *slots, const float *gates, int32_t choices, int64_t x_rows,
                        float eps, void *sum, void *out, uint8_t *scales, float *rstd, void *hip_stream) {
    try {
        return norm_impl(dtype, x, residual, weight, tokens, cols, slots, gates, choices, x_rows, eps, sum, out, scales,
                         rstd, hip_stream);
    } catch (...) {
        return CSF_E_HIP;
    }
}

int64_t csf_rms_norm_backward_workspace(int32_t tokens, int32_t cols) {
    if (tokens < 0 || cols <= 0) return 0;
    return int64_t(4) * cols * csf::norm_backward_groups(uint32_t(tokens), uint32_t(cols));
}

csf_status csf_rms_norm_backward(int32_t dtype, const void *dy, const void *sum, const float *weight, const float *rstd,
                                 const void *dsum, int32_t tokens, int32_t cols, void *dx, float *dweight,
                                 void *workspace, int64_t workspace_bytes, void *hip_stream) {
    try {
        return norm_backward_impl(dtype, dy, sum, weight, rstd, dsum, tokens, cols, dx, dweight, workspace,
                                  workspace_bytes, hip_stream);
    } catch (...) {
        return CSF_E_HIP;
    }
}

int64_t csf_route_workspace(int32_t tokens, int32_t num_experts) {
    if (tokens < 0 || num_experts <= 0 || route_groups(tokens) <= 1) return 0;
    const int64_t E = num_experts, groups = route_groups(tokens);
    return 4 * E * (groups + 1) + groups * int64_t(csf::route_stride(uint32_t(num_experts)));
}

csf_status csf_route(int32_t dtype, const void *logits, int32_t tokens, int32_t num_experts, int32_t topk,
                     int32_t renorm, int32_t *experts, float *gates, int32_t *expert_start, int32_t *rows,
                     int32_t *slots, void *workspace, int64_t workspace_bytes, void *hip_stream) {
    try {
        return route_impl(dtype, logits, tokens, num_experts, topk, renorm, experts, gates, expert_start, rows, slots,
                          workspace, workspace_bytes, hip_stream);
    } catch (...) {
        return CSF_E_HIP;
    }
}

csf_status csf_combine_backward(int32_t dtype, const void *dout, const float *y, const int32_t *slots,
                                const float *gates, int32_t tokens, int32_t choices, int32_t cols, int64_t y_rows,
                                void *dy, float *dgates, void *hip_stream) {
    try {
        return combine_backward_impl(dtype, dout, y, slots, gates, tokens, choices, cols, y_rows, dy, dgates, hip_stream);
    } catch (...) {
        return CSF_E_HIP;
    }
}

csf_status csf_route_backward(int32_t dtype, const float *dgates, const void *logits, const int32_t *experts,
                              const float *gates, int32_t tokens, int32_t num_experts, int32_t topk, int32_t renorm,
                              void *dlogits, void *hip_stream) {
    try {
        return route_backward_impl(dtype, dgates, logits, experts, gates, tokens, num_experts, topk, renorm, dlogits,
                                   hip_stream);
    } catch (...) {
        return CSF_E_HIP;
    }
}

int64_t csf_moe_gated_workspace(const csf_stack *scales, int32_t num_slots) {
    int64_t K = 0;
    if (gated_stack(scales, false, K) != CSF_OK || num_slots < 0) return 0;
    return csf::gated_by_tiles(uint32_t(scales->num_experts), uint32_t(num_slots))
               ? csf::kGatedQueueBytes + int64_t(scales->num_experts) * scales->rows * scales->cols
               : 0;
}

csf_status csf_moe_gated(const csf_stack *scales, const uint8_t *dense_scales, const uint8_t *weights, const void *x,
                         const uint8_t *x_scales, int32_t num_tokens, const float *alpha, const int32_t *expert_start,
                         const int32_t *rows, int32_t num_slots, uint16_t *h, uint16_t *gate_up, void *workspace,
                         int64_t workspace_bytes, void *hip_stream) {
    try {
        return gated_impl(scales, dense_scales, weights, x, x_scales, num_tokens, alpha, expert_start, rows, num_slots,
                          h, gate_up, workspace, workspace_bytes, hip_stream);
    } catch (...) {
        return CSF_E_HIP;
    }
}

csf_status csf_moe_gated_backward(const csf_stack *scales, const uint8_t *dense_scales, const uint8_t *weights,
                                  const uint16_t *dh, const uint16_t *gate_up, int32_t num_slots, const float *alpha,
                                  const int32_t *expert_start, uint16_t *dx, uint16_t *dgate_up, void *hip_stream) {
    try {
        return gated_backward_impl(scales, dense_scales, weights, dh, gate_up, num_slots, alpha, expert_start, dx,
                                   dgate_up, hip_stream);
    } catch (...) {
        return CSF_E_HIP;
    }
}

}  // extern "C"

// Internal interface between the C ABI of the layer operators
// (csf_layer_api.cpp) and their gfx950 kernels (csf_norm.hip, csf_route.hip,
// csf_gated.hip).  Not installed; the public ABI is include/csf.h.
#pragma once

#include "csf_launch.h"

namespace csf {

constexpr uint32_t kCus = 256;             // compute units of an MI355X: grids are sized for them
constexpr uint32_t kNormMaxCols = 32768;  // columns of a norm (a row is held in registers)
constexpr uint32_t kGatedMaxK = 8192;     // columns of a gated projection's weights
constexpr uint32_t kRouteMaxTopk = 64;    // choices of a token (one lane each)
constexpr uint32_t kRouteTokens = 64;     // tokens per routing workgroup (one bit each of a 64-bit mask)

enum Dtype : int32_t { kBF16 = 0, kF16 = 1, kF32 = 2 };

struct NormArgs {
    const void *x;           // [T][D], or float32 [x_rows][D] with slots
    const void *residual;    // [T][D] or nullptr
    const float *weight;     // [D]
    const int32_t *slots;    // [T][k] or nullptr
    const float *gates;      // [T][k]
    void *sum;               // [T][D] or nullptr
    void *out;               // [T][D]: the type's, or E4M3 codes with scales
    uint8_t *scales;         // E8M0 [T][ceil(D / 32)] or nullptr
    float *rstd;             // [T] or nullptr
    int64_t x_rows;
    float eps;
    uint32_t T, D, k;
    uint32_t first;          // first workgroup of the launch
};

struct NormBackwardArgs {
    const void *dy, *sum;    // [T][D]
    const float *weight;     // [D]
    const float *rstd;       // [T]
    const void *dsum;        // [T][D] or nullptr
    void *dx;                // [T][D]
    float *dweight;          // [D]
    float *partial;          // [groups][D]: each workgroup's share of dweight
    uint32_t T, D, groups;
};

// Workgroups of a norm's backward pass: one row of partial sums each.
uint32_t norm_backward_groups(uint32_t T, uint32_t D);
hipError_t launch_norm(int32_t dtype, const NormArgs &a, hipStream_t stream);
hipError_t launch_norm_backward(int32_t dtype, const NormBackwardArgs &a, hipStream_t stream);

struct RouteArgs {
    const void *logits;      // [T][E]
    int32_t *experts;        // [T][k]
    float *gates;            // [T][k]
    int32_t *expert_start;   // [E + 1]
    int32_t *rows;           // [T * k]
    int32_t *slots;          // [T][k]
    uint8_t *count;          // workspace [groups][route_stride(E)]: entries of a workgroup per expert (at most 64)
    uint32_t *base;          // workspace [groups][E]: entries of earlier workgroups per expert
    uint32_t *total;         // workspace [E]
    uint32_t T, E, k, renorm, groups;
    uint32_t first;          // first workgroup of the launch
};

// Bytes between two workgroups' counts: whole 16-byte loads.
__host__ __device__ inline uint32_t route_stride(uint32_t E) { return (E + 15u) & ~15u; }

struct CombineBackwardArgs {
    const void *dout;        // [T][D]
    const float *y;          // [S][D]
    const int32_t *slots;    // [T][k]
    const float *gates;      // [T][k]
    void *dy;                // [S][D]
    float *dgates;           // [T][k]
    int64_t S;
    uint32_t T, D, k;
    uint32_t first;          // first workgroup of the launch
};

struct RouteBackwardArgs {
    const float *dgates;     // [T][k]
    const void *logits;      // [T][E]
    const int32_t *experts;  // [T][k]
    const float *gates;      // [T][k]
    void *dlogits;           // [T][E]
    uint32_t T, E, k, renorm;
    uint32_t first;          // first workgroup of the launch
};

hipError_t launch_route(int32_t dtype, const RouteArgs &a, hipStream_t stream);
hipError_t launch_combine_backward(int32_t dtype, const CombineBackwardArgs &a, hipStream_t stream);
hipError_t launch_route_backward(int32_t dtype, const RouteBackwardArgs &a, hipStream_t stream);

struct GatedArgs {
    StackArgs st;                  // scale stack of the 2 F rows (gate rows first)
    const uint8_t *dense;          // dense scales [E][2F][C], or nullptr: expanded in LDS
    const uint8_t *w;              // E2M1 codes [E][2F][K/2]
    const void *x;                 // bfloat16 [T][K], or E4M3 codes [T][K] with x_scales
    const uint8_t *x_scales;       // E8M0 [T][K / 32] or nullptr
    const float *alpha;            // [E]
    const int32_t *expert_start;   // [E + 1]
    const int32_t *rows;           // [S]
    uint16_t *h;                   // bfloat16 [S][F]
    uint16_t *gu;                  // bfloat16 [S][2F] or nullptr
    uint32_t *queue;               // workspace for the tiles' counters (kGatedQueueBytes), or nullptr
    uint32_t E, F, K, C, T, S;
    uint32_t mx;                   // MXFP4 (else NVFP4)
};

struct GatedBackwardArgs {
    const uint8_t *dense;          // dense scales [E][2F][C]
    const uint8_t *w;              // E2M1 codes [E][2F][K/2]
    const uint16_t *dh;            // bfloat16 [S][F]
    const uint16_t *gu;            // bfloat16 [S][2F]
    const float *alpha;            // [E]
    const int32_t *expert_start;   // [E + 1]
    uint16_t *dx;                  // bfloat16 [S][K]
    uint16_t *dgu;                 // bfloat16 [S][2F]
    uint32_t E, F, K, C, S;
    uint32_t mx;
};

constexpr uint32_t kGatedQueueBytes = 64;  // one counter per XCD

// A tile's share of the blocks of 16 slots of an expert with m of them: its
// first block and how many.
struct TileBlocks {
    uint32_t first, count;
};

// Tile j of the `tiles` that an expert's slots are spread over: all have q
// blocks, the first r of them one more.  No product passes the blocks' number,
// as blocks * j would (32 bits hold it up to three million slots only).
__host__ __device__ inline TileBlocks tile_blocks(uint32_t m, uint32_t j, uint32_t tiles) {
    const uint32_t blocks = (m + 15u) / 16u, q = blocks / tiles, r = blocks - q * tiles;
    return {q * j + (j < r ? j : r), q + (j < r ? 1u : 0u)};
}

// Whether a call has enough slots per expert for the tile kernel (which reads
// dense scales), and whether its activations lie within that one's reach.
bool gated_by_tiles(uint32_t E, uint32_t S);
bool tiles_reach(uint32_t T, uint32_t K, bool x8);
hipError_t launch_gated_tiles(const GatedArgs &a, hipStream_t stream);
hipError_t launch_gated(const GatedArgs &a, hipStream_t stream);
hipError_t launch_gated_backward(const GatedBackwardArgs &a, hipStream_t stream);

}  // namespace csf

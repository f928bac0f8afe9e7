// RMS norm with the residual's addition on gfx950, and its backward pass.
//
//     r    = x + residual                      (or sum_j gates[t][j] x[slots[t][j]] + residual)
//     rstd = (mean_d r^2 + eps)^(-1/2)
//     y    = r * rstd * weight
//
// A row is held in registers between the sum of squares and the scaling, so
// every input is read and every output written once: bound by memory.  Thread
// i of a row's THREADS holds columns 8 i .. 8 i + 7 of every chunk of
// 8 THREADS columns; all arithmetic is in float32, and each output is rounded
// once.  The routed combination adds its terms in the choices' order, then
// the residual.
//
// The 8-bit output is MXFP8: for every 32 columns the least power of two s
// with max |y| / s <= 448 (E4M3's largest value) as an E8M0 byte, and
// y / s rounded to E4M3, ties to even.  448 = 1.75 * 2^8, so the byte follows
// from the bits of max |y|: its exponent less 8, and one more where its
// fraction is above 1.75.
//
// A row is taken by one wave up to 1024 columns and by a workgroup above, since
// a wave's 64 lanes would need more registers than hide the loads' latency.
// Measured: 16384 x 5120 bfloat16 123 us, 5.4 TB/s (a large copy's rate); 512 x
// 5120 with 8 experts' outputs combined and 8-bit output 17.0 to 17.5 us, 5.6 TB/s; one
// row of 2048 4.1 us, a launch and two round trips.
#include "csf_layer_device.h"

namespace csf {
namespace {

// Sum over the row's THREADS threads (a wave, or the whole workgroup).
template <uint32_t THREADS>
__device__ __forceinline__ float row_sum(float v, float *lds) {
    v = wave_sum(v);
    if constexpr (THREADS == kWave) {
        return v;
    } else {
        if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
        __syncthreads();
        float s = lds[0];
#pragma unroll
        for (uint32_t i = 1; i < THREADS / kWave; ++i) s += lds[i];
        return s;
    }
}

__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0xB1, 0xF, 0xF, true)));
    return fmaxf(v, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x4E, 0xF, 0xF, true)));
}

// E8M0 byte of a block whose largest magnitude is m >= 0 (0 for m = 0, 254 at most).
__device__ __forceinline__ uint32_t mx8_byte(float m) {
    const uint32_t b = __float_as_uint(m);
    const int32_t e = (int32_t)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)min(max(e, 0), 254);
}

template <typename T, uint32_t CHUNKS, uint32_t THREADS, bool COMBINE, bool MX>
__global__ __launch_bounds__(THREADS < 256 ? 256 : THREADS) void csf_norm_kernel(NormArgs a) {
    __shared__ float lds[THREADS / kWave];
    uint32_t row = a.first + blockIdx.x, tid = threadIdx.x;
    if constexpr (THREADS == kWave) {
        row = __builtin_amdgcn_readfirstlane(row * 4u + threadIdx.x / kWave);
        tid = threadIdx.x % kWave;
        if (row >= a.T) return;  // no barriers on this path
    }
    const uint32_t D = a.D;
    const uint64_t at = (uint64_t)row * D;
    uint32_t d[CHUNKS], n[CHUNKS];
#pragma unroll
    for (uint32_t c = 0; c < CHUNKS; ++c) {
        d[c] = (c * THREADS + tid) * 8u;
        n[c] = d[c] < D ? D - d[c] : 0u;
    }
    float r[CHUNKS][8], res[CHUNKS][8];
    if (a.residual != nullptr) {
#pragma unroll
        for (uint32_t c = 0; c < CHUNKS; ++c) load8(static_cast<const T *>(a.residual) + at + d[c], n[c], res[c]);
    }
    if constexpr (COMBINE) {
#pragma unroll
        for (uint32_t c = 0; c < CHUNKS; ++c)
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) r[c][i] = 0.f;
        for (uint32_t j = 0; j < a.k; ++j) {
            const int32_t slot = a.slots[(uint64_t)row * a.k + j];
            if (slot < 0 || slot >= a.x_rows) continue;  // no expert there
            const float g = a.gates[(uint64_t)row * a.k + j];
            const float *x = static_cast<const float *>(a.x) + (int64_t)slot * D;
#pragma unroll
            for (uint32_t c = 0; c < CHUNKS; ++c) {
                float v[8];
                load8(x + d[c], n[c], v);
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) r[c][i] = fmaf(g, v[i], r[c][i]);
            }
        }
    } else {
#pragma unroll
        for (uint32_t c = 0; c < CHUNKS; ++c) load8(static_cast<const T *>(a.x) + at + d[c], n[c], r[c]);
    }
    float w[CHUNKS][8];
#pragma unroll
    for (uint32_t c = 0; c < CHUNKS; ++c) load8(a.weight + d[c], n[c], w[c]);
    float square = 0.f;
#pragma unroll
    for (uint32_t c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            if (a.residual != nullptr) r[c][i] += res[c][i];
            square = fmaf(r[c][i], r[c][i], square);
        }
    if (a.sum != nullptr) {
#pragma unroll
        for (uint32_t c = 0; c < CHUNKS; ++c) store8(static_cast<T *>(a.sum) + at + d[c], n[c], r[c]);
    }
    const float rstd = 1.0f / sqrtf(row_sum<THREADS>(square, lds) / (float)D + a.eps);
    if (tid == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
    const uint32_t blocks = (D + 31u) / 32u;
#pragma unroll
    for (uint32_t c = 0; c < CHUNKS; ++c) {
        float y[8];
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) y[i] = r[c][i] * rstd * w[c][i];
        if constexpr (MX) {
            float most = 0.f;
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) most = fmaxf(most, fabsf(y[i]));
            const uint32_t byte = mx8_byte(quad_max(most));  // the quad's 32 columns
            const int32_t up = 127 - (int32_t)byte;
            uint32_t code[2];
#pragma unroll
            for (uint32_t i = 0; i < 2; ++i) {
                int p = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(y[4 * i], up), ldexpf(y[4 * i + 1], up), 0, false);
                p = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(y[4 * i + 2], up), ldexpf(y[4 * i + 3], up), p, true);
                code[i] = (uint32_t)p;
            }
            uint8_t *out = static_cast<uint8_t *>(a.out) + at + d[c];
            if (n[c] >= 8u) {
                *reinterpret_cast<u32x2_byte *>(out) = (u32x2_byte){code[0], code[1]};
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i)
                    if (i < n[c]) out[i] = (uint8_t)(code[i / 4] >> (8u * (i % 4)));
            }
            if (tid % 4 == 0 && n[c] > 0) a.scales[(uint64_t)row * blocks + d[c] / 32u] = (uint8_t)byte;
        } else {
            store8(static_cast<T *>(a.out) + at + d[c], n[c], y);
        }
    }
}

// Backward pass: with xh = sum * rstd and c = dy * weight,
//     dx      = rstd * (c - xh * mean_d(c xh)) + dsum
//     dweight = sum_t dy * xh
// Workgroup g takes rows g, g + groups, ... and keeps its share of dweight in
// registers (a thread's columns are the same for every row); the shares are
// added in the groups' order by a second kernel, so the result does not
// depend on timing.  Bound by memory and, in short calls, by the second launch:
// 8191 x 2048 bfloat16 30.2 to 31.1 us, 4.4 TB/s.  Slower for what it moves are
// up to 1024 rows above 1024 columns, each a group with a row of partial sums of
// its own (1024 x 5120 22.8 us, 1.8 TB/s), and more than 8192 columns: 1024
// threads leave 128 registers each, and 275 to 309 are spilled (4096 x 16384
// 705 us, 0.8 TB/s).
template <typename T, uint32_t CHUNKS, uint32_t THREADS>
__global__ __launch_bounds__(THREADS) void csf_norm_backward_kernel(NormBackwardArgs a) {
    __shared__ float lds[2][THREADS / kWave];
    const uint32_t tid = threadIdx.x, D = a.D;
    uint32_t d[CHUNKS], n[CHUNKS];
    float w[CHUNKS][8], dw[CHUNKS][8];
#pragma unroll
    for (uint32_t c = 0; c < CHUNKS; ++c) {
        d[c] = (c * THREADS + tid) * 8u;
        n[c] = d[c] < D ? D - d[c] : 0u;
        load8(a.weight + d[c], n[c], w[c]);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) dw[c][i] = 0.f;
    }
    uint32_t turn = 0;  // two buffers: a row's partial sums are read while the next row's are written
    for (uint32_t row = blockIdx.x; row < a.T; row += a.groups, turn ^= 1u) {
        const uint64_t at = (uint64_t)row * D;
        const float rstd = a.rstd[row];
        float dy[CHUNKS][8], xh[CHUNKS][8], ds[CHUNKS][8];
#pragma unroll
        for (uint32_t c = 0; c < CHUNKS; ++c) {
            load8(static_cast<const T *>(a.dy) + at + d[c], n[c], dy[c]);
            load8(static_cast<const T *>(a.sum) + at + d[c], n[c], xh[c]);
            if (a.dsum != nullptr) {
                load8(static_cast<const T *>(a.dsum) + at + d[c], n[c], ds[c]);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) ds[c][i] = 0.f;
            }
        }
        float dot = 0.f;
#pragma unroll
        for (uint32_t c = 0; c < CHUNKS; ++c)
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) {
                xh[c][i] *= rstd;
                dw[c][i] = fmaf(dy[c][i], xh[c][i], dw[c][i]);
                dy[c][i] *= w[c][i];
                dot = fmaf(dy[c][i], xh[c][i], dot);
            }
        const float mean = row_sum<THREADS>(dot, lds[turn]) / (float)D;
#pragma unroll
        for (uint32_t c = 0; c < CHUNKS; ++c) {
            float dx[8];
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) dx[i] = fmaf(rstd, fmaf(-xh[c][i], mean, dy[c][i]), ds[c][i]);
            store8(static_cast<T *>(a.dx) + at + d[c], n[c], dx);
        }
    }
#pragma unroll
    for (uint32_t c = 0; c < CHUNKS; ++c) store8(a.partial + (uint64_t)blockIdx.x * D + d[c], n[c], dw[c]);
}

// dweight[d] = sum over groups of partial[g][d]: 32 columns per workgroup, its
// 32 half waves take every 32nd group (16 loads in flight each), then the
// shares are added in their order.
constexpr uint32_t kDweightCols = 32;

__global__ __launch_bounds__(1024) void csf_norm_dweight_kernel(NormBackwardArgs a) {
    __shared__ float lds[32][kDweightCols + 1u];
    const uint32_t col = threadIdx.x % kDweightCols, part = threadIdx.x / kDweightCols, d = blockIdx.x * kDweightCols + col;
    float s = 0.f;
    if (d < a.D) {
#pragma unroll 16
        for (uint32_t g = part; g < a.groups; g += 32u) s += a.partial[(uint64_t)g * a.D + d];
    }
    lds[part][col] = s;
    __syncthreads();
    if (part == 0 && d < a.D) {
#pragma unroll
        for (uint32_t i = 1; i < 32; ++i) s += lds[i][col];
        a.dweight[d] = s;
    }
}

template <typename T, uint32_t CHUNKS, uint32_t THREADS>
void start_norm(const NormArgs &all, hipStream_t stream) {
    const dim3 block(THREADS < 256 ? 256 : THREADS);
    launch_groups(all, THREADS == kWave ? (all.T + 3u) / 4u : all.T, [&](const NormArgs &a, dim3 grid) {
        if (a.slots != nullptr) {
            if (a.scales != nullptr) hipLaunchKernelGGL((csf_norm_kernel<T, CHUNKS, THREADS, true, true>), grid, block, 0, stream, a);
            else hipLaunchKernelGGL((csf_norm_kernel<T, CHUNKS, THREADS, true, false>), grid, block, 0, stream, a);
        } else {
            if (a.scales != nullptr) hipLaunchKernelGGL((csf_norm_kernel<T, CHUNKS, THREADS, false, true>), grid, block, 0, stream, a);
            else hipLaunchKernelGGL((csf_norm_kernel<T, CHUNKS, THREADS, false, false>), grid, block, 0, stream, a);
        }
    });
}

// Threads and chunks that cover the columns: a wave per row up to 1024
// columns, a workgroup of 4 waves up to 8192, of 16 above.
template <typename T>
void pick_norm(const NormArgs &a, hipStream_t stream) {
    if (a.D <= 512) start_norm<T, 1, 64>(a, stream);
    else if (a.D <= 1024) start_norm<T, 2, 64>(a, stream);
    else if (a.D <= 2048) start_norm<T, 1, 256>(a, stream);
    else if (a.D <= 4096) start_norm<T, 2, 256>(a, stream);
    else if (a.D <= 6144) start_norm<T, 3, 256>(a, stream);
    else if (a.D <= 8192) start_norm<T, 4, 256>(a, stream);
    else start_norm<T, 4, 1024>(a, stream);
}

template <typename T, uint32_t CHUNKS, uint32_t THREADS>
void start_backward(const NormBackwardArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL((csf_norm_backward_kernel<T, CHUNKS, THREADS>), dim3(a.groups), dim3(THREADS), 0, stream, a);
}

template <typename T>
void pick_backward(const NormBackwardArgs &a, hipStream_t stream) {
    if (a.D <= 512) start_backward<T, 1, 64>(a, stream);
    else if (a.D <= 1024) start_backward<T, 2, 64>(a, stream);
    else if (a.D <= 2048) start_backward<T, 1, 256>(a, stream);
    else if (a.D <= 4096) start_backward<T, 2, 256>(a, stream);
    else if (a.D <= 8192) start_backward<T, 4, 256>(a, stream);
    else start_backward<T, 4, 1024>(a, stream);
    hipLaunchKernelGGL(csf_norm_dweight_kernel, dim3((a.D + kDweightCols - 1u) / kDweightCols), dim3(1024), 0, stream, a);
}

}  // namespace

uint32_t norm_backward_groups(uint32_t T, uint32_t D) {
    const uint32_t most = kCus * (D <= 1024 ? 16u : 4u);
    return T < most ? (T > 0 ? T : 1u) : most;
}

hipError_t launch_norm(int32_t dtype, const NormArgs &a, hipStream_t stream) {
    if (dtype == kBF16) pick_norm<__bf16>(a, stream);
    else if (dtype == kF16) pick_norm<_Float16>(a, stream);
    else pick_norm<float>(a, stream);
    return hipGetLastError();
}

hipError_t launch_norm_backward(int32_t dtype, const NormBackwardArgs &a, hipStream_t stream) {
    if (dtype == kBF16) pick_backward<__bf16>(a, stream);
    else if (dtype == kF16) pick_backward<_Float16>(a, stream);
    else pick_backward<float>(a, stream);
    return hipGetLastError();
}

}  // namespace csf

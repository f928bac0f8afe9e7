// Gated half of a routed feed-forward block on FP4 experts, gfx950, and its
// backward pass.  For slot s of expert e (rows[s] its token), with the gate
// rows W_g = W[e][0 .. F) and the up rows W_u = W[e][F .. 2F):
//     g = alpha[e] W_g x,  u = alpha[e] W_u x,  h = g sigmoid(g) u
//     dg = dh u p (1 + g (1 - p)),  du = dh g p   (p = sigmoid(g)),
//     dx = alpha[e] (dg W_g + du W_u)
// W = E2M1 code x block scale (E4M3 per 16 for NVFP4, E8M0 per 32 for MXFP4),
// x bfloat16, or (with MXFP4 weights) E4M3 codes with E8M0 scales per 32.
//
// Sums are float32 in the matrix cores.  bfloat16 activations meet weights
// widened to bfloat16, which holds them exactly (at most 6 significant bits);
// 8-bit activations meet the codes themselves in the scaled matrix
// instruction, in two classes (low_codes).  No factor is rounded in either.
#include "csf_layer_device.h"

#include <type_traits>

namespace csf {
namespace {

constexpr uint32_t kGatedThreads = 256;  // 4 waves (the tile code's workgroup)
constexpr uint32_t kGatedWaves = kGatedThreads / kWave;
constexpr uint32_t kGatedCols = 16;      // columns of h per unit: 16 gate and 16 up rows
constexpr uint32_t kGatedChunk = 128;    // K per chunk (4 lane groups x 32)

typedef float v4f32 __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf16 __attribute__((ext_vector_type(8)));
typedef int v8i32 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float e4m3_scale(uint32_t b) { return __builtin_amdgcn_cvt_f32_fp8((int)b, 0); }

// An E8M0 byte as the float whose exponent field it is: the conversions below
// read only that field (byte 0, 2^-127, is passed as 0.0).
__device__ __forceinline__ float e8m0_field(uint32_t b) {
    return b == 0xffu ? __uint_as_float(0x7fc00000u) : __uint_as_float(b << 23);
}

// The upper halves of two floats that bfloat16 holds exactly.
__device__ __forceinline__ uint32_t pack_upper(float lo, float hi) {
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

// 8 codes of a word (byte j: codes 2j low, 2j + 1 high) as bfloat16 weights.
// The conversion's own scale acts through its exponent only: it carries an
// E8M0 scale; an E4M3 scale is multiplied in (exact: at most 6 bits).
template <bool MX>
__device__ __forceinline__ v8bf16 widen8(uint32_t codes, float scale) {
    uint32_t w[4];
    if constexpr (MX) {
        w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
        w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
        w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
        w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
    } else {
        const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
        const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
        const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2);
        const v2f d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
        w[0] = pack_upper(a.x * scale, a.y * scale);
        w[1] = pack_upper(b.x * scale, b.y * scale);
        w[2] = pack_upper(c.x * scale, c.y * scale);
        w[3] = pack_upper(d.x * scale, d.y * scale);
    }
    return __builtin_bit_cast(v8bf16, (u32x4){w[0], w[1], w[2], w[3]});
}

template <bool MX>
__device__ __forceinline__ float block_scale(uint32_t b) {
    if constexpr (MX) return e8m0_field(b);
    else return e4m3_scale(b);
}

// The scaled matrix instruction adds products of 8 consecutive k first, and cuts
// each toward zero below 2^-13 of the power of two of the largest; the eights'
// sums and the running sum are joined in 24 bits (measured by small products
// next to large ones).  An E2M1 code is a multiple of 1/2 up to 6, an E4M3 code of
// power 2^e a multiple of 2^(e - 3): nothing is cut where the eight activations'
// powers lie within 2^7 of each other.  E4M3's 15 powers are therefore taken in
// two classes, 2^1 and above (bit 6 set) and 2^0 and below, each with an
// instruction of its own and zeros for the others' codes.  In one class sums of 32
// random codes were off by up to 2^-12.4 of the terms' magnitudes; in two nothing
// is left of that beyond the rounding of the result.
//
// The codes below 2 of four.  The bytes' masks are the signs of x << 1's bytes.
__device__ __forceinline__ uint32_t low_codes(uint32_t x) {
    return x & ~__builtin_amdgcn_perm(x << 9, x << 1, 0x090b080au);
}

__device__ __forceinline__ v8i32 low_class(v8i32 x) {
    v8i32 low;
#pragma unroll
    for (int i = 0; i < 8; ++i) low[i] = (int)low_codes((uint32_t)x[i]);
    return low;
}

// acc + the products of 128 weight codes w and one class x of E4M3 codes.
__device__ __forceinline__ v4f32 scaled_products(v8i32 w, v8i32 x, v4f32 acc, uint32_t w_scale, uint32_t x_scale) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 4, 0, 0, (int)w_scale, 0, (int)x_scale);
}

// sigmoid(g) and 1 - sigmoid(g) from e = exp(-|g|), which cannot overflow; both
// keep their relative precision.  With n the whole part of -|g| log2(e), e =
// 2^n 2^f: f, at most a half, is a fused difference with log2(e) in two parts,
// so that large |g| lose nothing.  Below -200 e is 0 either way, and NaN stays
// with g's own factors.
__device__ __forceinline__ v2f sigmoid2(float g) {
    const float x = fmaxf(-fabsf(g), -200.0f);
    const float n = rintf(x * 1.44269504f);
    const float f = fmaf(x, 1.92596303e-8f, fmaf(x, 1.44269504f, -n));
    const float e = __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    return g >= 0.f ? (v2f){r, e * r} : (v2f){e * r, r};
}

// ---------------------------------------------------------------- few tokens
//
// Unit: 16 columns of h (16 gate and 16 up rows) of a routed expert, all of its
// slots in passes of 16.  The weights' bytes bound it, so a unit's loads
// go out as early as their addresses are known: the routing first; then the
// codes (all of a wave's share of K), the scales' streams,
// the slots' tokens; the exceptions once the tile index is in; the first
// activations once the tokens are.  The scales are expanded in LDS meanwhile.
// The waves take every eighth chunk of K, NCH of them each (they cover it), their
// sums meet in LDS and are added in the waves' order.  Several workgroups per compute unit cover each other's
// round trips.

// 16 scale bytes of run `pos` (a multiple of 16) of a plane, from its offset
// group and the row bases of rows r_lo .. in LDS.
template <bool MX>
__device__ __forceinline__ u32x4 expand_run(const StackArgs &st, u32x4 group, uint32_t pos, const uint8_t *bases, uint32_t r_lo) {
    constexpr uint32_t WB = MX ? 1u : 4u, MASK = MX ? 0x01010101u : 0x0f0f0f0fu;
    const u32x4 field = (group >> (WB * ((pos >> 4) & (8u / WB - 1u)))) & MASK;
    switch (st.row_mode) {
        case kRowSplat: return add_bytes4(field, run_bases<kRowSplat>(bases, pos, r_lo, st.C, st.rcp_cols));
        case kRowTwo: return add_bytes4(field, run_bases<kRowTwo>(bases, pos, r_lo, st.C, st.rcp_cols));
        default: return add_bytes4(field, run_bases<kRowBytes>(bases, pos, r_lo, st.C, st.rcp_cols));
    }
}

constexpr uint32_t kUnitWaves = 8;       // the vector work of widening a unit's weights is spread over 8 waves
constexpr uint32_t kUnitThreads = kUnitWaves * kWave;
constexpr uint32_t kUnitChunks = 8;      // chunks of a wave, at most
static_assert(kUnitChunks * kUnitWaves * kGatedChunk >= kGatedMaxK, "a unit's waves hold all of K");
constexpr uint32_t kUnitBases = 2u * kGatedCols + kBasesSlack;  // row bases of a half's span, its neighbours among them

template <bool MX, bool X8, bool DENSE, uint32_t NCH>
__global__ __launch_bounds__(kUnitThreads, NCH > 4 ? 2 : 4) void csf_gated_unit_kernel(GatedArgs a) {
    constexpr uint32_t BLOCK = MX ? 32u : 16u, GROUP = MX ? 128u : 32u;
    constexpr uint32_t STRIDE = kUnitWaves * kGatedChunk;  // a wave's chunks are this far apart
    extern __shared__ __align__(16) uint8_t dyn_lds[];
    __shared__ __align__(16) v4f32 s_part[kUnitWaves][2][kWave];
    __shared__ uint8_t s_bases[2][kUnitBases];
    __shared__ uint32_t s_nact;
    __shared__ int32_t s_rows[kUnitThreads];
    const uint32_t F = a.F, K = a.K, C = a.C, span = 16u * C + 32u;
    // dynamic LDS: scales of the gate and the up rows | expert_start | routed experts
    uint8_t *s_scales = dyn_lds;
    int32_t *s_es = reinterpret_cast<int32_t *>(dyn_lds + 2u * span);
    uint16_t *act = reinterpret_cast<uint16_t *>(s_es + a.E + 1u);
    const uint32_t tid = threadIdx.x, lane = tid % kWave, row = lane & 15u, kq = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    // with few slots their tokens come along with the routing: one round trip less
    const bool posted = a.S <= kUnitThreads;
    if (posted && tid < a.S) s_rows[tid] = a.rows[tid];
    for (uint32_t i = tid; i <= a.E; i += kUnitThreads) s_es[i] = a.expert_start[i];
    __syncthreads();
    if (tid < kWave) {
        const uint32_t n = list_experts(static_cast<const int32_t *>(s_es), a.E, act);
        if (tid == 0) s_nact = n;
    }
    __syncthreads();
    const uint32_t ntiles = (F + kGatedCols - 1u) / kGatedCols, total = s_nact * ntiles;
    for (uint32_t u = blockIdx.x; u < total; u += gridDim.x) {
        const uint32_t kx = u / ntiles, e = __builtin_amdgcn_readfirstlane(act[kx]), n0 = (u - kx * ntiles) * kGatedCols;
        const uint32_t cols = min(kGatedCols, F - n0);
        const uint32_t s0 = (uint32_t)min(max(__builtin_amdgcn_readfirstlane(s_es[e]), 0), (int32_t)a.S);
        const uint32_t s1 = (uint32_t)min(max(__builtin_amdgcn_readfirstlane(s_es[e + 1]), (int32_t)s0), (int32_t)a.S);
        const uint32_t m = s1 - s0;
        if (m == 0) continue;

        // ---- loads: tile index, tokens of the first pass, codes, scale streams
        uint32_t lo[2] = {}, hi[2] = {}, q0[2], skew[2];
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            q0[h] = (h * F + n0) * C;
            skew[h] = DENSE ? 0u : q0[h] & 15u;
            if constexpr (!DENSE) {
                const int32_t *index = a.st.tile_index + (uint64_t)e * a.st.index_tiles;
                lo[h] = (uint32_t)index[q0[h] / kIndexTile];
                hi[h] = (uint32_t)index[min((q0[h] + cols * C + kIndexTile - 1u) / kIndexTile, a.st.index_tiles)];
            }
        }
        auto token = [&](uint32_t s) {
            const uint32_t slot = s0 + min(s, m - 1u);
            return (uint64_t)min(max(posted ? s_rows[slot] : a.rows[slot], 0), (int32_t)a.T - 1);
        };
        uint64_t at = token(row);
        const float alpha = a.alpha[e];
        // a range per half: rows past the unit's columns and chunks past K read 0
        rsrc_t rw[2];
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) rw[h] = make_rsrc(a.w + ((uint64_t)e * 2u * F + h * F + n0) * (K / 2u), cols * (K / 2u));
        u32x4 codes[NCH][2];
#pragma unroll
        for (uint32_t c = 0; c < NCH; ++c) {
            const uint32_t k = c * STRIDE + wave * kGatedChunk + 32u * kq;
            const uint32_t off = k < K ? row * (K / 2u) + k / 2u : 0x80000000u;
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) codes[c][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw[h], (int)off, 0, kNonTemporal));
        }
        // ---- scale bytes of the unit's rows into LDS
        if constexpr (DENSE) {
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {
                const uint8_t *src = a.dense + (uint64_t)e * 2u * F * C + q0[h];
                for (uint32_t i = tid; i < cols * C; i += kUnitThreads) s_scales[h * span + i] = src[i];
            }
        } else {
            uint32_t r_lo[2], runs[2];
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {
                const uint32_t q1 = q0[h] + cols * C, qa = q0[h] - skew[h];
                r_lo[h] = div_exact(qa, a.st.rcp_cols);
                runs[h] = (q1 - qa + kRunBytes - 1u) / kRunBytes;
                const uint32_t rows = div_exact(q1 - 1u, a.st.rcp_cols) - r_lo[h] + 1u;  // at most 16 + 15 / C + 1
                if (tid / kWave == h && lane < rows) s_bases[h][lane] = a.st.bases[(uint64_t)e * a.st.R + r_lo[h] + lane];
            }
            const uint8_t *offsets = a.st.offsets + (uint64_t)e * a.st.stride;
            auto run_pos = [&](uint32_t j) { return j < runs[0] ? q0[0] - skew[0] + kRunBytes * j : q0[1] - skew[1] + kRunBytes * (j - runs[0]); };
            u32x4 group = {0u, 0u, 0u, 0u};
            if (tid < runs[0] + runs[1]) group = *reinterpret_cast<const u32x4 *>(offsets + (run_pos(tid) / GROUP) * 16u);
            uint32_t first[2], count[2], entry[2];
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {  // the first entries while the runs are expanded
                const uint32_t end = min((uint32_t)max((int32_t)hi[h], 0), a.st.n_exc);
                first[h] = min((uint32_t)max((int32_t)lo[h], 0), end);
                count[h] = end - first[h];
                entry[h] = tid < count[h] ? a.st.exc[first[h] + tid] : 0u;
            }
            __syncthreads();
            for (uint32_t j = tid; j < runs[0] + runs[1]; j += kUnitThreads) {
                const uint32_t h = j < runs[0] ? 0u : 1u, pos = run_pos(j);
                if (j != tid) group = *reinterpret_cast<const u32x4 *>(offsets + (pos / GROUP) * 16u);
                *reinterpret_cast<u32x4 *>(s_scales + h * span + (pos - (q0[h] - skew[h]))) = expand_run<MX>(a.st, group, pos, s_bases[h], h ? r_lo[1] : r_lo[0]);
            }
            __syncthreads();
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h)
                for (uint32_t i = tid; i < count[h]; i += kUnitThreads) {
                    const uint32_t x = i == tid ? entry[h] : a.st.exc[first[h] + i], p = x >> 8;
                    if (p >= q0[h] && p < q0[h] + cols * C) s_scales[h * span + p - q0[h] + skew[h]] = (uint8_t)(x & 0xffu);
                }
        }

                    constexpr uint32_t XV = X8 ? 2u : 4u;
                    u32x4 x[2][XV];
                    uint32_t xs[2];
                    auto load_x = [&](uint32_t kc, auto bufc) {  // kc: the wave's chunk
                        constexpr uint32_t BUF = decltype(bufc)::value;
                        const u32x4 zero = {0u, 0u, 0u, 0u};
                        if constexpr (X8) {
                            // 8-bit operands: lane group q holds k = 16 q .. + 15 and 64 + 16 q .. + 15 of the chunk, but the
                            // scale of block q, as 4-bit ones hold 32 q .. + 31
                            const uint8_t *p = static_cast<const uint8_t *>(a.x) + at * K + kc + 16u * kq;
                            x[BUF][0] = kc + 16u * kq < K ? *reinterpret_cast<const u32x4 *>(p) : zero;
                            x[BUF][1] = kc + 64u + 16u * kq < K ? *reinterpret_cast<const u32x4 *>(p + 64) : zero;
                            xs[BUF] = kc + 32u * kq < K ? a.x_scales[at * (K / 32u) + kc / 32u + kq] : 0u;
                        } else {
                            const u32x4 *p = reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.x) + at * K + kc + 32u * kq);
        #pragma unroll
                            for (uint32_t s = 0; s < 4; ++s) x[BUF][s] = kc + 32u * kq < K ? p[s] : zero;
                        }
                    };
        const std::integral_constant<uint32_t, 0> even;
        const std::integral_constant<uint32_t, 1> odd;
        uint32_t kc = wave * kGatedChunk;
        load_x(kc, even);
        __syncthreads();  // the scales are in LDS
        for (uint32_t tb = 0; tb < m; tb += 16u) {
            // Widened anew for every 16 slots, and compared with K anew: kept from pass to pass, as the compiler would
            // have it, the weights and the comparisons' results do not fit the registers.
            asm volatile("" : "+s"(kc));
#pragma unroll
            for (uint32_t c = 0; c < NCH; ++c) asm volatile("" : "+v"(codes[c][0]), "+v"(codes[c][1]));
            if (tb > 0) {
                at = token(tb + row);
                load_x(kc, even);
            }
            v4f32 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            auto products = [&](uint32_t kc, const u32x4 (&code)[2], auto bufc) {
                constexpr uint32_t BUF = decltype(bufc)::value;
                const uint32_t k = kc + 32u * kq;
                __builtin_amdgcn_sched_barrier(0);  // the next chunk's activations are on their way, no more
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    const bool ok = k < K && row < cols;
                    const uint8_t *sc = s_scales + h * span + skew[h] + row * C + k / BLOCK;
                    const uint32_t sc0 = ok ? sc[0] : 0u, sc1 = ok && !MX ? sc[1] : sc0;
                    if constexpr (X8) {
                        const v8i32 wv = {(int)code[h].x, (int)code[h].y, (int)code[h].z, (int)code[h].w, 0, 0, 0, 0};
                        const v8i32 xv = {(int)x[BUF][0].x, (int)x[BUF][0].y, (int)x[BUF][0].z, (int)x[BUF][0].w,
                                          (int)x[BUF][1].x, (int)x[BUF][1].y, (int)x[BUF][1].z, (int)x[BUF][1].w};
                        const v8i32 low = low_class(xv);
                        acc[h] = scaled_products(wv, low, acc[h], sc0, xs[BUF]);
                        acc[h] = scaled_products(wv, xv ^ low, acc[h], sc0, xs[BUF]);
                    } else {
                        const uint32_t wd[4] = {code[h].x, code[h].y, code[h].z, code[h].w};
                        const float f[2] = {block_scale<MX>(sc0), block_scale<MX>(sc1)};
#pragma unroll
                        for (uint32_t s = 0; s < 4; ++s)
                            acc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<MX>(wd[s], f[s >> 1]),
                                                                             __builtin_bit_cast(v8bf16, x[BUF][s]), acc[h], 0, 0, 0);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            };
#pragma unroll
            for (uint32_t c = 0; c < NCH; c += 2u) {
                if (c + 1u < NCH) load_x(kc + (c + 1u) * STRIDE, odd);
                products(kc + c * STRIDE, codes[c], even);
                if (c + 1u < NCH) {
                    if (c + 2u < NCH) load_x(kc + (c + 2u) * STRIDE, even);
                    products(kc + (c + 1u) * STRIDE, codes[c + 1u < NCH ? c + 1u : 0u], odd);
                }
            }
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) s_part[wave][h][lane] = acc[h];
            __syncthreads();
            // thread i: column i % 16 of slot i / 16; lane l of a wave's sums holds columns 4 (l / 16) .. + 3 of slot l % 16
            const uint32_t n = tid & 15u, t = (tid >> 4) & 15u, l = 16u * (n / 4u) + t;
            float g = 0.f, up = 0.f;
#pragma unroll
            for (uint32_t w = 0; w < kUnitWaves; ++w) {
                g += reinterpret_cast<const float *>(&s_part[w][0][l])[n & 3u];
                up += reinterpret_cast<const float *>(&s_part[w][1][l])[n & 3u];
            }
            if (tid < 256u && n < cols && tb + t < m) {
                const uint64_t slot = s0 + tb + t;
                g *= alpha, up *= alpha;
                reinterpret_cast<__bf16 *>(a.h)[slot * F + n0 + n] = (__bf16)(g * sigmoid2(g).x * up);
                if (a.gu != nullptr) {
                    __bf16 *gu = reinterpret_cast<__bf16 *>(a.gu) + slot * 2u * F + n0 + n;
                    gu[0] = (__bf16)g;
                    gu[F] = (__bf16)up;
                }
            }
            __syncthreads();  // the sums are read before they, or the scales, are written again
        }
    }
}

// ---------------------------------------------------------------- many tokens
//
// Tiles of 128 slots x 128 columns of h (256 weight rows) of one expert.  A
// wave owns 32 columns (two 16-row blocks of the gate and two of the up half)
// for all of the tile's slots, so no weight is read or widened twice in a
// tile: codes go from memory straight to the wave's registers, up to two steps
// ahead, scales through LDS 16 bytes of a row at a time.  The slots'
// activations are shared: gathered by rows[] and copied to LDS by the load
// itself, 256 bytes of K per slot and step, two buffers, one barrier per step.
// A row's 16-byte pieces are stored with their index xored by the row, so the 16
// rows of an operand read lie in different banks.  The scales are dense (decoded
// ahead of the kernel): a tile would spend three dependent round trips on
// expanding its own.
//
// 131,072 slots through 512 experts, K = 2048, 2 x 800 rows, NVFP4, bfloat16
// activations: 1.15 to 1.21 ms, 720 to 750 TFLOP/s.  Of that the matrix cores
// are busy 0.38 ms and vector instructions, most of them widening (two to a
// weight, two to three to a matrix instruction), issue for 0.35 ms; the two
// waves of a SIMD spend a third of their time issuing, a third waiting for the
// other's instructions and a third for loads, LDS and barriers.  Neither bounds
// it alone: what does not overlap is a tile's first loads and its stores, and
// the last of seven column tiles, in which one wave of four has columns (800 of
// 896).  35 to 53 vector registers are spilled in a tile's beginning and end and
// between steps; one load of them a step lies among the products (8 bits).
// 8-bit activations need no widening, but two products for their two classes:
// 65,536 slots through 384 experts, K = 5120, 2 x 512 rows, MXFP4: 0.80 to 0.85
// ms, 840 TFLOP/s (in one class, with sums cut as said above, 0.58 ms).  The
// matrix cores are busy 0.31 ms, vector instructions issue for 0.28 ms, and the
// loads take 3.7 GB through the L2s; waits are shared as above.  The same with
// bfloat16 activations takes 0.79 ms.

constexpr uint32_t kTileTokens = 128;
constexpr uint32_t kTileCols = 128;
constexpr uint32_t kStepBytes = 256;           // bytes of K per slot and step
constexpr uint32_t kTileLds = kTileTokens * kStepBytes;
constexpr uint32_t kOutside = 0x80000000u;     // buffer offset past every range used here: reads 0
constexpr int kLoadsButFour = 0x0f74;          // s_waitcnt: all but the wave's last four loads have arrived
constexpr int kLoadsDone = 0x0f70;             // s_waitcnt: every load of the wave has arrived, those into LDS too
constexpr uint32_t kXcds = 8;                  // workgroups go round-robin to 8 XCDs

__device__ __forceinline__ u32x4 buf_b128(rsrc_t r, uint32_t off, uint32_t add) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, (int)add, 0));
}

// Tiles of an expert's m slots.
__device__ __forceinline__ uint32_t expert_tiles(const int32_t *expert_start, uint32_t e, uint32_t S, uint32_t &s0, uint32_t &m) {
    s0 = (uint32_t)min(max(expert_start[e], 0), (int32_t)S);
    m = (uint32_t)min(max(expert_start[e + 1u], (int32_t)s0), (int32_t)S) - s0;
    return (m + kTileTokens - 1u) / kTileTokens;
}

// Tiles before each thread's run of experts (ceil(E / kGatedThreads) of them):
// prefix[i].  Returns the number of all.
__device__ __forceinline__ uint32_t tile_prefix(const int32_t *expert_start, uint32_t E, uint32_t S, uint32_t *prefix, uint32_t *scan) {
    const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const uint32_t per = (E + kGatedThreads - 1u) / kGatedThreads, e0 = tid * per;
    uint32_t sum = 0, s0, m;
    for (uint32_t i = 0; i < per && e0 + i < E; ++i) sum += expert_tiles(expert_start, e0 + i, S, s0, m);
    uint32_t s = sum;
#pragma unroll
    for (uint32_t d = 1; d < kWave; d *= 2) {
        const uint32_t o = (uint32_t)__shfl_up((int)s, d);
        if (lane >= d) s += o;
    }
    if (lane == kWave - 1u) scan[wave] = s;
    __syncthreads();
    uint32_t before = s - sum, all = 0;
#pragma unroll
    for (uint32_t w = 0; w < kGatedWaves; ++w) {
        if (w < wave) before += scan[w];
        all += scan[w];
    }
    prefix[tid] = before;
    __syncthreads();
    return all;
}

struct Tile {
    uint32_t e, t0, count, pairs;  // expert, first slot, slots, blocks of 32 slots
};

// Tile number `tile` of all: the last run of experts that begins at or before
// it, then the expert in the run.  An expert's slots are spread evenly over its
// tiles, in blocks of 16.
__device__ __forceinline__ Tile find_tile(const uint32_t *prefix, const int32_t *expert_start, uint32_t E, uint32_t S, uint32_t tile) {
    uint32_t lo = 0;
#pragma unroll
    for (uint32_t d = kGatedThreads / 2u; d > 0; d /= 2u)
        if (prefix[lo + d] <= tile) lo += d;
    lo = __builtin_amdgcn_readfirstlane(lo);
    uint32_t before = __builtin_amdgcn_readfirstlane(prefix[lo]), e = lo * ((E + kGatedThreads - 1u) / kGatedThreads), s0, m;
    uint32_t mts = expert_tiles(expert_start, e, S, s0, m);
    while (e + 1u < E && tile >= before + mts) {
        before += mts;
        ++e;
        mts = expert_tiles(expert_start, e, S, s0, m);
    }
    const TileBlocks b = tile_blocks(m, tile - before, mts);
    return {e, s0 + 16u * b.first, min(16u * b.count, m - 16u * b.first), (b.count + 1u) / 2u};
}

// Tiles left are handed out by counters in `queue`, one for each XCD's
// contiguous range of them (few experts' activations and weights per L2); a
// workgroup whose range is used up takes from the next one's.  Without a queue
// the tiles are dealt out in turn.  Every id is taken once, so a workgroup
// comes to an end after at most kXcds empty answers.
struct TileQueue {
    uint32_t *queue;
    uint32_t per, total, x, left;

    __device__ __forceinline__ uint32_t ask() const { return atomicAdd(queue + x, 1u); }
    // the tile that answer i stands for, asking on where a range is used up; total when nothing is left
    __device__ __forceinline__ uint32_t settle(uint32_t i) {
        for (;;) {
            const uint32_t u = x * per + i;
            if (i < per && u < total) return u;
            if (--left == 0) return total;
            x = (x + 1u) & (kXcds - 1u);
            i = ask();
        }
    }
};

template <bool MX, bool X8>
__global__ __launch_bounds__(kGatedThreads, 2) void csf_gated_tile_kernel(GatedArgs a) {
    constexpr uint32_t BLOCK = MX ? 32u : 16u;
    constexpr uint32_t STEP = X8 ? kStepBytes : kStepBytes / 2u;  // K per step
    constexpr uint32_t XB = X8 ? 1u : 2u;                         // bytes per activation
    constexpr uint32_t LOADS = kTileLds / (16u * kGatedThreads);  // 16-byte pieces per lane and step
    constexpr uint32_t SB = STEP / BLOCK;                         // scale bytes per weight row and step (4 or 8)
    constexpr uint32_t PERIOD = 16u / SB;                         // steps that 16 scale bytes of a row last
    // arrays of their own, chosen at compile time: reads of one must not wait for loads into the other
    __shared__ __align__(16) uint8_t s_x0[kTileLds], s_x1[kTileLds];
    __shared__ __align__(16) uint8_t s_sc[kGatedWaves][kWave * 16u];             // scales of a wave's 64 weight rows
    __shared__ __align__(8) uint8_t s_xs[2][X8 ? kTileTokens * 8u : 8u];         // the slots' scales of the step
    __shared__ uint32_t s_prefix[kGatedThreads];
    __shared__ uint32_t s_scan[kGatedWaves];
    __shared__ uint32_t s_next;
    const uint32_t tid = threadIdx.x, lane = tid % kWave, row = lane & 15u, kq = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const uint32_t F = a.F, K = a.K, C = a.C;
    const uint32_t mtiles = tile_prefix(a.expert_start, a.E, a.S, s_prefix, s_scan);
    const uint32_t ntiles = (F + kTileCols - 1u) / kTileCols, total = mtiles * ntiles;
    const uint32_t steps = (K + STEP - 1u) / STEP;
    const rsrc_t rx = make_rsrc(a.x, a.T * K * XB);

    TileQueue q = {a.queue, (total + kXcds - 1u) / kXcds, total, blockIdx.x & (kXcds - 1u), kXcds};
    uint32_t u = blockIdx.x;
    if (a.queue != nullptr) {
        if (tid == 0) s_next = q.settle(q.ask());
        __syncthreads();
        u = __builtin_amdgcn_readfirstlane(s_next);
    }
    while (u < total) {
        uint32_t answer = 0;
        const uint32_t mt = u / ntiles, nt = u - mt * ntiles;
        const Tile at = find_tile(s_prefix, a.expert_start, a.E, a.S, mt);
        const uint32_t e = at.e, t0 = at.t0, count = at.count;
        const uint32_t n0 = nt * kTileCols + 32u * wave;  // the wave's first column
        const float alpha = a.alpha[e];
        const uint32_t plane = 2u * F * K / 2u;
        const rsrc_t rw = make_rsrc(a.w + (uint64_t)e * plane, plane);

        uint32_t xoff[LOADS];
#pragma unroll
        for (uint32_t i = 0; i < LOADS; ++i) {
            const uint32_t r = (wave * LOADS + i) * 4u + lane / 16u, c = (lane ^ r) & 15u;
            const int32_t t = a.rows[t0 + min(r, count - 1u)];
            // rows past the tile's blocks are not read
            xoff[i] = r < 32u * at.pairs ? (uint32_t)min(max(t, 0), (int32_t)a.T - 1) * K * XB + 16u * c : kOutside;
        }
        // Weight row `row` of block f: gate rows n0 + 16 (f % 2) .. for f < 2, up rows for the others.  A gate
        // block that passes F reads up rows, an up block that passes 2F reads 0: columns that are not stored.
        // A quad of lanes loads 64 contiguous bytes of a row (its 16-byte pieces spread over the rows of 16
        // lanes load at a third of the rate); the operand wants lane (row, group) instead: a lane permutation.
        const uint32_t woff = (lane >> 2) * (K / 2u) + 16u * (lane & 3u);
        const int from = (int)(4u * (4u * row + kq));
        // scales are copied to LDS 16 bytes of a row at a time: lane l takes row l % 16 of block l / 16
        const uint8_t *scales = a.dense + ((uint64_t)e * 2u * F + min(n0 + 16u * (kq & 1u) + row, F - 1u) + (kq >> 1) * F) * C;
        const uint8_t *xscales = nullptr;  // thread i: half i % 2 of slot i / 2
        if constexpr (X8) {
            const int32_t t = a.rows[t0 + min(tid / 2u, count - 1u)];
            xscales = a.x_scales + (uint64_t)min(max(t, 0), (int32_t)a.T - 1) * (K / 32u);
        }

        auto tile = [&](auto nbc) {
            constexpr uint32_t NB = decltype(nbc)::value;
            v4f32 acc[4][NB];
#pragma unroll
            for (uint32_t f = 0; f < 4; ++f)
#pragma unroll
                for (uint32_t b = 0; b < NB; ++b) acc[f][b] = (v4f32){0.f, 0.f, 0.f, 0.f};
            u32x4 staged = {0u, 0u, 0u, 0u};  // the next period's scales on their way to LDS
            uint32_t xstaged = 0;

            // bytes at .. at + 3 of a row of `size` bytes, 0 past its end
            auto bytes = [](const uint8_t *p, uint32_t at, uint32_t size) {
                uint32_t v = 0;
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i)
                    if (at + i < size) v |= (uint32_t)p[at + i] << (8u * i);
                return v;
            };
            auto load_scales = [&](uint32_t period) {
                const uint32_t at = 16u * period;
                typedef u32x4 any128 __attribute__((aligned(1)));
                if (at + 16u <= C) staged = *reinterpret_cast<const any128 *>(scales + at);
                else if (at < C) staged = (u32x4){bytes(scales, at, C), bytes(scales, at + 4u, C), bytes(scales, at + 8u, C), bytes(scales, at + 12u, C)};
            };
            auto store_scales = [&]() { *reinterpret_cast<u32x4 *>(s_sc[wave] + lane * 16u) = staged; };
            auto load_xscales = [&](uint32_t step) {
                typedef uint32_t any32 __attribute__((aligned(1)));
                const uint32_t at = step * 8u + 4u * (tid & 1u);
                if ((step + 1u) * STEP <= K) xstaged = *reinterpret_cast<const any32 *>(xscales + at);
                else xstaged = bytes(xscales, at, K / 32u);
            };
            auto store_xscales = [&](uint32_t step) {
                if constexpr (X8) reinterpret_cast<uint32_t *>(s_xs[step & 1u])[tid] = xstaged;
            };
            auto buffer = [&](auto parity) -> uint8_t * {
                if constexpr (decltype(parity)::value == 0) return s_x0;
                else return s_x1;
            };
            const std::integral_constant<uint32_t, 0> even;
            const std::integral_constant<uint32_t, 1> odd;
            // piece i of a step's activations into an LDS buffer
            auto load_x = [&](uint32_t step, auto parity, uint32_t i) {
                const uint32_t kb = step * STEP;
                uint32_t off = xoff[i];
                if (kb + STEP > K) {
                    const uint32_t r = (wave * LOADS + i) * 4u + lane / 16u, c = (lane ^ r) & 15u;
                    off = kb + c * (16u / XB) < K ? off : kOutside;
                }
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rx, (__attribute__((address_space(3))) void *)(buffer(parity) + (wave * LOADS + i) * 1024u), 16, (int)off, (int)(min(kb, K) * XB), 0, 0);
            };
            // codes of 128 of K of block f, as loaded and as the operands take them
            auto load_w = [&](uint32_t part, uint32_t f) {
                const uint32_t kb = part * 128u;
                // no scalar offset passes the range's end: the bound less it must not wrap
                return buf_b128(rw, kb + 32u * (lane & 3u) < K ? woff : kOutside, min(((f >> 1) * F + n0 + 16u * (f & 1u)) * (K / 2u) + kb / 2u, plane));
            };
            auto load_codes = [&](uint32_t part, u32x4 (&codes)[4]) {
#pragma unroll
                for (uint32_t f = 0; f < 4; ++f) codes[f] = load_w(part, f);
            };
            auto spread = [&](const u32x4 (&codes)[4], u32x4 (&code)[4]) {
#pragma unroll
                for (uint32_t f = 0; f < 4; ++f) {
                    const u32x4 c = codes[f];
                    code[f] = (u32x4){(uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)c.x), (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)c.y),
                                      (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)c.z), (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)c.w)};
                }
            };
            const bool some = n0 < F;  // the wave has columns

            // every step in turn; waves without columns take part in the loads and barriers only, in a loop of their own,
            // so that no wait in the other one depends on a branch
            auto idle = [&](uint32_t step, auto, auto other) {
                __builtin_amdgcn_s_waitcnt(kLoadsDone);
                __syncthreads();
                if constexpr (X8) load_xscales(step + 1u);
                if (step == 0 && tid == 0 && a.queue != nullptr) answer = q.ask();
#pragma unroll
                for (uint32_t i = 0; i < LOADS; ++i) load_x(step + 1u, other, i);
                store_xscales(step + 1u);
            };
            auto every = [&](auto &&one) {
                for (uint32_t step = 0; step < steps; step += 2u) {
                    one(step, even, odd);
                    if (step + 1u < steps) one(step + 1u, odd, even);
                }
            };
            load_scales(0u);
            if constexpr (X8) load_xscales(0u);
#pragma unroll
            for (uint32_t i = 0; i < LOADS; ++i) load_x(0u, even, i);
            store_scales();
            store_xscales(0u);
            if (!some) {
                every(idle);
            } else if constexpr (X8) {
                // 128 of K: half h of the step's buffer
                auto compute = [&](uint32_t step, auto parity, const u32x4 (&codes)[4], uint32_t h, auto &&between) {
                    const uint8_t *x = buffer(parity) + row * kStepBytes, *sc = s_sc[wave] + row * 16u + (step % PERIOD) * SB;
                    u32x4 code[4];
                    spread(codes, code);
                    const uint8_t *lo = x + (((8u * h + kq) ^ row) * 16u), *hi = x + (((8u * h + 4u + kq) ^ row) * 16u);
                    const uint8_t *xs = s_xs[step & 1u] + row * 8u + 4u * h + kq;
                    auto read = [&](uint32_t b) {
                        const u32x4 l = *reinterpret_cast<const u32x4 *>(lo + b * 16u * kStepBytes);
                        const u32x4 u = *reinterpret_cast<const u32x4 *>(hi + b * 16u * kStepBytes);
                        return (v8i32){(int)l.x, (int)l.y, (int)l.z, (int)l.w, (int)u.x, (int)u.y, (int)u.z, (int)u.w};
                    };
                    uint32_t ws[4];
#pragma unroll
                    for (uint32_t f = 0; f < 4; ++f) ws[f] = sc[f * 256u + 4u * h + kq];
                    v8i32 next = read(0u);
                    uint32_t xs_next = xs[0];
#pragma unroll
                    for (uint32_t b = 0; b < NB; ++b) {
                        const v8i32 xv = next;
                        const uint32_t xscale = xs_next;
                        if (b + 1u < NB) next = read(b + 1u), xs_next = xs[(b + 1u) * 128u];
                        const v8i32 low = low_class(xv), high = xv ^ low;
#pragma unroll
                        for (uint32_t i = 0; i < 8; ++i) {  // a class at a time: no product waits for the last one's sum
                            const uint32_t f = i % 4u;
                            const u32x4 c = code[f];
                            const v8i32 wv = {(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
                            acc[f][b] = scaled_products(wv, i < 4u ? low : high, acc[f][b], ws[f], xscale);
                        }
                        between(b);
                        // one block's operands ahead, no more: read all at once they would not fit the registers
                        __builtin_amdgcn_sched_barrier(0);
                    }
                };
                u32x4 codes[2][4];
                __builtin_amdgcn_sched_barrier(0);  // the waits below count on the order of the loads
                load_codes(0u, codes[0]);
                auto one = [&](uint32_t step, auto parity, auto other) {
                    // all but the last four loads, this step's first codes, have arrived
                    __builtin_amdgcn_s_waitcnt(kLoadsButFour);
                    __syncthreads();  // this step's activations and scales are in LDS, the other buffer is free
                    // past K the loads read nothing: no wait depends on a branch
                    if ((step + 1u) % PERIOD == 0) load_scales((step + 1u) / PERIOD);
                    load_xscales(step + 1u);
                    load_codes(2u * step + 1u, codes[1]);
                    if (step == 0 && tid == 0 && a.queue != nullptr) answer = q.ask();
                    __builtin_amdgcn_sched_barrier(0);
                    // the other loads go out between the products, one at a time: sent all at once they hold the wave up
                    compute(step, parity, codes[0], 0u, [&](uint32_t b) {
#pragma unroll
                        for (uint32_t i = 0; i < LOADS; ++i)
                            if (i * NB / LOADS == b) load_x(step + 1u, other, i);
                    });
                    compute(step, parity, codes[1], 1u, [&](uint32_t b) {
#pragma unroll
                        for (uint32_t f = 0; f < 4; ++f)
                            if (f * NB / 4u == b) codes[0][f] = load_w(2u * step + 2u, f);
                    });
                    if ((step + 1u) % PERIOD == 0) store_scales();  // the wave has read the old ones
                    store_xscales(step + 1u);
                };
                every(one);
            } else {
                // A phase is 32 of K.  While its products run, the next phase's weights are widened, the operands of
                // the next two blocks of slots are on their way from LDS and the next step's loads go out; the codes
                // are two steps ahead, since they need not pass a barrier.
                u32x4 codes[4], code[4];
                v8bf16 wv[2][4];
                float f0[4], f1[4];
                auto factors = [&](uint32_t step) {
                    const uint8_t *sc = s_sc[wave] + row * 16u + (step % PERIOD) * SB;
#pragma unroll
                    for (uint32_t f = 0; f < 4; ++f) {
                        if constexpr (MX) {
                            f0[f] = f1[f] = e8m0_field(sc[f * 256u + kq]);
                        } else {
                            const uint32_t pair = *reinterpret_cast<const uint16_t *>(sc + f * 256u + 2u * kq);
                            f0[f] = __builtin_amdgcn_cvt_f32_fp8((int)pair, 0), f1[f] = __builtin_amdgcn_cvt_f32_fp8((int)pair, 1);
                        }
                    }
                };
                auto widen = [&](uint32_t s, uint32_t f) {
                    const uint32_t wd[4] = {code[f].x, code[f].y, code[f].z, code[f].w};
                    return widen8<MX>(wd[s], MX || s < 2 ? f0[f] : f1[f]);
                };
                // Always true, but for the compiler a branch: a step as one block of code does not fit the registers.
                uint32_t products = 1u;
                asm volatile("" : "+s"(products));
                const uint32_t xat = row * kStepBytes + ((4u * kq) ^ row) * 16u;
                __builtin_amdgcn_sched_barrier(0);  // the waits below count on the order of the loads
                load_codes(0u, codes);
                spread(codes, code);
                factors(0u);
                load_codes(1u, codes);
#pragma unroll
                for (uint32_t f = 0; f < 4; ++f) wv[0][f] = widen(0u, f);
                auto one = [&](uint32_t step, auto parity, auto other) {
                    // all but the last four loads, the next step's codes, have arrived
                    __builtin_amdgcn_s_waitcnt(kLoadsButFour);
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup", "local");
                    __builtin_amdgcn_s_barrier();  // this step's activations are in LDS, the other buffer is free
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup", "local");
                    __builtin_amdgcn_sched_barrier(0);
                    if ((step + 1u) % PERIOD == 0) load_scales((step + 1u) / PERIOD);
                    if (step == 0 && tid == 0 && a.queue != nullptr) answer = q.ask();
                    const uint8_t *x = buffer(parity);
                    auto read = [&](uint32_t i) {  // block i % NB of phase i / NB
                        return *reinterpret_cast<const u32x4 *>(x + (xat ^ (16u * (i / NB))) + (i % NB) * 16u * kStepBytes);
                    };
                    u32x4 xv[3];
                    xv[0] = read(0u), xv[1] = read(1u);
                    auto phase = [&](auto sc) {
                        constexpr uint32_t s = decltype(sc)::value;
                        // a third of the next step's activations, or the codes of the one after it
#pragma unroll
                        for (uint32_t l = 0; l < LOADS; ++l)
                            if (s < 3 && l * 3u / LOADS == s) load_x(step + 1u, other, l);
                        if constexpr (s == 3) load_codes(step + 2u, codes);
                        __builtin_amdgcn_sched_barrier(0);
                        if (products) {
#pragma unroll
                            for (uint32_t b = 0; b < NB; ++b) {
                                constexpr uint32_t G = 4u * NB;
                                const uint32_t i = s * NB + b;
                                if (i + 2u < G) xv[(i + 2u) % 3u] = read(i + 2u);
                                const v8bf16 xb = __builtin_bit_cast(v8bf16, xv[i % 3u]);
#pragma unroll
                                for (uint32_t f = 0; f < 4; ++f) acc[f][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[s & 1u][f], xb, acc[f][b], 0, 0, 0);
#pragma unroll
                                for (uint32_t f = 0; f < 4; ++f)
                                    if (f * NB / 4u == b) wv[(s + 1u) & 1u][f] = widen((s + 1u) & 3u, f);
                                __builtin_amdgcn_sched_barrier(0);
                            }
                        }
                        if constexpr (s == 2) {  // the codes and scales of the next step, whose first weights the last phase widens
                            if ((step + 1u) % PERIOD == 0) store_scales();  // the wave has read the old ones
                            spread(codes, code);
                            factors(step + 1u);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    };
                    phase(std::integral_constant<uint32_t, 0>{});
                    phase(std::integral_constant<uint32_t, 1>{});
                    phase(std::integral_constant<uint32_t, 2>{});
                    phase(std::integral_constant<uint32_t, 3>{});
                };
                every(one);
            }
            // Epilogue: h, then g and u, through LDS (the buffers in turn), so that 16 lanes store 256 contiguous
            // bytes of a row.  A lane holds 4 consecutive columns of a slot; 16-byte pieces are xored by the slot.
            auto put = [&](uint8_t *lds, uint32_t f, uint32_t b, const float (&v)[4]) {
                const uint32_t piece = (4u * wave + 2u * f + kq / 2u) ^ row;
                *reinterpret_cast<uint2 *>(lds + (16u * b + row) * 256u + 16u * piece + 8u * (kq & 1u)) =
                    make_uint2(pack2<__bf16>(v[0], v[1]), pack2<__bf16>(v[2], v[3]));
            };
            auto write = [&](const uint8_t *lds, uint16_t *dst, uint32_t stride) {
                __syncthreads();
                const uint32_t col = nt * kTileCols + 8u * (tid % 16u), t = tid / 16u;
                const uint8_t *src = lds + t * 256u + 16u * ((tid ^ t) & 15u);  // t and t + 16 i have the same xor
                uint16_t *d = dst + (uint64_t)(t0 + t) * stride + col;
                if (col + 8u <= F) {
                    u32x4 v[NB];
#pragma unroll
                    for (uint32_t i = 0; i < NB; ++i) v[i] = *reinterpret_cast<const u32x4 *>(src + 4096u * i);
                    __builtin_amdgcn_sched_barrier(0);  // all reads, then all stores: no store waits for the next read
#pragma unroll
                    for (uint32_t i = 0; i < NB; ++i)
                        if (t + 16u * i < count) *reinterpret_cast<u32x4_any *>(d + (uint64_t)(16u * i) * stride) = v[i];
                } else {
#pragma unroll 1
                    for (uint32_t n = 0; col + n < F; ++n)
#pragma unroll 1
                        for (uint32_t i = t; i < count; i += 16u)
                            d[(uint64_t)(i - t) * stride + n] = *reinterpret_cast<const uint16_t *>(src + 256u * (i - t) + 2u * n);
                }
            };
            __builtin_amdgcn_s_waitcnt(kLoadsDone);  // no load into LDS outlives the tile
            if (tid == 0 && a.queue != nullptr) s_next = q.settle(answer);
            __syncthreads();                         // the last step's operands are read
#pragma unroll
            for (uint32_t b = 0; b < NB; ++b)
#pragma unroll
                for (uint32_t f = 0; f < 2; ++f) {
                    float h[4];
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) {
                        acc[f][b][i] *= alpha, acc[2 + f][b][i] *= alpha;
                        h[i] = acc[f][b][i] * sigmoid2(acc[f][b][i]).x * acc[2 + f][b][i];
                    }
                    put(s_x0, f, b, h);
                }
            write(s_x0, a.h, F);
            if (a.gu != nullptr) {
#pragma unroll
                for (uint32_t half = 0; half < 2; ++half) {
#pragma unroll
                    for (uint32_t b = 0; b < NB; ++b)
#pragma unroll
                        for (uint32_t f = 0; f < 2; ++f) {
                            const v4f32 g = acc[2u * half + f][b];
                            put(half == 0 ? s_x1 : s_x0, f, b, {g.x, g.y, g.z, g.w});
                        }
                    write(half == 0 ? s_x1 : s_x0, a.gu + half * F, 2u * F);
                }
            }
            __syncthreads();  // the buffers are free for the next tile
        };
        switch (at.pairs) {
            case 1: tile(std::integral_constant<uint32_t, 2>{}); break;
            case 2: tile(std::integral_constant<uint32_t, 4>{}); break;
            case 3: tile(std::integral_constant<uint32_t, 6>{}); break;
            default: tile(std::integral_constant<uint32_t, 8>{}); break;
        }
        u = a.queue != nullptr ? __builtin_amdgcn_readfirstlane(s_next) : u + gridDim.x;
    }
}

__global__ void csf_gated_queue_kernel(uint32_t *queue) {
    if (threadIdx.x < kXcds) queue[threadIdx.x] = 0u;
}

// dgu of every routed slot: a workgroup takes rows in turn.
__global__ __launch_bounds__(kGatedThreads) void csf_gated_dgu_kernel(GatedBackwardArgs a) {
    const uint32_t F = a.F, used = (uint32_t)min(max(a.expert_start[a.E], 0), (int32_t)a.S);
    for (uint32_t s = (uint32_t)max(a.expert_start[0], 0) + blockIdx.x; s < used; s += gridDim.x) {
        const __bf16 *gu = reinterpret_cast<const __bf16 *>(a.gu) + (uint64_t)s * 2u * F;
        const __bf16 *dh = reinterpret_cast<const __bf16 *>(a.dh) + (uint64_t)s * F;
        __bf16 *dgu = reinterpret_cast<__bf16 *>(a.dgu) + (uint64_t)s * 2u * F;
        for (uint32_t f = threadIdx.x * 8u; f < F; f += kGatedThreads * 8u) {
            float g[8], u[8], d[8];
            load8(gu + f, F - f, g);
            load8(gu + F + f, F - f, u);
            load8(dh + f, F - f, d);
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) {
                const v2f p = sigmoid2(g[i]);
                const float dgi = d[i] * u[i] * p.x * fmaf(g[i], p.y, 1.0f);
                u[i] = d[i] * g[i] * p.x;
                g[i] = dgi;
            }
            store8(dgu + f, F - f, g);
            store8(dgu + F + f, F - f, u);
        }
    }
}

// dx = alpha dgu W.  The sum runs over the 2F weight rows, along which a
// matrix operand wants 8 consecutive values per lane, while the codes lie
// along K: a lane takes, of 8 rows, the 4 codes of its 4 columns, and operand
// j is made of code j of each row, so that column l % 16 of product j is the
// wave's column 4 (l % 16) + j and a lane's products over j are 4 consecutive
// columns of dx: one 8-byte store, 128 contiguous bytes of 16 lanes.
//
// Tiles of up to 128 slots x 256 columns of one expert, two workgroups of 4
// waves per compute unit; a wave owns 64 columns for all of the tile's slots,
// so a weight is widened once per tile.  Per step of 64 weight rows the slots'
// dgu (128 bytes each) and the codes (128 bytes a row) are copied to LDS by
// the loads themselves, the scale bytes through registers; three buffers, one
// barrier per step.  LDS pieces are xored (by slot, by 8 rows) so that the lanes
// a read serves at once find theirs in different banks.  dgu enters as rounded
// to bfloat16, the form it is returned in: half a step of 2^-8 on each factor,
// as the result's own rounding, for matrix cores that take 16 bits.
//
// 131,072 slots, K = 2048, 2 x 800 rows, NVFP4 in 1.29 to 1.33 ms, 655 TFLOP/s:
// the decode 0.05 ms, the pass over dgu 0.2 ms (bound by memory), then the
// products 1.05 ms, of which the matrix cores are busy 0.38 and vector
// instructions issue for 0.32; a third of the waves' time are waits for loads,
// LDS and barriers.
constexpr uint32_t kDxCols = 256;   // columns of dx per tile
constexpr uint32_t kDxWave = 64;    // per wave
constexpr uint32_t kDxRows = 64;    // weight rows per step

template <bool MX>
__global__ __launch_bounds__(kGatedThreads, 2) void csf_gated_dx_kernel(GatedBackwardArgs a) {
    constexpr uint32_t BLOCK = MX ? 32u : 16u;
    constexpr uint32_t WAVE_SCALES = kDxWave / BLOCK, SCALES = kDxCols / BLOCK;  // per weight row
    constexpr uint32_t PER = SCALES / 4u;                                        // staged by a thread
    // dgu, then codes: arrays of their own, chosen at compile time, as the compiler lets a read of LDS wait for every
    // load into LDS under way but where both are in arrays of which it knows that they differ
    constexpr uint32_t CODES_AT = kTileTokens * 128u;
    __shared__ __align__(16) uint8_t s_0[CODES_AT + kDxRows * 128u], s_1[CODES_AT + kDxRows * 128u], s_2[CODES_AT + kDxRows * 128u];
    __shared__ __align__(16) uint8_t s_s[3][SCALES * kDxRows];  // a block's scales of all rows lie together
    __shared__ uint32_t s_prefix[kGatedThreads];
    __shared__ uint32_t s_scan[kGatedWaves];
    const uint32_t tid = threadIdx.x, lane = tid % kWave, row = lane & 15u, kq = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const uint32_t F = a.F, K = a.K, C = a.C, N = 2u * F;
    const uint32_t mtiles = tile_prefix(a.expert_start, a.E, a.S, s_prefix, s_scan);
    const uint32_t ktiles = (K + kDxCols - 1u) / kDxCols, total = mtiles * ktiles;
    const uint32_t steps = (N + kDxRows - 1u) / kDxRows;
    // An offset past every tile's range of dgu: a constant would not be, since 128 slots of up to 2^24 - 2 rows reach
    // 2^32 - 512 bytes.
    const uint32_t past = kTileTokens * N * 2u;

    uint32_t u = blockIdx.x, ustep = gridDim.x, uend = total;
    if ((gridDim.x & (kXcds - 1u)) == 0) {
        const uint32_t per = (total + kXcds - 1u) / kXcds, x = blockIdx.x & (kXcds - 1u);
        u = x * per + blockIdx.x / kXcds;
        ustep = gridDim.x / kXcds;
        uend = min(total, (x + 1u) * per);
    }
    for (; u < uend; u += ustep) {
        const uint32_t mt = u / ktiles, k0 = (u - mt * ktiles) * kDxCols;
        const Tile at = find_tile(s_prefix, a.expert_start, a.E, a.S, mt);
        const uint32_t e = at.e, t0 = at.t0, count = at.count;
        const float alpha = a.alpha[e];
        const rsrc_t rd = make_rsrc(a.dgu + (uint64_t)t0 * N, count * N * 2u);  // slots past the tile's read 0
        const rsrc_t rw = make_rsrc(a.w + (uint64_t)e * N * (K / 2u), N * (K / 2u));
        const uint8_t *scales = a.dense + (uint64_t)e * N * C;
        const bool some = k0 + kDxWave * wave < K;  // the wave has columns

        auto tile = [&](auto nbc) {
            constexpr uint32_t NB = decltype(nbc)::value;
            v4f32 acc[4][NB];
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c)
#pragma unroll
                for (uint32_t b = 0; b < NB; ++b) acc[c][b] = (v4f32){0.f, 0.f, 0.f, 0.f};
            uint32_t staged = 0;

            // dgu and codes of a step into its LDS buffer (past 2F they read 0)
            auto buffer = [&](auto which) -> uint8_t * {
                if constexpr (decltype(which)::value == 0) return s_0;
                else if constexpr (decltype(which)::value == 1) return s_1;
                else return s_2;
            };
            auto load = [&](uint32_t step, auto which) {
                const uint32_t nb = step * kDxRows, from = min(nb, N);  // scalar offsets within the ranges
                if (nb + kDxRows <= N || N % 8u == 0) {
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) {
                        const uint32_t r = (wave * 4u + i) * 8u + lane / 8u, c = (lane ^ (r >> 1)) & 7u;
                        const uint32_t off = nb + 8u * c < N ? r * N * 2u + 16u * c : past;
                        __builtin_amdgcn_raw_ptr_buffer_load_lds(
                            rd, (__attribute__((address_space(3))) void *)(buffer(which) + (wave * 4u + i) * 1024u), 16, (int)off, (int)(from * 2u), 0, 0);
                    }
                } else {  // a 16-byte piece of the last step passes the row's end: 4 bytes at a time (N is even)
                    for (uint32_t i = 0; i < 16; ++i) {
                        const uint32_t r = (wave * 16u + i) * 2u + lane / 32u, c = ((lane % 32u) / 4u ^ (r >> 1)) & 7u;
                        const uint32_t n = 8u * c + 2u * (lane & 3u);
                        const uint32_t off = nb + n < N ? r * N * 2u + n * 2u : past;
                        __builtin_amdgcn_raw_ptr_buffer_load_lds(
                            rd, (__attribute__((address_space(3))) void *)(buffer(which) + (wave * 16u + i) * 256u), 4, (int)off, (int)(from * 2u), 0, 0);
                    }
                }
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i) {
                    const uint32_t n = (wave * 2u + i) * 8u + lane / 8u, c = (lane & 7u) ^ (2u * ((n >> 3) & 3u));
                    const uint32_t off = k0 + 32u * c < K ? n * (K / 2u) + k0 / 2u + 16u * c : kOutside;  // K is a multiple of 32
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(
                        rw, (__attribute__((address_space(3))) void *)(buffer(which) + (CODES_AT + (wave * 2u + i) * 1024u)), 16, (int)off, (int)(from * (K / 2u)), 0, 0);
                }
                // scales: thread i takes quarter i % 4 of row i / 4
                const uint32_t n = nb + tid / 4u, c = k0 / BLOCK + PER * (tid & 3u);
                const uint8_t *p = scales + (uint64_t)n * C + c;
                if (n < N && c + PER <= C) {
                    typedef uint32_t any32 __attribute__((aligned(1)));
                    typedef uint16_t any16 __attribute__((aligned(1)));
                    if constexpr (PER == 4) staged = *reinterpret_cast<const any32 *>(p);
                    else staged = *reinterpret_cast<const any16 *>(p);
                } else {
                    staged = 0;
#pragma unroll
                    for (uint32_t i = 0; i < PER; ++i)
                        if (n < N && c + i < C) staged |= (uint32_t)p[i] << (8u * i);
                }
            };
            auto store_scales = [&](auto which) {
                const uint32_t n = tid / 4u, block = PER * (tid & 3u);
#pragma unroll
                for (uint32_t i = 0; i < PER; ++i) s_s[decltype(which)::value][(block + i) * kDxRows + n] = (uint8_t)(staged >> (8u * i));
            };
            // A phase is 32 weight rows, two to a step.  While its products run, the next phase's weights are widened
            // from codes and scales read a phase before, and the slots' operands come two blocks ahead.  The barrier
            // lies between a step's phases: there the next step's operands are in LDS and the last step's buffer, of
            // three, is free for the loads of the step after, so that reading ahead never has to stop for it.
            uint32_t raw[8];
            uint2 factor[2];  // scale bytes of the 8 rows of each phase
            v8bf16 wv[2][4];
            u32x4 dv[3];
            auto read_raw = [&](auto which, uint32_t s) {
                const uint32_t at = CODES_AT + (32u * s + 8u * kq) * 128u + ((wave ^ kq) & 3u) * 32u + 2u * row;
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) raw[i] = *reinterpret_cast<const uint16_t *>(buffer(which) + (at + 128u * i));
            };
            // both phases' at once, while no load into LDS is under way
            auto read_factors = [&](auto which) {
                const uint8_t *sc = s_s[decltype(which)::value] + (wave * WAVE_SCALES + row * 4u / BLOCK) * kDxRows + 8u * kq;
                factor[0] = *reinterpret_cast<const uint2 *>(sc), factor[1] = *reinterpret_cast<const uint2 *>(sc + 32u);
            };
            auto scale = [&](uint32_t s, uint32_t i) {
                const uint32_t w = i < 4 ? factor[s].x : factor[s].y;
                if constexpr (MX) {  // 2^-127 is no float of the exponent field alone
                    const uint32_t b = (w >> (8u * (i & 3u))) & 0xffu;
                    return __builtin_amdgcn_ldexpf(b == 0xffu ? __builtin_nanf("") : 1.0f, (int)b - 127);
                } else {
                    return (i & 3u) == 0   ? __builtin_amdgcn_cvt_f32_fp8((int)w, 0)
                           : (i & 3u) == 1 ? __builtin_amdgcn_cvt_f32_fp8((int)w, 1)
                           : (i & 3u) == 2 ? __builtin_amdgcn_cvt_f32_fp8((int)w, 2)
                                           : __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
                }
            };
            // word q / 2 of columns 2 (q % 2) and the next: rows 2 (q / 2) and the next
            auto widen = [&](uint32_t s, uint32_t q, v8bf16 (&out)[4]) {
                const uint32_t i = 2u * (q / 2u), h = q % 2u;
                const v2f a = h == 0 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(raw[i], 1.0f, 0) : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(raw[i], 1.0f, 1);
                const v2f b = h == 0 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(raw[i + 1u], 1.0f, 0) : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(raw[i + 1u], 1.0f, 1);
                const float fa = scale(s, i), fb = scale(s, i + 1u);
                u32x4 lo = __builtin_bit_cast(u32x4, out[2u * h]), hi = __builtin_bit_cast(u32x4, out[2u * h + 1u]);
                lo[q / 2u] = pack_upper(a.x * fa, b.x * fb);
                hi[q / 2u] = pack_upper(a.y * fa, b.y * fb);
                out[2u * h] = __builtin_bit_cast(v8bf16, lo), out[2u * h + 1u] = __builtin_bit_cast(v8bf16, hi);
            };
            const uint32_t dat = row * 128u + ((kq ^ (row >> 1)) & 7u) * 16u;
            auto read_d = [&](auto which, uint32_t s, uint32_t b) {
                return *reinterpret_cast<const u32x4 *>(buffer(which) + ((dat ^ (64u * s)) + b * 2048u));
            };
            // products of phase s of the step in `which`, whose first two blocks are in dv[FIRST ..]; `next` holds the phase after it
            auto phase = [&](auto which, auto next, auto sc) {
                constexpr uint32_t s = decltype(sc)::value, FIRST = s * NB;
                if (some) {
#pragma unroll
                    for (uint32_t b = 0; b < NB; ++b) {
                        u32x4 &ahead = dv[(FIRST + b + 2u) % 3u];
                        const v8bf16 x = __builtin_bit_cast(v8bf16, dv[(FIRST + b) % 3u]);
                        if (b + 2u < NB) ahead = read_d(which, s, b + 2u);
                        else ahead = read_d(next, s ^ 1u, b + 2u - NB);
#pragma unroll
                        for (uint32_t c = 0; c < 4; ++c) acc[c][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, wv[s][c], acc[c][b], 0, 0, 0);
#pragma unroll
                        for (uint32_t q = 0; q < 8; ++q)
                            if (1u + q * (NB - 1u) / 8u == b) widen(s ^ 1u, q, wv[s ^ 1u]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            };
            // the ring goes on from one step to the next: after a step it has turned by 2 NB blocks
            auto turn = [&]() {
                constexpr uint32_t R = 2u * NB % 3u;
                if constexpr (R != 0) {
                    const u32x4 t0 = dv[R], t1 = dv[(R + 1u) % 3u];
                    dv[0] = t0, dv[1] = t1;
                }
            };
            auto meet = [&](auto next) {  // every wave's part of the step in buffer `next` is in LDS
                __builtin_amdgcn_s_waitcnt(kLoadsDone);
                store_scales(next);
                __syncthreads();
            };
            const std::integral_constant<uint32_t, 0> b0;
            const std::integral_constant<uint32_t, 1> b1;
            const std::integral_constant<uint32_t, 2> b2;
            load(0u, b0);
            meet(b0);
            if (some) {
                read_factors(b0);
                read_raw(b0, 0u);
#pragma unroll
                for (uint32_t q = 0; q < 8; ++q) widen(0u, q, wv[0]);
                read_raw(b0, 1u);
                dv[0] = read_d(b0, 0u, 0u), dv[1] = read_d(b0, 0u, 1u);
            }
            load(1u, b1);
            auto one = [&](uint32_t step, auto which, auto next, auto free) {
                phase(which, which, std::integral_constant<uint32_t, 0>{});
                meet(next);
                if (some) {
                    read_factors(next);
                    read_raw(next, 0u);
                }
                load(step + 2u, free);
                __builtin_amdgcn_sched_barrier(0);
                phase(which, next, std::integral_constant<uint32_t, 1>{});
                if (some) read_raw(next, 1u);
                turn();
            };
            for (uint32_t step = 0; step < steps; step += 3u) {
                one(step, b0, b1, b2);
                if (step + 1u < steps) one(step + 1u, b1, b2, b0);
                if (step + 2u < steps) one(step + 2u, b2, b0, b1);
            }
            __builtin_amdgcn_s_waitcnt(kLoadsDone);  // no load into LDS outlives the tile
            __syncthreads();                         // the buffers are free for the next one
            const uint32_t k = k0 + kDxWave * wave + 4u * row;
            if (k < K) {
#pragma unroll
                for (uint32_t b = 0; b < NB; ++b)
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) {
                        const uint32_t t = 16u * b + 4u * kq + i;
                        if (t < count)
                            *reinterpret_cast<uint2 *>(a.dx + (uint64_t)(t0 + t) * K + k) =
                                make_uint2(pack2<__bf16>(acc[0][b][i] * alpha, acc[1][b][i] * alpha),
                                           pack2<__bf16>(acc[2][b][i] * alpha, acc[3][b][i] * alpha));
                    }
            }
        };
        switch (at.pairs) {
            case 1: tile(std::integral_constant<uint32_t, 2>{}); break;
            case 2: tile(std::integral_constant<uint32_t, 4>{}); break;
            case 3: tile(std::integral_constant<uint32_t, 6>{}); break;
            default: tile(std::integral_constant<uint32_t, 8>{}); break;
        }
    }
}

}  // namespace

// Units take every expert's weights once per 16 slots, tiles once per 128, after a decode of the scales: 64 experts,
// K = 2048, 2 x 800 rows, with 16, 32 and 64 slots each 79, 116 and 198 us by units, 90, 92 and 103 us by tiles.  The
// host knows the slots' number, not how they spread: 6000 slots of 384 experts take 340 us by units and 313 by tiles
// where all have as many, 198 and 97 us where 8 experts have them all.
bool gated_by_tiles(uint32_t E, uint32_t S) { return S >= 20u * E; }

// 31-bit buffer offsets reach the activations; units take more of them.
bool tiles_reach(uint32_t T, uint32_t K, bool x8) { return uint64_t(T) * K * (x8 ? 1u : 2u) < (uint64_t(1) << 31); }

hipError_t launch_gated_tiles(const GatedArgs &a, hipStream_t stream) {
    const dim3 grid(2u * kCus), block(kGatedThreads);
    if (a.queue != nullptr) hipLaunchKernelGGL(csf_gated_queue_kernel, dim3(1), dim3(kWave), 0, stream, a.queue);
    if (a.mx && a.x_scales) hipLaunchKernelGGL((csf_gated_tile_kernel<true, true>), grid, block, 0, stream, a);
    else if (a.mx) hipLaunchKernelGGL((csf_gated_tile_kernel<true, false>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((csf_gated_tile_kernel<false, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <bool MX, bool X8, bool DENSE>
static void start_units(const GatedArgs &a, hipStream_t stream) {
    // at most min(E, S) experts have slots
    const uint64_t units = uint64_t(a.E < a.S ? a.E : a.S) * ((a.F + kGatedCols - 1u) / kGatedCols), cap = uint64_t(kCus) * 2u;
    const dim3 grid(uint32_t(units < cap ? units : cap)), block(kUnitThreads);
    const size_t lds = 2u * (16u * size_t(a.C) + 32u) + 4u * (size_t(a.E) + 1u) + 2u * size_t(a.E);
    const uint32_t chunks = (a.K + kUnitWaves * kGatedChunk - 1u) / (kUnitWaves * kGatedChunk);  // per wave
    if (chunks <= 1) hipLaunchKernelGGL((csf_gated_unit_kernel<MX, X8, DENSE, 1>), grid, block, lds, stream, a);
    else if (chunks <= 2) hipLaunchKernelGGL((csf_gated_unit_kernel<MX, X8, DENSE, 2>), grid, block, lds, stream, a);
    else if (chunks <= 4) hipLaunchKernelGGL((csf_gated_unit_kernel<MX, X8, DENSE, 4>), grid, block, lds, stream, a);
    else hipLaunchKernelGGL((csf_gated_unit_kernel<MX, X8, DENSE, kUnitChunks>), grid, block, lds, stream, a);
}

hipError_t launch_gated(const GatedArgs &a, hipStream_t stream) {
    if (a.mx && a.x_scales) {
        if (a.dense) start_units<true, true, true>(a, stream);
        else start_units<true, true, false>(a, stream);
    } else if (a.mx) {
        if (a.dense) start_units<true, false, true>(a, stream);
        else start_units<true, false, false>(a, stream);
    } else {
        if (a.dense) start_units<false, false, true>(a, stream);
        else start_units<false, false, false>(a, stream);
    }
    return hipGetLastError();
}

hipError_t launch_gated_backward(const GatedBackwardArgs &a, hipStream_t stream) {
    const dim3 block(kGatedThreads);
    hipLaunchKernelGGL(csf_gated_dgu_kernel, dim3(a.S < kCus * 8u ? a.S : kCus * 8u), block, 0, stream, a);
    const dim3 grid(2u * kCus);
    if (a.mx) hipLaunchKernelGGL(csf_gated_dx_kernel<true>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(csf_gated_dx_kernel<false>, grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace csf

// Router of a mixture-of-experts layer on gfx950: the k best experts of every
// token, their softmax gates and the routing grouped by expert; the backward
// pass of the routed combination and of the gates.
//
// Choice.  16 lanes take a token (64 in small calls, where latency counts, and
// where 16 would hold too many logits); each holds EPL consecutive logits, so a
// lane's experts lie below the next lane's.  Floats become unsigned keys of the
// same order (-0 as +0; -infinity and NaN as 0, which no round takes).  bfloat16
// logits leave room for the expert's complement in the key's lower half: keys
// are then distinct, and the next largest after t is t + max(key - t) in
// wrapping arithmetic, one subtraction and half a three-way maximum per key.
// Other types' keys find the maximum, then its lowest index, and are cleared.  The
// maximum over the lanes comes from cross-lane steps; lane j keeps choice j.
// The vector instructions of the rounds bound it: about 45 (bfloat16) or 110
// (others) a round of 24 keys per lane, for four tokens.
//
// Gates: exp(l_j - max) / sum, the sum over the chosen logits (renorm) or over
// all of the token's, in float32; 0 where there is no expert left.
//
// Grouping: a stable counting sort by expert of the T k choices.  A workgroup
// takes 64 tokens and sets bit t of a 64-bit mask per expert in LDS; a
// choice's rank among its workgroup's is the number of bits below its own, so
// the result does not depend on the order of the atomics.  With one workgroup
// the offsets follow at once.  Up to kRouteSumGroups of them, the second kernel's
// workgroups each add up all counts (a byte each) for themselves; beyond, a
// kernel of its own turns them into every workgroup's offsets first.
#include "csf_layer_device.h"

#include <type_traits>

namespace csf {
namespace {

constexpr uint32_t kRouteThreads = 1024;
// Counts of so many workgroups are added up in 16 bits, all in flight at once: four loads of 16 bytes a lane (the bits
// would do for 1023 workgroups).  A kernel of its own for the offsets costs more up to there (8192 x 384: 39.5 against
// 34.8 us, 16384: 52.9 against 52.3, calls from Python); beyond, where every workgroup reads all counts, it was not tried.
constexpr uint32_t kRouteSumGroups = 256;

__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 -> +0
    const uint32_t key = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
    return (v > -__builtin_inff()) ? key : 0u;  // -infinity, NaN: never chosen
}
__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// Exclusive prefix of the threads' values over the workgroup (256 to 1024
// threads); lds holds 16 words.  Every thread of the workgroup calls it.
__device__ __forceinline__ uint32_t exclusive_scan(uint32_t v, uint32_t *lds, uint32_t &total) {
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
    uint32_t s = v;
#pragma unroll
    for (uint32_t d = 1; d < kWave; d *= 2) {
        const uint32_t o = (uint32_t)__shfl_up((int)s, d);
        if (lane >= d) s += o;
    }
    if (lane == kWave - 1u) lds[wave] = s;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (uint32_t w = 0; w < waves; ++w) {
        const uint32_t x = lds[w];
        before += w < wave ? x : 0u;
        all += x;
    }
    __syncthreads();  // lds may be written again
    total = all;
    return before + s - v;
}

// Elements p[0 .. EPL) of which n exist, as floats, -infinity past them.
template <typename T, uint32_t EPL>
__device__ __forceinline__ void load_logits(const T *p, uint32_t n, float (&v)[EPL]) {
    if constexpr (EPL % 8u == 0) {
#pragma unroll
        for (uint32_t g = 0; g < EPL; g += 8u) {
            float w[8];
            const uint32_t left = n > g ? n - g : 0u;
            load8(p + g, left, w);
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) v[g + i] = i < left ? w[i] : -__builtin_inff();
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < EPL; ++i) v[i] = i < n ? (float)p[i] : -__builtin_inff();
    }
}

// Sum over the wave, the same in every lane (two 16-bit halves that do not overflow are summed apart).
__device__ __forceinline__ uint32_t wave_total(uint32_t v) {
    v += dpp_or_zero<0x111, 0xF>(v);
    v += dpp_or_zero<0x112, 0xF>(v);
    v += dpp_or_zero<0x114, 0xF>(v);
    v += dpp_or_zero<0x118, 0xF>(v);
    v += dpp_or_zero<0x142, 0xA>(v);
    v += dpp_or_zero<0x143, 0xC>(v);
    return __builtin_amdgcn_readlane(v, 63);
}

// Largest key, and sum, over a token's LANES lanes, the same in each of them.
template <uint32_t LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if constexpr (LANES == kWave) return wave_max(v);
    v = max(v, dpp_or_zero<0x128, 0xF>(v));  // rotations within 16 lanes
    v = max(v, dpp_or_zero<0x124, 0xF>(v));
    v = max(v, dpp_or_zero<0x122, 0xF>(v));
    return max(v, dpp_or_zero<0x121, 0xF>(v));
}
template <uint32_t LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (LANES == kWave) return wave_sum(v);
    v += dpp_or_zero<0x128>(v);
    v += dpp_or_zero<0x124>(v);
    v += dpp_or_zero<0x122>(v);
    return v + dpp_or_zero<0x121>(v);
}

template <typename T, uint32_t LANES, uint32_t EPL>
__global__ __launch_bounds__(kRouteThreads) void csf_route_kernel(RouteArgs a) {
    constexpr bool PACKED = std::is_same<T, __bf16>::value;  // the upper half of its float32 key holds a logit whole
    constexpr uint32_t PER = kWave / LANES;  // tokens of a wave at a time
    extern __shared__ __align__(16) uint8_t dyn_lds[];
    __shared__ uint32_t s_scan[kRouteThreads / kWave];
    uint64_t *mask = reinterpret_cast<uint64_t *>(dyn_lds);            // [E]
    uint32_t *start = reinterpret_cast<uint32_t *>(mask + a.E);        // [E] (one workgroup)
    int16_t *chosen = reinterpret_cast<int16_t *>(start + a.E);        // [64][k]
    const uint32_t waves = blockDim.x / kWave, sub = threadIdx.x % LANES;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t group = a.first + blockIdx.x, t0 = group * kRouteTokens;
    const uint32_t tokens = min(kRouteTokens, a.T - t0);
    const uint32_t E = a.E, k = a.k;
    for (uint32_t e = threadIdx.x; e < E; e += blockDim.x) mask[e] = 0;
    __syncthreads();

    for (uint32_t tb = wave * PER; tb < tokens; tb += waves * PER) {
        const uint32_t t = tb + threadIdx.x % kWave / LANES;
        const bool real = t < tokens;  // lanes past the last token repeat it
        const uint64_t row = t0 + min(t, tokens - 1u);
        const uint32_t first = sub * EPL;
        float v[EPL];
        load_logits(static_cast<const T *>(a.logits) + row * E + first, first < E ? E - first : 0u, v);
        uint32_t key[EPL];
#pragma unroll
        for (uint32_t i = 0; i < EPL; ++i) {
            key[i] = order_key(v[i]);
            if constexpr (PACKED) key[i] = key[i] == 0u ? 0u : (key[i] & 0xffff0000u) | (0xffffu - first - i);
        }
        int32_t expert = -1;  // lane j: choice j
        float logit = -__builtin_inff(), most = 0.f;
        uint32_t top = 0u;    // bfloat16: the last choice's key (0 at first: then key - top is the key)
        bool left = true;
        for (uint32_t j = 0; j < k; ++j) {
            uint32_t best = 0u, e;
            float l;
            if constexpr (PACKED) {
#pragma unroll
                for (uint32_t i = 0; i < EPL; ++i) best = max(best, key[i] - top);
                const uint32_t next = lanes_max<LANES>(best) + top;
                left = left && next != 0u;  // a masked key is 0; after it key - top would begin anew
                top = left ? next : 0u;
                e = 0xffffu - (top & 0xffffu);
                l = key_value((top & 0xffff0000u) | ((top >> 31) ? 0u : 0xffffu));  // the lower half as order_key leaves it
            } else {
#pragma unroll
                for (uint32_t i = 0; i < EPL; ++i) best = max(best, key[i]);
                top = lanes_max<LANES>(best);
                left = top != 0u;
                uint32_t at = 0u;
#pragma unroll
                for (uint32_t i = EPL; i-- > 0u;) at = key[i] == top ? i : at;
                const uint64_t offer = __ballot(best == top);
                const uint32_t base = threadIdx.x % kWave / LANES * LANES;
                const uint32_t winner = (uint32_t)__builtin_ctzll((offer >> base) | (1ull << 63));
                e = (uint32_t)__shfl((int)(first + at), (int)(base + (winner & (LANES - 1u))));
                const uint32_t mine = sub == winner && left ? at : EPL;
#pragma unroll
                for (uint32_t i = 0; i < EPL; ++i) key[i] = i == mine ? 0u : key[i];
                l = key_value(top);
            }
            if (j == 0 && left) most = l;
            if (sub == j && left) expert = (int32_t)e, logit = l;
        }
        const float p = expert < 0 ? 0.f : expf(logit - most);
        float whole;
        if (a.renorm) {
            whole = lanes_sum<LANES>(p);
        } else {
            float s = 0.f;
#pragma unroll
            for (uint32_t i = 0; i < EPL; ++i) s += v[i] > -__builtin_inff() ? expf(v[i] - most) : 0.f;
            whole = lanes_sum<LANES>(s);
        }
        if (sub < k && real) {
            a.experts[row * k + sub] = expert;
            a.gates[row * k + sub] = expert < 0 ? 0.f : p / whole;
            chosen[t * k + sub] = (int16_t)expert;
            if (expert >= 0) atomicOr(reinterpret_cast<unsigned long long *>(&mask[expert]), 1ull << t);
        }
    }
    __syncthreads();
    const bool one = a.groups == 1;
    if (one) {
        // offsets of the experts: thread i owns experts i per .. i per + per - 1
        const uint32_t per = (E + blockDim.x - 1u) / blockDim.x, e0 = threadIdx.x * per;
        uint32_t sum = 0, all;
        for (uint32_t i = 0; i < per && e0 + i < E; ++i) sum += (uint32_t)__popcll(mask[e0 + i]);
        uint32_t at = exclusive_scan(sum, s_scan, all);
        for (uint32_t i = 0; i < per && e0 + i < E; ++i) {
            start[e0 + i] = at;
            a.expert_start[e0 + i] = (int32_t)at;
            at += (uint32_t)__popcll(mask[e0 + i]);
        }
        if (threadIdx.x == 0) a.expert_start[E] = (int32_t)all;
        for (uint32_t i = all + threadIdx.x; i < tokens * k; i += blockDim.x) a.rows[i] = -1;
        __syncthreads();
    } else {
        const uint32_t stride = route_stride(E);
        for (uint32_t e = threadIdx.x; e < stride; e += blockDim.x)
            a.count[(uint64_t)group * stride + e] = e < E ? (uint8_t)__popcll(mask[e]) : 0u;
    }
    for (uint32_t i = threadIdx.x; i < tokens * k; i += blockDim.x) {
        const int32_t e = chosen[i];
        const uint32_t t = i / k;
        int32_t slot = -1;
        if (e >= 0) {
            slot = __popcll(mask[e] & ((1ull << t) - 1ull));
            if (one) {
                slot += (int32_t)start[e];
                a.rows[slot] = (int32_t)t;
            }
        }
        a.slots[(uint64_t)t0 * k + i] = slot;
    }
}

// Offset of every workgroup's choices within its experts, and the experts'
// totals: lane = expert, the 16 waves take consecutive ranges of workgroups.
__global__ __launch_bounds__(kRouteThreads) void csf_route_offsets_kernel(RouteArgs a) {
    __shared__ uint32_t s_sum[kRouteThreads / kWave][kWave];
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, waves = kRouteThreads / kWave;
    const uint32_t e = blockIdx.x * kWave + lane;
    const uint32_t per = (a.groups + waves - 1u) / waves, g0 = min(wave * per, a.groups), g1 = min(g0 + per, a.groups);
    uint32_t sum = 0;
    if (e < a.E) {
#pragma unroll 8
        for (uint32_t g = g0; g < g1; ++g) sum += a.count[(uint64_t)g * route_stride(a.E) + e];
    }
    s_sum[wave][lane] = sum;
    __syncthreads();
    uint32_t at = 0;
    for (uint32_t w = 0; w < wave; ++w) at += s_sum[w][lane];
    if (e >= a.E) return;
#pragma unroll 8
    for (uint32_t g = g0; g < g1; ++g) {
        a.base[(uint64_t)g * a.E + e] = at;
        at += a.count[(uint64_t)g * route_stride(a.E) + e];
    }
    if (wave == waves - 1u) a.total[e] = at;
}

// Slots and rows: expert's start + workgroup's offset + rank (left in slots).
// SUM: the workgroup adds up the counts itself: a wave takes 16 experts, its
// lanes every 64th workgroup's 16 bytes, two sums to a register (at most
// 64 * kRouteSumGroups < 2^16 each), joined across the lanes.
template <bool SUM>
__global__ __launch_bounds__(kRouteThreads) void csf_route_place_kernel(RouteArgs a) {
    extern __shared__ __align__(16) uint8_t dyn_lds[];
    __shared__ uint32_t s_scan[kRouteThreads / kWave];
    const uint32_t group = a.first + blockIdx.x, t0 = group * kRouteTokens;
    const uint32_t E = a.E, k = a.k, tokens = min(kRouteTokens, a.T - t0);
    const uint32_t stride = route_stride(E);
    uint32_t *total = reinterpret_cast<uint32_t *>(dyn_lds), *start = total + stride;  // [stride] each
    const uint32_t tid = threadIdx.x;
    // the first choices and their ranks arrive while the counts are added up
    const uint64_t choice = (uint64_t)t0 * k;
    const uint32_t i0 = min(tid, tokens * k - 1u);
    const int32_t e_first = a.experts[choice + i0];
    const uint32_t rank_first = (uint32_t)a.slots[choice + i0];
    if constexpr (SUM) {
        const uint32_t lane = tid % kWave;
        for (uint32_t c = tid / kWave; c < stride / 16u; c += kRouteThreads / kWave) {
            u32x4 v[kRouteSumGroups / kWave];
#pragma unroll
            for (uint32_t i = 0; i < kRouteSumGroups / kWave; ++i) {
                const uint32_t g = lane + kWave * i;
                v[i] = g < a.groups ? *reinterpret_cast<const u32x4 *>(a.count + (uint64_t)g * stride + 16u * c) : (u32x4){0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (uint32_t w = 0; w < 4; ++w) {
                uint32_t even = 0, odd = 0, even_before = 0, odd_before = 0;
#pragma unroll
                for (uint32_t i = 0; i < kRouteSumGroups / kWave; ++i) {
                    const uint32_t lo = v[i][w] & 0x00ff00ffu, hi = (v[i][w] >> 8) & 0x00ff00ffu;
                    const bool before = lane + kWave * i < group;
                    even += lo, odd += hi;
                    even_before += before ? lo : 0u, odd_before += before ? hi : 0u;
                }
                even = wave_total(even), odd = wave_total(odd), even_before = wave_total(even_before), odd_before = wave_total(odd_before);
                if (lane == 0) {
                    *reinterpret_cast<u32x4 *>(total + 16u * c + 4u * w) = (u32x4){even & 0xffffu, odd & 0xffffu, even >> 16, odd >> 16};
                    *reinterpret_cast<u32x4 *>(start + 16u * c + 4u * w) =
                        (u32x4){even_before & 0xffffu, odd_before & 0xffffu, even_before >> 16, odd_before >> 16};
                }
            }
        }
    } else {
        for (uint32_t e = tid; e < E; e += kRouteThreads) {
            total[e] = a.total[e];
            start[e] = a.base[(uint64_t)group * E + e];
        }
    }
    __syncthreads();
    const uint32_t per = (E + kRouteThreads - 1u) / kRouteThreads, e0 = tid * per;
    uint32_t sum = 0, all;
    for (uint32_t i = 0; i < per && e0 + i < E; ++i) sum += total[e0 + i];
    uint32_t at = exclusive_scan(sum, s_scan, all);
    for (uint32_t i = 0; i < per && e0 + i < E; ++i) {
        start[e0 + i] += at;
        if (group == 0) a.expert_start[e0 + i] = (int32_t)at;
        at += total[e0 + i];
    }
    if (group == 0 && tid == 0) a.expert_start[E] = (int32_t)all;
    __syncthreads();
    for (uint32_t i = tid; i < tokens * k; i += kRouteThreads) {
        const uint64_t at_choice = choice + i;
        if (at_choice >= all) a.rows[at_choice] = -1;
        const int32_t e = i == tid ? e_first : a.experts[at_choice];
        if (e < 0) continue;
        const uint32_t slot = start[e] + (i == tid ? rank_first : (uint32_t)a.slots[at_choice]);
        a.slots[at_choice] = (int32_t)slot;
        a.rows[slot] = (int32_t)(t0 + i / k);
    }
}

// Backward pass of out[t] = sum_j gates[t][j] y[slots[t][j]]: a wave takes a
// token; dy[slot] = gate dout, dgate = y[slot] . dout.
template <typename T>
__global__ __launch_bounds__(256) void csf_combine_backward_kernel(CombineBackwardArgs a) {
    const uint32_t lane = threadIdx.x % kWave;
    const uint32_t t = __builtin_amdgcn_readfirstlane((a.first + blockIdx.x) * 4u + threadIdx.x / kWave);
    if (t >= a.T) return;
    const uint32_t D = a.D;
    const T *dout = static_cast<const T *>(a.dout) + (uint64_t)t * D;
    for (uint32_t j = 0; j < a.k; ++j) {
        const int32_t slot = a.slots[(uint64_t)t * a.k + j];
        float dot = 0.f;
        if (slot >= 0 && slot < a.S) {
            const float g = a.gates[(uint64_t)t * a.k + j];
            const float *y = a.y + (int64_t)slot * D;
            T *dy = static_cast<T *>(a.dy) + (int64_t)slot * D;
            for (uint32_t d = lane * 8u; d < D; d += 8u * kWave) {
                float o[8], v[8];
                load8(dout + d, D - d, o);
                load8(y + d, D - d, v);
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) {
                    dot = fmaf(o[i], v[i], dot);
                    o[i] *= g;
                }
                store8(dy + d, D - d, o);
            }
        }
        dot = wave_sum(dot);
        if (lane == 0) a.dgates[(uint64_t)t * a.k + j] = dot;
    }
}

// Gradient of the logits: with p the softmax over all logits, or over the
// chosen ones (renorm), dl_e = p_e (dg_e [e chosen] - sum_j g_j dg_j).  A wave
// takes a token and holds its logits, EPL consecutive ones a lane; the chosen
// experts' terms reach their lanes through LDS.  Bound by memory.
template <typename T, uint32_t EPL>
__global__ __launch_bounds__(256) void csf_route_backward_kernel(RouteBackwardArgs a) {
    __shared__ __align__(16) float s_added[4][kWave * EPL];
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    float *added = s_added[wave];  // the chosen experts' p_e (dg_e - ..)
    const uint32_t t = __builtin_amdgcn_readfirstlane((a.first + blockIdx.x) * 4u + wave);
    if (t >= a.T) return;  // no barriers: a wave's LDS row is its own
    const uint32_t E = a.E, k = a.k, first = lane * EPL, left = first < E ? E - first : 0u;
    const uint64_t row = (uint64_t)t * E;
    float v[EPL];
    if (!a.renorm) load_logits(static_cast<const T *>(a.logits) + row + first, left, v);
    int32_t expert = -1;
    float g = 0.f, dg = 0.f;
    if (lane < k) {
        expert = a.experts[(uint64_t)t * k + lane];
        if (expert >= (int32_t)E) expert = -1;
        if (expert >= 0) g = a.gates[(uint64_t)t * k + lane], dg = a.dgates[(uint64_t)t * k + lane];
    }
#pragma unroll
    for (uint32_t i = 0; i < EPL; ++i) added[first + i] = 0.f;
    const float mean = wave_sum(g * dg);
    __builtin_amdgcn_wave_barrier();
    if (expert >= 0) added[expert] = g * (dg - (a.renorm ? mean : 0.f));
    __builtin_amdgcn_wave_barrier();
    float out[EPL];
#pragma unroll
    for (uint32_t i = 0; i < EPL; ++i) out[i] = added[first + i];
    if (!a.renorm) {
        float most = -__builtin_inff(), sum = 0.f;
#pragma unroll
        for (uint32_t i = 0; i < EPL; ++i) most = fmaxf(most, v[i]);
        const uint32_t top = wave_max(order_key(most));
        most = key_value(top);  // of no use where every logit is masked
#pragma unroll
        for (uint32_t i = 0; i < EPL; ++i) {
            v[i] = v[i] > -__builtin_inff() ? expf(v[i] - most) : -1.f;  // below 0: masked
            sum += fmaxf(v[i], 0.f);
        }
        const float scale = top == 0u ? 0.f : mean / wave_sum(sum);
        // a masked logit gets 0, not 0 times a mean that may be infinite or NaN
#pragma unroll
        for (uint32_t i = 0; i < EPL; ++i) out[i] = v[i] < 0.f ? out[i] : fmaf(-v[i], scale, out[i]);
    }
    T *dst = static_cast<T *>(a.dlogits) + row + first;
    if constexpr (EPL % 8u == 0) {
#pragma unroll
        for (uint32_t i = 0; i < EPL; i += 8u) {
            const float w[8] = {out[i], out[i + 1], out[i + 2], out[i + 3], out[i + 4], out[i + 5], out[i + 6], out[i + 7]};
            store8(dst + i, left > i ? left - i : 0u, w);
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < EPL; ++i)
            if (i < left) dst[i] = (T)out[i];
    }
}

template <typename T, uint32_t LANES, uint32_t EPL>
void start_route(const RouteArgs &all, uint32_t threads, size_t lds, hipStream_t stream) {
    launch_groups(all, all.groups, [&](const RouteArgs &a, dim3 grid) {
        hipLaunchKernelGGL((csf_route_kernel<T, LANES, EPL>), grid, dim3(threads), lds, stream, a);
    });
}

template <typename T>
void pick_route(const RouteArgs &a, hipStream_t stream) {
    const size_t lds = size_t(a.E) * 12 + size_t(kRouteTokens) * a.k * 2;
    // 16 lanes a token where there are tokens for most of the chip and the lanes hold the logits and the choices
    if (a.T >= 2048u && a.E <= 512u && a.k <= 16u) {
        const uint32_t epl = (a.E + 15u) / 16u;
        if (epl <= 2) start_route<T, 16, 2>(a, kRouteThreads, lds, stream);
        else if (epl <= 4) start_route<T, 16, 4>(a, kRouteThreads, lds, stream);
        else if (epl <= 8) start_route<T, 16, 8>(a, kRouteThreads, lds, stream);
        else if (epl <= 16) start_route<T, 16, 16>(a, kRouteThreads, lds, stream);
        else if (epl <= 24) start_route<T, 16, 24>(a, kRouteThreads, lds, stream);
        else start_route<T, 16, 32>(a, kRouteThreads, lds, stream);
    } else {
        const uint32_t threads = a.T >= 16 ? kRouteThreads : a.T > 4 ? 512 : 256;
        const uint32_t epl = (a.E + kWave - 1u) / kWave;
        if (epl <= 1) start_route<T, 64, 1>(a, threads, lds, stream);
        else if (epl <= 2) start_route<T, 64, 2>(a, threads, lds, stream);
        else if (epl <= 4) start_route<T, 64, 4>(a, threads, lds, stream);
        else if (epl <= 8) start_route<T, 64, 8>(a, threads, lds, stream);
        else if (epl <= 16) start_route<T, 64, 16>(a, threads, lds, stream);
        else start_route<T, 64, 32>(a, threads, lds, stream);
    }
    if (a.groups > 1) {
        const size_t place = 8u * size_t(route_stride(a.E));
        if (a.groups <= kRouteSumGroups) {
            hipLaunchKernelGGL(csf_route_place_kernel<true>, dim3(a.groups), dim3(kRouteThreads), place, stream, a);
        } else {
            hipLaunchKernelGGL(csf_route_offsets_kernel, dim3((a.E + kWave - 1u) / kWave), dim3(kRouteThreads), 0, stream, a);
            launch_groups(a, a.groups, [&](const RouteArgs &part, dim3 grid) {
                hipLaunchKernelGGL(csf_route_place_kernel<false>, grid, dim3(kRouteThreads), place, stream, part);
            });
        }
    }
}

}  // namespace

hipError_t launch_route(int32_t dtype, const RouteArgs &a, hipStream_t stream) {
    if (dtype == kBF16) pick_route<__bf16>(a, stream);
    else if (dtype == kF16) pick_route<_Float16>(a, stream);
    else pick_route<float>(a, stream);
    return hipGetLastError();
}

hipError_t launch_combine_backward(int32_t dtype, const CombineBackwardArgs &all, hipStream_t stream) {
    const dim3 block(256);
    launch_groups(all, (all.T + 3u) / 4u, [&](const CombineBackwardArgs &a, dim3 grid) {
        if (dtype == kBF16) hipLaunchKernelGGL(csf_combine_backward_kernel<__bf16>, grid, block, 0, stream, a);
        else if (dtype == kF16) hipLaunchKernelGGL(csf_combine_backward_kernel<_Float16>, grid, block, 0, stream, a);
        else hipLaunchKernelGGL(csf_combine_backward_kernel<float>, grid, block, 0, stream, a);
    });
    return hipGetLastError();
}

template <typename T>
static void pick_route_backward(const RouteBackwardArgs &all, hipStream_t stream) {
    const dim3 block(256);
    const uint32_t epl = (all.E + kWave - 1u) / kWave;
    launch_groups(all, (all.T + 3u) / 4u, [&](const RouteBackwardArgs &a, dim3 grid) {
        if (epl <= 1) hipLaunchKernelGGL((csf_route_backward_kernel<T, 1>), grid, block, 0, stream, a);
        else if (epl <= 2) hipLaunchKernelGGL((csf_route_backward_kernel<T, 2>), grid, block, 0, stream, a);
        else if (epl <= 4) hipLaunchKernelGGL((csf_route_backward_kernel<T, 4>), grid, block, 0, stream, a);
        else if (epl <= 8) hipLaunchKernelGGL((csf_route_backward_kernel<T, 8>), grid, block, 0, stream, a);
        else if (epl <= 16) hipLaunchKernelGGL((csf_route_backward_kernel<T, 16>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((csf_route_backward_kernel<T, 32>), grid, block, 0, stream, a);
    });
}

hipError_t launch_route_backward(int32_t dtype, const RouteBackwardArgs &a, hipStream_t stream) {
    if (dtype == kBF16) pick_route_backward<__bf16>(a, stream);
    else if (dtype == kF16) pick_route_backward<_Float16>(a, stream);
    else pick_route_backward<float>(a, stream);
    return hipGetLastError();
}

}  // namespace csf

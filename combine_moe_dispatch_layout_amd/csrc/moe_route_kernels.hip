// The router: experts and weights of each token from its logits, and the logits'
// gradient.
//
// What is chosen is decided by keys that are compared exactly: without a bias and
// without groups the logit itself (binary32; the score grows with it), otherwise
// score + bias in binary64, so that two experts closer than binary32 can tell are
// still taken in the formula's order.  The weights need no more than binary32.
//
// A token's logits sit in the registers of W lanes, expert u * W + l in lane l's u-th.
// Instructions bound the kernel: the k rounds of a maximum over those lanes, and with
// scores an exponential in 64 bits for each logit.  Scores take a whole wavefront for
// a token: what one lane found then is in scalar registers for all, and rounds compare
// 32 bits (4096 tokens of 256 experts in 8 groups, 8 chosen: 9.7 us; rounds of 64 bits
// 11.2; on 16 lanes 17.5).  Logits of up to 256 experts take 16 lanes, whose
// maximum needs no step between rows of lanes (8192 tokens of 64 experts, 6 chosen:
// 4.8 us; a wavefront each 7.1).
#include <type_traits>

#include "moe_ep.h"
#include "moe_internal.h"
#include "moe_layer.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// The value of the lane whose number differs in bit STEP, or of one that holds the same (what
// a reduction over aligned runs of lanes needs): quads, then mirrored halves of 16 lanes, then exchanges.
template <int STEP>
__device__ __forceinline__ uint32_t other(uint32_t v) {
    if constexpr (STEP == 1) return __builtin_amdgcn_update_dpp(v, v, 0xB1, 0xF, 0xF, true);
    else if constexpr (STEP == 2) return __builtin_amdgcn_update_dpp(v, v, 0x4E, 0xF, 0xF, true);
    else if constexpr (STEP == 4) return __builtin_amdgcn_update_dpp(v, v, 0x141, 0xF, 0xF, true);
    else if constexpr (STEP == 8) return __builtin_amdgcn_update_dpp(v, v, 0x140, 0xF, 0xF, true);
    else return __shfl_xor(v, STEP, 64);
}
template <int STEP, class T>
__device__ __forceinline__ T other_of(T v) {
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, other<STEP>(__builtin_bit_cast(uint32_t, v)));
    } else {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        return __builtin_bit_cast(T, ((uint64_t)other<STEP>((uint32_t)(b >> 32)) << 32) | other<STEP>((uint32_t)b));
    }
}
// f(f(..)) over the W lanes of a token; every lane gets the result.
template <int W, class T, class F>
__device__ __forceinline__ T over(T v, F f) {
    v = f(v, other_of<1>(v));
    v = f(v, other_of<2>(v));
    v = f(v, other_of<4>(v));
    v = f(v, other_of<8>(v));
    if constexpr (W == 64) {
        v = f(v, other_of<16>(v));
        v = f(v, other_of<32>(v));
    }
    return v;
}
struct Max {
    template <class T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a > b ? a : b; }
};
struct Min {
    template <class T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a < b ? a : b; }
};
struct Add {
    template <class T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

// Lane `from`'s value, for all (it is the same for all of them).
__device__ __forceinline__ int lane_of(int v, int from) { return __builtin_amdgcn_readlane(v, from); }
__device__ __forceinline__ float lane_of(float v, int from) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), from));
}
__device__ __forceinline__ double lane_of(double v, int from) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), from) << 32 |
                                          (uint32_t)__builtin_amdgcn_readlane((int)b, from));
}

// The row broadcasts of a reduction: CTRL 0x142 gives rows 1 and 3 the last lane of the row before, 0x143 the upper half lane
// 31; the others keep their own.
template <int CTRL>
__device__ __forceinline__ uint32_t from_row32(uint32_t v) {
    return __builtin_amdgcn_update_dpp(v, v, CTRL, CTRL == 0x142 ? 0xA : 0xC, 0xF, false);
}
template <int CTRL, class T>
__device__ __forceinline__ T from_row(T v) {
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, from_row32<CTRL>(__builtin_bit_cast(uint32_t, v)));
    } else {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        return __builtin_bit_cast(T, ((uint64_t)from_row32<CTRL>((uint32_t)(b >> 32)) << 32) | from_row32<CTRL>((uint32_t)b));
    }
}

template <class Key>
__device__ __forceinline__ Key lowest() { return -(Key)__builtin_inff(); }

// An integer in the order of binary32 numbers, zeros equal.
__device__ __forceinline__ int ordered(float v) {
    const int b = __builtin_bit_cast(int, v + 0.0f);
    return b ^ (b >> 31 & 0x7fffffff);
}

__device__ __forceinline__ float logit_of(const void* logits, int64_t at, bool bf16) {
    return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[at] << 16)
                : static_cast<const float*>(logits)[at];
}

// 1 / (1 + e^-v) and its complement, both without cancellation.
__device__ __forceinline__ float sigmoid32(float v) { return 1.0f / (1.0f + expf(-v)); }

// The largest of a token's lanes' values, for all of them.
template <int W, class T>
__device__ __forceinline__ T largest(T v) {
    v = Max()(v, other_of<1>(v));
    v = Max()(v, other_of<2>(v));
    v = Max()(v, other_of<4>(v));
    v = Max()(v, other_of<8>(v));
    if constexpr (W == 16) return v;
    // rows of 16: each second one gets the one before, then the upper half the lower; the last lane has all
    v = Max()(v, from_row<0x142>(v));
    v = Max()(v, from_row<0x143>(v));
    return lane_of(v, 63);
}

// 1 / d, to about a step; d and its reciprocal normal numbers
__device__ __forceinline__ double inverse(double d) {
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
    return __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
}

// A token on W lanes, PER logits a lane.  Key: float where keys are logits, double where they are scores (W = 64).
template <bool BF16, class Key, int W, int PER>
__global__ __launch_bounds__(kThreads) void k_route(RouteArgs a) {
    constexpr bool kScored = sizeof(Key) == 8;
    constexpr float kNone = -__builtin_inff();
    const int lane = threadIdx.x & 63, l = lane & (W - 1);
    const int t = (int)blockIdx.x * (kThreads / W) + (int)threadIdx.x / W;
    const bool live = t < a.T;
    float v[PER];
    bool bad = false;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int e = u * W + l;
        v[u] = live && e < a.E ? logit_of(a.logits, t * a.stride + e, BF16) : kNone;
    }
#pragma unroll
    for (int u = 0; u < PER; ++u)
        if (!(v[u] < __builtin_inff())) {   // infinite or NaN: not chosen, and reported; -inf: not chosen
            bad = true;
            v[u] = kNone;
        }
    if (__ballot(bad) != 0 && lane == 0) atomicOr(a.err, kErrNonFinite);
    float top = 0.0f;
    if (!a.sigmoid) {
        top = v[0];
#pragma unroll
        for (int u = 1; u < PER; ++u) top = fmaxf(top, v[u]);
        top = largest<W>(top);
        if (!(top > kNone)) top = 0.0f;   // nothing can be chosen: every exponential is zero
    }

    Key key[PER];
    float total = 0.0f;   // of the softmax's exponentials
    if constexpr (!kScored) {
#pragma unroll
        for (int u = 0; u < PER; ++u) key[u] = v[u];
        if (!a.sigmoid && !a.normalize) {
#pragma unroll
            for (int u = 0; u < PER; ++u) total += expf(v[u] - top);
            total = over<W>(total, Add());
        }
    } else {
        static_assert(W == 64);
        if (a.sigmoid) {
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const double x = v[u], tail = exp(-fabs(x));   // the smaller of the score and its complement, times a number from 1 to 2
                key[u] = (x < 0.0 ? tail : 1.0) * inverse(1.0 + tail);
            }
        } else {
            double sum = 0.0;
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                key[u] = exp((double)v[u] - (double)top);
                sum += key[u];
            }
            sum = over<64>(sum, Add());
            total = (float)sum;
            const double by = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
            for (int u = 0; u < PER; ++u) key[u] *= by;
        }
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int e = u * 64 + lane;
            if (a.bias != nullptr && e < a.E) key[u] += (double)a.bias[e];
            if (!(v[u] > kNone) || key[u] != key[u]) key[u] = lowest<Key>();
        }
        if (a.groups > 1) {
            // Group g's best two by `per` lanes, from g * per on, which take its experts in turn from LDS and put their own
            // together; then every group counts those before it.
            extern __shared__ double shared[];
            double* mine = shared + (threadIdx.x >> 6) * a.E;
#pragma unroll
            for (int u = 0; u < PER; ++u)
                if (u * 64 + lane < a.E) mine[u * 64 + lane] = key[u];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
            const int size = a.E / a.groups, per = a.group_lanes, g = lane / per;
            double first = lowest<Key>(), second = lowest<Key>();
            if (g < a.groups)
                for (int n = lane & (per - 1); n < size; n += per) {
                    const double x = mine[g * size + n];
                    second = Max()(second, first < x ? first : x);
                    first = Max()(first, x);
                }
            auto join = [&](double f, double s) {
                const double low = first < f ? first : f;
                first = Max()(first, f);
                second = Max()(Max()(second, s), low);
            };
            if (per > 1) join(other_of<1>(first), other_of<1>(second));
            if (per > 2) join(other_of<2>(first), other_of<2>(second));
            if (per > 4) join(other_of<4>(first), other_of<4>(second));
            if (per > 8) join(other_of<8>(first), other_of<8>(second));
            if (per > 16) join(other_of<16>(first), other_of<16>(second));
            const double score = a.top > 1 && second > lowest<Key>() ? first + second : first;
            int rank = 0;
            for (int j = 0; j < a.groups; ++j) {
                const double s = lane_of(score, j * per);
                rank += s > score || (s == score && j < g);
            }
            const uint64_t kept = __ballot(g < a.groups && rank < a.keep);
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const uint32_t e = u * 64 + lane;
                const uint32_t of = a.group_magic ? __umulhi(e, a.group_magic) : e;
                if (!(kept >> (of * per & 63) & 1)) key[u] = lowest<Key>();
            }
        }
    }

    // The best of what is left, k times; of equal keys the lowest expert.  Lane j keeps the j-th (k <= 32: two on 16 lanes).
    constexpr int kSlots = W == 64 ? 1 : 2;
    int mine_e[kSlots];
    float mine_v[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        mine_e[i] = -1;
        mine_v[i] = kNone;
    }
    auto keep = [&](int j, int e, float x) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
            if (i * W + l == j) {
                mine_e[i] = e;
                mine_v[i] = x;
            }
    };
    if constexpr (W == 64) {
        // Rounded to binary32, keys keep their order but for ties, and those are rare enough to be settled on the side.
        int fast[PER];
#pragma unroll
        for (int u = 0; u < PER; ++u) fast[u] = ordered((float)key[u]);
        for (int j = 0; j < a.k; ++j) {
            int best = fast[0];
#pragma unroll
            for (int u = 1; u < PER; ++u) best = Max()(best, fast[u]);
            best = largest<W>(best);
            if (best == ordered(kNone)) break;
            uint64_t equal[PER];
            int count = 0;
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                equal[u] = __ballot(fast[u] == best);
                count += __popcll(equal[u]);
            }
            if (kScored && count > 1) {
                Key m = lowest<Key>();
#pragma unroll
                for (int u = 0; u < PER; ++u)
                    if (fast[u] == best) m = Max()(m, key[u]);
                m = largest<W>(m);
#pragma unroll
                for (int u = 0; u < PER; ++u) equal[u] = __ballot(fast[u] == best && key[u] == m);
            }
            int chosen = 0, from = 0;
            float x = kNone;
#pragma unroll
            for (int u = PER - 1; u >= 0; --u)
                if (equal[u] != 0) {
                    chosen = u;
                    from = __ffsll((unsigned long long)equal[u]) - 1;
                    x = lane_of(v[u], from);
                }
#pragma unroll
            for (int u = 0; u < PER; ++u)
                if (u == chosen && lane == from) fast[u] = ordered(kNone);
            keep(j, chosen * W + from, x);
        }
    } else {
        for (int j = 0; j < a.k; ++j) {
            Key m = key[PER - 1];
            int e = (PER - 1) * W + l;
            float x = v[PER - 1];
#pragma unroll
            for (int u = PER - 2; u >= 0; --u)
                if (key[u] >= m) {
                    m = key[u];
                    e = u * W + l;
                    x = v[u];
                }
            const Key best = largest<W>(m);
            if (__ballot(best > lowest<Key>()) == 0) break;
            e = m == best ? e : INT32_MAX;
            const int chosen = over<W>(e, Min());
            x = over<W>(e == chosen ? x : kNone, Max());
            if (best > lowest<Key>()) {
#pragma unroll
                for (int u = 0; u < PER; ++u)
                    if (u * W + l == chosen) key[u] = lowest<Key>();
                keep(j, chosen, x);
            }
        }
    }
    // weights: shares of the chosen scores' sum, or the scores themselves
    float peak = kNone;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) peak = fmaxf(peak, mine_v[i]);
    peak = largest<W>(peak);
    float w[kSlots], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const float x = mine_v[i];
        if (mine_e[i] < 0) w[i] = 0.0f;
        else if (a.sigmoid) {
            // shares do not change when every score is divided by e^peak: a sum of small scores stays away from zero
            if (a.normalize && peak < 0.0f) w[i] = expf(x - peak) / (1.0f + expf(x));
            else w[i] = sigmoid32(x);
        } else w[i] = expf(x - (a.normalize ? peak : top));
        sum += w[i];
    }
    float by = a.scale;
    if (a.normalize) {
        sum = over<W>(sum, Add());
        by = sum > 0.0f ? a.scale / sum : 0.0f;
    } else if (!a.sigmoid) {
        by = a.scale / (total > 0.0f ? total : 1.0f);
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int j = i * W + l;
        if (live && j < a.k) {
            a.idx[(int64_t)t * a.k + j] = mine_e[i];
            a.weights[(int64_t)t * a.k + j] = w[i] * by;
        }
    }
}

// The gradient of a token's logits.  With r the weights without their factor c and g their gradients:
//   sigmoid              c g s (1 - s) for each slot's expert
//   shares (normalised)  c r_i sum over j of r_j (g_i - g_j) for each slot's expert, for sigmoids times 1 - s as well
//   softmax              the same over all experts, p for r, with g the sum of an expert's slots: -c p (sum of p g) for one
//                        that has no slot, for the others c p_i (sum over experts j with slots of p_j (g_i - g_j) + g_i times
//                        the p of those without)
// Differences are taken before they are added up: r_i (g_i - sum of r g), which is the same number, loses all of it for
// an expert that has nearly all of the weight, where the sum is nearly its own g.  Sums are
// binary64: an error of the scores' sum is one of all r together, and that of differences grows with the slots.
// Bound by latency: loads of the slots, of their logits, sums over the lanes, rounds over the slots, stores (8192 tokens of 64
// experts, 6 chosen, replayed: shares 3.9 us, 3.6 without differences; softmax 5.5 and 4.1).
template <bool BF16, int W, int PER>
__global__ __launch_bounds__(kThreads) void k_route_bwd(RouteBwdArgs a) {
    constexpr float kNone = -__builtin_inff();
    constexpr int kSlots = W == 64 ? 1 : 2;
    const int l = threadIdx.x & (W - 1);
    const int t = (int)blockIdx.x * (kThreads / W) + (int)threadIdx.x / W;
    const bool live = t < a.T;
    const bool spread = !a.sigmoid && !a.normalize;   // every expert has a gradient
    float v[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int e = u * W + l;
        v[u] = spread && live && e < a.E ? logit_of(a.logits, t * a.stride + e, BF16) : kNone;
        if (!(v[u] < __builtin_inff())) v[u] = kNone;
    }
    int e[kSlots];
    float x[kSlots], g[kSlots], peak = kNone;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int j = i * W + l;
        const int64_t id = live && j < a.k ? a.idx[(int64_t)t * a.k + j] : -1;
        if (id < -1 || id >= a.E) atomicOr(a.err, kErrBadTopk);
        e[i] = id >= 0 && id < a.E ? (int)id : -1;
        x[i] = e[i] >= 0 ? logit_of(a.logits, t * a.stride + e[i], BF16) : kNone;
        if (!(x[i] < __builtin_inff() && x[i] > kNone)) e[i] = -1;   // it cannot have been chosen
        if (e[i] < 0) x[i] = kNone;
        g[i] = e[i] >= 0 ? a.grad[(int64_t)t * a.k + j] : 0.0f;
        peak = fmaxf(peak, x[i]);
    }
    peak = over<W>(peak, Max());
    float top = kNone;
    double sum = 0.0;   // of the scores that share it
    if (spread) {
#pragma unroll
        for (int u = 0; u < PER; ++u) top = fmaxf(top, v[u]);
        top = over<W>(top, Max());
        if (!(top > kNone)) top = 0.0f;
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            v[u] = expf(v[u] - top);   // p times the sum
            sum += v[u];
        }
    }
    float r[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        if (e[i] < 0) r[i] = 0.0f;
        else if (a.sigmoid) r[i] = a.normalize && peak < 0.0f ? expf(x[i] - peak) / (1.0f + expf(x[i])) : sigmoid32(x[i]);
        else r[i] = expf(x[i] - (a.normalize ? peak : top));
        if (a.normalize) sum += r[i];
    }
    if (a.normalize || spread) {
        sum = over<W>(sum, Add());
        sum = sum > 0.0 ? inverse(sum) : 0.0;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) r[i] = (float)(r[i] * sum);
    }
    // slot j's value, for the token's lanes
    auto slot = [&](const auto (&of)[kSlots], int j) {
        if constexpr (W == 64) return lane_of(of[0], j);
        else return __shfl(j < W ? of[0] : of[kSlots - 1], (threadIdx.x & 63 & ~(W - 1)) | (j & (W - 1)), 64);
    };
    float d[kSlots], out[PER] = {};
    // d_i = start_i + sum over the slots of r_j (of_i - of_j)
    auto differences = [&](const float (&of)[kSlots], const float (&start)[kSlots]) {
        double sums[kSlots];
#pragma unroll
        for (int i = 0; i < kSlots; ++i) sums[i] = start[i];
        for (int j = 0; j < a.k; ++j) {
            const double rj = slot(r, j), oj = slot(of, j);
#pragma unroll
            for (int i = 0; i < kSlots; ++i) sums[i] = __builtin_fma(rj, of[i] - oj, sums[i]);
        }
#pragma unroll
        for (int i = 0; i < kSlots; ++i) d[i] = (float)sums[i];
    };
    if (a.normalize) {
        const float zero[kSlots] = {};
        differences(g, zero);
    } else if (spread) {
        // an expert's slots together in its first one, and the experts without any
        float own[kSlots];
        bool first[kSlots];
        uint32_t has = 0;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            own[i] = 0.0f;
            first[i] = true;
        }
        for (int j = 0; j < a.k; ++j) {
            const int ej = slot(e, j);
            const float gj = slot(g, j);
#pragma unroll
            for (int i = 0; i < kSlots; ++i)
                if (ej == e[i]) {
                    own[i] += gj;
                    first[i] = first[i] && j >= i * W + l;
                }
#pragma unroll
            for (int u = 0; u < PER; ++u) has |= (uint32_t)(u * W + l == ej) << u;
        }
        double none = 0.0, mean = 0.0;
#pragma unroll
        for (int u = 0; u < PER; ++u) none += has >> u & 1 ? 0.0f : v[u];
        none = over<W>(none, Add()) * sum;
        float start[kSlots];
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            if (!first[i]) r[i] = 0.0f;
            mean += (double)r[i] * own[i];
            start[i] = (float)(none * own[i]);
        }
        mean = over<W>(mean, Add());
        differences(own, start);
        const float rest = (float)(a.scale * mean * sum);
#pragma unroll
        for (int u = 0; u < PER; ++u) out[u] = has >> u & 1 ? 0.0f : -v[u] * rest;
    } else {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) d[i] = g[i];
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        d[i] *= a.scale * r[i];
        if (a.sigmoid && e[i] >= 0) d[i] *= sigmoid32(-x[i]);
    }
    // each slot's, from the lane that has it
    for (int j = 0; j < a.k; ++j) {
        const int ej = slot(e, j);
        const float dj = slot(d, j);
#pragma unroll
        for (int u = 0; u < PER; ++u)
            if (u * W + l == ej) out[u] += dj;
    }
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int ex = u * W + l;
        if (live && ex < a.E) a.grad_logits[(int64_t)t * a.E + ex] = out[u];
    }
}

template <class F16, class F64>
hipError_t by_experts(int E, F16 on16, F64 on64) {
    using std::integral_constant;
    if (E <= 16) return on16(integral_constant<int, 1>());
    if (E <= 64) return on16(integral_constant<int, 4>());
    if (E <= 128) return on16(integral_constant<int, 8>());
    if (E <= 256) return on16(integral_constant<int, 16>());
    if (E <= 512) return on64(integral_constant<int, 8>());
    return on64(integral_constant<int, 16>());
}

template <bool BF16, class Key>
hipError_t route(const RouteArgs& a, hipStream_t s) {
    auto go = [&](auto w, auto per) {
        constexpr int W = decltype(w)::value, tokens = kThreads / W;
        const size_t lds = sizeof(Key) == 8 && a.groups > 1 ? (size_t)tokens * a.E * sizeof(double) : 0;
        k_route<BF16, Key, W, decltype(per)::value><<<dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(kThreads), lds, s>>>(a);
        return hipGetLastError();
    };
    using std::integral_constant;
    if constexpr (sizeof(Key) == 4) {
        const integral_constant<int, 16> w;
        if (a.E <= 16) return go(w, integral_constant<int, 1>());
        if (a.E <= 64) return go(w, integral_constant<int, 4>());
        if (a.E <= 128) return go(w, integral_constant<int, 8>());
        if (a.E <= 256) return go(w, integral_constant<int, 16>());
    }
    const integral_constant<int, 64> w;
    if constexpr (sizeof(Key) == 8) {
        if (a.E <= 64) return go(w, integral_constant<int, 1>());
        if (a.E <= 128) return go(w, integral_constant<int, 2>());
        if (a.E <= 256) return go(w, integral_constant<int, 4>());
    }
    if (a.E <= 512) return go(w, integral_constant<int, 8>());
    return go(w, integral_constant<int, 16>());
}

template <bool BF16>
hipError_t route_bwd(const RouteBwdArgs& a, hipStream_t s) {
    auto go = [&](auto w, auto per) {
        constexpr int W = decltype(w)::value, PER = decltype(per)::value;
        const int tokens = kThreads / W;
        k_route_bwd<BF16, W, PER><<<dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(kThreads), 0, s>>>(a);
        return hipGetLastError();
    };
    return by_experts(a.E, [&](auto per) { return go(std::integral_constant<int, 16>(), per); },
                      [&](auto per) { return go(std::integral_constant<int, 64>(), per); });
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t s) {
    const bool scored = a.bias != nullptr || a.groups > 1;
    if (bf16) return scored ? route<true, double>(a, s) : route<true, float>(a, s);
    return scored ? route<false, double>(a, s) : route<false, float>(a, s);
}

hipError_t launch_route_bwd(const RouteBwdArgs& a, bool bf16, hipStream_t s) {
    return bf16 ? route_bwd<true>(a, s) : route_bwd<false>(a, s);
}

}  // namespace moe

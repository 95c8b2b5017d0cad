// Rotary positions of Q and K: y = amplitude * R(pos) x per head, from the model's token-major
// layout into the head-major bf16 layout of the attention calls, and the gradient
// dx = amplitude * R(pos)^T dy back. A pair (a, b) turned by the angle pos * freq becomes
// (a cos - b sin, a sin + b cos); elements past the rotated width pass through unscaled.
//
// Angles are formed in turns as 64-bit fixed point: freq / 2 pi is held as a fraction of 2^64 and
// pos times it, modulo 2^64, is the angle's fraction of a turn, of which the upper 32 bits are kept. For
// every 32-bit position the error is below 2^-32 turn (1.5e-9 rad) for that cut, and |pos| 2^-52
// max(1, |freq| / 2 pi) turns, since the quotient comes from a double division by a rounded 2 pi.
#include <math.h>
#include <string.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "sparsepr.h"

namespace spr {
namespace {

constexpr int kMaxPairs = 64;
constexpr int kThreads = 128;

struct RopeParams {
    unsigned long long turn[kMaxPairs];   // freq / 2 pi modulo 1, as a fraction of 2^64
    uint8_t axis[kMaxPairs];
    uint8_t first[kMaxPairs], second[kMaxPairs];      // the pairs' elements
    uint8_t vec_a[8], vec_b[8];           // vector kernel: a thread's two 8-element vectors
    uint8_t pair_a[8], pair_b[8];         // and the first pairs of its eight: the first four, the other four
    long long sb, sn, sh, spos;           // token-major strides; batch stride of the positions
    const int32_t* pos;
    const void* src;
    void* dst;
    int H, N, axes, pairs;
    int tokens, slots, heads;             // per block: tokens, heads at a time, heads in all
    int wide;                             // the fp32 side's vectors all start on 32 bytes
    float amplitude;
};

// The parameters by generic address, for tables indexed by the thread: the constant cache serves
// one address at a time, so a warp's 32 entries of a table would come one after another.
__device__ __forceinline__ const RopeParams* tables(const RopeParams& p) {
    const RopeParams* t = &p;
    asm volatile("" : "+l"(t));
    return t;
}

// amplitude * (cos, sin) of pair i at the token whose coordinates are `at`; sin negated for the
// transposed map.
template <bool BWD>
__device__ __forceinline__ void turn_of(const RopeParams& p, const RopeParams* tab, int i, const int32_t* at, float& cs, float& sn) {
    const uint32_t t = (uint32_t)(((unsigned long long)(long long)at[tab->axis[i]] * tab->turn[i]) >> 32);
    // nearest quarter turn q and the rest r in [-1/8, 1/8] turn, exact until its conversion to fp32
    const uint32_t q = (t + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(t - (q << 30)) * 1.4629180792671596e-9f;      // 2 pi / 2^32
    // Taylor sums on |x| <= pi / 4: the first terms left out are below 2e-9 (sin) and 3e-8 (cos)
    const float z = x * x;
    const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 40320.f, -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
    cs = (q & 1) ? s : c;
    sn = (q & 1) ? c : s;
    const float a = p.amplitude, b = BWD ? -a : a;
    cs *= ((q + 1) & 2) ? -a : a;      // cos(x + q pi / 2) = c, -s, -c, s
    sn *= (q & 2) ? -b : b;            // sin(x + q pi / 2) = s, c, -s, -c
}

// Eight consecutive elements, as loaded.
struct Raw8b { uint4 u; };
struct Raw8f { float4 a, b; };
__device__ __forceinline__ Raw8b load8(const bf16* p, bool) { return {__ldg(reinterpret_cast<const uint4*>(p))}; }
__device__ __forceinline__ Raw8f load8(const float* p, bool wide) {
    Raw8f r;
    if (wide)
        asm volatile("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(r.a.x), "=f"(r.a.y), "=f"(r.a.z), "=f"(r.a.w), "=f"(r.b.x), "=f"(r.b.y), "=f"(r.b.z), "=f"(r.b.w)
                     : "l"(p));
    else
        r = {__ldg(reinterpret_cast<const float4*>(p)), __ldg(reinterpret_cast<const float4*>(p) + 1)};
    return r;
}
__device__ __forceinline__ void widen8(const Raw8b& r, float (&v)[8]) {
    const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void widen8(const Raw8f& r, float (&v)[8]) {
    v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
    v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
__device__ __forceinline__ void store8(bf16* p, const float (&v)[8], bool) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                     "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                     : "memory");
        return;
    }
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A thread's token and first head of the block, its last head, and the addresses of both sides.
template <typename T, int D, bool BWD>
struct Walk {
    using Src = typename std::conditional<BWD, bf16, T>::type;
    using Dst = typename std::conditional<BWD, T, bf16>::type;
    const Src* src;
    Dst* dst;
    const int32_t* at;
    long long src_step, dst_step;   // per head
    int h, end;
    bool any;
    __device__ __forceinline__ Walk(const RopeParams& p, int row) {
        const int n = blockIdx.x * p.tokens + row % p.tokens, b = blockIdx.y;
        h = blockIdx.z * p.heads + row / p.tokens;
        end = min(p.H, (blockIdx.z + 1) * p.heads);
        any = n < p.N && h < end;
        const long long model = b * p.sb + n * p.sn, head = ((long long)b * p.H * p.N + n) * D;
        src = static_cast<const Src*>(p.src) + (BWD ? head : model);
        dst = static_cast<Dst*>(p.dst) + (BWD ? model : head);
        src_step = BWD ? (long long)p.N * D : p.sh;
        dst_step = BWD ? p.sh : (long long)p.N * D;
        at = p.pos + b * p.spos + (long long)n * p.axes;
    }
};

// Vector kernel: a thread holds 16 elements (two 8-element vectors, eight whole pairs) of a token's
// head and walks over the block's heads with the angles in registers. Consecutive threads hold
// consecutive vectors, so that every store fills whole 32-byte sectors. Bound by HBM: bf16 queries of
// 32760 tokens x 24 heads take 67 us (6.0 TB/s, 0.92 of the measured copy rate), the fp32 gradient
// of 75600 tokens x 8 heads 75 us (6.2 TB/s, 0.95), fp32 queries of 32760 x 24 94 us (6.4 TB/s, 0.98).
template <typename T, int D, bool HALF, bool BWD>
__global__ void __launch_bounds__(kThreads) rope_vec_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kUnits = D / 16;
    const int u = threadIdx.x % kUnits;
    Walk<T, D, BWD> w(p, threadIdx.x / kUnits);
    if (!w.any) return;
    const RopeParams* tab = tables(p);
    const int a = 8 * tab->vec_a[u], b = 8 * tab->vec_b[u], pa = tab->pair_a[u], pb = tab->pair_b[u];
    const bool wide = p.wide;
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int pair = (i < 4 ? pa : pb) + (i & 3);
        cs[i] = 1.f;
        sn[i] = 0.f;
        if (pair < p.pairs) turn_of<BWD>(p, tab, pair, w.at, cs[i], sn[i]);
    }
    // 256 bytes a thread are in flight before the first head is turned: with 128-byte batches the
    // 32760-token x 24-head case takes 68 us and the fp32 gradient below 80 us
    constexpr int kBatch = sizeof(typename Walk<T, D, BWD>::Src) == 2 ? 8 : 4;
    using Raw = decltype(load8(w.src, wide));
    for (int h0 = w.h; h0 < w.end; h0 += kBatch * p.slots) {
        Raw xr[kBatch], yr[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int h = h0 + j * p.slots;
            if (h >= w.end) break;
            xr[j] = load8(w.src + h * w.src_step + a, wide);
            yr[j] = load8(w.src + h * w.src_step + b, wide);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int h = h0 + j * p.slots;
            if (h >= w.end) break;
            float x[8], y[8];
            widen8(xr[j], x);
            widen8(yr[j], y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // pairs past the last one, where cos = 1 and sin = 0, are left as they are: 0 * inf is NaN
                if ((i < 4 ? pa : pb) + (i & 3) >= p.pairs) continue;
                float* q = HALF ? x + i : i < 4 ? x + 2 * i : y + 2 * (i - 4);
                float* r = HALF ? y + i : q + 1;
                const float v = *q;
                *q = v * cs[i] - *r * sn[i];
                *r = v * sn[i] + *r * cs[i];
            }
            store8(w.dst + h * w.dst_step + a, x, wide);
            store8(w.dst + h * w.dst_step + b, y, wide);
        }
    }
}

// Scalar kernel, for half layouts whose sections do not split into vectors: a lane holds pairs
// `lane` and `lane + 32` of a token's head, consecutive lanes consecutive elements. Each load and store moves
// one element a lane, so that there are eight times as many as the vector kernel needs for bf16 and too
// few bytes are in flight: sections of 44, 42 and 42, 32760 tokens x 24 heads, bf16 take 121 us (3.3 TB/s, 0.51 of
// the measured copy rate), their gradient 116 us.
template <typename T, int D, bool BWD>
__global__ void __launch_bounds__(kThreads) rope_scalar_kernel(const __grid_constant__ RopeParams p) {
    const int lane = threadIdx.x & 31;
    Walk<T, D, BWD> w(p, threadIdx.x >> 5);
    if (!w.any) return;
    const RopeParams* tab = tables(p);
    float cs[2], sn[2];
    int a[2], b[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = lane + 32 * j;
        cs[j] = 1.f;
        sn[j] = 0.f;
        // past the pairs: elements that pass through, two at a time
        a[j] = i < p.pairs ? tab->first[i] : 2 * i;
        b[j] = i < p.pairs ? tab->second[i] : 2 * i + 1;
        if (i < p.pairs) turn_of<BWD>(p, tab, i, w.at, cs[j], sn[j]);
    }
#pragma unroll 4
    for (int h = w.h; h < w.end; h += p.slots) {
        const auto* s = w.src + h * w.src_step;
        auto* d = w.dst + h * w.dst_step;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            const float x = (float)s[a[j]], y = (float)s[b[j]];
            const bool turned = lane + 32 * j < p.pairs;
            d[a[j]] = turned ? x * cs[j] - y * sn[j] : x;
            d[b[j]] = turned ? x * sn[j] + y * cs[j] : y;
        }
    }
}

template <typename T, int D>
void launch(RopeParams& p, int B, bool half, bool vec, bool bwd, int sms, cudaStream_t s) {
    // A block has rows of (token, head) to hand out: up to 16 or 32 (vector) or 4 (scalar) tokens;
    // with fewer tokens than that, the other rows take further heads. A block walks over as many heads
    // as leave eight blocks per SM, so that the angles of a token are formed once for all of them
    // and a few tokens still spread over the GPU (twice as many blocks: 71 us against 69 on the
    // 32760-token case, 5.2 against 4.7 us on 2 x 1001 tokens, both with blocks of 256).
    const int rows = vec ? kThreads / (D / 16) : kThreads / 32;
    p.tokens = rows;
    while (p.tokens / 2 >= p.N) p.tokens /= 2;
    p.slots = rows / p.tokens;
    const long long groups = (long long)B * ((p.N + p.tokens - 1) / p.tokens);
    long long heads = groups * p.H / (8ll * sms);
    heads = heads < 1 ? 1 : heads > p.H ? p.H : heads;
    heads = (heads + p.slots - 1) / p.slots * p.slots;
    p.heads = (int)heads;
    const dim3 grid((unsigned)((p.N + p.tokens - 1) / p.tokens), (unsigned)B, (unsigned)((p.H + heads - 1) / heads));
    if (!vec) bwd ? rope_scalar_kernel<T, D, true><<<grid, kThreads, 0, s>>>(p) : rope_scalar_kernel<T, D, false><<<grid, kThreads, 0, s>>>(p);
    else if (half) bwd ? rope_vec_kernel<T, D, true, true><<<grid, kThreads, 0, s>>>(p) : rope_vec_kernel<T, D, true, false><<<grid, kThreads, 0, s>>>(p);
    else bwd ? rope_vec_kernel<T, D, false, true><<<grid, kThreads, 0, s>>>(p) : rope_vec_kernel<T, D, false, false><<<grid, kThreads, 0, s>>>(p);
}

// Do the byte ranges [a, a + na) and [b, b + nb) meet?
bool overlap(const void* a, long long na, const void* b, long long nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

sparsepr_status rope(const sparsepr_rope_config* c, const void* src, const int32_t* pos, void* dst, bool bwd,
                     void* stream) {
    if (!c || !src || !dst || !pos) return SPARSEPR_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15u) != 0 ||
        (reinterpret_cast<uintptr_t>(pos) & 3u) != 0)
        return SPARSEPR_ERR_INVALID_ARG;
    if (c->B < 1 || c->H < 1 || c->N < 1) return SPARSEPR_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128) return SPARSEPR_ERR_UNSUPPORTED;
    if (c->layout != SPARSEPR_ROPE_INTERLEAVED && c->layout != SPARSEPR_ROPE_HALF) return SPARSEPR_ERR_INVALID_ARG;
    if (c->dtype != SPARSEPR_BF16 && c->dtype != SPARSEPR_FP32) return SPARSEPR_ERR_INVALID_ARG;
    if (c->axes < 1 || c->axes > 3 || !isfinite((float)c->amplitude)) return SPARSEPR_ERR_INVALID_ARG;
    int sum = 0;
    for (int a = 0; a < c->axes; ++a) {
        if (c->width[a] < 2 || c->width[a] % 2 != 0 || c->width[a] > c->d) return SPARSEPR_ERR_INVALID_ARG;
        sum += c->width[a];
    }
    if (sum > c->d) return SPARSEPR_ERR_INVALID_ARG;
    const int per16 = c->dtype == SPARSEPR_FP32 ? 4 : 8, size = 16 / per16;
    if (c->pos_stride_b < 0) return SPARSEPR_ERR_INVALID_ARG;
    const long long size_of[3] = {c->B, c->N, c->H}, stride_of[3] = {c->stride_b, c->stride_n, c->stride_h};
    const long long rows = (long long)c->B * c->N;
    if (c->B > 65535 || c->H > 65535 || rows > (1ll << 31) || rows * c->H > (1ll << 31)) return SPARSEPR_ERR_UNSUPPORTED;
    // every row of the token-major side starts on 16 bytes
    long long extent = c->d;
    for (int i = 0; i < 3; ++i) {
        if (size_of[i] == 1) continue;
        if (stride_of[i] < 0 || stride_of[i] % per16 != 0) return SPARSEPR_ERR_INVALID_ARG;
        if (stride_of[i] > (1ll << 40) / size_of[i]) return SPARSEPR_ERR_UNSUPPORTED;      // no sum below overflows
        extent += (size_of[i] - 1) * stride_of[i];
    }
    if (bwd) {
        // rows that are written must not overlap: taken by ascending stride, each step clears all before it
        int order[3] = {0, 1, 2};
        for (int i = 0; i < 3; ++i)
            for (int j = i + 1; j < 3; ++j)
                if (stride_of[order[j]] < stride_of[order[i]]) {
                    const int t = order[i];
                    order[i] = order[j];
                    order[j] = t;
                }
        long long span = c->d;
        for (int i = 0; i < 3; ++i) {
            const int k = order[i];
            if (size_of[k] == 1) continue;
            if (stride_of[k] < span) return SPARSEPR_ERR_INVALID_ARG;
            span += (size_of[k] - 1) * stride_of[k];
        }
    }
    const long long model = extent * size;
    const long long head = rows * c->H * c->d * 2;
    if (c->B > 1 && c->pos_stride_b > (1ll << 40) / c->B) return SPARSEPR_ERR_UNSUPPORTED;
    const long long at_bytes = 4 * ((c->B - 1) * c->pos_stride_b + (long long)c->N * c->axes);
    if (overlap(src, bwd ? head : model, dst, bwd ? model : head) || overlap(pos, at_bytes, dst, bwd ? model : head))
        return SPARSEPR_ERR_INVALID_ARG;
    RopeParams p;
    memset(&p, 0, sizeof(p));
    int at = 0;
    for (int a = 0; a < c->axes; ++a) {
        const int w = c->width[a];
        for (int i = 0; i < w / 2; ++i, ++p.pairs) {
            const double f = c->freq[p.pairs] / 6.283185307179586476925286766559;
            if (!isfinite(f)) return SPARSEPR_ERR_INVALID_ARG;
            // the fraction in two exact halves: 2^64 does not fit a double's integer conversion
            const double frac = f - floor(f), hi = floor(frac * 4294967296.0), lo = (frac * 4294967296.0 - hi) * 4294967296.0;
            p.turn[p.pairs] = ((unsigned long long)hi << 32) + (unsigned long long)lo;
            p.axis[p.pairs] = (uint8_t)a;
            p.first[p.pairs] = (uint8_t)(c->layout == SPARSEPR_ROPE_HALF ? at + i : at + 2 * i);
            p.second[p.pairs] = (uint8_t)(c->layout == SPARSEPR_ROPE_HALF ? at + w / 2 + i : at + 2 * i + 1);
        }
        at += w;
    }
    // the stride of a dimension of one is never used
    p.sb = c->B > 1 ? c->stride_b : 0; p.sn = c->N > 1 ? c->stride_n : 0; p.sh = c->H > 1 ? c->stride_h : 0;
    p.spos = c->B > 1 ? c->pos_stride_b : 0;
    p.pos = pos;
    p.src = src;
    p.dst = dst;
    p.H = c->H; p.N = c->N; p.axes = c->axes;
    p.amplitude = (float)c->amplitude;
    // The vector kernel's threads: two vectors and the pairs they hold. Interleaved pairs lie within
    // a vector; a half layout takes a vector and its partner, where every section's halves are
    // whole vectors. Vectors past the rotated width are paired likewise, without pairs.
    const bool half = c->layout == SPARSEPR_ROPE_HALF;
    bool vec = true;
    if (half) {
        int u = 0, start = 0, pair = 0;
        for (int a = 0; a < c->axes; ++a) {
            const int w = c->width[a];
            if (w % 16 != 0) vec = false;
            for (int i = 0; vec && i < w / 16; ++i, ++u, pair += 8) {
                p.vec_a[u] = (uint8_t)(start / 8 + i);
                p.vec_b[u] = (uint8_t)(start / 8 + w / 16 + i);
                p.pair_a[u] = (uint8_t)pair;
                p.pair_b[u] = (uint8_t)(pair + 4);
            }
            start += w;
        }
        for (int i = 0, rest = (c->d - start) / 16; vec && i < rest; ++i, ++u) {
            p.vec_a[u] = (uint8_t)(start / 8 + i);
            p.vec_b[u] = (uint8_t)(start / 8 + rest + i);
            p.pair_a[u] = p.pair_b[u] = kMaxPairs;
        }
    } else {
        for (int u = 0; u < c->d / 16; ++u) {
            p.vec_a[u] = (uint8_t)u;
            p.vec_b[u] = (uint8_t)(c->d / 16 + u);
            p.pair_a[u] = (uint8_t)(4 * u);
            p.pair_b[u] = (uint8_t)(4 * (c->d / 16 + u));
        }
    }
    const void* model_side = bwd ? dst : src;
    p.wide = (reinterpret_cast<uintptr_t>(model_side) & 31u) == 0 && p.sb % 8 == 0 && p.sn % 8 == 0 && p.sh % 8 == 0;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return SPARSEPR_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f32 = c->dtype == SPARSEPR_FP32;
    if (c->d == 128) f32 ? launch<float, 128>(p, c->B, half, vec, bwd, sms, s) : launch<bf16, 128>(p, c->B, half, vec, bwd, sms, s);
    else f32 ? launch<float, 64>(p, c->B, half, vec, bwd, sms, s) : launch<bf16, 64>(p, c->B, half, vec, bwd, sms, s);
    return cudaGetLastError() == cudaSuccess ? SPARSEPR_OK : SPARSEPR_ERR_CUDA;
}

}  // namespace
}  // namespace spr

extern "C" {

sparsepr_status sparsepr_rope(const sparsepr_rope_config* cfg, const void* X, const int32_t* pos, void* Y, void* stream) {
    return spr::rope(cfg, X, pos, Y, false, stream);
}

sparsepr_status sparsepr_rope_bwd(const sparsepr_rope_config* cfg, const void* dY, const int32_t* pos, void* dX,
                                  void* stream) {
    return spr::rope(cfg, dY, pos, dX, true, stream);
}

}  // extern "C"

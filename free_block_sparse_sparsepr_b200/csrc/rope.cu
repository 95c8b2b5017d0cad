// Rotary positions of Q and K: y = amplitude * R(pos) x per head, from the model's token-major
// layout into the head-major bf16 layout of the attention calls, and the gradient
// dx = amplitude * R(pos)^T dy back. A pair (a, b) turned by the angle pos * freq becomes
// (a cos - b sin, a sin + b cos); elements past the rotated width pass through unscaled.
//
// Angles are formed in turns as 64-bit fixed point: freq / 2 pi is held as a fraction of 2^64, so
// pos times it, modulo 2^64, is the angle's fraction of a turn with an error below
// |pos| 2^-53 turns (the fraction comes from a double), for every 32-bit position.
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "kernels.h"
#include "sparsepr.h"

namespace spr {
namespace {

constexpr int kMaxPairs = 64;

struct RopeParams {
    unsigned long long turn[kMaxPairs];   // freq / 2 pi modulo 1, as a fraction of 2^64
    uint8_t axis[kMaxPairs], first[kMaxPairs], second[kMaxPairs];
    long long sb, sn, sh, spos;           // token-major strides; batch stride of the positions
    const int32_t* pos;
    int H, N, axes, pairs;
    float amplitude;
};

// One warp per (b, n, h) row.
template <typename T, int D, bool BWD>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p, const void* src_, void* dst_, long long rows) {
    const long long r = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (r >= rows) return;
    const int h = (int)(r % p.H);
    const long long bn = r / p.H;
    const int n = (int)(bn % p.N), b = (int)(bn / p.N);
    const long long model = b * p.sb + n * p.sn + h * p.sh, head = (((long long)b * p.H + h) * p.N + n) * D;
    auto load = [&](int e) {
        if (BWD) return bf16_to_f32(static_cast<const bf16*>(src_)[head + e]);
        return (float)static_cast<const T*>(src_)[model + e];
    };
    auto store = [&](int e, float v) {
        if (BWD) static_cast<T*>(dst_)[model + e] = (T)v;
        else static_cast<bf16*>(dst_)[head + e] = __float2bfloat16_rn(v);
    };
    for (int i = lane; i < p.pairs; i += 32) {
        const int32_t at = p.pos[b * p.spos + (long long)n * p.axes + p.axis[i]];
        const long long turns = (long long)((unsigned long long)(long long)at * p.turn[i]);
        float sn, cs;
        sincospif((float)(int32_t)(turns >> 32) * 4.656612873077393e-10f, &sn, &cs);   // 2^-31: half turns
        if (BWD) sn = -sn;
        const float u = load(p.first[i]), v = load(p.second[i]);
        store(p.first[i], p.amplitude * (u * cs - v * sn));
        store(p.second[i], p.amplitude * (u * sn + v * cs));
    }
    for (int e = 2 * p.pairs + lane; e < D; e += 32) store(e, load(e));
}

template <typename T, int D>
void launch(const RopeParams& p, const void* src, void* dst, long long rows, bool bwd, cudaStream_t s) {
    const unsigned blocks = (unsigned)((rows * 32 + 255) / 256);
    if (bwd) rope_kernel<T, D, true><<<blocks, 256, 0, s>>>(p, src, dst, rows);
    else rope_kernel<T, D, false><<<blocks, 256, 0, s>>>(p, src, dst, rows);
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
    if (c->axes < 1 || c->axes > 3 || !isfinite(c->amplitude)) return SPARSEPR_ERR_INVALID_ARG;
    int sum = 0;
    for (int a = 0; a < c->axes; ++a) {
        if (c->width[a] < 2 || c->width[a] % 2 != 0 || c->width[a] > c->d) return SPARSEPR_ERR_INVALID_ARG;
        sum += c->width[a];
    }
    if (sum > c->d) return SPARSEPR_ERR_INVALID_ARG;
    const int vec = c->dtype == SPARSEPR_FP32 ? 4 : 8, size = 16 / vec;
    if (c->pos_stride_b < 0) return SPARSEPR_ERR_INVALID_ARG;
    const long long size_of[3] = {c->B, c->N, c->H}, stride_of[3] = {c->stride_b, c->stride_n, c->stride_h};
    const long long rows = (long long)c->B * c->N;
    if (rows > (1ll << 31) || rows * c->H > (1ll << 31)) return SPARSEPR_ERR_UNSUPPORTED;
    // every row of the token-major side starts on 16 bytes
    long long extent = c->d;
    for (int i = 0; i < 3; ++i) {
        if (size_of[i] == 1) continue;
        if (stride_of[i] < 0 || stride_of[i] % vec != 0) return SPARSEPR_ERR_INVALID_ARG;
        if (stride_of[i] > (1ll << 40)) return SPARSEPR_ERR_UNSUPPORTED;
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
    if (overlap(src, bwd ? head : model, dst, bwd ? model : head)) return SPARSEPR_ERR_INVALID_ARG;
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
    p.H = c->H; p.N = c->N; p.axes = c->axes;
    p.amplitude = (float)c->amplitude;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long n = rows * c->H;
    const bool f32 = c->dtype == SPARSEPR_FP32;
    if (c->d == 128) f32 ? launch<float, 128>(p, src, dst, n, bwd, s) : launch<bf16, 128>(p, src, dst, n, bwd, s);
    else f32 ? launch<float, 64>(p, src, dst, n, bwd, s) : launch<bf16, 64>(p, src, dst, n, bwd, s);
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

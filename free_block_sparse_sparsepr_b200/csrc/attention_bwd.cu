// Backward passes of the attention steps: gradients of O = softmax(Q K^T / sqrt(d)) V over all keys
// (dense) or over each query group's kept key groups (block-sparse), from the forward pass's
// inputs, output and lse. With s = q.k / sqrt(d) and the probabilities recomputed, for every kept
// pair (i, j):
//   P_ij = exp(s_ij - lse_i),  D_i = dO_i . O_i,  dS_ij = P_ij (dO_i . v_j - D_i),
//   dV_j = sum_i P_ij dO_i,  dK_j = sum_i dS_ij q_i / sqrt(d),  dQ_i = sum_j dS_ij k_j / sqrt(d);
// dK and dV also sum over the query heads that share the KV head. Each gradient row is summed by
// one owner in a fixed order (no atomics), so results repeat bit for bit.
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "kernels.h"

namespace spr {
namespace {

constexpr int kTile = 128;                  // rows per query or key tile
constexpr float kLog2e = 1.4426950408889634f;

struct BwdParams {
    const bf16 *Q, *K, *V;
    const bf16* dO;
    const float *nlse2, *nD;                // per query row: -lse log2(e), -dO.O
    bf16 *dQ, *dK, *dV;
    const int32_t *qperm, *kperm;           // output row of each position (null: the position itself)
    const int32_t *qoff, *koff;             // group offsets (null: one group of N rows)
    const int2 *klist, *qlist;              // kept key tiles of each query group, query tiles of each key group
    const int32_t *kcnt, *qcnt;             // their numbers
    int kcap, qcap;                         // list entries per group
    int* status;
    int N, g, Gq, Gk;
    float scale, scale_log2;
};

// ---------------------------------------------------------------- per-row terms
// D_i = dO_i . O_i and -lse_i log2(e), negated as the kernels add them. One 16-byte vector of a
// row per thread, D / 8 threads a row.
template <int D>
__global__ void __launch_bounds__(256) bwd_rows_kernel(const uint4* __restrict__ O, const uint4* __restrict__ dO,
                                                       const float* __restrict__ lse, float* __restrict__ nlse2,
                                                       float* __restrict__ nD, long long rows) {
    constexpr int kV = D / 8;
    const long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long row = t / kV;
    float s = 0.f;
    if (row < rows) {
        const uint4 a = __ldg(O + t), b = __ldg(dO + t);
        const uint32_t *x = &a.x, *y = &b.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 u = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(x + i));
            const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(y + i));
            s = fmaf(u.x, v.x, fmaf(u.y, v.y, s));
        }
    }
#pragma unroll
    for (int o = kV / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    if (row < rows && t % kV == 0) {
        nD[row] = -s;
        nlse2[row] = lse[row] == -INFINITY ? -INFINITY : -lse[row] * kLog2e;   // an empty row: P = 0
    }
}

// ---------------------------------------------------------------- tile lists
// One warp per (KV head z, group): the tiles (start row, valid rows <= 128) of the other side's
// groups that the route pairs with it, runs of touching groups merged. Warps [0, P Gq) walk their
// route row; warps from P Gq on collect the rows that hold their key group (binary search, the
// kept ids ascend). Ids and offsets out of range are skipped and reported in the status word, so
// the lists stay inside [0, N).
__global__ void __launch_bounds__(256) bwd_lists_kernel(const int32_t* __restrict__ rowptr,
                                                        const int32_t* __restrict__ kg,
                                                        const int32_t* __restrict__ qoff,
                                                        const int32_t* __restrict__ koff, int2* klist, int32_t* kcnt,
                                                        int2* qlist, int32_t* qcnt, int kcap, int qcap, int P, int N,
                                                        int Gq, int Gk, int* status) {
    const int wid = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (wid >= P * (Gq + Gk)) return;
    const bool rows = wid < P * Gq;
    const int z = rows ? wid / Gq : (wid - P * Gq) / Gk;
    const int own = rows ? wid % Gq : (wid - P * Gq) % Gk;
    const int32_t* rp = rowptr + (long long)z * (Gq + 1);
    const int32_t* kept = kg + (long long)z * Gq * Gk;
    const int32_t* off = rows ? koff + (long long)z * (Gk + 1) : qoff + (long long)z * (Gq + 1);
    const int cap = rows ? kcap : qcap;
    int2* out = (rows ? klist + ((long long)z * Gq + own) * cap : qlist + ((long long)z * Gk + own) * cap);
    bool bad = false;
    // the bounds of route row a, empty if they are no range of the kept list
    auto row_range = [&](int a) {
        int2 r = make_int2(rp[a], rp[a + 1]);
        if (r.x < 0 || r.y < r.x || r.y > Gq * Gk) {
            bad = true;
            r = make_int2(0, 0);
        }
        return r;
    };
    int nt = 0, cur_lo = 0, cur_hi = 0;
    auto emit = [&]() {
        const int n = (cur_hi - cur_lo + kTile - 1) / kTile;
        if (nt + n > cap) {     // more tiles than disjoint groups can have
            bad = true;
            return;
        }
        for (int t = lane; t < n; t += 32)
            out[nt + t] = make_int2(cur_lo + t * kTile, min(kTile, cur_hi - cur_lo - t * kTile));
        nt += n;
    };
    const int2 own_row = rows ? row_range(own) : make_int2(0, Gq);
    for (int c0 = own_row.x; c0 < own_row.y; c0 += 32) {
        const int c = c0 + lane;
        int lo = 0, hi = 0;
        if (c < own_row.y) {
            int grp = -1;
            if (rows) {
                grp = kept[c];
                if (grp < 0 || grp >= Gk) {
                    bad = true;
                    grp = -1;
                }
            } else {
                const int2 r = row_range(c);
                int b = r.x, e = r.y;
                while (b < e) {
                    const int m = (b + e) >> 1;
                    if (kept[m] < own) b = m + 1; else e = m;
                }
                if (b < r.y && kept[b] == own) grp = c;
            }
            if (grp >= 0) {
                lo = off[grp];
                hi = off[grp + 1];
                if (lo < 0 || hi < lo || hi > N) {
                    bad = true;
                    lo = hi = 0;
                }
            }
        }
        unsigned todo = __ballot_sync(kFull, hi > lo);
        while (todo) {
            const int i = __ffs(todo) - 1;
            todo &= todo - 1;
            const int l = __shfl_sync(kFull, lo, i), h = __shfl_sync(kFull, hi, i);
            if (l != cur_hi) {
                emit();
                cur_lo = l;
            }
            cur_hi = h;
        }
    }
    emit();
    if (lane == 0) (rows ? kcnt + (long long)z * Gq : qcnt + (long long)z * Gk)[own] = nt;
    if (__any_sync(kFull, bad) && lane == 0) set_status(status, kDevBounds);
}

// ---------------------------------------------------------------- gradients
// Group and list of position `pos`.
__device__ __forceinline__ int group_of(const int32_t* off, int z, int G, int pos) {
    return off ? upper_index(off + (long long)z * (G + 1), G, pos) : 0;
}

template <int D>
__device__ __forceinline__ void load_row(const bf16* p, int lane, float (&r)[D / 32]) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) r[i] = bf16_to_f32(p[lane + 32 * i]);
}

template <int D>
__device__ __forceinline__ float dot_row(const float (&a)[D / 32], const float (&b)[D / 32]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) s = fmaf(a[i], b[i], s);
    return warp_sum(s);
}

template <int D>
__device__ __forceinline__ void store_row(bf16* base, const int32_t* perm, int N, int pos, int lane,
                                          const float (&r)[D / 32], int* status) {
    const int row = perm ? perm[pos] : pos;
    if (row < 0 || row >= N) {
        if (lane == 0) set_status(status, kDevBounds);
        return;
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) base[(long long)row * D + lane + 32 * i] = __float2bfloat16_rn(r[i]);
}

// One warp per query row, over its group's key tiles.
template <int D>
__global__ void __launch_bounds__(256) bwd_dq_kernel(const BwdParams p) {
    const int lane = threadIdx.x & 31, pos = blockIdx.x * 8 + (threadIdx.x >> 5), x = blockIdx.y, z = x / p.g;
    if (pos >= p.N) return;
    const long long row = (long long)x * p.N + pos;
    const int a = group_of(p.qoff, z, p.Gq, pos);
    const int2* list = p.klist + ((long long)z * p.Gq + a) * p.kcap;
    const int nt = p.kcnt ? p.kcnt[(long long)z * p.Gq + a] : (p.N + kTile - 1) / kTile;
    float q[D / 32], o[D / 32], acc[D / 32] = {};
    load_row<D>(p.Q + row * D, lane, q);
    load_row<D>(p.dO + row * D, lane, o);
    const float nl = p.nlse2[row], nd = p.nD[row];
    for (int t = 0; t < nt; ++t) {
        const int2 e = p.kcnt ? list[t] : make_int2(t * kTile, min(kTile, p.N - t * kTile));
        for (int j = e.x; j < e.x + e.y; ++j) {
            float k[D / 32], v[D / 32];
            load_row<D>(p.K + ((long long)z * p.N + j) * D, lane, k);
            load_row<D>(p.V + ((long long)z * p.N + j) * D, lane, v);
            const float P = exp2f(fmaf(dot_row<D>(q, k), p.scale_log2, nl));
            const float dS = P * (dot_row<D>(o, v) + nd);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) acc[i] = fmaf(dS, k[i], acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] *= p.scale;
    store_row<D>(p.dQ + (long long)x * p.N * D, p.qperm ? p.qperm + (long long)z * p.N : nullptr, p.N, pos, lane, acc,
                 p.status);
}

// One warp per key row, over its group's query tiles of every query head of the KV head.
template <int D>
__global__ void __launch_bounds__(256) bwd_dkv_kernel(const BwdParams p) {
    const int lane = threadIdx.x & 31, pos = blockIdx.x * 8 + (threadIdx.x >> 5), z = blockIdx.y;
    if (pos >= p.N) return;
    const long long row = (long long)z * p.N + pos;
    const int a = group_of(p.koff, z, p.Gk, pos);
    const int2* list = p.qlist + ((long long)z * p.Gk + a) * p.qcap;
    const int nt = p.qcnt ? p.qcnt[(long long)z * p.Gk + a] : (p.N + kTile - 1) / kTile;
    float k[D / 32], v[D / 32], dk[D / 32] = {}, dv[D / 32] = {};
    load_row<D>(p.K + row * D, lane, k);
    load_row<D>(p.V + row * D, lane, v);
    for (int x = z * p.g; x < (z + 1) * p.g; ++x)
        for (int t = 0; t < nt; ++t) {
            const int2 e = p.qcnt ? list[t] : make_int2(t * kTile, min(kTile, p.N - t * kTile));
            for (int i = e.x; i < e.x + e.y; ++i) {
                const long long r = (long long)x * p.N + i;
                float q[D / 32], o[D / 32];
                load_row<D>(p.Q + r * D, lane, q);
                load_row<D>(p.dO + r * D, lane, o);
                const float P = exp2f(fmaf(dot_row<D>(q, k), p.scale_log2, p.nlse2[r]));
                const float dS = P * (dot_row<D>(o, v) + p.nD[r]);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    dv[c] = fmaf(P, o[c], dv[c]);
                    dk[c] = fmaf(dS, q[c], dk[c]);
                }
            }
        }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) dk[c] *= p.scale;
    const int32_t* perm = p.kperm ? p.kperm + (long long)z * p.N : nullptr;
    store_row<D>(p.dK + (long long)z * p.N * D, perm, p.N, pos, lane, dk, p.status);
    store_row<D>(p.dV + (long long)z * p.N * D, perm, p.N, pos, lane, dv, p.status);
}

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

// Byte offsets of the workspace's parts.
struct BwdLayout {
    size_t nlse2, nD, klist, qlist, kcnt, qcnt, bytes;
    int kcap, qcap;
};

BwdLayout bwd_layout(int P, int g, int N, int d, int Gq, int Gk, bool sparse) {
    BwdLayout l;
    memset(&l, 0, sizeof(l));
    size_t at = 0;
    auto take = [&](size_t b) {
        const size_t o = at;
        at += align256(b);
        return o;
    };
    const size_t rows = (size_t)P * g * N * sizeof(float), tiles = (size_t)((N + kTile - 1) / kTile);
    l.nlse2 = take(rows);
    l.nD = take(rows);
    if (sparse) {
        // the runs of a list are disjoint: at most N / 128 full tiles and one ragged tile per group
        l.kcap = (int)(tiles + Gk);
        l.qcap = (int)(tiles + Gq);
        l.klist = take((size_t)P * Gq * l.kcap * sizeof(int2));
        l.qlist = take((size_t)P * Gk * l.qcap * sizeof(int2));
        l.kcnt = take((size_t)P * Gq * sizeof(int32_t));
        l.qcnt = take((size_t)P * Gk * sizeof(int32_t));
    }
    l.bytes = at;
    return l;
}

template <int D>
cudaError_t launch_bwd(const AttnBwdArgs& a, cudaStream_t s) {
    const bool sparse = a.rowptr != nullptr;
    const BwdLayout l = bwd_layout(a.P, a.g, a.N, D, a.Gq, a.Gk, sparse);
    char* ws = static_cast<char*>(a.workspace);
    float *nlse2 = reinterpret_cast<float*>(ws + l.nlse2), *nD = reinterpret_cast<float*>(ws + l.nD);
    const long long rows = (long long)a.P * a.g * a.N;
    bwd_rows_kernel<D><<<(unsigned)((rows * (D / 8) + 255) / 256), 256, 0, s>>>(
        reinterpret_cast<const uint4*>(a.O), reinterpret_cast<const uint4*>(a.dO), a.lse, nlse2, nD, rows);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    BwdParams p;
    memset(&p, 0, sizeof(p));
    p.Q = a.Q; p.K = a.K; p.V = a.V; p.dO = a.dO;
    p.nlse2 = nlse2; p.nD = nD;
    p.dQ = a.dQ; p.dK = a.dK; p.dV = a.dV;
    p.N = a.N; p.g = a.g; p.Gq = 1; p.Gk = 1;
    p.status = a.status;
    p.scale = (float)(1.0 / sqrt((double)D));
    p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
    if (sparse) {
        int2 *klist = reinterpret_cast<int2*>(ws + l.klist), *qlist = reinterpret_cast<int2*>(ws + l.qlist);
        int32_t *kcnt = reinterpret_cast<int32_t*>(ws + l.kcnt), *qcnt = reinterpret_cast<int32_t*>(ws + l.qcnt);
        const long long warps = (long long)a.P * (a.Gq + a.Gk);
        bwd_lists_kernel<<<(unsigned)((warps * 32 + 255) / 256), 256, 0, s>>>(
            a.rowptr, a.kg, a.qoff, a.koff, klist, kcnt, qlist, qcnt, l.kcap, l.qcap, a.P, a.N, a.Gq, a.Gk, a.status);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        p.qoff = a.qoff; p.koff = a.koff; p.qperm = a.qperm; p.kperm = a.kperm;
        p.klist = klist; p.qlist = qlist; p.kcnt = kcnt; p.qcnt = qcnt;
        p.kcap = l.kcap; p.qcap = l.qcap;
        p.Gq = a.Gq; p.Gk = a.Gk;
    }
    const unsigned blocks = (unsigned)((a.N + 7) / 8);
    if (a.dQ) {
        bwd_dq_kernel<D><<<dim3(blocks, a.P * a.g), 256, 0, s>>>(p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (a.dK) bwd_dkv_kernel<D><<<dim3(blocks, a.P), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t attn_bwd_workspace(int P, int g, int N, int d, int Gq, int Gk, bool sparse) {
    return bwd_layout(P, g, N, d, Gq, Gk, sparse).bytes;
}

int attn_bwd_launches(const AttnBwdArgs& a) { return 1 + (a.rowptr != nullptr) + (a.dQ != nullptr) + (a.dK != nullptr); }

cudaError_t launch_attn_bwd(const AttnBwdArgs& a, cudaStream_t s) {
    return a.d == 128 ? launch_bwd<128>(a, s) : a.d == 64 ? launch_bwd<64>(a, s) : cudaErrorInvalidValue;
}

}  // namespace spr

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
#include "tc_primitives.cuh"
#include "tmap.h"

namespace spr {
namespace {

constexpr int kTile = 128;                  // rows per query or key tile
constexpr float kLog2e = 1.4426950408889634f;

struct BwdParams {
    const float *nlse2, *nD;                // per query row: -lse log2(e), -dO.O
    bf16 *dQ, *dK, *dV;
    const int32_t *qperm, *kperm;           // output row of each position (null: the position itself)
    const int32_t *qoff, *koff;             // group offsets (null: one group of N rows)
    const int2 *klist, *qlist;              // kept key tiles of each query group, query tiles of each key group
    const int32_t *kcnt, *qcnt;             // their numbers
    const int32_t *qtile_off, *ktile_off;   // [P][G + 1] 128-row tiles before each group
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
// route row; the next P Gk collect the rows that hold their key group (binary search, the kept ids
// ascend); the last 2 P sum up the tiles of each side's own groups. Ids and offsets out of range
// are skipped and reported in the status word, so every tile stays inside [0, N).
__global__ void __launch_bounds__(256) bwd_lists_kernel(const int32_t* __restrict__ rowptr,
                                                        const int32_t* __restrict__ kg,
                                                        const int32_t* __restrict__ qoff,
                                                        const int32_t* __restrict__ koff, int2* klist, int32_t* kcnt,
                                                        int2* qlist, int32_t* qcnt, int32_t* qtile_off,
                                                        int32_t* ktile_off, int kcap, int qcap, int P, int N, int Gq,
                                                        int Gk, int* status) {
    const int wid = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (wid >= P * (Gq + Gk)) {
        const int i = wid - P * (Gq + Gk), z = i >> 1, G = (i & 1) ? Gk : Gq;
        if (z >= P) return;
        const int32_t* off = (i & 1) ? koff + (long long)z * (Gk + 1) : qoff + (long long)z * (Gq + 1);
        int32_t* out = (i & 1) ? ktile_off + (long long)z * (Gk + 1) : qtile_off + (long long)z * (Gq + 1);
        bool bad = false;
        int before = 0;
        for (int g0 = 0; g0 < G; g0 += 32) {
            int n = 0;
            if (g0 + lane < G) {
                const int lo = off[g0 + lane], hi = off[g0 + lane + 1];
                if (lo < 0 || hi < lo || hi > N) bad = true;
                else n = (hi - lo + kTile - 1) / kTile;
            }
            int sum = n;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, sum, o);
                if (lane >= o) sum += v;
            }
            if (g0 + lane < G) out[g0 + lane] = before + sum - n;
            before += __shfl_sync(kFull, sum, 31);
        }
        if (lane == 0) out[G] = before;
        if (__any_sync(kFull, bad) && lane == 0) set_status(status, kDevBounds);
        return;
    }
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
// Both kernels run ten warps: two warpgroups that form P and dS (thread r of warpgroup w owns TMEM
// lane r of columns 64 w .. 64 w + 63), warp 8 loads tiles (TMA), warp 9 allocates TMEM and issues
// every MMA. P and dS go back to TMEM as bf16 pairs over the fp32 columns they were formed from
// (warpgroup w at column 64 w) and are the A operands of the next product, so no transposed copy is
// ever made: the dK/dV kernel keeps keys in the lanes (S^T = K Q^T), the dQ kernel queries.
// Rows of a streamed tile past its valid ones belong to another group or head: the loading warp
// zeroes them in shared memory, so that no value there, finite or not, reaches a sum.
constexpr int kRegion = 16384;              // one [128 rows][64 bf16] region, 128-byte swizzle
constexpr int kThreads = 320;
constexpr uint32_t kTmemCols = 512;

// Set-up shared by the kernels: aligned shared memory, barriers, TMEM.
struct Cta {
    uint32_t base, bars, tmem;
    unsigned char* sbase;
    volatile int* abort_flag;
    int warp, lane;
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * (uint32_t)i; }
};

__device__ __forceinline__ Cta cta_setup(unsigned char* smem_raw, int off_bar, const int* counts, int nbars) {
    Cta c;
    const uint32_t raw = tc::smem_addr(smem_raw);
    c.base = (raw + 1023u) & ~1023u;
    c.sbase = smem_raw + (c.base - raw);
    c.bars = c.base + off_bar;
    c.warp = threadIdx.x >> 5;
    c.lane = threadIdx.x & 31;
    uint32_t* slot = reinterpret_cast<uint32_t*>(c.sbase + off_bar + 8 * nbars);
    c.abort_flag = reinterpret_cast<volatile int*>(slot + 1);
    if (threadIdx.x == 0) {
        for (int i = 0; i < nbars; ++i) tc::mbar_init(c.bar(i), counts[i]);
        *c.abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (c.warp == 9) {
        tc::tmem_alloc(tc::smem_addr(slot), kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    c.tmem = *slot;
    return c;
}

// Releases TMEM and reports a wait that gave up; every thread of the CTA calls it last.
__device__ __forceinline__ void cta_finish(const Cta& c, int* status) {
    tc::fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && *c.abort_flag) set_status(status, kDevTimeout);
    if (c.warp == 9) {
        tc::fence_after_sync();
        tc::tmem_dealloc(c.tmem, kTmemCols);
    }
}

// D[tmem] = A B^T over D columns of two swizzled tiles (both K-major).
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint32_t a, uint32_t b) {
    constexpr uint32_t id = tc::idesc_bf16_f32(kTile, kTile, 0);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (uint32_t)((k >> 2) * kRegion + (k & 3) * 32);
        tc::mma_f16_ss(d_tmem, tc::smem_desc_sw128(a + off, 16, 1024), tc::smem_desc_sw128(b + off, 16, 1024), id,
                       k > 0 ? 1u : 0u);
    }
}

// D[tmem] (+)= A B over the 128 rows of tile b (MN-major); A is bf16 pairs in TMEM, its columns
// 64..127 packed from column a_tmem + 64.
template <int D>
__device__ __forceinline__ void mma_sums(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, bool accumulate) {
    constexpr uint32_t id = tc::idesc_bf16_f32(kTile, D, 1);
#pragma unroll
    for (int k = 0; k < kTile / 16; ++k)
        tc::mma_f16_ts(d_tmem, a_tmem + (uint32_t)(64 * (k >> 2) + 8 * (k & 3)),
                       tc::smem_desc_sw128(b + (uint32_t)(k * 2048), kRegion, 1024), id, (accumulate || k > 0) ? 1u : 0u);
}

template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int row) {
    tc::mbar_arrive_expect_tx(bar, D / 64 * kRegion);
#pragma unroll
    for (int h = 0; h < D / 64; ++h) tc::tma_load_2d(dst + h * kRegion, map, bar, 64 * h, row);
}

// The loading warp's tile of rows [row, row + 128), `valid` of them kept, completing `full`. A
// ragged tile lands on `land` first (its phase in `nland`); the warp then zeroes the other rows.
template <int D>
__device__ __forceinline__ bool load_tile_zeroed(const Cta& c, uint32_t dst, const CUtensorMap* map, int full, int land,
                                                 int& nland, int row, int valid) {
    if (valid >= kTile) {
        if (c.lane == 0) load_tile<D>(dst, map, c.bar(full), row);
        __syncwarp();
        return true;
    }
    if (c.lane == 0) load_tile<D>(dst, map, c.bar(land), row);
    __syncwarp();
    int never = 0;      // the copy is in flight and completes: an abort elsewhere does not end this wait
    const bool ok = __all_sync(kFull, tc::mbar_wait(c.bar(land), nland & 1, &never));
    ++nland;
    if (!ok) return false;
    uint4* p = reinterpret_cast<uint4*>(c.sbase + (dst - c.base));
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
        for (int i = valid * 8 + c.lane; i < kTile * 8; i += 32) p[h * (kRegion / 16) + i] = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (c.lane == 0) tc::mbar_arrive(c.bar(full));
    return true;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Pairs of fp32 in one 64-bit register (packed f32x2 arithmetic).
__device__ __forceinline__ uint64_t pk2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void up2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
}

// One fp32 accumulator row of D TMEM columns, times `scale`, rounded to bf16 into `out`.
template <int D>
__device__ __forceinline__ void store_acc_row(uint32_t tacc, float scale, bf16* out, bool zero) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        tc::tmem_ld32(tacc + 32 * c, v);
        tc::tmem_wait_ld();
        tc::regs_after_wait(v);
        if (!out) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = zero ? 0u
                            : bf16x2(__uint_as_float(v[8 * q + 2 * e]) * scale, __uint_as_float(v[8 * q + 2 * e + 1]) * scale);
            *reinterpret_cast<uint4*>(out + 32 * c + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Output row of position `pos` (null: out of range, reported, or not wanted).
template <int D>
__device__ __forceinline__ bf16* out_row(bf16* base, const int32_t* perm, long long head, int N, int pos, bool want,
                                         long long perm_head, int* status) {
    if (!want) return nullptr;
    const int row = perm ? perm[perm_head * N + pos] : pos;
    if (row < 0 || row >= N) {
        set_status(status, kDevBounds);
        return nullptr;
    }
    return base + (head * N + row) * D;
}

// The tile of CTA `pair` on one side: rows [lo, lo + n) of group `grp`; false past the last tile.
__device__ __forceinline__ bool find_tile(const int32_t* off, const int32_t* tile_off, int z, int G, int N, int pair,
                                          int& grp, int& lo, int& n) {
    grp = 0;
    if (!off) {
        lo = pair * kTile;
        n = min(kTile, N - lo);
        return true;
    }
    const int32_t* toff = tile_off + (long long)z * (G + 1);
    if (pair >= toff[G]) return false;
    grp = upper_index(toff, G, pair);
    const int32_t* o = off + (long long)z * (G + 1);
    lo = o[grp] + (pair - toff[grp]) * kTile;
    n = min(kTile, o[grp + 1] - lo);
    return true;
}

// ---------------------------------------------------------------- dK and dV
// One CTA per 128-key tile, streaming the (Q, dO) tiles of every query head of the KV head and
// every query tile that keeps the key group. Per tile, with keys in the TMEM lanes:
//   S^T = K Q^T -> P^T (over S^T);  dV += P^T dO;  dP^T = V dO^T -> dS^T (over dP^T);  dK += dS^T Q.
// Issue order dV(i), S(i+1), dK(i), dP(i+1): the exponentials of tile i + 1 run beside dK(i) and
// dP(i+1), dS(i) beside dV(i) and S(i+1).
namespace kv {
constexpr int kStages = 2;
constexpr int kOffK = 0, kOffV = 2 * kRegion, kOffQ = 4 * kRegion, kOffO = kOffQ + kStages * 2 * kRegion,
              kOffRows = kOffO + kStages * 2 * kRegion;         // per warp: 2 buffers of 64 -lse and 64 -D
constexpr int kOffBar = kOffRows + 8 * 2 * 128 * 4;
enum { kKV = 0, kQf = 1, kOf = kQf + kStages, kQe = kOf + kStages, kOe = kQe + kStages, kS = kOe + kStages, kP = kS + 1,
       kDP = kP + 1, kDS = kDP + 1, kDone = kDS + 1, kLand = kDone + 1, kBars = kLand + 1 };
constexpr int kSmem = kOffBar + 8 * kBars + 16 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr uint32_t kTS = 0, kTDP = 128, kTDV = 256, kTDK = 384;
}  // namespace kv

template <int D>
__global__ void __launch_bounds__(kThreads, 1) bwd_dkv_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                              const __grid_constant__ CUtensorMap tmK,
                                                              const __grid_constant__ CUtensorMap tmV,
                                                              const __grid_constant__ CUtensorMap tmO,
                                                              const BwdParams p) {
    using namespace kv;
    extern __shared__ unsigned char smem_raw[];
    if (p.status && *reinterpret_cast<volatile int*>(p.status) == kDevTimeout) return;
    const int z = blockIdx.y;
    int grp, klo, kn;
    if (!find_tile(p.koff, p.ktile_off, z, p.Gk, p.N, blockIdx.x, grp, klo, kn)) return;
    const int2* list = p.qlist + ((long long)z * p.Gk + grp) * p.qcap;
    const int nt = p.qcnt ? p.qcnt[(long long)z * p.Gk + grp] : (p.N + kTile - 1) / kTile;
    const int iters = nt * p.g;
    // tile `it`: head, first row and valid rows
    auto tile = [&](int t) { return p.qcnt ? list[t] : make_int2(t * kTile, min(kTile, p.N - t * kTile)); };
    const int counts[kBars] = {1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 256, 1, 256, 1, 1};
    const Cta c = cta_setup(smem_raw, kOffBar, counts, kBars);

    if (c.warp == 8) {
        if (c.lane == 0) {
            tc::mbar_arrive_expect_tx(c.bar(kKV), 2 * (D / 64) * kRegion);
            for (int h = 0; h < D / 64; ++h) {
                tc::tma_load_2d(c.base + kOffK + h * kRegion, &tmK, c.bar(kKV), 64 * h, z * p.N + klo);
                tc::tma_load_2d(c.base + kOffV + h * kRegion, &tmV, c.bar(kKV), 64 * h, z * p.N + klo);
            }
        }
        __syncwarp();
        int nland = 0, nq = 0, no = 0, t = 0, x = z * p.g;
        for (int it = 0; it < iters; ++it) {
            const int2 e = tile(t);
            const int s = it % kStages, row = x * p.N + e.x;
            if (it >= kStages && !__all_sync(kFull, tc::mbar_wait(c.bar(kQe + s), (it / kStages - 1) & 1, c.abort_flag))) break;
            if (!load_tile_zeroed<D>(c, c.base + kOffQ + s * 2 * kRegion, &tmQ, kQf + s, kLand, nland, row, e.y)) break;
            nq = it + 1;
            if (it >= kStages && !__all_sync(kFull, tc::mbar_wait(c.bar(kOe + s), (it / kStages - 1) & 1, c.abort_flag))) break;
            if (!load_tile_zeroed<D>(c, c.base + kOffO + s * 2 * kRegion, &tmO, kOf + s, kLand, nland, row, e.y)) break;
            no = it + 1;
            if (++t == nt) {
                t = 0;
                ++x;
            }
        }
        // every issued load lands before the CTA can exit
        int never = 0;
        for (int m = max(0, nq - kStages); m < nq; ++m) tc::mbar_wait(c.bar(kQf + m % kStages), (m / kStages) & 1, &never);
        for (int m = max(0, no - kStages); m < no; ++m) tc::mbar_wait(c.bar(kOf + m % kStages), (m / kStages) & 1, &never);
        tc::mbar_wait(c.bar(kKV), 0, &never);
    } else if (c.warp == 9) {
        auto wait = [&](int b, int parity) {
            const bool ok = __all_sync(kFull, tc::mbar_wait(c.bar(b), parity & 1, c.abort_flag));
            tc::fence_after_sync();
            return ok;
        };
        const uint32_t tS = c.tmem + kTS, tDP = c.tmem + kTDP;
        auto q = [&](int it) { return c.base + kOffQ + (it % kStages) * 2 * kRegion; };
        auto o = [&](int it) { return c.base + kOffO + (it % kStages) * 2 * kRegion; };
        bool ok = iters > 0 && wait(kKV, 0) && wait(kQf, 0);
        if (ok) {
            if (c.lane == 0) {
                mma_rows<D>(tS, c.base + kOffK, q(0));
                tc::commit(c.bar(kS));
            }
            __syncwarp();
            ok = wait(kOf, 0);
        }
        if (ok) {
            if (c.lane == 0) {
                mma_rows<D>(tDP, c.base + kOffV, o(0));
                tc::commit(c.bar(kDP));
            }
            __syncwarp();
        }
        for (int it = 0; ok && it < iters; ++it) {
            const bool more = it + 1 < iters;
            if (more && !wait(kQf + (it + 1) % kStages, (it + 1) / kStages)) break;
            if (!wait(kP, it)) break;
            if (c.lane == 0) {
                mma_sums<D>(c.tmem + kTDV, tS, o(it), it > 0);
                tc::commit(c.bar(kOe + it % kStages));
                if (more) {
                    mma_rows<D>(tS, c.base + kOffK, q(it + 1));
                    tc::commit(c.bar(kS));
                }
            }
            __syncwarp();
            if (more && !wait(kOf + (it + 1) % kStages, (it + 1) / kStages)) break;
            if (!wait(kDS, it)) break;
            if (c.lane == 0) {
                mma_sums<D>(c.tmem + kTDK, tDP, q(it), it > 0);
                tc::commit(c.bar(kQe + it % kStages));
                if (more) {
                    mma_rows<D>(tDP, c.base + kOffV, o(it + 1));
                    tc::commit(c.bar(kDP));
                }
            }
            __syncwarp();
        }
        // every issued MMA completes before the sums are read and TMEM is released
        if (c.lane == 0) tc::commit(c.bar(kDone));
        __syncwarp();
        int never = 0;
        tc::mbar_wait(c.bar(kDone), 0, &never);
    } else {
        const int w = c.warp >> 2, r = threadIdx.x & 127;
        const uint32_t lane_off = (uint32_t)((c.warp & 3) * 32) << 16;
        const uint32_t tS = c.tmem + kTS + 64 * w + lane_off, tDP = c.tmem + kTDP + 64 * w + lane_off;
        float* buf = reinterpret_cast<float*>(c.sbase + kOffRows) + c.warp * 256;
        const uint64_t cc = pk2(p.scale_log2, p.scale_log2);
        // this lane's two columns of -lse log2(e) and -D of a tile; rows past its end give P = 0
        float nl[2], nd[2];
        auto fetch = [&](int2 e, int x) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = 64 * w + 32 * i + c.lane;
                const long long at = (long long)x * p.N + e.x + col;
                nl[i] = col < e.y ? __ldg(p.nlse2 + at) : -INFINITY;
                nd[i] = col < e.y ? __ldg(p.nD + at) : 0.f;
            }
        };
        int t = 0, x = z * p.g;
        auto advance = [&]() {
            if (++t == nt) {
                t = 0;
                ++x;
            }
        };
        if (iters > 0) fetch(tile(0), x);
        advance();
        int2 next = iters > 1 ? tile(t) : make_int2(0, 0);
        bool ok = true;
        for (int it = 0; it < iters; ++it) {
            float* row = buf + (it & 1) * 128;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                row[32 * i + c.lane] = nl[i];
                row[64 + 32 * i + c.lane] = nd[i];
            }
            __syncwarp();
            if (it + 1 < iters) {
                fetch(next, x);
                advance();
                if (it + 2 < iters) next = tile(t);
            }
            if (!__all_sync(kFull, tc::mbar_wait(c.bar(kS), it & 1, c.abort_flag))) { ok = false; break; }
            tc::fence_after_sync();
            uint32_t pv[2][32];
            tc::tmem_ld32(tS, pv[0]);
            tc::tmem_ld32(tS + 32, pv[1]);
            tc::tmem_wait_ld();
            tc::regs_after_wait(pv[0]);
            tc::regs_after_wait(pv[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float4 l4 = *reinterpret_cast<const float4*>(row + 32 * h + 2 * e);
                    const float ls[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int i = 2 * (e + u);
                        float x0, x1;
                        up2(fma2(pk2(__uint_as_float(pv[h][i]), __uint_as_float(pv[h][i + 1])), cc, pk2(ls[2 * u], ls[2 * u + 1])),
                            x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        pk[e + u] = bf16x2(x0, x1);
                        pv[h][i] = __float_as_uint(x0);
                        pv[h][i + 1] = __float_as_uint(x1);
                    }
                }
                tc::tmem_st16(tS + 16 * h, pk);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(c.bar(kP));
            if (!__all_sync(kFull, tc::mbar_wait(c.bar(kDP), it & 1, c.abort_flag))) { ok = false; break; }
            tc::fence_after_sync();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t dv[32], pk[16];
                tc::tmem_ld32(tDP + 32 * h, dv);
                tc::tmem_wait_ld();
                tc::regs_after_wait(dv);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float4 d4 = *reinterpret_cast<const float4*>(row + 64 + 32 * h + 2 * e);
                    const float ds[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int i = 2 * (e + u);
                        float x0, x1;
                        up2(mul2(add2(pk2(__uint_as_float(dv[i]), __uint_as_float(dv[i + 1])), pk2(ds[2 * u], ds[2 * u + 1])),
                                 pk2(__uint_as_float(pv[h][i]), __uint_as_float(pv[h][i + 1]))),
                            x0, x1);
                        pk[e + u] = bf16x2(x0, x1);
                    }
                }
                tc::tmem_st16(tDP + 16 * h, pk);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(c.bar(kDS));
        }
        // warpgroup 0 stores dV, warpgroup 1 dK
        if (__all_sync(kFull, ok && tc::mbar_wait(c.bar(kDone), 0, c.abort_flag))) {
            tc::fence_after_sync();
            bf16* out = out_row<D>(w ? p.dK : p.dV, p.kperm, z, p.N, klo + r, r < kn, z, p.status);
            store_acc_row<D>(c.tmem + (w ? kTDK : kTDV) + lane_off, w ? p.scale : 1.f, out, iters == 0);
        }
    }
    cta_finish(c, p.status);
}

// ---------------------------------------------------------------- dQ
// One CTA per 128-query tile of a query head, streaming the (K, V) tiles of its kept keys. Per
// tile, with queries in the TMEM lanes: S = Q K^T -> P;  dP = dO V^T;  dS (over S);  dQ += dS K.
// S has two buffers, so S(j+1) is ready when the warpgroups turn to it; dP(j+1) is issued as soon
// as dP(j) has been read.
namespace dq {
constexpr int kKStages = 3, kVStages = 2;
constexpr int kOffQ = 0, kOffO = 2 * kRegion, kOffK = 4 * kRegion, kOffV = kOffK + kKStages * 2 * kRegion,
              kOffBar = kOffV + kVStages * 2 * kRegion;
enum { kQO = 0, kKf = 1, kVf = kKf + kKStages, kKe = kVf + kVStages, kVe = kKe + kKStages, kS = kVe + kVStages, kDP = kS + 2,
       kRead = kDP + 1, kDS = kRead + 1, kDone = kDS + 1, kLand = kDone + 1, kBars = kLand + 1 };
constexpr int kSmem = kOffBar + 8 * kBars + 16 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr uint32_t kTS = 0, kTDP = 256, kTDQ = 384;
}  // namespace dq

template <int D>
__global__ void __launch_bounds__(kThreads, 1) bwd_dq_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                             const __grid_constant__ CUtensorMap tmK,
                                                             const __grid_constant__ CUtensorMap tmV,
                                                             const __grid_constant__ CUtensorMap tmO, const BwdParams p) {
    using namespace dq;
    extern __shared__ unsigned char smem_raw[];
    if (p.status && *reinterpret_cast<volatile int*>(p.status) == kDevTimeout) return;
    const int x = blockIdx.y, z = x / p.g;
    int grp, qlo, qn;
    if (!find_tile(p.qoff, p.qtile_off, z, p.Gq, p.N, blockIdx.x, grp, qlo, qn)) return;
    const int2* list = p.klist + ((long long)z * p.Gq + grp) * p.kcap;
    const int nt = p.kcnt ? p.kcnt[(long long)z * p.Gq + grp] : (p.N + kTile - 1) / kTile;
    auto tile = [&](int t) { return p.kcnt ? list[t] : make_int2(t * kTile, min(kTile, p.N - t * kTile)); };
    const int counts[kBars] = {1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 256, 256, 1, 1};
    const Cta c = cta_setup(smem_raw, kOffBar, counts, kBars);

    if (c.warp == 8) {
        if (c.lane == 0) {
            tc::mbar_arrive_expect_tx(c.bar(kQO), 2 * (D / 64) * kRegion);
            for (int h = 0; h < D / 64; ++h) {
                tc::tma_load_2d(c.base + kOffQ + h * kRegion, &tmQ, c.bar(kQO), 64 * h, x * p.N + qlo);
                tc::tma_load_2d(c.base + kOffO + h * kRegion, &tmO, c.bar(kQO), 64 * h, x * p.N + qlo);
            }
        }
        __syncwarp();
        int nland = 0, nk = 0, nv = 0;
        for (int t = 0; t < nt; ++t) {
            const int2 e = tile(t);
            const int sk = t % kKStages, sv = t % kVStages, row = z * p.N + e.x;
            if (t >= kKStages && !__all_sync(kFull, tc::mbar_wait(c.bar(kKe + sk), (t / kKStages - 1) & 1, c.abort_flag))) break;
            if (!load_tile_zeroed<D>(c, c.base + kOffK + sk * 2 * kRegion, &tmK, kKf + sk, kLand, nland, row, e.y)) break;
            nk = t + 1;
            if (t >= kVStages && !__all_sync(kFull, tc::mbar_wait(c.bar(kVe + sv), (t / kVStages - 1) & 1, c.abort_flag))) break;
            if (!load_tile_zeroed<D>(c, c.base + kOffV + sv * 2 * kRegion, &tmV, kVf + sv, kLand, nland, row, e.y)) break;
            nv = t + 1;
        }
        int never = 0;
        for (int m = max(0, nk - kKStages); m < nk; ++m) tc::mbar_wait(c.bar(kKf + m % kKStages), (m / kKStages) & 1, &never);
        for (int m = max(0, nv - kVStages); m < nv; ++m) tc::mbar_wait(c.bar(kVf + m % kVStages), (m / kVStages) & 1, &never);
        tc::mbar_wait(c.bar(kQO), 0, &never);
    } else if (c.warp == 9) {
        auto wait = [&](int b, int parity) {
            const bool ok = __all_sync(kFull, tc::mbar_wait(c.bar(b), parity & 1, c.abort_flag));
            tc::fence_after_sync();
            return ok;
        };
        auto k = [&](int t) { return c.base + kOffK + (t % kKStages) * 2 * kRegion; };
        auto v = [&](int t) { return c.base + kOffV + (t % kVStages) * 2 * kRegion; };
        auto tS = [&](int t) { return c.tmem + kTS + 128 * (t & 1); };
        auto issue_S = [&](int t) {      // S(t) once K(t) has landed; its buffer's reader is done in issue order
            if (!wait(kKf + t % kKStages, t / kKStages)) return false;
            if (c.lane == 0) {
                mma_rows<D>(tS(t), c.base + kOffQ, k(t));
                tc::commit(c.bar(kS + (t & 1)));
            }
            __syncwarp();
            return true;
        };
        auto issue_dP = [&](int t) {
            if (!wait(kVf + t % kVStages, t / kVStages)) return false;
            if (c.lane == 0) {
                mma_rows<D>(c.tmem + kTDP, c.base + kOffO, v(t));
                tc::commit(c.bar(kDP));
                tc::commit(c.bar(kVe + t % kVStages));
            }
            __syncwarp();
            return true;
        };
        bool ok = nt > 0 && wait(kQO, 0) && issue_S(0) && issue_dP(0) && (nt < 2 || issue_S(1));
        for (int t = 0; ok && t < nt; ++t) {
            if (!wait(kRead, t)) break;                     // dP(t) is in registers
            if (t + 1 < nt && !issue_dP(t + 1)) break;
            if (!wait(kDS, t)) break;
            if (c.lane == 0) {
                mma_sums<D>(c.tmem + kTDQ, tS(t), k(t), t > 0);
                tc::commit(c.bar(kKe + t % kKStages));
            }
            __syncwarp();
            if (t + 2 < nt && !issue_S(t + 2)) break;
        }
        if (c.lane == 0) tc::commit(c.bar(kDone));
        __syncwarp();
        int never = 0;
        tc::mbar_wait(c.bar(kDone), 0, &never);
    } else {
        const int w = c.warp >> 2, r = threadIdx.x & 127;
        const uint32_t lane_off = (uint32_t)((c.warp & 3) * 32) << 16;
        const uint32_t tDP = c.tmem + kTDP + 64 * w + lane_off;
        const long long row = (long long)x * p.N + qlo + r;
        const float nl = r < qn ? p.nlse2[row] : -INFINITY, nd = r < qn ? p.nD[row] : 0.f;
        const uint64_t cc = pk2(p.scale_log2, p.scale_log2), nl2 = pk2(nl, nl), nd2 = pk2(nd, nd);
        bool ok = true;
        int valid_next = nt > 0 ? tile(0).y : 0;
        for (int t = 0; t < nt; ++t) {
            const int valid = valid_next;
            if (t + 1 < nt) valid_next = tile(t + 1).y;
            const uint32_t tS = c.tmem + kTS + 128 * (t & 1) + 64 * w + lane_off;
            if (!__all_sync(kFull, tc::mbar_wait(c.bar(kS + (t & 1)), (t >> 1) & 1, c.abort_flag))) { ok = false; break; }
            tc::fence_after_sync();
            uint32_t pv[2][32];
            tc::tmem_ld32(tS, pv[0]);
            tc::tmem_ld32(tS + 32, pv[1]);
            tc::tmem_wait_ld();
            tc::regs_after_wait(pv[0]);
            tc::regs_after_wait(pv[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float x0, x1;
                    up2(fma2(pk2(__uint_as_float(pv[h][i]), __uint_as_float(pv[h][i + 1])), cc, nl2), x0, x1);
                    pv[h][i] = __float_as_uint(ex2(x0));
                    pv[h][i + 1] = __float_as_uint(ex2(x1));
                }
                if (valid < kTile) {      // keys past the tile's end
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (64 * w + 32 * h + i >= valid) pv[h][i] = 0u;
                }
            }
            if (!__all_sync(kFull, tc::mbar_wait(c.bar(kDP), t & 1, c.abort_flag))) { ok = false; break; }
            tc::fence_after_sync();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t dv[32], pk[16];
                tc::tmem_ld32(tDP + 32 * h, dv);
                tc::tmem_wait_ld();
                tc::regs_after_wait(dv);
                if (h == 1) {
                    tc::fence_before_sync();
                    tc::mbar_arrive(c.bar(kRead));
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float x0, x1;
                    up2(mul2(add2(pk2(__uint_as_float(dv[2 * e]), __uint_as_float(dv[2 * e + 1])), nd2),
                             pk2(__uint_as_float(pv[h][2 * e]), __uint_as_float(pv[h][2 * e + 1]))),
                        x0, x1);
                    pk[e] = bf16x2(x0, x1);
                }
                tc::tmem_st16(tS + 16 * h, pk);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(c.bar(kDS));
        }
        if (__all_sync(kFull, ok && tc::mbar_wait(c.bar(kDone), 0, c.abort_flag))) {
            tc::fence_after_sync();
            // each warpgroup stores half of the row's columns
            bf16* out = out_row<D>(p.dQ, p.qperm, x, p.N, qlo + r, r < qn, z, p.status);
            store_acc_row<D / 2>(c.tmem + kTDQ + w * (D / 2) + lane_off, p.scale, out ? out + w * (D / 2) : nullptr, nt == 0);
        }
    }
    cta_finish(c, p.status);
}

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

// Byte offsets of the workspace's parts.
struct BwdLayout {
    size_t nlse2, nD, klist, qlist, kcnt, qcnt, qtile_off, ktile_off, bytes;
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
        l.qtile_off = take((size_t)P * (Gq + 1) * sizeof(int32_t));
        l.ktile_off = take((size_t)P * (Gk + 1) * sizeof(int32_t));
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
    p.nlse2 = nlse2; p.nD = nD;
    p.dQ = a.dQ; p.dK = a.dK; p.dV = a.dV;
    p.N = a.N; p.g = a.g; p.Gq = 1; p.Gk = 1;
    p.status = a.status;
    p.scale = (float)(1.0 / sqrt((double)D));
    p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
    if (sparse) {
        int2 *klist = reinterpret_cast<int2*>(ws + l.klist), *qlist = reinterpret_cast<int2*>(ws + l.qlist);
        int32_t *kcnt = reinterpret_cast<int32_t*>(ws + l.kcnt), *qcnt = reinterpret_cast<int32_t*>(ws + l.qcnt);
        int32_t *qt = reinterpret_cast<int32_t*>(ws + l.qtile_off), *kt = reinterpret_cast<int32_t*>(ws + l.ktile_off);
        const long long warps = (long long)a.P * (a.Gq + a.Gk + 2);
        bwd_lists_kernel<<<(unsigned)((warps * 32 + 255) / 256), 256, 0, s>>>(
            a.rowptr, a.kg, a.qoff, a.koff, klist, kcnt, qlist, qcnt, qt, kt, l.kcap, l.qcap, a.P, a.N, a.Gq, a.Gk, a.status);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        p.qoff = a.qoff; p.koff = a.koff; p.qperm = a.qperm; p.kperm = a.kperm;
        p.klist = klist; p.qlist = qlist; p.kcnt = kcnt; p.qcnt = qcnt;
        p.qtile_off = qt; p.ktile_off = kt;
        p.kcap = l.kcap; p.qcap = l.qcap;
        p.Gq = a.Gq; p.Gk = a.Gk;
    }
    CUtensorMap mq, mk, mv, mo;
    const long long krows = (long long)a.P * a.N;
    if (!make_tmap_bf16_sw128(&mq, a.Q, rows, D, kTile, 64) || !make_tmap_bf16_sw128(&mk, a.K, krows, D, kTile, 64) ||
        !make_tmap_bf16_sw128(&mv, a.V, krows, D, kTile, 64) || !make_tmap_bf16_sw128(&mo, a.dO, rows, D, kTile, 64))
        return cudaErrorInvalidValue;
    const unsigned tiles = (unsigned)((a.N + kTile - 1) / kTile);
    if (a.dQ) {
        e = cudaFuncSetAttribute(bwd_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, dq::kSmem);
        if (e != cudaSuccess) return e;
        bwd_dq_kernel<D><<<dim3(tiles + (sparse ? a.Gq : 0), a.P * a.g), kThreads, dq::kSmem, s>>>(mq, mk, mv, mo, p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (a.dK) {
        e = cudaFuncSetAttribute(bwd_dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kv::kSmem);
        if (e != cudaSuccess) return e;
        bwd_dkv_kernel<D><<<dim3(tiles + (sparse ? a.Gk : 0), a.P), kThreads, kv::kSmem, s>>>(mq, mk, mv, mo, p);
    }
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

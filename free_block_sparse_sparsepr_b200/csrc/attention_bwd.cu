// Backward passes of the attention steps: gradients of O = softmax(Q K^T / sqrt(d)) V over all keys
// (dense) or over each query group's kept key groups (block-sparse), from the forward pass's
// inputs, output and lse. With s = q.k / sqrt(d) and the probabilities recomputed, for every kept
// pair (i, j):
//   P_ij = exp(s_ij - lse_i),  D_i = dO_i . O_i,  dS_ij = P_ij (dO_i . v_j - D_i),
//   dV_j = sum_i P_ij dO_i,  dK_j = sum_i dS_ij q_i / sqrt(d),  dQ_i = sum_j dS_ij k_j / sqrt(d);
// dK and dV also sum over the query heads that share the KV head. Each gradient row is summed in a
// fixed order by one CTA, or by a fixed number of CTAs whose sums are joined in order (no atomics), so
// results repeat bit for bit.
//
// Roundings: P and dS become bf16 (2^-8 of each element at most) because the tensor cores take no fp32
// operand, and TF32 would halve their rate. In the 2-norm against fp64 that leaves dQ at 2.5 to 3.0e-3, dK and dV at
// 2.2 to 2.4e-3, where rounding the exact gradients to bf16 costs 1.7e-3. dQ suffers most: sum_j dS_ij = 0 takes
// the keys' common part out of the gradient but not out of the errors. The caller may have dS in two bf16 parts
// there (SPLIT): dQ is then at 1.66e-3 for an eighth product, 10 to 14% more time a call (12 heads x 4096 rows
// 314 -> 359 us, 24 x 8192 2.31 -> 2.57 ms, d = 64 24 x 4096 422 -> 470 us; 24 x 8192 at 22% kept 755 -> 829 us).
// lse, D, the logits and all sums are fp32.
//
// Bound by the tensor pipe (74% of its cycles at 4096 rows, d = 128) and, in long calls, by the power cap; at d = 64,
// where the products are half as long and the arithmetic is not, by the hand-over between the two (tensor pipe
// 50%, issue slots 60%). A call among others, the power cap settled: 12 heads x 4096 rows, d = 128 309 us (834
// TFLOP/s of 10 N^2 d a head), 24 x 8192 2.27 ms (907 TFLOP/s, the seven products at 1.27 PFLOP/s), 24 x 4096 at
// d = 64 416 us (619 TFLOP/s). Short graph runs, before it settles: 268 to 290 us, 2.21 to 2.25 ms, 380 us.
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
    const int2 *klist, *qlist;              // kept key tiles of each query group (or two), query tiles of each key group
    const int32_t *kcnt, *qcnt;             // their numbers
    const int4 *qtile, *ktile;              // [P][q_tiles], [P][kv_tiles]: list, first row, rows of each tile (0: none); joined:
                                            // rows of the first group (0: of one group) << 8, and the list's length
    int kcap, qcap;                         // list entries per group
    int* status;
    long long krows, qrows;                 // P N, P g N
    int N, g, Gq, Gk;                       // Gq, Gk: lists per KV head
    int kv_tiles, q_tiles;                  // most key tiles of a KV head, query tiles of a query head
    int kv_parts, q_parts;                  // CTAs that share a tile's stream
    float *kv_part, *q_part;                // their fp32 sums: [part][dV, dK][P N][D], [part][P g N][D]
    int kv_blocks;                          // CTAs of dK and dV
    int kv_first, q_early;                  // launch order: so many of dK and dV, so many of dQ, then the others of each
    float scale, scale_log2;
    const int32_t* loose;                   // [P][query groups, key groups]: whether their offsets leave rows out (null: dense)
    int stall;                              // test only: the tile that a CTA owns is not loaded, so that the wait for it runs out
};

// Tensor maps of [rows][64] boxes of 128 rows.
struct BwdMaps {
    CUtensorMap q, k, v, o;
};

// ---------------------------------------------------------------- per-row terms
// D_i = dO_i . O_i and -lse_i log2(e), negated as the kernels add them. One 16-byte vector of a
// row per thread, D / 8 threads a row; `t` counts threads. Reads O and dO once: bound by HBM.
template <int D>
__device__ __forceinline__ void row_terms(const uint4* __restrict__ O, const uint4* __restrict__ dO,
                                          const float* __restrict__ lse, float* __restrict__ nlse2,
                                          float* __restrict__ nD, long long rows, long long t) {
    constexpr int kV = D / 8;
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
// ascend); without `joined` the last 2 P cut each side's own groups into tiles. Ids out of range or order and
// offsets out of range are skipped and reported in the status word, so every tile stays inside [0, N).
//
// Joined: a tile may hold the last rows of one group and the first of the next that is not empty, so that
// groups of 100 or 130 rows do not leave half of the lanes idle. Its list is the union of both groups' lists,
// each entry with the groups that keep it (1 the first, 2 the second, 3 both; two more warps per group), and
// the sums skip the other group's lanes. Which tiles to join depends on how much the lists share: the cut is
// chosen per KV head and side with the lists at hand (joined_tiles). 24 heads x 8192 tokens, 64 uneven groups,
// 22% kept: the owned tiles are filled to 1.0 in place of 0.67, 660 us in place of 930; 12 x 16384 1174 and 1370.
constexpr int kMaxGroups = 1024;            // of a side
struct ListParams {
    const int32_t *rowptr, *kg, *qoff, *koff;
    int2 *klist, *qlist;
    int32_t *kcnt, *qcnt;
    int4 *qtile, *ktile;
    int32_t* loose;
    int* status;
    int kcap, qcap, q_tiles, kv_tiles, P, N, Gq, Gk, g, joined;
};

// Cuts the runs of a list into tiles as they are found.
struct Runs {
    int2* out;
    int cap, lane, nt = 0, lo = 0, hi = 0, cls = 0;
    bool bad = false;
    __device__ __forceinline__ void emit() {
        const int n = (hi - lo + kTile - 1) / kTile;
        if (nt + n > cap) {     // more tiles than disjoint groups can have
            bad = true;
            return;
        }
        for (int t = lane; t < n; t += 32) out[nt + t] = make_int2(lo + t * kTile, min(kTile, hi - lo - t * kTile) | cls << 8);
        nt += n;
    }
    // the rows [l, h) that each lane holds (none: h <= l), in lane order, of class c
    __device__ __forceinline__ void add(int l, int h, int c) {
        unsigned todo = __ballot_sync(kFull, h > l);
        while (todo) {
            const int i = __ffs(todo) - 1;
            todo &= todo - 1;
            const int nl = __shfl_sync(kFull, l, i), nh = __shfl_sync(kFull, h, i), nc = __shfl_sync(kFull, c, i);
            if (nl != hi || nc != cls) {
                emit();
                lo = nl;
                cls = nc;
            }
            hi = nh;
        }
    }
};

// Whether the ascending ids kept[r.x .. r.y) hold `id`; the next search, for an id above, starts at `r.x`.
__device__ __forceinline__ bool holds(const int32_t* kept, int2& r, int id) {
    int e = r.y;
    while (r.x < e) {
        const int m = (r.x + e) >> 1;
        if (kept[m] < id) r.x = m + 1; else e = m;
    }
    return r.x < r.y && kept[r.x] == id;
}

__device__ void tile_lists(const ListParams& l, int wid, int lane) {
    const int P = l.P, N = l.N, Gq = l.Gq, Gk = l.Gk, lists = P * (Gq + Gk);
    int* status = l.status;
    if (!l.joined && wid >= lists) {
        const int i = wid - lists, z = i >> 1, G = (i & 1) ? Gk : Gq;
        if (z >= P) return;
        const int32_t* off = (i & 1) ? l.koff + (long long)z * (Gk + 1) : l.qoff + (long long)z * (Gq + 1);
        const int cap = (i & 1) ? l.kv_tiles : l.q_tiles;
        int4* out = ((i & 1) ? l.ktile : l.qtile) + (long long)z * cap;
        bool bad = off[0] != 0 || off[G] != N;       // rows that no group holds would get no gradient
        int before = 0;
        for (int g0 = 0; g0 < G; g0 += 32) {
            int n = 0, lo = 0, hi = 0;
            if (g0 + lane < G) {
                lo = off[g0 + lane];
                hi = off[g0 + lane + 1];
                if (lo < 0 || hi < lo || hi > N) bad = true;
                else n = (hi - lo + kTile - 1) / kTile;
            }
            int sum = n;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, sum, o);
                if (lane >= o) sum += v;
            }
            for (int t = 0; t < n; ++t) {
                const int at = before + sum - n + t;
                if (at < cap) out[at] = make_int4(g0 + lane, lo + t * kTile, min(kTile, hi - lo - t * kTile), 0);
                else bad = true;       // more tiles than disjoint groups can have
            }
            before += __shfl_sync(kFull, sum, 31);
        }
        for (int t = before + lane; t < cap; t += 32) out[t] = make_int4(0, 0, 0, 0);
        bad = __any_sync(kFull, bad);
        if (lane == 0) {
            l.loose[i] = bad;
            if (bad) set_status(status, kDevBounds);
        }
        return;
    }
    if (wid >= lists * (l.joined ? 2 : 1)) return;
    const bool pair = wid >= lists;
    wid -= pair ? lists : 0;
    const bool rows = wid < P * Gq;
    const int z = rows ? wid / Gq : (wid - P * Gq) / Gk, G = rows ? Gq : Gk, others = rows ? Gk : Gq;
    const int own = rows ? wid % Gq : (wid - P * Gq) % Gk;
    const int32_t* rp = l.rowptr + (long long)z * (Gq + 1);
    const int32_t* kept = l.kg + (long long)z * Gq * Gk;
    const int32_t *koff = l.koff + (long long)z * (Gk + 1), *qoff = l.qoff + (long long)z * (Gq + 1);
    const int32_t *off = rows ? koff : qoff, *own_off = rows ? qoff : koff;
    const int lists_z = G * (l.joined ? 2 : 1);
    const long long id = (long long)z * lists_z + (pair ? G : 0) + own;
    int32_t* count = (rows ? l.kcnt : l.qcnt) + id;
    Runs runs;
    runs.cap = rows ? l.kcap : l.qcap;
    runs.out = (rows ? l.klist : l.qlist) + id * runs.cap;
    runs.lane = lane;
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
    // the rows of the other side's group k
    auto bounds = [&](int k) {
        int2 r = make_int2(off[k], off[k + 1]);
        if (r.x < 0 || r.y < r.x || r.y > N) {
            bad = true;
            r = make_int2(0, 0);
        }
        return r;
    };
    if (pair) {
        int next = G;       // the next group that is not empty
        for (int g0 = own + 1; g0 < G && next == G; g0 += 32) {
            const unsigned some = __ballot_sync(kFull, g0 + lane < G && own_off[min(g0 + lane, G - 1) + 1] > own_off[min(g0 + lane, G - 1)]);
            if (some) next = g0 + __ffs(some) - 1;
        }
        if (next < G && own_off[own + 1] > own_off[own]) {
            const int2 r0 = rows ? row_range(own) : make_int2(0, 0), r1 = rows ? row_range(next) : make_int2(0, 0);
            for (int k0 = 0; k0 < others; k0 += 32) {
                const int k = k0 + lane;
                int2 b = make_int2(0, 0);
                int cls = 0;
                if (k < others) {
                    b = bounds(k);
                    int2 r = rows ? r0 : row_range(k), other = r1;
                    cls = holds(kept, r, rows ? k : own);
                    if (!rows) other = make_int2(r.x, min(r.y, r.x + next - own + 1));      // ids ascend
                    cls |= holds(kept, other, rows ? k : next) << 1;
                    if (!cls) b = make_int2(0, 0);
                }
                runs.add(b.x, b.y, cls);
            }
            runs.emit();
        }
    } else {
        const int2 own_row = rows ? row_range(own) : make_int2(0, Gq);
        for (int c0 = own_row.x; c0 < own_row.y; c0 += 32) {
            const int c = c0 + lane;
            int2 b = make_int2(0, 0);
            if (c < own_row.y) {
                int grp = -1;
                if (rows) {
                    grp = kept[c];
                    if (grp < 0 || grp >= Gk || (c > own_row.x && kept[c - 1] >= grp)) {      // out of range or order
                        bad = true;
                        grp = -1;
                    }
                } else {
                    int2 r = row_range(c);
                    if (holds(kept, r, own)) grp = c;
                }
                if (grp >= 0) b = bounds(grp);
            }
            runs.add(b.x, b.y, 0);
        }
        runs.emit();
    }
    if (lane == 0) *count = runs.nt;
    if (__any_sync(kFull, bad || runs.bad) && lane == 0) set_status(status, kDevBounds);
}

// The cut of one side of one KV head (z = i / 2; keys where i is odd) into tiles of one or two groups, by four
// warps. Four ways to deal with a group's last rows, r < 128 of them: a tile of their own; joined with the next
// group's own last rows where both fit a tile (a tile fewer, and the list no longer than both), those moved to
// its front; the same filled up; filled up with the next group's first rows always. Each warp walks one
// and counts streamed tiles, 3.5 more for a CTA's start and end; the cheapest is written.
__device__ void joined_tiles(const ListParams& l, int i, int warp, int lane) {
    __shared__ unsigned long long s_cost[4];
    __shared__ int4 s_group[kMaxGroups];         // first row, rows, streamed tiles alone and with the next group
    __shared__ unsigned short s_id[kMaxGroups];
    const int z = i >> 1, keys = i & 1, G = keys ? l.Gk : l.Gq, N = l.N;
    const int32_t* off = keys ? l.koff + (long long)z * (G + 1) : l.qoff + (long long)z * (G + 1);
    const int32_t* cnt = (keys ? l.qcnt : l.kcnt) + (long long)z * 2 * G;
    const int cap = keys ? l.kv_tiles : l.q_tiles;
    int4* out = (keys ? l.ktile : l.qtile) + (long long)z * cap;
    bool bad = off[0] != 0 || off[G] != N;       // rows that no group holds would get no gradient
    int m = 0;                                   // groups that are not empty
    for (int g0 = 0; g0 < G; g0 += 32) {         // (every warp counts them, the first keeps them)
        const int grp = g0 + lane;
        int lo = 0, hi = 0;
        if (grp < G) {
            lo = off[grp];
            hi = off[grp + 1];
            if (lo < 0 || hi < lo || hi > N) {
                bad = true;
                lo = hi = 0;
            }
        }
        const unsigned some = __ballot_sync(kFull, hi > lo);
        if (hi > lo && warp == 0) {
            const int at = m + __popc(some & ((1u << lane) - 1));
            s_group[at] = make_int4(lo, hi - lo, cnt[grp], cnt[G + grp]);
            s_id[at] = (unsigned short)grp;
        }
        m += __popc(some);
    }
    tc::named_bar_sync(1, 128);
    // calls tile(list, first row, rows, split, streamed tiles, number of such tiles after one another)
    auto walk = [&](int mode, auto tile) {
        int o = 0;                               // rows of the group that are in tiles
        int4 e = s_group[0];
        for (int j = 0; j < m;) {
            const int id = s_id[j], lo = e.x + o, rest = e.y - o, whole = rest / kTile, r = rest % kTile;
            const int4 next = s_group[min(j + 1, m - 1)];
            if (whole) tile(id, lo, kTile, 0, e.z, whole);
            const int at = lo + whole * kTile;
            int take = 0;
            if (r && mode > 0 && j + 1 < m && next.x == at + r) {
                const int room = kTile - r, last = (next.y - 1) % kTile + 1;
                take = mode == 3 ? min(room, next.y) : last > room ? 0 : mode == 2 ? min(room, next.y) : last;
            }
            if (r) tile(take ? G + id : id, at, r + take, take ? r : 0, take ? e.w : e.z, 1);
            ++j;
            o = take;
            e = next;
            if (take && take == next.y) {
                ++j;
                o = 0;
                e = s_group[min(j, m - 1)];
            }
        }
    };
    const int heads = keys ? l.g : 1;
    unsigned long long cost = 0;
    walk(warp, [&](int, int, int, int, int streamed, int n) { cost += n * (2ull * streamed * heads + 7); });
    if (lane == 0) s_cost[warp] = cost;
    tc::named_bar_sync(1, 128);
    if (warp != 0) return;
    int mode = 0;
    for (int k = 1; k < 4; ++k)
        if (s_cost[k] < s_cost[mode]) mode = k;
    int nt = 0;
    walk(mode, [&](int list, int lo, int rows, int split, int streamed, int n) {
        for (int t = lane; t < n && nt + t < cap; t += 32) out[nt + t] = make_int4(list, lo + t * kTile, rows | split << 8, streamed);
        nt += n;
    });
    if (nt > cap) bad = true;                    // more tiles than disjoint groups can have
    for (int t = nt + lane; t < cap; t += 32) out[t] = make_int4(0, 0, 0, 0);
    if (__any_sync(kFull, bad) && lane == 0) set_status(l.status, kDevBounds);
}

// The lists (blocks before `list_blocks`) and the rows' terms (the others) in one launch; the joined tiles
// read the lists, so then these have a launch of their own and the tiles take their place.
template <int D>
__global__ void __launch_bounds__(256) bwd_prepare_kernel(const ListParams l, int list_blocks, const uint4* O, const uint4* dO,
                                                          const float* lse, float* nlse2, float* nD, long long rows) {
    if ((int)blockIdx.x < list_blocks) {
        if (!l.joined) tile_lists(l, (blockIdx.x * blockDim.x + threadIdx.x) >> 5, threadIdx.x & 31);
        else if (threadIdx.x < 128) joined_tiles(l, blockIdx.x, threadIdx.x >> 5, threadIdx.x & 31);
        return;
    }
    row_terms<D>(O, dO, lse, nlse2, nD, rows, (long long)(blockIdx.x - list_blocks) * blockDim.x + threadIdx.x);
}

__global__ void __launch_bounds__(256) bwd_lists_kernel(const ListParams l) {
    tile_lists(l, (blockIdx.x * blockDim.x + threadIdx.x) >> 5, threadIdx.x & 31);
}

// ---------------------------------------------------------------- gradients
// Both kernels run two or four warpgroups that form P and dS (thread r of a warpgroup owns TMEM lane r of
// the warpgroup's share of the 128 columns), a warp that loads tiles (TMA) and one that allocates TMEM and
// issues every MMA. P and dS go back to TMEM as bf16 pairs, where they are the A operands of the next
// product, so no transposed copy is ever made: the dK/dV kernel keeps keys in the lanes
// (S^T = K Q^T), the dQ kernel queries. They have columns of their own, so the fp32 columns of S and
// dP are free again as soon as they have been read, and the next product into them runs beside the
// arithmetic on the last.
// Rows of a streamed tile past its valid ones belong to another group or head: the loading warp
// zeroes them in shared memory, so that no value there, finite or not, reaches a sum.
constexpr int kRegion = 16384;              // one [128 rows][64 bf16] region, 128-byte swizzle
// Warpgroups that form P and dS, and the warps after them. d = 64 halves the products' time but not the
// arithmetic's, so it takes four where d = 128 takes two (24 heads x 4096 rows, d = 64: 433 us with two, 416
// with four; 12 heads, d = 128: 278 and 280).
template <int D>
struct Warps {
    static constexpr int kWgs = D == 64 ? 4 : 2, kTma = 4 * kWgs, kMma = kTma + 1, kThreads = 32 * (kMma + 1);
    static constexpr int kArrivals = 128 * kWgs;
    static constexpr int kCols = kTile / kWgs, kH = kCols / 32;     // columns of a thread, in blocks of 32
};
constexpr uint32_t kTmemCols = 512;

// Set-up shared by the kernels: aligned shared memory, barriers (`count` arrivals each), TMEM; the loading
// warp starts on the tiles that stay (`early`) while the others set up.
struct Cta {
    uint32_t base, bars, tmem;
    unsigned char* sbase;
    volatile int* abort_flag;
    int warp, lane, mma_warp;
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * (uint32_t)i; }
};

// A CTA that timed out earlier (in this launch or call) makes the rest abort at their first wait.
template <int D, typename Count, typename Early>
__device__ __forceinline__ Cta cta_setup(unsigned char* smem_raw, int off_bar, int nbars, const int* status, Count count, Early early) {
    Cta c;
    const uint32_t raw = tc::smem_addr(smem_raw);
    c.base = (raw + 1023u) & ~1023u;
    c.sbase = smem_raw + (c.base - raw);
    c.bars = c.base + off_bar;
    c.warp = threadIdx.x >> 5;
    c.lane = threadIdx.x & 31;
    c.mma_warp = Warps<D>::kMma;
    uint32_t* slot = reinterpret_cast<uint32_t*>(c.sbase + off_bar + 8 * nbars);
    c.abort_flag = reinterpret_cast<volatile int*>(slot + 1);
    if (c.warp == Warps<D>::kTma && c.lane == 0) {
        const int before = *reinterpret_cast<const volatile int*>(status);
        for (int i = 0; i < nbars; ++i) tc::mbar_init(c.bar(i), count(i));
        tc::fence_mbar_init();
        early(c);
        *c.abort_flag = before == kDevTimeout;
    }
    if (c.warp == Warps<D>::kMma) {
        tc::tmem_alloc(tc::smem_addr(slot), kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    c.tmem = *slot;
    return c;
}

// Whether every MMA has completed (barrier `done`) and no wait of the CTA gave up, for a converged warp whose own
// waits went `ok`. The flag is read after the barrier: a warp that leaves its loop early, the one that issues the
// MMAs too, raises it before it arrives there, and a CTA that found the timeout of an earlier one has it up from
// the start, though each of its waits may succeed at once. Without it such a CTA would store sums that lack a product.
__device__ __forceinline__ bool sums_complete(const Cta& c, bool ok, int done) {
    ok = ok && tc::mbar_wait(c.bar(done), 0, c.abort_flag) && !*c.abort_flag;
    tc::fence_after_sync();
    return __all_sync(kFull, ok);
}

// Releases TMEM and reports a wait that gave up; every thread of the CTA calls it last.
__device__ __forceinline__ void cta_finish(const Cta& c, int* status) {
    tc::fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && *c.abort_flag) set_status(status, kDevTimeout);
    if (c.warp == c.mma_warp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(c.tmem, kTmemCols);
    }
}

// D[tmem] = A B^T over D columns of two swizzled tiles (both K-major).
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t go) {
    constexpr uint32_t id = tc::idesc_bf16_f32(kTile, kTile, 0);
    const uint64_t da = tc::smem_desc_sw128(a, 16, 1024), db = tc::smem_desc_sw128(b, 16, 1024);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (uint32_t)((k >> 2) * kRegion + (k & 3) * 32) >> 4;     // address field of the descriptors
        tc::mma_f16_ss_go(d_tmem, da + off, db + off, id, k > 0 ? 1u : 0u, go);
    }
}

// Lanes of a tile of two groups, split after `split` rows, that a streamed tile of class `cls` leaves alone.
struct Lanes {
    uint32_t first[4];                      // the first group's
    __device__ __forceinline__ explicit Lanes(int split) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = min(max(split - 32 * i, 0), 32);
            first[i] = n == 32 ? kFull : (1u << n) - 1;
        }
    }
    __device__ __forceinline__ void off(int cls, uint32_t (&o)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = cls == 1 ? ~first[i] : cls == 2 ? first[i] : 0u;
    }
};

// D[tmem] (+)= A B over the 128 rows of tile b (MN-major); A is bf16 pairs in 64 TMEM columns. The lanes of
// `off` (JOINED) stay as they are, whatever their rows of A hold.
template <int D, bool JOINED>
__device__ __forceinline__ void mma_sums(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, const uint32_t (&off)[4], bool accumulate,
                                         uint32_t go) {
    constexpr uint32_t id = tc::idesc_bf16_f32(kTile, D, 1);
    const uint64_t db = tc::smem_desc_sw128(b, kRegion, 1024);
#pragma unroll
    for (int k = 0; k < kTile / 16; ++k) {
        const uint32_t at = a_tmem + (uint32_t)(8 * k);
        const uint64_t bk = db + (uint64_t)(k * 2048 >> 4);
        if (JOINED) tc::mma_f16_ts_off_go(d_tmem, at, bk, id, off, 1u, go);
        else tc::mma_f16_ts_go(d_tmem, at, bk, id, (accumulate || k > 0) ? 1u : 0u, go);
    }
}

// D[tmem] += A B^T over one K step of 16: [128][8] blocks without swizzle, each with the same block of zeros, which
// lies behind both, as the other 8 columns.
constexpr int kExtBlock = kTile * 16;
__device__ __forceinline__ void mma_ext(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t zeros, uint32_t go) {
    constexpr uint32_t id = tc::idesc_bf16_f32(kTile, kTile, 0);
    tc::mma_f16_ss_go(d_tmem, tc::smem_desc_none(a, zeros - a, 128), tc::smem_desc_none(b, zeros - b, 128), id, 1u, go);
}

// x as three bf16 parts that sum to it within 24 bits, in the first of 8 columns; the others are zero.
__device__ __forceinline__ uint4 split3(float x) {
    uint32_t o[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const bf16 h = __float2bfloat16_rn(x);
        o[i] = __bfloat16_as_ushort(h);
        x -= bf16_to_f32(h);
    }
    return make_uint4(o[0] | o[1] << 16, o[2], 0, 0);
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

// What rounding a and b to the bf16 pair `v` left over, rounded in turn.
__device__ __forceinline__ uint32_t bf16x2_rest(float a, float b, uint32_t v) {
    return bf16x2(a - __uint_as_float(v << 16), b - __uint_as_float(v & 0xffff0000u));
}

// 2^x of a pair on the FMA pipe: x = n + f with n the nearest integer (by adding 1.5 2^23) and |f| <= 1/2,
// 2^f by a least-maximum polynomial of degree 4 (relative error 2.7e-6, 2^-18.5, fitted here), 2^n from
// exponent bits. Exponents below -126.5 give 0 (n = -127, whose bits are those of 0), as ex2 gives 0 below
// -126; NaN stays NaN (the product keeps it, an addition to the exponent bits would not).
__device__ __forceinline__ uint64_t ex2_fma(uint64_t x2) {
    float a, b;
    up2(x2, a, b);
    asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(a));      // -127
    asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(b));
    const uint64_t x = pk2(a, b);
    const uint64_t t = add2(x, pk2(12582912.f, 12582912.f));
    const uint64_t f = fma2(add2(t, pk2(-12582912.f, -12582912.f)), pk2(-1.f, -1.f), x);
    uint64_t q = pk2(0.009570096619427204f, 0.009570096619427204f);
    q = fma2(q, f, pk2(0.05591785907745361f, 0.05591785907745361f));
    q = fma2(q, f, pk2(0.240247443318367f, 0.240247443318367f));
    q = fma2(q, f, pk2(0.6931217908859253f, 0.6931217908859253f));
    q = fma2(q, f, pk2(0.9999992847442627f, 0.9999992847442627f));
    float t0, t1;
    up2(t, t0, t1);
    constexpr int one = 127 << 23;
    return mul2(q, pk2(__int_as_float((__float_as_int(t0) << 23) + one), __int_as_float((__float_as_int(t1) << 23) + one)));
}

// 2^x of pair i of a row. The special-function unit alone would take 1024 cycles a 128 x 128 tile,
// most of the arithmetic's time; three pairs of eight go to the FMA pipe instead (12 heads x 4096 rows,
// d = 128, both passes: 297 us with none, 290, 282, 281.5 and 287 us with one to four).
__device__ __forceinline__ void ex2_pair(uint64_t x2, int i, uint32_t& a, uint32_t& b) {
    float x0, x1;
    if (i % 8 < 3) {
        up2(ex2_fma(x2), x0, x1);
    } else {
        up2(x2, x0, x1);
        x0 = ex2(x0);
        x1 = ex2(x1);
    }
    a = __float_as_uint(x0);
    b = __float_as_uint(x1);
}

// This thread's 32 kH columns of an fp32 tile.
template <int kH>
__device__ __forceinline__ void load_cols(uint32_t taddr, uint32_t (&v)[kH][32]) {
    static_assert(kH == 1 || kH == 2, "blocks of 32 columns");
    tc::tmem_ld32(taddr, v[0]);
    if (kH == 2) tc::tmem_ld32(taddr + 32, v[kH - 1]);
    tc::tmem_wait_ld();
    tc::regs_after_wait(v[0]);
    if (kH == 2) tc::regs_after_wait(v[kH - 1]);
}

// A warp's 32 accumulator rows of N TMEM columns, times `scale`, to global rows of T (bf16, or fp32 for
// partial sums); `row` is the place of this lane's row (null: not stored). The lanes hold a row each, so
// storing from there would touch 32 rows with every instruction. The rows go through `stage` instead (room
// for 32 N elements of T, their 16-byte pieces swapped within a row against bank conflicts) and leave as
// whole rows: 3260 cycles of a tile's 90000 for dV and dK at N = 4096, d = 128, where stores from the
// lanes took 6350, and 1750 for dQ, where they took 3190; 1-2% of the call.
template <int N, typename T>
__device__ __forceinline__ void store_acc_rows(uint32_t tacc, unsigned char* stage, int lane, float scale, bool zero, T* row) {
    constexpr int kPer = 16 / sizeof(T), kPieces = N / kPer, kRows = 32 / kPieces;      // elements a piece, pieces a row, rows a step
    uint4* st = reinterpret_cast<uint4*>(stage);
#pragma unroll
    for (int c = 0; c < N / 32; ++c) {
        uint32_t v[32];
        tc::tmem_ld32(tacc + 32 * c, v);
        tc::tmem_wait_ld();
        tc::regs_after_wait(v);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = zero ? 0u : __float_as_uint(__uint_as_float(v[i]) * scale);
#pragma unroll
        for (int q = 0; q < 32 / kPer; ++q) {
            uint4 u;
            if (sizeof(T) == 2)
                u = make_uint4(bf16x2(__uint_as_float(v[8 * q]), __uint_as_float(v[8 * q + 1])),
                               bf16x2(__uint_as_float(v[8 * q + 2]), __uint_as_float(v[8 * q + 3])),
                               bf16x2(__uint_as_float(v[8 * q + 4]), __uint_as_float(v[8 * q + 5])),
                               bf16x2(__uint_as_float(v[8 * q + 6]), __uint_as_float(v[8 * q + 7])));
            else
                u = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            st[lane * kPieces + ((c * (32 / kPer) + q) ^ (lane & (kPieces - 1)))] = u;
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int r = i * kRows + lane / kPieces, piece = lane % kPieces;
        T* to = reinterpret_cast<T*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(row), r));
        const uint4 u = st[r * kPieces + (piece ^ (r & (kPieces - 1)))];
        if (to) *reinterpret_cast<uint4*>(to + piece * kPer) = u;
    }
}

// Zeros in N TMEM columns of the warp's lanes.
template <int N>
__device__ __forceinline__ void zero_cols(uint32_t taddr) {
    const uint32_t z[32] = {};
#pragma unroll
    for (int c = 0; c < N; c += 32) tc::tmem_st32(taddr + c, z);
    tc::tmem_wait_st();
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

// Tile `pair` of one side: rows [lo, lo + n) that stream list `grp`; joined: its length `count`, and the first
// `split` rows' own group. False past the last tile. (A table: a
// search of the group offsets costs a CTA some eight reads of memory one after another.)
__device__ __forceinline__ bool find_tile(const int4* table, int z, int tiles, int N, int pair, int& grp, int& lo, int& n, int& split, int& count) {
    const int4 e = table ? __ldg(table + (long long)z * tiles + pair) : make_int4(0, pair * kTile, min(kTile, N - pair * kTile), 0);
    grp = e.x;
    lo = e.y;
    n = e.z & 255;
    split = e.z >> 8;
    count = e.w;
    return n > 0;
}

// ---------------------------------------------------------------- dK and dV
// One CTA per 128-key tile, streaming the (Q, dO) tiles of every query head of the KV head and
// every query tile that keeps the key group. Per tile, with keys in the TMEM lanes:
//   S^T = K Q^T -> P^T;  dV += P^T dO;  dP^T = V dO^T -> dS^T;  dK += dS^T Q.
// At d = 128, dV and dK take 256 of the 512 TMEM columns, P and dS 64 each; S and dP share the other 128 in
// turn: dP(i) is issued when S(i) has been read, S(i+1) when dP(i) has. Issue order dP(i),
// dK(i-1), S(i+1), dV(i): dP and dK run beside the exponentials, S and dV beside dS.
// The terms -lse and -D of a query vary along the columns here, so a thread would need every query's:
// they are added by the products instead. One more K step of 16 multiplies ones on the key side with
// the three bf16 parts (24 bits) of -lse sqrt(d), or of -D, on the query side. Each has a block of its own: in
// one, zeros would have to keep the other's parts out of the product, and zero times NaN is NaN.
// At d = 64 S and dP have columns of their own: S(i+1) follows the reading of S(i), dP(i+1) that of dP(i).
// At d = 128 four 128-row buffers hold the streamed tiles. dO(i) is done with a product before Q(i), and Q(i+2)
// is wanted before dO(i+2): Q(i+2) takes the buffer of dO(i), dO(i+2) that of Q(i).
namespace kv {
constexpr int kOffK = 0, kOffV = 2 * kRegion, kOffBuf = 4 * kRegion;
constexpr int kKV = 0, kQf = 1;             // the first barriers
constexpr uint32_t kTS = 0;
// What depends on d: d = 128 has two stages of Q and dO and S and dP in the same columns, d = 64 (tiles of
// half the size, sums of half the columns) four stages and columns of their own.
template <int D>
struct Layout {
    static constexpr int kStages = D == 64 ? 4 : 2;
    // parts of -lse and of -D of each stage, the ones, the zeros
    static constexpr int kOffExt = kOffBuf + 8 * kRegion, kOffOne = kOffExt + kStages * 2 * kExtBlock, kOffZero = kOffOne + kExtBlock,
                         kOffBar = kOffZero + kExtBlock;
    // full / empty stages (Q's full one also stands for the row terms); S and dP ready, read; P and dS written;
    // all MMAs done; ragged loads
    enum { kOf = kQf + kStages, kQe = kOf + kStages, kOe = kQe + kStages, kS = kOe + kStages, kDP, kDone, kLand, kSread, kDPread,
           kP, kDS, kBars };
    static constexpr int kSmem = kOffBar + 8 * kBars + 16 + 1024;
    static constexpr uint32_t kTDP = D == 64 ? 128 : 0, kTP = D == 64 ? 256 : 128, kTDS = kTP + 64, kTDV = D == 64 ? 384 : 256,
                              kTDK = kTDV + D;
    static_assert(kSmem <= 232448 && kTDK + D <= kTmemCols, "shared memory or TMEM budget");
    // Buffers of tile i. d = 128: stage i % 2 has two, which Q and dO swap from one use of the stage to the next.
    static __device__ __forceinline__ int q(int i) {
        return kOffBuf + (D == 64 ? (i & 3) * kRegion : (2 * (i & 1) + ((i >> 1) & 1)) * 2 * kRegion);
    }
    static __device__ __forceinline__ int o(int i) {
        return kOffBuf + (D == 64 ? (4 + (i & 3)) * kRegion : (2 * (i & 1) + (((i >> 1) & 1) ^ 1)) * 2 * kRegion);
    }
};
}  // namespace kv

template <int D, bool PARTS, bool JOINED>
__device__ __forceinline__ void dkv_tile(const BwdMaps& m, const BwdParams& p, unsigned char* smem_raw, int z, int pair, int part) {
    using namespace kv;
    using W = Warps<D>;
    using L = Layout<D>;
    constexpr int kStages = L::kStages, kTP = L::kTP, kTDS = L::kTDS, kTDV = L::kTDV, kTDK = L::kTDK;
    constexpr int kOffExt = L::kOffExt, kOffOne = L::kOffOne, kOffZero = L::kOffZero, kOffBar = L::kOffBar;
    constexpr int kOf = L::kOf, kQe = L::kQe, kOe = L::kOe, kS = L::kS, kDP = L::kDP, kDone = L::kDone, kLand = L::kLand, kSread = L::kSread,
                  kDPread = L::kDPread, kP = L::kP, kDS = L::kDS, kBars = L::kBars;
    int grp, klo, kn, split, count;
    if (!find_tile(p.ktile, z, p.kv_tiles, p.N, pair, grp, klo, kn, split, count)) return;
    const int2* list = p.qlist + ((long long)z * p.Gk + grp) * p.qcap;
    const int nt = JOINED ? count : p.qcnt ? p.qcnt[(long long)z * p.Gk + grp] : (p.N + kTile - 1) / kTile;
    // this CTA's share of the (query head, query tile) stream
    const long long all = (long long)nt * p.g;
    const int first = PARTS ? (int)(all * part / p.kv_parts) : 0;
    const int iters = PARTS ? (int)(all * (part + 1) / p.kv_parts) - first : (int)all;
    auto tile = [&](int t) { return p.qcnt ? list[t] : make_int2(t * kTile, min(kTile, p.N - t * kTile)); };
    const int t0 = PARTS && nt ? first % nt : 0;
    const int2 e0 = JOINED && iters > 0 ? tile(t0) : make_int2(0, 0);      // read while the CTA sets up
    {
        // ones under the parts (columns 0-2), and the zeros
        const uint32_t off = ((tc::smem_addr(smem_raw) + 1023u) & ~1023u) - tc::smem_addr(smem_raw);
        uint4* ext = reinterpret_cast<uint4*>(smem_raw + off + kOffOne);
        constexpr uint32_t one = 0x3f80u;
        for (int i = threadIdx.x; i < 2 * kTile; i += W::kThreads)
            ext[i] = i < kTile ? make_uint4(one | one << 16, one, 0, 0) : make_uint4(0, 0, 0, 0);
        tc::fence_proxy_async_smem();
    }
    const Cta c = cta_setup<D>(
        smem_raw, kOffBar, kBars, p.status, [](int i) { return i >= kSread ? W::kArrivals : i >= kQf && i < kOf ? 2 : 1; },
        [&](const Cta& c) {
            if (p.stall) return;
            tc::mbar_arrive_expect_tx(c.bar(kKV), 2 * (D / 64) * kRegion);
            for (int h = 0; h < D / 64; ++h) {
                tc::tma_load_2d(c.base + kOffK + h * kRegion, &m.k, c.bar(kKV), 64 * h, z * p.N + klo);
                tc::tma_load_2d(c.base + kOffV + h * kRegion, &m.v, c.bar(kKV), 64 * h, z * p.N + klo);
            }
        });

    if (c.warp == W::kTma) {
        int nland = 0, nq = 0, no = 0, t = t0, x = z * p.g + (PARTS && nt ? first / nt : 0);
        // this lane's four rows of the next tile's terms; rows past its end give P = 2^(-huge) = 0 (and their
        // Q and dO are zeroed)
        float nl[4], nd[4];
        auto fetch = [&](int2 e, int head) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 32 * j + c.lane, valid = JOINED ? e.y & 255 : e.y;
                const long long at = (long long)head * p.N + e.x + r;
                nl[j] = r < valid ? __ldg(p.nlse2 + at) : -INFINITY;
                nd[j] = r < valid ? __ldg(p.nD + at) : 0.f;
            }
        };
        const float inv = 1.f / p.scale_log2;
        int2 e = JOINED ? e0 : iters > 0 ? tile(t) : make_int2(0, 0);
        if (iters > 0) fetch(e, x);
        for (int it = 0; it < iters; ++it) {
            const int s = it % kStages, row = x * p.N + e.x, valid = JOINED ? e.y & 255 : e.y;
            if (++t == nt) {
                t = 0;
                ++x;
            }
            const int2 next = it + 1 < iters ? tile(t) : make_int2(0, 0);
            // d = 128: Q(it) follows dO(it - 2) in its buffer, dO(it) follows Q(it - 2)
            if (it >= kStages && !__all_sync(kFull, tc::mbar_wait(c.bar((D == 64 ? kQe : kOe) + s), (it / kStages - 1) & 1, c.abort_flag))) break;
            if (!load_tile_zeroed<D>(c, c.base + L::q(it), &m.q, kQf + s, kLand, nland, row, valid)) break;
            nq = it + 1;
            uint4* ext = reinterpret_cast<uint4*>(c.sbase + kOffExt + s * 2 * kExtBlock);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint4 a = split3(fmaxf(nl[j] * inv, -1e30f));
                if (isnan(nl[j])) a.x = 0x7fffu;        // fmaxf drops NaN
                ext[32 * j + c.lane] = a;
                ext[kTile + 32 * j + c.lane] = split3(nd[j]);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (c.lane == 0) tc::mbar_arrive(c.bar(kQf + s));
            if (it + 1 < iters) fetch(next, x);
            if (it >= kStages && !__all_sync(kFull, tc::mbar_wait(c.bar((D == 64 ? kOe : kQe) + s), (it / kStages - 1) & 1, c.abort_flag)))
                break;
            if (!load_tile_zeroed<D>(c, c.base + L::o(it), &m.o, kOf + s, kLand, nland, row, valid)) break;
            no = it + 1;
            e = next;
        }
        // every issued load lands before the CTA can exit
        int never = 0;
        for (int i = max(0, nq - kStages); i < nq; ++i) tc::mbar_wait(c.bar(kQf + i % kStages), (i / kStages) & 1, &never);
        for (int i = max(0, no - kStages); i < no; ++i) tc::mbar_wait(c.bar(kOf + i % kStages), (i / kStages) & 1, &never);
        if (!p.stall) tc::mbar_wait(c.bar(kKV), 0, &never);
    } else if (c.warp == W::kMma) {
        const uint32_t go = tc::elect_one();
        auto wait = [&](int b, int parity) {
            const bool ok = __all_sync(kFull, tc::mbar_wait(c.bar(b), parity & 1, c.abort_flag));
            tc::fence_after_sync();
            return ok;
        };
        const uint32_t tS = c.tmem + kTS, tDP = c.tmem + L::kTDP;
        auto q = [&](int it) { return c.base + L::q(it); };
        auto o = [&](int it) { return c.base + L::o(it); };
        auto ext = [&](int it) { return c.base + kOffExt + (it % kStages) * 2 * kExtBlock; };
        auto issue_S = [&](int it) {
            mma_rows<D>(tS, c.base + kOffK, q(it), go);
            mma_ext(tS, c.base + kOffOne, ext(it), c.base + kOffZero, go);
            tc::commit_go(c.bar(kS), go);
        };
        // joined: the lanes that the last tile's and this tile's sums leave alone
        const Lanes lanes(split);
        uint32_t off_last[4] = {}, off[4] = {};
        int t = 0, cls = e0.y >> 8;
        auto issue_dK = [&](int it, const uint32_t (&skip)[4]) {
            if (!wait(kDS, it)) return false;
            mma_sums<D, JOINED>(c.tmem + kTDK, c.tmem + kTDS, q(it), skip, it > 0, go);
            tc::commit_go(c.bar(kQe + it % kStages), go);
            return true;
        };
        bool ok = iters > 0 && wait(kKV, 0) && wait(kQf, 0);
        if (ok) issue_S(0);
        auto issue_dP = [&](int it) {
            mma_rows<D>(tDP, c.base + kOffV, o(it), go);
            mma_ext(tDP, c.base + kOffOne, ext(it) + kExtBlock, c.base + kOffZero, go);
            tc::commit_go(c.bar(kDP), go);
        };
        for (int it = 0; ok && it < iters; ++it) {
            const bool more = it + 1 < iters;
            if (JOINED) {
                lanes.off(cls, off);
                if (++t == nt) t = 0;
                if (more) cls = tile(t).y >> 8;
            }
            if (!wait(kOf + it % kStages, it / kStages)) break;
            if (D == 64) {
                if (it > 0 && !wait(kDPread, it - 1)) break;
                issue_dP(it);
                if (more) {
                    if (!wait(kQf + (it + 1) % kStages, (it + 1) / kStages) || !wait(kSread, it)) break;
                    issue_S(it + 1);
                }
                if (it > 0 && !issue_dK(it - 1, off_last)) break;
            } else {
                if (!wait(kSread, it)) break;
                issue_dP(it);
                if (it > 0 && !issue_dK(it - 1, off_last)) break;
                if (more) {
                    if (!wait(kQf + (it + 1) % kStages, (it + 1) / kStages) || !wait(kDPread, it)) break;
                    issue_S(it + 1);
                }
            }
            if (!wait(kP, it)) break;
            mma_sums<D, JOINED>(c.tmem + kTDV, c.tmem + kTP, o(it), off, it > 0, go);
            tc::commit_go(c.bar(kOe + it % kStages), go);
            if (!more) issue_dK(it, off);
#pragma unroll
            for (int i = 0; i < 4; ++i) off_last[i] = off[i];
        }
        // every issued MMA completes before the sums are read and TMEM is released; a raised abort flag is seen first
        __threadfence_block();
        tc::commit_go(c.bar(kDone), go);
        int never = 0;
        tc::mbar_wait(c.bar(kDone), 0, &never);
    } else {
        const int w = c.warp >> 2, r = threadIdx.x & 127;
        const uint32_t lane_off = (uint32_t)((c.warp & 3) * 32) << 16;
        const uint32_t tS = c.tmem + kTS + W::kCols * w + lane_off, tDP = c.tmem + L::kTDP + W::kCols * w + lane_off;
        const uint32_t tP = c.tmem + kTP + W::kCols / 2 * w + lane_off, tDS = c.tmem + kTDS + W::kCols / 2 * w + lane_off;
        const uint64_t cc = pk2(p.scale_log2, p.scale_log2);
        // the first sums into a lane need not be the tile's first: all start from zero, before this thread says
        // that it has written P
        if (JOINED) zero_cols<2 * D / W::kWgs>(c.tmem + kTDV + 2 * D / W::kWgs * w + lane_off);
        // even warpgroups store dV, odd ones dK, each its share of the row's columns; many short streams: where to
        // is read beforehand (8192 tokens x 24 heads, 22% kept: 719 us without, 705 with; dense 272 and 276)
        constexpr int kN = D / (W::kWgs / 2);
        const int is_dk = w & 1, col = (w >> 1) * kN;
        auto place = [&] { return out_row<D>(is_dk ? p.dK : p.dV, p.kperm, z, p.N, klo + r, r < kn, z, p.status); };
        bf16* const early = JOINED ? place() : nullptr;
        bool ok = true;
        for (int it = 0; it < iters; ++it) {
            if (!__all_sync(kFull, tc::mbar_wait(c.bar(kS), it & 1, c.abort_flag))) { ok = false; break; }
            tc::fence_after_sync();
            uint32_t pv[W::kH][32];
            load_cols(tS, pv);
            tc::fence_before_sync();
            tc::mbar_arrive(c.bar(kSread));
#pragma unroll
            for (int h = 0; h < W::kH; ++h)
#pragma unroll
                for (int i = 0; i < 32; i += 2)
                    ex2_pair(mul2(pk2(__uint_as_float(pv[h][i]), __uint_as_float(pv[h][i + 1])), cc), i / 2, pv[h][i],
                             pv[h][i + 1]);
            // P(it) and dS(it) follow P(it - 1) and dS(it - 1) once dV and dK have taken those in
            const int prev = (it - 1) % kStages, phase = ((it - 1) / kStages) & 1;
            if (it > 0 && !__all_sync(kFull, tc::mbar_wait(c.bar(kOe + prev), phase, c.abort_flag))) { ok = false; break; }
            tc::fence_after_sync();
#pragma unroll
            for (int h = 0; h < W::kH; ++h) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) pk[e] = bf16x2(__uint_as_float(pv[h][2 * e]), __uint_as_float(pv[h][2 * e + 1]));
                tc::tmem_st16(tP + 16 * h, pk);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(c.bar(kP));
            if (!__all_sync(kFull, tc::mbar_wait(c.bar(kDP), it & 1, c.abort_flag))) { ok = false; break; }
            tc::fence_after_sync();
            uint32_t dv[W::kH][32];
            load_cols(tDP, dv);
            tc::fence_before_sync();
            tc::mbar_arrive(c.bar(kDPread));
#pragma unroll
            for (int h = 0; h < W::kH; ++h)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float x0, x1;
                    up2(mul2(pk2(__uint_as_float(dv[h][2 * e]), __uint_as_float(dv[h][2 * e + 1])),
                             pk2(__uint_as_float(pv[h][2 * e]), __uint_as_float(pv[h][2 * e + 1]))),
                        x0, x1);
                    pv[h][e] = bf16x2(x0, x1);      // over columns that have been used
                }
            if (it > 0 && !__all_sync(kFull, tc::mbar_wait(c.bar(kQe + prev), phase, c.abort_flag))) { ok = false; break; }
            tc::fence_after_sync();
#pragma unroll
            for (int h = 0; h < W::kH; ++h) tc::tmem_st16(tDS + 16 * h, pv[h]);
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(c.bar(kDS));
        }
        if (sums_complete(c, ok, kDone)) {
            const uint32_t acc = c.tmem + (is_dk ? kTDK : kTDV) + col + lane_off;
            // the streamed tiles have all been used: their buffers take the rows
            unsigned char* stage = c.sbase + kOffBuf + c.warp * (32 * kN * 4);
            static_assert(4 * W::kWgs * 32 * kN * 4 <= 8 * kRegion, "staging");
            if (PARTS && p.kv_parts > 1) {
                const long long row = (part * 2 + is_dk) * p.krows + (long long)z * p.N + klo + r;
                store_acc_rows<kN, float>(acc, stage, c.lane, 1.f, iters == 0, r < kn ? p.kv_part + row * D + col : nullptr);
            } else {
                bf16* out = JOINED ? early : place();
                store_acc_rows<kN, bf16>(acc, stage, c.lane, is_dk ? p.scale : 1.f, iters == 0, out ? out + col : nullptr);
            }
        }
    }
    cta_finish(c, p.status);
}

// ---------------------------------------------------------------- dQ
// One CTA per 128-query tile of a query head, streaming the (K, V) tiles of its kept keys. Per
// tile, with queries in the TMEM lanes: S = Q K^T -> P;  dP = dO V^T -> dS;  dQ += dS K. S(j+1) is
// issued as soon as S(j) has been read, dP(j+1) as soon as dP(j) has.
namespace dq {
constexpr int kKStages = 3, kVStages = 2;
constexpr int kOffQ = 0, kOffO = 2 * kRegion, kOffK = 4 * kRegion, kOffV = kOffK + kKStages * 2 * kRegion,
              kOffBar = kOffV + kVStages * 2 * kRegion;
enum { kQO = 0, kKf = 1, kVf = kKf + kKStages, kKe = kVf + kVStages, kVe = kKe + kKStages, kS = kVe + kVStages, kDP, kDSfree,
       kDone, kLand, kSread, kDPread, kDS, kBars };
constexpr int kSmem = kOffBar + 8 * kBars + 16 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr uint32_t kTS = 0, kTDP = 128, kTDQ = 256, kTDS = 384, kTDSlow = 448;
}  // namespace dq

// With SPLIT dS enters dQ as two bf16 parts (16 bits), an eighth product; the second has the last 64 TMEM columns.
template <int D, bool PARTS, bool JOINED, bool SPLIT>
__device__ __forceinline__ void dq_tile(const BwdMaps& m, const BwdParams& p, unsigned char* smem_raw, int x, int pair, int part) {
    using namespace dq;
    using W = Warps<D>;
    const int z = x / p.g;
    int grp, qlo, qn, split, count;
    if (!find_tile(p.qtile, z, p.q_tiles, p.N, pair, grp, qlo, qn, split, count)) return;
    const int2* list = p.klist + ((long long)z * p.Gq + grp) * p.kcap;
    // this CTA's share of the key tiles
    const int all = JOINED ? count : p.kcnt ? p.kcnt[(long long)z * p.Gq + grp] : (p.N + kTile - 1) / kTile;
    const int first = PARTS ? (int)((long long)all * part / p.q_parts) : 0;
    const int nt = PARTS ? (int)((long long)all * (part + 1) / p.q_parts) - first : all;
    auto tile = [&](int t) {
        t += first;
        return p.kcnt ? list[t] : make_int2(t * kTile, min(kTile, p.N - t * kTile));
    };
    const int2 e0 = JOINED && nt > 0 ? tile(0) : make_int2(0, 0);
    const Cta c = cta_setup<D>(
        smem_raw, kOffBar, kBars, p.status, [](int i) { return i >= kSread ? W::kArrivals : 1; },
        [&](const Cta& c) {
            if (p.stall) return;
            tc::mbar_arrive_expect_tx(c.bar(kQO), 2 * (D / 64) * kRegion);
            for (int h = 0; h < D / 64; ++h) {
                tc::tma_load_2d(c.base + kOffQ + h * kRegion, &m.q, c.bar(kQO), 64 * h, x * p.N + qlo);
                tc::tma_load_2d(c.base + kOffO + h * kRegion, &m.o, c.bar(kQO), 64 * h, x * p.N + qlo);
            }
        });

    if (c.warp == W::kTma) {
        int nland = 0, nk = 0, nv = 0;
        int2 next = e0;
        for (int t = 0; t < nt; ++t) {
            int2 e = JOINED ? next : tile(t);
            if (JOINED) {
                e.y &= 255;
                if (t + 1 < nt) next = tile(t + 1);
            }
            const int sk = t % kKStages, sv = t % kVStages, row = z * p.N + e.x;
            if (t >= kKStages && !__all_sync(kFull, tc::mbar_wait(c.bar(kKe + sk), (t / kKStages - 1) & 1, c.abort_flag))) break;
            if (!load_tile_zeroed<D>(c, c.base + kOffK + sk * 2 * kRegion, &m.k, kKf + sk, kLand, nland, row, e.y)) break;
            nk = t + 1;
            if (t >= kVStages && !__all_sync(kFull, tc::mbar_wait(c.bar(kVe + sv), (t / kVStages - 1) & 1, c.abort_flag))) break;
            if (!load_tile_zeroed<D>(c, c.base + kOffV + sv * 2 * kRegion, &m.v, kVf + sv, kLand, nland, row, e.y)) break;
            nv = t + 1;
        }
        int never = 0;
        for (int i = max(0, nk - kKStages); i < nk; ++i) tc::mbar_wait(c.bar(kKf + i % kKStages), (i / kKStages) & 1, &never);
        for (int i = max(0, nv - kVStages); i < nv; ++i) tc::mbar_wait(c.bar(kVf + i % kVStages), (i / kVStages) & 1, &never);
        if (!p.stall) tc::mbar_wait(c.bar(kQO), 0, &never);
    } else if (c.warp == W::kMma) {
        const uint32_t go = tc::elect_one();
        auto wait = [&](int b, int parity) {
            const bool ok = __all_sync(kFull, tc::mbar_wait(c.bar(b), parity & 1, c.abort_flag));
            tc::fence_after_sync();
            return ok;
        };
        auto k = [&](int t) { return c.base + kOffK + (t % kKStages) * 2 * kRegion; };
        auto v = [&](int t) { return c.base + kOffV + (t % kVStages) * 2 * kRegion; };
        auto issue_S = [&](int t) {
            if (!wait(kKf + t % kKStages, t / kKStages)) return false;
            mma_rows<D>(c.tmem + kTS, c.base + kOffQ, k(t), go);
            tc::commit_go(c.bar(kS), go);
            return true;
        };
        auto issue_dP = [&](int t) {
            if (!wait(kVf + t % kVStages, t / kVStages)) return false;
            mma_rows<D>(c.tmem + kTDP, c.base + kOffO, v(t), go);
            tc::commit_go(c.bar(kDP), go);
            tc::commit_go(c.bar(kVe + t % kVStages), go);
            return true;
        };
        const Lanes lanes(split);
        uint32_t off[4] = {};
        int cls = e0.y >> 8;
        bool ok = nt > 0 && wait(kQO, 0) && issue_S(0) && issue_dP(0);
        for (int t = 0; ok && t < nt; ++t) {
            if (JOINED) {
                lanes.off(cls, off);
                if (t + 1 < nt) cls = tile(t + 1).y >> 8;
            }
            if (t + 1 < nt && !(wait(kSread, t) && issue_S(t + 1) && wait(kDPread, t) && issue_dP(t + 1))) break;
            if (!wait(kDS, t)) break;
            mma_sums<D, JOINED>(c.tmem + kTDQ, c.tmem + kTDS, k(t), off, t > 0, go);
            if (SPLIT) mma_sums<D, JOINED>(c.tmem + kTDQ, c.tmem + kTDSlow, k(t), off, true, go);
            tc::commit_go(c.bar(kKe + t % kKStages), go);
            tc::commit_go(c.bar(kDSfree), go);
        }
        __threadfence_block();
        tc::commit_go(c.bar(kDone), go);
        int never = 0;
        tc::mbar_wait(c.bar(kDone), 0, &never);
    } else {
        const int w = c.warp >> 2, r = threadIdx.x & 127;
        const uint32_t lane_off = (uint32_t)((c.warp & 3) * 32) << 16;
        const uint32_t tS = c.tmem + kTS + W::kCols * w + lane_off, tDP = c.tmem + kTDP + W::kCols * w + lane_off;
        const uint32_t tDS = c.tmem + kTDS + W::kCols / 2 * w + lane_off;
        const long long row = (long long)x * p.N + qlo + r;
        const float nl = r < qn ? p.nlse2[row] : -INFINITY, nd = r < qn ? p.nD[row] : 0.f;
        auto place = [&] { return out_row<D>(p.dQ, p.qperm, x, p.N, qlo + r, r < qn, z, p.status); };
        bf16* const early = JOINED ? place() : nullptr;      // as in the other pass
        const uint64_t cc = pk2(p.scale_log2, p.scale_log2), nl2 = pk2(nl, nl), nd2 = pk2(nd, nd);
        bool ok = true;
        if (JOINED && w < 2) zero_cols<D / 2>(c.tmem + kTDQ + D / 2 * w + lane_off);
        int valid_next = JOINED ? e0.y : nt > 0 ? tile(0).y : 0;
        for (int t = 0; t < nt; ++t) {
            const int valid = JOINED ? valid_next & 255 : valid_next;
            if (t + 1 < nt) valid_next = tile(t + 1).y;
            if (!__all_sync(kFull, tc::mbar_wait(c.bar(kS), t & 1, c.abort_flag))) { ok = false; break; }
            tc::fence_after_sync();
            uint32_t pv[W::kH][32], pk[16 * W::kH], low[16 * W::kH];
            load_cols(tS, pv);
            tc::fence_before_sync();
            tc::mbar_arrive(c.bar(kSread));
#pragma unroll
            for (int h = 0; h < W::kH; ++h) {
#pragma unroll
                for (int i = 0; i < 32; i += 2)
                    ex2_pair(fma2(pk2(__uint_as_float(pv[h][i]), __uint_as_float(pv[h][i + 1])), cc, nl2), i / 2, pv[h][i],
                             pv[h][i + 1]);
                if (valid < kTile) {      // keys past the tile's end
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (W::kCols * w + 32 * h + i >= valid) pv[h][i] = 0u;
                }
            }
            if (!__all_sync(kFull, tc::mbar_wait(c.bar(kDP), t & 1, c.abort_flag))) { ok = false; break; }
            tc::fence_after_sync();
            uint32_t dv[W::kH][32];
            load_cols(tDP, dv);
            tc::fence_before_sync();
            tc::mbar_arrive(c.bar(kDPread));
#pragma unroll
            for (int h = 0; h < W::kH; ++h) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float x0, x1;
                    up2(mul2(add2(pk2(__uint_as_float(dv[h][2 * e]), __uint_as_float(dv[h][2 * e + 1])), nd2),
                             pk2(__uint_as_float(pv[h][2 * e]), __uint_as_float(pv[h][2 * e + 1]))),
                        x0, x1);
                    pk[16 * h + e] = bf16x2(x0, x1);
                    if (SPLIT) low[16 * h + e] = bf16x2_rest(x0, x1, pk[16 * h + e]);
                }
            }
            if (t > 0 && !__all_sync(kFull, tc::mbar_wait(c.bar(kDSfree), (t - 1) & 1, c.abort_flag))) { ok = false; break; }
            tc::fence_after_sync();
            if (W::kH == 2) tc::tmem_st32(tDS, pk);
            else tc::tmem_st16(tDS, pk);
            if (SPLIT && W::kH == 2) tc::tmem_st32(tDS + kTDSlow - kTDS, low);
            if (SPLIT && W::kH == 1) tc::tmem_st16(tDS + kTDSlow - kTDS, low);
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(c.bar(kDS));
        }
        // the first two warpgroups store half of the row's columns each
        constexpr int kN = D / 2;
        if (w < 2 && sums_complete(c, ok, kDone)) {
            const uint32_t acc = c.tmem + kTDQ + w * kN + lane_off;
            unsigned char* stage = c.sbase + kOffK + c.warp * (32 * kN * 4);     // as in the other pass
            static_assert(8 * 32 * kN * 4 <= (kKStages + kVStages) * 2 * kRegion, "staging");
            if (PARTS && p.q_parts > 1) {
                float* sums = p.q_part + (part * p.qrows + (long long)x * p.N + qlo + r) * D + w * kN;
                store_acc_rows<kN, float>(acc, stage, c.lane, 1.f, nt == 0, r < qn ? sums : nullptr);
            } else {
                bf16* out = JOINED ? early : place();
                store_acc_rows<kN, bf16>(acc, stage, c.lane, p.scale, nt == 0, out ? out + w * kN : nullptr);
            }
        }
    }
    cta_finish(c, p.status);
}

// Both passes in one launch: the CTAs of dK and dV come first, being the longer ones, and those of dQ
// fill the SMs that they leave idle at their end; where that ends sooner, some of dQ go before the last of
// dK and dV.
template <int D>
constexpr int kSmemBytes = kv::Layout<D>::kSmem > dq::kSmem ? kv::Layout<D>::kSmem : dq::kSmem;

template <int D, bool PARTS, bool JOINED, bool SPLIT>
__global__ void __launch_bounds__(Warps<D>::kThreads, 1) bwd_kernel(const __grid_constant__ BwdMaps m, const __grid_constant__ BwdParams p) {
    extern __shared__ unsigned char smem_raw[];
    const int b = blockIdx.x, early = b - p.kv_first;
    if (early < 0 || (early >= p.q_early && b < p.kv_blocks + p.q_early)) {
        const int i = early < 0 ? b : b - p.q_early, t = PARTS ? i / p.kv_parts : i;
        dkv_tile<D, PARTS, JOINED>(m, p, smem_raw, t / p.kv_tiles, t % p.kv_tiles, PARTS ? i % p.kv_parts : 0);
    } else {
        const int i = early < p.q_early ? early : b - p.kv_blocks, t = PARTS ? i / p.q_parts : i;
        dq_tile<D, PARTS, JOINED, SPLIT>(m, p, smem_raw, t / p.q_tiles, t % p.q_tiles, PARTS ? i % p.q_parts : 0);
    }
}

// Sums of the parts in their order, scaled, rounded and written to the output rows: D / 8 threads a row. After a
// timeout, in this call or one not yet read, sums may be missing and nothing is written.
template <int D>
__global__ void __launch_bounds__(256) bwd_join_kernel(const __grid_constant__ BwdParams p) {
    const int before = *reinterpret_cast<const volatile int*>(p.status);       // looked at last, beside the sums' loads
    const long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    long long row = t / (D / 8);
    const int col = (int)(t % (D / 8)) * 8;
    const long long kv = p.kv_parts > 1 && p.dK ? 2 * p.krows : 0;
    const bool q = row >= kv;
    if (q) row -= kv;
    if (q && (p.q_parts <= 1 || !p.dQ || row >= p.qrows)) return;
    const int parts = q ? p.q_parts : p.kv_parts;
    const bool is_dv = !q && row < p.krows;
    const long long step = (q ? p.qrows : 2 * p.krows) * D, own = q || is_dv ? row : row - p.krows;
    const long long head = own / p.N, z = q ? head / p.g : head;
    const int pos = (int)(own % p.N);
    const bool loose = p.loose && p.loose[2 * z + !q];
    const float* src = (q ? p.q_part : p.kv_part) + row * D + col;
    float s[8] = {};
    for (int i = 0; i < parts; ++i, src += step) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(src)), b = __ldg(reinterpret_cast<const float4*>(src) + 1);
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += v[e];
    }
    const float scale = is_dv ? 1.f : p.scale;
    if (loose) {        // only rows that a tile holds have sums (bad offsets alone come here)
        const int4* tile = q ? p.qtile + z * p.q_tiles : p.ktile + z * p.kv_tiles;
        bool held = false;
        for (int i = 0; i < (q ? p.q_tiles : p.kv_tiles); ++i) held |= pos >= tile[i].y && pos < tile[i].y + tile[i].z;
        if (!held) return;
    }
    bf16* out = out_row<D>(q ? p.dQ : is_dv ? p.dV : p.dK, q ? p.qperm : p.kperm, head, p.N, pos, true, z, p.status);
    if (!out || before == kDevTimeout) return;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = bf16x2(s[2 * e] * scale, s[2 * e + 1] * scale);
    *reinterpret_cast<uint4*>(out + col) = make_uint4(w[0], w[1], w[2], w[3]);
}

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

// Byte offsets of the workspace's parts.
struct BwdLayout {
    size_t nlse2, nD, kv_part, q_part, klist, qlist, kcnt, qcnt, qtile, ktile, loose, bytes;
    int kcap, qcap;
};

BwdLayout bwd_layout(int P, int g, int N, int d, int Gq, int Gk, const BwdParts& parts, bool sparse) {
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
    if (parts.kv > 1) l.kv_part = take((size_t)parts.kv * 2 * P * N * d * sizeof(float));
    if (parts.q > 1) l.q_part = take((size_t)parts.q * P * g * N * d * sizeof(float));
    if (sparse) {
        // the runs of a list are disjoint: at most N / 128 full tiles and one ragged tile per group
        l.kcap = (int)(tiles + Gk);
        l.qcap = (int)(tiles + Gq);
        const size_t lists = (size_t)P * (parts.joined ? 2 : 1);
        l.klist = take(lists * Gq * l.kcap * sizeof(int2));
        l.qlist = take(lists * Gk * l.qcap * sizeof(int2));
        l.kcnt = take(lists * Gq * sizeof(int32_t));
        l.qcnt = take(lists * Gk * sizeof(int32_t));
        l.qtile = take((size_t)P * l.qcap * sizeof(int4));
        l.ktile = take((size_t)P * l.kcap * sizeof(int4));
        l.loose = take((size_t)P * 2 * sizeof(int32_t));
    }
    l.bytes = at + 240;      // the parts start on 256 bytes, the workspace on 16
    return l;
}

template <int D>
cudaError_t launch_bwd(const AttnBwdArgs& a, cudaStream_t s) {
    const bool sparse = a.rowptr != nullptr;
    const BwdLayout l = bwd_layout(a.P, a.g, a.N, D, a.Gq, a.Gk, a.parts, sparse);
    char* ws = reinterpret_cast<char*>(align256(reinterpret_cast<uintptr_t>(a.workspace)));
    float *nlse2 = reinterpret_cast<float*>(ws + l.nlse2), *nD = reinterpret_cast<float*>(ws + l.nD);
    const long long rows = (long long)a.P * a.g * a.N, krows = (long long)a.P * a.N;
    BwdParams p;
    memset(&p, 0, sizeof(p));
    p.nlse2 = nlse2; p.nD = nD;
    p.dQ = a.dQ; p.dK = a.dK; p.dV = a.dV;
    p.krows = krows; p.qrows = rows;
    p.N = a.N; p.g = a.g; p.Gq = 1; p.Gk = 1;
    p.kv_parts = a.parts.kv; p.q_parts = a.parts.q;
    p.kv_part = reinterpret_cast<float*>(ws + l.kv_part); p.q_part = reinterpret_cast<float*>(ws + l.q_part);
    p.status = a.status;
    p.stall = a.stall;
    p.scale = (float)(1.0 / sqrt((double)D));
    p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
    const int tiles = (a.N + kTile - 1) / kTile;
    p.kv_tiles = tiles + (sparse ? a.Gk : 0);
    p.q_tiles = tiles + (sparse ? a.Gq : 0);
    ListParams lp;
    memset(&lp, 0, sizeof(lp));
    int list_blocks = 0;
    if (sparse) {
        lp.rowptr = a.rowptr; lp.kg = a.kg; lp.qoff = a.qoff; lp.koff = a.koff;
        lp.klist = reinterpret_cast<int2*>(ws + l.klist); lp.qlist = reinterpret_cast<int2*>(ws + l.qlist);
        lp.kcnt = reinterpret_cast<int32_t*>(ws + l.kcnt); lp.qcnt = reinterpret_cast<int32_t*>(ws + l.qcnt);
        lp.qtile = reinterpret_cast<int4*>(ws + l.qtile);
        lp.ktile = reinterpret_cast<int4*>(ws + l.ktile);
        lp.loose = reinterpret_cast<int32_t*>(ws + l.loose);
        lp.q_tiles = p.q_tiles; lp.kv_tiles = p.kv_tiles;
        lp.status = a.status;
        lp.kcap = l.kcap; lp.qcap = l.qcap; lp.P = a.P; lp.N = a.N; lp.Gq = a.Gq; lp.Gk = a.Gk;
        lp.g = a.g; lp.joined = a.parts.joined;
        const long long warps = (long long)a.P * (a.parts.joined ? 2 * (a.Gq + a.Gk) : a.Gq + a.Gk + 2);
        list_blocks = (int)((warps * 32 + 255) / 256);
        if (a.parts.joined) {
            bwd_lists_kernel<<<list_blocks, 256, 0, s>>>(lp);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
            list_blocks = 2 * a.P;
        }
        p.qperm = a.qperm; p.kperm = a.kperm;
        p.klist = lp.klist; p.qlist = lp.qlist; p.kcnt = lp.kcnt; p.qcnt = lp.qcnt;
        p.qtile = lp.qtile; p.ktile = lp.ktile;
        p.loose = lp.loose;
        p.kcap = l.kcap; p.qcap = l.qcap;
        p.Gq = a.parts.joined ? 2 * a.Gq : a.Gq; p.Gk = a.parts.joined ? 2 * a.Gk : a.Gk;
    }
    const long long row_blocks = (rows * (D / 8) + 255) / 256;
    bwd_prepare_kernel<D><<<(unsigned)(list_blocks + row_blocks), 256, 0, s>>>(
        lp, list_blocks, reinterpret_cast<const uint4*>(a.O), reinterpret_cast<const uint4*>(a.dO), a.lse, nlse2, nD, rows);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    BwdMaps m;
    if (!make_tmap_bf16_sw128(&m.q, a.Q, rows, D, kTile, 64) || !make_tmap_bf16_sw128(&m.k, a.K, krows, D, kTile, 64) ||
        !make_tmap_bf16_sw128(&m.v, a.V, krows, D, kTile, 64) || !make_tmap_bf16_sw128(&m.o, a.dO, rows, D, kTile, 64))
        return cudaErrorInvalidValue;
    p.kv_blocks = a.dK ? p.kv_tiles * a.P * p.kv_parts : 0;
    const long long blocks = p.kv_blocks + (a.dQ ? (long long)p.q_tiles * a.P * a.g * p.q_parts : 0);
    const bool both = a.dK && a.dQ;
    p.kv_first = both ? p.kv_blocks - a.parts.kv_late : p.kv_blocks;
    p.q_early = both ? a.parts.q_early : 0;
    const bool parts = p.kv_parts > 1 || p.q_parts > 1;
    const int variant = parts ? 1 : a.parts.joined ? 2 : 0, bit = 1 << (variant + (a.split ? 3 : 0));
    static decltype(&bwd_kernel<D, false, false, false>) const kernels[2][3] = {
        {bwd_kernel<D, false, false, false>, bwd_kernel<D, true, false, false>, bwd_kernel<D, false, true, false>},
        {bwd_kernel<D, false, false, true>, bwd_kernel<D, true, false, true>, bwd_kernel<D, false, true, true>}};
    const auto kernel = kernels[a.split][variant];
    if (!(*a.attributes & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<D>);
        if (e != cudaSuccess) return e;
        *a.attributes |= bit;
    }
    kernel<<<(unsigned)blocks, Warps<D>::kThreads, kSmemBytes<D>, s>>>(m, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const long long join = (p.kv_parts > 1 && a.dK ? 2 * krows : 0) + (p.q_parts > 1 && a.dQ ? rows : 0);
    if (join) bwd_join_kernel<D><<<(unsigned)((join * (D / 8) + 255) / 256), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

// How many CTAs share a tile's stream, and the order of the launch: what a model of it expects to end
// first. An SM runs one CTA at a time, in launch order. Times in microseconds at 1.9 GHz, fitted to whole
// launches: 1.42 for a dK/dV tile, 1.0 for a dQ tile, 2.5 for a CTA's start and end; the join of the parts'
// sums takes 2.5 for its launch and 1 per 4 MB written and read back. Few CTAs with long streams gain most, and a number of
// CTAs just past a multiple of the SMs is stepped over. On the device, whole against shared (d = 128, one
// sample): 4 query heads on 1 KV head, 1000 tokens 54 against 17 us; 3 on 1, 4096 tokens 142 against 85;
// 12 heads, 1024 tokens 30 against 45 (left whole). The times are those of d = 128. At d = 64 a tile takes 0.7 to
// 0.8 of them, which moves few borders, and the choices hold: 39 against 17 us, 103 against 62, 24 (left whole)
// against 28; 2 heads, 1300 tokens 17.5 against 15.1; 1 head, 8192 tokens 72 (left whole) against 105.
struct BwdModel {
    double nk, nq, tk, tq;                  // CTAs of dK and dV, of dQ; their times
    int sms;
    // The end of the launch if `m` SMs go on to dQ a turn of dK and dV before the others.
    double end(double m) const {
        const double whole = floor(nk / sms), rest = nk - whole * sms;
        // SMs, and when they turn to dQ
        const double n[3] = {m, sms - 2 * m - rest, rest + m}, at[3] = {(whole - 1) * tk, whole * tk, (whole + 1) * tk};
        double t = fmax((nk * tk + nq * tq) / sms, n[2] > 0 ? at[2] : at[1]);
        for (int i = 0; i < 64; ++i) {
            double fit = 0, next = 1e30;
            for (int c = 0; c < 3; ++c) {
                if (n[c] <= 0) continue;
                const double ran = floor((t - at[c]) / tq + 1e-6);
                fit += n[c] * fmax(ran, 0.0);
                next = fmin(next, at[c] + (ran + 1) * tq);
            }
            if (fit >= nq) break;
            t = next;       // on to the next end of a dQ CTA
        }
        return t;
    }
};

BwdParts attn_bwd_parts(int P, int g, int N, int d, int Gq, int Gk, bool sparse, int sms) {
    BwdParts best = {1, 1, 0, 0, false};
    const double tiles = (N + kTile - 1) / kTile;
    // of a route neither the density nor the groups' sizes are known here: a quarter of the keys, and
    // a quarter more tiles than whole ones
    const double len = sparse ? ceil(tiles / 4) : tiles, ctas = sparse ? ceil(1.25 * tiles) : tiles;
    // Joined tiles take a launch more. They pay where the tiles fill the SMs, and where groups have some rows.
    auto joined = [&](const BwdParts& b) { return sparse && b.kv == 1 && b.q == 1 && P * (tiles + Gk) > sms && N >= 32 * max(Gq, Gk); };
    best.joined = joined(best);
    if (ctas * P > 8.0 * sms) return best;
    static const int kChoices[] = {1, 2, 3, 4, 6, 8, 12, 16};
    double best_t = 1e30;
    for (int kv : kChoices)
        for (int q : kChoices) {
            if ((kv > 1 && kv > len * g) || (q > 1 && q > len)) continue;
            const BwdModel w = {ctas * P * kv, ctas * P * g * q, 1.42 * ceil(len * g / kv) + 2.5, ceil(len / q) + 2.5, sms};
            double t = w.end(0);
            const double mb = 4e-6 * d * N * (double)P * ((kv > 1 ? 2.0 * kv : 0) + (q > 1 ? (double)g * q : 0));
            if (kv > 1 || q > 1) t += 2.5 + 2 * mb / 4;
            if (t < best_t * 0.97) {      // a gain below the model's error is none
                best_t = t;
                best = {kv, q, 0, 0, false};
            }
        }
    best.joined = joined(best);
    // The order, for equal streams: m SMs turn to dQ before their last CTA of dK and dV, m others run one
    // more of those (12 heads, 4096 tokens: 277 -> 271 us with m = 28; 16 on 4 heads, 2 x 2311: 257 -> 252 with
    // 32; at d = 64 208 -> 205 and 192.2 -> 191.0). Here the times are those of steady tiles and of whole CTAs at
    // d = 128, by clock reads in long launches.
    if (!sparse && best.kv == 1 && best.q == 1) {
        const BwdModel w = {ctas * P, ctas * P * g, 1.35 * len * g + 4.4, 0.98 * len + 3.1, sms};
        const int rest = (int)w.nk % sms, each = (int)ceil(w.tk / w.tq);
        best_t = w.end(0);
        for (int m = 1; w.nk >= sms && rest + 2 * m <= sms && (double)m * each <= w.nq; ++m) {
            const double t = w.end(m);
            if (t < best_t * 0.995) {
                best_t = t;
                best.kv_late = rest + m;
                best.q_early = m * each;
            }
        }
    }
    return best;
}

size_t attn_bwd_workspace(int P, int g, int N, int d, int Gq, int Gk, const BwdParts& parts, bool sparse) {
    return bwd_layout(P, g, N, d, Gq, Gk, parts, sparse).bytes;
}

int attn_bwd_launches(const AttnBwdArgs& a) { return 2 + (a.rowptr && a.parts.joined) + ((a.dK && a.parts.kv > 1) || (a.dQ && a.parts.q > 1)); }

cudaError_t launch_attn_bwd(const AttnBwdArgs& a, cudaStream_t s) {
    return a.d == 128 ? launch_bwd<128>(a, s) : a.d == 64 ? launch_bwd<64>(a, s) : cudaErrorInvalidValue;
}

}  // namespace spr

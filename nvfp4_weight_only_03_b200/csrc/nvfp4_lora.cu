// Low-rank adapters of many requests beside a shared projection (nvfp4_lora_add):
//
//   out[m] = bf16( y[m] + scale_a * B_a (A_a x[m]) ),   a = index[m];  out[m] = y[m] without one
//
// * Two kernels: the first forms T = A x (rank values per row), the second adds B T.  Rows that
//   share an adapter form a group, found from `index` by every CTA itself (at most 128 rows), so
//   each adapter leaves HBM once and the host needs no copy of the index.
// * HBM bound: rank * (K + N) bf16 per adapter against a few rows.  The weights go from global
//   memory straight into mma.sync fragments, 16 bytes per lane and load: k (and the rank) may be
//   permuted as long as both operands are, so a lane's 8 consecutive values serve as the 4 pairs
//   of two MMAs, and no shared-memory pass is needed.  tcgen05 would have to stage them.
// * First kernel: weights are the 16 rows of the MMA, x rows its 8 columns; a cluster of up to 8 CTAs
//   takes (group, 16 ranks), splits K over its warps and adds their sums in order through distributed
//   shared memory.  Second kernel: output channels are the MMA's rows, permuted so that a lane ends
//   up with 4 consecutive ones, and T rows its columns; a warp per (group, 32 channels) and many warps,
//   so that others load while one multiplies.
// * T leaves the first kernel as two bf16 values (high and remainder), scaled, so it is carried to
//   2^-17; the only other rounding is the output's.
// * The second kernel is launched while the first runs and has its groups, its first weights and y
//   before it waits for T.
// * Measured (B200, calls of a captured graph): 128 rows over 48 adapters of rank 64, 10240 x 5120:
//   23.8 us, 3.9 TB/s, 60% of the copy rate (two kernels of 5 and 9 us of traffic, each with its
//   start and its last wave); one row of rank 16: 5.6 us, latency alone.  One kernel with a cluster
//   per 16 rows of a group for both products took 36.5 and 8.2 us: eight SMs per adapter draw too
//   little.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "nvfp4.h"
#include "nvfp4_host.h"

namespace {

using nvfp4_host::misaligned;
using nvfp4_host::overlaps;

constexpr int kDownWarps = 8, kDownThreads = kDownWarps * 32;
constexpr int kWarps = 4, kThreads = kWarps * 32;  // of the second kernel
constexpr int kMaxM = NVFP4_MAX_ROWS;
constexpr int kMaxRank = NVFP4_LORA_MAX_RANK;
constexpr int kChunkN = kWarps * 32;  // output channels per item of the second kernel
constexpr int kColTiles = 2;          // tiles of 8 rows that share one pass over A
constexpr int kStepK = 128;           // k of one step of a warp: 16 rows of A, 4 KB

struct Params {
    const uint16_t* a;
    int64_t a_stride, a_ld;  // adapter, rank row
    const uint16_t* b;
    int64_t b_stride, b_ld;  // adapter, output channel
    const float* scales;
    const int32_t* ranks;  // or null: all `rank`
    const int32_t* index;
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* y;
    int64_t ldy;
    uint16_t* out;
    int64_t ldo;
    uint16_t* t;  // T: [m][2][rank32] bf16, values and remainders
    int m, adapters, rank, rank16, rank32, n, k;
};

// Rows by adapter: `row` lists the rows group by group; group g is adapter[g], its rows are
// row[first[g]] .. row[first[g + 1] - 1].  Rows without an adapter are a last group of rank 0.
struct Groups {
    int count;
    int16_t adapter[kMaxM + 1], rank[kMaxM + 1], first[kMaxM + 2], row[kMaxM];
    int16_t lead[kMaxM + 1];  // by leading row (kMaxM: none): its group's first place in `row`
    __align__(16) int32_t index[kMaxM];
};

// Thread t (< kMaxM) places row t.  One pass over the indexes gives it the set of rows with its
// adapter, as bits: the first of them leads the group, and prefix sums over the leaders' sizes place
// the groups.
__device__ __forceinline__ void find_groups(const Params& p, Groups& g) {
    static_assert(kThreads >= kMaxM && kDownThreads >= kMaxM, "a thread per row");
    __shared__ int32_t warp_sum[kMaxM / 32], warp_lead[kMaxM / 32];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int a = -2;  // not a row
    if (t < p.m) {
        a = p.index[t];
        if (a < 0 || a >= p.adapters) a = -1;
    }
    if (t < kMaxM) g.index[t] = a;
    __syncthreads();
    uint32_t same[4] = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w * 32 >= p.m) break;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const int4 v = *reinterpret_cast<const int4*>(&g.index[w * 32 + i]);
            same[w] |= (v.x == a ? 1u << i : 0u) | (v.y == a ? 2u << i : 0u) |
                       (v.z == a ? 4u << i : 0u) | (v.w == a ? 8u << i : 0u);
        }
    }
    int lead = kMaxM, before = 0, size = 0;
#pragma unroll
    for (int w = 3; w >= 0; --w) {
        if (same[w]) lead = w * 32 + __ffs(same[w]) - 1;
        size += __popc(same[w]);
        if (w <= warp) before += __popc(w < warp ? same[w] : same[w] & ((1u << lane) - 1));
    }
    // the rows without an adapter come last, whatever their first row is
    const bool leads = a >= 0 && lead == t;
    int sum = leads ? size : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(~0u, sum, d);
        if (lane >= d) sum += v;
    }
    const uint32_t vote = __ballot_sync(~0u, leads);
    if (lane == 31 && t < kMaxM) {
        warp_sum[warp] = sum;
        warp_lead[warp] = __popc(vote);
    }
    __syncthreads();
    int start = sum - (leads ? size : 0), group = __popc(vote & ((1u << lane) - 1)), all = 0,
        leaders = 0;
#pragma unroll
    for (int w = 0; w < kMaxM / 32; ++w) {
        if (w < warp) start += warp_sum[w], group += warp_lead[w];
        all += warp_sum[w], leaders += warp_lead[w];
    }
    const bool first_bare = a == -1 && before == 0;
    if (first_bare) start = all, group = leaders;
    if (leads || first_bare) {
        int r = 0;
        if (a >= 0) r = p.ranks ? min(max(p.ranks[a], 0), p.rank) : p.rank;
        g.adapter[group] = (int16_t)a;
        g.rank[group] = (int16_t)r;
        g.first[group] = (int16_t)start;
        g.first[group + 1] = (int16_t)(start + size);  // the next group's start, if there is one
        g.lead[a >= 0 ? t : kMaxM] = (int16_t)start;
    }
    if (t == 0) g.count = leaders + (all < p.m);
    __syncthreads();
    if (t < p.m) g.row[g.lead[a >= 0 ? lead : kMaxM] + before] = (int16_t)t;
    __syncthreads();
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_stream(const uint16_t* p) {  // read once
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// ---- T = A x -----------------------------------------------------------------------------
__global__ void __launch_bounds__(kDownThreads, 3) nvfp4_lora_down_kernel(const Params p) {
    __shared__ Groups g;
    __shared__ __align__(16) float part[kDownWarps][kColTiles][16][8];
    __shared__ __align__(16) float sum[kColTiles * 128];
    // (the second kernel reads y and the index as soon as it may start: not before this one may)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const auto cluster = cooperative_groups::this_cluster();
    const int ctas = (int)cluster.num_blocks(), cta = (int)cluster.block_rank();
    find_groups(p, g);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
    const int blocks = p.rank16 / 16;
    const int item = blockIdx.x / ctas, blk = item % blocks, gi = item / blocks;
    if (gi >= g.count) return;  // (the whole cluster)
    const int rank = g.rank[gi], r0 = blk * 16;
    if (r0 >= rank) return;
    const int first = g.first[gi], rows = g.first[gi + 1] - first;
    const uint16_t* const a = p.a + g.adapter[gi] * p.a_stride;
    const float scale = p.scales[g.adapter[gi]];
    // this lane's two rank rows; a row past the rank counts as zeros and is not read
    const bool on0 = r0 + gr < rank, on1 = r0 + gr + 8 < rank;
    const uint16_t* const a0 = a + (int64_t)(r0 + gr) * p.a_ld;
    const uint16_t* const a1 = a0 + 8 * p.a_ld;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int c0 = 0; c0 < rows; c0 += 8 * kColTiles) {
        const int tiles = min((rows - c0 + 7) / 8, kColTiles);
        const uint16_t* xr[kColTiles];
#pragma unroll
        for (int c = 0; c < kColTiles; ++c) {
            const int i = c0 + c * 8 + gr;
            xr[c] = i < rows ? p.x + (int64_t)g.row[first + i] * p.ldx : nullptr;
        }
        float acc[kColTiles][4];
#pragma unroll
        for (int c = 0; c < kColTiles; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][e] = 0.f;
        const int stride = ctas * kDownWarps * kStepK;
        for (int k0 = (cta * kDownWarps + warp) * kStepK; k0 < p.k; k0 += stride) {
            uint4 w0[4], w1[4], x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = k0 + u * 32 + t * 8;
                w0[u] = on0 && k < p.k ? load_stream(a0 + k) : zero;
                w1[u] = on1 && k < p.k ? load_stream(a1 + k) : zero;
            }
#pragma unroll
            for (int c = 0; c < kColTiles; ++c) {
                if (c >= tiles) break;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int k = k0 + u * 32 + t * 8;
                    x[u] = xr[c] && k < p.k ? __ldg(reinterpret_cast<const uint4*>(xr[c] + k))
                                            : zero;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    mma_bf16(acc[c], w0[u].x, w1[u].x, w0[u].y, w1[u].y, x[u].x, x[u].y);
                    mma_bf16(acc[c], w0[u].z, w1[u].z, w0[u].w, w1[u].w, x[u].z, x[u].w);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < kColTiles; ++c) {
            if (c >= tiles) break;
            *reinterpret_cast<float2*>(&part[warp][c][gr][2 * t]) =
                make_float2(acc[c][0], acc[c][1]);
            *reinterpret_cast<float2*>(&part[warp][c][gr + 8][2 * t]) =
                make_float2(acc[c][2], acc[c][3]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < tiles * 128; i += kDownThreads) {
            const float* const from = &part[0][0][0][0] + i;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kDownWarps; ++w) v += from[w * kColTiles * 128];
            sum[i] = v;  // [tile][rank][row]
        }
        cluster.sync();
        if (cta == 0) {
            for (int i = threadIdx.x; i < tiles * 128; i += kDownThreads) {
                const int r = i & 15, col = (i >> 4) & 7, c = i >> 7;
                const int at = c * 128 + r * 8 + col;  // neighbours write neighbouring ranks
                float v = 0.f;
                for (int q = 0; q < ctas; ++q) v += cluster.map_shared_rank(sum, q)[at];
                const int row = c0 + c * 8 + col;
                if (row < rows) {
                    v = r0 + r < rank ? v * scale : 0.f;
                    const __nv_bfloat16 h = __float2bfloat16_rn(v);
                    const float rest = v - __bfloat162float(h);
                    uint16_t* const to =
                        p.t + (int64_t)g.row[first + row] * 2 * p.rank32 + r0 + r;
                    to[0] = __bfloat16_as_ushort(h);
                    to[p.rank32] = __bfloat16_as_ushort(
                        __float2bfloat16_rn(isfinite(__bfloat162float(h)) ? rest : 0.f));
                }
            }
        }
        cluster.sync();  // before the sums are written again, or their CTA is gone
    }
}

// ---- out = y + B T -----------------------------------------------------------------------
// CTAs that an SM holds at once (more than that at rank 64, in a second wave: 27.4 us, not 23.9).
template <int STEPS>
constexpr int kUp = STEPS == 1 ? 6 : STEPS == 2 ? 5 : 3;

template <int STEPS>  // 32 ranks each
__global__ void __launch_bounds__(kThreads, kUp<STEPS>)
    nvfp4_lora_up_kernel(const Params p) {
    __shared__ Groups g;
    find_groups(p, g);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
    const int chunks = (p.n + kChunkN - 1) / kChunkN;
    const int items = g.count * chunks;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    bool waited = false;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int gi = it / chunks, n0 = (it - gi * chunks) * kChunkN + warp * 32;
        const int rank = g.rank[gi], first = g.first[gi], rows = g.first[gi + 1] - first;
        // row c + 8 h (c < 8) of tile j is channel n0 + 4 c + 2 j + h: a lane's rows c = gr are its
        // channels n0 + 4 gr .. + 3
        uint4 w[2][2][STEPS];
        const int n = n0 + gr * 4;
        const uint16_t* const b = p.b + (int64_t)max((int)g.adapter[gi], 0) * p.b_stride +
                                  (int64_t)n * p.b_ld + t * 8;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
                    w[j][h][s] = n < p.n && s * 32 + t * 8 < rank
                                     ? load_stream(b + (2 * j + h) * p.b_ld + s * 32)
                                     : zero;
        if (rank % 8) {  // ranks past the adapter's own within a lane's 8: zeros, whatever is there
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int left = rank - (s * 32 + t * 8);
                if (left > 0 && left < 8) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t* const v = &w[j >> 1][j & 1][s].x;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] &= (2 * e < left ? 0xffffu : 0u) |
                                    (2 * e + 1 < left ? 0xffff0000u : 0u);
                    }
                }
            }
        }
        for (int m0 = 0; m0 < rows; m0 += 8) {
            // a lane multiplies T of row gr and writes rows 2t and 2t + 1
            const int left = rows - m0;
            const int mul_row = gr < left ? g.row[first + m0 + gr] : 0;
            int row[2];
            uint2 y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                row[e] = 2 * t + e < left && n < p.n ? g.row[first + m0 + 2 * t + e] : -1;
                y[e] = make_uint2(0, 0);
                if (row[e] >= 0)
                    y[e] = *reinterpret_cast<const uint2*>(p.y + (int64_t)row[e] * p.ldy + n);
            }
            if (!waited) {  // T, from here on
                asm volatile("griddepcontrol.wait;" ::: "memory");
                waited = true;
            }
            float acc[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
            const uint16_t* const from = p.t + (int64_t)mul_row * 2 * p.rank32 + t * 8;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                // (16 ranks that the adapter does not reach were not written)
                const bool live = gr < left && s * 32 + t * 8 < ((rank + 15) & ~15);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint4 v = live ? *reinterpret_cast<const uint4*>(
                                               from + half * p.rank32 + s * 32)
                                         : zero;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 c = w[j][0][s], d = w[j][1][s];
                        mma_bf16(acc[j], c.x, d.x, c.y, d.y, v.x, v.y);
                        mma_bf16(acc[j], c.z, d.z, c.w, d.w, v.z, v.w);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (row[e] < 0) continue;
                if (rank) {
                    uint32_t* const v = &y[e].x;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {  // channels 2j and 2j + 1
                        const float e0 = __uint_as_float(v[j] << 16) + acc[j][e];
                        const float e1 = __uint_as_float(v[j] & 0xffff0000u) + acc[j][2 + e];
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v[j]) : "f"(e1), "f"(e0));
                    }
                }
                *reinterpret_cast<uint2*>(p.out + (int64_t)row[e] * p.ldo + n) = y[e];
            }
        }
    }
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// CTAs of a cluster: enough items of (group, 16 ranks, part of K) for two per SM, no more than K has
// steps for.  The group count is on the device; its bound is not.
int choose_cluster(int m, int adapters, int rank, int64_t k, int sms) {
    const int64_t items = (int64_t)(m < adapters ? m : adapters) * ((rank + 15) / 16);
    int ctas = 1;
    while (ctas < 8 && items * ctas < 2 * sms && 2 * ctas * kDownWarps * kStepK / 2 < k) ctas *= 2;
    return ctas;
}

size_t t_bytes(int m, int rank) { return (size_t)m * 2 * ((rank + 31) / 32 * 32) * 2; }

int check_shape(int m, int adapters, int rank, int64_t k) {
    if (m < 0 || m > NVFP4_MAX_ROWS) return NVFP4_ERR_ROWS;
    if (adapters < 0 || adapters > 32767 || rank < 0 || rank > kMaxRank || rank % 8 || k < 0 ||
        k % 8 || k > (1 << 30))
        return NVFP4_ERR_SHAPE;
    return NVFP4_OK;
}

// Everything that a call is refused for but the device and the workspace.
int check_call(const nvfp4_lora_t* lora, const void* x, int64_t ldx, const void* y, int64_t ldy,
               void* out, int64_t ldo, int m, int64_t n, int64_t k) {
    if (!lora) return NVFP4_ERR_NULL;
    const nvfp4_lora_t& l = *lora;
    const int st = check_shape(m, l.adapters, l.rank, k);
    if (st != NVFP4_OK) return st;
    if (n < 0 || n % 8 || n > (1 << 30) || ldx < k || ldy < n || ldo < n || l.a_ld < k ||
        l.b_ld < l.rank || l.a_stride < 0 || l.b_stride < 0)
        return NVFP4_ERR_SHAPE;
    if (m == 0 || n == 0) return NVFP4_OK;
    const bool any = l.adapters > 0 && l.rank > 0;
    if (!y || !out || !l.index || (any && (!l.a || !l.b || !l.scales)) || (any && k && !x))
        return NVFP4_ERR_NULL;
    if (misaligned(x, 16) || misaligned(y, 16) || misaligned(out, 16) || misaligned(l.a, 16) ||
        misaligned(l.b, 16) || misaligned(l.index, 4) || misaligned(l.scales, 4) ||
        misaligned(l.ranks, 4) || ldx % 8 || ldy % 8 || ldo % 8 || l.a_ld % 8 || l.b_ld % 8 ||
        l.a_stride % 8 || l.b_stride % 8)
        return NVFP4_ERR_ALIGN;
    using nvfp4_host::span;
    const uint64_t ob = 2 * span(1, 0, 1, 0, m, ldo, n), yb = 2 * span(1, 0, 1, 0, m, ldy, n);
    // in place is y itself, row for row
    if (overlaps(out, ob, y, yb) && !(out == y && (ldo == ldy || m == 1))) return NVFP4_ERR_ALIAS;
    if (overlaps(out, ob, l.index, 4ull * m)) return NVFP4_ERR_ALIAS;
    if (any && (overlaps(out, ob, x, 2 * span(1, 0, 1, 0, m, ldx, k)) ||
                overlaps(out, ob, l.a, 2 * span(1, 0, l.adapters, l.a_stride, l.rank, l.a_ld, k)) ||
                overlaps(out, ob, l.b, 2 * span(1, 0, l.adapters, l.b_stride, n, l.b_ld, l.rank)) ||
                overlaps(out, ob, l.scales, 4ull * l.adapters) ||
                overlaps(out, ob, l.ranks, 4ull * l.adapters)))
        return NVFP4_ERR_ALIAS;
    return NVFP4_OK;
}

template <int STEPS>
int launch_up(const Params& p, int sms, bool after_down, cudaStream_t stream) {
    const int64_t groups = (p.m < p.adapters ? p.m : p.adapters) + 1;
    const int64_t items = groups * ((p.n + kChunkN - 1) / kChunkN);
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)(items < kUp<STEPS> * sms ? items : kUp<STEPS> * sms));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    // only behind the first kernel, which itself began after all earlier work: this one reads y
    // and the weights before it waits
    cfg.attrs = attr;
    cfg.numAttrs = after_down ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, nvfp4_lora_up_kernel<STEPS>, p) != cudaSuccess) {
        cudaGetLastError();
        return NVFP4_ERR_LAUNCH;
    }
    return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_lora_workspace_bytes(int m, int adapters, int rank, int64_t k, size_t* bytes) {
    if (!bytes) return NVFP4_ERR_NULL;
    int st = check_shape(m, adapters, rank, k);
    if (st != NVFP4_OK) return st;
    int dev, sms;
    nvfp4_host::EncodeFn encode;
    st = nvfp4_host::device(&dev, &sms, &encode);
    if (st != NVFP4_OK) return st;
    *bytes = t_bytes(m, rank);
    return NVFP4_OK;
}

int nvfp4_lora_check(const nvfp4_lora_t* lora, const void* x, int64_t ldx, const void* y,
                     int64_t ldy, void* out, int64_t ldo, int m, int64_t n, int64_t k) {
    return check_call(lora, x, ldx, y, ldy, out, ldo, m, n, k);
}

int nvfp4_lora_add(const nvfp4_lora_t* lora, const void* x, int64_t ldx, const void* y,
                   int64_t ldy, void* out, int64_t ldo, int m, int64_t n, int64_t k,
                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check_call(lora, x, ldx, y, ldy, out, ldo, m, n, k);
    if (st != NVFP4_OK || m == 0 || n == 0) return st;
    const nvfp4_lora_t& l = *lora;
    const bool any = l.adapters > 0 && l.rank > 0;
    if (overlaps(out, 2 * nvfp4_host::span(1, 0, 1, 0, m, ldo, n), workspace, t_bytes(m, l.rank)))
        return NVFP4_ERR_ALIAS;
    int dev, sms;
    nvfp4_host::EncodeFn encode;
    st = nvfp4_host::device(&dev, &sms, &encode);
    if (st != NVFP4_OK) return st;
    Params p;
    memset(&p, 0, sizeof(p));
    p.a = static_cast<const uint16_t*>(l.a);
    p.a_stride = l.a_stride;
    p.a_ld = l.a_ld;
    p.b = static_cast<const uint16_t*>(l.b);
    p.b_stride = l.b_stride;
    p.b_ld = l.b_ld;
    p.scales = l.scales;
    p.ranks = l.ranks;
    p.index = l.index;
    p.x = static_cast<const uint16_t*>(x);
    p.ldx = ldx;
    p.y = static_cast<const uint16_t*>(y);
    p.ldy = ldy;
    p.out = static_cast<uint16_t*>(out);
    p.ldo = ldo;
    p.m = m;
    p.adapters = any ? l.adapters : 0;
    p.rank = l.rank;
    p.rank16 = (l.rank + 15) / 16 * 16;
    p.n = (int)n;
    p.k = (int)k;
    p.rank32 = (l.rank + 31) / 32 * 32;
    const size_t need = t_bytes(m, l.rank);
    if (need && (!workspace || misaligned(workspace, 16) || workspace_bytes < need))
        return NVFP4_ERR_WORKSPACE;
    p.t = static_cast<uint16_t*>(workspace);
    if (any) {
        const int64_t groups = m < l.adapters ? m : l.adapters;
        const int ctas = choose_cluster(m, l.adapters, l.rank, k, sms);
        st = nvfp4_host::launch_behind(nvfp4_lora_down_kernel,
                                       dim3((unsigned)(groups * (p.rank16 / 16) * ctas)),
                                       kDownThreads, 0, ctas, stream, p);
        if (st != NVFP4_OK) return st;
    }
    if (p.rank <= 32) return launch_up<1>(p, sms, any, stream);
    if (p.rank <= 64) return launch_up<2>(p, sms, any, stream);
    return launch_up<4>(p, sms, any, stream);
}

}  // extern "C"

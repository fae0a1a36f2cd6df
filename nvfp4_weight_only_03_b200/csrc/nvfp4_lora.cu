// Low-rank adapters of many requests beside a shared projection (nvfp4_lora_add):
//
//   out[m] = bf16( y[m] + scale_a * B_a (A_a x[m]) ),   a = index[m];  out[m] = y[m] without one
//
// * Two kernels: the first forms T = A x (rank values per row), the second adds B T.  Rows that
//   share an adapter form a group, found from `index` by every CTA itself (at most 128 rows), so each adapter leaves HBM once and the host needs no copy of the index.
// * HBM bound: rank * (K + N) bf16 per adapter against a few rows.  The weights go from global
//   memory straight into mma.sync fragments, 16 bytes per lane and load: k (and the rank) may be
//   permuted as long as both operands are, so a lane's 8 consecutive values serve as the 4 pairs
//   of two MMAs, and no shared-memory pass is needed.  tcgen05 would have to stage them.
// * First kernel: weights are the 16 rows of the MMA, x rows its 8 columns; 8 warps split a CTA's
//   K range and CTAs split K further when there are few groups; sums over warps and ranges are
//   formed in a fixed order.  Second kernel: T rows are the MMA's 16 rows and the columns are
//   output channels, permuted so that a lane ends up with 8 consecutive ones.
// * T stays fp32 between the kernels and enters the second MMA as two bf16 values (high and
//   remainder), so it is carried to 2^-17; the only other rounding is the output's.
// * The second kernel is launched while the first runs and has its weights and y in registers
//   before it waits for T.
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

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kMaxM = NVFP4_MAX_ROWS;
constexpr int kMaxRank = NVFP4_LORA_MAX_RANK;
constexpr int kChunkN = kWarps * 32;  // output channels per item of the second kernel
constexpr int kColTiles = 4;          // tiles of 8 rows that share one pass over A

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
    float* t;  // [splits][m][rank16] partial sums of T
    int m, adapters, rank, rank16, n, k, splits, chunk;  // chunk: k of one split, % 256 == 0
};

// Rows by adapter: `row` lists the rows group by group; group g is adapter[g], its rows are
// row[first[g]] .. row[first[g + 1] - 1].  Rows without an adapter are a last group of rank 0.
struct Groups {
    int count;
    int16_t adapter[kMaxM + 1], rank[kMaxM + 1], first[kMaxM + 2], row[kMaxM];
    int16_t lead[kMaxM];  // the first row with this row's adapter; kMaxM without one
    int32_t index[kMaxM];
};

// Thread t places row t: it counts the rows of earlier groups, and the earlier ones of its own.
__device__ __forceinline__ void find_groups(const Params& p, Groups& g) {
    const int t = threadIdx.x;
    int a = -1;
    if (t < p.m) {
        a = p.index[t];
        if (a < 0 || a >= p.adapters) a = -1;
        g.index[t] = a;
    }
    if (t == 0) g.count = 0;
    __syncthreads();
    int lead = kMaxM;
    if (t < p.m) {
        if (a >= 0)
            for (int i = t; i >= 0; --i)
                if (g.index[i] == a) lead = i;
        g.lead[t] = (int16_t)lead;
    }
    __syncthreads();
    if (t < p.m) {
        int group = 0, start = 0, before = 0, size = 0;
        for (int i = 0; i < p.m; ++i) {
            const int l = g.lead[i];
            group += l == i && l < lead;
            start += l < lead;
            before += l == lead && i < t;
            size += l == lead;
        }
        g.row[start + before] = (int16_t)t;
        if (before == 0) {
            int r = 0;
            if (a >= 0) r = p.ranks ? min(max(p.ranks[a], 0), p.rank) : p.rank;
            g.adapter[group] = (int16_t)a;
            g.rank[group] = (int16_t)r;
            g.first[group] = (int16_t)start;
            g.first[group + 1] = (int16_t)(start + size);  // the next group's start, if there is one
            atomicAdd(&g.count, 1);
        }
    }
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
__global__ void __launch_bounds__(kThreads, 2) nvfp4_lora_down_kernel(const Params p) {
    __shared__ Groups g;
    __shared__ __align__(16) float part[kWarps][kColTiles][16][8];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    find_groups(p, g);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
    const int blocks = p.rank16 / 16;
    const int items = g.count * blocks * p.splits;
    constexpr int kUnroll = 4;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int split = it % p.splits, gb = it / p.splits, blk = gb % blocks, gi = gb / blocks;
        const int rank = g.rank[gi], r0 = blk * 16;
        if (r0 >= rank) continue;
        const int first = g.first[gi], rows = g.first[gi + 1] - first;
        const uint16_t* const a = p.a + g.adapter[gi] * p.a_stride;
        // this lane's two rank rows; a row past the rank counts as zeros and is not read
        const bool on0 = r0 + gr < rank, on1 = r0 + gr + 8 < rank;
        const uint16_t* const a0 = a + (int64_t)(r0 + gr) * p.a_ld;
        const uint16_t* const a1 = a0 + 8 * p.a_ld;
        const int end = min((split + 1) * p.chunk, p.k);
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
            for (int k0 = split * p.chunk + warp * 32 + t * 8; k0 - t * 8 < end;
                 k0 += kWarps * 32 * kUnroll) {
                uint4 w0[kUnroll], w1[kUnroll], xv[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int kk = k0 + u * kWarps * 32;
                    w0[u] = on0 && kk < end ? load_stream(a0 + kk) : zero;
                    w1[u] = on1 && kk < end ? load_stream(a1 + kk) : zero;
                }
#pragma unroll
                for (int c = 0; c < kColTiles; ++c) {
                    if (c >= tiles) break;
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u) {
                        const int kk = k0 + u * kWarps * 32;
                        xv[u] = xr[c] && kk < end
                                    ? __ldg(reinterpret_cast<const uint4*>(xr[c] + kk))
                                    : zero;
                    }
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u) {
                        mma_bf16(acc[c], w0[u].x, w1[u].x, w0[u].y, w1[u].y, xv[u].x, xv[u].y);
                        mma_bf16(acc[c], w0[u].z, w1[u].z, w0[u].w, w1[u].w, xv[u].z, xv[u].w);
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
            for (int i = threadIdx.x; i < tiles * 128; i += kThreads) {
                const int c = i >> 7, r = i & 15, col = (i >> 4) & 7;
                if (c0 + c * 8 + col < rows) {
                    float s = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) s += part[w][c][r][col];
                    p.t[((int64_t)split * p.m + g.row[first + c0 + c * 8 + col]) * p.rank16 + r0 +
                        r] = s;
                }
            }
            __syncthreads();
        }
    }
}

// ---- out = y + B T -----------------------------------------------------------------------
template <int STEPS>  // 32 ranks each
__global__ void __launch_bounds__(kThreads, STEPS > 2 ? 1 : 2)
    nvfp4_lora_up_kernel(const Params p) {
    __shared__ Groups g;
    constexpr int kR = STEPS * 32, kPad = kR + 8;  // a row's stride keeps 16-byte reads apart
    extern __shared__ __align__(16) uint16_t t_smem[];
    uint16_t* const hi = t_smem;                     // [m][kPad]
    uint16_t* const lo = t_smem + p.m * kPad;
    find_groups(p, g);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
    const int chunks = (p.n + kChunkN - 1) / kChunkN;
    const int64_t items = (int64_t)g.count * chunks;
    const int64_t i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
    int loaded = -1;
    bool waited = false;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t it = i0; it < i1; ++it) {
        const int gi = (int)(it / chunks), n0 = (int)(it % chunks) * kChunkN + warp * 32;
        const int rank = g.rank[gi], first = g.first[gi], rows = g.first[gi + 1] - first;
        // column c of tile j is channel n0 + (c / 2) * 8 + 2 j + c % 2: tile j's columns 2t, 2t+1
        // are a lane's channels n0 + 8 t + 2 j + {0, 1}
        uint4 w[4][STEPS];
        const uint16_t* const b = p.b + (int64_t)max((int)g.adapter[gi], 0) * p.b_stride;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + (gr >> 1) * 8 + 2 * j + (gr & 1);
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int r = s * 32 + t * 8;
                w[j][s] = n < p.n && r < rank ? load_stream(b + (int64_t)n * p.b_ld + r) : zero;
            }
        }
        const int n_out = n0 + t * 8;
        auto y_at = [&](int i) {
            return i < rows && n_out < p.n
                       ? *reinterpret_cast<const uint4*>(p.y + (int64_t)g.row[first + i] * p.ldy + n_out)
                       : zero;
        };
        uint4 y0 = y_at(gr), y1 = y_at(gr + 8);
        if (rank % 8) {  // ranks past the adapter's own within a lane's 8: zeros, whatever is there
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int left = rank - (s * 32 + t * 8);
                if (left > 0 && left < 8) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t* const v = &w[j][s].x;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] &= (2 * e < left ? 0xffffu : 0u) |
                                    (2 * e + 1 < left ? 0xffff0000u : 0u);
                    }
                }
            }
        }
        if (!waited) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            waited = true;
        }
        if (gi != loaded) {
            __syncthreads();
            const float scale = rank ? p.scales[g.adapter[gi]] : 0.f;
            for (int i = threadIdx.x; i < rows * kR; i += kThreads) {
                const int q = i / kR, r = i % kR;
                float v = 0.f;
                if (r < rank) {
                    const float* src = p.t + (int64_t)g.row[first + q] * p.rank16 + r;
                    for (int s = 0; s < p.splits; ++s) v += __ldcg(src + (int64_t)s * p.m * p.rank16);
                    v *= scale;
                }
                const __nv_bfloat16 h = __float2bfloat16_rn(v);
                const float rest = v - __bfloat162float(h);
                hi[q * kPad + r] = __bfloat16_as_ushort(h);
                lo[q * kPad + r] = __bfloat16_as_ushort(
                    __float2bfloat16_rn(isfinite(__bfloat162float(h)) ? rest : 0.f));
            }
            loaded = gi;
            __syncthreads();
        }
        for (int m0 = 0; m0 < rows; m0 += 16) {
            if (m0) y0 = y_at(m0 + gr), y1 = y_at(m0 + gr + 8);
            float acc[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
            const bool on0 = m0 + gr < rows, on1 = m0 + gr + 8 < rows;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                if (s * 32 >= rank) break;
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const uint16_t* const src = (part ? lo : hi) + (m0 + gr) * kPad + s * 32 + t * 8;
                    const uint4 u = on0 ? *reinterpret_cast<const uint4*>(src) : zero;
                    const uint4 v = on1 ? *reinterpret_cast<const uint4*>(src + 8 * kPad) : zero;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        mma_bf16(acc[j], u.x, v.x, u.y, v.y, w[j][s].x, w[j][s].y);
                        mma_bf16(acc[j], u.z, v.z, u.w, v.w, w[j][s].z, w[j][s].w);
                    }
                }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!(half ? on1 : on0) || n_out >= p.n) continue;
                uint16_t* const dst =
                    p.out + (int64_t)g.row[first + m0 + gr + half * 8] * p.ldo + n_out;
                uint4 o = half ? y1 : y0;
                if (rank) {
                    uint32_t* const v = &o.x;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float e0 = __uint_as_float(v[j] << 16) + acc[j][2 * half];
                        const float e1 = __uint_as_float(v[j] & 0xffff0000u) + acc[j][2 * half + 1];
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v[j]) : "f"(e1), "f"(e0));
                    }
                }
                *reinterpret_cast<uint4*>(dst) = o;
            }
        }
    }
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

struct Split {
    int splits, chunk;
};

// K ranges: enough items of (group, 16 ranks, range) for three per SM, each range a multiple of
// the 256 k that a CTA's warps take per step.  The group count is on the device; its bound is not.
Split choose_split(int m, int adapters, int rank, int64_t k, int sms) {
    const int64_t groups = m < adapters ? m : adapters;
    const int64_t steps = (k + 255) / 256;
    const int64_t per = groups * ((rank + 15) / 16);
    int64_t want = (3 * sms + per - 1) / (per > 0 ? per : 1);
    if (want > steps) want = steps;
    if (want < 1) want = 1;
    const int64_t each = (steps + want - 1) / want;
    Split s;
    s.chunk = (int)(each * 256);
    s.splits = (int)((steps + each - 1) / each);
    if (s.splits < 1) s.splits = 1;
    return s;
}

int check_shape(int m, int adapters, int rank, int64_t k) {
    if (m < 0 || m > NVFP4_MAX_ROWS) return NVFP4_ERR_ROWS;
    if (adapters < 0 || adapters > 32767 || rank < 0 || rank > kMaxRank || rank % 8 || k < 0 ||
        k % 8 || k > (1 << 30))
        return NVFP4_ERR_SHAPE;
    return NVFP4_OK;
}

template <int STEPS>
int launch_up(const Params& p, int sms, bool after_down, cudaStream_t stream) {
    const size_t smem = (size_t)2 * p.m * (STEPS * 32 + 8) * 2;
    static bool ready[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !ready[dev]) {
        if (cudaFuncSetAttribute(nvfp4_lora_up_kernel<STEPS>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 2 * kMaxM * (STEPS * 32 + 8) * 2) != cudaSuccess) {
            cudaGetLastError();
            return NVFP4_ERR_LAUNCH;
        }
        ready[dev] = true;
    }
    const int64_t groups = (p.m < p.adapters ? p.m : p.adapters) + 1;
    const int64_t items = groups * ((p.n + kChunkN - 1) / kChunkN);
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)(items < 2 * sms ? items : 2 * sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
    const Split s = choose_split(m, adapters, rank, k, sms);
    *bytes = (size_t)s.splits * m * ((rank + 15) / 16 * 16) * 4;
    return NVFP4_OK;
}

int nvfp4_lora_add(const nvfp4_lora_t* lora, const void* x, int64_t ldx, const void* y,
                   int64_t ldy, void* out, int64_t ldo, int m, int64_t n, int64_t k,
                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!lora) return NVFP4_ERR_NULL;
    const nvfp4_lora_t& l = *lora;
    int st = check_shape(m, l.adapters, l.rank, k);
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
    const uint64_t ob = 2ull * ((uint64_t)(m - 1) * ldo + n), yb = 2ull * ((uint64_t)(m - 1) * ldy + n);
    // in place is y itself, row for row
    if (overlaps(out, ob, y, yb) && !(out == y && (ldo == ldy || m == 1))) return NVFP4_ERR_ALIAS;
    if (any && overlaps(out, ob, x, 2ull * ((uint64_t)(m - 1) * ldx + k))) return NVFP4_ERR_ALIAS;
    int dev, sms;
    nvfp4_host::EncodeFn encode;
    st = nvfp4_host::device(&dev, &sms, &encode);
    if (st != NVFP4_OK) return st;
    const Split s = choose_split(m, l.adapters, l.rank, k, sms);
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
    p.splits = s.splits;
    p.chunk = s.chunk;
    const size_t need = (size_t)s.splits * m * p.rank16 * 4;
    if (need && (!workspace || misaligned(workspace, 16) || workspace_bytes < need))
        return NVFP4_ERR_WORKSPACE;
    p.t = static_cast<float*>(workspace);
    if (any) {
        const int64_t groups = m < l.adapters ? m : l.adapters;
        const int64_t items = groups * (p.rank16 / 16) * s.splits;
        const int grid = (int)(items < 4 * sms ? items : 4 * sms);
        nvfp4_lora_down_kernel<<<grid, kThreads, 0, stream>>>(p);
        if (cudaGetLastError() != cudaSuccess) return NVFP4_ERR_LAUNCH;
    }
    if (p.rank <= 32) return launch_up<1>(p, sms, any, stream);
    if (p.rank <= 64) return launch_up<2>(p, sms, any, stream);
    return launch_up<4>(p, sms, any, stream);
}

}  // extern "C"

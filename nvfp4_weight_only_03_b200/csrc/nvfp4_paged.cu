// The paged key/value cache around the attention: block tables and slot maps from request
// lengths (nvfp4_paged_plan), and new rows into the cache (nvfp4_kv_append).  The decode plan
// launches the latter as reshape_and_cache ("Blueprint - circuit executor" page for
// qwen3.8-27b-nvfp4 on GB10, table "Kernels the plan launches").
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "nvfp4.h"
#include "nvfp4_host.h"

namespace {

using nvfp4_host::misaligned;
using nvfp4_host::overlaps;

// ------------------------------------------------------------------------------------------
// Plan.  With b = block_size, old = ceil(len / b), want = max(old, min(ceil((len + new) / b),
// columns)), need = want - old:
//   starts = exclusive sums of new;  first = exclusive sums of need
//   table[r][c] = free[head + first[r] + c - old[r]] for old <= c < want, -1 past the list's end
//   slot of token t = page * b + pos % b, pos = len[r] + t - starts[r], page = table[r][pos / b]
//
// The two sums are the only step that needs every request; a few thousand integers from L2 cost
// less than a second launch or a grid-wide wait, so every CTA forms them itself in shared memory
// and then takes its share of the tokens and of the new pages, finding a token's (a page's)
// request by binary search.  Nothing is read that another CTA writes: an entry that this call
// fills is taken from the free list again instead of from the table.  Latency bound: the chain
// is lengths -> sums -> search -> table -> slot: 4.2 us for 32 requests, 6.6 us for 1024 with 10200
// tokens (B200).
constexpr int kPlanThreads = 512;

struct PlanParams {
    const int32_t* lens;
    const int32_t* fresh;  // new tokens
    int32_t* table;
    int64_t ld_table, columns;
    const int32_t* free_pages;
    int64_t n_free;
    const int32_t* head;
    int64_t tokens;  // capacity of the per-token outputs
    int32_t *starts, *lens_out, *slots, *request, *positions, *head_out, *missing;
    int requests, block;
};

__device__ __forceinline__ int32_t saturate(int64_t v) {
    return v > INT32_MAX ? INT32_MAX : (int32_t)v;
}

struct Pages {
    int64_t old, need, lost;  // pages held, to take, and wanted beyond the table's columns
};

__device__ __forceinline__ Pages pages_of(const PlanParams& p, int64_t len, int64_t fresh) {
    const int64_t old = (len + p.block - 1) / p.block;
    const int64_t all = (len + fresh + p.block - 1) / p.block;
    const int64_t held = all < p.columns ? all : p.columns;
    Pages g;
    g.old = old;
    g.need = held > old ? held - old : 0;
    g.lost = all - old - g.need;
    return g;
}

// Index of the last i in [0, n) with a[i] <= v, for ascending a with a[0] <= v.
__device__ __forceinline__ int last_at_most(const int64_t* a, int n, int64_t v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) nvfp4_plan_kernel(const PlanParams p) {
    extern __shared__ int64_t sums[];  // starts[requests], first[requests]
    int64_t* const starts = sums;
    int64_t* const first = sums + p.requests;
    __shared__ int64_t warp_sum[3][kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int64_t carry_tok = 0, carry_page = 0, lost = 0;
    for (int base = 0; base < p.requests; base += kPlanThreads) {
        const int r = base + tid;
        int64_t tok = 0, need = 0;
        if (r < p.requests) {
            const int64_t len = max(p.lens[r], 0);
            tok = max(p.fresh[r], 0);
            const Pages g = pages_of(p, len, tok);
            need = g.need;
            lost += g.lost;
        }
        int64_t st = tok, sp = need;  // inclusive sums over the warp
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t a = __shfl_up_sync(~0u, st, d), b = __shfl_up_sync(~0u, sp, d);
            if (lane >= d) st += a, sp += b;
        }
        if (lane == 31) warp_sum[0][warp] = st, warp_sum[1][warp] = sp;
        __syncthreads();
        int64_t bt = carry_tok, bp = carry_page;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            const int64_t a = warp_sum[0][w], b = warp_sum[1][w];
            if (w < warp) bt += a, bp += b;
            carry_tok += a, carry_page += b;
        }
        if (r < p.requests) {
            starts[r] = bt + st - tok;
            first[r] = bp + sp - need;
            if (blockIdx.x == 0) {
                p.starts[r] = saturate(bt + st - tok);
                p.lens_out[r] = saturate((int64_t)max(p.lens[r], 0) + tok);
            }
        }
        __syncthreads();  // starts, first; and warp_sum may be written again
    }
    const int64_t total = carry_tok, wanted = carry_page;
    const int64_t head = max(p.head[0], 0);
    const int64_t left = p.n_free > head ? p.n_free - head : 0;
    const int64_t got = wanted < left ? wanted : left;
    if (blockIdx.x == 0) {
#pragma unroll
        for (int d = 16; d; d >>= 1) lost += __shfl_down_sync(~0u, lost, d);
        if (lane == 0) warp_sum[2][warp] = lost;
        __syncthreads();
        if (tid == 0) {
            int64_t all = wanted - got;
            for (int w = 0; w < kPlanThreads / 32; ++w) all += warp_sum[2][w];
            p.starts[p.requests] = saturate(total);
            p.head_out[0] = saturate(head + got);
            p.missing[0] = saturate(all);
        }
    }
    const int64_t stride = (int64_t)gridDim.x * kPlanThreads;
    const int64_t me = (int64_t)blockIdx.x * kPlanThreads + tid;
    for (int64_t i = me; i < wanted; i += stride) {
        const int r = last_at_most(first, p.requests, i);  // the last one: need > 0
        const int64_t old = ((int64_t)max(p.lens[r], 0) + p.block - 1) / p.block;
        const int64_t c = old + i - first[r];
        // (always true unless the lengths change while the call runs)
        if (c < p.columns) p.table[r * p.ld_table + c] = i < left ? p.free_pages[head + i] : -1;
    }
    for (int64_t t = me; t < p.tokens; t += stride) {
        int32_t slot = -1, req = -1, at = 0;
        if (t < total) {
            const int r = last_at_most(starts, p.requests, t);
            const int64_t len = max(p.lens[r], 0);
            const int64_t pos = len + t - starts[r];
            const int64_t c = pos / p.block, old = (len + p.block - 1) / p.block;
            int64_t page = -1;
            if (c < p.columns) {
                const int64_t i = first[r] + c - old;
                if (c < old) page = p.table[r * p.ld_table + c];
                else if (i >= 0 && i < left) page = p.free_pages[head + i];
            }
            const int64_t s = page * p.block + pos % p.block;
            if (page >= 0 && s <= INT32_MAX) slot = (int32_t)s;
            req = r;
            at = saturate(pos);
        }
        p.slots[t] = slot;
        if (p.request) p.request[t] = req;
        if (p.positions) p.positions[t] = at;
    }
}

// ------------------------------------------------------------------------------------------
// Append.  A warp per token, or per token and side (K or V); a lane moves pieces of 16 bytes of the
// cache (8 bf16 values, or 16 codes), so loads and stores are whole sectors and the slot is looked up
// once per row.  HBM bound, 4 bytes of traffic per value (3 with an 8-bit cache).  Measured (B200):
// 8192 tokens of 4 heads of 256 into an e4m3 cache 11.1 us, 63% of the copy rate; 128 tokens, bf16,
// 1.8 us.
//
// An e4m3 code is e4m3_rn(x / scale) of the fp32 quotient, saturated at 448.  A division per value was
// the bound (a hundred instructions per eight values).  The quotient is formed from 1 / scale in two
// fp32 terms, r and the rest of it, as q = fma(x, r, x * rest), which is off by little more than the
// rounding itself, so within one place; Markstein's correction (IBM J. Res. Dev. 34, 1990: with r the
// rounded reciprocal and q within a place, q + r (x - q scale) in two fused steps is the rounded
// quotient) then makes it exact, as long as nothing on the way leaves fp32's range: values of 2^63 scales
// and more (infinities and NaN among them), and all values at scales below 1e-15 or above 1e15, are
// divided.
constexpr int kAppendThreads = 256;

struct AppendParams {
    const uint16_t* src[2];
    int64_t ld[2], head_stride[2];
    uint8_t* cache[2];
    float scale[2], inverse[2], rest[2];  // 1 / scale = inverse + rest
    uint32_t far[2];  // sets bits 15 and 31 when added to two bf16 exponents that want a division
    const int32_t* slots;
    int64_t tokens, blocks, block_stride, slot_stride, cache_head_stride;
    int heads, dim, block;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// 8 bf16 values -> 8 codes.
__device__ __forceinline__ uint2 quantise(uint4 v, float scale, float inverse, float rest,
                                          uint32_t far) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top |= (w[i] & 0x7f807f80u) + far;
    const bool divide = top & 0x80008000u;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
        const float a = fmaf(x, inverse, x * rest);
        // (sums that are zero are +0: the sign is x's)
        q[i] = __uint_as_float(__float_as_uint(fmaf(fmaf(-a, scale, x), inverse, a)) |
                               (__float_as_uint(x) & 0x80000000u));
    }
    if (divide) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[i] = __fdiv_rn(i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]), scale);
    }
    return make_uint2(e4m3_pair(q[0], q[1]) | e4m3_pair(q[2], q[3]) << 16,
                      e4m3_pair(q[4], q[5]) | e4m3_pair(q[6], q[7]) << 16);
}

template <bool F8, int SIDES>  // K and V of a token in one warp, or one of them
__global__ void __launch_bounds__(kAppendThreads) nvfp4_append_kernel(const AppendParams p) {
    constexpr int kPiece = F8 ? 16 : 8;  // values
    const int lane = threadIdx.x & 31;
    const int per = p.dim / kPiece, pieces = p.heads * per;  // of a head, of a row
    const int log_per = 31 - __clz(per);
    const int64_t warps = (int64_t)gridDim.x * (kAppendThreads / 32);
    const int64_t me = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t i = me; i < p.tokens * (3 - SIDES); i += warps) {
        const int64_t t = SIDES == 2 ? i : i >> 1;
        const int32_t slot = __ldg(p.slots + t);
        const int32_t page = slot / p.block;
        if (slot < 0 || page >= p.blocks) continue;
        const int64_t at = page * p.block_stride + (int64_t)(slot - page * p.block) * p.slot_stride;
#pragma unroll 2
        for (int j = lane; j < pieces; j += 32) {
            const int h = j >> log_per, c = (j - (h << log_per)) * kPiece;
            const int64_t to = at + h * p.cache_head_stride + c;
            uint4 v[SIDES][F8 ? 2 : 1];
#pragma unroll
            for (int s = 0; s < SIDES; ++s) {  // (no load waits for a store)
                const int which = SIDES == 2 ? s : (int)(i & 1);
                const uint4* const from = reinterpret_cast<const uint4*>(
                    p.src[which] + t * p.ld[which] + h * p.head_stride[which] + c);
                v[s][0] = __ldg(from);
                if (F8) v[s][F8] = __ldg(from + 1);
            }
#pragma unroll
            for (int s = 0; s < SIDES; ++s) {
                const int which = SIDES == 2 ? s : (int)(i & 1);
                uint8_t* const dst = p.cache[which] + (F8 ? to : 2 * to);
                if (F8) {
                    const float scale = p.scale[which], inverse = p.inverse[which],
                                rest = p.rest[which];
                    const uint32_t far = p.far[which];
                    const uint2 x = quantise(v[s][0], scale, inverse, rest, far);
                    const uint2 y = quantise(v[s][F8], scale, inverse, rest, far);
                    *reinterpret_cast<uint4*>(dst) = make_uint4(x.x, x.y, y.x, y.y);
                } else {
                    *reinterpret_cast<uint4*>(dst) = v[s][0];
                }
            }
        }
    }
}

}  // namespace

namespace nvfp4_host {

int check_cache(const nvfp4_kv_cache_t* c) {
    if (!c) return NVFP4_ERR_NULL;
    if (c->type != NVFP4_KV_BF16 && c->type != NVFP4_KV_E4M3) return NVFP4_ERR_SHAPE;
    if (c->heads < 1 || c->heads > 1024 || (c->dim != 64 && c->dim != 128 && c->dim != 256) ||
        c->block_size < 16 || c->block_size % 16 || c->block_size > (1 << 20) || c->blocks < 0 ||
        c->blocks > INT32_MAX || c->blocks * c->block_size > INT32_MAX)
        return NVFP4_ERR_SHAPE;
    if (c->type == NVFP4_KV_E4M3 &&
        (!(c->k_scale > 0) || !(c->v_scale > 0) || isinf(c->k_scale) || isinf(c->v_scale)))
        return NVFP4_ERR_SHAPE;
    const int size = c->type == NVFP4_KV_E4M3 ? 1 : 2;
    const int64_t most = (int64_t)1 << 39;  // a tensor map's strides are below 2^40 bytes
    const int64_t strides[3] = {c->block_stride, c->slot_stride, c->head_stride};
    for (int64_t s : strides) {
        if (s < c->dim || s * size >= most) return NVFP4_ERR_SHAPE;
        if (s * size % 16) return NVFP4_ERR_ALIGN;
    }
    if (c->blocks > 0) {
        if (!c->k || !c->v) return NVFP4_ERR_NULL;
        if (misaligned(c->k, 16) || misaligned(c->v, 16)) return NVFP4_ERR_ALIGN;
    }
    return NVFP4_OK;
}

}  // namespace nvfp4_host

extern "C" {

int nvfp4_paged_plan(const nvfp4_paged_plan_t* plan, cudaStream_t stream) {
    if (!plan) return NVFP4_ERR_NULL;
    const nvfp4_paged_plan_t& a = *plan;
    if (a.requests < 0 || a.requests > NVFP4_MAX_REQUESTS || a.table_columns < 0 ||
        a.ld_table < a.table_columns || a.block_size < 1 || a.free_count < 0 || a.tokens < 0 ||
        a.tokens > INT32_MAX || a.free_count > INT32_MAX || a.table_columns > INT32_MAX)
        return NVFP4_ERR_SHAPE;
    if (!a.head || !a.starts || !a.head_out || !a.missing || (a.free_count && !a.free_pages) ||
        (a.tokens && !a.slots) || (a.requests && (!a.lens || !a.new_tokens || !a.lens_out)) ||
        (a.requests && a.table_columns && !a.table))
        return NVFP4_ERR_NULL;
    const void* all[] = {a.lens, a.new_tokens, a.table, a.free_pages, a.head, a.starts, a.lens_out,
                         a.slots, a.request, a.positions, a.head_out, a.missing};
    for (const void* q : all)
        if (misaligned(q, 4)) return NVFP4_ERR_ALIGN;
    // nothing that is written may overlap anything else: every CTA reads the inputs
    const uint64_t rb = 4ull * a.requests, tb = 4ull * a.tokens;
    const uint64_t bytes[] = {
        rb, rb,
        a.requests ? 4 * nvfp4_host::span(1, 0, 1, 0, a.requests, a.ld_table, a.table_columns) : 0,
        4ull * a.free_count, 4, rb + 4, rb, tb, a.request ? tb : 0, a.positions ? tb : 0, 4, 4};
    const int inputs[] = {0, 1, 3, 4}, outputs[] = {2, 5, 6, 7, 8, 9, 10, 11};
    for (int i = 0; i < 8; ++i) {
        for (int j : inputs)
            if (overlaps(all[outputs[i]], bytes[outputs[i]], all[j], bytes[j]))
                return NVFP4_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(all[outputs[i]], bytes[outputs[i]], all[outputs[j]], bytes[outputs[j]]))
                return NVFP4_ERR_ALIAS;
    }
    int dev, sms;
    nvfp4_host::EncodeFn encode;
    int st = nvfp4_host::device(&dev, &sms, &encode);
    if (st != NVFP4_OK) return st;
    PlanParams p;
    memset(&p, 0, sizeof(p));
    p.lens = a.lens;
    p.fresh = a.new_tokens;
    p.table = a.table;
    p.ld_table = a.ld_table;
    p.columns = a.table_columns;
    p.free_pages = a.free_pages;
    p.n_free = a.free_count;
    p.head = a.head;
    p.tokens = a.tokens;
    p.starts = a.starts;
    p.lens_out = a.lens_out;
    p.slots = a.slots;
    p.request = a.request;
    p.positions = a.positions;
    p.head_out = a.head_out;
    p.missing = a.missing;
    p.requests = a.requests;
    p.block = a.block_size;
    const size_t smem = 16ull * a.requests;
    if (smem > 40 * 1024 &&  // (48 KB are open without, the kernel's own arrays among them)
        cudaFuncSetAttribute(nvfp4_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             16 * NVFP4_MAX_REQUESTS) != cudaSuccess) {
        cudaGetLastError();
        return NVFP4_ERR_LAUNCH;
    }
    const int64_t want = (a.tokens + a.requests + kPlanThreads - 1) / kPlanThreads;
    const int grid = (int)(want < 1 ? 1 : want > sms ? sms : want);
    return nvfp4_host::launch_behind(nvfp4_plan_kernel, grid, kPlanThreads, smem, 0, stream, p);
}

int nvfp4_kv_append(const void* k, int64_t ldk, int64_t k_head_stride, const void* v, int64_t ldv,
                    int64_t v_head_stride, int64_t tokens, const int32_t* slots,
                    const nvfp4_kv_cache_t* cache, cudaStream_t stream) {
    int st = nvfp4_host::check_cache(cache);
    if (st != NVFP4_OK) return st;
    const nvfp4_kv_cache_t& c = *cache;
    if (tokens < 0 || tokens > INT32_MAX || ldk < c.dim || ldv < c.dim || k_head_stride < c.dim ||
        v_head_stride < c.dim)
        return NVFP4_ERR_SHAPE;
    if (tokens == 0 || c.blocks == 0) return NVFP4_OK;
    if (!k || !v || !slots) return NVFP4_ERR_NULL;
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(slots, 4) || ldk % 8 || ldv % 8 ||
        k_head_stride % 8 || v_head_stride % 8)
        return NVFP4_ERR_ALIGN;
    const uint64_t cache_bytes = nvfp4_host::cache_bytes(c);
    const uint64_t kb = 2 * nvfp4_host::span(1, 0, tokens, ldk, c.heads, k_head_stride, c.dim);
    const uint64_t vb = 2 * nvfp4_host::span(1, 0, tokens, ldv, c.heads, v_head_stride, c.dim);
    const void* caches[2] = {c.k, c.v};
    if (c.k == c.v) return NVFP4_ERR_ALIAS;  // (they may lie in one buffer, page by page)
    for (const void* dst : caches)
        if (overlaps(dst, cache_bytes, k, kb) || overlaps(dst, cache_bytes, v, vb) ||
            overlaps(dst, cache_bytes, slots, 4ull * tokens))
            return NVFP4_ERR_ALIAS;
    int dev, sms;
    nvfp4_host::EncodeFn encode;
    st = nvfp4_host::device(&dev, &sms, &encode);
    if (st != NVFP4_OK) return st;
    AppendParams p;
    memset(&p, 0, sizeof(p));
    p.src[0] = static_cast<const uint16_t*>(k);
    p.src[1] = static_cast<const uint16_t*>(v);
    p.ld[0] = ldk;
    p.ld[1] = ldv;
    p.head_stride[0] = k_head_stride;
    p.head_stride[1] = v_head_stride;
    p.cache[0] = static_cast<uint8_t*>(c.k);
    p.cache[1] = static_cast<uint8_t*>(c.v);
    p.scale[0] = c.k_scale;
    p.scale[1] = c.v_scale;
    for (int i = 0; i < 2; ++i) {
        int exponent = 0;  // biased, of the least values that are divided: all of them by default
        if (p.scale[i] >= 1e-15f && p.scale[i] <= 1e15f) {
            p.inverse[i] = 1.f / p.scale[i];
            p.rest[i] = (float)(1.0 / p.scale[i] - p.inverse[i]);
            int e;  // scale is in [2^(e - 1), 2^e)
            frexpf(p.scale[i], &e);
            exponent = 127 + 63 + e;  // 141 to 240: quotients below are less than 2^64
        }
        p.far[i] = (0x8000u - ((uint32_t)exponent << 7)) * 0x10001u;
    }
    p.slots = slots;
    p.tokens = tokens;
    p.blocks = c.blocks;
    p.block_stride = c.block_stride;
    p.slot_stride = c.slot_stride;
    p.cache_head_stride = c.head_stride;
    p.heads = c.heads;
    p.dim = c.dim;
    p.block = c.block_size;
    // Few rows: a warp each.  More than the GPU's warps can be at once: K and V of a token in one, with
    // twice the loads under way (e4m3: 8192 tokens 11.1 us against 12.9, 4000 tokens 6.6 against 8.0, 128
    // tokens 2.5 against 2.1; bf16: 13.1 against 12.5, 8.2 against 7.7, 2.7 against 1.8).
    const int most = 8 * sms;
    const bool both = tokens * 2 > (int64_t)most * (kAppendThreads / 32);
    const int64_t want = (tokens * (both ? 1 : 2) * 32 + kAppendThreads - 1) / kAppendThreads;
    const int grid = (int)(want > most ? most : want);
    const bool f8 = c.type == NVFP4_KV_E4M3;
    return nvfp4_host::launch_behind(
        both ? f8 ? nvfp4_append_kernel<true, 2> : nvfp4_append_kernel<false, 2>
             : f8 ? nvfp4_append_kernel<true, 1> : nvfp4_append_kernel<false, 1>,
        grid, kAppendThreads, 0, 0, stream, p);
}

}  // extern "C"

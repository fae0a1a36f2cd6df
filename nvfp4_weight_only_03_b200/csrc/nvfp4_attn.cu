// Attention of each request's newest tokens over its paged key/value cache (nvfp4_paged_attn):
// one token of a decode step, the rows of a verify round, a prefill chunk.  The decode plan
// launches it as paged_decode_attn ("Blueprint - circuit executor" page for qwen3.8-27b-nvfp4 on
// GB10, table "Kernels the plan launches").
//
//   token t of request r, starts[r] <= t < starts[r + 1]: p = lens[r] - starts[r + 1] + t
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j),  over the keys j <= p that have a page
//
// * Rows: the query heads that share a kv head are rows of one matrix product, row g of a request
//   being (token g / G, head g % G); 128 rows are a tile (the MMA's M), so a key or value row
//   leaves HBM once per tile and kv head.  A decode step fills 6 of the 128 rows: the tensor
//   cores have the time (1024 cycles of MMA against some 2800 of HBM per 64 KB of cache), and one
//   kernel serves every row count.
// * Work: units of TK keys of one (request, kv head, row tile).  All units in order are cut into
//   equal ranges, one per CTA (one CTA per SM), from the lengths in device memory: the host knows
//   none of them, so a captured call serves every later length.  A tile that a range boundary
//   cuts leaves (max, sum, O) in the workspace, and a second kernel joins the parts in order (or,
//   where all rows are few, the CTA that is last to leave its part).  Results are the same in every
//   run.
// * One pass over the cache: S = Q K^T in tensor memory, one thread per row keeps the running
//   maximum and sum, P goes back to tensor memory as the A operand of O += P V.  O stays in tensor
//   memory; it is rescaled only when a row's maximum rose by more than 2^8 (P is then at most
//   2^8 and the sums are fp32, so nothing overflows).  S and P have two buffers each, so the MMAs
//   of one unit run under the softmax of another.
// * Roles: 8 softmax warps, one warp each for the scores' MMAs, the values' MMAs, K, and Q and V; with
//   an e4m3 cache 4 more that widen V to f16 (exact) and split Q.  All else goes to the MMA as it lies
//   in memory.  The roles share the instruction cache: uniform operands, elected lanes and short loops
//   decide the time more than their count of operations.
// * P is rounded to the MMA's 16-bit type (bf16, or f16 with the e4m3 cache): half a step, 2^-8
//   (2^-11) of each weight.  f16 weights are 2^7 times the formula's, so they reach 2^15 and keep all
//   their bits down to 2^-21 of the row's reference; below, half a step is 2^-32 of it (without the
//   factor 2^-25 a key, and the many small weights beside a dominating one were lost).  The sums
//   carry the factor as well.  With the e4m3 cache K is read by 8-bit MMAs as it lies, q being carried
//   as two e4m3 terms times a power of two per row (an error of at most 2^-17 of the row's largest).
//   S, O, maxima and sums are fp32.
// * Measured (B200, calls of a captured graph): 64 requests of up to 8192 keys, 24 heads on 4 of
//   256, one token each: 166 us, 6.05 TB/s, 94% of the copy rate; one request of 131072 keys: 103 us,
//   80% (parts of its 4 heads' single row tiles are joined by one CTA each); 16 requests x 8 tokens,
//   e4m3, 32 heads on 8 of 128: 93 us, 48% (widening V and the one softmax warp that has rows);
//   2048 tokens over 16384 keys: 705 us, 1096 TFLOP/s, 65% of the matrix rate (the tensor pipe is busy
//   for half of its cycles).  The least call is some 7 us: lengths, first pages, keys, scores, weights
//   and values follow on one another, each with its latency.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "nvfp4.h"
#include "nvfp4_host.h"
#include "nvfp4_ptx.h"

namespace nvfp4_host {
int check_cache(const nvfp4_kv_cache_t* c);
}

namespace {

using namespace nvfp4_ptx;
using nvfp4_host::misaligned;
using nvfp4_host::overlaps;

constexpr int kRows = 128;  // rows of a tile: the MMA's M and tensor memory's lanes
constexpr int kSoftmaxWarps = 8, kScoresWarp = 8, kTmaWarp = 9, kValuesWarp = 10, kQWarp = 11;
constexpr int kWidenWarp = 12, kWidenWarps = 4;
constexpr int kTmemCols = 512;
constexpr size_t kSmemMost = 232448;  // shared memory of a block

// The small things in shared memory, ahead of the tiles.
template <int NK, int NV, int NR, bool F8>
struct Small {
    uint64_t full[NK + NV], empty[NK + NV];  // of the K places, then of the V places
    uint64_t raw_full[NR], raw_empty[NR];
    uint64_t q_full, q_free, s_full[2], p_full[2], pv_done[2], o_full, o_free, drained[2];
    int64_t sums[20];
    int start[2][12];  // a Cursor: where the range begins; then, by turns, the softmax's next tile
    uint32_t tmem;
    int stop, last;
    int partly[8];  // item + 1 where V of a key that not all rows see is not finite; [item's place]
    float row_max[2][kRows];  // a unit's reference maximum: [its parity][row]
    float row_sum[2][kRows];  // a row tile's sum of weights: [warpgroup][row]
    // biased exponents of the 8-bit Q rows' scales.  Q may be two row tiles ahead of the softmax.
    uint8_t q_scale[F8 ? 4 : 1][F8 ? kRows : 1];
};

template <int D, bool F8>
struct Cfg {
    static constexpr int TK = D == 256 ? 64 : 128;    // keys per unit
    static constexpr int kQBytes = kRows * D * 2;     // bf16, or two 8-bit terms
    static constexpr int kKey = TK * D * (F8 ? 1 : 2);  // a K tile
    static constexpr int kVal = TK * D * 2;           // a V tile, 16-bit
    static constexpr int kRaw = F8 ? TK * D : 0;      // the same in e4m3
    static constexpr int kRow = F8 && D == 64 ? 64 : 128;  // bytes of a row of a panel of Q and K
    static constexpr int kRowKeys = F8 ? kRow : 64;   // its values
    static constexpr int kPanels = D / kRowKeys;      // panels of Q and K
    static constexpr int kThreads = 32 * (F8 ? kWidenWarp + kWidenWarps : kQWarp + 1);
    static constexpr size_t kHead = F8 ? 4096 : 3 * 1024;  // Small, in front of the tiles
    // Places of K, of V and of V as it lies in an e4m3 cache.  K and V have rings of their own, since
    // their readers go on independently (with one ring, a reader could take the phase of the
    // other's tile for that of its own).
    static constexpr int kStages = (int)((kSmemMost - kHead - kQBytes) / kVal);
    static constexpr int NK = F8 ? (D == 64 ? 6 : D == 128 ? 4 : 3) : kStages / 2;
    static constexpr int NV = F8 ? (D == 64 ? 4 : 2) : kStages - NK;
    static constexpr int NR = F8 ? (D == 64 ? 6 : D == 128 ? 3 : 2) : 1;
    static constexpr size_t kSmem = kHead + kQBytes + (size_t)NK * kKey + (size_t)NV * kVal +
                                    (F8 ? (size_t)NR * kRaw : 0);
    using Shared = Small<NK, NV, NR, F8>;
    // tensor memory columns: O, then two S, then two P (two 16-bit values per column)
    static constexpr int kS = D, kP = D + 2 * TK, kEnd = D + 2 * TK + TK;
    static_assert(kEnd <= kTmemCols, "tensor memory");
    static_assert(NK >= 1 && NV >= 2, "rings");
    static_assert(kSmem <= kSmemMost && sizeof(Shared) <= kHead, "shared memory");
};

// A row tile that was cut: its parts lie with the CTAs `owner` (which holds its first unit) to
// owner + parts - 1.
struct Cut {
    int32_t parts;  // 0: this CTA owns none
    int32_t token0, row0, rows, head;
    int32_t pad[3];
};

// n / d for 0 <= n < 2^31 by a multiplication with ceil(2^(31 + L) / d), L = ceil(log2 d), whose
// excess over 2^(31 + L) / d is below 1 and so moves the quotient by less than 2^-L <= 1 / d.  (A
// division by a variable is a longer sequence, and the roles of a block share the instruction cache.)
struct Divisor {
    uint32_t mul, shift;
};
__device__ __forceinline__ uint32_t div_by(uint32_t n, Divisor d) {
    return d.mul ? __umulhi(n, d.mul) >> d.shift : n;
}
inline Divisor divisor_of(uint32_t d) {
    uint32_t log = 0;
    while ((1ull << log) < d) ++log;
    Divisor r = {0, 0};  // d = 1
    if (log > 0) {
        r.mul = (uint32_t)(((1ull << (31 + log)) + d - 1) / d);
        r.shift = log - 1;
    }
    return r;
}
// a / b, neither negative.  Every call waits for three of these before its first load, so small ones are
// approximated in fp32 (off by one at most) and put right.
__device__ __noinline__ int64_t div64(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if ((uint64_t)(a | b) >> 22) return div64(a, b);
    const int x = (int)a, y = (int)b;
    int q = (int)__fdividef((float)x, (float)y);
    const int left = x - q * y;
    q += left >= y;
    return q - (left < 0);
}

struct Params {
    const uint16_t* q;
    int64_t ldq, q_head_stride;
    uint16_t* o;
    int64_t ldo, o_head_stride;
    const int32_t* table;
    int64_t ld_table;
    const int32_t *starts, *lens;
    int requests, tokens, kv_heads, group, block, blocks, box;
    Divisor by_group, by_block;
    int outside;       // a page index past the tensor: its boxes arrive as zeros
    int capacity;      // keys that a table row can hold
    const void* v;     // the cache's values and strides (elements), for what is read without TMA
    int64_t block_stride, slot_stride, head_stride;
    // What beginning and ending a row tile costs, in units: Q's rows, the first scores and the epilogue
    // pass without overlap.  The split counts it, or a CTA with many short row tiles would be the
    // last by far.
    int tile_cost;
    float c;           // scale * k_scale * log2(e)
    float v_scale;     // (1 with a bf16 cache)
    int32_t* error;
    int join_here;     // rows are few: the last CTA of a cut row tile joins its parts itself
    int32_t* arrived;  // [grid]: parts of CTA i's cut row tile written so far; zero between calls
    Cut* cuts;         // [grid]
    float2* part_ml;   // [grid][2][128]: maximum (of q.k) and sum
    float* part_o;     // [grid][2][D / 4][128][4]: a warp's rows side by side
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack16(bool f16, float lo, float hi) {
    uint32_t r;
    if (f16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four e4m3 codes (bytes 0..3) -> f16 values times 2^-8, exact, as the pairs {0, 2} and {1, 3}: a
// code's exponent and mantissa, seven bits, moved to the same place below f16's exponent bias (15
// against 7), subnormals included; the factor goes into the output's scale.  Seven
// shifts and masks; cvt has the rate of the exponentials and shares their pipe.  O comes out in the
// pairs' order and is put right where it is written.
__device__ __forceinline__ void widen(uint32_t w, uint32_t& even, uint32_t& odd) {
    even = ((w << 8) & 0x80008000u) | ((w << 7) & 0x3f803f80u);
    odd = (w & 0x80008000u) | ((w >> 1) & 0x3f803f80u);
}
// The same by cvt, for words with a NaN code (which the above takes for 480).
__device__ __forceinline__ void widen_nan(uint32_t w, uint32_t& even, uint32_t& odd) {
    const uint32_t x = __byte_perm(w, 0, 0x3120);
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t"
        "mul.rn.f16x2 %0, %0, %3;\n\tmul.rn.f16x2 %1, %1, %3;\n\t}"
        : "=&r"(even), "=&r"(odd)
        : "r"(x), "r"(0x1c001c00u));  // 2^-8 twice
}
constexpr float kWidened = 256.f;
constexpr float kLift = 7.f;  // f16 weights are stored times 2^kLift
constexpr uint32_t kWidenedNan = 0x3f80;  // what widen makes of a NaN code, 480 / 256: above all others
// The larger magnitude of each half (its sign is of no use).
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two f16 values as e4m3 codes, and back.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t f16x2) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(f16x2));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_values(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return h;
}

// ---- the order of the work ---------------------------------------------------------------

struct Request {
    int token0, n, pos;  // first row, rows, position of the first row's token (below 0: sees no key)
};

// Device data is taken as it is, within bounds: a request outside [0, tokens] is cut to it.  What is
// cut off at its end still counts for the positions: starts[r + 1] is the one behind the last of lens[r].
__device__ __forceinline__ Request request_of(const Params& p, int r) {
    const int end = p.starts[r + 1];
    Request q;
    q.token0 = min(max(p.starts[r], 0), p.tokens);
    q.n = min(max(end, q.token0), p.tokens) - q.token0;
    q.pos = max(p.lens[r], 0) - (max(end, q.token0) - q.token0);
    return q;
}

__device__ __forceinline__ int row_tiles(const Params& p, const Request& q) {
    return (q.n * p.group + kRows - 1) / kRows;  // (tokens * group is at most 2^30)
}

// Keys below this are loaded for a row tile: the last row's own position, within the table.
__device__ __forceinline__ int key_end(const Params& p, const Request& q, int tile) {
    const int rows = min((tile + 1) * kRows, q.n * p.group);
    const int last = (int)div_by(rows - 1, p.by_group);
    return min(max(q.pos + last + 1, 0), p.capacity);
}

// Keys from this one on are seen by some rows of the row tile only: its first row's position + 1.
__device__ __forceinline__ int key_open(const Params& p, const Request& q, int tile) {
    return max(q.pos + (int)div_by(tile * kRows, p.by_group) + 1, 0);
}

template <int TK>
__device__ __forceinline__ int units_of(const Params& p, const Request& q, int tile) {
    return max(1, (key_end(p, q, tile) + TK - 1) / TK);  // 1: rows without keys are written too
}

template <int TK>
struct Cursor {
    int r, h, tile, tiles, u, n;  // unit u of the row tile's n
    int lead;                     // how much of tile_cost counts here: all, unless a cut fell in it
    Request q;
    // Units of this row tile in a range with `left` to go; none: the range is done.
    __device__ __forceinline__ int take(int left) const {
        return min(n - u, left - lead);
    }
    __device__ __forceinline__ void enter(const Params& p) {
        tiles = row_tiles(p, q);
        n = units_of<TK>(p, q, tile);
    }
    __device__ __forceinline__ void next(const Params& p) {  // the next row tile
        u = 0;
        lead = p.tile_cost;
        if (++tile == tiles) {
            tile = 0;
            if (++h == p.kv_heads) {
                h = 0;
                do {
                    if (++r >= p.requests) return;  // the last one: nothing is left to do
                    q = request_of(p, r);
                } while (q.n == 0);
                tiles = row_tiles(p, q);
            }
        }
        n = units_of<TK>(p, q, tile);
    }
};

// A reader's or writer's place in a ring of N tiles, and the phase of its barriers.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t phase;
    __device__ explicit Ring(uint32_t first) : phase(first) {}
    __device__ __forceinline__ void step() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1;
        }
    }
};

constexpr int kMinUnits = 2;  // fewest units worth a CTA of their own

struct Range {
    int64_t begin, end, total;
    int ctas;
};

__device__ __forceinline__ int64_t range_begin(int64_t total, int ctas, int c) {
    return quotient(total * c, ctas);
}

// This CTA's units and the row tile they start in.  Every thread sums the units of a run of
// requests; the thread that holds the first one walks to it.
template <int TK, int THREADS>
__device__ __forceinline__ Range find_range(const Params& p, Cursor<TK>* start, int64_t* sums) {
    const int tid = threadIdx.x;
    if (tid == 0) start->r = -1;  // behind the first __syncthreads at the latest
    const int per = (p.requests + THREADS - 1) / THREADS;
    const int r0 = min(tid * per, p.requests), r1 = min(r0 + per, p.requests);
    int64_t mine = 0, s = 0;
    Request q;
    auto weigh = [&](int r) {  // q, and s: the units of one of its heads
        q = request_of(p, r);
        const int tiles = row_tiles(p, q);
        s = 0;
        for (int t = 0; t < tiles; ++t) s += units_of<TK>(p, q, t) + p.tile_cost;
    };
    for (int r = r0; r < r1; ++r) {
        weigh(r);
        mine += s * p.kv_heads;
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t a = __shfl_up_sync(~0u, incl, d);
        if ((tid & 31) >= d) incl += a;
    }
    if ((tid & 31) == 31) sums[tid >> 5] = incl;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < (tid >> 5)) before += sums[w];
        total += sums[w];
    }
    before += incl - mine;
    Range g;
    g.total = total;
    const int64_t most = (total + kMinUnits - 1) / kMinUnits;
    g.ctas = (int)(most < (int64_t)gridDim.x ? most : (int64_t)gridDim.x);
    g.begin = g.end = 0;
    if ((int)blockIdx.x < g.ctas) {
        g.begin = range_begin(total, g.ctas, blockIdx.x);
        g.end = range_begin(total, g.ctas, blockIdx.x + 1);
    }
    if (g.end > g.begin && before <= g.begin && g.begin < before + mine) {
        int64_t at = g.begin - before;
        for (int r = r0; r < r1; ++r) {
            if (per > 1) weigh(r);
            if (at >= s * p.kv_heads) {
                at -= s * p.kv_heads;
                continue;
            }
            Cursor<TK> c;
            c.r = r;
            c.q = q;
            c.h = (int)quotient(at, s);
            at -= c.h * s;
            c.tile = 0;
            while (at >= units_of<TK>(p, q, c.tile) + p.tile_cost)
                at -= units_of<TK>(p, q, c.tile++) + p.tile_cost;
            c.lead = (int)max((int64_t)p.tile_cost - at, (int64_t)0);
            c.u = (int)max(at - p.tile_cost, (int64_t)0);
            c.enter(p);
            *start = c;
            break;
        }
    }
    __syncthreads();
    // lengths that change while the call runs (another stream writes them) may leave no row tile
    // to start in: the results are then whatever they are, but nothing is read out of bounds
    if (g.end > g.begin && start->r < 0) g.end = g.begin;
    return g;
}

// ---- V that is not finite -------------------------------------------------------------------
// In the product a weight of zero times an infinity or NaN is NaN, and a key that comes after a
// row's own position has such a weight.  So where V of a key that only some rows of the row tile see
// is not finite, the product gets a zero in its place, and the rows that see it get the value
// itself here: it decides their result whatever the weights are.  One thread, its row's columns
// col .. col + cols - 1, behind the result (out) or the part that it wrote.
template <bool F8>
__device__ __noinline__ void add_not_finite(const Params& p, const int32_t* table, int head, int key,
                                            int key_to, int col, int cols, uint16_t* out, float* part) {
    for (; key < key_to; ++key) {
        const int c = (int)div_by(key, p.by_block), page = table[c];
        if ((unsigned)page >= (unsigned)p.blocks) continue;
        const int64_t at = page * p.block_stride + (key - c * p.block) * p.slot_stride +
                           head * p.head_stride;
        for (int i = col; i < col + cols; ++i) {
            float v;
            if (F8)
                v = (static_cast<const uint8_t*>(p.v)[at + i] & 0x7f) == 0x7f ? NAN : 0.f;
            else
                v = __uint_as_float((uint32_t)static_cast<const uint16_t*>(p.v)[at + i] << 16);
            if (isfinite(v)) continue;
            if (part)
                part[i / 4 * (kRows * 4) + i % 4] += v;
            else
                out[i] = (uint16_t)pack16(false, __uint_as_float((uint32_t)out[i] << 16) + v, 0.f);
        }
    }
}

// A unit's scores in tensor memory, less a lane's `by`.  (Rare, and so out of the way of the code that
// every unit runs.)
template <int TK>
__device__ __noinline__ void subtract_scores(uint32_t at, float by) {
#pragma unroll 1
    for (int i = 0; i < TK / 32; ++i) {
        uint32_t s[32];
        tmem_ld(at + i * 32, s);
        tmem_wait_ld(s);
#pragma unroll
        for (int e = 0; e < 32; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) - by);
        tmem_st(at + i * 32, s);
    }
    tmem_wait_st();
}

// Row `row` (of all the request's) of the cursor's head.
template <int TK>
__device__ __forceinline__ const uint16_t* q_row(const Params& p, const Cursor<TK>& cur, int row) {
    const int tok = (int)div_by(row, p.by_group);
    return p.q + (int64_t)(cur.q.token0 + tok) * p.ldq +
           (int64_t)(cur.h * p.group + row - tok * p.group) * p.q_head_stride;
}

// ---- joining the parts of a cut row tile, in their order -------------------------------------
// Part 0 lies with its CTA's cut at the end, the others with their cuts at the start.  A thread
// takes 8 columns of a row, its neighbours those of the next rows, as the parts lie.
template <int D, bool F8>
__device__ __noinline__ void join_rows(const Params& p, int owner, const Cut& cut, int item, int step) {
    for (; item < cut.rows * (D / 8); item += step) {
        const int oct = item / cut.rows, row = item - oct * cut.rows;
        auto at = [&](int i) { return ((int64_t)(owner + i) * 2 + (i == 0)) * kRows; };
        float acc[8], sum = 0.f, top = -INFINITY;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        constexpr int kSome = 8;  // parts read at once: the loads' latency is what this takes
#pragma unroll 1
        for (int i0 = 0; i0 < cut.parts; i0 += kSome) {
            float2 ml[kSome];
            float4 u[kSome], v[kSome];
#pragma unroll
            for (int j = 0; j < kSome; ++j) {
                ml[j] = make_float2(-INFINITY, 0.f);
                u[j] = v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + j < cut.parts) {
                    const int64_t a = at(i0 + j);
                    const float4* const src =
                        reinterpret_cast<const float4*>(p.part_o + a * D) + oct * 2 * kRows + row;
                    ml[j] = __ldcg(&p.part_ml[a + row]);
                    u[j] = __ldcg(src), v[j] = __ldcg(src + kRows);
                }
            }
            const float was = top;
#pragma unroll
            for (int j = 0; j < kSome; ++j) top = fmaxf(top, ml[j].x);
            // (parts that saw no key have a weight of zero and zeros to weigh)
            const float ref = top == -INFINITY ? 0.f : top, f = exp2_approx((was - ref) * p.c);
            sum *= f;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] *= f;
#pragma unroll
            for (int j = 0; j < kSome; ++j) {
                const float w = exp2_approx((ml[j].x - ref) * p.c);
                sum = fmaf(w, ml[j].y, sum);
                acc[0] = fmaf(w, u[j].x, acc[0]), acc[1] = fmaf(w, u[j].y, acc[1]);
                acc[2] = fmaf(w, u[j].z, acc[2]), acc[3] = fmaf(w, u[j].w, acc[3]);
                acc[4] = fmaf(w, v[j].x, acc[4]), acc[5] = fmaf(w, v[j].y, acc[5]);
                acc[6] = fmaf(w, v[j].z, acc[6]), acc[7] = fmaf(w, v[j].w, acc[7]);
            }
        }
        const float inv = sum == 0.f ? 0.f : (F8 ? kWidened : p.v_scale) / sum;
        const float last = F8 ? p.v_scale : 1.f;  // (its product with the others may leave fp32's range)
        const int tok = (int)div_by(cut.row0 + row, p.by_group);
        uint4 o;
        uint32_t* const oo = &o.x;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            oo[e] = pack16(false, acc[2 * e] * inv * last, acc[2 * e + 1] * inv * last);
        *reinterpret_cast<uint4*>(
            p.o + (int64_t)(cut.token0 + tok) * p.ldo +
            (int64_t)(cut.head * p.group + cut.row0 + row - tok * p.group) * p.o_head_stride +
            oct * 8) = o;
    }
}

constexpr int kJoinThreads = 256;

template <int D, bool F8>
__global__ void __launch_bounds__(kJoinThreads) nvfp4_attn_join_kernel(const __grid_constant__ Params p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Cut cut = p.cuts[blockIdx.y];
    if (cut.parts <= 0) return;
    join_rows<D, F8>(p, blockIdx.y, cut, blockIdx.x * kJoinThreads + threadIdx.x,
                 gridDim.x * kJoinThreads);
}

// ---- the kernel --------------------------------------------------------------------------

template <int D, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::kThreads, 1)
    nvfp4_attn_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
    using C = Cfg<D, F8>;
    constexpr int TK = C::TK, NK = C::NK, NV = C::NV, NR = C::NR;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    typename C::Shared& sm = *reinterpret_cast<typename C::Shared*>(smem_raw);
    uint8_t* const q_tile = smem_raw + C::kHead;
    uint8_t* const key_ring = q_tile + C::kQBytes;
    uint8_t* const val_ring = key_ring + NK * C::kKey;
    uint8_t* const raw = val_ring + NV * C::kVal;
    uint64_t *const full = sm.full, *const empty = sm.empty, *const s_full = sm.s_full,
             *const p_full = sm.p_full;
    // (the tiles' swizzle wants 1024-byte alignment, which the block's only allocation has)
    if (smem_u32(smem_raw) & 1023u) {
        if (threadIdx.x == 0) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            atomicCAS(p.error, 0, 10);
            p.cuts[blockIdx.x].parts = 0;
        }
        return;
    }
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    if (warp == kScoresWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sm.tmem)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        for (int i = 0; i < NK + NV; ++i) {
            mbar_init(&full[i], F8 && i >= NK ? kWidenWarps : 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NR; ++i) {
            mbar_init(&sm.raw_full[i], 1);
            mbar_init(&sm.raw_empty[i], kWidenWarps);
        }
        mbar_init(&sm.q_full, F8 ? kWidenWarps : 1);
        mbar_init(&sm.q_free, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], kSoftmaxWarps / 2);
            mbar_init(&sm.pv_done[i], 1);
            mbar_init(&sm.drained[i], 1);
        }
        mbar_init(&sm.o_full, 1);
        mbar_init(&sm.o_free, kSoftmaxWarps);
        sm.stop = 0;
        for (int i = 0; i < 8; ++i) sm.partly[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&map_k);
        prefetch_map(&map_v);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_before_sync();
    Cursor<TK>* const start = reinterpret_cast<Cursor<TK>*>(sm.start[0]);
    static_assert(sizeof(Cursor<TK>) <= sizeof(sm.start[0]) && C::kThreads / 32 <= 20, "Small");
    const Range range = find_range<TK, C::kThreads>(p, start, sm.sums);  // two __syncthreads
    tc_after_sync();
    const uint32_t tmem = sm.tmem;
    volatile int* const stop_v = &sm.stop;
    int left = (int)min(range.end - range.begin, (int64_t)INT32_MAX);
    Cursor<TK> cur = *start;
    bool ok = true;
    int code = 0;

    if (tid == 0) p.cuts[blockIdx.x].parts = 0;
    if (left == 0) {
        // nothing to do
    } else if (warp == kTmaWarp || warp == kQWarp) {
        // ---- what the products read: one warp copies the K tiles, another gathers Q's rows (bf16) and
        // copies the V tiles (of an e4m3 cache, to where they are widened); one warp alone was the
        // kernel's bound with pages of 16 keys.  A tile is TK / box groups of `box` keys of one page
        // each (lane i knows group i's page and place), and a group is a box per panel.  Keys past the
        // end, and pages that do not exist, are boxes outside the tensor, which arrive as zeros.  One
        // elected lane issues all of a tile's boxes: a divergent issue, a lane per box, was slower.
        constexpr int kMost = TK / 16;
        const bool second = warp == kQWarp;
        const int groups = TK / p.box;
        const int places = !second ? NK : F8 ? NR : NV;
        uint64_t* const fulls = !second ? full : F8 ? sm.raw_full : full + NK;
        uint64_t* const empties = !second ? empty : F8 ? sm.raw_empty : empty + NK;
        const uint32_t room = smem_u32(!second ? key_ring : F8 ? raw : val_ring);
        const int bytes = !second ? C::kKey : F8 ? C::kRaw : C::kVal;
        const CUtensorMap* const map = second ? &map_v : &map_k;
        // 128-byte (64-byte) rows of a panel, or, where V is widened, whole rows
        const bool whole_rows = F8 && second;
        const int step = p.box * (whole_rows ? D : C::kRow);  // bytes of a group (in a panel)
        int slot = 0, it = 0, item = 0;
        uint32_t phase = 1;  // (the first lap finds every place free)
        // Q's rows in the MMA's layout (K-major, 128-byte swizzle): a lane finds the address of a row
        // in 32, D / 8 lanes copy it
        auto gather = [&]() {
            if (item > 0 &&
                !(ok = __all_sync(~0u, mbar_wait(&sm.q_free, (item - 1) & 1, stop_v))))
                return;
            const int row0 = cur.tile * kRows;
            const int rows = min(kRows, cur.q.n * p.group - row0);
            constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;  // lanes per row, rows at once
            const int c = lane % kLanes, sub = lane / kLanes;
            const uint32_t dst0 = smem_u32(q_tile) + (c >> 3) * (kRows * 128);
            for (int r0 = 0; r0 < rows; r0 += 32) {
                const uint16_t* const mine = q_row(p, cur, row0 + min(r0 + lane, rows - 1));
                const int some = min(32, rows - r0);
#pragma unroll 8
                for (int i = 0; i < some; i += kAtOnce) {
                    const int r = r0 + i + sub;
                    const uint16_t* const src = reinterpret_cast<const uint16_t*>(
                        __shfl_sync(~0u, reinterpret_cast<unsigned long long>(mine), i + sub));
                    if (r < rows)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                         dst0 + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                                     "l"(src + c * 8)
                                     : "memory");
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_full);
        };
        while (left > 0 && ok) {
            const int cnt = uniform(cur.take(left));
            if (cnt <= 0) break;
            if (!F8 && second) {
                gather();
                if (!ok) break;
            }
            const int end = key_end(p, cur.q, cur.tile), head = uniform(cur.h);
            const int32_t* const row = p.table + cur.r * p.ld_table;
            // this lane's page and place in unit j of the range
            auto page_at = [&](int j, int& place) {
                const int key = (cur.u + j) * TK + lane * p.box;  // (j may be past cnt)
                place = 0;
                if (j >= cnt || lane >= groups || key >= end) return p.outside;
                const int col = (int)div_by(key, p.by_block);
                place = key - col * p.block;
                return row[col];
            };
            // pages are read ahead of their unit's first box
            int place0, place1, place2;
            int page0 = page_at(0, place0), page1 = page_at(1, place1), page2 = page_at(2, place2);
            for (int i = 0; i < cnt; ++i) {
                const int at = (unsigned)page0 < (unsigned)p.blocks ? page0 : p.outside;
                int w[kMost], y[kMost];
#pragma unroll
                for (int x = 0; x < kMost; ++x) {
                    w[x] = __shfl_sync(~0u, at, x);
                    y[x] = __shfl_sync(~0u, place0, x);
                }
                const uint32_t fb = uniform(smem_u32(fulls + slot));
                const uint32_t dst = uniform(room + slot * bytes);
                ok = __all_sync(~0u, mbar_wait(empties + slot, phase, stop_v));
                if (!ok) break;
                if (elect_one()) {
                    mbar_expect_tx(fb, bytes);
#pragma unroll
                    for (int x = 0; x < kMost; ++x) {
                        if (x >= groups) break;
                        if (whole_rows) {
                            tma_load_4d(dst + x * step, map, 0, y[x], head, w[x], fb);
                        } else {
#pragma unroll
                            for (int pn = 0; pn < C::kPanels; ++pn)
                                tma_load_4d(dst + pn * (TK * C::kRow) + x * step, map,
                                            pn * C::kRowKeys, y[x], head, w[x], fb);
                        }
                    }
                }
                __syncwarp();
                ++it;
                if (++slot == places) {
                    slot = 0;
                    phase ^= 1;
                }
                page0 = page1, place0 = place1;
                page1 = page2, place1 = place2;
                page2 = page_at(i + 3, place2);
            }
            ++item;
            left -= cur.lead + cnt;
            cur.next(p);
        }
        if (!ok) {  // a CTA that gives up leaves no copy in flight behind it
            code = second ? 7 : 5;
            volatile int none = 0;
            for (int k = max(0, it - places); k < it; ++k)
                mbar_wait(fulls + k % places, (k / places) & 1, &none, 20000000ll);
        }
    } else if (warp == kScoresWarp || warp == kValuesWarp) {
        // ---- MMAs, one elected lane: a warp for S = Q K^T and one for O += P V, so that the next
        // product waits in the tensor core's queue while a warp looks after its barriers.
        // Unit g's scores need the weights of g - 2 formed (whose scores had their place).
        const bool values = warp == kValuesWarp;
        constexpr uint32_t id_s = F8 ? idesc_8(TK) : idesc_16(true, TK, false);
        constexpr uint32_t id_o = idesc_16(!F8, D, true);
        const uint32_t q_low = uniform(smem_u32(q_tile) >> 4);
        int g = 0, item = 0;
        Ring<NK> keys(0);
        Ring<NV> vals(0);
        auto ready = [&](uint64_t* b, uint32_t parity) {
            ok = __all_sync(~0u, mbar_wait(b, parity, stop_v));
            return ok;
        };
        while (left > 0 && ok) {
            const int cnt = uniform(cur.take(left));
            if (cnt <= 0) break;
            if (!values) {
                if (!ready(&sm.q_full, item & 1)) break;
                for (int j = 0; j < cnt; ++j, ++g) {
                    const int slot = keys.slot;
                    if (!ready(&full[slot], keys.phase)) break;
                    if (g >= 2 && !ready(&p_full[g & 1], ((g >> 1) - 1) & 1)) break;
                    const uint32_t low = uniform((smem_u32(key_ring) + slot * C::kKey) >> 4);
                    const uint32_t d = uniform(tmem + C::kS + (g & 1) * TK);
                    tc_after_sync();
                    if (elect_one()) {
                        // 32 bytes of a row per step: 16 values, or 32 of 8 bits
                        constexpr int kSteps = F8 ? D / 32 : D / 16, kPer = C::kRow / 32;
#pragma unroll
                        for (int x = 0; x < (F8 ? 2 : 1) * kSteps; ++x) {
                            const int kk = x % kSteps;  // (the second time: Q's second term)
                            const uint64_t a =
                                desc_at(q_low, 16, x / kSteps * (kRows * D) +
                                                       kk / kPer * (kRows * C::kRow) + kk % kPer * 32,
                                        C::kRow);
                            const uint64_t b = desc_at(
                                low, 16, kk / kPer * (TK * C::kRow) + kk % kPer * 32, C::kRow);
                            if (F8) mma_ss_8(d, a, b, id_s, x > 0);
                            else mma_ss(d, a, b, id_s, x > 0);
                        }
                        mma_commit(&s_full[g & 1]);
                        mma_commit(&empty[slot]);
                        if (j + 1 == cnt) mma_commit(&sm.q_free);
                    }
                    __syncwarp();
                    keys.step();
                }
            } else {
                for (int j = 0; j < cnt; ++j, ++g) {
                    const int slot = vals.slot;
                    if (!ready(&full[NK + slot], vals.phase)) break;
                    if (!ready(&p_full[g & 1], (g >> 1) & 1)) break;
                    if (j == 0 && item > 0 && !ready(&sm.o_free, (item - 1) & 1)) break;
                    const uint32_t low = uniform((smem_u32(val_ring) + slot * C::kVal) >> 4);
                    const uint32_t a = uniform(tmem + C::kP + (g & 1) * (TK / 2));
                    const uint32_t d = uniform(tmem);
                    tc_after_sync();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < TK / 16; ++kk)
                            mma_ts(d, a + kk * 8, desc_at(low, TK * 128, kk * 2048), id_o,
                                   kk > 0 || j > 0);
                        mma_commit(&empty[NK + slot]);
                        mma_commit(&sm.pv_done[g & 1]);
                        if (j + 1 == cnt) mma_commit(&sm.o_full);
                    }
                    __syncwarp();
                    vals.step();
                }
            }
            ++item;
            left -= cur.lead + cnt;
            cur.next(p);
        }
        __syncwarp();
        if (!ok) {  // let the MMAs that were issued end before tensor memory is freed
            code = 6;
            volatile int none = 0;
            if (elect_one()) mma_commit(&sm.drained[values]);
            mbar_wait(&sm.drained[values], 0, &none, 20000000ll);
        }
    } else if (F8 && warp >= kWidenWarp) {
        // ---- with an e4m3 cache: Q in two e4m3 terms, and V tiles to f16 in the MMA's layout (K goes
        // to the MMA as it lies; for P the two terms would be three conversions per weight).  A piece is
        // 16 codes of a key: two 16-byte units of its row.  Of 8 lanes, four take the four pieces of a panel of an even key and four those
        // of the next panel of the odd key after it, so that neither the loads nor the stores, whose
        // units are turned by the key's number, meet in a bank.
        constexpr int kKeys = kWidenWarps * 8, P = D / 64;  // keys at once; panels of a key
        constexpr int kPieces = TK / kKeys * P, kBatch = kPieces < 4 ? kPieces : 4;
        const int t = tid - kWidenWarp * 32, piece = t & 3, odd_key = (t >> 2) & 1;
        const int key = (t >> 3) * 2 + odd_key;  // and kKeys, 2 kKeys ... further on
        static_assert(kKeys % 8 == 0, "the swizzle of a thread's pieces is one");
        const uint32_t unit0 = ((2 * piece) ^ (key & 7)) << 4, unit1 = unit0 ^ 16;
        Ring<NR> raws(0);
        Ring<NV> values(1);
        int item = 0;  // (at most NV <= 4 ahead of the softmax warps')
        // Q as two e4m3 terms of x = q 2^e, with the row's largest magnitude in [2^7, 2^8): the first
        // is x rounded to its 4 bits, and what that leaves of bf16's 8 bits is at most 8 of its last
        // place, 4 bits again, so the two are exact down to e4m3's smallest step, 2^-9: an error of at
        // most 2^-10, 2^-17 of the row's largest value.  In between x is f16, exact down to 2^-17.  An
        // infinity makes the row NaN, as its scores would.  D / 8 lanes take a row, 16 bytes each; a
        // warp reads kSome such groups of rows at once, since a row alone is a memory latency and
        // a chain of conversions.  (One warp alone took 45 us for 128 rows at D = 256.)
        auto split_q = [&]() {
            constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kSome = 4;
            const int row0 = cur.tile * kRows;
            const int rows = min(kRows, cur.q.n * p.group - row0);
            const int sub = lane / kLanes, c = lane % kLanes;
            const int panel = c * 8 / C::kRowKeys, in_row = c * 8 % C::kRowKeys;
            constexpr int kStep = kWidenWarps * kAtOnce * kSome;
            uint4 ahead[kSome];
            auto read = [&](int r0) {
#pragma unroll
                for (int i = 0; i < kSome; ++i) {
                    const int r = min(r0 + i * kAtOnce + sub, rows - 1);
                    ahead[i] =
                        __ldg(reinterpret_cast<const uint4*>(q_row(p, cur, row0 + r) + c * 8));
                }
            };
            int r0 = (warp - kWidenWarp) * kAtOnce * kSome;
            read(r0);
#pragma unroll 1
            for (; r0 < rows; r0 += kStep) {
                uint4 v[kSome];
#pragma unroll
                for (int i = 0; i < kSome; ++i) v[i] = ahead[i];
                read(r0 + kStep);
#pragma unroll
                for (int i = 0; i < kSome; ++i) {
                    const int r = r0 + i * kAtOnce + sub;
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint32_t two = 0;  // largest magnitudes' bits; NaN and infinity lead
#pragma unroll
                    for (int e = 0; e < 4; ++e) two = __vmaxu2(two, w[e] & 0x7fff7fffu);
#pragma unroll
                    for (int d = kLanes / 2; d; d >>= 1)
                        two = __vmaxu2(two, __shfl_xor_sync(~0u, two, d));
                    const uint32_t big = max(two & 0xffffu, two >> 16);
                    // up: the biased exponent of 2^e.  At most 2^64: a row whose largest value is
                    // below 2^-57 has scores of zero to fp32 either way.
                    const int up = min(127 + 7 + 127 - (int)(big >> 7), 127 + 64);
                    const float mul = __uint_as_float((uint32_t)up << 23);
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x = pack16(true, __uint_as_float(w[e] << 16) * mul,
                                                  __uint_as_float(w[e] & 0xffff0000u) * mul);
                        const uint32_t h = e4m3_pair(x), f = e4m3_values(h);
                        uint32_t rest;
                        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(x), "r"(f));
                        const uint32_t l = e4m3_pair(rest);
                        hi[e >> 1] = e & 1 ? hi[e >> 1] | h << 16 : h;
                        lo[e >> 1] = e & 1 ? lo[e >> 1] | l << 16 : l;
                    }
                    if (big >= 0x7f80u) lo[0] = lo[1] = 0x7f7f7f7fu;
                    if (r < rows) {
                        if (c == 0) sm.q_scale[item & 3][r] = (uint8_t)(254 - up);
                        // 16-byte units turned by the row, as TMA turns K's
                        const int turn = C::kRow == 128 ? r & 7 : (r >> 1) & 3;
                        uint8_t* const to = q_tile + panel * (kRows * C::kRow) + r * C::kRow +
                                            (((in_row >> 4) ^ turn) << 4) + (in_row & 8);
                        *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
                        *reinterpret_cast<uint2*>(to + kRows * D) = make_uint2(lo[0], lo[1]);
                    }
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_full);
        };
        while (left > 0 && ok) {
            const int cnt = uniform(cur.take(left));
            if (cnt <= 0) break;
            if (item > 0) ok = __all_sync(~0u, mbar_wait(&sm.q_free, (item - 1) & 1, stop_v));
            if (!ok) break;
            split_q();
            const int end = key_end(p, cur.q, cur.tile), open = key_open(p, cur.q, cur.tile);
            for (int i = 0; i < cnt; ++i) {
                const int rs = raws.slot, ts = values.slot;
                ok = __all_sync(~0u, mbar_wait(&sm.raw_full[rs], raws.phase, stop_v) &&
                                         mbar_wait(&empty[NK + ts], values.phase, stop_v));
                if (!ok) break;  // (all lanes or none: what follows is for whole warps)
                const uint8_t* const src = raw + rs * C::kRaw + key * D + piece * 16;
                uint8_t* const dst = val_ring + ts * C::kVal + key * 128;
                // piece x of this thread: its key, and its panel
                auto key_of = [&](int x) { return x / P * kKeys; };
                auto panel_of = [&](int x) { return (x + odd_key) % P; };
                uint32_t most = 0;  // largest magnitudes, in two halves
#pragma unroll 1
                for (int x0 = 0; x0 < kPieces; x0 += kBatch) {
                    uint4 w[kBatch];
#pragma unroll
                    for (int y = 0; y < kBatch; ++y)
                        w[y] = *reinterpret_cast<const uint4*>(src + key_of(x0 + y) * D +
                                                               panel_of(x0 + y) * 64);
#pragma unroll
                    for (int y = 0; y < kBatch; ++y) {
                        const uint32_t in[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
                        uint32_t out[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            widen(in[j], out[2 * j], out[2 * j + 1]);
                            most = larger(larger(most, out[2 * j]), out[2 * j + 1]);
                        }
                        uint8_t* const to =
                            dst + key_of(x0 + y) * 128 + panel_of(x0 + y) * (TK * 128);
                        *reinterpret_cast<uint4*>(to + unit0) =
                            make_uint4(out[0], out[1], out[2], out[3]);
                        *reinterpret_cast<uint4*>(to + unit1) =
                            make_uint4(out[4], out[5], out[6], out[7]);
                    }
                }
                // What is rare is done over: NaN codes, which only cvt knows and which are zeros here
                // if not all rows see the key, and values past the end, which are zeros.
                const int valid = end - (cur.u + i) * TK;
                if (valid < TK || (most & 0x7fffu) >= kWidenedNan ||
                    (most >> 16 & 0x7fffu) >= kWidenedNan) {
#pragma unroll 1
                    for (int x = 0; x < kPieces; ++x) {
                        const uint32_t* const in = reinterpret_cast<const uint32_t*>(
                            src + key_of(x) * D + panel_of(x) * 64);
                        uint8_t* const to = dst + key_of(x) * 128 + panel_of(x) * (TK * 128);
#pragma unroll 1
                        for (int j = 0; j < 4; ++j) {
                            uint32_t even = 0, odd = 0;
                            if (key + key_of(x) < valid) {
                                uint32_t codes = in[j];
                                if ((cur.u + i) * TK + key + key_of(x) >= open) {
                                    const uint32_t nan =
                                        ((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                                    codes &= ~((nan >> 7) * 0xffu);
                                    if (nan) sm.partly[item & 7] = item + 1;
                                }
                                widen_nan(codes, even, odd);
                            }
                            *reinterpret_cast<uint2*>(to + (j < 2 ? unit0 : unit1) + (j & 1) * 8) =
                                make_uint2(even, odd);
                        }
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&full[NK + ts]);
                    mbar_arrive(&sm.raw_empty[rs]);
                }
                raws.step();
                values.step();
            }
            ++item;
            left -= cur.lead + cnt;
            cur.next(p);
        }
        if (!ok) code = 8;
    } else if (warp < kSoftmaxWarps) {
        // ---- softmax: thread = row = tensor memory lane.  Two warpgroups take the units by turns, so
        // that one waits for scores and finds their maximum while the other forms weights; the
        // reference maximum is handed from unit to unit, and each keeps a sum of its own.
        // The warps meet at barriers, so they must all take the same way: one thread reads what
        // comes next for all of them, and after a wait that gave up they go on (without waiting,
        // on whatever is there) to the end of the range.
        const int wg = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        int g = 0, item = 0;
        auto wait = [&](uint64_t* b, uint32_t parity) {
            if (ok && !mbar_wait(b, parity, stop_v)) ok = false;
        };
        while (left > 0) {
            const int cnt = cur.take(left);
            if (cnt <= 0) break;
            if (tid == 0) {
                Cursor<TK> after = cur;
                after.next(p);
                *reinterpret_cast<Cursor<TK>*>(sm.start[(item + 1) & 1]) = after;
            }
            const int row0 = cur.tile * kRows;
            const int rows = min(kRows, cur.q.n * p.group - row0);
            const bool busy = quarter * 32 < rows;  // this warp has rows
            const bool mine = row < rows;  // lanes past the rows compute on whatever is there
            const int tok = (int)div_by(row0 + row, p.by_group);
            const int end = key_end(p, cur.q, cur.tile), open = key_open(p, cur.q, cur.tile);
            // the last key this row sees
            const int last = mine ? min(cur.q.pos + tok, end - 1) : INT32_MAX;
            const int32_t* const table = p.table + cur.r * p.ld_table;
            auto page_at = [&](int j) {  // lane i: the page of 16 keys of the unit
                const int key = (cur.u + j) * TK + lane * 16;
                return j >= cnt || lane >= TK / 16 || key >= end ? 0
                                                                     : table[div_by(key, p.by_block)];
            };
            int page = page_at((g ^ wg) & 1);  // of this warpgroup's first unit; read a turn ahead
            float m = -INFINITY, l = 0.f, c = p.c;
            // (a row of zeros, or of 2^-57 and less, at a tiny scale: its factor may fall below fp32's
            // range, and a factor of zero would make a masked score NaN.  Its scores are zero either way.)
            auto row_factor = [&](float unit) { return fmaxf(p.c * unit, 1.1754944e-38f); };
            auto scale_of_q = [&]() {  // (where scores of the row tile have arrived)
                return __uint_as_float((uint32_t)sm.q_scale[item & 3][F8 ? row : 0] << 23);
            };

            // unit j's weights
            auto weigh = [&](int j) {
                constexpr int kChunks = TK / 32;
                const uint32_t from = tmem + lanes + C::kS + wg * TK;
                const uint32_t to = tmem + lanes + C::kP + wg * (TK / 2);
                const uint32_t holes = __ballot_sync(~0u, (unsigned)page >= (unsigned)p.blocks);
                const int see = last - (cur.u + j) * TK;  // keys 0..see of the unit
                const bool masked = holes || __any_sync(~0u, see < TK - 1);
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                for (int i = 0; i < kChunks; ++i) {
                    uint32_t s[32];
                    tmem_ld(from + i * 32, s);
                    tmem_wait_ld(s);
                    if (masked) {  // the second pass reads them masked
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (i * 32 + e > see || ((holes >> (i * 2 + e / 16)) & 1))
                                s[e] = 0xff800000u;  // -inf
                        tmem_st(from + i * 32, s);
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(s[e]));
                }
                if (masked) tmem_wait_st();
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (g > 0) bar_sync(1 + quarter * 2 + (wg ^ 1), 64);
                const float was = j > 0 ? sm.row_max[wg ^ 1][row] : top;
                // the reference rises only when it has to: weights stay below 2^8
                const bool rise = j > 0 && mine && (top - was) * c > 8.f;
                const float now = rise ? top : was;
                sm.row_max[wg][row] = now;
                bar_arrive(1 + quarter * 2 + wg, 64);
                if (l > 0.f) l *= exp2_approx((m - now) * c);
                m = now;
                // the rounding of mc, below, is a factor of all weights of this reference; with large scores
                // it would be many powers of two, and another one for the next reference
                const float far = fabsf(m * c);  // (infinite: no key yet)
                bool large = mine && far > 65536.f && far < INFINITY;
                const bool rare = __any_sync(~0u, rise || large);
                if (rare) {
                    large = __any_sync(~0u, large);
                    if (large) subtract_scores<TK>(from, m == -INFINITY ? 0.f : m);
                }
                if (rare && __any_sync(~0u, rise)) {
                    const float f = rise ? exp2_approx((was - top) * c) : 1.f;
                    wait(&sm.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
                    __syncwarp();
                    tc_after_sync();
#pragma unroll 1
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t o[32];
                        tmem_ld(tmem + lanes + i * 32, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st(tmem + lanes + i * 32, o);
                    }
                }
                const float lift = F8 ? kLift : 0.f;
                const float mc = (m == -INFINITY || large ? 0.f : m * c) - lift;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                // a chunk is read while the one before it is worked on
                uint32_t s[2][32];
                tmem_ld(from, s[0]);
#pragma unroll 1
                for (int i = 0; i < kChunks; i += 2) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        tmem_wait_ld(s[h]);
                        if (h == 0 || i + 2 < kChunks) tmem_ld(from + (i + h + 1) * 32, s[h ^ 1]);
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float a =
                                exp2_approx(fmaf(__uint_as_float(s[h][2 * e]), c, -mc));
                            const float b =
                                exp2_approx(fmaf(__uint_as_float(s[h][2 * e + 1]), c, -mc));
                            sum[(2 * e) & 3] += a;
                            sum[(2 * e + 1) & 3] += b;
                            w[e] = pack16(F8, a, b);
                        }
                        tmem_st(to + (i + h) * 16, w);
                    }
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_wait_st();
            };

            for (int j = 0; j < cnt; ++j, ++g) {
                if ((g & 1) != wg) continue;  // the other warpgroup's
                const int page_next = page_at(j + 2);
                wait(&s_full[wg], (g >> 1) & 1);
                // P's place is free once unit g - 2 is through (and V's of that unit, so that the
                // phase of a V place below is not taken for an earlier one's: NV >= 2)
                if (g >= 2) wait(&sm.pv_done[wg], ((g >> 1) - 1) & 1);
                tc_after_sync();
                const int unit0 = (cur.u + j) * TK;
                if (!F8 && unit0 + TK > min(open, end)) {
                    // Values past the end are whatever the page held: zeros, so that their weights
                    // of zero add nothing.  Those that not all rows see: zeros where not finite.
                    const int slot = g % NV;
                    wait(&full[NK + slot], (g / NV) & 1);
                    const int from = max(min(open, end) - unit0, 0);
                    uint8_t* const v = val_ring + slot * C::kVal;
#pragma unroll 1
                    for (int i = row; i < (TK - from) * (D / 8); i += kRows) {
                        const int key = from + i / (D / 8), x = i % (D / 8);
                        uint4* const at = reinterpret_cast<uint4*>(
                            v + (x >> 3) * (TK * 128) + key * 128 + (x & 7) * 16);
                        uint4 w = make_uint4(0, 0, 0, 0);
                        if (unit0 + key < end) {
                            w = *at;
                            uint32_t* const ww = &w.x;
                            uint32_t any = 0;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {  // an exponent of all ones
                                const uint32_t bad =
                                    ((ww[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
                                any |= bad;
                                ww[e] &= ~((bad >> 15) * 0xffffu);
                            }
                            if (!any) continue;
                            sm.partly[item & 7] = item + 1;
                        }
                        *at = w;
                    }
                    fence_async_smem();
                }
                __syncwarp();
                if (F8 && j < 2 && mine) c = row_factor(scale_of_q());  // this warpgroup's first unit
                if (busy) {
                    weigh(j);
                } else {
                    if (g > 0) bar_sync(1 + quarter * 2 + (wg ^ 1), 64);
                    bar_arrive(1 + quarter * 2 + wg, 64);
                }
                tc_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[wg]);
                page = page_next;
            }
            wait(&sm.o_full, item & 1);
            __syncwarp();
            tc_after_sync();

            // ---- O: divided by the sum and written, or left as a part
            bar_sync(9, kSoftmaxWarps * 32);
            const float unit = F8 && mine ? scale_of_q() : 1.f;
            if (F8) c = row_factor(unit);  // (also if it had no unit)
            const float most = busy ? sm.row_max[(g - 1) & 1][row] : -INFINITY;  // the last unit's
            sm.row_sum[wg][row] = l > 0.f ? l * exp2_approx((m - most) * c) : l;
            bar_sync(9, kSoftmaxWarps * 32);
            const float total = sm.row_sum[0][row] + sm.row_sum[1][row];
            const bool whole = cur.u == 0 && cnt == cur.n;
            const int which = cur.u == 0 ? 1 : 0;  // this CTA's cut at its end, or at its start
            const int64_t part0 = ((int64_t)blockIdx.x * 2 + which) * kRows;
            const float inv = total == 0.f ? 0.f : (F8 ? kWidened : p.v_scale) / total;
            const float v_scale = F8 ? p.v_scale : 1.f;  // (as in join_rows)
            if (!whole && mine && wg == 0)
                p.part_ml[part0 + row] = make_float2(most * unit, total);
            if (busy) {
                uint16_t* const out =
                    p.o + (int64_t)(cur.q.token0 + tok) * p.ldo +
                    (int64_t)(cur.h * p.group + (row0 + row) - tok * p.group) * p.o_head_stride;
#pragma unroll 1
                for (int i = 0; i < D / 64; ++i) {
                    const int col = wg * (D / 2) + i * 32;
                    uint32_t o[32];
                    tmem_ld(tmem + lanes + col, o);
                    tmem_wait_ld(o);
                    if (F8) {  // the values' own order
#pragma unroll
                        for (int e = 1; e < 32; e += 4) {
                            const uint32_t x = o[e];
                            o[e] = o[e + 1];
                            o[e + 1] = x;
                        }
                    }
                    if (mine && whole) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint4 w;
                            uint32_t* const ww = &w.x;
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                ww[x] = pack16(false,
                                               __uint_as_float(o[e * 8 + 2 * x]) * inv * v_scale,
                                               __uint_as_float(o[e * 8 + 2 * x + 1]) * inv *
                                                   v_scale);
                            *reinterpret_cast<uint4*>(out + col + e * 8) = w;
                        }
                    } else if (mine) {
                        uint4* const dst = reinterpret_cast<uint4*>(p.part_o + part0 * D) +
                                           col / 4 * kRows + row;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e * kRows] = make_uint4(
                                o[e * 4], o[e * 4 + 1], o[e * 4 + 2], o[e * 4 + 3]);
                    }
                }
            }
            if (mine && sm.partly[item & 7] == item + 1)
                add_not_finite<F8>(
                    p, table, cur.h, max(open, cur.u * TK), min(last + 1, (cur.u + cnt) * TK),
                    wg * (D / 2), D / 2,
                    p.o + (int64_t)(cur.q.token0 + tok) * p.ldo +
                        (int64_t)(cur.h * p.group + (row0 + row) - tok * p.group) * p.o_head_stride,
                    whole ? nullptr : p.part_o + part0 * D + row * 4);
            tc_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.o_free);
            ++item;
            if (!whole && (cur.u == 0 || p.join_here)) {
                // the CTA with unit x (as the ranges count) of this row tile's 0 .. n - 1 from `zero`
                const int64_t zero = cur.u == 0 ? range.end - cnt : range.begin - cur.u;
                auto cta_of = [&](int64_t x) {
                    const int64_t e = quotient((x + 1) * range.ctas + range.total - 1, range.total) - 1;
                    return (int)min(max(e, (int64_t)0), (int64_t)range.ctas - 1);
                };
                const int owner = cur.u == 0 ? (int)blockIdx.x : cta_of(zero);
                Cut cut;
                memset(&cut, 0, sizeof(cut));
                cut.parts = cta_of(zero + cur.n - 1) - owner + 1;
                cut.token0 = cur.q.token0;
                cut.row0 = row0;
                cut.rows = rows;
                cut.head = cur.h;
                if (!p.join_here) {  // the last row tile goes on in later CTAs
                    if (tid == 0) p.cuts[blockIdx.x] = cut;
                } else {
                    __threadfence();
                    bar_sync(9, kSoftmaxWarps * 32);
                    if (tid == 0)
                        sm.last = atomicAdd(&p.arrived[owner], 1) == cut.parts - 1;
                    bar_sync(9, kSoftmaxWarps * 32);
                    if (sm.last) {
                        __threadfence();
                        join_rows<D, F8>(p, owner, cut, tid, kSoftmaxWarps * 32);
                        if (tid == 0) p.arrived[owner] = 0;
                    }
                }
            }
            left -= cur.lead + cnt;
            cur = *reinterpret_cast<const Cursor<TK>*>(sm.start[item & 1]);
        }
        if (!ok) code = 9;
    }

    if (code) {
        *stop_v = 1;
        if (lane == 0) atomicCAS(p.error, 0, code);
    }
    tc_before_sync();
    __syncthreads();
    if (warp == kScoresWarp) {
        tc_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols));
    }
}

// ---- host --------------------------------------------------------------------------------

struct Layout {
    size_t arrived, cuts, ml, o, total;
};

Layout workspace_layout(int sms, int dim) {
    Layout w;
    w.arrived = 512;
    w.cuts = w.arrived + ((size_t)sms * 4 + 255) / 256 * 256;
    w.ml = w.cuts + (size_t)sms * sizeof(Cut);
    w.ml = (w.ml + 255) / 256 * 256;
    w.o = w.ml + (size_t)sms * 2 * kRows * sizeof(float2);
    w.total = w.o + (size_t)sms * 2 * kRows * dim * 4;
    return w;
}

int gcd(int a, int b) {
    while (b) {
        const int t = a % b;
        a = b;
        b = t;
    }
    return a;
}

template <int D, bool F8>
int launch(Params p, const CUtensorMap& mk, const CUtensorMap& mv, int dev, int grid,
           cudaStream_t stream) {
    using C = Cfg<D, F8>;
    static std::atomic<bool> ready[64];
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(nvfp4_attn_kernel<D, F8>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)C::kSmem) != cudaSuccess) {
            cudaGetLastError();
            return NVFP4_ERR_LAUNCH;
        }
        ready[dev] = true;
    }
    // Times (B200, us) with a cost of 0 / 2 / 4 / 7 / 10 units: 64 decode requests to 2000 keys 65 / 60 / 61
    // / 61 / 64 (D = 256, bf16), 87 / 63 / 62 / 67 / 70 (128, bf16), 88 / 70 / 66 / 71 / 76 (128, e4m3);
    // 3 chunks of up to 1024 tokens over 4000 keys 173 / 156 / 144 / 145 / 146 (128, bf16), 245 / 200 /
    // 166 / 148 / 152 (256, bf16), 263 / 236 / 226 / 212 / 192 (256, e4m3, where Q is split into two
    // terms first); 2048 over 16384, 256: 754 / 761 / 763 / 791 / 769 in bf16, 706 / 775 / 774 / 756 /
    // 780 in e4m3.
    p.tile_cost = F8 && D == 256 ? 7 : 4;
    const int st = nvfp4_host::launch_behind(nvfp4_attn_kernel<D, F8>, grid, C::kThreads, C::kSmem, 0,
                                             stream, p, mk, mv);
    if (st != NVFP4_OK || p.join_here) return st;
    // a thread for 8 columns of a row, by the average request's rows (16 blocks for each CTA, most of
    // which have no cut, are a microsecond of launching)
    const int64_t each = ((int64_t)p.tokens * p.group + p.requests - 1) / p.requests;
    const int rows = each < kRows ? (int)each : kRows;
    return nvfp4_host::launch_behind(
        (nvfp4_attn_join_kernel<D, F8>), dim3((rows * (D / 8) + kJoinThreads - 1) / kJoinThreads, grid),
        kJoinThreads, 0, 0, stream, p);
}

}  // namespace

extern "C" {

int nvfp4_paged_attn_workspace_bytes(int dim, size_t* bytes) {
    if (!bytes) return NVFP4_ERR_NULL;
    if (dim != 64 && dim != 128 && dim != 256) return NVFP4_ERR_SHAPE;
    int dev, sms;
    nvfp4_host::EncodeFn encode;
    const int st = nvfp4_host::device(&dev, &sms, &encode);
    if (st != NVFP4_OK) return st;
    *bytes = workspace_layout(sms, dim).total;
    return NVFP4_OK;
}

int nvfp4_paged_attn(const nvfp4_paged_attn_t* attn, const nvfp4_kv_cache_t* cache,
                     void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!attn) return NVFP4_ERR_NULL;
    int st = nvfp4_host::check_cache(cache);
    if (st != NVFP4_OK) return st;
    const nvfp4_paged_attn_t& a = *attn;
    const nvfp4_kv_cache_t& kv = *cache;
    if (a.heads < 1 || a.heads % kv.heads || a.heads > 16384 || a.tokens < 0 ||
        a.tokens > (1 << 30) / (a.heads / kv.heads) || a.requests < 0 ||
        a.requests > NVFP4_MAX_REQUESTS || a.table_columns < 0 || a.table_columns > INT32_MAX ||
        a.ld_table < a.table_columns || !(a.scale > 0) || isinf(a.scale) || a.ldq < kv.dim ||
        a.q_head_stride < kv.dim || a.ldo < kv.dim || a.o_head_stride < kv.dim)
        return NVFP4_ERR_SHAPE;
    if (a.tokens == 0 || a.requests == 0) return NVFP4_OK;
    if (!a.q || !a.o || !a.starts || !a.lens || (a.table_columns && !a.table))
        return NVFP4_ERR_NULL;
    if (misaligned(a.q, 16) || misaligned(a.o, 16) || misaligned(a.starts, 4) ||
        misaligned(a.lens, 4) || misaligned(a.table, 4) || a.ldq % 8 || a.q_head_stride % 8 ||
        a.ldo % 8 || a.o_head_stride % 8)
        return NVFP4_ERR_ALIGN;
    using nvfp4_host::span;
    const uint64_t ob = 2 * span(1, 0, a.tokens, a.ldo, a.heads, a.o_head_stride, kv.dim);
    const uint64_t cb = kv.blocks ? nvfp4_host::cache_bytes(kv) : 0;
    if (overlaps(a.o, ob, a.q, 2 * span(1, 0, a.tokens, a.ldq, a.heads, a.q_head_stride, kv.dim)) ||
        overlaps(a.o, ob, kv.k, cb) || overlaps(a.o, ob, kv.v, cb) ||
        overlaps(a.o, ob, a.table, 4 * span(1, 0, 1, 0, a.requests, a.ld_table, a.table_columns)) ||
        overlaps(a.o, ob, a.starts, 4ull * a.requests + 4) ||
        overlaps(a.o, ob, a.lens, 4ull * a.requests))
        return NVFP4_ERR_ALIAS;
    if (!workspace || misaligned(workspace, 16)) return NVFP4_ERR_WORKSPACE;
    int dev, sms;
    nvfp4_host::EncodeFn encode;
    st = nvfp4_host::device(&dev, &sms, &encode);
    if (st != NVFP4_OK) return st;
    const Layout w = workspace_layout(sms, kv.dim);
    if (workspace_bytes < w.total) return NVFP4_ERR_WORKSPACE;
    if (overlaps(a.o, ob, workspace, w.total)) return NVFP4_ERR_ALIAS;

    const bool f8 = kv.type == NVFP4_KV_E4M3;
    const int tk = kv.dim == 256 ? 64 : 128;
    const int box = gcd(kv.block_size, tk);
    const int size = f8 ? 1 : 2;
    CUtensorMap maps[2];
    memset(maps, 0, sizeof(maps));
    const void* tensors[2] = {kv.k, kv.v};
    for (int i = 0; i < 2; ++i) {
        const cuuint64_t dims[4] = {(cuuint64_t)kv.dim, (cuuint64_t)kv.block_size,
                                    (cuuint64_t)kv.heads, (cuuint64_t)(kv.blocks ? kv.blocks : 1)};
        const cuuint64_t strides[3] = {(cuuint64_t)kv.slot_stride * size,
                                       (cuuint64_t)kv.head_stride * size,
                                       (cuuint64_t)kv.block_stride * size};
        // K, and V in bf16, panel by panel as the MMA reads them; V in e4m3 in whole rows
        const bool panels = !f8 || i == 0;
        const int row = f8 && kv.dim == 64 ? 64 : 128;
        const cuuint32_t boxes[4] = {(cuuint32_t)(panels ? row / size : kv.dim), (cuuint32_t)box, 1,
                                     1};
        const CUtensorMapSwizzle swizzle = !panels      ? CU_TENSOR_MAP_SWIZZLE_NONE
                                           : row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                                        : CU_TENSOR_MAP_SWIZZLE_64B;
        const cuuint32_t one[4] = {1, 1, 1, 1};
        // L2 fetches no more of a line than the head's row has: the next head's is another CTA's, later
        const CUtensorMapL2promotion promotion = kv.dim * size >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                                 : kv.dim * size >= 128
                                                     ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                     : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
        // without pages nothing is read: every box then lies outside, on any valid address
        void* const at = const_cast<void*>(kv.blocks ? tensors[i] : workspace);
        if (encode(&maps[i], f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   4, at, dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   swizzle, promotion,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return NVFP4_ERR_LAUNCH;
    }
    Params p;
    memset(&p, 0, sizeof(p));
    p.q = static_cast<const uint16_t*>(a.q);
    p.ldq = a.ldq;
    p.q_head_stride = a.q_head_stride;
    p.o = static_cast<uint16_t*>(a.o);
    p.ldo = a.ldo;
    p.o_head_stride = a.o_head_stride;
    p.table = a.table;
    p.ld_table = a.ld_table;
    p.starts = a.starts;
    p.lens = a.lens;
    p.requests = a.requests;
    p.tokens = (int)a.tokens;
    p.kv_heads = kv.heads;
    p.group = a.heads / kv.heads;
    p.block = kv.block_size;
    p.by_group = divisor_of(p.group);
    p.by_block = divisor_of(p.block);
    p.blocks = (int)kv.blocks;
    p.outside = kv.blocks ? (int)kv.blocks : 1;
    p.box = box;
    p.v = kv.v;
    p.block_stride = kv.block_stride;
    p.slot_stride = kv.slot_stride;
    p.head_stride = kv.head_stride;
    const int64_t cap = a.table_columns * kv.block_size;  // (below 2^51)
    p.capacity = (int)(cap > INT32_MAX - 8192 ? INT32_MAX - 8192 : cap);
    p.c = a.scale * (f8 ? kv.k_scale : 1.f) * 1.4426950408889634f;
    p.v_scale = f8 ? kv.v_scale : 1.f;
    // a factor that left fp32's normal range would turn a masked score of -infinity into NaN
    if (!(p.c >= 1.1754944e-38f) || isinf(p.c)) return NVFP4_ERR_SHAPE;
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    p.error = reinterpret_cast<int32_t*>(ws);
    p.arrived = reinterpret_cast<int32_t*>(ws + w.arrived);
    // few rows at all: joining takes a CTA a microsecond or two, less than another launch does (with
    // 8 x 6 rows in 37 parts it would be 12)
    p.join_here = a.tokens * p.group <= 16;
    p.cuts = reinterpret_cast<Cut*>(ws + w.cuts);
    p.part_ml = reinterpret_cast<float2*>(ws + w.ml);
    p.part_o = reinterpret_cast<float*>(ws + w.o);
    switch (kv.dim) {
        case 64:
            return f8 ? launch<64, true>(p, maps[0], maps[1], dev, sms, stream)
                      : launch<64, false>(p, maps[0], maps[1], dev, sms, stream);
        case 128:
            return f8 ? launch<128, true>(p, maps[0], maps[1], dev, sms, stream)
                      : launch<128, false>(p, maps[0], maps[1], dev, sms, stream);
        default:
            return f8 ? launch<256, true>(p, maps[0], maps[1], dev, sms, stream)
                      : launch<256, false>(p, maps[0], maps[1], dev, sms, stream);
    }
}

}  // extern "C"

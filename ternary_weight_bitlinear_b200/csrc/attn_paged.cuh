// attn_paged.cuh -- attention of the new rows of a batch over the paged
// key/value cache (kvcache.cuh has the batch's description).
//
//   out[r, h] = sum_j p_j v_j,  p = softmax_j(scale q[r, h] . k_j),
// j over the positions of r's sequence (up to r's own when causal), key/value
// head h / (H / H_kv).  A row that sees no position gets zeros.
//
// One kernel for every mixture of decode rows, drafted tokens, chunks and
// prompts, on the tensor cores:
//  * Tiles.  A sub-tile is 128 rows of one sequence and key/value head: 128 /
//    group tokens times the group's heads, so keys and values are read once
//    for the group.  Per step of 64 positions S = Q K^T and O += P V are
//    tcgen05.mma (M = 128) with S, P (bf16, over S's columns) and O in tensor
//    memory; a softmax thread owns a row: no shuffles.
//  * Work.  An item is two sub-tiles (or a sequence's last, single one) of one
//    key/value head.  The items' tiles are laid end to end over sequences,
//    heads and sub-tiles, and every CTA (one per SM) takes an equal share of
//    them, found from the lengths on the device: no length is known on the
//    host, a captured call replays with other lengths, and one long sequence
//    spreads over the GPU as well as many short ones.  An item cut by shares
//    leaves (max, sum, vector) partials, merged by attn_merge_kernel in the
//    order of the CTAs: results do not depend on timing.
//  * Two softmax warpgroups, each working in steps of 64 positions with two
//    score buffers: while it works on one step, the scores of its next are
//    made and the probabilities of its last are multiplied with the values, so
//    neither the group nor the tensor core waits for the other.  (A product of
//    eight dependent instructions takes 790 cycles alone, 512 with another's
//    between them.)  In a pair item each group has one sub-tile; in a single
//    item each takes one half of every tile for the same rows, merged at the
//    end.
//  * Loads.  Pages arrive by TMA (a box per page part, no multicast) into a
//    ring that holds K and V tiles in turn, running ahead across items.  int8
//    pages land in a raw ring; a converter warpgroup writes their codes, exact
//    in bf16, in the operand layout; the steps multiply scores (K) and
//    probabilities (V) in binary32.
//  * Rows behind an item's last position are no part of the values' product:
//    its K extent ends at the last 16 positions, where the rows left are zeroed.
//  * Probability zero times an infinity or NaN in a hidden position is NaN.
//    Where a row comes out non-finite that such a position may have made so,
//    the CTA goes over its items a second time: in the steps that only some of
//    a sub-tile's rows see (its own last tokens) the hidden values are looked
//    through, and a run of 16 positions with an infinity or NaN among them is
//    left out of the product and added by the softmax threads, each row over
//    what it sees.  (Looking in the first pass costs a prompt of 2000
//    tokens without any 2 %, with as many key/value heads as query heads 5 %.
//    A prompt of 2048 with a NaN in every page takes 159 us instead of 52.)
// The running maximum moves only when a tile's exceeds it by 2^8 (the sums
// stay far inside binary32), so O is seldom rescaled.
// No unit is at its rate (prompt of 8192, bf16: XU pipe 44 to 51 % busy, tensor
// pipe 43 %, issue 41 %; six chunks, int8: 31, 32 and 51 %): the time is the two
// groups' dependent chains of tensor-memory loads, exponentials and products,
// under the power limit.  Measured, 20/5 heads of 128: a prompt of 8192 tokens,
// bf16, 372 to 391 us, 924 to 879 TFLOP/s of what the rows see (0.56 to 0.53 of
// the measured matrix rate); six chunks of up to 600 over 6800 positions on
// average, int8, 272 us, 645 TFLOP/s.  Five documents of up to 1777, 16/2 heads, not
// causal: 102 us, 637 TFLOP/s.  Tried without gain: a polynomial for some of the
// exponentials, one score buffer with the probabilities beside it, merging in
// this kernel (one SM's latency: prompts of a few hundred tokens 26 -> 66 us).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "attn.cuh"
#include "common.cuh"
#include "gemm_tc.cuh"
#include "kvcache.cuh"
#include "skinny.cuh"

namespace bl {

constexpr int kPaRows = 128;     // rows of a sub-tile (MMA M)
constexpr int kPaTile = 128;     // positions of a tile (a ring place)
constexpr int kPaStep = 64;      // positions of a softmax step
constexpr int kPaItemUnits = 1;  // cost of an item beside its tiles, in tiles of one sub-tile
constexpr int kNoMask = 1 << 30;
constexpr float kPaMaxGrowth = 8.0f;  // log2 growth of the maximum that a row's sums absorb

// Two codes (the low bytes of t's halves; the high ones may be anything) as
// bf16: a code in two's complement is m - 128 s (m: low 7 bits, s: sign), and
// (128 + m) - (128 + 128 s) has exact terms and an exact difference.  The masks
// come as kernel arguments: a logic instruction takes one constant, so (t & m) | c
// with both written out is two instructions.
struct PaCodes {
    uint32_t m, s, c;  // 0x007F007F, 0x00800080, 0x43004300 (128 twice)
    __device__ __forceinline__ uint32_t two(uint32_t t) const {
        const uint32_t x = (t & m) | c, y = (t & s) | c;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
        return *reinterpret_cast<const uint32_t*>(&d);
    }
};

struct PagedAttnArgs {
    KvCacheArgs c;
    KvBatchArgs b;
    const uint16_t* q;   // bf16 [T, heads, D], rows q_stride apart
    uint16_t* out;       // bf16 [T, heads, D], rows o_stride apart
    int64_t q_stride, o_stride;
    int group;           // query heads of a key/value head
    FastDiv by_group;
    int tokens;          // tokens of a sub-tile: 128 / group
    int causal;
    int box;             // positions of a page box: the largest power of two up to 128 dividing page_size
    float qscale;        // scale * log2(e)
    PaCodes codes;
    // workspace
    float* part;         // [grid, 2, part_rows, D] unnormalised vectors
    float* part_ml;      // [grid, 2, part_rows, 2] maximum (log2 domain) and sum
    int4* desc;          // [grid, 2] what the CTA left (PaDesc)
    int part_rows;
};

// What a CTA left in the workspace.  Word 0 of desc[2 c]: the state of its
// first share -- 0 nothing, 1 a continuing part of an item, 2 the end of one;
// desc[2 c + 1]: an item that begins in this CTA and does not end there
// (x: tokens, 0 for none; y: first row; z: key/value head; w: positions that
// its first token sees, below zero where it has no place).

// ---- items ------------------------------------------------------------------
// An item and this CTA's part of it, as the scheduler warp leaves it in shared
// memory for the other roles.  (64 bytes in aligned words: as 14 loose words the
// items cost chunks over an int8 cache 4%, 270 -> 282 us.)
struct alignas(16) PaItem {
    int b, g;        // sequence, key/value head; b < 0: no more items
    int row;         // first token's row in the batch
    int tokens;      // tokens of the item
    int nsub;        // sub-tiles: 1 or 2
    int nt;          // position tiles of the item
    int t0, t1;      // those of this CTA
    int end0;        // positions that some row of the first sub-tile sees
    int end;         // positions that some row of the item sees
    int vend;        // positions that its first token sees; below zero where it has no place
    int len;         // positions of the sequence
    int slot;        // running number of its first Q tile; a pair whose first sub-tile has no tile here loads the
    int nq;          // second only (nq of them, 0 without tiles)
};
constexpr int kPaItems = 4;      // ring of items

__device__ __forceinline__ int pa_tiles(int end) { return (end + kPaTile - 1) / kPaTile; }

// Positions that a row with `tok_end` tokens of its sequence up to and with itself sees.
__device__ __forceinline__ int pa_end(const PagedAttnArgs& a, const KvSeq& s, int tok_end) {
    return a.causal ? min(max(s.len - s.n + tok_end, 0), s.len) : s.len;
}
__device__ __forceinline__ int pa_items(const PagedAttnArgs& a, int n) {
    const int subs = (n + a.tokens - 1) / a.tokens;
    return (subs + 1) / 2;
}
// Positions that the first token of an item's sub-tile sees.
__device__ __forceinline__ int pa_first(const PagedAttnArgs& a, const PaItem& it, int sub) {
    return a.causal ? min(max(it.vend + sub * a.tokens, 0), it.len) : it.len;
}
// The positions of step u that a sub-tile's product with the values takes while
// some of its rows do not see them: from the first that its first token does not
// see to the end of the last run of 16, or the item's last position.
struct PaSpan {
    int from, to;  // in the step
    __device__ __forceinline__ bool some() const { return from < to; }
};
__device__ __forceinline__ PaSpan pa_hidden(int first, int own_end, int item_end, int u) {
    const int at = u * kPaStep;
    return {max(first - at, 0), min((min(kPaStep, own_end - at) + 15) & ~15, item_end - at)};
}
// Cost of item i of a sequence, and its shape.
__device__ __forceinline__ int pa_cost(const PagedAttnArgs& a, const KvSeq& s, int i, int* nsub, int* nt) {
    const int first = 2 * i * a.tokens;
    *nsub = s.n > first + a.tokens ? 2 : 1;
    *nt = pa_tiles(pa_end(a, s, min(first + *nsub * a.tokens, s.n)));
    return kPaItemUnits + *nsub * *nt;
}

// Walks the items of this CTA's share in unit order (the scheduler warp).
struct PaWalk {
    const PagedAttnArgs& a;
    int64_t u0, u1;      // this CTA's units
    int64_t at;          // first unit of the current item
    int b, g, i;         // current item: sequence, head, index within (sequence, head)
    KvSeq s;
    int items;           // items per head of the sequence
    int slot = 0;        // Q tiles so far

    __device__ __forceinline__ PaWalk(const PagedAttnArgs& args, const int64_t* plan, const KvSeq* seq) : a(args) {
        u0 = plan[0];
        u1 = plan[1];
        at = plan[2];
        b = (int)plan[3];
        g = (int)plan[4];
        i = (int)plan[5];
        s = *seq;
        items = pa_items(a, s.n);
    }
    __device__ __forceinline__ void load() {
        s = kv_seq(a.b, b);
        items = pa_items(a, s.n);
    }
    __device__ __forceinline__ bool next(PaItem& it) {
        while (at < u1) {
            int nsub, nt;
            const int c = pa_cost(a, s, i, &nsub, &nt);
            const int64_t from = u0 - at, to = u1 - at;
            const int lo = from > kPaItemUnits ? (int)((from - kPaItemUnits + nsub - 1) / nsub) : 0;
            const int hi = to >= c ? nt : to > kPaItemUnits ? (int)((to - kPaItemUnits + nsub - 1) / nsub) : 0;
            const int first = 2 * i * a.tokens;
            it.b = b;
            it.g = g;
            it.row = s.q0 + first;
            it.tokens = min(nsub * a.tokens, s.n - first);
            it.nsub = nsub;
            it.nt = nt;
            it.t0 = lo;
            it.t1 = hi;
            it.end0 = pa_end(a, s, min(first + a.tokens, s.n));
            it.end = pa_end(a, s, first + it.tokens);
            it.vend = a.causal ? s.len - s.n + first + 1 : s.len;
            it.len = s.len;
            it.nq = lo == hi ? 0 : nsub == 2 && it.end0 > lo * kPaTile ? 2 : 1;
            it.slot = slot;
            slot += it.nq;
            const bool mine = lo < hi || (nt == 0 && from <= 0);
            at += c;
            // (the next item is looked up when there is one in the share: a padded batch may end in many empty sequences)
            if (at < u1 && ++i == items) {
                i = 0;
                if (++g == a.c.kv_heads) {
                    g = 0;
                    ++b;  // (a share that goes on has a sequence with rows left)
                    if (b < a.b.batch) load();
                    if (b < a.b.batch && s.n <= 0 && (b = kv_next(a.b, b)) < a.b.batch) load();
                    if (b >= a.b.batch) at = u1;
                }
            }
            if (mine) return true;
        }
        return false;
    }
};

// How the items of a sequence are cut and what they cost (attn_rows.cuh has another way).
struct PaCut {
    static __device__ __forceinline__ int items(const PagedAttnArgs& a, int n) { return pa_items(a, n); }
    static __device__ __forceinline__ int cost(const PagedAttnArgs& a, const KvSeq& s, int i) {
        int nsub, nt;
        return pa_cost(a, s, i, &nsub, &nt);
    }
};

// Units of one head of a sequence.
template <class Cut>
__device__ __forceinline__ int64_t pa_seq_units(const PagedAttnArgs& a, const KvSeq& s) {
    const int items = Cut::items(a, s.n);
    int64_t u = 0;
    for (int i = 0; i < items; ++i) u += Cut::cost(a, s, i);
    return u;
}

// Inclusive scan over the CTA (blockDim.x threads, a multiple of 32).
__device__ __forceinline__ int64_t pa_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
        if (w == warp) before = all;
        all += warp_sums[w];
    }
    __syncthreads();
    *total = all;
    return v + before;
}

// This CTA's share of `total` units.
__device__ __forceinline__ void pa_share(int64_t total, int64_t* u0, int64_t* u1) {
    if (total < (1 << 22)) {  // 32-bit division (the grid has at most a few hundred CTAs)
        *u0 = (uint32_t)total * blockIdx.x / gridDim.x;
        *u1 = (uint32_t)total * (blockIdx.x + 1) / gridDim.x;
    } else {
        *u0 = total * blockIdx.x / gridDim.x;
        *u1 = total * (blockIdx.x + 1) / gridDim.x;
    }
}

// This CTA's share of all units, and the item that its first unit lies in:
// plan = {u0, u1, first unit of that item, sequence, head, item, all units},
// seq = that sequence.  Every thread of the CTA calls it; warp_sums has 16 words.
template <class Cut>
__device__ __forceinline__ void pa_plan(const PagedAttnArgs& a, int64_t* plan, KvSeq* seq, int64_t* warp_sums) {
    int64_t total = 0, mine = 0, upto = 0, per = 0;
    KvSeq s = {0, 0, 0};
    auto units = [&](int b) {
        per = 0;
        if (b < a.b.batch) {
            s = kv_seq(a.b, b);
            per = pa_seq_units<Cut>(a, s);
        }
        return per * a.c.kv_heads;
    };
    // the thread whose sequence b holds unit u0 leaves the plan
    auto locate = [&](int b, int64_t u0) {
        if (mine > 0 && u0 >= upto - mine && u0 < upto) {
            int64_t at = upto - mine;
            const int g = total < (1 << 22) ? (int)((uint32_t)(u0 - at) / (uint32_t)per) : (int)((u0 - at) / per);
            at += g * per;
            int i = 0;
            for (;;) {
                const int c = Cut::cost(a, s, i);
                if (u0 < at + c) break;
                at += c;
                ++i;
            }
            plan[2] = at;
            plan[3] = b;
            plan[4] = g;
            plan[5] = i;
            *seq = s;
        }
    };
    int64_t u0, u1;
    const auto leave = [&]() {
        if (threadIdx.x == 0) {
            plan[0] = u0;
            plan[1] = u1;
            plan[6] = total;
            if (u0 >= u1) plan[2] = u1;  // nothing
        }
    };
    if (a.b.batch <= 32) {  // one warp's work: the others need not be waited for in between
        if (threadIdx.x < 32) {
            const int lane = threadIdx.x;
            mine = upto = units(lane);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            total = __shfl_sync(0xffffffffu, upto, 31);
            pa_share(total, &u0, &u1);
            leave();
            if (u0 < u1) locate(lane, u0);
        }
        __syncthreads();
        return;
    }
    const int nthr = blockDim.x;
    for (int b0 = 0; b0 < a.b.batch; b0 += nthr) {
        mine = units(b0 + threadIdx.x);
        int64_t sum;
        upto = total + pa_scan(mine, warp_sums, &sum);
        total += sum;
    }
    pa_share(total, &u0, &u1);
    leave();
    if (u0 < u1) {
        int64_t sum = 0;
        for (int b0 = 0; b0 < a.b.batch; b0 += nthr) {
            if (a.b.batch > nthr) {  // the sequences are passed over again
                mine = units(b0 + threadIdx.x);
                int64_t all;
                upto = sum + pa_scan(mine, warp_sums, &all);
                sum += all;
            }
            locate(b0 + threadIdx.x, u0);
        }
    }
    __syncthreads();
}

template <int D, bool I8>
struct PaCfg {
    static constexpr int kHalves = D / 64;                    // 64-column (128-byte) halves of a bf16 tile
    static constexpr int kHalfBytes = kPaTile * 128;
    static constexpr int kTileBytes = kHalves * kHalfBytes;   // a bf16 tile of K, V or Q
    static constexpr int kStages = I8 ? (D == 128 ? 3 : 4) : (D == 128 ? 5 : 10);  // K and V operand ring
    static constexpr int kRawBytes = kPaTile * D;             // an int8 tile
    static constexpr int kRaw = I8 ? (D == 128 ? 3 : 8) : 0;
    static constexpr int kSteps = I8 ? 4 : 0;                 // ring of the tiles' steps (K and V)
    static constexpr int kThreads = I8 ? 512 : 384;
    // registers a thread: the launch's (65536 / kThreads, in eights), and each role's share of the same total
    static constexpr int kRegs = I8 ? 128 : 168, kRegsSoft = I8 ? 184 : 216, kRegsRest = 72, kRegsConv = 72;
    static_assert(2 * kRegsSoft + kRegsRest + (I8 ? kRegsConv : 0) <= kRegs * (kThreads / 128), "register shares");
    static constexpr int kOffRing = 2 * kTileBytes;           // after two Q slots
    static constexpr int kOffRaw = kOffRing + kStages * kTileBytes;
    static constexpr int kOffStep = kOffRaw + kRaw * kRawBytes;
    static constexpr int kOffMl = kOffStep + kSteps * 2 * kPaTile * 4;  // second group's (max, sum)
    static constexpr int kOffItems = kOffMl + kPaRows * 8;
    static constexpr int kOffBar = kOffItems + kPaItems * (int)sizeof(PaItem);
    // barriers: operand ring full/empty, raw full/empty, steps full/empty, Q full/empty,
    // scores, probabilities, products with the values (a group's two buffers each), merge full/empty, drain, items full/empty
    static constexpr int kBars = 2 * kStages + 2 * kRaw + 2 * kSteps + 4 + 12 + 2 + 2 + 2 * kPaItems;
    static constexpr int kOffPlan = kOffBar + 8 * kBars;
    static constexpr int kSmem = kOffPlan + 256 + 1024;       // plan words, alignment slack
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

// ---- tcgen05 and TMA wrappers -------------------------------------------------
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// bf16 x bf16 -> binary32: A and B from shared memory.
__device__ __forceinline__ void tc_mma_f16_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// A from tensor memory.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptors: binary32 accumulate, bf16 A and B, M = 128; N = 64
// positions with B (keys) K-major, or N = D with B (values) N-major.
constexpr uint32_t kPaIdescQk = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kPaStep >> 3) << 17) |
                                ((uint32_t)(kPaRows >> 4) << 24);
template <int D>
constexpr uint32_t pa_idesc_pv() {
    return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) |
           ((uint32_t)(kPaRows >> 4) << 24);
}
// Values: rows are positions (the contraction), 128-byte-swizzled halves of 64
// columns: 8-row groups 1024 bytes apart (stride offset), halves kHalfBytes
// apart (leading offset).
__device__ __forceinline__ uint64_t pa_desc_v(uint32_t addr, int half_bytes) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(half_bytes >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// A value that every lane of the warp has, in a form that the compiler knows to be one.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// 32 consecutive columns of this thread's lane (no wait).
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
        " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31},"
        " [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}

// One column of this thread's lane.
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
    tmem_ld_wait();
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Eight 16-byte pieces of a lane's row exchanged among eight lanes: afterwards
// x[i] is piece (lane & 7) of the row of lane (lane & ~7) + i, so that storing
// x[i] writes whole 128-byte lines of four rows (a lane storing its own row's
// pieces writes 32 half sectors).
__device__ __forceinline__ void transpose8(uint4 (&x)[8], int lane) {
#pragma unroll
    for (int s = 1; s < 8; s *= 2) {
        const bool up = lane & s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i & s) continue;
            uint4& a = x[i];
            uint4& b = x[i + s];
            const uint4 y = make_uint4(__shfl_xor_sync(0xffffffffu, up ? a.x : b.x, s), __shfl_xor_sync(0xffffffffu, up ? a.y : b.y, s),
                                       __shfl_xor_sync(0xffffffffu, up ? a.z : b.z, s), __shfl_xor_sync(0xffffffffu, up ? a.w : b.w, s));
            if (up) a = y; else b = y;
        }
    }
}

// Registers moved between the warpgroups of a CTA (every warp of a group calls it).
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Two binary32 operations at once.
__device__ __forceinline__ void fma2(float& x, float& y, float bx, float by, float cx, float cy) {
    asm("{\n\t.reg .b64 A, B, C;\n\t"
        "mov.b64 A, {%0, %1};\n\tmov.b64 B, {%2, %3};\n\tmov.b64 C, {%4, %5};\n\t"
        "fma.rn.f32x2 A, A, B, C;\n\tmov.b64 {%0, %1}, A;\n\t}"
        : "+f"(x), "+f"(y) : "f"(bx), "f"(by), "f"(cx), "f"(cy));
}
__device__ __forceinline__ void mul2(float& x, float& y, float bx, float by) {
    asm("{\n\t.reg .b64 A, B;\n\t"
        "mov.b64 A, {%0, %1};\n\tmov.b64 B, {%2, %3};\n\t"
        "mul.rn.f32x2 A, A, B;\n\tmov.b64 {%0, %1}, A;\n\t}"
        : "+f"(x), "+f"(y) : "f"(bx), "f"(by));
}
__device__ __forceinline__ void add2(float& x, float& y, float bx, float by) {
    asm("{\n\t.reg .b64 A, B;\n\t"
        "mov.b64 A, {%0, %1};\n\tmov.b64 B, {%2, %3};\n\t"
        "add.rn.f32x2 A, A, B;\n\tmov.b64 {%0, %1}, A;\n\t}"
        : "+f"(x), "+f"(y) : "f"(bx), "f"(by));
}

// ---- infinities and NaN among hidden values --------------------------------------
// Whether rows [from, to) of a bf16 tile of values hold an infinity or NaN,
// for a whole warp (rows 128 bytes long, their halves HALF bytes apart): such a
// value times zero is NaN, any other is zero.
template <int D, int HALF>
__device__ __forceinline__ bool pa_non_finite(const uint8_t* tile, int from, int to, int lane) {
    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.0f, 0.0f);
    __nv_bfloat162 acc[2] = {zero, zero};
    for (int e = from * 8 + lane; e < to * 8; e += 32)
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            const uint4 v = *reinterpret_cast<const uint4*>(tile + h * HALF + e * 16);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i & 1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), zero, acc[i & 1]);
        }
    const __nv_bfloat162 sum = __hadd2(acc[0], acc[1]);
    return __any_sync(0xffffffffu, (*reinterpret_cast<const uint32_t*>(&sum) & 0x7FFF7FFFu) != 0);
}

// Which of the runs of 16 positions of a step hold one in rows [from, to), a bit each.
template <int D, int HALF>
__device__ __noinline__ uint32_t pa_runs_non_finite(const uint8_t* tile, int from, int to, int lane) {
    uint32_t runs = 0;
    for (int e = from * 8 + lane; e < to * 8; e += 32)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
            if (kv_absmax8(*reinterpret_cast<const uint4*>(tile + h * HALF + e * 16)) >= 0x7F80u) runs |= 1u << (e >> 7);
    return __reduce_or_sync(0xffffffffu, runs);
}

// The products of a step's probabilities p (bf16 pairs, tensor memory) and
// values over those runs, added to this thread's row of the output o (in tensor
// memory too; begun at zero when `fresh`): over the `vis` positions of the step
// that the row sees and no others.  (Seldom needed: some 25 us a run.)
template <int D, int HALF>
__device__ __noinline__ void pa_add_runs(uint32_t o, uint32_t p, const uint8_t* tile, uint32_t runs, int vis, bool fresh) {
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        uint32_t r[32];
        if (fresh) {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0;
        } else {
            tmem_ld32(o + c, r);
        }
#pragma unroll 1
        for (int j = 0; j < kPaStep; ++j) {
            if (!((runs >> (j >> 4)) & 1u)) continue;
            __syncwarp();
            const uint32_t pair = tmem_ld1(p + (j >> 1));
            if (j >= vis) continue;
            const float x = __uint_as_float((j & 1) ? pair & 0xFFFF0000u : pair << 16);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint4 v = *reinterpret_cast<const uint4*>(tile + (c >> 6) * HALF + sw128_offset(j, ((c & 63) >> 3) + y));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t& lo = r[8 * y + 2 * i];
                    uint32_t& hi = r[8 * y + 2 * i + 1];
                    lo = __float_as_uint(fmaf(x, __uint_as_float(w[i] << 16), __uint_as_float(lo)));
                    hi = __float_as_uint(fmaf(x, __uint_as_float(w[i] & 0xFFFF0000u), __uint_as_float(hi)));
                }
            }
        }
        __syncwarp();
        tmem_st32(o + c, r);
    }
    tmem_st_wait();
}

// ---- the kernel -----------------------------------------------------------------
template <int D, bool I8>
__global__ void __launch_bounds__(PaCfg<D, I8>::kThreads, 1) attn_paged_kernel(
    const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ PagedAttnArgs a) {
    using C = PaCfg<D, I8>;
    constexpr int NS = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (base - raw);
    const uint32_t bars = base + C::kOffBar;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (NS + s); };
    auto rfull_bar = [&](int s) { return bars + 8u * (2 * NS + s); };
    auto rempty_bar = [&](int s) { return bars + 8u * (2 * NS + C::kRaw + s); };
    constexpr int kB1 = 2 * NS + 2 * C::kRaw;
    auto sfull_bar = [&](int s) { return bars + 8u * (kB1 + s); };              // steps
    auto sempty_bar = [&](int s) { return bars + 8u * (kB1 + C::kSteps + s); };
    constexpr int kB2 = kB1 + 2 * C::kSteps;
    auto qfull_bar = [&](int s) { return bars + 8u * (kB2 + s); };
    auto qempty_bar = [&](int s) { return bars + 8u * (kB2 + 2 + s); };
    // step j of group w: buffer j & 1, phase j >> 1
    auto score_bar = [&](int w, uint32_t j) { return bars + 8u * (kB2 + 4 + 2 * w + (j & 1)); };
    auto prob_bar = [&](int w, uint32_t j) { return bars + 8u * (kB2 + 8 + 2 * w + (j & 1)); };
    auto pv_bar = [&](int w, uint32_t j) { return bars + 8u * (kB2 + 12 + 2 * w + (j & 1)); };
    const uint32_t mfull_bar = bars + 8u * (kB2 + 16), mempty_bar = bars + 8u * (kB2 + 17);
    auto drain_bar = [&](int w) { return bars + 8u * (kB2 + 18 + w); };
    const uint32_t item_bars = bars + 8u * (kB2 + 20);  // full, then empty
    auto ifull_bar = [&](uint32_t i) { return item_bars + 8u * (i % kPaItems); };
    auto iempty_bar = [&](uint32_t i) { return item_bars + 8u * (kPaItems + i % kPaItems); };
    static_assert(kB2 + 20 + 2 * kPaItems == C::kBars, "barrier count");
    PaItem* ring = reinterpret_cast<PaItem*>(sm + C::kOffItems);
    int64_t* plan = reinterpret_cast<int64_t*>(sm + C::kOffPlan);       // 7 words
    int64_t* warp_sums = plan + 8;                                      // 16 words
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(plan + 24);
    KvSeq* seq = reinterpret_cast<KvSeq*>(plan + 26);
    // runs of 16 positions that a product with the values leaves out: of group w's step in buffer j & 1
    volatile uint32_t* left_out = reinterpret_cast<volatile uint32_t*>(plan + 28);
    unsigned* redo = reinterpret_cast<unsigned*>(plan + 30);            // bit 0: the share is gone over again, bit 1: a wait ran out
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(full_bar(s), I8 ? 4 : 1);  // converter warps, or the loader's expect
            mbar_init(empty_bar(s), 2);          // one by each group
        }
        for (int s = 0; s < C::kRaw; ++s) {
            mbar_init(rfull_bar(s), 1);
            mbar_init(rempty_bar(s), 4);
        }
        for (int s = 0; s < C::kSteps; ++s) {
            mbar_init(sfull_bar(s), 1);
            mbar_init(sempty_bar(s), 8);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(qfull_bar(s), 1);
            mbar_init(qempty_bar(s), 2);
            mbar_init(drain_bar(s), 1);
            for (int j = 0; j < 2; ++j) {
                mbar_init(score_bar(s, j), 1);
                mbar_init(prob_bar(s, j), 4);
                mbar_init(pv_bar(s, j), 1);
            }
        }
        mbar_init(mfull_bar, 4);
        mbar_init(mempty_bar, 4);
        for (int i = 0; i < kPaItems; ++i) {
            mbar_init(ifull_bar(i), 1);
            mbar_init(iempty_bar(i), I8 ? 15 : 11);  // page loader, MMA issuers, softmax (and converter) warps
        }
        *redo = 0;
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc(smem_addr(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
    // columns: scores (and probabilities) of group w's step j at 128 w + 64 (j & 1), its output at 256 + 128 w
    pdl_wait();
    pdl_launch_dependents();
    pa_plan<PaCut>(a, plan, seq, warp_sums);

    bool ok = true;
    uint32_t ii = 0;  // items taken from the ring
    // the next item for a whole warp (nullptr: none left, or a wait ran out), and its release
    auto take = [&]() -> const PaItem* {
        ok = __all_sync(0xffffffffu, mbar_wait(ifull_bar(ii), (ii / kPaItems) & 1u));
        if (!ok) return nullptr;
        const PaItem* it = ring + ii % kPaItems;
        return it->b < 0 ? nullptr : it;
    };
    auto release = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(iempty_bar(ii));
        ++ii;
    };
    // Every role goes over the CTA's items once, and where a row came out non-finite that an infinity or NaN in a hidden
    // position may have made so, once more with a look at those positions (see PaSpan).  Every warp asks once, with
    // nothing of its own under way in tensor memory, so that the CTA may end without another barrier.
    bool careful = false;
    auto again = [&](bool takes) {
        if constexpr (!I8) {  // (codes are finite)
            if (careful) return false;
            if (!ok) atomicOr(redo, 2u);
            tc_fence_before();
            __syncthreads();
            careful = *reinterpret_cast<volatile unsigned*>(redo) == 1u;
            if (careful && takes) release();  // the items' end
        }
        return careful;
    };
    if (warp < 4) {
    setmaxnreg_dec<C::kRegsRest>();
    if (warp == 3) {
        // ---------------- scheduler, and the queries: one slot per sub-tile ----------------
        uint32_t n = 0, flying = 0;
        do {
        if (lane == 0) {
            PaWalk walk(a, plan, seq);
            walk.slot = (int)n;
            PaItem it;
            for (bool more = true; more && ok; ++ii) {
                more = walk.next(it);
                if (!more) {
                    it.b = -1;
                    it.nq = 0;
                }
                ok = mbar_wait(iempty_bar(ii), ((ii / kPaItems) & 1u) ^ 1u);
                if (!ok) break;
                ring[ii % kPaItems] = it;
                mbar_arrive(ifull_bar(ii));
                for (int x = 0; x < it.nq; ++x, ++n) {
                    const int st = (int)(n & 1);
                    ok = mbar_wait(qempty_bar(st), ((n >> 1) & 1u) ^ 1u);
                    if (!ok) break;
                    flying = n >= 2 ? n - 1 : 0;
                    mbar_arrive_expect_tx(qfull_bar(st), (uint32_t)(a.tokens * a.group * D * 2));
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
                        tma_load_4d(base + st * C::kTileBytes + h * C::kHalfBytes, &map_q, h * 64, 0,
                                    it.row + (it.nsub - it.nq + x) * a.tokens, it.g, qfull_bar(st));
                }
            }
            if (!ok)
                for (uint32_t j = flying; j < n; ++j) mbar_wait(qfull_bar((int)(j & 1)), (j >> 1) & 1u);
        }
        } while (again(false));
    } else if (warp == 0) {
        // ---------------- pages: K and V tiles (and steps) ----------------
        constexpr int NR = I8 ? C::kRaw : NS;
        const int box = a.box, chunks = kPaTile / box;  // boxes of a tile: lane c loads box c
        uint32_t n = 0;        // ring places used (K and V in turn)
        uint32_t flying = 0;   // oldest place that may still be landing
        uint32_t tile = 0, tile_flying = 0;
        do {
        while (const PaItem* item = take()) {
            const PaItem it = *item;
            release();
            const int end = it.end;
            auto page_of = [&](int t) {  // this lane's page of tile t, -1 where it has none
                const int p = t * kPaTile + lane * box;
                return lane < chunks && t < it.t1 && p < end ? kv_page(a.c, a.b, it.b, p) : -1;
            };
            int page = page_of(it.t0);
            for (int t = it.t0; t < it.t1; ++t, ++tile) {
                const int page_next = page_of(t + 1);
                const int slot0 = a.c.by_page.mod(t * kPaTile + lane * box);
                const int boxes = __popc(__ballot_sync(0xffffffffu, page >= 0));
                if constexpr (I8) {
                    const int ss = (int)(tile % C::kSteps);
                    ok = __all_sync(0xffffffffu, mbar_wait(sempty_bar(ss), ((tile / C::kSteps) & 1u) ^ 1u));
                    if (!ok) break;
                    tile_flying = tile >= C::kSteps ? tile - C::kSteps + 1 : 0;
                    if (lane == 0) mbar_arrive_expect_tx(sfull_bar(ss), (uint32_t)(boxes * box * 8));
                    __syncwarp();
                    if (page >= 0) {
                        const uint32_t dst = base + C::kOffStep + (uint32_t)(ss * 2 * kPaTile + lane * box) * 4;
                        const int64_t off = ((int64_t)page * a.c.kv_heads + it.g) * a.c.page_size + slot0;
                        bulk_g2s(dst, a.c.k_step + off, (uint32_t)box * 4, sfull_bar(ss));
                        bulk_g2s(dst + kPaTile * 4, a.c.v_step + off, (uint32_t)box * 4, sfull_bar(ss));
                    }
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++n) {
                    const int st = (int)(n % NR);
                    const uint32_t fb = I8 ? rfull_bar(st) : full_bar(st), eb = I8 ? rempty_bar(st) : empty_bar(st);
                    ok = __all_sync(0xffffffffu, mbar_wait(eb, ((n / NR) & 1u) ^ 1u));
                    if (!ok) break;
                    flying = n >= NR ? n - NR + 1 : 0;
                    if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)(boxes * box * D * (I8 ? 1 : 2)));
                    __syncwarp();
                    if (page >= 0) {
                        const CUtensorMap* map = kv ? &map_v : &map_k;
                        if constexpr (I8) {
                            tma_load_4d(base + C::kOffRaw + st * C::kRawBytes + lane * box * D, map, 0, it.g, slot0, page, fb);
                        } else {
#pragma unroll
                            for (int h = 0; h < C::kHalves; ++h)
                                tma_load_4d(base + C::kOffRing + st * C::kTileBytes + h * C::kHalfBytes + lane * box * 128,
                                            map, h * 64, it.g, slot0, page, fb);
                        }
                    }
                    __syncwarp();
                }
                if (!ok) break;
                page = page_next;
            }
            if (!ok) break;
        }
        } while (again(true));
        // after a failed wait, let the copies still in flight land first
        if (!ok && lane == 0) {
            for (uint32_t j = flying; j < n; ++j)
                mbar_wait(I8 ? rfull_bar((int)(j % NR)) : full_bar((int)(j % NR)), (j / NR) & 1u);
            if constexpr (I8)
                for (uint32_t j = tile_flying; j < tile + 1; ++j) mbar_wait(sfull_bar((int)(j % C::kSteps)), (j / C::kSteps) & 1u);
        }
    } else {
        // ---------------- MMA issuers: warp 1 + w for softmax group w ----------------
        // Two steps of a group are in flight: while its softmax works on one, the next one's scores are made in the other
        // buffer, and the last one's probabilities are multiplied with the values.
        // The whole warp runs this, one lane issues: what the instructions take is then uniform, and an instruction's
        // issue is hidden behind the one before it (from a lane's own branch it took up to 195 cycles, against 48 to 64
        // of the tensor core's).
        const int w = warp - 1;
        const uint32_t sc = tmem + 128u * w, oc = tmem + 256u + 128u * w;
        uint32_t n = 0;               // ring fills passed
        uint32_t made = 0, used = 0;  // steps whose scores (whose product with the values) are issued
        uint32_t info0 = 0, info1 = 0;  // of the steps between the two, by parity (see below)
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar, parity));
            return ok;
        };
        // Every group takes every fill of the rings in order, used or not: a phase's parity tells it from the ones
        // beside it alone.
        auto skip = [&]() {
            const int st = (int)(n % NS);
            if (!wait(full_bar(st), (n / NS) & 1u)) return;
            if (elect_one()) mbar_arrive(empty_bar(st));
            __syncwarp();
            ++n;
        };
        auto finish = [&]() {  // O (+)= P V of step `used`
            const uint32_t x = used & 1 ? info1 : info0;
            const int st = (int)(x & 0xFF), half = (int)(x >> 8) & 1, ksteps = (int)(x >> 12) & 7;
            if (!wait(full_bar(st), (x >> 9) & 1u) || !wait(prob_bar(w, used), (used >> 1) & 1u)) return;
            tc_fence_after();
            const uint64_t vd = pa_desc_v(base + C::kOffRing + st * C::kTileBytes + half * (kPaStep * 128), C::kHalfBytes);
            const uint32_t out = !I8 && (x >> 15) ? (uint32_t)uniform((int)left_out[2 * w + (used & 1)]) : 0u;
            const uint32_t p = sc + 64u * (used & 1), add = (x >> 10) & 1u && !out ? 0u : 1u;  // (the group began O where it left some out)
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kPaStep / 16; ++k)  // 16 positions: 8 columns of P, two 8-row groups of V
                    if (k < ksteps && !((out >> k) & 1u)) tc_mma_f16_ts(oc, p + 8u * k, vd + (uint64_t)(k * 2048 >> 4), pa_idesc_pv<D>(), k ? 1u : add);
                tc_commit(pv_bar(w, used));
                if ((x >> 11) & 1u) tc_commit(empty_bar(st));
            }
            __syncwarp();
            ++used;
        };
        do {
        while (ok) {
            if (!wait(ifull_bar(ii), (ii / kPaItems) & 1u)) break;
            const PaItem& it = ring[ii % kPaItems];
            if (uniform(it.b) < 0) break;
            const bool pair = uniform(it.nsub) == 2;
            const int t0 = uniform(it.t0), t1 = uniform(it.t1), nq = uniform(it.nq);
            const int item_end = uniform(it.end), end = pair && w == 0 ? uniform(it.end0) : item_end;
            const uint32_t slot = (uint32_t)uniform(it.slot);
            const int first = I8 ? 0 : uniform(pa_first(a, it, pair ? w : 0));
            release();
            // this group's Q tile (a single item's one is both groups')
            const uint32_t own = slot + (nq == 2 ? w : 0);
            const int from = 2 * t0 + (pair ? 0 : w), to = min(2 * t1, (end + kPaStep - 1) / kPaStep);  // its steps
            for (int x = 0; ok && x < nq; ++x) {
                const uint32_t q = slot + x;
                if (wait(qfull_bar((int)(q & 1)), (q >> 1) & 1u) && (q != own || from >= to) && elect_one())
                    mbar_arrive(qempty_bar((int)(q & 1)));
                __syncwarp();
            }
            const uint64_t qd = smem_desc_sw128(base + (own & 1) * C::kTileBytes);
            for (int t = t0; ok && t < t1; ++t) {
                const int h0 = pair ? 0 : w, h1 = min(pair ? 2 : w + 1, to - 2 * t);  // its halves of the tile
                if (h0 >= h1) {
                    while (ok && used != made) finish();
                    if (ok) skip();
                    if (ok) skip();
                    continue;
                }
                const int st = (int)(n % NS), vst = (int)((n + 1) % NS);
                const uint32_t ph = (n / NS) & 1u, vph = ((n + 1) / NS) & 1u;
                n += 2;
                for (int h = h0; h < h1; ++h) {
                    if (made - used == 2) finish();
                    if (!ok || (h == h0 && !wait(full_bar(st), ph))) break;
                    tc_fence_after();
                    const uint64_t kd = smem_desc_sw128(base + C::kOffRing + st * C::kTileBytes + h * (kPaStep * 128));
                    const uint32_t s64 = sc + 64u * (made & 1);
                    if (elect_one()) {
#pragma unroll
                        for (int c = 0; c < C::kHalves; ++c)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {  // 16 dimensions (32 bytes) an instruction
                                const uint64_t o = (uint64_t)((c * C::kHalfBytes + k * 32) >> 4);
                                tc_mma_f16_ss(s64, qd + o, kd + o, kPaIdescQk, (c | k) != 0);
                            }
                        tc_commit(score_bar(w, made));
                        if (h == h1 - 1) tc_commit(empty_bar(st));
                        if (2 * t + h + (pair ? 1 : 2) >= to) tc_commit(qempty_bar((int)(own & 1)));
                    }
                    __syncwarp();
                    const int valid = min(kPaStep, end - (2 * t + h) * kPaStep);
                    // ring place, half, its phase, first step of the item, last of the tile, products of 16 positions,
                    // whether runs of 16 may be left out
                    const uint32_t x = (uint32_t)vst | (uint32_t)h << 8 | vph << 9 | (2 * t + h == from ? 1u << 10 : 0u) |
                                       (h == h1 - 1 ? 1u << 11 : 0u) | (uint32_t)((valid + 15) / 16) << 12 |
                                       (!I8 && careful && pa_hidden(first, end, item_end, 2 * t + h).some() ? 1u << 15 : 0u);
                    if (made & 1) info1 = x; else info0 = x;
                    ++made;
                }
            }
            // the item's last products with the values: the group's next step may be items away, and need the ring
            // place these hold
            while (ok && used != made) finish();
        }
        // every MMA this warp issued has finished before TMEM is freed (elect.sync names the same lane every time)
        if (elect_one()) {
            tc_commit(drain_bar(w));
            mbar_wait(drain_bar(w), careful ? 1u : 0u);
        }
        __syncwarp();
        } while (again(true));
    }
    } else if (warp >= 12) {
        // ---------------- int8 codes -> bf16 operand tiles ----------------
        if constexpr (I8) {
            setmaxnreg_dec<C::kRegsConv>();
            const int th = threadIdx.x - 384;
            const PaCodes codes = a.codes;
            uint32_t n = 0;
            while (const PaItem* item = take()) {
                const int parts = 2 * (item->t1 - item->t0);  // K and V of each tile
                release();
                for (int x = 0; x < parts; ++x, ++n) {
                    const int rs = (int)(n % C::kRaw), st = (int)(n % NS);
                    const bool got = mbar_wait(rfull_bar(rs), (n / C::kRaw) & 1u) &&
                                     mbar_wait(empty_bar(st), ((n / NS) & 1u) ^ 1u);
                    ok = __all_sync(0xffffffffu, got);
                    if (!ok) break;
                    const uint8_t* src = sm + C::kOffRaw + rs * C::kRawBytes;
                    uint8_t* dst = sm + C::kOffRing + st * C::kTileBytes;
                    constexpr int kRuns = D / 16, kPer = kPaTile * kRuns / 128;  // runs of 16 codes: of a row, of a thread
                    uint4 w[kPer];
#pragma unroll
                    for (int x = 0; x < kPer; ++x)
                        w[x] = *reinterpret_cast<const uint4*>(src + (th + 128 * x) * 16);
#pragma unroll
                    for (int x = 0; x < kPer; ++x) {
                        const int r = (th + 128 * x) / kRuns, ch = (th + 128 * x) % kRuns;
                        const uint32_t ws[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
                        uint32_t o[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                o[2 * i + y] = codes.two(__byte_perm(ws[i], 0, y ? 0x4342 : 0x4140));
                            }
                        uint8_t* half = dst + (ch >> 2) * C::kHalfBytes;
                        *reinterpret_cast<uint4*>(half + sw128_offset(r, (ch & 3) * 2)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(half + sw128_offset(r, (ch & 3) * 2 + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                    fence_proxy_async_smem();  // generic writes -> visible to the tensor core
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(full_bar(st));
                        mbar_arrive(rempty_bar(rs));
                    }
                }
                if (!ok) break;
            }
        }
    } else {
        // ---------------- softmax: a row per thread ----------------
        setmaxnreg_inc<C::kRegsSoft>();
        const int w = (warp - 4) >> 2, quad = warp & 3;
        const int row = quad * 32 + lane;
        const int tok = a.by_group.div(row);
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t ts = tmem + lanes + 128u * w, to_o = tmem + lanes + 256u + 128u * w;
        float2* ml = reinterpret_cast<float2*>(sm + C::kOffMl);
        uint32_t step = 0, merges = 0, tile = 0;  // steps of this group, merges, tiles
        int state = 0;      // of this CTA's first share (see desc)
        int4 began = make_int4(0, 0, 0, 0);
        do {
        while (const PaItem* item = take()) {
            const bool pair = item->nsub == 2;
            const int t0 = item->t0, t1 = item->t1, end = item->end;
            const int sub = pair ? w : 0;  // this group's sub-tile of the item
            const int tokens = min(a.tokens, item->tokens - sub * a.tokens);
            const bool live = tok < tokens;
            const bool warp_live = quad * 32 < tokens * a.group;
            // positions that this row sees (a lane without a row is masked nowhere: its results go nowhere)
            const int vend = !live ? kNoMask : a.causal ? min(max(item->vend + sub * a.tokens + tok, 0), item->len) : item->len;
            const int own = pair && w == 0 ? item->end0 : end;
            const int first = pa_first(a, *item, sub);
            const int to = min(2 * t1, (own + kPaStep - 1) / kPaStep);
            const uint32_t step0 = step;
            float m = -INFINITY, l = 0.0f;
            for (int t = t0; t < t1; ++t, ++tile) {
                const float* ks = nullptr;
                if constexpr (I8) {  // a tile without a step of this group too: the ring's phases go by both
                    const int ss = (int)(tile % C::kSteps);
                    ok = __all_sync(0xffffffffu, mbar_wait(sfull_bar(ss), (tile / C::kSteps) & 1u));
                    if (!ok) break;
                    ks = reinterpret_cast<const float*>(sm + C::kOffStep) + ss * 2 * kPaTile;
                }
                const int h1 = min(pair ? 2 : w + 1, to - 2 * t);
                for (int h = pair ? 0 : w; h < h1; ++h, ++step) {
                    ok = __all_sync(0xffffffffu, mbar_wait(score_bar(w, step), (step >> 1) & 1u));
                    if (!ok) break;
                    tc_fence_after();
                    const int u = 2 * t + h;
                    const int valid = end - u * kPaStep;  // positions of the step that some row of the item sees
                    const uint32_t tb = ts + 64u * (step & 1);
                    if (warp_live) {
                        float s[kPaStep];
                        tmem_ld32_nowait(tb, reinterpret_cast<uint32_t*>(s));
                        tmem_ld32_nowait(tb + 32, reinterpret_cast<uint32_t*>(s) + 32);
                        tmem_ld_wait();
                        if constexpr (I8) {
#pragma unroll
                            for (int e = 0; e < kPaStep; e += 4) {
                                const float4 k4 = *reinterpret_cast<const float4*>(ks + h * kPaStep + e);
                                mul2(s[e], s[e + 1], k4.x, k4.y);
                                mul2(s[e + 2], s[e + 3], k4.z, k4.w);
                            }
                        }
                        const int vis = vend - u * kPaStep;  // columns that this row sees
                        const bool masked = __any_sync(0xffffffffu, vis < kPaStep);
                        if (masked) {
#pragma unroll
                            for (int e = 0; e < kPaStep; ++e)
                                if (e >= vis) s[e] = -INFINITY;
                        }
                        float x0 = s[0], x1 = s[1], x2 = s[2], x3 = s[3];
#pragma unroll
                        for (int e = 4; e < kPaStep - 4; e += 8) {
                            x0 = fmaxf(fmaxf(x0, s[e]), s[e + 1]);
                            x1 = fmaxf(fmaxf(x1, s[e + 2]), s[e + 3]);
                            x2 = fmaxf(fmaxf(x2, s[e + 4]), s[e + 5]);
                            x3 = fmaxf(fmaxf(x3, s[e + 6]), s[e + 7]);
                        }
                        x0 = fmaxf(fmaxf(x0, s[kPaStep - 4]), s[kPaStep - 3]);
                        x1 = fmaxf(fmaxf(x1, s[kPaStep - 2]), s[kPaStep - 1]);
                        const float top = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
                        if (step == step0) {
                            m = top;
                        } else if (__any_sync(0xffffffffu, live && (top - m) * a.qscale > kPaMaxGrowth)) {
                            // the output so far to the new maximum, once the last step's product is in it
                            ok = __all_sync(0xffffffffu, mbar_wait(pv_bar(w, step - 1), ((step - 1) >> 1) & 1u));
                            if (!ok) break;
                            tc_fence_after();
                            const float mn = fmaxf(m, top);
                            const float alpha = m == mn ? 1.0f : ex2((m - mn) * a.qscale);
                            m = mn;
                            l *= alpha;
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t o[32];
                                tmem_ld32(to_o + c, o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st32(to_o + c, o);
                            }
                        }
                        const float off = m == -INFINITY ? 0.0f : -m * a.qscale;
                        float l0 = 0.0f, l1 = 0.0f, l2 = 0.0f, l3 = 0.0f;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float* r = s + 32 * c;
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                fma2(r[e], r[e + 1], a.qscale, a.qscale, off, off);
                                fma2(r[e + 2], r[e + 3], a.qscale, a.qscale, off, off);
#pragma unroll
                                for (int x = 0; x < 4; ++x) r[e + x] = ex2(r[e + x]);
                                add2(l0, l1, r[e], r[e + 1]);
                                add2(l2, l3, r[e + 2], r[e + 3]);
                            }
                            if constexpr (I8) {
                                // (before the rounding to bf16, so that a weight is rounded once: the code beside it is exact.
                                // A probability of one is not exact then: 0.0023 of the outputs' norm is error, 0.0019 with
                                // a bf16 cache)
                                const float* vs = ks + kPaTile + h * kPaStep + 32 * c;
#pragma unroll
                                for (int e = 0; e < 32; e += 4) {
                                    const float4 v4 = *reinterpret_cast<const float4*>(vs + e);
                                    mul2(r[e], r[e + 1], v4.x, v4.y);
                                    mul2(r[e + 2], r[e + 3], v4.z, v4.w);
                                }
                                if (masked) {  // a step behind the last position may be anything
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        if (32 * c + e >= vis) r[e] = 0.0f;
                                }
                            }
                            // the probabilities over columns of scores that have been read
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(r[2 * e], r[2 * e + 1]);
                            tmem_st16(tb + 16u * c, pk);
                        }
                        l += (l0 + l1) + (l2 + l3);
                        tmem_st_wait();
                    }
                    if constexpr (!I8) {
                        // The product takes whole runs of 16 positions.  Probability zero times an infinity or NaN would
                        // not be zero, so values behind the last position that anything sees are zeroed, and runs with
                        // such values where some row does not see them are left to this group's threads.
                        const bool tail = valid < kPaStep && valid % 16 != 0;
                        PaSpan hidden = {0, 0};
                        if (careful) hidden = pa_hidden(first, own, end, u);
                        if (tail || hidden.some()) {
                            const uint32_t n = 2 * tile + 1;
                            const int st = (int)(n % NS);
                            ok = __all_sync(0xffffffffu, mbar_wait(full_bar(st), (n / NS) & 1u));
                            if (!ok) break;
                            uint8_t* vt = sm + C::kOffRing + st * C::kTileBytes + h * kPaStep * 128;
                            if (tail) {
                                const int rows = 16 - valid % 16;
                                for (int e = quad * 32 + lane; e < rows * 8 * C::kHalves; e += 128)
                                    *reinterpret_cast<uint4*>(vt + valid * 128 + e / (rows * 8) * C::kHalfBytes + e % (rows * 8) * 16) = make_uint4(0, 0, 0, 0);
                                fence_proxy_async_smem();
                            }
                            if (hidden.some() && warp_live) {
                                uint32_t runs = 0;
                                if (pa_non_finite<D, C::kHalfBytes>(vt, hidden.from, hidden.to, lane)) {
                                    if (step != step0) {  // the output so far, once the last step's product is in it
                                        ok = __all_sync(0xffffffffu, mbar_wait(pv_bar(w, step - 1), ((step - 1) >> 1) & 1u));
                                        if (!ok) break;
                                        tc_fence_after();
                                    }
                                    runs = pa_runs_non_finite<D, C::kHalfBytes>(vt, hidden.from, hidden.to, lane);
                                    pa_add_runs<D, C::kHalfBytes>(to_o, tb, vt, runs, min(vend, end) - u * kPaStep, step == step0);
                                }
                                if (quad == 0 && lane == 0) left_out[2 * w + (step & 1)] = runs;  // (quad 0 has the first row)
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(prob_bar(w, step));
                }
                if (!ok) break;
                if constexpr (I8) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sempty_bar((int)(tile % C::kSteps)));
                }
            }
            if (!ok) break;
            // ---- the rows' results over [t0, t1) ----
            const bool some = step != step0;
            if (some) {
                ok = __all_sync(0xffffffffu, mbar_wait(pv_bar(w, step - 1), ((step - 1) >> 1) & 1u));
                if (!ok) break;
                tc_fence_after();
            }
            const bool whole = t0 == 0 && t1 == item->nt;
            const bool merge = !pair && t1 > t0 && min(2 * t1, (end + kPaStep - 1) / kPaStep) > 2 * t0 + 1;  // both have steps
            float f0 = 1.0f, f1 = 0.0f;
            if (merge && w == 1) {
                ml[row] = make_float2(m, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(mfull_bar);
            }
            if (merge && w == 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(mfull_bar, merges & 1u));
                if (!ok) break;
                tc_fence_after();
                const float2 other = ml[row];
                const float mn = fmaxf(m, other.x);
                f0 = m == mn ? 1.0f : ex2((m - mn) * a.qscale);
                f1 = other.x == mn ? 1.0f : ex2((other.x - mn) * a.qscale);
                m = mn;
                l = l * f0 + other.y * f1;
            }
            if ((pair || w == 0) && warp_live) {
                const int slot = t0 == 0 ? 1 : 0;
                const int64_t part0 = ((int64_t)blockIdx.x * 2 + slot) * a.part_rows + sub * kPaRows;
                const int64_t prow = part0 + row;
                const float inv = 1.0f / l;
                float poison = 0.0f;
                // 32 columns of this row's output over both groups' parts
                auto columns = [&](int c, uint32_t (&o)[32]) {
                    if (some) {
                        tmem_ld32(to_o + c, o);
                        if (merge) {
                            uint32_t o1[32];
                            tmem_ld32(to_o + 128u + c, o1);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), f1, __uint_as_float(o[e]) * f0));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0;
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) poison = fmaf(__uint_as_float(o[e]), 0.0f, poison);
                };
                const int rows = tokens * a.group, r8 = quad * 32 + (lane & ~7);  // of the sub-tile; the exchange's first row
                // (rolled: code that runs once an item is paid for in instruction fetches)
                if (whole) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 64) {
                        uint4 x[8];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            uint32_t o[32];
                            columns(c + 32 * y, o);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t pk[4];
#pragma unroll
                                for (int z = 0; z < 4; ++z)
                                    pk[z] = vend > 0 ? pack_bf16x2(__uint_as_float(o[8 * e + 2 * z]) * inv,
                                                                   __uint_as_float(o[8 * e + 2 * z + 1]) * inv) : 0u;
                                x[4 * y + e] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                            }
                        }
                        transpose8(x, lane);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = r8 + i, tk = a.by_group.div(r);
                            if (r < rows)
                                *reinterpret_cast<uint4*>(a.out + (int64_t)(item->row + sub * a.tokens + tk) * a.o_stride +
                                                          (int64_t)(item->g * a.group + r - tk * a.group) * D + c + 8 * (lane & 7)) = x[i];
                        }
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        columns(c, o);
                        uint4 x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        transpose8(x, lane);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (r8 + i < rows)
                                *reinterpret_cast<uint4*>(a.part + (part0 + r8 + i) * D + c + 4 * (lane & 7)) = x[i];
                    }
                }
                __syncwarp();
                if (live && !whole)
                    *reinterpret_cast<float2*>(a.part_ml + prow * 2) = make_float2(m == -INFINITY ? m : m * a.qscale, l);
                // an infinity or NaN came out of products that took positions which the row does not see
                if (!I8 && !careful && live && !(poison == 0.0f) && vend < min(min(end, (own + 15) & ~15), t1 * kPaTile)) atomicOr(redo, 1u);
                __syncwarp();
            }
            if (merge) {
                tc_fence_before();
                __syncwarp();
                if (w == 0) {
                    if (lane == 0) mbar_arrive(mempty_bar);
                } else {
                    ok = __all_sync(0xffffffffu, mbar_wait(mempty_bar, merges & 1u));
                }
                ++merges;
            }
            if (!whole) {
                if (t0 == 0)
                    began = make_int4(item->tokens, item->row, item->g, item->vend);
                else
                    state = t1 == item->nt ? 2 : 1;
            }
            if (!ok) break;
            release();
        }
        } while (again(true));
        if (w == 0 && quad == 0 && lane == 0) {
            a.desc[2 * blockIdx.x] = make_int4(state, 0, 0, 0);
            a.desc[2 * blockIdx.x + 1] = began;
        }
    }

    if (I8 || careful) {
        tc_fence_before();
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- merging the parts of items cut by shares ----------------------------------
// CTA (c, y): the item that began in CTA c of the attention kernel and did not
// end there; kPaMergeRows of its rows by each warp.  Its parts lie in CTA c and
// the following ones up to the first that ends it, merged in that order,
//   out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c.
// Bound by the latency of its loads: those of the first two parts (mostly all
// there are) go out together with those that say which CTAs hold one, the
// others' four at a time.
constexpr int kPaMergeThreads = 128;
constexpr int kPaMergeRows = 2;
constexpr int kPaMergeBlock = kPaMergeThreads / 32 * kPaMergeRows;

template <int D>
__global__ void __launch_bounds__(kPaMergeThreads) attn_merge_kernel(const __grid_constant__ PagedAttnArgs a, int grid) {
    constexpr int DL = D / 32, R = kPaMergeRows;
    const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row0 = blockIdx.y * kPaMergeBlock + warp * R;  // this warp's rows of a part
    pdl_wait();
    pdl_launch_dependents();
    float mx[R], den[R], num[R][DL];
    // N parts' loads, then their sums in order; used: bits of those that count
    auto parts = [&](auto n_tag, const int* x, uint32_t& some, auto&& used) {
        constexpr int N = decltype(n_tag)::value;
        float v[N][R][DL];
        float2 ml[N][R];
#pragma unroll
        for (int p = 0; p < N; ++p) {
            const int64_t base = ((int64_t)x[p] * 2 + (x[p] == c ? 1 : 0)) * a.part_rows;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int64_t at = base + min(row0 + i, a.part_rows - 1);
                ml[p][i] = __ldcg(reinterpret_cast<const float2*>(a.part_ml + at * 2));
                const float* src = a.part + at * D + lane * DL;
                if constexpr (DL == 4)
                    *reinterpret_cast<float4*>(v[p][i]) = __ldcg(reinterpret_cast<const float4*>(src));
                else
                    *reinterpret_cast<float2*>(v[p][i]) = __ldcg(reinterpret_cast<const float2*>(src));
            }
        }
        const uint32_t count = used(some);
#pragma unroll
        for (int p = 0; p < N; ++p) {
            if (!((count >> p) & 1u)) continue;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float mn = fmaxf(mx[i], ml[p][i].x);
                const float keep = mx[i] == -INFINITY ? 0.0f : exp2f(mx[i] - mn);
                const float f = ml[p][i].x == -INFINITY ? 0.0f : exp2f(ml[p][i].x - mn);
                den[i] = fmaf(den[i], keep, f * ml[p][i].y);
#pragma unroll
                for (int e = 0; e < DL; ++e) num[i][e] = fmaf(f, v[p][i][e], num[i][e] * keep);
                mx[i] = mn;
            }
        }
    };
#pragma unroll
    for (int i = 0; i < R; ++i) {
        mx[i] = -INFINITY;
        den[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < DL; ++e) num[i][e] = 0.0f;
    }
    const int4 it = __ldcg(a.desc + 2 * c + 1);
    if (it.x == 0 || (row0 >= kPaRows && it.x <= a.tokens)) return;  // no item began here and went on; no second sub-tile
    int state = c + lane >= grid ? 0 : lane == 0 ? 1 : __ldcg(&a.desc[2 * (c + lane)].x);
    // which of CTAs x0 .. x0 + 31 hold a part: up to and with the first that ends the item
    uint32_t ends = 0, some = 0;
    auto holders = [&]() {
        ends = __ballot_sync(0xffffffffu, state == 2);
        const uint32_t have = __ballot_sync(0xffffffffu, state != 0);
        return ends ? have & ((ends & (0u - ends)) * 2 - 1) : have;
    };
    const int near[2] = {c, min(c + 1, grid - 1)};
    parts(std::integral_constant<int, 2>{}, near, some, [&](uint32_t& left) {
        const uint32_t all = holders();
        left = all & ~3u;
        return all & 3u;
    });
    for (int x0 = c;;) {
        while (some) {
            int x[4];
            uint32_t count = 0;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                count |= some ? 1u << p : 0u;
                x[p] = some ? x0 + __ffs(some) - 1 : c;
                some &= some - 1;
            }
            parts(std::integral_constant<int, 4>{}, x, some, [&](uint32_t&) { return count; });
        }
        if (ends || (x0 += 32) >= grid) break;
        state = x0 + lane >= grid ? 0 : __ldcg(&a.desc[2 * (x0 + lane)].x);
        some = holders();
    }
    const int rows0 = min(it.x, a.tokens) * a.group, rows1 = (it.x - min(it.x, a.tokens)) * a.group;  // of its sub-tiles
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int sub = (row0 + i) / kPaRows, rr = (row0 + i) % kPaRows;
        if (rr >= (sub == 0 ? rows0 : rows1)) continue;
        const int in_sub = a.by_group.div(rr), tok = sub * a.tokens + in_sub, hh = rr - in_sub * a.group;
        const int vend = a.causal ? it.w + tok : it.w;
        const float inv = 1.0f / den[i];
        uint16_t* dst = a.out + (int64_t)(it.y + tok) * a.o_stride + (int64_t)(it.z * a.group + hh) * D + lane * DL;
#pragma unroll
        for (int e = 0; e < DL; e += 2)
            *reinterpret_cast<uint32_t*>(dst + e) = vend > 0 ? pack_bf16x2(num[i][e] * inv, num[i][e + 1] * inv) : 0u;
    }
}

}  // namespace bl

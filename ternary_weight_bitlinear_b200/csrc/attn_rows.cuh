// attn_rows.cuh -- attention over the paged cache for batches with few rows a
// sequence and key/value head on average (decode steps, a few drafted tokens):
// the same operation as attn_paged.cuh's, made for streaming the cache.
//
// With at most 16 rows against each position the products are far below what
// the keys and values cost to read, so the kernel is built as a stream: a
// position is read once for the (up to) 16 rows of its head, straight from its
// page, and everything after the load stays in a warp's registers.
//  * A loader warp moves chunks of 32 positions (keys, values, an int8 cache's
//    steps) by TMA into stages; chunk n of the CTA goes to consumer warp
//    n mod W, so a warp's stages are its own ring and no two warps wait for
//    one another between items.
//  * A consumer warp scores its chunk with mma.sync (m16n8k16, bf16: the
//    positions are its 16 rows and the item's rows its 8 columns, where a
//    tcgen05 tile has 64 rows at least and would also pass scores and
//    probabilities through tensor memory), keeps the running maximum, sum and
//    output of its positions, and feeds the probabilities of one product to the
//    next without leaving registers.  int8 codes become bf16 (exactly) in
//    registers, in the order in which shared memory gives them up in whole
//    16-byte words: the positions and dimensions of a product may stand in any
//    order as long as both operands agree.
//  * What a row does not see has no part in it: probability zero times an
//    infinity or NaN would be NaN, so a position that only some of an item's
//    rows see (among its last 15) and that holds one is left out of the
//    product, and added row by row to those that see it.
//  * Items ((sequence, head, 16 rows) times their chunks) are shared out
//    evenly over the CTAs as in attn_paged.cuh.  The warps of a CTA merge
//    through shared memory; of the CTAs that hold parts of one item the last
//    to arrive merges them (in groups where there are many), in the order of
//    the CTAs, so the result does not depend on which it is.  One launch.
// Bound by some 10 us of latency (launch, plan, first loads, merge) and the
// stream behind it; with int8 by the conversions too (ALU pipe 60 % busy): with
// the consumers' arithmetic left out the cases below take 59.5, 31.6 and 9.9 us.
// Ten consumer warps for int8 (144 registers each): 77.8.  Measured, one new row
// a sequence: 64 sequences of 3800 positions on average, 20/5 heads of 128, int8:
// 71 us, 4.55 TB/s of the cache (0.69 of the measured copy rate); two of 107,000
// with one key/value head, bf16: 33 us, 3.3 TB/s; one of 2048, bf16: 10.1 us, of
// which the launch, the plan and the merge are most (its bytes take 0.8).
// The tensor-memory kernel took 292, 69 and 18.8 us for these.
#pragma once

#include "attn_paged.cuh"

namespace bl {

constexpr int kRwRows = 16;       // most rows of an item
constexpr int kRwChunk = 32;      // positions of a chunk
constexpr int kRwItemUnits = 4;   // cost of an item beside its chunks, in chunks
constexpr int kRwItems = 4;       // ring of items
constexpr int kRwGroup = 16;      // parts of an item that one CTA merges at once, where there are more than kRwAlone
constexpr int kRwAlone = 32;
constexpr int kRwCounters = 3;    // counters a CTA

// NR: rows of an item, 8 or 16.
template <int D, bool I8, int NR>
struct RwCfg {
    static constexpr int kWarps = D == 128 && !I8 ? 4 : 8;                    // consumer warps
    static constexpr int kTileBytes = kRwChunk * D * (I8 ? 1 : 2);            // keys (or values) of a chunk
    static constexpr int kStepBytes = I8 ? 2 * kRwChunk * 4 : 0;
    static constexpr int kStageBytes = (2 * kTileBytes + kStepBytes + 1023) / 1024 * 1024;
    static constexpr int kDepth = D == 128 ? (I8 ? 2 : 3) : (I8 ? 4 : 2);     // stages of a warp
    static constexpr int kLoaders = 4;                                        // loader warps: chunk n is loader n mod kLoaders'
    // registers a thread: with eight consumer warps the loaders hand theirs over (a warpgroup each way)
    static constexpr int kRegsLoad = 72, kRegsUse = 216;
    static_assert(kWarps == 4 || kRegsLoad + 2 * kRegsUse <= 3 * 168, "register shares");
    static constexpr int kThreads = 32 * (kWarps + kLoaders);
    // floats of a merged row: four more than D keep its stores free of bank conflicts (16 rows of 128 bf16 have no room)
    static constexpr int kOStride = D == 128 && !I8 && NR == 16 ? D : D + 4;
    static constexpr int kOffO = kWarps * kDepth * kStageBytes;               // [warps][NR][kOStride] outputs
    static constexpr int kOffMl = kOffO + kWarps * NR * kOStride * 4;         // [warps][NR] (maximum, sum)
    static constexpr int kOffItems = kOffMl + kWarps * NR * 8;
    static constexpr int kBars = 2 * kWarps * kDepth + 2 * kRwItems + 4;
    static constexpr int kOffBar = kOffItems + kRwItems * 64;
    static constexpr int kOffPlan = kOffBar + 8 * kBars;
    static constexpr int kSmem = kOffPlan + 256 + 1024;  // plan words (28, of 8 bytes), alignment slack
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
    static_assert((kWarps * kDepth) % kLoaders == 0, "a stage has one loader");
};

// An item and this CTA's part of it.
struct RwItem {
    int b, g;            // sequence, key/value head; b < 0: no more items
    int q0;              // first row of the sequence in the batch
    int row0, rows;      // rows of the item among the sequence's n * group of this head
    int nt, t0, t1;      // its chunks, and this CTA's
    int end;             // positions that some row of the item sees
    int vbase, len;      // position of the sequence's first new token, positions of the sequence
    int cta0, parts;     // first CTA with a part of the item, and how many have one
    int spread;          // total < grid: a chunk a CTA, from unit (unit_hi, unit_lo) on
    int unit_hi, unit_lo;
};
static_assert(sizeof(RwItem) == 64, "item words");

template <int NR>
__device__ __forceinline__ int rw_cost(const PagedAttnArgs& a, const KvSeq& s, int i, int* nt) {
    const int last = min((i + 1) * NR, s.n * a.group) - 1;  // the item's last row
    *nt = (pa_end(a, s, a.by_group.div(last) + 1) + kRwChunk - 1) / kRwChunk;
    return kRwItemUnits + *nt;
}
template <int NR>
__device__ __forceinline__ int rw_items(const PagedAttnArgs& a, int n) {
    return (n * a.group + NR - 1) / NR;
}
template <int NR>
struct RwCut {
    static __device__ __forceinline__ int items(const PagedAttnArgs& a, int n) { return rw_items<NR>(a, n); }
    static __device__ __forceinline__ int cost(const PagedAttnArgs& a, const KvSeq& s, int i) {
        int nt;
        return rw_cost<NR>(a, s, i, &nt);
    }
};
// The CTA whose share [total x / grid, total (x + 1) / grid) holds unit u.
__device__ __forceinline__ int rw_cta_of(int64_t u, int64_t total) {
    if (total < (1 << 22))  // 32-bit division (the grid has at most a few hundred CTAs)
        return (int)((((uint32_t)u + 1) * gridDim.x + (uint32_t)total - 1) / (uint32_t)total) - 1;
    return (int)(((u + 1) * gridDim.x + total - 1) / total) - 1;
}

template <int NR>
struct RwWalk {
    const PagedAttnArgs& a;
    int64_t u0, u1, at, total;
    int b, g, i, items;
    KvSeq s;
    __device__ __forceinline__ RwWalk(const PagedAttnArgs& args, const int64_t* plan, const KvSeq* seq) : a(args) {
        u0 = plan[0];
        u1 = plan[1];
        at = plan[2];
        b = (int)plan[3];
        g = (int)plan[4];
        i = (int)plan[5];
        total = plan[6];
        s = *seq;
        items = rw_items<NR>(a, s.n);
    }
    __device__ __forceinline__ void load() {
        s = kv_seq(a.b, b);
        items = rw_items<NR>(a, s.n);
    }
    __device__ __forceinline__ bool next(RwItem& it) {
        while (at < u1) {
            int nt;
            const int c = rw_cost<NR>(a, s, i, &nt);
            const int64_t from = u0 - at - kRwItemUnits, to = u1 - at - kRwItemUnits;
            const int lo = from > 0 ? (int)from : 0, hi = to >= nt ? nt : to > 0 ? (int)to : 0;
            const bool mine = lo < hi || (nt == 0 && u0 <= at);
            if (mine) {
                it.b = b;
                it.g = g;
                it.q0 = s.q0;
                it.row0 = i * NR;
                it.rows = min(NR, s.n * a.group - it.row0);
                it.nt = nt;
                it.t0 = lo;
                it.t1 = hi;
                it.end = pa_end(a, s, a.by_group.div(it.row0 + it.rows - 1) + 1);
                it.vbase = s.len - s.n;
                it.len = s.len;
                const int64_t first = at + kRwItemUnits;
                it.spread = total < gridDim.x;
                it.cta0 = it.parts = 0;
                if (lo > 0 || hi < nt) {
                    it.cta0 = rw_cta_of(first, total);
                    it.parts = it.spread ? nt : rw_cta_of(at + c - 1, total) - it.cta0 + 1;
                }
                it.unit_hi = (int)(first >> 32);
                it.unit_lo = (int)(first & 0xFFFFFFFF);
            }
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

__device__ __forceinline__ void st_counter(unsigned long long* p, unsigned long long v) {
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
// An arrival: releases what this thread (and those it synchronised with) wrote, acquires what earlier ones released.
__device__ __forceinline__ unsigned long long arrive_counter(unsigned long long* p) {
    unsigned long long v;
    asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], 1;" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long ld_acquire(const unsigned long long* p) {
    unsigned long long v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values transposed across the warp.
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// The position that slot j of a product's eight stands for.  int8 rows of 128
// bytes (in the 128-byte swizzle) are read 16 bytes a lane by slots 2k and
// 2k + 1 together for the keys, and by the even or the odd slots together for
// the values: rows 2k and 2k ^ 5 keep both free of bank conflicts.
template <int D, bool I8>
__device__ __forceinline__ int rw_slot(int j) {
    if constexpr (I8 && D == 128) return (j & 1) ? (j - 1) ^ 5 : j;
    return j;
}
// The dimension that column x of a merged output row stands for, and back
// (int8: a lane reads D/8 neighbouring dimensions, one of each 8-column block).
template <int D, bool I8>
__device__ __forceinline__ int rw_column(int d) {
    if constexpr (I8) return (d % (D / 8)) * 8 + d / (D / 8);
    return d;
}

// Which of positions [from, to) of a chunk (bf16) hold an infinity or NaN among
// their values, a bit each, for a whole warp.
template <int D>
__device__ __forceinline__ uint32_t rw_non_finite(const uint8_t* vtile, int from, int to, int lane) {
    if (from >= to) return 0;
    uint32_t bad = 0;
    for (int e = from * 8 + lane; e < to * 8; e += 32)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
            if (kv_absmax8(*reinterpret_cast<const uint4*>(vtile + h * kRwChunk * 128 + e * 16)) >= 0x7F80u) bad |= 1u << (e >> 3);
    return __reduce_or_sync(0xffffffffu, bad);
}

template <int D, bool I8, int NR>
__global__ void __launch_bounds__(RwCfg<D, I8, NR>::kThreads, 1) attn_rows_kernel(
    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
    const __grid_constant__ PagedAttnArgs a, unsigned long long* counters, unsigned long long epoch) {
    using C = RwCfg<D, I8, NR>;
    constexpr int W = C::kWarps, NST = W * C::kDepth;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (base - raw);
    const uint32_t bars = base + C::kOffBar;
    auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bars + 8u * (NST + s); };
    auto ifull_bar = [&](uint32_t i) { return bars + 8u * (2 * NST + i % kRwItems); };
    auto iempty_bar = [&](uint32_t i) { return bars + 8u * (2 * NST + kRwItems + i % kRwItems); };
    const uint32_t put_bar = bars + 8u * (2 * NST + 2 * kRwItems);      // the warps' results are in shared memory
    const uint32_t got_bar = put_bar + 8u, sent_bar = put_bar + 16u, told_bar = put_bar + 24u;
    RwItem* ring = reinterpret_cast<RwItem*>(sm + C::kOffItems);
    int64_t* plan = reinterpret_cast<int64_t*>(sm + C::kOffPlan);       // 7 words
    int64_t* warp_sums = plan + 8;                                      // 16 words
    KvSeq* seq = reinterpret_cast<KvSeq*>(plan + 26);
    volatile int* last_flag = reinterpret_cast<volatile int*>(plan + 24);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int i = 0; i < kRwItems; ++i) {
            mbar_init(ifull_bar(i), 1);
            mbar_init(iempty_bar(i), W);
        }
        mbar_init(put_bar, W);
        mbar_init(got_bar, W);
        mbar_init(sent_bar, W);
        mbar_init(told_bar, 1);
        mbar_init_fence();
    }
    if (warp == 0 && lane == 0) {
        prefetch_map(&map_k);
        prefetch_map(&map_v);
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    // this CTA's counters (an item that begins here and goes on in others; a group that its parts are first of): this
    // launch's, and nothing counted yet
    if (threadIdx.x < 3) st_counter(threadIdx.x == 0 ? counters + blockIdx.x : counters + gridDim.x + 2 * blockIdx.x + threadIdx.x - 1, epoch);
    pa_plan<RwCut<NR>>(a, plan, seq, warp_sums);

    bool ok = true;
    uint32_t ii = 0;
    auto take = [&]() -> const RwItem* {
        ok = __all_sync(0xffffffffu, mbar_wait(ifull_bar(ii), (ii / kRwItems) & 1u));
        if (!ok) return nullptr;
        const RwItem* it = ring + ii % kRwItems;
        return it->b < 0 ? nullptr : it;
    };
    auto release = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(iempty_bar(ii));
        ++ii;
    };
    if (warp < C::kLoaders) {
        if constexpr (W == 8) setmaxnreg_dec<C::kRegsLoad>();
        // ---------------- the items (loader 0 hands them out), and their chunks ----------------
        const int ld = warp;
        const int box = min(a.box, kRwChunk), boxes = kRwChunk / box;
        uint32_t n0 = 0, loaded = ld;  // chunks passed; this loader's next chunk
        RwWalk<NR> walk(a, plan, seq);
        RwItem it;
        for (bool more = true; more; ++ii) {
            more = walk.next(it);
            if (!more) {
                it.b = -1;
                it.t0 = it.t1 = 0;
            }
            // the page table's next 32 entries, a lane each, and the 32 after them (on their way while the first are used)
            const int32_t* table = a.b.pages + (int64_t)it.b * a.b.max_pages;
            const int pages = more ? a.c.by_page.div(it.end + a.c.page_size - 1) : 0;
            auto entries = [&](int at) { return at + lane < pages ? __ldcg(table + at + lane) : -1; };
            const int skip = (int)((ld + C::kLoaders - n0 % C::kLoaders) % C::kLoaders);
            const uint32_t n = n0;  // the item's first chunk
            int p0 = a.c.by_page.div((it.t0 + skip) * kRwChunk);
            int now = entries(p0), next = entries(p0 + 32);
            if (ld == 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(iempty_bar(ii), ((ii / kRwItems) & 1u) ^ 1u));
                if (!ok) break;
                if (lane == 0) {
                    ring[ii % kRwItems] = it;
                    mbar_arrive(ifull_bar(ii));
                }
                __syncwarp();
            }
            if (!more) break;
            n0 += it.t1 - it.t0;
            for (int t = it.t0 + skip; t < it.t1; t += C::kLoaders) {
                // lane x: box x of the chunk (which spans at most two pages)
                const int p = t * kRwChunk + lane * box;
                const int at = a.c.by_page.div(p);
                const int first = __shfl_sync(0xffffffffu, at, 0);
                if (first + 1 >= p0 + 32) {  // the entries up to this chunk's are done with
                    const int keep = first - p0;
                    if (keep < 32) {
                        const int x = __shfl_sync(0xffffffffu, now, (lane + keep) & 31), y = __shfl_sync(0xffffffffu, next, (lane + keep) & 31);
                        now = lane + keep < 32 ? x : y;
                    } else {
                        now = entries(first);
                    }
                    p0 = first;
                    next = entries(p0 + 32);
                }
                const int entry = __shfl_sync(0xffffffffu, now, (lane < boxes ? at - p0 : 0) & 31);
                const int slot = p - at * a.c.page_size;
                const bool wanted = lane < boxes && p < it.end, here = (unsigned)entry < (unsigned)a.c.num_pages;
                if (wanted && !here) atomicOr(&g_status, kStatusBadPage);
                const int page = wanted && here ? entry : -1;
                const int some = __popc(__ballot_sync(0xffffffffu, page >= 0));
                const uint32_t c = n + (t - it.t0), st = c % NST, fb = full_bar(st);
                ok = __all_sync(0xffffffffu, mbar_wait(empty_bar(st), ((c / NST) & 1u) ^ 1u));
                if (!ok) break;
                loaded = c + C::kLoaders;
                if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)(some * box * (2 * D * (I8 ? 1 : 2) + (I8 ? 8 : 0))));
                __syncwarp();
                if (page >= 0) {
                    const uint32_t kd = base + st * C::kStageBytes, vd = kd + C::kTileBytes;
                    if constexpr (I8) {
                        tma_load_4d(kd + lane * box * D, &map_k, 0, it.g, slot, page, fb);
                        tma_load_4d(vd + lane * box * D, &map_v, 0, it.g, slot, page, fb);
                        const int64_t off = ((int64_t)page * a.c.kv_heads + it.g) * a.c.page_size + slot;
                        const uint32_t sd = vd + C::kTileBytes + lane * box * 4;
                        bulk_g2s(sd, a.c.k_step + off, (uint32_t)box * 4, fb);
                        bulk_g2s(sd + kRwChunk * 4, a.c.v_step + off, (uint32_t)box * 4, fb);
                    } else {
#pragma unroll
                        for (int h = 0; h < D / 64; ++h) {
                            tma_load_4d(kd + h * kRwChunk * 128 + lane * box * 128, &map_k, h * 64, it.g, slot, page, fb);
                            tma_load_4d(vd + h * kRwChunk * 128 + lane * box * 128, &map_v, h * 64, it.g, slot, page, fb);
                        }
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        // after a failed wait, let this loader's copies still in flight land first (a stage has at most one)
        if (!ok && lane == 0)
            for (uint32_t j = 1; j <= NST / C::kLoaders; ++j) {
                const uint32_t c = loaded - j * C::kLoaders;
                if ((int)c >= 0) mbar_wait(full_bar(c % NST), (c / NST) & 1u);
            }
    } else {
        // ---------------- consumers ----------------
        if constexpr (W == 8) setmaxnreg_inc<C::kRegsUse>();
        const int ct = threadIdx.x - 32 * C::kLoaders;  // thread among the consumers
        // The products have the positions (or dimensions) as their 16-row side and the item's rows as columns of eight:
        //   S^T = K Q^T,  O^T = V^T P^T,
        // so eight rows are a whole product.  In a result this lane holds rows 8 x + 2 kq and 8 x + 2 kq + 1 at position
        // (dimension) slots r8 and r8 + 8.
        constexpr int X = NR / 8;
        const PaCodes codes = a.codes;
        const int w = ct >> 5, r8 = lane >> 2, kq = lane & 3;
        float* osm = reinterpret_cast<float*>(sm + C::kOffO);
        float2* ml = reinterpret_cast<float2*>(sm + C::kOffMl);
        int used_ctr = 0;  // counters of this CTA that others arrive at (the last of them resets it)
        uint32_t n0 = 0, merges = 0, sent = 0, told = 0;  // chunks passed; phases of the barriers
        while (const RwItem* item = take()) {
            const int t0 = item->t0, t1 = item->t1, rows = item->rows, end = item->end;
            const int64_t head0 = (int64_t)item->g * a.group;
            // the queries of rows 8 x + r8 as the products' B operand
            uint32_t q[D / 16][X][2];
            int vend[X][2];
#pragma unroll
            for (int x = 0; x < X; ++x) {
                const int row = item->row0 + 8 * x + r8, tok = a.by_group.div(row);
                const bool live = 8 * x + r8 < rows;
                const uint16_t* src = a.q + (int64_t)(item->q0 + tok) * a.q_stride + (head0 + a.by_group.mod(row)) * D;
                if constexpr (I8) {
#pragma unroll
                    for (int blk = 0; blk < D / 64; ++blk)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint4 v = live ? __ldcg(reinterpret_cast<const uint4*>(src + 64 * blk + 16 * kq + 8 * y))
                                                 : make_uint4(0, 0, 0, 0);
                            q[4 * blk + 2 * y][x][0] = v.x;
                            q[4 * blk + 2 * y][x][1] = v.y;
                            q[4 * blk + 2 * y + 1][x][0] = v.z;
                            q[4 * blk + 2 * y + 1][x][1] = v.w;
                        }
                } else {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            q[k][x][y] = live ? __ldcg(reinterpret_cast<const uint32_t*>(src + 16 * k + 8 * y + 2 * kq)) : 0u;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {  // positions that rows 8 x + 2 kq + j see
                    const int r = 8 * x + 2 * kq + j, tk = a.by_group.div(item->row0 + r);
                    vend[x][j] = r >= rows ? 0 : a.causal ? min(max(item->vbase + tk + 1, 0), item->len) : item->len;
                }
            }
            const int vmin = a.causal ? item->vbase + a.by_group.div(item->row0) + 1 : item->len;  // of the item's first row
            float o[D / 16][X][4], m[X][2], l[X][2];
#pragma unroll
            for (int x = 0; x < X; ++x) {
                m[x][0] = m[x][1] = -INFINITY;
                l[x][0] = l[x][1] = 0.0f;
#pragma unroll
                for (int db = 0; db < D / 16; ++db)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[db][x][c] = 0.0f;
            }
            const int skip = (int)((w + W - n0 % W) % W);
            for (int t = t0 + skip; t < t1; t += W) {
                const uint32_t n = n0 + (t - t0), st = n % NST;
                ok = __all_sync(0xffffffffu, mbar_wait(full_bar(st), (n / NST) & 1u));
                if (!ok) break;
                uint8_t* ktile = sm + st * C::kStageBytes;
                uint8_t* vtile = ktile + C::kTileBytes;
                const uint32_t ka = base + st * C::kStageBytes, va = ka + C::kTileBytes;
                float ks[2][2], vs[2][2];  // steps of this lane's four positions
                if constexpr (I8) {
                    const float* steps = reinterpret_cast<const float*>(vtile + C::kTileBytes) + rw_slot<D, I8>(r8);
#pragma unroll
                    for (int pb = 0; pb < 2; ++pb)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            ks[pb][h] = steps[16 * pb + 8 * h] * a.qscale;
                            vs[pb][h] = steps[kRwChunk + 16 * pb + 8 * h];
                        }
                }
                float s[2][X][4];
#pragma unroll
                for (int pb = 0; pb < 2; ++pb)
#pragma unroll
                    for (int x = 0; x < X; ++x)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[pb][x][c] = 0.0f;
                if constexpr (I8) {
#pragma unroll
                    for (int blk = 0; blk < D / 64; ++blk) {
                        uint4 y[4];  // 16 codes of the four positions
#pragma unroll
                        for (int nb = 0; nb < 4; ++nb) {
                            const int r = nb * 8 + rw_slot<D, I8>(r8);
                            y[nb] = *reinterpret_cast<const uint4*>(ktile + r * D + (D == 128 ? (4 * blk + kq) ^ (r & 7) : kq) * 16);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int pb = 0; pb < 2; ++pb) {
                                const uint4 &u = y[2 * pb], &v = y[2 * pb + 1];
                                const uint32_t u1 = k == 0 ? u.x : k == 1 ? u.y : k == 2 ? u.z : u.w;
                                const uint32_t v1 = k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
                                const uint32_t ak[4] = {codes.two(__byte_perm(u1, 0, 0x4140)), codes.two(__byte_perm(v1, 0, 0x4140)),
                                                        codes.two(__byte_perm(u1, 0, 0x4342)), codes.two(__byte_perm(v1, 0, 0x4342))};
#pragma unroll
                                for (int x = 0; x < X; ++x) mma_bf16(s[pb][x], ak, q[4 * blk + k][x][0], q[4 * blk + k][x][1]);
                            }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
#pragma unroll
                        for (int pb = 0; pb < 2; ++pb) {
                            const int p = 16 * pb + ((lane >> 3) & 1) * 8 + (lane & 7), ch = 2 * (k & 3) + (lane >> 4);
                            uint32_t ak[4];
                            ldsm4(ka + (k >> 2) * kRwChunk * 128 + p * 128 + ((ch ^ (p & 7)) << 4), ak);
#pragma unroll
                            for (int x = 0; x < X; ++x) mma_bf16(s[pb][x], ak, q[k][x][0], q[k][x][1]);
                        }
                }
                // scores in the log2 domain, the hidden ones out
                const bool masked = t * kRwChunk + kRwChunk > vmin;
                const int p0 = t * kRwChunk + rw_slot<D, I8>(r8);
                float top[X][2];
                bool grows = false;
#pragma unroll
                for (int x = 0; x < X; ++x)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float y = -INFINITY;
#pragma unroll
                        for (int pb = 0; pb < 2; ++pb)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float& z = s[pb][x][2 * h + j];
                                z *= I8 ? ks[pb][h] : a.qscale;
                                if (masked && p0 + 16 * pb + 8 * h >= vend[x][j]) z = -INFINITY;
                                y = fmaxf(y, z);
                            }
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                        top[x][j] = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                        grows |= top[x][j] - m[x][j] > kPaMaxGrowth;
                    }
                if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                    for (int x = 0; x < X; ++x)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float mn = fmaxf(m[x][j], top[x][j]);
                            const float alpha = m[x][j] == mn ? 1.0f : ex2(m[x][j] - mn);
                            m[x][j] = mn;
                            l[x][j] *= alpha;
#pragma unroll
                            for (int db = 0; db < D / 16; ++db) {
                                o[db][x][j] *= alpha;
                                o[db][x][2 + j] *= alpha;
                            }
                        }
                }
                uint32_t p[2][X][2];  // the probabilities as the products' B operand
#pragma unroll
                for (int x = 0; x < X; ++x) {
                    const float ref[2] = {m[x][0] == -INFINITY ? 0.0f : m[x][0], m[x][1] == -INFINITY ? 0.0f : m[x][1]};
#pragma unroll
                    for (int pb = 0; pb < 2; ++pb)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float e[2];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                e[j] = ex2(s[pb][x][2 * h + j] - ref[j]);
                                l[x][j] += e[j];
                                // (a step behind the last position may be anything; rounded to bf16 with the probability,
                                // as in attn_paged.cuh)
                                if constexpr (I8) e[j] = masked && p0 + 16 * pb + 8 * h >= vend[x][j] ? 0.0f : e[j] * vs[pb][h];
                            }
                            p[pb][x][h] = movm_t(pack_bf16x2(e[0], e[1]));
                        }
                }
                if constexpr (!I8) {
                    const int valid = end - t * kRwChunk;
                    if (valid < kRwChunk) {
                        // values behind the last position that anything sees: zeros (probability zero times whatever
                        // the page holds there would not be)
                        for (int e = lane; e < (kRwChunk - valid) * 8 * (D / 64); e += 32) {
                            const int h = e / ((kRwChunk - valid) * 8), y = e % ((kRwChunk - valid) * 8);
                            *reinterpret_cast<uint4*>(vtile + h * kRwChunk * 128 + valid * 128 + y * 16) = make_uint4(0, 0, 0, 0);
                        }
                        __syncwarp();
                    }
                    // positions [from, to) are hidden from some of the item's rows
                    const int from = max(vmin - t * kRwChunk, 0), to = min(valid, kRwChunk);
                    const uint32_t bad = rw_non_finite<D>(vtile, from, to, lane);
                    for (uint32_t left = bad; left; left &= left - 1) {
                        const int y = __ffs(left) - 1;
#pragma unroll
                        for (int x = 0; x < X; ++x)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                // its probability for row 8 x + 2 kq + j, as the products take it
                                const uint32_t w2 = y < 16 ? (y < 8 ? p[0][x][0] : p[0][x][1]) : (y < 24 ? p[1][x][0] : p[1][x][1]);
                                const uint32_t both = __shfl_sync(0xffffffffu, w2, (2 * kq + j) * 4 + ((y & 7) >> 1));
                                if (t * kRwChunk + y >= vend[x][j]) continue;
                                const float e = __uint_as_float((y & 1) ? both & 0xFFFF0000u : both << 16);
#pragma unroll
                                for (int db = 0; db < D / 16; ++db)
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        const int ch = 2 * (db & 3) + h;
                                        const uint16_t v = *reinterpret_cast<const uint16_t*>(
                                            vtile + (db >> 2) * kRwChunk * 128 + y * 128 + ((ch ^ (y & 7)) << 4) + r8 * 2);
                                        o[db][x][2 * h + j] = fmaf(e, bf16_bits_to_float(v), o[db][x][2 * h + j]);
                                    }
                            }
                        __syncwarp();
                        if (lane < D / 8)
                            *reinterpret_cast<uint4*>(vtile + (lane >> 3) * kRwChunk * 128 + y * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                        __syncwarp();
                    }
                }
#pragma unroll
                for (int pb = 0; pb < 2; ++pb) {
                    if constexpr (I8) {
                        constexpr int N = D / 32;  // words of a lane's run of D/8 dimensions
                        uint32_t v[4][N];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {  // slots 2 kq and 2 kq + 1 of both eights
                            const int r = (2 * pb + (y >> 1)) * 8 + rw_slot<D, I8>(2 * kq + (y & 1));
                            if constexpr (D == 128) {
                                const uint4 z = *reinterpret_cast<const uint4*>(vtile + r * D + ((r8 ^ (r & 7)) << 4));
                                v[y][0] = z.x;
                                v[y][1] = z.y;
                                v[y][2] = z.z;
                                v[y][3] = z.w;
                            } else {
                                const uint2 z = *reinterpret_cast<const uint2*>(vtile + r * D + r8 * 8);
                                v[y][0] = z.x;
                                v[y][1] = z.y;
                            }
                        }
#pragma unroll
                        for (int db = 0; db < D / 16; ++db) {
                            uint32_t av[4];  // dimensions 2 db and 2 db + 1 of the run, both eights
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const int b = 2 * db + (y & 1);
                                const uint32_t pick = (uint32_t)((b & 3) | ((4 + (b & 3)) << 8));  // its bytes 0 and 2
                                av[y] = codes.two(__byte_perm(v[2 * (y >> 1)][b >> 2], v[2 * (y >> 1) + 1][b >> 2], pick));
                            }
#pragma unroll
                            for (int x = 0; x < X; ++x) mma_bf16(o[db][x], av, p[pb][x][0], p[pb][x][1]);
                        }
                    } else {
#pragma unroll
                        for (int db = 0; db < D / 16; ++db) {
                            const int r = 16 * pb + (lane >> 4) * 8 + (lane & 7), ch = 2 * (db & 3) + ((lane >> 3) & 1);
                            uint32_t av[4];
                            ldsm4t(va + (db >> 2) * kRwChunk * 128 + r * 128 + ((ch ^ (r & 7)) << 4), av);
#pragma unroll
                            for (int x = 0; x < X; ++x) mma_bf16(o[db][x], av, p[pb][x][0], p[pb][x][1]);
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(empty_bar(st));
            }
            if (!ok) break;
            n0 += t1 - t0;
            // ---- merge the CTA's warps ----
            const bool whole = t0 == 0 && t1 == item->nt;
            if (merges > 0) ok = __all_sync(0xffffffffu, mbar_wait(got_bar, (merges - 1) & 1u));  // the last item's are read
            if (!ok) break;
#pragma unroll
            for (int x = 0; x < X; ++x)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int y = 4; y < 32; y *= 2) l[x][j] += __shfl_xor_sync(0xffffffffu, l[x][j], y);
                    const int r = 8 * x + 2 * kq + j;
                    if (r < rows && t0 + skip < t1) {
                        if (r8 == 0) ml[w * NR + r] = make_float2(m[x][j], l[x][j]);
#pragma unroll
                        for (int db = 0; db < D / 16; ++db) {
                            osm[(w * NR + r) * C::kOStride + 16 * db + r8] = o[db][x][j];
                            osm[(w * NR + r) * C::kOStride + 16 * db + 8 + r8] = o[db][x][2 + j];
                        }
                    }
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(put_bar);
            ok = __all_sync(0xffffffffu, mbar_wait(put_bar, merges & 1u));
            if (!ok) break;
            const int slot = t0 == 0 ? 1 : 0;
            const int64_t prow = ((int64_t)blockIdx.x * 2 + slot) * kRwRows;
            const int done0 = (int)((n0 - (t1 - t0)) % W);  // warp of the item's first chunk
            const int used = min(t1 - t0, W);               // warps with chunks, from done0 on
            for (int x = ct; x < rows * (D / 2); x += 32 * W) {
                const int r = x / (D / 2), d = x % (D / 2) * 2;
                // the warps in the order of their first chunks
                float2 v[W];
                float mx = -INFINITY, den = 0.0f, n_0 = 0.0f, n_1 = 0.0f;
#pragma unroll
                for (int y = 0; y < W; ++y) {
                    v[y] = y < used ? ml[(done0 + y) % W * NR + r] : make_float2(-INFINITY, 0.0f);
                    mx = fmaxf(mx, v[y].x);
                }
#pragma unroll
                for (int y = 0; y < W; ++y) {
                    const float f = v[y].x == -INFINITY ? 0.0f : ex2(v[y].x - mx);
                    den = fmaf(f, v[y].y, den);
                    if (y < used) {
                        const float* src = osm + ((done0 + y) % W * NR + r) * C::kOStride;
                        n_0 = fmaf(f, src[rw_column<D, I8>(d)], n_0);
                        n_1 = fmaf(f, src[rw_column<D, I8>(d + 1)], n_1);
                    }
                }
                if (whole) {
                    const int row = item->row0 + r, tok = a.by_group.div(row);
                    const int ve = a.causal ? item->vbase + tok + 1 : item->len;
                    *reinterpret_cast<uint32_t*>(a.out + (int64_t)(item->q0 + tok) * a.o_stride + (head0 + a.by_group.mod(row)) * D + d) =
                        ve > 0 ? pack_bf16x2(n_0 / den, n_1 / den) : 0u;
                } else {
                    *reinterpret_cast<float2*>(a.part + (prow + r) * D + d) = make_float2(n_0, n_1);
                    if (d == 0) *reinterpret_cast<float2*>(a.part_ml + (prow + r) * 2) = make_float2(mx, den);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(got_bar);
            ++merges;
            if (!whole) {
                // ---- merge the item's parts over the CTAs ----
                // Up to kRwAlone parts: the last CTA to arrive merges them.  More: the last of each kRwGroup neighbours
                // merges those into the first one's place, and the last group's merges the groups.
                const int parts = item->parts, cta0 = item->cta0;
                const int groups = parts > kRwAlone ? (parts + kRwGroup - 1) / kRwGroup : 1;
                const int64_t unit0 = ((int64_t)item->unit_hi << 32) | (uint32_t)item->unit_lo, total = plan[6];
                // place of part y: slot 1 of the CTA the item begins in, slot 0 of the others
                auto place = [&](int y) {
                    const int x = item->spread ? rw_cta_of(unit0 + y, total) : cta0 + y;
                    return 2 * x + (y == 0 ? 1 : 0);
                };
                // This CTA arrives at a counter of the launch; whether it is the last of `count`.  The counter was set
                // by its CTA, which was started before this one and set it first of all: an arrival that still finds
                // another launch's value is overwritten by that, and made again.
                auto arrive_last = [&](unsigned long long* ctr, int count) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sent_bar);
                    ok = __all_sync(0xffffffffu, mbar_wait(sent_bar, sent & 1u));
                    ++sent;
                    if (!ok) return false;
                    if (ct == 0) {
                        const unsigned long long tag = epoch >> 32;
                        unsigned long long old = arrive_counter(ctr);
                        for (int tries = 0; old >> 32 != tag && tries < 64; ++tries) {
                            for (int spin = 0; spin < (1 << 16) && ld_acquire(ctr) >> 32 != tag; ++spin) {}
                            old = arrive_counter(ctr);
                        }
                        if (old >> 32 != tag) atomicOr(&g_status, kStatusTimeout);
                        const bool last = old >> 32 == tag && (int)(old & 0xFFFFFFFFull) + 1 == count;
                        if (last) st_counter(ctr, 0);  // nothing is left behind: a captured launch is replayed with its epoch
                        *last_flag = last;
                        mbar_arrive(told_bar);
                    }
                    __syncwarp();
                    ok = __all_sync(0xffffffffu, mbar_wait(told_bar, told & 1u));
                    ++told;
                    return ok && *last_flag;
                };
                constexpr int DL = D / 32;
                // parts first, first + step, ... (count of them), a row by a warp: into the place of the first (again a
                // part), or normalised into out
                auto merge_parts = [&](int first, int step, int count, bool final) {
                    for (int r = w; r < rows; r += W) {
                        float mx = -INFINITY, den = 0.0f, num[DL] = {};
                        for (int y0 = 0; y0 < count; y0 += kRwGroup) {
                            const int64_t from = (int64_t)place(first + min(y0 + (lane & (kRwGroup - 1)), count - 1) * step) * kRwRows + r;
                            float v[kRwGroup][DL];
#pragma unroll
                            for (int z = 0; z < kRwGroup; ++z) {
                                const float* src = a.part + __shfl_sync(0xffffffffu, from, z) * D + lane * DL;
                                if constexpr (DL == 4)
                                    *reinterpret_cast<float4*>(v[z]) = __ldcg(reinterpret_cast<const float4*>(src));
                                else
                                    *reinterpret_cast<float2*>(v[z]) = __ldcg(reinterpret_cast<const float2*>(src));
                            }
                            float2 y = __ldcg(reinterpret_cast<const float2*>(a.part_ml + from * 2));
                            if (y0 + (lane & (kRwGroup - 1)) >= count) y = make_float2(-INFINITY, 0.0f);
                            const float mn = fmaxf(mx, warp_max_f(y.x));
                            const float f = y.x == -INFINITY ? 0.0f : ex2(y.x - mn);
                            const float keep = mx == -INFINITY ? 0.0f : ex2(mx - mn);
                            den = fmaf(den, keep, warp_sum_f(lane < kRwGroup ? f * y.y : 0.0f));
#pragma unroll
                            for (int e = 0; e < DL; ++e) num[e] *= keep;
#pragma unroll
                            for (int z = 0; z < kRwGroup; ++z) {
                                const float fz = __shfl_sync(0xffffffffu, f, z);
                                if (y0 + z < count) {
#pragma unroll
                                    for (int e = 0; e < DL; ++e) num[e] = fmaf(fz, v[z][e], num[e]);
                                }
                            }
                            mx = mn;
                        }
                        if (final) {
                            const int row = item->row0 + r, tok = a.by_group.div(row);
                            const int ve = a.causal ? item->vbase + tok + 1 : item->len;
                            uint16_t* dst = a.out + (int64_t)(item->q0 + tok) * a.o_stride + (head0 + a.by_group.mod(row)) * D + lane * DL;
#pragma unroll
                            for (int e = 0; e < DL; e += 2)
                                *reinterpret_cast<uint32_t*>(dst + e) = ve > 0 ? pack_bf16x2(num[e] / den, num[e + 1] / den) : 0u;
                        } else {
                            const int64_t at = (int64_t)place(first) * kRwRows + r;
#pragma unroll
                            for (int e = 0; e < DL; ++e) a.part[at * D + lane * DL + e] = num[e];
                            if (lane == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(mx, den);
                        }
                    }
                };
                used_ctr |= t0 == 0 ? 1 : 0;
                bool final = true;
                if (groups > 1) {
                    const int mine = item->spread ? t0 : (int)blockIdx.x - cta0, head = mine / kRwGroup * kRwGroup;
                    const int count = min(kRwGroup, parts - head);
                    used_ctr |= mine == head ? (mine == 0 ? 4 : 2) : 0;
                    final = arrive_last(counters + gridDim.x + place(head), count);
                    if (final) merge_parts(head, 1, count, false);
                }
                if (final && ok && arrive_last(counters + cta0, groups > 1 ? groups : parts))
                    merge_parts(0, groups > 1 ? kRwGroup : 1, groups > 1 ? groups : parts, true);
                if (!ok) break;
            }
            release();
        }
        if (ct == 0) {  // counters of this CTA that nobody arrives at
            if (!(used_ctr & 1)) st_counter(counters + blockIdx.x, 0);
            if (!(used_ctr & 2)) st_counter(counters + gridDim.x + 2 * blockIdx.x, 0);
            if (!(used_ctr & 4)) st_counter(counters + gridDim.x + 2 * blockIdx.x + 1, 0);
        }
    }
    __syncthreads();
}

}  // namespace bl

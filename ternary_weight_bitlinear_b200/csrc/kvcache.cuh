// kvcache.cuh -- the paged key/value cache: new rows written into it
// (quantised per row when the cache holds int8) and read back out of it.
//
// A batch is described by three device arrays: cu_q[b] is the first new row
// of sequence b, kv_len[b] its positions (the new ones included), and
// pages[b, p / page_size] the page that holds position p.  Row i of the n
// new rows of a sequence stands at position kv_len - n + i, so the write, the
// read and the attention share one description of a step.
//
// int8 rows: the activation quantiser's codes (quant.cuh) per (position,
// key/value head), s = RN32(127 / max(max|x|, 1e-5)),
// code = clamp(rint(RN32(x s)), -128, 127), and step = RN32(1 / s) kept in
// binary32 beside them; a code stands for RN32(code step).  A row that holds
// an infinity or NaN has no scale: it is written as zero codes with a NaN
// step, so every reader of that row (and no other) gets NaN.
//
// Both kernels move each row once.  bf16 rows are bound by HBM bytes, int8 rows
// and a few rows by the latency of look-ups and loads (int8: DRAM 23 to 35 %,
// issue slots under half).  A group of d/8 lanes (int8: d/16) takes one or several (row,
// head) pairs, 16 bytes of the cache a lane; a warp looks up 32 sequences at
// once, a lane each, so a row costs two rounds of dependent loads (its
// sequence, its page) before its own; the row's maximum costs log2(d/16)
// shuffles.  Measured: 30,000 rows of 8 heads of 64 into a bf16 cache 24.0 us
// (5.1 TB/s of rows read and written); 43,500 positions of 5 heads of 128 read
// back from int8 38.2 us (4.4 TB/s); 333 rows read 2.3 us.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace bl {

constexpr int kKvThreads = 128;
constexpr int64_t kKvMaxPositions = 1 << 30;  // of a page table's row: position arithmetic stays in 32 bits
constexpr int64_t kKvMaxPairs = INT32_MAX - 1024;  // (row, key/value head) pairs: a grid's last block stays in 32 bits too

// Division of x < 2^31 by a divisor known on the host: with s = ceil(log2 d)
// and m = ceil(2^(31 + s) / d), m d exceeds 2^(31 + s) by less than d <= 2^s,
// so x m / 2^(31 + s) exceeds x / d by less than 1 / d and floors the same.
struct FastDiv {
    uint32_t d, m;
    int s;
    __device__ __forceinline__ int div(int x) const { return d == 1 ? x : (int)(__umulhi((uint32_t)x, m) >> (s - 1)); }
    __device__ __forceinline__ int mod(int x) const { return x - div(x) * (int)d; }
};
inline FastDiv fast_div(int64_t d) {
    FastDiv f = {(uint32_t)d, 0, 0};
    while (((int64_t)1 << f.s) < d) ++f.s;
    f.m = (uint32_t)((((uint64_t)1 << (31 + f.s)) + d - 1) / d);
    return f;
}

struct KvCacheArgs {
    void* k;                     // bf16 or int8 pages
    void* v;
    float* k_step;               // [num_pages, kv_heads, page_size] (int8 only)
    float* v_step;
    int64_t sp, ss, sh;          // strides in elements: page, slot, head
    int num_pages, page_size, kv_heads;
    FastDiv by_page, by_heads;
};

struct KvBatchArgs {
    const int32_t* cu_q;         // [batch + 1]
    const int32_t* kv_len;       // [batch]
    const int32_t* pages;        // [batch, max_pages]
    int batch;
    int max_pages;
    int T;                       // rows the caller's buffers have
    int max_len;                 // max_pages * page_size, at most kKvMaxPositions
};

// A sequence as the kernels see it: whatever the arrays hold, the rows lie
// inside [0, T) and the length inside the page table.
struct KvSeq {
    int q0, n, len;
};

__device__ __forceinline__ KvSeq kv_seq(const KvBatchArgs& a, int b) {
    KvSeq s;
    s.q0 = min(max(__ldcg(a.cu_q + b), 0), a.T);
    s.n = max(min(__ldcg(a.cu_q + b + 1), a.T) - s.q0, 0);
    s.len = min(max(__ldcg(a.kv_len + b), 0), a.max_len);
    return s;
}

// The sequence of row t, searched by a whole warp: the number of starts
// cu_q[1..batch] at or below t (batch when no sequence has the row).  The
// starts are in ascending order, so empty sequences are passed over; each
// round's 32 probes leave a 32nd of them.
__device__ __forceinline__ int kv_seq_of_row(const KvBatchArgs& a, int t, int lane) {
    uint32_t lo = 0, n = (uint32_t)a.batch;  // the answer lies in [lo, lo + n]
    while (n > 0) {
        const uint32_t step = (n + 31) / 32, at = (lane + 1) * step - 1;
        const bool below = at < n && __ldcg(a.cu_q + 1 + lo + at) <= t;
        const uint32_t c = __popc(__ballot_sync(0xffffffffu, below)) * step;
        lo += c;
        n = min(step - 1, n - c);
    }
    return (int)lo;
}

// The first sequence after b that has rows (batch: none).  Eight at a time: a
// step's batch may be padded with many that have none.
__device__ __forceinline__ int kv_next(const KvBatchArgs& a, int b) {
    for (++b; b < a.batch; b += 8) {
        int cu[9];
#pragma unroll
        for (int i = 0; i < 9; ++i) cu[i] = min(max(__ldcg(a.cu_q + min(b + i, a.batch)), 0), a.T);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (cu[i + 1] > cu[i]) return b + i;
    }
    return a.batch;
}

// Page of position p of sequence b, or -1 (recorded in the status word) when
// the table's entry is not a page of the cache.
__device__ __forceinline__ int kv_page(const KvCacheArgs& c, const KvBatchArgs& a, int b, int p) {
    const int page = __ldcg(a.pages + (int64_t)b * a.max_pages + c.by_page.div(p));
    if ((unsigned)page < (unsigned)c.num_pages) return page;
    atomicOr(&g_status, kStatusBadPage);
    return -1;
}

// 32 neighbouring sequences, one a lane of a warp.
struct KvWindow {
    int base, next;  // the window's first sequence; where this lane's sequence ends in the arrays (as it stands there)
    KvSeq s;
    // The window that holds the sequence of row t (the warp's first): with up to 32 sequences there is one only.
    __device__ __forceinline__ KvWindow(const KvBatchArgs& a, int t, int lane) {
        base = a.batch <= 32 ? 0 : min(kv_seq_of_row(a, t, lane), a.batch - 1);
        const bool have = base + lane < a.batch;
        next = have ? __ldcg(a.cu_q + base + lane + 1) : INT32_MAX;
        s = {0, 0, 0};
        if (have) s = kv_seq(a, base + lane);
    }
    // Where row t lies in the cache (element offset of (page, slot, head) and of its step); false when it has no place.
    // Every lane of the warp calls it, each with its own row.
    __device__ __forceinline__ bool place(const KvCacheArgs& c, const KvBatchArgs& a, int t, int head, int64_t* off,
                                          int64_t* step_off) const {
        int i = 0;  // sequences of the window that end at or before t (the ends ascend)
#pragma unroll
        for (int step = 16; step > 0; step >>= 1)
            if (__shfl_sync(0xffffffffu, next, i + step - 1) <= t) i += step;
        const bool past = __shfl_sync(0xffffffffu, next, i) <= t;  // behind the window
        KvSeq q = {__shfl_sync(0xffffffffu, s.q0, i), __shfl_sync(0xffffffffu, s.n, i), __shfl_sync(0xffffffffu, s.len, i)};
        int b = base + i;
        if (past) {
            while (b < a.batch && __ldcg(a.cu_q + b + 1) <= t) b = kv_next(a, b);
            if (b < a.batch) q = kv_seq(a, b);
        }
        const int pos = q.len - q.n + (t - q.q0);
        if (b >= a.batch || t < q.q0 || t >= q.q0 + q.n || pos < 0) return false;
        const int page = kv_page(c, a, b, pos);
        if (page < 0) return false;
        const int slot = c.by_page.mod(pos);
        *off = page * c.sp + slot * c.ss + head * c.sh;
        *step_off = ((int64_t)page * c.kv_heads + head) * c.page_size + slot;
        return true;
    }
};

// Largest |x| of eight bf16 values, as bf16 bits (above every finite value
// when one is an infinity or NaN).
__device__ __forceinline__ uint32_t kv_absmax8(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    return max(m & 0xFFFFu, m >> 16);
}

// Eight codes of one row's scale.  Adding 1.5 2^23 rounds to an integer (ties
// to even, as rint) and leaves it in two's complement in the low bits, without
// the slower conversion instructions; |x s| <= 127 (1 + 2^-23), so the clamp at
// -128 never binds.
__device__ __forceinline__ uint2 kv_codes8(const uint4& x, float s) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
        c[i] = __float_as_uint(__fadd_rn(__fmul_rn(f, s), 12582912.0f));
    }
    auto four = [&](int i) {
        return __byte_perm(__byte_perm(c[i], c[i + 1], 0x0040), __byte_perm(c[i + 2], c[i + 3], 0x0040), 0x5410);
    };
    return make_uint2(four(0), four(4));
}

// One row quantised by its group of LANES lanes, 16 elements a lane.
template <int LANES>
__device__ __forceinline__ void kv_store_i8(const uint4 (&x)[2], int8_t* dst, float* step, int part, bool live) {
    uint32_t m = max(kv_absmax8(x[0]), kv_absmax8(x[1]));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!live) return;
    const bool finite = m < 0x7F80u;
    const float s = __fdiv_rn(127.0f, fmaxf(bf16_bits_to_float(m), kScaleFloor));
    const uint2 lo = kv_codes8(x[0], s), hi = kv_codes8(x[1], s);
    *reinterpret_cast<uint4*>(dst + part * 16) = finite ? make_uint4(lo.x, lo.y, hi.x, hi.y) : make_uint4(0, 0, 0, 0);
    if (part == 0) *step = finite ? __frcp_rn(s) : __int_as_float(0x7FC00000);
}

// 16-byte vectors of bf16 a lane: one, or the two whose codes fill one.
template <bool I8>
constexpr int kKvVecs = I8 ? 2 : 1;

// R rows a group, GROUPS apart, so neighbouring groups have neighbouring heads
// and tokens.
template <int D, bool I8, int R>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const KvCacheArgs c, const KvBatchArgs a,
                                                              const uint16_t* __restrict__ k, int64_t k_stride,
                                                              const uint16_t* __restrict__ v, int64_t v_stride) {
    constexpr int V = kKvVecs<I8>, LANES = D / (8 * V), GROUPS = kKvThreads / LANES;
    const int lane = threadIdx.x & 31, part = threadIdx.x % LANES;
    const int pairs = a.T * c.kv_heads;  // (row, head) pairs
    const int block0 = blockIdx.x * (GROUPS * R);
    const int warp0 = block0 + (threadIdx.x & ~31) / LANES, first = block0 + threadIdx.x / LANES;
    pdl_wait();
    pdl_launch_dependents();
    if (warp0 >= pairs) return;  // warp-uniform
    uint4 kx[R][V], vx[R][V];
    int t[R], head[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const int pair = min(first + u * GROUPS, pairs - 1);
        t[u] = c.by_heads.div(pair);
        head[u] = pair - t[u] * c.kv_heads;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            kx[u][e] = __ldcg(reinterpret_cast<const uint4*>(k + t[u] * k_stride + head[u] * D) + part * V + e);
            vx[u][e] = __ldcg(reinterpret_cast<const uint4*>(v + t[u] * v_stride + head[u] * D) + part * V + e);
        }
    }
    const KvWindow window(a, c.by_heads.div(warp0), lane);
#pragma unroll
    for (int u = 0; u < R; ++u) {
        int64_t off = 0, step_off = 0;
        const bool live = window.place(c, a, t[u], head[u], &off, &step_off) && first + u * GROUPS < pairs;
        if constexpr (I8) {
            kv_store_i8<LANES>(kx[u], static_cast<int8_t*>(c.k) + off, c.k_step + step_off, part, live);
            kv_store_i8<LANES>(vx[u], static_cast<int8_t*>(c.v) + off, c.v_step + step_off, part, live);
        } else if (live) {
            *(reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.k) + off) + part) = kx[u][0];
            *(reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.v) + off) + part) = vx[u][0];
        }
    }
}

// Eight bf16 values of eight codes: RN_bf16(RN32(code * step)).  A code with its
// sign bit flipped is code + 128 >= 0: as the low byte of the binary32 2^23 it
// makes 2^23 + 128 + code, exactly.
__device__ __forceinline__ uint4 kv_values8(const uint2& c, float step) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = (i < 2 ? c.x : c.y) ^ 0x80808080u;
        const float lo = __uint_as_float(__byte_perm(w, 0x4B000000u, (i & 1) ? 0x7442 : 0x7440));
        const float hi = __uint_as_float(__byte_perm(w, 0x4B000000u, (i & 1) ? 0x7443 : 0x7441));
        r[i] = pack_bf16x2(__fmul_rn(__fsub_rn(lo, 8388736.0f), step), __fmul_rn(__fsub_rn(hi, 8388736.0f), step));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int D, bool I8, int R>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvCacheArgs c, const KvBatchArgs a,
                                                             uint16_t* __restrict__ k, int64_t k_stride,
                                                             uint16_t* __restrict__ v, int64_t v_stride) {
    constexpr int V = kKvVecs<I8>, LANES = D / (8 * V), GROUPS = kKvThreads / LANES;
    using Held = typename std::conditional<I8, int8_t, uint16_t>::type;
    const int lane = threadIdx.x & 31, part = threadIdx.x % LANES;
    const int pairs = a.T * c.kv_heads;
    const int block0 = blockIdx.x * (GROUPS * R);
    const int warp0 = block0 + (threadIdx.x & ~31) / LANES, first = block0 + threadIdx.x / LANES;
    pdl_wait();
    pdl_launch_dependents();
    if (warp0 >= pairs) return;
    const KvWindow window(a, c.by_heads.div(warp0), lane);
    uint4 kx[R], vx[R];  // as they are held
    float ks[R], vs[R];
    int64_t to_k[R], to_v[R];
    bool live[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const int pair = min(first + u * GROUPS, pairs - 1), t = c.by_heads.div(pair), head = pair - t * c.kv_heads;
        int64_t off, step_off;
        live[u] = window.place(c, a, t, head, &off, &step_off) && first + u * GROUPS < pairs;
        if (live[u]) {
            kx[u] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const Held*>(c.k) + off) + part);
            vx[u] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const Held*>(c.v) + off) + part);
            if constexpr (I8) {
                ks[u] = __ldcg(c.k_step + step_off);
                vs[u] = __ldcg(c.v_step + step_off);
            }
        }
        to_k[u] = t * k_stride + head * D;
        to_v[u] = t * v_stride + head * D;
    }
#pragma unroll
    for (int u = 0; u < R; ++u) {
        if (!live[u]) continue;
        uint4* const ko = reinterpret_cast<uint4*>(k + to_k[u]) + part * V;
        uint4* const vo = reinterpret_cast<uint4*>(v + to_v[u]) + part * V;
        if constexpr (I8) {
            ko[0] = kv_values8(make_uint2(kx[u].x, kx[u].y), ks[u]);
            ko[1] = kv_values8(make_uint2(kx[u].z, kx[u].w), ks[u]);
            vo[0] = kv_values8(make_uint2(vx[u].x, vx[u].y), vs[u]);
            vo[1] = kv_values8(make_uint2(vx[u].z, vx[u].w), vs[u]);
        } else {
            ko[0] = kx[u];
            vo[0] = vx[u];
        }
    }
}

}  // namespace bl

// chunk_plan.cuh -- the schedule shared by the attention kernels over paged
// caches: packed rows of a (sequence, KV head) cut into items, items into
// 128-key tiles, and the whole work into equal contiguous ranges, one per CTA
// (all computed on the device, where the lengths are).
#pragma once

#include "cache_kernels.h"

namespace hta {

constexpr int kPlanUnits = 2048;

// `bytes` contiguous bytes to shared memory (both ends 16-byte aligned, bytes a
// multiple of 16), counted on `bar`
__device__ __forceinline__ void bulk_load(void *dst, const void *src, int bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void bar_sync(int id, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// bits [lo, hi) of a 32-bit word (lo, hi any integers)
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
    const int h = min(max(hi, 0), 32), l = min(max(lo, 0), 32);
    const uint32_t below_h = h == 0 ? 0u : 0xffffffffu >> (32 - h);
    const uint32_t below_l = l == 0 ? 0u : 0xffffffffu >> (32 - l);
    return below_h & ~below_l;
}

// --------------------------------------------------------------- work items
struct Seq {
    int s0, n, L, rows, tiles;      // first token, tokens, prefix, packed rows, items per KV head
    bool bad;                       // prefix length out of range: rows come out as NaN
};

__device__ __forceinline__ Seq load_seq(const ChunkParams &p, int b) {
    Seq s;
    s.L = p.prefix_len[b];
    if (p.tree) {
        s.s0 = 0;
        s.n = p.N;
        s.bad = s.L < 0 || s.L > p.L_cap;
    } else {
        s.s0 = p.q_start[b];
        const int s1 = p.q_start[b + 1];
        s.n = (s.s0 < 0 || s1 < s.s0 || s1 > p.N) ? 0 : s1 - s.s0;   // (reported by check_ranges)
        s.bad = s.L < 0 || s.L > p.L_cap || s.n > p.L_cap - s.L;
    }
    s.rows = s.n * p.G;
    s.tiles = (s.rows + p.item_rows - 1) / p.item_rows;
    return s;
}

// x / G for 0 <= x < 2^31 (g_mul = floor(2^(31 + g_shift) / G) + 1 with 2^(g_shift - 1) < G <= 2^g_shift)
__device__ __forceinline__ int div_g(const ChunkParams &p, int x) {
    return p.G == 1 ? x : static_cast<int>(__umulhi(2u * static_cast<uint32_t>(x), p.g_mul) >> p.g_shift);
}

struct Item {
    int r0, rows;                   // packed rows [r0, r0 + rows)
    int two;                        // more than one 128-row tile
    int lo, hi, base;               // cache keys any row may see; first key of tile 0 (whole blocks)
    int all_lo, all_hi;             // keys every row sees
    int cache_tiles, nt;            // key tiles from the cache, and with the tree's
};

__device__ __forceinline__ Item item_of(const ChunkParams &p, const Seq &s, int tile) {
    Item it;
    it.r0 = tile * p.item_rows;
    it.rows = min(p.item_rows, s.rows - it.r0);
    it.two = it.rows > 128 ? 1 : 0;
    it.lo = it.all_lo = 0;
    if (s.bad) {
        it.hi = it.all_hi = 0;
    } else if (p.tree) {
        it.hi = it.all_hi = s.L;
    } else {
        const int t0 = div_g(p, it.r0), t1 = div_g(p, it.r0 + it.rows - 1);
        it.all_hi = s.L + t0 + 1;
        it.hi = s.L + t1 + 1;
        if (p.window > 0) {
            it.lo = max(0, s.L + t0 - p.window + 1);
            it.all_lo = max(0, s.L + t1 - p.window + 1);
        }
    }
    it.base = it.lo & ~(p.cache.block_size - 1);
    it.cache_tiles = (it.hi - it.base + 127) / 128;
    it.nt = it.cache_tiles + p.tree_tiles;
    if (it.nt == 0) it.nt = it.cache_tiles = 1;        // no key at all: one tile, wholly masked
    return it;
}

__device__ __forceinline__ int item_cost(const ChunkParams &p, const Item &it) {
    return p.c0 + it.nt * (it.two ? p.c2 : p.c1);
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
    return v;
}
template <typename T>
__device__ __forceinline__ T scan_add(T v) {                     // inclusive, over the warp
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const T o = __shfl_up_sync(0xffffffffu, v, k);
        if (lane >= k) v += o;
    }
    return v;
}

// cost of one KV head's items of a sequence, `first` by `step` of them
__device__ __forceinline__ long long seq_cost(const ChunkParams &p, const Seq &s, int first, int step) {
    long long cost = 0;
    for (int i = first; i < s.tiles; i += step) cost += item_cost(p, item_of(p, s, i));
    return cost;
}

struct Start {
    int b, kvh, tile, pad;
    long long at, begin, end;       // units: start of that item, this CTA's range
    Seq s;                          // sequence b
};

// The share of the work of each CTA, and where this CTA's begins (the whole
// CTA calls).  `plan` (shared scratch) takes the cost of each sequence, or of
// each 32 in batches of more than kPlanUnits: of long sequences a warp sums
// one's items, of short ones a thread.
static __device__ void plan_start(const ChunkParams &p, long long *plan, Start *out) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int per = p.B <= kPlanUnits ? 1 : 32, units = (p.B + per - 1) / per;
    if (per == 32) {
        for (int u = warp; u < units; u += warps) {
            const int b = u * 32 + lane;
            const long long c = warp_sum(b < p.B ? seq_cost(p, load_seq(p, b), 0, 1) : 0);
            if (lane == 0) plan[u] = c;
        }
    } else if (static_cast<long long>(p.N) * p.G > 512LL * (p.tree ? 1 : p.B)) {
        for (int b = warp; b < p.B; b += warps) {
            const long long c = warp_sum(seq_cost(p, load_seq(p, b), lane, 32));
            if (lane == 0) plan[b] = c;
        }
    } else {
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) plan[b] = seq_cost(p, load_seq(p, b), 0, 1);
    }
    __syncthreads();
    if (warp == 0) {
        long long total = 0;
        for (int u = lane; u < units; u += 32) total += plan[u];
        const long long work = (units == 1 ? plan[0] : warp_sum(total)) * p.Hkv;
        // Work of less than 2^31 units is counted in 32 bits: a call of few keys
        // has little else to do.  (Every CTA computes the same share; grid * share
        // >= work.)
        const bool small = work < (1LL << 31);
        const long long share = max(small ? static_cast<long long>(static_cast<uint32_t>(work) / gridDim.x + 1)
                                          : static_cast<long long>(static_cast<double>(work) / gridDim.x) + 1,
                                    static_cast<long long>(p.min_share));
        const long long begin = share * blockIdx.x, end = min(work, begin + share);
        Start st = {p.B, 0, 0, 0, 0, begin, end, {}};
        if (begin < work) {
            // the unit of sequences, the sequence, the KV head and the item that hold `begin`;
            // `before`: the work before it
            long long before = 0;
            auto find = [&](long long c, int &k) {      // c: the lanes' costs (of all KV heads)
                const long long cum = before + (small ? scan_add(static_cast<int>(c)) : scan_add(c));
                const uint32_t past = __ballot_sync(0xffffffffu, cum > begin);
                k = past ? __ffs(past) - 1 : 31;
                before = __shfl_sync(0xffffffffu, past ? cum - c : cum, k);
                return past != 0;
            };
            int k = 0, u = 0;
            if (units > 1)
                while (!find(u + lane < units ? plan[u + lane] * p.Hkv : 0, k) && u < units) u += 32;
            u = min(u + k, units - 1);
            st.b = u;
            long long cost = plan[u];
            if (per == 32) {
                const int b = u * 32 + lane;
                const long long c = b < p.B ? seq_cost(p, load_seq(p, b), 0, 1) : 0;
                find(c * p.Hkv, k);
                st.b = min(u * 32 + k, p.B - 1);
                cost = __shfl_sync(0xffffffffu, c, k);
            }
            const Seq s = load_seq(p, st.b);
            st.kvh = small ? static_cast<int>(static_cast<uint32_t>(begin - before) / static_cast<uint32_t>(cost))
                           : static_cast<int>(static_cast<double>(begin - before) / cost);
            if ((st.kvh + 1) * cost <= begin - before) ++st.kvh;     // (the division's rounding)
            if (st.kvh * cost > begin - before) --st.kvh;
            before += cost * st.kvh;
            k = 0;
            if (s.tiles > 1)        // (bounded: lengths that another stream changed meanwhile must not hang the search)
                while (!find(st.tile + lane < s.tiles ? item_cost(p, item_of(p, s, st.tile + lane)) : 0, k) &&
                       st.tile < s.tiles)
                    st.tile += 32;
            st.tile += k;
            st.s = s;
            st.at = before;
        }
        if (lane == 0) *out = st;
    }
    __syncthreads();
}

// The items of this CTA's range, in order; every role walks them alike.
struct Walk {
    int b, kvh, tile;
    long long at, begin, end;
    Seq s;
    Item it;
    int cur_kvh, cur_b;             // of `it`
    int j0, j1;                     // this CTA's key tiles of `it`

    __device__ __forceinline__ void start(const ChunkParams &p, const Start *st) {
        b = st->b;
        kvh = st->kvh;
        tile = st->tile;
        at = st->at;
        begin = st->begin;
        end = st->end;
        s = st->s;
    }
    __device__ __forceinline__ bool next(const ChunkParams &p) {
        for (;;) {
            if (b >= p.B || at >= end) return false;
            if (tile >= s.tiles) {
                tile = 0;
                if (s.tiles == 0 || ++kvh >= p.Hkv) {
                    kvh = 0;
                    if (++b >= p.B) return false;
                    s = load_seq(p, b);
                }
                continue;
            }
            it = item_of(p, s, tile);
            const int c = it.two ? p.c2 : p.c1;
            // tile j is this CTA's where at + c0 + j * c lies in [begin, end)
            const long long x0 = at + p.c0, x1 = x0 + static_cast<long long>(it.nt) * c;
            auto first_from = [&](long long x) {        // (differences below x1 - x0 fit an int)
                return x <= x0 ? 0 : x >= x1 ? it.nt : (static_cast<int>(x - x0) + c - 1) / c;
            };
            j0 = first_from(begin);
            j1 = first_from(end);
            cur_kvh = kvh;
            cur_b = b;
            at = x1;
            ++tile;
            if (j0 < j1) return true;
        }
    }
    __device__ __forceinline__ int key0(int j) const { return it.base + j * 128; }
    // a tile of cache keys that not every row of the item sees whole
    __device__ __forceinline__ bool partial(int j) const {
        return key0(j) < it.all_lo || key0(j) + 128 > it.all_hi;
    }
};

__device__ __forceinline__ long long slot_row(const ChunkParams &p, int cta, int which) {
    return (2LL * cta + which) * p.slot_rows;
}


// The header of this CTA's partial of item w.it.
__device__ __forceinline__ void write_head(const ChunkParams &p, const Walk &w, const Start *st, int which) {
    // segments: up to the CTA that holds the item's last tile
    const long long tail = w.at - (w.it.two ? p.c2 : p.c1), share = st->end - st->begin;
    PartHead hd;
    hd.b = w.cur_b;
    hd.kvh = w.cur_kvh;
    hd.r0 = w.it.r0;
    hd.rows = w.it.rows;
    hd.s0 = w.s.s0;
    hd.n = 1;
    for (long long e = w.end; e <= tail; e += share) ++hd.n;
    hd.pad0 = hd.pad1 = 0;
    p.heads[2 * blockIdx.x + which] = hd;
}

// A bounded wait that also ends when another wait of the CTA has given up.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort, uint32_t *status) {
    const uint32_t a = smem_u32(bar);
    if (mbar_test(a, parity & 1)) return true;
    const long long t0 = clock64();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(a, parity & 1)) return true;
        if ((i & 63u) == 0) {
            if (*abort) return false;
            if (clock64() - t0 > kWaitLimitCycles) {
                *abort = 1;
                raise_status(status, kStatusPipelineTimeout);
                return false;
            }
        }
    }
}

}  // namespace hta

// cache_kernels.h -- parameter blocks and launchers of the operators that
// take tokens into a paged KV cache and read it back: norm and rotation of
// query/key heads, append, chunk attention, and the e4m3 form of the cache
// (internal to liblongspec_hta.so).
//
// e4m3 cache rows: a row x of D values is kept as D e4m3 codes c and one
// byte e (the exponent format of block-scaled 8-bit floats, bias 127), with
//   x ~ c * 2^(e - 127),  2^(e - 127) the smallest power of two with
//   max|x| <= 448 * 2^(e - 127),  e clamped to [16, 134].
// A power of two costs an e4m3 row nothing that a free scale would save (the
// codes are floating point: their relative spacing does not move, only the
// 18-octave range shifts by less than one octave), and the attention kernels
// can then scale codes exactly: they feed f16 tensor-core products, in which
// every code and every value the format holds (up to 448 * 2^7 = 57344, the
// upper clamp; larger ones saturate) is a number.  A row holding a NaN or an
// infinity is stored as e = 255 with NaN codes and reads back as NaN.
#pragma once

#include "hta_kernels.h"

namespace hta {

// status bits beside those of hta_common.cuh
constexpr uint32_t kStatusBadRanges = 1u << 6;   // q_start not ascending inside [0, N]

constexpr int kScaleMin = 16, kScaleMax = 134, kScaleNan = 255;

// A paged cache: [num_blocks][Hkv][block_size][D], bf16, or e4m3 when
// k_scale/v_scale [num_blocks][Hkv][block_size] are set.
struct CacheView {
    void *k, *v;
    uint8_t *k_scale, *v_scale;
    const int32_t *block_table;       // [B][max_blocks]
    int block_size, max_blocks, num_blocks;
};

// [..][H][D] rows of bf16 at b*sb + h*sh + t*st elements
struct HeadRows {
    __nv_bfloat16 *p;
    long long sb, sh, st;
};

// Norm + rotation of q and k rows and/or append of k and v rows.
// Token n (0 <= n < B*T for dense rows, < N for a ragged chunk, where b = 0).
struct RowsParams {
    int Hq, Hkv, D;
    int T;                            // tokens per b of the strided views; N for ragged chunks
    int tokens;
    HeadRows q, k, v, q_out, k_out;   // q_out/k_out: dense outputs (k_out null when appending)
    const int32_t *positions;         // [tokens]; null: prefix_len[b] + place in the chunk
    // rotation (rotate = 0: none) and norms (null weight: none)
    int rotate, rot_dim, interleaved;
    const float *inv_freq;            // [rot_dim / 2]
    float rope_scale, eps;
    const __nv_bfloat16 *q_weight, *k_weight;
    // append (cache.k null: none)
    CacheView cache;
    const int32_t *prefix_len, *q_start;
    int B, L_cap;
    uint32_t *status;
    int n_split;                      // warps that share a token's heads
};
cudaError_t launch_rows(const RowsParams &p, int num_sms, cudaStream_t stream);

// commit of the accepted path into an e4m3 cache
struct CommitQ8Params {
    int B, Hkv, D, T, L_cap;
    CacheView cache;
    int32_t *prefix_len;
    const __nv_bfloat16 *k_tree, *v_tree;
    const int32_t *accept_len, *path;
    uint32_t *status;
};
cudaError_t launch_commit_q8(const CommitQ8Params &p, cudaStream_t stream);

// Which rows a partial of chunk_tc_kernel belongs to.
struct PartHead {
    int b, kvh, r0, rows;             // rows 0: the slot is empty
    int s0, n, pad0, pad1;            // n (slot 1): segments of the item
};

// Attention of query rows to a paged cache.  Two row layouts:
//   chunk (tree = 0): q [N][Hq][D] (token stride q_stride), token t of
//     sequence b at position prefix_len[b] + t, sees keys (pos - window, pos];
//   tree  (tree = 1): q [B][Hq][N][D], every row of b sees keys [0, prefix_len[b])
//     and, with tree_tiles = ceil(N / 128) > 0, its node's ancestors and
//     itself among the tree's keys k_tree, v_tree [B][Hkv][N][D].
// Output row = token*Hq + h (chunk) or (b*Hq + h)*N + t (tree).
struct ChunkParams {
    int B, Hq, Hkv, G, D, N, L_cap, window, tree, tree_tiles;
    float scale_log2;
    const __nv_bfloat16 *q;
    long long q_stride;
    CacheView cache;
    const int32_t *prefix_len, *q_start;
    const __nv_bfloat16 *k_tree, *v_tree;
    const int32_t *parent;
    __nv_bfloat16 *out;
    float *lse;
    uint32_t *status;
    // schedule and partials (chunk_plan.cuh): grid CTAs, two slots of slot_rows
    // rows each
    int grid, slot_rows;
    uint32_t g_mul;                   // division by G (div_g)
    int g_shift;
    int item_rows;                    // packed rows of an item, at most
    int c0, c1, c2, min_share;        // units of work: an item, a key tile of one / two row tiles; least share of a CTA
    PartHead *heads;                  // [2 * grid]
    float *o_part, *lse_part;         // [2 * grid][slot_rows][D], [2 * grid][slot_rows]
};
// tm: K and V cache as [num_blocks*Hkv*block_size][D], bf16 in boxes of 64
// columns by block_size rows with 128B swizzle, e4m3 in whole rows without;
// K and V of the tree as [B*Hkv*N][D], box 64 x 128, 128B swizzle (not used
// without tree tiles)
// few rows of each sequence, e4m3 cache; K and V maps: whole rows of codes,
// 128B (D = 128) or 64B (D = 64) swizzle
cudaError_t launch_chunk_decode(const ChunkParams &p, const CUtensorMap (&tm)[4], cudaStream_t stream);
cudaError_t launch_chunk_merge(const ChunkParams &p, cudaStream_t stream);
cudaError_t launch_chunk_tc(const ChunkParams &p, const CUtensorMap (&tm)[4], cudaStream_t stream);

// A launch whose start may overlap the end of the kernel before it (every
// kernel here waits for that one before it touches memory).
struct OverlappedLaunch {
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg;
    OverlappedLaunch(dim3 grid, dim3 block, size_t smem, cudaStream_t stream) : attr(), cfg() {
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        cfg.gridDim = grid;
        cfg.blockDim = block;
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
    }
    OverlappedLaunch(const OverlappedLaunch &) = delete;
};

// -------------------------------------------------------------- device parts
// The sequence of token i: the largest b with q_start[b] <= i, run by a whole
// warp as a 32-way search (two rounds for up to 1024 sequences).  Returns -1
// where no sequence holds i (padding).  Only reads q_start[0..B]; in an array
// that is out of order it may find a wrong b, but never one with i outside
// [q_start[b], q_start[b+1]).
__device__ __forceinline__ int find_sequence(const int32_t *q_start, int B, int i, int &s0, int &s1) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;                    // b in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int b = lo + lane * step;
        const bool below = lane * step < n && q_start[b] <= i;
        const uint32_t m = __ballot_sync(0xffffffffu, below);
        if (m == 0) return -1;
        const int k = 31 - __clz(m);
        lo += k * step;
        n = min(step, n - k * step);
    }
    s0 = q_start[lo];
    s1 = q_start[lo + 1];
    return (s0 <= i && i < s1 && s0 >= 0) ? lo : -1;
}

// q_start ascending inside [0, N], checked by one warp of the grid; raises
// kStatusBadRanges.
__device__ __forceinline__ void check_ranges(const int32_t *q_start, int B, int N, uint32_t *status) {
    bool bad = false;
    for (int b = threadIdx.x & 31; b < B; b += 32) {
        const int a = q_start[b], c = q_start[b + 1];
        bad |= a < 0 || c < a || c > N;
    }
    if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) raise_status(status, kStatusBadRanges);
}

// Scale byte of an e4m3 row from the largest |bf16| bit pattern of the row.
// 448 = 1.75 * 2^8: a mantissa above 1.75 (96/128) needs the next power.
__device__ __forceinline__ int e4m3_scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7f80u) return kScaleNan;
    const int e = static_cast<int>(amax_bits >> 7) - 8 + ((amax_bits & 127u) > 96u ? 1 : 0);
    return min(max(e, kScaleMin), kScaleMax);
}

// Four values to four e4m3 codes (round to nearest even, saturating).
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

}  // namespace hta

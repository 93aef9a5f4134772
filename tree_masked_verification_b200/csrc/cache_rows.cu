// cache_rows.cu -- rows of new tokens on their way into attention: the norm
// of each query and key head, the rotation by position, and the append of K
// and V to a paged cache (bf16 or e4m3), in one pass over the projection's
// output; and the commit of an accepted path into an e4m3 cache.
//
// Per row x of D values (one head of one token):
//   norm      y = x / sqrt(mean(x^2) + eps) * w                (optional)
//   rotation  for i < rot/2, the pair (a, b) = (y[i], y[i + rot/2]) or, when
//             interleaved, (y[2i], y[2i+1]):
//             (a cos - b sin, b cos + a sin), angle = position * inv_freq[i]
//   append    the row rounded to bf16, copied or quantised to e4m3
// all in fp32, rounded once to bf16 (what the 16-bit cache holds is what the
// 8-bit cache quantises, so both caches come from the same keys).
//
// The angle: positions reach the millions, where an fp32 product is off by
// whole turns' hundredths.  position * inv_freq / pi is formed in fp64 (the
// device has a full-rate unit for the few needed: rot/2 per token, shared by
// all its heads), reduced to [-1, 1] half-turns there and only then rounded
// to fp32 for sincospif.
//
// Bound by memory: every value is read once and written once.  A thread
// holds 16 values of a row as two 16-byte pieces, D/2 apart (piece 0: values
// 8l..8l+7, piece 1: D/2 + 8l..), so that with a full rotation in halves both
// values of a pair sit in the same thread; interleaved pairs always do.  Only
// a partial rotation in halves goes through shared memory.  D/16 lanes make a
// row, a warp works on 4 (D = 128) or 8 (D = 64) heads of one token at a time
// and keeps that token's cos/sin in registers; the next rows' loads are
// issued before the current rows are computed.  Few tokens: a token's heads
// are spread over n_split warps.  16k tokens of 32 KV heads: bf16 88 us, 0.94 of the
// measured copy, e4m3 68-74 us; 7 ragged chunks (4062 tokens of 32 over 8 heads)
// normed and rotated 26 us into either cache: 0.86 of a wave of warps, each with 12
// blocks of heads one behind the other.
#include "cache_kernels.h"

namespace hta {

namespace {

constexpr int kRowWarps = 8;
constexpr int kRowThreads = kRowWarps * 32;

enum RotMode : int { kRotNone = 0, kRotHalves = 1, kRotInterleaved = 2, kRotHalvesPartial = 3 };

// a 16-byte piece as 8 fp32 values and back
__device__ __forceinline__ void unpack8(uint4 u, float *x) {
    x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x);
    x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z);
    x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float *x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// largest |bf16| bit pattern of the row whose 16-value parts the LPR lanes hold
template <int LPR>
__device__ __forceinline__ uint32_t row_amax_bits(uint4 a, uint4 b) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// the codes of one 8-value piece; mul = 2^(127 - e) (unused for e = 255)
__device__ __forceinline__ uint2 quantise8(uint4 u, int e) {
    if (e == kScaleNan) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    const float mul = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    float x[8];
    unpack8(u, x);
    return make_uint2(pack_e4m3x4(x[0] * mul, x[1] * mul, x[2] * mul, x[3] * mul),
                      pack_e4m3x4(x[4] * mul, x[5] * mul, x[6] * mul, x[7] * mul));
}

// Row (slot, h) of the cache <- the row whose parts the LPR lanes hold.  The
// whole warp calls this (the row maximum is a shuffle); `ok` lanes store.
template <int D>
__device__ __forceinline__ void store_cache_row(void *cache, uint8_t *scale, size_t row, uint4 a, uint4 b, int l,
                                                bool ok) {
    if (scale) {
        const int e = e4m3_scale_byte(row_amax_bits<D / 16>(a, b));
        if (ok) {
            uint8_t *dst = static_cast<uint8_t *>(cache) + row * D;
            *reinterpret_cast<uint2 *>(dst + 8 * l) = quantise8(a, e);
            *reinterpret_cast<uint2 *>(dst + D / 2 + 8 * l) = quantise8(b, e);
            if (l == 0) scale[row] = static_cast<uint8_t>(e);
        }
    } else if (ok) {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(cache) + row * D);
        dst[l] = a;
        dst[D / 16 + l] = b;
    }
}

// Four CTAs an SM (64 registers) hide more latency where they fit: rotated
// append of ragged chunks 29.6 -> 25.6 us; interleaved pairs need 80 (a 16k
// chunk: 67 us with three CTAs, 78 with four).
template <int D, int MODE>
__global__ void __launch_bounds__(kRowThreads, MODE == kRotInterleaved ? 3 : 4)
rows_kernel(const RowsParams p) {
    constexpr int LPR = D / 16;           // lanes per row
    constexpr int RPW = 32 / LPR;         // rows a warp works on at a time
    // cos | sin of the token's pairs; with a partial rotation in halves also
    // the warp's normalised rows
    __shared__ float s_cs[kRowWarps][D];
    __shared__ float s_rows[MODE == kRotHalvesPartial ? kRowWarps * RPW * D : 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane / LPR, l = lane % LPR;
    // (tokens * n_split stays below 2^31: n_split > 1 only for few tokens)
    const unsigned unit = blockIdx.x * kRowWarps + warp;
    const int token = static_cast<int>(unit / p.n_split), split = static_cast<int>(unit % p.n_split);
    const bool append = p.cache.k != nullptr;
    if (append && unit == 0) check_ranges(p.q_start, p.B, p.tokens, p.status);
    if (token >= p.tokens) return;        // (whole warps)
    // Padding: its rows need not exist, so none is read ahead of this.  (Tokens in front of
    // q_start[B] that no sequence holds, ranges out of order, are found below.)
    if (append && token >= p.q_start[p.B]) return;

    // blocks of RPW heads: q, then k, then v
    const bool has_q = p.q.p != nullptr;
    const int qb = has_q ? (p.Hq + RPW - 1) / RPW : 0, kb = (p.Hkv + RPW - 1) / RPW;
    const int nb = qb + kb + (append ? kb : 0);
    const int bi = token / p.T, ti = token % p.T;
    struct Piece { uint4 a, b; };
    auto load = [&](int blk) {
        Piece x = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        const HeadRows &src = blk < qb ? p.q : blk < qb + kb ? p.k : p.v;
        const int h = (blk < qb ? blk : blk < qb + kb ? blk - qb : blk - qb - kb) * RPW + g;
        if (blk < nb && h < (blk < qb ? p.Hq : p.Hkv)) {
            const uint4 *r = reinterpret_cast<const uint4 *>(src.p + bi * src.sb + h * src.sh + ti * src.st);
            x.a = r[l];
            x.b = r[LPR + l];
        }
        return x;
    };
    Piece next = load(split);             // in flight while the position is looked up

    int seq = 0, pos = 0;
    bool bad = false;
    long long slot = 0;                   // block * Hkv * block_size + place in the block
    if (append) {
        int s0 = 0, s1 = 0;
        seq = find_sequence(p.q_start, p.B, token, s0, s1);
        if (seq < 0) return;              // nothing is written for it
        const int L = p.prefix_len[seq];
        if (L < 0 || L > p.L_cap || s1 - s0 > p.L_cap - L) {
            if (lane == 0) raise_status(p.status, kStatusPrefixLenRange);
            bad = true;
        } else {
            pos = L + token - s0;
            const int blk = p.cache.block_table[static_cast<size_t>(seq) * p.cache.max_blocks + pos / p.cache.block_size];
            if (blk < 0 || blk >= p.cache.num_blocks) {
                if (lane == 0) raise_status(p.status, kStatusBadBlock);
                bad = true;
            }
            slot = static_cast<long long>(blk) * p.Hkv * p.cache.block_size + pos % p.cache.block_size;
        }
    } else {
        pos = p.positions[token];
    }

    // cos and sin of this token's pairs, two per lane, through shared memory
    // into the registers of the lanes that use them
    float c0[8], s0v[8];                  // halves: pairs 8l..8l+7; interleaved: pairs 4l.. and D/4 + 4l..
    if constexpr (MODE != kRotNone) {
        const int half = p.rot_dim / 2;
        float *cs = s_cs[warp], *sn = cs + D / 2;
        for (int i = lane; i < D / 2; i += 32) {
            float c = 1.f, s = 0.f;
            if (i < half) {
                double y = static_cast<double>(pos) * static_cast<double>(p.inv_freq[i]) * 0.3183098861837906715;
                y -= 2.0 * rint(y * 0.5);
                sincospif(static_cast<float>(y), &s, &c);
                c *= p.rope_scale;
                s *= p.rope_scale;
            }
            cs[i] = c;
            sn[i] = s;
        }
        __syncwarp();
        if constexpr (MODE == kRotHalves || MODE == kRotInterleaved) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int i = MODE == kRotHalves ? 8 * l + 4 * j : j * (D / 4) + 4 * l;
                const float4 c = *reinterpret_cast<const float4 *>(cs + i);
                const float4 s = *reinterpret_cast<const float4 *>(sn + i);
                c0[4 * j] = c.x; c0[4 * j + 1] = c.y; c0[4 * j + 2] = c.z; c0[4 * j + 3] = c.w;
                s0v[4 * j] = s.x; s0v[4 * j + 1] = s.y; s0v[4 * j + 2] = s.z; s0v[4 * j + 3] = s.w;
            }
        }
    }

    for (int blk = split; blk < nb; blk += p.n_split) {
        Piece x = next;
        next = load(blk + p.n_split);
        const int kind = blk < qb ? 0 : blk < qb + kb ? 1 : 2;
        const int h = (kind == 0 ? blk : kind == 1 ? blk - qb : blk - qb - kb) * RPW + g;
        const bool ok = h < (kind == 0 ? p.Hq : p.Hkv);
        if constexpr (MODE != kRotNone) {
            if (kind != 2) {
                float y[16];
                unpack8(x.a, y);
                unpack8(x.b, y + 8);
                const __nv_bfloat16 *w = kind == 0 ? p.q_weight : p.k_weight;
                if (w) {
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float f = 1.f / sqrtf(ss * (1.f / D) + p.eps);
                    float wv[16];
                    unpack8(reinterpret_cast<const uint4 *>(w)[l], wv);
                    unpack8(reinterpret_cast<const uint4 *>(w)[LPR + l], wv + 8);
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] *= f * wv[i];
                }
                if constexpr (MODE == kRotHalves) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float a = y[i], b = y[8 + i];
                        y[i] = a * c0[i] - b * s0v[i];
                        y[8 + i] = b * c0[i] + a * s0v[i];
                    }
                } else if constexpr (MODE == kRotInterleaved) {
                    const int half = p.rot_dim / 2;   // the pairs from there on pass through
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const bool in = (i < 4 ? 0 : D / 4 - 4) + 4 * l + i < half;
                        const float a = y[2 * i], b = y[2 * i + 1];
                        y[2 * i] = in ? a * c0[i] - b * s0v[i] : a;
                        y[2 * i + 1] = in ? b * c0[i] + a * s0v[i] : b;
                    }
                } else {
                    float *row = s_rows + (warp * RPW + g) * D;
                    const float *cs = s_cs[warp], *sn = cs + D / 2;
                    const int half = p.rot_dim / 2;
#pragma unroll
                    for (int i = 0; i < 16; ++i) row[(i < 8 ? 0 : D / 2 - 8) + 8 * l + i] = y[i];
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int d = (i < 8 ? 0 : D / 2 - 8) + 8 * l + i;
                        if (d < half) y[i] = y[i] * cs[d] - row[d + half] * sn[d];
                        else if (d < p.rot_dim) y[i] = y[i] * cs[d - half] + row[d - half] * sn[d - half];
                    }
                    __syncwarp();
                }
                x.a = pack8(y);
                x.b = pack8(y + 8);
            }
        }
        if (kind == 2 || (kind == 1 && append)) {
            const size_t row = static_cast<size_t>(slot + static_cast<long long>(h) * p.cache.block_size);
            store_cache_row<D>(kind == 1 ? p.cache.k : p.cache.v, kind == 1 ? p.cache.k_scale : p.cache.v_scale, row,
                               x.a, x.b, l, ok && !bad);
        } else if (ok) {
            const HeadRows &dst = kind == 0 ? p.q_out : p.k_out;
            if (bad) {                    // the sequence's length or block is out of range
                x.a = x.b = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
            }
            uint4 *r = reinterpret_cast<uint4 *>(dst.p + bi * dst.sb + h * dst.sh + ti * dst.st);
            r[l] = x.a;
            r[LPR + l] = x.b;
        }
    }
}

template <int D>
cudaError_t launch_rows_d(const RowsParams &p, unsigned grid, cudaStream_t stream) {
    OverlappedLaunch l(dim3(grid), dim3(kRowThreads), 0, stream);
    if (!p.rotate) return cudaLaunchKernelEx(&l.cfg, rows_kernel<D, kRotNone>, p);
    if (p.interleaved) return cudaLaunchKernelEx(&l.cfg, rows_kernel<D, kRotInterleaved>, p);
    if (p.rot_dim == D) return cudaLaunchKernelEx(&l.cfg, rows_kernel<D, kRotHalves>, p);
    return cudaLaunchKernelEx(&l.cfg, rows_kernel<D, kRotHalvesPartial>, p);
}

}  // namespace

cudaError_t launch_rows(const RowsParams &p0, int num_sms, cudaStream_t stream) {
    RowsParams p = p0;
    const int rpw = 512 / p.D;
    const int kb = (p.Hkv + rpw - 1) / rpw;
    const int nb = (p.q.p ? (p.Hq + rpw - 1) / rpw : 0) + kb + (p.cache.k ? kb : 0);
    // about 16 warps per SM before a warp takes more than one block of heads
    const int want = (16 * num_sms + p.tokens - 1) / p.tokens;
    p.n_split = want < 1 ? 1 : want > nb ? nb : want;
    const long long units = 1LL * p.tokens * p.n_split;
    const unsigned grid = static_cast<unsigned>((units + kRowWarps - 1) / kRowWarps);
    return p.D == 128 ? launch_rows_d<128>(p, grid, stream) : launch_rows_d<64>(p, grid, stream);
}

// ------------------------------------------------------- commit, e4m3 cache
// One CTA per sequence (the in-place prefix_len update then needs no
// grid-wide order), as for the bf16 cache; a group of D/16 lanes per row.
namespace {

constexpr int kCommitThreads = 256;

template <int D>
__global__ void __launch_bounds__(kCommitThreads)
commit_q8_kernel(const CommitQ8Params p) {
    constexpr int LPR = D / 16;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ int s_path[kTMax];
    __shared__ int s_blk[kTMax];
    __shared__ int s_bad;
    const int b = blockIdx.x, T = p.T;
    const int L = p.prefix_len[b];
    const int n = p.accept_len[b];
    if (n < 0 || n > T || L < 0 || L > p.L_cap || n > p.L_cap - L) {
        if (threadIdx.x == 0) raise_status(p.status, n < 0 || n > T ? kStatusBadPath : kStatusPrefixLenRange);
        return;
    }
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    for (int d = threadIdx.x; d < n; d += kCommitThreads) {
        const int node = p.path[static_cast<size_t>(b) * T + d];
        const int blk = p.cache.block_table[static_cast<size_t>(b) * p.cache.max_blocks + (L + d) / p.cache.block_size];
        if (node < 0 || node >= T) { raise_status(p.status, kStatusBadPath); s_bad = 1; }
        if (blk < 0 || blk >= p.cache.num_blocks) { raise_status(p.status, kStatusBadBlock); s_bad = 1; }
        s_path[d] = node;
        s_blk[d] = blk;
    }
    __syncthreads();
    if (s_bad) return;                    // the sequence is left as it was

    // row r of (kv, h, d); every warp makes the same number of rounds so that
    // the row maximum is taken by whole warps
    const int total = 2 * p.Hkv * n;
    const int l = threadIdx.x % LPR;
    for (int r0 = 0; r0 < total; r0 += kCommitThreads / LPR) {
        const int r = r0 + threadIdx.x / LPR;
        const bool ok = r < total;
        const int d = ok ? r % n : 0, hk = ok ? r / n : 0;
        const int h = hk % p.Hkv, kv = hk / p.Hkv;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            (kv ? p.v_tree : p.k_tree) + ((static_cast<size_t>(b) * p.Hkv + h) * T + s_path[d]) * D);
        const uint4 x = src[l], y = src[LPR + l];
        const size_t row = (static_cast<size_t>(s_blk[d]) * p.Hkv + h) * p.cache.block_size + (L + d) % p.cache.block_size;
        store_cache_row<D>(kv ? p.cache.v : p.cache.k, kv ? p.cache.v_scale : p.cache.k_scale, row, x, y, l, ok);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();                      // every thread has read L before it changes
    if (threadIdx.x == 0) p.prefix_len[b] = L + n;
}

}  // namespace

cudaError_t launch_commit_q8(const CommitQ8Params &p, cudaStream_t stream) {
    OverlappedLaunch l(dim3(p.B), dim3(kCommitThreads), 0, stream);
    return p.D == 128 ? cudaLaunchKernelEx(&l.cfg, commit_q8_kernel<128>, p)
                      : cudaLaunchKernelEx(&l.cfg, commit_q8_kernel<64>, p);
}

}  // namespace hta

// Products of int4 weight rows (group scales) with a few tokens
// (moe_w4_matvec):  y[t][n] = sum_g s[n][g] sum_{k in g} c[n][k] xr[t][k].
//
// The weights are read once, so the bound is their stream; the arithmetic runs
// on v_mfma_f32_16x16x32_bf16 with 16 weight rows on one side and 16 columns of
// x on the other, because unpacking to MFMA operands costs one VALU operation
// a weight whatever the number of tokens is.
//
// Exactness: code c enters as the bf16 value 24 + c (16 <= . < 32: the nibble,
// its sign bit flipped, in mantissa bits 3..6 of 16.0), and 24 sum(x) is taken
// off by starting each group's sums at -24 times the sum of x over the group.  x
// enters as 1 to 3 bf16 columns that add up to it (bf16 is itself; fp16 and
// rotated values are two, 16 bits, or three, 24 bits, for fp32 results), so every
// product is exact and only the fp32 sums round.
//
// Work: a workgroup takes a run of 16-row tiles and makes one sequence of their
// 128-blocks of K, of which its waves take equal parts, so that neither few rows
// nor an odd number of tiles leaves waves idle; where a tile's blocks fall to
// several waves, their sums meet in LDS at the end, in order.
//
// One launch, if the operands of x fit LDS: each workgroup makes them there while
// its first weights are on their way.  Otherwise a launch before makes them in the
// workspace, and the waves read them through the caches.
//
// Measured (MI355X): 1 token, 2048 x 2048 5.3 us (latency: a launch of nothing takes
// about 2, x's way through LDS 1.5); 4 tokens, 12288 x 2048 7.7 us; 150144 x 2048: 1
// token 33 us (4.8 TB/s; the loads alone 29), 8 tokens 36, 32 tokens 47 (3.8 TB/s with
// y: each wave reads all of x from LDS for its 16 rows, which takes 20 us of the LDS
// beside the stream).
#include <type_traits>

#include "common.h"
#include "launch.h"

namespace moe_w4 {

struct MatvecPlan {
    int cols;       // columns of x
    int tiles;      // 16-row tiles
    int run;        // tiles of a workgroup, one more in the first `more`
    int more;
    uint32_t inv;   // ceil(2^32 / blocks of a row)
};

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kLdsBytes = 160 * 1024;

__device__ __forceinline__ f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

__device__ __forceinline__ uint2 bload8(__amdgpu_buffer_rsrc_t r, uint32_t voff) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, voff, 0, 0);
    return make_uint2(v[0], v[1]);
}

// Lanes 8..15 of every 16 of a change places with lanes 0..7 of b.
__device__ __forceinline__ void swap_halves(uint32_t &a, uint32_t &b) {
    const uint32_t c = __builtin_amdgcn_update_dpp(a, b, 0x128, 0xf, 0xc, false);
    b = __builtin_amdgcn_update_dpp(b, a, 0x128, 0xf, 0x3, false);
    a = c;
}

// Eight codes -> eight bf16 values 24 + c in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 codes_to_bf16(uint32_t w) {
    constexpr uint32_t kField = 0x00780078u, kSixteen = 0x41c041c0u;   // 16.0 with the sign bit of the code flipped
    return make_uint4(((w << 3) & kField) ^ kSixteen, ((w >> 1) & kField) ^ kSixteen, ((w >> 5) & kField) ^ kSixteen,
                      ((w >> 9) & kField) ^ kSixteen);
}

// Lane 16 g + t holds four dwords; afterwards dword i of lane 16 g + t is dword g of lane 16 i + t.
__device__ __forceinline__ void transpose4(uint4 &v) {
    auto p = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
    auto q = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
    auto r = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
    auto s = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
    v = make_uint4(r[0], r[1], s[0], s[1]);
}

__device__ __forceinline__ uint32_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// A token takes as many columns as its parts (three: four, the last unused), so
// that its parts' sums meet in one lane.
constexpr int column_stride(int parts) { return parts == 3 ? 4 : parts; }

// Operands of blocks [b0, b0 + n) of x: xs[block][4][4][cols] of 16 bytes (element (i,
// g, c): k = 32 i + 8 g .. + 8 of the block, column c, in the order of
// codes_to_bf16) and starts[group][16 CT], -24 times each group's sum.  Called by
// whole waves, `step` threads in all, this one number tid of them.
template <int GROUP, int CT, int PARTS>
__device__ __forceinline__ void make_operands(const MatvecArgs &a, int cols, int b0, int n, int tid, int step, uint4 *xs,
                                              float *starts) {
    constexpr int kGroups = 128 / GROUP, kStride = column_stride(PARTS), kTokens = 16 / kStride;
    const int places = n * 16;   // 8 elements each, 16 to a block; a thread keeps its place and walks the tokens
    const int at_once = max(step / places, 1);
    constexpr int kAhead = 4;    // tokens loaded together
    for (int place = step >= places ? tid % places : tid; place < places; place += step >= places ? places : step) {
        const int j = place & 15, blk = place >> 4, tok0 = step >= places ? tid / places : 0;
        if (tok0 >= at_once) break;
        const uint16_t *from = static_cast<const uint16_t *>(a.x) + (size_t)(b0 + blk) * 128 + j * 8;
        for (int tok = tok0; tok < a.m; tok += kAhead * at_once) {
            uint4 q[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                q[u] = *reinterpret_cast<const uint4 *>(from + (size_t)min(tok + u * at_once, a.m - 1) * a.k);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int token = tok + u * at_once;
                if (token >= a.m) break;
                const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
                float v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] = a.x_type == kElemBf16 ? bf16lo(w[i]) : half_lo(w[i]);
                    v[2 * i + 1] = a.x_type == kElemBf16 ? bf16hi(w[i]) : half_hi(w[i]);
                }
                if (a.rotate) fwht128_lanes16(v, tid & 63);   // (the 16 lanes of a block take every branch here together)
                const int col = (token / kTokens) * 16 + (token % kTokens) * kStride;
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    uint32_t b[8];
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        b[i] = bf16_bits(v[i]);
                        const float h = __uint_as_float(b[i] << 16);
                        sum += h;
                        v[i] -= h;
                    }
#pragma unroll
                    for (int d = 1; d < GROUP / 8; d <<= 1) sum += shfl_xor_f(sum, d);
                    // (one group a block: codes as a lane loads them, its 32 in the four MFMAs)
                    const int to = GROUP == 128 ? (place & ~15) | (j & 3) << 2 | j >> 2 : place;
                    xs[to * cols + col + p] =
                        make_uint4(b[0] | (b[4] << 16), b[1] | (b[5] << 16), b[2] | (b[6] << 16), b[3] | (b[7] << 16));
                    if (j % (GROUP / 8) == 0) starts[(blk * kGroups + j / (GROUP / 8)) * (16 * CT) + col + p] = -24.0f * sum;
                }
            }
        }
    }
}

}  // namespace

// All operands of x into the workspace: xs of every block, then starts.
template <int GROUP, int CT, int PARTS>
__global__ __launch_bounds__(256) void k_matvec_x(MatvecArgs a, MatvecPlan plan) {
    const int blocks = a.k / 128;
    uint4 *xs = static_cast<uint4 *>(a.ws);
    make_operands<GROUP, CT, PARTS>(a, plan.cols, 0, blocks, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256, xs,
                                    reinterpret_cast<float *>(xs + (size_t)blocks * 16 * plan.cols));
}

// Waves of a workgroup, and waves a SIMD that the registers are cut for.  One
// column tile: two workgroups of 8 a CU.  Two: one of 16, as x fills LDS.  More need
// the registers of two waves a SIMD.  Where a wave keeps the sums of its head (the
// last blocks of a tile that others begin) until the end: in registers, and with more
// column tiles in LDS, behind x.
constexpr int waves_of(int ct) { return ct == 2 ? 16 : 8; }
constexpr int simd_waves(int ct) { return ct <= 2 ? 4 : 2; }
constexpr bool head_in_lds(int ct) { return ct > 2; }

// PARTS parts of x; CT tiles of 16 columns; LDS: x's operands (xs, then starts) are
// there.  The waves' sums take their place, or follow.
template <int GROUP, int CT, int PARTS, bool LDS>
__global__ __launch_bounds__(64 * waves_of(CT), simd_waves(CT)) void k_matvec(MatvecArgs a, MatvecPlan plan) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    constexpr int kWaves = waves_of(CT);
    constexpr int kGroups = 128 / GROUP, kPer = GROUP / 32;   // groups a block, MFMAs a group
    constexpr int kStride = column_stride(PARTS), kTokens = 16 / kStride;
    constexpr int kBatch = 2;   // blocks whose weights a wave loads at a time, two such batches in flight
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t = lane & 15, g = lane >> 4;
    const int blocks = a.k / 128;
    const int cols = CT == 1 ? plan.cols : 16 * CT;
    uint4 *xs = reinterpret_cast<uint4 *>(smem);
    float *starts = reinterpret_cast<float *>(smem + (size_t)blocks * 256 * cols);
    const uint4 *xw = static_cast<const uint4 *>(a.ws);
    const float *startsw = reinterpret_cast<const float *>(xw + (size_t)blocks * 16 * cols);

    // tiles [tile0, tile1) of this workgroup; of their blocks in a row this wave's [begin, end)
    const int block0 = (int)blockIdx.x, tile0 = block0 * plan.run + min(block0, plan.more);
    const int all = (plan.run + (block0 < plan.more)) * blocks;
    // at / blocks, at <= 2^21 (at most 2^12 tiles of 2^9 blocks), by a product
    auto tile_of = [&](int at) { return blocks == 1 ? at : (int)__umulhi((uint32_t)at, plan.inv); };
    auto part = [&](int w) {   // from even blocks of a tile on
        const int at = (int)((uint32_t)(all * w) / kWaves);
        return at - ((at - tile_of(at) * blocks) & 1);
    };
    const int begin = __builtin_amdgcn_readfirstlane(part(wave)), end = __builtin_amdgcn_readfirstlane(part(wave + 1));

    // A batch: n blocks from block b of a tile.
    struct Place {
        int tile, b, n, left;   // left: this wave's blocks from here on
    };
    auto fill = [&](Place &p) { p.n = min(min(kBatch, blocks - p.b), p.left); };
    auto next = [&](Place &p) {
        p.left -= p.n;
        p.b += p.n;
        if (p.b == blocks) p.b = 0, ++p.tile;
        fill(p);
    };
    // Scales come for kWindow batches at a time, those of batch i of a window in the
    // lanes of g = i; the other batches' loads are out of range, which keeps the
    // count of loads the same for every batch.  Group size 128: where rows of an odd
    // number of blocks or the tensor's start are aligned to 2 bytes only, the second
    // scale of a batch is loaded apart.
    constexpr int kWords = kBatch * kGroups / 2, kWindow = 4;
    const bool even = !(blocks & 1) && (reinterpret_cast<uintptr_t>(a.scales) & 3) == 0;
    struct Batch {
        uint4 codes[kBatch];
        uint32_t scales[kWords], odd;
    };
    // A batch's codes are 128 bytes of each of 16 rows, loaded as whole lines of 8 rows
    // at a time (loads alone, one token, 150144 x 2048: 29 us, and 34 with 64 bytes of 16
    // rows); swap_halves gives each lane its row's.
    // Rows behind the last are out of the buffers' range and read as zeros.
    const uint32_t code_pitch = (uint32_t)a.k / 2, scale_pitch = (uint32_t)a.k / GROUP * 2;
    const uint32_t code_at = (t & 7) * code_pitch + 16 * (g + (t >> 3) * 4), scale_at = t * scale_pitch + g * (4 * kWords);
    auto new_window = [&](const Place &p) { return p.b % (kBatch * kWindow) == 0 || p.left == end - begin; };
    auto load = [&](Batch &w, const Place &p) {
        const int64_t row = (int64_t)p.tile * 16;
        const uint32_t left = p.left > 0 ? (uint32_t)min(16, a.n - (int)row) : 0u;   // nothing is read behind the last
        const __amdgpu_buffer_rsrc_t codes = make_buf(a.codes + row * code_pitch, left * code_pitch);
        const __amdgpu_buffer_rsrc_t scales = make_buf(reinterpret_cast<const uint8_t *>(a.scales) + row * scale_pitch, left * scale_pitch);
        const uint32_t at = scale_at + p.b / (kBatch * kWindow) * (kWindow * 4 * kWords) + (new_window(p) ? 0u : 0x80000000u);
        if constexpr (GROUP == 32) {
            const uint4 q = bload16(scales, at, 0);
            w.scales[0] = q.x, w.scales[1] = q.y, w.scales[2] = q.z, w.scales[3] = q.w;
        } else if constexpr (GROUP == 64) {
            const uint2 q = bload8(scales, at);
            w.scales[0] = q.x, w.scales[1] = q.y;
        } else if (even) {
            w.scales[0] = bload4(scales, at, 0);
        } else {
            w.scales[0] = bload2(scales, at, 0);
            w.odd = bload2(scales, at + 2, 0);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) w.codes[u] = bload16_nt(codes, code_at + u * 8 * code_pitch + p.b * 64, 0);
    };

    constexpr bool kHeadLds = head_in_lds(CT);
    f32x4_t *red = reinterpret_cast<f32x4_t *>(kHeadLds && LDS ? smem + (size_t)blocks * (256 * cols + kGroups * 64 * CT) : smem);
    f32x4_t sum[CT], head[kHeadLds ? 1 : CT];   // of the tile at hand; of the head
#pragma unroll
    for (int c = 0; c < CT; ++c) sum[c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const int first = tile_of(begin), begin_at = begin - first * blocks;   // tile and block where this wave begins
    const bool has_head = begin < end && begin_at != 0;
    // Operands of x that come through the caches are loaded before the next weights, as
    // loads return in order (64 tokens, 12288 x 6144: 43 us, and 62 when they are loaded
    // at the products; more column tiles have no registers for it)
    constexpr bool kFetch = !LDS && CT <= 4;
    uint4 ahead[kFetch ? kBatch : 1][kFetch ? CT : 1][kFetch ? 4 : 1];
    uint32_t window[kWords], window_odd = 0, scales[kWords], odd = 0;
    auto block = [&](Batch &w, int u, int b) {
        if constexpr (GROUP != 128) transpose4(w.codes[u]);
        const uint32_t wd[4] = {w.codes[u].x, w.codes[u].y, w.codes[u].z, w.codes[u].w};
        const int at = (b * 16 + g) * cols + (CT == 1 ? min(t, cols - 1) : t);
        const int st = b * kGroups * (16 * CT) + 4 * g;
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr) {
            const int i = u * kGroups + gr;
            float s = (i & 1) ? bf16hi(scales[i >> 1]) : bf16lo(scales[i >> 1]);
            if (GROUP == 128 && u == 1 && !even) s = bf16lo(odd);
            uint4 q[kPer];
#pragma unroll
            for (int k = 0; k < kPer; ++k) q[k] = codes_to_bf16(wd[gr * kPer + k]);
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                f32x4_t acc = *reinterpret_cast<const f32x4_t *>((LDS ? starts : startsw) + st + (gr * CT + c) * 16);
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    const int i = gr * kPer + k;
                    acc = mfma16(kFetch ? ahead[kFetch ? u : 0][kFetch ? c : 0][kFetch ? i : 0]
                                        : (LDS ? xs : xw)[at + i * 4 * cols + c * 16], q[k], acc);
                }
                sum[c] += s * acc;
            }
        }
    };
    auto fetch = [&](const Place &p) {
        if constexpr (kFetch) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        ahead[u][c][i] = xw[(min(p.b + u, blocks - 1) * 16 + g + 4 * i) * cols + (CT == 1 ? min(t, cols - 1) : t) + c * 16];
        }
    };
    auto store = [&](int tile) {   // element i of sum[c] is column 16 c + 4 g + i of row t
        const int row = tile * 16 + t;
        if (row >= a.n) return;
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int i = 0; i < 4; i += kStride) {
                const int token = c * kTokens + (4 * g + i) / kStride;
                if (token >= a.m) continue;
                float v = sum[c][i];
                if (PARTS > 1) v += sum[c][i + 1];
                if (PARTS > 2) v += sum[c][i + 2];
                const size_t o = (size_t)token * a.n + row;
                if (a.y_type == kElemF32) static_cast<float *>(a.y)[o] = v;
                else if (a.y_type == kElemF16) static_cast<_Float16 *>(a.y)[o] = (_Float16)v;
                else static_cast<uint16_t *>(a.y)[o] = (uint16_t)bf16_bits(v);
            }
    };
    auto compute = [&](Batch &w, const Place &p) {
        swap_halves(w.codes[0].x, w.codes[1].x);
        swap_halves(w.codes[0].y, w.codes[1].y);
        swap_halves(w.codes[0].z, w.codes[1].z);
        swap_halves(w.codes[0].w, w.codes[1].w);
        const bool fresh = new_window(p);
        const int from = (t + 16 * (p.b / kBatch % kWindow)) * 4;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            window[i] = fresh ? w.scales[i] : window[i];
            scales[i] = __builtin_amdgcn_ds_bpermute(from, window[i]);
        }
        if (GROUP == 128 && !even) {
            window_odd = fresh ? w.odd : window_odd;
            odd = __builtin_amdgcn_ds_bpermute(from, window_odd);
        }
        if (p.n == kBatch) {   // no branch between the blocks: their loads and products overlap
#pragma unroll
            for (int u = 0; u < kBatch; ++u) block(w, u, p.b + u);
        } else {
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (u < p.n) block(w, u, p.b + u);
        }
        if (p.b + p.n < blocks) return;
        // the tile's last block: it is whole, or (the first one) the head
        const bool is_head = has_head && p.tile == tile0 + first;
        if (!is_head) store(p.tile);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            if (is_head) {
                if constexpr (kHeadLds) red[(wave * CT + c) * 64 + lane] = sum[c];
                else head[c] = sum[c];
            }
            sum[c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
    };

    // products one batch behind the loads
    Place p{tile0 + first, begin_at, 0, end - begin};
    fill(p);
    Batch w0, w1;
    load(w0, p);
    if constexpr (LDS) {
        make_operands<GROUP, CT, PARTS>(a, cols, 0, blocks, tid, 64 * kWaves, xs, starts);
        __syncthreads();
    }
    while (p.left > 0) {
        Place p1 = p;
        next(p1);
        fetch(p);
        load(w1, p1);
        compute(w0, p);
        if (p1.left <= 0) break;
        p = p1;
        next(p);
        fetch(p1);
        load(w0, p);
        compute(w1, p1);
    }

    // Tiles that several waves share: the wave with the first blocks adds the others' sums.
    const int last = tile_of(max(end - 1, 0));
    const bool middle = has_head && first == last && end != (last + 1) * blocks;   // neither end is this wave's
    const bool has_tail = begin < end && end != (last + 1) * blocks && !middle;
    if (!kHeadLds) __syncthreads();   // the sums take the place of x
    if (has_head && (middle || !kHeadLds)) {
#pragma unroll
        for (int c = 0; c < CT; ++c) red[(wave * CT + c) * 64 + lane] = middle || kHeadLds ? sum[c] : head[kHeadLds ? 0 : c];
    }
    __syncthreads();
    if (has_tail) {
        const int stop = (last + 1) * blocks;
        for (int w = wave + 1; w < kWaves && part(w) < stop; ++w) {
            if (part(w) == part(w + 1)) continue;   // no blocks
#pragma unroll
            for (int c = 0; c < CT; ++c) sum[c] += red[(w * CT + c) * 64 + lane];
        }
        store(tile0 + last);
    }
}

// bf16 columns that hold one value of x.
static int x_parts(const MatvecArgs &a) {
    if (a.rotate) return a.y_type == kElemF32 ? 3 : 2;
    return a.x_type == kElemBf16 ? 1 : 2;
}

// Column tiles of m tokens of `parts` parts: 1, 2, 4, 8 or 16.
static int column_tiles(int m, int parts) {
    const int tokens = 16 / column_stride(parts), want = (m + tokens - 1) / tokens;
    return want <= 1 ? 1 : want <= 2 ? 2 : want <= 4 ? 4 : want <= 8 ? 8 : 16;
}

// Room for all operands of m tokens of three parts (a block: 16 columns of 256 bytes,
// and the starts of its four groups, a column tile).
size_t matvec_workspace_bytes(int m, int k) { return (size_t)(k / 128) * column_tiles(m, 3) * (16 * 256 + 4 * 64) + 256; }

// Bytes of the operands of m tokens, and whether they fit LDS (with the waves' heads).
static int64_t x_bytes(const MatvecArgs &a, int m, int parts) {
    const int ct = column_tiles(m, parts), cols = ct == 1 ? m * column_stride(parts) : 16 * ct;
    return (int64_t)(a.k / 128) * (256 * cols + (128 / a.group) * 64 * ct);
}
static bool x_fits(const MatvecArgs &a, int m, int parts) {
    const int ct = column_tiles(m, parts);
    return x_bytes(a, m, parts) + (head_in_lds(ct) ? waves_of(ct) * ct * 1024 : 0) <= kLdsBytes;
}

void launch_matvec(const MatvecArgs &a, hipStream_t s) {
    const int parts = x_parts(a), ct = column_tiles(a.m, parts);
    const bool in_lds = x_fits(a, a.m, parts);
    // In two halves, which read the weights twice:
    //   sixteen column tiles, and eight of group size 32 without LDS: their sums would
    //   spill (64 rotated tokens to fp32, 12288 x 2048: 54 us against 127; 64 rotated
    //   fp16 tokens, 2048 x 2048, group size 32: 23 against 37, but 128: 41 against 29);
    //   operands that only fit LDS so, and many rows to read them for (64 tokens,
    //   150144 x 2048: 92 us against 186 with x read through the caches; 16 tokens, 2048
    //   x 6144: 27 us against 10)
    const int half = (a.m + 1) / 2;
    if (ct == 16 || (!in_lds && ((ct == 8 && a.group == 32) || (a.n >= 32768 && x_fits(a, half, parts))))) {
        MatvecArgs h = a;
        h.m = half;
        launch_matvec(h, s);
        if (hipPeekAtLastError() != hipSuccess) return;
        h.m = a.m - half;
        h.x = static_cast<const uint16_t *>(a.x) + (size_t)half * a.k;
        h.y = static_cast<uint8_t *>(a.y) + (size_t)half * a.n * (a.y_type == kElemF32 ? 4 : 2);
        launch_matvec(h, s);
        return;
    }
    MatvecPlan p;
    p.cols = ct == 1 ? a.m * column_stride(parts) : 16 * ct;
    p.tiles = (a.n + 15) / 16;
    const int blocks = a.k / 128, waves = waves_of(ct), join = waves * ct * 1024, x = in_lds ? (int)x_bytes(a, a.m, parts) : 0;
    const int lds = head_in_lds(ct) ? x + join : x > join ? x : join;
    // two workgroups of one column tile a CU, if no tile more falls to a CU so
    const int one = (p.tiles + 255) / 256, two = 2 * ((p.tiles + 511) / 512);
    const int slots = ct == 1 && kLdsBytes / lds >= 2 && (two <= one || one > 8) ? 512 : 256;
    const unsigned grid = (unsigned)(p.tiles < slots ? p.tiles : slots);
    p.run = p.tiles / (int)grid;
    p.more = p.tiles % (int)grid;
    p.inv = (uint32_t)(((1ull << 32) + blocks - 1) / blocks);
    auto go = [&](auto G, auto C, auto P) {
        if constexpr (C() < 8 || G() > 32) {
            if (!in_lds) {
                hipLaunchKernelGGL((k_matvec_x<G(), C(), P()>), dim3((unsigned)((a.m * blocks + 15) / 16)), dim3(256), 0, s, a, p);
                if (hipPeekAtLastError() != hipSuccess) return;
                hipLaunchKernelGGL((k_matvec<G(), C(), P(), false>), dim3(grid), dim3(64 * waves), lds, s, a, p);
                return;
            }
        }
        hipLaunchKernelGGL((k_matvec<G(), C(), P(), true>), dim3(grid), dim3(64 * waves), lds, s, a, p);
    };
    auto by_parts = [&](auto G, auto C) {   // (eight column tiles: only two and three parts need so many)
        if constexpr (C() < 8) {
            if (parts == 1) return go(G, C, std::integral_constant<int, 1>{});
        }
        if (parts == 2) go(G, C, std::integral_constant<int, 2>{});
        else go(G, C, std::integral_constant<int, 3>{});
    };
    auto by_tiles = [&](auto G) {
        if (ct == 1) by_parts(G, std::integral_constant<int, 1>{});
        else if (ct == 2) by_parts(G, std::integral_constant<int, 2>{});
        else if (ct == 4) by_parts(G, std::integral_constant<int, 4>{});
        else by_parts(G, std::integral_constant<int, 8>{});
    };
    if (a.group == 32) by_tiles(std::integral_constant<int, 32>{});
    else if (a.group == 64) by_tiles(std::integral_constant<int, 64>{});
    else by_tiles(std::integral_constant<int, 128>{});
}

}  // namespace moe_w4

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
// off by starting each group's sums at x times a constant -24 operand.  x enters
// as 1 to 3 bf16 columns that add up to it (bf16 is itself; fp16 and rotated
// values are two, 16 bits, or three, 24 bits, for fp32 results), so every
// product is exact and only the fp32 sums round.
#include "common.h"
#include "launch.h"

namespace moe_w4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

// Eight codes -> eight bf16 values 24 + c in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 codes_to_bf16(uint32_t w) {
    constexpr uint32_t kField = 0x00780078u, kSixteen = 0x41c041c0u;   // 16.0 with the sign bit of the code flipped
    return make_uint4(((w << 3) & kField) ^ kSixteen, ((w >> 1) & kField) ^ kSixteen, ((w >> 5) & kField) ^ kSixteen,
                      ((w >> 9) & kField) ^ kSixteen);
}
constexpr uint32_t kMinus24 = 0xc1c0c1c0u;   // two bf16 -24

// Lane 16 g + t holds four dwords; afterwards dword i of lane 16 g + t is dword g of lane 16 i + t.
__device__ __forceinline__ void transpose4(uint4 &v) {
    auto p = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
    auto q = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
    auto r = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
    auto s = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
    v = make_uint4(r[0], r[1], s[0], s[1]);
}

__device__ __forceinline__ uint32_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// Columns of x: tile c / 16 of kTile = 16 / parts tokens.
constexpr int tokens_per_tile(int parts) { return 16 / parts; }

}  // namespace

// x -> MFMA operands in ws: [column tile][k / 32][lane][8 bf16], lane 16 g + c
// holding k = 32 i + 8 g .. + 8 of column c in the order of codes_to_bf16.  16
// lanes a 128-block of a token.
template <bool BF16, int PARTS>
__global__ __launch_bounds__(256) void k_matvec_x(const uint16_t *__restrict__ x, int m, int k, bool rotate, uint4 *ws) {
    const int blocks = k / 128;
    const int item = blockIdx.x * 16 + (threadIdx.x >> 4), j = threadIdx.x & 15;
    const bool live = item < m * blocks;
    const int tok = live ? item / blocks : 0, blk = live ? item % blocks : 0;
    const uint4 q = *reinterpret_cast<const uint4 *>(x + (size_t)tok * k + blk * 128 + j * 8);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = BF16 ? bf16lo(w[i]) : half_lo(w[i]);
        v[2 * i + 1] = BF16 ? bf16hi(w[i]) : half_hi(w[i]);
    }
    if (rotate) fwht128_lanes16(v, threadIdx.x & 63);
    if (!live) return;
    constexpr int kTokens = tokens_per_tile(PARTS);
    const int tile = tok / kTokens, c = (tok % kTokens) * PARTS;
    uint4 *out = ws + ((size_t)tile * (k / 32) + blk * 4 + j / 4) * 64 + (j & 3) * 16 + c;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        uint32_t b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            b[i] = bf16_bits(v[i]);
            v[i] -= __uint_as_float(b[i] << 16);
        }
        out[p] = make_uint4(b[0] | (b[4] << 16), b[1] | (b[5] << 16), b[2] | (b[6] << 16), b[3] | (b[7] << 16));
    }
}

// 16 weight rows and CT column tiles a workgroup, its WAVES waves taking every
// WAVES-th 128-block of K; their sums are added in order through LDS.
template <int GROUP, int CT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_matvec(MatvecArgs a, int parts, int tiles) {
    __shared__ f32x4_t red[WAVES][CT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, ct0 = blockIdx.y * CT;
    const int blocks = a.k / 128, chunks = a.k / 32;
    constexpr int kGroups = 128 / GROUP, kPer = GROUP / 32;
    const int row = min(n0 + t, a.n - 1);   // rows behind the last are computed and not stored
    const uint4 *codes = reinterpret_cast<const uint4 *>(a.codes + (size_t)row * (a.k / 2)) + g;
    const uint16_t *scales = a.scales + (size_t)row * (a.k / GROUP);
    const uint4 *xf[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
        xf[c] = static_cast<const uint4 *>(a.ws) + (size_t)min(ct0 + c, tiles - 1) * chunks * 64 + lane;
    f32x4_t sum[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) sum[c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = wave; b < blocks; b += WAVES) {
        uint4 w = codes[b * 4];
        transpose4(w);
        const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr) {
            const float s = bf16_to_f32(scales[b * kGroups + gr]);
            uint4 q[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) q[i] = codes_to_bf16(wd[gr * kPer + i]);
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
                uint4 xv[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    xv[i] = xf[c][(size_t)(b * 4 + gr * kPer + i) * 64];
                    acc = mfma16(xv[i], make_uint4(kMinus24, kMinus24, kMinus24, kMinus24), acc);
                }
#pragma unroll
                for (int i = 0; i < kPer; ++i) acc = mfma16(xv[i], q[i], acc);
                sum[c] += s * acc;
            }
        }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) red[wave][c][lane] = sum[c];
    __syncthreads();
    // column 4 g + i of row t is element i of lane 16 g + t
    const int per_tile = 16 / parts;
    for (int o = threadIdx.x; o < CT * per_tile * 16; o += 64 * WAVES) {
        const int r = o & 15, tok = o >> 4, c = tok / per_tile, col = (tok % per_tile) * parts;
        const int token = (ct0 + c) * per_tile + tok % per_tile;
        if (n0 + r >= a.n || token >= a.m) continue;
        float v = 0.0f;
        for (int p = 0; p < parts; ++p)
            for (int wv = 0; wv < WAVES; ++wv) v += red[wv][c][((col + p) >> 2) * 16 + r][(col + p) & 3];
        const size_t at = (size_t)token * a.n + n0 + r;
        if (a.y_type == kElemF32) static_cast<float *>(a.y)[at] = v;
        else if (a.y_type == kElemF16) static_cast<_Float16 *>(a.y)[at] = (_Float16)v;
        else static_cast<uint16_t *>(a.y)[at] = (uint16_t)bf16_bits(v);
    }
}

// bf16 columns that hold one value of x.
static int x_parts(const MatvecArgs &a) {
    if (a.rotate) return a.y_type == kElemF32 ? 3 : 2;
    return a.x_type == kElemBf16 ? 1 : 2;
}

size_t matvec_workspace_bytes(int m, int k) {
    const int per = tokens_per_tile(3);
    return (size_t)((m + per - 1) / per) * (size_t)k * 32 + 256;
}

template <int GROUP>
static void launch_group(const MatvecArgs &a, int parts, int tiles, hipStream_t s) {
    const unsigned gx = (unsigned)((a.n + 15) / 16);
    if (tiles == 1)
        hipLaunchKernelGGL((k_matvec<GROUP, 1, 4>), dim3(gx, 1), dim3(256), 0, s, a, parts, tiles);
    else if (tiles == 2)
        hipLaunchKernelGGL((k_matvec<GROUP, 2, 4>), dim3(gx, 1), dim3(256), 0, s, a, parts, tiles);
    else
        hipLaunchKernelGGL((k_matvec<GROUP, 4, 4>), dim3(gx, (tiles + 3) / 4), dim3(256), 0, s, a, parts, tiles);
}

void launch_matvec(const MatvecArgs &a, hipStream_t s) {
    const int parts = x_parts(a), per = tokens_per_tile(parts), tiles = (a.m + per - 1) / per;
    const dim3 grid((unsigned)((a.m * (a.k / 128) + 15) / 16));
    const uint16_t *x = static_cast<const uint16_t *>(a.x);
    uint4 *ws = static_cast<uint4 *>(a.ws);
    const bool b = a.x_type == kElemBf16;
    if (parts == 1) hipLaunchKernelGGL((k_matvec_x<true, 1>), grid, dim3(256), 0, s, x, a.m, a.k, a.rotate, ws);
    else if (parts == 2 && b) hipLaunchKernelGGL((k_matvec_x<true, 2>), grid, dim3(256), 0, s, x, a.m, a.k, a.rotate, ws);
    else if (parts == 2) hipLaunchKernelGGL((k_matvec_x<false, 2>), grid, dim3(256), 0, s, x, a.m, a.k, a.rotate, ws);
    else if (b) hipLaunchKernelGGL((k_matvec_x<true, 3>), grid, dim3(256), 0, s, x, a.m, a.k, a.rotate, ws);
    else hipLaunchKernelGGL((k_matvec_x<false, 3>), grid, dim3(256), 0, s, x, a.m, a.k, a.rotate, ws);
    if (hipPeekAtLastError() != hipSuccess) return;
    if (a.group == 32) launch_group<32>(a, parts, tiles, s);
    else if (a.group == 64) launch_group<64>(a, parts, tiles, s);
    else launch_group<128>(a, parts, tiles, s);
}

}  // namespace moe_w4

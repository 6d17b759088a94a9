// Matrix products grouped by expert with ragged row counts, in bf16 or fp16
// with fp32 sums (moe_w4_grouped_mm, _dx, _dw):
//   mm:  y[r][n]     = sum_k x[r][k]  w[e][n][k]
//   dx:  dx[r][k]    = sum_n dy[r][n] w[e][n][k]
//   dw:  dw[e][n][k] = add[e][n][k] + sum_r dy[r][n] x[r][k]
// for the rows offsets[e] <= r < offsets[e + 1] of group e.
//
// One tile kernel serves the three: out[m][c] = sum_l A(m, l) B(c, l), where an
// operand is either "K-major" (l contiguous in memory: x and w of mm, dy of
// dx) or "MN-major" (its m or c contiguous, one row per l: w of dx, dy and x
// of dw).  l advances kStep = 64 a step.  Both kinds go from global memory to
// LDS with 16-byte buffer loads that bypass the registers, STAGES - 1 steps
// ahead; a K-major fragment of v_mfma_f32_16x16x32 is one 16-byte LDS read, an
// MN-major one two transposing 8-byte LDS reads (ds_read_b64_tr_b16: in each
// group of 16 lanes, lane t receives element t of 4 rows of 16 elements).
//
// Edges need no branches in the loop: the descriptor of each load ends with
// the group's (or the expert's) last row, and lanes past the contiguous
// extent aim past every descriptor; the hardware's range check makes both
// zeros in LDS.  Descriptors of MN-major operands move with l, so offsets
// stay small whatever the tensors' sizes are.
#include "common.h"
#include "launch.h"

namespace moe_w4 {

struct GroupedArgs {
    const uint8_t *a, *b;     // mm: x, w; dx: dy, w; dw: dy, x
    const int *offsets;
    void *out;
    const void *add;          // dw: added to the sums, or null
    int groups, rows;
    int n, k;
};

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
typedef __attribute__((address_space(3))) s16x8_t lds_s16x8;

constexpr int kStep = 64;                  // contraction elements per step
constexpr uint32_t kPast = 0x80000000u;    // a byte offset behind every descriptor (their sizes stay below 2^31)
constexpr int kXcd = 8;

enum { kMm = 0, kDx = 1, kDw = 2 };

template <bool BF16>
__device__ __forceinline__ f32x4_t mfma16(s16x8_t a, s16x8_t b, f32x4_t c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                       c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                      0, 0, 0);
}

template <bool BF16>
__device__ __forceinline__ uint16_t round16(float v) {
    if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);   // round to nearest even
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}
template <bool BF16>
__device__ __forceinline__ float widen16(uint16_t v) {
    if constexpr (BF16) return bf16_to_f32(v);
    return (float)__builtin_bit_cast(_Float16, v);
}

// 16 bytes a lane from a buffer straight to LDS (lane i's to lds + 16 i; lanes out of the buffer's range write zeros).
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, lds_u8 *lds, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds, 16, off, 0, 0, 0);
}
__device__ __forceinline__ s16x4_t read_transposed(const lds_u8 *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
}

// Where the operand tile of one matrix comes from: base of its first row, the
// pitch of its rows and the number of rows and of contiguous elements.
struct Operand {
    const uint8_t *base;
    uint32_t pitch;   // bytes
    int rows;         // K-major: m or c left in the tile; MN-major: l left
    int cols;         // K-major: l; MN-major: m or c left, from the tile's first
};

// LDS image of one operand tile of one step: R m- or c-positions x 64 l.
//   K-major:  row r of 128 bytes; 16-byte chunk q at slot q ^ ((r >> 1) & 7), so
//             the reads of one chunk by 16 consecutive rows hit all 64 banks.
//   MN-major: row l of 2R bytes; chunk q at slot q ^ (2 h(l)),
//             h = (l & 3) | (l >> 1 & 4): the 16 rows that a transposing read
//             takes 32 bytes of spread over 8 slots of 32 bytes.
template <int R, bool MN, int NT>
struct Tile {
    static constexpr int kBytes = R * kStep * 2;
    static constexpr int kLoads = kBytes / (16 * NT);
    static constexpr int kChunks = MN ? R / 8 : kStep / 8;      // per LDS row
    static_assert(kBytes % (16 * NT) == 0, "whole loads");
    uint32_t off[kLoads];   // byte offset of each of this thread's loads at l = 0
    int chunk;              // K-major: the first l / 8 of this thread's loads

    // Per thread load i: LDS bytes [16 (tid + NT i), +16) of the tile.
    __device__ __forceinline__ void init(const Operand &o, int tid) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int p = tid + NT * i, row = p / kChunks, slot = p % kChunks;
            if constexpr (MN) {
                const int h = (row & 3) | ((row >> 1) & 4);
                const int q = slot ^ (2 * h & (kChunks - 1));
                off[i] = 8 * q < o.cols ? (uint32_t)row * o.pitch + 16 * q : kPast;
            } else {
                const int q = slot ^ ((row >> 1) & 7);
                off[i] = row < o.rows ? (uint32_t)row * o.pitch + 16 * q : kPast;
                chunk = q;   // NT is a multiple of 16 rows: the same for every i
            }
        }
    }

    // Starts the loads of step s into the image at lds.
    __device__ __forceinline__ void load(const Operand &o, int s, lds_u8 *lds, int wave) const {
        const int l = s * kStep;
        if constexpr (MN) {
            const int left = o.rows - l;
            const uint32_t bytes = left <= 0 ? 0u : (uint32_t)min(left, kStep) * o.pitch;
            const __amdgpu_buffer_rsrc_t r = make_buf(o.base + (size_t)l * o.pitch, bytes);
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                load_to_lds(r, lds + 16 * (NT * i + 64 * wave), off[i]);
        } else {
            const __amdgpu_buffer_rsrc_t r = make_buf(o.base, (uint32_t)o.rows * o.pitch);
            const bool in = l + 8 * chunk < o.cols;
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                load_to_lds(r, lds + 16 * (NT * i + 64 * wave), in ? off[i] + 2u * l : kPast);
        }
    }

    // Fragment of 16 m (or c) from position p0 and 32 l from 32 kk: lane t + 16 g holds
    // position p0 + t, l = 32 kk + 8 g .. + 8.
    static __device__ __forceinline__ s16x8_t frag(const lds_u8 *lds, int p0, int kk, int lane) {
        const int t = lane & 15, g = lane >> 4;
        if constexpr (MN) {
            const int h = (t >> 2) | ((g & 1) << 2);
            const int row = 32 * kk + 8 * g + (t >> 2);
            const int q = (p0 / 8 + ((t & 3) >> 1)) ^ (2 * h & (kChunks - 1));
            const lds_u8 *a = lds + row * (2 * R) + q * 16 + (t & 1) * 8;
            const s16x4_t lo = read_transposed(a);
            const s16x4_t hi = read_transposed(a + 4 * (2 * R));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            const int row = p0 + t;
            const int q = (4 * kk + g) ^ ((row >> 1) & 7);
            return *(const lds_s16x8 *)(lds + row * 128 + q * 16);
        }
    }
};

// Finds m tile `want` among the groups' tiles (ceil(count / BM) each, groups in
// order): {group, first row, rows of the tile, ...}.  Every thread calls it.
// Offsets are clamped to [0, rows] and to their predecessor, so that no tile
// leaves the arrays whatever they hold.
struct TileOf {
    int group, row, count, total;
};
template <int BM, int NT>
__device__ __forceinline__ TileOf find_tile(const int *__restrict__ offsets, int groups, int rows, int want_in, int tiles_n,
                                            int *sh) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (groups + NT - 1) / NT;
    const int e0 = min(tid * per, groups), e1 = min(e0 + per, groups);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        const int lo = min(max(offsets[e], 0), rows), hi = min(max(offsets[e + 1], lo), rows);
        sum += (hi - lo + BM - 1) / BM;
    }
    int pre = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(pre, d, 64);
        if (lane >= d) pre += v;
    }
    if (lane == 63) sh[wave] = pre;
    if (tid == 0) sh[NT / 64 + 0] = -1;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        const int v = sh[w];
        if (w < wave) base += v;
        total += v;
    }
    pre += base - sum;   // tiles before this thread's groups
    // XCD b % 8 takes a contiguous run of the tiles (row tiles outer, column
    // tiles inner), so that the tiles that share rows or weights share an L2
    const int all = total * tiles_n, run = (all + kXcd - 1) / kXcd;
    const int t = (want_in % kXcd) * run + want_in / kXcd;
    const bool none = want_in / kXcd >= run || t >= all;
    const int want = t / tiles_n;
    if (!none && want >= pre && want < pre + sum) {
        int at = pre;
        for (int e = e0; e < e1; ++e) {
            const int lo = min(max(offsets[e], 0), rows), hi = min(max(offsets[e + 1], lo), rows);
            const int c = (hi - lo + BM - 1) / BM;
            if (want < at + c) {
                const int r = lo + (want - at) * BM;
                sh[NT / 64 + 0] = e;
                sh[NT / 64 + 1] = r;
                sh[NT / 64 + 2] = min(hi - r, BM);
                break;
            }
            at += c;
        }
    }
    __syncthreads();
    TileOf o;
    o.group = __builtin_amdgcn_readfirstlane(sh[NT / 64 + 0]);
    o.row = __builtin_amdgcn_readfirstlane(sh[NT / 64 + 1]);
    o.count = __builtin_amdgcn_readfirstlane(sh[NT / 64 + 2]);
    o.total = t % tiles_n;   // the column tile
    return o;
}

template <int N>
__device__ __forceinline__ void wait_vm() {   // at most N vector memory operations of this wave outstanding, no LDS read
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}
__device__ __forceinline__ void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace

// One BM x BN tile by WM x WN waves.
template <int MODE, bool BF16, bool F32OUT, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(64 * WM *WN) void k_grouped_mm(GroupedArgs g) {
    constexpr int NT = 64 * WM * WN;
    constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
    typedef Tile<BM, MODE == kDw, NT> TA;
    typedef Tile<BN, MODE != kMm, NT> TB;
    constexpr int kStageBytes = TA::kBytes + TB::kBytes;
    constexpr int kLoads = TA::kLoads + TB::kLoads;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * kStageBytes];
    lds_u8 *lds = (lds_u8 *)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;

    Operand A, B;
    int group, row0, mcount, c0, ccount, len;
    const int C = MODE == kMm ? g.n : g.k;   // columns of the output
    if constexpr (MODE == kDw) {
        const int tn = (g.k + BN - 1) / BN;
        group = blockIdx.y;
        row0 = (blockIdx.x / tn) * BM;
        c0 = (blockIdx.x % tn) * BN;
        mcount = min(g.n - row0, BM);
        const int lo = min(max(g.offsets[group], 0), g.rows), hi = min(max(g.offsets[group + 1], lo), g.rows);
        len = hi - lo;
        A.pitch = 2u * g.n;
        A.base = g.a + (size_t)lo * A.pitch + 2 * (size_t)row0;
        A.cols = mcount;
        A.rows = len;
        B.pitch = 2u * g.k;
        B.base = g.b + (size_t)lo * B.pitch + 2 * (size_t)c0;
        B.rows = len;
    } else {
        const TileOf t = find_tile<BM, NT>(g.offsets, g.groups, g.rows, blockIdx.x, (C + BN - 1) / BN,
                                           reinterpret_cast<int *>(smem));
        if (t.group < 0) return;
        __syncthreads();   // smem is the tiles' from here on
        group = t.group;
        row0 = t.row;
        mcount = t.count;
        c0 = t.total * BN;
        len = MODE == kMm ? g.k : g.n;
        A.pitch = 2u * len;
        A.base = g.a + (size_t)row0 * A.pitch;
        A.rows = mcount;
        A.cols = len;
        const uint8_t *w = g.b + (size_t)group * g.n * g.k * 2;
        B.pitch = 2u * g.k;
        if constexpr (MODE == kMm) {
            B.base = w + (size_t)c0 * B.pitch;
            B.rows = min(C - c0, BN);
            B.cols = len;
        } else {
            B.base = w + 2 * (size_t)c0;
            B.rows = len;
        }
    }
    ccount = min(C - c0, BN);
    if constexpr (MODE != kMm) B.cols = ccount;

    TA ta;
    TB tb;
    ta.init(A, tid);
    tb.init(B, tid);
    const int steps = (len + kStep - 1) / kStep;

    f32x4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

    auto issue = [&](int s, int slot) {
        ta.load(A, s, lds + slot * kStageBytes, wave);
        tb.load(B, s, lds + slot * kStageBytes + TA::kBytes, wave);
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) issue(s, s);
    int slot = 0, fill = STAGES - 1;
    for (int s = 0; s < steps; ++s) {
        // step s has arrived for this wave (STAGES - 2 later ones may be in
        // flight); behind the barrier it has for all, and all have read step
        // s - 1, whose slot the loads issued next overwrite.  Loads behind the
        // last step read nothing (every lane out of range)
        wait_vm<(STAGES - 2) * kLoads>();
        barrier();
        issue(s + STAGES - 1, fill);
        const lds_u8 *la = lds + slot * kStageBytes, *lb = la + TA::kBytes;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            s16x8_t fa[FM], fb[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) fa[i] = TA::frag(la, wm * TM + 16 * i, kk, lane);
#pragma unroll
            for (int j = 0; j < FN; ++j) fb[j] = TB::frag(lb, wn * TN + 16 * j, kk, lane);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<BF16>(fb[j], fa[i], acc[i][j]);
        }
        if (++slot == STAGES) slot = 0;
        if (++fill == STAGES) fill = 0;
    }
    wait_vm<0>();

    // lane t + 16 g holds out row t, columns 4 g .. + 4 of each 16 x 16 tile
    const int t = lane & 15, q = lane >> 4;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = wm * TM + 16 * i + t;
        if (m >= mcount) continue;
        const size_t row = MODE == kDw ? (size_t)group * g.n + row0 + m : (size_t)row0 + m;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int c = wn * TN + 16 * j + 4 * q;
            if (c >= ccount) continue;   // extents are multiples of 8: all four or none
            f32x4_t v = acc[i][j];
            const size_t at = row * C + c0 + c;
            if constexpr (F32OUT) {
                float *o = static_cast<float *>(g.out) + at;
                if (g.add) v += *reinterpret_cast<const f32x4_t *>(static_cast<const float *>(g.add) + at);
                *reinterpret_cast<f32x4_t *>(o) = v;
            } else {
                uint16_t *o = static_cast<uint16_t *>(g.out) + at;
                if constexpr (MODE == kDw) {
                    if (g.add) {
                        const ushort4 u = *reinterpret_cast<const ushort4 *>(static_cast<const uint16_t *>(g.add) + at);
                        v += f32x4_t{widen16<BF16>(u.x), widen16<BF16>(u.y), widen16<BF16>(u.z), widen16<BF16>(u.w)};
                    }
                }
                *reinterpret_cast<ushort4 *>(o) = make_ushort4(round16<BF16>(v[0]), round16<BF16>(v[1]),
                                                               round16<BF16>(v[2]), round16<BF16>(v[3]));
            }
        }
    }
}

template <int MODE, bool BF16, bool F32OUT, int BM, int BN, int WM, int WN, int STAGES>
static void launch_tile(const GroupedArgs &g, hipStream_t s) {
    const int C = MODE == kMm ? g.n : g.k;
    const int tn = (C + BN - 1) / BN;
    dim3 grid;
    if (MODE == kDw)
        grid = dim3((unsigned)((g.n + BM - 1) / BM * tn), (unsigned)g.groups);
    else   // at most this many row tiles: one ragged tile a group
        grid = dim3((unsigned)((((int64_t)g.rows + BM - 1) / BM + min(g.groups, g.rows)) * tn + kXcd));
    hipLaunchKernelGGL((k_grouped_mm<MODE, BF16, F32OUT, BM, BN, WM, WN, STAGES>), grid, dim3(64 * WM * WN), 0, s, g);
}

template <bool BF16>
static void launch_rows(const GroupedArgs &g, bool dx, hipStream_t s) {
    if (dx)
        launch_tile<kDx, BF16, false, 128, 128, 2, 2, 3>(g, s);
    else
        launch_tile<kMm, BF16, false, 128, 128, 2, 2, 3>(g, s);
}

void launch_grouped_mm(const void *x, const void *w, const int *offsets, int groups, int rows, int n, int k, bool bf16,
                       void *y, hipStream_t s) {
    const GroupedArgs g{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(w), offsets, y, nullptr, groups, rows, n, k};
    if (bf16) launch_rows<true>(g, false, s); else launch_rows<false>(g, false, s);
}

void launch_grouped_mm_dx(const void *dy, const void *w, const int *offsets, int groups, int rows, int n, int k, bool bf16,
                          void *dx, hipStream_t s) {
    const GroupedArgs g{static_cast<const uint8_t *>(dy), static_cast<const uint8_t *>(w), offsets, dx, nullptr, groups, rows, n, k};
    if (bf16) launch_rows<true>(g, true, s); else launch_rows<false>(g, true, s);
}

void launch_grouped_mm_dw(const void *x, const void *dy, const int *offsets, int groups, int rows, int n, int k, bool bf16,
                          bool f32_out, const void *add, void *dw, hipStream_t s) {
    const GroupedArgs g{static_cast<const uint8_t *>(dy), static_cast<const uint8_t *>(x), offsets, dw, add, groups, rows, n, k};
    if (bf16) {
        if (f32_out) launch_tile<kDw, true, true, 128, 128, 2, 2, 3>(g, s);
        else launch_tile<kDw, true, false, 128, 128, 2, 2, 3>(g, s);
    } else {
        if (f32_out) launch_tile<kDw, false, true, 128, 128, 2, 2, 3>(g, s);
        else launch_tile<kDw, false, false, 128, 128, 2, 2, 3>(g, s);
    }
}

}  // namespace moe_w4

// Matrix products grouped by expert with ragged row counts, in bf16 or fp16
// with fp32 sums (moe_w4_grouped_mm, _dx, _dw):
//   mm:  y[r][n]     = sum_k x[r][k]  w[e][n][k]
//   dx:  dx[r][k]    = sum_n dy[r][n] w[e][n][k]
//   dw:  dw[e][n][k] = add[e][n][k] + sum_r dy[r][n] x[r][k]
// for the rows offsets[e] <= r < offsets[e + 1] of group e.
//
// One tile kernel serves the three: out[m][c] = sum_l A(m, l) B(c, l), where an
// operand is either "K-major" (l contiguous in memory: x and w of mm, dy of
// dx) or "MN-major" (its m or c contiguous, one row per l: w of dx, dy and x of
// dw).  l advances kStep = 64 a step.  Both kinds go from global memory to LDS
// with 16-byte buffer loads that bypass the registers, STAGES steps ahead; a
// K-major fragment of v_mfma_f32_16x16x32 is one 16-byte LDS read, an MN-major one
// two transposing 8-byte LDS reads (ds_read_b64_tr_b16: in each group of 16 lanes,
// lane t receives element t of 4 rows of 16 elements).
//
// Workgroups are as many as the chip holds, and each walks its share of the tiles
// as one stream of steps: the loads run ahead across the borders of the tiles,
// so a tile's first steps arrive under the stores of the one before (a tile a
// workgroup cost 10 us a tile more).  The LDS reads of a half step run under the
// MFMAs of the half before, from two register sets.  (Other shapes tried at 256 x
// 393216 x 1024 x 2048: 32x32x16 MFMAs 1650 us against 1540; 32 l a step and 4
// stages 1790 against 1620; 4 waves of 128 x 128 each 1950 against 1620.)
//
// Edges need no branches in the loop: the descriptor of each load ends with
// the group's (or the expert's) last row, and lanes past the contiguous
// extent aim past every descriptor; the hardware's range check makes both
// zeros in LDS.  Descriptors of MN-major operands move with l, so offsets
// stay small whatever the tensors' sizes are.
//
// Measured (MI355X): 256 experts, 1024 x 2048, bf16: 192 rows 99 us (5.7 TB/s, the
// weights' stream), 12288 uneven rows 218 us (5.3 TB/s), 393216 rows 1529 us (1079
// TFLOP/s: a large library product reaches 1478); dw of 98304 rows into fp32, added
// to, 1094 us (4.5 TB/s, a copy reaches 4.9); dx of 20011 fp16 rows of 60 experts,
// 1400 x 2056, 184 us (626 TFLOP/s: the ninth column tile holds 8 columns, and 1080
// tiles are five rounds of the CUs where 4.2 would do).
#include <type_traits>

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
    int slices;               // dw: parts that each group's rows are split into (groups counts the parts)
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
constexpr int kCus = 256;
constexpr int kLdsBytes = 160 * 1024;

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
__device__ __forceinline__ uint32_t pack16(float a, float b) {   // round to nearest even
    if constexpr (!BF16) return pack_half2(a, b);
    const __bf16 x = (__bf16)a, y = (__bf16)b;
    return (uint32_t)__builtin_bit_cast(uint16_t, x) | ((uint32_t)__builtin_bit_cast(uint16_t, y) << 16);
}
template <bool BF16>
__device__ __forceinline__ float widen16(uint16_t v) {
    if constexpr (BF16) return bf16_to_f32(v);
    return (float)__builtin_bit_cast(_Float16, v);
}

// 16 bytes a lane from a buffer straight to LDS (lane i's to lds + 16 i; lanes out of the buffer's range write zeros).
// In assembler, because behind the builtin the compiler waits for every load in
// flight before a transposing read of LDS, which ends the overlap of loads and
// products (dw of 8 groups x 8192 rows, 2048 x 4096: 935 TFLOP/s with the builtin,
// 1056 so).  The instruction writes no register, so
// nothing of it is in the compiler's hands; its address is read as it issues, and
// wait_vm() and barrier() order it with the LDS reads; s_nop 4 covers the wait states of an SGPR from a VALU operation.
__device__ __forceinline__ void load_to_lds(u32x4_t r, uint32_t lds, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(r)
                 : "memory");
}
__device__ __forceinline__ u32x4_t buffer_of(const void *base, uint32_t bytes) {
    const uint64_t a = (uint64_t)(uintptr_t)base;
    auto uniform = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); };   // (an SGPR)
    return u32x4_t{uniform((uint32_t)a), uniform((uint32_t)(a >> 32) & 0xffffu), uniform(bytes), 0x00020000u};
}
__device__ __forceinline__ s16x4_t read_transposed(const lds_u8 *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
}

// A bit that puts an offset behind every descriptor, unless `in` (arithmetic, not
// a choice: each load has to stay one instruction of the whole wave, as the
// waits count them).
__device__ __forceinline__ uint32_t past_unless(bool in) { return ((uint32_t)in - 1u) & kPast; }

// Where the operand tile of one matrix comes from: base of its first row, the
// number of rows and of contiguous elements (K-major: m or c, and l; MN-major:
// l, and m or c; all from the tile's first).
struct Operand {
    const uint8_t *base;
    int rows, cols;
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
    static constexpr int kRows = NT / kChunks;                  // rows that one load of the workgroup covers
    static_assert(kBytes % 1024 == 0 && kBytes % (16 * NT) == 0 && kRows % 16 == 0, "whole loads; one swizzle for all of a thread's loads");
    uint32_t pitch;   // bytes from row to row
    uint32_t off;     // byte offset of this thread's first load at l = 0
    int q;            // the 16-byte chunk of its row that this thread loads

    // Load i of a thread: LDS bytes [16 (tid + NT i), +16) of the image.
    __device__ __forceinline__ void init(uint32_t row_bytes, int tid) {
        const int row = tid / kChunks, slot = tid % kChunks;
        pitch = row_bytes;
        q = MN ? slot ^ (2 * ((row & 3) | ((row >> 1) & 4)) & (kChunks - 1)) : slot ^ ((row >> 1) & 7);
        off = (uint32_t)row * pitch + 16 * q;
    }

    // Starts the loads of step s into the image at lds.
    __device__ __forceinline__ void load(const Operand &o, int s, uint32_t lds, int wave) const {
        const int l = s * kStep;
        if constexpr (MN) {
            const int left = min(o.rows - l, kStep);
            const u32x4_t r = buffer_of(o.base + (size_t)l * pitch, left <= 0 ? 0u : (uint32_t)left * pitch);
            const uint32_t past = past_unless(8 * q < o.cols);
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                load_to_lds(r, lds + 16 * (NT * i + 64 * wave), (off + (uint32_t)(i * kRows) * pitch) | past);
        } else {
            const u32x4_t r = buffer_of(o.base, (uint32_t)o.rows * pitch);
            const uint32_t past = past_unless(l + 8 * q < o.cols);
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                load_to_lds(r, lds + 16 * (NT * i + 64 * wave), (off + (uint32_t)(i * kRows) * pitch + 2u * l) | past);
        }
    }

    // Fragment of 16 m (or c) and 32 l: lane t + 16 g holds position 16 block + t, l
    // = 32 kk + 8 g .. + 8.  Its LDS address is this lane's own part, from lane_part()
    // for the blocks that share the bits of `block`, changed by constants in the
    // rest of the block's bits, `more` (disjoint), and kk.
    static constexpr int kMask = (kChunks / 2 - 1) & 7;   // MN: block bits that the swizzle mixes
    static __device__ __forceinline__ uint32_t lane_part(int block, int lane) {
        const int t = lane & 15, g = lane >> 4;
        if constexpr (MN) {
            const int h = (t >> 2) | ((g & 1) << 2);
            return (8 * g + (t >> 2)) * (2 * R) + (((block ^ h) & kMask) << 5) + ((block & ~kMask) << 5) +
                   ((t & 3) >> 1) * 16 + (t & 1) * 8;
        } else {
            return (16 * block + t) * 128 + ((g ^ (t >> 1)) << 4);
        }
    }
    static __device__ __forceinline__ s16x8_t frag(uint32_t part, int more, int kk) {
        if constexpr (MN) {
            const lds_u8 *a = (const lds_u8 *)(uintptr_t)(part ^ ((more & kMask) << 5)) + ((more & ~kMask) << 5) + kk * (64 * R);
            const s16x4_t lo = read_transposed(a);
            const s16x4_t hi = read_transposed(a + 4 * (2 * R));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            return *(const lds_s16x8 *)((const lds_u8 *)(uintptr_t)(part ^ (kk * 64)) + more * 2048);
        }
    }
};

template <int N>
__device__ __forceinline__ void wait_vm() {   // at most N vector memory operations of this wave outstanding, no LDS read
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}
__device__ __forceinline__ void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The groups as a workgroup holds them in LDS, and the tiles that it takes.
struct Groups {
    const int *first;    // [groups] first row, clamped
    const int *count;    // [groups] rows
    const int *before;   // [groups + 1] tiles of the groups before
};
__device__ __forceinline__ int lds_int(const int *p) { return __builtin_amdgcn_readfirstlane(*p); }

struct Range {
    int begin, end;   // tiles of this workgroup's XCD
};

// Inclusive sum over the lanes of a wave (data-parallel primitives: six
// operations of the VALU, without the LDS crossbar's latency).
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);   // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);   // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);   // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
    return v;
}

// Reads the offsets once: rows and tiles of each group into LDS, and the run of
// tiles of XCD x.  Offsets are clamped to [0, rows] and to their predecessor,
// so that no tile leaves the arrays whatever they hold.  Tiles are numbered
// group by group; an XCD takes a contiguous run of them, so that the tiles that
// share rows or weights share an L2.  Runs have equal work: for mm and dx equal
// numbers of tiles, for dw tiles weighted by their steps (kTileFixed: steps that
// an epilogue is worth), in units that keep the sums within 31 bits.
constexpr int kTileFixed = 16;
template <int MODE, int BM, int NT>
__device__ __forceinline__ Range survey(const GroupedArgs &g, int tiles_m, int tiles_n, int x, int *first, int *count,
                                        int *before, int *sh) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (g.groups + NT - 1) / NT;
    const int e0 = min(tid * per, g.groups), e1 = min(e0 + per, g.groups);
    auto tiles_of = [&](int rows) { return MODE == kDw ? tiles_m * tiles_n : (rows + BM - 1) / BM * tiles_n; };
    auto weight = [&](int rows) { return (rows + kStep - 1) / kStep + kTileFixed; };   // dw: of each tile of the group
    int tiles = 0, work = 0;
    for (int e = e0; e < e1; ++e) {
        const int of = MODE == kDw ? e / g.slices : e;
        int lo = min(max(g.offsets[of], 0), g.rows), hi = min(max(g.offsets[of + 1], lo), g.rows);
        if (MODE == kDw && g.slices > 1) {   // slice e % slices, of whole steps
            const int each = ((hi - lo + kStep - 1) / kStep + g.slices - 1) / g.slices * kStep;
            lo = min(lo + e % g.slices * each, hi);
            hi = min(lo + each, hi);
        }
        first[e] = lo;
        count[e] = hi - lo;
        tiles += tiles_of(hi - lo);
        if (MODE == kDw) work += weight(hi - lo);   // (every group has as many tiles)
    }
    const int pt = wave_scan(tiles), pw = MODE == kDw ? wave_scan(work) : 0;
    constexpr int kW = NT / 64;
    if (lane == 63) {
        sh[wave] = pt;
        if (MODE == kDw) sh[kW + wave] = pw;
    }
    __syncthreads();
    int bt = 0, bw = 0, all_t = 0, all_w = 0;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
        const int vt = sh[w], vw = MODE == kDw ? sh[kW + w] : 0;
        if (w < wave) bt += vt, bw += vw;
        all_t += vt;
        all_w += vw;
    }
    int t = pt - tiles + bt, w0 = pw - work + bw;   // tiles and work before this thread's groups
    const int from = (int)((int64_t)all_w * x / kXcd), to = (int)((int64_t)all_w * (x + 1) / kXcd);
    for (int e = e0; e < e1; ++e) {
        before[e] = t;
        if (MODE == kDw) {
            // the share of the group's tiles that lies before a point of the work
            const int n = tiles_of(0), unit = weight(count[e]);
            if (from >= w0 && from < w0 + unit) sh[2 * kW] = t + (int)((int64_t)n * (from - w0) / unit);
            if (to >= w0 && to < w0 + unit) sh[2 * kW + 1] = t + (int)((int64_t)n * (to - w0) / unit);
            w0 += unit;
        }
        t += tiles_of(count[e]);
    }
    if (tid == 0) before[g.groups] = all_t;
    if (MODE == kDw && tid == 0 && x == kXcd - 1) sh[2 * kW + 1] = all_t;   // (to == all_w lies in no group)
    __syncthreads();
    Range r;
    if (MODE == kDw) {
        r.begin = lds_int(sh + 2 * kW);
        r.end = lds_int(sh + 2 * kW + 1);
    } else {
        const int run = (__builtin_amdgcn_readfirstlane(all_t) + kXcd - 1) / kXcd;
        r.begin = min(x * run, all_t);
        r.end = min(r.begin + run, all_t);
        r.begin = __builtin_amdgcn_readfirstlane(r.begin);
        r.end = __builtin_amdgcn_readfirstlane(r.end);
    }
    return r;
}

// The group of a tile: the last one that begins at it or before (64-way search, twice).
__device__ __forceinline__ int group_of(const int *before, int groups, int tile) {
    const int lane = threadIdx.x & 63, step = (groups + 63) / 64;
    const int a = lane * step;
    const int hi = __popcll(__ballot(a < groups && before[min(a, groups)] <= tile)) - 1;
    const int b = hi * step + lane;
    return hi * step + __popcll(__ballot(lane < step && b < groups && before[min(b, groups)] <= tile)) - 1;
}

// A place in a workgroup's sequence of tiles (tile, tile + stride, ..), and that tile.
template <int MODE, int BM, int BN>
struct Walker {
    int tile, group;
    int row0, mcount, c0, ccount, steps;   // output rows (dw: within n) and columns, steps of l
    Operand A, B;

    __device__ __forceinline__ void enter(const GroupedArgs &g, const Groups &gs, int tiles_n, int end) {
        const int C = MODE == kMm ? g.n : g.k;
        if (tile >= end) {   // behind the last: operands of which nothing is in range
            A.rows = A.cols = B.rows = B.cols = steps = 0;
            A.base = g.a;
            B.base = g.b;
            return;
        }
        group = __builtin_amdgcn_readfirstlane(group_of(gs.before, g.groups, tile));
        const int local = tile - lds_int(gs.before + group);
        const int mt = __builtin_amdgcn_readfirstlane(local / tiles_n), nt = local - mt * tiles_n;   // (a division is VALU work)
        const int lo = lds_int(gs.first + group), rows = lds_int(gs.count + group);
        c0 = nt * BN;
        ccount = __builtin_amdgcn_readfirstlane(min(C - c0, BN));
        if constexpr (MODE == kDw) {
            row0 = mt * BM;
            mcount = __builtin_amdgcn_readfirstlane(min(g.n - row0, BM));
            A.base = g.a + ((size_t)lo * g.n + row0) * 2;
            B.base = g.b + ((size_t)lo * g.k + c0) * 2;
            A.rows = B.rows = rows;
            A.cols = mcount;
            B.cols = ccount;
            steps = (rows + kStep - 1) / kStep;
        } else {
            const int len = MODE == kMm ? g.k : g.n;
            row0 = lo + mt * BM;
            mcount = __builtin_amdgcn_readfirstlane(min(rows - mt * BM, BM));
            A.base = g.a + (size_t)row0 * len * 2;
            A.rows = mcount;
            A.cols = len;
            const uint8_t *w = g.b + (size_t)group * g.n * g.k * 2;
            B.base = MODE == kMm ? w + (size_t)c0 * g.k * 2 : w + (size_t)c0 * 2;
            B.rows = MODE == kMm ? ccount : len;
            B.cols = MODE == kMm ? len : ccount;
            steps = (len + kStep - 1) / kStep;
        }
    }
};

}  // namespace

// BM x BN tiles by WM x WN waves.  A workgroup walks its tiles as one stream of
// steps: loads run STAGES steps ahead across the tiles' borders, so a tile's
// first steps arrive while the tile before is stored.
template <int MODE, bool BF16, bool F32OUT, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(64 * WM *WN) void k_grouped_mm(GroupedArgs g) {
    constexpr int NT = 64 * WM * WN;
    constexpr int FM = BM / WM / 16, TN = BN / WN, FN = TN / 16;
    typedef Tile<BM, MODE == kDw, NT> TA;
    typedef Tile<BN, MODE != kMm, NT> TB;
    constexpr int kStageBytes = TA::kBytes + TB::kBytes;
    constexpr int kLoads = TA::kLoads + TB::kLoads;
    constexpr int kElem = F32OUT ? 4 : 2;
    static_assert(F32OUT || FN % 2 == 0, "16-bit blocks are stored in pairs");
    // one LDS object: with more, the compiler waits for every load in flight before an LDS read
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const uint32_t lds_base = (uint32_t)(uintptr_t)(lds_u8 *)smem;        // the stages (a multiple of 1024)
    int *scan = reinterpret_cast<int *>(smem);                     // only before the first load
    int *tables = reinterpret_cast<int *>(smem + STAGES * kStageBytes);   // first, count, before
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int C = MODE == kMm ? g.n : g.k;   // columns of the output
    const int tiles_n = (C + BN - 1) / BN, tiles_m = (g.n + BM - 1) / BM;
    const int xcd = blockIdx.x % kXcd, stride = gridDim.x / kXcd;

    const Range range = survey<MODE, BM, NT>(g, tiles_m, tiles_n, xcd, tables, tables + g.groups, tables + 2 * g.groups, scan);
    const Groups gs{tables, tables + g.groups, tables + 2 * g.groups};
    typedef Walker<MODE, BM, BN> Walk;
    Walk at;   // the tile being multiplied
    at.tile = range.begin + (int)blockIdx.x / kXcd;
    if (at.tile >= range.end) return;
    at.enter(g, gs, tiles_n, range.end);
    Walk ld = at;   // the tile being loaded, and the step
    int ld_step = 0;
    auto skip = [&]() {   // on to the next tile that has the step
        while (ld_step >= ld.steps && ld.tile < range.end) {
            ld.tile += stride;
            ld_step = 0;
            ld.enter(g, gs, tiles_n, range.end);
        }
    };
    skip();

    TA ta;
    TB tb;
    ta.init(2u * (MODE == kMm ? g.k : g.n), tid);
    tb.init(2u * g.k, tid);
    auto issue = [&](int slot) {
        ta.load(ld.A, ld_step, lds_base + slot * kStageBytes, wave);
        tb.load(ld.B, ld_step, lds_base + slot * kStageBytes + TA::kBytes, wave);
        ++ld_step;
    };

    f32x4_t acc[FM][FN];
    // fragments of one half step (32 l), in two register sets: the reads of a
    // half run under the products of the one before.  The waves that share
    // columns take the tile's 16-row blocks in turn, so that a tile of few rows
    // is few products for all of them: AF blocks each
    s16x8_t fa[2][FM], fb[2][FN];
    auto row_of = [&](int i) { return 16 * (i * WM + wm); };
    int slot = 0;
    const uint32_t part_a = TA::lane_part(wm, lane), part_b = TB::lane_part(wn * FN, lane);
    auto read = [&](auto AF, int kk) {
        const uint32_t pa = part_a + lds_base + slot * kStageBytes, pb = part_b + lds_base + slot * kStageBytes + TA::kBytes;
#pragma unroll
        for (int i = 0; i < AF(); ++i) fa[kk][i] = TA::frag(pa, i * WM, kk);
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[kk][j] = TB::frag(pb, j, kk);
    };
    auto multiply = [&](auto AF, int kk) {
#pragma unroll
        for (int i = 0; i < AF(); ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<BF16>(fb[kk][j], fa[kk][i], acc[i][j]);
    };
    auto interleave = [&](auto AF) {   // one LDS read, then its share of the MFMAs, throughout the half step
        constexpr int kReads = AF() * (MODE == kDw ? 2 : 1) + FN * (MODE == kMm ? 1 : 2);
        constexpr int per = AF() * FN / kReads > 0 ? AF() * FN / kReads : 1;
#pragma unroll
        for (int i = 0; i < kReads; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, per, 0);
        }
    };
    auto steps = [&](auto AF) {
        read(AF, 0);
        for (int s = 0; s < at.steps; ++s) {
            skip();
            read(AF, 1);
            multiply(AF, 0);
            interleave(AF);
            // the next step of the stream has arrived for this wave (STAGES - 2
            // later ones may be in flight) and its reads of this step are done;
            // behind the barrier both hold for all waves, and the loads issued
            // next may overwrite this step.  Loads behind the last tile read
            // nothing (every lane out of range)
            wait_vm<(STAGES - 2) * kLoads>();
            barrier();
            issue(slot);
            if (++slot == STAGES) slot = 0;
            read(AF, 0);   // (behind a tile's last step: of the next tile, read again there)
            multiply(AF, 1);
            interleave(AF);
        }
    };

    // Stores the tile.  Lane t + 16 q holds row t, columns 4 q .. + 4 of each 16 x 16
    // block: 16 bytes of fp32, or, after neighbours q and q ^ 1 have exchanged
    // halves of two blocks, 16 bytes of 8 columns (64 bytes a row for each store
    // either way).  Rows and columns behind the tile's are out of the buffers'
    // range: no branch, so that the loads of `add` go out together.
    auto store = [&]() {
        int l2 = lane;
        asm volatile("" : "+v"(l2));   // keeps the addresses below out of the registers of the loop above
        const int t = l2 & 15, q = l2 >> 4;
        const uint32_t pitch = (uint32_t)C * kElem;
        const size_t first = ((MODE == kDw ? (size_t)at.group * g.n + at.row0 : (size_t)at.row0) * C + at.c0) * kElem;
        const __amdgpu_buffer_rsrc_t out = make_buf(static_cast<uint8_t *>(g.out) + first, (uint32_t)at.mcount * pitch);
        const __amdgpu_buffer_rsrc_t add = make_buf(static_cast<const uint8_t *>(g.add) + first, (uint32_t)at.mcount * pitch);
        // the column of this lane's first 16 bytes, and its next ones'
        const int col = wn * TN + (F32OUT ? 4 * q : 16 * (q & 1) + 8 * (q >> 1));
        constexpr int kNext = F32OUT ? 16 : 32, kStores = FN * 16 / kNext;
        uint32_t past[kStores];
#pragma unroll
        for (int j = 0; j < kStores; ++j) past[j] = past_unless(col + j * kNext < at.ccount);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if (row_of(i) >= at.mcount) break;
            const uint32_t off = (uint32_t)(row_of(i) + t) * pitch + (uint32_t)col * kElem;
            uint4 old[kStores];
            if (MODE == kDw && g.add) {
#pragma unroll
                for (int j = 0; j < kStores; ++j) old[j] = bload16(add, (off + j * kNext * kElem) | past[j], 0);
            }
#pragma unroll
            for (int j = 0; j < kStores; ++j) {
                u32x4_t v;
                if constexpr (F32OUT) {
                    f32x4_t f = acc[i][j];
                    if (MODE == kDw && g.add)
                        f += f32x4_t{__uint_as_float(old[j].x), __uint_as_float(old[j].y), __uint_as_float(old[j].z), __uint_as_float(old[j].w)};
                    v = __builtin_bit_cast(u32x4_t, f);
                } else {
                    f32x4_t a = acc[i][2 * j], b = acc[i][2 * j + 1];
                    // a, b: columns 4q of blocks 2j and 2j + 1 -> lo, hi: the 4 + 4 columns of `col`
                    f32x4_t lo, hi;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(a[k]), __float_as_uint(b[k]), false, false);
                        lo[k] = __uint_as_float(p[0]);
                        hi[k] = __uint_as_float(p[1]);
                    }
                    if (MODE == kDw && g.add) {
                        const uint32_t o[4] = {old[j].x, old[j].y, old[j].z, old[j].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            (k < 2 ? lo : hi)[2 * (k & 1)] += widen16<BF16>((uint16_t)o[k]);
                            (k < 2 ? lo : hi)[2 * (k & 1) + 1] += widen16<BF16>((uint16_t)(o[k] >> 16));
                        }
                    }
                    v = u32x4_t{pack16<BF16>(lo[0], lo[1]), pack16<BF16>(lo[2], lo[3]), pack16<BF16>(hi[0], hi[1]),
                                pack16<BF16>(hi[2], hi[3])};
                }
                __builtin_amdgcn_raw_buffer_store_b128(v, out, (off + j * kNext * kElem) | past[j], 0, 0);
            }
        }
    };

#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
        skip();
        issue(s);
    }
    wait_vm<(STAGES - 1) * kLoads>();
    barrier();
    for (;;) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        const int blocks = (at.mcount + 16 * WM - 1) / (16 * WM);   // 16-row blocks of a wave
        constexpr int kQ = FM >= 4 ? FM / 4 : 1;
        if (blocks <= kQ) steps(std::integral_constant<int, kQ>{});
        else if (blocks <= 2 * kQ) steps(std::integral_constant<int, (2 * kQ < FM ? 2 * kQ : FM)>{});
        else if (FM > 2 && blocks <= 3 * kQ) steps(std::integral_constant<int, (3 * kQ < FM ? 3 * kQ : FM)>{});
        else steps(std::integral_constant<int, FM>{});

        store();
        at.tile += stride;
        if (at.tile >= range.end) break;
        if (ld.tile == at.tile) at = ld;   // the loads are one tile ahead unless tiles have fewer steps than there are stages
        else at.enter(g, gs, tiles_n, range.end);
    }
    wait_vm<0>();   // nothing may land in LDS behind the workgroup's end
}

template <int MODE, bool BF16, bool F32OUT, int BM, int BN, int WM, int WN, int STAGES>
static void launch_tile(const GroupedArgs &g, hipStream_t s) {
    const int C = MODE == kMm ? g.n : g.k;
    const int64_t tn = (C + BN - 1) / BN;
    // at most this many tiles (mm, dx: one ragged row tile a group)
    const int64_t most = MODE == kDw ? (int64_t)((g.n + BM - 1) / BM) * tn * g.groups
                                     : ((int64_t)g.rows / BM + min(g.groups, g.rows)) * tn;
    const int lds = STAGES * (BM + BN) * kStep * 2 + (3 * g.groups + 1) * (int)sizeof(int);
    const int resident = kCus * (kLdsBytes / lds);   // workgroups that the chip holds at once
    const unsigned grid = (unsigned)(most >= resident ? resident : (most + kXcd - 1) / kXcd * kXcd);
    hipLaunchKernelGGL((k_grouped_mm<MODE, BF16, F32OUT, BM, BN, WM, WN, STAGES>), dim3(grid), dim3(64 * WM * WN), lds, s, g);
}

// The tile by the rows a group has on average and by how many tiles there are
// for the 256 CUs (the offsets are on the device, so half a ragged tile a group
// is assumed).  us on MI355X, E groups x rows in all x n x k, tiles as named:
//                            256x256  128x128  64x128  32x64
//   256 x 98304 x 1024 x 2048    513      569     731            products bound it: the fewest LDS and L2 reads a product
//   256 x 24576 x 1024 x 2048    243      252     277    492
//   256 x 12288 x 1024 x 2048    260      223     221    296     (uneven groups) weights bound it: little work on absent rows
//   256 x   192 x 1024 x 2048    136      116     101    100
//     1 x  4096 x 2048 x 2048     52       37      50    114     too few large tiles for the CUs
//     8 x  7168 x 2048 x 2048    102       75                    264 large tiles: a second round of the CUs for 8
//     8 x 14336 x 2048 x 2048    106      133                    488 large tiles: two full rounds
//    16 x 12288 x 1152 x 2048 dx  98       66                    285 large tiles
//     8 x   256 x 2048 x 2048     31       23      22     19     latency: the most, smallest tiles
constexpr int kMinRows = 80, kFewRows = 16;        // rows a group
constexpr int kFewTiles128 = 128;
// Large tiles go in whole rounds of the CUs; small ones, two a CU, so evenly that a
// part of a round counts as a part, and 512 of them take 0.8 of a large round.
constexpr int kSmallPerRound = 640;

template <int MODE, bool BF16>
static void launch_rows(const GroupedArgs &g, hipStream_t s) {
    const int C = MODE == kMm ? g.n : g.k;
    const int held = min(g.groups, g.rows), per = g.rows / held;
    auto tiles = [&](int bm, int bn) { return ((int64_t)g.rows / bm + held / 2 + 1) * ((C + bn - 1) / bn); };
    if (per >= kMinRows && tiles(128, 128) >= (tiles(256, 256) + kCus - 1) / kCus * kSmallPerRound)
        launch_tile<MODE, BF16, false, 256, 256, 2, 4, 2>(g, s);
    else if (MODE == kMm && (per <= kFewRows || tiles(128, 128) <= kFewTiles128))
        launch_tile<kMm, BF16, false, 32, 64, 2, 2, 4>(g, s);   // (dx of few rows: 117 us against 110 at 256 x 192 rows)
    else if (per < kMinRows)
        launch_tile<MODE, BF16, false, 64, 128, 2, 2, 2>(g, s);
    else
        launch_tile<MODE, BF16, false, 128, 128, 2, 2, 2>(g, s);
}

// out[i] = add[i] + the sum of the slices' [i] in order, 8 elements a thread.
template <bool BF16, bool F32OUT>
__global__ __launch_bounds__(256) void k_grouped_join(const float *parts, int slices, int64_t each, int64_t all, const void *add,
                                                      void *out) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= all) return;
    const float *p = parts + i / each * slices * each + i % each;   // each: one group's elements, a multiple of 64
    f32x4_t a = {0.0f, 0.0f, 0.0f, 0.0f}, b = a;
#pragma unroll 4
    for (int s = 0; s < slices; ++s) {
        a += *reinterpret_cast<const f32x4_t *>(p + s * each);
        b += *reinterpret_cast<const f32x4_t *>(p + s * each + 4);
    }
    if constexpr (F32OUT) {
        if (add) {
            a += *reinterpret_cast<const f32x4_t *>(static_cast<const float *>(add) + i);
            b += *reinterpret_cast<const f32x4_t *>(static_cast<const float *>(add) + i + 4);
        }
        *reinterpret_cast<f32x4_t *>(static_cast<float *>(out) + i) = a;
        *reinterpret_cast<f32x4_t *>(static_cast<float *>(out) + i + 4) = b;
    } else {
        if (add) {
            const uint4 o = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(add) + i);
            const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                (k < 2 ? a : b)[2 * (k & 1)] += widen16<BF16>((uint16_t)w[k]);
                (k < 2 ? a : b)[2 * (k & 1) + 1] += widen16<BF16>((uint16_t)(w[k] >> 16));
            }
        }
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + i) = make_uint4(
            pack16<BF16>(a[0], a[1]), pack16<BF16>(a[2], a[3]), pack16<BF16>(b[0], b[1]), pack16<BF16>(b[2], b[3]));
    }
}

// dw of few tiles and many rows: the rows of each group in this many slices, so
// that about two workgroups a CU have work, of at least 16 steps each on average (1 x
// 65536 rows, 512 x 512: 48 us against 629; of 8 steps, 4 x 2000 rows: 26 against 23);
// the slices' sums go to the workspace in fp32 and are joined by a second launch.
int grouped_dw_slices(int groups, int rows, int n, int k) {
    const int64_t tiles = (int64_t)groups * ((n + 127) / 128) * ((k + 127) / 128);
    const int64_t fill = 2 * kCus / tiles, steps = (int64_t)rows / groups / (16 * kStep);
    const int64_t s = fill < steps ? fill : steps;
    return s > 1 ? (int)s : 1;
}

// dw: large tiles for many of them with many rows to sum over (256 groups x 384
// rows, 1024 x 2048: 1090 us against 1295); else twice the workgroups, whose
// stores and products overlap (256 x 48 rows: 930 against 981; 1 x 65536 rows,
// 2048 x 2048, 64 large tiles: 846 against 1488).
template <bool BF16, bool F32OUT>
static void launch_dw(const GroupedArgs &g, float *parts, hipStream_t s) {
    const int64_t tiles = (int64_t)g.groups * ((g.n + 255) / 256) * ((g.k + 255) / 256);
    const int slices = parts ? grouped_dw_slices(g.groups, g.rows, g.n, g.k) : 1;
    if (slices > 1) {
        GroupedArgs h = g;
        h.groups = g.groups * slices;
        h.slices = slices;
        h.out = parts;
        h.add = nullptr;
        launch_tile<kDw, BF16, true, 128, 128, 2, 2, 2>(h, s);
        if (hipPeekAtLastError() != hipSuccess) return;
        const int64_t each = (int64_t)g.n * g.k, all = each * g.groups;
        hipLaunchKernelGGL((k_grouped_join<BF16, F32OUT>), dim3((unsigned)((all + 2047) / 2048)), dim3(256), 0, s, parts, slices, each,
                           all, g.add, g.out);
    } else if (tiles >= 2048 && g.rows / g.groups >= kMinRows) {
        launch_tile<kDw, BF16, F32OUT, 256, 256, 2, 4, 2>(g, s);
    } else {
        launch_tile<kDw, BF16, F32OUT, 128, 128, 2, 2, 2>(g, s);
    }
}

void launch_grouped_mm(const void *x, const void *w, const int *offsets, int groups, int rows, int n, int k, bool bf16,
                       void *y, hipStream_t s) {
    const GroupedArgs g{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(w), offsets, y, nullptr, groups, rows, n, k, 1};
    if (bf16) launch_rows<kMm, true>(g, s); else launch_rows<kMm, false>(g, s);
}

void launch_grouped_mm_dx(const void *dy, const void *w, const int *offsets, int groups, int rows, int n, int k, bool bf16,
                          void *dx, hipStream_t s) {
    const GroupedArgs g{static_cast<const uint8_t *>(dy), static_cast<const uint8_t *>(w), offsets, dx, nullptr, groups, rows, n, k, 1};
    if (bf16) launch_rows<kDx, true>(g, s); else launch_rows<kDx, false>(g, s);
}

void launch_grouped_mm_dw(const void *x, const void *dy, const int *offsets, int groups, int rows, int n, int k, bool bf16,
                          bool f32_out, const void *add, void *dw, float *parts, hipStream_t s) {
    const GroupedArgs g{static_cast<const uint8_t *>(dy), static_cast<const uint8_t *>(x), offsets, dw, add, groups, rows, n, k, 1};
    if (bf16) {
        if (f32_out) launch_dw<true, true>(g, parts, s); else launch_dw<true, false>(g, parts, s);
    } else {
        if (f32_out) launch_dw<false, true>(g, parts, s); else launch_dw<false, false>(g, parts, s);
    }
}

}  // namespace moe_w4

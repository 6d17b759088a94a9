// The norms before and after a block, with the block's gate and residual scale
// (moe_w4_norm_residual and its backward).  Per row of H elements:
//   n  = y / sqrt(mean(y^2) + eps)          (post-norm; without it n = y)
//   s  = n * post_gain
//   r' = r + scale * gate * s               (the residual stream behind the block)
//   x  = r' / sqrt(mean(r'^2) + eps) * pre_gain     (the next block's input)
// and backward, given d r' (from the stream) and d x, with q = 1 / sqrt(..) of
// the pre-norm, p of the post-norm, u = r' q:
//   d r  = d r' + q (h - u mean(h u)),   h = d x * pre_gain
//   d s  = scale * gate * d r,           d gate = scale * d r * s  (summed over what it is shared by)
//   d y  = p (k - n mean(k n)),          k = d s * post_gain       (without post-norm d y = d s)
//   d pre_gain = sum_t d x u,            d post_gain = sum_t d s n
// All statistics, sums and intermediate values are fp32; each output is
// rounded once.
//
// Both are bound by memory: a row stays in registers between its one load and
// its one store (8 neighbouring elements a lane), and the backward pass
// recomputes the two inverse norms from the rows that it has to read anyway.
// Both of its row sums of a norm come from one reduction, as
// mean(h u) = q sum(h r') / H needs no q inside the sum.
//
// Sums over rows (gains, channel gate): each workgroup takes every G-th row and
// keeps its columns' sums in registers, writes them once, and a second launch
// adds the G partial rows in a fixed order: no atomics, the same result each
// time.
//
// Measured (MI355X, bf16 with an fp32 stream; a copy reaches 4.9 TB/s): forward 65536
// x 2048 276 us (5.8 TB/s), 1 x 2048 2.3 us on the device; backward 16384 x 2048 124 us
// (4.8 TB/s, of it 6 us the second launch), 65536 x 2048 471 (5.1), 4000 x 8192 137
// (4.3), 30000 x 512 in bf16 44 (4.2), 1001 x 1000 in fp16 13 (latency of two launches).
#include <type_traits>

#include "common.h"
#include "launch.h"

namespace moe_w4 {

namespace {

constexpr int kBf16 = kElemBf16, kF16 = kElemF16, kF32 = kElemF32;

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_v __attribute__((ext_vector_type(4)));

// 8 neighbouring elements as fp32, and back (round to nearest even).
template <int DT>
__device__ __forceinline__ void load8(const void *p, size_t at, float (&v)[8]) {
    if constexpr (DT == kF32) {
        const f32x4_t *q = reinterpret_cast<const f32x4_t *>(static_cast<const float *>(p) + at);
        const f32x4_t a = q[0], b = q[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    } else {
        const u32x4_v q = *reinterpret_cast<const u32x4_v *>(static_cast<const uint16_t *>(p) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = DT == kBf16 ? bf16lo(q[i]) : half_lo(q[i]);
            v[2 * i + 1] = DT == kBf16 ? bf16hi(q[i]) : half_hi(q[i]);
        }
    }
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (DT == kF16) return pack_half2(a, b);
    const __bf16 x = (__bf16)a, y = (__bf16)b;   // v_cvt_pk_bf16_f32, round to nearest even
    return (uint32_t)__builtin_bit_cast(uint16_t, x) | ((uint32_t)__builtin_bit_cast(uint16_t, y) << 16);
}
template <int DT>
__device__ __forceinline__ void store8(void *p, size_t at, const float (&v)[8]) {
    if constexpr (DT == kF32) {
        f32x4_t *q = reinterpret_cast<f32x4_t *>(static_cast<float *>(p) + at);
        q[0] = f32x4_t{v[0], v[1], v[2], v[3]};
        q[1] = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
        *reinterpret_cast<u32x4_v *>(static_cast<uint16_t *>(p) + at) =
            u32x4_v{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
    }
}
template <int DT>
__device__ __forceinline__ float load1(const void *p, size_t at) {
    if constexpr (DT == kF32) return static_cast<const float *>(p)[at];
    if constexpr (DT == kF16) return (float)static_cast<const _Float16 *>(p)[at];
    return bf16_to_f32(static_cast<const uint16_t *>(p)[at]);
}

// N sums over the WAVES waves that share a row, the result in every lane.  buf:
// this row's [N][WAVES] floats, not in use by an earlier call that a wave may
// still read.
template <int N, int WAVES>
__device__ __forceinline__ void row_sums(float (&v)[N], float *buf, int wave) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) buf[i * WAVES + wave] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) s += buf[i * WAVES + w];
            v[i] = s;
        }
    }
}

}  // namespace

// ROWS rows per workgroup, WAVES waves a row, V chunks of 8 elements a lane.
template <int ACT, int RES, int WAVES, int V, int ROWS>
__global__ __launch_bounds__(64 * WAVES *ROWS) void k_norm(NormArgs a) {
    __shared__ float red[2][ROWS][WAVES];
    const int wave = (threadIdx.x >> 6) % WAVES, sub = (threadIdx.x >> 6) / WAVES;
    const int64_t row = (int64_t)blockIdx.x * ROWS + sub;
    const bool live = row < a.T;
    const int c0 = (wave * 64 + (threadIdx.x & 63)) * 8;
    const size_t at = (size_t)(live ? row : 0) * a.H;
    float r[V][8], y[V][8];
    bool in[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = c0 + v * WAVES * 512;
        in[v] = live && c < a.H;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[v][i] = y[v][i] = 0.0f;
        if (in[v]) {
            load8<RES>(a.resid, at + c, r[v]);
            if (a.y) load8<ACT>(a.y, at + c, y[v]);
        }
    }
    if (a.y) {
        float mul = a.scale;
        if (a.flags & kNormPost) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) ss[0] += y[v][i] * y[v][i];
            row_sums<1, WAVES>(ss, red[0][sub], wave);
            mul *= 1.0f / sqrtf(ss[0] / (float)a.H + a.eps);
        }
        if (a.gate_kind == kGateToken && live) mul *= load1<ACT>(a.gate, (size_t)row);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!in[v]) continue;
            const int c = c0 + v * WAVES * 512;
            float t[8];
            if (a.post_gain) {
                load8<ACT>(a.post_gain, c, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[v][i] *= t[i];
            }
            if (a.gate_kind >= kGateChannel) {
                load8<ACT>(a.gate, a.gate_kind == kGateFull ? at + c : (size_t)c, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[v][i] *= t[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) r[v][i] += mul * y[v][i];
            store8<RES>(a.resid_out, at + c, r[v]);
        }
    }
    if (!(a.flags & kNormPre)) return;
    // (x is the norm of the unrounded r')
    float ss[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] += r[v][i] * r[v][i];
    row_sums<1, WAVES>(ss, red[1][sub], wave);
    const float q = 1.0f / sqrtf(ss[0] / (float)a.H + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (!in[v]) continue;
        const int c = c0 + v * WAVES * 512;
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = 1.0f;
        if (a.pre_gain) load8<ACT>(a.pre_gain, c, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] *= r[v][i] * q;
        store8<ACT>(a.x_out, at + c, t);
    }
}

// Backward.  With w = scale * post_gain * (channel gate) of a column, e = d r * n
// and the gate of the row or element g (1 otherwise), all that depends on y is
//   k = g w d r,    d gate = w e   (full: stored; token: summed over the row,
//   which is also sum(k n) / g),
// and both d post_gain and the channel gate's gradient are a constant of the column
// times Q = sum_t g e: one sum in registers serves the two, and one more d pre_gain.
// Column sums of a workgroup's rows go to parts[which][workgroup][H].
template <int ACT, int RES, int WAVES, int V, int ROWS, int KIND>   // KIND: kGateToken, kGateFull, or kGateChannel (none too)
__global__ __launch_bounds__(64 * WAVES *ROWS) void k_norm_back(NormBackArgs a) {
    __shared__ float red[3][ROWS][3 * WAVES];   // first sums of even and odd rounds, second sums
    const int wave = (threadIdx.x >> 6) % WAVES, sub = (threadIdx.x >> 6) / WAVES;
    const int c0 = (wave * 64 + (threadIdx.x & 63)) * 8;
    const bool post = a.flags & kNormPost, pre = a.flags & kNormPre;
    const int slice = blockIdx.x * ROWS + sub, slices = gridDim.x * ROWS;
    const float inv_h = 1.0f / (float)a.H;
    float s_pre[V][8], s_q[V][8];
    auto gain = [&](int v, float (&b)[8]) {   // pre_gain of this lane's columns
        const int c = c0 + v * WAVES * 512;
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = 1.0f;
        if (c < a.H && a.pre_gain) load8<ACT>(a.pre_gain, c, b);
    };
    auto weight = [&](int v, float (&w)[8]) {
        const int c = c0 + v * WAVES * 512;
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = a.scale, g[i] = 1.0f;
        if (c >= a.H) return;
        if (a.post_gain) load8<ACT>(a.post_gain, c, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] *= g[i];
        if (KIND == kGateChannel && a.gate) {
            load8<ACT>(a.gate, c, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] *= g[i];
        }
    };
    // both held over the rows, but in workgroups of 16 waves, whose registers they
    // would overflow (4000 x 8192: 137 us so, 162 held and spilled)
    constexpr bool kHold = WAVES < 16;
    float held_b[kHold ? V : 1][8], held_w[kHold ? V : 1][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s_pre[v][i] = s_q[v][i] = 0.0f;
        if constexpr (kHold) {
            gain(v, held_b[v]);
            weight(v, held_w[v]);
        }
    }
    // every row of a workgroup runs as many rounds, so that all meet at the barriers
    const int64_t rounds = (a.T + slices - 1) / slices;
    for (int64_t n = 0; n < rounds; ++n) {
        const int64_t row = slice + n * slices;
        const bool live = row < a.T;
        const size_t at = (size_t)(live ? row : 0) * a.H;
        float r[V][8], y[V][8], dr[V][8], dx[V][8];
        bool in[V];
        float sums[3] = {0.0f, 0.0f, 0.0f};   // r'^2, h r', y^2
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = c0 + v * WAVES * 512;
            in[v] = live && c < a.H;
#pragma unroll
            for (int i = 0; i < 8; ++i) r[v][i] = y[v][i] = dr[v][i] = dx[v][i] = 0.0f;
            if (!in[v]) continue;
            if (pre) {
                load8<RES>(a.resid_out, at + c, r[v]);
                load8<ACT>(a.d_x, at + c, dx[v]);
            }
            if (a.y) load8<ACT>(a.y, at + c, y[v]);
            if (a.d_resid_out) load8<RES>(a.d_resid_out, at + c, dr[v]);
        }
        const float tok = KIND == kGateToken && live ? load1<ACT>(a.gate, (size_t)row) : 1.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float own[8];
            if constexpr (!kHold) gain(v, own);
            const float(&b)[8] = kHold ? held_b[kHold ? v : 0] : own;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sums[0] += r[v][i] * r[v][i];
                sums[1] += b[i] * dx[v][i] * r[v][i];
                sums[2] += y[v][i] * y[v][i];
            }
        }
        row_sums<3, WAVES>(sums, red[n & 1][sub], wave);
        const float q = pre ? 1.0f / sqrtf(sums[0] * inv_h + a.eps) : 0.0f;
        const float m = q * q * sums[1] * inv_h;   // mean(h u) q
        const float p = post ? 1.0f / sqrtf(sums[2] * inv_h + a.eps) : 1.0f;
        float kn[1] = {0.0f};   // sum of w d r n (full gate: of k n)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!in[v]) continue;
            const int c = c0 + v * WAVES * 512;
            float own[8];
            if constexpr (!kHold) gain(v, own);
            const float(&b)[8] = kHold ? held_b[kHold ? v : 0] : own;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s_pre[v][i] += dx[v][i] * (r[v][i] * q);
                dr[v][i] += q * (b[i] * dx[v][i] - r[v][i] * m);
            }
            store8<RES>(a.d_resid, at + c, dr[v]);
            if (!a.y) continue;
            float g[8], dg[8];
            if (KIND == kGateFull) load8<ACT>(a.gate, at + c, g);
            float own_w[8];
            if constexpr (!kHold) weight(v, own_w);
            const float(&w)[8] = kHold ? held_w[kHold ? v : 0] : own_w;
#pragma unroll
            for (int i = 0; i < 8; ++i) {   // from here on y: n, dr: w d r, and k with a full gate
                y[v][i] *= p;
                const float e = dr[v][i] * y[v][i];
                dr[v][i] *= w[i];
                if constexpr (KIND == kGateFull) {
                    dg[i] = dr[v][i] * y[v][i];
                    s_q[v][i] += g[i] * e;
                    dr[v][i] *= g[i];
                } else {
                    s_q[v][i] += tok * e;
                }
                kn[0] += dr[v][i] * y[v][i];
            }
            if (KIND == kGateFull && a.d_gate) store8<ACT>(a.d_gate, at + c, dg);
        }
        if (!a.y) continue;
        if (post || KIND == kGateToken) row_sums<1, WAVES>(kn, red[2][sub], wave);
        const float mk = post ? kn[0] * inv_h : 0.0f, out = p * tok;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!in[v]) continue;
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = out * (dr[v][i] - y[v][i] * mk);
            store8<ACT>(a.d_y, at + c0 + v * WAVES * 512, t);
        }
        if (KIND == kGateToken && a.d_gate && live && wave == 0 && (threadIdx.x & 63) == 0) static_cast<float *>(a.d_gate)[row] = kn[0];
    }
    // Q times scale and the gate is d post_gain, times scale and post_gain the gate's
    const bool want[3] = {a.d_pre_gain != nullptr, a.d_post_gain != nullptr, KIND == kGateChannel && a.gate && a.d_gate};
    if (ROWS > 1 && (want[0] || want[1] || want[2])) {   // the workgroup's rows side by side: theirs first become one
        __shared__ float side[ROWS > 1 ? ROWS - 1 : 1][WAVES * 512];
        static_assert(ROWS == 1 || V == 1, "one chunk a lane");
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float (&sum)[8] = k == 0 ? s_pre[0] : s_q[0];
            __syncthreads();
            if (sub > 0) store8<kF32>(side[sub - 1], c0, sum);
            __syncthreads();
            if (sub > 0) continue;
#pragma unroll
            for (int o = 0; o < ROWS - 1; ++o) {
                float t[8];
                load8<kF32>(side[o], c0, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] += t[i];
            }
        }
    }
    if (sub > 0) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = c0 + v * WAVES * 512;
        if (c >= a.H) continue;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (!want[k]) continue;
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = 1.0f;
            if (k == 1 && KIND == kGateChannel && a.gate) load8<ACT>(a.gate, c, t);
            if (k == 2 && a.post_gain) load8<ACT>(a.post_gain, c, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = k == 0 ? s_pre[v][i] : a.scale * t[i] * s_q[v][i];
            store8<kF32>(a.parts, ((size_t)k * gridDim.x + blockIdx.x) * a.H + c, t);
        }
    }
}

// out[c] = sum over the slices, 32 columns a workgroup: 8 threads of 4 columns by
// 64 runs of slices, 16 loads of each in flight; the runs are then added in order,
// eight by eight.
__global__ __launch_bounds__(512) void k_norm_parts(const float *parts, int slices, int H, float *d_pre, float *d_post,
                                                    float *d_gate) {
    __shared__ f32x4_t sh[64][8];
    float *out = blockIdx.y == 0 ? d_pre : blockIdx.y == 1 ? d_post : d_gate;
    if (!out) return;
    const int q = threadIdx.x & 7, run = threadIdx.x >> 3;
    const int c = blockIdx.x * 32 + q * 4;
    f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < H) {
        const float *p = parts + (size_t)blockIdx.y * slices * H + c;
#pragma unroll 16
        for (int i = run; i < slices; i += 64) s += *reinterpret_cast<const f32x4_t *>(p + (size_t)i * H);
    }
    sh[run][q] = s;
    __syncthreads();
    if (run < 8) {
        s = sh[8 * run][q];
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sh[8 * run + i][q];
    }
    __syncthreads();
    if (run < 8) sh[run][q] = s;
    __syncthreads();
    if (run == 0 && c < H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sh[i][q];
        *reinterpret_cast<f32x4_t *>(out + c) = s;
    }
}

// Waves a row and chunks a lane by the row's width: the fewest that hold it at
// 8 elements a lane, and four narrow rows (or two of two waves) a workgroup.
template <int ACT, int RES, class F>
static void by_width(int H, F f) {
    if (H <= 512) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
    else if (H <= 1024) f(std::integral_constant<int, 2>{}, std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{});
    else if (H <= 2048) f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
    else if (H <= 4096) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
    else f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
}

template <class F>
static void by_types(int act, int res, F f) {
    typedef std::integral_constant<int, kBf16> B;
    typedef std::integral_constant<int, kF16> H;
    typedef std::integral_constant<int, kF32> S;
    if (act == kF32) f(S{}, S{});
    else if (act == kBf16) { if (res == kF32) f(B{}, S{}); else f(B{}, B{}); }
    else { if (res == kF32) f(H{}, S{}); else f(H{}, H{}); }
}

void launch_norm_residual(const NormArgs &a, int act, int res, hipStream_t s) {
    by_types(act, res, [&](auto A, auto R) {
        by_width<A(), R()>(a.H, [&](auto W, auto V, auto N) {
            const unsigned grid = (unsigned)((a.T + N() - 1) / N());
            hipLaunchKernelGGL((k_norm<A(), R(), W(), V(), N()>), dim3(grid), dim3(64 * W() * N()), 0, s, a);
        });
    });
}

// Workgroups of the backward pass, each of which leaves one partial row: 16 waves
// a CU, which the registers allow.
int norm_back_slices(int64_t T, int H) {
    const int rows = H <= 512 ? 4 : H <= 1024 ? 2 : 1;   // side by side in a workgroup
    const int64_t want = (T + rows - 1) / rows, most = H <= 2048 ? 1024 : H <= 4096 ? 512 : 256;
    return (int)(want < most ? want : most);
}

void launch_norm_residual_backward(const NormBackArgs &a, int act, int res, hipStream_t s) {
    const int slices = norm_back_slices(a.T, a.H);
    if (a.T > 0) {
        by_types(act, res, [&](auto A, auto R) {
            by_width<A(), R()>(a.H, [&](auto W, auto V, auto N) {
                if (a.gate_kind == kGateToken)
                    hipLaunchKernelGGL((k_norm_back<A(), R(), W(), V(), N(), kGateToken>), dim3(slices), dim3(64 * W() * N()), 0, s, a);
                else if (a.gate_kind == kGateFull)
                    hipLaunchKernelGGL((k_norm_back<A(), R(), W(), V(), N(), kGateFull>), dim3(slices), dim3(64 * W() * N()), 0, s, a);
                else
                    hipLaunchKernelGGL((k_norm_back<A(), R(), W(), V(), N(), kGateChannel>), dim3(slices), dim3(64 * W() * N()), 0, s, a);
            });
        });
        if (hipPeekAtLastError() != hipSuccess) return;
    }
    float *gate = a.gate_kind == kGateChannel ? static_cast<float *>(a.d_gate) : nullptr;
    if (a.d_pre_gain || a.d_post_gain || gate)
        hipLaunchKernelGGL(k_norm_parts, dim3((a.H + 31) / 32, 3), dim3(512), 0, s, a.parts, slices, a.H, a.d_pre_gain,
                           a.d_post_gain, gate);
}

}  // namespace moe_w4

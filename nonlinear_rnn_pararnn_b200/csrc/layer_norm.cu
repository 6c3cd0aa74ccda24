// Layer norm, forward and backward, over each of `groups` equal slices of a
// row (one slice: the whole row; a slice for each head behind an attention):
//   y = (x - mean) rstd w + b,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   dx = rstd (p - mean(p) - xhat mean(p xhat)),  p = dy w,  xhat = (x - mean) rstd
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
// A slice is held in the registers of its TPR threads (NV pieces of 8 elements
// each, 16-byte loads where the width and the pointers allow), so x (and dy)
// are read once; the variance is the mean of the squared deviations from the
// mean, not a difference of squares.  All sums are fp32.  Bound by the bytes of
// the tensors: forward 65536 x 1024, fp32 in, bf16 out, 65 us (6.2 TB/s);
// backward 65536 x 8 slices of 128, bf16, 83 us (4.9 TB/s).
//
// dw and db: a block keeps one slice index, walks a strided set of its rows and
// sums them in the registers that hold its columns; the blocks' partial rows
// are added up by a second launch in a fixed order, so the result does not
// change from run to run.
#include <cuda_bf16.h>

#define SLSTM_FILE_ID 12
#include "checked.cuh"
#include "common.cuh"
#include "launchers.h"

namespace slstm {
namespace {

constexpr int LN_THREADS = 256;

SLSTM_DEVINL float ln_f(float v) { return v; }
SLSTM_DEVINL float ln_f(__nv_bfloat16 v) { return __bfloat162float(v); }
SLSTM_DEVINL void ln_put(float *p, float v) { *p = v; }
SLSTM_DEVINL void ln_put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// N elements (4 or 8) by 16-byte accesses, 8-byte ones for four bf16.
template <int N>
SLSTM_DEVINL void load_n(const float *p, float *v)
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p + i);
        v[i] = a.x;
        v[i + 1] = a.y;
        v[i + 2] = a.z;
        v[i + 3] = a.w;
    }
}
template <int N>
SLSTM_DEVINL void load_n(const __nv_bfloat16 *p, float *v)
{
    unsigned w[N / 2];
    if (N == 8) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        w[0] = q.x;
        w[1] = q.y;
        w[N / 2 - 2] = q.z;
        w[N / 2 - 1] = q.w;
    } else {
        const uint2 q = *reinterpret_cast<const uint2 *>(p);
        w[0] = q.x;
        w[1] = q.y;
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <int N>
SLSTM_DEVINL void store_n(float *p, const float *v)
{
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int N>
SLSTM_DEVINL void store_n(__nv_bfloat16 *p, const float *v)
{
    unsigned w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const unsigned *>(&r);
    }
    if (N == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[N / 2 - 2], w[N / 2 - 1]);
    else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

// The columns of a slice's thread `t`, 8 NV of them: W (8, or 4 where a type is
// fp32, so that a warp's 16-byte accesses are consecutive) at a time, or with
// W = 1 (any width and alignment) one at a time, TPR apart.
template <int TPR, int W>
SLSTM_DEVINL int ln_col(int t, int i, int e)
{
    return ((8 / W * i + e / W) * TPR + t) * W + e % W;
}

template <int TPR, int NV, int W, typename T>
SLSTM_DEVINL void ln_load(const T *p, int d, int t, float (&v)[NV][8])
{
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; e += W) {
            const int c = ln_col<TPR, W>(t, i, e);
            if (c < d) {
                if constexpr (W > 1) load_n<W>(p + c, &v[i][e]);
                else v[i][e] = ln_f(p[c]);
            } else {
#pragma unroll
                for (int k = 0; k < W; ++k) v[i][e + k] = 0.0f;
            }
        }
}

// (base, n: the tensor that p points into, for the bounds-checked build)
template <int TPR, int NV, int W, typename T>
SLSTM_DEVINL void ln_store(T *p, int d, int t, const float (&v)[NV][8], [[maybe_unused]] const T *base,
                           [[maybe_unused]] long long n)
{
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; e += W) {
            const int c = ln_col<TPR, W>(t, i, e);
            if (c < d && SLSTM_PIN(p + c + W - 1, base, n)) {
                if constexpr (W > 1) store_n<W>(p + c, &v[i][e]);
                else ln_put(p + c, v[i][e]);
            }
        }
}

// A thread's columns as they are stored: bf16 pairs stay packed.
template <typename T, int NV, int W>
struct LnRaw {
    float v[NV][8];
    template <int TPR>
    SLSTM_DEVINL void load(const T *p, int d, int t)
    {
        ln_load<TPR, NV, W>(p, d, t, v);
    }
    SLSTM_DEVINL void get(float (&o)[NV][8]) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[i][e] = v[i][e];
    }
};
template <int NV>
struct LnRaw<__nv_bfloat16, NV, 8> {
    uint4 v[NV];
    template <int TPR>
    SLSTM_DEVINL void load(const __nv_bfloat16 *p, int d, int t)
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = ln_col<TPR, 8>(t, i, 0);
            v[i] = c < d ? *reinterpret_cast<const uint4 *>(p + c) : make_uint4(0, 0, 0, 0);
        }
    }
    SLSTM_DEVINL void get(float (&o)[NV][8]) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const unsigned w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                o[i][2 * k] = __uint_as_float(w[k] << 16);
                o[i][2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
        }
    }
};

// Sums of `a` and `b` over the TPR threads of a slice, to all of them.
template <int TPR>
SLSTM_DEVINL float2 ln_sum(float a, float b, float2 *red)
{
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (TPR <= 32) return make_float2(a, b);
    constexpr int W = TPR / 32;
    const int slot = threadIdx.x / TPR, w = (threadIdx.x % TPR) >> 5;
    __syncthreads();   // the values of the last sum have been read
    if ((threadIdx.x & 31) == 0) red[slot * W + w] = make_float2(a, b);
    __syncthreads();
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float2 r = red[slot * W + i];
        s.x += r.x;
        s.y += r.y;
    }
    return s;
}

template <int TPR>
constexpr int ln_block()
{
    return TPR > LN_THREADS ? TPR : LN_THREADS;
}

template <typename TX, typename TY, int TPR, int NV, int W>
__global__ void __launch_bounds__(ln_block<TPR>())
    ln_forward_kernel(const TX *__restrict__ x, const float *__restrict__ w, const float *__restrict__ b, TY *y,
                      float *mean, float *rstd, long long n, int groups, int d, float eps)
{
    constexpr int SLOTS = ln_block<TPR>() / TPR;
    __shared__ float2 red[32];
    const int t = threadIdx.x % TPR;
    const long long r = (long long)blockIdx.x * SLOTS + threadIdx.x / TPR;
    const bool on = r < n;
    const long long at = (on ? r : 0) * d;
    const int g0 = (int)((on ? r : 0) % groups) * d;
    float v[NV][8];
    // (a slot without a row reads none: y may be x, and another block's to write)
    ln_load<TPR, NV, W>(x + at, on ? d : 0, t, v);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[i][e];
    const float mu = ln_sum<TPR>(s, 0.0f, red).x / d;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[i][e] -= mu;
            if (ln_col<TPR, W>(t, i, e) < d) q = fmaf(v[i][e], v[i][e], q);
        }
    const float rs = 1.0f / sqrtf(ln_sum<TPR>(q, 0.0f, red).x / d + eps);
    if (!on) return;
    if (t == 0 && SLSTM_IN(r, n)) {
        mean[r] = mu;
        rstd[r] = rs;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float wv[1][8], bv[1][8];
        ln_load<TPR, 1, W>(w + g0 + i * TPR * 8, d - i * TPR * 8, t, wv);
        if (b) ln_load<TPR, 1, W>(b + g0 + i * TPR * 8, d - i * TPR * 8, t, bv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[i][e] = v[i][e] * rs * wv[0][e];
            if (b) v[i][e] += bv[0][e];
        }
    }
    ln_store<TPR, NV, W>(y + at, d, t, v, y, n * d);
}

// part: [gridDim.x][2][groups d], the blocks' sums of dy xhat and dy.
template <typename TX, typename TY, int TPR, int NV, int W>
__global__ void __launch_bounds__(ln_block<TPR>())
    ln_backward_kernel(const TX *__restrict__ x, const float *__restrict__ w, const TY *__restrict__ dy,
                       const float *__restrict__ mean, const float *__restrict__ rstd, TX *dx, float *part,
                       long long rows, int groups, int d)
{
    constexpr int SLOTS = ln_block<TPR>() / TPR;
    __shared__ float2 red[32];
    __shared__ float join[SLOTS > 1 ? SLOTS : 1][SLOTS > 1 ? 8 * TPR : 1];
    const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    const int g = blockIdx.y;
    float wv[NV][8], dw[NV][8], db[NV][8];
    ln_load<TPR, NV, W>(w + (long long)g * d, d, t, wv);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.0f;
    // the next row is on its way while this one is summed, as it is stored, where
    // barriers hold a block's threads together anyway; slices of a warp or less
    // hide their loads behind one another
    constexpr bool AHEAD = TPR > 32;
    const long long step = (long long)gridDim.x * SLOTS;
    LnRaw<TX, NV, W> xn;
    LnRaw<TY, NV, W> yn;
    float mn = 0.0f, rn = 0.0f;
    auto fetch = [&](long long r) {
        const long long n = (r < rows ? r : 0) * groups + g;
        const int w = r < rows ? d : 0;   // no row, no reads: dx may be dy
        xn.template load<TPR>(x + n * d, w, t);
        yn.template load<TPR>(dy + n * d, w, t);
        mn = mean[n];
        rn = rstd[n];
    };
    if (AHEAD) fetch((long long)blockIdx.x * SLOTS + slot);
    for (long long r0 = (long long)blockIdx.x * SLOTS; r0 < rows; r0 += step) {
        const long long r = r0 + slot;
        const bool on = r < rows;
        const long long n = (on ? r : 0) * groups + g;
        if (!AHEAD) fetch(r);
        float xv[NV][8], yv[NV][8];
        xn.get(xv);
        yn.get(yv);
        const float mu = mn, rs = rn;
        if (AHEAD && r0 + step < rows) fetch(r + step);
        float sp = 0.0f, sx = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (xv[i][e] - mu) * rs;
                const float p = yv[i][e] * wv[i][e];   // 0 behind the slice: dy and w are
                if (on) {
                    dw[i][e] = fmaf(yv[i][e], xh, dw[i][e]);
                    db[i][e] += yv[i][e];
                }
                sp += p;
                sx = fmaf(p, xh, sx);
                xv[i][e] = xh;
                yv[i][e] = p;
            }
        const float2 s = ln_sum<TPR>(sp, sx, red);
        const float mp = s.x / d, mx = s.y / d;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) xv[i][e] = rs * (yv[i][e] - mp - xv[i][e] * mx);
        if (on) ln_store<TPR, NV, W>(dx + n * d, d, t, xv, dx, rows * groups * d);
    }
    // the block's sums, its slots in order
    float *pw = part + (long long)blockIdx.x * 2 * groups * d + (long long)g * d;
    [[maybe_unused]] const long long all = (long long)gridDim.x * 2 * groups * d;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float(&v)[8] = z == 0 ? dw[i] : db[i];
            if (SLOTS > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 8; ++e) join[slot][e * TPR + t] = v[e];
                __syncthreads();
                for (int j = threadIdx.x; j < 8 * TPR; j += ln_block<TPR>()) {
                    float s = 0.0f;
#pragma unroll 8
                    for (int k = 0; k < SLOTS; ++k) s += join[k][j];
                    const int c = ln_col<TPR, W>(j % TPR, i, j / TPR);
                    if (c < d && SLSTM_PIN(pw + (long long)z * groups * d + c, part, all))
                        pw[(long long)z * groups * d + c] = s;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = ln_col<TPR, W>(t, i, e);
                    if (c < d && SLSTM_PIN(pw + (long long)z * groups * d + c, part, all))
                        pw[(long long)z * groups * d + c] = v[e];
                }
            }
        }
    }
}

// out[c] = sum over k of part[k][c], c < 2 D (dw, then db): 32 columns and 8
// strided shares of the partial rows a block, the shares in order.
__global__ void __launch_bounds__(256) ln_reduce_kernel(const float *__restrict__ part, float *dw, float *db, int nb,
                                                        long long D)
{
    __shared__ float s[8][33];
    const long long c = (long long)blockIdx.x * 32 + (threadIdx.x & 31);
    const int y = threadIdx.x >> 5;
    float v = 0.0f;
    if (c < 2 * D)
#pragma unroll 8
        for (int k = y; k < nb; k += 8) v += part[k * 2 * D + c];
    s[y][threadIdx.x & 31] = v;
    __syncthreads();
    if (y == 0 && c < 2 * D) {
#pragma unroll
        for (int k = 1; k < 8; ++k) v += s[k][threadIdx.x];
        if (c < D) {
            if (SLSTM_IN(c, D)) dw[c] = v;
        } else if (SLSTM_IN(c - D, D)) {
            db[c - D] = v;
        }
    }
}

bool vec_ok(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Blocks that share the rows of one slice index in the backward pass: a few for
// every SM over all slice indices, so that the partial rows stay small beside
// the tensors.
int backward_blocks(long long rows, int groups, int slots)
{
    const long long want = max((148LL * 4 + groups - 1) / groups, 1LL);
    return (int)min(want, (rows + slots - 1) / slots);
}

// The threads and pieces of a slice of d columns, measured on both sides (2^26
// elements, bf16 / fp32 / fp32 to bf16, us; twice and half the threads, where
// another choice was near).
// Forward: 16 columns a thread up to 512, 32 above.
//   d          64        128        256        512       2048       4096       8192      16384
//   taken   66 86 82   62 84 70   62 82 70   64 82 71   70 86 70   70 85 70   66 86 70   78 133 108
//   twice   80 88 78   82 89 79   82 90 80   90 98 89   70 86 76   72 84 70   94 104 90  135 153 131
//   half   108 154 142 68 101 80  66 92 66   66 92 66                83 131 72            102 145 76
// Up to 1024 the sums need no barriers (65536 x 1024 fp32 to bf16 in 65 us; four
// warps took 100).
#define LN_FWD(F)                            \
    (d <= 64     ? F<TX, TY, 4, 2, W>(a)     \
     : d <= 128  ? F<TX, TY, 8, 2, W>(a)     \
     : d <= 256  ? F<TX, TY, 16, 2, W>(a)    \
     : d <= 512  ? F<TX, TY, 32, 2, W>(a)    \
     : d <= 1024 ? F<TX, TY, 32, 4, W>(a)    \
     : d <= 2048 ? F<TX, TY, 64, 4, W>(a)    \
     : d <= 4096 ? F<TX, TY, 128, 4, W>(a)   \
     : d <= 8192 ? F<TX, TY, 256, 4, W>(a)   \
                 : F<TX, TY, 512, 4, W>(a))
// Backward: x, dy, w and the sums of dw and db are all in registers, which bounds
// the columns of a thread: 8 up to 256, 16 to 32 above, by the types where the
// sides differ (those taken in brackets).
//   d            64          128         256          512         2048           4096          8192           16384
//   taken     89 131 113  85 131 110  86 131 109   115 146 117  [90 163] 190  109 [139 174] 149 151 176   281 420 368
//   twice    145 174 155 142 178 153 186 201 272   113 147 164  125 199 [172] [104] 183 205 139 188 171
//   half     133 137 138 122 131 140 114 149 132   126 150 158   99 135 173   341 697 615
// (up to 1024: at ln_bwd_d; above 8192 all bf16 takes 319 us the other way, fp32
// 863, fp32 to bf16 365)
#define LN_BWD(F, T1024, N1024, T2048, N2048, T4096, N4096, TMAX, NMAX) \
    (d <= 64     ? F<TX, TY, 8, 1, W>(a)                                \
     : d <= 128  ? F<TX, TY, 16, 1, W>(a)                               \
     : d <= 256  ? F<TX, TY, 32, 1, W>(a)                               \
     : d <= 512  ? F<TX, TY, 32, 2, W>(a)                               \
     : d <= 1024 ? F<TX, TY, T1024, N1024, W>(a)                        \
     : d <= 2048 ? F<TX, TY, T2048, N2048, W>(a)                        \
     : d <= 4096 ? F<TX, TY, T4096, N4096, W>(a)                        \
     : d <= 8192 ? F<TX, TY, 256, 4, W>(a)                              \
                 : F<TX, TY, TMAX, NMAX, W>(a))

struct LnArgs {
    const void *x, *dy;
    const float *w, *b, *mean_in, *rstd_in;
    void *y, *dx;
    float *mean, *rstd, *dw, *db, *part;
    long long rows;
    int groups, d;
    float eps;
    cudaStream_t st;
};

template <typename TX, typename TY, int TPR, int NV, int W>
cudaError_t ln_fwd(const LnArgs &a)
{
    constexpr int SLOTS = ln_block<TPR>() / TPR;
    const long long n = a.rows * a.groups;
    ln_forward_kernel<TX, TY, TPR, NV, W><<<(unsigned)((n + SLOTS - 1) / SLOTS), ln_block<TPR>(), 0, a.st>>>(
        static_cast<const TX *>(a.x), a.w, a.b, static_cast<TY *>(a.y), a.mean, a.rstd, n, a.groups, a.d, a.eps);
    return cudaGetLastError();
}

template <typename TX, typename TY, int TPR, int NV, int W>
cudaError_t ln_bwd(const LnArgs &a)
{
    constexpr int SLOTS = ln_block<TPR>() / TPR;
    const int nb = backward_blocks(a.rows, a.groups, SLOTS);
    ln_backward_kernel<TX, TY, TPR, NV, W><<<dim3(nb, a.groups), ln_block<TPR>(), 0, a.st>>>(
        static_cast<const TX *>(a.x), a.w, static_cast<const TY *>(a.dy), a.mean_in, a.rstd_in,
        static_cast<TX *>(a.dx), a.part, a.rows, a.groups, a.d);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long D = (long long)a.groups * a.d;
    ln_reduce_kernel<<<(unsigned)((2 * D + 31) / 32), 256, 0, a.st>>>(a.part, a.dw, a.db, nb, D);
    return cudaGetLastError();
}

template <typename TX, typename TY, int W>
cudaError_t ln_fwd_d(const LnArgs &a)
{
    const int d = a.d;
    return LN_FWD(ln_fwd);
}
template <typename TX, typename TY, int W>
cudaError_t ln_bwd_d(const LnArgs &a)
{
    const int d = a.d;
    // all bf16: two warps of 16 columns a thread (65536 x 1024 in 88 us; four warps of
    // 8 take 119), with fp32, twice the registers, four (165 and 185 us)
    if constexpr (W == 8) return LN_BWD(ln_bwd, 64, 2, 128, 2, 256, 2, 1024, 2);
    else if constexpr (sizeof(TX) == sizeof(TY)) return LN_BWD(ln_bwd, 128, 1, 128, 2, 128, 4, 256, 8);
    else return LN_BWD(ln_bwd, 128, 1, 256, 1, 128, 4, 256, 8);
}

}  // namespace

size_t layer_norm_workspace_bytes(long long rows, int groups, int d)
{
    return (size_t)backward_blocks(rows, groups, 1) * 2 * groups * d * 4;
}

cudaError_t layer_norm_forward(const void *x, int x_dtype, const float *w, const float *b, void *y, int y_dtype,
                               float *mean, float *rstd, long long rows, int groups, int d, float eps, cudaStream_t st)
{
    LnArgs a{};
    a.x = x;
    a.w = w;
    a.b = b;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.rows = rows;
    a.groups = groups;
    a.d = d;
    a.eps = eps;
    a.st = st;
    const bool v = d % 8 == 0 && vec_ok(x) && vec_ok(w) && vec_ok(y) && (b == nullptr || vec_ok(b));
    const bool xf = x_dtype == SLSTM_F32, yf = y_dtype == SLSTM_F32;
    typedef __nv_bfloat16 h;
    if (xf && yf) return v ? ln_fwd_d<float, float, 4>(a) : ln_fwd_d<float, float, 1>(a);
    if (xf) return v ? ln_fwd_d<float, h, 4>(a) : ln_fwd_d<float, h, 1>(a);
    if (yf) return v ? ln_fwd_d<h, float, 4>(a) : ln_fwd_d<h, float, 1>(a);
    return v ? ln_fwd_d<h, h, 8>(a) : ln_fwd_d<h, h, 1>(a);
}

cudaError_t layer_norm_backward(const void *x, int x_dtype, const float *w, const void *dy, int y_dtype,
                                const float *mean, const float *rstd, void *dx, float *dw, float *db, long long rows,
                                int groups, int d, void *ws, cudaStream_t st)
{
    LnArgs a{};
    a.x = x;
    a.w = w;
    a.dy = dy;
    a.mean_in = mean;
    a.rstd_in = rstd;
    a.dx = dx;
    a.dw = dw;
    a.db = db;
    a.part = static_cast<float *>(ws);
    a.rows = rows;
    a.groups = groups;
    a.d = d;
    a.st = st;
    const bool v = d % 8 == 0 && vec_ok(x) && vec_ok(w) && vec_ok(dy) && vec_ok(dx);
    const bool xf = x_dtype == SLSTM_F32, yf = y_dtype == SLSTM_F32;
    typedef __nv_bfloat16 h;
    if (xf && yf) return v ? ln_bwd_d<float, float, 4>(a) : ln_bwd_d<float, float, 1>(a);
    if (xf) return v ? ln_bwd_d<float, h, 4>(a) : ln_bwd_d<float, h, 1>(a);
    if (yf) return v ? ln_bwd_d<h, float, 4>(a) : ln_bwd_d<h, float, 1>(a);
    return v ? ln_bwd_d<h, h, 8>(a) : ln_bwd_d<h, h, 1>(a);
}

}  // namespace slstm

// Linear attention with a decay for each head, on the CUDA cores: every size,
// fp32 and bf16, dense and packed; the step of single tokens; and the small
// kernels that the tensor-core path (linear_attention_tc.cu) shares.
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
//
// Over a chunk of C rows, with c_i the sum of the log decays up to row i:
//   o_i     = scale (sum_{j<=i} D_ij (q_i . k_j) v_j + e^{c_i} S_n^T q_i),  D_ij = e^{c_i - c_j}
//   S_{n+1} = e^{c_C} S_n + sum_j e^{c_C - c_j} k_j v_j^T
// so three launches do it, all parallel over chunks but the second: what each
// chunk adds to the state, the scan of the states over the chunks (one thread
// for each state element), and the outputs.  The backward pass runs the same
// first two launches on (q, dO) from the end for dS and one more for the rest:
//   dq_i = scale (sum_j D_ij (dO_i . v_j) k_j + e^{c_i} S_n dO_i)
//   dk_j = scale sum_i D_ij (dO_i . v_j) q_i + e^{c_C - c_j} dS_{n+1} v_j
//   dv_j = scale sum_i D_ij (q_i . k_j) dO_i + e^{c_C - c_j} dS_{n+1}^T k_j
//   dg_t = sum_{i>=t>j} W_ij + sum_{i>=t} u_i + sum_{j<t} w_j + e^{c_C} <S_n, dS_{n+1}>
// with W_ij = scale D_ij (q_i . k_j)(dO_i . v_j), u_i = q_i . (the state part of
// dq_i), w_j = k_j . (the state part of dk_j).  dg is put together inside its
// chunk: the sum of q . dq - k . dk over all later rows is the same number, but
// cancels over the whole row and keeps little of it.
//
// All products are fp32 fused multiply-adds over 64 x 64 tiles (RT x 4 for each
// of 1024 / RT threads), the next 32 of the depth on their way from memory
// meanwhile; fp32 in, fp32 out needs that, and sizes that are no multiple
// of 8 come here too.  Bound: the FMA pipes, of
// which the gradients of 8 x 1024 rows, 4 heads of 64, keep a third busy (fetching
// instructions and operands the rest of the time).
#include <cuda_bf16.h>

#define SLSTM_FILE_ID 11
#include "checked.cuh"
#include "la.cuh"
#include "launchers.h"

namespace slstm {
namespace {

constexpr int LC = 64;        // rows of a chunk
constexpr int KB = 32;        // depth of the tiles in shared memory
constexpr int LDT = 68;       // padded row of a tile (floats)
// Rows of a thread's tile.  8: 128 threads, the fewest reads of shared memory for
// a multiply-add, where the blocks fill the GPU; 4: 256 threads, twice the warps
// to hide the latencies behind, where they do not (2 x 777 rows, 4 heads of 64:
// 25 and 40 us; gradients of 8 x 1024 rows: 200 and 127).
template <int RT>
constexpr int nt() { return 1024 / RT; }
template <int RT>
constexpr int nf() { return 64 * KB / nt<RT>(); }   // elements of a tile that a thread fetches

SLSTM_DEVINL float to_f(float v) { return v; }
SLSTM_DEVINL float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
SLSTM_DEVINL void put(float *p, float v) { *p = v; }
SLSTM_DEVINL void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

[[maybe_unused]] SLSTM_DEVINL long long la_rows(const LaArgs &a)
{
    return a.cu ? (long long)a.T : (long long)a.B * a.T;
}

// An operand of a 64 x 64 product: element (m, k) at p[m sm + k sk] for
// m < nm, k < nk, zero outside, times coef[k] where given.
template <typename T>
struct Op {
    const T *p;
    long long sm, sk;
    int nm, nk;
    const float *coef;
};

// Thread t's elements of the 64 x KB tiles of an operand, and where they go in
// shared memory.  Where k is contiguous in memory a warp's lanes take the 32 k
// of four rows m and write the four of a lane at once (one by one, 32 rows of
// shared memory apart, they would meet in the same banks); where m is, 32 m.
template <typename T, int RT>
struct Feed {
    const T *p;           // the first element at depth 0
    int m, k;
    bool kc;
    SLSTM_DEVINL explicit Feed(const Op<T> &a)
    {
        const int t = threadIdx.x;
        kc = a.sk == 1;
        m = kc ? 4 * (t / KB) : t % 64;
        k = kc ? t % KB : t / 64;
        p = a.p + m * a.sm + k * a.sk;
    }
    SLSTM_DEVINL static constexpr int dm(int i) { return (i & 3) + (i >> 2) * 4 * (nt<RT>() / KB); }
    SLSTM_DEVINL static constexpr int dk(int i) { return i * (nt<RT>() / 64); }
    SLSTM_DEVINL void fetch(float (&v)[nf<RT>()], const Op<T> &a, int k0) const
    {
        const T *q = p + k0 * a.sk;
        if (kc) {
            const bool on = k0 + k < a.nk;
            const float w = a.coef && on ? a.coef[k0 + k] : 1.0f;
#pragma unroll
            for (int i = 0; i < nf<RT>(); ++i) v[i] = on && m + dm(i) < a.nm ? to_f(q[dm(i) * a.sm]) : 0.0f;
            if (a.coef)
#pragma unroll
                for (int i = 0; i < nf<RT>(); ++i) v[i] *= w;
        } else {
            const bool on = m < a.nm;
#pragma unroll
            for (int i = 0; i < nf<RT>(); ++i) {
                const int kk = k0 + k + dk(i);
                v[i] = on && kk < a.nk ? to_f(q[dk(i) * a.sk]) : 0.0f;
                if (a.coef) v[i] *= kk < a.nk ? a.coef[kk] : 0.0f;
            }
        }
    }
    SLSTM_DEVINL void stow(float *dst, const float (&v)[nf<RT>()]) const
    {
        if (kc) {
#pragma unroll
            for (int i = 0; i < nf<RT>(); i += 4)
                *reinterpret_cast<float4 *>(dst + k * LDT + m + dm(i)) =
                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < nf<RT>(); ++i) dst[(k + dk(i)) * LDT + m] = v[i];
        }
    }
};

// acc += A B^T over k < K: thread (ty, tx) = (t / 16, t % 16) holds rows
// RT ty .. and columns 4 tx ...
template <int RT, typename TA, typename TB>
SLSTM_DEVINL void product(float (&acc)[RT][4], const Op<TA> &A, const Op<TB> &B, int K, float *sA, float *sB)
{
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    float va[nf<RT>()], vb[nf<RT>()];
    const Feed<TA, RT> fa(A);
    const Feed<TB, RT> fb(B);
    // what an operand in shared memory was written by is behind this barrier
    __syncthreads();
    fa.fetch(va, A, 0);
    fb.fetch(vb, B, 0);
    for (int k0 = 0; k0 < K; k0 += KB) {
        if (k0 > 0) __syncthreads();
        fa.stow(sA, va);
        fb.stow(sB, vb);
        __syncthreads();
        if (k0 + KB < K) {
            fa.fetch(va, A, k0 + KB);
            fb.fetch(vb, B, k0 + KB);
        }
#pragma unroll 8
        for (int k = 0; k < KB; ++k) {
            float av[RT], bv[4];
#pragma unroll
            for (int i = 0; i < RT; i += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(sA + k * LDT + ty * RT + i);
                av[i] = a.x;
                av[i + 1] = a.y;
                av[i + 2] = a.z;
                av[i + 3] = a.w;
            }
            const float4 b = *reinterpret_cast<const float4 *>(sB + k * LDT + tx * 4);
            bv[0] = b.x;
            bv[1] = b.y;
            bv[2] = b.z;
            bv[3] = b.w;
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
    }
}

template <int RT>
SLSTM_DEVINL void clear(float (&acc)[RT][4])
{
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
}

struct Decays {
    double cum[LC];
    int first[LC];
    float row[LC], col[LC];
    float tot;
};

SLSTM_DEVINL void chunk_decays(Decays &d, const LaArgs &a, const LaChunk &c, int h)
{
    if (threadIdx.x < 32)
        la_decays<LC / 32>(a.g, a.per_head ? h : c.row * a.H + h, a.per_head ? 0 : a.H, c.len, threadIdx.x, d.cum,
                           d.first, d.row, d.col, &d.tot);
    __syncthreads();
}

// e^{c_i - c_j} for j <= i < len of one run between clears, else 0.
SLSTM_DEVINL float decay_ij(const Decays &d, int i, int j, int len)
{
    return (j <= i && i < len && j >= d.first[i]) ? exp2f((float)(d.cum[i] - d.cum[j])) : 0.0f;
}

// What a chunk adds to the state: out[c][h] (d_k x d_v) = sum_j w_j X_j Y_j^T,
// with X = k, Y = v, w = e^{c_C - c_j} forward, or X = q, Y = dO,
// w = scale e^{c_i} from the end.
template <typename T, int RT>
__global__ void __launch_bounds__(nt<RT>(), RT == 8 ? 5 : 2)
    la_delta_kernel(LaArgs a, LaChunks ch, bool back, float *out, float *tot)
{
    __shared__ __align__(16) float sA[KB * LDT], sB[KB * LDT];
    __shared__ Decays d;
    __shared__ float w[LC];
    const int c = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const LaChunk ck = la_chunk(ch, c);
    if (ck.len <= 0) return;
    const int m0 = blockIdx.y * 64, n0 = blockIdx.z * 64;
    chunk_decays(d, a, ck, h);
    if (threadIdx.x < LC) w[threadIdx.x] = back ? a.scale * d.row[threadIdx.x] : d.col[threadIdx.x];
    if (threadIdx.x == 0 && m0 == 0 && n0 == 0) tot[(long long)c * a.H + h] = d.tot;
    const int hq = h / (a.H / a.Hqk);
    const long long ldx = back ? a.ldq : a.ldk, ldy = back ? (long long)a.H * a.dv : a.ldv;
    const T *X = static_cast<const T *>(back ? a.q : a.k) + ck.row * ldx + (long long)hq * a.dk + m0;
    const T *Y = static_cast<const T *>(back ? a.dO : a.v) + ck.row * ldy + (long long)h * a.dv + n0;
    float acc[RT][4];
    clear(acc);
    product(acc, Op<T>{X, 1, ldx, a.dk - m0, ck.len, w}, Op<T>{Y, 1, ldy, a.dv - n0, ck.len, nullptr}, ck.len, sA, sB);
    float *dst = out + ((long long)c * a.H + h) * a.dk * a.dv;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty * RT + i, n = n0 + tx * 4 + j;
            if (m < a.dk && n < a.dv &&
                SLSTM_PIN(dst + (long long)m * a.dv + n, out, (long long)ch.total * a.H * a.dk * a.dv))
                dst[(long long)m * a.dv + n] = acc[i][j];
        }
}

// The states over the chunks of each sequence, V elements a thread: the deltas
// in `buf` give way to the state that enters each chunk (forward) or the
// gradient of the state that leaves it (back).  first: s0 or dsT (null: zero);
// last: sT or ds0 (may be null).  Bound by the bytes of buf, read and written
// once; eight chunks are loaded at a time, ahead of their joining.
template <int V>
__global__ void __launch_bounds__(128) la_scan_kernel(LaChunks ch, int H, int E, bool back, float *buf,
                                                      const float *__restrict__ tot, const float *first, float *last,
                                                      int skip)
{
    const int e = (blockIdx.y * 128 + threadIdx.x) * V;
    const int seq = blockIdx.x / H, h = blockIdx.x % H;
    if (e >= E) return;
    const int c0 = ch.pos ? ch.coff[seq] : seq * ch.nc;
    const int n = ch.pos ? ch.coff[seq + 1] - c0 : ch.nc;
    if (n == skip) return;
    const long long at = ((long long)seq * H + h) * E + e;
    auto load = [](const float *p, float (&v)[V]) {
        if (V == 4) {
            const float4 f = *reinterpret_cast<const float4 *>(p);
            v[0] = f.x;
            v[V > 1 ? 1 : 0] = f.y;
            v[V > 2 ? 2 : 0] = f.z;
            v[V > 3 ? 3 : 0] = f.w;
        } else {
            v[0] = *p;
        }
    };
    auto store = [](float *p, const float (&v)[V]) {
        if (V == 4)
            *reinterpret_cast<float4 *>(p) =
                make_float4(v[0], v[V > 1 ? 1 : 0], v[V > 2 ? 2 : 0], v[V > 3 ? 3 : 0]);
        else
            *p = v[0];
    };
    float s[V];
#pragma unroll
    for (int k = 0; k < V; ++k) s[k] = 0.0f;
    if (first) load(first + at, s);
    const long long step = (back ? -1LL : 1LL) * H * E;
    float *p = buf + ((long long)(back ? c0 + n - 1 : c0) * H + h) * E + e;
    const float *t = tot + (long long)(back ? c0 + n - 1 : c0) * H + h;
    const int ts = back ? -H : H;
    for (int i0 = 0; i0 < n; i0 += 8, p += 8 * step, t += 8 * ts) {
        float dl[8][V], tt[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i0 + i < n) {
                load(p + i * step, dl[i]);
                tt[i] = t[i * ts];
            }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i0 + i < n) {
                if (SLSTM_PIN(p + i * step + V - 1, buf, (long long)ch.total * H * E)) store(p + i * step, s);
#pragma unroll
                for (int k = 0; k < V; ++k) s[k] = la_carry(tt[i], s[k], dl[i][k]);
            }
    }
    if (last && SLSTM_IN(at + V - 1, (long long)ch.n_seq * H * E)) store(last + at, s);
}

// The outputs of a chunk and head.
template <typename T, int RT>
__global__ void __launch_bounds__(nt<RT>(), RT == 8 ? 5 : 2)
    la_out_kernel(LaArgs a, LaChunks ch, const float *__restrict__ states)
{
    __shared__ __align__(16) float sA[KB * LDT], sB[KB * LDT];
    __shared__ float P[LC][LC + 1];
    __shared__ Decays d;
    const int c = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const LaChunk ck = la_chunk(ch, c);
    if (ck.len <= 0) return;
    chunk_decays(d, a, ck, h);
    const int hq = h / (a.H / a.Hqk);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const T *q = static_cast<const T *>(a.q) + ck.row * a.ldq + (long long)hq * a.dk;
    const T *k = static_cast<const T *>(a.k) + ck.row * a.ldk + (long long)hq * a.dk;
    const T *v = static_cast<const T *>(a.v) + ck.row * a.ldv + (long long)h * a.dv;
    const float *S = states + ((long long)c * a.H + h) * a.dk * a.dv;
    T *o = static_cast<T *>(a.o) + ck.row * (long long)a.H * a.dv + (long long)h * a.dv;
    float acc[RT][4];
    clear(acc);
    product(acc, Op<T>{q, a.ldq, 1, ck.len, a.dk, nullptr}, Op<T>{k, a.ldk, 1, ck.len, a.dk, nullptr}, a.dk, sA, sB);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = ty * RT + i, s = tx * 4 + j;
            const float w = decay_ij(d, r, s, ck.len);
            P[r][s] = w == 0.0f ? 0.0f : acc[i][j] * w;
        }
    for (int n0 = 0; n0 < a.dv; n0 += 64) {
        clear(acc);
        product(acc, Op<T>{q, a.ldq, 1, ck.len, a.dk, nullptr}, Op<float>{S + n0, 1, a.dv, a.dv - n0, a.dk, nullptr},
                a.dk, sA, sB);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const float r = d.row[ty * RT + i];
            const bool on = d.first[ty * RT + i] < 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = on ? acc[i][j] * r : 0.0f;
        }
        product(acc, Op<float>{&P[0][0], LC + 1, 1, LC, ck.len, nullptr},
                Op<T>{v + n0, 1, a.ldv, a.dv - n0, ck.len, nullptr}, ck.len, sA, sB);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty * RT + i, n = n0 + tx * 4 + j;
                if (r < ck.len && n < a.dv &&
                    SLSTM_PIN(o + (long long)r * a.H * a.dv + n, static_cast<T *>(a.o), la_rows(a) * a.H * a.dv))
                    put(o + (long long)r * a.H * a.dv + n, acc[i][j] * a.scale);
            }
    }
}

// Sum over the 16 threads that share rows (half a warp).
SLSTM_DEVINL float sum16(float v)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct BackShared {
    float sA[KB * LDT], sB[KB * LDT];
    float P[LC][LC + 1], Pd[LC][LC + 1];
    float r[LC], u[LC], w[LC];
    float cs[16][LC];     // column sums of W of each thread row
    float red[8];
    Decays d;
};

// The gradients of a chunk and head.  part_q, part_k: [row][h][d_k] fp32 where
// heads share a query and key head; dgc: the chunk's sum of dg, [c][h], where
// the decay belongs to the head.
template <typename T, int RT>
__global__ void __launch_bounds__(nt<RT>(), RT == 8 ? 4 : 2)
    la_back_kernel(LaArgs a, LaChunks ch, const float *__restrict__ states, const float *__restrict__ dstates,
                   float *part_q, float *part_k, float *dgc)
{
    extern __shared__ __align__(16) char smem[];
    BackShared &s = *reinterpret_cast<BackShared *>(smem);
    const int c = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const LaChunk ck = la_chunk(ch, c);
    if (ck.len <= 0) return;
    chunk_decays(s.d, a, ck, h);
    const int len = ck.len;
    const int hq = h / (a.H / a.Hqk);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const long long ldo = (long long)a.H * a.dv;
    const T *q = static_cast<const T *>(a.q) + ck.row * a.ldq + (long long)hq * a.dk;
    const T *k = static_cast<const T *>(a.k) + ck.row * a.ldk + (long long)hq * a.dk;
    const T *v = static_cast<const T *>(a.v) + ck.row * a.ldv + (long long)h * a.dv;
    const T *g = static_cast<const T *>(a.dO) + ck.row * ldo + (long long)h * a.dv;
    const float *S = states + ((long long)c * a.H + h) * a.dk * a.dv;
    const float *dS = dstates + ((long long)c * a.H + h) * a.dk * a.dv;
    for (int i = threadIdx.x; i < LC; i += nt<RT>()) s.u[i] = s.w[i] = 0.0f;

    // D (q k) and scale D (dO v), their products' sums over rows and columns
    float p[RT][4], t[RT][4];
    clear(p);
    clear(t);
    product(p, Op<T>{q, a.ldq, 1, len, a.dk, nullptr}, Op<T>{k, a.ldk, 1, len, a.dk, nullptr}, a.dk, s.sA, s.sB);
    product(t, Op<T>{g, ldo, 1, len, a.dv, nullptr}, Op<T>{v, a.ldv, 1, len, a.dv, nullptr}, a.dv, s.sA, s.sB);
    float cs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        float rs = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = ty * RT + i, m = tx * 4 + j;
            const float w = a.scale * decay_ij(s.d, r, m, len);
            const float P = w == 0.0f ? 0.0f : w * p[i][j], Pd = w == 0.0f ? 0.0f : w * t[i][j];
            s.P[r][m] = P;
            s.Pd[r][m] = Pd;
            const float W = r > m && w != 0.0f ? P * t[i][j] : 0.0f;
            rs += W;
            cs[j] += W;
        }
        rs = sum16(rs);
        if (tx == 0) s.r[ty * RT + i] = rs;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s.cs[ty][tx * 4 + j] = cs[j];

    for (int n0 = 0; n0 < a.dk; n0 += 64) {
        clear(p);
        product(p, Op<T>{g, ldo, 1, len, a.dv, nullptr},
                Op<float>{S + (long long)n0 * a.dv, a.dv, 1, a.dk - n0, a.dv, nullptr}, a.dv, s.sA, s.sB);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = ty * RT + i;
            const float f = a.scale * s.d.row[r];
            const bool on = s.d.first[r] < 0;
            float u = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx * 4 + j;
                p[i][j] = on ? p[i][j] * f : 0.0f;
                if (r < len && n < a.dk) u = fmaf(to_f(q[r * a.ldq + n]), p[i][j], u);
            }
            u = sum16(u);
            if (tx == 0) s.u[r] += u;
        }
        product(p, Op<float>{&s.Pd[0][0], LC + 1, 1, LC, len, nullptr},
                Op<T>{k + n0, 1, a.ldk, a.dk - n0, len, nullptr}, len, s.sA, s.sB);
        clear(t);
        product(t, Op<T>{v, a.ldv, 1, len, a.dv, nullptr},
                Op<float>{dS + (long long)n0 * a.dv, a.dv, 1, a.dk - n0, a.dv, nullptr}, a.dv, s.sA, s.sB);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = ty * RT + i;
            const float f = s.d.col[r];
            const bool on = s.d.first[LC - 1] <= r;
            float w = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx * 4 + j;
                t[i][j] = on ? t[i][j] * f : 0.0f;
                if (r < len && n < a.dk) w = fmaf(to_f(k[r * a.ldk + n]), t[i][j], w);
            }
            w = sum16(w);
            if (tx == 0) s.w[r] += w;
        }
        product(t, Op<float>{&s.Pd[0][0], 1, LC + 1, LC, len, nullptr},
                Op<T>{q + n0, 1, a.ldq, a.dk - n0, len, nullptr}, len, s.sA, s.sB);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty * RT + i, n = n0 + tx * 4 + j;
                if (r >= len || n >= a.dk) continue;
                if (part_q) {
                    const long long at = ((ck.row + r) * a.H + h) * a.dk + n;
                    if (!SLSTM_IN(at, la_rows(a) * a.H * a.dk)) continue;
                    part_q[at] = p[i][j];
                    part_k[at] = t[i][j];
                } else {
                    const long long at = ((ck.row + r) * a.Hqk + hq) * a.dk + n;
                    if (!SLSTM_IN(at, la_rows(a) * a.Hqk * a.dk)) continue;
                    put(static_cast<T *>(a.dq) + at, p[i][j]);
                    put(static_cast<T *>(a.dk_) + at, t[i][j]);
                }
            }
    }
    for (int n0 = 0; n0 < a.dv; n0 += 64) {
        clear(t);
        product(t, Op<T>{k, a.ldk, 1, len, a.dk, nullptr}, Op<float>{dS + n0, 1, a.dv, a.dv - n0, a.dk, nullptr}, a.dk,
                s.sA, s.sB);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const float f = s.d.col[ty * RT + i];
            const bool on = s.d.first[LC - 1] <= ty * RT + i;
#pragma unroll
            for (int j = 0; j < 4; ++j) t[i][j] = on ? t[i][j] * f : 0.0f;
        }
        product(t, Op<float>{&s.P[0][0], 1, LC + 1, LC, len, nullptr},
                Op<T>{g + n0, 1, ldo, a.dv - n0, len, nullptr}, len, s.sA, s.sB);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty * RT + i, n = n0 + tx * 4 + j;
                if (r < len && n < a.dv &&
                    SLSTM_IN((ck.row + r) * ldo + (long long)h * a.dv + n, la_rows(a) * ldo))
                    put(static_cast<T *>(a.dv_) + (ck.row + r) * ldo + (long long)h * a.dv + n, t[i][j]);
            }
    }
    if (a.dg == nullptr) return;
    // <S_n, dS_{n+1}>, then dg by one warp
    float dot = 0.0f;
    for (int i = threadIdx.x; i < a.dk * a.dv; i += nt<RT>()) dot = fmaf(S[i], dS[i], dot);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    dot = 0.0f;
    for (int i = 0; i < nt<RT>() / 32; ++i) dot += s.red[i];
    dot = s.d.tot < 0.0f ? 0.0f : dot * s.d.tot;
    // two rows a lane; sums of up to 64 terms, in 64 bits: they cancel
    double x[2], w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = lane * 2 + i;
        double col = 0.0;
        for (int y = 0; y < 64 / RT; ++y) col += s.cs[y][r];
        x[i] = (double)s.r[r] + s.u[r] - col;
        w[i] = s.w[r];
    }
    double xs = x[0] + x[1], ws = w[0] + w[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double xu = __shfl_down_sync(0xffffffffu, xs, o), wu = __shfl_up_sync(0xffffffffu, ws, o);
        if (lane + o < 32) xs += xu;
        if (lane >= o) ws += wu;
    }
    // rows behind, rows before this lane's (no differences: a sum may be no number)
    double xa = __shfl_down_sync(0xffffffffu, xs, 1), wb = __shfl_up_sync(0xffffffffu, ws, 1);
    if (lane == 31) xa = 0.0;
    if (lane == 0) wb = 0.0;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = lane * 2 + i;
        float dgv = (float)(xa + (i == 0 ? x[0] + x[1] : x[1]) + wb + (i == 0 ? 0.0 : w[0]) + (double)dot);
        if (r >= len || s.d.first[r] == r) dgv = 0.0f;   // nothing passes a row that clears the state
        if (r < len && !a.per_head && SLSTM_IN((ck.row + r) * a.H + h, la_rows(a) * a.H))
            a.dg[(ck.row + r) * a.H + h] = dgv;
        sum += dgv;
    }
    if (a.per_head) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0 && SLSTM_IN((long long)c * a.H + h, (long long)ch.total * a.H))
            dgc[(long long)c * a.H + h] = sum;
    }
}

// V elements of dq (blockIdx.y = 0) or dk a thread.
template <typename T, int V>
__global__ void __launch_bounds__(256) la_share_kernel(const float *__restrict__ pq, const float *__restrict__ pk, T *dq,
                                                       T *dk_, LaChunks ch, long long rows, int Hqk, int rep, int dk)
{
    const float *part = blockIdx.y ? pk : pq;
    T *out = blockIdx.y ? dk_ : dq;
    // packed: the rows of the sequences only
    const int per = dk / V;   // pieces of a head
    const long long w = (long long)Hqk * per, i0 = ch.pos ? ch.pos[0] * w : 0;
    const long long n = ch.pos ? ch.pos[ch.n_seq] * w : rows * w;
    for (long long i = i0 + (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const long long rh = i / per;   // row * Hqk + hq
        const int d = (int)(i - rh * per) * V;
        const float *p = part + rh * rep * dk + d;
        float s[V];
#pragma unroll
        for (int k = 0; k < V; ++k) s[k] = 0.0f;
#pragma unroll 4
        for (int r = 0; r < rep; ++r, p += dk) {
            if (V == 4) {
                const float4 f = *reinterpret_cast<const float4 *>(p);
                s[0] += f.x;
                s[V > 1 ? 1 : 0] += f.y;
                s[V > 2 ? 2 : 0] += f.z;
                s[V > 3 ? 3 : 0] += f.w;
            } else {
                s[0] += *p;
            }
        }
        // (four elements of a type stand on their own width: out is aligned to them)
        struct alignas(V * sizeof(T)) Piece {
            T v[V];
        } piece;
#pragma unroll
        for (int k = 0; k < V; ++k) put(&piece.v[k], s[k]);
        if (SLSTM_IN(rh * dk + d + V - 1, rows * Hqk * dk)) *reinterpret_cast<Piece *>(out + rh * dk + d) = piece;
    }
}

__global__ void __launch_bounds__(256) la_head_sum_kernel(const float *__restrict__ part, float *dg, LaChunks ch,
                                                          int H)
{
    __shared__ double red[8];
    const int h = blockIdx.x;
    const int n = ch.pos ? ch.coff[ch.n_seq] : ch.total;
    double s = 0.0;
    for (int c = threadIdx.x; c < n; c += 256) s += part[(long long)c * H + h];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) s += red[w];
        if (SLSTM_IN(h, H)) dg[h] = (float)s;
    }
}

// The table of packed sequences: offsets clamped into [0, T] and raised to the
// largest before them, and the chunks before each sequence.  One block a table,
// 1024 offsets at a time.  The second table's chunks are also put in an order,
// long ones first (by 64 classes of length; within one, as it comes): blocks take
// them in that order, and what is left for the last SMs is short.
__global__ void __launch_bounds__(1024) la_table_kernel(const int *__restrict__ cu, int n_seq, int T, int C, int *pos,
                                                        int *coff, int C2, int *pos2, int *coff2, int *order)
{
    if (blockIdx.x == 1) {
        C = C2;
        pos = pos2;
        coff = coff2;
    }
    __shared__ int wm[32], ws[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int top = 0, sum = 0;   // the largest offset, and the chunks, of the tiles before
    for (int k0 = 0; k0 <= n_seq; k0 += 1024) {
        const int k = k0 + threadIdx.x;
        int m = k <= n_seq ? min(max(cu[k], 0), T) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, m, o);
            if (lane >= o) m = max(m, u);
        }
        if (lane == 31) wm[warp] = m;
        __syncthreads();
        int before = top;
        for (int w = 0; w < warp; ++w) before = max(before, wm[w]);
        m = max(m, before);
        int prev = __shfl_up_sync(0xffffffffu, m, 1);
        if (lane == 0) prev = before;
        for (int w = 0; w < 32; ++w) top = max(top, wm[w]);
        // chunks of sequence k - 1, which ends at offset k
        int n = k >= 1 && k <= n_seq && m > prev ? (m - prev - 1) / C + 1 : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += u;
        }
        if (lane == 31) ws[warp] = n;
        __syncthreads();
        int off = sum;
        for (int w = 0; w < warp; ++w) off += ws[w];
        if (k <= n_seq) {
            pos[k] = m;
            coff[k] = off + n;
        }
        for (int w = 0; w < 32; ++w) sum += ws[w];
        __syncthreads();
    }
    if (blockIdx.x == 0 || order == nullptr) return;
    __shared__ int at[64];
    const LaChunks t{n_seq, T, C, 0, 0, pos, coff, nullptr};
    auto kind = [&](int i) { return 63 - (int)((long long)(la_chunk(t, i).len - 1) * 64 / C); };
    if (threadIdx.x < 64) at[threadIdx.x] = 0;
    __syncthreads();   // the table is written, too
    for (int i = threadIdx.x; i < sum; i += 1024) atomicAdd(&at[kind(i)], 1);
    __syncthreads();
    if (threadIdx.x == 0)
        for (int k = 0, n = 0; k < 64; ++k) {
            const int m = at[k];
            at[k] = n;
            n += m;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < sum; i += 1024) order[atomicAdd(&at[kind(i)], 1)] = i;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t la_table_bytes(const LaArgs &a) { return a.cu ? 2 * up256(4 * ((size_t)a.B + 1)) : 0; }

int la_chunk_bound(const LaArgs &a, int C)
{
    return a.cu ? a.T / C + a.B : a.B * ((a.T - 1) / C + 1);
}

size_t la_order_bytes(const LaArgs &a, int C) { return a.cu ? up256(4 * (size_t)la_chunk_bound(a, C)) : 0; }

cudaError_t la_chunks(const LaArgs &a, int C, void *mem, LaChunks *out, cudaStream_t st, int C2, void *mem2,
                      LaChunks *out2, void *order)
{
    int *tab[2][2] = {};
    for (int i = 0; i < 2; ++i) {
        LaChunks *o = i ? out2 : out;
        if (o == nullptr) break;
        const int c = i ? C2 : C;
        *o = LaChunks{a.B, a.T, c, (a.T - 1) / c + 1, la_chunk_bound(a, c), nullptr, nullptr, nullptr};
        if (a.cu == nullptr) continue;
        char *p = static_cast<char *>(i ? mem2 : mem);
        o->pos = tab[i][0] = reinterpret_cast<int *>(p);
        o->coff = tab[i][1] = reinterpret_cast<int *>(p + up256(4 * ((size_t)a.B + 1)));
    }
    if (a.cu == nullptr) return cudaSuccess;
    if (out2) out2->order = static_cast<int *>(order);
    la_table_kernel<<<out2 ? 2 : 1, 1024, 0, st>>>(a.cu, a.B, a.T, C, tab[0][0], tab[0][1], C2, tab[1][0], tab[1][1],
                                                   static_cast<int *>(order));
    return cudaGetLastError();
}

cudaError_t la_scan(const LaChunks &ch, int H, int E, bool back, float *buf, const float *tot, const float *first,
                    float *last, cudaStream_t st, int skip)
{
    if (E % 4 == 0)
        la_scan_kernel<4><<<dim3((unsigned)ch.n_seq * H, (E + 511) / 512), 128, 0, st>>>(ch, H, E, back, buf, tot,
                                                                                       first, last, skip);
    else
        la_scan_kernel<1><<<dim3((unsigned)ch.n_seq * H, (E + 127) / 128), 128, 0, st>>>(ch, H, E, back, buf, tot,
                                                                                       first, last, skip);
    return cudaGetLastError();
}

namespace {

template <typename T>
cudaError_t share_sum(const float *pq, const float *pk, const LaChunks &ch, const LaArgs &a, cudaStream_t st)
{
    const long long rows = a.cu ? a.T : (long long)a.B * a.T;
    T *dq = static_cast<T *>(a.dq), *dk = static_cast<T *>(a.dk_);
    const uintptr_t at = reinterpret_cast<uintptr_t>(dq) | reinterpret_cast<uintptr_t>(dk);
    const bool four = a.dk % 4 == 0 && at % (4 * sizeof(T)) == 0;
    const long long n = rows * a.Hqk * (four ? a.dk / 4 : a.dk);
    const dim3 grid((unsigned)min((n + 255) / 256, (long long)148 * 16), 2);
    if (four) la_share_kernel<T, 4><<<grid, 256, 0, st>>>(pq, pk, dq, dk, ch, rows, a.Hqk, a.H / a.Hqk, a.dk);
    else la_share_kernel<T, 1><<<grid, 256, 0, st>>>(pq, pk, dq, dk, ch, rows, a.Hqk, a.H / a.Hqk, a.dk);
    return cudaGetLastError();
}

}  // namespace

cudaError_t la_share_sum(const float *pq, const float *pk, const LaChunks &ch, const LaArgs &a, cudaStream_t st)
{
    return a.dtype == SLSTM_F32 ? share_sum<float>(pq, pk, ch, a, st) : share_sum<__nv_bfloat16>(pq, pk, ch, a, st);
}

cudaError_t la_head_sum(const float *part, float *dg, const LaChunks &ch, int H, cudaStream_t st)
{
    la_head_sum_kernel<<<H, 256, 0, st>>>(part, dg, ch, H);
    return cudaGetLastError();
}

namespace {

struct SimtWs {
    char *table;
    float *S, *totS, *dS, *totD, *pq, *pk, *dgc;
    size_t bytes;
};

SimtWs simt_layout(const LaArgs &a, bool backward, void *ws)
{
    SimtWs w{};
    char *p = static_cast<char *>(ws);
    const size_t nc = (size_t)la_chunk_bound(a, LC), E = (size_t)a.dk * a.dv;
    const size_t rows = a.cu ? (size_t)a.T : (size_t)a.B * a.T;
    auto take = [&](size_t bytes) {
        char *r = p;
        p += up256(bytes);
        return r;
    };
    w.table = take(la_table_bytes(a));
    w.S = reinterpret_cast<float *>(take(4 * nc * a.H * E));
    w.totS = reinterpret_cast<float *>(take(4 * nc * a.H));
    if (backward) {
        w.dS = reinterpret_cast<float *>(take(4 * nc * a.H * E));
        w.totD = reinterpret_cast<float *>(take(4 * nc * a.H));
        w.dgc = reinterpret_cast<float *>(take(4 * nc * a.H));
        if (a.H != a.Hqk) {
            w.pq = reinterpret_cast<float *>(take(4 * rows * a.H * a.dk));
            w.pk = reinterpret_cast<float *>(take(4 * rows * a.H * a.dk));
        }
    }
    w.bytes = (size_t)(p - static_cast<char *>(ws));
    return w;
}

template <typename T, int RT>
cudaError_t states(const LaArgs &a, const LaChunks &ch, bool back, float *buf, float *tot, cudaStream_t st)
{
    const int E = a.dk * a.dv;
    const dim3 grid((unsigned)ch.total * a.H, (a.dk + 63) / 64, (a.dv + 63) / 64);
    la_delta_kernel<T, RT><<<grid, nt<RT>(), 0, st>>>(a, ch, back, buf, tot);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return la_scan(ch, a.H, E, back, buf, tot, back ? a.dsT : a.s0, back ? a.ds0 : a.sT, st);
}

template <typename T, int RT>
cudaError_t forward(const LaArgs &a, const LaChunks &ch, const SimtWs &w, cudaStream_t st)
{
    cudaError_t e = states<T, RT>(a, ch, false, w.S, w.totS, st);
    if (e != cudaSuccess) return e;
    la_out_kernel<T, RT><<<(unsigned)ch.total * a.H, nt<RT>(), 0, st>>>(a, ch, w.S);
    return cudaGetLastError();
}

template <typename T, int RT>
cudaError_t backward(const LaArgs &a, const LaChunks &ch, const SimtWs &w, cudaStream_t st)
{
    cudaError_t e = states<T, RT>(a, ch, false, w.S, w.totS, st);
    if (e == cudaSuccess) e = states<T, RT>(a, ch, true, w.dS, w.totD, st);
    if (e == cudaSuccess)
        e = la_allow_shared<la_back_kernel<T, RT>>((int)sizeof(BackShared));
    if (e != cudaSuccess) return e;
    la_back_kernel<T, RT><<<(unsigned)ch.total * a.H, nt<RT>(), sizeof(BackShared), st>>>(a, ch, w.S, w.dS, w.pq, w.pk,
                                                                                       w.dgc);
    e = cudaGetLastError();
    if (e == cudaSuccess && w.pq) e = la_share_sum(w.pq, w.pk, ch, a, st);
    if (e == cudaSuccess && a.dg && a.per_head) e = la_head_sum(w.dgc, a.dg, ch, a.H, st);
    return e;
}

// Whether the blocks of a pass leave the SMs fewer than two each.
bool few(const LaArgs &a, const LaChunks &ch) { return (long long)ch.total * a.H < 2 * 148; }

}  // namespace

size_t la_simt_workspace(const LaArgs &a, bool backward)
{
    return simt_layout(a, backward, reinterpret_cast<void *>((uintptr_t)256)).bytes;
}

cudaError_t la_simt_forward(const LaArgs &a, void *ws, cudaStream_t st)
{
    const SimtWs w = simt_layout(a, false, ws);
    LaChunks ch;
    const cudaError_t e = la_chunks(a, LC, w.table, &ch, st);
    if (e != cudaSuccess) return e;
    typedef __nv_bfloat16 bf16;
    if (a.dtype == SLSTM_F32) return few(a, ch) ? forward<float, 4>(a, ch, w, st) : forward<float, 8>(a, ch, w, st);
    return few(a, ch) ? forward<bf16, 4>(a, ch, w, st) : forward<bf16, 8>(a, ch, w, st);
}

cudaError_t la_simt_backward(const LaArgs &a, void *ws, cudaStream_t st)
{
    const SimtWs w = simt_layout(a, true, ws);
    LaChunks ch;
    const cudaError_t e = la_chunks(a, LC, w.table, &ch, st);
    if (e != cudaSuccess) return e;
    typedef __nv_bfloat16 bf16;
    if (a.dtype == SLSTM_F32) return few(a, ch) ? backward<float, 4>(a, ch, w, st) : backward<float, 8>(a, ch, w, st);
    return few(a, ch) ? backward<bf16, 4>(a, ch, w, st) : backward<bf16, 8>(a, ch, w, st);
}

// ---------------------------------------------------------------------------
// the step of single tokens
// ---------------------------------------------------------------------------
namespace {

constexpr int STEP_WARPS = 4;
constexpr int STEP_COLS = 32;

// A block takes 32 columns of one state: LPR lanes hold a row of them (VEC
// columns each), the warps walk the rows, and the partial products with q meet
// in shared memory.  The state is read once and written once, in 16-byte pieces
// that are not to stay in the caches (the next token comes after everything
// else); s_next may be s_prev, as each element is read and written by one
// thread.  Bound by those bytes: 128 sequences of 8 heads of 128 x 128 in 25.7 us,
// 5.2 TB/s (blocks of 128 columns and 8 warps: 33 us).
template <typename T, int VEC>
__global__ void __launch_bounds__(STEP_WARPS * 32) la_step_kernel(LaArgs a, const float *s_prev, float *s_next)
{
    constexpr int COLS = STEP_COLS;
    constexpr int LPR = COLS / VEC;                     // lanes of a row
    constexpr int RPW = 32 / LPR;                       // rows a warp takes at once
    constexpr int ROWS = STEP_WARPS * RPW;
    __shared__ float red[ROWS][COLS];
    const int b = blockIdx.x / a.H, h = blockIdx.x % a.H, hq = h / (a.H / a.Hqk);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.y * COLS + (lane % LPR) * VEC;
    const int slot = warp * RPW + lane / LPR;
    const T *q = static_cast<const T *>(a.q) + b * a.ldq + (long long)hq * a.dk;
    const T *k = static_cast<const T *>(a.k) + b * a.ldk + (long long)hq * a.dk;
    const T *v = static_cast<const T *>(a.v) + b * a.ldv + (long long)h * a.dv;
    const float g = a.g[a.per_head ? h : (long long)b * a.H + h], decay = expf(g);
    if (la_clears(g)) s_prev = nullptr;   // not times zero: what is cleared may be infinite or no number
    const long long base = ((long long)b * a.H + h) * a.dk * a.dv;
    float o[VEC], vv[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        o[i] = 0.0f;
        vv[i] = col + i < a.dv ? to_f(v[col + i]) : 0.0f;
    }
    if (col < a.dv) {
#pragma unroll 8
        for (int r = slot; r < a.dk; r += ROWS) {
            const float kr = to_f(k[r]), qr = to_f(q[r]);
            const long long at = base + (long long)r * a.dv + col;
            float s[VEC];
            if (VEC == 4) {
                const float4 f =
                    s_prev ? __ldcs(reinterpret_cast<const float4 *>(s_prev + at)) : make_float4(0, 0, 0, 0);
                s[0] = f.x;
                s[VEC > 1 ? 1 : 0] = f.y;
                s[VEC > 2 ? 2 : 0] = f.z;
                s[VEC > 3 ? 3 : 0] = f.w;
            } else {
                s[0] = s_prev ? s_prev[at] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s[i] = fmaf(decay, s[i], kr * vv[i]);
                o[i] = fmaf(qr, s[i], o[i]);
            }
            if (!SLSTM_IN(at + VEC - 1, (long long)a.B * a.H * a.dk * a.dv)) continue;
            if (VEC == 4)
                __stcs(reinterpret_cast<float4 *>(s_next + at),
                       make_float4(s[0], s[VEC > 1 ? 1 : 0], s[VEC > 2 ? 2 : 0], s[VEC > 3 ? 3 : 0]));
            else
                s_next[at] = s[0];
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) red[slot][(lane % LPR) * VEC + i] = o[i];
    __syncthreads();
    const int n = blockIdx.y * COLS + threadIdx.x;
    if (threadIdx.x < COLS && n < a.dv) {
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) sum += red[r][threadIdx.x];
        if (SLSTM_IN(((long long)b * a.H + h) * a.dv + n, (long long)a.B * a.H * a.dv))
            put(static_cast<T *>(a.o) + ((long long)b * a.H + h) * a.dv + n, sum * a.scale);
    }
}

template <typename T>
cudaError_t step(const LaArgs &a, float *s_next, cudaStream_t st)
{
    const dim3 grid((unsigned)a.B * a.H, (a.dv + STEP_COLS - 1) / STEP_COLS);
    if (a.dv % 4 == 0) la_step_kernel<T, 4><<<grid, STEP_WARPS * 32, 0, st>>>(a, a.s0, s_next);
    else la_step_kernel<T, 1><<<grid, STEP_WARPS * 32, 0, st>>>(a, a.s0, s_next);
    return cudaGetLastError();
}

}  // namespace

cudaError_t la_step_launch(const LaArgs &a, float *s_next, cudaStream_t st)
{
    return a.dtype == SLSTM_F32 ? step<float>(a, s_next, st) : step<__nv_bfloat16>(a, s_next, st);
}

}  // namespace slstm

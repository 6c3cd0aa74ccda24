// Linear attention with a decay for each head, bf16 on the sm_100a tensor
// cores (tcgen05 + TMEM, fed by TMA); the formulas are at linear_attention.cu.
// d_k and d_v up to 128, multiples of 8; chunks of 128 rows, so that a chunk's
// products are 128 x 128 x d tiles.
//
// What needs how many bits: products of q, k, v and dO with one another are
// exact in the fp32 accumulators, and the state is held in fp32 registers.  What
// it sums, rows of v or dO times their decays, are split into three bf16 terms,
// all of an fp32 number, so that states and their gradients are those of fp32
// arithmetic.  So are the states that the gradients start from in each chunk,
// as that of the decay, an fp32 output, needs them.  What a bf16 output alone
// depends on, the weights D (q k) and D (dO v), the state in q S and its gradient
// in k dS, has two terms, which leave 2^-17 of it at most: the output is rounded
// once.  (With one term there and two for the rest, 8 rows of 8192 steps: o 2.35e-3
// off in the 2-norm, 1.66e-3 of it its own rounding, final states and the decays'
// gradients 2.4e-6 and 3.5e-6, now 2e-7 and 6.3e-7; 169 us forward and 542 for the
// gradients, now 213 and 712.)
//
// Every mbarrier wait is bounded in its tries (of about 4 us each when they
// fail); on expiry the block marks itself, waits (bounded) for its own loads and
// MMAs, writes NaN over the outputs that it has not made, frees its tensor memory
// and returns.
#include <cuda_bf16.h>

#define SLSTM_FILE_ID 13
#include "checked.cuh"
#include "la.cuh"
#include "launchers.h"
#include "tc.cuh"

namespace slstm {
namespace {

constexpr int TCC = 128;                     // rows of a chunk
constexpr uint32_t BOX = TCC * 128;          // bytes of 128 rows of 64 bf16
constexpr uint64_t TC_WAIT_NS = 1000000000ull;
constexpr int TRY_US = 4;                    // a try of a wait that fails: 3.96 us, measured

// A block's waits, in shared memory.
struct Waits {
    int gave_up, tries;
};
constexpr int ND = 4;                        // chunks whose decays are held

// The decays of a chunk.  D_ij = e^{c_i - c_j} of rows i in 32-row block q and
// j in an earlier one is rq[i] cq[q][j], by way of the block's first row (both
// factors are at most 1 where nothing grows): one exponential a row and three a
// column in place of one an element.  Inside a block it is the exponential of
// c_i - c_j: c_i less that of the block's first row as a multiple of 1/16 (16 bits,
// so that differences are exact) and a rest, as behind strong decays both numbers
// are large and their difference is not.
struct alignas(16) TcDecays {
    float loc[TCC], rest[TCC];
    float row[TCC], col[TCC];
    float rq[TCC];             // e^{loc}, 0 behind a row of the block that clears
    uint32_t mask[TCC];        // rows of the row's 32 that it reaches: itself and those behind it, up to a clear
    float cq_[192];            // cq(q)[j], j < 32 q; 0 where the state is cleared after j, up to row 32 q
    signed char first[TCC];    // the last row up to this one that clears the state, or -1
    float tot;                 // e^{c_C}, or -1 where a row clears
    SLSTM_DEVINL float *cq(int q) { return cq_ + 16 * q * (q - 1); }
    SLSTM_DEVINL const float *cq(int q) const { return cq_ + 16 * q * (q - 1); }
};
static_assert(sizeof(TcDecays) % 16 == 0, "an array of them in shared memory, read 16 bytes at a time");

// Blocks of one pass: a segment (a run of chunks of one sequence) of one head
// and 64 columns of the state.
struct TcArgs {
    LaArgs a;
    const TcDecays *dec;      // [chunk][h]
    LaChunks seg;             // the segments
    LaChunks ch;              // the chunks (packed: the table's second view)
    int tiles;                // 64-column tiles of d_v
    // states: where a segment starts and what it leaves
    const float *init;        // entry states [segment][h] of sequences of several segments
    const float *first;       // entry states [sequence][h] (null: zero) of the others
    float *fin;               // the pass for `init`: final states [segment][h], of several segments
    float *fin_tot;           // [segment][h] decay of a segment (-1: it clears)
    float *last;              // final states [sequence][h] of one segment, or null
    __nv_bfloat16 *st;        // states that each chunk starts from, [term][chunk][h] (dk x dv), or null
    const __nv_bfloat16 *pst; // from the end: the forward states, for `dot`
    float *dot;               // [chunk][h][2][8]: a warp's share of <S_n, dS_{n+1}>, or null
    bool back;                // from the end: (q, dO) in place of (k, v)
};

SLSTM_DEVINL float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One lane of the warp.  Chosen so, and not by its number, the compiler knows that
// one thread runs what follows, and keeps the operands of MMAs and copies in
// uniform registers without finding out lane by lane (186 -> 174 us a forward pass).
SLSTM_DEVINL bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0u;
}

SLSTM_DEVINL uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

SLSTM_DEVINL __nv_bfloat16 bf16_nan() { return __float2bfloat16(__int_as_float(0x7fc00000)); }

SLSTM_DEVINL float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
SLSTM_DEVINL float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 products, or differences, in one instruction.
SLSTM_DEVINL void mul2(float &d0, float &d1, float a0, float a1, float b0, float b1)
{
    asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 a, a, b;\n"
        " mov.b64 {%0, %1}, a;\n}\n"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
SLSTM_DEVINL void sub2(float &d0, float &d1, float a0, float a1, float b0, float b1)
{
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %6};\n"
        " fma.rn.f32x2 a, b, c, a;\n mov.b64 {%0, %1}, a;\n}\n"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(-1.0f));
}

// Byte offset of 16-byte piece p of a row in a 128-byte-swizzled box.
SLSTM_DEVINL uint32_t swz(int row, int p) { return (uint32_t)row * 128u + (uint32_t)((p ^ (row & 7)) << 4); }

// A box of a tensor on its way into the L2 cache.
SLSTM_DEVINL void tma_prefetch_4d(const CUtensorMap *map, int c0, int c1, int c2, int c3)
{
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}

// The first 1024-byte boundary in dynamic shared memory, by an offset: a pointer
// that goes through an integer is no longer known to be shared memory, and every
// access through it becomes a generic one (563 against 503 us, when this was found).
SLSTM_DEVINL uint8_t *aligned_smem(uint8_t *raw) { return raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u); }

// Wait for a phase of an mbarrier: the hardware suspends the thread in each try
// (for a time of its own), and the tries are counted, which costs the
// waiting warps' neighbours less than reading a clock.  False after the last, or
// once this block has given up.
SLSTM_DEVINL bool lane_wait(uint64_t *bar, uint32_t parity, Waits *w)
{
    const uint32_t addr = smem_u32(bar);
#pragma unroll 1
    for (int i = 1;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n"
            " .reg .pred p;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n"
            "}\n"
            : "=r"(ok)
            : "r"(addr), "r"(parity)
            : "memory");
        if (ok) return true;
        if (*(volatile int *)&w->gave_up) return false;
        if (i >= w->tries) break;
    }
    *(volatile int *)&w->gave_up = 1;
    return false;
}
// Whether a phase has completed, without being suspended.
SLSTM_DEVINL bool done(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0u;
}
// One wait of a whole warp: every lane the same answer.
SLSTM_DEVINL bool warp_wait(uint64_t *bar, uint32_t parity, Waits *w)
{
    return __all_sync(0xffffffffu, lane_wait(bar, parity, w));
}

// The warp's shared-memory writes (and its reads of tensor memory) before the
// arrival on `bar`.
SLSTM_DEVINL void warp_arrive(uint64_t *bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The log decays of a lane's four rows 4 l .. of a chunk; 0 behind `len`.
SLSTM_DEVINL void load_decays(float (&gv)[4], const LaArgs &a, long long row, int len, int h, int lane)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = lane * 4 + i;
        gv[i] = t < len ? __ldg(a.g + (a.per_head ? h : (row + t) * a.H + h)) : 0.0f;
    }
}

// The decays of a chunk by one warp into `d` (la_decays for the fields there).
// The sums and their differences run in 64 bits.
SLSTM_DEVINL void tc_decays(TcDecays &d, const float (&gv)[4], int lane)
{
    constexpr uint32_t ALL = 0xffffffffu;
    double c[4], run = 0.0;
    int f[4], last = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (la_clears(gv[i])) last = lane * 4 + i;
        else run += (double)gv[i] * 1.4426950408889634074;
        c[i] = run;
        f[i] = last;
    }
    double pre = run;
    int pf = last;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double u = __shfl_up_sync(ALL, pre, o);
        const int w = __shfl_up_sync(ALL, pf, o);
        if (lane >= o) {
            pre += u;
            pf = max(pf, w);
        }
    }
    const double all = __shfl_sync(ALL, pre, 31);
    const int allf = __shfl_sync(ALL, pf, 31);
    double before = __shfl_up_sync(ALL, pre, 1);
    int bf = __shfl_up_sync(ALL, pf, 1);
    if (lane == 0) {
        before = 0.0;
        bf = -1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[i] += before;
        f[i] = max(bf, f[i]);
    }
    const double base = __shfl_sync(ALL, c[0], lane & 24);   // of the block's first row
    const int b = 32 * (lane >> 3);
    double to_q[3];
    int fq[3];
#pragma unroll
    for (int q = 1; q < 4; ++q) {
        to_q[q - 1] = __shfl_sync(ALL, c[0], 8 * q);
        fq[q - 1] = __shfl_sync(ALL, f[0], 8 * q);
    }
    float loc[4], rest[4], row[4], col[4], rq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = lane * 4 + i;
        const double x = c[i] - base;
        loc[i] = rintf((float)x * 16.0f) * 0.0625f;
        rest[i] = (float)(x - (double)loc[i]);
        row[i] = f[i] >= 0 ? 0.0f : ex2((float)c[i]);
        col[i] = allf > t ? 0.0f : ex2((float)(all - c[i]));
        rq[i] = f[i] > b ? 0.0f : ex2((float)x);
    }
    // the block's rows that clear, then for each row the run up to the next of them
    uint32_t clears = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) clears |= (f[i] == lane * 4 + i ? 1u : 0u) << ((lane * 4 + i) & 31);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) clears |= __shfl_xor_sync(ALL, clears, o);
    uint32_t mk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t from = ~0u << ((lane * 4 + i) & 31);
        const uint32_t next = clears & (from << 1);
        mk[i] = from & (next ? (next & (0u - next)) - 1u : ~0u);
    }
    *reinterpret_cast<uint4 *>(d.mask + lane * 4) = make_uint4(mk[0], mk[1], mk[2], mk[3]);
    *reinterpret_cast<float4 *>(d.loc + lane * 4) = make_float4(loc[0], loc[1], loc[2], loc[3]);
    *reinterpret_cast<float4 *>(d.row + lane * 4) = make_float4(row[0], row[1], row[2], row[3]);
    *reinterpret_cast<float4 *>(d.col + lane * 4) = make_float4(col[0], col[1], col[2], col[3]);
    *reinterpret_cast<float4 *>(d.rq + lane * 4) = make_float4(rq[0], rq[1], rq[2], rq[3]);
    *reinterpret_cast<float4 *>(d.rest + lane * 4) = make_float4(rest[0], rest[1], rest[2], rest[3]);
    *reinterpret_cast<char4 *>(d.first + lane * 4) =
        make_char4((signed char)f[0], (signed char)f[1], (signed char)f[2], (signed char)f[3]);
#pragma unroll
    for (int q = 1; q < 4; ++q)
        if (b < 32 * q) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = fq[q - 1] > lane * 4 + i ? 0.0f : ex2((float)(to_q[q - 1] - c[i]));
            *reinterpret_cast<float4 *>(d.cq(q) + lane * 4) = make_float4(e[0], e[1], e[2], e[3]);
        }
    if (lane == 0) d.tot = allf >= 0 ? -1.0f : ex2((float)all);
}

// The decays of every chunk and head, [chunk][h], a warp each: about 250
// instructions one after another, which inside the kernels below took two warps
// 2500 cycles a chunk, longer than anything else there.
__global__ void __launch_bounds__(256) la_decay_kernel(LaArgs a, LaChunks ch, TcDecays *out)
{
    const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int h = (int)(i % a.H);
    if (i / a.H >= ch.total) return;
    const LaChunk c = la_chunk(ch, (int)(i / a.H));
    if (c.len <= 0) return;
    float gv[4];
    load_decays(gv, a, c.row, c.len, h, threadIdx.x & 31);
    tc_decays(out[i], gv, threadIdx.x & 31);
}

// Two numbers as two bf16 terms each: the number rounded, and what that leaves,
// rounded (2^-17 of the number is lost at most).
SLSTM_DEVINL void two_terms(float a, float b, uint32_t &hi, uint32_t &lo)
{
    float c, d;
    hi = pack2(a, b);
    sub2(c, d, a, b, lo_of(hi), hi_of(hi));
    lo = pack2(c, d);
}

// Two numbers as three bf16 terms each: all that fp32 holds of them, but for an
// eighth of its last bit.
SLSTM_DEVINL void three_terms(float a, float b, uint32_t (&t)[3])
{
    float c, d;
    t[0] = pack2(a, b);
    sub2(c, d, a, b, lo_of(t[0]), hi_of(t[0]));
    t[1] = pack2(c, d);
    sub2(a, b, c, d, lo_of(t[1]), hi_of(t[1]));
    t[2] = pack2(a, b);
}

// Pieces p0 .. p1 - 1 (8 columns each) of row t of a 64-column box of v (or dO)
// times w as three bf16 terms, the first into the box at hi (which may be the row's
// own), the others into the two at lo; zero where !on.  The loops over columns in
// these kernels are rolled up on purpose: the warps of a block run six different
// codes at once, and unrolled they do not fit the instruction cache.
SLSTM_DEVINL void scale_row(const uint8_t *src, uint8_t *hi, uint8_t *lo, int t, int p0, int p1, float w, bool on)
{
#pragma unroll 1
    for (int p = p0; p < p1; ++p) {
        const uint32_t o = swz(t, p);
        uint4 v = *reinterpret_cast<const uint4 *>(src + o);
        if (!on) v = make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
        uint32_t z[4][3];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float a, b;
            mul2(a, b, lo_of(x[k]), hi_of(x[k]), w, w);
            three_terms(a, b, z[k]);
        }
        *reinterpret_cast<uint4 *>(hi + o) = make_uint4(z[0][0], z[1][0], z[2][0], z[3][0]);
        *reinterpret_cast<uint4 *>(lo + o) = make_uint4(z[0][1], z[1][1], z[2][1], z[3][1]);
        *reinterpret_cast<uint4 *>(lo + BOX + o) = make_uint4(z[0][2], z[1][2], z[2][2], z[3][2]);
    }
}

// One term of eight numbers, added to what there is of them.
SLSTM_DEVINL void add_terms(float (&f)[8], uint4 v)
{
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] += lo_of(x[j]);
        f[2 * j + 1] += hi_of(x[j]);
    }
}

SLSTM_DEVINL void zero_row(uint8_t *box, int t)
{
#pragma unroll
    for (int p = 0; p < 8; ++p) *reinterpret_cast<uint4 *>(box + t * 128 + p * 16) = make_uint4(0, 0, 0, 0);
}

// Where a segment lies.
struct Seg {
    int seq, nch, len;        // sequence, chunks, rows
    int item;                 // its index
    long long row;            // first row
    int t, b;                 // TMA coordinates of the first row
    long long c0;             // index of its first chunk
    bool only;                // the sequence is one segment
};

// The i-th segment in the order in which the blocks take them.
SLSTM_DEVINL bool seg_of(const TcArgs &g, int i, Seg *s)
{
    if (g.seg.pos && i >= g.seg.coff[g.seg.n_seq]) return false;
    i = g.seg.order ? g.seg.order[i] : i;
    const LaChunk c = la_chunk(g.seg, i);
    s->item = i;
    s->seq = c.seq;
    s->len = c.len;
    s->nch = (c.len + TCC - 1) / TCC;
    s->row = c.row;
    const bool packed = g.seg.pos != nullptr;
    s->t = packed ? (int)c.row : c.n * g.seg.C;
    s->b = packed ? 0 : c.seq;
    s->c0 = (packed ? (long long)g.ch.coff[c.seq] : (long long)c.seq * g.ch.nc) + (long long)c.n * (g.seg.C / TCC);
    s->only = c.count == 1;
    return true;
}

// The share of a thread of eight warps (two on each quarter of the
// accumulator's lanes) in a state tile of DK rows and 64 columns: with DK = 128
// half a row; with DK = 64 lanes 64..127 repeat lanes 0..63 (the MMA is given
// its 64 rows twice), and a thread holds a quarter.
template <int DK>
struct Share {
    static constexpr int N = DK == 128 ? 32 : 16;
    SLSTM_DEVINL static int row(int warp, int lane) { return (DK == 128 ? warp & 3 : warp & 1) * 32 + lane; }
    SLSTM_DEVINL static int col(int warp) { return 32 * (warp >> 2) + (DK == 128 ? 0 : 16 * ((warp >> 1) & 1)); }
};

// S <- tot S (nothing where it is cleared) + the sum of the two accumulators at
// `at` and 64 columns on.
template <int N>
SLSTM_DEVINL void state_add(float (&S)[N], float tot, uint32_t at)
{
#pragma unroll
    for (int z = 0; z < N; z += 16) {
        float v[16], w[16];
        tmem_ld16x2(at + z, at + 64 + z, v, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) S[z + i] = la_carry(tot, S[z + i], v[i] + w[i]);
    }
}

template <int N>
SLSTM_DEVINL void state_load(float (&S)[N], const float *src, int dk, int dv, int r, int col)
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        float4 f = make_float4(0, 0, 0, 0);
        if (src && r < dk && col + i < dv) f = *reinterpret_cast<const float4 *>(src + (long long)r * dv + col + i);
        S[i] = f.x;
        S[i + 1] = f.y;
        S[i + 2] = f.z;
        S[i + 3] = f.w;
    }
}

template <int N>
SLSTM_DEVINL void state_store(const float (&S)[N], float *dst, int dk, int dv, int r, int col,
                              [[maybe_unused]] const float *base, [[maybe_unused]] long long n)
{
    if (r >= dk) return;
#pragma unroll
    for (int i = 0; i < N; i += 4)
        if (col + i < dv && SLSTM_PIN(dst + (long long)r * dv + col + i + 3, base, n))
            *reinterpret_cast<float4 *>(dst + (long long)r * dv + col + i) =
                make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
}

// ---------------------------------------------------------------------------
// The states of a segment: one block walks its chunks and keeps the state of
// its 64 columns in registers,
//   S <- e^{c_C} S + X^T (w Y):  X = k, Y = v, w = e^{c_C - c_j} (forward)
//                                X = q, Y = dO, w = scale e^{c_i} (from the end)
// and writes the state that each chunk starts from (three bf16 terms, for the
// backward kernel) and / or the final one.  The work of a chunk is split over
// warps that run a chunk apart, since each part of it is a chain of latencies:
// warps 0-7 hold the state (lane = row of d_k), warps 8-15 scale Y, warp 16
// loads (a ring of NST chunks), warp 17 issues the MMAs.  Bound: the bytes of X
// and Y and of the states written.  Those go out through shared memory by TMA (warps
// 18-25): a lane holds a row of them, and stores from the registers, a line for
// each lane, took 5500 cycles a chunk where the rest takes 2000.
// ---------------------------------------------------------------------------
template <int DK>
struct StateShared {
    static constexpr int NST = DK == 128 ? 2 : 3;
    static constexpr int NB = DK / 64;
    static constexpr uint32_t STAGE = (NB + 1) * BOX;
    static constexpr uint32_t Y = NST * STAGE;          // two buffers of the lower two terms; the first: in Y's place
    static constexpr uint32_t OUT = Y + 4 * BOX;        // DK rows of each term
    static constexpr uint32_t DEC = OUT + 3 * DK * 128;
    static constexpr uint32_t BYTES = DEC + ND * sizeof(TcDecays) + 1024;
};
static_assert(StateShared<128>::BYTES + 512 <= 227 * 1024, "state shared memory");

constexpr int STATE_THREADS = 832;

template <int DK>
__global__ void __launch_bounds__(STATE_THREADS, 1)
    la_state_kernel(const __grid_constant__ CUtensorMap mx0, const __grid_constant__ CUtensorMap my0,
                    const __grid_constant__ CUtensorMap mx1, const __grid_constant__ CUtensorMap my1,
                    const __grid_constant__ CUtensorMap ms,
                    const __grid_constant__ TcArgs g0, const __grid_constant__ TcArgs g1)
{
    typedef StateShared<DK> SM;
    constexpr int NST = SM::NST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = aligned_smem(smem_raw);
    TcDecays *dec = reinterpret_cast<TcDecays *>(smem + SM::DEC);
    __shared__ uint64_t full[NST], empty[NST], dfull[ND], dempty[ND], yready[2], delta[2], drained[2];
    __shared__ uint64_t staged, unstaged, fin;
    __shared__ uint32_t s_tmem;
    __shared__ Waits s_wait;
    __shared__ int s_loaded;
    // the passes of both directions for the segments' first states run in one launch
    const TcArgs &g = blockIdx.y == 0 ? g0 : g1;
    const CUtensorMap *mx = blockIdx.y == 0 ? &mx0 : &mx1, *my = blockIdx.y == 0 ? &my0 : &my1;
    const LaArgs &a = g.a;
    const int tile = blockIdx.x % g.tiles, h = (blockIdx.x / g.tiles) % a.H, item = blockIdx.x / (g.tiles * a.H);
    Seg sg;
    if (!seg_of(g, item, &sg) || (g.fin && sg.only)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool back = g.back, packed = g.seg.pos != nullptr;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < ND; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], 16);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&yready[i], 8);
            mbar_init(&delta[i], 1);
            mbar_init(&drained[i], 8);
        }
        mbar_init(&staged, 8);
        mbar_init(&unstaged, 8);
        mbar_init(&fin, 1);
        mbar_init_fence();
        s_wait.gave_up = 0;
        s_wait.tries = a.tries;
        s_loaded = 0;
    }
    if (warp == 0) tmem_alloc<256>(&s_tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int nch = sg.nch;
    // the n-th chunk walked, and its rows
    auto chunk = [&](int n) { return back ? nch - 1 - n : n; };
    auto rows = [&](int n) { return min(TCC, sg.len - chunk(n) * TCC); };

    if (warp == 16) {
        if (elect_one()) {
            const int hq = h / (a.H / a.Hqk);
            int n = 0;
            for (; n < nch && n + 1 != a.debug_fault; ++n) {
                const int s = n % NST;
                if (!lane_wait(&empty[s], ((uint32_t)(n / NST) & 1u) ^ 1u, &s_wait)) break;
                if (!lane_wait(&dempty[n % ND], ((uint32_t)(n / ND) & 1u) ^ 1u, &s_wait)) break;
                uint8_t *st = smem + s * SM::STAGE;
                mbar_expect_tx(&dfull[n % ND], sizeof(TcDecays));
                bulk_load(&dec[n % ND], g.dec + (sg.c0 + chunk(n)) * a.H + h, sizeof(TcDecays), &dfull[n % ND]);
                mbar_expect_tx(&full[s], SM::STAGE);
                const int t = sg.t + chunk(n) * TCC;
#pragma unroll
                for (int i = 0; i < SM::NB; ++i) tma_load_4d(st + i * BOX, mx, &full[s], 64 * i, hq, t, sg.b);
                tma_load_4d(st + SM::NB * BOX, my, &full[s], 64 * tile, h, t, sg.b);
                if (n + NST < nch) {   // the chunk that takes this one's place, as far as the L2 cache
                    const int u = sg.t + chunk(n + NST) * TCC;
#pragma unroll
                    for (int i = 0; i < SM::NB; ++i) tma_prefetch_4d(mx, 64 * i, hq, u, sg.b);
                    tma_prefetch_4d(my, 64 * tile, h, u, sg.b);
                }
            }
            s_loaded = n;
        }
    } else if (warp == 17) {
        if (elect_one()) {
            constexpr uint32_t id_kv = idesc_bf16(128, 128, true, true), id_k3 = idesc_bf16(128, 64, true, true);
            for (int n = 0; n < nch; ++n) {
                const int s = n % NST;
                if (!lane_wait(&full[s], (uint32_t)(n / NST) & 1u, &s_wait)) break;
                if (!lane_wait(&yready[n & 1], (uint32_t)(n >> 1) & 1u, &s_wait)) break;
                if (!lane_wait(&drained[n & 1], ((uint32_t)(n >> 1) & 1u) ^ 1u, &s_wait)) break;
                tc_fence_after();
                // the 64 rows of a narrow d_k twice: no step from one 64 to the next
                const uint64_t ad = smem_desc_mn_sw128(smem_u32(smem + s * SM::STAGE), DK == 128 ? BOX : 0u);
                // two terms of w Y side by side, X being read once for them, and the third
                // into the sum of the second
                const uint32_t y = smem_u32(smem + s * SM::STAGE + SM::NB * BOX);
                const uint32_t z = smem_u32(smem + SM::Y + (n & 1) * 2 * BOX);
                const uint64_t bd = smem_desc_mn_sw128(y, z - y), cd = smem_desc_mn_sw128(z + BOX, BOX);
                const uint32_t d = tmem + (n & 1) * 128;
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                    umma_bf16(d, ad + (2048u >> 4) * k, bd + (2048u >> 4) * k, id_kv, k > 0 ? 1u : 0u);
                    umma_bf16(d + 64, ad + (2048u >> 4) * k, cd + (2048u >> 4) * k, id_k3, 1u);
                }
                umma_commit(&delta[n & 1]);
                umma_commit(&empty[s]);
            }
            umma_commit(&fin);
        }
    } else if (warp >= 18) {
        // the state in shared memory: stored, and met with the forward one for dg
        const long long E = (long long)a.dk * a.dv, plane = (long long)g.ch.total * a.H;
        for (int n = 0; n < nch && g.st; ++n) {
            const long long ci = (sg.c0 + chunk(n)) * a.H + h;
            float s = 0.0f;
            constexpr int NP = DK / 32;   // 16-byte pieces of a thread
            // of the forward state, all of it on its way before the wait: added up only
            // behind it (389 -> 339 us for both directions at the training shape)
            uint4 y[3][NP];
            if (g.dot) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const int idx = (warp - 18) * 32 + lane + 256 * i, r = idx >> 3, c = tile * 64 + (idx & 7) * 8;
                    const __nv_bfloat16 *p = g.pst + ci * E + (long long)r * a.dv + c;
#pragma unroll
                    for (int t = 0; t < 3; ++t)
                        y[t][i] = r < a.dk && c < a.dv ? __ldg(reinterpret_cast<const uint4 *>(p + t * plane * E))
                                                       : make_uint4(0, 0, 0, 0);
                }
            }
            if (g.dot && n + 1 < nch) {
                // the next one's rows of 64 columns (a line each) into the L2 cache
#pragma unroll 1
                for (int i = (warp - 18) * 32 + lane; i < 3 * DK; i += 256) {
                    const int t = i / DK, r = i % DK;
                    const long long at = t * plane + (sg.c0 + chunk(n + 1)) * a.H + h;
                    const __nv_bfloat16 *p = g.pst + at * E + (long long)r * a.dv + 64 * tile;
                    if (r < a.dk) asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
                }
            }
            if (!warp_wait(&staged, (uint32_t)n & 1u, &s_wait)) break;
            if (warp == 18 && lane == 0) {
#pragma unroll
                for (int t = 0; t < 3; ++t)
                    tma_store_3d(&ms, smem + SM::OUT + t * DK * 128, 64 * tile, 0, (int)(t * plane + ci));
                bulk_commit();
            }
            if (g.dot) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const int idx = (warp - 18) * 32 + lane + 256 * i;
                    const uint8_t *at = smem + SM::OUT + swz(idx >> 3, idx & 7);
                    float d[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                    float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int t = 0; t < 3; ++t) add_terms(f, y[t][i]);
#pragma unroll
                    for (int t = 0; t < 3; ++t) add_terms(d, *reinterpret_cast<const uint4 *>(at + t * DK * 128));
#pragma unroll
                    for (int j = 0; j < 8; ++j) s = fmaf(d[j], f[j], s);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (lane == 0 && SLSTM_IN((ci * 2 + tile) * 8 + warp - 18, (long long)g.ch.total * a.H * 16))
                    g.dot[(ci * 2 + tile) * 8 + warp - 18] = s;
            }
            if (warp == 18 && lane == 0) bulk_wait_read_all();
            warp_arrive(&unstaged);
        }
        if (warp == 18 && lane == 0) bulk_wait_all();
    } else if (warp >= 8) {
        const int t = (warp & 3) * 32 + lane, half = (warp >> 2) & 1;
        for (int n = 0; n < nch; ++n) {
            const int s = n % NST;
            if (!warp_wait(&dfull[n % ND], (uint32_t)(n / ND) & 1u, &s_wait)) break;
            if (!warp_wait(&full[s], (uint32_t)(n / NST) & 1u, &s_wait)) break;
            // the product that read this buffer two chunks ago
            if (n > 1 && !warp_wait(&delta[n & 1], ((uint32_t)(n >> 1) & 1u) ^ 1u, &s_wait)) break;
            uint8_t *st = smem + s * SM::STAGE;
            const TcDecays &d = dec[n % ND];
            const int len = rows(n);
            uint8_t *y = st + SM::NB * BOX;
            scale_row(y, y, smem + SM::Y + (n & 1) * 2 * BOX, t, 4 * half, 4 * half + 4,
                      back ? a.scale * d.row[t] : d.col[t], t < len);
            // rows behind a packed sequence belong to another one
            if (packed && t >= len)
                for (int i = half; i < SM::NB; i += 2) zero_row(st + i * BOX, t);
            tma_store_fence();
            warp_arrive(&yready[n & 1]);
            warp_arrive(&dempty[n % ND]);
        }
    } else {
        typedef Share<DK> SH;
        const int r = SH::row(warp, lane), c0 = SH::col(warp), col = tile * 64 + c0;
        const long long E = (long long)a.dk * a.dv;
        const float *src = g.init && !sg.only ? g.init + ((long long)sg.item * a.H + h) * E
                                              : (g.first ? g.first + ((long long)sg.seq * a.H + h) * E
                                                         : nullptr);
        float S[SH::N];
        state_load(S, src, a.dk, a.dv, r, col);
        float run = 1.0f;
        bool ok = true;
        for (int n = 0; n < nch; ++n) {
            if (g.st) {
                if (n > 0 && !warp_wait(&unstaged, (uint32_t)(n - 1) & 1u, &s_wait)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < SH::N; i += 8) {
                    uint32_t y[4][3];
#pragma unroll
                    for (int j = 0; j < 4; ++j) three_terms(S[i + 2 * j], S[i + 2 * j + 1], y[j]);
                    uint8_t *at = smem + SM::OUT + swz(r, (c0 + i) / 8);
#pragma unroll
                    for (int t = 0; t < 3; ++t)
                        *reinterpret_cast<uint4 *>(at + t * DK * 128) =
                            make_uint4(y[0][t], y[1][t], y[2][t], y[3][t]);
                }
                tma_store_fence();
                warp_arrive(&staged);
            }
            if (!warp_wait(&dfull[n % ND], (uint32_t)(n / ND) & 1u, &s_wait) ||
                !warp_wait(&delta[n & 1], (uint32_t)(n >> 1) & 1u, &s_wait)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const float tot = dec[n % ND].tot;
            run = run < 0.0f || tot < 0.0f ? -1.0f : run * tot;
            state_add(S, tot, tmem + (n & 1) * 128 + c0 + ((uint32_t)((warp & 3) * 32) << 16));
            tc_fence_before();
            warp_arrive(&drained[n & 1]);
            warp_arrive(&dempty[n % ND]);
        }
        if (!ok) {
#pragma unroll
            for (int i = 0; i < SH::N; ++i) S[i] = __int_as_float(0x7fc00000);
        }
        float *dst = g.fin ? g.fin + ((long long)sg.item * a.H + h) * E
                           : (g.last && sg.only ? g.last + ((long long)sg.seq * a.H + h) * E : nullptr);
        if (dst)
            state_store(S, dst, a.dk, a.dv, r, col, g.fin ? g.fin : g.last,
                        (long long)(g.fin ? g.seg.total : g.seg.n_seq) * a.H * E);
        if (g.fin && tile == 0 && threadIdx.x == 0 &&
            SLSTM_IN((long long)sg.item * a.H + h, (long long)g.seg.total * a.H))
            g.fin_tot[(long long)sg.item * a.H + h] = run;
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        if (s_wait.gave_up)
            for (int n = max(0, s_loaded - NST); n < s_loaded; ++n)
                {
                (void)mbar_wait(&full[n % NST], (uint32_t)(n / NST) & 1u, TC_WAIT_NS);
                (void)mbar_wait(&dfull[n % ND], (uint32_t)(n / ND) & 1u, TC_WAIT_NS);
            }
        (void)mbar_wait(&fin, 0u, TC_WAIT_NS);
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_free<256>(tmem);
    }
    if (!s_wait.gave_up || !g.st) return;
    // what this block has not stored is not known any more
    Seg lost;
    seg_of(g, item, &lost);
    const int cols = min(64, a.dv - 64 * tile);
#pragma unroll 1
    for (int n = 0; n < lost.nch; ++n) {
        const long long ci = (lost.c0 + n) * a.H + h;
#pragma unroll 1
        for (int i = threadIdx.x; i < a.dk * cols; i += STATE_THREADS)
            g.st[ci * a.dk * a.dv + (long long)(i / cols) * a.dv + 64 * tile + i % cols] = bf16_nan();
        if (g.dot && threadIdx.x < 8) g.dot[(ci * 2 + tile) * 8 + threadIdx.x] = __int_as_float(0x7fc00000);
    }
}

// ---------------------------------------------------------------------------
// The forward pass of a segment: one block walks the chunks of one head and 64
// columns of v and does all of it while q, k and v are in shared memory, the
// state in registers:
//   warps 0-7   the state (lane = row of d_k), its two terms into shared memory
//               and half of v times its decays as three bf16 terms
//   warps 8-11  the other half
//   warps 12-19 the weights D (q k) from tensor memory and back as two bf16 terms
//               (lane = query row, half of the keys each)
//   warps 20-23 the outputs
//   warp 24     the MMAs of k^T (w v);  warp 25 the other MMAs
//   warp 26     loads (a ring of NST chunks)
// Each of these is a chain of latencies some 1500 cycles long; apart from one
// another they run a chunk or two ahead or behind, and a chunk takes as long as
// the longest of them, not as all.
// A chunk's products: q k^T (128 x 128; of the next chunk ahead of the last of
// this one where its rows have come), k^T (w v), and into an accumulator each
// q S, whose rows are scaled in fp32 as they are read, and D(q k) v with the
// weights in tensor memory, in the place of their scores.
// 8 rows of 8192 steps, 8 heads of 128: 205 us; reading and writing each tensor
// once would take 84.  No one part of the work bounds it: with k^T (w v) left out
// the call takes 91 % of its time, without the outputs' products or their stores
// 92 %, without splitting w v 97 %, without the scores, the weights or the loads
// all of it; what is left is the waits of a chunk's parts for one another.
// ---------------------------------------------------------------------------
template <int DK>
struct FwdShared {
    static constexpr int NST = DK == 128 ? 2 : 3;
    static constexpr int NB = DK / 64;
    static constexpr uint32_t STAGE = (2 * NB + 1) * BOX;   // q, k, v
    static constexpr uint32_t Y = NST * STAGE;              // three terms
    // The state's two terms: a buffer of their own where there is room for one (1 x
    // 65536, 16 heads of 64 x 128: 474 us, in the place of the keys 493).
    static constexpr bool OWN = DK == 64;
    static constexpr uint32_t S = Y + 3 * BOX;
    static constexpr uint32_t DEC = S + (OWN ? 2 * DK * 128 : 0);
    static constexpr uint32_t BYTES = DEC + ND * sizeof(TcDecays) + 1024;
};
static_assert(FwdShared<64>::BYTES + 512 <= 227 * 1024, "forward shared memory");
static_assert(FwdShared<128>::BYTES + 1024 <= 227 * 1024, "forward shared memory");

constexpr int FWD_THREADS = 864;

[[maybe_unused]] SLSTM_DEVINL long long tc_rows(const LaArgs &a)
{
    return a.cu ? (long long)a.T : (long long)a.B * a.T;
}

template <int DK>
__global__ void __launch_bounds__(FWD_THREADS, 1)
    la_forward_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, TcArgs g)
{
    typedef FwdShared<DK> SM;
    constexpr int NST = SM::NST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = aligned_smem(smem_raw);
    TcDecays *dec = reinterpret_cast<TcDecays *>(smem + SM::DEC);
    __shared__ uint64_t full[NST], empty[NST], vfull[NST], vempty[NST], dfull[ND], dempty[ND], scfull[2];
    __shared__ uint64_t yready, delta, sready[2], sfree, pready[2], ofull, oempty, tready, drained,
        fin;
    __shared__ uint32_t s_tmem;
    __shared__ Waits s_wait;
    __shared__ int s_loaded;
    const LaArgs &a = g.a;
    const int tile = blockIdx.x % g.tiles, h = (blockIdx.x / g.tiles) % a.H, item = blockIdx.x / (g.tiles * a.H);
    Seg sg;
    if (!seg_of(g, item, &sg)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool packed = g.seg.pos != nullptr;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 2);
            mbar_init(&vfull[i], 1);
            mbar_init(&vempty[i], 1);
        }
        for (int i = 0; i < ND; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], 24);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&scfull[i], 1);
        mbar_init(&yready, 12);
        mbar_init(&delta, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sready[i], 8);
            mbar_init(&pready[i], 8);
        }
        mbar_init(&sfree, 1);
        mbar_init(&ofull, 1);
        mbar_init(&oempty, 4);
        mbar_init(&tready, 4);
        mbar_init(&drained, 8);
        mbar_init(&fin, 2);
        mbar_init_fence();
        s_wait.gave_up = 0;
        s_wait.tries = a.tries;
        s_loaded = 0;
    }
    if (warp == 0) tmem_alloc<512>(&s_tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t t_o = tmem + 256, t_delta = tmem + 384;   // scores: 0 and 128; q S and D(q k) v: t_o and 64 on
    const int nch = sg.nch;
    // the last chunk of a packed sequence holds rows of the next one
    const int ragged = packed && sg.len % TCC != 0 ? nch - 1 : -1;

    if (warp == 26) {
        if (elect_one()) {
            const int hq = h / (a.H / a.Hqk);
            // q and k come back into use before v does
            auto load = [&](int n) -> bool {
                const int s = n % NST;
                const uint32_t ph = ((uint32_t)(n / NST) & 1u) ^ 1u;
                if (!lane_wait(&empty[s], ph, &s_wait)) return false;
                uint8_t *st = smem + s * SM::STAGE;
                mbar_expect_tx(&full[s], 2 * SM::NB * BOX);
                const int t = sg.t + n * TCC;
#pragma unroll
                for (int i = 0; i < SM::NB; ++i) {
                    tma_load_4d(st + i * BOX, &mq, &full[s], 64 * i, hq, t, sg.b);
                    tma_load_4d(st + (SM::NB + i) * BOX, &mk, &full[s], 64 * i, hq, t, sg.b);
                }
                s_loaded = 2 * n + 1;
                if (!lane_wait(&dempty[n % ND], ((uint32_t)(n / ND) & 1u) ^ 1u, &s_wait)) return false;
                if (!lane_wait(&vempty[s], ph, &s_wait)) return false;
                mbar_expect_tx(&dfull[n % ND], sizeof(TcDecays));
                bulk_load(&dec[n % ND], g.dec + (sg.c0 + n) * a.H + h, sizeof(TcDecays), &dfull[n % ND]);
                mbar_expect_tx(&vfull[s], BOX);
                tma_load_4d(st + 2 * SM::NB * BOX, &mv, &vfull[s], 64 * tile, h, t, sg.b);
                s_loaded = 2 * n + 2;
                return true;
            };
            for (int n = 0; n < nch && n + 1 != a.debug_fault; ++n)
                if (!load(n)) break;
        }
    } else if (warp == 24) {
        if (elect_one()) {
            constexpr uint32_t id_kv = idesc_bf16(128, 128, true, true), id_k3 = idesc_bf16(128, 64, true, true);
            bool ok = true;
            for (int n = 0; n < nch && ok; ++n) {
                const int s = n % NST;
                const uint32_t ph = (uint32_t)n & 1u;
                ok = lane_wait(&full[s], (uint32_t)(n / NST) & 1u, &s_wait) && lane_wait(&yready, ph, &s_wait) &&
                     lane_wait(&drained, ph ^ 1u, &s_wait);
                if (!ok) break;
                tc_fence_after();
                // two terms of w v side by side, k being read once for them, and the
                // third into the sum of the second; the 64 rows of a narrow d_k twice
                // (no step from one 64 to the next)
                const uint64_t kt =
                    smem_desc_mn_sw128(smem_u32(smem + s * SM::STAGE + SM::NB * BOX), DK == 128 ? BOX : 0u);
                const uint64_t yd = smem_desc_mn_sw128(smem_u32(smem + SM::Y), BOX);
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                    umma_bf16(t_delta, kt + (2048u >> 4) * k, yd + (2048u >> 4) * k, id_kv, k > 0 ? 1u : 0u);
                    umma_bf16(t_delta + 64, kt + (2048u >> 4) * k, yd + (2 * BOX >> 4) + (2048u >> 4) * k, id_k3, 1u);
                }
                umma_commit(&delta);
                umma_commit(&empty[s]);
            }
            umma_commit(&fin);
        }
    } else if (warp == 25) {
        if (elect_one()) {
            constexpr uint32_t id_qk = idesc_bf16(128, 128, false, false);
            constexpr uint32_t id_o = idesc_bf16(128, 64, false, true);
            // q k^T of chunk n; unless `must`, only if its rows are there
            int scored = 0;
            auto scores = [&](int n, bool must) -> bool {
                const int s = n % NST;
                if (!must && (!done(&full[s], (uint32_t)(n / NST) & 1u) || (n == ragged && !done(&tready, 0u))))
                    return true;
                if (!lane_wait(&full[s], (uint32_t)(n / NST) & 1u, &s_wait)) return false;
                if (n == ragged && !lane_wait(&tready, 0u, &s_wait)) return false;
                scored = n + 1;
                tc_fence_after();
                const uint8_t *st = smem + s * SM::STAGE;
#pragma unroll
                for (int i = 0; i < SM::NB; ++i) {
                    const uint64_t qd = smem_desc_k_sw128(smem_u32(st + i * BOX));
                    const uint64_t kd = smem_desc_k_sw128(smem_u32(st + (SM::NB + i) * BOX));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16(tmem + (n & 1) * 128, qd + 2 * k, kd + 2 * k, id_qk, (i > 0 || k > 0) ? 1u : 0u);
                }
                umma_commit(&scfull[n & 1]);
                return true;
            };
            bool ok = true;
            for (int n = 0; n < nch && ok; ++n) {
                const int s = n % NST;
                const uint32_t ph = (uint32_t)n & 1u;
                const uint8_t *st = smem + s * SM::STAGE;
                ok = scored > n || scores(n, true);
                if (!ok) break;
                // the next chunk's scores go ahead of this one's outputs when its
                // rows have come, and never make them wait
                if (n + 1 < nch) {
#pragma unroll 1
                    for (int i = 0; i < (1 << 20); ++i) {
                        if (scored > n + 1 || done(&pready[ph], (uint32_t)(n >> 1) & 1u) ||
                            *(volatile int *)&s_wait.gave_up)
                            break;
                        scores(n + 1, false);
                    }
                }
                ok = lane_wait(&sready[ph], (uint32_t)(n >> 1) & 1u, &s_wait) &&
                     lane_wait(&oempty, ph ^ 1u, &s_wait);
                if (!ok) break;
                tc_fence_after();
                const uint64_t sd =
                    smem_desc_mn_sw128(smem_u32(SM::OWN ? smem + SM::S : st + SM::NB * BOX), BOX);
                const uint64_t vd = smem_desc_mn_sw128(smem_u32(st + 2 * SM::NB * BOX), BOX);
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int i = 0; i < SM::NB; ++i) {
                        const uint64_t qd = smem_desc_k_sw128(smem_u32(st + i * BOX));
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_bf16(t_o, qd + 2 * k, sd + (DK * 128u >> 4) * t + (2048u >> 4) * (4 * i + k), id_o,
                                      (t > 0 || i > 0 || k > 0) ? 1u : 0u);
                    }
                }
                if (SM::OWN) umma_commit(&sfree);
                umma_commit(&empty[s]);
                ok = lane_wait(&vfull[s], (uint32_t)(n / NST) & 1u, &s_wait) &&
                     lane_wait(&pready[ph], (uint32_t)(n >> 1) & 1u, &s_wait);
                if (!ok) break;
                tc_fence_after();
                const uint32_t ta = tmem + ph * 128;
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                    umma_bf16_ta(t_o + 64, ta + 16 * k, vd + (2048u >> 4) * k, id_o, k > 0 ? 1u : 0u);
                    umma_bf16_ta(t_o + 64, ta + 16 * k + 8, vd + (2048u >> 4) * k, id_o, 1u);
                }
                umma_commit(&vempty[s]);
                umma_commit(&ofull);
            }
            umma_commit(&fin);
        }
    } else if (warp < 8) {
        typedef Share<DK> SH;
        const int r = SH::row(warp, lane), c0 = SH::col(warp), col = tile * 64 + c0;
        const long long E = (long long)a.dk * a.dv;
        const float *src = g.init && !sg.only ? g.init + ((long long)sg.item * a.H + h) * E
                                              : (g.first ? g.first + ((long long)sg.seq * a.H + h) * E
                                                         : nullptr);
        float S[SH::N];
        state_load(S, src, a.dk, a.dv, r, col);
        // the other half of v's columns: w v is what the next chunk's product waits for
        auto scale = [&](int n) -> bool {
            const int s = n % NST, t = (warp & 3) * 32 + lane, p = 4 + 2 * (warp >> 2);
            if (!warp_wait(&vfull[s], (uint32_t)(n / NST) & 1u, &s_wait) ||
                !warp_wait(&dfull[n % ND], (uint32_t)(n / ND) & 1u, &s_wait))
                return false;
            scale_row(smem + s * SM::STAGE + 2 * SM::NB * BOX, smem + SM::Y, smem + SM::Y + BOX, t, p, p + 2,
                      dec[n % ND].col[t], t < sg.len - n * TCC);
            tma_store_fence();
            warp_arrive(&yready);
            return true;
        };
        bool ok = scale(0);
        for (int n = 0; n < nch && ok; ++n) {
            const uint32_t ph = (uint32_t)n & 1u;
            // The state's terms, row r: the B operands of q S.  Where there is no room for
            // a buffer of their own they go where the chunk's keys were, once both products
            // that read those are done.
            if (SM::OWN) ok = n == 0 || warp_wait(&sfree, ph ^ 1u, &s_wait);
            else ok = warp_wait(&delta, ph, &s_wait) && warp_wait(&scfull[n & 1], (uint32_t)(n >> 1) & 1u, &s_wait);
            if (!ok) break;
            uint8_t *at = smem + (SM::OWN ? SM::S : (n % NST) * SM::STAGE + SM::NB * BOX);
#pragma unroll
            for (int i = 0; i < SH::N / 8; ++i) {
                uint32_t y[4], z[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) two_terms(S[8 * i + 2 * j], S[8 * i + 2 * j + 1], y[j], z[j]);
                *reinterpret_cast<uint4 *>(at + swz(r, c0 / 8 + i)) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4 *>(at + DK * 128 + swz(r, c0 / 8 + i)) = make_uint4(z[0], z[1], z[2], z[3]);
            }
            tma_store_fence();
            warp_arrive(&sready[ph]);
            if (SM::OWN) ok = warp_wait(&delta, ph, &s_wait);
            ok = ok && (n + 1 >= nch || scale(n + 1));
            if (!ok) break;
            tc_fence_after();
            state_add(S, dec[n % ND].tot, t_delta + c0 + ((uint32_t)((warp & 3) * 32) << 16));
            tc_fence_before();
            warp_arrive(&drained);
            warp_arrive(&dempty[n % ND]);
        }
        if (!ok)
#pragma unroll
            for (int i = 0; i < SH::N; ++i) S[i] = __int_as_float(0x7fc00000);
        if (g.last && sg.only)
            state_store(S, g.last + ((long long)sg.seq * a.H + h) * E, a.dk, a.dv, r, col, g.last,
                        (long long)g.seg.n_seq * a.H * E);
    } else if (warp < 12) {
        const int t = (warp & 3) * 32 + lane;
        for (int n = 0; n < nch; ++n) {
            const int s = n % NST, len = min(TCC, sg.len - n * TCC);
            uint8_t *st = smem + s * SM::STAGE;
            if (!warp_wait(&vfull[s], (uint32_t)(n / NST) & 1u, &s_wait)) break;
            if (n == ragged) {
                if (!warp_wait(&full[s], (uint32_t)(n / NST) & 1u, &s_wait)) break;
                if (t >= len)
                    for (int i = 0; i < 2 * SM::NB + 1; ++i) zero_row(st + i * BOX, t);
                tma_store_fence();
                warp_arrive(&tready);
            }
            if (!warp_wait(&dfull[n % ND], (uint32_t)(n / ND) & 1u, &s_wait)) break;
            // the product that read the last terms
            if (n > 0 && !warp_wait(&delta, (uint32_t)(n - 1) & 1u, &s_wait)) break;
            const float w = dec[n % ND].col[t];
            scale_row(st + 2 * SM::NB * BOX, smem + SM::Y, smem + SM::Y + BOX, t, 0, 4, w, t < len);
            tma_store_fence();
            warp_arrive(&yready);
            warp_arrive(&dempty[n % ND]);
        }
    } else if (warp < 20) {
        const int q = warp & 3, half = ((warp - 12) >> 2) & 1;
        const int i = q * 32 + lane;   // query row
        const uint32_t la = (uint32_t)(q * 32) << 16;
        for (int n = 0; n < nch; ++n) {
            if (!warp_wait(&dfull[n % ND], (uint32_t)(n / ND) & 1u, &s_wait)) break;
            if (!warp_wait(&scfull[n & 1], (uint32_t)(n >> 1) & 1u, &s_wait)) break;
            tc_fence_after();
            const TcDecays &d = dec[n % ND];
            // 64 keys of this warp; the two terms of 16 weights in the place of their scores
            const uint32_t sc = tmem + (n & 1) * 128 + 64 * half + la;
            const float ri = d.rq[i], li = d.loc[i], mi = d.rest[i];
            const int f = max(d.first[i] - 32 * q, 0);   // first key of its own 32 that reaches the query
            const uint32_t span = (uint32_t)(lane - f);
#pragma unroll 1
            for (int z = 0; z < 4; ++z) {   // 16 keys at a time
                const int b = 2 * half + (z >> 1), key = 64 * half + 16 * z;
                uint32_t p[16];   // 8 columns of the upper terms, 8 of the lower
                if (b <= q) {
                    float v[16];
                    tmem_ld16(sc + 16 * z, v);
                    if (b < q) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 e = *reinterpret_cast<const float4 *>(d.cq(q) + key + j);
                            two_terms(v[j] * (ri * e.x), v[j + 1] * (ri * e.y), p[j / 2], p[8 + j / 2]);
                            two_terms(v[j + 2] * (ri * e.z), v[j + 3] * (ri * e.w), p[j / 2 + 1], p[9 + j / 2]);
                        }
                    } else {
                        const int k0 = 16 * (z & 1) - f;
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 l = *reinterpret_cast<const float4 *>(&d.loc[key + j]);
                            const float4 m = *reinterpret_cast<const float4 *>(&d.rest[key + j]);
                            const float e[4] = {ex2((li - l.x) + (mi - m.x)), ex2((li - l.y) + (mi - m.y)),
                                                ex2((li - l.z) + (mi - m.z)), ex2((li - l.w) + (mi - m.w))};
                            float x[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                x[k] = (uint32_t)(k0 + j + k) <= span ? v[j + k] * e[k] : 0.0f;
                            two_terms(x[0], x[1], p[j / 2], p[8 + j / 2]);
                            two_terms(x[2], x[3], p[j / 2 + 1], p[9 + j / 2]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) p[j] = 0u;
                }
                tmem_st16(sc + 16 * z, p);
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&pready[n & 1]);
            warp_arrive(&dempty[n % ND]);
        }
    } else {
        const int i = (warp & 3) * 32 + lane;   // query row
        const uint32_t la = (uint32_t)((warp & 3) * 32) << 16;
        [[maybe_unused]] const long long all = tc_rows(a) * a.H * a.dv;
        [[maybe_unused]] const __nv_bfloat16 *base = static_cast<const __nv_bfloat16 *>(a.o);
        const int cols = min(64, a.dv - tile * 64);
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + (sg.row + i) * (long long)a.H * a.dv +
                           (long long)h * a.dv + tile * 64;
        const long long step = (long long)TCC * a.H * a.dv;
        bool ok = true;
        int n = 0;
        for (; n < nch; ++n) {
            ok = warp_wait(&dfull[n % ND], (uint32_t)(n / ND) & 1u, &s_wait);
            if (!ok) break;
            const float rowc = dec[n % ND].row[i] * a.scale;
            const bool open = dec[n % ND].first[i] < 0;   // the state reaches the row
            warp_arrive(&dempty[n % ND]);
            ok = warp_wait(&ofull, (uint32_t)n & 1u, &s_wait);
            if (!ok) break;
            tc_fence_after();
            const bool on = n * TCC + i < sg.len;
#pragma unroll 1
            for (int c = 0; c < 64; c += 16) {
                float u[16], w[16];
                tmem_ld16x2(t_o + la + c, t_o + 64 + la + c, u, w);
                if (c == 48) {
                    tc_fence_before();
                    warp_arrive(&oempty);
                }
                uint32_t p[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    p[j] = pack2(fmaf(rowc, open ? u[2 * j] : 0.0f, a.scale * w[2 * j]),
                                 fmaf(rowc, open ? u[2 * j + 1] : 0.0f, a.scale * w[2 * j + 1]));
                uint4 *dst = reinterpret_cast<uint4 *>(o + n * step + c);
                if (on && c < cols && SLSTM_PIN(o + n * step + c + 7, base, all))
                    dst[0] = make_uint4(p[0], p[1], p[2], p[3]);
                if (on && c + 8 < cols && SLSTM_PIN(o + n * step + c + 15, base, all))
                    dst[1] = make_uint4(p[4], p[5], p[6], p[7]);
            }
        }
        if (!ok)
            for (; n < nch && n * TCC + i < sg.len; ++n)
                for (int j = 0; j < cols; ++j) o[n * step + j] = bf16_nan();
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        if (s_wait.gave_up)
            for (int n = max(0, (s_loaded + 1) / 2 - NST); 2 * n < s_loaded; ++n) {
                (void)mbar_wait(&full[n % NST], (uint32_t)(n / NST) & 1u, TC_WAIT_NS);
                if (2 * n + 1 >= s_loaded) break;
                (void)mbar_wait(&vfull[n % NST], (uint32_t)(n / NST) & 1u, TC_WAIT_NS);
                (void)mbar_wait(&dfull[n % ND], (uint32_t)(n / ND) & 1u, TC_WAIT_NS);
            }
        (void)mbar_wait(&fin, 0u, TC_WAIT_NS);
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_free<512>(tmem);
    }
}

// ---------------------------------------------------------------------------
// The gradients of a chunk and head, given the state that enters it and the
// gradient of the state that leaves it (three bf16 terms each).  Persistent
// blocks; item = chunk * H + head.  Everything with a key's row per lane:
//   q k^T and dO v^T transposed (lane = key j, column = query i), from which
//   come P_ij = scale D_ij (q_i . k_j), Pd_ij = scale D_ij (dO_i . v_j) and the
//   row and column sums of W = P (dO v) for dg;  then
//   dq = Pd k + scale e^{c_i} dO S^T,   dk = Pd^T q + e^{c_C - c_j} v dS^T,
//   dv = P^T dO + e^{c_C - c_j} k dS
// with two terms each of P^T in tensor memory and of Pd^T in shared memory (read
// both ways round).  The products with the states come first; their rows are
// scaled in tensor memory, where the other products are then added.  u_i and w_j
// of dg are the dot products of q_i and k_j with those rows.
//   warps 0-15  lane quarter q = warp & 3, columns 32 b .. of b = warp >> 2
//   warp 16     loads;  warp 17 MMAs;  warp 18 dg
// Tensor memory: [0, 128) q k^T, then dv; [128, 256) dO v^T, then P^T;
// [256, 384) dq; [384, 512) dk.  Shared memory holds q, k, v, dO and five slots
// of 16 KB: the tiles of S and then of dS, a term of 64 columns each, go through
// them as a ring, and the terms of Pd^T take the first four after that.  Bound:
// the bytes of q, k, v, dO, the two states and the gradients (1.7 GB for 8 rows of
// 8192 steps, 8 heads of 128, 270 us at the measured rate; it takes 360: no one part,
// left out, takes off more than 13 %).
// ---------------------------------------------------------------------------
struct BackArgs {
    LaArgs a;
    const TcDecays *dec;   // [chunk][h]
    LaChunks ch;
    int total;             // items where the sequences are dense
    float *part_q, *part_k;
    float *dgc;            // [chunk][h]
    const float *dot;
    int tiles;
};

template <int DK, int DV>
struct BackShared {
    static constexpr int NK = DK / 64, NV = DV / 64;
    static constexpr uint32_t Q = 0, K = NK * BOX, V = 2 * NK * BOX, G = V + NV * BOX, X = G + NV * BOX;
    static constexpr int NT = 6 * NV;     // tiles of the states, a term of 64 columns each, S's and then dS's
    static constexpr int NS = 5;          // slots that they go through
    // Term and 64 columns of tile i.  Of dS the third terms come first: the others
    // stay until q k^T and dO v^T have been read, and their slots are free by then.
    static constexpr int term(int i) { return i < 3 * NV ? i % 3 : i < 4 * NV ? 2 : (i - 4 * NV) / NV; }
    static constexpr int half(int i) { return i < 3 * NV ? i / 3 : i % NV; }
    static constexpr uint32_t DEC = X + NS * BOX;
    static constexpr uint32_t SUMS = DEC + 2 * sizeof(TcDecays);
    // the parts of r, u, w of each column block and of c of each lane quarter's columns
    static constexpr uint32_t BYTES = SUMS + 16 * TCC * 4 + 1024;
};
static_assert((4 * 2 + 1) % 5 == 4 && (5 * 2) % 5 == 0, "the two halves of a term of dS in slots one behind the other");
static_assert(BackShared<128, 128>::BYTES + 1024 <= 227 * 1024, "backward shared memory");

constexpr int BACK_THREADS = 608;

// A thread's 32 columns of a row in bf16 from a swizzled box pair.
SLSTM_DEVINL float dot_row(const uint8_t *tile, int row, int b, const float (&v)[32])
{
    const uint8_t *box = tile + (b >> 1) * BOX;
    float s = 0.0f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint4 x = *reinterpret_cast<const uint4 *>(box + swz(row, 4 * (b & 1) + p));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s = fmaf(lo_of(w[j]), v[8 * p + 2 * j], s);
            s = fmaf(hi_of(w[j]), v[8 * p + 2 * j + 1], s);
        }
    }
    return s;
}

// A warp's 32 rows (one a lane) of 32 columns to global memory, `cols` of them
// and rows below `rows`, ld elements apart, by way of 2 KB (bf16) or 4 KB (fp32)
// of shared memory of its own: lanes that stand in a row then write its pieces
// side by side, 8 (4) rows an access.  Straight from the registers an access
// goes to 32 lines, and the outputs of a chunk took 9000 cycles, now 5000.
SLSTM_DEVINL void put_rows(__nv_bfloat16 *dst, long long ld, const float (&v)[32], int cols, int rows, uint8_t *stage,
                           int lane, [[maybe_unused]] const __nv_bfloat16 *base, [[maybe_unused]] long long n)
{
#pragma unroll
    for (int p = 0; p < 4; ++p)
        *reinterpret_cast<uint4 *>(stage + lane * 64 + ((p ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(pack2(v[8 * p], v[8 * p + 1]), pack2(v[8 * p + 2], v[8 * p + 3]),
                       pack2(v[8 * p + 4], v[8 * p + 5]), pack2(v[8 * p + 6], v[8 * p + 7]));
    __syncwarp();
    const int p = lane & 3;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = 8 * k + (lane >> 2);
        const uint4 x = *reinterpret_cast<const uint4 *>(stage + r * 64 + ((p ^ ((r >> 1) & 3)) << 4));
        if (r < rows && 8 * p < cols && SLSTM_PIN(dst + r * ld + 8 * p + 7, base, n))
            *reinterpret_cast<uint4 *>(dst + r * ld + 8 * p) = x;
    }
    __syncwarp();
}
SLSTM_DEVINL void put_rows(float *dst, long long ld, const float (&v)[32], int cols, int rows, uint8_t *stage,
                           int lane, [[maybe_unused]] const float *base, [[maybe_unused]] long long n)
{
#pragma unroll
    for (int p = 0; p < 8; ++p)
        *reinterpret_cast<float4 *>(stage + lane * 128 + ((p ^ (lane & 7)) << 4)) =
            make_float4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
    __syncwarp();
    const int p = lane & 7;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int r = 4 * k + (lane >> 3);
        const uint4 x = *reinterpret_cast<const uint4 *>(stage + r * 128 + ((p ^ (r & 7)) << 4));
        if (r < rows && 4 * p < cols && SLSTM_PIN(dst + r * ld + 4 * p + 3, base, n))
            *reinterpret_cast<uint4 *>(dst + r * ld + 4 * p) = x;
    }
    __syncwarp();
}

template <int DK, int DV>
__global__ void __launch_bounds__(BACK_THREADS, 1)
    la_backward_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mg,
                       const __grid_constant__ CUtensorMap ms, const __grid_constant__ CUtensorMap md, BackArgs g)
{
    typedef BackShared<DK, DV> SM;
    constexpr int NK = SM::NK, NV = SM::NV, NT = SM::NT, NS = SM::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = aligned_smem(smem_raw);
    TcDecays *dec = reinterpret_cast<TcDecays *>(smem + SM::DEC);
    float(*sums)[TCC] = reinterpret_cast<float(*)[TCC]>(smem + SM::SUMS);   // r: 0-3, c: 4-7, u: 8-11, w: 12-15
    uint8_t *x0 = smem + SM::X, *x1 = x0 + 2 * BOX;
    __shared__ uint64_t full1, full2, sfull[NS], sempty[NS], dfull[2], dempty[2], bsc, bdqi, bdki, scfree, pready,
        bout, tfree, xfree, tready, sumfree, fin;
    __shared__ uint32_t s_tmem;
    __shared__ Waits s_wait;
    __shared__ int s_items, s_tiles;   // items whose loads have begun, and tiles of the last of them
    const LaArgs &a = g.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool packed = g.ch.pos != nullptr;
    const int items = packed ? g.ch.coff[g.ch.n_seq] * a.H : g.total;
    if ((int)blockIdx.x >= items) return;
    if (threadIdx.x == 0) {
        mbar_init(&full1, 1);
        mbar_init(&full2, 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&sempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], 17);
        }
        mbar_init(&bsc, 1);
        mbar_init(&bdqi, 1);
        mbar_init(&bdki, 1);
        mbar_init(&scfree, 16);
        mbar_init(&pready, 16);
        mbar_init(&bout, 1);
        mbar_init(&tfree, 16);
        mbar_init(&xfree, 16);
        mbar_init(&tready, 16);
        mbar_init(&sumfree, 1);
        mbar_init(&fin, 1);
        mbar_init_fence();
        s_wait.gave_up = 0;
        s_wait.tries = a.tries;
        s_items = s_tiles = 0;
    }
    if (warp == 0) tmem_alloc<512>(&s_tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t R0 = tmem, R1 = tmem + 128, R2 = tmem + 256, R3 = tmem + 384;
    const int rep = a.H / a.Hqk;
    // tile i of the it-th item: its slot's phase
    auto phase = [](int it, int i) { return (uint32_t)(it * ((NT - i % NS + NS - 1) / NS) + i / NS); };

    if (warp == 16) {
        if (elect_one()) {
            const int plane = g.ch.total * a.H;
            int it = 0;
            for (int item = blockIdx.x; item < items; item += gridDim.x, ++it) {
                if (it + 1 == a.debug_fault) break;
                const int h = item % a.H, c = item / a.H, hq = h / rep;
                const LaChunk ck = la_chunk(g.ch, c);
                const int t = packed ? (int)ck.row : ck.n * TCC, b = packed ? 0 : ck.seq;
                const uint32_t ph = (uint32_t)it & 1u;
                if (it > 0 && !lane_wait(&bout, ph ^ 1u, &s_wait)) break;
                if (!lane_wait(&dempty[it & 1], ((uint32_t)(it >> 1) & 1u) ^ 1u, &s_wait)) break;
                mbar_expect_tx(&dfull[it & 1], sizeof(TcDecays));
                bulk_load(&dec[it & 1], g.dec + item, sizeof(TcDecays), &dfull[it & 1]);
                mbar_expect_tx(&full1, 2 * NK * BOX);
#pragma unroll
                for (int i = 0; i < NK; ++i) {
                    tma_load_4d(smem + SM::Q + i * BOX, &mq, &full1, 64 * i, hq, t, b);
                    tma_load_4d(smem + SM::K + i * BOX, &mk, &full1, 64 * i, hq, t, b);
                }
                mbar_expect_tx(&full2, 2 * NV * BOX);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    tma_load_4d(smem + SM::V + i * BOX, &mv, &full2, 64 * i, h, t, b);
                    tma_load_4d(smem + SM::G + i * BOX, &mg, &full2, 64 * i, h, t, b);
                }
                s_tiles = 0;
                s_items = it + 1;
                if (it > 0 && !lane_wait(&xfree, ph ^ 1u, &s_wait)) break;
                bool ok = true;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int s = i % NS;
                    if (i >= NS) ok = ok && lane_wait(&sempty[s], (phase(it, i) - 1u) & 1u, &s_wait);
                    if (!ok) break;
                    mbar_expect_tx(&sfull[s], DK * 128);
                    tma_load_3d(x0 + s * BOX, i < 3 * NV ? &ms : &md, &sfull[s], 64 * SM::half(i), 0,
                                SM::term(i) * plane + item);
                    s_tiles = i + 1;
                }
                if (!ok) break;
                // the next item's rows into the L2 cache while this one is
                // computed: a block has room for one item
                const int next = item + gridDim.x;
                if (next < items) {
                    const int h2 = next % a.H, hq2 = h2 / rep;
                    const LaChunk c2 = la_chunk(g.ch, next / a.H);
                    const int t2 = packed ? (int)c2.row : c2.n * TCC, b2 = packed ? 0 : c2.seq;
#pragma unroll
                    for (int i = 0; i < NK; ++i) {
                        tma_prefetch_4d(&mq, 64 * i, hq2, t2, b2);
                        tma_prefetch_4d(&mk, 64 * i, hq2, t2, b2);
                    }
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        tma_prefetch_4d(&mv, 64 * i, h2, t2, b2);
                        tma_prefetch_4d(&mg, 64 * i, h2, t2, b2);
                    }
                }
            }
        }
    } else if (warp == 17) {
        if (elect_one()) {
            constexpr uint32_t id_ss = idesc_bf16(128, 128, false, false);   // q k^T, dO v^T
            constexpr uint32_t id_si = idesc_bf16(128, DK, false, false);    // dO S^T, v dS^T
            constexpr uint32_t id_kd = idesc_bf16(128, DV, false, true);     // k dS, P^T dO
            constexpr uint32_t id_dk = idesc_bf16(128, DK, false, true);     // Pd^T q
            constexpr uint32_t id_dq = idesc_bf16(128, DK, true, true);      // Pd k
            // A (128 rows) by B over 64 NB deep K-major tiles
            auto inner = [&](uint32_t d, uint32_t at, uint32_t bt, uint32_t bstride, int nb, uint32_t id, bool add) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (i >= nb) break;
                    const uint64_t ad = smem_desc_k_sw128(at + i * BOX), bd = smem_desc_k_sw128(bt + i * bstride);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16(d, ad + 2 * k, bd + 2 * k, id, (add || i > 0 || k > 0) ? 1u : 0u);
                }
            };
            const uint32_t sm = smem_u32(smem), sx0 = smem_u32(x0), sx1 = smem_u32(x1);
            auto tile = [&](int it, int i) {
                const bool ok = lane_wait(&sfull[i % NS], phase(it, i) & 1u, &s_wait);
                tc_fence_after();
                return ok;
            };
            int it = 0, ragged = 0;
            for (int item = blockIdx.x; item < items; item += gridDim.x, ++it) {
                const uint32_t ph = (uint32_t)it & 1u;
                if (!lane_wait(&full1, ph, &s_wait)) break;
                if (packed && la_chunk(g.ch, item / a.H).len < TCC) {
                    // rows behind a ragged chunk are cleared before they are read
                    if (!lane_wait(&tready, (uint32_t)ragged & 1u, &s_wait)) break;
                    ++ragged;
                }
                if (it > 0 && !lane_wait(&tfree, ph ^ 1u, &s_wait)) break;
                tc_fence_after();
                inner(R0, sm + SM::K, sm + SM::Q, BOX, NK, id_ss, false);
                if (!lane_wait(&full2, ph, &s_wait)) break;
                tc_fence_after();
                inner(R1, sm + SM::V, sm + SM::G, BOX, NV, id_ss, false);
                umma_commit(&bsc);
                bool ok = true;
#pragma unroll
                for (int i = 0; i < 3 * NV && ok; ++i) {
                    if (!(ok = tile(it, i))) break;
                    inner(R2, sm + SM::G + SM::half(i) * BOX, sx0 + i % NS * BOX, 0, 1, id_si, i > 0);
                    umma_commit(&sempty[i % NS]);
                }
                if (!ok) break;
                umma_commit(&bdqi);
#pragma unroll
                for (int i = 3 * NV; i < NT && ok; ++i) {
                    if (!(ok = tile(it, i))) break;
                    const uint32_t x = sx0 + i % NS * BOX;
                    inner(R3, sm + SM::V + SM::half(i) * BOX, x, 0, 1, id_si, i > 3 * NV);
                    if (SM::term(i) == 2) umma_commit(&sempty[i % NS]);
                    if (SM::term(i) == 2 || SM::half(i) < NV - 1) continue;
                    // all columns of a term are there, in slots one behind the other
                    if (SM::term(i) == 0 && !(ok = lane_wait(&scfree, ph, &s_wait))) break;
                    tc_fence_after();
                    const uint32_t y = x - (NV - 1) * BOX;
#pragma unroll
                    for (int z = 0; z < NK; ++z) {
                        const uint64_t ad = smem_desc_k_sw128(sm + SM::K + z * BOX);
                        const uint64_t bd = smem_desc_mn_sw128(y + z * 64 * 128, BOX);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_bf16(R0, ad + 2 * k, bd + (2048u >> 4) * k, id_kd,
                                      (SM::term(i) > 0 || z > 0 || k > 0) ? 1u : 0u);
                    }
#pragma unroll
                    for (int z = NV - 1; z >= 0; --z) umma_commit(&sempty[(i - z) % NS]);
                }
                if (!ok) break;
                umma_commit(&bdki);
                if (!lane_wait(&pready, ph, &s_wait)) break;
                tc_fence_after();
                const uint64_t gd = smem_desc_mn_sw128(sm + SM::G, BOX), qd = smem_desc_mn_sw128(sm + SM::Q, BOX),
                               kd = smem_desc_mn_sw128(sm + SM::K, BOX);
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                    umma_bf16_ta(R0, R1 + 16 * k, gd + (2048u >> 4) * k, id_kd, 1u);
                    umma_bf16_ta(R0, R1 + 16 * k + 8, gd + (2048u >> 4) * k, id_kd, 1u);
                }
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    const uint32_t x = t ? sx1 : sx0;   // the terms of Pd^T
                    const uint64_t pdt = smem_desc_mn_sw128(x, BOX);
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) {
                        const uint64_t pt = smem_desc_k_sw128(x + (k >> 2) * BOX) + 2 * (k & 3);
                        umma_bf16(R3, pt, qd + (2048u >> 4) * k, id_dk, 1u);
                        umma_bf16(R2, pdt + (2048u >> 4) * k, kd + (2048u >> 4) * k, id_dq, 1u);
                    }
                }
                umma_commit(&bout);
            }
            umma_commit(&fin);
        }
    } else if (warp == 18) {
        // dg of four rows a lane from the parts of r, c, u, w, in 64 bits: the
        // sums over the chunk cancel
        int it = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x, ++it) {
            const int h = item % a.H, c = item / a.H;
            const uint32_t ph = (uint32_t)it & 1u;
            if (!warp_wait(&dfull[it & 1], (uint32_t)(it >> 1) & 1u, &s_wait)) break;
            if (!warp_wait(&pready, ph, &s_wait)) break;
            if (a.dg) {
                const TcDecays &d = dec[it & 1];
                const LaChunk ck = la_chunk(g.ch, c);
                double x[4], w[4], xs = 0.0, ws = 0.0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = lane * 4 + i;
                    double v = 0.0, y = 0.0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k <= (t >> 5)) v += sums[k][t];          // r: parts of the keys' blocks up to its own
                        if (k >= (t >> 5)) v -= sums[4 + k][t];      // c: of the queries' blocks from its own
                        if (k < DK / 32) {
                            v += sums[8 + k][t];
                            y += sums[12 + k][t];
                        }
                    }
                    x[i] = v;
                    w[i] = y;
                    xs += v;
                    ws += y;
                }
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double xu = __shfl_down_sync(0xffffffffu, xs, o), wu = __shfl_up_sync(0xffffffffu, ws, o);
                    if (lane + o < 32) xs += xu;
                    if (lane >= o) ws += wu;
                }
                double dot = 0.0;
                if (lane < 16 && lane / 8 < g.tiles) dot = g.dot[((long long)c * a.H + h) * 16 + lane];
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                dot = __shfl_sync(0xffffffffu, dot, 0) * (double)d.tot;
                if (d.tot < 0.0f) dot = 0.0;
                // rows behind this lane's, rows before (no differences: a sum may be no number)
                double back = __shfl_down_sync(0xffffffffu, xs, 1), front = __shfl_up_sync(0xffffffffu, ws, 1);
                if (lane == 31) back = 0.0;
                if (lane == 0) front = 0.0;
                double out[4];
                float sum = 0.0f;
#pragma unroll
                for (int i = 3; i >= 0; --i) {
                    back += x[i];
                    out[i] = back;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = lane * 4 + i;
                    float v = (float)(out[i] + front + dot);
                    front += w[i];
                    if (t >= ck.len || d.first[t] == t) v = 0.0f;   // nothing passes a row that clears the state
                    if (t < ck.len && !a.per_head && SLSTM_IN((ck.row + t) * a.H + h, tc_rows(a) * a.H))
                        a.dg[(ck.row + t) * a.H + h] = v;
                    sum += v;
                }
                if (a.per_head) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane == 0 && SLSTM_IN((long long)c * a.H + h, (long long)g.ch.total * a.H))
                        g.dgc[(long long)c * a.H + h] = sum;
                }
            }
            warp_arrive(&sumfree);
            warp_arrive(&dempty[it & 1]);
        }
    } else {
        const int q = warp & 3, b = warp >> 2;
        const int r = q * 32 + lane;                  // row: key or query
        const uint32_t at = ((uint32_t)(q * 32) << 16) + 32 * b;
        int it = 0;
        bool ok = true;
        LaChunk ck;
        int h = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x, ++it) {
            const uint32_t ph = (uint32_t)it & 1u;
            h = item % a.H;
            ck = la_chunk(g.ch, item / a.H);
            if (packed && ck.len < TCC) {
                ok = warp_wait(&full1, ph, &s_wait) && warp_wait(&full2, ph, &s_wait);
                if (!ok) break;
                if (r >= ck.len)
                    for (int i = b; i < 2 * (NK + NV); i += 4) zero_row(smem + i * BOX, r);
                tma_store_fence();
                warp_arrive(&tready);
            }
            ok = warp_wait(&dfull[it & 1], (uint32_t)(it >> 1) & 1u, &s_wait) && warp_wait(&bsc, ph, &s_wait);
            if (ok && it > 0) ok = warp_wait(&sumfree, ph ^ 1u, &s_wait);
            if (!ok) break;
            tc_fence_after();
            const TcDecays &d = dec[it & 1];
            uint32_t pd[16], pl[16];   // the two terms of Pd
            if (b >= q) {
                float csum = 0.0f;
                // e^{c_i - c_j}: column i, this thread's j
                const float cj = b > q ? d.cq(b)[r] * a.scale : 0.0f, lj = d.loc[r], mj = d.rest[r];
                const uint32_t mask = d.mask[r];
#pragma unroll
                for (int z = 0; z < 32; z += 16) {
                    float s[16], t[16];
                    uint32_t p[16];   // 8 columns of the upper terms of P, 8 of the lower
                    tmem_ld16x2(R0 + at + z, R1 + at + z, s, t);
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        float w[4];
                        if (b > q) {
                            const float4 e = *reinterpret_cast<const float4 *>(&d.rq[32 * b + z + j]);
                            w[0] = cj * e.x;
                            w[1] = cj * e.y;
                            w[2] = cj * e.z;
                            w[3] = cj * e.w;
                        } else {
                            const float4 l = *reinterpret_cast<const float4 *>(&d.loc[32 * b + z + j]);
                            const float4 m = *reinterpret_cast<const float4 *>(&d.rest[32 * b + z + j]);
                            w[0] = ex2((l.x - lj) + (m.x - mj)) * a.scale;
                            w[1] = ex2((l.y - lj) + (m.y - mj)) * a.scale;
                            w[2] = ex2((l.z - lj) + (m.z - mj)) * a.scale;
                            w[3] = ex2((l.w - lj) + (m.w - mj)) * a.scale;
                        }
                        float pp[4], pq[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const bool on = b > q || ((mask >> (z + j + k)) & 1u);
                            pp[k] = on ? w[k] * s[j + k] : 0.0f;
                            pq[k] = on ? w[k] * t[j + k] : 0.0f;
                            // W, without the diagonal; s keeps it for the sums over this warp's keys
                            const bool off = b > q || (on && z + j + k != lane);
                            s[j + k] = off ? pp[k] * t[j + k] : 0.0f;
                            csum += s[j + k];
                        }
                        two_terms(pp[0], pp[1], p[j / 2], p[8 + j / 2]);
                        two_terms(pp[2], pp[3], p[j / 2 + 1], p[9 + j / 2]);
                        two_terms(pq[0], pq[1], pd[(z + j) / 2], pl[(z + j) / 2]);
                        two_terms(pq[2], pq[3], pd[(z + j) / 2 + 1], pl[(z + j) / 2 + 1]);
                    }
                    tmem_st16(R1 + at + z, p);
                    // 16 columns summed over the lanes: each step halves the columns a lane holds
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) {
                        const bool up = lane & o;
#pragma unroll
                        for (int k = 0; k < o; ++k) {
                            const float send = up ? s[k] : s[k + o], keep = up ? s[k + o] : s[k];
                            s[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                        }
                    }
                    s[0] += __shfl_xor_sync(0xffffffffu, s[0], 16);
                    if (lane < 16) sums[q][32 * b + z + lane] = s[0];
                }
                sums[4 + b][r] = csum;
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) pd[j] = pl[j] = 0u;
                tmem_st16(R1 + at, pd);
                tmem_st16(R1 + at + 16, pd);
            }
            tc_fence_before();
            warp_arrive(&scfree);
            // the states' part of dq and dk: scaled in place, dotted with q and k
            ok = warp_wait(&bdqi, ph, &s_wait);
            if (!ok) break;
            tc_fence_after();
            if (b < DK / 32) {
                float v[32];
                tmem_ld32(R2 + at, v);
                const float f = a.scale * d.row[r];
                const bool open = d.first[r] < 0;   // the state reaches the row
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = open ? v[j] * f : 0.0f;
                tmem_st32(R2 + at, v);
                sums[8 + b][r] = dot_row(smem + SM::Q, r, b, v);
            }
            ok = warp_wait(&bdki, ph, &s_wait);
            if (!ok) break;
            tc_fence_after();
            const float colr = d.col[r];
            const bool out = d.first[TCC - 1] <= r;   // the row reaches the state
            if (b < DK / 32) {
                float v[32];
                tmem_ld32(R3 + at, v);
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = out ? v[j] * colr : 0.0f;
                tmem_st32(R3 + at, v);
                sums[12 + b][r] = dot_row(smem + SM::K, r, b, v);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t o = (b >> 1) * BOX + swz(r, 4 * (b & 1) + k);
                *reinterpret_cast<uint4 *>(x0 + o) = make_uint4(pd[4 * k], pd[4 * k + 1], pd[4 * k + 2], pd[4 * k + 3]);
                *reinterpret_cast<uint4 *>(x1 + o) = make_uint4(pl[4 * k], pl[4 * k + 1], pl[4 * k + 2], pl[4 * k + 3]);
            }
            // the states' part of dv
            if (b < DV / 32) {
                float v[32];
                tmem_ld32(R0 + at, v);
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = out ? v[j] * colr : 0.0f;
                tmem_st32(R0 + at, v);
            }
            tmem_wait_st();
            tma_store_fence();
            tc_fence_before();
            warp_arrive(&pready);
            warp_arrive(&dempty[it & 1]);
            ok = warp_wait(&bout, ph, &s_wait);
            if (!ok) break;
            tc_fence_after();
            const long long row = ck.row + q * 32;
            const int rows = ck.len - q * 32;
            // (every product has read the two buffers)
            uint8_t *stage = x0 + warp * 4096;
            const long long ldv = (long long)a.H * a.dv;
            if (b < DV / 32) {
                float v[32];
                tmem_ld32(R0 + at, v);
                __nv_bfloat16 *dv = static_cast<__nv_bfloat16 *>(a.dv_);
                put_rows(dv + row * ldv + (long long)h * a.dv + 32 * b, ldv, v, a.dv - 32 * b, rows, stage, lane, dv,
                         tc_rows(a) * ldv);
            }
            if (b < DK / 32) {
                const int cols = a.dk - 32 * b;
#pragma unroll 1
                for (int z = 0; z < 2; ++z) {
                    float v[32];
                    tmem_ld32((z ? R3 : R2) + at, v);
                    if (g.part_q) {
                        float *dst = z ? g.part_k : g.part_q;
                        put_rows(dst + (row * a.H + h) * a.dk + 32 * b, (long long)a.H * a.dk, v, cols, rows, stage,
                                 lane, dst, tc_rows(a) * a.H * a.dk);
                    } else {
                        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(z ? a.dk_ : a.dq);
                        put_rows(dst + (row * a.Hqk + h) * a.dk + 32 * b, (long long)a.Hqk * a.dk, v, cols, rows,
                                 stage, lane, dst, tc_rows(a) * a.Hqk * a.dk);
                    }
                }
            }
            tma_store_fence();   // these writes before the next loads into the buffers
            warp_arrive(&xfree);
            tc_fence_before();
            warp_arrive(&tfree);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        if (s_wait.gave_up && s_items > 0) {
            const int it = s_items - 1;
            const uint32_t ph = (uint32_t)it & 1u;
            (void)mbar_wait(&dfull[it & 1], (uint32_t)(it >> 1) & 1u, TC_WAIT_NS);
            (void)mbar_wait(&full1, ph, TC_WAIT_NS);
            (void)mbar_wait(&full2, ph, TC_WAIT_NS);
            for (int i = max(0, s_tiles - NS); i < s_tiles; ++i)
                (void)mbar_wait(&sfull[i % NS], phase(it, i) & 1u, TC_WAIT_NS);
        }
        (void)mbar_wait(&fin, 0u, TC_WAIT_NS);
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_free<512>(tmem);
    }
    if (!s_wait.gave_up) return;
    // which of its parts a block has finished is not known: all its items
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int h = item % a.H, c = item / a.H;
        const LaChunk ck = la_chunk(g.ch, c);
        const float nan = __int_as_float(0x7fc00000);
        for (int r = warp; r < ck.len; r += BACK_THREADS / 32) {
            const long long row = ck.row + r;
            for (int j = lane; j < a.dv; j += 32)
                static_cast<__nv_bfloat16 *>(a.dv_)[(row * a.H + h) * a.dv + j] = bf16_nan();
            for (int j = lane; j < a.dk; j += 32)
                if (g.part_q) {
                    g.part_q[(row * a.H + h) * a.dk + j] = nan;
                    g.part_k[(row * a.H + h) * a.dk + j] = nan;
                } else {
                    static_cast<__nv_bfloat16 *>(a.dq)[(row * a.Hqk + h) * a.dk + j] = bf16_nan();
                    static_cast<__nv_bfloat16 *>(a.dk_)[(row * a.Hqk + h) * a.dk + j] = bf16_nan();
                }
            if (a.dg && !a.per_head && lane == 0) a.dg[row * a.H + h] = nan;
        }
        if (a.dg && a.per_head && threadIdx.x == 0) g.dgc[(long long)c * a.H + h] = nan;
    }
}

// Packed sequences without a row: their final state is their first.
__global__ void __launch_bounds__(256) la_empty_kernel(LaChunks ch, long long HE, const float *first, float *last)
{
    const int seq = blockIdx.x;
    if (ch.coff[seq + 1] != ch.coff[seq]) return;
    for (long long i = (long long)blockIdx.y * 256 + threadIdx.x; i < HE; i += (long long)gridDim.y * 256)
        if (SLSTM_IN(seq * HE + i, ch.n_seq * HE)) last[seq * HE + i] = first ? first[seq * HE + i] : 0.0f;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// (features, heads, rows of a sequence, sequences) of a token tensor with rows
// ld elements apart, in boxes of 64 features of one head and 128 rows.
bool token_map(CUtensorMap *m, const void *p, int d, int heads, long long ld, const LaArgs &a)
{
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const uint64_t T = (uint64_t)a.T, B = a.cu ? 1u : (uint64_t)a.B;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, T, B};
    cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * T};
    cuuint32_t box[4] = {64u, 1u, (cuuint32_t)TCC, 1u};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Chunks of a segment: whole sequences where their blocks fill the GPU, else
// as many equal segments as make the fewest idle SMs of whole waves (one block
// an SM), of four chunks at least, since a segment's first state costs a pass
// over its k and v.  Measured, forward and gradients, in segments and whole:
// 1 x 65536, 16 heads of 64 x 128: 429, 1091 and 1220, 1787 us; 1 x 4096, 8 heads
// of 128: 44, 105 and 101, 161; 4 x 8192: 159, 417 and 184, 411; but 8 x 1024, 4
// heads of 128 (64 blocks of 8 chunks): 47, 106 and 38, 84; 9 x 2048: 61, 164 and
// 56, 135.
int seg_chunks(const LaArgs &a, int per_item)
{
    const int nc = (a.T - 1) / TCC + 1;
    if (a.cu) {
        // packed: the lengths are not known here; a segment is as long as an even
        // share of all chunks, so that the longest sequence takes no longer than
        // the rest of the work, and one that is no longer is one segment
        const long long share = ((long long)nc * per_item + 147) / 148;
        return (int)min((long long)nc, max(share, 4LL));
    }
    const long long base = (long long)a.B * per_item;
    if (base >= 120 || nc < 8) return nc;
    int best = nc;
    double best_t = 1e300;
    for (int n = 1; n <= nc / 4 && n <= 64; ++n) {
        const int len = (nc + n - 1) / n;
        const long long waves = (base * n + 147) / 148;
        // the pass for the first states costs about half a segment and, with the scan
        // of them, two launches, about four chunks; a block's start costs about three
        // chunks, and a segment's state in the scan something too
        const double t = (double)waves * (len + 3) * (n > 1 ? 1.5 : 1.0) + (n > 1 ? 4.0 : 0.0) + 0.1 * n;
        if (t < best_t) {
            best_t = t;
            best = len;
        }
    }
    return best;
}

struct FwdWs {
    char *table, *seg_table, *order;
    TcDecays *dec;
    float *states, *tot;
    size_t bytes;
};

FwdWs fwd_layout(const LaArgs &a, int L, void *ws)
{
    FwdWs w{};
    char *p = static_cast<char *>(ws);
    auto take = [&](size_t n) {
        char *r = p;
        p += up256(n);
        return r;
    };
    w.table = take(la_table_bytes(a));
    w.seg_table = take(la_table_bytes(a));
    w.order = take(la_order_bytes(a, L * TCC));
    w.dec = reinterpret_cast<TcDecays *>(take(sizeof(TcDecays) * la_chunk_bound(a, TCC) * a.H));
    if (L < (a.T - 1) / TCC + 1) {
        const size_t items = (size_t)la_chunk_bound(a, L * TCC);
        w.states = reinterpret_cast<float *>(take(4 * items * a.H * a.dk * a.dv));
        w.tot = reinterpret_cast<float *>(take(4 * items * a.H));
    }
    w.bytes = (size_t)(p - static_cast<char *>(ws));
    return w;
}

cudaError_t launch_decays(const LaArgs &a, const LaChunks &ch, TcDecays *dec, cudaStream_t st)
{
    la_decay_kernel<<<(unsigned)(((long long)ch.total * a.H + 7) / 8), 256, 0, st>>>(a, ch, dec);
    return cudaGetLastError();
}

// One direction (g1 null) or both; st: where the chunks' states go, if they do.
template <int DK>
cudaError_t launch_state(const CUtensorMap *xy, const CUtensorMap *st_map, const TcArgs &g0, const TcArgs *g1,
                         cudaStream_t st)
{
    const int bytes = StateShared<DK>::BYTES;
    cudaError_t e = la_allow_shared<la_state_kernel<DK>>(bytes);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)g0.seg.total * g0.a.H * g0.tiles, g1 ? 2 : 1);
    la_state_kernel<DK><<<grid, STATE_THREADS, bytes, st>>>(xy[0], xy[1], xy[g1 ? 2 : 0], xy[g1 ? 3 : 1],
                                                          *st_map, g0, g1 ? *g1 : g0);
    return cudaGetLastError();
}

cudaError_t launch_states(const CUtensorMap *xy, const CUtensorMap *st_map, const TcArgs &g0, const TcArgs *g1,
                          cudaStream_t st)
{
    return g0.a.dk <= 64 ? launch_state<64>(xy, st_map, g0, g1, st) : launch_state<128>(xy, st_map, g0, g1, st);
}

template <int DK>
cudaError_t launch_forward(const CUtensorMap *m, const TcArgs &g, cudaStream_t st)
{
    const int bytes = FwdShared<DK>::BYTES;
    cudaError_t e = la_allow_shared<la_forward_kernel<DK>>(bytes);
    if (e != cudaSuccess) return e;
    la_forward_kernel<DK>
        <<<(unsigned)g.seg.total * g.a.H * g.tiles, FWD_THREADS, bytes, st>>>(m[0], m[1], m[2], g);
    return cudaGetLastError();
}

// The states of the chunks: (d_v, d_k, term * n + chunk * H + h), boxes of 64
// columns and DK rows.
bool state_map(CUtensorMap *m, const void *p, const LaArgs &a, long long n, int DK)
{
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)a.dv, (cuuint64_t)a.dk, (cuuint64_t)n * 3};
    cuuint64_t strides[2] = {(cuuint64_t)a.dv * 2, (cuuint64_t)a.dv * a.dk * 2};
    cuuint32_t box[3] = {64u, (cuuint32_t)DK, 1u};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct BackWs {
    char *table, *seg_table, *order;
    TcDecays *dec;
    float *seg[2], *tot[2];            // a segment's first states, forward and from the end
    __nv_bfloat16 *st[2];              // the chunks' states, three terms
    float *dot, *dgc, *pq, *pk;
    size_t bytes;
};

BackWs back_layout(const LaArgs &a, int L, void *ws)
{
    BackWs w{};
    char *p = static_cast<char *>(ws);
    auto take = [&](size_t n) {
        char *r = p;
        p += up256(n);
        return r;
    };
    const size_t E = (size_t)a.dk * a.dv, n = (size_t)la_chunk_bound(a, TCC) * a.H;
    const size_t rows = a.cu ? (size_t)a.T : (size_t)a.B * a.T;
    w.table = take(la_table_bytes(a));
    w.seg_table = take(la_table_bytes(a));
    w.order = take(la_order_bytes(a, L * TCC));
    w.dec = reinterpret_cast<TcDecays *>(take(sizeof(TcDecays) * n));
    for (int i = 0; i < 2; ++i) {
        if (L < (a.T - 1) / TCC + 1) {
            const size_t items = (size_t)la_chunk_bound(a, L * TCC) * a.H;
            w.seg[i] = reinterpret_cast<float *>(take(4 * items * E));
            w.tot[i] = reinterpret_cast<float *>(take(4 * items));
        }
        w.st[i] = reinterpret_cast<__nv_bfloat16 *>(take(3 * 2 * n * E));
    }
    w.dot = reinterpret_cast<float *>(take(4 * n * 16));
    w.dgc = reinterpret_cast<float *>(take(4 * n));
    if (a.H != a.Hqk) {
        w.pq = reinterpret_cast<float *>(take(4 * rows * a.H * a.dk));
        w.pk = reinterpret_cast<float *>(take(4 * rows * a.H * a.dk));
    }
    w.bytes = (size_t)(p - static_cast<char *>(ws));
    return w;
}

template <int DK, int DV>
cudaError_t launch_back(const CUtensorMap *m, const BackArgs &g, int items, cudaStream_t st)
{
    const int bytes = BackShared<DK, DV>::BYTES;
    cudaError_t e = la_allow_shared<la_backward_kernel<DK, DV>>(bytes);
    if (e != cudaSuccess) return e;
    la_backward_kernel<DK, DV><<<min(items, 148), BACK_THREADS, bytes, st>>>(m[0], m[1], m[2], m[3], m[4], m[5], g);
    return cudaGetLastError();
}

}  // namespace

bool la_tc_takes(const LaArgs &a)
{
    return a.dtype == SLSTM_BF16 && a.dk <= 128 && a.dv <= 128 && a.dk % 8 == 0 && a.dv % 8 == 0 && a.ldq % 8 == 0 &&
           a.ldk % 8 == 0 && a.ldv % 8 == 0;
}

int la_tc_tries(int wait_limit_us)
{
    const int us = wait_limit_us ? wait_limit_us : 2000000;
    return us / TRY_US + 1;
}

size_t la_tc_forward_workspace(const LaArgs &a)
{
    return fwd_layout(a, seg_chunks(a, a.H * ((a.dv + 63) / 64)), reinterpret_cast<void *>((uintptr_t)256)).bytes;
}

cudaError_t la_tc_forward(const LaArgs &a, void *ws, cudaStream_t st)
{
    TcArgs g{};
    g.a = a;
    g.tiles = (a.dv + 63) / 64;
    const int L = seg_chunks(a, a.H * g.tiles);
    const FwdWs w = fwd_layout(a, L, ws);
    cudaError_t e = la_chunks(a, TCC, w.table, &g.ch, st, L * TCC, w.seg_table, &g.seg,
                              w.order);
    if (e == cudaSuccess) e = launch_decays(a, g.ch, w.dec, st);
    if (e != cudaSuccess) return e;
    g.dec = w.dec;
    CUtensorMap m[4];
    if (!token_map(&m[0], a.q, a.dk, a.Hqk, a.ldq, a) || !token_map(&m[1], a.k, a.dk, a.Hqk, a.ldk, a) ||
        !token_map(&m[2], a.v, a.dv, a.H, a.ldv, a))
        return cudaErrorInvalidValue;
    g.first = a.s0;
    g.last = a.sT;
    if (w.states) {
        TcArgs s = g;
        s.first = nullptr;
        s.fin = w.states;
        s.fin_tot = w.tot;
        const CUtensorMap xy[4] = {m[1], m[2], m[1], m[2]};
        e = launch_states(xy, xy, s, nullptr, st);   // (it stores no chunk's state)
        if (e == cudaSuccess) e = la_scan(g.seg, a.H, a.dk * a.dv, false, w.states, w.tot, a.s0, a.sT, st, 1);
        if (e != cudaSuccess) return e;
        g.init = w.states;
    } else if (a.cu && a.sT) {
        const long long HE = (long long)a.H * a.dk * a.dv;
        la_empty_kernel<<<dim3(a.B, (unsigned)min((HE + 1023) / 1024, 64LL)), 256, 0, st>>>(g.seg, HE, a.s0, a.sT);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return a.dk <= 64 ? launch_forward<64>(m, g, st) : launch_forward<128>(m, g, st);
}

size_t la_tc_backward_workspace(const LaArgs &a)
{
    return back_layout(a, seg_chunks(a, a.H * ((a.dv + 63) / 64)), reinterpret_cast<void *>((uintptr_t)256)).bytes;
}

cudaError_t la_tc_backward(const LaArgs &a, void *ws, cudaStream_t st)
{
    TcArgs g{};
    g.a = a;
    g.tiles = (a.dv + 63) / 64;
    const int L = seg_chunks(a, a.H * g.tiles);
    const BackWs w = back_layout(a, L, ws);
    const int DK = a.dk <= 64 ? 64 : 128, DV = a.dv <= 64 ? 64 : 128;
    cudaError_t e = la_chunks(a, TCC, w.table, &g.ch, st, L * TCC, w.seg_table, &g.seg,
                              w.order);
    if (e == cudaSuccess) e = launch_decays(a, g.ch, w.dec, st);
    if (e != cudaSuccess) return e;
    g.dec = w.dec;
    const long long n = (long long)g.ch.total * a.H;
    CUtensorMap m[6];
    bool ok = token_map(&m[0], a.q, a.dk, a.Hqk, a.ldq, a) && token_map(&m[1], a.k, a.dk, a.Hqk, a.ldk, a) &&
              token_map(&m[2], a.v, a.dv, a.H, a.ldv, a) &&
              token_map(&m[3], a.dO, a.dv, a.H, (long long)a.H * a.dv, a);
    for (int i = 0; i < 2; ++i) ok = ok && state_map(&m[4 + i], w.st[i], a, n, DK);
    if (!ok) return cudaErrorInvalidValue;
    const CUtensorMap xy[4] = {m[1], m[2], m[0], m[3]};
    TcArgs dir[2] = {g, g};
    const float *first[2] = {a.s0, a.dsT};
    float *last[2] = {nullptr, a.ds0};
    dir[1].back = true;
    if (w.seg[0]) {
        for (int i = 0; i < 2; ++i) {
            dir[i].fin = w.seg[i];
            dir[i].fin_tot = w.tot[i];
        }
        e = launch_states(xy, xy, dir[0], &dir[1], st);
        for (int i = 0; i < 2 && e == cudaSuccess; ++i)
            e = la_scan(g.seg, a.H, a.dk * a.dv, i == 1, w.seg[i], w.tot[i], first[i], last[i], st, 1);
        if (e != cudaSuccess) return e;
    } else if (a.cu && a.ds0) {
        const long long HE = (long long)a.H * a.dk * a.dv;
        la_empty_kernel<<<dim3(a.B, (unsigned)min((HE + 1023) / 1024, 64LL)), 256, 0, st>>>(g.seg, HE, a.dsT, a.ds0);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    // the chunks' states: forward, then from the end (which meets the forward ones for dg)
    for (int i = 0; i < 2; ++i) {
        TcArgs &s = dir[i];
        s.fin = nullptr;
        s.fin_tot = nullptr;
        s.init = w.seg[i];
        s.first = first[i];
        s.last = last[i];
        s.st = w.st[i];
        if (i == 1 && a.dg) {
            s.pst = w.st[0];
            s.dot = w.dot;
        }
        e = launch_states(xy + 2 * i, &m[4 + i], s, nullptr, st);
        if (e != cudaSuccess) return e;
    }
    BackArgs b{};
    b.a = a;
    b.ch = g.ch;
    b.dec = w.dec;
    b.total = (int)n;
    b.part_q = w.pq;
    b.part_k = w.pk;
    b.dgc = w.dgc;
    b.dot = w.dot;
    b.tiles = g.tiles;
    if (DK == 64) e = DV == 64 ? launch_back<64, 64>(m, b, (int)n, st) : launch_back<64, 128>(m, b, (int)n, st);
    else e = DV == 64 ? launch_back<128, 64>(m, b, (int)n, st) : launch_back<128, 128>(m, b, (int)n, st);
    if (e == cudaSuccess && w.pq) e = la_share_sum(w.pq, w.pk, g.ch, a, st);
    if (e == cudaSuccess && a.dg && a.per_head) e = la_head_sum(w.dgc, a.dg, g.ch, a.H, st);
    return e;
}

}  // namespace slstm

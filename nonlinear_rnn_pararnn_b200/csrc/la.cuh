// Device helpers of the linear attention: where a chunk lies, and the decays
// inside it.
#pragma once

#include "common.cuh"
#include "la.h"

namespace slstm {

struct LaChunk {
    int seq;          // sequence
    int n;            // index of the chunk in its sequence
    long long row;    // first row
    int len;          // rows, 1..C; 0: the sequences have fewer chunks than the grid
    int count;        // chunks of the sequence
};

// Chunk c of the sequences in order.
SLSTM_DEVINL LaChunk la_chunk(const LaChunks &t, int c)
{
    LaChunk r;
    if (t.pos == nullptr) {
        r.seq = c / t.nc;
        r.n = c - r.seq * t.nc;
        r.count = t.nc;
        r.row = (long long)r.seq * t.T + (long long)r.n * t.C;
        r.len = min(t.C, t.T - r.n * t.C);
        return r;
    }
    if (c >= t.coff[t.n_seq]) return LaChunk{0, 0, 0, 0, 0};
    int lo = 0, hi = t.n_seq;   // the last sequence with coff <= c
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.coff[mid] <= c) lo = mid;
        else hi = mid;
    }
    r.seq = lo;
    r.n = c - t.coff[lo];
    r.count = t.coff[lo + 1] - t.coff[lo];
    const int p = t.pos[lo], e = t.pos[lo + 1];
    r.row = (long long)p + (long long)r.n * t.C;
    r.len = min(t.C, e - (int)r.row);
    return r;
}

// A log decay in base 2.  Below 2^-126 (-inf among them) the factor is zero in
// fp32: such a step clears the state and takes no part in the sums, so that
// neither -inf nor a large finite value spoils the differences of the others.
SLSTM_DEVINL bool la_clears(float g) { return g < -87.3f; }

// What a state becomes over a chunk: tot s + delta, or delta alone where the
// chunk clears it (tot < 0), since zero times what is cleared need not be zero.
SLSTM_DEVINL float la_carry(float tot, float s, float delta) { return tot < 0.0f ? delta : fmaf(tot, s, delta); }

// The decays inside a chunk of C = 32 P rows, by one warp; lane l holds rows
// P l .. P l + P - 1.  With c_i the sum of log2 decays up to and with row i:
//   cum[i]    c_i in 64 bits (differences of far rows stay exact)
//   first[i]  the last row <= i that clears the state, or -1
//   row[i]    e^{c_i}: from the state that enters to row i (0 behind a clear)
//   col[j]    e^{c_C - c_j}: from row j to the state that leaves (0 before one)
//   *tot      e^{c_C}, or -1 where a row clears (la_carry)
// Rows behind `len` decay nothing.
template <int P>
SLSTM_DEVINL void la_decays(const float *g, long long g0, int gstride, int len, int lane, double *cum, int *first,
                            float *row, float *col, float *tot)
{
    double s[P];
    int f[P];
    double run = 0.0;
    int last = -1;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int t = lane * P + i;
        const float gv = t < len ? g[g0 + (long long)t * gstride] : 0.0f;
        if (la_clears(gv)) last = t;
        else run += (double)gv * 1.4426950408889634074;
        s[i] = run;
        f[i] = last;
    }
    double pre = run;
    int pf = last;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double u = __shfl_up_sync(0xffffffffu, pre, o);
        const int w = __shfl_up_sync(0xffffffffu, pf, o);
        if (lane >= o) {
            pre += u;
            pf = max(pf, w);
        }
    }
    const double all = __shfl_sync(0xffffffffu, pre, 31);
    const int allf = __shfl_sync(0xffffffffu, pf, 31);
    double before = __shfl_up_sync(0xffffffffu, pre, 1);
    int bf = __shfl_up_sync(0xffffffffu, pf, 1);
    if (lane == 0) {
        before = 0.0;
        bf = -1;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int t = lane * P + i;
        const double c = before + s[i];
        const int fi = max(bf, f[i]);
        cum[t] = c;
        first[t] = fi;
        row[t] = fi >= 0 ? 0.0f : exp2f((float)c);
        col[t] = allf > t ? 0.0f : exp2f((float)(all - c));
    }
    if (lane == 0) *tot = allf >= 0 ? -1.0f : exp2f((float)all);
}

}  // namespace slstm

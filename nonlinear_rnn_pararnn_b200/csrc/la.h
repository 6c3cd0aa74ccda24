// Linear attention with a decay for each head: the arguments shared by its
// launchers (linear_attention.cu: any sizes and types on the CUDA cores;
// linear_attention_tc.cu: bf16 on the tensor cores), behind the C ABI in
// slstm_api.cu.
#pragma once

#include <atomic>

#include <cuda_runtime.h>
#include <stddef.h>

#include "../../include/slstm.h"

namespace slstm {

// One call.  Rows are tokens: B sequences of T rows each, or (cu != null)
// n_seq packed sequences over T rows.
struct LaArgs {
    int B, T;                 // dense: B x T rows; packed: B = n_seq, T = total rows
    int H, Hqk, dk, dv;
    long long ldq, ldk, ldv;  // elements between rows
    int dtype;
    int per_head;             // g is (H,), not (rows, H)
    float scale;
    const int *cu;            // packed offsets (n_seq + 1), or null
    const void *q, *k, *v;
    const float *g, *s0;
    void *o;
    float *sT;
    // backward only
    const void *dO;
    const float *dsT;
    void *dq, *dk_, *dv_;
    float *dg, *ds0;
    // tensor cores: what a wait may try, and the self-test of its running out
    int tries, debug_fault;
};

size_t la_simt_workspace(const LaArgs &a, bool backward);
cudaError_t la_simt_forward(const LaArgs &a, void *ws, cudaStream_t st);
cudaError_t la_simt_backward(const LaArgs &a, void *ws, cudaStream_t st);
cudaError_t la_step_launch(const LaArgs &a, float *s_next, cudaStream_t st);

// The chunks of C rows that the sequences are cut into, each sequence from its
// own first row.  Dense sequences need no table; of packed ones, pos[k] is the
// first row of sequence k (the offsets clamped into the rows and made
// nondecreasing, so that malformed ones lead nowhere out of range) and coff[k]
// the number of chunks before it.
struct LaChunks {
    int n_seq, T, C;          // T: rows of a dense sequence
    int nc;                   // dense: chunks of a sequence
    int total;                // an upper bound of the chunks (dense: the number)
    const int *pos, *coff;    // packed: [n_seq + 1] each; else null
    const int *order;         // packed, where asked for: the chunks, long ones first; else null
};
size_t la_table_bytes(const LaArgs &a);
int la_chunk_bound(const LaArgs &a, int C);
size_t la_order_bytes(const LaArgs &a, int C);   // of the order of chunks of C rows
// Fill the table (packed) at `mem` on `st`; with out2, a second one for chunks of
// C2 rows at mem2 in the same launch, its order at `order` (la_order_bytes).
cudaError_t la_chunks(const LaArgs &a, int C, void *mem, LaChunks *out, cudaStream_t st, int C2 = 0,
                      void *mem2 = nullptr, LaChunks *out2 = nullptr, void *order = nullptr);

// The states over the chunks (or segments) of each sequence, elementwise: the
// E-element deltas in buf[chunk][h], with the decays tot[chunk][h] (negative: the
// state is cleared), give way to the state that enters each (back: the gradient of the one that leaves it),
// starting from first[sequence][h] (null: zero); the last one to `last` (or
// null).  Sequences of `skip` chunks are left alone.
cudaError_t la_scan(const LaChunks &ch, int H, int E, bool back, float *buf, const float *tot, const float *first,
                    float *last, cudaStream_t st, int skip = -1);

// bf16 on the tensor cores.
bool la_tc_takes(const LaArgs &a);
int la_tc_tries(int wait_limit_us);
size_t la_tc_forward_workspace(const LaArgs &a);
cudaError_t la_tc_forward(const LaArgs &a, void *ws, cudaStream_t st);
size_t la_tc_backward_workspace(const LaArgs &a);
cudaError_t la_tc_backward(const LaArgs &a, void *ws, cudaStream_t st);

// Lets kernel F have `bytes` of dynamic shared memory; asks the runtime once for
// each device.
template <auto *F>
cudaError_t la_allow_shared(int bytes)
{
    static std::atomic<unsigned long long> asked{0ull};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (asked.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(F, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) asked.fetch_or(bit, std::memory_order_release);
    return e;
}

// Sums of the fp32 per-head partial gradients over the heads that share a query
// and key head, into a.dq and a.dk_: dq[row][hq][d] = sum over r of
// pq[row][hq * rep + r][d].
cudaError_t la_share_sum(const float *pq, const float *pk, const LaChunks &ch, const LaArgs &a, cudaStream_t st);
// dg[h] = sum of part[c][h] over the chunks in order.
cudaError_t la_head_sum(const float *part, float *dg, const LaChunks &ch, int H, cudaStream_t st);

}  // namespace slstm

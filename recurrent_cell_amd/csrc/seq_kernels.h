// Arguments and launchers of the sequence-block kernels (layer norm, dropout,
// causal convolution, selective scan).  Element pointers are void*: the
// launchers pick the instantiation by `type` (seq_dtype).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace seq {

constexpr int kMaxSumSegs = 5;

// out[n] = sum over r < R of in[r * stride + n], n < N; fp64 sums in an order
// fixed by R, rounded once to the output's type.
struct SumSeg {
    const float* in;
    void* out;
    int64_t R, N, stride;
    int type;        // of out
    int64_t block0;  // first workgroup (filled by the launcher)
};
struct SumArgs {
    SumSeg seg[kMaxSumSegs];
    int nseg;
};
int64_t sum_rows_blocks(int64_t R, int64_t N);   // of 256 lanes, for one segment; a launch has fewer than 2^24
hipError_t launch_sum_rows(SumArgs a, hipStream_t s);

struct LnArgs {
    const void* x;
    const void* dy;        // backward
    void* out;             // y, or dx
    int64_t ldx, lddy, ldo;
    const float* w;        // or NULL: ones
    const float* b;        // or NULL: zeros
    float* mean;
    float* rstd;
    float* part;           // backward: [parts][2][C] (NULL: no parameter gradients)
    int64_t rows;
    int C, type, parts;
    float eps;
};
int ln_bwd_parts(int64_t rows, int C, int type);
hipError_t launch_ln_fwd(const LnArgs& a, hipStream_t s);
hipError_t launch_ln_bwd(const LnArgs& a, hipStream_t s);

struct DropArgs {
    const void* x;
    const void* r;         // residual or NULL
    void* y;
    int64_t ldx, ldr, ldy, rows, C;
    uint64_t seed, offset;
    uint32_t threshold;    // an element is kept when its word is >= this
    float scale;
    int type;
};
hipError_t launch_dropout(const DropArgs& a, hipStream_t s);

// How rows fall into sequences (SeqMap in seq_device.h, without the piece).
struct Rows {
    const int* cu;
    int64_t total, L;
    int n;
};

struct ConvArgs {
    const void* x;
    const void* dy;         // backward
    void* out;              // y, or dx
    int64_t ldx, lddy, ldo;
    const float* w;         // [D, K]
    const float* b;         // [D] or NULL
    const void* state_in;   // [n, K - 1, D] or NULL: zeros
    void* state_out;        // the same or NULL
    float* part;            // backward: [parts][D K + D]
    Rows rows;
    int D, K, type, silu;
    unsigned blocks;        // of channels (filled by the launcher)
};
int64_t conv_bwd_parts(const Rows& r, int D);
bool conv_fits(const Rows& r, int D);   // every launch has fewer than 2^32 lanes, what a grid's first axis can hold
hipError_t launch_conv_fwd(ConvArgs a, hipStream_t s);
hipError_t launch_conv_bwd(ConvArgs a, hipStream_t s);

struct ConvStepArgs {
    const void* x;
    void* state;            // [S, K - 1, D], shifted in place
    void* y;
    int64_t ldx, ldy;
    const float* w;
    const float* b;
    int64_t S;
    int D, K, type, silu;
};
hipError_t launch_conv_step(const ConvStepArgs& a, hipStream_t s);

// Rows between the states a training pass keeps: the piece of the backward
// kernel, 16 lanes of 4 rows.
constexpr int kScanKeep = 64;

struct ScanArgs {
    const void *u, *dt, *z, *B, *C, *dy;
    int64_t ldu, lddt, ldz, ldb, ldc, lddy;
    void *y, *du, *ddt, *dz;
    int64_t ldy, lddu, ldddt, lddz;
    const float *A, *skip, *dt_bias, *h0, *dh_last;
    float *h_last, *dh0;
    float* hist;     // [slots of kScanKeep rows][N][D]: the state before each
    float* st;       // [slots][N][D]: a piece's own end state, then (after the join) the state that enters it
    float* sd;       // [slots][D]: the piece's sum of delta
    float* part_bc;  // backward: [channel blocks][2][rows][G][N]
    float* part_p;   // backward: [slots][(N + 2)][D]: dA, dskip, ddt_bias
    Rows rows;
    int piece;       // rows per piece, a multiple of kScanKeep (in a backward pass those)
    int chans;       // backward: channels per workgroup (a multiple of 16)
    int join;        // st holds the pieces' own states: the main pass joins them itself
    int D, N, G, type, softplus;
};
int64_t scan_slots(const Rows& r, int piece);
bool scan_fits(const Rows& r, int D, int G);   // as conv_fits
bool scan_in_rows(const Rows& r, int D, int G);
bool scan_joins(const Rows& r, int D, int G);   // ScanArgs::join; without it launch_scan_join comes first
int scan_piece(const Rows& r, int D, int G);
int scan_bwd_chans(const Rows& r, int D, int G);
inline int scan_bwd_blocks(int D, int G, int chans) { return (D / G + chans - 1) / chans; }
bool scan_one_piece(const Rows& r, int piece);   // no sequence can have a second piece
hipError_t launch_scan_state(const ScanArgs& a, bool reverse, hipStream_t s);
hipError_t launch_scan_join(const ScanArgs& a, bool reverse, hipStream_t s);
hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t s);

struct ScanStepArgs {
    const void *u, *dt, *z, *B, *C;
    int64_t ldu, lddt, ldz, ldb, ldc, ldy;
    void* y;
    const float *A, *skip, *dt_bias;
    float* h;   // [S, N, D], updated in place
    int64_t S;
    int D, N, G, type, softplus;
};
hipError_t launch_scan_step(const ScanStepArgs& a, hipStream_t s);

}  // namespace seq

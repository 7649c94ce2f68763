// Selective state space scan, channels innermost.  Per sequence, channel d and
// state n (g the channel's group):
//   x = dt + dt_bias,  delta = softplus(x)            (or x)
//   h_t[n] = exp(delta A[n]) h_{t-1}[n] + delta u B_t[g, n]
//   y_t = (sum_n C_t[g, n] h_t[n] + skip u) * z sigmoid(z)
// The recurrence is linear in h, so a sequence is cut into pieces that run in
// parallel: a first pass forms each piece's end state from zero, a join
// carries the states over the pieces (a piece's decay is exp(A sum delta)),
// and the main pass starts every piece from the state that enters it.
// Everything is fp32; the states never leave fp32.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../../include/seq.h"
#include "seq_device.h"
#include "seq_kernels.h"

namespace seq {

namespace {

constexpr int kBatch = 8;    // rows whose loads are in flight together

__device__ __forceinline__ float delta_of(float dt, float bias, int softplus)
{
    const float x = dt + bias;
    return softplus ? softplus_e(x, exp_neg_abs(x)) : x;
}

// A log2(e), an infinite rate of decay held at the largest finite one: rows past
// the end of a piece have delta = 0, and 0 times infinity would be NaN.
__device__ __forceinline__ float rate2(float A)
{
    const float r = A * kLog2e;
    return r < -3.402823466e38f ? -3.402823466e38f : r;
}

// What a wavefront of the channel-per-lane kernels works on: one piece of a
// sequence and 64 channels of a group.  Neighbouring wavefronts take
// neighbouring channels of the same piece.
struct WaveItem {
    int slot, g, c;   // .. group, first channel within it
};

__device__ __forceinline__ WaveItem wave_item(int D, int G)
{
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const unsigned item = blockIdx.x * 4 + wave;   // below 2^26: scan_fits
    const unsigned per = (unsigned)(D / G + 63) / 64, all = per * (unsigned)G;
    WaveItem w;
    w.slot = (int)(item / all);
    const unsigned r = item - (unsigned)w.slot * all;
    w.g = (int)(r / per);
    w.c = (int)(r - (unsigned)w.g * per) * 64;
    return w;
}

// One batch of rows of B or C for a wavefront: each lane loads E adjacent
// values of one row, so that the batch is one load per lane; in LDS they are
// fp32 [row][NS], zeros past N and past the piece.  Only the wavefront itself
// reads them, so no barrier is needed: its LDS operations keep their order.
template <typename T, int NS>
struct RowStage {
    static constexpr int E = NS >= 8 ? NS / 8 : 1;
    Pack<T, E> q;

    __device__ __forceinline__ void fetch(const T* src, int64_t ld, int row, int rows, int N, int lane)
    {
        const int t = lane * E / NS, n = lane * E % NS;
        const bool in = lane * E < kBatch * NS && row + t < rows;
        q = load_some<T, E>(src + (int64_t)(in ? row + t : 0) * ld + n, in ? N - n : 0);
    }
    __device__ __forceinline__ void put(float (*dst)[NS], int lane) const
    {
        if (kBatch * NS < 64 * E && lane * E >= kBatch * NS) return;
        float v[E];
        unpack(q, v);
        float* p = &dst[0][0] + lane * E;
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] = v[i];
    }
};

// LDS written before, by any lane of the wavefront, is read after.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int SB>
__device__ __forceinline__ void read_states(const float* p, float (&o)[SB])   // 16-byte aligned
{
#pragma unroll
    for (int n = 0; n < SB; n += 4) {
        const float4 x = *reinterpret_cast<const float4*>(p + n);
        o[n] = x.x, o[n + 1] = x.y, o[n + 2] = x.z, o[n + 3] = x.w;
    }
}

// States read from LDS together: the next unit (row, block of states) is read
// while the present one is computed.
template <int NS>
constexpr int kUnit = NS < 8 ? NS : 8;

// Keeps a unit's products and reads where they stand: what depends on x and y
// is formed after this point, reads do not cross it.  Left alone, the compiler
// reads and multiplies a whole batch ahead and runs out of registers.
__device__ __forceinline__ void pin(float& x, float& y) { asm volatile("" : "+v"(x), "+v"(y)::"memory"); }

// Rows [row, row + kBatch) of channel d (the lane's), p the piece's first row;
// past its end the last row again.
template <typename T>
__device__ __forceinline__ void fetch_rows(T (&q)[kBatch], const T* p, int64_t ld, int row, int rows, int d)
{
#pragma unroll
    for (int i = 0; i < kBatch; ++i) q[i] = (p + (int64_t)min(row + i, rows - 1) * ld)[d];
}

// A batch's values past the end set to 0 (only the last batch has any).
__device__ __forceinline__ void zero_past(float (&o)[kBatch], int left)
{
    if (left < kBatch) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) o[i] = i < left ? o[i] : 0.0f;
    }
}

// delta of a batch, 0 past the end.
template <typename T>
__device__ __forceinline__ void batch_delta(float (&o)[kBatch], const T (&qt)[kBatch], float bias, int softplus, int left)
{
    if (softplus) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) o[i] = delta_of(to_f<T>(qt[i]), bias, 1);
    } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) o[i] = to_f<T>(qt[i]) + bias;
    }
    zero_past(o, left);
}

// ---------------------------------------------------------------------------
// A piece's own contribution, from a zero state.  Forward: the end state and
// sum(delta).  Reverse: the gradient that leaves the piece at its start,
// a_t0 G_t0 with G_t = C_t dS_t + a_{t+1} G_{t+1}, dS = dy z sigmoid(z).
// A lane is a channel with its NS states in registers; B or C is the same for
// every lane and read from LDS as a broadcast.  The next batch's loads are
// issued before the present one's rows; rows past the end of the piece run
// with delta = 0 and an input of 0, which change nothing.  With four wavefronts
// per SIMD bound by the vector ALU, 82 % busy: [4, 4096, 2048] bf16 with 16 states
// 117 us.  With the two that [4, 2048, 1024] has it is 52 % busy, and what the two
// wait for shows: 38 us.
// ---------------------------------------------------------------------------
template <typename T, int NS, bool REV>
__global__ __launch_bounds__(256) void scan_state_kernel(ScanArgs a, SeqMap m, int slots)
{
    __shared__ __align__(16) float bc[4][2][kBatch][NS];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const WaveItem w = wave_item(a.D, a.G);
    if (w.slot >= slots) return;
    const Piece p = seq_locate(m, w.slot);
    const int64_t t0 = p.index * m.piece;
    // forward: nothing follows a sequence's last piece; reverse: nothing
    // precedes its first, unless the initial state's gradient is wanted
    const bool last = t0 + m.piece >= p.len;
    if (!p.live || p.len == 0 || (REV ? p.index == 0 && !a.dh0 : last)) return;
    const int rows = (int)min((int64_t)m.piece, p.len - t0);
    const int Dg = a.D / a.G;
    const bool on = w.c + lane < Dg;
    const int d = w.g * Dg + (on ? w.c + lane : Dg - 1);   // a lane past the group repeats its last channel
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f;
    float A2[NS], h[NS], sd = 0.0f;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        A2[n] = n < a.N ? rate2(a.A[(int64_t)n * a.D + d]) : 0.0f;
        h[n] = 0.0f;
    }
    const int64_t r0 = p.row + t0;
    const T* pt = (const T*)a.dt + r0 * a.lddt;
    const T* pu = REV ? (const T*)a.dy + r0 * a.lddy : (const T*)a.u + r0 * a.ldu;
    const T* pz = REV && a.z ? (const T*)a.z + r0 * a.ldz : nullptr;
    const int64_t ldu = REV ? a.lddy : a.ldu, ldb = REV ? a.ldc : a.ldb;
    const T* pb = (const T*)(REV ? a.C : a.B) + r0 * ldb + (int64_t)w.g * a.N;
    const int batches = (rows + kBatch - 1) / kBatch;
    T qt[kBatch], qu[kBatch], qz[kBatch];
    RowStage<T, NS> sb;
    auto fetch = [&](int b) {
        const int row = (REV ? batches - 1 - b : b) * kBatch;
        sb.fetch(pb, ldb, row, rows, a.N, lane);
        fetch_rows(qt, pt, a.lddt, row, rows, d);
        fetch_rows(qu, pu, ldu, row, rows, d);
        if (REV && pz) fetch_rows(qz, pz, a.ldz, row, rows, d);
    };
    fetch(0);
    for (int b = 0; b < batches; ++b) {
        const int row = (REV ? batches - 1 - b : b) * kBatch;
        float(*B)[NS] = bc[wave][b & 1];
        sb.put(B, lane);
        float delta[kBatch], v[kBatch];
        batch_delta<T>(delta, qt, bias, a.softplus, rows - row);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) v[i] = REV ? to_f<T>(qu[i]) : to_f<T>(qu[i]) * delta[i];
        if (REV && pz) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v[i] *= to_f<T>(qz[i]) * sigmoid(to_f<T>(qz[i]));
        }
        zero_past(v, rows - row);
        if (b + 1 < batches) fetch(b + 1);
        wave_fence();
        constexpr int SB = kUnit<NS>, PER = NS / SB, UNITS = kBatch * PER;
        float bq[2][SB];
        auto row_of = [](int k) { return REV ? kBatch - 1 - k / PER : k / PER; };
        read_states<SB>(&B[row_of(0)][0], bq[0]);
#pragma unroll
        for (int k = 0; k < UNITS; ++k) {
            const int i = row_of(k), n0 = k % PER * SB;
            if (k + 1 < UNITS) read_states<SB>(&B[row_of(k + 1)][(k + 1) % PER * SB], bq[(k + 1) & 1]);
            pin(delta[i], v[i]);
            if (n0 == 0) sd += delta[i];
#pragma unroll
            for (int j = 0; j < SB; ++j) {
                const int n = n0 + j;
                const float e = exp2_hw(delta[i] * A2[n]);
                h[n] = REV ? e * fmaf(bq[k & 1][j], v[i], h[n]) : fmaf(e, h[n], v[i] * bq[k & 1][j]);
            }
        }
    }
    if (!on) return;
    float* st = a.st + (int64_t)w.slot * a.N * a.D + d;
#pragma unroll
    for (int n = 0; n < NS; ++n)
        if (n < a.N) st[(int64_t)n * a.D] = h[n];
    a.sd[(int64_t)w.slot * a.D + d] = sd;
}

// Carries states over a sequence's pieces, one thread per (sequence, state,
// channel): forward leaves in st[slot] the state that enters the piece;
// reverse the gradient that enters it from the right, and dh0.  Eight pieces'
// loads are in flight at a time, and one dependent product and sum per piece
// remains: 8 us for the 32 pieces of 64 rows of [4, 2048, 1024] with 16 states.
__global__ __launch_bounds__(256) void scan_join_kernel(ScanArgs a, SeqMap m, int reverse)
{
    const Piece p = seq_piece_of(m, (int)blockIdx.x);
    const int d = (int)blockIdx.y * 256 + (int)threadIdx.x, n = blockIdx.z;
    if (d >= a.D) return;
    const int64_t nd = (int64_t)n * a.D + d, ND = (int64_t)a.N * a.D;
    const float A2 = rate2(a.A[nd]);
    const int64_t pieces = p.len == 0 ? 1 : (p.len + m.piece - 1) / m.piece;
    float* st = a.st + (int64_t)p.slot0 * ND + nd;
    const float* sd = a.sd + (int64_t)p.slot0 * a.D + d;
    const float* from = reverse ? a.dh_last : a.h0;
    float h = from ? from[(int64_t)p.s * ND + nd] : 0.0f;
    // links: the pieces whose own contribution was formed
    const int64_t links = reverse ? (p.len == 0 ? 0 : (a.dh0 ? pieces : pieces - 1)) : pieces - 1;
    int64_t k = 0;
    auto at = [&](int64_t i) { return reverse ? pieces - 1 - i : i; };
    for (; k + 8 <= links; k += 8) {
        float e[8], f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            e[i] = st[at(k + i) * ND];
            f[i] = sd[at(k + i) * a.D];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            st[at(k + i) * ND] = h;
            h = fmaf(exp2_hw(f[i] * A2), h, e[i]);
        }
    }
    for (; k < links; ++k) {
        const float e = st[at(k) * ND], f = sd[at(k) * a.D];
        st[at(k) * ND] = h;
        h = fmaf(exp2_hw(f * A2), h, e);
    }
    if (k < pieces) st[at(k) * ND] = h;
    if (reverse && a.dh0) a.dh0[(int64_t)p.s * ND + nd] = h;
}

// What scan_join_kernel leaves for one (state, channel) of piece p, formed by the
// pass that needs it, in the same order: forward from the pieces before, reverse
// from those after (and dh0, by the first).  For few pieces: each joins its own.
template <bool REV>
__device__ __forceinline__ float join_own(const ScanArgs& a, const SeqMap& m, const Piece& p, int64_t nd, int d, float A)
{
    const int64_t ND = (int64_t)a.N * a.D;
    const float A2 = rate2(A);
    const float* from = REV ? a.dh_last : a.h0;
    float h = from ? from[(int64_t)p.s * ND + nd] : 0.0f;
    const int pieces = p.len == 0 ? 0 : (int)((p.len + m.piece - 1) / m.piece), own = (int)p.index;
    const int links = REV ? max(pieces - 1 - own, 0) : own;
    const float* st = a.st + (int64_t)p.slot0 * ND + nd;
    const float* sd = a.sd + (int64_t)p.slot0 * a.D + d;
    for (int k = 0; k < links; k += 4) {
        float e[4], f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // past the last link: the last again, unused
            const int l = min(k + i, links - 1), at = REV ? pieces - 1 - l : l;
            e[i] = st[at * ND];
            f[i] = sd[(int64_t)at * a.D];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k + i < links) h = fmaf(exp2_hw(f[i] * A2), h, e[i]);
    }
    if (REV && own == 0 && a.dh0) a.dh0[(int64_t)p.s * ND + nd] = pieces ? fmaf(exp2_hw(sd[0] * A2), h, st[0]) : h;
    return h;
}

// ---------------------------------------------------------------------------
// Main forward pass: a lane is a channel, its NS states in registers, one row
// at a time.  Per row and state one exp2 and four products or sums.  With four
// wavefronts per SIMD bound by the vector ALU, 84 % busy: [4, 4096, 2048] bf16 with
// 16 states 158 us, of whose 119 vector instructions per row 80 are the
// recurrence.  With two ([4, 2048, 1024]) 57 % busy: 48 us.
// Where N is not NS (FULL), a row ends with its last state: the B and C of 0 past
// it would turn an infinite input into NaN, which y would take.  At
// [4, 2048, 1024] with 11 states the forward pass takes 84.5 us so, 85.5 over all
// 16, and 87.1 with a select per sum.
// ---------------------------------------------------------------------------
template <typename T, int NS, bool FULL>
__global__ __launch_bounds__(256) void scan_fwd_kernel(ScanArgs a, SeqMap m, SeqMap keep, int slots)
{
    __shared__ __align__(16) float bs[4][2][kBatch][NS];
    __shared__ __align__(16) float cs[4][2][kBatch][NS];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const WaveItem w = wave_item(a.D, a.G);
    if (w.slot >= slots) return;
    const Piece p = seq_locate(m, w.slot);
    if (!p.live) return;
    const int64_t t0 = p.index * m.piece;
    const int rows = (int)min((int64_t)m.piece, p.len - t0);
    const int Dg = a.D / a.G;
    const bool on = w.c + lane < Dg;
    const int d = w.g * Dg + (on ? w.c + lane : Dg - 1);
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f, skip = a.skip ? a.skip[d] : 0.0f;
    const int64_t ND = (int64_t)a.N * a.D;
    float A2[NS], h[NS];
    const float* h_in = a.st ? a.st + (int64_t)w.slot * ND : (a.h0 ? a.h0 + (int64_t)p.s * ND : nullptr);
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        A2[n] = n < a.N ? rate2(a.A[(int64_t)n * a.D + d]) : 0.0f;
        h[n] = n < a.N && h_in ? h_in[(int64_t)n * a.D + d] : 0.0f;
    }
    float* hist = nullptr;
    if (a.hist) hist = a.hist + (seq_slot0(keep, p.s, p.row) + t0 / keep.piece) * ND + d;
    if (rows > 0) {
        const int64_t r0 = p.row + t0;
        const T* pt = (const T*)a.dt + r0 * a.lddt;
        const T* pu = (const T*)a.u + r0 * a.ldu;
        const T* pz = a.z ? (const T*)a.z + r0 * a.ldz : nullptr;
        const T* pb = (const T*)a.B + r0 * a.ldb + (int64_t)w.g * a.N;
        const T* pc = (const T*)a.C + r0 * a.ldc + (int64_t)w.g * a.N;
        T* py = (T*)a.y + r0 * a.ldy;
        T qt[kBatch], qu[kBatch], qz[kBatch];
        RowStage<T, NS> sb, sc;
        auto fetch = [&](int row) {
            sb.fetch(pb, a.ldb, row, rows, a.N, lane);
            sc.fetch(pc, a.ldc, row, rows, a.N, lane);
            fetch_rows(qt, pt, a.lddt, row, rows, d);
            fetch_rows(qu, pu, a.ldu, row, rows, d);
            if (pz) fetch_rows(qz, pz, a.ldz, row, rows, d);
        };
        fetch(0);
        for (int row = 0; row < rows; row += kBatch) {
            if (hist && on && row % keep.piece == 0) {
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    if (n < a.N) hist[(int64_t)n * a.D] = h[n];
                hist += ND;
            }
            float(*B)[NS] = bs[wave][row / kBatch & 1];
            float(*C)[NS] = cs[wave][row / kBatch & 1];
            sb.put(B, lane);
            sc.put(C, lane);
            float delta[kBatch], du[kBatch], y[kBatch], gate[kBatch];
            batch_delta<T>(delta, qt, bias, a.softplus, rows - row);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float u = to_f<T>(qu[i]);
                du[i] = delta[i] * u;
                y[i] = skip * u;
                gate[i] = 1.0f;
            }
            zero_past(du, rows - row);
            if (pz) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const float z = to_f<T>(qz[i]);
                    gate[i] = z * sigmoid(z);
                }
            }
            if (row + kBatch < rows) fetch(row + kBatch);
            wave_fence();
            constexpr int SB = kUnit<NS>, PER = NS / SB, UNITS = kBatch * PER;
            float bq[2][SB], cq[2][SB], y1 = 0.0f;
            read_states<SB>(&B[0][0], bq[0]);
            read_states<SB>(&C[0][0], cq[0]);
#pragma unroll
            for (int k = 0; k < UNITS; ++k) {
                const int i = k / PER, n0 = k % PER * SB;
                if (k + 1 < UNITS) {
                    read_states<SB>(&B[(k + 1) / PER][(k + 1) % PER * SB], bq[(k + 1) & 1]);
                    read_states<SB>(&C[(k + 1) / PER][(k + 1) % PER * SB], cq[(k + 1) & 1]);
                }
                pin(delta[i], du[i]);
                if (!FULL && n0 == 0) y1 = 0.0f;
#pragma unroll
                for (int j = 0; j < SB; ++j) {
                    const int n = n0 + j;
                    if (!FULL && n >= (NS > 4 ? NS / 2 : 1) && n >= a.N) break;   // more than half of NS exist
                    const float e = exp2_hw(delta[i] * A2[n]);
                    h[n] = fmaf(e, h[n], du[i] * bq[k & 1][j]);
                    if (FULL && n == 1) y1 = cq[k & 1][j] * h[n];
                    else if (n & 1) y1 = fmaf(cq[k & 1][j], h[n], y1);
                    else y[i] = fmaf(cq[k & 1][j], h[n], y[i]);
                }
                if (n0 + SB == NS) y[i] += y1;
                pin(y[i], y1);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) y[i] *= gate[i];
            if (on) {
                T* q = py + (int64_t)row * a.ldy;
                if (row + kBatch <= rows) {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) (q + i * a.ldy)[d] = (T)y[i];
                } else {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        if (row + i < rows) (q + i * a.ldy)[d] = (T)y[i];
                }
            }
        }
    } else if (hist && on) {   // the one slot of a sequence without rows
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (n < a.N) hist[(int64_t)n * a.D] = h[n];
    }
    if (on && a.h_last && t0 + rows == p.len) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (n < a.N) a.h_last[(int64_t)p.s * ND + (int64_t)n * a.D + d] = h[n];
    }
}

// ---------------------------------------------------------------------------
// Main backward pass over one piece of 64 rows and `chans` channels.
//
// Lane layout of a wavefront: lane = 16 q + seg.  Row q of 16 lanes holds
// NSL of its group's 4 NSL states, lane seg of the row the R rows from R seg
// of the piece on; the wavefront takes its channels one after another.  So
//  - the sums over channels (dB, dC) are register accumulators of the lane
//    that owns the row and the state: no exchange until the end;
//  - the recurrence is a scan over a lane's R rows in registers, then over the
//    16 lanes of a DPP row (four shift-and-add levels), forward from the
//    stored state and backward from the joined gradient;
//  - the exponentials of a row and state are formed once and serve both.
// With R = 4 and NSL = 4 a lane's B, C, dB, dC, decays and states take about 205
// registers, two wavefronts per SIMD.  (R = 8, three wavefronts per SIMD, and two
// channels at a time all spilled and were slower.  With at most 8 states R = 8
// fits: [8, 2048, 1024] with 8 states 237 us against 261, but half as many
// pieces to fill the chip with: at [4, 2048, 512] the backward pass takes 92
// against 90 and the forward 66 against 49, with 4 states 77 against 72 and 57
// against 39.  So R is 4 throughout.)  Bound by the vector ALU, 76 % busy:
// [4, 2048, 1024] bf16 with 16 states 158 us.
// With N > 16 states the four wavefronts share channels: NG groups of 16
// states each, 4 / NG channels side by side.
// Per-row values of 16 channels at a time (delta, u, dS, slopes) are formed once,
// coalesced, and handed over in LDS as [channel][row]; the per-row sums over
// states come back the same way for the elementwise tail.
// ---------------------------------------------------------------------------
constexpr int kCB = 16;                  // channels per LDS round
constexpr int R = 4;                     // rows per lane
constexpr int kRows = 16 * R;            // rows per piece
static_assert(kRows == kScanKeep, "the backward pass starts from the states kept");
constexpr int kLd = kRows + 4;           // row pitch in LDS: the staging writes of 4 channels fall on distinct banks

template <int NG>
struct BwdLds {
    float delta[kCB][kLd], u[kCB][kLd], ds[kCB][kLd];   // ds = dy z sigmoid(z)
    float sg[kCB][kLd], gz[kCB][kLd];                   // d delta / d dt, d (y gate) / dz over y: each thread's own
    float y[NG][kCB][kLd], s1[NG][kCB][kLd], s2[NG][kCB][kLd];
    float A2[kCB][NG * 16], hin[kCB][NG * 16], gin[kCB][NG * 16], dA[kCB][NG * 16];
    float red[4][2][kCB];
};

// v[0 .. 4) summed over the four rows of 16 lanes: lane (q, seg) stores element
// q of its four to out.
__device__ __forceinline__ void quad_rows_sum(const float (&v)[R], float* out, int q)
{
    out[q] = pair_sum16(pair_sum32(v[0], v[2]), pair_sum32(v[1], v[3]));
}

// Lane k < NSL of each row of 16 gets v[k] summed over the row.
template <int NSL>
__device__ __forceinline__ float rows_of_16_sum(const float (&v)[NSL], int seg)
{
    constexpr int kXor1 = 0xB1, kXor2 = 0x4E;   // quad_perm [1,0,3,2] and [2,3,0,1]
    float x;
    if constexpr (NSL == 1) {
        x = v[0] + dpp0<kXor1>(v[0]);
        x += dpp0<kXor2>(x);
    } else {
        const bool odd = seg & 1, high = seg & 2;
        x = (odd ? v[1] : v[0]) + dpp0<kXor1>(odd ? v[0] : v[1]);
        if constexpr (NSL == 2) {
            x += dpp0<kXor2>(x);
        } else {
            const float y = (odd ? v[3] : v[2]) + dpp0<kXor1>(odd ? v[2] : v[3]);
            x = (high ? y : x) + dpp0<kXor2>(high ? x : y);
        }
    }
    x += dpp0<kRowRor(4)>(x);
    return x + dpp0<kRowRor(8)>(x);
}

__device__ __forceinline__ void load_r(const float* p, float (&o)[R])   // 16-byte aligned
{
    const float4 x = *reinterpret_cast<const float4*>(p);
    o[0] = x.x, o[1] = x.y, o[2] = x.z, o[3] = x.w;
}

template <int CTRL>
__device__ __forceinline__ float dpp_or(float old, float x)   // lanes without a source keep old
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, x),
                                                                CTRL, 0xf, 0xf, false));
}

// Inclusive scans of pairs (P, H) over the 16 lanes of a row, H += P H(before),
// P *= P(before), shifted right (forward) or left; lanes without a source read
// 0.  Written as instructions because the shifted operand of a multiply-add is
// otherwise moved first.  A register is read through a shift at the earliest
// two instructions after it was written: four pairs per statement see to that,
// smaller groups wait.
#define SEQ_LEVEL(sh)                                                                                                      \
    if constexpr (NSL == 4) {                                                                                             \
        asm volatile("s_nop 1\n\t"                                                                                        \
                     "v_fmac_f32_dpp %0, %0, %4 " sh " row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"                       \
                     "v_fmac_f32_dpp %1, %1, %5 " sh " row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"                       \
                     "v_fmac_f32_dpp %2, %2, %6 " sh " row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"                       \
                     "v_fmac_f32_dpp %3, %3, %7 " sh " row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"                       \
                     "v_mul_f32_dpp %4, %4, %4 " sh " row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"                        \
                     "v_mul_f32_dpp %5, %5, %5 " sh " row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"                        \
                     "v_mul_f32_dpp %6, %6, %6 " sh " row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"                        \
                     "v_mul_f32_dpp %7, %7, %7 " sh " row_mask:0xf bank_mask:0xf bound_ctrl:1"                            \
                     : "+v"(H[0]), "+v"(H[1]), "+v"(H[2]), "+v"(H[3]), "+v"(P[0]), "+v"(P[1]), "+v"(P[2]), "+v"(P[3])); \
    } else {                                                                                                              \
        for (int j = 0; j < NSL; ++j)                                                                                     \
            asm volatile("s_nop 1\n\t"                                                                                    \
                         "v_fmac_f32_dpp %0, %0, %1 " sh " row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"                   \
                         "v_mul_f32_dpp %1, %1, %1 " sh " row_mask:0xf bank_mask:0xf bound_ctrl:1"                        \
                         : "+v"(H[j]), "+v"(P[j]));                                                                       \
    }

template <bool LEFT, int LEVEL, int NSL>
__device__ __forceinline__ void scan_level(float (&P)[NSL], float (&H)[NSL])
{
    if constexpr (!LEFT && LEVEL == 1) { SEQ_LEVEL("row_shr:1") }
    if constexpr (!LEFT && LEVEL == 2) { SEQ_LEVEL("row_shr:2") }
    if constexpr (!LEFT && LEVEL == 4) { SEQ_LEVEL("row_shr:4") }
    if constexpr (!LEFT && LEVEL == 8) { SEQ_LEVEL("row_shr:8") }
    if constexpr (LEFT && LEVEL == 1) { SEQ_LEVEL("row_shl:1") }
    if constexpr (LEFT && LEVEL == 2) { SEQ_LEVEL("row_shl:2") }
    if constexpr (LEFT && LEVEL == 4) { SEQ_LEVEL("row_shl:4") }
    if constexpr (LEFT && LEVEL == 8) { SEQ_LEVEL("row_shl:8") }
}
#undef SEQ_LEVEL

template <bool LEFT, int NSL>
__device__ __forceinline__ void row_scan(float (&P)[NSL], float (&H)[NSL])
{
    scan_level<LEFT, 1>(P, H);
    scan_level<LEFT, 2>(P, H);
    scan_level<LEFT, 4>(P, H);
    scan_level<LEFT, 8>(P, H);
    asm volatile("s_nop 1");   // the caller shifts the results once more
}

// Sums over states leave out those past N.  B and C are 0 there, but 0 times an
// infinite input is NaN.  So a lane none of whose states exist computes on zeros
// (here), and where N cuts a lane's states its sums take only those that exist:
// the backward pass of [4, 2048, 1024] takes 205 us with 11 states, 195 without
// these selects.
enum Cut { kFull, kWholeLanes, kWithinLane };   // N fills the lanes, ends between two, within one

template <int CUT>
__device__ __forceinline__ bool exists(int n, int j, int N)   // the lane's state j is n; of a lane with states, the first exists
{
    return CUT != kWithinLane || j == 0 || n < N;
}
__device__ __forceinline__ void zero_without_states(bool none, float (&x)[R])
{
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = none ? 0.0f : x[i];
}
__device__ __forceinline__ void zero_without_states(bool none, float (&x)[R], float (&y)[R], float& sum)
{
    zero_without_states(none, x);
    zero_without_states(none, y);
    sum = none ? 0.0f : sum;
}

// The lane's R rows of NSL states of B or C as fp32, zeros past the piece's rows
// and past N.  All loads are issued before the first is converted.
template <typename T, int NSL>
__device__ __forceinline__ void load_states(const T* src, int64_t ld, int row0, int rows, int n0, int N, float (&o)[R][NSL])
{
    Pack<T, NSL> q[R];
    if (N % NSL == 0) {   // no lane has a tail: one load each, inside the buffer, unused where there is nothing
        const int n = n0 < N ? n0 : 0;
#pragma unroll
        for (int i = 0; i < R; ++i) q[i] = load_pack<T, NSL>(src + (int64_t)min(row0 + i, rows - 1) * ld + n);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) q[i] = load_some<T, NSL>(src + (int64_t)min(row0 + i, rows - 1) * ld + n0, N - n0);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        unpack(q[i], o[i]);
        if (row0 + i >= rows || n0 >= N) {
#pragma unroll
            for (int j = 0; j < NSL; ++j) o[i][j] = 0.0f;
        }
    }
}

// JOIN (ScanArgs::join) is a constant: with both ways in one kernel it took 162 us
// where it takes 158 without the other.
template <typename T, int NSL, int NG, bool JOIN, int CUT>
__global__ __launch_bounds__(256, 2) void scan_bwd_kernel(ScanArgs a, SeqMap m)
{
    extern __shared__ __align__(16) char smem[];
    using Lds = BwdLds<NG>;
    Lds& L = *reinterpret_cast<Lds*>(smem);
    constexpr int NP = 4 * NSL * NG;   // states, padded
    const int tid = (int)threadIdx.x, wave = tid >> 6, lane = tid & 63, q = lane >> 4, seg = lane & 15;
    const int ng = wave % NG, cs = wave / NG;
    const int n0 = ng * 4 * NSL + q * NSL;   // the lane's first state
    const int slot = (int)blockIdx.x;
    const Piece p = seq_locate(m, slot);
    const int g = blockIdx.z, Dg = a.D / a.G;
    const int c_begin = (int)blockIdx.y * a.chans, c_end = min(Dg, c_begin + a.chans);
    const int64_t ND = (int64_t)a.N * a.D;
    float* part_p = a.part_p + (int64_t)slot * (ND + 2 * (int64_t)a.D);
    const int64_t t0 = p.index * m.piece;
    if (!p.live || p.len == 0) {   // a slot without rows adds nothing to the parameters' gradients
        const int w = c_end - c_begin;
        for (int i = tid; i < (a.N + 2) * w; i += 256)
            part_p[(int64_t)(i / w) * a.D + g * Dg + c_begin + i % w] = 0.0f;
        if (JOIN && p.live)   // a sequence without rows hands dh_last on
            for (int i = tid; i < a.N * w; i += 256) {
                const int d = g * Dg + c_begin + i % w;
                join_own<true>(a, m, p, (int64_t)(i / w) * a.D + d, d, 0.0f);
            }
        return;
    }
    const int rows = (int)min((int64_t)kRows, p.len - t0);
    const int64_t r0 = p.row + t0;

    float Bv[R][NSL], Cv[R][NSL], dB[R][NSL], dC[R][NSL];
    load_states<T, NSL>((const T*)a.B + r0 * a.ldb + (int64_t)g * a.N, a.ldb, seg * R, rows, n0, a.N, Bv);
    load_states<T, NSL>((const T*)a.C + r0 * a.ldc + (int64_t)g * a.N, a.ldc, seg * R, rows, n0, a.N, Cv);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < NSL; ++j) dB[i][j] = dC[i][j] = 0.0f;

    const int chg = tid & 3, r_of = tid >> 2;   // elementwise work: 4 channels of row r_of
    const float* hist = a.hist + (int64_t)slot * ND;
    const float* gin = a.st ? a.st + (int64_t)slot * ND : (a.dh_last ? a.dh_last + (int64_t)p.s * ND : nullptr);

    struct Raw {
        Pack<T, 4> u, dt, dy, z;
    } raw;
    // whole groups of four channels: one load each, at a place inside the
    // buffers for threads that have none; what they load is not used
    const bool quads = Dg % 4 == 0;
    auto fetch = [&](int cb) {
        const int c = cb + chg * 4, dch = g * Dg + (c < c_end ? c : c_begin);
        const int64_t r = r0 + (r_of < rows ? r_of : 0);
        const T* pu = (const T*)a.u + r * a.ldu + dch;
        const T* pt = (const T*)a.dt + r * a.lddt + dch;
        const T* py = (const T*)a.dy + r * a.lddy + dch;
        const T* pz = (const T*)a.z + r * a.ldz + dch;
        if (quads) {
            raw.u = load_pack<T, 4>(pu);
            raw.dt = load_pack<T, 4>(pt);
            raw.dy = load_pack<T, 4>(py);
            if (a.z) raw.z = load_pack<T, 4>(pz);
        } else {
            const int n = c_end - c;
            raw.u = load_some<T, 4>(pu, n);
            raw.dt = load_some<T, 4>(pt, n);
            raw.dy = load_some<T, 4>(py, n);
            if (a.z) raw.z = load_some<T, 4>(pz, n);
        }
    };
    constexpr int kPer = NP * kCB > 256 ? NP * kCB / 256 : 1;   // a thread's (channel, state) pairs of a round
    float rA[kPer], rh[kPer], rg[kPer];
    auto fetch_states = [&](int cb) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = tid + 256 * k, n = i / kCB, c = cb + i % kCB;
            const bool in = n < a.N && c < c_end;
            const int64_t at = (int64_t)n * a.D + g * Dg + c;
            rA[k] = in ? a.A[at] : 0.0f;
            rh[k] = in ? hist[at] : 0.0f;
            if (JOIN) rg[k] = in ? join_own<true>(a, m, p, at, g * Dg + c, rA[k]) : 0.0f;
            else rg[k] = in && gin ? gin[at] : 0.0f;
        }
    };
    fetch(c_begin);
    fetch_states(c_begin);
    for (int cb = c_begin; cb < c_end; cb += kCB) {
        const int dch = g * Dg + cb + chg * 4, nch = c_end - cb - chg * 4;   // the thread's channels
        float skip[4];
        {
            float bias[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                bias[e] = e < nch && a.dt_bias ? a.dt_bias[dch + e] : 0.0f;
                skip[e] = e < nch && a.skip ? a.skip[dch + e] : 0.0f;
            }
            const int n = r_of < rows ? nch : 0;
            float u[4], x[4], dy[4], sg[4];
            unpack(raw.u, u);
            unpack(raw.dt, x);
            unpack(raw.dy, dy);
            if (a.softplus) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float xb = x[e] + bias[e], ex = exp_neg_abs(xb);
                    x[e] = softplus_e(xb, ex);
                    sg[e] = sigmoid_e(xb, ex);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] += bias[e], sg[e] = 1.0f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {   // past the rows and channels: zeros
                L.delta[chg * 4 + e][r_of] = e < n ? x[e] : 0.0f;
                L.u[chg * 4 + e][r_of] = e < n ? u[e] : 0.0f;
                L.sg[chg * 4 + e][r_of] = sg[e];
            }
            if (a.z) {
                float z[4];
                unpack(raw.z, z);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float s = sigmoid(z[e]);
                    L.gz[chg * 4 + e][r_of] = dy[e] * (s * fmaf(z[e], 1.0f - s, 1.0f));
                    dy[e] *= z[e] * s;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) L.ds[chg * 4 + e][r_of] = e < n ? dy[e] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = tid + 256 * k, n = i / kCB, c = i % kCB;
            if (n >= NP) break;
            L.A2[c][n] = rate2(rA[k]);
            L.hin[c][n] = rh[k];
            L.gin[c][n] = rg[k];
        }
        lds_barrier();
        if (cb > c_begin && tid < 2 * kCB) {   // the round before: its sums over rows
            const int k = tid / kCB, c = tid % kCB;
            part_p[(int64_t)(a.N + k) * a.D + g * Dg + cb - kCB + c] =
                (L.red[0][k][c] + L.red[1][k][c]) + (L.red[2][k][c] + L.red[3][k][c]);
        }

        if (cb + kCB < c_end) {
            fetch(cb + kCB);
            fetch_states(cb + kCB);
        }
        const int nc = min(kCB, c_end - cb);
        for (int c = cs; c < nc; c += 4 / NG) {
            float A2[NSL], P[NSL], P0[NSL], H[NSL], hv[NSL], av[R][NSL], ah[R][NSL];
            float dl[R], du[R], ds[R], sd = 0.0f;
            load_r(&L.delta[c][seg * R], dl);
            load_r(&L.u[c][seg * R], du);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                du[i] *= dl[i];
                sd += dl[i];
            }
            if (CUT != kFull) zero_without_states(n0 >= a.N, dl, du, sd);
#pragma unroll
            for (int j = 0; j < NSL; ++j) {
                A2[j] = L.A2[c][n0 + j];
                hv[j] = L.hin[c][n0 + j];
                P0[j] = P[j] = exp2_hw(A2[j] * sd);
                H[j] = 0.0f;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    av[i][j] = exp2_hw(dl[i] * A2[j]);
                    H[j] = fmaf(av[i][j], H[j], du[i] * Bv[i][j]);
                }
                if (seg == 0) H[j] = fmaf(P[j], hv[j], H[j]);
            }
            row_scan<false>(P, H);
#pragma unroll
            for (int j = 0; j < NSL; ++j) hv[j] = dpp_or<0x111>(hv[j], H[j]);   // the state that enters this lane's rows
            float y[R];
            load_r(&L.ds[c][seg * R], ds);
            if (CUT != kFull) zero_without_states(n0 >= a.N, ds);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                y[i] = 0.0f;
#pragma unroll
                for (int j = 0; j < NSL; ++j) {
                    ah[i][j] = av[i][j] * hv[j];
                    hv[j] = fmaf(du[i], Bv[i][j], ah[i][j]);
                    dC[i][j] = fmaf(ds[i], hv[j], dC[i][j]);
                    const float t = fmaf(Cv[i][j], hv[j], y[i]);
                    y[i] = exists<CUT>(n0 + j, j, a.N) ? t : y[i];
                }
            }
            if (a.z) quad_rows_sum(y, &L.y[ng][c][seg * R], q);
            if (rows < kRows) {   // past the piece's end delta is 0, but 0 times an infinite state is NaN
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int j = 0; j < NSL; ++j) ah[i][j] = seg * R + i < rows ? ah[i][j] : 0.0f;
            }
            float G[NSL], gi[NSL], dA[NSL], s1[R], s2[R];
#pragma unroll
            for (int j = 0; j < NSL; ++j) {
                gi[j] = L.gin[c][n0 + j];
                G[j] = dA[j] = 0.0f;
#pragma unroll
                for (int i = R - 1; i >= 0; --i) G[j] = av[i][j] * fmaf(Cv[i][j], ds[i], G[j]);
                if (seg == 15) G[j] = fmaf(P0[j], gi[j], G[j]);
            }
            row_scan<true>(P0, G);
#pragma unroll
            for (int j = 0; j < NSL; ++j) G[j] = dpp_or<0x101>(gi[j], G[j]);   // what enters from the rows after this lane's
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                s1[i] = s2[i] = 0.0f;
#pragma unroll
                for (int j = 0; j < NSL; ++j) {
                    G[j] = fmaf(Cv[i][j], ds[i], G[j]);
                    dB[i][j] = fmaf(G[j], du[i], dB[i][j]);
                    const float t1 = fmaf(G[j], Bv[i][j], s1[i]), k = G[j] * ah[i][j], t2 = fmaf(k, A2[j], s2[i]);
                    s1[i] = exists<CUT>(n0 + j, j, a.N) ? t1 : s1[i];
                    s2[i] = exists<CUT>(n0 + j, j, a.N) ? t2 : s2[i];
                    dA[j] = fmaf(k, dl[i], dA[j]);
                    G[j] *= av[i][j];
                }
            }
            const float dAs = rows_of_16_sum(dA, seg);
            if (seg < NSL) L.dA[c][n0 + seg] = dAs;
            quad_rows_sum(s1, &L.s1[ng][c][seg * R], q);
            quad_rows_sum(s2, &L.s2[ng][c][seg * R], q);
        }
        lds_barrier();

        float rs[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};   // dskip, ddt_bias
        if (r_of < rows && nch > 0) {
            const int64_t r = r0 + r_of;
            float odu[4], oddt[4], odz[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = chg * 4 + e;
                const float u = L.u[c][r_of], ds = L.ds[c][r_of];
                float s1 = 0.0f, s2 = 0.0f, y = skip[e] * u;
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    s1 += L.s1[i][c][r_of];
                    s2 += L.s2[i][c][r_of];
                    y += L.y[i][c][r_of];   // without z: not written, not used
                }
                odz[e] = L.gz[c][r_of] * y;
                odu[e] = fmaf(L.delta[c][r_of], s1, skip[e] * ds);
                oddt[e] = fmaf(u, s1, s2 * kLn2) * L.sg[c][r_of];
                if (e < nch) {
                    rs[0][e] = fmaf(ds, u, rs[0][e]);
                    rs[1][e] += oddt[e];
                }
            }
            if (quads) {
                store_pack<T, 4>((T*)a.du + r * a.lddu + dch, odu);
                store_pack<T, 4>((T*)a.ddt + r * a.ldddt + dch, oddt);
                if (a.z) store_pack<T, 4>((T*)a.dz + r * a.lddz + dch, odz);
            } else {
                store_some<T, 4>((T*)a.du + r * a.lddu + dch, odu, nch);
                store_some<T, 4>((T*)a.ddt + r * a.ldddt + dch, oddt, nch);
                if (a.z) store_some<T, 4>((T*)a.dz + r * a.lddz + dch, odz, nch);
            }
        }
        // sums over the wavefront's rows: lanes 4 apart, then the four rows of
        // 16 lanes, of which row i ends with channel 4 chg + i
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                rs[k][e] += dpp0<kRowRor(8)>(rs[k][e]);
                rs[k][e] += dpp0<kRowRor(4)>(rs[k][e]);
            }
            const float v = pair_sum32(pair_sum16(rs[k][0], rs[k][1]), pair_sum16(rs[k][2], rs[k][3]));
            if (seg < 4) L.red[wave][k][seg * 4 + q] = v;
        }
        for (int i = tid; i < a.N * kCB; i += 256) {
            const int n = i / kCB, c = i % kCB;
            if (cb + c < c_end) part_p[(int64_t)n * a.D + g * Dg + cb + c] = L.dA[c][n];
        }
    }
    __syncthreads();
    if (tid < 2 * kCB) {
        const int k = tid / kCB, c = tid % kCB, cb = c_begin + (c_end - c_begin - 1) / kCB * kCB;
        if (cb + c < c_end)
            part_p[(int64_t)(a.N + k) * a.D + g * Dg + cb + c] =
                (L.red[0][k][c] + L.red[1][k][c]) + (L.red[2][k][c] + L.red[3][k][c]);
    }
    __syncthreads();
    // dB and dC over the wavefronts that share states: added in order in LDS
    float(*acc)[kRows][NP + 1] = reinterpret_cast<float(*)[kRows][NP + 1]>(smem);
    static_assert(sizeof(float) * 2 * kRows * (NP + 1) <= sizeof(Lds), "the exchange fits the round's LDS");
    for (int w = 0; w < 4 / NG; ++w) {
        if (cs == w) {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < NSL; ++j) {
                    float* b = &acc[0][seg * R + i][n0 + j];
                    float* c = &acc[1][seg * R + i][n0 + j];
                    *b = w == 0 ? dB[i][j] : *b + dB[i][j];
                    *c = w == 0 ? dC[i][j] : *c + dC[i][j];
                }
        }
        __syncthreads();
    }
    const int64_t GN = (int64_t)a.G * a.N;
    float* o = a.part_bc + (int64_t)blockIdx.y * 2 * a.rows.total * GN + r0 * GN + (int64_t)g * a.N;
    for (int i = tid; i < rows * a.N; i += 256) {
        const int t = i / a.N, n = i % a.N;
        o[t * GN + n] = acc[0][t][n];
        o[a.rows.total * GN + t * GN + n] = acc[1][t][n];
    }
}

// ---------------------------------------------------------------------------
// The state passes and the forward pass for little work, in the backward
// kernel's lane layout: a wavefront takes 64 rows of a channel at once, so a
// small batch of short sequences occupies rows x channels / 64 wavefronts
// instead of rows x channels / (64 x its rows one after another).  Per row and
// state it costs about a third more than a channel per lane.  One round of 16
// channels per workgroup; the piece is the backward kernel's.  Bound by latency:
// 32 sequences of ~65 rows, 128 channels, 32 states 11 us per state pass, 14 us
// forward.
// ---------------------------------------------------------------------------
enum RowsMode { kStateFwd, kStateRev, kForward };

template <int NG>
struct RowsLds {
    float delta[kCB][kLd], v[kCB][kLd];            // v: u, or dS in reverse
    float gate[kCB][kLd], y[NG][kCB][kLd];         // forward
    float A2[kCB][NG * 16], hin[kCB][NG * 16];
};

template <typename T, int NSL, int NG, int MODE, int CUT>
__global__ __launch_bounds__(256) void scan_rows_kernel(ScanArgs a, SeqMap m)
{
    using Lds = RowsLds<NG>;
    __shared__ __align__(16) Lds L;
    constexpr int NP = 4 * NSL * NG;
    const int tid = (int)threadIdx.x, wave = tid >> 6, lane = tid & 63, q = lane >> 4, seg = lane & 15;
    const int ng = wave % NG, cs = wave / NG, n0 = ng * 4 * NSL + q * NSL;
    const int slot = (int)blockIdx.x;
    const Piece p = seq_locate(m, slot);
    const int64_t t0 = p.index * m.piece;
    const bool last = t0 + m.piece >= p.len;
    if (!p.live) return;
    if (MODE == kStateFwd && last) return;
    if (MODE == kStateRev && (p.len == 0 || (p.index == 0 && !a.dh0))) return;
    const int rows = (int)min((int64_t)kRows, p.len - t0);
    const int64_t r0 = p.row + t0, ND = (int64_t)a.N * a.D;
    const int g = blockIdx.z, Dg = a.D / a.G, cb = (int)blockIdx.y * kCB, d0 = g * Dg + cb;
    const int nc = min(kCB, Dg - cb);

    // every load goes out before the first wait
    const int chg = tid & 3, r_of = tid >> 2, nch = nc - chg * 4, dch = d0 + chg * 4;
    const bool gated = MODE != kStateFwd && a.z;
    Pack<T, 4> qx = {}, qv = {}, qz = {};
    if (rows > 0) {
        const int at = nch > 0 ? dch : d0;   // inside the buffers for threads that have no channels
        const bool quads = Dg % 4 == 0;
        const int64_t r = r0 + min(r_of, rows - 1);
        const T* pt = (const T*)a.dt + r * a.lddt + at;
        const T* pv = MODE == kStateRev ? (const T*)a.dy + r * a.lddy + at : (const T*)a.u + r * a.ldu + at;
        const T* pz = (const T*)a.z + r * a.ldz + at;
        if (quads) {
            qx = load_pack<T, 4>(pt);
            qv = load_pack<T, 4>(pv);
            if (gated) qz = load_pack<T, 4>(pz);
        } else {
            qx = load_some<T, 4>(pt, nch);
            qv = load_some<T, 4>(pv, nch);
            if (gated) qz = load_some<T, 4>(pz, nch);
        }
    }
    float Bv[R][NSL] = {}, Cv[R][NSL] = {};
    if (rows > 0) {   // (a sequence without rows hands its state on)
        if (MODE != kStateRev)
            load_states<T, NSL>((const T*)a.B + r0 * a.ldb + (int64_t)g * a.N, a.ldb, seg * R, rows, n0, a.N, Bv);
        if (MODE != kStateFwd)
            load_states<T, NSL>((const T*)a.C + r0 * a.ldc + (int64_t)g * a.N, a.ldc, seg * R, rows, n0, a.N, Cv);
    }
    const float* h_in = nullptr;
    if (MODE == kForward) h_in = a.st ? a.st + (int64_t)slot * ND : (a.h0 ? a.h0 + (int64_t)p.s * ND : nullptr);
    for (int i = tid; i < NP * kCB; i += 256) {
        const int n = i / kCB, c = i % kCB;
        const bool in = n < a.N && c < nc;
        const int64_t at = (int64_t)n * a.D + d0 + c;
        float h = 0.0f;
        if (MODE == kForward && in) h = a.join ? join_own<false>(a, m, p, at, d0 + c, a.A[at]) : (h_in ? h_in[at] : 0.0f);
        L.A2[c][n] = in ? rate2(a.A[at]) : 0.0f;
        if (MODE == kForward) {
            L.hin[c][n] = h;
            if (in && a.hist) a.hist[(int64_t)slot * ND + at] = h;
        }
    }
    const int n = r_of < rows ? nch : 0;
    float x[4], v[4], z[4];
    unpack(qx, x);
    unpack(qv, v);
    if (gated) unpack(qz, z);
#pragma unroll
    for (int e = 0; e < 4; ++e) {   // past the rows and channels: zeros
        const float dlt = delta_of(x[e], e < n && a.dt_bias ? a.dt_bias[dch + e] : 0.0f, a.softplus);
        const float gate = gated ? z[e] * sigmoid(z[e]) : 1.0f;
        L.delta[chg * 4 + e][r_of] = e < n ? dlt : 0.0f;
        L.v[chg * 4 + e][r_of] = e < n ? (MODE == kStateRev ? v[e] * gate : v[e]) : 0.0f;
        if (MODE == kForward) L.gate[chg * 4 + e][r_of] = gate;
    }
    __syncthreads();
    for (int c = cs; c < nc; c += 4 / NG) {
        float A2[NSL], P[NSL], H[NSL], hv[NSL], av[R][NSL], dl[R], v[R], sd = 0.0f;
        load_r(&L.delta[c][seg * R], dl);
        load_r(&L.v[c][seg * R], v);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            sd += dl[i];
            if (MODE != kStateRev) v[i] *= dl[i];
        }
        if (CUT != kFull) zero_without_states(n0 >= a.N, dl, v, sd);
#pragma unroll
        for (int j = 0; j < NSL; ++j) {
            A2[j] = L.A2[c][n0 + j];
            P[j] = exp2_hw(A2[j] * sd);
            H[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < R; ++i) av[i][j] = exp2_hw(dl[i] * A2[j]);
            if (MODE == kStateRev) {
#pragma unroll
                for (int i = R - 1; i >= 0; --i) H[j] = av[i][j] * fmaf(Cv[i][j], v[i], H[j]);
            } else {
#pragma unroll
                for (int i = 0; i < R; ++i) H[j] = fmaf(av[i][j], H[j], v[i] * Bv[i][j]);
            }
            if (MODE == kForward) {
                hv[j] = L.hin[c][n0 + j];
                if (seg == 0) H[j] = fmaf(P[j], hv[j], H[j]);
            }
        }
        row_scan<MODE == kStateRev>(P, H);
        const int64_t d = d0 + c;
        if (MODE != kForward) {
            sd = row_sum(sd);
            if (seg == (MODE == kStateRev ? 0 : 15)) {
#pragma unroll
                for (int j = 0; j < NSL; ++j)
                    if (n0 + j < a.N) a.st[(int64_t)slot * ND + (int64_t)(n0 + j) * a.D + d] = H[j];
                if (n0 == 0) a.sd[(int64_t)slot * a.D + d] = sd;
            }
        } else {
            // rows past the end change nothing: lane 15 holds the state after the last
            if (a.h_last && last && seg == 15) {
#pragma unroll
                for (int j = 0; j < NSL; ++j)
                    if (n0 + j < a.N) a.h_last[(int64_t)p.s * ND + (int64_t)(n0 + j) * a.D + d] = H[j];
            }
            float y[R];
#pragma unroll
            for (int j = 0; j < NSL; ++j) hv[j] = dpp_or<0x111>(hv[j], H[j]);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                y[i] = 0.0f;
#pragma unroll
                for (int j = 0; j < NSL; ++j) {
                    hv[j] = fmaf(av[i][j], hv[j], v[i] * Bv[i][j]);
                    const float t = fmaf(Cv[i][j], hv[j], y[i]);
                    y[i] = exists<CUT>(n0 + j, j, a.N) ? t : y[i];
                }
            }
            quad_rows_sum(y, &L.y[ng][c][seg * R], q);
        }
    }
    if (MODE != kForward) return;
    __syncthreads();
    if (r_of < rows && nch > 0) {
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = chg * 4 + e;
            float y = e < nch && a.skip ? a.skip[dch + e] * L.v[c][r_of] : 0.0f;
#pragma unroll
            for (int i = 0; i < NG; ++i) y += L.y[i][c][r_of];
            o[e] = y * L.gate[c][r_of];
        }
        store_some<T, 4>((T*)a.y + (r0 + r_of) * a.ldy + dch, o, nch);
    }
}

// ---------------------------------------------------------------------------
// One token: a workgroup takes 64 V channels of one sequence (64 lanes of V),
// its four wavefronts a quarter of the states each; y's quarters meet in LDS.
// The state is read and written once.  V divides the group's channels.  Bound by
// memory: 256 sequences of 2048 channels with 16 states 76 MB in 17 us, 4.4 TB/s;
// one sequence 4 us, a launch's latency.
// ---------------------------------------------------------------------------
template <typename T, int NQ, int V>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanStepArgs a)
{
    __shared__ float ys[4][64 * V];
    const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
    const int64_t s = blockIdx.x;
    const int g = blockIdx.z, Dg = a.D / a.G;
    const int c = (int)blockIdx.y * 64 * V + lane * V;
    const bool on = c < Dg;
    const int d = g * Dg + (on ? c : 0);
    const int n0 = wave * NQ;
    float* h = a.h + (s * a.N + n0) * a.D + d;
    const T* pb = (const T*)a.B + s * a.ldb + (int64_t)g * a.N;
    const T* pc = (const T*)a.C + s * a.ldc + (int64_t)g * a.N;
    Pack<float, V> hq[NQ], aq[NQ];
    float B[NQ], C[NQ];
    // a state past N repeats the last: not used, not stored
#pragma unroll
    for (int j = 0; j < NQ; ++j) hq[j] = load_pack<float, V>(h + (int64_t)(min(n0 + j, a.N - 1) - n0) * a.D);
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int n = min(n0 + j, a.N - 1);
        aq[j] = load_pack<float, V>(a.A + (int64_t)n * a.D + d);
        B[j] = to_f<T>(pb[n]);
        C[j] = n0 + j < a.N ? to_f<T>(pc[n]) : 0.0f;
    }
    float u[V], x[V], z[V], bias[V], skip[V], y[V];
#pragma unroll
    for (int e = 0; e < V; ++e) bias[e] = skip[e] = y[e] = z[e] = 0.0f;
    unpack(load_pack<T, V>((const T*)a.u + s * a.ldu + d), u);
    unpack(load_pack<T, V>((const T*)a.dt + s * a.lddt + d), x);
    if (a.z) unpack(load_pack<T, V>((const T*)a.z + s * a.ldz + d), z);
    if (a.dt_bias) unpack(load_pack<float, V>(a.dt_bias + d), bias);
    if (a.skip) unpack(load_pack<float, V>(a.skip + d), skip);
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = delta_of(x[e], bias[e], a.softplus);
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        float hn[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            hn[e] = fmaf(exp2_hw(x[e] * rate2(aq[j].v[e])), hq[j].v[e], x[e] * u[e] * B[j]);
            if (n0 + j < a.N) y[e] = fmaf(C[j], hn[e], y[e]);
        }
        if (on && n0 + j < a.N) store_pack<float, V>(h + (int64_t)j * a.D, hn);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) ys[wave][lane * V + e] = y[e];
    __syncthreads();
    if (wave != 0 || !on) return;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int i = lane * V + e;
        y[e] = fmaf(skip[e], u[e], (ys[0][i] + ys[1][i]) + (ys[2][i] + ys[3][i]));
        if (a.z) y[e] *= z[e] * sigmoid(z[e]);
    }
    store_pack<T, V>((T*)a.y + s * a.ldy + d, y);
}

// ---------------------------------------------------------------- host

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

SeqMap map_of(const Rows& r, int piece)
{
    return SeqMap{r.cu, r.total, r.L, (int)std::max<int64_t>(1, ceil_div(r.L, piece)), r.n, piece};
}

template <typename F>
hipError_t type_dispatch(int type, F&& f)
{
    if (type == SEQ_F32) return f(float{});
    if (type == SEQ_BF16) return f(bf16{});
    return f(f16{});
}

template <typename F>
hipError_t states_dispatch(int N, F&& f)
{
    if (N <= 4) return f(std::integral_constant<int, 4>{});
    if (N <= 8) return f(std::integral_constant<int, 8>{});
    if (N <= 16) return f(std::integral_constant<int, 16>{});
    if (N <= 32) return f(std::integral_constant<int, 32>{});
    return f(std::integral_constant<int, 64>{});
}

// f(states per lane, groups of 16 states, how N fills them) of the kernels in
// rows.
template <typename F>
hipError_t rows_dispatch(int N, F&& f)
{
    auto cut = [&](auto nsl, auto ng) {
        constexpr int NSL = decltype(nsl)::value;
        if (N == 4 * NSL * decltype(ng)::value) return f(nsl, ng, std::integral_constant<int, kFull>{});
        if (N % NSL == 0) return f(nsl, ng, std::integral_constant<int, kWholeLanes>{});
        return f(nsl, ng, std::integral_constant<int, NSL == 1 ? kWholeLanes : kWithinLane>{});
    };
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I4 = std::integral_constant<int, 4>;
    if (N <= 4) return cut(I1{}, I1{});
    if (N <= 8) return cut(I2{}, I1{});
    if (N <= 16) return cut(I4{}, I1{});
    if (N <= 32) return cut(I4{}, I2{});
    return cut(I4{}, I4{});
}

template <int MODE>
hipError_t launch_rows(const ScanArgs& a, hipStream_t s)
{
    const SeqMap m = map_of(a.rows, a.piece);
    const dim3 grid((unsigned)scan_slots(a.rows, a.piece), (unsigned)ceil_div(a.D / a.G, kCB), (unsigned)a.G);
    return type_dispatch(a.type, [&](auto t) {
        return rows_dispatch(a.N, [&](auto nsl, auto ng, auto cut) {
            // only the forward pass sums over states
            hipLaunchKernelGGL((scan_rows_kernel<decltype(t), decltype(nsl)::value, decltype(ng)::value, MODE,
                                                 MODE == kForward ? decltype(cut)::value : kFull>), grid, dim3(256), 0, s, a, m);
            return hipGetLastError();
        });
    });
}

// The channel-per-lane kernels: four wavefronts per workgroup, each an item.
dim3 wave_grid(const ScanArgs& a, int64_t slots)
{
    return dim3((unsigned)ceil_div(slots * a.G * ceil_div(a.D / a.G, 64), 4));
}

}  // namespace

int64_t scan_slots(const Rows& r, int piece)
{
    return r.cu ? r.total / piece + r.n : r.n * std::max<int64_t>(1, ceil_div(r.L, piece));
}

// Pieces have at least kScanKeep rows; wavefronts of 64 lanes, four to a workgroup.
bool scan_fits(const Rows& r, int D, int G)
{
    return ceil_div(scan_slots(r, kScanKeep) * G * ceil_div(D / G, 64), 4) < (int64_t)1 << 24;
}

bool scan_one_piece(const Rows& r, int piece) { return (r.cu ? r.total : r.L) <= piece; }

// Whether the state and forward passes run in rows: where pieces between kept
// states, a channel per lane, give fewer than one wavefront per SIMD (1,024).
// [32 x ~65, 128] with 32 states: the three forward launches 31 us in rows, 52
// in 16-row pieces with a channel per lane.  16 states, training, forward and
// backward in us: with 256 such wavefronts 31 and 48 in rows against 59 and 61,
// with 512 46 and 72 against 60 and 81, with 1,024 75 and 120 against 65 and 117,
// with 2,048 124 and 207 against 86 and 194.
bool scan_in_rows(const Rows& r, int D, int G)
{
    return scan_slots(r, kScanKeep) * G * ceil_div(D / G, 64) < 1024;
}

// Whether the main passes join the pieces' states themselves: in rows, where a
// launch costs more than what they read again.  Forward and backward, in us,
// with joins of their own and so: [4, 250, 256], 16 states, 64 wavefronts (a
// channel per lane, as above), 16.1 and 25.4 against 13.7 and 22.5; [16 x ~130,
// 256], 204: 27.7 and 46.9 against 24.9 and 44.2; [64 x ~100, 256], 664: 52 and
// 92 both ways; [100, 100, 256] with 32 states, 800: 92 and 166 against 89 and
// 170.  With many pieces to a sequence each would read many: on average at most
// four slots, and no sequence of more than 64 pieces.
bool scan_joins(const Rows& r, int D, int G)
{
    const int64_t slots = scan_slots(r, kScanKeep), longest = (r.cu ? r.total : r.L) / kScanKeep;
    return slots * G * ceil_div(D / G, 64) < 512 && longest < 64 && slots <= 4 * (int64_t)r.n;
}

// Rows per piece: in rows, those between kept states; else a multiple of them.
// One wavefront carries 64 channels; about four per SIMD (4,096) keep its pipes
// busy, and pieces beyond that only add states to form and join (32-row pieces
// at [4, 2048, 1024]: the state passes 40 -> 37 us, the joins 8 -> 11).
int scan_piece(const Rows& r, int D, int G)
{
    const int64_t waves = (int64_t)G * ceil_div(D / G, 64), keep = kScanKeep;
    if (scan_in_rows(r, D, G)) return kScanKeep;
    const int64_t rows = std::max<int64_t>(1, ceil_div(r.total, ceil_div(4096, waves)));
    return (int)std::min<int64_t>(ceil_div(rows, keep) * keep, 1 << 20);
}

// Channels of a backward workgroup: as many as bring the grid down to the two
// workgroups that each CU holds (512), in rounds of 16; more channels mean fewer partial dB and dC.
int scan_bwd_chans(const Rows& r, int D, int G)
{
    const int64_t slots = scan_slots(r, kScanKeep);
    const int64_t rounds = slots * G * ceil_div(D / G, kCB);
    const int64_t per = std::max<int64_t>(1, std::min<int64_t>(ceil_div(rounds, 512), ceil_div(D / G, kCB)));
    return (int)(per * kCB);
}

hipError_t launch_scan_state(const ScanArgs& a, bool reverse, hipStream_t s)
{
    if (scan_in_rows(a.rows, a.D, a.G)) return reverse ? launch_rows<kStateRev>(a, s) : launch_rows<kStateFwd>(a, s);
    const SeqMap m = map_of(a.rows, a.piece);
    const int64_t slots = scan_slots(a.rows, a.piece);
    const dim3 grid = wave_grid(a, slots), block(256);
    return type_dispatch(a.type, [&](auto t) {
        return states_dispatch(a.N, [&](auto ns) {
            using T = decltype(t);
            constexpr int NS = decltype(ns)::value;
            if (reverse) hipLaunchKernelGGL((scan_state_kernel<T, NS, true>), grid, block, 0, s, a, m, (int)slots);
            else hipLaunchKernelGGL((scan_state_kernel<T, NS, false>), grid, block, 0, s, a, m, (int)slots);
            return hipGetLastError();
        });
    });
}

hipError_t launch_scan_join(const ScanArgs& a, bool reverse, hipStream_t s)
{
    const SeqMap m = map_of(a.rows, a.piece);
    const dim3 grid((unsigned)a.rows.n, (unsigned)ceil_div(a.D, 256), (unsigned)a.N);
    hipLaunchKernelGGL(scan_join_kernel, grid, dim3(256), 0, s, a, m, reverse ? 1 : 0);
    return hipGetLastError();
}

hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t s)
{
    if (scan_in_rows(a.rows, a.D, a.G)) return launch_rows<kForward>(a, s);
    const SeqMap m = map_of(a.rows, a.piece), keep = map_of(a.rows, kScanKeep);
    const int64_t slots = scan_slots(a.rows, a.piece);
    const dim3 grid = wave_grid(a, slots), block(256);
    return type_dispatch(a.type, [&](auto t) {
        return states_dispatch(a.N, [&](auto ns) {
            using T = decltype(t);
            constexpr int NS = decltype(ns)::value;
            if (a.N == NS) hipLaunchKernelGGL((scan_fwd_kernel<T, NS, true>), grid, block, 0, s, a, m, keep, (int)slots);
            else hipLaunchKernelGGL((scan_fwd_kernel<T, NS, false>), grid, block, 0, s, a, m, keep, (int)slots);
            return hipGetLastError();
        });
    });
}

hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t s)
{
    const SeqMap m = map_of(a.rows, kScanKeep);
    const dim3 grid((unsigned)scan_slots(a.rows, kScanKeep), (unsigned)scan_bwd_blocks(a.D, a.G, a.chans), (unsigned)a.G);
    auto run = [&](auto t, auto nsl, auto ng, auto join, auto cut) {
        constexpr auto kernel =
            scan_bwd_kernel<decltype(t), decltype(nsl)::value, decltype(ng)::value, decltype(join)::value, decltype(cut)::value>;
        constexpr int bytes = (int)sizeof(BwdLds<decltype(ng)::value>);
        if constexpr (bytes > 65536) {
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL(kernel, grid, dim3(256), bytes, s, a, m);
        return hipGetLastError();
    };
    return type_dispatch(a.type, [&](auto t) {
        return rows_dispatch(a.N, [&](auto nsl, auto ng, auto cut) {
            return a.join ? run(t, nsl, ng, std::true_type{}, cut) : run(t, nsl, ng, std::false_type{}, cut);
        });
    });
}

hipError_t launch_scan_step(const ScanStepArgs& a, hipStream_t s)
{
    const int Dg = a.D / a.G, V = Dg % 4 == 0 ? 4 : (Dg % 2 == 0 ? 2 : 1);
    const dim3 grid((unsigned)a.S, (unsigned)ceil_div(Dg, 64 * V), (unsigned)a.G);
    return type_dispatch(a.type, [&](auto t) {
        return states_dispatch(a.N, [&](auto ns) {
            using T = decltype(t);
            constexpr int NQ = decltype(ns)::value / 4;
            if (V == 4) hipLaunchKernelGGL((scan_step_kernel<T, NQ, 4>), grid, dim3(256), 0, s, a);
            else if (V == 2) hipLaunchKernelGGL((scan_step_kernel<T, NQ, 2>), grid, dim3(256), 0, s, a);
            else hipLaunchKernelGGL((scan_step_kernel<T, NQ, 1>), grid, dim3(256), 0, s, a);
            return hipGetLastError();
        });
    });
}

}  // namespace seq

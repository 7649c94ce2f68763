// Causal depthwise convolution over time, channels innermost: forward,
// backward and the single-token step.  Memory bound: a wavefront holds 64 V
// adjacent channels and walks the rows of one piece of a sequence with the
// last K - 1 inputs in registers, so each row is read once (the K - 1 rows
// before a piece twice).  [8, 2048, 2048] bf16, K = 4: forward 134 MB in 31 us,
// 4.3 TB/s; backward 201 MB in 43 us, 4.7 TB/s, with the vector ALU 59 % busy.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../../include/seq.h"
#include "seq_device.h"
#include "seq_kernels.h"

namespace seq {

namespace {

constexpr int kFwdRows = 16;   // rows of one wavefront's piece: all their loads are in flight together
constexpr int kBatch = 8;      // backward: rows whose loads are in flight while the batch before is computed

template <typename T, int V>
__device__ __forceinline__ void load_row(const T* p, float (&o)[V])
{
    unpack(load_pack<T, V>(p), o);
}

// The first of a lane's V channels.  A lane whose channels would pass D takes
// the last V: it computes what other lanes compute too, bit for bit, and stores
// the same values.  D >= V.
template <int V>
__device__ __forceinline__ int lane_channel(int at, int D)
{
    return min(at, D - V);
}

// win[j] = the input at row t - (K - 1) + j of the sequence; rows before its
// start come from the state (row -1 is the state's last).
template <typename T, int K, int V>
__device__ __forceinline__ void first_window(const ConvArgs& a, const Piece& p, int64_t t, int c, float (&win)[K][V])
{
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int64_t q = t - (K - 1) + j;
        if (q >= 0) {
            load_row<T, V>((const T*)a.x + (p.row + q) * a.ldx + c, win[j]);
        } else if (a.state_in) {
            load_row<T, V>((const T*)a.state_in + ((int64_t)p.s * (K - 1) + (K - 1 + q)) * a.D + c, win[j]);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) win[j][e] = 0.0f;
        }
    }
}

template <int K, int V>
__device__ __forceinline__ void load_taps(const float* taps, const float* bias, int c, float (&w)[K][V], float (&b)[V])
{
    float q[V * K];   // the taps of V adjacent channels lie together
    unpack(load_pack<float, V * K>(taps + (int64_t)c * K), q);
#pragma unroll
    for (int e = 0; e < V; ++e)
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][e] = q[e * K + k];
#pragma unroll
    for (int e = 0; e < V; ++e) b[e] = 0.0f;
    if (bias) unpack(load_pack<float, V>(bias + c), b);
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }

template <int K, int V>
__device__ __forceinline__ void shift(float (&win)[K][V])
{
#pragma unroll
    for (int j = 0; j + 1 < K; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) win[j][e] = win[j + 1][e];
}

template <typename T, int K, int V>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a, SeqMap m, int slots)
{
    const int slot = (int)(blockIdx.x / a.blocks) * 4 + wave_id();
    if (slot >= slots) return;
    const Piece p = seq_locate(m, slot);
    const int c = lane_channel<V>(((int)(blockIdx.x % a.blocks) * 64 + (int)(threadIdx.x & 63)) * V, a.D);
    if (!p.live) return;
    const int64_t t0 = p.index * kFwdRows;
    const int rows = (int)min((int64_t)kFwdRows, p.len - t0);
    const T* x = (const T*)a.x + (p.row + t0) * a.ldx;
    T* y = (T*)a.out + (p.row + t0) * a.ldo;
    Pack<T, V> q[kFwdRows];
    if (rows > 0) {
#pragma unroll
        for (int i = 0; i < kFwdRows; ++i)   // past the end: the last row again, unused
            q[i] = load_pack<T, V>(x + (int64_t)min(i, rows - 1) * a.ldx + c);
    }
    float w[K][V], b[V], win[K][V];
    load_taps<K, V>(a.w, a.b, c, w, b);
    first_window<T, K, V>(a, p, t0, c, win);
    auto walk = [&](auto full) {
#pragma unroll
        for (int i = 0; i < kFwdRows; ++i) {
            unpack(q[i], win[K - 1]);
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                o[e] = b[e];
#pragma unroll
                for (int k = 0; k < K; ++k) o[e] = fmaf(w[k][e], win[k][e], o[e]);
            }
            if (a.silu) {
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] *= sigmoid(o[e]);
            }
            if (decltype(full)::value || i < rows) store_pack<T, V>(y + (int64_t)i * a.ldo + c, o);
            shift<K, V>(win);
        }
    };
    if (rows == kFwdRows) walk(std::true_type{});
    else if (rows > 0) walk(std::false_type{});
    // the piece that ends the sequence keeps its last K - 1 inputs
    if (a.state_out && t0 + rows == p.len) {
        first_window<T, K, V>(a, p, p.len, c, win);
#pragma unroll
        for (int j = 0; j + 1 < K; ++j)
            store_pack<T, V>((T*)a.state_out + ((int64_t)p.s * (K - 1) + j) * a.D + c, win[j]);
    }
}

// Backward.  da_t = dy_t act'(a_t) with a_t formed again from x;
//   dx_t = sum_k w_k da_{t + K - 1 - k}:  da_t is added into the K pending
//   sums of rows t - K + 1 .. t, the oldest of which is then complete;
//   dw_k += da_t x_{t - K + 1 + k},  db += da_t  over the piece's own rows.
// The K - 1 rows after the piece are formed twice (by it and by the next).
// The workgroup's four wavefronts take four pieces of the same channels and
// add their dw and db through LDS: one partial row per workgroup.
template <typename T, int K, int V>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvArgs a, SeqMap m, int slots)
{
    __shared__ float comb[4][64 * V];
    const int wave = wave_id(), lane = (int)threadIdx.x & 63;
    const int slot = (int)(blockIdx.x / a.blocks) * 4 + wave;
    const int cblock = (int)(blockIdx.x % a.blocks), c = lane_channel<V>((cblock * 64 + lane) * V, a.D);
    float dw[K][V], db[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        db[e] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][e] = 0.0f;
    }
    Piece p{};
    if (slot < slots) p = seq_locate(m, slot);
    if (p.live && p.len > 0) {
        const int64_t t0 = p.index * m.piece;
        const int rows = (int)min((int64_t)m.piece, p.len - t0);
        const int all = (int)min((int64_t)rows + K - 1, p.len - t0);   // rows of da there are
        float w[K][V], b[V], win[K][V], acc[K][V];
        load_taps<K, V>(a.w, a.b, c, w, b);
        first_window<T, K, V>(a, p, t0, c, win);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[k][e] = 0.0f;
        const T* x = (const T*)a.x + (p.row + t0) * a.ldx;
        const T* dy = (const T*)a.dy + (p.row + t0) * a.lddy;
        T* dx = (T*)a.out + (p.row + t0) * a.ldo;
        Pack<T, V> nx[kBatch], ny[kBatch];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t r = min(i0 + i, all - 1);
                nx[i] = load_pack<T, V>(x + r * a.ldx + c);
                ny[i] = load_pack<T, V>(dy + r * a.lddy + c);
            }
        };
        // first: the batch that starts the piece; full: all its rows are the
        // piece's own.  Known at compile time, they leave no branch around a
        // store, and the loads in flight need not wait for stores.
        auto walk = [&](int i0, auto first, auto full) {
            Pack<T, V> qx[kBatch], qy[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) qx[i] = nx[i], qy[i] = ny[i];
            if (i0 + kBatch < rows + K - 1) fetch(i0 + kBatch);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int t = i0 + i;
                float g[V];
                unpack(qx[i], win[K - 1]);
                unpack(qy[i], g);
                if (a.silu) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float s = b[e];
#pragma unroll
                        for (int k = 0; k < K; ++k) s = fmaf(w[k][e], win[k][e], s);
                        const float sg = sigmoid(s);
                        g[e] *= sg * fmaf(s, 1.0f - sg, 1.0f);
                    }
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (!decltype(full)::value) g[e] = t < all ? g[e] : 0.0f;   // no da past the sequence's end
#pragma unroll
                    for (int k = 0; k + 1 < K; ++k) acc[k][e] = fmaf(w[k][e], g[e], acc[k + 1][e]);
                    acc[K - 1][e] = w[K - 1][e] * g[e];
                }
                if (!decltype(first)::value || i >= K - 1) {
                    if (decltype(full)::value || t < rows + K - 1)
                        store_pack<T, V>(dx + (int64_t)(t - (K - 1)) * a.ldo + c, acc[0]);
                }
                if (decltype(full)::value || t < rows) {   // the next piece counts the rest
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        db[e] += g[e];
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k][e] = fmaf(g[e], win[k][e], dw[k][e]);
                    }
                }
                shift<K, V>(win);
            }
        };
        fetch(0);
        if (rows >= kBatch) walk(0, std::true_type{}, std::true_type{});
        else walk(0, std::true_type{}, std::false_type{});
        int i0 = kBatch;
        for (; i0 + kBatch <= rows; i0 += kBatch) walk(i0, std::false_type{}, std::true_type{});
        for (; i0 < rows + K - 1; i0 += kBatch) walk(i0, std::false_type{}, std::false_type{});
    }
    float* part = a.part + (int64_t)(blockIdx.x / a.blocks) * a.D * (K + 1);
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) comb[wave][lane * V + e] = k < K ? dw[k < K ? k : 0][e] : db[e];
        __syncthreads();
        for (int i = (int)threadIdx.x; i < 64 * V; i += 256) {
            const int d = lane_channel<V>(cblock * 64 * V + i / V * V, a.D) + i % V;
            part[k < K ? (int64_t)d * K + k : (int64_t)a.D * K + d] =
                (comb[0][i] + comb[1][i]) + (comb[2][i] + comb[3][i]);
        }
    }
}

// One token per sequence: the state's K - 1 rows and the input in, the state
// moved on by one row and the output back.  Bound by a launch's latency (2 us
// for one sequence of 2048 channels, 4 us for 256).
template <typename T, int K, int V>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvStepArgs a)
{
    const int64_t s = blockIdx.x;
    const int at = ((int)blockIdx.y * 256 + (int)threadIdx.x) * V;
    if (at >= a.D) return;
    // the state is changed in place: a lane that shares channels with another
    // (the last, shifted back) leaves theirs alone
    const int c = lane_channel<V>(at, a.D), dup = at - c;
    T* st = (T*)a.state + s * (K - 1) * a.D + c;
    Pack<T, V> in[K];
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) in[j] = load_pack<T, V>(st + (int64_t)j * a.D);
    in[K - 1] = load_pack<T, V>((const T*)a.x + s * a.ldx + c);
    float x[K][V], w[K][V], o[V];
    load_taps<K, V>(a.w, a.b, c, w, o);
#pragma unroll
    for (int j = 0; j < K; ++j) unpack(in[j], x[j]);
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < K; ++k) o[e] = fmaf(w[k][e], x[k][e], o[e]);
        if (a.silu) o[e] *= sigmoid(o[e]);
    }
    T* y = (T*)a.y + s * a.ldy + c;
    if (dup == 0) {
        store_pack<T, V>(y, o);
#pragma unroll
        for (int j = 0; j + 1 < K; ++j) store_pack<T, V>(st + (int64_t)j * a.D, x[j + 1]);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e >= dup) {
                y[e] = (T)o[e];
#pragma unroll
                for (int j = 0; j + 1 < K; ++j) st[(int64_t)j * a.D + e] = in[j + 1].v[e];
            }
    }
}

SeqMap map_of(const Rows& r, int piece)
{
    return SeqMap{r.cu, r.total, r.L, (int)std::max<int64_t>(1, (r.L + piece - 1) / piece), r.n, piece};
}

int64_t slots_of(const Rows& r, int piece)
{
    return r.cu ? r.total / piece + r.n : r.n * std::max<int64_t>(1, (r.L + piece - 1) / piece);
}

// f(element type, K, V).  A lane takes two adjacent channels (one, where there is
// only one).  More a lane take registers from rows in flight: with four, 27 and
// 44 us at [8, 2048, 2048] bf16 and 6.5 and 28 at 256 channels, against 27 and
// 42, 6.0 and 21; with eight, 64 and 141 at 2048.
template <typename F>
hipError_t conv_dispatch(int type, int K, int vec, F&& f)
{
    auto by_k = [&](auto t, auto v) {
        if (K == 2) return f(t, std::integral_constant<int, 2>{}, v);
        if (K == 3) return f(t, std::integral_constant<int, 3>{}, v);
        return f(t, std::integral_constant<int, 4>{}, v);
    };
    auto by_v = [&](auto t) {
        return vec == 2 ? by_k(t, std::integral_constant<int, 2>{}) : by_k(t, std::integral_constant<int, 1>{});
    };
    if (type == SEQ_F32) return by_v(float{});
    if (type == SEQ_BF16) return by_v(bf16{});
    return by_v(f16{});
}

int vec_of(int D) { return D >= 2 ? 2 : 1; }

// Rows per piece of the backward pass.  A short piece forms its K - 1 following
// rows again for fewer of its own and leaves more partial gradients to add; a
// long one leaves the chip empty.  With pieces of 16, 32 and 64 rows (us):
// [8, 2048, 2048] bf16, 4,096 wavefronts of 64 rows: 55, 45, 43; [8, 2048, 512],
// 1,024: 23, 21, 23; [8, 2048, 256], 512: 17, 16, 21; [8, 2048, 128], 256: 14, 15,
// 20; [1, 64, 256]: 9, 11, 16.
int bwd_rows(const Rows& r, int D)
{
    const int64_t waves = r.total / 64 * ((D + 127) / 128);
    return waves >= 2048 ? 64 : (waves >= 384 ? 32 : 16);
}

}  // namespace

int64_t conv_bwd_parts(const Rows& r, int D) { return (slots_of(r, bwd_rows(r, D)) + 3) / 4; }

// The forward pass has the shortest pieces; workgroups of 256 lanes.
bool conv_fits(const Rows& r, int D)
{
    const int cols = 64 * vec_of(D);
    return (slots_of(r, kFwdRows) + 3) / 4 * ((D + cols - 1) / cols) < (int64_t)1 << 24;
}

hipError_t launch_conv_fwd(ConvArgs a, hipStream_t s)
{
    const int vec = vec_of(a.D);
    const int64_t slots = slots_of(a.rows, kFwdRows);
    const int cols = 64 * vec;
    // neighbouring workgroups take neighbouring channels: what runs at a time
    // covers whole rows (one block of channels over all rows first: 55 us
    // against 51, when each took that long)
    a.blocks = (unsigned)((a.D + cols - 1) / cols);
    const dim3 grid((unsigned)((slots + 3) / 4) * a.blocks);
    const SeqMap m = map_of(a.rows, kFwdRows);
    return conv_dispatch(a.type, a.K, vec, [&](auto t, auto k, auto v) {
        hipLaunchKernelGGL((conv_fwd_kernel<decltype(t), decltype(k)::value, decltype(v)::value>), grid, dim3(256), 0, s,
                           a, m, (int)slots);
        return hipGetLastError();
    });
}

hipError_t launch_conv_bwd(ConvArgs a, hipStream_t s)
{
    const int vec = vec_of(a.D);
    const int piece = bwd_rows(a.rows, a.D);
    const int64_t slots = slots_of(a.rows, piece);
    const int cols = 64 * vec;
    a.blocks = (unsigned)((a.D + cols - 1) / cols);
    const dim3 grid((unsigned)((slots + 3) / 4) * a.blocks);
    const SeqMap m = map_of(a.rows, piece);
    return conv_dispatch(a.type, a.K, vec, [&](auto t, auto k, auto v) {
        hipLaunchKernelGGL((conv_bwd_kernel<decltype(t), decltype(k)::value, decltype(v)::value>), grid, dim3(256), 0, s,
                           a, m, (int)slots);
        return hipGetLastError();
    });
}

hipError_t launch_conv_step(const ConvStepArgs& a, hipStream_t s)
{
    const int vec = vec_of(a.D);
    const int cols = 256 * vec;
    const dim3 grid((unsigned)a.S, (unsigned)((a.D + cols - 1) / cols));
    return conv_dispatch(a.type, a.K, vec, [&](auto t, auto k, auto v) {
        hipLaunchKernelGGL((conv_step_kernel<decltype(t), decltype(k)::value, decltype(v)::value>), grid, dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace seq

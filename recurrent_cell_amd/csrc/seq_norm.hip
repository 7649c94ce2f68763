// Layer norm (forward, backward with the weight gradient's partial sums),
// dropout from a counter-based generator, and the row sum that finishes
// per-workgroup partial gradients.  No atomics: every sum has an order fixed
// by the sizes.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../../include/seq.h"
#include "seq_device.h"
#include "seq_kernels.h"

namespace seq {

namespace {

// ---------------------------------------------------------------------------
// Layer norm.  A row is held in registers: NV vectors of V elements by each of
// the W lanes that share it (16 or 32 lanes, one wavefront, four or eight), so x
// is read once, and the variance is the mean square of the centred values (two
// passes over registers, no cancellation).  Workers walk the rows with a
// stride; where one has a next row (the grid stops at 4,096 workgroups: more than
// 16,384 rows of a wavefront each), its loads are issued before the present row's
// sums.  With a row per worker, as at [16384, 2048], the registers for it buy
// nothing.  w and b come from the caches (kept in registers they cost half the
// wavefronts per SIMD: 44 us against 31 at [16384, 2048] bf16).  Bound by memory:
// 134 MB in 31 us, 4.3 TB/s; short rows by latency ([2048, 128] f32: 3 us).
// ---------------------------------------------------------------------------
template <int W>
__device__ __forceinline__ float worker_sum(float x, float (*red)[W >= 64 ? W / 64 : 1], int& turn)
{
    x = row_sum(x);
    if constexpr (W >= 32) x = pair_sum16(x, x);
    if constexpr (W >= 64) x = pair_sum32(x, x);
    if constexpr (W > 64) {
        // two buffers in turn: a wave can be at most one sum ahead of another
        const int wv = (int)threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) red[turn][wv] = x;
        __syncthreads();
        x = 0.0f;
#pragma unroll
        for (int i = 0; i < W / 64; ++i) x += red[turn][i];
        turn ^= 1;
    }
    return x;
}

template <int W>
constexpr int kLnThreads = W <= 256 ? 256 : W;

// The lane's vector v of a row: whole vectors throughout.  A vector that would
// pass the row's end is shifted back to end with it; its first `dup` elements
// then belong to other lanes (all of them, where the lane has none of its own):
// they are left out of the row's sums, and otherwise computed alike, bit for
// bit.  C >= V.
template <int W, int V>
struct LnCol {
    int c, dup;
    __device__ __forceinline__ LnCol(int v, int lane, int C)
    {
        const int at = (v * W + lane) * V;
        c = min(at, C - V);
        dup = min(at - c, V);
    }
};

template <typename T, int V, int W, int NV>
__global__ __launch_bounds__(kLnThreads<W>) void ln_fwd_kernel(LnArgs a)
{
    constexpr int PER = kLnThreads<W> / W;
    using Col = LnCol<W, V>;
    __shared__ float red[2][W >= 64 ? W / 64 : 1];
    int turn = 0;
    const int lane = (int)threadIdx.x % W;
    const int64_t step = (int64_t)gridDim.x * PER;
    int64_t r = (int64_t)blockIdx.x * PER + (int)threadIdx.x / W;
    const float invC = 1.0f / (float)a.C;
    Pack<T, V> nx[NV];
    auto fetch = [&](int64_t row) {
        const T* p = (const T*)a.x + row * a.ldx;
#pragma unroll
        for (int v = 0; v < NV; ++v) nx[v] = load_pack<T, V>(p + Col(v, lane, a.C).c);
    };
    if (r < a.rows) fetch(r);
    for (; r < a.rows; r += step) {
        float x[NV][V];
#pragma unroll
        for (int v = 0; v < NV; ++v) unpack(nx[v], x[v]);
        if (r + step < a.rows) fetch(r + step);
        float t = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int dup = Col(v, lane, a.C).dup;
#pragma unroll
            for (int e = 0; e < V; ++e) t += e >= dup ? x[v][e] : 0.0f;
        }
        const float mean = worker_sum<W>(t, red, turn) * invC;
        t = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int dup = Col(v, lane, a.C).dup;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                x[v][e] -= mean;
                const float q = e >= dup ? x[v][e] : 0.0f;
                t = fmaf(q, q, t);
            }
        }
        const float rstd = 1.0f / sqrtf(fmaf(worker_sum<W>(t, red, turn), invC, a.eps));
        if (lane == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
        T* q = (T*)a.out + r * a.ldo;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const Col k(v, lane, a.C);
            float w[V], b[V];
#pragma unroll
            for (int e = 0; e < V; ++e) w[e] = 1.0f, b[e] = 0.0f;
            if (a.w) unpack(load_pack<float, V>(a.w + k.c), w);
            if (a.b) unpack(load_pack<float, V>(a.b + k.c), b);
#pragma unroll
            for (int e = 0; e < V; ++e) x[v][e] = fmaf(x[v][e] * rstd, w[e], b[e]);
            if (k.dup < V) store_pack<T, V>(q + k.c, x[v]);
        }
    }
}

// Backward: xh = (x - mean) rstd, g = dy w,
//   dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum dy xh,  db = sum dy.
// One pass over x and dy.  A thread sums dw and db of its columns over the
// rows it meets; the workgroup's 512 / W workers (W <= 64) add theirs through
// LDS, and each workgroup writes one partial row [2][C], summed by
// sum_rows_kernel.  Bound by memory: [16384, 2048] bf16, 201 MB in 37 us, 5.4 TB/s
// (part of the operands lies in the cache); [2048, 128] f32 4 us.
template <int W>
constexpr int kLnBwdThreads = W == 256 ? 256 : 512;

template <typename T, int V, int W, int NV>
__global__ __launch_bounds__(kLnBwdThreads<W>) void ln_bwd_kernel(LnArgs a)
{
    constexpr int PER = kLnBwdThreads<W> / W;
    using Col = LnCol<W, V>;
    __shared__ float red[2][W >= 64 ? W / 64 : 1];
    __shared__ float comb[PER > 1 ? PER : 1][PER > 1 ? W * V : 1];
    int turn = 0;
    const int lane = (int)threadIdx.x % W, worker = (int)threadIdx.x / W;
    const int64_t step = (int64_t)gridDim.x * PER;
    int64_t r = (int64_t)blockIdx.x * PER + worker;
    float dw[NV][V], db[NV][V];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < V; ++e) dw[v][e] = db[v][e] = 0.0f;
    const float invC = 1.0f / (float)a.C;
    Pack<T, V> nx[NV], ny[NV];
    float nmean = 0.0f, nrstd = 0.0f;
    auto fetch = [&](int64_t row) {
        const T* p = (const T*)a.x + row * a.ldx;
        const T* q = (const T*)a.dy + row * a.lddy;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = Col(v, lane, a.C).c;
            nx[v] = load_pack<T, V>(p + c);
            ny[v] = load_pack<T, V>(q + c);
        }
        nmean = a.mean[row];
        nrstd = a.rstd[row];
    };
    // with eight vectors a lane the next row's would not fit beside the present's
    constexpr bool kAhead = NV < 8;
    if (kAhead && r < a.rows) fetch(r);
    for (; r < a.rows; r += step) {
        if (!kAhead) fetch(r);
        float x[NV][V], g[NV][V];
        const float mean = nmean, rstd = nrstd;
        float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const Col k(v, lane, a.C);
            float w[V];
#pragma unroll
            for (int e = 0; e < V; ++e) w[e] = 1.0f;
            if (a.w) unpack(load_pack<float, V>(a.w + k.c), w);
            unpack(nx[v], x[v]);
            unpack(ny[v], g[v]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                x[v][e] = (x[v][e] - mean) * rstd;
                dw[v][e] = fmaf(g[v][e], x[v][e], dw[v][e]);
                db[v][e] += g[v][e];
                g[v][e] *= w[e];
                const float own = e >= k.dup ? g[v][e] : 0.0f;
                t1 += own;
                t2 = fmaf(own, x[v][e], t2);
            }
        }
        if (kAhead && r + step < a.rows) fetch(r + step);
        t1 = worker_sum<W>(t1, red, turn) * invC;
        t2 = worker_sum<W>(t2, red, turn) * invC;
        T* q = (T*)a.out + r * a.ldo;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const Col k(v, lane, a.C);
#pragma unroll
            for (int e = 0; e < V; ++e) g[v][e] = rstd * (g[v][e] - t1 - x[v][e] * t2);
            if (k.dup < V) store_pack<T, V>(q + k.c, g[v]);
        }
    }
    if (!a.part) return;
    float* p = a.part + (int64_t)blockIdx.x * 2 * a.C;
    if constexpr (PER == 1) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const Col k(v, lane, a.C);
            if (k.dup < V) {
                store_pack<float, V>(p + k.c, dw[v]);
                store_pack<float, V>(p + a.C + k.c, db[v]);
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < V; ++e) comb[worker][lane * V + e] = k ? db[v][e] : dw[v][e];
                __syncthreads();
                for (int i = (int)threadIdx.x; i < W * V; i += kLnBwdThreads<W>) {
                    const Col q(v, i / V, a.C);
                    float t = 0.0f;
#pragma unroll
                    for (int j = 0; j < PER; ++j) t += comb[j][i];
                    if (q.dup < V) p[k * a.C + q.c + i % V] = t;
                }
            }
    }
}

// The narrowest worker that holds the row, with at most four vectors a lane up
// to four wavefronts: fewer lanes per row mean fewer exchanges per sum, and of a
// short row fewer idle lanes ([65536, 64] bf16: 7.5 us with 16 lanes, 18 with a
// wavefront); eight wavefronts rather than sixteen leave a lane the registers
// for its sums ([2048, 16384] f32 backward: 70 us against 167, spilled).
struct LnShape {
    int W, nv;
};

LnShape ln_shape(int C, int type)
{
    const int V = type == SEQ_F32 ? 4 : 8;
    if (C <= 16 * V) return {16, 1};
    if (C <= 32 * V) return {32, 1};
    for (int nv = 1; nv <= 4; nv *= 2)
        if (C <= 64 * V * nv) return {64, nv};
    for (int nv = 2; nv <= 4; nv *= 2)
        if (C <= 256 * V * nv) return {256, nv};
    return {512, C <= 512 * V * 4 ? 4 : 8};
}

// Calls f with V, W and NV as compile-time constants; rows shorter than a vector
// go element by element.
template <typename T, typename F>
hipError_t ln_dispatch(int C, int type, F&& f)
{
    using std::integral_constant;
    using V = integral_constant<int, kVec<T>>;
    const LnShape s = ln_shape(C, type);
    if (C < kVec<T>) return f(integral_constant<int, 1>{}, integral_constant<int, 16>{}, integral_constant<int, 1>{});
    if (s.W == 16) return f(V{}, integral_constant<int, 16>{}, integral_constant<int, 1>{});
    if (s.W == 32) return f(V{}, integral_constant<int, 32>{}, integral_constant<int, 1>{});
    if (s.W == 64 && s.nv == 1) return f(V{}, integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (s.W == 64 && s.nv == 2) return f(V{}, integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (s.W == 64) return f(V{}, integral_constant<int, 64>{}, integral_constant<int, 4>{});
    if (s.W == 256 && s.nv == 2) return f(V{}, integral_constant<int, 256>{}, integral_constant<int, 2>{});
    if (s.W == 256) return f(V{}, integral_constant<int, 256>{}, integral_constant<int, 4>{});
    // 16-bit rows of at most SEQ_MAX_C need no more than four vectors
    if (s.nv == 4 || sizeof(T) == 2) return f(V{}, integral_constant<int, 512>{}, integral_constant<int, 4>{});
    return f(V{}, integral_constant<int, 512>{}, integral_constant<int, sizeof(T) == 2 ? 4 : 8>{});
}

template <typename F>
hipError_t type_dispatch(int type, F&& f)
{
    if (type == SEQ_F32) return f(float{});
    if (type == SEQ_BF16) return f(bf16{});
    return f(f16{});
}

// ---------------------------------------------------------------------------
// Row sums of per-workgroup partials.  A workgroup is RS row slices x (256 /
// RS) lanes of 4 adjacent columns; slice i sums its contiguous rows in
// ascending order in fp64, the slices are added in order through LDS.  RS
// depends on R alone.  Bound by latency: 256 rows of [2, 2048] 6 us, the five
// tensors of a scan's backward pass 5 us.
// ---------------------------------------------------------------------------
__host__ __device__ inline int sum_slices(int64_t R) { return R >= 128 ? 32 : (R >= 16 ? 8 : 1); }

template <int RS>
__device__ __forceinline__ void sum_seg(const SumSeg& g, double (*part)[4])
{
    constexpr int LANES = 256 / RS;
    const int slice = (int)threadIdx.x / LANES, lane = (int)threadIdx.x % LANES;
    const int64_t c = ((int64_t)(blockIdx.x - g.block0) * LANES + lane) * 4;
    const int64_t per = (g.R + RS - 1) / RS;
    const int64_t rb = slice * per, re = min(rb + per, g.R);
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    const int n = (int)min(g.N - c, (int64_t)4);
    if (n > 0) {
        const float* p = g.in + rb * g.stride + c;
        int64_t r = rb;
        for (; r + 8 <= re; r += 8, p += 8 * g.stride) {
            float v[8][4];
#pragma unroll
            for (int k = 0; k < 8; ++k) unpack(load_some<float, 4>(p + k * g.stride, n), v[k]);
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] += (double)v[k][e];
        }
        for (; r < re; ++r, p += g.stride) {
            float v[4];
            unpack(load_some<float, 4>(p, n), v);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] += (double)v[e];
        }
    }
    if constexpr (RS > 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) part[threadIdx.x][e] = acc[e];
        __syncthreads();
        if (slice == 0) {
#pragma unroll
            for (int i = 1; i < RS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] += part[i * LANES + lane][e];
        }
    }
    if (slice == 0 && n > 0) {
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = (float)acc[e];
        if (g.type == SEQ_F32) store_some<float, 4>((float*)g.out + c, o, n);
        else if (g.type == SEQ_BF16) store_some<bf16, 4>((bf16*)g.out + c, o, n);
        else store_some<f16, 4>((f16*)g.out + c, o, n);
    }
}

__global__ __launch_bounds__(256) void sum_rows_kernel(SumArgs a)
{
    __shared__ double part[256][4];
    int k = 0;
#pragma unroll
    for (int i = 1; i < kMaxSumSegs; ++i)
        if (i < a.nseg && (int64_t)blockIdx.x >= a.seg[i].block0) k = i;
    const SumSeg g = a.seg[k];
    const int rs = sum_slices(g.R);
    if (rs == 32) sum_seg<32>(g, part);
    else if (rs == 8) sum_seg<8>(g, part);
    else sum_seg<1>(g, part);
}

// ---------------------------------------------------------------------------
// Dropout.  Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as
// 1, 2, 3", 2011): counter (offset + i / 4, 0), key = seed; element i takes
// word i mod 4, i its place in the row-major [rows, C] whatever the strides.
// Forward and backward form the same words, so no mask is stored.  A dropped
// element gives 0 (or the residual) even where x is not finite.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void philox4(uint64_t ctr, uint64_t key, uint32_t (&o)[4])
{
    uint32_t c0 = (uint32_t)ctr, c1 = (uint32_t)(ctr >> 32), c2 = 0, c3 = 0;
    uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)p1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    o[0] = c0, o[1] = c1, o[2] = c2, o[3] = c3;
}

constexpr int kDropElems = 8;   // per thread, dense tensors

// Dense rows: one flat run of elements.  Bound by memory; two generator calls
// per eight elements keep the vector ALU 47 % busy: [16384, 2048] bf16 with a
// residual, 201 MB in 37 us, 5.4 TB/s.
template <typename T, bool RES>
__global__ __launch_bounds__(256) void dropout_kernel(DropArgs a)
{
    const int64_t total = a.rows * a.C;
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * kDropElems;
    if (i >= total) return;
    const int n = (int)min(total - i, (int64_t)kDropElems);
    float x[kDropElems], r[kDropElems];
    unpack(load_some<T, kDropElems>((const T*)a.x + i, n), x);
    if (RES) unpack(load_some<T, kDropElems>((const T*)a.r + i, n), r);
#pragma unroll
    for (int h = 0; h < kDropElems / 4; ++h) {
        uint32_t u[4];
        philox4(a.offset + (uint64_t)(i / 4 + h), a.seed, u);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float k = u[e] >= a.threshold ? x[4 * h + e] * a.scale : 0.0f;
            x[4 * h + e] = RES ? r[4 * h + e] + k : k;
        }
    }
    store_some<T, kDropElems>((T*)a.y + i, x, n);
}

// Rows with strides of their own: four elements of the flat order per thread,
// each at its row and column.
template <typename T, bool RES>
__global__ __launch_bounds__(256) void dropout_strided_kernel(DropArgs a)
{
    const int64_t total = a.rows * a.C;
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= total) return;
    uint32_t u[4];
    philox4(a.offset + (uint64_t)(i / 4), a.seed, u);
    int64_t row = i / a.C, c = i - row * a.C;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (i + e >= total) break;
        const float x = to_f<T>(((const T*)a.x)[row * a.ldx + c]);
        float k = u[e] >= a.threshold ? x * a.scale : 0.0f;
        if (RES) k = to_f<T>(((const T*)a.r)[row * a.ldr + c]) + k;
        ((T*)a.y)[row * a.ldy + c] = (T)k;
        if (++c == a.C) c = 0, ++row;
    }
}

}  // namespace

// Workgroups of the backward pass, one partial row each: a function of the
// sizes alone.
int ln_bwd_parts(int64_t rows, int C, int type)
{
    const int W = ln_shape(C, type).W;
    const int64_t per = W <= 64 ? 512 / W : 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, W == 256 ? 512 : 256));
}

hipError_t launch_ln_fwd(const LnArgs& a, hipStream_t s)
{
    return type_dispatch(a.type, [&](auto t) {
        using T = decltype(t);
        return ln_dispatch<T>(a.C, a.type, [&](auto v, auto w, auto nv) {
            constexpr int V = decltype(v)::value, W = decltype(w)::value, NV = decltype(nv)::value;
            constexpr int64_t per = kLnThreads<W> / W;
            const dim3 grid((unsigned)std::min<int64_t>((a.rows + per - 1) / per, 4096));
            hipLaunchKernelGGL((ln_fwd_kernel<T, V, W, NV>), grid, dim3(kLnThreads<W>), 0, s, a);
            return hipGetLastError();
        });
    });
}

hipError_t launch_ln_bwd(const LnArgs& a, hipStream_t s)
{
    return type_dispatch(a.type, [&](auto t) {
        using T = decltype(t);
        return ln_dispatch<T>(a.C, a.type, [&](auto v, auto w, auto nv) {
            constexpr int V = decltype(v)::value, W = decltype(w)::value, NV = decltype(nv)::value;
            hipLaunchKernelGGL((ln_bwd_kernel<T, V, W, NV>), dim3((unsigned)a.parts), dim3(kLnBwdThreads<W>), 0, s, a);
            return hipGetLastError();
        });
    });
}

// Workgroups of the row sum of an R x N segment.
int64_t sum_rows_blocks(int64_t R, int64_t N)
{
    const int64_t cols = 256 / sum_slices(R) * 4;
    return (N + cols - 1) / cols;
}

hipError_t launch_sum_rows(SumArgs a, hipStream_t s)
{
    int64_t blocks = 0;
    int n = 0;
    for (int i = 0; i < a.nseg; ++i) {
        SumSeg g = a.seg[i];
        if (g.N <= 0 || !g.out) continue;
        g.block0 = blocks;
        blocks += sum_rows_blocks(g.R, g.N);
        a.seg[n++] = g;
    }
    a.nseg = n;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(sum_rows_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_dropout(const DropArgs& a, hipStream_t s)
{
    const int64_t total = a.rows * a.C;
    const bool dense = a.rows <= 1 || (a.ldx == a.C && a.ldy == a.C && (!a.r || a.ldr == a.C));
    const int per = 256 * (dense ? kDropElems : 4);
    const unsigned grid = (unsigned)((total + per - 1) / per);
    return type_dispatch(a.type, [&](auto t) {
        using T = decltype(t);
        if (dense && a.r) hipLaunchKernelGGL((dropout_kernel<T, true>), dim3(grid), dim3(256), 0, s, a);
        else if (dense) hipLaunchKernelGGL((dropout_kernel<T, false>), dim3(grid), dim3(256), 0, s, a);
        else if (a.r) hipLaunchKernelGGL((dropout_strided_kernel<T, true>), dim3(grid), dim3(256), 0, s, a);
        else hipLaunchKernelGGL((dropout_strided_kernel<T, false>), dim3(grid), dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace seq

// Device helpers shared by the sequence-block kernels: element types, vector
// moves at element alignment, wavefront sums, the elementary functions, and
// the map from a workgroup's slot to its piece of a sequence.
//
// Activations are fp32, bf16 or fp16 (one type per call); everything is
// computed in fp32 and rounded to the activation type once, when stored.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace seq {

using bf16 = __bf16;
using f16 = _Float16;

// Elements of one 16-byte move.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

template <typename T>
__device__ __forceinline__ float to_f(T v)
{
    return (float)v;
}
template <>
__device__ __forceinline__ float to_f<bf16>(bf16 v)
{
    return __builtin_bit_cast(float, (uint32_t)__builtin_bit_cast(uint16_t, v) << 16);
}

// V elements moved as words of 16, 8, 4 or 2 bytes at the element's alignment:
// the hardware serves a misaligned wide access, so odd row lengths and views
// take the same moves as aligned ones.  (The words are vector types: an array's
// elements would be split up and merged with the moves of a row's tail.)
template <typename T, int V>
struct Pack {
    T v[V];
};

using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using u32x2 = uint32_t __attribute__((ext_vector_type(2)));

template <int BYTES>
struct Word;
template <>
struct Word<16> {
    using type = u32x4;
};
template <>
struct Word<8> {
    using type = u32x2;
};
template <>
struct Word<4> {
    using type = uint32_t;
};
template <>
struct Word<2> {
    using type = uint16_t;
};

constexpr int word_bytes(int left) { return left >= 16 ? 16 : left >= 8 ? 8 : left >= 4 ? 4 : 2; }

template <typename T, int V, int I = 0>
__device__ __forceinline__ void load_words(const T* p, Pack<T, V>& r)
{
    if constexpr (I < V) {
        constexpr int B = word_bytes((V - I) * (int)sizeof(T)), N = B / (int)sizeof(T);
        using W = typename Word<B>::type;
        typedef W WA __attribute__((aligned(sizeof(T))));
        const W w = *reinterpret_cast<const WA*>(p + I);
        const Pack<T, N> q = __builtin_bit_cast(Pack<T, N>, w);
#pragma unroll
        for (int i = 0; i < N; ++i) r.v[I + i] = q.v[i];
        load_words<T, V, I + N>(p, r);
    }
}

template <typename T, int V, int I = 0>
__device__ __forceinline__ void store_words(T* p, const Pack<T, V>& r)
{
    if constexpr (I < V) {
        constexpr int B = word_bytes((V - I) * (int)sizeof(T)), N = B / (int)sizeof(T);
        using W = typename Word<B>::type;
        typedef W WA __attribute__((aligned(sizeof(T))));
        Pack<T, N> q;
#pragma unroll
        for (int i = 0; i < N; ++i) q.v[i] = r.v[I + i];
        *reinterpret_cast<WA*>(p + I) = __builtin_bit_cast(W, q);
        store_words<T, V, I + N>(p, r);
    }
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p)
{
    Pack<T, V> r;
    load_words<T, V>(p, r);
    return r;
}

// The first n of V elements (n <= 0: none), zeros beyond; reads nothing past
// the n-th.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_some(const T* p, int n)
{
    Pack<T, V> r;
    if (n >= V) {
        load_words<T, V>(p, r);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) r.v[i] = i < n ? p[i] : (T)0.0f;
    }
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V>& q, float (&o)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = to_f<T>(q.v[i]);
}

template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const float (&x)[V])
{
    Pack<T, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) q.v[i] = (T)x[i];
    store_words<T, V>(p, q);
}

template <typename T, int V>
__device__ __forceinline__ void store_some(T* p, const float (&x)[V], int n)
{
    Pack<T, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) q.v[i] = (T)x[i];
    if (n >= V) {
        store_words<T, V>(p, q);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i] = q.v[i];
    }
}

// ---------------------------------------------------------------- wavefront

template <int CTRL>
__device__ __forceinline__ float dpp0(float x)   // lanes without a source read 0
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

constexpr int kRowShl(int n) { return 0x100 + n; }   // lane i reads lane i + n of its row of 16
constexpr int kRowShr(int n) { return 0x110 + n; }   // lane i reads lane i - n
constexpr int kRowRor(int n) { return 0x120 + n; }

// Sum over the 16 lanes of a row, in every lane of the row.
__device__ __forceinline__ float row_sum(float x)
{
    x += dpp0<kRowRor(8)>(x);
    x += dpp0<kRowRor(4)>(x);
    x += dpp0<kRowRor(2)>(x);
    x += dpp0<kRowRor(1)>(x);
    return x;
}

// (x, y) -> lower half of the wavefront: x summed with its upper half; upper
// half: y summed with its lower half.
__device__ __forceinline__ float pair_sum32(float x, float y)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y),
                                                    false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The same within each half: even rows of 16 hold x's sum, odd rows y's.
__device__ __forceinline__ float pair_sum16(float x, float y)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y),
                                                    false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum over the wavefront, in every lane; a fixed tree.
__device__ __forceinline__ float wave_sum(float x)
{
    x = row_sum(x);
    x = pair_sum16(x, x);
    return pair_sum32(x, x);
}

// Barrier for LDS traffic only: global loads and stores stay in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// ---------------------------------------------------------------- functions

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

// exp(-|x|): the product with log2(e) is rounded once, so the relative error is
// |x| 2^-24 and one rounding more.
__device__ __forceinline__ float exp_neg_abs(float x) { return exp2_hw(fabsf(x) * -kLog2e); }

// log(1 + exp(x)) = max(x, 0) + log1p(e), e = exp_neg_abs(x); log1p by the log of the rounded sum
// corrected by e / (rounded sum - 1), which keeps small e exact.  The max is a
// select: 0 at x = -inf (a row whose step is masked), and NaN comes through.
__device__ __forceinline__ float softplus_e(float x, float e)
{
    const float w = 1.0f + e, d = w - 1.0f;
    const float l = d == 0.0f ? e : __builtin_amdgcn_logf(w) * kLn2 * (e * rcp_hw(d));
    return (x < 0.0f ? 0.0f : x) + l;
}

// 1 / (1 + exp(-x)): the product with log2(e) is rounded once, so for negative x
// the relative error is |x| 2^-24 and two roundings more.
// The same from e = exp_neg_abs(x).
__device__ __forceinline__ float sigmoid_e(float x, float e)
{
    const float r = rcp_hw(1.0f + e);
    return x < 0.0f ? e * r : r;
}

__device__ __forceinline__ float sigmoid(float x) { return rcp_hw(1.0f + exp2_hw(x * -kLog2e)); }

// ---------------------------------------------------------------- sequences

// Rows are numbered over all sequences.  Without cu, sequence s is rows
// [s L, (s + 1) L); with it, rows [cu[s], cu[s + 1]).  Sequences are cut into
// pieces of `piece` rows, numbered by slots: nch slots per sequence without
// cu; with it sequence s starts at slot cu[s] / piece + s, which leaves room
// for every piece (and, here and there, a slot that holds none).  A sequence
// without rows has one (empty) slot.
struct SeqMap {
    const int* cu;     // [n + 1] on the device, or NULL
    int64_t total;     // rows
    int64_t L;         // rows per sequence without cu
    int nch;           // pieces per sequence without cu
    int n;             // sequences
    int piece;
};

struct Piece {
    int64_t row;     // first row of the sequence
    int64_t len;     // rows of the sequence
    int slot0;       // its first slot
    int64_t index;   // this piece's number in the sequence
    int s;
    bool live;       // the slot holds a piece
};

// What cu holds is not known to the host: every value is brought into
// [0, total], so no row outside the buffers is touched whatever it is.
__device__ __forceinline__ int64_t seq_start(const SeqMap& m, int s)
{
    if (!m.cu) return (int64_t)s * m.L;
    const int64_t v = m.cu[s];
    return v < 0 ? 0 : (v > m.total ? m.total : v);
}

// Slots are fewer than 2^31: a piece has at least 16 of at most 2^28 rows, and
// there are at most 2^20 sequences.
__device__ __forceinline__ int seq_slot0(const SeqMap& m, int s, int64_t start)
{
    return m.cu ? (int)((unsigned)start / (unsigned)m.piece) + s : s * m.nch;
}

__device__ __forceinline__ Piece seq_piece_of(const SeqMap& m, int s)
{
    Piece p;
    p.s = s;
    p.row = seq_start(m, s);
    const int64_t end = m.cu ? seq_start(m, s + 1) : p.row + m.L;
    p.len = end > p.row ? end - p.row : 0;
    p.slot0 = seq_slot0(m, s, p.row);
    p.index = 0;
    p.live = true;
    return p;
}

// The piece of a slot.  Called by whole wavefronts: with cu the sequence is
// found by a 64-way search, each lane looking at one candidate per level; with
// fewer than 64 sequences one load does, lane s holding cu[s].  Row numbers fit
// 32 bits; the result is the same in every lane, and said to be.
__device__ __forceinline__ Piece seq_locate(const SeqMap& m, int slot)
{
    int s, row, end;
    if (!m.cu) {
        s = (int)((unsigned)slot / (unsigned)m.nch);
        row = (int)(s * m.L);
        end = row + (int)m.L;
    } else {
        const int lane = (int)(threadIdx.x & 63);
        if (m.n < 64) {
            const int v = (int)seq_start(m, min(lane, m.n));
            const unsigned long long b = __ballot(lane < m.n && seq_slot0(m, lane, v) <= slot);
            s = b ? 63 - __clzll(b) : 0;
            row = __builtin_amdgcn_readlane(v, s);
            end = __builtin_amdgcn_readlane(v, s + 1);
        } else {
            int lo = 0, n = m.n;   // the last s in [lo, lo + n) whose first slot is <= slot
            while (n > 1) {
                const int step = (n + 63) / 64;
                const int c = lo + lane * step;
                const bool ok = c < lo + n && seq_slot0(m, c, seq_start(m, c)) <= slot;
                const unsigned long long b = __ballot(ok);
                const int k = b ? 63 - __clzll(b) : 0;
                const int nlo = lo + k * step;
                const int left = lo + n - nlo;
                n = left < step ? left : step;
                lo = nlo;
                n = n < 1 ? 1 : n;
            }
            s = __builtin_amdgcn_readfirstlane(lo);
            row = (int)seq_start(m, s);
            end = (int)seq_start(m, s + 1);
        }
        row = __builtin_amdgcn_readfirstlane(row);
        end = __builtin_amdgcn_readfirstlane(end);
    }
    Piece p;
    p.s = s;
    p.row = row;
    p.len = end > row ? end - row : 0;
    p.slot0 = seq_slot0(m, s, row);
    p.index = slot - p.slot0;
    p.live = p.index >= 0 && (p.index == 0 || p.index * m.piece < p.len);
    return p;
}

}  // namespace seq

// glr.hip -- the gated linear recurrence: one number of state per channel, with a gate on the decay and one on
// the input.
//
//   s = sigmoid(r + r_bias),  g = sigmoid(i + i_bias),  a = exp(s A)          (A <= 0)
//   h_t = a_t h_{t-1} + m_t g_t x_t,  m = sqrt(1 - a^2),  y_t = h_t
//
// and backward, from gy and the state after the row's last token:
//   lam_t = gy_t + a_{t+1} lam_{t+1}
//   dx = lam m g,  di = lam m x g (1 - g),  dl = lam (a h_{t-1} - g x a^2 / m),  dr = dl A s (1 - s)
//   dA = sum dl s,  dr_bias = sum dr,  di_bias = sum di
// (where m is 0 the second part of dl is taken as 0; a subnormal 1 - a^2, below 2^-126, counts as 0 for both).
//
// A stretch of tokens maps the state h that enters it to A h + H (A the product of its decays, H what it gathers from a
// zero state), and two stretches after one another compose: A = A1 A2, H = A2 H1 + H2.  A tile is kWaves stretches, one a
// wave, of some tokens by 128 channels; every lane keeps the decays and inputs of its two channels in registers, so that
// the tokens are read once.  A tile's waves join in LDS; tiles join through the workspace in the same launch: each
// publishes its (A, H), composes those before it in its group of 8 with the state that enters the group, and the group's
// last tile publishes the state that leaves it.  A document's start cuts: what was before is dropped, NaN included.  Tokens
// behind a row's length are decays of 1.  Both are chosen, not multiplied, so what stands there is not used.
//
// Every wait ends: a workgroup takes its place in the chain from a counter when it starts, so all places before its own
// belong to workgroups that have started, and these wait only for places before theirs.  A published pair is one 64-bit
// word with its own mark of validity, written and read by single relaxed atomics of device scope: no other memory is
// ordered by it.  What is composed, and in which order, does not depend on the timing: results are deterministic.
//
// Bound.  The forward cannot do without 4 activations an element, the backward without 7; a copy runs at 5.2 TB/s.  In bf16
// the gates' arithmetic (six transcendentals and some 27 other instructions an element and pass) and a tile's latencies (its
// place, its loads, the tiles before it) take about as long as the bytes, and two workgroups a CU overlap them.
// Measured (B x L x D):
//   forward, bf16, 1 x 65536 x 2048: 236 us, 4.6 TB/s (209 us with the arithmetic left out, 220 with operands from the
//   cache); tiles of 64 tokens in place of 128: 318 us; tiles, their composition and the scan as three launches: 603 us
//   forward, fp32, 2 x 16384 x 2048 or 4 x 8192 x 2048: 215 us, 5.0 TB/s; with its backward 624 (567 at a copy's rate)
//   off pairs, 4 x 8192 x 2047, forward and both passes: bf16 152 and 438 us (122 and 357 for 2048 channels), fp32 233 and 686
//   few channels, bf16, 1 x 65536 x 256: 120 us, with its backward 355 (the chain of groups, whatever the channels; 26 and 71 at
//   a copy's rate)
//   forward and backward, bf16, 4 x 8192 x 2048, packed documents: 124 and 230 us, 368 with the chains' memory and the sums
#include <algorithm>
#include <cfloat>

#include "layer_launch.hpp"
#include "ssd_device.hpp"

namespace ssd {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves, kCols = 128;
template <typename T> constexpr int kTw = sizeof(T) == 2 ? 16 : 8;      // tokens of a wave, forward
template <typename T> constexpr int kTile = kTw<T> * kWaves;

// ------------------------------------------------------------ a lane's two channels
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void narrow(float* p, float v) { *p = v; }
__device__ __forceinline__ void narrow(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16_bits(v); }

// Column c of a row whose address is the wave's.
template <typename V, typename T>
__device__ __forceinline__ const V* column(const T* row, uint32_t c) {
    return reinterpret_cast<const V*>(reinterpret_cast<const char*>(row) + c * (uint32_t)sizeof(T));
}
template <typename V, typename T>
__device__ __forceinline__ V* column(T* row, uint32_t c) {
    return reinterpret_cast<V*>(reinterpret_cast<char*>(row) + c * (uint32_t)sizeof(T));
}

// PAIR: neighbours, read together (even widths and strides, bases on pairs); else 64 apart.  Channels past the last are
// read from it and not written.
template <bool PAIR>
struct Lane {
    uint32_t c[2];
    bool on, on1;
    __device__ __forceinline__ Lane(int blk, int D) {
        const int l = threadIdx.x % 64, c0 = blk * kCols + (PAIR ? 2 * l : l), c1 = PAIR ? c0 + 1 : c0 + 64;
        on = c0 < D;
        on1 = c1 < D;                               // PAIR: D is even
        c[0] = (uint32_t)min(c0, PAIR ? D - 2 : D - 1);
        c[1] = (uint32_t)min(c1, D - 1);
    }
};

// two channels of a row as they are in memory
// hide(): the compiler forgets what it knows of the values, so that it does not keep what it has made of them
template <typename T> struct Two;
template <> struct Two<float> {
    float2 v;
    __device__ __forceinline__ float get(int j) const { return j ? v.y : v.x; }
    __device__ __forceinline__ void hide() { asm volatile("" : "+v"(v.x), "+v"(v.y)); }
    __device__ __forceinline__ void keep(bool on, float off) { v = make_float2(on ? v.x : off, on ? v.y : off); }
};
template <> struct Two<uint16_t> {
    uint32_t v;
    __device__ __forceinline__ float get(int j) const { return j ? bf16_hi(v) : bf16_lo(v); }
    __device__ __forceinline__ void hide() { asm volatile("" : "+v"(v)); }
    __device__ __forceinline__ void keep(bool on, float off) { v = on ? v : (__float_as_uint(off) >> 16) * 0x10001u; }
};
// The rows of a wave's tokens as one buffer: a row is a scalar offset, a lane's channels a vector offset that all rows share,
// so that no address is computed per row and lane.  Rows past the batch row's end are its last one.
template <typename T>
struct Rows {
    __amdgpu_buffer_rsrc_t rsrc;
    int stride, most;                               // bytes; tokens after the first
    __device__ __forceinline__ Rows(const T* p, int64_t s, int b, int t0, int L) {
        const int t = min(t0, L - 1);
        rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p) + ((int64_t)b * L + t) * s, 0, 0x7fffffff, 0x00020000);
        stride = (int)(s * (int)sizeof(T));          // 16 rows of at most 2^24 bytes
        most = L - 1 - t;
    }
    __device__ __forceinline__ int at(int t) const { return min(t, most) * stride; }
};
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <bool PAIR>
__device__ __forceinline__ Two<float> load2(const Rows<float>& r, int t, const Lane<PAIR>& ln) {
    if constexpr (PAIR) {
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r.rsrc, ln.c[0] * 4, r.at(t), 0));
        return {make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]))};
    } else {
        return {make_float2(__uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r.rsrc, ln.c[0] * 4, r.at(t), 0)),
                            __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r.rsrc, ln.c[1] * 4, r.at(t), 0)))};
    }
}
template <bool PAIR>
__device__ __forceinline__ Two<uint16_t> load2(const Rows<uint16_t>& r, int t, const Lane<PAIR>& ln) {
    if constexpr (PAIR) return {(uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r.rsrc, ln.c[0] * 2, r.at(t), 0)};
    else
        return {(uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r.rsrc, ln.c[0] * 2, r.at(t), 0) |
                (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r.rsrc, ln.c[1] * 2, r.at(t), 0) << 16};
}
template <bool PAIR>
__device__ __forceinline__ void store2(const Rows<float>& r, int t, const Lane<PAIR>& ln, float a, float b) {
    if constexpr (PAIR) {
        const u32x2 v = {__float_as_uint(a), __float_as_uint(b)};
        if (ln.on) __builtin_amdgcn_raw_buffer_store_b64(v, r.rsrc, ln.c[0] * 4, r.at(t), 0);
    } else {
        if (ln.on) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(a), r.rsrc, ln.c[0] * 4, r.at(t), 0);
        if (ln.on1) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(b), r.rsrc, ln.c[1] * 4, r.at(t), 0);
    }
}
template <bool PAIR>
__device__ __forceinline__ void store2(const Rows<uint16_t>& r, int t, const Lane<PAIR>& ln, float a, float b) {
    const uint32_t v = pack_bf16x2(a, b);
    if constexpr (PAIR) {
        if (ln.on) __builtin_amdgcn_raw_buffer_store_b32(v, r.rsrc, ln.c[0] * 2, r.at(t), 0);
    } else {
        if (ln.on) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)v, r.rsrc, ln.c[0] * 2, r.at(t), 0);
        if (ln.on1) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(v >> 16), r.rsrc, ln.c[1] * 2, r.at(t), 0);
    }
}
// of a row of states
template <bool PAIR>
__device__ __forceinline__ Two<float> load2(const float* row, const Lane<PAIR>& ln) {
    if (PAIR) return {*column<float2>(row, ln.c[0])};
    return {make_float2(*column<float>(row, ln.c[0]), *column<float>(row, ln.c[1]))};
}
template <bool PAIR>
__device__ __forceinline__ void store2(float* row, const Lane<PAIR>& ln, float a, float b) {
    if (PAIR) {
        if (ln.on) *column<float2>(row, ln.c[0]) = make_float2(a, b);
    } else {
        if (ln.on) *column<float>(row, ln.c[0]) = a;
        if (ln.on1) *column<float>(row, ln.c[1]) = b;
    }
}
// ------------------------------------------------------------ the gates
__device__ __forceinline__ float sigmoid_f(float v) { return fast_rcp(1.0f + fast_exp2(-v * kLog2e)); }

// decay a = e^-n = 2^-z and 1 - a, z = n log2 e.  A decay near 1 is what a long memory rests on: there 1 - a comes from its
// series (5 terms in z, off by n^5 / 6! of itself, 4e-8 at the border) and a from 1 - a by one rounding, so that neither
// the hardware exp2's error nor the difference's shows: over thousands of tokens a decay that is off by one step the same
// way each time would move the state by some 1e-5.  From the border on the hardware's exp2 and the difference are within
// 2^-20 of 1 - a.
constexpr float kNear = 0.18f;                       // n < 0.125
__device__ __forceinline__ float one_minus(float z) {
    float q = fmaf(z, -0.0013333558146428443f, 0.009618129107628477f);
    q = fmaf(z, -q, 0.05550410866482158f);
    q = fmaf(z, -q, 0.2402265069591007f);
    q = fmaf(z, -q, 0.6931471805599453f);
    return q * z;
}
__device__ __forceinline__ void decay(float z, float& a, float& om) {
    const float q = one_minus(z), e = fast_exp2(-z);
    const bool near = z < kNear;
    a = near ? 1.0f - q : e;
    om = near ? q : 1.0f - e;
}

// bit t set: a document starts at token t0 + t (t < n <= 64)
__device__ __forceinline__ uint64_t starts_in(const int32_t* doc, int t0, int n, int L) {
    if (!doc) return 0;
    const int l = threadIdx.x % 64, t = t0 + l;
    return __ballot(l < n && t > 0 && t < L && doc[max(min(t, L - 1), 0)] != doc[max(min(t, L - 1) - 1, 0)]);
}

// A of a stretch that a document starts in: nothing passes through, in either direction, whatever the stretch's decays are.  It is
// set after their product: a NaN decay behind the start belongs to the state (H is NaN then, too), but would undo the cut for
// the adjoint, which comes from behind.
constexpr uint32_t kCut = 0x80000000u;              // -0.0
__device__ __forceinline__ bool is_cut(float A) { return __float_as_uint(A) == kCut; }
__device__ __forceinline__ float through(float A, float H, float h) { return is_cut(A) ? H : fmaf(A, h, H); }
// (A, H) and then (A2, H2); a product of -0.0 and a decay is -0.0
__device__ __forceinline__ void then(float& A, float& H, float A2, float H2) {
    H = through(A2, H2, H);
    A = is_cut(A2) ? A2 : A * A2;
}

// Infinite parameters as the largest finite numbers: the same decay of 0 and gate of 1, but with a gate of 0 no 0 * inf.  NaN
// stays.  Where they are applied costs: with both on every parameter as it is loaded 4 x 8192 x 2048 took 371 us in place of 368.
__device__ __forceinline__ float at_most(float v) { return v > FLT_MAX ? FLT_MAX : v; }
__device__ __forceinline__ float at_least(float v) { return v < -FLT_MAX ? -FLT_MAX : v; }

// the wave's number, known to the compiler to be the same for its lanes: rows are then addressed by scalars
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// a lane's parameters: -A log2 e and the biases times -log2 e, for sigmoid(v + bias) = 1 / (1 + 2^(-v log2 e - bias log2 e))
struct Params {
    float zA[2], rb[2], ib[2];
    template <bool PAIR>
    __device__ __forceinline__ void load(const GlrArgs& a, const Lane<PAIR>& ln) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            zA[j] = at_most(*column<float>(a.A, ln.c[j]) * -kLog2e);
            rb[j] = a.r_bias ? -kLog2e * *column<float>(a.r_bias, ln.c[j]) : 0.0f;
            ib[j] = a.i_bias ? -kLog2e * *column<float>(a.i_bias, ln.c[j]) : 0.0f;
        }
    }
    // for waves with tokens that are not real, whose r is -inf: with an infinite bias that would be inf - inf
    __device__ __forceinline__ void bounded() { rb[0] = at_least(rb[0]), rb[1] = at_least(rb[1]); }
    __device__ __forceinline__ float r_gate(float v, int j) const { return fast_rcp(1.0f + fast_exp2(fmaf(v, -kLog2e, rb[j]))); }
    __device__ __forceinline__ float i_gate(float v, int j) const { return fast_rcp(1.0f + fast_exp2(fmaf(v, -kLog2e, ib[j]))); }
};

// What a wave knows of its place: batch row, tile, first token, tokens that are real
struct Place {
    int b, c, blk, t0, len;
    __device__ __forceinline__ Place(const GlrArgs& a, int id, int tile, int Tw) {
        const int nblk = (a.D + kCols - 1) / kCols;
        blk = id % nblk;
        b = id / nblk % a.B;
        c = id / nblk / a.B;
        t0 = c * tile + wave_id() * Tw;
        len = a.lengths ? max(0, min(a.lengths[b], a.L)) : a.L;
    }
};

// Bits of a wave's n <= 16 tokens: those that start a document, those that are real.  In vector registers, though the same
// in every lane: of scalars the compiler makes a branch a token.  plain: none starts and all are real.
struct Masks {
    uint32_t starts, lives;
    bool plain;
    __device__ __forceinline__ Masks(const GlrArgs& g, const Place& p, int n) {
        lives = (1u << max(0, min(p.len - p.t0, n))) - 1;
        starts = (uint32_t)starts_in(g.doc ? g.doc + (size_t)p.b * g.L : nullptr, p.t0, n, g.L) & lives;
        plain = starts == 0 && lives == (1u << n) - 1;
        asm volatile("" : "+v"(starts), "+v"(lives));
    }
};
__device__ __forceinline__ bool bit(uint32_t mask, int t) { return (mask >> t) & 1; }

// A token that is not real decays by 1 and takes nothing in: its decay gate is that of -inf, its inputs are 0.
template <typename T>
__device__ __forceinline__ void blank(Two<T>& x, Two<T>& r, Two<T>& i, bool live) {
    x.keep(live, 0.0f);
    r.keep(live, -INFINITY);
    i.keep(live, 0.0f);
}

// decays and inputs of a wave's tokens, and their composition
template <typename T, bool PAIR, int Tw>
struct Stretch {
    float a[Tw][2], v[Tw][2];
    float A[2], H[2];
    __device__ __forceinline__ void gates(const Two<T> (&x)[Tw], const Two<T> (&r)[Tw], const Two<T> (&i)[Tw], const Params& w,
                                          const Masks& m) {
#pragma unroll
        for (int t = 0; t < Tw; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float s = w.r_gate(r[t].get(j), j);
                float om;
                decay(s * w.zA[j], a[t][j], om);
                v[t][j] = __builtin_amdgcn_sqrtf(fmaf(om, a[t][j], om)) * w.i_gate(i[t].get(j), j) * x[t].get(j);
                // here and now: the compiler would put part of every token off, and hold what that part needs
                asm volatile("" : "+v"(a[t][j]), "+v"(v[t][j]));
            }
        A[0] = A[1] = 1.0f;
        H[0] = H[1] = 0.0f;
        if (m.plain) {
#pragma unroll
            for (int t = 0; t < Tw; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    A[j] *= a[t][j];
                    H[j] = fmaf(a[t][j], H[j], v[t][j]);
                }
        } else {
#pragma unroll
            for (int t = 0; t < Tw; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    A[j] *= a[t][j];
                    H[j] = bit(m.starts, t) ? v[t][j] : fmaf(a[t][j], H[j], v[t][j]);
                }
            if (m.starts) A[0] = A[1] = __uint_as_float(kCut);
        }
    }
};

// ------------------------------------------------------------ tiles in a chain
// Places 0, 1, ... along each row of the batch (forward: its tiles in order, backward: from the last).  All bits set: not
// written yet.  A's own NaNs have other bits.  Groups of 8, a place a wave: with 16 a tile fetches twice the pairs, 5 % of
// the forward's traffic in bf16, and takes 1 % longer.
constexpr int kGroup = kWaves;
constexpr uint32_t kUnset = 0xffffffffu;
struct Chain {
    uint32_t* ticket;                               // kUnset at the start
    uint64_t* pairs;                                // [B][tiles][D]
    uint64_t* enter;                                // [B][groups - 1][D]: the state that leaves a group
    int groups;
};
__device__ __forceinline__ uint64_t pack_pair(float A, float H) {
    return (uint64_t)__float_as_uint(H) << 32 | (A == A ? __float_as_uint(A) : 0x7fc00000u);
}
__device__ __forceinline__ float pair_A(uint64_t w) { return __uint_as_float((uint32_t)w); }
__device__ __forceinline__ float pair_H(uint64_t w) { return __uint_as_float((uint32_t)(w >> 32)); }
__device__ __forceinline__ bool is_set(uint64_t w) { return (uint32_t)w != kUnset; }
__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <bool PAIR>
__device__ __forceinline__ void publish(uint64_t* row, const Lane<PAIR>& ln, float2 A, float2 H) {
    if (ln.on) __hip_atomic_store(column<uint64_t>(row, ln.c[0]), pack_pair(A.x, H.x), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (ln.on1) __hip_atomic_store(column<uint64_t>(row, ln.c[1]), pack_pair(A.y, H.y), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <bool PAIR>
__device__ __forceinline__ void await(const uint64_t* row, const Lane<PAIR>& ln, uint64_t (&w)[2]) {
    for (;;) {
        w[0] = peek(column<uint64_t>(row, ln.c[0]));
        w[1] = peek(column<uint64_t>(row, ln.c[1]));
        if (__all(is_set(w[0]) && is_set(w[1]))) return;
        __builtin_amdgcn_s_sleep(4);
    }
}
__device__ __forceinline__ int chain_place(const Chain& ch) {
    __shared__ uint32_t place;
    if (threadIdx.x == 0) place = atomicAdd(ch.ticket, 1u) + 1u;
    __syncthreads();
    return (int)__builtin_amdgcn_readfirstlane(place);
}
// What stands before place k of a row: each wave fetches one of the places before k in k's group into pA, pH, wave 0 also
// the state that enters the group.  Followed by a barrier and chain_enter().
template <bool PAIR>
__device__ __forceinline__ void chain_gather(const Chain& ch, int b, int k, int tiles, int D, const Lane<PAIR>& ln, float2 (*pA)[64],
                                             float2 (*pH)[64], float2* in) {
    const int wave = wave_id(), l = threadIdx.x % 64, group = k / kGroup, place = group * kGroup + wave;
    uint64_t w[2];
    if (place < k) {
        await(ch.pairs + ((size_t)b * tiles + place) * D, ln, w);
        pA[wave][l] = make_float2(pair_A(w[0]), pair_A(w[1]));
        pH[wave][l] = make_float2(pair_H(w[0]), pair_H(w[1]));
    }
    if (wave == 0 && group > 0) {
        await(ch.enter + ((size_t)b * (ch.groups - 1) + group - 1) * D, ln, w);
        in[l] = make_float2(pair_H(w[0]), pair_H(w[1]));
    }
}
__device__ __forceinline__ void chain_enter(int k, const float2 (*pA)[64], const float2 (*pH)[64], const float2* in, float (&h)[2]) {
    const int l = threadIdx.x % 64, n = k % kGroup;
    if (k >= kGroup) {
        h[0] = in[l].x;
        h[1] = in[l].y;
    }
    for (int w = 0; w < n; ++w) {
        const float2 A = pA[w][l], H = pH[w][l];
        h[0] = through(A.x, H.x, h[0]);
        h[1] = through(A.y, H.y, h[1]);
    }
}
// the chain's memory to all bits set, 16 bytes a thread
__global__ __launch_bounds__(256) void ssd_glr_unset_kernel(uint4* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        p[i] = make_uint4(kUnset, kUnset, kUnset, kUnset);
}

// ------------------------------------------------------------ forward
// CHAIN: one tile a workgroup, rows of many; else a workgroup walks a row's tiles
// Two workgroups a CU, except where 16-bit channels are read one by one (twice the registers on their way) or walked.
// 16 tokens of a wave in bf16, 8 in fp32: the same bytes on their way, and what the registers of two workgroups hold.
template <typename T, bool PAIR, bool CHAIN>
__global__ __launch_bounds__(kThreads, (CHAIN && (PAIR || sizeof(T) == 4) ? 4 : 2)) void ssd_glr_scan_kernel(GlrArgs g, Chain ch) {
    constexpr int Tw = kTw<T>;
    __shared__ float2 sA[2][kWaves][64], sH[2][kWaves][64], pA[CHAIN ? kWaves : 1][64], pH[CHAIN ? kWaves : 1][64], in[64];
    Place p(g, CHAIN ? chain_place(ch) : blockIdx.x, kTile<T>, Tw);
    const Lane<PAIR> ln(p.blk, g.D);
    const int wave = wave_id(), l = threadIdx.x % 64;
    Params w;
    w.load(g, ln);
    float h[2] = {0.0f, 0.0f};
    if (p.c == 0 && g.init_state) {
        const Two<float> e = load2(g.init_state + (size_t)p.b * g.D, ln);
        h[0] = e.get(0);
        h[1] = e.get(1);
    }
    for (;;) {
        Stretch<T, PAIR, Tw> s;
        Two<T> x[Tw], r[Tw], i[Tw];
        {
            const Rows<T> xr(static_cast<const T*>(g.x), g.x_stride, p.b, p.t0, g.L),
                rr(static_cast<const T*>(g.r), g.r_stride, p.b, p.t0, g.L),
                ir(static_cast<const T*>(g.i), g.i_stride, p.b, p.t0, g.L);
#pragma unroll
            for (int t = 0; t < Tw; ++t) {
                x[t] = load2(xr, t, ln);
                r[t] = load2(rr, t, ln);
                i[t] = load2(ir, t, ln);
            }
        }
        const Masks m(g, p, Tw);
        if (!m.plain) {
            w.bounded();
#pragma unroll
            for (int t = 0; t < Tw; ++t) blank(x[t], r[t], i[t], bit(m.lives, t));
        }
        s.gates(x, r, i, w, m);
        const int turn = CHAIN ? 0 : p.c & 1;        // a walk's next tile leaves these alone
        sA[turn][wave][l] = make_float2(s.A[0], s.A[1]);
        sH[turn][wave][l] = make_float2(s.H[0], s.H[1]);
        // init_state has been read by all, for final_state may be it: h itself, not a load of it, passes the barrier
        asm volatile("" : "+v"(h[0]), "+v"(h[1]));
        __syncthreads();
        if constexpr (CHAIN) {
            if (wave == kWaves - 1) {                // the first tile starts from the row's own state: a cut
                float2 A = p.c == 0 ? make_float2(__uint_as_float(kCut), __uint_as_float(kCut)) : make_float2(1.0f, 1.0f);
                float2 H = make_float2(h[0], h[1]);
#pragma unroll
                for (int k = 0; k < kWaves; ++k) {
                    const float2 a = sA[0][k][l], v = sH[0][k][l];
                    then(A.x, H.x, a.x, v.x);
                    then(A.y, H.y, a.y, v.y);
                }
                publish(ch.pairs + ((size_t)p.b * g.tiles + p.c) * g.D, ln, A, H);
            }
            chain_gather(ch, p.b, p.c, g.tiles, g.D, ln, pA, pH, in);
            __syncthreads();
            chain_enter(p.c, pA, pH, in, h);
        }
        const float enter[2] = {h[0], h[1]};
        for (int k = 0; k < wave; ++k) {
            const float2 a = sA[turn][k][l], v = sH[turn][k][l];
            h[0] = through(a.x, v.x, h[0]);
            h[1] = through(a.y, v.y, h[1]);
        }
        if constexpr (CHAIN) {
            if (wave == kWaves - 1 && p.c % kGroup == kGroup - 1 && p.c + 1 < g.tiles)
                publish(ch.enter + ((size_t)p.b * (ch.groups - 1) + p.c / kGroup) * g.D, ln, make_float2(0.0f, 0.0f),
                        make_float2(through(s.A[0], s.H[0], h[0]), through(s.A[1], s.H[1], h[1])));
        }
        if (p.t0 < g.L) {
            if (g.states && p.t0 % 64 == 0)
                store2(g.states + ((size_t)p.b * ((g.L + 63) / 64) + p.t0 / 64) * g.D, ln, h[0], h[1]);
            const Rows<T> yr(static_cast<const T*>(g.y), g.y_stride, p.b, p.t0, g.L);
            if (m.plain && g.y) {
#pragma unroll
                for (int t = 0; t < Tw; ++t) {
                    h[0] = fmaf(s.a[t][0], h[0], s.v[t][0]);
                    h[1] = fmaf(s.a[t][1], h[1], s.v[t][1]);
                    store2(yr, t, ln, h[0], h[1]);
                }
            } else if (g.y || g.final_state) {
#pragma unroll
                for (int t = 0; t < Tw; ++t) {
                    const bool live = bit(m.lives, t), start = bit(m.starts, t);
#pragma unroll
                    for (int j = 0; j < 2; ++j) h[j] = start ? s.v[t][j] : fmaf(s.a[t][j], h[j], s.v[t][j]);
                    if (g.y && p.t0 + t < g.L) store2(yr, t, ln, live ? h[0] : 0.0f, live ? h[1] : 0.0f);
                }
            }
            if (g.final_state && p.t0 + Tw >= g.L) store2(g.final_state + (size_t)p.b * g.D, ln, h[0], h[1]);
        }
        if (CHAIN || p.c + 1 == g.tiles) break;
        h[0] = enter[0];
        h[1] = enter[1];
        for (int k = 0; k < kWaves; ++k) {
            const float2 a = sA[turn][k][l], v = sH[turn][k][l];
            h[0] = through(a.x, v.x, h[0]);
            h[1] = through(a.y, v.y, h[1]);
        }
        ++p.c;
        p.t0 += kTile<T>;
    }
}

// ------------------------------------------------------------ backward
constexpr int kTb = 8, kTileB = kTb * kWaves;         // tokens of a wave and of a tile: a chunk of 64
static_assert(kTileB == 64, "a tile starts at a chunk's state");

// What a wave needs of its tokens in both directions
template <typename T, bool PAIR>
struct Back {
    Two<T> x[kTb], gy[kTb];
    float a[kTb][2], v[kTb][2], s[kTb][2], gi[kTb][2];    // decay, input (later a h_{t-1}), gates
    float A[2], H[2], N[2];                               // compositions: of the state, and of the adjoint from behind
    __device__ __forceinline__ void gates(const Two<T> (&r)[kTb], const Two<T> (&i)[kTb], const Params& w, const Masks& k) {
#pragma unroll
        for (int t = 0; t < kTb; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float om;
                s[t][j] = w.r_gate(r[t].get(j), j);
                gi[t][j] = w.i_gate(i[t].get(j), j);
                decay(s[t][j] * w.zA[j], a[t][j], om);
                v[t][j] = __builtin_amdgcn_sqrtf(fmaf(om, a[t][j], om)) * gi[t][j] * x[t].get(j);
                // here and now: the compiler would put part of every token off, and hold what that part needs
                asm volatile("" : "+v"(a[t][j]), "+v"(v[t][j]), "+v"(s[t][j]), "+v"(gi[t][j]));
            }
        A[0] = A[1] = 1.0f;
        H[0] = H[1] = N[0] = N[1] = 0.0f;
        if (k.plain) {
#pragma unroll
            for (int t = 0; t < kTb; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    A[j] *= a[t][j];
                    H[j] = fmaf(a[t][j], H[j], v[t][j]);
                }
#pragma unroll
            for (int t = kTb - 1; t >= 0; --t)
#pragma unroll
                for (int j = 0; j < 2; ++j) N[j] = a[t][j] * (gy[t].get(j) + N[j]);
        } else {
#pragma unroll
            for (int t = 0; t < kTb; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    A[j] *= a[t][j];
                    H[j] = bit(k.starts, t) ? v[t][j] : fmaf(a[t][j], H[j], v[t][j]);
                }
            if (k.starts) A[0] = A[1] = __uint_as_float(kCut);
#pragma unroll
            for (int t = kTb - 1; t >= 0; --t)
#pragma unroll
                for (int j = 0; j < 2; ++j) N[j] = bit(k.starts, t) ? 0.0f : a[t][j] * (gy[t].get(j) + N[j]);
        }
    }
    // a h_{t-1} in the inputs' place; h: the state that enters
    __device__ __forceinline__ void hold(float (&h)[2], const Masks& k) {
#pragma unroll
        for (int t = 0; t < kTb; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float was = bit(k.starts, t) ? 0.0f : a[t][j] * h[j];
                h[j] = was + v[t][j];
                v[t][j] = bit(k.lives, t) ? was : 0.0f;
            }
        // so that nothing made of these above is kept for below
#pragma unroll
        for (int t = 0; t < kTb; ++t) {
            x[t].hide();
            gy[t].hide();
#pragma unroll
            for (int j = 0; j < 2; ++j) asm volatile("" : "+v"(s[t][j]), "+v"(gi[t][j]));
        }
    }
    // the gradients; nu: the adjoint that enters from behind, then the one that leaves
    __device__ __forceinline__ void grads(const GlrArgs& g, const Place& p, const Lane<PAIR>& ln, const Masks& k, float (&nu)[2],
                                          float (&sum)[3][2]) {
        const Rows<T> xr(static_cast<const T*>(g.dx), g.dx_stride, p.b, p.t0, g.L),
            rr(static_cast<const T*>(g.dr), g.dr_stride, p.b, p.t0, g.L),
            ir(static_cast<const T*>(g.di), g.di_stride, p.b, p.t0, g.L);
        // not held from above; -inf would be inf - inf below
        float A2[2] = {at_least(*column<float>(g.A, ln.c[0])), at_least(*column<float>(g.A, ln.c[1]))};
#pragma unroll
        for (int t = kTb - 1; t >= 0; --t) {
            float dx[2], dr[2], di[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float all = gy[t].get(j) + nu[j], lam = bit(k.lives, t) ? all : 0.0f;
                nu[j] = bit(k.starts, t) ? 0.0f : a[t][j] * all;
                const float z = s[t][j] * (A2[j] * -kLog2e);
                float q = one_minus(z);
                asm volatile("" : "+v"(q));              // no branch around it, nor below
                const float om = z < kNear ? q : 1.0f - a[t][j], m2 = fmaf(om, a[t][j], om);
                float inv = __builtin_amdgcn_rsqf(m2);
                asm volatile("" : "+v"(inv));
                inv = m2 >= 0x1p-126f ? inv : 0.0f;      // 1 / m, 0 where m is: the units take a subnormal m2 as 0
                const float gx = gi[t][j] * x[t].get(j), lm = lam * (m2 * inv);
                dx[j] = lm * gi[t][j];
                di[j] = lm * fmaf(-gx, gi[t][j], gx);
                const float ds = lam * (v[t][j] - gx * (a[t][j] * a[t][j]) * inv) * s[t][j];
                dr[j] = ds * fmaf(-A2[j], s[t][j], A2[j]);
                sum[0][j] += ds;
                sum[1][j] += dr[j];
                sum[2][j] += di[j];
            }
            if (p.t0 + t < g.L) {
                store2(xr, t, ln, dx[0], dx[1]);
                store2(rr, t, ln, dr[0], dr[1]);
                store2(ir, t, ln, di[0], di[1]);
            }
        }
    }
};

// The chain runs from a row's last tile.  part: [tile of all rows][3][D], a tile's sums of dA, dr_bias and di_bias.
// fp32 operands take the registers of one workgroup a CU; as many bytes are on their way then as with two in bf16.
// 8 tokens of a wave, so that a tile starts at a state that the forward kept: 4 x 8192 x 2048 in bf16 takes 230 us (1.0 GB with
// the kept states and the partial sums, 4.4 TB/s).  Decays are formed again where the gradients need them: held, they would
// spill.
template <typename T, bool PAIR, bool CHAIN>
__global__ __launch_bounds__(kThreads, (CHAIN && sizeof(T) == 2 ? 4 : 2)) void ssd_glr_back_kernel(GlrArgs g, Chain ch, float* part) {
    __shared__ float2 sA[kWaves][64], sH[kWaves][64], sN[kWaves][64], pA[CHAIN ? kWaves : 1][64], pN[CHAIN ? kWaves : 1][64], in[64];
    Place p(g, CHAIN ? chain_place(ch) : blockIdx.x, kTileB, kTb);
    const Lane<PAIR> ln(p.blk, g.D);
    const int wave = wave_id(), l = threadIdx.x % 64;
    Params w;
    w.load(g, ln);
    float nu[2] = {0.0f, 0.0f};
    int place = p.c;
    if (place == 0 && g.g_final) {
        const Two<float> e = load2(g.g_final + (size_t)p.b * g.D, ln);
        nu[0] = e.get(0);
        nu[1] = e.get(1);
    }
    for (;;) {
        p.c = g.tiles - 1 - place;
        p.t0 = p.c * kTileB + wave * kTb;
        const size_t tile = (size_t)p.b * g.tiles + p.c;
        Back<T, PAIR> s;
        const Two<float> e = load2(g.states + tile * g.D, ln);
        Two<T> r[kTb], i[kTb];
        {
            const Rows<T> xr(static_cast<const T*>(g.x), g.x_stride, p.b, p.t0, g.L),
                rr(static_cast<const T*>(g.r), g.r_stride, p.b, p.t0, g.L),
                ir(static_cast<const T*>(g.i), g.i_stride, p.b, p.t0, g.L),
                yr(static_cast<const T*>(g.gy), g.gy_stride, p.b, p.t0, g.L);
#pragma unroll
            for (int t = 0; t < kTb; ++t) {
                s.x[t] = load2(xr, t, ln);
                r[t] = load2(rr, t, ln);
                i[t] = load2(ir, t, ln);
                s.gy[t] = load2(yr, t, ln);
            }
        }
        const Masks m(g, p, kTb);
        if (!m.plain) {
            w.bounded();
#pragma unroll
            for (int t = 0; t < kTb; ++t) {
                blank(s.x[t], r[t], i[t], bit(m.lives, t));
                s.gy[t].keep(bit(m.lives, t), 0.0f);
            }
        }
        s.gates(r, i, w, m);
        float h[2] = {e.get(0), e.get(1)};
        sA[wave][l] = make_float2(s.A[0], s.A[1]);
        sH[wave][l] = make_float2(s.H[0], s.H[1]);
        sN[wave][l] = make_float2(s.N[0], s.N[1]);
        __syncthreads();
        if constexpr (CHAIN) {
            if (wave == kWaves - 1) {
                float2 A = place == 0 ? make_float2(__uint_as_float(kCut), __uint_as_float(kCut)) : make_float2(1.0f, 1.0f);
                float2 N = make_float2(nu[0], nu[1]);
#pragma unroll 2
                for (int k = kWaves - 1; k >= 0; --k) {
                    const float2 a = sA[k][l], n = sN[k][l];
                    then(A.x, N.x, a.x, n.x);
                    then(A.y, N.y, a.y, n.y);
                }
                publish(ch.pairs + ((size_t)p.b * g.tiles + place) * g.D, ln, A, N);
            }
            chain_gather(ch, p.b, place, g.tiles, g.D, ln, pA, pN, in);
            __syncthreads();
            chain_enter(place, pA, pN, in, nu);
        }
        const float enter[2] = {nu[0], nu[1]};
        for (int k = 0; k < wave; ++k) {
            const float2 a = sA[k][l], v = sH[k][l];
            h[0] = through(a.x, v.x, h[0]);
            h[1] = through(a.y, v.y, h[1]);
        }
        for (int k = kWaves - 1; k > wave; --k) {
            const float2 a = sA[k][l], v = sN[k][l];
            nu[0] = through(a.x, v.x, nu[0]);
            nu[1] = through(a.y, v.y, nu[1]);
        }
        float next[2] = {nu[0], nu[1]};
        if constexpr (CHAIN) {
            if (wave == 0 && place % kGroup == kGroup - 1 && place + 1 < g.tiles)
                publish(ch.enter + ((size_t)p.b * (ch.groups - 1) + place / kGroup) * g.D, ln, make_float2(0.0f, 0.0f),
                        make_float2(through(s.A[0], s.N[0], nu[0]), through(s.A[1], s.N[1], nu[1])));
        } else {
            next[0] = enter[0];
            next[1] = enter[1];
            for (int k = kWaves - 1; k >= 0; --k) {
                const float2 a = sA[k][l], v = sN[k][l];
                next[0] = through(a.x, v.x, next[0]);
                next[1] = through(a.y, v.y, next[1]);
            }
        }
        float sum[3][2] = {};
        s.hold(h, m);
        s.grads(g, p, ln, m, nu, sum);
        if (g.g_init && p.t0 == 0) store2(g.g_init + (size_t)p.b * g.D, ln, nu[0], nu[1]);
        // the waves' sums in their order
        __syncthreads();
        sA[wave][l] = make_float2(sum[0][0], sum[0][1]);
        sH[wave][l] = make_float2(sum[1][0], sum[1][1]);
        sN[wave][l] = make_float2(sum[2][0], sum[2][1]);
        __syncthreads();
        if (wave < 3) {
            const float2(*from)[64] = wave == 0 ? sA : wave == 1 ? sH : sN;
            float a = 0.0f, b = 0.0f;
#pragma unroll
            for (int k = 0; k < kWaves; ++k) {
                a += from[k][l].x;
                b += from[k][l].y;
            }
            store2(part + (tile * 3 + wave) * g.D, ln, a, b);
        }
        if (CHAIN || p.c == 0) break;
        nu[0] = next[0];
        nu[1] = next[1];
        ++place;
        __syncthreads();                             // the sums have been read
    }
}

// dA, dr_bias and di_bias: the tiles' sums in a fixed order, in 64 bits.  32 columns a workgroup, 32 threads a column, each
// with eight rows on their way at a time: 512 rows of 6144 in 4.6 us, one at a time 12.
__global__ __launch_bounds__(1024) void ssd_glr_sum_kernel(const float* part, int64_t rows, int D, float* dA, float* dr_bias,
                                                           float* di_bias) {
    __shared__ double s[32][33];
    const int x = threadIdx.x % 32, k = threadIdx.x / 32, c = blockIdx.x * 32 + x;
    double v = 0.0;
    if (c < 3 * D) {
        const float* p = part + c;
        int64_t r = k;
        for (; r + 7 * 32 < rows; r += 8 * 32) {
            float u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = p[(r + 32 * j) * 3 * D];
#pragma unroll
            for (int j = 0; j < 8; ++j) v += u[j];
        }
        for (; r < rows; r += 32) v += p[r * 3 * D];
    }
    s[k][x] = v;
    __syncthreads();
    if (k || c >= 3 * D) return;
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][x];
    if (c < D) dA[c] = (float)t;
    else if (c < 2 * D) {
        if (dr_bias) dr_bias[c - D] = (float)t;
    } else if (di_bias) di_bias[c - 2 * D] = (float)t;
}

// to = from, or 0 where there is none: a state through a row of no tokens
__global__ __launch_bounds__(256) void ssd_glr_copy_kernel(const float* from, float* to, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) to[i] = from ? from[i] : 0.0f;
}

// ------------------------------------------------------------ one token
// V channels a thread: 8 where every row, state and parameter starts on a 16-byte boundary and D % 8 == 0, else 1.  Bound by HBM:
// 8 bytes of state and four activations a channel.  256 x 8192 in fp32: 10.8 us (50 MB, 9.7 at a copy's rate); in bf16: 8.3 us (33.6 MB; 7.8 in a graph, where an
// empty step takes 2.4), 15.8 with the parameters read one by one, 8.9 in a graph with four rows a thread.
template <typename T, int V> __device__ __forceinline__ void step_ld(const T* p, float (&o)[V]) {
    if constexpr (V == 1) {
        o[0] = widen(*p);
    } else if constexpr (sizeof(T) == 2) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        o[0] = bf16_lo(v.x); o[1] = bf16_hi(v.x); o[2] = bf16_lo(v.y); o[3] = bf16_hi(v.y);
        o[4] = bf16_lo(v.z); o[5] = bf16_hi(v.z); o[6] = bf16_lo(v.w); o[7] = bf16_hi(v.w);
    } else {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
        o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
    }
}
template <typename T, int V> __device__ __forceinline__ void step_st(T* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        narrow(p, v[0]);
    } else if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
}
template <typename T, int V>
__global__ __launch_bounds__(256) void ssd_glr_step_kernel(GlrArgs g) {
    const uint32_t n = g.D / V, at = blockIdx.x * 256u + threadIdx.x;      // V > 1: D % 8 == 0; B * D < 2^31
    if (at >= g.B * n) return;
    const int b = (int)(at / n), c = (int)(at % n) * V;
    float x[V], r[V], i[V], A[V], rb[V], ib[V], h[V];
    step_ld<T, V>(static_cast<const T*>(g.x) + b * g.x_stride + c, x);
    step_ld<T, V>(static_cast<const T*>(g.r) + b * g.r_stride + c, r);
    step_ld<T, V>(static_cast<const T*>(g.i) + b * g.i_stride + c, i);
    float* state = g.final_state + (int64_t)b * g.D + c;
    step_ld<float, V>(state, h);
#pragma unroll
    for (int j = 0; j < V; ++j) rb[j] = ib[j] = 0.0f;
    step_ld<float, V>(g.A + c, A);
    if (g.r_bias) step_ld<float, V>(g.r_bias + c, rb);
    if (g.i_bias) step_ld<float, V>(g.i_bias + c, ib);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float d, om;
        decay(sigmoid_f(r[j] + rb[j]) * at_most(A[j] * -kLog2e), d, om);
        h[j] = fmaf(d, h[j], __builtin_amdgcn_sqrtf(fmaf(om, d, om)) * sigmoid_f(i[j] + ib[j]) * x[j]);
    }
    step_st<float, V>(state, h);
    step_st<T, V>(static_cast<T*>(g.y) + b * g.y_stride + c, h);
}

int cols(int D) { return (D + kCols - 1) / kCols; }
int tiles_of(int L, int tile) { return (int)(((int64_t)L + tile - 1) / tile); }
size_t pad16(size_t n) { return (n + 15) / 16 * 16; }

// Rows of at most this many tiles are walked by one workgroup: the chain's memory is another launch, 3.7 us of the host's
// time, against some 3 us a tile.  3 x 77 x 201 in fp32: 12.0 us walked, 16.7 in a chain.
constexpr int kWalk = 2;

// the chain of a launch over `tiles` tiles a row, in n bytes at `ws`
size_t chain_bytes(int B, int D, int tiles) {
    if (tiles <= kWalk) return 0;
    return 256 + pad16((size_t)B * D * (tiles + (tiles + kGroup - 1) / kGroup - 1) * sizeof(uint64_t));
}
hipError_t make_chain(Chain& ch, int B, int D, int tiles, char* ws, hipStream_t s) {
    ch.groups = (tiles + kGroup - 1) / kGroup;
    ch.ticket = reinterpret_cast<uint32_t*>(ws);
    ch.pairs = reinterpret_cast<uint64_t*>(ws + 256);
    ch.enter = ch.pairs + (size_t)B * tiles * D;
    const int64_t n = (int64_t)(chain_bytes(B, D, tiles) / 16);
    hipLaunchKernelGGL(ssd_glr_unset_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 2048)), dim3(256), 0, s,
                       reinterpret_cast<uint4*>(ws), n);
    return hipGetLastError();
}

template <typename T, bool PAIR>
hipError_t fwd_t(GlrArgs a, char* ws, hipStream_t s) {
    a.tiles = tiles_of(a.L, kTile<T>);
    const int64_t rows = (int64_t)a.B * cols(a.D);
    Chain ch{};
    if (a.tiles > kWalk) {
        if (hipError_t e = make_chain(ch, a.B, a.D, a.tiles, ws, s)) return e;
        hipLaunchKernelGGL((ssd_glr_scan_kernel<T, PAIR, true>), dim3((unsigned)(a.tiles * rows)), dim3(kThreads), 0, s, a, ch);
    } else {
        hipLaunchKernelGGL((ssd_glr_scan_kernel<T, PAIR, false>), dim3((unsigned)rows), dim3(kThreads), 0, s, a, ch);
    }
    return hipGetLastError();
}

size_t fwd_bytes(int B, int L, int D, int dtype) {
    return chain_bytes(B, D, tiles_of(L, dtype == 0 ? kTile<float> : kTile<uint16_t>));
}
size_t states_bytes(int B, int L, int D) { return pad16((size_t)B * tiles_of(L, kTileB) * D * sizeof(float)); }

template <typename T, bool PAIR>
hipError_t bwd_t(GlrArgs a, char* ws, hipStream_t s) {
    if (!a.states) {
        a.states = reinterpret_cast<float*>(ws);
        ws += states_bytes(a.B, a.L, a.D);
        GlrArgs f = a;
        f.y = nullptr;
        f.final_state = nullptr;
        if (hipError_t e = fwd_t<T, PAIR>(f, ws, s)) return e;
        ws += fwd_bytes(a.B, a.L, a.D, a.dtype);
    }
    a.tiles = tiles_of(a.L, kTileB);
    float* part = reinterpret_cast<float*>(ws);
    ws += pad16((size_t)a.B * a.tiles * 3 * a.D * sizeof(float));
    const int64_t rows = (int64_t)a.B * cols(a.D);
    Chain ch{};
    if (a.tiles > kWalk) {
        if (hipError_t e = make_chain(ch, a.B, a.D, a.tiles, ws, s)) return e;
        hipLaunchKernelGGL((ssd_glr_back_kernel<T, PAIR, true>), dim3((unsigned)(a.tiles * rows)), dim3(kThreads), 0, s, a, ch, part);
    } else {
        hipLaunchKernelGGL((ssd_glr_back_kernel<T, PAIR, false>), dim3((unsigned)rows), dim3(kThreads), 0, s, a, ch, part);
    }
    if (hipError_t e = hipGetLastError()) return e;
    hipLaunchKernelGGL(ssd_glr_sum_kernel, dim3((unsigned)((3LL * a.D + 31) / 32)), dim3(1024), 0, s, part,
                       (int64_t)a.B * a.tiles, a.D, a.dA, a.dr_bias, a.di_bias);
    return hipGetLastError();
}

}  // namespace

size_t glr_fwd_workspace_bytes(int B, int L, int D, int dtype) { return fwd_bytes(B, L, D, dtype); }
size_t glr_bwd_workspace_bytes(int B, int L, int D, int dtype) {
    const int tiles = tiles_of(L, kTileB);
    return states_bytes(B, L, D) + fwd_bytes(B, L, D, dtype) + pad16((size_t)B * tiles * 3 * D * sizeof(float)) +
           chain_bytes(B, D, tiles);
}

hipError_t launch_glr_fwd(const GlrArgs& a, void* workspace, hipStream_t s) {
    char* ws = static_cast<char*>(workspace);
    if (a.dtype == 0) return a.pair ? fwd_t<float, true>(a, ws, s) : fwd_t<float, false>(a, ws, s);
    return a.pair ? fwd_t<uint16_t, true>(a, ws, s) : fwd_t<uint16_t, false>(a, ws, s);
}
hipError_t launch_glr_bwd(const GlrArgs& a, void* workspace, hipStream_t s) {
    char* ws = static_cast<char*>(workspace);
    if (a.dtype == 0) return a.pair ? bwd_t<float, true>(a, ws, s) : bwd_t<float, false>(a, ws, s);
    return a.pair ? bwd_t<uint16_t, true>(a, ws, s) : bwd_t<uint16_t, false>(a, ws, s);
}
hipError_t launch_glr_copy(const float* from, float* to, int64_t n, hipStream_t s) {
    if (n == 0) return hipSuccess;
    hipLaunchKernelGGL(ssd_glr_copy_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, from, to, n);
    return hipGetLastError();
}
hipError_t launch_glr_step(const GlrArgs& a, hipStream_t s) {
    const int64_t n = (int64_t)a.B * (a.vec ? a.D / 8 : a.D);
    const dim3 grid((unsigned)((n + 255) / 256));
    if (a.dtype == 0) {
        if (a.vec) hipLaunchKernelGGL((ssd_glr_step_kernel<float, 8>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((ssd_glr_step_kernel<float, 1>), grid, dim3(256), 0, s, a);
    } else {
        if (a.vec) hipLaunchKernelGGL((ssd_glr_step_kernel<uint16_t, 8>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((ssd_glr_step_kernel<uint16_t, 1>), grid, dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace ssd

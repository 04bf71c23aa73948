// proj.hip -- the 8-bit projection: activations and weights in e4m3, each with a scale for every 128 columns of K.
//
//   y[m][n] = sum_b as[m][b] ws[n / 128][b] (sum_{k in block b} a[m][k] w[n][k])
//
// A block's inner sum starts from zero and joins the accumulator by one fma with the two scales' product, so no scale is
// rounded to fewer bits.  The weights are the product's row operand and the activations its columns: a lane then holds
// four neighbouring columns of one row of y, and needs one activation scale.
//
// The inner sum, for y in bf16: one v_mfma_f32_16x16x128 on e4m3.  That unit adds eight products at a time and cuts each
// at 2^-13 of the largest one's exponent before they join an fp32 sum (measured, with single products at every place and
// size): at most 7 * 2^-13 of the largest of every eight, 1.5e-5 of y where inputs are normal, against a half step of
// 2^-9 by which y is rounded.  For y in fp32 that would show, so the bytes are widened to bf16, which holds them exactly,
// and the sum taken on v_mfma_f32_16x16x32_bf16 (6e-8 of y), whose rate is half.
//
// Operand layout of the 16x16x128 product, for lane l: row l % 16 and 32 bytes of the block, the same ones of both operands.
// The bf16 products take them eight at a time.
#include <hip/hip_runtime.h>
#include <algorithm>
#include <type_traits>

#include "layer_launch.hpp"
#include "ssd_device.hpp"

namespace ssd {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
union Bytes {                                       // a lane's 32 bytes of a block
    u32x4_t h[2];
    uint32_t u[8];
    i32x8 v;
};
// an operand of the inner sum, and the sum
template <typename T> struct Frag;
template <> struct Frag<uint16_t> {
    i32x8 v;
    __device__ __forceinline__ explicit Frag(const Bytes& b) : v(b.v) {}
};
template <> struct Frag<float> {
    bf16x8 v[4];
    __device__ __forceinline__ explicit Frag(const Bytes& b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const auto two = j & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b.u[2 * i + j / 2], 1.0f, true)
                                       : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b.u[2 * i + j / 2], 1.0f, false);
                v[i][2 * j] = two[0];
                v[i][2 * j + 1] = two[1];
            }
        }
    }
};
__device__ __forceinline__ f32x4 inner(const Frag<uint16_t>& a, const Frag<uint16_t>& b) {
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, zero, 0, 0, 0, 0, 0, 0);    // both e4m3, no block scales
}
__device__ __forceinline__ f32x4 inner(const Frag<float>& a, const Frag<float>& b) {
    f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], d, 0, 0, 0);
    return d;
}

// four neighbouring columns of a row of y; `wide`: rows and bases on four elements
__device__ __forceinline__ void store4(float* p, int left, bool wide, f32x4 v) {
    if (wide && left >= 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = v[i];
}
__device__ __forceinline__ void store4(uint16_t* p, int left, bool wide, f32x4 v) {
    if (wide && left >= 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = (uint16_t)f32_to_bf16_bits(v[i]);
}

// ------------------------------------------------------------ few rows: weights streamed from HBM into registers
// A workgroup owns 16 columns of y and 16 MT rows; its four waves take every fourth block of K and their sums meet in
// LDS, in order.  The weights' bytes are the work: nothing is staged, a lane's 32 bytes of a block are two loads, and U
// blocks are on their way at once.  M = 4, N = 5152, K = 2048 to bf16: 5.7 us (10.6 MB; a copy of as much 2.0 us and a launch
// 2 to 3).  Eight waves: the same there, M = 16, N = 1024, K = 8192 11.4 in place of 11.7.
constexpr int kSkinnyWaves = 4;
template <typename T, int MT, int U>
__global__ __launch_bounds__(64 * kSkinnyWaves) void ssd_proj_rows_kernel(ProjArgs p) {
    __shared__ f32x4 part[kSkinnyWaves][MT][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64, i = l % 16, g = l / 16;
    const int tn = (p.N + 15) / 16, n0 = blockIdx.x % tn * 16, m0 = blockIdx.x / tn * 16 * MT;
    const int blocks = (p.K + 127) / 128;
    const uint8_t* w = p.w + (int64_t)min(n0 + i, p.N - 1) * p.w_stride;
    const uint8_t* a[MT];
    const float* as[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t row = min(m0 + 16 * t + i, p.M - 1);
        a[t] = p.a + row * p.a_stride;
        as[t] = p.a_scale + row * p.a_scale_stride;
    }
    const float* ws = p.w_scale + (int64_t)(n0 / 128) * p.w_scale_stride;
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int b0 = wave; b0 < blocks; b0 += kSkinnyWaves * U) {
        Bytes fw[U], fa[U][MT];
        float s[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u * kSkinnyWaves;
            if (b >= blocks) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // past K the row's last bytes stand in, against activations of 0
                const int k = b * 128 + g * 32 + h * 16, kc = min(k, p.K - 16);
                fw[u].h[h] = *reinterpret_cast<const u32x4_t*>(w + kc);
#pragma unroll
                for (int t = 0; t < MT; ++t) fa[u][t].h[h] = *reinterpret_cast<const u32x4_t*>(a[t] + kc);
            }
            const float sw = ws[b];
#pragma unroll
            for (int t = 0; t < MT; ++t) s[u][t] = as[t][b] * sw;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u * kSkinnyWaves;
            if (b >= blocks) break;
            if (b * 128 + 128 > p.K) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (b * 128 + g * 32 + h * 16 >= p.K) {
#pragma unroll
                        for (int t = 0; t < MT; ++t) fa[u][t].h[h] = u32x4_t{0, 0, 0, 0};
                    }
            }
            const Frag<T> wide(fw[u]);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const f32x4 d = inner(wide, Frag<T>(fa[u][t]));
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(d[e], s[u][t], acc[t][e]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][t][l] = acc[t];
    __syncthreads();
    if (wave >= MT) return;
    f32x4 v = part[0][wave][l];
#pragma unroll
    for (int k = 1; k < kSkinnyWaves; ++k) v += part[k][wave][l];
    const int m = m0 + 16 * wave + i, n = n0 + 4 * g;
    if (m < p.M && n < p.N) store4(static_cast<T*>(p.y) + (int64_t)m * p.y_stride + n, p.N - n, p.wide, v);
}

// ------------------------------------------------------------ many rows: tiles through LDS
// LDS DMA, 16 bytes a lane to lds + 16 l (4 bytes to lds + 4 l), written so that the compiler does not model it (it would
// wait for every copy in flight before each LDS read); base and lds are the wave's.
#define SSD_DMA(width)                                                                                           \
    uint32_t m0_saved;                                                                                           \
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_" width " %1, %2\n\ts_mov_b32 m0, %0" \
                 : "=&s"(m0_saved)                                                                               \
                 : "v"(voff), "s"(base), "s"(lds)                                                                \
                 : "memory")
__device__ __forceinline__ void dma16(const void* base, uint32_t voff, uint32_t lds) { SSD_DMA("dwordx4"); }
__device__ __forceinline__ void dma4(const void* base, uint32_t voff, uint32_t lds) { SSD_DMA("dword"); }
#undef SSD_DMA

// Byte of piece c (16 bytes) of row r in a tile of 128-byte rows: sixteen rows at one piece fall on sixteen different
// sixteenths of the LDS banks.
__device__ __forceinline__ uint32_t at(int r, int c) { return (uint32_t)(r * 128 + ((c ^ ((r >> 1) & 7)) << 4)); }
// The h-th piece of a block that lane group g holds (the same of both operands, so that any assignment will do).  A 16-byte
// LDS read takes sixteen lanes a clock, and not sixteen neighbours: eight rows of one group go with the other eight rows
// of the next, whose piece differs in the last bit only, which at() keeps apart.  (With pieces 2 g and 2 g + 1 every read
// took twice as long.)
__device__ __forceinline__ int piece_of(int g, int h) { return (g & 1) | h << 1 | (g >> 1) << 2; }

// A workgroup of NWN x NWM waves owns a tile of y; a wave's part of it is WN x WM products of 16 x 16.  The two operands'
// block of 128 bytes a row goes through one of two LDS stages while the other is computed, and so do the activations'
// scales of 16 blocks at a time: read by the lanes that need them, they would be as many requests as the operands.
// M = 16384, N = 4096, K = 8192 to bf16: 472 to 495 us, 2.33 to 2.22 PFLOP/s (to fp32, tiles of 128 x 128: 943); a library's 8-bit product without block scales
// takes 412 us there.  Matrix instructions alone would take 300 us at the clock they leave, with their LDS reads and barriers 405;
// copies and scales add the rest, and the scales' fmas nothing.  A row of products is scaled while the next one's run (one
// after the other: 666 us).
// KG groups of waves take every KG-th block each, in stages of their own, and their sums meet in LDS: in a small tile a wave's
// steps of a block are a chain that nothing else covers (64 x 64 of K = 4096: 14.2 us with one group and four stages, 11.0
// with two groups of two; 256 x 4096 x 4096 16.0 and 13.3).  Four groups: 9.9 and 12.5, 128 x 8192 x 8192 23.7 in place of 29.4,
// but 512 x 4096 x 4096, where a CU has two workgroups, 24.4 in place of 19.5.
template <int BN, int BM, int KG> constexpr int kTileLds = KG * 2 * (BN + BM) * 128 + 2 * BM * 16 * 4;
template <typename T, int WN, int WM, int NWN, int NWM, int KG>
__global__ __launch_bounds__(64 * NWN * NWM * KG, 2) void ssd_proj_tiles_kernel(ProjArgs p) {
    constexpr int NW = NWN * NWM, BN = 16 * WN * NWN, BM = 16 * WM * NWM, kStage = (BN + BM) * 128;
    constexpr int kCopies = (BN + BM) / 8 / NW;     // of a wave: 8 rows each
    constexpr int kPerRow = (2 * kCopies + WN - 1) / WN;      // copies beside a row of products: all in a block's first half
    static_assert(kCopies * 8 * NW == BN + BM && 128 % (16 * WN) == 0 && WM == 4 && 16 % KG == 0, "tile");
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int l = threadIdx.x % 64, i = l % 16, g = l / 16, any = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wave = any % NW, group = any / NW;
    const int wn = wave % NWN, wm = wave / NWN;
    // tiles of y in an order that keeps an XCD's workgroups (every eighth of the launch) on neighbouring tiles: panels of
    // 8 tiles of rows, column by column
    const int tn = (p.N + BN - 1) / BN, tm = (p.M + BM - 1) / BM, total = tn * tm;
    int id = blockIdx.x;
    const int per = total / 8;
    if (id < per * 8) id = id % 8 * per + id / 8;
    const int panel = id / (8 * tn), rows = min(8, tm - panel * 8), in = id - panel * 8 * tn;
    const int n0 = in / rows * BN, m0 = (panel * 8 + in % rows) * BM;

    const int blocks = (p.K + 127) / 128;
    // What a wave copies: kCopies times 8 rows, of the weights or (the later waves) the activations; lane l the piece at
    // place l % 8 of the l / 8-th.  Rows past the operand's last are that one; where there are none, an 8-row step is a
    // scalar's and a lane's offset is one register.
    static_assert(kCopies % 2 == 0 && BN % (8 * kCopies) == 0, "a wave copies rows of one operand");
    const int piece0 = 16 * ((l % 8) ^ (l >> 4));   // at(): (r >> 1) & 7 = 4 (j & 1) + l / 16
    const int row0 = 8 * wave * kCopies;
    const bool of_w = row0 < BN;
    const uint8_t* base = of_w ? p.w + (int64_t)(n0 + row0) * p.w_stride : p.a + (int64_t)(m0 + row0 - BN) * p.a_stride;
    const int most = of_w ? p.N - 1 - n0 - row0 : p.M - 1 - m0 - (row0 - BN);     // rows of the operand after row0
    const uint32_t row_bytes = (uint32_t)(of_w ? p.w_stride : p.a_stride);
    const bool whole = most >= 8 * kCopies - 1;
    if (most < 0) base += (int64_t)most * row_bytes;                              // row0 itself is past the last
    const uint32_t lane_off = (uint32_t)(l / 8) * row_bytes;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
    auto stage_of = [&](int b) { return (group * 2 + (b / KG & 1)) * kStage; };
    // the wave's j-th copy of block b
    auto copy = [&](int b, int j, auto full) {
        const uint32_t k = (uint32_t)min(b * 128 + (j & 1 ? piece0 ^ 64 : piece0), p.K - 16);
        const uint32_t to = lds0 + stage_of(b) + wave * kCopies * 1024 + j * 1024;
        if constexpr (decltype(full)::value) dma16(base + (size_t)(8 * j) * row_bytes, lane_off + k, to);
        else dma16(base, (uint32_t)min(8 * j + l / 8, max(most, 0)) * row_bytes + k, to);
    };
    // the scales of blocks 16 q .. + 15 go to rows of 16, block c of row r at place c ^ (r % 16): sixteen rows' scales of one
    // block are in sixteen banks.  Rows of at most 2^24 bytes, 255 of them: offsets fit 32 bits.
    constexpr int kScales = KG * 2 * kStage, kScaleCopies = BM / 4 / NW;       // of a wave: 4 rows each
    static_assert(kScaleCopies * 4 * NW == BM, "scales");
    const char* as = reinterpret_cast<const char*>(p.a_scale + (int64_t)m0 * p.a_scale_stride);
    auto copy_scales = [&](int q) {
#pragma unroll
        for (int j = 0; j < kScaleCopies; ++j) {
            const int first = 4 * (wave * kScaleCopies + j), r = first + g;
            const uint32_t row = (uint32_t)min(r, p.M - 1 - m0) * (uint32_t)(p.a_scale_stride * 4);
            dma4(as, row + 4 * (uint32_t)min(16 * q + (i ^ (r & 15)), blocks - 1), lds0 + kScales + (q & 1) * BM * 64 + first * 64);
        }
    };
    // of the wave's rows, block b
    auto a_scale = [&](int b, int t) {
        return *reinterpret_cast<const float*>(lds + kScales + (b >> 4 & 1) * BM * 64 + (16 * (wm * WM + t) + i) * 64 + ((b & 15) ^ i) * 4);
    };
    const float* ws = p.w_scale + (int64_t)(min(n0 + 16 * wn * WN, p.N - 1) / 128) * p.w_scale_stride;

    f32x4 acc[WN][WM], d[WM];                       // d: inner sums of a row of products, until the next row's take their place
#pragma unroll
    for (int t = 0; t < WM; ++t) {
        d[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < WN; ++u) acc[u][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    float s[WM], last[WM], nw = ws[min(group, blocks - 1)];
#pragma unroll
    for (int t = 0; t < WM; ++t) s[t] = 0.0f;
    if (group == 0) copy_scales(0);
    const int steps = (blocks + KG - 1) / KG;        // of every group; a last one past the last block adds 0
#pragma unroll
    for (int j = 0; j < kCopies; ++j) copy(group, j, std::false_type{});
    auto block = [&](int b, auto more, auto full) {
        constexpr bool MORE = decltype(more)::value;
        // this wave's copies of block b have landed, and then everyone's; the other stage has been read by all
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int t = 0; t < WM; ++t) {
            last[t] = s[t];
            s[t] = a_scale(b, t) * nw;
            if (!MORE && KG > 1 && b >= blocks) s[t] = 0.0f;
        }
        if (MORE) {
            nw = ws[KG == 1 ? b + 1 : min(b + KG, blocks - 1)];
            if (b % 16 == 0) copy_scales(b / 16 + 1);            // group 0's: KG divides 16
        }
        const uint8_t* stage = lds + stage_of(b);
        auto weights = [&](int u) {
            Bytes w;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w.h[h] = *reinterpret_cast<const u32x4_t*>(stage + at(16 * (wn * WN + u) + i, piece_of(g, h)));
            return w;
        };
        Bytes bw = weights(0), ba[WM];
#pragma unroll
        for (int t = 0; t < WM; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                ba[t].h[h] = *reinterpret_cast<const u32x4_t*>(stage + BN * 128 + at(16 * (wm * WM + t) + i, piece_of(g, h)));
        if (!MORE && b * 128 + 128 > p.K) {          // past K the row's last bytes stand in, against activations of 0
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (b * 128 + piece_of(g, h) * 16 >= p.K) {
#pragma unroll
                    for (int t = 0; t < WM; ++t) ba[t].h[h] = u32x4_t{0, 0, 0, 0};
                }
        }
        Frag<T> fa[WM] = {Frag<T>(ba[0]), Frag<T>(ba[1]), Frag<T>(ba[2]), Frag<T>(ba[3])};
#pragma unroll
        for (int u = 0; u < WN; ++u) {
            if (sizeof(T) == 2) __builtin_amdgcn_sched_barrier(0);      // a row at a time: the registers
            const Frag<T> fw(bw);
            if (u + 1 < WN) bw = weights(u + 1);
            if (MORE) {
#pragma unroll
                for (int j = u * kPerRow; j < min((u + 1) * kPerRow, kCopies); ++j) copy(b + KG, j, full);
            }
            // the products of this row while the last row's are scaled and added
#pragma unroll
            for (int t = 0; t < WM; ++t) {
                f32x4& to = acc[u ? u - 1 : WN - 1][t];
                const float f = u ? s[t] : last[t];
#pragma unroll
                for (int e = 0; e < 4; ++e) to[e] = fmaf(d[t][e], f, to[e]);
                d[t] = inner(fw, fa[t]);
                if (!MORE) asm volatile("" : "+v"(to));      // here: the compiler would hold d for additions at the stores
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);                           // vector
                __builtin_amdgcn_sched_group_barrier(0x008, sizeof(T) == 2 ? 1 : 4, 0);      // matrix
            }
        }
    };
    const int end = (steps - 1) * KG + group;
    if (whole)
        for (int b = group; b < end; b += KG) block(b, std::true_type{}, std::true_type{});
    else
        for (int b = group; b < end; b += KG) block(b, std::true_type{}, std::false_type{});
    block(end, std::false_type{}, std::false_type{});
#pragma unroll
    for (int t = 0; t < WM; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[WN - 1][t][e] = fmaf(d[t][e], s[t], acc[WN - 1][t][e]);
#pragma unroll
    for (int t = 0; t < WM; ++t) asm volatile("" : "+v"(acc[WN - 1][t]));
    if constexpr (KG > 1) {                          // the groups' sums, in order; the stages have been read by all
        f32x4* sums = reinterpret_cast<f32x4*>(lds);
        __syncthreads();
        if (group) {
#pragma unroll
            for (int t = 0; t < WM; ++t)
#pragma unroll
                for (int u = 0; u < WN; ++u) sums[(((group - 1) * NW + wave) * WN * WM + t * WN + u) * 64 + l] = acc[u][t];
        }
        __syncthreads();
        if (group) return;
#pragma unroll
        for (int k = 0; k < KG - 1; ++k)
#pragma unroll
            for (int t = 0; t < WM; ++t)
#pragma unroll
                for (int u = 0; u < WN; ++u) acc[u][t] += sums[((k * NW + wave) * WN * WM + t * WN + u) * 64 + l];
    }
    T* y = static_cast<T*>(p.y);
#pragma unroll
    for (int t = 0; t < WM; ++t) {
        const int m = m0 + 16 * (wm * WM + t) + i;
        if (m >= p.M) continue;
#pragma unroll
        for (int u = 0; u < WN; ++u) {
            const int n = n0 + 16 * (wn * WN + u) + 4 * g;
            if (n < p.N) store4(y + (int64_t)m * p.y_stride + n, p.N - n, p.wide, acc[u][t]);
        }
    }
}

template <typename T, int MT, int U>
hipError_t rows(const ProjArgs& p, hipStream_t s) {
    const int64_t n = (int64_t)((p.N + 15) / 16), m = (int64_t)((p.M + 16 * MT - 1) / (16 * MT));
    const dim3 grid((unsigned)(n * m));
    hipLaunchKernelGGL((ssd_proj_rows_kernel<T, MT, U>), grid, dim3(64 * kSkinnyWaves), 0, s, p);
    return hipGetLastError();
}
template <typename T, int WN, int WM, int NWN, int NWM, int KG>
hipError_t tiles(const ProjArgs& p, hipStream_t s) {
    constexpr int BN = 16 * WN * NWN, BM = 16 * WM * NWM, lds = kTileLds<BN, BM, KG>;
    const auto kernel = &ssd_proj_tiles_kernel<T, WN, WM, NWN, NWM, KG>;
    if (hipError_t e = prepare_launch(reinterpret_cast<const void*>(kernel), lds)) return e;
    const int64_t n = (int64_t)((p.N + BN - 1) / BN) * ((p.M + BM - 1) / BM);
    hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(64 * NWN * NWM * KG), lds, s, p);
    return hipGetLastError();
}

// The kernel by its estimated time in us, from sweeps of M, N and K (256 CUs, one workgroup each before any has two):
//  - rows: a workgroup reads 16 rows of w and 16 MT of a, 2 KB a block each, at some 28 bytes a ns and CU (a CU's lines on
//    their way), 40 where an XCD's 4 MB of L2 hold the weights; 3 us around it.
//  - tiles of 64 x 64, K in two groups: 0.24 to 0.31 us a block (0.4 to 0.5 with widened operands), the chain of a block's
//    steps; 3.5 us.
//  - tiles of 128 x 128: 0.5 to 0.8 us a block (1.1 to 1.25) as the CUs fill; 5 us.
//  - tiles of 256 x 256, one a CU: 1.85 us a block, against 0.7 a 128 x 128 tile when there are many.
// Measured, us, in that order (rows: the better MT; -: not built):
//   bf16  M = 32, N = K = 4096        9.8  11.4  20    42      fp32  M = 777, N = 1000, K = 1040  10.2   8.5  15.9   -
//         M = 64, N = 5152, K = 2048   13   8.5  12.3  24            M = 300, N = K = 2048        20.6  10.7  23.3   -
//         M = 16, N = 1024, K = 8192   11    19    37  78            M = 512, N = K = 4096         115  31.3  41.6   -
//         M = 256, N = K = 4096        59  13.3  21.7  48      bf16  M = 4096, N = 5152, K = 2048    -     -    60  64
//         M = 512, N = K = 4096       115    19    28  49            M = N = K = 4096                -     -    95  66
//         M = 800, N = K = 4096         -    35    29  50            M = 2000, N = 8192, K = 256     53    29    18  17
// The answer is the rows of y that a workgroup computes; each number is one kernel.
enum : int { kRows16 = 16, kRows32 = 32, kTiles64 = 64, kTiles128 = 128, kTiles256 = 256 };
int choose(int M, int N, int K, bool wide) {         // wide: widened operands
    const auto over = [](double n, int d) { return (double)(((int64_t)n + d - 1) / d); };
    const auto more = [](double n) { return std::max(0.0, n / 256 - 1.0); };      // workgroups a CU after the first
    const double blocks = over(K, 128), n16 = over(N, 16), t64 = over(N, 64) * over(M, 64), t128 = over(N, 128) * over(M, 128);
    const double piece = (int64_t)N * K <= 4 << 20 ? 0.05 : 0.073, most = 0xffffffffu;          // threads that a launch counts
    double best = 5.0 + blocks * (wide ? 1.1 + 0.15 * std::min(1.0, t128 / 256) + 0.9 * more(t128)
                                       : 0.5 + 0.3 * std::min(1.0, t128 / 256) + 0.6 * more(t128));
    int kind = kTiles128;
    const auto consider = [&](int k, double t, double threads) {
        if (t >= best || threads > most) return;
        kind = k;
        best = t;
    };
    consider(kTiles64, 3.5 + blocks * (wide ? 0.4 + 0.09 * std::min(1.0, t64 / 256) + 0.5 * more(t64)
                                           : 0.24 + 0.07 * std::min(1.0, t64 / 256) + 0.3 * more(t64)), t64 * 512);
    for (int k : {1, 2}) {
        const double wgs = n16 * over(M, 16 * k);
        consider(k == 1 ? kRows16 : kRows32, 3.0 + blocks * piece * (1 + k) * (1.0 + more(wgs)), wgs * 64 * kSkinnyWaves);
    }
    // widened operands take too many registers for the largest tile
    if (kind == kTiles128 && !wide && over(over(N, 256) * over(M, 256), 256) * 1.85 < 0.7 * t128 / 256) return kTiles256;
    return kind;
}
template <typename T>
hipError_t proj_t(const ProjArgs& p, hipStream_t s) {
    constexpr bool kWide = sizeof(T) == 4;
    const int kind = choose(p.M, p.N, p.K, kWide);
    if (kind == kRows16) return rows<T, 1, 4>(p, s);
    if (kind == kRows32) return rows<T, 2, 2>(p, s);
    if (kind == kTiles64) return tiles<T, 1, 4, 4, 1, 2>(p, s);
    if constexpr (!kWide) {
        if (kind == kTiles256) return tiles<T, 8, 4, 2, 4, 1>(p, s);
    }
    return tiles<T, 4, 4, 2, 2, 1>(p, s);
}

}  // namespace

int proj_tile_rows(int M, int N, int K, int dtype) { return choose(M, N, K, dtype == 0); }
hipError_t launch_proj(const ProjArgs& p, hipStream_t s) { return p.dtype == 0 ? proj_t<float>(p, s) : proj_t<uint16_t>(p, s); }

}  // namespace ssd

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
// Operand layout of the 16x16x128 product, for lane l: row l % 16, bytes 32 (l / 16) .. + 32 of the block.  The bf16
// products take the same bytes eight at a time: only that both operands agree matters.
#include <hip/hip_runtime.h>
#include <algorithm>
#include <type_traits>

#include "ssd_device.hpp"
#include "ssd_launch.hpp"

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
// A workgroup owns 16 columns of y and 16 MT rows; its eight waves take every eighth block of K and their sums meet in
// LDS, in order.  The weights' bytes are the work: nothing is staged, a lane's 32 bytes of a block are two loads, and U
// blocks are on their way at once.
constexpr int kSkinnyWaves = 8;
template <typename T, int MT, int U>
__global__ __launch_bounds__(64 * kSkinnyWaves) void ssd_proj_rows_kernel(ProjArgs p) {
    __shared__ f32x4 part[kSkinnyWaves][MT][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64, i = l % 16, g = l / 16;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MT;
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
// LDS DMA, 16 bytes a lane to lds + 16 l, written so that the compiler does not model it (it would wait for every copy in
// flight before each LDS read); base and lds are the wave's.
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t voff, uint32_t lds) {
    uint32_t m0_saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %3\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, %2\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(m0_saved)
        : "v"(voff), "s"(base), "s"(lds)
        : "memory");
}

// Byte of piece c (16 bytes) of row r in a tile of 128-byte rows: sixteen rows at one piece fall on sixteen different
// sixteenths of the LDS banks.
__device__ __forceinline__ uint32_t at(int r, int c) { return (uint32_t)(r * 128 + ((c ^ ((r >> 1) & 7)) << 4)); }

// A workgroup of NWN x NWM waves owns a tile of y; a wave's part of it is WN x WM products of 16 x 16.  The two operands'
// block of 128 bytes a row goes through one of two LDS stages while the other is computed.
template <typename T, int WN, int WM, int NWN, int NWM>
__global__ __launch_bounds__(64 * NWN * NWM, 2) void ssd_proj_tiles_kernel(ProjArgs p) {
    constexpr int NW = NWN * NWM, BN = 16 * WN * NWN, BM = 16 * WM * NWM, kStage = (BN + BM) * 128;
    constexpr int kCopies = (BN + BM) / 8 / NW;     // of a wave: 8 rows each
    static_assert(kCopies * 8 * NW == BN + BM && 128 % (16 * WN) == 0 && WM == 4, "tile");
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64, i = l % 16, g = l / 16;
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
    // what a lane copies: piece c of row 8 j + l / 8 for the wave's j-th copy, weights first
    static_assert(kCopies % 2 == 0, "the place of a lane's piece goes by j's parity");
    uint32_t row_off[kCopies];
    const uint8_t* base[kCopies];
    const int piece0 = 16 * ((l % 8) ^ (l >> 4));   // at(): (r >> 1) & 7 = 4 (j & 1) + l / 16
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
        const int first = 8 * (wave * kCopies + j), r = first + l / 8;
        if (first < BN) {
            base[j] = p.w + (int64_t)n0 * p.w_stride;
            row_off[j] = (uint32_t)min(r, p.N - 1 - n0) * (uint32_t)p.w_stride;
        } else {
            base[j] = p.a + (int64_t)m0 * p.a_stride;
            row_off[j] = (uint32_t)min(r - BN, p.M - 1 - m0) * (uint32_t)p.a_stride;
        }
    }
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
    // the wave's j-th copy of block b
    auto copy = [&](int b, int j) {
        dma16(base[j], row_off[j] + (uint32_t)min(b * 128 + (j & 1 ? piece0 ^ 64 : piece0), p.K - 16),
              lds0 + (b & 1) * kStage + wave * kCopies * 1024 + j * 1024);
    };
    // rows of the activations' scales: 255 of at most 2^24 bytes each fit 32 bits
    uint32_t as_off[WM];
#pragma unroll
    for (int t = 0; t < WM; ++t)
        as_off[t] = (uint32_t)min(16 * (wm * WM + t) + i, p.M - 1 - m0) * (uint32_t)(p.a_scale_stride * 4);
    const char* as = reinterpret_cast<const char*>(p.a_scale + (int64_t)m0 * p.a_scale_stride);
    auto a_scale = [&](int b, int t) { return *reinterpret_cast<const float*>(as + (size_t)b * 4 + as_off[t]); };
    const float* ws = p.w_scale + (int64_t)(min(n0 + 16 * wn * WN, p.N - 1) / 128) * p.w_scale_stride;

    f32x4 acc[WN][WM], d[2][WM];                    // d: inner sums, one row of products behind its addition to acc
#pragma unroll
    for (int t = 0; t < WM; ++t) {
        d[1][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < WN; ++u) acc[u][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    static_assert(WN % 2 == 0, "the last row of products is d[1]");
    float next[WM], s[WM], last[WM], nw = ws[0];
#pragma unroll
    for (int t = 0; t < WM; ++t) {
        next[t] = a_scale(0, t);
        s[t] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < kCopies; ++j) copy(0, j);
    auto block = [&](int b, auto more) {
        constexpr bool MORE = decltype(more)::value;
#pragma unroll
        for (int t = 0; t < WM; ++t) {
            last[t] = s[t];
            s[t] = next[t] * nw;
        }
        // this wave's copies of block b have landed, and then everyone's; the other stage has been read by all
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (MORE) {
            nw = ws[b + 1];
#pragma unroll
            for (int t = 0; t < WM; ++t) next[t] = a_scale(b + 1, t);
        }
        const uint8_t* stage = lds + (b & 1) * kStage;
        auto weights = [&](int u) {
            Bytes w;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w.h[h] = *reinterpret_cast<const u32x4_t*>(stage + at(16 * (wn * WN + u) + i, 2 * g + h));
            return w;
        };
        Bytes bw = weights(0), ba[WM];
#pragma unroll
        for (int t = 0; t < WM; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                ba[t].h[h] = *reinterpret_cast<const u32x4_t*>(stage + BN * 128 + at(16 * (wm * WM + t) + i, 2 * g + h));
        if (!MORE && b * 128 + 128 > p.K) {          // past K the row's last bytes stand in, against activations of 0
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (b * 128 + g * 32 + h * 16 >= p.K) {
#pragma unroll
                    for (int t = 0; t < WM; ++t) ba[t].h[h] = u32x4_t{0, 0, 0, 0};
                }
        }
        Frag<T> fa[WM] = {Frag<T>(ba[0]), Frag<T>(ba[1]), Frag<T>(ba[2]), Frag<T>(ba[3])};
#pragma unroll
        for (int u = 0; u < WN; ++u) {
            const Frag<T> fw(bw);
            if (u + 1 < WN) bw = weights(u + 1);
            if (MORE) {
#pragma unroll
                for (int j = u * kCopies / WN; j < (u + 1) * kCopies / WN; ++j) copy(b + 1, j);
            }
            // the products of this row while the last row's are scaled and added
#pragma unroll
            for (int t = 0; t < WM; ++t) {
                d[u & 1][t] = inner(fw, fa[t]);
                const f32x4 v = d[1 - (u & 1)][t];
                f32x4& to = acc[u ? u - 1 : WN - 1][t];
                const float f = u ? s[t] : last[t];
#pragma unroll
                for (int e = 0; e < 4; ++e) to[e] = fmaf(v[e], f, to[e]);
                if (!MORE) asm volatile("" : "+v"(to));      // here: the compiler would hold d for additions at the stores
                __builtin_amdgcn_sched_group_barrier(0x008, sizeof(T) == 2 ? 1 : 4, 0);      // matrix
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);                           // vector
            }
        }
    };
    for (int b = 0; b + 1 < blocks; ++b) block(b, std::true_type{});
    block(blocks - 1, std::false_type{});
#pragma unroll
    for (int t = 0; t < WM; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[WN - 1][t][e] = fmaf(d[1][t][e], s[t], acc[WN - 1][t][e]);
#pragma unroll
    for (int t = 0; t < WM; ++t) asm volatile("" : "+v"(acc[WN - 1][t]));
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
    const dim3 grid((p.N + 15) / 16, (p.M + 16 * MT - 1) / (16 * MT));
    hipLaunchKernelGGL((ssd_proj_rows_kernel<T, MT, U>), grid, dim3(64 * kSkinnyWaves), 0, s, p);
    return hipGetLastError();
}
template <typename T, int WN, int WM, int NWN, int NWM>
hipError_t tiles(const ProjArgs& p, hipStream_t s) {
    constexpr int BN = 16 * WN * NWN, BM = 16 * WM * NWM, lds = 2 * (BN + BM) * 128;
    const auto kernel = &ssd_proj_tiles_kernel<T, WN, WM, NWN, NWM>;
    if (hipError_t e = prepare_launch(reinterpret_cast<const void*>(kernel), lds)) return e;
    const int64_t n = (int64_t)((p.N + BN - 1) / BN) * ((p.M + BM - 1) / BM);
    hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(64 * NWN * NWM), lds, s, p);
    return hipGetLastError();
}

template <typename T>
hipError_t proj_t(const ProjArgs& p, hipStream_t s) {
    if (p.M <= 16) return rows<T, 1, 4>(p, s);
    if (p.M <= 32) return rows<T, 2, 2>(p, s);
    if (p.M <= 256) return rows<T, 4, 2>(p, s);
    if ((int64_t)((p.N + 255) / 256) * ((p.M + 255) / 256) >= 192) {
        if constexpr (sizeof(T) == 2) return tiles<T, 8, 4, 2, 4>(p, s);
        else return tiles<T, 4, 4, 2, 4>(p, s);     // widened operands take twice the registers
    }
    if constexpr (sizeof(T) == 2) return tiles<T, 4, 4, 2, 2>(p, s);
    else return tiles<T, 2, 4, 4, 2>(p, s);
}

}  // namespace

hipError_t launch_proj(const ProjArgs& p, hipStream_t s) { return p.dtype == 0 ? proj_t<float>(p, s) : proj_t<uint16_t>(p, s); }

}  // namespace ssd

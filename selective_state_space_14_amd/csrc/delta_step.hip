// delta_step.hip -- one token of the gated delta rule for each of B sequences.
//
//   a = exp(dt A);  u = beta (v - a S k);  S' = a S + u k^T;  y = scale S' q
// with S the head's state [P][N], k and q its group's rows (of unit length
// with qk_norm).  S' q = a (S q) + u (k . q), so a row of S gives both of its
// products in one pass and is written back from the registers it was read to:
// the state's bytes, read and written once, are the whole cost.
//
// A row of S lies in N / 4 lanes, four entries each, so a wave reads whole
// 256-byte lines; each lane holds its four entries of k and q for every row.
// A thread takes F rows' parts, all loaded before the first is used.
//
// Measured: B=256 H=64 N=128, 1.07 GB read and written, 178 us (6.0 TB/s; a
// large copy reaches 5.1).  B=1 H=32 N=64: 3.6 us on the GPU, the call's host time more.
#include <hip/hip_runtime.h>

#include "ssd_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const uint16_t* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
}
__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16_bits(v); }
__device__ __forceinline__ float dot4(float4 a, float4 b) {
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, a.x * b.x)));
}

template <typename T, int N, int F, bool STREAM>
__global__ __launch_bounds__(kThreads) void ssd_delta_step_kernel(DeltaArgs a) {
    constexpr int NQ = N / 4;                       // lanes of a state row
    constexpr int kRows = kThreads / NQ;            // state rows of the workgroup at a time
    const int tiles = a.P / (kRows * F);            // workgroups of a head
    const int bh = blockIdx.x / tiles;
    const int p0 = (blockIdx.x % tiles) * kRows * F + threadIdx.x / NQ;
    const int b = bh / a.H, h = bh % a.H;
    const int n0 = (threadIdx.x % NQ) * 4;
    const int g = h / (a.H / a.G);

    float* S = a.final_state + ((size_t)bh * a.P + p0) * N + n0;
    float4 s[F];
    float vv[F];
    const T* vrow = static_cast<const T*>(a.v) + (size_t)b * a.v_stride + (size_t)h * a.P + p0;
#pragma unroll
    for (int f = 0; f < F; ++f) {
        const f32x4* at = reinterpret_cast<const f32x4*>(S + (size_t)f * kRows * N);
        const f32x4 z = STREAM ? __builtin_nontemporal_load(at) : *at;
        s[f] = make_float4(z[0], z[1], z[2], z[3]);
        vv[f] = ld1(vrow + f * kRows);
    }
    float4 q = ld4(static_cast<const T*>(a.q) + (size_t)b * a.q_stride + (size_t)g * N + n0);
    float4 k = ld4(static_cast<const T*>(a.k) + (size_t)b * a.k_stride + (size_t)g * N + n0);
    float dt = a.dt[(size_t)b * a.dt_stride + h];
    float beta = a.beta[(size_t)b * a.beta_stride + h];
    if (a.dt_softplus) dt = softplus_f(dt + (a.dt_bias ? a.dt_bias[h] : 0.0f));
    if (a.beta_sigmoid) beta = 1.0f / (1.0f + expf(-beta));
    const float dec = expf(dt * a.A[h]);
    float qs = a.scale;
    if (a.qk_norm) {
        const float rk = 1.0f / sqrtf(lanes_sum<NQ>(dot4(k, k)) + kQkEps);
        k = make_float4(k.x * rk, k.y * rk, k.z * rk, k.w * rk);
        qs *= 1.0f / sqrtf(lanes_sum<NQ>(dot4(q, q)) + kQkEps);
    }
    const float kq = lanes_sum<NQ>(dot4(k, q));
    T* yrow = static_cast<T*>(a.y) + (size_t)b * a.y_stride + (size_t)h * a.P + p0;
#pragma unroll
    for (int f = 0; f < F; ++f) {
        const float sk = lanes_sum<NQ>(dot4(s[f], k)), sq = lanes_sum<NQ>(dot4(s[f], q));
        const float u = beta * (vv[f] - dec * sk);
        const f32x4 o = {fmaf(dec, s[f].x, u * k.x), fmaf(dec, s[f].y, u * k.y), fmaf(dec, s[f].z, u * k.z), fmaf(dec, s[f].w, u * k.w)};
        f32x4* to = reinterpret_cast<f32x4*>(S + (size_t)f * kRows * N);
        if (STREAM) __builtin_nontemporal_store(o, to);
        else *to = o;
        if (n0 == 0) st1(yrow + f * kRows, qs * fmaf(dec, sq, u * kq));
    }
}

template <typename T, int N>
hipError_t launch_n(const DeltaArgs& a, hipStream_t stream) {
    // the most rows a thread that leave 1024 workgroups, four on every CU.  Measured: the 1.07 GB of B=256 H=64 N=128,
    // past the last-level cache, take 179 us with F = 8, 178 with 4 and 214 to 218 with 1; B=1 H=32 N=64 3.9 us with F = 1
    // and 4.1 with 4
    const int64_t work = (int64_t)a.B * a.H * a.P * N / (kThreads * 4);   // workgroups at F = 1
    const int most = a.P * N / (kThreads * 4);                            // F of a whole head: >= 2
    int f = 8;
    while (f > 1 && (f > most || work / f < 1024)) f /= 2;
    const dim3 grid((unsigned)(work / f));
    switch (f) {
        case 1: hipLaunchKernelGGL((ssd_delta_step_kernel<T, N, 1, false>), grid, dim3(kThreads), 0, stream, a); break;
        case 2: hipLaunchKernelGGL((ssd_delta_step_kernel<T, N, 2, false>), grid, dim3(kThreads), 0, stream, a); break;
        case 4: hipLaunchKernelGGL((ssd_delta_step_kernel<T, N, 4, false>), grid, dim3(kThreads), 0, stream, a); break;
        default:
            // A state that the last-level cache cannot hold until the next token goes past it: 512 MB take 179 us this way
            // and 199 without, but 256 MB 87 and 83, 64 MB 22.3 and 21.0.
            if (work * kThreads * 16 > (256LL << 20)) hipLaunchKernelGGL((ssd_delta_step_kernel<T, N, 8, true>), grid, dim3(kThreads), 0, stream, a);
            else hipLaunchKernelGGL((ssd_delta_step_kernel<T, N, 8, false>), grid, dim3(kThreads), 0, stream, a);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const DeltaArgs& a, hipStream_t stream) {
    switch (a.N) {
        case 32: return launch_n<T, 32>(a, stream);
        case 64: return launch_n<T, 64>(a, stream);
        case 128: return launch_n<T, 128>(a, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_delta_step(const DeltaArgs& a, hipStream_t stream) {
    return a.dtype == 0 ? launch_t<float>(a, stream) : launch_t<uint16_t>(a, stream);
}

}  // namespace ssd

// Dropout with a counter-based generator: y = [residual +] keep * x / (1 - p).
//
// No mask is stored: whether element i is kept follows from (seed, offset, i)
// alone, so the backward pass is the same call on the gradient. Elements 4 g
// .. 4 g + 3 take the four 32-bit words of Philox4x32-10 (Salmon, Moraes, Dror
// and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) with counter
// {g, g >> 32, offset, offset >> 32} and key {seed, seed >> 32}; an element is
// kept when its word is at least p * 2^32 (rounded to an integer), so the
// probability is right to 2^-33.
//
// Bound by memory with fp32 elements (33.5 M: 41 us, 6.5 TB/s) or a residual
// (33.5 M bf16: 34 to 38 us, 5.3 to 5.9 TB/s), by integer work without (31 us,
// 4.4 TB/s): ten rounds of two 32 x 32 -> 64 products serve four elements, and
// the pipe of wide products is the busiest (65 % of the time, DRAM 32 %, issue
// 58 %). Each thread takes two runs
// of 16 bytes at a time (four or eight elements, one or two generator calls
// each). seed and offset are read from
// device memory so that a captured graph draws anew when they are changed
// between replays.
#include "kernels.cuh"
#include "rowvec.cuh"

namespace dlrm {
namespace {

// The ten rounds' keys, the same for every element.
struct RoundKeys {
    uint32_t a[10], b[10];
    __device__ __forceinline__ RoundKeys(unsigned long long seed) {
#pragma unroll
        for (int r = 0; r < 10; ++r) {
            a[r] = (uint32_t)seed + 0x9E3779B9u * r;
            b[r] = (uint32_t)(seed >> 32) + 0xBB67AE85u * r;
        }
    }
};

__device__ __forceinline__ uint4 philox4x32_10(unsigned long long group, uint32_t c2, uint32_t c3, const RoundKeys& k) {
    uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const unsigned long long a = (unsigned long long)0xD2511F53u * c0;
        const unsigned long long b = (unsigned long long)0xCD9E8D57u * c2;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k.a[r];
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k.b[r];
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
    }
    return make_uint4(c0, c1, c2, c3);
}

struct DropArgs {
    long long n;
    const void* x;
    const void* residual;       // or null
    void* y;
    const unsigned long long* rng;   // {seed, offset}
    uint32_t threshold;              // kept when word >= threshold ...
    bool any;                        // ... unless p * 2^32 rounds to 2^32: nothing is kept
    float scale;
};

// VEC = elements per 16 bytes, or 4 with element-wise accesses (ALIGNED = false). SMALL: the counter's low half
// fits 32 bits, so that two of the twenty products are the same for all elements and leave the loop.
template <typename T, bool RES, bool ALIGNED, bool SMALL>
__global__ void __launch_bounds__(256, 5) dropout_kernel(const __grid_constant__ DropArgs a) {
    pdl_wait();
    constexpr int VEC = ALIGNED ? 16 / (int)sizeof(T) : 4;
    const T* x = static_cast<const T*>(a.x);
    const T* res = static_cast<const T*>(a.residual);
    T* y = static_cast<T*>(a.y);
    const unsigned long long seed = a.rng[0], off = a.rng[1];
    const RoundKeys keys(seed);
    const uint32_t c2 = (uint32_t)off, c3 = (uint32_t)(off >> 32);
    // a block's turn: two runs per thread, loaded together
    for (long long turn = blockIdx.x; turn * (2 * VEC * 256) < a.n; turn += gridDim.x) {
        RowRaw<T, VEC> rx[2], rr[2];
        const long long i0 = (turn * 512 + threadIdx.x) * VEC;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const long long i = i0 + u * (256 * VEC);
            if (ALIGNED && i + VEC <= a.n) {
                rx[u].load(x + i);
                if constexpr (RES) rr[u].load(res + i);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (i + e < a.n) {
                        rx[u].e[e] = x[i + e];
                        if constexpr (RES) rr[u].e[e] = res[i + e];
                    }
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const long long i = i0 + u * (256 * VEC);
            float v[VEC];
#pragma unroll
            for (int g = 0; g < VEC / 4; ++g) {
                const uint4 w = philox4x32_10(SMALL ? (unsigned long long)(uint32_t)(i / 4 + g) : (unsigned long long)(i / 4 + g), c2, c3, keys);
                const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // a dropped element gives zero whatever x holds there (infinity and NaN too)
                    const int q = 4 * g + e;
                    v[q] = word[e] >= a.threshold && a.any ? Cvt<T>::to_f(rx[u].e[q]) * a.scale : 0.f;
                    if constexpr (RES) v[q] += Cvt<T>::to_f(rr[u].e[q]);
                }
            }
            RowRaw<T, VEC> out;
            out.set(v);
            if (ALIGNED && i + VEC <= a.n) {
                out.store(y + i);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (i + e < a.n) y[i + e] = out.e[e];
            }
        }
    }
}

template <typename T>
dlrm_status launch_t(const DropArgs& a, cudaStream_t st) {
    const bool al = rows_on(a.x, 0, 16) && rows_on(a.y, 0, 16) && rows_on(a.residual, 0, 16);
    const int vec = al ? 16 / (int)sizeof(T) : 4;
    const long long want = (a.n + 512ll * vec - 1) / (512ll * vec);
    // many short blocks: 40 an SM where one wave of five, eight, 16 or 80 take longer (33.5 M: bf16 with residual 34.1 us and
    // 36.2, 35.3, 34.8, 34.5; without 30.5 and 32.3, 31.1, 30.6, 31.2; fp32 41.2 and 43.6, 50.5, 42.6, 41.6)
    const long long most = 40ll * device_sms();
    const dim3 grid((unsigned)(want < most ? want : most));
    const bool small = a.n <= 4ll << 32;
#define DLRM_DROP(RES, AL)                                                                          \
    do {                                                                                            \
        if (small) DLRM_PDL_CHECK(launch_pdl(dropout_kernel<T, RES, AL, true>, grid, dim3(256), 0, st, a)); \
        else DLRM_PDL_CHECK(launch_pdl(dropout_kernel<T, RES, AL, false>, grid, dim3(256), 0, st, a));      \
    } while (0)
    if (a.residual) {
        if (al) DLRM_DROP(true, true);
        else DLRM_DROP(true, false);
    } else {
        if (al) DLRM_DROP(false, true);
        else DLRM_DROP(false, false);
    }
#undef DLRM_DROP
    return DLRM_OK;
}

}  // namespace

dlrm_status launch_dropout(long long n, const void* x, const void* residual, dlrm_dtype dt, double p,
                           const int64_t* rng, void* y, cudaStream_t st) {
    DropArgs a;
    a.n = n;
    a.x = x;
    a.residual = residual;
    a.y = y;
    a.rng = reinterpret_cast<const unsigned long long*>(rng);
    const double t = p * 4294967296.0 + 0.5;
    a.any = t < 4294967296.0;
    a.threshold = a.any ? (uint32_t)t : 0u;
    a.scale = a.any ? (float)(1.0 / (1.0 - p)) : 0.f;
    if (dt == DLRM_F32) return launch_t<float>(a, st);
    if (dt == DLRM_F16) return launch_t<__half>(a, st);
    return launch_t<__nv_bfloat16>(a, st);
}

}  // namespace dlrm

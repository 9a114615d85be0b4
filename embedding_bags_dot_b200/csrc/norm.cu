// Root-mean-square norm with the residual's addition, and its backward pass.
//
//   h = x + residual                     (fp32, stored rounded once)
//   rstd = 1 / sqrt(mean_c h_c^2 + eps)
//   y_c = h_c * rstd * w_c               (from the unrounded h)
// y is rounded once to x's type, or to e4m3 codes with one fp32 scale per row:
//   s = max_c |y_c| / 448,  q_c = rn(y_c / s),  y_c ~ q_c s.
// Backward, with xh = h * rstd from the stored h and g = dy * w:
//   dx = rstd * (g - xh * mean_c(g xh)) + dh,      dw_c = sum_rows dy_c xh_c.
//
// Both passes move each row once, so memory bounds them, with instruction issue
// close behind (16,384 x 4,096 bf16 to e4m3 with residual: 78 to 84 us, 5.6 to
// 6.0 TB/s, 77 % of issue slots; backward of 20,000 x 2,040 fp16: 65 to 67 us,
// 4.9 TB/s). A row's elements stay with their threads between the statistics and
// the output. A warp takes rows of up to one run per lane (no block barrier), a
// block longer ones, two runs per thread; where rows allow whole 16-byte runs the
// next rows are on their way to shared memory meanwhile. Rows of more than 16,384
// 16-bit or 8,192 other elements (fp32, and widths without whole runs) take 32
// elements a thread, which do not fit its 64 registers with their weights: 124 to
// 660 bytes of each thread's go through local memory forward, 540 to 960 backward
// (76 in the backward pass of 4,097 to 16,384 16-bit columns), and the time shows
// it (4,096 rows with residual, forward and backward: 32,768 bf16 218 and 585 us,
// 16,384 fp32 364 and 515, where the bytes take 164; 10,001 bf16 576 and 861,
// where they take 50). Blocks are as many as fit at once; they keep their columns
// of w in registers, and in the backward pass their columns'
// sums of dw, written once per block and added in block order by a second
// kernel. All sums are fp32 in an order fixed by the shape.
#include <algorithm>

#include "kernels.cuh"
#include "rowvec.cuh"

namespace dlrm {
namespace {

struct NormFwdArgs {
    int rows, d;
    float eps, inv_d;
    const void* x;
    long long ldx;
    const void* res;
    long long ldres;
    const float* w;    // or null: ones
    void* h;
    long long ldh;
    void* y;
    long long ldy;
    float* y_scale;    // e4m3 output only
    float* rstd;
};

struct NormBwdArgs {
    int rows, d;
    float inv_d;
    const void* dy;
    long long lddy;
    const void* h;
    long long ldh;
    const float* rstd;
    const float* w;
    const void* dh;
    long long lddh;
    void* dx;
    long long lddx;
    float* partial;    // [gridDim.x][d] or null
};

// Sum (or unsigned maximum) over the row's threads: one warp, or the whole block through shared memory.
// Consecutive calls alternate `slot`, so one barrier per call is enough.
template <bool BLOCK>
__device__ __forceinline__ float row_sum(float v, float (*red)[32], int slot) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (BLOCK) {
        const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
        if (lane == 0) red[slot][threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < nw ? red[slot][lane] : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}
template <bool BLOCK>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float (*red)[32], int slot) {
    v = __reduce_max_sync(0xffffffffu, v);
    if constexpr (BLOCK) {
        const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
        if (lane == 0) red[slot][threadIdx.x >> 5] = __uint_as_float(v);
        __syncthreads();
        v = __reduce_max_sync(0xffffffffu, lane < nw ? __float_as_uint(red[slot][lane]) : 0u);
    }
    return v;
}

// Means below this are taken apart (FAR). Only where eps is below it too: the branch beside the row's registers costs up to
// a half of odd widths (16,384 x 1,001 bf16 42 us without, 49 with; 4,096 x 10,001: 569, 866).
constexpr float FAR_MEAN = 0x1p-100f;

// rstd of a row whose mean square (with eps) left fp32's ordinary range: from its values times 2^100 or 2^-80 (exact for
// all that count), whose squares and their sum stay inside. It is at most fp32's largest number (a mean below 2^-256).
// A row of zeros without eps has 0: its output is zeros, and it adds nothing to a gradient. An infinity or NaN spreads as
// in other rows. All threads of a row come here together.
template <int NV, int VEC, bool BLOCK>
__device__ __forceinline__ float far_rstd(const float (&v)[NV][VEC], bool small, const NormFwdArgs& a, float (*red)[32], int slot) {
    const float up = small ? 0x1p100f : 0x1p-80f;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float u = v[i][e] * up;
            ss = fmaf(u, u, ss);
        }
    const float mean = fmaf(row_sum<BLOCK>(ss, red, slot), a.inv_d, a.eps * up * up);
    const float rstd = mean == 0.f ? 0.f : 1.f / sqrtf(mean) * up;
    return rstd > 3.402823466e38f ? 3.402823466e38f : rstd;
}

// Rows ahead of the one being reduced are copied into shared memory asynchronously (cp.async): each thread copies
// the 16-byte runs that it will itself read, so the ring needs no barrier.
__device__ __forceinline__ void copy16_async(uint4* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

constexpr int FWD_RING = 3, BWD_RING = 2;    // rows in the ring: one in use, the others on their way

// Thread t of the row's G threads holds runs t, t + G, ... (NV of them) of VEC elements. FAR: eps is too small to keep
// every mean above 2^-100, so rows are watched for it.
template <typename T, int VEC, int NV, bool BLOCK, bool Q8, int MAXT, bool RING, bool FAR>
__global__ void __launch_bounds__(MAXT, MAXT == 1024 ? 1 : 1024 / MAXT) rmsnorm_fwd_kernel(const __grid_constant__ NormFwdArgs a) {
    pdl_wait();
    __shared__ float red[4][32];
    const int G = BLOCK ? blockDim.x : 32;
    const int t = BLOCK ? threadIdx.x : (threadIdx.x & 31);
    const long long first = BLOCK ? blockIdx.x : (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const long long step = BLOCK ? gridDim.x : (long long)gridDim.x * (blockDim.x >> 5);
    float w[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = (t + i * G) * VEC + e;
            w[i][e] = a.w && c < a.d ? a.w[c] : 1.f;
        }
    int slot = 0, stage = 0;
    RowRaw<T, VEC> raw[NV], rres[NV];
    extern __shared__ uint4 ring[];      // RING: [row][x, residual][run][thread]
    auto place = [&](int s, int arr, int i) { return ring + ((s * 2 + arr) * NV + i) * blockDim.x + threadIdx.x; };
    auto send = [&](long long r, int s) {
        if (r < a.rows) {
            const T* x = static_cast<const T*>(a.x) + r * a.ldx;
            const T* res = static_cast<const T*>(a.res) + r * a.ldres;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t + i * G) * VEC;
                if (c < a.d) {
                    copy16_async(place(s, 0, i), x + c);
                    if (a.res) copy16_async(place(s, 1, i), res + c);
                }
            }
        }
        copy_commit();
    };
    if constexpr (RING) {
#pragma unroll
        for (int s = 0; s < FWD_RING - 1; ++s) send(first + s * step, s);
    }
    for (long long r = first; r < a.rows; r += step) {
        if constexpr (RING) {
            send(r + (FWD_RING - 1) * step, stage == 0 ? FWD_RING - 1 : stage - 1);
            copy_wait<FWD_RING - 1>();
        }
        const T* x = static_cast<const T*>(a.x) + r * a.ldx;
        const T* res = static_cast<const T*>(a.res) + r * a.ldres;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * G) * VEC;
            if (c < a.d) {
                if constexpr (RING) {
                    raw[i].a[0] = *place(stage, 0, i);
                    if (a.res) rres[i].a[0] = *place(stage, 1, i);
                } else {
                    raw[i].load(x + c);
                    if (a.res) rres[i].load(res + c);
                }
            } else {
                raw[i].zero();
                rres[i].zero();
            }
        }
        if constexpr (RING) stage = stage + 1 == FWD_RING ? 0 : stage + 1;
        float v[NV][VEC], ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            raw[i].get(v[i]);
            if (a.res) {
                float q[VEC];
                rres[i].get(q);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[i][e] += q[e];
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) ss = fmaf(v[i][e], v[i][e], ss);
        }
        if (a.h) {
            T* h = static_cast<T*>(a.h) + r * a.ldh;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t + i * G) * VEC;
                if (c < a.d) {
                    raw[i].set(v[i]);
                    raw[i].store(h + c);
                }
            }
        }
        ss = row_sum<BLOCK>(ss, red, slot);
        slot ^= 1;
        float rstd;
        if constexpr (FAR) {
            const float mean = fmaf(ss, a.inv_d, a.eps);
            rstd = 1.f / sqrtf(mean);
            // Squares below 2^-126 lose bits, each at most 2^-150: nothing next to a mean of 2^-100. All threads of the
            // row have the same mean.
            if (!(mean >= FAR_MEAN && mean <= 3.402823466e38f)) {
                rstd = far_rstd<NV, VEC, BLOCK>(v, mean < 1.f, a, red, slot);
                slot ^= 1;
            }
        } else {
            rstd = 1.f / sqrtf(fmaf(ss, a.inv_d, a.eps));
        }
        if (a.rstd && t == 0) a.rstd[r] = rstd;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i][e] = v[i][e] * rstd * w[i][e];
        if constexpr (Q8) {
            // the largest magnitude as its bit pattern: a NaN compares above every number, so it reaches the
            // scale (and with it the whole row) instead of being passed over
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if ((t + i * G) * VEC < a.d) m = max(m, __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
            m = row_max<BLOCK>(m, red, slot + 2);
            const float amax = __uint_as_float(m), scale = amax / 448.f;
            if (t == 0) a.y_scale[r] = scale;
            uint8_t* y = static_cast<uint8_t*>(a.y) + r * a.ldy;
            if (amax >= 1e-30f || m > 0x7F800000u) {
                const float inv = 448.f / amax;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (t + i * G) * VEC;
                    if (c < a.d) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) v[i][e] *= inv;
                        store_e4m3<VEC>(y + c, v[i]);
                    }
                }
            } else {
                // 448 / amax could overflow here, and the scale may be a subnormal that says little about it
                // (or zero): these rows divide by the scale as stored
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (t + i * G) * VEC;
                    if (c < a.d) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) v[i][e] = scale > 0.f ? v[i][e] / scale : 0.f;
                        store_e4m3<VEC>(y + c, v[i]);
                    }
                }
            }
        } else {
            T* y = static_cast<T*>(a.y) + r * a.ldy;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t + i * G) * VEC;
                if (c < a.d) {
                    raw[i].set(v[i]);
                    raw[i].store(y + c);
                }
            }
        }
    }
}

template <typename T, int VEC, int NV, bool BLOCK, int MAXT, bool RING>
__global__ void __launch_bounds__(MAXT, MAXT == 1024 ? 1 : MAXT == 256 ? 3 : 4) rmsnorm_bwd_kernel(const __grid_constant__ NormBwdArgs a) {
    pdl_wait();
    __shared__ float red[2][32];
    const int G = BLOCK ? blockDim.x : 32;
    const int t = BLOCK ? threadIdx.x : (threadIdx.x & 31);
    const long long first = BLOCK ? blockIdx.x : (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const long long step = BLOCK ? gridDim.x : (long long)gridDim.x * (blockDim.x >> 5);
    float w[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = (t + i * G) * VEC + e;
            w[i][e] = a.w && c < a.d ? a.w[c] : 1.f;
            dw[i][e] = 0.f;
        }
    int slot = 0, stage = 0;
    RowRaw<T, VEC> ry[NV], rh[NV], rd[NV];
    extern __shared__ uint4 ring[];      // RING: [row][dy, h, dh][run][thread]
    auto place = [&](int s, int arr, int i) { return ring + ((s * 3 + arr) * NV + i) * blockDim.x + threadIdx.x; };
    auto send = [&](long long r, int s) {
        if (r < a.rows) {
            const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
            const T* h = static_cast<const T*>(a.h) + r * a.ldh;
            const T* dh = static_cast<const T*>(a.dh) + r * a.lddh;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t + i * G) * VEC;
                if (c < a.d) {
                    copy16_async(place(s, 0, i), dy + c);
                    copy16_async(place(s, 1, i), h + c);
                    if (a.dh) copy16_async(place(s, 2, i), dh + c);
                }
            }
        }
        copy_commit();
    };
    if constexpr (RING) {
#pragma unroll
        for (int s = 0; s < BWD_RING - 1; ++s) send(first + s * step, s);
    }
    float next_rstd = first < a.rows ? a.rstd[first] : 0.f;
    for (long long r = first; r < a.rows; r += step) {
        const float rstd = next_rstd;
        if (r + step < a.rows) next_rstd = a.rstd[r + step];
        if constexpr (RING) {
            send(r + (BWD_RING - 1) * step, stage == 0 ? BWD_RING - 1 : stage - 1);
            copy_wait<BWD_RING - 1>();
        }
        const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
        const T* h = static_cast<const T*>(a.h) + r * a.ldh;
        const T* dh = static_cast<const T*>(a.dh) + r * a.lddh;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * G) * VEC;
            if (c < a.d) {
                if constexpr (RING) {
                    ry[i].a[0] = *place(stage, 0, i);
                    rh[i].a[0] = *place(stage, 1, i);
                    if (a.dh) rd[i].a[0] = *place(stage, 2, i);
                } else {
                    ry[i].load(dy + c);
                    rh[i].load(h + c);
                    if (a.dh) rd[i].load(dh + c);
                }
            } else {
                ry[i].zero();
                rh[i].zero();
            }
        }
        if constexpr (RING) stage = stage + 1 == BWD_RING ? 0 : stage + 1;
        float along = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float y[VEC], xh[VEC];
            ry[i].get(y);
            rh[i].get(xh);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                xh[e] *= rstd;
                dw[i][e] = fmaf(y[e], xh[e], dw[i][e]);
                along = fmaf(y[e] * w[i][e], xh[e], along);
            }
        }
        along = row_sum<BLOCK>(along, red, slot) * a.inv_d;
        slot ^= 1;
        T* dx = static_cast<T*>(a.dx) + r * a.lddx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * G) * VEC;
            if (c < a.d) {
                float y[VEC], xh[VEC], o[VEC];
                ry[i].get(y);
                rh[i].get(xh);
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = rstd * (y[e] * w[i][e] - xh[e] * rstd * along);
                if (a.dh) {
                    rd[i].get(y);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[e] += y[e];
                }
                ry[i].set(o);
                ry[i].store(dx + c);
            }
        }
    }
    if (!a.partial) return;
    float* p = a.partial + (long long)blockIdx.x * a.d;
    if constexpr (BLOCK) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int c = (t + i * G) * VEC + e;
                if (c < a.d) p[c] = dw[i][e];
            }
    } else {
        // the block's warps add their sums in warp order
        float* sums = reinterpret_cast<float*>(ring);   // [warps][NV * VEC * 32]
        constexpr int W = NV * VEC * 32;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) sums[(threadIdx.x >> 5) * W + (t + i * 32) * VEC + e] = dw[i][e];
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
            float s = 0.f;
            for (int q = 0; q < (int)(blockDim.x >> 5); ++q) s += sums[q * W + c];
            p[c] = s;
        }
    }
}

// dw[c] = sum over blocks of partial[block][c]: 16 columns a block, 64 row groups, all in fixed order.
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(int nparts, int d, const float* __restrict__ partial,
                                                          float* __restrict__ dw) {
    pdl_wait();
    __shared__ float part[64][17];
    const int lane = threadIdx.x & 15, g = threadIdx.x >> 4, c = blockIdx.x * 16 + lane;
    float s = 0.f;
    if (c < d) {
#pragma unroll 8
        for (int p = g; p < nparts; p += 64) s += partial[(long long)p * d + c];
    }
    part[g][lane] = s;
    __syncthreads();
    // eight sums of eight groups, then one of those
    if (g < 8) {
        s = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += part[g * 8 + q][lane];
    }
    __syncthreads();
    if (g < 8) part[g][lane] = s;
    __syncthreads();
    if (g == 0 && c < d) {
        s = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += part[q][lane];
        dw[c] = s;
    }
}

// Widest run (elements) that every row of every given array allows.
struct Runs {
    int es;
    int bytes = 16;
    void add(const void* p, long long ld, int elem) {
        if (!p) return;
        // e4m3 rows hold one byte per element: a run of VEC elements needs VEC bytes there
        const int scale = es / elem;
        while (bytes > es && !rows_on(p, ld * elem, bytes / scale)) bytes >>= 1;
    }
    int vec() const { return bytes / es; }
};

int norm_threads(int d, int per) { return ((d + per - 1) / per + 31) / 32 * 32; }

// Launches a norm kernel with `smem` bytes of ring: at most 1,024 threads of 192 bytes. Above 48 KB in all the kernel has
// to be told; always the same value, so that calls from several host threads agree.
constexpr int RING_MOST = 1024 * 192;
template <typename Args>
dlrm_status norm_launch(void (*kern)(Args), unsigned grid, int threads, size_t smem, const Args& a, cudaStream_t st) {
    if (smem > 40 * 1024) cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_MOST);
    DLRM_PDL_CHECK(launch_pdl(kern, dim3(grid), dim3(threads), smem, st, a));
    return DLRM_OK;
}

template <typename T, int VEC, bool Q8, bool FAR>
dlrm_status fwd_vec(const NormFwdArgs& a, cudaStream_t st) {
    constexpr int W = 16 / (int)sizeof(T);
    constexpr int NV = W / VEC;             // one 16-byte run's elements, however they are loaded
    const int one = norm_threads(a.d, W);
    if (one == 32) {
        const long long want = (a.rows + 3ll) / 4, most = 8ll * device_sms();
        return norm_launch(rmsnorm_fwd_kernel<T, VEC, NV, false, Q8, 128, false, FAR>, (unsigned)std::min(want, most), 128, 0, a, st);
    }
    const long long sms = device_sms();
    // few rows: the latency of a row counts, so it is spread over as many threads as it has runs
    if (a.rows <= sms && one <= 1024)
        return norm_launch(rmsnorm_fwd_kernel<T, VEC, NV, true, Q8, 1024, false, FAR>, (unsigned)a.rows, one, 0, a, st);
    // two runs a thread where the runs are whole, else eight elements in smaller pieces (16 of them a thread took
    // 70 us where 8 take 45: 16,384 odd-width bf16 rows)
    constexpr int PT = VEC == W ? 2 * W : 8;
    const int two = norm_threads(a.d, PT);
    if (two > 1024) {
        const int t = norm_threads(a.d, 32);
        return norm_launch(rmsnorm_fwd_kernel<T, VEC, 32 / VEC, true, Q8, 1024, false, FAR>,
                           (unsigned)std::min<long long>(a.rows, sms), t, 0, a, st);
    }
    const unsigned grid = (unsigned)std::min<long long>(a.rows, sms * (1024 / two));
    const size_t smem = VEC == W ? (size_t)FWD_RING * 2 * 2 * 16 * two : 0;
    if (two > 256) return norm_launch(rmsnorm_fwd_kernel<T, VEC, PT / VEC, true, Q8, 1024, VEC == W, FAR>, grid, two, smem, a, st);
    return norm_launch(rmsnorm_fwd_kernel<T, VEC, PT / VEC, true, Q8, 256, VEC == W, FAR>, grid, two, smem, a, st);
}

template <typename T, bool FAR>
dlrm_status fwd_t(const NormFwdArgs& a, bool q8, cudaStream_t st) {
    Runs u{(int)sizeof(T)};
    u.add(a.x, a.ldx, sizeof(T));
    u.add(a.res, a.ldres, sizeof(T));
    u.add(a.h, a.ldh, sizeof(T));
    u.add(a.y, a.ldy, q8 ? 1 : sizeof(T));
    constexpr int W = 16 / (int)sizeof(T);
    int vec = u.vec();
    while (a.d % vec) vec >>= 1;
    if (vec == W) return q8 ? fwd_vec<T, W, true, FAR>(a, st) : fwd_vec<T, W, false, FAR>(a, st);
    if constexpr (W > 4)
        if (vec == 4) return q8 ? fwd_vec<T, 4, true, FAR>(a, st) : fwd_vec<T, 4, false, FAR>(a, st);
    if (vec >= 2) return q8 ? fwd_vec<T, 2, true, FAR>(a, st) : fwd_vec<T, 2, false, FAR>(a, st);
    return q8 ? fwd_vec<T, 1, true, FAR>(a, st) : fwd_vec<T, 1, false, FAR>(a, st);
}

template <typename T>
dlrm_status fwd_far(const NormFwdArgs& a, bool q8, cudaStream_t st) {
    return a.eps < FAR_MEAN ? fwd_t<T, true>(a, q8, st) : fwd_t<T, false>(a, q8, st);
}

// Blocks of `threads` threads that are resident at once: 64 registers a thread above 256 threads, 80 below.
long long bwd_resident(int threads) {
    return (long long)device_sms() * std::max(1, (threads > 256 ? 1024 : 768) / threads);
}
// Most blocks of the backward pass, each of which writes a row of partial sums: those of a 16-bit type, whose rows
// take the fewest threads.
long long bwd_most(int d) { return bwd_resident(std::max(96, norm_threads(d, 16))); }

template <typename T, int VEC>
dlrm_status bwd_vec(const NormBwdArgs& a, int& nblocks, cudaStream_t st) {
    constexpr int W = 16 / (int)sizeof(T);
    constexpr int NV = W / VEC;
    if (norm_threads(a.d, W) == 32) {
        nblocks = (int)std::min<long long>((a.rows + 3ll) / 4, std::min(bwd_resident(128), bwd_most(a.d)));
        const size_t smem = a.partial ? sizeof(float) * 4 * W * 32 : 0;
        return norm_launch(rmsnorm_bwd_kernel<T, VEC, NV, false, 128, false>, nblocks, 128, smem, a, st);
    }
    constexpr int PT = VEC == W ? 2 * W : 8;
    const int two = norm_threads(a.d, PT), wide = norm_threads(a.d, 32);
    nblocks = (int)std::min<long long>(a.rows, std::min(bwd_resident(two > 1024 ? wide : two), bwd_most(a.d)));
    if (two > 1024)
        return norm_launch(rmsnorm_bwd_kernel<T, VEC, 32 / VEC, true, 1024, false>, nblocks, wide, 0, a, st);
    const size_t smem = VEC == W ? (size_t)BWD_RING * 3 * 2 * 16 * two : 0;
    if (two > 256)
        return norm_launch(rmsnorm_bwd_kernel<T, VEC, PT / VEC, true, 1024, VEC == W>, nblocks, two, smem, a, st);
    return norm_launch(rmsnorm_bwd_kernel<T, VEC, PT / VEC, true, 256, VEC == W>, nblocks, two, smem, a, st);
}

template <typename T>
dlrm_status bwd_t(const NormBwdArgs& a, int& nblocks, cudaStream_t st) {
    Runs u{(int)sizeof(T)};
    u.add(a.dy, a.lddy, sizeof(T));
    u.add(a.h, a.ldh, sizeof(T));
    u.add(a.dh, a.lddh, sizeof(T));
    u.add(a.dx, a.lddx, sizeof(T));
    constexpr int W = 16 / (int)sizeof(T);
    int vec = u.vec();
    while (a.d % vec) vec >>= 1;
    if (vec == W) return bwd_vec<T, W>(a, nblocks, st);
    if constexpr (W > 4)
        if (vec == 4) return bwd_vec<T, 4>(a, nblocks, st);
    if (vec >= 2) return bwd_vec<T, 2>(a, nblocks, st);
    return bwd_vec<T, 1>(a, nblocks, st);
}

}  // namespace

dlrm_status launch_rmsnorm_fwd(int rows, int d, const void* x, long long ldx, const void* res, long long ldres,
                               const float* w, float eps, dlrm_dtype dt, void* h, long long ldh, void* y,
                               long long ldy, float* y_scale, float* rstd, cudaStream_t st) {
    const NormFwdArgs a{rows, d, eps, 1.f / (float)d, x, ldx, res, ldres, w, h, ldh, y, ldy, y_scale, rstd};
    const bool q8 = y_scale != nullptr;
    if (dt == DLRM_F32) return fwd_far<float>(a, q8, st);
    if (dt == DLRM_F16) return fwd_far<__half>(a, q8, st);
    return fwd_far<__nv_bfloat16>(a, q8, st);
}

size_t rmsnorm_bwd_partial_floats(int rows, int d) { return (size_t)std::min<long long>(rows, bwd_most(d)) * d; }

dlrm_status launch_rmsnorm_bwd(int rows, int d, const void* dy, long long lddy, const void* h, long long ldh,
                               const float* rstd, const float* w, const void* dh, long long lddh, dlrm_dtype dt,
                               void* dx, long long lddx, float* dw, float* partial, cudaStream_t st) {
    const NormBwdArgs a{rows, d,  1.f / (float)d, dy, lddy, h, ldh, rstd, w, dh, lddh, dx, lddx,
                        dw ? partial : nullptr};
    int nblocks = 0;
    if (rows > 0) {
        const dlrm_status r = dt == DLRM_F32   ? bwd_t<float>(a, nblocks, st)
                              : dt == DLRM_F16 ? bwd_t<__half>(a, nblocks, st)
                                               : bwd_t<__nv_bfloat16>(a, nblocks, st);
        if (r != DLRM_OK) return r;
    }
    if (dw) DLRM_PDL_CHECK(launch_pdl(rmsnorm_dw_kernel, dim3((d + 15) / 16), dim3(1024), 0, st, nblocks, d,
                                      (const float*)partial, dw));
    return DLRM_OK;
}

}  // namespace dlrm

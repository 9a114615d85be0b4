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
// Both passes move each row once, so memory bounds them: a row's elements stay
// in registers between the statistics and the output. One warp takes a row of
// up to 32 runs per lane group below (no block barrier); longer rows take a
// block. Blocks are persistent (a few per SM) and keep their columns of w in
// registers; the backward pass also keeps its columns' sums of dw there and
// writes them once per block, a second kernel adds the blocks' sums in block
// order. All sums are fp32 in an order fixed by the shape.
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

// Thread t of the row's G threads holds runs t, t + G, ... (NV of them) of VEC elements.
template <typename T, int VEC, int NV, bool BLOCK, bool Q8, int MAXT>
__global__ void __launch_bounds__(MAXT) rmsnorm_fwd_kernel(const __grid_constant__ NormFwdArgs a) {
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
    int slot = 0;
    for (long long r = first; r < a.rows; r += step) {
        const T* x = static_cast<const T*>(a.x) + r * a.ldx;
        RowRaw<T, VEC> raw[NV], rres[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * G) * VEC;
            if (c < a.d) raw[i].load(x + c);
            else raw[i].zero();
        }
        if (a.res) {
            const T* res = static_cast<const T*>(a.res) + r * a.ldres;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t + i * G) * VEC;
                if (c < a.d) rres[i].load(res + c);
                else rres[i].zero();
            }
        }
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
        const float rstd = 1.f / sqrtf(fmaf(ss, a.inv_d, a.eps));
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
            // 1 / scale would overflow or lose its subnormal bits for the smallest rows: those divide
            const bool tiny = amax < 1e-30f;
            const float inv = tiny ? 0.f : 448.f / amax;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t + i * G) * VEC;
                if (c < a.d) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        v[i][e] = tiny ? (scale > 0.f ? v[i][e] / scale : 0.f) : v[i][e] * inv;
                    store_e4m3<VEC>(y + c, v[i]);
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

template <typename T, int VEC, int NV, bool BLOCK, int MAXT>
__global__ void __launch_bounds__(MAXT) rmsnorm_bwd_kernel(const __grid_constant__ NormBwdArgs a) {
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
    int slot = 0;
    for (long long r = first; r < a.rows; r += step) {
        const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
        const T* h = static_cast<const T*>(a.h) + r * a.ldh;
        RowRaw<T, VEC> ry[NV], rh[NV], rd[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * G) * VEC;
            if (c < a.d) {
                ry[i].load(dy + c);
                rh[i].load(h + c);
            } else {
                ry[i].zero();
                rh[i].zero();
            }
        }
        if (a.dh) {
            const T* dh = static_cast<const T*>(a.dh) + r * a.lddh;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t + i * G) * VEC;
                if (c < a.d) rd[i].load(dh + c);
            }
        }
        const float rstd = a.rstd[r];
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
        extern __shared__ float sums[];   // [warps][NV * VEC * 32]
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

// dw[c] = sum over blocks of partial[block][c]: 32 columns a block, 32 row groups, all in fixed order.
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(int nparts, int d, const float* __restrict__ partial,
                                                          float* __restrict__ dw) {
    pdl_wait();
    __shared__ float part[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    float s = 0.f;
    if (c < d)
        for (int p = g; p < nparts; p += 32) s += partial[(long long)p * d + c];
    part[g][threadIdx.x & 31] = s;
    __syncthreads();
    if (g == 0 && c < d) {
        s = 0.f;
#pragma unroll
        for (int q = 0; q < 32; ++q) s += part[q][threadIdx.x];
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

template <typename T, int VEC, int NV, bool Q8>
dlrm_status fwd_nv(const NormFwdArgs& a, cudaStream_t st) {
    const int runs = (a.d + VEC - 1) / VEC;
    if (runs <= 32 * NV) {
        const int warps = 4;
        const long long want = (a.rows + warps - 1) / warps, most = 16ll * device_sms();
        DLRM_PDL_CHECK(launch_pdl(rmsnorm_fwd_kernel<T, VEC, NV, false, Q8, 128>,
                                  dim3((unsigned)std::min(want, most)), dim3(32 * warps), 0, st, a));
        return DLRM_OK;
    }
    const int threads = ((runs + NV - 1) / NV + 31) / 32 * 32;
    const dim3 grid((unsigned)std::min<long long>(a.rows, (long long)device_sms() * std::max(1, 2048 / threads)));
    if (threads <= 256)
        DLRM_PDL_CHECK(launch_pdl(rmsnorm_fwd_kernel<T, VEC, NV, true, Q8, 256>, grid, dim3(threads), 0, st, a));
    else if (threads <= 1024)
        DLRM_PDL_CHECK(launch_pdl(rmsnorm_fwd_kernel<T, VEC, NV, true, Q8, 1024>, grid, dim3(threads), 0, st, a));
    else
        return DLRM_ERR_UNSUPPORTED;
    return DLRM_OK;
}

template <typename T, int VEC, bool Q8>
dlrm_status fwd_vec(const NormFwdArgs& a, cudaStream_t st) {
    constexpr int W = 16 / (int)sizeof(T);       // elements of a full run
    // few rows: the latency of one row counts, so it is spread over more threads
    const bool few = a.rows <= device_sms();
    const int runs = (a.d + VEC - 1) / VEC;
    if (few && runs <= 1024) return fwd_nv<T, VEC, 1, Q8>(a, st);
    if (runs <= 1024 * 2 * (W / VEC)) return fwd_nv<T, VEC, 2 * (W / VEC), Q8>(a, st);
    return fwd_nv<T, VEC, 32 / VEC, Q8>(a, st);
}

template <typename T>
dlrm_status fwd_t(const NormFwdArgs& a, bool q8, cudaStream_t st) {
    Runs u{(int)sizeof(T)};
    u.add(a.x, a.ldx, sizeof(T));
    u.add(a.res, a.ldres, sizeof(T));
    u.add(a.h, a.ldh, sizeof(T));
    u.add(a.y, a.ldy, q8 ? 1 : sizeof(T));
    constexpr int W = 16 / (int)sizeof(T);
    int vec = u.vec();
    while (a.d % vec) vec >>= 1;
    if (vec == W) return q8 ? fwd_vec<T, W, true>(a, st) : fwd_vec<T, W, false>(a, st);
    if (vec >= 2) return q8 ? fwd_vec<T, 2, true>(a, st) : fwd_vec<T, 2, false>(a, st);
    return q8 ? fwd_vec<T, 1, true>(a, st) : fwd_vec<T, 1, false>(a, st);
}

// Launch shape of the backward pass, shared with its workspace query: the number of blocks does not depend
// on alignment, only on rows, so that the query needs no pointers.
int bwd_blocks(int rows) { return std::max(1, std::min(rows, 4 * device_sms())); }

template <typename T, int VEC, int NV>
dlrm_status bwd_nv(const NormBwdArgs& a, int& nblocks, cudaStream_t st) {
    const int runs = (a.d + VEC - 1) / VEC;
    if (runs <= 32 * NV) {
        const int warps = 4;
        nblocks = bwd_blocks((a.rows + warps - 1) / warps);
        const dim3 grid(nblocks);
        const size_t smem = a.partial ? sizeof(float) * warps * NV * VEC * 32 : 0;
        DLRM_PDL_CHECK(launch_pdl(rmsnorm_bwd_kernel<T, VEC, NV, false, 128>, grid, dim3(32 * warps), smem, st, a));
        return DLRM_OK;
    }
    const int threads = ((runs + NV - 1) / NV + 31) / 32 * 32;
    nblocks = bwd_blocks(a.rows);
    const dim3 grid(nblocks);
    if (threads <= 256)
        DLRM_PDL_CHECK(launch_pdl(rmsnorm_bwd_kernel<T, VEC, NV, true, 256>, grid, dim3(threads), 0, st, a));
    else if (threads <= 1024)
        DLRM_PDL_CHECK(launch_pdl(rmsnorm_bwd_kernel<T, VEC, NV, true, 1024>, grid, dim3(threads), 0, st, a));
    else
        return DLRM_ERR_UNSUPPORTED;
    return DLRM_OK;
}

template <typename T, int VEC>
dlrm_status bwd_vec(const NormBwdArgs& a, int& nblocks, cudaStream_t st) {
    constexpr int W = 16 / (int)sizeof(T);
    const int runs = (a.d + VEC - 1) / VEC;
    if (runs <= 1024 * 2 * (W / VEC)) return bwd_nv<T, VEC, 2 * (W / VEC)>(a, nblocks, st);
    return bwd_nv<T, VEC, 32 / VEC>(a, nblocks, st);
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
    if (vec >= 2) return bwd_vec<T, 2>(a, nblocks, st);
    return bwd_vec<T, 1>(a, nblocks, st);
}

}  // namespace

dlrm_status launch_rmsnorm_fwd(int rows, int d, const void* x, long long ldx, const void* res, long long ldres,
                               const float* w, float eps, dlrm_dtype dt, void* h, long long ldh, void* y,
                               long long ldy, float* y_scale, float* rstd, cudaStream_t st) {
    const NormFwdArgs a{rows, d, eps, 1.f / (float)d, x, ldx, res, ldres, w, h, ldh, y, ldy, y_scale, rstd};
    const bool q8 = y_scale != nullptr;
    if (dt == DLRM_F32) return fwd_t<float>(a, q8, st);
    if (dt == DLRM_F16) return fwd_t<__half>(a, q8, st);
    return fwd_t<__nv_bfloat16>(a, q8, st);
}

size_t rmsnorm_bwd_partial_floats(int rows, int d) { return (size_t)bwd_blocks(rows) * d; }

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
    if (dw) DLRM_PDL_CHECK(launch_pdl(rmsnorm_dw_kernel, dim3((d + 31) / 32), dim3(1024), 0, st, nblocks, d,
                                      (const float*)partial, dw));
    return DLRM_OK;
}

}  // namespace dlrm

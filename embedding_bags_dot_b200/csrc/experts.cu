// Products grouped by expert, ragged: expert e owns rows [offsets[e],
// offsets[e + 1]) of the activations and one weight matrix W_e [N][K].
//   forward  Y  = act(X W_e^T + b_e)      per row          A = X  (K),  B = W_e (K)
//   dgrad    dX = dP W_e                  per row          A = dP (K),  B = W_e (MN)
//   wgrad    dW_e = dP_e^T X_e            over e's rows    A = dP (MN), B = X   (MN)
// with dP = dY where the forward's output is positive (ReLU) or dY itself.
// Operands are 16-bit (fp16 or bf16), the forward also e4m3 with one fp32
// scale per row of X and per row of W; accumulation is fp32.
//
// The offsets stay on the device: every CTA reads them after the previous
// kernel, checks them, and walks the same list of tiles (experts in order,
// then row blocks, then column blocks), taking every gridDim-th one. A row
// block past its expert's end multiplies rows of the next expert (or zeros)
// into accumulator rows that are never stored: rows do not mix. In wgrad rows
// are the reduction, so an expert's last, incomplete 64-row block is read from
// a copy padded with zeros (expert_prep_kernel), and no other row's infinity
// or NaN can reach it. Weights are three-dimensional tensor maps, so a block
// past row N of W_e reads zeros, not the next expert's weights.
//
// Two kernels on tcgen05 with TMA-fed 128-byte-swizzled shared memory:
//  - expert_pair_kernel: 256 x 256 tiles on SM pairs (cta_group::2): the forward,
//    or both products of the backward pass in one launch. Bound by the tensor
//    pipe at large sizes.
//  - expert_tile_kernel: tiles of 128 rows and 64 or 128 columns on one SM,
//    forward only, for calls too small to fill the pairs, where reading the
//    weights bounds the time. A row block of at most 32 rows loads 32 rows
//    instead of 128.
// The tensor core truncates as it accumulates, so no accumulator runs longer
// than 8 k-blocks (512 16-bit or 1,024 8-bit terms): the epilogue warps add each
// finished part to fp32 registers, rounding to nearest, while the next part
// accumulates in the other TMEM buffer.
// All waits are bounded: on timeout the kernel records DLRM_ERR_TIMEOUT, drains
// its copies and MMAs (again bounded), frees TMEM and returns. A warp gives up as one: what follows a wait is issued by
// all its lanes or by none. No multicast load.
//
// Alone, at burst clocks: 16,384 rows by 16 experts of 4,096 x 2,048 in e4m3 108 us
// (2.5 PFLOP/s, tensor pipe 85 % busy); dX and dW of 16,384 rows by 8 experts of
// 4,096 x 1,024 in bf16 198 us (1.39 PFLOP/s, 87 %), after 75 us of masking dY and
// summing the bias gradient (5.4 TB/s). Back to back at the 1,000 W cap 137 to 147
// and 326 us. 12 rows by 8 experts of 4,096 x 1,024: 12 to 15 us for the weights of
// the four to six experts that had rows, 34 to 50 MB, at 3 to 3.5 TB/s; in e4m3 11.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "kernels.cuh"
#include "rowvec.cuh"
#include "tcgen05.cuh"

namespace dlrm {
namespace tc {

constexpr int EX_MAX = DLRM_MAX_EXPERTS;
constexpr int PART = 8;                             // k-blocks per accumulator
constexpr int EX_THREADS2 = 384;                    // pair kernel: warps 0..3 TMA, MMA, idle; 4..11 epilogue
constexpr int EX_REGS_LOW = 40, EX_REGS_HIGH = 232;
static_assert(128 * EX_REGS_LOW + 256 * EX_REGS_HIGH <= 168 * EX_THREADS2, "register split exceeds the launch allocation");
constexpr int EX_STAGE2_BYTES = 32768;              // 128 rows x 128 bytes of A, as much of B
// Six stages: a pair multiplies a 16-bit stage in about 500 cycles and a load takes some 2,500 from the freed stage to
// the filled one (by the clock, all SMs loading), so every stage counts; five stages with a second output buffer per
// epilogue warp measured 32.6 us where six take 31.5 (20,000 rows, 24 experts of 1,024 x 479).
constexpr int EX_STAGES2 = 6;

enum ExpertOp { EX_FWD = 0, EX_BWD = 1 };
enum ExpertTile { ET_FWD = 0, ET_DGRAD = 1, ET_WGRAD = 2 };   // what a tile of the pair kernel computes
enum ExpertKind { EX_F16 = 0, EX_F8 = 1 };

struct ExpertArgs {
    int E, M;                 // experts; rows of the activations
    int J;                    // output columns: N (fwd), K (dX and dW)
    int I;                    // dW: output rows per expert (N), 0 without dW
    int R;                    // reduction length of fwd (K) and dX (N)
    bool rows_out;            // whether there is an output with rows (Y, dX)
    const int32_t* offsets;
    bool count;               // whether this launch reports bad ranges
    const float* bias;        // fwd, or null: [E][J]
    const float* x_scale;     // e4m3: [M]
    const float* w_scale;     // e4m3: [E][J]
    bool relu;
    void* C;                  // Y or dX
    long long ldc;
    void* D;                  // dW
    long long ldd;
    ErrRecord* err;
    bool give_up;             // test hook: every warp gives up before its first tile, as if that tile's wait had run out
};

struct ExpertMaps {
    CUtensorMap a, b, c;      // row operand, weights, output with rows
    CUtensorMap a32;          // tile kernel: 32-row boxes of A
};
struct GradMaps {
    CUtensorMap a, b, c;      // dX: dP, W, dX
    CUtensorMap wa, wb, wc;   // dW: dP, X, dW
    CUtensorMap at, bt;       // zero-padded last blocks of dP and X
};
template <int OP> struct PairMaps { using t = ExpertMaps; };
template <> struct PairMaps<EX_BWD> { using t = GradMaps; };

struct Ranges {
    int begin[EX_MAX];
    int end[EX_MAX];
};

template <int NS>
struct ExBars {
    unsigned long long full[NS];
    unsigned long long empty[NS];
    unsigned long long tfull[2];
    unsigned long long tempty[2];
    unsigned long long drain;
    unsigned int tmem_base;
    int abort;
};

// One warp fills the ranges. An expert whose range decreases, leaves [0, M] or starts before an earlier offset
// has no rows (and is counted), so ranges never overlap.
__device__ __forceinline__ void read_ranges(const ExpertArgs& a, Ranges* rg, bool count) {
    const int lane = threadIdx.x & 31;
    const int per = (a.E + 31) / 32;
    const int e0 = lane * per < a.E ? lane * per : a.E, e1 = e0 + per < a.E ? e0 + per : a.E;
    int most = 0;                 // largest offset in [e0, e1)
    for (int e = e0; e < e1; ++e) most = max(most, a.offsets[e]);
    int before = most;            // inclusive scan, then shifted: the largest offset before e0
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before = max(before, up);
    }
    before = __shfl_up_sync(0xffffffffu, before, 1);
    if (lane == 0) before = 0;
    unsigned bad = 0;
    for (int e = e0; e < e1; ++e) {
        const int s = a.offsets[e], t = a.offsets[e + 1];
        const bool ok = s >= before && t >= s && t <= a.M;
        before = max(before, s);
        bad += !ok;
        rg->begin[e] = ok ? s : 0;
        rg->end[e] = ok ? t : 0;
    }
    if (count) report_warp(a.err, 0, bad);
}

// Position in the list of tiles: experts in order, `per` column blocks for each of an expert's row blocks
// (a fixed number of tiles per expert in wgrad).
struct TileWalk {
    const Ranges* rg;
    int E, nb;                // experts; column blocks
    int rows_per;             // rows per row block; 0: `fixed` row blocks per expert
    int fixed;
    int e = 0;
    long long base = 0;       // tiles before expert e
    __device__ __forceinline__ long long tiles() const {
        const long long rb = rows_per ? (rg->end[e] - rg->begin[e] + rows_per - 1) / rows_per : fixed;
        return rb * nb;
    }
    // Moves on to the expert of tile t (t never decreases); false past the last tile.
    __device__ __forceinline__ bool seek(long long t, int& mb, int& cb) {
        while (e < E) {
            const long long n = tiles();
            if (t < base + n) {
                const int local = (int)(t - base);
                mb = local / nb;
                cb = local - mb * nb;
                return true;
            }
            base += n;
            ++e;
        }
        return false;
    }
};

// The pair kernel's list: the tiles of the output with rows first, then those of dW. In one launch, because either
// alone leaves SMs idle in its last round (270 and 512 tiles over 74 pairs in a batch of 16,384 rows).
struct TileList {
    TileWalk rows, mats;
    bool in_mats = false;
    long long off = 0;
    __device__ __forceinline__ bool seek(long long t, int& mb, int& cb) {
        if (!in_mats) {
            if (rows.seek(t, mb, cb)) return true;
            in_mats = true;
            off = rows.base;
        }
        return mats.seek(t - off, mb, cb);
    }
    __device__ __forceinline__ int expert() const { return in_mats ? mats.e : rows.e; }
};

// MN-major 16-bit operand with 128-byte swizzle: each reduction row is 128 bytes (64 consecutive M/N elements),
// 8-row groups are 1,024 bytes apart, 64-wide M/N blocks one 64-row box (8 KB) apart.
__device__ __forceinline__ uint64_t sdesc_mn16(uint32_t addr) {
    uint64_t d = (uint64_t)((addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(8192 >> 4) << 16;   // leading byte offset: next 64-wide M/N block
    d |= (uint64_t)(1024 >> 4) << 32;   // stride byte offset: next 8 reduction rows
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Instruction descriptor: fp32 accumulate; fmt: f16 kind 0 = fp16, 1 = bf16; f8f6f4 kind 0 = e4m3.
__host__ __device__ constexpr uint32_t ex_idesc(int fmt, bool a_mn, bool b_mn, int m, int n) {
    return (1u << 4) | ((uint32_t)fmt << 7) | ((uint32_t)fmt << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// The TMA and MMA warps run their loops with all lanes and issue from one elected lane: what the instructions
// take (descriptors, coordinates, addresses) is then the same for the warp and stays in uniform registers.
// Issued from a one-lane branch instead, a k-block of four MMAs took 640 cycles whatever its width (measured with
// the clock at 32, 64 and 128 columns), most of it moving operands into uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int uni(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint64_t desc64(uint32_t hi, uint32_t lo) { return ((uint64_t)hi << 32) | lo; }

template <int KIND, int CG>
__device__ __forceinline__ void ex_umma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accum) {
    if constexpr (KIND == EX_F16 && CG == 2) {
        umma2(d, a, b, id, accum);
    } else if constexpr (KIND == EX_F16) {
        umma(d, a, b, id, accum);
    } else if constexpr (CG == 2) {
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(accum));
    } else {
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(accum));
    }
}

__device__ __forceinline__ void ex_load_3d(uint32_t dst, const CUtensorMap* map, unsigned long long* bar, int x, int y,
                                           int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(su32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void ex_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t leader_bar, int x, int y,
                                                int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
        "%5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(leader_bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void ex_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// 32 TMEM columns straight into fp32 registers (valid after tmem_ld_wait)
__device__ __forceinline__ void tmem_ld32_f(uint32_t taddr, float (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%"
        "19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr));
}

// acc[c] += the 32 TMEM columns at taddr + 32 c, two loads in flight
template <int NC>
__device__ __forceinline__ void ex_promote(float (&acc)[NC][32], uint32_t taddr) {
#pragma unroll
    for (int c = 0; c < NC; c += 2) {
        float r[2][32];
        tmem_ld32_f(taddr + 32 * c, r[0]);
        tmem_ld32_f(taddr + 32 * c + 32, r[1]);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            acc[c][e] += r[0][e];
            acc[c + 1][e] += r[1][e];
        }
    }
}

// What the forward's epilogue needs besides the sums, fetched while the tile is still being multiplied: lane l
// holds the bias and weight scale of column 32 c + l of each 32-column group c, and the scale of its row.
template <int NC>
struct EpiRow {
    float bias[NC], wsc[NC], xs;
    bool far;          // whether any of the warp's scales is neither zero nor within 2^-60 .. 2^60
};
__device__ __forceinline__ bool far_scale(float s) { return s != 0.f && !(fabsf(s) >= 0x1p-60f && fabsf(s) <= 0x1p60f); }
template <int NC, int OP, int KIND>
__device__ __forceinline__ void ex_fetch(EpiRow<NC>& er, int row0, int nvalid, int j0, int e, const ExpertArgs& a) {
    if constexpr (OP == ET_FWD) {
        const int lane = threadIdx.x & 31;
        er.xs = KIND == EX_F8 && lane < nvalid ? __ldg(a.x_scale + row0 + lane) : 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = j0 + 32 * c + lane;
            const bool in = col < a.J;
            er.bias[c] = a.bias && in ? __ldg(a.bias + (long long)e * a.J + col) : 0.f;
            er.wsc[c] = KIND == EX_F8 && in ? __ldg(a.w_scale + (long long)e * a.J + col) : 0.f;
        }
        if constexpr (KIND == EX_F8) {
            bool far = far_scale(er.xs);
#pragma unroll
            for (int c = 0; c < NC; ++c) far |= far_scale(er.wsc[c]);
            er.far = __any_sync(0xffffffffu, far);
        }
    }
}

// Scales, bias and ReLU of 32 columns (group g of the warp's). A row's and a column's scale are multiplied first; where
// their product could leave fp32's range although the result does not, all three factors are multiplied in fp64.
template <int NC, int KIND>
__device__ __forceinline__ void ex_affine(float (&v)[32], const EpiRow<NC>& er, int g, const ExpertArgs& a) {
    if constexpr (KIND == EX_F8) {
        if (er.far) {
#pragma unroll
            for (int q = 0; q < 32; ++q)
                v[q] = (float)((double)v[q] * (double)er.xs * (double)__shfl_sync(0xffffffffu, er.wsc[g], q));
        } else {
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] *= er.xs * __shfl_sync(0xffffffffu, er.wsc[g], q);
        }
    }
    if (a.bias) {
#pragma unroll
        for (int q = 0; q < 32; ++q) v[q] += __shfl_sync(0xffffffffu, er.bias[g], q);
    }
    if (a.relu) {
        // not fmaxf: a NaN stays one
#pragma unroll
        for (int q = 0; q < 32; ++q) v[q] = v[q] < 0.f ? 0.f : v[q];
    }
}

// One warp's share of a finished tile: 32 rows (one per lane) x 32 NC columns from column j0. Rows go out
// through the warp's 4 KB stage, 128 bytes of columns at a time: whole 32-row groups by TMA, a group that holds the
// expert's last row by 16-byte stores of its valid rows only. TMA clips a box at 16 bytes: of a width that is no multiple
// of that it has the columns before, and the others go out one by one (by TMA they would take up to 15 bytes beside the
// matrix with them).
//   row0: first output row of the warp; nvalid: its rows that exist (<= 0: none); e: expert
template <typename TC, int NC, int OP, int KIND>
__device__ __forceinline__ void ex_store(float (&acc)[NC][32], const EpiRow<NC>& er, int row0, int nvalid, int j0, int e,
                                         const ExpertArgs& a, const CUtensorMap* mapC, unsigned char* stage,
                                         uint32_t stage_s) {
    constexpr int CW = 128 / (int)sizeof(TC);   // columns per 128 bytes: 32 (fp32) or 64
    constexpr int PER = CW / 32;                // 32-column groups per 128 bytes
    const int lane = threadIdx.x & 31;
    if (nvalid <= 0) return;                    // uniform across the warp
#pragma unroll
    for (int c = 0; c < NC / PER; ++c) {
        const int n0 = j0 + c * CW;
        if (n0 >= a.J) break;                   // uniform across the warp
        if constexpr (OP == ET_FWD) {
#pragma unroll
            for (int p = 0; p < PER; ++p) ex_affine<NC, KIND>(acc[c * PER + p], er, c * PER + p, a);
        }
        if (lane == 0) bulk_wait_read0();       // the previous chunk's store has read the stage
        __syncwarp();
        unsigned char* row = stage + lane * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            uint4 w;
            if constexpr (sizeof(TC) == 2) {
                union {
                    uint32_t t[4];
                    uint4 w;
                } u;
#pragma unroll
                for (int k = 0; k < 8; k += 2)
                    u.t[k / 2] = Pair<TC>::from_f(acc[c * PER + q / 4][(q % 4) * 8 + k], acc[c * PER + q / 4][(q % 4) * 8 + k + 1]);
                w = u.w;
            } else {
                w = make_uint4(__float_as_uint(acc[c][4 * q]), __float_as_uint(acc[c][4 * q + 1]),
                               __float_as_uint(acc[c][4 * q + 2]), __float_as_uint(acc[c][4 * q + 3]));
            }
            *reinterpret_cast<uint4*>(row + 16 * (q ^ (lane & 7))) = w;
        }
        constexpr int E16 = 16 / (int)sizeof(TC);
        auto out = [&](int r, int col) {
            return OP == ET_WGRAD ? static_cast<TC*>(a.D) + ((long long)e * a.I + row0 + r) * a.ldd + col
                                  : static_cast<TC*>(a.C) + (long long)(row0 + r) * a.ldc + col;
        };
        if (OP == ET_WGRAD || nvalid >= 32) {
            const int whole = a.J / E16 * E16;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0 && n0 < whole) {
                if constexpr (OP == ET_WGRAD) ex_store_3d(mapC, stage_s, n0, row0, e);
                else tma_store_2d(mapC, stage_s, n0, row0);
            }
            if (whole < a.J && n0 + CW > whole && lane < nvalid) {
                const uint4 w = *reinterpret_cast<const uint4*>(row + 16 * (((whole - n0) / E16) ^ (lane & 7)));
                const TC* src = reinterpret_cast<const TC*>(&w);
                TC* dst = out(lane, whole);
#pragma unroll
                for (int k = 0; k < E16 - 1; ++k)
                    if (whole + k < a.J) dst[k] = src[k];
            }
        } else {
            __syncwarp();
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const int r = it * 4 + (lane >> 3), q = lane & 7;
                const int col = n0 + q * E16;
                if (r < nvalid && col < a.J) {
                    const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 128 + 16 * (q ^ (r & 7)));
                    TC* dst = out(r, col);
                    if (col + E16 <= a.J) {
                        *reinterpret_cast<uint4*>(dst) = w;
                    } else {
                        const TC* src = reinterpret_cast<const TC*>(&w);
#pragma unroll
                        for (int k = 0; k < E16; ++k)
                            if (col + k < a.J) dst[k] = src[k];
                    }
                }
            }
            __syncwarp();
        }
    }
}

// k-blocks of a reduction.
template <int KIND>
__device__ __forceinline__ int ex_kblocks(int len) {
    constexpr int KE = KIND == EX_F8 ? 128 : 64;
    return (len + KE - 1) / KE;
}

// TC: type of the output with rows; TW: of dW (EX_BWD)
template <typename TC, typename TW, int OP, int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(EX_THREADS2, 1)
    expert_pair_kernel(const __grid_constant__ typename PairMaps<OP>::t maps, const __grid_constant__ ExpertArgs a, uint32_t id,
                       uint32_t id_dw) {
    constexpr bool BMN = OP != EX_FWD;
    constexpr int KE = KIND == EX_F8 ? 128 : 64;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = su32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    constexpr int NS = EX_STAGES2;
    Ranges* rg = reinterpret_cast<Ranges*>(gbase + NS * EX_STAGE2_BYTES + OUT_BYTES);
    ExBars<NS>* bars = reinterpret_cast<ExBars<NS>*>(rg + 1);
    const int warp = uni(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int npair = gridDim.x >> 1, pair = blockIdx.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->tfull[i], 1);
            mbar_init(&bars->tempty[i], 2 * EPI_WARPS);
        }
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&bars->tmem_base)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    pdl_wait();
    if (warp == 2) read_ranges(a, rg, a.count && blockIdx.x == 0);
    fence_before();
    cluster_sync_all();
    fence_after();
    const uint32_t tmem = uni(bars->tmem_base);
    volatile int* abort = &bars->abort;
    bool timed_out = false;
    const int nbj = (a.J + 255) / 256, E = a.give_up ? 0 : a.E;
    TileList walk{{rg, E, a.rows_out ? nbj : 0, 256, 0}, {rg, OP == EX_BWD ? E : 0, nbj, 0, (a.I + 255) / 256}};
    int mb, cb;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(EX_REGS_LOW));
        if (warp == 0) {
            int s = 0;
            uint32_t ph = 0;
            for (long long t = pair; !timed_out && uni(walk.seek(t, mb, cb)); t += npair) {
                const int e = uni(walk.expert()), r0 = uni(rg->begin[e]), rows = uni(rg->end[e]) - r0;
                const bool dw = OP == EX_BWD && uni(walk.in_mats);
                const int nk = ex_kblocks<KIND>(dw ? rows : a.R);
                const int arow = uni(mb) * 256 + (int)rank * 128, brow = uni(cb) * 256 + (int)rank * 128;
                for (int kb = 0; kb < nk; ++kb) {
                    if (!__all_sync(0xffffffffu, mbar_wait(&bars->empty[s], ph ^ 1u, abort))) {
                        timed_out = true;
                        break;
                    }
                    const uint32_t sa = base + s * EX_STAGE2_BYTES, sb = sa + EX_STAGE2_BYTES / 2;
                    const uint32_t bar = map_rank(su32(&bars->full[s]), 0);
                    if (elect_one()) {
                        if (leader) mbar_expect_tx(&bars->full[s], 2 * EX_STAGE2_BYTES);
                        if constexpr (OP == EX_FWD) {
                            tma_load_2d_pair(sa, &maps.a, bar, kb * KE, r0 + arow);
                            ex_load_3d_pair(sb, &maps.b, bar, kb * KE, brow, e);
                        } else if (!dw) {
                            tma_load_2d_pair(sa, &maps.a, bar, kb * KE, r0 + arow);
#pragma unroll
                            for (int b = 0; b < 2; ++b)
                                ex_load_3d_pair(sb + b * 8192, &maps.b, bar, brow + 64 * b, kb * KE, e);
                        } else if (kb * KE + KE <= rows) {
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                tma_load_2d_pair(sa + b * 8192, &maps.wa, bar, arow + 64 * b, r0 + kb * KE);
                                tma_load_2d_pair(sb + b * 8192, &maps.wb, bar, brow + 64 * b, r0 + kb * KE);
                            }
                        } else {
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                ex_load_3d_pair(sa + b * 8192, &maps.at, bar, arow + 64 * b, 0, e);
                                ex_load_3d_pair(sb + b * 8192, &maps.bt, bar, brow + 64 * b, 0, e);
                            }
                        }
                    }
                    __syncwarp();
                    if (++s == NS) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
        timed_out |= a.give_up;
        if (timed_out) *abort = 1;
            // every load this CTA issued completes before it may exit: the leader's MMA commits release
            // each stage after consuming it (bounded)
            for (int q = 0; q < NS; ++q) {
                mbar_wait(&bars->empty[s], ph ^ 1u, abort, true);
                if (++s == NS) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        } else if (warp == 1) {
            if (leader) {
                const uint64_t ak = sdesc(base), am = sdesc_mn16(base);      // A of rows, A of dW
                const uint64_t b0 = BMN ? sdesc_mn16(base + EX_STAGE2_BYTES / 2) : sdesc(base + EX_STAGE2_BYTES / 2);
                const uint32_t bhi = (uint32_t)(b0 >> 32);
                constexpr uint32_t BSTEP = (BMN ? 2048 : 32) >> 4;           // one MMA's depth
                int s = 0;
                uint32_t ph = 0, part = 0;   // accumulator parts so far: part n uses TMEM buffer n & 1
                for (long long t = pair; !timed_out && uni(walk.seek(t, mb, cb)); t += npair) {
                    const int e = walk.expert();
                    const bool dw = OP == EX_BWD && uni(walk.in_mats);
                    const int nk = uni(ex_kblocks<KIND>(dw ? rg->end[e] - rg->begin[e] : a.R));
                    const uint64_t a0 = dw ? am : ak;
                    const uint32_t ahi = (uint32_t)(a0 >> 32), astep = (dw ? 2048 : 32) >> 4, idt = dw ? id_dw : id;
                    for (int kb = 0; kb < nk; ++kb) {
                        const uint32_t acc = part & 1u;
                        bool ok = true;
                        if ((kb % PART) == 0) ok = mbar_wait(&bars->tempty[acc], ((part >> 1) & 1u) ^ 1u, abort);
                        ok = ok && mbar_wait(&bars->full[s], ph, abort);
                        if (!__all_sync(0xffffffffu, ok)) {
                            timed_out = true;
                            break;
                        }
                        fence_after();
                        const uint32_t d = tmem + acc * 256u;
                        const uint32_t alo = (uint32_t)a0 + s * (EX_STAGE2_BYTES >> 4);
                        const uint32_t blo = (uint32_t)b0 + s * (EX_STAGE2_BYTES >> 4);
                        const bool last = (kb % PART) == PART - 1 || kb + 1 == nk;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                ex_umma<KIND, 2>(d, desc64(ahi, alo + k * astep), desc64(bhi, blo + k * BSTEP), idt,
                                                 ((kb % PART) | k) != 0);
                            umma2_commit_both(&bars->empty[s]);
                            if (last) umma2_commit_both(&bars->tfull[acc]);
                        }
                        __syncwarp();
                        part += last;
                        if (++s == NS) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                }
        timed_out |= a.give_up;
        if (timed_out) *abort = 1;
                if (elect_one()) umma2_commit_both(&bars->drain);
                __syncwarp();
            }
            // the peer has nothing to issue; it waits for the leader's last MMA like the leader itself
            mbar_wait(&bars->drain, 0, abort, true);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EX_REGS_HIGH));
        const int ew = warp - 4, q = warp & 3, h = ew >> 2;
        unsigned char* stage = gbase + NS * EX_STAGE2_BYTES + ew * STAGE_OUT_BYTES;
        const uint32_t stage_s = base + NS * EX_STAGE2_BYTES + ew * STAGE_OUT_BYTES;
        const uint32_t lead_tempty0 = map_rank(su32(&bars->tempty[0]), 0);
        const uint32_t lead_tempty1 = map_rank(su32(&bars->tempty[1]), 0);
        uint32_t part = 0;
        for (long long t = pair; !timed_out && walk.seek(t, mb, cb); t += npair) {
            const int e = walk.expert(), r0 = rg->begin[e], rows = rg->end[e] - r0;
            const bool dw = OP == EX_BWD && walk.in_mats;
            const int parts = (ex_kblocks<KIND>(dw ? rows : a.R) + PART - 1) / PART;
            const int in_tile = mb * 256 + (int)rank * 128 + q * 32, j0 = cb * 256 + h * 128;
            const int row0 = dw ? in_tile : r0 + in_tile;
            const int nvalid = (dw ? a.I : rows) - in_tile;
            EpiRow<4> er;
            if constexpr (OP == EX_FWD) ex_fetch<4, ET_FWD, KIND>(er, row0, nvalid, j0, e, a);
            float acc[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int x = 0; x < 32; ++x) acc[c][x] = 0.f;
            for (int p = 0; p < parts; ++p, ++part) {
                const int b = (int)(part & 1u);
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->tfull[b], (part >> 1) & 1u, abort))) {
                    timed_out = true;
                    break;
                }
                fence_after();
                ex_promote<4>(acc, tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * 256 + h * 128));
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(b ? lead_tempty1 : lead_tempty0);
            }
            if (timed_out) break;
            if constexpr (OP == EX_FWD) {
                ex_store<TC, 4, ET_FWD, KIND>(acc, er, row0, nvalid, j0, e, a, &maps.c, stage, stage_s);
            } else if (dw) {
                ex_store<TW, 4, ET_WGRAD, KIND>(acc, er, row0, nvalid, j0, e, a, &maps.wc, stage, stage_s);
            } else {
                ex_store<TC, 4, ET_DGRAD, KIND>(acc, er, row0, nvalid, j0, e, a, &maps.c, stage, stage_s);
            }
        }
        timed_out |= a.give_up;
        if (timed_out) *abort = 1;
        if (lane == 0) bulk_wait_all0();
    }
    if (timed_out && lane == 0) atomicOr(&a.err->flags, (unsigned)ERR_TIMEOUT);
    fence_before();
    cluster_sync_all();   // no CTA frees TMEM or exits while its pair still signals it
    fence_after();
    if (warp == 1) {
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

// ------------------------------------------------------------------ one SM per tile (forward)

template <int BNT>
struct ExTile {
    static constexpr int NS = BNT == 64 ? 8 : 6;
    static constexpr int STAGE = (128 + BNT) * 128;
    static constexpr int TMEM = 2 * BNT;
    static constexpr int WC = 64;                            // columns per epilogue warp
    static constexpr int SMEM = NS * STAGE + OUT_BYTES + (int)sizeof(Ranges) + (int)sizeof(ExBars<NS>) + 256;
};

template <typename TC, int KIND, int BNT>
__global__ void __launch_bounds__(THREADS, 1)
    expert_tile_kernel(const __grid_constant__ ExpertMaps maps, const __grid_constant__ ExpertArgs a, uint32_t id) {
    using T = ExTile<BNT>;
    constexpr int NS = T::NS;
    constexpr int KE = KIND == EX_F8 ? 128 : 64;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = su32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    Ranges* rg = reinterpret_cast<Ranges*>(gbase + NS * T::STAGE + OUT_BYTES);
    ExBars<NS>* bars = reinterpret_cast<ExBars<NS>*>(rg + 1);
    const int warp = uni(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int nk = ex_kblocks<KIND>(a.R);
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->tfull[i], 1);
            mbar_init(&bars->tempty[i], EPI_WARPS);
        }
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&bars->tmem_base)),
                     "r"(T::TMEM));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.b)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.a32)) : "memory");
    }
    pdl_wait();
    if (warp == 2) read_ranges(a, rg, a.count && blockIdx.x == 0);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uni(bars->tmem_base);
    volatile int* abort = &bars->abort;
    bool timed_out = false;
    TileWalk walk{rg, a.give_up ? 0 : a.E, (a.J + BNT - 1) / BNT, 128, 0};
    int mb, cb;

    if (warp == 0) {
        int s = 0;
        uint32_t ph = 0;
        for (long long t = blockIdx.x; !timed_out && uni(walk.seek(t, mb, cb)); t += gridDim.x) {
            const int e = uni(walk.e), row = uni(rg->begin[e] + mb * 128), col = uni(cb) * BNT;
            const bool few = uni(rg->end[e]) - row <= 32;
            const uint32_t tx = (uint32_t)((few ? 32 : 128) + BNT) * 128u;
            for (int kb = 0; kb < nk; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->empty[s], ph ^ 1u, abort))) {
                    timed_out = true;
                    break;
                }
                const uint32_t sa = base + s * T::STAGE;
                if (elect_one()) {
                    mbar_expect_tx(&bars->full[s], tx);
                    if (few) tma_load_2d(sa, &maps.a32, &bars->full[s], kb * KE, row);
                    else tma_load_2d(sa, &maps.a, &bars->full[s], kb * KE, row);
                    ex_load_3d(sa + 128 * 128, &maps.b, &bars->full[s], kb * KE, col, e);
                }
                __syncwarp();
                if (++s == NS) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        timed_out |= a.give_up;
        if (timed_out) *abort = 1;
        // drain, also when another role gave up: every stage whose load may still be in flight completes its
        // full phase before the CTA may exit (a stage never loaded, or already consumed, passes at once)
        for (int q = 0; q < NS; ++q) {
            if (--s < 0) {
                s = NS - 1;
                ph ^= 1u;
            }
            mbar_wait(&bars->full[s], ph, abort, true);
        }
    } else if (warp == 1) {
        const uint64_t a0 = sdesc(base), b0 = sdesc(base + 128 * 128);
        const uint32_t ahi = (uint32_t)(a0 >> 32), bhi = (uint32_t)(b0 >> 32);
        int s = 0;
        uint32_t ph = 0, part = 0;
        for (long long t = blockIdx.x; !timed_out && uni(walk.seek(t, mb, cb)); t += gridDim.x) {
            for (int kb = 0; kb < nk; ++kb) {
                const uint32_t acc = part & 1u;
                bool ok = true;
                if ((kb % PART) == 0) ok = mbar_wait(&bars->tempty[acc], ((part >> 1) & 1u) ^ 1u, abort);
                ok = ok && mbar_wait(&bars->full[s], ph, abort);
                if (!__all_sync(0xffffffffu, ok)) {
                    timed_out = true;
                    break;
                }
                fence_after();
                const uint32_t d = tmem + acc * BNT;
                const uint32_t alo = (uint32_t)a0 + s * (T::STAGE >> 4), blo = (uint32_t)b0 + s * (T::STAGE >> 4);
                const bool last = (kb % PART) == PART - 1 || kb + 1 == nk;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        ex_umma<KIND, 1>(d, desc64(ahi, alo + 2 * k), desc64(bhi, blo + 2 * k), id, ((kb % PART) | k) != 0);
                    umma_commit(&bars->empty[s]);
                    if (last) umma_commit(&bars->tfull[acc]);
                }
                __syncwarp();
                part += last;
                if (++s == NS) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        timed_out |= a.give_up;
        if (timed_out) *abort = 1;
        if (elect_one()) umma_commit(&bars->drain);
        __syncwarp();
        mbar_wait(&bars->drain, 0, abort, true);
    } else {
        constexpr int NC = T::WC / 32;
        const int ew = warp - 2, q = warp & 3, h = ew >> 2;
        const bool active = h * T::WC < BNT;
        unsigned char* stage = gbase + NS * T::STAGE + ew * STAGE_OUT_BYTES;
        const uint32_t stage_s = base + NS * T::STAGE + ew * STAGE_OUT_BYTES;
        const int parts = (nk + PART - 1) / PART;
        uint32_t part = 0;
        for (long long t = blockIdx.x; !timed_out && walk.seek(t, mb, cb); t += gridDim.x) {
            const int e = walk.e, row = rg->begin[e] + mb * 128 + q * 32;
            const bool some = active && row < rg->end[e];
            const int nvalid = active ? rg->end[e] - row : 0, j0 = cb * BNT + h * T::WC;
            EpiRow<NC> er;
            ex_fetch<NC, ET_FWD, KIND>(er, row, nvalid, j0, e, a);
            float acc[NC][32];
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int x = 0; x < 32; ++x) acc[c][x] = 0.f;
            for (int p = 0; p < parts; ++p, ++part) {
                const int b = (int)(part & 1u);
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->tfull[b], (part >> 1) & 1u, abort))) {
                    timed_out = true;
                    break;
                }
                fence_after();
                if (some) ex_promote<NC>(acc, tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * BNT + h * T::WC));
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->tempty[b]);
            }
            if (timed_out) break;
            if (some) ex_store<TC, NC, ET_FWD, KIND>(acc, er, row, nvalid, j0, e, a, &maps.c, stage, stage_s);
        }
        timed_out |= a.give_up;
        if (timed_out) *abort = 1;
        if (lane == 0) bulk_wait_all0();
    }
    if (timed_out && lane == 0) atomicOr(&a.err->flags, (unsigned)ERR_TIMEOUT);
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(T::TMEM));
    }
}

constexpr int EX_SMEM2 =
    EX_STAGES2 * EX_STAGE2_BYTES + OUT_BYTES + (int)sizeof(Ranges) + (int)sizeof(ExBars<EX_STAGES2>) + 256;
static_assert(EX_SMEM2 <= 227 * 1024, "shared memory");
static_assert(ExTile<64>::SMEM <= 227 * 1024 && ExTile<128>::SMEM <= 227 * 1024, "shared memory");

// ------------------------------------------------------------------ backward: dP, bias sums, padded last blocks

struct PrepArgs {
    ExpertArgs x;             // E, M, offsets, count, err
    int N, K;
    int nslices;              // column slices of dY; the slices after them are X's
    const void* dY;
    long long lddy;
    const void* Y;            // ReLU: the forward's output
    long long ldyy;
    const void* X;
    long long ldx;
    void* dP;                 // ReLU: the masked gradient [M][ldp]
    long long ldp;
    float* part;              // bias sums: [chunk][N], or null
    void* tail_dp;            // [E][64][ldp], or null
    void* tail_x;             // [E][64][ldtx]
    long long ldtx;
};

constexpr int PREP_ROWS = 64;     // rows per chunk: one reduction block of wgrad
constexpr int PREP_COLS = 8;      // columns per thread: 16 bytes
constexpr int PREP_RUNS = 64;     // column runs of a block: 512 columns, each run by four threads of 16 rows
constexpr int PREP_SPAN = PREP_RUNS * PREP_COLS;

// The expert and first row of chunk number `chunk` (experts in order, each cut into 64-row chunks from its first
// row), found by the whole block's first warp; e = E if there is no such chunk.
__device__ __forceinline__ void find_chunk(const Ranges* rg, int E, long long chunk, int* e_out, long long* j_out) {
    const int lane = threadIdx.x & 31;
    long long seen = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        const long long mine = e < E ? (rg->end[e] - rg->begin[e] + PREP_ROWS - 1) / PREP_ROWS : 0;
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const bool here = chunk >= seen + incl - mine && chunk < seen + incl;
        if (here) {
            *e_out = e;
            *j_out = chunk - (seen + incl - mine);
        }
        if (__any_sync(0xffffffffu, here)) return;
        seen += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) *e_out = E;
}

// A run of which the first `valid` columns exist: the rest reads as zeros.
template <typename T>
__device__ __forceinline__ void load_run(RowRaw<T, PREP_COLS>& v, const T* p, int valid) {
    if (valid == PREP_COLS) {
        v.load(p);
    } else {
        v.zero();
#pragma unroll
        for (int k = 0; k < PREP_COLS; ++k)
            if (k < valid) v.e[k] = p[k];
    }
}

// Blocks take (chunk, slice) after (chunk, slice): up to 64 rows x 512 columns. Thread (run, quarter) has a run of
// 8 columns of 16 rows, so that a chunk takes two rounds of eight loads, not sixteen of four; the quarters' column
// sums are added in order.
template <typename T>
__global__ void __launch_bounds__(256) expert_prep_kernel(const __grid_constant__ PrepArgs a) {
    pdl_wait();
    __shared__ Ranges rg;
    __shared__ int se;
    __shared__ long long sj;
    __shared__ float quarter[3][PREP_RUNS][PREP_COLS + 1];
    if (threadIdx.x < 32) read_ranges(a.x, &rg, a.x.count && blockIdx.x == 0 && blockIdx.y == 0);
    const bool is_x = (int)blockIdx.y >= a.nslices;
    const int run = threadIdx.x % PREP_RUNS, q = threadIdx.x / PREP_RUNS;
    const long long c = (is_x ? blockIdx.y - a.nslices : blockIdx.y) * (long long)PREP_SPAN + run * PREP_COLS;
    const long long width = is_x ? a.K : a.N;
    const int valid = width - c >= PREP_COLS ? PREP_COLS : width > c ? (int)(width - c) : 0;
    const bool mask = a.Y != nullptr;
    for (long long chunk = blockIdx.x;; chunk += gridDim.x) {
        __syncthreads();
        if (threadIdx.x < 32) find_chunk(&rg, a.x.E, chunk, &se, &sj);
        __syncthreads();
        const int e = se;
        if (e >= a.x.E) return;
        const long long r0 = rg.begin[e] + sj * PREP_ROWS;
        const int rows = (int)(rg.end[e] - r0 < PREP_ROWS ? rg.end[e] - r0 : PREP_ROWS);
        const bool tail = rows < PREP_ROWS && a.tail_dp;
        // X only has its last, incomplete blocks copied; so has dY where neither ReLU nor bias sums are wanted
        if (is_x || (!mask && !a.part))
            if (!tail) continue;
        const T* src = is_x ? static_cast<const T*>(a.X) + r0 * a.ldx + c : static_cast<const T*>(a.dY) + r0 * a.lddy + c;
        const long long ld = is_x ? a.ldx : a.lddy, ldt = is_x ? a.ldtx : a.ldp;
        const T* y = mask && !is_x ? static_cast<const T*>(a.Y) + r0 * a.ldyy + c : nullptr;
        T* dp = mask && !is_x ? static_cast<T*>(a.dP) + r0 * a.ldp + c : nullptr;
        T* tl = tail ? static_cast<T*>(is_x ? a.tail_x : a.tail_dp) + (long long)e * PREP_ROWS * ldt + c : nullptr;
        float sum[PREP_COLS];
#pragma unroll
        for (int k = 0; k < PREP_COLS; ++k) sum[k] = 0.f;
        constexpr int U = 8, PER = PREP_ROWS / 4;
        if (valid > 0) {
#pragma unroll 1
            for (int i = 0; i < PER; i += U) {
                RowRaw<T, PREP_COLS> g[U], f[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = q * PER + i + u;
                    if (r < rows) {
                        load_run(g[u], src + r * ld, valid);
                        if (y) load_run(f[u], y + r * a.ldyy, valid);
                    } else {
                        g[u].zero();
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = q * PER + i + u;
                    float v[PREP_COLS];
                    g[u].get(v);
                    if (y && r < rows) {
                        float o[PREP_COLS];
                        f[u].get(o);
#pragma unroll
                        for (int k = 0; k < PREP_COLS; ++k)
                            if (!(o[k] > 0.f)) v[k] = 0.f;
                        g[u].set(v);
                        g[u].store(dp + r * a.ldp);
                    }
                    if (tl) g[u].store(tl + r * ldt);       // rows past the last are the zeros
#pragma unroll
                    for (int k = 0; k < PREP_COLS; ++k) sum[k] += v[k];
                }
            }
        }
        if (!a.part || is_x) continue;
        if (q > 0) {
#pragma unroll
            for (int k = 0; k < PREP_COLS; ++k) quarter[q - 1][run][k] = sum[k];
        }
        __syncthreads();
        if (q == 0) {
#pragma unroll
            for (int k = 0; k < PREP_COLS; ++k) {
                float s = sum[k];
#pragma unroll
                for (int p = 0; p < 3; ++p) s += quarter[p][run][k];
                if (k < valid) a.part[chunk * a.N + c + k] = s;
            }
        }
    }
}

// db[e][n] = sum over the expert's chunks: 32 columns a block, eight contiguous shares of the chunks added in order.
__global__ void __launch_bounds__(256) expert_bias_kernel(const __grid_constant__ ExpertArgs a, int N,
                                                          const float* __restrict__ part, float* __restrict__ db) {
    pdl_wait();
    __shared__ Ranges rg;
    __shared__ long long first;
    __shared__ float share[8][33];
    const int e = blockIdx.y;
    if (threadIdx.x < 32) {
        read_ranges(a, &rg, a.count && blockIdx.x == 0 && e == 0);
        __syncwarp();
        long long s = 0;
        for (int q = threadIdx.x; q < e; q += 32) s += (rg.end[q] - rg.begin[q] + PREP_ROWS - 1) / PREP_ROWS;
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) first = s;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int n = blockIdx.x * 32 + lane;
    const int chunks = (rg.end[e] - rg.begin[e] + PREP_ROWS - 1) / PREP_ROWS;
    const int per = (chunks + 7) / 8;
    const int j0 = g * per, j1 = j0 + per < chunks ? j0 + per : chunks;
    float s = 0.f;
    if (n < N) {
        const float* p = part + first * N + n;
#pragma unroll 8
        for (int j = j0; j < j1; ++j) s += p[(long long)j * N];
    }
    share[g][lane] = s;
    __syncthreads();
    if (g == 0 && n < N) {
        s = share[0][lane];
#pragma unroll
        for (int q = 1; q < 8; ++q) s += share[q][lane];
        db[(long long)e * N + n] = s;
    }
}

// ------------------------------------------------------------------ host side

namespace {

std::atomic<bool> g_give_up{false};     // dlrm_set_wait_polls(0)

bool ex_map(CUtensorMap* m, const void* p, int es, dlrm_dtype dt, int rank, long long inner, long long mid, long long outer,
            long long ld, int box_inner, int box_mid) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)mid, (cuuint64_t)outer};
    const cuuint64_t strides[2] = {(cuuint64_t)(ld * es), (cuuint64_t)(mid * ld * es)};
    const cuuint32_t box[3] = {(cuuint32_t)box_inner, (cuuint32_t)box_mid, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUtensorMapDataType t = dt == DLRM_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                  : dt == DLRM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                  : dt == DLRM_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                   : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    return enc(m, t, rank, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Columns of an output's map: whole runs of 16 bytes (a map has at least one; of narrower outputs TMA stores nothing).
long long ex_whole(long long cols, int es) { return std::max<long long>(cols * es / 16, 1) * (16 / es); }

int ex_size(dlrm_dtype dt) { return dt == DLRM_F32 ? 4 : dt == DLRM_E4M3 ? 1 : 2; }

// Most tiles a call can have: row blocks of every expert, the experts with rows being at most min(E, M).
long long most_tiles(int E, long long M, int rows_per, long long nb) {
    return (M / rows_per + std::min<long long>(E, M)) * nb;
}

template <typename TC, typename TW, int OP, int KIND>
dlrm_status launch_pair(const typename PairMaps<OP>::t& maps, const ExpertArgs& a, uint32_t id, uint32_t id_dw,
                        long long tiles, cudaStream_t st) {
    auto kern = expert_pair_kernel<TC, TW, OP, KIND>;
    cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, EX_SMEM2);
    const int pairs = device_sms() / 2;
    const dim3 grid((unsigned)(2 * std::min<long long>(tiles, pairs)));
    DLRM_PDL_CHECK(launch_pdl(kern, grid, dim3(EX_THREADS2), (size_t)EX_SMEM2, st, maps, a, id, id_dw));
    return DLRM_OK;
}

template <typename TC, int KIND, int BNT>
dlrm_status launch_tile(const ExpertMaps& maps, const ExpertArgs& a, int fmt, cudaStream_t st) {
    auto kern = expert_tile_kernel<TC, KIND, BNT>;
    constexpr int SMEM = ExTile<BNT>::SMEM;
    cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    const long long tiles = most_tiles(a.E, a.M, 128, (a.J + BNT - 1) / BNT);
    const dim3 grid((unsigned)std::min<long long>(tiles, device_sms()));
    DLRM_PDL_CHECK(launch_pdl(kern, grid, dim3(THREADS), (size_t)SMEM, st, maps, a,
                              ex_idesc(fmt, false, false, 128, BNT)));
    return DLRM_OK;
}

}  // namespace
}  // namespace tc

dlrm_status launch_experts_fwd(int E, int M, int N, int K, const int32_t* offsets, const void* X, long long ldx,
                               const float* x_scale, dlrm_dtype dt, const void* W, long long ldw, const float* w_scale,
                               const float* bias, bool relu, void* Y, long long ldy, dlrm_dtype y_dt, ErrRecord* err,
                               cudaStream_t st) {
    using namespace tc;
    const int es = ex_size(dt), ke = 128 / es;
    const ExpertArgs a{E, M, N, 0, K, true, offsets, true, bias, x_scale, w_scale, relu, Y, ldy, nullptr, 0, err,
                       g_give_up.load(std::memory_order_relaxed)};
    // Tiles of 256 x 256 on SM pairs, or of 128 x 128 or 128 x 64 on single SMs: whichever rounds of tiles take least,
    // by times of whole rounds (us: a round's k-blocks and what it costs besides; the pairs' later start). Short reductions
    // and calls of few rounds take up to twice as long as these say, all shapes alike, so the choice holds. Measured
    // (pairs; 128 columns; 64): 4 experts of 4,096 x 1,024 bf16, 8,192 rows 57, 71, 106, 512 rows 15.6, 15.0, 16.0;
    // 4 of 1,024 x 4,096, 4,096 rows 35, 37, 58, 2,048 rows 26, 21, 32; 8 of 4,096 x 1,024, 64 rows 19.6, 16.0, 19.3,
    // 12 rows 19.9, 14.8, 15.7 (and 17.6 at 32 columns beside 13.6 at 128 then: a k-block's issue costs 420 to 465 cycles
    // at any width); 24 of 1,024 x 479 fp16, 20,000 rows 26.7, 31.3, 41.4; 8 of 2,048 x 256, 5,000 rows 14.9, 12.5, 16.2;
    // 16 of 4,096 x 2,048 e4m3, 16,384 rows 127, 154, 227, 1,000 rows 35.7, 30.8, 36.8.
    const long long sms = device_sms(), used = std::min(E, M);
    const double nk = (K + ke - 1) / ke;
    auto rounds = [&](long long rows_per, long long cols, long long units) {
        // row blocks of unevenly filled experts: half a block each is lost to their last rows, and where most fit one
        // block some need two
        const double full = (double)M / rows_per;
        const double rb = full >= used ? full + 0.5 * used : used + 0.4 * full;
        return std::ceil(rb * (double)((N + cols - 1) / cols) / (double)units);
    };
    const double t256 = rounds(256, 256, sms / 2) * (0.3 * nk + 1.5) + 2.5;
    const double t128 = rounds(128, 128, sms) * (0.245 * nk + 1.0), t64 = rounds(128, 64, sms) * (0.22 * nk + 1.0);
    const bool pair = t256 < std::min(t128, t64), narrow = t64 < t128;
    ExpertMaps maps{};
    // the tile kernel's A comes in boxes of 128 rows or, for row blocks of at most 32, of 32
    const bool only32 = !pair && M <= 32;
    if ((!only32 && !ex_map(&maps.a, X, es, dt, 2, K, M, 1, ldx, ke, 128)) ||
        (!pair && !ex_map(&maps.a32, X, es, dt, 2, K, M, 1, ldx, ke, 32)) ||
        !ex_map(&maps.b, W, es, dt, 3, K, N, E, ldw, ke, pair || !narrow ? 128 : 64) ||
        !ex_map(&maps.c, Y, ex_size(y_dt), y_dt, 2, ex_whole(N, ex_size(y_dt)), M, 1, ldy, 128 / ex_size(y_dt), 32))
        return DLRM_ERR_CUDA;
    const int fmt = dt == DLRM_BF16 ? 1 : 0;
#define DLRM_EX_FWD(TC, KIND)                                                                     \
    return pair ? launch_pair<TC, TC, EX_FWD, KIND>(maps, a, ex_idesc(fmt, false, false, 256, 256), \
                                                    0u, most_tiles(E, M, 256, (N + 255) / 256), st) \
           : narrow ? launch_tile<TC, KIND, 64>(maps, a, fmt, st)                                 \
                    : launch_tile<TC, KIND, 128>(maps, a, fmt, st);
    if (dt == DLRM_E4M3) {
        if (y_dt == DLRM_F32) DLRM_EX_FWD(float, EX_F8)
        if (y_dt == DLRM_BF16) DLRM_EX_FWD(__nv_bfloat16, EX_F8)
        DLRM_EX_FWD(__half, EX_F8)
    }
    if (y_dt == DLRM_F32) DLRM_EX_FWD(float, EX_F16)
    if (y_dt == DLRM_BF16) DLRM_EX_FWD(__nv_bfloat16, EX_F16)
    DLRM_EX_FWD(__half, EX_F16)
#undef DLRM_EX_FWD
}

ExpertsLayout experts_layout(int E, long long M, int N, int K, bool relu) {
    ExpertsLayout L;
    size_t off = align_up(DLRM_ERR_RECORD_BYTES, 256);
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = align_up(off + bytes, 256);
        return o;
    };
    L.ldp = (N + 7) / 8 * 8;
    L.ldtx = (K + 7) / 8 * 8;
    L.dp = take(relu ? (size_t)2 * M * L.ldp : 0);
    L.tail_dp = take((size_t)2 * E * tc::PREP_ROWS * L.ldp);
    L.tail_x = take((size_t)2 * E * tc::PREP_ROWS * L.ldtx);
    L.part = take(sizeof(float) * (size_t)(M / tc::PREP_ROWS + E) * N);
    L.total = off;
    return L;
}

dlrm_status launch_experts_bwd(int E, int M, int N, int K, const int32_t* offsets, const void* dY, long long lddy,
                               const void* Y, long long ldyy, const void* X, long long ldx, const void* W, long long ldw,
                               dlrm_dtype dt, void* dX, long long lddx, dlrm_dtype dx_dt, void* dW, long long lddw,
                               dlrm_dtype dw_dt, float* db, char* ws, cudaStream_t st) {
    using namespace tc;
    const bool relu = Y != nullptr;
    const ExpertsLayout L = experts_layout(E, M, N, K, relu);
    ErrRecord* err = reinterpret_cast<ErrRecord*>(ws);
    ExpertArgs a{E, M, K, dW ? N : 0, N, dX != nullptr, offsets, true, nullptr, nullptr, nullptr, false, dX, lddx, dW, lddw, err,
                 g_give_up.load(std::memory_order_relaxed)};
    float* part = reinterpret_cast<float*>(ws + L.part);
    const void* dP = relu ? (const void*)(ws + L.dp) : dY;
    const long long ldp = relu ? L.ldp : lddy;
    // every map is encoded before anything is launched
    GradMaps maps{};
    const long long nbk = (K + 255) / 256;
    long long tiles = 0;
    a.rows_out = dX && M > 0;
    if (a.rows_out) {
        if (!ex_map(&maps.a, dP, 2, dt, 2, N, M, 1, ldp, 64, 128) || !ex_map(&maps.b, W, 2, dt, 3, K, N, E, ldw, 64, 64) ||
            !ex_map(&maps.c, dX, ex_size(dx_dt), dx_dt, 2, ex_whole(K, ex_size(dx_dt)), M, 1, lddx, 128 / ex_size(dx_dt), 32))
            return DLRM_ERR_CUDA;
        tiles += most_tiles(E, M, 256, nbk);
    }
    if (dW) {
        // without rows nothing is loaded; the maps still need an address
        const void* pa = M > 0 ? dP : ws + L.tail_dp;
        const void* pb = M > 0 ? X : ws + L.tail_x;
        const long long rows = M > 0 ? M : 1;
        if (!ex_map(&maps.wa, pa, 2, dt, 2, N, rows, 1, M > 0 ? ldp : L.ldp, 64, 64) ||
            !ex_map(&maps.wb, pb, 2, dt, 2, K, rows, 1, M > 0 ? ldx : L.ldtx, 64, 64) ||
            !ex_map(&maps.at, ws + L.tail_dp, 2, dt, 3, N, PREP_ROWS, E, L.ldp, 64, 64) ||
            !ex_map(&maps.bt, ws + L.tail_x, 2, dt, 3, K, PREP_ROWS, E, L.ldtx, 64, 64) ||
            !ex_map(&maps.wc, dW, ex_size(dw_dt), dw_dt, 3, ex_whole(K, ex_size(dw_dt)), N, E, lddw, 128 / ex_size(dw_dt), 32))
            return DLRM_ERR_CUDA;
        tiles += (long long)E * ((N + 255) / 256) * nbk;
    }
    if (M > 0 && (relu || db || dW)) {
        PrepArgs p{};
        p.x = a;
        p.N = N;
        p.K = K;
        p.nslices = (N + PREP_SPAN - 1) / PREP_SPAN;
        const int xs = dW ? (K + PREP_SPAN - 1) / PREP_SPAN : 0;
        p.dY = dY;
        p.lddy = lddy;
        p.Y = Y;
        p.ldyy = ldyy;
        p.X = X;
        p.ldx = ldx;
        p.dP = ws + L.dp;
        p.ldp = L.ldp;
        p.part = db ? part : nullptr;
        p.tail_dp = dW ? ws + L.tail_dp : nullptr;
        p.tail_x = dW ? ws + L.tail_x : nullptr;
        p.ldtx = L.ldtx;
        // at most six blocks per SM, each of which looks up its ranges once
        const int chunks = M / PREP_ROWS + std::min(E, M), slices = p.nslices + xs;
        const dim3 grid((unsigned)std::min(chunks, std::max(1, 6 * device_sms() / slices)), slices);
        if (dt == DLRM_BF16) DLRM_PDL_CHECK(launch_pdl(expert_prep_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, p));
        else DLRM_PDL_CHECK(launch_pdl(expert_prep_kernel<__half>, grid, dim3(256), 0, st, p));
        a.count = false;
    }
    if (db) {
        DLRM_PDL_CHECK(launch_pdl(expert_bias_kernel, dim3((N + 31) / 32, E), dim3(256), 0, st, a, N,
                                  (const float*)part, db));
        a.count = false;
    }
    if (tiles == 0) return DLRM_OK;
    const int fmt = dt == DLRM_BF16 ? 1 : 0;
    const uint32_t id = ex_idesc(fmt, false, true, 256, 256), id_dw = ex_idesc(fmt, true, true, 256, 256);
    // an output that is not asked for takes the other's type
    const bool fx = dX ? dx_dt == DLRM_F32 : dw_dt == DLRM_F32, fw = dW ? dw_dt == DLRM_F32 : fx;
#define DLRM_EX_BWD(T)                                                                                               \
    return fx && fw ? launch_pair<float, float, EX_BWD, EX_F16>(maps, a, id, id_dw, tiles, st)                       \
           : fx     ? launch_pair<float, T, EX_BWD, EX_F16>(maps, a, id, id_dw, tiles, st)                           \
           : fw     ? launch_pair<T, float, EX_BWD, EX_F16>(maps, a, id, id_dw, tiles, st)                           \
                    : launch_pair<T, T, EX_BWD, EX_F16>(maps, a, id, id_dw, tiles, st);
    if (dt == DLRM_BF16) {
        DLRM_EX_BWD(__nv_bfloat16)
    }
    DLRM_EX_BWD(__half)
#undef DLRM_EX_BWD
}

void set_wait_polls_experts(long long polls) { tc::g_give_up.store(polls == 0, std::memory_order_relaxed); }

bool experts_supported() { return tc::encode_fn() != nullptr; }

}  // namespace dlrm

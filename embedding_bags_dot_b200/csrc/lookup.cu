// Unpooled lookups with scaling, and their gradient by sorted ids.
//
//   forward    out[i] = scale * T[idx_i]          (zeros for an index outside the table, which is counted)
//   backward   dT[r]  = scale * sum_{i : idx_i = r} dout[i], in order of i, for every row r of the table
//
// Forward: bound by memory (n rows read, n written). Each thread moves runs of
// up to 16 bytes of several rows, so that several row reads are in flight
// (65,536 rows of 1,024 bf16: 36 us, 7.5 TB/s with the frequent rows in L2).
//
// Backward: n rows of dout read once, m rows of the table's gradient written
// once; no atomics on values, so the result does not depend on timing.
//   1. (id, position) pairs are sorted by id, stably: an LSD radix sort whose
//      digits are as wide as the table needs (two passes up to 2^20 rows), in
//      one block up to 2,048 pairs, a cluster of sixteen up to 65,536 (7,375
//      pairs 15 us the call where blocks of eight with their pairs in memory took
//      24; 23,517 pairs 19 where four launches took 32), else, and where the
//      device cannot place sixteen blocks together, with a histogram and a
//      scatter launch per pass over blocks of 2,048.
//      The sort takes few SMs and little bandwidth, so the other blocks of
//      its launches write the table's zeros meanwhile; rows with lookups are
//      written again by the next steps.
//   2. The sorted pairs are cut into windows of fixed length, each summed by
//      one group of threads per column slice, whatever rows they belong to, so
//      that here a row looked up thousands of times costs no more per lookup
//      than any other. A run of equal ids inside a window is final and goes
//      straight to its row; the parts of a run that crosses windows go to a
//      partial buffer.
//   3. The partial sums of the crossing runs are added in window order, a run's
//      by one block per column slice. Here one id's share counts: all of 65,536
//      ids the same take 49 us at 512 columns where spread ids take 44, 60 at 8
//      columns where those take 28; all of 1,000,000 630 at 8 columns (80), 547
//      at 512 (268).
// 65,536 ids into 100,000 x 512 fp32 from bf16: 67 us, of which the sort with
// the zeros (205 MB) takes about 39, the sums 20 and the join 8; the least bytes
// would take 41. Calls of a few hundred ids take three launches, 11 us. Past the
// cluster's sort: 131,072 ids into the same 94 us (52), 1,000,000 ids into
// 100,000 x 64 107 us (24).
#include <algorithm>
#include <atomic>

#include "kernels.cuh"
#include "rowvec.cuh"
#include "tcgen05.cuh"

namespace dlrm {
namespace {

// ------------------------------------------------------------------ forward

struct LookupArgs {
    long long n;
    int d;
    long long rows;        // of the table
    const void* table;     // its first row
    const int32_t* idx;
    float scale;
    void* out;
    long long ldo;
    ErrRecord* err;
};

// blockDim = (TX, 256 / TX): TX threads along a row, each on run tx, tx + TX, ...; R rows at once per thread.
template <typename TI, typename TO, int VEC, int R>
__global__ void __launch_bounds__(256) lookup_kernel(const __grid_constant__ LookupArgs a) {
    pdl_wait();
    const TI* table = static_cast<const TI*>(a.table);
    TO* out = static_cast<TO*>(a.out);
    const int runs = a.d / VEC;
    for (long long i0 = ((long long)blockIdx.x * blockDim.y + threadIdx.y) * R; i0 < a.n;
         i0 += (long long)gridDim.x * blockDim.y * R) {
        long long row[R];
        unsigned bad = 0;
#pragma unroll
        for (int u = 0; u < R; ++u) {
            row[u] = -1;
            if (i0 + u < a.n) {
                const int v = a.idx[i0 + u];
                if (v >= 0 && v < a.rows) row[u] = v;
                else ++bad;
            }
        }
        if (bad && threadIdx.x == 0) report(a.err, bad, 0);
        for (int c = threadIdx.x; c < runs; c += blockDim.x) {
            RowRaw<TI, VEC> in[R];
#pragma unroll
            for (int u = 0; u < R; ++u) {
                if (row[u] >= 0) in[u].load(table + row[u] * a.d + (long long)c * VEC);
                else in[u].zero();
            }
#pragma unroll
            for (int u = 0; u < R; ++u) {
                if (i0 + u >= a.n) break;
                float v[VEC];
                in[u].get(v);
                // a skipped row is zero also under an infinite scale
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[e] = row[u] >= 0 ? v[e] * a.scale : 0.f;
                RowRaw<TO, VEC> o;
                o.set(v);
                o.store(out + (i0 + u) * a.ldo + (long long)c * VEC);
            }
        }
    }
}

int pow2_at_least(int n, int most) {
    int p = 1;
    while (p < n && p < most) p <<= 1;
    return p;
}

template <typename TI, typename TO, int VEC>
dlrm_status lookup_vec(const LookupArgs& a, cudaStream_t st) {
    const int tx = pow2_at_least(a.d / VEC, 256);
    const dim3 block(tx, 256 / tx);
    // four rows per thread once that still gives every SM several blocks
    const bool many = a.n / (4ll * block.y) >= 2ll * device_sms();
    const long long per = (long long)block.y * (many ? 4 : 1);
    const dim3 grid((unsigned)std::min<long long>((a.n + per - 1) / per, 1ll << 30));
    if (many) DLRM_PDL_CHECK(launch_pdl(lookup_kernel<TI, TO, VEC, 4>, grid, block, 0, st, a));
    else DLRM_PDL_CHECK(launch_pdl(lookup_kernel<TI, TO, VEC, 1>, grid, block, 0, st, a));
    return DLRM_OK;
}

template <typename TI, typename TO>
dlrm_status lookup_to(const LookupArgs& a, cudaStream_t st) {
    // runs of 16 bytes of the narrower type where every row allows it, else the widest that do
    constexpr int W = 16 / (int)(sizeof(TI) < sizeof(TO) ? sizeof(TI) : sizeof(TO));
    auto fits = [&](int vec) {
        const int bi = std::min(16, vec * (int)sizeof(TI)), bo = std::min(16, vec * (int)sizeof(TO));
        return a.d % vec == 0 && rows_on(a.table, (long long)a.d * sizeof(TI), bi) &&
               rows_on(a.out, a.ldo * (long long)sizeof(TO), bo);
    };
    if (fits(W)) return lookup_vec<TI, TO, W>(a, st);
    if constexpr (W > 4)
        if (fits(4)) return lookup_vec<TI, TO, 4>(a, st);
    if (fits(2)) return lookup_vec<TI, TO, 2>(a, st);
    return lookup_vec<TI, TO, 1>(a, st);
}

template <typename TI>
dlrm_status lookup_ti(const LookupArgs& a, dlrm_dtype out_dt, cudaStream_t st) {
    if (out_dt == DLRM_F32) return lookup_to<TI, float>(a, st);
    if (out_dt == DLRM_F16) return lookup_to<TI, __half>(a, st);
    return lookup_to<TI, __nv_bfloat16>(a, st);
}

// ------------------------------------------------------------------ sort of (id, position)

constexpr int DIG_BITS_MAX = 10;       // digits of up to 10 bits
constexpr int RS_ITEMS = 8;            // keys per thread and tile
// Ranking a warp's 32 keys costs about a hundred instructions, so a pass takes an SM the longer the more of them it
// has: 8,192 pairs on one SM took 10 us a pass. Blocks are small, and short calls alone stay in one.
constexpr int RS_THREADS = 256;
constexpr int RS_WARPS = RS_THREADS / 32;
constexpr int RS_TILE = RS_THREADS * RS_ITEMS;
constexpr int RS_BLOCKS_MAX = 296;
constexpr int SORT1_MAX = RS_TILE;      // pairs the one-block sort takes
constexpr int SORTC_MAX = 65536;        // pairs a cluster's sort takes

// A share of the table's bytes, zeroed by the blocks of a sorting launch that do not sort.
struct Zeros {
    char* base;
    long long begin, end;     // bytes
    int sorters;              // blocks of the launch that sort
};
__device__ __forceinline__ void write_zeros(const Zeros& z) {
    const long long nb = gridDim.x - z.sorters, b = (long long)blockIdx.x - z.sorters;
    // 16-byte stores from the first aligned address of the share; its ragged ends byte by byte
    char* p0 = z.base + z.begin;
    char* p1 = z.base + z.end;
    char* q0 = reinterpret_cast<char*>(((uintptr_t)p0 + 15) & ~(uintptr_t)15);
    if (q0 > p1) q0 = p1;
    char* q1 = q0 + ((p1 - q0) & ~(long long)15);
    const long long n16 = (q1 - q0) / 16;
    for (long long i = b * blockDim.x + threadIdx.x; i < n16; i += nb * blockDim.x)
        reinterpret_cast<uint4*>(q0)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (b == 0) {
        if ((long long)threadIdx.x < q0 - p0) p0[threadIdx.x] = 0;
        if ((long long)threadIdx.x < p1 - q1) q1[threadIdx.x] = 0;
    }
}

// Radix pass: block b owns keys [b * chunk, (b + 1) * chunk). FIRST reads the indices themselves.
template <bool FIRST>
__device__ __forceinline__ uint32_t pass_key(const void* in, long long i, long long m) {
    if constexpr (FIRST) {
        const int v = static_cast<const int32_t*>(in)[i];
        return v >= 0 && v < m ? (uint32_t)v : (uint32_t)m;
    } else {
        return static_cast<const uint32_t*>(in)[i];
    }
}

// Shared memory of a sorting block.
struct SortMem {
    unsigned short* wc;     // [warps][radix]: keys of a digit in each warp, then their places by warp
    int* tot;               // [radix]
    int* wsum;              // [32]
    uint32_t* keys;         // [tile]: the tile's pairs in order (the cluster's sort: [tile] of uint2)
    uint32_t* vals;
};
template <int WARPS = RS_WARPS>
__device__ __forceinline__ SortMem sort_mem(unsigned char* p, int radix) {
    SortMem s;
    s.wc = reinterpret_cast<unsigned short*>(p);
    s.tot = reinterpret_cast<int*>(p + 2 * WARPS * radix);
    s.wsum = s.tot + radix;
    s.keys = reinterpret_cast<uint32_t*>(s.wsum + 32);
    s.vals = s.keys + RS_TILE;
    return s;
}
constexpr size_t sort_bytes(int radix, int threads = RS_THREADS, int items = RS_ITEMS) {
    return (size_t)threads / 16 * radix + 4 * (size_t)radix + 128 + 8 * (size_t)threads * items;
}

// place[e] = how many keys of the block with the same digit come before the thread's e-th; sm.tot[digit] = how many
// there are. Key e of lane l in warp w is number (w * ITEMS + e) * 32 + l of the tile; those from `cnt` on do not count.
// Each warp counts its own keys 32 at a time (equal digits find each other by ballots, 2,400 cycles a block;
// match.any took 3,400), then each digit's counts
// are summed over the warps.
template <int THREADS, int ITEMS>
__device__ __forceinline__ void rank_keys(const uint32_t (&key)[ITEMS], int cnt, int shift, int radix, const SortMem& sm,
                                          int (&place)[ITEMS]) {
    constexpr int WARPS = THREADS / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = warp * (32 * ITEMS) + lane;
    for (int i = threadIdx.x; i < WARPS * radix / 8; i += THREADS)
        reinterpret_cast<uint4*>(sm.wc)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    unsigned short* mine = sm.wc + warp * radix;
    const unsigned lt = (1u << lane) - 1u;
    // lanes with the same digit, bit by bit, all keys side by side; the counts below depend on one another
    unsigned peers[ITEMS];
#pragma unroll
    for (int e = 0; e < ITEMS; ++e) peers[e] = __ballot_sync(0xffffffffu, first + e * 32 < cnt);
    for (int b = 0; 1 << b < radix; ++b) {
#pragma unroll
        for (int e = 0; e < ITEMS; ++e) {
            const unsigned bit = (key[e] >> (shift + b)) & 1u;
            const unsigned set = __ballot_sync(0xffffffffu, bit);
            peers[e] &= set ^ (bit - 1u);        // the lanes with this lane's bit
        }
    }
#pragma unroll
    for (int e = 0; e < ITEMS; ++e) {
        const bool valid = first + e * 32 < cnt;
        const int dg = (int)((key[e] >> shift) & (radix - 1));
        const int ahead = __popc(peers[e] & lt);
        const int seen = valid ? mine[dg] : 0;
        place[e] = seen + ahead;
        __syncwarp();
        if (valid && ahead == 0) mine[dg] = (unsigned short)(seen + __popc(peers[e]));
        __syncwarp();
    }
    __syncthreads();
    // two neighbouring digits a thread (one word of counts per warp), all warps' words loaded before any is written
    for (int d2 = threadIdx.x; d2 < radix / 2; d2 += THREADS) {
        uint32_t* col = reinterpret_cast<uint32_t*>(sm.wc) + d2;
        uint32_t c[WARPS], run = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) c[w] = col[w * (radix / 2)];
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            col[w * (radix / 2)] = run;
            run += c[w];          // both halves at once: a tile's counts stay below 2^16
        }
        sm.tot[2 * d2] = (int)(run & 0xffffu);
        sm.tot[2 * d2 + 1] = (int)(run >> 16);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < ITEMS; ++e)
        if (first + e * 32 < cnt) place[e] += mine[(key[e] >> shift) & (radix - 1)];
}

// x[0..radix) becomes its exclusive prefix sums, by the whole block (radix <= 4 blockDim).
__device__ __forceinline__ void scan_digits(int* x, int radix, int* wsum) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (radix + blockDim.x - 1) / blockDim.x;
    int v[4], s = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = threadIdx.x * per + e;
        v[e] = e < per && i < radix ? x[i] : 0;
        s += v[e];
    }
    int incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int run = incl - s;
    for (int q = 0; q < warp; ++q) run += wsum[q];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = threadIdx.x * per + e;
        if (e < per && i < radix) x[i] = run;
        run += v[e];
    }
    __syncthreads();
}

// The whole sort in one block, the pairs going round through shared memory. Indices outside the table get id m
// and end up last.
__global__ void __launch_bounds__(RS_THREADS) sort_one_block_kernel(int n, long long m, int passes, int bits,
                                                                    const int32_t* __restrict__ idx,
                                                                    uint32_t* __restrict__ keys,
                                                                    uint32_t* __restrict__ vals, ErrRecord* err,
                                                                    const __grid_constant__ Zeros zeros) {
    pdl_wait();
    extern __shared__ __align__(16) unsigned char sort_smem[];
    if (blockIdx.x > 0) {
        write_zeros(zeros);
        return;
    }
    const int radix = 1 << bits;
    const SortMem sm = sort_mem(sort_smem, radix);
    const int first = (threadIdx.x >> 5) * (32 * RS_ITEMS) + (threadIdx.x & 31);
    uint32_t key[RS_ITEMS], val[RS_ITEMS];
    unsigned bad = 0;
#pragma unroll
    for (int e = 0; e < RS_ITEMS; ++e) {
        const int i = first + e * 32;
        key[e] = val[e] = 0;
        if (i < n) {
            key[e] = pass_key<true>(idx, i, m);
            val[e] = (uint32_t)i;
            bad += key[e] == (uint32_t)m;
        }
    }
    report_warp(err, bad, 0);
    for (int p = 0; p < passes; ++p) {
        int place[RS_ITEMS];
        rank_keys<RS_THREADS, RS_ITEMS>(key, n, p * bits, radix, sm, place);
        scan_digits(sm.tot, radix, sm.wsum);
#pragma unroll
        for (int e = 0; e < RS_ITEMS; ++e)
            if (first + e * 32 < n) {
                const int at = sm.tot[(key[e] >> (p * bits)) & (radix - 1)] + place[e];
                sm.keys[at] = key[e];
                sm.vals[at] = val[e];
            }
        __syncthreads();
        if (p + 1 < passes) {
#pragma unroll
            for (int e = 0; e < RS_ITEMS; ++e)
                if (first + e * 32 < n) {
                    key[e] = sm.keys[first + e * 32];
                    val[e] = sm.vals[first + e * 32];
                }
        }
    }
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        keys[i] = sm.keys[i];
        vals[i] = sm.vals[i];
    }
}

// The whole sort in one cluster of sixteen blocks, which keep THREADS * ITEMS pairs each in shared memory, read one
// another's digit counts there and write each pair to its next place in the block that it falls to. Two cluster
// barriers a pass stand in for two launches. The other clusters of the launch write zeros.
constexpr int SORTC_CTAS = 16;
template <int THREADS, int ITEMS>
__global__ void __cluster_dims__(SORTC_CTAS, 1, 1) __launch_bounds__(THREADS)
    sort_cluster_kernel(int n, long long m, int passes, int bits, const int32_t* __restrict__ idx,
                        uint32_t* __restrict__ keys, uint32_t* __restrict__ vals, ErrRecord* err,
                        const __grid_constant__ Zeros zeros) {
    pdl_wait();
    extern __shared__ __align__(16) unsigned char sort_smem[];
    __shared__ int next[1 << DIG_BITS_MAX], earlier[1 << DIG_BITS_MAX];
    if (blockIdx.x >= SORTC_CTAS) {
        write_zeros(zeros);
        return;
    }
    constexpr int TILE = THREADS * ITEMS;
    const int radix = 1 << bits;
    const SortMem sm = sort_mem<THREADS / 32>(sort_smem, radix);
    uint2* pairs = reinterpret_cast<uint2*>(sm.keys);
    const int rank = (int)tc::cluster_rank(), t0 = rank * TILE;
    const int cnt = n - t0 < 0 ? 0 : n - t0 < TILE ? n - t0 : TILE;
    const int first = (threadIdx.x >> 5) * (32 * ITEMS) + (threadIdx.x & 31);
    const uint32_t tot_s = tc::su32(sm.tot), pairs_s = tc::su32(pairs);
    for (int p = 0; p < passes; ++p) {
        uint32_t key[ITEMS], val[ITEMS];
        unsigned bad = 0;
#pragma unroll
        for (int e = 0; e < ITEMS; ++e) {
            const int i = first + e * 32;
            key[e] = val[e] = 0;
            if (i < cnt) {
                if (p == 0) {
                    key[e] = pass_key<true>(idx, t0 + i, m);
                    val[e] = (uint32_t)(t0 + i);
                    bad += key[e] == (uint32_t)m;
                } else {
                    const uint2 kv = pairs[i];
                    key[e] = kv.x;
                    val[e] = kv.y;
                }
            }
        }
        if (p == 0) report_warp(err, bad, 0);
        int place[ITEMS];
        rank_keys<THREADS, ITEMS>(key, cnt, p * bits, radix, sm, place);
        tc::cluster_sync_all();      // every block's counts are there, and its pairs in registers
        for (int dg = threadIdx.x; dg < radix; dg += THREADS) {
            int all = 0, before = 0;
#pragma unroll
            for (int q = 0; q < SORTC_CTAS; ++q) {
                int v;
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(tc::map_rank(tot_s + 4 * dg, q)) : "memory");
                all += v;
                before += q < rank ? v : 0;
            }
            next[dg] = all;
            earlier[dg] = before;
        }
        __syncthreads();
        scan_digits(next, radix, sm.wsum);
#pragma unroll
        for (int e = 0; e < ITEMS; ++e)
            if (first + e * 32 < cnt) {
                const int dg = (int)((key[e] >> (p * bits)) & (radix - 1));
                const int at = next[dg] + earlier[dg] + place[e];       // < n: block at / TILE holds it
                asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(
                                 tc::map_rank(pairs_s + 8 * (at % TILE), at / TILE)),
                             "r"(key[e]), "r"(val[e])
                             : "memory");
            }
        tc::cluster_sync_all();      // counts read, pairs written
    }
    for (int i = threadIdx.x; i < cnt; i += THREADS) {
        const uint2 kv = pairs[i];
        keys[t0 + i] = kv.x;
        vals[t0 + i] = kv.y;
    }
}

// hist[b][digit] = keys of block b with that digit
template <bool FIRST>
__global__ void __launch_bounds__(RS_THREADS) rs_hist_kernel(long long n, long long m, const void* __restrict__ in,
                                                             int shift, int bits, long long chunk,
                                                             int* __restrict__ hist, ErrRecord* err,
                                                             const __grid_constant__ Zeros zeros) {
    pdl_wait();
    __shared__ int h[1 << DIG_BITS_MAX];
    if ((int)blockIdx.x >= zeros.sorters) {
        write_zeros(zeros);
        return;
    }
    const int radix = 1 << bits;
    for (int i = threadIdx.x; i < radix; i += blockDim.x) h[i] = 0;
    __syncthreads();
    const long long b0 = (long long)blockIdx.x * chunk, b1 = b0 + chunk < n ? b0 + chunk : n;
    unsigned bad = 0;
    for (long long i0 = b0 + threadIdx.x; i0 < b1; i0 += RS_TILE) {
        uint32_t key[RS_ITEMS];
#pragma unroll
        for (int e = 0; e < RS_ITEMS; ++e)
            if (i0 + e * RS_THREADS < b1) key[e] = pass_key<FIRST>(in, i0 + e * RS_THREADS, m);
#pragma unroll
        for (int e = 0; e < RS_ITEMS; ++e)
            if (i0 + e * RS_THREADS < b1) {
                if (FIRST) bad += key[e] == (uint32_t)m;
                atomicAdd(&h[(key[e] >> shift) & (radix - 1)], 1);
            }
    }
    if (FIRST) {
        __syncwarp();
        report_warp(err, bad, 0);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < radix; i += blockDim.x) hist[(long long)blockIdx.x * radix + i] = h[i];
}

// Stable scatter of block b's keys. Its first position for a digit is the count of smaller digits in all
// blocks plus that of the same digit in earlier blocks, summed here from the histograms (at most 296 of them).
template <bool FIRST>
__global__ void __launch_bounds__(RS_THREADS) rs_scatter_kernel(long long n, long long m, const void* __restrict__ in,
                                                                const uint32_t* __restrict__ vin, int shift, int bits,
                                                                long long chunk, const int* __restrict__ hist,
                                                                uint32_t* __restrict__ kout,
                                                                uint32_t* __restrict__ vout,
                                                                const __grid_constant__ Zeros zeros) {
    pdl_wait();
    extern __shared__ __align__(16) unsigned char sort_smem[];
    __shared__ int next[1 << DIG_BITS_MAX];      // the block's next output position per digit
    if ((int)blockIdx.x >= zeros.sorters) {
        write_zeros(zeros);
        return;
    }
    const int radix = 1 << bits;
    const SortMem sm = sort_mem(sort_smem, radix);
    const long long b0 = (long long)blockIdx.x * chunk, b1 = b0 + chunk < n ? b0 + chunk : n;
    const int first = (threadIdx.x >> 5) * (32 * RS_ITEMS) + (threadIdx.x & 31);
    uint32_t key[RS_ITEMS], val[RS_ITEMS];
    auto load_tile = [&](long long t0) {
#pragma unroll
        for (int e = 0; e < RS_ITEMS; ++e) {
            const long long i = t0 + first + e * 32;
            const bool valid = i < b1;
            key[e] = valid ? pass_key<FIRST>(in, i, m) : 0u;
            val[e] = valid ? (FIRST ? (uint32_t)i : vin[i]) : 0u;
        }
    };
    load_tile(b0);      // on its way while the positions are worked out
    {
        // totals and prefixes over blocks: each thread takes four neighbouring digits, and the threads left over
        // share the blocks' rows between them
        int* tot = reinterpret_cast<int*>(sm.keys);          // [groups][radix]: 4 * RS_THREADS sums
        int* bef = tot + 4 * RS_THREADS;
        const int per_group = radix / 4, groups = RS_THREADS / per_group;
        const int g = threadIdx.x / per_group, d4 = threadIdx.x - g * per_group;
        const int nb = zeros.sorters, mine = (nb + groups - 1) / groups;
        const int q0 = g * mine, q1 = q0 + mine < nb ? q0 + mine : nb;
        int4 all = make_int4(0, 0, 0, 0), before = all;
        const int4* row = reinterpret_cast<const int4*>(hist) + d4;
#pragma unroll 8
        for (int q = q0; q < q1; ++q) {
            const int4 v = __ldg(row + (long long)q * per_group);
            all.x += v.x, all.y += v.y, all.z += v.z, all.w += v.w;
            if (q < (int)blockIdx.x) before.x += v.x, before.y += v.y, before.z += v.z, before.w += v.w;
        }
        reinterpret_cast<int4*>(tot)[threadIdx.x] = all;
        reinterpret_cast<int4*>(bef)[threadIdx.x] = before;
        __syncthreads();
        for (int dg = threadIdx.x; dg < radix; dg += RS_THREADS) {
            int x = 0, y = 0;
            for (int q = 0; q < groups; ++q) {
                x += tot[q * radix + dg];
                y += bef[q * radix + dg];
            }
            next[dg] = x;
            bef[dg] = y;        // only this thread reads or writes column dg
        }
        __syncthreads();
        scan_digits(next, radix, sm.wsum);
        for (int dg = threadIdx.x; dg < radix; dg += RS_THREADS) next[dg] += bef[dg];
        __syncthreads();
    }
    for (long long t0 = b0; t0 < b1; t0 += RS_TILE) {
        if (t0 > b0) load_tile(t0);
        const int cnt = (int)(b1 - t0 < RS_TILE ? b1 - t0 : RS_TILE);
        int place[RS_ITEMS];
        rank_keys<RS_THREADS, RS_ITEMS>(key, cnt, shift, radix, sm, place);
        scan_digits(sm.tot, radix, sm.wsum);
        // in order of digit through shared memory, so that neighbouring threads write neighbouring pairs
#pragma unroll
        for (int e = 0; e < RS_ITEMS; ++e)
            if (first + e * 32 < cnt) {
                const int at = sm.tot[(key[e] >> shift) & (radix - 1)] + place[e];
                sm.keys[at] = key[e];
                sm.vals[at] = val[e];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < cnt; i += RS_THREADS) {
            const uint32_t k = sm.keys[i];
            const int dg = (int)((k >> shift) & (radix - 1));
            const long long at = (long long)next[dg] + (i - sm.tot[dg]);
            kout[at] = k;
            vout[at] = sm.vals[i];
        }
        __syncthreads();
        for (int dg = threadIdx.x; dg < radix; dg += RS_THREADS)
            next[dg] += (dg + 1 < radix ? sm.tot[dg + 1] : cnt) - sm.tot[dg];
        __syncthreads();
    }
}

// ------------------------------------------------------------------ sums over runs of equal ids

struct SumArgs {
    long long n, m;
    int d;
    long long windows;
    int P;                    // sorted pairs per window
    int slices;               // column slices
    const uint32_t* keys;
    const uint32_t* vals;
    const void* dout;
    long long ldd;
    float scale;
    float* partial;           // [windows][2][d]: the run entering from before, the run leaving into the next
    void* dT;
};

// How many windows after w begin with `key`, by the whole warp: the 32 next ones at a glance, further ones by their
// number, 32 probes at a time (the keys are sorted, so these windows follow one another).
__device__ __forceinline__ long long warp_windows_of(const SumArgs& a, long long w, uint32_t key, int lane) {
    const long long at = w + 1 + lane;
    const unsigned same = __ballot_sync(0xffffffffu, at < a.windows && a.keys[at * a.P] == key);
    if (same != 0xffffffffu) return __popc(same);
    long long lo = w + 33, hi = a.windows;      // the first window that begins with another key is in [lo, hi]
    while (hi - lo > 0) {
        const long long step = (hi - lo + 31) / 32;
        const long long last = lo + step * (lane + 1) - 1;              // last window of the lane's piece
        const bool in = last < hi && a.keys[last * a.P] == key;
        const int pieces = __popc(__ballot_sync(0xffffffffu, in));      // pieces wholly of this key
        lo += step * pieces;
        if (lo > hi) lo = hi;
        if (step == 1) break;
        hi = lo + step - 1 < hi ? lo + step - 1 : hi;
    }
    return lo - w - 1;
}

// blockDim = (TX, 128 / TX): TX threads along the column slice, one window per threadIdx.y. A thread has NV runs of
// VEC columns, TX runs apart: 16 bytes of the narrower type in all, so that what a pair costs besides its columns
// is spread over as many of them where the rows allow only short runs.
template <typename TI, typename TO, int VEC, int NV>
__global__ void __launch_bounds__(128) run_sum_kernel(const __grid_constant__ SumArgs a) {
    pdl_wait();
    TO* dT = static_cast<TO*>(a.dT);
    const long long wb = blockIdx.x / a.slices;
    const int slice = (int)(blockIdx.x - wb * a.slices);
    const long long w = wb * blockDim.y + threadIdx.y;
    const int c = (slice * NV * blockDim.x + threadIdx.x) * VEC, cstep = blockDim.x * VEC;
    if (w >= a.windows || c >= a.d) return;
    const long long i0 = w * a.P, i1 = i0 + a.P < a.n ? i0 + a.P : a.n;
    const TI* dout = static_cast<const TI*>(a.dout) + c;
    const uint32_t m = (uint32_t)a.m;
    constexpr int U = 8;
    // ids and positions one group ahead of the rows they name; id m: no pair
    uint32_t key[U], val[U], nkey[U], nval[U];
    auto fetch = [&](long long i, uint32_t(&k)[U], uint32_t(&v)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = i + u < i1;
            k[u] = in ? a.keys[i + u] : m;
            v[u] = in ? a.vals[i + u] : 0u;
        }
    };
    fetch(i0, key, val);
    // the first run of the window is a continuation when the pair before it has the same id; the last one goes on
    // when the pair after the window has
    const uint32_t before = i0 > 0 ? a.keys[i0 - 1] : m, beyond = i1 < a.n ? a.keys[i1] : m;
    bool entering = before == key[0];
    float acc[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[j][e] = 0.f;
    for (long long i = i0; i < i1; i += U) {
        RowRaw<TI, VEC> in[U][NV];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (key[u] != m) {
                const TI* p = dout + (long long)val[u] * a.ldd;
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (j == 0 || c + j * cstep < a.d) in[u][j].load(p + j * cstep);
            }
        fetch(i + U, nkey, nval);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (key[u] == m) break;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j == 0 || c + j * cstep < a.d) {
                    float v[VEC];
                    in[u][j].get(v);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) acc[j][e] += v[e];
                }
            const bool last_here = i + u + 1 == i1;          // the window's last pair
            const uint32_t after = last_here ? beyond : u + 1 < U ? key[u + 1 < U ? u + 1 : 0] : nkey[0];
            const bool ends = after != key[u];
            if (!ends && !last_here) continue;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j == 0 || c + j * cstep < a.d) {
                    if (entering || !ends) {
                        // part of a run that crosses windows
                        float* p = a.partial + (w * 2 + (entering ? 0 : 1)) * a.d + c + j * cstep;
#pragma unroll
                        for (int e = 0; e < VEC; ++e) p[e] = acc[j][e];
                    } else {
                        RowRaw<TO, VEC> o;
#pragma unroll
                        for (int e = 0; e < VEC; ++e) acc[j][e] *= a.scale;
                        o.set(acc[j]);
                        o.store(dT + (long long)key[u] * a.d + c + j * cstep);
                    }
#pragma unroll
                    for (int e = 0; e < VEC; ++e) acc[j][e] = 0.f;
                }
            entering = false;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            key[u] = nkey[u];
            val[u] = nval[u];
        }
    }
}

// Adds partial[w + j][0] for j in [j0, j1) to s, in order, 64 bytes of loads in flight at most (four of 16 bytes: 65,536
// ids of 512 67.0 us the call, 67.7 with eight, 72.3 with sixteen; eight of 4 bytes: 23,517 of 29 18.6, 19.2 with four).
template <int VEC>
__device__ __forceinline__ void add_parts(const SumArgs& a, long long w, long long j0, long long j1, int c, float (&s)[VEC]) {
    constexpr int U = VEC == 4 ? 4 : 8;
    for (long long j = j0; j < j1; j += U) {
        RowRaw<float, VEC> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u < j1) r[u].load(a.partial + (w + j + u) * 2 * a.d + c);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u < j1) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[e] += r[u].e[e];
            }
    }
}

// A run that starts inside window w and goes on into w + 1: its parts are partial[w][1], partial[w + 1][0],
// ... up to the window where it ends. blockDim = (32, 8): each warp looks at one window and adds up a run of few
// parts by itself, VEC columns a lane; the block's warps share each longer run in eight contiguous pieces, added
// in order. Which of the two depends on the run's length alone.
constexpr int JOIN_SHORT = 32;
template <typename TO, int VEC>
__global__ void __launch_bounds__(256) run_join_kernel(const __grid_constant__ SumArgs a) {
    pdl_wait();
    __shared__ float part[8][32][VEC + 1];
    __shared__ long long parts_of[8];            // parts after the first of each warp's run (0: none, or done)
    __shared__ uint32_t key_of[8];
    const long long w0 = (long long)blockIdx.x * 8, w = w0 + threadIdx.y;
    const int c = (blockIdx.y * 32 + threadIdx.x) * VEC;
    const long long i0 = w * a.P, i1 = i0 + a.P;
    long long cnt = 0;
    uint32_t key = 0;
    if (i1 < a.n) {
        key = a.keys[i1 - 1];
        const uint32_t next = a.keys[i1], first = a.keys[i0], prev = i0 > 0 ? a.keys[i0 - 1] : ~key;
        // it leaves this window, and did not start before it
        if (key == next && key != (uint32_t)a.m && !(first == key && prev == key))
            cnt = warp_windows_of(a, w, key, threadIdx.x);
    }
    float s[VEC];
    auto first_part = [&](long long win) {
        RowRaw<float, VEC> r;
        r.load(a.partial + (win * 2 + 1) * a.d + c);
        r.get(s);
    };
    auto write = [&](uint32_t k) {
        TO* p = static_cast<TO*>(a.dT) + (long long)k * a.d + c;
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = Cvt<TO>::from_f(s[e] * a.scale);
    };
    if (cnt > 0 && cnt <= JOIN_SHORT) {
        if (c < a.d) {
            first_part(w);
            add_parts<VEC>(a, w, 1, cnt + 1, c, s);
            write(key);
        }
        cnt = 0;
    }
    if (threadIdx.x == 0) {
        parts_of[threadIdx.y] = cnt;
        key_of[threadIdx.y] = key;
    }
    __syncthreads();
    for (int q = 0; q < 8; ++q) {
        const long long n = parts_of[q];
        if (n == 0) continue;                    // the same for the whole block
        const long long per = (n + 7) / 8;
        const long long j0 = 1 + threadIdx.y * per, j1 = j0 + per < n + 1 ? j0 + per : n + 1;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[e] = 0.f;
        if (c < a.d) {
            if (threadIdx.y == 0) first_part(w0 + q);
            add_parts<VEC>(a, w0 + q, j0, j1, c, s);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) part[threadIdx.y][threadIdx.x][e] = s[e];
        __syncthreads();
        if (threadIdx.y == 0 && c < a.d) {
#pragma unroll
            for (int g = 1; g < 8; ++g)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[e] += part[g][threadIdx.x][e];
            write(key_of[q]);
        }
        __syncthreads();
    }
}

// Pairs per window: short windows while long ones would leave SMs without work. us a call with 16 and with 64, at n * d of
// 2^22 22.5 and 28.3; 2^23 31 and 34 to 35; 2^24 41 and 39, 38 and 40, 49 and 45 (1,024, 256, 64 columns); 2^25 53 and 47,
// 74 and 67.
int window_len(long long n, int d) { return n * (long long)d >= (1ll << 24) ? 64 : 16; }

template <typename TI, typename TO, int VEC, int NV>
dlrm_status sum_launch(SumArgs a, cudaStream_t st) {
    const int runs = a.d / VEC;
    const int tx = pow2_at_least((runs + NV - 1) / NV, 128);
    const dim3 block(tx, 128 / tx);
    a.slices = (runs + NV * tx - 1) / (NV * tx);
    const long long blocks = (a.windows + block.y - 1) / block.y * a.slices;      // lookup_grad_fits: below 2^31
    if (blocks == 0) return DLRM_OK;
    // few blocks: a run a thread (288 ids of 19 fp16: 10.6 us the call, 16.9 with eight runs)
    if constexpr (NV > 1)
        if (blocks < 2ll * device_sms()) return sum_launch<TI, TO, VEC, 1>(a, st);
    DLRM_PDL_CHECK(launch_pdl(run_sum_kernel<TI, TO, VEC, NV>, dim3((unsigned)blocks), block, 0, st, a));
    if (a.windows > 1) {
        const unsigned nw = (unsigned)((a.windows - 1 + 7) / 8);
        if (a.d % 4 == 0)
            DLRM_PDL_CHECK(launch_pdl(run_join_kernel<TO, 4>, dim3(nw, (a.d + 127) / 128), dim3(32, 8), 0, st, a));
        else
            DLRM_PDL_CHECK(launch_pdl(run_join_kernel<TO, 1>, dim3(nw, (a.d + 31) / 32), dim3(32, 8), 0, st, a));
    }
    return DLRM_OK;
}

template <typename TI, typename TO, int VEC>
dlrm_status sum_vec(const SumArgs& a, cudaStream_t st) {
    constexpr int W = 16 / (int)(sizeof(TI) < sizeof(TO) ? sizeof(TI) : sizeof(TO));
    return sum_launch<TI, TO, VEC, W / VEC>(a, st);
}

template <typename TI, typename TO>
dlrm_status sum_to(const SumArgs& a, cudaStream_t st) {
    constexpr int W = 16 / (int)(sizeof(TI) < sizeof(TO) ? sizeof(TI) : sizeof(TO));
    auto fits = [&](int vec) {
        const int bi = std::min(16, vec * (int)sizeof(TI)), bo = std::min(16, vec * (int)sizeof(TO));
        return a.d % vec == 0 && rows_on(a.dout, a.ldd * (long long)sizeof(TI), bi) &&
               rows_on(a.dT, (long long)a.d * sizeof(TO), bo);
    };
    if (fits(W)) return sum_vec<TI, TO, W>(a, st);
    if constexpr (W > 4)
        if (fits(4)) return sum_vec<TI, TO, 4>(a, st);
    if (fits(2)) return sum_vec<TI, TO, 2>(a, st);
    return sum_vec<TI, TO, 1>(a, st);
}

template <typename TI>
dlrm_status sum_ti(const SumArgs& a, dlrm_dtype dt, cudaStream_t st) {
    if (dt == DLRM_F32) return sum_to<TI, float>(a, st);
    if (dt == DLRM_F16) return sum_to<TI, __half>(a, st);
    return sum_to<TI, __nv_bfloat16>(a, st);
}

static_assert(sort_bytes(1 << DIG_BITS_MAX) + 2 * 4 * (1 << DIG_BITS_MAX) <= 48 * 1024, "sorting blocks");

static_assert(SORTC_MAX == SORTC_CTAS * 512 * 8, "the cluster's largest variant");
std::atomic<bool> g_clusters{true};     // dlrm_set_sort_clusters

// Whether the current device can place a cluster of this variant: sixteen blocks are more than every device, partition or
// context has room for, the largest variant's taking an SM each. Asked once per device; the answer does not change.
template <int THREADS, int ITEMS>
bool cluster_fits() {
    static std::atomic<signed char> known[64];
    auto kern = sort_cluster_kernel<THREADS, ITEMS>;
    const int most = (int)sort_bytes(1 << DIG_BITS_MAX, THREADS, ITEMS);
    int dev = 0;
    // sixteen blocks a cluster, and shared memory past 48 KB, are asked for; always the same values
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    const bool slot = dev >= 0 && dev < 64;
    if (slot && known[dev].load(std::memory_order_relaxed)) return known[dev].load(std::memory_order_relaxed) > 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(SORTC_CTAS);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = most;
    int n = 0;
    const bool fits = cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0;
    if (!fits) (void)cudaGetLastError();
    if (slot) known[dev].store(fits ? 1 : -1, std::memory_order_relaxed);
    return fits;
}

// The fewest pairs a thread that hold them all: ranking takes longer the more there are.
#define DLRM_SORT_CLUSTER(n, CALL)                                        \
    ((n) <= SORTC_CTAS * 256 * 2   ? CALL(256, 2)                          \
     : (n) <= SORTC_CTAS * 256 * 4 ? CALL(256, 4)                          \
     : (n) <= SORTC_CTAS * 256 * 8 ? CALL(256, 8)                          \
                                   : CALL(512, 8))

template <int THREADS, int ITEMS>
dlrm_status sort_cluster(dim3 grid, int n, long long m, int passes, int bits, const int32_t* idx, uint32_t* keys,
                         uint32_t* vals, ErrRecord* err, const Zeros& z, cudaStream_t st) {
    DLRM_PDL_CHECK(launch_pdl(sort_cluster_kernel<THREADS, ITEMS>, grid, dim3(THREADS), sort_bytes(1 << bits, THREADS, ITEMS),
                              st, n, m, passes, bits, idx, keys, vals, err, z));
    return DLRM_OK;
}

struct GradLayout {
    bool one, cluster;      // the one-block sort; the cluster's where the device can place it
    int nblocks, passes, bits;
    long long chunk;
    size_t keys[2], vals[2], hist, partial, total;
};

GradLayout grad_layout(long long m, int d, long long n) {
    GradLayout L;
    int kb = 1;
    while ((1ll << kb) <= m) ++kb;             // ids 0 .. m
    L.one = n <= SORT1_MAX;
    L.cluster = !L.one && n <= SORTC_MAX;
    L.passes = (kb + DIG_BITS_MAX - 1) / DIG_BITS_MAX;
    L.bits = std::max(5, (kb + L.passes - 1) / L.passes);
    const long long tiles = (n + RS_TILE - 1) / RS_TILE;
    const long long per = (tiles + RS_BLOCKS_MAX - 1) / RS_BLOCKS_MAX;
    L.chunk = std::max(1ll, per) * RS_TILE;
    L.nblocks = (int)std::max(1ll, (n + L.chunk - 1) / L.chunk);
    size_t off = align_up(DLRM_ERR_RECORD_BYTES, 256);
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = align_up(off + bytes, 256);
        return o;
    };
    // the cluster's sizes have the space of the many-block sort, so that the size does not depend on the device
    const int pairs = L.one ? 1 : 2;
    for (int i = 0; i < 2; ++i) L.keys[i] = i < pairs ? take(sizeof(uint32_t) * (size_t)n) : 0;
    for (int i = 0; i < 2; ++i) L.vals[i] = i < pairs ? take(sizeof(uint32_t) * (size_t)n) : 0;
    L.hist = take(!L.one ? sizeof(int) * ((size_t)L.nblocks << L.bits) : 0);
    const long long windows = (n + window_len(n, d) - 1) / window_len(n, d);
    L.partial = take(sizeof(float) * 2 * (size_t)windows * d);
    L.total = off;
    return L;
}

}  // namespace

dlrm_status launch_lookup(const void* table, dlrm_dtype dt, long long rows, int d, long long n, const int32_t* idx,
                          float scale, void* out, long long ldo, dlrm_dtype out_dt, ErrRecord* err, cudaStream_t st) {
    const LookupArgs a{n, d, rows, table, idx, scale, out, ldo, err};
    if (dt == DLRM_F32) return lookup_ti<float>(a, out_dt, st);
    if (dt == DLRM_F16) return lookup_ti<__half>(a, out_dt, st);
    return lookup_ti<__nv_bfloat16>(a, out_dt, st);
}

void set_sort_clusters(bool allowed) { g_clusters.store(allowed, std::memory_order_relaxed); }

// A block sums at least one window of at least 512 columns, or all of them.
bool lookup_grad_fits(int d, long long n) {
    const long long p = window_len(n, d);
    return (n + p - 1) / p * ((d + 511) / 512) < 1ll << 31;
}

size_t lookup_grad_workspace(long long m, int d, long long n) { return grad_layout(m, d, n).total; }

dlrm_status launch_lookup_grad(long long m, int d, long long n, const int32_t* idx, float scale, const void* dout,
                               long long ldd, dlrm_dtype dt, void* dT, dlrm_dtype dT_dt, char* ws, cudaStream_t st) {
    GradLayout L = grad_layout(m, d, n);
#define DLRM_FITS(T, I) cluster_fits<T, I>()
    L.cluster = L.cluster && g_clusters.load(std::memory_order_relaxed) && DLRM_SORT_CLUSTER(n, DLRM_FITS);
#undef DLRM_FITS
    ErrRecord* err = reinterpret_cast<ErrRecord*>(ws);
    uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(ws + L.keys[0]), reinterpret_cast<uint32_t*>(ws + L.keys[1])};
    uint32_t* vals[2] = {reinterpret_cast<uint32_t*>(ws + L.vals[0]), reinterpret_cast<uint32_t*>(ws + L.vals[1])};
    int* hist = reinterpret_cast<int*>(ws + L.hist);
    const long long bytes = m * d * (long long)(dT_dt == DLRM_F32 ? 4 : 2);
    // launches of the sort: a histogram takes about a third of a scatter's time, and writes so much of the zeros
    const int shares = L.one || L.cluster ? 1 : 4 * L.passes;
    long long done = 0;
    auto zeros = [&](int sorters, int share) {
        Zeros z{static_cast<char*>(dT), bytes * done / shares, bytes * (done + share) / shares, sorters};
        done += share;
        return z;
    };
    // blocks that write a share's zeros: 16 KB each at least, `most` per SM at most. Eight of the small sorts' blocks, two
    // where the sort is as long as the zeros, which then hold it up. us a call with eight and with two, into 100,000 x 512
    // fp32: 2,500 ids 41 and 46, 8,192 46 and 51, 32,768 56 and 60; 32,769 65 and 62, 50,000 67 and 65, 65,536 70 and 67.
    auto writers = [&](const Zeros& z, int most) {
        return (unsigned)std::max<long long>(1, std::min<long long>((z.end - z.begin + 16383) / 16384, (long long)most * device_sms()));
    };
    // with the static arrays under 48 KB: 8 warps, up to 1,024 digits, the pairs of a tile
    const size_t smem = sort_bytes(1 << L.bits);
    int cur = 0;
    if (L.one) {
        const Zeros z = zeros(1, 1);
        DLRM_PDL_CHECK(launch_pdl(sort_one_block_kernel, dim3(1 + writers(z, 8)), dim3(RS_THREADS), smem, st, (int)n, m,
                                  L.passes, L.bits, idx, keys[0], vals[0], err, z));
    } else if (L.cluster) {
        const Zeros z = zeros(SORTC_CTAS, 1);
        const unsigned nw = writers(z, n <= SORTC_CTAS * 256 * 8 ? 8 : 2);
        const dim3 grid(SORTC_CTAS + (nw + SORTC_CTAS - 1) / SORTC_CTAS * SORTC_CTAS);
#define DLRM_SORT(T, I) sort_cluster<T, I>(grid, (int)n, m, L.passes, L.bits, idx, keys[0], vals[0], err, z, st)
        const dlrm_status r = DLRM_SORT_CLUSTER(n, DLRM_SORT);
#undef DLRM_SORT
        if (r != DLRM_OK) return r;
    } else {
        const dim3 block(RS_THREADS);
        for (int p = 0; p < L.passes; ++p) {
            const int shift = p * L.bits;
            const Zeros zh = zeros(L.nblocks, 1), zs = zeros(L.nblocks, 3);
            const dim3 gh(L.nblocks + writers(zh, 2)), gs(L.nblocks + writers(zs, 2));
            if (p == 0) {
                DLRM_PDL_CHECK(launch_pdl(rs_hist_kernel<true>, gh, block, 0, st, n, m, (const void*)idx, shift,
                                          L.bits, L.chunk, hist, err, zh));
                DLRM_PDL_CHECK(launch_pdl(rs_scatter_kernel<true>, gs, block, smem, st, n, m, (const void*)idx,
                                          (const uint32_t*)nullptr, shift, L.bits, L.chunk, (const int*)hist,
                                          keys[0], vals[0], zs));
            } else {
                DLRM_PDL_CHECK(launch_pdl(rs_hist_kernel<false>, gh, block, 0, st, n, m, (const void*)keys[cur], shift,
                                          L.bits, L.chunk, hist, err, zh));
                DLRM_PDL_CHECK(launch_pdl(rs_scatter_kernel<false>, gs, block, smem, st, n, m, (const void*)keys[cur],
                                          (const uint32_t*)vals[cur], shift, L.bits, L.chunk, (const int*)hist,
                                          keys[cur ^ 1], vals[cur ^ 1], zs));
                cur ^= 1;
            }
        }
    }
    SumArgs a;
    a.n = n;
    a.m = m;
    a.d = d;
    a.P = window_len(n, d);
    a.windows = (n + a.P - 1) / a.P;
    a.slices = 0;
    a.keys = keys[cur];
    a.vals = vals[cur];
    a.dout = dout;
    a.ldd = ldd;
    a.scale = scale;
    a.partial = reinterpret_cast<float*>(ws + L.partial);
    a.dT = dT;
    if (dt == DLRM_F32) return sum_ti<float>(a, dT_dt, st);
    if (dt == DLRM_F16) return sum_ti<__half>(a, dT_dt, st);
    return sum_ti<__nv_bfloat16>(a, dT_dt, st);
}

}  // namespace dlrm

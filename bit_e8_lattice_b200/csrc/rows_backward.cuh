// Backward of the row lookup (identity straight-through estimator, "E8-QAT",
// Figure 2 (b)): every latent row gets the sum of the output gradients of
// the tokens that read it,
//   G[r] (+)= alpha * sum_{t : id_t - first_row = r} g[t],
// in fp32, in token order, rounded once.  No sum is formed with an atomic (one
// counter tells which CTA adds the parts of a long run, always in the same
// order), so the result does not depend on timing.
//
// Tokens are first sorted by row, ties by position:
//   n <= kRbRankMax   k_rb_rank: the place of a token is the number of tokens
//                     before it in (row, position) order, counted against all
//                     n ids held in shared memory; n^2 comparisons over all
//                     SMs cost less than the launches of a radix sort;
//   above             k_rb_sort: a stable radix sort by one cluster of CTAs.
// Then
//   k_rb_sum          one CTA per (chunk of sorted tokens, 1,024 columns): a
//                     thread owns 8 columns and keeps a batch of rows in
//                     flight.  The run of a row is summed by the chunk that it
//                     begins in, past the border if need be, and written at
//                     once; only a run longer than a chunk is cut at the
//                     borders and leaves fp32 partial sums (at most two a
//                     chunk), which the last CTA to write one of the run adds
//                     in order (a padding id may fill thousands of chunks).
//                     Further CTAs of the same launch write the zeros of the
//                     rows without a token, so that every output byte is
//                     written once.
// Short batches (n <= kRbDirectMax) need no sort: k_rb_direct has one CTA per
// (token, 1,024 columns), and the first token of a row sums the others'.
//
// Measured: 16,384 bf16 gradients (natural-language-like ids) into a 32000 x
// 4096 bf16 table: 92 us, of which the sort about 18 and the sums 68 to 72 (396
// MB read and written once: 5.5 TB/s, 84 % of the measured copy bandwidth), 68 us
// accumulated (5,408 rows touched); 5,003 fp32 gradients of 768 columns into
// 25,011 rows: 29.5 us (rank 11, sums 19), 24 us accumulated.
// The sums are bound by HBM; the sort by its barriers (8 SMs).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace e8q {

constexpr int kRbThreads = 128;
constexpr int kRbSliceCols = kRbThreads * 8;
// 128 ids into 1000 x 2048: 2.4 us without a sort, 7.5 us with (on one row: 9.5 and 9.0)
constexpr int kRbDirectMax = 128;
// into 32000 x 1024, 4,096 ids: 12 us ranked, 22 us by the cluster's sort; 8,192: 21 and 24
constexpr int kRbRankMax = 8192;
constexpr int kRbGroup = 32;  // parts of a long run that are added together
constexpr int kRbRankKeys = 32;  // keys a rank CTA places
constexpr int kRbRankThreads = 512;
constexpr int kRbZeroRows = 32;
constexpr int kRbMaxChunk = 128;
constexpr int kRbCluster = 8;
constexpr int kRbSortThreads = 1024;
constexpr int kRbDigitBits = 9;
constexpr int kRbBins = 1 << kRbDigitBits;
constexpr size_t kRbSortSmem = (1 + kRbSortThreads / 32) * kRbBins * 4;

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// barrier of all threads of the cluster; earlier writes are visible after it
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// *p of CTA r of the cluster (p: the place in this CTA's shared memory)
__device__ __forceinline__ uint32_t cluster_load(const uint32_t* p, unsigned r) {
    uint32_t at, v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(r));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

struct RbIds {
    const void* ids;
    long long first_row;
    int32_t id64;
    int32_t rows;
};

// Row of token i, or `rows` for an id outside the table (it sorts last).
__device__ __forceinline__ int rb_key(const RbIds& p, long long i) {
    const long long id = p.id64 ? __ldg(static_cast<const long long*>(p.ids) + i)
                                : static_cast<long long>(__ldg(static_cast<const int*>(p.ids) + i));
    // unsigned, since the distance of two 64-bit ids may not fit a signed one
    const unsigned long long d = static_cast<unsigned long long>(id) - static_cast<unsigned long long>(p.first_row);
    return (id >= p.first_row && d < static_cast<unsigned long long>(p.rows)) ? static_cast<int>(d) : p.rows;
}

// Rows of tokens i, i + step, ..; past the end: `pad`.  All loads go out before the first is used.
template <int N>
__device__ __forceinline__ void rb_keys(const RbIds& p, long long i, int step, long long end, int pad, int (&key)[N]) {
    long long id[N];
    if (p.id64) {
#pragma unroll
        for (int k = 0; k < N; ++k) id[k] = i + k * step < end ? __ldg(static_cast<const long long*>(p.ids) + i + k * step) : 0;
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) id[k] = i + k * step < end ? __ldg(static_cast<const int*>(p.ids) + i + k * step) : 0;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const unsigned long long d = static_cast<unsigned long long>(id[k]) - static_cast<unsigned long long>(p.first_row);
        key[k] = i + k * step >= end ? pad
                 : (id[k] >= p.first_row && d < static_cast<unsigned long long>(p.rows)) ? static_cast<int>(d) : p.rows;
    }
}

// ------------------------------------------------------------------ sorting
struct RbRankParams {
    RbIds ids;
    int32_t n;
    int32_t* keys;   // out: sorted rows
    int32_t* order;  // out: their tokens
    int32_t* done;   // out: zeros (RbSumParams)
    int32_t dones;
};

// Lane = key, the warps share the comparisons; keys before and behind the
// CTA's own need one comparison each, since ties go by position.
__global__ void __launch_bounds__(kRbRankThreads) k_rb_rank(const __grid_constant__ RbRankParams p) {
    constexpr int W = kRbRankThreads / 32;
    __shared__ __align__(16) int s_key[kRbRankMax];
    __shared__ int s_part[W][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    const int npad = (p.n + 4 * W - 1) / (4 * W) * (4 * W);
    for (int i = blockIdx.x * kRbRankThreads + tid; i < p.dones; i += gridDim.x * kRbRankThreads) p.done[i] = 0;
    for (int i = tid; i < npad; i += 8 * kRbRankThreads) {
        int k[8];
        rb_keys(p.ids, i, kRbRankThreads, p.n, 0x7FFFFFFF, k);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j * kRbRankThreads < npad) s_key[i + j * kRbRankThreads] = k[j];
    }
    __syncthreads();
    const int base = blockIdx.x * 32, me = base + lane;
    const int key = me < p.n ? s_key[me] : 0;
    const int each = npad / W, j0 = warp * each, j1 = j0 + each;  // multiples of 4
    int cnt = 0;
    const int mid0 = min(max(base, j0), j1), mid1 = min(max(base + 32, j0), j1);
#pragma unroll 4
    for (int j = j0; j < mid0; j += 4) {
        const int4 v = *reinterpret_cast<const int4*>(s_key + j);
        cnt += (v.x <= key) + (v.y <= key) + (v.z <= key) + (v.w <= key);
    }
    for (int j = mid0; j < mid1; ++j) cnt += s_key[j] < key || (s_key[j] == key && j < me);
#pragma unroll 4
    for (int j = mid1; j < j1; j += 4) {
        const int4 v = *reinterpret_cast<const int4*>(s_key + j);
        cnt += (v.x < key) + (v.y < key) + (v.z < key) + (v.w < key);
    }
    s_part[warp][lane] = cnt;
    __syncthreads();
    if (warp == 0 && me < p.n) {
        int at = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) at += s_part[w][lane];
        p.keys[at] = key;
        p.order[at] = me;
    }
}

struct RbSortParams {
    RbIds ids;
    long long n;
    int32_t* keys[2];   // pass i writes [i & 1]
    int32_t* order[2];
    int32_t* done;      // zeros (RbSumParams)
    long long dones;
    int32_t passes, digit;
};

// Stable radix sort by one cluster of 8 CTAs (the largest portable size): every
// warp owns a contiguous range of keys, counts its digits, and the counts of
// all warps give each its places.  The CTAs read one another's counts through
// the cluster's shared memory and meet at the cluster barrier, so a pass needs
// no launch of its own.
__global__ void __cluster_dims__(kRbCluster, 1, 1) __launch_bounds__(kRbSortThreads)
    k_rb_sort(const __grid_constant__ RbSortParams p) {
    extern __shared__ __align__(16) uint32_t s_sort[];
    uint32_t* s_total = s_sort;                      // [kRbBins] of this CTA
    uint32_t* s_warp = s_sort + kRbBins;             // [warps][kRbBins]
    __shared__ uint32_t s_scan[kRbSortThreads / 32];
    constexpr int W = kRbSortThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = cluster_rank();
    const int bins = 1 << p.digit;
    // keys a warp, a multiple of 32; the warps of all CTAs in order
    const long long per = (p.n + 32ll * W * kRbCluster - 1) / (32ll * W * kRbCluster) * 32;
    const long long t0 = (static_cast<long long>(rank) * W + warp) * per, t1 = min(p.n, t0 + per);
    uint32_t* mine = s_warp + warp * kRbBins;
    for (long long i = static_cast<long long>(rank) * kRbSortThreads + tid; i < p.dones; i += kRbCluster * kRbSortThreads)
        p.done[i] = 0;
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.digit;
        const int32_t* kin = p.keys[(pass & 1) ^ 1];
        const int32_t* oin = p.order[(pass & 1) ^ 1];
        int32_t* kout = p.keys[pass & 1];
        int32_t* oout = p.order[pass & 1];
        auto load = [&](long long t, int (&key)[4]) {  // 128 keys, through L2: other SMs wrote them
            if (pass == 0) {
                rb_keys(p.ids, t + lane, 32, t1, -1, key);
                return;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) key[i] = t + 32 * i + lane < t1 ? __ldcg(kin + t + 32 * i + lane) : -1;
        };
        for (int i = lane; i < bins; i += 32) mine[i] = 0;
        __syncwarp();
        for (long long t = t0; t < t1; t += 128) {
            int key[4];
            load(t, key);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (t + 32 * i >= t1) break;
                const int d = key[i] < 0 ? bins : (key[i] >> shift) & (bins - 1);
                const unsigned peers = __match_any_sync(0xFFFFFFFFu, d);
                if (d < bins && (peers & lanemask_lt()) == 0) mine[d] += __popc(peers);
                __syncwarp();
            }
        }
        __syncthreads();
        for (int b = tid; b < bins; b += kRbSortThreads) {  // counts before each warp in this CTA
            uint32_t run = 0;
#pragma unroll 8
            for (int w = 0; w < W; ++w) {
                const uint32_t c = s_warp[w * kRbBins + b];
                s_warp[w * kRbBins + b] = run;
                run += c;
            }
            s_total[b] = run;
        }
        cluster_sync();
        // first place of this CTA's keys of bin tid: smaller bins of all CTAs, then this bin's earlier CTAs
        uint32_t total = 0, before = 0;
        if (tid < bins) {
            uint32_t of[kRbCluster];
#pragma unroll
            for (unsigned r = 0; r < kRbCluster; ++r) of[r] = cluster_load(s_total + tid, r);
#pragma unroll
            for (unsigned r = 0; r < kRbCluster; ++r) {
                if (r < rank) before += of[r];
                total += of[r];
            }
        }
        uint32_t run = total;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, run, d);
            if (lane >= d) run += v;
        }
        if (lane == 31) s_scan[warp] = run;
        __syncthreads();
        uint32_t first = run - total + before;
        for (int w = 0; w < min(warp, kRbBins / 32); ++w) first += s_scan[w];
        if (tid < bins) {
#pragma unroll 8
            for (int w = 0; w < W; ++w) s_warp[w * kRbBins + tid] += first;
        }
        __syncthreads();
        for (long long t = t0; t < t1; t += 128) {
            int key[4], tok[4];
            load(t, key);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long at = t + 32 * i + lane;
                tok[i] = at < t1 ? (pass ? __ldcg(oin + at) : static_cast<int>(at)) : 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (t + 32 * i >= t1) break;
                const int d = key[i] < 0 ? bins : (key[i] >> shift) & (bins - 1);
                const unsigned peers = __match_any_sync(0xFFFFFFFFu, d);
                const uint32_t at = d < bins ? mine[d] : 0;
                __syncwarp();
                if (d < bins) {
                    const uint32_t to = at + __popc(peers & lanemask_lt());
                    kout[to] = key[i];
                    oout[to] = tok[i];
                    if ((peers & lanemask_lt()) == 0) mine[d] = at + __popc(peers);
                }
                __syncwarp();
            }
        }
        cluster_sync();  // the pass is written, and every CTA is done with the counts
    }
}

// ------------------------------------------------------------------ summing
struct RbSumParams {
    RbIds ids;
    const int32_t* keys;
    const int32_t* order;
    const void* grad;
    void* latent;
    float* part;    // [chunk][2][cols]
    int32_t* done;  // [chunk][slice][3]: of the run that begins in the chunk, its first group's parts written and its
                    // groups added; of the run that goes on there, the parts written of the group that begins so
    long long n;
    float alpha;
    int32_t cols;
    int32_t slices;
    int32_t chunk;       // sorted tokens a CTA
    int32_t accumulate;
    long long sum_ctas;  // CTAs that sum; the rest write zeros
};

__device__ __forceinline__ void rb_load(const void* base, size_t at, bool f32, uint4 (&v)[2]) {
    if (f32) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
        v[0] = __ldcs(s);
        v[1] = __ldcs(s + 1);
    } else {
        v[0] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    }
}

__device__ __forceinline__ void rb_floats(const uint4 (&v)[2], bool f32, float (&f)[8]) {
    if (f32) {
        const unsigned w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    } else {
        const unsigned w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// latent[row][col .. col + 7] = alpha * acc (+ what is there)
template <bool kLatF32>
__device__ __forceinline__ void rb_store(void* latent, size_t at, const float (&acc)[8], float alpha, bool accumulate) {
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = alpha * acc[i];
    if (accumulate) {
        uint4 v[2];
        rb_load(latent, at, kLatF32, v);
        float f[8];
        rb_floats(v, kLatF32, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = fmaf(alpha, acc[i], f[i]);
    }
    if (kLatF32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(latent) + at);
        d[0] = make_float4(o[0], o[1], o[2], o[3]);
        d[1] = make_float4(o[4], o[5], o[6], o[7]);
    } else {
        unsigned w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
            w[i] = *reinterpret_cast<const unsigned*>(&b);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(latent) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Zeros in the rows of this block of kRbZeroRows whose bit in `absent` is set.
template <bool kLatF32>
__device__ __forceinline__ void rb_zero_rows(void* latent, long long r0, int cols, unsigned absent) {
    const int per_row = cols >> (kLatF32 ? 2 : 3);
    while (absent) {
        const int r = __ffs(absent) - 1;
        absent &= absent - 1;
        uint4* d = reinterpret_cast<uint4*>(static_cast<unsigned char*>(latent) +
                                            static_cast<size_t>(r0 + r) * cols * (kLatF32 ? 4 : 2));
        for (int i = threadIdx.x; i < per_row; i += kRbThreads) __stcs(d + i, make_uint4(0, 0, 0, 0));
    }
}

// Chunk c has written its part of a run longer than a chunk.  Whoever writes
// the last part of a group of kRbGroup (in these columns) adds the group's, in
// order; whoever adds the last group of the run adds the groups' sums: the
// result does not depend on who that is, and no sum is longer than a group
// plus the groups (8,192 ids that are one padding id, 1,024 columns: 32 us, not
// 120).  A launch of its own for this took 6 us.  Reached by the whole CTA.
template <bool kLatF32>
__device__ __forceinline__ void rb_join(const RbSumParams& p, long long c, int key, int col) {
    const int tid = threadIdx.x;
    // chunks that begin with this row, back from c and on from c + 1
    long long back = 0, on = 0;
    for (int q = kRbThreads; q == kRbThreads; back += q) {
        const long long k = c - back - tid;
        q = __syncthreads_count(k >= 0 && p.keys[k * p.chunk] == key);
    }
    for (int q = kRbThreads; q == kRbThreads; on += q) {
        const long long at = (c + 1 + on + tid) * p.chunk;
        q = __syncthreads_count(at < p.n && p.keys[at] == key);
    }
    long long first = c - back + 1;  // the first of them
    const bool inside = first > 0 && p.keys[first * p.chunk - 1] == key;
    if (inside) --first;  // the run begins inside the chunk before
    const int m = static_cast<int>(c + on - first + 1), lead = static_cast<int>(c - first) / kRbGroup * kRbGroup;
    const int size = min(kRbGroup, m - lead), groups = (m + kRbGroup - 1) / kRbGroup;
    __shared__ int s_last;
    auto last = [&](long long chunk, int level, int all) {  // of `all` arrivals, earlier writes of the others visible
        __threadfence();
        __syncthreads();
        if (tid == 0) s_last = atomicAdd(p.done + 3 * (chunk * p.slices + blockIdx.x % p.slices) + level, 1) == all - 1;
        __syncthreads();
        if (s_last) __threadfence();
        return s_last != 0;
    };
    auto place = [&](int k) {  // part k of the run
        return reinterpret_cast<float4*>(p.part + (2 * (first + k) + (k == 0 && inside ? 1 : 0)) * p.cols + col);
    };
    float acc[8];
    auto add = [&](int k0, int step, int count) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
        if (col >= p.cols) return;
#pragma unroll 4
        for (int k = 0; k < count; ++k) {
            const float4* s = place(k0 + k * step);
            const float4 x = __ldcg(s), y = __ldcg(s + 1);
            acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
            acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
        }
    };
    // (a chunk can end one run and begin another: the run's first group has a counter of its own)
    if (!last(first + lead, lead == 0 ? 0 : 2, size)) return;
    add(lead, 1, size);
    if (groups > 1) {
        if (col < p.cols) {  // in place of the group's first part
            float4* d = place(lead);
            d[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            d[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        }
        if (!last(first, 1, groups)) return;
        add(0, kRbGroup, groups);
    }
    if (col < p.cols) rb_store<kLatF32>(p.latent, static_cast<size_t>(key) * p.cols + col, acc, p.alpha, p.accumulate);
}

template <bool kGradF32, bool kLatF32>
__global__ void __launch_bounds__(kRbThreads) k_rb_sum(const __grid_constant__ RbSumParams p) {
    constexpr int U = kGradF32 ? 4 : 8;  // rows in flight a thread
    __shared__ int s_key[2 * kRbMaxChunk + 1], s_tok[2 * kRbMaxChunk];
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x >= p.sum_ctas) {  // rows without a token
        const long long r0 = (static_cast<long long>(blockIdx.x) - p.sum_ctas) * kRbZeroRows;
        const int row = static_cast<int>(r0) + (tid & 31);
        bool absent = false;
        if (row < p.ids.rows) {  // first sorted place whose key is >= row
            long long lo = 0, hi = p.n;
            while (lo < hi) {
                const long long mid = (lo + hi) >> 1;
                if (p.keys[mid] < row) lo = mid + 1;
                else hi = mid;
            }
            absent = lo == p.n || p.keys[lo] != row;
        }
        rb_zero_rows<kLatF32>(p.latent, r0, p.cols, __ballot_sync(0xFFFFFFFFu, absent));
        return;
    }
    const long long c = blockIdx.x / p.slices;
    const int col = static_cast<int>(blockIdx.x - c * p.slices) * kRbSliceCols + 8 * tid;
    const long long p0 = c * p.chunk;
    const int len = static_cast<int>(min(static_cast<long long>(p.chunk), p.n - p0));
    // places p0 .. p0 + 2 chunk - 1 (past the end: -1)
    for (int i = tid; i <= 2 * p.chunk; i += kRbThreads) {
        const bool on = p0 + i < p.n;
        s_key[i] = on ? p.keys[p0 + i] : -1;
        if (i < 2 * p.chunk) s_tok[i] = on ? p.order[p0 + i] : 0;
    }
    const int before = tid < p.chunk && p0 > tid ? p.keys[p0 - 1 - tid] : -1;
    __syncthreads();
    // the runs of equal keys that cross this chunk's borders
    const int k0 = s_key[0], k1 = s_key[len - 1];
    const int lead = __syncthreads_count(before == k0);                                      // of its first key, before it
    const int head = __syncthreads_count(tid < len && s_key[tid] == k0);                     // inside
    const int tail = __syncthreads_count(tid < len && s_key[tid] == k1);                     // of its last key, inside
    const int past = __syncthreads_count(tid < p.chunk && s_key[len + tid] == k1);           // behind it
    const bool one_run = k0 == k1;
    const int more = one_run ? past : 0;
    // a run longer than a chunk is cut at the borders; a shorter one belongs to the chunk that it begins in
    const bool lead_long = lead + head + more > p.chunk;
    int i_begin = 0, i_end = len;
    if (lead > 0 && !lead_long) i_begin = head;
    const bool tail_mine = !(one_run && lead > 0);  // the last run begins here
    const bool tail_long = tail_mine ? tail + past > p.chunk : lead_long;
    if (tail_mine && !tail_long) i_end = len + past;
    const bool col_on = col < p.cols;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    bool cut = lead > 0;  // (of a run that is processed here: a long one)
    int start = i_begin;
    if (i_begin > 0) cut = false;
    for (int i0 = i_begin; i0 < i_end; i0 += U) {
        uint4 v[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = col_on && i0 + u < i_end && s_key[i0 + u] < p.ids.rows;
            if (on) rb_load(p.grad, static_cast<size_t>(s_tok[i0 + u]) * p.cols + col, kGradF32, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            if (i >= i_end) break;
            const int key = s_key[i];
            if (key >= p.ids.rows) break;  // ids outside the table sort last
            float f[8];
            rb_floats(v[u], kGradF32, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] += f[q];
            if (i + 1 == i_end || s_key[i + 1] != key) {
                const bool goes_on = i + 1 == len && i + 1 == i_end && tail_long && past > 0;
                if (!col_on) {
                } else if (cut || goes_on) {
                    float4* d = reinterpret_cast<float4*>(p.part + (2 * c + (start == 0 ? 0 : 1)) * p.cols + col);
                    d[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    d[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
                } else {
                    rb_store<kLatF32>(p.latent, static_cast<size_t>(key) * p.cols + col, acc, p.alpha, p.accumulate);
                }
                cut = false;
                start = i + 1;
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] = 0.f;
            }
        }
    }
    // long runs that this chunk has a part of: its first and its last
    const bool lead_cut = lead > 0 && lead_long && k0 < p.ids.rows;
    const bool tail_cut = tail_mine && tail_long && past > 0 && k1 < p.ids.rows;
    if (lead_cut) rb_join<kLatF32>(p, c, k0, col);
    if (tail_cut) rb_join<kLatF32>(p, c, k1, col);
}

// Short batches: no sort, one launch.
template <bool kGradF32, bool kLatF32>
__global__ void __launch_bounds__(kRbThreads) k_rb_direct(const __grid_constant__ RbSumParams p) {
    constexpr int U = kGradF32 ? 4 : 8;
    __shared__ int s_key[kRbDirectMax];
    __shared__ int s_tok[kRbDirectMax];
    const int tid = threadIdx.x, n = static_cast<int>(p.n);
    if (tid < n) s_key[tid] = rb_key(p.ids, tid);
    __syncthreads();
    if (blockIdx.x >= p.sum_ctas) {
        const long long r0 = (static_cast<long long>(blockIdx.x) - p.sum_ctas) * kRbZeroRows;
        const int row = static_cast<int>(r0) + (tid & 31);
        bool absent = row < p.ids.rows;
        for (int i = 0; i < n; ++i) absent = absent && s_key[i] != row;
        rb_zero_rows<kLatF32>(p.latent, r0, p.cols, __ballot_sync(0xFFFFFFFFu, absent));
        return;
    }
    const int t = static_cast<int>(blockIdx.x / p.slices);
    const int col = static_cast<int>(blockIdx.x - t * p.slices) * kRbSliceCols + 8 * tid;
    const int key = s_key[t];
    if (key >= p.ids.rows) return;
    // the tokens of this row, in order; an earlier one means another CTA sums it
    int m = 0;
    bool first = true;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + (tid & 31);
        const unsigned same = __ballot_sync(0xFFFFFFFFu, i < n && s_key[i] == key);
        if (same && i0 + __ffs(same) - 1 < t) first = false;
        if (((same >> (tid & 31)) & 1u) && tid < 32) s_tok[m + __popc(same & lanemask_lt())] = i;
        m += __popc(same);
    }
    if (!first) return;  // the same in every thread
    __syncthreads();
    if (col >= p.cols) return;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int i0 = 0; i0 < m; i0 += U) {
        uint4 v[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u < m) rb_load(p.grad, static_cast<size_t>(s_tok[i0 + u]) * p.cols + col, kGradF32, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u >= m) break;
            float f[8];
            rb_floats(v[u], kGradF32, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] += f[q];
        }
    }
    rb_store<kLatF32>(p.latent, static_cast<size_t>(key) * p.cols + col, acc, p.alpha, p.accumulate);
}

}  // namespace e8q

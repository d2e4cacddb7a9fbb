// Backward of the row lookup (identity straight-through estimator, "E8-QAT",
// Figure 2 (b)): every latent row gets the sum of the output gradients of
// the tokens that read it,
//   G[r] (+)= alpha * sum_{t : id_t - first_row = r} g[t],
// in fp32, in token order, rounded once.  Nothing is added with an atomic, so
// the result does not depend on timing.
//
// Tokens are first sorted by row, ties by position:
//   n <= kRbRankMax   k_rb_rank: the place of a token is the number of tokens
//                     before it in (row, position) order, counted against all
//                     n ids held in shared memory; n^2 comparisons over all
//                     SMs cost less than the launches of a radix sort;
//   above             k_rb_hist + k_rb_scatter a digit of up to 9 bits: each
//                     CTA's histogram, then every CTA derives its own bases
//                     from all histograms and places its keys in order.
// Then
//   k_rb_sum          one CTA per (chunk of sorted tokens, 1,024 columns): a
//                     thread owns 8 columns and keeps a batch of rows in
//                     flight.  A row whose tokens lie in one chunk is written at
//                     once; a row cut by a chunk border leaves fp32 partial
//                     sums (at most two a chunk).  Further CTAs of the same
//                     launch write the zeros of the rows without a token, so
//                     that every output byte is written once;
//   k_rb_join         the rows cut by chunk borders: their partial sums in
//                     order, the list split over 16 warps (a padding id may
//                     fill thousands of chunks).
// Short batches (n <= kRbDirectMax) need no sort: k_rb_direct has one CTA per
// (token, 1,024 columns), and the first token of a row sums the others'.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace e8q {

constexpr int kRbThreads = 128;
constexpr int kRbSliceCols = kRbThreads * 8;
constexpr int kRbDirectMax = 128;
constexpr int kRbRankMax = 8192;
constexpr int kRbRankKeys = 64;  // keys a rank CTA places
constexpr int kRbRankThreads = 256;
constexpr int kRbZeroRows = 32;
constexpr int kRbMaxChunk = 128;
constexpr int kRbTile = 2048;  // keys of a radix CTA
constexpr int kRbDigitBits = 9;
constexpr int kRbBins = 1 << kRbDigitBits;
constexpr int kRbJoinThreads = 512;
constexpr int kRbJoinCols = 256;

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

// ------------------------------------------------------------------ sorting
struct RbRankParams {
    RbIds ids;
    int32_t n;
    int32_t* keys;   // out: sorted rows
    int32_t* order;  // out: their tokens
};

__global__ void __launch_bounds__(kRbRankThreads) k_rb_rank(const __grid_constant__ RbRankParams p) {
    __shared__ __align__(16) int s_key[kRbRankMax];
    __shared__ int s_part[kRbRankThreads];
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    const int npad = (p.n + 15) & ~15;
    for (int i = tid; i < npad; i += kRbRankThreads) s_key[i] = i < p.n ? rb_key(p.ids, i) : 0x7FFFFFFF;
    __syncthreads();
    // thread (k, q): key k of this CTA against the q-th quarter of all keys
    const int k = tid % kRbRankKeys, q = tid / kRbRankKeys;
    const int base = blockIdx.x * kRbRankKeys, me = base + k;
    const int key = me < p.n ? s_key[me] : 0;
    const int quarter = npad >> 2;  // a multiple of 4
    int cnt = 0;
    for (int j = q * quarter; j < (q + 1) * quarter; j += 4) {
        const int4 v = *reinterpret_cast<const int4*>(s_key + j);
        if (j + 4 <= base) {  // all before this CTA's keys: ties come first
            cnt += (v.x <= key) + (v.y <= key) + (v.z <= key) + (v.w <= key);
        } else if (j >= base + kRbRankKeys) {
            cnt += (v.x < key) + (v.y < key) + (v.z < key) + (v.w < key);
        } else {
            cnt += (v.x < key || (v.x == key && j < me)) + (v.y < key || (v.y == key && j + 1 < me)) +
                   (v.z < key || (v.z == key && j + 2 < me)) + (v.w < key || (v.w == key && j + 3 < me));
        }
    }
    s_part[tid] = cnt;
    __syncthreads();
    if (q == 0 && me < p.n) {
        const int at = s_part[k] + s_part[k + kRbRankKeys] + s_part[k + 2 * kRbRankKeys] + s_part[k + 3 * kRbRankKeys];
        p.keys[at] = key;
        p.order[at] = me;
    }
}

struct RbRadixParams {
    RbIds ids;
    long long n;
    const int32_t* keys_in;  // NULL: the ids, in token order
    const int32_t* order_in;
    int32_t* keys;
    int32_t* order;
    uint32_t* hist;  // [CTA][kRbBins]
    int32_t shift;
    int32_t mask;
};

__global__ void __launch_bounds__(256) k_rb_hist(const __grid_constant__ RbRadixParams p) {
    __shared__ uint32_t s_h[kRbBins];
    for (int i = threadIdx.x; i < kRbBins; i += 256) s_h[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const long long t0 = static_cast<long long>(blockIdx.x) * kRbTile;
    for (int i = threadIdx.x; i < kRbTile; i += 256) {
        if (t0 + i >= p.n) break;
        const int key = p.keys_in ? p.keys_in[t0 + i] : rb_key(p.ids, t0 + i);
        atomicAdd(&s_h[(key >> p.shift) & p.mask], 1u);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kRbBins; i += 256) p.hist[static_cast<size_t>(blockIdx.x) * kRbBins + i] = s_h[i];
}

__global__ void __launch_bounds__(256) k_rb_scatter(const __grid_constant__ RbRadixParams p) {
    __shared__ uint32_t s_w[8][kRbBins];
    __shared__ uint32_t s_base[kRbBins];
    __shared__ uint32_t s_scan[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < 8 * kRbBins; i += 256) (&s_w[0][0])[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const long long t0 = static_cast<long long>(blockIdx.x) * kRbTile + 256 * warp;
    int key[8], dig[8];
    unsigned peers[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const long long i = t0 + 32 * j + lane;
        key[j] = i < p.n ? (p.keys_in ? p.keys_in[i] : rb_key(p.ids, i)) : 0;
        dig[j] = i < p.n ? ((key[j] >> p.shift) & p.mask) : kRbBins;  // lanes past the end match only each other
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        peers[j] = __match_any_sync(0xFFFFFFFFu, dig[j]);
        if (dig[j] < kRbBins && (peers[j] & lanemask_lt()) == 0) s_w[warp][dig[j]] += __popc(peers[j]);
        __syncwarp();
    }
    // first place of this CTA's keys of every bin: smaller bins of all CTAs, then this bin's earlier CTAs
    uint32_t total[2] = {0, 0}, before[2] = {0, 0};
    for (unsigned c = 0; c < gridDim.x; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t v = p.hist[static_cast<size_t>(c) * kRbBins + 2 * tid + h];
            if (c < blockIdx.x) before[h] += v;
            total[h] += v;
        }
    }
    const uint32_t mine = total[0] + total[1];
    uint32_t run = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, run, d);
        if (lane >= d) run += v;
    }
    if (lane == 31) s_scan[warp] = run;
    __syncthreads();
    uint32_t first = run - mine;
    for (int w = 0; w < warp; ++w) first += s_scan[w];
    s_base[2 * tid] = first + before[0];
    s_base[2 * tid + 1] = first + total[0] + before[1];
    __syncthreads();
    for (int b = tid; b < kRbBins; b += 256) {
        uint32_t at = s_base[b];
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const uint32_t c = s_w[w][b];
            s_w[w][b] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const long long i = t0 + 32 * j + lane;
        uint32_t at = 0;
        if (dig[j] < kRbBins) at = s_w[warp][dig[j]] + __popc(peers[j] & lanemask_lt());
        __syncwarp();
        if (dig[j] < kRbBins) {
            if ((peers[j] & lanemask_lt()) == 0) s_w[warp][dig[j]] += __popc(peers[j]);
            p.keys[at] = key[j];
            p.order[at] = p.order_in ? p.order_in[i] : static_cast<int32_t>(i);
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------ summing
struct RbSumParams {
    RbIds ids;
    const int32_t* keys;
    const int32_t* order;
    const void* grad;
    void* latent;
    float* part;  // [chunk][2][cols]
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

template <bool kGradF32, bool kLatF32>
__global__ void __launch_bounds__(kRbThreads) k_rb_sum(const __grid_constant__ RbSumParams p) {
    constexpr int U = kGradF32 ? 4 : 8;  // rows in flight a thread
    __shared__ int s_key[kRbMaxChunk + 2], s_tok[kRbMaxChunk];
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
    for (int i = tid; i < len + 2; i += kRbThreads) {  // s_key[i + 1] is the key of place p0 + i
        const long long at = p0 + i - 1;
        s_key[i] = (at >= 0 && at < p.n) ? p.keys[at] : -1;
    }
    for (int i = tid; i < len; i += kRbThreads) s_tok[i] = p.order[p0 + i];
    __syncthreads();
    if (col >= p.cols) return;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    bool cut = s_key[0] == s_key[1];  // the current row began in an earlier chunk
    int start = 0;
    for (int i0 = 0; i0 < len; i0 += U) {
        uint4 v[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = i0 + u < len && s_key[i0 + u + 1] < p.ids.rows;
            if (on) rb_load(p.grad, static_cast<size_t>(s_tok[i0 + u]) * p.cols + col, kGradF32, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            if (i >= len) break;
            const int key = s_key[i + 1];
            if (key >= p.ids.rows) break;  // ids outside the table sort last
            float f[8];
            rb_floats(v[u], kGradF32, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] += f[q];
            const bool last = i + 1 == len;
            if (last || s_key[i + 2] != key) {
                const bool goes_on = last && s_key[i + 2] == key;
                if (cut || goes_on) {
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
}

// Rows cut by chunk borders: CTA (border b = chunk b | chunk b + 1, 256
// columns) acts where a cut row's first chunk is b.
template <bool kLatF32>
__global__ void __launch_bounds__(kRbJoinThreads) k_rb_join(const __grid_constant__ RbSumParams p) {
    __shared__ __align__(16) float s_sum[kRbJoinThreads / 32][kRbJoinCols];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    const int slices = (p.cols + kRbJoinCols - 1) / kRbJoinCols;
    const long long b = blockIdx.x / slices;
    const int col = static_cast<int>(blockIdx.x - b * slices) * kRbJoinCols + 8 * lane;
    const long long border = (b + 1) * p.chunk;
    const int key = p.keys[border];
    if (key >= p.ids.rows || p.keys[border - 1] != key) return;
    if (b > 0 && p.keys[border - p.chunk - 1] == key) return;  // began earlier
    const long long chunks = (p.n + p.chunk - 1) / p.chunk;
    long long lo = b + 1, hi = chunks - 1;  // last chunk that begins with this row
    while (lo < hi) {
        const long long mid = (lo + hi + 1) >> 1;
        if (p.keys[mid * p.chunk] == key) lo = mid;
        else hi = mid - 1;
    }
    const long long m = lo - b + 1;  // partial sums
    const int first_slot = p.keys[b * p.chunk] == key ? 0 : 1;
    constexpr int W = kRbJoinThreads / 32;
    const long long per = (m + W - 1) / W;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    if (col < p.cols) {
        const long long k1 = min(m, (warp + 1) * per);
#pragma unroll 4
        for (long long k = warp * per; k < k1; ++k) {
            const float4* s = reinterpret_cast<const float4*>(p.part + (2 * (b + k) + (k == 0 ? first_slot : 0)) * p.cols + col);
            const float4 x = __ldcs(s), y = __ldcs(s + 1);
            acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
            acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
        }
    }
    float4* d = reinterpret_cast<float4*>(&s_sum[warp][8 * lane]);
    d[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    d[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    __syncthreads();
    if (warp != 0 || col >= p.cols) return;
    const int used = static_cast<int>((m + per - 1) / per);
    for (int w = 1; w < used; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += s_sum[w][8 * lane + i];
    rb_store<kLatF32>(p.latent, static_cast<size_t>(key) * p.cols + col, acc, p.alpha, p.accumulate);
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

// Low-rank adapters of many requests beside a shared projection, forward
// and backward.  Token t has the adapter a = slots[t] (none: outside 0..n-1):
//
//   u_t = A_a x_t,   y_t = base_t + s_a B_a u_t
//   v_t = s_a B_a^T gy_t,   gx_t = gx0_t + A_a^T v_t
//   gA_a = sum_t v_t x_t^T,   gB_a = sum_t gy_t (s_a u_t)^T
//
// The tokens are grouped by adapter first (k_lr_plan); everything after it
// works on tiles of up to 64 (8 in small batches) tokens of one adapter:
//
//   k_lr_down   p = W z, a long sum over the columns of z and a short result
//               (u from x and A; v / s from gy and B): tensor cores with the
//               rank as M and the tokens as N (8 a tile, so that one token wastes
//               7 columns, not 15), operands straight from global memory in
//               16-byte loads.  The sum's order is free, so lane q takes the
//               columns 8q..8q+7 of a 32-column block as they lie in memory and
//               both operands use that order.  The columns are split over the
//               warps of a CTA and over CTAs; partial sums are added in a
//               fixed order;
//   k_lr_up     out = base + W w, a short sum and a long result (y from u and
//               B; gx from v and A): tokens as M, columns as N; the columns of
//               the four 8-column MMA tiles of a 32-column chunk are dealt so
//               that a lane ends up with 8 neighbouring ones (16-byte loads of
//               base and stores of out);
//   k_lr_split  (backward) w = s u and v as bf16 high + low parts;
//   k_lr_grad   sums over tokens: gB from gy and s u, gA from x and v, both in
//               one launch.  z^T and w come from shared memory by transposing
//               ldmatrix; long token ranges are split into units whose partial
//               sums k_lr_join adds in order.
//
// The fp32 factors u, v enter the tensor cores as a bf16 high part plus a
// bf16 low part (two MMAs, about 16 bits), so that the only rounding to bf16
// that counts is the result's.  Everything is bound by reading and writing
// the token matrices; ranks up to 128 leave the tensor cores far from busy,
// which is why these are warp-level MMAs fed from registers.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace e8q {

constexpr int kLrMaxTokens = 65536;
constexpr int kLrMaxAdapters = 2048;
constexpr int kLrMaxRank = 128;
constexpr int64_t kLrMaxWidth = 1 << 20;
constexpr int kLrPlanThreads = 1024;
constexpr int kLrTile = 64;        // tokens a tile
constexpr int kLrSmallTile = 8;    // in batches of up to kLrSmallTokens
constexpr int kLrSmallTokens = 128;
constexpr int kLrDownThreads = 256;
constexpr int kLrUpThreads = 128;
constexpr int kLrGradThreads = 256;
constexpr int kLrGradCols = 256;

struct LrTile {  // of tokens of one adapter, in the grouped order
    int32_t first, len, slot, pad;
};

// ------------------------------------------------------------------ grouping
struct LrPlanParams {
    const int32_t* slots;
    int32_t tokens, n;
    int32_t tile, unit;   // tokens a tile, a unit
    int32_t* head;        // out: tiles, units, grouped tokens that have an adapter
    int32_t* order;       // out: tokens by adapter, those without one last; original order inside
    LrTile* tiles;        // out
    LrTile* units;        // out (with adapters only), pad = the unit's place among the partial sums, or -1
    int32_t* unit_base;   // out: [n] first partial sum of each adapter, [n] its units
};

// One CTA: a stable counting sort by adapter, each warp over its own range.
__global__ void __launch_bounds__(kLrPlanThreads) k_lr_plan(const __grid_constant__ LrPlanParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nb = p.n + 1;  // bin n: no adapter
    int* s_tok = reinterpret_cast<int*>(smem);   // [nb + 1] first token, tile, unit of each bin
    int* s_tile = s_tok + nb + 1;
    int* s_unit = s_tile + nb + 1;
    int* s_part = s_unit + nb + 1;  // units of adapters that have several: those need partial sums
    uint16_t* hist = reinterpret_cast<uint16_t*>(s_part + nb + 1);  // [32][nb]
    __shared__ int s_scan[4][32];
    pdl_launch_dependents();
    for (int i = tid; i < 32 * nb; i += kLrPlanThreads) hist[i] = 0;
    __syncthreads();
    const int per = ((p.tokens + 1023) / 1024) * 32, t0 = warp * per, t1 = min(p.tokens, t0 + per);
    uint16_t* mine = hist + warp * nb;
    const unsigned below = (1u << lane) - 1u;
    for (int t = t0; t < t1; t += 32) {
        int bin = nb;  // past the end: matched only by its like
        if (t + lane < t1) {
            const int s = __ldg(p.slots + t + lane);
            bin = (s >= 0 && s < p.n) ? s : p.n;
        }
        const unsigned peers = __match_any_sync(0xFFFFFFFFu, bin);
        if (bin < nb && (peers & below) == 0) mine[bin] = static_cast<uint16_t>(mine[bin] + __popc(peers));
        __syncwarp();
    }
    __syncthreads();
    // bins 3 tid .. 3 tid + 2: counts before each warp, then the scan over the bins
    int cnt[3], sum[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int b = 3 * tid + i;
        int run = 0;
        if (b < nb)
            for (int w = 0; w < 32; ++w) {
                const int c = hist[w * nb + b];
                hist[w * nb + b] = static_cast<uint16_t>(run);
                run += c;
            }
        cnt[i] = run;
        sum[0] += run;
        sum[1] += (run + p.tile - 1) / p.tile;
        if (b < p.n) {
            const int u = (run + p.unit - 1) / p.unit;
            sum[2] += u;
            sum[3] += u > 1 ? u : 0;
        }
    }
    int inc[4] = {sum[0], sum[1], sum[2], sum[3]};
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, inc[i], d);
            if (lane >= d) inc[i] += v;
        }
    if (lane == 31)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_scan[i][warp] = inc[i];
    __syncthreads();
    int at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        at[i] = inc[i] - sum[i];
        for (int w = 0; w < warp; ++w) at[i] += s_scan[i][w];
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int b = 3 * tid + i;
        if (b > nb) break;
        s_tok[b] = at[0];
        s_tile[b] = at[1];
        s_unit[b] = at[2];
        s_part[b] = at[3];
        if (b == nb) break;
        at[0] += cnt[i];
        at[1] += (cnt[i] + p.tile - 1) / p.tile;
        if (b < p.n) {
            const int u = (cnt[i] + p.unit - 1) / p.unit;
            at[2] += u;
            at[3] += u > 1 ? u : 0;
        }
    }
    __syncthreads();
    for (int t = t0; t < t1; t += 32) {
        int bin = nb;
        if (t + lane < t1) {
            const int s = __ldg(p.slots + t + lane);
            bin = (s >= 0 && s < p.n) ? s : p.n;
        }
        const unsigned peers = __match_any_sync(0xFFFFFFFFu, bin);
        const int before = bin < nb ? mine[bin] : 0;
        __syncwarp();
        if (bin < nb) {
            p.order[s_tok[bin] + before + __popc(peers & below)] = t + lane;
            if ((peers & below) == 0) mine[bin] = static_cast<uint16_t>(before + __popc(peers));
        }
        __syncwarp();
    }
    const int ntiles = s_tile[nb], nunits = s_unit[p.n];
    for (int k = tid; k < ntiles; k += kLrPlanThreads) {
        int lo = 0, hi = nb - 1;  // last bin whose first tile is <= k (empty bins share theirs with the next)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_tile[mid] <= k) lo = mid;
            else hi = mid - 1;
        }
        const int first = s_tok[lo] + (k - s_tile[lo]) * p.tile;
        p.tiles[k] = LrTile{first, min(p.tile, s_tok[lo + 1] - first), lo < p.n ? lo : -1, 0};
    }
    for (int k = tid; k < nunits; k += kLrPlanThreads) {
        int lo = 0, hi = p.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_unit[mid] <= k) lo = mid;
            else hi = mid - 1;
        }
        const int first = s_tok[lo] + (k - s_unit[lo]) * p.unit;
        const int several = s_unit[lo + 1] - s_unit[lo] > 1;
        p.units[k] = LrTile{first, min(p.unit, s_tok[lo + 1] - first), lo, several ? s_part[lo] + k - s_unit[lo] : -1};
    }
    for (int b = tid; b < p.n; b += kLrPlanThreads) {
        p.unit_base[b] = s_part[b];
        p.unit_base[p.n + b] = s_unit[b + 1] - s_unit[b];
    }
    if (tid == 0) {
        p.head[0] = ntiles;
        p.head[1] = nunits;
        p.head[2] = s_tok[p.n];
    }
}

// ------------------------------------------------------------------ helpers
__device__ __forceinline__ void lr_mma(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                       unsigned b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// four 8x8 b16 matrices from shared memory, transposed; lane l gives row l % 8 of matrix l / 8
__device__ __forceinline__ void ldsm_t4(unsigned (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16-byte copy, or 16 zero bytes where it is off (nothing is read then)
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ unsigned lr_pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&h);
}
__device__ __forceinline__ float lr_lo(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float lr_hi(unsigned w) { return __uint_as_float(w & 0xFFFF0000u); }
// (a, b) = high parts + low parts; a part that is not finite leaves no rest
__device__ __forceinline__ void lr_split2(float a, float b, unsigned& high, unsigned& low) {
    high = lr_pack(a, b);
    const float ra = a - lr_lo(high), rb = b - lr_hi(high);
    low = lr_pack(fabsf(ra) <= fabsf(a) ? ra : 0.f, fabsf(rb) <= fabsf(b) ? rb : 0.f);
}

// ------------------------------------------------------------------ p = W z
struct LrDownParams {
    const int32_t* head;
    const int32_t* order;
    const LrTile* tiles;
    const uint16_t* z;  // [tokens][cols]
    const uint16_t* w;  // [n][rank][cols], or [n][cols][rank] (kTrans)
    float* part;        // [split][tokens][rank]
    int32_t tokens, cols, rank;
    int32_t per;        // columns a CTA, a multiple of 256
};

// Column n of a 32-column block -> row of the staged block, such that the
// eight rows of each 8x8 matrix of the MMA's A operand follow one another.
__device__ __forceinline__ int lr_stage_row(int n) { return 16 * ((n >> 2) & 1) + 8 * ((n >> 1) & 1) + 2 * (n >> 3) + (n & 1); }

// MT: 16-row tiles of the rank (4 at most: higher ranks in gridDim.z parts).
// kSmall: tiles of 8 tokens, 8 warps along the columns; else 64 tokens, 2 x 4.
template <int MT, bool kSmall, bool kTrans>
__global__ void __launch_bounds__(kLrDownThreads) k_lr_down(const __grid_constant__ LrDownParams p) {
    constexpr int KW = kSmall ? 8 : 4, NT = kSmall ? 1 : 4;
    constexpr int STEP = 32 * KW;                // columns a round
    constexpr int ROW = MT * 16 * 2 + 16;        // bytes of a staged row (kTrans), padded against bank conflicts
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q = lane & 3, c = lane >> 2;
    const int kq = kSmall ? warp : (warp & 3), th = kSmall ? 0 : (warp >> 2);
    pdl_wait();
    pdl_launch_dependents();
    if (static_cast<int>(blockIdx.x) >= p.head[0]) return;
    const LrTile tile = p.tiles[blockIdx.x];
    if (tile.slot < 0) return;
    const int k0 = static_cast<int>(blockIdx.y) * p.per, k1 = min(p.cols, k0 + p.per);
    const int r0 = static_cast<int>(blockIdx.z) * 64;
    const uint16_t* w = p.w + static_cast<size_t>(tile.slot) * p.rank * p.cols;
    const uint16_t* zr[NT];
    bool on[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int t = 32 * th + 8 * i + c;
        on[i] = t < tile.len;
        zr[i] = p.z + static_cast<size_t>(on[i] ? p.order[tile.first + t] : 0) * p.cols;
    }
    const int live = min(NT, (tile.len - 32 * th + 7) >> 3);  // token tiles with a token (the same in the whole warp)
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][i][e] = 0.f;
    const uint4 zero = make_uint4(0, 0, 0, 0);

    auto load_z = [&](int kb, uint4 (&x)[NT]) {
        const int k = kb + 8 * q;
#pragma unroll
        for (int i = 0; i < NT; ++i)
            x[i] = (on[i] && k < k1) ? __ldg(reinterpret_cast<const uint4*>(zr[i] + k)) : zero;
    };
    auto multiply = [&](const unsigned (&a)[MT][2][4], const uint4 (&x)[NT]) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (i >= live) break;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                lr_mma(acc[m][i], a[m][0][0], a[m][0][1], a[m][0][2], a[m][0][3], x[i].x, x[i].y);
                lr_mma(acc[m][i], a[m][1][0], a[m][1][1], a[m][1][2], a[m][1][3], x[i].z, x[i].w);
            }
        }
    };

    if (!kTrans) {
        auto load_w = [&](int kb, uint4 (&v)[MT][2]) {
            const int k = kb + 8 * q;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = r0 + 16 * m + 8 * h + c;
                    v[m][h] = (r < p.rank && k < k1) ? __ldg(reinterpret_cast<const uint4*>(w + static_cast<size_t>(r) * p.cols + k)) : zero;
                }
        };
        uint4 x[NT], v[MT][2];
        int kb = k0 + 32 * kq;
        load_z(kb, x);
        load_w(kb, v);
        for (; kb < k1; kb += STEP) {
            uint4 xn[NT], vn[MT][2];
            load_z(kb + STEP, xn);
            load_w(kb + STEP, vn);
            unsigned a[MT][2][4];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                a[m][0][0] = v[m][0].x; a[m][0][1] = v[m][1].x; a[m][0][2] = v[m][0].y; a[m][0][3] = v[m][1].y;
                a[m][1][0] = v[m][0].z; a[m][1][1] = v[m][1].z; a[m][1][2] = v[m][0].w; a[m][1][3] = v[m][1].w;
            }
            multiply(a, x);
#pragma unroll
            for (int i = 0; i < NT; ++i) x[i] = xn[i];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                v[m][0] = vn[m][0];
                v[m][1] = vn[m][1];
            }
        }
    } else {
        // the weights of a round, [STEP columns][16 MT ranks], through shared memory, two rounds deep
        constexpr int CH = 2 * MT;  // 16-byte pieces of a row
        const uint32_t base = smem_addr(smem);
        auto stage = [&](int kb, int buf) {
            for (int i = tid; i < STEP * CH; i += kLrDownThreads) {
                const int n = i / CH, piece = i - n * CH, k = kb + n, r = r0 + 8 * piece;
                const uint32_t dst = base + (buf * STEP + (n & ~31) + lr_stage_row(n & 31)) * ROW + 16 * piece;
                const bool in = k < k1 && r < p.rank;
                cp_async16_or_zero(dst, in ? w + static_cast<size_t>(k) * p.rank + r : w, in);
            }
            cp_async_commit();
        };
        uint4 x[NT];
        stage(k0, 0);
        load_z(k0 + 32 * kq, x);
        int buf = 0;
        for (int kr = k0; kr < k1; kr += STEP, buf ^= 1) {
            uint4 xn[NT];
            load_z(kr + STEP + 32 * kq, xn);
            cp_async_wait<0>();
            __syncthreads();  // the round's weights are there, and the other buffer is read
            if (kr + STEP < k1) stage(kr + STEP, buf ^ 1);
            unsigned a[MT][2][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    ldsm_t4(a[m][h], base + (buf * STEP + 32 * kq + 16 * h + 8 * (lane >> 4) + (lane & 7)) * ROW +
                                         32 * m + 16 * ((lane >> 3) & 1));
            multiply(a, x);
#pragma unroll
            for (int i = 0; i < NT; ++i) x[i] = xn[i];
        }
        __syncthreads();  // the staging memory becomes the reduction's
    }

    // the column warps' sums, in order
    float* red = reinterpret_cast<float*>(smem);
    constexpr int V = MT * NT * 4;
    if (kq > 0) {
        float* d = red + ((kq - 1) * (kSmall ? 1 : 2) + th) * V * 32 + lane;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[((m * NT + i) * 4 + e) * 32] = acc[m][i][e];
    }
    __syncthreads();
    if (kq > 0) return;
    for (int k = 1; k < KW; ++k) {
        const float* d = red + ((k - 1) * (kSmall ? 1 : 2) + th) * V * 32 + lane;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][i][e] += d[((m * NT + i) * 4 + e) * 32];
    }
    float* out = p.part + static_cast<size_t>(blockIdx.y) * p.tokens * p.rank;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 32 * th + 8 * i + 2 * q + e;
            if (t >= tile.len) continue;
            float* row = out + static_cast<size_t>(p.order[tile.first + t]) * p.rank;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = r0 + 16 * m + 8 * h + c;
                    if (r < p.rank) row[r] = acc[m][i][2 * h + e];
                }
        }
}

__host__ __device__ constexpr size_t lr_down_smem(int mt, bool small, bool trans) {
    const size_t kw = small ? 8 : 4, nt = small ? 1 : 4;
    const size_t red = (kw - 1) * (small ? 1 : 2) * mt * nt * 4 * 32 * 4;
    const size_t stage = trans ? 2 * 32 * kw * (static_cast<size_t>(mt) * 32 + 16) : 0;
    return red > stage ? red : stage;
}

// ------------------------------------------------------------------ out = base + W w
struct LrUpParams {
    const int32_t* head;
    const int32_t* order;
    const LrTile* tiles;
    const float* part;      // [splits][tokens][rank]
    const float* scale;
    const uint16_t* w;      // [n][cols][rank], or [n][rank][cols] (kTrans)
    const uint16_t* base;   // [tokens][cols] or NULL
    uint16_t* out;          // [tokens][cols]
    float* sum;             // [tokens][rank]: the sum of the parts, or NULL
    int32_t tokens, cols, rank;
    int32_t splits;
    int32_t range;          // columns a CTA, a multiple of 128
};

template <bool kTrans>
__global__ void __launch_bounds__(kLrUpThreads) k_lr_up(const __grid_constant__ LrUpParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    uint4* s_w = reinterpret_cast<uint4*>(smem);  // [token tile of 16][16 ranks][high | low][lane]
    __shared__ int s_tok[kLrTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q = lane & 3, c = lane >> 2;
    pdl_wait();
    pdl_launch_dependents();
    if (static_cast<int>(blockIdx.x) >= p.head[0]) return;
    const LrTile tile = p.tiles[blockIdx.x];
    const int c0 = static_cast<int>(blockIdx.y) * p.range, c1 = min(p.cols, c0 + p.range);
    for (int i = tid; i < tile.len; i += kLrUpThreads) s_tok[i] = p.order[tile.first + i];
    __syncthreads();
    const int per_row = (c1 - c0) >> 3;
    if (tile.slot < 0) {  // tokens without an adapter
        if (p.sum && blockIdx.y == 0)
            for (int i = tid; i < tile.len * p.rank; i += kLrUpThreads)
                p.sum[static_cast<size_t>(s_tok[i / p.rank]) * p.rank + i % p.rank] = 0.f;
        if (p.base == p.out) return;
        for (int i = tid; i < tile.len * per_row; i += kLrUpThreads) {
            const int t = i / per_row;
            const size_t at = static_cast<size_t>(s_tok[t]) * p.cols + c0 + 8 * (i - t * per_row);
            *reinterpret_cast<uint4*>(p.out + at) =
                p.base ? *reinterpret_cast<const uint4*>(p.base + at) : make_uint4(0, 0, 0, 0);
        }
        return;
    }
    // A operands: lane (c, q) holds tokens c and c + 8, ranks 4q..4q+3 of every 16
    const int mt = (tile.len + 15) >> 4, ks = (p.rank + 15) >> 4;
    const float s = __ldg(p.scale + tile.slot);
    for (int i = warp; i < mt * ks; i += kLrUpThreads / 32) {
        const int m = i / ks, r = 16 * (i - m * ks) + 4 * q;
        unsigned hi[4], lo[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = 16 * m + 8 * h + c;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < tile.len && r < p.rank) {
                const size_t at = static_cast<size_t>(s_tok[t]) * p.rank + r;
                f = *reinterpret_cast<const float4*>(p.part + at);
                for (int k = 1; k < p.splits; ++k) {
                    const float4 g = *reinterpret_cast<const float4*>(p.part + static_cast<size_t>(k) * p.tokens * p.rank + at);
                    f.x += g.x; f.y += g.y; f.z += g.z; f.w += g.w;
                }
                if (p.sum && blockIdx.y == 0) *reinterpret_cast<float4*>(p.sum + at) = f;
            }
            lr_split2(s * f.x, s * f.y, hi[h], lo[h]);
            lr_split2(s * f.z, s * f.w, hi[2 + h], lo[2 + h]);
        }
        s_w[(2 * i) * 32 + lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        s_w[(2 * i + 1) * 32 + lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    __syncthreads();

    const uint16_t* w = p.w + static_cast<size_t>(tile.slot) * p.rank * p.cols;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int col = c0 + 32 * warp; col < c1; col += 32 * (kLrUpThreads / 32)) {
        const bool col_on = col + 8 * q < c1;
        uint4 base[4][2];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = 16 * m + 8 * h + c;
                base[m][h] = zero;
                if (p.base && col_on && t < tile.len)
                    base[m][h] = *reinterpret_cast<const uint4*>(p.base + static_cast<size_t>(s_tok[t]) * p.cols + col + 8 * q);
            }
        float acc[4][4][4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
        for (int k = 0; k < ks; ++k) {
            const int r = 16 * k + 4 * q;
            unsigned b[4][2];  // MMA tile j, its column c: column 8 (c / 2) + 2 j + c % 2 of the chunk
            if (!kTrans) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = col + 8 * (c >> 1) + 2 * j + (c & 1);
                    uint2 v = make_uint2(0, 0);
                    if (n < c1 && r < p.rank) v = __ldg(reinterpret_cast<const uint2*>(w + static_cast<size_t>(n) * p.rank + r));
                    b[j][0] = v.x;
                    b[j][1] = v.y;
                }
            } else {
                uint4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = (r < p.rank && col + 8 * (c >> 1) < c1)
                               ? __ldg(reinterpret_cast<const uint4*>(w + static_cast<size_t>(r + i) * p.cols + col + 8 * (c >> 1)))
                               : zero;
                const unsigned sel = (c & 1) ? 0x7632u : 0x5410u;
                b[0][0] = prmt(v[0].x, v[1].x, sel); b[0][1] = prmt(v[2].x, v[3].x, sel);
                b[1][0] = prmt(v[0].y, v[1].y, sel); b[1][1] = prmt(v[2].y, v[3].y, sel);
                b[2][0] = prmt(v[0].z, v[1].z, sel); b[2][1] = prmt(v[2].z, v[3].z, sel);
                b[3][0] = prmt(v[0].w, v[1].w, sel); b[3][1] = prmt(v[2].w, v[3].w, sel);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (m >= mt) break;
                const uint4 h = s_w[2 * (m * ks + k) * 32 + lane], l = s_w[(2 * (m * ks + k) + 1) * 32 + lane];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    lr_mma(acc[m][j], h.x, h.y, h.z, h.w, b[j][0], b[j][1]);
                    lr_mma(acc[m][j], l.x, l.y, l.z, l.w, b[j][0], b[j][1]);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = 16 * m + 8 * h + c;
                if (t >= tile.len || !col_on) continue;
                const unsigned bw[4] = {base[m][h].x, base[m][h].y, base[m][h].z, base[m][h].w};
                unsigned o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = lr_pack(lr_lo(bw[j]) + acc[m][j][2 * h], lr_hi(bw[j]) + acc[m][j][2 * h + 1]);
                *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(s_tok[t]) * p.cols + col + 8 * q) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
    }
}

__host__ __device__ constexpr size_t lr_up_smem(int rank) { return size_t{4} * ((rank + 15) / 16) * 2 * 32 * 16; }

// ------------------------------------------------------------------ backward: the factors in two bf16 parts
struct LrSplitParams {
    const int32_t* head;
    const int32_t* order;
    const int32_t* slots;
    const float* u;      // [tokens][rank]
    const float* part;   // [splits][tokens][rank]: B^T gy
    const float* scale;
    uint16_t* parts;     // out: s u high, low, v high, low, each [tokens][rank] in the grouped order
    int32_t tokens, rank, splits;
};

__global__ void __launch_bounds__(256) k_lr_split(const __grid_constant__ LrSplitParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int quads = p.rank >> 2;
    const size_t all = static_cast<size_t>(p.tokens) * p.rank;
    for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < static_cast<size_t>(p.head[2]) * quads;
         i += static_cast<size_t>(gridDim.x) * 256) {
        const int at = static_cast<int>(i / quads), r = 4 * static_cast<int>(i - static_cast<size_t>(at) * quads);
        const int t = p.order[at];
        const float s = __ldg(p.scale + __ldg(p.slots + t));
        const size_t src = static_cast<size_t>(t) * p.rank + r, dst = static_cast<size_t>(at) * p.rank + r;
        const float4 u = *reinterpret_cast<const float4*>(p.u + src);
        float4 v = *reinterpret_cast<const float4*>(p.part + src);
        for (int k = 1; k < p.splits; ++k) {
            const float4 g = *reinterpret_cast<const float4*>(p.part + k * all + src);
            v.x += g.x; v.y += g.y; v.z += g.z; v.w += g.w;
        }
        uint2 h, l;
        lr_split2(s * u.x, s * u.y, h.x, l.x);
        lr_split2(s * u.z, s * u.w, h.y, l.y);
        *reinterpret_cast<uint2*>(p.parts + dst) = h;
        *reinterpret_cast<uint2*>(p.parts + all + dst) = l;
        lr_split2(s * v.x, s * v.y, h.x, l.x);
        lr_split2(s * v.z, s * v.w, h.y, l.y);
        *reinterpret_cast<uint2*>(p.parts + 2 * all + dst) = h;
        *reinterpret_cast<uint2*>(p.parts + 3 * all + dst) = l;
    }
}

// ------------------------------------------------------------------ backward: sums over tokens
struct LrGradParams {
    const int32_t* head;
    const int32_t* order;
    const LrTile* units;
    const int32_t* unit_base;
    const uint16_t* gy;     // [tokens][rows]
    const uint16_t* x;      // [tokens][cols]
    const uint16_t* parts;  // k_lr_split's
    float* part;            // [partial sum][rows][rank], then its [rank][cols]
    uint16_t* grad_b;       // [n][rows][rank]
    uint16_t* grad_a;       // [n][rank][cols]
    int32_t tokens, rows, cols, rank, n;
    int32_t row_ctas;       // CTAs along the rows of B; the rest take the columns of A
};

// NT: 8-wide tiles of the rank
template <int NT>
__global__ void __launch_bounds__(kLrGradThreads) k_lr_grad(const __grid_constant__ LrGradParams p) {
    constexpr int WROW = NT * 16 + 16;                 // bytes of a row of w, padded against bank conflicts
    constexpr int ZBYTES = 64 * kLrGradCols * 2, WBYTES = 64 * WROW, STAGE = ZBYTES + 2 * WBYTES;
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q = lane & 3, c = lane >> 2;
    pdl_wait();
    pdl_launch_dependents();
    if (static_cast<int>(blockIdx.x) >= p.head[1]) return;
    const LrTile unit = p.units[blockIdx.x];
    const bool is_b = static_cast<int>(blockIdx.y) < p.row_ctas;
    const int width = is_b ? p.rows : p.cols;
    const int c0 = (is_b ? static_cast<int>(blockIdx.y) : static_cast<int>(blockIdx.y) - p.row_ctas) * kLrGradCols;
    const uint16_t* z = is_b ? p.gy : p.x;
    const size_t all = static_cast<size_t>(p.tokens) * p.rank;
    const uint16_t* wh = p.parts + (is_b ? 0 : 2 * all);
    const uint32_t base = smem_addr(smem);

    // 64 tokens: z [64][256] (16-byte pieces xored with the row against bank conflicts), w high and low [64][rank]
    auto stage = [&](int t0, int buf) {
        const uint32_t d = base + buf * STAGE;
        const int piece = tid & 31;
        const bool col_on = c0 + 8 * piece < width;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = (tid >> 5) + 8 * i;
            const bool on = col_on && t0 + row < unit.len;
            const uint16_t* src = z;
            if (on) src = z + static_cast<size_t>(p.order[unit.first + t0 + row]) * width + c0 + 8 * piece;
            cp_async16_or_zero(d + row * (kLrGradCols * 2) + 16 * (piece ^ (row & 7)), src, on);
        }
        for (int i = tid; i < 2 * 64 * NT; i += kLrGradThreads) {
            const int half = i / (64 * NT), j = i - half * 64 * NT, row = j / NT, pc = j - row * NT;
            const bool on = t0 + row < unit.len && 8 * pc < p.rank;
            const uint16_t* src = wh;
            if (on) src = wh + half * all + static_cast<size_t>(unit.first + t0 + row) * p.rank + 8 * pc;
            cp_async16_or_zero(d + ZBYTES + half * WBYTES + row * WROW + 16 * pc, src, on);
        }
        cp_async_commit();
    };

    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
    stage(0, 0);
    int buf = 0;
    for (int t0 = 0; t0 < unit.len; t0 += 64, buf ^= 1) {
        cp_async_wait<0>();
        __syncthreads();  // this stage is there, and the other one is read
        if (t0 + 64 < unit.len) stage(t0 + 64, buf ^ 1);
        const uint32_t zs = base + buf * STAGE, ws = zs + ZBYTES;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            unsigned a[2][4];
            const int row = 16 * k + 8 * (lane >> 4) + (lane & 7);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int piece = 4 * warp + 2 * m + ((lane >> 3) & 1);
                ldsm_t4(a[m], zs + row * (kLrGradCols * 2) + 16 * (piece ^ (row & 7)));
            }
            const int wrow = 16 * k + 8 * ((lane >> 3) & 1) + (lane & 7);
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    unsigned b[4];
                    ldsm_t4(b, ws + half * WBYTES + wrow * WROW + 16 * (j + (lane >> 4)));
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        lr_mma(acc[m][j], a[m][0], a[m][1], a[m][2], a[m][3], b[0], b[1]);
                        lr_mma(acc[m][j + 1], a[m][0], a[m][1], a[m][2], a[m][3], b[2], b[3]);
                    }
                }
            }
        }
    }
    const bool whole = unit.pad < 0;  // the adapter's only unit
    float* part = whole ? nullptr : p.part + (static_cast<size_t>(unit.pad) * (p.rows + p.cols) + (is_b ? 0 : p.rows)) * p.rank;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int col = c0 + 32 * warp + 16 * m + 8 * h + c;
            if (col >= width) continue;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int r = 8 * j + 2 * q;
                if (r >= p.rank) continue;
                const float lo = acc[m][j][2 * h], hi = acc[m][j][2 * h + 1];
                if (!whole && is_b) {
                    *reinterpret_cast<float2*>(part + static_cast<size_t>(col) * p.rank + r) = make_float2(lo, hi);
                } else if (!whole) {
                    part[static_cast<size_t>(r) * p.cols + col] = lo;
                    part[static_cast<size_t>(r + 1) * p.cols + col] = hi;
                } else if (is_b) {
                    *reinterpret_cast<unsigned*>(p.grad_b + (static_cast<size_t>(unit.slot) * p.rows + col) * p.rank + r) = lr_pack(lo, hi);
                } else {
                    uint16_t* d = p.grad_a + (static_cast<size_t>(unit.slot) * p.rank + r) * p.cols + col;
                    const unsigned v = lr_pack(lo, hi);
                    d[0] = static_cast<uint16_t>(v & 0xFFFFu);
                    d[p.cols] = static_cast<uint16_t>(v >> 16);
                }
            }
        }
}

__host__ __device__ constexpr size_t lr_grad_smem(int nt) { return 2 * (size_t{64} * kLrGradCols * 2 + 2 * 64 * (size_t(nt) * 16 + 16)); }

// Adapters of several units: their sums in order; adapters without a token: zeros.
__global__ void __launch_bounds__(256) k_lr_join(const __grid_constant__ LrGradParams p) {
    pdl_wait();
    const int slot = static_cast<int>(blockIdx.y);
    const int u0 = p.unit_base[slot], nu = p.unit_base[p.n + slot];
    if (nu == 1) return;
    const size_t each = static_cast<size_t>(p.rows + p.cols) * p.rank;
    const int quads_b = p.rows * (p.rank >> 2), quads = quads_b + p.cols * (p.rank >> 2);
    for (int i = static_cast<int>(blockIdx.x) * 256 + threadIdx.x; i < quads; i += static_cast<int>(gridDim.x) * 256) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4* src = reinterpret_cast<const float4*>(p.part + u0 * each) + i;
#pragma unroll 4
        for (int k = 0; k < nu; ++k) {
            const float4 g = __ldcs(src + k * (each >> 2));
            s.x += g.x; s.y += g.y; s.z += g.z; s.w += g.w;
        }
        uint2* d = i < quads_b ? reinterpret_cast<uint2*>(p.grad_b) + static_cast<size_t>(slot) * quads_b + i
                               : reinterpret_cast<uint2*>(p.grad_a) + static_cast<size_t>(slot) * (quads - quads_b) + (i - quads_b);
        *d = make_uint2(lr_pack(s.x, s.y), lr_pack(s.z, s.w));
    }
}

}  // namespace e8q

// Low-rank adapters of many requests beside a shared projection, forward
// and backward.  Token t has the adapter a = slots[t] (none: outside 0..n-1):
//
//   u_t = A_a x_t,   y_t = base_t + s_a B_a u_t
//   v_t = s_a B_a^T gy_t,   gx_t = gx0_t + A_a^T v_t
//   gA_a = sum_t v_t x_t^T,   gB_a = sum_t gy_t (s_a u_t)^T
//
// The tokens are grouped by adapter first (k_lr_plan; in small batches each
// CTA groups for itself); everything after it works on tiles of up to 64 (8
// in small batches) tokens of one adapter:
//
//   k_lr_down   p = W z, a long sum over the columns of z and a short result
//               (u from x and A; v / s from gy and B): tensor cores with the
//               rank as M and the tokens as N.  The columns are split over the
//               warps of a CTA and over CTAs; partial sums are added in a fixed
//               order;
//   k_lr_up     out = base + W w, a short sum and a long result (y from u and
//               B; gx from v and A): tokens as M, columns as N;
//   k_lr_split  (backward) w = s u and v as bf16 high + low parts;
//   k_lr_grad   sums over tokens: gB from gy and s u, gA from x and v, both in
//               one launch.  z^T and w come from shared memory by transposing
//               ldmatrix; long token ranges are split into units whose partial
//               sums k_lr_join adds in order.
//
// The fp32 factors u, v enter the tensor cores as a bf16 high part plus a
// bf16 low part (two MMAs, about 16 bits), so that the only rounding to bf16
// that counts is the result's (measured error 1.7e-3, the plain rounding's; 0.2 %
// of the results are the bf16 neighbour of the exact value's rounding, 0.05 %
// with the factors in fp32).
//
// Measured on one B200 (kernel alone, cold L2; bytes of the token matrices):
//   k_lr_down   4,096 tokens, rank 32, 4096 columns: 13 us (34 MB); rank 16,
//               14336 columns from B: 24 us (117 MB, 4.9 TB/s); 64 tokens of 64
//               adapters, 14336 columns: 10 us (29 MB of A)
//   k_lr_up     4,096 tokens, rank 32, 14336 columns: 68 us (235 MB, 3.5 TB/s);
//               rank 128: 166 us; 8,192 tokens, rank 64, 14336 columns from A:
//               123 us (470 MB, 3.8 TB/s); 64 tokens of 64 adapters, 4096
//               columns: 8 us
//   k_lr_grad   4,096 tokens, rank 16, 18,432 columns: 41 us (151 MB, 3.7 TB/s);
//               rank 128: 167 us; 8,192 tokens, rank 64: 118 us (302 MB, tensor
//               pipe 58 %)
//   k_lr_plan   9 us at 4,096 tokens, k_lr_split and k_lr_join 5 us each
// Long kernels of low ranks are bound by the waits of their pipelines (issue
// 0.4 to 0.45 a cycle, tensor pipe 14 to 22 %).  From rank 64 on the token sums
// wait for the tensor pipe first (58 %), the up kernel for its own steps and
// the pipe alike (43 %).  Small batches are bound by the latency of two
// dependent kernels.  All are warp-level MMAs fed from registers; a tcgen05
// form has not been tried.
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
// Rank 16, 4096 x 4096, each CTA grouping for itself at 128 tokens, and
// k_lr_plan with tiles of 64 at 129: 11.0 and 17.6 us on one adapter, 11.2 and
// 18.9 on 8, 11.5 and 20.5 on 64.  The times cross somewhere above 128, which
// is what the grouping's shared arrays (one thread a token) hold.
constexpr int kLrSmallTokens = 128;
// Most tokens a unit of k_lr_grad sums in its MMA accumulators (256 MMAs on
// each, of high and low parts).  The tensor cores cut off what lies below an
// accumulator's last bit, so a sum of one sign falls short by about half a
// step, 2^-24, an MMA.  65,536 tokens in one accumulator (8,192 MMAs) moved
// 4.8 % of the bf16 results to another value than the exact sum's; 256 MMAs
// lose no more than 2^-15.  The partial sums of longer runs leave take at
// most 4 rank / 2,048 of the token matrices' bytes; units of any length
// measured 1.5 % faster at 16,384 tokens of rank 64 (277 and 281 us), 4 %
// at 65,536 of rank 16 on 8 adapters (718 and 745 us).
constexpr int kLrUnitMax = 2048;
constexpr int kLrFewThreads = 256;
constexpr int kLrDownThreads = 256;

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
    extern __shared__ __align__(128) unsigned char smem[];
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
    auto bins = [&](int t, int (&bin)[8]) {  // of 256 tokens; past the range: nb, matched only by its like
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = t + 32 * i + lane;
            bin[i] = at < t1 ? __ldg(p.slots + at) : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = t + 32 * i + lane;
            bin[i] = at >= t1 ? nb : (bin[i] >= 0 && bin[i] < p.n) ? bin[i] : p.n;
        }
    };
    for (int t = t0; t < t1; t += 256) {
        int bin[8];
        bins(t, bin);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (t + 32 * i >= t1) break;
            const unsigned peers = __match_any_sync(0xFFFFFFFFu, bin[i]);
            if (bin[i] < nb && (peers & below) == 0) mine[bin[i]] = static_cast<uint16_t>(mine[bin[i]] + __popc(peers));
            __syncwarp();
        }
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
    for (int t = t0; t < t1; t += 256) {
        int bin[8];
        bins(t, bin);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (t + 32 * i >= t1) break;
            const unsigned peers = __match_any_sync(0xFFFFFFFFu, bin[i]);
            const int before = bin[i] < nb ? mine[bin[i]] : 0;
            __syncwarp();
            if (bin[i] < nb) {
                p.order[s_tok[bin[i]] + before + __popc(peers & below)] = t + 32 * i + lane;
                if ((peers & below) == 0) mine[bin[i]] = static_cast<uint16_t>(before + __popc(peers));
            }
            __syncwarp();
        }
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
__device__ __forceinline__ void ldsm_4(unsigned (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
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

// Small batches (up to kLrSmallTokens tokens): every CTA finds its own tile of
// up to 8 tokens, which costs less than a launch that would tell it.  A tile
// begins at each token that has a multiple of 8 tokens of its adapter before
// it; tiles are numbered by their first token.
struct LrSmall {
    int slot[kLrSmallTokens];  // n: no adapter
    int before[kLrSmallTokens];
    int warp_heads[kLrSmallTokens / 32];
    int head;
    int tok[kLrSmallTile];
};

__device__ __forceinline__ LrTile lr_find_tile(LrSmall& s, const int32_t* slots, int tokens, int n, int index) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int mine = -1, before = 0;
    if (tid < kLrSmallTokens) {
        if (tid < tokens) {
            mine = __ldg(slots + tid);
            if (mine < 0 || mine >= n) mine = n;
        }
        s.slot[tid] = mine;
    }
    if (tid == 0) s.head = -1;
    __syncthreads();
    bool head = false;
    if (tid < kLrSmallTokens) {
        for (int j = 0; j < min(tokens, 32 * warp); ++j) before += s.slot[j] == mine;
        before += __popc(__match_any_sync(0xFFFFFFFFu, mine) & ((1u << lane) - 1u));
        s.before[tid] = before;
        head = tid < tokens && (before & (kLrSmallTile - 1)) == 0;
        const unsigned heads = __ballot_sync(0xFFFFFFFFu, head);
        if (lane == 0) s.warp_heads[warp] = __popc(heads);
        before = __popc(heads & ((1u << lane) - 1u));  // heads before this token in its warp
    }
    __syncthreads();
    if (head) {
        for (int w = 0; w < warp; ++w) before += s.warp_heads[w];
        if (before == index) s.head = tid;
    }
    __syncthreads();
    LrTile t{0, 0, -2, 0};
    if (s.head < 0) return t;  // no such tile
    const int h = s.head, first = s.before[h], slot = s.slot[h];
    if (tid < kLrSmallTokens && mine == slot && s.before[tid] >= first && s.before[tid] < first + kLrSmallTile)
        s.tok[s.before[tid] - first] = tid;
    t.len = __syncthreads_count(tid < kLrSmallTokens && mine == slot && s.before[tid] >= first && s.before[tid] < first + kLrSmallTile);
    t.slot = slot == n ? -1 : slot;
    return t;
}

// ------------------------------------------------------------------ p = W z
struct LrDownParams {
    const int32_t* head;
    const int32_t* order;
    const LrTile* tiles;
    const int32_t* slots;
    const uint16_t* z;  // [tokens][cols]
    const uint16_t* w;  // [n][rank][cols], or [n][cols][rank] (kTrans)
    float* part;        // [split][tokens][rank]
    int32_t tokens, cols, rank, n;
    int32_t per;        // columns a CTA, a multiple of 256
};

// Column n of a 32-column block -> row of the staged block, such that the
// eight rows of each 8x8 matrix of the MMA's A operand follow one another.
__device__ __forceinline__ int lr_stage_row(int n) { return 16 * ((n >> 2) & 1) + 8 * ((n >> 1) & 1) + 2 * (n >> 3) + (n & 1); }

// Tiles of up to 8 tokens: 8 warps along the columns, z and the weights
// straight from global memory in 16-byte loads.  MT: 16-row tiles of the
// rank (4 at most: higher ranks in gridDim.z parts).
template <int MT, bool kTrans>
__global__ void __launch_bounds__(kLrFewThreads) k_lr_down_few(const __grid_constant__ LrDownParams p) {
    constexpr int KW = 8, STEP = 32 * KW;   // columns a round
    constexpr int ROW = MT * 16 * 2 + 16;   // bytes of a staged row (kTrans), padded against bank conflicts
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ LrSmall s_small;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q = lane & 3, c = lane >> 2;
    pdl_wait();
    pdl_launch_dependents();
    const LrTile tile = lr_find_tile(s_small, p.slots, p.tokens, p.n, blockIdx.x);
    if (tile.slot < 0) return;
    const int k0 = static_cast<int>(blockIdx.y) * p.per, k1 = min(p.cols, k0 + p.per);
    const int r0 = static_cast<int>(blockIdx.z) * 64;
    const uint16_t* w = p.w + static_cast<size_t>(tile.slot) * p.rank * p.cols;
    const bool on = c < tile.len;
    const uint16_t* zr = p.z + static_cast<size_t>(on ? s_small.tok[c] : 0) * p.cols;
    float acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][e] = 0.f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto load_z = [&](int kb) {
        const int k = kb + 8 * q;
        return (on && k < k1) ? __ldg(reinterpret_cast<const uint4*>(zr + k)) : zero;
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
        uint4 x, v[MT][2];
        int kb = k0 + 32 * warp;
        x = load_z(kb);
        load_w(kb, v);
        for (; kb < k1; kb += STEP) {
            uint4 vn[MT][2];
            const uint4 xn = load_z(kb + STEP);
            load_w(kb + STEP, vn);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                lr_mma(acc[m], v[m][0].x, v[m][1].x, v[m][0].y, v[m][1].y, x.x, x.y);
                lr_mma(acc[m], v[m][0].z, v[m][1].z, v[m][0].w, v[m][1].w, x.z, x.w);
            }
            x = xn;
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
            for (int i = tid; i < STEP * CH; i += kLrFewThreads) {
                const int n = i / CH, piece = i - n * CH, k = kb + n, r = r0 + 8 * piece;
                const uint32_t dst = base + (buf * STEP + (n & ~31) + lr_stage_row(n & 31)) * ROW + 16 * piece;
                const bool in = k < k1 && r < p.rank;
                cp_async16_or_zero(dst, in ? w + static_cast<size_t>(k) * p.rank + r : w, in);
            }
            cp_async_commit();
        };
        stage(k0, 0);
        uint4 x = load_z(k0 + 32 * warp);
        int buf = 0;
        for (int kr = k0; kr < k1; kr += STEP, buf ^= 1) {
            const uint4 xn = load_z(kr + STEP + 32 * warp);
            cp_async_wait<0>();
            __syncthreads();  // the round's weights are there, and the other buffer is read
            if (kr + STEP < k1) stage(kr + STEP, buf ^ 1);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    unsigned a[4];
                    ldsm_t4(a, base + (buf * STEP + 32 * warp + 16 * h + 8 * (lane >> 4) + (lane & 7)) * ROW + 32 * m +
                                   16 * ((lane >> 3) & 1));
                    lr_mma(acc[m], a[0], a[1], a[2], a[3], h ? x.z : x.x, h ? x.w : x.y);
                }
            x = xn;
        }
        __syncthreads();  // the staging memory becomes the reduction's
    }

    // the warps' sums, in order
    float* red = reinterpret_cast<float*>(smem);
    constexpr int V = MT * 4;
    if (warp > 0)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[((warp - 1) * V + 4 * m + e) * 32 + lane] = acc[m][e];
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int k = 0; k < KW - 1; ++k)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][e] += red[(k * V + 4 * m + e) * 32 + lane];
    float* out = p.part + static_cast<size_t>(blockIdx.y) * p.tokens * p.rank;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int t = 2 * q + e;
        if (t >= tile.len) continue;
        float* row = out + static_cast<size_t>(s_small.tok[t]) * p.rank;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = r0 + 16 * m + 8 * h + c;
                if (r < p.rank) row[r] = acc[m][2 * h + e];
            }
    }
}

__host__ __device__ constexpr size_t lr_down_few_smem(int mt, bool trans) {
    const size_t red = size_t{7} * mt * 4 * 32 * 4;
    const size_t stage = trans ? size_t{2} * 256 * (static_cast<size_t>(mt) * 32 + 16) : 0;
    return red > stage ? red : stage;
}

// Tiles of up to 64 tokens: z [64][128 columns] and the weights of the same
// columns come through shared memory, three or four rounds deep (two CTAs an
// SM: a round's compute is short, and the loads of the next ones have to be
// out).  8 warps: 4 along the round's columns, 2 along the tokens.
constexpr int kLrRound = 128;
__host__ __device__ constexpr int lr_down_stages(int mt) { return mt == 4 ? 3 : 4; }

template <int MT, bool kTrans>
__global__ void __launch_bounds__(kLrDownThreads) k_lr_down(const __grid_constant__ LrDownParams p) {
    constexpr int NT = 4, kStages = lr_down_stages(MT);
    constexpr int ZB = kLrTile * kLrRound * 2;                           // 16-byte pieces xored with the row
    constexpr int ROW = MT * 16 * 2 + 16;                                // staged row (kTrans), padded
    constexpr int WB = kTrans ? kLrRound * ROW : MT * 16 * kLrRound * 2;  // (else) pieces xored with the row
    constexpr int STAGE = ZB + WB;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int s_tok[kLrTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q = lane & 3, c = lane >> 2;
    const int kq = warp & 3, th = warp >> 2;
    pdl_wait();
    pdl_launch_dependents();
    if (static_cast<int>(blockIdx.x) >= p.head[0]) return;
    const LrTile tile = p.tiles[blockIdx.x];
    if (tile.slot < 0) return;
    const int k0 = static_cast<int>(blockIdx.y) * p.per, k1 = min(p.cols, k0 + p.per);
    const int r0 = static_cast<int>(blockIdx.z) * 64;
    const uint16_t* w = p.w + static_cast<size_t>(tile.slot) * p.rank * p.cols;
    if (tid < tile.len) s_tok[tid] = p.order[tile.first + tid];
    __syncthreads();
    const uint32_t base = smem_addr(smem);
    // this thread's pieces of a round of z: rows tid / 16 + 16 i, piece tid % 16
    const uint16_t* zr[4];
    bool on[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (tid >> 4) + 16 * i;
        on[i] = row < tile.len;
        zr[i] = p.z + static_cast<size_t>(on[i] ? s_tok[row] : 0) * p.cols + 8 * (tid & 15);
    }
    auto stage = [&](int kb, int buf) {
        const uint32_t d = base + buf * STAGE;
        if (kb < k1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (tid >> 4) + 16 * i;
                const bool in = on[i] && kb + 8 * (tid & 15) < k1;
                cp_async16_or_zero(d + row * (kLrRound * 2) + 16 * ((tid & 15) ^ (row & 7)), in ? zr[i] + kb : p.z, in);
            }
            if (kTrans) {
                constexpr int CH = 2 * MT;
#pragma unroll
                for (int i = tid; i < kLrRound * CH; i += kLrDownThreads) {
                    const int n = i / CH, piece = i - n * CH, k = kb + n, r = r0 + 8 * piece;
                    const bool in = k < k1 && r < p.rank;
                    cp_async16_or_zero(d + ZB + n * ROW + 16 * piece, in ? w + static_cast<size_t>(k) * p.rank + r : w, in);
                }
            } else {
#pragma unroll
                for (int i = tid; i < MT * 16 * 16; i += kLrDownThreads) {
                    const int row = i >> 4, piece = i & 15, k = kb + 8 * piece;
                    const bool in = r0 + row < p.rank && k < k1;
                    cp_async16_or_zero(d + ZB + row * (kLrRound * 2) + 16 * (piece ^ (row & 7)),
                                       in ? w + static_cast<size_t>(r0 + row) * p.cols + k : w, in);
                }
            }
        }
        cp_async_commit();
    };
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][i][e] = 0.f;
    const int live = tile.len - 32 * th;  // tokens of this warp (maybe none)
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) stage(k0 + i * kLrRound, i);
    int buf = 0;
    for (int kb = k0; kb < k1; kb += kLrRound) {
        cp_async_wait<kStages - 2>();
        __syncthreads();  // this round is there, and the stage read last is free
        stage(kb + (kStages - 1) * kLrRound, buf == 0 ? kStages - 1 : buf - 1);
        const uint32_t zs = base + buf * STAGE, ws = zs + ZB;
        buf = buf + 1 == kStages ? 0 : buf + 1;
        if (live > 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 16 columns each: pieces 4 kq + 2 h, + 1
                unsigned a[MT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (kTrans) {
                        ldsm_t4(a[m], ws + (32 * kq + 16 * h + 8 * (lane >> 4) + (lane & 7)) * ROW + 32 * m + 16 * ((lane >> 3) & 1));
                    } else {
                        const int row = 16 * m + (lane & 15), piece = 4 * kq + 2 * h + (lane >> 4);
                        ldsm_4(a[m], ws + row * (kLrRound * 2) + 16 * (piece ^ (row & 7)));
                    }
                }
#pragma unroll
                for (int i = 0; i < NT; i += 2) {
                    if (8 * i >= live) break;
                    unsigned b[4];
                    const int row = 32 * th + 8 * i + 8 * (lane >> 4) + (lane & 7), piece = 4 * kq + 2 * h + ((lane >> 3) & 1);
                    ldsm_4(b, zs + row * (kLrRound * 2) + 16 * (piece ^ (row & 7)));
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        lr_mma(acc[m][i], a[m][0], a[m][1], a[m][2], a[m][3], b[0], b[1]);
                        lr_mma(acc[m][i + 1], a[m][0], a[m][1], a[m][2], a[m][3], b[2], b[3]);
                    }
                }
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();  // the stages become the reduction's

    // the column warps' sums, in order
    float* red = reinterpret_cast<float*>(smem);
    constexpr int V = MT * NT * 4;
    if (kq > 0) {
        float* d = red + ((kq - 1) * 2 + th) * V * 32 + lane;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[((m * NT + i) * 4 + e) * 32] = acc[m][i][e];
    }
    __syncthreads();
    if (kq > 0 || live <= 0) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const float* d = red + (k * 2 + th) * V * 32 + lane;
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
            float* row = out + static_cast<size_t>(s_tok[t]) * p.rank;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = r0 + 16 * m + 8 * h + c;
                    if (r < p.rank) row[r] = acc[m][i][2 * h + e];
                }
        }
}

__host__ __device__ constexpr size_t lr_down_smem(int mt, bool trans) {
    const size_t red = size_t{3} * 2 * mt * 16 * 32 * 4;
    const size_t stages = lr_down_stages(mt) * (size_t{kLrTile} * kLrRound * 2 + (trans ? kLrRound * (static_cast<size_t>(mt) * 32 + 16)
                                                                              : static_cast<size_t>(mt) * 16 * kLrRound * 2));
    return red > stages ? red : stages;
}

// ------------------------------------------------------------------ out = base + W w
struct LrUpParams {
    const int32_t* head;
    const int32_t* order;
    const LrTile* tiles;
    const int32_t* slots;
    const float* part;      // [splits][tokens][rank]
    const float* scale;
    const uint16_t* w;      // [n][cols][rank], or [n][rank][cols] (kTrans)
    const uint16_t* base;   // [tokens][cols] or NULL
    uint16_t* out;          // [tokens][cols]
    float* sum;             // [tokens][rank]: the sum of the parts, or NULL
    int32_t tokens, cols, rank, n;
    int32_t splits;
};

// base [tokens][64 columns] and the weights of the same columns come through
// shared memory, three steps deep; the factors w stay in registers.  TOK: 8
// tokens (small batches; four warps along the columns), or 64
// (four warps along the tokens).  Small CTAs, four an SM, because a step is a
// chain of short waits (copies, barrier, ldmatrix, MMA, store) that only other
// CTAs fill: 256 threads on 128 columns measured 4 % slower, tiles of 128
// tokens 5 to 20 %.  KS: 16-rank steps.
constexpr int kLrUpStages = 3, kLrUpThreads = 128, kLrUpCols = 64;

template <int KS, int TOK, bool kTrans>
__global__ void __launch_bounds__(kLrUpThreads) k_lr_up(const __grid_constant__ LrUpParams p) {
    constexpr bool kSmall = TOK == kLrSmallTile;
    constexpr int kThreads = kLrUpThreads, kStages = kLrUpStages, COLS = kLrUpCols;
    constexpr int NT = kSmall ? 2 : 8;              // 8-column tiles a warp
    constexpr int ROWS = TOK;
    constexpr int BB = ROWS * COLS * 2;        // 16-byte pieces xored with the row
    constexpr int WROW = kTrans ? COLS * 2 : KS * 32 + 16;  // (kTrans) xored with the row, else padded
    constexpr int WB = (kTrans ? KS * 16 : COLS) * WROW;
    constexpr int STAGE = BB + WB;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ LrSmall s_small;
    __shared__ int s_rows[kLrTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q = lane & 3, c = lane >> 2;
    LrTile tile;
    if (kSmall) {
        // Grouping and the first stages read the caller's inputs only.  The first kernel of a call starts after
        // everything before it, so this may go ahead of the wait for the previous kernel.
        tile = lr_find_tile(s_small, p.slots, p.tokens, p.n, blockIdx.x);
        if (tile.len == 0) {
            pdl_wait();
            return;
        }
    } else {
        pdl_wait();
        pdl_launch_dependents();
        if (static_cast<int>(blockIdx.x) >= p.head[0]) return;
        tile = p.tiles[blockIdx.x];
        if (tid < tile.len) s_rows[tid] = p.order[tile.first + tid];
        __syncthreads();
    }
    const int* s_tok = kSmall ? s_small.tok : s_rows;
    // this CTA's steps: every gridDim.y-th, so that the CTAs of a tile work on neighbouring columns of its rows
    const int c0 = static_cast<int>(blockIdx.y) * COLS, c1 = p.cols, next = static_cast<int>(gridDim.y) * COLS;
    const uint16_t* w = p.w + static_cast<size_t>(max(tile.slot, 0)) * p.rank * p.cols;
    const uint32_t sbase = smem_addr(smem);
    const int m0 = kSmall ? 0 : 16 * warp, j0 = kSmall ? 2 * warp : 0;  // the warp's tokens and column tiles
    // this thread's rows of base and out: kSmall one, of 64 threads; else four of its warp's 16
    constexpr int OWN = kSmall ? 1 : 4;
    const int row0 = kSmall ? (tid >> 3) : m0 + (lane >> 3), piece = tid & 7;
    long long off[OWN];  // their first element in this thread's column piece; negative: none
    uint32_t own[OWN];   // their place in a stage
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int row = row0 + 4 * i;
        off[i] = row < tile.len ? static_cast<long long>(s_tok[row]) * p.cols + 8 * piece : -1;
        own[i] = row * (COLS * 2) + 16 * (piece ^ (row & 7));
    }
    auto stage = [&](int col, int buf) {
        const uint32_t d = sbase + buf * STAGE;
        if (col < c1) {
            const int k = col + 8 * piece;
            if (p.base && (!kSmall || tid < 8 * ROWS))
#pragma unroll
                for (int i = 0; i < OWN; ++i) {
                    const bool in = off[i] >= 0 && k < c1;
                    cp_async16_or_zero(d + own[i], in ? p.base + off[i] + col : p.base, in);
                }
            if (kTrans) {
#pragma unroll
                for (int i = tid; i < KS * 16 * (COLS / 8); i += kThreads) {
                    const int row = i / (COLS / 8), pc = i % (COLS / 8);
                    const bool in = row < p.rank && col + 8 * pc < c1;
                    cp_async16_or_zero(d + BB + row * WROW + 16 * (pc ^ (row & 7)),
                                       in ? w + static_cast<size_t>(row) * p.cols + col + 8 * pc : w, in);
                }
            } else {
#pragma unroll
                for (int i = tid; i < COLS * 2 * KS; i += kThreads) {
                    const int n = i / (2 * KS), pc = i - n * 2 * KS;
                    const bool in = col + n < c1 && 8 * pc < p.rank;
                    cp_async16_or_zero(d + BB + n * WROW + 16 * pc, in ? w + static_cast<size_t>(col + n) * p.rank + 8 * pc : w, in);
                }
            }
        }
        cp_async_commit();
    };
    if (tile.slot >= 0)
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) stage(c0 + i * next, i);
    if (kSmall) {
        pdl_wait();
        pdl_launch_dependents();
    }
    if (tile.slot < 0) {  // tokens without an adapter
        if (p.sum && blockIdx.y == 0)
            for (int i = tid; i < tile.len * p.rank; i += kThreads)
                p.sum[static_cast<size_t>(s_tok[i / p.rank]) * p.rank + i % p.rank] = 0.f;
        if (p.base == p.out) return;
        // copied, the loads of two steps out before their stores
        constexpr int AT_ONCE = kThreads / (COLS / 8), R = (ROWS + AT_ONCE - 1) / AT_ONCE;
        const int mine = 8 * (tid % (COLS / 8)), first = tid / (COLS / 8);
        for (int col = c0 + mine; col < c1; col += 2 * next) {
            uint4 v[2][R];
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int row = first + AT_ONCE * i, k = col + d * next;
                    v[d][i] = make_uint4(0, 0, 0, 0);
                    if (p.base && row < tile.len && k < c1)
                        v[d][i] = *reinterpret_cast<const uint4*>(p.base + static_cast<size_t>(s_tok[row]) * p.cols + k);
                }
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int row = first + AT_ONCE * i, k = col + d * next;
                    if (row < tile.len && k < c1)
                        *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(s_tok[row]) * p.cols + k) = v[d][i];
                }
        }
        return;
    }

    // A operands: lane (c, q) holds tokens c and c + 8 of the warp's 16, ranks 16 k + 2q, + 1, + 8, + 9
    unsigned hi[KS][4], lo[KS][4];
    const float s = __ldg(p.scale + tile.slot);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = m0 + 8 * (e & 1) + c, r = 16 * k + 8 * (e >> 1) + 2 * q;
            float2 f = make_float2(0.f, 0.f);
            if (t < tile.len && r < p.rank) {
                const size_t at = static_cast<size_t>(s_tok[t]) * p.rank + r;
                f = *reinterpret_cast<const float2*>(p.part + at);
#pragma unroll 4
                for (int i = 1; i < p.splits; ++i) {
                    const float2 g = *reinterpret_cast<const float2*>(p.part + static_cast<size_t>(i) * p.tokens * p.rank + at);
                    f.x += g.x;
                    f.y += g.y;
                }
                if (p.sum && blockIdx.y == 0 && (!kSmall || warp == 0)) *reinterpret_cast<float2*>(p.sum + at) = f;
            }
            lr_split2(s * f.x, s * f.y, hi[k][e], lo[k][e]);
        }

    int buf = 0;
    for (int col = c0; col < c1; col += next) {
        cp_async_wait<kStages - 2>();
        __syncthreads();  // this step is there, and the stage stored last is free
        stage(col + (kStages - 1) * next, buf == 0 ? kStages - 1 : buf - 1);
        const uint32_t bs = sbase + buf * STAGE, ws = bs + BB;
        unsigned char* tile_mem = smem + buf * STAGE;
        unsigned char* mine = tile_mem + (m0 + c) * (COLS * 2) + 4 * q;  // rows m0 + c, + 8 (the same xor)
        buf = buf + 1 == kStages ? 0 : buf + 1;
        if (m0 < tile.len) {
            // the sums begin with base; the result takes its place in the stage
            constexpr int H = kSmall ? 1 : 2;
            float acc[NT][4];
            if (p.base) {
                unsigned b[NT][2];
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int h = 0; h < H; ++h) b[j][h] = *reinterpret_cast<const unsigned*>(mine + h * 8 * (COLS * 2) + 16 * ((j0 + j) ^ c));
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    acc[j][0] = lr_lo(b[j][0]);
                    acc[j][1] = lr_hi(b[j][0]);
                    acc[j][2] = kSmall ? 0.f : lr_lo(b[j][H - 1]);
                    acc[j][3] = kSmall ? 0.f : lr_hi(b[j][H - 1]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                unsigned b[NT / 2][4];  // columns 8 (j0 + 2 i) .. + 15
#pragma unroll
                for (int i = 0; i < NT / 2; ++i) {
                    if (kTrans) {
                        const int row = 16 * k + 8 * ((lane >> 3) & 1) + (lane & 7), pc = j0 + 2 * i + (lane >> 4);
                        ldsm_t4(b[i], ws + row * WROW + 16 * (pc ^ (row & 7)));
                    } else {
                        ldsm_4(b[i], ws + (8 * (j0 + 2 * i) + 8 * (lane >> 4) + (lane & 7)) * WROW + 32 * k + 16 * ((lane >> 3) & 1));
                    }
                }
                // high parts of all tiles, then low parts: MMAs on one accumulator lie NT apart
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    lr_mma(acc[j], hi[k][0], hi[k][1], hi[k][2], hi[k][3], b[j >> 1][2 * (j & 1)], b[j >> 1][2 * (j & 1) + 1]);
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    lr_mma(acc[j], lo[k][0], lo[k][1], lo[k][2], lo[k][3], b[j >> 1][2 * (j & 1)], b[j >> 1][2 * (j & 1) + 1]);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int h = 0; h < H; ++h)
                    *reinterpret_cast<unsigned*>(mine + h * 8 * (COLS * 2) + 16 * ((j0 + j) ^ c)) =
                        lr_pack(acc[j][2 * h], acc[j][2 * h + 1]);
        }
        if (kSmall) __syncthreads();
        else __syncwarp();
        if (!kSmall || tid < 8 * ROWS) {
            uint4 o[OWN];
#pragma unroll
            for (int i = 0; i < OWN; ++i) o[i] = *reinterpret_cast<const uint4*>(tile_mem + own[i]);
#pragma unroll
            for (int i = 0; i < OWN; ++i)
                if (off[i] >= 0 && col + 8 * piece < c1) *reinterpret_cast<uint4*>(p.out + off[i] + col) = o[i];
        }
    }
}

__host__ __device__ constexpr size_t lr_up_smem(int ks, int tok, bool trans) {
    return kLrUpStages * (size_t(tok) * kLrUpCols * 2 +
                          (trans ? size_t(ks) * 16 * kLrUpCols * 2 : size_t(kLrUpCols) * (size_t(ks) * 32 + 16)));
}

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

constexpr int kLrGradCols = 256;  // of a CTA, 32 a warp

// NT: 8-wide tiles of the rank
template <int NT>
__global__ void __launch_bounds__(kLrGradCols) k_lr_grad(const __grid_constant__ LrGradParams p) {
    constexpr int kCols = kLrGradCols;                 // and threads
    constexpr int WROW = NT * 16 + 16;                 // bytes of a row of w, padded against bank conflicts
    constexpr int ZBYTES = 64 * kCols * 2, WBYTES = 64 * WROW, STAGE = ZBYTES + 2 * WBYTES;
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q = lane & 3, c = lane >> 2;
    pdl_wait();
    pdl_launch_dependents();
    if (static_cast<int>(blockIdx.x) >= p.head[1]) return;
    const LrTile unit = p.units[blockIdx.x];
    const bool is_b = static_cast<int>(blockIdx.y) < p.row_ctas;
    const int width = is_b ? p.rows : p.cols;
    const int c0 = (is_b ? static_cast<int>(blockIdx.y) : static_cast<int>(blockIdx.y) - p.row_ctas) * kCols;
    const uint16_t* z = is_b ? p.gy : p.x;
    const size_t all = static_cast<size_t>(p.tokens) * p.rank;
    const uint16_t* wh = p.parts + (is_b ? 0 : 2 * all);
    const uint32_t base = smem_addr(smem);

    // 64 tokens: z [64][kCols] (16-byte pieces xored with the row against bank conflicts), w high and low [64][rank]
    constexpr int PIECES = kCols / 8, ROWS = kCols / PIECES;  // rows copied at once: 8
    const int piece = tid % PIECES, row0 = tid / PIECES;
    const bool col_on = c0 + 8 * piece < width;
    const uint16_t* zc = z + c0 + 8 * piece;
    int tok[64 / ROWS];  // of this thread's rows of the next stage (row0 + 8 i), loaded a stage ahead
    auto tokens = [&](int t0) {
#pragma unroll
        for (int i = 0; i < 64 / ROWS; ++i) {
            const int row = t0 + row0 + ROWS * i;
            tok[i] = row < unit.len ? __ldg(p.order + unit.first + row) : -1;
        }
    };
    auto stage = [&](int t0, int buf) {
        const uint32_t d = base + buf * STAGE;
#pragma unroll
        for (int i = 0; i < 64 / ROWS; ++i) {
            const int row = row0 + ROWS * i;
            const bool on = col_on && tok[i] >= 0;
            cp_async16_or_zero(d + row * (kCols * 2) + 16 * (piece ^ (row & 7)),
                               on ? zc + static_cast<size_t>(tok[i]) * width : z, on);
        }
        tokens(t0 + 64);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = tid; i < 64 * NT; i += kCols) {
                const int row = i / NT, pc = i - row * NT;
                const bool on = t0 + row < unit.len && 8 * pc < p.rank;
                cp_async16_or_zero(d + ZBYTES + half * WBYTES + row * WROW + 16 * pc,
                                   on ? wh + half * all + static_cast<size_t>(unit.first + t0 + row) * p.rank + 8 * pc : wh, on);
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
    tokens(0);
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
                ldsm_t4(a[m], zs + row * (kCols * 2) + 16 * (piece ^ (row & 7)));
            }
            const int wrow = 16 * k + 8 * ((lane >> 3) & 1) + (lane & 7);
#pragma unroll
            for (int half = 0; half < 2; ++half)  // high parts of all tiles, then low parts
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
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

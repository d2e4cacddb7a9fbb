// Chosen rows of an encoded matrix, decoded and scaled: the lookup of an
// embedding table that is held in the 2-bit form ("E8-QAT", abstract: the
// core encoding and the sparse extension keep the lattice points exactly).
//
//   out[t] = alpha * w~[id_t - first_row],  w~ as in e8q_decode;
//   an id outside [first_row, first_row + rows) gives a row of zeros.
//
// One warp per (token, window of 2,048 columns = 256 groups).  Lane l owns
// the groups 32 j + l (j = 0..7), so that index reads and 16-byte stores of
// consecutive lanes are contiguous.  The row's records (CSR range, sorted or
// not) are scattered into the warp's 256-entry map group -> root + 1 /
// 0x8000 | slot of an overflow point; a lane's eight entries lie together (one
// 16-byte read, which also clears them).  What the next task needs first (its
// row, indices, record ranges) is loaded while the current one is computed.
//
// Original basis: the Hadamard transform of the window, on exact integers.
// Write an element's index inside the window as bits e10..e0: e2..e0 inside
// a group, e7..e3 the lane, e10..e8 the register j.  H_B is a product of
// one 2x2 transform per index bit below log2 B, so the bits may be taken in
// any grouping and order:
//   - e8..e10: butterflies over the lane's registers, in f16 pairs;
//   - MMA 1 (m16n8k16, f16): k = (e2, e3, e4, e0), n = lane / 4.  A codeword
//     pair (P_i, P_i+4) is one f16x2 B register as it comes out of the
//     nibbles;
//   - MMA 2: k = (e5, e6, e7, e1).  The f16 accumulator of MMA 1 (rows k', two
//     columns n a register) IS the B operand of its transpose, register for
//     register, so nothing moves between the two.  Its fp32 accumulator
//     holds, in lane l, the eight elements of lane l's own group again: they
//     are scaled, signed, rounded and stored at once.
// The transform needs no shuffle and no shared memory.  Bits at or above
// log2 B get a 2x2 identity in the MMA's A operand, so every block size takes
// the same path.  f16 is exact here: integers up to 2,048 are, the steps
// before MMA 2 combine at most 32 groups, and the sum of |P_i| over a group is
// below 28 for core points and core + root (|P| <= sqrt 48 + sqrt 8, sum
// |P_i| <= sqrt 8 |P|); an overflow point takes part when its sum is at most
// 64 (32 x 64 = 2,048).  Points farther out (rare), and those past the 32
// that the warp's staging holds, are left out of the f16 path and added in
// fp32.
//
// Measured: 8,192 rows of 4,096 columns at kappa = 1 (a fifth of the groups
// have records), original basis, bf16: 36 us for 84 MB, 2.3 TB/s, 35 % of the
// measured copy bandwidth; fp32 52 us, rotated basis 41 (bf16) and 53 (fp32).
// Bound by instructions and latency together (0.53 issued a cycle, 16 warps an
// SM at 124 registers); the codeword gathers take one L1 wavefront per line
// (the load pipe is 55 % busy).  Copies without the records run in 31 us, with
// the butterflies after the MMAs in fp32 43 us (64 more live values), with the
// prefetch in registers 55 us (two CTAs fewer).
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"
#include "gemv.cuh"
#include "lattice.cuh"
#include "ptx.cuh"

namespace e8q {

constexpr int kDrWarps = 8;
constexpr int kDrThreads = 32 * kDrWarps;
constexpr int kDrCtas = 2;  // an SM
constexpr int kDrNearSum = 64;  // largest sum of |P_i| of an overflow point in the f16 path
constexpr int kDrSlots = 32;     // overflow points of a window staged in f16
// what is added to a group's codeword, by map entry: 0 none, 1..240 roots, then every warp's staged points, then a void
constexpr int kDrFirstSlot = 241;
constexpr int kDrVoid = kDrFirstSlot + kDrWarps * kDrSlots;
constexpr int kDrFar = 0xFFFF;  // left out: contributes in fp32
constexpr int kDrEscStage = 128;  // records of a row staged ahead of their use; further ones are read in place
constexpr int kDrOvfStage = 32;

struct DecodeRowsParams {
    const uint16_t* idx;
    const float* scale;
    const int8_t* signs;
    const e8q_escape* esc;
    const int64_t* esc_rp;
    const e8q_overflow* ovf;
    const int64_t* ovf_rp;
    const void* ids;
    void* out;
    uint32_t esc_n, ovf_n;
    long long first_row;
    long long n;
    float alpha, sqrt_b;
    int32_t rows, cols, logb;
    int32_t nwin;
    int32_t id64;
    int32_t idx_copy;  // bytes an asynchronous copy of indices may take: 16, 4, or 0 (2-byte rows)
    uint32_t group_base;
};

__device__ __forceinline__ void mma_f16_m16n8k16(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ unsigned fma_f16x2(unsigned a, unsigned b, unsigned c) {
    unsigned d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ unsigned add_f16x2(unsigned a, unsigned b) {
    unsigned d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ unsigned pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&h);
}
__device__ __forceinline__ void mma_f16_m16n8k16(unsigned (&d)[2], const unsigned (&a)[4], unsigned b0, unsigned b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f16.f16.f16.f16 {%0,%1}, {%2,%3,%4,%5}, {%6,%7}, {%8,%8};"
        : "=r"(d[0]), "=r"(d[1])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(0u));
}

// A operand: the product over the four index bits of the 2x2 Hadamard matrix
// (bits set in `active`) or the 2x2 identity.
__device__ __forceinline__ unsigned dr_entry(int m, int k, int active) {
    if ((m ^ k) & ~active & 15) return 0u;
    return (__popc(m & k & active) & 1) ? 0xBC00u : 0x3C00u;  // -1 : 1
}
__device__ __forceinline__ void dr_matrix(unsigned (&a)[4], int lane, int active) {
    const int m = lane >> 2, k = 2 * (lane & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int mi = m + 8 * (i & 1), ki = k + 8 * (i >> 1);
        a[i] = dr_entry(mi, ki, active) | (dr_entry(mi, ki + 1, active) << 16);
    }
}

// Two tasks ahead: the ends of the row's record ranges, as loaded (nothing
// computes on them before the next iteration).  Their low words: records,
// like the groups that they belong to, number at most 2^32.
struct DrRow {
    unsigned esc, esc_end, ovf, ovf_end;
    float s;
    int row;  // -1: zeros
};
// A task's row once its records are known; its indices and first records are
// on their way to (or in) one of the warp's two shared-memory stages.
struct DrTask {
    int ne, no;
    float s;
    int row;
};
struct __align__(16) DrStage {
    uint16_t idx[256];
    uint2 esc[kDrEscStage];
    uint32_t ovf[kDrOvfStage * 5];
};

constexpr size_t kDrStageBytes = 2 * kDrWarps * sizeof(DrStage);
__host__ __device__ constexpr size_t dr_smem_bytes(bool original, int cols) {
    return kDrStageBytes + (original ? static_cast<size_t>(cols) * 2 : 0);
}

__device__ __forceinline__ long long dr_id(const DecodeRowsParams& p, long long t) {
    return p.id64 ? __ldg(static_cast<const long long*>(p.ids) + t)
                  : static_cast<long long>(__ldg(static_cast<const int*>(p.ids) + t));
}

__device__ __forceinline__ void dr_load(const DecodeRowsParams& p, long long id, DrRow& k) {
    // unsigned, since the distance of two 64-bit ids may not fit a signed one
    const unsigned long long d = static_cast<unsigned long long>(id) - static_cast<unsigned long long>(p.first_row);
    k.row = (id >= p.first_row && d < static_cast<unsigned long long>(p.rows)) ? static_cast<int>(d) : -1;
    if (k.row < 0) return;
    if (p.esc_rp) {
        k.esc = __ldg(reinterpret_cast<const unsigned*>(p.esc_rp + k.row));
        k.esc_end = __ldg(reinterpret_cast<const unsigned*>(p.esc_rp + k.row + 1));
    }
    if (p.ovf_rp) {
        k.ovf = __ldg(reinterpret_cast<const unsigned*>(p.ovf_rp + k.row));
        k.ovf_end = __ldg(reinterpret_cast<const unsigned*>(p.ovf_rp + k.row + 1));
    }
    k.s = __ldg(p.scale + k.row);
}

// records [first, end) of the n readable ones
__device__ __forceinline__ int dr_count(unsigned& first, unsigned end, unsigned n) {
    first = min(first, n);
    return static_cast<int>(min(max(min(end, n), first) - first, 1u << 30));
}

// The records of a row, past those that are staged (rare: the row's range is read again).
__device__ __forceinline__ const e8q_escape* dr_esc(const DecodeRowsParams& p, int row) {
    return p.esc + min(__ldg(reinterpret_cast<const unsigned*>(p.esc_rp + row)), p.esc_n);
}
__device__ __forceinline__ const uint32_t* dr_ovf(const DecodeRowsParams& p, int row) {
    return reinterpret_cast<const uint32_t*>(p.ovf + min(__ldg(reinterpret_cast<const unsigned*>(p.ovf_rp + row)), p.ovf_n));
}

// Start the copies of a task's indices and first records into a stage.
__device__ __forceinline__ void dr_stage(const DecodeRowsParams& p, DrRow& a, int w, int lane, DrTask& k, DrStage& st) {
    k.row = a.row;
    k.ne = k.no = 0;
    if (k.row >= 0) {
        k.s = a.s;
        const int gpr = p.cols >> 3, ng = min(256, gpr - 256 * w);
        const uint16_t* src = p.idx + static_cast<size_t>(k.row) * gpr + 256 * w;
        if (p.idx_copy == 16) {
            if (8 * lane < ng) cp_async16(st.idx + 8 * lane, src + 8 * lane);
        } else if (p.idx_copy == 4) {
            for (int g = 2 * lane; g < ng; g += 64) cp_async4(st.idx + g, src + g);
        } else {
            for (int g = lane; g < ng; g += 32) st.idx[g] = __ldg(src + g);
        }
        if (p.esc_rp) {
            k.ne = dr_count(a.esc, a.esc_end, p.esc_n);
            const int n = min(k.ne, kDrEscStage);
            for (int e = lane; e < n; e += 32) cp_async8(st.esc + e, p.esc + a.esc + e);
        }
        if (p.ovf_rp) {
            k.no = dr_count(a.ovf, a.ovf_end, p.ovf_n);
            const int n = 5 * min(k.no, kDrOvfStage);
            for (int o = lane; o < n; o += 32) cp_async4(st.ovf + o, reinterpret_cast<const uint32_t*>(p.ovf + a.ovf) + o);
        }
    }
    cp_async_commit();
}

__device__ __forceinline__ float dr_coord(const unsigned* o, int i) {  // coordinate i of a loaded overflow record
    return static_cast<float>(static_cast<short>(o[1 + (i >> 1)] >> (16 * (i & 1))));
}

__device__ __forceinline__ void dr_point(const uint32_t* rec, float (&f)[8]) {
    unsigned o[5];
#pragma unroll
    for (int q = 1; q < 5; ++q) o[q] = __ldg(rec + q);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = dr_coord(o, i);
}

// place of group gl of the window in the warp's map: a lane's entries together
__device__ __forceinline__ int dr_place(unsigned gl) { return static_cast<int>((gl & 31) * 8 + (gl >> 5)); }

// The groups left out of the f16 path (bit j of a lane's `far`: its group
// 32 j + lane), added to the transformed elements of group g: with T the
// transform inside a group, group gf adds +-T(P_gf), the sign being that of
// H at (g, gf), where both lie in one block.
__device__ __forceinline__ void dr_add_far(const DecodeRowsParams& p, float (&d0)[4], float (&d1)[4], unsigned far,
                                        const uint16_t* far_rec, int row, int g) {
    const int gmask = p.logb >= 3 ? (1 << (p.logb - 3)) - 1 : 0;
#pragma unroll 1
    for (int jj = 0; jj < 8; ++jj) {
        unsigned todo = __ballot_sync(0xFFFFFFFFu, (far >> jj) & 1u);
#pragma unroll 1
        while (todo) {
            const int gf = 32 * jj + __ffs(todo) - 1;
            todo &= todo - 1;
            float f[8];
            dr_point(dr_ovf(p, row) + 5 * far_rec[gf], f);
            if (p.logb >= 3) fwht_reg<8>(f);
            if ((g ^ gf) & ~gmask) continue;
            const float s = (__popc(g & gf & gmask) & 1) ? -1.f : 1.f;
            d0[0] = fmaf(s, f[0], d0[0]);
            d0[1] = fmaf(s, f[4], d0[1]);
            d0[2] = fmaf(s, f[2], d0[2]);
            d0[3] = fmaf(s, f[6], d0[3]);
            d1[0] = fmaf(s, f[1], d1[0]);
            d1[1] = fmaf(s, f[5], d1[1]);
            d1[2] = fmaf(s, f[3], d1[2]);
            d1[3] = fmaf(s, f[7], d1[3]);
        }
    }
}

// kFull: the width is a multiple of 2,048, so that every window is whole.
template <bool kOriginal, bool kF32, bool kFull>
__global__ void __launch_bounds__(kDrThreads, kDrCtas) k_decode_rows(const __grid_constant__ DecodeRowsParams p) {
    __shared__ __align__(16) uint16_t s_map[kDrWarps][256];
    __shared__ __align__(16) uint4 s_add[kDrVoid + 1];  // pairs (i, i + 4) in f16; roots less the nibbles' bias of 1032
    __shared__ uint16_t s_far[kDrWarps][256];           // record of each group left out, in the row
    __shared__ __align__(16) uint4 s_a[2][32];          // the MMAs' A operands
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kDrFirstSlot; i += kDrThreads) {
        const uint2 c = i > 0 ? __ldg(g_root8 + i - 1) : make_uint2(0, 0);
        unsigned h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            h[q] = pack_f16x2(static_cast<float>(coord_of(c, q)) - 1032.f, static_cast<float>(coord_of(c, q + 4)) - 1032.f);
        s_add[i] = make_uint4(h[0], h[1], h[2], h[3]);
    }
    if (tid == 0) s_add[kDrVoid] = make_uint4(0, 0, 0, 0);
    const int gpr = p.cols >> 3;
    extern __shared__ __align__(16) unsigned char smem[];
    DrStage* stage = reinterpret_cast<DrStage*>(smem) + 2 * warp;
    // a group's eight sign bits in the sign places of its bf16 output, lane by lane
    uint4* s_sign = reinterpret_cast<uint4*>(smem + kDrStageBytes);
    if (kOriginal) {
        if (warp < 2) {  // e2, e3, e4, e0 | e5, e6, e7, e1
            const int act = (1 << p.logb) - 1;
            unsigned a[4];
            dr_matrix(a, lane, ((act >> (2 + 3 * warp)) & 7) | (((act >> warp) & 1) << 3));
            s_a[warp][lane] = make_uint4(a[0], a[1], a[2], a[3]);
        }
        for (int g = tid; g < gpr; g += kDrThreads) {
            const uint2 d = __ldg(reinterpret_cast<const uint2*>(p.signs) + g);
            s_sign[g] = make_uint4(prmt(d.x, 0u, 0x1404u) & 0x80008000u, prmt(d.x, 0u, 0x3424u) & 0x80008000u,
                                   prmt(d.y, 0u, 0x1404u) & 0x80008000u, prmt(d.y, 0u, 0x3424u) & 0x80008000u);
        }
    }
    uint16_t* map = s_map[warp];
    uint16_t* far_rec = s_far[warp];
    uint4* lane_map = reinterpret_cast<uint4*>(map) + lane;
    *lane_map = make_uint4(0, 0, 0, 0);
    __syncthreads();

    // this warp's tasks: (token t, window w), advanced by the grid's warps (n <= 2^30: the sums fit 32 bits)
    const int n = static_cast<int>(p.n);
    const int stride = static_cast<int>(gridDim.x) * kDrWarps, task = static_cast<int>(blockIdx.x) * kDrWarps + warp;
    const int dt = stride / p.nwin, dw = stride - dt * p.nwin;
    int t = task / p.nwin, w = task - t * p.nwin;
    if (t >= n) return;
    auto advance = [&](int& tt, int& ww) {
        tt += dt;
        ww += dw;
        if (ww >= p.nwin) {
            ww -= p.nwin;
            ++tt;
        }
    };
    DrRow ahead;
    DrTask cur, nxt;
    dr_load(p, dr_id(p, t), ahead);
    int t1 = t, w1 = w;  // one task ahead
    advance(t1, w1);
    int t2 = t1, w2 = w1;  // two
    advance(t2, w2);
    const long long id1 = t1 < n ? dr_id(p, t1) : 0;
    dr_stage(p, ahead, w, lane, nxt, stage[0]);
    if (t1 < n) dr_load(p, id1, ahead);
    long long id2 = t2 < n ? dr_id(p, t2) : 0;

    for (int k = 0; t < n; ++k) {
        const DrStage& st = stage[k & 1];
        cp_async_wait_all();
        __syncwarp();  // this task's stage is filled, and every lane is done with the other one
        cur = nxt;
        // the next two tasks' loads go out before this task's work
        if (t1 < n) {
            dr_stage(p, ahead, w1, lane, nxt, stage[(k + 1) & 1]);
            if (t2 < n) dr_load(p, id2, ahead);
        }
        const int w_now = w;
        const int ng = kFull ? 256 : min(256, gpr - 256 * w_now);  // groups of this window
        unsigned char* out = static_cast<unsigned char*>(p.out) +
                             (static_cast<size_t>(t) * p.cols + 2048 * static_cast<size_t>(w_now)) * (kF32 ? 4 : 2);
        t = t1;
        w = w1;
        t1 = t2;
        w1 = w2;
        advance(t2, w2);
        if (t2 < n) id2 = dr_id(p, t2);
        if (cur.row < 0) {
            for (int g = lane; g < ng; g += 32) {
                uint4* o = reinterpret_cast<uint4*>(out) + (kF32 ? 2 : 1) * g;
                o[0] = make_uint4(0, 0, 0, 0);
                if (kF32) o[1] = make_uint4(0, 0, 0, 0);
            }
            continue;
        }
        unsigned wd[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) wd[j] = 32 * j + lane < ng ? __ldg(g_gv_tab + st.idx[32 * j + lane]) : 0x88888888u;  // the origin
        const float as = p.alpha * cur.s;
        unsigned pr[8][4];  // codeword pairs (P_i, P_i+4), i = 0..3, of the lane's groups in f16
        unsigned far = 0;   // groups (bit j) left out
        bool any_far = false;
        // group ids are 32-bit and the matrix's all fit (checked by the caller), so differences modulo 2^32 do
        const unsigned g0 = p.group_base + static_cast<unsigned>(cur.row) * gpr + 256 * w_now;
        auto escape = [&](uint2 r) {
            const unsigned gl = r.x - g0, root = (r.y >> 16) & 0xFFu;
            if (gl < static_cast<unsigned>(ng) && root < 240) map[dr_place(gl)] = static_cast<uint16_t>(root + 1);
        };
#pragma unroll 2
        for (int e = lane; e < min(cur.ne, kDrEscStage); e += 32) escape(st.esc[e]);
        if (cur.ne > kDrEscStage) {
            const uint2* more = reinterpret_cast<const uint2*>(dr_esc(p, cur.row));
#pragma unroll 1
            for (int e = lane + kDrEscStage; e < cur.ne; e += 32) escape(__ldg(more + e));
        }
        __syncwarp();
        int used = 0;
#pragma unroll 1
        for (int o0 = 0; o0 < cur.no; o0 += 32) {
            const bool on = o0 + lane < cur.no;
            unsigned rec[5] = {0, 0, 0, 0, 0};
            if (on)
#pragma unroll
                for (int q = 0; q < 5; ++q) rec[q] = o0 == 0 ? st.ovf[5 * lane + q] : __ldg(dr_ovf(p, cur.row) + 5 * (o0 + lane) + q);
            const unsigned gl = on ? rec[0] - g0 : 0xFFFFFFFFu;
            const bool mine = gl < static_cast<unsigned>(ng);
            if (!__any_sync(0xFFFFFFFFu, mine)) continue;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += fabsf(dr_coord(rec, i));
            const bool near = mine && kOriginal && sum <= static_cast<float>(kDrNearSum);
            const unsigned peers = __ballot_sync(0xFFFFFFFFu, near);
            const int slot = used + __popc(peers & lanemask_lt());
            used += __popc(peers);
            if (near && slot < kDrSlots) {
                const int at = kDrFirstSlot + warp * kDrSlots + slot;
                s_add[at] = make_uint4(pack_f16x2(dr_coord(rec, 0), dr_coord(rec, 4)), pack_f16x2(dr_coord(rec, 1), dr_coord(rec, 5)),
                                       pack_f16x2(dr_coord(rec, 2), dr_coord(rec, 6)), pack_f16x2(dr_coord(rec, 3), dr_coord(rec, 7)));
                map[dr_place(gl)] = static_cast<uint16_t>(at);
            } else if (mine && o0 + lane < 0x7FFF) {
                far_rec[gl] = static_cast<uint16_t>(o0 + lane);
                map[dr_place(gl)] = kDrFar;
                any_far = true;
            }
        }
        __syncwarp();
        any_far = __any_sync(0xFFFFFFFFu, any_far);
        const uint4 mp = *lane_map;
        *lane_map = make_uint4(0, 0, 0, 0);
        unsigned mw[4] = {mp.x, mp.y, mp.z, mp.w};
        if (any_far) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (((mw[j >> 1] >> (16 * (j & 1))) & 0xFFFFu) == kDrFar) {
                    far |= 1u << j;
                    mw[j >> 1] ^= static_cast<unsigned>(kDrFar ^ kDrVoid) << (16 * (j & 1));
                }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const unsigned m = (j & 1) ? mw[j >> 1] >> 16 : mw[j >> 1] & 0xFFFFu;
            const uint4 add = s_add[m];
            const unsigned keep = m < kDrFirstSlot ? 0x3C003C00u : 0u;  // an overflow point takes the codeword's place
            // (1024 + nibble) x 1 + (root - 1032), exact
            pr[j][0] = fma_f16x2((wd[j] & 0x000F000Fu) | 0x64006400u, keep, add.x);
            pr[j][1] = fma_f16x2(((wd[j] >> 4) & 0x000F000Fu) | 0x64006400u, keep, add.y);
            pr[j][2] = fma_f16x2(((wd[j] >> 8) & 0x000F000Fu) | 0x64006400u, keep, add.z);
            pr[j][3] = fma_f16x2(((wd[j] >> 12) & 0x000F000Fu) | 0x64006400u, keep, add.w);
        }

        if (kOriginal) {
            const uint4 m1 = s_a[0][lane], m2 = s_a[1][lane];
            const unsigned a1[4] = {m1.x, m1.y, m1.z, m1.w}, a2[4] = {m2.x, m2.y, m2.z, m2.w};
#pragma unroll
            for (int h = 1; h < 8; h <<= 1) {
                if ((256 * h) < (1 << p.logb)) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if ((j & h) == 0) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const unsigned x = pr[j][i], y = pr[j + h][i];
                                pr[j][i] = add_f16x2(x, y);
                                pr[j + h][i] = hsub2_bits(x, y);
                            }
                        }
                }
            }
            const float mul = 0.5f * (as / p.sqrt_b);
            const float2 mul2 = make_float2(mul, mul);
            auto finish = [&](int g, const unsigned (&x)[4], auto&& more) {
                unsigned c0[2], c1[2];
                mma_f16_m16n8k16(c0, a1, x[0], x[1]);  // e1 = 0: elements 0, 4 | 1, 5
                mma_f16_m16n8k16(c1, a1, x[2], x[3]);  // e1 = 1
                float d0[4], d1[4];
                mma_f16_m16n8k16(d0, a2, c0[0], c1[0]);  // e0' = 0: elements 0, 4 | 2, 6
                mma_f16_m16n8k16(d1, a2, c0[1], c1[1]);  // e0' = 1: elements 1, 5 | 3, 7
                more(d0, d1);
                if (g >= ng) return;
                const float2 y0 = __fmul2_rn(make_float2(d0[0], d0[1]), mul2), y1 = __fmul2_rn(make_float2(d1[0], d1[1]), mul2);
                const float2 y2 = __fmul2_rn(make_float2(d0[2], d0[3]), mul2), y3 = __fmul2_rn(make_float2(d1[2], d1[3]), mul2);
                const uint4 m = s_sign[256 * w_now + g];
                if (kF32) {
                    uint4* o = reinterpret_cast<uint4*>(out) + 2 * g;
                    o[0] = make_uint4(__float_as_uint(y0.x) ^ (m.x << 16), __float_as_uint(y1.x) ^ (m.x & 0x80000000u),
                                      __float_as_uint(y2.x) ^ (m.y << 16), __float_as_uint(y3.x) ^ (m.y & 0x80000000u));
                    o[1] = make_uint4(__float_as_uint(y0.y) ^ (m.z << 16), __float_as_uint(y1.y) ^ (m.z & 0x80000000u),
                                      __float_as_uint(y2.y) ^ (m.w << 16), __float_as_uint(y3.y) ^ (m.w & 0x80000000u));
                } else {
                    auto word = [](float lo, float hi, unsigned sign) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
                        return *reinterpret_cast<const unsigned*>(&h) ^ sign;
                    };
                    reinterpret_cast<uint4*>(out)[g] = make_uint4(word(y0.x, y1.x, m.x), word(y2.x, y3.x, m.y),
                                                                  word(y0.y, y1.y, m.z), word(y2.y, y3.y, m.w));
                }
            };
            if (!any_far) {
#pragma unroll
                for (int j = 0; j < 8; ++j) finish(32 * j + lane, pr[j], [](float (&)[4], float (&)[4]) {});
            } else {  // apart, so that the rare case costs the other no registers
                unsigned x[8][4];
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[j][i] = pr[j][i];
#pragma unroll 1
                for (int j = 0; j < 8; ++j)
                    finish(32 * j + lane, x[j], [&](float (&d0)[4], float (&d1)[4]) {
                        dr_add_far(p, d0, d1, far, far_rec, cur.row, 32 * j + lane);
                    });
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int g = 32 * j + lane;
                if (g >= ng) continue;
                float f[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&pr[j][i]));
                    f[i] = x.x;
                    f[i + 4] = x.y;
                }
                if ((far >> j) & 1u) dr_point(dr_ovf(p, cur.row) + 5 * far_rec[g], f);
                if (kF32) {
                    float4* o = reinterpret_cast<float4*>(out) + 2 * g;
                    o[0] = make_float4(as * (0.5f * f[0]), as * (0.5f * f[1]), as * (0.5f * f[2]), as * (0.5f * f[3]));
                    o[1] = make_float4(as * (0.5f * f[4]), as * (0.5f * f[5]), as * (0.5f * f[6]), as * (0.5f * f[7]));
                } else {
                    reinterpret_cast<uint4*>(out)[g] =
                        make_uint4(bf16x2_of_half_products(as, f[0], f[1]), bf16x2_of_half_products(as, f[2], f[3]),
                                   bf16x2_of_half_products(as, f[4], f[5]), bf16x2_of_half_products(as, f[6], f[7]));
                }
            }
        }
        __syncwarp();  // the map and the staged points are free for the next task
    }
}

}  // namespace e8q

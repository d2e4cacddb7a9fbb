// Entry points of the low-rank adapters (include/e8q.h) over lora.cuh.
#include "lora.cuh"

#include <algorithm>
#include <mutex>

#include "host.cuh"

namespace e8q {
namespace {

// CTAs that run at once where two fit an SM; a constant, so that the order of the
// sums is the same on any device.
constexpr int64_t kAtOnce = 2 * 148;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct LrGeom {
    int tile, mt;            // tokens a tile; 16-row tiles of the rank in a k_lr_down CTA
    int64_t tiles;           // most tiles
    int64_t zparts;          // rank parts of k_lr_down
    int64_t unit, units, parts;  // tokens a unit, most units, most partial sums (backward)
};

LrGeom geometry(const e8q_adapters& a, int64_t tokens) {
    LrGeom g;
    g.tile = tokens <= kLrSmallTokens ? kLrSmallTile : kLrTile;
    // every group (the tokens without an adapter are one) adds at most one tile that is not full
    g.tiles = std::min(tokens, ceil_div(tokens, g.tile) + std::min<int64_t>(tokens, int64_t{a.n} + 1));
    g.mt = a.rank <= 16 ? 1 : a.rank <= 32 ? 2 : 4;
    g.zparts = ceil_div(a.rank, 64);
    const int64_t along = ceil_div(a.rows, kLrGradCols) + ceil_div(a.cols, kLrGradCols);
    // cuts of the tokens into units: as many as run at once, and units of at most kLrUnitMax tokens
    const int64_t cuts = std::max(std::max<int64_t>(1, kAtOnce / along), ceil_div(tokens, kLrUnitMax));
    g.unit = ceil_div(ceil_div(tokens, cuts), 64) * 64;
    const int64_t full = std::min(cuts, ceil_div(tokens, 64));  // at least ceil(tokens / unit), and growing with the tokens
    g.units = full + std::min<int64_t>(tokens, a.n);
    g.parts = 2 * full;  // an adapter of several units has all but one full
    return g;
}

// Columns a CTA of k_lr_down: as many as let all CTAs run at once (a second
// wave would wait for the first), at most 4,096 so that a warp's sum has at
// most 64 MMAs.  Small batches take three CTAs an SM (two and four measured 6 %
// and 8 % slower on 64 tokens of 64 adapters).
int64_t down_at_once(const LrGeom& g) { return 148 * (g.tile == kLrSmallTile ? 3 : 2); }
int64_t down_columns(const LrGeom& g, int64_t cols) {
    const int64_t least = ceil_div(cols, 4096), most = ceil_div(cols, 256);
    const int64_t splits = std::min(most, std::max(least, down_at_once(g) / (g.tiles * g.zparts)));
    return ceil_div(ceil_div(cols, splits), 256) * 256;
}

struct LrWs {
    size_t head, order, tiles, units, unit_base, part, parts, grads, total;
};

// Every part is a bound that grows with the tokens, so that a workspace serves
// smaller calls too.
LrWs workspace(const e8q_adapters& a, int64_t tokens, const LrGeom& g, bool backward) {
    LrWs w = {};
    size_t at = 0;
    auto take = [&at](size_t bytes) {
        const size_t o = at;
        at += align256(bytes);
        return o;
    };
    w.head = take(16);
    w.order = take(static_cast<size_t>(tokens) * 4);
    const int64_t few = std::min<int64_t>(tokens, kLrSmallTokens);
    w.tiles = take(static_cast<size_t>(std::max(g.tiles, geometry(a, few).tiles)) * sizeof(LrTile));
    w.units = take(static_cast<size_t>(g.units) * sizeof(LrTile));
    w.unit_base = take(static_cast<size_t>(a.n) * 8);
    const int64_t cols = backward ? a.rows : a.cols;
    // tokens x splits: the splits are the least, or at most down_at_once / tiles with tiles >= tokens / tile
    const int64_t rows = std::max(tokens * ceil_div(cols, 4096), std::min(tokens * ceil_div(cols, 256), down_at_once(g) * g.tile));
    w.part = take(static_cast<size_t>(rows) * a.rank * 4);
    if (backward) {
        w.parts = take(static_cast<size_t>(4) * tokens * a.rank * 2);
        w.grads = take(static_cast<size_t>(g.parts) * (a.rows + a.cols) * a.rank * 4);
    }
    w.total = at;
    return w;
}

e8q_status check(const e8q_adapters* a, int64_t tokens) {
    if (!a || tokens < 0 || a->n < 0 || a->rows <= 0 || a->cols <= 0 || a->rank <= 0) return E8Q_ERR_INVALID_ARG;
    if (a->rows % 8 != 0 || a->cols % 8 != 0 || a->rank % 8 != 0) return E8Q_ERR_INVALID_ARG;
    if (a->rows > kLrMaxWidth || a->cols > kLrMaxWidth || a->rank > kLrMaxRank || a->n > kLrMaxAdapters ||
        tokens > kLrMaxTokens)
        return E8Q_ERR_UNSUPPORTED;
    if (a->n > 0 && (!a->a || !a->b || !a->scale || !aligned(a->a, 16) || !aligned(a->b, 16) || !aligned(a->scale, 4)))
        return E8Q_ERR_INVALID_ARG;
    return E8Q_OK;
}

// whether a buffer lies in the adapters' own
bool overlaps_adapters(const e8q_adapters& a, const void* p, size_t bytes) {
    if (a.n == 0) return false;
    const size_t each = static_cast<size_t>(a.n) * a.rank * 2;
    return overlap(p, bytes, a.a, each * a.cols) || overlap(p, bytes, a.b, each * a.rows) ||
           overlap(p, bytes, a.scale, static_cast<size_t>(a.n) * 4);
}

size_t plan_smem(int n) { return static_cast<size_t>(n + 2) * 16 + static_cast<size_t>(n + 1) * 64; }

template <typename K>
e8q_status allow(K kernel, size_t smem) {
    return cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
}

template <int MT, bool kTrans>
e8q_status allow_down() {
    e8q_status st = allow(k_lr_down<MT, kTrans>, lr_down_smem(MT, kTrans));
    return st == E8Q_OK ? allow(k_lr_down_few<MT, kTrans>, lr_down_few_smem(MT, kTrans)) : st;
}

template <int KS, bool kTrans>
e8q_status allow_up() {
    e8q_status st = allow(k_lr_up<KS, kLrTile, kTrans>, lr_up_smem(KS, kLrTile, kTrans));
    return st == E8Q_OK ? allow(k_lr_up<KS, kLrSmallTile, kTrans>, lr_up_smem(KS, kLrSmallTile, kTrans)) : st;
}

template <bool kTrans>
e8q_status allow_all() {
    e8q_status st = allow_down<1, kTrans>();
    if (st == E8Q_OK) st = allow_down<2, kTrans>();
    if (st == E8Q_OK) st = allow_down<4, kTrans>();
    if (st == E8Q_OK) st = allow_up<1, kTrans>();
    if (st == E8Q_OK) st = allow_up<2, kTrans>();
    if (st == E8Q_OK) st = allow_up<4, kTrans>();
    if (st == E8Q_OK) st = allow_up<8, kTrans>();
    return st;
}

// Shared-memory limits of the kernels, once per device.
e8q_status ensure_lora() {
    static std::mutex mu;
    static bool ready[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return E8Q_ERR_CUDA;
    if (dev < 0 || dev >= 64) return E8Q_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(mu);
    if (ready[dev]) return E8Q_OK;
    e8q_status st = allow(k_lr_plan, plan_smem(kLrMaxAdapters));
    if (st == E8Q_OK) st = allow_all<false>();
    if (st == E8Q_OK) st = allow_all<true>();
    if (st == E8Q_OK) st = allow(k_lr_grad<2>, lr_grad_smem(2));
    if (st == E8Q_OK) st = allow(k_lr_grad<4>, lr_grad_smem(4));
    if (st == E8Q_OK) st = allow(k_lr_grad<8>, lr_grad_smem(8));
    if (st == E8Q_OK) st = allow(k_lr_grad<16>, lr_grad_smem(16));
    ready[dev] = st == E8Q_OK;
    return st;
}

e8q_status launch_plan(const e8q_adapters& a, const int32_t* slots, int64_t tokens, const LrGeom& g, const LrWs& l,
                       unsigned char* w, cudaStream_t s) {
    LrPlanParams p;
    p.slots = slots;
    p.tokens = static_cast<int32_t>(tokens);
    p.n = a.n;
    p.tile = g.tile;
    p.unit = static_cast<int32_t>(g.unit);
    p.head = reinterpret_cast<int32_t*>(w + l.head);
    p.order = reinterpret_cast<int32_t*>(w + l.order);
    p.tiles = reinterpret_cast<LrTile*>(w + l.tiles);
    p.units = reinterpret_cast<LrTile*>(w + l.units);
    p.unit_base = reinterpret_cast<int32_t*>(w + l.unit_base);
    k_lr_plan<<<1, kLrPlanThreads, plan_smem(a.n), s>>>(p);
    return cuda_ok(cudaGetLastError());
}

template <bool kTrans>
e8q_status launch_down(const e8q_adapters& a, const int32_t* slots, const void* z, const void* weights, int64_t cols,
                       int64_t tokens, const LrGeom& g, const LrWs& l, unsigned char* w, cudaStream_t s, bool overlaps) {
    LrDownParams p;
    p.slots = slots;
    p.n = a.n;
    p.head = reinterpret_cast<const int32_t*>(w + l.head);
    p.order = reinterpret_cast<const int32_t*>(w + l.order);
    p.tiles = reinterpret_cast<const LrTile*>(w + l.tiles);
    p.z = static_cast<const uint16_t*>(z);
    p.w = static_cast<const uint16_t*>(weights);
    p.part = reinterpret_cast<float*>(w + l.part);
    p.tokens = static_cast<int32_t>(tokens);
    p.cols = static_cast<int32_t>(cols);
    p.rank = a.rank;
    p.per = static_cast<int32_t>(down_columns(g, cols));
    const dim3 grid(static_cast<unsigned>(g.tiles), static_cast<unsigned>(ceil_div(cols, p.per)), static_cast<unsigned>(g.zparts));
    if (g.tile == kLrSmallTile) {
        const size_t smem = lr_down_few_smem(g.mt, kTrans);
        if (g.mt == 1) return launch_pdl(k_lr_down_few<1, kTrans>, grid, kLrFewThreads, smem, s, p, overlaps);
        if (g.mt == 2) return launch_pdl(k_lr_down_few<2, kTrans>, grid, kLrFewThreads, smem, s, p, overlaps);
        return launch_pdl(k_lr_down_few<4, kTrans>, grid, kLrFewThreads, smem, s, p, overlaps);
    }
    const size_t smem = lr_down_smem(g.mt, kTrans);
    if (g.mt == 1) return launch_pdl(k_lr_down<1, kTrans>, grid, kLrDownThreads, smem, s, p);
    if (g.mt == 2) return launch_pdl(k_lr_down<2, kTrans>, grid, kLrDownThreads, smem, s, p);
    return launch_pdl(k_lr_down<4, kTrans>, grid, kLrDownThreads, smem, s, p);
}

template <int KS, bool kTrans>
e8q_status launch_up_rank(const LrGeom& g, cudaStream_t s, LrUpParams& p) {
    const bool small = g.tile == kLrSmallTile;
    // two rounds of the four CTAs that an SM holds: enough steps to share the factors' preparation, and a short
    // tail (one round: 5 % slower on a 4,096-token prefill)
    const int64_t parts = std::min(std::max<int64_t>(1, 8 * 148 / g.tiles), ceil_div(p.cols, kLrUpCols));
    const dim3 grid(static_cast<unsigned>(g.tiles), static_cast<unsigned>(parts));
    constexpr int T = kLrTile, S = kLrSmallTile;
    return small ? launch_pdl(k_lr_up<KS, S, kTrans>, grid, kLrUpThreads, lr_up_smem(KS, S, kTrans), s, p)
                 : launch_pdl(k_lr_up<KS, T, kTrans>, grid, kLrUpThreads, lr_up_smem(KS, T, kTrans), s, p);
}

template <bool kTrans>
e8q_status launch_up(const e8q_adapters& a, const int32_t* slots, const void* weights, const void* base, void* out, float* sum, int64_t cols,
                     int64_t sum_cols, int64_t tokens, const LrGeom& g, const LrWs& l, unsigned char* w, cudaStream_t s) {
    LrUpParams p;
    p.slots = slots;
    p.n = a.n;
    p.head = reinterpret_cast<const int32_t*>(w + l.head);
    p.order = reinterpret_cast<const int32_t*>(w + l.order);
    p.tiles = reinterpret_cast<const LrTile*>(w + l.tiles);
    p.part = reinterpret_cast<const float*>(w + l.part);
    p.scale = a.scale;
    p.w = static_cast<const uint16_t*>(weights);
    p.base = static_cast<const uint16_t*>(base);
    p.out = static_cast<uint16_t*>(out);
    p.sum = sum;
    p.tokens = static_cast<int32_t>(tokens);
    p.cols = static_cast<int32_t>(cols);
    p.rank = a.rank;
    p.splits = static_cast<int32_t>(ceil_div(sum_cols, down_columns(g, sum_cols)));
    if (a.rank <= 16) return launch_up_rank<1, kTrans>(g, s, p);
    if (a.rank <= 32) return launch_up_rank<2, kTrans>(g, s, p);
    if (a.rank <= 64) return launch_up_rank<4, kTrans>(g, s, p);
    return launch_up_rank<8, kTrans>(g, s, p);
}

}  // namespace
}  // namespace e8q

using namespace e8q;

extern "C" {

size_t e8q_lora_workspace_bytes(const e8q_adapters* a, int64_t tokens, int32_t backward) {
    if (check(a, tokens) != E8Q_OK || tokens == 0) return 256;
    return workspace(*a, tokens, geometry(*a, tokens), backward != 0).total;
}

e8q_status e8q_lora(const e8q_adapters* a, const void* x, const int32_t* slots, int64_t tokens, const void* base,
                    void* y, float* u, void* ws, size_t ws_bytes, e8q_stream stream) {
    e8q_status st = check(a, tokens);
    if (st != E8Q_OK || tokens == 0) return st;
    if (!x || !slots || !y || !aligned(x, 16) || !aligned(slots, 4) || !aligned(y, 16) || !aligned(base, 16) || !aligned(u, 16))
        return E8Q_ERR_INVALID_ARG;
    const size_t xb = static_cast<size_t>(tokens) * a->cols * 2, yb = static_cast<size_t>(tokens) * a->rows * 2;
    const size_t ub = static_cast<size_t>(tokens) * a->rank * 4, sb = static_cast<size_t>(tokens) * 4;
    if (overlap(x, xb, y, yb) || overlap(slots, sb, y, yb) || (base && base != y && overlap(base, yb, y, yb)))
        return E8Q_ERR_INVALID_ARG;
    if (u && (overlap(u, ub, x, xb) || overlap(u, ub, y, yb) || overlap(u, ub, slots, sb) || (base && overlap(u, ub, base, yb))))
        return E8Q_ERR_INVALID_ARG;
    if (overlaps_adapters(*a, y, yb) || (u && overlaps_adapters(*a, u, ub))) return E8Q_ERR_INVALID_ARG;
    const LrGeom g = geometry(*a, tokens);
    const LrWs l = workspace(*a, tokens, g, false);
    if (!ws || ws_bytes < l.total || !aligned(ws, 256)) return E8Q_ERR_WORKSPACE;
    st = ensure_lora();
    if (st != E8Q_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    unsigned char* w = static_cast<unsigned char*>(ws);
    if (g.tile != kLrSmallTile) st = launch_plan(*a, slots, tokens, g, l, w, s);
    if (st == E8Q_OK) st = launch_down<false>(*a, slots, x, a->a, a->cols, tokens, g, l, w, s, g.tile != kLrSmallTile);
    if (st == E8Q_OK) st = launch_up<false>(*a, slots, a->b, base, y, u, a->rows, a->cols, tokens, g, l, w, s);
    return st;
}

e8q_status e8q_lora_backward(const e8q_adapters* a, const void* grad_y, const void* x, const float* u,
                             const int32_t* slots, int64_t tokens, void* grad_a, void* grad_b, const void* grad_x_base,
                             void* grad_x, void* ws, size_t ws_bytes, e8q_stream stream) {
    e8q_status st = check(a, tokens);
    if (st != E8Q_OK) return st;
    const size_t ab = static_cast<size_t>(a->n) * a->rank * a->cols * 2, bb = static_cast<size_t>(a->n) * a->rank * a->rows * 2;
    if (a->n > 0 && (!grad_a || !grad_b || !aligned(grad_a, 16) || !aligned(grad_b, 16))) return E8Q_ERR_INVALID_ARG;
    if (a->n > 0 && (overlap(grad_a, ab, grad_b, bb) || overlaps_adapters(*a, grad_a, ab) || overlaps_adapters(*a, grad_b, bb)))
        return E8Q_ERR_INVALID_ARG;
    if (tokens > 0) {
        if (!grad_y || !x || !u || !slots || !aligned(grad_y, 16) || !aligned(x, 16) || !aligned(u, 16) ||
            !aligned(slots, 4) || !aligned(grad_x, 16) || !aligned(grad_x_base, 16) || (grad_x_base && !grad_x))
            return E8Q_ERR_INVALID_ARG;
        const size_t xb = static_cast<size_t>(tokens) * a->cols * 2, yb = static_cast<size_t>(tokens) * a->rows * 2;
        const size_t ub = static_cast<size_t>(tokens) * a->rank * 4, sb = static_cast<size_t>(tokens) * 4;
        const struct { const void* p; size_t n; } ins[] = {{grad_y, yb}, {x, xb}, {u, ub}, {slots, sb}};
        for (const auto& i : ins) {
            if (a->n > 0 && (overlap(i.p, i.n, grad_a, ab) || overlap(i.p, i.n, grad_b, bb))) return E8Q_ERR_INVALID_ARG;
            if (grad_x && overlap(i.p, i.n, grad_x, xb)) return E8Q_ERR_INVALID_ARG;
        }
        if (grad_x && overlaps_adapters(*a, grad_x, xb)) return E8Q_ERR_INVALID_ARG;
        if (grad_x && a->n > 0 && (overlap(grad_x, xb, grad_a, ab) || overlap(grad_x, xb, grad_b, bb))) return E8Q_ERR_INVALID_ARG;
        if (grad_x_base && grad_x_base != grad_x && overlap(grad_x_base, xb, grad_x, xb)) return E8Q_ERR_INVALID_ARG;
        if (grad_x_base && a->n > 0 && (overlap(grad_x_base, xb, grad_a, ab) || overlap(grad_x_base, xb, grad_b, bb)))
            return E8Q_ERR_INVALID_ARG;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (tokens == 0) {
        if (a->n == 0) return E8Q_OK;
        st = cuda_ok(cudaMemsetAsync(grad_a, 0, ab, s));
        return st == E8Q_OK ? cuda_ok(cudaMemsetAsync(grad_b, 0, bb, s)) : st;
    }
    const LrGeom g = geometry(*a, tokens);
    const LrWs l = workspace(*a, tokens, g, true);
    if (!ws || ws_bytes < l.total || !aligned(ws, 256)) return E8Q_ERR_WORKSPACE;
    st = ensure_lora();
    if (st != E8Q_OK) return st;
    unsigned char* w = static_cast<unsigned char*>(ws);
    st = launch_plan(*a, slots, tokens, g, l, w, s);
    if (st == E8Q_OK) st = launch_down<true>(*a, slots, grad_y, a->b, a->rows, tokens, g, l, w, s, true);
    if (st == E8Q_OK && a->n > 0) {
        LrSplitParams sp;
        sp.head = reinterpret_cast<const int32_t*>(w + l.head);
        sp.order = reinterpret_cast<const int32_t*>(w + l.order);
        sp.slots = slots;
        sp.u = u;
        sp.part = reinterpret_cast<const float*>(w + l.part);
        sp.scale = a->scale;
        sp.parts = reinterpret_cast<uint16_t*>(w + l.parts);
        sp.tokens = static_cast<int32_t>(tokens);
        sp.rank = a->rank;
        sp.splits = static_cast<int32_t>(ceil_div(a->rows, down_columns(g, a->rows)));
        st = launch_pdl(k_lr_split, static_cast<int>(std::min<int64_t>(2 * kAtOnce, ceil_div(tokens * (a->rank / 4), 256))), 256, 0, s, sp);
        if (st != E8Q_OK) return st;
        LrGradParams gp;
        gp.head = sp.head;
        gp.order = sp.order;
        gp.units = reinterpret_cast<const LrTile*>(w + l.units);
        gp.unit_base = reinterpret_cast<const int32_t*>(w + l.unit_base);
        gp.gy = static_cast<const uint16_t*>(grad_y);
        gp.x = static_cast<const uint16_t*>(x);
        gp.parts = sp.parts;
        gp.part = reinterpret_cast<float*>(w + l.grads);
        gp.grad_b = static_cast<uint16_t*>(grad_b);
        gp.grad_a = static_cast<uint16_t*>(grad_a);
        gp.tokens = sp.tokens;
        gp.rows = static_cast<int32_t>(a->rows);
        gp.cols = static_cast<int32_t>(a->cols);
        gp.rank = a->rank;
        gp.n = a->n;
        gp.row_ctas = static_cast<int32_t>(ceil_div(a->rows, kLrGradCols));
        const dim3 grid(static_cast<unsigned>(g.units), static_cast<unsigned>(gp.row_ctas + ceil_div(a->cols, kLrGradCols)));
        if (a->rank <= 16) st = launch_pdl(k_lr_grad<2>, grid, kLrGradCols, lr_grad_smem(2), s, gp);
        else if (a->rank <= 32) st = launch_pdl(k_lr_grad<4>, grid, kLrGradCols, lr_grad_smem(4), s, gp);
        else if (a->rank <= 64) st = launch_pdl(k_lr_grad<8>, grid, kLrGradCols, lr_grad_smem(8), s, gp);
        else st = launch_pdl(k_lr_grad<16>, grid, kLrGradCols, lr_grad_smem(16), s, gp);
        const int64_t quads = (a->rows + a->cols) * (a->rank / 4);
        const dim3 jgrid(static_cast<unsigned>(std::min<int64_t>(ceil_div(quads, 256), 2 * kAtOnce)), static_cast<unsigned>(a->n));
        if (st == E8Q_OK) st = launch_pdl(k_lr_join, jgrid, 256, 0, s, gp);
    }
    if (st == E8Q_OK && grad_x)
        st = launch_up<true>(*a, slots, a->a, grad_x_base, grad_x, nullptr, a->cols, a->rows, tokens, g, l, w, s);
    return st;
}

}  // extern "C"

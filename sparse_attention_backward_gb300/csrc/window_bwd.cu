// Windowed attention, gradient: launches of k_xdkv and k_xdq (xbwd.cuh) over the tiles that a window reaches.
//
// k_xdkv goes first, since its units are longer, and k_xdq does not wait for it:
// both need only k_xpre, which is complete once k_xdkv lets the next kernel's
// CTAs in.  They start as k_xdkv's leave, and take units by ticket, so the one's
// last, unfilled round is filled by the other.
//
// fp16: dS is rounded to 11 bits with an exponent for each row that it is summed
// into, which keeps 2^e |dS| <= 2^15 (|dS| <= |dP - Delta|):
//     dQ of row i    |dY_i| max |V_j| + |Delta_i|        over the keys j that i sees
//     dK of key j    max |dY_i| |V_j| + max |Delta_i|    over the rows i that see j
// With one for the whole sequence, rows out of reach took the bits of those within
// (8192 causal tokens, dY of the first 64 2^16 times the others': dK of the later
// half off by 0.6 %).  k_wscale forms them from norms that k_xpre leaves.
#include "xbwd.cuh"

namespace sag {

namespace {

constexpr int kScaleThreads = kXRows;

// Largest of elements a + i .. b + i of a sequence of n for thread i, of two numbers each: `value(x)` of an element, `top(t)` of
// the `per` elements of tile t.  Collective; `s` has room for two for each thread.
template <class Value, class Top>
__device__ __forceinline__ float2 reach_max(int a, int b, int n, int per, float2 (*s)[kScaleThreads], Value &&value, Top &&top) {
    const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
    auto more = [](float2 x, float2 y) { return make_float2(fmaxf(x.x, y.x), fmaxf(x.y, y.y)); };
    auto at = [&](int x) { return x >= 0 && x < n ? value(x) : make_float2(0.f, 0.f); };
    float2 best = make_float2(0.f, 0.f);
    if (b - a < kScaleThreads) {                         // short: each for itself
        s[0][i] = at(a + i);
        s[1][i] = at(a + kScaleThreads + i);
        __syncthreads();
        for (int k = i; k <= i + b - a; ++k) best = more(best, s[k / kScaleThreads][k % kScaleThreads]);
        return best;
    }
    // what all have in common, a + 128 .. b: whole tiles, and the elements around them
    const int lo = max(a + kScaleThreads, 0), hi = min(b, n - 1);
    if (lo <= hi) {
        const int t0 = (lo + per - 1) / per, t1 = hi + 1 == n ? (n + per - 1) / per : (hi + 1) / per;
        if (t0 < t1) {
            for (int t = t0 + i; t < t1; t += kScaleThreads) best = more(best, top(t));
            for (int x = lo + i; x < t0 * per; x += kScaleThreads) best = more(best, at(x));
            for (int x = t1 * per + i; x <= hi; x += kScaleThreads) best = more(best, at(x));
        } else {
            for (int x = lo + i; x <= hi; x += kScaleThreads) best = more(best, at(x));
        }
    }
    // from a + i on before those, and up to b + i behind them
    float2 from = at(a + i), to = at(b + i);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float2 f = make_float2(__shfl_down_sync(0xffffffffu, from.x, o), __shfl_down_sync(0xffffffffu, from.y, o));
        const float2 t = make_float2(__shfl_up_sync(0xffffffffu, to.x, o), __shfl_up_sync(0xffffffffu, to.y, o));
        const float2 c = make_float2(__shfl_xor_sync(0xffffffffu, best.x, o), __shfl_xor_sync(0xffffffffu, best.y, o));
        if (lane + o < 32) from = more(from, f);
        if (lane >= o) to = more(to, t);
        best = more(best, c);
    }
    if (lane == 0) s[0][warp] = from, s[0][4 + warp] = best;
    if (lane == 31) s[1][warp] = to;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kScaleThreads / 32; ++w) {
        best = more(best, s[0][4 + w]);
        if (w > warp) best = more(best, s[0][w]);
        if (w < warp) best = more(best, s[1][w]);
    }
    return more(best, more(from, to));
}

// A block a tile of query rows or keys.  Latency: a launch and two or three dependent reads (4 x 1500 padded tokens, 24 / 8 heads of
// 128: the gradient 116 -> 120 us; 8192 tokens, 32 / 8 heads, a window of 512: 245 -> 250 us).
__global__ void __launch_bounds__(kScaleThreads) k_wscale(const __grid_constant__ XArgs A) {
    __shared__ float2 s[2][kScaleThreads];
    __shared__ float reached[kXRows];
    const int i = threadIdx.x, G = A.group, q_units = A.q_tiles * A.n2;
    auto finite = [](float x) { return x < INFINITY ? x : 0.f; };
    grid_wait();                                         // k_xpre's norms
    grid_next();
    if ((int)blockIdx.x < q_units) {
        const XUnit u = x_decode<&SeqRow::qtile0>(A, blockIdx.x);
        const int a = u.tile * A.tpt + u.seq.klen - u.seq.qlen - A.left, b = a + A.left + A.right;
        auto place = [&](int tile) { return (int64_t)(u.seq.ktile0 + tile) * A.n2 + u.head; };
        auto norm = [&](int key) {
            return make_float2(finite(A.key_norms[place(key / kXRows) * kXRows + key % kXRows]), 0.f);
        };
        // token i's keys
        reached[i] = reach_max(a, b, u.seq.klen, kXRows, s, norm, [&](int t) { return A.k_tops[place(t)]; }).x;
        __syncthreads();
        const float dy = finite(A.row_norms[u.tile_id * kXRows + i]), far = fabsf(A.stats[u.tile_id * 256 + kXRows + i]);
        A.q_up[u.tile_id * kXRows + i] = ds_exponent(sqrtf(dy) * sqrtf(reached[i / G]) + far);
    } else {
        const XUnit u = x_decode<&SeqRow::ktile0>(A, blockIdx.x - q_units);
        const int a = u.tile * kXRows - (u.seq.klen - u.seq.qlen) - A.right, b = a + A.right + A.left;
        auto place = [&](int tile) { return (int64_t)(u.seq.qtile0 + tile) * A.n2 + u.head; };
        auto token = [&](int tok) {
            const int tile = tok / A.tpt, row = (tok - tile * A.tpt) * G;
            const float *dy = A.row_norms + place(tile) * kXRows + row, *far = A.stats + place(tile) * 256 + kXRows + row;
            float2 most = make_float2(0.f, 0.f);
            for (int h = 0; h < G; ++h)
                most = make_float2(fmaxf(most.x, finite(dy[h])), fmaxf(most.y, finite(fabsf(far[h]))));
            return most;
        };
        const float2 most = reach_max(a, b, u.seq.qlen, A.tpt, s, token, [&](int t) { return A.q_tops[place(t)]; });
        const float v = finite(A.key_norms[u.tile_id * kXRows + i]);
        A.k_up[u.tile_id * kXRows + i] = ds_exponent(sqrtf(most.x) * sqrtf(v) + most.y);
    }
}

}  // namespace

cudaError_t launch_wscale(const XArgs &a, cudaStream_t s) {
    const int64_t ctas = ((int64_t)a.q_tiles + a.k_tiles) * a.n2;
    return ctas ? x_launch(k_wscale, (int)ctas, kScaleThreads, 1, 0, true, s, a) : cudaSuccess;
}

cudaError_t launch_wdq(const XArgs &a, const sca_io &io, const sca_desc &d, cudaStream_t s) {
    return launch_bwd<true>(a, io, d, false, true, s);
}

cudaError_t launch_wdkv(const XArgs &a, const sca_io &io, const sca_desc &d, cudaStream_t s) {
    // without query rows there is no kernel of this call before it
    return launch_bwd<true>(a, io, d, true, a.q_tiles > 0, s);
}

}  // namespace sag

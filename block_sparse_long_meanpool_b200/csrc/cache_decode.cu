// Decode step over the paged 4-bit cache (moba_cache_decode).
//
// One new query per (sequence, head), at the sequence's last held token: the own block
// c = (L - 1) / chunk is attended whole, the topk - 1 best earlier blocks by q . k_mean are
// routed (topk = 0: all of them), and out = softmax(scale q K^T) V over the union, with the held
// keys and values.  The query heads of a KV head are taken together, up to kRowHeads at a time (a
// "row"), so that a block that several of them attend to is read once.
//   cache_plan_kernel  one CTA per row: gate scores, the heads' choices, their union
//   cache_attn_kernel  one CTA per row: online softmax over the row's blocks
#include <climits>

#include "cache_internal.cuh"
#include "moba_internal.cuh"

namespace moba {
namespace cache {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;
constexpr int kWindow = 1024;  // blocks scored at a time

struct Row {
    int seq, g, h0, nh;  // sequence, KV head, first query head, query heads
};
__device__ __forceinline__ Row row_of(const View& c, const DecodeArgs& a, int r) {
    Row w;
    const int per = c.hkv * a.hgroups;
    w.seq = r / per;
    w.g = (r - w.seq * per) / a.hgroups;
    const int p = r - w.seq * per - w.g * a.hgroups;
    w.h0 = w.g * a.group + p * kRowHeads;
    w.nh = min(kRowHeads, a.group - p * kRowHeads);
    return w;
}

// Tokens of a sequence, 0 where the length is out of range.
__device__ __forceinline__ int held_tokens(const View& c, int seq) {
    const int L = __ldg(c.lengths + seq);
    return L < 0 || L > (long long)c.max_blocks * c.chunk ? 0 : L;
}

// items[row] lists the row's blocks ascending, the own block last, as (page, heads that attend);
// counts[row] is their number (0: an empty sequence, whose outputs are written here).
template <int D, int K>
__global__ void __launch_bounds__(kThreads) cache_plan_kernel(View c, DecodeArgs a, DecodeWs ws) {
    constexpr int V = D / 32;
    __shared__ float qs[kRowHeads][D];
    __shared__ float score[kRowHeads][kWindow];
    __shared__ int pick[kRowHeads * 32];
    const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Row w = row_of(c, a, r);
    const int L = held_tokens(c, w.seq);
    if (L == 0) {
        if (tid == 0) {
            ws.counts[r] = 0;
            if (__ldg(c.lengths + w.seq) != 0) report(c, MOBA_ERR_INVALID_ARG);
        }
        for (int i = tid; i < w.nh * D; i += kThreads)
            a.out[((size_t)w.seq * a.hq + w.h0) * D + i] = __float2bfloat16(0.f);
        if (tid < w.nh) a.lse[(size_t)(w.h0 + tid) * c.seqs + w.seq] = -INFINITY;
        return;
    }
    const int own = (L - 1) / c.chunk;
    const int* row = c.table + (size_t)w.seq * c.max_blocks;
    int2* items = ws.items + (size_t)r * a.max_items;
    const int all = (1 << w.nh) - 1;
    const int n_route = min(a.topk - 1, own);
    if (a.topk == 0 || n_route == own) {  // every block
        if (tid == 0) ws.counts[r] = own + 1;
        if (a.topk)
            for (int j = tid; j <= own; j += kThreads) items[j] = make_int2(__ldg(row + j), all);
        return;
    }
    for (int i = tid; i < kRowHeads * D; i += kThreads) {
        const int h = i / D;
        qs[h][i - h * D] = h < w.nh ? __bfloat162float(a.q[((size_t)w.seq * a.hq + w.h0) * D + i]) : 0.f;
    }
    float val[K];
    int idx[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        val[i] = -INFINITY;
        idx[i] = INT_MAX;
    }
    for (int j0 = 0; j0 < own; j0 += kWindow) {
        const int n = min(kWindow, own - j0);
        __syncthreads();
        for (int j = warp; j < n; j += kThreads / 32) {
            const int page = __ldg(row + j0 + j);
            const bool ok = page >= 0 && page < c.pages;
            float s[kRowHeads];
#pragma unroll
            for (int h = 0; h < kRowHeads; ++h) s[h] = 0.f;
            if (ok) {
                const float* m = c.mean + ((size_t)page * c.hkv + w.g) * D + lane * V;
                float x[V];
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = __ldg(m + i);
#pragma unroll
                for (int h = 0; h < kRowHeads; ++h)
#pragma unroll
                    for (int i = 0; i < V; ++i) s[h] = fmaf(qs[h][lane * V + i], x[i], s[h]);
            }
#pragma unroll
            for (int h = 0; h < kRowHeads; ++h) {
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) s[h] += __shfl_xor_sync(0xffffffffu, s[h], off);
                // a NaN, and a page that is not there, ranks last
                if (lane == 0) score[h][j] = ok && s[h] == s[h] ? s[h] : -INFINITY;
            }
        }
        __syncthreads();
        for (int j = lane; j < n; j += 32) insert_ordered<K>(val, idx, score[warp][j], j0 + j);
    }
    // warp = head: n_route rounds of a warp argmax over the lists' heads, (score desc, block asc)
    for (int i = 0; i < n_route; ++i) {
        float bv = val[0];
        int bi = idx[0];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, off);
            const int oi = __shfl_xor_sync(0xffffffffu, bi, off);
            if (ov > bv || (ov == bv && oi < bi)) {
                bv = ov;
                bi = oi;
            }
        }
        if (idx[0] == bi) {
#pragma unroll
            for (int k = 0; k + 1 < K; ++k) {
                val[k] = val[k + 1];
                idx[k] = idx[k + 1];
            }
            val[K - 1] = -INFINITY;
            idx[K - 1] = INT_MAX;
        }
        if (lane == 0) pick[warp * n_route + i] = bi;
    }
    __syncthreads();
    // union of the heads' choices: a block's first mention leads; it counts the leaders before it
    const int n = w.nh * n_route;
    __shared__ int lead[kRowHeads * 32];
    int mine = -1, mask = 0;
    if (tid < n) {
        mine = pick[tid];
        bool first = true;
        for (int i = 0; i < n; ++i)
            if (pick[i] == mine) {
                mask |= 1 << (i / n_route);
                first = first && i >= tid;
            }
        lead[tid] = first;
        if (!first) mine = -1;
    }
    __syncthreads();
    if (mine >= 0) {
        int at = 0;
        for (int i = 0; i < n; ++i) at += lead[i] && pick[i] < mine;
        items[at] = make_int2(__ldg(row + mine), mask);
    }
    const int leaders = __syncthreads_count(mine >= 0);
    if (tid == 0) {
        items[leaders] = make_int2(__ldg(row + own), all);
        ws.counts[r] = leaders + 1;
    }
}

// Held values of one tile (rows [t0, t0 + n) of a page) into xs[kTile][D + 1], fp32.
template <int D>
__device__ __forceinline__ void load_tile(const uint8_t* codes, const uint8_t* scales, int n, float* xs) {
    constexpr int kPerTok = D / kGroup;
    for (int i = threadIdx.x; i < n * kPerTok; i += kThreads) {
        const int t = i / kPerTok, grp = i - t * kPerTok;
        const uint2 w = *reinterpret_cast<const uint2*>(codes + (size_t)t * (D / 2) + grp * 8);
        const float s = f16x2_to_f32(e4m3x2_to_f16x2(scales[(size_t)t * kPerTok + grp])).x;
        uint32_t h[4];
        float* x = xs + t * (D + 1) + grp * kGroup;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            e2m1x8_to_f16x2(k ? w.y : w.x, h);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = f16x2_to_f32(h[j]);
                x[8 * k + 2 * j] = f.x * s;
                x[8 * k + 2 * j + 1] = f.y * s;
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) cache_attn_kernel(View c, DecodeArgs a, DecodeWs ws) {
    constexpr int kSub = kThreads / D, kPer = kRowHeads / kSub;  // heads per thread of the value product
    __shared__ float qs[kRowHeads][D];
    __shared__ float xs[kTile * (D + 1)];
    __shared__ float ps[kRowHeads][kTile];
    __shared__ float alpha[kRowHeads];
    const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Row w = row_of(c, a, r);
    const int items = ws.counts[r];
    if (items == 0) return;
    const int L = held_tokens(c, w.seq), own = (L - 1) / c.chunk;
    for (int i = tid; i < kRowHeads * D; i += kThreads) {
        const int h = i / D;
        qs[h][i - h * D] =
            h < w.nh ? __bfloat162float(a.q[((size_t)w.seq * a.hq + w.h0) * D + i]) * a.scale_log2 : 0.f;
    }
    float m = -INFINITY, l = 0.f;  // of head `warp`
    float acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
    const int dim = tid % D, sub = tid / D;
    for (int it = 0; it < items; ++it) {
        const int2 item = a.topk ? ws.items[(size_t)r * a.max_items + it]
                                 : make_int2(__ldg(c.table + (size_t)w.seq * c.max_blocks + it), (1 << w.nh) - 1);
        const int tokens = it == items - 1 ? L - own * c.chunk : c.chunk;
        if (item.x < 0 || item.x >= c.pages) {
            if (tid == 0) report(c, MOBA_ERR_INVALID_ARG);
            continue;
        }
        const size_t cr = code_row(c, item.x, w.g), sr = scale_row(c, item.x, w.g);
        for (int t0 = 0; t0 < tokens; t0 += kTile) {
            const int n = min(kTile, tokens - t0);
            const size_t co = cr + (size_t)t0 * (D / 2), so = sr + (size_t)t0 * (D / kGroup);
            __syncthreads();
            load_tile<D>(c.kc + co, c.ks + so, n, xs);
            __syncthreads();
            for (int i = tid; i < kRowHeads * kTile; i += kThreads) {
                const int key = i % kTile, h = i / kTile;
                float s = 0.f;
                for (int e = 0; e < D; ++e) s = fmaf(qs[h][e], xs[key * (D + 1) + e], s);
                ps[h][key] = key < n && (item.y >> h & 1) ? s : -INFINITY;
            }
            __syncthreads();
            load_tile<D>(c.vc + co, c.vs + so, n, xs);
            {
                const float x = ps[warp][lane], y = ps[warp][lane + 32];
                float top = fmaxf(x, y);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
                const float al = exp2f(m - ref), px = exp2f(x - ref), py = exp2f(y - ref);
                float ts = px + py;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) ts += __shfl_xor_sync(0xffffffffu, ts, off);
                ps[warp][lane] = px;
                ps[warp][lane + 32] = py;
                l = l * al + ts;
                m = mn;
                if (lane == 0) alpha[warp] = al;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int h = sub * kPer + i;
                float o = acc[i] * alpha[h];
                for (int k = 0; k < n; ++k) o = fmaf(ps[h][k], xs[k * (D + 1) + dim], o);
                acc[i] = o;
            }
        }
    }
    __syncthreads();
    if (lane == 0) {
        ps[0][warp] = l > 0.f ? c.v_unit / l : l == 0.f ? 0.f : l;
        if (warp < w.nh)
            a.lse[(size_t)(w.h0 + warp) * c.seqs + w.seq] = m * 0.69314718055994531f + logf(l);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int h = sub * kPer + i;
        if (h < w.nh)
            a.out[((size_t)w.seq * a.hq + w.h0 + h) * D + dim] = __float2bfloat16_rn(acc[i] * ps[0][h]);
    }
}

template <int D>
cudaError_t launch_decode_d(const View& c, const DecodeArgs& a, const DecodeWs& ws, cudaStream_t st) {
    const int route = a.topk - 1;
    if (route <= 4)
        cache_plan_kernel<D, 4><<<a.rows, kThreads, 0, st>>>(c, a, ws);
    else if (route <= 8)
        cache_plan_kernel<D, 8><<<a.rows, kThreads, 0, st>>>(c, a, ws);
    else if (route <= 16)
        cache_plan_kernel<D, 16><<<a.rows, kThreads, 0, st>>>(c, a, ws);
    else
        cache_plan_kernel<D, 32><<<a.rows, kThreads, 0, st>>>(c, a, ws);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cache_attn_kernel<D><<<a.rows, kThreads, 0, st>>>(c, a, ws);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode(const View& c, const DecodeArgs& a, const DecodeWs& ws, cudaStream_t st) {
    return c.d == 64 ? launch_decode_d<64>(c, a, ws, st) : launch_decode_d<128>(c, a, ws, st);
}

}  // namespace cache
}  // namespace moba

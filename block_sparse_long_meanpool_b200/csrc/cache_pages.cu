// The page operators of the 4-bit cache: reserve, fork, free and compact.
//
// They read and write the int32 tables on the device, so a serving loop never waits for the
// host.  Free pages are those with refs = 0; a call takes the lowest ones in the order of its
// requests, so its result does not depend on timing.  Reserve, fork and compact are all or
// nothing: one CTA checks everything, finds the pages and leaves a verdict in the workspace,
// and only then is the cache written.  The planning CTAs are bound by the latency of a few dependent
// loads (4 to 8 us); the copies stream: 1024 pages of 577 KB are packed in 197 us, 6.2 TB/s.
#include "cache_internal.cuh"

namespace moba {
namespace cache {

namespace {

constexpr int kPlan = 1024;     // threads of the planning CTA
constexpr int kThreads = 256;
constexpr int kCopyTokens = 256;  // tokens of a page that one copying CTA takes

// Workspace words: [0] verdict (1: go ahead), [1] a count, from 64 on the call's lists.
constexpr int kVerdict = 0, kCount = 1, kLists = 64;

// Exclusive prefix sum over the CTA's threads of x; *total receives the sum.  All threads call it.
template <class T>
__device__ __forceinline__ T block_scan(T x, T* total) {
    __shared__ T warp_sum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        T s = lane < (int)(blockDim.x >> 5) ? warp_sum[lane] : T(0);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += y;
        }
        warp_sum[lane] = s;
    }
    __syncthreads();
    const T before = warp ? warp_sum[warp - 1] : T(0);
    *total = warp_sum[31];
    __syncthreads();
    return before + incl - x;
}

// The lowest `need` free pages into list[0 .. need); false when there are fewer.
__device__ __forceinline__ bool find_free(const View& c, int need, int* list) {
    int found = 0;
    for (int p0 = 0; p0 < c.pages && found < need; p0 += kPlan) {
        const int p = p0 + threadIdx.x;
        const int free = p < c.pages && c.refs[p] == 0;
        int n;
        const int at = found + block_scan(free, &n);
        if (free && at < need) list[at] = p;
        found += n;
    }
    return found >= need;
}

// Pages that sequence i holds: the first entries of its row, without gaps.
__device__ __forceinline__ int pages_held(const View& c, int i) {
    const int* row = c.table + (size_t)i * c.max_blocks;
    int lo = 0, hi = c.max_blocks;  // answer in [lo, hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (row[mid] >= 0) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// ws lists: held [seqs], first [seqs + 1], free pages [<= pages].
__global__ void __launch_bounds__(kPlan) reserve_kernel(View c, const int* __restrict__ upto, int* ws) {
    __shared__ int s_bad;
    int *held = ws + kLists, *first = held + c.seqs, *list = first + c.seqs + 1;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    long long total = 0;
    for (int i0 = 0; i0 < c.seqs; i0 += kPlan) {
        const int i = i0 + threadIdx.x;
        long long need = 0;  // up to max_blocks, so the CTA's sum may pass 32 bits
        if (i < c.seqs) {
            const int u = upto[i];
            if (u < 0 || u > c.max_blocks * (long long)c.chunk) {
                s_bad = MOBA_ERR_INVALID_ARG;
            } else {
                const int h = pages_held(c, i);
                held[i] = h;
                need = max(0LL, ((long long)u + c.chunk - 1) / c.chunk - h);
            }
        }
        long long n;
        const long long before = block_scan(need, &n);
        if (i < c.seqs) first[i] = (int)min(total + before, 0x7fffffffLL);
        total += n;
    }
    const bool fits = total <= c.pages, args_ok = !s_bad;
    __syncthreads();
    if (args_ok && (!fits || !find_free(c, (int)total, list))) {
        __syncthreads();
        if (threadIdx.x == 0) s_bad = MOBA_ERR_NO_PAGES;
    }
    __syncthreads();
    if (s_bad) {
        if (threadIdx.x == 0) report(c, s_bad);
        return;
    }
    for (int r = threadIdx.x; r < (int)total; r += kPlan) {
        int lo = 0, hi = c.seqs;  // the last sequence whose first request is <= r
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= r) lo = mid; else hi = mid;
        }
        const int page = list[r];
        c.table[(size_t)lo * c.max_blocks + held[lo] + r - first[lo]] = page;
        c.refs[page] = 1;
    }
}

// ws lists: length of the source [n], copied page's number among the copies or -1 [n], free pages.
__global__ void __launch_bounds__(kPlan)
fork_plan_kernel(View c, const int* __restrict__ src, const int* __restrict__ dst, int n, int* ws) {
    __shared__ unsigned named[65536 / 32];
    __shared__ int s_bad;
    int *len = ws + kLists, *copy = len + n, *list = copy + n;
    cudaTriggerProgrammaticLaunchCompletion();
    for (int i = threadIdx.x; i < (c.seqs + 31) / 32; i += kPlan) named[i] = 0;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    int copies = 0;
    for (int i0 = 0; i0 < n; i0 += kPlan) {
        const int i = i0 + threadIdx.x;
        int part = 0;
        bool bad = false;
        if (i < n) {
            const int a = src[i], b = dst[i];
            int L = 0;
            if (a < 0 || a >= c.seqs || b < 0 || b >= c.seqs || a == b) {
                bad = true;
            } else {
                L = c.lengths[a];
                bad = L < 0 || L > c.max_blocks * (long long)c.chunk || c.lengths[b] != 0 ||
                      c.table[(size_t)b * c.max_blocks] != -1 ||
                      (atomicOr(&named[b >> 5], 1u << (b & 31)) >> (b & 31) & 1u);
            }
            len[i] = L;
            part = !bad && L % c.chunk > 0;
        }
        int m;
        const int at = copies + block_scan(part, &m);
        if (i < n) copy[i] = part ? at : -1;
        copies += m;
        if (bad) s_bad = MOBA_ERR_INVALID_ARG;
    }
    __syncthreads();
    const bool named_ok = !s_bad;
    __syncthreads();
    if (named_ok)  // every page of every source is in range and in use
        for (int i = threadIdx.x >> 5; i < n; i += kPlan / 32)
            for (int j = threadIdx.x & 31; j < (len[i] + c.chunk - 1) / c.chunk; j += 32) {
                const int p = c.table[(size_t)src[i] * c.max_blocks + j];
                if (p < 0 || p >= c.pages || c.refs[p] <= 0) s_bad = MOBA_ERR_INVALID_ARG;
            }
    __syncthreads();
    const bool pages_ok = !s_bad;
    __syncthreads();
    if (pages_ok && (copies > c.pages || !find_free(c, copies, list))) {
        __syncthreads();
        if (threadIdx.x == 0) s_bad = MOBA_ERR_NO_PAGES;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        ws[kVerdict] = !s_bad;
        if (s_bad) report(c, s_bad);
    }
}

// Tokens [t0, t1) of head g of one page to another, t0 a multiple of kCopyTokens: codes and scales
// of keys and values.  A thread has kAhead 16-byte loads in flight before it stores; a token's
// scales are 4 or 8 bytes, so a last piece of up to 12 bytes is copied by words.
__device__ __forceinline__ void copy_tokens(const View& to, int q, const View& from, int p, int g, int t0, int t1) {
    constexpr int kAhead = 5;
    const int n = t1 - t0, cb = n * (from.d / 2) / 16, sb = n * (from.d / kGroup) / 16;  // whole pieces
    const size_t cf = code_row(from, p, g) + (size_t)t0 * (from.d / 2), ct = code_row(to, q, g) + (size_t)t0 * (from.d / 2);
    const size_t sf = scale_row(from, p, g) + (size_t)t0 * (from.d / kGroup);
    const size_t st = scale_row(to, q, g) + (size_t)t0 * (from.d / kGroup);
    const uint4* src[4] = {reinterpret_cast<const uint4*>(from.kc + cf), reinterpret_cast<const uint4*>(from.vc + cf),
                           reinterpret_cast<const uint4*>(from.ks + sf), reinterpret_cast<const uint4*>(from.vs + sf)};
    uint4* dst[4] = {reinterpret_cast<uint4*>(to.kc + ct), reinterpret_cast<uint4*>(to.vc + ct),
                     reinterpret_cast<uint4*>(to.ks + st), reinterpret_cast<uint4*>(to.vs + st)};
    const int all = 2 * (cb + sb);
    auto where = [&](int i, int& which) {  // the i-th piece
        which = i < cb ? 0 : i < 2 * cb ? 1 : i < 2 * cb + sb ? 2 : 3;
        return which == 0 ? i : which == 1 ? i - cb : which == 2 ? i - 2 * cb : i - 2 * cb - sb;
    };
    for (int i0 = threadIdx.x; i0 < all; i0 += kThreads * kAhead) {
        uint4 x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * kThreads;
            int which;
            const int at = where(i, which);
            if (i < all) x[j] = __ldcs((which == 0 ? src[0] : which == 1 ? src[1] : which == 2 ? src[2] : src[3]) + at);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * kThreads;
            int which;
            const int at = where(i, which);
            if (i < all) (which == 0 ? dst[0] : which == 1 ? dst[1] : which == 2 ? dst[2] : dst[3])[at] = x[j];
        }
    }
    const int words = n * (from.d / kGroup) / 4 - 4 * sb;  // of each kind of scales
    if (threadIdx.x < 2 * words) {
        const bool v = threadIdx.x >= words;
        const int at = 4 * sb + threadIdx.x - (v ? words : 0);
        reinterpret_cast<uint32_t*>(v ? dst[3] : dst[2])[at] = reinterpret_cast<const uint32_t*>(v ? src[3] : src[2])[at];
    }
}

// CTA (pair, head, slice): the slice's tokens of the pair's partial page; slice 0 of head 0 also
// writes the row, the references and the length.
__global__ void __launch_bounds__(kThreads)
fork_kernel(View c, const int* __restrict__ src, const int* __restrict__ dst, int n, const int* __restrict__ ws) {
    cudaGridDependencySynchronize();
    if (!__ldcg(ws + kVerdict)) return;
    const int *len = ws + kLists, *copy = len + n, *list = copy + n;
    const int i = blockIdx.x, g = blockIdx.y, z = blockIdx.z;
    const int L = len[i], full = L / c.chunk, rest = L % c.chunk;
    const int* from = c.table + (size_t)src[i] * c.max_blocks;
    const int page = rest ? list[copy[i]] : -1;
    if (g == 0 && z == 0) {
        int* to = c.table + (size_t)dst[i] * c.max_blocks;
        for (int j = threadIdx.x; j < c.max_blocks; j += kThreads) {
            int p = -1;
            if (j < full) {
                p = from[j];
                atomicAdd(c.refs + p, 1);
            } else if (j == full && rest) {
                p = page;
                c.refs[p] = 1;
            }
            to[j] = p;
        }
        if (threadIdx.x == 0) c.lengths[dst[i]] = L;
    }
    const int t0 = z * kCopyTokens, t1 = min(rest, t0 + kCopyTokens);
    if (t0 < t1) copy_tokens(c, page, c, from[full], g, t0, t1);
}

__global__ void __launch_bounds__(kThreads) free_kernel(View c, const int* __restrict__ seqs) {
    const int i = seqs[blockIdx.x];
    if (i < 0 || i >= c.seqs) {
        if (threadIdx.x == 0) report(c, MOBA_ERR_INVALID_ARG);
        return;
    }
    int* row = c.table + (size_t)i * c.max_blocks;
    for (int j = threadIdx.x; j < c.max_blocks; j += kThreads) {
        if (row[j] == -1) continue;
        const int p = atomicExch(row + j, -1);  // a slot named twice finds its row empty
        if (p < 0) continue;
        if (p >= c.pages)
            report(c, MOBA_ERR_INVALID_ARG);
        else
            atomicSub(c.refs + p, 1);
    }
    if (threadIdx.x == 0) c.lengths[i] = 0;
}

// ws lists: the page's new number or -1 [pages].
__global__ void __launch_bounds__(kPlan) compact_plan_kernel(View c, View to, int* ws) {
    cudaTriggerProgrammaticLaunchCompletion();
    int* name = ws + kLists;
    int live = 0;
    for (int p0 = 0; p0 < c.pages; p0 += kPlan) {
        const int p = p0 + threadIdx.x;
        const int used = p < c.pages && c.refs[p] > 0;
        int n;
        const int at = live + block_scan(used, &n);
        if (p < c.pages) name[p] = used ? at : -1;
        live += n;
    }
    if (threadIdx.x == 0) {
        ws[kVerdict] = live <= to.pages;
        ws[kCount] = live;
        if (live > to.pages) report(c, MOBA_ERR_NO_PAGES);
    }
}

// CTA (page, head, slice) copies; CTAs behind the pages write the tables.
__global__ void __launch_bounds__(kThreads) compact_kernel(View c, View to, const int* __restrict__ ws) {
    cudaGridDependencySynchronize();
    if (!__ldcg(ws + kVerdict)) return;
    const int* name = ws + kLists;
    const int p = blockIdx.x, g = blockIdx.y, z = blockIdx.z;
    if (p < c.pages) {
        const int q = name[p];
        if (q < 0) return;
        if (z == 0) {
            if (g == 0 && threadIdx.x == 0) to.refs[q] = c.refs[p];
            for (int i = threadIdx.x; i < c.d; i += kThreads)
                to.mean[((size_t)q * c.hkv + g) * c.d + i] = c.mean[((size_t)p * c.hkv + g) * c.d + i];
        }
        const int t0 = z * kCopyTokens;
        copy_tokens(to, q, c, p, g, t0, min(c.chunk, t0 + kCopyTokens));
        return;
    }
    if (g || z) return;
    const long long tables = gridDim.x - c.pages, me = p - c.pages;
    const long long entries = (long long)c.seqs * c.max_blocks;
    for (long long j = me * kThreads + threadIdx.x; j < entries; j += tables * kThreads) {
        int q = c.table[j];
        if (q >= 0) {
            q = q < c.pages ? name[q] : -1;
            if (q < 0) report(c, MOBA_ERR_INVALID_ARG);
        }
        to.table[j] = q < 0 ? -1 : q;
    }
    for (long long i = me * kThreads + threadIdx.x; i < c.seqs; i += tables * kThreads) to.lengths[i] = c.lengths[i];
    for (long long i = ws[kCount] + me * kThreads + threadIdx.x; i < to.pages; i += tables * kThreads) to.refs[i] = 0;
}

}  // namespace

cudaError_t launch_reserve(const View& c, const int* upto, int* ws, cudaStream_t st) {
    reserve_kernel<<<1, kPlan, 0, st>>>(c, upto, ws);
    return cudaGetLastError();
}

cudaError_t launch_fork(const View& c, const int* src, const int* dst, int n, int* ws, cudaStream_t st) {
    fork_plan_kernel<<<1, kPlan, 0, st>>>(c, src, dst, n, ws);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int slices = (c.chunk + kCopyTokens - 1) / kCopyTokens;
    return launch_early(fork_kernel, dim3(n, c.hkv, slices), kThreads, 0, st, c, src, dst, n, (const int*)ws);
}

cudaError_t launch_free(const View& c, const int* seqs, int n, cudaStream_t st) {
    free_kernel<<<n, kThreads, 0, st>>>(c, seqs);
    return cudaGetLastError();
}

cudaError_t launch_compact(const View& c, const View& into, int* ws, cudaStream_t st) {
    compact_plan_kernel<<<1, kPlan, 0, st>>>(c, into, ws);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int slices = (c.chunk + kCopyTokens - 1) / kCopyTokens;
    const int tables = 16;
    return launch_early(compact_kernel, dim3(c.pages + tables, c.hkv, slices), kThreads, 0, st, c, into, (const int*)ws);
}

}  // namespace cache
}  // namespace moba

// Pages of the 4-bit cache: room for new tokens with copy on write, branches,
// freeing, compaction.  All state is on the device and every call is a fixed
// number of launches, so a decode step that allocates can be captured.
//
// A page is free iff its reference count is 0.  The bookkeeping is done by one
// workgroup that walks the reference counts in ascending order, 16 a thread
// (16384 pages a step), so the pages handed out are those of lowest index
// whatever the timing: a few microseconds of latency for pools of that size.
// The payload is copied by a second launch over all compute units, bound by HBM
// (page bytes read and written once: 106 MB in 21 us, 5 TB/s).
#include "attn.h"

namespace moedec {
namespace attn {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kPer = 16;                           // reference counts per thread and step
constexpr int kStep = kThreads * kPer;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopyPart = kCopyThreads * 16 * kCopyUnroll;   // bytes a workgroup copies at a time
constexpr int kCopyGrid = 2048;

// Inclusive sums over the workgroup (every thread calls), the totals in `total`.
template <typename V>
__device__ __forceinline__ V block_scan(V v, V* total) {
    __shared__ V part[kWaves];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const V u = __shfl_up(v, o, kWave);
        if (lane >= o) v += u;
    }
    __syncthreads();                               // the last call's readers are done
    if (lane == kWave - 1) part[wave] = v;
    __syncthreads();
    V before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const V p = part[w];
        if (w < wave) before += p;
        all += p;
    }
    *total = all;
    return v + before;
}

// Bit k set: page p + k is free (pages past the pool are not).
__device__ __forceinline__ uint32_t free_mask(const Cache& c, int p) {
    uint32_t m = 0;
    if (p + kPer <= c.n_pages) {
        const int4* r = reinterpret_cast<const int4*>(c.ref + p);
#pragma unroll
        for (int i = 0; i < kPer / 4; ++i) {
            const int4 v = r[i];
            m |= (uint32_t)((v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3) << (4 * i);
        }
    } else {
        for (int k = 0; k < kPer && p + k < c.n_pages; ++k) m |= (uint32_t)(c.ref[p + k] == 0) << k;
    }
    return m;
}

// One thread per sequence.  The copies to make: ws[0] their number, then the
// source pages, then (from 1 + n_seqs) the destinations.  The first step of the
// free pages is read at once, beside the lengths: with up to 16384 pages the call
// waits for memory three times and scans once.
__global__ __launch_bounds__(kThreads) void kv4_reserve_kernel(Cache c, const int32_t* __restrict__ n_new,
                                                               int32_t* __restrict__ granted, int32_t* __restrict__ ws) {
    __shared__ int4 part_page4[kThreads / 4];      // the shared, partly filled page a sequence is to write, or -1
    __shared__ int64_t end_of[kThreads];           // pages asked for by sequences 0 .. s
    __shared__ int place[kThreads];                // table column of the sequence's first place
    __shared__ int list[kStep];                    // the free pages of a step
    __shared__ int copies[kThreads];               // the sequence's place in the list of copies, or -1
    __shared__ int refused, any_shared;
    int* part_page = reinterpret_cast<int*>(part_page4);
    const int s = threadIdx.x, pt = c.page_tokens(), cap = c.max_pages << c.pt_log2;
    const uint32_t mask0 = free_mask(c, min(s * kPer, c.n_pages));
    int len = 0, grow = 0, have = 0, want = 0, last = -1, refs = 0;
    if (s == 0) {
        refused = kThreads;
        any_shared = 0;
    }
    if (s < c.n_seqs) {
        len = c.held(s);
        grow = max(n_new[s], 0);
        if (grow > cap - len) grow = 0;
        have = (len + pt - 1) >> c.pt_log2;
        want = grow > 0 ? (len + grow + pt - 1) >> c.pt_log2 : have;
        if (grow > 0 && (len & (pt - 1))) {
            last = c.table[(int64_t)s * c.max_pages + have - 1];
            refs = c.good(last) ? c.ref[last] : 0;
        }
    }
    part_page[s] = refs > 1 ? last : -1;
    __syncthreads();
    if (refs > 1) any_shared = 1;
    __syncthreads();
    // of those that share a page and grow, every one but the last copies it
    bool cow = false;
    if (any_shared && refs > 1) {
        int before = 0;
        for (int j = 0; j < s; j += 4) {
            const int4 v = part_page4[j / 4];
            before += (v.x == last) + (j + 1 < s && v.y == last) + (j + 2 < s && v.z == last) +
                      (j + 3 < s && v.w == last);
        }
        cow = refs - before > 1;
    }
    // one scan: pages asked for (under 2^36) and, above them, the copies among them
    const int need = want - have + (cow ? 1 : 0);
    int64_t sums;
    const int64_t scan = block_scan<int64_t>((int64_t)need | (int64_t)cow << 48, &sums);
    const int64_t end = scan & ((1ll << 48) - 1), total = sums & ((1ll << 48) - 1);
    const int copies_to = (int)(scan >> 48);       // copies of sequences 0 .. s
    end_of[s] = end;
    place[s] = have - (cow ? 1 : 0);
    // enough free pages?
    int got, first0 = 0, first_got = 0;
    int64_t found = 0;
    for (int base = 0; base < c.n_pages && found < total; base += kStep) {
        const uint32_t m = base == 0 ? mask0 : free_mask(c, min(base + s * kPer, c.n_pages));
        const int f = block_scan<int>(__popc(m), &got);
        if (base == 0) {
            first0 = f;
            first_got = got;
        }
        found += got;
    }
    if (grow > 0 && end > found) atomicMin(&refused, s);
    __syncthreads();
    const bool go = grow > 0 && s < refused;
    const int64_t served = refused < kThreads ? (refused > 0 ? end_of[refused - 1] : 0) : total;
    copies[s] = go && cow ? copies_to - 1 : -1;
    if (s == (refused < kThreads ? refused : kThreads - 1)) ws[0] = copies_to - (refused < kThreads && cow ? 1 : 0);
    __syncthreads();
    // Free page number f (ascending) goes to the first sequence whose end is past f.
    // A step's free pages go to a list first: they lie in runs, and a thread that
    // searched for all sixteen of its own would keep the workgroup waiting.
    int64_t seen = 0;
    for (int base = 0; base < c.n_pages && seen < served; base += kStep) {
        const int p = min(base + s * kPer, c.n_pages);
        uint32_t m = base == 0 ? mask0 : free_mask(c, p);
        const int pop = __popc(m);
        int f = first0 - pop;
        got = first_got;
        if (base > 0) f = block_scan<int>(pop, &got) - pop;
        for (; m; m &= m - 1, ++f) list[f] = p + __ffs(m) - 1;
        __syncthreads();
        const int take = (int)min((int64_t)got, served - seen);
        for (int i = s; i < take; i += kThreads) {
            const int page = list[i];
            const int64_t at = seen + i;
            int lo = 0, hi = c.n_seqs - 1;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (end_of[mid] > at) hi = mid;
                else lo = mid + 1;
            }
            const int k = (int)(at - (lo > 0 ? end_of[lo - 1] : 0));
            if (k == 0 && copies[lo] >= 0) ws[1 + c.n_seqs + copies[lo]] = page;
            c.table[(int64_t)lo * c.max_pages + place[lo] + k] = page;
            c.ref[page] = 1;
        }
        __syncthreads();                           // the list is free again
        seen += got;
    }
    if (go && cow) {
        ws[1 + copies_to - 1] = last;
        atomicSub(c.ref + last, 1);
    }
    if (s < c.n_seqs) {
        granted[s] = go ? grow : 0;
        if (go) c.len[s] = len + grow;
    }
}

// Copies the pages src[i] -> dst[i], i < n, in every layer.
__device__ __forceinline__ void copy_pages(const Cache& c, int n, const int32_t* src, const int32_t* dst) {
    const int64_t bytes = c.page_bytes();
    const int parts = (int)((bytes + kCopyPart - 1) / kCopyPart);
    const int64_t jobs = (int64_t)n * c.layers * parts;
    for (int64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
        const int part = (int)(j % parts), layer = (int)(j / parts % c.layers), i = (int)(j / parts / c.layers);
        const int a = src[i], b = dst[i];
        const u32x4* from = reinterpret_cast<const u32x4*>(c.unit(layer, a, 0) + (int64_t)part * kCopyPart);
        u32x4* to = reinterpret_cast<u32x4*>(c.unit(layer, b, 0) + (int64_t)part * kCopyPart);
        const int64_t rest = bytes - (int64_t)part * kCopyPart;
        const int words = (int)((rest < kCopyPart ? rest : kCopyPart) / 16);
        u32x4 v[kCopyUnroll];
#pragma unroll
        for (int k = 0; k < kCopyUnroll; ++k) {
            const int w = threadIdx.x + k * kCopyThreads;
            if (w < words) v[k] = __builtin_nontemporal_load(from + w);
        }
#pragma unroll
        for (int k = 0; k < kCopyUnroll; ++k) {
            const int w = threadIdx.x + k * kCopyThreads;
            if (w < words) __builtin_nontemporal_store(v[k], to + w);
        }
    }
}

__global__ __launch_bounds__(kCopyThreads) void kv4_copy_kernel(Cache c, const int32_t* __restrict__ ws, int stride) {
    copy_pages(c, ws[0], ws + 1, ws + 1 + stride);
}

// Checks every entry against the state before the call; the lengths of the
// accepted ones are written once all are read.
__global__ __launch_bounds__(kThreads) void kv4_fork_check(Cache c, int n, const int32_t* __restrict__ src,
                                                           const int32_t* __restrict__ dst,
                                                           const int32_t* __restrict__ n_tokens,
                                                           int32_t* __restrict__ ok) {
    __shared__ int first[KV4_MAX_SEQS];            // the first entry that names a slot
    const int i = threadIdx.x;
    first[i] = kThreads;
    __syncthreads();
    int a = -1, b = -1, keep = 0;
    bool good = false;
    if (i < n) {
        a = src[i];
        b = dst[i];
        if ((unsigned)b < (unsigned)c.n_seqs) atomicMin(&first[b], i);
    }
    __syncthreads();
    if (i < n && (unsigned)a < (unsigned)c.n_seqs && (unsigned)b < (unsigned)c.n_seqs) {
        const int have = c.held(a);
        keep = n_tokens ? n_tokens[i] : have;
        good = first[b] == i && c.len[b] == 0 && keep >= 0 && keep <= have;
    }
    __syncthreads();
    if (i < n) {
        ok[i] = good;
        if (good) c.len[b] = keep;
    }
}

__global__ __launch_bounds__(kCopyThreads) void kv4_fork_pages(Cache c, const int32_t* __restrict__ src,
                                                               const int32_t* __restrict__ dst,
                                                               const int32_t* __restrict__ ok) {
    const int i = blockIdx.x;
    if (!ok[i]) return;
    const int64_t a = (int64_t)src[i] * c.max_pages, b = (int64_t)dst[i] * c.max_pages;
    const int pages = (c.held(dst[i]) + c.page_tokens() - 1) >> c.pt_log2;
    for (int p = threadIdx.x; p < pages; p += kCopyThreads) {
        const int page = c.table[a + p];
        c.table[b + p] = page;
        if (c.good(page)) atomicAdd(c.ref + page, 1);
    }
}

__global__ __launch_bounds__(kCopyThreads) void kv4_truncate_kernel(Cache c, const int32_t* __restrict__ new_len) {
    const int s = blockIdx.x, pt = c.page_tokens(), len = c.held(s), keep = new_len[s];
    if (keep < 0 || keep >= len) return;
    const int from = (keep + pt - 1) >> c.pt_log2, to = (len + pt - 1) >> c.pt_log2;
    for (int p = from + threadIdx.x; p < to; p += kCopyThreads) {
        int32_t* e = c.table + (int64_t)s * c.max_pages + p;
        if (c.good(*e)) atomicSub(c.ref + *e, 1);
        *e = -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) c.len[s] = keep;
}

// ws[0] = pages to move, then their sources, then (from 1 + n_pages / 2) their
// destinations: at most min(live, free) <= n_pages / 2 of them.
__global__ __launch_bounds__(kThreads) void kv4_compact_plan(Cache c, int32_t* __restrict__ remap,
                                                             int32_t* __restrict__ n_live, int32_t* __restrict__ ws) {
    const int t = threadIdx.x;
    int32_t *src = ws + 1, *dst = ws + 1 + c.n_pages / 2;
    const uint32_t mask0 = free_mask(c, min(t * kPer, c.n_pages));
    int live = 0, got;
    for (int base = 0; base < c.n_pages; base += kStep) {
        const int p = min(base + t * kPer, c.n_pages);
        const int in = min(c.n_pages - p, kPer);
        block_scan<int>(in - __popc(base == 0 ? mask0 : free_mask(c, p)), &got);
        live += got;
    }
    int holes = 0, moves = 0;
    for (int base = 0; base < c.n_pages; base += kStep) {
        const int p = min(base + t * kPer, c.n_pages);
        const int in = min(c.n_pages - p, kPer);
        const uint32_t all = (1u << in) - 1, below = p >= live ? 0 : live - p >= in ? all : (1u << (live - p)) - 1;
        const uint32_t fr = base == 0 ? mask0 : free_mask(c, p);
        uint32_t hole = fr & below, move = ~fr & all & ~below;
        // both counts (at most 16384 a step) in one scan
        const int both = block_scan<int>(__popc(hole) | __popc(move) << 16, &got);
        int h = holes + (both & 0xFFFF) - __popc(hole);
        holes += got & 0xFFFF;
        int v = moves + (both >> 16) - __popc(move);
        moves += got >> 16;
        for (int k = 0; k < in; ++k) {
            remap[p + k] = fr >> k & 1 ? -1 : p + k;
            if (hole >> k & 1) dst[h++] = p + k;
            if (move >> k & 1) src[v++] = p + k;
        }
    }
    __syncthreads();                               // the lists are complete (one workgroup wrote them)
    for (int i = t; i < moves; i += kThreads) {
        const int a = src[i], b = dst[i];
        remap[a] = b;
        c.ref[b] = c.ref[a];
        c.ref[a] = 0;
    }
    if (t == 0) {
        ws[0] = moves;
        *n_live = live;
    }
}

__global__ __launch_bounds__(kCopyThreads) void kv4_compact_move(Cache c, const int32_t* __restrict__ remap,
                                                                 const int32_t* __restrict__ ws) {
    for (int s = blockIdx.x; s < c.n_seqs; s += gridDim.x) {
        const int pages = (c.held(s) + c.page_tokens() - 1) >> c.pt_log2;
        for (int p = threadIdx.x; p < pages; p += kCopyThreads) {
            int32_t* e = c.table + (int64_t)s * c.max_pages + p;
            if (c.good(*e)) *e = remap[*e];
        }
    }
    copy_pages(c, ws[0], ws + 1, ws + 1 + c.n_pages / 2);
}

}  // namespace

hipError_t launch_reserve(const Cache& c, const int32_t* n_new, int32_t* granted, int32_t* ws, hipStream_t st) {
    hipLaunchKernelGGL(kv4_reserve_kernel, dim3(1), dim3(kThreads), 0, st, c, n_new, granted, ws);
    hipLaunchKernelGGL(kv4_copy_kernel, dim3(kCopyGrid), dim3(kCopyThreads), 0, st, c, ws, c.n_seqs);
    return hipGetLastError();
}

hipError_t launch_fork(const Cache& c, int n, const int32_t* src, const int32_t* dst, const int32_t* n_tokens,
                       int32_t* ok, hipStream_t st) {
    if (n == 0) return hipSuccess;
    hipLaunchKernelGGL(kv4_fork_check, dim3(1), dim3(kThreads), 0, st, c, n, src, dst, n_tokens, ok);
    hipLaunchKernelGGL(kv4_fork_pages, dim3(n), dim3(kCopyThreads), 0, st, c, src, dst, ok);
    return hipGetLastError();
}

hipError_t launch_truncate(const Cache& c, const int32_t* new_len, hipStream_t st) {
    hipLaunchKernelGGL(kv4_truncate_kernel, dim3(c.n_seqs), dim3(kCopyThreads), 0, st, c, new_len);
    return hipGetLastError();
}

hipError_t launch_compact(const Cache& c, int32_t* remap, int32_t* n_live, int32_t* ws, hipStream_t st) {
    hipLaunchKernelGGL(kv4_compact_plan, dim3(1), dim3(kThreads), 0, st, c, remap, n_live, ws);
    hipLaunchKernelGGL(kv4_compact_move, dim3(kCopyGrid), dim3(kCopyThreads), 0, st, c, remap, ws);
    return hipGetLastError();
}

}  // namespace attn
}  // namespace moedec

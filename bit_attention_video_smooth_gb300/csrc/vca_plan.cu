// vca_plan.cu -- places for the cache's new tokens: pages for the columns that
// begin, lengths, the cut of a call's rows, and every row's slot and position; or
// fresh pages for an eviction.  Integers alone: what bounds it is latency, a few
// dependent loads and barriers.
//
// No list of free pages is kept: free is what no live table entry names, found
// anew where pages are given out.  So no page is lost or given out twice, a
// shared page stays while one sequence names it, and a length of 0 gives a
// sequence's pages back.  The lowest free pages go to the sequences in order, so that
// equal calls have equal answers.
//
// One cluster does it all in one launch: every CTA adds up all sequences' rows and
// pages for itself (that sum needs no exchange), marks its share of the table's
// entries in a bitmap of its own, and joins its share of the words of all bitmaps;
// a warp then hands out the free pages of a word, a lane a page.  Where no page is
// needed (most decode steps) there is no bitmap.
#include "vca_cache.cuh"

namespace vca {

namespace {

using namespace cache;

constexpr int kErrFull = 6;              // mirrors VCA_ERR_FULL
constexpr int kPer = 8;                  // groups a thread sums: of one sequence or, of more sequences, of a few each
constexpr int kAhead = 8;                // loads of table entries under way
constexpr int kSmem = 220 * 1024;        // for sums and bitmap: 900,000 pages or more at a time
constexpr uint32_t kAll = 0xffffffffu;

struct PlanParams {
    PlanArgs a;
    int size, groups;                    // sequences of a group, and groups
    int words;                           // of a bitmap
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Also orders what its threads wrote to global memory before it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_read(const void *p, uint32_t rank) {
    uint32_t at, v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// Pages that hold n tokens.
__device__ __forceinline__ int up(int n) { return n / kBlk + (n % kBlk != 0); }

// What sequence b needs: new rows, the table columns [first, first + pages) that begin.
struct Need {
    int held, rows, first, pages;
    bool bad;
};
template <bool kFresh>
__device__ __forceinline__ Need need_of(const PlanArgs &a, int b) {
    Need n;
    n.held = a.held[b];
    n.rows = kFresh ? 0 : a.news[b];
    const int64_t most = static_cast<int64_t>(a.cols) * kBlk;
    n.bad = n.held < 0 || n.rows < 0 || static_cast<int64_t>(n.held) + n.rows > most;
    if (n.bad) return Need{0, 0, 0, 0, true};
    n.first = kFresh ? 0 : up(n.held);
    n.pages = kFresh ? up(min(n.held, a.budget)) : up(n.held + n.rows) - n.first;
    return n;
}

__device__ __forceinline__ int64_t warp_scan(int64_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += y;
    }
    return v;
}
// Sum over the threads before this one, and over all of them in `total`.
template <int kWarps>
__device__ __forceinline__ int64_t block_before(int64_t v, int64_t *red, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t incl = warp_scan(v);
    __syncthreads();
    if (lane == 31) red[warp] = incl;
    __syncthreads();
    const int64_t sums = warp_scan(lane < kWarps ? red[lane] : 0);
    total = __shfl_sync(kAll, sums, 31);
    const int64_t mine = __shfl_sync(kAll, sums, warp) - red[warp];
    return mine + incl - v;
}

// The last i with sum[i] <= x, of n + 1 rising sums that start with 0 <= x < sum[n].
__device__ __forceinline__ int find(const int *sum, int n, int x) {
    int a = 0, z = n;
    while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (sum[mid] <= x)
            a = mid;
        else
            z = mid;
    }
    return a;
}

template <bool kFresh, int kCluster, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) plan_kernel(const PlanParams p) {
    extern __shared__ int smem[];
    int *rows_to = smem, *pages_to = rows_to + p.groups + 1;                             // sums before each group
    int *held_s = pages_to + p.groups + 1;                                               // held, where a group is one sequence
    uint32_t *bits = reinterpret_cast<uint32_t *>(held_s + p.groups);                    // [words]: pages that are named
    int *free_to = reinterpret_cast<int *>(bits + p.words);                              // free pages before each of this CTA's words
    constexpr int kWarps = kThreads / 32;
    __shared__ int64_t red[32];
    __shared__ int free_here;

    const PlanArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = kCluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    auto everywhere = [&] {
        if constexpr (kCluster > 1)
            cluster_sync();
        else
            __syncthreads();
    };

    // rows and pages of all sequences, a run of groups a thread
    const bool single = p.size == 1;
    const int per = (p.groups + kThreads - 1) / kThreads, g0 = min(p.groups, tid * per), g1 = min(p.groups, g0 + per);
    int64_t rows = 0, pages = 0;
    bool bad = false;
    Need mine[kPer];      // of sequences g0 .. g1 - 1, where a group is one: their loads side by side
    if (single) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            mine[i] = Need{0, 0, 0, 0, false};
            if (g0 + i < g1) mine[i] = need_of<kFresh>(a, g0 + i);
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            rows += mine[i].rows;
            pages += mine[i].pages;
            bad |= mine[i].bad;
        }
    } else {
        for (int b = g0 * p.size; b < min(a.B, g1 * p.size); ++b) {
            const Need n = need_of<kFresh>(a, b);
            rows += n.rows;
            pages += n.pages;
            bad |= n.bad;
        }
    }
    int64_t all_rows, all_pages;
    int64_t row = block_before<kWarps>(rows, red, all_rows), page = block_before<kWarps>(pages, red, all_pages);
    int refused = __syncthreads_or(bad) || (!kFresh && all_rows > a.T) ? kErrInvalid : all_pages > a.pages ? kErrFull : 0;
    if (!refused) {
        if (single) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int b = g0 + i;
                if (b < g1) {
                    rows_to[b] = static_cast<int>(row);
                    pages_to[b] = static_cast<int>(page);
                    held_s[b] = mine[i].held;
                    if (!kFresh && rank == 0) a.start[b] = static_cast<int>(row);
                    row += mine[i].rows;
                    page += mine[i].pages;
                }
            }
        } else {
            for (int g = g0; g < g1; ++g) {
                rows_to[g] = static_cast<int>(row);
                pages_to[g] = static_cast<int>(page);
                for (int b = g * p.size; b < min(a.B, (g + 1) * p.size); ++b) {
                    const Need n = need_of<kFresh>(a, b);
                    if (!kFresh && rank == 0) a.start[b] = static_cast<int>(row);
                    row += n.rows;
                    page += n.pages;
                }
            }
        }
        if (tid == 0) {
            rows_to[p.groups] = static_cast<int>(all_rows);
            pages_to[p.groups] = static_cast<int>(all_pages);
            if (!kFresh && rank == 0) a.start[a.B] = static_cast<int>(all_rows);
        }
    }
    const int need = static_cast<int>(all_pages);
    __syncthreads();
    // Where the place `at` of group g's things lies, sum(b) of them a sequence: its sequence.
    auto within = [&](int g, int &at, auto sum) {
        if (single) return g;
        int b = g * p.size;
        for (int n; at >= (n = sum(b)); ++b) at -= n;
        return b;
    };

    if (!refused && need > 0) {
        const bool once = static_cast<int64_t>(p.words) * 32 >= a.pages;      // all pages in one window
        const int share = (p.words + kCluster - 1) / kCluster, word0 = min(p.words, rank * share), word1 = min(p.words, word0 + share);
        // pass 0 counts the free pages, pass 1 gives them out
        for (int pass = 0; pass < 2 && !refused; ++pass) {
            int taken = 0;
            for (int64_t from = 0; from < a.pages && taken < need; from += 32ll * p.words) {
                int64_t here = 0, before = 0;      // free pages of this window, and of it before this CTA's words
                if (pass == 0 || !once) {
                    for (int i = tid; i < p.words; i += kThreads) bits[i] = 0;
                    __syncthreads();
                    const int64_t window = 32ll * p.words;
                    auto mark = [&](int named) {
                        if (named < 0 || named >= a.pages)
                            report(a.dev_status, kErrInvalid);
                        else if (named >= from && named - from < window)
                            atomicOr(&bits[(named - from) >> 5], 1u << (named & 31));
                    };
                    const int warps = kCluster * kWarps, me = rank * kWarps + warp;
                    if (a.B < warps) {
                        // a few warps a sequence, a stride of 32 columns each
                        const int split = warps / a.B, b = me / split;
                        if (b < a.B) {
                            const int live = up(single ? held_s[b] : a.held[b]);
                            const int32_t *entries = a.table + static_cast<int64_t>(b) * a.cols;
                            for (int j = (me % split) * 32 + lane; j < live; j += kAhead * 32 * split) {
                                int named[kAhead];
#pragma unroll
                                for (int i = 0; i < kAhead; ++i)
                                    if (j + i * 32 * split < live) named[i] = entries[j + i * 32 * split];
#pragma unroll
                                for (int i = 0; i < kAhead; ++i)
                                    if (j + i * 32 * split < live) mark(named[i]);
                            }
                        }
                    } else {
                        // a warp's sequences, kAhead at a time
                        for (int b0 = me; b0 < a.B; b0 += kAhead * warps) {
                            int live[kAhead], named[kAhead], most = 0;
#pragma unroll
                            for (int i = 0; i < kAhead; ++i) {
                                const int b = b0 + i * warps;
                                live[i] = b < a.B ? up(single ? held_s[b] : a.held[b]) : 0;
                                most = max(most, live[i]);
                            }
                            for (int j = lane; j < most; j += 32) {
#pragma unroll
                                for (int i = 0; i < kAhead; ++i)
                                    if (j < live[i]) named[i] = a.table[static_cast<int64_t>(b0 + i * warps) * a.cols + j];
#pragma unroll
                                for (int i = 0; i < kAhead; ++i)
                                    if (j < live[i]) mark(named[i]);
                            }
                        }
                    }
                    everywhere();
                    // this CTA's words of all bitmaps; pages behind the last count as named
                    const int run = (word1 - word0 + kThreads - 1) / kThreads;
                    const int i0 = min(word1, word0 + tid * run), i1 = min(word1, i0 + run);
                    int free_mine = 0;
                    for (int i = i0; i < i1; ++i) {
                        uint32_t w = bits[i];
                        if constexpr (kCluster > 1) {
                            uint32_t v[kCluster];
#pragma unroll
                            for (int r = 0; r < kCluster; ++r) v[r] = cluster_read(&bits[i], r);
#pragma unroll
                            for (int r = 0; r < kCluster; ++r) w |= v[r];
                        }
                        const int64_t left = a.pages - from - 32ll * i;
                        if (left < 32) w |= left <= 0 ? kAll : kAll << left;
                        bits[i] = w;
                        free_mine += __popc(~w);
                    }
                    int64_t in_cta;
                    int64_t to = block_before<kWarps>(free_mine, red, in_cta);
                    for (int i = i0; i < i1; ++i) {
                        free_to[i - word0] = static_cast<int>(to);
                        to += __popc(~bits[i]);
                    }
                    if (tid == 0) free_here = static_cast<int>(in_cta);
                    everywhere();
                }
                if constexpr (kCluster > 1) {
                    uint32_t f[kCluster];
#pragma unroll
                    for (int r = 0; r < kCluster; ++r) f[r] = cluster_read(&free_here, r);
#pragma unroll
                    for (int r = 0; r < kCluster; ++r) {
                        here += f[r];
                        if (r < rank) before += f[r];
                    }
                } else {
                    here = free_here;
                }
                if (pass == 1) {
                    for (int i = word0 + warp; i < word1; i += kWarps) {
                        const uint32_t w = bits[i];
                        const int64_t first = taken + before + free_to[i - word0];
                        if (w == kAll || first >= need) continue;
                        const int64_t at = first + __popc(~w & ((1u << lane) - 1u));
                        if (((w >> lane) & 1u) || at >= need) continue;
                        const int g = find(pages_to, p.groups, static_cast<int>(at));
                        int left = static_cast<int>(at) - pages_to[g];
                        const int b = within(g, left, [&](int s) { return need_of<kFresh>(a, s).pages; });
                        const int got = static_cast<int>(from + 32ll * i + lane);
                        if constexpr (kFresh)
                            a.fresh[static_cast<int64_t>(b) * a.fresh_cols + left] = got;
                        else
                            a.table[static_cast<int64_t>(b) * a.cols + up(single ? held_s[b] : a.held[b]) + left] = got;
                    }
                }
                taken = static_cast<int>(min(static_cast<int64_t>(need), taken + here));
                if (!once) everywhere();      // before the bitmaps are cleared again
            }
            if (pass == 0 && taken < need) refused = kErrFull;
        }
    }
    if (refused && rank == 0) {
        if (!kFresh)
            for (int b = tid; b <= a.B; b += kThreads) a.start[b] = 0;
        if (tid == 0) report(a.dev_status, refused);
    }
    // the new entries are there, no CTA reads another's bitmap any more, and held, which
    // may be len, is read but where a group is more than a sequence
    if constexpr (kCluster > 1) cluster_sync();
    else __syncthreads();
    if constexpr (!kFresh) {
        if (refused) return;
        const int total = static_cast<int>(all_rows);
        if (a.slot || a.position) {
            for (int64_t t = rank * kThreads + tid; t < total; t += kCluster * kThreads) {
                const int g = find(rows_to, p.groups, static_cast<int>(t));
                int left = static_cast<int>(t) - rows_to[g];
                const int b = within(g, left, [&](int s) { return a.news[s]; });
                const int at = (single ? held_s[b] : a.held[b]) + left;
                if (a.position) a.position[t] = at;
                if (a.slot) {
                    const int named = __ldcg(a.table + static_cast<int64_t>(b) * a.cols + at / kBlk);
                    const bool there = named >= 0 && named < a.pages;
                    if (!there) report(a.dev_status, kErrInvalid);
                    a.slot[t] = there ? named * kBlk + at % kBlk : -1;
                }
            }
        }
        if (single) {
            for (int b = rank * kThreads + tid; b < a.B; b += kCluster * kThreads) a.len[b] = held_s[b] + rows_to[b + 1] - rows_to[b];
        } else {
            everywhere();
            for (int b = rank * kThreads + tid; b < a.B; b += kCluster * kThreads) a.len[b] = a.held[b] + a.news[b];
        }
    }
}

template <bool kFresh, int kCluster, int kThreads>
cudaError_t launch(const PlanParams &p, size_t smem, cudaStream_t st) {
    const auto kernel = plan_kernel<kFresh, kCluster, kThreads>;
    // the most that any call needs: another thread's call may be between this and the launch
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = kCluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(kCluster);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, p);
}

template <int kCluster, int kThreads>
cudaError_t launch_by(const PlanArgs &a, cudaStream_t st) {
    constexpr int kGroups = kPer * kThreads;
    PlanParams p;
    p.a = a;
    p.size = (a.B + kGroups - 1) / kGroups;
    p.groups = (a.B + p.size - 1) / p.size;
    const int sums = 4 * (3 * p.groups + 2);
    const int words = (a.pages + 31) / 32, most = (kSmem - sums) / 4 * kCluster / (kCluster + 1) - 1;
    p.words = words < most ? words : most;
    const size_t smem = sums + 4 * (static_cast<size_t>(p.words) + (p.words + kCluster - 1) / kCluster);
    return a.fresh ? launch<true, kCluster, kThreads>(p, smem, st) : launch<false, kCluster, kThreads>(p, smem, st);
}

}  // namespace

// Eight CTAs of 512 threads: 32 sequences of up to 32,768 tokens 7.5 us on the GPU,
// 4,096 of up to 2,000 15.5; of 256 threads 6.8 and 28.4, of 1,024 9.8 and 15.7, four
// of 512 6.9 and 20.8.
cudaError_t launch_cache_plan(const PlanArgs &a, cudaStream_t st) { return launch_by<8, 512>(a, st); }

}  // namespace vca

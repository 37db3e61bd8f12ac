// route.cu -- routing of tokens to the experts of a mixture-of-experts layer,
// and the grouping of rows by an index (expert or adapter) that the routed
// products and the low-rank adapters read.
//
// Routing.  For a token with logits l[0..E):
//   score   s_e = softmax(l)_e  or  1 / (1 + exp(-l_e))
//   choice  c_e = s_e + bias_e when a bias is given (it decides the selection
//           only); without one the order of the scores is the order of the
//           logits, and the logits themselves are compared
//   groups  (optional) the experts lie in n_groups equal runs; a run's value
//           is its largest choice or the sum of its two largest scores (with
//           the bias); only the top_groups best runs stay
//   ids     the top_k largest choices, largest first, ties to the lowest index
//   weights scale * s_e, or scale * s_e / (sum of the chosen s + 1e-20)
// A logit of -inf or NaN is an expert that is never chosen: a slot for which
// no expert is left gets id -1 and weight 0, so a padding token (all -inf)
// routes nowhere.  +inf counts as the largest finite float.
//
// Exactness of the selection.  Logits compare exactly.  Choices with a bias
// and sums of two scores are compared in 64 bits: two experts a few units of
// 2^-24 apart are common at thousands of tokens times hundreds of experts, and
// a 32-bit sigmoid would order them by its own rounding.
//
// One warp per token; lane l holds experts l, l + 32, ...  A value is kept as
// an unsigned key of the same order (0 = not there), so a selection step is a
// scan of the lane's keys and warp reductions of 32-bit words (redux), and
// the winner removes its key.  Bytes are few (E logits in, 16 bytes per slot
// out): the kernel is bound by the latency of these dependent reductions, so
// blocks are large (32 warps) and never more than one wave of SMs, which
// also bounds what the ordering pass has to sum over.
//
// Ordering (k_group): a stable counting sort.  Every block counts its chunk of
// items per group; the ordering kernel sums the counts of the blocks before
// its own (and of all blocks, for the groups' offsets), and each of its warps
// ranks 32 items at a time with a match of equal ids.  No atomic decides a
// position, so the order never varies.  A call small enough for one block
// does all of it in one launch.
#include <algorithm>
#include <cmath>

#include "device_common.cuh"
#include "kernels.h"

namespace uw {
namespace {

using namespace dev;

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kMaxFloat = 3.402823466e38f;
constexpr int kGroupCells = 10240;      // 40 KB of per-warp counters

struct GroupArgs {
    const int32_t *ids;     // [items]; outside [0, groups): no group
    int64_t items;
    int groups;
    int64_t per_block;      // items per block (the same chunks as `counts`)
    const int32_t *counts;  // [blocks][groups + 1]; null: one block, which counts itself
    int blocks;
    int warps;              // warps that rank (groups + 1 counters each)
    int32_t *offsets, *order, *slot;
};

struct RouteArgs {
    const void *logits;
    int64_t t, stride;
    const float *bias;
    int experts, top_k, n_groups, top_groups, group_size;
    int softmax, top2, renorm, bf16;
    float scale;
    int32_t *ids;
    float *weights;
    int64_t rows_per_block;
    int32_t *counts;        // [blocks][experts + 1]; null: one block, which also orders
    GroupArgs group;
};

__device__ __forceinline__ int group_of(int32_t id, int groups) { return uint32_t(id) < uint32_t(groups) ? id : groups; }

// exclusive scan of v[0..n) in shared memory by one warp
__device__ __forceinline__ void warp_exclusive_scan(int32_t *v, int n) {
    const int lane = threadIdx.x & 31;
    int32_t run = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int32_t x = i0 + lane < n ? v[i0 + lane] : 0;
        int32_t s = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t u = __shfl_up_sync(kAll, s, d);
            if (lane >= d) s += u;
        }
        if (i0 + lane < n) v[i0 + lane] = run + s - x;
        run += __shfl_sync(kAll, s, 31);
    }
}

// Orders one block's items.  Shared memory: base[groups + 1], then
// cell[warps][groups + 1].  All threads of the block take part.
__device__ __forceinline__ void order_block(const GroupArgs &a, int64_t block, int32_t *base, int32_t *cell) {
    const int g1 = a.groups + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t begin = block * a.per_block;
    const int64_t n = max(int64_t(0), min(a.per_block, a.items - begin));
    const int64_t per_warp = ((n + a.warps - 1) / a.warps + 31) / 32 * 32;
    const int64_t w0 = min(n, warp * per_warp), w1 = min(n, w0 + per_warp);
    for (int i = threadIdx.x; i < a.warps * g1; i += blockDim.x) cell[i] = 0;
    for (int i = threadIdx.x; i < g1; i += blockDim.x) base[i] = 0;
    __syncthreads();
    int32_t *mine = cell + warp * g1;
    if (warp < a.warps) {
        for (int64_t i0 = w0; i0 < w1; i0 += 32) {
            const bool live = i0 + lane < w1;
            const int key = live ? group_of(a.ids[begin + i0 + lane], a.groups) : -1;
            const uint32_t same = __match_any_sync(kAll, key);
            if (live && lane == __ffs(same) - 1) mine[key] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // base: where this block's first item of each group goes
    if (a.counts) {
        // part p of the columns' threads sums blocks p, p + parts, ...
        const int cols = (g1 + 31) / 32 * 32;
        const int parts = max(1, int(blockDim.x) / cols);
        int32_t *before = cell + a.warps * g1;
        for (int i = threadIdx.x; i < g1; i += blockDim.x) before[i] = 0;
        __syncthreads();
        for (int c0 = threadIdx.x; c0 < cols * parts; c0 += blockDim.x) {
            const int c = c0 % cols, p = c0 / cols;
            if (c < g1) {
                int32_t sum = 0, bef = 0;
#pragma unroll 8
                for (int b = p; b < a.blocks; b += parts) {
                    const int32_t v = a.counts[int64_t(b) * g1 + c];
                    sum += v;
                    bef += b < block ? v : 0;
                }
                atomicAdd(&base[c], sum);
                atomicAdd(&before[c], bef);
            }
        }
        __syncthreads();
        if (warp == 0) warp_exclusive_scan(base, g1);
        __syncthreads();
        if (block == 0)
            for (int i = threadIdx.x; i < g1; i += blockDim.x) a.offsets[i] = base[i];
        for (int i = threadIdx.x; i < g1; i += blockDim.x) {
            int32_t run = base[i] + before[i];
            for (int w = 0; w < a.warps; w++) {
                const int32_t v = cell[w * g1 + i];
                cell[w * g1 + i] = run;
                run += v;
            }
        }
    } else {
        for (int i = threadIdx.x; i < g1; i += blockDim.x) {
            int32_t sum = 0;
            for (int w = 0; w < a.warps; w++) sum += cell[w * g1 + i];
            base[i] = sum;
        }
        __syncthreads();
        if (warp == 0) warp_exclusive_scan(base, g1);
        __syncthreads();
        for (int i = threadIdx.x; i < g1; i += blockDim.x) {
            int32_t run = base[i];
            a.offsets[i] = run;
            for (int w = 0; w < a.warps; w++) {
                const int32_t v = cell[w * g1 + i];
                cell[w * g1 + i] = run;
                run += v;
            }
        }
    }
    __syncthreads();
    if (warp < a.warps) {
        for (int64_t i0 = w0; i0 < w1; i0 += 32) {
            const bool live = i0 + lane < w1;
            const int64_t item = begin + i0 + lane;
            const int key = live ? group_of(a.ids[item], a.groups) : -1;
            const uint32_t same = __match_any_sync(kAll, key);
            int32_t pos = 0;
            if (live) pos = mine[key] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (live) {
                if (lane == __ffs(same) - 1) mine[key] += __popc(same);
                a.order[pos] = int32_t(item);
                if (a.slot) a.slot[item] = key < a.groups ? pos : -1;
            }
            __syncwarp();
        }
    }
}

extern __shared__ int32_t smem_route[];

__global__ void __launch_bounds__(1024) k_group(const GroupArgs a) {
    pdl_wait();   // ids and counts are the previous kernel's output
    order_block(a, blockIdx.x, smem_route, smem_route + a.groups + 1);
}

__global__ void __launch_bounds__(1024) k_group_count(const int32_t *ids, int64_t items, int groups, int64_t per_block,
                                                      int32_t *counts) {
    pdl_trigger();
    const int g1 = groups + 1;
    for (int i = threadIdx.x; i < g1; i += blockDim.x) smem_route[i] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * per_block, end = min(items, begin + per_block);
    for (int64_t i = begin + threadIdx.x; i < end; i += blockDim.x)
        atomicAdd(&smem_route[group_of(ids[i], groups)], 1);
    __syncthreads();
    for (int i = threadIdx.x; i < g1; i += blockDim.x) counts[int64_t(blockIdx.x) * g1 + i] = smem_route[i];
}

// ---------------------------------------------------------------- keys

// unsigned key of the same order as the value; 0 is below every finite value
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);   // -0 compares equal to +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double v) {
    const uint64_t b = uint64_t(__double_as_longlong(v + 0.0));
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double value_of(uint64_t key) {
    return __longlong_as_double(static_cast<long long>(key >> 63 ? key & 0x7FFFFFFFFFFFFFFFull : ~key));
}

// largest key of the warp, in every lane
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kAll, uint32_t(k >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, uint32_t(k >> 32) == hi ? uint32_t(k) : 0u);
    return uint64_t(hi) << 32 | lo;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

__device__ __forceinline__ float load_logit(const RouteArgs &a, int64_t row, int e) {
    const int64_t at = row * a.stride + e;
    if (a.bf16) return __uint_as_float(uint32_t(static_cast<const uint16_t *>(a.logits)[at]) << 16);
    return static_cast<const float *>(a.logits)[at];
}

// s_e in 64 bits; m and sum: the row's largest logit and sum of exp(l - m)
__device__ __forceinline__ double score_of(const RouteArgs &a, float l, float m, double sum) {
    return a.softmax ? exp(double(l) - double(m)) / sum : 1.0 / (1.0 + exp(-double(l)));
}

// NV: experts per lane; Key: uint32_t compares logits, uint64_t choices in 64 bits
template <int NV, class Key>
__device__ __forceinline__ void route_row(const RouteArgs &a, int64_t row, int32_t *count) {
    const int lane = threadIdx.x & 31;
    constexpr bool kWide = sizeof(Key) == 8;
    float l[NV];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int e = 32 * i + lane;
        float v = e < a.experts ? load_logit(a, row, e) : -INFINITY;
        v = v > -INFINITY ? fminf(v, kMaxFloat) : -INFINITY;   // NaN, -inf: not there
        l[i] = v;
        m = fmaxf(m, v);
    }
    double sum = 1.0;
    if (a.softmax) {
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, d));
        if (kWide) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (l[i] >= -kMaxFloat) s += exp(double(l[i]) - double(m));
            sum = warp_sum(s);
        } else {
            // the sum only scales the weights here: 32 bits, all terms positive
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (l[i] >= -kMaxFloat) s += expf(l[i] - m);
            sum = double(warp_sum(s));
        }
    }
    Key key[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        key[i] = 0;
        if (l[i] >= -kMaxFloat) {
            if constexpr (kWide) {
                if (a.bias) {
                    const double c = score_of(a, l[i], m, sum) + double(__ldg(a.bias + 32 * i + lane));
                    key[i] = c > -INFINITY ? key_of(c) : 0;   // a bias of -inf or NaN: never chosen
                } else {
                    key[i] = key_of(double(l[i]));
                }
            } else {
                key[i] = key_of(l[i]);
            }
        }
    }

    if (a.n_groups > 1) {
        // lane g keeps group g's value as a key of its own order
        uint64_t value = 0;
        for (int g = 0; g < a.n_groups; g++) {
            const int lo = g * a.group_size, hi = lo + a.group_size;
            Key best = 0;
            int at = 0;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                if (32 * i + 31 < lo || 32 * i >= hi) continue;
                const int e = 32 * i + lane;
                if (e >= lo && e < hi && key[i] > best) {
                    best = key[i];
                    at = e;
                }
            }
            const Key first = warp_max(best);
            uint64_t v = uint64_t(first);
            if (kWide && a.top2 && first != 0) {
                // the second largest: the first's lowest place left out
                const int where = __reduce_min_sync(kAll, best == first ? at : 0x7FFFFFFF);
                Key next = 0;
#pragma unroll
                for (int i = 0; i < NV; i++) {
                    if (32 * i + 31 < lo || 32 * i >= hi) continue;
                    const int e = 32 * i + lane;
                    if (e >= lo && e < hi && e != where && key[i] > next) next = key[i];
                }
                const Key second = warp_max(next);
                double s;
                if (a.bias) {
                    s = value_of(uint64_t(first)) + (second ? value_of(uint64_t(second)) : 0.0);
                } else {
                    // the keys are logits: the two scores are summed
                    s = score_of(a, float(value_of(uint64_t(first))), m, sum) +
                        (second ? score_of(a, float(value_of(uint64_t(second))), m, sum) : 0.0);
                }
                v = key_of(s);
            }
            if (lane == g) value = v;
        }
        uint32_t keep = 0;
        for (int j = 0; j < a.top_groups; j++) {
            const uint64_t live = (keep >> lane) & 1u ? 0 : value;
            const uint64_t best = warp_max(live);
            if (best == 0) break;    // groups that are left hold nothing to choose
            keep |= 1u << (__ffs(__ballot_sync(kAll, live == best)) - 1);
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int e = 32 * i + lane;
            if (e < a.experts && !((keep >> (e / a.group_size)) & 1u)) key[i] = 0;
        }
    }

    int32_t my_id = -1;
    for (int s = 0; s < a.top_k; s++) {
        Key best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (key[i] > best) {
                best = key[i];
                at = 32 * i + lane;
            }
        const Key top = warp_max(best);
        if (top == 0) break;
        const int win = __reduce_min_sync(kAll, best == top ? at : 0x7FFFFFFF);
        if (lane == s) my_id = win;
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (win == 32 * i + lane) key[i] = 0;
    }
    // slot s is lane s's
    double w = 0.0;
    if (my_id >= 0) w = score_of(a, fminf(load_logit(a, row, my_id), kMaxFloat), m, sum);
    if (a.renorm) w = w / (warp_sum(w) + 1e-20);
    if (lane < a.top_k) {
        a.ids[row * a.top_k + lane] = my_id;
        a.weights[row * a.top_k + lane] = float(w * double(a.scale));
        if (count) atomicAdd(&count[my_id < 0 ? a.experts : my_id], 1);
    }
}

template <int NV>
constexpr int route_threads() { return NV <= 8 ? 1024 : 512; }

template <int NV, class Key>
__global__ void __launch_bounds__(route_threads<NV>()) k_route(const RouteArgs a) {
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t begin = blockIdx.x * a.rows_per_block, end = min(a.t, begin + a.rows_per_block);
    int32_t *count = a.counts ? smem_route : nullptr;
    pdl_trigger();
    if (count) {
        for (int i = threadIdx.x; i <= a.experts; i += blockDim.x) count[i] = 0;
        __syncthreads();
    }
    for (int64_t row = begin + warp; row < end; row += warps) route_row<NV, Key>(a, row, count);
    __syncthreads();
    if (count) {
        for (int i = threadIdx.x; i <= a.experts; i += blockDim.x)
            a.counts[int64_t(blockIdx.x) * (a.experts + 1) + i] = count[i];
    } else {
        order_block(a.group, 0, smem_route, smem_route + a.experts + 1);
    }
}

// ranking warps for `groups` groups and `items` items per block, at most `most`
int rank_warps(int groups, int64_t items, int most) {
    return int(std::max<int64_t>(1, std::min<int64_t>(std::min(most, kGroupCells / (groups + 1)), (items + 31) / 32)));
}

size_t group_smem(int groups, int warps) { return size_t(warps + 2) * size_t(groups + 1) * 4; }

}  // namespace

GroupGeometry group_geometry(int64_t rows, int per_row, int groups) {
    GroupGeometry g;
    // One block takes what its 32 warps rank in a few steps (4096 items: 5 us in
    // one block, 8 us in two launches); beyond that one block per SM, so that
    // the sum over blocks stays short.
    if (rows * per_row <= 8192) {
        g.blocks = 1;
        g.rows_per_block = std::max<int64_t>(rows, 1);
        g.bytes = 0;
        return g;
    }
    const int64_t most = 148;
    g.rows_per_block = (rows + most - 1) / most;
    // at least 256 items per block
    g.rows_per_block = std::max<int64_t>(g.rows_per_block, (256 + per_row - 1) / per_row);
    g.blocks = int((rows + g.rows_per_block - 1) / g.rows_per_block);
    g.bytes = (uint64_t(g.blocks) * uint64_t(groups + 1) * 4 + 255) / 256 * 256;
    return g;
}

// Routing: a block of 32 warps takes one row per warp at a time.  Two rounds in
// one block are quicker than a second launch; more are not.
GroupGeometry route_geometry(int64_t t, int top_k, int experts) {
    GroupGeometry g = group_geometry(t, top_k, experts);
    if (t <= 64) return g;
    const int64_t most = 148;
    g.rows_per_block = std::max<int64_t>((t + most - 1) / most, 32);
    g.blocks = int((t + g.rows_per_block - 1) / g.rows_per_block);
    g.bytes = (uint64_t(g.blocks) * uint64_t(experts + 1) * 4 + 255) / 256 * 256;
    return g;
}

cudaError_t launch_group_rows(const GroupLaunch &p, cudaStream_t stream) {
    const GroupGeometry geo = group_geometry(p.rows, p.per_row, p.groups);
    GroupArgs a{};
    a.ids = p.ids;
    a.items = p.rows * p.per_row;
    a.groups = p.groups;
    a.per_block = geo.rows_per_block * p.per_row;
    a.blocks = geo.blocks;
    a.offsets = p.offsets;
    a.order = p.order;
    a.slot = p.slot;
    const int threads = 1024;
    a.warps = rank_warps(p.groups, a.per_block, 32);
    const size_t smem = group_smem(p.groups, a.warps);
    if (geo.bytes) {
        int32_t *counts = static_cast<int32_t *>(p.ws);
        k_group_count<<<unsigned(geo.blocks), 1024, size_t(p.groups + 1) * 4, stream>>>(p.ids, a.items, p.groups,
                                                                                       a.per_block, counts);
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess) return err;
        a.counts = counts;
    }
    const cudaError_t err = launch_pdl(geo.bytes != 0, k_group, dim3(unsigned(geo.blocks)), dim3(threads), smem, stream, a);
    return err != cudaSuccess ? err : cudaGetLastError();
}

cudaError_t launch_route(const RouteLaunch &p, cudaStream_t stream) {
    const uw_router &r = *p.router;
    const GroupGeometry geo = route_geometry(p.t, r.top_k, r.experts);
    const int per_lane = (r.experts + 31) / 32;
    const int nv = per_lane <= 1 ? 1 : per_lane <= 2 ? 2 : per_lane <= 4 ? 4 : per_lane <= 8 ? 8 : per_lane <= 16 ? 16 : 32;
    const int threads = nv <= 8 ? 1024 : 512;
    RouteArgs a{};
    a.logits = p.logits;
    a.t = p.t;
    a.stride = p.stride;
    a.bias = p.bias;
    a.experts = r.experts;
    a.top_k = r.top_k;
    a.n_groups = r.n_groups;
    a.top_groups = r.top_groups;
    a.group_size = r.experts / r.n_groups;
    a.softmax = r.score == UW_SCORE_SOFTMAX;
    a.top2 = r.group_score == UW_GROUP_TOP2;
    a.renorm = r.renormalize;
    a.bf16 = r.logits_type == UW_TYPE_BF16;
    a.scale = r.scale;
    a.ids = p.ids;
    a.weights = p.weights;
    a.rows_per_block = geo.rows_per_block;
    GroupArgs &g = a.group;
    g.ids = p.ids;
    g.items = p.t * r.top_k;
    g.groups = r.experts;
    g.per_block = geo.rows_per_block * r.top_k;
    g.blocks = geo.blocks;
    g.offsets = p.offsets;
    g.order = p.order;
    g.slot = p.slot;
    a.counts = geo.bytes ? static_cast<int32_t *>(p.ws) : nullptr;
    g.warps = rank_warps(r.experts, g.per_block, threads / 32);
    const size_t smem = geo.bytes ? size_t(r.experts + 1) * 4 : group_smem(r.experts, g.warps);
    // 64-bit keys where the selection compares computed scores
    const bool wide = p.bias != nullptr || (r.n_groups > 1 && a.top2);
    const dim3 grid(static_cast<unsigned>(geo.blocks)), block(static_cast<unsigned>(threads));
#define UW_ROUTE(NV_)                                                    \
    case NV_:                                                            \
        if (wide) k_route<NV_, uint64_t><<<grid, block, smem, stream>>>(a); \
        else k_route<NV_, uint32_t><<<grid, block, smem, stream>>>(a);   \
        break;
    switch (nv) {
        UW_ROUTE(1)
        UW_ROUTE(2)
        UW_ROUTE(4)
        UW_ROUTE(8)
        UW_ROUTE(16)
        UW_ROUTE(32)
    }
#undef UW_ROUTE
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || !geo.bytes) return err;
    g.counts = a.counts;
    g.warps = rank_warps(r.experts, g.per_block, 32);
    err = launch_pdl(true, k_group, grid, dim3(1024), group_smem(r.experts, g.warps), stream, g);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace uw

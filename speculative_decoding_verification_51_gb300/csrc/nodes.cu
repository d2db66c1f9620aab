// nodes.cu -- the bookkeeping of a decoding step: where the drafted nodes
// stand (spec_tree_plan), and the kept path's rows after the verification
// (spec_kv_commit).
//
// k_tree_plan, grid 1 + B: CTA 1 + b checks request b's page table and lets
// one warp (lane v = node v) find the ancestors by pointer doubling: after
// round r a node's mask holds its 2^r nearest ancestors, so five rounds reach
// all of at most 32 nodes.  The depth is the number of bits.  CTA 0 forms the
// running sum of the requests' tiles from the lengths alone, so that no CTA
// waits for another.
//
// k_kv_commit, grid (B, caches): bit i of the last node's mask set means node
// i is on the path, and the path's d-th node (in index order, which is path
// order since a parent comes before its children) moves to the slot of node
// d.  Its index is d or more, so that a row is always read before a row with a
// greater d is written over it: a thread keeps its 16 bytes of the row
// through the whole path, in order, and no thread waits for another.
//
// Both are bound by latency: 256 trees of 32 nodes over up to 4000 tokens take
// 3.7 us of device time, the commit of their paths in one 8-bit cache 4.5 (a table
// entry, a slot and a row have to be read one after the other).
#include <algorithm>
#include <cfloat>

#include "cache.cuh"

namespace sv {
namespace {

constexpr int PLAN_T = 256;

struct PlanArgs {
    const int32_t* parents;
    const int32_t* nodes;
    const int32_t* ctx;
    const int32_t* table;
    int B, N, max_pages, page, num_pages;
    int32_t* positions;
    long long* slots;
    uint32_t* masks;
    PlanLists<int> plan;
    int rest;  // words of the plan after its lists
    int32_t* status;
};

// whether the request's length lies within its page table
__device__ __forceinline__ bool length_ok(const PlanArgs& A, int ctx, int n) {
    return ctx >= 0 && n >= 1 && n <= A.N &&
           (long long)ctx + n <= (long long)A.max_pages * A.page;
}

__global__ void __launch_bounds__(PLAN_T) k_tree_plan(const __grid_constant__ PlanArgs A) {
    begin_after_previous();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x == 0) {
        __shared__ int sums[PLAN_T / 32];
        int carry = 0;
        for (int base = 0; base < A.B; base += PLAN_T) {
            const int b = base + tid;
            int t = 0;
            if (b < A.B) {
                const int ctx = A.ctx[b], n = A.nodes[b];
                t = length_ok(A, ctx, n) ? (ctx + n + TREE_TILE - 1) / TREE_TILE : 1;
            }
            int incl = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            __syncthreads();
            if (lane == 31) sums[warp] = incl;
            __syncthreads();
            int before = carry, all = 0;
#pragma unroll
            for (int w = 0; w < PLAN_T / 32; ++w) {
                if (w < warp) before += sums[w];
                all += sums[w];
            }
            if (b < A.B) A.plan.tiles[b] = before + incl - t;
            carry += all;
        }
        if (tid == 0) A.plan.tiles[A.B] = carry;
        if (tid < A.rest) A.plan.tiles[A.B + 1 + tid] = 0;  // (less than 256 bytes)
        return;
    }
    const int b = blockIdx.x - 1;
    const int ctx = A.ctx[b], n = A.nodes[b];
    const bool fits = length_ok(A, ctx, n);
    const int32_t* table = A.table + (long long)b * A.max_pages;
    int bad = 0;
    if (n < 1 || n > A.N) bad = SPEC_BADBIT_NUM_DRAFT;
    else if (!fits) bad = SPEC_BADBIT_PAGE;
    if (fits) {
        const int used = (ctx + n - 1) / A.page + 1;
        for (int i = tid; i < used; i += PLAN_T) {
            const int p = table[i];
            if (p < 0 || p >= A.num_pages) bad |= SPEC_BADBIT_PAGE;
        }
    }
    uint32_t mask = 0;
    if (warp == 0 && fits) {
        int up = -1;
        if (lane >= 1 && lane < n) {
            up = A.parents[(long long)b * A.N + lane];
            if (up < 0 || up >= lane) {
                bad |= SPEC_BADBIT_TREE;
                up = -1;
            }
        }
        mask = lane < n ? 1u << lane : 0u;
#pragma unroll
        for (int r = 0; r < 5; ++r) {
            const uint32_t m = __shfl_sync(0xffffffffu, mask, up < 0 ? 0 : up);
            const int u = __shfl_sync(0xffffffffu, up, up < 0 ? 0 : up);
            if (up >= 0) {
                mask |= m;
                up = u;
            }
        }
    }
    __shared__ int all_bad;
    if (tid == 0) all_bad = 0;
    __syncthreads();
    if (bad) atomicOr(&all_bad, bad);
    __syncthreads();
    if (warp == 0) {
        const bool ok = all_bad == 0 && lane < n;
        if (lane < A.N) {
            const long long i = (long long)b * A.N + lane;
            const int t = ctx + lane;
            A.positions[i] = ok ? ctx + __popc(mask) - 1 : 0;
            A.slots[i] = ok ? (long long)table[t / A.page] * A.page + t % A.page : -1;
            A.masks[i] = ok ? mask : 0u;
        }
        if (lane == 0) {
            A.plan.ctx[b] = all_bad ? 0 : ctx;
            A.plan.nodes[b] = all_bad ? 0 : n;
            if (all_bad && A.status) atomicOr(A.status, all_bad);
        }
    }
}

struct CommitArgs {
    void* k[SPEC_MAX_COMMIT_CACHES];
    void* v[SPEC_MAX_COMMIT_CACHES];
    uint8_t* ks[SPEC_MAX_COMMIT_CACHES];
    uint8_t* vs[SPEC_MAX_COMMIT_CACHES];
    CacheView c;  // the shape they share
    const uint32_t* masks;
    const long long* slots;
    const int32_t* last;
    const int32_t* ctx;
    int N;
    int32_t* new_ctx;
    int32_t* status;
};

constexpr int COMMIT_T = 128;

__global__ void __launch_bounds__(COMMIT_T) k_kv_commit(const __grid_constant__ CommitArgs A) {
    begin_after_previous();
    const int b = blockIdx.x, l = blockIdx.y, tid = threadIdx.x;
    const int last = A.last[b];
    const long long* slots = A.slots + (long long)b * A.N;
    uint32_t path = 0;
    int bad = 0;
    if (last >= 0) {
        path = last < A.N ? A.masks[(long long)b * A.N + last] : 0u;
        if (!(path >> (last & 31) & 1u)) {  // no such node: nothing moves
            path = 0;
            bad = SPEC_BADBIT_TREE;
        }
    }
    __shared__ long long src[32], dst[32];  // element offsets of the rows to move
    __shared__ long long ssrc[32], sdst[32];
    __shared__ int moves;
    if (tid < 32) {
        const bool on = tid < A.N && (path >> tid & 1u);
        const int d = __popc(path & ((1u << tid) - 1u));
        long long a = -1, z = -1;
        if (on) {
            a = slots[tid];
            z = slots[d];
            if (a < 0 || z < 0 || a >= A.c.slots || z >= A.c.slots) {
                bad |= SPEC_BADBIT_PAGE;
                a = z = -1;
            }
        }
        const bool move = on && a >= 0 && d != tid;
        const unsigned m = __ballot_sync(0xffffffffu, move);
        if (move) {
            const int at = __popc(m & ((1u << tid) - 1u));
            const long long pa = a / A.c.page, pz = z / A.c.page;
            const int oa = int(a - pa * A.c.page), oz = int(z - pz * A.c.page);
            src[at] = pa * A.c.page_stride + oa * A.c.token_stride;
            dst[at] = pz * A.c.page_stride + oz * A.c.token_stride;
            ssrc[at] = pa * A.c.heads * A.c.page + oa;
            sdst[at] = pz * A.c.heads * A.c.page + oz;
        }
        if (tid == 0) moves = __popc(m);
        if (l == 0) {
            if (bad && A.status) atomicOr(A.status, bad);
            if (tid == 0) A.new_ctx[b] = A.ctx[b] + __popc(path);
        }
    }
    __syncthreads();
    const int n = moves;
    if (!n) return;
    const int es = A.c.dtype == SPEC_E4M3 ? 1 : 2;
    const int vecs = A.c.D * es / 16, per = A.c.heads * vecs;
    for (int i = tid; i < 2 * per; i += COMMIT_T) {
        const int side = i >= per, j = side ? i - per : i;
        const int h = j / vecs, x = j - h * vecs;
        char* base = static_cast<char*>(side ? A.v[l] : A.k[l]) + h * A.c.head_stride * es + x * 16;
        for (int r = 0; r < n; r += 8) {  // eight rows in flight, stores in path order
            uint4 w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (r + u < n) w[u] = *reinterpret_cast<const uint4*>(base + src[r + u] * es);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (r + u < n) *reinterpret_cast<uint4*>(base + dst[r + u] * es) = w[u];
        }
    }
    if (es == 1)
        for (int i = tid; i < 2 * A.c.heads; i += COMMIT_T) {
            const int side = i >= A.c.heads, h = side ? i - A.c.heads : i;
            uint8_t* base = (side ? A.vs[l] : A.ks[l]) + (long long)h * A.c.page;
            for (int r = 0; r < n; r += 8) {
                uint8_t w[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (r + u < n) w[u] = base[ssrc[r + u]];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (r + u < n) base[sdst[r + u]] = w[u];
            }
        }
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_tree_plan_size(int B) {
    if (B < 0 || B > (1 << 24)) return 0;
    return align256(plan_words(B) * 4);
}

spec_status spec_tree_plan(const int32_t* tree_parents, const int32_t* num_nodes,
                           const int32_t* context_len, const int32_t* page_table, int B, int N,
                           int max_pages, int page_size, int num_pages, int32_t* positions,
                           int64_t* slots, uint32_t* masks, void* plan, size_t plan_bytes,
                           int32_t* dev_status, spec_stream_t stream) {
    if (B < 0 || B > (1 << 24) || N < 1 || max_pages < 1 || num_pages < 1 || page_size < 1)
        return SPEC_ERR_INVALID_ARG;
    if (N > 32 || page_size % 16 || page_size > 65536) return SPEC_ERR_UNSUPPORTED;
    const long long longest = (long long)max_pages * page_size;
    if (longest >= (1ll << 31) - TREE_TILE || B * ((longest + TREE_TILE - 1) / TREE_TILE) >= (1ll << 31))
        return SPEC_ERR_UNSUPPORTED;
    if (B == 0) return SPEC_OK;
    if (!tree_parents || !num_nodes || !context_len || !page_table || !positions || !slots ||
        !masks || !plan)
        return SPEC_ERR_INVALID_ARG;
    if (!all_aligned(4, {tree_parents, num_nodes, context_len, page_table, positions, masks, dev_status}) || !aligned(slots, 8))
        return SPEC_ERR_UNSUPPORTED;
    if (!aligned(plan, 256) || plan_bytes < spec_tree_plan_size(B)) return SPEC_ERR_WORKSPACE;
    PlanArgs A;
    A.parents = tree_parents;
    A.nodes = num_nodes;
    A.ctx = context_len;
    A.table = page_table;
    A.B = B;
    A.N = N;
    A.max_pages = max_pages;
    A.page = page_size;
    A.num_pages = num_pages;
    A.positions = positions;
    A.slots = reinterpret_cast<long long*>(slots);
    A.masks = masks;
    A.plan = plan_lists(static_cast<int*>(plan), B);
    A.rest = int(spec_tree_plan_size(B) / 4 - plan_words(B));
    A.status = dev_status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dev_status && cudaMemsetAsync(dev_status, 0, 4, st) != cudaSuccess) return SPEC_ERR_CUDA;
    return launch_behind(k_tree_plan, dim3(unsigned(B) + 1), PLAN_T, 0, st, A) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_kv_commit(const spec_kv_cache* caches, int num_caches, const uint32_t* masks,
                           const int64_t* slots, const int32_t* last_node,
                           const int32_t* context_len, int B, int N, int32_t* new_context_len,
                           int32_t* dev_status, spec_stream_t stream) {
    if (!caches || num_caches < 1 || num_caches > SPEC_MAX_COMMIT_CACHES || B < 0 ||
        B > (1 << 24) || N < 1)
        return SPEC_ERR_INVALID_ARG;
    if (N > 32) return SPEC_ERR_UNSUPPORTED;
    CommitArgs A;
    for (int l = 0; l < num_caches; ++l) {
        const spec_kv_cache &c = caches[l], &f = caches[0];
        const spec_status cs = check_cache(&c);
        if (cs != SPEC_OK) return cs;
        if (c.dtype != f.dtype || c.num_pages != f.num_pages || c.page_size != f.page_size ||
            c.heads != f.heads || c.head_dim != f.head_dim || c.page_stride != f.page_stride ||
            c.head_stride != f.head_stride || c.token_stride != f.token_stride)
            return SPEC_ERR_INVALID_ARG;
        A.k[l] = c.k;
        A.v[l] = c.v;
        A.ks[l] = c.k_scale;
        A.vs[l] = c.v_scale;
    }
    if (B == 0) return SPEC_OK;
    if (!masks || !slots || !last_node || !context_len || !new_context_len)
        return SPEC_ERR_INVALID_ARG;
    if (!all_aligned(4, {masks, last_node, context_len, new_context_len, dev_status}) || !aligned(slots, 8))
        return SPEC_ERR_UNSUPPORTED;
    A.c = view_of(caches[0]);
    A.masks = masks;
    A.slots = reinterpret_cast<const long long*>(slots);
    A.last = last_node;
    A.ctx = context_len;
    A.N = N;
    A.new_ctx = new_context_len;
    A.status = dev_status;
    return launch_behind(k_kv_commit, dim3(unsigned(B), unsigned(num_caches)), COMMIT_T, 0,
                         reinterpret_cast<cudaStream_t>(stream), A) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}

}  // extern "C"

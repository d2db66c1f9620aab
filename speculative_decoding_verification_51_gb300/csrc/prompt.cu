// prompt.cu -- spec_prompt_plan: the pieces of packed prompts, their tokens' positions and
// cache slots; spec_prompt_attention: argument checks, tensor maps and the launch.
#include "prompt.cuh"

using namespace sv;

namespace {

constexpr int PLAN_T = 1024;
constexpr int BUCKETS = 2048;  // of the counting sort

struct PlanArgs {
    const int32_t* off;
    const int32_t* koff;  // or null: off
    const int32_t* table;
    int32_t* positions;
    long long* slots;
    PromptHead* plan;
    PromptItem* items;
    int* first;  // [B + 1] pieces of the prompts before b
    int32_t* status;
    int B, T, M, tokens, max_pages, page, num_pages;
};

// Whether offsets and k_offsets begin at 0 or more, never fall and end within their
// tensors.  Called by a whole CTA.
__device__ __forceinline__ bool offsets_good(const PlanArgs& A) {
    bool good = true;
    for (int b = threadIdx.x; b <= A.B; b += blockDim.x) {
        const int o = A.off[b], k = A.koff ? A.koff[b] : o;
        good = good && o >= 0 && o <= A.T && k >= 0 && k <= A.M;
        if (b) good = good && A.off[b - 1] <= o && (!A.koff || A.koff[b - 1] <= k);
    }
    return __syncthreads_and(good);
}

// the prompt that holds packed token t (offsets[b] <= t < offsets[b + 1]), or B
__device__ __forceinline__ int prompt_of(const int32_t* off, int B, int t) {
    int lo = 0, hi = B;  // the first b with offsets[b + 1] > t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (off[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo < B && off[lo] <= t ? lo : B;
}

// CTA 0 lists the pieces, the longest first: so that the pieces that are left when
// the SMs run out of work are short ones.  A counting sort by the keys that a piece
// sees.  The others write positions and slots.  Bound by latency: two passes over
// the pieces, a search of the prompt for each.
__global__ void __launch_bounds__(PLAN_T) k_prompt_plan(const __grid_constant__ PlanArgs A) {
    begin_after_previous();
    const bool good = offsets_good(A);
    if (blockIdx.x) {
        const int t = (blockIdx.x - 1) * PLAN_T + threadIdx.x;
        if (t >= A.T) return;
        int pos = 0;
        long long slot = -1;
        const int b = good ? prompt_of(A.off, A.B, t) : A.B;
        if (b < A.B) {
            const int n = A.off[b + 1] - A.off[b], m = A.koff ? A.koff[b + 1] - A.koff[b] : n;
            pos = t - A.off[b] + m - n;
            if (A.table && pos >= 0) {
                const int p = pos / A.page;
                const int page = p < A.max_pages ? A.table[(long long)b * A.max_pages + p] : -1;
                if (page >= 0 && page < A.num_pages) slot = (long long)page * A.page + pos % A.page;
                else if (A.status) atomicOr(A.status, int(SPEC_BADBIT_PAGE));
            }
        }
        if (A.positions) A.positions[t] = pos;
        if (A.slots) A.slots[t] = slot;
        return;
    }
    __shared__ int count[BUCKETS];
    __shared__ int sums[PLAN_T / 32];
    __shared__ int base;
    const int each = 2 * A.tokens, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // an exclusive sum over the CTA's threads; `base` is what came before, and grows
    auto scan = [&](int x) {
        int s = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (lane == 31) sums[warp] = s;
        __syncthreads();
        if (warp == 0) {
            int z = sums[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, z, o);
                if (lane >= o) z += y;
            }
            sums[lane] = z;
        }
        __syncthreads();
        const int before = base + (warp ? sums[warp - 1] : 0) + s - x;
        const int all = sums[PLAN_T / 32 - 1];
        __syncthreads();
        if (threadIdx.x == 0) base += all;
        __syncthreads();
        return before;
    };
    if (threadIdx.x == 0) base = 0;
    for (int i = threadIdx.x; i < BUCKETS; i += PLAN_T) count[i] = 0;
    __syncthreads();
    int longest = 0;
    if (good) {
        for (int b0 = 0; b0 < A.B; b0 += PLAN_T) {
            const int b = b0 + threadIdx.x;
            const int n = b < A.B ? A.off[b + 1] - A.off[b] : 0;
            if (b < A.B && A.koff) longest = max(longest, A.koff[b + 1] - A.koff[b]);
            else longest = max(longest, n);
            const int at = scan((n + each - 1) / each);
            if (b < A.B) A.first[b] = at;
        }
    }
    __syncthreads();
    const int total = good ? base : 0;
    for (int o = 16; o; o >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
    if (lane == 0) sums[warp] = longest;
    __syncthreads();
    for (int i = 0; i < PLAN_T / 32; ++i) longest = max(longest, sums[i]);
    __syncthreads();
    if (threadIdx.x == 0) {
        A.plan->items = total;
        A.plan->T = A.T;
        A.plan->M = A.M;
        A.plan->tokens = A.tokens;
        if (!good && A.status) atomicOr(A.status, int(SPEC_BADBIT_OFFSETS));
        A.first[A.B] = total;
        base = 0;
    }
    __syncthreads();
    const long long unit = max(1, longest / BUCKETS + 1);
    auto piece = [&](int i, int& bucket) {
        // (prompts without tokens have no piece: the search passes over them)
        int lo = 0, hi = A.B;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (A.first[mid + 1] > i) hi = mid;
            else lo = mid + 1;
        }
        const int b = lo, p = i - A.first[b];
        const int n = A.off[b + 1] - A.off[b];
        PromptItem x = {};
        x.k0 = A.koff ? A.koff[b] : A.off[b];
        x.m = A.koff ? A.koff[b + 1] - x.k0 : n;
        x.q0 = A.off[b] + p * each;
        x.n = min(each, n - p * each);
        x.last = x.m - n + p * each;
        bucket = BUCKETS - 1 - int(min((long long)(BUCKETS - 1), max(0, x.last + x.n) / unit));
        return x;
    };
    for (int i = threadIdx.x; i < total; i += PLAN_T) {
        int k;
        piece(i, k);
        atomicAdd(&count[k], 1);
    }
    __syncthreads();
    for (int k0 = 0; k0 < BUCKETS; k0 += PLAN_T) {
        const int at = scan(count[k0 + threadIdx.x]);
        count[k0 + threadIdx.x] = at;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < total; i += PLAN_T) {
        int k;
        const PromptItem x = piece(i, k);
        A.items[atomicAdd(&count[k], 1)] = x;  // (within a bucket in any order: it decides nothing but who begins)
    }
}

size_t items_bytes(int B, long long T, int G) { return align256(size_t(prompt_max_items(B, T, G)) * sizeof(PromptItem)); }

// A tensor [tokens, heads, D] as (channel, head of the group, group, token)
spec_status heads_map(CUtensorMap* map, const void* base, bool f16, int D, int group, int groups, long long tokens,
                      long long head, long long token, int box_heads, int box_tokens) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    if (!tensor_map_encoder(&enc)) return SPEC_ERR_CUDA;
    const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(group), cuuint64_t(groups), cuuint64_t(tokens)};
    const cuuint64_t strides[3] = {cuuint64_t(head) * 2, cuuint64_t(head) * 2 * group, cuuint64_t(token) * 2};
    const cuuint32_t box[4] = {64, cuuint32_t(box_heads), 1, cuuint32_t(box_tokens)};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    const CUresult r = enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                           const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SPEC_OK : SPEC_ERR_UNSUPPORTED;
}

constexpr long long MAX_TOKENS = (1ll << 30);

spec_status check_sizes(int B, long long T, long long M, int q_heads, int kv_heads) {
    if (B < 0 || T < 0 || M < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads) return SPEC_ERR_INVALID_ARG;
    if (B > (1 << 24) || T > MAX_TOKENS || M > MAX_TOKENS || kv_heads > 65535 || q_heads / kv_heads > PROMPT_ROWS)
        return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

}  // namespace

extern "C" {

size_t spec_prompt_plan_size(int B, int64_t T, int q_heads, int kv_heads) {
    if (check_sizes(B, T, 0, q_heads, kv_heads) != SPEC_OK) return 0;
    return 256 + items_bytes(B, T, q_heads / kv_heads) + align256((size_t(B) + 1) * 4);
}

spec_status spec_prompt_plan(const int32_t* offsets, const int32_t* k_offsets, int B, int64_t T, int64_t M, int q_heads,
                             int kv_heads, const int32_t* page_table, int max_pages, int page_size, int num_pages,
                             int32_t* positions, int64_t* slots, void* plan, size_t plan_bytes, int32_t* dev_status,
                             spec_stream_t stream) {
    const spec_status cs = check_sizes(B, T, M, q_heads, kv_heads);
    if (cs != SPEC_OK) return cs;
    if (!offsets || !plan || (!k_offsets && M != T)) return SPEC_ERR_INVALID_ARG;
    if (slots && !page_table) return SPEC_ERR_INVALID_ARG;
    if (page_table) {
        if (max_pages < 1 || page_size < 1 || num_pages < 1) return SPEC_ERR_INVALID_ARG;
        if (page_size % 16 || page_size > 65536) return SPEC_ERR_UNSUPPORTED;
    }
    if (!all_aligned(4, {offsets, k_offsets, page_table, positions, dev_status}) || !aligned(slots, 8))
        return SPEC_ERR_UNSUPPORTED;
    if (!aligned(plan, 256) || plan_bytes < spec_prompt_plan_size(B, T, q_heads, kv_heads)) return SPEC_ERR_WORKSPACE;
    const int G = q_heads / kv_heads;
    PlanArgs A = {};
    A.off = offsets;
    A.koff = k_offsets;
    A.table = page_table;
    A.positions = positions;
    A.slots = reinterpret_cast<long long*>(slots);
    A.plan = static_cast<PromptHead*>(plan);
    A.items = reinterpret_cast<PromptItem*>(static_cast<char*>(plan) + 256);
    A.first = reinterpret_cast<int*>(static_cast<char*>(plan) + 256 + items_bytes(B, T, G));
    A.status = dev_status;
    A.B = B;
    A.T = int(T);
    A.M = int(M);
    A.tokens = prompt_tokens(G);
    A.max_pages = max_pages;
    A.page = page_size;
    A.num_pages = num_pages;
    const unsigned grid = 1 + (positions || slots ? unsigned((T + PLAN_T - 1) / PLAN_T) : 0);
    const cudaError_t e = launch_behind(k_prompt_plan, dim3(grid), PLAN_T, 0, reinterpret_cast<cudaStream_t>(stream), A);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_prompt_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                                  int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                                  int64_t v_head_stride, spec_dtype dtype, int B, int64_t T, int64_t M, int q_heads,
                                  int kv_heads, int D, const void* plan, float scale, int window, void* out, float* lse,
                                  int32_t* dev_status, spec_stream_t stream) {
    const spec_status cs = check_sizes(B, T, M, q_heads, kv_heads);
    if (cs != SPEC_OK) return cs;
    if (D < 1 || window < 0 || !(scale > 0.f) || !(scale < 3.4e38f)) return SPEC_ERR_INVALID_ARG;
    if (dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (D % 8 || D > 256) return SPEC_ERR_UNSUPPORTED;
    if (T == 0 || B == 0) return SPEC_OK;
    if (!q || (M && (!k || !v)) || !plan || !out) return SPEC_ERR_INVALID_ARG;
    for (long long s : {(long long)q_token_stride, (long long)q_head_stride, (long long)k_token_stride,
                        (long long)k_head_stride, (long long)v_token_stride, (long long)v_head_stride})
        if (s < 0 || s % 8 || s >= (1ll << 38)) return SPEC_ERR_UNSUPPORTED;
    if (!all_aligned(16, {q, k, v, out}) || !all_aligned(4, {lse, dev_status})) return SPEC_ERR_UNSUPPORTED;
    if (!aligned(plan, 256)) return SPEC_ERR_WORKSPACE;
    const int G = q_heads / kv_heads, tokens = prompt_tokens(G);
    const bool f16 = dtype == SPEC_F16;
    PromptLaunch L;
    PromptArgs& A = L.A;
    A.plan = static_cast<const PromptHead*>(plan);
    A.out = out;
    A.lse = lse;
    A.v = v;
    A.v_token = v_token_stride;
    A.v_head = v_head_stride;
    A.T = int(T);
    A.M = int(M);
    A.Hq = q_heads;
    A.Hkv = kv_heads;
    A.G = G;
    A.D = D;
    A.tokens = tokens;
    A.window = window < M ? window : 0;  // (one that holds every key is none; sums with it stay in 32 bits)
    A.c = scale * 1.4426950408889634f;
    A.status = dev_status;
    // (without keys nothing is copied: any map will do)
    spec_status r = heads_map(&L.mq, q, f16, D, G, kv_heads, T, q_head_stride, q_token_stride, G, tokens);
    if (r == SPEC_OK) r = heads_map(&L.mo, out, f16, D, G, kv_heads, T, D, (long long)q_heads * D, G, tokens);
    if (r == SPEC_OK && M) r = heads_map(&L.mk, k, f16, D, 1, kv_heads, M, k_head_stride, k_token_stride, 1, PROMPT_KEYS);
    if (r == SPEC_OK && M) r = heads_map(&L.mv, v, f16, D, 1, kv_heads, M, v_head_stride, v_token_stride, 1, PROMPT_KEYS);
    if (r != SPEC_OK) return r;
    if (!M) L.mk = L.mv = L.mq;
    L.items = prompt_max_items(B, T, G) * kv_heads;
    if (L.items > (1ll << 30)) return SPEC_ERR_UNSUPPORTED;  // (places are 32 bits in the kernel)
    L.sms = sm_count();
    if (L.sms <= 0) return SPEC_ERR_CUDA;
    L.st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = f16 ? launch_prompt_f16(L) : launch_prompt_bf16(L);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"

// tree_attn.cu -- spec_tree_attention: argument checks, tensor maps and the
// choice of the kernel.
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "tree_attn.cuh"

using namespace sv;

namespace sv {
bool tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* out) {
    static std::mutex mu;
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    std::lock_guard<std::mutex> lk(mu);
    if (!encode) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !fn)
            return false;
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    *out = encode;
    return true;
}
}  // namespace sv

namespace {

// One side of a cache as (channel, token of the page, head, page), in boxes
// of 128 bytes of a row (channels past head_dim read as zeros) x `tokens` rows.
spec_status cache_map(CUtensorMap* map, const spec_kv_cache& c, void* base, int tokens) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    if (!tensor_map_encoder(&enc)) return SPEC_ERR_CUDA;
    const cuuint64_t es = cuuint64_t(dtype_bytes(c.dtype));
    const cuuint64_t dims[4] = {cuuint64_t(c.head_dim), cuuint64_t(c.page_size),
                                cuuint64_t(c.heads), cuuint64_t(c.num_pages)};
    const cuuint64_t strides[3] = {c.token_stride * es, c.head_stride * es, c.page_stride * es};
    const cuuint32_t box[4] = {cuuint32_t(128 / es), cuuint32_t(tokens), 1, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    const CUtensorMapDataType t = c.dtype == SPEC_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                  : c.dtype == SPEC_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUresult r = enc(map, t, 4, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SPEC_OK : SPEC_ERR_UNSUPPORTED;
}

constexpr int MAX_R = 128;  // rows of the largest tile

// channels of a part's row in the workspace, the most that a kernel lays out for D
// (k_attn_tiles 64 or 128, k_attn_rows 64, 96, 128 or 256)
int width_of(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
size_t part_o_bytes(int ctas, int D) { return align256(size_t(2) * ctas * MAX_R * width_of(D) * 4); }
size_t part_ml_bytes(int ctas) { return align256(size_t(2) * ctas * MAX_R * 2 * 4); }

// The parts that k_attn_tiles left: CTA (c, y) joins the item that starts in CTA
// c's share and ends in another's, its y-th share of the channels.  One row a
// thread (lanes side by side, so that reads are coalesced), 8 channels at most, up
// to 8 parts' reads in flight.  It finds its item while k_attn_tiles still runs
// (the plan was there before that began).
constexpr int JOIN_T = 256, JOIN_Y = 8;
__global__ void __launch_bounds__(JOIN_T) k_attn_join(const __grid_constant__ AttnArgs A, int width) {
    __shared__ PlanWindow window;
    Share share;
    Segment s = {};
    long long g0 = 0;
    bool mine = read_plan(A, window, share);
    if (mine) {
        const Lists L = {window, A.plan, window.b0};
        s = segment_at(A, L, share, share.end - 1, window.b0);
        g0 = s.g - s.t0;
        mine = g0 >= share.begin && s.t0 + 1 != s.tiles;  // not begun before this share, nor ended with it
    }
    // one CTA at least ends after k_attn_tiles, and so does this grid
    if (!mine && (blockIdx.x || blockIdx.y)) return;
    griddep_wait();
    if (!mine) return;
    const int c0 = blockIdx.x, parts = cta_of(share, g0 + s.tiles - 1) - c0 + 1;
    const int r = threadIdx.x & 127, row = s.rt * 128 + r, quads = width / 4;
    const int per = quads / JOIN_Y / (JOIN_T / 128);  // 2 (128 channels) or 1
    const int q0 = (blockIdx.y * (JOIN_T / 128) + (threadIdx.x >> 7)) * per;
    if (row >= A.rows) return;
    auto slot = [&](int c) { return 2ll * (c0 + c) + (c == 0 ? 1 : 0); };
    const float2* ml = reinterpret_cast<const float2*>(A.part_ml) + r;
    const float4* po = reinterpret_cast<const float4*>(A.part_o) + (long long)q0 * 128 + r;
    float ref = -INFINITY, total = 0.f, o[2][4] = {};
    for (int c = 0; c < parts; c += 8) {  // running sums, by the running reference
        float2 z[8];
        float4 x[8], y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool on = c + i < parts;
            z[i] = on ? __ldcg(ml + slot(c + i) * 128) : make_float2(-INFINITY, 0.f);
            x[i] = on ? __ldcg(po + slot(c + i) * quads * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
            y[i] = on && per == 2 ? __ldcg(po + slot(c + i) * quads * 128 + 128) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float to = ref;
#pragma unroll
        for (int i = 0; i < 8; ++i) to = fmaxf(to, z[i].x);
        const float at = to == -INFINITY ? 0.f : to, f = ex2_approx(ref - at);
        ref = to;
        total *= f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            o[0][e] *= f;
            o[1][e] *= f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float w = ex2_approx(z[i].x - at);  // 0 for a part that is not there
            total = fmaf(w, z[i].y, total);
            o[0][0] = fmaf(w, x[i].x, o[0][0]);
            o[0][1] = fmaf(w, x[i].y, o[0][1]);
            o[0][2] = fmaf(w, x[i].z, o[0][2]);
            o[0][3] = fmaf(w, x[i].w, o[0][3]);
            o[1][0] = fmaf(w, y[i].x, o[1][0]);
            o[1][1] = fmaf(w, y[i].y, o[1][1]);
            o[1][2] = fmaf(w, y[i].z, o[1][2]);
            o[1][3] = fmaf(w, y[i].w, o[1][3]);
        }
    }
    put_row(A, s, row, q0 * 4, o[0], total);
    if (per == 2) put_row(A, s, row, q0 * 4 + 4, o[1], total);
    if (q0 == 0) put_lse(A, s, row, ref, total);
}

}  // namespace

namespace sv {
cudaError_t launch_attn_join(const AttnLaunch& L, int width) {
    return launch_behind(k_attn_join, dim3(unsigned(L.ctas), JOIN_Y), JOIN_T, 0, L.st, L.A, width);
}
}  // namespace sv

extern "C" {

size_t spec_tree_attention_workspace_size(const spec_kv_cache* cache, int q_heads) {
    if (check_cache(cache) != SPEC_OK || q_heads < 1 || q_heads % cache->heads) return 0;
    const int sms = sm_count();
    if (sms <= 0) return 0;
    return part_o_bytes(sms, cache->head_dim) + part_ml_bytes(sms) + align256(size_t(sms) * 8);
}

spec_status spec_tree_attention(const void* q, int64_t q_batch_stride, int64_t q_node_stride,
                                int64_t q_head_stride, spec_dtype dtype, int B, int N, int q_heads,
                                const spec_kv_cache* cache, const int32_t* page_table,
                                int max_pages, const uint32_t* masks, const void* plan,
                                float scale, void* out, float* lse, void* workspace,
                                size_t workspace_bytes, int32_t* dev_status,
                                spec_stream_t stream) {
    const spec_status cs = check_cache(cache);
    if (cs != SPEC_OK) return cs;
    if (B < 0 || B > (1 << 24) || N < 1 || q_heads < 1 || max_pages < 1 || !(scale == scale))
        return SPEC_ERR_INVALID_ARG;
    if (dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (cache->dtype != SPEC_E4M3 && cache->dtype != int(dtype)) return SPEC_ERR_INVALID_ARG;
    if (N > 32 || q_heads % cache->heads || q_heads > 65536) return SPEC_ERR_UNSUPPORTED;
    if (B == 0) return SPEC_OK;
    if (!q || !page_table || !masks || !plan || !out || !workspace) return SPEC_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || q_batch_stride % 8 || q_node_stride % 8 ||
        q_head_stride % 8 || !all_aligned(4, {page_table, masks, lse, dev_status}))
        return SPEC_ERR_UNSUPPORTED;
    if (!aligned(workspace, 256) || !aligned(plan, 256) ||
        workspace_bytes < spec_tree_attention_workspace_size(cache, q_heads))
        return SPEC_ERR_WORKSPACE;
    const int sms = sm_count();
    if (sms <= 0) return SPEC_ERR_CUDA;

    AttnLaunch L;
    AttnArgs& A = L.A;
    A.q = q;
    A.qb = q_batch_stride;
    A.qn = q_node_stride;
    A.qh = q_head_stride;
    A.out = out;
    A.lse = lse;
    A.table = page_table;
    A.masks = masks;
    A.plan = plan_lists(static_cast<const int*>(plan), B);
    A.v = cache->v;
    A.ks = cache->k_scale;
    A.vs = cache->v_scale;
    A.v_page = cache->page_stride;
    A.v_head = cache->head_stride;
    A.v_token = cache->token_stride;
    A.B = B;
    A.N = N;
    A.Hq = q_heads;
    A.Hkv = cache->heads;
    A.G = q_heads / cache->heads;
    A.D = cache->head_dim;
    A.page = cache->page_size;
    A.max_pages = max_pages;
    A.num_pages = cache->num_pages;
    A.rows = N * A.G;
    A.c = scale * 1.4426950408889634f;
    A.q_f16 = dtype == SPEC_F16;
    // (the counts last: ahead of the parts they cost 7 narrow-headed requests 22.9 us, here 22.7)
    char* room = static_cast<char*>(workspace);
    A.part_o = reinterpret_cast<float*>(room);
    A.part_ml = reinterpret_cast<float*>(room += part_o_bytes(sms, A.D));
    A.arrived = reinterpret_cast<unsigned long long*>(room + part_ml_bytes(sms));
    A.status = dev_status;
    // More than 16 rows go to the tcgen05 kernels (128 a tile, heads of up to 128),
    // since k_attn_rows reads the cache again for every 16.  Measured (us, k_attn_rows /
    // tiles; 32 requests of 1000 to 16384 tokens, 200 of 30 to 1000):
    //   16 rows, 16 bits 177 / 198 and 106 / 121, 8 bits 166 / 184 and 115 / 182
    //   32 rows, 16 bits 342 / 201 and 206 / 124, 8 bits 322 / 184 and 223 / 184
    // (A form of k_attn_rows with 32 rows a tile took 212 and 148, 8 bits 233 and 164: over
    // short contexts of 8 bits it was the fastest, and over no others.)
    const bool e4 = cache->dtype == SPEC_E4M3;
    const bool tiles = A.rows > 16 && A.D <= 128;
    const int R = tiles ? 128 : 16;
    A.tiles_r = (A.rows + R - 1) / R;
    // A copy lies in one page: k_attn_rows takes chunks of 16 tokens,
    // k_attn_tiles the longest power of two up to a tile that divides a page.
    // What another item costs a CTA, in tiles: its queries, a pipeline that runs dry
    // and fills again, the join of the warps.  Measured (us without a lead / with 2 /
    // 4 / 8, or for the tile kernels 3 / 6 / 9 and 2 / 5 / 9):
    //   k_attn_rows, 256 chains over 64 to 4096 tokens 352 / 337 / 330 / 344, 64 over
    //     20 to 2000 tokens 87 / 66 / 56 / 60, heads of 256 178 / 147 / 153 / 165
    //   8 bits, 32 trees of 32 over 1000 to 16384 tokens 247 / 218 / 196 / 193, 32 rows over
    //     30 to 1000 223 / 190 / 184 / 185
    //   16 bits, the same 241 / 228 / 214 / 215
    A.lead = !tiles ? (A.D > 128 ? 2 : 4) : e4 ? 6 : 5;
    A.box = tiles ? std::min(TREE_TILE, A.page & -A.page) : 16;
    spec_status r = cache_map(&L.mk, *cache, cache->k, A.box);
    if (r == SPEC_OK) r = cache_map(&L.mv, *cache, cache->v, A.box);
    if (r != SPEC_OK) return r;
    L.ctas = sms;
    L.st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = e4                         ? launch_attn_e4m3(L, tiles)
                          : cache->dtype == SPEC_F16 ? launch_attn_f16(L, tiles)
                                                     : launch_attn_bf16(L, tiles);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"

// tree_attn_q8.cu -- attention of a tree of drafted tokens over the quantised
// paged cache (see include/indexcache.h).
//
// Row (b, i), head h, over the seen positions s (before the tree, or a node of
// the row's mask; restricted to idx[b,i,:] where it is given):
//   p = softmax_s(scale * q . KV[s, 0:576]),  out = sum_s p_s KV[s, 0:512].
//
// Simple form: one CTA per (row, 8 heads).  Tiles of 32 positions are decoded
// to float32 in shared memory; a warp computes the logits of one head and the
// online softmax, then every thread accumulates two columns of all 8 heads.
#include <algorithm>

#include "q8.cuh"

namespace ic {
namespace {

using namespace q8;

constexpr int HG = 8, KT = 32, THREADS = 256;

__global__ void __launch_bounds__(THREADS)
tree_attn_simple_kernel(const __nv_bfloat16* __restrict__ q, const uint8_t* __restrict__ cache,
                        const float* __restrict__ kv_scale,
                        const int32_t* __restrict__ idx, int k, const unsigned long long* __restrict__ tree,
                        ic_paged_rows pr, int Hq, float scale, __nv_bfloat16* __restrict__ out,
                        uint32_t* status) {
    extern __shared__ float sm[];
    float* qs = sm;                  // [HG][576]
    float* ks = qs + HG * KVW;       // [KT][577]
    float* ps = ks + KT * (KVW + 1); // [HG][KT]
    float* corr = ps + HG * KT;      // [HG]
    float* linv = corr + HG;         // [HG]
    __shared__ int seen[KT];
    const int row = blockIdx.x, h0 = blockIdx.y * HG;
    const int b = row / pr.Lq, i = row % pr.Lq;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    pdl_trigger();
    pdl_wait();
    int len = pr.seq_lens[b];
    if (len < pr.Lq || len > pr.T_max) {
        if (t == 0) flag_status(status, IC_DEV_INDEX_RANGE);
        len = 0;
    }
    const int ctx = len - pr.Lq;
    const unsigned long long own = i >= 63 ? ~0ull : (2ull << i) - 1;
    const unsigned long long mask = tree ? tree[row] : own;
    for (int c = t; c < HG * KVW; c += THREADS) {
        const int h = h0 + c / KVW;
        qs[c] = h < Hq ? __bfloat162float(q[((int64_t)row * Hq + h) * KVW + c % KVW]) * scale : 0.f;
    }
    float m = -INFINITY, l = 0.f, acc[HG][2];
    for (int h = 0; h < HG; ++h) acc[h][0] = acc[h][1] = 0.f;
    const int n = len == 0 ? 0 : idx ? k : len;
    for (int j0 = 0; j0 < n; j0 += KT) {
        __syncthreads();
        for (int kk = warp; kk < KT; kk += THREADS / 32) {
            int s = -1;
            if (j0 + kk < n) s = idx ? idx[(int64_t)row * k + j0 + kk] : j0 + kk;
            if (s != -1 && (s < 0 || s >= len)) {
                if (lane == 0) flag_status(status, IC_DEV_INDEX_RANGE);
                s = -1;
            }
            if (s >= 0 && s >= ctx && !((mask >> (s - ctx)) & 1)) s = -1;
            int64_t phys = -1;
            if (s >= 0) {
                const int page = pr.block_table[(int64_t)b * pr.max_pages + s / pr.page_size];
                if (page < 0 || page >= pr.num_pages) {
                    if (lane == 0) flag_status(status, IC_DEV_INDEX_RANGE);
                } else {
                    phys = (int64_t)page * pr.page_size + s % pr.page_size;
                }
            }
            if (lane == 0) seen[kk] = phys >= 0;
            const uint8_t* p = cache + phys * ROW;
            for (int c = lane; c < KVW; c += 32) {
                float v = 0.f;
                if (phys >= 0) {
                    if (c < DV) v = decode2(p[c]).x;
                    else v = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p + OFF_ROPE + 2 * (c - DV)));
                    v *= kv_scale[phys];
                }
                ks[kk * (KVW + 1) + c] = v;
            }
        }
        __syncthreads();
        {   // warp = head, lane = position
            float x = 0.f;
            for (int c = 0; c < KVW; ++c) x = fmaf(qs[warp * KVW + c], ks[lane * (KVW + 1) + c], x);
            if (!seen[lane]) x = -INFINITY;
            float mx = x;
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
            mx = fmaxf(mx, m);
            const float a = m == -INFINITY ? 0.f : __expf(m - mx);
            const float p = !seen[lane] ? 0.f : __expf(x - mx);
            float sum = p;
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            l = l * a + sum;
            m = mx;
            ps[warp * KT + lane] = p;
            if (lane == 0) corr[warp] = a;
        }
        __syncthreads();
        for (int h = 0; h < HG; ++h) {
            const float a = corr[h];
            acc[h][0] *= a;
            acc[h][1] *= a;
        }
        for (int kk = 0; kk < KT; ++kk) {
            if (!seen[kk]) continue;
            const float v0 = ks[kk * (KVW + 1) + t], v1 = ks[kk * (KVW + 1) + t + 256];
            for (int h = 0; h < HG; ++h) {
                acc[h][0] = fmaf(ps[h * KT + kk], v0, acc[h][0]);
                acc[h][1] = fmaf(ps[h * KT + kk], v1, acc[h][1]);
            }
        }
    }
    if (lane == 0) linv[warp] = l == 0.f ? 0.f : 1.f / l;
    __syncthreads();
    for (int h = 0; h < HG && h0 + h < Hq; ++h) {
        __nv_bfloat16* o = out + ((int64_t)row * Hq + h0 + h) * DV;
        o[t] = __float2bfloat16_rn(acc[h][0] * linv[h]);
        o[t + 256] = __float2bfloat16_rn(acc[h][1] * linv[h]);
    }
}

constexpr size_t SMEM = sizeof(float) * (HG * KVW + KT * (KVW + 1) + HG * KT + 2 * HG);

}  // namespace

size_t tree_attn_q8_scratch_bytes(const ic_paged_rows& pr, int k, int Hq) { return 0; }

ic_status launch_tree_attn_q8(const void* q, const void* kv_q8, const float* kv_scale,
                              const int32_t* idx, int k, const uint64_t* tree, const ic_paged_rows& pr, int Hq, float scale,
                              void* out, uint32_t* status, void* scratch, cudaStream_t s) {
    if ((int64_t)pr.B * pr.Lq > 0x7fffffffLL) return IC_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(tree_attn_simple_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)SMEM) != cudaSuccess)
        return cuda_error("tree_attn_q8");
    const int64_t rows = (int64_t)pr.B * pr.Lq;
    if (launch_ex(tree_attn_simple_kernel, dim3((unsigned)rows, (unsigned)ceil_div(Hq, HG)), dim3(THREADS),
                  SMEM, s, pdl_rows(rows), 0, static_cast<const __nv_bfloat16*>(q),
                  static_cast<const uint8_t*>(kv_q8), kv_scale, idx, k,
                  reinterpret_cast<const unsigned long long*>(tree), pr, Hq, scale,
                  static_cast<__nv_bfloat16*>(out), status) != cudaSuccess)
        return cuda_error("tree_attn_q8");
    count_launch(IC_LK_TREE);
    return last_launch_status();
}

}  // namespace ic

// cache_q8.cu -- writing the quantised cache and reading it back.
//
// Row n goes to (comes from) cache row slots[n]; see include/indexcache.h for
// the row format.  For a row x of 512 values (an indexer key: 128)
//   s = 2^e, e the smallest with max|x| <= 448 * 2^e;  code = e4m3(x / s),
// and back x' = code * s.  Both directions are bound by memory: a token is
// 1408 bytes of bfloat16 against 776 bytes of cache.  Measured on 64K tokens:
// writing latents and keys 24.7 us (5.8 TB/s, 89 % of a plain copy), reading
// latents back 22.6 us (5.2 TB/s, 79 %; two bytes in three are written).  That
// is the memory's rate for such a mix: without the decoding, with slots that
// need no load, with four warps a block or streaming stores it is the same to
// 1 %, two tokens a warp are no faster, a loop over tokens that loads the next
// slot ahead is slower (24.4), and so are sixteen warps a block (24.6).
//
// One warp per token, every load of the token in flight before the first is
// used; slot and data loads do not wait for one another when writing.  A lane
// takes the values of one 16-byte vector at a time (8 bfloat16 or 4 float32),
// so a warp's loads and stores are whole consecutive lines on both sides; the
// row's maximum is one integer reduction over the warp (non-negative floats
// order like their bits).  Writing was bound by its arithmetic first: vectors
// that stay packed until they are used (32 registers, a full SM of warps) took
// 64K tokens from 36.9 to 28.7 us, packed maxima and products to 24.6.
#include <algorithm>

#include "q8.cuh"

namespace ic {
namespace {

using namespace q8;

constexpr int WARPS = 8;

template <typename T> struct Vec;   // the values of one 16-byte vector
template <> struct Vec<float> { static constexpr int N = 4; };
template <> struct Vec<__nv_bfloat16> { static constexpr int N = 8; };

// N values at p, as they lie: one 16-byte load where rows start on 16-byte
// boundaries (ALIGNED), else element loads.
template <bool ALIGNED>
__device__ __forceinline__ uint4 load_vec(const float* p) {
    if (ALIGNED) return __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t* u = reinterpret_cast<const uint32_t*>(p);
    return make_uint4(__ldg(u), __ldg(u + 1), __ldg(u + 2), __ldg(u + 3));
}
template <bool ALIGNED>
__device__ __forceinline__ uint4 load_vec(const __nv_bfloat16* p) {
    if (ALIGNED) return __ldg(reinterpret_cast<const uint4*>(p));
    const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__ldg(u + 2 * i) | (uint32_t)__ldg(u + 2 * i + 1) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The values of a vector.
__device__ __forceinline__ void values_of(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void values_of(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool ALIGNED>
__device__ __forceinline__ void store_vec(float* p, const float (&x)[4]) {
    if (ALIGNED) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = x[i];
    }
}
template <bool ALIGNED>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&x)[8]) {
    if (ALIGNED) {
        *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]),
                                                  bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = __float2bfloat16_rn(x[i]);
    }
}

// The codes of a vector's values times inv, a power of two: 4 or 8 bytes.
// bfloat16 products with it are exact (what would fall under 2^-126 has the
// code 0 either way), two at a time.
__device__ __forceinline__ uint32_t mul_pair(uint32_t p, uint32_t inv2) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(p), "r"(inv2));
    return r;
}
__device__ __forceinline__ uint32_t twice(float pow2) { return (__float_as_uint(pow2) >> 16) * 0x10001u; }
__device__ __forceinline__ uint32_t encode_pair(uint32_t p) {
    return encode2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u), 1.f);
}
__device__ __forceinline__ void store_codes(uint8_t* p, const uint4& v, float inv, __nv_bfloat16) {
    const uint32_t i2 = twice(inv);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(encode_pair(mul_pair(v.x, i2)) | encode_pair(mul_pair(v.y, i2)) << 16,
                   encode_pair(mul_pair(v.z, i2)) | encode_pair(mul_pair(v.w, i2)) << 16);
}
__device__ __forceinline__ void store_codes(uint8_t* p, const uint4& v, float inv, float) {
    *reinterpret_cast<uint32_t*>(p) = encode2(__uint_as_float(v.x), __uint_as_float(v.y), inv) |
                                      encode2(__uint_as_float(v.z), __uint_as_float(v.w), inv) << 16;
}
// The same values as bfloat16, rounded once: 16 or 8 bytes.
__device__ __forceinline__ void store_scaled(uint8_t* p, const uint4& v, float inv, __nv_bfloat16) {
    const uint32_t i2 = twice(inv);
    *reinterpret_cast<uint4*>(p) = make_uint4(mul_pair(v.x, i2), mul_pair(v.y, i2), mul_pair(v.z, i2), mul_pair(v.w, i2));
}
__device__ __forceinline__ void store_scaled(uint8_t* p, const uint4& v, float inv, float) {
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(__uint_as_float(v.x) * inv, __uint_as_float(v.y) * inv),
                                              bf16_pair(__uint_as_float(v.z) * inv, __uint_as_float(v.w) * inv));
}
template <int N>
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&w)[N / 4]) {
    if constexpr (N == 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
}
template <int N>
__device__ __forceinline__ void decode_codes(const uint32_t (&w)[N / 4], float s, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const float2 a = decode2(w[i]), b = decode2(w[i] >> 16);
        x[4 * i] = a.x * s; x[4 * i + 1] = a.y * s; x[4 * i + 2] = b.x * s; x[4 * i + 3] = b.y * s;
    }
}

// Largest magnitude of a vector's values, as float32 bits: of all of them (two
// instructions a pair; 0x7f800000 or more where one is not finite), and of the
// finite ones.
__device__ __forceinline__ uint32_t vec_max(const uint4& v, __nv_bfloat16) {
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
}
__device__ __forceinline__ uint32_t vec_max(const uint4& v, float) {
    return max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
}
template <int N>
__device__ __forceinline__ uint32_t vec_finite_max(const uint4& v) {
    float x[N];
    values_of(v, x);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, finite_abs_bits(x[i]));
    return m;
}

// Exponent of the scale of a row, a warp's vectors x[0..IT).
template <typename T, int IT>
__device__ __forceinline__ int row_exponent(const uint4 (&x)[IT]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < IT; ++i) m = max(m, vec_max(x[i], T()));
    m = __reduce_max_sync(0xffffffffu, m);
    if (m >= 0x7f800000u) {
        m = 0;
#pragma unroll
        for (int i = 0; i < IT; ++i) m = max(m, vec_finite_max<Vec<T>::N>(x[i]));
        m = __reduce_max_sync(0xffffffffu, m);
    }
    return scale_exponent(m);
}

// The slot of row n: -1 for a padding row or one outside the cache.
__device__ __forceinline__ int64_t slot_of(const int32_t* slots, int64_t n, int64_t num_rows,
                                           uint32_t* status) {
    const int64_t s = slots ? (int64_t)__ldg(slots + n) : n;
    if (s >= 0 && s < num_rows) return s;
    if (s != -1 && (threadIdx.x & 31) == 0) flag_status(status, IC_DEV_INDEX_RANGE);
    return -1;
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(32 * WARPS)
cache_write_kernel(const T* __restrict__ kv, int64_t kv_stride, const T* __restrict__ k_idx,
                   int64_t k_stride, int64_t n_rows, const int32_t* __restrict__ slots,
                   uint8_t* __restrict__ kv_q8, float* __restrict__ kv_scale,
                   uint8_t* __restrict__ k_codes, float* __restrict__ k_scale, int64_t num_rows,
                   uint32_t* status) {
    constexpr int N = Vec<T>::N;
    constexpr int IT = DV / (32 * N);          // vectors of a lane in the quantised columns
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
    pdl_trigger();
    pdl_wait();
    if (n >= n_rows) return;
    // kept as they lie until they are used: 32 registers, a full SM of warps
    uint4 x[IT], rope, key[1] = {make_uint4(0u, 0u, 0u, 0u)};
    if (kv) {
        const T* p = kv + n * kv_stride;
#pragma unroll
        for (int i = 0; i < IT; ++i) x[i] = load_vec<ALIGNED>(p + (i * 32 + lane) * N);
        if (lane < DR / N) rope = load_vec<ALIGNED>(p + DV + lane * N);
    }
    if (k_idx && lane < DI / N) key[0] = load_vec<ALIGNED>(k_idx + n * k_stride + lane * N);
    const int64_t slot = slot_of(slots, n, num_rows, status);
    if (slot < 0) return;
    if (kv) {
        uint8_t* row = kv_q8 + slot * ROW;
        const int e = row_exponent<T>(x);
#pragma unroll
        for (int i = 0; i < IT; ++i) store_codes(row + (i * 32 + lane) * N, x[i], exp2_int(-e), T());
        if (lane == 0) kv_scale[slot] = exp2_int(e);
        if (lane < DR / N) store_scaled(row + OFF_ROPE + lane * N * 2, rope, exp2_int(-e), T());
    }
    if (k_idx) {
        const int e = row_exponent<T>(key);
        if (lane < DI / N) store_codes(k_codes + slot * DI + lane * N, key[0], exp2_int(-e), T());
        if (lane == 0) k_scale[slot] = exp2_int(e);
    }
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(32 * WARPS)
cache_read_kernel(const uint8_t* __restrict__ kv_q8, const float* __restrict__ kv_scale,
                  const uint8_t* __restrict__ k_codes, const float* __restrict__ k_scale,
                  int64_t num_rows, int64_t n_rows, const int32_t* __restrict__ slots,
                  T* __restrict__ kv, int64_t kv_stride, T* __restrict__ k_idx, int64_t k_stride,
                  uint32_t* status) {
    constexpr int N = Vec<T>::N;
    constexpr int IT = DV / (32 * N);
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
    pdl_trigger();
    pdl_wait();
    if (n >= n_rows) return;
    const int64_t slot = slot_of(slots, n, num_rows, status);
    uint32_t w[IT][N / 4], kw[N / 4];
    uint32_t rope[N / 2];
    float s = 0.f, ks = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int j = 0; j < N / 4; ++j) w[i][j] = 0u;
#pragma unroll
    for (int j = 0; j < N / 4; ++j) kw[j] = 0u;
#pragma unroll
    for (int j = 0; j < N / 2; ++j) rope[j] = 0u;
    if (kv && slot >= 0) {
        const uint8_t* row = kv_q8 + slot * ROW;
#pragma unroll
        for (int i = 0; i < IT; ++i) load_codes<N>(row + (i * 32 + lane) * N, w[i]);
        s = __ldg(kv_scale + slot);
        if (lane < DR / N) {
            const uint32_t* d = reinterpret_cast<const uint32_t*>(row + OFF_ROPE) + lane * (N / 2);
#pragma unroll
            for (int j = 0; j < N / 2; j += 2) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(d + j));
                rope[j] = v.x; rope[j + 1] = v.y;
            }
        }
    }
    if (k_idx && slot >= 0 && lane < DI / N) {
        load_codes<N>(k_codes + slot * DI + lane * N, kw);
        ks = __ldg(k_scale + slot);
    }
    float x[N];
    if (kv) {
        T* p = kv + n * kv_stride;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            decode_codes<N>(w[i], s, x);
            store_vec<ALIGNED>(p + (i * 32 + lane) * N, x);
        }
        if (lane < DR / N) {
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                x[2 * j] = __uint_as_float(rope[j] << 16) * s;
                x[2 * j + 1] = __uint_as_float(rope[j] & 0xffff0000u) * s;
            }
            store_vec<ALIGNED>(p + DV + lane * N, x);
        }
    }
    if (k_idx && lane < DI / N) {
        decode_codes<N>(kw, ks, x);
        store_vec<ALIGNED>(k_idx + n * k_stride + lane * N, x);
    }
}

// Every row of an array starts on a 16-byte boundary.
bool rows_aligned(const void* p, int64_t stride, int esize) {
    return p == nullptr || (((uintptr_t)p & 15) == 0 && stride * esize % 16 == 0);
}

template <typename T>
ic_status write_rows(const void* kv, int64_t kv_stride, const void* k_idx, int64_t k_stride, int64_t n,
                     const int32_t* slots, void* kv_q8, float* kv_scale, void* k_codes,
                     float* k_scale, int64_t num_rows, uint32_t* status, cudaStream_t s) {
    const bool aligned = rows_aligned(kv, kv_stride, sizeof(T)) && rows_aligned(k_idx, k_stride, sizeof(T));
    auto kern = aligned ? cache_write_kernel<T, true> : cache_write_kernel<T, false>;
    if (launch_ex(kern, dim3((unsigned)ceil_div64(n, WARPS)), dim3(32 * WARPS), 0, s, pdl_rows(n), 0,
                  static_cast<const T*>(kv), kv_stride, static_cast<const T*>(k_idx), k_stride, n,
                  slots, static_cast<uint8_t*>(kv_q8), kv_scale, static_cast<uint8_t*>(k_codes),
                  k_scale, num_rows, status) != cudaSuccess)
        return cuda_error("cache_q8");
    count_launch(IC_LK_CACHE);
    return last_launch_status();
}

template <typename T>
ic_status read_rows(const void* kv_q8, const float* kv_scale, const void* k_codes,
                    const float* k_scale, int64_t num_rows, int64_t n, const int32_t* slots, void* kv, int64_t kv_stride, void* k_idx,
                    int64_t k_stride, uint32_t* status, cudaStream_t s) {
    const bool aligned = rows_aligned(kv, kv_stride, sizeof(T)) && rows_aligned(k_idx, k_stride, sizeof(T));
    auto kern = aligned ? cache_read_kernel<T, true> : cache_read_kernel<T, false>;
    if (launch_ex(kern, dim3((unsigned)ceil_div64(n, WARPS)), dim3(32 * WARPS), 0, s, pdl_rows(n), 0,
                  static_cast<const uint8_t*>(kv_q8), kv_scale, static_cast<const uint8_t*>(k_codes),
                  k_scale, num_rows, n, slots, static_cast<T*>(kv), kv_stride, static_cast<T*>(k_idx), k_stride,
                  status) != cudaSuccess)
        return cuda_error("cache_q8");
    count_launch(IC_LK_CACHE);
    return last_launch_status();
}

}  // namespace

ic_status launch_cache_write_q8(const void* kv, int64_t kv_stride, const void* k_idx,
                                int64_t k_stride, ic_dtype dt, int64_t n, const int32_t* slots,
                                void* kv_q8, float* kv_scale, void* k_codes, float* k_scale,
                                int64_t num_rows, uint32_t* status, cudaStream_t s) {
    auto f = dt == IC_F32 ? write_rows<float> : write_rows<__nv_bfloat16>;
    return f(kv, kv_stride, k_idx, k_stride, n, slots, kv_q8, kv_scale, k_codes, k_scale, num_rows,
             status, s);
}

ic_status launch_cache_read_q8(const void* kv_q8, const float* kv_scale, const void* k_codes,
                               const float* k_scale, int64_t num_rows, int64_t n,
                               const int32_t* slots, ic_dtype dt, void* kv, int64_t kv_stride,
                               void* k_idx, int64_t k_stride, uint32_t* status, cudaStream_t s) {
    auto f = dt == IC_F32 ? read_rows<float> : read_rows<__nv_bfloat16>;
    return f(kv_q8, kv_scale, k_codes, k_scale, num_rows, n, slots, kv, kv_stride, k_idx, k_stride,
             status, s);
}

}  // namespace ic

// kv_common.h -- what the KV-cache operators' kernels share: the cache as a
// kernel sees it, element types and wave-wide steps. Internal to the library.
#ifndef UZIP_KV_COMMON_H
#define UZIP_KV_COMMON_H

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "uzip_kv.h"

namespace uzip_kv {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kBF16 = (int)UZIP_KV_BF16, kF16 = (int)UZIP_KV_F16, kE5M2 = (int)UZIP_KV_E5M2;
constexpr uint32_t kCUs = 256;                   // of the one GPU this library is for
constexpr uint64_t kLaunchThreads = 1ull << 32;  // a launch has fewer
constexpr int64_t kMaxTokenStride = 1ll << 26;   // elements: 16 rows' offsets fit 32 bits

constexpr uint32_t elem_size(int dtype) { return dtype >= kE5M2 ? 1u : 2u; }

// A cache as kernels see it; strides in bytes. Capacity, page table and pool
// bounds are the host's, so no device value can lead outside them.
struct CacheView {
    char *k, *v;
    const int32_t *table;
    int64_t ks0, ks1, ks2, vs0, vs1, vs2, ts;
    uint32_t tokens, shift, pages;
};

// Scales of an 8-bit cache as kernels see them; strides in elements: page or
// sequence, block, head. No offset reaches 2^30, so 32 bits do.
struct ScaleView {
    float *k, *v;
    uint32_t k0, k1, k2, v0, v1, v2;
    uint32_t shift;                                  // of a block's tokens
};

// a load at an address that is the same for a whole wave, of memory that the kernel does not write
__device__ inline float scalar_load(const float *p)
{
    return *(const __attribute__((address_space(4))) float *)p;
}

// Byte offset of token t's page or sequence plus its row, or false when it
// lies in an absent page. t < c.tokens.
__device__ inline bool locate(const CacheView &c, int64_t b, uint32_t t, int64_t s0, int64_t s1, int64_t &off)
{
    if (!c.table) {
        off = b * s0 + (int64_t)t * s1;
        return true;
    }
    const uint32_t p = (uint32_t)c.table[b * c.ts + (t >> c.shift)];
    off = (int64_t)p * s0 + (int64_t)(t & ((1u << c.shift) - 1)) * s1;
    return p < c.pages;
}

// length clamped to the capacity; the drafted count to [0, T]
__device__ inline int clamp_length(const int32_t *length, int b, uint32_t tokens)
{
    const int n = length[b];
    return n < 0 ? 0 : (uint32_t)n > tokens ? (int)tokens : n;
}

__device__ inline int clamp_drafted(const int32_t *drafted, int b, int T)
{
    if (!drafted) return T;
    const int n = drafted[b];
    return n < 0 ? 0 : n > T ? T : n;
}

__device__ inline float bf16_to_f32(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ inline float f16_to_f32(uint16_t x) { return (float)__builtin_bit_cast(_Float16, x); }

// two floats to two 16-bit values, each rounded once to nearest even
template <bool F16>
__device__ inline uint32_t pack2(float a, float b)
{
    const f32x2 v = {a, b};
    if constexpr (F16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// ... each cut off toward zero
template <bool F16>
__device__ inline uint32_t cut2(float a, float b)
{
    if constexpr (F16)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
    else
        return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

template <bool F16>
__device__ inline f32x2 unpack2(uint32_t w)
{
    if constexpr (F16) {
        const f16x2 h = __builtin_bit_cast(f16x2, w);
        return f32x2{(float)h.x, (float)h.y};
    } else {
        return f32x2{__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
    }
}

// four floats to four E5M2 bytes, to nearest even, out-of-range to infinity
__device__ inline uint32_t pack4_e5m2(float a, float b, float c, float d)
{
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
}

// max (a NaN loses) and sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48
__device__ inline float quad_max(float x)
{
    u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false));
    x = fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
    r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false));
    return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}

__device__ inline float quad_sum(float x)
{
    u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false));
    x = __uint_as_float(r.x) + __uint_as_float(r.y);
    r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false));
    return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// ------------------------------------------------------------- host checks --
inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline int hip_failed(hipError_t e, const char *what)
{
    fprintf(stderr, "uzip_kv: %s: %s\n", what, hipGetErrorString(e));
    return UZIP_EHIP;
}

#define UZIP_KV_LAUNCH_CHECK(what)                                      \
    do {                                                                \
        const hipError_t e_ = hipGetLastError();                        \
        if (e_ != hipSuccess) return uzip_kv::hip_failed(e_, what);     \
    } while (0)

inline bool valid_strides(const int64_t s[3])
{
    for (int i = 0; i < 3; i++)
        if (s[i] < 0 || (s[i] & 7) || s[i] > (1ll << 40)) return false;
    return s[1] < kMaxTokenStride;
}

inline bool valid_tensor(const uzip_kv_tensor_t &t) { return t.data && aligned(t.data, 16) && valid_strides(t.stride); }

inline bool same_tensor(const uzip_kv_tensor_t &a, const uzip_kv_tensor_t &b)
{
    return a.stride[0] == b.stride[0] && a.stride[1] == b.stride[1] && a.stride[2] == b.stride[2];
}

// a's queries, whose output they are, turned; checked by the caller
int turn_in_place(const uzip_kv_append_args_t *a, uint32_t seqs, uint32_t dim, const uzip_kv_rope_t *rope, hipStream_t s);

inline bool valid_dims(uint32_t seqs, uint32_t heads, uint32_t dim)
{
    return seqs >= 1 && seqs <= 65535 && heads >= 1 && heads <= 4096 && dim >= 8 && dim <= 256 && dim % 8 == 0;
}

// scaled: of the types that go with scales, else of the others
inline bool valid_cache(const uzip_kv_cache_t *c, bool scaled = false)
{
    if (!c || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return false;
    if (scaled ? c->dtype != UZIP_KV_E4M3 && c->dtype != UZIP_KV_I8 : c->dtype > UZIP_KV_E5M2) return false;
    if (!valid_dims(c->seqs, c->heads, c->dim) || !valid_strides(c->k_stride) || !valid_strides(c->v_stride)) return false;
    if (c->tokens < 1 || c->tokens > (1u << 30) || c->reserved) return false;
    if (!c->table) return true;
    return aligned(c->table, 4) && c->page >= 16 && c->page <= (1u << 30) && !(c->page & (c->page - 1)) &&
           c->tokens % c->page == 0 && c->pages >= 1 && c->pages <= 0x7fffffffu && c->table_stride >= 0 &&
           c->table_stride <= (1ll << 40);
}

inline bool valid_scales(const uzip_kv_scales_t *f, const uzip_kv_cache_t *c)
{
    if (!f || !f->k || !f->v || !aligned(f->k, 4) || !aligned(f->v, 4) || f->reserved) return false;
    if (f->block < 16 || f->block > 65536 || (f->block & (f->block - 1)) || (c->table && f->block > c->page)) return false;
    const uint64_t most[3] = {c->table ? c->pages : c->seqs, ((c->table ? c->page : c->tokens) + (uint64_t)f->block - 1) / f->block, c->heads};
    uint64_t k = 0, v = 0;
    for (int i = 0; i < 3; i++) {
        if (f->k_stride[i] < 0 || f->v_stride[i] < 0 || f->k_stride[i] >= (1ll << 30) || f->v_stride[i] >= (1ll << 30)) return false;
        k += (most[i] - 1) * (uint64_t)f->k_stride[i], v += (most[i] - 1) * (uint64_t)f->v_stride[i];
    }
    return k < (1ull << 30) && v < (1ull << 30);
}

inline ScaleView view_of(const uzip_kv_scales_t *f)
{
    const auto u = [](int64_t x) { return (uint32_t)x; };
    return {f->k, f->v, u(f->k_stride[0]), u(f->k_stride[1]), u(f->k_stride[2]), u(f->v_stride[0]), u(f->v_stride[1]), u(f->v_stride[2]),
            (uint32_t)__builtin_ctz(f->block)};
}

inline bool valid_rope(const uzip_kv_rope_t *r, uint32_t dim)
{
    if (r->reserved || (r->rot & 1) || r->rot > dim || (r->flags & ~(UZIP_KV_INTERLEAVED | UZIP_KV_INVERSE))) return false;
    if (r->rot && (!r->freq || !aligned(r->freq, 8))) return false;
    if (!(fabsf(r->amplitude) < INFINITY) || r->pos_stride < 0) return false;
    return aligned(r->pos, 4);
}

inline CacheView view_of(const uzip_kv_cache_t *c)
{
    CacheView v;
    const int64_t es = elem_size((int)c->dtype);
    v.k = static_cast<char *>(c->k);
    v.v = static_cast<char *>(c->v);
    v.table = c->table;
    v.ks0 = c->k_stride[0] * es, v.ks1 = c->k_stride[1] * es, v.ks2 = c->k_stride[2] * es;
    v.vs0 = c->v_stride[0] * es, v.vs1 = c->v_stride[1] * es, v.vs2 = c->v_stride[2] * es;
    v.ts = c->table_stride;
    v.tokens = c->tokens;
    v.shift = c->table ? (uint32_t)__builtin_ctz(c->page) : 0;
    v.pages = c->pages;
    return v;
}

}  // namespace uzip_kv

#endif

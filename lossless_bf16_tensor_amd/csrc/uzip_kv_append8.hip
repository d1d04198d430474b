// uzip_kv_append8.hip -- appending to a KV cache in 8 bits with a scale for
// each block of tokens and head (gfx950, wave64). The C-ABI is declared in
// include/uzip_kv.h.
//
// The new tokens of one block and head share a scale: the block's own, if its
// earlier tokens have one that holds them, else the smallest power of two that
// does. A power of two makes x / scale exact, so an element is rounded once;
// and where a block's scale grows under its earlier tokens, those lose bits at
// the end and nothing else. Growing by less than a factor of two is not
// possible, so that happens rarely: with amax / 127 every new maximum in a
// block, 3.4 in 16 tokens on average, would round all earlier ones again.
#include "kv_common.h"

namespace uzip_kv {
namespace {

constexpr int kThreads = 256, kAppendWaves = kThreads / 64;
constexpr int kKeep = 4;                          // units of 8 elements that a lane holds between the two passes, at most
constexpr int kAngles = 8192;                     // of a workgroup in LDS, at most

struct Append8Params {
    const char *q, *k, *v;
    char *y;
    int64_t qs0, qs1, qs2, ys0, ys1, ys2;         // bytes
    int64_t ks0, ks1, ks2, vs0, vs1, vs2;
    CacheView c;
    ScaleView f;
    const double *freq;
    const int32_t *pos, *length, *drafted;
    int64_t pos_stride;
    float amplitude;
    int T, Hq, H, D, rot;
    int interleaved, inverse;
    uint32_t per_magic;                           // 2^32 / (D / 8), rounded up; unused where that is 2^32
    int blocks, groups, items, waves;             // of a sequence; workgroups a block; heads' keys or values a workgroup; waves an item
    int kv_grid;                                  // workgroups before those of the queries
    int q_tokens, q_parts, q_share;               // tokens a workgroup, or workgroups a token and units of each
    int64_t q_count;                              // tokens of all sequences
    int angles;                                   // of a workgroup in LDS; 0: worked out where they are used
};

// cos and sin of position * freq turns: binary64 up to the fraction of a turn,
// and what its rounding to binary32 left over added in, since an element next
// to a border between two 8-bit values goes by its last bits.
__device__ inline float2 angle_of(const Append8Params &p, int64_t pos, int i)
{
    double turns = (double)pos * p.freq[i];
    turns -= rint(turns);
    const float half = (float)(2.0 * turns);
    const float left = (float)(2.0 * turns - (double)half) * 3.14159265f;
    float s, c;
    sincospif(half, &s, &c);
    const float s1 = fmaf(c, left, s), c1 = fmaf(-s, left, c);
    return make_float2(c1 * p.amplitude, p.inverse ? -s1 * p.amplitude : s1 * p.amplitude);
}

// How heads turn: not at all; as halves of whole units of 8 elements; in any
// other way, a unit's elements one by one; and so with more angles than LDS
// holds for a workgroup, which are worked out where they are used.
enum { kStill, kHalves, kAny, kFar };
constexpr int kept_units(int mode) { return mode <= kHalves ? kKeep : 1; }

// Eight elements of a head as they are read, and those they turn with.
struct Eight {
    u32x4 w, z;
};

template <bool F16>
__device__ inline void unpack8(u32x4 w, float (&x)[8])
{
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const f32x2 v = unpack2<F16>(w[e]);
        x[2 * e] = v.x, x[2 * e + 1] = v.y;
    }
}

template <int MODE>
__device__ inline Eight load8(const Append8Params &p, const char *row, int d, bool turns)
{
    Eight r;
    r.w = *reinterpret_cast<const u32x4 *>(row + d * 2);
    if constexpr (MODE == kHalves) {
        const int half = p.rot / 2;
        r.z = r.w;
        if (turns && d < p.rot) r.z = *reinterpret_cast<const u32x4 *>(row + (d < half ? d + half : d - half) * 2);
    } else if constexpr (MODE != kStill) {
        r.z = u32x4{0, 0, 0, 0};
        const int half = p.rot / 2;
        if (turns && !p.interleaved)
            for (int e = 0; e < 8; e += 2) {      // rot is even, so both turn or neither does
                if (d + e >= p.rot) break;
                const int i = d + e < half ? d + e + half : d + e - half, j = d + e + 1 < half ? d + e + 1 + half : d + e + 1 - half;
                const uint32_t two = *reinterpret_cast<const uint16_t *>(row + i * 2) | (uint32_t)*reinterpret_cast<const uint16_t *>(row + j * 2) << 16;
                r.z[0] = e == 0 ? two : r.z[0], r.z[1] = e == 2 ? two : r.z[1], r.z[2] = e == 4 ? two : r.z[2], r.z[3] = e == 6 ? two : r.z[3];
            }
    }
    return r;
}

// ... turned. cs: the token's angles.
template <bool F16, int MODE>
__device__ inline void turned8(const Append8Params &p, const Eight &r, int d, bool turns, const float2 *cs, int64_t pos, float (&y)[8])
{
    unpack8<F16>(r.w, y);
    if constexpr (MODE == kStill) return;
    if (!turns || d >= p.rot) return;
    const int half = p.rot / 2;
    float o[8];                                   // the elements' partners
    if constexpr (MODE == kHalves) {
        unpack8<F16>(r.z, o);
        const bool lead = d < half;
        const float sign = lead ? -1.f : 1.f;
        const float2 *at = cs + (lead ? d : d - half);
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const float2 a = at[e];
            y[e] = fmaf(y[e], a.x, o[e] * a.y * sign);
        }
    } else {
        unpack8<F16>(r.z, o);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float2 a[2];
            float sign[2];
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const int at = min(d + e + k, p.rot - 1);
                const bool lead = p.interleaved ? k == 0 : at < half;
                const int i = p.interleaved ? at >> 1 : lead ? at : at - half;
                a[k] = MODE == kFar ? angle_of(p, pos, i) : cs[i];
                sign[k] = lead ? -a[k].y : a[k].y;
            }
            const float x0 = y[e], x1 = y[e + 1], o0 = p.interleaved ? x1 : o[e], o1 = p.interleaved ? x0 : o[e + 1];
            const bool in = d + e < p.rot;
            y[e] = in ? fmaf(x0, a[0].x, o0 * sign[0]) : x0;
            y[e + 1] = in ? fmaf(x1, a[1].x, o1 * sign[1]) : x1;
        }
    }
}

// What an element type can hold, and rounding to it, to nearest even: beyond
// its range the largest value; NaN stays in E4M3 and is zero in integers.
template <bool I8>
struct Byte {
    static constexpr float kMost = I8 ? 127.f : 448.f;

    // the smallest power of two, 2^-60 or more, times which kMost is not below a finite a
    __device__ inline static float scale_for(float a)
    {
        const uint32_t u = __float_as_uint(a);
        const int down = I8 ? (u & 0x7fffffu) <= 0x7e0000u ? 7 : 6 : (u & 0x7fffffu) <= 0x600000u ? 9 : 8;
        const int e = max((int)(u >> 23) - 126 - down, -60);
        return __uint_as_float((uint32_t)(e + 127) << 23);
    }

    __device__ inline static float held(float x)
    {
        const float y = __builtin_amdgcn_fmed3f(x, -kMost, kMost);
        return x != x ? (I8 ? 0.f : x) : y;
    }

    __device__ inline static uint32_t pack4(float a, float b, float c, float d)
    {
        if constexpr (I8) {
            // an integer added to 1.5 * 2^23 is its low bits, rounded to nearest even
            constexpr float k = 12582912.f;
            const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(held(b) + k), __float_as_uint(held(a) + k), 0x0c0c0400u);
            return __builtin_amdgcn_perm(__float_as_uint(held(d) + k), __float_as_uint(held(c) + k), 0x04000c0cu) | lo;
        } else {
            const int w = __builtin_amdgcn_cvt_pk_fp8_f32(held(a), held(b), 0, false);
            return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(held(c), held(d), w, true);
        }
    }

    __device__ inline static u32x2 pack8(const float (&y)[8]) { return u32x2{pack4(y[0], y[1], y[2], y[3]), pack4(y[4], y[5], y[6], y[7])}; }

    __device__ inline static void unpack4(uint32_t w, float (&y)[8], int at)
    {
        if constexpr (I8) {
#pragma unroll
            for (int e = 0; e < 4; e++) y[at + e] = (float)(int8_t)(w >> 8 * e);
        } else {
            const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
            y[at] = a.x, y[at + 1] = a.y, y[at + 2] = b.x, y[at + 3] = b.y;
        }
    }
};

// x / s, correctly rounded: by the reciprocal where that is exact
__device__ inline void divide8(float (&y)[8], float s)
{
    if ((__float_as_uint(s) & 0x7fffffu) == 0 && s >= 0x1p-126f && s <= 0x1p126f) {
        const float inv = 1.f / s;
#pragma unroll
        for (int e = 0; e < 8; e++) y[e] *= inv;
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++) y[e] /= s;
    }
}

template <bool F16, int MODE>
__device__ inline void turn_queries(const Append8Params &p, float2 *cs)
{
    constexpr int KEEP = kept_units(MODE);
    const int id = (int)blockIdx.x - p.kv_grid, part = id % p.q_parts, tid = (int)threadIdx.x;
    const int64_t first = (int64_t)(id / p.q_parts) * p.q_tokens;
    const int tokens = (int)min((int64_t)p.q_tokens, p.q_count - first), half = p.rot / 2, per = p.D / 8;
    const auto position = [&](int64_t at) {
        const int64_t b = at / p.T, t = at - b * p.T;
        return p.pos ? (int64_t)p.pos[b * p.pos_stride + t] : (int64_t)p.length[b] + t;
    };
    const int u0 = part * p.q_share, u1 = min(u0 + p.q_share, tokens * p.Hq * per);
    Eight raw[KEEP];
    const auto fetch = [&](int base) {
#pragma unroll
        for (int r = 0; r < KEEP; r++) {
            if (base + r * kThreads >= u1) continue;
            const int u = min(base + r * kThreads + tid, u1 - 1), head = u / per % p.Hq;
            const int64_t at = first + u / per / p.Hq, b = at / p.T, t = at - b * p.T;
            raw[r] = load8<MODE>(p, p.q + b * p.qs0 + t * p.qs1 + head * p.qs2, u % per * 8, true);
        }
    };
    fetch(u0);
    if (MODE != kFar && MODE != kStill) {
        for (int j = tid; j < tokens * half; j += kThreads) cs[j] = angle_of(p, position(first + j / half), j % half);
        __syncthreads();
    }
    for (int base = u0; base < u1; base += KEEP * kThreads) {
        if (base > u0) fetch(base);
#pragma unroll
        for (int r = 0; r < KEEP; r++) {
            const int u = base + r * kThreads + tid;
            if (u >= u1) continue;
            const int d = u % per * 8, head = u / per % p.Hq, token = u / per / p.Hq;
            const int64_t at = first + token, b = at / p.T, t = at - b * p.T;
            float y[8];
            turned8<F16, MODE>(p, raw[r], d, true, cs + token * half, MODE == kFar ? position(at) : 0, y);
            u32x4 w = raw[r].w;
            const int keep = max(0, min(p.rot - d, 8));       // elements from here on keep their bits
#pragma unroll
            for (int e = 0; e < 4; e++) w[e] = 2 * e < keep ? pack2<F16>(y[2 * e], y[2 * e + 1]) : w[e];
            *reinterpret_cast<u32x4 *>(p.y + b * p.ys0 + t * p.ys1 + head * p.ys2 + d * 2) = w;
        }
    }
}

// One launch: workgroups for the keys and values of a block of tokens of some
// heads, then those that turn queries. A wave (or, of long blocks, the four of
// a workgroup) takes the keys or values of a head: turns the new tokens, finds
// their largest magnitude, and rounds what it holds in registers. Bound by
// memory where there is much: 2 x 8192 decoded tokens of 8 heads of 128 into
// integers in pages, blocks of 16, 25 us, 3.9 TB/s (a copy 5.1; every element is
// read once, and a wave's loads, their maximum and the stores follow each
// other). One token with 64 query heads 4.7 us: the trips to memory for the
// length, the tokens and the scale, and the angles. Long blocks are slow: one
// workgroup takes a block of a head, 2 x 8192 tokens of 8 heads into E4M3 in
// blocks of 64, 256 and 1024 22, 25 and 64 us; turned, by angles that LDS holds
// for 128 tokens of 128 dims and that every head works out for itself beyond, 54,
// 147 and 363. And where one token raises a block's scale, one wave rounds the
// earlier ones again, a trip to memory after the other: 8 heads of 128, the last
// token of blocks of 128, 1024 and 65536, 12, 71 and 6500 us a call.
template <bool F16, bool I8, int MODE>
__global__ __launch_bounds__(kThreads, MODE == kStill ? 4 : 3) void k_append8(Append8Params p)
{
    using E = Byte<I8>;
    constexpr int KEEP = kept_units(MODE);
    extern __shared__ float2 cs[];
    __shared__ float wave_top[kAppendWaves];
    if ((int)blockIdx.x >= p.kv_grid) {
        turn_queries<F16, MODE>(p, cs);
        return;
    }
    int id = (int)blockIdx.x;
    const int group = id % p.groups;
    id /= p.groups;
    const int b = id / p.blocks, j = id % p.blocks;
    const int tid = (int)threadIdx.x, half = p.rot / 2;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the block's tokens [s0, ..), of which [lo, hi) are new
    const int64_t n = p.length[b], nd = clamp_drafted(p.drafted, b, p.T);
    const int64_t s0 = ((max(n, (int64_t)0) >> p.f.shift) + j) << p.f.shift;
    const int64_t lo = max(s0, n), hi = min(min(s0 + (1ll << p.f.shift), n + nd), (int64_t)p.c.tokens);
    int64_t ko, vo;
    if (lo >= hi || !locate(p.c, b, (uint32_t)s0, p.c.ks0, p.c.ks1, ko)) return;
    locate(p.c, b, (uint32_t)s0, p.c.vs0, p.c.vs1, vo);
    const int rows = (int)(hi - lo), skip = (int)(lo - s0), t0 = (int)(lo - n);    // skip: earlier tokens
    const uint32_t first = p.c.table ? (uint32_t)p.c.table[b * p.c.ts + (s0 >> p.c.shift)] : (uint32_t)b;
    const uint32_t block = (uint32_t)((p.c.table ? s0 & ((1ll << p.c.shift) - 1) : s0) >> p.f.shift);
    const auto position = [&](int row) { return p.pos ? (int64_t)p.pos[b * p.pos_stride + t0 + row] : lo + row; };
    const int per = p.D / 8, units = rows * per;
    const int lanes = p.waves * 64, lane = p.waves == 1 ? tid & 63 : tid;
    const int item = group * p.items + (p.waves == 1 ? wave : 0);      // of the wave, or of all four
    const auto row_of = [&](int u) { return per == 1 ? u : (int)__umulhi((uint32_t)u, p.per_magic); };

    // where the item is, its scale and its first elements
    const bool there = item < 2 * p.H, val = item >= p.H;
    const int h = val ? item - p.H : item;
    const char *src = val ? p.v + b * p.vs0 + t0 * p.vs1 + h * p.vs2 : p.k + b * p.ks0 + t0 * p.ks1 + h * p.ks2;
    const int64_t ss = val ? p.vs1 : p.ks1, ds = val ? p.c.vs1 : p.c.ks1;
    char *dst = val ? p.c.v + vo + h * p.c.vs2 : p.c.k + ko + h * p.c.ks2;
    float *scale = val ? p.f.v + (first * p.f.v0 + block * p.f.v1 + h * p.f.v2) : p.f.k + (first * p.f.k0 + block * p.f.k1 + h * p.f.k2);
    float before = 0.f;
    Eight raw[KEEP];
    if (there) {
#pragma unroll
        for (int r = 0; r < KEEP; r++) {
            if (r * lanes >= units) continue;
            const int u = min(r * lanes + lane, units - 1), row = row_of(u);
            raw[r] = load8<MODE>(p, src + row * ss, (u - row * per) * 8, !val);
        }
        before = *scale;
    }
    if (MODE != kFar && MODE != kStill && group * p.items < p.H) {
        for (int i = tid; i < rows * half; i += kThreads) cs[i] = angle_of(p, position(i / half), i % half);
        __syncthreads();
    }
    if (!there) return;
    const auto elements = [&](const Eight &r, int u, float (&y)[8]) {
        const int row = row_of(u);
        turned8<F16, MODE>(p, r, (u - row * per) * 8, !val, cs + row * half, MODE == kFar && !val ? position(row) : 0, y);
    };
    const auto again = [&](int u) {
        const int row = row_of(u);
        return load8<MODE>(p, src + row * ss, (u - row * per) * 8, !val);
    };
    float top = 0.f;
    const auto look = [&](const float (&y)[8]) {
#pragma unroll
        for (int e = 0; e < 8; e++) top = fabsf(y[e]) < INFINITY ? fmaxf(top, fabsf(y[e])) : top;
    };
    float kept[KEEP][8];
#pragma unroll
    for (int r = 0; r < KEEP; r++) {
        if (r * lanes >= units) continue;
        elements(raw[r], min(r * lanes + lane, units - 1), kept[r]);
        look(kept[r]);
    }
    for (int u = KEEP * lanes + lane; u < units; u += lanes) {
        float y[8];
        elements(again(u), u, y);
        look(y);
    }
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    if (p.waves > 1) {
        if ((tid & 63) == 0) wave_top[wave] = top;
        __syncthreads();                      // and all waves have read the scale
        top = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));
    }
    const float now = skip && top <= before * E::kMost ? before : E::scale_for(top);
    if (skip && now != before) {              // the earlier tokens in the new scale
        const float ratio = before / now;
        for (int u = lane; u < skip * per; u += lanes) {
            const int row = row_of(u);
            u32x2 *at = reinterpret_cast<u32x2 *>(dst + row * ds + (u - row * per) * 8);
            const u32x2 w = *at;
            float y[8];
            E::unpack4(w.x, y, 0);
            E::unpack4(w.y, y, 4);
#pragma unroll
            for (int e = 0; e < 8; e++) y[e] *= ratio;
            *at = E::pack8(y);
        }
    }
    const auto put = [&](int u, float (&y)[8]) {
        const int row = row_of(u);
        divide8(y, now);
        *reinterpret_cast<u32x2 *>(dst + (skip + row) * ds + (u - row * per) * 8) = E::pack8(y);
    };
#pragma unroll
    for (int r = 0; r < KEEP; r++) {
        const int u = r * lanes + lane;
        if (u < units) put(u, kept[r]);
    }
    for (int u = KEEP * lanes + lane; u < units; u += lanes) {
        float y[8];
        elements(again(u), u, y);
        put(u, y);
    }
    if (lane == 0) *scale = now;
}

template <int MODE>
void launch_append8(const Append8Params &p, dim3 grid, bool f16, bool i8, hipStream_t s)
{
    const size_t lds = (size_t)p.angles * sizeof(float2);
    if (i8) {
        if (f16) k_append8<true, true, MODE><<<grid, kThreads, lds, s>>>(p);
        else k_append8<false, true, MODE><<<grid, kThreads, lds, s>>>(p);
    } else {
        if (f16) k_append8<true, false, MODE><<<grid, kThreads, lds, s>>>(p);
        else k_append8<false, false, MODE><<<grid, kThreads, lds, s>>>(p);
    }
}

}  // namespace
}  // namespace uzip_kv

extern "C" int uzip_kv_append_scaled(const uzip_kv_cache_t *cache, const uzip_kv_scales_t *scales, const uzip_kv_append_args_t *a,
                                     const uzip_kv_rope_t *rope, hipStream_t s)
{
    using namespace uzip_kv;
    if (!a || a->reserved || !valid_cache(cache, true) || !valid_scales(scales, cache) || !valid_tensor(a->k) || !valid_tensor(a->v)) return UZIP_EINVAL;
    if (a->dtype > UZIP_KV_F16 || !a->length || !aligned(a->length, 4) || !aligned(a->drafted, 4)) return UZIP_EINVAL;
    if (a->tokens < 1 || a->tokens > (1u << 30) || (uint64_t)cache->seqs * a->tokens >= (1ull << 31)) return UZIP_EINVAL;
    if (rope && !valid_rope(rope, cache->dim)) return UZIP_EINVAL;
    if (cache->k == cache->v || scales->k == scales->v) return UZIP_EINVAL;
    Append8Params p;
    memset(&p, 0, sizeof p);
    if (a->q.data || a->q_out.data) {
        if (!valid_tensor(a->q) || !valid_tensor(a->q_out) || a->heads < 1 || a->heads > 65535) return UZIP_EINVAL;
        if (a->q.data == a->q_out.data && !same_tensor(a->q, a->q_out)) return UZIP_EINVAL;
        if (a->q_out.data == a->k.data || a->q_out.data == a->v.data) return UZIP_EINVAL;      // read beside it
        p.q = static_cast<const char *>(a->q.data);
        p.y = static_cast<char *>(a->q_out.data);
        p.qs0 = a->q.stride[0] * 2, p.qs1 = a->q.stride[1] * 2, p.qs2 = a->q.stride[2] * 2;
        p.ys0 = a->q_out.stride[0] * 2, p.ys1 = a->q_out.stride[1] * 2, p.ys2 = a->q_out.stride[2] * 2;
        p.Hq = a->q.data == a->q_out.data ? 0 : (int)a->heads;    // in place: another thread reads an element's partner here
    }
    p.k = static_cast<const char *>(a->k.data);
    p.v = static_cast<const char *>(a->v.data);
    p.ks0 = a->k.stride[0] * 2, p.ks1 = a->k.stride[1] * 2, p.ks2 = a->k.stride[2] * 2;
    p.vs0 = a->v.stride[0] * 2, p.vs1 = a->v.stride[1] * 2, p.vs2 = a->v.stride[2] * 2;
    p.c = view_of(cache);
    p.f = view_of(scales);
    p.length = a->length;
    p.drafted = a->drafted;
    p.T = (int)a->tokens, p.H = (int)cache->heads, p.D = (int)cache->dim;
    if (rope) {
        p.freq = rope->freq, p.pos = rope->pos, p.pos_stride = rope->pos_stride, p.amplitude = rope->amplitude;
        p.rot = (int)rope->rot;
        p.interleaved = (rope->flags & UZIP_KV_INTERLEAVED) != 0, p.inverse = (rope->flags & UZIP_KV_INVERSE) != 0;
    }
    const int64_t unit = 1ll << p.f.shift, T = p.T, most = T < unit ? T : unit;    // new tokens a block, at most
    p.blocks = (int)((T + unit - 2) / unit + 1);
    const int64_t places = (int64_t)cache->seqs * p.blocks;
    // a wave an item where it can hold the block's elements; an item a wave
    p.waves = most * (p.D / 8) <= 64 * kKeep ? 1 : kAppendWaves;
    p.items = p.waves == 1 ? kAppendWaves : 1;
    p.groups = (2 * p.H + p.items - 1) / p.items;
    p.per_magic = (uint32_t)(((1ull << 32) + p.D / 8 - 1) / (p.D / 8));
    int64_t in_lds = most * (p.rot / 2), q_blocks = 0;
    if (p.Hq) {
        // queries: a round of loads or two for each workgroup's threads
        p.q_count = (int64_t)cache->seqs * T;
        const int64_t units = (int64_t)p.Hq * (p.D / 8);
        int64_t tokens = 4 * kThreads / units;
        if (p.rot && tokens > kAngles / (p.rot / 2)) tokens = kAngles / (p.rot / 2);
        if (tokens > p.q_count / (4 * kCUs)) tokens = p.q_count / (4 * kCUs);
        p.q_tokens = (int)(tokens < 1 ? 1 : tokens);
        int64_t parts = 1;
        if (p.q_count < 4 * kCUs) {
            parts = 4 * kCUs / p.q_count;
            const int64_t at_most = (units + kThreads - 1) / kThreads;
            if (parts > at_most) parts = at_most;
        }
        p.q_share = (int)((units * p.q_tokens + parts - 1) / parts);
        p.q_parts = (int)((units * p.q_tokens + p.q_share - 1) / p.q_share);
        q_blocks = (p.q_count + p.q_tokens - 1) / p.q_tokens * p.q_parts;
        if (in_lds < p.q_tokens * (p.rot / 2)) in_lds = p.q_tokens * (p.rot / 2);
    }
    const bool far = in_lds > kAngles;
    p.angles = far ? 0 : (int)in_lds;
    const int64_t kv = places * p.groups;
    if ((uint64_t)(kv + q_blocks) * kThreads >= kLaunchThreads) return UZIP_EINVAL;
    p.kv_grid = (int)kv;
    if (a->q.data && !p.Hq)
        if (const int rc = turn_in_place(a, cache->seqs, cache->dim, rope, s)) return rc;
    const dim3 grid((unsigned)(kv + q_blocks));
    const bool f16 = a->dtype == UZIP_KV_F16, i8 = cache->dtype == UZIP_KV_I8;
    if (!p.rot) launch_append8<kStill>(p, grid, f16, i8, s);
    else if (far) launch_append8<kFar>(p, grid, f16, i8, s);
    else if (!p.interleaved && p.rot % 16 == 0) launch_append8<kHalves>(p, grid, f16, i8, s);
    else launch_append8<kAny>(p, grid, f16, i8, s);
    UZIP_KV_LAUNCH_CHECK("k_append8");
    return UZIP_OK;
}

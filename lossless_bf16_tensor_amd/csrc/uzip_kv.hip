// uzip_kv.hip -- rotary positions, appending to a KV cache and cutting one
// down (gfx950, wave64). The C-ABI is declared in include/uzip_kv.h.
#include "kv_common.h"

namespace uzip_kv {
namespace {

// ------------------------------------------------------------------- rope --
constexpr int kRopeThreads = 256;
constexpr int kRopeUnits = 4;                     // units a thread loads before it computes

struct RopeParams {
    const char *q, *k, *v;
    char *y;
    int64_t qs0, qs1, qs2, ys0, ys1, ys2;         // bytes
    int64_t ks0, ks1, ks2, vs0, vs1, vs2;
    CacheView c;
    const double *freq;
    const int32_t *pos, *length, *drafted;
    int64_t pos_stride;
    float amplitude;
    int T, Hq, H, D, rot;                         // Hq 0: no queries; H 0: no cache
    int interleaved, inverse;
    int per_q, per_copy;                          // units of a rotated and of a copied head
    int units, share;                             // of a token; of a workgroup
    int parts;                                    // workgroups a token
};

// A unit of work: 8 elements of a head, or 8 and the 8 they turn with.
enum { kPair, kInterleaved, kCopy };
struct Unit {
    const char *src;
    char *dst;                                    // null: dropped
    int kind, i;                                  // i: the first pair's number
    int d;                                        // the first element in the head
    bool cached;                                  // dst is a cache row
};

template <int CT>
__device__ inline void store8(char *dst, const float (&y)[8])
{
    if constexpr (CT == kE5M2)
        *reinterpret_cast<u32x2 *>(dst) = u32x2{pack4_e5m2(y[0], y[1], y[2], y[3]), pack4_e5m2(y[4], y[5], y[6], y[7])};
    else
        *reinterpret_cast<u32x4 *>(dst) = u32x4{pack2<CT == kF16>(y[0], y[1]), pack2<CT == kF16>(y[2], y[3]),
                                                pack2<CT == kF16>(y[4], y[5]), pack2<CT == kF16>(y[6], y[7])};
}

template <bool F16>
__device__ inline void unpack8(u32x4 w, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const f32x2 v = unpack2<F16>(w[i]);
        x[2 * i] = v.x, x[2 * i + 1] = v.y;
    }
}

// (head row of) unit u of a token: source, destination, place in the head
__device__ inline Unit unit_at(const RopeParams &p, int u, int b, int t, char *krow, char *vrow)
{
    Unit r;
    int head, in;
    const int nq = p.Hq * p.per_q, nk = p.H * p.per_q;
    bool copy = false;
    if (u < nq) {
        head = u / p.per_q, in = u - head * p.per_q;
        r.src = p.q + b * p.qs0 + t * p.qs1 + head * p.qs2;
        r.dst = p.y + b * p.ys0 + t * p.ys1 + head * p.ys2;
        r.cached = false;
    } else if (u < nq + nk) {
        u -= nq;
        head = u / p.per_q, in = u - head * p.per_q;
        r.src = p.k + b * p.ks0 + t * p.ks1 + head * p.ks2;
        r.dst = krow ? krow + head * p.c.ks2 : nullptr;
        r.cached = true;
    } else {
        u -= nq + nk;
        head = u / p.per_copy, in = u - head * p.per_copy;
        r.src = p.v + b * p.vs0 + t * p.vs1 + head * p.vs2;
        r.dst = vrow ? vrow + head * p.c.vs2 : nullptr;
        r.cached = true;
        copy = true;
    }
    const int pairs = p.rot / 16;
    if (copy || p.rot == 0) r.kind = kCopy, r.d = in * 8;
    else if (p.interleaved) r.kind = in * 8 < p.rot ? kInterleaved : kCopy, r.d = in * 8;
    else if (in < pairs) r.kind = kPair, r.d = in * 8;
    else r.kind = kCopy, r.d = p.rot + (in - pairs) * 8;
    r.i = r.kind == kInterleaved ? r.d / 2 : r.d;
    return r;
}

// Rotates queries and keys and writes keys and values into the cache, one
// launch. A workgroup takes (a part of) one token: the angles of its rot / 2
// pairs are worked out once, in binary64 up to the fraction of a turn (a
// binary32 angle is wrong by 2^-24 of itself: 0.06 rad at position 2^20), and
// serve all its heads. Bound by memory: every element is read and written
// once, in 16-byte pieces; the loads of a thread's first units are on their
// way while the angles are computed.
// LANES: rot is not a whole number of units; elements find their partner
// through LDS instead.
template <bool F16, int CT, bool LANES>
__global__ __launch_bounds__(kRopeThreads) void k_rope(RopeParams p)
{
    constexpr int ces = CT == kE5M2 ? 1 : 2;
    __shared__ float2 cs[128];
    __shared__ uint16_t row[LANES ? kRopeThreads * 8 : 1];
    const int part = (int)(blockIdx.x % p.parts), token = (int)(blockIdx.x / p.parts);
    const int b = token / p.T, t = token - b * p.T;
    const int tid = (int)threadIdx.x;

    char *krow = nullptr, *vrow = nullptr;
    if (p.H) {
        const int64_t slot = (int64_t)p.length[b] + t;
        if (t < clamp_drafted(p.drafted, b, p.T) && slot >= 0 && slot < p.c.tokens) {
            int64_t ko, vo;
            if (locate(p.c, b, (uint32_t)slot, p.c.ks0, p.c.ks1, ko)) {
                locate(p.c, b, (uint32_t)slot, p.c.vs0, p.c.vs1, vo);
                krow = p.c.k + ko;
                vrow = p.c.v + vo;
            }
        }
    }
    const int u0 = part * p.share, u1 = min(u0 + p.share, p.units);

    Unit unit[kRopeUnits];
    u32x4 a[kRopeUnits], o[kRopeUnits];
    const auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < kRopeUnits; i++) {
            const int u = base + i * kRopeThreads + tid;
            unit[i].dst = nullptr;
            if (u >= u1) continue;
            unit[i] = unit_at(p, u, b, t, krow, vrow);
            if (!unit[i].dst) continue;
            a[i] = *reinterpret_cast<const u32x4 *>(unit[i].src + unit[i].d * 2);
            if (unit[i].kind == kPair) o[i] = *reinterpret_cast<const u32x4 *>(unit[i].src + unit[i].d * 2 + p.rot);
        }
    };
    if (!LANES) load(u0);

    if (tid < p.rot / 2) {
        const int64_t pos = p.pos ? p.pos[b * p.pos_stride + t] : p.length[b] + (int64_t)t;
        double turns = (double)pos * p.freq[tid];
        turns -= rint(turns);
        float s, c;
        sincospif((float)(2.0 * turns), &s, &c);
        cs[tid] = make_float2(c * p.amplitude, p.inverse ? -s * p.amplitude : s * p.amplitude);
    }
    __syncthreads();

    if constexpr (LANES) {
        // whole heads a step: per_q units of 8 elements each
        const int rows = kRopeThreads / p.per_q, half = p.rot / 2;
        for (int base = u0; base < u1; base += rows * p.per_q) {
            const int u = base + tid;
            Unit r;
            r.dst = nullptr;
            u32x4 w = {};
            if (tid < rows * p.per_q && u < u1) {
                r = unit_at(p, u, b, t, krow, vrow);
                const int in = tid % p.per_q;
                r.kind = u >= (p.Hq + p.H) * p.per_q ? kCopy : kPair;
                r.d = in * 8;
                if (r.dst) w = *reinterpret_cast<const u32x4 *>(r.src + r.d * 2);
                *reinterpret_cast<u32x4 *>(row + tid * 8) = w;
            }
            __syncthreads();
            if (r.dst) {
                float x[8], y[8];
                unpack8<F16>(w, x);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int d = r.d + e;
                    y[e] = x[e];
                    if (r.kind == kCopy || d >= p.rot) continue;
                    const int i = p.interleaved ? d >> 1 : d < half ? d : d - half;
                    const bool first = p.interleaved ? !(d & 1) : d < half;
                    const int other = p.interleaved ? d ^ 1 : first ? d + half : d - half;
                    const uint16_t z = row[tid * 8 - r.d + other];
                    const float f = F16 ? f16_to_f32(z) : bf16_to_f32(z);
                    y[e] = first ? x[e] * cs[i].x - f * cs[i].y : x[e] * cs[i].x + f * cs[i].y;
                }
                if (r.cached) store8<CT>(r.dst + r.d * ces, y);
                else store8<F16 ? kF16 : kBF16>(r.dst + r.d * 2, y);
            }
            __syncthreads();
        }
        return;
    }

    for (int base = u0;;) {
#pragma unroll
        for (int i = 0; i < kRopeUnits; i++) {
            const Unit &r = unit[i];
            if (!r.dst) continue;
            float x[8], y[8], z[8];
            unpack8<F16>(a[i], x);
            if (r.kind == kPair) {
                float w[8];
                unpack8<F16>(o[i], w);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float2 q = cs[r.i + e];
                    y[e] = x[e] * q.x - w[e] * q.y;
                    z[e] = w[e] * q.x + x[e] * q.y;
                }
            } else if (r.kind == kInterleaved) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 q = cs[r.i + e / 2];
                    y[e] = x[e] * q.x - x[e + 1] * q.y;
                    y[e + 1] = x[e + 1] * q.x + x[e] * q.y;
                }
            } else {
                if (!r.cached || CT != kE5M2) {   // unchanged bits
                    *reinterpret_cast<u32x4 *>(r.dst + r.d * 2) = a[i];
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 8; e++) y[e] = x[e];
            }
            if (r.cached) {
                store8<CT>(r.dst + r.d * ces, y);
                if (r.kind == kPair) store8<CT>(r.dst + (r.d + p.rot / 2) * ces, z);
            } else {
                store8<F16 ? kF16 : kBF16>(r.dst + r.d * 2, y);
                if (r.kind == kPair) store8<F16 ? kF16 : kBF16>(r.dst + (r.d + p.rot / 2) * 2, z);
            }
        }
        base += kRopeUnits * kRopeThreads;
        if (base >= u1) break;
        load(base);
    }
}

bool valid_rope(const uzip_kv_rope_t *r, uint32_t dim)
{
    if (r->reserved || (r->rot & 1) || r->rot > dim || (r->flags & ~(UZIP_KV_INTERLEAVED | UZIP_KV_INVERSE))) return false;
    if (r->rot && (!r->freq || !aligned(r->freq, 8))) return false;
    if (!(fabsf(r->amplitude) < INFINITY) || r->pos_stride < 0) return false;
    return aligned(r->pos, 4);
}

int launch_rope(RopeParams &p, const uzip_kv_rope_t *r, uint32_t seqs, bool f16, int ct, hipStream_t s)
{
    p.freq = r ? r->freq : nullptr;
    p.pos = r ? r->pos : nullptr;
    p.pos_stride = r ? r->pos_stride : 0;
    p.amplitude = r ? r->amplitude : 1.f;
    p.rot = r ? (int)r->rot : 0;
    p.interleaved = r && (r->flags & UZIP_KV_INTERLEAVED);
    p.inverse = r && (r->flags & UZIP_KV_INVERSE);
    const bool lanes = p.interleaved ? p.rot % 8 != 0 : p.rot % 16 != 0;
    p.per_copy = p.D / 8;
    p.per_q = lanes || p.interleaved ? p.D / 8 : p.rot / 16 + (p.D - p.rot) / 8;
    p.units = (p.Hq + p.H) * p.per_q + p.H * p.per_copy;
    // A token's units in one workgroup, so that its angles are worked out
    // once; with few tokens over several, whole heads each.
    const int64_t tokens = (int64_t)seqs * p.T;
    int64_t parts = 1;
    if (tokens < 4 * kCUs) {
        parts = 4 * kCUs / tokens;
        const int64_t most = (p.units + kRopeThreads - 1) / kRopeThreads;
        parts = parts > most ? most : parts;
    }
    if (lanes) {
        const int heads = p.units / p.per_copy;
        const int64_t each = (heads + parts - 1) / parts;
        p.share = (int)(each * p.per_copy);
    } else {
        p.share = (int)((p.units + parts - 1) / parts);
    }
    p.parts = (p.units + p.share - 1) / p.share;
    if (tokens * p.parts >= (1ll << 31)) return UZIP_EINVAL;
    const dim3 grid((unsigned)(tokens * p.parts));
#define UZIP_KV_ROPE(F, C)                                                                    \
    do {                                                                                      \
        if (lanes) k_rope<F, C, true><<<grid, kRopeThreads, 0, s>>>(p);                       \
        else k_rope<F, C, false><<<grid, kRopeThreads, 0, s>>>(p);                            \
    } while (0)
    if (ct == kE5M2 && f16) UZIP_KV_ROPE(true, kE5M2);
    else if (ct == kE5M2) UZIP_KV_ROPE(false, kE5M2);
    else if (f16) UZIP_KV_ROPE(true, kF16);
    else UZIP_KV_ROPE(false, kBF16);
#undef UZIP_KV_ROPE
    UZIP_KV_LAUNCH_CHECK("k_rope");
    return UZIP_OK;
}

bool same_tensor(const uzip_kv_tensor_t &a, const uzip_kv_tensor_t &b)
{
    return a.stride[0] == b.stride[0] && a.stride[1] == b.stride[1] && a.stride[2] == b.stride[2];
}

// ------------------------------------------------------------------ evict --
constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64;
constexpr int kBins = 2048, kCopies = 8;

struct EvictParams {
    CacheView c, o;
    const float *score;
    int64_t sc0, sc1;
    const int32_t *length;
    int32_t *index, *length_out;
    float *score_out;
    int heads, D, keep, sink, recent;
};

// scores in the order of unsigned integers; NaN as -inf, -0 as 0
__device__ inline uint32_t rank_of(float f)
{
    uint32_t u = __float_as_uint(f);
    if (f != f) u = 0xff800000u;
    if (f == 0.f) u = 0;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One workgroup a row of scores: the need-th largest of the tokens that are
// not kept anyway, by three histograms of 11, 11 and 10 bits, then the kept
// tokens in order. Histograms are held in 8 copies, one for every eighth lane:
// attention weights crowd into few bins, and lanes that add to the same word
// wait for each other.
__global__ __launch_bounds__(kSelThreads) void k_evict_select(EvictParams p)
{
    __shared__ uint32_t hist[kBins * kCopies];
    __shared__ uint32_t wsum[kSelWaves][2];
    __shared__ uint32_t found[2];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int h = (int)(blockIdx.x % p.heads), b = (int)(blockIdx.x / p.heads);
    const int n = clamp_length(p.length, b, p.c.tokens);
    const int kept = min(n, p.keep);
    const float *score = p.score + b * p.sc0 + h * p.sc1;
    int32_t *index = p.index + ((int64_t)b * p.heads + h) * p.keep;
    if (h == 0 && tid == 0 && p.length_out) p.length_out[b] = kept;
    for (int j = kept + tid; j < p.keep; j += kSelThreads) index[j] = -1;
    if (n <= p.keep) {
        for (int j = tid; j < n; j += kSelThreads) index[j] = j;
        return;
    }
    const int lo = p.sink, hi = n - p.recent;      // candidates: [lo, hi)
    uint32_t need = (uint32_t)(p.keep - p.sink - p.recent);
    uint32_t prefix = 0;                           // the bits found so far
    if (need == 0) prefix = 0xffffffffu;           // above every rank
    for (int level = 0; level < 3 && need; level++) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bins = level == 2 ? 1024 : 2048;
        for (int i = tid; i < kBins * kCopies; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int i = lo + tid; i < hi; i += kSelThreads) {
            const uint32_t r = rank_of(score[i]);
            const bool in = level == 0 || (level == 1 ? r >> 21 == prefix >> 21 : r >> 10 == prefix >> 10);
            if (in) atomicAdd(&hist[((r >> shift) & (bins - 1)) * kCopies + (lane & (kCopies - 1))], 1u);
        }
        __syncthreads();
        // thread t owns bins 2t and 2t + 1 from the top; prefix sums over them
        uint32_t c0 = 0, c1 = 0;
        const int top = kBins - 1 - 2 * tid;
        for (int k = 0; k < kCopies; k++) c0 += hist[top * kCopies + k], c1 += hist[(top - 1) * kCopies + k];
        uint32_t sum = c0 + c1;
        for (int x = 1; x < 64; x <<= 1) {
            const uint32_t v = __shfl_up(sum, x);
            if (lane >= x) sum += v;
        }
        if (lane == 63) wsum[wave][0] = sum;
        __syncthreads();
        uint32_t before = sum - c0 - c1;
        for (int w = 0; w < wave; w++) before += wsum[w][0];
        if (before < need && need <= before + c0 + c1) {
            const bool second = need > before + c0;
            found[0] = (uint32_t)(second ? top - 1 : top);
            found[1] = need - before - (second ? c0 : 0);
        }
        __syncthreads();
        prefix |= found[0] << shift;
        need = found[1];
        __syncthreads();
    }
    // need: how many of the ranks equal to prefix are kept, the lowest tokens

    const int seg = ((n + kSelWaves - 1) / kSelWaves + 63) & ~63, s0 = wave * seg, s1 = min(s0 + seg, n);
    uint32_t above = 0, equal = 0;
    for (int i = s0 + lane; i < s1; i += 64) {
        const bool free_ = i >= lo && i < hi;
        const uint32_t r = rank_of(score[i]);
        above += !free_ || r > prefix;
        equal += free_ && r == prefix;
    }
    for (int x = 1; x < 64; x <<= 1) above += __shfl_xor(above, x), equal += __shfl_xor(equal, x);
    if (lane == 0) wsum[wave][0] = above, wsum[wave][1] = equal;
    __syncthreads();
    above = equal = 0;
    for (int w = 0; w < wave; w++) above += wsum[w][0], equal += wsum[w][1];
    for (int i0 = s0; i0 < s1; i0 += 64) {
        const int i = i0 + lane;
        const bool free_ = i >= lo && i < hi;
        const uint32_t r = i < s1 ? rank_of(score[i]) : 0;
        const bool over = i < s1 && (!free_ || r > prefix), tie = i < s1 && free_ && r == prefix;
        const uint64_t mo = __builtin_amdgcn_ballot_w64(over), mt = __builtin_amdgcn_ballot_w64(tie);
        const uint64_t below = (1ull << lane) - 1;
        const uint32_t a = above + (uint32_t)__popcll(mo & below), e = equal + (uint32_t)__popcll(mt & below);
        if (over || (tie && e < need)) index[a + min(e, need)] = i;
        above += (uint32_t)__popcll(mo);
        equal += (uint32_t)__popcll(mt);
    }
}

// Copies the kept rows: bound by memory. A thread moves 8 elements of the key
// and of the value of four slots.
template <typename RawT>
__global__ __launch_bounds__(256) void k_evict_gather(EvictParams p)
{
    constexpr int kSlots = 4, es = sizeof(RawT) / 8;
    const int per = p.D / 8, rows = 256 / per;     // rows a step
    const int groups = (p.keep + rows * kSlots - 1) / (rows * kSlots);
    int id = (int)blockIdx.x;
    const int grp = id % groups;
    id /= groups;
    const int h = id % p.heads, b = id / p.heads;
    const int sub = (int)threadIdx.x / per, chunk = (int)threadIdx.x - sub * per;
    if (sub >= rows) return;
    const int64_t row = ((int64_t)b * p.heads + h) * p.keep;
    RawT k[kSlots], v[kSlots];
    int idx[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; i++) {
        const int j = grp * rows * kSlots + i * rows + sub;
        idx[i] = j < p.keep ? p.index[row + j] : -1;
    }
#pragma unroll
    for (int i = 0; i < kSlots; i++) {
        k[i] = RawT{}, v[i] = RawT{};
        int64_t ko, vo;
        if (idx[i] >= 0 && locate(p.c, b, (uint32_t)idx[i], p.c.ks0, p.c.ks1, ko)) {
            locate(p.c, b, (uint32_t)idx[i], p.c.vs0, p.c.vs1, vo);
            k[i] = *reinterpret_cast<const RawT *>(p.c.k + ko + h * p.c.ks2 + chunk * 8 * es);
            v[i] = *reinterpret_cast<const RawT *>(p.c.v + vo + h * p.c.vs2 + chunk * 8 * es);
        }
    }
#pragma unroll
    for (int i = 0; i < kSlots; i++) {
        const int64_t j = grp * rows * kSlots + i * rows + sub;
        if (j >= p.keep) continue;
        *reinterpret_cast<RawT *>(p.o.k + b * p.o.ks0 + j * p.o.ks1 + h * p.o.ks2 + chunk * 8 * es) = k[i];
        *reinterpret_cast<RawT *>(p.o.v + b * p.o.vs0 + j * p.o.vs1 + h * p.o.vs2 + chunk * 8 * es) = v[i];
        if (chunk == 0 && p.score_out) p.score_out[row + j] = idx[i] >= 0 ? p.score[b * p.sc0 + h * p.sc1 + idx[i]] : 0.f;
    }
}

}  // namespace
}  // namespace uzip_kv

extern "C" {

int uzip_kv_rope(const uzip_kv_tensor_t *x, const uzip_kv_tensor_t *y, uint32_t dtype, uint32_t seqs,
                 uint32_t tokens, uint32_t heads, uint32_t dim, const uzip_kv_rope_t *rope, hipStream_t s)
{
    using namespace uzip_kv;
    if (!x || !y || !valid_tensor(*x) || !valid_tensor(*y) || dtype > UZIP_KV_F16) return UZIP_EINVAL;
    if (!valid_dims(seqs, heads, dim) || tokens < 1 || tokens > (1u << 30) || (uint64_t)seqs * tokens >= (1ull << 31)) return UZIP_EINVAL;
    if (!rope || !valid_rope(rope, dim) || (rope->rot && !rope->pos)) return UZIP_EINVAL;
    if (x->data == y->data && !same_tensor(*x, *y)) return UZIP_EINVAL;
    RopeParams p;
    memset(&p, 0, sizeof p);
    p.q = static_cast<const char *>(x->data);
    p.y = static_cast<char *>(y->data);
    p.qs0 = x->stride[0] * 2, p.qs1 = x->stride[1] * 2, p.qs2 = x->stride[2] * 2;
    p.ys0 = y->stride[0] * 2, p.ys1 = y->stride[1] * 2, p.ys2 = y->stride[2] * 2;
    p.T = (int)tokens, p.Hq = (int)heads, p.D = (int)dim;
    return launch_rope(p, rope, seqs, dtype == UZIP_KV_F16, (int)dtype, s);
}

int uzip_kv_append(const uzip_kv_cache_t *cache, const uzip_kv_append_args_t *a, const uzip_kv_rope_t *rope,
                   hipStream_t s)
{
    using namespace uzip_kv;
    if (!a || a->reserved || !valid_cache(cache) || !valid_tensor(a->k) || !valid_tensor(a->v)) return UZIP_EINVAL;
    if (a->dtype > UZIP_KV_F16 || (cache->dtype != UZIP_KV_E5M2 && cache->dtype != a->dtype)) return UZIP_EINVAL;
    if (!a->length || !aligned(a->length, 4) || !aligned(a->drafted, 4)) return UZIP_EINVAL;
    if (a->tokens < 1 || a->tokens > (1u << 30) || (uint64_t)cache->seqs * a->tokens >= (1ull << 31)) return UZIP_EINVAL;
    if (rope && !valid_rope(rope, cache->dim)) return UZIP_EINVAL;
    RopeParams p;
    memset(&p, 0, sizeof p);
    if (a->q.data || a->q_out.data) {
        if (!valid_tensor(a->q) || !valid_tensor(a->q_out) || a->heads < 1 || a->heads > 65535) return UZIP_EINVAL;
        if (a->q.data == a->q_out.data && !same_tensor(a->q, a->q_out)) return UZIP_EINVAL;
        p.q = static_cast<const char *>(a->q.data);
        p.y = static_cast<char *>(a->q_out.data);
        p.qs0 = a->q.stride[0] * 2, p.qs1 = a->q.stride[1] * 2, p.qs2 = a->q.stride[2] * 2;
        p.ys0 = a->q_out.stride[0] * 2, p.ys1 = a->q_out.stride[1] * 2, p.ys2 = a->q_out.stride[2] * 2;
        p.Hq = (int)a->heads;
    }
    p.k = static_cast<const char *>(a->k.data);
    p.v = static_cast<const char *>(a->v.data);
    p.ks0 = a->k.stride[0] * 2, p.ks1 = a->k.stride[1] * 2, p.ks2 = a->k.stride[2] * 2;
    p.vs0 = a->v.stride[0] * 2, p.vs1 = a->v.stride[1] * 2, p.vs2 = a->v.stride[2] * 2;
    p.c = view_of(cache);
    p.length = a->length;
    p.drafted = a->drafted;
    p.T = (int)a->tokens, p.H = (int)cache->heads, p.D = (int)cache->dim;
    return launch_rope(p, rope, cache->seqs, a->dtype == UZIP_KV_F16, (int)cache->dtype, s);
}

uint64_t uzip_kv_evict_workspace_bytes(uint32_t seqs, uint32_t kv_heads, uint32_t cache_tokens)
{
    if (!uzip_kv::valid_dims(seqs, kv_heads, 8) || cache_tokens < 1 || cache_tokens > (1u << 30)) return 0;
    return 256;
}

int uzip_kv_evict(const uzip_kv_cache_t *cache, const uzip_kv_cache_t *out, const uzip_kv_evict_args_t *a,
                  void *d_ws, uint64_t ws_bytes, hipStream_t s)
{
    using namespace uzip_kv;
    if (!a || !valid_cache(cache) || !valid_cache(out) || out->table) return UZIP_EINVAL;
    if (a->score_tokens < 1 || a->score_tokens > cache->tokens) return UZIP_EINVAL;
    if (out->seqs != cache->seqs || out->heads != cache->heads || out->dim != cache->dim || out->dtype != cache->dtype) return UZIP_EINVAL;
    if (a->keep < 1 || out->tokens != a->keep || a->sink > a->keep || a->recent > a->keep - a->sink) return UZIP_EINVAL;
    if (!a->score || !aligned(a->score, 4) || a->score_stride[0] < 0 || a->score_stride[1] < 0) return UZIP_EINVAL;
    if (!a->length || !aligned(a->length, 4) || !a->index || !aligned(a->index, 4)) return UZIP_EINVAL;
    if (!aligned(a->score_out, 4) || !aligned(a->length_out, 4) || !d_ws || !aligned(d_ws, 16)) return UZIP_EINVAL;
    if (cache->k == out->k || cache->v == out->v) return UZIP_EINVAL;
    if (ws_bytes < uzip_kv_evict_workspace_bytes(cache->seqs, cache->heads, cache->tokens)) return UZIP_ENOSPC;
    EvictParams p;
    memset(&p, 0, sizeof p);
    p.c = view_of(cache);
    p.c.tokens = a->score_tokens;
    p.o = view_of(out);
    p.score = a->score;
    p.sc0 = a->score_stride[0], p.sc1 = a->score_stride[1];
    p.length = a->length;
    p.index = a->index;
    p.length_out = a->length_out;
    p.score_out = a->score_out;
    p.heads = (int)cache->heads, p.D = (int)cache->dim;
    p.keep = (int)a->keep, p.sink = (int)a->sink, p.recent = (int)a->recent;
    const uint64_t rows = (uint64_t)cache->seqs * cache->heads;
    const int each = 256 / (p.D / 8) * 4;
    const uint64_t grid = rows * ((a->keep + each - 1) / each);
    if (rows >= (1ull << 31) || grid >= (1ull << 31)) return UZIP_EINVAL;
    k_evict_select<<<(unsigned)rows, kSelThreads, 0, s>>>(p);
    UZIP_KV_LAUNCH_CHECK("k_evict_select");
    if (cache->dtype == UZIP_KV_E5M2) k_evict_gather<u32x2><<<(unsigned)grid, 256, 0, s>>>(p);
    else k_evict_gather<u32x4><<<(unsigned)grid, 256, 0, s>>>(p);
    UZIP_KV_LAUNCH_CHECK("k_evict_gather");
    return UZIP_OK;
}

}  // extern "C"

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
    int parts, tokens;                            // workgroups a token, or tokens a workgroup
    int64_t count;                                // tokens of all sequences
};

// A unit of work: 8 elements of a head, or 8 and the 8 they turn with.
enum { kPair, kInterleaved, kCopy };
struct Unit {
    const char *src;
    int64_t off;                                  // of the head from its token's place in `to`
    int kind, i;                                  // i: the first pair's number
    int d;                                        // the first element in the head
    int to, token;                                // to: 0 queries, 1 keys, 2 values, -1 nothing; token of the workgroup
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

// unit u of a workgroup's tokens, the first of them number `first` of all
__device__ inline Unit unit_at(const RopeParams &p, int u, int64_t first)
{
    Unit r;
    r.token = 0;
    if (p.tokens > 1) r.token = u / p.units, u -= r.token * p.units;
    const int64_t id = first + r.token;
    const int64_t b = id / p.T, t = id - b * p.T;
    int head, in;
    const int nq = p.Hq * p.per_q, nk = p.H * p.per_q;
    if (u < nq) {
        head = u / p.per_q, in = u - head * p.per_q;
        r.src = p.q + b * p.qs0 + t * p.qs1 + head * p.qs2;
        r.off = b * p.ys0 + t * p.ys1 + head * p.ys2;
        r.to = 0;
    } else if (u < nq + nk) {
        u -= nq;
        head = u / p.per_q, in = u - head * p.per_q;
        r.src = p.k + b * p.ks0 + t * p.ks1 + head * p.ks2;
        r.off = head * p.c.ks2;
        r.to = 1;
    } else {
        u -= nq + nk;
        head = u / p.per_copy, in = u - head * p.per_copy;
        r.src = p.v + b * p.vs0 + t * p.vs1 + head * p.vs2;
        r.off = head * p.c.vs2;
        r.to = 2;
    }
    const int pairs = p.rot / 16;
    if (r.to == 2 || p.rot == 0) r.kind = kCopy, r.d = in * 8;
    else if (p.interleaved) r.kind = in * 8 < p.rot ? kInterleaved : kCopy, r.d = in * 8;
    else if (in < pairs) r.kind = kPair, r.d = in * 8;
    else r.kind = kCopy, r.d = p.rot + (in - pairs) * 8;
    r.i = r.kind == kInterleaved ? r.d / 2 : r.d;
    return r;
}

// Rotates queries and keys and writes keys and values into the cache, one
// launch. A workgroup takes some tokens, as many as give its threads work (8 x
// 3068 tokens of one head of 128: 11 us, with one token a workgroup 60), or a
// part of one when there are few: the angles of a token's rot / 2 pairs are worked out
// once, in binary64 up to the fraction of a turn (a binary32 angle is wrong by
// 2^-24 of itself: 0.06 rad at position 2^20), and serve all its heads. Bound
// by memory: every element is read and written once, in 16-byte pieces; the
// loads of a thread's first units are on their way while the angles are
// computed. Queries of 2 x 16384 tokens of 64 heads of 128: 206 us, 5.2 TB/s,
// which is the rate of a large copy.
// LANES: rot is not a whole number of units; elements find their partner
// through LDS instead.
constexpr int kRopeTokens = 32, kRopeAngles = 1024;       // of a workgroup, at most
template <bool F16, int CT, bool LANES>
__global__ __launch_bounds__(kRopeThreads) void k_rope(RopeParams p)
{
    constexpr int ces = CT == kE5M2 ? 1 : 2;
    __shared__ float2 cs[kRopeAngles];
    __shared__ char *place[kRopeTokens][2];       // of a token's keys and values in the cache, null where dropped
    __shared__ uint16_t row[LANES ? kRopeThreads * 8 : 1];
    const int part = (int)(blockIdx.x % p.parts);
    const int64_t first = (int64_t)(blockIdx.x / p.parts) * p.tokens;
    const int tokens = (int)min((int64_t)p.tokens, p.count - first), half = p.rot / 2;
    const int tid = (int)threadIdx.x;
    const int u0 = part * p.share, u1 = min(u0 + p.share, p.units * tokens);

    Unit unit[kRopeUnits];
    u32x4 a[kRopeUnits], o[kRopeUnits];
    const auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < kRopeUnits; i++) {
            const int u = base + i * kRopeThreads + tid;
            unit[i].to = -1;
            if (u >= u1) continue;
            unit[i] = unit_at(p, u, first);
            a[i] = *reinterpret_cast<const u32x4 *>(unit[i].src + unit[i].d * 2);
            if (unit[i].kind == kPair) o[i] = *reinterpret_cast<const u32x4 *>(unit[i].src + unit[i].d * 2 + p.rot);
        }
    };
    if (!LANES) load(u0);

    for (int j = tid; j < tokens * half; j += kRopeThreads) {
        const int token = j / half, i = j - token * half;
        const int64_t id = first + token, b = id / p.T, t = id - b * p.T;
        const int64_t pos = p.pos ? p.pos[b * p.pos_stride + t] : p.length[b] + t;
        double turns = (double)pos * p.freq[i];
        turns -= rint(turns);
        float s, c;
        sincospif((float)(2.0 * turns), &s, &c);
        cs[j] = make_float2(c * p.amplitude, p.inverse ? -s * p.amplitude : s * p.amplitude);
    }
    if (p.H && tid < tokens) {
        const int64_t id = first + tid;
        const int b = (int)(id / p.T), t = (int)(id - (int64_t)b * p.T);
        const int64_t slot = (int64_t)p.length[b] + t;
        char *k = nullptr, *v = nullptr;
        if (t < clamp_drafted(p.drafted, b, p.T) && slot >= 0 && slot < p.c.tokens) {
            int64_t ko, vo;
            if (locate(p.c, b, (uint32_t)slot, p.c.ks0, p.c.ks1, ko)) {
                locate(p.c, b, (uint32_t)slot, p.c.vs0, p.c.vs1, vo);
                k = p.c.k + ko;
                v = p.c.v + vo;
            }
        }
        place[tid][0] = k, place[tid][1] = v;
    }
    __syncthreads();
    const auto where = [&](const Unit &r) {
        if (r.to < 0) return (char *)nullptr;
        char *at = r.to == 0 ? p.y : place[r.token][r.to - 1];
        return at ? at + r.off : at;
    };

    if constexpr (LANES) {
        // whole heads a step: per_q units of 8 elements each
        const int rows = kRopeThreads / p.per_q;
        for (int base = u0; base < u1; base += rows * p.per_q) {
            const int u = base + tid;
            Unit r;
            r.to = -1;
            u32x4 w = {};
            if (tid < rows * p.per_q && u < u1) {
                r = unit_at(p, u, first);
                r.d = u % p.per_q * 8;
                w = *reinterpret_cast<const u32x4 *>(r.src + r.d * 2);
                *reinterpret_cast<u32x4 *>(row + tid * 8) = w;
            }
            __syncthreads();
            if (char *dst = where(r)) {
                const float2 *angle = cs + r.token * half;
                float x[8], y[8];
                unpack8<F16>(w, x);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int d = r.d + e;
                    y[e] = x[e];
                    if (r.to == 2 || d >= p.rot) continue;
                    const int i = p.interleaved ? d >> 1 : d < half ? d : d - half;
                    const bool lead = p.interleaved ? !(d & 1) : d < half;
                    const int other = p.interleaved ? d ^ 1 : lead ? d + half : d - half;
                    const uint16_t z = row[tid * 8 - r.d + other];
                    const float f = F16 ? f16_to_f32(z) : bf16_to_f32(z);
                    y[e] = lead ? x[e] * angle[i].x - f * angle[i].y : x[e] * angle[i].x + f * angle[i].y;
                }
                const int keep = r.to == 2 ? 0 : max(0, min(p.rot - r.d, 8));   // elements from here on keep their bits
                if (r.to && CT == kE5M2) {
                    store8<CT>(dst + r.d * ces, y);
                } else {
                    u32x4 z;
#pragma unroll
                    for (int e = 0; e < 4; e++)    // rot is even
                        z[e] = 2 * e < keep ? pack2<F16>(y[2 * e], y[2 * e + 1]) : w[e];
                    *reinterpret_cast<u32x4 *>(dst + r.d * 2) = z;
                }
            }
            __syncthreads();
        }
        return;
    }

    for (int base = u0;;) {
#pragma unroll
        for (int i = 0; i < kRopeUnits; i++) {
            const Unit &r = unit[i];
            char *dst = where(r);
            if (!dst) continue;
            const float2 *angle = cs + r.token * half + r.i;
            float x[8], y[8], z[8];
            unpack8<F16>(a[i], x);
            if (r.kind == kPair) {
                float w[8];
                unpack8<F16>(o[i], w);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float2 q = angle[e];
                    y[e] = x[e] * q.x - w[e] * q.y;
                    z[e] = w[e] * q.x + x[e] * q.y;
                }
            } else if (r.kind == kInterleaved) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 q = angle[e / 2];
                    y[e] = x[e] * q.x - x[e + 1] * q.y;
                    y[e + 1] = x[e + 1] * q.x + x[e] * q.y;
                }
            } else {
                if (!r.to || CT != kE5M2) {       // unchanged bits
                    *reinterpret_cast<u32x4 *>(dst + r.d * 2) = a[i];
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 8; e++) y[e] = x[e];
            }
            if (r.to) {
                store8<CT>(dst + r.d * ces, y);
                if (r.kind == kPair) store8<CT>(dst + (r.d + half) * ces, z);
            } else {
                store8<F16 ? kF16 : kBF16>(dst + r.d * 2, y);
                if (r.kind == kPair) store8<F16 ? kF16 : kBF16>(dst + (r.d + half) * 2, z);
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
    // A workgroup's units are a round of loads or two of its threads: of
    // several tokens, as their angles and places fit; of a part of one (whole
    // heads) when there are few tokens.
    p.count = (int64_t)seqs * p.T;
    int64_t tokens = kRopeUnits * kRopeThreads / p.units;
    if (p.rot && tokens > kRopeAngles / (p.rot / 2)) tokens = kRopeAngles / (p.rot / 2);
    if (tokens > kRopeTokens) tokens = kRopeTokens;
    if (tokens > p.count / (4 * kCUs)) tokens = p.count / (4 * kCUs);
    p.tokens = (int)(tokens < 1 ? 1 : tokens);
    int64_t parts = 1;
    if (p.count < 4 * kCUs) {
        parts = 4 * kCUs / p.count;
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
    if (p.tokens > 1) p.parts = 1, p.share = p.units * p.tokens;
    const int64_t blocks = (p.count + p.tokens - 1) / p.tokens * p.parts;
    if (blocks >= (1ll << 31)) return UZIP_EINVAL;
    const dim3 grid((unsigned)blocks);
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
// The kept tokens of a row of scores are the first and last ones and the
// need-th largest of the others and all above it. Scores become unsigned ranks
// in the same order; the need-th largest rank is found by histograms of its
// upper 11 bits, the next 11 and the last 10, each of the ranks that agree with
// the bits found so far. Histograms in LDS are held in 4 copies, one for every
// fourth lane: attention weights crowd into few bins, and lanes that add to the
// same word wait for each other; clearing and adding up more copies costs short
// rows more than it saves (16 rows of 4096: 12 us, with 8 copies 13; 128 equal
// rows of 16384 104 and 101).
constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64;
constexpr int kBins = 2048, kCopies = 4;
constexpr int kOneTokens = 32 * kSelThreads;      // rows up to here are held in one workgroup's registers
constexpr int kSlice = 8 * kSelThreads;           // tokens a workgroup takes of a longer row
constexpr uint32_t kForced = 0xffffffffu, kOutside = 0;      // ranks of no score

struct EvictParams {
    CacheView c, o;
    const float *score;
    int64_t sc0, sc1;
    const int32_t *length;
    int32_t *index, *length_out;
    float *score_out;
    int heads, D, keep, sink, recent;
    int parts, share;                             // workgroups a row, slots each, where k_evict_one copies
    // long rows: per row, slices' histograms of one level [3][slices][kBins],
    // their numbers of kept tokens by level [2][slices], and what is found
    uint16_t *hist;
    uint32_t *count;
    uint2 *found;                                 // [row][2]: rank bits, how many are still needed
    int slices;
};

// Scores in the order of unsigned integers; NaN as -inf, -0 as 0. Tokens that
// are kept anyway rank above all, those outside the cache below.
__device__ inline uint32_t rank_of(const EvictParams &p, float f, int i, int n)
{
    if (i >= n) return kOutside;
    if (i < p.sink || i >= n - p.recent) return kForced;
    uint32_t u = __float_as_uint(f);
    if (f != f) u = 0xff800000u;
    if (f == 0.f) u = 0;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ inline int level_shift(int level) { return level == 0 ? 21 : level == 1 ? 10 : 0; }

// whether a rank is a score's and agrees with the bits found before this level
__device__ inline bool agrees(uint32_t r, uint32_t prefix, int level)
{
    if (r == kForced || r == kOutside) return false;
    return level == 0 || (level == 1 ? r >> 21 == prefix >> 21 : r >> 10 == prefix >> 10);
}

__device__ inline void add_to_hist(uint32_t *hist, uint32_t r, int level)
{
    atomicAdd(&hist[(r >> level_shift(level) & (level == 2 ? 1023 : 2047)) * kCopies + (threadIdx.x & (kCopies - 1))], 1u);
}

// Of bins counted from the top, two a thread (c0 in bin 2047 - 2 tid, c1 in the
// next lower one): the bin that holds the need-th, and how many of it are
// needed. out: {bin, needed}. wsum: one word a wave. Ends with a barrier.
__device__ inline void find_bin(uint32_t c0, uint32_t c1, uint32_t need, uint32_t *wsum, uint32_t *out)
{
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t sum = c0 + c1;
    for (int x = 1; x < 64; x <<= 1) {
        const uint32_t v = __shfl_up(sum, x);
        if (lane >= x) sum += v;
    }
    if (lane == 63) wsum[wave] = sum;
    __syncthreads();
    uint32_t before = sum - c0 - c1;
#pragma unroll
    for (int w = 0; w < kSelWaves; w += 4) {      // all waves' sums at once
        const u32x4 v = *reinterpret_cast<const u32x4 *>(wsum + w);
#pragma unroll
        for (int i = 0; i < 4; i++) before += w + i < wave ? v[i] : 0;
    }
    if (before < need && need <= before + c0 + c1) {
        const bool second = need > before + c0;
        out[0] = (uint32_t)(kBins - 1 - 2 * tid - second);
        out[1] = need - before - (second ? c0 : 0);
    }
    __syncthreads();
}

__device__ inline void fill_behind(const EvictParams &p, int32_t *index, int kept, int part, int parts)
{
    for (int j = kept + part * kSelThreads + (int)threadIdx.x; j < p.keep; j += parts * kSelThreads) index[j] = -1;
}

// Kept rows [j0, j1) of a sequence and head, to out in order: bound by memory.
// slot(j) is the token of slot j, -1 for none.
template <typename RawT, int SLOTS, typename Slot>
__device__ inline void copy_rows(const EvictParams &p, int b, int h, int j0, int j1, int threads, Slot slot)
{
    constexpr int es = sizeof(RawT) / 8;
    const int per = p.D / 8, rows = threads / per;           // 8-element pieces a row, rows a step
    const int sub = (int)threadIdx.x / per, piece = (int)threadIdx.x - sub * per;
    if (sub >= rows) return;
    const int64_t row = ((int64_t)b * p.heads + h) * p.keep;
    for (int base = j0 + sub; base < j1; base += rows * SLOTS) {
        RawT k[SLOTS], v[SLOTS];
        int idx[SLOTS];
#pragma unroll
        for (int i = 0; i < SLOTS; i++) idx[i] = base + i * rows < j1 ? slot(base + i * rows) : -1;
#pragma unroll
        for (int i = 0; i < SLOTS; i++) {
            k[i] = RawT{}, v[i] = RawT{};
            int64_t ko, vo;
            if (idx[i] >= 0 && locate(p.c, b, (uint32_t)idx[i], p.c.ks0, p.c.ks1, ko)) {
                locate(p.c, b, (uint32_t)idx[i], p.c.vs0, p.c.vs1, vo);
                k[i] = *reinterpret_cast<const RawT *>(p.c.k + ko + h * p.c.ks2 + piece * 8 * es);
                v[i] = *reinterpret_cast<const RawT *>(p.c.v + vo + h * p.c.vs2 + piece * 8 * es);
            }
        }
#pragma unroll
        for (int i = 0; i < SLOTS; i++) {
            const int64_t j = base + i * rows;
            if (j >= j1) continue;
            *reinterpret_cast<RawT *>(p.o.k + b * p.o.ks0 + j * p.o.ks1 + h * p.o.ks2 + piece * 8 * es) = k[i];
            *reinterpret_cast<RawT *>(p.o.v + b * p.o.vs0 + j * p.o.vs1 + h * p.o.vs2 + piece * 8 * es) = v[i];
            if (piece == 0 && p.score_out) p.score_out[row + j] = idx[i] >= 0 ? p.score[b * p.sc0 + h * p.sc1 + idx[i]] : 0.f;
        }
    }
}

// Rows of up to N * 1024 tokens, held in a workgroup's registers. COPY (rows
// and cuts up to 4096): each of a row's workgroups finds the kept tokens for
// itself and copies its share of them; a second launch would cost more than
// choosing again (8 rows of 4096, 1024 of 128 16-bit elements kept: 11 us, in
// two launches 17; 256 rows 45 and 55). Without, one workgroup a row writes the
// index, and k_evict_copy copies. Choosing is bound by the steps of its three
// levels, 22 us for 128 rows of 16384, where the copy of 4096 of each takes 104.
template <int N, bool COPY, typename RawT>
__global__ __launch_bounds__(kSelThreads) void k_evict_one(EvictParams p)
{
    __shared__ __attribute__((aligned(16))) uint32_t hist[kBins * kCopies];    // later the tokens of this workgroup's slots
    __shared__ uint32_t counts[N * kSelWaves];    // kept tokens before each wave's 64 of each round: above << 16 | equal
    __shared__ __attribute__((aligned(16))) uint32_t wsum[kSelWaves];
    __shared__ uint32_t out[2];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int part = (int)(blockIdx.x % p.parts), row = (int)(blockIdx.x / p.parts);
    const int h = row % p.heads, b = row / p.heads;
    const int n = clamp_length(p.length, b, p.c.tokens), kept = min(n, p.keep);
    const float *score = p.score + b * p.sc0 + h * p.sc1;
    int32_t *index = p.index + (int64_t)row * p.keep;
    const int j0 = part * p.share, j1 = min(j0 + p.share, p.keep);
    if (h == 0 && part == 0 && tid == 0 && p.length_out) p.length_out[b] = kept;
    fill_behind(p, index, kept, part, p.parts);
    if (n <= p.keep) {
        for (int j = j0 + tid; j < min(j1, n); j += kSelThreads) index[j] = j;
        if constexpr (COPY) copy_rows<RawT, 4>(p, b, h, j0, j1, kSelThreads, [&](int j) { return j < n ? j : -1; });
        return;
    }
    uint32_t r[N];
#pragma unroll
    for (int k = 0; k < N; k++) {
        const int i = k * kSelThreads + tid;
        r[k] = rank_of(p, i < n ? score[i] : 0.f, i, n);
    }
    uint32_t need = (uint32_t)(p.keep - p.sink - p.recent), prefix = need ? 0 : kForced - 1;
    for (int level = 0; level < 3 && need; level++) {
        for (int i = tid; i < kBins * kCopies / 4; i += kSelThreads) reinterpret_cast<u32x4 *>(hist)[i] = u32x4{0, 0, 0, 0};
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; k++)
            if (agrees(r[k], prefix, level)) add_to_hist(hist, r[k], level);
        __syncthreads();
        uint32_t c[2] = {0, 0};
        const u32x4 *bin = reinterpret_cast<const u32x4 *>(hist) + (kBins - 2 - 2 * tid) * (kCopies / 4);
#pragma unroll
        for (int i = 0; i < 2 * kCopies / 4; i++) c[i < kCopies / 4] += bin[i].x + bin[i].y + bin[i].z + bin[i].w;
        find_bin(c[0], c[1], need, wsum, out);
        prefix |= out[0] << level_shift(level);
        need = out[1];
        __syncthreads();
    }
    // need: how many of the ranks equal to prefix are kept, the lowest tokens.
    // A round's 64 tokens of a wave, rounds before waves, are in order.
#pragma unroll
    for (int k = 0; k < N; k++) {
        const uint32_t above = (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(r[k] > prefix)), equal = (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(r[k] == prefix));
        if (lane == 0) counts[k * kSelWaves + wave] = above << 16 | equal;
    }
    __syncthreads();
    if (wave == 0) {                              // prefix sums; halves stay below 2^16: 32768 tokens
        constexpr int each = (N * kSelWaves + 63) / 64;
        uint32_t c[each], sum = 0;
#pragma unroll
        for (int i = 0; i < each; i++) {
            c[i] = lane * each + i < N * kSelWaves ? counts[lane * each + i] : 0;
            sum += c[i];
        }
        uint32_t before = sum;
        for (int x = 1; x < 64; x <<= 1) {
            const uint32_t v = __shfl_up(before, x);
            if (lane >= x) before += v;
        }
        before -= sum;
#pragma unroll
        for (int i = 0; i < each; i++) {
            if (lane * each + i < N * kSelWaves) counts[lane * each + i] = before;
            before += c[i];
        }
    }
    __syncthreads();
    int *slots = reinterpret_cast<int *>(hist);
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll
    for (int k = 0; k < N; k++) {
        const uint32_t before = counts[k * kSelWaves + wave];
        const bool over = r[k] > prefix, tie = r[k] == prefix;
        const uint32_t a = (before >> 16) + (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(over) & below);
        const uint32_t e = (before & 0xffffu) + (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(tie) & below);
        const int at = (int)(a + min(e, need));
        if (!over && !(tie && e < need)) continue;
        if constexpr (COPY) {
            if (at >= j0 && at < j1) slots[at - j0] = k * kSelThreads + tid;
        } else {
            index[at] = k * kSelThreads + tid;
        }
    }
    if constexpr (COPY) {
        __syncthreads();
        for (int j = j0 + tid; j < j1; j += kSelThreads) index[j] = slots[j - j0];  // n > keep: every slot has a token
        copy_rows<RawT, 4>(p, b, h, j0, j1, kSelThreads, [&](int j) { return slots[j - j0]; });
    }
}

// Longer rows, by slices: a launch a level, each of whose workgroups adds up
// the slices' histograms of the level before, and one that writes the kept
// tokens. Nothing needs clearing and no sum depends on an order. Bound by the
// launches, which wait for each other: 16 rows of 120000 take 35 us to choose,
// and 28 for the copy of 12345 FP8 rows of 128 of each. Rows up to 32768 stay in registers: 128
// of them 122 us with their copy, by slices 128; only with few rows is it the
// other way (16 rows: 43 and 40). What decides is how many scores a row can
// hold, as the lengths are on the device: 128 rows of 2000 tokens take 20 us
// where it holds 2048, 29 at 32768 and 101 at 131072.
struct Slice {
    int row, slice, b, h, n, i0;
    const float *score;

    __device__ inline Slice(const EvictParams &p)
    {
        slice = (int)(blockIdx.x % p.slices), row = (int)(blockIdx.x / p.slices);
        h = row % p.heads, b = row / p.heads;
        n = clamp_length(p.length, b, p.c.tokens);
        i0 = slice * kSlice;
        score = p.score + b * p.sc0 + h * p.sc1;
    }

    __device__ inline void load(const EvictParams &p, uint32_t (&r)[kSlice / kSelThreads]) const
    {
#pragma unroll
        for (int k = 0; k < kSlice / kSelThreads; k++) {
            const int i = i0 + k * kSelThreads + (int)threadIdx.x;
            r[k] = rank_of(p, i < n ? score[i] : 0.f, i, n);
        }
    }

    // a level's histograms, of this row; a thread's two bins of one are one word
    __device__ inline const uint32_t *hist(const EvictParams &p, int level) const
    {
        return reinterpret_cast<const uint32_t *>(p.hist + ((int64_t)row * 3 + level) * p.slices * kBins) + (kBins / 2 - 1 - (int)threadIdx.x);
    }
};

__device__ inline uint32_t slices_used(int n) { return (uint32_t)((n + kSlice - 1) / kSlice); }

// adds up a level's histograms over the slices below `to`
__device__ inline void sum_hist(const uint32_t *h, uint32_t from, uint32_t to, uint32_t &c0, uint32_t &c1)
{
    for (uint32_t s = from; s < to; s += 8) {     // eight loads at a time: they come from other XCDs' writes
        uint32_t w[8];
#pragma unroll
        for (uint32_t i = 0; i < 8; i++) w[i] = s + i < to ? h[(s + i) * (kBins / 2)] : 0;
#pragma unroll
        for (uint32_t i = 0; i < 8; i++) c0 += w[i] >> 16, c1 += w[i] & 0xffffu;
    }
}

template <int LEVEL>
__global__ __launch_bounds__(kSelThreads) void k_evict_level(EvictParams p)
{
    __shared__ __attribute__((aligned(16))) uint32_t hist[kBins * kCopies];
    __shared__ __attribute__((aligned(16))) uint32_t wsum[kSelWaves];
    __shared__ uint32_t out[2], total;
    const Slice s(p);
    const int tid = (int)threadIdx.x;
    const uint32_t first_need = (uint32_t)(p.keep - p.sink - p.recent);
    if (s.n <= p.keep || s.i0 >= s.n || first_need == 0) return;       // nothing to choose
    uint32_t r[kSlice / kSelThreads];
    s.load(p, r);
    for (int i = tid; i < kBins * kCopies / 4; i += kSelThreads) reinterpret_cast<u32x4 *>(hist)[i] = u32x4{0, 0, 0, 0};
    if (tid == 0) total = 0;
    uint32_t prefix = 0;
    if constexpr (LEVEL > 0) {
        uint2 before = make_uint2(0, first_need);
        if constexpr (LEVEL == 2) before = p.found[s.row * 2];
        uint32_t c0 = 0, c1 = 0;
        sum_hist(s.hist(p, LEVEL - 1), 0, slices_used(s.n), c0, c1);
        find_bin(c0, c1, before.y, wsum, out);
        prefix = before.x | out[0] << level_shift(LEVEL - 1);
        if (s.slice == 0 && tid == 0) p.found[s.row * 2 + LEVEL - 1] = make_uint2(prefix, out[1]);
        // this slice's tokens that are kept for this level's bits
        uint32_t mine = 0;
#pragma unroll
        for (int k = 0; k < kSlice / kSelThreads; k++) {
            if (LEVEL == 1 && r[k] == kForced) mine++;
            else if (agrees(r[k], prefix, LEVEL - 1) && (r[k] >> level_shift(LEVEL - 1)) > (prefix >> level_shift(LEVEL - 1))) mine++;
        }
        for (int x = 1; x < 64; x <<= 1) mine += __shfl_xor(mine, x);
        if ((tid & 63) == 0 && mine) atomicAdd(&total, mine);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSlice / kSelThreads; k++)
        if (agrees(r[k], prefix, LEVEL)) add_to_hist(hist, r[k], LEVEL);
    __syncthreads();
    uint32_t c[2] = {0, 0};
    const u32x4 *bin = reinterpret_cast<const u32x4 *>(hist) + (kBins - 2 - 2 * tid) * (kCopies / 4);
#pragma unroll
    for (int i = 0; i < 2 * kCopies / 4; i++) c[i < kCopies / 4] += bin[i].x + bin[i].y + bin[i].z + bin[i].w;
    const_cast<uint32_t *>(s.hist(p, LEVEL))[s.slice * (kBins / 2)] = c[0] << 16 | c[1];      // at most 8192 each
    if (LEVEL > 0 && tid == 0) p.count[((int64_t)s.row * 2 + LEVEL - 1) * p.slices + s.slice] = total;
}

__global__ __launch_bounds__(kSelThreads) void k_evict_index(EvictParams p)
{
    __shared__ __attribute__((aligned(16))) uint32_t wsum[kSelWaves];
    __shared__ uint32_t counts[kSlice / kSelThreads * kSelWaves], out[2], sums[2];
    const Slice s(p);
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int kept = min(s.n, p.keep);
    int32_t *index = p.index + (int64_t)s.row * p.keep;
    if (s.h == 0 && s.slice == 0 && tid == 0 && p.length_out) p.length_out[s.b] = kept;
    fill_behind(p, index, kept, s.slice, p.slices);
    if (s.i0 >= s.n) return;
    if (s.n <= p.keep) {
        for (int i = s.i0 + tid; i < min(s.i0 + kSlice, s.n); i += kSelThreads) index[i] = i;
        return;
    }
    uint32_t r[kSlice / kSelThreads];
    s.load(p, r);
    uint32_t need = (uint32_t)(p.keep - p.sink - p.recent), prefix = kForced - 1;
    uint32_t above0 = 0, equal0 = 0;              // kept in earlier slices: for sure, and by tokens of the last rank
    if (need) {
        const uint2 before = p.found[s.row * 2 + 1];
        uint32_t p0 = 0, p1 = 0, c0, c1;
        const uint32_t *h = s.hist(p, 2);
        sum_hist(h, 0, (uint32_t)s.slice, p0, p1);
        c0 = p0, c1 = p1;
        sum_hist(h, (uint32_t)s.slice, slices_used(s.n), c0, c1);
        if (tid < 2) sums[tid] = 0;
        find_bin(c0, c1, before.y, wsum, out);
        prefix = before.x | out[0];
        need = out[1];
        const uint32_t bin = (uint32_t)(kBins - 1 - 2 * tid);
        uint32_t more = (bin > out[0] ? p0 : 0) + (bin - 1 > out[0] ? p1 : 0);
        for (int i = tid; i < s.slice; i += kSelThreads)
            more += p.count[(int64_t)s.row * 2 * p.slices + i] + p.count[((int64_t)s.row * 2 + 1) * p.slices + i];
        for (int x = 1; x < 64; x <<= 1) more += __shfl_xor(more, x);
        if (lane == 0 && more) atomicAdd(&sums[0], more);
        if (bin == out[0]) sums[1] = p0;
        if (bin - 1 == out[0]) sums[1] = p1;
        __syncthreads();
        above0 = sums[0], equal0 = sums[1];
    } else {
        above0 = (uint32_t)(min(s.i0, p.sink) + max(0, s.i0 - (s.n - p.recent)));      // the first and last tokens alone
    }
#pragma unroll
    for (int k = 0; k < kSlice / kSelThreads; k++) {
        const uint32_t above = (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(r[k] > prefix)), equal = (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(r[k] == prefix));
        if (lane == 0) counts[k * kSelWaves + wave] = above << 16 | equal;
    }
    __syncthreads();
    if (wave == 0) {
        constexpr int each = kSlice / kSelThreads * kSelWaves / 64;
        uint32_t c[each], sum = 0;
#pragma unroll
        for (int i = 0; i < each; i++) sum += c[i] = counts[lane * each + i];
        uint32_t before = sum;
        for (int x = 1; x < 64; x <<= 1) {
            const uint32_t v = __shfl_up(before, x);
            if (lane >= x) before += v;
        }
        before -= sum;
#pragma unroll
        for (int i = 0; i < each; i++) {
            counts[lane * each + i] = before;
            before += c[i];
        }
    }
    __syncthreads();
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll
    for (int k = 0; k < kSlice / kSelThreads; k++) {
        const uint32_t before = counts[k * kSelWaves + wave];
        const bool over = r[k] > prefix, tie = r[k] == prefix;
        const uint32_t a = above0 + (before >> 16) + (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(over) & below);
        const uint32_t e = equal0 + (before & 0xffffu) + (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(tie) & below);
        if (over || (tie && e < need)) index[a + min(e, need)] = s.i0 + k * kSelThreads + tid;
    }
}

template <typename RawT>
__global__ __launch_bounds__(256) void k_evict_copy(EvictParams p)
{
    const int each = 256 / (p.D / 8) * 4, groups = (p.keep + each - 1) / each;
    const int grp = (int)(blockIdx.x % groups), row = (int)(blockIdx.x / groups);
    const int32_t *index = p.index + (int64_t)row * p.keep;
    copy_rows<RawT, 4>(p, row / p.heads, row % p.heads, grp * each, min(grp * each + each, p.keep), 256, [&](int j) { return index[j]; });
}

template <typename RawT>
int launch_copy(const EvictParams &p, uint64_t rows, hipStream_t s)
{
    const int each = 256 / (p.D / 8) * 4;
    const uint64_t grid = rows * ((p.keep + each - 1) / each);
    k_evict_copy<RawT><<<(unsigned)grid, 256, 0, s>>>(p);
    UZIP_KV_LAUNCH_CHECK("k_evict_copy");
    return UZIP_OK;
}

template <typename RawT>
int launch_evict(EvictParams &p, uint64_t rows, hipStream_t s)
{
    p.parts = 1, p.share = p.keep;
    if (p.c.tokens <= 4 * kSelThreads && p.keep <= 4 * kSelThreads) {
        // workgroups a row: one a CU, as long as each has some slots to copy
        // (32 rows of 4096: 14 us, with two a CU 25)
        const uint64_t most = ((uint64_t)p.keep + 63) / 64, parts = kCUs / rows;
        p.parts = (int)(parts < 1 ? 1 : parts > most ? most : parts);
        p.share = (p.keep + p.parts - 1) / p.parts;
        k_evict_one<4, true, RawT><<<(unsigned)(rows * p.parts), kSelThreads, 0, s>>>(p);
        UZIP_KV_LAUNCH_CHECK("k_evict_one");
        return UZIP_OK;
    }
    if (p.slices == 0) {
        if (p.c.tokens <= 16 * kSelThreads) k_evict_one<16, false, RawT><<<(unsigned)rows, kSelThreads, 0, s>>>(p);
        else k_evict_one<32, false, RawT><<<(unsigned)rows, kSelThreads, 0, s>>>(p);
        UZIP_KV_LAUNCH_CHECK("k_evict_one");
        return launch_copy<RawT>(p, rows, s);
    }
    const unsigned grid = (unsigned)(rows * p.slices);
    k_evict_level<0><<<grid, kSelThreads, 0, s>>>(p);
    UZIP_KV_LAUNCH_CHECK("k_evict_level");
    k_evict_level<1><<<grid, kSelThreads, 0, s>>>(p);
    UZIP_KV_LAUNCH_CHECK("k_evict_level");
    k_evict_level<2><<<grid, kSelThreads, 0, s>>>(p);
    UZIP_KV_LAUNCH_CHECK("k_evict_level");
    k_evict_index<<<grid, kSelThreads, 0, s>>>(p);
    UZIP_KV_LAUNCH_CHECK("k_evict_index");
    return launch_copy<RawT>(p, rows, s);
}

struct EvictWs {
    uint64_t slices, off_count, off_found, bytes;
};

EvictWs evict_ws(uint64_t rows, uint32_t tokens)
{
    EvictWs w{};
    if (tokens <= (uint32_t)kOneTokens) return w;
    w.slices = (tokens + kSlice - 1) / kSlice;
    const auto up = [](uint64_t v) { return (v + 255) & ~255ull; };
    w.off_count = up(rows * 3 * w.slices * kBins * 2);
    w.off_found = w.off_count + up(rows * 2 * w.slices * 4);
    w.bytes = w.off_found + up(rows * 2 * 8);
    return w;
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
    if (cache->k == cache->v) return UZIP_EINVAL;
    RopeParams p;
    memset(&p, 0, sizeof p);
    if (a->q.data || a->q_out.data) {
        if (!valid_tensor(a->q) || !valid_tensor(a->q_out) || a->heads < 1 || a->heads > 65535) return UZIP_EINVAL;
        if (a->q.data == a->q_out.data && !same_tensor(a->q, a->q_out)) return UZIP_EINVAL;
        if (a->q_out.data == a->k.data || a->q_out.data == a->v.data) return UZIP_EINVAL;      // read beside it
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
    return uzip_kv::evict_ws((uint64_t)seqs * kv_heads, cache_tokens).bytes;
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
    if (!aligned(a->score_out, 4) || !aligned(a->length_out, 4) || !aligned(d_ws, 16)) return UZIP_EINVAL;
    if (cache->k == out->k || cache->v == out->v || cache->k == out->v || cache->v == out->k || out->k == out->v) return UZIP_EINVAL;
    const uint64_t rows = (uint64_t)cache->seqs * cache->heads;
    const EvictWs ws = evict_ws(rows, a->score_tokens);
    if (ws.bytes && !d_ws) return UZIP_EINVAL;
    if (ws_bytes < ws.bytes) return UZIP_ENOSPC;
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
    p.hist = static_cast<uint16_t *>(d_ws);
    p.count = reinterpret_cast<uint32_t *>(static_cast<char *>(d_ws) + ws.off_count);
    p.found = reinterpret_cast<uint2 *>(static_cast<char *>(d_ws) + ws.off_found);
    p.slices = (int)ws.slices;
    const uint64_t each = 256 / (p.D / 8) * 4, groups = (a->keep + each - 1) / each;
    if (rows * groups >= (1ull << 31) || rows * ws.slices >= (1ull << 31)) return UZIP_EINVAL;
    return cache->dtype == UZIP_KV_E5M2 ? launch_evict<u32x2>(p, rows, s) : launch_evict<u32x4>(p, rows, s);
}

}  // extern "C"

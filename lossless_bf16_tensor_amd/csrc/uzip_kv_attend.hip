// uzip_kv_attend.hip -- attention of drafted tokens over a KV cache (gfx950,
// wave64). The C-ABI is declared in include/uzip_kv.h.
//
// For one sequence and key/value head the R = tokens * group query rows share
// the keys. With c = scale * log2(e), a wave keeps for each row the running
// maximum m of s = q.k, the sum l of p = 2^(c (s - m)) and the unnormalised
// output o = sum p v, all in binary32, in one pass over its keys:
//   m' = max(m, max s),  l = l 2^(c (m - m')) + sum p,  o likewise.
// Pieces of the key axis are joined by the same rule: first the waves of a
// workgroup in LDS, then (k_attend_join) the workgroups of a row.
//
// Nothing goes through LDS on the way to the matrix cores. With
// v_mfma_f32_16x16x32 the wave computes S^T = K Q^T (16 keys x 16 rows): lane
// (x = lane % 16, g = lane / 16) needs for key x the 8 dims 32 ks + 8 g ..
// + 7, one 16-byte load, and gets for row x the keys 4 g .. 4 g + 3. Then
// O^T = V^T P^T over 32 keys at once needs from lane (x, g) the weights of
// row x for 8 keys: exactly the ones it has from two S^T tiles, if the key
// axis of the product runs (g, tile, i) instead of in order. So the weights
// stay where they are, and only V^T must follow that order: lane (x, g) loads
// 8 (or 4) dims of its 8 keys and transposes them with byte permutes.
// Maximum and sum of a row need only the four lanes with the same x.
// E5M2 is the upper byte of FP16, so the permute that transposes also widens.
#include "kv_common.h"

namespace uzip_kv {
namespace {

constexpr int kWaves = 4;                     // per workgroup
constexpr int kTileKeys = 32;
constexpr float kSlack = 8.f;

struct AttendParams {
    CacheView c;
    const char *q;
    char *out;
    float *lse, *score;
    const int32_t *length, *drafted;
    const uint8_t *tree;
    int64_t qs0, qs1, qs2, os0, os1, os2;     // bytes
    int64_t sc0, sc1, tr0, tr1;               // elements
    int score_tokens;
    float *part_o;                            // [row][split][DP], when nsplit > 1
    float2 *part_ml;                          // [row][split]: maximum (times c), sum
    int T, G, R, D, heads;                    // heads: key/value heads
    int nsplit, nrg, min_tiles;
    int wk;                                   // waves of a workgroup that share rows and split keys
    float c2;                                 // scale * log2(e)
    int q_f16;
};

// tiles per split: the same for the kernel that fills and the one that joins
__device__ inline int tiles_per_split(int ntiles, const AttendParams &p)
{
    int t = (ntiles + p.nsplit - 1) / p.nsplit;
    t = t < p.min_tiles ? p.min_tiles : t;
    return (t + p.wk - 1) / p.wk * p.wk;
}

template <int CT>
using Raw = typename std::conditional<CT == kE5M2, u32x2, u32x4>::type;       // 8 elements

template <int CT>
__device__ inline u32x4 widen(const Raw<CT> &r)
{
    if constexpr (CT == kE5M2)
        return u32x4{__builtin_amdgcn_perm(r.x, r.x, 0x010c000cu), __builtin_amdgcn_perm(r.x, r.x, 0x030c020cu),
                     __builtin_amdgcn_perm(r.y, r.y, 0x010c000cu), __builtin_amdgcn_perm(r.y, r.y, 0x030c020cu)};
    else
        return r;
}

template <int CT>
__device__ inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (CT == kBF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// infinities and NaN of packed elements: their bits where an element is not
// finite (all of the element), zero elsewhere
template <int CT>
__device__ inline uint32_t not_finite(uint32_t w)
{
    if constexpr (CT == kE5M2) {
        // exponent bits 6..2 of a byte all set: adding the lowest one carries into bit 7
        const uint32_t t = ((w & 0x7c7c7c7cu) + 0x04040404u) & 0x80808080u;
        return (t << 1) - (t >> 7);                  // 0xff in each such byte
    } else {
        constexpr uint32_t e = CT == kBF16 ? 0x7f80u : 0x7c00u, one = CT == kBF16 ? 0x80u : 0x400u;
        const uint32_t t = ((w & (e | e << 16)) + (one | one << 16)) & 0x80008000u;
        return (t << 1) - (t >> 15);
    }
}

// A row's 16-byte fragments of Q for the matrix cores (8 dims at 32 ks + 8 g).
// FP8 caches are multiplied in FP16. A BF16 row for them is scaled by a power
// of two that brings its largest finite element to [1, 2): what FP16 then
// rounds is below 2^-24 of that element, the last bit of the binary32 sum.
// Returns the factor that undoes it.
template <int CT, int KS, bool PAD>
__device__ inline float load_q(const AttendParams &p, const char *row, bool there, int g, u32x4 (&f)[KS])
{
#pragma unroll
    for (int ks = 0; ks < KS; ks++) {
        f[ks] = u32x4{0, 0, 0, 0};
        if (there && (!PAD || ks * 32 + g * 8 < p.D)) f[ks] = *reinterpret_cast<const u32x4 *>(row + (ks * 32 + g * 8) * 2);
    }
    if (CT != kE5M2 || p.q_f16) return 1.f;
    float top = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t w = f[ks][i] & ~not_finite<kBF16>(f[ks][i]);
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u))));
        }
    top = quad_max(top);
    int e = top > 0.f ? ilogbf(top) : 0;
    e = e < -60 ? -60 : e;                        // keeps c2 normal; smaller rows lose nothing a sum would keep
#pragma unroll
    for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const f32x2 v = unpack2<false>(f[ks][i]);
            f[ks][i] = pack2<true>(ldexpf(v.x, -e), ldexpf(v.y, -e));
        }
    return ldexpf(1.f, e);
}

// The two 16-key halves of a tile: where their rows start, and whether every
// key is a cached token that all queries see (fast).
struct Tile {
    const char *k[2], *v[2];
    int key;
    bool there[2];
    bool fast;
};

// Finds tiles for one wave. Page numbers of its next 32 tiles are held one
// half tile a lane, so a lookup costs a readlane and not a dependent load.
struct TileFinder {
    int batch = -1;
    int entry = -1;

    __device__ inline Tile at(const AttendParams &p, int b, int h, int i, int first, int n, int end)
    {
        Tile t;
        t.key = (first + i * p.wk) * kTileKeys;
        if (p.c.table && (i >> 5) != batch) {
            batch = i >> 5;
            const int lane = (int)(threadIdx.x & 63);
            const int64_t key = ((int64_t)first + ((int64_t)batch * 32 + (lane >> 1)) * p.wk) * kTileKeys + (lane & 1) * 16;
            entry = key < end ? p.c.table[b * p.c.ts + (key >> p.c.shift)] : -1;
        }
#pragma unroll
        for (int x = 0; x < 2; x++) {
            const int key = t.key + 16 * x;
            int64_t ko, vo;
            if (p.c.table) {
                const uint32_t page = (uint32_t)__builtin_amdgcn_readlane(entry, 2 * (i & 31) + x);
                t.there[x] = key < end && page < p.c.pages;
                const int64_t in = key & ((1 << p.c.shift) - 1);
                ko = (int64_t)page * p.c.ks0 + in * p.c.ks1;
                vo = (int64_t)page * p.c.vs0 + in * p.c.vs1;
            } else {
                t.there[x] = key < end;
                ko = b * p.c.ks0 + key * p.c.ks1;
                vo = b * p.c.vs0 + key * p.c.vs1;
            }
            t.k[x] = p.c.k + (t.there[x] ? ko + h * p.c.ks2 : 0);
            t.v[x] = p.c.v + (t.there[x] ? vo + h * p.c.vs2 : 0);
        }
        t.fast = t.there[0] && t.there[1] && t.key + kTileKeys <= n;
        return t;
    }
};

// What a lane's row sees of its eight keys, a bit each: keys 4 g .. 4 g + 3 of
// both halves of a tile.
// ... those before place `left` behind the lane's first key
__device__ inline uint32_t leading_bits(int left)
{
    const int a = min(max(left, 0), 4), c = min(max(left - 16, 0), 4);
    return ((1u << a) - 1) | ((1u << c) - 1) << 4;
}

// ... those whose page is there
__device__ inline uint32_t there_bits(const Tile &t) { return (t.there[0] ? 0x0fu : 0) | (t.there[1] ? 0xf0u : 0); }

// ... those of the drafted tokens, the first of them drafted token j0, that
// the mask names. Its bytes are read at places held inside it, all at once.
__device__ inline uint32_t tree_bits(const AttendParams &p, int b, int tok, int j0, int nd)
{
    const uint8_t *row = p.tree + b * p.tr0 + min(tok, nd - 1) * p.tr1;
    uint32_t bits = 0, named[8];
#pragma unroll
    for (int k = 0; k < 8; k++) named[k] = row[min(max(j0 + 16 * (k >> 2) + (k & 3), 0), nd - 1)];
#pragma unroll
    for (int k = 0; k < 8; k++) {
        const int j = j0 + 16 * (k >> 2) + (k & 3);
        bits |= named[k] && j >= 0 && j < nd ? 1u << k : 0;
    }
    return bits;
}

// 8 dims (32 ks + 8 g ..) of key x in each half
template <int CT, int KS, bool PAD, bool MASKED>
__device__ inline void load_keys(const AttendParams &p, const Tile &t, int end, int x, int g, uint32_t off, Raw<CT> (&r)[2][KS])
{
    constexpr int es = CT == kE5M2 ? 1 : 2;
#pragma unroll
    for (int hf = 0; hf < 2; hf++) {
        const bool row = !MASKED || (t.there[hf] && t.key + 16 * hf + x < end);
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
            if (MASKED || PAD) r[hf][ks] = Raw<CT>{};
            if (row && (!PAD || ks * 32 + g * 8 < p.D)) r[hf][ks] = *reinterpret_cast<const Raw<CT> *>(t.k[hf] + (off + ks * 32 * es));
        }
    }
}

// One wave's rows over its keys. DP: the head dim rounded up to 64, 128 or
// 256 (PAD: it is smaller than that); RB: row blocks of 16.
template <int CT, int DP, int RB, bool PAD>
__global__ __launch_bounds__(kWaves * 64, RB == 4 || DP == 256 ? 1 : 2) void k_attend(AttendParams p)
{
    constexpr int KS = DP / 32;                   // steps of the product over the head dim
    constexpr int VE = DP >= 128 ? 8 : 4;         // dims that a lane loads at once
    constexpr int VC = DP >= 128 ? DP / 128 : 1;  // ... and how often
    constexpr int NV = VE * VC;                   // output products; dim = c * 128 + (4 g + i) * VE + e
    constexpr int VW = VE * (CT == kE5M2 ? 1 : 2) / 4;   // dwords of a load
    constexpr int es = CT == kE5M2 ? 1 : 2;
    constexpr bool f16 = CT != kBF16;             // type of the products
    __shared__ float smem[2 * RB * 16 * DP + 2 * kWaves * RB * 16];

    const int lane = (int)(threadIdx.x & 63), x = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    int id = (int)blockIdx.x;
    const int h = id % p.heads;
    id /= p.heads;
    const int rg = id % p.nrg;
    id /= p.nrg;
    const int split = id % p.nsplit, b = id / p.nsplit;
    const int wkey = wave & (p.wk - 1), wrow = wave / p.wk;
    const int n = __builtin_amdgcn_readfirstlane(clamp_length(p.length, b, p.c.tokens));
    const int nd = __builtin_amdgcn_readfirstlane(clamp_drafted(p.drafted, b, p.T));
    const int end = nd == 0 ? 0 : (uint32_t)nd > p.c.tokens - (uint32_t)n ? (int)p.c.tokens : n + nd;
    const int ntiles = (end + kTileKeys - 1) / kTileKeys;
    const int tps = tiles_per_split(ntiles, p);
    const int t0 = split * tps, t1 = min(t0 + tps, ntiles);
    if (p.nsplit > 1 && t0 >= t1) return;         // the joining kernel knows

    // this wave's rows: their token, and Q
    const int row0 = (rg * (kWaves / p.wk) + wrow) * RB * 16;
    int tok[RB];
    float c2[RB];
    u32x4 q[RB][KS];
#pragma unroll
    for (int rb = 0; rb < RB; rb++) {
        const int r = row0 + rb * 16 + x;
        tok[rb] = r / p.G;
        c2[rb] = p.c2 * load_q<CT, KS, PAD>(p, p.q + b * p.qs0 + tok[rb] * p.qs1 + (int64_t)(h * p.G + r % p.G) * p.qs2, r < p.R, g, q[rb]);
    }
    // keys this wave can see: a chain's later tokens are not read for earlier rows
    int lim = end;
    if (!p.tree) lim = min(end, n + min((min(row0 + RB * 16, p.R) - 1) / p.G, p.T - 1) + 1);

    f32x4 acc[RB][NV] = {};
    float m[RB], l[RB];                           // l: of this lane's keys
#pragma unroll
    for (int rb = 0; rb < RB; rb++) m[rb] = -INFINITY, l[rb] = 0.f;

    const uint32_t koff = (uint32_t)(x * p.c.ks1) + g * 8 * es;
    const uint32_t voff = (uint32_t)(g * 4 * p.c.vs1) + x * VE * es;
    typedef uint32_t vraw __attribute__((ext_vector_type(VW)));

    const auto score_tile = [&](const Raw<CT> (&kr)[2][KS], f32x4 (&s)[RB][2]) {
#pragma unroll
        for (int hf = 0; hf < 2; hf++)
#pragma unroll
            for (int ks = 0; ks < KS; ks++) {
                const u32x4 a = widen<CT>(kr[hf][ks]);
#pragma unroll
                for (int rb = 0; rb < RB; rb++) s[rb][hf] = mfma<CT>(a, q[rb][ks], ks ? s[rb][hf] : f32x4{0.f, 0.f, 0.f, 0.f});
            }
    };
    // Scores to weights. m need not be the maximum so far, only near it: the
    // weights stay below 2^kSlack and nothing is lost in binary32, while the
    // output is scaled anew in the first tile and then hardly ever.
    const auto weigh_tile = [&](f32x4 (&s)[RB][2], u32x4 (&pw)[RB]) {
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            float top = fmaxf(fmaxf(fmaxf(s[rb][0][0], s[rb][0][1]), fmaxf(s[rb][0][2], s[rb][0][3])),
                              fmaxf(fmaxf(s[rb][1][0], s[rb][1][1]), fmaxf(s[rb][1][2], s[rb][1][3])));
            top = quad_max(top);
            if (__builtin_amdgcn_ballot_w64((top - m[rb]) * c2[rb] > kSlack)) {
                top = fmaxf(top, m[rb]);
                const float a = __builtin_amdgcn_exp2f((m[rb] - (top == -INFINITY ? 0.f : top)) * c2[rb]);
                m[rb] = top;
                l[rb] *= a;
#pragma unroll
                for (int e = 0; e < NV; e++) acc[rb][e] *= a;
            }
            const float base = (m[rb] == -INFINITY ? 0.f : m[rb]) * c2[rb];
#pragma unroll
            for (int hf = 0; hf < 2; hf++)
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    s[rb][hf][k] = __builtin_amdgcn_exp2f(fmaf(s[rb][hf][k], c2[rb], -base));
                    l[rb] += s[rb][hf][k];
                }
            // The one rounding of the weights, half a step of the products'
            // type. Their sum is taken before it: lse keeps binary32.
            pw[rb] = u32x4{pack2<f16>(s[rb][0][0], s[rb][0][1]), pack2<f16>(s[rb][0][2], s[rb][0][3]),
                           pack2<f16>(s[rb][1][0], s[rb][1][1]), pack2<f16>(s[rb][1][2], s[rb][1][3])};
        }
    };
    // element (c, e) of the lane's dims for its eight keys
    const auto value_fragment = [&](const vraw (&vr)[VC][8], int c, int e) {
        u32x4 a;
#pragma unroll
        for (int k = 0; k < 4; k++) {
            if constexpr (CT == kE5M2) {
                const uint32_t sel = ((4u + e % 4) << 24) | (0x0cu << 16) | ((uint32_t)(e % 4) << 8) | 0x0cu;
                a[k] = __builtin_amdgcn_perm(vr[c][2 * k + 1][e / 4], vr[c][2 * k][e / 4], sel);
            } else {
                a[k] = __builtin_amdgcn_perm(vr[c][2 * k + 1][e / 2], vr[c][2 * k][e / 2], e % 2 ? 0x07060302u : 0x05040100u);
            }
        }
        return a;
    };
    const auto add_tile = [&](const vraw (&vr)[VC][8], const u32x4 (&pw)[RB]) {
#pragma unroll
        for (int c = 0; c < VC; c++)
#pragma unroll
            for (int e = 0; e < VE; e++) {
                const u32x4 a = value_fragment(vr, c, e);
#pragma unroll
                for (int rb = 0; rb < RB; rb++) acc[rb][c * VE + e] = mfma<CT>(a, pw[rb], acc[rb][c * VE + e]);
            }
    };

    // Tiles that every row sees: keys one tile ahead in registers, values
    // loaded while the scores are worked out.
    const int first = t0 + wkey, count = row0 < p.R ? (t1 - first + p.wk - 1) / p.wk : 0;
    int i = 0;
    if (count > 0) {
        TileFinder finder;
        Tile t = finder.at(p, b, h, 0, first, n, lim);
        Raw<CT> kr[2][KS];
        if (t.fast) load_keys<CT, KS, PAD, false>(p, t, lim, x, g, koff, kr);
        while (t.fast) {
            Tile nxt = t;
            nxt.fast = false;
            if (++i < count) {
                const Tile f = finder.at(p, b, h, i, first, n, lim);
                if (f.fast) nxt = f;
            }
            vraw vr[VC][8];
#pragma unroll
            for (int c = 0; c < VC; c++)
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    if (PAD) vr[c][j] = vraw{};
                    if (!PAD || c * 128 + x * VE < p.D)
                        vr[c][j] = *reinterpret_cast<const vraw *>(t.v[j >> 2] + (j & 3) * p.c.vs1 + (voff + c * 128 * es));
                }
            f32x4 s[RB][2];
            u32x4 pw[RB];
            score_tile(kr, s);
            load_keys<CT, KS, PAD, false>(p, nxt, lim, x, g, koff, kr);   // the same ones again after the last
            weigh_tile(s, pw);
            add_tile(vr, pw);
            t = nxt;
        }
    }
    // The others: the drafted tokens' own tiles, the last one, absent pages.
    TileFinder finder;
    for (; i < count; i++) {
        const Tile t = finder.at(p, b, h, i, first, n, lim);
        if (t.key >= lim) break;
        Raw<CT> kr[2][KS];
        vraw vr[VC][8];
        load_keys<CT, KS, PAD, true>(p, t, lim, x, g, koff, kr);
#pragma unroll
        for (int c = 0; c < VC; c++)
#pragma unroll
            for (int j = 0; j < 8; j++) {
                vr[c][j] = vraw{};
                if ((!PAD || c * 128 + x * VE < p.D) && t.there[j >> 2] && t.key + 16 * (j >> 2) + 4 * g + (j & 3) < lim)
                    vr[c][j] = *reinterpret_cast<const vraw *>(t.v[j >> 2] + (j & 3) * p.c.vs1 + (voff + c * 128 * es));
            }
        f32x4 s[RB][2];
        u32x4 pw[RB];
        score_tile(kr, s);
        uint32_t seen[RB];
#pragma unroll
        for (int rb = 0; rb < RB; rb++) seen[rb] = 0;
        if (p.tree) {
#pragma unroll
            for (int rb = 0; rb < RB; rb++) seen[rb] = tree_bits(p, b, tok[rb], t.key + 4 * g - n, nd);
        }
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            seen[rb] |= leading_bits((p.tree ? n : min(lim, n + tok[rb] + 1)) - t.key - 4 * g);
            seen[rb] &= there_bits(t);
#pragma unroll
            for (int k = 0; k < 8; k++) s[rb][k >> 2][k & 3] = seen[rb] >> k & 1 ? s[rb][k >> 2][k & 3] : -INFINITY;
        }
        weigh_tile(s, pw);
        // A value that is not finite must reach only the rows that see its
        // key, and in a product it would reach all (0 * inf). Rare: count the
        // seen ones per row and dim with products of zeros and ones, +inf and
        // NaN in one, -inf and NaN in the other, and leave them out below.
        uint32_t any = 0;
#pragma unroll
        for (int c = 0; c < VC; c++)
#pragma unroll
            for (int j = 0; j < 8; j++)
#pragma unroll
                for (int w = 0; w < VW; w++) any |= not_finite<CT>(vr[c][j][w]);
        if (__builtin_amdgcn_ballot_w64(any != 0)) {
            constexpr uint32_t one = f16 ? 0x3c003c00u : 0x3f803f80u;
            u32x4 pi[RB];
#pragma unroll
            for (int rb = 0; rb < RB; rb++)
#pragma unroll
                for (int k = 0; k < 4; k++)
                    pi[rb][k] = (seen[rb] >> (2 * k) & 1 ? one & 0xffffu : 0) | (seen[rb] >> (2 * k + 1) & 1 ? one & 0xffff0000u : 0);
            constexpr uint32_t top16 = f16 ? 0x7c00u : 0x7f80u;
#pragma unroll
            for (int c = 0; c < VC; c++)
#pragma unroll
                for (int e = 0; e < VE; e++) {
                    const u32x4 a = value_fragment(vr, c, e);
                    u32x4 up, down;
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const uint32_t bad = not_finite<f16 ? kF16 : kBF16>(a[k]);
                        uint32_t u = 0, d = 0;
#pragma unroll
                        for (int half = 0; half < 2; half++) {
                            const uint32_t v = a[k] >> (16 * half) & 0xffffu, o = (one & 0xffffu) << (16 * half);
                            if (bad >> (16 * half) & 1) {
                                if (v != (top16 | 0x8000u)) u |= o;
                                if (v != top16) d |= o;
                            }
                        }
                        up[k] = u, down[k] = d;
                    }
#pragma unroll
                    for (int rb = 0; rb < RB; rb++) {
                        const f32x4 nu = mfma<CT>(up, pi[rb], f32x4{0.f, 0.f, 0.f, 0.f}), nn = mfma<CT>(down, pi[rb], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            if (nu[k] > 0.f) acc[rb][c * VE + e][k] += INFINITY;
                            if (nn[k] > 0.f) acc[rb][c * VE + e][k] -= INFINITY;
                        }
                    }
                }
#pragma unroll
            for (int c = 0; c < VC; c++)
#pragma unroll
                for (int j = 0; j < 8; j++)
#pragma unroll
                    for (int w = 0; w < VW; w++) vr[c][j][w] &= ~not_finite<CT>(vr[c][j][w]);
        }
        add_tile(vr, pw);
    }

    // join the waves that split the keys
#pragma unroll
    for (int rb = 0; rb < RB; rb++) {
        l[rb] = quad_sum(l[rb]);
        m[rb] *= c2[rb];                          // comparable between waves; -inf stays
    }
    if (p.wk > 1) {
        float *ml = smem + 2 * RB * 16 * DP;      // [wave][row][2]
        if (g == 0)
#pragma unroll
            for (int rb = 0; rb < RB; rb++) {
                ml[(wave * RB * 16 + rb * 16 + x) * 2] = m[rb];
                ml[(wave * RB * 16 + rb * 16 + x) * 2 + 1] = l[rb];
            }
        __syncthreads();
        const int w0 = wave - wkey;
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            float top = -INFINITY, sum = 0.f;
            for (int k = 0; k < p.wk; k++) top = fmaxf(top, ml[((w0 + k) * RB * 16 + rb * 16 + x) * 2]);
            const float base = top == -INFINITY ? 0.f : top;
            for (int k = 0; k < p.wk; k++)
                sum += ml[((w0 + k) * RB * 16 + rb * 16 + x) * 2 + 1] * __builtin_amdgcn_exp2f(ml[((w0 + k) * RB * 16 + rb * 16 + x) * 2] - base);
            const float a = __builtin_amdgcn_exp2f(m[rb] - base);
            m[rb] = top;
            l[rb] = sum;
#pragma unroll
            for (int e = 0; e < NV; e++) acc[rb][e] *= a;
        }
        for (int step = p.wk >> 1; step; step >>= 1) {
            // 4 waves: waves 2, 3 hand over to 0, 1, then 1 to 0; 2 + 2 waves: 1 to 0 and 3 to 2
            const int slot = p.wk == 4 ? wkey & 1 : wrow;
            float *buf = smem + slot * RB * 16 * DP;
            if (wkey >= step && wkey < 2 * step)
#pragma unroll
                for (int rb = 0; rb < RB; rb++)
#pragma unroll
                    for (int e = 0; e < NV; e++)
                        *reinterpret_cast<f32x4 *>(buf + ((rb * NV + e) * 64 + lane) * 4) = acc[rb][e];
            __syncthreads();
            if (wkey < step) {
                buf = smem + (p.wk == 4 ? (wkey + step) & 1 : wrow) * RB * 16 * DP;
#pragma unroll
                for (int rb = 0; rb < RB; rb++)
#pragma unroll
                    for (int e = 0; e < NV; e++)
                        acc[rb][e] += *reinterpret_cast<const f32x4 *>(buf + ((rb * NV + e) * 64 + lane) * 4);
            }
            __syncthreads();
        }
        if (wkey) return;
    }

#pragma unroll
    for (int rb = 0; rb < RB; rb++) {
        const int r = row0 + rb * 16 + x;
        if (r >= p.R) continue;
        if (p.nsplit > 1) {
            const int64_t at = (((int64_t)b * p.heads + h) * p.R + r) * p.nsplit + split;
            if (g == 0) p.part_ml[at] = make_float2(m[rb], l[rb]);
            float *o = p.part_o + at * DP;
#pragma unroll
            for (int c = 0; c < VC; c++)
#pragma unroll
                for (int ii = 0; ii < 4; ii++)
#pragma unroll
                    for (int e = 0; e < VE; e += 4)
                        *reinterpret_cast<f32x4 *>(o + c * 128 + (4 * g + ii) * VE + e) =
                            f32x4{acc[rb][c * VE + e][ii], acc[rb][c * VE + e + 1][ii], acc[rb][c * VE + e + 2][ii], acc[rb][c * VE + e + 3][ii]};
            continue;
        }
        const bool empty = l[rb] == 0.f || tok[rb] >= nd;      // a seen key's weight is 1 at the maximum, or NaN
        const float inv = empty ? 0.f : 1.f / l[rb];
        const int head = h * p.G + r % p.G;
        if (g == 0 && p.lse) p.lse[((int64_t)b * p.T + tok[rb]) * (p.heads * p.G) + head] = empty ? -INFINITY : (m[rb] + __log2f(l[rb])) * 0.6931471805599453f;
        char *o = p.out + b * p.os0 + tok[rb] * p.os1 + head * p.os2;
        const bool half = f16 && (CT == kF16 || p.q_f16);
#pragma unroll
        for (int c = 0; c < VC; c++)
#pragma unroll
            for (int ii = 0; ii < 4; ii++) {
                const int d = c * 128 + (4 * g + ii) * VE;
                if (PAD && d >= p.D) continue;
                uint32_t w[VE / 2];
#pragma unroll
                for (int e = 0; e < VE; e += 2) {
                    const float u = empty ? 0.f : acc[rb][c * VE + e][ii] * inv, v = empty ? 0.f : acc[rb][c * VE + e + 1][ii] * inv;
                    w[e / 2] = half ? pack2<true>(u, v) : pack2<false>(u, v);
                }
                if constexpr (VE == 8)
                    *reinterpret_cast<u32x4 *>(o + d * 2) = u32x4{w[0], w[1], w[2], w[3]};
                else
                    *reinterpret_cast<u32x2 *>(o + d * 2) = u32x2{w[0], w[1]};
            }
    }
}

// Joins a row's splits: W waves a row, each taking every W-th split.
template <int DP, int W>
__global__ __launch_bounds__(kWaves * 64) void k_attend_join(AttendParams p, int64_t rows, int half)
{
    constexpr int E = DP / 64, U = 8;             // dims a lane, splits whose loads are under way together
    __shared__ float so[W > 1 ? kWaves : 1][DP];
    const int lane = (int)(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t row = (int64_t)blockIdx.x * (kWaves / W) + wave / W;      // ((b * heads) + h) * R + r
    if (row >= rows) return;                      // W == 1 only: rows are whole workgroups otherwise
    const int part = wave % W;
    const int r = (int)(row % p.R), h = (int)(row / p.R % p.heads), b = (int)(row / p.R / p.heads);
    const int n = clamp_length(p.length, b, p.c.tokens), nd = clamp_drafted(p.drafted, b, p.T);
    const int end = nd == 0 ? 0 : (uint32_t)nd > p.c.tokens - (uint32_t)n ? (int)p.c.tokens : n + nd;
    const int ntiles = (end + kTileKeys - 1) / kTileKeys, tps = tiles_per_split(ntiles, p);
    const int used = (ntiles + tps - 1) / tps, tok = r / p.G, head = h * p.G + r % p.G;
    const float2 *ml = p.part_ml + row * p.nsplit;
    const float *po = p.part_o + row * p.nsplit * DP + lane * E;

    float top = -INFINITY;
    for (int k = lane; k < used; k += 64) top = fmaxf(top, ml[k].x);
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int k = lane; k < used; k += 64) sum += ml[k].y * __builtin_amdgcn_exp2f(ml[k].x - base);
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);

    typedef float fe __attribute__((ext_vector_type(E)));
    fe o = {};
    for (int k0 = part; k0 < used; k0 += W * U) {
        fe v[U];
        float a[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int k = min(k0 + u * W, used - 1);
            a[u] = ml[k].x;
            if constexpr (E == 1) v[u][0] = po[(int64_t)k * DP];
            else v[u] = *reinterpret_cast<const fe *>(po + (int64_t)k * DP);
        }
#pragma unroll
        for (int u = 0; u < U; u++)
            if (k0 + u * W < used) o += v[u] * __builtin_amdgcn_exp2f(a[u] - base);
    }
    if constexpr (W > 1) {
        if constexpr (E == 1) so[wave][lane] = o[0];
        else *reinterpret_cast<fe *>(&so[wave][lane * E]) = o;
        __syncthreads();
        if (part) return;
        for (int w = 1; w < W; w++)
            if constexpr (E == 1) o[0] += so[wave + w][lane];
            else o += *reinterpret_cast<const fe *>(&so[wave + w][lane * E]);
    }
    const bool empty = sum == 0.f || tok >= nd;
    if (lane == 0 && p.lse) p.lse[((int64_t)b * p.T + tok) * (p.heads * p.G) + head] = empty ? -INFINITY : (top + __log2f(sum)) * 0.6931471805599453f;
    if (lane * E >= p.D) return;
    const float inv = 1.f / sum;
    char *out = p.out + b * p.os0 + tok * p.os1 + head * p.os2 + lane * E * 2;
    if constexpr (E == 1) {
        const float u = empty ? 0.f : o[0] * inv;
        *reinterpret_cast<uint16_t *>(out) = (uint16_t)(half ? pack2<true>(u, 0.f) : pack2<false>(u, 0.f));
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float u = empty ? 0.f : o[e] * inv, v = empty ? 0.f : o[e + 1] * inv;
            *reinterpret_cast<uint32_t *>(out + e * 2) = half ? pack2<true>(u, v) : pack2<false>(u, v);
        }
    }
}

// score[key] += sum over a kv head's rows of exp(s - lse). With the rows' lse
// known, a wave owns 32 keys, keeps them in registers and passes over the
// rows: no atomics, each sum in one fixed order. The products are those of
// k_attend, bit for bit.
template <int CT, int DP, bool PAD>
__global__ __launch_bounds__(kWaves * 64, 2) void k_attend_weigh(AttendParams p)
{
    constexpr int KS = DP / 32;
    constexpr int es = CT == kE5M2 ? 1 : 2;
    const int lane = (int)(threadIdx.x & 63), x = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    int id = (int)blockIdx.x;
    const int h = id % p.heads;
    id /= p.heads;
    const int per = (int)((p.c.tokens + kTileKeys * kWaves - 1) / (kTileKeys * kWaves));
    const int tile = (id % per) * kWaves + wave, b = id / per;
    const int n = __builtin_amdgcn_readfirstlane(clamp_length(p.length, b, p.c.tokens));
    const int nd = __builtin_amdgcn_readfirstlane(clamp_drafted(p.drafted, b, p.T));
    const int end = nd == 0 ? 0 : (uint32_t)nd > p.c.tokens - (uint32_t)n ? (int)p.c.tokens : n + nd;
    if (tile * kTileKeys >= end) return;
    TileFinder finder;
    const Tile t = finder.at(p, b, h, 0, tile, n, end);
    Raw<CT> kr[2][KS];
    load_keys<CT, KS, PAD, true>(p, t, end, x, g, (uint32_t)(x * p.c.ks1) + g * 8 * es, kr);
    // the sum this lane will add to, on its way already
    const int key = t.key + 16 * (x >> 2 & 1) + 4 * g + (x & 3);
    const bool mine = (x & 4 ? t.there[1] : t.there[0]) && key < min(end, p.score_tokens);
    float *at = p.score + b * p.sc0 + h * p.sc1 + key;
    const float old = mine ? *at : 0.f;
    f32x4 sum[2] = {};
    const int rows = nd * p.G;
    u32x4 q[KS];
    float c2, lse;
    int tok;
    const auto load_row = [&](int r0) {
        const int r = r0 + x;
        tok = r / p.G;
        const int head = h * p.G + r % p.G;
        c2 = p.c2 * load_q<CT, KS, PAD>(p, p.q + b * p.qs0 + tok * p.qs1 + head * p.qs2, r < rows, g, q);
        lse = r < rows ? p.lse[((int64_t)b * p.T + tok) * (p.heads * p.G) + head] : -INFINITY;
    };
    load_row(0);
    for (int r0 = 0; r0 < rows; r0 += 16) {
        f32x4 s[2];
#pragma unroll
        for (int hf = 0; hf < 2; hf++)
#pragma unroll
            for (int ks = 0; ks < KS; ks++) s[hf] = mfma<CT>(widen<CT>(kr[hf][ks]), q[ks], ks ? s[hf] : f32x4{0.f, 0.f, 0.f, 0.f});
        const float base = lse * 1.4426950408889634f, scale = c2;
        const bool any = lse != -INFINITY;
        const int me = tok;
        if (r0 + 16 < rows) load_row(r0 + 16);
        if (t.fast) {
#pragma unroll
            for (int hf = 0; hf < 2; hf++)
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float w = __builtin_amdgcn_exp2f(fmaf(s[hf][k], scale, -base));
                    sum[hf][k] += any ? w : 0.f;
                }
            continue;
        }
        uint32_t seen = p.tree ? tree_bits(p, b, me, t.key + 4 * g - n, nd) : 0;
        seen |= leading_bits((p.tree ? n : min(end, n + me + 1)) - t.key - 4 * g);
        seen = any ? seen & there_bits(t) : 0;
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const float w = __builtin_amdgcn_exp2f(fmaf(s[k >> 2][k & 3], scale, -base));
            sum[k >> 2][k & 3] += seen >> k & 1 ? w : 0.f;
        }
    }
    // Sums over the 16 lanes of a row of lanes, halving the keys a lane holds
    // with each step: lane x ends with key x % 8 of the eight.
    float v[8] = {sum[0][0], sum[0][1], sum[0][2], sum[0][3], sum[1][0], sum[1][1], sum[1][2], sum[1][3]};
#pragma unroll
    for (int half = 4; half; half >>= 1) {
        const bool up = x & half;
#pragma unroll
        for (int k = 0; k < half; k++) {
            const float give = up ? v[k] : v[k + half], keep = up ? v[k + half] : v[k];
            v[k] = keep + __shfl_xor(give, half);
        }
    }
    v[0] += __shfl_xor(v[0], 8);
    if (x < 8 && mine) *at = old + v[0];
}

// ------------------------------------------------------------------- host --
struct Plan {
    int DP, RB, wk, nrg, nsplit, min_tiles;
    uint64_t rows, off_ml, off_lse, bytes;
};

// The split of the key axis: enough workgroups to fill the chip a few times,
// as far as each still has a share of keys worth its joining.
Plan make_plan(uint32_t seqs, uint32_t kv_heads, uint32_t dim, uint32_t cache_tokens, uint32_t T, uint32_t heads)
{
    Plan a;
    const uint32_t G = heads / kv_heads;
    const uint64_t R = (uint64_t)T * G;
    a.DP = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
    a.RB = R <= 16 ? 1 : R <= 32 || a.DP == 256 ? 2 : 4;
    const uint64_t blocks = (R + a.RB * 16 - 1) / (a.RB * 16);
    const int wr = blocks >= 4 ? 4 : blocks >= 2 ? 2 : 1;
    a.wk = kWaves / wr;
    a.nrg = (int)((blocks + wr - 1) / wr);
    a.min_tiles = 2 * a.wk;
    const uint64_t base = (uint64_t)seqs * kv_heads * a.nrg;
    const uint64_t tiles = ((uint64_t)cache_tokens + kTileKeys - 1) / kTileKeys;
    const uint64_t want = a.RB == 1 ? 8 * kCUs : a.RB == 2 ? 4 * kCUs : 2 * kCUs;
    uint64_t split = (want + base - 1) / base;
    const uint64_t most = (tiles + a.min_tiles - 1) / a.min_tiles;
    split = split > most ? most : split;
    a.nsplit = (int)(split < 1 ? 1 : split);
    a.rows = (uint64_t)seqs * heads * T;
    const auto up = [](uint64_t v) { return (v + 255) & ~255ull; };
    a.off_ml = a.nsplit > 1 ? up(a.rows * a.nsplit * a.DP * 4) : 0;
    a.off_lse = a.off_ml + (a.nsplit > 1 ? up(a.rows * a.nsplit * 8) : 0);
    a.bytes = a.off_lse + up(a.rows * 4);
    return a;
}

bool valid_shapes(uint32_t seqs, uint32_t kv_heads, uint32_t dim, uint32_t cache_tokens, uint32_t T, uint32_t heads)
{
    return valid_dims(seqs, kv_heads, dim) && cache_tokens >= 1 && cache_tokens <= (1u << 30) && T >= 1 && T <= (1u << 20) &&
           heads >= kv_heads && heads <= 65535 && heads % kv_heads == 0 && (uint64_t)seqs * T * heads < (1ull << 30);
}

template <int CT, int DP, int RB, bool PAD>
int launch(const AttendParams &p, uint64_t grid, hipStream_t s)
{
    k_attend<CT, DP, RB, PAD><<<(unsigned)grid, kWaves * 64, 0, s>>>(p);
    UZIP_KV_LAUNCH_CHECK("k_attend");
    return UZIP_OK;
}

template <int CT, int DP, bool PAD>
int run(const AttendParams &p, const Plan &plan, int seqs, int half, hipStream_t s)
{
    const uint64_t grid = (uint64_t)seqs * p.heads * p.nrg * p.nsplit;
    int rc;
    if (plan.RB == 1) rc = launch<CT, DP, 1, PAD>(p, grid, s);
    else if (plan.RB == 2) rc = launch<CT, DP, 2, PAD>(p, grid, s);
    else if constexpr (DP <= 128) rc = launch<CT, DP, 4, PAD>(p, grid, s);
    else rc = UZIP_EINVAL;
    if (rc) return rc;
    if (p.nsplit > 1) {
        // a wave a row while it can have all its splits' loads under way at once
        if (p.nsplit <= 16) k_attend_join<DP, 1><<<(unsigned)((plan.rows + kWaves - 1) / kWaves), kWaves * 64, 0, s>>>(p, (int64_t)plan.rows, half);
        else k_attend_join<DP, kWaves><<<(unsigned)plan.rows, kWaves * 64, 0, s>>>(p, (int64_t)plan.rows, half);
        UZIP_KV_LAUNCH_CHECK("k_attend_join");
    }
    if (p.score) {
        const uint64_t per = ((uint64_t)p.c.tokens + kTileKeys * kWaves - 1) / (kTileKeys * kWaves);
        k_attend_weigh<CT, DP, PAD><<<(unsigned)(per * seqs * p.heads), kWaves * 64, 0, s>>>(p);
        UZIP_KV_LAUNCH_CHECK("k_attend_weigh");
    }
    return UZIP_OK;
}

template <int CT>
int run_type(const AttendParams &p, const Plan &plan, int seqs, int half, hipStream_t s)
{
    if (plan.DP == 64) return p.D == 64 ? run<CT, 64, false>(p, plan, seqs, half, s) : run<CT, 64, true>(p, plan, seqs, half, s);
    if (plan.DP == 128) return p.D == 128 ? run<CT, 128, false>(p, plan, seqs, half, s) : run<CT, 128, true>(p, plan, seqs, half, s);
    return p.D == 256 ? run<CT, 256, false>(p, plan, seqs, half, s) : run<CT, 256, true>(p, plan, seqs, half, s);
}

}  // namespace
}  // namespace uzip_kv

extern "C" {

uint64_t uzip_kv_attend_workspace_bytes(uint32_t seqs, uint32_t kv_heads, uint32_t dim, uint32_t cache_tokens,
                                        uint32_t tokens, uint32_t heads)
{
    if (!uzip_kv::valid_shapes(seqs, kv_heads, dim, cache_tokens, tokens, heads)) return 0;
    return uzip_kv::make_plan(seqs, kv_heads, dim, cache_tokens, tokens, heads).bytes;
}

int uzip_kv_attend(const uzip_kv_cache_t *cache, const uzip_kv_attend_args_t *a, void *d_ws, uint64_t ws_bytes,
                   hipStream_t s)
{
    using namespace uzip_kv;
    if (!a || !valid_cache(cache) || !valid_tensor(a->q) || !valid_tensor(a->out)) return UZIP_EINVAL;
    if (!valid_shapes(cache->seqs, cache->heads, cache->dim, cache->tokens, a->tokens, a->heads)) return UZIP_EINVAL;
    if (a->dtype > UZIP_KV_F16 || (cache->dtype != UZIP_KV_E5M2 && cache->dtype != a->dtype)) return UZIP_EINVAL;
    if (!a->length || !aligned(a->length, 4) || !aligned(a->drafted, 4) || !aligned(a->lse, 4) || !aligned(a->score, 4)) return UZIP_EINVAL;
    if (!(a->scale >= 0x1p-60f) || !(a->scale <= 0x1p60f)) return UZIP_EINVAL;
    if (a->reserved || (a->score && (a->score_stride[0] < 0 || a->score_stride[1] < 0 || a->score_tokens > cache->tokens))) return UZIP_EINVAL;
    if (a->tree && (a->tree_stride[0] < 0 || a->tree_stride[1] < 0)) return UZIP_EINVAL;
    if (!d_ws || !aligned(d_ws, 16)) return UZIP_EINVAL;
    const Plan plan = make_plan(cache->seqs, cache->heads, cache->dim, cache->tokens, a->tokens, a->heads);
    if (ws_bytes < plan.bytes) return UZIP_ENOSPC;
    if ((uint64_t)cache->seqs * cache->heads * plan.nrg * plan.nsplit >= (1ull << 31) ||
        (uint64_t)cache->seqs * cache->heads * ((cache->tokens + 127) / 128) >= (1ull << 31)) return UZIP_EINVAL;

    AttendParams p;
    memset(&p, 0, sizeof p);
    p.c = view_of(cache);
    p.q = static_cast<const char *>(a->q.data);
    p.out = static_cast<char *>(a->out.data);
    p.qs0 = a->q.stride[0] * 2, p.qs1 = a->q.stride[1] * 2, p.qs2 = a->q.stride[2] * 2;
    p.os0 = a->out.stride[0] * 2, p.os1 = a->out.stride[1] * 2, p.os2 = a->out.stride[2] * 2;
    char *ws = static_cast<char *>(d_ws);
    p.lse = a->lse ? a->lse : a->score ? reinterpret_cast<float *>(ws + plan.off_lse) : nullptr;
    p.score = a->score;
    p.sc0 = a->score_stride[0], p.sc1 = a->score_stride[1];
    p.score_tokens = (int)a->score_tokens;
    p.length = a->length;
    p.drafted = a->drafted;
    p.tree = a->tree;
    p.tr0 = a->tree_stride[0], p.tr1 = a->tree_stride[1];
    p.part_o = reinterpret_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + plan.off_ml);
    p.T = (int)a->tokens;
    p.G = (int)(a->heads / cache->heads);
    p.R = p.T * p.G;
    p.D = (int)cache->dim;
    p.heads = (int)cache->heads;
    p.nsplit = plan.nsplit;
    p.nrg = plan.nrg;
    p.min_tiles = plan.min_tiles;
    p.wk = plan.wk;
    p.c2 = a->scale * 1.4426950408889634f;
    p.q_f16 = a->dtype == UZIP_KV_F16;
    const int seqs = (int)cache->seqs, half = p.q_f16;
    if (cache->dtype == UZIP_KV_BF16) return run_type<kBF16>(p, plan, seqs, half, s);
    if (cache->dtype == UZIP_KV_F16) return run_type<kF16>(p, plan, seqs, half, s);
    return run_type<kE5M2>(p, plan, seqs, half, s);
}

}  // extern "C"

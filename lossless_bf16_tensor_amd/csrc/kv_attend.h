// kv_attend.h -- attention of drafted tokens over a KV cache (gfx950, wave64):
// the kernels and their host side, for the files that make them for caches of
// 16 bits and E5M2 and for caches of 8 bits with scales. Internal to the
// library.
//
// For one sequence and key/value head the R = tokens * group query rows share
// the keys. With c = scale * log2(e), a wave keeps for each row the running
// maximum m of s = q.k, the sum l of p = 2^(c (s - m)) and the unnormalised
// output o = sum p v, all in binary32, in one pass over its keys:
//   m' = max(m, max s),  l = l 2^(c (m - m')) + sum p,  o likewise.
// Pieces of the key axis are joined by the same rule: first the waves of a
// workgroup in LDS, then (k_attend_join_few, _many) the workgroups of a row.
//
// With few rows the cache's bytes are the bound, and k_attend takes them from
// memory into registers: nothing goes through LDS on the way to the matrix
// cores. With more than 64, over enough keys, the products are, and
// k_attend_shared lets eight waves read the keys and values that one workgroup
// loads.
//
// In both nothing but keys and values moves between lanes. With
// v_mfma_f32_16x16x32 the wave computes S^T = K Q^T (16 keys x 16 rows): lane
// (x = lane % 16, g = lane / 16) needs for key x the 8 dims 32 ks + 8 g ..
// + 7, one 16-byte load, and gets for row x the keys 4 g .. 4 g + 3. Then
// O^T = V^T P^T over 32 keys at once needs from lane (x, g) the weights of
// row x for 8 keys: exactly the ones it has from two S^T tiles, if the key
// axis of the product runs (g, tile, i) instead of in order. So the weights
// stay where they are, and only V^T must follow that order: lane (x, g) loads
// 8 (or 4) dims of its 8 keys and transposes them with byte permutes.
// Maximum and sum of a row need only the four lanes with the same x.
// E5M2 is the upper byte of FP16, so the permute that transposes also widens;
// keys become the queries' type, BF16 by a conversion of two at a time.
//
// Caches in 8 bits with scales: a half tile of 16 keys lies in one block, so its
// scales are two numbers for the whole wave. Scores are multiplied by the keys',
// weights by the values', before they become BF16: a weight times a scale can be
// anything that binary32 holds, and FP16 would lose it.
#ifndef UZIP_KV_ATTEND_H
#define UZIP_KV_ATTEND_H

#include "kv_common.h"

namespace uzip_kv {
namespace {

constexpr int kWaves = 4;                     // per workgroup
constexpr int kTileKeys = 32;

enum { kParts, kRuns, kWalks };

struct AttendParams {
    CacheView c;
    const char *q;
    char *out;
    float *lse, *score;
    const int32_t *length, *drafted;
    const uint8_t *tree;
    int64_t qs0, qs1, qs2, os0, os1, os2;     // bytes
    int64_t sc0, sc1, tr0, tr1;               // elements
    ScaleView scales;
    int score_tokens, weigh_tiles;            // weigh_tiles: of each wave of k_attend_weigh
    float *part_o;                            // [row][split][DP], when nsplit > 1
    float2 *part_ml;                          // [row][split]: maximum (times c, less Rows::kLift), sum
    int T, G, R, D, heads, seqs;              // heads: key/value heads
    int *used;                                // parts of each sequence, when flat
    int flat;                                 // Walk, even_part
    int nsplit, nrg, slots, min_steps, unit;  // unit: tiles that a workgroup takes in one step
    int wk;                                   // waves of a workgroup that share rows and split keys
    float c2;                                 // scale * log2(e)
};

__device__ inline int end_of(const AttendParams &p, int n, int nd)
{
    return nd == 0 ? 0 : (uint32_t)nd > p.c.tokens - (uint32_t)n ? (int)p.c.tokens : n + nd;
}

// What a workgroup works on: tiles [t0, t1) of sequence b for its rows.
struct Place {
    int b, h, rg, split, n, nd, end, t0, t1;
    bool whole;                                   // all the tiles of b: the output is final

    // A wave's lanes may leave a loop apart, so that the compiler takes what
    // follows for different in each: says that it is the same.
    __device__ inline void uniform()
    {
        const auto same = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
        b = same(b), split = same(split), n = same(n), nd = same(nd), end = same(end), t0 = same(t0), t1 = same(t1), whole = same(whole);
    }
};

// Each sequence cut into p.nsplit parts or fewer, one workgroup each.
__device__ inline int tiles_per_split(const AttendParams &p, int tiles)
{
    const int t = max((tiles + p.nsplit - 1) / p.nsplit, p.min_steps * p.unit);
    return (t + p.unit - 1) / p.unit * p.unit;
}

__device__ inline int tiles_of(const AttendParams &p, int b)
{
    return (end_of(p, clamp_length(p.length, b, p.c.tokens), clamp_drafted(p.drafted, b, p.T)) + kTileKeys - 1) / kTileKeys;
}

__device__ inline Place part_of_sequence(const AttendParams &p)
{
    Place at;
    int id = (int)blockIdx.x;
    at.h = id % p.heads;
    id /= p.heads;
    at.rg = id % p.nrg;
    id /= p.nrg;
    at.split = id % p.nsplit, at.b = id / p.nsplit;
    at.n = __builtin_amdgcn_readfirstlane(clamp_length(p.length, at.b, p.c.tokens));
    at.nd = __builtin_amdgcn_readfirstlane(clamp_drafted(p.drafted, at.b, p.T));
    at.end = end_of(p, at.n, at.nd);
    const int tiles = (at.end + kTileKeys - 1) / kTileKeys, each = tiles_per_split(p, tiles);
    at.t0 = at.split * each, at.t1 = min(at.t0 + each, tiles);
    at.whole = tiles <= each;
    return at;
}

// What a workgroup's number says. spread: workgroups go to the 8 dies in turn,
// and those of all heads for the same keys, whose rows lie side by side, are on
// one (16 sequences of up to 30000 FP8 keys of 64 in pages: 105 us, 87 so).
struct Number {
    int h, rg, k;

    __device__ inline Number(const AttendParams &p, bool spread)
    {
        int id = (int)blockIdx.x, die = 0;
        if (spread) die = id & 7, id >>= 3;
        h = id % p.heads;
        id /= p.heads;
        rg = id % p.nrg;
        k = spread ? id / p.nrg * 8 + die : id / p.nrg;
    }
};

// The places of a workgroup of which there is one a CU, so that none may have
// more to do than another: the steps (`unit` tiles) of all sequences lie in a
// row, for each key/value head and group of rows, and each of p.slots
// workgroups takes the next `chunk` of them, however the lengths differ. A
// sequence that lies in several chunks is joined afterwards; p.used says of how
// many parts. (nsplit == 1: a workgroup a sequence.)
struct Walk {
    int b, start, s0, s1, chunk, slot, h, rg;     // start: of b's steps
    int len, cnt;                                 // lane i: of sequence i, when there are at most 64

    __device__ inline static int steps(const AttendParams &p, int n, int nd)
    {
        return ((end_of(p, n, nd) + kTileKeys - 1) / kTileKeys + p.unit - 1) / p.unit;
    }
    __device__ inline static int steps(const AttendParams &p, int b)
    {
        return steps(p, clamp_length(p.length, b, p.c.tokens), clamp_drafted(p.drafted, b, p.T));
    }

    __device__ inline Walk(const AttendParams &p, bool spread = false)
    {
        const Number num(p, spread);
        h = num.h, rg = num.rg, slot = num.k;
        b = slot, start = s0 = 0, s1 = 1, chunk = 1, len = cnt = 0;
        if (p.nsplit == 1) return;
        const int lane = (int)(threadIdx.x & 63);
        int total = 0, most = 0;
        if (p.seqs <= 64) {
            if (lane < p.seqs) len = clamp_length(p.length, lane, p.c.tokens), cnt = clamp_drafted(p.drafted, lane, p.T);
            total = most = lane < p.seqs ? steps(p, len, cnt) : 0;
        } else {
            for (int i = lane; i < p.seqs; i += 64) {
                const int st = steps(p, i);
                total += st;
                most = max(most, st);
            }
        }
        if (p.seqs > 1)
            for (int x = 1; x < 64; x <<= 1) total += __shfl_xor(total, x), most = max(most, __shfl_xor(most, x));
        total = __builtin_amdgcn_readfirstlane(total);
        most = __builtin_amdgcn_readfirstlane(most);
        // a sequence is in one part more than its length asks for when it begins inside a chunk
        const int parts = p.seqs > 1 ? p.nsplit - 1 : p.nsplit;
        chunk = max(max(p.min_steps, (total + p.slots - 1) / p.slots), (most + parts - 1) / parts);
        s0 = slot * chunk, s1 = s0 < total ? min(s0 + chunk, total) : 0;      // 0: nothing for this one, start is not below it
        b = 0;
        const bool tell = blockIdx.x == 0 && threadIdx.x < 64;
        if (p.seqs == 1) {
            if (tell && lane == 0) p.used[0] = (total + chunk - 1) / chunk;
            return;
        }
        bool found = false;
        for (int base = 0, before = 0; base < p.seqs && (!found || tell); base += 64) {
            const int st = base + lane >= p.seqs ? 0 : p.seqs <= 64 ? steps(p, len, cnt) : steps(p, base + lane);
            int sum = st;
            for (int x = 1; x < 64; x <<= 1) {
                const int v = __shfl_up(sum, x);
                if (lane >= x) sum += v;
            }
            if (tell && base + lane < p.seqs)
                p.used[base + lane] = st ? (before + sum - 1) / chunk - (before + sum - st) / chunk + 1 : 0;
            const uint64_t past = __builtin_amdgcn_ballot_w64(before + sum > s0);
            if (!found && past) {
                const int at = __builtin_ctzll(past);
                b = base + at;
                start = before + __builtin_amdgcn_readlane(sum, at) - __builtin_amdgcn_readlane(st, at);
                found = true;
            }
            before += __builtin_amdgcn_readlane(sum, 63);
        }
        if (!found) s1 = 0;
    }

    __device__ inline void uniform()
    {
        const auto same = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
        b = same(b), start = same(start), s0 = same(s0), s1 = same(s1), chunk = same(chunk);
    }

    __device__ inline bool next(const AttendParams &p, Place &at)
    {
        at.h = h, at.rg = rg;
        while (start < s1 && b < p.seqs) {
            at.b = b++;
            if (p.nsplit > 1 && p.seqs <= 64) {
                at.n = __builtin_amdgcn_readlane(len, at.b);
                at.nd = __builtin_amdgcn_readlane(cnt, at.b);
            } else {
                at.n = __builtin_amdgcn_readfirstlane(clamp_length(p.length, at.b, p.c.tokens));
                at.nd = __builtin_amdgcn_readfirstlane(clamp_drafted(p.drafted, at.b, p.T));
            }
            at.end = end_of(p, at.n, at.nd);
            const int tiles = (at.end + kTileKeys - 1) / kTileKeys, st = (tiles + p.unit - 1) / p.unit, from = start;
            if (p.nsplit == 1) {
                at.split = 0, at.t0 = 0, at.t1 = tiles, at.whole = true;
                start = s1;
                return true;
            }
            start += st;
            if (st == 0) continue;
            at.t0 = max(s0 - from, 0) * p.unit, at.t1 = min(min(s1 - from, st) * p.unit, tiles);
            at.split = slot - from / chunk;
            at.whole = (from + st - 1) / chunk == from / chunk;
            return true;
        }
        return false;
    }
};

// One place a workgroup, none longer than another's may be: each sequence is cut
// into runs of `chunk` steps, as many as it has, and each workgroup finds the
// sequence and run that its number falls into. p.used says of how many parts a
// sequence is. (Cut into as many parts each, long sequences would end last.)
__device__ inline bool even_part(const AttendParams &p, Place &at)
{
    const Number num(p, true);
    at.h = num.h, at.rg = num.rg;
    const int k = num.k, lane = (int)(threadIdx.x & 63);
    at.b = at.split = at.n = at.nd = at.end = at.t0 = at.t1 = 0, at.whole = false;
    if (p.nsplit == 1) {                          // a workgroup a sequence
        if (k >= p.seqs) return false;
        at.b = k;
        at.n = clamp_length(p.length, k, p.c.tokens), at.nd = clamp_drafted(p.drafted, k, p.T);
        at.end = end_of(p, at.n, at.nd);
        at.t1 = (at.end + kTileKeys - 1) / kTileKeys, at.whole = true;
        at.uniform();
        return true;
    }
    int len = 0, cnt = 0, total = 0, most = 0;
    for (int i = lane; i < p.seqs; i += 64) {
        len = clamp_length(p.length, i, p.c.tokens), cnt = clamp_drafted(p.drafted, i, p.T);
        const int st = Walk::steps(p, len, cnt);
        total += st;
        most = max(most, st);
    }
    for (int x = 1; x < 64; x <<= 1) total += __shfl_xor(total, x), most = max(most, __shfl_xor(most, x));
    total = __builtin_amdgcn_readfirstlane(total);
    most = __builtin_amdgcn_readfirstlane(most);
    const int chunk = max(max(p.min_steps, (total + p.slots - 1) / p.slots), (most + p.nsplit - 1) / p.nsplit);
    const bool tell = blockIdx.x == 0 && threadIdx.x < 64;
    bool found = false;
    for (int base = 0, before = 0; base < p.seqs && (!found || tell); base += 64) {
        const int i = base + lane;
        if (p.seqs > 64 && i < p.seqs) len = clamp_length(p.length, i, p.c.tokens), cnt = clamp_drafted(p.drafted, i, p.T);
        const int parts = i < p.seqs ? max((Walk::steps(p, len, cnt) + chunk - 1) / chunk, 1) : 0;
        int sum = parts;
        for (int x = 1; x < 64; x <<= 1) {
            const int v = __shfl_up(sum, x);
            if (lane >= x) sum += v;
        }
        if (tell && i < p.seqs) p.used[i] = parts;
        const uint64_t past = __builtin_amdgcn_ballot_w64(before + sum > k);
        if (!found && past) {
            const int l = __builtin_ctzll(past);
            const int of = __builtin_amdgcn_readlane(parts, l);
            at.b = base + l;
            at.split = k - (before + __builtin_amdgcn_readlane(sum, l) - of);
            at.n = __builtin_amdgcn_readlane(len, l), at.nd = __builtin_amdgcn_readlane(cnt, l);
            at.end = end_of(p, at.n, at.nd);
            const int tiles = (at.end + kTileKeys - 1) / kTileKeys;
            at.t0 = at.split * chunk * p.unit, at.t1 = min(at.t0 + chunk * p.unit, tiles);
            at.whole = of == 1;
            found = true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    at.uniform();
    return __builtin_amdgcn_readfirstlane(found);
}

// What a kernel is made for: the types of the cache and, where that has 8 bits,
// of the queries. E4M3 and 8-bit integers have a scale for each block of tokens
// and head, and a half tile lies in one block.
constexpr int kE5M2BF = 3;                    // BF16 queries; kE5M2: FP16 ones
constexpr int kE4M3 = 4, kE4M3BF = 5, kI8 = 6, kI8BF = 7;      // likewise
constexpr bool is_byte(int ct) { return ct >= kE5M2; }
constexpr bool is_e5m2(int ct) { return ct == kE5M2 || ct == kE5M2BF; }
constexpr bool is_i8(int ct) { return ct == kI8 || ct == kI8BF; }
constexpr bool is_scaled(int ct) { return ct >= kE4M3; }
constexpr bool f16_queries(int ct) { return ct == kF16 || ct == kE5M2 || ct == kE4M3 || ct == kI8; }      // the output's type, and that of the products with keys
// The type of the products with values. A weight times a scale can be anything
// that binary32 holds, so beside scales it is BF16.
constexpr bool f16_weights(int ct) { return ct != kBF16 && !is_scaled(ct); }

template <int CT>
using Raw = typename std::conditional<is_byte(CT), u32x2, u32x4>::type;        // 8 elements

// byte e of a dword, a signed integer, in binary32
__device__ inline float byte_to_f32(uint32_t w, int e) { return (float)(int8_t)(w >> 8 * e); }

// Eight elements of a key, in the queries' type: any E5M2, E4M3 or 8-bit integer
// value is one of FP16 and one of BF16, so products with either are exact.
template <int CT>
__device__ inline u32x4 widen(const Raw<CT> &r)
{
    if constexpr (CT == kE4M3BF)
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.x, 1.f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.x, 1.f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.y, 1.f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.y, 1.f, true))};
    else if constexpr (CT == kE4M3)
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r.x, 1.f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r.x, 1.f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r.y, 1.f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r.y, 1.f, true))};
    else if constexpr (is_i8(CT)) {
        u32x4 a;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t w = i < 2 ? r.x : r.y;
            if constexpr (CT == kI8BF) {      // exact, so cut off
                a[i] = cut2<false>(byte_to_f32(w, 2 * (i & 1)), byte_to_f32(w, 2 * (i & 1) + 1));
            } else {                          // 0x6400 + u is 1024 + u in FP16
                const uint32_t u = __builtin_amdgcn_perm(0x64646464u, w ^ 0x80808080u, i & 1 ? 0x04030402u : 0x04010400u);
                a[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, u) - f16x2{(_Float16)1152.f, (_Float16)1152.f});
            }
        }
        return a;
    } else if constexpr (CT == kE5M2BF)
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(r.x, 1.f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(r.x, 1.f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(r.y, 1.f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(r.y, 1.f, true))};
    else if constexpr (CT == kE5M2)
        return u32x4{__builtin_amdgcn_perm(r.x, r.x, 0x010c000cu), __builtin_amdgcn_perm(r.x, r.x, 0x030c020cu),
                     __builtin_amdgcn_perm(r.y, r.y, 0x010c000cu), __builtin_amdgcn_perm(r.y, r.y, 0x030c020cu)};
    else
        return r;
}

template <bool F16>
__device__ inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// infinities and NaN of packed elements: their bits where an element is not
// finite (all of the element), zero elsewhere
template <int CT>
__device__ inline uint32_t not_finite(uint32_t w)
{
    if constexpr (is_scaled(CT)) {
        if constexpr (is_i8(CT)) return 0u;
        // E4M3 has no infinities, and its NaN are 0x7f and 0xff
        const uint32_t t = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
        return (t << 1) - (t >> 7);
    } else if constexpr (is_byte(CT)) {
        // exponent bits 6..2 of a byte all set: adding the lowest one carries into bit 7
        const uint32_t t = ((w & 0x7c7c7c7cu) + 0x04040404u) & 0x80808080u;
        return (t << 1) - (t >> 7);                  // 0xff in each such byte
    } else {
        constexpr uint32_t e = CT == kBF16 ? 0x7f80u : 0x7c00u, one = CT == kBF16 ? 0x80u : 0x400u;
        const uint32_t t = ((w & (e | e << 16)) + (one | one << 16)) & 0x80008000u;
        return (t << 1) - (t >> 15);
    }
}

// Loaded elements are widened behind this and not before: the compiler would
// carry them from one tile to the next in their wide form, which the registers
// do not hold.
template <typename V, int N, int M>
__device__ inline void hold(V (&v)[N][M])
{
    constexpr int W = sizeof(V) / 4;
    typedef uint32_t Words __attribute__((ext_vector_type(W)));
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int j = 0; j < M; j++) {
            Words u = __builtin_bit_cast(Words, v[i][j]);
#pragma unroll
            for (int k = 0; k < W; k++) {
                uint32_t word = u[k];
                asm volatile("" : "+v"(word));
                u[k] = word;
            }
            v[i][j] = __builtin_bit_cast(V, u);
        }
}

// Byte e of each of eight dwords, a lane's values of one dim and eight keys, as
// BF16.
template <int CT>
__device__ inline u32x4 turned_over(const uint32_t (&w)[8], int e)
{
    u32x4 a;
    if constexpr (is_i8(CT)) {
#pragma unroll
        for (int k = 0; k < 4; k++) a[k] = cut2<false>(byte_to_f32(w[2 * k], e), byte_to_f32(w[2 * k + 1], e));
    } else {                                  // 4 x 4 bytes turned over, then widened
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
            const uint32_t sel = e < 2 ? 0x05010400u : 0x07030602u;
            const uint32_t low = __builtin_amdgcn_perm(w[k + 1], w[k], sel), high = __builtin_amdgcn_perm(w[k + 3], w[k + 2], sel);
            const uint32_t four = __builtin_amdgcn_perm(high, low, e % 2 ? 0x07060302u : 0x05040100u);
            a[k / 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, 1.f, false));
            a[k / 2 + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, 1.f, true));
        }
    }
    return a;
}

// A row's 16-byte fragments of Q for the matrix cores (8 dims at 32 ks + 8 g).
template <int KS, bool PAD>
__device__ inline void load_q(const AttendParams &p, const char *row, bool there, int g, u32x4 (&f)[KS])
{
#pragma unroll
    for (int ks = 0; ks < KS; ks++) {
        f[ks] = u32x4{0, 0, 0, 0};
        if (there && (!PAD || ks * 32 + g * 8 < p.D)) f[ks] = *reinterpret_cast<const u32x4 *>(row + (ks * 32 + g * 8) * 2);
    }
}

// The two 16-key halves of a tile: where their rows start, and whether every
// key is a cached token that all queries see (fast).
struct Tile {
    const char *k[2], *v[2];
    int key;
    bool there[2];
    bool fast;
    float ks[2], vs[2];                       // scales
};

// Finds tiles for one wave. Page numbers of its next 32 tiles are held one
// half tile a lane, so a lookup costs a readlane and not a dependent load.
template <bool SCALED>
struct TileFinder {
    int batch = -1;
    int entry = -1;

    __device__ inline Tile at(const AttendParams &p, int b, int h, int i, int first, int n, int end)
    {
        return find(p, b, h, i, first, p.wk, n, end);
    }

    __device__ inline Tile find(const AttendParams &p, int b, int h, int i, int first, int step, int n, int end)
    {
        Tile t;
        t.key = (first + i * step) * kTileKeys;
        if (p.c.table && (i >> 5) != batch) {
            batch = i >> 5;
            const int lane = (int)(threadIdx.x & 63);
            const int64_t key = ((int64_t)first + ((int64_t)batch * 32 + (lane >> 1)) * step) * kTileKeys + (lane & 1) * 16;
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
            if constexpr (SCALED) {           // by scalar loads; of a half tile that is not there, 0
                const uint32_t from = p.c.table ? (uint32_t)__builtin_amdgcn_readlane(entry, 2 * (i & 31) + x) : (uint32_t)b;
                const uint32_t block = (uint32_t)(p.c.table ? key & ((1 << p.c.shift) - 1) : key) >> p.scales.shift;
                const uint32_t ka = from * p.scales.k0 + block * p.scales.k1 + (uint32_t)h * p.scales.k2;
                const uint32_t va = from * p.scales.v0 + block * p.scales.v1 + (uint32_t)h * p.scales.v2;
                const float ks = scalar_load(p.scales.k + (t.there[x] ? ka : 0)), vs = scalar_load(p.scales.v + (t.there[x] ? va : 0));
                t.ks[x] = t.there[x] ? ks : 0.f;
                t.vs[x] = t.there[x] ? vs : 0.f;
            }
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
// the mask names and that lie in the cache: `in` of them, which may be fewer
// than the nd (> 0) that the mask is for. Its bytes are read at places held
// inside it, all at once.
__device__ inline uint32_t tree_bits(const AttendParams &p, int b, int tok, int j0, int nd, int in)
{
    const uint8_t *row = p.tree + b * p.tr0 + min(tok, nd - 1) * p.tr1;
    uint32_t bits = 0, named[8];
#pragma unroll
    for (int k = 0; k < 8; k++) named[k] = row[min(max(j0 + 16 * (k >> 2) + (k & 3), 0), nd - 1)];
#pragma unroll
    for (int k = 0; k < 8; k++) {
        const int j = j0 + 16 * (k >> 2) + (k & 3);
        bits |= named[k] && j >= 0 && j < min(nd, in) ? 1u << k : 0;
    }
    return bits;
}

// Scores that can be read. A product's result is there after eight wait states,
// which the hardware does not keep by itself; the compiler counts them, but
// where a branch between the products and the first use leaves instructions out
// it has counted those of the longer way (head dim 64: seven along the other).
// Behind such a branch they are waited for here; its own ones, a few of the
// thousands of cycles that a tile's memory takes, are then not needed.
template <int N>
__device__ inline void settle(f32x4 (&s)[N][2])
{
    static_assert(N <= 2, "every result is named");
    if constexpr (N == 1) asm("s_nop 7" : "+v"(s[0][0]), "+v"(s[0][1]));
    else asm("s_nop 7" : "+v"(s[0][0]), "+v"(s[0][1]), "+v"(s[1][0]), "+v"(s[1][1]));
}

// 8 dims (32 ks + 8 g ..) of key x in each half
template <int CT, int KS, bool PAD, bool MASKED>
__device__ inline void load_keys(const AttendParams &p, const Tile &t, int end, int x, int g, uint32_t off, Raw<CT> (&r)[2][KS])
{
    constexpr int es = is_byte(CT) ? 1 : 2;
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

// A wave's RB blocks of 16 query rows and what it holds for them. DP: the head
// dim rounded up to 64, 128 or 256 (PAD: it is smaller than that). FINE: the
// products with the values take the weights in two terms, the rounded ones and
// what that left over, so that nothing but the output's rounding shows.
template <int CT, int DP, int RB, bool PAD, bool FINE>
struct Rows {
    static constexpr int TERMS = FINE ? 2 : 1;           // of a weight
    static constexpr int KS = DP / 32;                   // steps of the product over the head dim
    static constexpr int VE = DP >= 128 ? 8 : 4;         // dims that a lane takes at once
    static constexpr int VC = DP >= 128 ? DP / 128 : 1;  // ... and how often
    static constexpr int NV = VE * VC;                   // output products; dim = c * 128 + (4 g + i) * VE + e
    static constexpr int VW = VE * (is_byte(CT) ? 1 : 2) / 4;    // dwords of a lane's dims
    static constexpr int es = is_byte(CT) ? 1 : 2;
    static constexpr bool f16 = f16_weights(CT), half = f16_queries(CT);
    // Weights are 2^kLift at the row's maximum so far and below 2^(kLift +
    // kSlack) until it is raised. FP16 has no bits below 2^-24, and a first
    // token often has a score 15 to 20 above thousands of others: with the
    // range used up to 2^15, their weights are kept to 2^-35 of the maximum,
    // where without a lift and with a slack of 8 those below 2^-25 were lost
    // from the output. BF16 reaches as low as binary32.
    static constexpr float kSlack = f16 ? 4.f : 8.f, kLift = f16 ? 11.f : 0.f;
    static constexpr float kLeast = f16 ? 0x1p-24f : 0x1p-126f;
    typedef uint32_t Values __attribute__((ext_vector_type(VW)));

    int x, g, row0, lim;
    bool odd;                                     // poison() has something to add
    bool far;                                     // raise() has a row to bring near zero
    int tok[RB];                                  // of the lane's rows
    float m[RB], l[RB];                           // l: of this lane's keys
    float base[RB];                               // m c2 - kLift; without m c2 when raise() has taken it off the scores; 0 while m is -inf
    u32x4 q[RB][KS];
    f32x4 acc[RB][NV];

    __device__ inline void init(const AttendParams &p, int b, int h, int first_row, int n, int end)
    {
        int tid = (int)threadIdx.x;
        asm volatile("" : "+v"(tid));             // what follows from it is made anew for each place, not kept in registers
        x = tid & 15, g = (tid & 63) >> 4;
        row0 = first_row;
        odd = far = false;
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            const int r = row0 + rb * 16 + x;
            tok[rb] = r / p.G;
            load_q<KS, PAD>(p, p.q + b * p.qs0 + tok[rb] * p.qs1 + (int64_t)(h * p.G + r % p.G) * p.qs2, r < p.R, g, q[rb]);
            m[rb] = -INFINITY, l[rb] = 0.f, base[rb] = 0.f;
#pragma unroll
            for (int e = 0; e < NV; e++) acc[rb][e] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        // keys these rows can see: of a chain's later tokens, earlier rows need
        // neither products nor, in k_attend, loads
        lim = end;
        if (!p.tree) lim = min(end, n + min((min(row0 + RB * 16, p.R) - 1) / p.G, p.T - 1) + 1);
    }

    __device__ inline void score(const u32x4 (&k)[2][KS], f32x4 (&s)[RB][2])
    {
#pragma unroll
        for (int hf = 0; hf < 2; hf++)
#pragma unroll
            for (int ks = 0; ks < KS; ks++)
#pragma unroll
                for (int rb = 0; rb < RB; rb++) s[rb][hf] = mfma<half>(k[hf][ks], q[rb][ks], ks ? s[rb][hf] : f32x4{0.f, 0.f, 0.f, 0.f});
    }

    // ... with the scales of the keys
    __device__ inline static void scaled(const float (&ks)[2], f32x4 (&s)[RB][2])
    {
        if constexpr (is_scaled(CT))
#pragma unroll
            for (int rb = 0; rb < RB; rb++) s[rb][0] *= ks[0], s[rb][1] *= ks[1];
    }

    // Brings m near the maximum of a tile's scores. It need not be the maximum
    // so far: the weights stay below 2^(kLift + kSlack) and nothing is lost in binary32,
    // while the output is scaled anew in the first tile and then hardly ever.
    // A row with a NaN is NaN by its sum, whatever m.
    // m c2 is rounded, and where a step of binary32 is a power of two the
    // weights would not be near 1 but anything, infinite in FP16: scores of
    // rows beyond 2^16 have m taken off, which is exact near it.
    __device__ inline void raise(float c2, f32x4 (&s)[RB][2])
    {
        float top[RB];
        bool any = false;
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            top[rb] = fmaxf(fmaxf(fmaxf(s[rb][0][0], s[rb][0][1]), fmaxf(s[rb][0][2], s[rb][0][3])),
                            fmaxf(fmaxf(s[rb][1][0], s[rb][1][1]), fmaxf(s[rb][1][2], s[rb][1][3])));
            if constexpr (!is_scaled(CT)) top[rb] = quad_max(top[rb]);
            any = any || (top[rb] - m[rb]) * c2 > kSlack;
        }
        if (__builtin_expect(__builtin_amdgcn_ballot_w64(any) != 0 || far, 0)) {
            far = false;
#pragma unroll
            for (int rb = 0; rb < RB; rb++) {
                if constexpr (is_scaled(CT)) top[rb] = quad_max(top[rb]);      // a row's lanes have to agree only here
                const float up = fmaxf(top[rb], m[rb]);
                const float a = __builtin_amdgcn_exp2f((m[rb] - (up == -INFINITY ? 0.f : up)) * c2);
                m[rb] = up;
                base[rb] = up == -INFINITY ? 0.f : fmaf(up, c2, -kLift);
                const bool off = fabsf(base[rb]) > 65536.f;
                far = far || __builtin_amdgcn_ballot_w64(off) != 0;
                if (off) s[rb][0] -= up, s[rb][1] -= up, base[rb] = -kLift;
                l[rb] *= a;
#pragma unroll
                for (int e = 0; e < NV; e++) acc[rb][e] *= a;
            }
        }
    }

    // Scores to weights, as the products with the values take them: with the values' scales.
    __device__ inline void weigh(float c2, const f32x4 (&s)[RB][2], const float (&vs)[2], u32x4 (&pw)[TERMS][RB])
    {
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            f32x4 w[2];
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int hf = 0; hf < 2; hf++)
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    w[hf][k] = __builtin_amdgcn_exp2f(fmaf(s[rb][hf][k], c2, -base[rb]));
                    sum[hf] += w[hf][k];
                }
            l[rb] += sum[0] + sum[1];
            if constexpr (is_scaled(CT)) w[0] *= vs[0], w[1] *= vs[1];
            // One term is a rounding to half a step of the products' type; the
            // sum was taken before it: lse keeps binary32. Of two the first is
            // cut off toward zero, so that the second is never negative, and
            // that is made kLeast at least where the weight is not less: an
            // infinite value times zero would be NaN, and infinities of both
            // signs too.
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float a = w[i >> 1][2 * (i & 1)], b = w[i >> 1][2 * (i & 1) + 1];
                if constexpr (FINE) {
                    pw[0][rb][i] = cut2<f16>(a, b);
                    const f32x2 had = unpack2<f16>(pw[0][rb][i]);
                    if constexpr (is_scaled(CT)) pw[1][rb][i] = pack2<f16>(a - had.x, b - had.y);      // no infinities there
                    else pw[1][rb][i] = pack2<f16>(__builtin_amdgcn_fmed3f(a - had.x, kLeast, a), __builtin_amdgcn_fmed3f(b - had.y, kLeast, b));
                } else {
                    pw[0][rb][i] = pack2<f16>(a, b);
                }
            }
        }
    }

    // element (c, e) of the lane's dims for its eight keys
    __device__ inline static u32x4 fragment(const Values (&v)[VC][8], int c, int e)
    {
        u32x4 a;
        if constexpr (is_scaled(CT)) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; k++) w[k] = v[c][k][e / 4];
            return turned_over<CT>(w, e % 4);
        }
#pragma unroll
        for (int k = 0; k < 4; k++) {
            if constexpr (is_byte(CT)) {
                const uint32_t sel = ((4u + e % 4) << 24) | (0x0cu << 16) | ((uint32_t)(e % 4) << 8) | 0x0cu;
                a[k] = __builtin_amdgcn_perm(v[c][2 * k + 1][e / 4], v[c][2 * k][e / 4], sel);
            } else {
                a[k] = __builtin_amdgcn_perm(v[c][2 * k + 1][e / 2], v[c][2 * k][e / 2], e % 2 ? 0x07060302u : 0x05040100u);
            }
        }
        return a;
    }

    __device__ inline void add(const Values (&v)[VC][8], const u32x4 (&pw)[TERMS][RB])
    {
#pragma unroll
        for (int c = 0; c < VC; c++)
#pragma unroll
            for (int e = 0; e < VE; e++) {
                const u32x4 a = fragment(v, c, e);
#pragma unroll
                for (int t = 0; t < TERMS; t++)
#pragma unroll
                    for (int rb = 0; rb < RB; rb++) acc[rb][c * VE + e] = mfma<f16>(a, pw[t][rb], acc[rb][c * VE + e]);
            }
    }

    // values of the lane's eight keys
    template <bool MASKED>
    __device__ inline void load_values(const AttendParams &p, const Tile &t, Values (&v)[VC][8])
    {
        const uint32_t off = (uint32_t)(g * 4 * p.c.vs1) + x * VE * es;
#pragma unroll
        for (int c = 0; c < VC; c++)
#pragma unroll
            for (int j = 0; j < 8; j++) {
                if (MASKED || PAD) v[c][j] = Values{};
                if ((!PAD || c * 128 + x * VE < p.D) && (!MASKED || (t.there[j >> 2] && t.key + 16 * (j >> 2) + 4 * g + (j & 3) < lim)))
                    v[c][j] = *reinterpret_cast<const Values *>(t.v[j >> 2] + (j & 3) * p.c.vs1 + (off + c * 128 * es));
            }
    }

    // Scores of keys that a row does not see become -inf, and the values' scale
    // of a half tile that no row sees 0: it may be anything, and a weight of
    // zero times it NaN.
    __device__ inline void hide(const AttendParams &p, const Tile &t, const Place &at, f32x4 (&s)[RB][2], float (&vs)[2])
    {
        uint32_t any = 0;
        const int n = at.n, nd = at.nd;
        uint32_t seen[RB];
#pragma unroll
        for (int rb = 0; rb < RB; rb++) seen[rb] = 0;
        if (p.tree && t.key + kTileKeys > n) {
#pragma unroll
            for (int rb = 0; rb < RB; rb++) seen[rb] = tree_bits(p, at.b, tok[rb], t.key + 4 * g - n, nd, at.end - n);
        }
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            seen[rb] |= leading_bits((p.tree ? n : min(lim, n + tok[rb] + 1)) - t.key - 4 * g);
            seen[rb] &= there_bits(t);
            any |= seen[rb];
#pragma unroll
            for (int i = 0; i < 8; i++) s[rb][i >> 2][i & 3] = seen[rb] >> i & 1 ? s[rb][i >> 2][i & 3] : -INFINITY;
        }
        if constexpr (is_scaled(CT))
#pragma unroll
            for (int x = 0; x < 2; x++) vs[x] = __builtin_amdgcn_ballot_w64((any >> 4 * x & 15) != 0) != 0 ? vs[x] : 0.f;
    }

    // One tile. values() is called for the values when the scores are done.
    // Not `fast`: one that not every row sees whole (the drafted tokens' own,
    // the last one, one with an absent page).
    template <typename F>
    __device__ inline void tile(const AttendParams &p, const Tile &t, const Place &at, const u32x4 (&k)[2][KS], Values (&v)[VC][8], F values)
    {
        const int n = at.n;
        f32x4 s[RB][2];
        u32x4 pw[TERMS][RB];
        score(k, s);
        scaled(t.ks, s);
        values(v);
        if constexpr (!is_scaled(CT)) settle(s);          // the scaled ones have been read above
        float vs[2] = {1.f, 1.f};
        if constexpr (is_scaled(CT)) vs[0] = t.vs[0], vs[1] = t.vs[1];
        if (!t.fast) hide(p, t, at, s, vs);
        raise(p.c2, s);
        weigh(p.c2, s, vs, pw);
        if (!is_i8(CT) && t.key + kTileKeys > n) {
            // A value that is not finite must reach only the rows that see its
            // key, and in a product it would reach all (0 * inf): poison() adds it.
            uint32_t any = 0;
#pragma unroll
            for (int c = 0; c < VC; c++)
#pragma unroll
                for (int j = 0; j < 8; j++)
#pragma unroll
                    for (int i = 0; i < VW; i++) {
                        const uint32_t bad = not_finite<CT>(v[c][j][i]);
                        any |= bad;
                        v[c][j][i] &= ~bad;
                    }
            odd = odd || __builtin_amdgcn_ballot_w64(any != 0) != 0;
        }
        add(v, pw);
    }

    // ... from the cache itself
    __device__ inline void masked_tile(const AttendParams &p, const Tile &t, const Place &at)
    {
        Raw<CT> kr[2][KS];
        u32x4 k[2][KS];
        Values v[VC][8];
        load_keys<CT, KS, PAD, true>(p, t, lim, x, g, (uint32_t)(x * p.c.ks1) + g * 8 * es, kr);
        constexpr bool together = RB * NV <= 16;          // registers for keys and values at once: one wait, not two
        if (together) load_values<true>(p, t, v);
#pragma unroll
        for (int hf = 0; hf < 2; hf++)
#pragma unroll
            for (int ks = 0; ks < KS; ks++) k[hf][ks] = widen<CT>(kr[hf][ks]);
        tile(p, t, at, k, v, [&](Values (&u)[VC][8]) {
            if (!together) load_values<true>(p, t, u);
        });
    }

    // After the last tile: whole sums, and maxima that waves can compare.
    __device__ inline void close(float c2)
    {
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            l[rb] = quad_sum(l[rb]);
            m[rb] = fmaf(m[rb], c2, -kLift);
        }
    }

    // Joins the wk (2 or 4) waves that split these rows' keys into the one
    // with wkey 0. wave0: the first of them; buf: join_words(waves) words for
    // all waves of the workgroup, which all call this; out: wk / 2 blocks of
    // RB * 16 * DP floats for these waves.
    static constexpr int join_words(int waves) { return (2 * RB * 16 + 1) * waves; }
    __device__ inline void join(int waves, int wk, int wkey, int wave0, float *buf, float *out)
    {
        const int lane = (int)(threadIdx.x & 63);
        if (g == 0)
#pragma unroll
            for (int rb = 0; rb < RB; rb++) {
                buf[((wave0 + wkey) * RB * 16 + rb * 16 + x) * 2] = m[rb];
                buf[((wave0 + wkey) * RB * 16 + rb * 16 + x) * 2 + 1] = l[rb];
            }
        int *flags = reinterpret_cast<int *>(buf + 2 * waves * RB * 16);
        if (lane == 0) flags[wave0 + wkey] = odd;
        __syncthreads();
        for (int k = 0; k < wk; k++) odd = odd || flags[wave0 + k];
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            const float *ml = buf + (wave0 * RB * 16 + rb * 16 + x) * 2;
            float top = -INFINITY, sum = 0.f;
            for (int k = 0; k < wk; k++) top = fmaxf(top, ml[k * RB * 32]);
            const float base = top == -INFINITY ? 0.f : top;
            for (int k = 0; k < wk; k++) sum += ml[k * RB * 32 + 1] * __builtin_amdgcn_exp2f(ml[k * RB * 32] - base);
            const float a = __builtin_amdgcn_exp2f(m[rb] - base);
            m[rb] = top;
            l[rb] = sum;
#pragma unroll
            for (int e = 0; e < NV; e++) acc[rb][e] *= a;
        }
        for (int step = wk >> 1; step; step >>= 1) {      // the upper half hands over to the lower
            float *at = out + (wkey & (step - 1)) * RB * 16 * DP + lane * 4;
            if (wkey >= step && wkey < 2 * step)
#pragma unroll
                for (int rb = 0; rb < RB; rb++)
#pragma unroll
                    for (int e = 0; e < NV; e++) *reinterpret_cast<f32x4 *>(at + (rb * NV + e) * 256) = acc[rb][e];
            __syncthreads();
            if (wkey < step)
#pragma unroll
                for (int rb = 0; rb < RB; rb++)
#pragma unroll
                    for (int e = 0; e < NV; e++) acc[rb][e] += *reinterpret_cast<const f32x4 *>(at + (rb * NV + e) * 256);
            __syncthreads();
        }
    }

    // What masked_tile left out: adds values that are not finite, among the
    // keys [lo, hi) of the drafted tokens' tiles, to the stored output of the
    // rows that see them, unless all their scores are -inf: those are zeros (of
    // a split row the join says so). Rare, and so written for few registers: a
    // lane goes over its own outputs, after store().
    __device__ inline void poison(const AttendParams &p, const Place &at)
    {
        const int b = at.b, h = at.h, n = at.n, nd = at.nd;
        const int lo = max(at.t0 * kTileKeys, n & ~(kTileKeys - 1)), hi = min(at.t1 * kTileKeys, at.end);
        uint32_t none = 0;
#pragma unroll
        for (int rb = 0; rb < RB; rb++) none |= at.whole && l[rb] == 0.f ? 1u << rb : 0;
        for (int rb = 0; rb < RB; rb++) {
            const int r = row0 + rb * 16 + x, token = r / p.G, head = h * p.G + r % p.G;
            if (r >= p.R || token >= nd || none >> rb & 1) continue;
            for (int i = 0; i < DP / 4; i++) {
                const int d = (i / (DP / VC / 4)) * 128 + g * 4 * VE + i % (DP / VC / 4);
                if (d >= p.D) continue;
                bool up = false, down = false;
                for (int key = lo; key < hi; key++) {
                    if (key >= n && !(p.tree ? p.tree[b * p.tr0 + token * p.tr1 + (key - n)] != 0 : key - n <= token)) continue;
                    int64_t off;
                    if (!locate(p.c, b, (uint32_t)key, p.c.vs0, p.c.vs1, off)) continue;
                    const char *from = p.c.v + off + h * p.c.vs2 + d * es;
                    const float v = is_scaled(CT) ? ((*reinterpret_cast<const uint8_t *>(from) & 0x7f) == 0x7f ? NAN : 0.f)
                                  : is_byte(CT) ? f16_to_f32((uint16_t)(*reinterpret_cast<const uint8_t *>(from) << 8))
                                                : CT == kBF16 ? bf16_to_f32(*reinterpret_cast<const uint16_t *>(from)) : f16_to_f32(*reinterpret_cast<const uint16_t *>(from));
                    if (fabsf(v) < INFINITY) continue;
                    up = up || !(v < 0.f);
                    down = down || !(v > 0.f);
                }
                if (!up && !down) continue;
                const float add = up && down ? NAN : up ? INFINITY : -INFINITY;
                if (!at.whole) {
                    p.part_o[((((int64_t)b * p.heads + h) * p.R + r) * p.nsplit + at.split) * DP + d] += add;
                } else {
                    uint16_t *o = reinterpret_cast<uint16_t *>(p.out + b * p.os0 + token * p.os1 + head * p.os2) + d;
                    const float sum = (half ? f16_to_f32(*o) : bf16_to_f32(*o)) + add;
                    *o = (uint16_t)(half ? pack2<true>(sum, 0.f) : pack2<false>(sum, 0.f));
                }
            }
        }
    }

    // The rows' output, or their part of it when the key axis is split.
    __device__ inline void store(const AttendParams &p, const Place &place)
    {
        const int b = place.b, h = place.h, nd = place.nd;
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            const int r = row0 + rb * 16 + x;
            if (r >= p.R) continue;
            if (!place.whole) {
                const int64_t at = (((int64_t)b * p.heads + h) * p.R + r) * p.nsplit + place.split;
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
            const bool empty = l[rb] == 0.f || tok[rb] >= nd;      // the weight of the row's maximum is at least 1, or NaN
            const float inv = 1.f / l[rb];
            const int head = h * p.G + r % p.G;
            if (g == 0 && p.lse) p.lse[((int64_t)b * p.T + tok[rb]) * (p.heads * p.G) + head] = empty ? -INFINITY : (m[rb] + __log2f(l[rb])) * 0.6931471805599453f;
            char *o = p.out + b * p.os0 + tok[rb] * p.os1 + head * p.os2;
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
};

// Few rows: bound by the cache's bytes. Waves work alone until they join, each
// on every wk-th tile; keys one tile ahead in registers, values loaded while
// the scores are worked out. One wave a SIMD at the larger head dims, two at
// the others, keep 32 KB a CU on their way and more. A chain of 4 tokens of 64
// heads over 2 x 131072 FP8 tokens of 8 heads of 128, 537 MB: 110 us, 4.9 TB/s
// (a copy of 1 GiB: 5.2); one token of 32 heads over 32 ragged sequences in
// pages: 103 us, 4.5 TB/s; one over 2048 tokens: 9.4 us, mostly the start of a
// launch and a first trip to memory.
// Weights go in two terms, which the matrix cores have the time for: BF16 rows
// of 128 over 2048 keys are off by 1.72e-3 of their norm, as if only the output
// were rounded, and by 2.22e-3 with one; in 14.9 us both. Not so the FP16
// weights of BF16 queries, three bits finer than the output: 1.689e-3 and
// 1.698e-3, in 130 and 120 us (2 x 4 tokens over 131072 FP8 keys).
// With scales: the same chain over 2 x 131072 tokens in 8-bit integers 105 us,
// 5.1 TB/s, the rate of a copy; 32 ragged sequences of up to 16384 E4M3 tokens
// in pages 116 us, 4.5 TB/s, where rows of a head are 128 bytes, 1 KB apart (side
// by side 104); one over 2048 tokens 11 us.
template <int CT, int DP, int RB, bool PAD, int SPLIT>
__global__ __launch_bounds__(kWaves * 64, DP == 256 ? 1 : 2) void k_attend(AttendParams p)
{
    using W = Rows<CT, DP, RB, PAD, CT != kE5M2BF>;
    constexpr int KS = W::KS;
    __shared__ float smem[2 * RB * 16 * DP + W::join_words(kWaves)];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wkey = wave & (p.wk - 1), wrow = wave / p.wk;
    const auto work = [&](const Place &at) {
        W w;
        w.init(p, at.b, at.h, (at.rg * (kWaves / p.wk) + wrow) * RB * 16, at.n, at.end);

        const int first = at.t0 + wkey, count = w.row0 < p.R ? (at.t1 - first + p.wk - 1) / p.wk : 0;
        int i = 0;
        if (count > 0) {
            const uint32_t koff = (uint32_t)(w.x * p.c.ks1) + w.g * 8 * W::es;
            Raw<CT> kr[2][KS];
            const auto next_of = [&](TileFinder<is_scaled(CT)> &finder, const Tile &t) {
                Tile nxt = t;
                nxt.fast = false;
                if (++i < count) {
                    const Tile f = finder.at(p, at.b, at.h, i, first, at.n, w.lim);
                    if (f.fast) nxt = f;
                }
                return nxt;
            };
            TileFinder<is_scaled(CT)> finder;
            Tile t = finder.at(p, at.b, at.h, 0, first, at.n, w.lim);
            if constexpr (is_scaled(CT)) {
                // The elements of a tile are few enough registers for all of the
                // next one to be under way: its keys once this one's are widened,
                // its values once this one's are multiplied.
                typename W::Values v[W::VC][8];
                if (t.fast) {
                    load_keys<CT, KS, PAD, false>(p, t, w.lim, w.x, w.g, koff, kr);
                    w.template load_values<false>(p, t, v);
                }
                while (t.fast) {
                    const Tile nxt = next_of(finder, t);
                    u32x4 k[2][KS];
                    hold(kr);
#pragma unroll
                    for (int hf = 0; hf < 2; hf++)
#pragma unroll
                        for (int ks = 0; ks < KS; ks++) k[hf][ks] = widen<CT>(kr[hf][ks]);
                    // before the products: no branch between them and the first
                    // use of the scores, and no wait of settle()
                    if (nxt.fast) load_keys<CT, KS, PAD, false>(p, nxt, w.lim, w.x, w.g, koff, kr);
                    f32x4 s[RB][2];
                    u32x4 pw[W::TERMS][RB];
                    w.score(k, s);
                    w.scaled(t.ks, s);
                    w.raise(p.c2, s);
                    w.weigh(p.c2, s, t.vs, pw);
                    hold(v);
                    w.add(v, pw);
                    if (nxt.fast) w.template load_values<false>(p, nxt, v);
                    t = nxt;
                }
            } else {
                if (t.fast) load_keys<CT, KS, PAD, false>(p, t, w.lim, w.x, w.g, koff, kr);
                while (t.fast) {
                    const Tile nxt = next_of(finder, t);
                    typename W::Values v[W::VC][8];
                    w.template load_values<false>(p, t, v);
                    u32x4 k[2][KS];
#pragma unroll
                    for (int hf = 0; hf < 2; hf++)
#pragma unroll
                        for (int ks = 0; ks < KS; ks++) k[hf][ks] = widen<CT>(kr[hf][ks]);
                    f32x4 s[RB][2];
                    u32x4 pw[W::TERMS][RB];
                    w.score(k, s);
                    if (nxt.fast) load_keys<CT, KS, PAD, false>(p, nxt, w.lim, w.x, w.g, koff, kr);
                    settle(s);
                    w.raise(p.c2, s);
                    w.weigh(p.c2, s, t.vs, pw);
                    w.add(v, pw);
                    t = nxt;
                }
            }
        }
        TileFinder<is_scaled(CT)> finder;
        for (; i < count; i++) {
            const Tile t = finder.at(p, at.b, at.h, i, first, at.n, w.lim);
            if (t.key >= w.lim) break;
            w.masked_tile(p, t, at);
        }

        w.close(p.c2);
        if (p.wk > 1) {
            w.join(kWaves, p.wk, wkey, wave - wkey, smem + 2 * RB * 16 * DP, smem + (p.wk == 4 ? 0 : wrow) * RB * 16 * DP);
            if (wkey) return;
        }
        w.store(p, at);
        if (w.odd) w.poison(p, at);
    };
    if constexpr (SPLIT == kRuns) {
        Place at;
        if (even_part(p, at)) work(at);
    } else if constexpr (SPLIT == kWalks) {
        Walk walk(p, true);
        walk.uniform();
        Place at;
        while (walk.next(p, at)) {
            at.uniform();
            work(at);
        }
    } else {
        const Place at = part_of_sequence(p);
        if (at.split && at.t0 >= at.t1) return;
        work(at);
    }
}

// Many rows: bound by the matrix cores and the exponentials. Eight waves of 32
// rows each, two on a SIMD so that one's products run beside the other's
// exponentials, read keys and values from LDS. A workgroup keeps a ring of
// stages of 64 keys there. All but two are under way, one being worked on and
// one just done with: a stage is worked on in less than half the time memory
// takes to answer, so that it is the bytes under way that keep the matrix cores
// fed (two stages of 32 KB of 16-bit heads of 128, six of 16 KB of half that,
// six of 8 KB of FP8 heads of 64). They go from memory to LDS without passing
// registers. Every wave's rows go over all of the workgroup's stages, also
// those of a chain's tokens that they do not see: their products are left out,
// their loads are not.
// Trees of 64 tokens of 64 heads over 8 ragged sequences of up to 4109 keys of
// 128: 91 us, of which 28 are the products at the rate of a large matrix
// product; a place begins in 9 us and ends in 4, and a stage takes 3. The
// matrix cores are busy for 20 % of the time and the vector units for 45, with
// permutes, maxima and moves (one vector instruction of 17 is an exponential);
// waves wait a third of it for loads and barriers, and a third to issue.
//
// A row is kept in 16-byte pieces, piece c of row r at place c ^ mixed(r), so
// that what 16 lanes read at once lies on all 64 banks; a load writes 64 places
// in order, so it is the source that is mixed.
// wk == 1: every wave takes both tiles of a stage; wk == 2: pairs of waves
// share rows and take one each.
//
// Weights go in one term here, rounded to half a step: the trees above take 118
// us with two, 105 with one, and are off by 1.68e-3 and 2.08e-3 of their norm;
// 32 FP16 rows' weights over 4 x 16384 keys 102 and 91 us, 2.16e-4 and 2.41e-4.
constexpr int kShared = 8;                        // waves

// A 16-byte read takes lanes {0-3, 12-15, 20-27}, then {4-11, 16-19, 28-31} and
// the same of the upper half. Keys: lane (x, g) reads piece 4 ks + g of row x;
// values: piece x of row 4 g + j. With 16 pieces a row fills the banks, and
// both are free of conflicts if flipping bit 2 of a row flips the upper two
// bits of the mix (measured: row & 7 doubles the time of every read). With 8
// pieces, two rows fill the banks, and a row's low bits do.
template <int PIECES>
__device__ constexpr int mixed(int row)
{
    return PIECES == 16 ? (row & 15) ^ (row & 4) << 1 : row & (PIECES < 8 ? PIECES - 1 : 7);
}

__device__ const u32x4 kZeros[1] = {};            // what dims behind the head's own are read from

template <int CT, int DP, bool PAD, bool PAGED>
__global__ __launch_bounds__(kShared * 64, 2) void k_attend_shared(AttendParams p)
{
    constexpr int RB = 2;
    using W = Rows<CT, DP, RB, PAD, false>;
    constexpr int KS = W::KS, es = W::es, ROW = DP * es, PIECES = ROW / 16;
    constexpr int LOADS = 2 * 64 * ROW / (kShared * 64 * 16);      // 16-byte pieces a thread loads a stage
    constexpr int STAGE = 2 * 64 * ROW, RING = ROW == 256 ? 4 : 8;
    static_assert(RING * STAGE >= 4 * RB * 16 * DP * 4, "the waves' outputs are joined in the ring");
    __shared__ __attribute__((aligned(16))) char smem[RING * STAGE + W::join_words(kShared) * 4];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wkey = wave & (p.wk - 1), wrow = wave / p.wk;
    Walk walk(p);
    Place at;
    while (walk.next(p, at)) {
        int tid = (int)threadIdx.x;
        asm volatile("" : "+v"(tid));
        __syncthreads();                              // the ring is free

        // Stages of 64 keys, the first `fast` of them all cached tokens, which
        // every row sees; in pages, up to the first that touches an absent one.
        const int key0 = at.t0 * kTileKeys, stages = (at.t1 - at.t0 + 1) / 2;
        int fast = min((at.t1 - at.t0) / 2, max(at.n - key0, 0) / 64);
        if constexpr (PAGED) {
            const int lane = tid & 63;
            for (int i = 0; i < fast * 4; i += 64) {
                const bool bad = i + lane < fast * 4 && (uint32_t)p.c.table[at.b * p.c.ts + ((key0 + (i + lane) * 16) >> p.c.shift)] >= p.c.pages;
                const uint64_t any = __builtin_amdgcn_ballot_w64(bad);
                if (any) fast = (i + __builtin_ctzll(any)) / 4;
            }
        }
        // A thread's place `lin` of load j: the keys' 64 rows, then the values'. A
        // wave's 64 places lie in one half tile, so that a page is looked up once.
        const char *src[LOADS];
        bool pad[LOADS];
    #pragma unroll
        for (int j = 0; j < LOADS; j++) {
            const int lin0 = j * kShared * 64 + wave * 64, lin = lin0 + (tid & 63);
            const bool val = lin0 >= 64 * PIECES;
            const int row = (lin / PIECES) & 63, piece = lin % PIECES ^ mixed<PIECES>(row);
            const int64_t step = val ? p.c.vs1 : p.c.ks1;
            src[j] = (val ? p.c.v + at.h * p.c.vs2 : p.c.k + at.h * p.c.ks2) + piece * 16 + (PAGED ? (row & 15) * step : at.b * (val ? p.c.vs0 : p.c.ks0) + (key0 + row) * step);
            if (PAD) pad[j] = piece * 16 >= p.D * es;
        }
        int entry = 0;
        const auto issue = [&](int i) {
            char *to = smem + i % RING * STAGE + wave * 1024;
            // page numbers of the next 64 half tiles, one a lane; -1 behind the
            // last token. The wait for them is one for the stages under way too.
            if (PAGED && (i & 15) == 0) {
                const int key = key0 + (i * 4 + (tid & 63)) * 16;
                entry = key < at.end ? p.c.table[at.b * p.c.ts + (key >> p.c.shift)] : -1;
                __builtin_amdgcn_s_waitcnt(0x0f70);
            }
    #pragma unroll
            for (int j = 0; j < LOADS; j++) {
                const int lin0 = j * kShared * 64 + wave * 64;
                const bool val = lin0 >= 64 * PIECES;
                const int64_t step = val ? p.c.vs1 : p.c.ks1;
                const char *from = src[j];
                if constexpr (PAGED) {
                    const int half = (lin0 / PIECES & 63) >> 4;
                    const uint32_t page = (uint32_t)__builtin_amdgcn_readlane(entry, (i & 15) * 4 + half);
                    const uint32_t in = (uint32_t)(key0 + i * 64 + half * 16) & ((1u << p.c.shift) - 1);
                    from += (int64_t)page * (val ? p.c.vs0 : p.c.ks0) + (int64_t)in * step;
                    if (page >= p.c.pages) from = reinterpret_cast<const char *>(kZeros);
                } else {
                    // behind the last token the last one again, which the mask leaves out
                    if (i >= fast) from -= max(key0 + i * 64 + ((lin0 + (tid & 63)) / PIECES & 63) - (at.end - 1), 0) * step;
                    src[j] += 64 * step;
                }
                if (PAD && pad[j]) from = reinterpret_cast<const char *>(kZeros);
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                                 (__attribute__((address_space(3))) void *)(to + j * kShared * 1024), 16, 0, 0);
            }
        };
        // The queries are waited for here: a wait for them inside the loop would be
        // one for every stage under way. The first stages arrive meanwhile.
        int issued = 0;
        while (issued < RING - 2 && issued < stages) issue(issued++);
        W w;
        w.init(p, at.b, at.h, (at.rg * (kShared / p.wk) + wrow) * RB * 16, at.n, at.end);
        __builtin_amdgcn_s_waitcnt(0x0f70);
        const auto keys_of = [&](const char *stage, int tile, u32x4 (&k)[2][KS]) {
            const char *kb = stage + (tile * 32 + w.x) * ROW;
    #pragma unroll
            for (int hf = 0; hf < 2; hf++)
    #pragma unroll
                for (int ks = 0; ks < KS; ks++) {
                    const int o = (ks * 32 + w.g * 8) * es;
                    k[hf][ks] = widen<CT>(*reinterpret_cast<const Raw<CT> *>(kb + hf * 16 * ROW + ((((o >> 4) ^ mixed<PIECES>(w.x)) << 4) | (o & 15))));
                }
        };
        const auto values_of = [&](const char *stage, int tile, typename W::Values (&v)[W::VC][8]) {
            const char *vb = stage + (64 + tile * 32 + w.g * 4) * ROW;
    #pragma unroll
            for (int j = 0; j < 8; j++) {
                const int o = w.x * W::VE * es, mix = mixed<PIECES>(w.g * 4 + (j & 3));
                v[0][j] = *reinterpret_cast<const typename W::Values *>(vb + ((j >> 2) * 16 + (j & 3)) * ROW + ((((o >> 4) ^ mix) << 4) | (o & 15)));
            }
        };

        // Makes stage i readable and starts the load of a later one. This wave's
        // loads of it are done when no more than the later stages' are outstanding
        // (they end in order); other loads in between make the wait longer, never
        // shorter. Behind the barrier all waves' are, and all are past the values
        // of stage i - 2, whose place is free.
        const auto enter = [&](int i) {
            if (issued - i == RING - 2) __builtin_amdgcn_s_waitcnt(0x0f70 | ((RING - 3) * LOADS & 15) | ((RING - 3) * LOADS >> 4) << 14);
            else __builtin_amdgcn_s_waitcnt(0x0f70);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (issued < stages) issue(issued++);
        };
        // One tile's weights and output beside the next tile's scores: a wave's
        // exponentials run while its own products do (64 rows over 16384 keys: 379
        // against 395 us without).
        const bool rows = w.row0 < p.R;               // else this wave only loads
        if (fast > 0) {
            f32x4 s[RB][2];
            const auto step = [&](const char *stage, int tile, const char *next_stage, int next_tile) {
                typename W::Values v[W::VC][8];
                u32x4 k[2][KS], pw[W::TERMS][RB];
                f32x4 next[RB][2];
                const float none[2] = {1.f, 1.f};     // no scales
                keys_of(next_stage, next_tile, k);
                values_of(stage, tile, v);
                w.weigh(p.c2, s, none, pw);
                w.score(k, next);
                w.add(v, pw);
    #pragma unroll
                for (int rb = 0; rb < RB; rb++)
    #pragma unroll
                    for (int hf = 0; hf < 2; hf++) s[rb][hf] = next[rb][hf];
                w.raise(p.c2, s);
            };
            enter(0);
            if (rows) {
                u32x4 k[2][KS];
                keys_of(smem, p.wk == 1 ? 0 : wkey, k);
                w.score(k, s);
                w.raise(p.c2, s);
            }
            for (int i = 0; i < fast; i++) {
                const char *stage = smem + i % RING * STAGE, *next = i + 1 < fast ? smem + (i + 1) % RING * STAGE : stage;
                // after the last tile its own scores again, which change nothing
                if (p.wk == 1 && rows) step(stage, 0, stage, 1);
                if (i + 1 < fast) enter(i + 1);
                if (rows) step(stage, p.wk == 1 ? 1 : wkey, next, p.wk == 1 ? 0 : wkey);
            }
        }
        for (int i = fast; i < stages; i++) {
            enter(i);
            const char *stage = smem + i % RING * STAGE;
            for (int tile = wkey; tile < 2; tile += p.wk) {
                Tile t;
                t.key = key0 + i * 64 + tile * kTileKeys;
                t.fast = false;
                if (!rows || t.key >= w.lim) break;
    #pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    const int key = t.key + 16 * hf;
                    t.there[hf] = key < at.end && (!PAGED || (uint32_t)p.c.table[at.b * p.c.ts + (key >> p.c.shift)] < p.c.pages);
                }
                u32x4 k[2][KS];
                typename W::Values v[W::VC][8];
                keys_of(stage, tile, k);
                w.tile(p, t, at, k, v, [&](typename W::Values (&u)[W::VC][8]) { values_of(stage, tile, u); });
            }
        }
        w.close(p.c2);
        if (p.wk == 2) {
            __syncthreads();                          // the ring's memory is free
            w.join(kShared, 2, wkey, wave - wkey, reinterpret_cast<float *>(smem + RING * STAGE), reinterpret_cast<float *>(smem) + wrow * RB * 16 * DP);
            if (wkey) continue;
        }
        w.store(p, at);
        if (w.odd) w.poison(p, at);
    }
}

// The same for 8 bits with scales, whose elements take longer to widen than to
// multiply: a workgroup does it once for all its waves. Threads read the
// elements of the stage after the next into registers, and write those of the
// next one to LDS in 16 bits, keys in rows as above, values as the matrix cores
// take them: for dim e of each lane's, the 16 bytes of all 64 lanes in order.
// So a stage is read from one of three places while the next one fills another,
// with one barrier a stage. Half the waves widen values, right behind it, half
// keys, a tile later, so that the two waves of a SIMD are not at the same thing.
// Trees of 64 tokens of 64 FP16 heads over 8 ragged sequences of up to 8205 E4M3
// keys of 128: 199 us under the profiler, with every wave widening for itself 277,
// with all of them widening at once 10 more, with values read from LDS where they
// are used 8 more (keys read two fragments at a time, 3 more). The products, in
// two terms, are 43 us at the dense peak; the vector units are busy for 57 % of
// the time, the matrix cores for 38.
template <int CT, int DP, bool PAD, bool PAGED>
__global__ __launch_bounds__(kShared * 64, 2) void k_attend_wide(AttendParams p)
{
    constexpr int RB = 2;
    // Two terms of a weight, as with few rows: it is BF16 beside scales, and one
    // would be as coarse as a BF16 output and save 4 to 6 %
    using W = Rows<CT, DP, RB, PAD, true>;
    constexpr int KS = W::KS, VE = W::VE, ROW = DP * 2, PIECES = ROW / 16;
    constexpr int TILE = DP * 64, STAGE = 64 * ROW + 2 * TILE, RING = 3;      // a tile's values, and bytes of a stage
    constexpr int UNITS = DP / 64;                // of 16 elements of keys, a thread
    static_assert(RING * STAGE >= 4 * RB * 16 * DP * 4, "the waves' outputs are joined in the ring");
    __shared__ __attribute__((aligned(16))) char smem[RING * STAGE + W::join_words(kShared) * 4];
    __shared__ float lscale[RING * 8];            // of the four half tiles, the keys' and the values'
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wkey = wave & (p.wk - 1), wrow = wave / p.wk;
    Walk walk(p);
    walk.uniform();
    Place at;
    while (walk.next(p, at)) {
        at.uniform();
        int tid = (int)threadIdx.x;
        asm volatile("" : "+v"(tid));
        __syncthreads();                              // the ring is free

        // Stages of 64 keys, the first `fast` of them all cached tokens, which
        // every row sees; in pages, up to the first that touches an absent one.
        const int key0 = at.t0 * kTileKeys, stages = (at.t1 - at.t0 + 1) / 2;
        int fast = min((at.t1 - at.t0) / 2, max(at.n - key0, 0) / 64);
        if constexpr (PAGED) {
            const int lane = tid & 63;
            for (int i = 0; i < fast * 4; i += 64) {
                const bool bad = i + lane < fast * 4 && (uint32_t)p.c.table[at.b * p.c.ts + ((key0 + (i + lane) * 16) >> p.c.shift)] >= p.c.pages;
                const uint64_t any = __builtin_amdgcn_ballot_w64(bad);
                if (any) fast = (i + __builtin_ctzll(any)) / 4;
            }
        }
        // What a thread reads of a stage. Values: 4 dims of the eight keys of a
        // lane; keys: 16 elements of a row, UNITS times. first[]: their keys'
        // numbers in the stage, two of which may lie in different pages.
        const bool val = wave < kShared / 2, some = !val || tid < 2 * DP;
        const int quad = tid % (DP / 4), vg = tid / (DP / 4) & 3, vtile = tid / DP & 1;
        int row[2];
#pragma unroll
        for (int j = 0; j < 2; j++) row[j] = val ? vtile * 32 + j * 16 + 4 * vg : ((tid & 255) + j * 256) / (DP / 16) & 63;
        const int chunk = (tid & 255) % (DP / 16);
        const bool pad = PAD && (val ? quad * 4 : chunk * 16) >= p.D;
        const char *base = (val ? p.c.v + at.h * p.c.vs2 + quad * 4 : p.c.k + at.h * p.c.ks2 + chunk * 16) + (PAGED ? 0 : at.b * (val ? p.c.vs0 : p.c.ks0));
        const int64_t step1 = val ? p.c.vs1 : p.c.ks1, step0 = val ? p.c.vs0 : p.c.ks0;
        const int shalf = tid & 3;                    // threads 0 to 7: a half tile's scale, of values from 4 on
        uint32_t raw[8], page[2] = {0, 0}, spage = 0;
        float sraw = 0.f;
        const auto look_up = [&](int i) {             // pages of a stage
            if constexpr (PAGED) {
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int key = key0 + i * 64 + row[j];
                    page[j] = key < at.end ? (uint32_t)p.c.table[at.b * p.c.ts + (key >> p.c.shift)] : ~0u;
                }
                if (tid < 8) {
                    const int key = key0 + i * 64 + shalf * 16;
                    spage = key < at.end ? (uint32_t)p.c.table[at.b * p.c.ts + (key >> p.c.shift)] : ~0u;
                }
            }
        };
        const auto fetch = [&](int i) {
#pragma unroll
            for (int r = 0; r < 8; r++) raw[r] = 0;
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int key = key0 + i * 64 + row[j];
                const bool there = some && !pad && (!PAGED || page[j] < p.c.pages);
                const int64_t in = PAGED ? key & ((1 << p.c.shift) - 1) : key;
                const char *from = base + (PAGED ? (int64_t)page[j] * step0 : 0) + in * step1;
                if (val) {
#pragma unroll
                    for (int r = 0; r < 4; r++)
                        if (there && key + r < at.end) raw[j * 4 + r] = *reinterpret_cast<const uint32_t *>(from + r * step1);
                } else if (j < UNITS && there && key < at.end) {
                    const u32x4 w = *reinterpret_cast<const u32x4 *>(from);
#pragma unroll
                    for (int r = 0; r < 4; r++) raw[j * 4 + r] = w[r];
                }
            }
            if (tid < 8) {
                const int key = key0 + i * 64 + shalf * 16;
                const uint32_t from = PAGED ? spage : (uint32_t)at.b;
                const uint32_t block = (uint32_t)(PAGED ? key & ((1 << p.c.shift) - 1) : key) >> p.scales.shift;
                sraw = 0.f;
                if (key < at.end && (!PAGED || spage < p.c.pages))
                    sraw = tid & 4 ? p.scales.v[from * p.scales.v0 + block * p.scales.v1 + (uint32_t)at.h * p.scales.v2]
                                   : p.scales.k[from * p.scales.k0 + block * p.scales.k1 + (uint32_t)at.h * p.scales.k2];
            }
            if (i + 1 < stages) look_up(i + 1);
        };
        const auto put = [&](int i) {
            char *stage = smem + i % RING * STAGE;
            if (val) {
                if (some)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int d = quad * 4 + e;
                        *reinterpret_cast<u32x4 *>(stage + 64 * ROW + vtile * TILE + d % VE * 1024 + vg * 256 + d / VE * 16) = turned_over<CT>(raw, e);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < UNITS; j++)
#pragma unroll
                    for (int k = 0; k < 2; k++)
                        *reinterpret_cast<u32x4 *>(stage + row[j] * ROW + (((2 * chunk + k) ^ mixed<PIECES>(row[j])) << 4)) =
                            widen<CT>(Raw<CT>{raw[j * 4 + 2 * k], raw[j * 4 + 2 * k + 1]});
            }
            if (tid < 8) lscale[i % RING * 8 + tid] = sraw;
        };
        look_up(0);
        fetch(0);
        W w;
        w.init(p, at.b, at.h, (at.rg * (kShared / p.wk) + wrow) * RB * 16, at.n, at.end);
        put(0);
        if (stages > 1) fetch(1);
        // Behind the barrier all waves have written stage i, and none reads stage
        // i - 2 any more, whose place is that of i + 1.
        const auto refill = [&](int i) {
            if (i + 1 < stages) put(i + 1);
            if (i + 2 < stages) fetch(i + 2);
        };
        const auto enter = [&](int i, bool whole) {
            __syncthreads();
            if (val || whole) refill(i);
        };
        const auto keys_of = [&](int i, int tile, u32x4 (&k)[2][KS], float (&ks)[2]) {
            const char *kb = smem + i % RING * STAGE + (tile * 32 + w.x) * ROW;
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
#pragma unroll
                for (int kk = 0; kk < KS; kk++)
                    k[hf][kk] = *reinterpret_cast<const u32x4 *>(kb + hf * 16 * ROW + (((kk * 4 + w.g) ^ mixed<PIECES>(w.x)) << 4));
                ks[hf] = lscale[i % RING * 8 + tile * 2 + hf];
            }
        };
        const auto scales_of = [&](int i, int tile, float (&vs)[2]) {
#pragma unroll
            for (int hf = 0; hf < 2; hf++) vs[hf] = lscale[i % RING * 8 + 4 + tile * 2 + hf];
        };
        // Products with the values, two dims of a lane's at a time, the next two on
        // their way from LDS meanwhile; the first two are read by ready(), before
        // what else there is to do. check: those that are not finite are left to
        // poison().
        u32x4 two[2][2];
        const auto read_two = [&](int i, int tile, int e) {
            const char *vb = smem + i % RING * STAGE + 64 * ROW + tile * TILE + w.g * 256 + w.x * 16;
#pragma unroll
            for (int k = 0; k < 2; k++) two[e / 2 & 1][k] = *reinterpret_cast<const u32x4 *>(vb + (e + k) * 1024);
        };
        const auto ready = [&](int i, int tile) { read_two(i, tile, 0); };
        const auto add = [&](int i, int tile, const u32x4 (&pw)[W::TERMS][RB], bool check) {
            uint32_t any = 0;
#pragma unroll
            for (int e = 0; e < VE; e += 2) {
                if (e + 2 < VE) {
                    read_two(i, tile, e + 2);
                    __builtin_amdgcn_sched_barrier(0);        // not moved down to where they are used
                }
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    u32x4 a = two[e / 2 & 1][j];
                    if (!is_i8(CT) && check)
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const uint32_t bad = not_finite<kBF16>(a[k]);
                            any |= bad;
                            a[k] &= ~bad;
                        }
#pragma unroll
                    for (int t = 0; t < W::TERMS; t++)
#pragma unroll
                        for (int rb = 0; rb < RB; rb++) w.acc[rb][e + j] = mfma<false>(a, pw[t][rb], w.acc[rb][e + j]);
                }
            }
            if (check) w.odd = w.odd || __builtin_amdgcn_ballot_w64(any != 0) != 0;
        };
        // One tile's weights and output beside the next tile's scores.
        const bool rows = w.row0 < p.R;               // else this wave only widens
        if (fast > 0) {
            f32x4 s[RB][2];
            const auto step = [&](int i, int tile, int next_i, int next_tile) {
                u32x4 k[2][KS], pw[W::TERMS][RB];
                f32x4 next[RB][2];
                float ks[2], vs[2];
                scales_of(i, tile, vs);
                keys_of(next_i, next_tile, k, ks);
                w.weigh(p.c2, s, vs, pw);
                ready(i, tile);
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(1);
                w.score(k, next);
                w.scaled(ks, next);
                add(i, tile, pw, false);
                __builtin_amdgcn_s_setprio(0);
#pragma unroll
                for (int rb = 0; rb < RB; rb++)
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) s[rb][hf] = next[rb][hf];
                w.raise(p.c2, s);
            };
            enter(0, true);
            if (rows) {
                u32x4 k[2][KS];
                float ks[2];
                keys_of(0, p.wk == 1 ? 0 : wkey, k, ks);
                w.score(k, s);
                w.scaled(ks, s);
                w.raise(p.c2, s);
            }
            for (int i = 0; i < fast; i++) {
                // after the last tile its own scores again, which change nothing
                if (p.wk == 1 && rows) step(i, 0, i, 1);
                if (i + 1 < fast) enter(i + 1, false);
                if (rows) step(i, p.wk == 1 ? 1 : wkey, i + 1 < fast ? i + 1 : i, i + 1 < fast ? p.wk == 1 ? 0 : wkey : p.wk == 1 ? 1 : wkey);
                if (i + 1 < fast && !val) refill(i + 1);
            }
        }
        for (int i = fast; i < stages; i++) {
            enter(i, true);
            for (int tile = wkey; tile < 2; tile += p.wk) {
                Tile t;
                t.key = key0 + i * 64 + tile * kTileKeys;
                t.fast = false;
                if (!rows || t.key >= w.lim) break;
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    const int key = t.key + 16 * hf;
                    t.there[hf] = key < at.end && (!PAGED || (uint32_t)p.c.table[at.b * p.c.ts + (key >> p.c.shift)] < p.c.pages);
                }
                u32x4 k[2][KS], pw[W::TERMS][RB];
                f32x4 s[RB][2];
                keys_of(i, tile, k, t.ks);
                scales_of(i, tile, t.vs);
                w.score(k, s);
                w.scaled(t.ks, s);
                w.hide(p, t, at, s, t.vs);
                w.raise(p.c2, s);
                w.weigh(p.c2, s, t.vs, pw);
                ready(i, tile);
                add(i, tile, pw, t.key + kTileKeys > at.n);
            }
        }
        w.close(p.c2);
        if (p.wk == 2) {
            __syncthreads();                          // the ring's memory is free
            w.join(kShared, 2, wkey, wave - wkey, reinterpret_cast<float *>(smem + RING * STAGE), reinterpret_cast<float *>(smem) + wrow * RB * 16 * DP);
            if (wkey) continue;
        }
        w.store(p, at);
        if (w.odd) w.poison(p, at);
    }
}

// Joins a row's splits. Few of them: 16 lanes a row, one split a lane to weigh
// and then DP / 16 dims a lane; a row's loads are few and wait for each other,
// so rows must run side by side. Many: a workgroup a row, below.
struct Joined {
    int b, h, tok, head, nd, used;

    __device__ inline Joined(const AttendParams &p, int64_t row)      // ((b * heads) + h) * R + r
    {
        const int r = (int)(row % p.R);
        h = (int)(row / p.R % p.heads), b = (int)(row / p.R / p.heads);
        nd = clamp_drafted(p.drafted, b, p.T);
        const int tiles = tiles_of(p, b), each = tiles_per_split(p, tiles);
        used = p.flat ? p.used[b] : max((tiles + each - 1) / each, 1);
        tok = r / p.G, head = h * p.G + r % p.G;
    }

    __device__ inline bool empty(float sum) const { return sum == 0.f || tok >= nd; }
    __device__ inline char *out(const AttendParams &p) const { return p.out + b * p.os0 + tok * p.os1 + head * p.os2; }
    __device__ inline void put_lse(const AttendParams &p, float top, float sum) const
    {
        if (p.lse) p.lse[((int64_t)b * p.T + tok) * (p.heads * p.G) + head] = empty(sum) ? -INFINITY : (top + __log2f(sum)) * 0.6931471805599453f;
    }
};

template <int DP>
__global__ __launch_bounds__(256) void k_attend_join_few(AttendParams p, int64_t rows, int half)
{
    constexpr int E = DP / 64;                    // 16-byte pieces a lane, 64 dims apart
    const int x = (int)(threadIdx.x & 15);
    const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    if (row >= rows) return;
    const Joined j(p, row);
    if (j.used == 1) return;                      // whole already
    const float *po = p.part_o + row * p.nsplit * DP + x * 4;
    const float2 *ml = p.part_ml + row * p.nsplit;
    f32x4 v[2][E];                                // two splits ahead
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
        for (int e = 0; e < E; e++) v[u][e] = u < j.used ? *reinterpret_cast<const f32x4 *>(po + u * DP + e * 64) : f32x4{0.f, 0.f, 0.f, 0.f};
    float top = -INFINITY;
    for (int k = x; k < j.used; k += 16) top = fmaxf(top, ml[k].x);
    for (int y = 1; y < 16; y <<= 1) top = fmaxf(top, __shfl_xor(top, y));
    float sum = 0.f;
    f32x4 o[E] = {};
    for (int k0 = 0; k0 < j.used; k0 += 16) {
        const float2 mine = k0 + x < j.used ? ml[k0 + x] : make_float2(-INFINITY, 0.f);
        const float a = __builtin_amdgcn_exp2f(mine.x - (top == -INFINITY ? 0.f : top));
        sum += mine.y * a;
        for (int k = k0; k < min(j.used, k0 + 16); k += 2)
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const float w = __shfl(a, (int)(threadIdx.x & 48) + ((k + u) & 15));
#pragma unroll
                for (int e = 0; e < E; e++) {
                    if (k + u < j.used) o[e] += v[u][e] * w;
                    if (k + u + 2 < j.used) v[u][e] = *reinterpret_cast<const f32x4 *>(po + (k + u + 2) * DP + e * 64);
                }
            }
    }
    for (int y = 1; y < 16; y <<= 1) sum += __shfl_xor(sum, y);
    if (x == 0) j.put_lse(p, top, sum);
    const bool empty = j.empty(sum);
    const float inv = 1.f / sum;
#pragma unroll
    for (int e = 0; e < E; e++) {
        if (x * 4 + e * 64 >= p.D) continue;
        float r[4];
#pragma unroll
        for (int i = 0; i < 4; i++) r[i] = empty ? 0.f : o[e][i] * inv;
        *reinterpret_cast<u32x2 *>(j.out(p) + (x * 4 + e * 64) * 2) =
            half ? u32x2{pack2<true>(r[0], r[1]), pack2<true>(r[2], r[3])} : u32x2{pack2<false>(r[0], r[1]), pack2<false>(r[2], r[3])};
    }
}

template <int DP>
__global__ __launch_bounds__(kWaves * 64) void k_attend_join_many(AttendParams p, int half)
{
    constexpr int E = DP / 64, U = 8;             // dims a lane, splits whose loads are under way together
    typedef float fe __attribute__((ext_vector_type(E)));
    __shared__ __attribute__((aligned(16))) float so[kWaves][DP];
    const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
    const int64_t row = blockIdx.x;
    const Joined j(p, row);
    if (j.used == 1) return;
    const float2 *ml = p.part_ml + row * p.nsplit;
    const float *po = p.part_o + row * p.nsplit * DP + lane * E;

    float top = -INFINITY;
    for (int k = lane; k < j.used; k += 64) top = fmaxf(top, ml[k].x);
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int k = lane; k < j.used; k += 64) sum += ml[k].y * __builtin_amdgcn_exp2f(ml[k].x - base);
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);

    fe o = {};
    for (int k0 = wave; k0 < j.used; k0 += kWaves * U) {
        fe v[U];
        float a[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int k = min(k0 + u * kWaves, j.used - 1);
            a[u] = ml[k].x;
            if constexpr (E == 1) v[u][0] = po[(int64_t)k * DP];
            else v[u] = *reinterpret_cast<const fe *>(po + (int64_t)k * DP);
        }
#pragma unroll
        for (int u = 0; u < U; u++)
            if (k0 + u * kWaves < j.used) o += v[u] * __builtin_amdgcn_exp2f(a[u] - base);
    }
    if constexpr (E == 1) so[wave][lane] = o[0];
    else *reinterpret_cast<fe *>(&so[wave][lane * E]) = o;
    __syncthreads();
    if (threadIdx.x == 0) j.put_lse(p, top, sum);
    const int d = 2 * (int)threadIdx.x;
    if (d >= p.D) return;
    const bool empty = j.empty(sum);
    const float inv = 1.f / sum;
    const float u = empty ? 0.f : (so[0][d] + so[1][d] + so[2][d] + so[3][d]) * inv;
    const float v = empty ? 0.f : (so[0][d + 1] + so[1][d + 1] + so[2][d + 1] + so[3][d + 1]) * inv;
    *reinterpret_cast<uint32_t *>(j.out(p) + d * 2) = half ? pack2<true>(u, v) : pack2<false>(u, v);
}

// score[key] += sum over a kv head's rows of exp(s - lse). With the rows' lse
// known, a wave owns 32 keys at a time, keeps them in registers and passes over
// the rows: no atomics, each sum in one fixed order. The products are those of
// k_attend, bit for bit. A workgroup has its rows in LDS, as the matrix cores
// take them, for p.weigh_tiles tiles of each wave; read from memory for every
// tile they took twice the time (32 tokens of 32 heads over 4 x 16384 keys of
// 64: 30 and 50 us). Bound by vector instructions, busy for 76 % of that; the
// matrix cores are for 13, LDS for 12.
template <int CT, int DP, bool PAD>
__global__ __launch_bounds__(kWaves * 64, 2) void k_attend_weigh(AttendParams p)
{
    constexpr int KS = DP / 32;
    constexpr int es = is_byte(CT) ? 1 : 2;
    constexpr int BLOCKS = KS <= 4 ? 16 : 8;      // of 16 rows, at a time
    __shared__ __attribute__((aligned(16))) u32x4 lq[BLOCKS * KS * 64];
    __shared__ float lrow[BLOCKS * 16];           // lse * log2(e); +inf: takes no part
    const int lane = (int)(threadIdx.x & 63), x = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    int id = (int)blockIdx.x;
    const int h = id % p.heads;
    id /= p.heads;
    const int each = kWaves * p.weigh_tiles, per = (int)(((p.c.tokens + kTileKeys - 1) / kTileKeys + each - 1) / each);
    const int first = id % per * each, b = id / per;
    const int n = __builtin_amdgcn_readfirstlane(clamp_length(p.length, b, p.c.tokens));
    const int nd = __builtin_amdgcn_readfirstlane(clamp_drafted(p.drafted, b, p.T));
    const int end = end_of(p, n, nd), rows = nd * p.G;
    if (first * kTileKeys >= end) return;
    const uint32_t koff = (uint32_t)(x * p.c.ks1) + g * 8 * es;

    for (int r0 = 0; r0 < rows; r0 += BLOCKS * 16) {
        const int blocks = min((rows - r0 + 15) / 16, BLOCKS);
        __syncthreads();                          // the rows before have been used
        for (int i = wave; i < blocks; i += kWaves) {
            const int r = r0 + i * 16 + x, tok = r / p.G, head = h * p.G + r % p.G;
            u32x4 q[KS];
            load_q<KS, PAD>(p, p.q + b * p.qs0 + tok * p.qs1 + head * p.qs2, r < rows, g, q);
#pragma unroll
            for (int ks = 0; ks < KS; ks++) lq[(i * KS + ks) * 64 + lane] = q[ks];
            const float lse = r < rows ? p.lse[((int64_t)b * p.T + tok) * (p.heads * p.G) + head] : -INFINITY;
            if (g == 0) lrow[i * 16 + x] = lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;
        }
        __syncthreads();

        TileFinder<is_scaled(CT)> finder;
        Tile nxt;
        Raw<CT> kr[2][KS];
        // where this lane adds, and what is there, on its way with the keys
        const auto fetch = [&](int i, float *&at, float &old) {
            nxt = finder.find(p, b, h, i, first + wave, kWaves, n, end);
            load_keys<CT, KS, PAD, true>(p, nxt, end, x, g, koff, kr);
            const int key = nxt.key + 16 * (x >> 2 & 1) + 4 * g + (x & 3);
            const bool mine = x < 8 && (x & 4 ? nxt.there[1] : nxt.there[0]) && key < min(end, p.score_tokens);
            at = mine ? p.score + b * p.sc0 + h * p.sc1 + key : nullptr;
            old = mine ? *at : 0.f;
        };
        float *at, *at_next = nullptr;
        float old, old_next = 0.f;
        if ((first + wave) * kTileKeys < end) fetch(0, at_next, old_next);
        for (int i = 0; i < p.weigh_tiles && (first + wave + i * kWaves) * kTileKeys < end; i++) {
            const Tile t = nxt;
            at = at_next, old = old_next;
            u32x4 k[2][KS];
#pragma unroll
            for (int hf = 0; hf < 2; hf++)
#pragma unroll
                for (int ks = 0; ks < KS; ks++) k[hf][ks] = widen<CT>(kr[hf][ks]);
            if (i + 1 < p.weigh_tiles && (first + wave + (i + 1) * kWaves) * kTileKeys < end) fetch(i + 1, at_next, old_next);
            f32x4 sum[2] = {};
            for (int j = 0; j < blocks; j++) {
                const float row = lrow[j * 16 + x];
                f32x4 sc[1][2], (&s)[2] = sc[0];
#pragma unroll
                for (int ks = 0; ks < KS; ks++) {
                    const u32x4 q = lq[(j * KS + ks) * 64 + lane];
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) s[hf] = mfma<f16_queries(CT)>(k[hf][ks], q, ks ? s[hf] : f32x4{0.f, 0.f, 0.f, 0.f});
                }
                if constexpr (is_scaled(CT)) s[0] *= t.ks[0], s[1] *= t.ks[1];
                uint32_t seen = row == INFINITY ? 0u : 0xffu;
                if (!t.fast) {
                    const int tok = (r0 + j * 16 + x) / p.G;
                    uint32_t bits = p.tree ? tree_bits(p, b, tok, t.key + 4 * g - n, nd, end - n) : 0;
                    bits |= leading_bits((p.tree ? n : min(end, n + tok + 1)) - t.key - 4 * g);
                    seen &= bits & there_bits(t);
                }
                if constexpr (!is_scaled(CT)) settle(sc);
#pragma unroll
                for (int i8 = 0; i8 < 8; i8++) {
                    const float w = __builtin_amdgcn_exp2f(fmaf(s[i8 >> 2][i8 & 3], p.c2, -row));
                    sum[i8 >> 2][i8 & 3] += seen >> i8 & 1 ? w : 0.f;
                }
            }
            // Sums over the 16 lanes of a row of lanes, halving the keys a lane
            // holds with each step: lane x ends with key x % 8 of the eight.
            float v[8] = {sum[0][0], sum[0][1], sum[0][2], sum[0][3], sum[1][0], sum[1][1], sum[1][2], sum[1][3]};
#pragma unroll
            for (int half = 4; half; half >>= 1) {
                const bool up = x & half;
#pragma unroll
                for (int y = 0; y < half; y++) {
                    const float give = up ? v[y] : v[y + half], keep = up ? v[y + half] : v[y];
                    v[y] = keep + __shfl_xor(give, half);
                }
            }
            v[0] += __shfl_xor(v[0], 8);
            if (at) *at = old + v[0];
        }
    }
}

// ------------------------------------------------------------------- host --
struct Plan {
    int DP, RB, wk, nrg, nsplit, slots, min_steps, unit;
    bool shared, flat, walks;                     // k_attend_shared, Walk or even_part, Walk without sharing keys
    uint64_t rows, grid, off_ml, off_used, off_lse, bytes;
};

// may_share: the cache's rows begin on 16 bytes and end on them.
Plan make_plan(uint32_t seqs, uint32_t kv_heads, uint32_t dim, uint32_t cache_tokens, uint32_t T, uint32_t heads, bool may_share, bool scaled)
{
    Plan a;
    const uint32_t G = heads / kv_heads;
    const uint64_t R = (uint64_t)T * G;
    a.DP = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
    const uint64_t tiles = ((uint64_t)cache_tokens + kTileKeys - 1) / kTileKeys;
    // Sharing keys doubles the rate of many rows but begins and ends slowly:
    // it has to have more than 100 tiles of 32 keys by 32 rows for each CU, and
    // with several sequences a workgroup they have to be long. Of 8 key/value
    // heads of 128, shared against not: 4 x 16384 keys of 96 rows 69 against 93
    // us, of 64 rows 59 against 64 (not worth the losses: 64 ragged sequences
    // of up to 1024 93 against 40); 16 x 1024 keys of 512 rows 61 against 81,
    // 1 x 2048 of them 40 against 31; 64 ragged sequences of up to 1024 keys
    // of 96 rows 113 against 62, 16 of up to 4096 66 against 77.
    // The lengths are on the device, so this goes by the capacity, and where
    // that is loose shares keys of too few tokens: 16 sequences of 480, 96 rows,
    // 20 us in capacities up to 2048 and 32 from 8192; one of 1000, 512 rows, 28
    // and 35; 64 of 480, 96 rows, 55 and 59; 16 of 2000 49 both.
    const uint64_t groups = (uint64_t)seqs * kv_heads * (R > 128 ? (R + 255) / 256 : 1);
    a.shared = may_share && R > 64 && a.DP <= 128 && seqs * kv_heads * ((R + 31) / 32) * tiles > 100 * kCUs && (tiles >= 64 || groups <= kCUs);
    a.RB = !a.shared && R <= 16 ? 1 : 2;
    const int waves = a.shared ? kShared : kWaves;
    const uint64_t blocks = (R + a.RB * 16 - 1) / (a.RB * 16);
    // Waves side by side on rows; the others split the keys. Shared, up to 128
    // rows: 128 rows of 64 over 4 x 16384 keys 53 us, with 8 instead of 4 waves
    // 56; 160 rows of 128 over 4 x 8192 keys with 4 instead of 8 68, not 61.
    const int wr = a.shared ? (R > 128 ? 8 : 4) : blocks >= 4 ? 4 : blocks >= 2 ? 2 : 1;
    a.wk = waves / wr;
    a.nrg = (int)((blocks + wr - 1) / wr);
    a.unit = a.shared ? 2 : a.wk;
    a.min_steps = 2;                              // 1: 24 for 20 us where 16384 keys are split; 4: 15 for 13 at 2048
    // Workgroups: one a CU, and eight where they are small, so that one's loads
    // run beside another's join and long sequences are cut as short as others
    // end: 16 rows, 32 sequences of very different lengths up to 8192 101 us,
    // with three a CU 116 (64 of up to 1024 37 and 33, 4 equal ones of 16384
    // FP8 keys 39 and 34). 32 rows, 2 x 131072 FP8 keys: 120 us, with two 140,
    // with four 143; a head dim of 256, 16 rows, 9155 keys: 36 us, with two 38.
    // More sequences than that leaves for each head: a workgroup each.
    // Beside scales, where a wave has all of its next tile under way: two a CU
    // (32 rows, 2 x 131072 keys 116 us, with one 168, with four 133; 16 rows, 4
    // x 16384 keys 35 and, with eight, 45), and eight of heads of 64, whose
    // tiles are half as long (105 and 87 us where Number says). Heads of 256 too,
    // though their registers hold one at a time: 32 ragged sequences of up to
    // 16384 keys, 4 rows, 296 us and, with one, 327, 4 of them 51 and 68; but
    // equal lengths, 2 x 131072 keys of 32 rows, 251 and 239.
    uint64_t want = !a.shared && a.RB == 1 && a.DP < 256 ? 8 * kCUs : kCUs;
    if (scaled && !a.shared && a.DP > 64) want = 2 * kCUs;
    const uint64_t each = (uint64_t)kv_heads * a.nrg;
    const uint64_t slots = want > each ? want / each : 1;
    const uint64_t steps = (tiles + a.unit - 1) / a.unit, most = (steps + a.min_steps - 1) / a.min_steps;
    a.slots = (int)slots;
    a.nsplit = 1;
    a.flat = (a.shared || scaled) && most > 1 && seqs < 4 * slots && (slots > 1 || seqs > 1);
    // Runs in workgroups of their own end apart by as much as one is long; where
    // that is more than 4096 keys, each workgroup takes its share of all
    // sequences instead, one place after the other, though a place begins and
    // ends in some 6 us: 32 ragged sequences of up to 16384 keys, 4 rows, 124 us
    // and, in runs, 169; of up to 8192 84 and 106; of up to 4096 58 both; 64 of up
    // to 4096 76 and 91, of up to 1024 37 and 29; equal ones, 2 of 131072 keys, 104
    // and 103. Made and measured for up to 16 rows of heads of 65 to 128; others
    // take runs.
    a.walks = a.flat && scaled && !a.shared && a.RB == 1 && a.DP == 128 && seqs > 1 && seqs * tiles >= 128 * slots;
    if (a.flat) {
        // parts of one sequence: up to four times what equal lengths give
        uint64_t n = seqs == 1 ? slots : 4 * ((slots + seqs - 1) / seqs) + 1;
        n = n > most + 1 ? most + 1 : n;
        a.nsplit = (int)(n < 2 ? 2 : n);
    } else if (!a.shared) {
        const uint64_t n = (slots + seqs - 1) / seqs;
        a.nsplit = (int)(n > most ? most : n);
    }
    const uint64_t runs = !a.flat ? (uint64_t)seqs * a.nsplit : a.shared || a.walks ? slots : slots + seqs;
    a.grid = each * (scaled && !a.shared ? (runs + 7) / 8 * 8 : runs);
    a.rows = (uint64_t)seqs * heads * T;
    const auto up = [](uint64_t v) { return (v + 255) & ~255ull; };
    a.off_ml = a.nsplit > 1 ? up(a.rows * a.nsplit * a.DP * 4) : 0;
    a.off_used = a.off_ml + (a.nsplit > 1 ? up(a.rows * a.nsplit * 8) : 0);
    a.off_lse = a.off_used + (a.nsplit > 1 ? up(seqs * 4ull) : 0);
    a.bytes = a.off_lse + up(a.rows * 4);
    return a;
}

bool valid_shapes(uint32_t seqs, uint32_t kv_heads, uint32_t dim, uint32_t cache_tokens, uint32_t T, uint32_t heads)
{
    return valid_dims(seqs, kv_heads, dim) && cache_tokens >= 1 && cache_tokens <= (1u << 30) && T >= 1 && T <= (1u << 20) &&
           heads >= kv_heads && heads <= 65535 && heads % kv_heads == 0 && (uint64_t)seqs * T * heads < (1ull << 30);
}

// workgroups of k_attend_weigh
uint64_t weigh_grid(uint32_t cache_tokens, uint64_t seqs, uint64_t heads, uint64_t weigh_tiles)
{
    const uint64_t each = kWaves * weigh_tiles, tiles = ((uint64_t)cache_tokens + kTileKeys - 1) / kTileKeys;
    return (tiles + each - 1) / each * seqs * heads;
}

template <int CT, int DP, int RB, bool PAD>
int launch(const AttendParams &p, uint64_t grid, bool walks, hipStream_t s)
{
    if constexpr (is_scaled(CT) && RB == 1 && DP == 128)
        if (walks) {
            k_attend<CT, DP, RB, PAD, kWalks><<<(unsigned)grid, kWaves * 64, 0, s>>>(p);
            UZIP_KV_LAUNCH_CHECK("k_attend");
            return UZIP_OK;
        }
    k_attend<CT, DP, RB, PAD, is_scaled(CT) ? kRuns : kParts><<<(unsigned)grid, kWaves * 64, 0, s>>>(p);
    UZIP_KV_LAUNCH_CHECK("k_attend");
    return UZIP_OK;
}

template <int CT, int DP, bool PAD>
int run(const AttendParams &p, const Plan &plan, int half, hipStream_t s)
{
    const uint64_t grid = plan.grid;
    int rc = UZIP_EINVAL;
    if (plan.shared) {
        if constexpr (DP <= 128) {
            if constexpr (is_scaled(CT)) {
                if (p.c.table) k_attend_wide<CT, DP, PAD, true><<<(unsigned)grid, kShared * 64, 0, s>>>(p);
                else k_attend_wide<CT, DP, PAD, false><<<(unsigned)grid, kShared * 64, 0, s>>>(p);
            } else {
                if (p.c.table) k_attend_shared<CT, DP, PAD, true><<<(unsigned)grid, kShared * 64, 0, s>>>(p);
                else k_attend_shared<CT, DP, PAD, false><<<(unsigned)grid, kShared * 64, 0, s>>>(p);
            }
            UZIP_KV_LAUNCH_CHECK("k_attend_shared");
            rc = UZIP_OK;
        }
    } else if (plan.RB == 1) rc = launch<CT, DP, 1, PAD>(p, grid, plan.walks, s);
    else rc = launch<CT, DP, 2, PAD>(p, grid, false, s);
    if (rc) return rc;
    if (p.nsplit > 1) {
        if (p.nsplit <= 16 || (p.flat && p.nsplit <= 64)) k_attend_join_few<DP><<<(unsigned)((plan.rows + 15) / 16), 256, 0, s>>>(p, (int64_t)plan.rows, half);
        else k_attend_join_many<DP><<<(unsigned)plan.rows, kWaves * 64, 0, s>>>(p, half);
        UZIP_KV_LAUNCH_CHECK("k_attend_join");
    }
    if (p.score) {
        k_attend_weigh<CT, DP, PAD><<<(unsigned)weigh_grid(p.c.tokens, p.seqs, p.heads, p.weigh_tiles), kWaves * 64, 0, s>>>(p);
        UZIP_KV_LAUNCH_CHECK("k_attend_weigh");
    }
    return UZIP_OK;
}

template <int CT>
int run_type(const AttendParams &p, const Plan &plan, int half, hipStream_t s)
{
    if (plan.DP == 64) return p.D == 64 ? run<CT, 64, false>(p, plan, half, s) : run<CT, 64, true>(p, plan, half, s);
    if (plan.DP == 128) return p.D == 128 ? run<CT, 128, false>(p, plan, half, s) : run<CT, 128, true>(p, plan, half, s);
    return p.D == 256 ? run<CT, 256, false>(p, plan, half, s) : run<CT, 256, true>(p, plan, half, s);
}

uint64_t workspace_bytes(uint32_t seqs, uint32_t kv_heads, uint32_t dim, uint32_t cache_tokens, uint32_t tokens, uint32_t heads, bool scaled)
{
    if (!valid_shapes(seqs, kv_heads, dim, cache_tokens, tokens, heads)) return 0;
    const uint64_t a = make_plan(seqs, kv_heads, dim, cache_tokens, tokens, heads, true, scaled).bytes;
    const uint64_t b = make_plan(seqs, kv_heads, dim, cache_tokens, tokens, heads, false, scaled).bytes;
    return a > b ? a : b;
}

// SCALED: the cache is E4M3 or 8-bit integers with these scales
template <bool SCALED>
int attend(const uzip_kv_cache_t *cache, const uzip_kv_scales_t *scales, const uzip_kv_attend_args_t *a, void *d_ws, uint64_t ws_bytes,
           hipStream_t s)
{
    if (!a || !valid_cache(cache, SCALED) || !valid_tensor(a->q) || !valid_tensor(a->out)) return UZIP_EINVAL;
    if (!valid_shapes(cache->seqs, cache->heads, cache->dim, cache->tokens, a->tokens, a->heads)) return UZIP_EINVAL;
    if (a->dtype > UZIP_KV_F16 || (cache->dtype < UZIP_KV_E5M2 && cache->dtype != a->dtype)) return UZIP_EINVAL;
    if (SCALED && !valid_scales(scales, cache)) return UZIP_EINVAL;
    if (a->q.data == a->out.data) return UZIP_EINVAL;          // the accumulated weights read q again
    if (!a->length || !aligned(a->length, 4) || !aligned(a->drafted, 4) || !aligned(a->lse, 4) || !aligned(a->score, 4)) return UZIP_EINVAL;
    if (!(a->scale >= 0x1p-60f) || !(a->scale <= 0x1p60f)) return UZIP_EINVAL;
    if (a->reserved || (a->score && (a->score_stride[0] < 0 || a->score_stride[1] < 0 || a->score_tokens > cache->tokens))) return UZIP_EINVAL;
    if (a->tree && (a->tree_stride[0] < 0 || a->tree_stride[1] < 0)) return UZIP_EINVAL;
    if (!d_ws || !aligned(d_ws, 16)) return UZIP_EINVAL;
    if (ws_bytes < workspace_bytes(cache->seqs, cache->heads, cache->dim, cache->tokens, a->tokens, a->heads, SCALED)) return UZIP_ENOSPC;
    int64_t bits = cache->dim * elem_size((int)cache->dtype);
    for (int i = 0; i < 3; i++) bits |= (cache->k_stride[i] | cache->v_stride[i]) * elem_size((int)cache->dtype);
    const Plan plan = make_plan(cache->seqs, cache->heads, cache->dim, cache->tokens, a->tokens, a->heads, (bits & 15) == 0, SCALED);
    if (plan.grid * (plan.shared ? kShared : kWaves) * 64 >= kLaunchThreads || (uint64_t)cache->seqs * ((cache->tokens + 31) / 32) >= (1ull << 31)) return UZIP_EINVAL;
    // accumulated weights: enough workgroups to fill the chip four times, rows read once for up to eight tiles of a wave
    const uint64_t waves = (uint64_t)cache->seqs * cache->heads * ((cache->tokens + kTileKeys - 1) / kTileKeys);
    const uint64_t share = waves / (4 * kCUs * kWaves), weigh_tiles = share < 1 ? 1 : share > 8 ? 8 : share;
    if (a->score && weigh_grid(cache->tokens, cache->seqs, cache->heads, weigh_tiles) * kWaves * 64 >= kLaunchThreads) return UZIP_EINVAL;

    AttendParams p;
    memset(&p, 0, sizeof p);
    p.c = view_of(cache);
    if (SCALED) p.scales = view_of(scales);
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
    p.slots = plan.slots;
    p.min_steps = plan.min_steps;
    p.seqs = (int)cache->seqs;
    p.used = reinterpret_cast<int *>(ws + plan.off_used);
    p.flat = plan.flat;
    p.weigh_tiles = (int)weigh_tiles;
    p.wk = plan.wk;
    p.unit = plan.unit;
    p.c2 = a->scale * 1.4426950408889634f;
    const int half = a->dtype == UZIP_KV_F16;
    if constexpr (SCALED) {
        if (cache->dtype == UZIP_KV_E4M3) return half ? run_type<kE4M3>(p, plan, half, s) : run_type<kE4M3BF>(p, plan, half, s);
        return half ? run_type<kI8>(p, plan, half, s) : run_type<kI8BF>(p, plan, half, s);
    } else {
        if (cache->dtype == UZIP_KV_BF16) return run_type<kBF16>(p, plan, half, s);
        if (cache->dtype == UZIP_KV_F16) return run_type<kF16>(p, plan, half, s);
        return half ? run_type<kE5M2>(p, plan, half, s) : run_type<kE5M2BF>(p, plan, half, s);
    }
}

}  // namespace
}  // namespace uzip_kv

#endif

// uzip_kv_step.hip -- between two steps with drafted tokens (gfx950, wave64):
// which of them the target accepts, the accepted ones moved up in the cache,
// and the page tables of the next step. The C-ABI is declared in
// include/uzip_kv.h.
#include "kv_common.h"

namespace uzip_kv {
namespace {

// ----------------------------------------------------------------- verify --
// A node's children are tried in their order. With p the target's and q the
// drafting model's probabilities behind the node, c = 0 and mass = 1 at first:
// child x is accepted if u q(x) mass < max(p(x) - c q(x), 0); if it is not, c
// grows by mass, and mass becomes the sum of max(p - c q, 0), the probability
// that is left. (The usual rule takes max(r - q, 0), normalised, from r at each
// rejection; c adds those steps up, so that p and q are read as they came.)
// Without q, x was chosen, not drawn: q is 1 at x, which is taken out of p.
//
// What tells tokens apart are sums over the vocabulary, compared with a random
// number: they are binary64, since of 2^17 borders between tokens a binary32
// sum crosses some in one case of a hundred.
//
// The walk down the tree reads a value of p and q for each node, all at once.
// Only the sums read whole rows: k_verify's workgroups each walk and then sum
// a slice of the row where the walk ended, and k_verify_end finds the token in
// it. Where a walk asks for a sum (a second child, with q), it goes on there.
constexpr int kVerifyThreads = 256, kVerifyWaves = kVerifyThreads / 64, kEndThreads = 1024;
constexpr int kSeg = 1024;                        // tokens whose sum is kept
constexpr int kNodes = 1024;                      // of a tree, at most

struct Walked {
    int at, next, count, rejected;                // rejected: children of `at`, whose tokens are listed
    double c, mass;
    int pending;                                  // mass has to become a sum before node `next` is tried
    int at_sums;                                  // which of the two places its sums are in
};

struct VerifyParams {
    const char *p, *q;
    int64_t p0, p1, q0, q1;                       // bytes
    const int32_t *tokens, *parent, *drafted;
    int64_t tok0, par0, u0;
    const float *uniform;
    int32_t *path, *count, *token;
    int T, V, slices, segs;
    double *sums;                                 // [2][sequence][segs]
    Walked *state;                                // [2][sequence]
    int seqs, rounds;                             // launches of k_verify_more
    int32_t *rejected;                            // [sequence][T]
};

template <int PT>
__device__ inline float prob(const char *row, int64_t i)
{
    float x;
    if constexpr (PT == 2) x = reinterpret_cast<const float *>(row)[i];
    else if constexpr (PT == kF16) x = f16_to_f32(reinterpret_cast<const uint16_t *>(row)[i]);
    else x = bf16_to_f32(reinterpret_cast<const uint16_t *>(row)[i]);
    return x > 0.f && x < INFINITY ? x : 0.f;     // what is no probability counts as none
}

// One wave goes on with the walk. list: the rejected children's tokens, in LDS.
template <int PT>
__device__ void walk(const VerifyParams &p, int b, int nd, Walked &w, int32_t *list, bool tell)
{
    const int lane = (int)(threadIdx.x & 63);
    bool whole = true;                            // mass is what it says
    w.pending = 0;
    for (int base = w.next & ~63; base < nd; base += 64) {
        const int node = base + lane;
        const bool in = node >= 1 && node < nd;
        int par = in ? p.parent ? p.parent[b * p.par0 + node] : node - 1 : -1;
        const int x = in ? p.tokens[b * p.tok0 + node] : -1;
        if (par >= node || x < 0 || x >= p.V) par = -1;
        float px = 0.f, qx = 1.f, u = 0.f;
        if (par >= 0) {
            u = p.uniform[b * p.u0 + node];
            px = prob<PT>(p.p + b * p.p0 + par * p.p1, x);
            if (p.q) qx = prob<PT>(p.q + b * p.q0 + par * p.q1, x);
        }
        const int end = min(64, nd - base);
        for (int k = max(w.next - base, 0); k < end; k++) {
            if (__builtin_amdgcn_readlane(par, k) != w.at) continue;
            if (!whole) {
                w.next = base + k;
                w.pending = 1;
                return;
            }
            const double pk = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(px), k));
            const double qk = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(qx), k));
            const double uk = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(u), k));
            const int xk = __builtin_amdgcn_readlane(x, k);
            bool again = false;                   // a token that was taken out
            if (!p.q)
                for (int i = 0; i < w.rejected; i += 64) again = again || __builtin_amdgcn_ballot_w64(i + lane < w.rejected && list[i + lane] == xk) != 0;
            const double left = p.q ? pk - w.c * qk : pk;
            if (left > 0. && !again && uk * qk * w.mass < left) {
                w.at = base + k;
                if (tell && lane == 0) p.path[(int64_t)b * p.T + w.count] = w.at;
                w.count++;
                w.c = 0., w.mass = 1., w.rejected = 0;
            } else if (p.q) {
                w.c += w.mass;
                whole = false;
            } else if (!again) {
                w.mass -= pk;
                if (lane == 0) list[w.rejected] = xk;
                // read by the wave's other lanes from here on
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
                w.rejected++;
            }
        }
        w.next = base + 64;
    }
    w.next = nd;
}

// What is left of the lane's tokens of a segment, and its sum over the wave.
template <int PT>
__device__ inline double left_of(const VerifyParams &p, const char *pr, const char *qr, const Walked &w, const int32_t *list, int i)
{
    const double x = prob<PT>(pr, i);
    if (qr) return fmax(fma(-w.c, (double)prob<PT>(qr, i), x), 0.);
    for (int k = 0; k < w.rejected; k++)
        if (list[k] == i) return 0.;
    return x;
}

template <int PT>
__device__ inline double segment_sum(const VerifyParams &p, const char *pr, const char *qr, const Walked &w, const int32_t *list, int seg)
{
    constexpr int ES = PT == 2 ? 4 : 2, VEC = 16 / ES;
    const int lane = (int)(threadIdx.x & 63), first = seg * kSeg;
    double sum = 0.;
    bool listed = false;                          // a token that was taken out is here
    if (!qr)
        for (int i = 0; i < w.rejected; i += 64)
            listed = listed || __builtin_amdgcn_ballot_w64(i + lane < w.rejected && (list[i + lane] ^ first) < kSeg && list[i + lane] >= first) != 0;
    if (listed) {
        for (int i = first + lane; i < min(first + kSeg, p.V); i += 64) sum += left_of<PT>(p, pr, qr, w, list, i);
    } else if (first + kSeg <= p.V && (((uintptr_t)pr | (uintptr_t)qr) & 15) == 0) {
        u32x4 a[kSeg / 64 / VEC], c[kSeg / 64 / VEC];
#pragma unroll
        for (int j = 0; j < kSeg / 64 / VEC; j++) {
            const int64_t at = (int64_t)(first + (j * 64 + lane) * VEC) * ES;
            a[j] = *reinterpret_cast<const u32x4 *>(pr + at);
            if (qr) c[j] = *reinterpret_cast<const u32x4 *>(qr + at);
        }
#pragma unroll
        for (int j = 0; j < kSeg / 64 / VEC; j++)
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                const double x = prob<PT>(reinterpret_cast<const char *>(&a[j]), e);
                sum += qr ? fmax(fma(-w.c, (double)prob<PT>(reinterpret_cast<const char *>(&c[j]), e), x), 0.) : x;
            }
    } else {
#pragma unroll
        for (int j = 0; j < kSeg / 64; j++) {
            const int i = first + j * 64 + lane;
            if (i >= p.V) continue;
            const double x = prob<PT>(pr, i);
            sum += qr ? fmax(fma(-w.c, (double)prob<PT>(qr, i), x), 0.) : x;
        }
    }
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
    return sum;
}

// Bound by trips to memory that depend on each other: tokens, their
// probabilities, the row where the walk ends, its sums, a segment again. A chain
// of 5 nodes over 32000 tokens 5 us and, for k_verify_end, 7; 16 trees of 32
// over 131072 9, twice 7, and 10.
template <int PT>
__global__ __launch_bounds__(kVerifyThreads) void k_verify(VerifyParams p)
{
    __shared__ int32_t list[kNodes];
    __shared__ Walked shared;
    const int slice = (int)blockIdx.x % p.slices, b = (int)blockIdx.x / p.slices;
    const int tid = (int)threadIdx.x, nd = clamp_drafted(p.drafted, b, p.T);
    if (nd == 0) return;
    if (tid < 64) {
        Walked w = {0, 1, 1, 0, 0., 1., 0, 0};
        if (slice == 0 && tid == 0) p.path[(int64_t)b * p.T] = 0;
        walk<PT>(p, b, nd, w, list, slice == 0);
        if (tid == 0) {
            shared = w;
            if (slice == 0) p.state[b] = w;
        }
        if (slice == 0)
            for (int i = tid; i < w.rejected; i += 64) p.rejected[(int64_t)b * p.T + i] = list[i];
    }
    __syncthreads();
    const Walked w = shared;
    const char *pr = p.p + b * p.p0 + w.at * p.p1, *qr = p.q ? p.q + b * p.q0 + w.at * p.q1 : nullptr;
    for (int seg = slice * kVerifyWaves + (tid >> 6); seg < p.segs; seg += p.slices * kVerifyWaves) {
        const double sum = segment_sum<PT>(p, pr, qr, w, list, seg);
        if ((tid & 63) == 0) p.sums[(int64_t)b * p.segs + seg] = sum;
    }
}

// Sum over the workgroup of what its threads have, in one order; wave_sum: a word a wave.
__device__ inline double whole_sum(double sum, double *wave_sum, int waves)
{
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
    if ((threadIdx.x & 63) == 0) wave_sum[threadIdx.x >> 6] = sum;
    __syncthreads();
    double total = 0.;
    for (int i = 0; i < waves; i++) total += wave_sum[i];
    __syncthreads();
    return total;
}

// Walks that wait for a sum go on. What they wait for was written by the launch
// before, and they write to the other place, since all of a sequence's
// workgroups read it.
template <int PT>
__global__ __launch_bounds__(kVerifyThreads) void k_verify_more(VerifyParams p, int round)
{
    __shared__ int32_t list[kNodes];              // of rejected tokens: none with q
    __shared__ Walked shared;
    __shared__ double wave_sum[kVerifyWaves];
    const int slice = (int)blockIdx.x % p.slices, b = (int)blockIdx.x / p.slices;
    const int tid = (int)threadIdx.x, nd = clamp_drafted(p.drafted, b, p.T);
    if (nd == 0) return;
    const Walked was = p.state[(int64_t)(round & 1) * p.seqs + b];
    Walked *out = p.state + (int64_t)(~round & 1) * p.seqs + b;
    if (!was.pending) {
        if (slice == 0 && tid == 0) *out = was;
        return;
    }
    const double *sums = p.sums + ((int64_t)was.at_sums * p.seqs + b) * p.segs;
    double sum = 0.;
    for (int i = tid; i < p.segs; i += kVerifyThreads) sum += sums[i];
    const double total = whole_sum(sum, wave_sum, kVerifyWaves);
    if (tid < 64) {
        Walked w = was;
        w.mass = total;
        walk<PT>(p, b, nd, w, list, slice == 0);
        if (w.at != was.at || w.c != was.c) w.at_sums ^= 1;
        if (tid == 0) {
            shared = w;
            if (slice == 0) *out = w;
        }
    }
    __syncthreads();
    const Walked w = shared;
    if (w.at_sums == was.at_sums) return;         // the same sums
    const char *pr = p.p + b * p.p0 + w.at * p.p1, *qr = p.q + b * p.q0 + w.at * p.q1;
    for (int seg = slice * kVerifyWaves + (tid >> 6); seg < p.segs; seg += p.slices * kVerifyWaves) {
        const double one = segment_sum<PT>(p, pr, qr, w, list, seg);
        if ((tid & 63) == 0) p.sums[((int64_t)w.at_sums * p.seqs + b) * p.segs + seg] = one;
    }
}

template <int PT>
__global__ __launch_bounds__(kEndThreads) void k_verify_end(VerifyParams p)
{
    __shared__ int32_t list[kNodes];
    __shared__ Walked shared;
    __shared__ double wave_sum[kEndThreads / 64];
    const int threads = (int)blockDim.x, waves = threads / 64;
    const int b = (int)blockIdx.x, tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nd = clamp_drafted(p.drafted, b, p.T);
    if (nd == 0) {
        for (int i = tid; i < p.T; i += threads) p.path[(int64_t)b * p.T + i] = -1;
        if (tid == 0) p.count[b] = 0, p.token[b] = -1;
        return;
    }
    Walked w = p.state[(int64_t)(p.rounds & 1) * p.seqs + b];
    for (int i = tid; i < w.rejected; i += threads) list[i] = p.rejected[(int64_t)b * p.T + i];
    __syncthreads();
    double *sums = p.sums + ((int64_t)w.at_sums * p.seqs + b) * p.segs;
    const char *pr, *qr;
    double total;
    bool plain = false;                           // nothing was left: from p itself
    for (;;) {
        pr = p.p + b * p.p0 + w.at * p.p1, qr = p.q && !plain ? p.q + b * p.q0 + w.at * p.q1 : nullptr;
        double sum = 0.;
        for (int i = tid; i < p.segs; i += threads) sum += sums[i];
        total = whole_sum(sum, wave_sum, waves);
        if (w.pending) {
            if (wave == 0) {
                const int at = w.at;
                const double c = w.c;
                w.mass = total;
                walk<PT>(p, b, nd, w, list, true);
                w.at_sums = w.at != at || w.c != c;       // other sums are needed
                if (lane == 0) shared = w;
            }
            __syncthreads();
            w = shared;
            __syncthreads();
            if (!w.at_sums) continue;                 // mass was 0, and c is what it was
        } else if (!(total > 0.) && !plain) {
            plain = true;
            w.rejected = 0;
        } else {
            break;
        }
        pr = p.p + b * p.p0 + w.at * p.p1, qr = p.q && !plain ? p.q + b * p.q0 + w.at * p.q1 : nullptr;
        for (int seg = wave; seg < p.segs; seg += waves) {
            const double s = segment_sum<PT>(p, pr, qr, w, list, seg);
            if (lane == 0) sums[seg] = s;
        }
        __syncthreads();
    }
    for (int i = w.count + tid; i < p.T; i += threads) p.path[(int64_t)b * p.T + i] = -1;
    if (wave) return;
    // the first segment, and in it the first token, where the sum so far is beyond u * total
    const double goal = (double)p.uniform[b * p.u0] * total;
    int seg = -1, last = 0;                       // last: with something left
    double before = 0.;
    for (int base = 0; base < p.segs && seg < 0; base += 64) {
        const double mine = base + lane < p.segs ? sums[base + lane] : 0.;
        double sum = mine;
        for (int x = 1; x < 64; x <<= 1) {
            const double v = __shfl_up(sum, x);
            if (lane >= x) sum += v;
        }
        const uint64_t past = __builtin_amdgcn_ballot_w64(before + sum > goal), some = __builtin_amdgcn_ballot_w64(mine > 0.);
        if (some) last = base + 63 - __builtin_clzll(some);
        if (past) {
            const int k = __builtin_ctzll(past);
            seg = base + k;
            if (k) before += __shfl(sum, k - 1);
        } else {
            before += __shfl(sum, 63);
        }
    }
    const bool end = seg < 0;                     // rounding: the last token there is
    if (end) seg = last;
    constexpr int EACH = kSeg / 64;
    double mine[EACH], sum = 0.;
    int top = -1;
#pragma unroll
    for (int e = 0; e < EACH; e++) {
        const int i = seg * kSeg + lane * EACH + e;
        mine[e] = i < p.V ? left_of<PT>(p, pr, qr, w, list, i) : 0.;
        sum += mine[e];
        if (mine[e] > 0.) top = i;
    }
    double run = sum;
    for (int x = 1; x < 64; x <<= 1) {
        const double v = __shfl_up(run, x);
        if (lane >= x) run += v;
    }
    const uint64_t past = end ? 0 : __builtin_amdgcn_ballot_w64(before + run > goal);
    int token = -1;                               // no probability at all
    if (past) {
        const int k = __builtin_ctzll(past);
        double so_far = before + (run - sum);
        int found = -1;
#pragma unroll
        for (int e = 0; e < EACH; e++) {
            so_far += mine[e];
            if (found < 0 && so_far > goal && mine[e] > 0.) found = seg * kSeg + lane * EACH + e;
        }
        if (found < 0) found = top;
        token = __builtin_amdgcn_readlane(found, k);
    } else {
        const uint64_t some = __builtin_amdgcn_ballot_w64(top >= 0);
        token = some ? __builtin_amdgcn_readlane(top, 63 - __builtin_clzll(some)) : -1;
    }
    if (lane == 0) p.count[b] = w.count, p.token[b] = token;
}

struct VerifyWs {
    uint64_t off_state, off_rejected, bytes;
};

VerifyWs verify_ws(uint64_t seqs, uint64_t nodes, uint64_t vocab)
{
    const auto up = [](uint64_t v) { return (v + 255) & ~255ull; };
    VerifyWs w;
    w.off_state = up(2 * seqs * ((vocab + kSeg - 1) / kSeg) * 8);
    w.off_rejected = w.off_state + up(2 * seqs * sizeof(Walked));
    w.bytes = w.off_rejected + up(seqs * nodes * 4);
    return w;
}

bool valid_verify(uint32_t seqs, uint32_t nodes, uint32_t vocab)
{
    return seqs >= 1 && seqs <= 65535 && nodes >= 1 && nodes <= (uint32_t)kNodes && vocab >= 1 && vocab <= (1u << 30);
}

template <int PT>
int run_verify(const VerifyParams &p, int seqs, hipStream_t s)
{
    k_verify<PT><<<(unsigned)(seqs * p.slices), kVerifyThreads, 0, s>>>(p);
    UZIP_KV_LAUNCH_CHECK("k_verify");
    for (int i = 0; i < p.rounds; i++) {
        k_verify_more<PT><<<(unsigned)(seqs * p.slices), kVerifyThreads, 0, s>>>(p, i);
        UZIP_KV_LAUNCH_CHECK("k_verify_more");
    }
    // a walk that asks for sums has them made by the one workgroup: as wide as it can be
    k_verify_end<PT><<<(unsigned)seqs, p.q && p.parent ? kEndThreads : kVerifyThreads, 0, s>>>(p);
    UZIP_KV_LAUNCH_CHECK("k_verify_end");
    return UZIP_OK;
}

// ----------------------------------------------------------------- accept --
// Token length + path[j] becomes token length + j. A way down a tree goes up
// in its numbers, so path[j] >= j, and a row is read before or when it is
// written if each thread, for its 8 elements, goes through the rows in order;
// kMoved rows' loads are under way together. Bound by the chain of trips: count,
// path, page numbers, rows; 64 sequences of 64 nodes in pages 7 us, one 2.
constexpr int kAcceptThreads = 256, kMoved = 8, kChunk = 64;

struct AcceptParams {
    CacheView c;
    const int32_t *length, *path, *count;
    int64_t path0;
    int T, H, per, parts;                         // per: units of 8 elements a head; workgroups a sequence
};

template <typename U>
__global__ __launch_bounds__(kAcceptThreads) void k_accept(AcceptParams p)
{
    __shared__ int64_t from[2][kChunk], to[2][kChunk];
    const int part = (int)blockIdx.x % p.parts, b = (int)blockIdx.x / p.parts, tid = (int)threadIdx.x;
    const int u = part * kAcceptThreads + tid, head = u / p.per % p.H, kv = u / p.per / p.H;
    const int n = max(0, min(p.count[b], p.T));
    char *base = kv == 0 ? p.c.k + head * p.c.ks2 : p.c.v + head * p.c.vs2;
    base += u % p.per * (int64_t)sizeof(U);
    for (int j0 = 0; j0 < n; j0 += kChunk) {
        if (tid < kChunk) {
            const int j = j0 + tid;
            int64_t ks = -1, kd = -1, vs = -1, vd = -1;
            if (j < n) {
                const int way = p.path[b * p.path0 + j];
                const int64_t src = (int64_t)p.length[b] + way, dst = (int64_t)p.length[b] + j;
                if (way > j && way < p.T && dst >= 0 && src < p.c.tokens && locate(p.c, b, (uint32_t)src, p.c.ks0, p.c.ks1, ks) &&
                    locate(p.c, b, (uint32_t)dst, p.c.ks0, p.c.ks1, kd)) {
                    locate(p.c, b, (uint32_t)src, p.c.vs0, p.c.vs1, vs);
                    locate(p.c, b, (uint32_t)dst, p.c.vs0, p.c.vs1, vd);
                } else {
                    ks = -1;
                }
            }
            from[0][tid] = ks, to[0][tid] = kd, from[1][tid] = ks < 0 ? -1 : vs, to[1][tid] = vd;
        }
        __syncthreads();
        if (kv < 2)
            for (int j = 0; j < min(kChunk, n - j0); j += kMoved) {
                U row[kMoved];
#pragma unroll
                for (int i = 0; i < kMoved; i++)
                    if (from[kv][j + i] >= 0) row[i] = *reinterpret_cast<const U *>(base + from[kv][j + i]);
#pragma unroll
                for (int i = 0; i < kMoved; i++)
                    if (from[kv][j + i] >= 0) *reinterpret_cast<U *>(base + to[kv][j + i]) = row[i];
            }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ pages --
// What holds a page is read off the table itself, so there are no counts that
// could go wrong: a word a page, which its holders mark, and for a fork another,
// the least of the sequences that have it as their partly filled last one.
// Marks, the plan and the table are launches of their own, since each needs all
// of the one before: 256 sequences of up to 512 pages of 11000 in 2 + 4 + 7 + 4
// us. The plan is one workgroup's, which looks at 8192 pages at a time.
constexpr uint32_t kFree = 0xffffffffu;
constexpr uint32_t kHeld = 0;                     // fork: whole, or held outside; compact: held outside
// compact: 1 of the table; then 2 + where it goes
constexpr int kPageThreads = 256, kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;

struct PageParams {
    const int32_t *table, *length, *parent;
    const uint8_t *held;
    int64_t t0;
    int32_t *out_table, *out_length, *moves, *left;
    uint32_t *mark;                               // [pages]
    uint32_t *first;                              // fork: [pages], 1 + the first sequence that fills it on
    int32_t *given;                               // pages handed out, in order
    int32_t *offset;                              // [seqs]: of a sequence's first one
    int rows, seqs, entries, pages, shift, room;  // rows: of table
    int most;                                     // moves
    int compact;
};

// Sequence b after the step: its old row, tokens, whole pages, and what its table then holds.
struct Branch {
    int row, n, full, end;
    bool part;
    __device__ inline Branch(const PageParams &p, int b)
    {
        row = p.parent ? p.parent[b] : b;
        const bool live = row >= 0 && row < p.rows;
        if (!live) row = -1;
        const int64_t cap = (int64_t)p.entries << p.shift;
        n = live ? (int)max((int64_t)0, min((int64_t)p.length[row], cap)) : 0;
        full = n >> p.shift;
        part = (n & ((1 << p.shift) - 1)) != 0;
        end = live ? (int)min(((int64_t)n + p.room + (1 << p.shift) - 1) >> p.shift, (int64_t)p.entries) : 0;
    }
    __device__ inline uint32_t page(const PageParams &p, int e) const { return (uint32_t)p.table[row * p.t0 + e]; }
};

__global__ __launch_bounds__(kPageThreads) void k_pages_clear(PageParams p)
{
    const int i = (int)(blockIdx.x * kPageThreads + threadIdx.x);
    if (i >= p.pages) return;
    p.mark[i] = p.held && p.held[i] ? kHeld : kFree;
    if (p.first) p.first[i] = kFree;
}

__global__ __launch_bounds__(kPageThreads) void k_pages_mark(PageParams p, int parts)
{
    const int b = (int)blockIdx.x / parts, e = ((int)blockIdx.x % parts) * kPageThreads + (int)threadIdx.x;
    const Branch s(p, b);
    if (s.row < 0 || e >= s.full + s.part) return;
    const uint32_t x = s.page(p, e);
    if (x >= (uint32_t)p.pages) return;
    // Stores of one value need no atomics; the words that a minimum is taken of
    // are others, since dies would not see each other's stores before it. (256
    // sequences of 270 pages 3.5 us; 12 with atomics for all or with atomic stores.)
    if (p.compact || e < s.full) {
        const uint32_t as = p.compact ? 1u : kHeld;
        if (p.mark[x] > as) p.mark[x] = as;
    } else {
        atomicMin(p.first + x, 1u + (uint32_t)b);
    }
}

// inclusive sum over the workgroup's threads, and of all; wsum: one word a wave
__device__ inline int sum_before(int v, int *wsum, int &all)
{
    const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
    int sum = v;
    for (int x = 1; x < 64; x <<= 1) {
        const int o = __shfl_up(sum, x);
        if (lane >= x) sum += o;
    }
    __syncthreads();                              // the words have been read
    if (lane == 63) wsum[wave] = sum;
    __syncthreads();
    all = 0;
    int before = 0;
    for (int w = 0; w < kPlanWaves; w++) {
        if (w < wave) before += wsum[w];
        all += wsum[w];
    }
    return before + sum - v;
}

__device__ inline bool copied(const PageParams &p, const Branch &s, int b)
{
    if (!s.part) return false;
    const uint32_t x = s.page(p, s.full);
    return x < (uint32_t)p.pages && (p.mark[x] == kHeld || p.first[x] != 1u + (uint32_t)b);
}

constexpr int kPlanPages = 8;                     // pages a thread looks at, at a time

// a fork's are kHeld, kFree or a first sequence
template <bool FORK>
__device__ inline void load_marks(const PageParams &p, int first, uint32_t (&m)[kPlanPages])
{
    if (first + kPlanPages <= p.pages) {
        const u32x4 a = *reinterpret_cast<const u32x4 *>(p.mark + first), c = *reinterpret_cast<const u32x4 *>(p.mark + first + 4);
#pragma unroll
        for (int i = 0; i < 4; i++) m[i] = a[i], m[4 + i] = c[i];
        if constexpr (FORK) {
            const u32x4 d = *reinterpret_cast<const u32x4 *>(p.first + first), e = *reinterpret_cast<const u32x4 *>(p.first + first + 4);
#pragma unroll
            for (int i = 0; i < 4; i++) m[i] = min(m[i], d[i]), m[4 + i] = min(m[4 + i], e[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPlanPages; i++) {
            m[i] = first + i < p.pages ? p.mark[first + i] : kHeld;
            if (FORK && first + i < p.pages) m[i] = min(m[i], p.first[first + i]);
        }
    }
}

__global__ __launch_bounds__(kPlanThreads) void k_fork_plan(PageParams p)
{
    __shared__ int wsum[kPlanWaves];
    const int tid = (int)threadIdx.x;
    int need = 0, all;
    for (int base = 0; base < p.seqs; base += kPlanThreads) {
        const int b = base + tid;
        int mine = 0;
        if (b < p.seqs) {
            const Branch s(p, b);
            if (s.row >= 0) mine = max(0, s.end - s.full - (s.part && !copied(p, s, b) ? 1 : 0));
        }
        const int at = need + sum_before(mine, wsum, all);
        if (b < p.seqs) p.offset[b] = at;
        need += all;
    }
    int have = 0;
    for (int base = 0; base < p.pages; base += kPlanThreads * kPlanPages) {
        const int first = base + tid * kPlanPages;
        uint32_t m[kPlanPages];
        load_marks<true>(p, first, m);
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kPlanPages; i++) mine += m[i] == kFree;
        int at = have + sum_before(mine, wsum, all);
#pragma unroll
        for (int i = 0; i < kPlanPages; i++)
            if (m[i] == kFree) {
                if (at < need) p.given[at] = first + i;
                at++;
            }
        have += all;
    }
    for (int i = have + tid; i < need; i += kPlanThreads) p.given[i] = -1;
    if (tid == 0) p.left[0] = have - need;
}

__global__ __launch_bounds__(kPageThreads) void k_fork_fill(PageParams p, int parts)
{
    const int b = (int)blockIdx.x / parts, e = ((int)blockIdx.x % parts) * kPageThreads + (int)threadIdx.x;
    const Branch s(p, b);
    const bool copy = s.row >= 0 && copied(p, s, b);
    const int own = s.full + (s.part && !copy ? 1 : 0);           // entries that stay
    if (e < p.entries) {
        int x = -1;
        if (s.row >= 0 && e < own) {
            const uint32_t old = s.page(p, e);
            x = old < (uint32_t)p.pages ? (int)old : -1;
        } else if (s.row >= 0 && e < s.end) {
            x = p.given[p.offset[b] + e - own];
        }
        p.out_table[(int64_t)b * p.entries + e] = x;
    }
    if (e == 0) {
        p.out_length[b] = s.n;
        const int to = copy ? p.given[p.offset[b]] : -1;
        p.moves[2 * b] = to >= 0 ? (int)s.page(p, s.full) : -1;
        p.moves[2 * b + 1] = to;
    }
}

__global__ __launch_bounds__(kPlanThreads) void k_compact_plan(PageParams p)
{
    __shared__ int wsum[kPlanWaves];
    const int tid = (int)threadIdx.x;
    int used = 0, all;
    for (int base = 0; base < p.pages; base += kPlanThreads * kPlanPages) {
        uint32_t m[kPlanPages];
        load_marks<false>(p, base + tid * kPlanPages, m);
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kPlanPages; i++) mine += base + tid * kPlanPages + i < p.pages && m[i] != kFree;
        sum_before(mine, wsum, all);
        used += all;
    }
    int holes = 0;
    for (int base = 0; base < used; base += kPlanThreads * kPlanPages) {
        const int first = base + tid * kPlanPages;
        uint32_t m[kPlanPages];
        load_marks<false>(p, first, m);
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kPlanPages; i++) mine += first + i < used && m[i] == kFree;
        int at = holes + sum_before(mine, wsum, all);
#pragma unroll
        for (int i = 0; i < kPlanPages; i++)
            if (first + i < used && m[i] == kFree) p.given[at++] = first + i;
        holes += all;
    }
    __syncthreads();
    int moved = 0;
    for (int base = used / (kPlanThreads * kPlanPages) * (kPlanThreads * kPlanPages); base < p.pages; base += kPlanThreads * kPlanPages) {
        const int first = base + tid * kPlanPages;
        uint32_t m[kPlanPages];
        load_marks<false>(p, first, m);
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kPlanPages; i++) mine += first + i >= used && m[i] == 1u;
        int at = moved + sum_before(mine, wsum, all);
#pragma unroll
        for (int i = 0; i < kPlanPages; i++)
            if (first + i >= used && m[i] == 1u) {
                const int to = p.given[at];
                p.moves[2 * at] = first + i, p.moves[2 * at + 1] = to;
                p.mark[first + i] = 2u + (uint32_t)to;
                at++;
            }
        moved += all;
    }
    for (int i = moved + tid; i < p.most; i += kPlanThreads) p.moves[2 * i] = p.moves[2 * i + 1] = -1;
    if (tid == 0) p.left[0] = used;
}

__global__ __launch_bounds__(kPageThreads) void k_compact_fill(PageParams p, int parts)
{
    const int b = (int)blockIdx.x / parts, e = ((int)blockIdx.x % parts) * kPageThreads + (int)threadIdx.x;
    if (e >= p.entries) return;
    const Branch s(p, b);
    int x = -1;
    if (e < s.full + s.part) {
        const uint32_t old = s.page(p, e);
        if (old < (uint32_t)p.pages) x = p.mark[old] >= 2u ? (int)(p.mark[old] - 2u) : (int)old;
    }
    p.out_table[(int64_t)b * p.entries + e] = x;
}

// Pages are copied as bytes, in units of U, kCopied of which a thread has under
// way. Each workgroup takes a piece of one page of one pool. 4000 pages of 64 KB
// in two pools: 207 us, the rate of a copy.
constexpr int kPools = 8, kCopied = 4;
struct Pool {
    char *data;
    int64_t page, s0, s1;                         // bytes
    uint32_t n0, n1, run, units;                  // a page: n0 x n1 runs of `run` units; units: of a page
    uint32_t parts;                               // workgroups a page
};
struct CopyParams {
    const int32_t *moves;
    Pool pool[kPools];
    uint32_t pages, parts;                        // parts: of all pools
    int pools;
};

template <typename U>
__global__ __launch_bounds__(kPageThreads) void k_copy_pages(CopyParams p)
{
    const uint32_t move = blockIdx.x / p.parts;
    uint32_t part = blockIdx.x % p.parts;
    const uint32_t src = (uint32_t)p.moves[2 * (int64_t)move], dst = (uint32_t)p.moves[2 * (int64_t)move + 1];
    if (src >= p.pages || dst >= p.pages || src == dst) return;
    int k = 0;
    while (part >= p.pool[k].parts) part -= p.pool[k++].parts;
    const Pool &q = p.pool[k];
    const char *from = q.data + (int64_t)src * q.page;
    char *to = q.data + (int64_t)dst * q.page;
    U v[kCopied];
    int64_t at[kCopied];
#pragma unroll
    for (int i = 0; i < kCopied; i++) {
        const uint32_t u = (part * kCopied + i) * kPageThreads + threadIdx.x;
        at[i] = -1;
        if (u >= q.units) continue;
        const uint32_t run = u / q.run;
        at[i] = (run / q.n1) * q.s0 + (run % q.n1) * q.s1 + (int64_t)(u - run * q.run) * sizeof(U);
        v[i] = *reinterpret_cast<const U *>(from + at[i]);
    }
#pragma unroll
    for (int i = 0; i < kCopied; i++)
        if (at[i] >= 0) *reinterpret_cast<U *>(to + at[i]) = v[i];
}

struct PagesWs {
    uint64_t off_first, off_given, off_offset, bytes;
};

PagesWs pages_ws(uint64_t pages, uint64_t seqs, uint64_t entries)
{
    const auto up = [](uint64_t v) { return (v + 255) & ~255ull; };
    PagesWs w;
    w.off_first = up(pages * 4);
    w.off_given = w.off_first + up(pages * 4);
    const uint64_t given = seqs * entries > pages ? seqs * entries : pages;
    w.off_offset = w.off_given + up(given * 4);
    w.bytes = w.off_offset + up(seqs * 4);
    return w;
}

bool valid_pages(uint64_t pages, uint64_t seqs, uint64_t entries)
{
    return pages >= 1 && pages <= (1u << 30) && seqs >= 1 && seqs <= 65535 && entries >= 1 && entries <= (1u << 26) && seqs * entries < (1ull << 31);
}

int plan_pages(const uzip_kv_pages_t *a, bool compact, void *d_ws, uint64_t ws_bytes, hipStream_t s)
{
    if (!a || !a->table || !aligned(a->table, 4) || !a->length || !aligned(a->length, 4) || !aligned(a->parent, 4)) return UZIP_EINVAL;
    if (!a->out_table || !aligned(a->out_table, 4) || !a->moves || !aligned(a->moves, 4) || !a->left || !aligned(a->left, 4)) return UZIP_EINVAL;
    if (!valid_pages(a->pages, a->seqs, a->entries) || a->rows < 1 || a->rows > 65535 || a->reserved) return UZIP_EINVAL;
    if (a->table_stride < 0 || a->table_stride > (1ll << 40)) return UZIP_EINVAL;
    if (a->page < 16 || a->page > (1u << 30) || (a->page & (a->page - 1)) || (uint64_t)a->entries * a->page > (1u << 30) || a->room > (1u << 30)) return UZIP_EINVAL;
    if (compact ? a->parent || a->rows != a->seqs || a->room || a->out_length : !a->parent || !a->out_length || !aligned(a->out_length, 4)) return UZIP_EINVAL;
    if (a->out_table == a->table || (!compact && a->out_length == a->length)) return UZIP_EINVAL;       // read beside it
    if (!d_ws || !aligned(d_ws, 16)) return UZIP_EINVAL;
    const PagesWs ws = pages_ws(a->pages, a->seqs, a->entries);
    if (ws_bytes < ws.bytes) return UZIP_ENOSPC;
    PageParams p;
    memset(&p, 0, sizeof p);
    p.table = a->table, p.length = a->length, p.parent = a->parent, p.held = a->held, p.t0 = a->table_stride;
    p.out_table = a->out_table, p.out_length = a->out_length, p.moves = a->moves, p.left = a->left;
    char *w = static_cast<char *>(d_ws);
    p.mark = reinterpret_cast<uint32_t *>(w);
    p.first = compact ? nullptr : reinterpret_cast<uint32_t *>(w + ws.off_first);
    p.given = reinterpret_cast<int32_t *>(w + ws.off_given);
    p.offset = reinterpret_cast<int32_t *>(w + ws.off_offset);
    p.rows = (int)a->rows, p.seqs = (int)a->seqs, p.entries = (int)a->entries, p.pages = (int)a->pages;
    p.shift = __builtin_ctz(a->page), p.room = (int)a->room;
    p.compact = compact;
    const uint64_t cells = (uint64_t)a->seqs * a->entries;
    p.most = (int)(cells < a->pages / 2 ? cells : a->pages / 2);
    const int parts = (p.entries + kPageThreads - 1) / kPageThreads;
    const unsigned grid = (unsigned)(p.seqs * parts);
    k_pages_clear<<<(unsigned)((p.pages + kPageThreads - 1) / kPageThreads), kPageThreads, 0, s>>>(p);
    k_pages_mark<<<grid, kPageThreads, 0, s>>>(p, parts);
    if (compact) {
        k_compact_plan<<<1, kPlanThreads, 0, s>>>(p);
        k_compact_fill<<<grid, kPageThreads, 0, s>>>(p, parts);
    } else {
        k_fork_plan<<<1, kPlanThreads, 0, s>>>(p);
        k_fork_fill<<<grid, kPageThreads, 0, s>>>(p, parts);
    }
    UZIP_KV_LAUNCH_CHECK("k_pages");
    return UZIP_OK;
}

}  // namespace
}  // namespace uzip_kv

extern "C" {

uint64_t uzip_kv_verify_workspace_bytes(uint32_t seqs, uint32_t nodes, uint32_t vocab)
{
    return uzip_kv::valid_verify(seqs, nodes, vocab) ? uzip_kv::verify_ws(seqs, nodes, vocab).bytes : 0;
}

int uzip_kv_verify(const uzip_kv_verify_args_t *a, void *d_ws, uint64_t ws_bytes, hipStream_t s)
{
    using namespace uzip_kv;
    if (!a || a->reserved || !valid_verify(a->seqs, a->nodes, a->vocab) || a->dtype > UZIP_KV_F32) return UZIP_EINVAL;
    const uint32_t es = a->dtype == UZIP_KV_F32 ? 4 : 2;
    if (!a->target || !aligned(a->target, es) || !aligned(a->draft, es) || !a->tokens || !aligned(a->tokens, 4)) return UZIP_EINVAL;
    if (!aligned(a->parent, 4) || !aligned(a->drafted, 4) || !a->uniform || !aligned(a->uniform, 4)) return UZIP_EINVAL;
    if (!a->path || !aligned(a->path, 4) || !a->count || !aligned(a->count, 4) || !a->token || !aligned(a->token, 4)) return UZIP_EINVAL;
    for (int i = 0; i < 2; i++)
        if (a->target_stride[i] < 0 || a->target_stride[i] > (1ll << 40) || a->draft_stride[i] < 0 || a->draft_stride[i] > (1ll << 40)) return UZIP_EINVAL;
    if (a->tokens_stride < 0 || a->parent_stride < 0 || a->uniform_stride < 0) return UZIP_EINVAL;
    if (!d_ws || !aligned(d_ws, 16)) return UZIP_EINVAL;
    const VerifyWs ws = verify_ws(a->seqs, a->nodes, a->vocab);
    if (ws_bytes < ws.bytes) return UZIP_ENOSPC;
    VerifyParams p;
    memset(&p, 0, sizeof p);
    p.p = static_cast<const char *>(a->target), p.q = static_cast<const char *>(a->draft);
    p.p0 = a->target_stride[0] * es, p.p1 = a->target_stride[1] * es;
    p.q0 = a->draft_stride[0] * es, p.q1 = a->draft_stride[1] * es;
    p.tokens = a->tokens, p.parent = a->parent, p.drafted = a->drafted, p.uniform = a->uniform;
    p.tok0 = a->tokens_stride, p.par0 = a->parent_stride, p.u0 = a->uniform_stride;
    p.path = a->path, p.count = a->count, p.token = a->token;
    p.T = (int)a->nodes, p.V = (int)a->vocab;
    p.segs = (p.V + kSeg - 1) / kSeg;
    // a segment a wave while there are workgroups to spare, four a CU
    const int64_t most = (p.segs + kVerifyWaves - 1) / kVerifyWaves, want = (4 * kCUs + a->seqs - 1) / a->seqs;
    p.slices = (int)(most < want ? most : want);
    // Two launches that make one more sum, where rows are long and some of the
    // sequences will ask for sums again and again. Trees of 32 nodes over 131072
    // tokens, calls' means over 12 drawings and without: 4 of them 27 and 28 us, 16
    // 38 and 55, 32 50 and 70; 16 over 70000 39 and 43. One tree (23 us) and 64
    // over 50000 (57) do without.
    p.seqs = (int)a->seqs;
    p.rounds = a->draft && a->parent && p.T > 2 && p.segs >= 64 && p.seqs >= 4 && p.seqs <= 32 ? 2 : 0;
    char *w = static_cast<char *>(d_ws);
    p.sums = reinterpret_cast<double *>(w);
    p.state = reinterpret_cast<Walked *>(w + ws.off_state);
    p.rejected = reinterpret_cast<int32_t *>(w + ws.off_rejected);
    if (a->dtype == UZIP_KV_F32) return run_verify<2>(p, (int)a->seqs, s);
    return a->dtype == UZIP_KV_F16 ? run_verify<kF16>(p, (int)a->seqs, s) : run_verify<kBF16>(p, (int)a->seqs, s);
}

int uzip_kv_accept(const uzip_kv_cache_t *cache, const uzip_kv_accept_args_t *a, hipStream_t s)
{
    using namespace uzip_kv;
    if (!a || a->reserved || !valid_cache(cache) || cache->k == cache->v) return UZIP_EINVAL;
    if (!a->length || !aligned(a->length, 4) || !a->path || !aligned(a->path, 4) || !a->count || !aligned(a->count, 4)) return UZIP_EINVAL;
    if (a->nodes < 1 || a->nodes > (uint32_t)kNodes || a->path_stride < 0) return UZIP_EINVAL;
    AcceptParams p;
    memset(&p, 0, sizeof p);
    p.c = view_of(cache);
    p.length = a->length, p.path = a->path, p.count = a->count, p.path0 = a->path_stride;
    p.T = (int)a->nodes, p.H = (int)cache->heads, p.per = (int)cache->dim / 8;
    p.parts = (2 * p.H * p.per + kAcceptThreads - 1) / kAcceptThreads;
    if ((uint64_t)cache->seqs * p.parts * kAcceptThreads >= kLaunchThreads) return UZIP_EINVAL;
    const unsigned grid = (unsigned)(cache->seqs * p.parts);
    if (elem_size((int)cache->dtype) == 2) k_accept<u32x4><<<grid, kAcceptThreads, 0, s>>>(p);
    else k_accept<u32x2><<<grid, kAcceptThreads, 0, s>>>(p);
    UZIP_KV_LAUNCH_CHECK("k_accept");
    return UZIP_OK;
}

uint64_t uzip_kv_pages_workspace_bytes(uint32_t pages, uint32_t seqs, uint32_t entries)
{
    return uzip_kv::valid_pages(pages, seqs, entries) ? uzip_kv::pages_ws(pages, seqs, entries).bytes : 0;
}

int uzip_kv_fork(const uzip_kv_pages_t *a, void *d_ws, uint64_t ws_bytes, hipStream_t s)
{
    return uzip_kv::plan_pages(a, false, d_ws, ws_bytes, s);
}

int uzip_kv_compact(const uzip_kv_pages_t *a, void *d_ws, uint64_t ws_bytes, hipStream_t s)
{
    return uzip_kv::plan_pages(a, true, d_ws, ws_bytes, s);
}

int uzip_kv_copy_pages(const int32_t *moves, uint32_t count, const uzip_kv_pool_t *pools, uint32_t n, uint32_t pages, hipStream_t s)
{
    using namespace uzip_kv;
    if (!moves || !aligned(moves, 4) || count > (1u << 30) || !pools || n < 1 || n > (uint32_t)kPools || pages < 1 || pages > 0x7fffffffu) return UZIP_EINVAL;
    uint64_t bits = 0;
    for (uint32_t i = 0; i < n; i++) {
        const uzip_kv_pool_t &q = pools[i];
        if (!q.data || q.n[0] < 1 || q.n[1] < 1 || q.run < 1 || q.run > (1u << 30) || q.reserved) return UZIP_EINVAL;
        if (q.page_stride < 0 || q.page_stride > (1ll << 42) || q.stride[0] < 0 || q.stride[0] > (1ll << 42) || q.stride[1] < 0 || q.stride[1] > (1ll << 42)) return UZIP_EINVAL;
        if ((uint64_t)q.n[0] * q.n[1] > (1u << 30) || (uint64_t)q.n[0] * q.n[1] * q.run > (1u << 30)) return UZIP_EINVAL;
        bits |= (uintptr_t)q.data | (uint64_t)q.page_stride | q.run | (q.n[0] > 1 ? (uint64_t)q.stride[0] : 0) | (q.n[1] > 1 ? (uint64_t)q.stride[1] : 0);
    }
    if (count == 0) return UZIP_OK;
    const uint32_t unit = !(bits & 15) ? 16 : !(bits & 3) ? 4 : 1;
    CopyParams p;
    memset(&p, 0, sizeof p);
    p.pages = pages;
    for (uint32_t i = 0; i < n; i++) {
        const uzip_kv_pool_t &q = pools[i];
        Pool &o = p.pool[i];
        o.data = static_cast<char *>(q.data);
        o.page = q.page_stride, o.s0 = q.stride[0], o.s1 = q.stride[1];
        o.n0 = q.n[0], o.n1 = q.n[1], o.run = q.run / unit;
        o.units = o.n0 * o.n1 * o.run;
        o.parts = (o.units + kCopied * kPageThreads - 1) / (kCopied * kPageThreads);
        p.parts += o.parts;
    }
    p.pools = (int)n;
    // as many moves a launch as it can hold: at most 2^20 workgroups each of 8 pools
    const uint32_t most = (uint32_t)((kLaunchThreads - 1) / kPageThreads / p.parts);
    for (uint32_t first = 0; first < count; first += most) {
        const unsigned grid = (count - first < most ? count - first : most) * p.parts;
        p.moves = moves + 2 * (int64_t)first;
        if (unit == 16) k_copy_pages<u32x4><<<grid, kPageThreads, 0, s>>>(p);
        else if (unit == 4) k_copy_pages<uint32_t><<<grid, kPageThreads, 0, s>>>(p);
        else k_copy_pages<uint8_t><<<grid, kPageThreads, 0, s>>>(p);
        UZIP_KV_LAUNCH_CHECK("k_copy_pages");
    }
    return UZIP_OK;
}

}  // extern "C"

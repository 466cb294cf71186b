// nq_verify_drafts.cu -- drafted tokens against the model's probabilities, from given random numbers.
//
// A request's walk through its tree needs one probability of each draft, at the draft's parent and token: both are known before the
// walk, so a warp loads them all at once and walks in registers.  Only what follows a rejection needs the vocabulary: the sum of what
// is left, w = max(p - A q, 0), where A adds up the S of the node's rejections (max(max(p - a, 0) - b, 0) = max(p - a - b, 0), so
// no w is ever stored), and in the end the token where the running sum of w passes its part of the whole.
//
// A cluster of blocks takes a request, each a part of the vocabulary.  The first block loads what the walk needs, 32 nodes at a time, and
// writes it into every block's shared memory; from there all warps of all blocks walk alike, so that nobody waits to be told what to sum.
// Each block forms its part of a sum and writes that into every other's shared memory; after a barrier of the cluster all know the
// whole and walk on, and in the end the block whose part holds the token finds it.  What decides how often the blocks meet comes from
// that one load, so that inputs that change meanwhile, by mistake, cannot part them.
//
// Sums decide between whole numbers, so they are off by no more than 2^-37 of the sum of p for each rejection and one: 2^-38 of themselves
// for the additions (see Sums), 2^-45 for a term's and A's own roundings, and an error of A only shrinks, since more taken leaves less.
// That is no fraction of what is left: with a draft near the model p - A q is small and has p's roundings (S = 2e-7 has 30 bits), but
// then it is as seldom needed.  The GPU's 64-bit units are too slow for that (used for no more
// than the threads' totals and the search they took four fifths of the time), so a number that matters is the sum of two fp32: an
// addition's rounding error is found by Knuth's two-sum, a product's by a fused multiply-add.
//
// Measured (median of graph replays): one request, a chain of 5 drafts, 32000 tokens in bf16 9.1 us: the launch, 1.7 us of loads for the
// walk (three after one another), 0.6 us for each barrier, 1.3 us of sum, 3 us of search, all latency; every further sum 2.6 us, of
// 128256 tokens in fp32 4.8 us.  64 requests, 128256 tokens in fp32: 18.6 us with one sum (3.5 TB/s of p and q), 12 us for a further one
// of all (5.5 TB/s, the rows come from the L2 in part); sampled trees of 16 35 us, 3 to 3.6 sums on average.  256 chains of 3 drafts 63 us.
// Chosen drafts, 256 requests, 32000 tokens in fp32 18 us.
// At the ends of the range (one request, 32000 tokens in fp32, calls timed by events): a chain of 256 accepted drafts 68 us, of 4096 0.79 ms;
// a star of 256 chosen drafts that are all rejected 0.14 ms, of 1024 0.76 ms, of 4096 8.6 ms, since each draft is held against all earlier
// ones for a repeated token, and past 64 rejected tokens in a warp's part every vector is held against all of them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "nq_paged.h"
#include "nq_paged_cluster.cuh"

namespace nq {
namespace {

// 1024 threads on a multiprocessor: four blocks, so that 64 requests' clusters all run at once.  (Blocks of 512 threads take 1.2 to 2
// times as long for 64 requests and more, of 128 up to 1.3 times for few, clusters of 16 such 4% less to 7% more; of 16 blocks of 256 10% to
// 20% less for few requests and up to 1.5 times for many.)
constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32, kBlocksPerSm = 4;
constexpr int kMostBlocks = 8;       // of a cluster
constexpr int kRejectedTokens = 64;  // of a warp's part of the vocabulary

struct VerifyArgs {
    const void *probs, *draft_probs;
    int64_t probs_stride, draft_stride;
    const int32_t *drafts, *parents, *q_start;
    const float* uniform;
    int32_t *accepted, *path, *tokens_out;
    int vocab, tokens;
};

// -------------------------------------------------------------------- values

__device__ __forceinline__ float weight_of(float x) { return fmaxf(x, 0.0f); }  // NaN counts as 0

template <typename T>
struct Vec {  // 16 bytes of a row
    static constexpr int N = 16 / sizeof(T);
    uint32_t w[4];
    __device__ __forceinline__ float2 pair(int i) const {  // elements 2i, 2i + 1
        if constexpr (sizeof(T) == 4)
            return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else if constexpr (std::is_same<T, __half>::value)
            return __half22float2(*reinterpret_cast<const __half2*>(w + i));
        else
            return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
};
template <typename T>
__device__ __forceinline__ Vec<T> as_vec(uint4 x) {
    return Vec<T>{{x.x, x.y, x.z, x.w}};
}
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* p) {
    return as_vec<T>(__ldg(reinterpret_cast<const uint4*>(p)));
}
template <typename T>
__device__ __forceinline__ float load_one(const T* p) {
    if constexpr (std::is_same<T, float>::value)
        return __ldg(p);
    else if constexpr (std::is_same<T, __half>::value)
        return __half2float(__ushort_as_half(__ldg(reinterpret_cast<const unsigned short*>(p))));
    else
        return __uint_as_float(uint32_t(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
}

// A number as the sum of two fp32, the second no more than the first's rounding.
struct Pair {
    float s, e;
};
__device__ __forceinline__ Pair normal(float s, float e) {  // |s| >= |e|
    const float t = s + e;
    return Pair{t, e - (t - s)};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    const float t = a.s + b.s, v = t - a.s;
    return normal(t, ((a.s - (t - v)) + (b.s - v)) + (a.e + b.e));
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b) { return a + Pair{-b.s, -b.e}; }
__device__ __forceinline__ Pair operator*(Pair a, float x) {
    const float h = a.s * x;
    return normal(h, __fmaf_rn(a.s, x, -h) + a.e * x);
}
__device__ __forceinline__ bool operator<(Pair a, Pair b) { return a.s < b.s || (a.s == b.s && a.e < b.e); }
__device__ __forceinline__ bool positive(Pair a) { return a.s > 0.0f; }
__device__ __forceinline__ Pair shfl_up(Pair a, int d) {
    return Pair{__shfl_up_sync(0xffffffffu, a.s, d), __shfl_up_sync(0xffffffffu, a.e, d)};
}
__device__ __forceinline__ Pair shfl(Pair a, int from) {
    return Pair{__shfl_sync(0xffffffffu, a.s, from), __shfl_sync(0xffffffffu, a.e, from)};
}
__device__ __forceinline__ uint64_t bits_of(Pair a) {
    return uint64_t(__float_as_uint(a.s)) | uint64_t(__float_as_uint(a.e)) << 32;
}

// Two fp32 in one operation.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.0f, -1.0f), a); }

// Two running sums side by side, with their rounding errors.  What is lost is the rounding of the errors' own sum: for each vector ten times
// 2^-48 of the running sum at most, and a thread adds 64 vectors of 2^19 tokens: 2^-38.
struct Sums {
    float2 s = {0.0f, 0.0f}, e = {0.0f, 0.0f};
    __device__ __forceinline__ void add(float2 x, float2 low) {
        const float2 t = add2(s, x), v = sub2(t, s);
        e = add2(e, add2(add2(sub2(s, sub2(t, v)), sub2(x, v)), low));
        s = t;
    }
    __device__ __forceinline__ void settle() {  // what the errors add up to goes over into the sums
        const float2 t = add2(s, e);
        e = sub2(e, sub2(t, s));
        s = t;
    }
    __device__ __forceinline__ Pair total() const { return normal(s.x, e.x) + normal(s.y, e.y); }
};

// 32 nodes of a request, from `first` on.
struct __align__(8) Nodes {
    int2 drafts[32];    // parent (-1: not to be walked to), token
    float2 chances[32];  // its random number, p at its parent and token
    float2 q[32];       // q there; q[0].y and q[1].y hold the request's first row and its rows, as whole numbers
};
constexpr int kNodeWords = sizeof(Nodes) / 8;

struct __align__(8) VerifyShared {
    Nodes nodes[2];             // by turns
    Pair part[2][kMostBlocks];  // of each block, by turns
    Pair warp[2][kVerifyWarps];  // of each warp's part; of its part of the warp's part that holds the token
    int rejected[kVerifyWarps][kRejectedTokens], rejected_count[kVerifyWarps];
};

// A row of p (and of q) as a warp of the cluster sees it.  Index order: the elements before the first 16-byte boundary, whole vectors
// in equal parts for all warps, the elements after the last boundary.
template <typename T, bool SAMPLED>
struct Slice {
    static constexpr int N = Vec<T>::N;
    const T *p, *q;
    int head, tail_at, vocab;  // tail_at: first element after the vectors
    int v0, v1;                // this warp's vectors
    bool first, last, together;  // together: q's vectors begin where p's do

    __device__ __forceinline__ Slice(const VerifyArgs& a, int row, int segment, int segments) {
        p = static_cast<const T*>(a.probs) + int64_t(row) * a.probs_stride;
        q = SAMPLED ? static_cast<const T*>(a.draft_probs) + int64_t(row) * a.draft_stride : nullptr;
        vocab = a.vocab;
        head = min(int((0 - reinterpret_cast<uintptr_t>(p)) & 15) / int(sizeof(T)), vocab);
        v0 = 0;
        v1 = (vocab - head) / N;
        tail_at = head + v1 * N;
        first = last = true;
        narrow(segment, segments);
        together = SAMPLED && ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    }
    // To part i of `parts` of what it is.
    __device__ __forceinline__ void narrow(int i, int parts) {
        const int n = v1 - v0;
        v1 = v0 + int(int64_t(n) * (i + 1) / parts);
        v0 += int(int64_t(n) * i / parts);
        first = first && i == 0;
        last = last && i == parts - 1;
    }
    // The tokens that this warp's part begins and ends with.
    __device__ __forceinline__ int begin() const { return first ? 0 : head + v0 * N; }
    __device__ __forceinline__ int end() const { return last ? vocab : head + v1 * N; }
    __device__ __forceinline__ const T* at_p(int v) const { return p + head + int64_t(v) * N; }
    __device__ __forceinline__ const T* at_q(int v) const { return q + head + int64_t(v) * N; }
    __device__ __forceinline__ Vec<T> load_p(int v) const { return load_vec(at_p(v)); }
    __device__ __forceinline__ Vec<T> load_q(int v) const {
        const T* from = at_q(v);
        if (together) return load_vec(from);
        Vec<T> x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4)
                x.w[i] = __ldg(reinterpret_cast<const uint32_t*>(from) + i);
            else
                x.w[i] = __ldg(reinterpret_cast<const unsigned short*>(from) + 2 * i) |
                         uint32_t(__ldg(reinterpret_cast<const unsigned short*>(from) + 2 * i + 1)) << 16;
        }
        return x;
    }
};

// The tokens of rejected drafts (without draft probabilities), of which nothing is left: those of a warp's part, or, when they
// are too many to be kept, all of the request's nodes after `node`.
struct Rejected {
    const int* tokens;
    int count;
    const int32_t *parents, *drafts;  // of the request
    int node, n;  // node < 0: none of them counts
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        if (count <= kRejectedTokens) {
            for (int j = 0; j < count; ++j) f(tokens[j]);
        } else {
            for (int j = node + 1; j < n; ++j)
                if (parents[j] == node) f(drafts[j]);
        }
    }
    // The vector that begins at token x, without them.
    template <typename T>
    __device__ __forceinline__ void clear(Vec<T>& v, int x) const {
        each([&](int token) {
            const int64_t i = int64_t(token) - x;
            if (i < 0 || i >= Vec<T>::N) return;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (int(i) * int(sizeof(T)) / 4 == k) v.w[k] &= sizeof(T) == 4 ? 0u : i & 1 ? 0xffffu : 0xffff0000u;
        });
    }
    __device__ __forceinline__ bool has(int x) const {
        bool found = false;
        each([&](int token) { found |= token == x; });
        return found;
    }
};

// What is left of two tokens' probabilities, d + l: p - A q with its rounding errors.  Where p is above A q, p - d is exact, and where it
// is not, q is cut down to what leaves nothing.
struct Left2 {
    float2 d, l;
};
template <bool SAMPLED, bool ONE>
__device__ __forceinline__ Left2 left_of(float2 p, float2 q, Pair taken) {
    const float2 zero = make_float2(0.0f, 0.0f);
    p = make_float2(weight_of(p.x), weight_of(p.y));
    if constexpr (!SAMPLED) {
        return Left2{p, zero};
    } else {
        q = make_float2(weight_of(q.x), weight_of(q.y));
        if constexpr (ONE) {  // one rejection, A = 1
            q = make_float2(fminf(q.x, p.x), fminf(q.y, p.y));
            const float2 d = sub2(p, q);
            return Left2{d, sub2(sub2(p, d), q)};
        } else {
            const float2 high = make_float2(taken.s, taken.s), low = make_float2(taken.e, taken.e);
            const float2 h = fma2(high, q, zero);  // A q, and what its rounding left
            const float2 below = fma2(low, q, fma2(high, q, make_float2(-h.x, -h.y)));
            const float2 d = sub2(p, h), l = sub2(sub2(sub2(p, d), h), below);
            const bool x = d.x + l.x > 0.0f, y = d.y + l.y > 0.0f;
            return Left2{make_float2(x ? d.x : 0.0f, y ? d.y : 0.0f), make_float2(x ? l.x : 0.0f, y ? l.y : 0.0f)};
        }
    }
}
// ... of one of the tokens before or after the vectors.
template <typename T, bool SAMPLED>
__device__ __forceinline__ Pair edge_left(const Slice<T, SAMPLED>& s, Pair taken, const Rejected& rejected, int x) {
    if (!SAMPLED && rejected.has(x)) return Pair{0.0f, 0.0f};
    const float p = load_one(s.p + x), q = SAMPLED ? load_one(s.q + x) : 0.0f;
    const Left2 w = left_of<SAMPLED, false>(make_float2(p, 0.0f), make_float2(q, 0.0f), taken);
    return normal(w.d.x, w.l.x);
}
template <typename T, bool SAMPLED, bool ONE>
__device__ __forceinline__ void add_vec(Sums& sums, const Vec<T>& p, const Vec<T>& q, Pair taken) {
#pragma unroll
    for (int i = 0; i < Vec<T>::N / 2; ++i) {
        const Left2 w = left_of<SAMPLED, ONE>(p.pair(i), SAMPLED ? q.pair(i) : p.pair(i), taken);
        sums.add(w.d, w.l);
    }
    sums.settle();
}

constexpr int kRing = 5, kFindAhead = 2;  // vectors of each row that a thread has on their way

// A thread's next vectors; those past the warp's part are zeros, which count for nothing.
template <int AHEAD, typename T, bool SAMPLED>
__device__ __forceinline__ void load_ahead(const Slice<T, SAMPLED>& s, const Rejected& rejected, int v, Vec<T> (&p)[AHEAD],
                                           Vec<T> (&q)[AHEAD]) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
        p[u] = q[u] = Vec<T>{{0, 0, 0, 0}};
        if (v + 32 * u < s.v1) {
            p[u] = s.load_p(v + 32 * u);
            if (SAMPLED) q[u] = s.load_q(v + 32 * u);
        }
    }
    if (!SAMPLED && rejected.count > 0)
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) rejected.clear(p[u], s.head + (v + 32 * u) * Vec<T>::N);
}

// Sixteen bytes of a row into this thread's place, as part of the thread's open group of copies.
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(to))), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {  // all groups but the last N have ended
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's vectors come through a ring in shared memory, kRing of them ahead of each thread, which reads only what it copied itself.
template <typename T, bool SAMPLED, bool ONE>
__device__ __forceinline__ Pair sum_slice(const Slice<T, SAMPLED>& s, Pair taken, const Rejected& rejected, int lane, uint4* ring) {
    Pair edges{0.0f, 0.0f};
    if (s.first && lane < s.head) edges = edge_left(s, taken, rejected, lane);
    if (s.last && s.tail_at + lane < s.vocab) edges = edges + edge_left(s, taken, rejected, s.tail_at + lane);
    Sums sums;
    constexpr int ROWS = SAMPLED ? 2 : 1;
    auto ask = [&](int v, int stage) {
        if (v < s.v1) {
            copy_async(ring + (stage * ROWS) * 32 + lane, s.at_p(v));
            if (SAMPLED && s.together) copy_async(ring + (stage * ROWS + 1) * 32 + lane, s.at_q(v));
        }
        copy_group();
    };
    int v = s.v0 + lane;
#pragma unroll
    for (int i = 0; i < kRing; ++i) ask(v + 32 * i, i);
    for (int stage = 0; v < s.v1; v += 32, stage = stage + 1 == kRing ? 0 : stage + 1) {
        copy_wait<kRing - 1>();
        Vec<T> p = as_vec<T>(ring[(stage * ROWS) * 32 + lane]), q = p;
        if (SAMPLED) q = s.together ? as_vec<T>(ring[(stage * ROWS + 1) * 32 + lane]) : s.load_q(v);
        if (!SAMPLED && rejected.count > 0) rejected.clear(p, s.head + v * Vec<T>::N);
        ask(v + 32 * kRing, stage);
        add_vec<T, SAMPLED, ONE>(sums, p, q, taken);
    }
    copy_wait<0>();
    return edges + sums.total();
}
template <typename T, bool SAMPLED>
__device__ __forceinline__ void warp_sum(const Slice<T, SAMPLED>& s, Pair taken, const Rejected& rejected, int lane, uint4* ring,
                                         Pair* to) {
    Pair sum;  // a loop for A = 1, which most sums have: one loop that tests A takes up to 5% longer
    if (SAMPLED && taken.s == 1.0f && taken.e == 0.0f)
        sum = sum_slice<T, SAMPLED, true>(s, taken, rejected, lane, ring);
    else
        sum = sum_slice<T, SAMPLED, false>(s, taken, rejected, lane, ring);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        sum = sum + Pair{__shfl_xor_sync(0xffffffffu, sum.s, d), __shfl_xor_sync(0xffffffffu, sum.e, d)};
    if (lane == 0) *to = sum;
}

// The sum of n numbers, at most MOST, for every lane of a warp.
template <int MOST>
__device__ __forceinline__ Pair sum_few(const Pair* x, int n, int lane) {
    Pair sum = (lane & (MOST - 1)) < n ? x[lane & (MOST - 1)] : Pair{0.0f, 0.0f};
#pragma unroll
    for (int d = MOST / 2; d > 0; d >>= 1)
        sum = sum + Pair{__shfl_xor_sync(0xffffffffu, sum.s, d), __shfl_xor_sync(0xffffffffu, sum.e, d)};
    return sum;
}

// Which of n parts the target lies in, the last with anything in it when the additions' roundings leave none; `before` becomes
// what the parts before it have.
__device__ __forceinline__ int part_of(const Pair* parts, int n, Pair target, Pair& before) {
    Pair upto = before;
    int found = 0;
    for (int i = 0; i < n; ++i) {
        if (positive(parts[i])) {
            found = i;
            before = upto;
        }
        upto = upto + parts[i];
        if (target < upto) break;
    }
    return found;
}

// The lowest token of a warp's part whose running sum, from `before` on, is above the target, -1 when the additions' roundings leave
// none; LAST: the last token with anything left.
template <typename T, bool SAMPLED, bool LAST>
__device__ __forceinline__ int find_token(const Slice<T, SAMPLED>& s, Pair taken, const Rejected& rejected, int lane, Pair before,
                                          Pair target) {
    int token = -1;
    // A lane's `mine` is what its tokens have together, `upto` what the lanes up to it have; `pick` goes through its tokens from a
    // running sum.  Returns whether the search is over.
    auto step = [&](Pair mine, Pair upto, auto pick) {
        const uint32_t hit = __ballot_sync(0xffffffffu, positive(mine) && (LAST || target < before + upto));
        if (hit) {
            const int from = LAST ? 31 - __clz(hit) : __ffs(hit) - 1;
            const Pair last = shfl_up(upto, 1);
            int got = -1;
            if (lane == from) got = pick(lane > 0 ? before + last : before);
            token = __shfl_sync(0xffffffffu, got, from);
        }
        before = before + shfl(upto, 31);
        return !LAST && hit;
    };
    auto edge = [&](int x, int end) {
        const Pair mine = x < end ? edge_left(s, taken, rejected, x) : Pair{0.0f, 0.0f};
        Pair upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Pair y = shfl_up(upto, d);
            if (lane >= d) upto = y + upto;
        }
        return step(mine, upto, [&](Pair) { return x; });
    };
    if (s.first && edge(lane, s.head)) return token;
    for (int v = s.v0 + lane; v - lane < s.v1; v += 32 * kFindAhead) {
        Vec<T> p[kFindAhead], q[kFindAhead];
        Pair mine[kFindAhead], upto[kFindAhead];
        load_ahead(s, rejected, v, p, q);
#pragma unroll
        for (int u = 0; u < kFindAhead; ++u) {
            Sums sums;
            add_vec<T, SAMPLED, false>(sums, p[u], q[u], taken);
            mine[u] = upto[u] = sums.total();
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)  // side by side: one after the other they would be all latency
#pragma unroll
            for (int u = 0; u < kFindAhead; ++u) {
                const Pair y = shfl_up(upto[u], d);
                if (lane >= d) upto[u] = y + upto[u];
            }
#pragma unroll
        for (int u = 0; u < kFindAhead; ++u) {
            const bool over = step(mine[u], upto[u], [&](Pair run) {
                int got = -1;
                bool done = false;
#pragma unroll
                for (int i = 0; i < Vec<T>::N / 2; ++i) {
                    const Left2 w = left_of<SAMPLED, false>(p[u].pair(i), SAMPLED ? q[u].pair(i) : p[u].pair(i), taken);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const Pair y = normal(k ? w.d.y : w.d.x, k ? w.l.y : w.l.x);
                        if (!positive(y) || done) continue;
                        got = s.head + (v + 32 * u) * Vec<T>::N + 2 * i + k;
                        run = run + y;
                        done = !LAST && target < run;
                    }
                }
                return got;
            });
            if (over) return token;
        }
    }
    if (s.last) edge(s.tail_at + lane, s.vocab);
    return token;
}

template <typename T, bool SAMPLED>
__global__ void __launch_bounds__(kVerifyThreads, kBlocksPerSm) verify_drafts_kernel(const VerifyArgs a) {
    __shared__ VerifyShared sh;
    __shared__ uint4 rings[kVerifyWarps][kRing * (SAMPLED ? 2 : 1) * 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, V = a.vocab;
    const uint32_t rank = cluster_rank(), blocks = cluster_size();
    const int r = blockIdx.x / blocks;
    uint4* ring = rings[warp];
    cluster_arrive();  // the blocks' shared memory exists
    const int segments = kVerifyWarps * int(blocks), segment = int(rank) * kVerifyWarps + warp;

    // ------------------------------------------------------------------ nodes
    int begin = 0, n = 0;
    int loaded = -1, parent = -1, drafted = -1;  // of node loaded + lane
    float u = 0.0f, p = 0.0f, q = 1.0f;
    int loads = 0;
    // Nodes i0 .. i0 + 31 for every warp of the cluster.  All call it together.
    auto load = [&](int i0) {
        loaded = i0;
        Nodes& nodes = sh.nodes[loads & 1];
        if (rank == 0) {
            if (warp == 0) {
                if (loads == 0) {
                    begin = min(max(a.q_start[r], 0), a.tokens);
                    n = max(min(max(a.q_start[r + 1], 0), a.tokens) - begin, 0);
                }
                const int i = i0 + lane;
                parent = drafted = -1;
                if (i < n && i > 0) {
                    parent = a.parents[begin + i];
                    drafted = a.drafts[begin + i];
                    u = weight_of(a.uniform[begin + i]);
                    if (parent < 0 || parent >= i || drafted < 0 || drafted >= V) {
                        parent = -1;
                    } else {
                        const int64_t row = begin + parent;
                        p = weight_of(load_one(static_cast<const T*>(a.probs) + row * a.probs_stride + drafted));
                        if (SAMPLED) q = weight_of(load_one(static_cast<const T*>(a.draft_probs) + row * a.draft_stride + drafted));
                    }
                }
                nodes.drafts[lane] = make_int2(parent, drafted);
                nodes.chances[lane] = make_float2(u, p);
                nodes.q[lane] = make_float2(q, __int_as_float(lane == 0 ? begin : n));
            }
            __syncthreads();
            if (loads == 0) cluster_wait();
            if (warp > 0 && warp < int(blocks)) {  // a warp for each other block
                uint64_t* place = reinterpret_cast<uint64_t*>(&nodes);
#pragma unroll
                for (int i = 0; i < kNodeWords; i += 32) store_remote(place + i + lane, warp, place[i + lane]);
            }
            __syncwarp();
        } else if (loads == 0) {
            cluster_wait();
        }
        cluster_arrive();
        cluster_wait();
        ++loads;
        parent = nodes.drafts[lane].x;
        drafted = nodes.drafts[lane].y;
        u = nodes.chances[lane].x;
        p = nodes.chances[lane].y;
        q = nodes.q[lane].x;
        begin = __float_as_int(nodes.q[0].y);
        n = __float_as_int(nodes.q[1].y);
    };
    load(0);
    if (n == 0) {
        if (rank == 0 && threadIdx.x == 0) a.accepted[r] = 0;
        return;
    }

    // --------------------------------------------------------------- the walk
    const bool writes = rank == 0 && warp == 0 && lane == 0;
    int cur = 0, at = 1, kept = 1;
    Pair taken{0.0f, 0.0f}, total{1.0f, 0.0f};
    bool pending = false;  // a sum that the next draft needs, or the token that follows
    // Up to a rejection that another draft follows (false), or to the end (true).
    auto walk = [&]() {
        while (at < n) {
            const int i0 = at & ~31;
            if (loaded != i0) load(i0);
            const uint32_t mine = __ballot_sync(0xffffffffu, parent == cur && i0 + lane >= at);
            if (mine == 0) {
                at = i0 + 32;
                continue;
            }
            if (pending) {
                pending = false;
                return false;
            }
            const int from = __ffs(mine) - 1, node = i0 + from;
            const int token = __shfl_sync(0xffffffffu, drafted, from);
            const float uu = __shfl_sync(0xffffffffu, u, from), qq = __shfl_sync(0xffffffffu, q, from);
            Pair w{__shfl_sync(0xffffffffu, p, from), 0.0f};
            if constexpr (SAMPLED) {
                w = w - taken * qq;
                if (!positive(w)) w = Pair{0.0f, 0.0f};
            } else {  // an earlier child with the same token has been rejected: nothing is left of it
                bool again = parent == cur && lane < from && drafted == token;
                for (int j = cur + 1 + lane; j < i0; j += 32)
                    again |= a.parents[begin + j] == cur && a.drafts[begin + j] == token;
                if (__any_sync(0xffffffffu, again)) w = Pair{0.0f, 0.0f};
            }
            at = node + 1;
            if (total * qq * uu < w) {
                if (writes) {
                    a.tokens_out[begin + kept - 1] = token;
                    a.path[begin + kept] = node;
                }
                ++kept;
                cur = node;
                taken = Pair{0.0f, 0.0f};
                total = Pair{1.0f, 0.0f};
            } else if (SAMPLED) {
                taken = taken + total;
                pending = true;
            } else {
                total = total - w;
            }
        }
        return true;
    };

    // ------------------------------------------------------------------- sums
    int turn = 0;
    // The sum over this block's part, into every block's shared memory; the whole after a barrier.
    auto sum = [&](int node, Pair less, const Rejected& rejected) {
        warp_sum(Slice<T, SAMPLED>(a, begin + node, segment, segments), less, rejected, lane, ring, sh.warp[0] + warp);
        __syncthreads();
        if (warp == 0) {
            const Pair mine = sum_few<kVerifyWarps>(sh.warp[0], kVerifyWarps, lane);
            if (lane < int(blocks)) store_remote(&sh.part[turn & 1][rank], lane, bits_of(mine));
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        return sum_few<kMostBlocks>(sh.part[turn++ & 1], int(blocks), lane);
    };
    Rejected rejected{sh.rejected[warp], 0, a.parents + begin, a.drafts + begin, 0, n};
    while (true) {
        const bool end = walk();
        if (!SAMPLED) {  // the walk is over: the node's children have all been rejected
            const Slice<T, SAMPLED> mine(a, begin + cur, segment, segments);
            rejected.node = cur;
            for (int j0 = cur + 1; j0 < n; j0 += 32) {
                const int j = j0 + lane, token = j < n && a.parents[begin + j] == cur ? a.drafts[begin + j] : -1;
                const bool here = token >= mine.begin() && token < mine.end();
                const uint32_t all = __ballot_sync(0xffffffffu, here);
                const int slot = rejected.count + __popc(all & ((1u << lane) - 1));
                if (here && slot < kRejectedTokens) sh.rejected[warp][slot] = token;
                rejected.count += __popc(all);
            }
            if (lane == 0) sh.rejected_count[warp] = rejected.count;
            __syncwarp();
        }
        total = sum(cur, taken, rejected);
        if (end) break;
    }
    Pair less = taken;
    if (!positive(total)) {  // nothing is left: the node's own probabilities
        rejected.count = 0;
        rejected.node = -1;
        less = Pair{0.0f, 0.0f};
        total = sum(cur, less, rejected);
    }

    // ------------------------------------------------- the token that follows
    const int last = begin + kept - 1;
    if (rank == 0) {
        if (threadIdx.x == 0) {
            a.accepted[r] = kept;
            a.path[begin] = 0;
            if (!positive(total)) a.tokens_out[last] = -1;
        }
        for (int k = kept + threadIdx.x; k < n; k += kVerifyThreads) a.path[begin + k] = a.tokens_out[begin + k] = -1;
    }
    if (!positive(total)) return;
    const Pair target = total * weight_of(a.uniform[begin]);
    Pair before{0.0f, 0.0f};
    if (part_of(sh.part[(turn - 1) & 1], int(blocks), target, before) != int(rank)) return;
    // The warp whose part it is in; that part in turn in equal parts for all the block's warps: one warp alone would be all latency.
    const int holder = part_of(sh.warp[0], kVerifyWarps, target, before);
    Slice<T, SAMPLED> x(a, begin + cur, int(rank) * kVerifyWarps + holder, segments);
    x.narrow(warp, kVerifyWarps);
    if (!SAMPLED) {
        rejected.tokens = sh.rejected[holder];
        if (rejected.node >= 0) rejected.count = sh.rejected_count[holder];
    }
    warp_sum(x, less, rejected, lane, ring, sh.warp[1] + warp);
    __syncthreads();
    if (part_of(sh.warp[1], kVerifyWarps, target, before) != warp) return;
    int token = find_token<T, SAMPLED, false>(x, less, rejected, lane, before, target);
    if (token < 0) token = find_token<T, SAMPLED, true>(x, less, rejected, lane, before, target);
    if (lane == 0) a.tokens_out[last] = token;
}

// Blocks of a cluster: so many that a thread has four vectors of a row, at most a portable cluster's eight; fewer, with up to sixteen
// vectors a thread, while there are more blocks than run at once (four on each of 152 multiprocessors).  8, 4, 2 blocks: 256
// requests, 32000 tokens in fp32, 38, 28, 25 us (chains of 3 drafts that were drawn), 50, 41, 43 (trees of 8), 37, 26, 21 (chosen);
// 128 requests 21, 16, 16, then 29, 25, 30, then 19, 15, 15; 128256 tokens in fp32, 128 requests, 38, 38, 37, then 54, 65, 86, then 34, 31, 38.
int cluster_blocks(int vocab, int size, int requests) {
    const int64_t vectors = int64_t(vocab) * size / 16;
    int blocks = 1;
    while (blocks < kMostBlocks && blocks * kVerifyThreads * 4 < vectors) blocks *= 2;
    while (blocks > 1 && int64_t(requests) * blocks > 152 * kBlocksPerSm && vectors <= blocks / 2 * kVerifyThreads * 16) blocks /= 2;
    return blocks;
}

template <typename T>
int launch_verify(const VerifyArgs& a, int requests, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(cluster_blocks(a.vocab, sizeof(T), requests));
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(requests) * attr.val.clusterDim.x);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = a.draft_probs ? cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T, true>, a)
                                        : cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T, false>, a);
    return e == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

}  // namespace
}  // namespace nq

extern "C" int nq_verify_drafts(const void* probs, int64_t probs_stride, const void* draft_probs, int64_t draft_stride,
                                int32_t dtype, int32_t vocab, const int32_t* drafts, const int32_t* parents,
                                const float* uniform, int32_t tokens, const int32_t* q_start, int32_t requests,
                                int32_t* accepted, int32_t* path, int32_t* tokens_out, void* stream) {
    if (dtype != NQ_F16 && dtype != NQ_BF16 && dtype != NQ_F32) return NQ_ERR_UNSUPPORTED;
    if (tokens < 0 || requests < 0 || requests > INT32_MAX / nq::kMostBlocks || vocab < 1 || vocab > INT32_MAX - 65536)
        return NQ_ERR_ARG;
    if (tokens > 1 && (probs_stride < vocab || (draft_probs && draft_stride < vocab))) return NQ_ERR_ARG;
    if (requests == 0) return NQ_OK;
    if (!q_start || !accepted) return NQ_ERR_ARG;
    if (tokens > 0 && (!probs || !drafts || !parents || !uniform || !path || !tokens_out)) return NQ_ERR_ARG;
    const uintptr_t size = dtype == NQ_F32 ? 4 : 2;
    if (!nq::paged_aligned(probs, size) || !nq::paged_aligned(draft_probs, size)) return NQ_ERR_ARG;
    for (const void* p : {static_cast<const void*>(drafts), static_cast<const void*>(parents),
                          static_cast<const void*>(uniform), static_cast<const void*>(q_start),
                          static_cast<const void*>(accepted), static_cast<const void*>(path),
                          static_cast<const void*>(tokens_out)})
        if (!nq::paged_aligned(p, 4)) return NQ_ERR_ARG;
    // a request's results are written while other requests' blocks read
    struct Range {
        uintptr_t at, bytes;
    };
    auto range = [](const void* p, uint64_t n) { return Range{reinterpret_cast<uintptr_t>(p), uintptr_t(n)}; };
    auto rows = [&](const void* p, int64_t stride) {  // as far as 64 bits go
        const unsigned __int128 n = p && tokens > 0 ? ((unsigned __int128)(tokens - 1) * uint64_t(tokens > 1 ? stride : 0) + vocab) * size : 0;
        return range(p, uint64_t(std::min<unsigned __int128>(n, UINT64_MAX - reinterpret_cast<uintptr_t>(p))));
    };
    const uint64_t bytes = uint64_t(tokens) * 4;
    const Range all[] = {range(accepted, uint64_t(requests) * 4), range(path, bytes), range(tokens_out, bytes),
                         range(drafts, bytes), range(parents, bytes), range(uniform, bytes),
                         range(q_start, (uint64_t(requests) + 1) * 4), rows(probs, probs_stride), rows(draft_probs, draft_stride)};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 9; ++j)
            if (all[i].bytes > 0 && all[j].bytes > 0 && all[i].at < all[j].at + all[j].bytes && all[j].at < all[i].at + all[i].bytes)
                return NQ_ERR_ARG;
    const nq::VerifyArgs a{probs,   draft_probs, probs_stride, draft_stride, drafts, parents, q_start,
                           uniform, accepted,    path,         tokens_out,   vocab,  tokens};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == NQ_F32) return nq::launch_verify<float>(a, requests, s);
    return dtype == NQ_F16 ? nq::launch_verify<__half>(a, requests, s) : nq::launch_verify<__nv_bfloat16>(a, requests, s);
}

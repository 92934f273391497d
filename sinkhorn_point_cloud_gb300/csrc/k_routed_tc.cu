// k_routed_tc.cu -- the routed layer for a few tokens on the tensor cores, 16-bit types.
//
// After the scores (k_routed.cu) one cooperative kernel, a CTA an SM, does the rest:
//   choose  the tokens' experts (few tokens: every CTA for itself), then every CTA each expert's list of tokens;
//   up      products gate_up x^T: an expert's rows are the M of a tcgen05.mma (64 gate rows and the 64 up rows that
//           belong to them), its tokens the N.  The units of all experts (16 KB of weights, K = 64, or twice that) are
//           dealt out evenly, so a CTA starts and ends inside a tile; it leaves a partial sum for each piece;
//   act     h = silu(gate) up of the joined pieces, as a sum of two numbers of the type;
//   down    products down h^T, the same way, both parts of h into one accumulator;
//   join    the weighted sum over a token's experts.
// The weights are read once and bound it.  They come by TMA through a ring of stages, 16 or 32 KB each, from a warp that waits
// for nothing but free stages: across the phases' grid barriers the next phase's weights are already on their way.
// Every wait is bounded; one that runs out ends the call with NaN outputs and the timeout status.
//
// bf16, H = 4096, F = 1408, 8 of 128 experts, 64 tokens: 650 us for 4.36 GB, 0.99 of the measured copy bandwidth.  H = 2048,
// F = 1024, 8 of 64 experts: one token 31.3 us for 101 MB (about 4.5 us until the first weights, 16 of weights, the rest waits of
// phases on one another), 8 tokens 98 us, 128 tokens 158 us (fp16 160; 0.75: the tokens' side of the units takes a third of
// the ring and more).
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "kernels.h"
#include "routed.cuh"
#include "tc_ptx.cuh"

namespace sot {

namespace {

constexpr int LOADERS = 8;  // warps that fetch the tokens' side, a unit each in turn (as many of them as the ring has stages)
constexpr int NWARP = 6 + LOADERS, NT = NWARP * 32;
constexpr int W_PRODUCER = 0, W_MMA = 1, W_EPI = 2, W_LOAD = 6;  // first warps of each role (4 in the epilogue)
constexpr int WORKERS = (4 + LOADERS) * 32;                      // threads of the last two
constexpr int KSTEP = 64, A_BYTES = 128 * KSTEP * 2;  // columns of a swizzled row (128 bytes), 128 rows of them
constexpr int MIN_STAGES = 3, MAX_STAGES = 12, HEAD = 3;
constexpr unsigned long long WAIT_NS = 2000000000ull;
constexpr int PHASES = 2;  // 0: up, 1: down
constexpr int FUSED_PAIRS = 16;

struct Layout {  // byte offsets in dynamic shared memory (from a 1024-byte boundary, where the ring is)
    int ring, most;  // bytes of the ring; tokens that an expert may have, in sixteens
    int bars, weight, toks, list, act, id, info, mask, place, total;
};
// Numbers of the type that h is the sum of.  One alone would be most of the output's error (bf16: 2.4e-3 of it, where its
// own rounding makes 1.6e-3); two cost 0 to 5 % (one token 31.3 us, was 30.7; 37 fp16 tokens of 10 experts 44.6, was 42.5).
constexpr int PARTS = 2;

// How the ring is cut for experts of at most npad tokens: weights, then the parts of the tokens' side of each slice.
struct Cut {
    int npad, wide;  // wide: slices of KSTEP columns in a unit: two where that leaves four stages (a unit costs the
                     // multiplying thread 250 ns whatever its width), else one
    int part, stage, stages;
    __host__ __device__ Cut(int npad_, int ring) : npad(npad_), part(npad_ * KSTEP * 2) {
        wide = 4 * 2 * (A_BYTES + PARTS * part) <= ring ? 2 : 1;
        stage = wide * (A_BYTES + PARTS * part);
        stages = ring / stage;
        if (stages > MAX_STAGES) stages = MAX_STAGES;
    }
};

struct TcArgs {
    RoutedArgs r;
    Layout L;
    unsigned* barrier;   // [4] grid barriers, zeroed by the scores' kernel
    unsigned* status;    // the device's status word
    float* part[PHASES];  // [pieces][T K][2 F or H]
    unsigned* peak;       // fp16: [2][T K] largest |gate| and |up| of a pair's pieces, as bits; zeroed like the barriers
    void* h;              // [PARTS][T K][F]
    int pieces[PHASES];   // of a tile, at most
    bool fused;           // the loading warps form h
    unsigned long long wait_ns;  // limit of a wait
    int hold;  // testing hook: what CTA 0 withholds, its arrival at meeting 0 to 3 or its units from hold - 4 on (-1: nothing)
};

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int k, int row, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3}], [%4], "
        "%5;" ::"r"(dst),
        "l"(map), "r"(k), "r"(row), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {  // bytes 0: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// One lane of a warp that has come here as a whole.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void worker_sync() { asm volatile("bar.sync 1, %0;" ::"n"(WORKERS) : "memory"); }

struct Info {  // an expert that some token chose
    int expert, start, n;
};

// What the roles share: where things lie, and how the units of a phase are dealt out.
struct Ctx {
    unsigned char* sm;
    uint32_t base, bars;
    volatile int *abort, *met;  // a wait has run out; the last meeting took place
    float* weight;
    unsigned short *toks, *list, *act;  // by expert: tokens, pairs (token, choice); by pair: its expert's place in info
    short* id;
    Info* info;
    int P, active;
    int KS[PHASES], tiles[PHASES];
    int chunk[PHASES];  // units of a CTA
    int first[PHASES], end[PHASES];
    int npad, wide, part, stage, S;  // the ring's cut
    int doublings;                   // of a bound: a tile has at most two to this many pieces
    __device__ __forceinline__ uint32_t full(int s) const { return bars + 8 * s; }
    __device__ __forceinline__ uint32_t empty(int s) const { return bars + 8 * (MAX_STAGES + s); }
    __device__ __forceinline__ uint32_t accfull(int b) const { return bars + 8 * (2 * MAX_STAGES + b); }
    __device__ __forceinline__ uint32_t accempty(int b) const { return bars + 8 * (2 * MAX_STAGES + 2 + b); }
    __device__ __forceinline__ uint32_t drain() const { return bars + 8 * (2 * MAX_STAGES + 4); }
    __device__ __forceinline__ uint32_t go() const { return bars + 8 * (2 * MAX_STAGES + 5); }
};
constexpr int BAR_BYTES = 8 * (2 * MAX_STAGES + 6) + 16;  // and the TMEM address, and the two flags

// A piece: units [u, u + n) of one tile.
struct Piece {
    int job, ks, n;
};
__device__ __forceinline__ Piece piece_at(const Ctx& c, int ph, int u) {
    const int job = u / c.KS[ph], ks = u - job * c.KS[ph];
    return Piece{job, ks, min(c.KS[ph] - ks, c.end[ph] - u)};
}
// A role's place in the ring, counted without divisions: these would be most of what a unit costs the
// producing and the multiplying thread (400 ns a unit with them).
struct Turn {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ void skip(int n, int stages) {
        s += n;
        while (s >= stages) {
            s -= stages;
            phase ^= 1;
        }
    }
};
__device__ __forceinline__ int pad16(int n) { return (n + 15) & ~15; }

// Returns the units that were requested.
__device__ int produce(const Ctx& c, const TcArgs& t, const CUtensorMap* up, const CUtensorMap* down) {
    const uint64_t policy = policy_drop();
    const int stages = c.S, stage = c.stage, wide = c.wide, step = wide * KSTEP;
    Turn at;
    int issued = 0;
    bool ok = true;
    for (int ph = 0; ok && ph < PHASES; ++ph) {
        const CUtensorMap* const map = ph ? down : up;
        for (int u = c.first[ph]; ok && u < c.end[ph];) {
            const Piece p = piece_at(c, ph, u);
            const int a = p.job / c.tiles[ph], tile = p.job - a * c.tiles[ph], e = c.info[a].expert;
            const int r0 = ph ? e * t.r.H + tile * 128 : e * 2 * t.r.F + tile * 64, r1 = ph ? r0 + 64 : r0 + t.r.F;
            for (int k = p.ks * step, end = k + p.n * step; k < end; k += step) {
                if (t.hold >= 4 && issued >= t.hold - 4 && blockIdx.x == 0) return issued;
                // The loading warps' first requests go out before most of the ring's: behind all of it they take 5 us.
                if (issued == HEAD) ok = mbar_wait_bounded(c.go(), 0, c.abort, t.wait_ns);
                ok = ok && mbar_wait_bounded(c.empty(at.s), at.phase ^ 1, c.abort, t.wait_ns);
                if (!ok) break;
                const uint32_t full = c.full(at.s), dst = c.base + at.s * stage;
                mbar_arrive_expect_tx(full, wide * A_BYTES);
                for (int i = 0; i < wide; ++i) {  // (columns past the matrix's last one come as zeros)
                    tma_rows(dst + i * A_BYTES, map, k + i * KSTEP, r0, full, policy);
                    tma_rows(dst + i * A_BYTES + A_BYTES / 2, map, k + i * KSTEP, r1, full, policy);
                }
                at.next(stages);
                ++issued;
            }
            u += p.n;
        }
    }
    return issued;
}
// After a wait that ran out, once no role is at work any more: copies in flight land before the CTA goes.  A unit's barrier
// wants the arrival of its loading warp too, which may have given up before it; loaded: units that each has arrived for.
__device__ void settle(const Ctx& c, int issued, const int* loaded) {
    const int stages = c.S, loaders = min(LOADERS, stages);
    int dummy = 0;
    for (int i = max(0, issued - stages); i < issued; ++i) {
        const int s = i % stages;
        if (i / loaders >= loaded[i % loaders]) mbar_arrive(c.full(s));
        mbar_wait_bounded(c.full(s), (i / stages) & 1, &dummy, WAIT_NS);
    }
}

template <int DT>
__device__ void multiply(const Ctx& c, const TcArgs& t, uint32_t tmem) {
    constexpr uint32_t format = DT == SOT_BF16 ? (1u << 7) | (1u << 10) : 0u;
    const int stages = c.S;
    const uint64_t a0 = sw128_desc(c.base), step = c.stage >> 4;
    const int wide = c.wide;
    const uint64_t tokens = wide * A_BYTES >> 4, part = c.part >> 4;
    Turn at;
    int seg = 0;
    bool ok = true, issued = false;
    for (int ph = 0; ok && ph < PHASES; ++ph)
        for (int u = c.first[ph]; ok && u < c.end[ph]; ++seg) {
            const Piece p = piece_at(c, ph, u);
            const uint32_t idesc = f16_idesc(128, pad16(c.info[p.job / c.tiles[ph]].n)) | format;
            const uint32_t d = tmem + (seg & 1) * c.npad;
            ok = mbar_wait_bounded(c.accempty(seg & 1), ((seg >> 1) & 1) ^ 1, c.abort, t.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            for (int i = 0; ok && i < p.n; ++i) {
                ok = mbar_wait_bounded(c.full(at.s), at.phase, c.abort, t.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint64_t a = a0 + at.s * step, b = a + tokens;
                if (elect_one()) {
                    const auto product = [&](uint64_t a, uint64_t b, bool first) {
#pragma unroll
                        for (int k = 0; k < KSTEP / 16; ++k) tc_mma_f16(d, a + 2 * k, b + 2 * k, idesc, !first || k > 0);
                    };
                    product(a, b, i == 0);
                    if (ph) product(a, b + part, false);
                    if (wide == 2) {
                        product(a + (A_BYTES >> 4), b + PARTS * part, false);
                        if (ph) product(a + (A_BYTES >> 4), b + (PARTS + 1) * part, false);
                    }
                    tc_commit(c.empty(at.s));
                    if (i == p.n - 1) tc_commit(c.accfull(seg & 1));
                }
                __syncwarp();
                issued = true;
                at.next(stages);
            }
            u += p.n;
        }
    if (issued && elect_one()) {  // nothing is under way when the CTA frees its TMEM
        int dummy = 0;
        tc_commit(c.drain());
        mbar_wait_bounded(c.drain(), 0, &dummy, WAIT_NS);
    }
}

__device__ __forceinline__ float silu_times(float gate, float up) { return gate / (1.f + expf(-gate)) * up; }

// Pieces of a tile: the CTAs that have units of it.
__device__ __forceinline__ int pieces_of(const Ctx& c, int ph, int job) {
    const int u = job * c.KS[ph];
    return (u + c.KS[ph] - 1) / c.chunk[ph] - u / c.chunk[ph] + 1;
}

// Four columns of the pieces of a tile: three are fetched before the first is added, and before other tiles' are.
struct Pieces {
    static constexpr int MOST = 3;
    const float* from;
    long long step;
    int n;
    float4 v[MOST];
    __device__ __forceinline__ void fetch(const float* from_, long long step_, int n_) {
        from = from_;
        step = step_;
        n = n_;
#pragma unroll
        for (int j = 0; j < MOST; ++j)  // (a piece that is not there: another one again, not added)
            v[j] = __ldcg(reinterpret_cast<const float4*>(from + max(0, min(j, n - 1)) * step));
    }
    __device__ __forceinline__ float4 sum() const {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        const auto add = [&](const float4& a) { s = make_float4(s.x + a.x, s.y + a.y, s.z + a.z, s.w + a.w); };
#pragma unroll
        for (int j = 0; j < MOST; ++j)
            if (j < n) add(v[j]);
#pragma unroll 1
        for (int j = MOST; j < n; ++j) add(__ldcg(reinterpret_cast<const float4*>(from + j * step)));
        return s;
    }
};
// fp16 has too few exponents for h, so a pair's h is multiplied by a power of two, which its products are divided by as they
// leave the accumulators.  |h| <= |gate| |up|, each at most as many times its largest piece as a tile has pieces: with
// that bound below 2^15 nothing overflows, and what two parts cannot hold is 2^-40 of the bound.  (A bound, because
// the exact maximum of a pair would be known a phase too late; the exponent alone, so that no bit of h changes.)
template <int DT>
__device__ __forceinline__ int exponent_of(const Ctx& c, unsigned gate, unsigned up) {
    if constexpr (DT != SOT_F16) return 0;
    // |v| < 2^(e - 126) with e the exponent's bits; an h that is finite at all is below 2^128
    const int bound = min(128, (int)(gate >> 23) - 126 + (int)(up >> 23) - 126 + 2 * c.doublings);
    return min(126, 15 - bound);
}
template <int DT>
__device__ __forceinline__ int exponent_at(const Ctx& c, const TcArgs& t, int p) {
    if constexpr (DT != SOT_F16) return 0;
    return exponent_of<DT>(c, __ldcg(t.peak + p), __ldcg(t.peak + c.P + p));
}
__device__ __forceinline__ float two_to(int k) { return __uint_as_float((unsigned)(k + 127) << 23); }  // -127 < k < 128

template <int DT>
struct Most {  // the type's largest number
    static constexpr float value = DT == SOT_F16 ? 65504.f : 3.3895313892515355e38f;
};
// Four numbers h 2^k as two parts each; infinities and NaN are in the second one.
template <int DT>
__device__ __forceinline__ void activated(const Pieces& gate, const Pieces& up, int k, uint2 (&part)[PARTS]) {
    const float4 g = gate.sum(), u = up.sum();
    float h[4] = {silu_times(g.x, u.x), silu_times(g.y, u.y), silu_times(g.z, u.z), silu_times(g.w, u.w)};
    float2 a[Elem<DT>::N / 2] = {}, b[Elem<DT>::N / 2] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == SOT_F16) h[i] *= two_to(k);
        const float first = Elem<DT>::get(Elem<DT>::put(fminf(fmaxf(h[i], -Most<DT>::value), Most<DT>::value)));
        (i & 1 ? a[i / 2].y : a[i / 2].x) = first;
        (i & 1 ? b[i / 2].y : b[i / 2].x) = h[i] - first;
    }
    const uint4 v = pack<DT>(a), w = pack<DT>(b);
    part[0] = make_uint2(v.x, v.y);
    part[1] = make_uint2(w.x, w.y);
}

// A half-warp takes 64 columns of a pair, two at a time.
template <int DT>
__device__ void activate(const Ctx& c, const TcArgs& t) {
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - W_EPI, tiles = c.tiles[0], F = t.r.F, all = c.P * tiles;
    const int teams = gridDim.x * (WORKERS / 32) * 2;
    const long long step = (long long)c.P * 2 * F;
#pragma unroll 1
    for (int i = (blockIdx.x + w * gridDim.x) * 2 + (lane >> 4); i < all; i += 2 * teams) {
        Pieces gate[2], up[2];
        unsigned short* to[2];
        int k[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int at = min(i + j * teams, all - 1), p = at / tiles, tile = at - p * tiles, f = tile * 64 + (lane & 15) * 4;
            const bool real = i + j * teams < all && c.id[p] >= 0 && f < F;
            const int n = real ? pieces_of(c, 0, c.act[p] * tiles + tile) : 0;
            const float* const from = t.part[0] + (long long)p * 2 * F + (real ? f : 0);
            gate[j].fetch(from, step, n);
            up[j].fetch(from + F, step, n);
            k[j] = exponent_at<DT>(c, t, p);
            to[j] = real ? static_cast<unsigned short*>(t.h) + (long long)p * F + f : nullptr;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint2 h[PARTS];
            activated<DT>(gate[j], up[j], k[j], h);
            if (to[j]) {
                *reinterpret_cast<uint2*>(to[j]) = h[0];
                *reinterpret_cast<uint2*>(to[j] + (long long)c.P * F) = h[1];
            }
        }
    }
}

// For few tokens the loading warps do that for themselves, each unit's columns as it is loaded: every tile of an expert
// does it again, but there is no phase of its own and no barrier behind it
// (H = 2048, F = 1024, 8 of 64 experts: one token 31.4 us, else 33.7; two 44.6, else 45.7; four 71.9, else 71.0).
// 64 columns from k on of pair p's h, for the swizzled row at `row` of a slice at `dst`: four columns a lane, 16 lanes a slice.
template <int DT>
__device__ __forceinline__ void activate_into(const Ctx& c, const TcArgs& t, uint32_t dst, int row, int p, int expert, int k0) {
    const int lane = threadIdx.x & 31, F = t.r.F;
    const int slice = lane >> 4, k = k0 + lane * 4, tile = k >> 6;
    if (slice >= c.wide) return;
    const bool real = k < F;
    const int n = real ? pieces_of(c, 0, expert * c.tiles[0] + tile) : 0;
    const float* const from = t.part[0] + (long long)p * 2 * F + (real ? k : 0);
    Pieces gate, up;
    gate.fetch(from, (long long)c.P * 2 * F, n);
    up.fetch(from + F, (long long)c.P * 2 * F, n);
    uint2 h[PARTS];
    activated<DT>(gate, up, exponent_at<DT>(c, t, p), h);
    const int ch = lane >> 1 & 7;
    const uint32_t to = dst + slice * PARTS * c.part + (row >> 3) * 1024 + (row & 7) * 128 + ((ch ^ (row & 7)) << 4) + (lane & 1) * 8;
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(to + i * c.part), "r"(h[i].x), "r"(h[i].y) : "memory");
}

// The tokens' side of a phase: rows of x or of h's parts, swizzled as the tensor cores read them.  A row past the expert's
// last token is not written: what it holds only reaches columns that nobody reads.
template <int DT>
__device__ bool load_tokens(const Ctx& c, const TcArgs& t, int ph, Turn& at, int& turn, int& loaded) {
    const int lane = threadIdx.x & 31, ch = lane & 7, stages = c.S, stage = c.stage, wide = c.wide;
    const int K = ph ? t.r.F : t.r.H;
    const long long ld = ph ? t.r.F : t.r.ldx, second = (long long)c.P * t.r.F;
    const unsigned short* const from = static_cast<const unsigned short*>(ph ? t.h : t.r.x) + ch * 8;
    const unsigned short* const rows = ph ? c.list : c.toks;
    // A warp's next unit must not lie more than a ring ahead of its last one: further on, the parity it waits for
    // could be that of the use before the last, and the place still taken.
    const int loaders = min(LOADERS, stages);
    bool first = ph == 0;
    if ((threadIdx.x >> 5) - W_LOAD >= loaders) {
        if (first && lane == 0) mbar_arrive(c.go());
        return true;
    }
    for (int u = c.first[ph]; u < c.end[ph];) {
        const Piece p = piece_at(c, ph, u);
        const int place = p.job / c.tiles[ph];
        const Info e = c.info[place];
        // turn: units until this warp's next one, whose place in the ring is `at`
        for (; turn < p.n; turn += loaders) {
            const int k0 = (p.ks + turn) * wide * KSTEP;
            const bool ok = mbar_wait_bounded(c.empty(at.s), at.phase ^ 1, c.abort, t.wait_ns);
            if (!__all_sync(0xffffffffu, ok)) return false;
            const uint32_t dst = c.base + at.s * stage + wide * A_BYTES;
            if (ph && t.fused)
                for (int row = 0; row < e.n; ++row) activate_into<DT>(c, t, dst, row, rows[e.start + row], place, k0);
            else
              for (int row = lane >> 3; row < e.n; row += 4) {
                const unsigned short* const src = from + rows[e.start + row] * ld;
                const uint32_t to = dst + (row >> 3) * 1024 + (row & 7) * 128 + ((ch ^ (row & 7)) << 4);
                for (int i = 0; i < wide; ++i) {
                    const int k = k0 + i * KSTEP;
                    const bool real = k + ch * 8 < K;
                    copy16(to + i * PARTS * c.part, real ? src + k : src, real ? 16 : 0);
                    if (ph) copy16(to + (i * PARTS + 1) * c.part, real ? src + second + k : src, real ? 16 : 0);
                }
            }
            if (first && lane == 0) mbar_arrive(c.go());
            first = false;
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.full(at.s));
            ++loaded;
            at.skip(loaders, stages);
        }
        turn -= p.n;
        u += p.n;
    }
    if (first && lane == 0) mbar_arrive(c.go());  // (a warp without a unit)
    return true;
}

// The accumulators of a phase's pieces, as partial sums [piece of the tile][pair][row].
template <int DT>
__device__ bool store_pieces(const Ctx& c, const TcArgs& t, int ph, int& seg, uint32_t tmem) {
    const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3, m = q * 32 + lane;
    const int ld = ph ? t.r.H : 2 * t.r.F;
    for (int u = c.first[ph]; u < c.end[ph]; ++seg) {
        const Piece p = piece_at(c, ph, u);
        const int a = p.job / c.tiles[ph], tile = p.job - a * c.tiles[ph];
        const Info e = c.info[a];
        const int col = ph ? tile * 128 + m : tile * 64 + (m & 63) + (m < 64 ? 0 : t.r.F);
        const bool real = ph ? col < t.r.H : tile * 64 + (m & 63) < t.r.F;
        const int ord = blockIdx.x - p.job * c.KS[ph] / c.chunk[ph];
        float* const to = t.part[ph] + (long long)ord * c.P * ld + col;
        // fp16: what lane n's token of the next sixteen multiplies h by
        const auto exponent = [&](int n0) { return lane < 16 && n0 + lane < e.n ? exponent_at<DT>(c, t, c.list[e.start + n0 + lane]) : 0; };
        int k = DT == SOT_F16 && ph ? exponent(0) : 0;
        bool ok = mbar_wait_bounded(c.accfull(seg & 1), (seg >> 1) & 1, c.abort, t.wait_ns);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tc_fence_after();
        const uint32_t from = tmem + (seg & 1) * c.npad + ((uint32_t)(q * 32) << 16);
        for (int n0 = 0; n0 < e.n; n0 += 16) {
            float v[16];
            tmem_ld16(from + n0, v);
            if (DT == SOT_F16 && ph) {
                if (n0 > 0) k = exponent(n0);
#pragma unroll
                for (int n = 0; n < 16; ++n) v[n] *= two_to(-__shfl_sync(0xffffffffu, k, n));
            }
#pragma unroll
            for (int n = 0; n < 16; ++n)
                if (n0 + n < e.n && real) __stcg(to + (long long)c.list[e.start + n0 + n] * ld, v[n]);
            if (DT == SOT_F16 && !ph) {
                unsigned most = 0;
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                    const unsigned w = __reduce_max_sync(0xffffffffu, real ? __float_as_uint(fabsf(v[n])) : 0u);
                    if (lane == n) most = w;
                }
                if (lane < 16 && n0 + lane < e.n) atomicMax(t.peak + (q < 2 ? 0 : c.P) + c.list[e.start + n0 + lane], most);
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(c.accempty(seg & 1));
        u += p.n;
    }
    return true;
}

__device__ __forceinline__ unsigned load_acquire(const unsigned* at) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
    return v;
}
// One thread of each CTA, for all that the CTA has done before: whether all CTAs have come this far (what they wrote is
// then seen) and this one has not given up.
__device__ __forceinline__ bool meet(const Ctx& c, const TcArgs& t, int which) {
    unsigned* const at = t.barrier + which;
    __threadfence();
    // (a CTA that gave up holds the others, whose waits then run out too)
    if (!*c.abort && !(t.hold == which && blockIdx.x == 0)) atomicAdd(at, 1u);
    const uint64_t t0 = globaltimer_ns();
    bool ok = false;
    while (!*c.abort && !(ok = load_acquire(at) >= gridDim.x))
        if (globaltimer_ns() - t0 > t.wait_ns) *c.abort = 1;
    __threadfence();
    return ok;
}
// All workers of a CTA get one answer.  (The flag itself may be raised by another role between two of them looking at it, and
// they would wait for each other at different barriers.  Nobody else writes the answer, and the next one is
// written behind a barrier that comes after all have read this one.)
__device__ bool grid_barrier(const Ctx& c, const TcArgs& t, int which) {
    worker_sync();
    if (threadIdx.x == W_EPI * 32) *c.met = meet(c, t, which);
    worker_sync();
    return *c.met != 0;
}

// A warp takes 32 columns of a token: four lanes share four columns and take a quarter of the experts each.
template <int DT>
__device__ void join(const Ctx& c, const TcArgs& t) {
    using T = typename Elem<DT>::T;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - W_EPI, H = t.r.H, per = (H + 31) / 32;
    for (int i = blockIdx.x + w * gridDim.x; i < t.r.T * per; i += gridDim.x * (WORKERS / 32)) {
        const int tok = i / per, col = (i - tok * per) * 32 + (lane & 7) * 4;
        const bool real = col < H;
        float s[4] = {};
#pragma unroll 1
        for (int k0 = lane >> 3; k0 < t.r.K; k0 += 8) {
            Pieces y[2];
            float wt[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = k0 + 4 * j, p = tok * t.r.K + min(k, t.r.K - 1);
                const bool chosen = k < t.r.K && c.id[p] >= 0 && real;
                wt[j] = k < t.r.K ? c.weight[p] : 0.f;  // (not chosen: 0, or NaN)
                const int n = chosen ? pieces_of(c, 1, c.act[p] * c.tiles[1] + (col >> 7)) : 0;
                y[j].fetch(t.part[1] + (long long)p * H + (real ? col : 0), (long long)c.P * H, n);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 v = y[j].n > 0 ? y[j].sum() : make_float4(1.f, 1.f, 1.f, 1.f);
                s[0] = fmaf(wt[j], v.x, s[0]);
                s[1] = fmaf(wt[j], v.y, s[1]);
                s[2] = fmaf(wt[j], v.z, s[2]);
                s[3] = fmaf(wt[j], v.w, s[3]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[j] += __shfl_xor_sync(0xffffffffu, s[j], 8);
            s[j] += __shfl_xor_sync(0xffffffffu, s[j], 16);
        }
        if (lane < 8 && real) {
            T* const to = static_cast<T*>(t.r.out) + tok * t.r.ldo + col;
#pragma unroll
            for (int j = 0; j < 4; ++j) to[j] = Elem<DT>::put(s[j]);
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(NT, 1) routed_tc_kernel(const TcArgs t, const __grid_constant__ CUtensorMap up,
                                                          const __grid_constant__ CUtensorMap down) {
    extern __shared__ unsigned char raw[];
    __shared__ int counts[2], issued, loaded[LOADERS];
    const uint32_t lead = smem_u32(raw);
    const uint32_t skip = (1024 - (lead & 1023)) & 1023;
    Ctx c;
    c.sm = raw + skip;
    c.base = lead + skip;
    c.bars = c.base + t.L.bars;
    uint32_t* const slot = reinterpret_cast<uint32_t*>(c.sm + t.L.bars + BAR_BYTES - 16);
    c.abort = reinterpret_cast<volatile int*>(slot + 1);
    c.met = c.abort + 1;
    c.weight = reinterpret_cast<float*>(c.sm + t.L.weight);
    c.toks = reinterpret_cast<unsigned short*>(c.sm + t.L.toks);
    c.list = reinterpret_cast<unsigned short*>(c.sm + t.L.list);
    c.act = reinterpret_cast<unsigned short*>(c.sm + t.L.act);
    c.id = reinterpret_cast<short*>(c.sm + t.L.id);
    c.info = reinterpret_cast<Info*>(c.sm + t.L.info);
    uint4* const mask = reinterpret_cast<uint4*>(c.sm + t.L.mask);  // the tokens of each expert
    unsigned short* const place = reinterpret_cast<unsigned short*>(c.sm + t.L.place);  // of each expert in info
    c.P = t.r.T * t.r.K;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = t.r.E, K = t.r.K;
    if (tid == 0) {
        for (int s = 0; s < MAX_STAGES; ++s) {
            mbar_init(c.full(s), 2);  // the producer's arrival and a loading warp's
            mbar_init(c.empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(c.accfull(b), 1);
            mbar_init(c.accempty(b), 4);
        }
        mbar_init(c.drain(), 1);
        mbar_init(c.go(), LOADERS);
        fence_mbar_init();
        *c.abort = 0;
    }
    int cols = 32;
    while (cols < 2 * t.L.most) cols *= 2;
    if (warp == W_MMA) {
        tmem_alloc(smem_u32(slot), cols);
        tmem_relinquish();
    }
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&up) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&down) : "memory");
    }
    // Choose: a warp a token.  Every CTA does it for all tokens where that takes a round; otherwise the tokens are shared out
    // and read back behind a barrier (64 tokens of 128 experts: products begin after 8 us, with all in every CTA after 20).
    for (int i = tid; i < E; i += NT) mask[i] = make_uint4(0u, 0u, 0u, 0u);
    const auto take = [&](int p, int id, float w) {
        c.id[p] = (short)id;
        c.weight[p] = w;
        if (id >= 0) atomicOr(reinterpret_cast<unsigned*>(mask + id) + (p / K >> 5), 1u << (p / K & 31));
    };
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores, and the barriers' zeros
    const bool shared = t.r.T > NWARP;
#pragma unroll 1
    for (int tok = shared ? blockIdx.x + warp * gridDim.x : warp; tok < t.r.T; tok += NWARP * (shared ? gridDim.x : 1)) {
        int id;
        float w;
        routed_choose(t.r.logits + (long long)tok * E, E, K, t.r.renorm, t.r.scale, id, w);
        if (lane < K) {
            const int p = tok * K + lane;
            if (!shared) take(p, id, w);
            if (shared || tok % gridDim.x == blockIdx.x) {
                t.r.ids[p] = id;
                t.r.weights[p] = w;
            }
        }
    }
    __syncthreads();
    if (shared) {
        if (tid == 0) meet(c, t, 3);
        __syncthreads();
        if (!*c.abort) {  // (otherwise some tokens' choices may not be there, only what the memory held before)
#pragma unroll 1
            for (int p = tid; p < c.P; p += NT) take(p, __ldcg(t.r.ids + p), __ldcg(t.r.weights + p));
        }
        __syncthreads();
    }
    // The experts in use, in order, and where their lists start.  (Loops stay loops here: this runs once, and fetching
    // instructions is most of what it costs.)
    if (warp == 0) {
        int used = 0, start = 0, most = 0;
#pragma unroll 1
        for (int e0 = 0; e0 < E; e0 += 32) {
            const uint4 m = e0 + lane < E ? mask[e0 + lane] : make_uint4(0u, 0u, 0u, 0u);
            const int n = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
            const unsigned on = __ballot_sync(0xffffffffu, n > 0);
            int upto = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            if (n > 0) {
                const int a = used + __popc(on & ((1u << lane) - 1u));
                c.info[a] = Info{e0 + lane, start + upto - n, n};
                place[e0 + lane] = (unsigned short)a;
            }
            used += __popc(on);
            start += __shfl_sync(0xffffffffu, upto, 31);
            most = max(most, n);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) {
            counts[0] = *c.abort ? 0 : used;
            counts[1] = most;
        }
    }
    __syncthreads();
    c.active = counts[0];
    const Cut cut(max(16, pad16(counts[1])), t.L.ring);
    c.npad = cut.npad;
    c.wide = cut.wide;
    c.part = cut.part;
    c.stage = cut.stage;
    c.S = cut.stages;
    // A pair's place in its expert's list: the tokens before its own.
#pragma unroll 1
    for (int p = tid; p < c.P; p += NT) {
        const int id = c.id[p], tok = p / K;
        if (id < 0 || c.active == 0) continue;
        const unsigned* const m = reinterpret_cast<const unsigned*>(mask + id);
        int at = __popc(m[tok >> 5] & ((1u << (tok & 31)) - 1u));
        for (int q = 0; q < tok >> 5; ++q) at += __popc(m[q]);
        at += c.info[place[id]].start;
        c.toks[at] = (unsigned short)tok;
        c.list[at] = (unsigned short)p;
        c.act[p] = place[id];
    }
    const int dims[PHASES] = {t.r.H, t.r.F};
    c.tiles[0] = (t.r.F + 63) / 64;
    c.tiles[1] = (t.r.H + 127) / 128;
    for (int ph = 0; ph < PHASES; ++ph) {
        c.KS[ph] = (dims[ph] + c.wide * KSTEP - 1) / (c.wide * KSTEP);
        const int U = c.active * c.tiles[ph] * c.KS[ph];
        // An even share each, but not so small that a tile has more pieces than there is room for.
        c.chunk[ph] = max(1, max((U + (int)gridDim.x - 1) / (int)gridDim.x,
                                 t.pieces[ph] > 1 ? (c.KS[ph] + t.pieces[ph] - 2) / (t.pieces[ph] - 1) : c.KS[ph]));
        c.first[ph] = (int)min((long long)U, (long long)blockIdx.x * c.chunk[ph]);
        c.end[ph] = min(U, c.first[ph] + c.chunk[ph]);
    }
    c.doublings = 32 - __clz(min(c.KS[0], (c.KS[0] + c.chunk[0] - 2) / c.chunk[0] + 1) - 1);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;

    if (warp == W_PRODUCER) {
        if (lane == 0) issued = produce(c, t, &up, &down);
    } else if (warp == W_MMA) {
        multiply<DT>(c, t, tmem);
    } else {
        int seg = 0, turn = warp - W_LOAD, units = 0;
        Turn at;
        if (warp < W_LOAD) store_pieces<DT>(c, t, 0, seg, tmem);
        else {
            at.skip(turn, c.S);
            load_tokens<DT>(c, t, 0, at, turn, units);
        }
        bool ok = grid_barrier(c, t, 0);
        if (ok && !t.fused) {
            activate<DT>(c, t);
            ok = grid_barrier(c, t, 1);
        }
        if (ok) {
            if (warp < W_LOAD) store_pieces<DT>(c, t, 1, seg, tmem);
            else load_tokens<DT>(c, t, 1, at, turn, units);
            ok = grid_barrier(c, t, 2);
        }
        if (ok) join<DT>(c, t);
        else {
            using T = typename Elem<DT>::T;
            for (long long i = (long long)blockIdx.x * WORKERS + tid - W_EPI * 32; i < (long long)t.r.T * t.r.H;
                 i += (long long)gridDim.x * WORKERS)
                static_cast<T*>(t.r.out)[i / t.r.H * t.r.ldo + i % t.r.H] = Elem<DT>::put(NAN);
            if (tid == W_EPI * 32) atomicOr(t.status, SOT_DEV_TIMEOUT);
        }
        if (warp >= W_LOAD && lane == 0) loaded[warp - W_LOAD] = units;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) tmem_dealloc(tmem, cols);
    if (tid == 0 && *c.abort) settle(c, issued, loaded);
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static const EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// rows x cols of 16-bit elements in boxes of 64 x 64, 128-byte swizzle.
bool weight_map(CUtensorMap* map, const void* p, int dtype, long long rows, int cols) {
    const EncodeTiled encode = encoder();
    if (!encode) return false;
    const cuuint64_t dim[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)cols * 2};
    const cuuint32_t box[2] = {KSTEP, 64}, step[2] = {1, 1};
    return encode(map, dtype == SOT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                  const_cast<void*>(p), dim, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Host-side settings that every launch takes.
std::atomic<int> g_hold{-1};
std::atomic<unsigned long long> g_wait_ns{WAIT_NS};

constexpr int MAX_SMEM = 227 * 1024 - 1024;  // the kernel's static part is below 1 KB

Layout layout(const RoutedArgs& a) {
    Layout L = {};
    const int P = a.T * a.K;
    int at = 0;
    const auto place = [&](int bytes) {
        const int here = at;
        at = (at + bytes + 15) / 16 * 16;
        return here;
    };
    L.most = (a.T + 15) / 16 * 16;
    const int other = (BAR_BYTES + 15) / 16 * 16 + (4 * P + 15) / 16 * 16 + 4 * ((2 * P + 15) / 16 * 16) +
                      ((int)sizeof(Info) * a.E + 15) / 16 * 16 + 16 * a.E + (2 * a.E + 15) / 16 * 16;
    L.ring = (MAX_SMEM - 1024 - other) / 1024 * 1024;
    place(L.ring);
    L.bars = place(BAR_BYTES);
    L.weight = place(4 * P);
    L.toks = place(2 * P);
    L.list = place(2 * P);
    L.act = place(2 * P);
    L.id = place(2 * P);
    L.info = place((int)sizeof(Info) * a.E);
    L.mask = place(16 * a.E);
    L.place = place(2 * a.E);
    L.total = at + 1024;
    return L;
}

// Pieces of a tile that there is room for: those an even share leaves where the tokens choose no more than K experts.
int pieces(const RoutedArgs& a, int ph, int sms) {
    const int KS = ((ph ? a.F : a.H) + KSTEP - 1) / KSTEP, tiles = ph ? (a.H + 127) / 128 : (a.F + 63) / 64;
    const int p = (sms + tiles * a.K - 1) / (tiles * a.K) + 1;
    return p < KS ? p : KS;
}

}  // namespace

void routed_set_test_hold(int what, unsigned long long wait_ns) {
    g_hold.store(what < 0 ? -1 : what);
    g_wait_ns.store(wait_ns > 0 ? wait_ns : WAIT_NS);
}

bool routed_tc_fits(const RoutedArgs& a) {
    return a.dtype != SOT_F32 && a.H % 8 == 0 && a.F % 8 == 0 && a.ldx % 8 == 0 && (unsigned long long)a.x % 16 == 0 &&
           (unsigned long long)a.gate_up % 16 == 0 && (unsigned long long)a.down % 16 == 0 &&
           (long long)a.E * 2 * a.F < 1ll << 31 && (long long)a.E * a.H < 1ll << 31 &&
           // (units are counted in 32 bits)
           (long long)a.E * ((a.F + 63) / 64) * ((a.H + 63) / 64) < 1ll << 30 &&
           (long long)a.E * ((a.H + 127) / 128) * ((a.F + 63) / 64) < 1ll << 30 && Cut(layout(a).most, layout(a).ring).stages >= MIN_STAGES;
}

RoutedTcPlan routed_tc_plan(const RoutedArgs& a, int sms) {
    RoutedTcPlan p = {};
    const auto place = [&](size_t bytes) {
        const size_t at = p.scratch;
        p.scratch = (at + bytes + 255) & ~(size_t)255;
        return at;
    };
    const size_t P = (size_t)a.T * a.K;
    p.zeros = 4 + (a.dtype == SOT_F16 ? 2 * (int)P : 0);
    p.barrier_at = place(p.zeros * sizeof(unsigned));
    p.up_at = place(sizeof(float) * pieces(a, 0, sms) * P * 2 * a.F);
    p.down_at = place(sizeof(float) * pieces(a, 1, sms) * P * a.H);
    p.h_at = place(2 * PARTS * P * a.F);
    return p;
}

cudaError_t launch_routed_tc(const RoutedArgs& a, const RoutedTcPlan& p, unsigned char* scratch, int sms, cudaStream_t st) {
    TcArgs t = {};
    t.r = a;
    t.L = layout(a);
    t.barrier = reinterpret_cast<unsigned*>(scratch + p.barrier_at);
    t.peak = t.barrier + 4;
    t.part[0] = reinterpret_cast<float*>(scratch + p.up_at);
    t.part[1] = reinterpret_cast<float*>(scratch + p.down_at);
    t.h = scratch + p.h_at;
    for (int ph = 0; ph < PHASES; ++ph) t.pieces[ph] = pieces(a, ph, sms);
    t.fused = a.T * a.K <= FUSED_PAIRS;
    t.wait_ns = g_wait_ns.load();
    t.hold = g_hold.load();
    cudaError_t e = async_status_address(&t.status);
    if (e != cudaSuccess) return e;
    CUtensorMap up, down;
    if (!weight_map(&up, a.gate_up, a.dtype, (long long)a.E * 2 * a.F, a.H) ||
        !weight_map(&down, a.down, a.dtype, (long long)a.E * a.H, a.F))
        return cudaErrorInvalidValue;
    const void* const kern = a.dtype == SOT_BF16 ? (const void*)routed_tc_kernel<SOT_BF16> : (const void*)routed_tc_kernel<SOT_F16>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
    if (e != cudaSuccess) return e;
    void* args[] = {&t, &up, &down};
    count_launches(1);
    // All CTAs wait for one another, so all have to be there; and they may come while the scores are still being
    // formed, which they wait for before they read them.
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(sms, 1, 1);
    cfg.blockDim = dim3(NT, 1, 1);
    cfg.dynamicSmemBytes = t.L.total;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

}  // namespace sot

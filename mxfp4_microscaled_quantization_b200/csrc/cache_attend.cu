// cache_attend.cu -- single-token attention over the 8-bit paged cache for
// sm_100a.
//
// For sequence b, query head h (key head g = h / (Hq / Hkv)) and the cached
// tokens j < lens[b]:  s_j = scale q . (kc_j 2^ek),  o = sum_j e^(s_j - M)
// (vc_j 2^ev) / sum_j e^(s_j - M),  lse = M + ln sum_j e^(s_j - M), with the
// exponents of j's page.  lens[b] = 0 gives zeros and -inf.
//
// What bounds it is the cache's bytes, 2 d a token and key head, so the codes
// go from HBM to the tensor core untouched: TMA brings pages into shared
// memory, where they are the first operand of both products, in E4M3
// (tcgen05 kind::f8f6f4, 128 tokens a tile):
//   S^T [128 tokens, heads] = K Q^T,   O^T [d, heads] += V^T P^T.
// Only Q and P are converted, each into E4M3 parts whose sum is the value:
//   * Q, scaled by a power of two a head so that its largest element is in
//     (224, 448]:  q = q1 + q2 (+ q3), every part the rounded rest of those
//     before.  A part takes 4 bits, so two hold bf16's 8 significant bits and
//     three fp16's 11, down to 2^-10 (2^-18 of the largest element).  The
//     parts' products add up in one accumulator.
//   * P as p1 + p2 / 16 (+ p3 / 256), the rest scaled by 16 before it is
//     rounded, so it does not run out of exponent:  relative error 2^-8 (bf16;
//     bf16's own rounding) or 2^-12 (fp16), and 2^-19 (2^-23) of the largest
//     weight where that is more.  The parts are further columns of the second
//     product, added up in the end.
// A token's K exponent scales its scores; its V exponent goes into P, relative
// to the largest one so far.  Maxima, sums and O are fp32.
//
// Work.  All (sequence, key head) pairs' tiles of 128 tokens form one list, cut
// into equal runs, one a block (two blocks an SM), whatever the lengths: a run
// covers the end of one pair, whole pairs, the start of another.  A whole
// pair's result is final; a part of one goes to the block's slot in the
// workspace, and a second kernel (started early by programmatic launch) joins
// the parts in the order of the list, so results do not depend on timing.
//
// Roles (224 threads):
//   warps 0-3  softmax, a thread per token of the tile (= TMEM lane of S^T), all
//              heads of the group: maxima over the tile (redux, then shared
//              memory), P's parts to shared memory; O^T rescaled only when a
//              maximum has grown by more than 2^3 (P stays below 448) or a
//              larger V exponent came; the end of each piece.
//   warp 4     TMA producer, a lane per page, one ring for K and V tiles.
//   warp 5     MMA issuer: S(n + 1) before PV(n), so the softmax never waits
//              for a product it could have had.
//   warp 6     Q: loads the next piece's queries while the current one runs.
// Every mbarrier wait is bounded, as in attention.cu.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <cstring>

#include "kernels.cuh"
#include "serve.cuh"

namespace mxattn {
namespace {

constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per wait
constexpr int kTile = 128;                      // tokens
constexpr int kThreads = 224;
constexpr int kCtasPerSm = 2;
constexpr int kMaxCols = 32;                    // query heads a block handles together
constexpr float kGrow = 3.f;                    // log2 of the growth of a maximum that is put up with
constexpr float kPUnit = 32.f;                  // P's unit: 32 * 2^3 <= 448

// D channels, GC query heads (1 .. GC used), PARTS E4M3 parts of Q and P.
template <int D, int GC, int PARTS>
struct Cfg {
    static constexpr int NC = GC < 16 ? 16 : GC;     // columns of S^T
    static constexpr int NO = NC * PARTS;            // columns of O^T
    static constexpr int kTileBytes = kTile * D;     // a K or V tile
    static constexpr int kQBytes = NC * D;           // one part of Q
    static constexpr int kPBytes = kTile * NO;       // P of a tile, [column chunk of 16][token][16]
    static constexpr int kFixed = PARTS * kQBytes + 2 * kPBytes + 2048;
    // 228 KB an SM, 1 KB of each block is the system's
    static constexpr int kSlots = ((228 * 1024) / kCtasPerSm - 1024 - 1024 - kFixed) / kTileBytes;
    static_assert(kSlots >= 4, "ring");
    static constexpr int kOffQ = 0;
    static constexpr int kOffRing = (kOffQ + PARTS * kQBytes + 1023) / 1024 * 1024;
    static constexpr int kOffP = kOffRing + kSlots * kTileBytes;  // [2]
    static constexpr int kOffMax = kOffP + 2 * kPBytes;           // float [2][NC][4], then u32 [2][4]
    static constexpr int kOffBar = kOffMax + 2 * NC * 16 + 32;
    // q_full, q_empty, kv_full[S], kv_empty[S], s_full[2], s_empty[2], p_full[2], pv_done[2], drain
    static constexpr int kNumBars = 2 + 2 * kSlots + 8 + 1;
    static constexpr int kOffCol = kOffBar + kNumBars * 8;        // float [NC]: 2^eq * scale * log2 e
    static constexpr int kOffMisc = kOffCol + NC * 4;             // TMEM base, abort flag, run start
    static constexpr int kSmemBytes = kOffMisc + 64 + 1024;
    static_assert(kSmemBytes <= 113 * 1024, "two blocks an SM");
    // TMEM: S [2][NC], O [NO]
    static constexpr uint32_t kCols = 2 * NC + NO <= 64 ? 64 : 2 * NC + NO <= 128 ? 128 : 256;
    static_assert(kCtasPerSm * kCols <= 512, "TMEM");
    static constexpr uint32_t kLayout = D == 128 ? kLayoutSw128 : kLayoutSw64;
    static constexpr uint32_t kSbo = 8 * D;          // 8 rows of K, V or Q
    static constexpr size_t kSlotFloats = static_cast<size_t>(GC) * (D + 1);  // workspace slot: o [GC][D], L [GC]
};

struct KParams {
    AttendArgs a;
    float kq;     // softmax scale * log2(e)
    int G;        // query heads of a key head
    int chunks;   // blocks of at most GC heads that a group is cut into
    int per;      // heads of a chunk (the last may have fewer)
    int ctas;
};

// Instruction descriptor of tcgen05.mma kind::f8f6f4, E4M3 operands, fp32 accumulator.
__host__ __device__ constexpr uint32_t f8_idesc(uint32_t m, uint32_t n, bool a_mn, bool b_mn) {
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// N consecutive fp32 columns of this thread's TMEM lane (N = 4, 8, 16 or 32).
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* v) {
#define MXATTN_R4(b) "=r"(v[b]), "=r"(v[b + 1]), "=r"(v[b + 2]), "=r"(v[b + 3])
    if constexpr (N == 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
                     : MXATTN_R4(0)
                     : "r"(taddr)
                     : "memory");
    } else if constexpr (N == 8) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : MXATTN_R4(0), MXATTN_R4(4)
            : "r"(taddr)
            : "memory");
    } else if constexpr (N == 16) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
            "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
            : MXATTN_R4(0), MXATTN_R4(4), MXATTN_R4(8), MXATTN_R4(12)
            : "r"(taddr)
            : "memory");
    } else {
        tmem_ld<16>(taddr, v);
        tmem_ld<16>(taddr + 16, v + 16);
    }
#undef MXATTN_R4
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Largest value over the warp (NaN is passed over, as by fmaxf).
__device__ __forceinline__ float redux_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float log2_to_float(uint32_t e8m0) {  // 2^(byte - 127)
    return e8m0 == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(e8m0 << 23);
}

// 2^-k for k >= 0; 0 where that would leave the normal numbers.
__device__ __forceinline__ float pow2_neg(uint32_t k) { return k > 126 ? 0.f : __uint_as_float((127 - k) << 23); }

// A length as the kernels take it: within [0, max_pages * page].
__device__ __forceinline__ int clean_len(const AttendArgs& a, int b) {
    return max(0, min(a.lens[b], a.max_pages << a.page_shift));
}

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// The list of tiles.  Position x of the list: sequences in order, each its key
// heads' chunks in order, each its tiles in order.  `run` is called by all
// threads of the block (blockDim.x a multiple of 32, at most 256) and gives the
// total and, for the position `want(total)`, its sequence and the position
// that the sequence starts at.  All threads get the same.
struct Where {
    int64_t total, at, base;
    int b;
};
template <class F>
__device__ Where locate(const AttendArgs& a, int pairs, F want) {
    __shared__ int64_t s_sum[8];
    __shared__ int64_t s_base;
    __shared__ int s_b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
    int64_t mine = 0;
    for (int b = lo; b < hi; ++b) mine += tiles_of(clean_len(a, b));
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_sum[warp] = incl;
    if (tid == 0) {
        s_b = 0;
        s_base = 0;
    }
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) incl += s_sum[w];
        total += s_sum[w];
    }
    Where r;
    r.total = total * pairs;
    r.at = want(r.total);
    int64_t base = (incl - mine) * pairs;
    if (r.at >= base && r.at < incl * pairs) {
        int b = lo;
        for (;; ++b) {
            const int64_t n = static_cast<int64_t>(tiles_of(clean_len(a, b))) * pairs;
            if (r.at < base + n) break;
            base += n;
        }
        s_b = b;
        s_base = base;
    }
    __syncthreads();
    r.b = s_b;
    r.base = s_base;
    return r;
}

// Run of block c of C: positions [start(c), start(c + 1)) of the list.
__device__ __forceinline__ int64_t run_start(int64_t total, int c, int C) { return total / C * c + total % C * c / C; }

// The pieces of a run, in order.
struct Pieces {
    const AttendArgs& a;
    int64_t x, end, base;
    int pairs, b, len, tiles;
    // the current piece
    int pair, tile0, n;
    bool begins, ends;  // at the pair's first tile; behind its last

    __device__ Pieces(const AttendArgs& args, int pairs_, int64_t x_, int64_t end_, int64_t base_, int b_)
        : a(args), x(x_), end(end_), base(base_), pairs(pairs_), b(b_) {
        len = x < end ? clean_len(a, b) : 0;
        tiles = tiles_of(len);
    }
    __device__ bool next() {
        if (x >= end) return false;
        while (x >= base + static_cast<int64_t>(tiles) * pairs) {
            base += static_cast<int64_t>(tiles) * pairs;
            len = clean_len(a, ++b);
            tiles = tiles_of(len);
        }
        const int64_t off = x - base;
        pair = static_cast<int>(off / tiles);
        tile0 = static_cast<int>(off - static_cast<int64_t>(pair) * tiles);
        n = static_cast<int>(min(static_cast<int64_t>(tiles - tile0), end - x));
        begins = tile0 == 0;
        ends = tile0 + n == tiles;
        x += n;
        return true;
    }
};

__device__ __forceinline__ int page_at(const AttendArgs& a, int b, int index) {
    return a.table[static_cast<int64_t>(b) * a.table_stride + index];
}

template <int D, bool FP16, int GC>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    cache_attend_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ KParams p) {
    constexpr int PARTS = FP16 ? 3 : 2;
    using C = Cfg<D, GC, PARTS>;
    constexpr int S = C::kSlots, NC = C::NC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sQ = smem + C::kOffQ;
    uint8_t* sRing = smem + C::kOffRing;
    uint8_t* sP = smem + C::kOffP;
    float* sMax = reinterpret_cast<float*>(smem + C::kOffMax);             // [2][NC][4]
    uint32_t* sEv = reinterpret_cast<uint32_t*>(sMax + 2 * NC * 4);        // [2][4]
    float* sCol = reinterpret_cast<float*>(smem + C::kOffCol);             // [NC]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* bar_q_full = bars;
    uint64_t* bar_q_empty = bars + 1;
    uint64_t* bar_kv_full = bars + 2;
    uint64_t* bar_kv_empty = bar_kv_full + S;
    uint64_t* bar_s_full = bar_kv_empty + S;
    uint64_t* bar_s_empty = bar_s_full + 2;
    uint64_t* bar_p_full = bar_s_empty + 2;
    uint64_t* bar_pv_done = bar_p_full + 2;
    uint64_t* bar_drain = bar_pv_done + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    const AttendArgs& a = p.a;
    uint32_t* status = a.status;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int P = a.page_shift, pairs = a.Hkv * p.chunks;

    if (tid == 0) {
        mbar_init(bar_q_full, 1);
        mbar_init(bar_q_empty, 2);  // the products that read Q, and the softmax's reads of its scales
        for (int s = 0; s < S; ++s) {
            mbar_init(bar_kv_full + s, 1);
            mbar_init(bar_kv_empty + s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar_s_full + s, 1);
            mbar_init(bar_s_empty + s, 128);
            mbar_init(bar_p_full + s, 128);
            mbar_init(bar_pv_done + s, 1);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    // Q's rows behind the group's heads stay zero.
    for (int i = tid; i < PARTS * C::kQBytes / 16; i += kThreads) reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == 5) {
        tmem_alloc(tmem_holder, C::kCols);
        tmem_relinquish();
    }
    const int cta = blockIdx.x;
    const Where at = locate(a, pairs, [&](int64_t total) { return run_start(total, cta, p.ctas); });
    const int64_t x0 = at.at, x1 = run_start(at.total, cta + 1, p.ctas);
    // Sequences without a token, and reports of lengths out of range.
    for (int b = cta; b < a.B; b += p.ctas) {
        const int given = a.lens[b];
        const int len = clean_len(a, b);
        if (given != len && tid == 0) atomicOr(status, kStatusInvalid);
        if (len > 0) continue;
        for (int i = tid; i < a.Hq * (D / 8); i += kThreads)
            *reinterpret_cast<uint4*>(a.o + b * a.o_seq + (i / (D / 8)) * a.o_head + i % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
        if (a.lse != nullptr)
            for (int h = tid; h < a.Hq; h += kThreads) a.lse[static_cast<int64_t>(b) * a.Hq + h] = -INFINITY;
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tbase = *tmem_holder;
    const uint32_t col_o = 2 * NC;

    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu,
                          mbar_wait_bounded(bar, parity, abort_flag, status, kStatusTimeout, kTimeoutNs));
    };
    Pieces it(a, pairs, x0, x1, at.base, at.b);

    if (warp == 4) {
        // ---------------------------------------------------------------- TMA producer, a lane per page of the tile
        const int ppt = kTile >> P;  // pages of a tile
        int slot = 0;
        bool ok = true;
        while (ok && it.next()) {
            const int head = it.pair / p.chunks;
            const int used = (it.len + a.page - 1) >> P;  // pages that hold tokens
            auto page_of = [&](int tile) {
                const int index = tile * ppt + lane;
                return lane < ppt && index < used ? page_at(a, it.b, index) : -2;
            };
            int pg = page_of(it.tile0);
            for (int t = it.tile0; ok && t < it.tile0 + it.n; ++t) {
                const int ahead = t + 1 < it.tile0 + it.n ? page_of(t + 1) : -2;
                const bool good = pg >= 0 && pg < a.num_pages;
                if (!good && pg != -2) atomicOr(status, kStatusInvalid);
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, good)) * (a.page * D);
                for (int kv = 0; kv < 2; ++kv) {
                    const int s = slot % S;
                    if (slot >= S && !wait(bar_kv_empty + s, ((slot / S) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(bar_kv_full + s, bytes);
                    __syncwarp();
                    if (good)
                        tma_load_3d(sRing + s * C::kTileBytes + lane * a.page * D, kv ? &tmV : &tmK, bar_kv_full + s, 0, 0,
                                    pg * a.Hkv + head);
                    __syncwarp();
                    ++slot;
                }
                pg = ahead;
            }
        }
        // Every copy issued must land before the block exits.
        int dummy = 0;
        for (int i = max(0, slot - S); i < slot; ++i)
            mbar_wait_bounded(bar_kv_full + i % S, (i / S) & 1, &dummy, status, kStatusTimeout, kTimeoutNs);
        __syncwarp();
    } else if (warp == 5) {
        // ---------------------------------------------------------------- MMA issuer
        const bool leader = elect_one_sync();
        constexpr uint32_t kIdescS = f8_idesc(128, NC, false, false);
        constexpr uint32_t kIdescO = f8_idesc(D, C::NO, true, true);
        const uint64_t qd = smem_desc(smem_u32(sQ), 16, C::kSbo, C::kLayout);
        const uint64_t rd = smem_desc(smem_u32(sRing), 16, C::kSbo, C::kLayout);
        // P: 16-column chunks kTile * 16 bytes apart, in them 8 tokens of 16 bytes, then the next 8
        const uint64_t pd = smem_desc(smem_u32(sP), 128, kTile * 16, kLayoutNone);
        auto kv_ready = [&](int i) { return wait(bar_kv_full + i % S, (i / S) & 1); };
        // S(n) of the piece that it belongs to
        auto issue_s = [&](int n) -> bool {
            const int i = 2 * n, s = i % S;
            if (!kv_ready(i)) return false;
            if (n >= 2 && !wait(bar_s_empty + (n & 1), (n / 2 - 1) & 1)) return false;
            tc_fence_after_sync();
            if (leader) {
                const uint64_t kd = rd + static_cast<uint32_t>(s * (C::kTileBytes >> 4));
#pragma unroll
                for (int part = 0; part < PARTS; ++part)
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk)
                        tc_mma_f8(tbase + (n & 1) * NC, kd + 2 * kk, qd + part * (C::kQBytes >> 4) + 2 * kk, kIdescS,
                                  part > 0 || kk > 0 ? 1u : 0u);
                tc_commit(bar_s_full + (n & 1));
                tc_commit(bar_kv_empty + s);
            }
            __syncwarp();
            return true;
        };
        auto issue_pv = [&](int n, bool first) -> bool {
            const int i = 2 * n + 1, s = i % S;
            if (!kv_ready(i) || !wait(bar_p_full + (n & 1), (n / 2) & 1)) return false;
            tc_fence_after_sync();
            if (leader) {
                const uint64_t vd = rd + static_cast<uint32_t>(s * (C::kTileBytes >> 4));
                const uint64_t b = pd + static_cast<uint32_t>((n & 1) * (C::kPBytes >> 4));
#pragma unroll
                for (int kk = 0; kk < kTile / 32; ++kk)
                    tc_mma_f8(tbase + col_o, vd + kk * ((32 * D) >> 4), b + kk * ((32 * 16) >> 4), kIdescO,
                              first && kk == 0 ? 0u : 1u);
                tc_commit(bar_pv_done + (n & 1));
                tc_commit(bar_kv_empty + s);
            }
            __syncwarp();
            return true;
        };
        int n = 0;  // running number of the tile
        bool ok = true;
        for (int k = 0; ok && it.next(); ++k) {
            ok = wait(bar_q_full, k & 1) && issue_s(n);
            for (int i = 0; ok && i < it.n; ++i) {
                if (i + 1 < it.n) ok = issue_s(n + 1);
                else if (leader) tc_commit(bar_q_empty);
                __syncwarp();
                ok = ok && issue_pv(n, i == 0);
                ++n;
            }
        }
        if (leader) tc_commit(bar_drain);
        __syncwarp();
        int dummy = 0;
        mbar_wait_bounded(bar_drain, 0, &dummy, status, kStatusTimeout, kTimeoutNs);
        __syncwarp();
    } else if (warp == 6) {
        // ---------------------------------------------------------------- Q: a row (head) at a time, D / 32 channels a lane
        constexpr int E = D / 32;
        for (int k = 0; it.next(); ++k) {
            const int head0 = it.pair / p.chunks * p.G + it.pair % p.chunks * p.per;
            const int heads = min(p.per, p.G - it.pair % p.chunks * p.per);
            uint32_t raw[GC][E / 2];
#pragma unroll
            for (int g = 0; g < GC; ++g)
#pragma unroll
                for (int i = 0; i < E / 2; ++i)
                    raw[g][i] = g < heads ? *reinterpret_cast<const uint32_t*>(a.q + it.b * a.q_seq + (head0 + g) * a.q_head +
                                                                               lane * E + 2 * i)
                                          : 0u;
            if (k > 0 && !wait(bar_q_empty, (k - 1) & 1)) break;
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                float x[E], top = 0.f;
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    widen2<FP16>(raw[g][i], x[2 * i], x[2 * i + 1]);
                    top = fmaxf(top, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
                }
                top = redux_max(top);
                const int e = e4m3_exponent(top);
                // an infinite query has no finite parts: NaN, as its products with the keys are
                const float down = isinf(top) ? NAN : exp2_neg_int(e);
#pragma unroll
                for (int i = 0; i < E; ++i) x[i] *= down;
                if (lane == 0) sCol[g] = log2_to_float(e + 127) * p.kq;
#pragma unroll
                for (int part = 0; part < PARTS; ++part) {
                    uint32_t w = 0;
#pragma unroll
                    for (int i = 0; i < E; i += 2) {
                        const uint32_t c = pack_e4m3x2(x[i], x[i + 1]);
                        float v0, v1;
                        unpack_e4m3x2(c, v0, v1);
                        x[i] -= v0;
                        x[i + 1] -= v1;
                        w |= c << (8 * i);
                    }
                    // swizzled like a TMA tile of D-byte rows
                    const int byte = lane * E;
                    const int chunk = D == 128 ? (byte >> 4) ^ (g & 7) : (byte >> 4) ^ ((g >> 1) & 3);
                    uint8_t* at8 = sQ + part * C::kQBytes + g * D + chunk * 16 + (byte & 15);
                    if constexpr (E == 4) *reinterpret_cast<uint32_t*>(at8) = w;
                    else *reinterpret_cast<uint16_t*>(at8) = static_cast<uint16_t>(w);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_q_full);
        }
    } else {
        // ---------------------------------------------------------------- softmax: a thread per token
        // The four warps meet at named barriers, so none of them leaves early: a wait that gave up is recorded
        // (the flag makes the others give up at once) and the run goes on to its end, its results unspecified.
        const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
        const uint32_t t_o = tbase + lane_base + col_o;
        int n = 0;
        for (int k = 0; it.next(); ++k) {
            const int chunk = it.pair % p.chunks, head = it.pair / p.chunks;
            const int head0 = head * p.G + chunk * p.per, heads = min(p.per, p.G - chunk * p.per);
            const int last = it.tile0 + it.n;
            // The token's page two tiles ahead, its page's exponents one ahead.
            auto page_of = [&](int tile) {
                const int token = tile * kTile + tid;
                return tile < last && token < it.len ? page_at(a, it.b, token >> P) : -1;
            };
            auto scales_of = [&](int pg) -> uint32_t {  // K's exponent byte, V's << 8, bit 16: valid
                if (pg < 0 || pg >= a.num_pages) return 0;
                const int64_t cell = static_cast<int64_t>(pg) * a.Hkv + head;
                return a.k_scales[cell] | a.v_scales[cell] << 8 | 1u << 16;
            };
            uint32_t sc = scales_of(page_of(it.tile0));
            int pg1 = page_of(it.tile0 + 1);
            float m[GC], l[GC], col[GC];
            uint32_t ev = 0;  // largest exponent of V so far
            wait(bar_q_full, k & 1);
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                m[g] = -INFINITY;
                l[g] = 0.f;
                col[g] = sCol[g];
            }
            named_barrier_sync(2, 128);  // all have read sCol
            if (tid == 0) mbar_arrive(bar_q_empty);
            for (int t = it.tile0; t < last; ++t, ++n) {
                const uint32_t sc1 = scales_of(pg1);
                const int pg2 = page_of(t + 2);
                wait(bar_s_full + (n & 1), (n / 2) & 1);
                tc_fence_after_sync();
                float s[GC];
                {
                    uint32_t r[GC];
                    tmem_ld<GC>(tbase + lane_base + (n & 1) * NC, r);
#pragma unroll
                    for (int g = 0; g < GC; ++g) s[g] = __uint_as_float(r[g]);
                }
                tc_fence_before_sync();
                mbar_arrive(bar_s_empty + (n & 1));
                const bool valid = sc >> 16;
                const float ks = log2_to_float(sc & 0xFFu);
                const uint32_t my_ev = (sc >> 8) & 0xFFu;
                float* mx = sMax + (n & 1) * NC * 4;
                float keep = 0.f;
#pragma unroll
                for (int g = 0; g < GC; ++g) {
                    s[g] = valid ? s[g] * (ks * col[g]) : -INFINITY;
                    const float top = redux_max(s[g]);
                    if (lane == g) keep = top;
                }
                if (lane < GC) mx[lane * 4 + warp] = keep;
                const uint32_t top_ev = __reduce_max_sync(0xffffffffu, valid ? my_ev : 0u);
                if (lane == 0) sEv[(n & 1) * 4 + warp] = top_ev;
                named_barrier_sync(2, 128);
                const uint4 e4 = *reinterpret_cast<const uint4*>(sEv + (n & 1) * 4);
                const uint32_t ev_tile = max(max(e4.x, e4.y), max(e4.z, e4.w));
                const bool first = t == it.tile0;
                bool grown = first || ev_tile > ev;
                float m_tile[GC];
#pragma unroll
                for (int g = 0; g < GC; ++g) {
                    const float4 v = *reinterpret_cast<const float4*>(mx + g * 4);
                    m_tile[g] = fmaxf(fmax3(v.x, v.y, v.z), v.w);
                    grown |= m_tile[g] > m[g] + kGrow || (m[g] == -INFINITY && m_tile[g] > -INFINITY);
                }
                // P's buffer: PV(n - 2) has read it
                if (n >= 2) wait(bar_pv_done + (n & 1), (n / 2 - 1) & 1);
                if (grown) {  // the same in every thread
                    const uint32_t ev_new = first ? ev_tile : max(ev, ev_tile);
                    const float f = first ? 1.f : pow2_neg(ev_new - ev);
                    float alpha[GC];
#pragma unroll
                    for (int g = 0; g < GC; ++g) {
                        const bool up = m_tile[g] > m[g] + kGrow || (m[g] == -INFINITY && m_tile[g] > -INFINITY);
                        const float m_new = up ? m_tile[g] : m[g];
                        alpha[g] = up ? ex2_approx(m[g] - m_new) : 1.f;
                        l[g] *= alpha[g];
                        alpha[g] *= f;
                        m[g] = m_new;
                    }
                    ev = ev_new;
                    if (!first) {
                        wait(bar_pv_done + ((n - 1) & 1), ((n - 1) / 2) & 1);
                        tc_fence_after_sync();
#pragma unroll
                        for (int c = 0; c < C::NO / 16; ++c) {
                            uint32_t r[16];
                            tmem_ld<16>(t_o + 16 * c, r);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int g = (16 * c + i) % NC;
                                r[i] = g < GC ? __float_as_uint(__uint_as_float(r[i]) * alpha[g < GC ? g : 0]) : 0u;
                            }
                            tmem_st16(t_o + 16 * c, r);
                        }
                        tmem_st_wait();
                    }
                }
                // P in units of 2^ev: weights times 2^(own exponent - ev) * 32
                const float vf = valid ? pow2_neg(ev - my_ev) * kPUnit : 0.f;
                uint8_t* pb = sP + (n & 1) * C::kPBytes + tid * 16;
#pragma unroll
                for (int c = 0; c < NC / 16; ++c) {
                    uint32_t w[PARTS][4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int g = 16 * c + 4 * q + i;
                            if (g < GC) {
                                const float pr = ex2_approx(s[g < GC ? g : 0] - (m[g < GC ? g : 0] == -INFINITY ? 0.f : m[g < GC ? g : 0]));
                                l[g < GC ? g : 0] += pr;
                                x[i] = pr * vf;
                            } else {
                                x[i] = 0.f;
                            }
                        }
#pragma unroll
                        for (int part = 0; part < PARTS; ++part) {
                            if (16 * c + 4 * q >= GC) {
                                w[part][q] = 0;
                                continue;
                            }
                            const uint32_t lo = pack_e4m3x2(x[0], x[1]), hi = pack_e4m3x2(x[2], x[3]);
                            w[part][q] = lo | hi << 16;
                            if (part + 1 < PARTS) {
                                float v[4];
                                unpack_e4m3x2(lo, v[0], v[1]);
                                unpack_e4m3x2(hi, v[2], v[3]);
#pragma unroll
                                for (int i = 0; i < 4; ++i) x[i] = (x[i] - v[i]) * 16.f;
                            }
                        }
                    }
#pragma unroll
                    for (int part = 0; part < PARTS; ++part)
                        *reinterpret_cast<uint4*>(pb + (part * (NC / 16) + c) * (kTile * 16)) =
                            make_uint4(w[part][0], w[part][1], w[part][2], w[part][3]);
                }
                // V rows of no token: zero, so that 0 * (what they hold) is 0.
                if (__any_sync(0xffffffffu, !valid)) {
                    const int i = 2 * n + 1, sl = i % S;
                    wait(bar_kv_full + sl, (i / S) & 1);
                    if (!valid) {
                        uint4* vr = reinterpret_cast<uint4*>(sRing + sl * C::kTileBytes + tid * D);
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) vr[c] = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                mbar_arrive(bar_p_full + (n & 1));
                sc = sc1;
                pg1 = pg2;
            }
            // End of the piece: the row sums over the tile's threads, then O^T / l.
            float* sum = sMax + (n & 1) * NC * 4;  // free until the next tile's maxima
            float keep = 0.f;
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                const float v = warp_sum(l[g]);
                if (lane == g) keep = v;
            }
            if (lane < GC) sum[lane * 4 + warp] = keep;
            wait(bar_pv_done + ((n - 1) & 1), ((n - 1) / 2) & 1);
            tc_fence_after_sync();
            named_barrier_sync(2, 128);
            float o[GC];
#pragma unroll
            for (int part = PARTS - 1; part >= 0; --part) {
                uint32_t r[GC];
                tmem_ld<GC>(t_o + part * NC, r);
#pragma unroll
                for (int g = 0; g < GC; ++g)
                    o[g] = part == PARTS - 1 ? __uint_as_float(r[g]) : fmaf(o[g], 1.f / 16.f, __uint_as_float(r[g]));
            }
            tc_fence_before_sync();
            const float unit = log2_to_float(ev) * (1.f / kPUnit);
            // lane -> channel: 128 rows lie in all lanes, 64 in the first 16 of each warp
            const int ch = D == 128 ? tid : warp * 16 + lane;
            const bool mine = D == 128 || lane < 16;
            const bool whole = it.begins && it.ends;
            float* slot = reinterpret_cast<float*>(a.scratch) + (2 * static_cast<size_t>(cta) + (it.x - it.n == x0 ? 0 : 1)) * C::kSlotFloats;
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                const float4 v = *reinterpret_cast<const float4*>(sum + g * 4);
                const float lt = (v.x + v.y) + (v.z + v.w);
                const bool none = lt == 0.f;  // every token left out
                const float val = none ? 0.f : o[g] * (1.f / lt) * unit;
                const float L = none ? -INFINITY : m[g] + log2f(lt);  // log2 of the sum of weights
                if (g < heads) {
                    if (whole) {
                        if (mine) a.o[it.b * a.o_seq + (head0 + g) * a.o_head + ch] = static_cast<uint16_t>(narrow2<FP16>(val, 0.f));
                        if (a.lse != nullptr && tid == g)
                            a.lse[static_cast<int64_t>(it.b) * a.Hq + head0 + g] = L * 0.693147180559945f;
                    } else {
                        if (mine) slot[g * D + ch] = val;
                        if (tid == g) slot[GC * D + g] = L;
                    }
                }
            }
            named_barrier_sync(2, 128);  // the sums are read before the next piece writes maxima there
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after_sync();
        tmem_dealloc(tbase, C::kCols);
    }
}

// Joins the parts of the pairs that several blocks had, in the order of the
// list: o = sum_c w_c o_c / sum_c w_c, w_c = 2^(L_c - max L).  Block c takes the
// pair that begins in run c and goes on behind it, if there is one; a warp a
// head, D / 32 channels a lane.
template <int D, bool FP16, int GC>
__global__ void __launch_bounds__(256) cache_join_kernel(const __grid_constant__ KParams p) {
    constexpr int E = D / 32;
    using C = Cfg<D, GC, FP16 ? 3 : 2>;
    const AttendArgs& a = p.a;
    const int cta = blockIdx.x, pairs = a.Hkv * p.chunks, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Where at = locate(a, pairs, [&](int64_t total) { return run_start(total, cta + 1, p.ctas) - 1; });
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t lo = run_start(at.total, cta, p.ctas), hi = at.at + 1;
    if (hi <= lo) return;
    const int tiles = tiles_of(clean_len(a, at.b));
    const int pair = static_cast<int>((at.at - at.base) / tiles);
    const int64_t first = at.base + static_cast<int64_t>(pair) * tiles, end = first + tiles;
    if (end == hi || first < lo) return;  // ends here, or began before
    int c1 = cta + 1;
    while (run_start(at.total, c1 + 1, p.ctas) < end) ++c1;  // the last run with a part
    const int head = pair / p.chunks, chunk = pair % p.chunks;
    const int head0 = head * p.G + chunk * p.per, heads = min(p.per, p.G - chunk * p.per);
    const float* slots = reinterpret_cast<const float*>(a.scratch);
    auto slot_of = [&](int c) { return slots + (2 * static_cast<size_t>(c) + (c == cta && first > lo ? 1 : 0)) * C::kSlotFloats; };
    for (int g = warp; g < heads; g += 8) {
        float top = -INFINITY;
        for (int c = cta + lane; c <= c1; c += 32)
            if (run_start(at.total, c, p.ctas) < run_start(at.total, c + 1, p.ctas)) top = fmaxf(top, slot_of(c)[GC * D + g]);
        top = warp_max(top);
        const float base = top == -INFINITY ? 0.f : top;
        float acc[E] = {}, total = 0.f;
        for (int c = cta; c <= c1; ++c) {
            if (run_start(at.total, c, p.ctas) == run_start(at.total, c + 1, p.ctas)) continue;  // an empty run
            const float* slot = slot_of(c);
            const float w = exp2f(slot[GC * D + g] - base);
            total += w;
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = fmaf(w, slot[g * D + lane * E + i], acc[i]);
        }
        const float inv = total == 0.f ? 0.f : 1.f / total;  // 0: every part's tokens were left out
        uint16_t* out = a.o + at.b * a.o_seq + (head0 + g) * a.o_head + lane * E;
#pragma unroll
        for (int i = 0; i < E; i += 2) *reinterpret_cast<uint32_t*>(out + i) = narrow2<FP16>(acc[i] * inv, acc[i + 1] * inv);
        if (a.lse != nullptr && lane == 0)
            a.lse[static_cast<int64_t>(at.b) * a.Hq + head0 + g] =
                (base + log2f(total)) * 0.693147180559945f;
    }
}

// Codes [cells, page, d]: boxes of one page.
bool encode_pages(CUtensorMap* map, const void* base, int d, int page, int64_t cells) {
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page), static_cast<cuuint64_t>(cells)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(d) * page};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(page), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool FP16, int GC>
cudaError_t launch_impl(const AttendArgs& a, int dev, int G, int chunks, int per, cudaStream_t stream) {
    using C = Cfg<D, GC, FP16 ? 3 : 2>;
    static bool ready[kMaxDevices] = {};
    if (!ready[dev]) {
        cudaError_t e = cudaFuncSetAttribute(cache_attend_kernel<D, FP16, GC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             C::kSmemBytes);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    CUtensorMap tk, tv;
    if (a.num_pages > 0) {
        const int64_t cells = static_cast<int64_t>(a.num_pages) * a.Hkv;
        if (!encode_pages(&tk, a.k_codes, D, a.page, cells) || !encode_pages(&tv, a.v_codes, D, a.page, cells))
            return cudaErrorInvalidValue;
    } else {  // never read: no page is in range
        memset(&tk, 0, sizeof(tk));
        tv = tk;
    }
    KParams p{};
    p.a = a;
    p.kq = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    p.G = G;
    p.chunks = chunks;
    p.per = per;
    p.ctas = min(sm_count(dev), kMaxSms) * kCtasPerSm;
    cache_attend_kernel<D, FP16, GC><<<p.ctas, kThreads, C::kSmemBytes, stream>>>(tk, tv, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.ctas);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_join_kernel<D, FP16, GC>, p);
}

template <int D, bool FP16>
cudaError_t launch_heads(const AttendArgs& a, int dev, cudaStream_t stream) {
    const int G = a.Hq / a.Hkv, chunks = (G + kMaxCols - 1) / kMaxCols, per = (G + chunks - 1) / chunks;
    if (per <= 4) return launch_impl<D, FP16, 4>(a, dev, G, chunks, per, stream);
    if (per <= 8) return launch_impl<D, FP16, 8>(a, dev, G, chunks, per, stream);
    if (per <= 16) return launch_impl<D, FP16, 16>(a, dev, G, chunks, per, stream);
    return launch_impl<D, FP16, 32>(a, dev, G, chunks, per, stream);
}

}  // namespace

// Two slots a block, each with a part's O and log-sums of up to kMaxCols heads.
size_t cache_attend_scratch_bytes(int Hq, int Hkv, int d) {
    const int G = Hq / Hkv, chunks = (G + kMaxCols - 1) / kMaxCols, per = (G + chunks - 1) / chunks;
    const size_t gc = per <= 4 ? 4 : per <= 8 ? 8 : per <= 16 ? 16 : 32;
    return 2 * static_cast<size_t>(kMaxSms) * kCtasPerSm * gc * (d + 1) * sizeof(float);
}

cudaError_t launch_cache_attend(const AttendArgs& a, cudaStream_t stream) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (a.d == 128) return a.fp16 ? launch_heads<128, true>(a, dev, stream) : launch_heads<128, false>(a, dev, stream);
    return a.fp16 ? launch_heads<64, true>(a, dev, stream) : launch_heads<64, false>(a, dev, stream);
}

}  // namespace mxattn

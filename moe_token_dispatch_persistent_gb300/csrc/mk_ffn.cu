// mk_ffn.cu -- mk_moe_ffn_decode: the whole gated expert layer for a few
// tokens in one persistent kernel.
//
//   experts of token t: the k largest logits; gates: softmax over them (an
//   expert whose logit is -inf is left out)
//   h = silu(x . W1[e]) * (x . W3[e]),   out[t] = sum_j gate_j h . W2[e_j]
//
// For a few tokens the chosen experts' weights are all the traffic, each used
// for the few rows routed to its expert, so the kernel is a stream of weights
// (read once for up to 64 rows of an expert, twice for one with 65 to 128).
// One step is 32 KiB of them, 256 columns wide; a unit of work is a few
// consecutive steps of one block of columns: first the units of W1 and W3 of
// every chosen expert, then those of W2, taken in order from one counter.
// SMs that read slower take fewer, and by the time the first expert's W2 is
// reached its h has long been complete, unless it is the only one.
//
// The products run on tcgen05 with the weights as the 128-row operand (their
// columns are its rows, M-major as they lie in memory, loaded by TMA) and the
// expert's rows of x or h as the columns (N = 16..128), gathered by TMA
// tile::gather4.  Roles of a CTA's warps: one takes units and loads their
// weights, waiting for nothing but free stages, so the stream goes on while an
// h is still being completed; one gathers rows (and waits for an expert's h
// before its first use); one issues products; eight drain accumulators; one
// counts the pieces of h and three complete it.
//
// A unit's sums are a piece in fp32 in the workspace.  The CTA that delivers
// the last piece of 256 columns of h adds them up, applies SwiGLU and
// publishes them; after the last barrier of the grid the combine adds the
// pieces of each token's k rows.  Both add in the order of K: which CTA
// computed a piece, and when, changes nothing.
//
// 16-bit weights: h is kept as the sum of two bf16 values, which take
// neighbouring columns of the same product (16 significant bits): the tensor
// core has columns to spare here, and one rounding fewer reaches the output.
// 8-bit weights: a weight scale per 128 x 128 block and a scale of x and h per
// row and 128 columns, so one step is one block of K; its products leave the
// tensor core after each step and are added up in fp32 registers with their
// scales.
//
// Measured on GB300: 128 tokens over 256 e4m3 experts of 7168 x 2048 1.55 to
// 1.59 ms, 48 tokens over 112 bf16 experts of 4096 x 1536 0.58 to 0.59 ms (both
// 7.0 TB/s of weights or more), one token over two of 4096 x 14336 0.112 ms (6.3
// TB/s), two tokens through a layer of 512 x 1024 22 us (latency).  More rows an
// expert cost more: 77 tokens over 7 bf16 experts of 3840 x 1984 (44 rows each)
// 104 us, 3.1 TB/s; over 4 of 4096 x 14336 64 rows each 351 us, 128 rows 621.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "mk.h"
#include "mk_common.h"
#include "mk_host.h"
#include "mk_ptx.cuh"
#include "mk_quant.cuh"
#include "mk_wait.cuh"

namespace mk {
namespace {

constexpr int FFN_MAX_T = 128;
constexpr int FFN_MAX_ROWS = FFN_MAX_T * MAX_K;
constexpr int FFN_MAX_CTAS = 160;

// Warps: weight loads, products, eight draining accumulators (TMEM lanes
// 32 * (warp % 4); two warps share a quarter and take turns at its column
// blocks), row loads, counting of pieces, three that complete h.
constexpr int WARP_A = 0, WARP_MMA = 1, WARP_EPI = 2, EPI_WARPS = 8, WARP_B = WARP_EPI + EPI_WARPS;
constexpr int WARP_COUNT = WARP_B + 1, WARP_FIN = WARP_COUNT + 1, FIN_WARPS = 3;
constexpr int FFN_WARPS = WARP_FIN + FIN_WARPS;
constexpr int FFN_THREADS = FFN_WARPS * 32;  // 128 registers each: about 200 bytes of them are spilled

// Rows of an expert that are multiplied together; an expert with more is
// taken in parts, each reading its weights.  (Two accumulators of 64 columns
// for the value and the remainder of h, twice, fill TMEM; with 8 bits the
// sums of a step are kept in registers, and those end there too.)
constexpr int MAX_N = 64;
constexpr int MAX_PARTS = MAX_E + FFN_MAX_ROWS / MAX_N;

constexpr int STEP_BYTES = 32768;  // weights of one step
constexpr int ACC_COLS = 256;      // weight columns of a tile: two accumulators of 128
constexpr int GROUP8 = 128;        // rows and columns of an 8-bit scale block
// Stages of the ring.  Four hold 19 MB of weights in flight over the GPU, 2.9
// us of its bandwidth; with six every other access (row loads, pieces,
// counters) waited behind 4.3 us of them and the kernel took 1-5% longer.
constexpr int STAGES_F = 4;
constexpr int FFN_MAX_BUFS = 8;
// A stage: the step's weights, then up to 64 rows (16 bits: twice, for h's values and remainders).
template <bool FP8>
constexpr int STAGE_F = STEP_BYTES + (FP8 ? 1 : 2) * MAX_N * 128;
constexpr int RING_BYTES = STAGES_F * STAGE_F<false>;
// 8 bits: the scales of a step (up to 64 rows, then the two weight blocks) in
// a ring of their own after the stages, longer than the stages and accumulator
// buffers that lie between their load and their use.
constexpr int SCALE_SLOTS = 16, SCALE_FLOATS = MAX_N + 4;
constexpr int SCALE_AT = STAGES_F * STAGE_F<true>;
static_assert(SCALE_SLOTS >= STAGES_F + FFN_MAX_BUFS && SCALE_AT + SCALE_SLOTS * SCALE_FLOATS * 4 <= RING_BYTES, "scale ring");
constexpr int MAX_TILES1 = MAX_PARTS * (32768 / ACC_COLS);
// Units: about this many per CTA, of at least this many steps.  Pieces of more
// floats than this only where one unit covers all of K.
constexpr uint32_t UNITS_PER_CTA = 8, MIN_CHUNK = 4;
constexpr size_t PIECE_FLOATS = size_t(8) << 20;
constexpr int INFO_SLOTS = 8;
constexpr int JOBS = 2;  // blocks of h handed to the completing warps
constexpr long long FFN_SPIN_NS = 2000000000LL;

struct FfnCtl {
    uint32_t routed;  // CTAs whose tokens are routed
    uint32_t done;    // CTAs whose output pieces are written
    uint32_t exited;
    uint32_t abort;
    uint32_t next;    // units taken beyond the first of every CTA
    uint32_t pad[59];
    uint32_t ready[MAX_PARTS];        // blocks of h published, per part of the chosen experts
    uint32_t arrived[MAX_TILES1];     // pieces of each block of h delivered
};

struct FfnParams {
    const float* logits;
    const float* x_scale;
    const float* w1_scale;
    const float* w3_scale;
    const float* w2_scale;
    __nv_bfloat16* out;
    FfnCtl* ctl;
    uint8_t* ids;       // [T*k] chosen experts, and
    float* gates;       // [T*k] their gates (when routing is shared out)
    uint8_t* h;         // [2][T*k][F] bf16 (value and remainder) or [T*k][F] e4m3
    float* h_scale;     // [T*k][F/128]
    float* piece[2];    // sums of the units: [matrix and chunk of K][T*k][columns, whole blocks]
    size_t room[2];     // floats of each
    DevError* err;
    int T, H, F, E, k;
};

struct FfnMaps {
    CUtensorMap x, w1, w3, w2, h;
};

// A unit of work as its CTA's warps see it.
struct Unit {
    int half, second;  // first or second half of the layer; W3 instead of W1
    int a, expert;     // part of the chosen experts and its expert,
    int n, off;        // its rows and the first of them
    int blk, c;        // block of columns, chunk of K
    uint32_t k0, k1;   // steps along K
    int end;           // 1: no more units
};

struct FfnSmem {
    uint64_t weights_in[STAGES_F], rows_in[STAGES_F], empty[STAGES_F];
    uint64_t acc_full[FFN_MAX_BUFS], acc_empty[FFN_MAX_BUFS];
    uint64_t scales_in[SCALE_SLOTS], scales_out[SCALE_SLOTS];
    uint64_t info_in[INFO_SLOTS], info_out[INFO_SLOTS], piece_in[INFO_SLOTS];
    uint64_t drain;
    Unit unit[INFO_SLOTS];         // this CTA's units in turn
    uint32_t tmem_base;
    int ok, parts, most;           // most: rows of the largest part
    int scan[8];
    uint64_t job_in[JOBS], job_out[JOBS];
    Unit job[JOBS];                // blocks of h being completed,
    uint32_t job_left[JOBS];       // and the warps at work on them
    uint16_t off[MAX_PARTS];       // per part of the chosen experts: its first row,
    uint8_t expert[MAX_PARTS];     // its expert
    uint8_t count[MAX_PARTS];      // and its rows
    uint8_t row_token[FFN_MAX_ROWS];
    uint16_t row_of[FFN_MAX_ROWS]; // per (token, choice): its row or NO_ROW
    float gate[FFN_MAX_ROWS];      // and its gate or MASKED
};
constexpr int FFN_SMEM = RING_BYTES + int(sizeof(FfnSmem)) + 1024;
static_assert(FFN_SMEM <= 232448, "dynamic shared memory of one CTA on sm_103");

// The gate of a chosen expert whose logit is -inf, which gets no row: its
// weights are not read, and nothing that they hold reaches the output.
constexpr float MASKED = -1.f;
constexpr uint16_t NO_ROW = 0xffff;

// Routing scratch, in the ring before the first load.
constexpr int RS_IDS = 0, RS_MASK = FFN_MAX_ROWS, RS_FIRST = RS_MASK + MAX_E * (FFN_MAX_T / 8);

// The layer's units, the same in every CTA.  Index 0: W1 and W3 (K = H,
// columns F), 1: W2 (K = F, columns H).
struct Plan {
    uint32_t ms[2];      // steps along K of a matrix
    uint32_t blocks[2];  // blocks of 256 columns
    uint32_t chunk[2];   // steps of a unit
    uint32_t chunks[2];  // units along K
    uint32_t first_down, units;
};

__device__ __forceinline__ Plan make_plan(const FfnParams& p, int step_rows, uint32_t parts, uint32_t most) {
    Plan q;
    q.ms[0] = uint32_t(p.H / step_rows);
    q.ms[1] = uint32_t(p.F / step_rows);
    q.blocks[0] = uint32_t((p.F + ACC_COLS - 1) / ACC_COLS);
    q.blocks[1] = uint32_t((p.H + ACC_COLS - 1) / ACC_COLS);
    const uint32_t steps[2] = {parts * 2 * q.ms[0] * q.blocks[0], parts * q.ms[1] * q.blocks[1]};
    const uint32_t share = (steps[0] + steps[1]) / gridDim.x;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // Small units even out the SMs' speeds, but each leaves a piece of `most` rows
        // of 1 KiB beside its 32 KiB a step, to be stored, counted and added up: about
        // 8 units per CTA (16 cost up to 15%), and as many steps as rows while that
        // leaves every CTA two units of either half (half as many steps: +18% with 12
        // rows an expert).
        const uint32_t want = max(max(MIN_CHUNK, share / UNITS_PER_CTA), min(most, steps[h] / gridDim.x / 2));
        const uint32_t rows = uint32_t(p.T * p.k) * (h == 0 ? 2 : 1);
        const uint32_t fit = uint32_t(p.room[h] / (size_t(rows) * q.blocks[h] * ACC_COLS));
        const uint32_t n = max(1u, min((q.ms[h] + want / 2) / want, fit));
        q.chunk[h] = (q.ms[h] + n - 1) / n;
        q.chunks[h] = (q.ms[h] + q.chunk[h] - 1) / q.chunk[h];
    }
    q.first_down = parts * 2 * q.chunks[0] * q.blocks[0];
    q.units = q.first_down + parts * q.chunks[1] * q.blocks[1];
    return q;
}

// Neighbours in the order read neighbouring columns of the same rows of
// weights (measured against a block of columns after the other: 109 us instead
// of 114 on one token and two experts of 4096 x 14336, no change elsewhere).
__device__ __forceinline__ Unit unit_of(const FfnSmem* sm, const Plan& q, uint32_t u) {
    Unit s;
    s.end = 0;
    s.half = u >= q.first_down;
    const uint32_t mats = s.half ? 1 : 2, blocks = q.blocks[s.half];
    if (s.half) u -= q.first_down;
    const uint32_t per = mats * q.chunks[s.half] * blocks;
    s.a = int(u / per);
    u -= uint32_t(s.a) * per;
    s.c = int(u / (mats * blocks));
    u -= uint32_t(s.c) * mats * blocks;
    s.second = u >= blocks;
    s.blk = int(s.second ? u - blocks : u);
    s.k0 = uint32_t(s.c) * q.chunk[s.half];
    s.k1 = min(q.ms[s.half], s.k0 + q.chunk[s.half]);
    s.expert = sm->expert[s.a];
    s.n = sm->count[s.a];
    s.off = sm->off[s.a];
    return s;
}

// Row r of a unit's piece.
__device__ __forceinline__ float* piece_row(const FfnParams& p, const Plan& q, int half, uint32_t part, int row) {
    return p.piece[half] + (size_t(part) * (p.T * p.k) + row) * (size_t(q.blocks[half]) * ACC_COLS);
}

__device__ __forceinline__ uint8_t* ffn_ring() {
    extern __shared__ uint8_t ffn_raw[];
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ffn_raw) + 1023) & ~uintptr_t(1023));
}

__device__ __forceinline__ int pad16(int n) { return (n + 15) & ~15; }

// ------------------------------------------------------------- routing -----

// Order of the logits as unsigned integers, above 0: -0 counts as 0, NaN as -inf.
__device__ __forceinline__ uint32_t ordered(float v) {
    if (v != v) v = -INFINITY;
    const uint32_t u = __float_as_uint(v + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}

// One token by one warp: the k largest logits in descending order, ties to
// the lower expert, and the softmax over them (MASKED where the logit is -inf).
__device__ void route_token(const FfnParams& p, int t, uint8_t* ids, float* gates) {
    const int lane = threadIdx.x & 31;
    const float* row = p.logits + size_t(t) * p.E;
    uint32_t key[MAX_E / 32];
#pragma unroll
    for (int i = 0; i < MAX_E / 32; ++i) key[i] = lane + 32 * i < p.E ? ordered(__ldg(row + lane + 32 * i)) : 0u;
    float value = -INFINITY;
    int id = 0;
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < MAX_E / 32; ++i)
            if (key[i] > best) {
                best = key[i];
                at = lane + 32 * i;
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        const int e = int(__reduce_min_sync(0xffffffffu, best == top ? uint32_t(at) : 0xffffu));
#pragma unroll
        for (int i = 0; i < MAX_E / 32; ++i)
            if (lane + 32 * i == e) key[i] = 0;
        if (lane == j) {
            value = unordered(top);
            id = e;
        }
    }
    const float v0 = __shfl_sync(0xffffffffu, value, 0);
    const float w = lane < p.k && value > -INFINITY ? expf(value - v0) : 0.f;
    float sum = 0.f;
    for (int j = 0; j < p.k; ++j) sum += __shfl_sync(0xffffffffu, w, j);
    if (lane < p.k) {
        ids[t * p.k + lane] = uint8_t(id);
        gates[t * p.k + lane] = value == -INFINITY ? MASKED : sum > 0.f ? w / sum : 0.f;
    }
}

// The tables of every CTA from the chosen experts in the scratch: rows sorted
// by (expert, token).  An expert's tokens are a bit mask, so a row's place is
// a count of bits and no order of arrival matters.
__device__ void build_rows(const FfnParams& p, FfnSmem* sm, uint8_t* scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int WORDS = FFN_MAX_T / 32;
    const uint8_t* ids = scratch + RS_IDS;
    uint32_t* mask = reinterpret_cast<uint32_t*>(scratch + RS_MASK);
    uint16_t* first_row = reinterpret_cast<uint16_t*>(scratch + RS_FIRST);
    const int rows = p.T * p.k;
    for (int i = tid; i < p.E * WORDS; i += FFN_THREADS) mask[i] = 0;
    if (tid == 0) sm->most = 0;
    __syncthreads();
    for (int i = tid; i < rows; i += FFN_THREADS) {
        if (sm->gate[i] == MASKED) continue;
        const int t = i / p.k;
        atomicOr(&mask[ids[i] * WORDS + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    // rows and parts before each expert, 16 bits each
    uint32_t mine = 0;
    if (tid < p.E) {
        int c = 0;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) c += __popc(mask[tid * WORDS + w]);
        mine = uint32_t(c) | uint32_t((c + MAX_N - 1) / MAX_N) << 16;
    }
    uint32_t run = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += o;
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, min(mine & 0xffffu, uint32_t(MAX_N)));
    if (warp < MAX_E / 32) {
        if (lane == 31) sm->scan[warp] = int(run);
        if (lane == 0) atomicMax(&sm->most, int(top));
    }
    __syncthreads();
    if (tid < MAX_E) {
        uint32_t base = run - mine;
        for (int w = 0; w < warp; ++w) base += uint32_t(sm->scan[w]);
        const int a = int(base >> 16), first = int(base & 0xffffu), c = int(mine & 0xffffu);
        for (int i = 0; i < int(mine >> 16); ++i) {
            sm->expert[a + i] = uint8_t(tid);
            sm->count[a + i] = uint8_t(min(MAX_N, c - i * MAX_N));
            sm->off[a + i] = uint16_t(first + i * MAX_N);
        }
        first_row[tid] = uint16_t(first);
        if (tid == MAX_E - 1) sm->parts = int((base + mine) >> 16);
    }
    __syncthreads();
    for (int i = tid; i < rows; i += FFN_THREADS) {
        if (sm->gate[i] == MASKED) {
            sm->row_of[i] = NO_ROW;
            continue;
        }
        const int t = i / p.k, e = ids[i];
        int before = 0;
        for (int w = 0; w < (t >> 5); ++w) before += __popc(mask[e * WORDS + w]);
        before += __popc(mask[e * WORDS + (t >> 5)] & ((1u << (t & 31)) - 1u));
        const int r = first_row[e] + before;
        sm->row_of[i] = uint16_t(r);
        sm->row_token[r] = uint8_t(t);
    }
}

// --------------------------------------------------------------- roles -----

struct Accs {
    uint32_t bufs, acc_stride;  // accumulator pairs, TMEM columns of one accumulator
};

struct Turn {  // position in a ring of n slots
    uint32_t i = 0, phase = 0;
    __device__ void next(uint32_t n) {
        if (++i == n) {
            i = 0;
            phase ^= 1u;
        }
    }
};

// The stages that a loading warp has issued, so that after a wait gave up it
// can let its loads land before the CTA exits.
struct Issued {
    uint32_t any = 0, parity = 0;  // per stage: issued at all, the phase of its last load
    __device__ void note(const Turn& t) {
        any |= 1u << t.i;
        parity = (parity & ~(1u << t.i)) | (t.phase << t.i);
    }
    __device__ void settle(uint64_t* bars) const {
        const uint64_t t0 = globaltimer();
        for (uint32_t i = 0; i < STAGES_F; ++i)
            if (any >> i & 1u)
                while (!mbar_try_wait(&bars[i], parity >> i & 1u) && globaltimer() - t0 < 5000000ull) {
                }
        __syncwarp();
    }
};

// The CTA's next unit, as the weight loads publish it.  False: no more, or a
// wait gave up (ok is then false).
__device__ __forceinline__ bool next_unit(FfnSmem* sm, Turn& in, const Waiter& w, Unit& s, bool& ok) {
    if (!(ok = warp_await_mbar(&sm->info_in[in.i], in.phase, w, SITE_INFO_FULL))) return false;
    s = sm->unit[in.i];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sm->info_out[in.i]);
    in.next(INFO_SLOTS);
    return s.end == 0;
}

template <bool FP8>
__device__ void weight_loads(const FfnParams& p, const FfnMaps& m, FfnSmem* sm, const Plan& pl,
                             const Waiter& w) {
    constexpr int KB = FP8 ? 128 : 64;   // rows of K in a step
    constexpr int CB = FP8 ? 128 : 64;   // columns of a box
    constexpr int BOX = KB * 128;        // bytes of a box
    const int lane = threadIdx.x & 31;
    uint8_t* ring = ffn_ring();
    const uint64_t pol = l2_policy_evict_first();  // weights are read once, but for experts of more than 64 rows
    Turn st, out;
    Issued mine;
    uint32_t u = blockIdx.x;  // the first unit of every CTA needs no counter
    while (true) {
        if (!warp_await_mbar(&sm->info_out[out.i], out.phase ^ 1u, w, SITE_INFO_EMPTY)) break;
        const bool more = u < pl.units;
        uint32_t ahead = 0;  // taken while this unit's loads are issued
        if (more && lane == 0) ahead = atom_add_relaxed_u32(&p.ctl->next, 1u);
        Unit s = unit_of(sm, pl, more ? u : 0u);
        s.end = !more;
        if (lane == 0) {
            sm->unit[out.i] = s;
            mbar_arrive(&sm->info_in[out.i]);
        }
        out.next(INFO_SLOTS);
        if (!more) return;
        const int ncol = s.half ? p.H : p.F;
        const int row0 = s.expert * (s.half ? p.F : p.H);
        const CUtensorMap* map = s.half ? &m.w2 : s.second ? &m.w3 : &m.w1;
#pragma unroll 1
        for (uint32_t k = s.k0; k < s.k1; ++k) {
            if (!warp_await_mbar(&sm->empty[st.i], st.phase ^ 1u, w, SITE_STAGE_EMPTY)) {
                mine.settle(sm->weights_in);
                return;
            }
            uint64_t* fb = &sm->weights_in[st.i];
            uint8_t* dst = ring + st.i * STAGE_F<FP8>;
            mine.note(st);
            mbar_arrive_expect_tx_elect(fb, STEP_BYTES);
#pragma unroll
            for (int q = 0; q < STEP_BYTES / BOX; ++q) {
                // boxes past the matrix's edge read as zeros
                const int c = s.blk * ACC_COLS + q * CB;
                tma_load_2d_elect_hint(dst + q * BOX, map, c < ncol ? c : ncol, row0 + int(k) * KB, fb, pol);
            }
            st.next(STAGES_F);
        }
        u = gridDim.x + __shfl_sync(0xffffffffu, ahead, 0);
    }
    mine.settle(sm->weights_in);
}

__device__ __forceinline__ void cp_async_4(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <bool FP8>
__device__ void row_loads(const FfnParams& p, const FfnMaps& m, FfnSmem* sm, const Plan& pl,
                          const Waiter& w) {
    constexpr int KB = FP8 ? 128 : 64;
    const int lane = threadIdx.x & 31;
    uint8_t* ring = ffn_ring();
    Turn st, sc, in;
    Issued mine;
    int known = -1;  // the part whose h is known to be complete
    Unit s;
    bool ok;
    while (next_unit(sm, in, w, s, ok)) {
        const int n = s.n, N = pad16(n), off = s.off;
        const int parts = s.half && !FP8 ? 2 : 1;  // h: value and remainder
        if (s.half && s.a != known) {
            ok = __all_sync(0xffffffffu, await_geq(&p.ctl->ready[s.a], pl.blocks[0], w, SITE_TILE_READY));
            fence_proxy_async();  // the other CTAs' stores to h before the loads below
            known = s.a;
        }
        // Lanes take four rows each, the next ones the last n % 4 one by one: no
        // row is read twice (what the rest of the N columns holds is never used).
        const int fours = n >> 2, singles = n & 3;
        const bool four = lane < fours, one = !four && lane < fours + singles;
        const int first = four ? 4 * lane : 4 * fours + (lane - fours);
        int r[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = off + min(first + q, n - 1);
            r[q] = s.half ? i : sm->row_token[i];
        }
        // 8 bits: scales of this lane's rows lane, lane + 32, ... and of the two weight blocks
        const int KB8 = (s.half ? p.F : p.H) / GROUP8, NB8 = (s.half ? p.H : p.F) / GROUP8;
        const float* sx[MAX_N / 32];
        const float* sw = nullptr;
        if constexpr (FP8) {
#pragma unroll
            for (int q = 0; q < MAX_N / 32; ++q) {
                const int i = off + min(lane + 32 * q, n - 1);
                sx[q] = s.half ? p.h_scale + size_t(i) * KB8 : p.x_scale + size_t(sm->row_token[i]) * KB8;
            }
            sw = (s.half ? p.w2_scale : s.second ? p.w3_scale : p.w1_scale) +
                 size_t(s.expert) * KB8 * NB8 + min(2 * s.blk + (lane & 1), NB8 - 1);
        }
#pragma unroll 1
        for (uint32_t k = s.k0; ok && k < s.k1; ++k) {
            if (!(ok = warp_await_mbar(&sm->empty[st.i], st.phase ^ 1u, w, SITE_STAGE_EMPTY))) break;
            uint64_t* fb = &sm->rows_in[st.i];
            uint8_t* dst = ring + st.i * STAGE_F<FP8> + STEP_BYTES;
            mine.note(st);
            mbar_arrive_expect_tx_elect(fb, uint32_t(n * 128 * parts));
            __syncwarp();
            for (int q = 0; q < parts; ++q) {
                const CUtensorMap* map = s.half ? &m.h : &m.x;
                uint8_t* to = dst + (q * N + first) * 128;
                const int R = q * p.T * p.k;
                if (four) tma_gather4(to, map, int(k) * KB, R + r[0], R + r[1], R + r[2], R + r[3], fb);
                else if (one) tma_load_2d(to, map, int(k) * KB, R + r[0], fb);
            }
            if constexpr (FP8) {
                if (!(ok = warp_await_mbar(&sm->scales_out[sc.i], sc.phase ^ 1u, w, SITE_ACC_EMPTY))) break;
                const uint32_t to = smem_u32(ring + SCALE_AT) + sc.i * (SCALE_FLOATS * 4);
#pragma unroll
                for (int q = 0; q < MAX_N / 32; ++q)
                    if (lane + 32 * q < N) cp_async_4(to + (lane + 32 * q) * 4, sx[q] + k);
                if (lane < 2) cp_async_4(to + (MAX_N + lane) * 4, sw + size_t(k) * NB8);
                cp_async_mbar_arrive_noinc(&sm->scales_in[sc.i]);
                sc.next(SCALE_SLOTS);
            }
            __syncwarp();
            st.next(STAGES_F);
        }
        if (!ok) break;
    }
    if (!ok) {
        if (FP8) cp_async_wait_all();
        mine.settle(sm->rows_in);
    }
}

// A value that is the same on every lane, in a uniform register: without this
// the compiler moves each operand of each product there one by one, and the
// issue of the products takes longer than a step's loads.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

template <bool FP8>
__device__ void products(FfnSmem* sm, const Accs& accs, const Waiter& w) {
    const uint32_t bufs = uniform(accs.bufs), acc_stride = uniform(accs.acc_stride);
    const uint32_t tmem = uniform(sm->tmem_base), ring = uniform(smem_u32(ffn_ring()));
    Turn st, buf, in;
    bool issued = false, ok = true;
    Unit s;
    while (ok && next_unit(sm, in, w, s, ok)) {
        // 16 bits: h's values and remainders are columns side by side
        const uint32_t half = uniform(uint32_t(s.half)), steps = uniform(s.k1 - s.k0);
        const uint32_t N = uniform(uint32_t(pad16(s.n))) * (FP8 ? 1 : 1 + half);
        const uint32_t idesc = FP8 ? umma_idesc_e4m3(128, N, true, false) : umma_idesc_bf16(128, N, true, false);
#pragma unroll 1
        for (uint32_t k = 0; k < steps; ++k) {
            // 16 bits: one accumulation per unit; 8 bits: one per step
            if (FP8 || k == 0) {
                if (!(ok = warp_await_mbar(&sm->acc_empty[buf.i], buf.phase ^ 1u, w, SITE_ACC_EMPTY))) break;
            }
            if (!(ok = warp_await_mbar(&sm->rows_in[st.i], st.phase, w, SITE_STAGE_FULL))) break;
            if (!(ok = warp_await_mbar(&sm->weights_in[st.i], st.phase, w, SITE_STAGE_FULL))) break;
            tc_fence_after();
            const uint32_t d = tmem + buf.i * 2u * acc_stride;
            const uint32_t a = ring + st.i * STAGE_F<FP8>, b = a + STEP_BYTES;
            issued = true;
            // Rows K-major: 32 bytes per instruction along their swizzle span.
            // Weights M-major, K rows in groups of 8 that lie 1024 bytes apart.  8
            // bits: 128 columns are one swizzle span, 4 KiB per K = 32.  16 bits: two
            // 64-column chunks 8 KiB apart, 2 KiB per K = 16.
            constexpr uint32_t CHUNK = FP8 ? 16384 : 8192, ADVANCE = FP8 ? 4096 : 2048;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint64_t a0 = umma_desc_sw128(a + kk * ADVANCE, CHUNK, 1024);
                const uint64_t a1 = umma_desc_sw128(a + 16384 + kk * ADVANCE, CHUNK, 1024);
                const uint64_t bd = umma_desc_sw128(b + kk * 32, 16, 1024);
                if constexpr (FP8) {
                    tc_mma_f8_elect(d, a0, bd, idesc, kk != 0);
                    tc_mma_f8_elect(d + acc_stride, a1, bd, idesc, kk != 0);
                } else {
                    tc_mma_f16_elect(d, a0, bd, idesc, k != 0 || kk != 0);
                    tc_mma_f16_elect(d + acc_stride, a1, bd, idesc, k != 0 || kk != 0);
                }
            }
            tc_commit_elect(&sm->empty[st.i]);
            st.next(STAGES_F);
            if (FP8 || k + 1 == steps) {
                tc_commit_elect(&sm->acc_full[buf.i]);
                buf.next(bufs);
            }
        }
    }
    if (issued) {
        // every product has completed before TMEM is freed
        tc_commit_elect(&sm->drain);
        const uint64_t t0 = globaltimer();
        while (!__all_sync(0xffffffffu, mbar_try_wait(&sm->drain, 0u)) && globaltimer() - t0 < 5000000ull) {
        }
    }
    __syncwarp();
}

// Two values of h as the sum of two bf16 values each: the value cut off, and
// what remains with 2^-23 of the value, so that both have its sign and their
// products with an infinite weight are one infinity (rounded to nearest, the
// remainder may be 0 or of the other sign, and the sum NaN).  Of an infinite or
// NaN value both are that.
__device__ __forceinline__ void split_pair(float h0, float h1, uint32_t& hi, uint32_t& lo) {
    const float c0 = __uint_as_float(__float_as_uint(h0) & 0xffff0000u), c1 = __uint_as_float(__float_as_uint(h1) & 0xffff0000u);
    constexpr float ABOVE = 1.1920928955078125e-7f;
    const float r0 = fabsf(h0) < INFINITY ? fmaf(h0, ABOVE, h0 - c0) : h0, r1 = fabsf(h1) < INFINITY ? fmaf(h1, ABOVE, h1 - c1) : h1;
    hi = __byte_perm(__float_as_uint(h0), __float_as_uint(h1), 0x7632);
    const __nv_bfloat162 l = __floats2bfloat162_rn(r0, r1);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}

// ROWS rows from i0 on of a block of 256 columns of a part's h, from their
// pieces, by one warp: eight columns per lane.  BATCH pieces of each matrix are
// loaded together.
template <bool FP8, int ROWS, int BATCH>
__device__ __forceinline__ void complete_rows(const FfnParams& p, const Plan& pl, const Unit& s, int i0) {
    const int lane = threadIdx.x & 31, col = s.blk * ACC_COLS + lane * 8;
    const bool in = col < p.F;  // F is a multiple of 64
    const size_t R = size_t(p.T) * p.k, stride = size_t(pl.blocks[0]) * ACC_COLS;
    const int chunks = int(pl.chunks[0]);
    {
        float v[2][ROWS][8];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[m][r][i] = 0.f;
        const float* src = piece_row(p, pl, 0, 0, s.off + i0) + col;
        for (int c = 0; c < chunks; c += BATCH) {
            float4 u[2][BATCH][ROWS][2];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int x = 0; x < BATCH; ++x)
#pragma unroll
                    for (int r = 0; r < ROWS; ++r)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            u[m][x][r][q] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (in && c + x < chunks && i0 + r < s.n)
                                u[m][x][r][q] = __ldcg(reinterpret_cast<const float4*>(
                                    src + (size_t(m * chunks + c + x) * R + r) * stride + 4 * q));
                        }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int x = 0; x < BATCH; ++x)
#pragma unroll
                    for (int r = 0; r < ROWS; ++r)
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[m][r][i] += (&u[m][x][r][i >> 2].x)[i & 3];
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (i0 + r >= s.n) break;
            float* h = v[0][r];
            // SwiGLU.  The fast exponential is off by 2^-17 of it where a is -88 and far
            // less where the gate is open.  The fast division gives 0 where a
            // denominator lies above 2^126, so a quarter of both is divided.
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[i] = __fdividef(0.25f * h[i], fmaf(0.25f, __expf(-h[i]), 0.25f)) * v[1][r][i];
            const int row = s.off + i0 + r;
            const size_t at = size_t(row) * p.F + col;
            if constexpr (FP8) {
                // 16 lanes hold a group of 128 columns
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(h[i]));
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
                const GroupScale scale(top);
                uint32_t q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    q[i] = __nv_cvt_float2_to_fp8x2(make_float2(scale.of(h[2 * i]), scale.of(h[2 * i + 1])), __NV_SATFINITE,
                                                    __NV_E4M3);
                if (in) {
                    *reinterpret_cast<uint2*>(p.h + at) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
                    if ((lane & 15) == 0) p.h_scale[size_t(row) * (p.F / GROUP8) + 2 * s.blk + (lane >> 4)] = scale.scale;
                }
            } else if (in) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) split_pair(h[2 * i], h[2 * i + 1], hi[i], lo[i]);
                *reinterpret_cast<uint4*>(p.h + at * 2) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(p.h + (R * p.F + at) * 2) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
    }
}

// The counting warp: follows the CTA's units, counts each piece of h once it is
// stored, and hands a block whose last piece that was to the completing warps.
// The weights in flight make any round trip to L2 take several microseconds, so
// while the next piece is there already, a count's result is looked at only
// after the next count has been sent.
__device__ void count_pieces(const FfnParams& p, FfnSmem* sm, const Plan& pl, const Waiter& w) {
    const int lane = threadIdx.x & 31;
    const uint32_t all = 2 * pl.chunks[0];
    Turn in, out;
    Unit open;  // the unit whose count has been sent but not looked at
    uint32_t open_count = 0;
    bool is_open = false;
    auto hand = [&](const Unit& s) {
        if (!warp_await_mbar(&sm->job_out[out.i], out.phase ^ 1u, w, SITE_INFO_EMPTY)) return false;
        if (lane == 0) {
            __threadfence();  // the pieces that the other CTAs released
            sm->job[out.i] = s;
            sm->job_left[out.i] = FIN_WARPS;
            mbar_arrive(&sm->job_in[out.i]);
        }
        out.next(JOBS);
        return true;
    };
    while (true) {
        if (is_open) {
            const bool more = mbar_test(&sm->info_in[in.i], in.phase) && mbar_test(&sm->piece_in[in.i], in.phase);
            if (!__all_sync(0xffffffffu, more)) {
                is_open = false;
                if (__shfl_sync(0xffffffffu, open_count, 0) == all && !hand(open)) return;
            }
        }
        if (!warp_await_mbar(&sm->info_in[in.i], in.phase, w, SITE_INFO_FULL)) return;
        const Unit s = sm->unit[in.i];
        if (s.end) {
            hand(s);
            return;
        }
        // the slot is given back only after its piece, so that no second one comes in unseen
        if (!warp_await_mbar(&sm->piece_in[in.i], in.phase, w, SITE_INFO_FULL)) return;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->info_out[in.i]);
        in.next(INFO_SLOTS);
        uint32_t count = 0;
        if (s.half == 0 && lane == 0)  // releases the draining warps' stores, which the wait above has seen
            count = atom_add_release_u32(&p.ctl->arrived[uint32_t(s.a) * pl.blocks[0] + s.blk], 1u) + 1u;
        if (is_open && __shfl_sync(0xffffffffu, open_count, 0) == all && !hand(open)) return;
        is_open = s.half == 0;
        open = s;
        open_count = count;
    }
}

// A completing warp: its share of the rows of each block handed on.
template <bool FP8>
__device__ void complete_h(const FfnParams& p, FfnSmem* sm, const Plan& pl, const Waiter& w) {
    const int lane = threadIdx.x & 31, me = threadIdx.x / 32 - WARP_FIN;
    Turn in;
    int turn = 0;
    while (true) {
        if (!warp_await_mbar(&sm->job_in[in.i], in.phase, w, SITE_INFO_FULL)) return;
        const Unit s = sm->job[in.i];
        if (s.end) return;
        if (me == 0 && lane == 0) p.ctl->arrived[uint32_t(s.a) * pl.blocks[0] + s.blk] = 0u;  // for the next call
        // the warps take turns at the first rows: many blocks have few
        const int me_now = (me + turn++) % FIN_WARPS;
        // about as many loads in flight either way
        const int rows = pl.chunks[0] == 1 ? 4 : pl.chunks[0] == 2 ? 2 : 1;
        if (rows == 4)
            for (int i = me_now * 4; i < s.n; i += FIN_WARPS * 4) complete_rows<FP8, 4, 1>(p, pl, s, i);
        else if (rows == 2)
            for (int i = me_now * 2; i < s.n; i += FIN_WARPS * 2) complete_rows<FP8, 2, 2>(p, pl, s, i);
        else
            for (int i = me_now; i < s.n; i += FIN_WARPS) complete_rows<FP8, 1, 4>(p, pl, s, i);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            // The warp that had all the rows publishes, or the last of them, which has
            // then seen the other warps' rows: fences around the count, and the release
            // below covers what this thread has seen.
            bool publish = me_now == 0;
            if (s.n > rows) {
                __threadfence_block();
                publish = atomicSub(&sm->job_left[in.i], 1u) == 1u;
                __threadfence_block();
            }
            if (publish) atom_add_acq_rel_u32(&p.ctl->ready[s.a], 1u);  // releases the rows
            mbar_arrive(&sm->job_out[in.i]);
        }
        in.next(JOBS);
    }
}

// 8 bits: `steps` steps of one matrix, each with its own scales, summed in
// registers: up to B blocks of 16 rows for this warp (set, set + 2, ...).
template <int B, typename Put>
__device__ __forceinline__ bool drain_steps8(FfnSmem* sm, const Accs& rg, const Waiter& w, uint32_t tq, uint32_t steps,
                                             int set, int nblk, Turn& buf, Turn& sc, bool ok, const Put& put) {
    const int lane = threadIdx.x & 31;
    const float* scales = reinterpret_cast<const float*>(ffn_ring() + SCALE_AT);
    float acc0[B][16], acc1[B][16];
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc0[b][i] = acc1[b][i] = 0.f;
#pragma unroll 1
    for (uint32_t k = 0; k < steps; ++k) {
        if (ok) ok = warp_await_mbar(&sm->scales_in[sc.i], sc.phase, w, SITE_ACC_FULL);
        if (ok) ok = warp_await_mbar(&sm->acc_full[buf.i], buf.phase, w, SITE_ACC_FULL);
        if (ok) {
            tc_fence_after();
            const uint32_t t0 = tq + buf.i * 2u * rg.acc_stride;
            const float* scale = scales + sc.i * SCALE_FLOATS;
            const float c0 = scale[MAX_N], c1 = scale[MAX_N + 1];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int blk = set + 2 * b;
                if (blk < nblk) {
                    uint32_t r0[16], r1[16];
                    tmem_ld_32x32b_x16(t0 + blk * 16, r0);
                    tmem_ld_32x32b_x16(t0 + rg.acc_stride + blk * 16, r1);
                    float4 x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(scale + blk * 16 + 4 * i);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float v = (&x[i >> 2].x)[i & 3];
                        acc0[b][i] = fmaf(__uint_as_float(r0[i]), v * c0, acc0[b][i]);
                        acc1[b][i] = fmaf(__uint_as_float(r1[i]), v * c1, acc1[b][i]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm->acc_empty[buf.i]);
                mbar_arrive(&sm->scales_out[sc.i]);
            }
        }
        buf.next(rg.bufs);
        sc.next(SCALE_SLOTS);
    }
    if (ok) {
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (set + 2 * b < nblk) put(set + 2 * b, acc0[b], acc1[b]);
    }
    return ok;
}

template <bool FP8>
__device__ void drain_accumulators(const FfnParams& p, FfnSmem* sm, const Accs& rg, const Plan& pl, const Waiter& w) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp & 3, set = (warp - WARP_EPI) >> 2;
    const uint32_t tq = sm->tmem_base + (uint32_t(quad * 32) << 16);
    Turn buf, sc, in, done;
    bool ok = true;
    Unit s;
    while (ok && next_unit(sm, in, w, s, ok)) {
        const int n = s.n, nblk = pad16(n) / 16;
        // where the sums go: row i, this lane's columns f (first accumulator) and 128 + f
        const size_t stride = size_t(pl.blocks[s.half]) * ACC_COLS;
        float* to = piece_row(p, pl, s.half, s.second * pl.chunks[0] + s.c, s.off) + s.blk * ACC_COLS + quad * 32 + lane;
        auto put = [&](int blk, const float (&v0)[16], const float (&v1)[16]) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = blk * 16 + i;
                if (r < n) {
                    __stcg(to + size_t(r) * stride, v0[i]);
                    __stcg(to + size_t(r) * stride + 128, v1[i]);
                }
            }
        };
        if constexpr (!FP8) {
            ok = warp_await_mbar(&sm->acc_full[buf.i], buf.phase, w, SITE_ACC_FULL);
            if (ok) {
                tc_fence_after();
                const uint32_t t0 = tq + buf.i * 2u * rg.acc_stride;
#pragma unroll 1
                for (int blk = set; blk < nblk; blk += 2) {
                    uint32_t r0[16], r1[16];
                    float v0[16], v1[16];
                    tmem_ld_32x32b_x16(t0 + blk * 16, r0);
                    tmem_ld_32x32b_x16(t0 + rg.acc_stride + blk * 16, r1);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        v0[i] = __uint_as_float(r0[i]);
                        v1[i] = __uint_as_float(r1[i]);
                    }
                    if (s.half) {
                        // the products of h's remainders
                        tmem_ld_32x32b_x16(t0 + (nblk + blk) * 16, r0);
                        tmem_ld_32x32b_x16(t0 + rg.acc_stride + (nblk + blk) * 16, r1);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            v0[i] += __uint_as_float(r0[i]);
                            v1[i] += __uint_as_float(r1[i]);
                        }
                    }
                    put(blk, v0, v1);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->acc_empty[buf.i]);
            }
            buf.next(rg.bufs);
        } else {
            // as few registers as the rows need
            const uint32_t steps = s.k1 - s.k0;
            if ((nblk - set + 1) / 2 <= 1) ok = drain_steps8<1>(sm, rg, w, tq, steps, set, nblk, buf, sc, ok, put);
            else ok = drain_steps8<2>(sm, rg, w, tq, steps, set, nblk, buf, sc, ok, put);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->piece_in[done.i]);
        done.next(INFO_SLOTS);
    }
}

__device__ __forceinline__ void add4(float4& a, const float4& b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
}
__device__ __forceinline__ void fma4(float4& a, float g, const float4& b) {
    a.x = fmaf(g, b.x, a.x);
    a.y = fmaf(g, b.y, a.y);
    a.z = fmaf(g, b.z, a.z);
    a.w = fmaf(g, b.w, a.w);
}
__device__ __forceinline__ void store_out(const FfnParams& p, int t, int col, const float4& v) {
    const __nv_bfloat162 b0 = __floats2bfloat162_rn(v.x, v.y), b1 = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p.out + size_t(t) * p.H + col) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
}

// out[t] = sum over the k choices, in order, of gate * the row's pieces, in order.
__device__ void combine_rows(const FfnParams& p, const FfnSmem* sm, const Plan& pl) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int chunks = int(pl.chunks[1]), all = p.k * chunks;  // pieces of a token, choice by choice
    // piece i of token t at column col, and its gate
    auto load = [&](int t, int i, int col, float& g) {
        const int j = i / chunks, c = i - j * chunks, row = sm->row_of[t * p.k + j];
        if (row == NO_ROW) return make_float4(0.f, 0.f, 0.f, 0.f);
        g = sm->gate[t * p.k + j];
        return __ldcg(reinterpret_cast<const float4*>(piece_row(p, pl, 1, uint32_t(c), row) + col));
    };
    const int nb128 = (p.H + 127) / 128;
    constexpr int TOGETHER = 8;  // loads in flight
    if (all <= TOGETHER || p.T * nb128 >= int(gridDim.x) * FFN_WARPS / 2) {
        // 128 columns of a token per warp
        for (int item = blockIdx.x * FFN_WARPS + (tid >> 5); item < p.T * nb128; item += gridDim.x * FFN_WARPS) {
            const int t = item / nb128, col = (item - t * nb128) * 128 + lane * 4;
            if (col >= p.H) continue;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i = 0; i < all; i += TOGETHER) {
                float4 u[TOGETHER];
                float g[TOGETHER];
#pragma unroll
                for (int x = 0; x < TOGETHER; ++x) {
                    u[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                    g[x] = 0.f;
                    if (i + x < all) u[x] = load(t, i + x, col, g[x]);
                }
#pragma unroll
                for (int x = 0; x < TOGETHER; ++x)
                    if (i + x < all) fma4(acc, g[x], u[x]);
            }
            store_out(p, t, col, acc);
        }
        return;
    }
    // few rows in many pieces: 64 columns of a token per CTA, the pieces over
    // its threads, summed in shared memory
    constexpr int COLS = 16, SHARE = FFN_THREADS / COLS;  // float4 columns, threads per column
    float4* red = reinterpret_cast<float4*>(ffn_ring());
    const int c4 = tid % COLS, who = tid / COLS;
    const int nb = p.H / 64, each = (all + SHARE - 1) / SHARE;
    for (int item = blockIdx.x; item < p.T * nb; item += gridDim.x) {
        const int t = item / nb, col = (item - t * nb) * 64 + c4 * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const int i1 = min(all, (who + 1) * each);
        constexpr int BATCH = 4;
        for (int i = who * each; i < i1; i += BATCH) {
            float4 u[BATCH];
            float g[BATCH];
#pragma unroll
            for (int x = 0; x < BATCH; ++x) {
                u[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                g[x] = 0.f;
                if (i + x < i1) u[x] = load(t, i + x, col, g[x]);
            }
#pragma unroll
            for (int x = 0; x < BATCH; ++x)
                if (i + x < i1) fma4(acc, g[x], u[x]);
        }
        red[tid] = acc;
        __syncthreads();
        if (who == 0) {
            for (int x = 1; x < SHARE; ++x) add4(acc, red[x * COLS + c4]);
            store_out(p, t, col, acc);
        }
        __syncthreads();
    }
}

template <bool FP8>
__global__ void __launch_bounds__(FFN_THREADS, 1)
    mk_moe_ffn_decode_kernel(const FfnParams p, const __grid_constant__ FfnMaps m) {
    uint8_t* ring = ffn_ring();
    FfnSmem* sm = reinterpret_cast<FfnSmem*>(ring + RING_BYTES);
    const int tid = threadIdx.x, warp = tid >> 5;
    const Waiter w{p.err, &p.ctl->abort, FFN_SPIN_NS};
    // waits inside the pipeline and for the other CTAs' ends stall because something
    // upstream does: they get longer, so that the one that is recorded is the one at the root
    const Waiter wp{p.err, &p.ctl->abort, 2 * FFN_SPIN_NS};

    if (tid == 0) {
        for (int i = 0; i < STAGES_F; ++i) {
            mbar_init(&sm->weights_in[i], 1);
            mbar_init(&sm->rows_in[i], 1);
            mbar_init(&sm->empty[i], 1);
        }
        for (int i = 0; i < FFN_MAX_BUFS; ++i) {
            mbar_init(&sm->acc_full[i], 1);
            mbar_init(&sm->acc_empty[i], EPI_WARPS);
        }
        for (int i = 0; i < SCALE_SLOTS; ++i) {
            mbar_init(&sm->scales_in[i], 32);
            mbar_init(&sm->scales_out[i], EPI_WARPS);
        }
        for (int i = 0; i < INFO_SLOTS; ++i) {
            mbar_init(&sm->info_in[i], 1);
            mbar_init(&sm->info_out[i], 3 + EPI_WARPS);  // row loads, products, draining, counting
            mbar_init(&sm->piece_in[i], EPI_WARPS);
        }
        mbar_init(&sm->drain, 1);
        for (int i = 0; i < JOBS; ++i) {
            mbar_init(&sm->job_in[i], 1);
            mbar_init(&sm->job_out[i], FIN_WARPS);
        }
        fence_barrier_init();
        sm->ok = 1;
        tma_prefetch_desc(&m.w1);
        tma_prefetch_desc(&m.w3);
        tma_prefetch_desc(&m.x);
        tma_prefetch_desc(&m.w2);
        tma_prefetch_desc(&m.h);
    }
    if (warp == WARP_MMA) {
        tmem_alloc(&sm->tmem_base, 512);
        tmem_relinquish();
    }

    // ---- routing: a warp per token, in every CTA for itself, or shared out
    // over the CTAs and read back after a barrier once there are more tokens
    // than a CTA has warps (a second token per warp would cost about what the
    // barrier does)
    uint8_t* ids = ring + RS_IDS;
    const int rows = p.T * p.k;
    if (p.T <= FFN_WARPS) {
        if (warp < p.T) route_token(p, warp, ids, sm->gate);
        __syncthreads();
    } else {
        for (int t = blockIdx.x + int(gridDim.x) * warp; t < p.T; t += int(gridDim.x) * FFN_WARPS)
            route_token(p, t, p.ids, p.gates);
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            atom_add_acq_rel_u32(&p.ctl->routed, 1u);
            sm->ok = await_geq(&p.ctl->routed, gridDim.x, w, SITE_BAR_ROUTED);
        }
        __syncthreads();
        for (int i = tid; i < rows; i += FFN_THREADS) {
            ids[i] = __ldcg(p.ids + i);
            sm->gate[i] = __ldcg(p.gates + i);
        }
        __syncthreads();
    }
    if (sm->ok) {
        build_rows(p, sm, ring);
        fence_proxy_async_shared();  // the scratch's generic accesses before TMA writes there
        tc_fence_before();
        __syncthreads();
        tc_fence_after();

        const Plan pl = make_plan(p, FP8 ? 128 : 64, uint32_t(sm->parts), uint32_t(sm->most));
        Accs rg;
        const int N = pad16(max(sm->most, 1));  // no rows at all: every logit is -inf
        rg.acc_stride = uint32_t(N * (FP8 ? 1 : 2));
        rg.bufs = min(uint32_t(FFN_MAX_BUFS), 512u / (2u * rg.acc_stride));

        if (warp == WARP_A) weight_loads<FP8>(p, m, sm, pl, wp);
        else if (warp == WARP_B) row_loads<FP8>(p, m, sm, pl, w);
        else if (warp == WARP_MMA) products<FP8>(sm, rg, wp);
        else if (warp == WARP_COUNT) count_pieces(p, sm, pl, wp);
        else if (warp >= WARP_FIN) complete_h<FP8>(p, sm, pl, wp);
        else drain_accumulators<FP8>(p, sm, rg, pl, wp);

        __syncthreads();
        if (tid == 0) {
            // releases what the whole CTA has stored
            atom_add_acq_rel_u32(&p.ctl->done, 1u);
            sm->ok = await_geq(&p.ctl->done, gridDim.x, wp, SITE_BAR_COMPUTED) && ld_relaxed_u32(w.abort) == 0u;
        }
        __syncthreads();
        if (sm->ok) combine_rows(p, sm, pl);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(sm->tmem_base, 512);
    }
    if (tid == 0 && atom_add_acq_rel_u32(&p.ctl->exited, 1u) == gridDim.x - 1) {
        // the last CTA out leaves the control block ready for the next call
        FfnCtl* c = p.ctl;
        c->routed = 0;
        c->done = 0;
        c->next = 0;
        for (int i = 0; i < MAX_PARTS; ++i) c->ready[i] = 0;
        if (c->abort != 0)
            for (int i = 0; i < MAX_TILES1; ++i) c->arrived[i] = 0;  // a call that gave up left some
        c->abort = 0;
        c->exited = 0;
        __threadfence();
    }
}

struct FfnLayout {
    size_t ctl, ids, gates, h, h_scale, piece[2], room[2], total;
};

FfnLayout ffn_layout(int T, int H, int F, int k, bool fp8) {
    const size_t R = size_t(T) * k;
    FfnLayout L{};
    size_t o = 0;
    L.ctl = o;      o = ws_align(o + sizeof(FfnCtl));
    L.ids = o;      o = ws_align(o + R);
    L.gates = o;    o = ws_align(o + R * 4);
    L.h = o;        o = ws_align(o + R * F * (fp8 ? 1 : 4));
    L.h_scale = o;  o = ws_align(o + (fp8 ? R * (F / GROUP8) * 4 : 0));
    for (int i = 0; i < 2; ++i) {
        const size_t cols = (size_t(i == 0 ? F : H) + ACC_COLS - 1) / ACC_COLS * ACC_COLS;
        L.room[i] = std::max(PIECE_FLOATS, R * cols * (i == 0 ? 2 : 1));  // one unit along K always fits
        L.piece[i] = o;
        o = ws_align(o + L.room[i] * 4);
    }
    L.total = o;
    return L;
}

mk_status_t ffn_sizes(int T, int H, int E, int k, int F, int weights) {
    if (T < 0 || E < 1 || k < 1 || k > E || k > MAX_K) return MK_ERR_INVALID_ARG;
    if (weights != MK_WEIGHT_BF16 && weights != MK_WEIGHT_E4M3) return MK_ERR_INVALID_ARG;
    if (E > MAX_E || T > FFN_MAX_T) return MK_ERR_UNSUPPORTED;
    const int unit = weights == MK_WEIGHT_E4M3 ? GROUP8 : 64;
    if (H < unit || F < unit || H % unit != 0 || F % unit != 0) return MK_ERR_INVALID_ARG;
    if (H > 32768 || F > 32768) return MK_ERR_UNSUPPORTED;
    return MK_OK;
}

template <bool FP8>
cudaError_t launch_ffn(const FfnParams& p, const FfnMaps& m, int grid, cudaStream_t st) {
    // the CTAs wait for one another: a cooperative launch has all of them resident
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(FFN_THREADS);
    cfg.dynamicSmemBytes = FFN_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mk_moe_ffn_decode_kernel<FP8>, p, m);
}

}  // namespace

cudaError_t ffn_kernel_attributes() {
    const cudaError_t e =
        cudaFuncSetAttribute(mk_moe_ffn_decode_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, FFN_SMEM);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(mk_moe_ffn_decode_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, FFN_SMEM);
}

}  // namespace mk

using namespace mk;

extern "C" size_t mk_moe_ffn_decode_workspace_size(int T, int H, int F, int E, int k, int weights) {
    if (ffn_sizes(T, H, E, k, F, weights) != MK_OK) return 0;
    return ffn_layout(T, H, F, k, weights == MK_WEIGHT_E4M3).total;
}

extern "C" mk_status_t mk_moe_ffn_decode(const void* x, const float* x_scale, const float* logits, int T, int H, int E,
                                         int k, const void* W1, const void* W3, const void* W2, const float* W1_scale,
                                         const float* W3_scale, const float* W2_scale, int F, int weights, void* out,
                                         void* stream, void* workspace, size_t ws_bytes) {
    mk_status_t s = ffn_sizes(T, H, E, k, F, weights);
    if (s != MK_OK) return s;
    const bool fp8 = weights == MK_WEIGHT_E4M3;
    if (T > 0) {
        if (!x || !logits || !W1 || !W3 || !W2 || !out) return MK_ERR_INVALID_ARG;
        if (!host_aligned(x, 16) || !host_aligned(W1, 16) || !host_aligned(W3, 16) || !host_aligned(W2, 16) ||
            !host_aligned(out, 16) || !host_aligned(logits, 4))
            return MK_ERR_INVALID_ARG;
        const float* scales[4] = {x_scale, W1_scale, W3_scale, W2_scale};
        for (const float* v : scales)
            if ((v != nullptr) != fp8 || !host_aligned(v, 4)) return MK_ERR_INVALID_ARG;
    }
    int dev = 0, sms = 0;
    DevError* err = nullptr;
    if ((s = host_device(&dev, &sms, &err)) != MK_OK) return s;
    if (T == 0) return MK_OK;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const FfnLayout L = ffn_layout(T, H, F, k, fp8);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Workspace cached;  // held until the launch below
    if (ws) {
        if (ws_bytes < L.total || !host_aligned(ws, 256)) return MK_ERR_WORKSPACE;
    } else {
        if ((s = cached.get(WS_FFN, dev, st, L.total, L.total)) != MK_OK) return s;
        ws = cached.data();
    }
    FfnParams p{};
    p.logits = logits;
    p.x_scale = x_scale;
    p.w1_scale = W1_scale;
    p.w3_scale = W3_scale;
    p.w2_scale = W2_scale;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.ctl = reinterpret_cast<FfnCtl*>(ws + L.ctl);
    p.ids = ws + L.ids;
    p.gates = reinterpret_cast<float*>(ws + L.gates);
    p.h = ws + L.h;
    p.h_scale = reinterpret_cast<float*>(ws + L.h_scale);
    for (int i = 0; i < 2; ++i) {
        p.piece[i] = reinterpret_cast<float*>(ws + L.piece[i]);
        p.room[i] = L.room[i];
    }
    p.err = err;
    p.T = T;
    p.H = H;
    p.F = F;
    p.E = E;
    p.k = k;

    const CUtensorMapDataType type = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t size = fp8 ? 1 : 2;
    const uint32_t box = fp8 ? 128 : 64;  // one 128-byte swizzle span, and the rows of K of a step
    const uint64_t R = uint64_t(T) * k * (fp8 ? 1 : 2);
    FfnMaps m;
    std::memset(&m, 0, sizeof(m));
    if (host_encode_2d(&m.x, type, x, H, T, H * size, box, 1) != CUDA_SUCCESS ||
        host_encode_2d(&m.w1, type, W1, F, uint64_t(E) * H, F * size, box, box) != CUDA_SUCCESS ||
        host_encode_2d(&m.w3, type, W3, F, uint64_t(E) * H, F * size, box, box) != CUDA_SUCCESS ||
        host_encode_2d(&m.w2, type, W2, H, uint64_t(E) * F, H * size, box, box) != CUDA_SUCCESS ||
        host_encode_2d(&m.h, type, p.h, F, R, F * size, box, 1) != CUDA_SUCCESS)
        return MK_ERR_CUDA;
    const int grid = std::min(sms, FFN_MAX_CTAS);
    const cudaError_t e = fp8 ? launch_ffn<true>(p, m, grid, st) : launch_ffn<false>(p, m, grid, st);
    return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

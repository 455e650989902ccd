// kvattend.cu -- attention of one query token a sequence over the paged 8-bit
// cache.
//
// For a query row q and the n visible rows of its sequence,
//   s_l = scale * q . k_l,  out = sum_l exp(s_l - m) v_l / sum_l exp(s_l - m),
// in one pass with a running maximum m: when it grows, the sums so far are
// multiplied by exp(old m - new m).  With codes c and a scale a row,
//   s_l = (q . ck_l) (scale kscale_l),  weight of cv_l = exp(s_l - m) vscale_l,
// so codes are multiplied as they are and every scale is applied to a sum.
//
// Bound by memory: each visible row's 2 D code bytes and two scales are read
// once for a whole group of query heads, at 4 operations a byte and head.  On
// the tensor cores that leaves most of their rate unused; on the plain float
// units a group of 8 heads would need three times what they have.
//
// Products.  Both run as 16x8x16 matrix instructions with the rows of the
// cache as the wide operand: scores = K (16 tokens x D) times q^T (D x 8
// heads), and out^T = V^T (D x 16 tokens) times weights^T (16 tokens x 8
// heads), so a tile wastes nothing when a key head serves 8 query heads.
// (The fifth-generation instructions take 8-bit operands of one type on both
// sides, or 16-bit ones from shared or tensor memory: the codes would have to
// be widened into shared memory first, twice the traffic that bounds this.)
// Codes become 16-bit floats exactly, in registers: |code| <= 448 and at most 7
// significant bits.  The order of the D values within the scores' product is
// free, so a lane loads 16 consecutive bytes of a row and uses them as they
// come; the transposed use of V pairs the bytes of two tokens' words.
//
// Rounding.  q is divided by a power of two (its row's maximum becomes 2^7 to
// 2^8) and rounded to half precision: for a bfloat16 q that is exact down to 2^-32
// of the row's maximum; a float32 one takes two parts (22 bits; the result's
// error, 1.3e-7 at up to 2047 tokens of 64, is plain float32's, 1.2e-7).  Weights
// exp(s - m) vscale are split into three bfloat16 parts, float32's 24 bits and its
// range, as a channel's only nonzero codes may belong to tokens of tiny weight
// (two parts would be up to 9 % faster where instructions are the bound, 9 to 16
// query heads a key head or head_dim 64, and 1 to 3 % where memory is).  Sums are
// float32.  The matrix instructions drop what an addition shifts out instead of
// rounding it: about 2^-25 of the sum each time, always towards 0.  So a step's
// products start from 0, smallest parts first, and are added by ordinary rounded
// additions: in float32, the error against 64 bits of 35936 tokens went from
// 3.4e-6 to 4.7e-7 (plain float32 arithmetic gives 1.4e-6); in bfloat16, the loss
// was 2e-6 of the values over 128 pieces of one warp and 0.5 %, more than the
// result's rounding, after 27 thousand (2^31 tokens of head_dim 16); the additions
// cost 2 %, and 5 to 8 for rows of 256 values or 16 heads.  Two sums of bfloat16
// calls stay in the instructions, being short: a score's 4 to 16 steps, and a
// cluster's weighted sums, as its warps have at most 24 steps each.
//
// Split.  A row of work is one sequence, key head and block of 8 or 16 of its
// query heads; its tokens are cut into pieces of 32 (16 for the widest rows).
// All rows' pieces in one line are dealt out to a fixed number of warps, an
// equal run of consecutive pieces each, whatever the lengths: a warp walks its
// run across row ends with the next pieces' copies always in flight (a ring of
// stages in shared memory, 16-byte asynchronous copies: whole tiles where pages
// are made of them, else row by row), and leaves (m, sum, weighted sums) of each
// row it touched in the workspace.  A second kernel joins each row's, in order.
// Few and short rows take a second way: each row has a cluster of blocks, whose
// warps take equal shares of its pieces and join their parts in shared memory,
// a block's warps first, then the cluster's blocks; so one launch (cluster_of).
//
// Measured (bfloat16 q, 32 + 8 heads of 128): 4 sequences of 131071 tokens, e4m3,
// 172-175 us, 6.4 TB/s of cache; 64 uneven ones up to 8192 tokens, int8, 73 us
// (4.8 TB/s), of which the join is 5; without the arithmetic the copies alone
// take 56.  Cutting each sequence into chunks of one block instead took 200 and
// 100 us: a block's start and end cost about 4 us, and uneven lengths left SMs
// idle.  One sequence of 4099 tokens takes 11 us in clusters of 16 blocks: a warp
// alone on its scheduler needs 1.1 us for a piece, most of it one instruction
// waiting for the other, and has two or three.
//
#include <cuda_fp16.h>

#include "heads.cuh"
#include "launch.h"

namespace rdx {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * kWarpSize;
constexpr int kTile = 16;              // tokens of one matrix tile
constexpr int kScan = 1024;             // sequences whose lengths the join adds up itself, at most
constexpr int kRowUnits = 2;           // see units_of
constexpr int kFewest = 2;             // units of a warp's run, at least
constexpr float kSlack = 8.f;          // powers of two a score may exceed the reference by
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

struct AttendParams {
    KvCacheView cache;
    RowView q, out;
    const int32_t* table;
    const int32_t* lens;
    float* lse;
    // a warp's part of a row: slot = warp + row (both grow along the line of
    // pieces, one at a time, so every part has a slot of its own)
    float* sums;        // [slot][block_heads][head_dim]
    float2* stats;      // [slot][block_heads] (m in powers of two, sum)
    int64_t* firsts;    // [batch + 1] units of one row before each sequence
    int64_t slots;
    int64_t table_stride;
    int64_t table_pages;
    int64_t batch;
    int max_len;
    int q_heads;
    int group;          // query heads of a key head
    int head_blocks;    // blocks over a group
    int block_heads;    // query heads of one
    int rows;           // key heads * head_blocks: rows of a sequence
    int warps;          // runs
    int cluster;        // blocks for each row, which join its parts themselves; 0: the line and the join
    float scale;
    uint32_t page_magic;  // l / page_size = (umulhi(page_magic, l) + l) >> page_shift
    int page_shift;
    bool wide_q, wide_out;  // four values of a row at a time
};

__device__ __forceinline__ float nan_value() { return __uint_as_float(0x7fffffffu); }

// d += a (16x16) times b (16x8) into float32: half precision, or bfloat16.
__device__ __forceinline__ void matrix_step_half(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void matrix_step_bf16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// a += x and b += y in one instruction, each rounded.
__device__ __forceinline__ void add_two(float& a, float& b, float x, float y) {
    asm("{\n.reg .b64 s, t;\nmov.b64 s, {%0, %1};\nmov.b64 t, {%2, %3};\nadd.rn.f32x2 s, s, t;\nmov.b64 {%0, %1}, s;\n}"
        : "+f"(a), "+f"(b)
        : "f"(x), "f"(y));
}
// An 8x8 matrix of 16-bit values, a row's pair a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// Four codes of one word as two pairs in half precision, bytes 0 1 and 2 3.
template <int kFormat>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (kFormat == RDX_KV_INT8) {
        // the usual conversion by a fixed exponent: 0x64uu is the 16-bit float
        // 1024 + u, whose last bit is 1; u = code + 128
        const uint32_t u = w ^ 0x80808080u;
        const __half2 bias = __floats2half2_rn(1152.f, 1152.f);
        uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias), y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
        lo = *reinterpret_cast<const uint32_t*>(&x);
        hi = *reinterpret_cast<const uint32_t*>(&y);
    } else {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(uint16_t(w)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(uint16_t(w >> 16)));
    }
}

// Byte i of two words as a pair of bfloat16s, divided by kCodeUnit.
template <int kFormat>
constexpr float kCodeUnit = kFormat == RDX_KV_INT8 ? 128.f : 1.f;
template <int kFormat>
__device__ __forceinline__ uint32_t widen_pair(uint32_t w0, uint32_t w1, int i) {
    uint32_t r, z;
    if constexpr (kFormat == RDX_KV_INT8) {
        // u = code + 128 as the lowest bits of a bfloat16 is u 2^-133 (below
        // 0x80 a subnormal number, from there a normal one); times 2^126, less 1,
        // is code 2^-7
        z = __byte_perm(w0, w1, 0x4400 + 0x1111 * i);  // each byte twice
        const uint32_t x = (z ^ 0x00800080u) & 0x00ff00ffu;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0x7e807e80u), "r"(0xbf80bf80u));
    } else {
        // the exponent's 4 and the mantissa's 3 bits in a bfloat16's places are
        // the value times 2^-120 (subnormal codes too); NaN codes are never
        // stored.  Each code is the high byte of its half, and the byte between
        // them is the first code's sign: the shift brings both signs to their
        // halves' top bits.
        asm("prmt.b32 %0, %1, %2, %3;" : "=r"(z) : "r"(w0), "r"(w1), "r"(0x4800 + 0x1111 * i));
        const uint32_t x = uint32_t(int32_t(z) >> 4) & 0x87f087f0u;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x7b807b80u));
    }
    return r;
}

// Where 16-byte chunk c of row r of a 16-row tile lies.  Rows of 128 bytes and
// more all begin at the same bank; the exchange of chunks by row makes the
// eight lanes of a shared-memory phase meet eight different ones, both when
// they read two rows' first or second four chunks (scores) and when they read
// two chunks of every second row (weighted sums).
template <int kDim>
__device__ __forceinline__ int tile_offset(int r, int c) {
    if constexpr (kDim == 64) {
        const int line = r >> 1;
        return line * 128 + ((((r & 1) * 4 + c) ^ ((line & 3) << 1)) << 4);
    } else {
        const int s = (((r ^ (r >> 2)) & 1) << 2) | (r & 2);
        return r * kDim + ((c ^ s) << 4);
    }
}

// Four consecutive values: one load where rows allow it.
template <class T>
__device__ __forceinline__ void load_four(const RowView& v, const char* at, bool wide, float (&f)[4]) {
    if (wide) {
        typename Elems<T, 4>::R r;
        load_in(r, at, v.p, v.span);
        Elems<T, 4>::widen(r, f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            typename Elems<T, 1>::R r;
            float one[1];
            load_in(r, at + i * int(sizeof(T)), v.p, v.span);
            Elems<T, 1>::widen(r, one);
            f[i] = one[0];
        }
    }
}

// One warp's next tokens on their way: two tiles, or one of the widest rows.
template <int kDim>
struct Stage {
    static constexpr int kTiles = kDim == 256 ? 1 : 2;
    static constexpr int kTokens = kTiles * kTile;
    unsigned char k[kTiles][kTile * kDim];
    unsigned char v[kTiles][kTile * kDim];
    float scales[2][kTokens];
};
constexpr int kRing = 2;               // stages of a warp: one read, one on its way
constexpr int kCluster = 16;           // blocks of a row's cluster, at most

// 2^x to about 2 units in the last place; results below 2^-126 are 0.
__device__ __forceinline__ float power2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A sequence's visible tokens; 0 for a length outside [0, max_len], whose rows
// the join makes NaN.
__device__ __forceinline__ int length_of(const AttendParams& p, int64_t b) {
    const int len = guard(p.lens + b, 4, p.lens, size_t(p.batch) * 4) ? __ldg(p.lens + b) : 0;
    return len < 0 || len > p.max_len ? 0 : len;
}
template <int kTokens>
__device__ __forceinline__ int pieces_of(int len) {
    return len / kTokens + (len % kTokens != 0);
}
__device__ __forceinline__ void put_first(const AttendParams& p, int64_t b, int64_t first) {
    if (guard(p.firsts + b, 8, p.firsts, size_t(p.batch + 1) * 8)) p.firsts[b] = first;
}
// A row's length on the line: its pieces, and kRowUnits for what a warp does
// once a row (queries, sums out), so that runs over many short rows are no
// longer than others.
template <int kTokens>
__device__ __forceinline__ int units_of(int len) {
    return len == 0 ? 0 : kRowUnits + pieces_of<kTokens>(len);
}
// a / b of numbers >= 0, in 32 bits where they fit.
__device__ __forceinline__ int64_t over(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? int64_t(unsigned(a) / unsigned(b)) : a / b;
}
// Units of one warp's run.
__device__ __forceinline__ int64_t run_of(int64_t all, int warps) {
    const int64_t run = over(all + warps - 1, warps);
    return run < kFewest ? kFewest : run;
}
// A piece on the line.
struct Place {
    int64_t b;
    int row;      // key head and block of its query heads
    int key_head;
    int piece;    // of the row's `pieces`
    int pieces;
    int len;
    int64_t unit;  // where the piece lies on the line
};

// Four of a head's results from d on, rounded and stored.
template <class T>
__device__ __forceinline__ void put_four(const AttendParams& p, int64_t b, int head, int d, const float (&y)[4]) {
    char* const out = p.out.p + b * p.out.token_bytes + head * p.out.head_bytes;
    if (p.wide_out) {
        typename Elems<T, 4>::R r;
        Elems<T, 4>::narrow(y, r);
        store_in(r, out + d * int(sizeof(T)), p.out.p, p.out.span);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float one[1] = {y[i]};
            typename Elems<T, 1>::R r;
            Elems<T, 1>::narrow(one, r);
            store_in(r, out + (d + i) * int(sizeof(T)), p.out.p, p.out.span);
        }
    }
}
__device__ __forceinline__ void put_lse(const AttendParams& p, int64_t b, int head, float lse) {
    float* at = p.lse + b * p.q_heads + head;
    if (guard(at, 4, p.lse, size_t(p.batch) * p.q_heads * 4)) *at = lse;
}

// Shared memory of the cluster's blocks.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t of_block(const void* shared, int block) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(uint32_t(__cvta_generic_to_shared(shared))), "r"(block));
    return at;
}
__device__ __forceinline__ float2 load_two(uint32_t at) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float4 load_quad(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}

// Parts of a row, four of a head's values, joined in order.
struct Joined {
    float top = -INFINITY, sum = 0.f;
    float4 x = {0.f, 0.f, 0.f, 0.f};
    template <int kParts>
    __device__ __forceinline__ void add(const float2 (&st)[kParts], const float4 (&v)[kParts]) {
        float grown = top;
#pragma unroll
        for (int i = 0; i < kParts; ++i) grown = fmaxf(grown, st[i].x);
        const float down = grown == -INFINITY ? 1.f : exp2f(top - grown);
        top = grown;
        sum *= down, x.x *= down, x.y *= down, x.z *= down, x.w *= down;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const float f = top == -INFINITY ? 1.f : exp2f(st[i].x - top);
            sum += f * st[i].y;
            x.x += f * v[i].x, x.y += f * v[i].y, x.z += f * v[i].z, x.w += f * v[i].w;
        }
    }
};

// Blocks of an SM, as its shared memory and registers allow.  More blocks hide
// more of each other's latency, until the accumulators spill: 16 sequences of
// 16384 tokens on 8 key heads of 128 take, at 16 query heads a key head, 155 us
// with two blocks of 255 registers and 207 us with three of 168; in float32, at
// 4 query heads, 108 us and 115 us.
constexpr int blocks_per_sm(size_t type_bytes, int dim, int tiles) {
    return dim == 64 ? (tiles == 1 ? 4 : 3) : dim == 128 && type_bytes == 2 && tiles == 1 ? 3 : 2;
}

// T: the type of q and out; kDim: head_dim rounded up to 64, 128 or 256 (the
// rest is zeros); kTiles: tiles of 8 query heads; kClustered: a cluster of
// blocks for each row, not runs of the line.
template <class T, int kFormat, int kDim, int kTiles, bool kClustered>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(sizeof(T), kDim, kTiles))
    kv_attend_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kParts = sizeof(T) == 4 ? 2 : 1;   // of a query
    constexpr int kWeightParts = 3;
    constexpr bool kFreshScores = kParts == 2;       // a step's products added by rounded additions
    constexpr bool kFreshSums = kParts == 2 || !kClustered;
    constexpr int kSteps = kDim / 16;                // of the scores' product
    constexpr int kRowChunks = kDim / 16;
    constexpr int kOutTiles = kDim / 16;             // of 16 values of out^T
    using S = Stage<kDim>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t starts[kThreads];             // units before each thread's share of the sequences
    __shared__ int64_t warp_sums[kWarps];
    pdl_wait();
    pdl_release();
    const KvCacheView& cache = p.cache;
    const int warp = threadIdx.x / kWarpSize, lane = threadIdx.x % kWarpSize, gid = lane >> 2, tig = lane & 3;

    // chunks of a row past head_dim are never copied: zeros, once
    if (cache.head_dim < kDim)
        for (int i = threadIdx.x; i < int(kWarps * kRing * sizeof(S) / 16); i += kThreads)
            reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);

    // ---- this warp's pieces: places of the worker, and of the reader ahead of it
    const int index = blockIdx.x * kWarps + warp;
    Place at;
    int64_t last;
    if constexpr (kClustered) {                      // an equal share of one row
        __syncthreads();                             // the zeros
        const int row = blockIdx.x / p.cluster, share = index - row * p.cluster * kWarps, shares = p.cluster * kWarps;
        at.b = row / p.rows;
        at.row = row - int(at.b) * p.rows;
        at.key_head = at.row / p.head_blocks;
        at.len = length_of(p, at.b);
        at.pieces = pieces_of<S::kTokens>(at.len);
        at.piece = int(over(int64_t(at.pieces) * share, shares));
        at.unit = at.piece;
        last = over(int64_t(at.pieces) * (share + 1), shares);
    } else {
        // a run of the line of units
        const int share = int((p.batch + kThreads - 1) / kThreads);
        const int mine = int(min(int64_t(threadIdx.x) * share, p.batch)), mine_end = int(min(int64_t(mine) + share, p.batch));
        int64_t count = 0;
        for (int i = mine; i < mine_end; ++i) count += units_of<S::kTokens>(length_of(p, i));
        int64_t before = count;
#pragma unroll
        for (int off = 1; off < kWarpSize; off <<= 1) {
            const int64_t below = __shfl_up_sync(kFullMask, before, off);
            if (lane >= off) before += below;
        }
        if (lane == kWarpSize - 1) warp_sums[warp] = before;
        __syncthreads();
        int64_t all = 0;
        before -= count;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += warp_sums[w];
            all += warp_sums[w];
        }
        starts[threadIdx.x] = before;
        if (p.batch > kScan && threadIdx.x % gridDim.x == blockIdx.x) {  // for the join, each share by one block
            for (int i = mine; i < mine_end; ++i) {
                put_first(p, i, before);
                before += units_of<S::kTokens>(length_of(p, i));
            }
            if (mine < mine_end && mine_end == p.batch) put_first(p, p.batch, before);
        }
        __syncthreads();
        const int64_t run = run_of(all * p.rows, p.warps);
        const int64_t first = index * run;
        last = min(all * p.rows, first + run);
        if (first >= last) return;
        {
            int part = -1;
#pragma unroll
            for (int i = 0; i < kThreads / kWarpSize; ++i)
                part += __popc(__ballot_sync(kFullMask, starts[i * kWarpSize + lane] * p.rows <= first));
            int64_t from = starts[part];
            at.b = part * share;
            at.len = length_of(p, at.b);
            while ((from + units_of<S::kTokens>(at.len)) * p.rows <= first) {
                from += units_of<S::kTokens>(at.len);
                ++at.b;
                at.len = length_of(p, at.b);
            }
            const int64_t rest = first - from * p.rows;
            const int units = units_of<S::kTokens>(at.len);
            at.row = int(over(rest, units));
            at.key_head = at.row / p.head_blocks;
            const int unit = int(rest - int64_t(at.row) * units);
            at.piece = max(unit - kRowUnits, 0);
            at.pieces = units - kRowUnits;
            at.unit = first + max(kRowUnits - unit, 0);
        }
    }
    Place ahead = at;
    const auto step = [&](Place& x) {
        ++x.unit;
        if (++x.piece < x.pieces) return;
        x.piece = 0;
        x.unit += kRowUnits;
        x.row = x.row + 1 == p.rows ? 0 : x.row + 1;
        x.key_head = x.row / p.head_blocks;
        if (x.row > 0 || x.unit >= last) return;
        do {  // the line goes on, so some later sequence has tokens
            ++x.b;
            x.len = length_of(p, x.b);
        } while (x.len == 0);
        x.pieces = pieces_of<S::kTokens>(x.len);
    };

    S* const ring = reinterpret_cast<S*>(smem) + warp * kRing;
    const int token_lane = lane % S::kTokens;
    const bool whole_tiles = cache.page_size % kTile == 0;
    const int row_chunks = cache.head_dim / 16;
    const unsigned chunk_magic = 65536u / row_chunks + 1;  // x / row_chunks = x * this >> 16, for x < 512
    // where this lane's 16 bytes of a tile's runs of 512 go: the exchange of
    // chunks repeats every 8 rows
    constexpr int kPeriod = kDim / 64;
    int lane_offset[kPeriod];
#pragma unroll
    for (int n = 0; n < kPeriod; ++n) {
        const int x = n * kWarpSize + lane;
        lane_offset[n] = tile_offset<kDim>(x / kRowChunks, x % kRowChunks) - n * 512;
    }
    const auto page_index = [&](int l) -> int { return int((__umulhi(p.page_magic, uint32_t(l)) + uint32_t(l)) >> p.page_shift); };
    const auto page_of = [&](const Place& x) -> int {  // of this lane's token, -1 past the end
        const int l = x.piece * S::kTokens + token_lane;
        if (l >= x.len) return -1;
        const int32_t* entry = p.table + x.b * p.table_stride + page_index(l);
        return guard(entry, 4, p.table, (size_t(p.batch - 1) * p.table_stride + p.table_pages) * 4) ? __ldg(entry) : -2;
    };
    int page = page_of(ahead);
    const auto issue = [&](int slot) {
        if (ahead.unit < last) {
            S& st = ring[slot];
            const int l = ahead.piece * S::kTokens + token_lane;
            bool there = l < ahead.len;
            if (there && (page < 0 || page >= cache.pages)) there = false;
            const int row = there ? (page * cache.heads + ahead.key_head) * cache.page_size + (l - page_index(l) * cache.page_size) : -1;
            if (whole_tiles && cache.head_dim == kDim) {
                // 16 tokens of one page are one run of bytes; rows past the
                // sequence's end are copied as they are, or a tile of them not
                // at all: their scores are masked, and whatever their codes
                // are, they widen to numbers that their weights of 0 cancel
#pragma unroll
                for (int t = 0; t < S::kTiles; ++t) {
                    const int from = __shfl_sync(kFullMask, row, t * kTile);
                    if (from < 0) continue;
                    const int64_t off = int64_t(from) * kDim + 16 * lane;
                    if (!guard(cache.codes[0] + off, (kTile * kDim / 512 - 1) * 512 + 16, cache.codes[0],
                               size_t(cache.rows) * kDim)) continue;
#pragma unroll
                    for (int n = 0; n < kTile * kDim / 512; ++n) {
                        copy_async<16>(st.k[t] + lane_offset[n % kPeriod] + n * 512, cache.codes[0] + off + n * 512, true);
                        copy_async<16>(st.v[t] + lane_offset[n % kPeriod] + n * 512, cache.codes[1] + off + n * 512, true);
                    }
                }
            } else if (whole_tiles) {
#pragma unroll
                for (int t = 0; t < S::kTiles; ++t) {
                    const int from = __shfl_sync(kFullMask, row, t * kTile);
                    if (from < 0) continue;
                    const int64_t off = int64_t(from) * cache.head_dim;
                    for (int x = lane; x < kTile * row_chunks; x += kWarpSize) {
                        if (!guard(cache.codes[0] + off + 16 * x, 16, cache.codes[0], size_t(cache.rows) * cache.head_dim)) continue;
                        const int r = int(x * chunk_magic >> 16), at = tile_offset<kDim>(r, x - r * row_chunks);
                        copy_async<16>(st.k[t] + at, cache.codes[0] + off + 16 * x, true);
                        copy_async<16>(st.v[t] + at, cache.codes[1] + off + 16 * x, true);
                    }
                }
            } else {
#pragma unroll
                for (int t = 0; t < S::kTiles; ++t)
#pragma unroll
                    for (int n = 0; n < kTile * kRowChunks / kWarpSize; ++n) {
                        const int x = n * kWarpSize + lane, r = x / kRowChunks, c = x % kRowChunks;
                        const int from = __shfl_sync(kFullMask, row, t * kTile + r);
                        if (16 * c < cache.head_dim) {
                            const int64_t off = from < 0 ? 0 : int64_t(from) * cache.head_dim + 16 * c;
                            const bool take = from >= 0 && guard(cache.codes[0] + off, 16, cache.codes[0],
                                                                 size_t(cache.rows) * cache.head_dim);
                            copy_async<16>(st.k[t] + tile_offset<kDim>(r, c), cache.codes[0] + off, take);
                            copy_async<16>(st.v[t] + tile_offset<kDim>(r, c), cache.codes[1] + off, take);
                        }
                    }
            }
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                if (S::kTiles == 1 && lane / kTile != side) continue;
                float* const to = &st.scales[side][token_lane];
                if (l < ahead.len && !there)
                    *to = nan_value();               // a visible token on a page that the cache does not have
                else
                    copy_async<4>(to, reinterpret_cast<const char*>(cache.scales[side] + (row < 0 ? 0 : row)), row >= 0);
            }
            step(ahead);
            if (ahead.unit < last) page = page_of(ahead);
        }
        copies_commit();
    };
    issue(0);

    // ---- queries as the scores' second operand: this lane's values of head gid
    uint32_t q[kTiles][kParts][kSteps][2];
    float qscale[kTiles][2];                         // of heads 2 tig and 2 tig + 1
    const auto load_queries = [&](const Place& x) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const int in_group = x.row % p.head_blocks * p.block_heads + 8 * t + gid;
            const bool mine = 8 * t + gid < p.block_heads && in_group < p.group;
            const int head = x.key_head * p.group + (mine ? in_group : 0);
            const char* row = p.q.p + x.b * p.q.token_bytes + head * p.q.head_bytes;
            float f[kSteps][4], top = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int j = (tig + 4 * (s / 4)) * 16 + 4 * (s % 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[s][i] = 0.f;
                if (mine && j < cache.head_dim) load_four<T>(p.q, row + j * int(sizeof(T)), p.wide_q, f[s]);
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(f[s][i]));
            }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, off));
            // 2^e above the row's maximum (at least 2^-100); q 2^(8 - e) stays below 2^8
            int e = int(__float_as_uint(top) >> 23) - 126;
            e = min(max(e, -100), 127);
            const float down = __uint_as_float(uint32_t(127 + 8 - e) << 23);   // 2^(8 - e)
            const float up = __uint_as_float(uint32_t(127 + e - 8) << 23);
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float x = f[s][2 * i] * down, y = f[s][2 * i + 1] * down;
                    const uint32_t h = pack_half(x, y);
                    q[t][0][s][i] = h;
                    if constexpr (kParts == 2) {
                        const float2 g = unpack_half(h);
                        q[t][1][s][i] = pack_half(x - g.x, y - g.y);
                    }
                }
            const float mult = up * p.scale * kLog2e;
#pragma unroll
            for (int i = 0; i < 2; ++i) qscale[t][i] = __shfl_sync(kFullMask, mult, (2 * tig + i) * 4);
        }
    };

    float acc[kTiles][kOutTiles][4];
    float m[kTiles][2], total[kTiles][2];
    const auto clear = [&] {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            m[t][0] = m[t][1] = -INFINITY, total[t][0] = total[t][1] = 0.f;
#pragma unroll
            for (int o = 0; o < kOutTiles; ++o) acc[t][o][0] = acc[t][o][1] = acc[t][o][2] = acc[t][o][3] = 0.f;
        }
    };
    // the part of a row as it stands: head 0's place for the sums and the statistics
    const auto leave = [&](float* sums, float2* stats, bool shared) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int off = 4; off < kWarpSize; off <<= 1) total[t][h] += __shfl_xor_sync(kFullMask, total[t][h], off);
                const int head = 8 * t + 2 * tig + h;
                if (head >= p.block_heads) continue;
                const size_t parts = size_t(p.slots) * p.block_heads;
                // tile o's rows gid and gid + 8 are two neighbouring values; a run of tiles is a run of values
                constexpr int kRun = kDim == 64 ? 4 : 8;
#pragma unroll
                for (int o = 0; o < kOutTiles; o += 2) {
                    const int d = kDim == 64 ? gid * 8 + 2 * o : (gid + 8 * (o / kRun)) * 16 + 2 * (o % kRun);
                    float* const out = sums + head * cache.head_dim + d;
                    if (d < cache.head_dim && (shared || guard(out, 16, p.sums, parts * cache.head_dim * 4)))
                        *reinterpret_cast<float4*>(out) =
                            make_float4(acc[t][o][h], acc[t][o][2 + h], acc[t][o + 1][h], acc[t][o + 1][2 + h]);
                }
                if (gid == 0 && (shared || guard(stats + head, 8, p.stats, parts * 8)))
                    stats[head] = make_float2(m[t][h], total[t][h]);
            }
    };
    clear();
    int slot = 0;
#pragma unroll 1
    for (bool begins = true; at.unit < last;) {
        if (begins) {                                // this warp's part of a row
            load_queries(at);
            clear();
        }
        copies_wait<0>();
        __syncwarp();
        const S& st = ring[slot];
        slot ^= 1;
        issue(slot);                                 // in place of the piece before
        const int l0 = at.piece * S::kTokens;

        // scores: tokens gid and gid + 8 of each tile, heads 2 tig and 2 tig + 1
        float s[S::kTiles][kTiles][4] = {};
#pragma unroll
        for (int x = 0; x < S::kTiles; ++x) {
            float low[kTiles][4] = {};               // of q's second part
#pragma unroll
            for (int i = 0; i < kDim / 64; ++i) {
                float run[kTiles][4] = {};
                const uint4 lo = *reinterpret_cast<const uint4*>(st.k[x] + tile_offset<kDim>(gid, tig + 4 * i));
                const uint4 hi = *reinterpret_cast<const uint4*>(st.k[x] + tile_offset<kDim>(gid + 8, tig + 4 * i));
                const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t a[4];
                    widen4<kFormat>(wl[j], a[0], a[2]);
                    widen4<kFormat>(wh[j], a[1], a[3]);
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) {
                        if constexpr (kFreshScores) {
                            matrix_step_half(run[t], a, q[t][0][4 * i + j]);
                            if constexpr (kParts == 2) matrix_step_half(low[t], a, q[t][1][4 * i + j]);
                        } else {
                            matrix_step_half(s[x][t], a, q[t][0][4 * i + j]);
                        }
                    }
                }
                if constexpr (kFreshScores)
#pragma unroll
                    for (int t = 0; t < kTiles; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[x][t][e] += run[t][e];
            }
            if constexpr (kParts == 2)
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[x][t][e] += low[t][e];
        }
#pragma unroll
        for (int x = 0; x < S::kTiles; ++x)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float ks = st.scales[0][x * kTile + gid + 8 * i];
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) s[x][t][2 * i + h] *= qscale[t][h] * ks;
            }
        if (at.len - l0 < S::kTokens) {              // the row's last piece
#pragma unroll
            for (int x = 0; x < S::kTiles; ++x)
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (l0 + x * kTile + gid + 8 * (i / 2) >= at.len) s[x][t][i] = -INFINITY;
        }

        // The weights' reference m only has to keep 2^(s - m) in range: it moves
        // when a score passes it by 2^kSlack, and then to the maximum so far.
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            float top[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[h] = fmaxf(s[0][t][h], s[0][t][2 + h]);
                if (S::kTiles == 2) top[h] = fmaxf(top[h], fmaxf(s[S::kTiles - 1][t][h], s[S::kTiles - 1][t][2 + h]));
            }
            if (__any_sync(kFullMask, top[0] > m[t][0] + kSlack || top[1] > m[t][1] + kSlack)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int off = 4; off < kWarpSize; off <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(kFullMask, top[h], off));
                    const float grown = fmaxf(m[t][h], top[h]);
                    const float down = grown == -INFINITY ? 1.f : power2(m[t][h] - grown);
                    m[t][h] = grown;
                    total[t][h] *= down;
#pragma unroll
                    for (int o = 0; o < kOutTiles; ++o) acc[t][o][h] *= down, acc[t][o][2 + h] *= down;
                }
            }
        }

#pragma unroll
        for (int x = 0; x < S::kTiles; ++x) {
            uint32_t w[kTiles][kWeightParts][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float vs = st.scales[1][x * kTile + gid + 8 * i] * kCodeUnit<kFormat>;
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    float y[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float e = power2(s[x][t][2 * i + h] - m[t][h]);
                        total[t][h] += e;
                        y[h] = e * vs;
                    }
#pragma unroll
                    for (int part = 0; part < kWeightParts; ++part) {
                        const uint32_t h = pack_bf16(y[0], y[1]);
                        y[0] -= __uint_as_float(h << 16);
                        y[1] -= __uint_as_float(h & 0xffff0000u);
                        w[t][part][i] = transpose8(h);
                    }
                }
            }
            // weighted sums: out^T rows (values) from tokens 2 tig, 2 tig + 1 and both + 8
#pragma unroll
            for (int u = 0; u < (kDim + 127) / 128; ++u) {
                constexpr int kWords = kDim == 64 ? 2 : 4;
                uint32_t v[4][kWords];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 2 * tig + (i & 1) + 8 * (i >> 1);
                    if constexpr (kDim == 64) {
                        const uint2 c = *reinterpret_cast<const uint2*>(st.v[x] + tile_offset<kDim>(r, gid >> 1) + 8 * (gid & 1));
                        v[i][0] = c.x, v[i][1] = c.y;
                    } else {
                        const uint4 c = *reinterpret_cast<const uint4*>(st.v[x] + tile_offset<kDim>(r, gid + 8 * u));
                        v[i][0] = c.x, v[i][1] = c.y, v[i][2] = c.z, v[i][3] = c.w;
                    }
                }
#pragma unroll
                for (int j = 0; j < kWords; ++j)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t a[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            a[i] = widen_pair<kFormat>(v[i & 2][j], v[(i & 2) + 1][j], 2 * half + (i & 1));
#pragma unroll
                        for (int t = 0; t < kTiles; ++t) {
                            float(&sum)[4] = acc[t][(u * kWords + j) * 2 + half];
                            if constexpr (kFreshSums) {
                                float fresh[4] = {};
#pragma unroll
                                for (int part = kWeightParts - 1; part >= 0; --part) matrix_step_bf16(fresh, a, w[t][part]);
                                add_two(sum[0], sum[1], fresh[0], fresh[1]);
                                add_two(sum[2], sum[3], fresh[2], fresh[3]);
                            } else {
#pragma unroll
                                for (int part = 0; part < kWeightParts; ++part) matrix_step_bf16(sum, a, w[t][part]);
                            }
                        }
                    }
            }
        }

        begins = at.piece + 1 == at.pieces;
        if (!kClustered && (begins || at.unit + 1 == last)) {  // the part's end
            const int64_t part = (index + at.b * p.rows + at.row) * p.block_heads;
            leave(p.sums + part * cache.head_dim, p.stats + part, false);
        }
        step(at);
    }
    copies_wait<0>();
    if (!kClustered) return;

    // ---- the row's parts joined, four values a thread: the block's warps, then the cluster's blocks
    constexpr int kPart = kTiles * 8 * (kDim + 2);   // words of a part: sums, then the statistics
    static_assert(kRing * sizeof(S) >= 2 * kPart * 4, "a warp's part and the block's fit one ring");
    const auto part_of = [&](int w) { return reinterpret_cast<float*>(reinterpret_cast<S*>(smem) + w * kRing); };
    const auto stats_of = [&](float* sums) { return reinterpret_cast<float2*>(sums + kTiles * 8 * kDim); };
    float* const joined = part_of(0) + kPart;
    __syncwarp();                                    // the ring is read no more
    leave(part_of(warp), stats_of(part_of(warp)), true);
    __syncthreads();
    const int fours = cache.head_dim / 4, all_fours = p.block_heads * fours;
    for (int o = threadIdx.x; o < all_fours; o += kThreads) {
        const int head = o / fours, d = 4 * (o - head * fours);
        float2 st[kWarps];
        float4 v[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            st[w] = stats_of(part_of(w))[head];
            v[w] = *reinterpret_cast<const float4*>(part_of(w) + head * cache.head_dim + d);
        }
        Joined y;
        y.add(st, v);
        *reinterpret_cast<float4*>(joined + head * cache.head_dim + d) = y.x;
        if (d == 0) stats_of(joined)[head] = make_float2(y.top, y.sum);
    }
    cluster_barrier();
    const int row = blockIdx.x / p.cluster, rank = blockIdx.x - row * p.cluster, b = row / p.rows;
    const int written = guard(p.lens + b, 4, p.lens, size_t(p.batch) * 4) ? __ldg(p.lens + b) : 0;
    const bool bad = written < 0 || written > p.max_len, none = written == 0;
    const int row_of_b = row - b * p.rows, in_group = row_of_b % p.head_blocks * p.block_heads;
    for (int o = rank * kThreads + threadIdx.x; o < all_fours; o += p.cluster * kThreads) {
        const int head = o / fours, d = 4 * (o - head * fours);
        if (in_group + head >= p.group) break;
        float2 st[kCluster];
        float4 v[kCluster];
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            st[c] = make_float2(-INFINITY, 0.f), v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < p.cluster) {
                st[c] = load_two(of_block(stats_of(joined) + head, c));
                v[c] = load_quad(of_block(joined + head * cache.head_dim + d, c));
            }
        }
        Joined y;
        y.add(st, v);
        const int to = row_of_b / p.head_blocks * p.group + in_group + head;
        float out[4] = {y.x.x / y.sum, y.x.y / y.sum, y.x.z / y.sum, y.x.w / y.sum};
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = bad ? nan_value() : none ? 0.f : out[i];
        put_four<T>(p, b, to, d, out);
        if (d == 0 && p.lse != nullptr)
            put_lse(p, b, to, bad ? nan_value() : none ? -INFINITY : (y.top + log2f(y.sum)) * kLn2);
    }
    cluster_barrier();                               // the other blocks have read this one's part
}

// The parts of one query head's row joined: kSplit warps for each head, each
// taking every kSplit-th part in order, eight at a time, its lanes four values
// each (eight where a row has more than 128); then the warps in order.  Where
// the row's parts lie follows from the lengths alone, which were there before
// the first kernel: for up to kScan sequences each warp adds them up while that
// kernel runs; else it reads what that kernel left.
template <int kSplit>
constexpr int kJoinWarps = kSplit < 8 ? 8 : kSplit;  // of a block
template <class T, int kTokens, int kSplit>
__global__ void __launch_bounds__(kJoinWarps<kSplit> * kWarpSize) kv_attend_join_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kBatch = 8;                        // parts read at once
    constexpr int kVecs = kTokens == kTile ? 2 : 1;  // of four values a lane
    __shared__ float4 shared_sums[kSplit > 1 ? kJoinWarps<kSplit> : 1][kVecs][kWarpSize];
    __shared__ float2 shared_stats[kJoinWarps<kSplit>];
    const int warp = threadIdx.x / kWarpSize, lane = threadIdx.x % kWarpSize, piece = warp % kSplit;
    const int64_t index = int64_t(blockIdx.x) * (kJoinWarps<kSplit> / kSplit) + warp / kSplit;  // batch * q_heads + head
    const bool on = index < p.batch * p.q_heads;
    const int64_t b = on ? over(index, p.q_heads) : 0;
    const int head = on ? int(index - b * p.q_heads) : 0;
    const int in_group = head % p.group, block = in_group / p.block_heads;
    const int row = head / p.group * p.head_blocks + block;
    const int written = guard(p.lens + b, 4, p.lens, size_t(p.batch) * 4) ? __ldg(p.lens + b) : 0;
    const bool bad = written < 0 || written > p.max_len;
    int64_t before = 0, all = 0;
    if (p.batch <= kScan) {
        for (int i = lane; i < p.batch; i += kWarpSize) {
            const int units = units_of<kTokens>(length_of(p, i));
            all += units;
            before += i < b ? units : 0;
        }
        before = group_sum(before, kWarpSize);
        all = group_sum(all, kWarpSize);
    }
    pdl_wait();
    pdl_release();
    if (p.batch > kScan) {
        const auto first_of = [&](int64_t i) -> int64_t {
            return guard(p.firsts + i, 8, p.firsts, size_t(p.batch + 1) * 8)
                       ? __ldcg(reinterpret_cast<const long long*>(p.firsts + i)) : 0;
        };
        before = first_of(b);
        all = first_of(p.batch);
    }
    const int pieces = pieces_of<kTokens>(bad ? 0 : written), units = units_of<kTokens>(bad ? 0 : written);
    const int64_t run = run_of(all * p.rows, p.warps);
    const int64_t from = before * p.rows + int64_t(row) * units + kRowUnits;
    const int first = int(over(from, run)), n = !on || pieces == 0 ? 0 : int(over(from + pieces - 1, run)) - first + 1;
    const int64_t part = (first + b * p.rows + row) * p.block_heads + in_group - block * p.block_heads;
    const size_t parts = size_t(p.slots) * p.block_heads;
    const int d_all = p.cache.head_dim;

    float top = -INFINITY, sum = 0.f;
    float4 x[kVecs] = {};
#pragma unroll 1
    for (int i0 = piece; i0 < n; i0 += kSplit * kBatch) {
        float2 st[kBatch];
        float4 v[kBatch][kVecs];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * kSplit;
            const int64_t at = part + int64_t(i) * p.block_heads;
            const bool there = i < n;
            st[j] = there && guard(p.stats + at, 8, p.stats, parts * 8) ? __ldcg(p.stats + at) : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int c = 0; c < kVecs; ++c) {
                const int d = 4 * (lane + c * kWarpSize);
                const float* from_d = p.sums + at * d_all + d;
                v[j][c] = there && d < d_all && guard(from_d, 16, p.sums, parts * d_all * 4)
                              ? __ldcg(reinterpret_cast<const float4*>(from_d)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        float grown = top;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) grown = fmaxf(grown, st[j].x);
        const float down = grown == -INFINITY ? 1.f : exp2f(top - grown);
        top = grown;
        sum *= down;
#pragma unroll
        for (int c = 0; c < kVecs; ++c) x[c].x *= down, x[c].y *= down, x[c].z *= down, x[c].w *= down;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const float f = top == -INFINITY ? 1.f : exp2f(st[j].x - top);
            sum += f * st[j].y;
#pragma unroll
            for (int c = 0; c < kVecs; ++c)
                x[c].x += f * v[j][c].x, x[c].y += f * v[j][c].y, x[c].z += f * v[j][c].z, x[c].w += f * v[j][c].w;
        }
    }
    if constexpr (kSplit > 1) {
#pragma unroll
        for (int c = 0; c < kVecs; ++c) shared_sums[warp][c][lane] = x[c];
        if (lane == 0) shared_stats[warp] = make_float2(top, sum);
        __syncthreads();
        if (piece != 0) return;
        float grown = top;
#pragma unroll
        for (int w = 1; w < kSplit; ++w) grown = fmaxf(grown, shared_stats[warp + w].x);
#pragma unroll
        for (int w = 0; w < kSplit; ++w) {
            const float2 st = shared_stats[warp + w];
            const float f = grown == -INFINITY ? 1.f : exp2f(st.x - grown);
            sum = (w == 0 ? 0.f : sum) + f * st.y;
#pragma unroll
            for (int c = 0; c < kVecs; ++c) {
                const float4 v = shared_sums[warp + w][c][lane];
                if (w == 0) x[c] = make_float4(0.f, 0.f, 0.f, 0.f);
                x[c].x += f * v.x, x[c].y += f * v.y, x[c].z += f * v.z, x[c].w += f * v.w;
            }
        }
        top = grown;
    }
    if (!on) return;
#pragma unroll
    for (int c = 0; c < kVecs; ++c) {
        const int d = 4 * (lane + c * kWarpSize);
        if (d >= d_all) continue;
        float y[4] = {x[c].x / sum, x[c].y / sum, x[c].z / sum, x[c].w / sum};
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = bad ? nan_value() : n == 0 ? 0.f : y[i];
        put_four<T>(p, b, head, d, y);
    }
    if (lane == 0 && p.lse != nullptr)
        put_lse(p, b, head, bad ? nan_value() : n == 0 ? -INFINITY : (top + log2f(sum)) * kLn2);
}

// ---- host ---------------------------------------------------------------------------------------------------------

struct Split {
    int tiles;        // of 8 query heads in a row of work
    int head_blocks;
    int block_heads;
    int rows;         // of a sequence
    int warps;
    int64_t slots;
};

// Rows of 8 query heads, or of 16 where a key head serves more than 8 and the
// accumulators fit.  Runs: one for every warp that a GB300's 152 SMs hold.
// Fixed, so that the order of the sums depends on the sizes and lengths alone.
Split split_of(const KvAttendPlan& p) {
    Split s;
    const int group = p.q_heads / p.cache.heads;
    s.tiles = group > 8 && p.cache.head_dim <= 128 ? 2 : 1;
    s.block_heads = group < 8 * s.tiles ? group : 8 * s.tiles;
    s.head_blocks = (group + s.block_heads - 1) / s.block_heads;
    s.rows = p.cache.heads * s.head_blocks;
    const int dim = p.cache.head_dim <= 64 ? 64 : p.cache.head_dim <= 128 ? 128 : 256;
    s.warps = kWarps * 152 * blocks_per_sm(p.type == RDX_TYPE_BF16 ? 2 : 4, dim, s.tiles);
    s.slots = s.warps + p.batch * s.rows;
    return s;
}

// Where each array starts in the workspace (firsts at 0), and its size.
struct Layout {
    size_t sums, stats, bytes;
};
Layout layout_of(const KvAttendPlan& p, const Split& s) {
    const auto up = [](size_t n) { return (n + 15) / 16 * 16; };
    Layout l;
    l.sums = up(size_t(p.batch + 1) * 8);
    l.stats = l.sums + size_t(s.slots) * s.block_heads * size_t(p.cache.head_dim) * 4;
    l.bytes = up(l.stats + size_t(s.slots) * s.block_heads * 8);
    return l;
}

// Blocks of a row's cluster, 0 for the line.  Where every row can have a cluster
// at once and a warp's share stays short, one kernel is faster than two: of 32
// query heads on 8 key heads of 128, one sequence of 512 tokens takes 7.4 us
// against 10.2, one of 4096 10.3 against 12.0, 16 of 500 11.6 against 13.8 (and
// on the host 6 us against 9).  From there on the line's even shares and full
// SMs count for as much or more: 8 sequences of 2000 tokens (four pieces a warp)
// 16.2 either way, 16 uneven ones up to 1000 (four) 13.4 against 12.2; with 12
// heads of 64, 16 up to 1000 (four) 11.8 against 10.0, up to 500 (two) 7.9
// against 9.0; with 4 key heads of 256, 32 of 1000 (eight pieces of 16) 22.6
// against 23.7.  Up to a piece a warp more blocks make a row faster (8 sequences
// of 500: one block a row 11.1 us, two 9.4, four 9.4), then no more; nor beyond
// four results a thread when they are joined (16 query heads a key head, 8
// sequences of 64 tokens: one block 13.2, four 11.8).
template <int kDim>
int cluster_of(const AttendParams& a) {
    constexpr int64_t kTokens = Stage<kDim>::kTokens, kMost = kDim == 64 ? 2 : kDim == 128 ? 3 : 8;  // pieces a warp
    const int64_t pieces = (int64_t(a.max_len) + kTokens - 1) / kTokens;
    const int64_t rows = a.batch * a.rows, places = a.warps / kWarps;
    int blocks = 1;
    const auto more = [&] { return pieces > blocks * kWarps || a.block_heads * a.cache.head_dim > 4 * blocks * kThreads; };
    while (blocks < kCluster && more() && 2 * blocks * rows <= places) blocks *= 2;
    return blocks * rows <= places && pieces <= blocks * kWarps * kMost ? blocks : 0;
}

template <class T, int kTokens, int kSplit>
cudaError_t join(const AttendParams& a, cudaStream_t stream) {
    constexpr int64_t kHeads = kJoinWarps<kSplit> / kSplit;  // of a block
    return launch_pdl(kv_attend_join_kernel<T, kTokens, kSplit>, dim3(unsigned((a.batch * a.q_heads + kHeads - 1) / kHeads)),
                      dim3(kJoinWarps<kSplit> * kWarpSize), stream, a);
}

template <class T, int kFormat, int kDim, int kTiles, bool kClustered>
cudaError_t start(bool early, unsigned blocks, const AttendParams& a, cudaStream_t stream) {
    const auto kernel = kv_attend_kernel<T, kFormat, kDim, kTiles, kClustered>;
    constexpr size_t kSmem = kWarps * kRing * sizeof(Stage<kDim>);
    static SharedMemoryGrant grant;
    const cudaError_t e = grant.ask(kernel, kSmem, kClustered);
    return e != cudaSuccess ? e : launch_smem(early, kernel, dim3(blocks), dim3(kThreads), kSmem, stream,
                                              kClustered ? unsigned(a.cluster) : 1u, a);
}

template <class T, int kFormat, int kDim, int kTiles>
cudaError_t launch(AttendParams a, cudaStream_t stream) {
    constexpr int kTokens = Stage<kDim>::kTokens;
    a.cluster = cluster_of<kDim>(a);
    if (a.cluster > 0) {
        const unsigned blocks = unsigned(a.batch * a.rows * a.cluster);
        return start<T, kFormat, kDim, kTiles, true>(blocks < unsigned(a.warps / kWarps), blocks, a, stream);
    }
    // no more blocks than the longest lengths could use
    const __int128 most = __int128(a.batch) * a.rows * (kRowUnits + (int64_t(a.max_len) + kTokens - 1) / kTokens);
    const __int128 blocks = (most + kFewest * kWarps - 1) / (kFewest * kWarps);
    const unsigned grid = blocks < 1 ? 1 : blocks < a.warps / kWarps ? unsigned(blocks) : unsigned(a.warps / kWarps);
    // A grid that needs all of every SM's shared memory starts on empty SMs: one
    // that still runs another kernel's last blocks keeps that kernel's division
    // of its memory, and with it room for fewer of these (64 uneven sequences up
    // to 8192 tokens, one call after the other: 93 us instead of 75).
    const bool early = grid < unsigned(a.warps / kWarps);
    const cudaError_t e = start<T, kFormat, kDim, kTiles, false>(early, grid, a, stream);
    if (e != cudaSuccess) return e;
    // The fewer heads there are, the more parts each has: 16 warps for each of up
    // to one head an SM (6 heads on one sequence of 16384 tokens: 15.0 us for the
    // call, 16.7 with 8 warps), 4 for a few a SM (512 heads of 64 uneven
    // sequences: 69.1 us; with 16, 77.7), else 2 (2048 heads: 72.5; with 4, 75.5).
    const int64_t heads = a.batch * a.q_heads;
    return heads <= 152 ? join<T, kTokens, 16>(a, stream)
                        : heads <= 1024 ? join<T, kTokens, 4>(a, stream) : join<T, kTokens, 2>(a, stream);
}

template <class T, int kFormat>
cudaError_t launch(const AttendParams& a, int tiles, cudaStream_t stream) {
    if (a.cache.head_dim <= 64) return tiles == 2 ? launch<T, kFormat, 64, 2>(a, stream) : launch<T, kFormat, 64, 1>(a, stream);
    if (a.cache.head_dim <= 128)
        return tiles == 2 ? launch<T, kFormat, 128, 2>(a, stream) : launch<T, kFormat, 128, 1>(a, stream);
    return launch<T, kFormat, 256, 1>(a, stream);
}

}  // namespace

RDX_DEFINE_VIOLATION_COUNTER(kv_attend_out_of_range)

size_t kv_attend_workspace_bytes(const KvAttendPlan& plan) {
    return plan.batch == 0 ? 0 : layout_of(plan, split_of(plan)).bytes;
}

cudaError_t kv_attend_launch(const KvAttendPlan& plan, cudaStream_t stream) {
    const Split s = split_of(plan);
    const Layout l = layout_of(plan, s);
    AttendParams a = {};
    a.cache = plan.cache;
    for (int i = 0; i < 2 && plan.cache.rows == 0; ++i) {  // never read, but an address for copies of no bytes
        a.cache.codes[i] = plan.workspace;
        a.cache.scales[i] = reinterpret_cast<float*>(plan.workspace);
    }
    a.q = plan.q;
    a.out = plan.out;
    a.table = plan.table;
    a.lens = plan.lens;
    a.lse = plan.lse;
    a.firsts = reinterpret_cast<int64_t*>(plan.workspace);
    a.sums = reinterpret_cast<float*>(plan.workspace + l.sums);
    a.stats = reinterpret_cast<float2*>(plan.workspace + l.stats);
    a.slots = s.slots;
    a.table_stride = plan.batch > 1 ? plan.table_stride : 0;
    a.table_pages = plan.table_pages;
    a.batch = plan.batch;
    a.max_len = int(plan.max_len);
    a.q_heads = plan.q_heads;
    a.group = plan.q_heads / plan.cache.heads;
    a.head_blocks = s.head_blocks;
    a.block_heads = s.block_heads;
    a.rows = s.rows;
    a.warps = s.warps;
    a.scale = plan.scale;
    const int four = plan.type == RDX_TYPE_BF16 ? 8 : 16;
    const auto wide = [four](const RowView& v) {
        return reinterpret_cast<uintptr_t>(v.p) % four == 0 && v.token_bytes % four == 0 && v.head_bytes % four == 0;
    };
    a.wide_q = wide(plan.q);
    a.wide_out = wide(plan.out);
    // Division by an invariant d (Granlund and Montgomery, 1994), for l < 2^31:
    // shift s = ceil(log2 d), magic = floor(2^32 (2^s - d) / d) + 1
    while (int64_t(1) << a.page_shift < plan.cache.page_size) ++a.page_shift;
    a.page_magic = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << a.page_shift) - plan.cache.page_size)) / plan.cache.page_size + 1);
    if (plan.type == RDX_TYPE_BF16)
        return plan.cache.format == RDX_KV_INT8 ? launch<Bf16, RDX_KV_INT8>(a, s.tiles, stream)
                                                : launch<Bf16, RDX_KV_E4M3>(a, s.tiles, stream);
    return plan.cache.format == RDX_KV_INT8 ? launch<float, RDX_KV_INT8>(a, s.tiles, stream)
                                            : launch<float, RDX_KV_E4M3>(a, s.tiles, stream);
}

}  // namespace rdx

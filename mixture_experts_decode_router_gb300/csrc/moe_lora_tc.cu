// moe_lora_tc.cu -- low-rank adapters of many rows on the tensor cores (sm_103a): the rows sorted by
// adapter, in tiles of up to 128 rows of one adapter (moe_lora.cu).
//
// Bound by HBM: x once, base and out once; the adapters' matrices come from L2, and the products
// are 4 n r (in + out) / 2 operations, a tenth of the tensor cores' rate at rank 64.
//
// v = A x (lora_shrink_kernel): a block takes a tile of rows and a stretch of K.  Rows of x are
// gathered where they lie by TMA (four rows an instruction, 64 elements of each), beside the adapter's
// rows; M = 128 rows, N = the rank; the fp32 sums in tensor memory are written as that stretch's part.
// (Of ranks above 16 the parts are then added by lora_sum_kernel.)
//
// out = base + B v (lora_expand_kernel): a block takes a tile of rows and a stretch of the outputs,
// 128 at a time.  v, summed over the stretches in their order, scaled and split into 16-bit parts
// (moe_lora.cu), stays in shared memory as the products' M = 128 rows; B's rows come by TMA.  Eight
// warps add the base to what they read of tensor memory.  They read it by fragments, of which a lane
// has column pairs 8 apart; B's rows are put into shared memory so that these are pieces of 16 bytes
// of neighbouring outputs, four lanes' side by side.  base comes by asynchronous copies, a tile ahead,
// to where the lane that wants it reads it, and out is written from the registers (8192 rows of 7168
// outputs, rank 64: 43 us, 5.4 TB/s, and the sums of v before it 26 and 5).  Of the other forms, when this
// one took 49 us: base loaded into registers a tile ahead 74, since waits for anything else waited for
// those loads too; results through shared memory, 128 bytes along a row, 61, bound by its traffic and
// steps.  Rows that are not of whole aligned pieces go through shared memory: their aligned 16 bytes, and
// single elements at the ends (6000 rows of 3551 outputs: 49 us; all by single elements 102).
#include <mutex>
#include <type_traits>

#include "moe_launch.cuh"
#include "moe_lora.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr int kM = kLoraTile;
constexpr int kBox = 64;                       // elements along a reduction: 128 bytes
constexpr int kBoxBytes = kM * kBox * 2;       // of 128 rows

struct TcArgs {
    LoraParams p;
    int N;            // rank, a multiple of 16
    int max_splits;   // of K: as many as part holds
    int stages;       // shrink: ring
    int tmem_cols;    // shrink
    int expand_blocks;
    bool summed;      // v's parts have been added into the first
    float* part;      // [splits][n][r]
};

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// Rows y of a [rows, K] map (box 64 x 1), 64 elements from x on, four times 128 bytes.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, int32_t x, int4 y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(ptx::smem_u32(bar))
        : "memory");
}

// 64 columns of 16 lanes of tensor memory by fragments: of lane (g, t) = (lane / 4, lane % 4), values
// 4 j .. 4 j + 3 are columns 8 j + 2 t and the next of row g, and of row g + 8.
__device__ __forceinline__ void tmem_ld_fragments(uint32_t taddr, float (&v)[32]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
        "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
          "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// 16 bytes from global to shared memory, asynchronously.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A box of a 3-D map.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(ptx::smem_u32(bar))
        : "memory");
}

// A wait of the whole warp that tries for some microseconds before it begins to count the time (the
// timer's first reading alone takes a microsecond, which every wait of a ring would pay).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* err, int32_t code) {
    for (int i = 0; i < 256; ++i)
        if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    return ptx::mbar_wait_warp(bar, parity, abort, err, code);
}

// Into how many pieces of `size` (boxes of K, tiles of outputs) each of `runs` tiles is cut, at most
// `most`: that for which the blocks' rounds are over soonest, where a piece costs 2% of a tile more
// than its part.  (Both kernels form the same from ctrl->n_active.)
struct Pieces {
    int n, size;
};
__device__ __forceinline__ Pieces pieces(int runs, int size, int most, int blocks) {
    // Lane i weighs i + 1 and i + 33 pieces; the costs, in whole warps' agreement, by their upper bits.
    const int lane = threadIdx.x & 31;
    uint32_t key = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = lane + 1 + 32 * i;
        if (c <= min(most, size)) {
            const int per = (size + c - 1) / c;
            const float cost = (float)((runs * c + blocks - 1) / blocks) * ((float)per / size + 0.02f);
            key = min(key, (__float_as_uint(cost) & ~63u) | (uint32_t)(c - 1));
        }
    }
    const int best = (int)(__reduce_min_sync(0xffffffffu, key) & 63u) + 1;
    const int per = (size + best - 1) / best;
    return {(size + per - 1) / per, per};
}

// A warp's 32 rows of a tile, from its row r0 on: how TMA is to fetch them.  Rows that follow one
// another in memory come as one box of 32 rows (rows behind the last come along, and are not used);
// others, four at a time (the last row again behind the last).  One lane issues: an instruction of
// many lanes is issued lane by lane, 64 cycles each.
struct RowFetch {
    int4 rows[8];
    int groups;       // of four; 0 where there are no rows
    bool together;
    __device__ __forceinline__ void start(const int32_t* perm, int first, int r0, int count) {
        const int here = min(32, count - r0);
        const int32_t* q = perm + first + r0;
        groups = here > 0 ? (here + 3) / 4 : 0;
        together = here > 0 && q[here - 1] - q[0] == here - 1;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < groups) {
                rows[i].x = q[4 * i];
                rows[i].y = q[min(4 * i + 1, here - 1)];
                rows[i].z = q[min(4 * i + 2, here - 1)];
                rows[i].w = q[min(4 * i + 3, here - 1)];
            }
    }
    __device__ __forceinline__ uint32_t bytes() const { return groups == 0 ? 0 : together ? 32 * 128 : groups * 512; }
    // 128 bytes of each row, from element x on.
    __device__ __forceinline__ void issue(uint8_t* dst, const CUtensorMap* one, const CUtensorMap* box, int x, uint64_t* bar) const {
        if (together) {
            ptx::tma_load_2d(dst, box, x, rows[0].x, bar);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < groups) tma_gather4(dst + 512 * i, one, x, rows[i], bar);
        }
    }
};

// Warp 0 fetches the adapter's rows, warp 1 issues the products, warps 2 to 5 fetch 32 rows of x each.
constexpr int kShrinkThreads = 192;

template <bool kBf16>
__global__ void __launch_bounds__(kShrinkThreads)
lora_shrink_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap xbox,
                   const __grid_constant__ CUtensorMap amap, const TcArgs g) {
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t* smem = align1024(raw);
    const LoraParams& p = g.p;
    const int stage_bytes = kBoxBytes + g.N * kBox * 2;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + g.stages * stage_bytes);
    uint64_t *empty = full + g.stages, *done = empty + g.stages;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < g.stages; ++i) {
            ptx::mbar_init(&full[i], 5);
            ptx::mbar_init(&empty[i], 1);
        }
        ptx::mbar_init(done, 1);
        *s_abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) ptx::tmem_alloc(s_tmem, g.tmem_cols);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *s_tmem;
    pdl_wait();
    pdl_trigger();   // (the next kernel's launch overlaps this one; it waits for its end)

    const int runs = p.ctrl->n_active, boxes = (p.K + kBox - 1) / kBox;
    const Pieces ks = pieces(runs, boxes, g.max_splits, kLoraBlocks);
    int slot = 0, unit_no = 0;
    uint32_t phase = 0;               // of the ring: the slot's use counted from 0, modulo 2
    bool used = false;                // the ring has been round
    for (int64_t unit = blockIdx.x; unit < (int64_t)runs * ks.n; unit += gridDim.x, ++unit_no) {
        const int tile = (int)(unit / ks.n), piece = (int)(unit % ks.n);
        const int adapter = p.segs[3 * tile], first = p.segs[3 * tile + 1], count = p.segs[3 * tile + 2];
        const int j0 = piece * ks.size, nj = min(boxes - j0, ks.size);
        auto next = [&]() {
            if (++slot == g.stages) {
                slot = 0;
                phase ^= 1;
                used = true;
            }
        };
        if (warp == 1) {
            const uint32_t idesc = ptx::idesc_f16(kM, g.N, kBf16);
            for (int j = 0; j < nj; ++j, next()) {
                if (!wait_warp(&full[slot], phase, s_abort, p.err, 32)) break;
                ptx::tc_fence_after();
                if (ptx::elect_one()) {
                    const uint64_t a = ptx::sw128_desc(ptx::smem_u32(smem + slot * stage_bytes));
                    const uint64_t b = ptx::sw128_desc(ptx::smem_u32(smem + slot * stage_bytes + kBoxBytes));
#pragma unroll
                    for (int k = 0; k < kBox / 16; ++k) ptx::mma_f16(tmem, a + 2 * k, b + 2 * k, idesc, j > 0 || k > 0);
                    ptx::mma_commit(&empty[slot]);
                    if (j == nj - 1) ptx::mma_commit(done);
                }
                __syncwarp();
            }
        } else {
            RowFetch f;
            if (warp > 1) f.start(p.perm, first, 32 * (warp - 2), count);
            const uint32_t bytes = warp == 0 ? g.N * kBox * 2 : f.bytes();
            for (int j = 0; j < nj; ++j, next()) {
                if (used && !wait_warp(&empty[slot], phase ^ 1, s_abort, p.err, 31)) break;
                uint8_t* at = smem + slot * stage_bytes;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(&full[slot], bytes);
                    const int k = (j0 + j) * kBox;
                    if (warp == 0) ptx::tma_load_2d(at + kBoxBytes, &amap, k, adapter * p.r, &full[slot]);
                    else if (bytes) f.issue(at + 4096 * (warp - 2), &xmap, &xbox, k, &full[slot]);
                }
                __syncwarp();
            }
        }
        __syncwarp();
        if (wait_warp(done, unit_no & 1, s_abort, p.err, 33)) {
            ptx::tc_fence_after();
            const int q = warp & 3, row = 32 * q + lane;     // (the quarter of tensor memory that the warp can read)
            float* to = g.part + ((int64_t)piece * p.n + first + row) * p.r;
            const uint32_t tb = tmem + ((uint32_t)(32 * q) << 16);
            if (warp > 1 && 32 * q < count)
                for (int c = 0; c < g.N; c += 16) {
                    float d[16];
                    ptx::tmem_ld16(tb + c, d);
                    if (row < count) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (c + 4 * i < p.r) *reinterpret_cast<float4*>(to + c + 4 * i) = make_float4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
                    }
                }
        }
        ptx::tc_fence_before();
        if (__syncthreads_or(*s_abort)) break;   // (and the accumulator is read)
        ptx::tc_fence_after();
    }
    // After a wait that gave up, copies may be in flight: they end before the block does.
    // The expansion finds no runs, and so writes nothing of a v that is not there.
    if (*s_abort && threadIdx.x == 0) p.ctrl->n_rsegs = 0;
    if (*s_abort && threadIdx.x == 0)
        for (int s = 0; s < g.stages; ++s) ptx::mbar_wait_quiet(&full[s], phase, ptx::kWaitLimitNs / 8);
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, g.tmem_cols);
    }
}

// v's parts added into the first, in their order, four elements a thread: where every block of the expansion would
// read and add many of them.
constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) lora_sum_kernel(const TcArgs g) {
    const LoraParams& p = g.p;
    pdl_wait();
    pdl_trigger();   // (the next kernel's launch overlaps this one; it waits for its end)
    const int n = pieces(p.ctrl->n_active, (p.K + kBox - 1) / kBox, g.max_splits, kLoraBlocks).n;
    const int64_t size = (int64_t)p.n * p.r / 4;
    float4* part = reinterpret_cast<float4*>(g.part);
    for (int64_t i = (int64_t)blockIdx.x * kSumThreads + threadIdx.x; n > 1 && i < size; i += (int64_t)gridDim.x * kSumThreads) {
        float4 v[kLoraMaxSplits];
#pragma unroll
        for (int k = 0; k < kLoraMaxSplits; ++k) v[k] = k < n ? part[i + k * size] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 1; k < kLoraMaxSplits; ++k)
            if (k < n) {
                v[0].x += v[k].x; v[0].y += v[k].y; v[0].z += v[k].z; v[0].w += v[k].w;
            }
        part[i] = v[0];
    }
}

constexpr int kNT = 128;                 // outputs of a tile
constexpr int kEpiWarps = 8;             // 32 rows and 64 outputs of a tile each
constexpr int kExpandThreads = 32 * (kEpiWarps + 2);
constexpr int kRing = 2;                 // tiles of B in flight
constexpr int kStageRow = 70;            // floats of a row of a warp's staging (64 and 6: fewest bank conflicts of both its sides)
constexpr int kStageBytes = 16 * kStageRow * 4;

__host__ __device__ constexpr int expand_parts(bool f32) { return f32 ? 3 : 2; }
constexpr size_t kMaxSmem = 226 * 1024;  // (beside 1 KB of static arrays)
// A warp's 32 rows and 64 outputs of base.
__host__ __device__ constexpr int ahead_bytes(bool f32) { return 32 * 64 * (f32 ? 4 : 2); }
inline size_t expand_smem(int rank16, bool f32, bool wide) {
    const int boxes = (rank16 + kBox - 1) / kBox;
    return 1024 + (size_t)(expand_parts(f32) + kRing) * boxes * kBoxBytes + kEpiWarps * (wide ? ahead_bytes(f32) : kStageBytes) + 256;
}

// Outputs o0 .. o1 of a row that has no adapter, by a warp: base's elements as they are (or zeros), 16 bytes at a
// time where the two rows are aligned alike, and then what is left at both ends; else by elements.
template <int kOut> __device__ __forceinline__ void copy_row(const LoraParams& p, int64_t row, int o0, int o1, int lane) {
    constexpr int kSize = kOut == MOE_F32 ? 4 : 2, kV = 16 / kSize, kU = 4;
    const int64_t from = row * p.base_stride, to = row * p.out_stride;
    const uint8_t* src = reinterpret_cast<const uint8_t*>(p.base) + from * kSize;
    uint8_t* dst = reinterpret_cast<uint8_t*>(p.out) + to * kSize;
    const uint32_t lag = (uint32_t)(reinterpret_cast<uintptr_t>(dst) + (uintptr_t)o0 * kSize);
    auto elements = [&](int a, int b) {
        for (int o = a + lane; o < b; o += 32 * 2 * kU) {
            uint32_t v[2 * kU];
#pragma unroll
            for (int u = 0; u < 2 * kU; ++u) v[u] = p.base && o + 32 * u < b ? load_bits<kOut>(src, o + 32 * u) : 0u;
#pragma unroll
            for (int u = 0; u < 2 * kU; ++u)
                if (o + 32 * u < b) store_bits<kOut>(dst, o + 32 * u, v[u]);
        }
    };
    int a = o0, b = o0;      // whole pieces: a .. b
    if (!p.base || ((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15) == 0) {
        a = min(o1, o0 + (int)((0u - lag) & 15) / kSize);
        b = a + (o1 - a) / kV * kV;
        for (int o = a + lane * kV; o < b; o += kU * kV * 32) {
            uint4 v[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u)
                v[u] = p.base && o + u * 32 * kV < b ? *reinterpret_cast<const uint4*>(src + (size_t)(o + u * 32 * kV) * kSize) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (o + u * 32 * kV < b) *reinterpret_cast<uint4*>(dst + (size_t)(o + u * 32 * kV) * kSize) = v[u];
        }
    }
    elements(o0, a);
    elements(b, o1);
}

// kWide: rows of base and out that are aligned to 16 bytes, of a multiple of 32 (fp32: 16) outputs.
template <bool kBf16, int kOut, bool kWide>
__global__ void __launch_bounds__(kExpandThreads, kOut == MOE_F32 ? 1 : 2)
lora_expand_kernel(const __grid_constant__ CUtensorMap bmap, const TcArgs g) {
    constexpr bool kF32 = kOut == MOE_F32;
    constexpr int kParts = expand_parts(kF32);
    extern __shared__ __align__(1024) uint8_t raw[];
    __shared__ int32_t s_rows[kM], s_exp[kM];
    const LoraParams& p = g.p;
    const int boxes = (g.N + kBox - 1) / kBox, vbytes = boxes * kBoxBytes;
    uint8_t* sV = align1024(raw);                       // [part][box][128 rows x 128 bytes]
    uint8_t* sB = sV + kParts * vbytes;                 // [stage][box][128 outputs x 128 bytes]
    uint8_t* sStage = sB + kRing * vbytes;
    uint64_t* bfull = reinterpret_cast<uint64_t*>(sStage + kEpiWarps * (kWide ? ahead_bytes(kF32) : kStageBytes));
    uint64_t *bempty = bfull + kRing, *tfull = bempty + kRing, *tempty = tfull + 2;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(tempty + 2);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            ptx::mbar_init(&bfull[i], 1);
            ptx::mbar_init(&bempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&tfull[i], 1);
            ptx::mbar_init(&tempty[i], kEpiWarps);
        }
        *s_abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == kEpiWarps) ptx::tmem_alloc(s_tmem, 2 * kNT);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *s_tmem;
    pdl_wait();
    pdl_trigger();   // (the next kernel's launch overlaps this one; it waits for its end)

    const int O = p.O, n_tiles = (O + kNT - 1) / kNT, runs = p.ctrl->n_rsegs;
    const int parts = g.summed ? 1 : pieces(p.ctrl->n_active, (p.K + kBox - 1) / kBox, g.max_splits, kLoraBlocks).n;
    const Pieces os = pieces(runs, n_tiles, 64, g.expand_blocks);
    int done_tiles = 0;      // of this block, before this unit
    constexpr int kSize = kF32 ? 4 : 2, kV = 16 / kSize;        // elements of 16 bytes
    constexpr int kPieces = 16 / kV;                            // of a lane's 16 outputs of a row
    for (int64_t unit = blockIdx.x; unit < (int64_t)runs * os.n; unit += gridDim.x) {
        const int tile = (int)(unit / os.n), t0 = (int)(unit % os.n) * os.size, nt = min(n_tiles - t0, os.size);
        const int adapter = p.segs[3 * tile], first = p.segs[3 * tile + 1], count = p.segs[3 * tile + 2];
        if (adapter < 0 && p.copy) {
            // Rows without an adapter: base's elements as they are.
            const int o0 = t0 * kNT, o1 = min(O, (t0 + nt) * kNT);
            for (int i = warp; i < count; i += kEpiWarps + 2) copy_row<kOut>(p, p.perm[first + i], o0, o1, lane);
        } else if (adapter >= 0) {
            const int q = warp & 3, half = warp >> 2, here = warp < kEpiWarps ? min(32, count - 32 * q) : 0;
            if (warp < 4 && lane < here) s_rows[32 * q + lane] = p.perm[first + 32 * q + lane];
            // kWide: rows 8 i + lane / 4 of the warp's (the last again behind it, which is not written), of each 4 kV
            // outputs kV from kV (lane % 4) on; base's of the first tile are on their way while v is formed.
            const uint8_t* from[4];
            uint8_t* to[4];
            const int left = O - (t0 * kNT + half * 64 + kV * (lane & 3));      // outputs from the lane's first one on
            uint8_t* mine = sStage + warp * ahead_bytes(kF32) + lane * 16;      // [row][piece][lane]
            // (Rows r that the warp has none of get no copies: no wait would stand between those and the next
            // unit's, which go to the same places.)
            auto fetch = [&](int i, int r) {
                if (p.base && i < nt && 8 * r < here) {
#pragma unroll
                    for (int w = 0; w < kPieces; ++w)
                        if (i * kNT + 4 * kV * w < left) cp_async16(mine + (r * kPieces + w) * 512, from[r] + (size_t)i * (kNT * kSize) + 64 * w);
                }
                cp_commit();
            };
            if constexpr (kWide) {
                if (here > 0) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int64_t row = p.perm[first + 32 * q + min(8 * r + (lane >> 2), here - 1)];
                        const int64_t o = t0 * kNT + half * 64 + kV * (lane & 3);
                        from[r] = reinterpret_cast<const uint8_t*>(p.base) + (row * p.base_stride + o) * kSize;
                        to[r] = reinterpret_cast<uint8_t*>(p.out) + (row * p.out_stride + o) * kSize;
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) fetch(0, r);
                }
            }
            // v of the tile's rows, split, in the products' layout: lanes of a row hold eight elements each.
            const int chunks = g.N / 8;
            int lanes = 2;
            while (lanes < chunks) lanes *= 2;
            const float scale = p.scale ? __ldg(p.scale + adapter) : 1.f;
            const int per_warp = 32 / lanes, c8 = lane % lanes;
            constexpr int kGroups = kWide ? 1 : 2;   // of rows whose loads are in flight together
            for (int g0 = warp * per_warp; warp < kEpiWarps && g0 < count; g0 += kGroups * kEpiWarps * per_warp) {
                float v[kGroups][8];
#pragma unroll
                for (int u = 0; u < kGroups; ++u) {
                    const int row = g0 + u * kEpiWarps * per_warp + lane / lanes;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
                    if (row < count && c8 * 8 < p.r) {
                        const float* part = g.part + (int64_t)(first + row) * p.r + c8 * 8;
#pragma unroll 2
                        for (int s = 0; s < parts; ++s, part += (int64_t)p.n * p.r) {
                            const float4 a = *reinterpret_cast<const float4*>(part), b = *reinterpret_cast<const float4*>(part + 4);
                            v[u][0] += a.x; v[u][1] += a.y; v[u][2] += a.z; v[u][3] += a.w;
                            v[u][4] += b.x; v[u][5] += b.y; v[u][6] += b.z; v[u][7] += b.w;
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < kGroups; ++u) {
                    const int row = g0 + u * kEpiWarps * per_warp + lane / lanes;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[u][i] *= scale;
                    int e = 0;
                    if constexpr (!kBf16) {
                        float most = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) most = fmaxf(most, finite_abs(v[u][i]));
                        for (int o = 1; o < lanes; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                        e = f16_shift(most);
                        if (row < count && c8 == 0) s_exp[row] = e;
                    }
                    uint16_t part[8][kParts];
#pragma unroll
                    for (int i = 0; i < 8; ++i) split<kBf16, kParts>(kBf16 ? v[u][i] : times_exp2(v[u][i], e), part[i]);
                    if (row < count && c8 < chunks) {
                        uint8_t* at = sV + (c8 >> 3) * kBoxBytes + row * 128 + (((c8 & 7) ^ (row & 7)) << 4);
#pragma unroll
                        for (int m = 0; m < kParts; ++m)
                            *reinterpret_cast<uint4*>(at + m * vbytes) =
                                make_uint4(part[0][m] | (uint32_t)part[1][m] << 16, part[2][m] | (uint32_t)part[3][m] << 16,
                                           part[4][m] | (uint32_t)part[5][m] << 16, part[6][m] | (uint32_t)part[7][m] << 16);
                    }
                }
            }
            if (warp <= kEpiWarps) {      // (the warp that fetches B has begun)
                ptx::fence_proxy_async_smem();
                ptx::named_bar(1, 32 * (kEpiWarps + 1));
            }

            // kWide: two fragments of 16 rows.
            auto epilogue = [&]() {
                float m0[4], m1[4];
                if (!kBf16) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = 8 * r + (lane >> 2), e = row < here ? -s_exp[32 * q + row] : 0;
                        m0[r] = exp2i(e >> 1);
                        m1[r] = exp2i(e - (e >> 1));
                    }
                }
                for (int i = 0; i < nt; ++i) {
                    const int buf = (done_tiles + i) & 1;
                    if (!wait_warp(&tfull[buf], ((done_tiles + i) >> 1) & 1, s_abort, p.err, 37)) return;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float d[32];
                        if (here > 16 * u) tmem_ld_fragments(tmem + ((uint32_t)(32 * q + 16 * u) << 16) + buf * kNT + half * 64, d);
                        if (u == 1) {                            // the accumulator is read
                            ptx::tc_fence_before();
                            __syncwarp();
                            ptx::mbar_arrive_elect(&tempty[buf]);
                        }
                        if (here <= 16 * u) {                    // (no rows: their groups all the same, so that the waits count right)
                            cp_commit();
                            cp_commit();
                            continue;
                        }
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const int r = 2 * u + s;
                            cp_wait<3>();                        // (a group a row: this one's is the oldest of four)
#pragma unroll
                            for (int w = 0; w < kPieces; ++w) {
                                float y[kV];
#pragma unroll
                                for (int j = 0; j < kV / 2; ++j) {
                                    y[2 * j] = d[4 * (kV / 2 * w + j) + 2 * s];
                                    y[2 * j + 1] = d[4 * (kV / 2 * w + j) + 2 * s + 1];
                                }
                                if constexpr (!kBf16) {
#pragma unroll
                                    for (int j = 0; j < kV; ++j) y[j] = y[j] * m0[r] * m1[r];
                                }
                                if (i * kNT + 4 * kV * w < left && 8 * r + (lane >> 2) < here) {
                                    if (p.base) add_raw<kOut>(*reinterpret_cast<const uint4*>(mine + (r * kPieces + w) * 512), y);
                                    *reinterpret_cast<uint4*>(to[r] + (size_t)i * (kNT * kSize) + 64 * w) = pack_raw<kOut>(y);
                                }
                            }
                            fetch(i + 1, r);                     // (to where this one was)
                        }
                    }
                }
            };
            // Any rows: 64 outputs of 16 rows at a time through the warp's staging.  Of each row its aligned pieces of 16
            // bytes belong to neighbouring lanes, and what is left before and behind them (8 elements of 16 bits, 4 of 32,
            // where the tile is full) to the same lanes by single elements.  All 32 rows of base are in flight while the
            // products run.
            auto any_rows = [&]() {
                constexpr int kCh = 64 / kV, kAt = 32 / kCh, kIt = 16 / kAt;   // pieces of a row, rows at a time, times of 16 rows
                float* stage = reinterpret_cast<float*>(sStage + warp * kStageBytes);
                const int c = lane % kCh, sub = lane / kCh;
                const bool alike = ((reinterpret_cast<uintptr_t>(p.base) ^ reinterpret_cast<uintptr_t>(p.out)) & 15) == 0 &&
                                   ((p.base_stride - p.out_stride) * kSize & 15) == 0;
                const uint32_t lag = (uint32_t)reinterpret_cast<uintptr_t>(p.out) / kSize;   // (in elements)
                for (int i = 0; i < nt; ++i) {
                    const int buf = (done_tiles + i) & 1, o0 = (t0 + i) * kNT + half * 64, lim = max(0, min(64, O - o0));
                    // Of row `w` of the warp's: its number, the outputs before the first whole piece, and the pieces.
                    auto place = [&](int w, int64_t& row, int& head, int& whole) {
                        row = s_rows[32 * q + w];
                        head = (int)((0u - lag - (uint32_t)row * (uint32_t)p.out_stride) & (kV - 1));
                        whole = max(0, lim - head) / kV;
                    };
                    uint4 was[2 * kIt];
                    uint32_t one[2 * kIt];
#pragma unroll
                    for (int t = 0; t < 2 * kIt; ++t) {
                        was[t] = make_uint4(0u, 0u, 0u, 0u);
                        one[t] = 0u;
                        const int w = kAt * t + sub;
                        if (p.base && w < here) {
                            int64_t row;
                            int head, whole;
                            place(w, row, head, whole);
                            const int64_t at = row * p.base_stride + o0;
                            if (c < whole) {
                                if (alike) was[t] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p.base) + (at + head + kV * c) * kSize);
                                else was[t] = gather_raw<kOut>(p.base, at + head + kV * c);
                            }
                            if (c < lim - kV * whole) one[t] = load_bits<kOut>(p.base, at + (c < head ? c : kV * whole + c));
                        }
                    }
                    if (!wait_warp(&tfull[buf], ((done_tiles + i) >> 1) & 1, s_abort, p.err, 37)) return;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        if (here > 16 * u) {
                            float d[32];
                            tmem_ld_fragments(tmem + ((uint32_t)(32 * q + 16 * u) << 16) + buf * kNT + half * 64, d);
                            float* to = stage + (lane >> 2) * kStageRow + 2 * (lane & 3);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                *reinterpret_cast<float2*>(to + 8 * j) = make_float2(d[4 * j], d[4 * j + 1]);
                                *reinterpret_cast<float2*>(to + 8 * kStageRow + 8 * j) = make_float2(d[4 * j + 2], d[4 * j + 3]);
                            }
                        }
                        if (u == 1) ptx::tc_fence_before();       // the accumulator is read
                        __syncwarp();
                        if (u == 1) ptx::mbar_arrive_elect(&tempty[buf]);
#pragma unroll
                        for (int t = kIt * u; t < kIt * (u + 1); ++t) {
                            const int w = kAt * t + sub;
                            if (w < here) {
                                int64_t row;
                                int head, whole;
                                place(w, row, head, whole);
                                const float* y0 = stage + (w - 16 * u) * kStageRow;
                                const int64_t at = row * p.out_stride + o0;
                                const int e = kBf16 ? 0 : -s_exp[32 * q + w];
                                if (c < whole) {
                                    float y[kV];
#pragma unroll
                                    for (int j = 0; j < kV; ++j) {
                                        y[j] = y0[head + kV * c + j];
                                        if constexpr (!kBf16) y[j] = times_exp2(y[j], e);
                                    }
                                    if (p.base) add_raw<kOut>(was[t], y);
                                    *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p.out) + (at + head + kV * c) * kSize) = pack_raw<kOut>(y);
                                }
                                auto single = [&](int k, uint32_t base) {
                                    float y = y0[k];
                                    if constexpr (!kBf16) y = times_exp2(y, e);
                                    store_one<kOut>(p.out, at + k, p.base ? of_bits<kOut>(base) + y : y);
                                };
                                const int rest = lim - kV * whole;
                                if (c < rest) single(c < head ? c : kV * whole + c, one[t]);
                                if (kV == 8 && c + kCh < rest) {         // (up to 14 at a row's end)
                                    const int k = c + kCh < head ? c + kCh : kV * whole + c + kCh;
                                    single(k, p.base ? load_bits<kOut>(p.base, row * p.base_stride + o0 + k) : 0u);
                                }
                            }
                        }
                        __syncwarp();                             // the staging is read
                    }
                }
            };
            if (warp == kEpiWarps + 1) {
                int sent = done_tiles;
                for (int i = 0; i < nt; ++i, ++sent) {
                    const int s = sent % kRing;
                    if (sent >= kRing && !wait_warp(&bempty[s], (sent / kRing - 1) & 1, s_abort, p.err, 34)) break;
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(&bfull[s], vbytes);
                        const int row = adapter * O + (t0 + i) * kNT;
                        for (int b = 0; b < boxes; ++b) {
                            uint8_t* at = sB + s * vbytes + b * kBoxBytes;
                            if constexpr (kWide) {
                                // Column 8 j + 2 t + e of a half is output 4 kV (j / (kV / 2)) + kV t + 2 (j % (kV / 2)) + e:
                                // a box of e and t for each j.
                                for (int c = 0; c < 16; ++c)
                                    tma_load_3d(at + c * 1024, &bmap, b * kBox, row + 64 * (c / 8) + 4 * kV * (c % 8 / (kV / 2)) + 2 * (c % (kV / 2)), 0, &bfull[s]);
                            } else {
                                ptx::tma_load_2d(at, &bmap, b * kBox, row, &bfull[s]);
                            }
                        }
                    }
                    __syncwarp();
                }
                if (ptx::aborted_warp(s_abort) && lane == 0)
                    for (int i = max(0, sent - kRing); i < sent; ++i) ptx::mbar_wait_quiet(&bfull[i % kRing], (i / kRing) & 1, ptx::kWaitLimitNs);
            } else if (warp == kEpiWarps) {
                const uint32_t idesc = ptx::idesc_f16(kM, kNT, kBf16);
                const int steps = g.N / 16;
                const uint64_t a_desc = ptx::sw128_desc(ptx::smem_u32(sV)), b_desc = ptx::sw128_desc(ptx::smem_u32(sB));
                for (int i = 0; i < nt; ++i) {
                    const int at = done_tiles + i, s = at % kRing, buf = at & 1;
                    if (!wait_warp(&bfull[s], (at / kRing) & 1, s_abort, p.err, 35)) break;
                    if (at >= 2 && !wait_warp(&tempty[buf], (at / 2 - 1) & 1, s_abort, p.err, 36)) break;
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) {
                        uint32_t more = 0;
                        const uint64_t b = b_desc + (uint32_t)(s * vbytes >> 4);
                        for (int m = kParts - 1; m >= 0; --m)     // the smallest part first
                            for (int box = 0; box < boxes; ++box) {
                                const uint32_t at = (uint32_t)(box * kBoxBytes >> 4);
                                const uint64_t a = a_desc + (uint32_t)(m * vbytes >> 4) + at;
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if (4 * box + k < steps) {
                                        ptx::mma_f16(tmem + buf * kNT, a + 2 * k, b + at + 2 * k, idesc, more);
                                        more = 1;
                                    }
                            }
                        ptx::mma_commit(&bempty[s]);
                        ptx::mma_commit(&tfull[buf]);
                    }
                    __syncwarp();
                }
            } else {
                if constexpr (kWide) {
                    epilogue();
                } else {
                    any_rows();
                }
            }
            done_tiles += nt;
        }
        if (__syncthreads_or(*s_abort)) break;   // (and v and the rows' numbers are read)
    }
    if (kWide) cp_wait<0>();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kEpiWarps) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 2 * kNT);
    }
}

template <typename Kern>
cudaError_t configure(Kern kern, int slot) {
    static std::mutex mu;
    static bool configured[128][14] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (configured[dev][slot]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e == cudaSuccess) configured[dev][slot] = true;
    return e;
}

}  // namespace

bool lora_maps(const LoraParams& p, int x_type, CUtensorMap (&maps)[5]) {
    // (Coordinates are 32-bit; strides fit 40 bits.)
    if ((int64_t)p.L * p.O > INT32_MAX - 1024 || p.x_stride * 2 >= (int64_t)1 << 40) return false;
    const CUtensorMapDataType t = x_type == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const uint32_t N = (p.r + 15) / 16 * 16;
    return make_map(&maps[0], p.x, t, 2, p.K, p.n, kBox, 1, CU_TENSOR_MAP_SWIZZLE_128B, p.x_stride) &&
           make_map(&maps[1], p.a, t, 2, p.K, (uint64_t)p.L * p.r, kBox, N, CU_TENSOR_MAP_SWIZZLE_128B) &&
           make_map(&maps[3], p.x, t, 2, p.K, p.n, kBox, 32, CU_TENSOR_MAP_SWIZZLE_128B, p.x_stride) &&
           make_map(&maps[2], p.b, t, 2, p.r, (uint64_t)p.L * p.O, kBox, kNT, CU_TENSOR_MAP_SWIZZLE_128B) &&
           make_map_pairs(&maps[4], p.b, t, p.r, (uint64_t)p.L * p.O, p.out_type == MOE_F32 ? 4 : 8);
}

cudaError_t launch_lora_tc(const LoraParams& p, int x_type, const CUtensorMap (&maps)[5], float* part, int max_segs, cudaStream_t st) {
    TcArgs g{};
    g.p = p;
    g.N = (p.r + 15) / 16 * 16;
    g.part = part;
    // Parts of v, one a stretch of K, that every block of the expansion would read and add are first added by a kernel
    // of their own, which costs less above a rank of 16 (us without and with it: 1000 rows of 7168, rank 64, 38.7 and 32.9;
    // 600 of 2048, rank 128, 39.0 and 22.7; 4000 of 4096, rank 64, 42.9 and 37.8; 1000 of 4096, rank 32, 23.7 and 21.5; 3001 of
    // 2048, rank 16, 26.6 and 28.2).
    g.summed = p.r > 16;
    g.max_splits = (int)std::min<int64_t>(kLoraMaxSplits, lora_part_rows(p.n) / p.n);
    const int stage = kBoxBytes + g.N * kBox * 2;
    g.stages = std::min((p.K + kBox - 1) / kBox, 100 * 1024 / stage);
    g.tmem_cols = 32;
    while (g.tmem_cols < g.N) g.tmem_cols *= 2;
    const size_t smem = 1024 + (size_t)g.stages * stage + 256;
    auto shrink = x_type == MOE_BF16 ? lora_shrink_kernel<true> : lora_shrink_kernel<false>;
    cudaError_t e = configure(shrink, x_type == MOE_BF16 ? 0 : 1);
    if (e != cudaSuccess) return e;
    if ((e = launch_pdl(shrink, dim3((unsigned)std::min<int64_t>(kLoraBlocks, (int64_t)max_segs * g.max_splits)), dim3(kShrinkThreads), smem, st,
                        maps[0], maps[3], maps[1], g)) != cudaSuccess)
        return e;

    if (g.summed &&
        (e = launch_pdl(lora_sum_kernel, dim3((unsigned)std::min<int64_t>(4 * kLoraBlocks, ((int64_t)p.n * p.r / 4 + kSumThreads - 1) / kSumThreads)),
                        dim3(kSumThreads), 0, st, g)) != cudaSuccess)
        return e;
    const bool f32 = p.out_type == MOE_F32, bf = x_type == MOE_BF16;
    const int64_t esize = f32 ? 4 : 2;
    const bool wide = !p.out_host && p.O * esize % 64 == 0 && p.vec * esize >= 16;
    const size_t expand_bytes = expand_smem(g.N, f32, wide);
    g.expand_blocks = f32 || expand_bytes > kMaxSmem / 2 ? kLoraBlocks / 2 : kLoraBlocks;
    const dim3 grid((unsigned)std::min<int64_t>(g.expand_blocks, (int64_t)max_segs * ((p.O + kNT - 1) / kNT)));
    auto of_out = [&](auto bf16, auto is_wide) {
        constexpr bool kB = decltype(bf16)::value, kW = decltype(is_wide)::value;
        return p.out_type == MOE_F32 ? lora_expand_kernel<kB, MOE_F32, kW> : p.out_type == MOE_BF16 ? lora_expand_kernel<kB, MOE_BF16, kW>
                                                                                                    : lora_expand_kernel<kB, MOE_F16, kW>;
    };
    using yes = std::true_type;
    using no = std::false_type;
    auto expand = bf ? (wide ? of_out(yes{}, yes{}) : of_out(yes{}, no{})) : (wide ? of_out(no{}, yes{}) : of_out(no{}, no{}));
    if ((e = configure(expand, 2 + (wide ? 6 : 0) + (bf ? 0 : 3) + p.out_type)) != cudaSuccess) return e;
    return launch_pdl(expand, grid, dim3(kExpandThreads), expand_bytes, st, maps[wide ? 4 : 2], g);
}

}  // namespace moe

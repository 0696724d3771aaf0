// moe_lora.cu -- low-rank adapters of many requests beside a shared projection (sm_103a):
//   out[t] = base[t] + scale[a] B_a (A_a x[t]),  a = idx[t];  out[t] = base[t] where a is no adapter
//
// Few rows: bound by the bytes of the adapters that occur and by latency.  One cluster takes up
// to eight rows that share an adapter, so that the adapter's matrices are read once for them (one row of
// 2048 -> 2048, rank 16: 3.8 us; 64 of 7168 -> 2048, rank 64, 8 adapters: 9.3; 256 of 2048 -> 5003 fp32,
// rank 32, 200 adapters: 15.5):
// its blocks split K for v = A x (each warp's products m16n8k16 with A as the rows and the
// eight x as the columns, 16-byte loads straight into the fragments), add their partial v over
// distributed shared memory, and split the outputs for B v.  No workspace and one launch.
//
// Exactness: products of 16-bit elements are exact in fp32 and summed there.  v enters the
// second product as a sum of 16-bit parts: two for outputs of 16 bits (16 bits of v, below the
// output's own rounding), three for fp32 outputs (24 bits of v).  fp16 parts are those of v
// times a power of two for each row, which takes its largest element to [2^14, 2^15).
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "moe_launch.cuh"
#include "moe_lora.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRows = 8;            // rows of a cluster (the n of the products)
constexpr int kScanRows = 1024;     // rows whose adapters a cluster goes through for itself, at most
constexpr int kGroupAdapters = 255; // adapters whose rows it counts, where it takes groups of rows
constexpr int kGroups = 448;        // of kRows at most

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// A float of block `rank`'s shared memory, at this block's address p.
__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), b;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(b) : "memory");
    return v;
}

template <bool kBf16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (kBf16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// out[row] = base[row] (zeros without a base), the block's part `part` of `parts`.
__device__ __forceinline__ void copy_row(const LoraParams& p, int64_t row, int part, int parts) {
    const int quads = (p.O + 3) / 4, step = p.vec >= 4 ? 1 : kThreads;
    for (int q0 = part * kThreads; q0 < quads; q0 += parts * kThreads) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        const int o = 4 * q0 + (step == 1 ? 4 : 1) * (int)threadIdx.x, left = p.O - o;
        if (p.base) load4(p.out_type, p.base, row * p.base_stride + o, step, left, v);
        store4(p.out_type, p.out, row * p.out_stride + o, step, left, v);
    }
}

// The rows in groups of kRows of an adapter, the adapters one after another, formed by each block for itself.  A
// row's rank among its adapter's rows: those before it in its 32 rows, and the counts of the 32s before, a byte
// each, 32 an adapter (table: (L + 1) times 32 bytes, the last one's of rows without an adapter).
struct Groups {
    uint16_t rows[kGroups * kRows], none[kScanRows], base[kThreads];
    uint8_t adapter[kGroups], count[kGroups];
};
struct Found {
    int groups, none;
};
__device__ __forceinline__ Found find_groups(const LoraParams& p, uint8_t* table, Groups& out) {
    constexpr int kH = kScanRows / kThreads, kWords = kScanRows / 128;
    static_assert(kGroupAdapters <= kThreads, "an adapter a thread");
    __shared__ int s_sum[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(table);
    for (int i = tid; i < 2 * (p.L + 1); i += kThreads) reinterpret_cast<uint4*>(table)[i] = make_uint4(0u, 0u, 0u, 0u);
    // (Of the kH times kThreads rows only those that are there are gone through: most calls have few.)
    int e[kH], rank[kH];
#pragma unroll
    for (int h = 0; h < kH; ++h) {
        const int row = tid + h * kThreads;
        e[h] = -2;
        rank[h] = 0;
        if (row < p.n) {
            e[h] = p.idx[row];
            if (e[h] < 0 || e[h] >= p.L) e[h] = p.L;
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kH; ++h) {
        if (h * kThreads >= p.n) continue;
        const uint32_t peers = __match_any_sync(0xffffffffu, e[h]);
        rank[h] = __popc(peers & ((1u << lane) - 1));
        if (rank[h] == 0 && e[h] >= 0) table[e[h] * 4 * kWords + warp + h * kWarps] = (uint8_t)__popc(peers);
    }
    __syncthreads();
    // Each adapter's groups: an adapter a thread.
    uint32_t total = 0, none = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        if (128 * i >= p.n) continue;
        if (tid < p.L) total = __dp4a(words[tid * kWords + i], 0x01010101u, total);
        none = __dp4a(words[p.L * kWords + i], 0x01010101u, none);
    }
    const int mine = (int)(total + kRows - 1) / kRows;
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
    }
    if (lane == 31) s_sum[warp] = before;
    before -= mine;
    __syncthreads();
    int groups = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        groups += s_sum[w];
    }
    out.base[tid] = (uint16_t)before;
    for (int j = 0; j < mine; ++j) {
        out.adapter[before + j] = (uint8_t)tid;
        out.count[before + j] = (uint8_t)min(kRows, (int)total - j * kRows);
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kH; ++h) {
        if (h * kThreads >= p.n) continue;
        const int b = warp + h * kWarps;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if (4 * i >= b) continue;
            const uint32_t c = words[max(e[h], 0) * kWords + i];
            const int here = min(b - 4 * i, 4);      // bytes of this word that count
            rank[h] = __dp4a(c, here == 4 ? 0x01010101u : 0x01010101u & ((1u << 8 * here) - 1), (uint32_t)rank[h]);
        }
        const int row = tid + h * kThreads;
        if (e[h] == p.L) out.none[rank[h]] = (uint16_t)row;
        else if (e[h] >= 0) out.rows[out.base[e[h]] * kRows + rank[h]] = (uint16_t)row;
    }
    __syncthreads();
    return {groups, (int)none};
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory"); }

// kRT: tiles of 16 of the rank.  kParts: parts of v.  kInGroups: a cluster for each group of rows (find_groups).
template <bool kBf16, int kRT, int kParts, bool kInGroups>
__global__ void __launch_bounds__(kThreads) lora_rows_kernel(const LoraParams p) {
    constexpr int kR = kRT * 16;
    constexpr int kPad = kRT == 1 ? 0 : 16;       // (no bank conflicts between rows of parts)
    constexpr int kSpan = kInGroups && kRT == 1 ? 2 * kWarps : kWarps;
    __shared__ __align__(16) float s_part[kSpan][kR][kRows];    // (first the counts,) then v's parts, [part][row][rank]
    __shared__ float s_mine[kR * kRows];
    __shared__ int s_rows[kWarps][kRows];         // (every warp finds them for itself)
    __shared__ uint32_t s_top[kRows];
    __shared__ std::conditional_t<kInGroups, Groups, int> s_groups;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int C = (int)cluster_size(), c = (int)cluster_rank(), group = blockIdx.x / C;
    if (tid < kRows) s_top[tid] = 0;
    pdl_wait();
    pdl_trigger();   // (the next kernel's launch overlaps this one; it waits for its end)

    // The cluster's rows: row `group`, if an adapter's rows before it fill whole clusters, and
    // the next ones of its adapter; kInGroups: the group-th of these; or a run of the rows sorted by adapter.
    int adapter, count;
    [[maybe_unused]] int none = 0;       // rows without an adapter that are to be written
    auto copy_none = [&]() {
        if constexpr (kInGroups)
            for (int i = group; i < none; i += p.groups) copy_row(p, s_groups.none[i], c, C);
    };
    if constexpr (kInGroups) {
        static_assert(sizeof(s_part) >= (kGroupAdapters + 1) * (kScanRows / 32), "the counts fit");
        const Found f = find_groups(p, reinterpret_cast<uint8_t*>(&s_part[0][0][0]), s_groups);
        none = p.copy ? f.none : 0;
        if (group >= f.groups) {
            copy_none();
            return;
        }
        adapter = s_groups.adapter[group];
        count = s_groups.count[group];
        if (lane < count) s_rows[warp][lane] = s_groups.rows[group * kRows + lane];
    } else if (p.segs) {
        if (group >= p.ctrl->n_rsegs) return;
        const int first = p.segs[3 * group + 1];
        adapter = p.segs[3 * group];
        count = p.segs[3 * group + 2];
        if (adapter < 0) {
            for (int i = 0; p.copy && i < count; ++i) copy_row(p, p.perm[first + i], c, C);
            return;
        }
        if (lane < count) s_rows[warp][lane] = p.perm[first + lane];
    } else {
        constexpr int kBatch = 4;   // of 32 rows whose loads are in flight
        adapter = p.idx[group];
        int before = 0, found = 0;
        for (int i0 = 0; i0 < p.n && found < kRows; i0 += 32 * kBatch) {
            int e[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) e[u] = i0 + 32 * u + lane < p.n ? p.idx[i0 + 32 * u + lane] : -1;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int row = i0 + 32 * u + lane;
                const uint32_t all = __ballot_sync(0xffffffffu, e[u] == adapter && row < p.n), late = __ballot_sync(0xffffffffu, row >= group);
                before += __popc(all & ~late);
                const int at = found + __popc(all & late & ((1u << lane) - 1));
                if ((all & late) >> lane & 1 && at < kRows) s_rows[warp][at] = row;
                found += __popc(all & late);
            }
        }
        if (adapter < 0 || adapter >= p.L) {
            if (p.copy) copy_row(p, group, c, C);
            return;
        }
        if (before % kRows) return;
        count = min(found, kRows);
    }
    __syncwarp();

    // v = A x: lane (g, t) holds elements 8 t .. 8 t + 7 of a step of 32 along K, of the rows g and
    // g + 8 of each tile and of x's row g.  (The products' order of k is any, the same for both.)
    const int K = p.K, r = p.r;
    const uint16_t* A = p.a + (int64_t)adapter * r * K;
    const uint16_t* x = g < count ? p.x + (int64_t)s_rows[warp][g] * p.x_stride : nullptr;
    const int steps = (K + 31) / 32, per = (steps + C - 1) / C, s1 = min(steps, (c + 1) * per);
    const int O = p.O, units = (O + 31) / 32, uper = (units + C - 1) / C, u1 = min(units, (c + 1) * uper);
    const uint16_t* Bm = p.b + (int64_t)adapter * O * r;
    // The block's part of B is asked for before the loads of A, by lines of 128 bytes.
    {
        const int64_t b0 = (int64_t)c * uper * 32 * r, b1 = (int64_t)min(O, u1 * 32) * r;
        for (int64_t e = b0 + tid * 64; e < b1; e += kThreads * 64) prefetch_l2(Bm + e);
    }
    const float scale = p.scale ? __ldg(p.scale + adapter) : 1.f;   // (long before it is used)
    float acc[kRT][4];
#pragma unroll
    for (int j = 0; j < kRT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    constexpr int kU = kRT >= 8 ? 1 : kRT == 4 ? 2 : 4 / kRT;   // steps in flight
    for (int s = c * per + warp; s < s1; s += kU * kWarps) {
        uint4 xv[kU], av[kU][kRT][2];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int su = s + u * kWarps, k = su * 32 + t * 8;
            const bool in = su < s1 && k < K;
            xv[u] = in && x ? __ldg(reinterpret_cast<const uint4*>(x + k)) : zero;
#pragma unroll
            for (int j = 0; j < kRT; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = j * 16 + i * 8 + g;
                    av[u][j][i] = in && row < r ? ld_stream_v4(A + (int64_t)row * K + k) : zero;
                }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int j = 0; j < kRT; ++j) {
                mma<kBf16>(acc[j], av[u][j][0].x, av[u][j][1].x, av[u][j][0].y, av[u][j][1].y, xv[u].x, xv[u].y);
                mma<kBf16>(acc[j], av[u][j][0].z, av[u][j][1].z, av[u][j][0].w, av[u][j][1].w, xv[u].z, xv[u].w);
            }
    }
#pragma unroll
    for (int j = 0; j < kRT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float2*>(&s_part[warp][j * 16 + i * 8 + g][2 * t]) = make_float2(acc[j][2 * i], acc[j][2 * i + 1]);
    __syncthreads();
    for (int e = tid; e < kR * kRows; e += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += (&s_part[w][0][0])[e];
        s_mine[e] = s;
    }
    // This lane's results are those of rows 2 t and 2 t + 1; outputs o .. o + 3 of a unit of 32 are rows g
    // and g + 8 of two tiles.  A unit's loads are made while the one before it is worked on, the first
    // one's before v is there (with more than 64 of rank there are no registers for that).
    int64_t orow[2];
    bool has[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        has[m] = 2 * t + m < count;
        orow[m] = has[m] ? s_rows[warp][2 * t + m] : 0;
    }
    uint2 bv[kRT][2][2];
    float was[2][4];
    // Output i of this lane's four of a unit: neighbouring ones where rows are read and written four at a time,
    // else 8 apart, so that neighbouring lanes have neighbouring ones.
    const bool fours = p.vec >= 4;
    const int ostep = fours ? 1 : 8, ofirst = fours ? 4 * g : g;
    auto fetch = [&](int u) {
        const int o = u * 32 + ofirst, left = u < u1 ? O - o : 0;
        const uint16_t* at = Bm + (int64_t)o * r + 4 * t;
#pragma unroll
        for (int j = 0; j < kRT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool in = i * ostep < left && j * 16 + 4 * t < r;
                bv[j][i >> 1][i & 1] = in ? ld_stream_v2(at + i * ostep * r + j * 16) : make_uint2(0u, 0u);
            }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int i = 0; i < 4; ++i) was[m][i] = 0.f;
            if (p.base && has[m]) load4(p.out_type, p.base, orow[m] * p.base_stride + o, ostep, left, was[m]);
        }
    };
    constexpr bool kEarly = kRT < 8;
    if (kEarly) fetch(c * uper + warp);
    cluster_arrive();
    copy_none();
    cluster_wait();
    // Each element of v is summed over the blocks in their order, and split, by one thread.
    constexpr int kMine = (kR * kRows + kThreads - 1) / kThreads;
    float v[kMine];
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
        const int i = tid + m * kThreads;
        v[m] = 0.f;
        if (i < kR * kRows) {
            float sum = 0.f;
            for (int b0 = 0; b0 < C; b0 += 8)
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    if (b0 + b < C) sum += ld_cluster(&s_mine[i], b0 + b);
            // (Elements behind the rank are 0, not what a 0 weight makes of an infinity.)
            if (i / kRows < r) v[m] = sum * scale;
            if (!kBf16) atomicMax(&s_top[i % kRows], __float_as_uint(finite_abs(v[m])));
        }
    }
    cluster_arrive();   // (the others' sums are read; waited for before the block ends)
    if (!kBf16) __syncthreads();
    uint16_t* s_v = reinterpret_cast<uint16_t*>(&s_part[0][0][0]);
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
        const int i = tid + m * kThreads;
        if (i < kR * kRows) {
            uint16_t part[kParts];
            split<kBf16, kParts>(kBf16 ? v[m] : times_exp2(v[m], f16_shift(__uint_as_float(s_top[i % kRows]))), part);
#pragma unroll
            for (int q = 0; q < kParts; ++q) s_v[(q * kRows + i % kRows) * (kR + kPad) + i / kRows] = part[q];
        }
    }
    __syncthreads();

    // out = base + B v: v's parts are the columns' operand; lane (g, t) holds elements 4 t .. 4 t + 3 of a
    // step of 16 along the rank.
    uint2 vb[kRT][kParts];
#pragma unroll
    for (int j = 0; j < kRT; ++j)
#pragma unroll
        for (int q = 0; q < kParts; ++q) vb[j][q] = *reinterpret_cast<const uint2*>(&s_v[(q * kRows + g) * (kR + kPad) + j * 16 + 4 * t]);
    float back[2][2];   // what takes this lane's results, rows 2 t and 2 t + 1, back to their size
    if constexpr (!kBf16) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int e = -f16_shift(__uint_as_float(s_top[2 * t + m]));
            back[m][0] = exp2i(e >> 1);
            back[m][1] = exp2i(e - (e >> 1));
        }
    }
    // (Not unrolled: every call runs this code for the first time, and its instructions are fetched as it goes:
    // four units at once took 4.9 us for a row of 2048 that takes 3.7 so.)
#pragma unroll 1
    for (int u = c * uper + warp; u < u1; u += kWarps) {
        const int o = u * 32 + ofirst, left = O - o;
        if (!kEarly) fetch(u);
        float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int j = 0; j < kRT; ++j)
#pragma unroll
            for (int q = kParts - 1; q >= 0; --q)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    mma<kBf16>(d[h], bv[j][h][0].x, bv[j][h][1].x, bv[j][h][0].y, bv[j][h][1].y, vb[j][q].x, vb[j][q].y);
        float y[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float w = d[i >> 1][2 * (i & 1) + m];
                if constexpr (!kBf16) w = w * back[m][0] * back[m][1];
                y[m][i] = was[m][i] + w;
            }
        if (kEarly && u + kWarps < u1) fetch(u + kWarps);
#pragma unroll
        for (int m = 0; m < 2; ++m)
            if (has[m]) store4(p.out_type, p.out, orow[m] * p.out_stride + o, ostep, left, y[m]);
    }
    cluster_wait();
}

// The rows sorted by adapter (stable), those of no adapter last, by one block: each warp counts and
// then places a stretch of the rows, 32 at a time, the equal ones among them found by a match.  No runs for the
// kernels behind it while `pending` (or null) has an error.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kBatch = 8;
__global__ void __launch_bounds__(kSortThreads)
lora_sort_kernel(const int32_t* __restrict__ idx, int n, int L, int tile, int32_t* __restrict__ perm, int32_t* __restrict__ segs, Ctrl* ctrl,
                 const int32_t* pending) {
    // cnt[e][w]: adapter e's rows (e = L: no adapter's) in warp w's stretch, then those before them;
    // total[e]: e's rows; first[e]: their first position.
    extern __shared__ int32_t cnt[];
    int32_t *total = cnt + (L + 1) * kSortWarps, *first = total + L + 1;
    __shared__ int32_t s_sum[2][32], s_all[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < (L + 1) * kSortWarps; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();   // (the next kernel's launch overlaps this one; it waits for its end)
    const bool stop = tid == 0 && pending && *pending >= kLoraErrFirst && *pending <= kLoraErrLast;
    const int per = (int)(((int64_t)n + kSortThreads - 1) / kSortThreads) * 32;
    const int64_t begin = (int64_t)warp * per, end = min((int64_t)n, begin + per);
    int ev[kBatch];
    auto fetch = [&](int64_t r0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t r = r0 + 32 * u + lane;
            ev[u] = r < end ? idx[r] : -1;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) ev[u] = r0 + 32 * u + lane < end ? (ev[u] >= 0 && ev[u] < L ? ev[u] : L) : -1;
    };
    for (int64_t r0 = begin; r0 < end; r0 += 32 * kBatch) {
        fetch(r0);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t peers = __match_any_sync(0xffffffffu, ev[u]);
            if (ev[u] >= 0 && lane == __ffs(peers) - 1) cnt[ev[u] * kSortWarps + warp] += __popc(peers);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int e = warp; e <= L; e += kSortWarps) {
        const int c = cnt[e * kSortWarps + lane];
        int s = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        cnt[e * kSortWarps + lane] = s - c;
        if (lane == 31) total[e] = s;
    }
    __syncthreads();
    // First position and first run of each adapter (L <= 1024, one a thread).
    const int c = tid < L ? total[tid] : 0, g = c / tile + (c % tile != 0);   // (c + tile may pass 2^31)
    int sc = c, sg = g;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int yc = __shfl_up_sync(0xffffffffu, sc, o), yg = __shfl_up_sync(0xffffffffu, sg, o);
        if (lane >= o) { sc += yc; sg += yg; }
    }
    if (lane == 31) { s_sum[0][warp] = sc; s_sum[1][warp] = sg; }
    __syncthreads();
    if (warp == 0) {
        const int c0 = s_sum[0][lane], g0 = s_sum[1][lane];
        int vc = c0, vg = g0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int yc = __shfl_up_sync(0xffffffffu, vc, o), yg = __shfl_up_sync(0xffffffffu, vg, o);
            if (lane >= o) { vc += yc; vg += yg; }
        }
        s_sum[0][lane] = vc - c0;
        s_sum[1][lane] = vg - g0;
        if (lane == 31) { s_all[0] = vc; s_all[1] = vg; }
    }
    __syncthreads();
    auto write_run = [&](int run, int e, int at, int count) {
        int32_t* s = segs + 3 * (int64_t)run;
        s[0] = e;
        s[1] = at;
        s[2] = min(tile, count);
    };
    if (tid < L) {
        const int at = s_sum[0][warp] + sc - c, run = s_sum[1][warp] + sg - g;
        first[tid] = at;
        for (int i = 0; i < g; ++i) write_run(run + i, tid, at + i * tile, c - i * tile);
    }
    const int none = total[L], runs = (int)(((int64_t)none + tile - 1) / tile);
    for (int i = tid; i < runs; i += kSortThreads) write_run(s_all[1] + i, -1, s_all[0] + i * tile, none - i * tile);
    if (tid == 0) {
        first[L] = s_all[0];
        ctrl->n_active = stop ? 0 : s_all[1];
        ctrl->n_rsegs = stop ? 0 : s_all[1] + runs;
        ctrl->err = 0;
    }
    __syncthreads();
    for (int64_t r0 = begin; r0 < end; r0 += 32 * kBatch) {
        if (per > 32 * kBatch) fetch(r0);   // (else they are still there)
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t peers = __match_any_sync(0xffffffffu, ev[u]);
            const int before = __popc(peers & ((1u << lane) - 1));
            int* mine = &cnt[max(ev[u], 0) * kSortWarps + warp];
            const int at = ev[u] >= 0 ? *mine + before : 0;
            __syncwarp();
            if (ev[u] >= 0) {
                perm[first[ev[u]] + at] = (int32_t)(r0 + 32 * u + lane);
                if (before == 0) *mine = at + __popc(peers);
            }
            __syncwarp();
        }
    }
}

template <bool kBf16, int kRT, int kParts, bool kInGroups>
cudaError_t launch_clusters(const LoraParams& p, int groups, int cluster, cudaStream_t st) {
    auto kern = lora_rows_kernel<kBf16, kRT, kParts, kInGroups>;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    auto blocks = [&](int of) {
        cfg.gridDim = dim3((unsigned)groups * of);
        attr[1].val.clusterDim.x = of;
    };
    if (cluster > 8) {   // (more than every GPU has to offer: to be asked for; eight blocks where there is no place for them)
        static std::mutex mu;
        static int fits[128] = {};   // 0: not known; -1: no; 1: yes
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lock(mu);
        if (!fits[dev]) {
            int at_once = 0;
            blocks(16);
            fits[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                                cudaOccupancyMaxActiveClusters(&at_once, kern, &cfg) == cudaSuccess && at_once > 0
                            ? 1 : -1;
            if (fits[dev] < 0) cudaGetLastError();   // (no error of the launch)
        }
        if (fits[dev] < 0) cluster = 8;
    }
    blocks(cluster);
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool kBf16, int kRT, int kParts>
cudaError_t launch_rows(const LoraParams& p, int groups, int cluster, cudaStream_t st) {
    return p.groups ? launch_clusters<kBf16, kRT, kParts, true>(p, groups, cluster, st)
                    : launch_clusters<kBf16, kRT, kParts, false>(p, groups, cluster, st);
}

template <bool kBf16, int kParts>
cudaError_t launch_rank(const LoraParams& p, int groups, int cluster, cudaStream_t st) {
    if (p.r <= 16) return launch_rows<kBf16, 1, kParts>(p, groups, cluster, st);
    if (p.r <= 32) return launch_rows<kBf16, 2, kParts>(p, groups, cluster, st);
    if (p.r <= 64) return launch_rows<kBf16, 4, kParts>(p, groups, cluster, st);
    return launch_rows<kBf16, 8, kParts>(p, groups, cluster, st);
}

cudaError_t launch_all(const LoraParams& p, int x_type, int groups, int cluster, cudaStream_t st) {
    const bool three = p.out_type == MOE_F32;
    if (x_type == MOE_BF16) return three ? launch_rank<true, 3>(p, groups, cluster, st) : launch_rank<true, 2>(p, groups, cluster, st);
    return three ? launch_rank<false, 3>(p, groups, cluster, st) : launch_rank<false, 2>(p, groups, cluster, st);
}

// Bytes of an adapter's matrices.
int64_t adapter_bytes(int K, int O, int r) { return (int64_t)r * ((int64_t)K + O) * 2; }

// The groups of kRows that L adapters' rows make at most, where so few clusters are launched; 0: one a row.  A
// cluster then costs the ranking of all rows, and saves the launches of those whose row another one takes.  (us a
// row each and so: 64 rows, 8 adapters of 131 KB 5.9 and 5.6; 30 rows, 3 of 2 MB 12.6 and 11.5; 200 rows, 20 of
// 1.1 MB 23.7 and 15.6; 500 rows, 8 of 262 KB 16.0 and 10.2; 8 rows of one adapter 4.1 and 4.9; 256 rows, 100 of
// 440 KB, 119 groups, 17.1 and 17.6.)
int most_groups(int n, int L) { return (int)((n + 7LL * std::min(n, L)) / 8); }
int group_count(int n, int L) {
    const int most = most_groups(n, L);
    return n > 16 && L <= kGroupAdapters && most <= std::min(n * 7 / 16, kGroups) ? most : 0;
}

// Rows that the clusters take as they come, each going through all of them for its own; more are sorted first.
// (us so and sorted: 500 rows, 131 KB an adapter 12.5 and 20.9, 64 adapters of 459 KB 26.5 and 43.8; of rank 64, 4 of
// 1.8 MB 27.5 and 33.6, 8 of 1 MB 18.1 and 25.4, 20 of 1.8 MB 35.3 and 31.3; 400 rows, 16 of rank 128 45 and 30.  In groups:
// 700 rows, 96 groups of 393 KB 15.4 and 22.5; 1024 rows, 215 of 131 KB 20.2 and 29.1; 1000 rows, 132 of 262 KB 21.2 and
// 22.8, 142 of 524 KB 31.2 and 26.4; 600 rows, 82 of 1 MB 33.4 and 26.3.)  What holds for n rows holds for fewer, so
// that a workspace for many serves few; above 512 rows L <= 182 makes them groups.
bool by_scan(int64_t n, int L, int K, int O, int r) {
    const int64_t bytes = adapter_bytes(K, O, r);
    if (n <= 256 || (n <= 512 && (bytes < 1 << 20 || (L <= 8 && r <= 64)))) return true;
    return n <= kScanRows && L <= 182 && most_groups((int)n, L) * bytes <= 48 << 20;
}

// Blocks of a cluster.  More share an adapter's bytes among them; but most rows' clusters find that
// another one has them, and all of them are launched.  (us with 4, 8 and 16 blocks: one row, 131 KB an
// adapter 4.2, 3.7, 3.8, 459 KB 7.9, 5.5, 4.8; 32 rows 4.9, 4.7, 6.8, 11.6, 8.5, 8.7, 1.8 MB 21.2, 14.5, 12.1;
// 128 rows 6.9, 7.7, 14.4, 15.4, 12.3, 19.0; 256 rows 8.6, 12.4, 22.7, 17.7, 19.2, 27.6.)
int cluster_blocks(int n, int64_t bytes) {
    constexpr int64_t kSmall = 256 << 10, kLarge = 1 << 20;
    if (n <= 32) return bytes >= kLarge || (n <= 8 && bytes >= kSmall) ? 16 : 8;
    if (n <= 128) return bytes < kSmall ? 4 : 8;
    return n > 384 && bytes < kSmall ? 2 : 4;
}

// The same where groups are launched, most of which have rows.  (us with 2, 4, 8 and 16 blocks: 6 groups of 2 MB 32,
// 20, 12.7, 11.5; 15 of 131 KB 7.7, 6.0, 5.6, 6.3; 15 of 1.1 MB 16.8, 11.0, 8.9, 10.6; 42 of 448 KB, rank 16, 21, 13.3, 11.9,
// 13.5; 40 of 1 MB, rank 64, 21.6, 16.5, 20.0, 32; 80 of 1.8 MB 48, 35, 50, 81; 118 of 131 KB 10.8, 11.4, 16.2, 27.6;
// 143 of 378 KB 19.8, 25.5, 37, 82.)
int group_blocks(int groups, int64_t bytes, int r) {
    const bool large = bytes >= 256 << 10;
    if (large && groups * 16 <= kLoraBlocks / 2) return 16;
    if (groups * 8 <= (large && r <= 32 ? 400 : 240)) return 8;
    return groups <= 100 ? 4 : 2;
}

struct Layout {
    size_t perm, segs, part, total;
};
Layout layout(int64_t n, int L, int K, int O, int r) {
    Layout l{};
    size_t off = sizeof(Ctrl);
    auto take = [&](size_t bytes) { const size_t o = off; off = align_up(off + bytes, 256); return o; };
    if (!by_scan(n, L, K, O, r)) {
        l.perm = take(sizeof(int32_t) * n);
        l.segs = take(sizeof(int32_t) * 3 * (n / kRows + std::min<int64_t>(n, L + 1) + 1));
        l.part = take(sizeof(float) * lora_part_rows(n) * r);
    }
    l.total = off;
    return l;
}

cudaError_t launch_sort(const LoraParams& p, int tile, int32_t* perm, int32_t* segs, const int32_t* pending, cudaStream_t st) {
    const size_t smem = sizeof(int32_t) * (p.L + 1) * (kSortWarps + 2);
    static std::mutex mu;
    static bool configured[128] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!configured[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(lora_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       (int)sizeof(int32_t) * (kMaxExperts + 1) * (kSortWarps + 2));
            if (e != cudaSuccess) return e;
            configured[dev] = true;
        }
    }
    return launch_pdl(lora_sort_kernel, dim3(1), dim3(kSortThreads), smem, st, p.idx, p.n, p.L, tile, perm, segs, p.ctrl, pending);
}

}  // namespace

size_t lora_workspace(int64_t n, int L, int K, int O, int r) { return layout(n, L, K, O, r).total; }

cudaError_t launch_lora(const LoraParams& given, int x_type, void* ws, cudaStream_t st) {
    LoraParams p = given;
    const int size = p.out_type == MOE_F32 ? 4 : 2;
    auto rows_of = [&](int v, const void* a, int64_t stride) {
        return !a || (reinterpret_cast<uintptr_t>(a) % (v * size) == 0 && (p.n == 1 || stride % v == 0));
    };
    p.vec = 1;
    for (int v : {4, 8})
        if (rows_of(v, p.out, p.out_stride) && rows_of(v, p.base, p.base_stride)) p.vec = v;
    p.copy = p.base != p.out;
    cudaError_t e;
    if (by_scan(p.n, p.L, p.K, p.O, p.r)) {
        const int64_t bytes = adapter_bytes(p.K, p.O, p.r);
        p.groups = group_count(p.n, p.L);
        e = p.groups ? launch_all(p, x_type, p.groups, group_blocks(p.groups, bytes, p.r), st)
                     : launch_all(p, x_type, p.n, cluster_blocks(p.n, bytes), st);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    const Layout l = layout(p.n, p.L, p.K, p.O, p.r);
    uint8_t* w = static_cast<uint8_t*>(ws);
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(w);
    p.ctrl = ctrl;
    if (!p.err) p.err = &ctrl->err;
    p.segs = reinterpret_cast<int32_t*>(w + l.segs);
    p.perm = reinterpret_cast<int32_t*>(w + l.perm);
    CUtensorMap maps[5];
    const bool tc = !p.x_host && lora_maps(p, x_type, maps);
    const int tile = tc ? kLoraTile : kRows;
    if ((e = launch_sort(p, tile, reinterpret_cast<int32_t*>(w + l.perm), reinterpret_cast<int32_t*>(w + l.segs), given.err, st)) != cudaSuccess)
        return e;
    const int max_segs = (int)(p.n / tile + std::min(p.n, p.L + 1) + 1);
    e = tc ? launch_lora_tc(p, x_type, maps, reinterpret_cast<float*>(w + l.part), max_segs, st)
           : launch_all(p, x_type, max_segs, 4, st);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe

// Gated feed-forward block on the 5th-generation tensor cores, forward and
// backward.
//
//   forward   g = x Wg^T, u = x Wu^T, a = act(g) u, y = a Wd^T (+ res)
//   backward  da = dy Wd, dg = da u act'(g), du = da act(g),
//             dx = [dg du] [Wg; Wu], dW = [dg du]^T x, dWd = dy^T a
//   act       SiLU g s(g), or GELU in its tanh form g s(2 z), z = sqrt(2/pi)
//             (g + 0.044715 g^3), s the logistic function
//
// Six products, one kernel template over the operands' layouts and the
// epilogue:
//   EPI_GLU    gate and up columns of the same channels side by side in one
//              accumulator; the activation and the product in the epilogue, so
//              g and u reach global memory only when the backward needs them
//   EPI_DGLU   da in the accumulator; the epilogue reads g and u and writes
//              dg and du
//   EPI_OUT    bf16 output, residual added in fp32 before the one rounding
//   EPI_PART   fp32 partial sums of a split contraction (few tiles: the
//              operands are read by all SMs), joined by a second kernel
// CLUSTER (up to 128 rows): the CTAs that split a tile's contraction are a
// cluster and add their sums through shared memory: no second kernel and
// nothing in global memory (one row, d 1152, f 1456: 19.0 us with partial sums
// and a join, 14.0 so; 3 rows, d 384, f 1952 in E4M3 17.0 and 11.3; one row,
// d 2560, f 10240 36.1 and 34.7; at worst 20 rows, d 384, f 7824 15.3 and 16.4).
// MIXED: waves of whole tiles; the stages of the tiles that do not fill a wave
// are dealt out evenly, in order, and a tile that several workers share leaves
// partial sums for the join (2048 rows, d 2560, f 10240, whose down projection
// has 80 tiles for 74 pairs: 247 us with two waves, 226 so; with the backward
// 791 and 725; n 4952, d 808, f 3232 with the backward 299 and 279).
// DUAL: a pair takes two neighbouring gate and up tiles at once, an accumulator
// each, and reads a stage of x once for both: where one wave of such holds all
// (256 rows, d 2560, f 10240: 55.0 us with two waves, 52.8 so; 700 rows, d 2048,
// f 4096, 46.1 and 43.3; not where less than that is saved: E4M3, 1000 rows,
// d 1024, f 2816, 30.5 and 32.1).
// An operand whose contraction index is the row of its matrix (Wd in da, Wgu
// in dx, both in the weight gradients) is loaded as it lies and multiplied
// MN-major: nothing is transposed in memory.
//
// Persistent, warp-specialised (416 threads): warps 0 and 2-4 TMA producers,
// warp 1 allocates TMEM and issues tcgen05.mma, warps 5-12 epilogue (two warps per
// TMEM lane quarter, taking turns on 16-column chunks).  Two accumulators of
// up to 256 columns: the epilogue of a tile overlaps the MMAs of the next.
// More than 128 rows run on CTA pairs (M = 256, each CTA stages its rows of A
// and half of the columns of B).  Every wait is bounded as in the projection
// kernels: on a timeout the status bit is set, the roles leave their loops,
// copies and MMAs in flight are drained and TMEM is freed.
#include <algorithm>
#include <mutex>

#include "ctx.cuh"
#include "tc.cuh"

namespace engram {
namespace {

enum { EPI_GLU = 0, EPI_DGLU = 1, EPI_OUT = 2, EPI_PART = 3 };

constexpr int BM = 128;                 // rows per CTA (UMMA M 128, or 256 over a pair)
constexpr int ROWB = 128;               // bytes of a swizzled shared-memory row: 64 bf16 or 128 E4M3
constexpr int BK = 64;                  // contraction indices per stage of MN-major (bf16) operands
constexpr int A_BYTES = BM * ROWB;      // 16 KB
constexpr int MAX_BN = 256;
constexpr int EPI_WARPS = 8;
constexpr int EPI_PARTS = EPI_WARPS / 4;   // warps per TMEM lane quarter, taking turns on 16-column chunks
constexpr int EPI_WARP0 = 5;            // warps 0-4: producers and MMA issuer
constexpr int THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
constexpr int TMEM_COLS = 512;

// Shared memory: a ring of stages, each A rows then B rows of 128 bytes.  Few
// rows stage only the rows they have, and a narrow tile only its columns, so
// that more stages are in flight: the ring's round trip (free slot -> load ->
// MMA -> free slot) is about 1.4 us, and a stage takes that over the number of
// stages at least.  A pair's epilogue keeps the end of the area for its patches or
// inputs, which leaves six or four stages of a 256 x 256 tile (with three it is
// slower, with seven no faster).
constexpr int TILE_AREA = 7 * 32768;
constexpr int STAGING = EPI_WARPS * 4096;    // a patch for each epilogue warp of a pair
// DGLU on a pair: two buffers per epilogue warp for 32 columns of its 32 rows'
// g and u: [g high 2 KB | u high 2 KB | g low 1 KB | u low 1 KB]
constexpr int IN_BUF = 6144;
constexpr int IN_AREA = EPI_WARPS * 2 * IN_BUF;
constexpr int MAX_STAGES = 14;
constexpr int SMEM_BYTES = TILE_AREA + 1024 + 1024;   // ring | barriers | alignment

struct __align__(8) Barriers {
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint64_t in[EPI_WARPS][2];     // DGLU on a pair: the warp's input buffers
    uint32_t tmem_base;
    volatile int abort_flag;
    int issued[5];            // stages loaded by each producer warp
    int consumed;
    uint32_t peer_abort;
};

struct FfnParams {
    int M, N;                   // output rows and columns (EPI_GLU: channels)
    int64_t ldo;                // elements from one row of out to the next
    int kb;                     // stages along the contraction
    int bn;                     // accumulator columns per tile (EPI_GLU: gate and up together)
    int n_tiles, m_units, splits, raster;
    int full, dealt, shares;    // MIXED: tiles computed whole, workers the others are dealt to, partial sums per tile at most
    uint32_t idesc;
    int a_bytes, b_bytes;       // of a stage
    int stages;
    int b_rows;                 // K-major B: rows per box
    int act;
    __nv_bfloat16* out;         // GLU: a [M][N]; DGLU: dgu [M][2N]; OUT: [M][N]
    uint4* gu_hi;               // upper 16 bits of g and u, 8 columns an element: written by GLU (or null), read by DGLU
    uint2* gu_lo;               // the next 8 bits
    const __nv_bfloat16* res;   // OUT: [M][N] or null
    const float* row_scale;     // FP8: [M]
    const float* col_scale;     // FP8: [2N]
    float4* part;               // PART: [splits] of a matrix [M][N] (GLU: [M][2N]); MIXED: [tiles][shares] of [256][bn]; see part_at
    uint32_t* status;
    int late_wait;              // nothing here depends on the kernel before: wait for it only before leaving
    int stall;                  // test hook: CTA 0 announces its first B stage but never loads it
};

// Bounded wait for the phase with `parity`; false when the CTA aborted or the
// wait ran out.  Operands arrive by the async proxy and accumulators are read
// behind tcgen05 fences, so CTA scope serves the pair's barriers too.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, Barriers* sb, uint32_t* status) {
    const uint32_t a = smem_u32(bar);
    if (mbar_try_wait(a, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (mbar_try_wait(a, parity)) return true;
        if (sb->abort_flag) return false;
        if (clock64() - t0 > kWaitCycles) {
            flag(status, ENGRAM_ERR_TIMEOUT);
            sb->abort_flag = 1;
            if (sb->peer_abort) st_remote_s32(sb->peer_abort, 1);
            return false;
        }
    }
}

// MN-major operand, 128-byte swizzle: boxes of 64 elements x 64 contraction
// rows of 128 bytes (8 KB); the leading offset steps from one 64-element box
// to the next, the stride offset from one group of 8 contraction rows to the next
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr) {
    uint64_t d = 0;
    d |= (uint64_t)((addr & 0x3FFFF) >> 4);
    d |= (uint64_t)((BK * ROWB) >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// bulk_g2s with an L2 policy: what is read once leaves first
__device__ __forceinline__ void bulk_g2s_hint(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

template <bool PAIR, bool F8>
__device__ __forceinline__ void umma(uint32_t tmem_d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR && F8)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d), "l"(da), "l"(db),
                     "r"(idesc), "r"(accumulate));
    else if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d), "l"(da), "l"(db),
                     "r"(idesc), "r"(accumulate));
    else if constexpr (F8)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d), "l"(da), "l"(db),
                     "r"(idesc), "r"(accumulate));
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d), "l"(da), "l"(db),
                     "r"(idesc), "r"(accumulate));
}

// ---------------------------------------------------------------- activation

// p = act(g) / g = 1 / (1 + exp(-k)): k = g, or 2 sqrt(2/pi) (g + 0.044715 g^3)
// = g k1, with exp(-k) = 2^(-k log2 e) by the hardware's base-2 exponential and
// reciprocal (2 and 1 ulp; an infinite denominator gives 0).  g2 = g^2, held
// below 1e4 so that k' stays finite where p is 0 or 1 anyway.
template <bool GELU>
__device__ __forceinline__ float act_p(float g, float& g2) {
    constexpr float kLog2e = 1.4426950409f;
    float k = -kLog2e * g, e, r;
    if (GELU) {
        g2 = fminf(g * g, 1e4f);
        k = g * fmaf(-0.0713548163f * kLog2e, g2, -1.5957691216f * kLog2e);
    }
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(k));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// act'(g) = p + g p (1 - p) k'(g), gp = g p
template <bool GELU>
__device__ __forceinline__ float act_d(float gp, float p, float g2) {
    if (GELU) gp *= fmaf(0.2140644488f, g2, 1.5957691216f);
    return fmaf(gp, 1.f - p, p);
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* f) { Vec<__nv_bfloat16>::load(p, f); }

// g and u are kept for the backward as 24 of their 32 bits:
// in bf16 their rounding would reach d_x and d_Wgu beside that of dg and du
// (measured against 64 bits: 3.5e-3 of the norm, with 24 bits 2.4e-3); the
// lower plane costs a byte per value.  Both planes are blocked as the
// epilogues hold them, [row / 32][column / 8][row % 32] elements of 8 columns:
// a warp's access is contiguous, where rows of 2 N would touch 32 lines
// (d_gate_up of 16372 rows, d 2560, f 6824: 1343 us by rows, 673 us blocked).
// Prefetching a tile of them into L2 ahead costs 45 us more than it saves.
__device__ __forceinline__ int64_t at24(const FfnParams& p, int64_t row, int col) {
    return ((row >> 5) * (p.N / 4) + col / 8) * 32 + (row & 31);
}

// Reading repeats the low byte L below itself, so the lower 16 bits stand for
// one of 257 L, L = 0 .. 255: zeros, infinities and NaN come back as they were.
// L is the nearest of them, (255 low + 32895) >> 16, which never carries into
// the upper half: a value is off by 128 units of 2^-23 at most, 2^-16 of itself.
// (Cutting L off would leave 2^-15; it takes two instructions less a value: 700
// rows, d 2048, f 4096 48 us, 49 so; 16372 rows, d 2560, f 6824 1318 us either way.)
__device__ __forceinline__ void put24(const FfnParams& p, int64_t at, const float* f) {
    uint32_t b[8], m[8], hi[4], lo[2];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        b[k] = __float_as_uint(f[k]);
        m[k] = (b[k] & 0xffffu) * 255u + 32895u;     // L in byte 2
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) hi[k] = __byte_perm(b[2 * k], b[2 * k + 1], 0x7632);
#pragma unroll
    for (int k = 0; k < 2; ++k)
        lo[k] = __byte_perm(__byte_perm(m[4 * k], m[4 * k + 1], 0x0062), __byte_perm(m[4 * k + 2], m[4 * k + 3], 0x0062), 0x5410);
    p.gu_hi[at] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    p.gu_lo[at] = make_uint2(lo[0], lo[1]);
}

struct Raw24 {
    uint4 hi;
    uint2 lo;
    __device__ __forceinline__ void load(const FfnParams& p, int64_t at) {
        hi = __ldcs(p.gu_hi + at);     // read once: leaves L2 to the operands
        lo = __ldcs(p.gu_lo + at);
    }
    __device__ __forceinline__ void get(float* f) const {
        const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[2] = {lo.x, lo.y};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            // bytes 3, 2 from a half of h, 1 and 0 both byte k % 4 of l
            f[k] = __uint_as_float(__byte_perm(l[k / 4], h[k / 2], (k & 1 ? 0x7600u : 0x5400u) + 0x11u * (k & 3)));
        }
    }
};

// Eight columns from c of one row, wherever the sums came from; *8 leave the
// values to store in their arguments.
template <bool GELU>
__device__ __forceinline__ void glu8(const FfnParams& p, int64_t row, int c, float* g, const float* u) {
    if (p.gu_hi) {
        put24(p, at24(p, row, c), g);
        put24(p, at24(p, row, p.N + c), u);
    }
    float g2;
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = g[k] * act_p<GELU>(g[k], g2) * u[k];
}

template <bool GELU>
__device__ __forceinline__ void dglu8(const Raw24& rg, const Raw24& ru, float* dg, float* du) {
    float g[8], u[8], g2;
    rg.get(g);
    ru.get(u);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float da = dg[k], pr = act_p<GELU>(g[k], g2), gp = g[k] * pr;
        du[k] = da * gp;
        dg[k] = da * u[k] * act_d<GELU>(gp, pr, g2);
    }
}

__device__ __forceinline__ void add8(float* v, const uint4& r) {
    float f[8];
    load8(reinterpret_cast<const __nv_bfloat16*>(&r), f);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += f[k];
}

__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// ---------------------------------------------------------------- work of a CTA or pair

// Row unit and column tile of tile t: groups of `raster` row units share the
// columns' slice of B while it is in L2.
__device__ __forceinline__ void place(const FfnParams& p, int t, int& row, int& nt) {
    const int per = p.raster * p.n_tiles;
    const int g = t / per, local = t - g * per;
    const int rows_g = min(p.raster, p.m_units - g * p.raster);
    row = g * p.raster + local % rows_g;
    nt = local / rows_g;
}

// MIXED: the stages of the tiles behind the first `full`, numbered through, are
// dealt to `dealt` workers: worker w has [w T / dealt, (w + 1) T / dealt).
__device__ __forceinline__ int64_t dealt_stages(const FfnParams& p) {
    return (int64_t)(p.n_tiles * p.m_units - p.full) * p.kb;
}
__device__ __forceinline__ int64_t deal_lo(const FfnParams& p, int64_t T, int w) { return w * T / p.dealt; }
// the worker that has stage x
__device__ __forceinline__ int deal_of(const FfnParams& p, int64_t T, int64_t x) {
    return (int)(((x + 1) * p.dealt - 1) / T);
}

// Partial sums lie four columns an element, [row / 32][column / 4][row % 32]: a
// warp's rows are contiguous where they are written and read (d 2560, f 10240,
// 256 rows: 62 us by rows, 55 so; n 615, d 496, f 4952 with its backward 92
// and 87).
__device__ __forceinline__ int64_t part_at(int cols, int64_t row, int col) {
    return ((row >> 5) * (cols / 4) + col / 4) * 32 + (row & 31);
}
__host__ __device__ inline int64_t part_size(int64_t rows, int cols) { return (rows + 31) / 32 * 32 * (cols / 4); }

__device__ __forceinline__ void add4(float* acc, const float4& a) {
    acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

// sums of eight columns over n matrices `next` elements apart
__device__ __forceinline__ void add_parts(float* acc, const float4* at, int n, int64_t next) {
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
        add4(acc, at[k * next]);
        add4(acc + 4, at[k * next + 32]);
    }
}

constexpr int MAX_CLUSTER = 8;      // CTAs; what every device of the kind takes

enum { WHOLE, SPLIT, MIXED_TAIL, TWO_TILES, CLUSTER };

struct Work {
    int row, nt;        // row unit, column tile
    int klo, khi;       // stages
    int split;          // PART
    int slot;           // MIXED: where the partial sums go, or -1: the whole tile
};

// The epilogue of eight columns whose sums are complete but for the FP8 scales.
template <int EPI, bool F8, bool GELU>
__device__ __forceinline__ void finish8(const FfnParams& p, int64_t row, int c, float* f, float* g) {
    if constexpr (F8) {
        const float rs = p.row_scale[row];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            f[k] *= rs * p.col_scale[c + k];
            g[k] *= rs * p.col_scale[p.N + c + k];
        }
    }
    if constexpr (EPI == EPI_GLU) glu8<GELU>(p, row, c, f, g);
    if constexpr (EPI == EPI_DGLU) {
        Raw24 rg, ru;
        rg.load(p, at24(p, row, c));
        ru.load(p, at24(p, row, p.N + c));
        dglu8<GELU>(rg, ru, f, g);
        *reinterpret_cast<uint4*>(p.out + row * p.ldo + p.N + c) = pack8(g);
    }
    if constexpr (EPI == EPI_OUT) {
        if (p.res) add8(f, *reinterpret_cast<const uint4*>(p.res + row * p.N + c));
    }
    *reinterpret_cast<uint4*>(p.out + row * p.ldo + c) = pack8(f);
}

// ---------------------------------------------------------------- kernel

// AMN / BMN: the operand is MN-major (contraction index = row of its matrix).
// GLU: B's two column halves are the gate and up rows of the same channels.
template <int EPI, bool GLU, bool AMN, bool BMN, bool PAIR, bool F8, bool GELU, int MODE>
__global__ void __launch_bounds__(THREADS, 1)
ffn_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const FfnParams p) {
    constexpr int NCTA = PAIR ? 2 : 1;
    constexpr bool MIXED = MODE == MIXED_TAIL, DUAL = MODE == TWO_TILES, CL = MODE == CLUSTER;
    const int STAGES = p.stages;
    const int stage_bytes = p.a_bytes + p.b_bytes;
    constexpr int KSTEP = F8 ? 128 : 64;        // contraction indices per stage
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
    const uint32_t tiles_u32 = smem_u32(smem);
    Barriers* sb = reinterpret_cast<Barriers*>(smem + TILE_AREA);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_rank() : 0u;
    const bool leader = rank == 0;
    const int unit0 = (int)blockIdx.x / NCTA, step = (int)gridDim.x / NCTA;
    const int tiles = p.n_tiles * p.m_units;
    const int num_units = tiles * p.splits;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sb->full[s], (2 + AMN + BMN) * NCTA);   // the producers of each CTA, on the leader's barrier
            mbar_init(&sb->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sb->tfull[a], 1);
            mbar_init(&sb->tempty[a], NCTA * EPI_WARPS);
        }
        mbar_init(&sb->drain, 1);
        for (int w = 0; w < 2 * EPI_WARPS; ++w) mbar_init(&sb->in[0][0] + w, 1);
        sb->abort_flag = 0;
        for (int w = 0; w < 5; ++w) sb->issued[w] = 0;
        sb->consumed = 0;
        sb->peer_abort = PAIR ? peer_addr(const_cast<const int*>(&sb->abort_flag), rank ^ 1u) : 0u;
        mbar_fence_init();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sb->tmem_base)),
                         "r"(TMEM_COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sb->tmem_base)),
                         "r"(TMEM_COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    if constexpr (PAIR) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = sb->tmem_base;
    grid_dep_launch_dependents();

    // this worker's units one after the other: every role walks the same list
    struct Cursor {
        int u;
        int64_t pos, end;
    };
    const int64_t T = MIXED ? dealt_stages(p) : 0;
    auto begin = [&]() {
        Cursor c{unit0, 0, 0};
        if (MIXED && unit0 < p.dealt) {
            c.pos = deal_lo(p, T, unit0);
            c.end = deal_lo(p, T, unit0 + 1);
        }
        return c;
    };
    auto next = [&](Cursor& c, Work& w) {
        w.split = 0;
        w.slot = -1;
        w.klo = 0;
        w.khi = p.kb;
        if (!MIXED) {
            if (c.u >= num_units) return false;
            w.split = CL ? c.u % p.splits : c.u / tiles;
            place(p, CL ? c.u / p.splits : c.u - w.split * tiles, w.row, w.nt);
            w.klo = (int)((int64_t)p.kb * w.split / p.splits);
            w.khi = (int)((int64_t)p.kb * (w.split + 1) / p.splits);
        } else if (c.u < p.full) {
            place(p, c.u, w.row, w.nt);
        } else {
            if (c.pos >= c.end) return false;
            const int tt = (int)(c.pos / p.kb);
            const int64_t t0 = (int64_t)tt * p.kb;
            w.klo = (int)(c.pos - t0);
            w.khi = (int)min((int64_t)p.kb, c.end - t0);
            place(p, p.full + tt, w.row, w.nt);
            if (w.klo != 0 || w.khi != p.kb) w.slot = tt * p.shares + unit0 - deal_of(p, T, t0);
            c.pos = t0 + w.khi;
            return true;
        }
        c.u += step;
        return true;
    };
    // bytes of B that producer `part` loads a stage: 64-column boxes in turn
    auto b_share = [&](int part) {
        if (!BMN) return p.b_bytes;
        const int boxes = p.b_bytes / (BK * ROWB);
        return (boxes + 1 - part) / 2 * (BK * ROWB);
    };

    if (warp == 0 || warp == 2 || (AMN && warp == 3) || (BMN && warp == 4)) {
        // ---------------- TMA producers, one load a stage each where it can
        // be (a thread that issues two is slower than the MMAs: 0.46 us a
        // stage, and 0.56 us with all four, against 0.36): warp 0 loads A and
        // warp 2 B, warps 3 and 4 the second halves of MN-major ones
        if (lane == 0) {
            const bool is_a = warp == 0 || warp == 3;
            const int part = warp >= 3;
            const bool remote = PAIR && !leader;
            const uint32_t bytes = (uint32_t)(is_a ? (AMN ? p.a_bytes / 2 : p.a_bytes) : b_share(part));
            int* issued = &sb->issued[warp];
            // A may come from a kernel of this call that is still running; B
            // (weights, x, the saved a) never does
            if (is_a && !p.late_wait) grid_dep_wait();
            int it = 0, s = 0;
            uint32_t ph = 0;
            Work w;
            for (Cursor cur = begin(); !sb->abort_flag && next(cur, w);) {
                const int m0 = (w.row * NCTA + (int)rank) * BM;
                bool ok = true;
                for (int kb = w.klo; kb < w.khi; ++kb, ++it) {
                    if (!wait_bounded(&sb->empty[s], ph ^ 1u, sb, p.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = remote ? peer_addr(&sb->full[s], 0u) : smem_u32(&sb->full[s]);
                    auto load = [&](const CUtensorMap* m, uint32_t dst, int x, int y) {
                        if (remote) tma_load_2d_peer_bar(m, dst, bar, x, y);
                        else tma_load_2d(m, dst, &sb->full[s], x, y);
                    };
                    if (remote) mbar_arrive_expect_tx_remote(bar, bytes);
                    else mbar_arrive_expect_tx(&sb->full[s], bytes);
                    const int k0 = kb * KSTEP;
                    const uint32_t a_dst = tiles_u32 + s * stage_bytes;
                    const uint32_t b_dst = a_dst + p.a_bytes;
                    if (p.stall && it == 0 && warp == 2 && blockIdx.x == 0) {
                        // bounded-wait test: announced above, never loaded
                    } else if (is_a) {
                        if (AMN) load(&map_a, a_dst + part * (BK * ROWB), m0 + part * 64, k0);
                        else load(&map_a, a_dst, k0, m0);
                    } else if constexpr (BMN) {
                        const int n0 = w.nt * p.bn + (int)rank * (p.bn / 2);
                        const int cols = PAIR ? p.bn / 2 : p.bn;
                        for (int c = part * 64; c < cols; c += 128) load(&map_b, b_dst + c * ROWB, n0 + c, k0);
                    } else if constexpr (GLU) {
                        // gate rows from nt * bn / 2, up rows N behind; a pair's second CTA stages the up rows
                        const int n0 = w.nt * p.b_rows;
                        load(&map_b, b_dst, k0, n0 + (PAIR ? (int)rank * p.N : 0));
                        if (!PAIR) load(&map_b, b_dst + p.b_rows * ROWB, k0, n0 + p.N);
                    } else {
                        load(&map_b, b_dst, k0, w.nt * p.bn + (int)rank * (p.bn / 2));
                    }
                    *issued = it + 1;
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
            }
        }
    } else if (warp == 1 && (!PAIR || leader)) {
        // ---------------- MMA issuer
        if (lane == 0) {
            int it = 0, tc = 0, s = 0;
            uint32_t ph = 0;
            Work w;
            for (Cursor cur = begin(); !sb->abort_flag && next(cur, w); tc += DUAL ? 2 : 1) {
                const int acc = tc & 1;
                const uint32_t aph = (uint32_t)(tc >> 1) & 1u;
                if (!wait_bounded(&sb->tempty[acc], aph ^ 1u, sb, p.status)) break;
                if (DUAL && !wait_bounded(&sb->tempty[1], aph ^ 1u, sb, p.status)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * MAX_BN);
                bool ok = true;
                for (int kb = w.klo; kb < w.khi; ++kb, ++it) {
                    if (!wait_bounded(&sb->full[s], ph, sb, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = tiles_u32 + s * stage_bytes;
                    const uint64_t da = AMN ? smem_desc_mn(a_addr) : smem_desc_sw128(a_addr);
                    const uint64_t db = BMN ? smem_desc_mn(a_addr + p.a_bytes) : smem_desc_sw128(a_addr + p.a_bytes);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        // 16 contraction indices: 32 bytes inside the swizzled row, or 16 rows of 128 bytes
                        umma<PAIR, F8>(d_tmem, da + (uint64_t)(kk * (AMN ? 128 : 2)), db + (uint64_t)(kk * (BMN ? 128 : 2)),
                                       p.idesc, (uint32_t)((kb != w.klo) | (kk != 0)));
                        if constexpr (DUAL)
                            umma<PAIR, F8>(d_tmem + MAX_BN, da + (uint64_t)(kk * 2), db + (uint64_t)(p.b_bytes / 32 + kk * 2), p.idesc,
                                           (uint32_t)((kb != w.klo) | (kk != 0)));
                    }
                    if constexpr (PAIR) umma_commit_pair_both(&sb->empty[s]);
                    else umma_commit(&sb->empty[s]);
                    sb->consumed = it + 1;
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                if constexpr (PAIR) umma_commit_pair_both(&sb->tfull[acc]);
                else umma_commit(&sb->tfull[acc]);
                if constexpr (DUAL) umma_commit_pair_both(&sb->tfull[1]);
            }
        }
    } else if (warp >= EPI_WARP0) {
        // ---------------- epilogue: a warp reads the TMEM lane quarter of its number
        const int q = warp & 3, part = (warp - EPI_WARP0) >> 2;
        const uint32_t leader_tempty[2] = {PAIR ? peer_addr(&sb->tempty[0], 0u) : 0u, PAIR ? peer_addr(&sb->tempty[1], 0u) : 0u};
        // A warp takes blocks of BLK columns in turn with the others of its
        // lane quarter.  STAGED: its lanes, a row each, leave their bf16 values
        // in a patch of shared memory [32 rows][128 bytes] (16-byte chunks
        // swizzled by the row), and the patch goes out four full lines per
        // instruction; by rows, a store touches 32 lines of 16 bytes.
        constexpr bool BULK = PAIR && EPI == EPI_DGLU;
        constexpr bool STAGED = PAIR && EPI != EPI_PART && !BULK;
        constexpr int BLK = STAGED ? 64 : 16;
        uint8_t* patch = smem + TILE_AREA - STAGING + (warp - EPI_WARP0) * (STAGING / EPI_WARPS);
        auto patch_at = [&](int r, int ch) {
            return reinterpret_cast<uint4*>(patch + r * 128 + ((ch ^ (r & 7)) << 4));
        };
        // the warp's k-th chunk of 16 columns
        auto chunk = [&](int k) { return part * BLK + k / (BLK / 16) * (BLK * EPI_PARTS) + k % (BLK / 16) * 16; };
        int tc = 0;
        if (!p.late_wait) grid_dep_wait();   // reads what earlier kernels wrote, writes what they may still read
        // BULK: 32 columns of g and u at a time, copied by the warp's lane 0 a
        // block ahead, over tiles too.  Loads into registers keep too few
        // bytes in flight: the epilogue of 16384 rows, f 6912 alone took 399
        // us with them, 149 us without any, 206 us (5.5 TB/s) with the copies.
        uint8_t* in_buf = smem + TILE_AREA - IN_AREA + (warp - EPI_WARP0) * 2 * IN_BUF;
        int in_sent = 0, in_used = 0;
        const uint64_t in_policy = l2_policy_evict_first();
        // columns of g (and of u) of block b of unit u that this warp reads: 0 where there is nothing
        auto in_cols = [&](const Work& w, int b) {
            const int64_t row0 = (int64_t)(w.row * NCTA + (int)rank) * BM + q * 32;
            return row0 < p.M && w.slot < 0 ? max(0, min(32, p.N - (w.nt * p.bn + b))) : 0;
        };
        auto in_copy = [&](const Work& w, int b) {
            const int cols = in_cols(w, b);
            if (cols == 0) return;
            if (lane == 0) {
                const int64_t row0 = (int64_t)(w.row * NCTA + (int)rank) * BM + q * 32;
                const int col = w.nt * p.bn + b;
                uint8_t* to = in_buf + (in_sent & 1) * IN_BUF;
                uint64_t* bar = &sb->in[warp - EPI_WARP0][in_sent & 1];
                const uint32_t hi = (uint32_t)cols * 64, lo = (uint32_t)cols * 32;
                mbar_arrive_expect_tx(bar, 2 * (hi + lo));
                bulk_g2s_hint(to, p.gu_hi + at24(p, row0, col), hi, bar, in_policy);
                bulk_g2s_hint(to + 2048, p.gu_hi + at24(p, row0, p.N + col), hi, bar, in_policy);
                bulk_g2s_hint(to + 4096, p.gu_lo + at24(p, row0, col), lo, bar, in_policy);
                bulk_g2s_hint(to + 5120, p.gu_lo + at24(p, row0, p.N + col), lo, bar, in_policy);
            }
            ++in_sent;
        };
        Work w, ahead;
        Cursor cur = begin();
        bool more = next(cur, ahead);
        if (BULK && more) in_copy(ahead, part * 32);
        for (; more || (DUAL && tc & 1); ++tc) {
            if (DUAL && tc & 1) {
                ++w.nt;
            } else {
                w = ahead;
                if (DUAL) w.nt *= 2;
                more = next(cur, ahead);
            }
            const int acc = tc & 1;
            const uint32_t aph = (uint32_t)(tc >> 1) & 1u;
            const int64_t row = (int64_t)(w.row * NCTA + (int)rank) * BM + q * 32 + lane;
            const bool live = row < p.M;
            const int width = GLU ? p.bn / 2 : p.bn;       // output columns of the tile
            const int c_tile = w.nt * width;
            // g and u of two chunks are held or in flight, the tile's first ones while its MMAs run
            Raw24 rg[2][2], ru[2][2];     // not BULK
            auto fetch = [&](int c, Raw24* fg, Raw24* fu) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int col = c_tile + c + h * 8;
                    if (live && c + h * 8 < width && col < p.N) {
                        fg[h].load(p, at24(p, row, col));
                        fu[h].load(p, at24(p, row, p.N + col));
                    }
                }
            };
            if constexpr (EPI == EPI_DGLU && !BULK && !CL) {
                fetch(chunk(0), rg[0], ru[0]);
                fetch(chunk(1), rg[1], ru[1]);
            }
            const bool ok = wait_bounded(&sb->tfull[acc], aph, sb, p.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + (uint32_t)(acc * MAX_BN) + ((uint32_t)(q * 32) << 16);
            float rs = 1.f;
            if (F8 && live) rs = __ldg(p.row_scale + row);
            if constexpr (BULK) {
                bool in_ok = true;
#pragma unroll 1
                for (int b = part * 32; b < p.bn; b += 32 * EPI_PARTS) {
                    // the next block: of this tile, or the first of the next one
                    if (b + 32 * EPI_PARTS < p.bn) in_copy(w, b + 32 * EPI_PARTS);
                    else if (more) in_copy(ahead, part * 32);
                    const int cols = in_cols(w, b);
                    if (cols == 0) continue;
                    const uint8_t* from = in_buf + (in_used & 1) * IN_BUF + lane * 16;
                    in_ok = wait_bounded(&sb->in[warp - EPI_WARP0][in_used & 1], (uint32_t)(in_used >> 1) & 1u, sb, p.status);
                    if (!__all_sync(0xffffffffu, in_ok)) break;
                    ++in_used;
                    uint4 o[4][2];
#pragma unroll
                    for (int c16 = 0; c16 < 32; c16 += 16) {
                        uint32_t x[16];
                        tmem_ld16(taddr + b + c16, x);
                        tmem_wait_ld(x);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int g8 = c16 / 8 + h;
                            Raw24 xg, xu;
                            xg.hi = *reinterpret_cast<const uint4*>(from + g8 * 512);
                            xu.hi = *reinterpret_cast<const uint4*>(from + 2048 + g8 * 512);
                            xg.lo = *reinterpret_cast<const uint2*>(from - lane * 8 + 4096 + g8 * 256);
                            xu.lo = *reinterpret_cast<const uint2*>(from - lane * 8 + 5120 + g8 * 256);
                            float f[8], g[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(x[h * 8 + k]);
                            dglu8<GELU>(xg, xu, f, g);
                            o[g8][0] = pack8(f);
                            o[g8][1] = pack8(g);
                        }
                    }
                    // out through the same buffer: [dg | du][32 rows][64 bytes], chunks swizzled by the row pair,
                    // then two full sectors a row, eight rows per instruction
                    uint8_t* const out_buf = in_buf + ((in_used - 1) & 1) * IN_BUF;
                    __syncwarp();
#pragma unroll
                    for (int g8 = 0; g8 < 4; ++g8)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            *reinterpret_cast<uint4*>(out_buf + k * 2048 + lane * 64 + ((g8 ^ ((lane >> 1) & 3)) << 4)) = o[g8][k];
                    __syncwarp();
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        const int r = it * 8 + (lane >> 2), ch = lane & 3;
                        const int64_t to_row = row - lane + r;
                        if (to_row < p.M && ch * 8 < cols) {
                            const uint8_t* at = out_buf + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
                            __nv_bfloat16* to = p.out + to_row * p.ldo + c_tile + b + ch * 8;
                            *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(at);
                            *reinterpret_cast<uint4*>(to + p.N) = *reinterpret_cast<const uint4*>(at + 2048);
                        }
                    }
                    // the buffer is read and written before the next copy into it
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (!__all_sync(0xffffffffu, in_ok)) break;
            }
            if (MIXED && w.slot >= 0) {
                // a share of the tile: the accumulator's columns as they are
                float4* const to = p.part + w.slot * part_size(2 * BM, p.bn) +
                                   part_at(p.bn, (int)rank * BM + q * 32 + lane, 0);
#pragma unroll 1
                for (int c = part * 16; c < p.bn; c += 16 * EPI_PARTS) {
                    uint32_t x[16];
                    tmem_ld16(taddr + c, x);
                    tmem_wait_ld(x);
                    if (live) {
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            to[(c + k) * 8] = make_float4(__uint_as_float(x[k]), __uint_as_float(x[k + 1]), __uint_as_float(x[k + 2]),
                                                          __uint_as_float(x[k + 3]));
                    }
                    __syncwarp();
                }
            }
            if constexpr (CL) {
                // this CTA's share of the sums, [column / 4][row], where the ring was: its MMAs are done
                float4* const to = reinterpret_cast<float4*>(smem) + q * 32 + lane;
#pragma unroll 1
                for (int c = part * 16; c < p.bn; c += 16 * EPI_PARTS) {
                    uint32_t x[16];
                    tmem_ld16(taddr + c, x);
                    tmem_wait_ld(x);
                    if (live) {
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            to[(c + k) / 4 * p.M] = make_float4(__uint_as_float(x[k]), __uint_as_float(x[k + 1]),
                                                                __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
                    }
                    __syncwarp();
                }
            }
            // the patch's lane: row r of four, 16-byte chunk lane % 8
            auto each_line = [&](int b0, auto&& f) {
#pragma unroll
                for (int it = 0; it < 8; ++it) {
                    const int r = it * 4 + (lane >> 3), ch = lane & 7;
                    const int64_t to_row = row - lane + r;
                    const int col = c_tile + b0 + ch * 8;
                    if (to_row < p.M && b0 + ch * 8 < width && col < p.N) f(r, ch, to_row, col);
                }
            };
            const int nk = BULK || CL || (MIXED && w.slot >= 0) ? 0
                           : STAGED ? (width + 64 * EPI_PARTS - 1) / (64 * EPI_PARTS) * 4
                                    : ((width + 16 * EPI_PARTS - 1) / (16 * EPI_PARTS) + 1) / 2 * 2;
#pragma unroll 1
            for (int k2 = 0; k2 < nk; k2 += 2) {
#pragma unroll
                for (int odd = 0; odd < 2; ++odd) {
                    const int k = k2 + odd, c = chunk(k), b0 = c / BLK * BLK;
                    if (b0 >= width) break;
                    if (STAGED && EPI == EPI_OUT && p.res && k % 4 == 0) {
                        each_line(b0, [&](int r, int ch, int64_t to_row, int col) {
                            *patch_at(r, ch) = *reinterpret_cast<const uint4*>(p.res + to_row * p.N + col);
                        });
                        __syncwarp();
                    }
                    uint32_t x[16], y[16];
                    tmem_ld16(taddr + c, x);
                    if (GLU) tmem_ld16(taddr + width + c, y);
                    tmem_wait_ld(x);
                    if (GLU) tmem_wait_ld(y);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int col = c_tile + c + h * 8;
                        if (!live || c + h * 8 >= width || col >= p.N) continue;
                        float f[8], g[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            f[k] = __uint_as_float(x[h * 8 + k]);
                            if (GLU) g[k] = __uint_as_float(y[h * 8 + k]);
                        }
                        if constexpr (F8) {
                            float sf[8], sg[8];
                            Vec<float>::load(p.col_scale + col, sf);
                            Vec<float>::load(p.col_scale + col + 4, sf + 4);
                            Vec<float>::load(p.col_scale + p.N + col, sg);
                            Vec<float>::load(p.col_scale + p.N + col + 4, sg + 4);
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                f[k] *= rs * sf[k];
                                g[k] *= rs * sg[k];
                            }
                        }
                        const int ch = (c - b0) / 8 + h;
                        if constexpr (EPI == EPI_PART) {
                            const int ld = GLU ? 2 * p.N : p.N;
                            float4* to = p.part + w.split * part_size(p.M, ld) + part_at(ld, row, col);
                            to[0] = make_float4(f[0], f[1], f[2], f[3]);
                            to[32] = make_float4(f[4], f[5], f[6], f[7]);
                            if (GLU) {
                                to += (int64_t)p.N * 8;
                                to[0] = make_float4(g[0], g[1], g[2], g[3]);
                                to[32] = make_float4(g[4], g[5], g[6], g[7]);
                            }
                        } else {
                            if constexpr (EPI == EPI_GLU) glu8<GELU>(p, row, col, f, g);
                            if constexpr (EPI == EPI_DGLU) dglu8<GELU>(rg[odd][h], ru[odd][h], f, g);
                            if constexpr (EPI == EPI_OUT) {
                                if (p.res)
                                    add8(f, STAGED ? *patch_at(lane, ch) : *reinterpret_cast<const uint4*>(p.res + row * p.N + col));
                            }
                            *(STAGED ? patch_at(lane, ch) : reinterpret_cast<uint4*>(p.out + row * p.ldo + col)) = pack8(f);
                            if constexpr (EPI == EPI_DGLU)
                                *reinterpret_cast<uint4*>(p.out + row * p.ldo + p.N + col) = pack8(g);
                        }
                    }
                    if constexpr (EPI == EPI_DGLU) fetch(chunk(k + 2), rg[odd], ru[odd]);
                    __syncwarp();
                    if (STAGED && k % 4 == 3) {
                        each_line(b0, [&](int r, int ch, int64_t to_row, int col) {
                            __nv_bfloat16* to = p.out + to_row * p.ldo + col;
                            *reinterpret_cast<uint4*>(to) = *patch_at(r, ch);
                        });
                        __syncwarp();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR && !leader) mbar_arrive_remote(leader_tempty[acc]);
                else mbar_arrive(&sb->tempty[acc]);
            }
        }
        // an aborted warp leaves no copy in flight
        for (; BULK && in_used < in_sent; ++in_used)
            mbar_wait_timed(&sb->in[warp - EPI_WARP0][in_used & 1], (uint32_t)(in_used >> 1) & 1u);
    }

    // this grid must not complete before the one it depends on: those behind it count on both
    if (p.late_wait) grid_dep_wait();
    __syncthreads();
    if constexpr (CL) {
        // every CTA of the tile adds the shares, in split order, of some of its columns and rows
        cluster_sync_all();
        const int width = GLU ? p.bn / 2 : p.bn, total = p.M * (width / 8);
        int unit, nt;
        place(p, (int)blockIdx.x / p.splits, unit, nt);
        for (int i = (int)cluster_rank() * THREADS + threadIdx.x; i < total; i += p.splits * THREADS) {
            const int v = i / p.M, row = i - v * p.M, c = nt * width + v * 8;
            if (c >= p.N) continue;
            float f[8] = {}, g[8] = {};
            const float4* const at = reinterpret_cast<const float4*>(smem) + v * 2 * p.M + row;
#pragma unroll 4
            for (int k = 0; k < p.splits; ++k) {
                add4(f, ld_cluster_f4(peer_addr(at, k)));
                add4(f + 4, ld_cluster_f4(peer_addr(at + p.M, k)));
                if constexpr (GLU) {
                    add4(g, ld_cluster_f4(peer_addr(at + width / 4 * p.M, k)));
                    add4(g + 4, ld_cluster_f4(peer_addr(at + (width / 4 + 1) * p.M, k)));
                }
            }
            finish8<EPI, F8, GELU>(p, row, c, f, g);
        }
    }
    bool aborted = sb->abort_flag != 0;
    if constexpr (PAIR) {
        cluster_sync_all();
        aborted = aborted || ld_remote_s32(sb->peer_abort) != 0;
    }
    if (aborted) {
        // copies issued but not consumed, the peer's among them; a stage that
        // not every producer reached never completes, so one limit covers all
        if (warp == 0 && lane == 0 && (!PAIR || leader)) {
            const long long t0 = clock64();
            int to = 0;
            for (int w = 0; w < 5; ++w) {
                to = max(to, sb->issued[w]);
                if (PAIR) to = max(to, ld_remote_s32(peer_addr(&sb->issued[w], 1u)));
            }
            for (int it = sb->consumed; it < to; ++it)
                while (!mbar_try_wait(smem_u32(&sb->full[it % STAGES]), (uint32_t)(it / STAGES) & 1u) &&
                       clock64() - t0 < kWaitCycles) {
                }
        }
        if (warp == 1 && lane == 0 && (!PAIR || leader)) {
            if constexpr (PAIR) umma_commit_pair_local(&sb->drain);
            else umma_commit(&sb->drain);
            const long long t0 = clock64();
            while (!mbar_try_wait(smem_u32(&sb->drain), 0) && clock64() - t0 < kWaitCycles) {
            }
        }
        __syncthreads();
    }
    if constexpr (PAIR || CL) cluster_sync_all();      // CL: shared memory is read by the others until here
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS) : "memory");
    }
}

// The partial sums of a split contraction in split order, then the epilogue
// (PART applied the FP8 scales): a thread takes eight columns of a row, its
// neighbours the block's other rows.
template <int EPI, bool GELU>
__global__ void ffn_join_kernel(const FfnParams p) {
    constexpr bool GLU = EPI == EPI_GLU;
    const int vec = p.N / 8, ld = GLU ? 2 * p.N : p.N;
    const int64_t next = part_size(p.M, ld), total = part_size(p.M, p.N) / 2;
    grid_dep_wait();
    grid_dep_launch_dependents();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t j = i >> 5, block = j / vec, row = block * 32 + (i & 31);
        const int c = (int)(j - block * vec) * 8;
        if (row >= p.M) continue;
        float f[8] = {}, g[8] = {};
        const float4* const at = p.part + part_at(ld, row, c);
        add_parts(f, at, p.splits, next);
        if (GLU) add_parts(g, at + (int64_t)p.N * 8, p.splits, next);
        finish8<EPI, false, GELU>(p, row, c, f, g);
    }
}

// MIXED: the tiles that several workers share, the shares in stage order.
template <int EPI, bool F8, bool GELU>
__global__ void ffn_join_mixed_kernel(const FfnParams p) {
    constexpr bool GLU = EPI == EPI_GLU;
    const int width = GLU ? p.bn / 2 : p.bn, vec = width / 8;
    const int64_t T = dealt_stages(p), next = part_size(2 * BM, p.bn);
    const int64_t total = (int64_t)(p.n_tiles * p.m_units - p.full) * (2 * BM) * vec;
    grid_dep_wait();
    grid_dep_launch_dependents();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        // lane: row within 32; then column group, row block, tile
        const int64_t j = i >> 5;
        const int v = (int)(j % vec), rb = (int)(j / vec % (2 * BM / 32)), tt = (int)(j / vec / (2 * BM / 32));
        const int first = deal_of(p, T, (int64_t)tt * p.kb);
        const int n = deal_of(p, T, (int64_t)(tt + 1) * p.kb - 1) - first + 1;
        int unit, nt;
        place(p, p.full + tt, unit, nt);
        const int ur = rb * 32 + (int)(i & 31), c = nt * width + v * 8;
        const int64_t row = (int64_t)unit * (2 * BM) + ur;
        if (n == 1 || row >= p.M || c >= p.N) continue;    // one worker: done there
        float f[8] = {}, g[8] = {};
        const float4* const at = p.part + (int64_t)tt * p.shares * next + part_at(p.bn, ur, v * 8);
        add_parts(f, at, n, next);
        if (GLU) add_parts(g, at + width * 8, n, next);
        finish8<EPI, F8, GELU>(p, row, c, f, g);
    }
}

// ---------------------------------------------------------------- host side

// [rows][cols] row-major operand; boxes of 128 bytes of a row x box_rows rows
// ld elements apart; rows and columns outside read as zero
bool operand_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows, bool f8) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t es = f8 ? 1 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * es};
    const cuuint32_t box[2] = {(cuuint32_t)(ROWB / es), (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return fn(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row pitch of the matrices this file keeps between products (a, [dg du]):
// whole 128-byte lines, or a row of a tile would touch five sectors for four
// (down projection of 16372 rows, f 6824: 478 us, on lines 400 us).
int64_t pitch(int64_t cols) { return (cols + 63) / 64 * 64; }

// How a product is cut: one CTA or a pair per tile, accumulator columns,
// splits of the contraction, bytes and number of the stages.
struct Plan {
    bool pair;
    int bn, m_units, n_tiles, kb, splits, a_bytes, b_bytes, stages;
    int dual;                   // two column tiles at once (n_tiles counts them as one)
    int full, dealt, shares;    // MIXED (dealt > 0)
    size_t part_bytes;
};

int resident_clusters(int num_sms, int size);

// M x N outputs (N: channels of GLU) over a contraction of kb stages: the cut
// with the least time by these rates (us; measured, see the header):
//   a stage   the larger of its MMAs, the ring's round trip over its stages,
//             and its bytes into one SM (full waves of pairs, several row units:
//             0.29 us at 64 columns, 0.32 at 128, 0.35 from 160 to 256)
//   all       the weights from HBM
//   a split, a share   the partial sums written and read back, and the join's
//             launch; in a cluster the exchange, and its clusters must all be
//             resident (a second wave took one row of d 1544, f 5656 from 24 to 32 us)
// Dealt stages are taken where they save a twentieth.  Not for one row unit,
// whose time is the weights' (256 rows, d 2560, f 10240: 55 us, with them 57),
// nor behind four waves (16384 rows 1666 us, with them 1706).
Plan search_plan(int num_sms, int64_t M, int64_t N, int kb, bool glu, bool dglu, bool amn, bool bmn) {
    Plan best{};
    double best_cost = 1e30;
    const bool pair = M > BM;
    const int workers = pair ? num_sms / 2 : num_sms;
    const int64_t cols = glu ? 2 * N : N;
    const int step = bmn ? (pair ? 128 : 64) : (pair ? 32 : 16);
    const int a_rows = !pair && !amn ? (int)(M + 7) / 8 * 8 : BM;
    const int64_t m_units = pair ? (M + 2 * BM - 1) / (2 * BM) : 1;
    int resident[MAX_CLUSTER + 1] = {};
    for (int k = 2; k <= MAX_CLUSTER && !pair; ++k) resident[k] = resident_clusters(num_sms, k);
    const int keep = pair ? (dglu ? IN_AREA : STAGING) : 0;      // the epilogue's end of the area
    for (int bn = MAX_BN; bn >= (bmn ? step : 64); bn -= step) {
        const int width = glu ? bn / 2 : bn;
        const int64_t n_tiles = (N + width - 1) / width;
        const int64_t tiles = m_units * n_tiles;
        const int a_bytes = a_rows * ROWB, b_bytes = (pair ? bn / 2 : bn) * ROWB;
        // the MMA reads 128 rows of A whatever was staged: the last stage's lie inside the ring too
        const int stages = std::min(MAX_STAGES, (TILE_AREA - keep - (A_BYTES - a_bytes)) / (a_bytes + b_bytes));
        const double bytes = (a_bytes + b_bytes) / 80e3;
        const double stage = std::max(std::max(0.365 * bn / 256, 1.4 / stages),
                                      m_units > 1 ? std::min(0.03 + bytes, 0.355) : bytes);
        for (int splits = 1; splits <= (pair ? 16 : MAX_CLUSTER) && splits * 4 <= std::max(kb, 4); ++splits) {
            if (splits > 1 && pair && tiles * (splits - 1) >= workers) break;
            if (splits > 1 && !pair && tiles > resident[splits]) continue;
            const int64_t waves = (tiles * splits + workers - 1) / workers;
            const double units = waves * ((kb + splits - 1) / splits) * stage, hbm = (double)kb * ROWB * cols / 6.4e6;
            double cost = std::max(units, hbm) + 0.2 * std::min(units, hbm);     // they overlap, but not wholly
            if (splits > 1)
                cost += pair ? 3.0 + (double)splits * M * cols * 8 / 6e6 : 0.7 + (double)M * (bn / 15e3 + 1 / 64.0);
            if (cost < best_cost * 0.98) {
                best_cost = cost;
                best = Plan{pair, bn, (int)m_units, (int)n_tiles, kb, splits, a_bytes, b_bytes, stages, 0, 0, 0, 0,
                            pair && splits > 1 ? align256((size_t)splits * part_size(M, (int)cols) * 16) : 0};
            }
        }
        // two column tiles at once, in one wave: A is read once for both; both epilogues come behind all MMAs (4 us)
        const int64_t twos = m_units * ((n_tiles + 1) / 2);
        if (glu && pair && n_tiles > 1 && twos <= workers) {
            const int ring = std::min(MAX_STAGES, (TILE_AREA - keep) / (a_bytes + 2 * b_bytes));
            const double units = kb * std::max(std::max(0.365 * bn / 128, 1.4 / ring), (a_bytes + 2 * b_bytes) / 80e3);
            const double hbm = (double)kb * ROWB * cols / 6.4e6;
            const double cost = std::max(units, hbm) + 0.2 * std::min(units, hbm) + 4.0;
            if (cost < best_cost * 0.98) {
                best_cost = cost;
                best = Plan{pair, bn, (int)m_units, (int)((n_tiles + 1) / 2), kb, 1, a_bytes, 2 * b_bytes, ring, 1, 0, 0, 0, 0};
            }
        }
        // whole waves, then the other tiles' stages dealt to all workers or to a few per tile
        const int64_t full = tiles / workers * workers, tail = tiles - full;
        for (int per_tile = 1; m_units > 1 && tail > 0 && full + tail < 4 * workers && per_tile <= 16; ++per_tile) {
            const int64_t dealt = per_tile == 1 ? workers : tail * per_tile;
            const int64_t total = tail * kb;
            if (dealt > workers || dealt <= tail || total < 4 * dealt) continue;
            const int64_t each = (total + dealt - 1) / dealt, shares = (kb + total / dealt - 1) / (total / dealt) + 1;
            const double units = ((double)(full / workers) * kb + each) * stage;
            // workers are at different stages: operands that L2 does not hold are read by each of them
            const bool shared = (double)kb * ROWB * (cols + M) < 1e8;
            const double hbm = (shared ? (double)kb * ROWB * cols : (double)total * 2 * (a_bytes + b_bytes)) / 6.4e6;
            const double cost = 1.05 * (std::max(units, hbm) + 0.2 * std::min(units, hbm) + 4.0 +
                                       (double)(dealt + tail) * std::min<int64_t>(M, 2 * BM) * bn * 8 / 6e6);
            if (cost < best_cost * 0.98) {
                best_cost = cost;
                best = Plan{pair, bn, (int)m_units, (int)n_tiles, kb, 1, a_bytes, b_bytes, stages, 0, (int)full, (int)dealt, (int)shares,
                            align256((size_t)tail * shares * 2 * BM * bn * 4)};
            }
        }
    }
    return best;
}

// The search takes about a microsecond and a call needs each of its plans
// three times: the last ones of this thread are kept, by their sizes.
Plan make_plan(const engram_ctx* c, int64_t M, int64_t N, int kb, bool glu, bool dglu, bool amn, bool bmn) {
    struct Entry {
        int64_t M = -1, N = 0;
        int kb = 0, num_sms = 0, kind = 0;
        Plan plan{};
    };
    constexpr int kEntries = 16;
    static thread_local Entry cache[kEntries];
    static thread_local int next = 0;
    const int kind = glu | amn << 1 | bmn << 2 | dglu << 3;
    for (const Entry& e : cache)
        if (e.M == M && e.N == N && e.kb == kb && e.num_sms == c->num_sms && e.kind == kind) return e.plan;
    Entry& e = cache[next];
    next = (next + 1) % kEntries;
    e.plan = search_plan(c->num_sms, M, N, kb, glu, dglu, amn, bmn);
    e.M = M;
    e.N = N;
    e.kb = kb;
    e.num_sms = c->num_sms;
    e.kind = kind;
    return e.plan;
}

// the kernel form that a cut takes
int form_of(const Plan& pl) {
    if (pl.splits > 1) return pl.pair ? SPLIT : CLUSTER;
    return pl.dual ? TWO_TILES : pl.dealt > 0 ? MIXED_TAIL : WHOLE;
}

// Clusters of `size` CTAs that the current device holds at once, at a CTA an SM
// (148 SMs in their partitions: 74 of 2, 45 of 3, 33 of 4, 26 of 5, 22 of 6, 15
// of 7 and of 8); the share of the SMs where it cannot be asked.
int resident_clusters(int num_sms, int size) {
    static std::mutex mu;
    static int known[64][MAX_CLUSTER + 1] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return num_sms * 4 / 5 / size;
    }
    std::lock_guard<std::mutex> lock(mu);
    int& n = known[dev][size];
    if (n == 0) {
        auto kernel = ffn_kernel<EPI_OUT, false, false, false, false, false, false, CLUSTER>;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = size;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(num_sms / size * size), 1, 1);
        cfg.blockDim = dim3(THREADS, 1, 1);
        cfg.dynamicSmemBytes = SMEM_BYTES;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = num_sms * 4 / 5 / size;
        }
    }
    return n;
}

template <int EPI, bool GLU, bool AMN, bool BMN, bool PAIR, bool F8, bool GELU, int MODE>
cudaError_t launch_one(const CUtensorMap& ma, const CUtensorMap& mb, const FfnParams& p, int num_sms, bool pdl,
                       cudaStream_t s) {
    auto kernel = ffn_kernel<EPI, GLU, AMN, BMN, PAIR, F8, GELU, MODE>;
    constexpr bool CL = MODE == CLUSTER;
    static std::mutex mu;
    static int max_units[64] = {};              // CTAs or pairs resident at once, per device
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 0;
    if (PAIR || CL) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = CL ? p.splits : 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
    }
    int cap = 0;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (max_units[dev] == 0) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
            if (e != cudaSuccess) return e;
            int mc = num_sms;
            if (PAIR) {
                cfg.gridDim = dim3((unsigned)(num_sms & ~1), 1, 1);
                if (cudaOccupancyMaxActiveClusters(&mc, kernel, &cfg) != cudaSuccess || mc < 1) {
                    cudaGetLastError();
                    mc = num_sms / 2;
                }
            }
            max_units[dev] = mc;
        }
        cap = max_units[dev];
    }
    const int64_t units = (int64_t)p.m_units * p.n_tiles * p.splits;
    if (units >= (int64_t)1 << 31) return cudaErrorInvalidValue;
    // CLUSTER: a unit each.  MIXED: every worker that stages are dealt to has to be there, resident at once or not
    const int64_t grid = MODE == MIXED_TAIL ? std::max<int64_t>(num_sms / 2, p.dealt) : CL ? units : std::min<int64_t>(units, cap);
    cfg.gridDim = dim3((unsigned)((PAIR ? 2 : 1) * grid), 1, 1);
    if (pdl) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, kernel, ma, mb, p);
}

// after: the kernel before on the stream is one of this call's, so this one
// may be its programmatic dependent (timed calls put events in between).
// One product: A [M][K] (or [K][M] with AMN), B [N][K] (or [K][N] with BMN;
// GLU: [2N][K]), and its epilogue, through partial sums when the plan splits.
// independent: it reads and writes nothing of the kernels before it in this
// call (it may run beside them, unless it needs the shared partial sums).
template <int EPI, bool AMN, bool BMN, bool F8 = false>
cudaError_t product(engram_ctx* c, const void* A, int64_t lda, const void* B, int64_t ldb, int64_t M, int64_t N, int64_t K,
                    FfnParams p, float4* part, const char* name, bool after, cudaStream_t s, bool independent = false) {
    constexpr bool GLU = EPI == EPI_GLU;
    const int kstep = F8 ? 128 : 64;
    const Plan pl = make_plan(c, M, N, (int)((K + kstep - 1) / kstep), GLU, EPI == EPI_DGLU, AMN, BMN);
    const bool pdl = after && !c->prof;
    p.M = (int)M;
    p.N = (int)N;
    p.kb = pl.kb;
    p.bn = pl.bn;
    p.n_tiles = pl.n_tiles;
    p.m_units = pl.m_units;
    p.splits = pl.splits;
    p.a_bytes = pl.a_bytes;
    p.b_bytes = pl.b_bytes;
    p.stages = pl.stages;
    p.raster = 8;
    p.late_wait = independent && pdl && pl.splits == 1 && pl.dealt == 0;
    p.full = pl.full;
    p.dealt = pl.dealt;
    p.shares = pl.shares;
    p.status = c->d_status;
    p.part = part;
    p.b_rows = pl.dual ? pl.bn : GLU || pl.pair ? pl.bn / 2 : pl.bn;
    // fp32 accumulator; formats bf16 (or E4M3: 0); MN-major bits; N / 8; M / 16
    p.idesc = (1u << 4) | (F8 ? 0u : (1u << 7) | (1u << 10)) | (AMN ? 1u << 15 : 0u) | (BMN ? 1u << 16 : 0u) |
              ((uint32_t)(pl.bn >> 3) << 17) | ((uint32_t)((pl.pair ? 256 : 128) >> 4) << 24);
    CUtensorMap ma, mb;
    const int64_t b_cols = GLU ? 2 * N : N;
    const bool ok = (AMN ? operand_map(&ma, A, K, M, lda, BK, F8) : operand_map(&ma, A, M, K, lda, pl.a_bytes / ROWB, F8)) &&
                    (BMN ? operand_map(&mb, B, K, b_cols, ldb, BK, F8) : operand_map(&mb, B, b_cols, K, ldb, p.b_rows, F8));
    if (!ok) return cudaErrorInvalidValue;
    prof_begin(c, s, name);
    cudaError_t e;
    constexpr bool ACT = EPI == EPI_GLU || EPI == EPI_DGLU;
    const bool gelu = ACT && p.act == ENGRAM_ACT_GELU;
    auto go = [&](auto pair, auto mode) {
        constexpr bool PAIR = decltype(pair)::value;
        constexpr int MODE = decltype(mode)::value;
        constexpr int E = MODE == SPLIT ? EPI_PART : EPI;
        return gelu && E == EPI ? launch_one<E, GLU, AMN, BMN, PAIR, F8, ACT && E == EPI, MODE>(ma, mb, p, c->num_sms, pdl, s)
                                : launch_one<E, GLU, AMN, BMN, PAIR, F8, false, MODE>(ma, mb, p, c->num_sms, pdl, s);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    switch (form_of(pl)) {
        case SPLIT: e = go(Yes{}, std::integral_constant<int, SPLIT>{}); break;
        case CLUSTER: e = go(No{}, std::integral_constant<int, CLUSTER>{}); break;
        case TWO_TILES: e = go(Yes{}, std::integral_constant<int, GLU ? TWO_TILES : WHOLE>{}); break;
        case MIXED_TAIL: e = go(Yes{}, std::integral_constant<int, MIXED_TAIL>{}); break;
        default: e = pl.pair ? go(Yes{}, std::integral_constant<int, WHOLE>{}) : go(No{}, std::integral_constant<int, WHOLE>{});
    }
    prof_end(c, s);
    if (e == cudaSuccess && pl.dealt > 0) {
        prof_begin(c, s, "ffn_join");
        const int64_t threads = ((int64_t)pl.n_tiles * pl.m_units - pl.full) * (2 * BM) * ((GLU ? pl.bn / 2 : pl.bn) / 8);
        const unsigned blocks = (unsigned)std::min<int64_t>((threads + 255) / 256, (int64_t)c->num_sms * 8);
        e = gelu ? launch_after(c, ffn_join_mixed_kernel<EPI, F8, ACT>, blocks, dim3(256), 0, s, p)
                 : launch_after(c, ffn_join_mixed_kernel<EPI, F8, false>, blocks, dim3(256), 0, s, p);
        prof_end(c, s);
    }
    if (e == cudaSuccess && pl.splits > 1 && pl.pair) {
        prof_begin(c, s, "ffn_join");
        const int64_t threads = part_size(M, (int)N) / 2;
        const unsigned blocks = (unsigned)std::min<int64_t>((threads + 255) / 256, (int64_t)c->num_sms * 8);
        e = gelu ? launch_after(c, ffn_join_kernel<EPI, ACT>, blocks, dim3(256), 0, s, p)
                 : launch_after(c, ffn_join_kernel<EPI, false>, blocks, dim3(256), 0, s, p);
        prof_end(c, s);
    }
    return e;
}

// What the forward keeps for the backward: the two planes of g and u, and
// a = act(g) u as the down projection read it.
struct Saved {
    __nv_bfloat16* a;       // [n][f], rows pitch(f) apart
    uint4* hi;              // [ceil(n / 32)][2f / 8][32]
    uint2* lo;
    size_t bytes;
};

Saved saved_of(const void* base, int64_t n, int64_t f) {
    char* p = static_cast<char*>(const_cast<void*>(base));
    const int64_t elems = (n + 31) / 32 * 32 * (f / 4);
    const int64_t a_bytes = n * pitch(f) * 2;
    return Saved{reinterpret_cast<__nv_bfloat16*>(p), reinterpret_cast<uint4*>(p + a_bytes),
                 reinterpret_cast<uint2*>(p + a_bytes + elems * 16), (size_t)(a_bytes + elems * 24)};
}

// Scratch: the products' shared partial sums, then the intermediate matrix
// (forward: a [n][f], unless it is saved; backward: dg and du [n][2f]).
struct FfnWs {
    float4* part;
    __nv_bfloat16* mid;
    size_t bytes;
};

// The products of a call, in the order that engram_debug_ffn_cut numbers them.
enum { GATE_UP, DOWN, D_GATE_UP, D_WD, D_X, D_WGU, PRODUCTS };

Plan plan_of(const engram_ctx* c, int64_t n, int64_t f, int product) {
    const int64_t d = c->cfg.hidden;
    const int k8 = c->cfg.dtype == ENGRAM_FP8 && product == GATE_UP ? 128 : 64;
    auto kb = [&](int64_t K) { return (int)((K + k8 - 1) / k8); };
    switch (product) {
        case GATE_UP: return make_plan(c, n, f, kb(d), true, false, false, false);
        case DOWN: return make_plan(c, n, d, kb(f), false, false, false, false);
        case D_GATE_UP: return make_plan(c, n, f, kb(d), false, true, false, true);
        case D_WD: return make_plan(c, d, f, kb(n), false, false, true, true);
        case D_X: return make_plan(c, n, d, kb(2 * f), false, false, false, true);
        default: return make_plan(c, 2 * f, d, kb(n), false, false, true, true);
    }
}

FfnWs ffn_carve(const engram_ctx* c, void* base, int64_t n, int64_t f, bool grad) {
    size_t part = 0;
    for (int k = grad ? D_GATE_UP : GATE_UP; k < (grad ? PRODUCTS : D_GATE_UP); ++k)
        part = std::max(part, plan_of(c, n, f, k).part_bytes);
    FfnWs w{};
    char* p = static_cast<char*>(base);
    auto take = [&](size_t bytes) {
        char* q = p;
        p += align256(bytes);
        return q;
    };
    w.part = reinterpret_cast<float4*>(take(part));
    w.mid = reinterpret_cast<__nv_bfloat16*>(take((size_t)n * pitch(grad ? 2 * f : f) * 2));
    w.bytes = (size_t)(p - static_cast<char*>(base));
    return w;
}

constexpr int32_t kMaxFfnWidth = 1 << 20;

engram_status ffn_shape(const engram_ctx* c, int64_t n, int32_t f, int32_t act, bool grad) {
    if (!c) return inval("null context");
    if (n < 0 || n >= (int64_t)1 << 31) return inval("the row count must be in [0, 2^31)");
    if (f < 8 || f % 8 != 0 || f > kMaxFfnWidth) return inval("f must be a multiple of 8 in [8, 2^20]");
    if (act != ENGRAM_ACT_SILU && act != ENGRAM_ACT_GELU) return inval("unknown activation");
    if (c->cfg.dtype == ENGRAM_F32 || (grad && c->cfg.dtype != ENGRAM_BF16)) {
        set_error(grad ? "the feed-forward backward takes bf16 contexts" : "the feed-forward block runs on the tensor cores (bf16 or FP8)");
        return ENGRAM_E_UNSUPPORTED;
    }
    if (!c->sm100) {
        set_error("the feed-forward block needs an sm_100 device");
        return ENGRAM_E_UNSUPPORTED;
    }
    return ENGRAM_OK;
}

engram_status check_ws(const void* workspace, size_t have, size_t need) {
    if (!workspace) return inval("null workspace");
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return inval("workspace must be 256-byte aligned");
    if (have < need) {
        set_error("the workspace is smaller than the call needs");
        return ENGRAM_E_NOMEM;
    }
    return ENGRAM_OK;
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" {

int32_t engram_debug_ffn_cut(const engram_ctx* c, int64_t n, int32_t f, int32_t product) {
    if (product < 0 || product >= PRODUCTS || n < 1 ||
        ffn_shape(c, n, f, ENGRAM_ACT_SILU, product >= D_GATE_UP) != ENGRAM_OK)
        return -1;
    const Plan pl = plan_of(c, n, f, product);
    return form_of(pl) * 2 + (pl.pair ? 1 : 0);
}

size_t engram_ffn_workspace_bytes(const engram_ctx* c, int64_t n, int32_t f) {
    if (ffn_shape(c, n, f, ENGRAM_ACT_SILU, false) != ENGRAM_OK) return 0;
    return ffn_carve(c, nullptr, std::max<int64_t>(1, n), f, false).bytes;
}

engram_status engram_ffn(engram_ctx* c, const void* x, const float* x_scale, int64_t n, int32_t f, int32_t act,
                         const void* Wgu, const float* gu_scale, const void* Wd, const void* res, void* y, void* saved,
                         void* workspace, size_t workspace_bytes, cudaStream_t s) {
    engram_status st = ffn_shape(c, n, f, act, false);
    if (st != ENGRAM_OK) return st;
    const bool f8 = c->cfg.dtype == ENGRAM_FP8;
    if (f8 && saved) return inval("saved is for the backward, which takes bf16 contexts");
    if (n == 0) return ENGRAM_OK;
    if (!x || !Wgu || !Wd || !y) return inval("null tensor pointer");
    if (f8 ? (!x_scale || !gu_scale) : (x_scale || gu_scale))
        return inval("x_scale and gu_scale go with ENGRAM_FP8, and are required there");
    if (!aligned16(x) || !aligned16(Wgu) || !aligned16(Wd) || !aligned16(res) || !aligned16(y) || !aligned16(saved) ||
        !aligned16(gu_scale))
        return inval("x, Wgu, gu_scale, Wd, res, y and saved must be 16-byte aligned");
    const FfnWs w = ffn_carve(c, workspace, n, f, false);
    st = check_ws(workspace, workspace_bytes, w.bytes);
    if (st == ENGRAM_OK) st = check_device(c);
    if (st != ENGRAM_OK) return st;
    prof_reset(c);
    const int64_t d = c->cfg.hidden;
    FfnParams p{};
    p.act = act;
    p.out = w.mid;
    p.ldo = pitch(f);
    if (saved) {
        const Saved sv = saved_of(saved, n, f);
        p.out = sv.a;
        p.gu_hi = sv.hi;
        p.gu_lo = sv.lo;
    }
    p.row_scale = x_scale;
    p.col_scale = gu_scale;
    p.stall = c->debug_stall;
    c->debug_stall = 0;
    cudaError_t e = f8 ? product<EPI_GLU, false, false, true>(c, x, d, Wgu, d, n, f, d, p, w.part, "ffn_gate_up_fp8", false, s)
                       : product<EPI_GLU, false, false>(c, x, d, Wgu, d, n, f, d, p, w.part, "ffn_gate_up", false, s);
    if (e != cudaSuccess) return cuda_fail("feed-forward gate/up launch", e);
    FfnParams o{};
    o.out = static_cast<__nv_bfloat16*>(y);
    o.ldo = d;
    o.res = static_cast<const __nv_bfloat16*>(res);
    e = product<EPI_OUT, false, false>(c, p.out, p.ldo, Wd, f, n, d, f, o, w.part, "ffn_down", true, s);
    return e == cudaSuccess ? ENGRAM_OK : cuda_fail("feed-forward down launch", e);
}

size_t engram_ffn_grad_workspace_bytes(const engram_ctx* c, int64_t n, int32_t f) {
    if (ffn_shape(c, n, f, ENGRAM_ACT_SILU, true) != ENGRAM_OK) return 0;
    return ffn_carve(c, nullptr, std::max<int64_t>(1, n), f, true).bytes;
}

size_t engram_ffn_saved_bytes(const engram_ctx* c, int64_t n, int32_t f) {
    if (ffn_shape(c, n, f, ENGRAM_ACT_SILU, true) != ENGRAM_OK) return 0;
    return saved_of(nullptr, n, f).bytes;
}

engram_status engram_ffn_grad(engram_ctx* c, const void* d_y, const void* x, const void* saved, int64_t n, int32_t f,
                              int32_t act, const void* Wgu, const void* Wd, void* d_x, void* d_Wgu, void* d_Wd,
                              void* workspace, size_t workspace_bytes, cudaStream_t s) {
    engram_status st = ffn_shape(c, n, f, act, true);
    if (st != ENGRAM_OK) return st;
    if (!d_Wgu || !d_Wd) return inval("null weight gradient");
    if (n > 0 && (!d_y || !x || !saved || !Wgu || !Wd || !d_x)) return inval("null tensor pointer");
    if (!aligned16(d_y) || !aligned16(x) || !aligned16(saved) || !aligned16(Wgu) || !aligned16(Wd) || !aligned16(d_x) ||
        !aligned16(d_Wgu) || !aligned16(d_Wd))
        return inval("tensors must be 16-byte aligned");
    FfnWs w{};
    if (n > 0) {
        w = ffn_carve(c, workspace, n, f, true);
        st = check_ws(workspace, workspace_bytes, w.bytes);
        if (st != ENGRAM_OK) return st;
    }
    st = check_device(c);
    if (st != ENGRAM_OK) return st;
    prof_reset(c);
    const int64_t d = c->cfg.hidden;
    if (n == 0) {
        cudaError_t e = cudaMemsetAsync(d_Wgu, 0, (size_t)2 * f * d * 2, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(d_Wd, 0, (size_t)f * d * 2, s);
        return e == cudaSuccess ? ENGRAM_OK : cuda_fail("clearing the weight gradients", e);
    }
    FfnParams p{};
    p.act = act;
    const Saved sv = saved_of(saved, n, f);
    p.out = w.mid;
    p.ldo = pitch(2 * (int64_t)f);
    p.gu_hi = sv.hi;
    p.gu_lo = sv.lo;
    cudaError_t e = product<EPI_DGLU, false, true>(c, d_y, d, Wd, f, n, f, d, p, w.part, "ffn_d_gate_up", false, s);
    // d_Wd needs neither dg nor du: its tiles fill the SMs that d_gate_up leaves
    FfnParams o{};
    if (e == cudaSuccess) {
        o.out = static_cast<__nv_bfloat16*>(d_Wd);
        o.ldo = f;
        e = product<EPI_OUT, true, true>(c, d_y, d, sv.a, pitch(f), d, f, n, o, w.part, "ffn_d_Wd", true, s, true);
    }
    if (e == cudaSuccess) {
        o.out = static_cast<__nv_bfloat16*>(d_x);
        o.ldo = d;
        e = product<EPI_OUT, false, true>(c, w.mid, p.ldo, Wgu, d, n, d, 2 * (int64_t)f, o, w.part, "ffn_d_x", true, s);
    }
    if (e == cudaSuccess) {
        o.out = static_cast<__nv_bfloat16*>(d_Wgu);
        e = product<EPI_OUT, true, true>(c, w.mid, p.ldo, x, d, 2 * (int64_t)f, d, n, o, w.part, "ffn_d_Wgu", true, s);
    }
    return e == cudaSuccess ? ENGRAM_OK : cuda_fail("feed-forward backward launches", e);
}

}  // extern "C"

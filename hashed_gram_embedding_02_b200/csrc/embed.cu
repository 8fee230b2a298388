// Token embedding of the hidden states and its gradient.
//
//   forward    h[i] = scale * E[tok_i]                     (fp32 product, one rounding)
//   gradient   dE[v] = scale * sum_{i : tok_i = v} dh[i]   (fp32 sums)
//
// Both move rows and compute next to nothing: the forward is bound by the
// bytes of the rows read and written, the gradient by dh and dE.
//
// The gradient sorts the tokens first, so that every sum runs over a
// contiguous list in increasing position and no float atomics are needed:
//   1. sort (token, position) by token, stable: least significant digit
//      first, kDigitBits per pass.  A pass cuts the list into at most
//      kMaxSortCtas contiguous parts; part p's digit counts are in
//      hist[p][digit]; its CTA sums the counts of the parts before it and
//      scatters its elements in order.  The counts of the next pass are made
//      by the scatter of this one.  At most kSortSmall positions are sorted
//      by one CTA in shared memory instead.
//   2. reduce: a piece is `piece` consecutive sorted entries, all columns.
//      A run of equal tokens that lies inside a piece is summed and stored; a
//      run cut by a piece's edge leaves its part's sum in `part`.  Work is
//      the same for every piece however often a token occurs, so a token that
//      takes half of the batch costs nothing extra.
//   3. join: the parts of each cut run, in order.
// Between 1 and 2 the rows of the tokens that do not occur are cleared (a small
// dE is cleared whole by the sort's first launch).
// The order of a token's sum is fixed by its positions and by where its run lies
// among the pieces, whose length depends on the row count and the SMs (piece_of).
// The launches behind the first are programmatic dependents of one another: each waits at its start
// for the one before, which hides most of its launch.
#include <algorithm>

#include "ctx.cuh"
#include "tc.cuh"

namespace engram {
namespace {

// ---------------------------------------------------------------- row geometry

// Threads of a CTA over rows of `cpr` 16-byte chunks: TPR threads per row
// (whole warps, or a power of two below a warp), RB rows side by side.
struct RowGeo {
    int tpr, rb;
};

RowGeo row_geo(int cpr) {
    RowGeo g{};
    if (cpr >= 32) {
        g.tpr = std::min(512, (cpr + 31) / 32 * 32);
        // two equal rounds rather than one full and one short
        if (cpr > 512) {
            const int rounds = (cpr + 511) / 512;
            g.tpr = ((cpr + rounds - 1) / rounds + 31) / 32 * 32;
        }
    } else {
        g.tpr = 1;
        while (g.tpr < cpr) g.tpr <<= 1;
    }
    g.rb = std::min(128, std::max(1, 256 / g.tpr));   // 128 long pieces: 34 KB of keys and positions
    return g;
}

// position i of the call -> its token (rows are sequence-major)
struct TokSource {
    const int32_t* tok;
    int64_t stride;
    int32_t t_begin, L, V;
    __device__ __forceinline__ int32_t at(int64_t i) const {
        const uint32_t b = (uint32_t)i / (uint32_t)L;      // i < 2^31
        return __ldg(tok + b * stride + t_begin + ((uint32_t)i - b * (uint32_t)L));
    }
};

// ---------------------------------------------------------------- forward

// Short calls: a row per thread row, nothing before its token's load.
template <typename T>
__global__ void embed_short_kernel(TokSource src, int64_t n, const T* __restrict__ E, float scale, T* __restrict__ h,
                                   int cpr, uint32_t* status) {
    constexpr int EPC = Vec<T>::N;
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= n) return;
    const int32_t v = src.at(row);
    const bool ok = v >= 0 && v < src.V;
    if (!ok && threadIdx.x == 0) flag(status, ENGRAM_ERR_TOKEN);
    for (int c = threadIdx.x; c < cpr; c += blockDim.x) {
        const uint4 q = ok ? __ldg(reinterpret_cast<const uint4*>(E) + (int64_t)v * cpr + c) : make_uint4(0, 0, 0, 0);
        float f[EPC];
        Vec<T>::load(reinterpret_cast<const T*>(&q), f);
#pragma unroll
        for (int k = 0; k < EPC; ++k) f[k] *= scale;
        Vec<T>::store(h + (row * cpr + c) * EPC, f);
    }
}

// Persistent: a CTA takes blockDim.y * kEmbedRows rows at a time, gridDim.x
// groups of rows apart.  The tokens of its next kTokBuf rows are read first (a
// row's address is then a shared-memory read away), and the next group of rows
// is in flight while one is stored.  8 x 4096 x 2560 bf16: 42 us, 5.0 TB/s (45 us
// with each group's tokens loaded a group ahead; 30 against 43 us when the rows
// come from the caches), four rows in flight or more CTAs 41 to 48 us.
constexpr int kEmbedRows = 2;
constexpr int kTokBuf = 256;

template <typename T>
__global__ void embed_kernel(TokSource src, int64_t n, const T* __restrict__ E, float scale, T* __restrict__ h,
                             int cpr, uint32_t* status) {
    constexpr int EPC = Vec<T>::N, RPT = kEmbedRows;
    __shared__ int32_t s_tok[kTokBuf];
    const int rows_cta = blockDim.y * RPT, tid = threadIdx.y * blockDim.x + threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * rows_cta;
    const int per_batch = kTokBuf / rows_cta;              // groups whose tokens fit (rows_cta <= kTokBuf)
    for (int64_t g0 = (int64_t)blockIdx.x * rows_cta; g0 < n; g0 += step * per_batch) {
        __syncthreads();
        for (int j = tid; j < per_batch * rows_cta; j += blockDim.x * blockDim.y) {
            const int64_t row = g0 + j / rows_cta * step + j % rows_cta;
            int32_t v = -1;
            if (row < n) {
                v = src.at(row);
                if (v < 0 || v >= src.V) {
                    v = -1;
                    flag(status, ENGRAM_ERR_TOKEN);
                }
            }
            s_tok[j] = v;
        }
        __syncthreads();
        const int64_t left = (n - g0 + step - 1) / step;
        const int groups = (int)min((int64_t)per_batch, left);
        for (int c = threadIdx.x; c < cpr; c += blockDim.x) {
            uint4 q[RPT];
            auto fetch = [&](int g) {
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    const int32_t v = g < groups ? s_tok[g * rows_cta + threadIdx.y * RPT + r] : -1;
                    q[r] = v >= 0 ? __ldg(reinterpret_cast<const uint4*>(E) + (int64_t)v * cpr + c) : make_uint4(0, 0, 0, 0);
                }
            };
            fetch(0);
            for (int g = 0; g < groups; ++g) {
                const int64_t row = g0 + g * step + threadIdx.y * RPT;
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    if (row + r < n) {
                        float f[EPC];
                        Vec<T>::load(reinterpret_cast<const T*>(&q[r]), f);
#pragma unroll
                        for (int k = 0; k < EPC; ++k) f[k] *= scale;
                        Vec<T>::store(h + ((row + r) * cpr + c) * EPC, f);
                    }
                }
                fetch(g + 1);
            }
        }
    }
}

template <typename T>
cudaError_t launch_embed(const TokSource& src, int64_t n, const void* E, float scale, void* h, int d, int num_sms,
                         uint32_t* status, cudaStream_t s) {
    const int cpr = d / Vec<T>::N;
    const RowGeo g = row_geo(cpr);
    const dim3 block(g.tpr, g.rb);
    const int per_sm = std::max(1, 1280 / (g.tpr * g.rb));
    const int64_t ctas = (int64_t)num_sms * per_sm, per = (int64_t)g.rb * kEmbedRows;
    if (n < ctas * per)       // less than a group for every CTA
        embed_short_kernel<T><<<(unsigned)((n + g.rb - 1) / g.rb), block, 0, s>>>(src, n, static_cast<const T*>(E), scale,
                                                                                  static_cast<T*>(h), cpr, status);
    else
        embed_kernel<T><<<(unsigned)ctas, block, 0, s>>>(src, n, static_cast<const T*>(E), scale, static_cast<T*>(h), cpr, status);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- sort

constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortIpt = 4;                                // elements per thread and tile
constexpr int kSortTile = kSortThreads * kSortIpt;
constexpr int kMaxSortCtas = 256;
constexpr int kSmallThreads = 512;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kSmallIpt = 4;                               // at most, elements per thread
// One CTA sorts 2048 positions in 6 us less than the launches of several (15
// against 21 us a call); with 16 elements a thread it takes 31 to 37 us for 8192.
constexpr int kSortSmall = kSmallThreads * kSmallIpt;
constexpr size_t small_smem(int ipt) { return (size_t)kSmallThreads * ipt * 6 + kSmallWarps * kDigits * 2; }
constexpr int64_t kMaxEmbedRows = (int64_t)1 << 24;
// Gradients of at most this many bytes are cleared whole: clearing 64 MB takes
// 9 us, the bitmap and a launch of their own cost as much (256 rows, V 4096, d
// 256: 20 us a call with them, 17 us without).
constexpr int64_t kClearWhole = (int64_t)64 << 20;

// A small gradient is cleared whole by the extra CTAs of the sort's first
// launch, ahead of the sums in the stream.
struct Zero {
    float4* to;
    int64_t vecs;
    // CTA k of `of`
    __device__ __forceinline__ void run(unsigned k, unsigned of) const {
        for (int64_t i = (int64_t)k * blockDim.x + threadIdx.x; i < vecs; i += (int64_t)of * blockDim.x)
            to[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
};

// tokens outside [0, V) sort behind all others as V
__device__ __forceinline__ uint32_t sort_key(const TokSource& src, int64_t i, uint32_t* status) {
    const int32_t v = src.at(i);
    if (v >= 0 && v < src.V) return (uint32_t)v;
    flag(status, ENGRAM_ERR_TOKEN);
    return (uint32_t)src.V;
}

// Rank of the warp's 32 elements among the earlier ones of the warp with the
// same digit: cnt[digit] is the count so far; one lane per digit adds to it.
__device__ __forceinline__ uint32_t warp_rank(uint32_t digit, bool live, uint32_t* cnt, int lane) {
    const uint32_t mask = __match_any_sync(0xffffffffu, live ? digit : 0xffffffffu);
    const uint32_t before = __popc(mask & ((1u << lane) - 1u));
    const uint32_t had = live ? cnt[digit] : 0u;
    __syncwarp();
    if (live && before == 0) cnt[digit] = had + __popc(mask);
    __syncwarp();
    return had + before;
}

// The keys, the first digit's counts of each part, and the bitmap of the
// tokens that occur (cleared before; null: not wanted).
__global__ void embed_keys_kernel(TokSource src, int64_t n, int64_t per, uint32_t* __restrict__ keys,
                                  uint32_t* __restrict__ pos, uint32_t* __restrict__ hist, uint32_t* touched,
                                  unsigned parts, Zero zero, uint32_t* status) {
    __shared__ uint32_t s_hist[kDigits];
    if (blockIdx.x >= parts) {
        zero.run(blockIdx.x - parts, gridDim.x - parts);
        return;
    }
    for (int k = threadIdx.x; k < kDigits; k += blockDim.x) s_hist[k] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * per, hi = min(n, lo + per);
    for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) {
        const uint32_t k = sort_key(src, i, status);
        keys[i] = k;
        pos[i] = (uint32_t)i;
        atomicAdd(&s_hist[k & (kDigits - 1)], 1u);
        if (touched) atomicOr(touched + (k >> 5), 1u << (k & 31));
    }
    __syncthreads();
    for (int k = threadIdx.x; k < kDigits; k += blockDim.x) hist[(int64_t)blockIdx.x * kDigits + k] = s_hist[k];
}

// One pass: stable scatter by the digit at `shift`.  hist_next (nullable,
// cleared before): counts of the next digit per part of the output.
__global__ void __launch_bounds__(kSortThreads)
embed_scatter_kernel(const uint32_t* keys, const uint32_t* pos, int64_t n, int64_t per, int shift, const uint32_t* hist,
                     uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out, uint32_t* hist_next) {
    __shared__ uint32_t s_base[kDigits];                   // where this part's next element of a digit goes
    __shared__ uint32_t s_cnt[kSortWarps][kDigits];
    __shared__ uint32_t s_scan[kSortWarps];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int parts = gridDim.x, me = blockIdx.x;
    // two digits per thread: totals, and the counts of the parts before this one
    uint32_t tot[2] = {0, 0}, mine[2] = {0, 0};
    for (int p = 0; p < parts; ++p) {
        const uint2 v = *(reinterpret_cast<const uint2*>(hist + (int64_t)p * kDigits) + tid);
        tot[0] += v.x;
        tot[1] += v.y;
        if (p < me) {
            mine[0] += v.x;
            mine[1] += v.y;
        }
    }
    uint32_t inc = tot[0] + tot[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    uint32_t base = inc - tot[0] - tot[1];
    for (int w = 0; w < warp; ++w) base += s_scan[w];
    s_base[2 * tid] = base + mine[0];
    s_base[2 * tid + 1] = base + tot[0] + mine[1];
    const int64_t lo = me * per, hi = min(n, lo + per);
    for (int64_t t0 = lo; t0 < hi; t0 += kSortTile) {
        __syncthreads();
        for (int k = tid; k < kSortWarps * kDigits; k += kSortThreads) (&s_cnt[0][0])[k] = 0;
        __syncthreads();
        uint32_t key[kSortIpt], ps[kSortIpt], rank[kSortIpt];
        const int64_t w0 = t0 + warp * (32 * kSortIpt);    // a warp's elements are contiguous
#pragma unroll
        for (int k = 0; k < kSortIpt; ++k) {
            const int64_t i = w0 + k * 32 + lane;
            key[k] = i < hi ? keys[i] : 0u;
            ps[k] = i < hi ? pos[i] : 0u;
        }
#pragma unroll
        for (int k = 0; k < kSortIpt; ++k)
            rank[k] = warp_rank((key[k] >> shift) & (kDigits - 1), w0 + k * 32 + lane < hi, s_cnt[warp], lane);
        __syncthreads();
        // counts of the warps -> the offset of each warp's first element of a digit
        for (int g = tid; g < kDigits; g += kSortThreads) {
            uint32_t run = s_base[g];
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t x = s_cnt[w][g];
                s_cnt[w][g] = run;
                run += x;
            }
            s_base[g] = run;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSortIpt; ++k) {
            const int64_t i = w0 + k * 32 + lane;
            if (i < hi) {
                const uint32_t to = s_cnt[warp][(key[k] >> shift) & (kDigits - 1)] + rank[k];
                keys_out[to] = key[k];
                pos_out[to] = ps[k];
                if (hist_next)
                    atomicAdd(hist_next + (to / per) * kDigits + ((key[k] >> (shift + kDigitBits)) & (kDigits - 1)),
                              1u);
            }
        }
    }
}

// At most kSmallThreads * IPT positions: all passes in one CTA's shared memory.
template <int IPT>
__global__ void __launch_bounds__(kSmallThreads)
embed_sort_small_kernel(TokSource src, int n, int passes, uint32_t* __restrict__ keys_out,
                        uint32_t* __restrict__ pos_out, uint32_t* touched, int64_t touched_words, uint32_t* count,
                        Zero zero, uint32_t* status) {
    if (blockIdx.x > 0) {
        zero.run(blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    extern __shared__ uint32_t s_key[];
    uint16_t* const s_pos = reinterpret_cast<uint16_t*>(s_key + kSmallThreads * IPT);
    uint16_t(*const s_cnt)[kDigits] = reinterpret_cast<uint16_t(*)[kDigits]>(s_pos + kSmallThreads * IPT);
    __shared__ uint32_t s_scan[kSmallWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int64_t k = tid; k < touched_words; k += kSmallThreads) touched[k] = 0;
    if (tid == 0) *count = 0;
    uint32_t key[IPT], ps[IPT], rank[IPT];
    const int w0 = warp * (32 * IPT);
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const int i = w0 + k * 32 + lane;
        key[k] = i < n ? sort_key(src, i, status) : 0u;
        ps[k] = (uint32_t)i;
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = p * kDigitBits;
        __syncthreads();
        for (int k = tid; k < kSmallWarps * kDigits; k += kSmallThreads) (&s_cnt[0][0])[k] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < IPT; ++k) {
            const bool live = w0 + k * 32 + lane < n;
            const uint32_t digit = (key[k] >> shift) & (kDigits - 1);
            const uint32_t mask = __match_any_sync(0xffffffffu, live ? digit : 0xffffffffu);
            const uint32_t before = __popc(mask & ((1u << lane) - 1u));
            const uint32_t had = live ? s_cnt[warp][digit] : 0u;
            __syncwarp();
            if (live && before == 0) s_cnt[warp][digit] = (uint16_t)(had + __popc(mask));
            __syncwarp();
            rank[k] = had + before;
        }
        __syncthreads();
        // one digit per thread: its total, the scan over digits, then the warps' offsets
        uint32_t tot = 0;
        for (int w = 0; w < kSmallWarps; ++w) tot += s_cnt[w][tid];
        uint32_t inc = tot;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        uint32_t run = inc - tot;
        for (int w = 0; w < warp; ++w) run += s_scan[w];
        for (int w = 0; w < kSmallWarps; ++w) {
            const uint32_t x = s_cnt[w][tid];
            s_cnt[w][tid] = (uint16_t)run;
            run += x;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < IPT; ++k) {
            if (w0 + k * 32 + lane < n) {
                const uint32_t to = s_cnt[warp][(key[k] >> shift) & (kDigits - 1)] + rank[k];
                s_key[to] = key[k];
                s_pos[to] = (uint16_t)ps[k];
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < IPT; ++k) {
            const int i = w0 + k * 32 + lane;
            if (i < n) {
                key[k] = s_key[i];
                ps[k] = s_pos[i];
            }
        }
    }
    // the bitmap was cleared above by this CTA alone; the barriers of the passes order the two
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const int i = w0 + k * 32 + lane;
        if (i < n) {
            keys_out[i] = key[k];
            pos_out[i] = ps[k];
            if (touched) atomicOr(touched + (key[k] >> 5), 1u << (key[k] & 31));
        }
    }
}

// ---------------------------------------------------------------- reduce

constexpr int kPieceLong = 32;    // sorted entries per piece
constexpr int kPieceShort = 8;    // few positions: more pieces in flight
constexpr int kAhead = 8;         // rows of dh in flight per thread

struct EmbedGrad {
    const uint32_t* keys;
    const uint32_t* pos;
    int64_t n;
    int64_t n_pieces;
    uint32_t V;
    int d;
    float scale;
    bool wide;                    // rows of dE are 32-byte aligned (d is a multiple of 8)
    float* d_E;
    float* part;                  // [n_pieces][2][d]: a piece's first run when it began earlier, its last when it goes on
    uint4* cut;                   // runs that a piece's edge cuts: piece where it begins, pieces it reaches, token
    uint32_t* count;
};

// EPC floats of a row.  A thread's eight go out as one 32-byte store where
// the rows are aligned for it: as two of 16 bytes, each warp store would fill
// half of its sectors.
template <int EPC>
__device__ __forceinline__ void store_row(float* to, const float* f, bool wide) {
    if (EPC == 8 && wide) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(f[0]), "f"(f[1]), "f"(f[2]),
                     "f"(f[3]), "f"(f[EPC - 4]), "f"(f[EPC - 3]), "f"(f[EPC - 2]), "f"(f[EPC - 1])
                     : "memory");
        return;
    }
#pragma unroll
    for (int k = 0; k < EPC; k += 4) *reinterpret_cast<float4*>(to + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
}

template <int EPC>
__device__ __forceinline__ void put_row(float* to, const float* f, float scale, bool accumulate, bool wide) {
    float o[EPC];
#pragma unroll
    for (int k = 0; k < EPC; ++k) o[k] = scale * f[k];
    if (accumulate) {
#pragma unroll
        for (int k = 0; k < EPC; k += 4) {
            const float4 was = *reinterpret_cast<const float4*>(to + k);
            o[k] += was.x; o[k + 1] += was.y; o[k + 2] += was.z; o[k + 3] += was.w;
        }
    }
    store_row<EPC>(to, o, wide);
}

// The rows of dE whose token does not occur, 32 of them (a word of the bitmap)
// to a CTA, a warp to a row.  V rows of d floats are most of what the gradient
// writes (8 x 4096 tokens, V 128000, d 2560: 173 us, 7.1 TB/s; CTAs that loop
// over the words reach 197 us, and clearing in the launch of the sums or on a
// side stream starves the sums: 316 and 292 us for a call, so 276 us).
constexpr int kFillThreads = 512;

__global__ void __launch_bounds__(kFillThreads) embed_fill_kernel(const uint32_t* touched, uint32_t V, int d,
                                                                  float* __restrict__ d_E) {
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t w = blockIdx.x, bits = touched[w];
    for (uint32_t r = warp; r < 32 && w * 32 + r < V; r += kFillThreads / 32) {
        if ((bits >> r) & 1u) continue;
        float4* row = reinterpret_cast<float4*>(d_E + (int64_t)(w * 32 + r) * d);
        for (int c = lane; c < d / 4; c += 32) row[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

template <typename T, int PIECE, bool ACC>
__global__ void embed_reduce_kernel(EmbedGrad p, const T* __restrict__ dh) {
    constexpr int EPC = Vec<T>::N;
    extern __shared__ uint32_t s_mem[];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int cpr = p.d / EPC;
    const int64_t piece = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    // keys of the piece with one neighbour on each side (kNone outside the list), and its positions
    constexpr uint32_t kNone = 0xffffffffu;
    uint32_t* s_key = s_mem + threadIdx.y * (2 * PIECE + 2);
    uint32_t* s_pos = s_key + PIECE + 2;
    const int64_t i0 = piece * PIECE;
    for (int k = threadIdx.x; k < PIECE + 2; k += blockDim.x) {
        const int64_t i = i0 + k - 1;
        s_key[k] = i >= 0 && i < p.n ? p.keys[i] : kNone;
        if (k > 0 && k <= PIECE) s_pos[k - 1] = i < p.n ? p.pos[i] : 0u;
    }
    __syncthreads();
    if (i0 >= p.n) return;
    const int len = (int)min((int64_t)PIECE, p.n - i0);
    const bool enters = s_key[0] == s_key[1];                    // the first run began before this piece
    const bool leaves = s_key[len] == s_key[len + 1];            // the last run goes on behind it
    if (threadIdx.x == 0 && leaves && s_key[len] < p.V && !(enters && s_key[1] == s_key[len])) {
        // the first piece behind this one that does not begin with the run's token: most runs reach one
        // piece further, so the step doubles from there before the search halves it
        const uint32_t key = s_key[len];
        int64_t lo = piece + 1, hi = piece + 2, step = 1;
        while (hi < p.n_pieces && p.keys[hi * PIECE] == key) {
            lo = hi;
            hi += step;
            step <<= 1;
        }
        hi = min(hi, p.n_pieces);
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (p.keys[mid * PIECE] == key) lo = mid;
            else hi = mid;
        }
        p.cut[atomicAdd(p.count, 1u)] = make_uint4((uint32_t)piece, (uint32_t)(hi - piece), key, 0u);
    }
    float* part = p.part + piece * 2 * p.d;
    for (int c = threadIdx.x; c < cpr; c += blockDim.x) {
        float acc[EPC];
#pragma unroll
        for (int k = 0; k < EPC; ++k) acc[k] = 0.f;
        const uint4* from = reinterpret_cast<const uint4*>(dh) + c;
        bool first = true;
#pragma unroll 1
        for (int e0 = 0; e0 < len; e0 += kAhead) {
            uint4 q[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
                q[a] = e0 + a < len ? __ldg(from + (int64_t)s_pos[e0 + a] * cpr) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int e = e0 + a;
                if (e >= len) break;
                float f[EPC];
                Vec<T>::load(reinterpret_cast<const T*>(&q[a]), f);
#pragma unroll
                for (int k = 0; k < EPC; ++k) acc[k] += f[k];
                const uint32_t key = s_key[e + 1];
                if (e + 1 == len || s_key[e + 2] != key) {
                    // the end of a run, or of the piece
                    if (key < p.V) {
                        if (first && enters) store_row<EPC>(part + c * EPC, acc, true);
                        else if (e + 1 == len && leaves) store_row<EPC>(part + p.d + c * EPC, acc, true);
                        else put_row<EPC>(p.d_E + (int64_t)key * p.d + c * EPC, acc, p.scale, ACC, p.wide);
                    }
#pragma unroll
                    for (int k = 0; k < EPC; ++k) acc[k] = 0.f;
                    first = false;
                }
            }
        }
    }
}

// The cut runs: a CTA takes 4 * `lanes` columns of one run; its 256 / lanes
// groups of threads sum consecutive shares of the run's parts, which are then
// added in order.  Narrow rows leave more groups (a token that takes 38 % of
// 6732 positions, d 96: 39 us with two groups, 13 us with eight).
constexpr int kJoinThreads = 256;

template <int PIECE, bool ACC>
__global__ void __launch_bounds__(kJoinThreads) embed_join_kernel(EmbedGrad p, int lanes) {
    __shared__ float4 s_sum[kJoinThreads];
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int t = threadIdx.x % lanes, group = threadIdx.x / lanes, groups = kJoinThreads / lanes;
    const int slices = (p.d + 4 * lanes - 1) / (4 * lanes);
    const int64_t work = (int64_t)*p.count * slices;
    for (int64_t u = blockIdx.x; u < work; u += gridDim.x) {
        const uint4 run = p.cut[u / slices];
        const int64_t p0 = run.x, m = run.y;               // parts: p0's last run, then the first runs of m - 1 pieces
        const int col = ((int)(u % slices) * lanes + t) * 4;
        const int64_t per = (m + groups - 1) / groups, a = group * per, b = min(m, a + per);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col < p.d) {
#pragma unroll 8
            for (int64_t k = a; k < b; ++k) {
                const float4 x = *reinterpret_cast<const float4*>(p.part + (p0 + k) * 2 * p.d + (k == 0 ? p.d : 0) + col);
                acc.x += x.x;
                acc.y += x.y;
                acc.z += x.z;
                acc.w += x.w;
            }
        }
        s_sum[threadIdx.x] = acc;
        __syncthreads();
        if (group == 0 && col < p.d) {
            for (int g = 1; g < groups && g * per < m; ++g) {
                const float4 x = s_sum[g * lanes + t];
                acc.x += x.x;
                acc.y += x.y;
                acc.z += x.z;
                acc.w += x.w;
            }
            const float f[4] = {acc.x, acc.y, acc.z, acc.w};
            put_row<4>(p.d_E + (int64_t)run.z * p.d + col, f, p.scale, ACC, false);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host side

int sort_passes(int32_t V) {
    int bits = 0;
    while (((int64_t)1 << bits) <= V) ++bits;              // keys 0 .. V
    return (bits + kDigitBits - 1) / kDigitBits;
}

int64_t sort_part(int64_t n) {
    const int64_t parts = std::min<int64_t>(kMaxSortCtas, (n + kSortTile - 1) / kSortTile);
    return (n + parts - 1) / parts;
}

int piece_of(int64_t n, int num_sms) { return n >= (int64_t)kPieceLong * num_sms * 4 ? kPieceLong : kPieceShort; }

struct EmbedWs {
    uint32_t* keys[2];
    uint32_t* pos[2];
    uint32_t* hist[2];
    uint32_t* touched;
    uint32_t* count;
    uint4* cut;
    float* part;
    void* clear;
    size_t clear_bytes[2];      // with the bitmap, and without
    int64_t hist_words, touched_words, n_pieces;
    int piece;
    size_t bytes;
};

EmbedWs embed_carve(const engram_ctx* c, void* base, int64_t n) {
    EmbedWs w{};
    char* p = static_cast<char*>(base);
    auto take = [&](size_t bytes) {
        char* q = p;
        p += align256(bytes);
        return q;
    };
    for (int k = 0; k < 2; ++k) {
        w.keys[k] = reinterpret_cast<uint32_t*>(take((size_t)n * 4));
        w.pos[k] = reinterpret_cast<uint32_t*>(take((size_t)n * 4));
    }
    if (n > kSortSmall) {
        const int64_t per = sort_part(n);
        w.hist_words = (n + per - 1) / per * kDigits;
        w.hist[0] = reinterpret_cast<uint32_t*>(take((size_t)w.hist_words * 4));
    }
    // one clear covers the second pass's counts, the run count and the bitmap
    char* const cleared = p;
    if (n > kSortSmall) w.hist[1] = reinterpret_cast<uint32_t*>(take((size_t)w.hist_words * 4));
    w.count = reinterpret_cast<uint32_t*>(take(4));
    const size_t no_map = (size_t)(p - cleared);
    w.touched_words = ((int64_t)c->cfg.vocab + 1 + 31) / 32;
    w.touched = reinterpret_cast<uint32_t*>(take((size_t)w.touched_words * 4));
    w.clear = cleared;
    w.clear_bytes[0] = (size_t)(p - cleared);
    w.clear_bytes[1] = no_map;
    w.piece = piece_of(n, c->num_sms);
    w.n_pieces = (n + w.piece - 1) / w.piece;
    w.cut = reinterpret_cast<uint4*>(take((size_t)w.n_pieces * 16));
    w.part = reinterpret_cast<float*>(take((size_t)w.n_pieces * 2 * c->cfg.hidden * 4));
    w.bytes = (size_t)(p - static_cast<char*>(base));
    return w;
}

template <typename T, int PIECE, bool ACC>
cudaError_t launch_reduce(const engram_ctx* c, const EmbedGrad& p, const void* dh, cudaStream_t s) {
    const RowGeo g = row_geo(p.d / Vec<T>::N);
    const dim3 block(g.tpr, g.rb);
    const unsigned pieces = (unsigned)((p.n_pieces + g.rb - 1) / g.rb);
    const size_t smem = (size_t)g.rb * (2 * PIECE + 2) * 4;
    return launch_after(c, embed_reduce_kernel<T, PIECE, ACC>, pieces, block, smem, s, p, static_cast<const T*>(dh));
}

template <int PIECE, bool ACC>
cudaError_t reduce_and_join(engram_ctx* c, const EmbedGrad& p, const void* dh, cudaStream_t s) {
    prof_begin(c, s, "embed_reduce");
    cudaError_t e = c->hs == 2 ? launch_reduce<__nv_bfloat16, PIECE, ACC>(c, p, dh, s)
                               : launch_reduce<float, PIECE, ACC>(c, p, dh, s);
    prof_end(c, s);
    if (e != cudaSuccess || p.n_pieces < 2) return e;
    prof_begin(c, s, "embed_join");
    int lanes = 1;
    while (lanes < 64 && lanes * 4 < p.d) lanes <<= 1;
    const int slices = (p.d + 4 * lanes - 1) / (4 * lanes);
    const unsigned blocks = (unsigned)std::min<int64_t>(p.n_pieces * slices, (int64_t)c->num_sms * 8);
    e = launch_after(c, embed_join_kernel<PIECE, ACC>, blocks, dim3(kJoinThreads), 0, s, p, lanes);
    prof_end(c, s);
    return e;
}

engram_status check_tokens(const engram_ctx* c, int32_t B, int32_t T, int64_t tok_stride, int32_t t_begin,
                           float scale) {
    engram_status st = check_forward_args(c, B, T, tok_stride, t_begin);
    if (st != ENGRAM_OK) return st;
    if (!(scale - scale == 0.f)) return inval("scale must be finite");
    return ENGRAM_OK;
}

}  // namespace
}  // namespace engram

using namespace engram;

extern "C" {

engram_status engram_embed(engram_ctx* c, const int32_t* tok, int32_t B, int32_t T, int64_t tok_stride,
                           int32_t t_begin, const void* E, float scale, void* h, cudaStream_t s) {
    engram_status st = check_tokens(c, B, T, tok_stride, t_begin, scale);
    if (st != ENGRAM_OK) return st;
    const int64_t n = (int64_t)B * (T - t_begin);
    if (n == 0) return ENGRAM_OK;
    if (n >= (int64_t)1 << 31) return inval("B * (T - t_begin) must be below 2^31");
    if (!tok || !E || !h) return inval("null tensor pointer");
    if (!aligned16(E) || !aligned16(h)) return inval("E and h must be 16-byte aligned");
    st = check_device(c);
    if (st != ENGRAM_OK) return st;
    prof_reset(c);
    const TokSource src{tok, tok_stride, t_begin, T - t_begin, c->cfg.vocab};
    prof_begin(c, s, "embed");
    cudaError_t e = c->hs == 2
                        ? launch_embed<__nv_bfloat16>(src, n, E, scale, h, c->cfg.hidden, c->num_sms, c->d_status, s)
                        : launch_embed<float>(src, n, E, scale, h, c->cfg.hidden, c->num_sms, c->d_status, s);
    prof_end(c, s);
    return e == cudaSuccess ? ENGRAM_OK : cuda_fail("embedding launch", e);
}

size_t engram_embed_grad_workspace_bytes(const engram_ctx* c, int64_t n_tok) {
    if (!c || n_tok < 0 || n_tok > kMaxEmbedRows) return 0;
    return embed_carve(c, nullptr, std::max<int64_t>(1, n_tok)).bytes;
}

engram_status engram_embed_grad(engram_ctx* c, const int32_t* tok, int32_t B, int32_t T, int64_t tok_stride,
                                int32_t t_begin, const void* d_h, float scale, float* d_E, int32_t accumulate,
                                void* workspace, size_t workspace_bytes, cudaStream_t s) {
    engram_status st = check_tokens(c, B, T, tok_stride, t_begin, scale);
    if (st != ENGRAM_OK) return st;
    const int64_t n = (int64_t)B * (T - t_begin);
    if (n > kMaxEmbedRows) return inval("B * (T - t_begin) must be at most 2^24");
    if (!d_E) return inval("null gradient pointer");
    if (n > 0 && (!tok || !d_h || !workspace)) return inval("null tensor pointer");
    if (!aligned16(d_h) || !aligned16(d_E)) return inval("d_h and d_E must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return inval("workspace must be 256-byte aligned");
    if (n > 0 && workspace_bytes < embed_carve(c, nullptr, n).bytes) {
        set_error("engram_embed_grad: the workspace is smaller than engram_embed_grad_workspace_bytes");
        return ENGRAM_E_NOMEM;
    }
    st = check_device(c);
    if (st != ENGRAM_OK) return st;
    prof_reset(c);
    const int64_t V = c->cfg.vocab;
    const int d = c->cfg.hidden;
    if (n == 0) {
        if (accumulate) return ENGRAM_OK;
        cudaError_t e = cudaMemsetAsync(d_E, 0, (size_t)V * d * 4, s);
        return e == cudaSuccess ? ENGRAM_OK : cuda_fail("clearing the embedding gradient", e);
    }
    EmbedWs w = embed_carve(c, workspace, n);
    const TokSource src{tok, tok_stride, t_begin, T - t_begin, c->cfg.vocab};
    const int passes = sort_passes(c->cfg.vocab);
    // what is not summed is cleared: a small dE whole, by the sort's launch; of a large one the rows of the
    // tokens that do not occur
    const bool whole = !accumulate && V * d * 4 <= kClearWhole, rest = !accumulate && !whole;
    const Zero zero{reinterpret_cast<float4*>(d_E), whole ? V * d / 4 : 0};
    const unsigned zero_ctas = whole ? (unsigned)std::min<int64_t>((zero.vecs + kSortThreads - 1) / kSortThreads, (int64_t)c->num_sms * 4) : 0;
    uint32_t* touched = rest ? w.touched : nullptr;
    const int64_t touched_words = rest ? w.touched_words : 0;
    int at = 0;
    cudaError_t e = cudaSuccess;
    prof_begin(c, s, "embed_sort");
    if (n <= kSortSmall) {
        auto go = [&](auto kern, int ipt) {
            kern<<<1 + zero_ctas, kSmallThreads, small_smem(ipt), s>>>(src, (int)n, passes, w.keys[0], w.pos[0], touched,
                                                                       touched_words, w.count, zero, c->d_status);
        };
        if (n <= kSmallThreads) go(embed_sort_small_kernel<1>, 1);
        else go(embed_sort_small_kernel<kSmallIpt>, kSmallIpt);
    } else {
        const int64_t per = sort_part(n);
        const unsigned parts = (unsigned)((n + per - 1) / per);
        e = cudaMemsetAsync(w.clear, 0, w.clear_bytes[rest ? 0 : 1], s);
        if (e == cudaSuccess)
            embed_keys_kernel<<<parts + zero_ctas, kSortThreads, 0, s>>>(src, n, per, w.keys[0], w.pos[0], w.hist[0], touched,
                                                                         parts, zero, c->d_status);
        for (int p = 0; p < passes && e == cudaSuccess; ++p) {
            const bool last = p + 1 == passes;
            // the counts of pass p + 1 go where those of pass p - 1 were
            if (p > 0 && !last) e = cudaMemsetAsync(w.hist[at ^ 1], 0, (size_t)w.hist_words * 4, s);
            if (e != cudaSuccess) break;
            // the third pass on follows a clear, not a kernel
            auto args = [&](auto&& go) {
                return go(w.keys[at], w.pos[at], n, per, p * kDigitBits, w.hist[at], w.keys[at ^ 1], w.pos[at ^ 1],
                          last ? nullptr : w.hist[at ^ 1]);
            };
            const bool plain = p > 0 && !last;
            e = args([&](auto... a) {
                if (!plain) return launch_after(c, embed_scatter_kernel, parts, dim3(kSortThreads), 0, s, a...);
                embed_scatter_kernel<<<parts, kSortThreads, 0, s>>>(a...);
                return cudaGetLastError();
            });
            if (e != cudaSuccess) break;
            at ^= 1;
        }
    }
    prof_end(c, s);
    if (rest && e == cudaSuccess) {
        prof_begin(c, s, "embed_fill");
        const unsigned blocks = (unsigned)((V + 31) / 32);
        e = launch_after(c, embed_fill_kernel, blocks, dim3(kFillThreads), 0, s, w.touched, (uint32_t)V, d, d_E);
        prof_end(c, s);
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail("embedding gradient sort launches", e);
    const EmbedGrad p{w.keys[at], w.pos[at], n, w.n_pieces, (uint32_t)V, d, scale,
                      (reinterpret_cast<uintptr_t>(d_E) & 31u) == 0, d_E, w.part, w.cut, w.count};
    if (w.piece == kPieceLong)
        e = accumulate ? reduce_and_join<kPieceLong, true>(c, p, d_h, s) : reduce_and_join<kPieceLong, false>(c, p, d_h, s);
    else
        e = accumulate ? reduce_and_join<kPieceShort, true>(c, p, d_h, s) : reduce_and_join<kPieceShort, false>(c, p, d_h, s);
    return e == cudaSuccess ? ENGRAM_OK : cuda_fail("embedding gradient launches", e);
}

}  // extern "C"

// token_dispatch.hip -- tokens sorted by expert: a stable counting sort of
// the slots t * k + j by their expert and the token rows in that order.
//
// The slots are cut into chunks of whole tokens (about kChunkSlots slots).
//   1. one workgroup per chunk counts its slots per expert;
//   2. with many chunks, one workgroup turns the counts into each chunk's
//      first position per expert (and writes counts and offsets);
//   3. workgroups of a few tokens each count the slots of their chunk that
//      come before them, place their own, and copy their rows: a token's
//      row is read once and written to its places.
// With few counts step 3 sums them itself, every workgroup all of them, in
// place of step 2's launch of one workgroup; by their number times a chunk's
// workgroups (8 places a token, rows of 1024, summed and scanned, us: 16384
// slots of 256 experts 19.6, 21.6; 32768 of 128 27.6, 32.1; 65536 of 64 43.5,
// 51.6; beyond the bound 16384 of 512 24.1, 22.2; 65536 of 128 57.6, 52.4, of
// 1024 272, 58; one place, order alone: 16384 of 64 13.4, 14.2, of 256 18.8,
// 15.4).  Up to kOneLaunchSlots slots it counts the slots themselves: the
// call is then one launch without workspace.
// Positions are integers counted in slot order: the result does not depend
// on which workgroup runs when.
// Bound by the rows' bytes, each read once and written to its k places: 4096
// rows of 7168 bf16 to 8 places each 115 us, 4.6 TB/s, of which the counts are
// 5 (writes alone reach 6.9 TB/s, a copy 5.0 to 5.5; one workgroup per place,
// reading its row again, 154 us).  9 tokens: one launch, 5.8 us.
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunkSlots = 1024;
constexpr int kMaxChunks = 2048;
constexpr int kOneLaunchSlots = 4096;
constexpr int64_t kSumWork = 1 << 19;  // counts times workgroups of a chunk
constexpr int kMaxTokSlots = 64;  // slots of one gather workgroup, at least one token

struct Plan {
    int chunk_tok, chunks;  // tokens per chunk, number of chunks
    int wg_tok, wgs;        // tokens per gather workgroup, workgroups per chunk
    bool one;               // one launch
    bool sums;              // the last launch sums the chunks' counts
};

// where place_rows_kernel gets the positions before its own chunk from
enum class First { kSlots, kCounts, kScanned };

Plan make_plan(int64_t T, int E, int k) {
    Plan p;
    const int64_t S = T * k;
    p.one = S <= kOneLaunchSlots;
    int64_t slots = (S + kMaxChunks - 1) / kMaxChunks;
    if (slots < kChunkSlots) slots = kChunkSlots;
    p.chunk_tok = p.one ? (int)T : (int)((slots + k - 1) / k);
    p.chunks = (int)((T + p.chunk_tok - 1) / p.chunk_tok);
    // one token a workgroup (4096 tokens to 8 places each: 115 us, 117 with
    // four, 121 with eight); of long chunks, which every workgroup recounts, a
    // fair share
    p.wg_tok = p.chunk_tok / 256 > 1 ? p.chunk_tok / 256 : 1;
    if (p.wg_tok * k > kMaxTokSlots) p.wg_tok = kMaxTokSlots / k;
    p.wgs = (p.chunk_tok + p.wg_tok - 1) / p.wg_tok;
    p.sums = !p.one && (int64_t)p.chunks * E * p.wgs <= kSumWork;
    return p;
}

__device__ inline bool held(int e, int E) { return (unsigned)e < (unsigned)E; }

__global__ void __launch_bounds__(kThreads)
chunk_count_kernel(const int32_t* ids, int64_t S, int chunk_slots, int E, int32_t* hist) {
    __shared__ int cnt[kMaxExperts];
    for (int e = threadIdx.x; e < E; e += kThreads) cnt[e] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * chunk_slots;
    const int64_t s1 = s0 + chunk_slots < S ? s0 + chunk_slots : S;
    for (int64_t s = s0 + threadIdx.x; s < s1; s += kThreads) {
        const int e = ids[s];
        if (held(e, E)) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) hist[(int64_t)blockIdx.x * E + e] = cnt[e];
}

// exclusive prefix sum of v over the kThreads threads of a workgroup; total in *sum
template <int THREADS>
__device__ inline int block_scan(int v, int* wave_sum, int* total) {
    const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
    int inc = v;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == kWave - 1) wave_sum[w] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / kWave; i++) {
        if (i < w) before += wave_sum[i];
        all += wave_sum[i];
    }
    *total = all;
    return before + inc - v;
}

// hist[c][e] -> first position of chunk c's slots of expert e; counts, offsets
__global__ void __launch_bounds__(1024)
chunk_scan_kernel(int32_t* hist, int chunks, int E, int32_t* counts, int32_t* offsets) {
    __shared__ int wave_sum[16];
    const int e = threadIdx.x;
    int n = 0;
    if (e < E)
        for (int c = 0; c < chunks; c++) n += hist[(int64_t)c * E + e];
    int total;
    int at = block_scan<1024>(n, wave_sum, &total);
    if (e < E) {
        if (counts) counts[e] = n;
        offsets[e] = at;
        if (e == E - 1) offsets[E] = total;
        for (int c = 0; c < chunks; c++) {
            const int h = hist[(int64_t)c * E + e];
            hist[(int64_t)c * E + e] = at;
            at += h;
        }
    }
}

// the bytes of one row copied to each of its places (4 loads of V in flight
// per thread before the first store; V a vector type of the compiler's, whose
// copies stay whole: with the uint4 structure 147 us for 4096 tokens, not 115)
template <typename V>
__device__ inline void copy_row(const uint8_t* src, uint8_t* dst, int64_t row_bytes, const int* place, int k) {
    constexpr int kBatch = 4;
    const int n = (int)(row_bytes / (int)sizeof(V));
    for (int i0 = threadIdx.x; i0 < n; i0 += kBatch * kThreads) {
        V v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; u++) v[u] = reinterpret_cast<const V*>(src)[min(i0 + u * kThreads, n - 1)];
        for (int j = 0; j < k; j++) {
            if (place[j] < 0) continue;
            V* d = reinterpret_cast<V*>(dst + place[j] * row_bytes);
#pragma unroll
            for (int u = 0; u < kBatch; u++) {
                if (i0 + u * kThreads >= n) break;
                d[i0 + u * kThreads] = v[u];
            }
        }
    }
}

__device__ inline void copy_rows(const uint8_t* src, uint8_t* dst, int64_t row_bytes, const int* place, int k,
                                 int vec) {
    if (vec == 16) copy_row<u32x4_t>(src, dst, row_bytes, place, k);
    else if (vec == 4) copy_row<uint32_t>(src, dst, row_bytes, place, k);
    else if (vec == 2) copy_row<uint16_t>(src, dst, row_bytes, place, k);
    else copy_row<uint8_t>(src, dst, row_bytes, place, k);
}

template <First FROM>
__global__ void __launch_bounds__(kThreads)
place_rows_kernel(moe_dispatch_args a, Plan p, const int32_t* first, int64_t row_bytes, int64_t x_row_bytes, int vec,
                  int scale_bytes, int scale_vec) {
    constexpr bool kAll = FROM != First::kScanned;   // the offsets are formed here
    __shared__ int before[kMaxExperts];              // slots of the expert ahead of this workgroup's
    __shared__ int all[kAll ? kMaxExperts : 1];
    __shared__ int own[kMaxTokSlots], place[kMaxTokSlots];
    __shared__ int wave_sum[kThreads / kWave];
    const int E = (int)a.num_experts, k = a.top_k, tid = threadIdx.x;
    const int chunk = blockIdx.x / p.wgs, wg = blockIdx.x % p.wgs;
    const int64_t c0 = (int64_t)chunk * p.chunk_tok;
    const int64_t t0 = c0 + (int64_t)wg * p.wg_tok;
    int64_t t1 = t0 + p.wg_tok;
    if (t1 > c0 + p.chunk_tok) t1 = c0 + p.chunk_tok;
    if (t1 > a.num_tokens) t1 = a.num_tokens;
    if (t0 >= t1) return;
    for (int e = tid; e < E; e += kThreads) {
        before[e] = kAll ? 0 : first[(int64_t)chunk * E + e];
        if (kAll) all[e] = 0;
    }
    const int n = (int)(t1 - t0) * k;
    if (tid < n) own[tid] = a.ids[t0 * k + tid];
    __syncthreads();
    if (FROM == First::kCounts) {
        const int cells = p.chunks * E;
        for (int i0 = tid; i0 < cells; i0 += 8 * kThreads) {
            int h[8];
#pragma unroll
            for (int u = 0; u < 8; u++) h[u] = i0 + u * kThreads < cells ? first[i0 + u * kThreads] : 0;
#pragma unroll
            for (int u = 0; u < 8; u++) {
                if (h[u] == 0) continue;
                const int c = (i0 + u * kThreads) / E, e = i0 + u * kThreads - c * E;
                atomicAdd(&all[e], h[u]);
                if (c < chunk) atomicAdd(&before[e], h[u]);
            }
        }
    }
    const int64_t send = FROM == First::kSlots ? a.num_tokens * k : t0 * k;
    for (int64_t s = c0 * k + tid; s < send; s += kThreads) {
        const int e = a.ids[s];
        if (!held(e, E)) continue;
        if (s < t0 * k) atomicAdd(&before[e], 1);
        if (FROM == First::kSlots) atomicAdd(&all[e], 1);
    }
    __syncthreads();
    if (kAll) {  // four experts per thread: the offsets of all of them
        int v[4], sum = 0, total;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = 4 * tid + i < E ? all[4 * tid + i] : 0;
            sum += v[i];
        }
        int at = block_scan<kThreads>(sum, wave_sum, &total);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int e = 4 * tid + i;
            if (e < E) {
                before[e] += at;
                if (blockIdx.x == 0) {
                    if (a.counts) a.counts[e] = v[i];
                    a.offsets[e] = at;
                    if (e == E - 1) a.offsets[E] = total;
                }
            }
            at += v[i];
        }
        __syncthreads();
    }
    if (tid < n) {
        const int e = own[tid];
        int at = -1;
        if (held(e, E)) {
            at = before[e];
            for (int i = 0; i < tid; i++) at += own[i] == e;
            if (a.sorted) a.sorted[at] = (int32_t)(t0 * k + tid);
        }
        place[tid] = at;
        a.pos[t0 * k + tid] = at;
    }
    if (!a.rows) return;
    __syncthreads();
    for (int64_t t = t0; t < t1; t++) {
        const int* pl = place + (t - t0) * k;
        copy_rows((const uint8_t*)a.x + t * x_row_bytes, (uint8_t*)a.rows, row_bytes, pl, k, vec);
        if (a.row_scales)
            copy_rows(a.x_scales + t * scale_bytes, a.row_scales, scale_bytes, pl, k, scale_vec);
    }
}

__global__ void __launch_bounds__(kThreads) no_slots_kernel(int E, int32_t* counts, int32_t* offsets) {
    for (int e = threadIdx.x; e <= E; e += kThreads) {
        offsets[e] = 0;
        if (counts && e < E) counts[e] = 0;
    }
}

// bytes a copy may move at once: the largest of 16, 4, 2, 1 that divides
// every row start
int copy_bytes(const void* p, const void* q, int64_t row, int64_t stride) {
    const uint64_t m = (uint64_t)(uintptr_t)p | (uint64_t)(uintptr_t)q | (uint64_t)row | (uint64_t)stride;
    return m % 16 == 0 ? 16 : m % 4 == 0 ? 4 : m % 2 == 0 ? 2 : 1;
}

}  // namespace

int64_t dispatch_workspace(int64_t T, int64_t E, int32_t k) {
    if (T == 0) return 0;
    const Plan p = make_plan(T, (int)E, k);
    return p.one ? 0 : (int64_t)p.chunks * E * 4;
}

hipError_t launch_dispatch(const moe_dispatch_args& a, hipStream_t stream) {
    const int E = (int)a.num_experts, k = a.top_k;
    if (a.num_tokens == 0) {
        no_slots_kernel<<<1, kThreads, 0, stream>>>(E, a.counts, a.offsets);
        return hipGetLastError();
    }
    const Plan p = make_plan(a.num_tokens, E, k);
    const int64_t esize = a.dtype == MOE_DT_BF16 ? 2 : a.dtype == MOE_DT_F32 ? 4 : 1;
    const int64_t row = a.hidden * esize, xrow = a.x_stride * esize;
    const int vec = copy_bytes(a.x, a.rows, row, xrow);
    const int srow = a.row_scales ? (int)(a.hidden / 32) : 0;
    const int svec = copy_bytes(a.x_scales, a.row_scales, srow, srow);
    const unsigned grid = (unsigned)(p.chunks * (int64_t)p.wgs);
    if (p.one) {
        place_rows_kernel<First::kSlots><<<grid, kThreads, 0, stream>>>(a, p, nullptr, row, xrow, vec, srow, svec);
        return hipGetLastError();
    }
    int32_t* hist = (int32_t*)a.workspace;
    chunk_count_kernel<<<p.chunks, kThreads, 0, stream>>>(a.ids, a.num_tokens * k, p.chunk_tok * k, E, hist);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (p.sums) {
        place_rows_kernel<First::kCounts><<<grid, kThreads, 0, stream>>>(a, p, hist, row, xrow, vec, srow, svec);
        return hipGetLastError();
    }
    chunk_scan_kernel<<<1, 1024, 0, stream>>>(hist, p.chunks, E, a.counts, a.offsets);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    place_rows_kernel<First::kScanned><<<grid, kThreads, 0, stream>>>(a, p, hist, row, xrow, vec, srow, svec);
    return hipGetLastError();
}

}  // namespace moe

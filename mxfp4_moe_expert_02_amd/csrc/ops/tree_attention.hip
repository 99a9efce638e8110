// tree_attention.hip -- attention of drafted tokens over the MXFP8 cache.
//
// The rows of one key/value head of a sequence are its drafted tokens times
// the query heads that share it; a workgroup takes 16, 32, 64 or 128 of them (a
// row tile) over a run of positions.  Its waves are WR groups of 16 R rows
// times WK that share the positions out, 32 at a time (a tile); each keeps a result of
// its own (m, sum, O), joined at the end of the run.  Per tile a wave computes
//
//   S^T = K Q^T           A = K, decoded from its codes in LDS, B = Q
//   P^T = 2^(c S^T - c m)
//   O^T += V^T P^T        A = V^T (bf16 in LDS), B = P^T: the lanes and
//                         registers that S^T came in, as bf16
//
// with v_mfma_f32_16x16x32_bf16.  Lane (c, g) = (l % 16, l / 16).  K's lane
// (c, g) holds quarter g of position c's elements, one contiguous run and its
// scale; the inner axis is then in another order than the elements', and Q is
// loaded in the same one.  Of the 32 positions of O's inner axis a lane of P^T
// holds 4g .. 4g+3 and 16 + 4g .. ; V^T comes in that order out of
// ds_read_b64_tr_b16, which hands a lane 4 rows of a column.  The sum of the
// weights is one more product, with ones in V's place: the sum of the weights
// as they were rounded to bf16, in float32.  (bf16 for K, P and V: E4M3 times a
// power of two is exact in bf16, and P's rounding, off by at most 2^-8 of a
// weight, is that of the output.)
//
// m is a row's running maximum, but it is moved only where a score passes it
// by more than 8 powers of two (P then stays below 2^8), so that most steps
// neither exchange maxima nor rescale O.
//
// Work is cut by units of 128 positions, all row tiles' units in one line, an
// equal run of them to each workgroup: ragged lengths cost nothing.  A row tile
// that one workgroup does whole is finished there; else its parts go to the
// workspace in float32 and tree_attention_join_kernel adds them in order.
//
// With few rows the cache's bytes bound it: 32 sequences of 9 tokens and 56
// heads (8 of keys) over up to 16384 positions of 128 elements take 178 us, 4.1 TB/s;
// 64 of 1 token over up to 8000 of 64 elements 77 us, 4.4 TB/s.  With
// many it is the waves' own work: 8 trees of up to 64 tokens over up to 16001
// positions take 141 us, 577 TFLOP/s.  Per tile a wave has 34 matrix
// instructions (544 cycles), 16 exponentials (256), 88 other vector instructions
// (350) and 65 scalar ones; the two waves of a SIMD take 2700 cycles for a
// tile each: they overlap little of it (the matrix cores are busy 26 %).
#include "attention_internal.h"

namespace moe {
namespace {

constexpr float kAttnSlack = 8.f;  // powers of two that a score may pass m by

struct AttnArgs {
    moe_tree_attention_args a;
    int T, B, G;               // tokens, sequences, query heads per key/value head
    uint32_t g_inverse;        // 2^32 / G, rounded up (G > 1)
    int page_shift, capacity;  // positions of a page (log2), of a sequence's table
    int groups;                // workgroups
    float c;                   // scale * log2 e
    int64_t part_floats;       // of one partial result
};

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));

// x / G for x < 2^16
__device__ inline int by_group(const AttnArgs& p, int x) {
    return p.G == 1 ? x : (int)__umulhi((uint32_t)x, p.g_inverse);
}

__device__ inline float minus_inf() { return -__builtin_inff(); }

// ----------------------------------------------------------- the line of units

// A sequence as the device holds it: its first token, its tokens, committed
// positions and all positions (lengths out of range taken as the header says)
struct Seq {
    int first, n, L, len;
};
__device__ inline Seq read_seq(const AttnArgs& p, int b) {
    Seq s;
    const int first = p.a.token_offsets[b], next = p.a.token_offsets[b + 1], L = p.a.context_lens[b];
    s.first = first;
    s.n = next - first;
    s.L = min(max(L, 0), p.capacity);
    s.len = min(s.L + s.n, p.capacity);
    return s;
}
template <int ROWS>
__device__ inline int tiles_of(const AttnArgs& p, const Seq& s) {
    return (s.n * p.G + ROWS - 1) / ROWS;
}
__device__ inline int units_of(const Seq& s) { return max(1, (s.len + kAttnUnit - 1) / kAttnUnit); }
// its row tiles, of all heads
template <int ROWS>
__device__ inline int items_of(const AttnArgs& p, const Seq& s) {
    return s.n ? tiles_of<ROWS>(p, s) * p.a.cache.kv_heads : 0;
}

// inclusive sums over the wave's lanes
__device__ inline int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);  // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);  // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);  // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31
    return v;
}

// All units in one line: sequence by sequence, in each its heads, in each head
// its row tiles, in each of them its units.  Every wave works the line out
// for itself, 64 sequences at a time, one a lane (the lengths are the device's).
// A workgroup does `per` units of the line.  A run that goes over the end of a
// row tile costs about as much as 4 units (its queries, the first load, the
// join): where it lets each row tile start a run of its own by at most 3 more
// units a run, the line is laid out so, each row tile's units rounded up to
// whole runs (1 sequence of 9 tokens over 8192 positions: 27 -> 20 us).  Past a
// wave's lanes of sequences it is not tried, and both kernels' waves go through
// the sequences 64 at a time, twice (1 token of 64 elements and 64 heads over up
// to 2000 positions: 64 sequences 32 us, 65 33, 256 105, 1024 361).  That grows
// with the square of their number (over up to 500 positions: 1024 sequences 0.2
// ms, 4096 1.0, 16384 8.3, where the cache's bytes alone would take 0.8).
//
// The line holds every unit of a sequence once for each row tile, also where no
// mask is given and a tile's tokens see only up to their own position: of a
// prompt's chunk without committed positions before it half of the units are
// passed over unread (2048 tokens of 56 heads of 128: 316 us, 190 TFLOP/s; behind
// 4096 positions 587, 512 TFLOP/s).
struct Line {
    int total;   // units; 0 if the offsets are not ascending in 0 .. T
    int per;     // units of a workgroup
    int round;   // a row tile's units on the line are a multiple of this
    // the last 64 sequences: the lane's, its units and those up to its end
    Seq s;
    int w, incl;
};
__device__ inline int on_line(int units, int round) {
    return round == 1 ? units : (int)(((uint32_t)units + round - 1) / (uint32_t)round) * round;
}
template <int ROWS>
__device__ inline void line_part(const AttnArgs& p, int b, Line* l, bool* bad) {
    l->s = read_seq(p, min(b, p.B - 1));
    if (l->s.first < 0 || l->s.first > p.T || l->s.n < 0 || l->s.n > p.T - l->s.first) {
        *bad = true;
        l->s.n = 0;
    }
    l->w = b < p.B ? items_of<ROWS>(p, l->s) * on_line(units_of(l->s), l->round) : 0;
    l->incl = wave_scan(l->w);
}
template <int ROWS>
__device__ inline Line line_of(const AttnArgs& p) {
    const int lane = threadIdx.x % kWave;
    Line l;
    l.total = 0;
    l.round = 1;
    bool bad = false;
    for (int b0 = 0; b0 < p.B; b0 += kWave) {
        line_part<ROWS>(p, b0 + lane, &l, &bad);
        l.total += __builtin_amdgcn_readlane(l.incl, kWave - 1);
    }
    if (__any(bad)) l.total = 0;
    l.per = max(1, (l.total + p.groups - 1) / p.groups);
    if (p.B <= kWave && l.per <= 1024) {  // (past that it does not matter, and w might overflow)
        const int items = lane < p.B ? items_of<ROWS>(p, l.s) : 0, units = units_of(l.s);
        for (int more = 0; more < 4; more++) {
            const int per = l.per + more, w = items * on_line(units, per), incl = wave_scan(w);
            const int total = __builtin_amdgcn_readlane(incl, kWave - 1);
            if (total <= p.groups * per && l.total) {
                l.total = total, l.per = per, l.round = per, l.w = w, l.incl = incl;
                break;
            }
        }
    }
    return l;
}

// The sequence of unit u (u < total), or with `token` of token u (-1: none),
// and the units before it; for a line that has units.
template <int ROWS>
__device__ inline int sequence_at(const AttnArgs& p, int u, bool token, Line* l, Seq* s, int* base) {
    const int lane = threadIdx.x % kWave;
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += kWave) {
        bool bad = false;
        if (p.B > kWave) line_part<ROWS>(p, b0 + lane, l, &bad);  // else line_of left it
        const bool mine = token ? b0 + lane < p.B && l->s.first <= u && u - l->s.first < l->s.n
                                : u - before < l->incl && u - before >= l->incl - l->w;
        const uint64_t at = __ballot(mine);
        if (at) {
            const int i = __builtin_ctzll(at);
            *base = before + __builtin_amdgcn_readlane(l->incl - l->w, i);
            s->first = __builtin_amdgcn_readlane(l->s.first, i);
            s->n = __builtin_amdgcn_readlane(l->s.n, i);
            s->L = __builtin_amdgcn_readlane(l->s.L, i);
            s->len = __builtin_amdgcn_readlane(l->s.len, i);
            return b0 + i;
        }
        before += __builtin_amdgcn_readlane(l->incl, kWave - 1);
    }
    return -1;
}

// ------------------------------------------------------------------ one wave

// How 32 positions of one head (a tile) go to the waves of a row group's
// workgroup.  In the cache a position's codes are D contiguous bytes.  A load
// takes whole lines: kLanes lanes of 16 bytes a position, kKeys positions at a
// time (16 lanes on 16 lines, as the matrix cores' operands would have them,
// cost 64 cycles a load in place of 16); the WR waves that share the tile take
// kLoads / WR each.  K lies in LDS as it came, its 16-byte pieces dealt so that
// 8 positions of an operand read are in different banks; V lies there in
// bf16, 16 bytes between its positions for the same reason.
template <int D>
struct Tile {
    typedef typename std::conditional<D == 64, uint16_t, typename std::conditional<D == 128, uint32_t, uint64_t>::type>::type scales_t;
    static constexpr int kLanes = D / 16, kKeys = kWave / kLanes, kLoads = 32 / kKeys;
    static constexpr int kValueRow = 2 * D + 16;              // bytes of a position's values in LDS
    static constexpr int kCodes = 32 * kValueRow;             // V, then K from here,
    static constexpr int kScales = kCodes + 32 * D;           // then K's scales,
    static constexpr int kBits = kScales + 32 * (D / 32);     // then for special tiles a bit for each value that is infinite
    static constexpr int kOdd = kBits + 32 * (D / 8);         // or no number, then whether there are any, a byte a load
    static constexpr int kBytes = kOdd + 16;
    // where piece `piece` of position `key`'s codes is: 8 neighbouring positions'
    // in different banks; pieces 2 i and 2 i + 1 stay neighbours, and 16
    // positions on the place is 16 D on
    __device__ static int code_at(int key, int piece) {
        return kCodes + key * D + (piece ^ (key / (256 / D) % (kLanes / 2) * 2)) * 16;
    }
};

// A wave's part of a tile as loaded: lane l has piece l % kLanes of position
// kKeys i + l / kLanes, that value's scale, and all scales of that key
template <int D, int N>
struct Part {
    u32x4_t k[N], v[N];
    uint32_t vs[N];
    typename Tile<D>::scales_t ks[N];
};

// The page numbers of a wave's tiles, 32 tiles at a time: lane l has that of half
// l % 2 of tile l / 2, as the table has it (past the last position its page is
// asked for again).  Read one by one a step before they are needed they would
// each be waited for: a value that is the same in all lanes goes to a scalar
// register as soon as it is there.
struct PageRun {
    int now, next;
};
__device__ inline int page_numbers(const AttnArgs& p, const int32_t* table, int p0, int stride, int len) {
    const int lane = threadIdx.x % kWave;
    const int64_t at = p0 + (int64_t)(lane / 2) * stride + 16 * (lane % 2);
    return table[max((int)(at < len ? at : len - 1), 0) >> p.page_shift];
}

// A tile's two halves: whether they are there, in pages of the cache, and
// their numbers (page 0 for one that is not)
struct Halves {
    uint32_t number[2];
    bool ok[2];
};
__device__ inline Halves halves_of(const AttnArgs& p, int pages, int tile, int p0, int len) {
    Halves h;
#pragma unroll
    for (int t = 0; t < 2; t++) {
        const uint32_t n = (uint32_t)__builtin_amdgcn_readlane(pages, 2 * (tile % 32) + t);
        h.ok[t] = p0 + 16 * t < len && n < (uint32_t)p.a.cache.num_pages;
        h.number[t] = h.ok[t] ? n : 0u;
    }
    return h;
}

// 32 bits of the lane's, and a constant, added to an address that is the same in all lanes and
// kept in scalar registers (memory, so that the load is no flat one, which
// would be counted among the LDS accesses)
template <typename X>
__device__ inline X load_at(const uint8_t* p, uint32_t offset, int more) {
    typedef const __attribute__((address_space(1))) uint8_t* global_t;
    uint64_t a = (uint64_t)p;
    asm volatile("" : "+s"(a));
    return *reinterpret_cast<const __attribute__((address_space(1))) X*>((global_t)a + offset + more);
}

// Where a wave's part of a tile is: its codes and scales in the tile's first and
// second half (only one of them where waves share the tile, WR > 1: the same
// then).  The addresses are worked out well before the loads, while the tile
// before is waited for in LDS: beside the loads they cost 400 to 600 cycles
// a step (8 trees of 64 tokens: 149 -> 141 us).
struct Source {
    const uint8_t *k[2], *v[2], *ks[2], *vs[2];
};
template <int D, int WR>
__device__ inline Source source_of(const AttnArgs& p, int h, int p0, int wr, const Halves& halves) {
    const moe_kv_cache& q = p.a.cache;
    Source r;
#pragma unroll
    for (int t = 0; t < (WR == 1 ? 2 : 1); t++) {
        const int first = WR == 1 ? 16 * t : 32 / WR * wr;
        const uint64_t n = first >= 16 ? halves.number[1] : halves.number[0];
        const uint32_t row = h * q.page_size + ((p0 + first) & (q.page_size - 1));
        const uint64_t code = n * (uint32_t)q.codes_page_stride + (uint64_t)row * D;
        const uint64_t scale = n * (uint32_t)q.scales_page_stride + (uint64_t)row * (D / 32);
        r.k[t] = q.k_codes + code, r.v[t] = q.v_codes + code;
        r.ks[t] = q.k_scales + scale, r.vs[t] = q.v_scales + scale;
    }
    return r;
}

template <int D, int WR, int N>
__device__ inline void load_part(const Source& from, int lane, Part<D, N>& r) {
    using T = Tile<D>;
    const uint32_t key = (uint32_t)lane / T::kLanes, piece = (uint32_t)lane % T::kLanes;
    constexpr int kOfHalf = WR == 1 ? N / 2 : N;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int t = i / kOfHalf, on = (i - t * kOfHalf) * T::kKeys;  // positions into the half
        r.k[i] = load_at<u32x4_t>(from.k[t], (uint32_t)lane * 16, on * D);
        r.v[i] = load_at<u32x4_t>(from.v[t], (uint32_t)lane * 16, on * D);
        r.ks[i] = load_at<typename T::scales_t>(from.ks[t], key * (D / 32), on * (D / 32));
        r.vs[i] = load_at<uint8_t>(from.vs[t], key * (D / 32) + piece / 2, on * (D / 32));
    }
}

__device__ inline f32x4_t mfma(const bf16x8_t& a, const bf16x8_t& b, const f32x4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// A wave's LDS accesses are carried out in order; this keeps the compiler
// from changing it.
__device__ inline void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The lane, anew: what is worked out from it is not kept in registers from
// where it was worked out before (rare paths, and the ends of a row tile)
__device__ inline int lane_again() {
    int lane;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(lane));
    return lane;
}

// A barrier that orders LDS alone: loads from memory stay on their way
__device__ inline void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Which of positions p0 .. p0+31 a drafted token sees (bit k: p0 + k)
__device__ inline uint32_t seen_bits(const AttnArgs& p, const Seq& s, int node, int p0, bool ok0, bool ok1) {
    const int js = p0 - s.L;  // the drafted token at p0, below 0: committed
    const int j0 = max(js, 0), shift = j0 - js;
    uint32_t seen = js >= 0 ? 0u : js <= -32 ? ~0u : (1u << shift) - 1u;
    if (js > -32 && j0 < s.n) {
        uint32_t bits;
        if (p.a.mask) {
            const uint64_t* m = p.a.mask + (int64_t)(s.first + node) * p.a.mask_words;
            const int w = j0 >> 6, o = j0 & 63;
            const uint64_t lo = w < p.a.mask_words ? m[w] : 0, hi = w + 1 < p.a.mask_words ? m[w + 1] : 0;
            bits = (uint32_t)(o ? (lo >> o) | (hi << (64 - o)) : lo);
        } else {
            const int k = node - j0 + 1;
            bits = k >= 32 ? ~0u : k <= 0 ? 0u : (1u << k) - 1u;
        }
        if (s.n - j0 < 32) bits &= (1u << (s.n - j0)) - 1u;
        seen |= bits << shift;
    }
    const int left = s.len - p0;
    if (left < 32) seen &= left <= 0 ? 0u : (1u << left) - 1u;
    return seen & (ok0 ? ~0u : 0xffff0000u) & (ok1 ? ~0u : 0xffffu);
}

template <int D, int R>
struct Wave {
    // per row tile, lane (c, g): row c.  O: elements 16 d + 4 g ..
    f32x4_t o[R][D / 16], sum[R];
    float m[R], mc[R];  // the reference score, and c * m (0 while there is none)
    float pass[R];      // the score past which the reference is moved
};

// A value that is infinite or no number makes one of what sees it, and of
// nothing else (0 times it would): in its place 2^127 is multiplied with 2^127
// where it is seen, or the negative, or for no number both: infinity less
// infinity.  Which it is the value's place holds (`store_part`).  For an O that
// is not scaled by 0 any more.  seen: as shifted for the lane's positions.
template <int D, int R>
__device__ inline void add_specials(const uint8_t* lds, const uint32_t (&seen)[R], Wave<D, R>& w) {
    using T = Tile<D>;
    const int lane = lane_again(), c = lane % 16, g = lane / 16;
    const uint16_t* bits = reinterpret_cast<const uint16_t*>(lds + T::kBits);
#pragma unroll
    for (int d = 0; d < D / 16; d++) {
        u32x4_t n, m;
#pragma unroll
        for (int i = 0; i < 4; i++) {  // the lane's positions 2 i, 2 i + 1 of 8
            const int at = 16 * (i / 2) + 4 * g + 2 * (i % 2);
            const uint32_t a = bits[at * T::kLanes + d] >> c & 1u, b = bits[(at + 1) * T::kLanes + d] >> c & 1u;
            const uint8_t* value = lds + at * T::kValueRow + (16 * d + c) * 2;
            const uint32_t va = *reinterpret_cast<const uint16_t*>(value);
            const uint32_t vb = *reinterpret_cast<const uint16_t*>(value + T::kValueRow);
            n[i] = 0x7f00u * (va != 0x8000u ? a : 0u) | 0x7f000000u * (vb != 0x8000u ? b : 0u);
            m[i] = 0xff00u * (va != 0 ? a : 0u) | 0xff000000u * (vb != 0 ? b : 0u);
        }
#pragma unroll
        for (int r = 0; r < R; r++) {
            auto pair = [&](int k) {  // of positions k, k + 1
                return 0x7f00u * (seen[r] >> k & 1u) | 0x7f000000u * (seen[r] >> (k + 1) & 1u);
            };
            const u32x4_t sees = {pair(0), pair(2), pair(16), pair(18)};
            w.o[r][d] = mfma(__builtin_bit_cast(bf16x8_t, n), __builtin_bit_cast(bf16x8_t, sees), w.o[r][d]);
            w.o[r][d] = mfma(__builtin_bit_cast(bf16x8_t, m), __builtin_bit_cast(bf16x8_t, sees), w.o[r][d]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// A wave's part of the tile at p0, into LDS.  special: some of the tile's
// positions are drafted ones or none at all; else all rows see all of them.
// There values that are infinite or no numbers are stored without their
// exponent (+0, -0, or for no number something small that is not 0), and their
// places kept: `weights` puts them back, by the same question of the same tile.
// The waves that share a tile have the same answer, whichever loop each is
// in.  (SPECIAL false: a loop that knows it is not.)
template <bool SPECIAL, int D, int N>
__device__ inline void store_part(const Seq& s, int p0, int wr, int lane, bool special, const Halves& h,
                                  Part<D, N>& r, uint8_t* lds) {
    using T = Tile<D>;
    const int key = lane / T::kLanes, piece = lane % T::kLanes;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int at = (wr * N + i) * T::kKeys + key;
        *reinterpret_cast<u32x4_t*>(lds + T::code_at(at, piece)) = r.k[i];
        // (all lanes of a position: the same word to the same place)
        reinterpret_cast<typename T::scales_t*>(lds + T::kScales)[at] = r.ks[i];
        u32x4_t v[2];
        const float f = e8m0_as_scale(r.vs[i]);
        v[0] = __builtin_bit_cast(u32x4_t, decode8_e4m3(r.v[i].x, r.v[i].y, f));
        v[1] = __builtin_bit_cast(u32x4_t, decode8_e4m3(r.v[i].z, r.v[i].w, f));
        if (SPECIAL && special) {
            const bool there = p0 + at < s.len && ((wr * N + i) * T::kKeys >= 16 ? h.ok[1] : h.ok[0]);
            uint32_t bits = 0;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                uint32_t w = there ? v[e / 4][e % 4] : 0u;
                if ((w & 0x7f80u) == 0x7f80u) bits |= 1u << (2 * e), w &= ~0x7f80u;
                if ((w & 0x7f800000u) == 0x7f800000u) bits |= 2u << (2 * e), w &= ~0x7f800000u;
                v[e / 4][e % 4] = w;
            }
            reinterpret_cast<uint16_t*>(lds + T::kBits)[at * T::kLanes + piece] = (uint16_t)bits;
            const bool odd = __any(bits != 0);
            if (lane == 0) lds[T::kOdd + wr * N + i] = odd;
        }
        u32x4_t* to = reinterpret_cast<u32x4_t*>(lds + at * T::kValueRow + piece * 32);
        to[0] = v[0];
        to[1] = v[1];
    }
}

// The weights of the 32 positions from p0, whose tile is in LDS, for a wave's
// rows; m and with it O and its sum are moved where a score asks for it.
// meanwhile: what is done while the keys are waited for.
template <bool SPECIAL, int D, int R, typename Node, typename Meanwhile>
__device__ inline void weights(const AttnArgs& p, const Seq& s, Node&& node_of, const bf16x8_t (&q)[R][D / 32], int p0,
                               int lane, bool special, const Halves& h, const uint8_t* lds, Wave<D, R>& w,
                               bf16x8_t (&pt)[R], Meanwhile&& meanwhile) {
    using T = Tile<D>;
    const int c = lane % 16, g = lane / 16;
    // lane (c, g): quarter g of position 16 t + c.  All reads are on their way
    // before the first is waited for (left to itself the compiler reads each
    // just before its use: 850 cycles a tile in place of 500)
    u32x4_t kx[2][D / 64];
    uint32_t ks[2];
#pragma unroll
    for (int t = 0; t < 2; t++) {
        const uint8_t* scales = lds + T::kScales + (16 * t + c) * (D / 32);
        if constexpr (D == 64) ks[t] = scales[g / 2];
        else if constexpr (D == 128) ks[t] = scales[g];
        else ks[t] = *reinterpret_cast<const uint16_t*>(scales + 2 * g);
#pragma unroll
        for (int j = 0; j < D / 64; j++)
            kx[t][j] = *reinterpret_cast<const u32x4_t*>(lds + T::code_at(c, g * (D / 64) + j / 2 * 2) + 16 * t * D + j % 2 * 16);
    }
    __builtin_amdgcn_sched_barrier(0);
    meanwhile();
    f32x4_t st[2][R];
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
        for (int r = 0; r < R; r++) st[t][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < D / 64; j++)
#pragma unroll
        for (int t = 0; t < 2; t++) {
            const float f = e8m0_as_scale(D == 256 ? (j < 2 ? ks[t] & 0xffu : ks[t] >> 8) : ks[t]);
            const bf16x8_t k0 = decode8_e4m3(kx[t][j].x, kx[t][j].y, f), k1 = decode8_e4m3(kx[t][j].z, kx[t][j].w, f);
#pragma unroll
            for (int r = 0; r < R; r++) st[t][r] = mfma(k0, q[r][2 * j], st[t][r]);
#pragma unroll
            for (int r = 0; r < R; r++) st[t][r] = mfma(k1, q[r][2 * j + 1], st[t][r]);
        }
    uint32_t seen[R];
    if (SPECIAL && special) {
#pragma unroll
        for (int r = 0; r < R; r++) {
            seen[r] = seen_bits(p, s, node_of(16 * r + c), p0, h.ok[0], h.ok[1]) >> (4 * g);
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t keep = (uint32_t)((int32_t)(seen[r] << (31 - 16 * t - i)) >> 31);
                    st[t][r][i] = __uint_as_float((__float_as_uint(st[t][r][i]) & keep) | (0xff800000u & ~keep));
                }
        }
    }
    // the reference score, where one has passed it
    float top[R];
    bool passed = false;
#pragma unroll
    for (int r = 0; r < R; r++) {
        top[r] = fmaxf(st[0][r][0], st[1][r][0]);
#pragma unroll
        for (int i = 1; i < 4; i++) top[r] = fmaxf(fmaxf(top[r], st[0][r][i]), st[1][r][i]);
        passed |= top[r] > w.pass[r];
    }
    if (__any(passed)) {
#pragma unroll
        for (int r = 0; r < R; r++) {
#pragma clang fp contract(off)
            float t = top[r];
            t = fmaxf(t, __shfl_xor(t, 16));
            t = fmaxf(t, __shfl_xor(t, 32));
            // (a row whose own has not passed keeps it, and f is 1, as c m is rounded
            // alike each time: its result does not depend on the other rows)
            const float m = t > w.pass[r] ? t : w.m[r], mc = m == minus_inf() ? 0.f : m * p.c;
            const float f = w.m[r] == minus_inf() ? 0.f : __builtin_amdgcn_exp2f(w.mc[r] - mc);
#pragma unroll
            for (int d = 0; d < D / 16; d++) w.o[r][d] *= f;
            w.sum[r] *= f;
            w.m[r] = m;
            w.mc[r] = mc;
            w.pass[r] = m + kAttnSlack / p.c;
        }
    }
    if (SPECIAL && special) {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < T::kLoads; i++) any |= lds[T::kOdd + i];
        if (uniform(any)) add_specials<D, R>(lds, seen, w);
    }
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                pt[r][4 * t + i] = (__bf16)__builtin_amdgcn_exp2f(fmaf(st[t][r][i], p.c, -w.mc[r]));
}

// O and its sum with the weights of the tile in LDS
template <int D, int R>
__device__ inline void product(const bf16x8_t (&pt)[R], int lane, const uint8_t* lds, Wave<D, R>& w) {
    using T = Tile<D>;
    const int c = lane % 16, g = lane / 16;
    typedef __attribute__((address_space(3))) s16x4_t lds4_t;
    const uint8_t* column = lds + (4 * g + c / 4) * T::kValueRow + (c % 4) * 8;
    auto value = [&](int d) {
        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4_t*)(column + 32 * d));
        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4_t*)(column + 16 * T::kValueRow + 32 * d));
        const s16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        return __builtin_bit_cast(bf16x8_t, v);
    };
    constexpr int kAhead = 4;
    bf16x8_t vt[kAhead];
#pragma unroll
    for (int d = 0; d < kAhead; d++) vt[d] = value(d);
    const s16x8_t one16 = {0x3f80, 0x3f80, 0x3f80, 0x3f80, 0x3f80, 0x3f80, 0x3f80, 0x3f80};
    const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, one16);
#pragma unroll
    for (int r = 0; r < R; r++) w.sum[r] = mfma(ones, pt[r], w.sum[r]);
#pragma unroll
    for (int d = 0; d < D / 16; d++) {
#pragma unroll
        for (int r = 0; r < R; r++) w.o[r][d] = mfma(vt[d % kAhead], pt[r], w.o[r][d]);
        if (d + kAhead < D / 16) vt[d % kAhead] = value(d + kAhead);
    }
}

// the statistic of rows without a position is -infinity: their weight is 0
__device__ inline float reference(float m) { return m == minus_inf() ? 0.f : m; }

// A workgroup's shape: WR groups of 16 R rows times WK runs of positions, a
// wave each.  The WR waves of a run share its tiles, which are then in LDS twice:
// the next one's parts are stored while this one is worked on.
template <int D_, int R_, int WR_, int WK_>
struct Shape {
    static constexpr int D = D_, R = R_, WR = WR_, WK = WK_;
    static constexpr int kRows = 16 * R * WR, kWaves = WR * WK, kThreads = kWave * kWaves;
    static constexpr int kParts = Tile<D>::kLoads / WR;
    static_assert(kParts * WR == Tile<D>::kLoads, "a tile is dealt evenly");
    static constexpr int kBuffers = WR == 1 ? 1 : 2, kTiles = kBuffers * WK * Tile<D>::kBytes;
    static constexpr int kResult = kWaves * 16 * R * (D + 4) * 4;  // at the end the waves' results
    static constexpr int kQuery = 16 * D * 2;                  // at the start 16 queries of each
    static constexpr int kLds = kTiles > kResult ? kTiles : kResult;
    static_assert(kWaves * kQuery <= kLds, "queries fit");
    // waves per SIMD that the registers and LDS leave room for
    static constexpr int kPerSimd = D == 256 ? 1 : 2;
};

template <typename S>
__global__ void __launch_bounds__(S::kThreads, S::kPerSimd) tree_attention_kernel(AttnArgs p) {
    constexpr int D = S::D, R = S::R, WR = S::WR, WK = S::WK, ROWS = S::kRows;
    __shared__ __align__(16) uint8_t buf[S::kLds];
    __shared__ float s_m[WK][ROWS], s_sum[WK][ROWS];
    const int wave = uniform((int)threadIdx.x / kWave);
    const int wr = wave % WR, wk = wave / WR;
    // Workgroups are dealt round the 8 XCDs; each XCD takes a run of the line, so
    // that the row tiles of a head, which read the same positions, share its L2
    const int group = (int)blockIdx.x % 8 * (p.groups / 8) + (int)blockIdx.x / 8;
    Line line = line_of<ROWS>(p);
    int u = uniform(group * line.per);
    const int end = uniform(min(u + line.per, line.total));
    if (u >= end) return;
    int base = 0;
    Seq s;
    int b = uniform(sequence_at<ROWS>(p, u, false, &line, &s, &base));
    while (u < end) {
        const int tiles = tiles_of<ROWS>(p, s), units = units_of(s), long_units = on_line(units, line.round);
        const int all = items_of<ROWS>(p, s) * long_units;
        if (u - base >= all) {  // on to the next sequence (there is one: u < total)
            base += all;
            b++;
            s = read_seq(p, b);
            s.first = uniform(s.first), s.n = uniform(s.n), s.L = uniform(s.L), s.len = uniform(s.len);
            continue;
        }
        // (unsigned: half the instructions of a signed division)
        const uint32_t item = (uint32_t)(u - base) / (uint32_t)long_units;
        const int u0 = u - base - (int)item * long_units, u1 = min(units, u0 + end - u);
        const int h = (int)(item / (uint32_t)tiles), row0 = ((int)item - h * tiles) * ROWS;
        const int here = min(ROWS, s.n * p.G - row0);  // rows of the tile
        const int node0 = (int)((uint32_t)row0 / (uint32_t)p.G), rest = row0 - node0 * p.G;
        // drafted token (from node0) of a row of the tile, past the last that one's
        auto node_of = [&](int row) { return by_group(p, rest + min(row, here - 1)); };

        // positions that some row of the workgroup, and of the wave, may see
        const int from = u0 * kAttnUnit;
        int stop = min(s.len, u1 * kAttnUnit), mine = stop;
        if (!p.a.mask) {
            stop = min(stop, s.L + node0 + node_of(ROWS - 1) + 1);
            mine = min(stop, s.L + node0 + node_of(16 * R * (wr + 1) - 1) + 1);
        }
        if (16 * R * wr >= here) mine = 0;
        const int32_t* table = p.a.block_table + (int64_t)b * p.a.block_table_stride;
        const int steps = stop > from ? (stop - from + 32 * WK - 1) / (32 * WK) : 0;
        int p0 = from + 32 * wk;
        constexpr int kStride = 32 * WK;  // from a wave's tile to its next
        PageRun run;
        run.now = page_numbers(p, table, p0, kStride, s.len);
        run.next = page_numbers(p, table, p0 + 32 * kStride, kStride, s.len);

        auto node_at = [&](int row) { return node0 + node_of(16 * R * wr + row); };  // of the wave's rows
        const int lane = lane_again(), c = lane % 16, g = lane / 16;
        bf16x8_t q[R][D / 32];
        Wave<D, R> w;
        // the queries, whole lines at a time and through LDS (past the last row that row again)
        constexpr int kRowLanes = D / 8, kRowsAtOnce = kWave / kRowLanes;  // lanes of 16 bytes a row
        const uint16_t* queries = (const uint16_t*)p.a.q + (int64_t)(s.first + node0) * p.a.q_stride + h * p.G * D;
        u32x4_t rows_in[R][16 / kRowsAtOnce];
#pragma unroll
        for (int r = 0; r < R; r++) {
#pragma unroll
            for (int i = 0; i < 16 / kRowsAtOnce; i++) {
                const int row = 16 * (R * wr + r) + kRowsAtOnce * i + lane / kRowLanes, at = node_of(row);
                const uint16_t* src = queries + (uint64_t)(uint32_t)at * (uint32_t)p.a.q_stride +
                                      (rest + min(row, here - 1) - at * p.G) * D + lane % kRowLanes * 8;
                rows_in[r][i] = *reinterpret_cast<const u32x4_t*>(src);
            }
        }
        Part<D, S::kParts> part;
        Halves halves = halves_of(p, run.now, 0, p0, s.len);
        load_part<D, WR>(source_of<D, WR>(p, h, p0, wr, halves), lane, part);
        uint8_t* qbuf = buf + wave * S::kQuery;
        auto query_at = [](int row, int piece) {  // 16-byte pieces, the 16 rows' in different banks
            return row * D * 2 + (piece ^ (D == 64 ? row / 2 : row)) * 16;
        };
#pragma unroll
        for (int r = 0; r < R; r++) {
#pragma unroll
            for (int i = 0; i < 16 / kRowsAtOnce; i++)
                *reinterpret_cast<u32x4_t*>(qbuf + query_at(kRowsAtOnce * i + lane / kRowLanes, lane % kRowLanes)) =
                    rows_in[r][i];
            wave_order();
#pragma unroll
            for (int j = 0; j < D / 32; j++)
                q[r][j] = *reinterpret_cast<const bf16x8_t*>(qbuf + query_at(c, g * (D / 32) + j));
            wave_order();
#pragma unroll
            for (int d = 0; d < D / 16; d++) w.o[r][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            w.sum[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            w.m[r] = minus_inf();
            w.mc[r] = 0.f;
            w.pass[r] = minus_inf();
        }
        lds_barrier();

        uint8_t* tile = buf + S::kBuffers * wk * Tile<D>::kBytes;
        auto is_special = [&](int at, const Halves& t) { return at + 32 > s.L || !t.ok[0] || !t.ok[1]; };
        Halves now = halves, next;  // of tile i, of the one after that in `part` (which has halves)
        auto source = [&](int i, int at) {  // of the wave's tile i, at position `at`
            if (i % 32 == 0) {
                run.now = run.next;
                run.next = page_numbers(p, table, at + 32 * kStride, kStride, s.len);
            }
            next = halves_of(p, run.now, i, at, s.len);
            return source_of<D, WR>(p, h, at, wr, next);
        };
        // A step: the weights and the product of tile i, the next tile stored and the
        // one after it loaded.  Tiles that all rows see whole have a loop of
        // their own, whose steps are one piece of code for the scheduler (8 trees
        // of 64 tokens: 155 -> 149 us); the waves of a workgroup may be in either
        // loop (a step has one barrier).
        bf16x8_t pt[R];
        int i = 0;
        Source ahead = source(1, p0 + kStride);  // of the tile after that in `part`
        auto step = [&](auto special) {
            constexpr bool SPECIAL = decltype(special)::value;
            // the rare loop works out what comes of the lane each time, the other keeps it
            const int lane = SPECIAL ? lane_again() : (int)threadIdx.x % kWave;
            uint8_t* lds = tile + (WR > 1 ? (i & 1) * Tile<D>::kBytes : 0);
            if constexpr (WR == 1) {  // a tile is its wave's own
                now = halves;
                store_part<SPECIAL>(s, p0, wr, lane, is_special(p0, now), now, part, lds);
                wave_order();
                halves = next;
                load_part<D, WR>(ahead, lane, part);
            }
            auto meanwhile = [&] { ahead = source(i + 2, p0 + 2 * kStride); };
            if (!SPECIAL || p0 < mine) {
                weights<SPECIAL, D, R>(p, s, node_at, q, p0, lane, is_special(p0, now), now, lds, w, pt, meanwhile);
                product<D, R>(pt, lane, lds, w);
            } else {
                meanwhile();
            }
            if constexpr (WR == 1) {
                wave_order();
            } else {
                now = halves;
                store_part<SPECIAL>(s, p0 + kStride, wr, lane, is_special(p0 + kStride, now), now, part,
                                    tile + (~i & 1) * Tile<D>::kBytes);
                halves = next;
                load_part<D, WR>(ahead, lane, part);
                lds_barrier();
            }
            i++;
            p0 += kStride;
        };
        if constexpr (WR == 1) {
            while (i < steps && !is_special(p0, halves)) step(std::false_type{});
            while (i < steps && p0 < mine) step(std::true_type{});
        } else if (steps > 0) {
            store_part<true>(s, p0, wr, lane, is_special(p0, halves), halves, part, tile);
            halves = next;
            load_part<D, WR>(ahead, lane, part);
            lds_barrier();
            // (two loops one after the other would hold O in other registers each)
            while (i < steps) {
#pragma unroll 1
                while (i < steps && mine && !is_special(p0, now) && !is_special(p0 + kStride, halves))
                    step(std::false_type{});
                if (i < steps) step(std::true_type{});
            }
        }
        lds_barrier();

        // the results of the waves of a row group joined
        const int own = lane_again(), oc = own % 16, og = own / 16, tid = wave * kWave + own;
        if (og == 0)
#pragma unroll
            for (int r = 0; r < R; r++)
                s_m[wk][16 * (R * wr + r) + oc] = w.m[r] == minus_inf() ? minus_inf() : w.mc[r];
        lds_barrier();
        auto top_of = [&](int row) {
            float m = s_m[0][row];
#pragma unroll
            for (int i = 1; i < WK; i++) m = fmaxf(m, s_m[i][row]);
            return m;
        };
        float* joined = reinterpret_cast<float*>(buf);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const float f = __builtin_amdgcn_exp2f((w.m[r] == minus_inf() ? minus_inf() : w.mc[r]) -
                                                   reference(top_of(16 * (R * wr + r) + oc)));
            float* to = joined + ((wave * R + r) * 16 + oc) * (D + 4) + 4 * og;
#pragma unroll
            for (int d = 0; d < D / 16; d++) *reinterpret_cast<f32x4_t*>(to + 16 * d) = w.o[r][d] * f;
            if (og == 0) s_sum[wk][16 * (R * wr + r) + oc] = w.sum[r][0] * f;
        }
        lds_barrier();
        const bool whole = u0 == 0 && u1 == units;
        float* left = (float*)p.a.workspace + (2 * (int64_t)group + (u0 ? 0 : 1)) * p.part_floats;
        uint16_t* out = (uint16_t*)p.a.out + (int64_t)(s.first + node0) * p.a.out_stride + h * p.G * D;
        constexpr int kPiece = 8, kPieces = D / kPiece;  // elements of a thread, threads of a row
#pragma unroll 1
        for (int i = tid; i < ROWS * kPieces; i += S::kThreads) {
            const int at = i / kPieces, d0 = i % kPieces * kPiece;
            const int from_wave = at / (16 * R), from_row = at % (16 * R);
            f32x4_t v[2] = {};
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < WK; k++) {
                const f32x4_t* src = reinterpret_cast<const f32x4_t*>(
                    joined + ((k * WR + from_wave) * 16 * R + from_row) * (D + 4) + d0);
                v[0] += src[0];
                v[1] += src[1];
                sum += s_sum[k][at];
            }
            if (!whole) {
                f32x4_t* dst = reinterpret_cast<f32x4_t*>(left + at * D + d0);
                dst[0] = v[0];
                dst[1] = v[1];
                if (d0 == 0) {
                    left[ROWS * D + 2 * at] = top_of(at);
                    left[ROWS * D + 2 * at + 1] = sum;
                }
            } else if (at < here) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const int node = node_of(at);
                float o[kPiece];
#pragma unroll
                for (int e = 0; e < kPiece; e++) o[e] = v[e / 4][e % 4] * inv;
                store_piece<kPiece>(out + (uint64_t)(uint32_t)node * (uint32_t)p.a.out_stride +
                                        (rest + at - node * p.G) * D + d0, o);
            }
        }
        lds_barrier();
        u += line.round > 1 ? line.per : u1 - u0;
    }
}

// The parts of row tiles that several workgroups did, in their order: HEADS
// heads of a token a wave.  A part's weight is 2^(its reference - the largest).
template <int D, int ROWS, int HEADS>
__global__ void __launch_bounds__(kJoinWaves * kWave) tree_attention_join_kernel(AttnArgs p) {
    const int lane = threadIdx.x % kWave, heads = p.a.num_heads, runs = (heads + HEADS - 1) / HEADS;
    const int idx = uniform(((int)blockIdx.y * (int)kJoinRow + (int)blockIdx.x) * kJoinWaves + (int)threadIdx.x / kWave);
    if (idx >= p.T * runs) return;
    const int token = (int)((uint32_t)idx / (uint32_t)runs), head0 = (idx - token * runs) * HEADS;
    Line line = line_of<ROWS>(p);
    if (line.total == 0) return;
    int base = 0;
    Seq s;
    if (sequence_at<ROWS>(p, token, true, &line, &s, &base) < 0) return;
    const int units = units_of(s), long_units = on_line(units, line.round), tiles = tiles_of<ROWS>(p, s);
    // 16 bytes a lane, kAtOnce parts at a time
    constexpr int kLanes = D / 4, kAtOnce = kWave / kLanes;
    const int which = lane / kLanes, e0 = lane % kLanes * 4;

    int first[HEADS], parts[HEADS], at[HEADS], most = 0;
#pragma unroll
    for (int j = 0; j < HEADS; j++) {
        const int head = min(head0 + j, heads - 1), h = by_group(p, head);
        const int row = (token - s.first) * p.G + head - h * p.G;
        const int u0 = base + (h * tiles + row / ROWS) * long_units;
        at[j] = row % ROWS;
        first[j] = (int)((uint32_t)u0 / (uint32_t)line.per);
        parts[j] = head0 + j < heads ? (int)((uint32_t)(u0 + units - 1) / (uint32_t)line.per) - first[j] + 1 : 1;
        most = max(most, parts[j]);
    }
    if (most == 1) return;
    auto part = [&](int j, int i) {
        return (const float*)p.a.workspace + (2 * (int64_t)(first[j] + i) + (i ? 0 : 1)) * p.part_floats;
    };
    // UNROLL * kAtOnce parts of COUNT heads from j0, in flight together; v and
    // sum relative to `top`
    auto add = [&](auto unroll, auto count, int j0, int i0, float (&top)[HEADS], f32x4_t (&v)[HEADS],
                   float (&sum)[HEADS]) {
        constexpr int UNROLL = decltype(unroll)::value, COUNT = decltype(count)::value;
        f32x4_t x[COUNT][UNROLL];
        float m[COUNT][UNROLL], l[COUNT][UNROLL];
#pragma unroll
        for (int j = 0; j < COUNT; j++)
#pragma unroll
            for (int k = 0; k < UNROLL; k++) {
                const int i = i0 + k * kAtOnce + which;
                const float* src = part(j0 + j, min(i, parts[j0 + j] - 1));
                x[j][k] = *reinterpret_cast<const f32x4_t*>(src + at[j0 + j] * D + e0);
                m[j][k] = i < parts[j0 + j] ? src[ROWS * D + 2 * at[j0 + j]] : minus_inf();
                l[j][k] = src[ROWS * D + 2 * at[j0 + j] + 1];
            }
#pragma unroll
        for (int j = 0; j < COUNT; j++) {
            float t = top[j0 + j];
#pragma unroll
            for (int k = 0; k < UNROLL; k++) t = fmaxf(t, m[j][k]);
#pragma unroll
            for (int a = kLanes; a < kWave; a *= 2) t = fmaxf(t, __shfl_xor(t, a));
            const float f = top[j0 + j] == minus_inf() ? 0.f : __builtin_amdgcn_exp2f(top[j0 + j] - t);
            top[j0 + j] = t;
            sum[j0 + j] *= f;
            v[j0 + j] *= f;
#pragma unroll
            for (int k = 0; k < UNROLL; k++) {
                if (i0 + k * kAtOnce + which >= parts[j0 + j]) continue;
                const float g = __builtin_amdgcn_exp2f(m[j][k] - reference(t));
                sum[j0 + j] = fmaf(l[j][k], g, sum[j0 + j]);
#pragma unroll
                for (int e = 0; e < 4; e++) v[j0 + j][e] = fmaf(x[j][k][e], g, v[j0 + j][e]);
            }
        }
    };
    float top[HEADS], sum[HEADS] = {};
    f32x4_t v[HEADS] = {};
#pragma unroll
    for (int j = 0; j < HEADS; j++) top[j] = minus_inf();
    constexpr int kFew = 4 / kAtOnce > 0 ? 4 / kAtOnce : 1, kMany = 16 / kAtOnce;
    if (most <= kFew * kAtOnce) {
        add(std::integral_constant<int, kFew>{}, std::integral_constant<int, HEADS>{}, 0, 0, top, v, sum);
    } else {
        static_for<HEADS>([&](auto j) {
            for (int i0 = 0; i0 < parts[j]; i0 += kMany * kAtOnce)
                add(std::integral_constant<int, kMany>{}, std::integral_constant<int, 1>{}, j, i0, top, v, sum);
        });
    }
#pragma unroll
    for (int j = 0; j < HEADS; j++) {
#pragma unroll
        for (int a = kLanes; a < kWave; a *= 2) {
            sum[j] += __shfl_xor(sum[j], a);
#pragma unroll
            for (int e = 0; e < 4; e++) v[j][e] += __shfl_xor(v[j][e], a);
        }
        if (which || parts[j] == 1) continue;
        const float inv = sum[j] == 0.f ? 0.f : 1.f / sum[j];
        const float o[4] = {v[j][0] * inv, v[j][1] * inv, v[j][2] * inv, v[j][3] * inv};
        store_piece<4>((uint16_t*)p.a.out + (int64_t)token * p.a.out_stride + (head0 + j) * D + e0, o);
    }
}

template <int D, int R, int WR, int WK>
hipError_t launch_shape(const AttnArgs& p, hipStream_t stream) {
    using S = Shape<D, R, WR, WK>;
    tree_attention_kernel<S><<<p.groups, S::kThreads, 0, stream>>>(p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const AttentionJoin join = attention_join(p.T, p.a.num_heads);
    const dim3 grid(join.x, join.y);
    if (join.heads == 4) tree_attention_join_kernel<D, S::kRows, 4><<<grid, kJoinWaves * kWave, 0, stream>>>(p);
    else tree_attention_join_kernel<D, S::kRows, 1><<<grid, kJoinWaves * kWave, 0, stream>>>(p);
    return hipGetLastError();
}

template <int D>
hipError_t launch_rows(const AttnArgs& p, int rows, hipStream_t stream) {
    if (rows == 16) return launch_shape<D, 1, 1, 4>(p, stream);
    if constexpr (D == 256) {
        return rows == 32   ? launch_shape<D, 1, 2, 2>(p, stream)
               : rows == 64 ? launch_shape<D, 1, 4, 1>(p, stream)
                            : launch_shape<D, 2, 4, 1>(p, stream);
    } else {
        if (rows == 32) return launch_shape<D, 2, 1, 4>(p, stream);
        if constexpr (D == 128)
            if (rows == 128) return launch_shape<D, 2, 4, 2>(p, stream);
        return launch_shape<D, 2, 2, 4>(p, stream);
    }
}

}  // namespace

hipError_t launch_tree_attention(const moe_tree_attention_args& a, hipStream_t stream) {
    const AttentionPlan plan =
        attention_plan(a.num_tokens, a.num_seqs, a.num_heads, a.cache.kv_heads, a.cache.head_dim);
    AttnArgs p;
    p.a = a;
    p.T = (int)a.num_tokens;
    p.B = (int)a.num_seqs;
    p.G = a.num_heads / a.cache.kv_heads;
    p.g_inverse = p.G > 1 ? (uint32_t)(((1ull << 32) + p.G - 1) / p.G) : 0;
    p.page_shift = __builtin_ctz(a.cache.page_size);
    p.capacity = (int)(a.max_pages * a.cache.page_size);
    p.groups = plan.groups;
    p.c = a.scale * 1.44269504088896340736f;
    p.part_floats = plan.part_floats;
    switch (a.cache.head_dim) {
        case 64: return launch_rows<64>(p, plan.rows, stream);
        case 128: return launch_rows<128>(p, plan.rows, stream);
        default: return launch_rows<256>(p, plan.rows, stream);
    }
}

}  // namespace moe

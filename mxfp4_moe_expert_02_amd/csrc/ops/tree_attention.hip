// tree_attention.hip -- attention of drafted tokens over the MXFP8 cache.
//
// The rows of one key/value head of a sequence are its drafted tokens times
// the query heads that share it; a workgroup takes 16 R of them (a row tile)
// over a run of positions.  Its four waves take 32 positions each in turn,
// all rows, and keep a result of their own (m, sum, O), joined at the end of
// the run.  Per 32 positions a wave computes
//
//   S^T = K Q^T     A = K (decoded in the registers it was loaded to), B = Q
//   P^T = 2^(c S^T - m)
//   O^T += V^T P^T  A = V^T (decoded, through LDS), B = P^T: the lanes and
//                   registers that S^T came in, as bf16
//
// with v_mfma_f32_16x16x32_bf16.  Lane (c, g) = (l % 16, l / 16).  K's lane
// (c, g) holds quarter g of position c's elements, which is how the cache lies
// (one contiguous run and its scale per lane); the inner axis is then in
// another order than the elements', and Q is loaded in the same one.  Of the 32
// positions of O's inner axis a lane of P^T holds 4g .. 4g+3 and 16 + 4g .. ; V^T
// comes in that order out of ds_read_b64_tr_b16, which hands a lane 4 rows of a
// column.  The sum of the weights is one more product, with ones in V's place.
//
// m is a row's running maximum, but it is moved only where a score passes it
// by more than 8 powers of two (P then stays below 2^8), so that most steps
// neither exchange maxima nor rescale O.
//
// Work is cut by units of 128 positions, all row tiles' units in one line, an
// equal run of them to each workgroup: ragged lengths cost nothing.  A row tile
// that one workgroup does whole is finished there; else its parts go to the
// workspace in float32 and tree_attention_join_kernel adds them in order.
#include "attention_internal.h"

namespace moe {
namespace {

constexpr int kJoinWaves = 4;
constexpr float kAttnSlack = 8.f;  // powers of two that a score may pass m by

struct AttnArgs {
    moe_tree_attention_args a;
    int T, B, G;               // tokens, sequences, query heads per key/value head
    int page_shift, capacity;  // positions of a page (log2), of a sequence's table
    int groups;                // workgroups
    float c;                   // scale * log2 e
    int64_t part_floats;       // of one partial result
};

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));

__device__ inline float minus_inf() { return -__builtin_inff(); }

// ----------------------------------------------------------- the line of units

// A sequence as the device holds it: its first token, its tokens, committed
// positions and all positions (lengths out of range taken as the header says)
struct Seq {
    int first, n, L, len;
};
__device__ inline Seq read_seq(const AttnArgs& p, int b) {
    Seq s;
    s.first = p.a.token_offsets[b];
    s.n = p.a.token_offsets[b + 1] - s.first;
    s.L = min(max(p.a.context_lens[b], 0), p.capacity);
    s.len = min(s.L + s.n, p.capacity);
    return s;
}
template <int ROWS>
__device__ inline int tiles_of(const AttnArgs& p, const Seq& s) {
    return (s.n * p.G + ROWS - 1) / ROWS;
}
__device__ inline int units_of(const Seq& s) { return max(1, (s.len + kAttnUnit - 1) / kAttnUnit); }

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
// for itself, 64 sequences at a time (the lengths are the device's).
struct Line {
    int total;  // units; 0 if the offsets are not ascending in 0 .. T
    int per;    // units of a workgroup
};
// units of a lane's sequence b
template <int ROWS>
__device__ inline int weight_of(const AttnArgs& p, int b, bool* bad) {
    if (b >= p.B) return 0;
    const Seq s = read_seq(p, b);
    if (s.first < 0 || s.first > p.T || s.n < 0 || s.n > p.T - s.first) {
        *bad = true;
        return 0;
    }
    return s.n ? tiles_of<ROWS>(p, s) * units_of(s) * p.a.cache.kv_heads : 0;
}
template <int ROWS>
__device__ inline Line line_of(const AttnArgs& p) {
    const int lane = threadIdx.x % kWave;
    int total = 0;
    bool bad = false;
    for (int b0 = 0; b0 < p.B; b0 += kWave)
        total += __builtin_amdgcn_readlane(wave_scan(weight_of<ROWS>(p, b0 + lane, &bad)), kWave - 1);
    Line l;
    l.total = __any(bad) ? 0 : total;
    l.per = max(1, (l.total + p.groups - 1) / p.groups);
    return l;
}

// The sequence of unit u (u < total), or with `token` of token u (-1: none),
// and the units before it.  After line_of found the offsets in order.
template <int ROWS>
__device__ inline int sequence_at(const AttnArgs& p, int u, bool token, int* base) {
    const int lane = threadIdx.x % kWave;
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += kWave) {
        bool bad = false;
        const int b = b0 + lane, w = weight_of<ROWS>(p, b, &bad), incl = wave_scan(w);
        const int total = __builtin_amdgcn_readlane(incl, kWave - 1);
        const bool mine = token ? b < p.B && p.a.token_offsets[b] <= u && u < p.a.token_offsets[b + 1]
                                : u - before < incl && u - before >= incl - w;
        const uint64_t at = __ballot(mine);
        if (at) {
            const int l = __builtin_ctzll(at);
            *base = before + __builtin_amdgcn_readlane(incl - w, l);
            return b0 + l;
        }
        before += total;
    }
    return -1;
}

// ------------------------------------------------------------------ one wave

// How 32 positions of one head go through a wave.  In the cache a position's
// codes are D contiguous bytes.  A load takes whole lines: kLanes lanes of 16
// bytes a position, kKeys positions at a time, kLoads times (16 lanes on 16
// lines, as the matrix cores' operands would have them, cost 64 cycles a load
// in place of 16).  K lies in LDS as it came, its 16-byte pieces dealt so that
// the 16 positions of an operand read are in different banks; V lies there in
// bf16, 16 bytes between its positions for the same reason.
template <int D>
struct Tile {
    static constexpr int kLanes = D / 16, kKeys = kWave / kLanes, kLoads = 32 / kKeys;
    static constexpr int kValueRow = 2 * D + 16;           // bytes of a position's values in LDS
    static constexpr int kValues = 32 * kValueRow;         // V, then
    static constexpr int kCodes = 32 * D;                  // K, then
    static constexpr int kScales = 2 * 32 * (D / 32);      // both's scales
    static constexpr int kBytes = kValues + kCodes + kScales;
    // where piece `piece` of position `key`'s codes is
    __device__ static int code_at(int key, int piece) {
        return key * D + (piece ^ (key / (256 / D) % kLanes)) * 16;
    }
};

// 32 positions' keys and values as loaded: lane l has piece l % kLanes of
// position kKeys i + l / kLanes; the scales of position l % 32, lanes 0 .. 31
// of K, the others of V
template <int D>
struct Raw {
    u32x4_t k[Tile<D>::kLoads], v[Tile<D>::kLoads];
    uint64_t scales;  // D / 32 bytes
    bool ok[2];    // the page of the first 16 positions and of the others is one of the cache's
};

// page numbers of positions p0 .. p0+15 and p0+16 .. p0+31 (-1: none)
__device__ inline void page_numbers(const AttnArgs& p, const int32_t* table, int p0, int len, int (&page)[2]) {
#pragma unroll
    for (int t = 0; t < 2; t++) page[t] = p0 + 16 * t < len ? table[(p0 + 16 * t) >> p.page_shift] : -1;
}

template <int D>
__device__ inline void load_raw(const AttnArgs& p, int h, int p0, const int (&page)[2], Raw<D>& r) {
    using T = Tile<D>;
    const moe_kv_cache& q = p.a.cache;
    const uint32_t lane = threadIdx.x % kWave;
    int64_t at[2];
    int row[2];
#pragma unroll
    for (int t = 0; t < 2; t++) {
        const int number = uniform(page[t]);
        r.ok[t] = (uint32_t)number < (uint32_t)q.num_pages;
        at[t] = r.ok[t] ? number : 0;
        row[t] = h * q.page_size + ((p0 + 16 * t) & (q.page_size - 1));
    }
#pragma unroll
    for (int i = 0; i < T::kLoads; i++) {
        const int t = i * T::kKeys / 16;
        const int64_t code = at[t] * q.codes_page_stride + (int64_t)(row[t] + i * T::kKeys % 16) * D;
        r.k[i] = *reinterpret_cast<const u32x4_t*>(q.k_codes + code + lane * 16);
        r.v[i] = *reinterpret_cast<const u32x4_t*>(q.v_codes + code + lane * 16);
    }
    const int t = lane / 16 % 2;
    const uint8_t* s = (lane < 32 ? q.k_scales : q.v_scales) +
                       ((t ? at[1] : at[0]) * q.scales_page_stride + (int64_t)(t ? row[1] : row[0]) * (D / 32)) +
                       lane % 16 * (D / 32);
    if constexpr (D == 64) r.scales = *reinterpret_cast<const uint16_t*>(s);
    else if constexpr (D == 128) r.scales = *reinterpret_cast<const uint32_t*>(s);
    else r.scales = *reinterpret_cast<const uint64_t*>(s);
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

// A word of two bf16 values: 2^127 for each that is no finite number, else zero
__device__ inline uint32_t specials(uint32_t w) {
    return ((w & 0x7f80u) == 0x7f80u ? 0x7f00u : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? 0x7f000000u : 0u);
}

// whether 16 values hold one that is no finite number: a NaN code or scale, or
// a scale that can take one out of range
__device__ inline bool has_specials(const u32x4_t& x, uint32_t s) {
    const uint32_t nan = ((x.x & 0x7f7f7f7fu) + 0x01010101u) | ((x.y & 0x7f7f7f7fu) + 0x01010101u) |
                         ((x.z & 0x7f7f7f7fu) + 0x01010101u) | ((x.w & 0x7f7f7f7fu) + 0x01010101u);
    return (nan & 0x80808080u) || s >= 246u;
}

template <int D, int R>
struct Wave {
    // per row tile, lane (c, g): row c.  O: elements 16 d + 4 g ..
    f32x4_t o[R][D / 16], sum[R];
    float m[R], mc[R];  // the reference score, and c * m (0 while there is none)
    float pass[R];      // the score past which the reference is moved
};

// One step: 32 positions from p0.  `ahead` issues the next step's loads.
template <int D, int R, typename Ahead>
__device__ inline void step(const AttnArgs& p, const Seq& s, const int (&node)[R], const bf16x8_t (&q)[R][D / 32],
                            int p0, Raw<D>& raw, uint8_t* lds, Wave<D, R>& w, Ahead&& ahead) {
    using T = Tile<D>;
    const int lane = threadIdx.x % kWave, c = lane % 16, g = lane / 16;
    const int key = lane / T::kLanes, piece = lane % T::kLanes;  // of a load
    uint8_t *codes = lds + T::kValues, *scales = codes + T::kCodes;
    // K and the scales as they are
    if constexpr (D == 64) *reinterpret_cast<uint16_t*>(scales + lane * 2) = (uint16_t)raw.scales;
    else if constexpr (D == 128) *reinterpret_cast<uint32_t*>(scales + lane * 4) = (uint32_t)raw.scales;
    else *reinterpret_cast<uint64_t*>(scales + lane * 8) = raw.scales;
#pragma unroll
    for (int i = 0; i < T::kLoads; i++)
        *reinterpret_cast<u32x4_t*>(codes + T::code_at(T::kKeys * i + key, piece)) = raw.k[i];
    wave_order();
    // V in bf16
    uint32_t vs[T::kLoads];
#pragma unroll
    for (int i = 0; i < T::kLoads; i++) vs[i] = scales[(32 + T::kKeys * i + key) * (D / 32) + piece / 2];
    const bool ok0 = raw.ok[0], ok1 = raw.ok[1];
    // whether some of them are drafted ones or none at all; else all rows see all
    const bool special = p0 + 32 > s.L || !ok0 || !ok1;
    bool odd = false;  // a drafted token's value is no number
    if (special) {
#pragma unroll
        for (int i = 0; i < T::kLoads; i++) {
            if (!(p0 + T::kKeys * i + key < s.len && (i * T::kKeys / 16 ? ok1 : ok0))) {  // nothing is there
                raw.v[i] = u32x4_t{0, 0, 0, 0};
                vs[i] = 0;
            }
            odd |= has_specials(raw.v[i], vs[i]);
        }
        odd = __any(odd);
    }
    uint8_t* mine = lds + key * T::kValueRow + piece * 32;
#pragma unroll
    for (int i = 0; i < T::kLoads; i++) {
        const float f = e8m0_as_scale(vs[i]);
        bf16x8_t* at = reinterpret_cast<bf16x8_t*>(mine + T::kKeys * i * T::kValueRow);
        at[0] = decode8_e4m3(raw.v[i].x, raw.v[i].y, f);
        at[1] = decode8_e4m3(raw.v[i].z, raw.v[i].w, f);
    }
    wave_order();
    ahead();

    f32x4_t st[2][R];
#pragma unroll
    for (int t = 0; t < 2; t++) {
#pragma unroll
        for (int r = 0; r < R; r++) st[t][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        // lane (c, g): quarter g of position 16 t + c
        uint32_t ks = 0;
        if constexpr (D == 64) ks = scales[(16 * t + c) * 2 + g / 2];
        else if constexpr (D == 128) ks = scales[(16 * t + c) * 4 + g];
        else ks = *reinterpret_cast<const uint16_t*>(scales + (16 * t + c) * 8 + 2 * g);
#pragma unroll
        for (int j = 0; j < D / 64; j++) {
            const uint4 x = *reinterpret_cast<const uint4*>(codes + T::code_at(16 * t + c, g * (D / 64) + j));
            const float f = e8m0_as_scale(D == 256 ? (j < 2 ? ks & 0xffu : ks >> 8) : ks);
            const bf16x8_t k0 = decode8_e4m3(x.x, x.y, f), k1 = decode8_e4m3(x.z, x.w, f);
#pragma unroll
            for (int r = 0; r < R; r++) st[t][r] = mfma(k0, q[r][2 * j], st[t][r]);
#pragma unroll
            for (int r = 0; r < R; r++) st[t][r] = mfma(k1, q[r][2 * j + 1], st[t][r]);
        }
    }
    typedef __attribute__((address_space(3))) s16x4_t lds4_t;
    const uint8_t* column = lds + (4 * g + c / 4) * T::kValueRow + (c % 4) * 8;
    auto value = [&](int d) {
        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4_t*)(column + 32 * d));
        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4_t*)(column + 16 * T::kValueRow + 32 * d));
        const s16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        return __builtin_bit_cast(bf16x8_t, v);
    };
    // the first of the product's operands are on their way before the softmax
    constexpr int kAhead = 4;
    bf16x8_t vt[kAhead];
#pragma unroll
    for (int d = 0; d < kAhead; d++) vt[d] = value(d);
    __builtin_amdgcn_sched_barrier(0);
    uint32_t seen[R];
    if (special) {
#pragma unroll
        for (int r = 0; r < R; r++) {
            seen[r] = seen_bits(p, s, node[r], p0, ok0, ok1) >> (4 * g);
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
            float t = top[r];
            t = fmaxf(t, __shfl_xor(t, 16));
            t = fmaxf(t, __shfl_xor(t, 32));
            const float m = fmaxf(w.m[r], t), mc = m == minus_inf() ? 0.f : m * p.c;
            const float f = w.m[r] == minus_inf() ? 0.f : __builtin_amdgcn_exp2f(w.mc[r] - mc);
#pragma unroll
            for (int d = 0; d < D / 16; d++) w.o[r][d] *= f;
            w.sum[r] *= f;
            w.m[r] = m;
            w.mc[r] = mc;
            w.pass[r] = m + kAttnSlack / p.c;
        }
    }
    bf16x8_t pt[R];
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                pt[r][4 * t + i] = (__bf16)__builtin_amdgcn_exp2f(fmaf(st[t][r][i], p.c, -w.mc[r]));
    const s16x8_t one16 = {0x3f80, 0x3f80, 0x3f80, 0x3f80, 0x3f80, 0x3f80, 0x3f80, 0x3f80};
    const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, one16);
#pragma unroll
    for (int r = 0; r < R; r++) w.sum[r] = mfma(ones, pt[r], w.sum[r]);

    if (odd) {
        // A value that is no number makes one of what sees it, and of
        // nothing else.  2^127 in its place is multiplied with 2^127 where
        // it is seen, and with the negative: infinity, then infinity less
        // infinity.  For the product below it is then zero.
#pragma unroll
        for (int r = 0; r < R; r++) {
            auto pair = [&](int k) {  // of positions k, k + 1
                return 0x7f00u * (seen[r] >> k & 1u) | 0x7f000000u * (seen[r] >> (k + 1) & 1u);
            };
            const uint4 sees = make_uint4(pair(0), pair(2), pair(16), pair(18));
#pragma unroll
            for (int d = 0; d < D / 16; d++) {
                const uint4 v = __builtin_bit_cast(uint4, value(d));
                const uint4 n = make_uint4(specials(v.x), specials(v.y), specials(v.z), specials(v.w));
                const uint4 m = make_uint4(n.x | (n.x << 1 & 0x80008000u), n.y | (n.y << 1 & 0x80008000u),
                                           n.z | (n.z << 1 & 0x80008000u), n.w | (n.w << 1 & 0x80008000u));
                w.o[r][d] = mfma(__builtin_bit_cast(bf16x8_t, n), __builtin_bit_cast(bf16x8_t, sees), w.o[r][d]);
                w.o[r][d] = mfma(__builtin_bit_cast(bf16x8_t, m), __builtin_bit_cast(bf16x8_t, sees), w.o[r][d]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        wave_order();
#pragma unroll 1
        for (int i = 0; i < 2 * T::kLoads; i++) {
            uint4* at = reinterpret_cast<uint4*>(mine + i / 2 * T::kKeys * T::kValueRow + i % 2 * 16);
            const uint4 v = *at;
            auto clean = [](uint32_t x) { const uint32_t n = specials(x);
                return x & ~((n & 0x4000u ? 0xffffu : 0u) | (n & 0x40000000u ? 0xffff0000u : 0u)); };
            *at = make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
        }
        wave_order();
#pragma unroll
        for (int d = 0; d < kAhead; d++) vt[d] = value(d);
    }
#pragma unroll
    for (int d = 0; d < D / 16; d++) {
#pragma unroll
        for (int r = 0; r < R; r++) w.o[r][d] = mfma(vt[d % kAhead], pt[r], w.o[r][d]);
        if (d + kAhead < D / 16) vt[d % kAhead] = value(d + kAhead);
    }
    wave_order();
}

// the statistic of rows without a position is -infinity: their weight is 0
__device__ inline float reference(float m) { return m == minus_inf() ? 0.f : m; }

// A workgroup's shape: WR groups of 16 R rows times WK runs of positions, a
// wave each.
template <int D_, int R_, int WR_, int WK_>
struct Shape {
    static constexpr int D = D_, R = R_, WR = WR_, WK = WK_;
    static constexpr int kRows = 16 * R * WR, kWaves = WR * WK, kThreads = kWave * kWaves;
    // a wave's 32 positions; at the end the waves' results, 16 rows of each
    static constexpr int kTile = Tile<D>::kBytes, kResult = 16 * (D + 4) * 4;
    static constexpr int kLds = kWaves * (kTile > kResult ? kTile : kResult);
    // waves per SIMD that the registers leave room for
    static constexpr int kPerSimd = D == 256 ? 1 : D * R <= 128 ? 3 : 2;
};

template <typename S>
__global__ void __launch_bounds__(S::kThreads, S::kPerSimd) tree_attention_kernel(AttnArgs p) {
    constexpr int D = S::D, R = S::R, WR = S::WR, WK = S::WK, ROWS = S::kRows;
    __shared__ __align__(16) uint8_t buf[S::kLds];
    __shared__ float s_m[WK][ROWS], s_sum[S::kWaves][16];
    const int tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave), c = lane % 16, g = lane / 16;
    const int wr = wave / WK, wk = wave % WK;
    // Workgroups are dealt round the 8 XCDs; each XCD takes a run of the line, so
    // that the row tiles of a head, which read the same positions, share its L2
    const int group = (int)blockIdx.x % 8 * (p.groups / 8) + (int)blockIdx.x / 8;
    const Line line = line_of<ROWS>(p);
    int u = uniform(group * line.per);
    const int end = uniform(min(u + line.per, line.total));
    if (u >= end) return;
    int base = 0;
    int b = uniform(sequence_at<ROWS>(p, u, false, &base));
    base = uniform(base);
    while (u < end) {
        Seq s = read_seq(p, b);
        s.first = uniform(s.first), s.n = uniform(s.n), s.L = uniform(s.L), s.len = uniform(s.len);
        const int tiles = tiles_of<ROWS>(p, s), units = units_of(s), all = s.n ? tiles * units * p.a.cache.kv_heads : 0;
        if (u - base >= all) {  // on to the next sequence (there is one: u < total)
            base += all;
            b++;
            continue;
        }
        const int item = (u - base) / units, u0 = (u - base) % units, u1 = min(units, u0 + end - u);
        const int h = item / tiles, row0 = item % tiles * ROWS, rows = s.n * p.G;

        int node[R];
        bf16x8_t q[R][D / 32];
        Wave<D, R> w;
#pragma unroll
        for (int r = 0; r < R; r++) {
            const int row = row0 + 16 * (R * wr + r) + c, live = row < rows;
            node[r] = (live ? row : rows - 1) / p.G;
            const uint16_t* src = (const uint16_t*)p.a.q + (int64_t)(s.first + node[r]) * p.a.q_stride +
                                  (h * p.G + (live ? row % p.G : 0)) * D + g * (D / 4);
#pragma unroll
            for (int j = 0; j < D / 32; j++) {
                const uint4 x = live ? reinterpret_cast<const uint4*>(src)[j] : make_uint4(0, 0, 0, 0);
                q[r][j] = __builtin_bit_cast(bf16x8_t, x);
            }
#pragma unroll
            for (int d = 0; d < D / 16; d++) w.o[r][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            w.sum[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            w.m[r] = minus_inf();
            w.mc[r] = 0.f;
            w.pass[r] = minus_inf();
        }
        // positions that some row of the wave may see
        int stop = s.len;
        if (!p.a.mask) stop = min(stop, s.L + (min(row0 + 16 * R * (wr + 1), rows) - 1) / p.G + 1);
        stop = row0 + 16 * R * wr < rows ? min(stop, u1 * kAttnUnit) : 0;
        const int32_t* table = p.a.block_table + (int64_t)b * p.a.block_table_stride;
        int p0 = u0 * kAttnUnit + 32 * wk;
        if (p0 < stop) {
            Raw<D> raw;
            int page[2];
            page_numbers(p, table, p0, s.len, page);
            load_raw<D>(p, h, p0, page, raw);
            page_numbers(p, table, p0 + 32 * WK, s.len, page);
            uint8_t* lds = buf + wave * S::kTile;
            for (; p0 < stop; p0 += 32 * WK) {
                auto ahead = [&] {
                    const int next = p0 + 32 * WK;
                    if (next < stop) {
                        load_raw<D>(p, h, next, page, raw);
                        page_numbers(p, table, next + 32 * WK, s.len, page);
                    }
                };
                step<D, R>(p, s, node, q, p0, raw, lds, w, ahead);
            }
        }

        // the results of the waves of a row group joined, 16 rows of each group at a time
        if (g == 0)
#pragma unroll
            for (int r = 0; r < R; r++)
                s_m[wk][16 * (R * wr + r) + c] = w.m[r] == minus_inf() ? minus_inf() : w.mc[r];
        __syncthreads();
        auto top_of = [&](int row) {
            float m = s_m[0][row];
#pragma unroll
            for (int i = 1; i < WK; i++) m = fmaxf(m, s_m[i][row]);
            return m;
        };
        const bool whole = u0 == 0 && u1 == units;
        float* part = (float*)p.a.workspace + (2 * (int64_t)group + (u0 ? 0 : 1)) * p.part_floats;
        float* joined = reinterpret_cast<float*>(buf);
        constexpr int kPiece = D * 16 * WR / S::kThreads, kPieces = D / kPiece;  // of a row: elements of a thread, threads
#pragma unroll
        for (int r = 0; r < R; r++) {
            const float f = __builtin_amdgcn_exp2f((w.m[r] == minus_inf() ? minus_inf() : w.mc[r]) -
                                                   reference(top_of(16 * (R * wr + r) + c)));
            float* mine = joined + (wave * 16 + c) * (D + 4) + 4 * g;
#pragma unroll
            for (int d = 0; d < D / 16; d++)
                *reinterpret_cast<f32x4_t*>(mine + 16 * d) = w.o[r][d] * f;
            if (g == 0) s_sum[wave][c] = w.sum[r][0] * f;
            __syncthreads();
            const int og = tid / (16 * kPieces), orow = tid / kPieces % 16, d0 = tid % kPieces * kPiece;
            const int at = 16 * (R * og + r) + orow;
            float v[kPiece] = {}, sum = 0.f;
#pragma unroll
            for (int i = 0; i < WK; i++) {
                sum += s_sum[og * WK + i][orow];
#pragma unroll
                for (int d = 0; d < kPiece; d++) v[d] += joined[((og * WK + i) * 16 + orow) * (D + 4) + d0 + d];
            }
            if (!whole) {
                float* dst = part + at * D + d0;
#pragma unroll
                for (int d = 0; d < kPiece; d++) dst[d] = v[d];
                if (d0 == 0) {
                    part[ROWS * D + 2 * at] = top_of(at);
                    part[ROWS * D + 2 * at + 1] = sum;
                }
            } else if (row0 + at < rows) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                uint16_t* dst = (uint16_t*)p.a.out + (int64_t)(s.first + (row0 + at) / p.G) * p.a.out_stride +
                                (h * p.G + (row0 + at) % p.G) * D + d0;
#pragma unroll
                for (int d = 0; d < kPiece; d += 4) {
                    const float o[4] = {v[d] * inv, v[d + 1] * inv, v[d + 2] * inv, v[d + 3] * inv};
                    store_piece<4>(dst + d, o);
                }
            }
            __syncthreads();
        }
        u += u1 - u0;
    }
}

// One wave per row: the parts of a row tile that several workgroups did, in
// their order.  A part's weight is 2^(its reference - the largest).
template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinWaves * kWave) tree_attention_join_kernel(AttnArgs p) {
    constexpr int N = D / kWave;
    const int lane = threadIdx.x % kWave;
    const int idx = uniform((int)blockIdx.x * kJoinWaves + (int)threadIdx.x / kWave);
    if (idx >= p.T * p.a.num_heads) return;
    const int token = idx / p.a.num_heads, head = idx % p.a.num_heads;
    const Line line = line_of<ROWS>(p);
    if (line.total == 0) return;
    int base = 0;
    const int b = uniform(sequence_at<ROWS>(p, token, true, &base));
    if (b < 0) return;
    const Seq s = read_seq(p, b);
    const int units = units_of(s), row = (token - s.first) * p.G + head % p.G, at = row % ROWS;
    const int u0 = base + (head / p.G * tiles_of<ROWS>(p, s) + row / ROWS) * units;
    const int first = u0 / line.per, parts = (u0 + units - 1) / line.per - first + 1;
    if (parts == 1) return;
    auto part = [&](int i) {
        return (const float*)p.a.workspace + (2 * (int64_t)(first + i) + (i ? 0 : 1)) * p.part_floats;
    };
    float top = minus_inf();
    for (int i = lane; i < parts; i += kWave) top = fmaxf(top, part(i)[ROWS * D + 2 * at]);
#pragma unroll
    for (int x = 1; x < kWave; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
    top = reference(top);
    float v[N] = {}, sum = 0.f;
    for (int i0 = 0; i0 < parts; i0 += kWave) {
        float f = 0.f, l = 0.f;
        if (i0 + lane < parts) {
            const float* stat = part(i0 + lane) + ROWS * D + 2 * at;
            f = __builtin_amdgcn_exp2f(stat[0] - top);
            l = stat[1] * f;
        }
        const int n = min(parts - i0, kWave);
        for (int i = 0; i < n; i++) {
            const float fi = __shfl(f, i);
            sum += __shfl(l, i);
            const float* src = part(i0 + i) + at * D + lane * N;
#pragma unroll
            for (int e = 0; e < N; e++) v[e] = fmaf(src[e], fi, v[e]);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* dst = (uint16_t*)p.a.out + (int64_t)token * p.a.out_stride + head * D + lane * N;
#pragma unroll
    for (int e = 0; e < N; e++) dst[e] = f32_to_bf16_rne(v[e] * inv);
}

template <int D, int R, int WR, int WK>
hipError_t launch_shape(const AttnArgs& p, hipStream_t stream) {
    using S = Shape<D, R, WR, WK>;
    tree_attention_kernel<S><<<p.groups, S::kThreads, 0, stream>>>(p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const unsigned blocks = ((unsigned)p.T * p.a.num_heads + kJoinWaves - 1) / kJoinWaves;
    tree_attention_join_kernel<D, S::kRows><<<blocks, kJoinWaves * kWave, 0, stream>>>(p);
    return hipGetLastError();
}

template <int D, int W>  // W: waves of the larger shapes
hipError_t launch_rows(const AttnArgs& p, int rows, hipStream_t stream) {
    switch (rows) {
        case 16: return launch_shape<D, 1, 1, 4>(p, stream);
        case 32: return launch_shape<D, 2, 1, 4>(p, stream);
        case 64: return launch_shape<D, 2, 2, W / 2>(p, stream);
        default: return launch_shape<D, 2, 4, W / 4>(p, stream);
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
    p.page_shift = __builtin_ctz(a.cache.page_size);
    p.capacity = (int)(a.max_pages * a.cache.page_size);
    p.groups = plan.groups;
    p.c = a.scale * 1.44269504088896340736f;
    p.part_floats = plan.part_floats;
    switch (a.cache.head_dim) {
        case 64: return launch_rows<64, 8>(p, plan.rows, stream);
        case 128: return launch_rows<128, 8>(p, plan.rows, stream);
        default: return launch_rows<256, 4>(p, plan.rows, stream);
    }
}

}  // namespace moe

// ln_mask.cuh -- the dropout mask, drawn wherever it is needed and never
// stored: the generator, and the form in which kernels apply it to packed
// fp32 pairs.
//
// Generator.  Philox4x32-10: J. Salmon, M. Moraes, R. Dror, D. Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011 (ten rounds are the
// paper's recommended safety margin).  Elements are numbered in memory order;
// element e belongs to group e / 8 and owns 16 bits of
//   Philox(key = (seed lo, seed hi), counter = (group lo, group hi, o lo, o hi)),
//   o = offset + *step (mod 2^64):
// half e % 2 of word (e % 8) / 2.  An element is kept where its 16 bits are at
// least T = round(65536 p).  A mask bit therefore depends on the keys and the
// element's index alone: not on the type, the kernel, the grid or alignment.
//
// Why 16 bits per element.  One Philox evaluation (20 wide multiplies and 20
// three-way xors) then serves eight elements, i.e. one 16-byte vector of a
// 16-bit type: about 7 integer instructions per element.  With 32 bits per
// element that doubles, and the elementwise kernel would leave the memory
// roofline (bf16: about 6 elements per clock and SM at the measured copy
// bandwidth).  A 16-byte vector of fp32 is half a group: the fused calls draw a
// group in both lanes that hold its halves, twice the work per element, for half
// the elements per byte; ln_dropout gives a thread whole groups and draws each
// once, and the scalar kernels draw one evaluation per element.  T / 65536 differs from p by at most 2^-17; kept elements are
// scaled by 65536 / (65536 - T), so the result stays unbiased for the rate
// actually drawn.
#pragma once

#include "ln_vec.cuh"

namespace lnk {

// What a kernel needs of the keys (filled in on the host, passed by value).
// The round keys and multipliers are kernel parameters, so that a round's xor
// and multiply read them from the constant bank: no instruction and no register
// goes into the key schedule.
constexpr int kPhiloxRounds = 10;
struct DropKeys {
    uint32_t key[2 * kPhiloxRounds];
    uint32_t mul[2];
    uint64_t offset;
    const uint64_t *step;   // device counter added to offset, or NULL
    uint32_t threshold;     // T in both halves
    float scale;            // 65536 / (65536 - T); 0 when nothing is kept
};
// T = 65536 (nothing is kept) does not fit 16 bits: then multipliers and round
// keys are zero, which makes every word zero after two rounds, and the
// threshold is 1.
inline DropKeys make_keys(uint32_t T, uint64_t seed, uint64_t offset, const uint64_t *step) {
    DropKeys k = {};
    const bool some = T < 65536u;
    uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
    for (int r = 0; some && r < kPhiloxRounds; ++r) {
        k.key[2 * r] = k0;
        k.key[2 * r + 1] = k1;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    k.mul[0] = some ? 0xD2511F53u : 0u;
    k.mul[1] = some ? 0xCD9E8D57u : 0u;
    k.offset = offset;
    k.step = step;
    k.threshold = (some ? T : 1u) * 0x10001u;
    k.scale = some ? float(65536.0 / double(65536u - T)) : 0.f;
    return k;
}

// The keys of one launch, with the counter read (after griddepcontrol.wait,
// so a counter written earlier on the stream is seen).
struct Mask {
    const DropKeys &k;
    uint32_t o_lo, o_hi;
    float scale;
};
__device__ __forceinline__ Mask make_mask(const DropKeys &k) {
    const uint64_t o = k.offset + (k.step ? *k.step : 0u);
    return Mask{k, uint32_t(o), uint32_t(o >> 32), k.scale};
}

// Philox4x32-10 of one group: the 128 bits of elements 8g .. 8g + 7.
__device__ __forceinline__ uint4 mask_bits(const Mask &m, uint64_t g) {
    uint32_t c0 = uint32_t(g), c1 = uint32_t(g >> 32), c2 = m.o_lo, c3 = m.o_hi;
#pragma unroll
    for (int r = 0; r < kPhiloxRounds; ++r) {
        const uint64_t a = uint64_t(m.k.mul[0]) * c0;
        const uint64_t b = uint64_t(m.k.mul[1]) * c2;
        c0 = uint32_t(b >> 32) ^ c1 ^ m.k.key[2 * r];
        c1 = uint32_t(b);
        c2 = uint32_t(a >> 32) ^ c3 ^ m.k.key[2 * r + 1];
        c3 = uint32_t(a);
    }
    return make_uint4(c0, c1, c2, c3);
}

// Whether the elements in the low and high half of a word are kept: one
// two-way 16-bit maximum, which also says of each half whether the word's was
// the larger.  Measured on B200 against a shift and two 32-bit comparisons: 9.6
// instructions per pair of a loop that selects by them instead of 13.8.
__device__ __forceinline__ void keep2(const Mask &m, uint32_t word, bool &lo, bool &hi) {
    (void)__vibmax_u16x2(word, m.k.threshold, &hi, &lo);
}

// The words of the P pairs of 16-byte vector number `vec` (counted over the
// whole array; arrays of this form start on a vector boundary).  A vector of
// a 16-bit type is one group; a vector of fp32 is half a group.
template <typename T>
__device__ __forceinline__ void vec_words(const Mask &m, int64_t vec,
                                          uint32_t (&w)[Vec<T>::E / 2]) {
    if constexpr (Vec<T>::E == 8) {
        const uint4 b = mask_bits(m, uint64_t(vec));
        w[0] = b.x;
        w[1] = b.y;
        w[2] = b.z;
        w[3] = b.w;
    } else {
        const uint4 b = mask_bits(m, uint64_t(vec) >> 1);
        w[0] = (vec & 1) ? b.z : b.x;
        w[1] = (vec & 1) ? b.w : b.y;
    }
}

// dropout of a pair: kept elements times the scale, dropped ones exactly zero
// whatever their value (a selection, so that an infinity or a NaN in a dropped
// place leaves no trace).
__device__ __forceinline__ f32x2 drop2(const Mask &m, uint32_t word, f32x2 v) {
    float lo, hi;
    bool keep_lo, keep_hi;
    split(mul2(v, pair(m.scale, m.scale)), lo, hi);
    keep2(m, word, keep_lo, keep_hi);
    return pair(keep_lo ? lo : 0.f, keep_hi ? hi : 0.f);
}
// base + dropout of a pair.  The product is rounded to fp32 before the sum
// rather than fused into it: the scale is itself rounded, and rounding the
// product undoes that where the true product has few bits (p = 1/4, scale
// 4/3, a branch that 3 divides), while a fused sum carries the scale's error
// past the ties of a 16-bit result (fp16, p = 1/4: 0.34 % of the elements one
// step off; rounded first: 0.007 %).
__device__ __forceinline__ f32x2 drop_add2(const Mask &m, uint32_t word, f32x2 v, f32x2 base) {
    return add2(base, drop2(m, word, v));
}

// resid + dropout(branch) for a vector with mask words `w`, each element
// rounded to T.
template <typename T>
__device__ __forceinline__ uint4 drop_add_round(const Mask &m, const uint32_t (&w)[Vec<T>::E / 2],
                                                const uint4 &resid, const uint4 &branch) {
    constexpr int P = Vec<T>::E / 2;
    f32x2 r[P], b[P];
    to_pairs<T>(resid, r);
    to_pairs<T>(branch, b);
#pragma unroll
    for (int q = 0; q < P; ++q) r[q] = drop_add2(m, w[q], b[q], r[q]);
    return from_pairs<T>(r);
}

// A 16-bit vector's mask in one word, for a warp that draws it for another:
// element k is kept where bit 7 of byte k is set (k < 4), or bit 6 of byte
// k - 4.  pack_mask makes it; mask_pair widens it to the 32 bits of pair q, all
// ones where kept, with one byte permutation that replicates sign bits.
__device__ __forceinline__ uint32_t pack_mask(const Mask &m, const uint4 &b) {
    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
    uint32_t r = 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        bool lo, hi;
        keep2(m, w[q], lo, hi);
        const uint32_t bit = (q < 2 ? 0x80u : 0x40u) << (q & 1 ? 16 : 0);
        r |= lo ? bit : 0u;
        r |= hi ? bit << 8 : 0u;
    }
    return r;
}
__device__ __forceinline__ uint32_t mask_pair(uint32_t packed, int q) {
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;"
        : "=r"(r)
        : "r"(q < 2 ? packed : packed << 1), "r"(q & 1 ? 0xBBAAu : 0x9988u));
    return r;
}
// dbranch = dropout(dx) for vector number `vec` of a 16-bit array by its packed
// mask: the scaled and rounded pair, with the dropped halves cleared.
template <typename T>
__device__ __forceinline__ void store_dbranch_packed(float scale, uint32_t packed, T *dbranch,
                                                     int64_t vec, const f32x2 (&dx)[4]) {
    static_assert(Vec<T>::E == 8, "16-bit types");
    f32x2 y[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = mul2(dx[q], pair(scale, scale));
    uint4 v = from_pairs<T>(y);
    v.x &= mask_pair(packed, 0);
    v.y &= mask_pair(packed, 1);
    v.z &= mask_pair(packed, 2);
    v.w &= mask_pair(packed, 3);
    __stcs(reinterpret_cast<uint4 *>(dbranch) + vec, v);
}

// What a backward kernel with MODE & kBwdDropout needs besides the arguments
// of the plain one (unused in the other modes).
template <typename T>
struct DropOut {
    T *dbranch;         // gradient of the dropped-out summand
    const T *prev;      // kBwdAccumulate: the gradient that reaches x from elsewhere
    DropKeys keys;
};
// dbranch = dropout(dx) for vector number `vec`, dx in fp32.
template <typename T>
__device__ __forceinline__ void store_dbranch(const Mask &m, T *dbranch, int64_t vec,
                                              const f32x2 (&dx)[Vec<T>::E / 2]) {
    constexpr int P = Vec<T>::E / 2;
    uint32_t w[P];
    f32x2 y[P];
    vec_words<T>(m, vec, w);
#pragma unroll
    for (int q = 0; q < P; ++q) y[q] = drop2(m, w[q], dx[q]);
    __stcs(reinterpret_cast<uint4 *>(dbranch) + vec, from_pairs<T>(y));
}

// Whether element e of the array is kept (scalar paths).
__device__ __forceinline__ bool keep_element(const Mask &m, int64_t e) {
    const uint4 b = mask_bits(m, uint64_t(e) >> 3);
    const uint32_t w = (e & 4) ? ((e & 2) ? b.w : b.z) : ((e & 2) ? b.y : b.x);
    bool lo, hi;
    keep2(m, w, lo, hi);
    return (e & 1) ? hi : lo;
}
// resid + dropout(branch) of one element, rounded to T: the value
// drop_add_round gives it.
template <typename T>
__device__ __forceinline__ float drop_add_round1(const Mask &m, int64_t e, T resid, T branch) {
    const float y = keep_element(m, e) ? __fmul_rn(to_f32(branch), m.scale) : 0.f;
    return to_f32(from_f32<T>(__fadd_rn(to_f32(resid), y)));
}

}  // namespace lnk

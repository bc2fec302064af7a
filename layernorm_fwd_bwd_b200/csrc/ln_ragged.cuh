// ln_ragged.cuh -- the dropout-residual forward and backward for rows of any
// length (arrays that start on a 16-byte boundary), for narrow rows, for
// backward calls of few rows, and for backward rows wider than the ring kernels
// serve.
//
// Operation: as ln_forward_dropout_residual and ln_backward_dropout_residual in
// include/ln.h state; arithmetic as in ln_kernels.cuh, mask from ln_mask.cuh.
//
// Why kernels of their own.  Row r starts at element r * C of its array, so
// when C is no multiple of 16 bytes most rows start inside a 16-byte vector,
// and the mask's groups of 8 elements straddle rows.  The scalar kernels take
// such rows an element at a time and draw the mask once per element.  Here a
// row is taken as the aligned vectors that cover it: row r has shift
// sh = (r * C) % E, covers nv = ceil((sh + C) / E) vectors, and its first and
// last vector may be shared with its neighbours.  Vectors are loaded whole (the
// array's very last one element by element where it is cut off), elements
// outside the row are set to zero before they are used and left out of every
// sum and store, and a vector is again one mask group (16-bit types; half a
// group in fp32).
//
// The shift is fixed per row group: rows are dealt out with a step that is a
// multiple of 8, and 8 * C is a multiple of E.  So each group keeps weight (and
// bias) in shared memory already shifted to its vectors, and the backward's
// column sums stay in registers, tied to fixed columns, as in the other
// kernels.
//
// L lanes share a row: 8 or 16 (several rows per warp: rows of up to 8 or 16
// vectors, where a whole warp per row would idle), 32, or several warps.
//
// What bounds them: memory and the instructions of a row, on a persistent grid.
// The forward loads whole rows into registers (up to 5 vectors of both arrays
// per lane); the backward, whose column sums take its registers, copies each
// group's next row to shared memory while it works on the current one.
#pragma once

#include "ln_kernels.cuh"
#include "ln_mask.cuh"

namespace lnk {

// Rows of up to so many vectors' elements take these kernels (several rows per
// warp) also where a whole number of vectors would suit the others.
constexpr int kNarrowVecs = 16;

// Most vectors that a row of C elements can cover.
template <typename T>
__host__ __device__ constexpr int ragged_vecs(int C) {
    return C % Vec<T>::E == 0 ? C / Vec<T>::E : (C + 2 * Vec<T>::E - 2) / Vec<T>::E;
}
template <typename T, int L, int GROUPS>
__host__ __device__ constexpr size_t fwd_ragged_smem(int C) {
    // weight and bias of every group, shifted to its vectors, and its slots
    return size_t(GROUPS) * 2 * ragged_vecs<T>(C) * 16 + (L > 32 ? size_t(GROUPS) * 3 * L / 8 : 0);
}
// Copies of the weight that a block of GROUPS row groups needs: one per shift
// (groups 8 apart share it).
template <int GROUPS>
__host__ __device__ constexpr int ragged_copies() {
    return GROUPS < 8 ? GROUPS : 8;
}
// Bytes of the backward's shared memory before its stages: the fp32 weight
// copies and the row groups' slots.
template <typename T, int L, int GROUPS>
__host__ __device__ constexpr size_t bwd_ragged_fixed(int C) {
    return size_t(ragged_copies<GROUPS>()) * ragged_vecs<T>(C) * Vec<T>::E * 4 +
           (L > 32 ? size_t(GROUPS) * L / 2 : 0);
}
// Two stages per group of NS arrays' rows; at the end every group's column
// sums (in its vectors' places, so that a lane stores whole vectors: by columns
// its scalar stores would meet 8 deep in the same banks, 3 us a launch) and the
// block's 2C lie over all of it.
template <typename T, int L, int GROUPS, int NS>
__host__ __device__ constexpr size_t bwd_ragged_smem(int C) {
    const size_t run = bwd_ragged_fixed<T, L, GROUPS>(C) +
                       size_t(GROUPS) * 2 * NS * ragged_vecs<T>(C) * 16;
    const size_t end = (size_t(GROUPS) * 2 * ragged_vecs<T>(C) * Vec<T>::E + 2 * size_t(C)) * 4;
    return run > end ? run : end;
}

// 16-byte asynchronous copy global -> shared of the first `bytes` (1 .. 16), zeros
// behind; committed in groups that the issuing thread waits for.
__device__ __forceinline__ void copy_async16(void *dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Sums over the L lanes of a row.
template <int L, int GROUPS>
__device__ __forceinline__ void row_sum2(float &a, float &b, float *slot, int group, int warp,
                                         int lane) {
    if constexpr (L >= 32) {
        group_sum2<L / 32, GROUPS>(a, b, slot, group, warp, lane);
    } else {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
    }
}
template <int L, int GROUPS>
__device__ __forceinline__ float row_sum(float v, float *slot, int group, int warp, int lane) {
    if constexpr (L >= 32) {
        return group_sum<L / 32, GROUPS>(v, slot, group, warp, lane);
    } else {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
}

// The part [lo, hi) of a vector that lies in the row, as bit masks, as factors
// for pair q, and for loads and stores.
template <typename T>
__device__ __forceinline__ uint4 inside_bits(int lo, int hi) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (Vec<T>::E == 4) {
            w[q] = q >= lo && q < hi ? 0xffffffffu : 0u;
        } else {
            w[q] = (2 * q >= lo && 2 * q < hi ? 0x0000ffffu : 0u) |
                   (2 * q + 1 >= lo && 2 * q + 1 < hi ? 0xffff0000u : 0u);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 and4(const uint4 &a, const uint4 &b) {
    return make_uint4(a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w);
}
__device__ __forceinline__ uint4 select4(const uint4 &m, const uint4 &a, uint32_t b) {
    return make_uint4((a.x & m.x) | (b & ~m.x), (a.y & m.y) | (b & ~m.y),
                      (a.z & m.z) | (b & ~m.z), (a.w & m.w) | (b & ~m.w));
}
// A value of T in every place of a word.
template <typename T>
__device__ __forceinline__ uint32_t spread(float v) {
    if constexpr (Vec<T>::E == 4) {
        return __float_as_uint(v);
    } else {
        const T e = from_f32<T>(v);
        uint16_t h;
        memcpy(&h, &e, 2);
        return h * 0x10001u;
    }
}
__device__ __forceinline__ f32x2 inside_pair(int q, int lo, int hi) {
    return pair(2 * q >= lo && 2 * q < hi ? 1.f : 0.f,
                2 * q + 1 >= lo && 2 * q + 1 < hi ? 1.f : 0.f);
}
// The array's cut-off last vector (elements vec * E .. total - 1), zeros behind.
template <typename T>
__device__ __forceinline__ uint4 load_cut(const T *p, int64_t vec, int64_t total) {
    constexpr int E = Vec<T>::E;
    T part[E];
#pragma unroll
    for (int k = 0; k < E; ++k)
        part[k] = vec * E + k < total ? p[vec * E + k] : from_f32<T>(0.f);
    uint4 v;
    memcpy(&v, part, 16);
    return v;
}
// Elements [lo, hi) of vector `vec`.
template <typename T>
__device__ __forceinline__ void store_part(T *p, int64_t vec, const uint4 &v, int lo, int hi) {
    constexpr int E = Vec<T>::E;
    T part[E];
    memcpy(part, &v, 16);
#pragma unroll
    for (int k = 0; k < E; ++k)
        if (k >= lo && k < hi) p[vec * E + k] = part[k];
}

// How a row group's rows lie on the vectors, and lane t's part of them: vector
// j = t + L * i for i < V, V = ceil(most vectors / L).  So the rounds before the
// last are whole, and only rounds 0, V - 2 and V - 1 can meet the row's ends.
template <typename T, int L, int V>
struct RowSpan {
    static constexpr int E = Vec<T>::E;
    int sh, C, nv, t;
    bool first, last;      // whether the first / last vector lies partly outside
    __device__ __forceinline__ RowSpan(int64_t r, int C_, int t_)
        : sh(int((r * C_) % E)), C(C_), nv((sh + C_ + E - 1) / E), t(t_), first(sh != 0),
          last((sh + C_) % E != 0) {}
    __device__ __forceinline__ int j(int i) const { return t + L * i; }
    __device__ __forceinline__ bool in(int i) const { return i < V - 1 || j(i) < nv; }
    __device__ __forceinline__ bool edge(int i) const {
        return (i == 0 && t == 0 && first) || (i >= V - 2 && j(i) == nv - 1 && last);
    }
    __device__ __forceinline__ int lo(int i) const { return i == 0 && t == 0 ? sh : 0; }
    __device__ __forceinline__ int hi(int i) const {
        const int left = sh + C - j(i) * E;
        return left < E ? left : E;
    }
    // Vector v0 + j(i); outside the row it may hold a neighbour's elements.
    __device__ __forceinline__ uint4 load(const T *p, int64_t v0, int i, int64_t total) const {
        const int64_t vec = v0 + j(i);
        if (i >= V - 2 && vec * E + E > total) return load_cut(p, vec, total);
        return __ldcs(reinterpret_cast<const uint4 *>(p) + vec);
    }
    // The same vector, asynchronously, to `dst`.
    __device__ __forceinline__ void load_async(uint4 *dst, const T *p, int64_t v0, int i,
                                               int64_t total) const {
        const int64_t vec = v0 + j(i);
        int bytes = 16;
        if (i >= V - 2) {
            const int64_t left = (total - vec * E) * int64_t(sizeof(T));
            bytes = left < 16 ? int(left) : 16;
        }
        copy_async16(dst, reinterpret_cast<const uint4 *>(p) + vec, bytes);
    }
    __device__ __forceinline__ void store(T *p, int64_t v0, int i, const uint4 &v) const {
        if (edge(i))
            store_part(p, v0 + j(i), v, lo(i), hi(i));
        else
            __stcs(reinterpret_cast<uint4 *>(p) + v0 + j(i), v);
    }
    // zeros outside the row
    __device__ __forceinline__ uint4 only(int i, const uint4 &v) const {
        return edge(i) ? and4(v, inside_bits<T>(lo(i), hi(i))) : v;
    }
    // one of the vector's own elements of the row in the places outside it: the
    // last in the row's first vector, else the first (V > 1: the row goes on past
    // its first vector)
    __device__ __forceinline__ uint4 only_own(int i, const uint4 &v) const {
        static_assert(V > 1, "a row in one vector may end before its last element");
        if (!edge(i)) return v;
        const bool start = i == 0 && t == 0 && first;
        const uint32_t w = start ? v.w : v.x;
        return select4(inside_bits<T>(lo(i), hi(i)), v,
                       E == 4 ? w : __byte_perm(w, 0u, start ? 0x3232u : 0x1010u));
    }
    // `fill` there
    __device__ __forceinline__ uint4 only_or(int i, const uint4 &v, uint32_t fill) const {
        return edge(i) ? select4(inside_bits<T>(lo(i), hi(i)), v, fill) : v;
    }
    __device__ __forceinline__ void only_or(int i, f32x2 (&d)[E / 2], float fill) const {
        if (edge(i)) {
#pragma unroll
            for (int q = 0; q < E / 2; ++q) {
                float a, b;
                split(d[q], a, b);
                d[q] = pair(2 * q >= lo(i) && 2 * q < hi(i) ? a : fill,
                            2 * q + 1 >= lo(i) && 2 * q + 1 < hi(i) ? b : fill);
            }
        }
    }
    __device__ __forceinline__ void only(int i, f32x2 (&d)[E / 2]) const {
        if (edge(i)) {
#pragma unroll
            for (int q = 0; q < E / 2; ++q) d[q] = mul2(d[q], inside_pair(q, lo(i), hi(i)));
        }
    }
};

// Element k (0 <= k < E) of a vector held in registers.
template <typename T>
__device__ __forceinline__ float element_of(const uint4 &v, int k) {
    constexpr int E = Vec<T>::E;
    const int q = E == 4 ? k : k >> 1;
    const uint32_t w = q & 2 ? (q & 1 ? v.w : v.z) : (q & 1 ? v.y : v.x);
    if constexpr (E == 4) {
        return __uint_as_float(w);
    } else {
        const uint16_t h = uint16_t(k & 1 ? w >> 16 : w);
        T e;
        memcpy(&e, &h, 2);
        return to_f32(e);
    }
}

// Rows shared by several warps: small blocks, 24 warps per SM (80 registers; 16
// warps at 64 lanes, which would spill), and the mask drawn vector by vector.
// Measured on B200 against blocks of 8 warps without a bound, the mask drawn
// ahead: bf16 6000 x 4001 50.1 -> 43.1 us, fp32 8000 x 2001 60.8 -> 47.0; one
// warp per row the other way round, bf16 24001 x 1023 51.7 against 57.9.
template <typename T, int V, int L, int GROUPS>
__global__ void __launch_bounds__(L * GROUPS, L > 64    ? 768 / (L * GROUPS)
                                              : L == 64 ? 512 / (L * GROUPS)
                                                        : 0)
ln_fwd_ragged_kernel(T *__restrict__ out, float *__restrict__ mean, float *__restrict__ rstd,
                     const T *__restrict__ resid, const T *__restrict__ weight,
                     const T *__restrict__ bias, T *__restrict__ resid_out,
                     const T *__restrict__ branch, int64_t N, int C, float inv_C, float eps,
                     const __grid_constant__ DropKeys keys) {
    pdl_enter();
    const Mask mask = make_mask(keys);
    constexpr int E = Vec<T>::E;
    constexpr int P = E / 2;
    const int CW = ragged_vecs<T>(C) * E;
    const int group = threadIdx.x / L;
    const int t = threadIdx.x - group * L;
    const int warp = t >> 5;
    const int lane = threadIdx.x & 31;
    T *s_w = reinterpret_cast<T *>(ln_dyn_smem) + size_t(group) * 2 * CW;
    T *s_b = s_w + CW;
    float *s_red = reinterpret_cast<float *>(reinterpret_cast<T *>(ln_dyn_smem) +
                                             size_t(GROUPS) * 2 * CW) + group * 3 * (L / 32);
    int64_t r = int64_t(blockIdx.x) * GROUPS + group;
    const int64_t rstep = int64_t(gridDim.x) * GROUPS;     // a multiple of 8 (host)
    // first row of this warp: the groups of a warp leave the loop together
    int64_t r_warp = L < 32 ? r - group % (32 / L) : r;
    const int64_t total = N * C;
    const RowSpan<T, L, V> row(r, C, t);
#pragma unroll 8
    for (int c = t; c < CW; c += L) {
        const bool in = c >= row.sh && c < row.sh + C;
        s_w[c] = in ? weight[c - row.sh] : from_f32<T>(0.f);
        s_b[c] = in ? bias[c - row.sh] : from_f32<T>(0.f);
    }
    __syncthreads();
    const uint4 *ws = reinterpret_cast<const uint4 *>(s_w);
    const uint4 *bs = reinterpret_cast<const uint4 *>(s_b);

    for (; r_warp < N; r += rstep, r_warp += rstep) {
        const bool valid = L >= 32 || r < N;
        const int64_t v0 = (r * C - row.sh) / E;           // exact
        uint4 xv[V], bv[V];
        constexpr bool EARLY = L <= 32;
        uint32_t words[EARLY ? V : 1][P];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            xv[i] = bv[i] = make_uint4(0u, 0u, 0u, 0u);
            if (valid && row.in(i)) {
                xv[i] = row.load(resid, v0, i, total);
                bv[i] = row.load(branch, v0, i, total);
            }
        }
        // one warp per row: the mask is drawn while the loads are on their way
        if constexpr (EARLY) {
#pragma unroll
            for (int i = 0; i < V; ++i) vec_words<T>(mask, v0 + row.j(i), words[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (valid && row.in(i)) {
                uint32_t (&w)[P] = words[EARLY ? i : 0];
                if constexpr (!EARLY) vec_words<T>(mask, v0 + row.j(i), w);
                xv[i] = row.only(i, drop_add_round<T>(mask, w, xv[i], bv[i]));
                row.store(resid_out, v0, i, xv[i]);
            }
        }
        float pivot;
        if constexpr (L <= 32)
            pivot = __shfl_sync(0xffffffffu, element_of<T>(xv[0], row.sh), lane & ~(L - 1));
        else
            pivot = drop_add_round1<T>(mask, r * C, resid[r * C], branch[r * C]);
        const f32x2 K = pair(pivot, pivot);
        f32x2 d[V][P];
        f32x2 acc = pair(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            to_pairs<T>(xv[i], d[i]);
            if (row.in(i)) {
#pragma unroll
                for (int q = 0; q < P; ++q) d[i][q] = sub2(d[i][q], K);
                row.only(i, d[i]);
#pragma unroll
                for (int q = 0; q < P; ++q) acc = add2(acc, d[i][q]);
            }
        }
        const float mean_d = row_sum<L, GROUPS>(hsum(acc), s_red, group, warp, lane) * inv_C;
        const f32x2 M = pair(mean_d, mean_d);
        const f32x2 MH = pair(coarse(mean_d), coarse(mean_d));
        f32x2 sq = pair(0.f, 0.f), rest = pair(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (row.in(i)) {
                f32x2 e[P];
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    e[q] = sub2(d[i][q], MH);
                    d[i][q] = sub2(d[i][q], M);
                }
                row.only(i, e);
                row.only(i, d[i]);
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    sq = fma2(d[i][q], d[i][q], sq);
                    rest = add2(rest, e[q]);
                }
            }
        }
        float var = hsum(sq), left = hsum(rest);
        row_sum2<L, GROUPS>(var, left, s_red + L / 32, group, warp, lane);
        const float rs = rsqrtf(var * inv_C + eps);
        const f32x2 R = pair(rs, rs);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (valid && row.in(i)) {
                f32x2 wp[P], bp[P], o[P];
                to_pairs<T>(ws[row.j(i)], wp);
                to_pairs<T>(bs[row.j(i)], bp);
#pragma unroll
                for (int q = 0; q < P; ++q) o[q] = fma2(mul2(d[i][q], R), wp[q], bp[q]);
                row.store(out, v0, i, from_pairs<T>(o));
            }
        }
        if (valid && t == 0) {
            mean[r] = mean_with_rest(pivot, mean_d, left, inv_C);
            rstd[r] = rs;
        }
    }
}

// Blocks of the cluster that takes a backward of few rows (more than the
// portable 8: the host asks the kernel's permission and whether one fits).
constexpr int kMaxCluster = 16;
// Address of `p` (this block's shared memory) in the cluster's block `rank`,
// and a load from there.
__device__ __forceinline__ float cluster_load(const float *p, uint32_t rank) {
    uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(p)), remote;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Where the column sums go: the blocks' partial rows, for ln_colsum_kernel to
// add, or, when the whole grid is one cluster, dweight and dbias themselves:
// the blocks then add their sums through distributed shared memory, each a
// slice of the columns, in block order.
struct ColumnSums {
    float *partial;        // NULL: one cluster
    float *dweight;
    float *dbias;
    int accumulate;
};

// Row groups take rows as above; each keeps the column sums of its own columns
// over its rows, and the block adds its groups' sums in group order.
template <typename T, int V, int L, int GROUPS, int MODE>
__global__ void __launch_bounds__(L * GROUPS, 1)
ln_bwd_ragged_kernel(T *__restrict__ dresid, const T *__restrict__ dout,
                     const T *__restrict__ inp, const T *__restrict__ weight,
                     const float *__restrict__ mean, const float *__restrict__ rstd, int64_t N,
                     int C, float inv_C, float eps, ColumnSums sums,
                     const __grid_constant__ DropOut<T> drop) {
    pdl_enter();
    static_assert((MODE & kBwdDropout) != 0, "a dropout kernel");
    constexpr bool ACC = (MODE & kBwdAccumulate) != 0;
    constexpr bool RECOMP = (MODE & kBwdRecompute) != 0;
    constexpr int NS = ACC ? 3 : 2;
    constexpr int W = L / 32;
    const Mask mask = make_mask(drop.keys);
    constexpr int E = Vec<T>::E;
    constexpr int P = E / 2;
    const int group = threadIdx.x / L;
    const int t = threadIdx.x - group * L;
    const int warp = t >> 5;
    const int lane = threadIdx.x & 31;
    const int NVM = ragged_vecs<T>(C);
    float *s_all = reinterpret_cast<float *>(ln_dyn_smem);
    float *s_w = s_all + size_t(group % ragged_copies<GROUPS>()) * NVM * E;
    float *s_red = s_all + size_t(ragged_copies<GROUPS>()) * NVM * E + group * 4 * W;
    // stage s, array k (inp, dout, prev), vector j: s_st[(s * NS + k) * NVM + j]
    uint4 *s_st = reinterpret_cast<uint4 *>(ln_dyn_smem + bwd_ragged_fixed<T, L, GROUPS>(C)) +
                  size_t(group) * 2 * NS * NVM;
    int64_t r = int64_t(blockIdx.x) * GROUPS + group;
    const int64_t rstep = int64_t(gridDim.x) * GROUPS;     // a multiple of 8 (host)
    int64_t r_warp = L < 32 ? r - group % (32 / L) : r;
    const int64_t total = N * C;
    const RowSpan<T, L, V> row(r, C, t);

    // A lane copies the vectors that it will use itself, one row ahead, so only
    // its own copies have to be waited for.
    int stage = 0;
    float m_next = 0.f, s_next = 0.f;
    auto fetch = [&](int64_t rr, int st) {
        if (rr < N) {
            const int64_t v0 = (rr * C - row.sh) / E;
            uint4 *to = s_st + st * NS * NVM;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (row.in(i)) {
                    row.load_async(to + row.j(i), inp, v0, i, total);
                    row.load_async(to + NVM + row.j(i), dout, v0, i, total);
                    if constexpr (ACC)
                        row.load_async(to + 2 * NVM + row.j(i), drop.prev, v0, i, total);
                }
            }
            if constexpr (!RECOMP) {
                m_next = __ldg(mean + rr);
                s_next = __ldg(rstd + rr);
            } else if constexpr (L > 32) {
                m_next = to_f32(inp[rr * C]);              // the pivot
            }
        } else {
            m_next = s_next = 0.f;                         // no row: xhat is zero below
        }
        copy_commit();
    };
    fetch(r, 0);
    if (group < ragged_copies<GROUPS>()) {
#pragma unroll 8
        for (int c = t; c < NVM * E; c += L)
            s_w[c] = c >= row.sh && c < row.sh + C ? to_f32(weight[c - row.sh]) : 0.f;
    }
    __syncthreads();

    f32x2 acc_w[V][P], acc_b[V][P];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int q = 0; q < P; ++q) {
            acc_w[i][q] = pair(0.f, 0.f);
            acc_b[i][q] = pair(0.f, 0.f);
        }
    int parity = 0;
    for (; r_warp < N; r += rstep, r_warp += rstep, stage ^= 1) {
        const bool valid = L >= 32 || r < N;
        const int64_t v0 = (r * C - row.sh) / E;           // exact
        const float m = m_next;
        float s = s_next;
        fetch(r + rstep, stage ^ 1);
        copy_wait<1>();
        const uint4 *xs = s_st + stage * NS * NVM, *ds = xs + NVM, *ps = ds + NVM;
        // Vector i.  Nothing of a neighbour's row may enter a sum (0 * infinity):
        // zeros outside the row, or for x the pivot.
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        auto vec = [&](const uint4 *from, int i) {
            return valid ? row.only(i, from[row.j(i)]) : zero;
        };
        uint32_t fill = 0u;
        auto vec_p = [&](int i) { return valid ? row.only_or(i, xs[row.j(i)], fill) : zero; };
        float k = m;                                       // K as a number
        f32x2 K = pair(m, m), MD = pair(0.f, 0.f);
        if constexpr (RECOMP) {
            float pivot;
            if constexpr (L <= 32)
                pivot = __shfl_sync(0xffffffffu,
                                    valid && row.in(0) ? element_of<T>(xs[row.j(0)], row.sh) : 0.f,
                                    lane & ~(L - 1));
            else
                pivot = m;
            k = pivot;
            K = pair(pivot, pivot);
            fill = spread<T>(pivot);
            f32x2 sd = pair(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (row.in(i)) {
                    f32x2 x[P];
                    to_pairs<T>(vec_p(i), x);
#pragma unroll
                    for (int q = 0; q < P; ++q) sd = add2(sd, sub2(x[q], K));
                }
            }
            const float md =
                row_sum<L, GROUPS>(hsum(sd), s_red + parity * 2 * W, group, warp, lane) * inv_C;
            parity ^= 1;
            MD = pair(md, md);
            f32x2 sq = pair(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (row.in(i)) {
                    f32x2 x[P];
                    to_pairs<T>(vec_p(i), x);
#pragma unroll
                    for (int q = 0; q < P; ++q) x[q] = sub2(sub2(x[q], K), MD);
                    row.only(i, x);
#pragma unroll
                    for (int q = 0; q < P; ++q) sq = fma2(x[q], x[q], sq);
                }
            }
            const float var =
                row_sum<L, GROUPS>(hsum(sq), s_red + parity * 2 * W, group, warp, lane) * inv_C;
            parity ^= 1;
            s = rsqrtf(var + eps);
        }
        const f32x2 S = pair(s, s);
        auto xhat = [&](f32x2 x) {
            f32x2 d = sub2(x, K);
            if constexpr (RECOMP) d = sub2(d, MD);
            return mul2(d, S);
        };
        // Outside the row dout is zero, and xhat must be finite for its product
        // with dout to be zero too.  For x = 0 it is -mean * rstd, which overflows
        // for a row of the type's lowest value (3.4e38 * 316).  So x there is one
        // of the vector's own elements, or, where a lane's one vector may hold the
        // whole row, K in the rows that need it; with recomputed statistics the
        // pivot, selected as bits or, with several warps a row, as numbers.
        // Measured on B200: the plain zeros 67.2 us at bf16 24001 x 1023, own
        // elements 68.0, K selected in every row 72.5; recomputed 8000 x 5001 as
        // numbers 122 against 147 as bits, 24001 x 1023 98 against 90.
        [[maybe_unused]] const bool far = !(fabsf(m * s) <= 3.402823466e38f);
        f32x2 s1 = pair(0.f, 0.f), s2 = pair(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (row.in(i)) {
                f32x2 x[P], dy[P], wp[P];
                if constexpr (!RECOMP && V > 1) {
                    to_pairs<T>(valid ? row.only_own(i, xs[row.j(i)]) : zero, x);
                } else if constexpr (!RECOMP) {
                    to_pairs<T>(vec(xs, i), x);
                    if (far) row.only_or(i, x, k);
                } else if constexpr (L > 64) {
                    to_pairs<T>(xs[row.j(i)], x);
                    row.only_or(i, x, k);
                } else {
                    to_pairs<T>(vec_p(i), x);
                }
                to_pairs<T>(vec(ds, i), dy);
                smem_pairs<P>(s_w + row.j(i) * E, wp);
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    const f32x2 xh = xhat(x[q]);
                    const f32x2 g = mul2(dy[q], wp[q]);
                    s1 = add2(s1, g);
                    s2 = fma2(g, xh, s2);
                    acc_w[i][q] = fma2(dy[q], xh, acc_w[i][q]);
                    acc_b[i][q] = add2(acc_b[i][q], dy[q]);
                }
            }
        }
        float a = hsum(s1), b = hsum(s2);
        row_sum2<L, GROUPS>(a, b, s_red + parity * 2 * W, group, warp, lane);
        parity ^= 1;
        // one warp per row has no barrier here; without this one the second
        // pass's loads move up and 130 bytes of registers spill (3 vectors)
        if constexpr (L == 32) __syncwarp();
        const float na = -s * (a * inv_C), nc = -s * (b * inv_C);
        const f32x2 NA = pair(na, na), NC = pair(nc, nc);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (valid && row.in(i)) {
                // what lies outside the row is not stored
                f32x2 x[P], dy[P], wp[P], o[P];
                uint32_t w[P];
                to_pairs<T>(xs[row.j(i)], x);
                to_pairs<T>(ds[row.j(i)], dy);
                smem_pairs<P>(s_w + row.j(i) * E, wp);
#pragma unroll
                for (int q = 0; q < P; ++q)
                    o[q] = fma2(mul2(dy[q], wp[q]), S, fma2(xhat(x[q]), NC, NA));
                if constexpr (ACC) {
                    f32x2 pp[P];
                    to_pairs<T>(ps[row.j(i)], pp);
#pragma unroll
                    for (int q = 0; q < P; ++q) o[q] = add2(o[q], pp[q]);
                }
                row.store(dresid, v0, i, from_pairs<T>(o));
                vec_words<T>(mask, v0 + row.j(i), w);
#pragma unroll
                for (int q = 0; q < P; ++q) o[q] = drop2(mask, w[q], o[q]);
                row.store(drop.dbranch, v0, i, from_pairs<T>(o));
            }
        }
    }
    copy_wait<0>();                                        // nothing in flight any more

    __syncthreads();                                       // weights and stages are done with
    const int span = NVM * E;                              // floats of one group's sums
    float *dst = s_all + size_t(group) * 2 * span;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (row.in(i)) {
            ulonglong2 *pw = reinterpret_cast<ulonglong2 *>(dst + row.j(i) * E);
            ulonglong2 *pb = reinterpret_cast<ulonglong2 *>(dst + span + row.j(i) * E);
#pragma unroll
            for (int q = 0; q < P / 2; ++q) {
                pw[q] = make_ulonglong2(acc_w[i][2 * q], acc_w[i][2 * q + 1]);
                pb[q] = make_ulonglong2(acc_b[i][2 * q], acc_b[i][2 * q + 1]);
            }
        }
    }
    __syncthreads();
    float *s_sum = s_all + size_t(GROUPS) * 2 * span;      // the block's 2C sums
    const int sh0 = int((int64_t(blockIdx.x) * GROUPS * C) % E);
    for (int c = threadIdx.x; c < 2 * C; c += blockDim.x) {
        const float *from = s_all + (c < C ? c : span + c - C);
        float sum = from[sh0];
#pragma unroll 4
        for (int g = 1; g < GROUPS; ++g)
            sum += from[size_t(g) * 2 * span + ((sh0 + g * C) & (E - 1))];
        if (sums.partial)
            sums.partial[int64_t(blockIdx.x) * 2 * C + c] = sum;
        else
            s_sum[c] = sum;
    }
    if (!sums.partial) {
        // the whole grid is this cluster: block b is rank b
        __syncthreads();                                   // whole warps at the barrier
        cluster_sync();
        for (int c = blockIdx.x * blockDim.x + threadIdx.x; c < 2 * C;
             c += gridDim.x * blockDim.x) {
            float v[kMaxCluster];                          // loads first, then the sum
#pragma unroll
            for (uint32_t k = 0; k < kMaxCluster; ++k)
                v[k] = k < gridDim.x ? cluster_load(s_sum + c, k) : 0.f;
            float sum = v[0];
#pragma unroll
            for (uint32_t k = 1; k < kMaxCluster; ++k) sum += v[k];
            float *to = c < C ? sums.dweight + c : sums.dbias + (c - C);
            *to = sums.accumulate ? *to + sum : sum;
        }
        __syncthreads();
        cluster_sync();                                    // no block leaves while it is read
    }
}

// Calls visitor.template ragged<V, L, GROUPS>() for the forward / backward
// variant that serves rows of C elements; false when none does.  V is
// ceil(most vectors / L) throughout; up to 5 vectors of each array per lane in
// the forward, 3 of 16-bit types and 4 of fp32 in the backward, whose column
// sums take its registers.  ragged_if: L lanes per row for rows of more than
// (V - 1) * L and up to V * L vectors, in blocks of about THREADS.
template <int V, int L, int THREADS, typename Visitor>
bool ragged_if(int nv, Visitor &v) {
    if (nv > V * L) return false;
    if constexpr (V > 1) {
        if (nv <= (V - 1) * L) return false;
    }
    v.template ragged<V, L, (THREADS / L)>();
    return true;
}
template <typename T, typename Visitor>
bool visit_fwd_ragged(int C, Visitor &v) {
    const int nv = ragged_vecs<T>(C);
    return ragged_if<1, 8, 256>(nv, v) || ragged_if<1, 16, 256>(nv, v) ||
           ragged_if<1, 32, 256>(nv, v) || ragged_if<2, 32, 256>(nv, v) ||
           ragged_if<3, 32, 256>(nv, v) || ragged_if<4, 32, 256>(nv, v) ||
           ragged_if<5, 32, 256>(nv, v) || ragged_if<3, 64, 128>(nv, v) ||
           ragged_if<4, 64, 128>(nv, v) || ragged_if<5, 64, 128>(nv, v) ||
           ragged_if<3, 128, 128>(nv, v) || ragged_if<4, 128, 128>(nv, v) ||
           ragged_if<5, 128, 128>(nv, v) || ragged_if<3, 256, 256>(nv, v) ||
           ragged_if<4, 256, 256>(nv, v) || ragged_if<5, 256, 256>(nv, v);
}
template <typename T, typename Visitor>
bool visit_bwd_ragged(int C, Visitor &v) {
    const int nv = ragged_vecs<T>(C);
    if (ragged_if<1, 8, 512>(nv, v) || ragged_if<1, 16, 512>(nv, v) || ragged_if<1, 32, 512>(nv, v) ||
        ragged_if<2, 32, 512>(nv, v) || ragged_if<3, 32, 512>(nv, v))
        return true;
    if constexpr (sizeof(T) == 2) {
        return ragged_if<2, 64, 512>(nv, v) || ragged_if<3, 64, 512>(nv, v) || ragged_if<3, 96, 512>(nv, v) ||
               ragged_if<3, 128, 512>(nv, v) || ragged_if<3, 192, 512>(nv, v) || ragged_if<3, 256, 512>(nv, v) ||
               ragged_if<3, 384, 512>(nv, v) || ragged_if<3, 512, 512>(nv, v);
    } else {
        return ragged_if<4, 32, 512>(nv, v) || ragged_if<3, 64, 512>(nv, v) ||
               ragged_if<4, 64, 512>(nv, v) || ragged_if<3, 128, 512>(nv, v) || ragged_if<4, 128, 512>(nv, v) ||
               ragged_if<3, 256, 512>(nv, v) || ragged_if<4, 256, 512>(nv, v) ||
               ragged_if<3, 512, 512>(nv, v) || ragged_if<4, 512, 512>(nv, v);
    }
}

}  // namespace lnk

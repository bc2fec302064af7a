// dropout_geometry.cu -- host-side check of the kernel selection and launch
// geometry of the dropout calls.  It runs on a machine without a GPU: nothing
// here calls the CUDA runtime, launches a kernel or instantiates one.
//
// For every row length from 1 channel to past the widest vector kernel, every
// element type and every variant it visits the selection as the launchers do,
// for arrays on 16-byte boundaries (with many rows and with few), and checks:
//   - ragged kernels: the lanes' vectors cover the row at any shift, all rounds
//     but the last are whole for every row, the block has whole warps and at
//     most 1024 threads, its named barriers fit, its shared memory fits and its
//     parts start on 16 bytes; the blocks of a grid or a cluster times the
//     groups are a multiple of 8 rows, so that a group's shift is fixed;
//   - forward tiles with dropout, one small tile a block: shared memory and
//     bulk copies;
//   - ring and split ring: coverage, depth, shared memory, barriers, at most 16
//     warps, bulk copies.
//
// Output: "use <kernel>" once for each kernel that some call reaches, one "FAIL
// ..." line per failed check, and "checks <n> failures <m>".  Exit status 1 on
// failure.
#include <cstdint>
#include <cstdio>
#include <set>
#include <string>
#include <vector>

#include "../layernorm_fwd_bwd_b200/csrc/ln_dispatch.cuh"

namespace {

std::vector<std::string> g_fail;
std::set<std::string> g_use;
long g_checks = 0;

void check(bool ok, const std::string &what) {
    ++g_checks;
    if (!ok) g_fail.push_back(what);
}

template <typename T> const char *tname();
template <> const char *tname<float>() { return "f32"; }
template <> const char *tname<lnk::bf16>() { return "bf16"; }
template <> const char *tname<lnk::f16>() { return "f16"; }

std::string num(long v) { return std::to_string(v); }

constexpr size_t kMax = lnk::kMaxSmemPerBlock;
constexpr size_t kMaxTx = (size_t(1) << 20) - 1;   // mbarrier transaction count limit
constexpr int kWidest = 2100;                      // vectors of the longest rows visited

void check_copies(const std::string &ctx, size_t row_bytes, int rows, int arrays) {
    check(row_bytes % 16 == 0, ctx + "bulk copies are whole 16-byte units");
    check(size_t(arrays) * rows * row_bytes <= kMaxTx,
          ctx + "one phase expects fewer than 2^20 bytes");
}

// What every ragged kernel needs of V, L and GROUPS.
template <typename T, int V, int L, int GROUPS>
void check_ragged(const std::string &ctx, int C, size_t smem) {
    constexpr int E = lnk::Vec<T>::E;
    const int most = lnk::ragged_vecs<T>(C);
    for (int sh = 0; sh < E; ++sh) {
        if ((int64_t(sh) * C) % E != 0 && C % E == 0) continue;
        const int shift = int((int64_t(sh) * C) % E);       // row sh's
        const int nv = (shift + C + E - 1) / E;
        check(nv <= most, ctx + "the widest span is the stated one");
        check(nv <= V * L, ctx + "lanes cover the row");
        check(nv >= (V - 1) * L, ctx + "rounds before the last are whole");
        check(nv - 1 >= (V >= 2 ? (V - 2) * L : 0), ctx + "the row ends in the last two rounds");
    }
    check(L * GROUPS <= 1024 && (L * GROUPS) % 32 == 0, ctx + "whole warps, at most 1024 threads");
    check(L <= 32 ? 32 % L == 0 : (L % 32 == 0 && GROUPS <= 15), ctx + "row groups and barriers");
    check(smem <= kMax, ctx + "shared memory fits: " + num(long(smem)));
    constexpr int kStep = lnh::ragged_step(GROUPS);
    check(kStep * GROUPS % 8 == 0, ctx + "blocks come in steps of 8 rows");
    for (int64_t N : {1, 7, 8, 9, 100, 1024, 5003, 65536})
        for (int64_t resident : {1, 3, 148, 592}) {
            const int64_t G = lnh::ragged_grid<GROUPS>(N, resident);
            check(G >= 1 && G * GROUPS % 8 == 0, ctx + "a group's rows lie 8 apart");
            check(G <= (N + GROUPS - 1) / GROUPS + 8, ctx + "no blocks without rows but the step's");
        }
}

template <typename T>
struct FwdChoice {
    int C;
    static constexpr int E = lnk::Vec<T>::E;
    std::string ctx() const { return std::string("fwd ") + tname<T>() + " C " + num(C) + ": "; }

    template <int V, int L, int GROUPS>
    void ragged() {
        g_use.insert("fwd_ragged " + std::string(tname<T>()) + " " + num(V) + " " + num(L) + " " +
                     num(GROUPS));
        check_ragged<T, V, L, GROUPS>(ctx(), C, lnk::fwd_ragged_smem<T, L, GROUPS>(C));
        check(size_t(GROUPS) * 2 * lnk::ragged_vecs<T>(C) * 16 % 16 == 0,
              ctx() + "slots start on 16 bytes");
    }
    template <int V, int RW, int NW>
    void tile(int tiles) {
        const int nvec = C / E;
        check(32 * RW * V >= nvec && 32 * RW * (V - 1) < nvec, ctx() + "a tile's rounds are whole");
        const size_t smem = tiles == 2 ? lnk::fwd_tile_smem<T, NW, 2, RW, 2>(C)
                                       : lnk::fwd_tile_smem<T, NW, 1, RW, 2>(C);
        check(smem <= kMax, ctx() + "tile shared memory fits");
        check_copies(ctx(), size_t(C) * sizeof(T), NW / RW, 2);
    }
    template <int V, int W, int GROUPS>
    void run() {
        using F = lnh::FwdVec<T, lnk::kFwdResidual | lnk::kFwdDropout>;
        if constexpr (W == 1)
            tile<V, 1, F::template kWarps<V>>(F::template kTiles<V>);
        else
            check(32 * W * V >= C / E && lnk::fwd_vec_smem<W, GROUPS>(C) <= kMax,
                  ctx() + "register-resident rows are covered and fit");
    }
    template <int V> void run_tile_two() { tile<V, 2, 4>(1); }
    template <int V> void run_tile_four() { tile<V, 4, 4>(1); }
};

template <typename T, int MODE>
struct BwdChoice {
    int C;
    static constexpr int E = lnk::Vec<T>::E;
    static constexpr int NS = lnk::BwdRingArrays<MODE>::value;
    std::string ctx() const {
        return std::string("bwd ") + tname<T>() + " mode " + num(MODE) + " C " + num(C) + ": ";
    }
    std::string use(const char *kernel) const {
        return std::string(kernel) + " " + tname<T>() + " " + num(MODE);
    }
    template <int V, int L, int GROUPS>
    void ragged() {
        g_use.insert(use("bwd_ragged") + " " + num(V) + " " + num(L) + " " + num(GROUPS));
        check_ragged<T, V, L, GROUPS>(ctx(), C, lnk::bwd_ragged_smem<T, L, GROUPS, NS>(C));
        check(lnk::bwd_ragged_fixed<T, L, GROUPS>(C) % 16 == 0, ctx() + "stages start on 16 bytes");
        int blocks = lnh::ragged_step(GROUPS);
        check(blocks <= lnk::kMaxCluster, ctx() + "a cluster holds one step of blocks");
        for (; blocks < lnk::kMaxCluster; blocks *= 2) {}
        check(blocks == lnk::kMaxCluster, ctx() + "a cluster of 16 at most");
    }
    template <int V, int W>
    void ring() {
        constexpr int NC = lnk::BwdRingConsumers<W>::value;
        constexpr int S = lnk::BwdStages<V, NC, NS>::value;
        g_use.insert(use("bwd_tma") + " " + num(V) + " " + num(W));
        check(32 * W * V >= C / E, ctx() + "ring rows are covered");
        check(S >= 2 && S <= 8, ctx() + "ring depth 2..8");
        check(NC % W == 0 && NC / W >= 2 && NC / W <= 15, ctx() + "ring row groups");
        check(lnk::bwd_tma_smem<T, NC, S, W, NS>(C) <= kMax, ctx() + "ring shared memory fits");
        check_copies(ctx(), size_t(C) * sizeof(T), NC / W, NS);
    }
    template <int VR, int VC>
    void split() {
        using Warps = lnk::SplitWarps<VR, MODE>;
        constexpr bool kStats = (MODE & lnk::kBwdRecompute) != 0;
        constexpr int kDeep = lnk::split_max_stages<MODE>();
        const int fit = lnk::split_stages<T, Warps::rows, NS, kStats>(C, kMax);
        const int S = fit < kDeep ? fit : kDeep;
        const int nvec = C / E;
        g_use.insert(use("bwd_split") + " " + num(VR) + " " + num(VC));
        check(VR == (nvec + 31) / 32, ctx() + "split rows take the fewest vectors per lane");
        check(32 * VC * Warps::cols >= nvec && 32 * VC >= (nvec + Warps::cols - 1) / Warps::cols,
              ctx() + "column warps cover the row");
        check(S >= 2, ctx() + "split ring depth");
        check((kStats ? 3 : 2) * kDeep * 8 <= 128, ctx() + "split barriers fit in 128 bytes");
        check(lnk::split_smem<T, Warps::rows, NS, kStats>(C, S) <= kMax,
              ctx() + "split shared memory fits");
        check(Warps::rows + Warps::cols + 1 <= 16, ctx() + "split block of at most 16 warps");
        check_copies(ctx(), size_t(C) * sizeof(T), Warps::rows, NS);
    }
};

template <typename T>
void forward_all() {
    constexpr int E = lnk::Vec<T>::E;
    for (int C = 1; C <= kWidest * E; ++C) {
        FwdChoice<T> c{C};
        if (C % E == 0 && C > lnk::kNarrowVecs * E && lnk::visit_fwd_vec<T>(C / E, c)) continue;
        const bool found = lnk::visit_fwd_ragged<T>(C, c);
        check(found == (lnk::ragged_vecs<T>(C) <= 5 * 256), c.ctx() + "ragged up to 1280 vectors");
    }
}

template <typename T, int MODE>
void backward_all() {
    constexpr int E = lnk::Vec<T>::E;
    for (int C = 1; C <= kWidest * E; ++C) {
        BwdChoice<T, MODE> c{C};
        // few rows take a ragged kernel wherever there is one, others where the
        // ring does not serve them
        const bool ragged = lnk::visit_bwd_ragged<T>(C, c);
        check(ragged == (lnk::ragged_vecs<T>(C) <= (E == 8 ? 1536 : 2048)),
              c.ctx() + "ragged up to 3 or 4 vectors a lane of 512");
        if (C % E == 0 && C > lnk::kNarrowVecs * E) lnk::visit_bwd_ring<T, MODE>(C / E, c);
    }
}

template <typename T>
void type_all() {
    constexpr int D = lnk::kBwdDropout, A = lnk::kBwdAccumulate, R = lnk::kBwdRecompute;
    forward_all<T>();
    backward_all<T, D>();
    backward_all<T, D | A>();
    backward_all<T, D | R>();
    backward_all<T, D | A | R>();
}

}  // namespace

int main() {
    type_all<float>();
    type_all<lnk::bf16>();
    type_all<lnk::f16>();
    for (const std::string &u : g_use) std::printf("use %s\n", u.c_str());
    for (const std::string &f : g_fail) std::printf("FAIL %s\n", f.c_str());
    std::printf("checks %ld failures %zu\n", g_checks, g_fail.size());
    return g_fail.empty() ? 0 : 1;
}

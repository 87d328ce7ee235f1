// The launch plans of the block-scaled FP8 products, without a GPU: abi.cpp linked with launchers of this file, which check what
// the kernels would be given -- every buffer inside the call's workspace, no two of them over each other, K ranges and work tiles that
// cover the call exactly, a form that exists, a grid that HIP takes.  Pointers are numbers, nothing is read or written.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <vector>

#include "fp8.h"
#include "glowq.h"

namespace glowq {

static char call[256];
static int failures = 0;
static uintptr_t ws_begin, ws_end;
static int64_t launches[2];

static void fail(const char* what) {
    if (failures++ < 20) std::printf("FAIL: %s: %s\n", call, what);
}

struct Region {
    uintptr_t from, to;
};
static std::vector<Region> held;

static void region(const void* p, size_t bytes, const char* what) {
    const uintptr_t from = reinterpret_cast<uintptr_t>(p), to = from + bytes;
    if (from < ws_begin || to > ws_end) fail(what);
    for (const Region& h : held)
        if (from < h.to && h.from < to) fail(what);
    held.push_back({from, to});
}

hipError_t launch_repack_fp8(const uint8_t*, const float*, int64_t, int64_t, uint8_t*, float*, int32_t*, hipStream_t) {
    return hipSuccess;
}

hipError_t launch_fp8_prep(const Fp8PrepArgs& a, int tt, int nj, bool join, const Fp8Args* experts, int64_t row_blocks, hipStream_t) {
    ++launches[0];
    const int64_t rows = experts != nullptr ? experts->n_rows : a.T;
    region(a.xq, (size_t)a.T * a.d, "codes");
    region(a.xs, (size_t)a.T * a.gp * 4, "scales");
    if (a.gp % 4 != 0 || a.gp < a.d / 128) fail("scale stride");
    if (a.r > 0) {
        if (a.rp % 64 != 0 || a.rp < a.r) fail("padded rank");
        if (a.part != nullptr) region(a.part, (size_t)a.ks * rows * a.rp * 4, "ranges of the projection");
        else if (a.ks > 1) fail("ranges without a place");
        region(a.R, (size_t)rows * a.rp * 2, "projection");
        if (a.range % 32 != 0 || (int64_t)a.range * a.ks < a.d || (int64_t)a.range * (a.ks - 1) >= a.d) fail("ranges cover the inputs");
        if (join && experts != nullptr && a.part != nullptr) fail("join of the experts' rows counts tokens");
    }
    const bool form = tt == 4 ? nj == 4 && experts != nullptr
                              : tt == 2 ? nj == 4 : tt == 1 && (nj == 1 || (nj == 4 && experts == nullptr));
    if (!form) fail("a form of the preparation");
    const int64_t cols = ceil_div(a.rp / 16, nj);
    const int64_t proj = a.r == 0 ? 0 : experts != nullptr ? 8 * ceil_div(row_blocks * cols, 8) * a.ks : ceil_div(a.T, 16 * tt) * cols * a.ks;
    if (experts != nullptr && row_blocks < ceil_div(rows, 16 * tt) + (rows < experts->n_exp ? rows : experts->n_exp)) fail("row blocks");
    if ((proj + ceil_div((int64_t)a.T * a.d / 8, 512)) * 512 > (int64_t)UINT32_MAX) fail("grid of the preparation");
    return hipSuccess;
}

hipError_t launch_fp8(const Fp8Args& a, const Fp8PrepArgs& p, int64_t items, hipStream_t) {
    ++launches[1];
    const int G = a.d / 128;
    int64_t blocks = 0;
    for (int i = 0; i < a.n_mod; ++i) {
        if (a.mod[i].block_begin != blocks) fail("first row block");
        blocks += ceil_div(ceil_div((int64_t)a.mod[i].n_out, 16), a.rr);
    }
    if (a.row_blocks != blocks || a.G != G || a.gp != p.gp) fail("row blocks, groups");
    if (a.r > 0 && a.R != (a.r_ranges > 0 ? (const void*)p.part : (const void*)p.R)) fail("projection's place");
    if (a.r > 0 && a.r_ranges > 0 && a.r_ranges != p.ks) fail("projection's ranges");
    if (a.r > 0 && a.r_rows != (a.offsets != nullptr && !a.r_by_token ? a.n_rows : a.T)) fail("projection's rows");
    const bool small = a.rr <= 2;
    const bool pieces = (a.tt == 1 && a.rr == 1) || (a.tt == 2 && a.rr == 2) || (a.tt == 4 && a.rr == 2);
    if (a.offsets != nullptr) {
        if (small ? !pieces : !(a.tt == 8 && a.rr == 16)) fail("a form of the experts' product");
        if (!small && a.r > 0 && a.r_ranges > 0) fail("tiles take R");
        if (!small && (a.gk % 4 != 0 || a.gk < G || a.ks != 1)) fail("groups of the tiles");
        const int64_t active = a.n_rows < a.n_exp ? a.n_rows : a.n_exp;
        if (items < blocks * (ceil_div((int64_t)a.n_rows, 16 * a.tt) + active - 1) || items * 512 > (int64_t)UINT32_MAX) fail("items");
        return hipSuccess;
    }
    if (a.m_blocks != ceil_div((int64_t)a.T, 16 * a.tt)) fail("token blocks");
    if (small) {
        if (!pieces || items != blocks * a.m_blocks || items * 512 > (int64_t)UINT32_MAX) fail("pieces");
        if (a.r > 0 && a.r_ranges == 0) fail("pieces add up the ranges");
        return hipSuccess;
    }
    const bool form = (a.tt == 8 && a.rr == 16 && a.kh == 1 && a.ks == 1) || (a.tt == 8 && a.rr == 8 && (a.kh == 2 ? a.ks > 1 : a.kh == 1 && a.ks == 1)) ||
                      (a.tt == 4 && a.rr == 8 && a.kh == 4);
    if (!form) fail("a form of the tiles");
    if (a.gk % (4 * a.kh) != 0 || (int64_t)a.gk * a.ks < G || (int64_t)a.gk * (a.ks - 1) >= G) fail("K ranges of whole turns cover the groups");
    if (G > 128) fail("scales of a workgroup's groups in two registers");
    if (a.r > 0 && a.r_ranges > 0 && (a.kh == 1 || a.ks > 1)) fail("ranges of the projection");
    const int64_t threads = 64 * (a.tt == 4 ? 2 : 4) * a.kh;
    const int64_t join = a.ks > 1 && a.r > 0 && p.part != nullptr ? ceil_div(ceil_div((int64_t)p.T * p.rp / 4, threads), 8) * 8 : 0;
    if ((join + 8 * ceil_div(blocks * a.ks, 8) * a.m_blocks) * threads > (int64_t)UINT32_MAX) fail("grid of the tiles");
    if (a.ks > 1) region(a.part, (size_t)(blocks * a.m_blocks * a.ks) * a.tt * a.rr * 1024, "the K ranges' tiles");
    return hipSuccess;
}

}  // namespace glowq

using namespace glowq;

namespace {

const void* at(uintptr_t p) { return reinterpret_cast<const void*>(p); }
constexpr uintptr_t kData = (uintptr_t)1 << 40, kWorkspace = (uintptr_t)1 << 44;

void set_workspace(size_t bytes) {
    ws_begin = kWorkspace;
    ws_end = kWorkspace + bytes;
    held.clear();
}

void group(int64_t T, int64_t d, const std::vector<int64_t>& rows, int32_t r) {
    const size_t need = glowq_fp8_workspace_bytes(T, d, r);
    std::snprintf(call, sizeof(call), "group T=%lld d=%lld r=%d %zu modules, first of %lld rows", (long long)T, (long long)d, r, rows.size(), (long long)rows[0]);
    if (need == 0) return fail("no workspace size");
    set_workspace(need);
    glowq_qweight w[8] = {};
    const void* a[8];
    void* y[8];
    for (size_t i = 0; i < rows.size(); ++i) {
        w[i].q = w[i].sz = a[i] = at(kData);
        y[i] = const_cast<void*>(at(kData));
        w[i].n_out = rows[i];
        w[i].k_in = d;
        w[i].format = GLOWQ_FMT_FP8_BLOCK;
    }
    const int status = glowq_group_forward_fp8(at(kData), T, d, (int32_t)rows.size(), w, at(kData), a, r, r > 0, const_cast<void*>(at(kWorkspace)),
                                               need, y, nullptr);
    if (status != GLOWQ_OK) {
        std::printf("status %d\n", status);
        fail("refused");
    }
}

void experts(int64_t T, int64_t n_rows, int32_t n_exp, int64_t d, const std::vector<int64_t>& rows, int32_t r, int32_t share) {
    const size_t need = glowq_moe_fp8_workspace_bytes(n_rows, T, d, r, share);
    std::snprintf(call, sizeof(call), "experts T=%lld rows=%lld E=%d d=%lld r=%d share=%d %zu modules of %lld rows", (long long)T, (long long)n_rows, n_exp,
                  (long long)d, r, share, rows.size(), (long long)rows[0]);
    if (need == 0) return fail("no workspace size");
    set_workspace(need);
    held.push_back({kWorkspace, kWorkspace + 8192});  // status words
    glowq_moe_module m[4] = {};
    for (size_t i = 0; i < rows.size(); ++i) {
        m[i].q = m[i].sz = m[i].a = at(kData);
        m[i].y = const_cast<void*>(at(kData));
        m[i].n_out = rows[i];
        m[i].k_in = d;
    }
    const int status = glowq_moe_forward_fp8(at(kData), T, d, n_exp, (int32_t)rows.size(), m, at(kData), share, r, r > 0,
                                             reinterpret_cast<const int32_t*>(kData), reinterpret_cast<const int32_t*>(kData), n_rows,
                                             const_cast<void*>(at(kWorkspace)), need, nullptr);
    if (status != GLOWQ_OK) {
        std::printf("status %d\n", status);
        fail("refused");
    }
}

}  // namespace

int main() {
    std::vector<int64_t> Ts;
    for (int64_t t = 1; t <= 200; ++t) Ts.push_back(t);
    for (int64_t t : {255, 256, 257, 400, 513, 600, 1000, 1025, 2048, 4095, 4096, 4097, 8191, 8192, 16384, 65535, 65536}) Ts.push_back(t);
    std::vector<int64_t> ds;
    for (int64_t g : {1, 2, 3, 4, 5, 7, 8, 15, 16, 23, 25, 31, 32, 33, 47, 48, 49, 56, 63, 64, 65, 96, 97, 112, 127, 128}) ds.push_back(128 * g);
    const std::vector<std::vector<int64_t>> sets = {{1}, {16, 17}, {130}, {1024}, {4096}, {4097, 20}, {9000}, {4096, 1024, 1024}, {11008, 11008},
                                                    {28672}, {33, 33, 33, 33, 33, 33, 33, 33}, {128256}};
    for (int64_t T : Ts)
        for (int64_t d : ds)
            for (const auto& rows : sets)
                for (int32_t r : {0, 8, 64, 72, 256}) group(T, d, rows, r);
    for (int64_t T : {(int64_t)1, (int64_t)40, (int64_t)1 << 17, (int64_t)1 << 20})
        for (int32_t r : {0, 256}) {
            group(T, 128, {(int64_t)1 << 18}, r);
            group(T, 1024, {4096, 1}, r);
        }
    for (int64_t T : {1, 2, 3, 8, 15, 16, 17, 33, 64, 65, 100, 257, 1000, 4095, 20000, 65536})
        for (int64_t k : {1, 2, 4, 8})
            for (int32_t E : {1, 2, 7, 60, 128, 255, 256})
                for (int64_t d : {128, 640, 2048, 4096, 7168, 16384})
                    for (const auto& rows : {std::vector<int64_t>{20}, {300, 17}, {1408, 1408}, {14336}, {2049, 1, 16, 4096}})
                        for (int32_t r : {0, 8, 64, 256})
                            for (int32_t share : {GLOWQ_MOE_SHARE_EXPERT, GLOWQ_MOE_SHARE_ALL}) experts(T, T * k, E, d, rows, r, share);
    std::printf("%lld preparations, %lld products, %d failures\n", (long long)launches[0], (long long)launches[1], failures);
    return failures != 0;
}

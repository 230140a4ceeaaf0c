// dg_train_api.cpp -- C ABI of the training operators (dg.h): argument validation,
// choice of the tile and launch of the kernels in dg_ragged.hip.  Host code only; like
// dg_api.cpp it never touches device memory, so every call is asynchronous on the
// caller's stream and graph-capturable.
#include <hip/hip_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>

#include "../../include/dg.h"
#include "dg_train.h"

namespace {

constexpr int kMaxConfigs = 64;
constexpr long kMaxLd = 1l << 22;      // a tile's copies use 31-bit offsets: 256 rows of ld elements

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

long ceil_div(long a, long b) { return (a + b - 1) / b; }

// Workgroups of config c that fit a CU (the same on every device the library runs on).
int blocks_per_cu(const dg::RaggedConfig* c, int index) {
    static std::atomic<int> known[kMaxConfigs];
    int v = known[index].load(std::memory_order_relaxed);
    if (v == 0) {
        if (c->occupancy(&v) != hipSuccess || v <= 0) {
            (void)hipGetLastError();
            v = 1;
        }
        known[index].store(v, std::memory_order_relaxed);
    }
    return v;
}

// Upper bound of the tiles of D: the rows' exact split over the groups is on the device.
long tiles_bound(int op, const dg::RaggedParams& p, int bm, int bn) {
    if (op == dg::kRaggedTN) return (long)p.groups * ceil_div(p.ni, bm) * ceil_div(p.nj, bn);
    const long filled = p.groups < p.rows ? p.groups : p.rows;
    return (p.rows / bm + filled) * ceil_div(p.nj, bn);
}

int launch_ragged(int op, int half, int out_f32, dg::RaggedParams& p, void* stream) {
    int count = 0;
    const dg::RaggedConfig* cfgs = dg::ragged_configs(&count);
    const int units = dg_get_num_cus();
    if (units < 0) return DG_ERR_HIP;
    int best = -1;
    for (int i = 0; i < count && i < kMaxConfigs; ++i)
        if (cfgs[i].op == op && cfgs[i].half == half && cfgs[i].out_f32 == out_f32) best = i;
    if (best < 0) return DG_ERR_UNSUPPORTED;
    const dg::RaggedConfig& c = cfgs[best];
    p.tiles_i = (int)ceil_div(p.ni, c.bm);
    p.tiles_j = (int)ceil_div(p.nj, c.bn);
    long grid = (long)units * blocks_per_cu(&c, best);
    const long tiles = tiles_bound(op, p, c.bm, c.bn);
    if (tiles < grid) grid = tiles;
    if (c.launch(p, (int)grid, static_cast<hipStream_t>(stream)) != hipSuccess) {
        (void)hipGetLastError();
        return DG_ERR_HIP;
    }
    return DG_OK;
}

// Checks shared by the three products: sizes, types, and each operand's row stride
// (width_a, width_b, width_d elements wide).
int check_ragged(const void* a, long lda, int width_a, const void* b, long ldb, int width_b, const void* d, long ldd,
                 int width_d, const int* offsets, int m_total, int n, int k, int num_groups, int dtype) {
    if (m_total < 0 || n < 0 || k < 0 || num_groups < 1) return DG_ERR_INVALID_ARG;
    if (dtype != DG_DTYPE_BF16 && dtype != DG_DTYPE_F16) return DG_ERR_INVALID_ARG;
    if (n % 8 || k % 8 || num_groups > dg::kMaxRaggedGroups) return DG_ERR_UNSUPPORTED;
    if (n == 0 || k == 0) return DG_OK;
    if (!d || !offsets || lda < width_a || ldb < width_b || ldd < width_d) return DG_ERR_INVALID_ARG;
    if (lda >= kMaxLd || ldb >= kMaxLd || ldd >= kMaxLd || n >= kMaxLd || k >= kMaxLd) return DG_ERR_UNSUPPORTED;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(d, 16) || lda % 8 || ldb % 8 || ldd % 8 || !aligned(offsets, 4))
        return DG_ERR_MISALIGNED;
    return DG_OK;
}

}  // namespace

extern "C" {

int dg_m_grouped_gemm_ragged_nt(const void* a, long lda, const void* b, void* d, long ldd, const int* offsets,
                                int m_total, int n, int k, int num_groups, int dtype, void* stream) {
    const int st = check_ragged(a, lda, k, b, k, k, d, ldd, n, offsets, m_total, n, k, num_groups, dtype);
    if (st != DG_OK) return st;
    if (m_total == 0 || n == 0) return DG_OK;
    if (k == 0) return DG_ERR_UNSUPPORTED;
    if (!a || !b) return DG_ERR_INVALID_ARG;
    dg::RaggedParams p{};
    p.p = static_cast<const uint16_t*>(a);
    p.ldp = lda;
    p.q = static_cast<const uint16_t*>(b);
    p.ldq = k;
    p.q_gstride = (long)n * k;
    p.d = d;
    p.ldd = ldd;
    p.offsets = offsets;
    p.rows = m_total;
    p.groups = num_groups;
    p.nj = n;
    p.nc = k;
    return launch_ragged(dg::kRaggedNT, dtype == DG_DTYPE_F16, 0, p, stream);
}

int dg_m_grouped_gemm_ragged_nn(const void* a, long lda, const void* b, void* d, long ldd, const int* offsets,
                                int m_total, int n, int k, int num_groups, int dtype, void* stream) {
    const int st = check_ragged(a, lda, n, b, k, k, d, ldd, k, offsets, m_total, n, k, num_groups, dtype);
    if (st != DG_OK) return st;
    if (m_total == 0 || k == 0) return DG_OK;
    if (n == 0) return DG_ERR_UNSUPPORTED;
    if (!a || !b) return DG_ERR_INVALID_ARG;
    dg::RaggedParams p{};
    p.p = static_cast<const uint16_t*>(a);
    p.ldp = lda;
    p.q = static_cast<const uint16_t*>(b);
    p.ldq = k;
    p.q_gstride = (long)n * k;
    p.d = d;
    p.ldd = ldd;
    p.offsets = offsets;
    p.rows = m_total;
    p.groups = num_groups;
    p.nj = k;
    p.nc = n;
    return launch_ragged(dg::kRaggedNN, dtype == DG_DTYPE_F16, 0, p, stream);
}

int dg_k_grouped_gemm_ragged_tn(const void* a, long lda, const void* b, long ldb, void* d, const int* offsets,
                                int m_total, int n, int k, int num_groups, int dtype, int d_dtype, int accumulate,
                                void* stream) {
    const int st = check_ragged(a, lda, n, b, ldb, k, d, k, k, offsets, m_total, n, k, num_groups, dtype);
    if (st != DG_OK) return st;
    if (d_dtype != dtype && d_dtype != DG_DTYPE_F32) return DG_ERR_INVALID_ARG;
    if (accumulate != 0 && accumulate != 1) return DG_ERR_INVALID_ARG;
    if (n == 0 || k == 0) return DG_OK;
    if (m_total == 0 && accumulate) return DG_OK;
    if (m_total > 0 && (!a || !b)) return DG_ERR_INVALID_ARG;
    dg::RaggedParams p{};
    p.p = static_cast<const uint16_t*>(a);
    p.ldp = lda;
    p.q = static_cast<const uint16_t*>(b);
    p.ldq = ldb;
    p.d = d;
    p.ldd = k;
    p.d_gstride = (long)n * k;
    p.offsets = offsets;
    p.rows = m_total;
    p.groups = num_groups;
    p.ni = n;
    p.nj = k;
    p.accumulate = accumulate;
    return launch_ragged(dg::kRaggedTN, dtype == DG_DTYPE_F16, d_dtype == DG_DTYPE_F32, p, stream);
}

}  // extern "C"

// train_host_check.cpp -- drives the training entry points (dg_train_api.cpp, compiled
// unchanged) on the CPU under sanitizers: stand-ins record the launches that the kernels
// would get, on a fake device of 256 CUs.
#include <climits>
#include <cstdio>
#include <vector>

#include "../../fp8_block_scaled_e4m3_amd/csrc/dg_train.h"
#include "../../include/dg.h"

namespace {
dg::RaggedParams g_ragged;
int g_grid = 0, g_launches = 0, g_op = -1, g_half = -1, g_f32 = -1;
dg::RaggedJoin g_join;
int g_joins = 0;
dg::AdamwParams g_adamw;
long g_chunks = 0;
int g_cus = 256;

template <int OP, int HALF, int F32>
hipError_t record(const dg::RaggedParams& p, int grid, hipStream_t) {
    g_ragged = p;
    g_grid = grid;
    g_op = OP;
    g_half = HALF;
    g_f32 = F32;
    ++g_launches;
    return hipSuccess;
}
hipError_t two(int* blocks) {
    *blocks = 2;
    return hipSuccess;
}
#define ROW(OP, HALF, F32) {OP, HALF, F32, 128, 128, 1.0, 1.0, 1.0, 1.0, 0.0, F32 ? 32 : 1, &record<OP, HALF, F32>, &two}
const dg::RaggedConfig kRows[] = {ROW(0, 0, 0), ROW(1, 0, 0), ROW(2, 0, 0), ROW(2, 0, 1),
                                  ROW(0, 1, 0), ROW(1, 1, 0), ROW(2, 1, 0), ROW(2, 1, 1)};
int g_failures = 0;
void expect(bool ok, const char* what) {
    if (!ok) {
        ++g_failures;
        std::printf("FAILED: %s\n", what);
    }
}
}  // namespace

namespace dg {
const RaggedConfig* ragged_configs(int* count) {
    *count = (int)(sizeof(kRows) / sizeof(kRows[0]));
    return kRows;
}
hipError_t launch_ragged_join(const RaggedJoin& p, hipStream_t) {
    g_join = p;
    ++g_joins;
    return hipSuccess;
}
hipError_t launch_adamw(const AdamwParams& p, long chunks, hipStream_t) {
    g_adamw = p;
    g_chunks = chunks;
    return hipSuccess;
}
}  // namespace dg

extern "C" int dg_get_num_cus(void) { return g_cus; }
extern "C" hipError_t hipGetLastError(void) { return hipSuccess; }
extern "C" hipError_t hipGetDevice(int* device) {
    *device = 0;
    return hipSuccess;
}
extern "C" hipError_t hipDeviceGetAttribute(int* value, hipDeviceAttribute_t, int) {
    *value = 256;
    return hipSuccess;
}

int main() {
    void* const a = (void*)0x1000;
    void* const b = (void*)0x2000;
    void* const d = (void*)0x3000;
    const int* off = (const int*)0x4000;
    const int big = (1 << 21) - 8;
    // the launches of ordinary calls
    expect(dg_m_grouped_gemm_ragged_nt(a, 64, b, d, 136, off, 10, 136, 64, 4, DG_DTYPE_BF16, nullptr, 0, nullptr) == DG_OK, "nt");
    expect(g_op == 0 && g_half == 0 && g_ragged.tiles_j == 2 && g_ragged.nc == 64 && g_ragged.q_gstride == 136 * 64 &&
           g_grid == 8, "nt launch: at most one row tile a group");
    expect(dg_m_grouped_gemm_ragged_nn(a, 136, b, d, 64, off, 100000, 136, 64, 4, DG_DTYPE_F16, nullptr, 0, nullptr) == DG_OK, "nn");
    expect(g_op == 1 && g_half == 1 && g_ragged.nj == 64 && g_ragged.nc == 136 && g_grid == 512, "nn launch");
    expect(dg_k_grouped_gemm_ragged_tn(a, 136, b, 64, d, off, 10, 136, 64, 3, DG_DTYPE_BF16, DG_DTYPE_F32, 1, nullptr, 0, nullptr) == DG_OK,
           "tn");
    expect(g_op == 2 && g_f32 == 1 && g_ragged.accumulate == 1 && g_grid == 6 && g_ragged.d_gstride == 136 * 64, "tn launch");
    // no row at all: the gradient's zeros are still written
    expect(dg_k_grouped_gemm_ragged_tn(nullptr, 136, nullptr, 64, d, off, 0, 136, 64, 3, DG_DTYPE_BF16, DG_DTYPE_BF16, 0, nullptr, 0,
                                       nullptr) == DG_OK && g_grid == 6, "tn without rows");
    // the largest sizes: no product overflows; too many tiles are refused
    expect(dg_m_grouped_gemm_ragged_nt(a, big, b, d, big, off, 1 << 20, 2048, big, 1024, DG_DTYPE_BF16, nullptr, 0, nullptr) == DG_OK &&
           g_grid == 512, "large nt");
    expect(dg_m_grouped_gemm_ragged_nt(a, big, b, d, big, off, 1 << 30, big, big, 1024, DG_DTYPE_BF16, nullptr, 0, nullptr) ==
           DG_ERR_UNSUPPORTED, "largest nt");
    expect(dg_k_grouped_gemm_ragged_tn(a, big, b, big, d, off, 1 << 30, big, big, 1024, DG_DTYPE_BF16, DG_DTYPE_F32, 1, nullptr, 0,
                                       nullptr) == DG_ERR_UNSUPPORTED, "largest tn");
    expect(dg_k_grouped_gemm_ragged_tn(a, big, b, big, d, off, 1 << 30, 8192, 8192, 1024, DG_DTYPE_BF16, DG_DTYPE_F32, 1, nullptr, 0,
                                       nullptr) == DG_OK && g_grid == 512, "large tn");
    expect(dg_m_grouped_gemm_ragged_nt(a, LONG_MAX, b, d, 136, off, 10, 136, 64, 4, DG_DTYPE_BF16, nullptr, 0, nullptr) ==
           DG_ERR_UNSUPPORTED, "lda past 63 bits' use");
    const int before = g_launches;
    g_cus = DG_ERR_HIP;
    expect(dg_m_grouped_gemm_ragged_nt(a, 64, b, d, 136, off, 10, 136, 64, 4, DG_DTYPE_BF16, nullptr, 0, nullptr) == DG_ERR_HIP &&
           g_launches == before, "no device");
    g_cus = 256;

    // few tiles, a long contraction: slices, where the workspace holds them
    const long ws = dg_ragged_workspace_bytes(DG_RAGGED_TN, 100000, 128, 128, 2, DG_DTYPE_BF16, DG_DTYPE_BF16);
    const long one = 2l * 128 * 128 * 4;
    expect(ws >= 2 * one && ws % one == 0 && g_joins == 0, "workspace of a long contraction");
    expect(dg_k_grouped_gemm_ragged_tn(a, 128, b, 128, d, off, 100000, 128, 128, 2, DG_DTYPE_BF16, DG_DTYPE_BF16, 1, (void*)0x6000,
                                       ws, nullptr) == DG_OK && g_joins == 1 && g_ragged.slices == ws / one &&
           g_ragged.slice_stride == 2 * 128 * 128 && g_ragged.d == (void*)0x6000 && g_ragged.accumulate == 0 &&
           g_join.accumulate == 1 && g_join.d == d && g_join.out == DG_DTYPE_BF16 && g_grid == 2 * ws / one, "slices");
    expect(dg_k_grouped_gemm_ragged_tn(a, 128, b, 128, d, off, 100000, 128, 128, 2, DG_DTYPE_BF16, DG_DTYPE_BF16, 1, nullptr,
                                       0, nullptr) == DG_OK && g_joins == 1 && g_ragged.slices == 1, "no workspace, no slices");
    expect(dg_ragged_workspace_bytes(DG_RAGGED_TN, 1 << 30, big, big, 1024, DG_DTYPE_BF16, DG_DTYPE_F32) == 0,
           "no slices of the largest");

    // the AdamW table, unaligned in host memory, and hostile sizes
    std::vector<dg_adamw_tensor> t(3);
    for (int i = 0; i < 3; ++i) {
        t[i] = dg_adamw_tensor{};
        t[i].param = a;
        t[i].grad = b;
        t[i].exp_avg = d;
        t[i].exp_avg_sq = (void*)0x5000;
        t[i].numel = 3000 * i;
    }
    const long bytes = dg_adamw_plan_bytes(t.data(), 3);
    expect(bytes == 3 * (long)sizeof(dg::AdamwEntry) + 5 * 4, "table bytes");
    std::vector<char> host(bytes + 1);
    expect(dg_adamw_plan(t.data(), 3, host.data() + 1, bytes) == DG_OK, "plan into unaligned host memory");
    expect(dg_adamw_step(a, 3, bytes, 1, 1e-3, 0.9, 0.999, 1e-8, 0.1, nullptr, nullptr) == DG_OK && g_chunks == 5 &&
           g_adamw.tensor_of == (const int*)((char*)a + 3 * sizeof(dg::AdamwEntry)), "step");
    expect(g_adamw.root2 > 31.6f && g_adamw.root2 < 31.7f && g_adamw.size > 0.0099f && g_adamw.size < 0.0101f,
           "bias corrections of step 1");
    expect(dg_adamw_step(a, 3, bytes, LONG_MAX, 1e-3, 0.9, 0.999, 1e-8, 0.1, nullptr, nullptr) == DG_OK &&
           g_adamw.root2 == 1.0f, "last step");
    expect(dg_adamw_step(a, INT_MAX, bytes, 1, 1e-3, 0.9, 0.999, 1e-8, 0.1, nullptr, nullptr) == DG_ERR_INVALID_ARG, "count");
    expect(dg_adamw_step(a, 0, LONG_MAX - 3, 1, 1e-3, 0.9, 0.999, 1e-8, 0.1, nullptr, nullptr) == DG_ERR_INVALID_ARG, "bytes");
    t[1].numel = LONG_MAX;
    expect(dg_adamw_plan_bytes(t.data(), 3) == DG_ERR_UNSUPPORTED, "elements past the limit");
    t[1].numel = (long)INT_MAX * 2048;
    expect(dg_adamw_plan_bytes(t.data(), 3) == DG_ERR_UNSUPPORTED, "chunks of all tensors past the limit");
    std::printf("%d failures\n", g_failures);
    return g_failures != 0;
}

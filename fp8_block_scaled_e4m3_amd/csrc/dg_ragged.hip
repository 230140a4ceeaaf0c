// dg_ragged.hip -- gfx950 kernels of the 16-bit matrix products grouped by expert with
// ragged segments: forward, input gradient, weight gradient (dg.h).
//
// All three are D[i][j] = sum_c P(i, c) Q(j, c) (RaggedOp in dg_train.h).  They differ in
// which extent is ragged (rows i of D, or the contraction c) and in how an operand lies
// in memory: with c contiguous (a row of P or Q is one i or j), or with c as the rows
// ("strided": a row holds all i or j of one c).
//
//  * V_MFMA_F32_16X16X32 with fp32 accumulation.  Q feeds the instruction's rows and P its
//    columns, so that a lane's four results are four adjacent j of one row of D.
//  * One K step holds 64 c of both operands in LDS, copied there directly from memory.
//    A contiguous operand keeps rows of 128 bytes; a fragment is one 16-byte read per
//    lane.  A strided one keeps rows of BM or BN elements; a fragment is two of gfx950's
//    transposing 8-byte reads, each of which hands lane l of a 16-lane group the four c of
//    column l.  Both are XOR-swizzled (16-byte chunks of a row; 32-byte units) so that the
//    lanes of one read fall into distinct banks; the swizzle is in the copies' source
//    address, because LDS receives a wave's copy in lane order.
//  * What lies outside a segment, a matrix or the contraction is never read: those lanes'
//    offsets are outside their buffer descriptor, which gives zeros.  Rows of D outside
//    the segment are not written.
//  * A persistent grid walks the tiles; the segments' row tiles are counted on the device
//    from the offsets, which the host never reads.
#include "dg_device.h"
#include "dg_train.h"

namespace dg {

using namespace dev;

namespace {

constexpr int kStep = 64;        // c per step
constexpr int kXcdCount = 8;

struct Bf16 {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    typedef __bf16 elem;
    static __device__ __forceinline__ v4f mfma(v4i a, v4i b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
};
struct F16 {
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    typedef _Float16 elem;
    static __device__ __forceinline__ v4f mfma(v4i a, v4i b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
};

// two fp32 values rounded to nearest even and packed
template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    typedef typename T::elem v2 __attribute__((ext_vector_type(2)));
    const v2 t = {(typename T::elem)x, (typename T::elem)y};
    return __builtin_bit_cast(uint32_t, t);
}
template <typename T>
__device__ __forceinline__ void unpack2(uint32_t w, float& x, float& y) {
    typedef typename T::elem v2 __attribute__((ext_vector_type(2)));
    const v2 t = __builtin_bit_cast(v2, w);
    x = (float)t.x;
    y = (float)t.y;
}

// Swizzles (see the head of the file).  Contiguous operand: 16-byte chunk of a 128-byte
// row.  A 16-byte read takes a wave's lanes sixteen at a time, and not in order: four runs of
// four that pair rows 0-3 and 12-15 of one chunk with rows 4-11 of its neighbour.  This one
// keeps those sixteen, as well as any sixteen lanes in order, in distinct banks (an earlier one
// that did only the latter doubled the reads' time: 4 conflict cycles in 8).
__device__ __forceinline__ int swz_row(int row) { return (row >> 1) & 7; }
// Strided operand: 32-byte unit of a row of one c.  Half a wave's transposing read covers
// four consecutive c in each of two groups eight apart: eight rows, eight distinct units.
__device__ __forceinline__ int swz_c(int c) { return (c & 3) | (((c >> 3) & 1) << 2); }

// Tile r of a group of ni x nj tiles: bands of kBand row tiles, down a band's column before
// the next column.  The 32 tiles that an XCD works on at a time are then a block of 8 x 4,
// whose operands its L2 fetches once.
constexpr int kBand = 8;
__device__ __forceinline__ void band_order(long r, int ni, int nj, int& ti, int& tj) {
    const int band = (int)(r / ((long)kBand * nj));
    const int rest = (int)(r - (long)band * kBand * nj), height = min(kBand, ni - band * kBand);
    ti = band * kBand + rest % height;
    tj = rest / height;
}

template <typename T, int OP, int BM, int BN, int WM, int WN, bool OUT32>
__global__ void __launch_bounds__(WM * WN * 64)
ragged_gemm_kernel(const RaggedParams p) {
    constexpr int NW = WM * WN;
    constexpr bool PS = OP == kRaggedTN, QS = OP != kRaggedNT;   // strided operands
    constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
    constexpr int P_BYTES = BM * kStep * 2, STAGE = (BM + BN) * kStep * 2;
    constexpr int P_SLOTS = BM / 8, Q_SLOTS = BN / 8;            // 1 KiB copies per step
    constexpr int P_PER = P_SLOTS / NW, Q_PER = Q_SLOTS / NW;
    static_assert(P_SLOTS % NW == 0 && Q_SLOTS % NW == 0, "copies are dealt evenly to the waves");
    static_assert(!PS || BM >= 128, "strided rows of whole 256-byte spans");
    static_assert(!QS || BN >= 128, "strided rows of whole 256-byte spans");
    static_assert(FN % 2 == 0, "the epilogue stores pairs of sub-tiles");

    // (each stage its own array, so that reads of one provably miss the copies into the other)
    __shared__ __attribute__((aligned(1024))) uint8_t smem0[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t smem1[STAGE];
    __shared__ int s_off[kMaxRaggedGroups + 1];                              // clamped, non-decreasing
    __shared__ int s_tiles[OP == kRaggedTN ? 1 : kMaxRaggedGroups + 1];      // row tiles before a group

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int l16 = lane & 15, lgrp = lane >> 4;
    const int G = p.groups;

    // ---- segments: s_off[g] = the largest of offsets[0..g], clamped to [0, rows], so that
    // no offsets, whatever they hold, lead outside the operands ----
    if (wave == 0) {
        const int per = (G + 1 + 63) / 64, g0 = lane * per;
        int top = 0;
        for (int i = 0; i < per; ++i)
            if (g0 + i <= G) top = max(top, min(p.offsets[g0 + i], p.rows));
        int before = top;
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(before, d, 64);
            if (lane >= d) before = max(before, v);
        }
        before = __shfl_up(before, 1, 64);
        if (lane == 0) before = 0;
        for (int i = 0; i < per; ++i)
            if (g0 + i <= G) {
                before = max(before, min(p.offsets[g0 + i], p.rows));
                s_off[g0 + i] = before;
            }
    }
    __syncthreads();
    long total;
    if constexpr (OP == kRaggedTN) {
        total = (long)G * p.tiles_i * p.tiles_j;
    } else {
        if (wave == 0) {
            const int per = (G + 63) / 64, g0 = lane * per;
            int own = 0;
            for (int i = 0; i < per; ++i)
                if (g0 + i < G) own += (s_off[g0 + i + 1] - s_off[g0 + i] + BM - 1) / BM;
            int incl = own;
            for (int d = 1; d < 64; d <<= 1) {
                const int v = __shfl_up(incl, d, 64);
                if (lane >= d) incl += v;
            }
            int run = incl - own;
            for (int i = 0; i < per; ++i)
                if (g0 + i < G) {
                    s_tiles[g0 + i] = run;
                    run += (s_off[g0 + i + 1] - s_off[g0 + i] + BM - 1) / BM;
                }
            if (lane == 63) s_tiles[G] = incl;
        }
        __syncthreads();
        total = (long)s_tiles[G] * p.tiles_j;
    }

    // ---- a lane's place in its copies.  A copy is 1 KiB of a stage: 8 rows of 128 bytes
    // (contiguous) or RPS rows of BM or BN elements (strided).  A wave's copies are NW slots
    // apart, a multiple of 16 rows, so that they share the lane's swizzled chunk and differ
    // by a whole number of rows. ----
    constexpr int P_RPS = PS ? 512 / BM : 8, Q_RPS = QS ? 512 / BN : 8;
    static_assert(NW * P_RPS % 16 == 0 && NW * Q_RPS % 16 == 0, "the swizzles' period");
    const int p_row = wave * P_RPS + lane / (64 / P_RPS), q_row = wave * Q_RPS + lane / (64 / Q_RPS);
    const int p_chunk = (lane % (64 / P_RPS)) ^ (PS ? swz_c(p_row) * 2 : swz_row(p_row));
    const int q_chunk = (lane % (64 / Q_RPS)) ^ (QS ? swz_c(q_row) * 2 : swz_row(q_row));
    const uint32_t p_lane = (uint32_t)(p_row * p.ldp + p_chunk * 8) * 2u, q_lane = (uint32_t)(q_row * p.ldq + q_chunk * 8) * 2u;
    const uint32_t p_next = (uint32_t)(NW * P_RPS * p.ldp) * 2u, q_next = (uint32_t)(NW * Q_RPS * p.ldq) * 2u;

    // ---- a lane's place in its fragments: byte offset in an operand's part of a stage of
    // sub-tile 0 of half 0; strided operands add (xor) the sub-tile's 32-byte unit to it, and
    // constants lead to the other sub-tiles and halves ----
    const int tr_c = lgrp * 8 + (l16 >> 2), tr_swz = swz_c(tr_c);
    const int p_frag = PS ? tr_c * BM * 2 + ((wm * (WTM / 16)) ^ tr_swz) * 32 + (l16 & 3) * 8
                          : (wm * WTM + l16) * 128 + (lgrp ^ swz_row(l16)) * 16;
    const int q_frag = QS ? tr_c * BN * 2 + ((wn * (WTN / 16)) ^ tr_swz) * 32 + (l16 & 3) * 8
                          : (wn * WTN + l16) * 128 + (lgrp ^ swz_row(l16)) * 16;

    for (long L0 = 0; L0 < total; L0 += gridDim.x) {
        const int P = gridDim.x, w = blockIdx.x;
        // neighbouring tiles to the workgroups of one XCD (they share its L2)
        const long L = L0 + (P % kXcdCount == 0 ? (w % kXcdCount) * (P / kXcdCount) + w / kXcdCount : w);
        if (L >= total) continue;      // uniform

        // ---- the tile: group, first i and j, rows of the segment ----
        int g, i0, j0, seg0, seg_rows;
        if constexpr (OP == kRaggedTN) {
            const int per = p.tiles_i * p.tiles_j;
            g = (int)(L / per);
            int ti, tj;
            band_order((int)(L - (long)g * per), p.tiles_i, p.tiles_j, ti, tj);
            i0 = ti * BM;
            j0 = tj * BN;
        } else {
            const int q = (int)(L / p.tiles_j);
            int lo = 0, hi = G;        // the last g with s_tiles[g] <= q
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_tiles[mid] <= q) lo = mid; else hi = mid;
            }
            g = lo;
            const int rt = s_tiles[g + 1] - s_tiles[g];
            int ti, tj;
            band_order(L - (long)s_tiles[g] * p.tiles_j, rt, p.tiles_j, ti, tj);
            i0 = ti * BM;
            j0 = tj * BN;
        }
        g = __builtin_amdgcn_readfirstlane(g);
        i0 = __builtin_amdgcn_readfirstlane(i0);
        j0 = __builtin_amdgcn_readfirstlane(j0);
        seg0 = __builtin_amdgcn_readfirstlane(s_off[g]);
        seg_rows = __builtin_amdgcn_readfirstlane(s_off[g + 1]) - seg0;

        const int ni = OP == kRaggedTN ? p.ni : seg_rows;
        const int nc = OP == kRaggedTN ? seg_rows : p.nc;
        const int steps = (nc + kStep - 1) / kStep;
        // base of P: its first row of the tile (contiguous) or of c = 0, at column i0 (strided)
        const uint16_t* pb = p.p + (PS ? (long)seg0 * p.ldp + i0 : (long)(seg0 + i0) * p.ldp);
        const uint16_t* qb = p.q + (OP == kRaggedTN ? (long)seg0 * p.ldq + j0
                                    : QS ? (long)g * p.q_gstride + j0
                                         : (long)g * p.q_gstride + (long)j0 * p.ldq);
        const uint32_t p_off = PS && i0 + p_chunk * 8 >= p.ni ? kOutside : p_lane;
        const uint32_t q_off = QS && j0 + q_chunk * 8 >= p.nj ? kOutside : q_lane;
        // contiguous operands: one descriptor for the tile, the step in the scalar offset, the
        // contraction's end by lane; strided ones: a descriptor per step, over the rows left
        const long p_bytes = (long)min(ni - i0, BM) * p.ldp * 2, q_bytes = (long)min(p.nj - j0, BN) * p.ldq * 2;
        struct Copies { __amdgpu_buffer_rsrc_t pr, qr; uint32_t po, qo, soff; };
        auto copies_of = [&](int s) DG_DEV_INLINE -> Copies {
            const int c0 = s * kStep, left = nc - c0;
            const bool some = left > 0, tail = left < kStep;
            return Copies{PS ? buffer_over(pb + (long)c0 * p.ldp, (long)min(left, kStep) * p.ldp * 2)
                             : buffer_over(pb, some ? p_bytes : 0),
                          QS ? buffer_over(qb + (long)c0 * p.ldq, (long)min(left, kStep) * p.ldq * 2)
                             : buffer_over(qb, some ? q_bytes : 0),
                          !PS && tail && p_chunk * 8 >= left ? kOutside : p_off,
                          !QS && tail && q_chunk * 8 >= left ? kOutside : q_off, some ? (uint32_t)c0 * 2u : 0u};
        };
        auto copy_one = [&](uint8_t* st, const Copies& c, int i) DG_DEV_INLINE {
            if (i < P_PER) {
                copy_to_lds16(c.pr, (lds_void*)(st + (wave + i * NW) * 1024), c.po + i * p_next, PS ? 0u : c.soff);
            } else {
                i -= P_PER;
                copy_to_lds16(c.qr, (lds_void*)(st + P_BYTES + (wave + i * NW) * 1024), c.qo + i * q_next, QS ? 0u : c.soff);
            }
        };

        // Fragment of sub-tile f, half h.  The lane's offset is hidden from the compiler at each
        // use, so that it computes the few addresses it needs (one xor or a constant offset
        // each) instead of keeping one register for every fragment of every stage.
        auto frag_row = [&](const uint8_t* b, int at, int f, int h) DG_DEV_INLINE -> v4i {
            typedef __attribute__((address_space(3))) const v4i lds_v4i;
            return *(lds_v4i*)((const lds_u8*)b + ((at ^ (h * 64)) + f * 2048));
        };
        auto frag_tr = [&](const uint8_t* b, int at, int f, int h, int width) DG_DEV_INLINE -> v4i {
            typedef short v4s __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) v4s lds_v4s;
            lds_u8* a = (lds_u8*)b + ((at ^ (f * 32)) + h * 32 * width * 2);
            const v2i lo = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)a));
            const v2i hi = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(a + 4 * width * 2)));
            return v4i{lo.x, lo.y, hi.x, hi.y};
        };

        v4f acc[FM][FN];
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
#pragma unroll
            for (int fn = 0; fn < FN; ++fn) acc[fm][fn] = v4f{0.f, 0.f, 0.f, 0.f};

        // fragments of half h of a step: one set is multiplied while the other is read
        v4i pf[2][FM], qf[2][FN];
        constexpr int NREAD = FM + FN, NCOPY = P_PER + Q_PER;
        // read i of a half, in the order in which the products need them
        auto read_one = [&](const uint8_t* st, int pa, int qa, int h, int i) DG_DEV_INLINE {
            if (i < FN) qf[h][i] = QS ? frag_tr(st + P_BYTES, qa, i, h, BN) : frag_row(st + P_BYTES, qa, i, h);
            else pf[h][i - FN] = PS ? frag_tr(st, pa, i - FN, h, BM) : frag_row(st, pa, i - FN, h);
        };
        // One half's products, row of sub-tiles by row, with the other half's reads and the copies
        // dealt out between the rows, so that neither the LDS nor the memory pipeline's queue
        // ever holds up the matrix core.  (The scheduling barriers keep the compiler from
        // collecting them again.)
        auto half = [&](auto which, const uint8_t* read_from, uint8_t* copy_to, const Copies* c) DG_DEV_INLINE {
            constexpr int h = decltype(which)::value;
            int pa = p_frag, qa = q_frag;
            asm volatile("" : "+v"(pa), "+v"(qa));
#pragma unroll
            for (int fm = 0; fm < FM; ++fm) {
#pragma unroll
                for (int fn = 0; fn < FN; ++fn) acc[fm][fn] = T::mfma(qf[h][fn], pf[h][fm], acc[fm][fn]);
                if constexpr (h == 1) {
#pragma unroll
                    for (int i = fm * NCOPY / FM; i < (fm + 1) * NCOPY / FM; ++i) copy_one(copy_to, *c, i);
                }
                // (a quarter of the rows is left for the last reads to land)
                constexpr int R = FM > 3 ? FM * 3 / 4 : FM;
#pragma unroll
                for (int i = fm * NREAD / R; i < (fm + 1) * NREAD / R && i < NREAD; ++i)
                    read_one(read_from, pa, qa, 1 - h, i);
                __builtin_amdgcn_sched_barrier(0);
            }
        };

        // ---- contraction.  The one barrier of a step sits between its halves: by then every
        // wave holds the second half's fragments, so the stage is free for the copies of the
        // step after next, and every wave's copies of the next step have landed, so its
        // first half is read while this step's second half is multiplied. ----
        if (steps > 0) {
            // Past the last step, copies read nothing and write zeros and reads bring what nobody
            // uses: the loop has no special last steps.
            constexpr std::integral_constant<int, 0> first{};
            constexpr std::integral_constant<int, 1> second{};
            wait_vmem<0>();      // the last tile's copies past its end
            const Copies c0 = copies_of(0), c1 = copies_of(1);
#pragma unroll
            for (int i = 0; i < NCOPY; ++i) copy_one(smem0, c0, i);
#pragma unroll
            for (int i = 0; i < NCOPY; ++i) copy_one(smem1, c1, i);
            wait_vmem<NCOPY>();
            barrier_only();
#pragma unroll
            for (int i = 0; i < NREAD; ++i) read_one(smem0, p_frag, q_frag, 0, i);
            auto step = [&](int s, uint8_t* cur, uint8_t* next) DG_DEV_INLINE {
                half(first, cur, cur, nullptr);
                wait_vmem<0>();
                wait_lds();
                barrier_only();
                const Copies c = copies_of(s + 2);
                half(second, next, cur, &c);
            };
            for (int s = 0; s < steps; s += 2) {
                step(s, smem0, smem1);
                if (s + 1 < steps) step(s + 1, smem1, smem0);
            }
        }

        // ---- epilogue: lane l16 holds row l16 of a sub-tile, columns 4 lgrp .. + 3 ----
        const int rows_left = ni - i0;
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            const int li = wm * WTM + fm * 16 + l16;
            const bool row_ok = li < rows_left;
            const long drow = OP == kRaggedTN ? (long)g * p.d_gstride + (long)(row_ok ? i0 + li : 0) * p.ldd
                                              : (long)(seg0 + (row_ok ? i0 + li : 0)) * p.ldd;
            if constexpr (OUT32) {
#pragma unroll
                for (int fn = 0; fn < FN; ++fn) {
                    const int col = j0 + wn * WTN + fn * 16 + lgrp * 4;
                    if (row_ok && col < p.nj) {
                        v4f* at = (v4f*)((float*)p.d + drow + col);
                        *at = p.accumulate ? *at + acc[fm][fn] : acc[fm][fn];
                    }
                }
            } else {
                // the swap of adjacent 16-lane rows gives every lane eight adjacent columns:
                // group lgrp then holds sub-tile fn + (lgrp & 1), columns 8 (lgrp >> 1) .. + 7
#pragma unroll
                for (int fn = 0; fn < FN; fn += 2) {
                    const v4f x = acc[fm][fn], y = acc[fm][fn + 1];
                    const int col = j0 + wn * WTN + (fn + (lgrp & 1)) * 16 + (lgrp >> 1) * 8;
                    const bool ok = row_ok && col < p.nj;
                    uint4* at = (uint4*)((uint16_t*)p.d + drow + (ok ? col : 0));
                    if (OP == kRaggedTN && p.accumulate) {
                        // the sums are added in fp32 and rounded once: exchange them unrounded
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const auto sw = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[e]), __float_as_uint(y[e]),
                                                                             false, false);
                            v[e] = __uint_as_float(sw[0]);
                            v[4 + e] = __uint_as_float(sw[1]);
                        }
                        if (ok) {
                            uint4 old = *at;
                            uint32_t* ow = (uint32_t*)&old;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float a, b;
                                unpack2<T>(ow[e], a, b);
                                ow[e] = pack2<T>(a + v[2 * e], b + v[2 * e + 1]);
                            }
                            *at = old;
                        }
                    } else {
                        const auto s0 = __builtin_amdgcn_permlane16_swap(pack2<T>(x[0], x[1]), pack2<T>(y[0], y[1]), false, false);
                        const auto s1 = __builtin_amdgcn_permlane16_swap(pack2<T>(x[2], x[3]), pack2<T>(y[2], y[3]), false, false);
                        if (ok) *at = uint4{s0[0], s1[0], s0[1], s1[1]};
                    }
                }
            }
        }
    }
}

template <typename T, int OP, int BM, int BN, int WM, int WN, bool OUT32>
hipError_t launch_ragged(const RaggedParams& p, int grid, hipStream_t stream) {
    hipLaunchKernelGGL((ragged_gemm_kernel<T, OP, BM, BN, WM, WN, OUT32>), dim3(grid), dim3(WM * WN * 64), 0, stream, p);
    return hipGetLastError();
}
template <typename T, int OP, int BM, int BN, int WM, int WN, bool OUT32>
hipError_t occupancy_ragged(int* blocks) {
    return hipOccupancyMaxActiveBlocksPerMultiprocessor(blocks, ragged_gemm_kernel<T, OP, BM, BN, WM, WN, OUT32>,
                                                        WM * WN * 64, 0);
}

// Relative times: 1024 256x256 tiles' worth of products take 4 (one workgroup a CU), with
// 128x128 tiles (two a CU) 1/0.85 of it, from the forward pass of 32768 x 4096 x 7168 in
// eight groups: 1647 us and 1929 us.  Few tiles: 64 x 4096 x 7168 in 16 groups 193 us and 156 us.
#define DG_RAGGED_256(T, HALF, OP, OUT32)                                                  \
    {OP, HALF, OUT32, 256, 256, 4.0, 4.0, &launch_ragged<T, OP, 256, 256, 2, 4, OUT32>,    \
     &occupancy_ragged<T, OP, 256, 256, 2, 4, OUT32>}
#define DG_RAGGED_128(T, HALF, OP, OUT32)                                                  \
    {OP, HALF, OUT32, 128, 128, 2.35, 1.4, &launch_ragged<T, OP, 128, 128, 2, 2, OUT32>,   \
     &occupancy_ragged<T, OP, 128, 128, 2, 2, OUT32>}
#define DG_RAGGED_TYPE(T, HALF)                                                            \
    DG_RAGGED_256(T, HALF, kRaggedNT, false), DG_RAGGED_128(T, HALF, kRaggedNT, false),    \
    DG_RAGGED_256(T, HALF, kRaggedNN, false), DG_RAGGED_128(T, HALF, kRaggedNN, false),    \
    DG_RAGGED_256(T, HALF, kRaggedTN, false), DG_RAGGED_128(T, HALF, kRaggedTN, false),    \
    DG_RAGGED_256(T, HALF, kRaggedTN, true), DG_RAGGED_128(T, HALF, kRaggedTN, true)

const RaggedConfig kConfigs[] = {DG_RAGGED_TYPE(Bf16, 0), DG_RAGGED_TYPE(F16, 1)};

}  // namespace

const RaggedConfig* ragged_configs(int* count) {
    *count = (int)(sizeof(kConfigs) / sizeof(kConfigs[0]));
    return kConfigs;
}

}  // namespace dg

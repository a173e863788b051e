// head_loss.cuh -- K15: losses over the tied head's vocabulary without keeping the logits: softmax
// cross entropy and distillation from a teacher's top logits, forward and backward.
//
// With the normalised hidden rows x [m][d] and the table T [vocab][d], s = x T^T:
//   forward   lse_r = log sum_v exp(s_rv / tau): logits tiles live in tensor memory only; each tile
//             leaves one (maximum, sum) pair per row, and a small kernel joins the pairs of a row.
//   backward  g_rv = c_r (exp(s_rv / tau - lse_r) - teacher_rv), dx = g T, dT = g^T x, in pieces of
//             the vocabulary: one launch recomputes a piece's logits and writes its g (bf16), one
//             launch forms both products from it. Nothing of size m x vocab is kept.
// Rows without a target are left out before any product: a scan lists the live rows, a gather copies
// them together, and every kernel reads the live count on the device (no host synchronisation, and
// what a dropped row holds, NaN included, reaches nothing).
//
// All three products are one warp-specialised tcgen05 kernel on pairs of CTAs (cta_group::2): a pair
// owns a 256 x 256 tile, each CTA loads its 128 rows of A and its 128 columns' half of B and holds its
// 128 x 256 of D, so that a k-block costs 32 KB of L2 reads per CTA; with single CTAs and 128 x 256
// tiles it is 48 KB, and those reads (13.5 TB/s) held the kernel at 1150 TFLOP/s. Per CTA a TMA
// producer thread and eight epilogue warps, one MMA thread in the pair's first CTA, persistent over
// tiles, two accumulators in tensor memory so that a tile's epilogue runs under the next tile's MMAs.
//
// Operands of a bf16 table are bf16; float32 rows beside it enter as three bf16 planes that add up to
// them exactly (8 + 8 + 8 significant bits, by truncation), and a product of float32 accuracy runs over
// the plane pairs (i, j) with i + j <= 2, smallest terms first.
//
// With a float32 table everything is fp16 in two planes instead, hi = fp16(v 2^k), lo = fp16(v 2^k -
// hi): 11 + 11 bits rounded to nearest, within 2^-22 of v, so three pairs (i + j <= 1; what they drop is
// 2^-22 too) do what six do in bf16. The power of two keeps fp16's range: one per row for x (taken out
// in the epilogue), one for the table (the forward: one per row of it), one for c x (c = dloss / tau),
// which is the rows' side of dT, and 2^15 for g / c = p - teacher, which lies in [-1, 1]. Values below
// 2^-17 of such a maximum lose bits one by one down to 2^-39 of it: less than float32's rounding of the
// sums they enter, though not of a single p far below 2^-17, nor of a row of dtable that only rows of a
// dloss far below the largest one reach.
//
// The tensor cores' float32 accumulator cuts bits off at every step of K = 16, towards zero: a bias of
// about half an ulp of the running sum per step, 1.3e-6 of logits of size 2 at d = 1024 and 3.8e-6 at
// 2560 (a float32 sum on the CUDA cores: below 1e-9). For the logits, and for every gradient with a
// float32 operand, the kernel therefore starts a new accumulator every FLUSH_KB k-blocks and the epilogue
// adds the pieces in registers, rounding to nearest. (Relative error of the loss at d = 1024: 1.2e-6
// without, 5.9e-7 with 8 k-blocks, 2.6e-7 with 4; of a float32 product 3.6e-7. With bf16 operands 4 k-blocks
// cost 9% of forward + backward at 16384 x 1024 against 8.) The backward's logits are added up as the
// forward's were, to the bit: p = exp(s / tau - lse) sums to one then, whatever s itself is off by, and
// 1 - p of a row that is sure of its target keeps its digits (before, 1 - p of some 1e-3 at d = 2560 was off
// by 6% and more; 1% of 16384 x 1024 forward + backward).
//
// Measured (32000 words, bf16, back to back): 16384 x 1024 forward + backward 3.56 ms = 1147 TFLOP/s of
// 8 m vocab d (5% of the rows left out), 0.83 of the sustained cuBLAS rate; 16384 x 2560 6.3 ms = 1185
// (0.86). Alone, 4096 x 1024: statistics 206 us (1306 TFLOP/s), g 220 (1222), products 392 (1369); the
// tensor pipe is active 73 / 66 / 79% of the cycles at 1.6 GHz. No other unit is near its limit: TMA loads
// 10 TB/s out of the L2 (a third of the crossbar's rate), shared memory's banks 17 to 19% busy reading and
// as much writing. What is lost: waits between a tile's accumulators, 28 rounds of tiles paid for 27.03,
// start and end of the launch (6%), and the clock, which the power cap holds below 1.65 GHz. Few rows
// (40 x 1024): 23 us forward, of which 11 us are the table's 65.5 MB and the rest set-up, HBM's first bytes
// and the join.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "pair_exit.cuh"

namespace mmf {
namespace hl {

constexpr int CM = 128;        // rows of D per CTA
constexpr int BM = 2 * CM;     // rows of D per tile (MMA M, over the pair)
constexpr int BN = 256;        // columns of D per tile (MMA N)
constexpr int BK = 64;         // bf16 per k-block: one 128-byte swizzle atom
constexpr int UK = 16;         // K per kind::f16 instruction
constexpr int STAGES = 5;
// k-blocks per accumulator where pieces are added in registers: with bf16 operands, and with float32 ones
// (whose lower planes' products share the first accumulator)
constexpr int FLUSH_KB = 8, FLUSH_KB_F32 = 4;
constexpr int BOX_BYTES = 64 * BK * 2;  // every TMA load box: 64 x 64 bf16, 8 KB
constexpr int A_BOXES = CM / 64, B_BOXES = BN / 2 / 64;  // per CTA
constexpr int STAGE_BYTES = (A_BOXES + B_BOXES) * BOX_BYTES;
constexpr int EPI_WARPS = 8;   // two per tensor-memory lane quarter, each half of the columns
constexpr int THREADS = (4 + EPI_WARPS) * 32;
constexpr int OUT_BYTES = 4096;  // a staging buffer of an epilogue warp: 32 rows x 128 bytes
constexpr int OUT_BUFS = 2;      // ... of which one is filled while the other one is being stored
constexpr int NUM_BARS = 2 * STAGES + 5;
constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_WARPS * OUT_BUFS * OUT_BYTES + NUM_BARS * 8 + 16;
constexpr uint32_t TMEM_COLS = 2 * BN;
constexpr int PLANES = 3;      // bf16 planes of a float32 operand
constexpr int MAX_PRODS = 6;
constexpr int MAX_TOP = 256;   // teacher entries per row
constexpr float kLog2e = 1.4426950408889634f;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");

enum Mode : int { kStats = 0, kGrad = 1, kProducts = 2 };

// Plane pairs of one product, smallest terms first.
struct Prods {
  int32_t n;
  uint8_t a[MAX_PRODS], b[MAX_PRODS];
};

struct Params {
  CUtensorMap x;    // live rows, planes   [px][m_pad][d], 16 bits, box 64 x 64 (all loads); kProducts with
                    // a float32 table: c x
  CUtensorMap t;    // table, planes       [pt][vocab][d]
  CUtensorMap g;    // the piece's g       [pg][m_pad][ldg], inner extent = piece columns; one plane
                    // rounded to nearest, three that split it exactly, or (fp16) two of g / c
  CUtensorMap g_out;   // the same array, box 64 x 32 (stores)
  CUtensorMap dx_out;  // float32 partials [splits][m_pad][d], box 32 x 32
  CUtensorMap dt_out;  // dtable's rows of the piece (its dtype), or float32 partials [planes][vocab][d]
  const int32_t* live;  // device: live rows; nullptr: rows of the caller's x, taken as they are (kStats)
  int32_t rows;
  int32_t d, vocab;
  int32_t v0, vn;       // vocabulary range of this launch
  int64_t m_pad;
  float scale;          // log2(e) / tau (kStats)
  float inv_tau;        // (kGrad)
  const int32_t* tgt;   // [m_pad] target of each live row, or nullptr (kStats, kGrad)
  const float* lse;     // [m_pad] (kGrad)
  const float* c;       // [m_pad] dloss / tau (kGrad)
  float2* part;         // [2 * column tiles][m_pad] (maximum, sum) (kStats)
  float* st;            // [m_pad] target logit (kStats)
  // distillation (kStats): the teacher's entries of every row in order of their ids
  const int2* top;      // [m][top_k] (id, entry), or nullptr
  const uint16_t* top_start;  // [2 * column tiles][m_pad] the row's first entry in the tile's half
  const int32_t* rowmap;      // [m_pad] row of each live row
  float* s_top;         // [m][top_k] out: the student's logits at the entries
  int32_t top_k;
  Prods fwd, dxp, dtp;
  int32_t dx_split;             // K splits of dx in this launch (0: no dx)
  int32_t dx_add;               // a later piece: dx's partials are added to
  int32_t dt_split;             // K splits of dT (0: no dT)
  int32_t dt_f32;               // dt_out holds float32
  // float32 tables (fp16 planes): the powers of two to take out, else nullptr
  const float* x_unit;          // [m_pad] of each row of x
  const float* t_unit;          // of the table (backward)
  const float* t_units;         // [vocab] of each row of the table (forward)
  const float* dt_unit;         // of c x
  int32_t dt_row0;              // first row of dt_out this launch writes
  // kProducts with few rows: dx^T = T^T g^T, so that M is 256 columns of d and N the rows, in 64s; with
  // 256 rows as M, 40 of them cost what 256 do
  int32_t few_n;                // N, or 0
  float* dx_part;               // dx_out's array
  uint32_t wait_limit_us;
};

// ---------------------------------------------------------------------------------------------
// PTX used here only
// ---------------------------------------------------------------------------------------------
// Load into this CTA's shared memory, counted on a barrier of either CTA of the pair (a
// shared::cluster address).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(src)
               : "memory");
}
// The same, added to what is there (float32).
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// all stores but the latest N have read their shared memory
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Programmatic dependent launch: the next kernel's blocks may start (their set-up overlaps this
// kernel's end), and nothing an earlier kernel wrote is read, and nothing written, before the wait.
__device__ __forceinline__ void let_dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependent() {
  let_dependents_start();
  dependency_wait();
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// shared::cluster address of `p` in the pair's CTA `rank`
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t in_first_cta(const uint64_t* bar) { return in_cta(bar, 0); }
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrives on `bar` (the same place in both CTAs) when all MMAs issued so far have completed.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tc_mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float r;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
  return r;
}
// 2^v by the hardware approximation (2 ulp over the range the softmax needs; 0 for -inf).
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// Shared-memory descriptor of an MN-major, 128-byte-swizzled operand: atoms of 64 MN elements (128
// bytes) x 8 k rows. Leading byte offset = the next 64 MN elements (one box), stride byte offset =
// the next 8 k rows.
__device__ __forceinline__ uint64_t mn128_desc(uint32_t smem_addr) {
  return (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | ((uint64_t)(BOX_BYTES >> 4) << 16) | ((uint64_t)64u << 32) |
         ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

// x = p0 + p1 + p2 exactly: each plane keeps the 8 leading significant bits of what is left
// (truncation never overflows). An infinity or NaN stays whole in the first plane.
__device__ __forceinline__ float trunc_bf16(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }
// Takes the leading plane off v and leaves the rest.
__device__ __forceinline__ float peel(float& v) {
  const bool finite = (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u;
  const float p = v != v ? __uint_as_float(0x7fc00000u) : trunc_bf16(v);
  v = finite ? v - p : 0.0f;
  return p;
}
__device__ __forceinline__ void split3(float v, float& p0, float& p1, float& p2) {
  p0 = peel(v);
  p1 = peel(v);
  p2 = peel(v);
}
// v 2^k as two fp16 planes; v leaves with the rest after the first. An infinity or NaN stays whole.
constexpr float kGradUnit = 32768.0f;  // g / c as fp16: |g / c| <= 1
__device__ __forceinline__ float peel_half(float& v) {
  const float h = __half2float(__float2half_rn(v));
  v = (__float_as_uint(h) & 0x7f800000u) == 0x7f800000u ? 0.0f : v - h;
  return h;
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// two finite values (or NaN) at once
__device__ __forceinline__ uint32_t peel_half2(float& a, float& b) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  a -= f.x;
  b -= f.y;
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^k that brings `most`, the largest finite magnitude, to [2^14, 2^15); 2^126 at most, the largest whose
// reciprocal is normal (below 2^-112 it falls short of 2^14).
__device__ __forceinline__ float unit_up(float most) {
  const int e = (int)(__float_as_uint(most) >> 23) - 127;  // floor(log2); -127 for zero and subnormals
  const int k = 14 - e > 126 ? 126 : 14 - e;               // -113 at least
  return most > 0.0f ? __uint_as_float((uint32_t)(127 + k) << 23) : 1.0f;
}
__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a <= 3.402823466e38f ? a : 0.0f;  // infinities and NaN do not count
}
__device__ __forceinline__ uint32_t pack_bf16_rn(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// two values to bf16, leaving what the rounding took off them
__device__ __forceinline__ uint32_t peel_bf16_rn(float& a, float& b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  const float2 f = __bfloat1622float2(p);
  a = (__float_as_uint(f.x) & 0x7f800000u) == 0x7f800000u ? 0.0f : a - f.x;
  b = (__float_as_uint(f.y) & 0x7f800000u) == 0x7f800000u ? 0.0f : b - f.y;
  return *reinterpret_cast<const uint32_t*>(&p);
}
// two values that are exact in bf16
__device__ __forceinline__ uint32_t pack_bf16_hi(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}

// ---------------------------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------------------------
struct Tile {
  int row, col;     // first row / column of D
  int kb0, nkb;     // k-blocks (per plane pair)
  int nprod;
  int kind;         // kProducts: 0 = dT, 1 = dx, 2 = dx of few rows; else 0
  int split;
  int n;            // columns of D (MMA N)
};

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return a / b + (a % b != 0); }

// What all tiles of a launch share, worked out once per thread.
struct Geo {
  int tiles;
  int nt, nt_dx;           // column tiles
  int mt;                  // row tiles (kStats, kGrad)
  int kb_d;                // k-blocks of d
  int per_dt, per_dx, end_dt;  // kProducts: tiles per split, tiles of dT
  int kb_dt, len_dt, kb_dx, len_dx;  // k-blocks, k-blocks per split
};

template <int MODE>
__device__ __forceinline__ Geo geometry(const Params& P, int live) {
  Geo G = {};
  if (MODE != kProducts) {
    G.mt = cdiv(live, BM);
    G.nt = cdiv(P.vn, BN);
    G.kb_d = cdiv(P.d, BK);
    G.tiles = G.mt * G.nt;
  } else {
    G.nt = cdiv(P.d, BN);
    G.per_dt = cdiv(P.vn, BM) * G.nt;
    G.nt_dx = P.few_n > 0 ? 1 : G.nt;
    G.per_dx = P.few_n > 0 ? (live > 0 ? cdiv(P.d, BM) : 0) : cdiv(live, BM) * G.nt;
    G.end_dt = P.dt_split * G.per_dt;
    G.tiles = G.end_dt + P.dx_split * G.per_dx;
    G.kb_dt = cdiv(live, BK);
    G.kb_dx = cdiv(P.vn, BK);
    G.len_dt = P.dt_split > 1 ? cdiv(G.kb_dt, P.dt_split) : G.kb_dt;
    G.len_dx = P.dx_split > 1 ? cdiv(G.kb_dx, P.dx_split) : G.kb_dx;
  }
  return G;
}

template <int MODE>
__device__ __forceinline__ Tile tile_at(const Params& P, const Geo& G, int t) {
  Tile T;
  T.kind = 0;
  T.split = 0;
  T.n = BN;
  if (MODE != kProducts) {
    // groups of sixteen row tiles, columns slow inside a group: the pairs of one wave share a few row
    // tiles and a few table tiles, which the L2 then serves (eight: 1.2% slower at 16384 x 1024)
    constexpr int R = 16;
    const int grp = t / (R * G.nt), rem = t - grp * (R * G.nt);
    const int gm = G.mt - grp * R < R ? G.mt - grp * R : R;
    const int c = gm == R ? rem / R : rem / gm;
    T.row = (grp * R + rem - c * gm) * BM;
    T.col = c * BN;
    T.kb0 = 0;
    T.nkb = G.kb_d;
    T.nprod = P.fwd.n;
    return T;
  }
  int kb, len, rem, nt = G.nt;
  if (t < G.end_dt) {
    T.split = P.dt_split > 1 ? t / G.per_dt : 0;
    rem = t - T.split * G.per_dt;
    kb = G.kb_dt;
    len = G.len_dt;
    T.nprod = P.dtp.n;
  } else {
    t -= G.end_dt;
    T.kind = 1;
    T.split = P.dx_split > 1 ? t / G.per_dx : 0;
    rem = t - T.split * G.per_dx;
    kb = G.kb_dx;
    len = G.len_dx;
    T.nprod = P.dxp.n;
    nt = G.nt_dx;
    if (P.few_n > 0) {
      T.kind = 2;
      T.n = P.few_n;
    }
  }
  const int m = rem / nt;
  T.row = m * BM;
  T.col = (rem - m * nt) * BN;
  T.kb0 = T.split * len;
  T.nkb = kb - T.kb0 < len ? kb - T.kb0 : len;
  if (T.nkb < 0) T.nkb = 0;
  return T;
}

// Accumulators (segments of K) of a tile, and the k-blocks of one: KB of the leading planes'
// product, the last in order. The products before it are 2^-8 or less of it, and so is what the
// accumulator cuts off them: they all go into the first segment.
template <bool FLUSH, int KB>
__device__ __forceinline__ int tile_segments(const Tile& T) {
  return FLUSH && T.nkb > KB ? cdiv(T.nkb, KB) : 1;
}
template <bool FLUSH, int KB>
__device__ __forceinline__ int segment_blocks(const Tile& T, int seg) {
  if (!FLUSH) return T.nprod * T.nkb;
  const int left = T.nkb - seg * KB;
  return (seg == 0 ? (T.nprod - 1) * T.nkb : 0) + (left < KB ? left : KB);
}

// How g is held (GP of kGrad and of its products).
enum GradPlanes : int {
  kOne = 1,    // one bf16 value
  kHalf2 = 2,  // two fp16 values of g / c (float32 table)
  kExact3 = 3, // three bf16 values, exact (float32 rows beside a bf16 table)
  kFine2 = 4   // two bf16 values rounded to nearest (few bf16 rows)
};
__host__ __device__ constexpr int grad_planes(int gp) { return gp == kFine2 ? 2 : gp; }

// GP: kGrad's GradPlanes; kStats and kProducts: 1 with bf16 results and operands, else 2.
template <int MODE, int GP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) head_loss_kernel(const __grid_constant__ Params P) {
  // kStats and kGrad add up the logits alike, to the bit, so that p = exp(s / tau - lse) fits its lse
  constexpr bool FLUSH = MODE != kProducts || GP > 1;
  constexpr int KB = GP > 1 && GP != kFine2 ? FLUSH_KB_F32 : FLUSH_KB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + STAGES * STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + EPI_WARPS * OUT_BUFS * OUT_BYTES);
  // full and accempty count in the pair's first CTA (both CTAs' copies and epilogue warps); empty,
  // accfull and drain are each CTA's own, reached by the MMA thread's multicast commits
  uint64_t* full = bars;                     // TMA -> MMA           (count 1 + both CTAs' bytes)
  uint64_t* empty = bars + STAGES;           // MMA commit -> TMA    (count 1)
  uint64_t* accfull = bars + 2 * STAGES;     // MMA commit -> epilogue, two accumulators
  uint64_t* accempty = accfull + 2;          // epilogues -> MMA     (count 2 * EPI_WARPS)
  uint64_t* drain = accempty + 2;            // everything the MMA thread issued
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // by rank, the same in both CTAs: stages the producer issued, with kGaveUp when one of its waits ran out
  volatile uint32_t* issued = tmem_slot + 2;
  constexpr uint32_t kGaveUp = 0x80000000u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t limit = P.wait_limit_us;
  const uint32_t rank = cluster_rank();
  let_dependents_start();
  const int first = (int)(blockIdx.x >> 1), stride = (int)(gridDim.x >> 1);  // this pair's tiles

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], 2 * EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 2) tmem_alloc_pair(tmem_slot, TMEM_COLS);
  if (warp == 3 && lane == 0) {
    tma_prefetch_desc(&P.x);
    tma_prefetch_desc(&P.t);
    if (MODE == kProducts) tma_prefetch_desc(&P.g);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and tensor memory are set up
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  dependency_wait();
  const int live = P.live ? *P.live : P.rows;
  const Geo G = geometry<MODE>(P, live);
  const int tiles = G.tiles;
  const int live64 = (live + 63) & ~63;
  // Fills iteration `it`'s stage with k-block kb of a plane pair; its slot has to be free.
  const auto fill = [&](const Tile& T, int pa, int pb, int kb, uint32_t it) {
    const uint32_t s = it % STAGES;
    const uint32_t sa = smem_u32(smem + s * STAGE_BYTES), sb = sa + A_BOXES * BOX_BYTES;
    const int k = (T.kb0 + kb) * BK;
    const uint32_t bar = in_first_cta(&full[s]);
    const int b_boxes = MODE == kProducts && T.n <= 128 ? 1 : B_BOXES;
    // kStats reads nothing of the rows past the last: boxes of such rows are left out (a row of A
    // reaches its own row of D only)
    int a_boxes = A_BOXES, a_both = 2 * A_BOXES;
    if (MODE == kStats) {
      const int left = live - T.row;
      a_both = left >= BM ? 2 * A_BOXES : (left + 63) >> 6;
      a_boxes = min(max(a_both - A_BOXES * (int)rank, 0), A_BOXES);
    }
    if (rank == 0) mbar_arrive_expect_tx(&full[s], (a_both + 2 * b_boxes) * BOX_BYTES);
    const int arow = T.row + CM * (int)rank, bcol = T.col + T.n / 2 * (int)rank;
    if (MODE == kProducts && T.kind == 2) {  // A MN-major, B K-major, k = vocabulary
#pragma unroll
      for (int i = 0; i < A_BOXES; ++i) tma_load_3d(sa + i * BOX_BYTES, &P.t, arow + 64 * i, P.v0 + k, pb, bar);
      for (int i = 0; i < b_boxes; ++i) tma_load_3d(sb + i * BOX_BYTES, &P.g, k, bcol + 64 * i, pa, bar);
    } else if (MODE != kProducts) {
#pragma unroll
      for (int i = 0; i < A_BOXES; ++i)
        if (i < a_boxes) tma_load_3d(sa + i * BOX_BYTES, &P.x, k, arow + 64 * i, pa, bar);
#pragma unroll
      for (int i = 0; i < B_BOXES; ++i) tma_load_3d(sb + i * BOX_BYTES, &P.t, k, P.v0 + bcol + 64 * i, pb, bar);
    } else if (T.kind == 0) {  // dT = g^T x: both operands MN-major, k = live rows
#pragma unroll
      for (int i = 0; i < A_BOXES; ++i) tma_load_3d(sa + i * BOX_BYTES, &P.g, arow + 64 * i, k, pa, bar);
#pragma unroll
      for (int i = 0; i < B_BOXES; ++i) tma_load_3d(sb + i * BOX_BYTES, &P.x, bcol + 64 * i, k, pb, bar);
    } else {  // dx = g T: A K-major, B MN-major, k = vocabulary
#pragma unroll
      for (int i = 0; i < A_BOXES; ++i) tma_load_3d(sa + i * BOX_BYTES, &P.g, k, arow + 64 * i, pa, bar);
#pragma unroll
      for (int i = 0; i < B_BOXES; ++i) tma_load_3d(sb + i * BOX_BYTES, &P.t, bcol + 64 * i, P.v0 + k, pb, bar);
    }
  };
  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += stride) {
        const Tile T = tile_at<MODE>(P, G, t);
        const Prods& pr = MODE != kProducts ? P.fwd : T.kind ? P.dxp : P.dtp;
        for (int p = 0; ok && p < T.nprod; ++p) {
          const int pa = pr.a[p], pb = pr.b[p];
          for (int kb = 0; kb < T.nkb; ++kb, ++it) {
            if (!mbar_wait_bounded(&empty[it % STAGES], ((it / STAGES) & 1u) ^ 1u, limit, abort_flag)) { ok = false; break; }
            fill(T, pa, pb, kb, it);
          }
        }
      }
      // the last stages' commits have reached this CTA before it ends
      for (uint32_t j = it > STAGES ? it - STAGES : 0; ok && j < it; ++j)
        ok = mbar_wait_bounded(&empty[j % STAGES], (j / STAGES) & 1u, limit, abort_flag);
      for (uint32_t r = 0; r < 2; ++r) st_cluster_u32(in_cta(const_cast<const uint32_t*>(issued) + rank, r), it | (ok ? 0u : kGaveUp));
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0 && rank == 0) {
      // kind::f16: D float32 (bits 4-5 = 1), A and B bf16 or fp16 (bits 7-9, 10-12), MN-major A / B at
      // bits 15 / 16, N >> 3 at bits 17-22, M >> 4 at bits 24-28
      const uint32_t fmt = P.x_unit ? 0u : 1u;  // fp16 : bf16
      const uint32_t idesc0 = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(BM >> 4) << 24);
      uint32_t it = 0, n = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += stride) {
        const Tile T = tile_at<MODE>(P, G, t);
        const bool a_mn = MODE == kProducts && T.kind != 1, b_mn = MODE == kProducts && T.kind != 2;
        const uint32_t idesc = idesc0 | ((uint32_t)(T.n >> 3) << 17) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
        const int segs = tile_segments<FLUSH, KB>(T);
        for (int seg = 0; ok && seg < segs; ++seg, ++n) {
          const uint32_t buf = n & 1u, acc = tmem + buf * BN;
          if (!mbar_wait_bounded(&accempty[buf], ((n >> 1) & 1u) ^ 1u, limit, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const int its = segment_blocks<FLUSH, KB>(T, seg);
          for (int i = 0; i < its; ++i, ++it) {
            const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
            if (!mbar_wait_bounded(&full[s], ph, limit, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + s * STAGE_BYTES), sb = sa + A_BOXES * BOX_BYTES;
#pragma unroll
            for (int kk = 0; kk < BK / UK; ++kk) {
              const uint64_t ad = a_mn ? mn128_desc(sa + kk * UK * 128) : sw128_desc(sa + kk * UK * 2);
              const uint64_t bd = b_mn ? mn128_desc(sb + kk * UK * 128) : sw128_desc(sb + kk * UK * 2);
              tc_mma_bf16_pair(acc, ad, bd, idesc, (i | kk) != 0 ? 1u : 0u);
            }
            tc_commit_pair(&empty[s]);
          }
          if (ok) tc_commit_pair(&accfull[buf]);
        }
      }
      // everything issued has completed before this thread reaches the teardown barrier
      tc_commit_pair(drain);
      mbar_wait_drain(drain, 0u);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t stg0 = smem_u32(staging + (warp - 4) * OUT_BUFS * OUT_BYTES);
    const uint32_t swz = (uint32_t)(lane & 7) << 4;
    uint32_t stg = stg0, stg_row = stg0 + lane * 128;  // the buffer being filled
    const auto next_buffer = [&] {
      if (OUT_BUFS > 1) stg = stg == stg0 ? stg0 + OUT_BYTES : stg0;
      stg_row = stg + lane * 128;
    };
    uint32_t n = 0;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += stride) {
      const Tile T = tile_at<MODE>(P, G, t);
      const int row0 = T.row + CM * (int)rank + quarter * 32, row = row0 + lane;
      const int nh = MODE == kProducts ? T.n / 2 : BN / 2;  // columns of this half
      const int col0 = T.col + half * nh;
      const bool zero = T.nprod * T.nkb == 0;  // no k-blocks: the accumulator was never written
      uint32_t acc = 0;
      float sum[FLUSH ? BN / 2 : 1];
      const int segs = tile_segments<FLUSH, KB>(T);
#pragma unroll 1
      for (int g = 0; g < segs; ++g, ++n) {
        const uint32_t buf = n & 1u;
        const bool have = mbar_wait_bounded(&accfull[buf], (n >> 1) & 1u, limit, abort_flag);
        if (!__all_sync(0xffffffffu, have)) { ok = false; break; }
        tc_fence_after();
        acc = tmem + buf * BN + half * nh + ((uint32_t)(quarter * 32) << 16);
        if (FLUSH) {
#pragma unroll
          for (int c0 = 0; c0 < BN / 2; c0 += 16) {
            if (MODE == kProducts && c0 >= nh) break;
            uint32_t w[16];
            tmem_ld_32x32b_x16(acc + c0, w);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              sum[c0 + e] = (g == 0 ? 0.0f : sum[c0 + e]) + __uint_as_float(w[e]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(in_first_cta(&accempty[buf]));
        }
      }
      if (!ok) break;
      if (FLUSH && zero) {
#pragma unroll
        for (int e = 0; e < (FLUSH ? BN / 2 : 1); ++e) sum[e] = 0.0f;
      }
      // the powers of two of fp16 operands: of the row and the table, or of dT's (dx's go where its
      // partials are added). A product of two that is past the range belongs to logits that are zero, or past
      // it too
      float unit = 1.0f;
      if (FLUSH && P.x_unit)
        unit = MODE == kStats   ? (row < live ? P.x_unit[row] : 0.0f)
               : MODE == kGrad  ? (row < live ? fminf(P.x_unit[row] * *P.t_unit, 3.402823466e38f) : 0.0f)
               : T.kind == 0    ? *P.dt_unit * (1.0f / kGradUnit)
                                : 1.0f;
      if (MODE == kStats && GP > 1 && P.t_units) {
        // s from the raw sum (2^45 at most): the smaller power first, so that a row of 2^-120 beside a word of
        // 2^120 stays in range on the way (what the sum loses below 2^-126 is 2^-36 of such a logit at most)
        const auto scaled = [&](float v, float u) { return v * fminf(unit, u) * fmaxf(unit, u); };
        const float4* u4 = reinterpret_cast<const float4*>(P.t_units + col0);  // one address for the warp
#pragma unroll
        for (int e = 0; e < (FLUSH ? BN / 2 : 0); e += 4) {
          const float4 u = u4[e / 4];
          sum[e] = scaled(sum[e], u.x);
          sum[e + 1] = scaled(sum[e + 1], u.y);
          sum[e + 2] = scaled(sum[e + 2], u.z);
          sum[e + 3] = scaled(sum[e + 3], u.w);
        }
      }
      // columns [c0, c0 + N) of D into v (with FLUSH they are in `sum` already)
      const auto cols32 = [&](int c0, float* v) {
        uint32_t w[32];
        tmem_ld_32x32b_x32(acc + c0, w);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = zero ? 0.0f : __uint_as_float(w[e]);
      };
      if (MODE == kStats) {
        constexpr int W = FLUSH ? BN / 2 : 1;  // kStats always runs with FLUSH
        const int left = P.vn - col0;
        if (left < W) {
#pragma unroll
          for (int e = 0; e < W; ++e)
            if (e >= left) sum[e] = -INFINITY;
        }
        const uint32_t tgt = P.tgt && row < live ? (uint32_t)P.tgt[row] - (uint32_t)(P.v0 + col0) : 0xffffffffu;
        if (tgt < (uint32_t)W) {
          float hit = 0.0f;
#pragma unroll
          for (int e = 0; e < W; ++e)
            if (tgt == (uint32_t)e) hit = sum[e];
          P.st[row] = hit;
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < W; ++e) m4[e & 3] = fmaxf(m4[e & 3], sum[e]);
        const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        const float scale = P.scale, off = top == -INFINITY ? 0.0f : -top * scale;
#pragma unroll
        for (int e = 0; e < W; ++e) s4[e & 3] += ex2(fmaf(sum[e], scale, off));
        if (row < live)
          P.part[(int64_t)((T.col / BN) * 2 + half) * P.m_pad + row] = make_float2(top, (s4[0] + s4[1]) + (s4[2] + s4[3]));
        if (P.top) {
          // the logits at the teacher's ids, while they are here: a group of 32 columns that holds one
          // of the warp's entries goes through the warp's staging rows, where it can be indexed
          int pos = P.top_k;
          int64_t base = 0;
          int2 ent = make_int2(0x7fffffff, 0);
          if (row < live) {
            const int32_t r = P.rowmap ? P.rowmap[row] : row;
            base = (int64_t)r * P.top_k;
            pos = P.top_start[(int64_t)((T.col / BN) * 2 + half) * P.m_pad + r];
            if (pos < P.top_k) ent = P.top[base + pos];
          }
#pragma unroll
          for (int c0 = 0; c0 < W; c0 += 32) {
            const int begin = col0 + c0;
            if (!__any_sync(0xffffffffu, ent.x < begin + 32)) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              st_shared_v4(stg_row + (((uint32_t)j << 4) ^ swz), __float_as_uint(sum[FLUSH ? c0 + 4 * j : 0]),
                           __float_as_uint(sum[FLUSH ? c0 + 4 * j + 1 : 0]), __float_as_uint(sum[FLUSH ? c0 + 4 * j + 2 : 0]),
                           __float_as_uint(sum[FLUSH ? c0 + 4 * j + 3 : 0]));
            while (ent.x < begin + 32) {  // at most top_k entries; a row reads what its own thread wrote
              const uint32_t c = (uint32_t)(ent.x - begin);
              P.s_top[base + ent.y] = ld_shared_f32(stg_row + (((c >> 2) << 4) ^ swz) + ((c & 3u) << 2));
              ent = ++pos < P.top_k ? P.top[base + pos] : make_int2(0x7fffffff, 0);
            }
          }
        }
      } else if (MODE == kGrad) {
        // pad rows have c = lse = 0: zeros, which dT's last k-block of rows relies on; past that nobody
        // reads what a row leaves
        const bool needed = row0 < live64;  // uniform across the warp
        constexpr bool halves = GP == kHalf2;
        const float c = !needed ? 0.0f : !halves ? P.c[row] : row < live ? kGradUnit : 0.0f;
        const float lse = needed ? P.lse[row] : 0.0f, inv_tau = P.inv_tau * unit;
        // s / tau - lse before the change of base: where p is near 1 it is a small difference, exact but for lse
        const auto prob = [&](float sv) { return ex2(fmaf(sv, inv_tau, -lse) * kLog2e); };
        const int tgt = needed && P.tgt ? P.tgt[row] - P.v0 - col0 : -1;
        if (needed && grad_planes(GP) != 2) {
#pragma unroll
          for (int e = 0; e < BN / 2; ++e) sum[FLUSH ? e : 0] = prob(sum[FLUSH ? e : 0]);
          if ((uint32_t)tgt < (uint32_t)(BN / 2)) {
#pragma unroll
            for (int e = 0; e < BN / 2; ++e)
              if (tgt == e) sum[FLUSH ? e : 0] -= 1.0f;
          }
#pragma unroll
          for (int e = 0; e < BN / 2; ++e) sum[FLUSH ? e : 0] *= c;
        }
#pragma unroll
        for (int c0 = 0; c0 < BN / 2; c0 += 64) {
          if (!needed || col0 + c0 >= P.vn) break;
          float* gv = sum + (FLUSH ? c0 : 0);
          if (grad_planes(GP) == 2) {
            // both planes at once, one per buffer: a value is worked out, split and gone
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int e = 8 * j + 2 * q;
                float a = prob(gv[e]), b = prob(gv[e + 1]);
                if (tgt - c0 == e) a -= 1.0f;
                if (tgt - c0 == e + 1) b -= 1.0f;
                a *= c;
                b *= c;
                hi[q] = halves ? peel_half2(a, b) : peel_bf16_rn(a, b);
                lo[q] = halves ? pack_half(a, b) : pack_bf16_rn(a, b);
              }
              const uint32_t at = lane * 128 + (((uint32_t)j << 4) ^ swz);
              st_shared_v4(stg0 + at, hi[0], hi[1], hi[2], hi[3]);
              st_shared_v4(stg0 + OUT_BYTES + at, lo[0], lo[1], lo[2], lo[3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&P.g_out, stg0, col0 + c0, row0, 0);
              tma_store_3d(&P.g_out, stg0 + OUT_BYTES, col0 + c0, row0, 1);
              bulk_commit();
            }
          } else {
#pragma unroll
            for (int p = 0; p < grad_planes(GP); ++p) {
              if (lane == 0) bulk_wait_read<OUT_BUFS - 1>();
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  float& a = gv[8 * j + 2 * q];
                  float& b = gv[8 * j + 2 * q + 1];
                  // keeps the compiler from splitting all values ahead of the stores, into spills
                  asm volatile("" : "+f"(a), "+f"(b));
                  w[q] = GP == kOne ? pack_bf16_rn(a, b) : pack_bf16_hi(peel(a), peel(b));
                }
                st_shared_v4(stg_row + (((uint32_t)j << 4) ^ swz), w[0], w[1], w[2], w[3]);
              }
              fence_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_3d(&P.g_out, stg, col0 + c0, row0, p);
                bulk_commit();
              }
              next_buffer();
            }
          }
        }
      } else if (T.kind == 2) {
        // lane = column of d, column = row: a row's 32 values leave as 128 bytes
        const int dcol = T.row + CM * (int)rank + quarter * 32 + lane;
        float* o = P.dx_part + ((int64_t)T.split * P.m_pad + col0) * P.d + dcol;
#pragma unroll
        for (int c0 = 0; c0 < BN / 2; c0 += 32) {
          if (c0 >= nh || col0 + c0 >= live) break;
          float own[FLUSH ? 1 : 32];
          float* v = FLUSH ? sum + (FLUSH ? c0 : 0) : own;
          if (!FLUSH) cols32(c0, v);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (dcol < P.d && col0 + c0 + e < live) {
              float* at = o + (int64_t)(c0 + e) * P.d;
              *at = P.dx_add ? *at + v[e] : v[e];
            }
        }
      } else {
        const int rows = T.kind ? (int)P.m_pad : P.vn;
        const bool f32 = T.kind || P.dt_f32;
        const CUtensorMap* map = T.kind ? &P.dx_out : &P.dt_out;
        const int out_row = T.kind ? row0 : P.dt_row0 + row0;
        // a value of dx gets one addition per piece, and the pieces are launches in order: the sum is too
        const bool add = T.kind && P.dx_add;
#pragma unroll
        for (int c0 = 0; c0 < BN / 2; c0 += 32) {
          if (row0 >= rows || col0 + c0 >= P.d) continue;
          float own[FLUSH ? 1 : 32];
          float* v = FLUSH ? sum + (FLUSH ? c0 : 0) : own;
          if (!FLUSH) cols32(c0, v);
          if (FLUSH) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= unit;
          }
          const int h = f32 ? 0 : (c0 >> 5) & 1;  // bf16: two groups of 32 columns fill a 128-byte row
          if (h == 0) {
            if (lane == 0) bulk_wait_read<OUT_BUFS - 1>();
            __syncwarp();
          }
          if (f32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              st_shared_v4(stg_row + (((uint32_t)j << 4) ^ swz), __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                           __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) w[q] = pack_bf16_rn(v[8 * j + 2 * q], v[8 * j + 2 * q + 1]);
              st_shared_v4(stg_row + (((uint32_t)(4 * h + j) << 4) ^ swz), w[0], w[1], w[2], w[3]);
            }
          }
          if (f32 || h == 1 || col0 + c0 + 32 >= P.d) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (add) tma_add_3d(map, stg, col0 + c0, out_row, T.split);
              else tma_store_3d(map, stg, col0 + c0 - 32 * h, out_row, T.split);
              bulk_commit();
            }
            next_buffer();
          }
        }
      }
      if (!FLUSH) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(in_first_cta(&accempty[(n - 1u) & 1u]));
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // neither CTA ends, or frees tensor memory, while the other one's MMAs, copies or arrivals can reach it
  if (rank == 1 && threadIdx.x == 0) mbar_wait_drain(drain, 0u);
  __syncthreads();
  cluster_sync();
  if ((issued[0] | issued[1]) & kGaveUp) {  // both CTAs see the same
    // The producers may have stopped at different iterations. Each issues what only the other one did, so
    // that every stage's barrier has both CTAs' bytes to come, and the first CTA waits for all of them.
    if (threadIdx.x == 0) {
      const PairExit e = pair_exit(issued[rank] & ~kGaveUp, issued[rank ^ 1u] & ~kGaveUp, STAGES);
      uint32_t it = 0;
      for (int t = first; it < e.to && t < tiles; t += stride) {
        const Tile T = tile_at<MODE>(P, G, t);
        const Prods& pr = MODE != kProducts ? P.fwd : T.kind ? P.dxp : P.dtp;
        for (int p = 0; p < T.nprod; ++p)
          for (int kb = 0; kb < T.nkb; ++kb, ++it)
            if (it >= e.from && it < e.to) fill(T, pr.a[p], pr.b[p], kb, it);
      }
      if (rank == 0)
        for (uint32_t j = e.drain; j < e.to; ++j) mbar_wait_drain(&full[j % STAGES], (j / STAGES) & 1u);
    }
    __syncthreads();
    cluster_sync();
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------------------------
// rows: which are live, gathered together
// ---------------------------------------------------------------------------------------------
struct Rows {
  const int32_t* targets;  // cross entropy: a row is live when its target is in [0, vocab)
  const uint8_t* flags;    // distillation: live flags of teacher_rows_kernel
  int32_t vocab;
  int32_t m;
};
__device__ __forceinline__ bool row_live(const Rows& R, int r) {
  return R.targets ? (uint32_t)R.targets[r] < (uint32_t)R.vocab : R.flags[r] != 0;
}

constexpr int kScanThreads = 1024;

// rowmap[i] = the i-th live row in order, *live = their number. One CTA: 4096 rows a turn, ballots
// inside a warp and a scan over the 32 warps' counts.
__global__ void __launch_bounds__(kScanThreads) live_rows_kernel(const Rows R, int32_t* __restrict__ rowmap,
                                                                 int32_t* __restrict__ live) {
  dependent();
  __shared__ int32_t count[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int base = 0, turn = 0;
  for (int r0 = 0; r0 < R.m; r0 += 4 * kScanThreads, turn ^= 1) {
    uint32_t mask[4];
    int mine = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t r = (int64_t)r0 + warp * 128 + u * 32 + lane;
      mask[u] = __ballot_sync(0xffffffffu, r < R.m && row_live(R, (int)r));
      mine += __popc(mask[u]);
    }
    if (lane == 0) count[turn][warp] = mine;
    __syncthreads();
    int before = lane < warp ? count[turn][lane] : 0, all = count[turn][lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      before += __shfl_xor_sync(0xffffffffu, before, o);
      all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    int at = base + before;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (mask[u] >> lane & 1u) rowmap[at + __popc(mask[u] & ((1u << lane) - 1u))] = r0 + warp * 128 + u * 32 + lane;
      at += __popc(mask[u]);
    }
    base += all;
  }
  if (threadIdx.x == 0) *live = base;
}

struct GatherArgs {
  Rows R;
  const int32_t* rowmap;
  const int32_t* live;
  const void* x;          // [m][d]
  int32_t d;
  int64_t m_pad;
  __nv_bfloat16* xg;      // [planes][m_pad][d], fp16 with a float32 table
  float* x_unit;          // fp16: [m_pad] the power of two to take out again, or nullptr
  float* row_most;        // fp16, backward: [m_pad] largest |c x| of each place
  // backward, per live row (pad rows: 0): c = dloss / tau, lse, target
  const float* dloss;     // [m] or nullptr
  const float* lse_in;    // [m]
  float inv_tau;
  float* c;
  float* lse;
  int32_t* tgt;           // nullptr: no targets
  // rows that are not live: zeros
  void* dx;               // [m][d] in x's dtype, or nullptr
  float* zero1;           // [m] or nullptr
  float* zero2;
};

constexpr int kRowThreads = 256;

__device__ __forceinline__ void store_planes(const GatherArgs& a, int64_t i, int c, const uint32_t (*p)[4], int planes) {
  for (int j = 0; j < planes; ++j)
    reinterpret_cast<uint4*>(a.xg + (j * a.m_pad + i) * a.d)[c] = make_uint4(p[j][0], p[j][1], p[j][2], p[j][3]);
}
template <mmf_dtype XT>
__device__ __forceinline__ void load_row8(const void* x, int64_t at, float (&v)[8]) {
  if (XT == MMF_F32) {
    const float4* s = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + at);
    const float4 u = s[0], w = s[1];
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    v[4] = w.x; v[5] = w.y; v[6] = w.z; v[7] = w.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(x) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float(w[q] << 16);
      v[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
    }
  }
}
// eight values as fp16 planes: two of them, or one (bf16 rows: eight bits fit in eleven)
template <int N>
__device__ __forceinline__ void half_planes(float (&v)[8], uint32_t (&p)[PLANES][4]) {
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) p[j][q] = pack_half(peel_half(v[2 * q]), peel_half(v[2 * q + 1]));
}

// Live row r -> place i (float32 rows as planes; fp16 rows by their own power of two). Whole warp, as
// the next two.
template <mmf_dtype XT>
__device__ __forceinline__ void place_row(const GatherArgs& a, int64_t i, int64_t r, int lane) {
  const int nck = a.d >> 3;
  float v[8];
  uint32_t p[PLANES][4];
  if (a.x_unit) {
    float most = 0.0f;
    for (int c = lane; c < nck; c += 32) {
      load_row8<XT>(a.x, r * a.d + 8 * c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, finite_abs(v[e]));
    }
    most = warp_max(most);
    const float up = unit_up(most);
    for (int c = lane; c < nck; c += 32) {
      load_row8<XT>(a.x, r * a.d + 8 * c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= up;
      half_planes<XT == MMF_F32 ? 2 : 1>(v, p);
      store_planes(a, i, c, p, XT == MMF_F32 ? 2 : 1);
    }
    if (lane == 0) {
      a.x_unit[i] = 1.0f / up;
      if (a.row_most) a.row_most[i] = finite_abs(most * (a.dloss[r] * a.inv_tau));
    }
  } else {
    for (int c = lane; c < nck; c += 32) {
      if (XT == MMF_BF16) {
        reinterpret_cast<uint4*>(a.xg + i * a.d)[c] =
            reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.x) + r * a.d)[c];
        continue;
      }
      load_row8<XT>(a.x, r * a.d + 8 * c, v);
#pragma unroll
      for (int j = 0; j < PLANES; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) p[j][q] = pack_bf16_hi(peel(v[2 * q]), peel(v[2 * q + 1]));
      store_planes(a, i, c, p, PLANES);
    }
  }
  if (lane == 0 && a.c) {
    a.c[i] = a.dloss[r] * a.inv_tau;
    a.lse[i] = a.lse_in[r];
  }
  if (lane == 0 && a.tgt) a.tgt[i] = a.R.targets[r];
}
// zeros in a place past the live rows
template <mmf_dtype XT>
__device__ __forceinline__ void zero_place(const GatherArgs& a, int64_t i, int lane) {
  for (int j = 0; j < (XT == MMF_F32 ? (a.x_unit ? 2 : PLANES) : 1); ++j)
    for (int c = lane; c < a.d >> 3; c += 32)
      reinterpret_cast<uint4*>(a.xg + (j * a.m_pad + i) * a.d)[c] = make_uint4(0u, 0u, 0u, 0u);
  if (lane == 0 && a.c) a.c[i] = a.lse[i] = 0.0f;
  if (lane == 0 && a.row_most) a.row_most[i] = 0.0f;
  if (lane == 0 && a.tgt) a.tgt[i] = -1;
}
// zeros in the outputs of a row that is not live
template <mmf_dtype XT>
__device__ __forceinline__ void zero_outputs(const GatherArgs& a, int64_t r, int lane) {
  if (a.dx) {
    const int n16 = (a.d >> 3) * (XT == MMF_F32 ? 2 : 1);
    for (int c = lane; c < n16; c += 32) reinterpret_cast<uint4*>(a.dx)[r * n16 + c] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (lane == 0 && a.zero1) a.zero1[r] = 0.0f;
  if (lane == 0 && a.zero2) a.zero2[r] = 0.0f;
}

// One warp per row i: fills place i from live row rowmap[i], or with zeros up to the next multiple of
// 256 past the live rows, and zeroes the outputs of row i when it is not live itself.
template <mmf_dtype XT>
__global__ void __launch_bounds__(kRowThreads) gather_rows_kernel(const GatherArgs a) {
  dependent();
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int live = *a.live;
  if (i < live) place_row<XT>(a, i, a.rowmap[i], lane);
  else if (i < (((int64_t)live + 255) & ~(int64_t)255)) zero_place<XT>(a, i, lane);
  if (i < a.R.m && !row_live(a.R, (int)i)) zero_outputs<XT>(a, i, lane);
}

// live_rows_kernel and gather_rows_kernel in one launch, for few rows: every CTA counts the live rows
// before its own eight (m / 256 flags a thread, out of the L2), a live row goes to the place that gives
// it, and the rows that are not live and those past m fill the places behind with zeros. Below
// kOneLaunchRows this is 2.5 us less than the two launches; the counting grows with m^2.
constexpr int kOneLaunchRows = 4096;
template <mmf_dtype XT>
__global__ void __launch_bounds__(kRowThreads) place_rows_kernel(const GatherArgs a, int32_t* __restrict__ rowmap,
                                                                 int32_t* __restrict__ live_out) {
  dependent();
  __shared__ int32_t counts[2][kRowThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r0 = blockIdx.x * (kRowThreads / 32);
  int before = 0, total = 0;
  for (int r = threadIdx.x; r < a.R.m; r += kRowThreads) {
    const int is = row_live(a.R, r) ? 1 : 0;
    total += is;
    if (r < r0) before += is;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) {
    counts[0][warp] = before;
    counts[1][warp] = total;
  }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int w = 0; w < kRowThreads / 32; ++w) {
    before += counts[0][w];
    total += counts[1][w];
  }
  const uint32_t mine = __ballot_sync(0xffffffffu, lane < kRowThreads / 32 && r0 + lane < a.R.m && row_live(a.R, r0 + lane));
  const int64_t r = r0 + warp;
  before += __popc(mine & ((1u << warp) - 1u));
  if (mine >> warp & 1u) {
    if (lane == 0) rowmap[before] = (int32_t)r;
    place_row<XT>(a, before, r, lane);
  } else {
    const int64_t i = total + (r - before);
    if (i < (((int64_t)total + 255) & ~(int64_t)255)) zero_place<XT>(a, i, lane);
    if (r < a.R.m) zero_outputs<XT>(a, r, lane);
  }
  if (r0 == 0 && threadIdx.x == 0) *live_out = total;
}

constexpr int kMostParts = 592;  // four CTAs per SM

__device__ __forceinline__ float reduce_most(float v, float* red) {  // red: 32 floats; all threads get the result
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = threadIdx.x < kRowThreads / 32 ? red[threadIdx.x] : 0.0f;
  if (threadIdx.x < 32) {
    v = warp_max(v);
    if (threadIdx.x == 0) red[0] = v;
  }
  __syncthreads();
  return red[0];
}

// Largest finite magnitude of a float32 table, one value per CTA.
__global__ void __launch_bounds__(kRowThreads) table_most_kernel(const float* __restrict__ t, int64_t count,
                                                                 float* __restrict__ parts) {
  __shared__ float red[32];
  dependent();
  const int64_t n4 = count >> 2;
  float most = 0.0f;
  for (int64_t e = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; e < n4; e += (int64_t)gridDim.x * kRowThreads) {
    const float4 u = reinterpret_cast<const float4*>(t)[e];
    most = fmaxf(most, fmaxf(fmaxf(finite_abs(u.x), finite_abs(u.y)), fmaxf(finite_abs(u.z), finite_abs(u.w))));
  }
  most = reduce_most(most, red);
  if (threadIdx.x == 0) parts[blockIdx.x] = most;
}

// float32 table -> two fp16 planes [2][count] and the power of two to take out again, 8 values a thread.
__global__ void __launch_bounds__(kRowThreads) split_table_kernel(const float* __restrict__ t, int64_t count,
                                                                  const float* __restrict__ parts, int nparts,
                                                                  __nv_bfloat16* __restrict__ out,
                                                                  float* __restrict__ unit) {
  __shared__ float red[32];
  dependent();
  float most = 0.0f;
  for (int i = threadIdx.x; i < nparts; i += kRowThreads) most = fmaxf(most, parts[i]);
  const float up = unit_up(reduce_most(most, red));
  if (blockIdx.x == 0 && threadIdx.x == 0) *unit = 1.0f / up;
  const int64_t n8 = count >> 3;
  for (int64_t e = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; e < n8; e += (int64_t)gridDim.x * kRowThreads) {
    float v[8];
    uint32_t p[PLANES][4];
    load_row8<MMF_F32>(t, 8 * e, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= up;
    half_planes<2>(v, p);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      reinterpret_cast<uint4*>(out + j * count)[e] = make_uint4(p[j][0], p[j][1], p[j][2], p[j][3]);
  }
}

// float32 table -> two fp16 planes [2][rows][d], every row by its own power of two (unit[row] to take it
// out again): the forward's, whose epilogue has a word per column; one pass over the table where a common
// power takes two (the backward's, in which words are summed over). One warp per row.
__global__ void __launch_bounds__(kRowThreads) split_rows_kernel(const float* __restrict__ t, int rows, int d,
                                                                 __nv_bfloat16* __restrict__ out,
                                                                 float* __restrict__ unit) {
  dependent();
  const int lane = threadIdx.x & 31, nck = d >> 3;
  const int64_t count = (int64_t)rows * d;
  for (int64_t r = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); r < rows;
       r += (int64_t)gridDim.x * (kRowThreads / 32)) {
    float most = 0.0f, v[8];
    for (int c = lane; c < nck; c += 32) {
      load_row8<MMF_F32>(t, r * d + 8 * c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, finite_abs(v[e]));
    }
    const float up = unit_up(warp_max(most));
    if (lane == 0) unit[r] = 1.0f / up;
    for (int c = lane; c < nck; c += 32) {
      uint32_t p[PLANES][4];
      load_row8<MMF_F32>(t, r * d + 8 * c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= up;
      half_planes<2>(v, p);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        reinterpret_cast<uint4*>(out + j * count + r * d)[c] = make_uint4(p[j][0], p[j][1], p[j][2], p[j][3]);
    }
  }
}

// c x of the live rows as fp16 planes under one power of two, the rows' side of dT with a float32
// table; zeros in the places up to the next multiple of 256. One warp per place; every CTA takes the
// largest |c x| over the places from row_most.
template <mmf_dtype XT>
__global__ void __launch_bounds__(kRowThreads) weigh_rows_kernel(const GatherArgs a, __nv_bfloat16* __restrict__ out,
                                                                 float* __restrict__ unit) {
  __shared__ float red[32];
  dependent();
  const int live = *a.live, lane = threadIdx.x & 31, nck = a.d >> 3;
  const int64_t places = ((int64_t)live + 255) & ~(int64_t)255;
  if ((int64_t)blockIdx.x * (kRowThreads / 32) >= places && blockIdx.x > 0) return;  // uniform
  float most = 0.0f;
  for (int i = threadIdx.x; i < live; i += kRowThreads) most = fmaxf(most, a.row_most[i]);
  const float up = unit_up(reduce_most(most, red));
  if (blockIdx.x == 0 && threadIdx.x == 0) *unit = 1.0f / up;
  for (int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); i < places;
       i += (int64_t)gridDim.x * (kRowThreads / 32)) {
    const float c = i < live ? a.c[i] : 0.0f;
    const int64_t r = i < live ? a.rowmap[i] : 0;
    for (int k = lane; k < nck; k += 32) {
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      uint32_t p[PLANES][4];
      if (i < live) load_row8<XT>(a.x, r * a.d + 8 * k, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * c * up;
      half_planes<2>(v, p);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        reinterpret_cast<uint4*>(out + (j * a.m_pad + i) * a.d)[k] = make_uint4(p[j][0], p[j][1], p[j][2], p[j][3]);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// joining the tiles' statistics
// ---------------------------------------------------------------------------------------------
// lse_i = top / tau + log sum_j S_j exp((M_j - top) / tau) over the row's parts, and for the cross
// entropy loss_i = lse_i - s_target / tau. Without live_p and rowmap every row of R is there, and those
// that are not live get zeros. CTA = 32 rows x 32 lanes over the parts, four parts in flight
// per lane (a lane's chain over 250 / 32 parts is what the call costs when there are few rows).
constexpr int kJoinThreads = 1024;
__global__ void __launch_bounds__(kJoinThreads) join_stats_kernel(const float2* __restrict__ part, int parts,
                                                                  int64_t m_pad, const int32_t* __restrict__ live_p,
                                                                  const int32_t* __restrict__ rowmap, const Rows R,
                                                                  const float* __restrict__ st, float inv_tau,
                                                                  float* loss, float* lse_out) {
  dependent();
  __shared__ float2 red[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int live = live_p ? *live_p : R.m;
  const int64_t i = (int64_t)blockIdx.x * 32 + tx;
  if ((int64_t)blockIdx.x * 32 >= live) return;
  float mx = -INFINITY, sum = 0.0f;
  if (i < live) {
    for (int j0 = ty; j0 < parts; j0 += 128) {
      float2 p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        p[u] = j0 + 32 * u < parts ? part[(int64_t)(j0 + 32 * u) * m_pad + i] : make_float2(-INFINITY, 0.0f);
      const float top = fmaxf(fmaxf(mx, fmaxf(p[0].x, p[1].x)), fmaxf(p[2].x, p[3].x));
      const float ref = top == -INFINITY ? 0.0f : top;
      sum *= expf((mx - ref) * inv_tau);
#pragma unroll
      for (int u = 0; u < 4; ++u) sum += p[u].y * expf((p[u].x - ref) * inv_tau);
      mx = top;
    }
  }
  red[ty][tx] = make_float2(mx, sum);
  __syncthreads();
  // warp ty joins row ty's 32 lanes
  const float2 p = red[tx][ty];
  const float top = warp_max(p.x);
  const float ref = top == -INFINITY ? 0.0f : top;
  const float s = warp_sum(p.y * expf((p.x - ref) * inv_tau));
  const int64_t row = (int64_t)blockIdx.x * 32 + ty;
  if (tx == 0 && row < live) {
    const bool is = rowmap || row_live(R, (int)row);
    const float l = is ? top * inv_tau + logf(s) : 0.0f;
    const int64_t r = rowmap ? rowmap[row] : row;
    lse_out[r] = l;
    if (st || !is) loss[r] = is ? l - st[row] * inv_tau : 0.0f;
  }
}

// out[row(i)][:] = sum over planes of part[p][i][:], in plane order; rows i < *count (or count_h),
// written to rowmap[i] when given, times c_p[i] and dx's fp16 units when given. 8 columns a thread.
template <mmf_dtype OT>
__global__ void __launch_bounds__(kRowThreads) join_planes_kernel(const float* __restrict__ part, int planes,
                                                                  int64_t plane_rows, int d,
                                                                  const int32_t* __restrict__ count_p, int64_t count_h,
                                                                  const int32_t* __restrict__ rowmap,
                                                                  const float* __restrict__ c_p,
                                                                  const float* __restrict__ unit, void* out) {
  dependent();
  const int nck = d >> 3;
  const int64_t rows = count_p ? *count_p : count_h;
  const int64_t total = rows * nck;
  for (int64_t e = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; e < total; e += (int64_t)gridDim.x * kRowThreads) {
    const int64_t i = e / nck;
    const int c = (int)(e - i * nck);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int p = 0; p < planes; ++p) {
      const float4* s = reinterpret_cast<const float4*>(part + (p * plane_rows + i) * d) + 2 * c;
      const float4 u = s[0], w = s[1];
      v[0] += u.x; v[1] += u.y; v[2] += u.z; v[3] += u.w;
      v[4] += w.x; v[5] += w.y; v[6] += w.z; v[7] += w.w;
    }
    const int64_t r = rowmap ? rowmap[i] : i;
    if (c_p) {
      // in 64 bits: the unit and c may leave float32's range one after the other, in either order
      const double u = (double)*unit * (1.0f / kGradUnit) * c_p[i];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (float)(v[e] * u);
    }
    if (OT == MMF_F32) {
      float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + r * d) + 2 * c;
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(out) + r * d)[c] =
          make_uint4(pack_bf16_rn(v[0], v[1]), pack_bf16_rn(v[2], v[3]), pack_bf16_rn(v[4], v[5]), pack_bf16_rn(v[6], v[7]));
    }
  }
}

// ---------------------------------------------------------------------------------------------
// the teacher's entries
// ---------------------------------------------------------------------------------------------
struct Teacher {
  const int32_t* ids;   // [m][k]
  const void* logits;   // [m][k]
  mmf_dtype dt;
  int32_t k;
  int32_t vocab;
  float inv_tau;
};
__device__ __forceinline__ bool teacher_valid(const Teacher& t, int64_t at, float& logit) {
  logit = load_as_float(t.logits, at, t.dt);
  return (uint32_t)t.ids[at] < (uint32_t)t.vocab && !(logit == -INFINITY);
}

// The row's teacher distribution over its valid entries: top = the largest valid logit, total = sum
// exp((t_j - top) / tau). Whole warp; the differences are taken before the division by tau, so that
// logits near the type's lowest value stay finite.
__device__ __forceinline__ void teacher_softmax(const Teacher& t, int64_t r, int lane, float& top, float& total) {
  top = -INFINITY;
  bool nan = false;
  for (int j = lane; j < t.k; j += 32) {
    float l;
    if (teacher_valid(t, r * t.k + j, l)) {
      nan |= l != l;
      top = fmaxf(top, l);
    }
  }
  top = warp_max(top);
  if (__any_sync(0xffffffffu, nan)) top = __int_as_float(0x7fc00000);
  total = 0.0f;
  for (int j = lane; j < t.k; j += 32) {
    float l;
    if (teacher_valid(t, r * t.k + j, l)) total += expf((l - top) * t.inv_tau);
  }
  total = warp_sum(total);
}

constexpr int kTeacherRows = 16;      // rows per CTA, one warp each
constexpr int kTeacherTiles = 128;    // tile halves per turn
// Per row: its live flag (it has a valid entry), and its entries in order of their ids (equal ids in
// order of the entries), entries that are not valid last with id 2^31 - 1. The place of an entry is the
// number of entries before it, counted over the row in shared memory, four at a time.
//   start (forward): start[h][r] = valid entries with an id below 128 h, so that the tile half at
//     columns 128 h finds its own without a search, and zeros in s_top at entries that are not valid;
//   q (backward): the teacher's weight of every entry, in the same order.
__global__ void __launch_bounds__(kTeacherRows * 32, 3) teacher_rows_kernel(const Teacher t, int64_t m, int64_t m_pad,
                                                                            int halves, uint8_t* __restrict__ flags,
                                                                            int2* __restrict__ top,
                                                                            uint16_t* __restrict__ start,
                                                                            float* __restrict__ s_top,
                                                                            float* __restrict__ q) {
  __shared__ __align__(16) int32_t ids[kTeacherRows][MAX_TOP];
  __shared__ int32_t sorted[kTeacherRows][MAX_TOP];
  __shared__ uint16_t turn[kTeacherTiles][kTeacherRows + 1];
  dependent();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r0 = (int64_t)blockIdx.x * kTeacherRows, r = r0 + warp;
  constexpr int32_t kNone = 0x7fffffff;
  int count = 0;  // valid entries
  if (r < m) {
    for (int j = lane; j < ((t.k + 31) & ~31); j += 32) {
      float l;
      int32_t id = kNone;  // past the row's entries too: counted by nobody
      if (j < t.k) {
        const int32_t given = t.ids[r * t.k + j];
        if (teacher_valid(t, r * t.k + j, l)) id = given;
        else if (s_top) s_top[r * t.k + j] = 0.0f;
      }
      ids[warp][j] = id;
      count += __popc(__ballot_sync(0xffffffffu, id != kNone));
    }
    if (lane == 0) flags[r] = count > 0 ? 1 : 0;
    float best = 0.0f, total = 1.0f;
    if (q) teacher_softmax(t, r, lane, best, total);
    __syncwarp();
    for (int j = lane; j < t.k; j += 32) {
      const int32_t id = ids[warp][j];
      int place = 0;
      for (int i = 0; i < t.k; i += 4) {
        const int4 o = *reinterpret_cast<const int4*>(&ids[warp][i]);
        place += (o.x < id || (o.x == id && i < j)) + (o.y < id || (o.y == id && i + 1 < j)) +
                 (o.z < id || (o.z == id && i + 2 < j)) + (o.w < id || (o.w == id && i + 3 < j));
      }
      sorted[warp][place] = id;
      top[r * t.k + place] = make_int2(id, j);
      if (q)
        q[r * t.k + place] = id != kNone ? expf((load_as_float(t.logits, r * t.k + j, t.dt) - best) * t.inv_tau) / total : 0.0f;
    }
  }
  if (!start) return;  // uniform
  __syncwarp();
  // the first entry of half h is the first one whose own half is h or later: entry p is it for the
  // halves past entry p - 1's up to its own, and the end of the row for those past the last entry's
  for (int h0 = 0; h0 < halves; h0 += kTeacherTiles) {
    for (int p = lane; p <= count; p += 32) {
      const int from = p == 0 ? h0 : max(sorted[warp][p - 1] / (BN / 2) + 1, h0);
      const int to = min(p == count ? h0 + kTeacherTiles - 1 : sorted[warp][p] / (BN / 2), h0 + kTeacherTiles - 1);
      for (int h = from; h <= to; ++h) turn[h - h0][warp] = (uint16_t)p;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kTeacherTiles * kTeacherRows; e += kTeacherRows * 32) {
      const int h = e / kTeacherRows, i = e % kTeacherRows;
      if (h0 + h < halves && r0 + i < m_pad) start[(int64_t)(h0 + h) * m_pad + r0 + i] = turn[h][i];
    }
    __syncthreads();
  }
}

// loss = sum_j q_j (log q_j - s_j / tau + lse) of the live rows. One warp per row.
__global__ void __launch_bounds__(kRowThreads) distill_loss_kernel(const Teacher t, int64_t m,
                                                                   const uint8_t* __restrict__ flags,
                                                                   const float* __restrict__ lse,
                                                                   const float* __restrict__ s_top, float* loss) {
  dependent();
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (r >= m || !flags[r]) return;  // the gather has zeroed the row's loss
  float top, total, sum = 0.0f;
  teacher_softmax(t, r, lane, top, total);
  const float log_total = logf(total), L = lse[r];
  for (int j = lane; j < t.k; j += 32) {
    float l;
    if (teacher_valid(t, r * t.k + j, l)) {
      const float e = (l - top) * t.inv_tau, q = expf(e) / total;
      // an entry whose q underflows adds nothing (0 log 0 = 0); NaN goes through
      if (!(q == 0.0f)) sum += q * ((e - log_total) - (s_top[r * t.k + j] * t.inv_tau - L));
    }
  }
  sum = warp_sum(sum);
  if (lane == 0) loss[r] = sum;
}

// The teacher's share of g for the piece [v0, v0 + vn): for every entry of live row i with its id in
// the piece, g[i][id] = c (exp(s_j / tau - lse) - sum of q over the row's entries with that id),
// computed whole in float32 from the kept s_j and stored over the softmax part (so nothing is rounded
// twice). One warp per row; the first entry of a run of equal ids writes.
__global__ void __launch_bounds__(kRowThreads) teacher_grad_kernel(const int2* __restrict__ top,
                                                                   const float* __restrict__ q, int k, float inv_tau,
                                                                   const int32_t* __restrict__ live_p,
                                                                   const int32_t* __restrict__ rowmap,
                                                                   const float* __restrict__ s_top,
                                                                   const float* __restrict__ c_p,
                                                                   const float* __restrict__ lse_p, int v0, int vn,
                                                                   __nv_bfloat16* g, int64_t m_pad, int64_t ldg,
                                                                   int gp) {
  dependent();
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (i >= *live_p) return;
  const int64_t base = (int64_t)rowmap[i] * k;
  const float c = c_p[i], L = lse_p[i];
  for (int p = lane; p < k; p += 32) {
    const int2 e = top[base + p];
    if (e.x < v0 || e.x >= v0 + vn || (p > 0 && top[base + p - 1].x == e.x)) continue;
    float w = q[base + p];
    for (int n = p + 1; n < k && top[base + n].x == e.x; ++n) w += q[base + n];
    float v = expf(s_top[base + e.y] * inv_tau - L) - w;
    __nv_bfloat16* o = g + i * ldg + (e.x - v0);
    if (gp == kHalf2) {  // without c
      v *= kGradUnit;
      for (int pl = 0; pl < 2; ++pl)
        *reinterpret_cast<__half*>(o + pl * m_pad * ldg) = __float2half_rn(peel_half(v));
      continue;
    }
    v *= c;
    if (gp == kOne) {
      *o = __float2bfloat16_rn(v);
    } else if (gp == kFine2) {
      float none = 0.0f;
      const uint32_t hi = peel_bf16_rn(v, none);
      *reinterpret_cast<uint16_t*>(o) = (uint16_t)hi;
      o[m_pad * ldg] = __float2bfloat16_rn(v);
    } else
      for (int pl = 0; pl < PLANES; ++pl) o[pl * m_pad * ldg] = __float2bfloat16_rn(peel(v));
  }
}

}  // namespace hl
}  // namespace mmf

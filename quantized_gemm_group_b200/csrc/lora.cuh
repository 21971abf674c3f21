// lora.cuh -- low-rank adapters beside a shared projection: for each row m of
// a segment with adapter a (rank r_a <= R, scale s_a)
//   forward         t = drop(x) A^T          y  = base + s (t B^T)
//   input gradient  dt = s (dy B)            dx = base + drop'(dt A)
// Both directions are one shape of work, "down" to the rank and "up" again,
// so one kernel does both (UP = 0 forward, 1 gradient); they differ in which
// pool comes first and in how its elements lie: A is [L, R, K] (contiguous
// along the contraction of the forward's down step), B is [L, N, R].
//
// This file's kernel takes short segments (up to 24 rows each on average),
// where the pools are most of the traffic; lora_tc.cuh takes longer ones.
// Bound: memory and, below 16 rows, the latency of the chain x -> t -> y.
// On mma.sync a warp works on its own and starts with the first bytes; 16 rows
// would leave 112 of the 128 rows of a tensor memory tile empty.
//
// Split: a cluster of CS CTAs owns 16 rows of one segment.  Each CTA contracts
// its share of the columns (down), the partial [16, R] sums meet in distributed
// shared memory (added in rank order: no atomics, the same bits every time),
// and each CTA then writes its share of the output columns (up).  t never goes
// through global memory (the training forward stores it once for the backward
// pass), and one launch does the whole adapter.  The grid has one cluster for
// each tile that S segments of M rows can need; a cluster finds its segment by
// a prefix sum over the segment lengths, so lengths stay on the device.
//
// Down: a warp takes every eighth run of 32 columns.  A lane's 16-byte load of
// a row (8 consecutive columns) is used as the fragments of two k-steps: the
// contraction may run in any order as long as both operands use the same one,
// so x needs no shared memory and dropout is applied to the loaded registers,
// one generator block a load.  The pool goes through a cp.async ring.
// Up: t (fp32) is split into two 16-bit parts t = hi + lo, two mma.sync a step:
// bf16 within 2^-16 (one bf16 would lose 2^-9 of t), fp16 within 2^-21 and 2^-38 of the
// row's largest, which a power of two brings into fp16's range first.  A warp takes
// 32 output columns of the tile; the column that fragment slot n of tile j stands for is 8 (n / 2) + 2 j + n % 2,
// so that a lane ends with 8 consecutive columns: base and y move as 16-byte
// vectors.
//
// Measured (bf16, each request its own adapter, 4096 columns in): 1 token to
// 4096 columns, rank 16 5.5 us; 16 requests to 28672, rank 16 14 us and to
// 14336, rank 64 17 us; 128 requests to 4096, rank 64 29 us (134 MB of pools:
// 71 % of the copy rate); 256 requests to 14336, rank 64 (64 adapters) 90 us.
// Few requests are bound by the chain of waits and by the warps' instructions
// (16 requests: one issued every 2.7 cycles by two warps a scheduler; sixteen
// warps a CTA were slower, as clusters of 8 then find 15 places instead of 33).
#pragma once
#include <cooperative_groups.h>

#include "common.cuh"
#include "dropout.cuh"
#include "gemv.cuh"

namespace bq {
namespace cg = cooperative_groups;

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraRows = 16;  // rows per tile
// Steps down (of two products each) that a CTA lets add up in the tensor core.  Its
// additions cut where fp32 additions round: 56 steps (14336 columns in one CTA)
// lost 2e-6 of t's norm, plain fp32 products 1e-6, 16 steps lose 0.6e-6.  CTAs with
// more (APART) add each step's products to the sums in fp32.  That costs up to 8 %
// (1536 rows in 64 segments, 14336 -> 4096, rank 16 48 instead of 45 us), so it is a
// kernel of its own.
constexpr int kLoraRun = 16;

struct LoraArgs {
  const uint16_t *x;      // [M, Ci] rows of stride ldx: x, or dy
  const uint16_t *A, *B;  // pools [L, R, K] and [L, N, R]
  const uint16_t *base;   // [M, Co] added to the output, or NULL
  uint16_t *y;            // [M, Co]; may be base
  float *t;               // [M, R] or NULL: t (UP = 0), dt (UP = 1)
  const int *ranks;
  const float *scales;
  const int *seg_off, *seg_adapter;
  int64_t M, ldx, ldbase, ldy;
  int Ci, Co, R, L, S, CS;
  int slice_c, slice_o;  // columns of the contraction / of the output per CTA
  DropArgs drop;
};

// One segment tile: rows [row0, row0 + rows), its adapter (-1: none).
struct LoraTile {
  int row0, rows, adapter;
  bool found;
};

// A segment as the kernels use it: its length, 0 where the offsets are unusable.
BQ_DEV int lora_segment(const int *seg_off, int s, int64_t M, int *start) {
  const int a = __ldcg(seg_off + s), b = __ldcg(seg_off + s + 1);
  *start = a;
  return (a >= 0 && b >= a && b <= M) ? b - a : 0;
}

// Tile `tile` of the segments cut into BM rows each.  Every lane of the warp
// takes part; the result is the same in all lanes.
template <int BM>
BQ_DEV LoraTile lora_find_tile(const int *seg_off, const int *seg_adapter, int S, int64_t M, int tile) {
  const int lane = threadIdx.x & 31;
  LoraTile r = {0, 0, -1, false};
  int before = 0;
  for (int s0 = 0; s0 < S; s0 += 32) {
    const int s = s0 + lane;
    int start = 0, len = 0, ad = -1;
    if (s < S) {
      ad = __ldcg(seg_adapter + s);
      len = lora_segment(seg_off, s, M, &start);
    }
    const int n = (len + BM - 1) / BM;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + incl > tile);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int i = tile - before - (__shfl_sync(0xffffffffu, incl, src) - __shfl_sync(0xffffffffu, n, src));
      const int st = __shfl_sync(0xffffffffu, start, src), ln = __shfl_sync(0xffffffffu, len, src);
      r.row0 = st + i * BM;
      r.rows = min(BM, ln - i * BM);
      r.adapter = __shfl_sync(0xffffffffu, ad, src);
      r.found = true;
      return r;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return r;
}

// Descending or overlong segments and unknown adapters or ranks are recorded
// in the device status (one warp of the grid looks at all of them).
BQ_DEV void lora_check_segments(const int *seg_off, const int *seg_adapter, const int *ranks, int S, int L, int R,
                                int64_t M) {
  bool bad = false;
  for (int s = threadIdx.x & 31; s < S; s += 32) {
    const int a = seg_off[s], b = seg_off[s + 1], ad = seg_adapter[s];
    bad |= a < 0 || b < a || b > M || ad < -1 || ad >= L;
    if (ad >= 0 && ad < L) bad |= ranks[ad] < 0 || ranks[ad] > R;
  }
  if (bad) bq_flag(BQ_FLAG_BADMAP);
}

// Rows without a contribution: base's (nothing to do in place), t zero.  The
// cluster's warps take a row each in turn; a lane has eight loads in flight
// while it stores the eight before.
BQ_DEV void lora_copy_load(uint4 (&v)[8], const uint16_t *from, int c, int n) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    v[k] = (from && c + 256 * k < n) ? ld_stream_v4(from + c + 256 * k) : make_uint4(0, 0, 0, 0);
}
BQ_DEV void lora_copy_store(const uint4 (&v)[8], uint16_t *to, int c, int n) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (c + 256 * k < n) st_v4(to + c + 256 * k, v[k]);
}
// (Not inlined, and without the kernel's argument struct: it is rarely run, and
// the struct's address would put a copy of it on every thread's stack.)
__device__ __noinline__ void lora_copy_some(const uint16_t *base, int64_t ldbase, uint16_t *y, int64_t ldy, float *t, int n,
                                            int R, int first, int rows, int step) {
  const int lane = threadIdx.x & 31;
  for (int m = first; m < rows; m += step) {
    if (base != y && n > 0) {
      const uint16_t *from = base ? base + m * ldbase : nullptr;
      uint16_t *to = y + m * ldy;
      uint4 v[8], w[8];
      int c = 8 * lane;
      lora_copy_load(v, from, c, n);
      for (; c < n; c += 2 * 2048) {
        lora_copy_load(w, from, c + 2048, n);
        lora_copy_store(v, to, c, n);
        lora_copy_load(v, from, c + 2 * 2048, n);
        lora_copy_store(w, to, c + 2048, n);
      }
    }
    if (t)
      for (int i = lane; i < R; i += 32) t[(int64_t)m * R + i] = 0.0f;
  }
}
BQ_DEV void lora_copy_rows(const LoraArgs &a, const LoraTile &tile, int rank, int CS, int threads) {
  const int warps = threads >> 5;
  const int64_t row = tile.row0;
  const bool copy = a.base != a.y;
  lora_copy_some(a.base ? a.base + row * a.ldbase : nullptr, a.ldbase, copy ? a.y + row * a.ldy : nullptr, a.ldy,
                 a.t ? a.t + row * a.R : nullptr, copy ? a.Co : 0, a.R, rank * warps + (int)(threadIdx.x >> 5), tile.rows,
                 CS * warps);
}

// The rank to use: 0 (no contribution) without an adapter or with a bad one.
BQ_DEV int lora_rank(const int *ranks, int adapter, int L, int R) {
  if (adapter < 0 || adapter >= L) return 0;
  const int r = __ldcg(ranks + adapter);
  return (r < 0 || r > R) ? 0 : r;
}

BQ_DEV void cp_async16(uint32_t dst, const void *src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
BQ_DEV void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
BQ_DEV void cp_async8(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
BQ_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> BQ_DEV void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

BQ_DEV void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t smem_addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr));
}
BQ_DEV uint2 lds_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
BQ_DEV void sts_u32(uint32_t addr, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory"); }
BQ_DEV void sts_v2f(uint32_t addr, float a, float b) {
  asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}
BQ_DEV uint4 ld_nc_v4(const void *p) {
  uint4 r;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// Two floats as bf16x2 (a in the lower half).
BQ_DEV uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// v = hi + lo in bf16 parts; an infinite or NaN v keeps lo = 0.
BQ_DEV void split_bf16(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16(a, b);
  float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xffff0000u);
  if (!(fabsf(ra) <= 3.402823466e38f)) ra = 0.0f;
  if (!(fabsf(rb) <= 3.402823466e38f)) rb = 0.0f;
  lo = pack_bf16(ra, rb);
}
// Two floats as the hi and lo parts of type XT (fp16: scaled by the caller).
template <int XT> BQ_DEV void tc_split(float a, float b, uint32_t &hi, uint32_t &lo) {
  if (XT == 1) {
    split_bf16(a, b, hi, lo);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    float ra = a - f.x, rb = b - f.y;
    if (!(fabsf(ra) <= 3.402823466e38f)) ra = 0.0f;
    if (!(fabsf(rb) <= 3.402823466e38f)) rb = 0.0f;
    const __half2 l = __floats2half2_rn(ra, rb);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
  }
}
// The parts for a product whose other factor may be infinite: hi is cut, lo = a - hi
// has its sign and is not 0 unless a is, so that both parts times an infinity give
// the same one (with hi rounded, lo of the other sign or 0 would make it NaN).  Off
// by 2^-16 of a (bf16), 2^-21 and 2^-24 (fp16).  Where lo would be 0 it is 2^-24 of hi;
// fp16 has no less than 2^-24, 2^-38 of the row's largest after tc_scale.  Values that
// are too small for that (bf16 below 2^-102, fp16 below 2^-24) keep lo = 0.
BQ_DEV float same_sign_rest(float a, float h, float least) {
  const float r = a - h;  // exact; NaN where a is not finite
  return fabsf(r) > 0.0f ? r : h * least;
}
template <int XT> BQ_DEV void split_same_sign(float a, float b, uint32_t &hi, uint32_t &lo) {
  if (XT == 1) {
    const float ha = isnan(a) ? a : __uint_as_float(__float_as_uint(a) & 0xffff0000u);
    const float hb = isnan(b) ? b : __uint_as_float(__float_as_uint(b) & 0xffff0000u);
    hi = pack_bf16(ha, hb);
    lo = pack_bf16(same_sign_rest(a, ha, 0x1p-24f), same_sign_rest(b, hb, 0x1p-24f));
  } else {
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
    const float2 h = Elem<0>::pair(hi);
    const __half2 l = __floats2half2_rn(same_sign_rest(a, h.x, 1.0f), same_sign_rest(b, h.y, 1.0f));
    lo = *reinterpret_cast<const uint32_t *>(&l);
    // exact values, and rests that round to 0
    if (h.x != 0.0f && (a == h.x || !(lo & 0x7fffu)) && fabsf(a) <= 3.402823466e38f)
      lo = (lo & 0xffff0000u) | (hi & 0x8000u) | 1u;
    if (h.y != 0.0f && (b == h.y || !(lo & 0x7fff0000u)) && fabsf(b) <= 3.402823466e38f)
      lo = (lo & 0x0000ffffu) | (hi & 0x80000000u) | 0x10000u;
  }
}
// 2^e that brings a largest magnitude m into [2^14, 2^15) when divided by it
// (1 where m is 0 or not finite), as the pair (2^e, 2^-e).
BQ_DEV float2 tc_scale(float m) {
  if (!(m > 0.0f) || !(m <= 3.402823466e38f)) return make_float2(1.0f, 1.0f);
  int e = (int)(__float_as_uint(m) >> 23) - 127 - 14;
  e = max(-126, min(e, 126));
  return make_float2(__uint_as_float((uint32_t)(e + 127) << 23), __uint_as_float((uint32_t)(127 - e) << 23));
}
// |v|, 0 where v is not finite (such values do not set a row's power of two).
BQ_DEV float finite_abs(float v) {
  v = fabsf(v);
  return v <= 3.402823466e38f ? v : 0.0f;
}

// Tile geometry for the padded rank RP.  Shared memory holds, one after the
// other, the down ring; the warps' partial sums (from 0); t (from 0), the up
// pool's staging (UP = 1) and the up ring (to MAIN); the owned sums from MAIN.
constexpr int lora_max(int a, int b) { return a > b ? a : b; }
template <int UP, int RP> struct LoraGeom {
  static constexpr int SC = 32 * kLoraWarps;                  // columns per step
  static constexpr int NST = RP == 128 ? 2 : 3;
  static constexpr int STAGE = RP * SC * 2;                   // pool bytes per stage
  static constexpr int PARTIAL = kLoraWarps * kLoraRows * RP * 4;  // the warps' partial sums
  static constexpr int T_BYTES = 2 * kLoraRows * RP * 2;      // t as two bf16 parts
  static constexpr int WT_BYTES = RP * 64;                    // a warp's 32 columns of A (UP = 1)
  // the up ring (UP = 0): a warp's 32 columns of base and B for two turns, stage 0
  // last (four turns: the same within 3 %)
  static constexpr int DU = UP == 1 ? 0 : 2;
  static constexpr int SLOT = UP == 1 ? 0 : kLoraRows * 64 + RP * 64;
  static constexpr int UP_STAGE = kLoraWarps * SLOT;
  static constexpr int LOW = T_BYTES + (UP == 0 ? 0 : kLoraWarps * WT_BYTES);
  static constexpr int MAIN = lora_max(lora_max(NST * STAGE, LOW + DU * UP_STAGE), lora_max(PARTIAL, LOW) + UP_STAGE);
  static constexpr int CLEAR = UP == 1 ? 0 : (MAIN - PARTIAL) / lora_max(UP_STAGE, 1);
  static constexpr int EARLY = CLEAR < DU ? CLEAR : DU;  // stages clear of the sums
  static constexpr int RECV = kLoraRows * RP * 4;
  static constexpr int SCALE = MAIN + RECV;  // fp16: the rows' powers of two
  static constexpr int TOTAL = SCALE + kLoraRows * 4;
};

// Shared-memory byte offset of 16-byte chunk c of row r in a stage of the
// down pool.  UP = 0: row = rank, SC columns; two rows of four chunks are
// read together.  UP = 1: row = contraction index, RP ranks; the eight rows
// 8 i + {0, 1} of one transposed fragment are read together.
template <int UP, int RP, int SC> BQ_DEV uint32_t down_offset(int r, int c) {
  if (UP == 0) return (uint32_t)(r * SC * 2 + ((c ^ ((r & 1) << 2)) << 4));
  const int f = RP >= 64 ? (((r >> 3) & 3) << 1) | (r & 1) : (r >> 3) & 1;
  return (uint32_t)(r * RP * 2 + ((c ^ f) << 4));
}

// grid = CS x tiles, cluster = (CS, 1, 1).
template <int XT, int UP, int RP, bool APART>
__global__ void __launch_bounds__(kLoraThreads, RP == 128 ? 1 : 2)
lora_kernel(LoraArgs a) {
  using G = LoraGeom<UP, RP>;
  constexpr int SC = G::SC, NST = G::NST;
  constexpr int NT = RP / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = a.CS, rank = (int)blockIdx.x % CS, tile_index = (int)blockIdx.x / CS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const uint32_t sbase = smem_u32(smem);

  pdl_wait();
  pdl_launch_dependents();  // everything before this kernel is complete
  if (blockIdx.x == 0 && warp == kLoraWarps - 1)
    lora_check_segments(a.seg_off, a.seg_adapter, a.ranks, a.S, a.L, a.R, a.M);
  const LoraTile tile = lora_find_tile<kLoraRows>(a.seg_off, a.seg_adapter, a.S, a.M, tile_index);
  if (!tile.found) return;  // the whole cluster
  const int r_a = lora_rank(a.ranks, tile.adapter, a.L, a.R);
  const int o_begin = rank * a.slice_o, o_end = min(a.Co, o_begin + a.slice_o);

  if (r_a == 0) {
    lora_copy_rows(a, tile, rank, CS, kLoraThreads);
    return;
  }

  const bool drop = a.drop.thr != 0;
  const DropState dst = drop_state(a.drop);
  const int K = UP ? a.Co : a.Ci, N = UP ? a.Ci : a.Co;
  const uint16_t *poolA = a.A + (int64_t)tile.adapter * a.R * K;  // [R, K]
  const uint16_t *poolB = a.B + (int64_t)tile.adapter * a.R * N;  // [N, R]
  const uint16_t *down = UP ? poolB : poolA;
  const int nt_used = (r_a + 7) / 8;
  const int c_begin = rank * a.slice_c, c_end = min(a.Ci, c_begin + a.slice_c);
  // every CTA has started before any writes into its shared memory
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  // ---- down: partial sums of this warp's rows over its columns -------------
  const int steps = (c_end > c_begin) ? (c_end - c_begin + SC - 1) / SC : 0;
  const uint16_t *xrow[2];
  bool xval[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int m = h * 8 + g;
    xval[h] = m < tile.rows;
    xrow[h] = a.x + (int64_t)(tile.row0 + (xval[h] ? m : 0)) * a.ldx;
  }
  const int lane_c = 32 * warp + 8 * t4;
  auto load_x = [&](uint4 (&v)[2], int step) {
    const int c = c_begin + step * SC + lane_c;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      v[h] = (step < steps && c < c_end && xval[h]) ? ld_stream_v4(xrow[h] + c) : make_uint4(0, 0, 0, 0);
  };
  auto load_pool = [&](int step) {
    if (step < steps) {
      const uint32_t stage = sbase + (step % NST) * G::STAGE;
      const int c0 = c_begin + step * SC;
      if (UP == 0) {
        constexpr int CH = SC / 8;
        for (int i = threadIdx.x; i < r_a * CH; i += kLoraThreads) {
          const int r = i / CH, c = i % CH;
          const bool ok = c0 + 8 * c < c_end;
          cp_async16(stage + down_offset<UP, RP, SC>(r, c), down + (int64_t)r * K + (ok ? c0 + 8 * c : 0), ok);
        }
      } else {
        for (int i = threadIdx.x; i < nt_used * SC; i += kLoraThreads) {
          const int r = i / nt_used, c = i - r * nt_used;
          const bool ok = c0 + r < c_end;
          cp_async16(stage + down_offset<UP, RP, SC>(r, c), down + (int64_t)(ok ? c0 + r : 0) * a.R + 8 * c, ok);
        }
      }
    }
    cp_async_commit();
  };

  float acc[NT][4];
  auto add4 = [](float (&s)[4], const float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] += v[i];
  };
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;

  uint4 xv[2][2];
  load_x(xv[0], 0);
#pragma unroll
  for (int s = 0; s < NST - 1; ++s) load_pool(s);
  auto run_step = [&](uint4 (&cur)[2], uint4 (&nxt)[2], int step) {
    load_x(nxt, step + 1);
    cp_async_wait<NST - 2>();
    __syncthreads();  // the stage is visible, and the one read last step is free
    load_pool(step + NST - 1);
    if (UP == 0 && drop) {
      const int c = c_begin + step * SC + lane_c;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 k = drop_mask8(drop_block(dst, (uint32_t)c >> 3, (uint32_t)(tile.row0 + h * 8 + g)), dst.thr_hi);
        cur[h].x &= k.x;
        cur[h].y &= k.y;
        cur[h].z &= k.z;
        cur[h].w &= k.w;
      }
    }
    const uint32_t stage = sbase + (step % NST) * G::STAGE;
    const uint32_t fa[2][4] = {{cur[0].x, cur[1].x, cur[0].y, cur[1].y}, {cur[0].z, cur[1].z, cur[0].w, cur[1].w}};
    if (UP == 0 && APART) {
      // four tiles at a time, so that their products do not wait for one another
      constexpr int TW = NT < 4 ? NT : 4;
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += TW)
        if (n0 < nt_used) {
          uint4 w[TW];
          float v[TW][4];
#pragma unroll
          for (int j = 0; j < TW; ++j) {
            w[j] = lds_v4(stage + down_offset<UP, RP, SC>((n0 + j) * 8 + g, 4 * warp + t4));
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = 0.0f;
          }
#pragma unroll
          for (int j = 0; j < TW; ++j) MmaT<XT>::mma(v[j], fa[0], w[j].x, w[j].y);
#pragma unroll
          for (int j = 0; j < TW; ++j) MmaT<XT>::mma(v[j], fa[1], w[j].z, w[j].w);
#pragma unroll
          for (int j = 0; j < TW; ++j) add4(acc[n0 + j], v[j]);
        }
    } else if (UP == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (nt < nt_used) {
          const uint4 w = lds_v4(stage + down_offset<UP, RP, SC>(nt * 8 + g, 4 * warp + t4));
          MmaT<XT>::mma(acc[nt], fa[0], w.x, w.y);
          MmaT<XT>::mma(acc[nt], fa[1], w.z, w.w);
        }
    } else {
      // lane i addresses row i % 8 of matrix i / 8: (nt, low), (nt, high), (nt + 1, low), (nt + 1, high)
      const int j = lane & 7, hi = (lane >> 3) & 1, nx = lane >> 4;
      const int row = 32 * warp + 8 * (j >> 1) + (j & 1) + 2 * hi;
#pragma unroll
      for (int nt = 0; nt < NT; nt += 2)
        if (nt < nt_used) {
          float v[2][4] = {};
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            uint32_t w[4];
            ldmatrix_x4_trans(w, stage + down_offset<UP, RP, SC>(row + 4 * ks, nt + nx));
            MmaT<XT>::mma(APART ? v[0] : acc[nt], fa[ks], w[0], w[1]);
            MmaT<XT>::mma(APART ? v[1] : acc[nt + 1], fa[ks], w[2], w[3]);
          }
          if (APART) {
            add4(acc[nt], v[0]);
            add4(acc[nt + 1], v[1]);
          }
        }
    }
  };
  // Two copies of the step that change the buffers over, as one copy and register
  // moves gained nothing on the whole: rank 64, 128 requests 14336 -> 4096 50.0 against
  // 47.6 us, but 61 requests 1032 -> 1000 6.6 against 6.8; 40 shapes within 5 % either
  // way, 0.3 % in the mean; rank 16 and 128 slower by up to 15 %.
  for (int step = 0; step < steps; step += 2) {
    run_step(xv[0], xv[1], step);
    if (step + 1 < steps) run_step(xv[1], xv[0], step + 1);
  }
  cp_async_wait<0>();
  __syncthreads();

  // ---- the sums meet: warps in this CTA's memory, CTAs in their owner's ----
  float *part = reinterpret_cast<float *>(smem);  // [kLoraWarps][16][RP]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float *p = part + ((warp * kLoraRows + g) * RP + nt * 8 + 2 * t4);
    *reinterpret_cast<float2 *>(p) = make_float2(acc[nt][0], acc[nt][1]);
    *reinterpret_cast<float2 *>(p + 8 * RP) = make_float2(acc[nt][2], acc[nt][3]);
  }
  // ---- up: this CTA's output columns, 32 per warp and turn -----------------
  // UP = 0: a turn's elements of B and base are asked for two turns ahead (the
  // first before the sums are exchanged), as a turn is shorter than the way to
  // memory and back.  A lane copies what it reads itself, so no warp waits for
  // another (through registers, B one turn ahead and base none: 16 requests to
  // 14336 columns, rank 64 23.6 us instead of 17, 1536 rows in 64 segments 48
  // instead of 37).  UP = 1 goes through registers: A's columns are transposed
  // on the way.
  constexpr int KC = (RP >= 32) ? RP / 32 : 1;  // runs of 32 ranks (one of 16 where RP = 16)
  constexpr int KS = (RP >= 32) ? 2 : 1;   // k-steps in a run
  constexpr int PER = 4 * KS;              // UP = 0: ranks that a lane holds of a run
  constexpr int NV = (RP >= 32) ? RP / 8 : 2;  // UP = 1: vectors per lane and turn
  const int w_rows = (RP >= 32) ? (r_a + 31) & ~31 : 16;       // UP = 1: rows of A to stage
  // UP = 1: the row of A in vector k of this lane; the eight rows of one store
  // instruction lie in different banks
  auto w_row = [&](int k) {
    const int i8 = lane >> 2;
    return (RP >= 32) ? 32 * (k >> 2) + 8 * (i8 >> 1) + 2 * (k & 3) + (i8 & 1) : 4 * (i8 >> 1) + 2 * k + (i8 & 1);
  };
  uint4 wv[NV];
  auto load_w = [&](int cb) {
#pragma unroll
    for (int k = 0; k < NV; ++k) wv[k] = make_uint4(0, 0, 0, 0);
    if (cb >= o_end) return;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int r = w_row(k), c = cb + 8 * (lane & 3);
      if (r < r_a && c < o_end) wv[k] = ld_nc_v4(poolA + (int64_t)r * K + c);
    }
  };
  constexpr int DU = UP == 0 ? G::DU : 1;
  auto up_stage = [&](int turn) { return sbase + G::MAIN - (turn % DU + 1) * G::UP_STAGE + warp * G::SLOT; };
  // What no copy fills is never used: rows behind the tile and columns behind the
  // slice are not stored, ranks behind r_a are masked.
  const int row_a = tile.row0 + g, first = o_begin + 32 * warp;
  const bool in0 = g < tile.rows, in1 = g + 8 < tile.rows;
  const uint16_t *wp = poolB + (int64_t)(first + 8 * (g >> 1) + (g & 1)) * a.R + PER * t4;
  const uint16_t *bp = a.base + row_a * a.ldbase + first + 8 * t4;
  int next = first;  // column of the next turn to ask for
  auto fetch = [&](int turn) {
    const uint32_t at = up_stage(turn) + lane * 16;
    if (a.base && next + 8 * t4 < o_end) {
      if (in0) cp_async16(at, bp);
      if (in1) cp_async16(at + 512, bp + 8 * a.ldbase);
    }
    if (next + 8 * (g >> 1) < o_end) {
#pragma unroll
      for (int i = 0; i < KC; ++i)
        if (32 * i + PER * t4 < r_a) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (KS == 2) cp_async16(at + 1024 + (j * KC + i) * 512, wp + 2 * j * a.R + 32 * i);
            else cp_async8(at + 1024 + j * 256 - lane * 8, wp + 2 * j * a.R);
          }
        }
    }
    cp_async_commit();
    next += 32 * kLoraWarps;
    bp += 32 * kLoraWarps;
    wp += 32 * kLoraWarps * a.R;
  };
  if (UP == 1) load_w(o_begin + 32 * warp);
#pragma unroll
  for (int i = 0; i < G::EARLY; ++i) fetch(i);

  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  const int per = kLoraRows * RP / CS;  // elements that one CTA owns
  float *recv = reinterpret_cast<float *>(smem + G::MAIN);  // [CS][per]
  for (int e = 4 * (int)threadIdx.x; e < kLoraRows * RP; e += 4 * kLoraThreads) {
    float4 s = *reinterpret_cast<const float4 *>(part + e);
#pragma unroll
    for (int q = 1; q < kLoraWarps; ++q) {
      const float4 v = *reinterpret_cast<const float4 *>(part + q * kLoraRows * RP + e);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    const int owner = e / per;
    *reinterpret_cast<float4 *>(cluster.map_shared_rank(recv, owner) + rank * per + (e - owner * per)) = s;
  }
  cluster.sync();
#pragma unroll
  for (int i = G::EARLY; i < G::DU; ++i) fetch(i);
  {
    const float sc = a.scales[tile.adapter];
    const float pre = (UP == 0) ? a.drop.inv_keep : sc;  // to t (or dt) as stored
    const float post = (UP == 0) ? sc : 1.0f;                          // to what the up step multiplies
    for (int i0 = 0; i0 < per; i0 += 4 * kLoraThreads) {  // all lanes take part in a row's maximum
      const int i = i0 + 4 * (int)threadIdx.x;
      const bool own = i < per;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int q = 0; own && q < CS; ++q) {
        const float4 p = *reinterpret_cast<const float4 *>(recv + q * per + i);
        v[0] += p.x;
        v[1] += p.y;
        v[2] += p.z;
        v[3] += p.w;
      }
      const int e = rank * per + i, m = e / RP, r = e % RP;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = (r + k < r_a) ? v[k] * pre : 0.0f;
      if (a.t && own && m < tile.rows && r < a.R)
        *reinterpret_cast<float4 *>(a.t + (int64_t)(tile.row0 + m) * a.R + r) = make_float4(v[0], v[1], v[2], v[3]);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] *= post;
      float2 rs = make_float2(1.0f, 1.0f);
      if (XT == 0) {
        float mx = fmaxf(fmaxf(finite_abs(v[0]), finite_abs(v[1])), fmaxf(finite_abs(v[2]), finite_abs(v[3])));
#pragma unroll
        for (int o = 1; o < RP / 4; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        rs = tc_scale(mx);
      }
      if (!own) continue;
      uint2 hi, lo;
      split_same_sign<XT>(v[0] * rs.y, v[1] * rs.y, hi.x, lo.x);
      split_same_sign<XT>(v[2] * rs.y, v[3] * rs.y, hi.y, lo.y);
      int c = r >> 3;
      if (RP >= 64) c ^= (m & 1) << 2;
      const int at = m * RP * 2 + c * 16 + (r & 7) * 2;
      for (int q = 0; q < CS; ++q) {
        uint8_t *tt = cluster.map_shared_rank(smem, q);
        *reinterpret_cast<uint2 *>(tt + at) = hi;
        *reinterpret_cast<uint2 *>(tt + kLoraRows * RP * 2 + at) = lo;
        if (XT == 0 && r == 0) *reinterpret_cast<float *>(tt + G::SCALE + 4 * m) = rs.x;
      }
    }
  }
  cluster.sync();

  const uint32_t tbase = sbase, wbase = sbase + G::T_BYTES + warp * G::WT_BYTES;
  const float out_scale = (UP == 1) ? a.drop.inv_keep : 1.0f;
  float row_scale[2] = {1.0f, 1.0f};
  if (XT == 0) {
    row_scale[0] = *reinterpret_cast<const float *>(smem + G::SCALE + 4 * g);
    row_scale[1] = *reinterpret_cast<const float *>(smem + G::SCALE + 4 * (g + 8));
  }
  int turn = 0;
  for (int cb = o_begin + 32 * warp; cb < o_end; cb += 32 * kLoraWarps, ++turn) {
    const uint32_t from = up_stage(turn) + lane * 16;
    if (UP == 0) cp_async_wait<DU - 1>();
    uint32_t w[4][KC][KS][2];  // fragments of the up pool: n-tile, run, k-step
    if (UP == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < KC; ++i) {
          uint32_t v[4];
          if (KS == 2) {
            const uint4 q = lds_v4(from + 1024 + (j * KC + i) * 512);
            v[0] = q.x;
            v[1] = q.y;
            v[2] = q.z;
            v[3] = q.w;
          } else {
            const uint2 q = lds_v2(from + 1024 + j * 256 - lane * 8);
            v[0] = q.x;
            v[1] = q.y;
          }
          const int left = r_a - (32 * i + PER * t4);
          if (left < PER)  // what lies behind the rank may be anything
#pragma unroll
            for (int k = 0; k < PER / 2; ++k)
              v[k] &= (left > 2 * k + 1) ? 0xffffffffu : (left > 2 * k) ? 0x0000ffffu : 0u;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            w[j][i][ks][0] = v[2 * ks];
            w[j][i][ks][1] = v[2 * ks + 1];
          }
        }
    } else {
      // 32 columns of A [R, K], stored so that a transposed read gives the
      // column order above: pair p = 4 q + j of a row goes to tile j, place q
      __syncwarp();
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int r = w_row(k);
        if (r < w_rows) {
          const int f = (RP >= 32) ? (r >> 3) & 3 : (r >> 2) & 3;
          const uint32_t at = wbase + r * 64 + (lane & 3) * 4;
          sts_u32(at + ((0 ^ f) << 4), wv[k].x);
          sts_u32(at + ((1 ^ f) << 4), wv[k].y);
          sts_u32(at + ((2 ^ f) << 4), wv[k].z);
          sts_u32(at + ((3 ^ f) << 4), wv[k].w);
        }
      }
      __syncwarp();
      const int l = lane & 7, hi = (lane >> 3) & 1, jx = lane >> 4;
#pragma unroll
      for (int i = 0; i < KC; ++i)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int r = (RP >= 32) ? 32 * i + 8 * (l >> 1) + 4 * ks + (l & 1) + 2 * hi : 4 * (l >> 1) + (l & 1) + 2 * hi;
          const int f = (RP >= 32) ? (r >> 3) & 3 : (r >> 2) & 3;
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            uint32_t q[4] = {0, 0, 0, 0};
            if (32 * i < r_a) ldmatrix_x4_trans(q, wbase + r * 64 + (((j + jx) ^ f) << 4));
            w[j][i][ks][0] = q[0];
            w[j][i][ks][1] = q[1];
            w[j + 1][i][ks][0] = q[2];
            w[j + 1][i][ks][1] = q[3];
          }
        }
    }
    if (UP == 1) load_w(cb + 32 * kLoraWarps);
    const int col = cb + 8 * t4;
    const bool ok0 = in0 && col < o_end, ok1 = in1 && col < o_end;
    uint4 b0 = make_uint4(0, 0, 0, 0), b1 = b0;
    if (UP == 1 && a.base) {
      if (ok0) b0 = *reinterpret_cast<const uint4 *>(a.base + row_a * a.ldbase + col);
      if (ok1) b1 = *reinterpret_cast<const uint4 *>(a.base + (row_a + 8) * a.ldbase + col);
    }
    float d[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) d[j][i] = 0.0f;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      if (32 * i >= r_a) break;
      uint32_t fh[KS][4], fl[KS][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // rows g, g + 8
        const int m = half * 8 + g;
        if (KS == 2) {
          int c = 4 * i + t4;
          if (RP >= 64) c ^= (m & 1) << 2;
          const uint32_t at = tbase + m * RP * 2 + c * 16;
          const uint4 h = lds_v4(at), l = lds_v4(at + kLoraRows * RP * 2);
          fh[0][half] = h.x;
          fh[0][2 + half] = h.y;
          fh[KS - 1][half] = h.z;
          fh[KS - 1][2 + half] = h.w;
          fl[0][half] = l.x;
          fl[0][2 + half] = l.y;
          fl[KS - 1][half] = l.z;
          fl[KS - 1][2 + half] = l.w;
        } else {
          const uint32_t at = tbase + m * RP * 2 + t4 * 8;
          const uint2 h = lds_v2(at), l = lds_v2(at + kLoraRows * RP * 2);
          fh[0][half] = h.x;
          fh[0][2 + half] = h.y;
          fl[0][half] = l.x;
          fl[0][2 + half] = l.y;
        }
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          MmaT<XT>::mma(d[j], fh[ks], w[j][i][ks][0], w[j][i][ks][1]);
          MmaT<XT>::mma(d[j], fl[ks], w[j][i][ks][0], w[j][i][ks][1]);
        }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (!(half ? ok1 : ok0)) continue;
      uint4 b = half ? b1 : b0;
      if (UP == 0 && a.base) b = lds_v4(from + 512 * half);
      uint32_t bw[4] = {b.x, b.y, b.z, b.w}, ow[4];
      uint4 keep = make_uint4(0, 0, 0, 0);
      if (UP == 1 && drop) keep = drop_block(dst, (uint32_t)col >> 3, (uint32_t)(row_a + 8 * half));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v0 = d[j][2 * half], v1 = d[j][2 * half + 1];
        if (XT == 0) {
          v0 *= row_scale[half];
          v1 *= row_scale[half];
        }
        if (UP == 1 && drop) {
          v0 = drop_keep(keep, 2 * j, dst.thr_hi) ? v0 * out_scale : 0.0f;
          v1 = drop_keep(keep, 2 * j + 1, dst.thr_hi) ? v1 * out_scale : 0.0f;
        }
        const float2 bf = Elem<XT>::pair(bw[j]);
        ow[j] = (uint32_t)Elem<XT>::from_float(bf.x + v0) | ((uint32_t)Elem<XT>::from_float(bf.y + v1) << 16);
      }
      *reinterpret_cast<uint4 *>(a.y + (row_a + 8 * half) * a.ldy + col) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
    }
    if (UP == 0) fetch(turn + DU);  // this turn's stage has been read
  }
  cp_async_wait<0>();
}

}  // namespace bq

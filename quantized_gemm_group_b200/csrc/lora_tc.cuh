// lora_tc.cuh -- low-rank adapters on the 5th-generation tensor cores, for
// segments of many rows (the kernel of lora.cuh takes short ones), and their
// weight gradients.  The operands' formulas are in lora.cuh.
//
// What bounds it is memory; mma.sync spent about 15 instructions for every
// matrix instruction on addresses, fragments and partial sums and reached a
// third of the copy rate (8192 rows, 14336 -> 4096, rank 64: 180 us, gradients
// of 4096 -> 14336 510 us).  Here tiles come by TMA, tcgen05.mma reads them from shared
// memory, and threads touch only t, the masks and the output.
//
// lora_tc_kernel: a cluster of up to 8 CTAs owns 128 rows of one segment.  Each
// contracts its share of the columns into tensor memory (down), sends its
// partial sums to the CTA that owns the row (distributed shared memory, added
// in rank order: the same bits every time), the owner sends the 16-bit parts of
// t to all of them, and each writes its share of the output columns (up).
// Roles (10 or 18 warps): warp 0 producer (one ring of slots: a chunk of x and
// of the down pool, later a chunk of base and of the up pool); warp 1 issues
// tcgen05.mma; the others (two or four per TMEM lane quadrant) mask x, exchange
// the sums and finish the output.
// Two persistent kernels instead (down, then up, one CTA per SM, equal runs of
// steps, sums through global scratch) took 92 us where this one takes 80, and
// 43 where it takes 33 (4096 rows, 4096 -> 4096, rank 64): a second launch and
// the sums' way through L2 cost more than the exchange.
//
// Rounding: t enters the up product as two 16-bit parts, t = hi + lo (bf16:
// relative error below 2^-17; fp16: the row is first scaled by a power of two so
// that its largest value lies in [2^14, 2^15), error below 2^-22 of the value and 2^-38
// of the largest).  Their products have sums of their own, so that those of hi say
// where an infinite element gives an infinity (lora.cuh's kernel gives lo hi's sign
// instead, which costs a bit).  One
// part would lose 2^-9; the second costs a matrix instruction and no traffic.
// Long sums leave the tensor core's accumulator every 16 instructions (kTcRun).
//
// What lies outside never enters a product: columns behind K, N or R are
// zero-filled by TMA (the pools are 3D maps, so an adapter's end is an edge),
// ranks behind an adapter's rank are zeroed in shared memory where they share
// a k-step of 16 with used ones, and rows behind a segment's end only reach
// output rows that are not stored (weight gradients: they are zeroed).
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "dropout.cuh"
#include "gemm.cuh"
#include "lora.cuh"

namespace bq {

constexpr int kTcRows = 128;                   // rows per tile (MMA M)
constexpr int kTcXBox = 64;                    // rows per TMA box of x and base
constexpr int kTcMaxCS = 8;                    // CTAs per cluster at most
// Steps down whose products add up in tensor memory: 16 instructions.  The
// accumulator cuts where fp32 additions round (up to 2^-23 of the running sum
// lost at each instruction, always towards zero), so a run this long loses about
// 3e-7 and the runs are added in registers.  In one run 14336 columns in clusters
// of 2 (448 instructions) lost 8e-6 of t's norm, in single CTAs 1.6e-5; plain fp32
// products lose about 1e-6.
constexpr int kTcRun = 4;

// ---------------------------------------------------------------------------
// primitives
// ---------------------------------------------------------------------------

// Shared-memory matrix descriptor, 128-byte swizzle.  K-major: 8-row groups
// SBO = 1024 bytes apart.  MN-major (rows run along the contraction, 64
// elements of the other index in a row): 8-row groups SBO = 1024 bytes
// apart, blocks of 64 elements LBO bytes apart.
BQ_DEV uint64_t tc_desc(uint32_t smem_addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
// Instruction descriptor (see gemm_idesc): M = 128, fp32 accumulation, both
// operands of type XT; MN-major operands set bit 15 (A) / 16 (B).
template <int XT> BQ_DEV uint32_t tc_idesc(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((uint32_t)XT << 7) | ((uint32_t)XT << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTcRows >> 4) << 24);
}
BQ_DEV void tc_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
BQ_DEV void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
// Arrive on the mbarrier at this shared-memory address of CTA `cta` of the cluster.
BQ_DEV void mbar_arrive_cta(uint32_t bar, uint32_t cta) {
  asm volatile(
      "{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\t"
      "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [ra];\n\t}" ::"r"(bar),
      "r"(cta)
      : "memory");
}
BQ_DEV bool mbar_wait_cluster(uint32_t bar, uint32_t parity) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}
BQ_DEV void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
BQ_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
BQ_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
BQ_DEV void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
BQ_DEV uint4 and4(uint4 a, uint4 b) { return make_uint4(a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w); }
BQ_DEV void sts_v4(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
BQ_DEV void tc_give_up(volatile int *abort) {  // a wait ran out: the other roles leave too
  if (!*abort) bq_flag(BQ_FLAG_TIMEOUT);
  *abort = 1;
}
// 16 consecutive fp32 columns of this thread's TMEM lane from each of two places.
BQ_DEV void tmem_ld16_two(uint32_t a, uint32_t b, float (&v)[16], float (&w)[16]) {
  uint32_t r[32];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[16 * k]), "=r"(r[16 * k + 1]), "=r"(r[16 * k + 2]), "=r"(r[16 * k + 3]), "=r"(r[16 * k + 4]),
          "=r"(r[16 * k + 5]), "=r"(r[16 * k + 6]), "=r"(r[16 * k + 7]), "=r"(r[16 * k + 8]), "=r"(r[16 * k + 9]),
          "=r"(r[16 * k + 10]), "=r"(r[16 * k + 11]), "=r"(r[16 * k + 12]), "=r"(r[16 * k + 13]), "=r"(r[16 * k + 14]),
          "=r"(r[16 * k + 15])
        : "r"(k == 0 ? a : b));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = __uint_as_float(r[i]);
    w[i] = __uint_as_float(r[16 + i]);
  }
}
// Zeros in 16 consecutive columns of this thread's TMEM lane.
BQ_DEV void tmem_zero16(uint32_t taddr) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1};" ::"r"(taddr),
               "r"(0)
               : "memory");
}
BQ_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------------------
// forward / input gradient
// ---------------------------------------------------------------------------

// DEEP: one CTA per SM with a deep ring and 16 worker warps, for grids that do
// not fill the GPU twice (and for ranks above 64, whose pools are twice as
// large); else two CTAs per SM, so that one's exchange hides behind the other's
// streams.
template <int RP, bool DEEP> struct TcGeom {
  static_assert(DEEP || RP == 64, "two CTAs of rank 128 do not fit an SM");
  static constexpr int NG = DEEP ? 4 : 2;           // worker warps per TMEM lane quadrant
  static constexpr int WORKERS = 4 * NG;            // worker warps
  static constexpr int THREADS = 32 * (2 + WORKERS);
  static constexpr int X_BYTES = kTcRows * 128;     // 128 rows x 64 columns
  static constexpr int W_BYTES = RP * 128;          // 64 x RP of a pool
  static constexpr int SLOT = X_BYTES + W_BYTES;
  static constexpr int NS = RP == 128 ? 4 : DEEP ? 7 : 3;
  static constexpr int BLOCKS = RP / 64;            // 64-rank blocks
  static constexpr int T_BYTES = 2 * BLOCKS * kTcRows * 128;  // hi and lo
  // the sums' buffer lies there before: [CS][ceil(128 / CS) rows][RP] fp32, at most 133 rows
  static constexpr int T_AREA = 136 * RP * 4;
  static_assert(T_AREA >= T_BYTES, "t and the sums share their place");
  static constexpr int TOTAL0 = NS * SLOT + T_AREA;
  static constexpr int bar_off = TOTAL0;
  static constexpr int nbar = 4 * NS + 2 * NG + 9;
  static constexpr int scale_off = bar_off + 8 * nbar;  // fp32 per row
  static constexpr int tmem_off = scale_off + 4 * kTcRows;
  static constexpr int abort_off = tmem_off + 4;
  static constexpr int total = abort_off + 4 + 1024;
  // two buffers of P; when all of P has been read, the output: for each of NG
  // groups 64 columns of hi's products and 64 of lo's
  static constexpr int TM_COLS = DEEP ? 512 : 256;
  static_assert(2 * RP <= TM_COLS && 128 * NG <= TM_COLS, "tensor memory");
  static constexpr int P_GROUPS = RP / 16 / NG;     // groups of 16 ranks whose sums a worker warp keeps
  static constexpr int PER_THREAD = kTcRows * RP / 4 / (32 * WORKERS);  // quads of sums per worker, CS = 1
};

struct TcBars {
  uint32_t full, masked, free_mma, free_out;  // [NS]
  uint32_t p_full, p_empty;                   // [2]
  uint32_t d_full, d_empty;                   // [ng]
  uint32_t recv, taken, t_in, t_ready, done;
  BQ_DEV TcBars(uint32_t base, int ns, int ng) {
    full = base;
    masked = full + 8u * ns;
    free_mma = masked + 8u * ns;
    free_out = free_mma + 8u * ns;
    p_full = free_out + 8u * ns;
    p_empty = p_full + 16u;
    d_full = p_empty + 16u;
    d_empty = d_full + 8u * ng;
    recv = d_empty + 8u * ng;
    taken = recv + 8u;
    t_in = taken + 8u;
    t_ready = t_in + 8u;
    done = t_ready + 8u;
  }
};

// Worker warps (NG per TMEM lane quadrant, thread = row of the tile).
template <int XT, int UP, int RP, bool DEEP>
BQ_DEV void lora_tc_workers(const LoraArgs &a, const LoraTile &tile, int r_a, int r16, int D, int U, bool patch, bool pad,
                            int rank, uint32_t tmem, uint32_t sbase, unsigned char *smem, const TcBars &B, volatile int *abort, cg::cluster_group &cluster) {
  const int CS = a.CS;
  using G = TcGeom<RP, DEEP>;
  constexpr int NS = G::NS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wt = (int)threadIdx.x - 64;
  const int quad = warp & 3, grp = (warp - 2) >> 2, m = quad * 32 + lane;
  const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
  const bool drop = a.drop.thr != 0;
  const DropState dst = drop_state(a.drop);
  bool ok = true;
  auto vote = [&](bool v) { return __all_sync(0xffffffffu, v) != 0; };

  // A finished run of the down product is added to this warp's sums: row m,
  // ranks 16 (grp + NG k) onwards.
  float psum[G::P_GROUPS][16];
#pragma unroll
  for (int k = 0; k < G::P_GROUPS; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) psum[k][i] = 0.0f;
  const int runs = (D + kTcRun - 1) / kTcRun;
  int run = 0;
  auto add_run = [&]() {
    const int buf = run & 1;
    ok = vote(!*abort && mbar_wait(B.p_full + 8u * buf, (run >> 1) & 1));
    if (!ok) return;
    tc_fence_after();
#pragma unroll
    for (int k = 0; k < G::P_GROUPS; ++k) {
      const int cgp = grp + G::NG * k;
      if (cgp < r16 / 16) {
        float v[16];
        tmem_ld16(tmem + lane_addr + buf * RP + cgp * 16, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) psum[k][i] += v[i];
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(B.p_empty + 8u * buf);
    ++run;
  };

  // ---- down: masks on x (drawn while x is on its way) -----------------------
  if (patch)
    for (int s = 0; s < D && ok; ++s) {
      const int slot = s % NS;
      constexpr int PT = kTcRows * 8 / (32 * G::WORKERS);  // 16-byte chunks per worker
      uint4 mask[PT];
      if (UP == 0 && drop) {
#pragma unroll
        for (int k = 0; k < PT; ++k) {
          const int i = wt + k * 32 * G::WORKERS;
          mask[k] = drop_mask8(drop_block(dst, (uint32_t)(8 * (rank + CS * s) + (i & 7)), (uint32_t)(tile.row0 + (i >> 3))),
                               dst.thr_hi);
        }
      }
      ok = vote(!*abort && mbar_wait(B.full + 8u * slot, (s / NS) & 1));
      if (!ok) break;
      if (UP == 0 && drop) {
        const uint32_t xs = sbase + slot * G::SLOT;
#pragma unroll
        for (int k = 0; k < PT; ++k) {
          const int i = wt + k * 32 * G::WORKERS, row = i >> 3;
          const uint32_t at = xs + row * 128 + (((i & 7) ^ (row & 7)) << 4);
          sts_v4(at, and4(lds_v4(at), mask[k]));
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(B.masked + 8u * slot);
      // the run before this one: by now its products are done, and its buffer is
      // free before the next run asks for it
      if (s % kTcRun == kTcRun - 2 && s >= kTcRun) add_run();
    }

  // ---- the sums meet -------------------------------------------------------
  // partial sums go to the owner of the row: [source CTA][own rows][RP], 16-byte
  // chunks XORed with the row so that a warp's rows lie in different banks
  const int own = (kTcRows + CS - 1) / CS;
  float *recv = reinterpret_cast<float *>(smem + NS * G::SLOT);
  while (ok && run < runs) add_run();
  cluster_wait();
  if (ok) {
    const int rr = rank * own + m % own;
    float *to = cluster.map_shared_rank(recv, m / own) + rr * RP;
#pragma unroll
    for (int k = 0; k < G::P_GROUPS; ++k) {
      const int cgp = grp + G::NG * k;
      if (cgp < r16 / 16) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<float4 *>(to + 4 * ((cgp * 4 + q) ^ (rr & 7))) =
              make_float4(psum[k][4 * q], psum[k][4 * q + 1], psum[k][4 * q + 2], psum[k][4 * q + 3]);
      }
    }
    __syncwarp();
    if (lane < CS) mbar_arrive_cta(B.recv, lane);
    ok = vote(mbar_wait_cluster(B.recv, 0));
  }
  float sum[G::PER_THREAD][4];
  if (ok) {
    const float sc = a.scales[tile.adapter];
    const float pre = (UP == 0) ? a.drop.inv_keep : sc;  // to t (or dt) as stored
#pragma unroll
    for (int k = 0; k < G::PER_THREAD; ++k) {
      const int i = wt + k * 32 * G::WORKERS, ml = i / (RP / 4), chunk = i % (RP / 4), r = 4 * chunk;
      const int row = rank * own + ml;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (ml < own && row < tile.rows && r < r_a)
        for (int q = 0; q < CS; ++q) {
          const int rr = q * own + ml;
          const float4 p = *reinterpret_cast<const float4 *>(recv + rr * RP + 4 * (chunk ^ (rr & 7)));
          v[0] += p.x;
          v[1] += p.y;
          v[2] += p.z;
          v[3] += p.w;
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[k][j] = (r + j < r_a) ? v[j] * pre : 0.0f;
      if (a.t && ml < own && row < tile.rows && r < a.R)
        *reinterpret_cast<float4 *>(a.t + (int64_t)(tile.row0 + row) * a.R + r) =
            make_float4(sum[k][0], sum[k][1], sum[k][2], sum[k][3]);
    }
    __syncwarp();
    if (lane < CS) mbar_arrive_cta(B.taken, lane);  // this CTA's buffer may be overwritten by t
    ok = vote(mbar_wait_cluster(B.taken, 0));
  }
  if (ok) {
    const float post = (UP == 0) ? a.scales[tile.adapter] : 1.0f;  // to what the up step multiplies
#pragma unroll
    for (int k = 0; k < G::PER_THREAD; ++k) {
      const int i = wt + k * 32 * G::WORKERS, ml = i / (RP / 4), r = 4 * (i % (RP / 4)), row = rank * own + ml;
      if (k * 32 * G::WORKERS >= own * (RP / 4)) break;
      float2 sc = make_float2(1.0f, 1.0f);
      if (XT == 0) {
        float mx = fmaxf(fmaxf(finite_abs(sum[k][0] * post), finite_abs(sum[k][1] * post)),
                         fmaxf(finite_abs(sum[k][2] * post), finite_abs(sum[k][3] * post)));
#pragma unroll
        for (int o = 1; o < RP / 4; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        sc = tc_scale(mx);
      }
      uint2 hi, lo;
      tc_split<XT>(sum[k][0] * post * sc.y, sum[k][1] * post * sc.y, hi.x, lo.x);
      tc_split<XT>(sum[k][2] * post * sc.y, sum[k][3] * post * sc.y, hi.y, lo.y);
      const int at = (r >> 6) * (kTcRows * 128) + row * 128 + ((((r & 63) >> 3) ^ (row & 7)) << 4) + (r & 7) * 2;
      if (ml < own && row < kTcRows && r < r16)
        for (int q = 0; q < CS; ++q) {
          unsigned char *to = cluster.map_shared_rank(smem, q);
          *reinterpret_cast<uint2 *>(to + NS * G::SLOT + at) = hi;
          *reinterpret_cast<uint2 *>(to + NS * G::SLOT + G::BLOCKS * kTcRows * 128 + at) = lo;
          if (XT == 0 && r == 0) *reinterpret_cast<float *>(to + G::scale_off + 4 * row) = sc.x;
        }
    }
    fence_proxy_async_all();  // t is read by the tensor cores
    __syncwarp();
    if (lane < CS) mbar_arrive_cta(B.t_in, lane);
    ok = vote(mbar_wait_cluster(B.t_in, 0));
    fence_proxy_async_all();
    __syncwarp();
    if (ok && lane == 0) mbar_arrive(B.t_ready);
  }

  // ---- up: base + t W2, 64 columns a step -------------------------------------
  // The warps of a quadrant take steps in turn (each its own buffer of tensor
  // memory), so that one's waits hide behind the others' work: a step is a
  // chain of waits, and with both warps of two on the same step it took 1.3 us.
  const float row_scale = (XT == 0 && ok) ? *reinterpret_cast<const float *>(smem + G::scale_off + 4 * m) : 1.0f;
  uint16_t *out = a.y + (int64_t)(tile.row0 + quad * 32 + (lane >> 3)) * a.ldy + 8 * (lane & 7);
  for (int j = grp; j < U && ok; j += G::NG) {
    const int s = D + j, slot = s % NS;
    const uint32_t xs = sbase + slot * G::SLOT, ws = xs + G::X_BYTES;
    const int col0 = 64 * (rank + CS * j);
    ok = vote(!*abort && mbar_wait(B.full + 8u * slot, (s / NS) & 1));
    if (!ok) break;
    if (patch) {
      const int wg = quad * 32 + lane;
      if (pad && UP == 0) {  // W2 [64 rows][ranks]: zero ranks r_a .. r16 - 1
        const int n = wg >> 1, r = r16 - 16 + 8 * (wg & 1), live = r_a - r;
        if (live < 8) {
          const uint32_t wat = ws + (r >> 6) * 8192 + n * 128 + ((((r & 63) >> 3) ^ (n & 7)) << 4);
          const uint4 v = lds_v4(wat);
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] &= (live > 2 * k + 1) ? 0xffffffffu : (live > 2 * k) ? 0x0000ffffu : 0u;
          sts_v4(wat, make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
      if (pad && UP == 1 && wg < 8 * (r16 - r_a)) sts_v4(ws + (r_a + (wg >> 3)) * 128 + (wg & 7) * 16, make_uint4(0, 0, 0, 0));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane < G::NG) mbar_arrive(B.masked + 8u * slot);  // for the quadrant's other warps too
    }
    ok = vote(mbar_wait(B.d_full + 8u * grp, (j / G::NG) & 1));
    if (!ok) break;
    tc_fence_after();
#pragma unroll
    for (int hc = 0; hc < 4; ++hc) {
      float d[16], lo[16];
      const uint32_t at_hi = tmem + lane_addr + 128 * grp + 16 * hc;
      tmem_ld16_two(at_hi, at_hi + 64, d, lo);
      if (hc == 3) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(B.d_empty + 8u * grp);
      }
      // lo is often 0 or of hi's other sign: where an infinite element of the pool made
      // its products NaN, hi's alone say what the formula gives
      float2 any = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < 16; i += 2) any = __fadd2_rn(any, make_float2(lo[i], lo[i + 1]));
      if (!(fabsf(any.x + any.y) <= 3.402823466e38f)) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!(fabsf(d[i]) <= 3.402823466e38f)) lo[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float2 v = __fadd2_rn(make_float2(d[i], d[i + 1]), make_float2(lo[i], lo[i + 1]));
        d[i] = v.x;
        d[i + 1] = v.y;
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t at = xs + m * 128 + (((2 * hc + q) ^ (m & 7)) << 4);
        uint4 b = make_uint4(0, 0, 0, 0);
        if (a.base) b = lds_v4(at);
        if (UP == 1 && drop) {
          const uint4 keep = drop_block(dst, (uint32_t)((col0 >> 3) + 2 * hc + q), (uint32_t)(tile.row0 + m));
#pragma unroll
          for (int i = 0; i < 8; ++i)
            d[8 * q + i] = drop_keep(keep, i, dst.thr_hi) ? d[8 * q + i] * a.drop.inv_keep : 0.0f;
        }
        const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
        uint32_t ow[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 v = make_float2(d[8 * q + 2 * i], d[8 * q + 2 * i + 1]);
          const float2 bf = Elem<XT>::pair(bw[i]);
          v = XT == 0 ? __ffma2_rn(v, make_float2(row_scale, row_scale), bf) : __fadd2_rn(v, bf);
          ow[i] = pack_pair<XT>(v);
        }
        sts_v4(at, make_uint4(ow[0], ow[1], ow[2], ow[3]));
      }
    }
    __syncwarp();
    // this warp's 32 rows x 128 bytes leave in whole lines; the slot is free
    // (its next contents come by TMA) before the stores are under way
    uint4 o[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int row = quad * 32 + q * 4 + (lane >> 3);
      o[q] = lds_v4(xs + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(B.free_out + 8u * slot);
    const bool in = col0 + 8 * (lane & 7) < a.Co;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (in && quad * 32 + q * 4 + (lane >> 3) < tile.rows) st_v4(out + (int64_t)(4 * q) * a.ldy + col0, o[q]);
  }
  if (!ok && lane == 0) tc_give_up(abort);
}

// grid = CS x tiles, cluster = (CS, 1, 1).  mx: x [M, Ci]; mA: A {K, R, L}, boxes
// of 64 columns x round_up(R, 16) ranks; mB: B {R, N, L}, boxes of 64 ranks x 64 rows;
// mbase: base [M, Co].
// Registers are handed out for whole groups of four warps, so two CTAs of 10
// warps fit an SM as two of 12 do.
template <int XT, int UP, int RP, bool DEEP>
__global__ void __launch_bounds__(DEEP ? TcGeom<RP, DEEP>::THREADS : 384, DEEP ? 1 : 2)
lora_tc_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mA,
               const __grid_constant__ CUtensorMap mB, const __grid_constant__ CUtensorMap mbase, const LoraArgs a) {
  using G = TcGeom<RP, DEEP>;
  constexpr int NS = G::NS;
  extern __shared__ __align__(1024) unsigned char tsm_raw[];
  const uint32_t raw = smem_u32(tsm_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char *smem = tsm_raw + (sbase - raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int CS = a.CS, rank = (int)blockIdx.x % CS, tile_index = (int)blockIdx.x / CS;
  volatile int *abort = reinterpret_cast<volatile int *>(smem + G::abort_off);
  const TcBars B(sbase + G::bar_off, NS, G::NG);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(B.full + 8u * i, 1);
      mbar_init(B.masked + 8u * i, G::WORKERS);
      mbar_init(B.free_mma + 8u * i, 1);
      mbar_init(B.free_out + 8u * i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(B.p_full + 8u * i, 1);
      mbar_init(B.p_empty + 8u * i, G::WORKERS);
    }
    for (int i = 0; i < G::NG; ++i) {
      mbar_init(B.d_full + 8u * i, 1);
      mbar_init(B.d_empty + 8u * i, 4);
    }
    mbar_init(B.recv, CS * G::WORKERS);
    mbar_init(B.taken, CS * G::WORKERS);
    mbar_init(B.t_in, CS * G::WORKERS);
    mbar_init(B.t_ready, G::WORKERS);
    mbar_init(B.done, 1);
    *abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + G::tmem_off),
                 "n"(G::TM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    prefetch_map(&mx);
    prefetch_map(UP ? &mB : &mA);
    if (a.Co > 0) prefetch_map(UP ? &mA : &mB);
    if (a.Co > 0 && a.base) prefetch_map(&mbase);
  }
  pdl_wait();
  if (blockIdx.x == 0 && warp == G::WORKERS + 1)
    lora_check_segments(a.seg_off, a.seg_adapter, a.ranks, a.S, a.L, a.R, a.M);
  const LoraTile tile = lora_find_tile<kTcRows>(a.seg_off, a.seg_adapter, a.S, a.M, tile_index);
  const int r_a = tile.found ? lora_rank(a.ranks, tile.adapter, a.L, a.R) : 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // everything before this kernel is complete, and this CTA has its tensor memory
  pdl_launch_dependents();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + G::tmem_off);
  if (r_a == 0) {  // the whole cluster: no such tile, or one without a contribution
    if (warp == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(G::TM_COLS) : "memory");
    if (tile.found) lora_copy_rows(a, tile, rank, CS, G::THREADS);
    return;
  }
  const int r16 = (r_a + 15) & ~15;
  // Steps down and up: the cluster's CTAs take the 64-column chunks of a row in
  // turn, so that at any time they read and write neighbouring pieces of it.
  const int D = ((a.Ci + 63) / 64 - rank + CS - 1) / CS, U = ((a.Co + 63) / 64 - rank + CS - 1) / CS;
  const bool drop = a.drop.thr != 0;
  // the last k-step of the up product needs zeros behind the rank (behind R there are)
  const bool pad = (r_a & 15) != 0 && r_a < a.R;
  const bool patch = pad || (UP == 0 && drop);     // workers touch the slots before the MMA
  const int blocks = (r_a + 63) / 64;              // 64-rank blocks in use

  cluster_arrive();  // barriers are initialised in every CTA before any remote arrival (the workers wait)
  const uint32_t t_smem = sbase + NS * G::SLOT;

  if (warp == 0) {
    if (lane == 0) {
      const int boxes = (tile.rows + kTcXBox - 1) / kTcXBox, ra16 = (a.R + 15) & ~15;
      const uint32_t a_bytes = ra16 * 128, b_bytes = blocks * 8192, x_bytes = boxes * kTcXBox * 128;
      int slot = 0, s = 0;
      for (; s < D + U; ++s) {
        const bool down = s < D;
        const int prev = s - NS;
        // the slot's last use: a step down is freed by its MMAs, a step up by the workers
        if (prev >= 0 && !(prev < D ? mbar_wait(B.free_mma + 8u * slot, (prev / NS) & 1)
                                    : mbar_wait(B.free_out + 8u * slot, ((prev - D) / NS) & 1))) {
          tc_give_up(abort);
          break;
        }
        const uint32_t xs = sbase + slot * G::SLOT, full = B.full + 8u * slot;
        const int c = 64 * (rank + CS * (down ? s : s - D));
        const bool from_a = down == (UP == 0);   // this step reads A, else B
        const bool rows_in = down || a.base;
        const CUtensorMap *map = down ? &mx : &mbase;
        mbar_arrive_expect_tx(full, (rows_in ? x_bytes : 0) + (from_a ? a_bytes : b_bytes));
        if (rows_in) {
          tma_load_2d(xs, map, c, tile.row0, full);
          if (boxes > 1) tma_load_2d(xs + kTcXBox * 128, map, c, tile.row0 + kTcXBox, full);
        }
        if (from_a) {
          tma_load_3d(xs + G::X_BYTES, &mA, c, 0, tile.adapter, full);
        } else {
          tma_load_3d(xs + G::X_BYTES, &mB, 0, c, tile.adapter, full);
          if (RP > 64 && blocks > 1) tma_load_3d(xs + G::X_BYTES + 8192, &mB, 64, c, tile.adapter, full);
        }
        if (++slot == NS) slot = 0;
      }
      // every copy has landed before the CTA may exit
      for (int j = 1; j <= NS && j <= s; ++j) mbar_wait(B.full + 8u * ((s - j) % NS), ((s - j) / NS) & 1, 1u << 20);
    }
    __syncwarp();
    cluster_wait();
  } else if (warp == 1) {
    // One thread issues everything, so a step is kept to its wait, its MMAs on
    // running descriptors and a commit (built anew for each MMA they took 80
    // cycles of this thread).
    if (lane == 0) {
      const uint32_t ready = patch ? B.masked : B.full;
      bool ok = true;
      int slot = 0;
      uint32_t use = 0;
      const uint64_t xd0 = tc_desc(sbase, 16);
      // down: P [128 rows, r16] = x . W1, A operand x (K-major); W1 = A [r][64 c]
      // (K-major) forward, B [64 c][r] (MN-major) in the gradient
      {
        const uint32_t id = tc_idesc<XT>(r16, false, UP == 1);
        const uint64_t wd0 = tc_desc(sbase + G::X_BYTES, UP == 0 ? 16 : 8192);
        constexpr uint64_t KW = UP == 0 ? 2 : 128;  // a k-step of W1 in a descriptor's units of 16 bytes
        for (int s = 0; s < D; ++s) {
          const int run = s / kTcRun, buf = run & 1;
          const bool first = s % kTcRun == 0, last = s % kTcRun == kTcRun - 1 || s == D - 1;
          // the buffer's last run has left it
          ok = mbar_wait(ready + 8u * slot, use) &&
               (!first || run < 2 || mbar_wait(B.p_empty + 8u * buf, ((run >> 1) & 1) ^ 1));
          if (!ok) break;
          tc_fence_after();
          const uint64_t at = (uint64_t)(slot * (G::SLOT >> 4));
#pragma unroll
          for (int k = 0; k < 4; ++k) tc_mma(tmem + buf * RP, xd0 + at + 2 * k, wd0 + at + KW * k, id, k > 0 || !first);
          umma_commit(B.free_mma + 8u * slot);
          if (last) umma_commit(B.p_full + 8u * buf);
          if (++slot == NS) {
            slot = 0;
            use ^= 1;
          }
        }
      }
      // up: 64 output columns a step, A operand t (hi and lo, their products apart; P's
      // columns are free, as t_ready comes after its last run was read); W2 = B [64 c][r]
      // (K-major) forward, A [r][64 c] (MN-major) in the gradient
      const uint32_t id = tc_idesc<XT>(64, false, UP == 1);
      const uint64_t td = tc_desc(t_smem, 16), wd0 = tc_desc(sbase + G::X_BYTES, UP == 0 ? 16 : 8192);
      const int ks = r16 / 16;
      if (ok && U > 0) ok = mbar_wait(B.t_ready, 0);
      for (int j = 0; j < U && ok; ++j) {
        const int buf = j % G::NG;
        ok = mbar_wait(ready + 8u * slot, use) && (j < G::NG || mbar_wait(B.d_empty + 8u * buf, ((j / G::NG) & 1) ^ 1));
        if (!ok) break;
        tc_fence_after();
        const uint64_t wd = wd0 + (uint64_t)(slot * (G::SLOT >> 4));
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int k = 0; k < RP / 16; ++k)
            if (k < ks)
              tc_mma(tmem + 128 * buf + 64 * part, td + (part * G::BLOCKS + k / 4) * (kTcRows * 128 >> 4) + 2 * (k % 4),
                     UP == 0 ? wd + (k / 4) * 512 + 2 * (k % 4) : wd + 128 * k, id, k > 0);
        umma_commit(B.d_full + 8u * buf);
        if (++slot == NS) {
          slot = 0;
          use ^= 1;
        }
      }
      if (!ok) tc_give_up(abort);
    }
    __syncwarp();
    cluster_wait();
  } else {
    lora_tc_workers<XT, UP, RP, DEEP>(a, tile, r_a, r16, D, U, patch, pad, rank, tmem, sbase, smem, B, abort, cluster);
  }

  // everything issued by this CTA has finished before the tensor memory goes
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (*abort && lane == 0) {
      umma_commit(B.done);
      mbar_wait(B.done, 0, 1u << 20);
    }
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(G::TM_COLS) : "memory");
  }
  cluster_arrive();  // no CTA leaves while another may still write into its shared memory
  cluster_wait();
}

// ---------------------------------------------------------------------------
// weight gradients
// ---------------------------------------------------------------------------
//   dA[a] = sum_m dt[m]^T drop(x)[m]        [R, K]
//   dB[a] = sum_m s_a dy[m]^T t[m]          [N, R]
// Both are G[c, r] = sum_m X[m, c] P[m, r] over the rows of the adapter's
// segments, X 16-bit and P fp32: tcgen05.mma with the column c as M and
// the rank as N, both operands MN-major (their rows run along the
// contraction, as they lie in memory).  One launch does both gradients: a
// cluster owns CT columns (256 up to rank 64) of one adapter's dA or dB, its CTAs take
// the adapter's 64-row tiles in turn, and their fp32 sums meet in distributed
// shared memory in rank order: no atomics, no partial gradients in global
// memory, and an adapter that occurs in several segments is summed by one
// cluster.
// P enters as 16-bit parts side by side along N, so that one matrix
// instruction multiplies all of them: bf16 three parts (24 bits); fp16 two,
// P scaled by a power of two that brings the largest of the CTA's rows into
// [2^14, 2^15).  X is read once; P once for each CT columns (from L2).
// The products of the first part leave tensor memory every kWgRun steps and are
// added in registers (as in lora_tc_kernel: in one run, 8192 rows lost 9e-6 of the
// gradient's norm).  So that the instructions go on meanwhile it has two places,
// before and behind the lower parts, which are 2^8 times smaller and stay:
// even runs multiply [first | lower], odd ones [lower | first] one place further.

struct WgradSide {
  const float *P;     // [M, R]
  float *out;         // dA [L, R, C], or dB [L, C, R]
  int C;
  int tiles;          // column tiles; 0 if this gradient is not wanted
};

struct WgradArgs {
  WgradSide dA, dB;
  const int *ranks;
  const float *scales;
  const int *seg_off, *seg_adapter;
  int64_t M;
  int R, L, S, CS;  // CS: CTAs per cluster, 1, 2, 4 or 8
  DropArgs drop;  // on dA's X
  bool check;     // bad segments are recorded here
};

constexpr int kWgRows = 64;      // rows per step
constexpr int kWgRun = 4;        // steps of a run: 16 instructions
constexpr int kWgGroups = 4;     // worker warps per TMEM lane quadrant
constexpr int kWgWorkers = 4 * kWgGroups;
constexpr int kWgThreads = 32 * (2 + kWgWorkers);

template <int RP> struct WgradGeom {
  static constexpr int MB = (RP == 64) ? 2 : 1;          // MMAs of 128 columns (tensor memory holds the parts of both)
  static constexpr int CT = 128 * MB;                    // columns per cluster
  static constexpr int X_BYTES = kWgRows * CT * 2;
  static constexpr int PB = 3 * RP / 64;                 // 64-wide blocks of P's parts
  static constexpr int P_BYTES = PB * kWgRows * 128;
  static constexpr int XS = 4, PS = 2;                   // stages
  static constexpr int RING = XS * X_BYTES + PS * P_BYTES;
  static constexpr int RECV = CT * RP * 4;
  static_assert(RECV <= RING, "the sums' buffer lies over the ring");
  static constexpr int PPT = kWgRows * RP / 4 / (32 * kWgWorkers);  // quads of P per worker and step
  static constexpr int wait_off = RING;                  // two steps' quads on their way, each worker its own
  static constexpr int WAIT_STAGE = PPT * 32 * kWgWorkers * 16;
  static constexpr int bar_off = RING + 2 * WAIT_STAGE;
  static constexpr int nbar = 2 * XS + 2 * PS + 2;
  static constexpr int max_off = bar_off + 8 * nbar;     // largest |P| (fp16), as bits
  static constexpr int tmem_off = max_off + 4;
  static constexpr int abort_off = tmem_off + 4;
  static constexpr int total = abort_off + 4 + 1024;
  static constexpr int TM_COLS = 512;                    // MB x (first, 2 lower, first) x RP columns
  static constexpr int D_COLS = 4 * RP;
  static_assert(MB * D_COLS <= TM_COLS, "tensor memory");
  static constexpr int SUMS = MB * RP / 16 / kWgGroups;  // groups of 16 ranks whose sums a worker warp keeps
};

// The 64-row tiles of one adapter, in order: every warp walks all of them and
// takes those whose number is its CTA's rank modulo the cluster's size.
struct WgradRows {
  int s0;            // first segment not looked at
  unsigned mask;     // segments of the last 32 that are left
  int start, len;    // this lane's segment
  int cur, cur_len;  // segment being cut: next row, rows left
  int count;         // tiles passed
  int row0, rows;    // the tile found
};

BQ_DEV bool wgrad_next(WgradRows &w, const WgradArgs &a, int adapter, int rank) {
  const int lane = threadIdx.x & 31;
  while (true) {
    while (w.cur_len <= 0) {
      while (!w.mask) {
        if (w.s0 >= a.S) return false;
        const int s = w.s0 + lane;
        bool hit = false;
        w.len = 0;
        if (s < a.S && __ldcg(a.seg_adapter + s) == adapter) {
          w.len = lora_segment(a.seg_off, s, a.M, &w.start);
          hit = w.len > 0;
        }
        w.mask = __ballot_sync(0xffffffffu, hit);
        w.s0 += 32;
      }
      const int src = __ffs(w.mask) - 1;
      w.mask &= w.mask - 1;
      w.cur = __shfl_sync(0xffffffffu, w.start, src);
      w.cur_len = __shfl_sync(0xffffffffu, w.len, src);
    }
    // tiles count .. count + n - 1 are this segment's; skip to this CTA's
    const int skip = (rank - w.count) & (a.CS - 1);
    const int n = (w.cur_len + kWgRows - 1) / kWgRows;
    if (skip >= n) {
      w.count += n;
      w.cur_len = 0;
      continue;
    }
    w.row0 = w.cur + skip * kWgRows;
    w.rows = min(kWgRows, w.cur_len - skip * kWgRows);
    w.count += skip + 1;
    w.cur += (skip + 1) * kWgRows;
    w.cur_len -= (skip + 1) * kWgRows;
    return true;
  }
}

struct WgradBars {
  uint32_t full, freed, ready, p_free, d_full, done;
  BQ_DEV WgradBars(uint32_t base, int xs, int ps) {
    full = base;                 // [XS] X has landed
    freed = full + 8u * xs;      // [XS] its MMAs are done
    ready = freed + 8u * xs;     // [PS] P is stored (and X patched)
    p_free = ready + 8u * ps;    // [PS] its MMAs are done
    d_full = p_free + 8u * ps;
    done = d_full + 8u;
  }
};

// P's quad v as parts at (row m, rank r) of a stage; the first part's ranks from
// column first_at on, the others' from low_at.
template <int XT>
BQ_DEV void wgrad_store_p(uint32_t stage, int m, int r, int r16, int first_at, int low_at, float4 v) {
  uint2 part[3];
  if (XT == 1) {
    float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      part[p].x = pack_bf16(f[0], f[1]);
      part[p].y = pack_bf16(f[2], f[3]);
      f[0] -= __uint_as_float(part[p].x << 16);
      f[1] -= __uint_as_float(part[p].x & 0xffff0000u);
      f[2] -= __uint_as_float(part[p].y << 16);
      f[3] -= __uint_as_float(part[p].y & 0xffff0000u);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!(fabsf(f[i]) <= 3.402823466e38f)) f[i] = 0.0f;  // infinite or NaN: the first part says it
    }
  } else {
    tc_split<0>(v.x, v.y, part[0].x, part[1].x);
    tc_split<0>(v.z, v.w, part[0].y, part[1].y);
  }
#pragma unroll
  for (int p = 0; p < (XT == 1 ? 3 : 2); ++p) {
    const int n = r + (p == 0 ? first_at : low_at + (p - 1) * r16);
    const uint32_t at = stage + (n >> 6) * (kWgRows * 128) + m * 128 + ((((n & 63) >> 3) ^ (m & 7)) << 4) + (n & 7) * 2;
    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at), "r"(part[p].x), "r"(part[p].y) : "memory");
  }
}

// grid = CS x (L x (dA tiles + dB tiles)), cluster = (CS, 1, 1); mx: x [M, K],
// mdy: dy [M, N], boxes of 64 columns x 64 rows.
template <int XT, int RP>
__global__ void __launch_bounds__(kWgThreads, 1)
lora_wgrad_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mdy, const WgradArgs a) {
  using G = WgradGeom<RP>;
  constexpr int XS = G::XS, PS = G::PS, PARTS = XT == 1 ? 3 : 2, CT = G::CT, MB = G::MB;
  extern __shared__ __align__(1024) unsigned char tsm_raw[];
  const uint32_t raw = smem_u32(tsm_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  unsigned char *smem = tsm_raw + (sbase - raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int CS = a.CS, rank = (int)blockIdx.x % CS, work = (int)blockIdx.x / CS;
  const int per_adapter = a.dA.tiles + a.dB.tiles, adapter = work / per_adapter;
  const bool is_b = work % per_adapter >= a.dA.tiles;
  const WgradSide side = is_b ? a.dB : a.dA;
  const CUtensorMap *map = is_b ? &mdy : &mx;
  const int c0 = (work % per_adapter - (is_b ? a.dA.tiles : 0)) * CT;
  const int r_a = lora_rank(a.ranks, adapter, a.L, a.R), r16 = (r_a + 15) & ~15;
  const int nfull = PARTS * r16, n0 = nfull < 192 ? nfull : 192, n1 = nfull - n0;  // columns of the two MMAs
  const int cblocks = min(2 * MB, (side.C - c0 + 63) / 64);  // 64-column blocks in use
  const bool masked = !is_b && a.drop.thr != 0;
  volatile int *abort = reinterpret_cast<volatile int *>(smem + G::abort_off);
  const WgradBars B(sbase + G::bar_off, XS, PS);

  if (threadIdx.x == 0) {
    for (int i = 0; i < XS; ++i) {
      mbar_init(B.full + 8u * i, 1);
      mbar_init(B.freed + 8u * i, 1);
    }
    for (int i = 0; i < PS; ++i) {
      mbar_init(B.ready + 8u * i, kWgWorkers);
      mbar_init(B.p_free + 8u * i, 1);
    }
    mbar_init(B.d_full, 1);
    mbar_init(B.done, 1);
    *abort = 0;
    *reinterpret_cast<volatile uint32_t *>(smem + G::max_off) = 0u;
    mbar_fence_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + G::tmem_off),
                 "n"(G::TM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0 && a.S > 0) prefetch_map(map);
  if (a.check && blockIdx.x == 0 && warp == 2) lora_check_segments(a.seg_off, a.seg_adapter, a.ranks, a.S, a.L, a.R, a.M);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + G::tmem_off);

  WgradRows w = {};
  int steps = 0;  // tiles taken
  float2 pscale = make_float2(1.0f, 1.0f);
  // worker warps: which 128 columns and ranks 16 (cg0 + CG k) onwards a warp's sums are of
  constexpr int CG = kWgGroups / MB;
  const int quad = warp & 3, grp = (warp - 2) >> 2, mb = MB == 2 ? grp & 1 : 0, cg0 = grp / MB;
  const uint32_t lane_tmem = tmem + ((uint32_t)(quad * 32) << 16) + mb * G::D_COLS;
  float psum[G::SUMS][16];
#pragma unroll
  for (int k = 0; k < G::SUMS; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) psum[k][i] = 0.0f;
  if (r_a == 0) {
    // no rank: nothing to sum
  } else if (warp == 0) {
    while (wgrad_next(w, a, adapter, rank)) {
      const int slot = steps % XS;
      bool ok = true;
      if (steps >= XS) ok = __all_sync(0xffffffffu, !*abort && mbar_wait(B.freed + 8u * slot, ((steps / XS) & 1) ^ 1)) != 0;
      if (!ok) {
        if (lane == 0) {
          if (!*abort) bq_flag(BQ_FLAG_TIMEOUT);
          *abort = 1;
        }
        break;
      }
      if (lane == 0) {
        const uint32_t xs = sbase + slot * G::X_BYTES, full = B.full + 8u * slot;
        mbar_arrive_expect_tx(full, cblocks * (kWgRows * 128));
#pragma unroll
        for (int b = 0; b < 2 * MB; ++b)
          if (b < cblocks) tma_load_2d(xs + b * (kWgRows * 128), map, c0 + 64 * b, w.row0, full);
      }
      __syncwarp();
      ++steps;
    }
    // every copy has landed before the ring is used for the sums
    for (int j = 1; j <= XS && j <= steps; ++j)
      mbar_wait(B.full + 8u * ((steps - j) % XS), ((steps - j) / XS) & 1, 1u << 20);
  } else if (warp == 1) {
    bool ok = true;
    const uint64_t xd0 = tc_desc(sbase, kWgRows * 128), pd0 = tc_desc(sbase + XS * G::X_BYTES, kWgRows * 128);
    const uint32_t id0 = tc_idesc<XT>(n0, true, true), id1 = tc_idesc<XT>(n1 > 0 ? n1 : 16, true, true);
    while (wgrad_next(w, a, adapter, rank)) {
      const int slot = steps % XS, ps = steps % PS;
      ok = __all_sync(0xffffffffu, !*abort && mbar_wait(B.full + 8u * slot, (steps / XS) & 1) &&
                                       mbar_wait(B.ready + 8u * ps, (steps / PS) & 1)) != 0;
      if (!ok) break;
      if (lane == 0) {
        tc_fence_after();
        const uint64_t xd = xd0 + (uint64_t)(slot * (G::X_BYTES >> 4)), pd = pd0 + (uint64_t)(ps * (G::P_BYTES >> 4));
        const int ks = (w.rows + 15) / 16;
        // the run's place holds zeros: every worker has added its last run and
        // cleared it before it stored P of a step that came before this one
        const uint32_t d = tmem + ((steps / kWgRun) & 1) * r16;
#pragma unroll
        for (int k = 0; k < kWgRows / 16; ++k) {
          if (k >= ks) break;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            if (2 * mb >= cblocks) break;
            tc_mma(d + mb * G::D_COLS, xd + 2 * mb * (kWgRows * 128 >> 4) + 128 * k, pd + 128 * k, id0, steps > 0 || k > 0);
            if (MB == 1 && n1 > 0)
              tc_mma(d + n0, xd + 128 * k, pd + 3 * (kWgRows * 128 >> 4) + 128 * k, id1, steps > 0 || k > 0);
          }
        }
        umma_commit(B.freed + 8u * slot);
        umma_commit(B.p_free + 8u * ps);
      }
      __syncwarp();
      ++steps;
    }
    if (lane == 0) {
      if (ok) umma_commit(B.d_full);
      else {
        if (!*abort) bq_flag(BQ_FLAG_TIMEOUT);
        *abort = 1;
      }
    }
    __syncwarp();
  } else {
    const int wt = (int)threadIdx.x - 64;
    const DropState dst = masked ? drop_state(a.drop) : DropState{};
    bool ok = true;
    auto first_col = [&](int place) { return lane_tmem + place * PARTS * r16; };
    // the first run's instructions start with zeros by themselves, the second's place is cleared here
#pragma unroll
    for (int k = 0; k < G::SUMS; ++k)
      if (cg0 + CG * k < r16 / 16) tmem_zero16(first_col(1) + (cg0 + CG * k) * 16);
    tmem_wait_st();
    tc_fence_before();
    if (!is_b) pdl_wait();  // dt is complete; all else was before the kernel that makes it began
    if (XT == 0) {  // the power of two that brings the largest |P| of these rows below fp16's range
      WgradRows v = {};
      float mx = 0.0f;
      while (wgrad_next(v, a, adapter, rank)) {
        float4 pv[G::PPT];
#pragma unroll
        for (int k = 0; k < G::PPT; ++k) {
          const int i = wt + k * 32 * kWgWorkers, m = i / (RP / 4), r = 4 * (i % (RP / 4));
          pv[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (m < v.rows && r < r_a) pv[k] = __ldcg(reinterpret_cast<const float4 *>(side.P + (int64_t)(v.row0 + m) * a.R + r));
        }
#pragma unroll
        for (int k = 0; k < G::PPT; ++k) {
          const int r = 4 * ((wt + k * 32 * kWgWorkers) % (RP / 4));
          const float q[4] = {fabsf(pv[k].x), fabsf(pv[k].y), fabsf(pv[k].z), fabsf(pv[k].w)};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (q[i] <= 3.402823466e38f && r + i < r_a) mx = fmaxf(mx, q[i]);  // infinite and NaN stay what they are
        }
      }
      mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
      if (lane == 0) atomicMax(reinterpret_cast<unsigned *>(smem + G::max_off), __float_as_uint(mx));
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kWgWorkers) : "memory");
      pscale = tc_scale(__uint_as_float(*reinterpret_cast<volatile uint32_t *>(smem + G::max_off)));
    }
    // P is read two steps ahead (one step is shorter than the way to L2 and back),
    // through shared memory that only this worker uses (in registers beside the sums:
    // dt and both gradients of 8192 rows of 4 adapters, rank 64, 174 us, so 138)
    const uint32_t mine = sbase + G::wait_off + wt * 16;
    int row0[2], rows[2];
    auto fetch = [&](int b) {
      rows[b] = 0;
      if (wgrad_next(w, a, adapter, rank)) {
        row0[b] = w.row0;
        rows[b] = w.rows;
#pragma unroll
        for (int k = 0; k < G::PPT; ++k) {
          const int i = wt + k * 32 * kWgWorkers, m = i / (RP / 4), r = 4 * (i % (RP / 4));
          if (m < w.rows && r < r_a)
            cp_async16(mine + b * G::WAIT_STAGE + k * (32 * kWgWorkers * 16), side.P + (int64_t)(w.row0 + m) * a.R + r);
        }
      }
      cp_async_commit();
    };
    int run = 0;  // runs added to psum
    auto add_run = [&](bool clear) {
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < G::SUMS; ++k) {
        const int cgp = cg0 + CG * k;
        if (cgp < r16 / 16) {
          float v[16];
          tmem_ld16(first_col(run & 1) + cgp * 16, v);
          if (clear) tmem_zero16(first_col(run & 1) + cgp * 16);
#pragma unroll
          for (int i = 0; i < 16; ++i) psum[k][i] += v[i];
        }
      }
      if (clear) tmem_wait_st();
      tc_fence_before();
      ++run;
    };
    auto step = [&](int b) {
      const int slot = steps % XS, first = row0[b], n = rows[b];
      const bool odd = (steps / kWgRun) & 1;
      const uint32_t xb = sbase + slot * G::X_BYTES, pb = sbase + XS * G::X_BYTES + b * G::P_BYTES;
      if (steps >= PS) ok = __all_sync(0xffffffffu, !*abort && mbar_wait(B.p_free + 8u * b, ((steps / PS) & 1) ^ 1)) != 0;
      if (!ok) return;
      // the wait above was for the last step of the run before this one
      if (b == 1 && steps % kWgRun == 1 && steps > kWgRun) add_run(true);
      cp_async_wait<1>();
#pragma unroll
      for (int k = 0; k < G::PPT; ++k) {
        const int i = wt + k * 32 * kWgWorkers, m = i / (RP / 4), r = 4 * (i % (RP / 4));
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (m < n && r < r_a) {
          const uint4 q = lds_v4(mine + b * G::WAIT_STAGE + k * (32 * kWgWorkers * 16));
          v.x = __uint_as_float(q.x);  // what lies behind the rank may be anything
          if (r + 1 < r_a) v.y = __uint_as_float(q.y);
          if (r + 2 < r_a) v.z = __uint_as_float(q.z);
          if (r + 3 < r_a) v.w = __uint_as_float(q.w);
        }
        if (XT == 0) v = make_float4(v.x * pscale.y, v.y * pscale.y, v.z * pscale.y, v.w * pscale.y);
        if (r < r16) wgrad_store_p<XT>(pb, m, r, r16, odd ? (PARTS - 1) * r16 : 0, odd ? 0 : r16, v);
      }
      fetch(b);
      if (masked || (n & 15)) {
        constexpr int PT = 2 * MB * kWgRows * 8 / (32 * kWgWorkers);  // 16-byte chunks per worker
        ok = __all_sync(0xffffffffu, mbar_wait(B.full + 8u * slot, (steps / XS) & 1)) != 0;
        if (!ok) return;
#pragma unroll 2
        for (int k = 0; k < PT; ++k) {
          const int i = wt + k * 32 * kWgWorkers, m = (i >> 3) % kWgRows, cb = i / (8 * kWgRows);
          const uint32_t at = xb + cb * (kWgRows * 128) + m * 128 + (((i & 7) ^ (m & 7)) << 4);
          if (cb >= cblocks) continue;
          if (m >= n) {
            sts_v4(at, make_uint4(0, 0, 0, 0));  // another segment's row
          } else if (masked) {
            const uint4 q = drop_block(dst, (uint32_t)(c0 >> 3) + 8 * cb + (i & 7), (uint32_t)(first + m));
            sts_v4(at, and4(lds_v4(at), drop_mask8(q, dst.thr_hi)));
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(B.ready + 8u * b);
      ++steps;
    };
    static_assert(PS == 2, "a buffer for each stage of P; step s waits for step s - 2");
    fetch(0);
    fetch(1);
    while (ok && rows[0] > 0) {
      step(0);
      if (!ok || rows[1] <= 0) break;
      step(1);
    }
    cp_async_wait<0>();  // no copy is on its way when the CTA leaves
    if (ok) ok = __all_sync(0xffffffffu, !*abort && mbar_wait(B.d_full, 0)) != 0;
    if (ok)
      while (run < (steps + kWgRun - 1) / kWgRun) add_run(false);
    if (!ok && lane == 0) {
      if (!*abort) bq_flag(BQ_FLAG_TIMEOUT);
      *abort = 1;
    }
  }

  // ---- the sums meet: every CTA's ring is idle, it holds the sums now --------
  pdl_wait();  // no CTA leaves before the kernel that makes dt is complete
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if (*abort && lane == 0) {
      umma_commit(B.done);
      mbar_wait(B.done, 0, 1u << 20);
    }
    __syncwarp();
  }
  cluster_arrive();
  cluster_wait();
  float *recv = reinterpret_cast<float *>(smem);
  const int per_r = r16 / CS, own = CT / CS;  // ranks of dA / columns of dB that one CTA owns
  if (warp >= 2 && r_a > 0) {
    // the warps of a quadrant share its blocks of 128 columns and the ranks
    const int c = mb * 128 + quad * 32 + lane;
#pragma unroll
    for (int k = 0; k < G::SUMS; ++k) {
      const int cgp = cg0 + CG * k;
      if (cgp >= r16 / 16) break;
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
      if (steps > 0) {
#pragma unroll
        for (int p = PARTS - 1; p > 0; --p) {  // the smallest part first
          float q[16];
          tmem_ld16(lane_tmem + p * r16 + cgp * 16, q);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += q[i];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)  // an infinity times a lower part that is 0 or of the other sign would give NaN
          v[i] = fabsf(psum[k][i]) <= 3.402823466e38f ? v[i] + psum[k][i] : psum[k][i];
      }
      if (XT == 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= pscale.x;
      }
      if (!is_b) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = cgp * 16 + i;
          cluster.map_shared_rank(recv, r / per_r)[(rank * per_r + r % per_r) * CT + c] = v[i];
        }
      } else {
        float *to = cluster.map_shared_rank(recv, c / own) + (rank * own + c % own) * RP;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<float4 *>(to + 4 * ((cgp * 4 + q) ^ (c & 7))) =
              make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      }
    }
  }
  tc_fence_before();
  cluster_arrive();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(G::TM_COLS) : "memory");
  }
  const float scale = is_b ? (r_a > 0 ? a.scales[adapter] : 0.0f) : (masked ? a.drop.inv_keep : 1.0f);
  auto finish = [&](float4 v) {  // an unused adapter's gradient is 0 whatever its scale
    return make_float4(v.x != 0.0f ? v.x * scale : 0.0f, v.y != 0.0f ? v.y * scale : 0.0f,
                       v.z != 0.0f ? v.z * scale : 0.0f, v.w != 0.0f ? v.w * scale : 0.0f);
  };
  if (!is_b) {
    // this CTA's ranks (and, behind r16, every CS-th zero row)
    const int zero_rows = a.R > r16 ? (a.R - r16 - rank + CS - 1) / CS : 0;
    for (int i = threadIdx.x; i < (per_r + zero_rows) * (CT / 4); i += kWgThreads) {
      const int rl = i / (CT / 4), c = 4 * (i % (CT / 4));
      const int r = rl < per_r ? rank * per_r + rl : r16 + rank + (rl - per_r) * CS;
      if (r >= a.R || c0 + c >= side.C) continue;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (r < r_a) {
        for (int q = 0; q < CS; ++q) {
          const float4 p = *reinterpret_cast<const float4 *>(recv + (q * per_r + rl) * CT + c);
          v.x += p.x;
          v.y += p.y;
          v.z += p.z;
          v.w += p.w;
        }
        v = finish(v);
      }
      *reinterpret_cast<float4 *>(side.out + ((int64_t)adapter * a.R + r) * side.C + c0 + c) = v;
    }
  } else {
    const int quads = a.R / 4;
    for (int i = threadIdx.x; i < own * quads; i += kWgThreads) {
      const int cl = i / quads, chunk = i % quads, c = c0 + rank * own + cl;
      if (c >= side.C) continue;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (4 * chunk < r_a) {
        for (int q = 0; q < CS; ++q) {
          const float4 p = *reinterpret_cast<const float4 *>(recv + (q * own + cl) * RP + 4 * (chunk ^ (cl & 7)));
          v.x += p.x;
          v.y += p.y;
          v.z += p.z;
          v.w += p.w;
        }
        v = finish(v);
        if (4 * chunk + 1 >= r_a) v.y = 0.0f;
        if (4 * chunk + 2 >= r_a) v.z = 0.0f;
        if (4 * chunk + 3 >= r_a) v.w = 0.0f;
      }
      *reinterpret_cast<float4 *>(side.out + ((int64_t)adapter * side.C + c) * a.R + 4 * chunk) = v;
    }
  }
}

}  // namespace bq

// dropout.cuh -- dropout from a counter-based generator, no mask stored:
//   y[i, j] = keep(i, j) ? x[i, j] / (1 - p) : 0
// The forward pass and the gradient are the same map (dx = mask dy / (1 - p)),
// so the mask is drawn again from its counter instead of being kept.
//
// Generator: Philox 4x32 with 10 rounds (J. Salmon, M. Moraes, R. Dror, D.
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011), key = seed,
// counter = (j / 8, i, offset low, offset high).  One block of 128 bits
// serves 8 consecutive columns of a row: element j takes the 16-bit field
// j % 8, and is kept where the field is at least thr = round(p 65536), so the
// probability is a multiple of 2^-16 and 1 / (1 - p) uses the same rounded p.
// 16 bits an element halve the generator's instructions against 32.
#pragma once
#include "common.cuh"

namespace bq {

// What a kernel needs to draw masks: thr = 0 keeps everything.
struct DropArgs {
  const unsigned long long *rng;  // DEVICE {seed, offset}
  uint32_t thr;                   // round(p 65536), at most 65535
  float inv_keep;                 // 65536 / (65536 - thr)
};

struct DropState {
  uint2 key;
  uint32_t c2, c3;   // offset
  uint32_t thr_hi;   // thr in the upper half-word
};

BQ_DEV DropState drop_state(const DropArgs &d) {
  DropState s = {};
  if (d.thr) {
    const unsigned long long seed = d.rng[0], off = d.rng[1];
    s.key = make_uint2((uint32_t)seed, (uint32_t)(seed >> 32));
    s.c2 = (uint32_t)off;
    s.c3 = (uint32_t)(off >> 32);
    s.thr_hi = d.thr << 16;
  }
  return s;
}

BQ_DEV uint4 philox4x32_10(uint4 c, uint2 k) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    // one wide product each (the low and the high half apart are two)
    const unsigned long long p0 = (unsigned long long)0xD2511F53u * c.x, p1 = (unsigned long long)0xCD9E8D57u * c.z;
    c = make_uint4((uint32_t)(p1 >> 32) ^ c.y ^ k.x, (uint32_t)p1, (uint32_t)(p0 >> 32) ^ c.w ^ k.y, (uint32_t)p0);
    k.x += 0x9E3779B9u;
    k.y += 0xBB67AE85u;
  }
  return c;
}

// The generator block of columns 8 blk .. 8 blk + 7 of a row.
BQ_DEV uint4 drop_block(const DropState &s, uint32_t blk, uint32_t row) {
  return philox4x32_10(make_uint4(blk, row, s.c2, s.c3), s.key);
}

// Kept halves of one 32-bit word of the block as a mask of 0xffff fields.
BQ_DEV uint32_t drop_mask2(uint32_t w, uint32_t thr_hi) {
  const uint32_t lo = ((w << 16) >= thr_hi) ? 0x0000ffffu : 0u;
  const uint32_t hi = (w >= thr_hi) ? 0xffff0000u : 0u;
  return lo | hi;
}
BQ_DEV uint4 drop_mask8(uint4 b, uint32_t thr_hi) {
  return make_uint4(drop_mask2(b.x, thr_hi), drop_mask2(b.y, thr_hi), drop_mask2(b.z, thr_hi),
                    drop_mask2(b.w, thr_hi));
}

// Element i (0..7) of the block is kept.
BQ_DEV bool drop_keep(const uint4 &b, int i, uint32_t thr_hi) {
  const uint32_t w = (i >> 1) == 0 ? b.x : (i >> 1) == 1 ? b.y : (i >> 1) == 2 ? b.z : b.w;
  return (i & 1) ? (w >= thr_hi) : ((w << 16) >= thr_hi);
}

// Two floats rounded to a pair of fp16 (XT = 0) or bf16.
template <int XT> BQ_DEV uint32_t pack_pair(float2 v) {
  uint32_t r;
  if (XT == 1) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
  return r;
}

template <int DT> struct DropElem { using T = uint16_t; };  // fp16, bf16
template <> struct DropElem<2> { using T = float; };

// One thread takes blocks of 8 columns, grid-stride over rows x blocks, kUnroll
// loads in flight.  VEC: both matrices have 16-byte aligned rows, whole blocks
// move as 16-byte vectors (the last block of a ragged row element by element).
// fp32 runs at the rate of a copy; 16-bit types are bound by the generator's
// instructions, so places advance by additions and pairs are scaled, rounded
// and masked together (8192 x 14336 bf16, p = 0.05: 110 -> 89 us; p = 0 73 us).
template <int DT, bool VEC>
__global__ void __launch_bounds__(256, 5)
dropout_kernel(const typename DropElem<DT>::T *x, uint32_t rows, int64_t cols, int64_t ldx,
               typename DropElem<DT>::T *out, int64_t ldo, DropArgs d) {
  using T = typename DropElem<DT>::T;
  constexpr int kVecs = (int)(8 * sizeof(T) / 16);
  constexpr int kUnroll = 2;
  const DropState st = drop_state(d);
  const uint32_t blocks = (uint32_t)((cols + 7) / 8);
  const bool ragged = (cols & 7) != 0;
  const int64_t step = (int64_t)gridDim.x * blockDim.x, first = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  // row, block and both places advance with the index
  const uint32_t drow = (uint32_t)(step / blocks), dblk = (uint32_t)(step - (int64_t)drow * blocks);
  const int64_t dx = drow * ldx + 8 * (int64_t)dblk, dout = drow * ldo + 8 * (int64_t)dblk;
  const int64_t wrap_x = ldx - 8 * (int64_t)blocks, wrap_o = ldo - 8 * (int64_t)blocks;
  int64_t row64 = first / blocks;
  if (row64 >= rows) return;
  uint32_t row = (uint32_t)row64, blk = (uint32_t)(first - row64 * blocks);
  const T *src = x + row * ldx + 8 * (int64_t)blk;
  T *dst = out + row * ldo + 8 * (int64_t)blk;
  while (row < rows) {
    uint32_t r[kUnroll], b[kUnroll];
    T *to[kUnroll];
    bool act[kUnroll], full[kUnroll];
    union {
      T e[8];
      uint4 v[kVecs];
    } buf[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      r[u] = row;
      b[u] = blk;
      to[u] = dst;
      act[u] = row < rows;
      full[u] = VEC && !(ragged && blk == blocks - 1);
      if (act[u]) {
        if (full[u]) {
#pragma unroll
          for (int k = 0; k < kVecs; ++k) buf[u].v[k] = reinterpret_cast<const uint4 *>(src)[k];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (8 * (int64_t)blk + i < cols) buf[u].e[i] = src[i];
        }
      }
      row += drow;
      blk += dblk;
      src += dx;
      dst += dout;
      if (blk >= blocks) {
        blk -= blocks;
        ++row;
        src += wrap_x;
        dst += wrap_o;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!act[u]) continue;
      if (d.thr) {
        const uint4 g = drop_block(st, b[u], r[u]);
        if constexpr (sizeof(T) == 2) {  // pairs: scaled and rounded together, then masked
          const uint4 k = drop_mask8(g, st.thr_hi);
          const float2 f = make_float2(d.inv_keep, d.inv_keep);
          uint4 v = buf[u].v[0];
          v.x = pack_pair<DT>(__fmul2_rn(Elem<DT>::pair(v.x), f)) & k.x;
          v.y = pack_pair<DT>(__fmul2_rn(Elem<DT>::pair(v.y), f)) & k.y;
          v.z = pack_pair<DT>(__fmul2_rn(Elem<DT>::pair(v.z), f)) & k.z;
          v.w = pack_pair<DT>(__fmul2_rn(Elem<DT>::pair(v.w), f)) & k.w;
          buf[u].v[0] = v;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) buf[u].e[i] = drop_keep(g, i, st.thr_hi) ? buf[u].e[i] * d.inv_keep : T(0);
        }
      }
      if (full[u]) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) reinterpret_cast<uint4 *>(to[u])[k] = buf[u].v[k];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * (int64_t)b[u] + i < cols) to[u][i] = buf[u].e[i];
      }
    }
  }
}

}  // namespace bq

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
    const uint32_t h0 = __umulhi(0xD2511F53u, c.x), l0 = 0xD2511F53u * c.x;
    const uint32_t h1 = __umulhi(0xCD9E8D57u, c.z), l1 = 0xCD9E8D57u * c.z;
    c = make_uint4(h1 ^ c.y ^ k.x, l1, h0 ^ c.w ^ k.y, l0);
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

template <int DT> struct DropElem {  // fp16, bf16
  using T = uint16_t;
  static BQ_DEV float load(T v) { return Elem<DT>::lo(v); }
  static BQ_DEV T store(float v) { return Elem<DT>::from_float(v); }
};
template <> struct DropElem<2> {  // fp32
  using T = float;
  static BQ_DEV float load(T v) { return v; }
  static BQ_DEV T store(float v) { return v; }
};

// One thread takes blocks of 8 columns, grid-stride over rows x blocks, kUnroll
// loads in flight.  VEC: both matrices have 16-byte aligned rows, whole blocks
// move as 16-byte vectors (the last block of a ragged row element by element).
template <int DT, bool VEC>
__global__ void __launch_bounds__(256)
dropout_kernel(const typename DropElem<DT>::T *x, int64_t rows, int64_t cols, int64_t ldx,
               typename DropElem<DT>::T *out, int64_t ldo, DropArgs d) {
  using E = DropElem<DT>;
  using T = typename E::T;
  constexpr int kVecs = (int)(8 * sizeof(T) / 16);
  constexpr int kUnroll = 2;
  const DropState st = drop_state(d);
  const int64_t blocks = (cols + 7) / 8, total = rows * blocks;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  int64_t idx = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  // (row, blk) advance with the index without a division a step
  const int64_t drow = step / blocks, dblk = step - drow * blocks;
  int64_t row = idx / blocks, blk = idx - row * blocks;
  while (idx < total) {
    int64_t r[kUnroll], b[kUnroll];
    bool act[kUnroll], full[kUnroll];
    union {
      T e[8];
      uint4 v[kVecs];
    } buf[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      act[u] = idx < total;
      r[u] = row;
      b[u] = blk;
      full[u] = VEC && (8 * blk + 8 <= cols);
      if (act[u]) {
        const T *src = x + row * ldx + 8 * blk;
        if (full[u]) {
#pragma unroll
          for (int k = 0; k < kVecs; ++k) buf[u].v[k] = reinterpret_cast<const uint4 *>(src)[k];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (8 * blk + i < cols) buf[u].e[i] = src[i];
        }
      }
      idx += step;
      row += drow;
      blk += dblk;
      if (blk >= blocks) {
        blk -= blocks;
        ++row;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!act[u]) continue;
      if (d.thr) {
        const uint4 g = drop_block(st, (uint32_t)b[u], (uint32_t)r[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          buf[u].e[i] = drop_keep(g, i, st.thr_hi) ? E::store(E::load(buf[u].e[i]) * d.inv_keep) : T(0);
      }
      T *dst = out + r[u] * ldo + 8 * b[u];
      if (full[u]) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) reinterpret_cast<uint4 *>(dst)[k] = buf[u].v[k];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * b[u] + i < cols) dst[i] = buf[u].e[i];
      }
    }
  }
}

}  // namespace bq

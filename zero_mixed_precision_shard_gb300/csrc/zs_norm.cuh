// sm_103a kernels of the root-mean-square norm and its gradients.
//
// Both move a few bytes per element for 6-10 flops: HBM is the bound, so each
// array is touched once.  A row stays in registers between its sum of squares
// (or its dot product) and its output: T threads (a multiple of 32) hold U
// units of 8 elements each, chosen by the row's length (norm_form); rows of one
// warp share a CTA, eight or four at a time (blockDim = 32 x 8, 32 x 4 with more
// than two units, otherwise T x 1).
// MAXT, the most threads of a form, bounds its registers.  The grid is what the
// GPU holds at once; the rows ahead are on their way into a ring in shared
// memory (cp.async) while a row is worked on, so that the bytes in flight cost
// no registers.  A unit is a 16-byte line and a thread copies, reads and writes
// lines that are its own:
//   kLines   every row of every array starts on a line;
//   kShifted every array's row starts at the same place in its line.  That
//            place repeats every 8 rows whatever the stride, so a CTA takes
//            rows of one residue modulo 8: its columns, weights and sums of
//            dweight stay where they are.  A row's first and last line may
//            hold elements of other rows (or of a gap); they are masked, and
//            such a line is copied whole only where it lies within the array
//            (gradients of 30000 x 1023: 66 us, 194 element by element);
//   kSingle  anything else: a thread takes elements t, t + T, ... one by one,
//            without a ring.
// Rows past the largest form are read again instead of held.
#pragma once

#include "zs_tensors.cuh"

namespace zs {

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;
  const uint16_t* w;
  uint16_t* sum;
  void* out;
  float* scales;
  float* rstd;
  int64_t rows, x_stride, res_stride, sum_stride, out_stride;
  int32_t cols;
  int32_t group, group_log2, groups;
  float eps, inv_cols;
};

struct NormBwdArgs {
  const uint16_t* dy;
  const uint16_t* h;
  const uint16_t* dsum;
  const uint16_t* w;
  const float* rstd;
  uint16_t* dx;
  float* part;  // gridDim.x (or row slices) x cols partial sums of dweight; null: one cluster
  float* dot;   // rows values, rows past the largest register form only
  float* dweight;  // one cluster only, with `accumulate`
  int64_t rows, dy_stride, h_stride, dsum_stride, dx_stride;
  int32_t cols, accumulate;
  float inv_cols;
};

enum NormAccess { kLines, kShifted, kSingle };

// Output of the norm: halves, E4M3 with a scale a row, E4M3 with a scale a group.
enum NormOut { kOutHalf = 0, kOutRow = 1, kOutGroup = 2 };

constexpr int kNormUnits = 2;     // largest U of a row that several warps share
constexpr int kNormCols = 16384;  // longest row held in registers

// Rows of a ring: the one worked on and the one ahead.  (A third costs the norm
// of 8192 x 8192 8 us of 90 with the same threads: more rows in flight spread
// the DRAM accesses over more pages.)
constexpr int kNormStages = 2;

// What the threads of a row combine: `turn` alternates between two buffers,
// so one barrier a call is enough -- a thread that writes a buffer again has
// passed the barrier of the call in between, which every reader of the buffer
// has reached.
struct RowShare {
  float (&sm)[2][32];
  int turn = 0;
  // Sum over the row's threads, the same bits in each.
  __device__ __forceinline__ float sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, off));
    if (blockDim.x == 32) return x;
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    float* const b = sm[turn];
    if (lane == 0) b[threadIdx.x >> 5] = x;
    __syncthreads();
    x = lane < warps ? b[lane] : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, off));
    turn ^= 1;
    return x;
  }
  // Maximum of magnitudes given as fp32 bits (an inf or NaN is the largest).
  __device__ __forceinline__ uint32_t top(uint32_t x) {
    x = __reduce_max_sync(0xffffffffu, x);
    if (blockDim.x == 32) return x;
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    float* const b = sm[turn];
    if (lane == 0) b[threadIdx.x >> 5] = __uint_as_float(x);
    __syncthreads();
    x = __reduce_max_sync(0xffffffffu, lane < warps ? __float_as_uint(b[lane]) : 0u);
    turn ^= 1;
    return x;
  }
  // Everything the row's threads wrote to shared memory is seen by all of them.
  __device__ __forceinline__ void sync() const {
    if (blockDim.x == 32) __syncwarp();
    else __syncthreads();
  }
};

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The scale past which a row's sum of squares leaves fp32 (bf16 values from
// about 1e18): squares of the values times 2^-100 instead (below 2^56, so that
// 2^31 of them stay in fp32; eps is nothing beside them).  An inf or NaN in the
// row stays one.
constexpr float kNormShrink = 0x1p-100f;
__device__ __forceinline__ float norm_rstd_big(float sum, float inv_cols) {
  return __fmul_rn(rsqrtf(__fmul_rn(sum, inv_cols)), kNormShrink);
}

// Element of register i of unit k of this thread; `off`: the row's place in
// its line.  In the one-element form T is hidden from the optimiser: it would
// keep every element's offset in registers across the rows (128 to 255 of them).
template <int ACC>
__device__ __forceinline__ int norm_at(int k, int i, int off) {
  int t = blockDim.x;
  if constexpr (ACC == kLines) return (threadIdx.x + k * t) * 8 + i;
  if constexpr (ACC == kShifted) return (threadIdx.x + k * t) * 8 + i - off;
  asm volatile("" : "+r"(t));
  return threadIdx.x + (k * 8 + i) * t;
}

// Whether the line of unit k holds an element of the row, and nothing else: for
// shifted rows a bit per unit (norm_lines), looked up in the loop over the rows.
struct NormBits {
  uint32_t live, whole;
};
template <int ACC>
__device__ __forceinline__ bool norm_live(NormBits b, int k, int cols) {
  return ACC == kLines ? norm_at<ACC>(k, 0, 0) < cols : (b.live >> k & 1u) != 0;
}
template <int ACC>
__device__ __forceinline__ bool norm_whole(NormBits b, int k, int cols) {
  return ACC == kLines ? norm_at<ACC>(k, 0, 0) < cols : (b.whole >> k & 1u) != 0;
}
template <int U, int ACC>
__device__ __forceinline__ NormBits norm_lines(int off, int cols) {
  NormBits b{0u, 0u};
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int e = norm_at<ACC>(k, 0, off);
    b.live |= (uint32_t)(e > -8 && e < cols) << k;
    b.whole |= (uint32_t)(e >= 0 && e + 8 <= cols) << k;
  }
  return b;
}

// A unit straight from memory, zeros past the row's ends.
template <int DT, int ACC>
__device__ __forceinline__ void norm_load(const uint16_t* p, int k, int off, int cols,
                                          float (&a)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = norm_at<ACC>(k, i, off);
    a[i] = e >= 0 && e < cols ? half_bits_to_float<DT>(p[e]) : 0.0f;
  }
}

template <int DT, int ACC>
__device__ __forceinline__ void norm_store(uint16_t* p, int k, int off, int cols, NormBits bits,
                                           const float (&a)[8]) {
  if (ACC != kSingle && norm_whole<ACC>(bits, k, cols)) {
    *reinterpret_cast<uint4*>(p + norm_at<ACC>(k, 0, off)) = pack8<DT>(a);
  } else if (ACC == kSingle || (ACC == kShifted && norm_live<ACC>(bits, k, cols))) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = norm_at<ACC>(k, i, off);
      if (e >= 0 && e < cols) p[e] = (uint16_t)float_to_half_bits<DT>(a[i]);
    }
  }
}

// This thread's weights, two halves a word.
template <int U, int ACC>
__device__ __forceinline__ void norm_weights(const uint16_t* w, int off, int cols,
                                             uint32_t (&w2)[U][4]) {
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if constexpr (ACC == kLines) {
      const int e = norm_at<ACC>(k, 0, off);
      const uint4 q = e < cols ? *reinterpret_cast<const uint4*>(w + e) : make_uint4(0u, 0u, 0u, 0u);
      w2[k][0] = q.x; w2[k][1] = q.y; w2[k][2] = q.z; w2[k][3] = q.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e0 = norm_at<ACC>(k, 2 * i, off), e1 = norm_at<ACC>(k, 2 * i + 1, off);
        w2[k][i] = (e0 >= 0 && e0 < cols ? (uint32_t)w[e0] : 0u) |
                   ((e1 >= 0 && e1 < cols ? (uint32_t)w[e1] : 0u) << 16);
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ float norm_weight(const uint32_t (&w2)[4], int i) {
  return half_bits_to_float<DT>(i & 1 ? w2[i / 2] >> 16 : w2[i / 2] & 0xFFFFu);
}

// The rows of a thread: the first, and the step from one to the next.
template <int ACC>
struct NormRows {
  int64_t row, step;
  __device__ __forceinline__ NormRows() {
    step = (int64_t)gridDim.x * blockDim.y;
    if constexpr (ACC == kShifted)  // (the grid is a multiple of 8)
      row = (blockIdx.x & 7) + 8 * ((int64_t)(blockIdx.x >> 3) * blockDim.y + threadIdx.y);
    else
      row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  }
};

// The ring of a thread's lines of N arrays (a null array is not there),
// kStages rows deep: [slot][array][unit][thread of the CTA]; for shifted rows
// masks of the lines' own elements follow, [unit][thread].  Single elements have
// no ring: they are read when the row's turn comes.
template <int U, int ACC, int kStages, int N>
struct NormRing {
  const uint16_t* p[N];
  int64_t step[N];
  int cols, off, plane, slot_bytes;
  int64_t rows;
  NormBits bits = {0u, 0u};
  uint8_t* mine;

  __device__ __forceinline__ void init(uint8_t* smem, int cols_, int64_t rows_, int64_t first) {
    cols = cols_;
    rows = rows_;
    off = ACC == kShifted
              ? (int)(reinterpret_cast<uintptr_t>(p[0] + first * step[0]) & 15u) / 2 : 0;
    const int threads = blockDim.x * blockDim.y;
    int arrays = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) arrays += p[i] != nullptr;
    plane = threads * 16;
    slot_bytes = arrays * U * plane;
    mine = smem + (threadIdx.y * blockDim.x + threadIdx.x) * 16;
    if constexpr (ACC == kShifted) bits = norm_lines<U, ACC>(off, cols);
    if constexpr (ACC == kShifted) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int e = norm_at<ACC>(k, 0, off);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = (e + 2 * j >= 0 && e + 2 * j < cols ? 0x0000FFFFu : 0u) |
                 (e + 2 * j + 1 >= 0 && e + 2 * j + 1 < cols ? 0xFFFF0000u : 0u);
        *mask(k) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }

  __device__ __forceinline__ uint4* mask(int k) const {
    return reinterpret_cast<uint4*>(mine + kStages * slot_bytes + k * plane);
  }

  // (The warp's reads of the slot come before the copies into it.)
  __device__ __forceinline__ void fill(int slot, int64_t r) {
    if constexpr (ACC == kSingle) return;
    __syncwarp();
    if (r < rows) {
      uint8_t* const d = mine + slot * slot_bytes;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (p[i] == nullptr) continue;
        const uint16_t* const q = p[i] + r * step[i];
        // a line on a row's edge lies within the array unless the row is one
        // of the first or last
        const bool inner = r * step[i] >= 8 && (rows - 1 - r) * step[i] >= 8;
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int e = norm_at<ACC>(k, 0, off);
          uint8_t* const to = d + (i * U + k) * plane;
          if (ACC == kLines || inner ? norm_live<ACC>(bits, k, cols)
                                     : norm_whole<ACC>(bits, k, cols)) {
            // (as a number: the line's start may lie in front of the row)
            cp_async<16>(to, reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(q) +
                                                           2 * (intptr_t)e));
          } else if (ACC == kShifted && norm_live<ACC>(bits, k, cols)) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (e + j >= 0 && e + j < cols) reinterpret_cast<uint16_t*>(to)[j] = q[e + j];
          }
        }
      }
    }
    cp_async_commit();
  }

  __device__ __forceinline__ void arrive() const {
    if constexpr (ACC != kSingle) cp_async_wait<kStages - 1>();
  }

  // Unit k of array i of row r as it is stored, zeros past the row's ends.
  __device__ __forceinline__ uint4 raw(int slot, int i, int k) const {
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (norm_live<ACC>(bits, k, cols))
      q = *reinterpret_cast<const uint4*>(mine + slot * slot_bytes + (i * U + k) * plane);
    if (ACC == kShifted && !norm_whole<ACC>(bits, k, cols)) {
      const uint4 m = *mask(k);
      q.x &= m.x; q.y &= m.y; q.z &= m.z; q.w &= m.w;
    }
    return q;
  }

  template <int DT>
  __device__ __forceinline__ void take(int slot, int64_t r, int i, int k, float (&x)[8]) const {
    if constexpr (ACC == kSingle) norm_load<DT, ACC>(p[i] + r * step[i], k, 0, cols, x);
    else unpack8<DT>(raw(slot, i, k), x);
  }
};

// Threads an SM that the norm's grid aims at, and that its registers are given
// out for: more of them hide more latency, fewer spill less and keep the rows in
// flight together.  Each against a step fewer and a step more, us for 64 million
// bf16 elements with residual, 16 bits out (fewer / taken / more):
//   whole lines    1 unit, 256 columns: 84 / 85 / 90 with 768, 1,024 and 1,536
//                  2 units, 4,096: 93 / 80 / 84 with 256, 512 and 1,024
//                  3 units, 768: 83 / 87 / 92 with 512, 768 and 1,024 (79 / 75 / 79 to 8 bits)
//                  4 units, 1,024: 82 / 83 / 90 with 384, 512 and 768
//   shifted rows   1 unit, 250: 134 / 135 / 153 with 768, 1,024 and 1,536
//                  2 units, 2,047: 92 / 86 / 98 with 512, 768 and 1,024
//                  3 units, 763: 120 / 92 / 92 with 384, 512 and 768
//                  4 units, 1,001: 98 / 88 / 91 with 256, 384 and 512
//   elements       1 unit, 1,000: 294 / 190 / 164 with 512, 768 and 1,024
//                  2 units, 4,096: 448 / 248 / 186 with 256, 512 and 768
// (One unit of whole lines would be faster with fewer where several warps share a
// row, 1,280 columns 78 / 88 / 91, and single elements with more.)  The gradients:
//   1 unit         lines, 256: 79 / 88 / 132 with 768, 1,024 and 1,536;
//                  shifted, 250: 238 / 166 / 299 with 512, 768 and 1,024
//   2 units        4,096: 94 / 81 / 122 with 256, 512 and 768; 2,047: 236 / 124 / 197
//   3 and 4        768: 79 / 79 / 100 with 256, 384 and 512; 763: 136 / 116 / 298;
//                  1,024: 80 / 82 / 85; 1,001: 109 / 95 / 240
__host__ __device__ constexpr int norm_sm_threads(int u, int acc) {
  return acc == kLines     ? (u == 1 ? 1024 : u == 2 ? 512 : u == 3 ? 768 : 512)
         : acc == kShifted ? (u == 1 ? 1024 : u == 2 ? 768 : u == 3 ? 512 : 384)
                           : (u == 1 ? 768 : 512);
}
__host__ __device__ constexpr int norm_bwd_sm_threads(int u, int acc) {
  return u == 1 ? (acc == kShifted ? 768 : 1024) : u == 2 ? 512 : 384;
}

// (Shifted rows of up to 512 threads are held to 64 registers for two CTAs an SM:
// 4,095 columns 107 us, 126 with one.)
template <int DT, int U, int OUT, int ACC, int MAXT>
__global__ void
__launch_bounds__(MAXT, MAXT == 512 && ACC == kShifted ? 2
                        : MAXT <= 512                  ? norm_sm_threads(U, ACC) / MAXT
                                                       : 1)
    k_norm(const __grid_constant__ NormArgs a) {
  pdl_enter_last(a.x, a.res, a.w, a.sum, a.out, a.scales, a.rstd);
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ float sm[2][32];
  // maxima of 32-column segments, for groups of single elements
  __shared__ uint32_t seg[OUT == kOutGroup && ACC == kSingle ? U * MAXT / 4 : 1];
  RowShare row_share{sm};
  constexpr int kStages = kNormStages;
  const int cols = a.cols;
  NormRows<ACC> at;
  NormRing<U, ACC, kStages, 2> ring{{a.x, a.res}, {a.x_stride, a.res_stride}};
  ring.init(norm_smem, cols, a.rows, at.row);
  const int off = ring.off;
#pragma unroll
  for (int s = 0; s < kStages; ++s) ring.fill(s, at.row + s * at.step);
  uint32_t w2[U][4];
  norm_weights<U, ACC>(a.w, off, cols, w2);
  int slot = 0;
  for (int64_t row = at.row; row < a.rows;
       row += at.step, slot = slot + 1 == kStages ? 0 : slot + 1) {
    float h[U][8];
    float ss = 0.0f;
    ring.arrive();
#pragma unroll
    for (int k = 0; k < U; ++k) {
      ring.template take<DT>(slot, row, 0, k, h[k]);
      if (a.res != nullptr) {
        float r[8];
        ring.template take<DT>(slot, row, 1, k, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] = __fadd_rn(h[k][i], r[i]);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) ss = __fadd_rn(ss, sq8f(h[k]));
    if (a.sum != nullptr) {
#pragma unroll
      for (int k = 0; k < U; ++k)
        norm_store<DT, ACC>(a.sum + row * a.sum_stride, k, off, cols, ring.bits, h[k]);
    }
    ss = row_share.sum(ss);
    ring.fill(slot, row + kStages * at.step);  // the slot's lines are in registers
    float rstd = rsqrtf(__fmaf_rn(ss, a.inv_cols, a.eps));
    if (!(ss <= 3.402823466e38f)) {  // the same in every thread of the row
      float s2 = 0.0f;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __fmul_rn(h[k][i], kNormShrink);
        s2 = __fadd_rn(s2, sq8f(q));
      }
      rstd = norm_rstd_big(row_share.sum(s2), a.inv_cols);
    }
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < U; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        h[k][i] = __fmul_rn(__fmul_rn(h[k][i], rstd), norm_weight<DT>(w2[k], i));
    }
    if constexpr (OUT == kOutHalf) {
#pragma unroll
      for (int k = 0; k < U; ++k)
        norm_store<DT, ACC>(static_cast<uint16_t*>(a.out) + row * a.out_stride, k, off, cols,
                            ring.bits, h[k]);
      continue;
    }
    uint8_t* const out = static_cast<uint8_t*>(a.out) + row * a.out_stride;
    float* const scales = a.scales + row * a.groups;
    float c = 0.0f;
    uint32_t* const segs = seg + threadIdx.y * (blockDim.x >> 5) * U * 8;
    if constexpr (OUT == kOutRow) {
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < U; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) top = abs_max_nan(top, h[k][i]);
      }
      c = e4m3_scale(row_share.top(abs_bits(top)));
      if (threadIdx.x == 0) scales[0] = c;
    } else if constexpr (ACC == kSingle) {
#pragma unroll
      for (int j = 0; j < U * 8; ++j) {  // columns j * T and on: a segment a warp
        const uint32_t top = __reduce_max_sync(0xffffffffu, abs_bits(h[j / 8][j % 8]));
        if ((threadIdx.x & 31) == 0) segs[j * (blockDim.x >> 5) + (threadIdx.x >> 5)] = top;
      }
      row_share.sync();
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if constexpr (ACC != kSingle) {
        const int e = norm_at<ACC>(k, 0, off);
        if constexpr (OUT == kOutGroup) {  // 4, 8 or 16 neighbouring lanes share a group
          float top = abs_max_nan(h[k][0], h[k][1]);
#pragma unroll
          for (int i = 2; i < 8; ++i) top = abs_max_nan(top, h[k][i]);
          top = abs_max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = abs_max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
          if (a.group > 32) top = abs_max_nan(top, __shfl_xor_sync(0xffffffffu, top, 4));
          if (a.group > 64) top = abs_max_nan(top, __shfl_xor_sync(0xffffffffu, top, 8));
          c = e4m3_scale(abs_bits(top));
          if (e < cols && (e & (a.group - 1)) == 0) scales[e >> a.group_log2] = c;
        }
        float (&q)[8] = h[k];
        by_scale(q, c);
        if (norm_whole<ACC>(ring.bits, k, cols)) {
          *reinterpret_cast<uint2*>(out + e) = pack8_e4m3(q);
        } else if (ACC == kShifted && norm_live<ACC>(ring.bits, k, cols)) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (e + i >= 0 && e + i < cols) out[e + i] = (uint8_t)float2_to_e4m3x2(q[i], 0.0f);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = norm_at<ACC>(k, i, off);
          if (e < cols) {
            if constexpr (OUT == kOutGroup) {
              // past the row's end the segments hold zeros or are not there
              const int per = a.group / 32, first = (e >> a.group_log2) * per;
              const int end = min(first + per, (int)(blockDim.x >> 5) * U * 8);
              uint32_t top = 0;
              for (int s = first; s < end; ++s) top = max(top, segs[s]);
              c = e4m3_scale(top);
              if ((e & (a.group - 1)) == 0) scales[e >> a.group_log2] = c;
            }
            float q[1] = {h[k][i]};
            by_scale(q, c);
            out[e] = (uint8_t)float2_to_e4m3x2(q[0], 0.0f);
          }
        }
      }
    }
    if constexpr (OUT == kOutGroup && ACC == kSingle) row_share.sync();  // written again
  }
}

// Rows past the largest register form: a CTA of 1024 threads reads its row
// two or three times (the later reads come from L2 for as long as the row is
// there).  Everything is written in the last pass, element by element after
// it was read, so that outputs may lie over inputs here too.
template <int DT>
__device__ __forceinline__ float wide_h(const NormArgs& a, int64_t row, int e) {
  float h = half_bits_to_float<DT>(a.x[row * a.x_stride + e]);
  if (a.res != nullptr) h = __fadd_rn(h, half_bits_to_float<DT>(a.res[row * a.res_stride + e]));
  return h;
}

template <int DT, int OUT>
__global__ void __launch_bounds__(1024) k_norm_wide(const __grid_constant__ NormArgs a) {
  pdl_enter_last(a.x, a.res, a.w, a.sum, a.out, a.scales, a.rstd);
  constexpr int T = 1024;
  __shared__ float sm[2][32];
  __shared__ uint32_t seg[32];
  RowShare row_share{sm};
  const int t = threadIdx.x;
  const int cols = a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float ss = 0.0f;
#pragma unroll 4
    for (int64_t e = t; e < cols; e += T) {
      const float h = wide_h<DT>(a, row, (int)e);
      ss = __fmaf_rn(h, h, ss);
    }
    ss = row_share.sum(ss);
    float rstd = rsqrtf(__fmaf_rn(ss, a.inv_cols, a.eps));
    if (!(ss <= 3.402823466e38f)) {
      float s2 = 0.0f;
      for (int64_t e = t; e < cols; e += T) {
        const float h = __fmul_rn(wide_h<DT>(a, row, (int)e), kNormShrink);
        s2 = __fmaf_rn(h, h, s2);
      }
      rstd = norm_rstd_big(row_share.sum(s2), a.inv_cols);
    }
    if (a.rstd != nullptr && t == 0) a.rstd[row] = rstd;
    float c = 0.0f;
    if constexpr (OUT == kOutRow) {
      uint32_t top = 0;
#pragma unroll 4
      for (int64_t e = t; e < cols; e += T)
        top = max(top, abs_bits(__fmul_rn(__fmul_rn(wide_h<DT>(a, row, (int)e), rstd),
                                          half_bits_to_float<DT>(a.w[e]))));
      c = e4m3_scale(row_share.top(top));
      if (t == 0) a.scales[row] = c;
    }
    for (int64_t e0 = 0; e0 < cols; e0 += T) {  // uniform: barriers inside
      const int64_t e = e0 + t;
      float h = 0.0f, y = 0.0f;
      if (e < cols) {
        h = wide_h<DT>(a, row, (int)e);
        y = __fmul_rn(__fmul_rn(h, rstd), half_bits_to_float<DT>(a.w[e]));
      }
      if constexpr (OUT == kOutGroup) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, abs_bits(y));
        __syncthreads();  // the last trip's segments have been read
        if ((t & 31) == 0) seg[t >> 5] = top;
        __syncthreads();
        const int per = a.group / 32, first = t / a.group * per;
        uint32_t m = seg[first];
        for (int s = 1; s < per; ++s) m = max(m, seg[first + s]);
        c = e4m3_scale(m);
        if (e < cols && t % a.group == 0) a.scales[row * a.groups + e / a.group] = c;
      }
      if (e < cols) {
        if (a.sum != nullptr)
          a.sum[row * a.sum_stride + e] = (uint16_t)float_to_half_bits<DT>(h);
        if constexpr (OUT != kOutHalf) {
          float q[1] = {y};
          by_scale(q, c);
          static_cast<uint8_t*>(a.out)[row * a.out_stride + e] =
              (uint8_t)float2_to_e4m3x2(q[0], 0.0f);
        } else {
          static_cast<uint16_t*>(a.out)[row * a.out_stride + e] =
              (uint16_t)float_to_half_bits<DT>(y);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- gradients

// dx of a row from registers, and dweight's partial sums: each thread keeps its
// columns' sums over all rows it meets in registers, and writes them once at
// the end (one row of `part` per CTA); k_norm_dw adds them up.  Few rows are one
// cluster of kNormCluster CTAs, which add up each other's sums in shared memory:
// the second launch costs a short call a third of its time.
constexpr int kNormCluster = 8;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}

// The float at shared address `at` of the cluster's CTA `rank`.
__device__ __forceinline__ float cluster_load(uint32_t at, int rank) {
  uint32_t there;
  float x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(there) : "memory");
  return x;
}

// (257 to 320 threads are a form of their own, two CTAs an SM at 102 registers: rows
// of 4,095 columns 123 us for 64 million elements, 145 among those of up to 512.)
template <int DT, int U, int ACC, int MAXT>
__global__ void
__launch_bounds__(MAXT, MAXT == 320 ? 2 : MAXT <= 512 ? norm_bwd_sm_threads(U, ACC) / MAXT : 1)
    k_norm_bwd(const __grid_constant__ NormBwdArgs a) {
  pdl_enter_last(a.dy, a.h, a.dsum, a.w, a.rstd, a.dx, a.part);
  extern __shared__ __align__(16) uint8_t norm_smem[];
  __shared__ float sm[2][32];
  RowShare row_share{sm};
  constexpr int kStages = kNormStages;
  const int cols = a.cols;
  const int threads = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
  NormRows<ACC> at;
  NormRing<U, ACC, kStages, 3> ring{{a.dy, a.h, a.dsum}, {a.dy_stride, a.h_stride, a.dsum_stride}};
  ring.init(norm_smem, cols, a.rows, at.row);
  const int off = ring.off;
#pragma unroll
  for (int s = 0; s < kStages; ++s) ring.fill(s, at.row + s * at.step);
  float dw[U][8];
  uint32_t w2[U][4];
  norm_weights<U, ACC>(a.w, off, cols, w2);
#pragma unroll
  for (int k = 0; k < U; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = 0.0f;
  }
  float rstd = at.row < a.rows ? a.rstd[at.row] : 0.0f;
  int slot = 0;
  for (int64_t row = at.row; row < a.rows;
       row += at.step, slot = slot + 1 == kStages ? 0 : slot + 1) {
    const float rstd_next = row + at.step < a.rows ? a.rstd[row + at.step] : 0.0f;
    // Where the registers run short a row is taken from the ring a second time
    // for dx instead of being held; the slot is filled again only after that.
    // (us for 64 million elements, taken twice and held: lines of 1,024 columns 82
    // and 105, 16,384 121 and 166; shifted rows of 763 116 and 212, 1,001 95 and
    // 172, 2,047 124 and 140, 4,095 123 and 190, 8,191 231 and 278; but lines of 768
    // 80 and 79, 8,192 85 and 83, shifted rows of 1,211 124 and 112, single
    // elements of 1,000 251 and 197.)
    constexpr bool kTwice =
        U == 4 || (U == 3 && ACC == kShifted) ||
        (U == 2 && (MAXT > 512 || MAXT == 320 || ACC == kShifted));
    float g[U][8], xh[U][8];
    uint4 ds[U];
    ring.arrive();
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      ring.template take<DT>(slot, row, 0, k, g[k]);
      ring.template take<DT>(slot, row, 1, k, xh[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[k][i] = __fmul_rn(xh[k][i], rstd);
        dw[k][i] = __fmaf_rn(g[k][i], xh[k][i], dw[k][i]);
        g[k][i] = __fmul_rn(g[k][i], norm_weight<DT>(w2[k], i));
        dot = __fmaf_rn(g[k][i], xh[k][i], dot);
      }
      if constexpr (!kTwice && ACC != kSingle)
        if (a.dsum != nullptr) ds[k] = ring.raw(slot, 2, k);
    }
    const float c = __fmul_rn(row_share.sum(dot), a.inv_cols);
    if constexpr (!kTwice) ring.fill(slot, row + kStages * at.step);  // its lines are in registers
    uint16_t* const dx = a.dx + row * a.dx_stride;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if constexpr (kTwice) {
        ring.template take<DT>(slot, row, 0, k, g[k]);
        ring.template take<DT>(slot, row, 1, k, xh[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xh[k][i] = __fmul_rn(xh[k][i], rstd);
          g[k][i] = __fmul_rn(g[k][i], norm_weight<DT>(w2[k], i));
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) g[k][i] = __fmul_rn(rstd, __fmaf_rn(-xh[k][i], c, g[k][i]));
      if (a.dsum != nullptr) {
        if constexpr (kTwice || ACC == kSingle) {
          float d[8];
          ring.template take<DT>(slot, row, 2, k, d);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[k][i] = __fadd_rn(g[k][i], d[i]);
        } else {
          add8<DT>(g[k], ds[k]);
        }
      }
      norm_store<DT, ACC>(dx, k, off, cols, ring.bits, g[k]);
    }
    if constexpr (kTwice) ring.fill(slot, row + kStages * at.step);
    rstd = rstd_next;
  }
  float* const red = reinterpret_cast<float*>(norm_smem);
  const bool cluster = a.part == nullptr;
  if (blockDim.y > 1 || cluster) {  // through shared memory: the ring is done with
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int k = 0; k < U; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = norm_at<ACC>(k, i, off);
        if (e >= 0 && e < cols) red[threadIdx.y * cols + e] = dw[k][i];
      }
    }
    __syncthreads();
  }
  if (cluster) {
    if (blockDim.y > 1) {
      for (int e = tid; e < cols; e += threads)
        for (int r = 1; r < (int)blockDim.y; ++r) red[e] = __fadd_rn(red[e], red[r * cols + e]);
    }
    cluster_sync();
    const uint32_t here = (uint32_t)__cvta_generic_to_shared(red);
    for (int e = blockIdx.x * threads + tid; e < cols; e += kNormCluster * threads) {
      float s = 0.0f;
#pragma unroll
      for (int r = 0; r < kNormCluster; ++r) s = __fadd_rn(s, cluster_load(here + e * 4, r));
      a.dweight[e] = a.accumulate ? __fadd_rn(a.dweight[e], s) : s;
    }
    cluster_sync();  // nobody leaves while its sums are read
    return;
  }
  float* const part = a.part + (int64_t)blockIdx.x * cols;
  if (blockDim.y > 1) {  // the CTA's rows hold sums of the same columns
    for (int e = tid; e < cols; e += threads) {
      float s = red[e];
      for (int r = 1; r < (int)blockDim.y; ++r) s = __fadd_rn(s, red[r * cols + e]);
      part[e] = s;
    }
  } else {
#pragma unroll
    for (int k = 0; k < U; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = norm_at<ACC>(k, i, off);
        if (e >= 0 && e < cols) part[e] = dw[k][i];
      }
    }
  }
}

// dweight (+)= the sum of nparts rows of partial sums: 32 columns a CTA, its 32
// warps take every 32nd row, in a fixed order.
__global__ void __launch_bounds__(1024)
    k_norm_dw(const float* __restrict__ part, int nparts, int cols, int accumulate,
              float* __restrict__ dweight) {
  pdl_enter_last(part, dweight);
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t e = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (e < cols) {
#pragma unroll 8
    for (int r = warp; r < nparts; r += 32) s = __fadd_rn(s, part[(int64_t)r * cols + e]);
  }
  red[warp][lane] = s;
  __syncthreads();
  s = red[lane][warp];  // warp w now holds column w's 32 sums
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
  const int64_t col = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && col < cols) dweight[col] = accumulate ? __fadd_rn(dweight[col], s) : s;
}

// Rows past the largest register form: first each row's mean(weight*dy*xhat),
// then columns: a thread takes one column and every gridDim.y-th row.
template <int DT>
__global__ void __launch_bounds__(1024) k_norm_bwd_dot(const __grid_constant__ NormBwdArgs a) {
  pdl_enter_last(a.dy, a.h, a.w, a.rstd, a.dot);
  __shared__ float sm[2][32];
  RowShare row_share{sm};
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float dot = 0.0f;
#pragma unroll 4
    for (int64_t e = threadIdx.x; e < a.cols; e += 1024)
      dot = __fmaf_rn(__fmul_rn(half_bits_to_float<DT>(a.dy[row * a.dy_stride + e]),
                                half_bits_to_float<DT>(a.w[e])),
                      __fmul_rn(half_bits_to_float<DT>(a.h[row * a.h_stride + e]), rstd), dot);
    dot = row_share.sum(dot);
    if (threadIdx.x == 0) a.dot[row] = __fmul_rn(dot, a.inv_cols);
  }
}

template <int DT>
__global__ void __launch_bounds__(256) k_norm_bwd_cols(const __grid_constant__ NormBwdArgs a) {
  pdl_enter_last(a.dy, a.h, a.dsum, a.w, a.rstd, a.dx, a.part, a.dot);
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= a.cols) return;
  const float w = half_bits_to_float<DT>(a.w[e]);
  float dw = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float rstd = a.rstd[row];
    const float g = half_bits_to_float<DT>(a.dy[row * a.dy_stride + e]);
    const float xh = __fmul_rn(half_bits_to_float<DT>(a.h[row * a.h_stride + e]), rstd);
    dw = __fmaf_rn(g, xh, dw);
    float d = __fmul_rn(rstd, __fmaf_rn(-xh, a.dot[row], __fmul_rn(g, w)));
    if (a.dsum != nullptr) d = __fadd_rn(d, half_bits_to_float<DT>(a.dsum[row * a.dsum_stride + e]));
    a.dx[row * a.dx_stride + e] = (uint16_t)float_to_half_bits<DT>(d);
  }
  a.part[(int64_t)blockIdx.y * a.cols + e] = dw;
}

}  // namespace zs

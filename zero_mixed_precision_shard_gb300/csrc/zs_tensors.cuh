// sm_103a kernels of the optimizer step over a list of tensors.
//
// Two passes over the list, each one launch whatever the number of tensors:
//   k_list_check   every gradient once: whether any is inf/NaN, and the sum of
//                  squares; the last CTA to finish resolves the step (overflow,
//                  clipping coefficient, Adam's constants, the loss scale);
//   k_list_apply   AdamW, the half copy, and the moments in 32 or in 8 bits.
// The overflow has to be known before any state is written, so the gradients
// are read twice; everything else moves once.
//
// Both are bound by HBM (measured at 124M elements: the update moves 28 bytes
// an element with fp16 gradients and 32-bit moments at 6.9 TB/s, 504 us, and 16
// with 8-bit ones at 6.6 TB/s, 304 us; the check reads 2 at 5.2 TB/s, 48 us with
// its fixed start and end, and at 5.9 over 1.07 GB).
//
// The update's CTA takes one chunk of one tensor (the plan's chunk table, built
// at creation), a warp a block of 256 elements at a time: through a ring of
// asynchronous copies where the tensor's arrays are 16-byte aligned and the
// unit of 2,048 elements is full, elements lane, lane + 32, ... one by one
// otherwise (any alignment, and the ragged ends).
//
// 8-bit moments: a block of 256 consecutive elements of one tensor shares an
// fp32 scale c = max|x| / 448, at least 2^-126; the stored byte is the E4M3
// value nearest to x / c.  m is stored so, and of v its root r = sqrt(v): the
// root halves v's range in binades, so that E4M3's 17 binades hold |g| ratios
// of 2^17 within a block, and r > 0 never rounds to 0 (it keeps at least the
// least code, 2^-9): a lost second moment would divide a living first moment
// by eps.  An inf or NaN among a block's values makes its scale inf or NaN, and the
// block reads back so.  The scale is fp32 and not a power of two so that a block whose
// values all decay by 0.1 % a step decays with it; a coarse scale would hold
// it still.
#pragma once

#include <cuda_fp8.h>

#include "zs_kernels.cuh"

namespace zs {

constexpr int kBlockElems = ZS_STATE_BLOCK;             // elements that share a state scale
constexpr int kListUnit = kThreads / 32 * kBlockElems;  // elements a CTA takes per trip
constexpr int kListChunkUnits = 4;                      // trips of a large list's chunk
constexpr int kListCheckCtas = 4;                       // resident CTAs per SM of the check pass
static_assert(kBlockElems == 256, "a warp takes a block as 8 elements a lane");

// Gradient addresses that one launch of k_list_set_grads carries by value.
#define ZS_LIST_GRADS_PER_LAUNCH 400

struct ListRec {
  const void* grad;
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  uint16_t* half;
  int64_t count;
  float lr_mult, wd_mult;
  int32_t grad_fp32;
  int32_t pad_;
};

struct ListChunk {
  int32_t tensor;  // -1: nothing to do (the one chunk of a list without elements)
  int32_t index;   // chunk number within the tensor
};

// Constants of the update with 8-bit moments, which takes the bias corrections
// and adamw1's eps together, root as an fp32 pair:
//   (m * inv_bc1) / (r * sbc2 + eps) = m / (r * root + eps / inv_bc1)
struct ListRatios {
  float root, root_lo, eps;
};

// From 1 - beta1^t and sqrt(1 / (1 - beta2^t)).
__host__ __device__ inline ListRatios list_ratios(double bc1, double sbc2, float eps) {
  ListRatios r;
  const double root = sbc2 * bc1;
  r.root = (float)root;
  r.root_lo = (float)(root - (double)r.root);
  r.eps = (float)((double)eps * bc1);
  return r;
}

// What the check pass leaves for the update.
struct ListStep {
  AdamArgs ad;
  float coef;      // clipping coefficient, 1 without clipping
  int32_t skip;    // the step overflowed: write nothing
  float inv_div;   // exact_inverse(grad_div)
  float g_mul;     // coef * inv_div, 0 where that is not exact
  ListRatios ratios;
  double inv_div2; // 1 / grad_div^2
};

// 1 / d where that is exact (a power of two, as loss scales are), 0 where not:
// a product with it is then the quotient by d, bit for bit.
__device__ __forceinline__ float exact_inverse(float d) {
  const uint32_t b = __float_as_uint(d), e = b >> 23;
  return (b & 0x7FFFFFu) == 0u && e >= 1u && e <= 253u ? __uint_as_float((254u - e) << 23) : 0.0f;
}

// A product of the sum of gradients with coef * inv_div is the averaged and
// clipped gradient as adamw1 forms it, by a quotient and a product, wherever the
// averaged gradient is no subnormal.
__device__ __forceinline__ float list_g_mul(float coef, float inv_div) {
  const float x = __fmul_rn(coef, inv_div);
  return x >= 0x1p-126f ? x : 0.0f;
}

// As pdl_enter, without letting the successor in early: it is launched when
// this grid's last CTA exits.  The list's kernels fill the GPU to their end,
// and a successor's CTAs waiting on it cost them more than the launch gap
// (124M elements, 8-bit moments: 370 us a step with the early launch, 344
// without; 11 us either way for a small list).
template <typename... P>
__device__ __forceinline__ void pdl_enter_last(const P*... ptrs) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  (pdl_escape(ptrs), ...);
}

struct ListPlan {
  ListRec* recs;
  const ListChunk* chunks;
  double* partials;   // one per CTA of the check pass
  uint32_t* counter;  // CTAs of the check pass that are done; zero between launches
  ListStep* step;
  int32_t nchunks;
  int32_t chunk_units;  // trips of kListUnit elements per chunk
};

// How the check pass ends: `dstate` non-null, the whole step is resolved from
// it; otherwise the flag and the sum go to the caller's words.
struct ListFinish {
  zs_device_state* dstate;
  zs_adam_hparams hp;
  zs_lr_schedule sched;
  int32_t has_sched, n, accum_steps;
  float max_norm;
  float* norm_out;
  int32_t* flag;
  double* sumsq;
  double inv_div2;
};

// Squares of single gradient values, summed apart by size so that none leaves
// fp32 at either end: past 1e15 in magnitude a value is scaled by 2^-80 first,
// below 2^-55 by 2^100 (its least square is then 2^-98).  An inf or NaN makes its
// sum inf or NaN and stays visible to the end.
constexpr float kListLow = 0x1p-55f;
struct ListSquares {
  float mid = 0.0f, big = 0.0f, low = 0.0f;
  __device__ __forceinline__ void add(float g) {
    if (fabsf(g) > 1e15f) {
      const float t = __fmul_rn(g, 0x1p-80f);
      big = __fmaf_rn(t, t, big);
    } else if (fabsf(g) < kListLow) {
      const float t = __fmul_rn(g, 0x1p100f);
      low = __fmaf_rn(t, t, low);
    } else {
      mid = __fmaf_rn(g, g, mid);
    }
  }
};

template <int DT>
__device__ __forceinline__ void unpack8(const uint4 h, float a[8]) {
  const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    a[2 * k] = half_bits_to_float<DT>(w[k] & 0xFFFFu);
    a[2 * k + 1] = half_bits_to_float<DT>(w[k] >> 16);
  }
}

template <int DT>
__device__ __forceinline__ uint4 pack8(const float a[8]) {
  bool unused = false;
  return pack8_hacc<DT>(a, &unused);
}

// 16 bytes of gradients: 8 halves (GT a zs_dtype) or 4 floats (ZS_FP32).
template <int GT>
__device__ __forceinline__ void unpack16(const uint4 q, float (&a)[GT == ZS_FP32 ? 4 : 8]) {
  if constexpr (GT == ZS_FP32) {
    a[0] = __uint_as_float(q.x);
    a[1] = __uint_as_float(q.y);
    a[2] = __uint_as_float(q.z);
    a[3] = __uint_as_float(q.w);
  } else {
    unpack8<GT>(q, a);
  }
}

// A thread's sum of squares: what rounding cuts off each addition is carried
// into the next, so that the sum of a thread that strides over a long list
// keeps 32 bits.  `big` and `low` are the sums of the scaled squares.
struct ListSum {
  float sum = 0.0f, cut = 0.0f, big = 0.0f, low = 0.0f;
  __device__ __forceinline__ void add(float x) {
    const float y = __fsub_rn(x, cut);
    const float t = __fadd_rn(sum, y);
    cut = __fsub_rn(__fsub_rn(t, sum), y);
    sum = t;
  }
  __device__ __forceinline__ void add(const ListSquares& q) {
    add(q.mid);
    big = __fadd_rn(big, q.big);
    low = __fadd_rn(low, q.low);
  }
};

// Gradients on their way through registers: kListBatch loads of 16 bytes.
constexpr int kListBatch = 4;

// Whether any of a batch's values is not a zero.
template <int GT>
__device__ __forceinline__ bool list_any(const uint4 (&q)[kListBatch]) {
  uint32_t any = 0;
#pragma unroll
  for (int j = 0; j < kListBatch; ++j) any |= q[j].x | q[j].y | q[j].z | q[j].w;
  return (any & (GT == ZS_FP32 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) != 0;
}

// Squares of a batch without a test (two instructions an element: the pass
// would be bound by issue otherwise), and again, with one, where the sum is
// large, not a number, or so small that squares were lost in it: at 2^-110 the
// 32 values' squares are off by at most 32 half units of 2^-149, 2^-35 of the
// sum.  (A half has no square below 2^-48; batches of zeros are common, and left
// at once.)
template <int GT>
__device__ __forceinline__ void list_squares(const uint4 (&q)[kListBatch], ListSum& s) {
  constexpr int kPer = GT == ZS_FP32 ? 4 : 8;
  float t[2] = {0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < kListBatch; ++j) {
    float a[kPer];
    unpack16<GT>(q[j], a);
#pragma unroll
    for (int k = 0; k < kPer; ++k) t[k & 1] = __fmaf_rn(a[k], a[k], t[k & 1]);
  }
  t[0] = __fadd_rn(t[0], t[1]);
  if (t[0] < 1e30f && (GT == ZS_FP16 || t[0] >= kListLow * kListLow)) {
    s.add(t[0]);
    return;
  }
  if (GT != ZS_FP16 && t[0] < 1e30f && !list_any<GT>(q)) return;
  ListSquares sq;
#pragma unroll
  for (int j = 0; j < kListBatch; ++j) {
    float a[kPer];
    unpack16<GT>(q[j], a);
#pragma unroll
    for (int k = 0; k < kPer; ++k) sq.add(a[k]);
  }
  s.add(sq);
}

// The elements of a chunk in front of its first 16-byte boundary and behind
// its last, 14 at most: a thread each.
template <int GT, typename E>
__device__ __forceinline__ void list_ends(const E* g, int head, int64_t tail, int64_t n,
                                          ListSum& s) {
  int64_t i = threadIdx.x;
  if (i >= head) i += tail - head;
  if (i >= n) return;
  ListSquares sq;
  if constexpr (GT == ZS_FP32) sq.add(g[i]);
  else sq.add(half_bits_to_float<GT>(g[i]));
  s.add(sq);
}

// Asynchronous copy of 4, 8 or 16 bytes from global to shared memory.
template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// Waits until at most N of this thread's copy groups are in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// As cp_async<16>, zeros in place of the bytes where `live` is false.
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(live ? 16 : 0)
               : "memory");
}

// A CTA's way over its chunks, a batch of every thread at a time.
template <int HT>
struct ListCursor {
  const ListPlan& pl;
  ListChunk next;      // the chunk after the current one, read ahead
  int c;               // its number
  const uint4* v = nullptr;
  int nv = 0, at = 0;  // 16-byte words of the current chunk, and the batch's first
  bool fp32 = false;

  __device__ __forceinline__ explicit ListCursor(const ListPlan& p) : pl(p), c(blockIdx.x) {
    next = pl.chunks[c];
  }

  // To the next batch; what a chunk holds beside its 16-byte words is squared
  // on entering it.  False at the end.
  __device__ __forceinline__ bool advance(ListSum& s) {
    at += kListBatch * kThreads;
    while (at >= nv) {
      if (c >= pl.nchunks) return false;
      const ListChunk now = next;
      c += gridDim.x;
      if (c < pl.nchunks) next = pl.chunks[c];
      at = nv = 0;
      if (now.tensor < 0) continue;
      const ListRec& rec = pl.recs[now.tensor];
      const int64_t chunk = (int64_t)pl.chunk_units * kListUnit;
      const int64_t base = (int64_t)now.index * chunk;
      const int64_t n = rec.count - base < chunk ? rec.count - base : chunk;
      fp32 = rec.grad_fp32 != 0;
      if (fp32) enter<ZS_FP32>(static_cast<const float*>(rec.grad) + base, n, s);
      else enter<HT>(static_cast<const uint16_t*>(rec.grad) + base, n, s);
    }
    return true;
  }

  template <int GT, typename E>
  __device__ __forceinline__ void enter(const E* g, int64_t n, ListSum& s) {
    constexpr int kPer = 16 / sizeof(E);
    const int off = (int)(reinterpret_cast<uintptr_t>(g) & 15u) / (int)sizeof(E);
    int head = off == 0 ? 0 : kPer - off;
    if (head > n) head = (int)n;
    nv = (int)((n - head) / kPer);
    v = reinterpret_cast<const uint4*>(g + head);
    list_ends<GT>(g, head, head + (int64_t)nv * kPer, n, s);
  }
};

// Norm and clipping coefficient of the averaged gradient's sum of squares, in
// fp64 and rounded once, as the flat step forms them: what one norm over
// several lists and shards clips is scaled alike everywhere.
__device__ __forceinline__ float list_coef(double sumsq, float max_norm, float* norm) {
  const double n = sqrt(sumsq);
  *norm = (float)n;
  return clip_coef_of_norm(n, max_norm);
}

// The step's constants by one warp: what device_step_args forms, its powers,
// reciprocals and roots side by side in lanes 0 and 1, the schedule's learning
// rate in lane 2 and grad_div's reciprocals in lane 3.
__device__ __forceinline__ void list_step_args(const ListFinish& fin, ListStep* step) {
  const int lane = threadIdx.x & 31;
  const zs_device_state* st = fin.dstate;
  const int64_t t = st->step + 1;
  const float div = (float)((double)fin.n * (double)fin.accum_steps * (double)st->scaler.scale);
  if (lane == 2) step->ad.lr = fin.has_sched ? lr_at(fin.sched, t) : fin.hp.lr;
  if (lane == 3) {
    step->inv_div = exact_inverse(div);
    step->inv_div2 = 1.0 / ((double)div * (double)div);
    step->ad.grad_div = div;
    step->ad.beta1 = fin.hp.beta1;
    step->ad.omb1 = 1.0f - fin.hp.beta1;
    step->ad.beta2 = fin.hp.beta2;
    step->ad.omb2 = 1.0f - fin.hp.beta2;
    step->ad.eps = fin.hp.eps;
    step->ad.wd = fin.hp.weight_decay;
  }
  double mine = 0.0;  // lane 0: 1 - beta1^t, lane 1: sqrt(1 / (1 - beta2^t))
  if (lane < 2) {
    const double bc = 1.0 - pow_int((double)(lane == 0 ? fin.hp.beta1 : fin.hp.beta2), t);
    const double inv = 1.0 / bc;
    const float hi = (float)inv;
    const float lo = (float)(inv - (double)hi);
    if (lane == 0) {
      mine = bc;
      step->ad.inv_bc1 = hi;
      step->ad.inv_bc1_lo = lo;
    } else {
      mine = sqrt(inv);
      step->ad.inv_bc2 = hi;
      step->ad.inv_bc2_lo = lo;
      step->ad.sbc2 = (float)mine;
      step->ad.sbc2_lo = (float)(mine - (double)step->ad.sbc2);
    }
  }
  const double sbc2 = __shfl_sync(0xffffffffu, mine, 1);
  if (lane == 0) step->ratios = list_ratios(mine, sbc2, fin.hp.eps);
}

// The end of the check pass (one thread): the step resolved from the sum of
// squares, which is not finite if any gradient is not.
__device__ __forceinline__ void list_finish(const ListPlan& pl, const ListFinish& fin,
                                            double sum) {
  const int bad = !(sum <= 1.7976931348623157e308);
  if (fin.dstate != nullptr) {
    float norm;
    const float coef = list_coef(sum * __ldcg(&pl.step->inv_div2), fin.max_norm, &norm);
    pl.step->coef = coef;
    pl.step->g_mul = list_g_mul(coef, __ldcg(&pl.step->inv_div));
    pl.step->skip = bad;
    AdamArgs ad;  // what device_state_step records
    ad.lr = __ldcg(&pl.step->ad.lr);
    ad.grad_div = __ldcg(&pl.step->ad.grad_div);
    device_state_step(fin.dstate, bad, ad);
    if (fin.norm_out != nullptr) *fin.norm_out = norm;
  } else {
    if (bad) atomicOr(fin.flag, 1);
    if (fin.sumsq != nullptr) *fin.sumsq = sum * fin.inv_div2;
  }
}

// Check pass.  HT: the list's half format (of the gradients that are not
// fp32).  The grid is what the GPU holds at once and strides over the chunks;
// each thread copies its words of the batches ahead into a ring in shared
// memory that it reads alone.  (A CTA per chunk instead pays the end of a CTA --
// its sum, the fence, the count of finished CTAs, about a microsecond -- for
// every chunk: 73 us for 124M fp16 gradients, 48 so; a kernel that only reads
// reaches 6.66 TB/s.)
constexpr int kCheckStages = 3;
template <int HT>
__global__ void __launch_bounds__(kThreads, kListCheckCtas)
    k_list_check(const ListPlan pl, const ListFinish fin) {
  pdl_enter_last(pl.recs, pl.chunks, pl.partials, pl.counter, pl.step, fin.dstate, fin.norm_out,
                 fin.flag, fin.sumsq);
  __shared__ uint4 ring[kCheckStages][kListBatch][kThreads];
  // CTA 0's last warp forms the constants while the gradients are read, not
  // the last CTA at the end
  if (fin.dstate != nullptr && blockIdx.x == 0 && threadIdx.x >= kThreads - 32)
    list_step_args(fin, pl.step);
  ListSum s;
  ListCursor<HT> cur(pl);
  uint32_t fp32 = 0;  // of the batches in flight, the oldest in bit 0
  int flying = 0;
  bool more = true;
  const auto fill = [&](int slot) {
    more = more && cur.advance(s);
    if (more) {
#pragma unroll
      for (int j = 0; j < kListBatch; ++j) {
        const int i = cur.at + j * kThreads + threadIdx.x;
        const bool live = i < cur.nv;
        cp_async16_or_zero(&ring[slot][j][threadIdx.x], cur.v + (live ? i : 0), live);
      }
      fp32 |= (uint32_t)cur.fp32 << flying;
      flying += 1;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kCheckStages; ++k) fill(k);
  for (int slot = 0; flying > 0; slot = slot + 1 == kCheckStages ? 0 : slot + 1) {
    cp_async_wait<kCheckStages - 1>();
    uint4 q[kListBatch];
#pragma unroll
    for (int j = 0; j < kListBatch; ++j) q[j] = ring[slot][j][threadIdx.x];
    if (fp32 & 1u) list_squares<ZS_FP32>(q, s);
    else list_squares<HT>(q, s);
    fp32 >>= 1;
    flying -= 1;
    __syncwarp();  // the warp's reads of the slot come before the copies into it
    fill(slot);
  }
  bool unused = false;
  double total = cta_norm_total(__fsub_rn(s.sum, s.cut), s.big, false, &unused);
  if (__syncthreads_or(s.low != 0.0f))
    total += cta_norm_total(s.low, 0.0f, false, &unused) * 0x1p-200;
  // the last CTA to finish folds the sums, in a fixed order whichever it is
  __shared__ int last;
  if (threadIdx.x == 0) {
    pl.partials[blockIdx.x] = total;
    __threadfence();
    last = atomicAdd(pl.counter, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  const double sum = fold_partials<true>(pl.partials, (int)gridDim.x);
  if (threadIdx.x != 0) return;
  *pl.counter = 0;
  list_finish(pl, fin, sum);
}

// The update's constants where the caller resolved the step (one thread).
__global__ void k_list_args(const int32_t* __restrict__ flag, const double* __restrict__ sumsq,
                            float max_norm, AdamArgs ad, ListRatios ratios,
                            ListStep* __restrict__ step) {
  pdl_enter(flag, sumsq, step);
  if (blockIdx.x != 0 || threadIdx.x != 0) return;
  float norm;
  const float coef = sumsq != nullptr ? list_coef(*sumsq, max_norm, &norm) : 1.0f;
  step->ad = ad;
  step->coef = coef;
  step->g_mul = list_g_mul(coef, exact_inverse(ad.grad_div));
  step->ratios = ratios;
  step->skip = *flag != 0;
}

// New gradient addresses, passed by value: they are the launch's own, so a
// captured graph keeps them and the caller's array can go at once.
struct ListGrads {
  const void* p[ZS_LIST_GRADS_PER_LAUNCH];
};
__global__ void k_list_set_grads(ListRec* __restrict__ recs, int first, int n,
                                 const __grid_constant__ ListGrads g) {
  pdl_enter(recs);
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) recs[first + i].grad = g.p[i];
}

// ---------------------------------------------------------------- update

// Two E4M3 bytes (the low one first) as floats, and back with saturation.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(__half2(h));
}

__device__ __forceinline__ uint32_t float2_to_e4m3x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ void unpack8_e4m3(const uint2 q, float a[8]) {
  const uint32_t w[4] = {q.x & 0xFFFFu, q.x >> 16, q.y & 0xFFFFu, q.y >> 16};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = e4m3x2_to_float2(w[k]);
    a[2 * k] = f.x;
    a[2 * k + 1] = f.y;
  }
}

__device__ __forceinline__ uint2 pack8_e4m3(const float a[8]) {
  return make_uint2(float2_to_e4m3x2(a[0], a[1]) | (float2_to_e4m3x2(a[2], a[3]) << 16),
                    float2_to_e4m3x2(a[4], a[5]) | (float2_to_e4m3x2(a[6], a[7]) << 16));
}

// x held to +-limit; a NaN stays one.
__device__ __forceinline__ float held_to(float x, float limit) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(-limit));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(limit));
  return x;
}

__device__ __forceinline__ float rcp_approx(float c) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(c));
  return r;
}

// x / c from the approximate reciprocal of c: a quotient 2 units off at most,
// corrected by its own residual, which one fma forms (Markstein 1990).  What is
// left beside the last rounding is 2^-21 of a unit.  For c in [2^-93, 2^126);
// beside smaller ones the residual of small quotients leaves fp32.
__device__ __forceinline__ float quotient(float x, float c, float rcp) {
  const float q = __fmul_rn(x, rcp);
  return __fmaf_rn(__fmaf_rn(-q, c, x), rcp, q);
}

// top / 448 rounded (a quotient by 7 lies a fourteenth of a unit from any midpoint
// or more, so the corrected one is it); inf and NaN stay.
__device__ __forceinline__ float over_448(float top) {
  const float c = quotient(top, 448.0f, 1.0f / 448.0f);
  return top <= 3.402823466e38f ? c : top;
}

// The scale of values whose largest magnitude has these fp32 bits.
__device__ __forceinline__ float e4m3_scale(uint32_t amax_bits) {
  const float c = over_448(__uint_as_float(amax_bits));
  return c < 0x1p-126f ? 0x1p-126f : c;
}

// Values by their scale, ready for E4M3 (small scales brought up, exactly).
template <int N>
__device__ __forceinline__ void by_scale(float (&x)[N], float c) {
  if (c < 0x1p-60f) {
    c = __fmul_rn(c, 0x1p64f);
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = __fmul_rn(x[k], 0x1p64f);
  }
  const float r = rcp_approx(c);
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = quotient(x[k], c, r);
}

// The root of v >= 0 in the same way, from the approximate reciprocal root:
// s = v * y, s + (v - s^2) * y / 2.  For v of 2^-100 and more; the root of
// smaller ones is 2 units off at most, that of zero is zero.
__device__ __forceinline__ float square_root(float v) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(v, 0x1p-126f)));
  const float s = __fmul_rn(v, y);
  return __fmaf_rn(__fmaf_rn(-s, s, v), __fmul_rn(0.5f, y), s);
}

// max(|a|, |b|), NaN if either is.
__device__ __forceinline__ float abs_max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// A block's values in the registers of one warp, 8 a lane.
struct ListVals {
  float g[8], p[8], m[8], v[8];
};

// What a CTA takes from the step's constants beside its tensor's multipliers.
struct ListConsts {
  float coef, g_mul;
  ListRatios ratios;
};

// AdamW of a block with 8-bit moments: m and v come as the codes' values and
// leave as the values to be encoded, mc and vc are their scales before and
// after.  The new moments are those of adamw1 bit for bit, the update is as good:
// the root of v_hat is taken as that of v, which is stored, times the bias
// corrections' ratio.  Quotients and roots are the corrected ones above (a step of
// the 124M-element list takes 353 us, 506 with CUDA's rounded division and root).
// The averaged gradient is held to +-2^63, where its square would leave fp32.
__device__ __forceinline__ void list_update_q8(ListVals& x, const AdamArgs& ad,
                                               const ListConsts& lc, float& mc, float& vc) {
  if (lc.g_mul != 0.0f) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x.g[k] = __fmul_rn(x.g[k], lc.g_mul);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x.g[k] = __fmul_rn(__fdiv_rn(x.g[k], ad.grad_div), lc.coef);
  }
  float mtop = 0.0f, vtop = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float g = held_to(x.g[k], 0x1p63f);
    const float r = __fmul_rn(x.v[k], vc);
    x.m[k] = __fmaf_rn(ad.beta1, __fmul_rn(x.m[k], mc), __fmul_rn(ad.omb1, g));
    x.v[k] = __fmaf_rn(ad.beta2, __fmul_rn(r, r), __fmul_rn(ad.omb2, __fmul_rn(g, g)));
    mtop = abs_max_nan(mtop, x.m[k]);
    vtop = abs_max_nan(vtop, x.v[k]);
  }
  // (an inf or NaN has the largest bits: its block's scale is not finite)
  mtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mtop)));
  vtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vtop)));
  // Small blocks, scaled up by powers of two: a root below 2^-20 of its block's
  // largest is stored as the least code, so the others are at least 2^-50.  (To
  // the update such a root, 2 units off at most, is nothing beside an eps of
  // 2^-48 or more.)
  float rs = 1.0f;
  if (vtop < 0x1p-60f) {
    rs = 0x1p-32f;
    vtop = __fmul_rn(vtop, 0x1p64f);
#pragma unroll
    for (int k = 0; k < 8; ++k) x.v[k] = __fmul_rn(x.v[k], 0x1p64f);
  }
  float cv = over_448(square_root(vtop));
  vc = __fmul_rn(cv, rs);
  if (vc < 0x1p-126f) {
    vc = 0x1p-126f;
    cv = rs == 1.0f ? 0x1p-126f : 0x1p-94f;
  }
  const float root = __fmul_rn(lc.ratios.root, rs), root_lo = __fmul_rn(lc.ratios.root_lo, rs),
              eps = lc.ratios.eps;
  if (mtop <= 3.402823466e38f && vtop <= 3.402823466e38f && eps >= 0x1p-72f &&
      eps <= 0x1p60f) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float s = square_root(x.v[k]);
      const float d = __fmaf_rn(s, root, __fmaf_rn(s, root_lo, eps));
      const float upd = quotient(x.m[k], d, rcp_approx(d));
      x.p[k] = __fmaf_rn(-ad.lr, __fmaf_rn(ad.wd, x.p[k], upd), x.p[k]);
      x.v[k] = s;
    }
  } else {  // values that are not finite, or an eps that d could lie far from
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float s = __fsqrt_rn(x.v[k]);
      float upd = __fdiv_rn(x.m[k], __fmaf_rn(s, root, __fmaf_rn(s, root_lo, eps)));
      if (upd != upd) upd = 0.0f;  // as adamw1 has it
      x.p[k] = __fmaf_rn(-ad.lr, __fmaf_rn(ad.wd, x.p[k], upd), x.p[k]);
      x.v[k] = s;
    }
  }
  mc = e4m3_scale(__float_as_uint(mtop));
  by_scale(x.m, mc);
  const float vi = rcp_approx(cv);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float q = quotient(x.v[k], cv, vi);
    x.v[k] = x.v[k] > 0.0f && q < 0x1p-9f ? 0x1p-9f : q;
  }
}

// The update of a block, in place.
template <int STATES>
__device__ __forceinline__ void list_update(ListVals& x, const AdamArgs& ad, const ListConsts& lc,
                                            float& mc, float& vc) {
  if constexpr (STATES == ZS_STATES_8BIT) {
    list_update_q8(x, ad, lc, mc, vc);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) adamw1<true>(ad, x.g[k], x.p[k], x.m[k], x.v[k], lc.coef);
  }
}

// A lane's elements of a full block: 4 from 4 * lane and 4 from 128 + 4 *
// lane, so that a warp's accesses cover 512 contiguous bytes of the fp32
// arrays.  (8 consecutive ones a lane would take half of each 32-byte sector
// per access: the L2 then serves every sector twice, 660 against 504 us for
// the 124M-element list with 32-bit moments.)  i0: the lane's first element.
constexpr int kListHalf = kBlockElems / 2;

template <int STATES, int HT>
__device__ __forceinline__ void list_store8(const ListRec& rec, int64_t i0, const ListVals& x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = i0 + h * kListHalf;
    __stcs(reinterpret_cast<float4*>(rec.master + i),
           make_float4(x.p[4 * h], x.p[4 * h + 1], x.p[4 * h + 2], x.p[4 * h + 3]));
    if constexpr (STATES == ZS_STATES_FP32) {
      __stcs(reinterpret_cast<float4*>(static_cast<float*>(rec.m) + i),
             make_float4(x.m[4 * h], x.m[4 * h + 1], x.m[4 * h + 2], x.m[4 * h + 3]));
      __stcs(reinterpret_cast<float4*>(static_cast<float*>(rec.v) + i),
             make_float4(x.v[4 * h], x.v[4 * h + 1], x.v[4 * h + 2], x.v[4 * h + 3]));
    } else {
      __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(rec.m) + i),
             float2_to_e4m3x2(x.m[4 * h], x.m[4 * h + 1]) |
                 (float2_to_e4m3x2(x.m[4 * h + 2], x.m[4 * h + 3]) << 16));
      __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(rec.v) + i),
             float2_to_e4m3x2(x.v[4 * h], x.v[4 * h + 1]) |
                 (float2_to_e4m3x2(x.v[4 * h + 2], x.v[4 * h + 3]) << 16));
    }
  }
  if (rec.half != nullptr) {
    const uint4 h = pack8<HT>(x.p);
    __stcs(reinterpret_cast<uint2*>(rec.half + i0), make_uint2(h.x, h.y));
    __stcs(reinterpret_cast<uint2*>(rec.half + i0 + kListHalf), make_uint2(h.z, h.w));
  }
}

// A block without the ring, for ragged ends and arrays off the 16-byte
// boundary: n <= kBlockElems elements from `at` on, lane, lane + 32, ... of them.
template <int STATES, int HT>
__device__ __forceinline__ void list_block(const ListRec& rec, const AdamArgs& ad,
                                           const ListConsts& lc, int64_t at, int n) {
  const int lane = threadIdx.x & 31;
  uint8_t* const mq = static_cast<uint8_t*>(rec.m);
  uint8_t* const vq = static_cast<uint8_t*>(rec.v);
  float* const mf = static_cast<float*>(rec.m);
  float* const vf = static_cast<float*>(rec.v);
  ListVals x;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x.g[k] = x.p[k] = x.m[k] = x.v[k] = 0.0f;
    const int j = lane + 32 * k;
    if (j < n) {
      x.g[k] = rec.grad_fp32
                   ? static_cast<const float*>(rec.grad)[at + j]
                   : half_bits_to_float<HT>(static_cast<const uint16_t*>(rec.grad)[at + j]);
      x.p[k] = rec.master[at + j];
      if constexpr (STATES == ZS_STATES_8BIT) {
        x.m[k] = e4m3x2_to_float2(mq[at + j]).x;
        x.v[k] = e4m3x2_to_float2(vq[at + j]).x;
      } else {
        x.m[k] = mf[at + j];
        x.v[k] = vf[at + j];
      }
    }
  }
  float mc = 0.0f, vc = 0.0f;
  const int64_t blk = at / kBlockElems;
  if constexpr (STATES == ZS_STATES_8BIT) {
    mc = rec.m_scale[blk];
    vc = rec.v_scale[blk];
  }
  list_update<STATES>(x, ad, lc, mc, vc);
  if constexpr (STATES == ZS_STATES_8BIT) {
    __syncwarp();  // every lane has read the block's scales
    if (lane == 0) {
      rec.m_scale[blk] = mc;
      rec.v_scale[blk] = vc;
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int j = lane + 32 * k;
    if (j < n) {
      rec.master[at + j] = x.p[k];
      if constexpr (STATES == ZS_STATES_8BIT) {
        mq[at + j] = (uint8_t)float2_to_e4m3x2(x.m[k], 0.0f);
        vq[at + j] = (uint8_t)float2_to_e4m3x2(x.v[k], 0.0f);
      } else {
        mf[at + j] = x.m[k];
        vf[at + j] = x.v[k];
      }
      if (rec.half != nullptr) rec.half[at + j] = (uint16_t)float_to_half_bits<HT>(x.p[k]);
    }
  }
}

// The update's ring in shared memory: each thread copies the elements of the
// units ahead that it will use itself (cp.async), so no barrier stands between
// a copy and its use, and the bytes in flight do not cost registers (457 us
// without a ring, 294 with it, for 124M elements with 8-bit moments; one to four
// stages are within 3 %).  A stage holds planes of 4 elements a thread, two of
// each array (16-byte places for the gradients, half filled by halves).
template <int STATES>
struct ListRing {
  static constexpr int kStages = STATES == ZS_STATES_8BIT ? 3 : 2;
  static constexpr int kStageBytes = kThreads * (STATES == ZS_STATES_8BIT ? 80 : 128);
  static constexpr int kBytes = kStages * kStageBytes;
};

template <int STATES>
__device__ __forceinline__ void ring_fill(uint8_t* stage, const ListRec& rec, int64_t i0) {
  uint4* const w = reinterpret_cast<uint4*>(stage) + threadIdx.x;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = i0 + h * kListHalf;
    if (rec.grad_fp32)
      cp_async<16>(w + h * kThreads, static_cast<const float*>(rec.grad) + i);
    else
      cp_async<8>(reinterpret_cast<uint2*>(stage) + h * kThreads + threadIdx.x,
                  static_cast<const uint16_t*>(rec.grad) + i);
    cp_async<16>(w + (2 + h) * kThreads, rec.master + i);
    if constexpr (STATES == ZS_STATES_8BIT) {
      uint32_t* const q = reinterpret_cast<uint32_t*>(stage + 64 * kThreads) + threadIdx.x;
      cp_async<4>(q + h * kThreads, static_cast<const uint8_t*>(rec.m) + i);
      cp_async<4>(q + (2 + h) * kThreads, static_cast<const uint8_t*>(rec.v) + i);
    } else {
      cp_async<16>(w + (4 + h) * kThreads, static_cast<const float*>(rec.m) + i);
      cp_async<16>(w + (6 + h) * kThreads, static_cast<const float*>(rec.v) + i);
    }
  }
}

__device__ __forceinline__ void plane_load8(const uint4* a, const uint4* b, float x[8]) {
  const uint4 q = *a, r = *b;
  x[0] = __uint_as_float(q.x); x[1] = __uint_as_float(q.y);
  x[2] = __uint_as_float(q.z); x[3] = __uint_as_float(q.w);
  x[4] = __uint_as_float(r.x); x[5] = __uint_as_float(r.y);
  x[6] = __uint_as_float(r.z); x[7] = __uint_as_float(r.w);
}

template <int STATES, int HT>
__device__ __forceinline__ void ring_take(const uint8_t* stage, const ListRec& rec, ListVals& x) {
  const uint4* const w = reinterpret_cast<const uint4*>(stage) + threadIdx.x;
  if (rec.grad_fp32) {
    plane_load8(w, w + kThreads, x.g);
  } else {
    const uint2* const g = reinterpret_cast<const uint2*>(stage) + threadIdx.x;
    const uint2 a = g[0], b = g[kThreads];
    unpack8<HT>(make_uint4(a.x, a.y, b.x, b.y), x.g);
  }
  plane_load8(w + 2 * kThreads, w + 3 * kThreads, x.p);
  if constexpr (STATES == ZS_STATES_8BIT) {
    const uint32_t* const q = reinterpret_cast<const uint32_t*>(stage + 64 * kThreads) + threadIdx.x;
    unpack8_e4m3(make_uint2(q[0], q[kThreads]), x.m);
    unpack8_e4m3(make_uint2(q[2 * kThreads], q[3 * kThreads]), x.v);
  } else {
    plane_load8(w + 4 * kThreads, w + 5 * kThreads, x.m);
    plane_load8(w + 6 * kThreads, w + 7 * kThreads, x.v);
  }
}

template <int STATES, int HT>
__global__ void __launch_bounds__(kThreads, 3) k_list_apply(const ListPlan pl) {
  extern __shared__ __align__(16) uint8_t ring[];
  using Ring = ListRing<STATES>;
  pdl_enter_last(pl.recs, pl.chunks, pl.step);
  // From the last chunk to the first: the check pass read the last gradients
  // last, and the L2 still holds some of them.
  const ListChunk ch = pl.chunks[pl.nchunks - 1 - blockIdx.x];
  if (pl.step->skip || ch.tensor < 0) return;
  const ListRec rec = pl.recs[ch.tensor];
  const uintptr_t wide = reinterpret_cast<uintptr_t>(rec.grad) |
                         reinterpret_cast<uintptr_t>(rec.master) |
                         reinterpret_cast<uintptr_t>(rec.half);
  const uintptr_t states = reinterpret_cast<uintptr_t>(rec.m) | reinterpret_cast<uintptr_t>(rec.v);
  const bool vec = (wide & 15u) == 0 && (states & (STATES == ZS_STATES_8BIT ? 3u : 15u)) == 0;
  const int64_t base = (int64_t)ch.index * pl.chunk_units * kListUnit;
  const int64_t left = rec.count - base;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int full = vec ? (int)(left / kListUnit < pl.chunk_units ? left / kListUnit : pl.chunk_units) : 0;
  const int64_t i0 = base + warp * kBlockElems + lane * 4;
#pragma unroll
  for (int s = 0; s < Ring::kStages; ++s) {
    if (s < full) ring_fill<STATES>(ring + s * Ring::kStageBytes, rec, i0 + s * kListUnit);
    cp_async_commit();
  }
  AdamArgs ad = pl.step->ad;
  ad.lr = __fmul_rn(ad.lr, rec.lr_mult);
  ad.wd = __fmul_rn(ad.wd, rec.wd_mult);
  const ListConsts lc = {pl.step->coef, pl.step->g_mul, pl.step->ratios};
  // the scales of this warp's block of unit u are kept by lane u
  static_assert(kListChunkUnits <= 32, "a lane for every unit of a chunk");
  float mcs = 0.0f, vcs = 0.0f;
  const int64_t blk = base / kBlockElems + lane * (kListUnit / kBlockElems) + warp;
  if constexpr (STATES == ZS_STATES_8BIT) {
    if (lane < full) {
      mcs = rec.m_scale[blk];
      vcs = rec.v_scale[blk];
    }
  }
  int slot = 0;
  for (int u = 0; u < full; ++u) {
    cp_async_wait<Ring::kStages - 1>();
    uint8_t* const stage = ring + slot * Ring::kStageBytes;
    slot = slot + 1 == Ring::kStages ? 0 : slot + 1;
    ListVals x;
    ring_take<STATES, HT>(stage, rec, x);
    float mc = 0.0f, vc = 0.0f;
    if constexpr (STATES == ZS_STATES_8BIT) {
      mc = __shfl_sync(0xffffffffu, mcs, u);
      vc = __shfl_sync(0xffffffffu, vcs, u);
    }
    list_update<STATES>(x, ad, lc, mc, vc);
    __syncwarp();  // the warp's reads of the stage come before the copies into it
    if (u + Ring::kStages < full)
      ring_fill<STATES>(stage, rec, i0 + (int64_t)(u + Ring::kStages) * kListUnit);
    cp_async_commit();
    if constexpr (STATES == ZS_STATES_8BIT) {
      if (lane == u) {
        mcs = mc;
        vcs = vc;
      }
    }
    list_store8<STATES, HT>(rec, i0 + (int64_t)u * kListUnit, x);
  }
  if constexpr (STATES == ZS_STATES_8BIT) {
    if (lane < full) {
      rec.m_scale[blk] = mcs;
      rec.v_scale[blk] = vcs;
    }
  }
  for (int u = full; u < pl.chunk_units; ++u) {
    const int64_t at = base + (int64_t)u * kListUnit + warp * kBlockElems;
    const int64_t n = rec.count - at;
    if (n <= 0) break;
    list_block<STATES, HT>(rec, ad, lc, at, n < kBlockElems ? (int)n : kBlockElems);
  }
}

}  // namespace zs

// Paged 8-bit KV cache: the step plan, the append and the attention that reads
// the cache (the serving form of the INT8 KV cache of "VAR-Compressor：在边缘GPU上
// 实现80亿参数视觉自回归模型的高效量化部署", INT8 KV缓存量化; the block-wise scale is
// the granularity that lets tokens join a cache without touching other blocks).
//
// Block b of the pool holds, for every key/value head h, `bs` tokens of d 8-bit
// codes (contiguous bs x d bytes at ((b kv + h) bs d)) and one fp32 scale for the
// keys and one for the values (at b kv + h): x ~ code * scale.
//
// Times in comments: device time on one B200 in a CUDA graph of 20 calls, where what
// fits the 126 MB L2 is read from it; "as a call" is a call among others from Python
// with inputs that change from call to call.
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "../../include/svdq.h"
#include "internal.h"
#include "ptx.cuh"

namespace svdq {
namespace paged {

using namespace svdq::dev;

constexpr int kMaxRequests = 16384;
// Tokens, lengths and rows stay this far from 2^31: the kernels round them up to tiles in 32 bits.
constexpr int kMaxCount = INT32_MAX - 65536;

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// ------------------------------------------------------------------ step plan
// new_i = max(0, target_i - prev_i); request i needs ceil(target/bs) -
// ceil(prev/bs) more blocks (taken from the front of the free ring in request
// order) or gives that many back (appended at its end).  Every CTA scans all B
// requests (three exclusive sums: new tokens, blocks taken, blocks given) into
// its own shared memory and then writes its share of the outputs, so one launch
// needs no communication between CTAs.  A token's block is found without reading
// what another CTA writes: blocks below ceil(prev/bs) come from the table, later
// ones from the ring.  Latency-bound: the lengths' load, the scan, one search.
// 3.8 us for 64 decoding requests, 7.6 us for a mixed step of 1000, 6.8 us for 256
// prompts of 570,000 slots (one slot at a time a thread: 9.2 us); as calls 6.8, 7.6, 10.4.
constexpr int kPlanThreads = 512, kPlanSlots = 4;

struct PlanArgs {
  const int* prev;
  const int* target;
  int* table;
  int* lens;
  int* cu;
  int* slots;
  int* ring;
  const int* state_in;
  int* state_out;
  int B, max_blocks, n_tokens, max_new, max_len, n_blocks, lb;
};

__device__ __forceinline__ int blocks_of(int tokens, int lb) {
  return (int)(((int64_t)tokens + ((1 << lb) - 1)) >> lb);
}

// Largest i in [0, n) with pre[i] <= k, for a non-decreasing pre with pre[0] = 0.
__device__ __forceinline__ int last_not_above(const int* pre, int n, int k) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= k) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanArgs A) {
  extern __shared__ int plan_smem[];
  int* s_new = plan_smem;            // [B + 1] exclusive sums
  int* s_take = s_new + A.B + 1;
  int* s_give = s_take + A.B + 1;
  __shared__ long long w_new[kPlanThreads / 32];
  __shared__ int w_take[kPlanThreads / 32], w_give[kPlanThreads / 32], s_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) s_bad = 0;
  griddep_wait();
  griddep_launch();
  __syncthreads();
  const int head = A.state_in[0], count = A.state_in[1];
  long long c_new = 0;
  int c_take = 0, c_give = 0;
  bool bad = head < 0 || head >= A.n_blocks || count < 0 || count > A.n_blocks;
  for (int i0 = 0; i0 < A.B; i0 += kPlanThreads) {
    const int i = i0 + tid;
    long long vn = 0;
    int vt = 0, vg = 0;
    if (i < A.B) {
      const int p = A.prev[i], t = A.target[i];
      if (p < 0 || t < 0 || t > A.max_len || p > (A.max_blocks << A.lb) || t > (A.max_blocks << A.lb) ||
          (t > p && t - p > A.max_new)) {
        bad = true;
      } else {
        const int a = blocks_of(p, A.lb), b = blocks_of(t, A.lb);
        vn = t > p ? t - p : 0;
        vt = b > a ? b - a : 0;
        vg = a > b ? a - b : 0;
      }
    }
    long long n = vn;
    int t = vt, g = vg;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n1 = __shfl_up_sync(0xffffffffu, n, o);
      const int t1 = __shfl_up_sync(0xffffffffu, t, o), g1 = __shfl_up_sync(0xffffffffu, g, o);
      if (lane >= o) { n += n1; t += t1; g += g1; }
    }
    if (lane == 31) { w_new[warp] = n; w_take[warp] = t; w_give[warp] = g; }
    __syncthreads();
    long long bn = c_new;
    int bt = c_take, bg = c_give;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) { bn += w_new[w]; bt += w_take[w]; bg += w_give[w]; }
      c_new += w_new[w]; c_take += w_take[w]; c_give += w_give[w];
    }
    if (i < A.B) {
      s_new[i] = (int)(bn + n - vn);
      s_take[i] = bt + t - vt;
      s_give[i] = bg + g - vg;
    }
    __syncthreads();
  }
  if (bad) s_bad = 1;
  if (tid == 0) { s_new[A.B] = (int)c_new; s_take[A.B] = c_take; s_give[A.B] = c_give; }
  __syncthreads();
  // entries given back are written from head + count on: they must not reach those being taken
  const bool wrong = s_bad != 0 || c_new > A.n_tokens || (int64_t)count + c_give > A.n_blocks;
  const int lacking = wrong ? -1 : (c_take > count ? c_take - count : 0);
  const bool ok = lacking == 0;
  const int gtid = blockIdx.x * kPlanThreads + tid, stride = gridDim.x * kPlanThreads;
  if (gtid == 0) {
    // head may be out of range when the call is refused: handed through as it is
    int h = head;
    if (ok) { h = head + c_take; if (h >= A.n_blocks) h -= A.n_blocks; }
    A.state_out[0] = h;
    A.state_out[1] = ok ? count - c_take + c_give : count;
    A.state_out[2] = lacking;
    A.state_out[3] = ok ? (int)c_new : 0;
  }
  for (int i = gtid; i <= A.B; i += stride) {
    A.cu[i] = ok ? s_new[i] : 0;
    if (i < A.B) A.lens[i] = ok ? A.target[i] : A.prev[i];
  }
  const auto wrap = [&](int64_t k) { return (int)(k >= 2ll * A.n_blocks ? k - 2ll * A.n_blocks : k >= A.n_blocks ? k - A.n_blocks : k); };   // k < 3 n_blocks
  if (ok) {
    for (int k = gtid; k < c_take; k += stride) {
      const int i = last_not_above(s_take, A.B, k);
      A.table[(size_t)i * A.max_blocks + blocks_of(A.prev[i], A.lb) + (k - s_take[i])] = A.ring[wrap((int64_t)head + k)];
    }
    for (int k = gtid; k < c_give; k += stride) {
      const int i = last_not_above(s_give, A.B, k);
      A.ring[wrap((int64_t)head + count + k)] =
          A.table[(size_t)i * A.max_blocks + blocks_of(A.target[i], A.lb) + (k - s_give[i])];
    }
  }
  // slots, four a thread at once: the searches step together and the loads of four slots overlap
  const int total = ok ? (int)c_new : 0;
  int top = 1;
  while (2 * top < A.B) top *= 2;
  for (int64_t k0 = (int64_t)blockIdx.x * (kPlanSlots * kPlanThreads) + tid; k0 < A.n_tokens; k0 += (int64_t)kPlanSlots * stride) {
    int i[kPlanSlots], p[kPlanSlots], slot[kPlanSlots];
#pragma unroll
    for (int u = 0; u < kPlanSlots; ++u) i[u] = 0;
    for (int step = top; step > 0; step >>= 1) {
#pragma unroll
      for (int u = 0; u < kPlanSlots; ++u) {
        const int mid = i[u] + step;
        if (mid < A.B && s_new[mid] <= k0 + u * kPlanThreads) i[u] = mid;
      }
    }
#pragma unroll
    for (int u = 0; u < kPlanSlots; ++u) p[u] = k0 + u * kPlanThreads < total ? A.prev[i[u]] : 0;
#pragma unroll
    for (int u = 0; u < kPlanSlots; ++u) {
      const int64_t k = k0 + u * kPlanThreads;
      slot[u] = -1;
      if (k < total) {
        const int pos = p[u] + ((int)k - s_new[i[u]]), held = blocks_of(p[u], A.lb), c = pos >> A.lb;
        int at = c;                                        // below `held` in the table, above it in the ring
        if (c >= held) {
          at = wrap((int64_t)head + s_take[i[u]] + (c - held));
        }
        const int blk = c < held ? A.table[(size_t)i[u] * A.max_blocks + at] : A.ring[at];
        slot[u] = blk < 0 || blk >= A.n_blocks ? -1 : (blk << A.lb) + (pos & ((1 << A.lb) - 1));
      }
    }
#pragma unroll
    for (int u = 0; u < kPlanSlots; ++u)
      if (k0 + u * kPlanThreads < A.n_tokens) A.slots[k0 + u * kPlanThreads] = slot[u];
  }
}

// -------------------------------------------------------------------- append
// One CTA per (block touched by a request's new tokens, kv head, keys or values).
// s = max(s_old, max |x| / qmax), codes = round(x / s); codes of the tokens that
// the block held before are re-rounded when s grows.  The new rows (at most one
// block: bs d values) are read once and stay in registers between the maximum
// and the codes.  Work index w -> request: request i owns the indices from
// floor(cu_i / bs) + 2 i, which leaves it at least as many as it touches blocks
// (<= floor(new / bs) + 2), so the grid needs only n_tokens and B on the host; + i
// where no request has more than one new token.  Bound by the chain lengths -> slots
// -> rows of each CTA, so by how many CTAs are resident: at most 80 registers, 24 warps
// an SM (at a time when a thread needed 80: 16 warps 25.8 us, 24 21.9, 32 with spills 22.4;
// now 72 and no spills).  Five prompts of 15,000 tokens in all, 8 heads of 128: 22.0 us,
// as a call 24.8 (3.5 TB/s); 48 single tokens 3.7 us, 1000 49 us (every CTA's search for
// its request is linear in B).
constexpr int append_threads(int BS, int D) { return BS * D >= 16384 ? 256 : 128; }

template <int FMT> struct Fmt;
template <> struct Fmt<SVDQ_KV_INT8> { static constexpr float qmax = 127.0f; };
template <> struct Fmt<SVDQ_KV_E4M3> { static constexpr float qmax = 448.0f; };

template <int DT>
__device__ __forceinline__ float load16(uint16_t h) {
  if constexpr (DT == SVDQ_BF16) return __uint_as_float((uint32_t)h << 16);
  else return __half2float(__ushort_as_half(h));
}
template <int DT> constexpr uint32_t kInf16 = DT == SVDQ_BF16 ? 0x7F80u : 0x7C00u;   // bits of +infinity

template <int DT>
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == SVDQ_BF16) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// x / s as IEEE division rounds it: q = RN(x rs) is within an ulp, e = q s - x is
// exact (one FMA), RN(q - e rs) is the correctly rounded quotient (Markstein) while
// nothing under- or overflows: for 2^-60 <= s <= 2^60, rs = RN(1 / s).  e is +0 where
// the quotient is exact, and -e rs + q then keeps the sign of a zero q (with x - q s
// for e a quotient of -0 came out as +0, another E4M3 code).
__device__ __forceinline__ float quotient(float x, float s, float rs) {
  const float q = __fmul_rn(x, rs);
  return __fmaf_rn(-__fmaf_rn(q, s, -x), rs, q);
}

__device__ __noinline__ float divide_rn(float x, float s) { return __fdiv_rn(x, s); }

// Four values to four codes, round to nearest even, saturating.
template <int FMT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  if constexpr (FMT == SVDQ_KV_INT8) {
    const auto q = [](float x) { return (uint32_t)(clampi(__float2int_rn(x), -127, 127) & 0xFF); };
    return q(a) | (q(b) << 8) | (q(c) << 16) | (q(d) << 24);
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
}

template <int FMT>
__device__ __forceinline__ float code_value(uint32_t byte) {
  if constexpr (FMT == SVDQ_KV_INT8) {
    return (float)(int8_t)byte;
  } else {
    // E4M3 -> fp16 of value / 256: the exponent field moves up by one place, exact for every finite code
    const uint16_t h = (uint16_t)(((byte & 0x80u) << 8) | ((byte & 0x7Fu) << 7));
    return __half2float(__ushort_as_half(h)) * 256.0f;
  }
}

struct AppendArgs {
  const uint16_t* x[2];    // keys, values
  int64_t stride[2];       // elements between tokens
  uint8_t* codes[2];
  float* scale[2];
  const int* cu;
  const int* slots;
  int B, n_tokens, kv, n_blocks, max_new, per;   // per: spare work indices a request
};

// The first token of [from, to) that has a slot, or `to`.  Called by all threads of the CTA, where a token without a
// slot stands at a place that others follow from; apart, so that the usual call's registers do not pay for it.
template <int THREADS>
__device__ __noinline__ int first_with_slot(const int* slots, int from, int to) {
  __shared__ int s_first;
  for (; from < to; from += THREADS) {
    const int t = from + threadIdx.x;
    if (threadIdx.x == 0) s_first = INT_MAX;
    __syncthreads();
    if (t < to && slots[t] >= 0) atomicMin(&s_first, t);
    __syncthreads();
    const int first = s_first;
    __syncthreads();
    if (first != INT_MAX) return first;
  }
  return to;
}

template <int DT, int FMT, int D, int LB>
__global__ void __launch_bounds__(append_threads(1 << LB, D), 768 / append_threads(1 << LB, D)) paged_append_kernel(const AppendArgs A) {
  constexpr int kAppendThreads = append_threads(1 << LB, D);
  constexpr int BS = 1 << LB, kPerRow = D / 8, kRows = kAppendThreads / kPerRow, kPass = BS / kRows > 0 ? BS / kRows : 1;
  __shared__ uint32_t s_top[kAppendThreads / 32];
  const int tid = threadIdx.x, w = blockIdx.x, h = blockIdx.y, which = blockIdx.z;
  griddep_wait();
  griddep_launch();
  // this work item's request: the last one whose first index is not above w
  int i = -1;
  for (int r0 = 0; r0 < A.B; r0 += kAppendThreads) {
    const int r = r0 + tid;
    const bool le = r < A.B && (clampi(A.cu[r], 0, A.n_tokens) >> LB) + A.per * r <= w;
    i += __syncthreads_count(le);
  }
  if (i < 0) return;
  const int a = clampi(A.cu[i], 0, A.n_tokens), e = clampi(A.cu[i + 1], 0, A.n_tokens);
  if (a >= e) return;
  if (e - a > A.max_new && tid == 0) record_status(SVDQ_ERR_INVALID_ARG);
  // o0: row of the request's first token in its block.  Where that token has no slot, any other one tells: the first
  // that has one among those that can be this item's (a longer search would make a long skipped prefix quadratic)
  const int j = w - (a >> LB) - A.per * i;
  int lead = a, slot0 = A.slots[a];
  if (slot0 < 0) {
    const int to = (int)min((int64_t)e, a + (j + 1) * (int64_t)BS);
    lead = first_with_slot<kAppendThreads>(A.slots, max(a, to - 2 * BS + 1), to);
    if (lead >= to) return;
    slot0 = A.slots[lead];
  }
  const int o0 = (slot0 - (lead - a)) & (BS - 1);
  const int64_t first = (int64_t)a + (j == 0 ? 0 : (int64_t)j * BS - o0);
  if (first >= e) return;
  // this item's tokens [t0, end), from the first one that has a slot
  int t0 = (int)first;
  const int end = t0 + min(e - t0, j == 0 ? BS - o0 : BS);
  slot0 = A.slots[t0];
  if (slot0 < 0) {
    t0 = first_with_slot<kAppendThreads>(A.slots, t0, end);
    if (t0 == end) return;
    slot0 = A.slots[t0];
  }
  const int blk = slot0 >> LB, off = slot0 & (BS - 1);
  if (blk >= A.n_blocks) {
    if (tid == 0) record_status(SVDQ_ERR_INVALID_ARG);
    return;
  }
  const int rows = min(end - t0, BS - off);
  const int c = tid % kPerRow, r0 = tid / kPerRow;
  // chosen, not indexed: an index into the arguments would copy them to local memory
  const int64_t stride = which ? A.stride[1] : A.stride[0];
  const uint16_t* x = (which ? A.x[1] : A.x[0]) + (int64_t)t0 * stride + h * D + 8 * c;
  float* scale = which ? A.scale[1] : A.scale[0];
  const size_t cell = (size_t)blk * A.kv + h;
  const float s_old = off > 0 ? scale[cell] : 0.0f;
  uint4 v[kPass];
  int at[kPass];
  uint32_t have = 0;
  // rows and their slots at once; a row counts only where the slot map puts it as far
  // from the block's first new row as its token is from that one's
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int r = r0 + p * kRows;
    v[p] = make_uint4(0, 0, 0, 0);
    at[p] = -1;
    if (r < rows) {
      v[p] = *reinterpret_cast<const uint4*>(x + (int64_t)r * stride);
      at[p] = A.slots[t0 + r];
    }
  }
  bool astray = ((slot0 - o0 - (t0 - a)) & (BS - 1)) != 0;
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    if (at[p] == slot0 + r0 + p * kRows) {
      have |= 1u << p;
    } else {
      v[p] = make_uint4(0, 0, 0, 0);
      astray = astray || at[p] >= 0;
    }
  }
  if (astray) record_status(SVDQ_ERR_INVALID_ARG);
  // the largest magnitude by its bits, two values at once: as whole numbers they order like the magnitudes, with
  // infinity and then NaN above all others, where a maximum of floats would let a NaN vanish
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const uint32_t u[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) top = __vmaxu2(top, u[k] & 0x7FFF7FFFu);
  }
  top = __reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xFFFFu));
  if ((tid & 31) == 0) s_top[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kAppendThreads / 32; ++k) top = max(top, s_top[k]);
  float amax = load16<DT>((uint16_t)top);
  if (top >= kInf16<DT>) {                              // the scale says so to every reader: what sees the block is NaN
    amax = INFINITY;
    if (tid == 0) record_status(SVDQ_ERR_INVALID_ARG);
  }
  const float s = fmaxf(s_old, __fdiv_rn(amax, Fmt<FMT>::qmax));
  uint8_t* base = (which ? A.codes[1] : A.codes[0]) + cell * (size_t)(BS * D);
  if (s > s_old) {
    if (tid == 0) scale[cell] = s;
    const float ratio = __fdiv_rn(s_old, s);
    for (int p = tid; p < off * D / 16; p += kAppendThreads) {
      uint4* at = reinterpret_cast<uint4*>(base) + p;
      uint4 q = *at;
      uint32_t* u = &q.x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) f[b] = __fmul_rn(code_value<FMT>((u[k] >> (8 * b)) & 0xFFu), ratio);
        u[k] = codes4<FMT>(f[0], f[1], f[2], f[3]);
      }
      *at = q;
    }
  } else if (off == 0 && tid == 0) {
    scale[cell] = 0.0f;                     // a fresh block of zeros
  }
  // two copies of the loop: with the division inlined at every value the code left the
  // instruction cache (five prompts of 15,000 tokens in all: 47 us, without it 26)
  const auto write = [&](auto divide) {
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      if (have >> p & 1u) {
        float f[8];
        unpack8<DT>(v[p], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = divide(f[k]);
        *reinterpret_cast<uint2*>(base + (size_t)(off + r0 + p * kRows) * D + 8 * c) =
            make_uint2(codes4<FMT>(f[0], f[1], f[2], f[3]), codes4<FMT>(f[4], f[5], f[6], f[7]));
      }
    }
  };
  if (s >= 0x1p-60f && s <= 0x1p+60f) {
    const float rs = __frcp_rn(s);
    write([&](float x) { return quotient(x, s, rs); });
  } else if (s > 0.0f && s < INFINITY) {
    write([&](float x) { return divide_rn(x, s); });
  } else {
    write([](float) { return 0.0f; });                  // zeros; or 0 times an infinite scale, which no reader mistakes
  }
}

// ----------------------------------------------------------------- attention
// Row r of request i, kv head h: new token r / G, query head h G + r % G.  With
// codes c and scales s per block: x_t = scale 2^e s_k (q' . c_t) log2(e), where
// q' = q 2^-e in fp16 (e: exponent of the row's largest entry, within [-120, 113], so q' is
// exact up to 2^-25 of that entry, of 2^-120 for smaller ones); out = sum_t p_t s_v c^v_t / sum_t p_t, p_t = 2^(x_t - m).
// Both products run on fp16 operands (8-bit codes are exact in fp16) with fp32
// accumulators.  The sum takes p relative to m, a score seen so far; the product takes
// p' = p s_v = 2^(x + log2 s_v - n), rounded to fp16, relative to n, 2^kRoom below a weighted
// magnitude x + log2 s_v seen so far.  Both come from what the row sees alone, so that
// a large scale behind a causal mask, or of no weight, costs nothing.  Both may lag by 2^kGrow:
// p' <= 2^14 does not overflow, what was summed is rarely rescaled, and a weight is
// off by 2^-11 of itself (the size of the rounding of an fp16 output) or, below fp16's
// normal numbers, by 2^-31 of the row's largest weighted magnitude.  At the end
// O 2^(n - m) / l; pieces of rows are kept so divided and joined as means with the weights
// 2^m l, which no sum of large values overflows.
struct AttnArgs {
  const uint16_t* q;
  uint16_t* out;
  const uint8_t* kc;
  const uint8_t* vc;
  const float* ks;
  const float* vs;
  const int* table;
  const int* lens;
  const int* cu;
  float* part_o;           // pieces of cut items: [CTA][2][rows][d]
  float* part_ml;          // [CTA][2][rows][2]
  struct Piece* pieces;    // [CTA][2]
  int64_t q_stride, out_stride;
  int B, max_blocks, n_tokens, max_new, max_len, n_blocks, kv, G, lb, causal, splits;
  float scale_log2;
  double inv_parts;        // 1 / CTAs of the schedule
  int snap;                // items are not cut
  uint32_t g_inv;          // ceil(2^32 / G), 0 for G = 1: x / G is exact for x G < 2^32
};

// What one request's rows see.
struct Rows {
  int a, n, L, rows;       // first token, new tokens, cached length, n G
};
__device__ __forceinline__ Rows request_rows(const AttnArgs& A, int i, bool note) {
  Rows R;
  R.a = clampi(A.cu[i], 0, A.n_tokens);
  const int e = clampi(A.cu[i + 1], 0, A.n_tokens), n = e - R.a, L = A.lens[i];
  R.n = clampi(n, 0, A.max_new);
  R.L = clampi(L, 0, min(A.max_len, A.max_blocks << A.lb));
  if (note && (n > A.max_new || L > R.L)) record_status(SVDQ_ERR_INVALID_ARG);
  R.rows = R.n * A.G;
  return R;
}
// A block number of a request's table: -1, and recorded, where it lies outside the pool.
__device__ __forceinline__ int pool_block(const AttnArgs& A, int id) {
  if (id >= 0 && id < A.n_blocks) return id;
  record_status(SVDQ_ERR_INVALID_ARG);
  return -1;
}
// Tokens that row r sees (its new token is r / G).
__device__ __forceinline__ int seen_by(const AttnArgs& A, const Rows& R, int r) {
  return A.causal ? max(0, R.L - R.n + r / A.G + 1) : R.L;
}

template <int DT>
__device__ __forceinline__ uint16_t store16(float f) {
  if constexpr (DT == SVDQ_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(f));
  else return __half_as_ushort(__float2half_rn(f));
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two codes (in bytes 0 and 1, or 2 and 3, of w) to an fp16 pair: the value for
// int8, value / 256 for E4M3 (kUnit undoes it).  int8: the byte with its sign bit
// flipped is u = code + 128; 0x6400 | u is the fp16 number 1024 + u.
template <int FMT> constexpr float kUnit = FMT == SVDQ_KV_INT8 ? 1.0f : 256.0f;
template <int FMT>
__device__ __forceinline__ uint32_t pre(uint32_t w) {
  return FMT == SVDQ_KV_INT8 ? w ^ 0x80808080u : w;
}
template <int FMT, int HI>
__device__ __forceinline__ uint32_t half2_of(uint32_t w) {
  if constexpr (FMT == SVDQ_KV_INT8) {
    const uint32_t x = __byte_perm(w, 0x64646464u, HI ? 0x4342 : 0x4140);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const uint32_t x = __byte_perm(w, 0u, HI ? 0x3424 : 0x1404);
    return (x & 0x80008000u) | ((x >> 1) & 0x3F803F80u);
  }
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The exponent e that a row of queries is divided by, from its largest magnitude.  Its limits leave every finite bf16
// query at most 2^15 after the division (an fp16 number) and 2^e scale within fp32; rows below 2^-120 keep
// what fp16 has of them after that much.
__device__ __forceinline__ int query_exponent(float top) { return clampi((int)(__float_as_uint(top) >> 23) - 127, -120, 113); }

constexpr float kGrow = 7.0f;   // a softmax reference may lag by this much (2^7)
// The largest weights are taken 2^kRoom above fp16's 1, so that many small ones keep as many more places.
constexpr float kRoom = 7.0f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// At least log2 s, at most one more (122, of the largest bf16 number over 127); -113 for smaller s, so that 2^(m - n)
// is a normal fp32 number.
__device__ __forceinline__ float scale_exponent(float s) {
  return fmaxf(__uint_as_float(0x4B000000u | (__float_as_uint(s) >> 23)) - 8388734.0f, -113.0f);   // 2^23 + field - (2^23 + 126)
}

// A row's accumulator in units of 2^n to its result, 2^(n - m) / l, as two factors that neither over- nor underflow.
__device__ __forceinline__ float2 result_factors(float n, float m, float l) {
  if (!(l > 0.0f)) return make_float2(0.0f, 0.0f);         // a row that sees nothing
  const float g = ex2(0.5f * (n - m));
  return make_float2(g, __fdiv_rn(g, l));
}

// NR rows of queries as normalised fp16 in shared memory (row pitch D + 8) and each
// row's factor 2^e |scale| log2(e), by W warps.  Rows past the request's are zero.
template <int DT, int D, int NR, int W>
__device__ __forceinline__ void load_queries(const AttnArgs& A, const Rows& R, int h, __half* sq, float* sf, int warp, int lane) {
  static_assert(NR % (2 * W) == 0, "rows in pairs");
#pragma unroll
  for (int i0 = 0; i0 < NR / W; i0 += 2) {
    uint2 w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = warp + (i0 + i) * W;
      w[i] = make_uint2(0, 0);
      if (r < R.rows && lane < D / 4)
        w[i] = *reinterpret_cast<const uint2*>(A.q + (int64_t)(R.a + r / A.G) * A.q_stride + (int64_t)(h * A.G + r % A.G) * D + 4 * lane);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = warp + (i0 + i) * W;
      const float v0 = load16<DT>((uint16_t)w[i].x), v1 = load16<DT>((uint16_t)(w[i].x >> 16));
      const float v2 = load16<DT>((uint16_t)w[i].y), v3 = load16<DT>((uint16_t)(w[i].y >> 16));
      float top = fmaxf(fmaxf(fabsf(v0), fabsf(v1)), fmaxf(fabsf(v2), fabsf(v3)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = query_exponent(top);
      // the factor is kept non-negative (maxima are taken before it): a negative scale turns the query instead
      const float down = copysignf(__uint_as_float((uint32_t)(127 - e) << 23), A.scale_log2);
      if (lane < D / 4) *reinterpret_cast<uint2*>(sq + r * (D + 8) + 4 * lane) = make_uint2(pack_half2(v0 * down, v1 * down), pack_half2(v2 * down, v3 * down));
      if (lane == 0) sf[r] = __uint_as_float((uint32_t)(127 + e) << 23) * fabsf(A.scale_log2);
    }
  }
}

// Few rows: up to 8 NB rows of one (request, kv head) against a range of its tokens.
// Bound by the cache's bytes, so the products run on mma.sync with the codes as the
// 16-row operand and the few rows as its 8 columns: S^T = K Q^T, O^T = V^T P^T (half
// the MMAs and accumulators of the other way round).  Each of the 4 warps takes every
// fourth tile of 32 tokens through a ring of its own (bulk copies, no barrier between
// warps) and keeps its own m, l and accumulator; the warps' results are joined at the
// end.  Few (request, kv head) cells: a cluster of CTAs shares a cell's tokens evenly and
// joins in shared memory (paged_rows_kernel).  Many cells, or long ones: the balanced
// schedule (paged_flat_kernel).  The fragments are read straight from the codes: the order of the
// contraction over d is free, so 16 bytes of a key row serve 4 k-steps, and 16 bytes
// of four value rows the 16 values of d that a lane needs.  One request of 333 tokens, 32
// heads: 7.1 us, a chain of loads (lengths, table, scales, codes) and two joins.
constexpr int kDecWarps = 4, kDecTile = 32, kDecStages = 2, kDecGroup = 32, kMaxCluster = 8;
constexpr int dec_stage_bytes(int D) { return kDecTile * D * 2; }
constexpr int dec_ring_bytes(int D) { return kDecWarps * kDecStages * dec_stage_bytes(D); }
struct DecMeta { float sk[2], sv[2]; };
constexpr int dec_smem(int D, int NB) {
  return dec_ring_bytes(D) + 8 * NB * (D + 8) * 2 + kDecWarps * 2 * kDecGroup * (16 + 8) + kDecWarps * NB * 8 * 8 + 8 * NB * 4 +
         kDecWarps * kDecStages * 8;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

template <int DT>
__device__ __forceinline__ void store_row4(uint16_t* dst, const float4& v) {
  uint2 w;
  w.x = (uint32_t)store16<DT>(v.x) | ((uint32_t)store16<DT>(v.y) << 16);
  w.y = (uint32_t)store16<DT>(v.z) | ((uint32_t)store16<DT>(v.w) << 16);
  *reinterpret_cast<uint2*>(dst) = w;
}

// The same pair as half2_of, E4M3 by the conversion instruction: its value, NaN codes NaN.
template <int FMT, int HI>
__device__ __forceinline__ uint32_t value2_of(uint32_t w) {
  if constexpr (FMT == SVDQ_KV_INT8) {
    return half2_of<FMT, HI>(w);
  } else {
    uint32_t y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"((uint16_t)(HI ? w >> 16 : w & 0xFFFFu)));
    return y;
  }
}

// One warp's rows against its tokens: the query fragments, maxima, sums, accumulators.
template <int FMT, int D, int NB>
struct RowState {
  static constexpr int KC = D / 64, VW = D / 32;
  uint32_t qf[NB][D / 16][2];
  float f[NB][2], o[D / 16][NB][4], m[NB][2], l[NB][2], n[NB][2];
  int see[NB][2], clear, last;                                   // clear: tiles that end at or below it need no mask

  // Q^T fragments: k-step s covers d = 64 (s / 4) + 16 q4 + 4 (s % 4) + {0, 1 | 2, 3}
  __device__ __forceinline__ void start(const AttnArgs& A, const Rows& R, const __half* sq, const float* sf, int t_end, int lane) {
    const int g = lane >> 2, q4 = lane & 3;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const uint2 w = *reinterpret_cast<const uint2*>(sq + (nb * 8 + g) * (D + 8) + (s >> 2) * 64 + q4 * 16 + 4 * (s & 3));
        qf[nb][s][0] = w.x;
        qf[nb][s][1] = w.y;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = nb * 8 + 2 * q4 + i;
        f[nb][i] = sf[r];
        see[nb][i] = r < R.rows ? min(t_end, seen_by(A, R, r)) : t_end;
        m[nb][i] = n[nb][i] = -INFINITY;
        l[nb][i] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[j][nb][0] = o[j][nb][1] = o[j][nb][2] = o[j][nb][3] = 0.0f;
    }
    clear = min(t_end, seen_by(A, R, 0));
    last = t_end;
  }

  // 32 tokens from t on
  __device__ __forceinline__ void step(const uint8_t* kt, const uint8_t* vt, const DecMeta& md, const int2& id, int t, int lane) {
    const int g = lane >> 2, q4 = lane & 3;
  // x[mt][nb]: tokens 16 mt + g (0, 1) and + 8 (2, 3), rows 8 nb + 2 q4 + {0, 1}
    float x[2][NB][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) x[mt][nb][0] = x[mt][nb][1] = x[mt][nb][2] = x[mt][nb][3] = 0.0f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint4 lo = *reinterpret_cast<const uint4*>(kt + (mt * 16 + g) * D + c * 64 + q4 * 16);
        const uint4 hi = *reinterpret_cast<const uint4*>(kt + (mt * 16 + g + 8) * D + c * 64 + q4 * 16);
        const uint32_t u[4] = {lo.x, lo.y, lo.z, lo.w}, w[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t y = pre<FMT>(u[i]), z = pre<FMT>(w[i]);
          const uint32_t a[4] = {value2_of<FMT, 0>(y), value2_of<FMT, 0>(z), value2_of<FMT, 1>(y), value2_of<FMT, 1>(z)};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma16816(x[mt][nb], a, qf[nb][c * 4 + i][0], qf[nb][c * 4 + i][1]);
        }
      }
    }
    if (t + kDecTile > clear || id.x < 0 || id.y < 0) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const bool gone = (mt == 0 ? id.x : id.y) < 0;
        const int tt = t + mt * 16 + g;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (gone || tt >= see[nb][0]) x[mt][nb][0] = -INFINITY;
          if (gone || tt >= see[nb][1]) x[mt][nb][1] = -INFINITY;
          if (gone || tt + 8 >= see[nb][0]) x[mt][nb][2] = -INFINITY;
          if (gone || tt + 8 >= see[nb][1]) x[mt][nb][3] = -INFINITY;
        }
      }
    }
    // factors to units of log2 (-inf stays -inf in a block of zeros); a new reference only where a lane's
    // scores, or weighted magnitudes, grew by 2^kGrow: no exchange between lanes otherwise
    float fac[2][NB][2], top[NB][2], vtop[NB][2];
    const float e0 = scale_exponent(md.sv[0]), e1 = scale_exponent(md.sv[1]);
    bool grow = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fac[0][nb][i] = fmaxf(f[nb][i] * md.sk[0], FLT_MIN);
        fac[1][nb][i] = fmaxf(f[nb][i] * md.sk[1], FLT_MIN);
        const float x0 = fmaxf(x[0][nb][i], x[0][nb][i + 2]) * fac[0][nb][i], x1 = fmaxf(x[1][nb][i], x[1][nb][i + 2]) * fac[1][nb][i];
        top[nb][i] = fmaxf(x0, x1);
        vtop[nb][i] = fmaxf(x0 + e0, x1 + e1);
        grow = grow || top[nb][i] > m[nb][i] + kGrow || vtop[nb][i] > n[nb][i] + (kGrow + kRoom);
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) {
            top[nb][i] = fmaxf(top[nb][i], __shfl_xor_sync(0xffffffffu, top[nb][i], s));
            vtop[nb][i] = fmaxf(vtop[nb][i], __shfl_xor_sync(0xffffffffu, vtop[nb][i], s));
          }
          if (top[nb][i] > m[nb][i] + kGrow) {
            l[nb][i] *= ex2(m[nb][i] - top[nb][i]);
            m[nb][i] = top[nb][i];
          }
          b[i] = 1.0f;
          if (vtop[nb][i] > n[nb][i] + (kGrow + kRoom)) {
            b[i] = ex2(n[nb][i] - (vtop[nb][i] - kRoom));
            n[nb][i] = vtop[nb][i] - kRoom;
          }
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          o[j][nb][0] *= b[0]; o[j][nb][1] *= b[1]; o[j][nb][2] *= b[0]; o[j][nb][3] *= b[1];
        }
      }
    }
    uint32_t pb[2][NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float z0 = m[nb][0] == -INFINITY ? 0.0f : m[nb][0], z1 = m[nb][1] == -INFINITY ? 0.0f : m[nb][1];
      // -122 <= m - n <= 127: n is at most a score (m + kGrow) plus 122 - kRoom; where m was set, n became at least
      // m - 113 - kGrow - kRoom
      const float rel0 = ex2(fminf(z0 - n[nb][0], 127.0f)), rel1 = ex2(fminf(z1 - n[nb][1], 127.0f));
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        // finite, so that a weight of 0 stays 0 beside a scale that the row does not see
        const float w0 = fminf(md.sv[mt] * rel0, FLT_MAX), w1 = fminf(md.sv[mt] * rel1, FLT_MAX);
        const float p0 = ex2(fmaf(x[mt][nb][0], fac[mt][nb][0], -z0)), p1 = ex2(fmaf(x[mt][nb][1], fac[mt][nb][1], -z1));
        const float p2 = ex2(fmaf(x[mt][nb][2], fac[mt][nb][0], -z0)), p3 = ex2(fmaf(x[mt][nb][3], fac[mt][nb][1], -z1));
        l[nb][0] += p0 + p2;
        l[nb][1] += p1 + p3;
        // [token][row] -> [row][token]: the column operand of the second product
        pb[mt][nb][0] = transpose8x8(pack_half2(p0 * w0, p1 * w1));
        pb[mt][nb][1] = transpose8x8(pack_half2(p2 * w0, p3 * w1));
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t u[4][VW];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint8_t* row = vt + (s * 16 + 2 * q4 + (r & 1) + (r >> 1) * 8) * D + g * (D / 8);
        if constexpr (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(row);
          u[r][0] = pre<FMT>(w.x); u[r][1] = pre<FMT>(w.y); u[r][2] = pre<FMT>(w.z); u[r][3] = pre<FMT>(w.w);
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(row);
          u[r][0] = pre<FMT>(w.x); u[r][1] = pre<FMT>(w.y);
        }
      }
      const int there = (s == 0 ? id.x : id.y) < 0 ? 0 : last;
      if (FMT == SVDQ_KV_E4M3 && t + s * 16 + 16 > there) {   // what no token wrote may be NaN codes
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (t + s * 16 + 2 * q4 + (r & 1) + (r >> 1) * 8 >= there) {
#pragma unroll
            for (int w = 0; w < VW; ++w) u[r][w] = 0;
          }
      }
      // accumulator tile j: operand row n is d = (D / 8) n + 2 j, row n + 8 the d after it
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        const uint32_t la = __byte_perm(u[0][w], u[1][w], 0x5140), ha = __byte_perm(u[0][w], u[1][w], 0x7362);
        const uint32_t lb = __byte_perm(u[2][w], u[3][w], 0x5140), hb = __byte_perm(u[2][w], u[3][w], 0x7362);
        const uint32_t a0[4] = {value2_of<FMT, 0>(la), value2_of<FMT, 1>(la), value2_of<FMT, 0>(lb), value2_of<FMT, 1>(lb)};
        const uint32_t a1[4] = {value2_of<FMT, 0>(ha), value2_of<FMT, 1>(ha), value2_of<FMT, 0>(hb), value2_of<FMT, 1>(hb)};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          mma16816(o[2 * w][nb], a0, pb[s][nb][0], pb[s][nb][1]);
          mma16816(o[2 * w + 1][nb], a1, pb[s][nb][0], pb[s][nb][1]);
        }
      }
    }
  }

  // Sums over the warp's lanes; maxima and sums to wml (this warp's NR entries).
  __device__ __forceinline__ void publish(float2* wml, int lane) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], s);
        if (lane < 4) wml[nb * 8 + 2 * lane + i] = make_float2(m[nb][i], l[nb][i]);
      }
  }
};

template <int DT, int FMT, int D, int NB>
__global__ void __launch_bounds__(kDecWarps * 32) paged_rows_kernel(const AttnArgs A) {
  constexpr int NST = kDecStages, kStage = dec_stage_bytes(D), NR = 8 * NB;
  extern __shared__ __align__(128) uint8_t dsm[];
  uint8_t* ring = dsm;
  __half* sq = reinterpret_cast<__half*>(dsm + dec_ring_bytes(D));
  DecMeta* meta = reinterpret_cast<DecMeta*>(sq + NR * (D + 8));           // [warp][2 groups]
  int2* ids = reinterpret_cast<int2*>(meta + kDecWarps * 2 * kDecGroup);   // [warp][2 groups]
  float2* wml = reinterpret_cast<float2*>(ids + kDecWarps * 2 * kDecGroup);  // [warp][NR]
  float* sf = reinterpret_cast<float*>(wml + kDecWarps * NR);              // [NR]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sf + NR);                   // [warp][NST]
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  const int h = blockIdx.y, req = blockIdx.z, split = blockIdx.x;
  griddep_wait();
  griddep_launch();
  const Rows R = request_rows(A, req, tid == 0);
  if (R.rows == 0) return;
  // the cluster shares what the rows see
  const int vis = seen_by(A, R, R.rows - 1), chunk = ((vis + A.splits - 1) / A.splits + kDecTile - 1) / kDecTile * kDecTile;
  const int t_begin = split * chunk, t_end = max(t_begin, min(vis, t_begin + chunk));
  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < kDecWarps * NST; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const int tiles = (t_end - t_begin + kDecTile - 1) / kDecTile;
  const int mine = tiles > warp ? (tiles - warp + kDecWarps - 1) / kDecWarps : 0;
  const int nblk = blocks_of(t_end, A.lb);
  uint8_t* wring = ring + warp * NST * kStage;
  uint64_t* wbar = bars + warp * NST;
  DecMeta* wmeta = meta + warp * 2 * kDecGroup;
  int2* wids = ids + warp * 2 * kDecGroup;
  const size_t blk_bytes = (size_t)(D << A.lb);

  // block ids and scales of kDecGroup tiles at a time, a lane each
  const auto load_group = [&](int k0) {
    const int k = k0 + lane;
    if (lane < kDecGroup) {
      int2 id = make_int2(-1, -1);
      DecMeta m = {{0.0f, 0.0f}, {0.0f, 0.0f}};
      if (k < mine) {
        const int t = t_begin + (warp + kDecWarps * k) * kDecTile, c0 = t >> A.lb, c1 = (t + 16) >> A.lb;
        const int* row = A.table + (size_t)req * A.max_blocks;
        id.x = pool_block(A, row[c0]);
        id.y = c1 == c0 ? id.x : (c1 < nblk ? pool_block(A, row[c1]) : -1);
        if (id.x >= 0) { const size_t c = (size_t)id.x * A.kv + h; m.sk[0] = A.ks[c]; m.sv[0] = A.vs[c]; }
        if (id.y >= 0) { const size_t c = (size_t)id.y * A.kv + h; m.sk[1] = A.ks[c]; m.sv[1] = A.vs[c]; }
      }
      wids[k & (2 * kDecGroup - 1)] = id;
      wmeta[k & (2 * kDecGroup - 1)] = m;
    }
    __syncwarp();
  };
  const auto issue = [&](int k) {
    if ((k & (kDecGroup - 1)) == 0) load_group(k);
    if (lane == 0) {
      const int t = t_begin + (warp + kDecWarps * k) * kDecTile, o = t & ((1 << A.lb) - 1);
      const int2 id = wids[k & (2 * kDecGroup - 1)];
      uint8_t* dst = wring + (k % NST) * kStage;
      uint64_t* bar = &wbar[k % NST];
      if (A.lb >= 5) {
        mbar_arrive_expect_tx(bar, id.x >= 0 ? 2 * kDecTile * D : 0);
        if (id.x >= 0) {
          const size_t at = ((size_t)id.x * A.kv + h) * blk_bytes + (size_t)o * D;
          bulk_load(dst, A.kc + at, kDecTile * D, bar);
          bulk_load(dst + kDecTile * D, A.vc + at, kDecTile * D, bar);
        }
      } else {
        mbar_arrive_expect_tx(bar, (id.x >= 0 ? kDecTile * D : 0) + (id.y >= 0 ? kDecTile * D : 0));
        if (id.x >= 0) {
          const size_t at = ((size_t)id.x * A.kv + h) * blk_bytes;
          bulk_load(dst, A.kc + at, 16 * D, bar);
          bulk_load(dst + kDecTile * D, A.vc + at, 16 * D, bar);
        }
        if (id.y >= 0) {
          const size_t at = ((size_t)id.y * A.kv + h) * blk_bytes;
          bulk_load(dst + 16 * D, A.kc + at, 16 * D, bar);
          bulk_load(dst + kDecTile * D + 16 * D, A.vc + at, 16 * D, bar);
        }
      }
    }
  };
  for (int k = 0; k < min(mine, NST); ++k) issue(k);

  load_queries<DT, D, NR, kDecWarps>(A, R, h, sq, sf, warp, lane);
  __syncthreads();
  RowState<FMT, D, NB> S;
  S.start(A, R, sq, sf, t_end, lane);

  for (int k = 0; k < mine; ++k) {
    const int st = k % NST, t = t_begin + (warp + kDecWarps * k) * kDecTile;
    if (!mbar_wait(&wbar[st], (k / NST) & 1, &s_abort)) {
      int own = 0;                                       // the copies in flight end before the CTA does
      for (int i = k; i < min(mine, k + NST); ++i) mbar_wait(&wbar[i % NST], (i / NST) & 1, &own);
      break;
    }
    const uint8_t* kt = wring + st * kStage;
    const uint8_t* vt = kt + kDecTile * D;
    S.step(kt, vt, wmeta[k & (2 * kDecGroup - 1)], wids[k & (2 * kDecGroup - 1)], t, lane);
    __syncwarp();
    if (k + NST < mine) issue(k + NST);
  }
  // join the four warps: each one's share of the CTA's rows
  S.publish(wml + warp * NR, lane);
  __syncthreads();                                       // every ring is free: the accumulators go there
  constexpr int AP = D + 4;                              // row pitch of the accumulators
  float* acc = reinterpret_cast<float*>(ring);           // [warp][NR][AP]
  float* mine_o = acc + kDecWarps * NR * AP;             // [NR][D]: this CTA's joined rows
  float2* mine_ml = reinterpret_cast<float2*>(mine_o + NR * D);
  static_assert((kDecWarps * NR * AP + NR * D + 2 * NR) * 4 <= dec_ring_bytes(D), "the join fits the ring");
  const auto total = [&](int r) {                        // maximum and sum of row r over the warps
    float2 y = make_float2(-INFINITY, 0.0f);
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) y.x = fmaxf(y.x, wml[w * NR + r].x);
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float2 u = wml[w * NR + r];
      y.y += u.x == -INFINITY ? 0.0f : ex2(u.x - y.x) * u.y;
    }
    return y;
  };
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = nb * 8 + 2 * q4 + i;
      const float2 ml = total(r), u = result_factors(S.n[nb][i], ml.x, ml.y);
      float* p = acc + (warp * NR + r) * AP + (D / 8) * g;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        *reinterpret_cast<float2*>(p + 2 * j) = make_float2(S.o[j][nb][i] * u.x * u.y, S.o[j][nb][i + 2] * u.x * u.y);
    }
  __syncthreads();
  for (int idx = tid; idx < NR * D / 4; idx += kDecWarps * 32) {
    const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
    if (r >= R.rows) break;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(acc + (w * NR + r) * AP + d);
      v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
    }
    *reinterpret_cast<float4*>(mine_o + r * D + d) = v;
    if (d == 0) mine_ml[r] = total(r);
  }
  // the cluster's CTAs in rank order, each taking its share of the values
  cluster_sync();
  const uint32_t o_at = smem_u32(mine_o), ml_at = smem_u32(mine_ml);
  for (int idx = split * (kDecWarps * 32) + tid; idx < NR * D / 4; idx += A.splits * kDecWarps * 32) {
    const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
    if (r >= R.rows) break;
    float2 ml[kMaxCluster];
    float M = -INFINITY, L = 0.0f;
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) {
      ml[s] = s < A.splits ? ld_cluster_f32x2(mapa_shared(ml_at + 8 * r, s)) : make_float2(-INFINITY, 0.0f);
      M = fmaxf(M, ml[s].x);
    }
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) {
      ml[s].y *= ml[s].x == -INFINITY ? 0.0f : ex2(ml[s].x - M);
      L += ml[s].y;
    }
    const float inv = L > 0.0f ? __frcp_rn(L) : 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) {
      if (s < A.splits) {
        const float w = ml[s].y * inv;
        const float4 y = ld_cluster_f32x4(mapa_shared(o_at + (r * D + d) * 4, s));
        v.x += w * y.x; v.y += w * y.y; v.z += w * y.z; v.w += w * y.w;
      }
    }
    const int token = R.a + r / A.G, head = h * A.G + r % A.G;
    store_row4<DT>(A.out + (int64_t)token * A.out_stride + (int64_t)head * D + d, v);
  }
  cluster_sync();                                        // nobody leaves while its rows are read
}

// ------------------------------------------------------- balanced schedule
// The calls' lengths are known on the device only, so every CTA works out its own
// share.  An item is `cr` rows of one (request, kv head); its cost is what its last
// row sees plus a tile for filling and emptying the pipeline, times G:
//   c_r = G (P + 128) + cr (r + 1) [causal],  P = L - n (causal) or L
// which sums in closed form over the row blocks r of a head, the heads and the
// requests.  CTA c of N takes the costs [T c / N, T (c + 1) / N); a border inside an
// item cuts its token tiles in proportion.  The two pieces of a cut item go to the
// workspace and paged_join_kernel joins them; everything else is written directly.
// Measured against a grid of (item, fixed split) when it was brought in: six ragged prompts, whose
// rows see 2 to 12 tiles, 283 -> 209 us; 256 equal items on 148 SMs took two full waves (782 -> 610 us).
constexpr int kTileTok = 128, kTileRows = 256;
struct Item {
  int req, h, a, n, L, rows, r0, lo, hi, out;              // token tiles [lo, hi); hi < 0: no more items
  int end[2];                                              // where the row tiles' token tiles end
};
enum { kItemWhole = 2 };                                   // out: 0, 1 a piece's slot in the workspace
struct Piece { int valid, last, token, n_rows, h, r0, pad0, pad1; };

__device__ __forceinline__ int64_t item_base(const AttnArgs& A, const Rows& R) {
  return (int64_t)A.G * ((A.causal ? max(0, R.L - R.n) : R.L) + kTileTok);
}
__device__ __forceinline__ int64_t head_cost(const AttnArgs& A, const Rows& R, int64_t r, int cr) {   // row blocks [0, r)
  return r * item_base(A, R) + (A.causal ? cr * (r * (r + 1) / 2) : 0);
}
__device__ __forceinline__ int64_t request_cost(const AttnArgs& A, const Rows& R, int cr) {
  return R.rows == 0 ? 0 : A.kv * head_cost(A, R, (R.rows + cr - 1) / cr, cr);
}

// A CTA's range of costs and the request that holds its start.  Called by all
// threads of the CTA; ends with a barrier.
struct Share { long long x0, x1, at; int req; };
template <int THREADS>
__device__ __forceinline__ Share cta_share(const AttnArgs& A, int cr, int part, int parts) {
  constexpr int W = THREADS / 32;
  __shared__ long long s_sum[W];
  __shared__ Share s_share;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const auto cost = [&](int i, bool note) { return i < A.B ? (long long)request_cost(A, request_rows(A, i, note), cr) : 0ll; };
  const long long first = cost(tid, part == 0);
  long long v = first;
  for (int i = tid + THREADS; i < A.B; i += THREADS) v += cost(i, part == 0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) s_sum[warp] = v;
  if (tid == 0) s_share.req = -1;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) total += s_sum[w];
  // a border is the same number for the CTAs on its two sides, which is all that it has to be
  const auto border = [&](int p) { return p == parts ? total : (long long)((double)total * (p * A.inv_parts)); };
  const long long x0 = border(part), x1 = border(part + 1);
  long long before = 0;
  for (int i0 = 0; i0 < A.B && before <= x0; i0 += THREADS) {
    const long long c = i0 == 0 ? first : cost(i0 + tid, false);
    long long p = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, p, o);
      if (lane >= o) p += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = p;
    __syncthreads();
    long long at = before + p - c;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) at += s_sum[w];
      before += s_sum[w];
    }
    if (at <= x0 && x0 < at + c) s_share = Share{x0, x1, at, i0 + tid};
  }
  __syncthreads();
  return s_share;
}

// The items of a share, one after another (by a converged warp).
struct Walk {
  Rows R;
  long long s, base;                                       // cost where the present item starts
  int req, h, r, nr;
  __device__ __forceinline__ void enter(const AttnArgs& A, int cr) {
    base = item_base(A, R);
    nr = (R.rows + cr - 1) / cr;
    h = r = 0;
  }
  __device__ __forceinline__ void start(const AttnArgs& A, const Share& S, int cr) {
    req = S.req;
    R = request_rows(A, req, false);
    enter(A, cr);
    const long long head = head_cost(A, R, nr, cr);
    long long y = S.x0 - S.at;
    h = (int)((double)y / (double)head);                   // within one of the quotient
    h -= (long long)h * head > y;
    h += (long long)(h + 1) * head <= y;
    y -= h * head;
    int hi = nr - 1;                                       // the last row block that starts at or below y
    while (r < hi) {
      const int mid = r + (hi - r + 1) / 2;
      if (head_cost(A, R, mid, cr) <= y) r = mid; else hi = mid - 1;
    }
    s = S.at + h * head + head_cost(A, R, r, cr);
  }
  // The present item's part of the share, then one step on; false past the share's end.
  __device__ __forceinline__ bool next(const AttnArgs& A, const Share& S, int cr, Item& it) {
    while (s < S.x1) {
      const long long c = base + (A.causal ? (long long)cr * (r + 1) : 0);
      const int vis = seen_by(A, R, min(R.rows, (r + 1) * cr) - 1), tiles = (vis + kTileTok - 1) / kTileTok;
      const auto cut = [&](long long x) { return min(tiles, (int)((double)(x - s) * tiles / (double)c)); };
      const int lo = s >= S.x0 ? 0 : A.snap ? tiles : cut(S.x0), hi = s + c <= S.x1 || A.snap ? tiles : cut(S.x1);
      const bool mine = tiles == 0 ? s >= S.x0 : hi > lo;
      it = Item{req, h, R.a, R.n, R.L, R.rows, r * cr, lo, hi, lo == 0 && hi == tiles ? (int)kItemWhole : (lo == 0 ? 1 : 0), {hi, lo}};
      if (cr == kTileRows) {
        const int first = r * cr, t0 = (seen_by(A, R, min(R.rows, first + 128) - 1) + kTileTok - 1) / kTileTok;
        it.end[0] = max(lo, min(hi, t0));
        if (first + 128 < R.rows) it.end[1] = hi;
      }
      s += c;
      if (++r == nr) {
        r = 0;
        if (++h == A.kv) {
          // the next request with rows, 32 at a time
          uint32_t some = 0;
          for (++req; req < A.B; req += 32) {
            const int i = req + (threadIdx.x & 31);
            some = __ballot_sync(0xffffffffu, i < A.B && request_rows(A, i, false).rows > 0);
            if (some) break;
          }
          if (some) {
            req += __ffs(some) - 1;
            R = request_rows(A, req, false);
            enter(A, cr);
          } else {
            s = S.x1;
          }
        }
      }
      if (mine) return true;
    }
    return false;
  }
};

// Few rows on the balanced schedule: every CTA streams its share of all tokens, item
// after item, the next item's tiles already on their way while one is finished.  A warp
// takes the 32 tokens at 32 w of each 128-token tile.  Pieces of cut items go to the
// workspace for paged_join_kernel; where A.snap is set items are not cut, and belong to
// the CTA in whose share they start.  64 requests of up to 4096 tokens (346 MB of int8
// codes): 71 us, 4.9 TB/s; one of 131071 (268 MB of E4M3): 57 us.  Beyond HBM's rate it
// pays the first chain of loads, 5 us, queries and joins, and bank conflicts: value rows of
// 128 bytes are read four lanes to a bank, key rows two, over a quarter of the kernel's cycles
// by the counter.  Tiles of 16 tokens in 16 warps an SM instead of 32 in 12: 89 and 62 us
// (against 80 and 60 then).
template <int D, int NB>
struct FlatSmem {
  uint8_t ring[dec_ring_bytes(D)];
  union {
    float sum[8 * NB][D + 4];                              // value d = (D / 8) g + 2 j + e at 2 (8 j + g) + e
    __half q[8 * NB][D + 8];
  };
  DecMeta meta[kDecWarps][2 * kDecGroup];
  int2 ids[kDecWarps][2 * kDecGroup];
  float2 ml[kDecWarps][8 * NB], total[8 * NB];
  float f[8 * NB];
  uint64_t bars[kDecWarps][kDecStages];
  int abort;
};

// CTAs an SM, which the schedule is sized by: four with 64 values a head and 8 rows; the accumulators of 16 rows, or
// the ring of 128 values, leave three, both two.  The launch bounds hold the compiler to it, the assertion the ring.
// 64 requests of up to 4096 tokens, 4 heads of 64 values, 16 query heads each: 47 us where a grid for four CTAs an SM, of
// which three fit, took 53, and one request of 131071 tokens 35 instead of 48 (41.5 and 34 us now).
constexpr int flat_per_sm(int head_dim, int rows) { return 4 - (head_dim > 64) - (rows > 8); }
constexpr int kSmemPerSm = 228 * 1024, kSmemPerCta = 1024;   // what an SM has, and what it takes for itself for each CTA

template <int DT, int FMT, int D, int NB>
__global__ void __launch_bounds__(kDecWarps * 32, flat_per_sm(D, 8 * NB)) paged_flat_kernel(const AttnArgs A) {
  static_assert(flat_per_sm(D, 8 * NB) * (sizeof(FlatSmem<D, NB>) + kSmemPerCta + 256) <= kSmemPerSm, "the rings fit");
  constexpr int NST = kDecStages, kStage = dec_stage_bytes(D), NR = 8 * NB;
  extern __shared__ __align__(128) uint8_t dsm[];
  FlatSmem<D, NB>& X = *reinterpret_cast<FlatSmem<D, NB>*>(dsm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    X.abort = 0;
    for (int s = 0; s < kDecWarps * NST; ++s) mbar_init(&X.bars[0][0] + s, 1);
    fence_mbar_init();
  }
  griddep_wait();
  griddep_launch();
  const Share share = cta_share<kDecWarps * 32>(A, NR, blockIdx.x, gridDim.x);   // ends with a barrier
  if (tid < 2 && A.pieces) A.pieces[blockIdx.x * 2 + tid].valid = 0;
  __syncthreads();
  if (share.req < 0) return;
  uint8_t* ring = X.ring + warp * NST * kStage;
  uint64_t* bar = X.bars[warp];
  DecMeta* meta = X.meta[warp];
  int2* ids = X.ids[warp];
  const size_t blk_bytes = (size_t)(D << A.lb);
  const auto end_of = [&](const Item& I) {                 // tokens that the piece's rows see
    const Rows R = {I.a, I.n, I.L, I.rows};
    return min(seen_by(A, R, I.rows - 1), I.hi * kTileTok);
  };

  // the tiles on their way: `sent` so far, the next one at token `t` of the item below `t_end`
  Walk ahead;
  ahead.start(A, share, NR);
  Walk walk = ahead;
  int sent = 0, t = 0, t_end = 0, h = 0, grouped = 0;
  const int* row = nullptr;
  const auto send = [&]() {
    while (t >= t_end) {
      Item I;
      if (!ahead.next(A, share, NR, I)) { t = 0; t_end = -1; return; }
      t = I.lo * kTileTok + 32 * warp;
      t_end = end_of(I);
      h = I.h;
      row = A.table + (size_t)I.req * A.max_blocks;
      grouped = 0;
    }
    if (grouped == 0) {                                    // block numbers and scales of the next tiles, a lane each
      const int tt = t + lane * kTileTok;
      if (lane < kDecGroup) {
        int2 id = make_int2(-1, -1);
        DecMeta m = {{0.0f, 0.0f}, {0.0f, 0.0f}};
        if (tt < t_end) {
          const int nblk = blocks_of(t_end, A.lb), c0 = tt >> A.lb, c1 = (tt + 16) >> A.lb;
          id.x = pool_block(A, row[c0]);
          id.y = c1 == c0 ? id.x : (c1 < nblk ? pool_block(A, row[c1]) : -1);
          if (id.x >= 0) { const size_t c = (size_t)id.x * A.kv + h; m.sk[0] = A.ks[c]; m.sv[0] = A.vs[c]; }
          if (id.y >= 0) { const size_t c = (size_t)id.y * A.kv + h; m.sk[1] = A.ks[c]; m.sv[1] = A.vs[c]; }
        }
        ids[(sent + lane) & (2 * kDecGroup - 1)] = id;
        meta[(sent + lane) & (2 * kDecGroup - 1)] = m;
      }
      grouped = kDecGroup;
      __syncwarp();
    }
    if (lane == 0) {
      const int o = t & ((1 << A.lb) - 1);
      const int2 id = ids[sent & (2 * kDecGroup - 1)];
      uint8_t* dst = ring + (sent % NST) * kStage;
      uint64_t* b = &bar[sent % NST];
      const int x = A.lb >= 5 ? 2 : 1;                     // halves of a tile that one copy brings
      mbar_arrive_expect_tx(b, ((id.x >= 0 ? x : 0) + (x == 1 && id.y >= 0 ? 1 : 0)) * 32 * D);
      if (id.x >= 0) {
        const size_t at = ((size_t)id.x * A.kv + h) * blk_bytes + (size_t)o * D;
        bulk_load(dst, A.kc + at, 16 * x * D, b);
        bulk_load(dst + kDecTile * D, A.vc + at, 16 * x * D, b);
      }
      if (x == 1 && id.y >= 0) {
        const size_t at = ((size_t)id.y * A.kv + h) * blk_bytes;
        bulk_load(dst + 16 * D, A.kc + at, 16 * D, b);
        bulk_load(dst + kDecTile * D + 16 * D, A.vc + at, 16 * D, b);
      }
    }
    ++sent;
    --grouped;
    t += kTileTok;
  };
  for (int s = 0; s < NST; ++s) send();

  Item I;
  int done = 0;
  bool dead = false;
  RowState<FMT, D, NB> S;
  while (walk.next(A, share, NR, I)) {
    const Rows R = {I.a, I.n, I.L, I.rows};
    const int end = end_of(I);
    __syncthreads();                                       // the sums of the item before are read
    load_queries<DT, D, NR, kDecWarps>(A, R, I.h, &X.q[0][0], X.f, warp, lane);
    __syncthreads();
    S.start(A, R, &X.q[0][0], X.f, end, lane);
    for (int at = I.lo * kTileTok + 32 * warp; at < end && !dead; at += kTileTok, ++done) {
      if (!mbar_wait(&bar[done % NST], (done / NST) & 1, &X.abort)) {
        int own = 0;                                       // the copies in flight end before the CTA does
        for (int i = done; i < sent; ++i) mbar_wait(&bar[i % NST], (i / NST) & 1, &own);
        dead = true;
        break;
      }
      const uint8_t* kt = ring + (done % NST) * kStage;
      S.step(kt, kt + kDecTile * D, meta[done & (2 * kDecGroup - 1)], ids[done & (2 * kDecGroup - 1)], at, lane);
      __syncwarp();
      send();
    }
    // join the four warps in order: each one's share of the rows
    S.publish(X.ml[warp], lane);
    __syncthreads();
    // maximum and sum of row `tid` over the warps: once, not by every lane at each use (64 requests: 74.9 -> 71.5 us)
    if (tid < NR) {
      const float M = fmaxf(fmaxf(X.ml[0][tid].x, X.ml[1][tid].x), fmaxf(X.ml[2][tid].x, X.ml[3][tid].x));
      float L = 0.0f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) L += X.ml[w][tid].x == -INFINITY ? 0.0f : ex2(X.ml[w][tid].x - M) * X.ml[w][tid].y;
      X.total[tid] = make_float2(M, L);
    }
    __syncthreads();
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 ml = X.total[nb * 8 + 2 * (lane & 3) + i];
        const float2 u = result_factors(S.n[nb][i], ml.x, ml.y);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          S.o[j][nb][i] = S.o[j][nb][i] * u.x * u.y;
          S.o[j][nb][i + 2] = S.o[j][nb][i + 2] * u.x * u.y;
        }
      }
    static_assert(kDecWarps == 4, "the join is written for four warps");
#pragma unroll 1
    for (int w = 0; w < kDecWarps; ++w) {
      if (warp == w) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = nb * 8 + 2 * (lane & 3) + i;
            // rows 16 bytes and lanes 8 bytes apart: no two lanes of a half warp on one bank
            float2* p = reinterpret_cast<float2*>(&X.sum[r][2 * (lane >> 2)]);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              const float2 v = w == 0 ? make_float2(0.0f, 0.0f) : p[8 * j];
              p[8 * j] = make_float2(v.x + S.o[j][nb][i], v.y + S.o[j][nb][i + 2]);
            }
          }
      }
      __syncthreads();
    }
    const int tiles = (seen_by(A, R, R.rows - 1) + kTileTok - 1) / kTileTok;
    if (tid == 0 && I.out != kItemWhole) A.pieces[blockIdx.x * 2 + I.out] = Piece{1, I.hi == tiles, I.a, I.rows, I.h, 0, 0, 0};
    for (int idx = tid; idx < NR * D / 4; idx += kDecWarps * 32) {
      const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
      if (r >= R.rows) break;
      const int at = 2 * (4 * (d % (D / 8)) + d / (D / 8));
      const float2 v0 = *reinterpret_cast<const float2*>(&X.sum[r][at]), v1 = *reinterpret_cast<const float2*>(&X.sum[r][at + 16]);
      const float4 v = make_float4(v0.x, v0.y, v1.x, v1.y);
      if (I.out == kItemWhole) {
        const int token = R.a + r / A.G, head = I.h * A.G + r % A.G;
        store_row4<DT>(A.out + (int64_t)token * A.out_stride + (int64_t)head * D + d, v);
      } else {
        const size_t cell = ((size_t)blockIdx.x * 2 + I.out) * NR + r;
        *reinterpret_cast<float4*>(A.part_o + cell * D + d) = v;
        if (d == 0) *reinterpret_cast<float2*>(A.part_ml + cell * 2) = X.total[r];
      }
    }
  }
}

// Many rows: items of 256 rows (two tiles of 128) on the tensor cores, one CTA per SM
// that works through its share without a break between items.  Codes become fp16
// operands in shared memory once per 128 tokens and serve both row tiles: S = Q K^T
// (both operands from shared memory, 128 x 128 fp32 in TMEM), P in fp16 over S's own
// columns, O += P V (P from TMEM; V as it lies, token rows of 64 d, an MN-major
// operand).  Roles:
//   warps 0-3, 4-7   softmax of row tile 0 / 1, a row per thread: maximum, weights,
//                    sum; rescales O only when the largest weighted magnitude grew
//                    by more than 2^7; the next item's queries; output
//   warps 8-11       codes -> fp16 (the next tile's codes already in registers)
//   warp 12          issues the MMAs: S0 S1 | P0V S0' | P1V S1' | ...
//   warp 13          walks the schedule, up to eight items ahead; writes the zeros of
//                    rows that see nothing.  Every item in the ring has a token tile: behind
//                    eight without, the MMA warp would wait for an item that the softmax
//                    warps hold back until it has served them
// The value scale goes into a weight's exponent, p' = 2^(x + log2 s_v - n), so it costs
// nothing per weight; the row sum takes each 16 tokens' sum times 2^(n - m) / s_v.
// 2048 rows x 32 heads at 16384 tokens, d = 128: 598 us, 862 TFLOP/s; as a call 658 us.  No unit
// is full: of about 4700 cycles that two row tiles take for 128 tokens, the products and the
// exponentials take 2048 each and the issue slots half; the rest are waits of the roles for one
// another, which two row tiles do not cover.  144, 128 and 96 registers, no spills (a spilled
// value missed what is left of L1 and cost 600 cycles).
constexpr int kTileThreads = 512, kTileMeta = 4, kItems = 8;
struct __align__(16) TileMeta { float sk, lsv; int gone, pad; };   // 16 tokens: key scale, log2 of the value scale
constexpr int kTileHalf = 128 * 128;                      // 128 rows of 64 fp16, 128-byte swizzle
constexpr int tile_bytes(int D) { return D / 64 * kTileHalf; }
constexpr int tiles_smem(int D) {
  return 6 * tile_bytes(D) + kTileRows * 4 + kTileMeta * 8 * 16 + kItems * (int)sizeof(Item) + 512 + 1024;
}

// MN-major operand with the 128-byte swizzle: rows of 64 values (128 bytes) along K,
// 8-row groups 1024 bytes apart, the next 64 values of MN kTileHalf further.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(kTileHalf >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// D[tmem] (+)= A[tmem] * B[smem], fp16 operands, fp32 accumulate.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// 2^d for a whole number d <= 0 (0 below the normal numbers).
__device__ __forceinline__ float power_of_two(float d) { return __uint_as_float((uint32_t)(max((int)d, -127) + 127) << 23); }

// threadIdx.x, read where it stands: what is computed from it is not kept in registers across the loops before.
__device__ __forceinline__ int tid_here() {
  int t;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
  return t;
}

// One lane of a converged warp; the compiler knows that the choice is uniform.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// 16 code bytes to 16 fp16 at columns 16 c .. of row r of an operand tile.
template <int FMT>
__device__ __forceinline__ void store_codes(uint8_t* tile, int r, int half, int c, const uint4& w) {
  const uint32_t u[4] = {pre<FMT>(w.x), pre<FMT>(w.y), pre<FMT>(w.z), pre<FMT>(w.w)};
  uint8_t* row = tile + half * kTileHalf + r * 128;
  *reinterpret_cast<uint4*>(row + (((2 * c) ^ (r & 7)) << 4)) =
      make_uint4(half2_of<FMT, 0>(u[0]), half2_of<FMT, 1>(u[0]), half2_of<FMT, 0>(u[1]), half2_of<FMT, 1>(u[1]));
  *reinterpret_cast<uint4*>(row + (((2 * c + 1) ^ (r & 7)) << 4)) =
      make_uint4(half2_of<FMT, 0>(u[2]), half2_of<FMT, 1>(u[2]), half2_of<FMT, 0>(u[3]), half2_of<FMT, 1>(u[3]));
}

// Codes are read once by an SM: they leave L1 to the block tables and scales.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Zeros for an item's rows, by one warp.
template <int D>
__device__ __forceinline__ void zero_rows(const AttnArgs& A, const Item& I) {
  constexpr int PER = D / 8;
  const int n = min(kTileRows, I.rows - I.r0) * PER;
  for (int x = threadIdx.x & 31; x < n; x += 32) {
    const int r = I.r0 + x / PER;
    *reinterpret_cast<uint4*>(A.out + (int64_t)(I.a + r / A.G) * A.out_stride + (int64_t)(I.h * A.G + r % A.G) * D + 8 * (x % PER)) = make_uint4(0, 0, 0, 0);
  }
}

template <int DT, int FMT, int D>
__global__ void __launch_bounds__(kTileThreads, 1) paged_tiles_kernel(const AttnArgs A) {
  constexpr int H = D / 64, TB = tile_bytes(D), kConsumers = 8 + 4 + 1;
  extern __shared__ uint8_t tsm_raw[];
  uint8_t* tsm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tsm_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sq = tsm;                                       // [2 row tiles]
  uint8_t* sk = sq + 2 * TB;                               // [2 stages]
  uint8_t* sv = sk + 2 * TB;                               // [2 stages]
  float* sf = reinterpret_cast<float*>(sv + 2 * TB);       // [256]
  TileMeta* meta = reinterpret_cast<TileMeta*>(sf + kTileRows);  // [kTileMeta][8]
  Item* items = reinterpret_cast<Item*>(meta + kTileMeta * 8);
  uint64_t* bars = reinterpret_cast<uint64_t*>(items + kItems);
  uint64_t *k_full = bars, *k_empty = bars + 2, *v_full = bars + 4, *v_empty = bars + 6, *s_full = bars + 8,
           *p_full = bars + 10, *o_full = bars + 12, *q_full = bars + 14, *p1_full = bars + 16,
           *o1_full = bars + 18, *i_full = bars + 20,
           *i_empty = i_full + kItems, *drained = i_empty + kItems;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 4);
      mbar_init(&v_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&p1_full[s], 4);
      mbar_init(&o1_full[s], 1);
      mbar_init(&o_full[s], 1);
      mbar_init(&q_full[s], 4);
    }
    for (int s = 0; s < kItems; ++s) {
      mbar_init(&i_full[s], 1);
      mbar_init(&i_empty[s], kConsumers);
    }
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  griddep_wait();
  // TMEM only now: a kernel before this one may still want its own, and would wait for ours
  if (warp == 12) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  const Share share = cta_share<kTileThreads>(A, kTileRows, blockIdx.x, gridDim.x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch();
  const uint32_t tm = s_tmem;
  // the k-th item, for one warp: false when there are no more; done with it: give_back
  const auto take = [&](int k) {
    return mbar_wait(&i_full[k % kItems], (k / kItems) & 1, &s_abort) && items[k % kItems].hi >= 0;
  };
  const auto give_back = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&i_empty[k % kItems]);
  };

  if (warp < 8) {
    regs_inc<144>();
    const int rt = warp >> 2, rl = tid & 127;
    const uint32_t ts = tm + rt * 128 + ((uint32_t)(warp & 3) << 21), to = tm + 256 + rt * D + ((uint32_t)(warp & 3) << 21);
    uint32_t n_s = 0, n_o = 0;                             // tiles and items of this row tile so far
    int flat = 0;                                          // token tiles of all items so far
    // An item's 32 rows of queries, normalised, as the A operand (16 or 8 lanes a row), and their factors.
    // The row tile's last S of the item before is done, so the operand is free.
    const auto queries = [&](const Item& N) {
      constexpr int PER = D / 8, RPI = 32 / PER, NQ = 8;                // rows in flight: NQ RPI
      if (N.end[rt] <= N.lo) return;
      const int here = tid_here(), c = here % PER, w0 = (here & 127) / 32 * 32 + here % 32 / PER, t0 = N.r0 / A.G, x0 = N.r0 - t0 * A.G + rt * 128 + w0;
      const uint16_t* q0 = A.q + (int64_t)(N.a + t0) * A.q_stride + (int64_t)N.h * A.G * D + 8 * c;
      uint8_t* dst = sq + rt * TB + (c >> 3) * kTileHalf;
#pragma unroll 1
      for (int b0 = 0; b0 < 32; b0 += NQ * RPI) {
      uint4 q[NQ];
#pragma unroll
      for (int b = 0; b < NQ; ++b) {
        const int x = x0 + b0 + b * RPI;
        const int dt = A.G == 1 ? x : (int)__umulhi((uint32_t)x, A.g_inv);   // x / G
        q[b] = make_uint4(0, 0, 0, 0);
        if (N.r0 + rt * 128 + w0 + b0 + b * RPI < N.rows) q[b] = *reinterpret_cast<const uint4*>(q0 + dt * A.q_stride + (int64_t)((x - dt * A.G) * D));
      }
#pragma unroll
      for (int b = 0; b < NQ; ++b) {
        const int rr = w0 + b0 + b * RPI;
        float v[8], top = 0.0f;
        unpack8<DT>(q[b], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
#pragma unroll
        for (int o = PER / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int e = query_exponent(top);
        // the factor is kept non-negative (maxima are taken before it): a negative scale turns the query instead
        const float down = copysignf(__uint_as_float((uint32_t)(127 - e) << 23), A.scale_log2);
        *reinterpret_cast<uint4*>(dst + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) =
            make_uint4(pack_half2(v[0] * down, v[1] * down), pack_half2(v[2] * down, v[3] * down),
                       pack_half2(v[4] * down, v[5] * down), pack_half2(v[6] * down, v[7] * down));
        if (c == 0) sf[rt * 128 + rr] = __uint_as_float((uint32_t)(127 + e) << 23) * fabsf(A.scale_log2) * kUnit<FMT>;
      }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[rt]);
    };
    int k = 0;
    bool some = take(0);
    if (some) queries(items[0]);
    while (some) {
      const Item& I = items[k % kItems];
      if (mbar_try_wait(&i_full[(k + 1) % kItems], ((k + 1) / kItems) & 1)) {   // the next item's queries, to L2
        const Item& N = items[(k + 1) % kItems];
        const int r = N.r0 + rt * 128 + rl;
        if (N.hi >= 0 && r < N.rows) {
          const uint16_t* row = A.q + (int64_t)(N.a + r / A.G) * A.q_stride + (int64_t)(N.h * A.G + r % A.G) * D;
          prefetch_l2(row);
          if (D == 128) prefetch_l2(row + 64);
        }
        __syncwarp();
      }
      const int lo = I.lo, end = I.end[rt], rows = I.rows - (I.r0 + rt * 128);   // rows of this row tile
      int see = INT_MAX, clear;
      {
        const Rows R = {I.a, I.n, I.L, I.rows};
        if (rl < rows) see = seen_by(A, R, I.r0 + rt * 128 + rl);
        clear = seen_by(A, R, I.r0 + rt * 128);
      }
      float m = -INFINITY, l = 0.0f, n = -INFINITY;
      const float f = sf[rt * 128 + rl];
      bool ok = true;
      for (int j = lo; j < end; ++j, ++n_s) {
        const int t = j * kTileTok;
        if (!(ok = mbar_wait(&s_full[rt], n_s & 1, &s_abort))) break;
        tc_fence_after();
        // 64 tokens at a time, whose products start while the next 64 are worked on; both references are
        // whole numbers, so that a growth rescales O and the sum by a power of two
        const TileMeta* M = meta + ((flat + j - lo) & (kTileMeta - 1)) * 8;
        uint32_t y[2][32];
#pragma unroll 1
        for (int q = 0; q < 2; ++q, M += 4) {
          const float4 M0 = reinterpret_cast<const float4*>(M)[0], M1 = reinterpret_cast<const float4*>(M)[1],
                       M2 = reinterpret_cast<const float4*>(M)[2], M3 = reinterpret_cast<const float4*>(M)[3];
          const auto sk_of = [&](int g) { return g == 0 ? M0.x : g == 1 ? M1.x : g == 2 ? M2.x : M3.x; };
          const auto lsv_of = [&](int g) { return g == 0 ? M0.y : g == 1 ? M1.y : g == 2 ? M2.y : M3.y; };
          const auto gone_of = [&](int g) { return __float_as_int(g == 0 ? M0.z : g == 1 ? M1.z : g == 2 ? M2.z : M3.z); };
          tmem_ld_32cols(ts + 64 * q, y[0]);
          tmem_ld_32cols(ts + 64 * q + 32, y[1]);
          tmem_ld_wait(y[0]);
          tmem_ld_wait(y[1]);
          const auto at = [&](int i) { return __uint_as_float(y[i >> 5][i & 31]); };
          if (t + 64 * q + 64 > clear || (gone_of(0) | gone_of(1) | gone_of(2) | gone_of(3))) {
            const int lim = see - t - 64 * q;
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= lim || gone_of(i >> 4)) y[i >> 5][i & 31] = __float_as_uint(-INFINITY);
          }
          float top = m, vtop = -INFINITY;
#pragma unroll
          for (int g = 0; g < 4; ++g) {                    // four chains: the unit is fast, its latency is not
            const int i = 16 * g;
            float t0 = fmaxf(fmaxf(at(i), at(i + 1)), at(i + 2)), t1 = fmaxf(fmaxf(at(i + 3), at(i + 4)), at(i + 5));
            float t2 = fmaxf(fmaxf(at(i + 6), at(i + 7)), at(i + 8)), t3 = fmaxf(fmaxf(at(i + 9), at(i + 10)), at(i + 11));
            t0 = fmaxf(fmaxf(t0, at(i + 12)), at(i + 13));
            t1 = fmaxf(fmaxf(t1, at(i + 14)), at(i + 15));
            // -inf stays -inf in a block of zeros
            const float x = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * fmaxf(f * sk_of(g), FLT_MIN);
            top = fmaxf(top, x);
            vtop = fmaxf(vtop, x + lsv_of(g));             // of what the row sees: -inf elsewhere
          }
          // new references only where one grew by 2^kGrow (or is the first)
          const bool grow = top > m + kGrow, vgrow = vtop > n + (kGrow + kRoom);   // -inf: any finite one
          if (__any_sync(0xffffffffu, grow || vgrow)) {
            const float m1 = grow ? ceilf(top) : m, n1 = vgrow ? ceilf(vtop) - kRoom : n;
            const float bo = n1 == n ? 1.0f : power_of_two(n - n1);
            l *= m1 == m ? 1.0f : power_of_two(m - m1);
            m = m1;
            n = n1;
            if (j > lo || q == 1) {
              // the first half's products of this tile may be under way
              if (q == 1 && !(ok = mbar_wait(&o1_full[rt], n_s & 1, &s_abort))) break;
              tc_fence_after();
#pragma unroll 1
              for (int e = 0; e < D / 8; ++e) {
                uint32_t o[8];
                tmem_ld_8cols(to + 8 * e, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * bo);
                tmem_st_8cols(to + 8 * e, o);
              }
            }
          }
          // an exponent below that of 2^-60 p counts as that: its values are lost beside the largest weighted one
          // either way, and the sum still gets p back
          const float z = m == -INFINITY ? 0.0f : m, nz = n == -INFINITY ? 0.0f : n, least = -60.0f - z;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float e0 = fmaxf(lsv_of(2 * h) - nz, least), e1 = fmaxf(lsv_of(2 * h + 1) - nz, least);
            const float a0 = fmaxf(f * sk_of(2 * h), FLT_MIN), a1 = fmaxf(f * sk_of(2 * h + 1), FLT_MIN);
            const float r0 = ex2(-z - e0), r1 = ex2(-z - e1);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[h][i] = __float_as_uint(ex2(fmaf(__uint_as_float(y[h][i]), i < 16 ? a0 : a1, i < 16 ? e0 : e1)));
            uint32_t p[16];
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float p0 = __uint_as_float(y[h][2 * i]), p1 = __uint_as_float(y[h][2 * i + 1]);
              p[i] = pack_half2(p0, p1);
              sum[(i >> 3) * 2] += p0;
              sum[(i >> 3) * 2 + 1] += p1;
            }
            l = fmaf(sum[0] + sum[1], r0, fmaf(sum[2] + sum[3], r1, l));
            tmem_st_16cols(ts + 32 * q + 16 * h, p);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(q == 0 ? &p1_full[rt] : &p_full[rt]);
        }
        if (!ok) break;
      }
      if (!ok) break;
      some = take(k + 1);
      if (some) queries(items[(k + 1) % kItems]);
      flat += I.hi - lo;
      if (rows > 0) {
      const int rl = tid_here() & 127;
      const bool any = end > lo, live = rl < rows, whole = I.out == kItemWhole;
      if (any) {
        if (!mbar_wait(&o_full[rt], n_o & 1, &s_abort)) break;
        ++n_o;
        tc_fence_after();
      }
      const float2 u = result_factors(n, m, l);
      const size_t cell = ((size_t)blockIdx.x * 2 + (whole ? 0 : I.out)) * kTileRows + rt * 128 + rl;
      const int r = I.r0 + rt * 128 + rl, token = I.a + r / A.G, head = I.h * A.G + r % A.G;
      if (!whole) *reinterpret_cast<float2*>(A.part_ml + cell * 2) = make_float2(m, l);
      // a loop: unrolled it pushes the tiles' code out of the instruction cache (chunk at 16384: 620 -> 598 us)
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        if (any) {
          tmem_ld_32cols(to + 32 * q, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
        if (live) {
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(o[i]) * (u.x * kUnit<FMT>) * u.y;
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(A.out + (int64_t)token * A.out_stride + (int64_t)head * D + 32 * q);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = (uint32_t)store16<DT>(y[8 * i + 2 * e]) | ((uint32_t)store16<DT>(y[8 * i + 2 * e + 1]) << 16);
              dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(A.part_o + cell * D + 32 * q);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
        }
      }
      }
      give_back(k++);
    }
  } else if (warp < 12) {
    regs_dec<128>();
    const int w = warp - 8, c = lane & 3, r4 = lane >> 2;   // rows 32 w + r4 + 8 i, 16-byte columns c and c + 4
    uint4 kr[4 * H], vr[4 * H];
    // a warp's 32 rows are two groups of 16 tokens: the tile's two block numbers are read a tile ahead of
    // its codes, which are read a tile ahead of their use
    struct Next { int id[2], h, o; };                      // o: row of the first group in its block
    float g_sk = 0.0f, g_sv = 0.0f;
    int g_gone = 0, k = -1, j = 0, hi = 0, h = 0, nblk = 0;
    const int* row = nullptr;
    Next nxt;
    const auto advance = [&](Next& N) {                    // one token tile on: false after the last
      if (++j >= hi) {
        if (k >= 0) give_back(k);
        if (!take(++k)) return false;
        const Item& I = items[k % kItems];
        j = I.lo;
        hi = I.hi;
        h = I.h;
        nblk = blocks_of(I.L, A.lb);
        row = A.table + (size_t)I.req * A.max_blocks;
      }
      const int t = j * kTileTok + 32 * w;
      N.h = h;
      N.o = t & ((1 << A.lb) - 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int b = (t + 16 * i) >> A.lb;
        N.id[i] = b < nblk ? row[b] : -1;                  // past the request's blocks
      }
      return true;
    };
    // codes and scales of tile N, the one that advance came to last (scales: lanes 0-15 and 16-31 hold the first
    // group's and the second's)
    const auto load = [&](Next N) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (N.id[i] < 0 || N.id[i] >= A.n_blocks) {
          if ((j * kTileTok + 32 * w + 16 * i) >> A.lb < nblk) record_status(SVDQ_ERR_INVALID_ARG);
          N.id[i] = -1;
        }
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int id = N.id[g], o = ((N.o + 16 * g) & ((1 << A.lb) - 1)) + r4;
        const size_t at = ((((size_t)max(id, 0) * A.kv + N.h) << A.lb) + o) * D + 16 * c;
        const uint4 *pk = reinterpret_cast<const uint4*>(A.kc + at), *pv = reinterpret_cast<const uint4*>(A.vc + at);
#pragma unroll
        for (int i = 2 * g; i < 2 * g + 2; ++i)
#pragma unroll
          for (int q = 0; q < H; ++q) {
            kr[i * H + q] = id >= 0 ? ld_stream(pk + (i & 1) * (8 * D / 16) + 4 * q) : make_uint4(0, 0, 0, 0);
            vr[i * H + q] = id >= 0 ? ld_stream(pv + (i & 1) * (8 * D / 16) + 4 * q) : make_uint4(0, 0, 0, 0);
          }
      }
      const int b = lane < 16 ? N.id[0] : N.id[1];
      g_gone = b < 0;
      g_sk = b < 0 ? 0.0f : A.ks[(size_t)b * A.kv + N.h];
      g_sv = b < 0 ? 0.0f : A.vs[(size_t)b * A.kv + N.h];
    };
    bool more = advance(nxt), after = false;
    if (more) {
      load(nxt);
      after = advance(nxt);
    }
    for (int t = 0; more; ++t) {
      const int st = t & 1;
      if (t >= 2 && !mbar_wait(&k_empty[st], ((t >> 1) & 1) ^ 1, &s_abort)) break;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < H; ++q) store_codes<FMT>(sk + st * TB, 32 * w + r4 + 8 * i, q, c, kr[i * H + q]);
      if ((lane & 15) == 0)
        meta[(t & (kTileMeta - 1)) * 8 + 2 * w + (lane >> 4)] = TileMeta{g_sk, g_sv > 0.0f ? fminf(log2f(g_sv), FLT_MAX) : -INFINITY, g_gone, 0};   // an infinite scale: -inf + it stays -inf
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[st]);
      if (t >= 2 && !mbar_wait(&v_empty[st], ((t >> 1) & 1) ^ 1, &s_abort)) break;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < H; ++q) store_codes<FMT>(sv + st * TB, 32 * w + r4 + 8 * i, q, c, vr[i * H + q]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[st]);
      // the next loads go out only here: the fences above wait for loads in flight
      more = after;
      if (more) {
        load(nxt);
        after = advance(nxt);
      }
    }
  } else {
  regs_dec<96>();
  if (warp == 12) {
    constexpr uint32_t kIdS = idesc_f16_f16(128, 128), kIdO = idesc_f16_f16(128, D) | (1u << 16);
    const uint64_t dq = desc_k_sw128(smem_u32(sq)), dk = desc_k_sw128(smem_u32(sk)), dv = desc_mn_sw128(smem_u32(sv));
    const bool leader = elect_one();
    // a token tile: its row tiles' tiles end at e0 and e1
    struct Tile { int j, lo, hi, e0, e1; };
    int k = 0;
    const auto advance = [&](Tile& T) {
      if (++T.j < T.hi) return true;
      if (!take(k)) return false;
      const Item& I = items[k % kItems];
      T = Tile{I.lo, I.lo, I.hi, I.end[0], I.end[1]};
      give_back(k++);
      return true;
    };
    const auto issue_s = [&](int rt, int st) {
      const uint64_t a = dq + rt * (TB >> 4), b = dk + st * (TB >> 4);
      if (leader) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          constexpr int kHalf = kTileHalf >> 4;
          const int o = (i >> 2) * kHalf + (i & 3) * 2;
          mma_f16(tm + rt * 128, a + o, b + o, kIdS, i > 0);
        }
        mma_commit(&s_full[rt]);
      }
    };
    const auto issue_o = [&](int rt, int st, int half, bool fresh) {   // 64 tokens
      const uint64_t b = dv + st * (TB >> 4);
      if (leader) {
#pragma unroll
        for (int i = 4 * half; i < 4 * half + 4; ++i)
          mma_f16_ts(tm + 256 + rt * D, tm + rt * 128 + 8 * i, b + i * (2048 >> 4), kIdO, !fresh || i > 0);
      }
    };
    const auto commit = [&](uint64_t* bar) { if (leader) mma_commit(bar); };
    uint32_t n_p[2] = {0, 0}, n_q[2] = {0, 0};
    bool ok = true;
    // S of row tile rt at tile T (flat index t), where rt has one there
    const auto next_s = [&](int rt, const Tile& T, int t) {
      const int e = rt == 0 ? T.e0 : T.e1;
      if (T.j >= e) return;
      if (T.j == T.lo) {
        ok = mbar_wait(&q_full[rt], n_q[rt] & 1, &s_abort);
        ++n_q[rt];
        if (!ok) return;
        tc_fence_after();
      }
      issue_s(rt, t & 1);
    };
    Tile cur = {0, 0, 0, 0, 0}, nxt;
    bool more = advance(cur);
    if (more) {
      ok = mbar_wait(&k_full[0], 0, &s_abort);
      tc_fence_after();
      for (int rt = 0; ok && rt < 2; ++rt) next_s(rt, cur, 0);
      commit(&k_empty[0]);
    }
    for (int t = 0; more && ok; ++t) {
      nxt = cur;
      more = advance(nxt);
      ok = mbar_wait(&v_full[t & 1], (t >> 1) & 1, &s_abort);
      if (ok && more) ok = mbar_wait(&k_full[(t + 1) & 1], ((t + 1) >> 1) & 1, &s_abort);
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        const int e = rt == 0 ? cur.e0 : cur.e1;
        if (ok && cur.j < e) {
          ok = mbar_wait(&p1_full[rt], n_p[rt] & 1, &s_abort);
          if (ok) {
            tc_fence_after();
            issue_o(rt, t & 1, 0, cur.j == cur.lo);
            commit(&o1_full[rt]);
            ok = mbar_wait(&p_full[rt], n_p[rt] & 1, &s_abort);
          }
          ++n_p[rt];
          if (ok) {
            tc_fence_after();
            issue_o(rt, t & 1, 1, false);
            if (cur.j + 1 == e) commit(&o_full[rt]);
          }
        }
        if (ok && more) next_s(rt, nxt, t + 1);
      }
      if (!ok) break;
      if (more) {
        commit(&v_empty[t & 1]);
        commit(&k_empty[(t + 1) & 1]);
      }
      cur = nxt;
    }
    if (!ok) {                                             // gave up: the MMAs in flight end before TMEM is freed
      int own = 0;
      commit(drained);
      mbar_wait(drained, 0, &own);
    }
    __syncwarp();
  } else if (warp == 13) {
    Walk walk;
    if (lane < 2 && A.pieces) A.pieces[blockIdx.x * 2 + lane].valid = 0;
    __syncwarp();
    bool left = share.req >= 0;
    if (left) walk.start(A, share, kTileRows);
    for (int k = 0;; ++k) {
      Item I;
      while ((left = left && walk.next(A, share, kTileRows, I)) && I.hi <= I.lo) zero_rows<D>(A, I);
      if (!left) I.hi = -1;
      if (k >= kItems && !mbar_wait(&i_empty[k % kItems], (k / kItems - 1) & 1, &s_abort)) break;
      if (lane == 0) {
        items[k % kItems] = I;
        mbar_arrive(&i_full[k % kItems]);
        if (left && I.out != kItemWhole) {
          const Rows R = {I.a, I.n, I.L, I.rows};
          const int tiles = (seen_by(A, R, min(I.rows, I.r0 + kTileRows) - 1) + kTileTok - 1) / kTileTok;
          A.pieces[blockIdx.x * 2 + I.out] = Piece{1, I.hi == tiles, I.a, min(kTileRows, I.rows - I.r0), I.h, I.r0, 0, 0};
        }
      }
      __syncwarp();
      if (!left) break;
    }
  }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

// Joins the pieces of the items that a border of the schedule cut: blockIdx.x is the
// CTA whose last item continues in the CTAs after it, blockIdx.y a part of its rows,
// `wide` warps a row (warp w of them takes every wide-th piece; then the warps in
// order).  One warp a row where an item has a few pieces, all eight where a long
// request is cut over many CTAs (55 pieces: 25 -> 4 us).
constexpr int kJoinWarps = 8, kMaxParts = 1024;
template <int DT, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const AttnArgs A, int parts, int rows, int wide) {
  constexpr int V = D / 32, kAhead = 4;                  // values a lane, pieces in flight
  __shared__ uint8_t s_valid[kMaxParts];
  __shared__ int s_last;
  __shared__ float s_v[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.x;
  griddep_wait();
  const Piece P = A.pieces[c0 * 2 + 1];
  if (!P.valid) return;
  if (threadIdx.x == 0) s_last = parts - 1;
  __syncthreads();
  for (int k = c0 + 1 + threadIdx.x; k < parts; k += kJoinWarps * 32) {
    const int valid = A.pieces[k * 2].valid;
    s_valid[k] = (uint8_t)valid;
    if (valid && A.pieces[k * 2].last) atomicMin(&s_last, k);   // the first last one ends this item
  }
  __syncthreads();
  const int last = s_last, per = kJoinWarps / wide, sub = warp % wide;
  for (int r0 = blockIdx.y * per; r0 < P.n_rows; r0 += gridDim.y * per) {
    const int r = r0 + warp / wide;
    const bool mine = r < P.n_rows;
    float m = -INFINITY, l = 0.0f, v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
    for (int k0 = c0 + sub; mine && k0 <= last; k0 += kAhead * wide) {
      float2 ml[kAhead];
      float x[kAhead][V], top = m;
#pragma unroll
      for (int b = 0; b < kAhead; ++b) {
        const int k = k0 + b * wide;
        ml[b] = make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) x[b][i] = 0.0f;
        if (k <= last && (k == c0 || s_valid[k])) {
          const size_t cell = ((size_t)k * 2 + (k == c0)) * rows + r;
          ml[b] = *reinterpret_cast<const float2*>(A.part_ml + cell * 2);
          const float* src = A.part_o + cell * D + V * lane;
          if constexpr (V == 4) {
            const float4 y = *reinterpret_cast<const float4*>(src);
            x[b][0] = y.x; x[b][1] = y.y; x[b][2] = y.z; x[b][3] = y.w;
          } else {
            const float2 y = *reinterpret_cast<const float2*>(src);
            x[b][0] = y.x; x[b][1] = y.y;
          }
        }
      }
#pragma unroll
      for (int b = 0; b < kAhead; ++b) top = fmaxf(top, ml[b].x);
      const float old = m == -INFINITY ? 0.0f : ex2(m - top) * l;
      m = top;
      l = old;
#pragma unroll
      for (int b = 0; b < kAhead; ++b) {
        ml[b].y *= ml[b].x == -INFINITY ? 0.0f : ex2(ml[b].x - m);
        l += ml[b].y;
      }
      const float inv = l > 0.0f ? __frcp_rn(l) : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= old * inv;
#pragma unroll
      for (int b = 0; b < kAhead; ++b) {
        const float w = ml[b].y * inv;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += w * x[b][i];
      }
    }
    if (wide > 1) {
      __syncthreads();                                   // the row before is read
      if (lane == 0) s_ml[warp] = make_float2(m, l);
#pragma unroll
      for (int i = 0; i < V; ++i) s_v[warp][V * lane + i] = v[i];
      __syncthreads();
      if (sub > 0) continue;
      float M = m;
      for (int w = 1; w < wide; ++w) M = fmaxf(M, s_ml[warp + w].x);
      const auto part = [&](const float2& ml) { return ml.x == -INFINITY ? 0.0f : ex2(ml.x - M) * ml.y; };
      const float own = part(make_float2(m, l));
      float all = own;
      for (int w = 1; w < wide; ++w) all += part(s_ml[warp + w]);
      const float inv = all > 0.0f ? __frcp_rn(all) : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= own * inv;
      for (int w = 1; w < wide; ++w) {
        const float b = part(s_ml[warp + w]) * inv;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += b * s_v[warp + w][V * lane + i];
      }
    }
    if (!mine) continue;
    const int row = P.r0 + r;
    uint16_t* dst = A.out + (int64_t)(P.token + row / A.G) * A.out_stride + (int64_t)(P.h * A.G + row % A.G) * D + V * lane;
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = (uint32_t)store16<DT>(v[2 * i]) | ((uint32_t)store16<DT>(v[2 * i + 1]) << 16);
    if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
  }
}

// ------------------------------------------------------------- host launchers
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// int32 arrays: a word that lies across words would end the CUDA context
template <class... P>
bool aligned4(const P*... p) { return ((reinterpret_cast<uintptr_t>(p) | ...) & 3) == 0; }

int log2_block(int bs) {
  switch (bs) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
  }
}

svdq_status check_cache(const svdq_paged_cache* c) {
  if (!c || c->reserved != 0) return SVDQ_ERR_INVALID_ARG;
  if (c->heads < 1 || c->kv_heads < 1 || c->heads % c->kv_heads != 0 || c->n_blocks < 1 || c->heads > 32768)
    return SVDQ_ERR_INVALID_ARG;
  if ((c->fmt != SVDQ_KV_INT8 && c->fmt != SVDQ_KV_E4M3) || (c->dtype != SVDQ_BF16 && c->dtype != SVDQ_F16))
    return SVDQ_ERR_INVALID_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128) || log2_block(c->block_size) < 0) return SVDQ_ERR_UNSUPPORTED;
  if ((int64_t)c->n_blocks * c->block_size > INT32_MAX) return SVDQ_ERR_UNSUPPORTED;
  if (!c->kcodes || !c->vcodes || !c->kscale || !c->vscale) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(c->kcodes) || !aligned16(c->vcodes) || !aligned16(c->kscale) || !aligned16(c->vscale))
    return SVDQ_ERR_ALIGNMENT;
  return SVDQ_OK;
}

svdq_status check_batch(const svdq_paged_batch* b, int bs) {
  if (!b || b->reserved != 0) return SVDQ_ERR_INVALID_ARG;
  if (b->B < 1 || b->B > kMaxRequests || b->max_blocks < 1 || b->n_tokens < 0 || b->max_new < 1 || b->max_len < 0)
    return SVDQ_ERR_INVALID_ARG;
  if ((int64_t)b->B * b->max_blocks > INT32_MAX || (int64_t)b->max_blocks * bs > INT32_MAX) return SVDQ_ERR_UNSUPPORTED;
  if (b->n_tokens > kMaxCount || b->max_len > kMaxCount) return SVDQ_ERR_UNSUPPORTED;
  if ((int64_t)b->max_len > (int64_t)b->max_blocks * bs) return SVDQ_ERR_INVALID_ARG;
  return SVDQ_OK;
}

constexpr int plan_smem_bytes(int B) { return 3 * (B + 1) * 4; }

// Per device, once: the sm_100 check, the SM count and the kernels' shared-memory
// attributes.
struct Device { std::atomic<int> state; int sms; };   // state: 0 unknown, 1 ready, 2 not an sm_100
Device g_devices[64];

template <int DT, int FMT, int D>
cudaError_t attention_attr() {
  const auto smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(paged_rows_kernel<DT, FMT, D, 1>, smem, dec_smem(D, 1));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(paged_rows_kernel<DT, FMT, D, 2>, smem, dec_smem(D, 2));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(paged_flat_kernel<DT, FMT, D, 1>, smem, (int)sizeof(FlatSmem<D, 1>));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(paged_flat_kernel<DT, FMT, D, 2>, smem, (int)sizeof(FlatSmem<D, 2>));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(paged_tiles_kernel<DT, FMT, D>, smem, tiles_smem(D));
  return e;
}

svdq_status device_ready(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return SVDQ_ERR_UNSUPPORTED;
  if (dev < 0 || dev >= 64) return SVDQ_ERR_UNSUPPORTED;
  Device& d = g_devices[dev];
  int state = d.state.load(std::memory_order_acquire);
  if (state == 0) {
    int major = 0, minor = 0, n = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SVDQ_ERR_UNSUPPORTED;
    if (major == 10 && minor == 0) {
      e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               plan_smem_bytes(kMaxRequests));
      if (e == cudaSuccess) e = attention_attr<SVDQ_BF16, SVDQ_KV_INT8, 64>();
      if (e == cudaSuccess) e = attention_attr<SVDQ_BF16, SVDQ_KV_INT8, 128>();
      if (e == cudaSuccess) e = attention_attr<SVDQ_BF16, SVDQ_KV_E4M3, 64>();
      if (e == cudaSuccess) e = attention_attr<SVDQ_BF16, SVDQ_KV_E4M3, 128>();
      if (e == cudaSuccess) e = attention_attr<SVDQ_F16, SVDQ_KV_INT8, 64>();
      if (e == cudaSuccess) e = attention_attr<SVDQ_F16, SVDQ_KV_INT8, 128>();
      if (e == cudaSuccess) e = attention_attr<SVDQ_F16, SVDQ_KV_E4M3, 64>();
      if (e == cudaSuccess) e = attention_attr<SVDQ_F16, SVDQ_KV_E4M3, 128>();
      if (e != cudaSuccess) return cuda_failure(e, "paged cache kernel attributes");
      state = 1;
    } else {
      state = 2;
    }
    d.sms = n;
    d.state.store(state, std::memory_order_release);
  }
  *sms = d.sms;
  return state == 1 ? SVDQ_OK : SVDQ_ERR_UNSUPPORTED;
}

// The SM count that the split aims at: fixed, so that workspace sizes can be asked
// for without a device.
constexpr int kSplitSms = 148;

// How a call's rows and tokens are split.  Up to 16 rows a request (few-row kernels,
// rows 8 or 16): fewer (request, kv head) cells than SMs take a cluster of up to
// kMaxCluster CTAs each, as long as those fill the chip; otherwise the balanced schedule
// over as many CTAs as are resident at once.  More rows: the tensor-core kernel (rows
// 256), a CTA per SM.  No CTA of a schedule is left with less than a token tile.
struct Split { int rows, ctas, cluster, snap; };
Split split_of(const svdq_paged_cache* c, const svdq_paged_batch* b) {
  const int64_t G = c->heads / c->kv_heads, rows = b->max_new * G, cells = (int64_t)b->B * c->kv_heads;
  const int64_t len = std::max(b->max_len, 1), tiles = (len + kTileTok - 1) / kTileTok;
  const auto within = [](int64_t n, int64_t hi) { return (int)std::clamp<int64_t>(n, 1, hi); };
  if (rows > 16) {
    const int64_t items = std::min((rows + kTileRows - 1) / kTileRows * b->B, b->n_tokens * G / kTileRows + b->B) * c->kv_heads;
    return Split{kTileRows, within(items * tiles, kSplitSms), 0, 0};
  }
  const int nr = rows <= 8 ? 8 : 16;
  const int64_t room = (int64_t)kSplitSms * flat_per_sm(c->head_dim, nr), want = std::min(room / cells, (len + 255) / 256);
  if (cells < kSplitSms && want <= kMaxCluster) return Split{nr, want >= 8 ? 8 : want >= 4 ? 4 : want >= 2 ? 2 : 1, 1, 0};
  // whole items where they are short: a cut costs a second kernel, an uneven share at most two tiles
  return Split{nr, within(cells * tiles, room), 0, tiles <= 2};
}
bool joins(const Split& s) { return !s.cluster && !s.snap && s.ctas > 1; }

size_t attention_ws(const svdq_paged_cache* c, const svdq_paged_batch* b) {
  const Split s = split_of(c, b);
  return joins(s) ? (size_t)s.ctas * 2 * (sizeof(Piece) + s.rows * (size_t)(c->head_dim + 2) * sizeof(float)) : 16;
}

// A launch that may start while the kernel before it on the stream still runs (each
// kernel waits for that one before it touches memory).
template <class... P, class... Q>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, int cluster, const Q&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int DT, int FMT, int D, int NB>
svdq_status launch_few(const AttnArgs& A, const Split& s, cudaStream_t stream) {
  cudaError_t e;
  if (s.cluster) {
    e = launch_after(paged_rows_kernel<DT, FMT, D, NB>, dim3((unsigned)s.ctas, (unsigned)A.kv, (unsigned)A.B), kDecWarps * 32,
                     dec_smem(D, NB), stream, s.ctas, A);
    return e == cudaSuccess ? SVDQ_OK : cuda_failure(e, "paged_rows_kernel launch");
  }
  e = launch_after(paged_flat_kernel<DT, FMT, D, NB>, dim3((unsigned)s.ctas), kDecWarps * 32, (int)sizeof(FlatSmem<D, NB>), stream, 1, A);
  return e == cudaSuccess ? SVDQ_OK : cuda_failure(e, "paged_flat_kernel launch");
}

template <int DT, int FMT, int D>
svdq_status launch_attention(const AttnArgs& A, const Split& s, cudaStream_t stream) {
  cudaError_t e;
  if (s.rows < kTileRows) {
    const svdq_status st = s.rows == 8 ? launch_few<DT, FMT, D, 1>(A, s, stream) : launch_few<DT, FMT, D, 2>(A, s, stream);
    if (st != SVDQ_OK) return st;
  } else {
    e = launch_after(paged_tiles_kernel<DT, FMT, D>, dim3((unsigned)s.ctas), kTileThreads, tiles_smem(D), stream, 1, A);
    if (e != cudaSuccess) return cuda_failure(e, "paged_tiles_kernel launch");
  }
  if (!joins(s)) return SVDQ_OK;
  const int64_t all = (int64_t)A.max_new * A.G, items = (all + s.rows - 1) / s.rows * A.B * A.kv;
  const int real = (int)std::min<int64_t>(s.rows, all), wide = s.ctas >= 8 * items ? kJoinWarps : 1, per = kJoinWarps / wide;
  const dim3 grid((unsigned)s.ctas, (unsigned)std::min(32, (real + per - 1) / per));
  e = launch_after(paged_join_kernel<DT, D>, grid, kJoinWarps * 32, 0, stream, 1, A, s.ctas, s.rows, wide);
  return e == cudaSuccess ? SVDQ_OK : cuda_failure(e, "paged_join_kernel launch");
}

template <int DT, int FMT, int D>
svdq_status launch_append(const AppendArgs& A, int lb, dim3 grid, cudaStream_t s) {
  cudaError_t e;
  switch (lb) {
    case 4: e = launch_after(paged_append_kernel<DT, FMT, D, 4>, grid, append_threads(16, D), 0, s, 1, A); break;
    case 5: e = launch_after(paged_append_kernel<DT, FMT, D, 5>, grid, append_threads(32, D), 0, s, 1, A); break;
    case 6: e = launch_after(paged_append_kernel<DT, FMT, D, 6>, grid, append_threads(64, D), 0, s, 1, A); break;
    default: e = launch_after(paged_append_kernel<DT, FMT, D, 7>, grid, append_threads(128, D), 0, s, 1, A); break;
  }
  return e == cudaSuccess ? SVDQ_OK : cuda_failure(e, "paged_append_kernel launch");
}

// The call's dtype, format and head size as template arguments.
template <class F>
svdq_status by_types(const svdq_paged_cache* c, F f) {
  const bool bf = c->dtype == SVDQ_BF16, i8 = c->fmt == SVDQ_KV_INT8, wide = c->head_dim == 128;
#define SVDQ_PAGED_CASE(BF_, I8_, W_, DT_, FMT_, D_) \
  if (bf == BF_ && i8 == I8_ && wide == W_) return f.template operator()<DT_, FMT_, D_>();
  SVDQ_PAGED_CASE(true, true, true, SVDQ_BF16, SVDQ_KV_INT8, 128)
  SVDQ_PAGED_CASE(true, true, false, SVDQ_BF16, SVDQ_KV_INT8, 64)
  SVDQ_PAGED_CASE(true, false, true, SVDQ_BF16, SVDQ_KV_E4M3, 128)
  SVDQ_PAGED_CASE(true, false, false, SVDQ_BF16, SVDQ_KV_E4M3, 64)
  SVDQ_PAGED_CASE(false, true, true, SVDQ_F16, SVDQ_KV_INT8, 128)
  SVDQ_PAGED_CASE(false, true, false, SVDQ_F16, SVDQ_KV_INT8, 64)
  SVDQ_PAGED_CASE(false, false, true, SVDQ_F16, SVDQ_KV_E4M3, 128)
  SVDQ_PAGED_CASE(false, false, false, SVDQ_F16, SVDQ_KV_E4M3, 64)
#undef SVDQ_PAGED_CASE
  return SVDQ_ERR_INVALID_ARG;
}

struct AppendCall {
  const AppendArgs& A;
  int lb;
  dim3 grid;
  cudaStream_t s;
  template <int DT, int FMT, int D> svdq_status operator()() const { return launch_append<DT, FMT, D>(A, lb, grid, s); }
};
struct AttnCall {
  const AttnArgs& A;
  const Split& sp;
  cudaStream_t s;
  template <int DT, int FMT, int D> svdq_status operator()() const { return launch_attention<DT, FMT, D>(A, sp, s); }
};

}  // namespace paged

cudaError_t paged_status_take(unsigned int* v) {
  *v = 0;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  // no call of the paged cache got as far as a launch on this device: nothing to read (a copy costs microseconds)
  if (e != cudaSuccess || device < 0 || device >= 64 || paged::g_devices[device].state.load(std::memory_order_acquire) != 1) return e;
  e = cudaMemcpyFromSymbol(v, dev::g_status, sizeof(*v));
  if (e == cudaSuccess && *v != 0) {
    const unsigned int z = 0;
    e = cudaMemcpyToSymbol(dev::g_status, &z, sizeof(z));
  }
  return e;
}

}  // namespace svdq

using namespace svdq;
using namespace svdq::paged;

extern "C" {

svdq_status svdq_paged_plan(const svdq_paged_batch* b, int32_t block_size, int32_t n_blocks, const int32_t* prev,
                            const int32_t* target, int32_t* ring, const int32_t* state_in, int32_t* state_out,
                            svdq_stream stream) {
  const int lb = log2_block(block_size);
  if (lb < 0) return SVDQ_ERR_UNSUPPORTED;
  svdq_status st = check_batch(b, block_size);
  if (st != SVDQ_OK) return st;
  if (n_blocks < 1 || !prev || !target || !ring || !state_in || !state_out || !b->table || !b->lens || !b->cu ||
      (b->n_tokens > 0 && !b->slots))
    return SVDQ_ERR_INVALID_ARG;
  if ((int64_t)n_blocks * block_size > INT32_MAX) return SVDQ_ERR_UNSUPPORTED;
  if (state_in == state_out || prev == b->lens || target == b->lens) return SVDQ_ERR_INVALID_ARG;
  if (!aligned4(b->table, b->lens, b->cu, b->slots, prev, target, ring, state_in, state_out)) return SVDQ_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = device_ready(&sms)) != SVDQ_OK) return st;
  PlanArgs A;
  A.prev = prev; A.target = target; A.table = b->table; A.lens = b->lens; A.cu = b->cu; A.slots = b->slots;
  A.ring = ring; A.state_in = state_in; A.state_out = state_out;
  A.B = b->B; A.max_blocks = b->max_blocks; A.n_tokens = b->n_tokens; A.max_new = b->max_new; A.max_len = b->max_len;
  A.n_blocks = n_blocks; A.lb = lb;
  // a CTA per 2048 slots: up to there one CTA's scan and writes are cheaper than another CTA's scan
  const int ctas = (int)std::min<int64_t>(sms, std::max<int64_t>(1, ((int64_t)b->n_tokens + b->B + 2047) / 2048));
  const cudaError_t e = launch_after(paged_plan_kernel, dim3((unsigned)ctas), kPlanThreads, plan_smem_bytes(b->B),
                                     reinterpret_cast<cudaStream_t>(stream), 1, A);
  return e == cudaSuccess ? SVDQ_OK : cuda_failure(e, "paged_plan_kernel launch");
}

svdq_status svdq_paged_append(const svdq_paged_cache* c, const svdq_paged_batch* b, const void* K, int64_t k_stride,
                              const void* V, int64_t v_stride, svdq_stream stream) {
  svdq_status st = check_cache(c);
  if (st != SVDQ_OK) return st;
  if ((st = check_batch(b, c->block_size)) != SVDQ_OK) return st;
  if (b->n_tokens == 0) return SVDQ_OK;
  if (!K || !V || !b->cu || !b->slots) return SVDQ_ERR_INVALID_ARG;
  const int64_t row = (int64_t)c->kv_heads * c->head_dim;
  if (k_stride < row || v_stride < row) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V) || k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned4(b->cu, b->slots)) return SVDQ_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = device_ready(&sms)) != SVDQ_OK) return st;
  AppendArgs A;
  A.x[0] = static_cast<const uint16_t*>(K); A.x[1] = static_cast<const uint16_t*>(V);
  A.stride[0] = k_stride; A.stride[1] = v_stride;
  A.codes[0] = c->kcodes; A.codes[1] = c->vcodes; A.scale[0] = c->kscale; A.scale[1] = c->vscale;
  A.cu = b->cu; A.slots = b->slots; A.B = b->B; A.n_tokens = b->n_tokens; A.kv = c->kv_heads; A.n_blocks = c->n_blocks;
  A.max_new = b->max_new; A.per = b->max_new == 1 ? 1 : 2;
  const int lb = log2_block(c->block_size);
  const dim3 grid((unsigned)((b->n_tokens >> lb) + A.per * b->B), (unsigned)c->kv_heads, 2u);
  return by_types(c, AppendCall{A, lb, grid, reinterpret_cast<cudaStream_t>(stream)});
}

size_t svdq_paged_attention_workspace_bytes(const svdq_paged_cache* c, const svdq_paged_batch* b) {
  if (check_cache(c) != SVDQ_OK || check_batch(b, c->block_size) != SVDQ_OK) return 0;
  if ((int64_t)b->max_new * (c->heads / c->kv_heads) > kMaxCount) return 0;
  return attention_ws(c, b);
}

svdq_status svdq_paged_attention(const svdq_paged_cache* c, const svdq_paged_batch* b, const void* Q, int64_t q_stride,
                                 int32_t causal, float scale, void* out, int64_t out_stride, void* workspace,
                                 size_t ws_bytes, svdq_stream stream) {
  svdq_status st = check_cache(c);
  if (st != SVDQ_OK) return st;
  if ((st = check_batch(b, c->block_size)) != SVDQ_OK) return st;
  if (b->n_tokens == 0) return SVDQ_OK;
  if (!Q || !out || !workspace || !b->cu || !b->lens || !b->table || (causal != 0 && causal != 1) || !std::isfinite(scale))
    return SVDQ_ERR_INVALID_ARG;
  if ((int64_t)b->max_new * (c->heads / c->kv_heads) > kMaxCount) return SVDQ_ERR_UNSUPPORTED;
  const int64_t row = (int64_t)c->heads * c->head_dim;
  if (q_stride < row || out_stride < row) return SVDQ_ERR_INVALID_ARG;
  if (ws_bytes < attention_ws(c, b)) return SVDQ_ERR_WORKSPACE;
  if (!aligned16(Q) || !aligned16(out) || !aligned16(workspace) || q_stride % 8 != 0 || out_stride % 8 != 0 ||
      !aligned4(b->table, b->lens, b->cu))
    return SVDQ_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = device_ready(&sms)) != SVDQ_OK) return st;
  const Split sp = split_of(c, b);
  AttnArgs A;
  A.q = static_cast<const uint16_t*>(Q); A.out = static_cast<uint16_t*>(out);
  A.kc = c->kcodes; A.vc = c->vcodes; A.ks = c->kscale; A.vs = c->vscale;
  A.table = b->table; A.lens = b->lens; A.cu = b->cu;
  A.pieces = nullptr;
  A.part_ml = A.part_o = nullptr;
  if (joins(sp)) {
    A.pieces = static_cast<Piece*>(workspace);
    A.part_ml = reinterpret_cast<float*>(A.pieces + sp.ctas * 2);
    A.part_o = A.part_ml + (size_t)sp.ctas * 2 * sp.rows * 2;
  }
  A.q_stride = q_stride; A.out_stride = out_stride;
  A.B = b->B; A.max_blocks = b->max_blocks; A.n_tokens = b->n_tokens; A.max_new = b->max_new; A.max_len = b->max_len;
  A.n_blocks = c->n_blocks; A.kv = c->kv_heads; A.G = c->heads / c->kv_heads;
  A.lb = log2_block(c->block_size); A.causal = causal; A.splits = sp.ctas; A.snap = sp.snap;
  A.scale_log2 = scale * 1.4426950408889634f;
  A.inv_parts = 1.0 / sp.ctas;
  A.g_inv = A.G == 1 ? 0u : (uint32_t)(((1ull << 32) + A.G - 1) / A.G);
  return by_types(c, AttnCall{A, sp, reinterpret_cast<cudaStream_t>(stream)});
}

}  // extern "C"

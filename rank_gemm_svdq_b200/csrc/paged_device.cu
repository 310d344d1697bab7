// Paged 8-bit KV cache: the step plan, the append and the attention that reads
// the cache (the serving form of the INT8 KV cache of "VAR-Compressor：在边缘GPU上
// 实现80亿参数视觉自回归模型的高效量化部署", INT8 KV缓存量化; the block-wise scale is
// the granularity that lets tokens join a cache without touching other blocks).
//
// Block b of the pool holds, for every key/value head h, `bs` tokens of d 8-bit
// codes (contiguous bs x d bytes at ((b kv + h) bs d)) and one fp32 scale for the
// keys and one for the values (at b kv + h): x ~ code * scale.
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
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
constexpr int kPlanThreads = 512;

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
  const bool wrong = s_bad != 0 || c_new > A.n_tokens || (int64_t)count - c_take + c_give > A.n_blocks;
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
  const auto wrap = [&](int64_t k) { return (int)(k % A.n_blocks); };
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
  const int total = ok ? (int)c_new : 0;
  for (int k = gtid; k < A.n_tokens; k += stride) {
    int slot = -1;
    if (k < total) {
      const int i = last_not_above(s_new, A.B, k);
      const int p = A.prev[i], pos = p + (k - s_new[i]), held = blocks_of(p, A.lb), c = pos >> A.lb;
      const int blk = c < held ? A.table[(size_t)i * A.max_blocks + c] : A.ring[wrap((int64_t)head + s_take[i] + (c - held))];
      slot = blk < 0 || blk >= A.n_blocks ? -1 : (blk << A.lb) + (pos & ((1 << A.lb) - 1));
    }
    A.slots[k] = slot;
  }
}

// -------------------------------------------------------------------- append
// One CTA per (block touched by a request's new tokens, kv head, keys or values).
// s = max(s_old, max |x| / qmax), codes = round(x / s); codes of the tokens that
// the block held before are re-rounded when s grows.  The new rows (at most one
// block: bs d values) are read once and stay in registers between the maximum
// and the codes.  Work index w -> request: request i owns the indices from
// floor(cu_i / bs) + 2 i, which leaves it at least as many as it touches blocks
// (<= floor(new / bs) + 2), so the grid needs only n_tokens and B on the host.
constexpr int kAppendThreads = 128;

template <int FMT> struct Fmt;
template <> struct Fmt<SVDQ_KV_INT8> { static constexpr float qmax = 127.0f; };
template <> struct Fmt<SVDQ_KV_E4M3> { static constexpr float qmax = 448.0f; };

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

// x / s as IEEE division rounds it: q = RN(x rs) is within an ulp, e = x - q s is
// exact (one FMA), RN(q + e rs) is the correctly rounded quotient (Markstein) while
// nothing under- or overflows; rs = 0 outside 2^-60 <= s <= 2^60 (division then).
__device__ __forceinline__ float quotient(float x, float s, float rs) {
  if (rs == 0.0f) return s > 0.0f ? __fdiv_rn(x, s) : 0.0f;
  const float q = __fmul_rn(x, rs);
  return __fmaf_rn(__fmaf_rn(-q, s, x), rs, q);
}

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
  int B, n_tokens, kv, n_blocks;
};

template <int DT, int FMT, int D, int LB>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendArgs A) {
  constexpr int BS = 1 << LB, kPerRow = D / 8, kRows = kAppendThreads / kPerRow, kPass = BS / kRows > 0 ? BS / kRows : 1;
  __shared__ float s_amax[kAppendThreads / 32];
  const int tid = threadIdx.x, w = blockIdx.x, h = blockIdx.y, which = blockIdx.z;
  // this work item's request: the last one whose first index is not above w
  int i = -1;
  for (int r0 = 0; r0 < A.B; r0 += kAppendThreads) {
    const int r = r0 + tid;
    const bool le = r < A.B && (clampi(A.cu[r], 0, A.n_tokens) >> LB) + 2 * r <= w;
    i += __syncthreads_count(le);
  }
  if (i < 0) return;
  const int a = clampi(A.cu[i], 0, A.n_tokens), e = clampi(A.cu[i + 1], 0, A.n_tokens);
  if (a >= e) return;
  const int j = w - (a >> LB) - 2 * i, o0 = A.slots[a] & (BS - 1);
  const int64_t first = (int64_t)a + (j == 0 ? 0 : (int64_t)j * BS - o0);
  if (first >= e) return;
  const int t0 = (int)first;
  const int slot0 = A.slots[t0];
  if (slot0 < 0) return;                             // a padded token
  const int blk = slot0 >> LB, off = slot0 & (BS - 1);
  if (blk >= A.n_blocks) {
    if (tid == 0) record_status(SVDQ_ERR_INVALID_ARG);
    return;
  }
  const int rows = min(min(e, a + (j + 1) * BS - o0) - t0, BS - off);
  const int c = tid % kPerRow, r0 = tid / kPerRow;
  const uint16_t* x = A.x[which] + (int64_t)t0 * A.stride[which] + h * D + 8 * c;
  const size_t cell = (size_t)blk * A.kv + h;
  const float s_old = off > 0 ? A.scale[which][cell] : 0.0f;
  uint4 v[kPass];
  int at[kPass];
  uint32_t have = 0;
  // rows and their slots at once; a row counts only where the slot map puts it next to
  // the block's first new row
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int r = r0 + p * kRows;
    v[p] = make_uint4(0, 0, 0, 0);
    at[p] = -1;
    if (r < rows) {
      v[p] = __ldg(reinterpret_cast<const uint4*>(x + (int64_t)r * A.stride[which]));
      at[p] = A.slots[t0 + r];
    }
  }
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    if (at[p] == slot0 + r0 + p * kRows) have |= 1u << p;
    else v[p] = make_uint4(0, 0, 0, 0);
  }
  float amax = 0.0f;
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    float f[8];
    unpack8<DT>(v[p], f);
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(f[k]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) s_amax[tid >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kAppendThreads / 32; ++k) amax = fmaxf(amax, s_amax[k]);
  const float s = fmaxf(s_old, __fdiv_rn(amax, Fmt<FMT>::qmax));
  uint8_t* base = A.codes[which] + cell * (size_t)(BS * D);
  if (s > s_old) {
    if (tid == 0) A.scale[which][cell] = s;
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
    A.scale[which][cell] = 0.0f;                     // a fresh block of zeros
  }
  const float rs = s >= 0x1p-60f && s <= 0x1p+60f ? __frcp_rn(s) : 0.0f;
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    if (have >> p & 1u) {
      float f[8];
      unpack8<DT>(v[p], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = quotient(f[k], s, rs);
      *reinterpret_cast<uint2*>(base + (size_t)(off + r0 + p * kRows) * D + 8 * c) =
          make_uint2(codes4<FMT>(f[0], f[1], f[2], f[3]), codes4<FMT>(f[4], f[5], f[6], f[7]));
    }
  }
}

// ----------------------------------------------------------------- attention
// Row r of request i, kv head h: new token r / G, query head h G + r % G.  With
// codes c and scales s per block: x_t = scale 2^e s_k (q' . c_t) log2(e), where
// q' = q 2^-e in fp16 (e: exponent of the row's largest entry, so q' is exact up to
// 2^-25 of that entry); out = sum_t p_t s_v c^v_t / sum_t p_t, p_t = 2^(x_t - m).
// Both products run on fp16 operands (8-bit codes are exact in fp16) with fp32
// accumulators.  The value scale is folded into p before it is rounded to fp16,
// relative to the largest value scale seen so far (p' <= 1, no overflow; one
// rounding of 2^-11 per weight, the size of the rounding of an fp16 output).
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
  float* part_o;           // [splits][n_tokens][heads][d]
  float* part_ml;          // [splits][n_tokens][heads][2]
  int64_t q_stride, out_stride;
  int B, max_blocks, n_tokens, max_new, max_len, n_blocks, heads, kv, G, lb, causal, splits, chunk;
  float scale_log2;
};

// What one request's rows see.
struct Rows {
  int a, n, L, rows;       // first token, new tokens, cached length, n G
};
__device__ __forceinline__ Rows request_rows(const AttnArgs& A, int i) {
  Rows R;
  R.a = clampi(A.cu[i], 0, A.n_tokens);
  const int e = clampi(A.cu[i + 1], 0, A.n_tokens), n = e - R.a, L = A.lens[i];
  R.n = clampi(n, 0, A.max_new);
  R.L = clampi(L, 0, min(A.max_len, A.max_blocks << A.lb));
  if (threadIdx.x == 0 && (n > A.max_new || L > R.L)) record_status(SVDQ_ERR_INVALID_ARG);
  R.rows = R.n * A.G;
  return R;
}
// Tokens that row r sees (its new token is r / G).
__device__ __forceinline__ int seen_by(const AttnArgs& A, const Rows& R, int r) {
  return A.causal ? max(0, R.L - R.n + r / A.G + 1) : R.L;
}

template <int DT>
__device__ __forceinline__ float load16(uint16_t h) {
  if constexpr (DT == SVDQ_BF16) return __uint_as_float((uint32_t)h << 16);
  else return __half2float(__ushort_as_half(h));
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 rows of queries as normalised fp16 in shared memory (row pitch D + 8) and
// each row's factor 2^e scale log2(e).  Rows past the request's are zero.
template <int DT, int D>
__device__ __forceinline__ void load_queries(const AttnArgs& A, const Rows& R, int h, int r0, int nrows, __half* sq,
                                             float* sf, int warp, int nwarps, int lane) {
  for (int rr = warp; rr < nrows; rr += nwarps) {
    const int r = r0 + rr;
    float v[D / 32], top = 0.0f;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) v[k] = 0.0f;
    if (r < R.rows) {
      const uint16_t* q = A.q + (int64_t)(R.a + r / A.G) * A.q_stride + (int64_t)(h * A.G + r % A.G) * D;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) { v[k] = load16<DT>(q[lane + 32 * k]); top = fmaxf(top, fabsf(v[k])); }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = clampi((int)(__float_as_uint(top) >> 23) - 127, -100, 100);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int k = 0; k < D / 32; ++k) sq[rr * (D + 8) + lane + 32 * k] = __float2half_rn(v[k] * down);
    if (lane == 0) sf[rr] = __uint_as_float((uint32_t)(127 + e) << 23) * A.scale_log2;
  }
}

// Few rows: up to 8 NB rows of one (request, kv head) against a range of its tokens.
// Bound by the cache's bytes, so the products run on mma.sync with the codes as the
// 16-row operand and the few rows as its 8 columns: S^T = K Q^T, O^T = V^T P^T (half
// the MMAs and accumulators of the other way round).  Each of the 4 warps takes every
// fourth tile of 32 tokens through a ring of its own (bulk copies, no barrier between
// warps) and keeps its own m, l and accumulator; the warps' results are joined at the
// end, then those of the CTAs of a cluster, which share the tokens of a (request, kv
// head) evenly.  The fragments are read straight from the codes: the order of the
// contraction over d is free, so 16 bytes of a key row serve 4 k-steps, and 16 bytes
// of four value rows the 16 values of d that a lane needs.
constexpr int kDecWarps = 4, kDecTile = 32, kDecStages = 2, kDecGroup = 16, kMaxCluster = 8;
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
__device__ __forceinline__ void store_row4(uint16_t* dst, const float4& v, float mul) {
  uint2 w;
  w.x = (uint32_t)store16<DT>(v.x * mul) | ((uint32_t)store16<DT>(v.y * mul) << 16);
  w.y = (uint32_t)store16<DT>(v.z * mul) | ((uint32_t)store16<DT>(v.w * mul) << 16);
  *reinterpret_cast<uint2*>(dst) = w;
}

template <int DT, int FMT, int D, int NB>
__global__ void __launch_bounds__(kDecWarps * 32) paged_rows_kernel(const AttnArgs A, int cluster) {
  constexpr int NST = kDecStages, kStage = dec_stage_bytes(D), KC = D / 64, VW = D / 32, NR = 8 * NB;
  extern __shared__ __align__(128) uint8_t dsm[];
  uint8_t* ring = dsm;
  __half* sq = reinterpret_cast<__half*>(dsm + dec_ring_bytes(D));
  DecMeta* meta = reinterpret_cast<DecMeta*>(sq + NR * (D + 8));           // [warp][2 groups]
  int2* ids = reinterpret_cast<int2*>(meta + kDecWarps * 2 * kDecGroup);   // [warp][2 groups]
  float2* wml = reinterpret_cast<float2*>(ids + kDecWarps * 2 * kDecGroup);  // [warp][NR]
  float* sf = reinterpret_cast<float*>(wml + kDecWarps * NR);              // [NR]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sf + NR);                   // [warp][NST]
  __shared__ int s_abort;
  __shared__ float s_vref[kDecWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  const int h = blockIdx.y, req = blockIdx.z, split = blockIdx.x;
  if (!cluster) griddep_launch();
  const Rows R = request_rows(A, req);
  if (R.rows == 0) return;
  const int vis = seen_by(A, R, R.rows - 1), first_vis = seen_by(A, R, 0);
  // a cluster shares what the rows see; otherwise a fixed chunk a split
  const int chunk = cluster ? ((vis + A.splits - 1) / A.splits + kDecTile - 1) / kDecTile * kDecTile : A.chunk;
  const int t_begin = split * chunk, t_end = max(t_begin, min(vis, t_begin + chunk));
  if (!cluster && split > 0 && t_begin >= vis) return;
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
        id.x = row[c0];
        id.y = c1 == c0 ? id.x : (c1 < nblk ? row[c1] : -2);
        if (id.x < 0 || id.x >= A.n_blocks) { id.x = -1; record_status(SVDQ_ERR_INVALID_ARG); }
        if (id.y != -2 && (id.y < 0 || id.y >= A.n_blocks)) { id.y = -1; record_status(SVDQ_ERR_INVALID_ARG); }
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

  load_queries<DT, D>(A, R, h, 0, NR, sq, sf, warp, kDecWarps, lane);
  __syncthreads();
  // Q^T fragments: k-step s covers d = 64 (s / 4) + 16 q4 + 4 (s % 4) + {0, 1 | 2, 3}
  uint32_t qf[NB][D / 16][2];
  float f[NB][2];
  int see[NB][2];
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
      f[nb][i] = sf[r] * kUnit<FMT>;
      see[nb][i] = r < R.rows ? min(t_end, seen_by(A, R, r)) : t_end;
    }
  }
  const int clear = min(t_end, first_vis);              // tiles that end at or below this need no mask
  float o[D / 16][NB][4], m[NB][2], l[NB][2], vref = 0.0f;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m[nb][0] = m[nb][1] = -INFINITY;
    l[nb][0] = l[nb][1] = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[j][nb][0] = o[j][nb][1] = o[j][nb][2] = o[j][nb][3] = 0.0f;
  }

  for (int k = 0; k < mine; ++k) {
    const int st = k % NST, t = t_begin + (warp + kDecWarps * k) * kDecTile;
    if (!mbar_wait(&wbar[st], (k / NST) & 1, &s_abort)) {
      int own = 0;                                       // the copies in flight end before the CTA does
      for (int i = k; i < min(mine, k + NST); ++i) mbar_wait(&wbar[i % NST], (i / NST) & 1, &own);
      break;
    }
    const uint8_t* kt = wring + st * kStage;
    const uint8_t* vt = kt + kDecTile * D;
    const DecMeta md = wmeta[k & (2 * kDecGroup - 1)];
    const int2 id = wids[k & (2 * kDecGroup - 1)];
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
          const uint32_t a[4] = {half2_of<FMT, 0>(y), half2_of<FMT, 0>(z), half2_of<FMT, 1>(y), half2_of<FMT, 1>(z)};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma16816(x[mt][nb], a, qf[nb][c * 4 + i][0], qf[nb][c * 4 + i][1]);
        }
      }
    }
    // scores in units of log2, masked
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float s0 = f[nb][0] * md.sk[mt], s1 = f[nb][1] * md.sk[mt];
        x[mt][nb][0] *= s0; x[mt][nb][1] *= s1; x[mt][nb][2] *= s0; x[mt][nb][3] *= s1;
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
    float top[NB][2];
    bool grow = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float a = fmaxf(fmaxf(x[0][nb][i], x[0][nb][i + 2]), fmaxf(x[1][nb][i], x[1][nb][i + 2]));
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, s));
        top[nb][i] = fmaxf(m[nb][i], a);
        grow = grow || top[nb][i] > m[nb][i];
      }
    const float vmax = fmaxf(vref, fmaxf(md.sv[0], md.sv[1]));
    if (__any_sync(0xffffffffu, grow || vmax > vref)) {
      const float fv = vmax > 0.0f ? __fdiv_rn(vref, vmax) : 1.0f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          b[i] = top[nb][i] == -INFINITY ? 1.0f : ex2(m[nb][i] - top[nb][i]);
          l[nb][i] *= b[i];
          m[nb][i] = top[nb][i];
          b[i] *= fv;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          o[j][nb][0] *= b[0]; o[j][nb][1] *= b[1]; o[j][nb][2] *= b[0]; o[j][nb][3] *= b[1];
        }
      }
      vref = vmax;
    }
    const float rv = vref > 0.0f ? __fdiv_rn(1.0f, vref) : 0.0f;
    uint32_t pb[2][NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float z0 = m[nb][0] == -INFINITY ? 0.0f : m[nb][0], z1 = m[nb][1] == -INFINITY ? 0.0f : m[nb][1];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const float wv = md.sv[mt] * rv;
        const float p0 = ex2(x[mt][nb][0] - z0), p1 = ex2(x[mt][nb][1] - z1);
        const float p2 = ex2(x[mt][nb][2] - z0), p3 = ex2(x[mt][nb][3] - z1);
        l[nb][0] += p0 + p2;
        l[nb][1] += p1 + p3;
        // [token][row] -> [row][token]: the column operand of the second product
        pb[mt][nb][0] = transpose8x8(pack_half2(p0 * wv, p1 * wv));
        pb[mt][nb][1] = transpose8x8(pack_half2(p2 * wv, p3 * wv));
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
      // accumulator tile j: operand row n is d = (D / 8) n + 2 j, row n + 8 the d after it
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        const uint32_t la = __byte_perm(u[0][w], u[1][w], 0x5140), ha = __byte_perm(u[0][w], u[1][w], 0x7362);
        const uint32_t lb = __byte_perm(u[2][w], u[3][w], 0x5140), hb = __byte_perm(u[2][w], u[3][w], 0x7362);
        const uint32_t a0[4] = {half2_of<FMT, 0>(la), half2_of<FMT, 1>(la), half2_of<FMT, 0>(lb), half2_of<FMT, 1>(lb)};
        const uint32_t a1[4] = {half2_of<FMT, 0>(ha), half2_of<FMT, 1>(ha), half2_of<FMT, 0>(hb), half2_of<FMT, 1>(hb)};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          mma16816(o[2 * w][nb], a0, pb[s][nb][0], pb[s][nb][1]);
          mma16816(o[2 * w + 1][nb], a1, pb[s][nb][0], pb[s][nb][1]);
        }
      }
    }
    __syncwarp();
    if (k + NST < mine) issue(k + NST);
  }
  // join the four warps: weights 2^(m_w - M) and the value reference of each
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int s = 4; s < 32; s <<= 1) l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], s);
      if (g == 0) wml[warp * NR + nb * 8 + 2 * q4 + i] = make_float2(m[nb][i], l[nb][i]);
    }
  if (lane == 0) s_vref[warp] = vref * kUnit<FMT>;
  __syncthreads();                                       // every ring is free: the accumulators go there
  constexpr int AP = D + 4;                              // row pitch of the accumulators
  float* acc = reinterpret_cast<float*>(ring);           // [warp][NR][AP]
  float* mine_o = acc + kDecWarps * NR * AP;             // [NR][D]: this CTA's joined rows
  float2* mine_ml = reinterpret_cast<float2*>(mine_o + NR * D);
  static_assert((kDecWarps * NR * AP + NR * D + 2 * NR) * 4 <= dec_ring_bytes(D), "the join fits the ring");
  const auto weight = [&](int w, int r, float M) { const float x = wml[w * NR + r].x; return x == -INFINITY ? 0.0f : ex2(x - M); };
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = nb * 8 + 2 * q4 + i;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, wml[w * NR + r].x);
      const float wt = weight(warp, r, M) * s_vref[warp];
      float* p = acc + (warp * NR + r) * AP + (D / 8) * g;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        *reinterpret_cast<float2*>(p + 2 * j) = make_float2(o[j][nb][i] * wt, o[j][nb][i + 2] * wt);
    }
  __syncthreads();
  const bool whole = !cluster && vis <= chunk;           // this CTA holds all that the rows see
  for (int idx = tid; idx < NR * D / 4; idx += kDecWarps * 32) {
    const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
    if (r >= R.rows) break;
    float M = -INFINITY, L = 0.0f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, wml[w * NR + r].x);
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) L += weight(w, r, M) * wml[w * NR + r].y;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(acc + (w * NR + r) * AP + d);
      v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
    }
    const int token = R.a + r / A.G, head = h * A.G + r % A.G;
    if (cluster) {
      *reinterpret_cast<float4*>(mine_o + r * D + d) = v;
      if (d == 0) mine_ml[r] = make_float2(M, L);
    } else if (whole) {
      store_row4<DT>(A.out + (int64_t)token * A.out_stride + (int64_t)head * D + d, v, L > 0.0f ? __fdiv_rn(1.0f, L) : 0.0f);
    } else {
      const size_t cell = ((size_t)split * A.n_tokens + token) * A.heads + head;
      *reinterpret_cast<float4*>(A.part_o + cell * D + d) = v;
      if (d == 0) *reinterpret_cast<float2*>(A.part_ml + cell * 2) = make_float2(M, L);
    }
  }
  if (!cluster) return;
  // the cluster's CTAs in rank order, each taking its share of the values
  cluster_sync();
  const uint32_t o_at = smem_u32(mine_o), ml_at = smem_u32(mine_ml);
  for (int idx = split * (kDecWarps * 32) + tid; idx < NR * D / 4; idx += A.splits * kDecWarps * 32) {
    const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
    if (r >= R.rows) break;
    float2 ml[kMaxCluster];
    float M = -INFINITY, L = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) {
      ml[s] = s < A.splits ? ld_cluster_f32x2(mapa_shared(ml_at + 8 * r, s)) : make_float2(-INFINITY, 0.0f);
      M = fmaxf(M, ml[s].x);
    }
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) {
      if (s < A.splits) {
        const float w = ml[s].x == -INFINITY ? 0.0f : ex2(ml[s].x - M);
        const float4 y = ld_cluster_f32x4(mapa_shared(o_at + (r * D + d) * 4, s));
        L += w * ml[s].y;
        v.x += w * y.x; v.y += w * y.y; v.z += w * y.z; v.w += w * y.w;
      }
    }
    const int token = R.a + r / A.G, head = h * A.G + r % A.G;
    store_row4<DT>(A.out + (int64_t)token * A.out_stride + (int64_t)head * D + d, v, L > 0.0f ? __fdiv_rn(1.0f, L) : 0.0f);
  }
  cluster_sync();                                        // nobody leaves while its rows are read
}

// Many rows: 128 or 256 rows of one (request, kv head) against a range of its
// tokens, on the tensor cores.  Codes become fp16 operands in shared memory once
// per 128 tokens and serve both 128-row tiles: S = Q K^T (both operands from shared
// memory, 128 x 128 fp32 in TMEM), P in fp16 over S's own columns, O += P V (P from
// TMEM; V as it lies, token rows of 64 d, an MN-major operand).  Roles:
//   warps 0-3, 4-7   softmax of row tile 0 / 1, a row per thread: maximum, weights,
//                    sum; rescales O only when a maximum grew by more than 2^8
//                    (weights stay below 2^8 in fp16)
//   warps 8-11       codes -> fp16 (the next tile's codes already in registers)
//   warp 12          issues the MMAs: S0 S1 | P0V S0' | P1V S1' | ...
// The value scale goes into a weight's exponent, p' = 2^(x - m + log2(s_v / s_ref))
// with s_ref the largest value scale of the range, so it costs nothing per weight;
// the row sum takes each 16 tokens' sum times s_ref / s_v.
constexpr int kTileThreads = 512, kTileTok = 128, kTileMeta = 4;
struct TileMeta { float sk, lsv, rsv; int gone; };        // 16 tokens: key scale, log2(s_v / s_ref), s_ref / s_v
constexpr int kTileHalf = 128 * 128;                      // 128 rows of 64 fp16, 128-byte swizzle
constexpr int tile_bytes(int D) { return D / 64 * kTileHalf; }
constexpr int tiles_smem(int D) { return 6 * tile_bytes(D) + 256 * 4 + kTileMeta * 8 * 16 + 128 + 1024; }

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

template <int DT, int FMT, int D>
__global__ void __launch_bounds__(kTileThreads, 1) paged_tiles_kernel(const AttnArgs A, int cta_rows) {
  constexpr int H = D / 64, TB = tile_bytes(D);
  extern __shared__ uint8_t tsm_raw[];
  uint8_t* tsm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tsm_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sq = tsm;                                       // [2 row tiles]
  uint8_t* sk = sq + 2 * TB;                               // [2 stages]
  uint8_t* sv = sk + 2 * TB;                               // [2 stages]
  float* sf = reinterpret_cast<float*>(sv + 2 * TB);       // [256]
  TileMeta* meta = reinterpret_cast<TileMeta*>(sf + 256);  // [kTileMeta][8]
  uint64_t* bars = reinterpret_cast<uint64_t*>(meta + kTileMeta * 8);
  uint64_t *k_full = bars, *k_empty = bars + 2, *v_full = bars + 4, *v_empty = bars + 6, *s_full = bars + 8,
           *p_full = bars + 10, *o_full = bars + 12, *drained = bars + 14;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ float s_ref;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // splits fastest, then kv heads and requests, then row CTAs: the longest rows of a prompt first
  const int split = blockIdx.x % A.splits, cell_id = (blockIdx.x / A.splits) % (A.B * A.kv);
  const int h = cell_id % A.kv, req = cell_id / A.kv, rts = (A.max_new * A.G + cta_rows - 1) / cta_rows;
  const int r0 = (rts - 1 - (int)(blockIdx.x / A.splits / (A.B * A.kv))) * cta_rows;
  griddep_launch();
  const Rows R = request_rows(A, req);
  if (r0 >= R.rows) return;
  const int last = min(R.rows, r0 + cta_rows) - 1;
  const int vis = seen_by(A, R, last);
  const int t_begin = split * A.chunk, t_end = min(vis, t_begin + A.chunk);
  if (split > 0 && t_begin >= vis) return;
  const int row_tiles = last - r0 >= 128 ? 2 : 1;
  // token tiles of a row tile: what its last row sees
  const auto tiles_of = [&](int rt) {
    const int e = min(t_end, seen_by(A, R, min(R.rows, r0 + rt * 128 + 128) - 1));
    return e > t_begin ? (e - t_begin + kTileTok - 1) / kTileTok : 0;
  };
  const int n0 = tiles_of(0), n1 = row_tiles == 2 ? tiles_of(1) : 0, tiles = max(n0, n1);
  const int nblk = blocks_of(t_end, A.lb);
  const int* row = A.table + (size_t)req * A.max_blocks;

  if (tid == 0) {
    s_abort = 0;
    s_ref = 0.0f;
    for (int s = 0; s < 2; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 4);
      mbar_init(&v_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 128);
      mbar_init(&o_full[s], 1);
    }
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  __syncthreads();
  // the largest value scale of the range (scales are not negative: their bits order them)
  {
    float top = 0.0f;
    for (int c = (t_begin >> A.lb) + tid; c < nblk; c += kTileThreads) {
      const int id = row[c];
      if (id >= 0 && id < A.n_blocks) top = fmaxf(top, A.vs[(size_t)id * A.kv + h]);
      else record_status(SVDQ_ERR_INVALID_ARG);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) atomicMax(reinterpret_cast<int*>(&s_ref), __float_as_int(top));
  }
  // queries, normalised, as the A operand; 16 (8) lanes a row
  if (warp < 8) {
    constexpr int PER = D / 8, RPI = 32 / PER;             // lanes per row, rows per instruction
    const int c = lane % PER;
#pragma unroll 4
    for (int k = 0; k < 32 / RPI; ++k) {
      const int rr = warp * 32 + k * RPI + lane / PER, r = r0 + rr;
      if (warp * 32 + k * RPI >= row_tiles * 128) break;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (r <= last)
        w = __ldg(reinterpret_cast<const uint4*>(A.q + (int64_t)(R.a + r / A.G) * A.q_stride + (int64_t)(h * A.G + r % A.G) * D) + c);
      float v[8], top = 0.0f;
      unpack8<DT>(w, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
#pragma unroll
      for (int o = PER / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = clampi((int)(__float_as_uint(top) >> 23) - 127, -100, 100);
      // the factor is kept non-negative (maxima are taken before it): a negative scale turns the query instead
      const float down = copysignf(__uint_as_float((uint32_t)(127 - e) << 23), A.scale_log2);
      uint8_t* dst = sq + (rr >> 7) * TB + (c >> 3) * kTileHalf + (rr & 127) * 128 + (((c & 7) ^ (rr & 7)) << 4);
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_half2(v[0] * down, v[1] * down), pack_half2(v[2] * down, v[3] * down),
                                                  pack_half2(v[4] * down, v[5] * down), pack_half2(v[6] * down, v[7] * down));
      if (c == 0) sf[rr] = __uint_as_float((uint32_t)(127 + e) << 23) * fabsf(A.scale_log2) * kUnit<FMT>;
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = s_tmem;
  const float vref = s_ref;

  if (warp < 8) {
    regs_inc<184>();
    const int rt = warp >> 2, n = rt == 0 ? n0 : n1;
    const uint32_t ts = tm + rt * 128 + ((uint32_t)(warp & 3) << 21), to = tm + 256 + rt * D + ((uint32_t)(warp & 3) << 21);
    const int r = r0 + rt * 128 + (tid & 127);
    const bool live = r <= last;
    if (rt < row_tiles) {
      const float f = sf[rt * 128 + (tid & 127)];
      const int see = live ? min(t_end, seen_by(A, R, r)) : t_end;
      const int clear = min(t_end, seen_by(A, R, r0 + rt * 128));
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < n; ++j) {
        const int t = t_begin + j * kTileTok;
        if (!mbar_wait(&s_full[rt], j & 1, &s_abort)) break;
        tc_fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld_32cols(ts + 32 * q, x[q]);
        tmem_ld_wait();
        const TileMeta* M = meta + (j & (kTileMeta - 1)) * 8;
        float a[8];
        int gone = 0;
#pragma unroll
        for (int g = 0; g < 8; ++g) { a[g] = f * M[g].sk; gone |= M[g].gone; }
        if (t + kTileTok > clear || gone) {
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const int lim = M[g].gone ? 0 : see - t - 16 * g;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              uint32_t& y = x[g >> 1][(g & 1) * 16 + i];
              y = __float_as_uint(i < lim ? __uint_as_float(y) * a[g] : -INFINITY);
            }
            a[g] = 1.0f;
          }
        }
        float top = m;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          float y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(x[g >> 1][(g & 1) * 16 + i]);
#pragma unroll
          for (int w = 8; w > 0; w >>= 1)
#pragma unroll
            for (int i = 0; i < w; ++i) y[i] = fmaxf(y[i], y[i + w]);
          top = fmaxf(top, y[0] * a[g]);
        }
        // a new reference maximum only where it grew by 2^8 (or is the first one)
        const bool grow = top > m + 8.0f;                  // m = -inf: any finite top
        if (__any_sync(0xffffffffu, grow)) {
          const float b = grow ? (m == -INFINITY ? 0.0f : ex2(m - top)) : 1.0f;
          if (grow) m = top;
          l *= b;
          if (j > 0) {
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
              uint32_t o[16];
              tmem_ld_16cols(to + 16 * q, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * b);
              tmem_st_16cols(to + 16 * q, o);
            }
          }
        }
        const float z = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int g2 = 0; g2 < 4; ++g2) {
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int g = 2 * g2 + k;
            const float b = M[g].lsv - z;
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float p0 = ex2(fmaf(__uint_as_float(x[g2][k * 16 + i]), a[g], b));
              const float p1 = ex2(fmaf(__uint_as_float(x[g2][k * 16 + i + 1]), a[g], b));
              s0 += p0;
              s1 += p1;
              p[k * 8 + i / 2] = pack_half2(p0, p1);
            }
            l = fmaf(s0 + s1, M[g].rsv, l);
          }
          tmem_st_16cols(ts + 16 * g2, p);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[rt]);
      }
      const bool whole = vis <= A.chunk;
      const int token = R.a + r / A.G, head = h * A.G + r % A.G;
      const bool ok = n == 0 || mbar_wait(&o_full[rt], 0, &s_abort);
      tc_fence_after();
      const size_t cell = ((size_t)split * A.n_tokens + token) * A.heads + head;
      const float u = vref * kUnit<FMT>, mul = whole ? (l > 0.0f ? __fdiv_rn(u, l) : 0.0f) : u;
      if (!whole && live) *reinterpret_cast<float2*>(A.part_ml + cell * 2) = make_float2(m, l);
#pragma unroll
      for (int q = 0; q < D / 16; ++q) {
        uint32_t o[16];
        if (n > 0 && ok) {
          tmem_ld_16cols(to + 16 * q, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0;
        }
        if (live) {
          float y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(o[i]) * mul;
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(A.out + (int64_t)token * A.out_stride + (int64_t)head * D + 16 * q);
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = (uint32_t)store16<DT>(y[2 * i]) | ((uint32_t)store16<DT>(y[2 * i + 1]) << 16);
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
          } else {
            float4* dst = reinterpret_cast<float4*>(A.part_o + cell * D + 16 * q);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
        }
      }
    }
  } else if (warp < 12) {
    regs_dec<96>();
    const int w = warp - 8, c = lane & 3, rl = 32 * w + (lane >> 2);   // rows rl + 8 i
    const size_t head_off = (size_t)h * (D << A.lb), blk_bytes = (size_t)A.kv * (D << A.lb);
    uint4 kr[4 * H], vr[4 * H];
    float g_sk = 0.0f, g_sv = 0.0f;
    int g_gone = 0, id[4];
    const auto ids = [&](int j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = (t_begin + j * kTileTok + rl + 8 * i) >> A.lb;
        const int v = b < nblk ? row[b] : -1;
        id[i] = v < A.n_blocks ? v : -1;
      }
    };
    const auto load = [&](const uint8_t* codes, int j, uint4 (&x)[4 * H]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int o = (t_begin + j * kTileTok + rl + 8 * i) & ((1 << A.lb) - 1);
        const uint4* at = reinterpret_cast<const uint4*>(codes + (id[i] < 0 ? 0 : id[i]) * blk_bytes + head_off + (size_t)o * D) + c;
#pragma unroll
        for (int q = 0; q < H; ++q) x[i * H + q] = id[i] >= 0 ? __ldg(at + 4 * q) : make_uint4(0, 0, 0, 0);
      }
    };
    // scales of this warp's two groups of 16 tokens: lanes 0-15 and 16-31 hold the first's and the second's
    const auto scales = [&]() {
      const int b = lane < 16 ? id[0] : id[2];
      g_gone = b < 0;
      g_sk = b < 0 ? 0.0f : A.ks[(size_t)b * A.kv + h];
      g_sv = b < 0 ? 0.0f : A.vs[(size_t)b * A.kv + h];
    };
    if (tiles > 0) {
      ids(0);
      load(A.kc, 0, kr);
      load(A.vc, 0, vr);
      scales();
    }
    for (int j = 0; j < tiles; ++j) {
      const int st = j & 1;
      if (j >= 2 && !mbar_wait(&k_empty[st], ((j >> 1) & 1) ^ 1, &s_abort)) break;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < H; ++q) store_codes<FMT>(sk + st * TB, rl + 8 * i, q, c, kr[i * H + q]);
      if ((lane & 15) == 0) {
        TileMeta* M = meta + (j & (kTileMeta - 1)) * 8 + 2 * w + (lane >> 4);
        // a scale below 2^-60 of the largest counts as that: its values are lost beside it either way
        const float ratio = vref > 0.0f ? fmaxf(__fdiv_rn(g_sv, vref), 0x1p-60f) : 1.0f;
        *M = TileMeta{g_sk, log2f(ratio), __fdiv_rn(1.0f, ratio), g_gone};
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[st]);
      if (j + 1 < tiles) {
        ids(j + 1);
        load(A.kc, j + 1, kr);
        scales();
      }
      if (j >= 2 && !mbar_wait(&v_empty[st], ((j >> 1) & 1) ^ 1, &s_abort)) break;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < H; ++q) store_codes<FMT>(sv + st * TB, rl + 8 * i, q, c, vr[i * H + q]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[st]);
      if (j + 1 < tiles) load(A.vc, j + 1, vr);
    }
  } else {
    regs_dec<48>();
    if (warp == 12 && lane == 0) {
      constexpr uint32_t kIdS = idesc_f16_f16(128, 128), kIdO = idesc_f16_f16(128, D) | (1u << 16);
      const auto issue_s = [&](int rt, int j) {
        const uint32_t a = smem_u32(sq + rt * TB), b = smem_u32(sk + (j & 1) * TB);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t o = (k >> 2) * kTileHalf + (k & 3) * 32;
          mma_f16(tm + rt * 128, desc_k_sw128(a + o), desc_k_sw128(b + o), kIdS, k > 0);
        }
        mma_commit(&s_full[rt]);
      };
      const auto issue_o = [&](int rt, int j) {
        const uint32_t b = smem_u32(sv + (j & 1) * TB);
#pragma unroll
        for (int k = 0; k < kTileTok / 16; ++k)
          mma_f16_ts(tm + 256 + rt * D, tm + rt * 128 + 8 * k, desc_mn_sw128(b + k * 2048), kIdO, j > 0 || k > 0);
      };
      bool ok = tiles == 0 || mbar_wait(&k_full[0], 0, &s_abort);
      if (ok && tiles > 0) {
        tc_fence_after();
        if (n0 > 0) issue_s(0, 0);
        if (n1 > 0) issue_s(1, 0);
        mma_commit(&k_empty[0]);
      }
      for (int j = 0; ok && j < tiles; ++j) {
        ok = mbar_wait(&v_full[j & 1], (j >> 1) & 1, &s_abort);
        if (ok && j + 1 < tiles) ok = mbar_wait(&k_full[(j + 1) & 1], ((j + 1) >> 1) & 1, &s_abort);
        for (int rt = 0; ok && rt < 2; ++rt) {
          const int n = rt == 0 ? n0 : n1;
          if (j >= n) continue;
          ok = mbar_wait(&p_full[rt], j & 1, &s_abort);
          if (!ok) break;
          tc_fence_after();
          issue_o(rt, j);
          if (j + 1 < n) issue_s(rt, j + 1);
          else mma_commit(&o_full[rt]);
        }
        if (!ok) break;
        mma_commit(&v_empty[j & 1]);
        if (j + 1 < tiles) mma_commit(&k_empty[(j + 1) & 1]);
      }
      if (!ok) {                                         // gave up: the MMAs in flight end before TMEM is freed
        int own = 0;
        mma_commit(drained);
        mbar_wait(drained, 0, &own);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

// Joins the splits of a row in a fixed order: a CTA per row, warp w takes splits w,
// w + 4, ..., then the warps in order.  Rows whose tokens fitted one split were
// written already.
constexpr int kJoinWarps = 4;
template <int DT, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const AttnArgs A, int tile_rows) {
  constexpr int V = D / 32;                              // values a lane
  __shared__ float s_v[kJoinWarps][D], s_m[kJoinWarps], s_l[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.x, h = blockIdx.y, req = blockIdx.z;
  griddep_wait();
  const Rows R = request_rows(A, req);
  if (r >= R.rows) return;
  const int vis = seen_by(A, R, min(R.rows, (r / tile_rows + 1) * tile_rows) - 1);
  if (vis <= A.chunk) return;
  const int n = (vis + A.chunk - 1) / A.chunk;
  const int token = R.a + r / A.G, head = h * A.G + r % A.G;
  const size_t cell = (size_t)token * A.heads + head, step = (size_t)A.n_tokens * A.heads;
  float m = -INFINITY, l = 0.0f, v[V];
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = 0.0f;
  for (int s0 = warp; s0 < n; s0 += 8 * kJoinWarps) {
    float2 ml[8];
    float x[8][V], top = m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int s = s0 + i * kJoinWarps;
      const size_t c = cell + (size_t)s * step;
      ml[i] = s < n ? *reinterpret_cast<const float2*>(A.part_ml + c * 2) : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int k = 0; k < V; ++k) x[i][k] = s < n ? A.part_o[c * D + V * lane + k] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, ml[i].x);
    const float b = m == -INFINITY ? 0.0f : ex2(m - top);
    m = top;
    l *= b;
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] *= b;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = ml[i].x == -INFINITY ? 0.0f : ex2(ml[i].x - m);
      l += w * ml[i].y;
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] += w * x[i][k];
    }
  }
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
  for (int k = 0; k < V; ++k) s_v[warp][V * lane + k] = v[k];
  __syncthreads();
  if (threadIdx.x >= D) return;
  float M = -INFINITY, L = 0.0f, y = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, s_m[w]);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float b = s_m[w] == -INFINITY ? 0.0f : ex2(s_m[w] - M);
    L += b * s_l[w];
    y += b * s_v[w][threadIdx.x];
  }
  A.out[(int64_t)token * A.out_stride + (int64_t)head * D + threadIdx.x] = store16<DT>(L > 0.0f ? __fdiv_rn(y, L) : 0.0f);
}

// ------------------------------------------------------------- host launchers
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

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
  if (c->heads < 1 || c->kv_heads < 1 || c->heads % c->kv_heads != 0 || c->n_blocks < 1 || c->heads > 65535)
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

svdq_status launched(const char* where) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SVDQ_OK : cuda_failure(e, where);
}

// The SM count that the split aims at: fixed, so that workspace sizes can be asked
// for without a device.
constexpr int kSplitSms = 148;

// How a call's rows and tokens are split: CTAs of `cta_rows` rows (8, 16: the few-row
// kernel; 128, 256: the tensor-core kernel) x `splits` ranges of tokens.  Up to
// kMaxCluster splits of the few-row kernel form a cluster, which shares each
// request's tokens evenly and joins in shared memory; otherwise a split is `chunk`
// tokens (a multiple of 128) and a second kernel joins them through the workspace.
struct Split { int cta_rows, row_ctas, splits, chunk, cluster; };
Split split_of(const svdq_paged_cache* c, const svdq_paged_batch* b, int sms) {
  Split s;
  const int64_t rows = (int64_t)b->max_new * (c->heads / c->kv_heads), cells = (int64_t)b->B * c->kv_heads;
  const auto ctas = [&](int per) { return (rows + per - 1) / per * cells; };
  const int64_t len = std::max(b->max_len, 1);
  if (rows <= 16) {
    s.cta_rows = rows <= 8 ? 8 : 16;
    s.row_ctas = 1;
    const int64_t unit = kDecWarps * kDecTile, want = std::min((4 * sms + cells - 1) / cells, (len + 2 * unit - 1) / (2 * unit));
    s.cluster = want > 1 && want <= kMaxCluster;
    s.splits = s.cluster ? (want > 4 ? 8 : want > 2 ? 4 : 2) : (int)std::max<int64_t>(1, want);
    s.chunk = (int)(((len + s.splits - 1) / s.splits + unit - 1) / unit * unit);
    if (!s.cluster) s.splits = (int)((len + s.chunk - 1) / s.chunk);
    return s;
  }
  s.cta_rows = rows > 128 && ctas(256) >= sms ? 256 : 128;
  s.row_ctas = (int)((rows + s.cta_rows - 1) / s.cta_rows);
  s.cluster = 0;
  const int64_t n = ctas(s.cta_rows), want = std::max<int64_t>(1, std::min((sms + n - 1) / n, (len + 1023) / 1024));
  s.chunk = (int)(((len + want - 1) / want + kTileTok - 1) / kTileTok * kTileTok);
  s.splits = (int)((len + s.chunk - 1) / s.chunk);
  return s;
}

size_t attention_ws(const svdq_paged_cache* c, const svdq_paged_batch* b) {
  const Split s = split_of(c, b, kSplitSms);
  if (s.splits <= 1 || s.cluster) return 16;
  return (size_t)s.splits * b->n_tokens * c->heads * (size_t)(c->head_dim + 2) * sizeof(float);
}

template <int DT, int FMT, int D, int NB>
cudaError_t launch_rows(const AttnArgs& A, const Split& s, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)s.splits, (unsigned)A.kv, (unsigned)A.B);
  cfg.blockDim = dim3(kDecWarps * 32);
  cfg.dynamicSmemBytes = dec_smem(D, NB);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)(s.cluster ? s.splits : 1);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_rows_kernel<DT, FMT, D, NB>, A, s.cluster);
}

template <int DT, int FMT, int D>
svdq_status launch_attention(const AttnArgs& A, const Split& s, cudaStream_t stream) {
  cudaError_t e;
  if (s.cta_rows <= 16) {
    e = s.cta_rows == 8 ? launch_rows<DT, FMT, D, 1>(A, s, stream) : launch_rows<DT, FMT, D, 2>(A, s, stream);
    if (e != cudaSuccess) return cuda_failure(e, "paged_rows_kernel launch");
  } else {
    const int64_t grid = (int64_t)s.splits * s.row_ctas * A.B * A.kv;
    if (grid > INT32_MAX) return SVDQ_ERR_UNSUPPORTED;
    paged_tiles_kernel<DT, FMT, D><<<(unsigned)grid, kTileThreads, tiles_smem(D), stream>>>(A, s.cta_rows);
    const svdq_status st = launched("paged_tiles_kernel launch");
    if (st != SVDQ_OK) return st;
  }
  if (s.splits <= 1 || s.cluster) return SVDQ_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(A.max_new * A.G), (unsigned)A.kv, (unsigned)A.B);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_join_kernel<DT, D>, A, s.cta_rows);
  return e == cudaSuccess ? SVDQ_OK : cuda_failure(e, "paged_join_kernel launch");
}

template <int DT, int FMT, int D>
svdq_status launch_append(const AppendArgs& A, int lb, dim3 grid, cudaStream_t s) {
  switch (lb) {
    case 4: paged_append_kernel<DT, FMT, D, 4><<<grid, kAppendThreads, 0, s>>>(A); break;
    case 5: paged_append_kernel<DT, FMT, D, 5><<<grid, kAppendThreads, 0, s>>>(A); break;
    case 6: paged_append_kernel<DT, FMT, D, 6><<<grid, kAppendThreads, 0, s>>>(A); break;
    default: paged_append_kernel<DT, FMT, D, 7><<<grid, kAppendThreads, 0, s>>>(A); break;
  }
  return launched("paged_append_kernel launch");
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
  cudaError_t e = cudaMemcpyFromSymbol(v, dev::g_status, sizeof(*v));
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
  int sms = 0;
  if ((st = device_ready(&sms)) != SVDQ_OK) return st;
  PlanArgs A;
  A.prev = prev; A.target = target; A.table = b->table; A.lens = b->lens; A.cu = b->cu; A.slots = b->slots;
  A.ring = ring; A.state_in = state_in; A.state_out = state_out;
  A.B = b->B; A.max_blocks = b->max_blocks; A.n_tokens = b->n_tokens; A.max_new = b->max_new; A.max_len = b->max_len;
  A.n_blocks = n_blocks; A.lb = lb;
  // a CTA per 2048 slots: up to there one CTA's scan and writes are cheaper than another CTA's scan
  const int ctas = (int)std::min<int64_t>(sms, std::max<int64_t>(1, ((int64_t)b->n_tokens + b->B + 2047) / 2048));
  paged_plan_kernel<<<ctas, kPlanThreads, plan_smem_bytes(b->B), reinterpret_cast<cudaStream_t>(stream)>>>(A);
  return launched("paged_plan_kernel launch");
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
  if (!aligned16(K) || !aligned16(V) || k_stride % 8 != 0 || v_stride % 8 != 0) return SVDQ_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = device_ready(&sms)) != SVDQ_OK) return st;
  AppendArgs A;
  A.x[0] = static_cast<const uint16_t*>(K); A.x[1] = static_cast<const uint16_t*>(V);
  A.stride[0] = k_stride; A.stride[1] = v_stride;
  A.codes[0] = c->kcodes; A.codes[1] = c->vcodes; A.scale[0] = c->kscale; A.scale[1] = c->vscale;
  A.cu = b->cu; A.slots = b->slots; A.B = b->B; A.n_tokens = b->n_tokens; A.kv = c->kv_heads; A.n_blocks = c->n_blocks;
  const int lb = log2_block(c->block_size);
  const dim3 grid((unsigned)((b->n_tokens >> lb) + 2 * b->B), (unsigned)c->kv_heads, 2u);
  return by_types(c, AppendCall{A, lb, grid, reinterpret_cast<cudaStream_t>(stream)});
}

size_t svdq_paged_attention_workspace_bytes(const svdq_paged_cache* c, const svdq_paged_batch* b) {
  if (check_cache(c) != SVDQ_OK || check_batch(b, c->block_size) != SVDQ_OK) return 0;
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
  const int64_t row = (int64_t)c->heads * c->head_dim;
  if (q_stride < row || out_stride < row) return SVDQ_ERR_INVALID_ARG;
  if (ws_bytes < attention_ws(c, b)) return SVDQ_ERR_WORKSPACE;
  if (!aligned16(Q) || !aligned16(out) || !aligned16(workspace) || q_stride % 8 != 0 || out_stride % 8 != 0)
    return SVDQ_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = device_ready(&sms)) != SVDQ_OK) return st;
  const Split sp = split_of(c, b, kSplitSms);
  AttnArgs A;
  A.q = static_cast<const uint16_t*>(Q); A.out = static_cast<uint16_t*>(out);
  A.kc = c->kcodes; A.vc = c->vcodes; A.ks = c->kscale; A.vs = c->vscale;
  A.table = b->table; A.lens = b->lens; A.cu = b->cu;
  A.part_o = static_cast<float*>(workspace);
  A.part_ml = A.part_o + (size_t)sp.splits * b->n_tokens * c->heads * c->head_dim;
  A.q_stride = q_stride; A.out_stride = out_stride;
  A.B = b->B; A.max_blocks = b->max_blocks; A.n_tokens = b->n_tokens; A.max_new = b->max_new; A.max_len = b->max_len;
  A.n_blocks = c->n_blocks; A.heads = c->heads; A.kv = c->kv_heads; A.G = c->heads / c->kv_heads;
  A.lb = log2_block(c->block_size); A.causal = causal; A.splits = sp.splits; A.chunk = sp.chunk;
  A.scale_log2 = scale * 1.4426950408889634f;
  return by_types(c, AttnCall{A, sp, reinterpret_cast<cudaStream_t>(stream)});
}

}  // extern "C"

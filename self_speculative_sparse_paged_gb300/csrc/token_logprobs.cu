// Log probability, rank and entropy of given tokens, and the most likely
// alternatives, in one read of the logits.
//
// For a row x of V logits, inverse temperature a, m = max x and
// Z = sum_i exp(a (x_i - m)):
//   logprob = a (x_tok - m) - ln Z,     entropy = ln Z - (1/Z) sum_i e_i a (x_i - m),
//   rank    = #{x_i > x_tok} + #{i < tok : x_i = x_tok},
//   top n   = the n largest logits above -inf, ties to the lower index.
//
// A cluster of CTAs shares a row.  Each thread streams 16-byte chunks with a
// running reference m (raised only when exceeded by 2^8, so the sums are
// rescaled a few times a row), fp32 sums of e and e (x - m), the rank's count
// and its own largest logit.  Instructions bound the stream before memory does,
// so pairs go through packed fp32 and (the maximum, the mask's clamp, the
// count) packed bf16 operations: about 8 instructions a logit.
// The n-th largest of the warps' four largest thread maxima bounds the n-th
// largest logit from below, so only the chunks of threads whose maximum reaches
// it are read again (by their whole warp, from L2); the logits that reach it
// are posted as unique 64-bit keys (value, then lower index first), and the n
// best of those are found by counting larger keys.  Should ties post more keys
// than the list holds, the n best are found one by one over the whole slice.
// Every CTA pushes its sums and its n keys to the cluster's first one through
// distributed shared memory, which joins them.
//
// 1000 rows of 151936 bf16 logits with 20 alternatives: 73 us, 4.2 TB/s (0.61 of
// the measured copy; instruction issue 67 % busy, the rest the rows' ends, where
// most warps wait for the few that find the n best).  240 rows of 50257 fp32
// logits: 14.2 us; 5 rows: 6.3 us, of which the stream is 1 us.
#include <cfloat>
#include <type_traits>

#include <cooperative_groups.h>

#include "kernels.h"
#include "vegas_common.cuh"

namespace cg = cooperative_groups;

namespace vegas {

namespace {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
// Batches of four chunks a thread asked for in L2 ahead of the loads (2 to 6 measured up to 15 % slower).
constexpr int kLpAhead = 1;
constexpr int kLpList = 1024;          // candidate keys a CTA can hold
constexpr float kLpSlack = 8.f;        // log2 units
constexpr float kLog2e = 1.4426950408889634f;

// A 16-byte chunk of logits: its values as fp32, or with -inf raised to the
// type's lowest; the maximum (of the raw values) of B chunks, and how many of
// their values lie above cmp (unordered: all of them where cmp is NaN).
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int N = 8;
  __nv_bfloat162 w[4];
  Chunk() = default;
  __device__ __forceinline__ explicit Chunk(const uint4& v) {
    w[0] = *reinterpret_cast<const __nv_bfloat162*>(&v.x);
    w[1] = *reinterpret_cast<const __nv_bfloat162*>(&v.y);
    w[2] = *reinterpret_cast<const __nv_bfloat162*>(&v.z);
    w[3] = *reinterpret_cast<const __nv_bfloat162*>(&v.w);
  }
  static __device__ __forceinline__ float2 wide(__nv_bfloat162 v) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&v);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  template <int B>
  static __device__ __forceinline__ float largest(const Chunk (&c)[B]) {
    __nv_bfloat162 m = __hmax2(__hmax2(c[0].w[0], c[0].w[1]), __hmax2(c[0].w[2], c[0].w[3]));
#pragma unroll
    for (int u = 1; u < B; ++u)
      m = __hmax2(m, __hmax2(__hmax2(c[u].w[0], c[u].w[1]), __hmax2(c[u].w[2], c[u].w[3])));
    const float2 f = wide(m);
    return fmaxf(f.x, f.y);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = wide(w[e]);
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
  __device__ __forceinline__ void finite(float (&x)[8]) const {
    const uint32_t low = 0xff7fff7fu;   // the lowest finite bf16, twice
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = wide(__hmax2(w[e], *reinterpret_cast<const __nv_bfloat162*>(&low)));
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
  using Cmp = __nv_bfloat162;
  static __device__ __forceinline__ Cmp pack(float x) { return __float2bfloat162_rn(x); }   // exact
  template <int B>
  static __device__ __forceinline__ float above(const Chunk (&c)[B], const Cmp (&cmp)[B]) {
    __nv_bfloat162 sum = __float2bfloat162_rn(0.f);   // counts to 4 B: exact in bf16
#pragma unroll
    for (int u = 0; u < B; ++u)
      sum = __hadd2(sum, __hadd2(__hadd2(__hgtu2(c[u].w[0], cmp[u]), __hgtu2(c[u].w[1], cmp[u])),
                                 __hadd2(__hgtu2(c[u].w[2], cmp[u]), __hgtu2(c[u].w[3], cmp[u]))));
    const float2 f = wide(sum);
    return f.x + f.y;
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  // the next number below x (not -inf) of this type
  static __device__ __forceinline__ float below(float x) {
    const uint32_t b = __float_as_uint(x);
    if ((b << 1) == 0) return __uint_as_float(0x80010000u);
    return __uint_as_float((b & 0x80000000u) ? b + 0x10000u : b - 0x10000u);
  }
};
template <>
struct Chunk<float> {
  static constexpr int N = 4;
  float w[4];
  Chunk() = default;
  __device__ __forceinline__ explicit Chunk(const uint4& v) {
    w[0] = __uint_as_float(v.x);
    w[1] = __uint_as_float(v.y);
    w[2] = __uint_as_float(v.z);
    w[3] = __uint_as_float(v.w);
  }
  template <int B>
  static __device__ __forceinline__ float largest(const Chunk (&c)[B]) {
    float m = c[0].w[0];
#pragma unroll
    for (int i = 1; i < 4 * B; ++i) m = fmaxf(m, c[i >> 2].w[i & 3]);
    return m;
  }
  __device__ __forceinline__ void values(float (&x)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = w[e];
  }
  __device__ __forceinline__ void finite(float (&x)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = fmaxf(w[e], -FLT_MAX);
  }
  using Cmp = float;
  static __device__ __forceinline__ Cmp pack(float x) { return x; }
  template <int B>
  static __device__ __forceinline__ float above(const Chunk (&c)[B], const Cmp (&cmp)[B]) {
    uint64_t sum = 0;
#pragma unroll
    for (int u = 0; u < B; ++u) {
      sum = add_f32x2(sum, pair_f32(set_gtu(c[u].w[0], cmp[u]), set_gtu(c[u].w[1], cmp[u])));
      sum = add_f32x2(sum, pair_f32(set_gtu(c[u].w[2], cmp[u]), set_gtu(c[u].w[3], cmp[u])));
    }
    float a, b;
    unpair_f32(sum, a, b);
    return a + b;
  }
  static __device__ __forceinline__ float set_gtu(float a, float b) {   // 1 or 0
    float r;
    asm("set.gtu.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ float below(float x) { return nextafterf(x, -INFINITY); }
};

// Unique order-preserving key: larger logit first, then the lower index.
// (x + 0 makes -0 equal to +0.)  A key of 0 stands for none.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ unsigned long long key_of(float x, int i) {
  return ((unsigned long long)order_of(x) << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float value_of(unsigned long long k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int index_of(unsigned long long k) { return (int)~(uint32_t)k; }

constexpr int kLpLead = 4;              // thread maxima a warp offers for the bound

// The sums of some logits relative to their maximum m: e = 2^((x - m) k) adds up to ones + s and
// e (x - m) to t.  The ones are kept apart: where one token has nearly all the probability, ln Z is
// ln(1 + s) of a small s, which the sum 1 + s would hold to 2^-24 only.
struct RowSums {
  float m, s, t;
  int ones;
};

struct LpShared {
  RowSums sums[kLpWarps];
  int cnt[kLpWarps];
  uint32_t lead[kLpWarps * kLpLead];    // as order_of()
  uint32_t bound;
  int posted;
  uint8_t owner[kLpWarps][32];
  unsigned long long best[kLpWarps];
  unsigned long long list[kLpList];
  // in the cluster's first CTA: what every CTA pushed
  RowSums parts[kMaxLogprobCluster];
  int count[kMaxLogprobCluster];
  unsigned long long all[kMaxLogprobCluster * kMaxTopLogprobs];
  float row_max, ln_z;
};

// (s, t) = sums of 2^((x - from) k) and of that times (x - from), moved to the reference `to`
// (>= from - slack; t stays in logit units).  Terms that vanish leave exact zeros.
__device__ __forceinline__ void move_sums(float from, float to, float k, float& s, float& t) {
  if (from > -INFINITY) {
    const float d = fmaxf(from - to, -FLT_MAX), f = ex2(d * k);
    t = f > 0.f ? f * fmaf(s, d, t) : 0.f;
    s *= f;
  } else {
    s = t = 0.f;
  }
}

// The sums of the first 2 * half lanes (the others hold none), joined at the largest maximum M.
__device__ __forceinline__ void join_sums(RowSums& v, float M, float k, int half) {
  if (v.m != M) {
    v.s += (float)v.ones;
    v.ones = 0;
    move_sums(v.m, M, k, v.s, v.t);
    v.m = M;
  }
  v.ones = __reduce_add_sync(0xffffffffu, v.ones);
#pragma unroll
  for (int o = half; o > 0; o >>= 1) {
    v.s += __shfl_xor_sync(0xffffffffu, v.s, o);
    v.t += __shfl_xor_sync(0xffffffffu, v.t, o);
  }
}

// a (x - m) for finite x <= m.  The difference alone may pass fp32's largest number (the lowest
// value beside a large maximum) where a brings it back: halves do not, and but for subnormal
// differences they round the same.
__device__ __forceinline__ float scaled_gap(float x, float m, float a) {
  return 2.f * ((0.5f * x - 0.5f * m) * a);
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kLpThreads, sizeof(T) == 2 ? 3 : 2)
    token_logprobs_kernel(const LogprobParams p) {
  constexpr int N = Chunk<T>::N;
  __shared__ LpShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = p.cluster, r = (int)cluster.block_rank();
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = p.top_n;
  if (r == 0)
    for (int i = tid; i < C * n; i += kLpThreads) sh.all[i] = 0;
  if (tid == 0) sh.posted = 0;
  // (waited for before the first push: the first CTA runs and its list is clear)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  griddep_begin();

  const T* x = reinterpret_cast<const T*>(p.logits) + size_t(row) * p.row_stride;
  const int V = p.vocab;
  int tok = p.tokens ? p.tokens[row] : -1;
  // Elements before the first 16-byte boundary and behind the last whole chunk
  // are taken one by one, by rank 0.
  const int skew = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const int head = min(V, skew ? N - skew : 0);
  const int chunks = (V - head) / N;
  const int tail0 = head + chunks * N, singles = head + (V - tail0);
  const int c0 = (int)((long long)chunks * r / C), c1 = (int)((long long)chunks * (r + 1) / C);
  const uint4* xc = reinterpret_cast<const uint4*>(x + head);
  auto single_at = [&](int i) { return i < head ? i : tail0 + (i - head); };
  const bool has_single = r == 0 && tid < singles;

  if (tok >= V) {
    if (tid == 0) set_error(p.err, kErrDeviceFault);
    tok = -1;
  }
  // One thread asks for the slice in L2 a few batches ahead of the loads.
  auto ahead = [&](int from, int chunks_wanted) {
    const int n16 = min(chunks_wanted, c1 - from);
    if (tid == 0 && n16 > 0)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(xc + from), "r"(n16 * 16)
                   : "memory");
  };
  ahead(c0, kLpAhead * 4 * kLpThreads);
  const float xt = tok >= 0 ? Chunk<T>::one(x + tok) : INFINITY;
  // x counts when x > xt, or x >= xt at a lower index: there x > (the number
  // below xt), or any x when xt = -inf (compared, unordered, with NaN)
  const float xt_low = xt == -INFINITY ? NAN : Chunk<T>::below(xt);
  const typename Chunk<T>::Cmp above_xt = Chunk<T>::pack(xt), above_low = Chunk<T>::pack(xt_low);
  const float k = p.inv_temperature * kLog2e, slack = kLpSlack / k;

  const int ctok = tok <= head ? 0 : (tok - head + N - 1) / N;   // chunks that begin before the token
  float m = -INFINITY, tm = -INFINITY;
  uint64_t s2 = 0, t2 = 0;   // pairs of partial sums
  int cnt = 0;
  float many = 0.f;          // counted in whole chunks: exact below 2^24 a thread
  auto raise = [&](float to) {
    if (to > m + slack) {   // (from -inf: any number)
      if (m > -INFINITY) {
        float sa, sb, ta, tb;
        unpair_f32(s2, sa, sb);
        unpair_f32(t2, ta, tb);
        move_sums(m, to, k, sa, ta);
        move_sums(m, to, k, sb, tb);
        s2 = pair_f32(sa, sb);
        t2 = pair_f32(ta, tb);
      }
      m = to;
    }
  };
  const uint64_t k2 = pair_f32(k, k);
  auto add2 = [&](float a, float b) {   // a, b finite or as low as the type goes
    const uint64_t u = add_f32x2(pair_f32(a, b), pair_f32(-m, -m));
    float ya, yb;
    unpair_f32(mul_f32x2(u, k2), ya, yb);
    const uint64_t e = pair_f32(ex2(ya), ex2(yb));
    s2 = add_f32x2(s2, e);
    t2 = fma_f32x2(e, u, t2);
  };
  auto add1 = [&](float v) {
    const float u = fmaxf(v - m, -FLT_MAX), e = ex2(u * k);
    s2 = add_f32x2(s2, pair_f32(e, 0.f));
    t2 = add_f32x2(t2, pair_f32(e * u, 0.f));
  };
  // B chunks, kLpThreads apart.  The branches are taken once per call.
  auto take = [&](auto batch, const uint4* raw, int c) {
    constexpr int B = decltype(batch)::value;
    Chunk<T> ch[B];
#pragma unroll
    for (int u = 0; u < B; ++u) ch[u] = Chunk<T>(raw[u]);
    const float mx = Chunk<T>::template largest<B>(ch);
    tm = fmaxf(tm, mx);
    raise(mx);
    if (fabsf(m) < 1e30f) {
#pragma unroll
      for (int u = 0; u < B; ++u) {
        float v[N];
        ch[u].finite(v);   // a masked logit counts 2^(-3e38 k) = 0, at a finite distance from m
#pragma unroll
        for (int e = 0; e < N; e += 2) add2(v[e], v[e + 1]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < B; ++u) {
        float v[N];
        ch[u].values(v);
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (v[e] > -INFINITY) add1(v[e]);
      }
    }
    // a chunk that begins before the token counts >= (the token's own is put right below)
    typename Chunk<T>::Cmp cmp[B];
#pragma unroll
    for (int u = 0; u < B; ++u)
      cmp[u] = c + u * kLpThreads < ctok ? above_low : above_xt;
    many += Chunk<T>::template above<B>(ch, cmp);
  };
  int c = c0 + tid;
  for (; c + 3 * kLpThreads < c1; c += 4 * kLpThreads) {
    ahead(c + kLpAhead * 4 * kLpThreads, 4 * kLpThreads);
    uint4 raw[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) raw[u] = __ldg(&xc[c + u * kLpThreads]);
    take(std::integral_constant<int, 4>{}, raw, c);
  }
  for (; c < c1; c += kLpThreads) {
    const uint4 raw = __ldg(&xc[c]);
    take(std::integral_constant<int, 1>{}, &raw, c);
  }
  if (tok > head && tok < tail0) {
    const int own = (tok - head) / N;   // its chunk counted the equal logits from the token on
    if (own < ctok && own >= c0 && own < c1 && (own - c0) % kLpThreads == tid) {
      float v[N];
      Chunk<T>(__ldg(&xc[own])).values(v);
#pragma unroll
      for (int e = 0; e < N; ++e) cnt -= v[e] == xt && head + own * N + e >= tok;
    }
  }
  if (has_single) {
    const int i = single_at(tid);
    const float v = Chunk<T>::one(x + i);
    tm = fmaxf(tm, v);
    raise(v);
    if (v > -INFINITY) add1(v);
    cnt += v > xt || (v == xt && i < tok);
  }

  // ---- the warp's sums, relative to its maximum, and its largest thread maxima
  {
    uint32_t left = order_of(tm);
    float Mw = -INFINITY;
#pragma unroll
    for (int j = 0; j < kLpLead; ++j) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, left);
      if (j == 0) Mw = value_of((unsigned long long)top << 32);
      if (lane == 0) sh.lead[warp * kLpLead + j] = top;
      const unsigned who = __ballot_sync(0xffffffffu, left == top);
      if (lane == __ffs(who) - 1) left = 0;
    }
    float s, t, sb, tb;
    unpair_f32(s2, s, sb);
    unpair_f32(t2, t, tb);
    // the thread's maximum (one of it) leaves the sums, as it was added, and counts one
    RowSums v{tm, 0.f, 0.f, 0};
    if (tm > -INFINITY) {
      const float u = fmaxf(tm - m, -FLT_MAX), e = ex2(u * k);
      const float sum = s + sb, z = sum - s, low = (s - (sum - z)) + (sb - z);   // sum + low = s + sb
      v.ones = 1;
      v.s = (sum - e) + low;
      v.t = t + fmaf(-e, u, tb);
      move_sums(m, tm, k, v.s, v.t);
    }
    join_sums(v, Mw, k, 16);
    cnt = __reduce_add_sync(0xffffffffu, cnt + (int)many);
    if (lane == 0) {
      sh.sums[warp] = v;
      sh.cnt[warp] = cnt;
    }
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  LpShared* first = cluster.map_shared_rank(&sh, 0);

  // the CTA's sums (last warp) and the bound on its n-th largest logit (first warps)
  if (warp == kLpWarps - 1) {
    const bool has = lane < kLpWarps;
    RowSums v = has ? sh.sums[lane] : RowSums{-INFINITY, 0.f, 0.f, 0};
    float M = v.m;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    join_sums(v, M, k, 8);
    const int total = __reduce_add_sync(0xffffffffu, has ? sh.cnt[lane] : 0);
    if (lane == 0) {
      first->parts[r] = v;
      first->count[r] = total;
    }
  }
  if (n > 0) {
    // the n-th largest of the offered maxima; each warp ranks its own against 32 at a time
    static_assert(kLpWarps * kLpLead == 64 && kLpLead * 16 >= kMaxTopLogprobs, "two per lane");
    const uint32_t lead0 = sh.lead[lane], lead1 = sh.lead[32 + lane];
#pragma unroll
    for (int j = 0; j < kLpLead; ++j) {
      const int i = warp * kLpLead + j;
      const uint32_t mine = __shfl_sync(0xffffffffu, i < 32 ? lead0 : lead1, i & 31);
      const int above =
          __popc(__ballot_sync(0xffffffffu, lead0 > mine || (lead0 == mine && lane < i))) +
          __popc(__ballot_sync(0xffffffffu, lead1 > mine || (lead1 == mine && 32 + lane < i)));
      if (above == n - 1 && lane == 0) sh.bound = mine;
    }
    __syncthreads();
    const uint32_t bound = sh.bound;
    auto post = [&](float v, int i) {
      if (v > -INFINITY && order_of(v) >= bound) {
        const int at = atomicAdd(&sh.posted, 1);
        if (at < kLpList) sh.list[at] = key_of(v, i);
      }
    };
    const bool reaches = tm > -INFINITY && order_of(tm) >= bound;
    const unsigned who = __ballot_sync(0xffffffffu, reaches);
    if (reaches) sh.owner[warp][__popc(who & ((1u << lane) - 1u))] = (uint8_t)lane;
    __syncwarp();
    if (reaches && has_single) post(Chunk<T>::one(x + single_at(tid)), single_at(tid));
    // the warp reads those threads' chunks, four a lane at a time
    const int each = (c1 - c0 + kLpThreads - 1) / kLpThreads, all = __popc(who) * each;
    for (int q0 = lane; q0 < all; q0 += 128) {
      uint4 raw[4];
      int at[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int q = q0 + 32 * u, o = q / each;
        at[u] = q < all ? c0 + warp * 32 + sh.owner[warp][o] + (q - o * each) * kLpThreads : c1;
        if (at[u] < c1) raw[u] = __ldg(&xc[at[u]]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (at[u] >= c1) continue;
        const Chunk<T> ch[1] = {Chunk<T>(raw[u])};
        if (order_of(Chunk<T>::template largest<1>(ch)) >= bound) {
          float v[N];
          ch[0].values(v);
#pragma unroll
          for (int e = 0; e < N; ++e) post(v[e], head + at[u] * N + e);
        }
      }
    }
    __syncthreads();
    const int posted = sh.posted;
    if (posted <= kLpList) {
      for (int i = warp; i < posted; i += kLpWarps) {   // a warp a key
        const unsigned long long mine = sh.list[i];
        int larger = 0;
        for (int j = 0; j < posted; j += 32)
          larger += __popc(__ballot_sync(0xffffffffu,
                                         j + lane < posted && sh.list[j + lane] > mine));
        if (larger < n && lane == 0) first->all[r * n + larger] = mine;
      }
    } else {
      unsigned long long last = ~0ull;
      for (int q = 0; q < n; ++q) {
        unsigned long long best = 0;
        auto see = [&](float v, int i) {
          if (v > -INFINITY) {
            const unsigned long long kk = key_of(v, i);
            if (kk < last && kk > best) best = kk;
          }
        };
        for (int cc = c0 + tid; cc < c1; cc += kLpThreads) {
          float v[N];
          Chunk<T>(__ldg(&xc[cc])).values(v);
#pragma unroll
          for (int e = 0; e < N; ++e) see(v[e], head + cc * N + e);
        }
        if (has_single) see(Chunk<T>::one(x + single_at(tid)), single_at(tid));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
          best = other > best ? other : best;
        }
        if (lane == 0) sh.best[warp] = best;
        __syncthreads();
        for (int w = 0; w < kLpWarps; ++w) best = sh.best[w] > best ? sh.best[w] : best;
        __syncthreads();
        if (tid == 0) first->all[r * n + q] = best;
        last = best;
        if (best == 0) break;
      }
    }
  }

  // ---- the row, in the cluster's first CTA; nothing reads the others' shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (r != 0) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    return;
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (warp == 0) {
    const bool has = lane < C;
    RowSums v = has ? sh.parts[lane] : RowSums{-INFINITY, 0.f, 0.f, 0};
    float M = v.m;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    join_sums(v, M, k, 8);
    const float s = (float)v.ones + v.s, t = v.t;
    const int count = __reduce_add_sync(0xffffffffu, has ? sh.count[lane] : 0);
    if (lane == 0) {
      const float ln_z = v.ones == 1 ? log1pf(v.s) : s > 0.f ? logf(s) : 0.f;
      sh.row_max = M;
      sh.ln_z = ln_z;
      if (p.logprob) {
        float lp = 0.f;
        if (tok >= 0) lp = xt > -INFINITY ? scaled_gap(xt, M, p.inv_temperature) - ln_z : -INFINITY;
        p.logprob[row] = lp;
      }
      if (p.rank) p.rank[row] = tok >= 0 ? count : -1;
      if (p.entropy) p.entropy[row] = s > 0.f ? ln_z - p.inv_temperature * (t / s) : 0.f;
    }
  }
  if (n > 0) {
    __syncthreads();   // row_max, ln_z
    int found = 0;
    for (int j = lane; j < C * n; j += 32) found += sh.all[j] != 0;
    found = __reduce_add_sync(0xffffffffu, found);
    for (int i = warp; i < C * n; i += kLpWarps) {
      const unsigned long long mine = sh.all[i];
      if (mine == 0) continue;
      int larger = 0;
      for (int j = 0; j < C * n; j += 32)
        larger += __popc(__ballot_sync(0xffffffffu, j + lane < C * n && sh.all[j + lane] > mine));
      if (larger < n && lane == 0) {
        p.top_ids[size_t(row) * n + larger] = index_of(mine);
        p.top_logprobs[size_t(row) * n + larger] =
            scaled_gap(value_of(mine), sh.row_max, p.inv_temperature) - sh.ln_z;
      }
    }
    if (tid >= found && tid < n) {   // fewer than n logits are left
      p.top_ids[size_t(row) * n + tid] = -1;
      p.top_logprobs[size_t(row) * n + tid] = -INFINITY;
    }
  }
}

template <typename T>
static cudaError_t launch_logprobs_t(const LogprobParams& p, cudaStream_t stream) {
  static std::atomic<uint32_t> configured{0};
  cudaError_t e = once_per_device(configured, [] {
    return cudaFuncSetAttribute(token_logprobs_kernel<T>,
                                cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.rows * p.cluster, 1, 1);
  cfg.blockDim = dim3(kLpThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T>, p);
}

cudaError_t launch_token_logprobs(const LogprobParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_logprobs_t<__nv_bfloat16>(p, stream) : launch_logprobs_t<float>(p, stream);
}

}  // namespace vegas

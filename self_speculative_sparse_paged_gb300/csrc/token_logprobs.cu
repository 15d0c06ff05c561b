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
// running reference maximum (raised only when exceeded by 2^8, so the sums are
// rescaled a few times a row), fp32 sums of e and e * y, the rank's count and
// its own largest logit.  The n-th largest of the threads' maxima bounds the
// n-th largest logit from below, so only threads whose maximum reaches it read
// their chunks again (from L2) and post the logits that reach it as unique
// 64-bit keys (value, then lower index first); the n best of those are found
// by counting larger keys.  Should ties post more keys than the list holds,
// the n best are found one by one over the whole slice.  The cluster's first
// CTA joins sums, counts and the CTAs' n keys through distributed shared memory.
#include <cooperative_groups.h>

#include "kernels.h"
#include "vegas_common.cuh"

namespace cg = cooperative_groups;

namespace vegas {

namespace {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpList = 1024;          // candidate keys a CTA can hold
constexpr float kLpSlack = 8.f;        // log2 units
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <>
struct Chunk<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};

// Unique order-preserving key: larger logit first, then the lower index.
// (x + 0 makes -0 equal to +0.)  A key of 0 stands for none.
__device__ __forceinline__ unsigned long long key_of(float x, int i) {
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((unsigned long long)o << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float value_of(unsigned long long k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int index_of(unsigned long long k) { return (int)~(uint32_t)k; }

struct LpShared {
  float m[kLpWarps], s[kLpWarps], t[kLpWarps];
  int cnt[kLpWarps];
  unsigned long long best[kLpWarps];
  float tmax[kLpThreads];
  float bound;
  int posted;
  unsigned long long list[kLpList];
  // the CTA's result, read by the cluster's first CTA
  float M, S, Tt;
  int count;
  unsigned long long top[32];
  unsigned long long all[32 * 16];
};

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_kernel(const LogprobParams p) {
  constexpr int N = Chunk<T>::N;
  __shared__ LpShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = p.cluster, r = C > 1 ? (int)cluster.block_rank() : 0;
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_begin();

  const T* x = reinterpret_cast<const T*>(p.logits) + size_t(row) * p.row_stride;
  const int V = p.vocab;
  int tok = p.tokens ? p.tokens[row] : -1;
  if (tok >= V) {
    if (tid == 0) set_error(p.err, kErrDeviceFault);
    tok = -1;
  }
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

  const float xt = tok >= 0 ? Chunk<T>::one(x + tok) : INFINITY;
  // x counts before the token when x > xt, or x >= xt at a lower index:
  // there x > (the number below xt), or any x when xt = -inf (not x <= NaN)
  const float xt_low = xt == -INFINITY ? NAN : nextafterf(xt, -INFINITY);
  const float k = p.inv_temperature * kLog2e;

  float m = -INFINITY, s = 0.f, t = 0.f, tm = -INFINITY;
  int cnt = 0;
  auto raise = [&](float to) {   // the reference maximum, with the sums moved to it
    if (to > -INFINITY && (m == -INFINITY || (to - m) * k > kLpSlack)) {
      if (m > -INFINITY) {
        const float d = (m - to) * k, f = ex2(d);
        t = f > 0.f ? f * (t + s * d) : 0.f;
        s *= f;
      }
      m = to;
    }
  };
  auto add = [&](float v) {
    const float y = fmaxf((v - m) * k, -200.f);   // (a masked logit: 2^-200 flushes to 0)
    const float e = ex2(y);
    s += e;
    t = fmaf(e, y, t);
  };
  auto take = [&](const uint4& raw, int c) {
    float v[N];
    Chunk<T>::unpack(raw, v);
    float mx = v[0];
#pragma unroll
    for (int e = 1; e < N; ++e) mx = fmaxf(mx, v[e]);
    tm = fmaxf(tm, mx);
    raise(mx);
#pragma unroll
    for (int e = 0; e < N; ++e) add(v[e]);
    const int i0 = head + c * N;
    if (tok >= i0 && tok < i0 + N) {
#pragma unroll
      for (int e = 0; e < N; ++e) cnt += v[e] > xt || (v[e] == xt && i0 + e < tok);
    } else {
      const float cmp = i0 < tok ? xt_low : xt;
#pragma unroll
      for (int e = 0; e < N; ++e) cnt += !(v[e] <= cmp);
    }
  };
  int c = c0 + tid;
  for (; c + 3 * kLpThreads < c1; c += 4 * kLpThreads) {
    uint4 raw[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) raw[u] = __ldg(&xc[c + u * kLpThreads]);
#pragma unroll
    for (int u = 0; u < 4; ++u) take(raw[u], c + u * kLpThreads);
  }
  for (; c < c1; c += kLpThreads) take(__ldg(&xc[c]), c);
  if (has_single) {
    const int i = single_at(tid);
    const float v = Chunk<T>::one(x + i);
    tm = fmaxf(tm, v);
    raise(v);
    add(v);
    cnt += v > xt || (v == xt && i < tok);
  }

  // ---- sums of the CTA
  float M = tm;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) sh.m[warp] = M;
  sh.tmax[tid] = tm;
  if (tid == 0) sh.posted = 0;
  __syncthreads();
  M = sh.m[0];
#pragma unroll
  for (int w = 1; w < kLpWarps; ++w) M = fmaxf(M, sh.m[w]);
  auto move_to = [&](float from, float to, float& ss, float& tt) {
    if (from > -INFINITY) {
      const float d = fmaxf((from - to) * k, -200.f), f = ex2(d);
      tt = f * (tt + ss * d);
      ss *= f;
    } else {
      ss = tt = 0.f;
    }
  };
  move_to(m, M, s, t);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
    cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
  }
  if (lane == 0) {
    sh.s[warp] = s;
    sh.t[warp] = t;
    sh.cnt[warp] = cnt;
  }

  // ---- the CTA's n best
  const int n = p.top_n;
  if (n > 0) {
    // the n-th largest of the threads' maxima
    int above = 0;
    const float4* t4 = reinterpret_cast<const float4*>(sh.tmax);
#pragma unroll 8
    for (int j = 0; j < kLpThreads / 4; ++j) {
      const float4 v = t4[j];
      above += (v.x > tm || (v.x == tm && 4 * j < tid)) + (v.y > tm || (v.y == tm && 4 * j + 1 < tid)) +
               (v.z > tm || (v.z == tm && 4 * j + 2 < tid)) + (v.w > tm || (v.w == tm && 4 * j + 3 < tid));
    }
    if (above == n - 1) sh.bound = tm;
    if (tid < 32) sh.top[tid] = 0;
    __syncthreads();
    const float bound = sh.bound;
    auto each = [&](auto&& f) {   // this thread's logits again
      for (int cc = c0 + tid; cc < c1; cc += kLpThreads) {
        float v[N];
        Chunk<T>::unpack(__ldg(&xc[cc]), v);
#pragma unroll
        for (int e = 0; e < N; ++e) f(v[e], head + cc * N + e);
      }
      if (has_single) f(Chunk<T>::one(x + single_at(tid)), single_at(tid));
    };
    if (tm >= bound && tm > -INFINITY)
      each([&](float v, int i) {
        if (v >= bound && v > -INFINITY) {
          const int at = atomicAdd(&sh.posted, 1);
          if (at < kLpList) sh.list[at] = key_of(v, i);
        }
      });
    __syncthreads();
    const int posted = sh.posted;
    if (posted <= kLpList) {
      for (int i = tid; i < posted; i += kLpThreads) {
        const unsigned long long mine = sh.list[i];
        int larger = 0;
        for (int j = 0; j < posted; ++j) larger += sh.list[j] > mine;
        if (larger < n) sh.top[larger] = mine;
      }
    } else {
      unsigned long long last = ~0ull;
      for (int q = 0; q < n; ++q) {
        unsigned long long best = 0;
        each([&](float v, int i) {
          if (v > -INFINITY) {
            const unsigned long long kk = key_of(v, i);
            if (kk < last && kk > best) best = kk;
          }
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
          best = other > best ? other : best;
        }
        if (lane == 0) sh.best[warp] = best;
        __syncthreads();
        for (int w = 0; w < kLpWarps; ++w) best = sh.best[w] > best ? sh.best[w] : best;
        __syncthreads();
        if (tid == 0) sh.top[q] = best;
        last = best;
        if (best == 0) break;
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    float S = 0.f, Tt = 0.f;
    int count = 0;
    for (int w = 0; w < kLpWarps; ++w) {
      S += sh.s[w];
      Tt += sh.t[w];
      count += sh.cnt[w];
    }
    sh.M = M;
    sh.S = S;
    sh.Tt = Tt;
    sh.count = count;
  }

  // ---- the row, in the cluster's first CTA
  if (C > 1)
    cluster.sync();
  else
    __syncthreads();
  if (r == 0) {
    float Mr = sh.M;
    for (int q = 1; q < C; ++q) Mr = fmaxf(Mr, cluster.map_shared_rank(&sh, q)->M);
    float S = 0.f, Tt = 0.f;
    int count = 0;
    for (int q = 0; q < C; ++q) {
      const LpShared* o = C > 1 ? cluster.map_shared_rank(&sh, q) : &sh;
      float ss = o->S, tt = o->Tt;
      move_to(o->M, Mr, ss, tt);
      S += ss;
      Tt += tt;
      count += o->count;
    }
    const float lnZ = S > 0.f ? logf(S) : 0.f;
    if (tid == 0) {
      if (p.logprob) {
        float lp = 0.f;
        if (tok >= 0) lp = xt > -INFINITY ? (xt - Mr) * p.inv_temperature - lnZ : -INFINITY;
        p.logprob[row] = lp;
      }
      if (p.rank) p.rank[row] = tok >= 0 ? count : -1;
      if (p.entropy) p.entropy[row] = S > 0.f ? lnZ - kLn2 * (Tt / S) : 0.f;
    }
    if (n > 0) {
      for (int i = tid; i < C * n; i += kLpThreads) {
        const int q = i / n;
        sh.all[i] = (C > 1 ? cluster.map_shared_rank(&sh, q) : &sh)->top[i - q * n];
      }
      if (tid < n) {
        p.top_ids[size_t(row) * n + tid] = -1;
        p.top_logprobs[size_t(row) * n + tid] = -INFINITY;
      }
      __syncthreads();
      for (int i = tid; i < C * n; i += kLpThreads) {
        const unsigned long long mine = sh.all[i];
        if (mine == 0) continue;
        int larger = 0;
        for (int j = 0; j < C * n; ++j) larger += sh.all[j] > mine;
        if (larger < n) {
          p.top_ids[size_t(row) * n + larger] = index_of(mine);
          p.top_logprobs[size_t(row) * n + larger] =
              (value_of(mine) - Mr) * p.inv_temperature - lnZ;
        }
      }
    }
  }
  if (C > 1) cluster.sync();   // no CTA leaves while its shared memory is read
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

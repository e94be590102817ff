// Routing of a mixture-of-experts layer: router logits -> the k experts of
// each token, their weights, and the dispatch plan that the grouped GEMMs and
// the combine read (pairs sorted by expert, tokens in order inside one).
//
// Selection orders the experts by a value: the logit itself without a bias (the
// scores are monotone in it), score + bias in float64 with one (float32 scores
// would tie or swap experts that the definition tells apart). A key is the
// value rounded to float32 as an unsigned integer of the same order, 0 for an
// expert that cannot be chosen; rounding is monotone, so only experts of equal
// keys need their float64 values compared, and that is rare. A token's experts
// lie in LANES lanes, NE neighbouring ones in each, so of equal values the
// lowest lane and the lowest register hold the lowest expert. A round takes the
// largest key: a register maximum, a rotation maximum over the 16-lane row
// (four lane-crossing maxima, no LDS), a ballot for the first lane that has it.
// Four tokens share a wave for up to 256 experts, and tokens of different
// waves do not wait for each other.
//
// Plan: workgroup c owns a chunk of consecutive tokens (at most 256 chunks)
// and counts its pairs per expert. The second kernel adds up the counts of all
// chunks and of those before its own, so every pair's place is known without
// a sort: segment start + pairs of earlier chunks + earlier tokens of the
// chunk with the same expert, the last by a 64-token bit mask per expert (a
// token takes an expert at most once). No order of atomics enters a result.
// One chunk (T <= 64) is routed and planned by one launch.

#include <type_traits>

#include "sharq_device.h"
#include "sharq_internal.h"

namespace sharq {
namespace {

constexpr int kMaxChunks = 256;
constexpr int kSlots = 64;  // largest k

template <int CTRL>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ uint64_t row_ror(uint64_t v) {
  return (uint64_t)row_ror<CTRL>((uint32_t)v) | (uint64_t)row_ror<CTRL>((uint32_t)(v >> 32)) << 32;
}
template <int CTRL>
__device__ __forceinline__ double row_ror(double v) {
  return __longlong_as_double((long long)row_ror<CTRL>((uint64_t)__double_as_longlong(v)));
}
template <int CTRL>
__device__ __forceinline__ float row_ror(float v) {
  return __uint_as_float(row_ror<CTRL>(__float_as_uint(v)));
}

// Reduction over a token's LANES lanes (16 or 64), the result in all of them.
template <int LANES, class T, class F>
__device__ __forceinline__ T token_reduce(T v, F f) {
  v = f(v, row_ror<0x128>(v));
  v = f(v, row_ror<0x124>(v));
  v = f(v, row_ror<0x122>(v));
  v = f(v, row_ror<0x121>(v));
  if constexpr (LANES == 64) {
    v = f(v, __shfl_xor(v, 16, 64));
    v = f(v, __shfl_xor(v, 32, 64));
  }
  return v;
}

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 and +0 are equal
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | (1ull << 63);
}

// NE logits of a row from expert e0 on; -inf for what cannot be chosen (no such
// expert, a padding row, -inf or NaN), +inf as the largest finite value.
template <int NE, class T>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int e0, int E, bool live, float (&x)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    float v = -__builtin_huge_valf();
    if (live && e0 + i < E) {
      if constexpr (std::is_same<T, uint16_t>::value)
        v = __uint_as_float((uint32_t)row[e0 + i] << 16);
      else
        v = (float)row[e0 + i];
    }
    x[i] = v > -__builtin_huge_valf() ? fminf(v, 3.4028234663852886e38f) : -__builtin_huge_valf();
  }
}

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

constexpr float kNegInf = -__builtin_huge_valf();

// The plan of one chunk: tokens [t0, t1), ids already in `expert`. totals[e]
// and before[e] (LDS) hold the pairs of expert e in all chunks and in those
// before this one; on return before[] is spent. All threads of the workgroup.
__device__ void plan_chunk(const RouteArgs& a, int64_t t0, int64_t t1, int* totals, int* before, uint64_t* bits,
                           int chunk, int chunks) {
  __shared__ int wave_sum[16];
  const int tid = threadIdx.x, nthreads = blockDim.x;
  // exclusive scan of totals over the experts, nthreads at a time
  int carry = 0;
  for (int e0 = 0; e0 < a.E; e0 += nthreads) {
    const int e = e0 + tid;
    const int v = e < a.E ? totals[e] : 0;
    int incl = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(incl, d, 64);
      if ((tid & 63) >= d) incl += u;
    }
    if ((tid & 63) == 63) wave_sum[tid >> 6] = incl;
    __syncthreads();
    int sum = carry;
    for (int w = 0; w < (tid >> 6); ++w) sum += wave_sum[w];
    int all = carry;
    for (int w = 0; w < (nthreads >> 6); ++w) all += wave_sum[w];
    if (e < a.E) {
      const int start = sum + incl - v;
      before[e] += start;
      if (chunk == 0) a.seg_offsets[e] = start;
    }
    carry = all;
    __syncthreads();
  }
  if (chunk == 0 && tid == 0) a.seg_offsets[a.E] = carry;
  // entries behind the last pair
  for (int64_t p = carry + (int64_t)chunk * nthreads + tid; p < a.T * a.k; p += (int64_t)chunks * nthreads)
    a.a_rows[p] = -1;
  const float per_token = 1.0f / (float)a.k;
  auto token_of = [&](int p) { return (int)(((float)p + 0.5f) * per_token); };  // p / k, exact for p < 4096
  for (int64_t s0 = t0; s0 < t1; s0 += 64) {
    const int pairs = (int)((t1 - s0 < 64 ? t1 - s0 : 64) * a.k);
    for (int e = tid; e < a.E; e += nthreads) bits[e] = 0;
    __syncthreads();
    for (int p = tid; p < pairs; p += nthreads) {
      const int e = a.expert[s0 * a.k + p];
      if (e >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&bits[e]), 1ull << token_of(p));
    }
    __syncthreads();
    for (int p = tid; p < pairs; p += nthreads) {
      const int e = a.expert[s0 * a.k + p], t = token_of(p);
      int at = -1;
      if (e >= 0) {
        at = before[e] + __popcll(bits[e] & ((1ull << t) - 1));
        a.a_rows[at] = (int32_t)(s0 + t);
      }
      a.pair_index[s0 * a.k + p] = at;
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += nthreads) before[e] += __popcll(bits[e]);
    __syncthreads();
  }
}

// LDS written by a wave and read by the same wave: in order as it is, kept so by the compiler.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Doubles of LDS that the groups of a token take: its values (or the two
// largest of each lane) and the groups' scores.
__host__ __device__ constexpr int group_doubles(int E, int groups, int lanes) {
  return (E > 2 * lanes ? E : 2 * lanes) + groups;
}

__device__ __forceinline__ void take_two(double v, double& first, double& second) {
  second = fmax(second, fmin(first, v));
  first = fmax(first, v);
}

// Clears the keys of experts outside the token's top_groups groups. v: what
// the groups compare, -inf for an expert that cannot be chosen; buf: the
// token's group_doubles in LDS.
template <int LANES, int NE>
__device__ __forceinline__ void keep_groups(const RouteArgs& a, const double (&v)[NE], uint32_t (&key)[NE], int lt,
                                            double* buf) {
  const int size = a.E / a.groups;
  double* gscore = buf + group_doubles(a.E, 0, LANES);
  const bool whole = size % NE == 0;  // a lane's experts belong to one group
  if (whole) {
    double first = kNegInf, second = kNegInf;
#pragma unroll
    for (int i = 0; i < NE; ++i) take_two(v[i], first, second);
    buf[2 * lt] = first;
    buf[2 * lt + 1] = second;
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (lt * NE + i < a.E) buf[lt * NE + i] = v[i];
  }
  wave_sync();
  const int per = whole ? 2 * (size / NE) : size;  // entries of a group
  for (int g = lt; g < a.groups; g += LANES) {
    double first = kNegInf, second = kNegInf;
    for (int e = g * per; e < (g + 1) * per; ++e) take_two(buf[e], first, second);
    gscore[g] = first + (a.sum2 && second > kNegInf ? second : 0.0);
  }
  wave_sync();
  int g = lt * NE / size, in = lt * NE - g * size, seen = -1;
  bool keep = false;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    if (g != seen && g < a.groups) {
      const double mine = gscore[g];
      int rank = 0;
      for (int o = 0; o < a.groups; ++o) {
        const double other = gscore[o];
        rank += other > mine || (other == mine && o < g);
      }
      keep = rank < a.top_groups;
      seen = g;
    }
    if (!keep) key[i] = 0;
    if (++in == size) in = 0, ++g;
  }
}

// Routes the tokens of chunk blockIdx.x. LDS: bit masks, counts and places of
// the experts, then k slots (expert, logit) of every token in flight, then,
// with groups, group_doubles of every token in flight.
template <int LANES, int NE, bool kBias>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a, int64_t chunk_tokens, int chunks) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int lt = lane % LANES;      // lane of the token
  const int slot = tid / LANES;     // token of the workgroup in flight
  const int flight = blockDim.x / LANES;
  uint64_t* bits = reinterpret_cast<uint64_t*>(lds);
  int* counts = reinterpret_cast<int*>(bits + a.E);
  int* before = counts + a.E;
  int2* chosen = reinterpret_cast<int2*>(before + a.E) + (int64_t)slot * a.k;
  double* gbuf = reinterpret_cast<double*>(reinterpret_cast<int2*>(before + a.E) + (int64_t)flight * a.k) +
                 (int64_t)slot * group_doubles(a.E, a.groups, LANES);
  for (int e = tid; e < a.E; e += blockDim.x) counts[e] = 0, before[e] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * chunk_tokens;
  const int64_t t1 = t0 + chunk_tokens < a.T ? t0 + chunk_tokens : a.T;
  const int64_t live_rows = a.num_tokens ? (int64_t)*a.num_tokens : a.T;
  const bool softmax = a.sigmoid == 0;
  auto add = [](double p, double q) { return p + q; };
  for (int64_t t = t0 + slot; t - lane / LANES < t1; t += flight) {  // uniform over a wave
    const bool row = t < t1 && t < live_rows;
    float x[NE];
    const int64_t at_row = row ? t * a.ld : 0;
    if (a.dtype == 0) load_row<NE>(static_cast<const float*>(a.logits) + at_row, lt * NE, a.E, row, x);
    else if (a.dtype == 1) load_row<NE>(static_cast<const uint16_t*>(a.logits) + at_row, lt * NE, a.E, row, x);
    else load_row<NE>(static_cast<const _Float16*>(a.logits) + at_row, lt * NE, a.E, row, x);
    double ref = 0.0, total = 1.0;  // softmax: the row's largest logit, and the sum of exp(x - ref)
    const bool all_scores = kBias || (a.groups > 1 && a.sum2);
    if (softmax && (all_scores || !a.renormalize)) {
      float top = x[0];
#pragma unroll
      for (int i = 1; i < NE; ++i) top = fmaxf(top, x[i]);
      top = token_reduce<LANES>(top, [](float p, float q) { return fmaxf(p, q); });
      if (top > kNegInf) ref = (double)top;
      total = 0.0;
#pragma unroll
      for (int i = 0; i < NE; ++i) total += exp((double)x[i] - ref);  // 0 for -inf
      total = token_reduce<LANES>(total, add);
    }
    uint32_t key[NE];
    double value[kBias ? NE : 1];
    if constexpr (kBias) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = min(lt * NE + i, a.E - 1);
        double v = (softmax ? exp((double)x[i] - ref) / total : sigmoid64(x[i])) + (double)a.bias[e];
        v = x[i] > kNegInf && v > kNegInf ? v : (double)kNegInf;
        value[i] = v;
        key[i] = v > kNegInf ? ordered((float)v) : 0;
      }
      if (a.groups > 1) keep_groups<LANES, NE>(a, value, key, lt, gbuf);
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) key[i] = x[i] > kNegInf ? ordered(x[i]) : 0;
      if (a.groups > 1) {
        double v[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i)
          v[i] = !(x[i] > kNegInf) ? (double)kNegInf
                 : !a.sum2         ? (double)x[i]
                 : softmax         ? exp((double)x[i] - ref) / total
                                   : sigmoid64(x[i]);
        keep_groups<LANES, NE>(a, v, key, lt, gbuf);
      }
    }
    // k rounds
    for (int j = 0; j < a.k; ++j) {
      uint32_t head = key[0];
#pragma unroll
      for (int i = 1; i < NE; ++i) head = max(head, key[i]);
      const uint32_t best = token_reduce<LANES>(head, [](uint32_t p, uint32_t q) { return max(p, q); });
      int at = 0, same = 0;
#pragma unroll
      for (int i = NE - 1; i >= 0; --i) {
        at = key[i] == best ? i : at;
        if constexpr (kBias) same += key[i] == best;
      }
      bool mine = head == best && best != 0;
      uint64_t have = __ballot(mine);
      auto of_token = [&](uint64_t m) {
        return LANES == 64 ? m : (m >> (lane & ~(LANES - 1))) & ((1ull << (LANES & 63)) - 1);
      };
      if constexpr (kBias) {  // several experts of this key: by their float64 values
        const uint64_t have_token = of_token(have);
        if (__any((mine && same > 1) || (have_token & (have_token - 1)) != 0)) {
          uint64_t top = 0;
#pragma unroll
          for (int i = 0; i < NE; ++i) top = key[i] == best && best != 0 ? max(top, ordered(value[i])) : top;
          const uint64_t highest = token_reduce<LANES>(top, [](uint64_t p, uint64_t q) { return p > q ? p : q; });
          mine = mine && top == highest;
          have = __ballot(mine);
#pragma unroll
          for (int i = NE - 1; i >= 0; --i) at = key[i] == best && ordered(value[i]) == highest ? i : at;
        }
      }
      const uint64_t token = of_token(have);
      const bool winner = mine && (token & ((1ull << lt) - 1)) == 0;
      if (winner || (token == 0 && lt == 0)) {
        float logit = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) logit = at == i ? x[i] : logit;
        chosen[j] = make_int2(winner ? lt * NE + at : -1, (int)__float_as_uint(logit));
      }
      if (!winner) at = -1;
#pragma unroll
      for (int i = 0; i < NE; ++i) key[i] = at == i ? 0 : key[i];
    }
    wave_sync();
    // weights, k slots over the token's lanes; renormalised ones relative to the largest chosen score, so that
    // they do not depend on how small the scores are
    double v[kSlots / LANES], w[kSlots / LANES], high = kNegInf, sum = 0.0;
#pragma unroll
    for (int s = 0; s < kSlots / LANES; ++s) {
      const int j = s * LANES + lt;
      v[s] = j < a.k && chosen[j].x >= 0 ? (double)__uint_as_float((uint32_t)chosen[j].y) : kNegInf;
      high = fmax(high, v[s]);
    }
    if (a.renormalize) high = token_reduce<LANES>(high, [](double p, double q) { return fmax(p, q); });
#pragma unroll
    for (int s = 0; s < kSlots / LANES; ++s) {
      w[s] = 0.0;
      if (v[s] > kNegInf) {
        if (!a.renormalize) w[s] = softmax ? exp(v[s] - ref) / total : sigmoid64(v[s]);
        else if (softmax) w[s] = exp(v[s] - high);
        else w[s] = v[s] > 0 ? sigmoid64(v[s]) : exp(v[s] - fmin(high, 0.0)) / (1.0 + exp(v[s]));
        sum += w[s];
      }
    }
    if (a.renormalize) {
      sum = token_reduce<LANES>(sum, add);
      sum = fmax(sum, 1e-300);
    } else {
      sum = 1.0;
    }
#pragma unroll
    for (int s = 0; s < kSlots / LANES; ++s) {
      const int j = s * LANES + lt;
      if (j < a.k && t < t1) {
        const int e = chosen[j].x;
        a.expert[t * a.k + j] = e;
        a.weight[t * a.k + j] = (float)(a.scale * (w[s] / sum));
        if (e >= 0) atomicAdd(&counts[e], 1);
      }
    }
    wave_sync();
  }
  __syncthreads();
  if (chunks == 1) {
    __threadfence_block();
    plan_chunk(a, t0, t1, counts, before, bits, 0, 1);
    return;
  }
  for (int e = tid; e < a.E; e += blockDim.x) a.counts[(int64_t)blockIdx.x * a.E + e] = counts[e];
}

// Places of chunk blockIdx.x from the counts of all chunks.
__global__ __launch_bounds__(1024) void moe_plan_kernel(RouteArgs a, int64_t chunk_tokens, int chunks) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  uint64_t* bits = reinterpret_cast<uint64_t*>(lds);
  int* totals = reinterpret_cast<int*>(bits + a.E);
  int* before = totals + a.E;
  const int tid = threadIdx.x, c = blockIdx.x;
  for (int e = tid; e < a.E; e += blockDim.x) totals[e] = 0, before[e] = 0;
  __syncthreads();
  // rows of the count table over groups of threads, an expert a thread
  const int width = a.E < (int)blockDim.x ? a.E : (int)blockDim.x;
  const int parts = blockDim.x / width, part = tid / width;
  if (part < parts)
    for (int e = tid - part * width; e < a.E; e += width) {
      int sum = 0, pre = 0;
#pragma unroll 8
      for (int r = part; r < chunks; r += parts) {
        const int v = a.counts[(int64_t)r * a.E + e];
        sum += v;
        pre += r < c ? v : 0;
      }
      atomicAdd(&totals[e], sum);
      atomicAdd(&before[e], pre);
    }
  __syncthreads();
  const int64_t t0 = (int64_t)c * chunk_tokens;
  plan_chunk(a, t0, t0 + chunk_tokens < a.T ? t0 + chunk_tokens : a.T, totals, before, bits, c, chunks);
}

// Tokens of a chunk: at most kMaxChunks chunks, 16 tokens or more; up to 64
// tokens in all are one chunk.
int64_t chunk_tokens(int64_t T) {
  if (T <= 64) return 64;
  const int64_t per = (T + kMaxChunks - 1) / kMaxChunks;
  return (per + 15) / 16 * 16;
}

template <int LANES, int NE>
void launch_route(const RouteArgs& a, int64_t per, int chunks, hipStream_t stream) {
  // tokens in flight: the chunk's, at most 256 threads' worth and 64 KB of LDS
  const int64_t token_bytes = 8 * a.k + (a.groups > 1 ? 8 * group_doubles(a.E, a.groups, LANES) : 0);
  const int64_t fixed = 16 * (int64_t)a.E;
  int64_t flight = (a.T < per ? a.T : per);
  if (flight > 256 / LANES) flight = 256 / LANES;
  if (flight < 1) flight = 1;
  while (flight > 1 && fixed + flight * token_bytes > 64 * 1024) flight /= 2;
  int threads = (int)((flight * LANES + 63) / 64 * 64);
  const size_t lds = (size_t)(fixed + (int64_t)(threads / LANES) * token_bytes);
  if (a.bias)
    hipLaunchKernelGGL((moe_route_kernel<LANES, NE, true>), dim3(chunks), dim3(threads), lds, stream, a, per, chunks);
  else
    hipLaunchKernelGGL((moe_route_kernel<LANES, NE, false>), dim3(chunks), dim3(threads), lds, stream, a, per, chunks);
}

}  // namespace

int64_t moe_route_workspace_bytes(int64_t T, int32_t E) {
  const int64_t per = chunk_tokens(T), chunks = (T + per - 1) / per;
  return chunks > 1 ? chunks * E * 4 : 0;
}

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream) {
  const int64_t per = chunk_tokens(a.T);
  const int chunks = a.T > 0 ? (int)((a.T + per - 1) / per) : 1;
  if (a.E <= 16) launch_route<16, 1>(a, per, chunks, stream);
  else if (a.E <= 32) launch_route<16, 2>(a, per, chunks, stream);
  else if (a.E <= 64) launch_route<16, 4>(a, per, chunks, stream);
  else if (a.E <= 128) launch_route<16, 8>(a, per, chunks, stream);
  else if (a.E <= 256) launch_route<16, 16>(a, per, chunks, stream);
  else if (a.E <= 512) launch_route<64, 8>(a, per, chunks, stream);
  else launch_route<64, 16>(a, per, chunks, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || chunks == 1) return e;
  const int threads = per * a.k >= 512 || a.E >= 512 ? 1024 : 512;
  hipLaunchKernelGGL(moe_plan_kernel, dim3(chunks), dim3(threads), 16 * (size_t)a.E, stream, a, per, chunks);
  return hipGetLastError();
}

}  // namespace sharq

// Routing of a mixture-of-experts layer: router logits -> the k experts of
// each token, their weights, and the dispatch plan that the grouped GEMMs and
// the combine read (pairs sorted by expert, tokens in order inside one).
//
// Selection orders the experts by a value: the logit itself without a bias (the
// scores are monotone in it), score + bias in float64 with one. Scores are
// first taken in float32 with a bound on their error; only where two of the
// values that decide (a round's largest and the next, two groups) lie within
// the bound is the order of the chosen found by their float64 values, or, where
// even the set is open, the wave's selection done again in float64, so the choice
// is float64's at about a third of its time. A token's experts lie in LANES lanes, NE
// neighbouring ones in each, so of equal values the lowest lane and the lowest
// register hold the lowest expert. A round takes the largest value as an
// unsigned integer of the same order (0: cannot be chosen): a register
// maximum, a rotation maximum over the 16-lane row and lane swaps beyond (no
// LDS), a ballot for the first lane that has it. Four tokens share a wave for
// up to 128 experts, and tokens of different waves do not wait for each other.
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

// f of a lane's value and that of the lane 16 or 32 away (rows of 16 or halves swapped, no LDS).
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
template <int D>
__device__ __forceinline__ v2u lane_swap(uint32_t v) {
  if constexpr (D == 16) return __builtin_amdgcn_permlane16_swap(v, v, false, false);
  else return __builtin_amdgcn_permlane32_swap(v, v, false, false);
}
template <int D, class T, class F>
__device__ __forceinline__ T swap_reduce(T v, F f) {
  if constexpr (sizeof(T) == 4) {
    const v2u p = lane_swap<D>(__builtin_bit_cast(uint32_t, v));
    return f(__builtin_bit_cast(T, (uint32_t)p[0]), __builtin_bit_cast(T, (uint32_t)p[1]));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const v2u lo = lane_swap<D>((uint32_t)u), hi = lane_swap<D>((uint32_t)(u >> 32));
    return f(__builtin_bit_cast(T, (uint64_t)hi[0] << 32 | lo[0]), __builtin_bit_cast(T, (uint64_t)hi[1] << 32 | lo[1]));
  }
}

// Reduction over a token's LANES lanes (16, 32 or 64), the result in all of them.
template <int LANES, class T, class F>
__device__ __forceinline__ T token_reduce(T v, F f) {
  v = f(v, row_ror<0x128>(v));
  v = f(v, row_ror<0x124>(v));
  v = f(v, row_ror<0x122>(v));
  v = f(v, row_ror<0x121>(v));
  if constexpr (LANES >= 32) v = swap_reduce<16>(v, f);
  if constexpr (LANES >= 64) v = swap_reduce<32>(v, f);
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

__device__ __forceinline__ float load_logit(const void* x, int dtype, int64_t i) {
  if (dtype == 0) return static_cast<const float*>(x)[i];
  if (dtype == 1) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(x)[i] << 16);
  return (float)static_cast<const _Float16*>(x)[i];
}

// NE logits of a row from expert e0 on; -inf for what cannot be chosen (no such
// expert, a padding row, -inf or NaN), +inf as the largest finite value. wide:
// rows are 16-byte aligned and a lane's experts are all there or all not.
template <class T>
__device__ __forceinline__ float widen(T v) {
  if constexpr (std::is_same<T, uint16_t>::value) return __uint_as_float((uint32_t)v << 16);
  else return (float)v;
}
template <int NE, class T>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int e0, int E, bool live, bool wide,
                                         float (&x)[NE]) {
  constexpr int kPer = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < NE; ++i) x[i] = -__builtin_huge_valf();
  if constexpr (NE % kPer == 0) {
    if (wide && live && e0 < E) {
      uint4 raw[NE / kPer];
#pragma unroll
      for (int q = 0; q < NE / kPer; ++q) raw[q] = reinterpret_cast<const uint4*>(row + e0)[q];
      T v[NE];
      __builtin_memcpy(v, raw, sizeof(v));
#pragma unroll
      for (int i = 0; i < NE; ++i) x[i] = widen(v[i]);
    }
  }
  if (NE % kPer != 0 || !wide) {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (live && e0 + i < E) x[i] = widen(row[e0 + i]);
  }
#pragma unroll
  for (int i = 0; i < NE; ++i)
    x[i] = x[i] > -__builtin_huge_valf() ? fminf(x[i], 3.4028234663852886e38f) : -__builtin_huge_valf();
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
  // this thread's first expert id, on its way while the scan runs
  const int first_id = tid < (t1 - t0 < 64 ? t1 - t0 : 64) * a.k ? a.expert[t0 * a.k + tid] : -1;
  auto id_of = [&](int64_t s0, int p) { return s0 == t0 && p == tid ? first_id : a.expert[s0 * a.k + p]; };
  // exclusive scan of totals over the experts, nthreads at a time
  int carry = 0;
  for (int e0 = 0; e0 < a.E; e0 += nthreads) {
    const int e = e0 + tid;
    const int v = e < a.E ? totals[e] : 0;
    const int incl = wave_inclusive_scan(v);
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
      const int e = id_of(s0, p);
      if (e >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&bits[e]), 1ull << token_of(p));
    }
    __syncthreads();
    for (int p = tid; p < pairs; p += nthreads) {
      const int e = id_of(s0, p), t = token_of(p);
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

// Doubles of LDS that the groups of a token take: its values (a.group_values of
// them), the groups' scores and which are kept. A group that is a power of two of
// whole lanes needs no values: its score is found by lane exchanges. (With the
// values always, 16384 x 256 with 8 groups had room for 16 tokens in flight
// instead of 32: 42 us, 35 so.)
__host__ __device__ inline int group_doubles(const RouteArgs& a) {
  return a.group_values + a.groups + (a.groups + 1) / 2;
}

template <class V>
__device__ __forceinline__ void take_two(V v, V& first, V& second) {
  second = max(second, min(first, v));
  first = max(first, v);
}

// Clears the keys of experts outside the token's top_groups groups. v: what
// the groups compare, -inf for an expert that cannot be chosen; buf: the
// token's group_doubles in LDS. True where scores at most `near` apart leave open
// whether a group stays (never for near < 0).
template <int LANES, int NE, class V, class Key>
__device__ __forceinline__ bool keep_groups(const RouteArgs& a, const V (&v)[NE], Key (&key)[NE], int lt, double* lds,
                                            V near) {
  const int size = a.E / a.groups;
  V* buf = reinterpret_cast<V*>(lds);
  V* gscore = buf + a.group_values;
  int* kept = reinterpret_cast<int*>(lds + a.group_values + a.groups);
  if (a.group_values == 0) {
    const int lanes = size / NE;
    // the two largest of each lane, then of the aligned lanes of a group
    V first = kNegInf, second = kNegInf;
#pragma unroll
    for (int i = 0; i < NE; ++i) take_two<V>(v[i], first, second);
    for (int d = 1; d < lanes; d <<= 1) {
      const V f = __shfl_xor(first, d, 64), s = __shfl_xor(second, d, 64);
      second = max(min(first, f), max(second, s));
      first = max(first, f);
    }
    if (lt % lanes == 0 && lt / lanes < a.groups)
      gscore[lt / lanes] = first + (a.sum2 && second > (V)kNegInf ? second : (V)0);
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (lt * NE + i < a.E) buf[lt * NE + i] = v[i];
    wave_sync();
    for (int g = lt; g < a.groups; g += LANES) {
      V first = kNegInf, second = kNegInf;
      for (int e = g * size; e < (g + 1) * size; ++e) take_two<V>(buf[e], first, second);
      gscore[g] = first + (a.sum2 && second > (V)kNegInf ? second : (V)0);
    }
  }
  wave_sync();
  bool close = false;
  for (int g = lt; g < a.groups; g += LANES) {
    const V mine = gscore[g];
    int rank = 0, above = 0, not_below = -1;  // -1: the group itself is not below
#pragma unroll 4
    for (int o = 0; o < a.groups; ++o) {
      const V other = gscore[o];
      rank += other > mine || (other == mine && o < g);
      above += other > mine + near;
      not_below += other >= mine - near;
    }
    kept[g] = rank < a.top_groups;
    close |= near >= 0 && mine > (V)kNegInf && above < a.top_groups && not_below >= a.top_groups;
  }
  wave_sync();
  int g = lt * NE / size, in = lt * NE - g * size;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    if (kept[min(g, a.groups - 1)] == 0) key[i] = 0;
    if (++in == size) in = 0, ++g;
  }
  wave_sync();
  return close;
}

__device__ __forceinline__ double score_exp(double x) { return exp(x); }
__device__ __forceinline__ float score_exp(float x) { return __expf(x); }
__device__ __forceinline__ double score_inverse(double x) { return 1.0 / x; }
__device__ __forceinline__ float score_inverse(float x) { return __builtin_amdgcn_rcpf(x); }

// What a selection by float32 values leaves to do.
enum : int { kTold, kOrder, kAgain };

// The k best experts of a wave's tokens, x their logits (-inf: cannot be
// chosen), into chosen[j] (an expert or -1). Where values of type V do not tell
// (V = double always does), the answer, the same for the wave, is kOrder if the
// first k + 1 (chosen[k] the first left out) are told from all others and only
// their order is open, else kAgain.
//
// Error of the float32 scores, u = 2^-24: exp(y), y a rounded difference, is
// off by at most (2.5 |y| + 2) u of it (the argument's two roundings, log2(e)'s
// and the instruction's), the reciprocal by 2 u, an addition by u. A sigmoid
// s = 1 / (1 + e): s (1 - s) (2.5 |x| + 2) u + 3 s u < 4e-7. A softmax score p =
// e / sum of at most 21 rounded additions of terms off by a mean of at most
// (2.5 ln 1024 + 2) u: p (2.5 |y| + 2 + 21 + 20 + 3) u < 3.5e-6 / sum, as p <=
// 1 / sum and p |y| < 0.37 / sum. Adding the bias rounds by u of the result.
// A key drops log2(NE) bits for the number of its register. Two values that
// follow each other in the order (the first two left out among them) and are
// closer than twice all that are taken for close.
template <int LANES, int NE, bool kBias, class V>
__device__ __forceinline__ int select(const RouteArgs& a, const float (&x)[NE], int lane, int* chosen,
                                       double* gbuf) {
  using Key = typename std::conditional<sizeof(V) == 8, uint64_t, uint32_t>::type;
  constexpr bool kRough = kBias && sizeof(V) == 4;
  const int lt = lane % LANES;
  const bool softmax = a.sigmoid == 0;
  Key key[NE];
  V value[NE];
  V bound = 0;
  bool again = false, order = false, last_close = false;
  const bool scores = kBias || (a.groups > 1 && a.sum2);
  if (scores) {
    V ref = 0, inv = 1;
    if (softmax) {
      float top = x[0];
#pragma unroll
      for (int i = 1; i < NE; ++i) top = fmaxf(top, x[i]);
      top = token_reduce<LANES>(top, [](float p, float q) { return fmaxf(p, q); });
      if (top > kNegInf) ref = (V)top;
      V total = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) total += score_exp((V)x[i] - ref);  // 0 for -inf
      total = token_reduce<LANES>(total, [](V p, V q) { return p + q; });
      inv = score_inverse(total);
    }
    bound = softmax ? (V)3.5e-6 * inv : (V)4e-7;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      V v = softmax ? score_exp((V)x[i] - ref) * inv : score_inverse((V)1 + score_exp(-(V)x[i]));
      if constexpr (kBias) v += (V)a.bias[min(lt * NE + i, a.E - 1)];
      value[i] = x[i] > kNegInf && v > (V)kNegInf ? v : (V)kNegInf;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i) value[i] = (V)x[i];
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const V v = kBias ? value[i] : (V)x[i];
    key[i] = v > (V)kNegInf ? ordered(v) : 0;
    if constexpr (kRough) key[i] = key[i] ? (key[i] & ~(Key)(NE - 1)) | (NE - 1 - i) : 0;  // says its register
  }
  if (a.groups > 1) {
    V near = -1;
    if (sizeof(V) == 4 && scores) {  // sums of up to two values, and their rounding
      V most = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) most = value[i] > (V)kNegInf ? max(most, (V)fabs(value[i])) : most;
      most = token_reduce<LANES>(most, [](V p, V q) { return p > q ? p : q; });
      near = 4 * bound + most * (V)5e-7;
      again = !(most < (V)8.5e37);  // below 2^126, so that no sum of two, nor a score + near, passes float32's range
    }
    again |= keep_groups<LANES, NE, V, Key>(a, value, key, lt, gbuf, near);
  }
  for (int j = lt; j < a.k + (kBias ? 1 : 0); j += LANES) chosen[j] = -1;
  wave_sync();
  // the lanes of this lane's token below it, in a half of a ballot
  const uint32_t shift = lane & 31 & ~(LANES - 1);
  const uint32_t below = ((1u << (lt & 31)) - 1u) << shift;
  auto lanes_of = [&](uint64_t m) { return lane < 32 ? (uint32_t)m : (uint32_t)(m >> 32); };
  float last = 0.0f;
  for (int j = 0; j < a.k + (kRough ? 2 : 0); ++j) {
    Key head = key[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) head = max(head, key[i]);
    const Key best = token_reduce<LANES>(head, [](Key p, Key q) { return max(p, q); });
    if constexpr (kRough) {  // the one before, and this one: far enough apart to tell? (NaN, of infinities, is not)
      const float v = __uint_as_float((uint32_t)(best >> 31 ? best ^ 0x80000000u : ~best));
      const float rounding = (float)(NE + 1) * 1.2e-7f * fmaxf(fabsf(v), fabsf(last));
      const bool close = j > 0 && best != 0 && !(last - v > 2.0f * ((float)bound + rounding));
      if (j == a.k + 1) {  // the last chosen, the first and the second left out: all close?
        again |= last_close && close;
        break;
      }
      order |= close;
      last_close = close;
      last = v;
    }
    const bool has = head == best && best != 0;
    const uint64_t have = __ballot(has);
    const bool first = LANES == 64 ? (have & ((1ull << lt) - 1)) == 0 : (lanes_of(have) & below) == 0;
    int at = -1;
    if constexpr (kRough) {
      if (has && first) at = NE - 1 - (int)(best & (NE - 1));
    } else {
#pragma unroll
      for (int i = NE - 1; i >= 0; --i) at = key[i] == best ? i : at;
      if (!(has && first)) at = -1;
    }
    if (at >= 0) chosen[j] = lt * NE + at;
#pragma unroll
    for (int i = 0; i < NE; ++i) key[i] = at == i ? 0 : key[i];
  }
  wave_sync();
  return __any(again) ? kAgain : __any(order) ? kOrder : kTold;
}

// chosen[0 .. k] into the order of float64's sigmoid + bias, a lane a slot (k <
// LANES). Lanes of tokens whose order was told find it again. One such wave in a
// launch is common (a pair of 4096 tokens' first nine of 128 is close in most of
// them) and decides its time: with the whole selection again instead, 4096 x 128
// with a bias 17.2 us, 15.3 so, with 4 of 8 groups 19.0 and 16.3.
template <int LANES>
__device__ __forceinline__ void order_chosen(const RouteArgs& a, int64_t t, int lane, int* chosen) {
  const int lt = lane % LANES;
  const int e = lt <= a.k ? chosen[lt] : -1;
  double v = kNegInf;
  if (e >= 0)
    v = sigmoid64((double)fminf(load_logit(a.logits, a.dtype, t * a.ld + e), 3.4028234663852886e38f)) +
        (double)a.bias[e];
  int rank = 0;
  for (int i = 0; i <= a.k; ++i) {
    const double other = __shfl(v, i, LANES);
    const int id = __shfl(e, i, LANES);
    rank += id >= 0 && (other > v || (other == v && id < e));
  }
  wave_sync();
  if (e >= 0 && rank < a.k) chosen[rank] = e;
  wave_sync();
}

// Threads of a routing workgroup: 1024 (128 registers a lane), 512 where a lane
// holds 16 experts.
template <int NE>
constexpr int kRouteThreads = NE <= 8 ? 1024 : 512;

// Routes the tokens of chunk blockIdx.x. LDS: bit masks, counts and places of
// the experts, then k slots (with a bias k + 1) of every token in flight, then, with groups,
// group_doubles of every token in flight. Bound by the chain of a token (load,
// k rounds of a maximum over its lanes, float64 weights) at few tokens: 1 x 128, k
// = 8: 6.3 us; 4096 x 128 bf16: 7.0 us. At many by vector instructions and by
// waiting, about half and half: 16384 x 256 with bias and 4 of 8 groups 27-28 us
// (16.8 MB read, 2.1 MB written: 4 us at the rate of a copy) with 10.0k vector
// instructions a SIMD, 17 us at four cycles each and 2.4 GHz. A CU holds one workgroup,
// four waves a SIMD, and a wave waits for 55% of its cycles.
template <int LANES, int NE, bool kBias>
__global__ __launch_bounds__(kRouteThreads<NE>) void moe_route_kernel(RouteArgs a, int64_t chunk_tokens, int chunks) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int lt = lane % LANES;      // lane of the token
  const int slot = tid / LANES;     // token of the workgroup in flight
  const int flight = blockDim.x / LANES;
  uint64_t* bits = reinterpret_cast<uint64_t*>(lds);
  int* counts = reinterpret_cast<int*>(bits + a.E);
  int* before = counts + a.E;
  const int slots = a.k + (kBias ? 1 : 0);
  int* chosen = before + a.E + (int64_t)slot * slots;
  double* gbuf = reinterpret_cast<double*>(before + a.E + ((int64_t)flight * slots + 1) / 2 * 2) +
                 (int64_t)slot * group_doubles(a);
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
    const int item = a.dtype == 0 ? 4 : 2;
    const bool wide = ((reinterpret_cast<uintptr_t>(a.logits) | (uintptr_t)(a.ld * item)) & 15) == 0 && a.E % NE == 0;
    if (a.dtype == 0) load_row<NE>(static_cast<const float*>(a.logits) + at_row, lt * NE, a.E, row, wide, x);
    else if (a.dtype == 1) load_row<NE>(static_cast<const uint16_t*>(a.logits) + at_row, lt * NE, a.E, row, wide, x);
    else load_row<NE>(static_cast<const _Float16*>(a.logits) + at_row, lt * NE, a.E, row, wide, x);
    const int left = select<LANES, NE, kBias, float>(a, x, lane, chosen, gbuf);
    if (kBias && left == kOrder && !softmax && a.k < LANES) order_chosen<LANES>(a, t, lane, chosen);
    else if (left != kTold) select<LANES, NE, kBias, double>(a, x, lane, chosen, gbuf);
    double ref = 0.0, total = 1.0;  // softmax: the row's largest logit, and the sum of exp(x - ref)
    if (softmax && !a.renormalize) {
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
    // weights, k slots over the token's lanes; renormalised ones relative to the largest chosen score, so that
    // they do not depend on how small the scores are
    double v[kSlots / LANES], w[kSlots / LANES], high = kNegInf, sum = 0.0;
#pragma unroll
    for (int s = 0; s < kSlots / LANES; ++s) {
      const int j = s * LANES + lt;
      const int e = j < a.k ? chosen[j] : -1;
      v[s] = e >= 0 ? (double)fminf(load_logit(a.logits, a.dtype, t * a.ld + e), 3.4028234663852886e38f) : kNegInf;
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
        const int e = chosen[j];
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

// Places of chunk blockIdx.x from the counts of all chunks: every workgroup
// reads the whole table (at most 256 rows, in L2) rather than wait for a scan
// of it in a launch between. 4096 x 128, k = 8: 6.2 us; 16384 x 256: 7.8 us.
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
      // rows on their way together: 32, then 4 at a time (the last row again behind the end)
      const int32_t* at = a.counts + (part * a.E + e);
      const int step = parts * a.E;
      int r = part;
      for (; r + 31 * parts < chunks; r += 32 * parts, at += 32 * step) {
        int v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = at[i * step];
#pragma unroll
        for (int i = 0; i < 32; ++i) sum += v[i], pre += r + i * parts < c ? v[i] : 0;
      }
      for (; r < chunks; r += 4 * parts, at += 4 * step) {
        int v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = r + i * parts < chunks ? at[i * step] : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += v[i], pre += r + i * parts < c ? v[i] : 0;
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
void launch_route(RouteArgs a, int64_t per, int chunks, hipStream_t stream) {
  const int size = a.E / a.groups, lanes = size / NE;
  a.group_values = size % NE == 0 && (lanes & (lanes - 1)) == 0 ? 0 : a.E;
  // tokens in flight: the chunk's, at most a workgroup's worth and 64 KB of LDS, in whole waves
  const int64_t token_bytes = 4 * (a.k + (a.bias ? 1 : 0)) + (a.groups > 1 ? 8 * group_doubles(a) : 0);
  const int64_t fixed = 16 * (int64_t)a.E + 8;  // 8: the groups' doubles are aligned
  constexpr int64_t kWaveTokens = 64 / LANES;
  int64_t waves = ((a.T < per ? a.T : per) + kWaveTokens - 1) / kWaveTokens;
  if (waves > kRouteThreads<NE> / 64) waves = kRouteThreads<NE> / 64;
  if (waves < 1) waves = 1;
  while (waves > 1 && fixed + waves * kWaveTokens * token_bytes > 64 * 1024) waves /= 2;
  const int threads = (int)(64 * waves);
  const size_t lds = (size_t)(fixed + waves * kWaveTokens * token_bytes);
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
  else if (a.E <= 256) launch_route<32, 8>(a, per, chunks, stream);
  else if (a.E <= 512) launch_route<64, 8>(a, per, chunks, stream);
  else launch_route<64, 16>(a, per, chunks, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || chunks == 1) return e;
  hipLaunchKernelGGL(moe_plan_kernel, dim3(chunks), dim3(1024), 16 * (size_t)a.E, stream, a, per, chunks);
  return hipGetLastError();
}

}  // namespace sharq

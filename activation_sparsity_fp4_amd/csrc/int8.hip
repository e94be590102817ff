// 8-bit integer coding with one scale a row (activations: a token, weights: an
// output channel), and the layout of the codes.
//
//   amax = max_k |x'[k]|,  s = fp32(amax / 127),  q[k] = clamp(rne(x'[k] / s), -127, 127)
//
// with x' = x, or the RMS-normed row bf16(x r) gamma. The quotient is the exact
// one, not its fp32 rounding. t = fma(x', 1 / s, 1.5 2^23) holds the integer nearest
// to x' (1 / s), which is at most 127 2^-24 off the quotient, so that q is the code
// or its neighbour. The rest x' - q s is one fma, exact (a multiple of the last bit
// of s or of x' below s), so q is the code wherever |rest| < s / 2; a thread that
// holds another entry settles its piece by the rest's sign. Rows of zeros have scale
// 0; a row that holds a NaN or an infinity has scale NaN and codes of zero, so that
// products with it are NaN.
//
// Layout: codes i8 [G][rows][64], G = ceil(K / 64), zeros past K: a stage of 64
// entries a row is the 64-byte row that the GEMM's LDS stage holds.

#include <type_traits>

#include "gemm_common.h"
#include "sharq_device.h"
#include "sharq_internal.h"

namespace sharq {
namespace {

constexpr int kPiece = 16;  // entries that a lane codes together: 16 bytes of codes

// The entries of a piece as they were loaded: two to a dword, or fp32.
template <class In>
struct Piece {
  static constexpr int kWords = sizeof(In) * kPiece / 4;
  uint32_t w[kWords];
};

__device__ __forceinline__ void widen(const Piece<uint16_t>& p, float (&v)[kPiece]) {  // bf16
#pragma unroll
  for (int i = 0; i < kPiece / 2; ++i) v[2 * i] = bf16_lo(p.w[i]), v[2 * i + 1] = bf16_hi(p.w[i]);
}
__device__ __forceinline__ void widen(const Piece<_Float16>& p, float (&v)[kPiece]) {
#pragma unroll
  for (int i = 0; i < kPiece / 2; ++i) {
    v[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)p.w[i]);
    v[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(p.w[i] >> 16));
  }
}
__device__ __forceinline__ void widen(const Piece<float>& p, float (&v)[kPiece]) {
#pragma unroll
  for (int i = 0; i < kPiece; ++i) v[i] = __uint_as_float(p.w[i]);
}

// Entries [16 p, 16 p + 16) of a row of K; those past K are zeros. kWide: K is a
// multiple of 8 and the row 16-byte aligned.
template <class In, bool kWide>
__device__ __forceinline__ Piece<In> load_piece(const In* __restrict__ row, uint32_t p, uint32_t K) {
  Piece<In> out;
#pragma unroll
  for (int i = 0; i < Piece<In>::kWords; ++i) out.w[i] = 0;
  if constexpr (kWide) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (kPiece * p + 8 * h < K) {
        constexpr int kHalf = Piece<In>::kWords / 2;
        const uint4* src = reinterpret_cast<const uint4*>(row + (uint64_t)kPiece * p + 8 * h);
#pragma unroll
        for (int i = 0; i < kHalf / 4; ++i) {
          const uint4 v = src[i];
          uint32_t* w = out.w + kHalf * h + 4 * i;
          w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        }
      }
  } else {
#pragma unroll
    for (int e = 0; e < kPiece; ++e) {
      const uint32_t k = kPiece * p + e;
      if (k < K) {
        if constexpr (sizeof(In) == 4) out.w[e] = __float_as_uint(row[k]);
        else out.w[e / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, row[k]) << (16 * (e & 1));
      }
    }
  }
  return out;
}

// Largest magnitude of a piece as a bit pattern of its type (NaN above infinity
// above all numbers), joined to m: two 16-bit patterns in a dword, or fp32's.
typedef unsigned short v2us __attribute__((ext_vector_type(2)));
template <class In>
__device__ __forceinline__ uint32_t join_amax(uint32_t m, const Piece<In>& p) {
#pragma unroll
  for (int i = 0; i < Piece<In>::kWords; ++i) {
    if constexpr (sizeof(In) == 4)
      m = max(m, p.w[i] & 0x7FFFFFFFu);
    else
      m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2us, m),
                                                                 __builtin_bit_cast(v2us, p.w[i] & 0x7FFF7FFFu)));
  }
  return m;
}
// The fp32 bits of the magnitude that join_amax found.
template <class In>
__device__ __forceinline__ uint32_t amax_f32(uint32_t m) {
  if constexpr (sizeof(In) == 4) return m;
  const uint32_t h = max(m & 0xFFFFu, m >> 16);
  if constexpr (std::is_same<In, uint16_t>::value) return h << 16;
  else return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)h));
}

// Over the wave, in all lanes: rotations within the rows of 16 lanes, then the four rows' values.
template <int kBy>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + kBy, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, row_ror<8>(v));
  v = max(v, row_ror<4>(v));
  v = max(v, row_ror<2>(v));
  v = max(v, row_ror<1>(v));
  uint32_t m = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) m = max(m, (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * r));
  return m;
}
template <int kBy>
__device__ __forceinline__ double row_ror_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)row_ror<kBy>((uint32_t)(b >> 32)) << 32 | row_ror<kBy>((uint32_t)b));
}
__device__ __forceinline__ double wave_sum(double v) {
  v += row_ror_f64<8>(v);
  v += row_ror_f64<4>(v);
  v += row_ror_f64<2>(v);
  v += row_ror_f64<1>(v);
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  double s = 0.0;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    s += __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), 16 * r) << 32 |
                                        (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 16 * r));
  return s;
}

// How a row is divided: x' up (1 / (s up)), up a power of two that keeps the
// reciprocal of a small scale finite.
struct Divisor {
  float up, scale, inverse;  // scale: s up
  bool tiny;                 // s may have lost bits of amax / 127, so that codes pass 127
};

__device__ __forceinline__ Divisor divisor(float s) {
  Divisor d;
  d.tiny = s < 0x1p-100f;
  d.up = d.tiny ? 0x1p64f : 1.0f;
  d.scale = s * d.up;
  d.inverse = s > 0.0f ? 1.0f / d.scale : 0.0f;
  return d;
}

// Sixteen codes, a byte each. x + 1.5 2^23 rounds x to the nearest integer, ties
// to even, and holds it in its low bits in two's complement.
__device__ __forceinline__ uint4 code_piece(float (&x)[kPiece], const Divisor& d) {
  constexpr float kMagic = 0x1.8p23f;
  const float half = 0.5f * d.scale;
  float off = 0.0f, t[kPiece];
  if (d.tiny) {  // uniform over the row
#pragma unroll
    for (int i = 0; i < kPiece; ++i) x[i] = fminf(fmaxf(x[i] * d.up, -127.0f * d.scale), 127.0f * d.scale);
  }
#pragma unroll
  for (int i = 0; i < kPiece; ++i) {
    t[i] = fmaf(x[i], d.inverse, kMagic);
    off = fmaxf(off, fabsf(fmaf(kMagic - t[i], d.scale, x[i])));
  }
  if (off >= half && half > 0.0f) {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const float rest = fmaf(kMagic - t[i], d.scale, x[i]);
      const bool over = fabsf(rest) > half || (fabsf(rest) == half && (__float_as_uint(t[i]) & 1u));
      if (over) t[i] += rest > 0.0f ? 1.0f : -1.0f;
    }
  }
  uint32_t w[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 1]), __float_as_uint(t[4 * h]), 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 3]), __float_as_uint(t[4 * h + 2]), 0x04000C0Cu);
    w[h] = lo | hi;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// fp32(1 / sqrt(v)), v > 0: the hardware's estimate y of 2^-23, and the third-order
// step y (1 + e / 2 + 3 e^2 / 8), e = 1 - v y^2, after which a few roundings of
// 2^-53 are left (with a division and a square root of float64 the normed 2048 x
// 4096 take 10.7 us, 10.1 so). Not finite where v is not.
__device__ __forceinline__ float inverse_root(double v) {
  const double y = __builtin_amdgcn_rsq(v), e = fma(-(v * y), y, 1.0);
  return (float)fma(y, e * fma(0.375, e, 0.5), y);
}

struct QuantArgs {
  const void* x;
  int64_t ldx;
  const uint16_t* gamma;  // norm: bf16 [K] or null
  float eps;
  double inverse_k;
  float* r_out;  // norm: fp32 [rows] or null
  uint32_t K, rows;
  uint32_t per;  // rows of a tensor (a stack holds rows / per of them)
  int8_t* codes;
  float* scales;
  const int32_t* seg;  // or null: rows outside [seg[0], seg[E]) are left as they are
  int32_t E;
};

// A workgroup has a row, a lane the pieces tid, tid + threads, ..., of which the
// first kHold stay in registers between the passes over the row (a sum for the
// norm, the maximum, the codes); later ones are read again. Many rows: bound by
// memory (16384 x 4096 39-45 us by card, 5.2-4.4 TB/s, the rate of a copy; of fp32 70 us,
// 4.8 TB/s; weights 128 x 1536 x 2048 209 us, 5.8 TB/s), with the norm by its instructions
// too (48-53 us). 2048 x 4096 8.1-8.6 us and 10.1-10.5, 4.9 at that rate: all rows are in
// flight at once and wait together. Few: by one row's round trips (8 x 8192 3.6 and 4.5).
// Rows that are not wide are read entry by entry: 16384 x 4097 145 us, of fp32 138, normed
// 269.
template <class In, bool kNorm, bool kWide, int kHold>
__global__ __launch_bounds__(1024) void quantize_int8_kernel(QuantArgs a) {
  __shared__ double s_sum[16];
  __shared__ uint32_t s_max[16];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  // Neighbouring rows go to one XCD: a 128-byte line holds a stage of two rows.
  const uint32_t t = blockIdx.y * gridDim.x + (uint32_t)xcd_item((int)blockIdx.x, (int)gridDim.x);
  if (t >= a.rows) return;  // uniform, like every branch to a barrier below
  if (a.seg) {
    const int64_t lo = a.seg[0], hi = a.seg[a.E];
    if ((int64_t)t < lo || (int64_t)t >= hi) return;
  }
  const In* row = static_cast<const In*>(a.x) + (int64_t)t * a.ldx;
  const uint32_t pieces = (a.K + kPiece - 1) / kPiece, stages = (a.K + 63) / 64, padded = 4 * stages;
  Piece<In> held[kHold];
  Piece<uint16_t> gam[kNorm ? kHold : 1];
#pragma unroll
  for (int q = 0; q < kHold; ++q) {
    const uint32_t p = tid + q * blockDim.x;
    held[q] = load_piece<In, kWide>(row, p, a.K);
    if constexpr (kNorm)
      if (a.gamma) gam[q] = load_piece<uint16_t, kWide>(a.gamma, p, a.K);
  }

  float r = 0.0f;
  if constexpr (kNorm) {
    // Sums of squares in float64 (each square exact), in an order set by the sizes alone.
    double sum = 0.0;
    auto add = [&](const Piece<In>& p) {
      float v[kPiece];
      widen(p, v);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) sum = fma((double)v[i], (double)v[i], sum);
    };
#pragma unroll
    for (int q = 0; q < kHold; ++q) add(held[q]);
    for (uint32_t p = tid + kHold * blockDim.x; p < pieces; p += blockDim.x) add(load_piece<In, kWide>(row, p, a.K));
    sum = wave_sum(sum);
    if (waves > 1) {
      if (lane == 0) s_sum[wave] = sum;
      __syncthreads();
      sum = 0.0;
      for (uint32_t i = 0; i < waves; ++i) sum += s_sum[i];
    }
    r = inverse_root(fma(sum, a.inverse_k, (double)a.eps));
    if (a.r_out && tid == 0) a.r_out[t] = r;
  }
  auto norm = [&](const Piece<In>& p, const Piece<uint16_t>& gamma, float (&v)[kPiece]) {
    widen(p, v);
    if constexpr (kNorm) {
#pragma unroll
      for (int i = 0; i < kPiece; i += 2) {
        const uint32_t b = bf16x2_rne(v[i] * r, v[i + 1] * r);
        v[i] = bf16_lo(b);
        v[i + 1] = bf16_hi(b);
      }
      if (a.gamma) {
        float g[kPiece];
        widen(gamma, g);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) v[i] *= g[i];
      }
    }
  };
  auto later = [&](uint32_t p, float (&v)[kPiece]) {
    Piece<uint16_t> g;
    if constexpr (kNorm)
      if (a.gamma) g = load_piece<uint16_t, kWide>(a.gamma, p, a.K);
    norm(load_piece<In, kWide>(row, p, a.K), g, v);
  };
  auto largest = [&](uint32_t m, const float (&v)[kPiece]) {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
  };

  // A normed row's held entries stay as their fp32 values, a plain row's as they were loaded.
  float value[kNorm ? kHold : 1][kPiece];
  uint32_t m = 0;
  if constexpr (kNorm) {
#pragma unroll
    for (int q = 0; q < kHold; ++q) {
      norm(held[q], gam[q], value[q]);
      m = largest(m, value[q]);
    }
    for (uint32_t p = tid + kHold * blockDim.x; p < pieces; p += blockDim.x) {
      float v[kPiece];
      later(p, v);
      m = largest(m, v);
    }
  } else {
#pragma unroll
    for (int q = 0; q < kHold; ++q) m = join_amax<In>(m, held[q]);
    for (uint32_t p = tid + kHold * blockDim.x; p < pieces; p += blockDim.x)
      m = join_amax<In>(m, load_piece<In, kWide>(row, p, a.K));
    m = amax_f32<In>(m);
  }
  m = wave_max(m);
  if (waves > 1) {
    if (lane == 0) s_max[wave] = m;
    __syncthreads();
    for (uint32_t i = 0; i < waves; ++i) m = max(m, s_max[i]);
  }
  const bool finite = m < 0x7F800000u;
  const float s = finite ? __uint_as_float(m) / 127.0f : __uint_as_float(0x7FC00000u);
  const Divisor d = divisor(finite ? s : 0.0f);
  if (tid == 0) a.scales[t] = s;

  const uint32_t tensor = t / a.per, at = t - tensor * a.per;
  const int64_t stage = (int64_t)a.per * 64;
  int8_t* out = a.codes + (int64_t)tensor * stages * stage + (int64_t)at * 64 + (tid >> 2) * stage + 16 * (tid & 3);
  const int64_t step = (blockDim.x >> 2) * stage;
#pragma unroll
  for (int q = 0; q < kHold; ++q) {
    if (tid + q * blockDim.x < padded) {
      uint4 c = make_uint4(0, 0, 0, 0);
      if (finite) {
        float v[kPiece];
        if constexpr (!kNorm) widen(held[q], v);
        c = code_piece(kNorm ? value[kNorm ? q : 0] : v, d);
      }
      *reinterpret_cast<uint4*>(out + q * step) = c;
    }
  }
  out += kHold * step;
  for (uint32_t p = tid + kHold * blockDim.x; p < padded; p += blockDim.x, out += step) {
    float v[kPiece];
    later(p, v);
    *reinterpret_cast<uint4*>(out) = finite ? code_piece(v, d) : make_uint4(0, 0, 0, 0);
  }
}

// Row-major codes [rows][K] to stages and back, a 16-byte piece of a stage a lane; kWide: rows are 16-byte aligned. Bound
// by memory then (14336 x 4096 24 us packed, 23 unpacked: 4.9-5.2 TB/s); others go byte by byte (14336 x 4100 98 and 140
// us: a weight is packed once).
template <bool kWide>
__global__ __launch_bounds__(256) void pack_int8_kernel(const int8_t* __restrict__ rm, uint32_t per, uint32_t K,
                                                        int64_t chunks, int8_t* __restrict__ sm) {
  const int64_t c = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  if (c >= chunks) return;
  const uint32_t stages = (K + 63) / 64;
  const int64_t row = c >> 2, tensor = row / ((int64_t)stages * per), in = row - tensor * stages * per;
  const uint32_t g = (uint32_t)(in / per), r = (uint32_t)(in - (int64_t)g * per), k = 64 * g + 16 * (uint32_t)(c & 3);
  const int8_t* src = rm + (tensor * per + r) * (int64_t)K;
  union {
    uint4 v;
    int8_t b[16];
  } u;
  u.v = make_uint4(0, 0, 0, 0);
  if (kWide && k + 16 <= K) {
    u.v = *reinterpret_cast<const uint4*>(src + k);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (k + e < K) u.b[e] = src[k + e];
  }
  reinterpret_cast<uint4*>(sm)[c] = u.v;
}

template <bool kWide>
__global__ __launch_bounds__(256) void unpack_int8_kernel(const int8_t* __restrict__ sm, uint32_t per, uint32_t K,
                                                          int64_t chunks, int8_t* __restrict__ rm) {
  const int64_t c = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  if (c >= chunks) return;
  const uint32_t stages = (K + 63) / 64;
  const int64_t row = c >> 2, tensor = row / ((int64_t)stages * per), in = row - tensor * stages * per;
  const uint32_t g = (uint32_t)(in / per), r = (uint32_t)(in - (int64_t)g * per), k = 64 * g + 16 * (uint32_t)(c & 3);
  int8_t* dst = rm + (tensor * per + r) * (int64_t)K;
  union {
    uint4 v;
    int8_t b[16];
  } u;
  u.v = reinterpret_cast<const uint4*>(sm)[c];
  if (kWide && k + 16 <= K) {
    *reinterpret_cast<uint4*>(dst + k) = u.v;
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (k + e < K) dst[k + e] = u.b[e];
  }
}

// At most 2^20 workgroups along x (fewer than 2^32 threads at 1024 each).
dim3 rows_grid(int64_t n) {
  const int64_t x = n < (1 << 20) ? n : 1 << 20;
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

template <class In, bool kNorm>
hipError_t launch_rows(const QuantArgs& a, hipStream_t stream) {
  const int64_t pieces = (a.K + kPiece - 1) / kPiece;
  // A piece a lane, which has most in flight: 2048 x 4096 8.1 us, 9.9 with two pieces
  // a lane in half the waves, 11.6 with four. Many long rows: two (2048 x 14336 20.7
  // us, 21.8 with one; normed 28.1 and 31.0).
  const int64_t each = a.rows >= 1024 && pieces > 512 ? 2 : 1;
  int64_t waves = (pieces + 64 * each - 1) / (64 * each);
  waves = waves <= 1 ? 1 : waves <= 2 ? 2 : waves <= 4 ? 4 : waves <= 8 ? 8 : 16;
  const int64_t hold = (pieces + 64 * waves - 1) / (64 * waves);
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.gamma);
  const bool wide = (at & 15) == 0 && a.K % 8 == 0 && a.ldx * (int64_t)sizeof(In) % 16 == 0;
  const dim3 grid = rows_grid(a.rows), block((unsigned)(64 * waves));
#define SHARQ_QUANT_INT8(W, H) \
  hipLaunchKernelGGL((quantize_int8_kernel<In, kNorm, W, H>), grid, block, 0, stream, a)
  if (!wide) SHARQ_QUANT_INT8(false, 2);
  else if (hold <= 1) SHARQ_QUANT_INT8(true, 1);
  else if (hold <= 2) SHARQ_QUANT_INT8(true, 2);
  else SHARQ_QUANT_INT8(true, 4);
#undef SHARQ_QUANT_INT8
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_int8(const void* x, int dtype, int64_t E, int64_t R, int64_t K, int64_t ldx, int8_t* codes,
                                float* scales, const int32_t* seg, int32_t segments, hipStream_t stream) {
  const QuantArgs a{x, ldx, nullptr, 0.0f, 0.0, nullptr, (uint32_t)K, (uint32_t)(E * R), (uint32_t)R, codes, scales,
                    seg, segments};
  if (dtype == 0) return launch_rows<float, false>(a, stream);
  if (dtype == 1) return launch_rows<uint16_t, false>(a, stream);
  return launch_rows<_Float16, false>(a, stream);
}

hipError_t launch_quantize_int8_rms(const uint16_t* x, int64_t T, int64_t K, int64_t ldx, const uint16_t* gamma,
                                    float eps, float* rms_scale, int8_t* codes, float* scales, hipStream_t stream) {
  const QuantArgs a{x, ldx, gamma, eps, 1.0 / (double)K, rms_scale, (uint32_t)K, (uint32_t)T, (uint32_t)T, codes, scales, nullptr, 0};
  return launch_rows<uint16_t, true>(a, stream);
}

hipError_t launch_pack_int8(const int8_t* codes_rm, int64_t E, int64_t R, int64_t K, int8_t* codes, bool unpack,
                            int8_t* out_rm, hipStream_t stream) {
  const int64_t chunks = E * R * ((K + 63) / 64) * 4;
  const dim3 grid = rows_grid((chunks + 255) / 256);
  const void* rm = unpack ? static_cast<const void*>(out_rm) : static_cast<const void*>(codes_rm);
  const bool wide = (reinterpret_cast<uintptr_t>(rm) & 15) == 0 && K % 16 == 0;
#define SHARQ_PACK_INT8(KERNEL, W, FROM, TO) \
  hipLaunchKernelGGL((KERNEL<W>), grid, dim3(256), 0, stream, FROM, (uint32_t)R, (uint32_t)K, chunks, TO)
  if (unpack) {
    if (wide) SHARQ_PACK_INT8(unpack_int8_kernel, true, codes, out_rm);
    else SHARQ_PACK_INT8(unpack_int8_kernel, false, codes, out_rm);
  } else {
    if (wide) SHARQ_PACK_INT8(pack_int8_kernel, true, codes_rm, codes);
    else SHARQ_PACK_INT8(pack_int8_kernel, false, codes_rm, codes);
  }
#undef SHARQ_PACK_INT8
  return hipGetLastError();
}

}  // namespace sharq

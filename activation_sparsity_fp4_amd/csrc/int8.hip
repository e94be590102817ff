// 8-bit integer coding with one scale a row (activations: a token, weights: an
// output channel), and the layout of the codes.
//
//   amax = max_k |x'[k]|,  s = fp32(amax / 127),  q[k] = clamp(rne(x'[k] / s), -127, 127)
//
// with x' = x, or the RMS-normed row bf16(x r) gamma. The quotient is the exact
// one, not its fp32 rounding: v = x' (1 / s) is at most 127 (2^-23 + 2^-47) <
// 2^-16 from it, so wherever v stays 2^-15 off the middle of two codes its
// nearest integer is the code; a thread that holds a closer one settles its
// entries by the sign of |x' - q s| - s / 2, where x' - q s is one fma, exact
// that near the middle (a multiple of the last bit of s below s). Rows of zeros
// have scale 0; a row that holds a NaN or an infinity has scale NaN and codes
// of zero, so that products with it are NaN.
//
// Layout: codes i8 [G][rows][64], G = ceil(K / 64), zeros past K: a stage of 64
// entries a row is the 64-byte row that the GEMM's LDS stage holds.

#include "gemm_common.h"
#include "sharq_device.h"
#include "sharq_internal.h"

namespace sharq {
namespace {

constexpr int kPiece = 8;  // entries of a lane's load

// The entries of a piece as they were loaded: 16 bytes of a 2-byte type, 32 of fp32.
template <class In>
struct Piece {
  uint32_t w[sizeof(In) * kPiece / 4];
};

__device__ __forceinline__ void widen(const Piece<uint16_t>& p, float (&v)[kPiece]) {  // bf16
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(p.w[i]), v[2 * i + 1] = bf16_hi(p.w[i]);
}
__device__ __forceinline__ void widen(const Piece<_Float16>& p, float (&v)[kPiece]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)p.w[i]);
    v[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(p.w[i] >> 16));
  }
}
__device__ __forceinline__ void widen(const Piece<float>& p, float (&v)[kPiece]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(p.w[i]);
}

// Entries [8 p, 8 p + 8) of a row of K; those past K are zeros. kWide: K is a
// multiple of 8 and the row 16-byte aligned.
template <class In, bool kWide>
__device__ __forceinline__ Piece<In> load_piece(const In* __restrict__ row, uint32_t p, uint32_t K) {
  Piece<In> out;
  constexpr int kWords = sizeof(Piece<In>) / 4;
#pragma unroll
  for (int i = 0; i < kWords; ++i) out.w[i] = 0;
  if constexpr (kWide) {
    if (kPiece * p < K) {
      const uint4* src = reinterpret_cast<const uint4*>(row + (uint64_t)kPiece * p);
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = src[i];
        out.w[4 * i] = v.x, out.w[4 * i + 1] = v.y, out.w[4 * i + 2] = v.z, out.w[4 * i + 3] = v.w;
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

// x' of a normed piece from its bf16 entries (x r, rounded) and gamma (exact in fp32).
__device__ __forceinline__ void times_gamma(float (&v)[kPiece], const Piece<uint16_t>& gamma) {
  float g[kPiece];
  widen(gamma, g);
#pragma unroll
  for (int i = 0; i < kPiece; ++i) v[i] *= g[i];
}

// How a row is divided: x' up (1 / (s up)), up a power of two that keeps the
// reciprocal of a small scale finite.
struct Divisor {
  float up, scale, inverse;  // scale: s up
  bool tiny;                 // s has lost bits of amax / 127, so codes may pass 127
};

__device__ __forceinline__ Divisor divisor(float s) {
  Divisor d;
  d.tiny = s < 0x1p-100f;
  d.up = d.tiny ? 0x1p64f : 1.0f;
  d.scale = s * d.up;
  d.inverse = s > 0.0f ? 1.0f / d.scale : 0.0f;
  return d;
}

// Eight codes, a byte each. x + 1.5 2^23 rounds x to the nearest integer, ties
// to even, and holds it in its low bits in two's complement.
__device__ __forceinline__ uint2 code_piece(float (&x)[kPiece], const Divisor& d) {
  constexpr float kMagic = 0x1.8p23f;
  float off = 0.0f, t[kPiece];
  if (d.tiny) {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) x[i] = fminf(fmaxf(x[i] * d.up, -127.0f * d.scale), 127.0f * d.scale);
  }
#pragma unroll
  for (int i = 0; i < kPiece; ++i) {
    const float v = x[i] * d.inverse;
    t[i] = v + kMagic;
    off = fmaxf(off, fabsf(v - (t[i] - kMagic)));
  }
  if (off > 0.5f - 0x1p-15f) {
    const float half = 0.5f * d.scale;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const float q = t[i] - kMagic, rest = fmaf(-q, d.scale, x[i]);
      const bool over = fabsf(rest) > half || (fabsf(rest) == half && (__float_as_uint(t[i]) & 1u));
      if (over && d.inverse > 0.0f) t[i] += rest > 0.0f ? 1.0f : -1.0f;
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 1]), __float_as_uint(t[4 * h]), 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 3]), __float_as_uint(t[4 * h + 2]), 0x04000C0Cu);
    w[h] = lo | hi;
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t amax_bits(const float (&v)[kPiece]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPiece; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

struct QuantArgs {
  const void* x;
  int64_t ldx;
  const uint16_t* gamma;  // norm: bf16 [K] or null
  float eps;
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
// norm, the maximum, the codes); later ones are read again. Bound by memory at
// many rows (3 bytes an entry), by the round trips of one row at few.
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
  const uint32_t pieces = (a.K + kPiece - 1) / kPiece, stages = (a.K + 63) / 64, padded = 8 * stages;
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
    // Squares of bf16 are exact in fp32; their sum is float64, in an order set by K alone.
    double sum = 0.0;
    auto add = [&](const Piece<In>& p) {
      float v[kPiece];
      widen(p, v);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) sum += (double)(v[i] * v[i]);
    };
#pragma unroll
    for (int q = 0; q < kHold; ++q) add(held[q]);
    for (uint32_t p = tid + kHold * blockDim.x; p < pieces; p += blockDim.x) add(load_piece<In, kWide>(row, p, a.K));
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
    if (waves > 1) {
      if (lane == 0) s_sum[wave] = sum;
      __syncthreads();
      sum = 0.0;
      for (uint32_t i = 0; i < waves; ++i) sum += s_sum[i];
    }
    r = (float)(1.0 / sqrt(sum / (double)a.K + (double)a.eps));
    if (a.r_out && tid == 0) a.r_out[t] = r;
  }
  auto values = [&](const Piece<In>& p, const Piece<uint16_t>& g, float (&v)[kPiece]) {
    widen(p, v);
    if constexpr (kNorm) {
#pragma unroll
      for (int i = 0; i < kPiece; i += 2) {
        const uint32_t b = bf16x2_rne(v[i] * r, v[i + 1] * r);
        v[i] = bf16_lo(b);
        v[i + 1] = bf16_hi(b);
      }
      if (a.gamma) times_gamma(v, g);
    }
  };
  auto later = [&](uint32_t p, float (&v)[kPiece]) {
    Piece<uint16_t> g;
    if constexpr (kNorm)
      if (a.gamma) g = load_piece<uint16_t, kWide>(a.gamma, p, a.K);
    values(load_piece<In, kWide>(row, p, a.K), g, v);
  };

  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < kHold; ++q) {
    float v[kPiece];
    values(held[q], gam[kNorm ? q : 0], v);
    m = max(m, amax_bits(v));
  }
  for (uint32_t p = tid + kHold * blockDim.x; p < pieces; p += blockDim.x) {
    float v[kPiece];
    later(p, v);
    m = max(m, amax_bits(v));
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
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
  int8_t* out = a.codes + ((int64_t)tensor * stages * a.per + at) * 64;
  auto emit = [&](uint32_t p, float (&v)[kPiece]) {
    const uint2 c = finite ? code_piece(v, d) : make_uint2(0, 0);
    *reinterpret_cast<uint2*>(out + (int64_t)(p >> 3) * a.per * 64 + 8 * (p & 7)) = c;
  };
#pragma unroll
  for (int q = 0; q < kHold; ++q) {
    const uint32_t p = tid + q * blockDim.x;
    if (p < padded) {
      float v[kPiece];
      values(held[q], gam[kNorm ? q : 0], v);
      emit(p, v);
    }
  }
  for (uint32_t p = tid + kHold * blockDim.x; p < padded; p += blockDim.x) {
    float v[kPiece];
    later(p, v);
    emit(p, v);
  }
}

// Row-major codes [rows][K] to stages and back, a 16-byte piece of a stage a lane; kWide: rows are 16-byte aligned.
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
  // Many rows: few waves a row, whose lanes hold four pieces (with gamma's) or
  // eight. Few: two a lane, for the row's own latency counts.
  constexpr int kMost = kNorm ? 4 : 8;
  const int64_t each = a.rows >= 1024 ? kMost : 2;
  int64_t waves = (pieces + 64 * each - 1) / (64 * each);
  waves = waves <= 1 ? 1 : waves <= 2 ? 2 : waves <= 4 ? 4 : waves <= 8 ? 8 : 16;
  const bool hold2 = pieces <= 128 * waves;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.gamma);
  const bool wide = (at & 15) == 0 && a.K % kPiece == 0 && a.ldx * (int64_t)sizeof(In) % 16 == 0;
  const dim3 grid = rows_grid(a.rows), block((unsigned)(64 * waves));
#define SHARQ_QUANT_INT8(W, H) \
  hipLaunchKernelGGL((quantize_int8_kernel<In, kNorm, W, H>), grid, block, 0, stream, a)
  if (wide) {
    if (hold2) SHARQ_QUANT_INT8(true, 2); else SHARQ_QUANT_INT8(true, kMost);
  } else {
    if (hold2) SHARQ_QUANT_INT8(false, 2); else SHARQ_QUANT_INT8(false, kMost);
  }
#undef SHARQ_QUANT_INT8
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_int8(const void* x, int dtype, int64_t E, int64_t R, int64_t K, int64_t ldx, int8_t* codes,
                                float* scales, const int32_t* seg, int32_t segments, hipStream_t stream) {
  const QuantArgs a{x, ldx, nullptr, 0.0f, nullptr, (uint32_t)K, (uint32_t)(E * R), (uint32_t)R, codes, scales,
                    seg, segments};
  if (dtype == 0) return launch_rows<float, false>(a, stream);
  if (dtype == 1) return launch_rows<uint16_t, false>(a, stream);
  return launch_rows<_Float16, false>(a, stream);
}

hipError_t launch_quantize_int8_rms(const uint16_t* x, int64_t T, int64_t K, int64_t ldx, const uint16_t* gamma,
                                    float eps, float* rms_scale, int8_t* codes, float* scales, hipStream_t stream) {
  const QuantArgs a{x, ldx, gamma, eps, rms_scale, (uint32_t)K, (uint32_t)T, (uint32_t)T, codes, scales, nullptr, 0};
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

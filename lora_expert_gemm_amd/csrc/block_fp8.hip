// Quantisation to OCP E4M3 with one scale per block of 128 along the
// contraction (rows) or per block of 128 x 128 (weights).
//
// The scale of a block is a power of two, the smallest 2^e with
// max|v| / 448 <= 2^e (448: the format's largest value; e >= -126), taken
// from the bits of max|v|.  v / 2^e is then exact in float32, so a code is
// one rounding of the input itself (nearest, ties to even) and no value sits
// on a border that depends on how a division was rounded; the price is up to
// one bit of the block's head room, which a floating-point code does not
// feel.  Elements that are not finite get the NaN code and do not count in
// max|v|.  Bound by HBM: a lane converts eight consecutive elements from
// registers, a code and 1/32 byte of scale are written per element.  25600
// gathered rows of 2880 bf16 (6400 tokens, each read four times, mostly from
// cache) take 31 us; 8 x 11008 x 4096 bf16 weights with their transposed copy
// 277 us (1.44 GB, 5.2 TB/s).
#include "common.h"
#include "kernels.h"
#include "ops.h"

namespace moelora {

namespace {

constexpr int kThreads = 256;
constexpr int kBlk = 128;    // elements a scale
constexpr int kLanes = 16;   // lanes on a block, 8 elements each
constexpr int kGroups = kThreads / kLanes;

// Eight elements of a row of K from element c on, zeros past K, as they are
// stored (bf16: two a dword).  Whole ones are 16-byte loads, which need no
// more than 2-byte alignment here.
template <typename DT> struct Raw8;
template <> struct Raw8<uint16_t> {
  u32x4_t v;
};
template <> struct Raw8<float> {
  u32x4_t v[2];
};
template <typename DT>
__device__ __forceinline__ Raw8<DT> load8(const DT *row, int c, int K) {
  typedef u32x4_t mem __attribute__((aligned(2)));
  const mem *p = reinterpret_cast<const mem *>(row + c);
  if (c + 8 <= K) {
    if constexpr (sizeof(DT) == 2) return {*p};
    else return {{p[0], p[1]}};
  }
  struct Eight {
    DT e[8];
  } f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f.e[i] = c + i < K ? row[c + i] : DT(0);
  return __builtin_bit_cast(Raw8<DT>, f);
}

__device__ __forceinline__ void to_f32(const Raw8<uint16_t> &r, float *f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(r.v[i] << 16);
    f[2 * i + 1] = __uint_as_float(r.v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void to_f32(const Raw8<float> &r, float *f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.v[i / 4][i % 4]);
}

// Largest magnitude of the eight as the bits of a non-negative float; not
// finite if any of them is not.  bf16: both halves of a dword at once.
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t amax_bits8(const Raw8<uint16_t> &r) {
  u16x2_t m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, r.v[i] & 0x7fff7fffu));
  return (uint32_t)max(m[0], m[1]) << 16;
}
__device__ __forceinline__ uint32_t amax_bits8(const Raw8<float> &r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, r.v[i / 4][i % 4] & 0x7fffffffu);
  return m;
}
constexpr uint32_t kInfBits = 0x7f800000u;
__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7fffffffu) < kInfBits; }
// ... of the finite ones only.
template <typename DT>
__device__ __forceinline__ uint32_t amax_finite8(const Raw8<DT> &r) {
  float f[8];
  to_f32(r, f);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, finite(f[i]) ? __float_as_uint(f[i]) & 0x7fffffffu : 0u);
  return m;
}

// e of the block's scale 2^e: amax = (1 + m) 2^q gives amax / 448 <= 2^(q - 8)
// exactly when 1 + m <= 1.75.
__device__ __forceinline__ int scale_exp(uint32_t amax) {
  const int q = (int)(amax >> 23) - 127;
  return max(-126, q - 8 + ((amax & 0x7fffffu) > 0x600000u));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Codes of the eight times inv.  `odd`: some element of the block is not
// finite (its code is set by hand).
template <typename DT>
__device__ __forceinline__ uint2 codes8(const Raw8<DT> &r, float inv, bool odd) {
  float f[8];
  to_f32(r, f);
  uint32_t u[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h] * inv, f[4 * h + 1] * inv, 0, false);
    u[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2] * inv, f[4 * h + 3] * inv, w, true);
  }
  if (odd) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!finite(f[i])) u[i / 4] = (u[i / 4] & ~(0xffu << 8 * (i % 4))) | (0x7fu << 8 * (i % 4));
  }
  return make_uint2(u[0], u[1]);
}

// 16 rows a workgroup, up to kBlocks blocks of each: 16 lanes a (row, block).
// The blocks' loads are all issued before the first is used; the rows'
// scales of one block are neighbours in memory.
constexpr int kBlocks = 4;
template <typename DT>
__global__ __launch_bounds__(kThreads) void k_quant_rows(QuantRowsArgs a, int KB) {
  const int g = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
  const int r = blockIdx.x * kGroups + g;
  if (r >= a.M) return;
  int src = r;
  if (a.rows) {
    const int p = a.rows[r];
    src = p < 0 ? -1 : p / a.div;
    if ((unsigned)src >= (unsigned)a.n_src) return;  // whole group: its row is left as it was
  }
  const DT *row = static_cast<const DT *>(a.x) + (size_t)src * a.K;
  uint8_t *out = a.codes + (size_t)r * KB * kBlk;
  const int b0 = blockIdx.y * kBlocks;
  Raw8<DT> v[kBlocks];
#pragma unroll
  for (int u = 0; u < kBlocks; ++u)
    if (b0 + u < KB) v[u] = load8<DT>(row, (b0 + u) * kBlk + l * 8, a.K);
#pragma unroll
  for (int u = 0; u < kBlocks; ++u) {
    if (b0 + u >= KB) break;
    uint32_t m = amax_bits8(v[u]);
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    const bool odd = m >= kInfBits;  // the same for the block's 16 lanes
    if (odd) {
      m = amax_finite8(v[u]);
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    }
    const int e = scale_exp(m);
    const uint2 c = codes8(v[u], pow2(-e), odd);
    __builtin_nontemporal_store(
        __builtin_bit_cast(unsigned long long, c),
        reinterpret_cast<unsigned long long *>(out + (size_t)(b0 + u) * kBlk + l * 8));
    if (l == 0) a.scales[(size_t)(b0 + u) * a.M + r] = pow2(e);
  }
}

// One 128 x 128 block a workgroup, held in registers between the maximum and
// the conversion; the transposed copy goes through LDS, four rows x four
// codes at a time.
constexpr int kPitch = kBlk + 4;  // LDS bytes per row of codes
template <typename DT>
__global__ __launch_bounds__(kThreads) void k_quant_weights(QuantWeightsArgs a, int NB, int KB) {
  __shared__ uint32_t wmax[kThreads / kWave];
  __shared__ __align__(16) uint8_t tile[kBlk * kPitch];
  const int tid = threadIdx.x, g = tid / kLanes, l = tid % kLanes;
  const int kb = blockIdx.x, nb = blockIdx.y, mat = blockIdx.z;
  const size_t P = (size_t)KB * kBlk, Pt = (size_t)NB * kBlk;
  const DT *w = static_cast<const DT *>(a.w) + (size_t)mat * a.N * a.K;
  const int n0 = nb * kBlk, k0 = kb * kBlk;
  constexpr int kPass = kBlk / kGroups;
  Raw8<DT> v[kPass];
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    const int n = n0 + i * kGroups + g;
    v[i] = load8<DT>(w + (size_t)min(n, a.N - 1) * a.K, k0 + l * 8, n < a.N ? a.K : 0);
  }
  auto block_max = [&](uint32_t m) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    if (tid % kWave == 0) wmax[tid / kWave] = m;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kThreads / kWave; ++q) m = max(m, wmax[q]);
    return m;
  };
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPass; ++i) m = max(m, amax_bits8(v[i]));
  m = block_max(m);
  const bool odd = m >= kInfBits;  // the same for the whole workgroup
  if (odd) {
    __syncthreads();
    m = 0;
#pragma unroll
    for (int i = 0; i < kPass; ++i) m = max(m, amax_finite8(v[i]));
    m = block_max(m);
  }
  const int e = scale_exp(m);
  const float inv = pow2(-e);
  if (tid == 0) {
    a.scales[((size_t)mat * NB + nb) * KB + kb] = pow2(e);
    if (a.scales_t) a.scales_t[((size_t)mat * KB + kb) * NB + nb] = pow2(e);
  }
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    const int nl = i * kGroups + g, n = n0 + nl;
    const uint2 c = codes8(v[i], inv, odd);
    if (n < a.N) *reinterpret_cast<uint2 *>(a.codes + ((size_t)mat * a.N + n) * P + k0 + l * 8) = c;
    if (a.codes_t) {
      uint32_t *t = reinterpret_cast<uint32_t *>(tile + nl * kPitch + l * 8);
      t[0] = c.x, t[1] = c.y;
    }
  }
  if (!a.codes_t) return;
  __syncthreads();
  // 32 lanes write one 128-byte line of a transposed row, 4 rows at a time
  const int n4 = tid % 32;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k4 = i * 8 + tid / 32;
    uint32_t r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      r[q] = *reinterpret_cast<const uint32_t *>(tile + (n4 * 4 + q) * kPitch + k4 * 4);
    // bytes q of r[0..3] side by side
    const uint32_t a01 = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u);  // r0.0 r1.0 r0.1 r1.1
    const uint32_t a23 = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u);
    const uint32_t b01 = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);  // r0.2 r1.2 r0.3 r1.3
    const uint32_t b23 = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
    const uint32_t o[4] = {
        __builtin_amdgcn_perm(a23, a01, 0x05040100u), __builtin_amdgcn_perm(a23, a01, 0x07060302u),
        __builtin_amdgcn_perm(b23, b01, 0x05040100u), __builtin_amdgcn_perm(b23, b01, 0x07060302u)};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = k0 + k4 * 4 + q;
      if (k < a.K)
        *reinterpret_cast<uint32_t *>(a.codes_t + ((size_t)mat * a.K + k) * Pt + n0 + n4 * 4) = o[q];
    }
  }
}

template <typename DT>
hipError_t rows_t(const QuantRowsArgs &a, hipStream_t st) {
  const int KB = (a.K + kBlk - 1) / kBlk;
  const int groups = (a.M + kGroups - 1) / kGroups;
  return launch_kernel(k_quant_rows<DT>, dim3(groups, (KB + kBlocks - 1) / kBlocks), dim3(kThreads), 0, st,
                       a, KB);
}

template <typename DT>
hipError_t weights_t(const QuantWeightsArgs &a, hipStream_t st) {
  const int KB = (a.K + kBlk - 1) / kBlk, NB = (a.N + kBlk - 1) / kBlk;
  return launch_kernel(k_quant_weights<DT>, dim3(KB, NB, a.mats), dim3(kThreads), 0, st, a, NB, KB);
}

}  // namespace

hipError_t launch_quantize_rows(const QuantRowsArgs &a, bool bf16, hipStream_t st) {
  return bf16 ? rows_t<uint16_t>(a, st) : rows_t<float>(a, st);
}

hipError_t launch_quantize_weights(const QuantWeightsArgs &a, bool bf16, hipStream_t st) {
  return bf16 ? weights_t<uint16_t>(a, st) : weights_t<float>(a, st);
}

}  // namespace moelora

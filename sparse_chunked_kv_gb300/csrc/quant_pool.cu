// Copies between bf16 rows and the 8-bit chunk pool (codes with one
// power-of-two scale per 16-row block of a slot and KV head).
//
// quantise: for a block with largest magnitude amax = (1 + f) 2^x the scale is
//   the smallest 2^e >= 2^-100 with amax <= M 2^e, M = 448 = 1.75 * 2^8 or
//   127 = 1.984375 * 2^6: e = x - 8 (or x - 6), one more when 1 + f passes
//   M's own 1.75 (1.984375).  Read off amax's bits, no logarithm.  Dividing by
//   2^e is exact, so a code is x rounded once.
// dequantise: value = code * 2^e, exact in bf16 for the scales written above.
//
// Both move 3 bytes per element and compute next to nothing: bound by HBM.
// One warp owns one (block, K or V, head): 16 rows of D values, 8 (or 4)
// 16-byte accesses per lane, all in flight before the first is used, and the
// block's maximum needs only a warp reduction.  Neighbouring warps take
// neighbouring heads, so neighbouring CTAs read the same token rows.  Small CTAs
// and a register bound keep 32 (36) warps on an SM: 1024 slots of 129 rows, 4
// heads of 128, are written in 66 us (6.1 TB/s; 75 us with 8 warps a CTA and 80
// registers), 512 slots of 100 to 129 rows read back in 30 us (6.0 TB/s; 35.6).
#include "pfd_internal.cuh"
#include "sm103_ptx.cuh"

namespace pfd {
namespace {

constexpr int kQuantThreads = kQuantWarps * 32;
constexpr int kMinExp = -100;   // smallest scale 2^-100: E4M3's 2^-9 steps stay normal bf16

// One slot of a call, checked.
struct Slot {
  long long src, dst;
  int len;
  int err;   // PFD_DEVERR_* of a slot that is skipped, else 0
};

// Slot j of a call; a slot's rows on the code side start at a multiple of 16.
template <bool kToCodes>
__device__ __forceinline__ Slot load_slot(const QuantParams& p, int j) {
  Slot s{0, 0, 0, 0};
  int at = j;
  if (!kToCodes && p.sel != nullptr) at = p.sel[j];
  const long long dst = p.dst_stride > 0 ? static_cast<long long>(j) * p.dst_stride : p.dst_row[j];
  if (at < 0 || at >= p.table_len) {
    s.err = PFD_DEVERR_SEL;
    return s;
  }
  const pfd_chunk_entry e = p.src_table[at];
  const long long code_row = kToCodes ? dst : e.row;
  if (e.row < 0 || e.len < 0 || static_cast<long long>(e.row) + e.len > p.src_rows ||
      (!kToCodes && code_row % kGroupRows != 0) || (p.dst_stride > 0 && e.len > p.dst_stride))
    s.err = PFD_DEVERR_TABLE;
  else if (dst < 0 || dst + e.len > p.dst_rows ||
           (kToCodes && code_row % kGroupRows != 0))
    s.err = PFD_DEVERR_SLOT;
  s.src = e.row;
  s.dst = dst;
  s.len = e.len;
  return s;
}

// The slot's destination table entry (an empty one for a skipped slot).
__device__ __forceinline__ void write_entry(const QuantParams& p, int j, const Slot& s) {
  if (s.err != 0) raise_dev_err(p.dev_err, s.err);
  if (p.dst_sel != nullptr) p.dst_sel[j] = j;
  if (p.dst_table == nullptr) return;
  pfd_chunk_entry e;
  e.row = s.err != 0 ? 0 : static_cast<int32_t>(s.dst);
  e.len = s.err != 0 ? 0 : s.len;
  p.dst_table[j] = e;
}

// The four bytes of codes of x[0..3] (already divided by the scale).
template <int kFmt>
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  if constexpr (kFmt == kFmtE4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  } else {
    const uint32_t i0 = static_cast<uint32_t>(__float2int_rn(a)) & 0xFFu;
    const uint32_t i1 = static_cast<uint32_t>(__float2int_rn(b)) & 0xFFu;
    const uint32_t i2 = static_cast<uint32_t>(__float2int_rn(c)) & 0xFFu;
    const uint32_t i3 = static_cast<uint32_t>(__float2int_rn(d)) & 0xFFu;
    return i0 | (i1 << 8) | (i2 << 16) | (i3 << 24);
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <int D, int kFmt>
__global__ void __launch_bounds__(kQuantThreads, 8) pool_quantize_kernel(const QuantParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  constexpr int kLanesPerRow = D / 8;              // 16-byte loads of a head's row
  constexpr int kLoads = 16 * kLanesPerRow / 32;   // per lane
  constexpr int kRowsPerLoad = 32 / kLanesPerRow;
  const int lane = threadIdx.x & 31;
  const int j = static_cast<int>(blockIdx.x) / p.ctas_per_slot;
  const int first = (static_cast<int>(blockIdx.x) % p.ctas_per_slot) * kQuantWarps +
                    static_cast<int>(threadIdx.x >> 5);
  const Slot s = load_slot<true>(p, j);
  if (first == 0 && lane == 0) write_entry(p, j, s);
  if (s.err != 0) return;
  const long long n_units = static_cast<long long>((s.len + kGroupRows - 1) / kGroupRows) * 2 * p.Hkv;
  const int r0 = lane / kLanesPerRow, col = (lane % kLanesPerRow) * 8;
  for (long long u = first; u < n_units; u += static_cast<long long>(p.ctas_per_slot) * kQuantWarps) {
    const int head = static_cast<int>(u % p.Hkv);
    const long long rest = u / p.Hkv;
    const bool is_v = (rest & 1) != 0;
    const int row0 = static_cast<int>(rest >> 1) * kGroupRows;
    const int rows = min(kGroupRows, s.len - row0);
    const bf16* src = (is_v ? p.v : p.k) + ((s.src + row0) * p.Hkv + head) * D + col;
    uint8_t* dst = (is_v ? p.code_v : p.code_k) + ((s.dst + row0) * p.Hkv + head) * D + col;
    const long long stride = static_cast<long long>(p.Hkv) * D;

    uint4 w[kLoads];
    uint32_t top = 0u;   // largest magnitude bits, two halves
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = r0 + i * kRowsPerLoad;
      w[i] = r < rows ? __ldg(reinterpret_cast<const uint4*>(src + r * stride))
                      : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      top = __vmaxu2(top, w[i].x & 0x7FFF7FFFu);
      top = __vmaxu2(top, w[i].y & 0x7FFF7FFFu);
      top = __vmaxu2(top, w[i].z & 0x7FFF7FFFu);
      top = __vmaxu2(top, w[i].w & 0x7FFF7FFFu);
    }
    const uint32_t amax = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
    const bool finite = amax < 0x7F80u;
    const int x = static_cast<int>(amax >> 7) - 127, frac = static_cast<int>(amax & 0x7Fu);
    int e = kFmt == kFmtE4M3 ? x - 8 + (frac > 96 ? 1 : 0) : x - 6 + (frac > 126 ? 1 : 0);
    e = max(e, kMinExp);   // zero and subnormal maxima too
    const float inv = finite ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 0.0f;
    if (lane == 0)
      (is_v ? p.exp_v : p.exp_k)[(s.dst + row0) / kGroupRows * p.Hkv + head] =
          static_cast<uint8_t>(finite ? e + 127 : 255);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = r0 + i * kRowsPerLoad;
      uint2 c = make_uint2(0u, 0u);
      if (finite) {
        c.x = pack_codes<kFmt>(bf16_lo(w[i].x) * inv, bf16_hi(w[i].x) * inv, bf16_lo(w[i].y) * inv,
                               bf16_hi(w[i].y) * inv);
        c.y = pack_codes<kFmt>(bf16_lo(w[i].z) * inv, bf16_hi(w[i].z) * inv, bf16_lo(w[i].w) * inv,
                               bf16_hi(w[i].w) * inv);
      }
      if (r < rows) *reinterpret_cast<uint2*>(dst + r * stride) = c;
    }
  }
}

// Two bf16 of two code bytes (the low 16 bits of c) times 2^e.
template <int kFmt>
__device__ __forceinline__ uint32_t codes2_to_bf16(uint32_t c, float scale) {
  float lo, hi;
  if constexpr (kFmt == kFmtE4M3) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
  } else {
    lo = static_cast<float>(static_cast<int8_t>(c & 0xFFu));
    hi = static_cast<float>(static_cast<int8_t>((c >> 8) & 0xFFu));
  }
  return pack_bf16x2(lo * scale, hi * scale);
}

template <int D, int kFmt>
__global__ void __launch_bounds__(kQuantThreads, 9) pool_dequantize_kernel(const QuantParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  constexpr int kLanesPerRow = D / 16;             // 16-byte loads of a head's code row
  constexpr int kLoads = 16 * kLanesPerRow / 32;   // per lane
  constexpr int kRowsPerLoad = 32 / kLanesPerRow;
  const int lane = threadIdx.x & 31;
  const int j = static_cast<int>(blockIdx.x) / p.ctas_per_slot;
  const int first = (static_cast<int>(blockIdx.x) % p.ctas_per_slot) * kQuantWarps +
                    static_cast<int>(threadIdx.x >> 5);
  const Slot s = load_slot<false>(p, j);
  if (first == 0 && lane == 0) write_entry(p, j, s);
  if (s.err != 0) return;
  const long long n_units = static_cast<long long>((s.len + kGroupRows - 1) / kGroupRows) * 2 * p.Hkv;
  const int r0 = lane / kLanesPerRow, col = (lane % kLanesPerRow) * 16;
  for (long long u = first; u < n_units; u += static_cast<long long>(p.ctas_per_slot) * kQuantWarps) {
    const int head = static_cast<int>(u % p.Hkv);
    const long long rest = u / p.Hkv;
    const bool is_v = (rest & 1) != 0;
    const int row0 = static_cast<int>(rest >> 1) * kGroupRows;
    const int rows = min(kGroupRows, s.len - row0);
    const uint8_t* src = (is_v ? p.code_v : p.code_k) + ((s.src + row0) * p.Hkv + head) * D + col;
    bf16* dst = (is_v ? p.v : p.k) + ((s.dst + row0) * p.Hkv + head) * D + col;
    const long long stride = static_cast<long long>(p.Hkv) * D;
    const uint32_t byte = __ldg((is_v ? p.exp_v : p.exp_k) + (s.src + row0) / kGroupRows * p.Hkv + head);
    uint4 w[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = r0 + i * kRowsPerLoad;
      w[i] = r < rows ? __ldg(reinterpret_cast<const uint4*>(src + r * stride))
                      : make_uint4(0u, 0u, 0u, 0u);
    }
    const float scale = byte == 255u ? __uint_as_float(0x7FC00000u)
                                     : byte == 0u ? __uint_as_float(0x00400000u)
                                                  : __uint_as_float(byte << 23);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = r0 + i * kRowsPerLoad;
      if (r >= rows) continue;
      const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[2 * k] = codes2_to_bf16<kFmt>(in[k] & 0xFFFFu, scale);
        o[2 * k + 1] = codes2_to_bf16<kFmt>(in[k] >> 16, scale);
      }
      uint4* out = reinterpret_cast<uint4*>(dst + r * stride);
      out[0] = make_uint4(o[0], o[1], o[2], o[3]);
      out[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

template <typename Kernel>
cudaError_t launch_rows(Kernel kernel, const QuantParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.ctas_per_slot) * static_cast<unsigned>(p.n_slots));
  return launch_pdl(kernel, grid, dim3(kQuantThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_pool_quantize(const QuantParams& p, int fmt, cudaStream_t stream) {
  if (fmt == kFmtE4M3)
    return p.D == 64 ? launch_rows(pool_quantize_kernel<64, kFmtE4M3>, p, stream)
                     : launch_rows(pool_quantize_kernel<128, kFmtE4M3>, p, stream);
  return p.D == 64 ? launch_rows(pool_quantize_kernel<64, kFmtInt8>, p, stream)
                   : launch_rows(pool_quantize_kernel<128, kFmtInt8>, p, stream);
}

cudaError_t launch_pool_dequantize(const QuantParams& p, int fmt, cudaStream_t stream) {
  if (fmt == kFmtE4M3)
    return p.D == 64 ? launch_rows(pool_dequantize_kernel<64, kFmtE4M3>, p, stream)
                     : launch_rows(pool_dequantize_kernel<128, kFmtE4M3>, p, stream);
  return p.D == 64 ? launch_rows(pool_dequantize_kernel<64, kFmtInt8>, p, stream)
                   : launch_rows(pool_dequantize_kernel<128, kFmtInt8>, p, stream);
}

}  // namespace pfd

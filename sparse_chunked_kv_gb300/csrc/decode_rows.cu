// Decode attention of few live rows over an 8-bit chunk pool (one token, a
// short draft): softmax over [selected slots ; live block] for the at most 32
// packed rows (token t, head j of the KV group, m = t * G + j) of a CTA.
//
// With so few rows a step is bound by reading the pool, and the 128-row
// tensor-memory tiles of the attention kernel are nearly empty: their chain
// (load, convert, QK, softmax, PV) takes the same time for 7 rows as for 128.
// Here each warp works alone on pairs of 16-key groups (a group is a scale block
// of the pool), with no barrier between the warps:
//   - a ring of pairs in shared memory, the warp's own, is filled by TMA; where the groups lie
//     and their exponents are looked up for 32 pairs at once, one pair per
//     lane, and the lane that looked a pair up loads it;
//   - codes become f16 (exact: at most 4, or 8, significant bits) and are the
//     left operands of m16n8k16 products with fp32 sums, 16 keys x 8 rows for
//     the logits, 16 columns of V x 8 rows for the output, so rows come in
//     eights (one token of 7 heads fills 7 of 8) and a code is converted once
//     for all of a warp's rows.  The order of the D dimensions in a product is
//     free as long as both factors agree, so lane c of a quad takes D / 4
//     neighbouring codes of a key, one or two 16-byte loads;
//   - Q is f16 too, each row divided by a power of two that brings its largest
//     element to 2^14..2^15: a bf16 within 2^-29 of that is exact, a smaller one
//     is off by less than 2^-40 of it, below the fp32 sums' own rounding;
//   - a group's K scale multiplies its 16 logits, its V scale the
//     probabilities.  A row keeps two references: m = max x over its logits x
//     (log2 units), for the denominator, and y = max (x + e), e the V exponent,
//     for the output, so probabilities enter the second product as
//     2^(x + e - y + 7), and nothing depends on how the scales of a row's blocks
//     differ.  The references move only when a logit passes one by more than 8
//     (a warp's vote, not a reduction over the keys each time), so f16 holds at
//     most 2^15, and 11 bits of contributions down to 2^-21 of the largest, less
//     of those down to 2^-32;
//   - live rows (bf16) are brought to f16 the same way, a power of two per
//     group of 16.
// The warps' states (m, y, l, O) are joined in shared memory in a fixed order,
// the splits' states by the merge kernel.
// 28 / 4 heads, D = 128: 1 token over 131,136 rows 30.9 us with the merge (4.3 TB/s;
// 55 with 16-row tiles loaded straight to registers, 35.8 with the rings); over 65,568 rows
// 16.6 us, 33.4 by the attention kernel, 4 tokens (28 rows) 30.2 and 33.7.  Which of the
// two takes 17 to 32 rows: few_rows_pays in pfd_api.cu.  (The join of
// 64 rows' outputs would not fit in shared memory.  At D = 128 the 32-row instances are at
// 255 registers and spill 136 to 148 bytes.)
#include "pfd_internal.cuh"
#include "sm103_ptx.cuh"

#include <cuda_fp16.h>

namespace pfd {
namespace {

constexpr int kWarps = kRowsWarps;
constexpr int kThreads = kWarps * 32;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNoRef = -1e30f;     // reference of a row that has seen no key (finite: no inf - inf)
constexpr float kLag = 8.0f;         // a reference may lag its maximum by this (log2)
constexpr float kProbBias = 7.0f;    // a probability at the reference enters as 2^7: at most 2^15

// Transposes an 8 x 8 matrix of f16 spread over a warp (lane l: row l / 4,
// columns 2 (l % 4) and + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// d += a b: 16 x 8 fp32, a 16 x 16 f16 (row major), b 16 x 8 f16.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void lds64(uint32_t addr, uint32_t& x, uint32_t& y) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(addr) : "memory");
}

// The four codes of w as f16 pairs (codes 0, 1 and 2, 3).
template <int kFmt>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kFmt == kFmtE4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // code + 128 under the exponent of 1024 is 1152 + code
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Largest magnitude bits of a word's two bf16 and m; infinities and NaN are left
// out, so the finite elements beside one keep their bits (it stays what it is
// under any scale).
__device__ __forceinline__ uint32_t max_mag(uint32_t m, uint32_t w) {
  const uint32_t x = w & 0x7FFF7FFFu;
  return __vmaxu2(m, x & __vcmpltu2(x, 0x7F807F80u));
}

// x of 2^x <= largest magnitude < 2^(x + 1) of bf16 magnitude bits (two halves
// of m, of this lane); -127 of zeros and subnormals.
__device__ __forceinline__ int top_exponent(uint32_t m) {
  const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
  return static_cast<int>(top >> 7) - 127;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float two_to(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// bf16 pair times 2^e1 2^e2, as an f16 pair (two factors: e may be as low as -240).
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float f1, float f2) {
  return pack_f16x2(bf16_lo(w) * f1 * f2, bf16_hi(w) * f1 * f2);
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t* w) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
}

// A pair of groups in a warp's ring: K of both, then V, 16 key rows of D bytes
// each in TMA's swizzle of D bytes (a row's 16-byte chunks are XORed with the
// row).  The eight lanes of an access phase find theirs in different banks:
// lane (g, c) reads chunks 2c, 2c + 1 (D = 64: c) of K rows g and g + 8, and chunk g
// (D = 64: half of chunk g / 2) of V rows 2c, 2c + 1, 2c + 8, 2c + 9.
template <int D>
struct Ring {
  static constexpr int kGroup = 16 * D;       // bytes of K or V of one group
  static constexpr int kBytes = 4 * kGroup;   // one pair
  static __device__ __forceinline__ uint32_t at(int row, int chunk) {
    return row * D + ((chunk ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4);
  }
};

// Pairs in a ring: 192 KB of them in a CTA.
template <int D>
constexpr int kStages = (192 * 1024) / (kWarps * Ring<D>::kBytes);

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t* src, bool ok) {
  static_assert(N % 4 == 0, "16-byte loads");
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint4 x = ok ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0u, 0u, 0u, 0u);
    w[4 * i] = x.x;
    w[4 * i + 1] = x.y;
    w[4 * i + 2] = x.z;
    w[4 * i + 3] = x.w;
  }
}

// State of a warp's rows: NT tiles of 8; a lane holds rows 2c and 2c + 1 of each
// (c = lane % 4): outputs of columns (lane / 4) * D / 8 + 2 mt + h in o[t][mt][2 h + i],
// relative to y, and this lane's share of l.
template <int D, int NT>
struct RowState {
  float o[NT][D / 16][4];
  float m[NT][2], y[NT][2], l[NT][2];
};

// Probabilities of NG groups' logits, as the second product's right operands b,
// with the references moved and the outputs rescaled to them.  s: the groups'
// raw products, [key lane / 4 + 8 h][row 2c + i] in s[..][2 h + i]; f: per group and
// row, what makes them log2-unit logits; ev: V's exponents (NaN: a NaN block);
// nv: the groups' existing keys.
template <int D, int NT, int NG>
__device__ __forceinline__ void weigh(RowState<D, NT>& st, float (&s)[NG][NT][4],
                                      const float (&f)[NT][2], const float (&ks)[NG],
                                      const float (&ev)[NG], const int (&nv)[NG], int g4,
                                      uint32_t (&b)[NG][NT][2]) {
  // How far the largest logits pass the references.
  float over = -INFINITY;
  bool ragged = false;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    if (nv[g] < kGroupRows) {   // warp-uniform
      ragged = true;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (8 * h + g4 >= nv[g]) s[g][t][2 * h] = s[g][t][2 * h + 1] = -INFINITY;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float x = fmaxf(s[g][t][i], s[g][t][2 + i]) * (f[t][i] * ks[g]);
        over = max3(over, x - st.m[t][i], x + ev[g] - st.y[t][i]);
      }
  }
  if (__any_sync(0xFFFFFFFFu, over > kLag)) {
    // Rare after a row's first keys: every reference moves to its maximum.
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float top = -INFINITY, top_y = -INFINITY;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float x = fmaxf(s[g][t][i], s[g][t][2 + i]) * (f[t][i] * ks[g]);
          top = fmaxf(top, x);
          top_y = fmaxf(top_y, x + ev[g]);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
          top_y = fmaxf(top_y, __shfl_xor_sync(0xFFFFFFFFu, top_y, o));
        }
        // (From kNoRef the factors are 0, and what they multiply is too.)
        const float m_new = fmaxf(st.m[t][i], top), y_new = fmaxf(st.y[t][i], top_y);
        const float ao = ex2_approx(st.y[t][i] - y_new);
        st.l[t][i] *= ex2_approx(st.m[t][i] - m_new);
        st.m[t][i] = m_new;
        st.y[t][i] = y_new;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          st.o[t][mt][i] *= ao;
          st.o[t][mt][2 + i] *= ao;
        }
      }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float f0 = f[t][0] * ks[g], f1 = f[t][1] * ks[g];
      const float y0 = ev[g] + kProbBias - st.y[t][0], y1 = ev[g] + kProbBias - st.y[t][1];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x0 = s[g][t][2 * h], x1 = s[g][t][2 * h + 1];
        float p0 = ex2_approx(fmaf(x0, f0, -st.m[t][0])), p1 = ex2_approx(fmaf(x1, f1, -st.m[t][1]));
        float w0 = ex2_approx(fmaf(x0, f0, y0)), w1 = ex2_approx(fmaf(x1, f1, y1));
        if (ragged && 8 * h + g4 >= nv[g]) p0 = p1 = w0 = w1 = 0.0f;
        st.l[t][0] += p0;
        st.l[t][1] += p1;
        b[g][t][h] = transpose8(pack_f16x2(w0, w1));
      }
    }
}

// Four floats of padding per 16 and a pitch of 4 mod 16: the lanes of an access
// fall into different banks.
template <int D>
struct Join {
  static constexpr int kPitch = D + D / 16 * 4 + 4;
  static __device__ __forceinline__ int at(int row, int d) { return row * kPitch + d + (d >> 4) * 4; }
};

// The rings, and after the last group the warps' outputs.
template <int D, int NT>
constexpr int rows_smem_bytes() {
  const int ring = 1024 + kWarps * kStages<D> * Ring<D>::kBytes;
  const int join = kWarps * 8 * NT * Join<D>::kPitch * 4;
  return ring > join ? ring : join;
}

// kSeqItems: items by sequence, of a ragged batch.
template <int D, int kFmt, int NT, bool kSeqItems>
__global__ void __launch_bounds__(kThreads, 1)
decode_rows_kernel(const __grid_constant__ RowsParams p) {
  using R = Ring<D>;
  constexpr int kRows = 8 * NT;
  constexpr int kStages = pfd::kStages<D>;
  constexpr int kPad = 8;
  extern __shared__ __align__(16) float o_sm[];   // rings; then the warps' outputs [warp][row][column]
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ int32_t seg_row[kMaxSegments], seg_len[kMaxSegments], seg_g0[kMaxSegments + 1];
  __shared__ float sm_m[kWarps][kRows], sm_y[kWarps][kRows], sm_l[kWarps][kRows];
  __shared__ float sm_scale[kRows];   // of a row: scale_log2 * 2^(its exponent)
  __shared__ __align__(16) uint16_t q_sm[kRows][D + kPad];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < kWarps * kStages) mbar_init(&full[0][0] + tid, 1);
  fence_barrier_init();
  grid_dependency_wait();
  int idx = static_cast<int>(blockIdx.x), seq = 0, n_splits = p.n_splits;
  if constexpr (kSeqItems) {
    seq = seq_of_item(p.seq, p.batch, idx);
    n_splits = p.seq.splits(seq);
    idx -= p.seq.first(seq);
  }
  const int split = idx % n_splits;
  idx /= n_splits;
  const int head = idx % p.Hkv;
  if constexpr (!kSeqItems) seq = idx / p.Hkv;
  const int lq0 = p.cu_lq[seq], lq1 = p.cu_lq[seq + 1];
  const int k0 = p.cu_k[seq], k1 = p.cu_k[seq + 1];
  if (lq0 < 0 || lq1 < lq0 || lq1 > p.total_lq || k0 < 0 || k1 < k0 || k1 > p.total_sel ||
      k1 - k0 >= kMaxSegments || lq1 - lq0 > kRows / p.G) {
    if (tid == 0) raise_dev_err(p.dev_err, PFD_DEVERR_SHAPE);
    return;
  }
  const int lq = lq1 - lq0, n_rows = lq * p.G;
  if (n_rows == 0) return;
  const int nsel = k1 - k0;

  // Selected slots, through the table.
  for (int i = tid; i < nsel; i += kThreads) {
    const int c = p.sel[k0 + i];
    int row = 0, len = 0;
    if (c < 0 || c >= p.table_len) {
      raise_dev_err(p.dev_err, PFD_DEVERR_SEL);
    } else {
      const pfd_chunk_entry e = p.table[c];
      if (e.row < 0 || e.len < 0 || static_cast<long long>(e.row) + e.len > p.pool_rows ||
          e.row % kGroupRows != 0 || e.len > p.max_chunk_len) {
        raise_dev_err(p.dev_err, PFD_DEVERR_TABLE);
      } else {
        row = e.row;
        len = e.len;
      }
    }
    seg_row[i] = row;
    seg_len[i] = len;
  }
  __syncthreads();
  if (warp == 0) {   // first group of every slot
    int carry = 0;
    for (int base = 0; base < nsel; base += 32) {
      const int i = base + lane;
      const int n = i < nsel ? (seg_len[i] + kGroupRows - 1) / kGroupRows : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += x;
      }
      if (i < nsel) seg_g0[i] = carry + incl - n;
      carry += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0) seg_g0[nsel] = carry;
  }
  __syncthreads();

  const int n_code = seg_g0[nsel];
  const int n_live = p.self_keys ? (lq + kGroupRows - 1) / kGroupRows : 0;
  const long long total = static_cast<long long>(n_code) + n_live;
  const int g_lo = static_cast<int>(total * split / n_splits);
  const int g_hi = static_cast<int>(total * (split + 1) / n_splits);
  // ------------------------------------------------------------ code groups --
  // The warp's i-th pair of groups begins at g_lo + 2 (warp + i * kWarps); the
  // last pair of the range may lack its second group (no keys).
  const int code_hi = min(g_hi, n_code);
  const int n_pairs = code_hi > g_lo ? (code_hi - g_lo + 1) / 2 : 0;
  const int n_it = warp < n_pairs ? (n_pairs - warp + kWarps - 1) / kWarps : 0;
  // Per group of a pair: its pool row, its existing keys (0: no group) and its
  // exponent bytes (K's, V's), which nothing waits for before the loads.
  struct Place {
    int row[2], nv[2];
    uint32_t ek[2], ev[2];
  };
  auto look_up = [&](int base) {   // lane l: pair base + l of the warp
    Place x{{0, 0}, {0, 0}, {0u, 0u}, {0u, 0u}};
    const int i = base + lane;
    if (i < n_it) {
      const int first = g_lo + 2 * (warp + i * kWarps);
      int lo = 0, hi = nsel;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seg_g0[mid] <= first) lo = mid;
        else hi = mid;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int grp = first + h;
        if (grp >= code_hi) break;
        while (seg_g0[lo + 1] <= grp) ++lo;   // ends: grp < n_code = seg_g0[nsel]
        const int ofs = (grp - seg_g0[lo]) * kGroupRows;
        x.row[h] = seg_row[lo] + ofs;
        const long long at = static_cast<long long>(x.row[h] / kGroupRows) * p.Hkv + head;
        x.nv[h] = min(kGroupRows, seg_len[lo] - ofs);
        x.ek[h] = __ldg(p.exp_k + at);
        x.ev[h] = __ldg(p.exp_v + at);
      }
    }
    return x;
  };
  uint8_t* const rings =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(o_sm) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const ring = rings + warp * (kStages * R::kBytes);
  int base = 0;   // the lanes hold the places of pairs base .. base + 31
  Place here = look_up(base);
  auto fill = [&](int i) {
    if (lane != i - base) return;
    uint64_t* bar = &full[warp][i % kStages];
    uint8_t* dst = ring + (i % kStages) * R::kBytes;
    const int n = here.nv[1] != 0 ? 2 : 1;
    mbar_arrive_expect_tx(bar, n * 2 * R::kGroup);
    for (int h = 0; h < n; ++h) {
      tma_load_3d(dst + h * R::kGroup, &p.tm_k, bar, 0, head, here.row[h]);
      tma_load_3d(dst + (2 + h) * R::kGroup, &p.tm_v, bar, 0, head, here.row[h]);
    }
  };
  for (int i = 0; i < min(kStages, n_it); ++i) fill(i);
  // Query rows in f16, a row per warp; rows past the last one are zero.
  for (int r = warp; r < kRows; r += kWarps) {
    constexpr int kWords = D / 64;   // bf16 pairs of a lane
    uint32_t w[kWords] = {};
    if (r < n_rows) {
      const int t = r / p.G, j = r - t * p.G;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          p.q + (static_cast<long long>(lq0 + t) * p.Hq + head * p.G + j) * D);
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __ldg(src + lane * kWords + i);
    }
    uint32_t mag = 0u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) mag = max_mag(mag, w[i]);
    const int e = max(top_exponent(mag), -100) - 14;   // to 2^14..2^15
    const float f1 = two_to(-e / 2), f2 = two_to(-e - (-e / 2));
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      reinterpret_cast<uint32_t*>(q_sm[r])[lane * kWords + i] = bf16x2_to_f16x2(w[i], f1, f2);
    if (lane == 0) sm_scale[r] = p.scale_log2 * two_to(e);
  }
  __syncthreads();
  const int c = lane & 3, g4 = lane >> 2;
  // Q's fragments: dimensions 4 kk.. of the lane's share, row g4 of each tile.
  // In registers for up to two tiles of rows, else read again for each pair.
  constexpr bool kQRegs = NT <= 2;
  const uint32_t q_addr = smem_u32(&q_sm[g4][c * (D / 4)]);
  auto q_frag = [&](int t, int kk, uint32_t (&b)[2]) {
    lds64(q_addr + (8 * t * (D + kPad) + 4 * kk) * 2, b[0], b[1]);
  };
  uint32_t qr[kQRegs ? NT : 1][kQRegs ? D / 16 : 1][2];
  if constexpr (kQRegs) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) q_frag(t, kk, qr[t][kk]);
  }
  float qf[NT][2];
  RowState<D, NT> st;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      qf[t][i] = sm_scale[8 * t + 2 * c + i];
      st.m[t][i] = st.y[t][i] = kNoRef;
      st.l[t][i] = 0.0f;
    }
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[t][mt][i] = 0.0f;
  }
  bool ok = true;
  for (int i = 0; i < n_it; ++i) {
    const int stage = i % kStages;
    if (!mbar_wait_warp(&full[warp][stage], (i / kStages) & 1)) {
      ok = false;   // what else is on its way lands before the ring is used again
      for (int k = i + 1; k < min(n_it, i + kStages); ++k)
        mbar_wait_warp(&full[warp][k % kStages], (k / kStages) & 1);
      break;
    }
    const uint32_t src = smem_u32(ring + stage * R::kBytes);
    int nv[2];
    float ks[2], ev[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint32_t info = __shfl_sync(
          0xFFFFFFFFu, static_cast<uint32_t>(here.nv[g]) | (here.ek[g] << 8) | (here.ev[g] << 16), i - base);
      const uint32_t ek = (info >> 8) & 0xFFu, e = info >> 16;
      const float nan = __uint_as_float(0x7FC00000u);
      nv[g] = static_cast<int>(info & 0xFFu);
      // 2^(ek - 127): the byte as an exponent, with the mantissa's upper bit for byte 0
      // (2^-127 is subnormal) and for byte 255 (a NaN)
      ks[g] = __uint_as_float((ek << 23) | (((ek + 1u) & 0xFEu) == 0u ? 0x00400000u : 0u));
      ev[g] = e == 255u ? nan : static_cast<float>(static_cast<int>(e) - 127);
    }
    float s[2][NT][4] = {};
#pragma unroll
    for (int k4 = 0; k4 < D / 64; ++k4) {   // four products of 16 dimensions
      uint32_t kw[2][2][4];
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          lds128(src + g * R::kGroup + R::at(g4 + 8 * h, c * (D / 64) + k4), kw[g][h]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t a[2][4];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          codes_to_f16<kFmt>(kw[g][0][k], a[g][0], a[g][2]);
          codes_to_f16<kFmt>(kw[g][1][k], a[g][1], a[g][3]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint32_t b[2];
          if constexpr (kQRegs) {
            b[0] = qr[t][4 * k4 + k][0];
            b[1] = qr[t][4 * k4 + k][1];
          } else {
            q_frag(t, 4 * k4 + k, b);
          }
#pragma unroll
          for (int g = 0; g < 2; ++g) mma_f16(s[g][t], a[g], b[0], b[1]);
        }
      }
    }
    uint32_t b[2][NT][2];
    weigh<D, NT, 2>(st, s, qf, ks, ev, nv, g4, b);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t vw[4][D / 32];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int key = 2 * c + (h & 1) + 8 * (h >> 1);
        const uint32_t at = src + (2 + g) * R::kGroup;
        if constexpr (D == 128) lds128(at + R::at(key, g4), vw[h]);
        else lds64(at + R::at(key, g4 >> 1) + (g4 & 1) * 8, vw[h][0], vw[h][1]);
      }
      if (nv[g] < kGroupRows) {   // rows behind the slot's last one may hold anything
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (2 * c + (h & 1) + 8 * (h >> 1) >= nv[g]) {
#pragma unroll
            for (int w = 0; w < D / 32; ++w) vw[h][w] = 0u;
          }
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
#pragma unroll
        for (int q = 0; q < 2; ++q) {   // bytes 2q, 2q + 1 of two keys' words, paired
          uint32_t a[4];
          codes_to_f16<kFmt>(__byte_perm(vw[0][w], vw[1][w], q ? 0x7362 : 0x5140), a[0], a[1]);
          codes_to_f16<kFmt>(__byte_perm(vw[2][w], vw[3][w], q ? 0x7362 : 0x5140), a[2], a[3]);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_f16(st.o[t][2 * w + q], a, b[g][t][0], b[g][t][1]);
        }
    }
    __syncwarp();   // the warp is done with the stage
    if (i + kStages >= base + 32 && base + 32 < n_it) {
      base = i + 1;
      here = look_up(base);
    }
    if (i + kStages < n_it) fill(i + kStages);
  }
  if (!ok && lane == 0) raise_dev_err(p.dev_err, PFD_DEVERR_TIMEOUT);
  // ------------------------------------------------------------ live groups --
  const long long stride = static_cast<long long>(p.Hkv) * D;
  for (int grp = max(g_lo, n_code) + warp; grp < g_hi; grp += kWarps) {
    const int row0 = (grp - n_code) * kGroupRows;
    const int nv[1] = {min(kGroupRows, lq - row0)};
    const bf16* kb = p.k_self + (lq0 + row0) * stride + head * D + c * (D / 4);
    const bf16* vb = p.v_self + (lq0 + row0) * stride + head * D + g4 * (D / 8);
    uint32_t k[2][D / 8], v[4][D / 16], mag = 0u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load_words(k[h], reinterpret_cast<const uint8_t*>(kb + (g4 + 8 * h) * stride), g4 + 8 * h < nv[0]);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) mag = max_mag(mag, k[h][i]);
    }
    const int ke = max(top_exponent(mag), -100) - 14;
    mag = 0u;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int key = 2 * c + (h & 1) + 8 * (h >> 1);
      load_words(v[h], reinterpret_cast<const uint8_t*>(vb + key * stride), key < nv[0]);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) mag = max_mag(mag, v[h][i]);
    }
    const int ve = max(top_exponent(mag), -100) - 8;   // to 2^8..2^9, about a code's size
    const float kf1 = two_to(-ke / 2), kf2 = two_to(-ke - (-ke / 2));
    const float vf1 = two_to(-ve / 2), vf2 = two_to(-ve - (-ve / 2));
    float s[1][NT][4] = {};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t a[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[h] = bf16x2_to_f16x2(k[h][2 * kk], kf1, kf2);
        a[2 + h] = bf16x2_to_f16x2(k[h][2 * kk + 1], kf1, kf2);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint32_t b[2];
        q_frag(t, kk, b);
        mma_f16(s[0][t], a, b[0], b[1]);
      }
    }
    const float ks[1] = {two_to(ke)}, ev[1] = {static_cast<float>(ve)};
    uint32_t b[1][NT][2];
    weigh<D, NT, 1>(st, s, qf, ks, ev, nv, g4, b);
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {   // columns 2 mt and + 1: the halves of word mt
      uint32_t a[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[2 * h] = bf16x2_to_f16x2(__byte_perm(v[2 * h][mt], v[2 * h + 1][mt], 0x5410), vf1, vf2);
        a[2 * h + 1] = bf16x2_to_f16x2(__byte_perm(v[2 * h][mt], v[2 * h + 1][mt], 0x7632), vf1, vf2);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) mma_f16(st.o[t][mt], a, b[0][t][0], b[0][t][1]);
    }
  }

  // ------------------------------------------------------- join the warps --
  __syncthreads();   // every warp is done with its ring
  using J = Join<D>;
  float* mine = o_sm + warp * (kRows * J::kPitch);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float l = st.l[t][i];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
      const int row = 8 * t + 2 * c + i;
      if (g4 == 0) {
        sm_m[warp][row] = st.m[t][i];
        sm_y[warp][row] = st.y[t][i];
        sm_l[warp][row] = l;
      }
#pragma unroll
      for (int q = 0; q < D / 32; ++q)
        *reinterpret_cast<float4*>(mine + J::at(row, g4 * (D / 8) + 4 * q)) =
            make_float4(st.o[t][2 * q][i], st.o[t][2 * q][2 + i], st.o[t][2 * q + 1][i],
                        st.o[t][2 * q + 1][2 + i]);
    }
  __syncthreads();
  const bool whole = p.n_splits == 1;
  for (int i = tid; i < n_rows * (D / 4); i += kThreads) {
    const int row = i / (D / 4), d = (i % (D / 4)) * 4;
    float m = kNoRef, y = kNoRef;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      m = fmaxf(m, sm_m[w][row]);
      y = fmaxf(y, sm_y[w][row]);
    }
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      l += sm_l[w][row] * ex2_approx(sm_m[w][row] - m);
      const float f = ex2_approx(sm_y[w][row] - y);
      const float4 x = *reinterpret_cast<const float4*>(
          o_sm + w * (kRows * J::kPitch) + J::at(row, d));
      o.x = fmaf(x.x, f, o.x);
      o.y = fmaf(x.y, f, o.y);
      o.z = fmaf(x.z, f, o.z);
      o.w = fmaf(x.w, f, o.w);
    }
    // O is relative to 2^(y - 7), l to 2^m.  (l is NaN where a logit was.)
    float e = y - kProbBias - m;
    if (e < -60.0f) {   // V scales near 2^-127: ex2_approx gives 0 below 2^-126, so two factors
      const float down = two_to(-64);
      o = make_float4(o.x * down, o.y * down, o.z * down, o.w * down);
      e += 64.0f;
    }
    const float f = l == 0.0f ? 0.0f : ex2_approx(e) / l;
    const int t = row / p.G, j = row - t * p.G;
    const long long at = static_cast<long long>(lq0 + t) * p.Hq + head * p.G + j;
    if (whole) {
      *reinterpret_cast<uint2*>(p.out + at * D + d) =
          make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
      if (d == 0 && p.lse != nullptr) p.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
    } else {
      const long long part = static_cast<long long>(split) * p.total_lq * p.Hq + at;
      *reinterpret_cast<float4*>(p.part_acc32 + part * D + d) =
          make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
      if (d == 0) {
        p.part_m[part] = l == 0.0f ? -INFINITY : m;
        p.part_l[part] = l;
        if (kSeqItems && split == 0)   // the splits that this sequence has not
          for (int s = n_splits; s < p.n_splits; ++s) {
            const long long none = static_cast<long long>(s) * p.total_lq * p.Hq + at;
            p.part_m[none] = -INFINITY;
            p.part_l[none] = 0.0f;
          }
      }
    }
  }
  grid_dependents_launch();
}

template <int D, int kFmt, int NT>
cudaError_t launch_t(const RowsParams& p, int grid, cudaStream_t stream) {
  constexpr int smem = rows_smem_bytes<D, NT>();
  const auto kernel =
      p.by_seq ? decode_rows_kernel<D, kFmt, NT, true> : decode_rows_kernel<D, kFmt, NT, false>;
  const cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  if (err != cudaSuccess) return err;
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, stream, p);
}

template <int D, int kFmt>
cudaError_t launch_fmt(const RowsParams& p, int grid, cudaStream_t stream) {
  switch (p.row_tiles) {
    case 1: return launch_t<D, kFmt, 1>(p, grid, stream);
    case 2: return launch_t<D, kFmt, 2>(p, grid, stream);
    default: return launch_t<D, kFmt, 4>(p, grid, stream);
  }
}

}  // namespace

cudaError_t launch_decode_rows(const RowsParams& p, int grid, cudaStream_t stream) {
  if (grid <= 0) return cudaSuccess;
  if (p.fmt == kFmtE4M3)
    return p.D == 64 ? launch_fmt<64, kFmtE4M3>(p, grid, stream) : launch_fmt<128, kFmtE4M3>(p, grid, stream);
  return p.D == 64 ? launch_fmt<64, kFmtInt8>(p, grid, stream) : launch_fmt<128, kFmtInt8>(p, grid, stream);
}

}  // namespace pfd

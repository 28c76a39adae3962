// Prefill GEMM against block-wise quantized weights:
//   Y[m][n] = sum_k X[m][k] * w_bf16[n][k]
// with w_bf16 = bf16(fp32 fma(S, C[q], Z)) for the 2-bit code
// ("On-The-Fly Weight Synthesizer (OTF-LLM Engine v4.0)", sections 2-4) or
// bf16(fp32 absmax * L[q]) for NF4 ("AirQuant" README, "Fundamentacao
// Teorica e Arquitetura" item 2). 2-bit anchor columns take bf16(out_w).
//
// Tiling: a 256-thread workgroup computes a 256 (M) x 256 (N) tile of Y; its
// four waves (2 x 2) each own 128 x 128 as 4 x 4 blocks of
// v_mfma_f32_32x32x16_bf16 (fp32 accumulators, 256 per lane). K advances 64
// at a time through two LDS buffers: while the waves multiply out of one,
// the next tile -- X copied, the packed W dequantized in registers straight
// to bf16 -- is written to the other and the one after that is in flight
// from memory; one LDS-only barrier per step. LDS rows are padded by 16
// bytes so 16-byte fragment reads of consecutive rows hit distinct banks.
// Workgroups are ordered M-tile fastest, so consecutive workgroups (spread
// over the eight XCDs) share a W tile and each XCD keeps one X slab in L2.
//
// 2-bit dequant: per group of 32 the four possible bf16 values
// v_q = bf16(fma(S, C[q], Z)) are formed once and packed into two dwords;
// a v_perm_b32 whose byte selectors are built from two code fields then
// assembles a bf16 pair, so each weight costs a few integer ops.
#include <stdlib.h>

#include "prefill_w.h"

namespace qw {
namespace {

// 32 codes of one group (two code dwords c0, c1 = elements 0..15, 16..31)
// -> 16 dwords of bf16 pairs in natural element order. The four possible
// values bf16(fma(S, C[q], Z)) are packed in T1:T0 (byte 2q, 2q+1 = value
// q); codes are unpacked to bytes (d_t byte j = code of element 4j + t of a
// 16-code half), one v_perm gathers the two codes of an output pair, a
// shift-add turns them into byte selectors and a second v_perm looks the
// pair up: three integer ops per two weights.
__device__ inline void dequant_group_2bit(uint32_t c0, uint32_t c1, uint32_t szw,
                                          uint32_t out[16]) {
  const float S = f16_bits_to_f32((uint16_t)(szw & 0xFFFFu));
  const float Z = f16_bits_to_f32((uint16_t)(szw >> 16));
  const uint32_t T0 = pack_bf16x2(__builtin_fmaf(S, -1.52f, Z), __builtin_fmaf(S, -0.45f, Z));
  const uint32_t T1 = pack_bf16x2(__builtin_fmaf(S, 0.45f, Z), __builtin_fmaf(S, 1.52f, Z));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c = h ? c1 : c0;
    uint32_t d[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) d[t] = (c >> (2 * t)) & 0x03030303u;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      // elements 2p, 2p+1 = 4j + t, 4j + t + 1 with j = p / 2, t = 2 (p % 2)
      const int j = p >> 1, t = 2 * (p & 1);
      const uint32_t gsel = (uint32_t)j * 0x0101u + (uint32_t)(4 + j) * 0x01010000u;
      const uint32_t r = __builtin_amdgcn_perm(d[t + 1], d[t], gsel);  // q0 q0 q1 q1
      out[h * 8 + p] = __builtin_amdgcn_perm(T1, T0, (r << 1) + 0x01000100u);
    }
  }
}

template <int FMT, bool F32OUT>
__global__ __launch_bounds__(NT) void prefill_kernel(PrefillArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  // two buffers of X [BM][LDA] and W [BN][LDA] tiles, then the NF4 table
  auto As = [&](int buf) { return smem + buf * BM * LDA; };
  auto Bs = [&](int buf) { return smem + 2 * BM * LDA + buf * BN * LDA; };
  float2 *ltab = reinterpret_cast<float2 *>(smem + 2 * (BM + BN) * LDA);  // NF4 [256]

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv >> 1, wn = wv & 1;
  const int b = blockIdx.x;
  const int m_tile = b % a.mt_count;
  const int n_tile = b / a.mt_count;
  const int m0 = m_tile * BM, n0 = n_tile * BN;
  const int K = a.K;
  const int KT = K / BK;

  if (FMT != QW_FMT_2BIT_G32) {  // NF4 levels, or u - 8 for INT4
    for (int v = tid; v < 256; v += NT) ltab[v] = make_float2(a.nf4[v & 15], a.nf4[v >> 4]);
  }

  // ---- global prefetch registers: 8 x 16 bytes of X, one W column ----
  uint4 ra[8];
  uint32_t rb[9];
  const int gn = n0 + tid;  // this thread's W column
  const bool bvalid = gn < a.N;

  auto load_x = [&](int kt) {
    const int k0 = kt * BK;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i * NT + tid;
      const int row = c >> 3, c16 = c & 7;
      const int gm = m0 + row;
      ra[i] = (gm < a.M)
                  ? *reinterpret_cast<const uint4 *>(a.X + (size_t)gm * K + k0 + c16 * 8)
                  : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_w = [&](int kt) {
    const int k0 = kt * BK;
    if (FMT == QW_FMT_2BIT_G32) {
      if (bvalid) {
        const u32x4 v = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4 *>(a.codes + (size_t)gn * (K / 16) + k0 / 16));
        rb[0] = v.x; rb[1] = v.y; rb[2] = v.z; rb[3] = v.w;
        const uint32_t *sp = reinterpret_cast<const uint32_t *>(a.scales) + (size_t)gn * (K / 32) + k0 / 32;
        rb[4] = __builtin_nontemporal_load(sp);
        rb[5] = __builtin_nontemporal_load(sp + 1);
      } else {
        rb[0] = rb[1] = rb[2] = rb[3] = rb[4] = rb[5] = 0;
      }
    } else {
      if (bvalid) {
        const u32x4 *cp = reinterpret_cast<const u32x4 *>(a.codes + (size_t)gn * (K / 8) + k0 / 8);
        const u32x4 v0 = __builtin_nontemporal_load(cp), v1 = __builtin_nontemporal_load(cp + 1);
        rb[0] = v0.x; rb[1] = v0.y; rb[2] = v0.z; rb[3] = v0.w;
        rb[4] = v1.x; rb[5] = v1.y; rb[6] = v1.z; rb[7] = v1.w;
        rb[8] = __builtin_bit_cast(uint32_t, __builtin_nontemporal_load(
            reinterpret_cast<const float *>(a.scales) + (size_t)gn * (K / 64) + k0 / 64));
      } else {
        for (int i = 0; i < 9; ++i) rb[i] = 0;
      }
    }
  };

  // X pieces of this thread (already in registers) into buffer buf
  auto store_x = [&](int buf) {
    uint16_t *A = As(buf);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i * NT + tid;
      const int row = c >> 3, c16 = c & 7;
      *reinterpret_cast<uint4 *>(A + row * LDA + c16 * 8) = ra[i];
    }
  };
  // one 32-element group (half h of the 64 k of tile kt) of this thread's W
  // column, dequantized to bf16, into buffer buf
  auto store_w = [&](int kt, int buf, int h) {
    uint4 *bp = reinterpret_cast<uint4 *>(Bs(buf) + tid * LDA);
    uint32_t out[16];
    if (FMT == QW_FMT_2BIT_G32) {
      dequant_group_2bit(rb[2 * h], rb[2 * h + 1], rb[4 + h], out);
      if (a.n_out > 0 && bvalid) {
        // anchor columns of this group: idx is ascending, find the first >= k_lo
        const int k_lo = kt * BK + 32 * h;
        int lo = 0, hi = a.n_out;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (a.idx[mid] < k_lo) lo = mid + 1; else hi = mid;
        }
        for (int o = lo; o < a.n_out && a.idx[o] < k_lo + 32; ++o) {
          const int e = a.idx[o] - k_lo;
          const float v = f16_bits_to_f32(a.wo[(size_t)gn * a.n_out_pad + o]);
          const uint32_t bb = f32_to_bf16_bits(v);
          // static indexing only, so out[] stays in registers
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            if (q == (e >> 1))
              out[q] = (e & 1) ? ((out[q] & 0xFFFFu) | (bb << 16)) : ((out[q] & 0xFFFF0000u) | bb);
          }
        }
      }
    } else {
      // NF4: one fp32 absmax per 64; INT4: the fp16 scale of group h
      const float am = FMT == QW_FMT_NF4_B64 ? __builtin_bit_cast(float, rb[8])
                                            : f16_bits_to_f32((uint16_t)(rb[8] >> (16 * h)));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t c = rb[4 * h + i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 l = ltab[(c >> (8 * j)) & 0xFFu];
          out[i * 4 + j] = pack_bf16x2(am * l.x, am * l.y);
        }
      }
      // INT4 anchors: permuted positions below n_out take bf16(out_w)
      const int k_lo = kt * BK + 32 * h;
      if (FMT == QW_FMT_INT4_G32 && bvalid && k_lo < a.n_out) {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int e = k_lo + 2 * q;
          const uint16_t *wr = a.wo + (size_t)gn * a.n_out_pad;
          const uint32_t b0 = e < a.n_out ? f32_to_bf16_bits(f16_bits_to_f32(wr[e])) : (out[q] & 0xFFFFu);
          const uint32_t b1 = e + 1 < a.n_out ? f32_to_bf16_bits(f16_bits_to_f32(wr[e + 1])) : (out[q] >> 16);
          out[q] = b0 | (b1 << 16);
        }
      }
    }
    bp[4 * h + 0] = make_uint4(out[0], out[1], out[2], out[3]);
    bp[4 * h + 1] = make_uint4(out[4], out[5], out[6], out[7]);
    bp[4 * h + 2] = make_uint4(out[8], out[9], out[10], out[11]);
    bp[4 * h + 3] = make_uint4(out[12], out[13], out[14], out[15]);
  };

  floatx16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // The products of tile kt out of buffer buf, with tile kt+1 written to the
  // other buffer between the 16-wide k slices (X after slice 0, the two W
  // groups after slices 1 and 2) so the writes and the dequantization run
  // beside the matrix cores; X and W of tile kt+2 are requested as soon as
  // their registers are free.
  auto read_frags = [&](int buf, int kk, bf16x8 (&af)[4], bf16x8 (&bfr)[4]) {
    const uint16_t *A = As(buf), *Bt = Bs(buf);
    const int kof = kk * 16 + (lane >> 5) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = wm * 128 + i * 32 + (lane & 31);
      af[i] = *reinterpret_cast<const bf16x8 *>(A + row * LDA + kof);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = wn * 128 + j * 32 + (lane & 31);
      bfr[j] = *reinterpret_cast<const bf16x8 *>(Bt + col * LDA + kof);
    }
  };
  // One K step: the products of tile kt out of buffer buf, with tile kt+1
  // written to the other buffer between the 16-wide k slices (X after slice
  // 0, the two W groups after slices 1 and 2) and X, W of tile kt+2
  // requested as soon as their registers are free. The side work is
  // unconditional (on the last step it fills the idle buffer; loads past the
  // end re-read the last tile) so each slice is one basic block, and
  // scheduling groups interleave it with the matrix-core instructions: with
  // one wave per SIMD, in-order issue would otherwise leave the matrix cores
  // idle while it runs.
  auto compute = [&](int kt, int buf) {
    const int kn = min(kt + 2, KT - 1);
    bf16x8 fa[2][4], fb[2][4];  // fragments of the current and the next k slice
    read_frags(buf, 0, fa[0], fb[0]);
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk) {
      if (kk + 1 < BK / 16) read_frags(buf, kk + 1, fa[(kk + 1) & 1], fb[(kk + 1) & 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[kk & 1][i], fb[kk & 1][j],
                                                               acc[i][j], 0, 0, 0);
      if (kk == 0) {
        store_x(buf ^ 1);
        load_x(kn);
      } else if (kk == 1) {
        store_w(kt + 1, buf ^ 1, 0);
      } else if (kk == 2) {
        store_w(kt + 1, buf ^ 1, 1);
        load_w(kn);
      }
      // 16 x {1 product, fragment reads, a few vector ops, an LDS write,
      // a memory read}
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // DS read
        __builtin_amdgcn_sched_group_barrier(0x002, 7, 0);  // VALU
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // DS write
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // VMEM read
      }
    }
  };

  // the NF4 table and tile 0 must be in LDS before the first step
  load_x(0);
  load_w(0);
  __syncthreads();
  store_x(0);
  store_w(0, 0, 0);
  store_w(0, 0, 1);
  if (KT > 1) {
    load_x(1);
    load_w(1);
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  for (int kt = 0; kt < KT; ++kt) {
    compute(kt, kt & 1);
    // LDS-only barrier: the loads of tile kt+2 stay in flight
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  }

  // ---- epilogue: lane holds D[8*g + 4*(lane>>5) + r][lane & 31] ----
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int gn_ = n0 + wn * 128 + j * 32 + (lane & 31);
      if (gn_ >= a.N) continue;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int gm = m0 + wm * 128 + i * 32 + 8 * g + 4 * (lane >> 5) + r;
          if (gm >= a.M) continue;
          const float v = acc[i][j][4 * g + r];
          const size_t o = (size_t)gm * a.N + gn_;
          if (F32OUT)
            reinterpret_cast<float *>(a.Y)[o] = v;
          else
            reinterpret_cast<uint16_t *>(a.Y)[o] = (uint16_t)f32_to_bf16_bits(v);
        }
      }
    }
  }
}


template <int FMT, bool F32, int NJ>
qw_status launch_w(const PrefillArgs &a, int n_begin, int n_tiles, hipStream_t s) {
  if (n_tiles <= 0) return QW_OK;
  PrefillArgs b = a;
  b.n_begin = n_begin;
  const size_t lds = (size_t)2 * BM * LDA * 2;  // the NF4 pair table is static
  // one wave per SIMD owning all 256 rows (WM = 1): measured on MI355X, two
  // waves per SIMD with 128 rows each (WM = 2) are slower, since the two
  // waves sharing a column both dequantize it
  constexpr int WM = 1;
  QW_HIP_TRY(hipFuncSetAttribute(reinterpret_cast<const void *>(&prefill_w_kernel<FMT, F32, NJ, WM, PrefillArgs>),
                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds));
  QW_HIP_TRY(launch(prefill_w_kernel<FMT, F32, NJ, WM, PrefillArgs>, a.mt_count * n_tiles, 256 * WM, lds, s, b));
  return QW_OK;
}

// Column split between 256-wide tiles and 128-wide tiles for the last
// columns: a whole number of rounds of wide tiles over the CUs, then one
// short round of narrow ones instead of a half-empty round of wide ones.
// Cost model in units of one wide-tile round; a narrow tile costs 0.55 of a
// wide one (half the products, same fixed per-step work).
int wide_column_tiles(int mt, int N, int cus) {
  const int nt = (N + 255) / 256;
  double best = 1e30;
  int best_n = nt;
  for (int n = nt; n >= 0; --n) {
    const long wide = (long)mt * n;
    const int rest = N - 256 * n;
    const long narrow = rest > 0 ? (long)mt * ((rest + 127) / 128) : 0;
    const double cost = (double)((wide + cus - 1) / cus) + 0.55 * (double)((narrow + cus - 1) / cus);
    if (cost < best - 1e-9) {
      best = cost;
      best_n = n;
    }
  }
  return best_n;
}

template <int FMT>
qw_status launch_fmt(const PrefillArgs &a, bool f32, int cus, hipStream_t s) {
  const size_t esz = f32 ? 4 : 2;
  const bool fits32 = (size_t)a.M * a.K * 2 < kPfOob && (size_t)a.M * a.N * esz < kPfOob &&
                      (size_t)a.N * (a.K / 2) < kPfOob;
  if (a.n_out == 0 && fits32) {  // W straight to registers
    // the test hook QW_TUNE_PREFILL_WIDE_TILES overrides the number of
    // 256-wide column tiles (tests run the 128-wide kernel on small shapes)
    const int nt = (a.N + 255) / 256;
    const int forced = tune(QW_TUNE_PREFILL_WIDE_TILES);
    const int nw = forced >= 0 ? min(forced, nt) : wide_column_tiles(a.mt_count, a.N, cus);
    const int rest = a.N - 256 * nw;
    const int nn = rest > 0 ? (rest + 127) / 128 : 0;
    if (f32) {
      QW_TRY((launch_w<FMT, true, 2>(a, 0, nw, s)));
      QW_TRY((launch_w<FMT, true, 1>(a, 256 * nw, nn, s)));
    } else {
      QW_TRY((launch_w<FMT, false, 2>(a, 0, nw, s)));
      QW_TRY((launch_w<FMT, false, 1>(a, 256 * nw, nn, s)));
    }
    return QW_OK;
  }
  const int nt = (a.N + BN - 1) / BN;
  const int grid = a.mt_count * nt;
  const size_t lds = (size_t)2 * (BM + BN) * LDA * 2 + (FMT != QW_FMT_2BIT_G32 ? 256 * 8 : 0);
  const void *fn = f32 ? reinterpret_cast<const void *>(&prefill_kernel<FMT, true>)
                       : reinterpret_cast<const void *>(&prefill_kernel<FMT, false>);
  QW_HIP_TRY(hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds));
  if (f32)
    QW_HIP_TRY(launch(prefill_kernel<FMT, true>, grid, NT, lds, s, a));
  else
    QW_HIP_TRY(launch(prefill_kernel<FMT, false>, grid, NT, lds, s, a));
  return QW_OK;
}

}  // namespace
}  // namespace qw

extern "C" qw_status qgemm_prefill(const qw_weight *w, const void *X, int M, void *Y,
                                   qw_dtype y_dtype, void *stream) {
  using namespace qw;
  CallScope scope;
  if (!w || !X || !Y || M < 1) return QW_ERR_INVALID_ARG;
  if (y_dtype != QW_DT_BF16 && y_dtype != QW_DT_F32) return QW_ERR_INVALID_ARG;
  if (!w || (w->format != QW_FMT_2BIT_G32 && w->format != QW_FMT_NF4_B64 && w->format != QW_FMT_INT4_G32))
    return QW_ERR_INVALID_ARG;
  qw_status st = check_weight_view(w, w->format, 0);
  if (st != QW_OK) return st;
  if (w->K % 64) return QW_ERR_UNSUPPORTED;
  if (!aligned16(X) || !aligned16(Y)) return QW_ERR_ALIGNMENT;
  int cus = 0;
  st = current_device(&cus);
  if (st != QW_OK) return st;
  PrefillArgs a{};
  a.X = reinterpret_cast<const uint16_t *>(X);
  a.codes = reinterpret_cast<const uint32_t *>(w->codes);
  a.scales = w->scales;
  a.idx = w->out_idx;
  a.wo = w->out_w;
  a.Y = Y;
  a.M = M;
  a.N = w->N;
  a.K = w->K;
  a.n_out = w->format == QW_FMT_NF4_B64 ? 0 : w->n_out;
  a.n_out_pad = w->n_out_pad;
  a.mt_count = (M + BM - 1) / BM;
  a.xcd_group = 4;  // row tiles an XCD walks per column sweep
  // level of each 4-bit code: the NF4 table, or u - 8 for INT4
  const float *L = nf4_levels_host();
  for (int i = 0; i < 16; ++i) a.nf4[i] = w->format == QW_FMT_INT4_G32 ? (float)(i - 8) : L[i];
  const bool f32 = y_dtype == QW_DT_F32;
  if (w->format == QW_FMT_2BIT_G32) return launch_fmt<QW_FMT_2BIT_G32>(a, f32, cus, as_stream(stream));
  if (w->format == QW_FMT_INT4_G32) return launch_fmt<QW_FMT_INT4_G32>(a, f32, cus, as_stream(stream));
  return launch_fmt<QW_FMT_NF4_B64>(a, f32, cus, as_stream(stream));
}

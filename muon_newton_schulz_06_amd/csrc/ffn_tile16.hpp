// Products of the gated feed-forward block on bf16 MFMA.
//
// C[i][j] = Σ_k A[i][k]·B[j][k] on TILE×TILE tiles (TILE 256: eight waves of
// 128×64; TILE 128: four waves of 64×64), k in steps of 32, with the 256-tile
// kernel's scheme of gemm.hpp: operands go straight from global memory into
// a 4-slot LDS ring (three k-tiles in flight), one barrier per k-tile with
// explicit vmcnt waits, fragments of the next quarter read while the MFMAs of
// the current one run.  What differs from it:
//  * an operand is k-contiguous (LDS rows of 32 k, read with 16-byte reads) or
//    row-contiguous (LDS panel of 32 k-rows, read with transposing reads):
//    the weights are used both ways and nothing is ever transposed in memory;
//  * no padded operands: the loads are buffer loads whose lanes point past the
//    buffer (and so deliver zeros) outside rows and k.  The k loop always runs
//    a multiple of four k-tiles, the surplus ones zero;
//  * FFN_GLU: a tile is TILE rows × TILE/2 columns of both projections.  Of a
//    wave's 64 B rows 32 are w_gate's and 32 w_up's, so g and u of one element
//    meet in one lane and the activation runs on fp32 registers.
// Bound by the matrix pipe at the power-limited clock (1.9–2.0 GHz, MFMA busy
// 49–62%): 0.77 µs per k-tile of a 256-tile on every CU.  At 4096 tokens,
// 3584×18944: gated projections with a, b 1087 µs (1020 TFLOP/s), dh 560 (990),
// dx 888 (1250), weight gradients 1310 (1270), y 490 (1130).  The 128-tile takes
// 0.62 µs per k-tile and pair of workgroups on a CU, which wins where 256-tiles
// would leave CUs idle (see the time estimate on the host).
// Operands need 16-byte aligned rows of whole 16-byte chunks; the host copies
// others once.
#pragma once

#include "dma.hpp"
#include "ffn_epi.hpp"
#include "gemm.hpp"

namespace muon {

typedef __bf16 fbf16x8 __attribute__((ext_vector_type(8)));

template <int TILE, int EPI, bool AROW, bool BROW>
__global__ __launch_bounds__(TILE * 2, 2) void ffn_tile16(const FfnLaunch L) {
  constexpr int TM = TILE, TN = TILE, SLOTS = 4;
  constexpr int NW = TILE / 32, WN = TN / 64, WTM = TM / 2, FM = WTM / 16, FN = 4;
  constexpr int KB = 32;                                             // k per k-tile
  constexpr int kA = TM * KB * 2, kB = TN * KB * 2, kSlot = kA + kB;  // bytes of the operands' tiles, of a slot
  constexpr int NA = TM / (16 * NW), NB = TN / (16 * NW);            // loads of a wave per operand and k-tile
  constexpr int NQ = FM / 2;  // quarters (pairs of block rows) per k-tile
  __shared__ __attribute__((aligned(1024))) char lds[SLOTS * kSlot];

  constexpr bool kTwo = EPI == FFN_STORE && !AROW && BROW;  // the launches with two k ranges
  // A slot's refill spread over the last quarter's MFMAs, one load after each:
  // dx 957 -> 900 µs, weight gradients 1390 -> 1341 µs, dh 571 -> 562 µs (4096
  // tokens, 3584×18944); FFN_GLU, whose loads need a buffer each, 1066 -> 1090
  // µs, so it issues them ahead of the MFMAs.
  constexpr bool kSpread = EPI != FFN_GLU;

  const int tid = threadIdx.x;
  int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int lc = lane & 15, lg = lane >> 4;

  // problem, tile and k split of this workgroup
  const int b = xcd_window_remap(blockIdx.x, gridDim.x, kXcdShift);
  int q = 0;
  while (q + 1 < L.nprob && b >= L.tiles[q + 1]) ++q;
  const FfnProb& P = L.prob[q];
  constexpr int TC = EPI == FFN_GLU ? TN / 2 : TN;  // columns of the result
  const int tilesM = (P.M + TM - 1) / TM, tilesN = (P.N + TC - 1) / TC;
  int t = b - L.tiles[q];
  const int split = t / (tilesM * tilesN);
  t -= split * (tilesM * tilesN);
  // bands of four tile rows, column by column inside a band
  const int band = t / (kBand * tilesN), r0 = band * kBand, bh = min(kBand, tilesM - r0);
  const int tb = t - r0 * tilesN, tj = tb / bh, ti = r0 + tb - tj * bh;
  const int64_t i0 = (int64_t)ti * TM, j0 = (int64_t)tj * TC;

  const int KT0 = (P.K[0] + KB - 1) / KB;
  const int KT = KT0 + (P.K[1] + KB - 1) / KB;
  const int per = L.splitTiles;  // k-tiles per split, a multiple of four
  const int kt0 = split * per;
  const int n = min(per, (KT - kt0 + 3) & ~3);

  // Each lane's place in the loads: byte offset from the operand's tile start
  // (nowhere if its row, or its chunk of a row-contiguous operand, does not
  // exist) and the k it holds.
  uint32_t offA[NA], offB[NB];
  [[maybe_unused]] uint32_t offB1[NB];  // the second k range's, whose stride may differ
  int kkA[NA], kkB[NB];
  auto place = [&](bool rowc, int T, int N, int64_t ld, int64_t first, int64_t extent, int p, uint32_t& off, int& k)
                   __attribute__((always_inline)) {
    if (rowc) {
      const int CH = T / 8, RPI = 64 / CH;  // chunks of a k-row, k-rows per load
      const int r = (wave * N + p) * RPI + lane / CH;
      const int c = (lane % CH) ^ tswz(r);
      k = r;
      off = first + c * 8 < extent ? (uint32_t)(r * ld * 2 + c * 16) : kFfnNowhere;
    } else {
      const int r = (wave * N + p) * 16 + (lane >> 2);
      const int c = (lane & 3) ^ swz4(r);
      k = c * 8;
      off = first + r < extent ? (uint32_t)(r * ld * 2 + c * 16) : kFfnNowhere;
    }
  };
  // FFN_GLU: rows 64·c + 0..31 of the B tile are w_gate's rows 32·c.., the next
  // 32 w_up's, so a wave's 32 rows are one matrix's
  static_assert(NB == 2, "a wave loads 32 rows of B");
  const bool up = EPI == FFN_GLU && (wave & 1);
  const int64_t ldB = up ? P.ldb[1] : P.ldb[0];
#pragma unroll
  for (int p = 0; p < NA; ++p) place(AROW, TM, NA, P.lda, i0, AROW ? P.extA : P.M, p, offA[p], kkA[p]);
#pragma unroll
  for (int p = 0; p < NB; ++p) {
    if constexpr (EPI == FFN_GLU) {
      const int r = (wave * NB + p) * 16 + (lane >> 2), c = (lane & 3) ^ swz4(r);
      const int f = (r >> 6) * 32 + (r & 31);
      kkB[p] = c * 8;
      offB[p] = j0 + f < P.N ? (uint32_t)(f * ldB * 2 + c * 16) : kFfnNowhere;
    } else {
      place(BROW, TN, NB, P.ldb[0], j0, BROW ? P.extB : P.N, p, offB[p], kkB[p]);
      if constexpr (kTwo) place(BROW, TN, NB, P.ldb[1], j0, BROW ? P.extB : P.N, p, offB1[p], kkB[p]);
    }
  }
  // tile starts and bytes per k of both k ranges
  const uint64_t a0 = (uint64_t)P.A[0] + (AROW ? (uint64_t)i0 : (uint64_t)i0 * P.lda) * 2;
  const uint64_t a1 = (uint64_t)P.A[1] + (AROW ? (uint64_t)i0 : (uint64_t)i0 * P.lda) * 2;
  const uint64_t b0 = (uint64_t)(up ? P.B[1] : P.B[0]) + (BROW ? (uint64_t)j0 : (uint64_t)j0 * ldB) * 2;
  const uint64_t b1 = (uint64_t)P.B[1] + (BROW ? (uint64_t)j0 : (uint64_t)j0 * P.ldb[1]) * 2;
  const uint32_t ka = AROW ? (uint32_t)P.lda * 2 : 2, kb0 = BROW ? (uint32_t)P.ldb[0] * 2 : 2,
                 kb1 = BROW ? (uint32_t)P.ldb[1] * 2 : 2;
  const int K0 = P.K[0], K1 = P.K[1];
  const uint32_t dst = __builtin_amdgcn_readfirstlane(lds_addr(lds) + wave * (NA * 1024));
  const uint32_t dstB = __builtin_amdgcn_readfirstlane(lds_addr(lds) + kA + wave * (NB * 1024));
  // load j of k-tile kt (A's, then B's) into the slot at byte `slot`
  auto issue_one = [=](int slot, int kt, auto jc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value;
    const bool z = kTwo && kt >= KT0;
    const int k0 = (z ? kt - KT0 : kt) * KB, left = (z ? K1 : K0) - k0;
    if constexpr (j < NA) {
      f_dma16(dst + slot + j * 1024, kkA[j] < left ? offA[j] : kFfnNowhere,
              f_buffer((z ? a1 : a0) + (uint64_t)k0 * ka));
    } else {
      constexpr int p = j - NA;
      uint32_t o = offB[p];
      if constexpr (kTwo) o = z ? offB1[p] : o;
      f_dma16(dstB + slot + p * 1024, kkB[p] < left ? o : kFfnNowhere,
              f_buffer((z ? b1 : b0) + (uint64_t)k0 * (z ? kb1 : kb0)));
    }
  };
  auto issue = [=](int slot, int kt) __attribute__((always_inline)) {
    static_for<0, NA + NB>([&](auto jc) __attribute__((always_inline)) { issue_one(slot, kt, jc); });
  };

  floatx4 acc[FM][FN];
#pragma unroll
  for (int fi = 0; fi < FM; ++fi)
#pragma unroll
    for (int fj = 0; fj < FN; ++fj) acc[fi][fj] = floatx4{0.f, 0.f, 0.f, 0.f};

  const int sw = swz4(lc);
  auto frag = [&](const char* pan, int row0, auto rowc, auto tc) __attribute__((always_inline)) {
    if constexpr (decltype(rowc)::value) {
      constexpr int T = decltype(tc)::value;
      auto rd = [&](int k0) {
        const int k = k0 + (lc >> 2), i = row0 + 4 * (lc & 3);
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s4_t)(pan + k * (T * 2) + (((i >> 3) ^ tswz(k)) << 4) + (i & 7) * 2));
      };
      const short4_t lo = rd(8 * lg), hi = rd(8 * lg + 4);
      return __builtin_bit_cast(fbf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *(const fbf16x8*)(pan + (row0 + lc) * 64 + ((lg ^ sw) << 4));
    }
  };
  constexpr auto kAr = std::bool_constant<AROW>{};
  constexpr auto kBr = std::bool_constant<BROW>{};
  fbf16x8 fb0[FN], fb1[FN], fax[2], fay[2];
  auto load_a = [&](fbf16x8 (&fa)[2], const char* st, int qq) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < 2; ++f) fa[f] = frag(st, wm * WTM + (2 * qq + f) * 16, kAr, std::integral_constant<int, TM>{});
  };
  auto load_b = [&](fbf16x8 (&fb)[FN], const char* st) __attribute__((always_inline)) {
#pragma unroll
    for (int fj = 0; fj < FN; ++fj) fb[fj] = frag(st + kA, wn * 64 + fj * 16, kBr, std::integral_constant<int, TN>{});
  };
  // operand roles swapped: a lane holds four consecutive columns of one row
  auto mma = [&](const fbf16x8 (&fa)[2], const fbf16x8 (&fb)[FN], auto qc) __attribute__((always_inline)) {
    constexpr int qq = decltype(qc)::value;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int fj = 0; fj < FN; ++fj)
        acc[2 * qq + f][fj] =
            __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[fj], fa[f], acc[2 * qq + f][fj], 0, 0, 0);
  };
  // One k-tile (its slot at byte cur, the next one's at nxt): all quarters but
  // the last while the next quarter's fragments are read; then the slot is free
  // for every wave, the next k-tile has landed (each is NA + NB loads per wave,
  // SLOTS − 2 stay in flight), the slot is refilled, and the last quarter runs
  // while the next k-tile's first fragments are read.
  auto step = [&](int cur, int nxt, int kt, const fbf16x8 (&fb)[FN], fbf16x8 (&fbn)[FN]) __attribute__((always_inline)) {
    const char* st = lds + cur;
    static_for<0, NQ - 1>([&](auto qc) __attribute__((always_inline)) {
      constexpr int qq = decltype(qc)::value;
      load_a(qq & 1 ? fax : fay, st, qq + 1);
      __builtin_amdgcn_sched_barrier(0);
      mma(qq & 1 ? fay : fax, fb, qc);
      __builtin_amdgcn_sched_barrier(0);
    });
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"((SLOTS - 2) * (NA + NB)) : "memory");
    const char* sn = lds + nxt;
    if constexpr (!kSpread) issue(cur, kt + SLOTS);
    load_b(fbn, sn);
    load_a(fax, sn, 0);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kSpread) {
      static_for<0, 2 * FN>([&](auto jc) __attribute__((always_inline)) {
        constexpr int j = decltype(jc)::value, f = j / FN, fj = j % FN, qq = NQ - 1;
        acc[2 * qq + f][fj] =
            __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[fj], fay[f], acc[2 * qq + f][fj], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (j < NA + NB) issue_one(cur, kt + SLOTS, jc);
        __builtin_amdgcn_sched_barrier(0);
      });
    } else {
      mma(fay, fb, std::integral_constant<int, NQ - 1>{});
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(NQ % 2 == 0, "the last quarter's fragments are in fay");
  if (n > 0) {
    // loads past this split's k-tiles, the next split's or zeros past the last
    // k, are never read
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) issue(i * kSlot, kt0 + i);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"i"((SLOTS - 1) * (NA + NB)) : "memory");
    load_b(fb0, lds);
    load_a(fax, lds, 0);
    for (int kt = kt0; kt < kt0 + n; kt += 4) {
      step(0, kSlot, kt, fb0, fb1);
      step(kSlot, 2 * kSlot, kt + 1, fb1, fb0);
      step(2 * kSlot, 3 * kSlot, kt + 2, fb0, fb1);
      step(3 * kSlot, 0, kt + 3, fb1, fb0);
    }
  }
  // no load may still be on its way into LDS when the workgroup ends
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  // the epilogue's addresses are formed here, not kept through the loop
  asm volatile("" : "+v"(lane));
  lc = lane & 15;
  lg = lane >> 4;

  // acc[fi][fj][r]: row fi·16 + lane%16, column fj·16 + 4·(lane/16) + r
  const int64_t iw = i0 + wm * WTM + lc;
  // results: f(i, j, fi, fj) for every group of four columns inside the rows
  // and the given width
  auto groups = [&](auto nfj, int cols, int64_t width, auto&& f) __attribute__((always_inline)) {
#pragma unroll
    for (int fi = 0; fi < FM; ++fi) {
      const int64_t i = iw + fi * 16;
      if (i >= P.M) continue;
#pragma unroll
      for (int fj = 0; fj < decltype(nfj)::value; ++fj) {
        const int64_t j = j0 + wn * cols + fj * 16 + 4 * lg;
        if (j < width) f(i, j, fi, fj);
      }
    }
  };
  auto four = [](const floatx4& c, float (&v)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = c[r];
  };
  constexpr auto kTwoF = std::integral_constant<int, 2>{};
  constexpr auto kAllF = std::integral_constant<int, FN>{};
  if (P.part) {
    if constexpr (EPI == FFN_GLU) {
      groups(kTwoF, 32, P.partN / 2, [&](int64_t i, int64_t j, int fi, int fj) __attribute__((always_inline)) {
        float g[4], u[4];
        four(acc[fi][fj], g);
        four(acc[fi][fj + 2], u);
        ffn_part4(P, split, i, j, true, 0, g);
        ffn_part4(P, split, i, j, true, 1, u);
      });
    } else {
      groups(kAllF, 64, P.partN, [&](int64_t i, int64_t j, int fi, int fj) __attribute__((always_inline)) {
        float c[4];
        four(acc[fi][fj], c);
        ffn_part4(P, split, i, j, false, 0, c);
      });
    }
    return;
  }
  // bf16 results are staged in the ring, which every wave has left behind,
  // and stored as whole rows, 16 bytes per lane: stored from the registers a
  // 256-tile's results (8 bytes per lane, 16 rows at a time) took about 15 µs.
  // A staged tile of W columns: chunk c of row r at c ^ r (mod W/8).
  auto soff = [](int W, int row, int col) __attribute__((always_inline)) {
    return row * W * 2 + (((col >> 3) ^ (row & (W / 8 - 1))) << 4) + (col & 7) * 2;
  };
  auto put = [&](char* st, int W, int row, int col, uint2 v) __attribute__((always_inline)) {
    *(uint2*)(st + soff(W, row, col)) = v;
  };
  // Rows of a staged tile → C, rows staged in `parts` groups per row half (the
  // staged row r is row (r / HR)·WTM + r % HR of part `part`).
  auto rows_out = [&](const char* st, auto wc, auto partsc, int part, void* C, int64_t ldc, int64_t width)
                      __attribute__((always_inline)) {
    constexpr int W = decltype(wc)::value, CH = W / 8, RPI = 64 / CH;
    constexpr int PARTS = decltype(partsc)::value, HR = WTM / PARTS, RW = TM / PARTS / NW;  // rows of a wave
#pragma unroll 4
    for (int p = 0; p < RW / RPI; ++p) {
      const int r = wave * RW + p * RPI + lane / CH, c = lane % CH;
      const int64_t i = i0 + (r / HR) * WTM + part * HR + r % HR, j = j0 + c * 8;
      const lu32x4 v = *(const lu32x4*)(st + soff(W, r, c * 8));
      if (i >= P.M || j >= width) continue;
      uint16_t* o = (uint16_t*)C + i * ldc + j;
      if (j + 8 <= width) {
        *(lu32x4*)o = v;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (j + e < width) o[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
      }
    }
  };
  constexpr auto kOne = std::integral_constant<int, 1>{};
  const int lrow = wm * WTM + lc;  // a lane's row of block row 0, and its column below
  if constexpr (EPI == FFN_GLU) {
    // half of every wave's rows at a time: h and the three planes of a and b
    constexpr int W = TN / 2, HR = WTM / 2;
    constexpr auto kW = std::integral_constant<int, W>{};
    constexpr int kPart = TM / 2 * W * 2;  // bytes of one array's half tile
    static_assert(4 * kPart <= SLOTS * kSlot, "staged arrays fit");
    // columns N .. ldh − 1 come out as zeros
    ffn_with_glu(L, [&](auto actc, auto savec) __attribute__((always_inline)) {
      constexpr bool SAVE = decltype(savec)::value;
      static_for<0, 2>([&](auto pc) __attribute__((always_inline)) {
        constexpr int part = decltype(pc)::value;
        __syncthreads();
#pragma unroll
        for (int fi = part * (FM / 2); fi < (part + 1) * (FM / 2); ++fi)
#pragma unroll
          for (int fj = 0; fj < 2; ++fj) {
            const int row = wm * HR + (fi - part * (FM / 2)) * 16 + lc, col = wn * 32 + fj * 16 + 4 * lg;
            float v[4], d[4], h[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float u = acc[fi][fj + 2][r];
              ffn_act<decltype(actc)::value, false>(acc[fi][fj][r], v[r], d[r]);
              h[r] = v[r] * u;
              d[r] *= u;
            }
            put(lds, W, row, col, make_uint2(l_f32_bf16x2(h[0], h[1]), l_f32_bf16x2(h[2], h[3])));
            if constexpr (SAVE) {
              put(lds + kPart, W, row, col, make_uint2(l_upper2(d[0], d[1]), l_upper2(d[2], d[3])));
              put(lds + 2 * kPart, W, row, col, make_uint2(l_upper2(v[0], v[1]), l_upper2(v[2], v[3])));
              put(lds + 3 * kPart, W, row, col,
                  make_uint2(l_lower2(d[0], v[0], d[1], v[1]), l_lower2(d[2], v[2], d[3], v[3])));
            }
          }
        __syncthreads();
        constexpr auto kHalves = std::integral_constant<int, 2>{};
        rows_out(lds, kW, kHalves, part, P.C, P.ldc, L.ldh);
        if constexpr (SAVE) {
#pragma unroll
          for (int p = 0; p < 3; ++p)
            rows_out(lds + (p + 1) * kPart, kW, kHalves, part, (uint16_t*)L.ab + p * L.ldh, 3 * L.ldh, L.ldh);
        }
      });
    });
  } else if constexpr (EPI == FFN_BACK) {
    // a quarter of every wave's rows at a time: the planes of a and b are loaded
    // into the staging, the upper halves multiplied in place (a lane reads and
    // writes the same addresses) and stored as dg and du
    constexpr auto kW = std::integral_constant<int, TN>{};
    constexpr auto kQuarters = std::integral_constant<int, 4>{};
    constexpr int CH = TN / 8, RPI = 64 / CH, HR = WTM / 4, RW = TM / 4 / NW;
    constexpr int kPlane = TM / 4 * TN * 2;  // bytes
    static_assert(3 * kPlane <= SLOTS * kSlot, "staged planes fit");
    static_for<0, 4>([&](auto pc) __attribute__((always_inline)) {
      constexpr int part = decltype(pc)::value;
      __syncthreads();
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) {
        const fi32x4 rs = f_buffer((uint64_t)L.ab + ((uint64_t)i0 * 3 * L.ldh + pl * L.ldh + j0) * 2);
#pragma unroll
        for (int p = 0; p < RW / RPI; ++p) {
          const int r = wave * RW + p * RPI + lane / CH, c = (lane % CH) ^ (r & (CH - 1));
          const int i = (r / HR) * WTM + part * HR + r % HR;
          const uint32_t off = i0 + i < P.M && j0 + c * 8 < L.ldh ? (uint32_t)((int64_t)i * 6 * L.ldh + c * 16) : kFfnNowhere;
          f_dma16(__builtin_amdgcn_readfirstlane(lds_addr(lds) + pl * kPlane + (wave * RW + p * RPI) * TN * 2), off, rs);
        }
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
#pragma unroll
      for (int f = 0; f < FM / 4; ++f)
#pragma unroll
        for (int fj = 0; fj < FN; ++fj) {
          char* const at = lds + soff(TN, wm * HR + f * 16 + lc, wn * 64 + fj * 16 + 4 * lg);
          const uint2 a = *(const uint2*)at, b = *(const uint2*)(at + kPlane), lower = *(const uint2*)(at + 2 * kPlane);
          const floatx4 c = acc[part * (FM / 4) + f][fj];
          *(uint2*)at = ffn_times24<0>(c, a, lower);
          *(uint2*)(at + kPlane) = ffn_times24<1>(c, b, lower);
        }
      __syncthreads();
      rows_out(lds, kW, kQuarters, part, P.C, P.ldc, L.ldh);
      rows_out(lds + kPlane, kW, kQuarters, part, (uint16_t*)P.C + L.ldh, P.ldc, L.ldh);
    });
  } else if (L.outBf16 && !L.accumulate && ((uintptr_t)P.C & 15) == 0 && (P.ldc & 7) == 0) {
    __syncthreads();
#pragma unroll
    for (int fi = 0; fi < FM; ++fi)
#pragma unroll
      for (int fj = 0; fj < FN; ++fj) {
        const floatx4 c = acc[fi][fj];
        put(lds, TN, lrow + fi * 16, wn * 64 + fj * 16 + 4 * lg,
            make_uint2(l_f32_bf16x2(c[0], c[1]), l_f32_bf16x2(c[2], c[3])));
      }
    __syncthreads();
    rows_out(lds, std::integral_constant<int, TN>{}, kOne, 0, P.C, P.ldc, P.N);
  } else {
    groups(kAllF, 64, P.N, [&](int64_t i, int64_t j, int fi, int fj) __attribute__((always_inline)) {
      float c[4];
      four(acc[fi][fj], c);
      ffn_store4(P.C, P.ldc, i, j, P.N, L.outBf16, L.accumulate, P.vecC, c);
    });
  }
}

template <int EPI, bool AROW, bool BROW>
void ffn16_launch(int tile, const FfnLaunch& L, hipStream_t st) {
  const dim3 grid(L.tiles[L.nprob]);
  if (tile == 256) hipLaunchKernelGGL((ffn_tile16<256, EPI, AROW, BROW>), grid, dim3(512), 0, st, L);
  else hipLaunchKernelGGL((ffn_tile16<128, EPI, AROW, BROW>), grid, dim3(256), 0, st, L);
}

}  // namespace muon

// Grouped products of expert-sorted rows with MXFP4 expert matrices.
//
//   forward   out[r, n] = sum_k A[r, k] W[e, n, k]       A MXFP4 (or gathered by route), W MXFP4
//   backward  dx[r, k]  = sum_n dy[r, n] W[e, n, k]      dy BF16, W MXFP4 as the forward read it
//
// with e the expert of row r. Codes and scales are read as the quantizer
// stores them (rows of Kd/2 and Kd/32 bytes). Both kernels bring tiles to LDS by
// loads that write LDS themselves (16 bytes a lane), in a ring of stages, and
// accumulate each output in one chain of FP32 matrix instructions whose order
// depends on Kd (N) alone: a row's bits do not depend on the other rows.
#include <type_traits>

#include "kernels.h"
#include "mx.h"

namespace pmoe {

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- loads into LDS
// A raw buffer of `bytes` bytes: reads at offsets >= bytes give zeros, which is
// how rows past a tile's end and elements past a row's end become zeros.
__device__ __forceinline__ intx4 raw_buffer(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return intx4{__builtin_amdgcn_readfirstlane((int)(uint32_t)a), __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
// An offset that is past every buffer, also with a row's offset added to it
// (row offsets are at most kRowLimit, and a row of nothing is kNoRow).
constexpr uint32_t kPast = 0x7FFFFF00u;
constexpr uint32_t kNoRow = 0x80000000u;

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p);
}
// Lane l's 16 bytes at `offset` go to lds + 16 l (4 bytes to lds + 4 l; one byte, extended
// with zeros to 4, to lds + 4 l). The loads are counted by vmcnt, in order.
__device__ __forceinline__ void load_lds16(intx4 buf, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(buf)
               : "memory");
}
__device__ __forceinline__ void load_lds4(intx4 buf, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(buf)
               : "memory");
}
__device__ __forceinline__ void load_lds1(intx4 buf, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(buf)
               : "memory");
}
template <int kLeft>
__device__ __forceinline__ void wait_loads() {  // until at most kLeft of the wave's loads are under way
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLeft) : "memory");
}

// ---------------------------------------------------------------- work items
// An item is one tile of BM rows of an expert by one column tile; items are
// numbered by expert, then column tile, then row tile, and each XCD (blockIdx %
// 8) takes a contiguous eighth, so that the row tiles that read one matrix tile
// run together on one L2. The item is found from the offsets by every wave: lane
// i scans experts i, 64 + i, ... Offsets are clamped to [0, R].
struct MxItem {
  int e, row0, rows, col;  // rows: of this tile, 1 .. BM
};
__device__ __forceinline__ int wave_scan(int v, int lane) {  // inclusive sum over the lanes
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(v, off, 64);
    if (lane >= off) v += y;
  }
  return v;
}
template <int BM>
__device__ __forceinline__ bool mx_item(const int* offsets, int E, int R, int col_tiles, MxItem& it) {
  const int lane = threadIdx.x & 63;
  auto rows_of = [&](int e, int& first) {
    first = 0;
    if (e >= E) return 0;
    first = min(max(offsets[e], 0), R);
    return max(min(offsets[e + 1], R) - first, 0);
  };
  int total = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    int first;
    total += (rows_of(e0 + lane, first) + BM - 1) / BM;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) total += __shfl_xor(total, off, 64);
  const long items = (long)total * col_tiles;
  const long per = (items + 7) >> 3;
  const long j = blockIdx.x >> 3;
  const long item = (blockIdx.x & 7) * per + j;
  if (j >= per || item >= items) return false;
  const int tile = (int)(item / col_tiles);  // row tiles before this item's expert are at most this
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    int first;
    const int rows = rows_of(e0 + lane, first);
    const int tiles = (rows + BM - 1) / BM;
    const int upto = before + wave_scan(tiles, lane);
    const uint64_t past = __ballot(upto > tile);
    if (past) {
      const int who = __builtin_ctzll(past);
      const int n = __builtin_amdgcn_readlane(tiles, who);
      const int start = __builtin_amdgcn_readlane(upto, who) - n;
      const int local = (int)(item - (long)start * col_tiles);
      const int m = local % n;
      it.e = e0 + who;
      it.col = local / n;
      it.row0 = __builtin_amdgcn_readlane(first, who) + m * BM;
      it.rows = min(__builtin_amdgcn_readlane(rows, who) - m * BM, BM);
      return true;
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// ---------------------------------------------------------------- forward
// v_mfma_scale_f32_32x32x64: a lane holds 32 consecutive codes, exactly one
// block, of row lane % 32 of either operand, and that block's scale byte. The
// matrix is the first operand, so that a lane's results are consecutive
// columns of one row. A stage is 256 elements of the reduction (128 bytes of
// codes, 8 scales a row); which blocks meet in one instruction is free as long as
// both operands agree: half h of the wave takes blocks 4h + j in step j, whose
// four scales are then one aligned dword, read once a stage, and the step selects the byte.
//
// In LDS a row of a stage is 8 slots of 16 bytes; piece p is in slot p ^ (row %
// 8), so the 8 lanes that one LDS access serves (8 rows, one piece) hit 8 slots.
// Loads write LDS in lane order, so the lanes' addresses carry the permutation.
template <int NW_, int MW_, int WN_, int WM_, int S_, bool kBytes_>
struct MxTile {
  static constexpr int NW = NW_, MW = MW_, WN = WN_, WM = WM_, S = S_;
  static constexpr bool kBytes = kBytes_;  // rows of scales are not whole dwords: loaded byte by byte
  static constexpr int kWaves = WN * WM, BN = 32 * NW * WN, BM = 32 * MW * WM, kRows = BN + BM;
  static constexpr int kScaleRow = kBytes ? 32 : 8;
  static constexpr int kStage = kRows * (128 + kScaleRow);
  static constexpr int kLoadW = BN / 8 / kWaves, kLoadX = BM / 8 / kWaves;  // 1 KB loads of a wave
  static constexpr int kScaleLoads = kRows / (kBytes ? 8 : 32);
  static constexpr int kLoadS = (kScaleLoads + kWaves - 1) / kWaves;
  static constexpr int kLoads = kLoadW + kLoadX + kLoadS;
  static_assert(BN % (8 * kWaves) == 0 && BM % (8 * kWaves) == 0, "whole loads");
};

template <class C>
__global__ __launch_bounds__(C::kWaves * 64) void mx_gemm_kernel(MxGemmParams P) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[C::S * C::kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  MxItem it;
  if (!mx_item<C::BM>(P.offsets, P.E, P.R, (P.N + C::BN - 1) / C::BN, it)) return;
  const int n0 = it.col * C::BN;
  const uint32_t krow = P.Kd / 2, srow = P.Kd / kMxBlock;
  const intx4 wq = raw_buffer(P.w_codes + (long)it.e * P.N * krow, (uint32_t)P.N * krow);
  const intx4 ws = raw_buffer(P.w_sf + (long)it.e * P.N * srow, (uint32_t)P.N * srow);
  const long base = P.route_of_row ? 0 : it.row0;
  const uint32_t a_rows = P.route_of_row ? P.a_rows : it.rows;
  const intx4 aq = raw_buffer(P.a_codes + base * krow, a_rows * krow);
  const intx4 as = raw_buffer(P.a_sf + base * srow, a_rows * srow);
  // Row m of the tile in A: its token, or the row itself; -1 past the tile's end.
  auto source = [&](int m) {
    if (m >= it.rows) return -1;
    if (!P.route_of_row) return m;
    const int f = P.route_of_row[it.row0 + m];
    return f >= 0 && f / P.topk < P.a_rows ? f / P.topk : -1;
  };

  // Loads of this lane: of a row of codes 16 bytes, of a row of scales one dword or byte.
  const int lr = lane >> 3;                              // row of the eight
  const uint32_t piece = ((lane & 7) ^ lr) * 16;         // its bytes within the stage's 128
  const uint32_t w_row = (uint32_t)(n0 + 8 * wave * C::kLoadW + lr) * krow;
  uint32_t x_row[C::kLoadX];
#pragma unroll
  for (int i = 0; i < C::kLoadX; ++i) {
    const int r = source(8 * (wave * C::kLoadX + i) + lr);
    x_row[i] = r < 0 ? kNoRow : (uint32_t)r * krow;
  }
  constexpr int kSRows = C::kBytes ? 8 : 32;             // rows of one load of scales
  const int sr = C::kBytes ? lane >> 3 : lane >> 1;
  const uint32_t s_at = C::kBytes ? lane & 7 : (lane & 1) * 4;
  uint32_t s_row[C::kLoadS];
#pragma unroll
  for (int i = 0; i < C::kLoadS; ++i) {
    const int q = min(wave * C::kLoadS + i, C::kScaleLoads - 1) * kSRows;
    if (q < C::BN) {
      s_row[i] = (uint32_t)(n0 + q + sr) * srow;
    } else {
      const int r = source(q - C::BN + sr);
      s_row[i] = r < 0 ? kNoRow : (uint32_t)r * srow;
    }
  }
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(lds));
  auto issue = [&](int st, int slot) {
    const uint32_t to = lds0 + slot * C::kStage;
    const uint32_t kb = (uint32_t)st * 128 + piece;
    const uint32_t k = kb < krow ? kb : kPast;
#pragma unroll
    for (int i = 0; i < C::kLoadW; ++i)
      load_lds16(wq, w_row + i * 8 * krow + k, to + (wave * C::kLoadW + i) * 1024);
#pragma unroll
    for (int i = 0; i < C::kLoadX; ++i)
      load_lds16(aq, x_row[i] + k, to + C::BN * 128 + (wave * C::kLoadX + i) * 1024);
    const uint32_t sb = (uint32_t)st * 8 + s_at;
    const uint32_t sk = sb < srow ? sb : kPast;
#pragma unroll
    for (int i = 0; i < C::kLoadS; ++i) {
      const int q = min(wave * C::kLoadS + i, C::kScaleLoads - 1);
      const intx4 buf = q * kSRows < C::BN ? ws : as;
      if constexpr (C::kBytes)
        load_lds1(buf, s_row[i] + sk, to + C::kRows * 128 + q * 256);
      else
        load_lds4(buf, s_row[i] + sk, to + C::kRows * 128 + q * 256);
    }
  };

  floatx16 acc[C::NW][C::MW];
#pragma unroll
  for (int f = 0; f < C::NW; ++f)
#pragma unroll
    for (int g = 0; g < C::MW; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][g][i] = 0.0f;

  const int wn = wave % C::WN, wm = wave / C::WN;
  const int half = lane >> 5, r32 = lane & 31;
  const int w_at = wn * C::NW * 32 + r32, x_at = C::BN + wm * C::MW * 32 + r32;  // rows of the stage
  auto compute = [&](int slot) {
    const uint8_t* b = lds + slot * C::kStage;
    const uint8_t* sc = b + C::kRows * 128;
    intx4 ws4[C::NW], xs4[C::MW];  // scales of the four steps: bytes of [0], or the words' low bytes
    auto scales = [&](int row) {
      if constexpr (C::kBytes) return *reinterpret_cast<const intx4*>(sc + row * 32 + half * 16);
      else return intx4{*reinterpret_cast<const int*>(sc + row * 8 + half * 4), 0, 0, 0};
    };
#pragma unroll
    for (int f = 0; f < C::NW; ++f) ws4[f] = scales(w_at + 32 * f);
#pragma unroll
    for (int g = 0; g < C::MW; ++g) xs4[g] = scales(x_at + 32 * g);
    auto step = [&](auto J) {
      constexpr int j = decltype(J)::value;
      const int at = ((4 * half + j) ^ (lane & 7)) * 16;
      auto frag = [&](int row) {
        const intx4 v = *reinterpret_cast<const intx4*>(b + row * 128 + at);
        return intx8{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
      };
      intx8 x[C::MW];
#pragma unroll
      for (int g = 0; g < C::MW; ++g) x[g] = frag(x_at + 32 * g);
#pragma unroll
      for (int f = 0; f < C::NW; ++f) {
        const intx8 w = frag(w_at + 32 * f);
#pragma unroll
        for (int g = 0; g < C::MW; ++g) {
          if constexpr (C::kBytes)
            acc[f][g] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x[g], acc[f][g], 4, 4, 0, ws4[f][j], 0, xs4[g][j]);
          else
            acc[f][g] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x[g], acc[f][g], 4, 4, j, ws4[f][0], j, xs4[g][0]);
        }
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  };

  // Stage st is in slot st % S. At its barrier every wave's loads of it have landed
  // and every wave is done with stage st - 1, whose slot the next loads take.
  const int stages = (P.Kd + 255) / 256;
#pragma unroll
  for (int s = 0; s < C::S - 1; ++s) issue(s, s);  // past the last stage: zeros
  int slot = 0;
  for (int st = 0; st < stages; ++st) {
    wait_loads<(C::S - 2) * C::kLoads>();
    lds_barrier();
    issue(st + C::S - 1, slot == 0 ? C::S - 1 : slot - 1);
    compute(slot);
    slot = slot == C::S - 1 ? 0 : slot + 1;
  }
  wait_loads<0>();  // no load may land in LDS after the workgroup's end

  // acc[f][g][i] is column 32 f + 8 (i / 4) + 4 half + i % 4 of row 32 g + r32 of the wave's part.
#pragma unroll
  for (int g = 0; g < C::MW; ++g) {
    const int m = (wm * C::MW + g) * 32 + r32;
    if (m >= it.rows) continue;
    const long row = (long)(it.row0 + m) * P.N;
#pragma unroll
    for (int f = 0; f < C::NW; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + (wn * C::NW + f) * 32 + 8 * q + 4 * half;
        if (n >= P.N) continue;
        const floatx16& a = acc[f][g];
        if (P.out_f32)
          *reinterpret_cast<float4*>(static_cast<float*>(P.out) + row + n) =
              make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.out) + row + n) =
              make_uint2(f32x2_to_bf16x2(a[4 * q], a[4 * q + 1]), f32x2_to_bf16x2(a[4 * q + 2], a[4 * q + 3]));
      }
  }
}

template <class C>
static hipError_t run_gemm(const MxGemmParams& p, hipStream_t s) {
  const long tiles = (long)p.R / C::BM + (p.E < p.R ? p.E : p.R);
  const long grid = (tiles * ((p.N + C::BN - 1) / C::BN) + 7) / 8 * 8;
  mx_gemm_kernel<C><<<(unsigned)grid, C::kWaves * 64, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_mx_gemm(const MxGemmParams& p, hipStream_t s) {
  const bool bytes = p.Kd % 128 != 0;
  const long mean = (long)p.R / p.E;
  if (mean <= 48) return bytes ? run_gemm<MxTile<1, 1, 4, 1, 3, true>>(p, s) : run_gemm<MxTile<1, 1, 4, 1, 3, false>>(p, s);
  return bytes ? run_gemm<MxTile<4, 2, 2, 2, 2, true>>(p, s) : run_gemm<MxTile<4, 2, 2, 2, 3, false>>(p, s);
}

// ---------------------------------------------------------------- backward
// v_mfma_f32_32x32x16_bf16 reduces over 16 rows n of the matrix; a lane needs 8
// consecutive n of one column k, while the codes run along k. So a lane reads
// the same 4 columns (16 bits) of 8 rows, converts each pair of columns with its
// row's scale (exact in BF16), and regroups the halves of row pairs: 4 fragments
// of 32 columns, columns 4c + i in fragment i for lane c, with no transposition
// through LDS. A wave owns 128 columns and every row of the tile, so a matrix tile
// is converted once a workgroup.
//
// A stage is 64 rows n of the matrix (512 columns: 256 bytes a row, 16 scales)
// and 64 columns of dy. Matrix rows with (n / 8) odd have their two halves of
// each 128 bytes exchanged, so that the two halves of a wave, 8 rows apart, read
// different banks.
template <int MW_, int S_, bool kBytes_>
struct MxBackTile {
  static constexpr int MW = MW_, S = S_;
  static constexpr bool kBytes = kBytes_;
  static constexpr int kWaves = 4, BK = 128 * kWaves, BM = 32 * MW, kN = 64;
  static constexpr int kScaleRow = kBytes ? 64 : 16;
  static constexpr int kW = kN * BK / 2, kS = kN * kScaleRow, kStage = kW + kS + BM * kN * 2;
  static constexpr int kLoadW = kW / 1024 / kWaves, kLoadS = kS / 256 / kWaves, kLoadY = BM / 8 / kWaves;
  static constexpr int kLoads = kLoadW + kLoadS + kLoadY;
};

template <class C>
__global__ __launch_bounds__(256) void mx_gemm_backward_kernel(MxGemmParams P) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[C::S * C::kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  MxItem it;
  if (!mx_item<C::BM>(P.offsets, P.E, P.R, (P.Kd + C::BK - 1) / C::BK, it)) return;
  const int k0 = it.col * C::BK;
  const uint32_t krow = P.Kd / 2, srow = P.Kd / kMxBlock, yrow = (uint32_t)P.N * 2;
  const intx4 wq = raw_buffer(P.w_codes + (long)it.e * P.N * krow, (uint32_t)P.N * krow);
  const intx4 ws = raw_buffer(P.w_sf + (long)it.e * P.N * srow, (uint32_t)P.N * srow);
  const intx4 dy = raw_buffer(P.a_codes + (long)it.row0 * yrow, (uint32_t)it.rows * yrow);

  // Loads of this lane: 16 bytes of codes of 1 in 4 rows, a dword (byte) of scales, 16 bytes of dy of 1 in 8 rows.
  const int wr = lane >> 4, slot16 = lane & 15;
  const int sr = C::kBytes ? lane >> 4 : lane >> 2;
  constexpr int kSRows = C::kBytes ? 4 : 16;
  const uint32_t s_k = k0 / kMxBlock + (C::kBytes ? lane & 15 : (lane & 3) * 4);
  const int yr = lane >> 3;
  const uint32_t y_piece = ((lane & 7) ^ yr) * 16;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(lds));
  auto issue = [&](int st, int slot) {
    const uint32_t to = lds0 + slot * C::kStage;
    const uint32_t n0 = (uint32_t)st * C::kN;
#pragma unroll
    for (int i = 0; i < C::kLoadW; ++i) {
      const int q = wave * C::kLoadW + i;                    // rows 4q .. 4q + 3
      const uint32_t k = k0 / 2 + ((slot16 ^ ((q >> 1 & 1) << 2)) * 16);
      const uint32_t n = n0 + 4 * q + wr;
      load_lds16(wq, n < (uint32_t)P.N && k < krow ? n * krow + k : kNoRow, to + q * 1024);
    }
#pragma unroll
    for (int i = 0; i < C::kLoadS; ++i) {
      const int q = wave * C::kLoadS + i;
      const uint32_t n = n0 + kSRows * q + sr;
      const uint32_t at = n < (uint32_t)P.N && s_k < srow ? n * srow + s_k : kNoRow;
      if constexpr (C::kBytes)
        load_lds1(ws, at, to + C::kW + q * 256);
      else
        load_lds4(ws, at, to + C::kW + q * 256);
    }
    const uint32_t yb = n0 * 2 + y_piece;
#pragma unroll
    for (int i = 0; i < C::kLoadY; ++i) {
      const int q = wave * C::kLoadY + i;
      const uint32_t m = 8 * q + yr;
      load_lds16(dy, m < (uint32_t)it.rows && yb < yrow ? m * yrow + yb : kNoRow, to + C::kW + C::kS + q * 1024);
    }
  };

  floatx16 acc[4][C::MW];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int g = 0; g < C::MW; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][g][i] = 0.0f;

  const int half = lane >> 5, c = lane & 31;
  const int w_at = half * 8 * (C::BK / 2) + ((wave * 64 + c * 2) ^ (half << 6));
  const int s_at = C::kBytes ? half * 8 * 64 + (wave * 4 + (c >> 3)) * 4 : half * 8 * 16 + wave * 4 + (c >> 3);
  auto compute = [&](int slot) {
    const uint8_t* b = lds + slot * C::kStage;
    const uint8_t* sc = b + C::kW + s_at;
    const uint8_t* y = b + C::kW + C::kS;
#pragma unroll
    for (int st = 0; st < C::kN / 16; ++st) {
      uint32_t lo[8], hi[8];  // columns 0, 1 and 2, 3 of each of 8 rows
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t q = *reinterpret_cast<const uint16_t*>(b + (16 * st + i) * (C::BK / 2) + w_at);
        const float s = mx_scale(sc[(16 * st + i) * C::kScaleRow]);
        lo[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
        hi[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
      }
      bf16x8_t w[4];
      auto regroup = [](const uint32_t(&v)[8], uint32_t sel) {
        const uint32_t p[4] = {__builtin_amdgcn_perm(v[1], v[0], sel), __builtin_amdgcn_perm(v[3], v[2], sel),
                               __builtin_amdgcn_perm(v[5], v[4], sel), __builtin_amdgcn_perm(v[7], v[6], sel)};
        bf16x8_t r;
        __builtin_memcpy(&r, p, 16);
        return r;
      };
      w[0] = regroup(lo, 0x05040100u);
      w[1] = regroup(lo, 0x07060302u);
      w[2] = regroup(hi, 0x05040100u);
      w[3] = regroup(hi, 0x07060302u);
#pragma unroll
      for (int g = 0; g < C::MW; ++g) {
        const int m = 32 * g + c;
        const bf16x8_t x = *reinterpret_cast<const bf16x8_t*>(y + m * 128 + (((2 * st + half) ^ (lane & 7)) * 16));
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[f][g] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[f], x, acc[f][g], 0, 0, 0);
      }
    }
  };

  const int stages = (P.N + C::kN - 1) / C::kN;
#pragma unroll
  for (int s = 0; s < C::S - 1; ++s) issue(s, s);
  int slot = 0;
  for (int st = 0; st < stages; ++st) {
    wait_loads<(C::S - 2) * C::kLoads>();
    lds_barrier();
    issue(st + C::S - 1, slot == 0 ? C::S - 1 : slot - 1);
    compute(slot);
    slot = slot == C::S - 1 ? 0 : slot + 1;
  }
  wait_loads<0>();

  // acc[f][g][i] is column 4 (8 (i / 4) + 4 half + i % 4) + f of the wave's 128, row 32 g + c.
#pragma unroll
  for (int g = 0; g < C::MW; ++g) {
    const int m = 32 * g + c;
    if (m >= it.rows) continue;
    uint16_t* out = static_cast<uint16_t*>(P.out) + (long)(it.row0 + m) * P.Kd;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = k0 + wave * 128 + 32 * q + 16 * half + 8 * i;
        if (k >= P.Kd) continue;
        const int a = 4 * q + 2 * i;
        const float v[8] = {acc[0][g][a],     acc[1][g][a],     acc[2][g][a],     acc[3][g][a],
                            acc[0][g][a + 1], acc[1][g][a + 1], acc[2][g][a + 1], acc[3][g][a + 1]};
        *reinterpret_cast<uint4*>(out + k) = pack8(v);
      }
  }
}

template <class C>
static hipError_t run_gemm_backward(const MxGemmParams& p, hipStream_t s) {
  const long tiles = (long)p.R / C::BM + (p.E < p.R ? p.E : p.R);
  const long grid = (tiles * ((p.Kd + C::BK - 1) / C::BK) + 7) / 8 * 8;
  mx_gemm_backward_kernel<C><<<(unsigned)grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_mx_gemm_backward(const MxGemmParams& p, hipStream_t s) {
  const bool bytes = p.Kd % 128 != 0;
  const long mean = (long)p.R / p.E;
  if (mean <= 48)
    return bytes ? run_gemm_backward<MxBackTile<1, 3, true>>(p, s) : run_gemm_backward<MxBackTile<1, 3, false>>(p, s);
  return bytes ? run_gemm_backward<MxBackTile<4, 3, true>>(p, s) : run_gemm_backward<MxBackTile<4, 4, false>>(p, s);
}

}  // namespace pmoe

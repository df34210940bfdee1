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
// with zeros to 4, to lds + 4 l). The loads are counted by vmcnt, in order. Each names M0 as
// overwritten, so that no M0 of the compiler's own is merged across it (the compiler allocates
// nothing there and warns that such a register is not saved, which nothing asks for).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(intx4 buf, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(__builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(buf)
               : "m0", "memory");
}
__device__ __forceinline__ void load_lds4(intx4 buf, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(__builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(buf)
               : "m0", "memory");
}
__device__ __forceinline__ void load_lds1(intx4 buf, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, 0 offen lds" ::"s"(__builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(buf)
               : "m0", "memory");
}
#pragma clang diagnostic pop
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
// Tile m of n of an expert with `rows` rows from `first`: the rows' groups of 32 are shared out evenly.
__device__ __forceinline__ MxItem mx_tile(int e, int first, int rows, int m, int n, int col) {
  const int groups = (rows + 31) / 32;
  const int from = (int)((long)m * groups / n) * 32, to = (int)((long)(m + 1) * groups / n) * 32;
  return MxItem{e, first + from, min(rows, to) - from, col};
}
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
      it = mx_tile(e0 + who, __builtin_amdgcn_readlane(first, who), __builtin_amdgcn_readlane(rows, who), local % n, n,
                   local / n);
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
// codes, 8 scales a row: whole lines, as loads of half lines reach half the rate);
// which blocks meet in one instruction is free as long as both operands agree: half
// h of the wave takes blocks 4h + j in step j, whose four scales are then one
// dword, read once a stage, and the step selects the byte.
//
// In LDS a row of a stage is 8 slots of 16 bytes; piece p is in slot p ^ (row /
// 2 % 8), so that the 16 lanes that one cycle serves (16 rows, one piece) meet
// the 16 slots of 64 banks. Loads write LDS in lane order, so the lanes'
// addresses carry the permutation: eight rows a load, the halves of 64 bytes
// exchanged in every second load.
// 16 tokens, 96 routes to 64 experts, N = Kd = 4096: 67 us, the 445 MB of the experts that are hit at
// 6.7 TB/s (reads alone, some of them from the 256 MB cache); 32 rows an expert 141 us (FP32 output: 152).
// 1100 tokens, 4 routes each, 32 experts, N = 1552, Kd = 2080: 33 us (FP32: 37), 0.85 PFLOP/s: byte loads
// of scales and 448 tiles on 256 CUs.
template <int NW_, int MW_, int WN_, int WM_, int S_, bool kBytes_>
struct MxTile {
  static constexpr int NW = NW_, MW = MW_, WN = WN_, WM = WM_, S = S_;
  static constexpr bool kBytes = kBytes_;  // rows of scales are not whole dwords: loaded byte by byte
  static constexpr int kWaves = WN * WM, BN = 32 * NW * WN, BM = 32 * MW * WM, kRows = BN + BM;
  static constexpr int kScaleRow = kBytes ? 32 : 8;
  static constexpr int kLoadW = BN / 8 / kWaves, kLoadX = (BM / 8 + kWaves - 1) / kWaves;  // 1 KB loads of a wave
  static constexpr int kScaleRows = kBytes ? 8 : 32;                                      // rows of one load of scales
  static constexpr int kScaleLoads = kRows / kScaleRows;
  static constexpr int kLoadS = (kScaleLoads + kWaves - 1) / kWaves;
  static constexpr int kLoads = kLoadW + kLoadX + kLoadS;
  static constexpr int kStage = kRows * (128 + kScaleRow);
  static constexpr int kOutRow = 64 * NW + 8;  // bytes of a row of the epilogue's LDS (BF16): banks 2 apart
  static constexpr int kLds = S * kStage > kWaves * 32 * kOutRow ? S * kStage : kWaves * 32 * kOutRow;
  static_assert(BN % (8 * kWaves) == 0 && BN % 32 == 0 && BM % 32 == 0, "whole loads");
};

template <class C>
__global__ __launch_bounds__(C::kWaves * 64) void mx_gemm_kernel(MxGemmParams P) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[C::kLds];
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

  // Loads of this lane: 16 bytes of a row of codes, a dword or byte of a row of
  // scales. A load past the operand's last one repeats the last (same bytes, same place).
  const int lr = lane >> 3;                        // row of the eight
  const uint32_t piece = ((lane & 7) ^ lr >> 1) * 16;  // its bytes within the stage's 128; ^ 64 in odd loads
  const uint32_t w_row = (uint32_t)(n0 + 8 * wave * C::kLoadW + lr) * krow;
  auto x_load = [&](int i) { return min(wave * C::kLoadX + i, C::BM / 8 - 1); };
  uint32_t x_row[C::kLoadX];
#pragma unroll
  for (int i = 0; i < C::kLoadX; ++i) {
    const int r = source(8 * x_load(i) + lr);
    x_row[i] = r < 0 ? kNoRow : (uint32_t)r * krow;
  }
  const int sr = C::kBytes ? lane >> 3 : lane >> 1;
  const uint32_t s_at = C::kBytes ? lane & 7 : (lane & 1) * 4;
  auto s_load = [&](int i) { return min(wave * C::kLoadS + i, C::kScaleLoads - 1); };
  uint32_t s_row[C::kLoadS];
  bool s_is_w[C::kLoadS];
#pragma unroll
  for (int i = 0; i < C::kLoadS; ++i) {
    const int q = s_load(i) * C::kScaleRows;
    s_is_w[i] = q < C::BN;
    const int r = s_is_w[i] ? n0 + q + sr : source(q - C::BN + sr);
    s_row[i] = r < 0 ? kNoRow : (uint32_t)r * srow;
  }
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(lds));
  auto issue = [&](int st, int slot) {
    const uint32_t to = lds0 + slot * C::kStage;
    auto k_of = [&](int load) {
      const uint32_t kb = (uint32_t)st * 128 + (piece ^ (load & 1) * 64);
      return kb < krow ? kb : kPast;
    };
    const uint32_t sb = (uint32_t)st * 8 + s_at;
    const uint32_t sk = sb < srow ? sb : kPast;
#pragma unroll
    for (int i = 0; i < C::kLoadS; ++i) {
      if constexpr (C::kBytes)
        load_lds1(s_is_w[i] ? ws : as, s_row[i] + sk, to + C::kRows * 128 + s_load(i) * 256);
      else
        load_lds4(s_is_w[i] ? ws : as, s_row[i] + sk, to + C::kRows * 128 + s_load(i) * 256);
    }
#pragma unroll
    for (int i = 0; i < C::kLoadX; ++i) load_lds16(aq, x_row[i] + k_of(x_load(i)), to + C::BN * 128 + x_load(i) * 1024);
#pragma unroll
    for (int i = 0; i < C::kLoadW; ++i)
      load_lds16(wq, w_row + i * 8 * krow + k_of(wave * C::kLoadW + i), to + (wave * C::kLoadW + i) * 1024);
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
  struct Frags {
    intx4 w[C::NW], x[C::MW];
  };
  // Scales of the four steps: the bytes of one word, or (kBytes) the low bytes of four.
  using Scale = std::conditional_t<C::kBytes, intx4, int>;
  struct Scales {
    Scale w[C::NW], x[C::MW];
  };
  auto read = [&](Frags& v, int slot, int j) {
    const uint8_t* b = lds + slot * C::kStage + ((4 * half + j) ^ (lane >> 1 & 7)) * 16;
#pragma unroll
    for (int g = 0; g < C::MW; ++g) v.x[g] = *reinterpret_cast<const intx4*>(b + (x_at + 32 * g) * 128);
#pragma unroll
    for (int f = 0; f < C::NW; ++f) v.w[f] = *reinterpret_cast<const intx4*>(b + (w_at + 32 * f) * 128);
  };
  auto read_scales = [&](Scales& v, int slot) {
    const uint8_t* b = lds + slot * C::kStage + C::kRows * 128 + half * (C::kScaleRow / 2);
#pragma unroll
    for (int g = 0; g < C::MW; ++g) v.x[g] = *reinterpret_cast<const Scale*>(b + (x_at + 32 * g) * C::kScaleRow);
#pragma unroll
    for (int f = 0; f < C::NW; ++f) v.w[f] = *reinterpret_cast<const Scale*>(b + (w_at + 32 * f) * C::kScaleRow);
  };
  auto multiply = [&](const Frags& v, const Scales& s, auto J) {
    constexpr int j = decltype(J)::value;
    auto wide = [](intx4 t) { return intx8{t[0], t[1], t[2], t[3], 0, 0, 0, 0}; };
#pragma unroll
    for (int f = 0; f < C::NW; ++f)
#pragma unroll
      for (int g = 0; g < C::MW; ++g) {
        if constexpr (C::kBytes)
          acc[f][g] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(v.w[f]), wide(v.x[g]), acc[f][g], 4, 4, 0,
                                                                      s.w[f][j], 0, s.x[g][j]);
        else
          acc[f][g] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(v.w[f]), wide(v.x[g]), acc[f][g], 4, 4, j,
                                                                      s.w[f], j, s.x[g]);
      }
  };

  // Stage st is in slot st % S. Fragments are read one step ahead of their
  // products, the first of a stage during the last step of the one before. The
  // barrier is there: every wave has then read all of stage st, whose slot the
  // loads of stage st + S may take, and its loads of stage st + 1 have landed.
  const int stages = (P.Kd + 255) / 256;
#pragma unroll
  for (int s = 0; s < C::S; ++s) issue(s, s);  // past the last stage: zeros
  wait_loads<(C::S - 1) * C::kLoads>();
  lds_barrier();
  Frags even, odd;
  Scales sc;
  read_scales(sc, 0);
  read(even, 0, 0);
  int slot = 0;
  for (int st = 0; st < stages; ++st) {
    const int next = slot == C::S - 1 ? 0 : slot + 1;
    read(odd, slot, 1);
    __builtin_amdgcn_sched_barrier(0);
    multiply(even, sc, std::integral_constant<int, 0>{});
    __builtin_amdgcn_sched_barrier(0);
    read(even, slot, 2);
    __builtin_amdgcn_sched_barrier(0);
    multiply(odd, sc, std::integral_constant<int, 1>{});
    __builtin_amdgcn_sched_barrier(0);
    read(odd, slot, 3);
    __builtin_amdgcn_sched_barrier(0);
    multiply(even, sc, std::integral_constant<int, 2>{});
    __builtin_amdgcn_sched_barrier(0);
    wait_loads<(C::S - 2) * C::kLoads>();
    lds_barrier();
    Scales sn;
    read(even, next, 0);
    read_scales(sn, next);
    issue(st + C::S, slot);
    __builtin_amdgcn_sched_barrier(0);
    multiply(odd, sc, std::integral_constant<int, 3>{});
    __builtin_amdgcn_sched_barrier(0);
    sc = sn;
    slot = next;
  }
  wait_loads<0>();  // no load may land in LDS after the workgroup's end, nor in what follows
  lds_barrier();

  // acc[f][g][i] is column 32 f + 8 (i / 4) + 4 half + i % 4 of row 32 g + r32 of
  // the wave's part. 32 rows at a time (FP32: in two halves of the columns) go
  // through this wave's own piece of LDS, so that a store covers whole rows of it.
  uint8_t* mine = lds + wave * 32 * C::kOutRow;
  const int cols = min(P.N - n0 - wn * C::NW * 32, C::NW * 32);  // of this wave's part that exist
#pragma unroll
  for (int g = 0; g < C::MW; ++g) {
    const int m0 = (wm * C::MW + g) * 32;
    const int rows = min(it.rows - m0, 32);
    const long out = (long)(it.row0 + m0) * P.N + n0 + wn * C::NW * 32;
    auto copy = [&](int size, int c0, int width) {  // columns c0 .. c0 + width of the 32 rows, 16 bytes a lane
      const int per = width * size / 16;            // lanes of a row: a power of two
      const int have = min(max(cols - c0, 0), width) * size;
      for (int i = lane; i < 32 * per; i += 64) {
        const int r = i / per, at = i % per * 16;
        const uint2* from = reinterpret_cast<const uint2*>(mine + r * C::kOutRow + at);
        const uint2 a = from[0], b = from[1];
        if (r < rows && at < have)
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(P.out) + (out + (long)r * P.N + c0) * size + at) =
              make_uint4(a.x, a.y, b.x, b.y);
      }
    };
    if (P.out_f32) {
      constexpr int kF = C::NW > 1 ? C::NW / 2 : 1;  // fragments of a half
#pragma unroll
      for (int h = 0; h < (C::NW > 1 ? 2 : 1) * (C::NW > 1 ? 1 : 2); ++h) {
        // NW > 1: fragments h * kF ..; NW = 1: quarters 2h, 2h + 1 of the one fragment
#pragma unroll
        for (int f = 0; f < kF; ++f)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (C::NW == 1 && q / 2 != h) continue;
            const floatx16& a = acc[C::NW > 1 ? h * kF + f : 0][g];
            const int at = (C::NW > 1 ? 32 * f + 8 * q : 8 * (q & 1)) + 4 * half;
            uint2* to = reinterpret_cast<uint2*>(mine + r32 * C::kOutRow + at * 4);
            to[0] = make_uint2(__float_as_uint(a[4 * q]), __float_as_uint(a[4 * q + 1]));
            to[1] = make_uint2(__float_as_uint(a[4 * q + 2]), __float_as_uint(a[4 * q + 3]));
          }
        copy(4, h * C::NW * 16, C::NW * 16);
      }
    } else {
#pragma unroll
      for (int f = 0; f < C::NW; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const floatx16& a = acc[f][g];
          *reinterpret_cast<uint2*>(mine + r32 * C::kOutRow + (32 * f + 8 * q + 4 * half) * 2) =
              make_uint2(f32x2_to_bf16x2(a[4 * q], a[4 * q + 1]), f32x2_to_bf16x2(a[4 * q + 2], a[4 * q + 3]));
        }
      copy(2, 0, C::NW * 32);
    }
  }
}

// ---------------------------------------------------------------- forward, many rows
// The same products in the same order by workgroups that stay: 256 x 256 tiles
// by eight waves (two a SIMD, each 64 columns by 128 rows), one workgroup a CU,
// which takes every 32nd tile of its XCD. Loads run ahead across tiles: while the last
// stages of one are multiplied, the first of the next are under way, so that
// only the epilogue stands between two tiles. Scales are loaded for two
// stages at once, 16 bytes of a row: a load moves whole lines whatever it uses of them,
// and two dwords of every row each stage cost as much as the codes.
// An expert's rows are shared out evenly over its tiles in groups of 32, and a wave
// multiplies the groups that its tile has. 49152 gathered rows, 64 experts, N = Kd = 4096: 536 us
// (527 to 547; FP32 output 630), 3080 TFLOP/s, the matrix pipes busy for 43 % of it at 1.8 GHz: what
// bounds it is the power that random codes draw (the instruction alone then runs at 5700 TFLOP/s,
// 9600 with constant ones) and LDS, into which a stage of 64 products a SIMD loads 64 KB and of
// which its waves read 192 KB (31 % of the cycles by its counter, which leaves the loads out),
// with two slots, so that a stage's loads are waited for three quarters of a stage after their
// issue. Three slots of smaller stages, half lines, loads in clumps and a prefetch into L2 measured no better.
// Where Kd is not a multiple of 128, rows of scales are not whole dwords: they are loaded
// byte by byte, each stage its own, 4 bytes of LDS a scale, beside tiles of 192 rows.
template <int MW_, bool kBytes_>
struct MxWide {
  static constexpr int NW = 2, MW = MW_, WN = 4, WM = 2, kWaves = WN * WM, BN = 32 * NW * WN, BM = 32 * MW * WM;
  static constexpr bool kBytes = kBytes_;
  static constexpr int kRows = BN + BM, kStage = kRows * 128;
  static constexpr int kScaleRow = kBytes ? 32 : 16, kScales = kRows * kScaleRow;  // of a stage, of a pair of stages
  static constexpr int kLoadW = BN / 8 / kWaves, kLoadX = BM / 8 / kWaves, kLoads = kLoadW + kLoadX;  // 1 KB loads of a wave
  static constexpr int kOutRow = 64 * NW + 8;
  static constexpr int kTable = 2 * kStage + 2 * kScales, kLds = kTable + kMaxExperts * 4;
  static_assert(kWaves * 32 * kOutRow <= kStage && kLds <= 163840 && (kBytes || kLoadX % 2 == 0), "room and whole loads");
};

template <class C, bool kF32>
__global__ __launch_bounds__(C::kWaves * 64) void mx_gemm_wide_kernel(MxGemmParams P) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[C::kLds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t krow = P.Kd / 2, srow = P.Kd / kMxBlock;
  const int col_tiles = (P.N + C::BN - 1) / C::BN;

  // Row tiles up to and with each expert, by wave 0.
  int* table = reinterpret_cast<int*>(lds + C::kTable);
  auto first_row = [&](int e) { return min(max(P.offsets[e], 0), P.R); };
  auto rows_of = [&](int e, int first) { return max(min(P.offsets[e + 1], P.R) - first, 0); };
  if (wave == 0) {
    int before = 0;
    for (int e0 = 0; e0 < P.E; e0 += 64) {
      const int e = e0 + lane;
      const int tiles = e < P.E ? (rows_of(e, first_row(e)) + C::BM - 1) / C::BM : 0;
      const int upto = before + wave_scan(tiles, lane);
      if (e < P.E) table[e] = upto;
      before = __builtin_amdgcn_readlane(upto, 63);
    }
  }
  __syncthreads();
  const int items = __builtin_amdgcn_readfirstlane(table[P.E - 1]) * col_tiles;  // below 2^23 by the launch's check
  const int per = (items + 7) >> 3;
  const int last_item = min((int)(blockIdx.x & 7) * per + per, items);
  int item = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (item >= last_item) return;
  const int step = gridDim.x >> 3;

  auto find = [&](int i) {
    const int tile = i / col_tiles;
    int e = 0;
    for (int e0 = 0; e0 < P.E; e0 += 64) {
      const int upto = table[min(e0 + lane, P.E - 1)];
      const uint64_t past = __ballot(upto > tile);
      if (past) {
        e = e0 + __builtin_ctzll(past);
        break;
      }
    }
    const int first = __builtin_amdgcn_readfirstlane(first_row(e));
    const int rows = __builtin_amdgcn_readfirstlane(rows_of(e, first));
    const int n = (rows + C::BM - 1) / C::BM;
    const int start = __builtin_amdgcn_readfirstlane(table[e]) - n;
    const int local = i - start * col_tiles;
    return mx_tile(e, first, rows, local % n, n, local / n);
  };

  // What a tile's loads need: where its operands begin, its column, and this lane's rows of A (-1: none).
  const int lr = lane >> 3;
  const uint32_t piece = ((lane & 7) ^ lr >> 1) * 16;
  const uint32_t a_rows = P.route_of_row ? P.a_rows : C::BM;  // rows past a tile's end are not asked for
  struct Source {
    const uint8_t *wq, *ws, *aq, *as;
    int n0, x[C::kLoadX];
  };
  auto source = [&](const MxItem& it, Source& s) {
    s.n0 = it.col * C::BN;
    s.wq = P.w_codes + (long)it.e * P.N * krow;
    s.ws = P.w_sf + (long)it.e * P.N * srow;
    const long base = P.route_of_row ? 0 : it.row0;
    s.aq = P.a_codes + base * krow;
    s.as = P.a_sf + base * srow;
#pragma unroll
    for (int i = 0; i < C::kLoadX; ++i) {
      const int m = 8 * (wave * C::kLoadX + i) + lr;
      s.x[i] = m < it.rows ? m : -1;
      if (P.route_of_row && m < it.rows) {
        const int f = P.route_of_row[it.row0 + m];
        s.x[i] = f >= 0 && f / P.topk < P.a_rows ? f / P.topk : -1;
      }
    }
  };
  // The rows' offsets are computed at each load: kept, they would not fit in registers.
  auto opaque = [](int v) {
    asm volatile("" : "+v"(v));
    return v;
  };
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(lds));
  // The loads of a stage's codes and of its scales (kBytes) or, in an even stage, of
  // its pair's, in parts; !any: zeros.
  auto row_of = [&](const Source& s, int i, uint32_t row) {
    const int x = opaque(s.x[i]);
    return x < 0 ? kNoRow : (uint32_t)x * row;
  };
  auto load_codes = [&](const Source& s, int st, int slot, bool any, int part, int parts) {
    const uint32_t to = lds0 + slot * C::kStage;
    const uint32_t kb = (uint32_t)st * 128 + piece, kx = kb ^ 64;
    const uint32_t k[2] = {any && kb < krow ? kb : kPast, any && kx < krow ? kx : kPast};
    const uint32_t w = (uint32_t)opaque(s.n0 + 8 * wave * C::kLoadW + lr) * krow;
    const intx4 wq = raw_buffer(s.wq, (uint32_t)P.N * krow), aq = raw_buffer(s.aq, a_rows * krow);
#pragma unroll
    for (int l = C::kLoads * part / parts; l < C::kLoads * (part + 1) / parts; ++l) {
      if (l < C::kLoadX) {
        const int q = wave * C::kLoadX + l;
        load_lds16(aq, row_of(s, l, krow) + k[q & 1], to + C::BN * 128 + q * 1024);
      } else {
        const int i = l - C::kLoadX;
        load_lds16(wq, w + i * 8 * krow + k[i & 1], to + (wave * C::kLoadW + i) * 1024);
      }
    }
  };
  auto load_scales = [&](const Source& s, int at, int buf, bool any, int part, int parts) {
    const uint32_t to = lds0 + 2 * C::kStage + buf * C::kScales;
    const intx4 ws = raw_buffer(s.ws, (uint32_t)P.N * srow), as = raw_buffer(s.as, a_rows * srow);
    if constexpr (C::kBytes) {  // 8 scales of 8 rows a load, stage `at`
      const uint32_t kb = (uint32_t)at * 8 + (lane & 7);
      const uint32_t k = any && kb < srow ? kb : kPast;
      const uint32_t w = (uint32_t)opaque(s.n0 + 8 * wave * C::kLoadW + lr) * srow + k;
#pragma unroll
      for (int l = C::kLoads * part / parts; l < C::kLoads * (part + 1) / parts; ++l) {
        if (l < C::kLoadX)
          load_lds1(as, row_of(s, l, srow) + k, to + C::BN * 32 + (wave * C::kLoadX + l) * 256);
        else
          load_lds1(ws, w + (l - C::kLoadX) * 8 * srow, to + (wave * C::kLoadW + l - C::kLoadX) * 256);
      }
    } else {  // 4 dwords of 16 rows a load, pair `at`; a lane's row of A is what lanes 8 (l / 4 % 8) have of codes' loads 2i + l / 32
      const uint32_t kb = (uint32_t)at * 16 + (lane & 3) * 4;
      const uint32_t k = any && kb < srow ? kb : kPast;
      const uint32_t w = (uint32_t)opaque(s.n0 + 8 * wave * C::kLoadW + (lane >> 2)) * srow + k;
      constexpr int kX = C::kLoadX / 2, kAll = kX + C::kLoadW / 2;
#pragma unroll
      for (int l = kAll * part / parts; l < kAll * (part + 1) / parts; ++l) {
        if (l < kX) {
          const int from = (lane >> 2 & 7) * 8;
          const int lo = __shfl(s.x[2 * l], from, 64), hi = __shfl(s.x[2 * l + 1 < C::kLoadX ? 2 * l + 1 : 0], from, 64);
          const int x = lane < 32 ? lo : hi;
          load_lds4(as, (x < 0 ? kNoRow : (uint32_t)x * srow) + k, to + C::BN * 16 + (wave * kX + l) * 256);
        } else {
          load_lds4(ws, w + (l - kX) * 16 * srow, to + (wave * (C::kLoadW / 2) + l - kX) * 256);
        }
      }
    }
  };

  const int wn = wave % C::WN, wm = wave / C::WN;
  const int half = lane >> 5, r32 = lane & 31;
  // Row groups of 32 alternate between the waves that share columns.
  const int w_at = wn * C::NW * 32 + r32, x_at = C::BN + wm * 32 + r32;
  struct Frags {
    intx4 w[C::NW], x[C::MW];
  };
  // Scales of the four steps of a stage: the bytes of one word, or (kBytes) the low bytes of four.
  using Scale = std::conditional_t<C::kBytes, intx4, int>;
  struct Scales {
    Scale w[C::NW], x[C::MW];
  };
  // Part `part` of `parts` of a step's fragments.
  auto read = [&](Frags& v, int slot, int j, int part, int parts) {
    constexpr int kAll = C::MW + C::NW;
    const uint8_t* b = lds + slot * C::kStage + ((4 * half + j) ^ (lane >> 1 & 7)) * 16;
#pragma unroll
    for (int i = kAll * part / parts; i < kAll * (part + 1) / parts; ++i) {
      if (i < C::MW)
        v.x[i] = *reinterpret_cast<const intx4*>(b + (x_at + 64 * i) * 128);
      else
        v.w[i - C::MW] = *reinterpret_cast<const intx4*>(b + (w_at + 32 * (i - C::MW)) * 128);
    }
  };
  auto read_scales = [&](Scales& v, int buf, int odd_stage) {
    const uint8_t* b = lds + 2 * C::kStage + buf * C::kScales + (C::kBytes ? half * 16 : odd_stage * 8 + half * 4);
#pragma unroll
    for (int g = 0; g < C::MW; ++g) v.x[g] = *reinterpret_cast<const Scale*>(b + (x_at + 64 * g) * C::kScaleRow);
#pragma unroll
    for (int f = 0; f < C::NW; ++f) v.w[f] = *reinterpret_cast<const Scale*>(b + (w_at + 32 * f) * C::kScaleRow);
  };

  // Stages come in pairs: stage st is in slot st % 2, its scales in the buffer of its pair,
  // or (kBytes) in buffer st % 2.
  const int pairs = (P.Kd + 511) / 512;
  MxItem it = find(item);
  Source src, nxt;
  source(it, src);
  load_scales(src, 0, 0, true, 0, 1);
  load_codes(src, 0, 0, true, 0, 1);
  load_codes(src, 1, 1, true, 0, 1);
  if constexpr (C::kBytes) load_scales(src, 1, 1, true, 0, 1);
  wait_loads<(C::kBytes ? 2 : 1) * C::kLoads>();
  lds_barrier();
  Frags even, odd;
  Scales sc;
  read_scales(sc, 0, 0);
  read(even, 0, 0, 0, 1);
  int buf = 0;
  bool more = false;

  // One tile, of which this wave multiplies kG groups of 32 rows.
  auto tile = [&](auto G) {
    constexpr int kG = decltype(G)::value;
    floatx16 acc[C::NW][kG];
#pragma unroll
    for (int f = 0; f < C::NW; ++f)
#pragma unroll
      for (int g = 0; g < kG; ++g)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[f][g][i] = 0.0f;
    // The products of step J, and between them what `behind` does in parts.
    auto multiply = [&](const Frags& v, auto J, auto behind) {
      constexpr int j = decltype(J)::value;
      auto wide = [](intx4 u) { return intx8{u[0], u[1], u[2], u[3], 0, 0, 0, 0}; };
#pragma unroll
      for (int g = 0; g < kG; ++g)
#pragma unroll
        for (int f = 0; f < C::NW; ++f) {
          if constexpr (C::kBytes)
            acc[f][g] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(v.w[f]), wide(v.x[g]), acc[f][g], 4, 4, 0,
                                                                        sc.w[f][j], 0, sc.x[g][j]);
          else
            acc[f][g] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(v.w[f]), wide(v.x[g]), acc[f][g], 4, 4, j,
                                                                        sc.w[f], j, sc.x[g]);
          __builtin_amdgcn_sched_barrier(0);
          behind(g * C::NW + f, kG * C::NW);
          __builtin_amdgcn_sched_barrier(0);
        }
    };
    // The stage in slot `slot`, the odd or the even one of its pair. At its barrier
    // every wave has read all of it, and the loads of the stage behind it have
    // landed; `load` may then fill its slot and, in an even stage, the other pair's scales.
    auto stage = [&](auto Slot, auto load) {
      constexpr int slot = decltype(Slot)::value;
      multiply(even, std::integral_constant<int, 0>{}, [&](int part, int parts) { read(odd, slot, 1, part, parts); });
      multiply(odd, std::integral_constant<int, 1>{}, [&](int part, int parts) { read(even, slot, 2, part, parts); });
      multiply(even, std::integral_constant<int, 2>{}, [&](int part, int parts) { read(odd, slot, 3, part, parts); });
      wait_loads<0>();
      lds_barrier();
      Scales next;
      if constexpr (slot == 1 && !C::kBytes) buf ^= 1;
      read_scales(next, C::kBytes ? slot ^ 1 : buf, slot ^ 1);
      multiply(odd, std::integral_constant<int, 3>{}, [&](int part, int parts) {
        read(even, slot ^ 1, 0, part, parts);
        load(part, parts);
      });
      sc = next;
    };
    constexpr auto slot0 = std::integral_constant<int, 0>{};
    constexpr auto slot1 = std::integral_constant<int, 1>{};
    for (int p = 0; p < pairs - 1; ++p) {
      stage(slot0, [&](int part, int parts) {
        load_codes(src, 2 * p + 2, 0, true, part, parts);
        load_scales(src, C::kBytes ? 2 * p + 2 : p + 1, C::kBytes ? 0 : buf ^ 1, true, part, parts);
      });
      stage(slot1, [&](int part, int parts) {
        load_codes(src, 2 * p + 3, 1, true, part, parts);
        if constexpr (C::kBytes) load_scales(src, 2 * p + 3, 1, true, part, parts);
      });
    }
    stage(slot0, [&](int part, int parts) {
      load_codes(nxt, 0, 0, more, part, parts);
      load_scales(nxt, 0, C::kBytes ? 0 : buf ^ 1, more, part, parts);
    });
    stage(slot1, [](int, int) {});
    // All products are issued before the epilogue: left to the compiler, some move into its branches.
#pragma unroll
    for (int f = 0; f < C::NW; ++f)
#pragma unroll
      for (int g = 0; g < kG; ++g) asm volatile("" : "+v"(acc[f][g]));

    // The second slot is free until the next tile's second stage. acc[f][g][i] is
    // column 32 f + 8 (i / 4) + 4 half + i % 4 of row r32 of group g; a group's rows
    // go through this wave's own piece of the slot, so that a store covers whole rows of it.
    uint8_t* mine = lds + C::kStage + wave * 32 * C::kOutRow;
    const int n0 = it.col * C::BN + wn * C::NW * 32;
    const int cols = min(P.N - n0, C::NW * 32);
    constexpr int kSize = kF32 ? 4 : 2, kPasses = kF32 ? 2 : 1, kWidth = C::NW * 32 / kPasses;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int m0 = (g * C::WM + wm) * 32;
      const int rows = min(it.rows - m0, 32);
      uint8_t* out = static_cast<uint8_t*>(P.out) + ((long)(it.row0 + m0) * P.N + n0) * kSize;
#pragma unroll
      for (int h = 0; h < kPasses; ++h) {
#pragma unroll
        for (int f = 0; f < C::NW; ++f) {
          if (f / (C::NW / kPasses) != h) continue;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const floatx16& a = acc[f][g];
            uint2* to = reinterpret_cast<uint2*>(mine + r32 * C::kOutRow + (32 * (f % (C::NW / kPasses)) + 8 * q + 4 * half) * kSize);
            if constexpr (kF32) {
              to[0] = make_uint2(__float_as_uint(a[4 * q]), __float_as_uint(a[4 * q + 1]));
              to[1] = make_uint2(__float_as_uint(a[4 * q + 2]), __float_as_uint(a[4 * q + 3]));
            } else {
              *to = make_uint2(f32x2_to_bf16x2(a[4 * q], a[4 * q + 1]), f32x2_to_bf16x2(a[4 * q + 2], a[4 * q + 3]));
            }
          }
        }
        const int have = min(max(cols - h * kWidth, 0), kWidth) * kSize;
#pragma unroll
        for (int i = 0; i < kWidth * kSize / 32; ++i) {  // a row's 16 bytes a lane
          constexpr int kPer = kWidth * kSize / 16;
          const int r = 64 / kPer * i + lane / kPer, at = lane % kPer * 16;
          const uint2* from = reinterpret_cast<const uint2*>(mine + r * C::kOutRow + at);
          const uint2 a = from[0], b = from[1];
          if (r < rows && at < have)
            *reinterpret_cast<uint4*>(out + (long)r * P.N * kSize + h * kWidth * kSize + at) = make_uint4(a.x, a.y, b.x, b.y);
        }
      }
    }
  };

  for (;;) {
    const int next_item = item + step;
    more = next_item < last_item;
    MxItem ahead = it;
    if (more) ahead = find(next_item);
    source(ahead, nxt);
    switch (((it.rows + 31) / 32 - wm + 1) / 2) {
      case 0:  // no row for this wave; it still loads, and meets the others at the barriers
      case 1: tile(std::integral_constant<int, 1>{}); break;
      case 2: tile(std::integral_constant<int, 2>{}); break;
      case 3: tile(std::integral_constant<int, 3>{}); break;
      default: tile(std::integral_constant<int, C::MW>{}); break;
    }
    if (!more) break;
    lds_barrier();
    load_codes(nxt, 1, 1, true, 0, 1);
    if constexpr (C::kBytes) load_scales(nxt, 1, 1, true, 0, 1);
    src = nxt;
    it = ahead;
    item = next_item;
  }
  wait_loads<0>();  // no load may land in LDS after the workgroup's end
}

template <class C>
static hipError_t run_gemm_wide(const MxGemmParams& p, hipStream_t s) {
  if (p.out_f32)
    mx_gemm_wide_kernel<C, true><<<256, C::kWaves * 64, 0, s>>>(p);
  else
    mx_gemm_wide_kernel<C, false><<<256, C::kWaves * 64, 0, s>>>(p);
  return hipGetLastError();
}

template <class C>
static hipError_t run_gemm(const MxGemmParams& p, hipStream_t s) {
  const long tiles = (long)p.R / C::BM + (p.E < p.R ? p.E : p.R);
  const long grid = (tiles * ((p.N + C::BN - 1) / C::BN) + 7) / 8 * 8;
  mx_gemm_kernel<C><<<(unsigned)grid, C::kWaves * 64, 0, s>>>(p);
  return hipGetLastError();
}

// Which tile: the largest that the rows of an expert fill to some part and that gives the
// chip enough workgroups (m: rows of an expert if all have alike). Measured at N = Kd =
// 4096: 64 experts, m = 1: 128 x 32 tiles 101 us, 256 x 128 109, 256 x 256 133; m = 32:
// 153, 126, 145; m = 192: 443, 265, 212. One expert, 1024 rows: 33, 23, 29, and 18
// with 128 x 128; 64 rows: 10, 18, 18, and 8 with 64 x 32.
// How many tiles the persistent kernel wants (N = 2064, 180 or 200 rows an expert): at 72, 108, 180, 288,
// 432 tiles, Kd = 4096, it takes 29, 30, 30, 55, 68 us and 256 x 128 tiles, which fill the chip once up
// to 256 of them, 22, 25, 43, 63, 93; with experts of unlike size (log-normal, 1) 29, 29, 37, 61, 91 and
// 24, 26, 47, 70, 96. With byte scales, Kd = 2080, at 180, 216, 432, 576: 25, 25, 47, 67 and 32, 32, 63,
// 81 where experts are alike, 40, 41, 62, 78 and 34, 33, 64, 84 where they are not: below 512 the
// gain of the first is the loss of the second, and the host cannot tell them apart.
template <bool kBytes>
static hipError_t run_gemm_any(const MxGemmParams& p, hipStream_t s) {
  const long experts = p.E < p.R ? p.E : p.R, m = (p.R + experts - 1) / experts;
  auto items = [&](int bm, int bn) { return experts * ((m + bm - 1) / bm) * ((p.N + bn - 1) / bn); };
  using Wide = MxWide<kBytes ? 3 : 4, kBytes>;
  if (m > 112 && items(Wide::BM, Wide::BN) >= (kBytes ? 512 : 160)) return run_gemm_wide<Wide>(p, s);
  if (m > 8 && items(128, 256) >= 128) return run_gemm<MxTile<2, 2, 4, 2, 2, kBytes>>(p, s);
  if (m > 8 && items(128, 128) >= 128) return run_gemm<MxTile<2, 2, 2, 2, 2, kBytes>>(p, s);
  if (items(32, 128) >= 256) return run_gemm<MxTile<1, 1, 4, 1, 3, kBytes>>(p, s);
  return run_gemm<MxTile<1, 1, 2, 1, 4, kBytes>>(p, s);
}

hipError_t launch_mx_gemm(const MxGemmParams& p, hipStream_t s) {
  return p.Kd % 128 != 0 ? run_gemm_any<true>(p, s) : run_gemm_any<false>(p, s);
}

// ---------------------------------------------------------------- backward
// v_mfma_f32_32x32x16_bf16 reduces over 16 rows n of the matrix; a lane needs 8
// consecutive n of one column k, while the codes run along k. So a lane reads
// the same 4 columns (16 bits) of 8 rows, converts each pair of columns with its
// row's scale (exact in BF16 up to the quantizer's largest scale, 252: subnormal values are
// kept by the convert and the product, and only 4 * 2^126 and 2 * 2^127 on are past its
// largest), and regroups the halves of row pairs: 4 fragments
// of 32 columns, columns 4c + i in fragment i for lane c, with no transposition
// through LDS. A wave owns 128 columns and every row of the tile, so a matrix tile
// is converted once a workgroup.
//
// A stage is 64 rows n of the matrix (KW * 128 columns: KW * 64 bytes a row, KW
// * 4 scales) and 64 columns of dy, four steps of 16. The codes of a step are read two steps
// ahead and converted one step ahead, between the products of the step before:
// products and conversions run in different pipes, but a wave issues in order.
// Matrix rows with (n / 8) odd have the halves of each 128 bytes exchanged, so
// that the two halves of a wave, 8 rows apart, read different banks.
// 24576 rows, 64 experts, N = Kd = 4096: 760 us (744 to 765), 1085 TFLOP/s (a large BF16 product of the library:
// 1266 to 1558), the matrix pipes busy for 63 % at 1.7 GHz, the vector ones, which convert, for 40 %. 777
// rows of 16 experts, N = 1536, Kd = 2048: 26 us, 24 stages of about 1 us in a row whatever the tile (24 to
// 28 us for five of them): the conversion of 64 x 128 codes by one wave is the chain.
template <int MW_, int KW_, int S_, bool kBytes_>
struct MxBackTile {
  static constexpr int MW = MW_, KW = KW_, S = S_;
  static constexpr bool kBytes = kBytes_;
  static constexpr int kWaves = KW, BK = 128 * KW, BM = 32 * MW, kN = 64, kRow = BK / 2;
  static constexpr int kScaleRow = kBytes ? 16 * KW : 4 * KW;
  static constexpr int kW = kN * kRow, kS = kN * kScaleRow, kStage = kW + kS + BM * kN * 2;
  static constexpr int kLoadW = kW / 1024 / kWaves, kLoadS = kS / 256 / kWaves, kLoadY = BM / 8 / kWaves;
  static constexpr int kLoads = kLoadW + kLoadS + kLoadY;
  static_assert(BM % (8 * kWaves) == 0 && (S - 2) * kLoads < 64, "whole loads, counted in 6 bits");
};

// One tile of G groups of 32 rows.
template <class C, int G>
__device__ __forceinline__ void mx_back_tile(const MxGemmParams& P, uint8_t* lds, const MxItem& it) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k0 = it.col * C::BK;
  const uint32_t krow = P.Kd / 2, srow = P.Kd / kMxBlock, yrow = (uint32_t)P.N * 2;
  const intx4 wq = raw_buffer(P.w_codes + (long)it.e * P.N * krow, (uint32_t)P.N * krow);
  const intx4 ws = raw_buffer(P.w_sf + (long)it.e * P.N * srow, (uint32_t)P.N * srow);
  const intx4 dy = raw_buffer(P.a_codes + (long)it.row0 * yrow, (uint32_t)it.rows * yrow);

  // Loads of this lane: 16 bytes of codes, a dword (byte) of scales, 16 bytes of dy.
  constexpr int kPer = C::kRow / 16, kWRows = 64 / kPer;            // lanes of a matrix row, rows of a load
  constexpr int kSPer = C::kBytes ? 4 * C::KW : C::KW, kSRows = 64 / kSPer;
  const int wr = lane / kPer, sr = lane / kSPer, yr = lane >> 3;
  const uint32_t s_k = k0 / kMxBlock + lane % kSPer * (C::kBytes ? 1 : 4);
  const uint32_t y_piece = ((lane & 7) ^ yr >> 1) * 16;  // ^ 64 in odd loads
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(lds));
  // Part `part` of `parts` of this wave's loads of stage st.
  auto issue = [&](int st, int slot, int part, int parts) {
    const uint32_t to = lds0 + slot * C::kStage;
    const uint32_t n0 = (uint32_t)st * C::kN;
#pragma unroll
    for (int l = C::kLoads * part / parts; l < C::kLoads * (part + 1) / parts; ++l) {
      if (l < C::kLoadW) {
        const int q = wave * C::kLoadW + l, row = kWRows * q + wr;
        const uint32_t k = k0 / 2 + ((lane % kPer) ^ (C::KW > 1 ? (row >> 3 & 1) << 2 : 0)) * 16;
        load_lds16(wq, n0 + row < (uint32_t)P.N && k < krow ? (n0 + row) * krow + k : kNoRow, to + q * 1024);
      } else if (l < C::kLoadW + C::kLoadS) {
        const int q = wave * C::kLoadS + l - C::kLoadW;
        const uint32_t n = n0 + kSRows * q + sr;
        const uint32_t at = n < (uint32_t)P.N && s_k < srow ? n * srow + s_k : kNoRow;
        if constexpr (C::kBytes)
          load_lds1(ws, at, to + C::kW + q * 256);
        else
          load_lds4(ws, at, to + C::kW + q * 256);
      } else {
        const int q = wave * C::kLoadY + l - C::kLoadW - C::kLoadS;
        const uint32_t m = 8 * q + yr, yb = n0 * 2 + (y_piece ^ (q & 1) * 64);
        load_lds16(dy, m < (uint32_t)it.rows && yb < yrow ? m * yrow + yb : kNoRow, to + C::kW + C::kS + q * 1024);
      }
    }
  };

  floatx16 acc[4][G];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][g][i] = 0.0f;

  const int half = lane >> 5, c = lane & 31;
  const int w_at = half * 8 * C::kRow + ((wave * 64 + c * 2) ^ (C::KW > 1 ? half << 6 : 0));
  const int s_at = half * 8 * C::kScaleRow + (wave * 4 + (c >> 3)) * (C::kBytes ? 4 : 1);
  struct Raw {
    uint32_t q[8];   // codes of columns 4c .. 4c + 3 of 8 rows
    uint32_t s[8];   // their scales
    bf16x8_t x[G];
  };
  // In 16 pieces: piece i < 8 reads row i, the others dy.
  auto read = [&](Raw& v, int slot, int j, int piece) {
    const uint8_t* b = lds + slot * C::kStage;
    if (piece < 8) {
      v.q[piece] = *reinterpret_cast<const uint16_t*>(b + (16 * j + piece) * C::kRow + w_at);
      v.s[piece] = b[C::kW + (16 * j + piece) * C::kScaleRow + s_at];
    } else if (piece - 8 < G) {
      v.x[piece - 8] = *reinterpret_cast<const bf16x8_t*>(b + C::kW + C::kS + (32 * (piece - 8) + c) * 128 +
                                                          (((2 * j + half) ^ (lane >> 1 & 7)) * 16));
    }
  };
  // Conversion in 16 pieces: piece i < 8 converts row i, piece 8 + i makes two words of the fragments.
  struct Frags {
    uint32_t lo[8], hi[8];  // columns 0, 1 and 2, 3 of each row
    uint32_t w[4][4];
  };
  auto convert = [&](const Raw& v, Frags& f, int piece) {
    if (piece < 8) {
      const float s = mx_scale(v.s[piece]);
      f.lo[piece] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v.q[piece], s, 0));
      f.hi[piece] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v.q[piece], s, 1));
    } else {
      const int p = piece - 8, pair = p & 3, h = p >> 2;
      const uint32_t a = h ? f.hi[2 * pair] : f.lo[2 * pair], b = h ? f.hi[2 * pair + 1] : f.lo[2 * pair + 1];
      f.w[2 * h][pair] = __builtin_amdgcn_perm(b, a, 0x05040100u);
      f.w[2 * h + 1][pair] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    }
  };
  // The products of one step, and between them the conversion of the next, the reads
  // of the one behind that, and, in one step of a stage, its loads.
  auto step = [&](const Frags& f, const Raw& v, const Raw& next, Frags& nf, auto behind) {
    constexpr int kProducts = 4 * G;
#pragma unroll
    for (int i = 0; i < kProducts; ++i) {
      const int g = i / 4, k = i % 4;
      bf16x8_t w;
      __builtin_memcpy(&w, f.w[k], 16);
      acc[k][g] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, v.x[g], acc[k][g], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int p = 16 * i / kProducts; p < 16 * (i + 1) / kProducts; ++p) {
        convert(next, nf, p);
        behind(p);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Stage st is in slot st % S. Its last codes are read in its second step; the barrier
  // behind that also says that stage st + 1 has landed for every wave.
  const int stages = (P.N + C::kN - 1) / C::kN;
#pragma unroll
  for (int s = 0; s < C::S; ++s) issue(s, s, 0, 1);
  wait_loads<(C::S - 1) * C::kLoads>();
  lds_barrier();
  Raw r0, r1, r2, r3;
  Frags even, odd;
#pragma unroll
  for (int p = 0; p < 16; ++p) {
    read(r0, 0, 0, p);
    read(r1, 0, 1, p);
  }
#pragma unroll
  for (int p = 0; p < 16; ++p) convert(r0, even, p);
  int slot = 0;
  for (int st = 0; st < stages; ++st) {
    const int next = slot == C::S - 1 ? 0 : slot + 1;
    step(even, r0, r1, odd, [&](int p) { read(r2, slot, 2, p); });
    step(odd, r1, r2, even, [&](int p) { read(r3, slot, 3, p); });
    wait_loads<(C::S - 2) * C::kLoads>();
    lds_barrier();
    step(even, r2, r3, odd, [&](int p) {
      read(r0, next, 0, p);
      issue(st + C::S, slot, p, 16);
    });
    step(odd, r3, r0, even, [&](int p) { read(r1, next, 1, p); });
    slot = next;
  }
  wait_loads<0>();
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int g = 0; g < G; ++g) asm volatile("" : "+a"(acc[f][g]));  // no product moves into the branches below

  // acc[f][g][i] is column 4 (8 (i / 4) + 4 half + i % 4) + f of the wave's 128, row 32 g + c.
#pragma unroll
  for (int g = 0; g < G; ++g) {
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
__global__ __launch_bounds__(C::kWaves * 64) void mx_gemm_backward_kernel(MxGemmParams P) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[C::S * C::kStage];
  MxItem it;
  if (!mx_item<C::BM>(P.offsets, P.E, P.R, (P.Kd + C::BK - 1) / C::BK, it)) return;
  switch ((it.rows + 31) / 32) {
    case 1: mx_back_tile<C, 1>(P, lds, it); break;
    case 2: mx_back_tile<C, C::MW < 2 ? C::MW : 2>(P, lds, it); break;
    case 3: mx_back_tile<C, C::MW < 3 ? C::MW : 3>(P, lds, it); break;
    default: mx_back_tile<C, C::MW>(P, lds, it); break;
  }
}

template <class C>
static hipError_t run_gemm_backward(const MxGemmParams& p, hipStream_t s) {
  const long tiles = (long)p.R / C::BM + (p.E < p.R ? p.E : p.R);
  const long grid = (tiles * ((p.Kd + C::BK - 1) / C::BK) + 7) / 8 * 8;
  mx_gemm_backward_kernel<C><<<(unsigned)grid, C::kWaves * 64, 0, s>>>(p);
  return hipGetLastError();
}

// Which tile, as for the forward product. Measured at N = Kd = 4096: 64 experts, m = 1:
// 32 x 512 tiles 104 us, 128 x 512 122; m = 48: 218, 169; m = 192: 584, 436. One expert,
// 1024 rows: 61, 84, and 58 with 32 x 128; 4096 rows: 183, 107, 228. Eight experts of 256 rows,
// N = Kd = 2048: 47, 48, 61, and 37 with 64 x 256.
template <bool kBytes>
static hipError_t run_gemm_backward_any(const MxGemmParams& p, hipStream_t s) {
  const long experts = p.E < p.R ? p.E : p.R, m = (p.R + experts - 1) / experts;
  auto items = [&](int bm, int bk) { return experts * ((m + bm - 1) / bm) * ((p.Kd + bk - 1) / bk); };
  if (m > 24 && items(128, 512) >= 200) return run_gemm_backward<MxBackTile<4, 4, 4, kBytes>>(p, s);
  if (m > 24 && items(64, 256) >= 256) return run_gemm_backward<MxBackTile<2, 2, 4, kBytes>>(p, s);
  if (items(32, 512) >= 256) return run_gemm_backward<MxBackTile<1, 4, 3, kBytes>>(p, s);
  return run_gemm_backward<MxBackTile<1, 1, 4, kBytes>>(p, s);
}

hipError_t launch_mx_gemm_backward(const MxGemmParams& p, hipStream_t s) {
  return p.Kd % 128 != 0 ? run_gemm_backward_any<true>(p, s) : run_gemm_backward_any<false>(p, s);
}

}  // namespace pmoe
